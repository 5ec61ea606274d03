"""Oracle of the paged-cache and sampling operators: plain numpy, fp64, loops.

Test infrastructure only; shares no code with the CUDA path.  Every function
takes host arrays and works one token, head or row at a time, from the
definitions in the comments.
"""
import numpy as np


def tokens(cu, kv_lens):
    """(token, sequence, position) of every new token."""
    for s in range(len(kv_lens)):
        for t in range(int(cu[s]), int(cu[s + 1])):
            yield t, s, int(kv_lens[s]) - int(cu[s + 1]) + t


def rotate(x, pos, freqs, interleaved):
    """Row(s) x [..., D] turned at position pos by freqs (radians per position)."""
    x = np.array(x, np.float64)
    r = 2 * len(freqs)
    a = np.mod(float(pos) * np.asarray(freqs, np.float64), 2 * np.pi)
    c, s = np.cos(a), np.sin(a)
    y = x.copy()
    i, j = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., j] * c + x[..., i] * s
    return y


def append(k, v, kc, vc, table, cu, kv_lens, freqs, interleaved=False, positions=None):
    """fp64 copies of the caches after the append; page size from kc [P, H, page, D]."""
    kc, vc = np.array(kc, np.float64), np.array(vc, np.float64)
    page = kc.shape[2]
    for t, s, pos in tokens(cu, kv_lens):
        if pos < 0 or pos // page >= table.shape[1] or not 0 <= table[s, pos // page] < kc.shape[0]:
            continue
        p = pos if positions is None else int(positions[t])
        kc[table[s, pos // page], :, pos % page] = rotate(k[t], p, freqs, interleaved)
        vc[table[s, pos // page], :, pos % page] = v[t]
    return kc, vc


def attention(q, kc, vc, table, cu, kv_lens, scale, window=0):
    """(out, lse, A, S) in fp64: A = sum p|v| and S = max over the seen keys of
    scale * sum |q_i k_i|, which the error bounds go by.  Rows of padding
    tokens are NaN; positions in bad pages are left out."""
    T, Hq, D = q.shape
    P, Hk, page, _ = kc.shape
    out = np.full((T, Hq, D), np.nan)
    lse = np.full((T, Hq), np.nan)
    A = np.zeros((T, Hq, D))
    S = np.zeros((T, Hq))
    for t, s, pos in tokens(cu, kv_lens):
        first = max(0, pos - window + 1) if window else 0
        seen = [(table[s, c // page], c % page) for c in range(first, pos + 1)
                if c // page < table.shape[1] and 0 <= table[s, c // page] < P]
        out[t] = 0
        lse[t] = -np.inf
        if not seen:
            continue
        pg, sl = np.array(seen).T
        for h in range(Hk):
            K, V = kc[pg, h, sl].astype(np.float64), vc[pg, h, sl].astype(np.float64)
            for j in range(h * Hq // Hk, (h + 1) * Hq // Hk):
                x = q[t, j].astype(np.float64)
                sc = scale * (K @ x)
                m = sc.max()
                w = np.exp(sc - m)
                out[t, j] = (w @ V) / w.sum()
                lse[t, j] = m + np.log(w.sum())
                A[t, j] = (w @ np.abs(V)) / w.sum()
                S[t, j] = abs(scale) * (np.abs(K) @ np.abs(x)).max()
    return out, lse, A, S


def sample(z, u, temperature=None, top_k=None, top_p=None, min_p=None):
    """(token, logprob, kept set in vocabulary order) of one row."""
    z = np.asarray(z, np.float64)
    z = np.where(np.isnan(z), -np.inf, z)
    M = z.max()
    if M == -np.inf:
        return -1, -np.inf, []
    order = sorted(range(len(z)), key=lambda i: (-z[i], i))
    order = [i for i in order if z[i] > -np.inf]
    t = 1.0 if temperature is None else float(temperature)
    if not t > 0 or (top_p is not None and top_p <= 0):
        return order[0], 0.0, order[:1]
    with np.errstate(invalid="ignore", over="ignore"):
        w = {i: 1.0 if z[i] == M else float(np.exp((z[i] - M) / t)) for i in order}
    if top_k is not None and top_k > 0:
        order = order[:int(top_k)]
    if top_p is not None and top_p < 1:
        total, run, n = sum(w[i] for i in order), 0.0, 0
        while n < len(order) and (n == 0 or run < float(top_p) * total):
            run += w[order[n]]
            n += 1
        order = order[:n]
    if min_p is not None and min_p > 0:
        order = [i for i in order if w[i] >= min(float(min_p), 1.0)]
    kept = sorted(order)
    mass, run = sum(w[i] for i in kept), 0.0
    token = None
    for i in kept:
        run += w[i]
        if w[i] > 0 and run > float(u) * mass:
            token = i
            break
    if token is None:
        token = [i for i in kept if w[i] > 0][-1]
    return token, float(np.log(w[token] / mass)), kept
