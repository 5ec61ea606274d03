"""Measured cases of the paged-cache and sampling operators.

Three operators of a decode step on q4_0 weights: appending keys and values
to a paged cache with the rotary rotation (``kv_append``), attention of the
new tokens over that cache (``kv_attention``) and sampling from the head's
logits with given random numbers (``logits_sample``).  ``run`` computes each in
elementary torch operations, or through the library when ``own`` is set.
"""
import math

import torch

own = False

GOLDEN = 0.6180339887498949


def listed():
    return [
        # one decode step of eight users on a sliding layer (8 query heads, 1 KV head of 256), straight from the f32 GEMV outputs
        append("append_decode_8", b=8, new=1, ctx=700, hq=8, hkv=1, d=256, inp="f32", dt="f16"),
        # a 64-token prefill chunk on a full layer (heads of 512), partial rotation
        append("append_chunk_64_d512", b=1, new=64, ctx=4096, hq=8, hkv=1, d=512, inp="f16", dt="f16", rot=128, theta=1e6),
        # prompts of sixteen users in one ragged call
        append("append_prompts_ragged", b=16, new=4096, ctx=6144, hq=8, hkv=1, d=256, inp="bf16", dt="bf16", page=64, ragged=True),
        # single-user decode on a sliding layer: 512 visible keys of 1000
        attend("attn_decode_1_window", b=1, new=1, ctx=1000, hq=8, hkv=1, d=256, dt="f16", window=512),
        # 64 users decoding on a full layer, ragged contexts up to 16384
        attend("attn_decode_64_ragged_d512", b=64, new=1, ctx=16384, hq=8, hkv=1, d=512, dt="f16", ragged=True),
        # one user far into a long document
        attend("attn_decode_long_d512", b=1, new=1, ctx=131071, hq=8, hkv=1, d=512, dt="f16", page=64),
        # four drafted tokens verified at once for 16 users, grouped heads of 128
        attend("attn_verify_4_gqa_d128", b=16, new=4, ctx=4001, hq=32, hkv=8, d=128, dt="bf16", page=32, ragged=True),
        # a 64-token prefill chunk behind 4032 cached tokens
        attend("attn_chunk_64", b=1, new=64, ctx=4096, hq=8, hkv=1, d=256, dt="f16"),
        # prompts of four users behind cached prefixes
        attend("attn_prompts_ragged", b=4, new=4096, ctx=8192, hq=8, hkv=1, d=256, dt="bf16", page=64, ragged=True),
        # the next token of one user: the usual top-64, top-0.95
        sample("sample_1", b=1, v=262144, dt="f32", k=64, p=0.95, m=0.0, t=1.0),
        # eight users, nucleus only: the set can be any part of the vocabulary
        sample("sample_8_top_p", b=8, v=262144, dt="f32", k=0, p=0.9, m=0.0, t=1.3),
        # a large batch with settings that differ from row to row
        sample("sample_192_mixed", b=192, v=262144, dt="f32", k=-1, p=-1.0, m=-1.0, t=-1.0),
    ]


def append(name=None, **kw):
    c = {"op": "append", "page": 16, "rot": kw["d"], "theta": 1e4, "interleaved": False, "ragged": False, **kw}
    return {"name": name, **c} if name else c


def attend(name=None, **kw):
    c = {"op": "attend", "page": 16, "window": 0, "ragged": False, **kw}
    return {"name": name, **c} if name else c


def sample(name=None, **kw):
    return {"name": name, "op": "sample", **kw} if name else {"op": "sample", **kw}


def log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "sample"])
    page = rng.choice([16, 32, 64, 128])
    dt = rng.choice(["f16", "bf16"])
    if op == "sample":
        b, v = log_int(rng, 1, 192), log_int(rng, 1000, 262144)
        k = rng.choice([0, 1, log_int(rng, 2, 1000), log_int(rng, 2, 200000)])
        p = rng.choice([1.0, rng.uniform(0.1, 0.99)])
        m = rng.choice([0.0, rng.uniform(0.001, 0.2)])
        return sample(b=b, v=v, dt=rng.choice(["f32", "f32", dt]), k=k, p=round(p, 4), m=round(m, 4), t=round(rng.uniform(0.3, 2.0), 3))
    d = rng.choice([64, 128, 256, 256, 512])
    hkv = rng.choice([1, 1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    ragged = rng.choice([True, False])
    if op == "append":
        b = log_int(rng, 1, 64)
        most = max(1, 16 * 4096 * 10 * 256 // (b * (group + 2) * hkv * d))
        new = log_int(rng, 1, min(4096, most))
        return append(b=b, new=new, ctx=new + log_int(rng, 1, 4096), hq=group * hkv, hkv=hkv, d=d, inp=rng.choice(["f32", dt]), dt=dt,
                      page=page, rot=rng.choice([d, d // 2]), theta=rng.choice([1e4, 1e6]), interleaved=rng.choice([True, False]), ragged=ragged)
    kind = rng.choice(["decode", "verify", "chunk"])
    new = {"decode": 1, "verify": rng.randint(2, 8), "chunk": log_int(rng, 9, 2048)}[kind]
    b = log_int(rng, 1, 4 if kind == "chunk" else 128)
    kv = max(64, 64 * 16384 * 512 // (b * hkv * d))                               # cache elements of the largest listed case
    sq = max(64, 4 * 4096 * 8192 * 8 * 256 // (b * new * group * hkv * d))        # work of the largest listed case
    ctx = new + log_int(rng, 1, max(1, min(32768, kv - new, sq - new)))
    return attend(b=b, new=new, ctx=ctx, hq=group * hkv, hkv=hkv, d=d, dt=dt, page=page, window=rng.choice([0, 0, 512, 1024]), ragged=ragged)


def lengths(case):
    """New tokens and cache length after the append, per sequence."""
    b, new, ctx = case["b"], case["new"], case["ctx"]
    f = [((i + 1) * GOLDEN) % 1.0 if case["ragged"] else 1.0 for i in range(b)]
    n = [max(1, round(new * (0.25 + 0.75 * x))) for x in f]
    return n, [n[i] + round((ctx - new) * (0.2 + 0.8 * ((f[i] * 7.3) % 1.0 if case["ragged"] else 1.0))) for i in range(b)]


DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def work(case):
    if case["op"] == "sample":
        n = case["b"] * case["v"]
        return {"bytes": n * SIZE[case["dt"]] + case["b"] * 28, "flops": 4.0 * n}
    n, kv = lengths(case)
    hq, hkv, d, t = case["hq"], case["hkv"], case["d"], sum(n)
    if case["op"] == "append":
        return {"bytes": t * (hq + 2 * hkv) * d * (SIZE[case["inp"]] + SIZE[case["dt"]]), "flops": 3.0 * t * (hq + hkv) * case["rot"]}
    w = case["window"]
    pairs = keys = 0
    pairs = sum(visible(n[i], kv[i], w) for i in range(case["b"]))
    keys = sum(min(kv[i], w + n[i] - 1) if w else kv[i] for i in range(case["b"]))
    return {"bytes": 2 * (2 * t * hq * d + 2 * keys * hkv * d) + 4 * t * hq, "flops": 4.0 * pairs * hq * d}


def visible(n, kv, w):
    """(query, key) pairs of n new tokens at the end of kv keys, with a window of w keys (0: none)."""
    first = kv - n + 1                                        # keys that the first new token sees
    if not w or kv <= w:
        return n * first + n * (n - 1) // 2
    full = max(0, min(n, kv - max(w, first) + 1)) if first <= w else n
    below = n - full
    return below * first + below * (below - 1) // 2 + full * w


def steps_of(rot, theta, device):
    """Turns per position of each rotary pair, in units of 2^-64."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    return (torch.pow(torch.tensor(theta, dtype=torch.float64), -2.0 * i / rot) / (2 * math.pi) * 2.0 ** 64).to(torch.int64).to(device)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    b = case["b"]

    def normal(*shape, dtype, std=1.0):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).mul_(std).to(dtype)

    if case["op"] == "sample":
        v = case["v"]
        z = torch.randn(b, v, generator=g, device=dev).mul_(2.5)
        z.scatter_add_(1, torch.randint(0, v, (b, 12), generator=g, device=dev), torch.rand(b, 12, generator=g, device=dev) * 8)   # the few likely words
        z = (30.0 * torch.tanh(z / 30.0)).to(DTYPES[case["dt"]])                   # as the head's softcap leaves them
        i = torch.arange(b, device=dev)
        mixed = case["k"] < 0
        k = torch.tensor([0, 64, 40, 1000, 1, 0], device=dev, dtype=torch.int32)[i % 6] if mixed else torch.full((b,), case["k"], dtype=torch.int32, device=dev)
        p = torch.tensor([0.9, 0.95, 1.0, 0.99, 1.0, 1.0], device=dev)[i % 6] if mixed else torch.full((b,), case["p"], device=dev)
        m = torch.tensor([0.0, 0.0, 0.05, 0.0, 0.0, 0.02], device=dev)[i % 6] if mixed else torch.full((b,), case["m"], device=dev)
        t = torch.tensor([0.8, 1.0, 0.7, 1.2, 1.0, 1.5, 0.6], device=dev)[i % 7] if mixed else torch.full((b,), case["t"], device=dev)
        return {"case": case, "z": z, "u": torch.rand(b, generator=g, device=dev), "k": k, "p": p, "m": m, "t": t}

    n, kv = lengths(case)
    hq, hkv, d, page, dt = case["hq"], case["hkv"], case["d"], case["page"], DTYPES[case["dt"]]
    pages = [-(-x // page) for x in kv]
    total, most = sum(pages) + 8, max(pages)
    order = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    start = torch.tensor([0] + pages, device=dev).cumsum(0)
    slot = torch.arange(most, device=dev)[None, :].expand(b, most)
    held = slot < torch.tensor(pages, device=dev)[:, None]
    table = torch.where(held, order[(start[:-1, None] + slot).clamp(max=total - 1)], torch.full_like(order[:1], -1)).contiguous()
    s = {
        "case": case, "table": table, "max_q": max(n),
        "cu": torch.tensor([0] + n, device=dev).cumsum(0).to(torch.int32),
        "kv": torch.tensor(kv, device=dev, dtype=torch.int32),
        "kc": normal(total, hkv, page, d, dtype=dt), "vc": normal(total, hkv, page, d, dtype=dt),
    }
    t = sum(n)
    if case["op"] == "append":
        fused = normal(t, (hq + 2 * hkv) * d, dtype=DTYPES[case["inp"]])           # one row of the fused projection per token
        s["q"] = fused[:, : hq * d].view(t, hq, d)
        s["k"] = fused[:, hq * d: (hq + hkv) * d].view(t, hkv, d)
        s["v"] = fused[:, (hq + hkv) * d:].view(t, hkv, d)
        s["steps"] = steps_of(case["rot"], case["theta"], dev)
    else:
        s["q"] = normal(t, hq, d, dtype=dt, std=1.7)
        s["scale"] = d ** -0.5
    return s


def run(s):
    op = s["case"]["op"]
    if op == "append":
        return run_append(s)
    return run_attend(s) if op == "attend" else run_sample(s)


def places(s):
    """Sequence of every token and its position in that sequence's cache."""
    cu, kv = s["cu"].long(), s["kv"].long()
    tok = torch.arange(s["q"].shape[0], device=cu.device)
    seq = torch.searchsorted(cu, tok, right=True) - 1
    return tok, seq, kv[seq] - cu[seq + 1] + tok


def run_append(s):
    case = s["case"]
    if own:
        import int4_q4_weight_gb300 as q4w
        q = q4w.kv_append(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["cu"], s["kv"], s["steps"], q=s["q"], interleaved=case["interleaved"])
        return {"q": q, "k_cache": s["kc"], "v_cache": s["vc"]}
    rot, page = case["rot"], case["page"]
    _, seq, pos = places(s)
    i = torch.arange(rot // 2, dtype=torch.float64, device=pos.device)
    angle = pos.double()[:, None] * torch.pow(torch.tensor(case["theta"], dtype=torch.float64, device=pos.device), -2.0 * i / rot)
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]

    def rotate(x):
        y = x.float()
        r = y[..., :rot]
        a, c = (r[..., 0::2], r[..., 1::2]) if case["interleaved"] else (r[..., : rot // 2], r[..., rot // 2:])
        a2, c2 = a * cos - c * sin, c * cos + a * sin
        r = torch.stack((a2, c2), -1).flatten(-2) if case["interleaved"] else torch.cat((a2, c2), -1)
        return torch.cat((r, y[..., rot:]), -1).to(s["kc"].dtype)

    where = s["table"].long()[seq, pos // page]
    s["kc"][where, :, pos % page] = rotate(s["k"])
    s["vc"][where, :, pos % page] = s["v"].to(s["vc"].dtype)
    return {"q": rotate(s["q"]), "k_cache": s["kc"], "v_cache": s["vc"]}


def run_attend(s):
    case = s["case"]
    if own:
        import int4_q4_weight_gb300 as q4w
        lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=s["q"].device)
        out, lse = q4w.kv_attention(s["q"], s["kc"], s["vc"], s["table"], s["cu"], s["kv"], s["max_q"], scale=s["scale"], window=case["window"], lse=lse)
        return {"out": out, "lse": lse}
    q, b, hkv, d, page, w = s["q"], case["b"], case["hkv"], case["d"], case["page"], case["window"]
    group = case["hq"] // hkv
    tok, seq, pos = places(s)
    most = s["table"].shape[1] * page
    table = s["table"].long().clamp(min=0)
    # keys and values of every sequence in order: [b, hkv, most, d]
    keys = s["kc"][table].transpose(1, 2).reshape(b, hkv, most, d).float()
    held = torch.arange(most, device=q.device)[None, :] < s["kv"].long()[:, None]
    vals = torch.where(held[:, None, :, None], s["vc"][table].transpose(1, 2).reshape(b, hkv, most, d).float(), 0.0)
    at = tok - s["cu"].long()[seq]
    rows = torch.zeros(b, s["max_q"], case["hq"], d, device=q.device)
    rows[seq, at] = q.float()
    here = torch.full((b, s["max_q"]), -1, dtype=torch.long, device=q.device)
    here[seq, at] = pos
    rows = rows.view(b, -1, hkv, group, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, d)
    score = (rows @ keys.transpose(2, 3)).mul_(s["scale"]).view(b, hkv, s["max_q"], group, most)
    c = torch.arange(most, device=q.device)[None, None, :]
    seen = c <= here[:, :, None]
    if w:
        seen &= c > here[:, :, None] - w
    score.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    e = score.sub_(top).exp_()
    total = e.sum(-1, keepdim=True)
    out = (e.view(b, hkv, -1, most) @ vals).view(b, hkv, s["max_q"], group, d) / total.clamp(min=1e-38)
    lse = (total.log() + top)[..., 0]
    out = out.permute(0, 2, 1, 3, 4).reshape(b, s["max_q"], case["hq"], d)[seq, at]
    return {"out": out.to(q.dtype), "lse": lse.permute(0, 2, 1, 3).reshape(b, s["max_q"], case["hq"])[seq, at].contiguous()}


def run_sample(s):
    if own:
        import int4_q4_weight_gb300 as q4w
        tokens, logprobs = q4w.logits_sample(s["z"], s["u"], s["t"], s["k"], s["p"], s["m"])
        return {"token": tokens, "logprob": logprobs}
    b, v = s["z"].shape
    # 64 bits: a sum of many small weights decides which side of a border a token falls on
    z = s["z"].double()
    z, index = torch.sort(z, dim=1, descending=True, stable=True)
    weight = ((z - z[:, :1]) / s["t"].double()[:, None]).exp()
    rank = torch.arange(v, device=z.device)[None, :]
    k = torch.where(s["k"] <= 0, torch.full_like(s["k"], v), s["k"]).long()[:, None]
    weight = torch.where(rank < k, weight, 0.0)
    before = weight.cumsum(1) - weight
    p, m = s["p"].double()[:, None], s["m"].double()[:, None]
    keep = (rank == 0) | ((p >= 1) | (before < p * weight.sum(1, keepdim=True))) & (weight >= m) & (rank < k)
    weight = torch.where(keep, weight, 0.0)
    total = weight.sum(1, keepdim=True)
    # back in the order of the vocabulary
    weight = torch.zeros_like(weight).scatter_(1, index, weight)
    running = weight.cumsum(1)
    token = ((running <= s["u"].double()[:, None] * total) | (weight == 0)).to(torch.int8).argmin(1, keepdim=True)
    logprob = (weight.gather(1, token) / total).log()
    return {"token": token[:, 0].to(torch.int32), "logprob": logprob[:, 0].float()}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return exact_append(s)
    return exact_attend(s) if case["op"] == "attend" else exact_sample(s)


def exact_append(s):
    """Each pair as a complex number, multiplied by exp(i angle)."""
    case = s["case"]
    n, kv = lengths(case)
    rot, page, kc, vc = case["rot"], case["page"], s["kc"].double(), s["vc"].double()
    qs, t0 = [], 0
    for i in range(case["b"]):
        pos = torch.arange(kv[i] - n[i], kv[i], device=kc.device)
        inv = torch.exp(torch.arange(rot // 2, device=kc.device, dtype=torch.float64) * (-2.0 * math.log(case["theta"]) / rot))
        turn = torch.polar(torch.ones(n[i], rot // 2, device=kc.device, dtype=torch.float64), torch.outer(pos.double(), inv))[:, None]
        span = slice(t0, t0 + n[i])

        def rotated(x):
            x = x[span].double().clone()
            if case["interleaved"]:
                x[..., :rot] = torch.view_as_real(torch.view_as_complex(x[..., :rot].reshape(*x.shape[:2], rot // 2, 2).contiguous()) * turn).flatten(-2)
            else:
                y = torch.complex(x[..., : rot // 2], x[..., rot // 2: rot]) * turn
                x[..., : rot // 2], x[..., rot // 2: rot] = y.real, y.imag
            return x

        pages = s["table"][i].long()[torch.div(pos, page, rounding_mode="floor")]
        kc[pages, :, pos % page] = rotated(s["k"])
        vc[pages, :, pos % page] = s["v"][span].double()
        qs.append(rotated(s["q"]))
        t0 += n[i]
    return {"q": torch.cat(qs), "k_cache": kc, "v_cache": vc}


def exact_attend(s):
    """One sequence and one KV head after the other, over its own keys."""
    case = s["case"]
    n, kv = lengths(case)
    hkv, hq, d, w = case["hkv"], case["hq"], case["d"], case["window"]
    if sum(4.0 * n[i] * kv[i] * hq * d for i in range(case["b"])) > 6e12:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=s["q"].device)
    t0 = 0
    for i in range(case["b"]):
        used = s["table"][i][s["table"][i] >= 0].long()
        mask = torch.ones(n[i], kv[i], dtype=torch.bool, device=out.device).tril(kv[i] - n[i])
        if w:
            mask &= ~torch.ones_like(mask).tril(kv[i] - n[i] - w)
        for h in range(hkv):
            k = s["kc"][used, h].reshape(-1, d)[: kv[i]].double()
            v = s["vc"][used, h].reshape(-1, d)[: kv[i]].double()
            for j in range(h * hq // hkv, (h + 1) * hq // hkv):
                sc = torch.where(mask, s["scale"] * (s["q"][t0: t0 + n[i], j].double() @ k.T), -math.inf)
                lse[t0: t0 + n[i], j] = torch.logsumexp(sc, 1)
                out[t0: t0 + n[i], j] = torch.softmax(sc, 1) @ v
        t0 += n[i]
    return {"out": out, "lse": lse}


def exact_sample(s):
    """Row by row over the kept tokens alone."""
    got = []
    for r in range(s["z"].shape[0]):
        z = s["z"][r].double()
        i = torch.argsort(z, descending=True, stable=True)
        i = i[: int(s["k"][r])] if int(s["k"][r]) > 0 else i
        prob = torch.softmax(z[i] / s["t"][r].double(), 0)
        if float(s["p"][r]) < 1:
            i = i[: 1 + int((prob.cumsum(0) < s["p"][r].double()).sum())]
        prob = prob[: i.numel()]
        i = i[prob / prob[0] >= s["m"][r].double()]
        i = torch.sort(i)[0]
        prob = torch.softmax(z[i] / s["t"][r].double(), 0)
        at = int((prob.cumsum(0) <= s["u"][r].double()).sum())
        got.append(torch.log(prob[min(at, i.numel() - 1)]))
    return {"token": None, "logprob": torch.stack(got)}
