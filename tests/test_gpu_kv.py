"""kv_append and kv_attention against the fp64 oracle.

Tolerances (eps: the type's machine epsilon; a rounding is off by at most
eps/2 of the value).
Append: the angle's fraction is rounded to fp32 once (2^-25 half turns, 1e-7
rad), sine and cosine are good to 2 ulp (2.4e-7), the two products and the sum
round three more times (1.8e-7): below 6e-7 of the pair's length, then one
rounding to the output type.  V and unturned elements are one rounding.
Attention: with A = sum p|v| the probabilities' rounding costs eps/2 A (and
2^-25 absolute per key where fp16 runs out of exponent), the output's eps/2 |o|.
A score is a sum of D products in fp32, S = scale sum |q k| at most: off by
8 2^-24 S for sums in pieces of a few dozen, twice that in a ratio; exponentials
and sums add 2e-6 of A.
"""
import math

import numpy as np
import pytest
import torch

from oracle import kv_oracle as O

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def normal(gen, *shape, dtype=F16, std=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)


class Case:
    """Tables and caches of sequences with n[i] new tokens at the end of kv[i]."""

    def __init__(self, n, kv, hq=8, hkv=1, D=256, page=16, dtype=F16, seed=0, std=1.0, pad=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.gen, self.n, self.kv, self.hq, self.hkv, self.D, self.page, self.dtype = g, n, kv, hq, hkv, D, page, dtype
        need = [-(-x // page) for x in kv]
        self.pages = sum(need) + 3
        self.max_pages = max(need + [1]) + 1
        order = torch.randperm(self.pages, generator=g, device="cuda").cpu().numpy()
        table = np.full((len(n), self.max_pages), -7, np.int32)
        at = 0
        for i, x in enumerate(need):
            table[i, :x] = order[at:at + x]
            at += x
        self.table = torch.from_numpy(table).cuda()
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).cuda()
        self.kvl = torch.tensor(kv, dtype=torch.int32, device="cuda")
        self.T = sum(n) + pad
        self.kc = normal(g, self.pages, hkv, page, D, dtype=dtype, std=std)
        self.vc = normal(g, self.pages, hkv, page, D, dtype=dtype)
        self.q = normal(g, self.T, hq, D, dtype=dtype, std=std)

    def stale(self, value):
        """Fills everything that holds no position."""
        keep = torch.zeros(self.pages, self.page, dtype=torch.bool)
        t = self.table.cpu().numpy()
        for i, x in enumerate(self.kv):
            for c in range(x):
                keep[t[i, c // self.page], c % self.page] = True
        drop = (~keep).cuda()[:, None, :, None].expand_as(self.kc)
        self.kc[drop] = value
        self.vc[drop] = value
        return self

    def host(self):
        return (self.kc.float().cpu().numpy(), self.vc.float().cpu().numpy(), self.table.cpu().numpy(),
                self.cu.cpu().numpy(), self.kvl.cpu().numpy())

    def tables(self):
        return self.kc, self.vc, self.table, self.cu, self.kvl


def check_attention(q4w, c, scale=None, window=0, max_q=None, q=None, err=0, **kw):
    scale = c.D ** -0.5 if scale is None else scale
    q = c.q if q is None else q
    lse = torch.full((c.T, c.hq), 77.0, device="cuda")
    out = torch.full((c.T, c.hq, c.D), 77.0, dtype=c.dtype, device="cuda")
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    q4w.kv_attention(q, *c.tables(), max_q=max(c.n) if max_q is None else max_q, scale=scale, window=window, out=out,
                     lse=lse, err=flag, **kw)
    q4w.q4_device_status()
    ro, rl, A, S = O.attention(q.float().cpu().numpy(), *c.host(), scale, window)
    go, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    pad = np.isnan(rl)
    assert np.all(gl[pad] == 77.0) and np.all(go[pad] == 77.0), "padding tokens were written"
    go, gl, ro, rl, A, S = go[~pad], gl[~pad], ro[~pad], rl[~pad], A[~pad], S[~pad]
    assert int(flag) == err
    empty = rl == -np.inf
    assert np.array_equal(gl == -np.inf, empty)
    assert np.all(go[empty] == 0)
    half = torch.finfo(c.dtype).eps / 2
    ds = 8 * 2.0 ** -24 * S
    n = max(c.kv + [1])
    vmax = np.abs(A).max() if A.size else 0
    small = n * 2.0 ** -25 * 4 * max(vmax, 1) / max(1.0, math.sqrt(n)) if c.dtype == F16 else 0.0
    tol = half * (A + np.abs(ro)) * 1.01 + (2 * ds[..., None] + 2e-6) * A + small + 1e-30
    bad = ~(np.abs(go - ro) <= tol)
    assert not bad.any(), (int(bad.sum()), float((np.abs(go - ro) / tol).max()))
    assert np.all(np.abs(gl[~empty] - rl[~empty]) <= (ds + 2e-6 * (1 + np.abs(rl)))[~empty])
    return out, lse


# ------------------------------------------------------------------ append ---
@pytest.mark.parametrize("D,hq,hkv,rot,inter,inp,dtype,page", [
    (256, 8, 1, 256, False, F32, F16, 16),
    (512, 8, 1, 128, False, F16, F16, 16),
    (512, 3, 1, 512, True, BF16, BF16, 48),
    (128, 6, 2, 64, True, F32, BF16, 32),
    (64, 1, 1, 64, False, BF16, F16, 128),
    (64, 10, 5, 16, False, F16, BF16, 16),
    (128, 0, 3, 0, False, F16, F16, 16),
])
def test_append(cuda_lib, D, hq, hkv, rot, inter, inp, dtype, page):
    q4w = cuda_lib
    n, kv = [1, 5, 0, 17, 1, 40], [1, 30, 9, 17, 200, 65]
    c = Case(n, kv, max(hq, 1), hkv, D, page, dtype, pad=2)
    fused = normal(c.gen, c.T, (hq + 2 * hkv) * D, dtype=inp)        # rows of a fused projection
    q = fused[:, :hq * D].view(c.T, hq, D) if hq else None
    k, v = fused[:, hq * D:(hq + hkv) * D].view(c.T, hkv, D), fused[:, (hq + hkv) * D:].view(c.T, hkv, D)
    freqs = 10000.0 ** (-np.arange(rot // 2) * 2.0 / max(rot, 1))
    before = c.host()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    steps = q4w.kv_rope_steps(rot, device="cuda") if rot else None
    q_out = torch.full((c.T, hq, D), 77.0, dtype=dtype, device="cuda") if hq else None
    q4w.kv_append(k, v, *c.tables(), steps=steps, q=q, interleaved=inter, q_out=q_out, err=err)
    assert int(err) == 0
    f = lambda t: t.double().cpu().numpy()   # noqa: E731
    rk, rv = O.append(f(k), f(v), *before, freqs, inter)
    half = torch.finfo(dtype).eps / 2

    def close(got, ref, src):
        length = np.abs(src).max(-1, keepdims=True) * 1.5
        assert np.all(np.abs(got - ref) <= half * np.abs(ref) * 1.01 + 6e-7 * length + 2.0 ** -25)

    assert np.array_equal(f(c.vc), rv if dtype == inp else torch.tensor(rv).to(F32).to(dtype).double().numpy())
    close(f(c.kc), rk, rk)
    if hq:
        for t, s, pos in O.tokens(before[3], before[4]):
            close(f(q_out[t]), O.rotate(f(q[t]), pos, freqs, inter), f(q[t]))
        assert torch.all(q_out[sum(n):] == 77.0)                    # padding tokens


def test_append_far_positions(cuda_lib):
    """Angles of positions that fp32 cannot hold, given and from the cache."""
    q4w = cuda_lib
    c = Case([4], [70], D=128)
    k = normal(c.gen, 4, 1, 128, dtype=F32)
    pos = torch.tensor([1048575, 16777217, 2 ** 31 - 1, -5], dtype=torch.int32, device="cuda")
    q = q4w.kv_append(k, k, *c.tables(), steps=q4w.kv_rope_steps(128), q=k, positions=pos)
    freqs = 10000.0 ** (-np.arange(64) / 64)
    x = k.double().cpu().numpy()
    for t in range(4):
        p = int(pos[t])
        ref = O.rotate(x[t], p, freqs, False)
        # the oracle's fp64 angle and the 2^-53 of the frequency are off by p 2^-52
        tol = 2.0 ** -11 * np.abs(ref) + (6e-7 + abs(p) * 2.0 ** -51) * np.abs(x[t]).max() * 1.5 + 2.0 ** -25
        assert np.all(np.abs(q[t].double().cpu().numpy() - ref) <= tol), t


def test_append_bad_places_store_nothing(cuda_lib):
    """Negative positions, positions behind the table and pages outside the cache."""
    q4w = cuda_lib
    c = Case([3, 2, 2, 1], [1, 40, 16, 5], D=64, hq=2)
    c.kvl[1] = 16 * c.max_pages + 1            # the second token is behind the table
    c.table[2, 0] = c.pages                    # no page
    before = c.host()
    k = normal(c.gen, c.T, 1, 64)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.table[1, c.max_pages - 1] = c.pages - 1  # the first one has a place
    before = c.host()
    q4w.kv_append(k, k, *c.tables(), err=err)
    torch.cuda.synchronize()
    assert int(err) == 1
    rk, rv = O.append(k.float().cpu().numpy(), k.float().cpu().numpy(), *before, [])
    assert np.array_equal(c.kc.double().cpu().numpy(), rk) and np.array_equal(c.vc.double().cpu().numpy(), rv)
    assert not np.array_equal(before[0], c.kc.float().cpu().numpy())


def test_append_many_sequences(cuda_lib):
    q4w = cuda_lib
    n = [(i * 7) % 3 for i in range(1500)]
    c = Case(n, [x + (i % 5) for i, x in enumerate(n)], D=64, hq=1)
    k = normal(c.gen, c.T, 1, 64)
    before = c.host()
    q4w.kv_append(k, k, *c.tables(), steps=q4w.kv_rope_steps(64))
    rk, rv = O.append(k.float().cpu().numpy(), k.float().cpu().numpy(), *before, 10000.0 ** (-np.arange(32) / 32))
    assert np.array_equal(c.vc.double().cpu().numpy(), rv)
    assert np.all(np.abs(c.kc.double().cpu().numpy() - rk) <= 2.0 ** -11 * np.abs(rk) * 1.01 + 6e-6 + 2.0 ** -25)


@pytest.mark.parametrize("D,K", [(256, 1536), (512, 12288)])
def test_append_right_behind_the_projection(cuda_lib, D, K):
    """The stage that writes q, k and v lets the next kernel start early: the append
    reads what it writes, not what lay there before, eagerly and in a graph."""
    q4w = cuda_lib
    c = Case([1], [37], 8, 1, D)
    rows = (8 * D, D, D)
    mats = [q4w.q4_quantize(normal(c.gen, n, K, dtype=F32, std=0.05)) for n in rows]
    out = [torch.empty(n, device="cuda") for n in rows]
    x = torch.empty(K, dtype=F16, device="cuda")
    steps = q4w.kv_rope_steps(D)
    q_out = torch.empty(1, 8, D, dtype=F16, device="cuda")

    def append(q, k, v):
        q4w.kv_append(k.view(1, 1, D), v.view(1, 1, D), *c.tables(), steps=steps, q=q.view(1, 8, D), q_out=q_out)

    def both():
        q4w.q4_gemv_stage(mats, x, q4w.Q4_IN_F16, out32=out)
        append(*out)

    page, slot = int(c.table[0, 36 // 16]), 36 % 16
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        both()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    for i in range(12):
        x.copy_(normal(c.gen, K))
        q4w.q4_gemv_stage(mats, x, q4w.Q4_IN_F16, out32=out)
        torch.cuda.synchronize()
        append(*[t.clone() for t in out])
        torch.cuda.synchronize()
        want = [t.clone() for t in (q_out, c.kc[page, 0, slot], c.vc[page, 0, slot])]
        for t in out:
            t.fill_(77.0)
        for t in (q_out, c.kc, c.vc):
            t.fill_(33.0)
        torch.cuda.synchronize()
        g.replay() if i % 2 else both()
        torch.cuda.synchronize()
        for a, b in zip(want, (q_out, c.kc[page, 0, slot], c.vc[page, 0, slot])):
            assert torch.equal(a, b), i


# --------------------------------------------------------------- attention ---
@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hq,hkv", [(8, 1), (4, 4), (6, 2), (5, 1), (16, 1), (1, 1)])
def test_attention_single_tokens(cuda_lib, D, dtype, hq, hkv):
    c = Case([1] * 6, [1, 2, 15, 16, 17, 333], hq, hkv, D, 16, dtype, seed=D + hq).stale(float("nan"))
    check_attention(cuda_lib, c)


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hq,hkv,page", [(8, 1, 16), (4, 2, 64), (7, 1, 48), (3, 3, 128)])
def test_attention_chunks(cuda_lib, D, dtype, hq, hkv, page):
    """Ragged chunks: no new token, one, the whole sequence, tiles that end inside pages."""
    c = Case([1, 64, 0, 33, 130, 5], [1, 64, 40, 200, 259, 128], hq, hkv, D, page, dtype, seed=D + hq, pad=3).stale(float("nan"))
    check_attention(cuda_lib, c)


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("hq,new", [(1, 7), (3, 3), (8, 2), (5, 4), (8, 3), (8, 4), (16, 2), (7, 5), (1, 40), (16, 9), (100, 1), (128, 2)])
def test_attention_any_number_of_query_rows(cuda_lib, D, hq, new):
    """1 to 256 query rows per KV head: every choice of kernel, groups that do not divide a tile."""
    check_attention(cuda_lib, Case([new, 1, new], [new, 100, 300 + new], hq, 1, D, 16, BF16, seed=hq))


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("rows", [7, 8, 9, 15, 16, 17, 31, 32, 33, 127, 128, 129, 255, 256, 257])
def test_attention_rows_next_to_the_kernels_limits(cuda_lib, D, rows):
    """Rows per KV head around the sizes at which another kernel or tile begins, as
    tokens of one head and as heads of few tokens."""
    for hq, new in [(1, rows)] + [(h, rows // h) for h in (rows, rows // 2, 3) if h <= 128 and rows % h == 0 and h > 1]:
        check_attention(cuda_lib, Case([new, 1, new], [new, 70, 190 + new], hq, 1, D, 16, F16, seed=rows + hq))


@pytest.mark.parametrize("D,hq,hkv", [(64, 8, 2), (256, 8, 1), (512, 8, 1), (128, 4, 4)])
@pytest.mark.parametrize("new", [1, 2, 4, 9, 70])
@pytest.mark.parametrize("window", [1, 17, 100, 512])
def test_attention_window(cuda_lib, D, hq, hkv, new, window):
    kv = [new, new + 16, new + 150, new + 777]
    c = Case([new] * 4, kv, hq, hkv, D, 16, F16, seed=window).stale(float("inf"))
    # pages that slid out of every token's reach are freed
    for i, x in enumerate(kv):
        c.table[i, :max(0, x - new + 1 - window) // 16] = -1
    check_attention(cuda_lib, c, window=window)


@pytest.mark.parametrize("D,hq", [(256, 8), (512, 8), (64, 2), (128, 1)])
@pytest.mark.parametrize("new", [1, 40])
def test_attention_long_and_split(cuda_lib, D, hq, new):
    """Lengths that are split over many CTAs next to short ones."""
    c = Case([new, new, 1], [5003, new, 2001], hq, 1, D, 32, BF16, seed=new, std=1.4)
    check_attention(cuda_lib, c)


@pytest.mark.parametrize("D,n,kv", [(256, [400, 3], [2000, 900]), (512, [100], [4000]), (512, [200, 3], [700, 900]),
                                    (128, [900], [2500]), (64, [1000, 70], [1500, 3000])])
def test_attention_several_steps_and_items_per_cta(cuda_lib, D, n, kv):
    """More steps than SMs: shares of several steps that end and begin inside items."""
    check_attention(cuda_lib, Case(n, kv, 8, 1, D, 64, F16, seed=D))


@pytest.mark.parametrize("D,hq,hkv,seqs,new", [(512, 16, 2, 100, 9), (512, 8, 8, 20, 90), (512, 64, 1, 200, 1), (256, 32, 2, 200, 9), (128, 40, 2, 200, 9),
                                               (64, 80, 2, 200, 9)])
@pytest.mark.parametrize("window", [0, 100])
def test_attention_many_short_items_one_after_the_other(cuda_lib, D, hq, hkv, seqs, new, window):
    """Items of a few steps, most of which end inside a step, whose keys come late (the
    cache is larger than L2): right, and the same bits every time."""
    g = np.random.default_rng(D + seqs)
    n = [int(x) for x in g.integers(1, new + 1, seqs)]
    kv = [x + int(g.choice([g.integers(0, 40), g.integers(100, 600), g.integers(0, 1500)])) for x in n]
    c = Case(n, kv, hq, hkv, D, 16, BF16, seed=seqs).stale(float("inf"))
    out, lse = check_attention(cuda_lib, c, window=window)
    again, flush = torch.empty_like(out), torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for i in range(60):
        if i % 2:
            flush.fill_(i)
        cuda_lib.kv_attention(c.q, *c.tables(), max_q=max(n), window=window, out=again)
        assert torch.equal(out, again), i


@pytest.mark.parametrize("D,hq,hkv,new", [(256, 8, 1, 1), (512, 8, 1, 1), (64, 3, 1, 1), (256, 8, 1, 64), (512, 4, 1, 50), (128, 4, 2, 90)])
def test_attention_rows_that_see_nothing(cuda_lib, D, hq, hkv, new):
    """A length of zero, and lengths shorter than the new tokens."""
    c = Case([new, new, new], [0, 3, 200], hq, hkv, D, 16, F16).stale(float("nan"))
    if new == 1:
        c = Case([1, 1, 1], [0, 1, 200], hq, hkv, D, 16, F16).stale(float("nan"))
    check_attention(cuda_lib, c)
    c.kvl.zero_()
    c.kv = [0, 0, 0]
    check_attention(cuda_lib, c)


@pytest.mark.parametrize("D,hq,new", [(256, 1, 6), (512, 1, 8), (64, 3, 9), (256, 8, 64), (512, 4, 50), (128, 4, 90)])
@pytest.mark.parametrize("window", [40, 2 ** 31 - 1])
def test_attention_lengths_shorter_than_the_new_tokens_with_a_window(cuda_lib, D, hq, new, window):
    """Tokens at negative positions see nothing, the others what the window leaves, as
    far as the largest window that there is."""
    c = Case([new, new, new, new], [0, 3, new - 1, 200], hq, 1, D, 16, F16, seed=new).stale(float("nan"))
    check_attention(cuda_lib, c, window=window)


@pytest.mark.parametrize("D,new", [(256, 1), (256, 40), (512, 1), (512, 40), (64, 6)])
def test_attention_scores_of_any_size(cuda_lib, D, new):
    """Scores far apart, all equal, huge, negative scale, and one key that takes all."""
    c = Case([new, new], [300, 77 + new], D=D, seed=3)
    check_attention(cuda_lib, c, scale=0.0)
    check_attention(cuda_lib, c, scale=-0.3)
    check_attention(cuda_lib, c, scale=1.0)
    c.kc[:, :, :, 0] = 0
    q = c.q.clone()
    q[..., 0] = 600.0
    t = c.table.cpu().numpy()
    for pos, val in ((290, 60.0), (17, 30.0), (250, -60.0)):
        if pos < 300 - new:
            c.kc[t[0, pos // 16], 0, pos % 16, 0] = val
    check_attention(cuda_lib, c, q=q, scale=1.0)


@pytest.mark.parametrize("D,new,seqs,n", [(256, 1, 160, 1500), (64, 3, 160, 1500), (128, 2, 160, 1500), (512, 1, 160, 1500), (256, 1, 1, 20000),
                                          (256, 40, 90, 600), (256, 40, 1, 20000), (64, 70, 1, 20000), (512, 20, 1, 20000)])
@pytest.mark.parametrize("depth", [12.0, 16.3, 20.4, 24.8])
def test_attention_many_keys_of_small_probability(cuda_lib, D, new, seqs, n, depth):
    """One key that takes nearly all, and thousands of 2^-depth each whose values alone
    make the output: their sum keeps the precision of 16 bits.  fp16 is the narrow type;
    its probabilities have an absolute error of 2^-32 of the largest (a key's is 2^-depth)."""
    q4w = cuda_lib
    c = Case([new] * seqs, [n] * seqs, 2, 1, D, 64, F16, seed=new)
    c.kc.zero_()
    c.kc[..., 0] = -depth * math.log(2.0)
    c.vc.fill_(1.0)
    sink = n // 3                                       # before every new token
    pages = c.table[:, sink // 64].long()
    c.kc[pages, 0, sink % 64, 0] = 0.0
    c.vc[pages, 0, sink % 64] = 0.0
    q = torch.zeros_like(c.q)
    q[..., 0] = 1.0
    out, _ = q4w.kv_attention(q, *c.tables(), max_q=new, scale=1.0)
    q4w.q4_device_status()
    ro, _, A, S = O.attention(q.float().cpu().numpy(), *c.host(), 1.0)
    tol = 2.0 ** -11 * (A + np.abs(ro)) * 1.01 + (16 * 2.0 ** -24 * S[..., None] + 2e-6) * A + 2.0 ** (depth - 32) * ro + 2.0 ** -25
    err = np.abs(out.double().cpu().numpy() - ro)
    assert np.all(err <= tol), float((err / tol).max())


@pytest.mark.parametrize("new,hq", [(1, 8), (64, 8), (4, 8)])
def test_attention_strided_queries_and_order(cuda_lib, new, hq):
    c = Case([new] * 3, [new + 100, new + 7, new], hq, 1, 256, 16, F16)
    fused = normal(c.gen, c.T, (hq + 2) * 256)
    check_attention(cuda_lib, c, q=fused[:, 256:(hq + 1) * 256].view(c.T, hq, 256))


@pytest.mark.parametrize("new,D", [(1, 256), (1, 512), (30, 256), (30, 512), (30, 64)])
def test_attention_bad_pages_are_left_out(cuda_lib, new, D):
    c = Case([new, new], [500, 90], 8, 1, D)
    c.table[0, 3] = c.pages
    c.table[0, 20] = -1
    c.table[1, 1] = 2 ** 31 - 1
    check_attention(cuda_lib, c, err=1)


@pytest.mark.parametrize("new,D", [(1, 256), (1, 64), (30, 256), (30, 512)])
def test_attention_lengths_beyond_the_table(cuda_lib, new, D):
    """A length that max_pages pages do not hold: the positions that they do hold."""
    c = Case([new, new], [300, 50], 8, 1, D)
    c.table[0] = c.table[0].clamp(min=0)
    c.kvl[0] = 16 * c.max_pages + 5
    check_attention(cuda_lib, c, err=1)


@pytest.mark.parametrize("new,D", [(1, 256), (1, 512), (50, 256), (50, 512)])
def test_attention_same_bits_again_streams_and_graphs(cuda_lib, new, D):
    q4w = cuda_lib
    c = Case([new] * 5, [new + x for x in (3000, 10, 555, 0, 1200)], 8, 1, D)
    out, lse = check_attention(q4w, c)
    ws = q4w.kv_attention_ws(new, 8, 1, D, "cuda")
    ws.fill_(0xFF)                                     # its contents do not matter
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out2, lse2 = q4w.kv_attention(c.q, *c.tables(), max_q=new, ws=ws, lse=torch.empty_like(lse))
    torch.cuda.synchronize()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    # captured once, replayed on new queries and lengths
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out3, lse3 = q4w.kv_attention(c.q, *c.tables(), max_q=new, ws=ws, lse=lse2)
    c.q.copy_(normal(c.gen, *c.q.shape))
    c.kvl -= 1
    c.kv = [x - 1 for x in c.kv]
    g.replay()
    torch.cuda.synchronize()
    want, wl = check_attention(q4w, c)
    assert torch.equal(out3, want) and torch.equal(lse3, wl)


def test_attention_workspace_of_any_size(cuda_lib):
    """Products of its arguments that pass 32 bits ask for the tiles' workspace, not for
    the smaller one of a few rows."""
    lib = cuda_lib.load()
    for D in (64, 128, 256, 512):
        tiles = lib.kv_attention_ws_bytes(4096, 8, 1, D)
        assert tiles > lib.kv_attention_ws_bytes(1, 8, 1, D)
        for max_q, n_q in ((2 ** 29, 8), (2 ** 30, 128), (2 ** 31 - 1, 128), (3 * 2 ** 29, 8)):
            assert lib.kv_attention_ws_bytes(max_q, n_q, 1, D) == tiles, (max_q, n_q, D)


def test_attention_longer_than_max_q(cuda_lib):
    """A sequence with more tokens than max_q: its first max_q tokens, and the flag."""
    q4w = cuda_lib
    c = Case([6, 2], [100, 50], 8, 1, 256)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((8, 8, 256), 77.0, dtype=F16, device="cuda")
    q4w.kv_attention(c.q, *c.tables(), max_q=2, out=out, err=err)
    q4w.q4_device_status()
    assert int(err) == 1
    full, _ = q4w.kv_attention(c.q, *c.tables(), max_q=6)
    torch.cuda.synchronize()
    for t in (0, 1, 6, 7):
        assert torch.allclose(out[t].float(), full[t].float(), rtol=0, atol=4e-3)
    assert torch.all(out[2:6] == 77.0)


def test_attention_cache_beyond_32_bits(cuda_lib):
    """Pages whose element offsets pass 2^32."""
    q4w = cuda_lib
    D, page, pages = 512, 128, 70000                 # 4.6e9 elements each
    kc = torch.zeros(pages, 1, page, D, dtype=F16, device="cuda")
    vc = torch.zeros_like(kc)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    ids = [69999, 3, 65536, 40000]
    for i in ids:
        kc[i] = normal(g, 1, page, D)
        vc[i] = normal(g, 1, page, D)
    table = torch.tensor([ids], dtype=torch.int32, device="cuda")
    for new in (1, 20):
        cu = torch.tensor([0, new], dtype=torch.int32, device="cuda")
        kvl = torch.tensor([500], dtype=torch.int32, device="cuda")
        k = normal(g, new, 1, D)
        q4w.kv_append(k, k, kc, vc, table, cu, kvl)
        assert torch.equal(vc[40000, 0, 500 - 384 - new:500 - 384], k[:, 0])
        q = normal(g, new, 8, D)
        out, _ = q4w.kv_attention(q, kc, vc, table, cu, kvl)
        small = torch.arange(4, dtype=torch.int32, device="cuda")[None]
        want, _ = q4w.kv_attention(q, kc[ids].contiguous(), vc[ids].contiguous(), small, cu, kvl)
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("D", [64, 256, 512])
def test_attention_zero_budget_times_out_then_recovers(cuda_lib, D):
    """The tiles' bounded waits: with a zero cycle budget the kernel gives up, returns
    and reports it; the next call is right again."""
    q4w = cuda_lib
    q4w.q4_device_status()
    c = Case([200, 90], [3000, 500], 8, 1, D)
    old = q4w.q4_set_wait_limit(0)
    try:
        q4w.kv_attention(c.q, *c.tables(), max_q=200)
        with pytest.raises(q4w.Q4Error, match="Q4_ERR_TIMEOUT"):
            q4w.q4_device_status()
    finally:
        q4w.q4_set_wait_limit(old)
    check_attention(q4w, c)
