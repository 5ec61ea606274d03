"""Appending with head norms, the int8 cache written, read back and attended over,
against the fp64 oracle.

Tolerances.  A norm: the sum of squares in fp32 has at most 16 additions in a thread
and 5 between threads, 21 2^-24 of itself, half of that in its root; rsqrt is good to
2 ulp (2^-22), two products round once each: below 1.2e-6 of the element.  The rotation
is below 6e-7 of the pair's length.  A code stands for a number that is half a scale off
at most; the scale is that of the largest magnitude, off by what the elements are off.
"""
import numpy as np
import pytest
import torch

from oracle import kv8_oracle as O8

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
OFF = 1.8e-6       # of a pair's length: an element before it is rounded


def normal(gen, *shape, dtype=F16, std=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)


def f64(t):
    return t.double().cpu().numpy()


class Case:
    """Tables, a 16-bit cache and an int8 cache of sequences with n[i] new tokens at the end of kv[i]."""

    def __init__(self, n, kv, hq=8, hkv=1, D=256, page=16, dtype=F16, seed=0, std=1.0, pad=0, plain=False):
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
        if plain:
            self.kc, self.vc = (normal(g, self.pages, hkv, page, D, dtype=dtype, std=std) for _ in "kv")
        else:
            self.kc, self.vc = ((torch.randint(-127, 128, (self.pages, hkv, page, D), generator=g, device="cuda", dtype=torch.int8),
                                 (torch.rand(self.pages, hkv, page, D // 32, generator=g, device="cuda") * 0.02 * std + 1e-3).to(F16)) for _ in "kv")
        self.q = normal(g, self.T, hq, D, dtype=dtype, std=std)

    def tables(self):
        return self.kc, self.vc, self.table, self.cu, self.kvl

    def places(self):
        """(token, sequence, position) on the host."""
        from oracle import kv_oracle as KV
        return list(KV.tokens(self.cu.cpu().numpy(), self.kv))


def appended(q4w, c, inp, rot, inter, norms, eps=1e-6, positions=None, bad=0):
    """Appends random rows by kv_append_norm or kv_append_q8 and checks everything that was written."""
    hq, hkv, D, plain = c.hq, c.hkv, c.D, isinstance(c.kc, torch.Tensor)
    fused = normal(c.gen, c.T, (hq + 2 * hkv) * D + 16, dtype=inp, std=3.0)
    q = fused[:, :hq * D].view(c.T, hq, D) if hq else None
    k, v = fused[:, hq * D:(hq + hkv) * D].view(c.T, hkv, D), fused[:, (hq + hkv) * D:(hq + 2 * hkv) * D].view(c.T, hkv, D)
    w = {x: normal(c.gen, D, dtype=F32, std=0.3) + 1 if x in norms else None for x in "qkv"}
    freqs = 10000.0 ** (-np.arange(rot // 2) * 2.0 / max(rot, 1))
    steps = q4w.kv_rope_steps(rot, device="cuda") if rot else None
    before = [x.clone() for x in ((c.kc, c.vc) if plain else (*c.kc, *c.vc))]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = torch.full((c.T, hq, D), 77.0, dtype=c.dtype, device="cuda") if hq else None
    more = {} if plain else {"dtype": c.dtype}
    call = q4w.kv_append_norm if plain else q4w.kv_append_q8
    call(k, v, *c.tables(), q_norm=w["q"], k_norm=w["k"], v_norm=w["v"], eps=eps, steps=steps, q=q, interleaved=inter, q_out=q_out,
         positions=positions, err=err, **more)
    assert int(err) == bad
    h = {x: None if w[x] is None else f64(w[x]) for x in "qkv"}
    rows, turned = O8.rows(f64(k), f64(v), None if q is None else f64(q), c.table.cpu().numpy(), c.cu.cpu().numpy(), c.kv, c.pages, c.page,
                           freqs, inter, None if positions is None else positions.cpu().numpy(), h["q"], h["k"], h["v"], eps)
    half = torch.finfo(c.dtype).eps / 2

    def close(got, ref):
        length = np.abs(ref).max(-1, keepdims=True) * 1.5
        assert np.all(np.abs(got - ref) <= half * np.abs(ref) * 1.01 + OFF * length + 2.0 ** -25), float(np.abs(got - ref).max())

    if hq:
        got, pad = f64(q_out), np.isnan(turned)
        assert np.all(got[pad] == 77.0), "padding tokens were written"
        close(got[~pad].reshape(-1, D), turned[~pad].reshape(-1, D))
    now = [x.clone() for x in ((c.kc, c.vc) if plain else (*c.kc, *c.vc))]
    for t, page, row, rk, rv in rows:
        if page is None:
            continue
        if plain:
            close(f64(now[0][page, :, row]), rk)
            close(f64(now[1][page, :, row]), rv)
            continue
        for i, ref in ((0, rk), (2, rv)):
            codes, scales = f64(now[i][page, :, row]), f64(now[i + 1][page, :, row])
            off = OFF * 1.5 * np.abs(ref).max(-1, keepdims=True)
            top = np.abs(ref.reshape(hkv, -1, 32)).max(-1)
            assert np.all(np.abs(codes) <= 127)
            assert np.all(scales * 127 * (1 + 1e-6) >= top - off) and np.all(scales * 127 <= (top + off) * (1 + 2.0 ** -10) + 127 * 2.0 ** -24)
            wide = np.repeat(scales, 32, axis=-1)
            assert np.all(np.abs(codes * wide - ref) <= wide / 2 * (1 + 1e-5) + off)
    for x, y in zip(now, before):      # nothing else was touched
        for t, page, row, rk, rv in rows:
            if page is not None:
                x[page, :, row] = y[page, :, row]
        assert torch.equal(x, y)
    return q_out


SHAPES = [
    (256, 8, 1, 256, False, F32, F16, 16, "qkv"),
    (512, 8, 1, 128, False, F16, F16, 16, "qk"),
    (512, 3, 1, 512, True, BF16, BF16, 48, "kv"),
    (128, 6, 2, 64, True, F32, BF16, 32, "q"),
    (64, 1, 1, 64, False, BF16, F16, 128, "k"),
    (64, 10, 5, 16, False, F16, BF16, 16, "v"),
    (64, 2, 2, 48, False, F16, F16, 16, "qkv"),
    (128, 0, 3, 0, False, F16, F16, 16, "kv"),
    (256, 2, 1, 80, True, F32, F16, 16, "qk"),
]


@pytest.mark.parametrize("plain", [True, False])
@pytest.mark.parametrize("D,hq,hkv,rot,inter,inp,dtype,page,norms", SHAPES)
def test_append(cuda_lib, D, hq, hkv, rot, inter, inp, dtype, page, norms, plain):
    c = Case([1, 5, 0, 17, 1, 40], [1, 30, 9, 17, 200, 65], hq, hkv, D, page, dtype, pad=2, plain=plain)
    appended(cuda_lib, c, inp, rot, inter, norms)


@pytest.mark.parametrize("plain", [True, False])
def test_append_without_norms_is_kv_append(cuda_lib, plain):
    """No weights: the 16-bit cache and the queries get the very bits of kv_append."""
    q4w = cuda_lib
    c = Case([3, 40], [10, 50], 4, 2, 128, plain=plain)
    d = Case([3, 40], [10, 50], 4, 2, 128, plain=True)
    k, v, q = (normal(c.gen, c.T, h, 128, dtype=F32) for h in (2, 2, 4))
    steps = q4w.kv_rope_steps(128, device="cuda")
    want = q4w.kv_append(k, v, *d.tables(), steps=steps, q=q)
    if plain:
        d2 = Case([3, 40], [10, 50], 4, 2, 128, plain=True)
        got = q4w.kv_append_norm(k, v, *d2.tables(), steps=steps, q=q)
        assert torch.equal(d.kc, d2.kc) and torch.equal(d.vc, d2.vc)
    else:
        got = q4w.kv_append_q8(k, v, *c.tables(), steps=steps, q=q)
    assert torch.equal(got, want)


@pytest.mark.parametrize("plain", [True, False])
@pytest.mark.parametrize("seqs,new", [(70, 1), (300, 3), (1, 700)])
def test_append_numbers_of_tokens(cuda_lib, seqs, new, plain):
    """One row a thread, and all rows of a token a thread; many sequences in a block."""
    appended(cuda_lib, Case([new] * seqs, [new + i % 37 for i in range(seqs)], 4, 2, 64, plain=plain, seed=seqs), F16, 64, False, "qk")


def test_append_explicit_positions_and_eps(cuda_lib):
    c = Case([2, 9], [2, 30], 4, 1, 128, plain=False)
    appended(cuda_lib, c, F32, 128, False, "qkv", eps=0.5, positions=torch.arange(c.T, dtype=torch.int32, device="cuda") * 1000 + 7)


def test_append_bad_places_store_nothing(cuda_lib):
    for plain in (True, False):
        c = Case([2, 3, 1], [2, 40, 20], 2, 1, 128, plain=plain)
        c.table[1, 2] = c.pages        # past the cache
        c.table[2, 1] = -1
        appended(cuda_lib, c, F16, 128, False, "k", bad=1)


def test_append_rows_of_zeros_and_of_small_and_large_numbers(cuda_lib):
    """Zeros keep scale 0; subnormal scales still cover their block; the largest that fit do."""
    q4w = cuda_lib
    c = Case([6], [6], 1, 1, 64)
    k = torch.zeros(6, 1, 64, device="cuda")
    k[1] = normal(c.gen, 1, 64, dtype=F32, std=1e-5)
    k[2] = normal(c.gen, 1, 64, dtype=F32, std=1e-7)
    k[3] = normal(c.gen, 1, 64, dtype=F32, std=2e4)
    k[3].clamp_(-65000, 65000)
    k[4, 0, 5], k[4, 0, 40] = 515.5 * 127, 1e-30
    k[5] = 1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q4w.kv_append_q8(k, k, *c.tables(), err=err)
    assert int(err) == 0
    for t in range(6):
        page, row = int(c.table[0, 0]), t
        codes, scales = f64(c.kc[0][page, 0, row]), f64(c.kc[1][page, 0, row])
        ref, rs, _ = O8.quantise(f64(k[t, 0]))
        assert np.array_equal(scales, rs)
        assert np.all(np.abs(codes * np.repeat(scales, 32) - f64(k[t, 0])) <= np.repeat(scales, 32) / 2 * (1 + 1e-5))
        assert np.abs(codes - ref).max() <= 1
        assert torch.equal(c.vc[0][page, 0, row], c.kc[0][page, 0, row])


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan"), 65500.0])
def test_append_blocks_that_cannot_be_held(cuda_lib, value):
    q4w = cuda_lib
    c = Case([2], [2], 1, 1, 128)
    k = normal(c.gen, 2, 1, 128, dtype=F32)
    v = k.clone()
    k[1, 0, 70] = value
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q4w.kv_append_q8(k, v, *c.tables(), err=err)
    assert int(err) == 1
    page = int(c.table[0, 0])
    codes, scales = c.kc[0][page, 0, 1], f64(c.kc[1][page, 0, 1])
    assert scales[2] == 0 and not codes[64:96].any()
    assert np.all(scales[[0, 1, 3]] > 0)
    assert np.all(f64(c.vc[1][page, 0, :2]) > 0)


# -------------------------------------------------------------------- read ---
@pytest.mark.parametrize("D,hkv,page,dtype", [(64, 3, 16, F16), (128, 2, 48, BF16), (256, 1, 32, F16), (512, 1, 128, BF16)])
def test_read(cuda_lib, D, hkv, page, dtype):
    """Parts of sequences and whole ones, an empty one, padding tokens left alone."""
    q4w = cuda_lib
    c = Case([1, 30, 0, 17, 150], [5, 30, 9, 40, 200], 1, hkv, D, page, dtype, pad=3)
    k, v = (torch.full((c.T, hkv, D), 77.0, dtype=dtype, device="cuda") for _ in "kv")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q4w.kv_read_q8(*c.tables(), c.T, dtype=dtype, k_out=k, v_out=v, err=err)
    assert int(err) == 0
    kn, vn = (torch.from_numpy(O8.values(x[0].cpu().numpy(), f64(x[1]))) for x in (c.kc, c.vc))
    t = c.table.cpu().numpy()
    for tok, s, pos in c.places():
        for got, ref in ((k, kn), (v, vn)):     # exact products in fp64: one rounding
            assert torch.equal(got[tok].cpu(), ref[t[s, pos // page], :, pos % page].to(dtype))
    assert bool((k[-3:] == 77).all()) and bool((v[-3:] == 77).all())


@pytest.mark.parametrize("D,hkv", [(64, 1), (128, 3), (512, 2)])
def test_read_more_sequences_than_a_warp_has_lanes(cuda_lib, D, hkv):
    """Short and empty ones, so that a warp's tokens are of several, far into the table."""
    n = [i % 3 for i in range(90)] + [0] * 40 + [5, 0, 1]
    c = Case(n, [x + i % 20 for i, x in enumerate(n)], 1, hkv, D, 16, BF16)
    k, v = cuda_lib.kv_read_q8(*c.tables(), c.T, dtype=BF16)
    kn, vn = (torch.from_numpy(O8.values(x[0].cpu().numpy(), f64(x[1]))) for x in (c.kc, c.vc))
    t = c.table.cpu().numpy()
    for tok, s, pos in c.places():
        for got, ref in ((k, kn), (v, vn)):
            assert torch.equal(got[tok].cpu(), ref[t[s, pos // 16], :, pos % 16].to(BF16))


def test_read_bad_places_are_zeros(cuda_lib):
    q4w = cuda_lib
    c = Case([20, 40], [20, 30], 1, 1, 64)      # the second has more tokens than positions
    c.table[0, 1] = c.pages
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    k, v = q4w.kv_read_q8(*c.tables(), c.T, err=err)
    assert int(err) == 1
    assert not k[16:20].any() and not v[16:20].any() and not k[20:30].any() and k[:16].any() and k[30:].any()


def test_written_rows_read_back(cuda_lib):
    """Appended, then read for the same tokens on a stream of its own."""
    q4w = cuda_lib
    c = Case([3, 64, 1], [10, 64, 500], 4, 2, 256, 32, BF16)
    k, v = (normal(c.gen, c.T, 2, 256, dtype=F32) for _ in "kv")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q4w.kv_append_q8(k, v, *c.tables(), dtype=BF16)
        gk, gv = q4w.kv_read_q8(*c.tables(), c.T, dtype=BF16)
    torch.cuda.synchronize()
    for got, x in ((gk, k), (gv, v)):
        top = x.reshape(c.T, 2, -1, 32).abs().amax(-1, keepdim=True)
        d = (got.float() - x).reshape(c.T, 2, -1, 32).abs()
        # half a scale, and the rounding to bf16
        assert bool((d <= top / 254 * (1 + 2.0 ** -10) * 1.00001 + top * 2.0 ** -8 * 1.01).all())


def test_read_offsets_beyond_32_bits(cuda_lib):
    """A cache of 5 GB of codes: pages beyond 2^32 bytes."""
    q4w = cuda_lib
    D, page, hkv = 512, 1024, 8
    pages = 1100
    kc = (torch.empty(pages, hkv, page, D, dtype=torch.int8, device="cuda"), torch.empty(pages, hkv, page, D // 32, dtype=F16, device="cuda"))
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device="cuda")
    cu, kvl = torch.tensor([0, 700], dtype=torch.int32, device="cuda"), torch.tensor([1000], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    k, v = (normal(g, 700, hkv, D, dtype=F32) for _ in "kv")
    vc = (torch.empty_like(kc[0]), torch.empty_like(kc[1]))
    q4w.kv_append_q8(k, v, kc, vc, table, cu, kvl)
    gk, gv = q4w.kv_read_q8(kc, vc, table, cu, kvl, 700)
    for got, x in ((gk, k), (gv, v)):
        top = x.reshape(700, hkv, -1, 32).abs().amax(-1, keepdim=True)
        assert bool(((got.float() - x).reshape(700, hkv, -1, 32).abs() <= top * (1 / 254 * 1.001 + 2.0 ** -11 * 1.01)).all())


# --------------------------------------------------------------- attention ---
# With A = sum p|v| and S the largest scale sum |q k|.  A score: products of 16-bit queries and
# codes are exact in fp32; a block's 32 are summed by two instructions (2^-23 each), then at most
# 16 blocks are added (2^-24 each) and two factors round: below 22 2^-24 S.  P and V are rounded
# to fp16 (2^-11 A each; P with an absolute error of 2^-25 of what lies 2^-7 under the largest, V
# of 2^-25 where it is subnormal), exponentials and sums add 2e-6 A, the output half a step.
def check_attention(q4w, c, scale=None, window=0, max_q=None, q=None, err=0, **kw):
    from oracle import kv_oracle as O
    scale = c.D ** -0.5 if scale is None else scale
    q = c.q if q is None else q
    lse = torch.full((c.T, c.hq), 77.0, device="cuda")
    out = torch.full((c.T, c.hq, c.D), 77.0, dtype=c.dtype, device="cuda")
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    q4w.kv_attention_q8(q, *c.tables(), max_q=max(c.n) if max_q is None else max_q, scale=scale, window=window, out=out, lse=lse, err=flag, **kw)
    q4w.q4_device_status()
    kn, vn = (O8.values(x[0].cpu().numpy(), f64(x[1])) for x in (c.kc, c.vc))
    ro, rl, A, S = O.attention(f64(q), kn, vn, c.table.cpu().numpy(), c.cu.cpu().numpy(), c.kvl.cpu().numpy(), scale, window)
    go, gl = f64(out), f64(lse)
    pad = np.isnan(rl)
    assert np.all(gl[pad] == 77.0) and np.all(go[pad] == 77.0), "padding tokens were written"
    go, gl, ro, rl, A, S = go[~pad], gl[~pad], ro[~pad], rl[~pad], A[~pad], S[~pad]
    assert int(flag) == err
    empty = rl == -np.inf
    assert np.array_equal(gl == -np.inf, empty)
    assert np.all(go[empty] == 0)
    ds = 22 * 2.0 ** -24 * S
    n = max(c.kv + [1])
    small = n * 2.0 ** -32 * max(A.max() if A.size else 0, 1) / max(1.0, np.sqrt(n)) * 4 + 2.0 ** -25
    tol = 2 * 2.0 ** -11 * A * 1.01 + torch.finfo(c.dtype).eps / 2 * np.abs(ro) * 1.01 + (2 * ds[..., None] + 2e-6) * A + small
    bad = ~(np.abs(go - ro) <= tol)
    assert not bad.any(), (int(bad.sum()), float((np.abs(go - ro) / tol).max()))
    assert np.all(np.abs(gl[~empty] - rl[~empty]) <= (ds + 2e-6 * (1 + np.abs(rl)))[~empty])
    return out, lse


def stale(c, value=float("nan")):
    """Scales of rows that hold no position."""
    keep = torch.zeros(c.pages, c.page, dtype=torch.bool)
    t = c.table.cpu().numpy()
    for i, x in enumerate(c.kv):
        for p in range(x):
            keep[t[i, p // c.page], p % c.page] = True
    drop = (~keep).cuda()[:, None, :, None].expand_as(c.kc[1])
    for x in (c.kc[1], c.vc[1]):
        x[drop] = value
    return c


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hq,hkv", [(8, 1), (4, 4), (6, 2), (5, 1), (16, 1), (1, 1)])
def test_attention_single_tokens(cuda_lib, D, dtype, hq, hkv):
    check_attention(cuda_lib, stale(Case([1] * 6, [1, 2, 15, 16, 17, 333], hq, hkv, D, 16, dtype, seed=D + hq)))


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hq,hkv,page", [(8, 1, 16), (4, 2, 64), (7, 1, 48), (3, 3, 128)])
def test_attention_chunks(cuda_lib, D, dtype, hq, hkv, page):
    """Ragged chunks: no new token, one, the whole sequence, tiles that end inside pages."""
    check_attention(cuda_lib, stale(Case([1, 64, 0, 33, 130, 5], [1, 64, 40, 200, 259, 128], hq, hkv, D, page, dtype, seed=D + hq, pad=3)))


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("rows", [1, 7, 8, 9, 15, 16, 17, 31, 32, 33, 127, 128, 129, 255, 256, 257])
def test_attention_rows_next_to_the_kernels_limits(cuda_lib, D, rows):
    """Rows per KV head around the sizes at which another kernel or tile begins, as tokens of
    one head and as heads of few tokens."""
    for hq, new in [(1, rows)] + [(h, rows // h) for h in (rows, rows // 2, 3) if h and h <= 128 and rows % h == 0 and h > 1]:
        check_attention(cuda_lib, Case([new, 1, new], [new, 70, 190 + new], hq, 1, D, 16, F16, seed=rows + hq))


@pytest.mark.parametrize("D,hq,hkv", [(64, 8, 2), (256, 8, 1), (512, 8, 1), (128, 4, 4)])
@pytest.mark.parametrize("new", [1, 2, 4, 9, 70])
@pytest.mark.parametrize("window", [1, 17, 100, 512])
def test_attention_window(cuda_lib, D, hq, hkv, new, window):
    kv = [new, new + 16, new + 150, new + 777]
    c = stale(Case([new] * 4, kv, hq, hkv, D, 16, F16, seed=window), float("inf"))
    for i, x in enumerate(kv):      # pages that slid out of every token's reach are freed
        c.table[i, :max(0, x - new + 1 - window) // 16] = -1
    check_attention(cuda_lib, c, window=window)


@pytest.mark.parametrize("D,hq", [(256, 8), (512, 8), (64, 2), (128, 1)])
@pytest.mark.parametrize("new", [1, 40])
def test_attention_long_and_split(cuda_lib, D, hq, new):
    """Lengths that are split over many CTAs next to short ones."""
    check_attention(cuda_lib, Case([new, new, 1], [5003, new, 2001], hq, 1, D, 32, BF16, seed=new, std=1.4))


@pytest.mark.parametrize("D,n,kv", [(256, [400, 3], [2000, 900]), (512, [100], [4000]), (512, [200, 3], [700, 900]),
                                    (128, [900], [2500]), (64, [1000, 70], [1500, 3000])])
def test_attention_several_steps_and_items_per_cta(cuda_lib, D, n, kv):
    check_attention(cuda_lib, Case(n, kv, 8, 1, D, 64, F16, seed=D))


@pytest.mark.parametrize("D,hq,hkv,seqs,new", [(512, 16, 2, 100, 9), (512, 8, 8, 20, 90), (512, 8, 1, 200, 1), (256, 32, 2, 200, 9), (128, 40, 2, 200, 9),
                                               (64, 80, 2, 200, 9), (256, 16, 1, 300, 1)])
@pytest.mark.parametrize("window", [0, 100])
def test_attention_many_short_items_one_after_the_other(cuda_lib, D, hq, hkv, seqs, new, window):
    """Items of a few steps, most of which end inside a step, whose keys come late: right, and
    the same bits every time."""
    g = np.random.default_rng(D + seqs)
    n = [int(x) for x in g.integers(1, new + 1, seqs)]
    kv = [x + int(g.choice([g.integers(0, 40), g.integers(100, 600), g.integers(0, 1500)])) for x in n]
    c = stale(Case(n, kv, hq, hkv, D, 16, BF16, seed=seqs), float("inf"))
    out, lse = check_attention(cuda_lib, c, window=window)
    again, flush = torch.empty_like(out), torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for i in range(30):
        if i % 2:
            flush.fill_(i)
        cuda_lib.kv_attention_q8(c.q, *c.tables(), max_q=max(n), window=window, out=again)
        assert torch.equal(out, again), i


@pytest.mark.parametrize("D,hq,hkv,new", [(256, 8, 1, 1), (512, 8, 1, 1), (64, 3, 1, 1), (256, 8, 1, 64), (512, 4, 1, 50), (128, 4, 2, 90)])
def test_attention_rows_that_see_nothing(cuda_lib, D, hq, hkv, new):
    """A length of zero, and lengths shorter than the new tokens."""
    c = stale(Case([new, new, new], [0, min(new, 3), 200], hq, hkv, D))
    check_attention(cuda_lib, c)
    c.kvl.zero_()
    c.kv = [0, 0, 0]
    check_attention(cuda_lib, stale(c))


@pytest.mark.parametrize("D", [64, 256, 512])
@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_attention_scores_of_any_size(cuda_lib, D, new, dtype):
    """Large and tiny scores, of either sign, a scale of zero, queries of zeros."""
    c = Case([new, new], [300, 700], 4, 1, D, dtype=dtype, std=3.0)
    for scale in (1.0, -0.5, 0.0, 1e-6, 30.0):
        check_attention(cuda_lib, c, scale=scale)
    c.q[0].zero_()
    c.q[-1, 1] *= 1e-3
    if dtype is BF16:       # a range that fp16 does not have
        c.q[0, 0], c.q[0, 1] = c.q[-1, 0] * 1e30, c.q[-1, 0] * 1e-30
        check_attention(cuda_lib, c, scale=1e-30)
    check_attention(cuda_lib, c)


@pytest.mark.parametrize("new", [1, 30])
def test_attention_small_and_large_values(cuda_lib, new):
    """Scales of V that fp16 holds as subnormal numbers, and up to its largest values."""
    c = Case([new, new], [100, 200], 4, 1, 128)
    half = c.pages // 2
    c.vc[1][:half] = 2.0 ** -20
    c.vc[1][half:] = 500.0
    check_attention(cuda_lib, c)


@pytest.mark.parametrize("D,new,depth", [(256, 1, 22), (128, 40, 24), (64, 3, 20)])
def test_attention_many_keys_of_small_probability(cuda_lib, D, new, depth):
    """Thousands of keys of 2^-depth of the largest: their sum counts."""
    c = Case([new], [6000 + new], 2, 1, D)
    for x in (c.kc, c.vc):
        x[0].zero_()
        x[1].fill_(1.0)
    c.q.zero_()
    c.q[..., 0] = 1.0
    first = int(c.table[0, 0])
    c.kc[0][first, 0, 0, 0] = depth                  # one key, scale ln 2: all others lie 2^-depth below it
    c.vc[0][..., 1] = 100
    c.vc[0][first, 0, 0, 1] = 0
    check_attention(cuda_lib, c, scale=float(np.log(2.0)))


@pytest.mark.parametrize("new,hq", [(1, 8), (50, 8)])
def test_attention_strided_queries_and_order(cuda_lib, new, hq):
    """Rows of a fused projection as queries; the sequences in another order give the same bits."""
    c = Case([new, new], [100, 400], hq, 2, 128)
    fused = normal(c.gen, c.T, (hq + 4) * 128)
    q = fused[:, 256:256 + hq * 128].view(c.T, hq, 128)
    check_attention(cuda_lib, c, q=q)


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("D", [64, 256, 512])
def test_attention_bad_pages_are_left_out(cuda_lib, new, D):
    c = Case([new, new], [200, 200], 4, 1, D)
    c.table[0, 3], c.table[1, 0], c.table[1, 5] = -1, c.pages, 2 ** 31 - 1
    check_attention(cuda_lib, c, err=1)


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("D", [128, 512])
def test_attention_lengths_beyond_the_table(cuda_lib, new, D):
    c = Case([new, new], [200, 200], 4, 1, D)
    c.kvl[1] += 64
    c.kv[1] += 64
    check_attention(cuda_lib, c, err=1)


@pytest.mark.parametrize("new,D", [(1, 256), (5, 512), (64, 256), (64, 512)])
def test_attention_same_bits_again_streams_and_graphs(cuda_lib, new, D):
    """Two streams at once with workspaces of their own, and a graph whose lengths change."""
    q4w = cuda_lib
    c = Case([new] * 3, [new + 50, new + 900, new + 3000], 8, 1, D, dtype=BF16)
    out, _ = check_attention(q4w, c)
    outs = [torch.empty_like(out) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    wss = [q4w.kv_attention_q8_ws(c.T, new, 8, 1, D, "cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(10):
        for st, o, ws in zip(streams, outs, wss):
            with torch.cuda.stream(st):
                q4w.kv_attention_q8(c.q, *c.tables(), max_q=new, out=o, ws=ws)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], out) and torch.equal(outs[1], out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q4w.kv_attention_q8(c.q, *c.tables(), max_q=new, out=outs[0], ws=wss[0])
    c.kvl -= 40
    c.kv = [x - 40 for x in c.kv]
    want, _ = check_attention(q4w, c)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want)


def test_attention_longer_than_max_q(cuda_lib):
    """The first max_q tokens are computed, the others' rows left, err set."""
    q4w = cuda_lib
    c = Case([4, 9], [50, 90], 4, 1, 128)
    out = torch.full((c.T, 4, 128), 77.0, dtype=F16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q4w.kv_attention_q8(c.q, *c.tables(), max_q=4, out=out, err=err)
    assert int(err) == 1 and bool((out[8:] == 77).all()) and bool((out[:8] != 77).any())


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("new", [1, 60])
def test_attention_fp16_error_in_the_mean(cuda_lib, D, new):
    """By both kernels, the error's root mean square against that of rounding the exact result to fp16
    (2^-11 at the most, of whatever its mantissa): V's rounding adds one like it, P in two pieces 2^-22 of
    itself, so sqrt(2) of it; 2 % for chance."""
    from oracle import kv_oracle as O
    c = Case([new] * 4, [500 + new, 130 + new, 1200 + new, 40 + new], 8, 1, D, 16, F16)
    out, _ = cuda_lib.kv_attention_q8(c.q, *c.tables(), max_q=new)
    kn, vn = (O8.values(x[0].cpu().numpy(), f64(x[1])) for x in (c.kc, c.vc))
    ro, _, _, _ = O.attention(f64(c.q), kn, vn, c.table.cpu().numpy(), c.cu.cpu().numpy(), c.kvl.cpu().numpy(), D ** -0.5, 0)
    off = np.sqrt(np.mean((f64(out) - ro) ** 2))
    alone = np.sqrt(np.mean((ro.astype(np.float16).astype(np.float64) - ro) ** 2))
    assert off <= 1.02 * 2 ** 0.5 * alone, off / alone


def test_attention_cache_beyond_32_bits(cuda_lib):
    """Pages beyond 2^32 bytes of codes, by both kernels."""
    q4w = cuda_lib
    D, page, hkv, pages = 512, 1024, 8, 1100
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    c = Case([1], [40], 8, hkv, D, 1024)
    kc, vc = (tuple(torch.zeros(pages, hkv, page, n, dtype=dt, device="cuda") for n, dt in ((D, torch.int8), (D // 32, F16))) for _ in "kv")
    for big, small in ((kc, c.kc), (vc, c.vc)):
        for b, x in zip(big, small):
            b[pages - 1] = x[int(c.table[0, 0])]
    far = c.table.clone()
    far[0, 0] = pages - 1
    for new in (1, 40):
        q = normal(c.gen, new, 8, D)
        cu = torch.tensor([0, new], dtype=torch.int32, device="cuda")
        near, _ = q4w.kv_attention_q8(q, c.kc, c.vc, c.table, cu, c.kvl)
        got, _ = q4w.kv_attention_q8(q, kc, vc, far, cu, c.kvl)
        assert torch.equal(got, near)


@pytest.mark.parametrize("D", [128, 512])
def test_attention_zero_budget_times_out_then_recovers(cuda_lib, D):
    """A wait of the tile kernel that runs out is reported, and the next call is right."""
    q4w = cuda_lib
    c = Case([40, 70], [400, 900], 8, 1, D)
    want, _ = check_attention(q4w, c)
    old = q4w.q4_set_wait_limit(0)
    try:
        q4w.kv_attention_q8(c.q, *c.tables(), max_q=70)
        with pytest.raises(q4w.Q4Error, match="imeout|timed|wait"):
            q4w.q4_device_status()
    finally:
        q4w.q4_set_wait_limit(old)
    again, _ = check_attention(q4w, c)
    assert torch.equal(want, again)


def test_a_step_with_norms_an_int8_cache_and_drafted_tokens(cuda_lib):
    """kv_append_q8 and kv_attention_q8 as a step calls them, over three steps, against attention
    in fp64 over the rows that kv_read_q8 gives back."""
    q4w = cuda_lib
    c = Case([4, 4], [4, 4], 8, 2, 128)
    table = torch.arange(32, dtype=torch.int32, device="cuda").view(2, 16)
    kc, vc = (tuple(torch.zeros(32, 2, 16, n, dtype=dt, device="cuda") for n, dt in ((128, torch.int8), (4, F16))) for _ in "kv")
    w = normal(c.gen, 128, dtype=F32, std=0.2) + 1
    steps = q4w.kv_rope_steps(128, device="cuda")
    c.kc, c.vc, c.table, c.pages = kc, vc, table, 32
    for step in range(3):
        c.kvl.fill_(4 * step + 4 + 30 * (step == 2))     # then a longer prefix: rows never appended stand for zeros
        c.kv = [int(x) for x in c.kvl]
        k, v, q = (normal(c.gen, 8, h, 128, dtype=F32) for h in (2, 2, 8))
        c.q = q4w.kv_append_q8(k, v, *c.tables(), q_norm=w, k_norm=w, steps=steps, q=q)
        check_attention(q4w, c)


def rows_of_any_size(D, inp, heads=2):
    """Normal rows times 10^-42 (subnormal numbers) to 10^37, and rows that span forty decades."""
    g = np.random.default_rng(D)
    scales = [1e-42, 1e-38, 1e-30, 1e-23, 1e-19, 1e-15, 1.0, 1e15, 1e19, 1e25, 1e37]
    x = np.stack([g.standard_normal((heads, D)) * s for s in scales] + [g.standard_normal((heads, D)) * 10.0 ** g.uniform(a, b, (heads, D)) for a, b in ((-40, 0), (-20, 20), (0, 37))])
    return torch.from_numpy(x.astype(np.float32)).to(inp).cuda()


@pytest.mark.parametrize("plain", [True, False])
@pytest.mark.parametrize("D", [64, 128, 512])
@pytest.mark.parametrize("inp", [F32, BF16])
@pytest.mark.parametrize("eps", [0.0, 1e-44, 1e-30, 1e-6, 1e36])
def test_append_norms_of_rows_of_any_size(cuda_lib, plain, D, inp, eps):
    """Squares that fp32 does not hold, above and below, next to rows whose squares it does: every element
    to the 1.2e-6 of a norm and its rounding (bf16: half a step, 2^-134 where it is subnormal).  (10^-42 is
    zero in bf16, whose least number is 2^-133: with eps = 0 that row is 0 / 0.)"""
    q4w = cuda_lib
    eps = float(np.float32(eps))
    x = rows_of_any_size(D, inp)
    T, half = x.shape[0], torch.finfo(BF16).eps / 2
    c = Case([T], [T], 2, 2, D, 16, BF16, plain=plain)
    w = normal(c.gen, D, dtype=F32, std=0.3) + 1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    call, more = (q4w.kv_append_norm, {}) if plain else (q4w.kv_append_q8, {"dtype": BF16})
    q = call(x, x, *c.tables(), q_norm=w, k_norm=w, v_norm=w, eps=eps, q=x, err=err, **more)
    with np.errstate(invalid="ignore"):
        ref = O8.norm(f64(x), f64(w), eps)
    empty = np.isnan(ref)
    assert empty.any() == (eps == 0 and inp is BF16) and int(err) == int(not plain and empty.any())
    tol = (half * 1.01 + 1.2e-6) * np.abs(ref) + 2.0 ** -134

    def near(got, t):
        return np.array_equal(np.isnan(got), empty[t]) and np.all((np.abs(got - ref[t]) <= tol[t]) | empty[t])

    assert near(f64(q), slice(None))
    table = c.table.cpu().numpy()[0]
    for t in range(T):
        for cache in (c.kc, c.vc):
            page, row = int(table[t // 16]), t % 16
            if plain:
                assert near(f64(cache[page, :, row]), t), t
                continue
            codes, scales = f64(cache[0][page, :, row]), f64(cache[1][page, :, row])
            if empty[t].any():
                assert not codes.any() and not scales.any()
                continue
            # (what is quantised is an fp32 number: below 2^-126 it is a multiple of 2^-149)
            wide, off = np.repeat(scales, 32, axis=-1), 1.2e-6 * np.abs(ref[t]) + 2.0 ** -149
            top = np.abs(ref[t].reshape(2, -1, 32)).max(-1)
            assert np.all(np.abs(codes * wide - ref[t]) <= wide / 2 * (1 + 1e-5) + off), t
            assert np.all(scales * 127 <= top * (1 + 1.2e-6) * (1 + 2.0 ** -10) + 127 * 2.0 ** -24), t


@pytest.mark.parametrize("inp", [F32, F16, BF16])
@pytest.mark.parametrize("plain", [True, False])
def test_append_norms_of_rows_of_zeros(cuda_lib, inp, plain):
    """Zeros with any eps above 0; 0 / 0, which is NaN, without: the int8 cache stores zeros and sets err."""
    q4w = cuda_lib
    for eps in (0.0, 1e-44, 1e-6, 3e38):
        c = Case([3], [3], 1, 1, 64, 16, BF16, plain=plain)
        x = torch.zeros(3, 1, 64, dtype=inp, device="cuda")
        x[1] = 1
        w = torch.ones(64, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        call, more = (q4w.kv_append_norm, {}) if plain else (q4w.kv_append_q8, {"dtype": BF16})
        q = call(x, x, *c.tables(), q_norm=w, k_norm=w, v_norm=w, eps=eps, q=x, err=err, **more)
        zeros = q[[0, 2]]
        assert bool(zeros.isnan().all()) if eps == 0.0 else not zeros.any()
        page = int(c.table[0, 0])
        for cache in (c.kc, c.vc):
            if plain:
                got = cache[page, 0, [0, 2]]
                assert bool(got.isnan().all()) if eps == 0.0 else not got.any()
            else:
                assert not cache[0][page, 0, [0, 2]].any() and not cache[1][page, 0, [0, 2]].any()
        assert int(err) == (0 if plain or eps > 0 else 1)
        assert float(q[1, 0, 0]) == (1.0 if eps < 1 else float(torch.tensor(3e38 ** -0.5).to(BF16)))


@pytest.mark.parametrize("D", [64, 256, 512])
def test_attention_workspace_of_fp16_queries(cuda_lib, D):
    """Queries that are read as they are need no room for themselves: a workspace that does not go by T is
    enough, and nothing is written behind it; bf16 ones are refused with it."""
    q4w = cuda_lib
    lib = q4w.load()
    big = lib.kv_attention_q8_ws_bytes(16384, 2048, 32, 4, D)
    small = lib.kv_attention_q8_ws_bytes(0, 2048, 32, 4, D)
    assert big - small >= 16384 * 32 * D * 2
    assert lib.kv_attention_q8_ws_bytes(0, 1, 8, 1, D) == lib.kv_attention_q8_ws_bytes(16384, 1, 8, 1, D) > 0
    assert q4w.kv_attention_q8_ws(16384, 2048, 32, 4, D, "cuda", dtype=F16).numel() == small
    assert q4w.kv_attention_q8_ws(16384, 2048, 32, 4, D, "cuda").numel() == big
    need = lib.kv_attention_q8_ws_bytes(0, 70, 8, 1, D)
    held = torch.full((need + 4096,), 201, dtype=torch.uint8, device="cuda")
    check_attention(q4w, Case([70, 40], [400, 900], 8, 1, D), ws=held[:need])
    assert bool((held[need:] == 201).all())
    c = Case([70, 40], [400, 900], 8, 1, D, dtype=BF16)
    with pytest.raises(q4w.Q4Error, match="ws must hold"):
        q4w.kv_attention_q8(c.q, *c.tables(), max_q=70, ws=held[:need])
    check_attention(q4w, c, ws=q4w.kv_attention_q8_ws(c.T, 70, 8, 1, D, "cuda", dtype=BF16))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows", [17, 20, 24, 25, 31, 32, 33])
def test_attention_bf16_rows_next_to_the_kernels_limits(cuda_lib, D, rows):
    """17 to 32 rows per KV head of bf16 queries, which are scaled and take one piece of P: as tokens of one
    head and as heads of few tokens, with rows of magnitudes that fp16 does not hold."""
    for hq, new in [(1, rows)] + [(h, rows // h) for h in (rows, rows // 2, 4) if h > 1 and rows % h == 0]:
        c = stale(Case([new, 1, new], [new, 70, 190 + new], hq, 1, D, 16, BF16, seed=rows + hq), float("inf"))
        check_attention(cuda_lib, c)
        check_attention(cuda_lib, c, window=60)
        c.q[-1] *= 1e30
        c.q[0] *= 1e-30
        check_attention(cuda_lib, c, scale=1e-30)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("seqs", [1, 120])
def test_attention_huge_scores_a_step_apart(cuda_lib, dtype, sign, seqs):
    """Two keys in different steps of the tile kernel whose scores are neighbouring numbers of fp32, 2^15 or more
    apart after the scale.  In one CTA (most items of 120 sequences) their difference is exact and the larger takes
    everything.  Parts of several CTAs (one sequence) are joined by references that are fp32 numbers: the scaled
    scores are one such number, here by construction, so the two may share the row.  Never anything else."""
    c = Case([40] * seqs, [400] * seqs, 8, 1, 64, 16, dtype)
    big, one = (2.0 ** 15, 2.0 ** -5) if dtype is F16 else (2.0 ** 20, 1.0)
    scale = 2.0 ** 20
    # scores big * 12 + one * i: i steps of fp32 above 1.5 2^k
    sc = np.float32(np.float32(scale) * np.float32(1.4426950408889634))
    score = [np.float32(12 * big + one * i) for i in range(100)]
    same = [i for i in range(1, 99) if score[i] < score[i + 1] and score[i] * sc == score[i + 1] * sc]
    assert same
    for x in (c.kc, c.vc):
        x[0].zero_()
        x[1].fill_(1.0)
    c.q.zero_()
    c.q[..., 0], c.q[..., 1] = big, one
    table = c.table.long()
    for i in same[:3]:
        for pos, step, value in ((3, i, 50), (200, i + 1, 100)):
            pages = table[:, pos // 16]
            c.kc[0][pages, 0, pos % 16, 0], c.kc[0][pages, 0, pos % 16, 1], c.vc[0][pages, 0, pos % 16] = sign * 12, sign * step, value
        out, _ = cuda_lib.kv_attention_q8(c.q, *c.tables(), max_q=40, scale=sign * scale)
        assert bool(((out >= 50) & (out <= 100)).all())
        assert seqs == 1 or float((out == 100).float().mean()) > 0.5
