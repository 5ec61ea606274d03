"""logits_sample against the fp64 oracle: tokens exactly, log probabilities to
the rounding of an fp32 (eps/2 of the value) and the weights' 2^-28."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import kv_oracle as O

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def check(q4w, z, u, t=None, k=None, p=None, m=None):
    """z [b, V] on the GPU; scalars stand for every row."""
    b = z.shape[0]
    dev = lambda x, dt: None if x is None else (x if torch.is_tensor(x) else torch.full((b,), x, dtype=dt, device="cuda"))   # noqa: E731
    t, k, p, m = dev(t, F32), dev(k, torch.int32), dev(p, F32), dev(m, F32)
    tok, lp = q4w.logits_sample(z, u, t, k, p, m)
    torch.cuda.synchronize()
    zh = z.float().cpu().numpy()
    at = lambda x, i: None if x is None else x[i].item()   # noqa: E731
    for i in range(b):
        rt, rl, _ = O.sample(zh[i], u[i].item(), at(t, i), at(k, i), at(p, i), at(m, i))
        assert int(tok[i]) == rt, (i, int(tok[i]), rt)
        if rl == -np.inf:
            assert float(lp[i]) == -np.inf
        else:
            assert abs(float(lp[i]) - rl) <= 2.0 ** -24 * abs(rl) + 2.0 ** -26, (i, float(lp[i]), rl)
    return tok, lp


def rows(b, V, seed=0, dtype=F32, std=2.5):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(b, V, generator=g, device="cuda") * std).to(dtype), torch.rand(b, generator=g, device="cuda")


@pytest.mark.parametrize("V", [1, 2, 31, 128, 129, 1000, 5003, 20001])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("kw", [dict(), dict(k=40), dict(p=0.9), dict(m=0.05), dict(k=50, p=0.95, t=0.7), dict(k=3000, p=0.9, m=0.001, t=1.5)])
def test_filters(cuda_lib, V, dtype, kw):
    z, u = rows(5, V, seed=V, dtype=dtype)
    check(cuda_lib, z, u, **kw)


@pytest.mark.parametrize("kw", [dict(t=3.0), dict(t=2.0, p=0.99), dict(k=100000, t=2.0), dict(k=100000, p=0.9, t=2.0), dict(t=2.0, m=1e-4), dict(t=1.0, k=64, p=0.95)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_wide_sets_of_a_large_vocabulary(cuda_lib, kw, dtype):
    z, u = rows(3, 262144, seed=7, dtype=dtype)
    check(cuda_lib, z, u, **kw)


@pytest.mark.parametrize("V", [1000, 40000, 262144])
def test_equal_logits(cuda_lib, V):
    """Ties: the set is the lowest indices, the token the index that u points at."""
    z = torch.full((6, V), 3.25, device="cuda")
    u = torch.tensor([0.0, 0.25, 0.5, 0.75, 0.999, 1 - 2.0 ** -24], device="cuda")
    for kw, n in ((dict(), V), (dict(k=V // 3), V // 3), (dict(p=0.25), V // 4), (dict(m=1.0), V)):
        tok, lp = cuda_lib.logits_sample(z, u, None, *(torch.full((6,), kw[x], dtype=d, device="cuda") if x in kw else None
                                                        for x, d in (("k", torch.int32), ("p", F32), ("m", F32))))
        torch.cuda.synchronize()
        want = [min(int(np.floor(float(x) * n)), n - 1) for x in u]
        assert tok.tolist() == want, kw
        assert np.allclose(lp.cpu().numpy(), -np.log(n), rtol=2.0 ** -23)


def test_many_ties_at_the_border(cuda_lib):
    """Logits on a coarse grid: thousands of equal ones at each border."""
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    z = torch.randint(0, 12, (4, 50000), generator=g, device="cuda").float()
    u = torch.rand(4, generator=g, device="cuda")
    for kw in (dict(k=5000), dict(p=0.5), dict(k=9000, p=0.7), dict(k=1500, m=0.5), dict(t=4.0, p=0.8)):
        check(cuda_lib, z, u, **kw)


@pytest.mark.parametrize("V", [70, 3001, 200000])
def test_infinities_and_nan(cuda_lib, V):
    z, u = rows(8, V, seed=9)
    z[0, :] = float("-inf")
    z[1, :] = float("nan")
    z[2, 5:] = float("-inf")                       # a grammar that leaves five
    z[3, ::2] = float("nan")
    z[4, 11] = float("inf")
    z[5, 7] = z[5, 60] = float("inf")
    z[6, :] = torch.finfo(F32).min                 # masks of the type's lowest value
    z[6, 3] = 1.0
    z[7, :] = torch.finfo(F32).min
    check(cuda_lib, z, u)
    check(cuda_lib, z, u, k=20, p=0.9)
    check(cuda_lib, z, u, p=0.5, t=0.1)
    check(cuda_lib, z, u, m=0.1, t=5.0)
    check(cuda_lib, z, u, k=V - 1)


def test_greedy_and_extreme_settings(cuda_lib):
    z, u = rows(4, 9000, seed=4, std=1.0)
    z[1, 77] = z[1, 400] = 9.0
    for kw in (dict(t=0.0), dict(t=-1.0), dict(k=1), dict(p=0.0), dict(t=1e-30), dict(t=float("inf")), dict(t=1e30, k=10),
               dict(t=1e-4, p=0.5), dict(m=1.0), dict(m=1e-30), dict(k=9000), dict(k=2 ** 31 - 1), dict(k=-3), dict(p=2.0), dict(p=1e-20)):
        check(cuda_lib, z, u, **kw)
    tok, lp = cuda_lib.logits_sample(z, u, torch.full((4,), float("nan"), device="cuda"))
    assert tok.tolist() == z.argmax(1).tolist() and lp.tolist() == [0.0] * 4
    # u outside [0, 1) is clamped
    edge = torch.tensor([-1.0, 1.0, 5.0, float("nan")], device="cuda")
    tok, _ = cuda_lib.logits_sample(z, edge, top_k=torch.full((4,), 10, dtype=torch.int32, device="cuda"))
    for i, x in enumerate((0.0, 1 - 2.0 ** -24, 1 - 2.0 ** -24, 0.0)):
        assert int(tok[i]) == O.sample(z[i].cpu().numpy(), x, top_k=10)[0]


def test_signed_zeros_tie(cuda_lib):
    z = torch.zeros(1, 300, device="cuda")
    z[0, ::2] = -0.0
    for x, want in ((0.0, 0), (0.99, 9)):
        tok, _ = cuda_lib.logits_sample(z, torch.tensor([x], device="cuda"), top_k=torch.tensor([10], dtype=torch.int32, device="cuda"))
        assert int(tok) == want


@pytest.mark.parametrize("V", [300, 5000, 60000, 262144])
def test_top_p_over_whole_rows(cuda_lib, V):
    """Borders from the first element to the last, spread and peaked rows, with min-p above and below the border."""
    z, u = rows(4, V, seed=V + 1)
    z[2] *= 3.0
    z[3] = (z[3] * 4).round() / 4
    for p in (1e-30, 1e-6, 0.01, 0.3, 0.9, 0.99, 0.999, 0.99999, 1 - 2.0 ** -24)[::1 if V < 200000 else 3]:
        check(cuda_lib, z, u, p=p)
        check(cuda_lib, z, u, p=p, t=2.5)
    for m in (1e-5, 0.003, 0.02, 0.3, 1.0)[::1 if V < 200000 else 2]:
        check(cuda_lib, z, u, p=0.7, m=m)
        check(cuda_lib, z, u, p=0.98, m=m, t=1.5)


def test_borders_next_to_zero(cuda_lib):
    """The border among the smallest negative numbers, with zeros of both signs above."""
    V = 12000
    z = torch.full((16, V), -30.0, device="cuda")
    u = torch.linspace(0.01, 0.99, 16, device="cuda")
    for i in range(16):
        z[i, 0] = 0.03 + 0.0013 * i   # the first bin ends at another key each time
        z[i, 1:3000], z[i, 3000:4000] = 0.0, -0.0
        for j in range(4):
            z[i, 4000 + 1000 * j:5000 + 1000 * j] = -(j + 1) * 2.0 ** -149
    for k in (4500, 5500, 6500, 7500):
        check(cuda_lib, z, u, k=k)
        check(cuda_lib, z, u, k=k, p=0.9)
    for p in (0.45, 0.55, 0.7, 0.8):
        check(cuda_lib, z, u, p=p)


def test_rows_with_their_own_settings_strides_streams_graphs(cuda_lib):
    q4w = cuda_lib
    z, u = rows(9, 30007, seed=11)
    i = torch.arange(9, device="cuda")
    k = torch.tensor([0, 64, 1, 2000, 0, 40, 0, 30006, 5], dtype=torch.int32, device="cuda")
    p = torch.tensor([0.9, 0.95, 1.0, 0.8, 1.0, 0.5, 0.99, 1.0, 0.1], device="cuda")
    m = torch.tensor([0.0, 0.0, 0.0, 0.01, 0.02, 0.3, 0.0, 0.0, 0.9], device="cuda")
    t = 0.5 + 0.25 * i.float()
    tok, lp = check(q4w, z, u, t, k, p, m)
    wide = torch.zeros(9, 30100, device="cuda")
    wide[:, 33:33 + 30007] = z
    with pytest.raises(q4w.Q4Error):
        q4w.logits_sample(wide[:, 33:33 + 30007], u, t, k, p, m)        # not 16-byte aligned
    wide[:, 32:32 + 30007] = z
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        tok2, lp2 = q4w.logits_sample(wide[:, 32:32 + 30007], u, t, k, p, m)
    torch.cuda.synchronize()
    assert torch.equal(tok, tok2) and torch.equal(lp, lp2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q4w.logits_sample(z, u, t, k, p, m, tokens=tok2, logprobs=lp2)
    u.copy_(torch.rand_like(u))
    g.replay()
    torch.cuda.synchronize()
    tok, lp = check(q4w, z, u, t, k, p, m)
    assert torch.equal(tok, tok2) and torch.equal(lp, lp2)


@pytest.mark.parametrize("b,V", [(512, 100), (700, 300), (1025, 70), (90, 9000)])
def test_more_rows_than_run_at_once(cuda_lib, b, V):
    """Rows are then taken by their settings, not in their order."""
    z, u = rows(b, V, seed=b)
    g = np.random.default_rng(b)
    pick = lambda x, dt: torch.tensor(g.choice(x, b), dtype=dt, device="cuda")   # noqa: E731
    t, k, p = pick([0.0, 0.5, 1.0, 2.0], F32), pick([0, 0, 1, 5, 50], torch.int32), pick([0.0, 0.5, 0.9, 1.0, 1.0], F32)
    check(cuda_lib, z, u, t, k, p, pick([0.0, 0.1], F32))
    check(cuda_lib, z, u, t)
    check(cuda_lib, z, u, k=k)
    check(cuda_lib, z, u, p=p)


def test_frequencies_follow_the_distribution(cuda_lib):
    """Evenly spread u: each token is drawn in proportion to its probability."""
    z = torch.tensor([0.1, 0.4, 0.1, 0.3, 0.1], device="cuda").log()
    n = 10000
    u = (torch.arange(n, device="cuda") + 0.5) / n
    tok, _ = cuda_lib.logits_sample(z.expand(n, 5).contiguous(), u)
    got = torch.bincount(tok.long(), minlength=5).tolist()
    assert all(abs(a - n * b) <= 1 for a, b in zip(got, (0.1, 0.4, 0.1, 0.3, 0.1)))


def test_largest_vocabulary(cuda_lib):
    z, u = rows(1, 1048576, seed=12)
    check(cuda_lib, z, u, t=2.0)
    check(cuda_lib, z, u, k=500000, p=0.9, t=2.0)


def tail_rows(V, near, depths, seed=3):
    """A row per depth: index 0 lies that far below the maximum, `near` others within a
    few of it, the rest where no weight counts (2^-200 and less)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    b = len(depths)
    z = 1.5 - 140 - torch.rand(b, V, generator=g, device="cuda")
    z[:, 1:1 + near] = 1.5 - 3 * torch.rand(b, near, generator=g, device="cuda")
    z[:, near] = 1.5
    z[:, 0] = 1.5 - torch.tensor(depths, device="cuda")
    return z


@pytest.mark.parametrize("V,near", [(2, 1), (300, 7), (9000, 100), (9000, 3000), (262144, 90), (262144, 5000)])
def test_log_probability_of_an_improbable_token(cuda_lib, V, near):
    """A drawn token of weight 2^-26 to 2^-42: its log probability keeps every digit."""
    depths = [18.0, 20.3, 24.0, 26.7, 28.0, 28.9, 29.05] if V < 200000 else [20.3, 29.05]
    z = tail_rows(V, near, depths)
    u = torch.tensor([np.exp(-x) / (4 * near) for x in depths], dtype=F32, device="cuda")
    for kw in (dict(), dict(k=near + 1), dict(m=1e-13)) if near + 1 < V else (dict(), dict(m=1e-13)):
        tok, _ = check(cuda_lib, z, u, **kw)
        assert tok.tolist() == [0] * len(depths)
        if V < 200000:
            check(cuda_lib, z * 0.5, u, t=0.5, **kw)


@pytest.mark.parametrize("V,near", [(2, 1), (300, 7), (9000, 100), (9000, 3000), (262144, 90), (262144, 5000)])
def test_zero_takes_the_first_of_the_set(cuda_lib, V, near):
    """u = 0: the first index of S, with weights from 2^-25 to 2^-126; u next to 0."""
    depths = [17.4, 22.0, 28.0, 29.2, 31.0, 35.0, 41.6, 60.0, 87.0] if V < 200000 else [22.0, 41.6, 87.0]
    z = tail_rows(V, near, depths)
    u = torch.zeros(len(depths), device="cuda")
    for kw in (dict(), dict(k=near + 1)) if near + 1 < V else (dict(),):
        tok, _ = check(cuda_lib, z, u, **kw)
        assert tok.tolist() == [0] * len(depths)
    check(cuda_lib, z[:7], u[:7], m=2.0 ** -58)
    # cut by a filter, it is not the first of S
    for kw in (dict(p=0.9), dict(k=near, p=0.9), dict(m=0.01), dict(k=near)) if V < 200000 else (dict(p=0.9), dict(k=near)):
        tok, _ = check(cuda_lib, z, u, **kw)
        assert min(tok.tolist()) >= 1
    # next to 0: below the weight of the first, and above it
    few = depths[:3] if V < 200000 else depths[:1]
    w = np.exp(-np.array(few))
    for f, first in ((0.25, True), (3.0 * near, False)):
        tok, _ = check(cuda_lib, z[:len(few)], torch.tensor(w * f / near, dtype=F32, device="cuda"))
        assert [t == 0 for t in tok.tolist()] == [first] * len(few)


@pytest.mark.parametrize("V", [20000, 262144])
def test_zero_with_a_wide_set(cuda_lib, V):
    """Top-p whose border lies among thousands of small weights, apart and tied."""
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    z = -13.0 - 0.7 * torch.rand(3, V, generator=g, device="cuda")
    z[1] = -13.5
    z[2, 1:] = (z[2, 1:] * 64).round() / 64
    z[:, V // 2] = 0.0
    z[:, 0] = -13.001
    z[1, 0] = -13.5
    u = torch.zeros(3, device="cuda")
    n = float(torch.exp(z[0].double()).sum()) - 1.0        # the tail's share
    for p in (1 - 0.5 * n / (1 + n), 1 - 0.2 * n / (1 + n)):
        tok, _ = check(cuda_lib, z, u, p=p)
        assert tok.tolist() == [0, 0, 0]
        check(cuda_lib, z, u, p=p, m=1e-6)
        check(cuda_lib, z, torch.full_like(u, 2.0 ** -24), p=p)
    check(cuda_lib, z, u, k=5000, p=0.9999999)
    check(cuda_lib, z, u, k=5000)


def test_top_p_over_the_largest_vocabulary(cuda_lib):
    """131072 indices a CTA: short weights of 14 bits, every segment."""
    z, u = rows(2, 1048576, seed=13)
    check(cuda_lib, z, u, p=0.9, t=2.0)
    check(cuda_lib, z[:1], u[:1], p=0.99, m=0.002)
    check(cuda_lib, z[:1], torch.zeros(1, device="cuda"), p=0.9999, t=3.0)


@pytest.mark.parametrize("V", [131072, 1048575, 1048576])
@pytest.mark.parametrize("p", [1e-7, 0.25, 0.7, 1 - 2.0 ** -24])
def test_equal_logits_of_the_largest_vocabulary_under_top_p(cuda_lib, V, p):
    """One bin holds every weight (2^31 a CTA at the largest size); the set is the lowest
    indices, the token where u points, in exact fractions."""
    us = [0.0, 2.0 ** -24, 0.3, 0.999, 1 - 2.0 ** -24]
    u = torch.tensor(us, device="cuda")
    P = Fraction(float(torch.tensor(p, dtype=F32)))
    n = math.ceil(P * V)
    for m in (None, 0.5):
        tok, lp = cuda_lib.logits_sample(torch.full((5, V), -2.5, device="cuda"), u, None, None, torch.full((5,), p, device="cuda"),
                                         None if m is None else torch.full((5,), m, device="cuda"))
        torch.cuda.synchronize()
        assert tok.tolist() == [math.floor(Fraction(float(x)) * n) for x in u]
        assert np.allclose(lp.cpu().numpy(), -np.log(n), rtol=2.0 ** -23, atol=0)


def test_rows_of_eight_ctas_that_read_again(cuda_lib):
    """More rows than fit one CTA an SM, fewer than take four: every kind of row."""
    z, u = rows(16, 262144, seed=21)
    t = torch.tensor([0.0, 0.7, 1.0, 1.6] * 4, device="cuda")
    k = torch.tensor([0, 0, 50, 0, 4000, 0, 0, 1] * 2, dtype=torch.int32, device="cuda")
    p = torch.tensor([1.0, 0.9, 0.95, 1.0, 0.8, 0.99, 0.5, 1.0] * 2, device="cuda")
    m = torch.tensor([0.0] * 12 + [0.02] * 4, device="cuda")
    check(cuda_lib, z, u, t, k, p, m)
    check(cuda_lib, z[:13], torch.zeros(13, device="cuda"), p=0.95)
