"""The paged-cache and sampling oracle against closed forms and brute force, the
cache's index arithmetic compiled for the host, and the refusals of the entry
points: all without a GPU."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest
import torch

import int4_q4_weight_gb300 as q4w
from oracle import kv_oracle as O

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "int4_q4_weight_gb300", "csrc")
A = 1 << 20   # an aligned, never-dereferenced stand-in address


@pytest.fixture(scope="module")
def lib():
    q4w.build()
    return q4w.load()


@pytest.fixture(scope="module")
def pages(tmp_path_factory):
    """q4w_pages.h compiled with the host compiler."""
    d = tmp_path_factory.mktemp("pages")
    src = d / "pages.cpp"
    src.write_text(f'#include "{CSRC}/q4w_pages.h"\nextern "C" {{\n'
                   "int page(const int32_t* r, int mp, int np, int ps, int pos) { return q4w::kv_page(r, mp, np, ps, pos); }\n"
                   "long long row(int p, int h, int ps, int i) { return q4w::kv_row(p, h, ps, i); }\n"
                   "int first(int pos, int w) { return q4w::kv_first(pos, w); }\n}\n")
    out = d / "pages.so"
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", str(src), "-o", str(out)], check=True)
    dll = ctypes.CDLL(str(out))
    dll.row.restype = ctypes.c_longlong
    return dll


def test_pages_stay_inside_the_cache(pages):
    table = np.array([3, 0, -1, 7, 8, 2 ** 31 - 1, -2 ** 31, 5], np.int32)
    p = table.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))
    for size in (16, 48, 128):
        for pos in (-2 ** 31, -1, 0, size - 1, size, 2 * size, 3 * size + 1, 4 * size, 5 * size, 6 * size, 7 * size,
                    8 * size - 1, 8 * size, 2 ** 31 - 1):
            at = pos // size
            want = int(table[at]) if 0 <= pos and at < 8 and 0 <= table[at] < 8 else -1
            assert pages.page(p, 8, 8, size, pos) == want, (size, pos)
    assert pages.row(2 ** 24, 8, 128, 7) == (2 ** 24 * 8 + 7) * 128      # passes 32 bits
    assert [pages.first(x, 4) for x in (-1, 0, 3, 4, 9)] == [0, 0, 0, 1, 6]
    assert pages.first(5, 0) == 0 and pages.first(2 ** 31 - 1, 2 ** 31 - 1) == 1


def test_first_position_of_a_window(pages):
    """Any position with any window, the largest among them; positions below zero too."""
    top = 2 ** 31 - 1
    for pos in (-top - 1, -top, -4096, -3, -2, -1, 0, 1, 5, 4096, top - 1, top):
        for w in (0, 1, 2, 3, 4096, top - 1, top):
            want = max(0, pos - w + 1) if w else 0
            assert pages.first(pos, w) == want, (pos, w)


def test_rotation_is_a_complex_product():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 32))
    f = 10000.0 ** (-np.arange(8) / 8)
    for inter in (False, True):
        y = O.rotate(x, 1237, f, inter)
        z = x[:, 0:16:2] + 1j * x[:, 1:16:2] if inter else x[:, :8] + 1j * x[:, 8:16]
        w = z * np.exp(1j * 1237 * f)
        got = y[:, 0:16:2] + 1j * y[:, 1:16:2] if inter else y[:, :8] + 1j * y[:, 8:16]
        assert np.allclose(got, w, rtol=0, atol=1e-11)
        assert np.array_equal(y[:, 16:], x[:, 16:])


def test_scores_of_rotated_rows_depend_on_the_distance_only():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal(16), rng.standard_normal(16)
    f = 10000.0 ** (-np.arange(8) / 8)
    a = O.rotate(q, 100, f, False) @ O.rotate(k, 93, f, False)
    b = O.rotate(q, 1007, f, False) @ O.rotate(k, 1000, f, False)
    assert abs(a - b) < 1e-10


def test_rope_steps():
    s = q4w.kv_rope_steps(8, 100.0, device="cpu")
    turns = (s.numpy().view(np.uint64).astype(np.float64)) / 2.0 ** 64
    assert np.allclose(turns, 100.0 ** (-np.arange(4) / 4) / (2 * math.pi), rtol=2 ** -52)
    assert q4w.kv_rope_steps(4, device="cpu", freqs=[0.0, math.pi]).tolist()[0] == 0
    # half a turn and more: the sign bit of the int64 is set
    assert q4w.kv_rope_steps(4, device="cpu", freqs=[math.pi, 1.5 * math.pi]).tolist() == [-2 ** 63, -2 ** 62]
    with pytest.raises(q4w.Q4Error):
        q4w.kv_rope_steps(8, device="cpu", freqs=[1.0])


def test_attention_oracle_closed_forms():
    kc = np.zeros((2, 1, 16, 64))
    vc = np.arange(2 * 16 * 64, dtype=np.float64).reshape(2, 1, 16, 64)
    table, cu, kv = np.array([[1, 0]]), [0, 1], [20]
    o, lse, _, _ = O.attention(np.ones((1, 1, 64)), kc, vc, table, cu, kv, 1.0)
    seq = np.concatenate([vc[1, 0], vc[0, 0, :4]])
    assert np.allclose(o[0, 0], seq.mean(0)) and abs(lse[0, 0] - math.log(20)) < 1e-12    # equal scores: the mean
    o, lse, _, _ = O.attention(np.ones((1, 1, 64)), kc, vc, table, cu, kv, 1.0, window=3)
    assert np.allclose(o[0, 0], seq[-3:].mean(0))
    o, lse, _, _ = O.attention(np.ones((1, 1, 64)), kc, vc, table, cu, [0], 1.0)
    assert np.all(o == 0) and lse[0, 0] == -np.inf
    kc[1, 0, 5] = 100.0                                                                    # one key that takes it all
    o, _, _, _ = O.attention(np.ones((1, 1, 64)), kc, vc, table, cu, kv, 1.0)
    assert np.allclose(o[0, 0], vc[1, 0, 5])


def test_sampling_oracle():
    z = np.log([0.1, 0.4, 0.1, 0.3, 0.1])
    pick = lambda u, **kw: O.sample(z, u, **kw)[0]   # noqa: E731
    assert [pick(u) for u in (0.0, 0.05, 0.11, 0.49, 0.51, 0.65, 0.91)] == [0, 0, 1, 1, 2, 3, 4]
    assert O.sample(z, 0.5, top_k=3)[2] == [0, 1, 3]              # a tie goes to the lower index
    assert O.sample(z, 0.5, top_p=0.65)[2] == [1, 3]
    assert O.sample(z, 0.5, top_k=2, top_p=0.5)[2] == [1]         # 0.4 of 0.7 reaches one half
    assert O.sample(z, 0.5, min_p=0.5)[2] == [1, 3]
    assert O.sample(z, 0.9, temperature=0.0)[0] == 1
    assert O.sample([-np.inf, np.nan], 0.5)[:2] == (-1, -np.inf)
    assert O.sample([np.inf, 1.0, np.inf], 0.6)[0] == 2
    t, lp, _ = O.sample(z, 0.5, top_k=2)
    assert t == 1 and abs(lp - math.log(0.4 / 0.7)) < 1e-12


def _cache(**kw):
    c = q4w.q4_kv_cache(A, A, A, A, A, 1, 8, 2, 16, 128, 3, 4)
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


@pytest.mark.parametrize("status,kw", [
    (1, dict(k=None)), (1, dict(v=None)), (1, dict(block_table=None)), (1, dict(cu_tokens=None)), (1, dict(kv_lens=None)),
    (3, dict(k=A + 8)), (3, dict(block_table=A + 4)), (3, dict(kv_lens=A + 4)),
    (2, dict(dtype=0)), (2, dict(dtype=3)), (2, dict(head_dim=96)), (2, dict(head_dim=1024)), (2, dict(page_size=8)),
    (2, dict(page_size=24)), (2, dict(page_size=2048)), (2, dict(n_pages=0)), (2, dict(n_kv=0)), (2, dict(n_seqs=0)),
    (2, dict(n_seqs=4097)), (2, dict(max_pages=0)), (2, dict(max_pages=2 ** 27 + 1)), (2, dict(n_pages=2 ** 26)),
])
def test_cache_refusals(lib, status, kw):
    assert lib.kv_append(_cache(**kw), 4, A, 256, A, 256, 1, None, 0, 0, None, A, 128, 0, None, None, None) == status
    assert lib.kv_attention(_cache(**kw), 4, 2, A, 512, 4, 0.1, 0, A, None, None, A, 1 << 30, None) == status
    assert lib.q4_last_error() != b""


def test_append_refusals(lib):
    def call(T=4, k=A, ks=256, v=A, vs=256, dt=1, q=A, qs=512, nq=4, qo=A, st=A, rot=128, inter=0, pos=None, err=None, cache=True):
        return lib.kv_append(_cache() if cache else None, T, k, ks, v, vs, dt, q, qs, nq, qo, st, rot, inter, pos, err, None)
    assert call(cache=False) == 1 and call(k=None) == 1 and call(v=None) == 1 and call(st=None) == 1
    assert call(k=A + 8) == 3 and call(qo=A + 4) == 3 and call(pos=A + 4) == 3 and call(err=A + 4) == 3
    assert call(ks=260) == 3 and call(vs=257) == 3 and call(qs=514) == 3          # strides that break the alignment
    assert call(T=0) == 2 and call(dt=3) == 2 and call(rot=136 + 8) == 2 and call(rot=24) == 2 and call(rot=-16) == 2
    assert call(inter=2) == 2 and call(ks=248) == 2 and call(qs=256) == 2 and call(nq=0) == 2
    assert call(q=None) == 2 and call(qo=None) == 2
    assert b"q_out" in lib.q4_last_error()


def test_attention_refusals(lib):
    def call(T=4, mq=2, q=A, qs=512, nq=4, scale=0.1, w=0, out=A, lse=None, err=None, cache=True):
        return lib.kv_attention(_cache() if cache else None, T, mq, q, qs, nq, scale, w, out, lse, err, A, 1 << 40, None)
    assert call(cache=False) == 1 and call(q=None) == 1 and call(out=None) == 1
    assert call(q=A + 2) == 3 and call(lse=A + 4) == 3 and call(qs=516) == 3
    assert call(T=0) == 2 and call(mq=0) == 2 and call(mq=5) == 2 and call(nq=3) == 2 and call(nq=0) == 2
    assert call(nq=2 * 129, qs=2 * 129 * 128) == 2 and call(w=-1) == 2 and call(qs=504) == 2
    assert call(scale=float("nan")) == 2 and call(scale=float("inf")) == 2
    assert b"scale" in lib.q4_last_error()


def test_sample_refusals(lib):
    def call(z=A, stride=100, dt=0, b=2, V=100, u=A, t=None, k=None, p=None, m=None, tok=A, lp=None):
        return lib.logits_sample(z, stride, dt, b, V, u, t, k, p, m, tok, lp, None)
    assert call(z=None) == 1 and call(u=None) == 1 and call(tok=None) == 1
    assert call(z=A + 4) == 3 and call(u=A + 4) == 3 and call(t=A + 4) == 3 and call(k=A + 8) == 3 and call(lp=A + 2) == 3
    assert call(dt=3) == 2 and call(b=0) == 2 and call(b=65536) == 2 and call(V=0) == 2 and call(V=2 ** 20 + 1, stride=2 ** 21) == 2
    assert call(stride=99) == 2
    assert b"stride" in lib.q4_last_error()


class _Lib:
    """Records which entry points were called; every call succeeds."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 0
        return call


@pytest.fixture
def fake(monkeypatch):
    f = _Lib()
    monkeypatch.setattr(q4w, "load", lambda: f)
    monkeypatch.setattr(q4w, "_dev", lambda t, dtype, name: None)
    monkeypatch.setattr(q4w, "_here", lambda t: True)
    monkeypatch.setattr(q4w, "_stream", lambda: None)
    return f


def _paged(T=5, hq=4, hkv=2, D=128, pages=6, seqs=2):
    z = lambda *s, dt=torch.float16: torch.zeros(*s, dtype=dt)   # noqa: E731
    return dict(q=z(T, hq, D), k=z(T, hkv, D), v=z(T, hkv, D),
                cache=[z(pages, hkv, 16, D), z(pages, hkv, 16, D), z(seqs, 3, dt=torch.int32),
                       z(seqs + 1, dt=torch.int32), z(seqs, dt=torch.int32)])


def test_binding_checks_sizes(fake):
    a = _paged()
    q4w.kv_append(a["k"], a["v"], *a["cache"], steps=torch.zeros(64, dtype=torch.int64), q=a["q"])
    q4w.kv_attention(a["q"], *a["cache"], ws=torch.zeros(16, dtype=torch.uint8))
    q4w.logits_sample(torch.zeros(3, 50), torch.zeros(3))
    assert fake.calls == ["kv_append", "kv_attention", "logits_sample"]
    c = a["cache"]
    bad = [
        lambda: q4w.kv_append(a["k"][:, :1], a["v"], *c),
        lambda: q4w.kv_append(a["k"], a["v"][:4], *c),
        lambda: q4w.kv_append(a["k"], a["v"], c[0], c[1][:5], *c[2:]),
        lambda: q4w.kv_append(a["k"], a["v"], c[0], c[1], c[2][:1], *c[3:]),
        lambda: q4w.kv_append(a["k"], a["v"], *c[:3], c[3][:2], c[4]),
        lambda: q4w.kv_append(a["k"], a["v"], *c, q=a["q"][..., :64]),
        lambda: q4w.kv_append(a["k"], a["v"], *c, q_out=a["q"]),
        lambda: q4w.kv_append(a["k"], a["v"], *c, positions=torch.zeros(4, dtype=torch.int32)),
        lambda: q4w.kv_append(a["k"].double(), a["v"].double(), *c),
        lambda: q4w.kv_attention(a["q"][:, :3], *c),
        lambda: q4w.kv_attention(a["q"], *c, out=a["q"][:4]),
        lambda: q4w.kv_attention(a["q"], *c, lse=torch.zeros(5, 3)),
        lambda: q4w.kv_attention(a["q"][0], *c),
        lambda: q4w.logits_sample(torch.zeros(50), torch.zeros(1)),
        lambda: q4w.logits_sample(torch.zeros(3, 50), torch.zeros(2)),
        lambda: q4w.logits_sample(torch.zeros(3, 50), torch.zeros(3), top_k=torch.zeros(2, dtype=torch.int32)),
        lambda: q4w.logits_sample(torch.zeros(3, 50, dtype=torch.float64), torch.zeros(3)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(q4w.Q4Error):
            f()
            print("case", i)
    assert len(fake.calls) == 3
    # no tokens, no rows: nothing to do
    assert q4w.kv_append(a["k"][:0], a["v"][:0], *c, q=a["q"][:0]).shape == (0, 4, 128)
    q4w.kv_attention(a["q"][:0], *c)
    q4w.logits_sample(torch.zeros(0, 50), torch.zeros(0))
    assert len(fake.calls) == 3


def test_workspace_sizes_belong_to_their_device(monkeypatch):
    """Two devices of different sizes: a size is that of the device that the workspace is
    for, whatever device is current and in whatever order they are asked for."""
    current = [0]

    class Lib:
        def kv_attention_ws_bytes(self, *a):
            return (1000, 3000)[current[0]]

    class Device:
        def __init__(self, i):
            self.i = i

        def __enter__(self):
            self.old, current[0] = current[0], self.i

        def __exit__(self, *a):
            current[0] = self.old

    monkeypatch.setattr(q4w, "load", lambda: Lib())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch, "empty", lambda n, dtype, device: (n, str(device)))
    q4w._attention_ws_bytes.cache_clear()
    try:
        ws = lambda d: q4w.kv_attention_ws(1, 8, 1, 256, d)[0]   # noqa: E731
        assert [ws("cuda"), ws("cuda:1"), ws("cuda:0")] == [1000, 3000, 1000]
        current[0] = 1
        assert [ws("cuda"), ws("cuda:0"), ws(torch.device("cuda", 1))] == [3000, 1000, 3000]
        assert current[0] == 1
        with pytest.raises(q4w.Q4Error):
            q4w.kv_attention_ws(1, 8, 1, 256, "cpu")
    finally:
        q4w._attention_ws_bytes.cache_clear()
