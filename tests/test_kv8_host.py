"""On the CPU: the refusals of the quantised cache's entry points and of draft_verify, the
binding's size checks, and the oracle of draft_verify against closed forms."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import int4_q4_weight_gb300 as q4w
from oracle import kv8_oracle as O8

A = 0x10000     # an aligned address; a refused call reads nothing


@pytest.fixture(scope="module")
def lib():
    q4w.build()
    return q4w.load()


def refused(lib, status, word):
    assert status != 0 and word in lib.q4_last_error(), (status, lib.q4_last_error())


def cache(**kw):
    c = q4w.q4_kv_cache(A, A, A, A, A, 1, 10, 2, 16, 128, 3, 4)
    q = q4w.q4_kv_cache_q8(c, A, A)
    for k, v in kw.items():
        setattr(q if k.endswith("scales") else q.c, k, v)
    return ctypes.byref(q)


@pytest.mark.parametrize("kw,word", [(dict(k_scales=None), b"k_scales"), (dict(v_scales=A + 2), b"v_scales"), (dict(head_dim=96), b"head_dim"),
                                     (dict(dtype=0), b"dtype"), (dict(page_size=8), b"page_size"), (dict(k=None), b"k is NULL"),
                                     (dict(v=A + 8), b"aligned"), (dict(n_seqs=0), b"n_seqs"), (dict(n_pages=1 << 30), b"2^31")])
def test_quantised_cache_refusals(lib, kw, word):
    refused(lib, lib.kv_read_q8(cache(**kw), 1, A, A, None, None), word)
    refused(lib, lib.kv_append_q8(cache(**kw), 1, A, 256, A, 256, 1, None, 0, 0, None, None, None, None, 0.0, None, 0, 0, None, None, None), word)
    refused(lib, lib.kv_attention_q8(cache(**kw), 1, 1, A, 256, 2, 1.0, 0, A, None, None, A, 1 << 30, None), word)


def test_append_norm_and_q8_refusals(lib):
    names = "T k ks v vs inp q qs nq out qn kn vn eps steps rot inter pos err".split()
    good = dict(zip(names, [4, A, 256, A, 256, 0, A, 512, 4, A, A, A, A, 1e-6, A, 128, 0, None, None]))
    plain = q4w.q4_kv_cache(A, A, A, A, A, 1, 10, 2, 16, 128, 3, 4)
    for call, c in ((lib.kv_append_norm, ctypes.byref(plain)), (lib.kv_append_q8, cache())):
        for kw, word in ((dict(T=0), b"T=0"), (dict(k=None), b"k is NULL"), (dict(inp=3), b"in_dtype"), (dict(ks=255), b"k_stride"), (dict(vs=257), b"v_stride"),
                         (dict(q=None), b"together"), (dict(q=None, out=None), b"q_norm without q"), (dict(qn=A + 4), b"q_norm"), (dict(kn=A + 4), b"k_norm"),
                         (dict(vn=A + 4), b"v_norm"), (dict(eps=-1.0), b"eps"), (dict(eps=float("nan")), b"eps"), (dict(eps=float("inf")), b"eps"),
                         (dict(rot=24), b"rot_dim"), (dict(rot=144), b"rot_dim"), (dict(steps=None), b"steps"), (dict(inter=2), b"interleaved"), (dict(err=A + 4), b"err")):
            refused(lib, call(c, *{**good, **kw}.values(), None), word)


def test_read_and_attention_refusals(lib):
    refused(lib, lib.kv_read_q8(cache(), 0, A, A, None, None), b"T=0")
    refused(lib, lib.kv_read_q8(cache(), 1, None, A, None, None), b"k_out")
    refused(lib, lib.kv_read_q8(cache(), 1, A, A + 8, None, None), b"v_out")
    refused(lib, lib.kv_read_q8(cache(), 1 << 30, A, A, None, None), b"2^31")
    names = "T max_q q qs nq scale window out lse err ws n".split()
    good = dict(zip(names, [4, 2, A, 512, 4, 1.0, 0, A, None, None, A, 1 << 30]))
    for kw, word in ((dict(T=0), b"T=0"), (dict(max_q=5), b"max_q"), (dict(q=None), b"q is NULL"), (dict(nq=3), b"n_q=3"), (dict(nq=512), b"n_q=512"),
                     (dict(window=-1), b"window"), (dict(scale=float("nan")), b"scale"), (dict(qs=511), b"q_stride"), (dict(ws=A + 8), b"ws")):
        refused(lib, lib.kv_attention_q8(cache(), *{**good, **kw}.values(), None), word)


def test_draft_verify_refusals(lib):
    names = "z us rs dtype b k V x u y dus drs t tok acc lp ws n".split()
    V = 1001
    good = dict(zip(names, [A + 4, 5 * V, V, 0, 3, 4, V, A, A, A + 8, 4 * V, V, A, A, A, A, A, 1 << 30]))
    call = lambda **kw: lib.draft_verify(*{**good, **kw}.values(), None)   # noqa: E731
    for kw, word in ((dict(z=None), b"logits"), (dict(z=A + 2), b"aligned"), (dict(y=A + 1), b"draft_logits"), (dict(dtype=3), b"dtype"), (dict(b=0), b"b=0"),
                     (dict(b=65536), b"b=65536"), (dict(k=-1), b"k=-1"), (dict(k=65), b"k=65"), (dict(V=0), b"V=0"), (dict(V=(1 << 20) + 1), b"V="),
                     (dict(x=None), b"drafts"), (dict(u=None), b"u is NULL"), (dict(tok=None), b"tokens"), (dict(acc=None), b"accepted"), (dict(x=A + 4), b"drafts"),
                     (dict(lp=A + 4), b"logprobs"), (dict(t=A + 4), b"temperature"), (dict(rs=V - 1), b"row_stride"), (dict(us=V - 1), b"user_stride"),
                     (dict(drs=V - 1), b"draft_row_stride"), (dict(dus=0), b"draft_user_stride"), (dict(us=1 << 40), b"user_stride"),
                     (dict(ws=A + 4), b"ws"), (dict(ws=None), b"ws must hold"), (dict(n=lib.draft_verify_ws_bytes(3, 4, V) - 1), b"ws must hold")):
        refused(lib, call(**kw), word)
    for sizes in ((0, 1, 10), (1, -1, 10), (1, 65, 10), (1, 1, 0), (65536, 1, 10), (1, 1, (1 << 20) + 1)):
        assert lib.draft_verify_ws_bytes(*sizes) == 0
    # the largest sizes do not wrap
    n = lib.draft_verify_ws_bytes(65535, 64, 1 << 20)
    assert n >= 65535 * (129 * 128 * 8 + 2 * 4096 * 8)


class _Lib:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 4096 if name.endswith("bytes") else 0
        return call


@pytest.fixture
def fake(monkeypatch):
    f = _Lib()
    monkeypatch.setattr(q4w, "load", lambda: f)
    monkeypatch.setattr(q4w, "_dev", lambda t, dtype, name: None if t is None or t.dtype == dtype and t.is_contiguous() else (_ for _ in ()).throw(q4w.Q4Error(name)))
    monkeypatch.setattr(q4w, "_here", lambda t: True)
    monkeypatch.setattr(q4w, "_stream", lambda: None)
    monkeypatch.setattr(q4w, "_raw_alloc", lambda n, stream: 4096)
    monkeypatch.setattr(q4w, "_raw_free", lambda p: None)
    q4w._draft_ws_bytes.cache_clear()
    yield f
    q4w._draft_ws_bytes.cache_clear()


def test_binding_checks_the_sizes_of_a_verification(fake):
    z, y = torch.zeros(3, 5, 50), torch.zeros(3, 4, 50)
    x, u, t = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, 5), torch.ones(3)
    q4w.draft_verify(z, x, u, y, t)
    q4w.draft_verify(torch.zeros(3, 5, 60)[..., 3:53], x, u, torch.zeros(4, 3, 50).transpose(0, 1))
    q4w.draft_verify(z[:, :1], x[:, :0], u[:, :1].contiguous(), y[:, :0])
    assert fake.calls.count("draft_verify") == 3
    for f in (lambda: q4w.draft_verify(z[0], x, u), lambda: q4w.draft_verify(z.double(), x, u), lambda: q4w.draft_verify(z, x[:, :3].contiguous(), u),
              lambda: q4w.draft_verify(z, x.long(), u), lambda: q4w.draft_verify(z, x, u[:, :4].contiguous()), lambda: q4w.draft_verify(z, x, u, y[:, :3]),
              lambda: q4w.draft_verify(z, x, u, y.half()), lambda: q4w.draft_verify(z, x, u, y, t[:2]), lambda: q4w.draft_verify(torch.zeros(3, 5, 100)[..., ::2], x, u),
              lambda: q4w.draft_verify(z, x, u, tokens=torch.zeros(3, 4, dtype=torch.int32)), lambda: q4w.draft_verify(z, x, u, accepted=torch.zeros(3)),
              lambda: q4w.draft_verify(z, x, u, logprobs=torch.zeros(15)), lambda: q4w.draft_verify(z, x.t().contiguous().t(), u)):
        with pytest.raises(q4w.Q4Error):
            f()
    assert fake.calls.count("draft_verify") == 3
    assert q4w.draft_verify(z[:0], x[:0], u[:0])[0].shape == (0, 5)


def test_oracle_of_the_verification():
    """Exact fractions: p, q of powers of two."""
    z = np.log(np.array([[0.5, 0.25, 0.25], [0.125, 0.5, 0.375]]))
    y = np.log(np.array([[0.25, 0.5, 0.25]]))
    # p(1) / q(1) = 1/2
    for u0, n in ((0.0, 1), (0.49, 1), (0.51, 0), (0.99, 0)):
        for u1, drawn in ((0.0, 0), (0.6, 1 if n else 0), (0.9, 2 if n else 0)):
            tok, acc, lp = O8.verify(z, [1], [u0, u1], y)
            assert acc == n and tok.tolist() == ([1, drawn] if n else [0, -1])
            assert np.allclose(lp, [np.log(0.25), z[1, drawn]] if n else [np.log(0.5), 0])
    # without probabilities: the draft is taken out of p
    assert O8.verify(z, [0], [0.5, 0.4])[0].tolist() == [1, -1] and O8.verify(z, [0], [0.49, 0.1])[0].tolist() == [0, 0]
    # none, greedy, empty rows
    assert O8.verify(z, [-1], [0.0, 0.8], y)[0].tolist() == [2, -1]
    assert O8.verify(z, [0], [0.9, 0.8], y, 0.0)[0].tolist() == [0, 1] and O8.verify(z, [1], [0.0, 0.0], y, 0.0)[0].tolist() == [0, -1]
    tok, acc, lp = O8.verify(np.full((2, 3), -np.inf), [1], [0.0, 0.0], y)
    assert tok.tolist() == [-1, -1] and acc == 0 and lp[0] == -np.inf


def test_rounding_a_scale_up():
    for x in (0.0, 1e-9, 2.0 ** -24, 5e-8, 6.1e-5, 0.1, 1.0, 1.0004, 515.4, 65504.0):
        up = O8.fp16_up(x)
        assert up == float(np.float16(up)) and up >= x and (up == 0 or float(np.nextafter(np.float16(up), np.float16(0))) < x)
    codes, scales, bad = O8.quantise(np.linspace(-3, 3, 64)[None])
    assert not bad.any() and (np.abs(O8.values(codes, scales) - np.linspace(-3, 3, 64)) <= np.repeat(scales, 32, -1) / 2).all()


@pytest.mark.parametrize("gone", [("alloc",), ("delete",), ("alloc", "delete")])
def test_the_package_without_the_private_allocator_calls(gone):
    """A build of torch that lacks them: the package is imported, its host checks answer, and a
    workspace is a tensor that is held until it is given back."""
    code = f"""
import torch
for n in {gone!r}:
    delattr(torch._C, "_cuda_cudaCachingAllocator_raw_" + n)
import int4_q4_weight_gb300 as q4w
assert q4w.load().kv_read_q8(None, 1, None, None, None, None) != 0
empty = torch.empty
torch.empty = lambda n, dtype, device: empty(n, dtype=dtype)
a, b = q4w._raw_alloc(4096, 0), q4w._raw_alloc(4096, 0)
assert a != b and a and b
q4w._raw_free(a)
assert list(q4w._held) == [b]
q4w._raw_free(b)
assert not q4w._held
"""
    q4w.build()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr


def test_workspace_sizes_of_the_quantised_attention(monkeypatch):
    """T counts for bf16 queries where the size grows with it, and is no part of what is kept elsewhere."""
    asked = []

    class Lib:
        def kv_attention_q8_ws_bytes(self, T, max_q, n_q, n_kv, head_dim):
            asked.append((T, max_q))
            return 1000 if max_q < 10 else 2000 + 10 * T

    class Device:
        def __init__(self, i):
            pass

        def __enter__(self):
            pass

        def __exit__(self, *a):
            pass

    monkeypatch.setattr(q4w, "load", lambda: Lib())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch, "empty", lambda n, dtype, device: n)
    for f in (q4w._attention_ws_bytes, q4w._attention_q8_grows):
        f.cache_clear()
    try:
        ws = lambda T, max_q, **kw: q4w.kv_attention_q8_ws(T, max_q, 8, 1, 256, "cuda", **kw)   # noqa: E731
        assert [ws(T, 40) for T in (40, 50)] == [2400, 2500]
        assert [ws(T, 40, dtype=torch.float16) for T in (40, 50)] == [2000, 2000]
        n = len(asked)
        assert {ws(T, 1, dtype=d) for T in range(1, 600) for d in (torch.float16, torch.bfloat16)} == {1000}
        assert len(asked) <= n + 2
        with pytest.raises(q4w.Q4Error):
            ws(40, 40, dtype=torch.float32)
    finally:
        for f in (q4w._attention_ws_bytes, q4w._attention_q8_grows):
            f.cache_clear()


@pytest.mark.parametrize("cache", [torch.zeros(3, 2, 16, 64, dtype=torch.int8), torch.zeros(()), None, (torch.zeros(3),), (1, 2, 3)])
def test_a_quantised_cache_is_a_pair(fake, cache):
    """A cache without its scales is refused by name, not by Python's unpacking."""
    pair = (torch.zeros(3, 2, 16, 64, dtype=torch.int8), torch.zeros(3, 2, 16, 2, dtype=torch.float16))
    cu, lens, table = torch.tensor([0, 1], dtype=torch.int32), torch.tensor([1], dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32)
    rows, q = torch.zeros(1, 2, 64), torch.zeros(1, 2, 64, dtype=torch.float16)
    for k, v in ((cache, pair), (pair, cache)):
        for call in (lambda: q4w.kv_read_q8(k, v, table, cu, lens, 1), lambda: q4w.kv_append_q8(rows, rows, k, v, table, cu, lens),
                     lambda: q4w.kv_attention_q8(q, k, v, table, cu, lens)):
            with pytest.raises(q4w.Q4Error, match="pair of codes and scales"):
                call()
    assert not fake.calls
