"""Python binding of libq4w.so, the q4_0 weight-only int4 decode kernels for GB300.

Argument marshalling only: every function here checks tensor placement and
dtypes, passes raw device pointers and the current CUDA stream to the C ABI
of the same name (declared in ``include/q4w.h``) and raises on a non-zero
status.  PyTorch provides device memory and streams; all computation runs in
the library's CUDA kernels.  There is no fallback: if the library cannot be
loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import struct

import torch

__all__ = [
    "load", "build", "Q4Error", "q4_quantize", "q4_gemv", "q4_gemv_weights_ro", "q4_gemv_stage", "q4_rmsnorm_f16",
    "q4_decode_pass", "q4_decode_pass_launches", "q2_gemv", "lmhead_softcap_argmax", "ple_gather_project", "q4_gemm_chunk",
    "q8_quantize", "ple_gather_project_q8", "q4_gemv_a8", "q4_gemm_chunk_a8", "q4_act_calibrate_a8",
    "kv_append", "kv_append_norm", "kv_rope_steps", "kv_attention", "kv_attention_ws", "logits_sample",
    "kv_append_q8", "kv_read_q8", "kv_attention_q8", "kv_attention_q8_ws", "draft_verify", "draft_verify_ws",
    "q4_workspace_bytes", "q4_version", "Q4_IN_F16", "Q4_IN_RMS_F16", "Q4_IN_RMS_F32",
    "Q4_IN_RMS2_F32", "Q4_OP_GEMV", "Q4_OP_GEMM_CHUNK", "Q4_OP_PLE", "Q4_OP_LMHEAD",
    "Q4_OP_DECODE_PASS", "q4_layer", "q4_matrix", "q4_kv_cache", "q4_kv_cache_q8",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libq4w.so")

Q4_IN_F16, Q4_IN_RMS_F16, Q4_IN_RMS_F32, Q4_IN_RMS2_F32 = 0, 1, 2, 3
Q4_OP_GEMV, Q4_OP_GEMM_CHUNK, Q4_OP_PLE, Q4_OP_LMHEAD, Q4_OP_DECODE_PASS = 0, 1, 2, 3, 4
_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}   # q4_dtype

_lib = None
_one_device = False   # set by load(): asking for the current device costs 1 us a tensor

vp = ctypes.c_void_p
ci = ctypes.c_int
cf = ctypes.c_float
csz = ctypes.c_size_t
cll = ctypes.c_longlong


class q4_matrix(ctypes.Structure):
    _fields_ = [("codes", vp), ("scales", vp)]


class q4_layer(ctypes.Structure):
    _fields_ = [("q_rows", ci), ("kv_rows", ci), ("mlp_rows", ci),
                ("q", q4_matrix), ("k", q4_matrix), ("v", q4_matrix), ("o", q4_matrix),
                ("gate", q4_matrix), ("up", q4_matrix), ("down", q4_matrix)]


class q4_kv_cache(ctypes.Structure):
    _fields_ = [("k", vp), ("v", vp), ("block_table", vp), ("cu_tokens", vp), ("kv_lens", vp),
                ("dtype", ci), ("n_pages", ci), ("n_kv", ci), ("page_size", ci), ("head_dim", ci),
                ("n_seqs", ci), ("max_pages", ci)]


class q4_kv_cache_q8(ctypes.Structure):
    _fields_ = [("c", q4_kv_cache), ("k_scales", vp), ("v_scales", vp)]


_SIGS = {
    "q4_quantize": (ci, [vp, ci, ci, vp, vp, vp, vp]),
    "q4_gemv": (ci, [vp, vp, vp, vp, ci, ci, ci, vp, csz, vp]),
    "q4_gemv_weights_ro": (ci, [vp, vp, vp, vp, ci, ci, ci, vp, csz, vp]),
    "q4_gemm_chunk": (ci, [vp, vp, vp, vp, ci, ci, ci, vp, csz, vp]),
    "q4_gemv_a8": (ci, [vp, vp, vp, cf, vp, ci, ci, vp]),
    "q4_gemm_chunk_a8": (ci, [vp, vp, vp, cf, vp, ci, ci, ci, vp, csz, vp]),
    "q4_act_calibrate_a8": (ci, [vp, ctypes.c_longlong, vp, vp]),
    "ple_gather_project": (ci, [vp, ci, vp, vp, ci, ci, ci, cf, vp, vp, ci, vp, cf, vp, vp, vp, vp]),
    "q8_quantize": (ci, [vp, ci, ci, vp, vp, vp, vp]),
    "ple_gather_project_q8": (ci, [vp, ci, vp, vp, ci, ci, ci, cf, vp, vp, vp, ci, vp, cf, vp, vp, vp, vp]),
    "lmhead_softcap_argmax": (ci, [vp, vp, vp, ci, ci, ci, cf, vp, vp, vp, vp, vp, csz, vp]),
    "lmhead_softcap_argmax_noalloc": (ci, [vp, vp, vp, ci, ci, ci, cf, vp, vp, vp, vp, vp]),
    "q4_decode_pass": (ci, [ctypes.POINTER(q4_layer), ci, ci, vp, vp, cf, vp, csz, vp]),
    "q4_decode_pass_launches": (ci, [ctypes.POINTER(q4_layer), ci, ci]),
    "q2_gemv": (ci, [vp, vp, vp, vp, ci, ci, vp]),
    "q4_gemv_stage": (ci, [ctypes.POINTER(q4_matrix), ctypes.POINTER(ci), ci, ci, vp, ci, cf, ci,
                           ctypes.POINTER(vp), ctypes.POINTER(vp), vp]),
    "q4_rmsnorm_f16": (ci, [vp, ci, cf, vp, vp]),
    "kv_append": (ci, [vp, ci, vp, cll, vp, cll, ci, vp, cll, ci, vp, vp, ci, ci, vp, vp,
                       vp]),
    "kv_append_norm": (ci, [vp, ci, vp, cll, vp, cll, ci, vp, cll, ci, vp, vp, vp, vp, cf, vp, ci, ci, vp, vp, vp]),
    "kv_append_q8": (ci, [vp, ci, vp, cll, vp, cll, ci, vp, cll, ci, vp, vp, vp, vp, cf, vp, ci, ci, vp, vp, vp]),
    "kv_read_q8": (ci, [vp, ci, vp, vp, vp, vp]),
    "kv_attention": (ci, [vp, ci, ci, vp, cll, ci, cf, ci, vp, vp, vp, vp, csz, vp]),
    "kv_attention_q8": (ci, [vp, ci, ci, vp, cll, ci, cf, ci, vp, vp, vp, vp, csz, vp]),
    "kv_attention_q8_ws_bytes": (csz, [ci, ci, ci, ci, ci]),
    "kv_attention_ws_bytes": (csz, [ci, ci, ci, ci]),
    "logits_sample": (ci, [vp, cll, ci, ci, ci, vp, vp, vp, vp, vp, vp, vp, vp]),
    "draft_verify": (ci, [vp, cll, cll, ci, ci, ci, ci, vp, vp, vp, cll, cll, vp, vp, vp, vp, vp, csz, vp]),
    "draft_verify_ws_bytes": (csz, [ci, ci, ci]),
    "q4_workspace_bytes": (csz, [ci, ci, ci, ci]),
    "q4_status_string": (ctypes.c_char_p, [ci]),
    "q4_last_error": (ctypes.c_char_p, []),
    "q4_version": (ci, []),
    "q4_device_status": (ci, [vp]),
    "q4_set_wait_limit": (ctypes.c_longlong, [ctypes.c_longlong]),
    "q4_set_trace": (ci, [vp, csz]),
}


class Q4Error(RuntimeError):
    pass


def build(force: bool = False) -> str:
    """Compile libq4w.so in-tree (nvcc, sm_103a)."""
    from . import _build
    return _build.build(force=force)


def load():
    """Load libq4w.so (raises if it is missing: there is no fallback path)."""
    global _lib, _one_device
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise Q4Error(f"{LIB_PATH} not found: build it first (int4_q4_weight_gb300.build())")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    _one_device = torch.cuda.device_count() == 1
    return lib


def _check(status: int, name: str):
    if status != 0:
        lib = load()
        raise Q4Error(f"{name}: {lib.q4_status_string(status).decode()}: "
                      f"{lib.q4_last_error().decode()}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream():
    # the current stream's handle without building a Stream object
    return torch._C._cuda_getCurrentRawStream(0 if _one_device else torch.cuda.current_device())


def _here(t):
    """Whether t is on the current CUDA device (the only one there is, as a rule)."""
    return t.get_device() == (0 if _one_device else torch.cuda.current_device())


def _numel(t, n, name):
    """An array a kernel reads or writes holds exactly the elements its sizes imply
    (the kernels trust the sizes, so a short buffer would be overrun)."""
    if t is not None and t.numel() != n:
        raise Q4Error(f"{name} has {t.numel()} elements; the sizes imply {n}")


def _dev(t, dtype, name):
    if t is None:
        return
    if _one_device and t.dtype is dtype and t.is_contiguous() and t.is_cuda and t.device.index == 0:
        return
    if not t.is_cuda:
        raise Q4Error(f"{name} must be a CUDA tensor")
    # every call launches on the current device's stream: a tensor on another
    # GPU would reach its kernels as a foreign pointer
    cur = torch.cuda.current_device()
    if t.device.index != cur:
        raise Q4Error(f"{name} is on cuda:{t.device.index}, the current device is cuda:{cur}")
    if t.dtype != dtype:
        raise Q4Error(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise Q4Error(f"{name} must be contiguous")


def q4_device_status():
    """Synchronise the current stream; raise if a kernel's bounded wait ran out."""
    _check(load().q4_device_status(_stream()), "q4_device_status")


def q4_set_wait_limit(cycles: int) -> int:
    return int(load().q4_set_wait_limit(cycles))


def q4_set_trace(buf=None):
    """Diagnostic stamps of the persistent decode pass into ``buf`` (uint64 CUDA tensor), or off."""
    if buf is None:
        _check(load().q4_set_trace(None, 0), "q4_set_trace")
    else:
        _dev(buf, torch.int64, "trace")
        _check(load().q4_set_trace(_ptr(buf), buf.numel() * 8), "q4_set_trace")


def q4_version() -> int:
    return load().q4_version()


def q4_workspace_bytes(op: int, a: int, b: int, c: int) -> int:
    return int(load().q4_workspace_bytes(op, a, b, c))


def q4_quantize(W, codes=None, scales=None, err=None):
    """fp32 W [N, K] -> (codes uint8 [N, K/2], scales fp16 [N, K/32])."""
    lib = load()
    _dev(W, torch.float32, "W")
    N, K = W.shape
    if codes is None:
        codes = torch.empty((N, K // 2), dtype=torch.uint8, device=W.device)
    if scales is None:
        scales = torch.empty((N, K // 32), dtype=torch.float16, device=W.device)
    _dev(codes, torch.uint8, "codes")
    _dev(scales, torch.float16, "scales")
    _dev(err, torch.int32, "err")
    _numel(codes, N * K // 2, "codes")
    _numel(scales, N * K // 32, "scales")
    _check(lib.q4_quantize(_ptr(W), N, K, _ptr(codes), _ptr(scales), _ptr(err), _stream()),
           "q4_quantize")
    return codes, scales


def q8_quantize(W, codes=None, scales=None, err=None):
    """fp32 W [N, K] -> (codes int8 [N, K], scales fp16 [N, K/32]), int8 per block of 32."""
    lib = load()
    _dev(W, torch.float32, "W")
    N, K = W.shape
    if codes is None:
        codes = torch.empty((N, K), dtype=torch.int8, device=W.device)
    if scales is None:
        scales = torch.empty((N, K // 32), dtype=torch.float16, device=W.device)
    _dev(codes, torch.int8, "codes")
    _dev(scales, torch.float16, "scales")
    _dev(err, torch.int32, "err")
    _numel(codes, N * K, "codes")
    _numel(scales, N * K // 32, "scales")
    _check(lib.q8_quantize(_ptr(W), N, K, _ptr(codes), _ptr(scales), _ptr(err), _stream()),
           "q8_quantize")
    return codes, scales


def q4_gemv(codes, scales, x, y=None):
    """y [b, N] f32 = dequant(codes, scales) @ x[b]  (x fp16 [b, K] or [K])."""
    return _gemv("q4_gemv", codes, scales, x, y)


def q4_gemv_weights_ro(codes, scales, x, y=None):
    """q4_gemv, promising that no earlier kernel still running on the stream
    writes codes or scales: the weight tiles stream before that kernel ends."""
    return _gemv("q4_gemv_weights_ro", codes, scales, x, y)


def _gemv(name, codes, scales, x, y):
    lib = load()
    _dev(codes, torch.uint8, "codes")
    _dev(scales, torch.float16, "scales")
    _dev(x, torch.float16, "x")
    N, K = codes.shape[0], codes.shape[1] * 2
    batch = 1 if x.dim() == 1 else x.shape[0]
    if y is None:
        y = torch.empty((batch, N) if x.dim() == 2 else (N,), dtype=torch.float32, device=x.device)
    _dev(y, torch.float32, "y")
    _numel(scales, N * K // 32, "scales")
    _numel(x, batch * K, "x")
    _numel(y, batch * N, "y")
    _check(getattr(lib, name)(_ptr(codes), _ptr(scales), _ptr(x), _ptr(y), N, K, batch, None, 0, _stream()), name)
    return y


def _matrix_shape(codes, scales, rows, cols, name):
    """codes uint8 [rows, cols/2] and rows * cols/32 scales, as the sizes imply."""
    if codes.dim() != 2 or tuple(codes.shape) != (rows, cols // 2):
        raise Q4Error(f"{name}.codes has shape {tuple(codes.shape)}; the sizes imply ({rows}, {cols // 2})")
    _numel(scales, rows * cols // 32, f"{name}.scales")


def q4_gemv_stage(mats, inp, in_mode, eps=1e-6, pair=False, out32=None, out16=None):
    """One fused decode-pass stage; ``mats`` is a list of (codes, scales)."""
    lib = load()
    n = len(mats)
    if not 1 <= n <= 3 or (pair and n != 2):
        raise Q4Error(f"q4_gemv_stage takes 1 to 3 matrices (exactly 2 with pair), got {n}")
    K = mats[0][0].shape[1] * 2
    for i, (c, s) in enumerate(mats):
        _matrix_shape(c, s, c.shape[0], K, f"mats[{i}]")
    if pair and mats[0][0].shape[0] != mats[1][0].shape[0]:
        raise Q4Error("pair: gate and up must have the same rows")
    _numel(inp, K, "in")
    arr = (q4_matrix * n)()
    rows = (ci * n)()
    o32 = (vp * n)()
    o16 = (vp * n)()
    out32 = list(out32) if out32 is not None else [None] * n
    out16 = list(out16) if out16 is not None else [None] * n
    for i, (c, s) in enumerate(mats):
        _dev(c, torch.uint8, f"mats[{i}].codes")
        _dev(s, torch.float16, f"mats[{i}].scales")
        arr[i] = q4_matrix(c.data_ptr(), s.data_ptr())
        rows[i] = c.shape[0]
        _dev(out32[i], torch.float32, f"out32[{i}]")
        _dev(out16[i], torch.float16, f"out16[{i}]")
        _numel(out32[i], c.shape[0], f"out32[{i}]")
        _numel(out16[i], c.shape[0], f"out16[{i}]")
        o32[i] = out32[i].data_ptr() if out32[i] is not None else None
        o16[i] = out16[i].data_ptr() if out16[i] is not None else None
    _dev(inp, torch.float16 if in_mode in (Q4_IN_F16, Q4_IN_RMS_F16) else torch.float32, "in")
    _check(lib.q4_gemv_stage(arr, rows, n, K, _ptr(inp), in_mode, eps, int(pair), o32, o16,
                             _stream()), "q4_gemv_stage")
    return out32, out16


def q4_rmsnorm_f16(inp, eps=1e-6, out=None):
    lib = load()
    _dev(inp, torch.float32, "in")
    if out is None:
        out = torch.empty(inp.shape, dtype=torch.float16, device=inp.device)
    _dev(out, torch.float16, "out")
    _numel(out, inp.numel(), "out")
    _check(lib.q4_rmsnorm_f16(_ptr(inp), inp.numel(), eps, _ptr(out), _stream()), "q4_rmsnorm_f16")
    return out


def _check_layers(layers, H):
    """Every matrix of every layer has the shape the pass reads for hidden H:
    q [Q, H], k and v [KV, H] (together or both absent), o [H, Q],
    gate and up [I, H], down [H, I]."""
    for i, lw in enumerate(layers):
        if ("k" in lw) != ("v" in lw):
            raise Q4Error(f"layers[{i}]: k and v must be given together")
        Q, I = lw["q"][0].shape[0], lw["g"][0].shape[0]
        KV = lw["k"][0].shape[0] if "k" in lw else 0
        want = {"q": (Q, H), "k": (KV, H), "v": (KV, H), "o": (H, Q), "g": (I, H), "u": (I, H), "d": (H, I)}
        for key, (r, c) in want.items():
            if key in lw:
                _matrix_shape(*lw[key], r, c, f"layers[{i}].{key}")
            elif key not in ("k", "v"):
                raise Q4Error(f"layers[{i}] has no '{key}' matrix")


def make_layers(layers, H=None):
    """Host descriptor array from a list of dicts name -> (codes, scales); every
    shape is checked against hidden size H (taken from layer 0's q when None)."""
    if H is None:
        H = layers[0]["q"][0].shape[1] * 2
    _check_layers(layers, H)
    arr = (q4_layer * len(layers))()
    for i, lw in enumerate(layers):
        d = q4_layer()
        d.q_rows = lw["q"][0].shape[0]
        d.kv_rows = lw["k"][0].shape[0] if "k" in lw else 0
        d.mlp_rows = lw["g"][0].shape[0]
        for fld, key in (("q", "q"), ("k", "k"), ("v", "v"), ("o", "o"), ("gate", "g"),
                         ("up", "u"), ("down", "d")):
            if key in lw:
                c, s = lw[key]
                _dev(c, torch.uint8, f"layers[{i}].{key}.codes")
                _dev(s, torch.float16, f"layers[{i}].{key}.scales")
                setattr(d, fld, q4_matrix(c.data_ptr(), s.data_ptr()))
        arr[i] = d
    return arr


def decode_pass_ws_bytes(layers, H):
    qkv = max(lw["q"][0].shape[0] + 2 * (lw["k"][0].shape[0] if "k" in lw else 0) for lw in layers)
    mlp = max(lw["g"][0].shape[0] for lw in layers)
    return q4_workspace_bytes(Q4_OP_DECODE_PASS, H, qkv, mlp)


def q4_decode_pass(layers, h0, h_out, ws, eps=1e-6, descs=None):
    """Run the weight pass over ``layers`` (list of dicts) from fp16 h0 [H] into
    fp16 h_out [H].  ``descs``: the descriptor array make_layers(layers, H) built
    for the same layers (the layers' shapes are checked either way)."""
    lib = load()
    _dev(h0, torch.float16, "h0")
    _dev(h_out, torch.float16, "h_out")
    _dev(ws, torch.uint8, "ws")
    H = h0.numel()
    _numel(h_out, H, "h_out")
    if descs is None:
        descs = make_layers(layers, H)
    else:
        if len(descs) != len(layers):
            raise Q4Error(f"descs holds {len(descs)} layers, layers {len(layers)}")
        _check_layers(layers, H)
    _check(lib.q4_decode_pass(descs, len(descs), h0.numel(), _ptr(h0), _ptr(h_out), eps, _ptr(ws),
                              ws.numel(), _stream()), "q4_decode_pass")
    return h_out


def lmhead_ws(V, K, b, device):
    return torch.empty(q4_workspace_bytes(Q4_OP_LMHEAD, V, K, b), dtype=torch.uint8, device=device)


def lmhead_softcap_argmax(codes, scales, h, cap=30.0, ws=None, idx=None, top1=None, top2=None,
                          logits=None):
    """Returns (idx int32 [b], top1 f32 [b], top2 f32 [b], logits or None)."""
    lib = load()
    _dev(codes, torch.uint8, "codes")
    _dev(scales, torch.float16, "scales")
    _dev(h, torch.float16, "h")
    V, K = codes.shape[0], codes.shape[1] * 2
    b = 1 if h.dim() == 1 else h.shape[0]
    dev = h.device
    if ws is None:
        ws = lmhead_ws(V, K, b, dev)
    idx = torch.empty(b, dtype=torch.int32, device=dev) if idx is None else idx
    top1 = torch.empty(b, dtype=torch.float32, device=dev) if top1 is None else top1
    top2 = torch.empty(b, dtype=torch.float32, device=dev) if top2 is None else top2
    for t, dt, nm in ((idx, torch.int32, "idx"), (top1, torch.float32, "top1"),
                      (top2, torch.float32, "top2"), (logits, torch.float32, "logits"),
                      (ws, torch.uint8, "ws")):
        _dev(t, dt, nm)
    _numel(scales, V * K // 32, "scales")
    _numel(h, b * K, "h")
    for t, nm in ((idx, "idx"), (top1, "top1"), (top2, "top2")):
        _numel(t, b, nm)
    _numel(logits, b * V, "logits")
    _check(lib.lmhead_softcap_argmax(_ptr(codes), _ptr(scales), _ptr(h), b, V, K, cap, _ptr(idx),
                                     _ptr(top1), _ptr(top2), _ptr(logits), _ptr(ws), ws.numel(),
                                     _stream()), "lmhead_softcap_argmax")
    return idx, top1, top2, logits


def _ple_sizes(S, V, L, ld, D, table, row_scale, hidden, norm_w, out, gathered):
    _numel(table, V * L * ld, "table (V rows of L*ld bytes)")
    _numel(row_scale, V, "row_scale")
    _numel(hidden, S * D, "hidden")
    _numel(norm_w, ld, "norm_w")
    _numel(out, S * L * ld, "out")
    _numel(gathered, S * L * ld, "gathered")


def ple_gather_project(ids, table, row_scale, proj, hidden, norm_w, L=35, ld=256,
                       embed_scale=16.0, eps=1e-6, out=None, gathered=None, err=None):
    """Returns (out f32 [S, L*ld], gathered int8 [S, L*ld] or None)."""
    lib = load()
    _dev(ids, torch.int32, "ids")
    _dev(table, torch.int8, "table")
    _dev(row_scale, torch.float32, "row_scale")
    _dev(proj, torch.float32, "proj")
    _dev(hidden, torch.float16, "hidden")
    _dev(norm_w, torch.float32, "norm_w")
    S = ids.numel()
    V = table.shape[0]
    D = proj.shape[1]
    if out is None:
        out = torch.empty((S, L * ld), dtype=torch.float32, device=ids.device)
    _dev(out, torch.float32, "out")
    _dev(gathered, torch.int8, "gathered")
    _dev(err, torch.int32, "err")
    _ple_sizes(S, V, L, ld, D, table, row_scale, hidden, norm_w, out, gathered)
    _numel(proj, L * ld * D, "proj")
    _check(lib.ple_gather_project(_ptr(ids), S, _ptr(table), _ptr(row_scale), V, L, ld, embed_scale,
                                  _ptr(proj), _ptr(hidden), D, _ptr(norm_w), eps, _ptr(out),
                                  _ptr(gathered), _ptr(err), _stream()), "ple_gather_project")
    return out, gathered


def ple_gather_project_q8(ids, table, row_scale, proj_codes, proj_scales, hidden, norm_w, L=35, ld=256,
                          embed_scale=16.0, eps=1e-6, out=None, gathered=None, err=None):
    """ple_gather_project with the projection as int8 codes [L*ld, D] and fp16
    scales [L*ld, D/32]; returns (out f32 [S, L*ld], gathered int8 or None)."""
    lib = load()
    _dev(ids, torch.int32, "ids")
    _dev(table, torch.int8, "table")
    _dev(row_scale, torch.float32, "row_scale")
    _dev(proj_codes, torch.int8, "proj_codes")
    _dev(proj_scales, torch.float16, "proj_scales")
    _dev(hidden, torch.float16, "hidden")
    _dev(norm_w, torch.float32, "norm_w")
    S = ids.numel()
    V = table.shape[0]
    D = proj_codes.shape[1]
    if out is None:
        out = torch.empty((S, L * ld), dtype=torch.float32, device=ids.device)
    _dev(out, torch.float32, "out")
    _dev(gathered, torch.int8, "gathered")
    _dev(err, torch.int32, "err")
    _ple_sizes(S, V, L, ld, D, table, row_scale, hidden, norm_w, out, gathered)
    _numel(proj_codes, L * ld * D, "proj_codes")
    _numel(proj_scales, L * ld * D // 32, "proj_scales")
    _check(lib.ple_gather_project_q8(_ptr(ids), S, _ptr(table), _ptr(row_scale), V, L, ld, embed_scale,
                                     _ptr(proj_codes), _ptr(proj_scales), _ptr(hidden), D, _ptr(norm_w), eps,
                                     _ptr(out), _ptr(gathered), _ptr(err), _stream()), "ple_gather_project_q8")
    return out, gathered


def q4_gemm_chunk(codes, scales, X, Y=None):
    """Y [64, N] f32 = bf16 tiles of dequant(codes, scales) times bf16(X [64, K])."""
    lib = load()
    _dev(codes, torch.uint8, "codes")
    _dev(scales, torch.float16, "scales")
    _dev(X, torch.float16, "X")
    N, K = codes.shape[0], codes.shape[1] * 2
    M = X.shape[0]
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float32, device=X.device)
    _dev(Y, torch.float32, "Y")
    _numel(scales, N * K // 32, "scales")
    _numel(X, M * K, "X")
    _numel(Y, M * N, "Y")
    nws = lib.q4_workspace_bytes(Q4_OP_GEMM_CHUNK, N, K, M)
    ws = torch.empty(max(nws, 1), dtype=torch.uint8, device=X.device)
    _check(lib.q4_gemm_chunk(_ptr(codes), _ptr(scales), _ptr(X), _ptr(Y), M, N, K, _ptr(ws), nws,
                             _stream()), "q4_gemm_chunk")
    return Y


def q4_gemv_a8(codes, scales, x, act_scale, y=None):
    """w4a8 GEMV: y [N] f32 = act_scale * dequant(codes, scales) @ q, q the int8
    codes clamp(rint(x / act_scale), -128, 127) of x (fp16 [K])."""
    lib = load()
    _dev(codes, torch.uint8, "codes")
    _dev(scales, torch.float16, "scales")
    _dev(x, torch.float16, "x")
    N, K = codes.shape[0], codes.shape[1] * 2
    if y is None:
        y = torch.empty(N, dtype=torch.float32, device=x.device)
    _dev(y, torch.float32, "y")
    _numel(scales, N * K // 32, "scales")
    _numel(x, K, "x")
    _numel(y, N, "y")
    _check(lib.q4_gemv_a8(_ptr(codes), _ptr(scales), _ptr(x), float(act_scale), _ptr(y), N, K, _stream()),
           "q4_gemv_a8")
    return y


def q4_gemm_chunk_a8(codes, scales, X, act_scale, Y=None):
    """w4a8 S=64 chunk: Y [64, N] f32 = act_scale * (bf16 tiles of dequant(codes, scales)) @ Q.T,
    Q the int8 codes of X [64, K] under act_scale."""
    lib = load()
    _dev(codes, torch.uint8, "codes")
    _dev(scales, torch.float16, "scales")
    _dev(X, torch.float16, "X")
    N, K = codes.shape[0], codes.shape[1] * 2
    M = X.shape[0]
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float32, device=X.device)
    _dev(Y, torch.float32, "Y")
    _numel(scales, N * K // 32, "scales")
    _numel(X, M * K, "X")
    _numel(Y, M * N, "Y")
    nws = lib.q4_workspace_bytes(Q4_OP_GEMM_CHUNK, N, K, M)
    ws = torch.empty(max(nws, 1), dtype=torch.uint8, device=X.device)
    _check(lib.q4_gemm_chunk_a8(_ptr(codes), _ptr(scales), _ptr(X), float(act_scale), _ptr(Y), M, N, K,
                                _ptr(ws), nws, _stream()), "q4_gemm_chunk_a8")
    return Y


def q4_act_calibrate_a8(samples, out=None):
    """Min-max calibration of a w4a8 activation scale: a one-element f32 CUDA
    tensor holding max |x| / 127 over every value of ``samples`` (fp16, any
    shape, e.g. [128, K]), or 1 when all are zero."""
    lib = load()
    _dev(samples, torch.float16, "samples")
    if out is None:
        out = torch.empty(1, dtype=torch.float32, device=samples.device)
    _dev(out, torch.float32, "out")
    _numel(out, 1, "out")
    if samples.numel() < 1:
        raise Q4Error("samples must hold at least one value")
    _check(lib.q4_act_calibrate_a8(_ptr(samples), samples.numel(), _ptr(out), _stream()),
           "q4_act_calibrate_a8")
    return out


def q2_gemv(codes, scales, x, y=None):
    """INT2 per-row symmetric GEMV: y [N] f32 = scale[n] * sum_k (code - 2) x[k] (x fp16 [K])."""
    lib = load()
    _dev(codes, torch.uint8, "codes")
    _dev(scales, torch.float32, "scales")
    _dev(x, torch.float16, "x")
    N, K = codes.shape[0], codes.shape[1] * 4
    if y is None:
        y = torch.empty(N, dtype=torch.float32, device=x.device)
    _dev(y, torch.float32, "y")
    _numel(scales, N, "scales")
    _numel(x, K, "x")
    _numel(y, N, "y")
    _check(lib.q2_gemv(_ptr(codes), _ptr(scales), _ptr(x), _ptr(y), N, K, _stream()), "q2_gemv")
    return y


def kv_rope_steps(rot_dim, theta=10000.0, device="cuda", freqs=None):
    """Rotary steps of kv_append: int64 [rot_dim/2] (uint64 bits), the turns per
    position in units of 2^-64.  ``freqs``: the frequencies in radians per
    position (float64, any sequence of rot_dim/2; 0 leaves a pair as it is)
    instead of theta^(-2i/rot_dim)."""
    if freqs is None:
        freqs = [theta ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)]
    freqs = [float(f) for f in freqs]
    if len(freqs) != rot_dim // 2:
        raise Q4Error(f"freqs has {len(freqs)} entries; rot_dim implies {rot_dim // 2}")
    turns = [int(round(math.fmod(f / (2 * math.pi), 1.0) * 2.0 ** 64)) % 2 ** 64 for f in freqs]
    return torch.tensor([t - 2 ** 64 if t >= 2 ** 63 else t for t in turns], dtype=torch.int64, device=device)


# The calls of a decode step are short enough on the device for the host's time
# to count, so the checks of the functions below avoid what is slow in Python:
# helper calls per tensor and ctypes structures.

# Memory of torch's caching allocator on a stream, without a tensor around it: a workspace that
# lives for one call (1 us; a tensor made and dropped between launches costs 5).  The calls are
# private ones of torch's CUDA builds: where they are missing, a tensor is held instead.
_raw_alloc = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_alloc", None)
_raw_free = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_delete", None)
if _raw_alloc is None or _raw_free is None:
    _held = {}

    def _raw_alloc(size, stream):
        t = torch.empty(size, dtype=torch.uint8, device="cuda")   # on the current stream, which `stream` is
        _held[t.data_ptr()] = t
        return t.data_ptr()

    def _raw_free(ptr):
        del _held[ptr]


def _heads(t, dtype, heads, dim, T, name):
    """A [T, heads, dim] tensor whose heads and elements are contiguous; returns the token stride."""
    if t.dtype is not dtype or not _here(t):
        _dev(t[:0], dtype, name)   # names the fault
    if t.shape != (T, heads, dim):
        raise Q4Error(f"{name} has shape {tuple(t.shape)}; the sizes imply ({T}, {heads}, {dim})")
    st, sh, se = t.stride()
    if se != 1 or (sh != dim and heads > 1):
        raise Q4Error(f"{name}: the heads and elements of a token must be contiguous, its strides are {(st, sh, se)}")
    return st if T > 1 else heads * dim


_CACHE = struct.Struct("@5P7i4x")   # q4_kv_cache
assert _CACHE.size == ctypes.sizeof(q4_kv_cache)


def _kv_cache(k_cache, v_cache, block_table, cu_tokens, kv_lens):
    """The checked cache as (the bytes of its q4_kv_cache, its dtype, n_kv, head_dim)."""
    dtype = k_cache.dtype
    if dtype is not torch.float16 and dtype is not torch.bfloat16:
        raise Q4Error(f"k_cache must be torch.float16 or torch.bfloat16, got {dtype}")
    i32 = torch.int32
    if not (v_cache.dtype is dtype and block_table.dtype is i32 and cu_tokens.dtype is i32 and kv_lens.dtype is i32
            and _here(k_cache) and _here(v_cache) and _here(block_table) and _here(cu_tokens) and _here(kv_lens)
            and k_cache.is_contiguous() and v_cache.is_contiguous() and block_table.is_contiguous()
            and cu_tokens.is_contiguous() and kv_lens.is_contiguous()):
        for t, dt, name in ((k_cache, dtype, "k_cache"), (v_cache, dtype, "v_cache"), (block_table, i32, "block_table"),
                            (cu_tokens, i32, "cu_tokens"), (kv_lens, i32, "kv_lens")):
            _dev(t, dt, name)   # names the fault
    shape, tshape = k_cache.shape, block_table.shape
    if len(shape) != 4 or shape != v_cache.shape:
        raise Q4Error(f"k_cache {tuple(shape)} and v_cache {tuple(v_cache.shape)} must both be "
                      "[n_pages, n_kv, page_size, head_dim]")
    n = kv_lens.numel()
    if len(tshape) != 2 or tshape[0] != n:
        raise Q4Error(f"block_table has shape {tuple(tshape)}; kv_lens implies ({n}, max_pages)")
    if cu_tokens.numel() != n + 1:
        _numel(cu_tokens, n + 1, "cu_tokens")
    pages, heads, page, dim = shape
    return _CACHE.pack(k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(), cu_tokens.data_ptr(),
                       kv_lens.data_ptr(), _DTYPES[dtype], pages, heads, page, dim, n, tshape[1]), dtype, heads, dim


def kv_append(k, v, k_cache, v_cache, block_table, cu_tokens, kv_lens, steps=None, q=None, positions=None,
              interleaved=False, q_out=None, err=None):
    """Store the K and V rows of new tokens (k, v [T, n_kv, D], f32/f16/bf16, any
    token stride) in the paged cache [n_pages, n_kv, page_size, D], K turned by
    the rotary ``steps`` (kv_rope_steps; None: not turned); returns the turned
    queries q [T, n_q, D] in the cache's type, or None without q.  kv_lens
    counts the new tokens already; see include/q4w.h for the layout."""
    lib = load()
    cache, dtype, n_kv, D = _kv_cache(k_cache, v_cache, block_table, cu_tokens, kv_lens)
    T, kt = k.shape[0], k.dtype
    if kt not in _DTYPES:
        raise Q4Error(f"k must be float32, float16 or bfloat16, got {kt}")
    if T == 0:
        return None if q is None else torch.empty((0, q.shape[1], D), dtype=dtype, device=k.device)
    ks = _heads(k, kt, n_kv, D, T, "k")
    vs = _heads(v, kt, n_kv, D, T, "v")
    qs = n_q = 0
    q_ptr = out_ptr = None
    if q is not None:
        n_q = q.shape[1] if q.dim() == 3 else 0
        qs = _heads(q, kt, n_q, D, T, "q")
        if q_out is None:
            q_out = torch.empty((T, n_q, D), dtype=dtype, device=q.device)
        else:
            _dev(q_out, dtype, "q_out")
            _numel(q_out, T * n_q * D, "q_out")
        q_ptr, out_ptr = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise Q4Error("q_out without q")
    steps_ptr, rot = None, 0
    if steps is not None:
        _dev(steps, torch.int64, "steps")
        steps_ptr, rot = steps.data_ptr(), 2 * steps.numel()
    if positions is not None:
        _dev(positions, torch.int32, "positions")
        _numel(positions, T, "positions")
    if err is not None:
        _dev(err, torch.int32, "err")
    status = lib.kv_append(cache, T, k.data_ptr(), ks, v.data_ptr(), vs, _DTYPES[kt], q_ptr, qs, n_q, out_ptr,
                           steps_ptr, rot, 1 if interleaved else 0, _ptr(positions), _ptr(err), _stream())
    if status:
        _check(status, "kv_append")
    return q_out


_CACHE_Q8 = struct.Struct("@5P7i4x2P")   # q4_kv_cache_q8
assert _CACHE_Q8.size == ctypes.sizeof(q4_kv_cache_q8)


def _kv_cache_q8(k_cache, v_cache, block_table, cu_tokens, kv_lens, dtype):
    """The checked quantised cache as (the bytes of its q4_kv_cache_q8, n_kv, head_dim)."""
    if dtype is not torch.float16 and dtype is not torch.bfloat16:
        raise Q4Error(f"the queries' type must be torch.float16 or torch.bfloat16, got {dtype}")
    try:
        (kc, ks), (vc, vs) = k_cache, v_cache
    except (TypeError, ValueError):
        raise Q4Error("k_cache and v_cache must each be a pair of codes and scales") from None
    i32, i8, f16 = torch.int32, torch.int8, torch.float16
    if not (kc.dtype is i8 and vc.dtype is i8 and ks.dtype is f16 and vs.dtype is f16 and block_table.dtype is i32 and cu_tokens.dtype is i32
            and kv_lens.dtype is i32 and _here(kc) and _here(vc) and _here(ks) and _here(vs) and _here(block_table) and _here(cu_tokens)
            and _here(kv_lens) and kc.is_contiguous() and vc.is_contiguous() and ks.is_contiguous() and vs.is_contiguous()
            and block_table.is_contiguous() and cu_tokens.is_contiguous() and kv_lens.is_contiguous()):
        for t, dt, name in ((kc, i8, "k_cache's codes"), (ks, f16, "k_cache's scales"), (vc, i8, "v_cache's codes"), (vs, f16, "v_cache's scales"),
                            (block_table, i32, "block_table"), (cu_tokens, i32, "cu_tokens"), (kv_lens, i32, "kv_lens")):
            _dev(t, dt, name)   # names the fault
    shape, tshape = kc.shape, block_table.shape
    if len(shape) != 4 or shape != vc.shape:
        raise Q4Error(f"the codes of k_cache {tuple(shape)} and v_cache {tuple(vc.shape)} must both be "
                      "[n_pages, n_kv, page_size, head_dim]")
    pages, heads, page, dim = shape
    if ks.shape != (pages, heads, page, dim // 32) or ks.shape != vs.shape:
        raise Q4Error(f"the scales of k_cache {tuple(ks.shape)} and v_cache {tuple(vs.shape)} must both be {(pages, heads, page, dim // 32)}")
    n = kv_lens.numel()
    if len(tshape) != 2 or tshape[0] != n:
        raise Q4Error(f"block_table has shape {tuple(tshape)}; kv_lens implies ({n}, max_pages)")
    if cu_tokens.numel() != n + 1:
        _numel(cu_tokens, n + 1, "cu_tokens")
    return _CACHE_Q8.pack(kc.data_ptr(), vc.data_ptr(), block_table.data_ptr(), cu_tokens.data_ptr(), kv_lens.data_ptr(),
                          _DTYPES[dtype], pages, heads, page, dim, n, tshape[1], ks.data_ptr(), vs.data_ptr()), heads, dim


def _vector(t, dtype, n, name):
    """Pointer of an array of n values."""
    if t.dtype is not dtype or t.numel() != n or not t.is_contiguous() or not _here(t):
        _dev(t, dtype, name)
        _numel(t, n, name)
    return t.data_ptr()


def _append_normed(name, cache, dtype, n_kv, D, k, v, q_norm, k_norm, v_norm, eps, steps, q, positions, interleaved, q_out, err):
    """The rest of kv_append_norm and kv_append_q8 once their cache is checked."""
    T, kt = k.shape[0], k.dtype
    if kt not in _DTYPES:
        raise Q4Error(f"k must be float32, float16 or bfloat16, got {kt}")
    if T == 0:
        return None if q is None else torch.empty((0, q.shape[1], D), dtype=dtype, device=k.device)
    ks = _heads(k, kt, n_kv, D, T, "k")
    vs = _heads(v, kt, n_kv, D, T, "v")
    qs = n_q = 0
    q_ptr = out_ptr = None
    if q is not None:
        n_q = q.shape[1] if q.dim() == 3 else 0
        qs = _heads(q, kt, n_q, D, T, "q")
        if q_out is None:
            q_out = torch.empty((T, n_q, D), dtype=dtype, device=q.device)
        else:
            _dev(q_out, dtype, "q_out")
            _numel(q_out, T * n_q * D, "q_out")
        q_ptr, out_ptr = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise Q4Error("q_out without q")
    f32 = torch.float32
    qn = None if q_norm is None else _vector(q_norm, f32, D, "q_norm")
    kn = None if k_norm is None else _vector(k_norm, f32, D, "k_norm")
    vn = None if v_norm is None else _vector(v_norm, f32, D, "v_norm")
    steps_ptr, rot = None, 0
    if steps is not None:
        rot = 2 * steps.numel()
        steps_ptr = _vector(steps, torch.int64, rot // 2, "steps")
    at = None if positions is None else _vector(positions, torch.int32, T, "positions")
    flag = None if err is None else _vector(err, torch.int32, 1, "err")
    status = getattr(load(), name)(cache, T, k.data_ptr(), ks, v.data_ptr(), vs, _DTYPES[kt], q_ptr, qs, n_q, out_ptr, qn, kn, vn, eps,
                                   steps_ptr, rot, 1 if interleaved else 0, at, flag, _stream())
    if status:
        _check(status, name)
    return q_out


def kv_append_norm(k, v, k_cache, v_cache, block_table, cu_tokens, kv_lens, q_norm=None, k_norm=None, v_norm=None, eps=1e-6,
                   steps=None, q=None, positions=None, interleaved=False, q_out=None, err=None):
    """kv_append with an RMS norm of each head before the rotation, x / sqrt(mean(x^2)
    + eps) * w, by weights f32 [D]: q_norm of the queries, k_norm of the keys, v_norm of
    the values; None: no norm of that kind."""
    load()
    cache, dtype, n_kv, D = _kv_cache(k_cache, v_cache, block_table, cu_tokens, kv_lens)
    return _append_normed("kv_append_norm", cache, dtype, n_kv, D, k, v, q_norm, k_norm, v_norm, eps, steps, q, positions, interleaved, q_out, err)


def kv_append_q8(k, v, k_cache, v_cache, block_table, cu_tokens, kv_lens, q_norm=None, k_norm=None, v_norm=None, eps=1e-6,
                 steps=None, q=None, positions=None, interleaved=False, q_out=None, err=None, dtype=torch.float16):
    """kv_append_norm into a quantised cache: k_cache and v_cache are pairs of int8
    codes [n_pages, n_kv, page_size, D] and fp16 scales [n_pages, n_kv, page_size, D/32].
    dtype: of the turned queries that come back (float16 or bfloat16)."""
    load()
    cache, n_kv, D = _kv_cache_q8(k_cache, v_cache, block_table, cu_tokens, kv_lens, dtype)
    return _append_normed("kv_append_q8", cache, dtype, n_kv, D, k, v, q_norm, k_norm, v_norm, eps, steps, q, positions, interleaved, q_out, err)


def kv_read_q8(k_cache, v_cache, block_table, cu_tokens, kv_lens, T, dtype=torch.float16, k_out=None, v_out=None, err=None):
    """The K and V rows of T tokens out of a quantised cache, as numbers of dtype:
    (k, v) [T, n_kv, D], the rows that kv_append_q8 stored for the same cu_tokens and
    kv_lens.  Rows of padding tokens are left as they are (of new tensors: undefined)."""
    lib = load()
    cache, n_kv, D = _kv_cache_q8(k_cache, v_cache, block_table, cu_tokens, kv_lens, dtype)
    if k_out is None:
        k_out = torch.empty((T, n_kv, D), dtype=dtype, device=kv_lens.device)
    else:
        _dev(k_out, dtype, "k_out")
        _numel(k_out, T * n_kv * D, "k_out")
    if v_out is None:
        v_out = torch.empty((T, n_kv, D), dtype=dtype, device=kv_lens.device)
    else:
        _dev(v_out, dtype, "v_out")
        _numel(v_out, T * n_kv * D, "v_out")
    if err is not None:
        _dev(err, torch.int32, "err")
        _numel(err, 1, "err")
    if T:
        status = lib.kv_read_q8(cache, T, k_out.data_ptr(), v_out.data_ptr(), _ptr(err), _stream())
        if status:
            _check(status, "kv_read_q8")
    return k_out, v_out


@functools.lru_cache(maxsize=256)
def _attention_ws_bytes(max_q, n_q, n_kv, head_dim, device, T=None):
    with torch.cuda.device(device):   # the size goes by the current device's SMs
        lib = load()
        n = lib.kv_attention_ws_bytes(max_q, n_q, n_kv, head_dim) if T is None else lib.kv_attention_q8_ws_bytes(T, max_q, n_q, n_kv, head_dim)
    if n == 0:
        raise Q4Error(f"no workspace size for max_q={max_q}, n_q={n_q}, n_kv={n_kv}, head_dim={head_dim} on this device")
    return n


@functools.lru_cache(maxsize=256)
def _attention_q8_grows(max_q, n_q, n_kv, head_dim, device):
    """Whether the workspace of bf16 queries grows with their tokens."""
    sizes = (max_q, n_q, n_kv, head_dim, device)
    return _attention_ws_bytes(*sizes, 1) > _attention_ws_bytes(*sizes, 0)


def _attention_q8_ws_bytes(T, dtype, *sizes):
    # (T is no part of the key where the size does not go by it)
    return _attention_ws_bytes(*sizes, T if dtype is torch.bfloat16 and _attention_q8_grows(*sizes) else 0)


def _ws_device(device):
    device = torch.device(device)
    if device.type != "cuda":
        raise Q4Error(f"a workspace lies on a CUDA device, not on {device}")
    return device, torch.cuda.current_device() if device.index is None else device.index


def kv_attention_ws(max_q, n_q, n_kv, head_dim, device):
    """A workspace for kv_attention calls of these sizes that do not overlap."""
    device, index = _ws_device(device)
    return torch.empty(max(_attention_ws_bytes(max_q, n_q, n_kv, head_dim, index), 16), dtype=torch.uint8, device=device)


def kv_attention_q8_ws(T, max_q, n_q, n_kv, head_dim, device, dtype=torch.bfloat16):
    """A workspace for kv_attention_q8 calls of up to T tokens that do not overlap; dtype: of their
    queries (one for bfloat16 serves float16 too)."""
    device, index = _ws_device(device)
    if dtype is not torch.float16 and dtype is not torch.bfloat16:
        raise Q4Error(f"the queries' type must be torch.float16 or torch.bfloat16, got {dtype}")
    return torch.empty(max(_attention_q8_ws_bytes(T, dtype, max_q, n_q, n_kv, head_dim, index), 16), dtype=torch.uint8, device=device)


def kv_attention(q, k_cache, v_cache, block_table, cu_tokens, kv_lens, max_q=None, scale=None, window=0, out=None,
                 lse=None, ws=None, err=None):
    """Attention of the new tokens' queries q [T, n_q, D] over the paged cache
    that holds them: returns (out [T, n_q, D], lse).  max_q: an upper bound of
    the new tokens of a sequence (None: T); scale None: 1/sqrt(D); window: how
    many positions a token sees (0: all); lse: f32 [T, n_q] to fill, or None."""
    load()
    cache, dtype, n_kv, D = _kv_cache(k_cache, v_cache, block_table, cu_tokens, kv_lens)
    return _attention("kv_attention", cache, dtype, n_kv, D, q, max_q, scale, window, out, lse, ws, err)


def kv_attention_q8(q, k_cache, v_cache, block_table, cu_tokens, kv_lens, max_q=None, scale=None, window=0, out=None,
                    lse=None, ws=None, err=None):
    """kv_attention over a quantised cache: k_cache and v_cache are the pairs of codes
    and scales that kv_append_q8 fills; q and out are float16 or bfloat16."""
    load()
    cache, n_kv, D = _kv_cache_q8(k_cache, v_cache, block_table, cu_tokens, kv_lens, q.dtype)
    return _attention("kv_attention_q8", cache, q.dtype, n_kv, D, q, max_q, scale, window, out, lse, ws, err)


def _attention(name, cache, dtype, n_kv, D, q, max_q, scale, window, out, lse, ws, err):
    """The rest of kv_attention and kv_attention_q8 once their cache is checked."""
    if q.dim() != 3:
        raise Q4Error(f"q has shape {tuple(q.shape)}; [T, n_q, head_dim] is wanted")
    T, n_q, _ = q.shape
    if T == 0:
        return (torch.empty_like(q) if out is None else out), lse
    qs = _heads(q, dtype, n_q, D, T, "q")
    if out is None:
        out = torch.empty((T, n_q, D), dtype=dtype, device=q.device)
    else:
        _dev(out, dtype, "out")
        _numel(out, T * n_q * D, "out")
    lse_ptr = None
    if lse is not None:
        _dev(lse, torch.float32, "lse")
        _numel(lse, T * n_q, "lse")
        lse_ptr = lse.data_ptr()
    if err is not None:
        _dev(err, torch.int32, "err")
    if max_q is None:
        max_q = T
    if n_q < 1 or n_q % n_kv:
        raise Q4Error(f"n_q={n_q} must be a multiple of n_kv={n_kv}")
    stream, mine = _stream(), None
    if ws is None:
        sizes = (max_q, n_q, n_kv, D, q.get_device())
        size = _attention_q8_ws_bytes(T, dtype, *sizes) if name == "kv_attention_q8" else _attention_ws_bytes(*sizes)
        ws_ptr = mine = _raw_alloc(size, stream)
    else:
        _dev(ws, torch.uint8, "ws")
        ws_ptr, size = ws.data_ptr(), ws.numel()
    try:
        status = getattr(load(), name)(cache, T, max_q, q.data_ptr(), qs, n_q, D ** -0.5 if scale is None else scale, window,
                                       out.data_ptr(), lse_ptr, _ptr(err), ws_ptr, size, stream)
    finally:
        if mine is not None:
            _raw_free(mine)   # for what comes behind on the stream
    if status:
        _check(status, name)
    return out, lse


def _row_setting(t, dtype, b, name):
    """Pointer of a per-row array of b values, or None."""
    if t is None:
        return None
    if t.dtype is not dtype or not _here(t) or t.shape != (b,) or not t.is_contiguous():
        _dev(t, dtype, name)
        _numel(t, b, name)
    return t.data_ptr()


def logits_sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, tokens=None, logprobs=None):
    """One token per row of logits [b, V] (f32/f16/bf16, any row stride) from the
    random numbers u [b] in [0, 1): returns (tokens int32 [b], logprobs f32 [b]).
    temperature, top_p, min_p: f32 [b]; top_k: int32 [b]; None turns one off."""
    lib = load()
    dtype = logits.dtype
    if logits.dim() != 2 or dtype not in _DTYPES:
        raise Q4Error(f"logits must be [b, V] of float32, float16 or bfloat16, got {tuple(logits.shape)} {dtype}")
    b, V = logits.shape
    f32, i32 = torch.float32, torch.int32
    if tokens is None:
        tokens = torch.empty(b, dtype=i32, device=logits.device)
    if logprobs is None:
        logprobs = torch.empty(b, dtype=f32, device=logits.device)
    if b == 0:
        return tokens, logprobs
    if not _here(logits):
        _dev(logits[:0], dtype, "logits")   # names the fault
    rs, es = logits.stride()
    if V > 1 and es != 1:
        raise Q4Error(f"a row of logits must be contiguous, the strides are {(rs, es)}")
    status = lib.logits_sample(logits.data_ptr(), rs if b > 1 else V, _DTYPES[dtype], b, V,
                               _row_setting(u, f32, b, "u"), _row_setting(temperature, f32, b, "temperature"),
                               _row_setting(top_k, i32, b, "top_k"), _row_setting(top_p, f32, b, "top_p"),
                               _row_setting(min_p, f32, b, "min_p"), _row_setting(tokens, i32, b, "tokens"),
                               _row_setting(logprobs, f32, b, "logprobs"), _stream())
    if status:
        _check(status, "logits_sample")
    return tokens, logprobs


@functools.lru_cache(maxsize=256)
def _draft_ws_bytes(b, k, V):
    n = load().draft_verify_ws_bytes(b, k, V)
    if n == 0:
        raise Q4Error(f"b={b} must be in [1, 65535], k={k} in [0, 64], V={V} in [1, 1048576]")
    return n


def draft_verify_ws(b, k, V, device):
    """A workspace for draft_verify calls of these sizes that do not overlap."""
    return torch.empty(_draft_ws_bytes(b, k, V), dtype=torch.uint8, device=device)


def _logit_rows(t, dtype, shape, name):
    """(user stride, row stride) of logits [b, rows, V] whose rows are contiguous."""
    if t.dtype is not dtype or not _here(t):
        _dev(t[:0], dtype, name)   # names the fault
    if t.shape != shape:
        raise Q4Error(f"{name} has shape {tuple(t.shape)}; the sizes imply {tuple(shape)}")
    b, rows, V = shape
    us, rs, es = t.stride()
    if V > 1 and es != 1:
        raise Q4Error(f"{name}: a row of logits must be contiguous, the strides are {(us, rs, es)}")
    rs = rs if rows > 1 else V
    return us if b > 1 else rows * rs, rs


def draft_verify(logits, drafts, u, draft_logits=None, temperature=None, tokens=None, accepted=None, logprobs=None, ws=None):
    """Which of each user's drafted tokens stand, and the token behind them: logits
    [b, k+1, V] of the target (f32/f16/bf16, any strides of users and rows), drafts
    int32 [b, k] (-1: none from here on), random numbers u f32 [b, k+1] in [0, 1),
    draft_logits [b, k, V] that the drafts were drawn from (None: drafts without
    probabilities), temperature f32 [b] (None: 1; <= 0: greedy).  Returns (tokens int32
    [b, k+1], accepted int32 [b], logprobs f32 [b, k+1]): the accepted drafts, one more
    token, then -1; see include/q4w.h."""
    lib = load()
    dtype = logits.dtype
    if logits.dim() != 3 or dtype not in _DTYPES:
        raise Q4Error(f"logits must be [b, k + 1, V] of float32, float16 or bfloat16, got {tuple(logits.shape)} {dtype}")
    b, rows, V = logits.shape
    k, device = rows - 1, logits.device
    f32, i32 = torch.float32, torch.int32
    if tokens is None:
        tokens = torch.empty((b, rows), dtype=i32, device=device)
    if accepted is None:
        accepted = torch.empty(b, dtype=i32, device=device)
    if logprobs is None:
        logprobs = torch.empty((b, rows), dtype=f32, device=device)
    if b == 0:
        return tokens, accepted, logprobs
    us, rs = _logit_rows(logits, dtype, logits.shape, "logits")
    dus = drs = 0
    if draft_logits is not None:
        dus, drs = _logit_rows(draft_logits, dtype, (b, k, V), "draft_logits") if k else (0, 0)
    rk, rr = (b, k), (b, rows)
    if not (drafts.dtype is i32 and u.dtype is f32 and tokens.dtype is i32 and accepted.dtype is i32 and logprobs.dtype is f32
            and drafts.shape == rk and u.shape == rr and tokens.shape == rr and accepted.shape == (b,) and logprobs.shape == rr
            and _here(drafts) and _here(u) and _here(tokens) and _here(accepted) and _here(logprobs)
            and drafts.is_contiguous() and u.is_contiguous() and tokens.is_contiguous() and accepted.is_contiguous() and logprobs.is_contiguous()):
        for t, dt, shape, name in ((drafts, i32, rk, "drafts"), (u, f32, rr, "u"), (tokens, i32, rr, "tokens"),
                                   (accepted, i32, (b,), "accepted"), (logprobs, f32, rr, "logprobs")):
            _dev(t, dt, name)   # names the fault
            if t.shape != shape:
                raise Q4Error(f"{name} has shape {tuple(t.shape)}; the logits imply {shape}")
    temperature_ptr = _row_setting(temperature, f32, b, "temperature")
    stream, mine = _stream(), None
    if ws is None:
        size = _draft_ws_bytes(b, k, V)
        ws_ptr = mine = _raw_alloc(size, stream)
    else:
        _dev(ws, torch.uint8, "ws")
        ws_ptr, size = ws.data_ptr(), ws.numel()
    try:
        status = lib.draft_verify(logits.data_ptr(), us, rs, _DTYPES[dtype], b, k, V, drafts.data_ptr(), u.data_ptr(), _ptr(draft_logits), dus, drs,
                                  temperature_ptr, tokens.data_ptr(), accepted.data_ptr(), logprobs.data_ptr(), ws_ptr, size, stream)
    finally:
        if mine is not None:
            _raw_free(mine)   # for what comes behind on the stream
    if status:
        _check(status, "draft_verify")
    return tokens, accepted, logprobs


def q4_decode_pass_launches(descs, H):
    """Kernels one q4_decode_pass call over ``descs`` (make_layers output) launches."""
    n = load().q4_decode_pass_launches(descs, len(descs), H)
    if n < 0:
        _check(-n, "q4_decode_pass_launches")
    return n


class Q4DecodePlan:
    """A decode weight pass bound to fixed device buffers and captured once into
    a CUDA graph, so that a step is one graph launch.

    ``layers``: list of dicts name -> (codes, scales) as for q4_decode_pass.
    ``step_device()`` replays the graph on the current stream (h_in -> h_out,
    both device buffers).  ``step_host(h_pinned, out_pinned)`` copies one fp16
    hidden vector host->device, replays, and copies the result back.
    """

    def __init__(self, layers, H, eps=1e-6, device="cuda"):
        self.layers = layers
        self.H = H
        self.eps = eps
        self.descs = make_layers(layers, H)
        self.ws = torch.empty(decode_pass_ws_bytes(layers, H), dtype=torch.uint8, device=device)
        self.h_in = torch.zeros(H, dtype=torch.float16, device=device)
        self.h_out = torch.zeros(H, dtype=torch.float16, device=device)
        self.stream = torch.cuda.Stream(device=device)
        self.graph = None

    def run_eager(self):
        q4_decode_pass(self.layers, self.h_in, self.h_out, self.ws, self.eps, descs=self.descs)

    def capture(self):
        with torch.cuda.stream(self.stream):
            self.run_eager()                       # warm-up outside the capture
        torch.cuda.current_stream().wait_stream(self.stream)
        torch.cuda.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph, stream=self.stream):
            self.run_eager()
        torch.cuda.synchronize()
        return self

    def step_device(self):
        self.graph.replay()

    def step_host(self, h_pinned, out_pinned):
        self.h_in.copy_(h_pinned, non_blocking=True)
        self.graph.replay()
        out_pinned.copy_(self.h_out, non_blocking=True)
        torch.cuda.current_stream().synchronize()
        return out_pinned

    @property
    def launches_per_step(self):
        """Kernels one replay launches (the library's own count)."""
        return q4_decode_pass_launches(self.descs, self.H)
