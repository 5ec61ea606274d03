"""How the attention kernels count a call's work, compiled for the host: the keys and
steps of a tile, the steps of a sequence, a CTA's share of them.  Without a GPU."""
import ctypes
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "int4_q4_weight_gb300", "csrc")


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("steps")
    src = d / "steps.cpp"
    src.write_text(f'#include "{CSRC}/q4w_pages.h"\nextern "C" {{\n'
                   "long long tile_steps(int pos0, int n, int end, int w, int tokens, int box, int first, int stride) {\n"
                   "  return q4w::kv_tile_steps(pos0, n, end, w, tokens, box, first, stride); }\n"
                   "int share(long long total, long long share, long long first) { return q4w::kv_share_steps(total, share, first); }\n"
                   "void span(int pos0, int n, int end, int w, int tokens, int t, int box, int* out) {\n"
                   "  const q4w::KvSpan x = q4w::kv_span(pos0, n, end, w, tokens, t, box);\n"
                   "  out[0] = x.lo, out[1] = x.base, out[2] = x.end, out[3] = x.steps; }\n}\n")
    out = d / "steps.so"
    subprocess.run(["g++", "-O1", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-shared", "-fPIC", str(src), "-o", str(out)],
                   check=True)
    dll = ctypes.CDLL(str(out))
    dll.tile_steps.restype = ctypes.c_longlong
    dll.share.argtypes = [ctypes.c_longlong] * 3
    return dll


def span(pos0, n, end, window, tokens, t, box):
    """From the definition: the union of what the tile's tokens see."""
    toks = range(t * tokens, min((t + 1) * tokens, n))
    lo = max(0, pos0 + toks[0] - window + 1) if window else 0
    stop = min(end, pos0 + toks[-1] + 1)
    base = lo // box * box
    return lo, base, stop, max(1, -(-(stop - base) // 128))


def test_spans_and_steps(lib):
    rng = random.Random(1)
    got = (ctypes.c_int * 4)()
    for _ in range(3000):
        n, tokens, box = rng.randint(1, 300), rng.choice([2, 3, 16, 32, 256]), rng.choice([16, 32, 64])
        length = rng.choice([rng.randint(0, n), rng.randint(n, 3000), rng.randint(n, 2 ** 31 - 8192)])
        window = rng.choice([0, 1, 7, 512, 2 ** 31 - 1])
        end = min(length, rng.choice([length, 16 * rng.randint(1, 200)]))
        want = [span(length - n, n, end, window, tokens, t, box) for t in range(-(-n // tokens))]
        for t, w in enumerate(want):
            lib.span(length - n, n, end, window, tokens, t, box, got)
            assert tuple(got) == w
        total = sum(w[3] for w in want)
        assert lib.tile_steps(length - n, n, end, window, tokens, box, 0, 1) == total
        assert sum(lib.tile_steps(length - n, n, end, window, tokens, box, x, 32) for x in range(32)) == total


def test_steps_of_a_sequence_pass_32_bits(lib):
    """128 heads on one KV head are one token a tile: 65536 new tokens over 8.45 million
    positions are more than 2^31 steps."""
    n, length = 65536, 8_454_144
    want = sum(-(-(length - n + 2 * t + 2) // 128) for t in range(n // 2))
    assert want > 2 ** 31
    assert lib.tile_steps(length - n, n, length, 0, 2, 64, 0, 1) == want
    assert sum(lib.tile_steps(length - n, n, length, 0, 2, 64, x, 32) for x in range(32)) == want


def test_shares(lib):
    for total in (0, 1, 75, 76, 77, 2_155_888_640, 2 ** 31 * 76):
        each = -(-total // 76)
        parts = [lib.share(total, each, each * c) for c in range(76)]
        if each > 2 ** 31 - 1:
            assert parts == [-1] * 76          # said, not cut off
        else:
            assert min(parts) >= 0 and sum(parts) == total
