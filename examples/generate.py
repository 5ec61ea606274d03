"""Generating tokens on q4_0 weights: a small decoder of random weights whose
step is one CUDA graph of the library's calls.

    python examples/generate.py [--layers 4] [--tokens 200] [--temperature 0.8]

Per layer (E2B-shaped: 8 query heads over 1 KV head, heads of 256 with a sliding
window on most layers and of 512 on every fourth): RMSNorm and the q, k, v
projections (q4_gemv_stage), the new key and value into the paged cache with the
rotary rotation and the query rotated (kv_append), attention over the cache
(kv_attention), output projection, gated MLP.  Then the LM head's softcapped
logits (lmhead_softcap_argmax) and the next token (logits_sample) from a given
random number; its embedding is the next step's input.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import int4_q4_weight_gb300 as q4w          # noqa: E402
from int4_q4_weight_gb300 import synth      # noqa: E402

N_Q, PAGE, WINDOW = 8, 16, 512


class Decoder:
    """A decoder of random q4_0 weights for one sequence, with its paged caches."""

    def __init__(self, layers=4, H=1536, mlp=6144, V=32768, max_len=2048, seed=1, device="cuda"):
        self.H, self.V, self.max_len, self.device = H, V, max_len, device
        q4 = lambda n, k, *tag: q4w.q4_quantize(synth.normal((n, k), 0.03, synth.sub_seed(seed, *tag), device))   # noqa: E731
        pages = -(-max_len // PAGE)
        self.block_table = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)[None].to(device)
        self.cu = torch.tensor([0, 1], dtype=torch.int32, device=device)
        self.kv_lens = torch.zeros(1, dtype=torch.int32, device=device)
        self.layers = []
        for i in range(layers):
            D = 512 if i % 4 == 3 else 256
            cache = lambda: torch.zeros((pages, 1, PAGE, D), dtype=torch.float16, device=device)   # noqa: B023, E731
            self.layers.append(dict(
                D=D, window=0 if D == 512 else WINDOW, steps=q4w.kv_rope_steps(D, 1e6 if D == 512 else 1e4, device),
                kc=cache(), vc=cache(), q=q4(N_Q * D, H, i, "q"), k=q4(D, H, i, "k"), v=q4(D, H, i, "v"), o=q4(H, N_Q * D, i, "o"),
                g=q4(mlp, H, i, "g"), u=q4(mlp, H, i, "u"), d=q4(H, mlp, i, "d"),
                qkv32=[torch.empty(n, dtype=torch.float32, device=device) for n in (N_Q * D, D, D)],
                q16=torch.empty((1, N_Q, D), dtype=torch.float16, device=device),
                att=torch.empty((1, N_Q, D), dtype=torch.float16, device=device),
                ws=q4w.kv_attention_ws(1, N_Q, 1, D, device)))
        self.embed = synth.normal((V, H), 1.0, synth.sub_seed(seed, "embed"), device).to(torch.float16)
        self.head = q4(V, H, "head")
        f32 = lambda *s: torch.empty(s, dtype=torch.float32, device=device)   # noqa: E731
        f16 = lambda *s: torch.empty(s, dtype=torch.float16, device=device)   # noqa: E731
        self.h, self.o32, self.m16, self.y32, self.hf = f16(H), f32(H), f16(mlp), f32(H), f16(1, H)
        self.logits, self.head_ws = f32(1, V), q4w.lmhead_ws(V, H, 1, device)
        self.idx, self.top1, self.top2 = torch.empty(1, dtype=torch.int32, device=device), f32(1), f32(1)
        # the step's inputs and outputs
        self.token = torch.zeros(1, dtype=torch.int32, device=device)
        self.u, self.logprob = torch.zeros(1, device=device), f32(1)
        self.settings = dict(temperature=torch.ones(1, device=device), top_k=torch.full((1,), 64, dtype=torch.int32, device=device),
                             top_p=torch.full((1,), 0.95, device=device), min_p=torch.zeros(1, device=device))

    def step(self):
        """One token: self.token in, the next one out (all on the current stream)."""
        self.kv_lens += 1
        torch.index_select(self.embed, 0, self.token, out=self.hf)
        x, mode = self.hf[0], q4w.Q4_IN_RMS_F16
        for L in self.layers:
            D, (q32, k32, v32) = L["D"], L["qkv32"]
            q4w.q4_gemv_stage([L["q"], L["k"], L["v"]], x, mode, out32=[q32, k32, v32])
            tables = (L["kc"], L["vc"], self.block_table, self.cu, self.kv_lens)
            q4w.kv_append(k32.view(1, 1, D), v32.view(1, 1, D), *tables, steps=L["steps"], q=q32.view(1, N_Q, D), q_out=L["q16"])
            q4w.kv_attention(L["q16"], *tables, max_q=1, window=L["window"], out=L["att"], ws=L["ws"])
            q4w.q4_gemv_stage([L["o"]], L["att"].view(-1), q4w.Q4_IN_F16, out32=[self.o32])
            q4w.q4_gemv_stage([L["g"], L["u"]], self.o32, q4w.Q4_IN_RMS_F32, pair=True, out16=[self.m16, None])
            q4w.q4_gemv_stage([L["d"]], self.m16, q4w.Q4_IN_F16, out32=[self.y32])
            x, mode = self.y32, q4w.Q4_IN_RMS_F32
        q4w.q4_rmsnorm_f16(self.y32, out=self.h)
        q4w.lmhead_softcap_argmax(*self.head, self.h.view(1, -1), ws=self.head_ws, idx=self.idx, top1=self.top1, top2=self.top2,
                                  logits=self.logits)
        q4w.logits_sample(self.logits, self.u, **self.settings, tokens=self.token, logprobs=self.logprob)

    def capture(self):
        """The step as a CUDA graph (call once; generate() then replays it)."""
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.step()
        torch.cuda.current_stream().wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.step()
        return self

    def generate(self, first, n, randoms, graph=True):
        """n tokens after `first`, from the random numbers given: (tokens, log probabilities)."""
        if n > self.max_len:
            raise ValueError(f"{n} tokens do not fit a cache of {self.max_len}")
        self.kv_lens.zero_()
        self.token.fill_(first)
        tokens = torch.empty(n, dtype=torch.int32, device=self.device)
        logprobs = torch.empty(n, device=self.device)
        for i in range(n):
            self.u.copy_(randoms[i:i + 1])
            if graph:
                self.graph.replay()
            else:
                self.step()
            tokens[i:i + 1].copy_(self.token)
            logprobs[i:i + 1].copy_(self.logprob)
        return tokens, logprobs


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=200)
    ap.add_argument("--temperature", type=float, default=0.8)
    a = ap.parse_args()
    dec = Decoder(layers=a.layers, max_len=a.tokens + 16)
    dec.settings["temperature"].fill_(a.temperature)
    dec.capture()
    randoms = torch.rand(a.tokens, generator=torch.Generator(device="cuda").manual_seed(0), device="cuda")
    dec.generate(1, 8, randoms)
    torch.cuda.synchronize()
    t = time.perf_counter()
    tokens, logprobs = dec.generate(1, a.tokens, randoms)
    q4w.q4_device_status()
    t = time.perf_counter() - t
    print(f"{a.tokens} tokens in {t * 1e3:.1f} ms ({a.tokens / t:.0f} tokens/s), mean log probability {logprobs.mean().item():.3f}")
    print("first tokens:", tokens[:12].tolist())


if __name__ == "__main__":
    main()
