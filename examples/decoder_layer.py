"""One decoder layer of an LLM server on the library's kernels, run the way a
server runs it: a batch of prompts packed into one call, then tokens one by
one for all requests over a paged cache, with requests of different lengths.

    python examples/decoder_layer.py [--steps N] [--fp8 0|1]

The attention half is qk_rope_append (per-head norms, rotation, cache write),
attn_prefill and attn_decode; the MoE half is forward_routed (router, expert
GEMMs on INT4 weights, combine).  The dense projections and the layer's two
RMS norms are plain torch calls.  Weights are random.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_moe_expert_align_gb300 as moe  # noqa: E402


def rms_norm(x, w, eps=1e-6):
    y = x.float()
    return (y * torch.rsqrt(y.pow(2).mean(-1, keepdim=True) + eps) * w.float()).to(x.dtype)


class PagedRequests:
    """The pages of a batch of requests: which page holds which tokens."""

    def __init__(self, cache, max_requests, max_len, device="cuda"):
        self.cache = cache
        self.page = cache.page_size
        self.free = list(range(cache.num_pages))
        self.table = torch.zeros(max_requests, -(-max_len // self.page), dtype=torch.int32)
        self.lens = torch.zeros(max_requests, dtype=torch.int32)
        self.device = device

    def extend(self, new_lens):
        """Gives request b `new_lens[b]` more tokens; returns their (positions,
        slots), request by request, on the device."""
        pos, slots = [], []
        for b, n in enumerate(new_lens):
            for t in range(int(self.lens[b]), int(self.lens[b]) + int(n)):
                if t % self.page == 0:
                    self.table[b, t // self.page] = self.free.pop()
                pos.append(t)
                slots.append(int(self.table[b, t // self.page]) * self.page + t % self.page)
            self.lens[b] += int(n)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=self.device)  # noqa: E731
        return i32(pos), i32(slots)

    def on_device(self):
        return self.table.to(self.device), self.lens.to(self.device)


class DecoderLayer:
    def __init__(self, H=512, Hq=8, Hkv=2, D=64, E=8, I=256, k=2, max_len=4096, rot=None, seed=0,
                 device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.H, self.Hq, self.Hkv, self.D, self.E, self.I, self.k = H, Hq, Hkv, D, E, I, k
        def rand(*shape, scale=1.0):
            return (torch.randn(*shape, generator=g, device=device) * scale).bfloat16()
        self.wqkv = rand((Hq + 2 * Hkv) * D, H, scale=H ** -0.5)
        self.wo = rand(H, Hq * D, scale=(Hq * D) ** -0.5)
        self.norm1, self.norm2 = 1 + rand(H, scale=0.1), 1 + rand(H, scale=0.1)
        self.q_norm, self.k_norm = 1 + rand(D, scale=0.1), 1 + rand(D, scale=0.1)
        self.router = rand(E, H, scale=H ** -0.5)
        self.cos_sin = moe.rope_table(max_len, D if rot is None else rot, device=device)

        def codes(N, K):
            q = torch.randint(0, 256, (E, N, K // 2), generator=g, device=device, dtype=torch.uint8)
            s = torch.rand(E, N, K // 32, generator=g, device=device) * 0.01 + 0.002
            return q, s.bfloat16()
        self.q13, self.s13 = codes(2 * I, H)
        self.q2, self.s2 = codes(H, I)
        self.w13 = moe.prepack(moe.MOE_PACK_W13, self.q13, self.s13)
        self.w2 = moe.prepack(moe.MOE_PACK_W2, self.q2, self.s2)

    def project(self, x):
        qkv = rms_norm(x, self.norm1) @ self.wqkv.T
        qkv = qkv.view(x.shape[0], self.Hq + 2 * self.Hkv, self.D)
        return qkv[:, :self.Hq], qkv[:, self.Hq:self.Hq + self.Hkv], qkv[:, self.Hq + self.Hkv:]

    def attend(self, x, requests, new_lens):
        """Attention of each request's new tokens (rows of x, request by
        request), which are appended to the cache.  Returns [T][Hq][D]."""
        before = requests.lens.clone()
        pos, slots = requests.extend(new_lens)
        q, k, v = self.project(x)
        whole = all(int(n) > 0 for n in before) and all(int(n) == 1 for n in new_lens)
        if whole:  # one token each: attention over the cache
            q = moe.qk_rope_append(q, k, v, self.cos_sin, pos, requests.cache, slots,
                                   q_norm=self.q_norm, k_norm=self.k_norm)
            table, lens = requests.on_device()
            return moe.attn_decode(q, requests.cache, table, lens)
        cu_q = torch.tensor([0] + list(torch.tensor(new_lens).cumsum(0)), dtype=torch.int32, device=x.device)
        q, k = moe.qk_rope_append(q, k, v, self.cos_sin, pos, requests.cache, slots, q_norm=self.q_norm,
                                  k_norm=self.k_norm, k_out=True)
        if int(before.sum()) == 0:  # first prompts: keys and values as they are
            return moe.attn_prefill(q, k, v, cu_q, cu_q)
        # later chunks of prompts: the whole context is read back from the cache
        table, lens = requests.on_device()
        total = int(requests.lens.sum())
        cu_k = torch.cat([torch.zeros(1, dtype=torch.int32, device=x.device),
                          lens.cumsum(0).to(torch.int32)])
        k, v = moe.kv_gather(requests.cache, table, cu_k, total)
        return moe.attn_prefill(q, k, v, cu_q, cu_k)

    def experts(self, h):
        y = rms_norm(h, self.norm2)
        logits = y.float() @ self.router.float().T
        out, _, _ = moe.forward_routed(y, logits, self.k, self.w13, self.w2, self.E, self.I)
        return out

    def __call__(self, x, requests, new_lens):
        a = self.attend(x, requests, new_lens)
        h = x + a.reshape(x.shape[0], -1) @ self.wo.T
        return h + self.experts(h)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--fp8", type=int, default=1)
    args = ap.parse_args()
    layer = DecoderLayer()
    prompts = [300, 17, 1024, 1]
    cache = moe.KVCache.empty(num_pages=64, Hkv=layer.Hkv, D=layer.D, page_size=64, fp8=bool(args.fp8))
    requests = PagedRequests(cache, len(prompts), 2048)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(sum(prompts), layer.H, generator=g, device="cuda").bfloat16()
    y = layer(x, requests, prompts)
    last = y[torch.tensor(prompts).cumsum(0) - 1]
    print(f"prompts of {prompts} tokens: output {tuple(y.shape)}, rms {y.float().pow(2).mean().sqrt().item():.3f}")
    for step in range(args.steps):
        last = layer(rms_norm(last, layer.norm1), requests, [1] * len(prompts))
    torch.cuda.synchronize()
    print(f"{args.steps} decode steps: lengths {requests.lens.tolist()}, rms {last.float().pow(2).mean().sqrt().item():.3f}")


if __name__ == "__main__":
    main()
