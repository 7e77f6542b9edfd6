"""examples/decoder_layer.py: the attention half and the MoE half together.

A request's tokens go through the layer as one prompt, as two chunks (the
second over the context read back from the cache) and token by token; all
three attentions are checked against a plain 64-bit one of the same
projections (attn_util.attention's bounds; norm and rotation are in 64 bits
there, and q and k rounded once to bf16 here: 2^-8 of each, which moves a
score by at most 2^-7 sum_d |q_d k_d| scale and a weight by twice that)."""
import math
import os
import sys

import numpy as np
import pytest

from tests import attn_util as au

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import decoder_layer
    return decoder_layer


def _rotated(x, w, cs):
    import torch
    x = x.double()
    x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.double()
    h = cs.shape[1] // 2
    c, s = cs.double()[:x.shape[0], None, :h], cs.double()[:x.shape[0], None, h:]
    a, b = x[..., :h], x[..., h:2 * h]
    return torch.cat([a * c - b * s, b * c + a * s, x[..., 2 * h:]], -1)


def test_prompt_chunks_and_tokens_agree(gpu):
    import torch
    import quantized_moe_expert_align_gb300 as moe
    ex = _example()
    layer = ex.DecoderLayer(seed=3)
    n = [150, 33]
    x = au.randn(5, sum(n), layer.H)
    ends = np.cumsum(n)

    def requests():
        return ex.PagedRequests(moe.KVCache.empty(16, layer.Hkv, layer.D, 16, fp8=False), 2, 256)
    whole = layer.attend(x, requests(), n)
    r = requests()
    first = [100, 32]
    part = lambda a, b: torch.cat([x[0 + a[0]:b[0]], x[n[0] + a[1]:n[0] + b[1]]])  # noqa: E731
    c1 = layer.attend(part([0, 0], first), r, first)
    c2 = layer.attend(part(first, [149, 32]), r, [49, 0])
    one = layer.attend(part([149, 32], n), r, [1, 1])
    got = [torch.cat([c1[:100], c2[:49], one[:1]]), torch.cat([c1[100:132], one[1:]])]
    q, k, v = layer.project(x)
    for b, (s, e) in enumerate([(0, ends[0]), (ends[0], ends[1])]):
        qr = _rotated(q[s:e], layer.q_norm, layer.cos_sin)
        kr = _rotated(k[s:e], layer.k_norm, layer.cos_sin)
        m = e - s
        ref, _, tol, _ = au.attention(qr, kr, v[s:e], layer.D ** -0.5,
                                      torch.arange(m, device="cuda") + 1)
        G = layer.Hq // layer.Hkv
        for h in range(layer.Hq):
            mags = (qr[:, h].abs() @ kr[:, h // G].abs().T) * layer.D ** -0.5
            moved = 2 * 2.0 ** -7 * mags.amax(-1, keepdim=True)
            p = torch.softmax((qr[:, h] @ kr[:, h // G].T * layer.D ** -0.5).masked_fill(
                ~torch.ones(m, m, dtype=torch.bool, device="cuda").tril(), -math.inf), -1)
            tol[:, h] += moved * (p @ v[s:e, h // G].double().abs())
        au.check(whole[s:e], ref, tol, f"whole {b}")
        au.check(got[b], ref, tol, f"chunks and tokens {b}")


@pytest.mark.parametrize("fp8", [False, True])
def test_layer_runs_and_its_experts_match_the_oracle(gpu, fp8):
    import torch
    import oracle
    import quantized_moe_expert_align_gb300 as moe
    from tests import gpu_util as gu
    ex = _example()
    layer = ex.DecoderLayer(seed=4)
    r = ex.PagedRequests(moe.KVCache.empty(16, layer.Hkv, layer.D, 64, fp8=fp8), 3, 512)
    x = au.randn(6, 80, layer.H)
    y = layer(x, r, [50, 1, 29])
    for _ in range(3):
        y = layer(ex.rms_norm(y[-3:], layer.norm1), r, [1, 1, 1])
    assert torch.isfinite(y).all() and r.lens.tolist() == [53, 4, 32]
    # the MoE half on the attention half's output
    h = au.randn(7, 5, layer.H)
    got = layer.experts(h)
    z = ex.rms_norm(h, layer.norm2)
    logits = (z.float() @ layer.router.float().T).cpu().numpy()
    ids, w, _ = oracle.route(logits, layer.k)
    bits = lambda t: t.view(torch.int16).cpu().numpy().view(np.uint16)  # noqa: E731
    ref = oracle.forward(bits(z), ids, w, layer.q13.cpu().numpy(), bits(layer.s13), layer.q2.cpu().numpy(),
                         bits(layer.s2), layer.E, layer.H, layer.I)
    gu.parity(gu.bf16_dev_to_f64(got), ref, "experts")


def test_example_runs(gpu):
    import subprocess
    out = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "decoder_layer.py"), "--steps", "3"],
                         capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stdout + out.stderr
    assert "3 decode steps" in out.stdout
