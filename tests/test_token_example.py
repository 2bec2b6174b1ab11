"""The example that runs the deformable layer and the token operators together,
and sizes whose offsets pass 32 bits."""
import importlib.util
import math
import os

import pytest
import torch

import modulated_deformable_convolution_gb300 as mdcn

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("feature_map_attention", os.path.join(ROOT, "examples", "feature_map_attention.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_example_trains_and_reads(example):
    losses, tokens = example.main(steps=6)
    assert losses[-1] < losses[0] and tokens.shape == (2, 4, example.CHANNELS) and torch.isfinite(tokens).all()


def test_example_gradients(example):
    """The chain's gradients in bfloat16 against torch's automatic ones of the
    same chain in 64 bits, from the convolution's output on. Every step of the
    chain rounds to 8 bits, five in a row on the way to the first weights: 5 x
    2^-8 of a gradient's norm in the worst case of errors that add up."""
    m = example.Model(seed=1)
    s = m.forward()
    g = m.backward(s)
    p = {n: t.double().requires_grad_() for n, t in m.p.items() if n != "conv"}
    qkv = (s["tokens"].double() @ p["qkv"]).view(len(s["tokens"]), -1, example.DIM)
    q, k, v = qkv.split([example.Q_HEADS, example.K_HEADS, example.K_HEADS], 1)

    def turned(x, w):
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
        t = torch.cat([m.positions[:, a:a + 1].double() * m.freq[16 * a:16 * a + 16].double() for a in range(2)], 1)[:, None]
        lo, hi = x[..., :32], x[..., 32:]
        return torch.cat([lo * t.cos() - hi * t.sin(), hi * t.cos() + lo * t.sin()], -1)

    q, k = turned(q, p["q_norm"]), turned(k, p["k_norm"])
    outs, at = [], 0
    for h, w in example.SIZES:
        n = h * w
        qi, ki, vi = (x[at:at + n].transpose(0, 1) for x in (q, k, v))
        ki, vi = ki.repeat_interleave(2, 0), vi.repeat_interleave(2, 0)
        outs.append((torch.softmax(qi @ ki.transpose(1, 2) * example.DIM**-0.5, -1) @ vi).transpose(0, 1))
        at += n
    y = torch.cat(outs).flatten(1) @ p["proj"]
    # from the library's own y, as the chain's first gradient is
    gy = (s["y"].double() - m.target.double()) / y.numel()
    (y * gy).sum().backward()
    for n, t in p.items():
        off = (g[n].double() - t.grad).norm() / t.grad.norm()
        assert off < 5 * 2.0**-8, (n, float(off))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_offsets_beyond_32_bits(dtype):
    """A cache of more than 2^31 elements: the last sequence lies past the
    2^31st, and gets what it gets from a cache of its own."""
    hk, d, n = 16, 128, 700
    tokens = 2**31 // (hk * d) + 1000
    kv = torch.zeros(tokens, hk, d, dtype=dtype, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    kv[-n:] = torch.randn(n, hk, d, generator=g, device="cuda").to(dtype)
    q = torch.randn(2, hk, d, generator=g, device="cuda").to(dtype)
    qs = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    ks = torch.tensor([0, tokens - n, tokens], dtype=torch.int32, device="cuda")
    used = torch.tensor([3, n], dtype=torch.int32, device="cuda")
    out, lse = mdcn.attention(q, kv, kv, qs, ks, k_lengths=used, causal=True)
    own, olse = mdcn.attention(q[1:], kv[-n:].clone(), kv[-n:].clone(), mdcn.sequence_starts([1]), mdcn.sequence_starts([n]), k_lengths=used[1:].clone(), causal=True)
    # the keys may be shared out differently: fp32 sums in another order, then one rounding
    u = {torch.bfloat16: 2.0**-8, torch.float32: 2.0**-20}[dtype]
    assert ((out[1:].double() - own.double()).abs() <= 2 * u * own.double().abs().amax()).all()
    assert ((lse[:, 1:] - olse).abs() <= 2.0**-20 * olse.abs()).all()
    # keys of zeros: every value alike
    assert (out[0] == 0).all()
    pos = torch.zeros(tokens, 1, dtype=torch.int32, device="cuda")
    yq, _ = mdcn.rotary(kv, None, pos, mdcn.rotary_frequencies((64,)), (64,), q_out=kv)  # angle 0: unchanged
    assert torch.equal(mdcn.attention(q[1:], yq[-n:], yq[-n:], mdcn.sequence_starts([1]), mdcn.sequence_starts([n]), k_lengths=used[1:].clone(), causal=True)[0], own)


def test_an_item_longer_than_a_wait_may_be():
    """One query against 400 million keys: its gradient is one work item of some
    three seconds, and the roles that have nothing to do in it (the one that
    clears the last tile's tail, the one that gets items) wait that long. All
    keys score 0, so that every probability is 1 / n; 1000 of them, the first
    and the last among these, have a value and a key of ones."""
    n, d, step = 400_000_005, 8, 400_000
    ones = torch.cat([torch.arange(0, n, step, device="cuda")[:999], torch.tensor([n - 1], device="cuda")])
    k = torch.zeros(n, 1, d, dtype=torch.bfloat16, device="cuda")
    k[ones] = 1
    q, g = torch.zeros(1, 1, d, dtype=k.dtype, device="cuda"), torch.ones(1, 1, d, dtype=k.dtype, device="cuda")
    out, lse = torch.zeros_like(q), torch.full((1, 1), math.log(n), device="cuda")
    qs, ks = mdcn.sequence_starts([1]), mdcn.sequence_starts([n])
    gq, gk, gv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(k)
    ws = torch.empty(mdcn.mdcn_attention_backward_workspace_size(g, q, k, k, out, lse, qs, ks, gq, gk, gv), dtype=torch.uint8, device="cuda")
    mdcn.mdcn_attention_backward(g, q, k, k, out, lse, qs, ks, gq, gk, gv, ws)
    assert mdcn.mdcn_query_status(ws) == (0, 0)
    # p is rounded once, ds once, each result once; lse, near 20, is off by 2^-20 in fp32
    p, tol = 1 / n, 4 * 2.0**-8
    assert ((gq.double() / (1000 * p * d * d**-0.5) - 1).abs() <= tol).all()
    assert ((gv.float().amin() / p - 1).abs() <= tol) and ((gv.float().amax() / p - 1).abs() <= tol)
    assert (gk == 0).all()
