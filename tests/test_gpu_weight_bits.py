"""Softmax weights with 24 bits where fp32 is written: tree attention and the decode with totals.

Two tokens, scores 0 and -1, V zero at the first: out = V w / (1 + w), w = exp(-scale), for a w that a high and a low
bf16 part leave 0.7 * 2^-18 short.  What else can go wrong, relative to out:
  * w itself, off by 2^-21 (the base-2 exponential's 2 ulp, its argument), enters by 1 / (1 + w) < 2/3;
  * the products of the parts with V are exact, their sum takes two additions that may drop 2^-23 each;
  * the sum 1 + w, its reciprocal and the last product take 2^-24, 2^-23 and 2^-24.
Together below 2^-21 * 2/3 + 2^-22 + 2^-22 = 8e-7; without the third part the result is off by more than 2e-6."""
import numpy as np
import pytest
import torch

from gpu_util import DEV
from paged_kv_gqa_06_gb300 import binding

TOL = 8e-7


def bf16(x):
    return torch.tensor(x, dtype=torch.float64).float().to(torch.bfloat16).double().item()


def two_parts(w):
    hi = bf16(w)
    return hi + bf16(w - hi)


def find_scale():
    """A scale whose weight the two parts leave short by 0.6 to 0.8 of the most they can, also 4 ulp away."""
    for i in range(1, 4000):
        scale = float(np.float32(0.3 + i * 1e-4))
        w = np.exp(-scale)
        if all(0.6 * 2.0 ** -18 < (x - two_parts(x)) / x < 0.8 * 2.0 ** -18
               for x in (float(np.float32(w)) + u * 2.0 ** -24 for u in range(-4, 5))):
            return scale
    raise AssertionError("no such scale")


def reference(v, scale):
    w = np.exp(-scale)
    return v.double() * (w / (1 + w))


def test_the_case_tells_two_parts_from_three():
    scale = find_scale()
    w = np.exp(-scale)
    short = abs(two_parts(w) / w - 1)
    assert short > 2.5 * TOL
    third = bf16(w - two_parts(w))
    assert abs((two_parts(w) + third) / w - 1) < 2.0 ** -24


def inputs(Hkv, D, tokens, gen):
    k = torch.zeros(1, Hkv, 16, D, dtype=torch.bfloat16)
    k[0, :, 1, 0] = -1.0
    v = torch.zeros_like(k)
    v[0, :, 1] = ((4 + 4 * torch.rand(Hkv, D, generator=gen)) * torch.where(torch.rand(Hkv, D, generator=gen) < 0.5, -1, 1)).to(torch.bfloat16)
    k[0, :, 2:tokens] = torch.randn(Hkv, tokens - 2, D, generator=gen).to(torch.bfloat16)
    return k.to(DEV), v.to(DEV)


def ones(rows, heads, D):
    q = torch.zeros(rows, heads, D, dtype=torch.bfloat16, device=DEV)
    q[:, :, 0] = 1.0
    return q


def check(out, v, G, scale):
    """out [rows, Hq, D]: every row the same."""
    ref = reference(v[0, :, 1], scale).repeat_interleave(G, dim=0)
    off = ((out.double() - ref) / ref).abs().max().item()
    print(f"relative error {off:.2e}")
    assert off <= TOL


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("nodes,G", [(2, 4), (16, 1), (16, 8)], ids=["64_rows", "64_rows_G1", "128_rows"])
def test_tree_weights_have_24_bits(nodes, G, D):
    """At most 64 rows a sequence: the parts in a tile's halves; more: all three in a row."""
    scale = find_scale()
    k, v = inputs(2, D, nodes, torch.Generator().manual_seed(D + G))
    out = torch.empty(nodes, 2 * G, D, device=DEV)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    binding.forge_paged_tree_attention(ones(nodes, 2 * G, D), k, v, i32([[0]]), i32([nodes]), i32([0, nodes]),
                                       torch.full((nodes, 1), 3, dtype=torch.int64, device=DEV), scale, out)
    assert binding.forge_paged_get_device_error() == 0
    check(out, v, G, scale)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_decode_with_totals_weights_have_24_bits(G, D):
    scale = find_scale()
    k, v = inputs(2, D, 2, torch.Generator().manual_seed(D + G))
    out, totals = torch.empty(1, 2 * G, D, device=DEV), torch.zeros(1, 2, 4, device=DEV)
    binding.forge_paged_gqa_decode_weights(ones(1, 2 * G, D), k, v, torch.zeros(1, 1, dtype=torch.int32, device=DEV),
                                           torch.tensor([2], dtype=torch.int32, device=DEV), scale, out, totals)
    assert binding.forge_paged_get_device_error() == 0
    check(out, v, G, scale)
