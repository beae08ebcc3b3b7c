"""forge_paged_tree_attention where one CTA sums over many thousand tokens: batches of so many long sequences that the
even split of the work leaves whole items, and more, to each CTA.

The number of products in one fp32 accumulation is bounded; the tests hold the constructed case of the largest
accumulation error to a bound that does not grow with the context, and the sums' joining to the plain 64-bit form: moving maxima, rows that see tokens of some accumulations only, infinities."""
import numpy as np
import pytest
import torch

import plain_select as plain
from gpu_util import DEV, TOL
from paged_kv_gqa_06_gb300 import binding
from paged_kv_gqa_06_gb300.workloads import STRESS_GAP

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.init()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def shared_pool(blocks, B, gen):
    """Tables of B sequences over the same blocks, each in an order of its own."""
    return torch.stack([torch.randperm(blocks, generator=gen) for _ in range(B)]).to(torch.int32).to(DEV)


# rows of an item: the halves of one tile, one tile, two tiles
@pytest.mark.parametrize("nodes,out_dtype", [(2, torch.bfloat16), (24, torch.bfloat16), (64, torch.bfloat16),
                                             (2, torch.float32), (24, torch.float32)])
def test_accumulation_error_does_not_grow_with_the_context(nodes, out_dtype):
    """Weights just above 0.5, every V of a dim of one sign and in [7, 8), 16384 tokens for each of 320 items on some
    300 CTAs: every addition of the P V products drops bits in the same direction.

    A sum starts anew after 384 products of 16 tokens at most for fp32 out; an addition drops less than 2^-23 of a sum
    that grows evenly, so 384 * 2^-24 of the result (|out| < 8: 1.83e-4).  2e-4 leaves the rest of the arithmetic a
    tenth of that.  bf16: the repository's bound."""
    B, Hkv, G, D, L = 40, 8, 4, 128, 16384
    gen = torch.Generator().manual_seed(nodes)
    k = torch.randn(L // 16, Hkv, 16, D, generator=gen)
    k[..., :G] = 0.0
    k[:, :, 0, :G] = STRESS_GAP
    sign = torch.where(torch.rand(Hkv, 1, D, generator=gen) < 0.5, -1.0, 1.0)
    v = sign * (7.0 + 0.97 * torch.rand(L // 16, Hkv, 16, D, generator=gen))
    k, v = k.to(torch.bfloat16).to(DEV), v.to(torch.bfloat16).to(DEV)
    T = B * nodes
    q = torch.zeros(T, Hkv * G, D, dtype=torch.bfloat16, device=DEV)
    for h in range(Hkv * G):
        q[:, h, h % G] = 1.0
    out = torch.full((T, Hkv * G, D), 7.25, dtype=out_dtype, device=DEV)
    binding.forge_paged_tree_attention(q, k, v, shared_pool(L // 16, B, gen), i32([L] * B), i32([nodes * b for b in range(B + 1)]),
                                       torch.full((T, 1), -1, dtype=torch.int64, device=DEV), D ** -0.5, out)
    assert binding.forge_paged_get_device_error() == 0
    kk, vv = [x.double().transpose(0, 1).reshape(Hkv, L, D) for x in (k, v)]
    w = torch.softmax(kk[:, :, :G].transpose(1, 2) * D ** -0.5, dim=-1)          # [Hkv, G, L]
    ref = (w @ vv).reshape(Hkv * G, D)
    assert ref.abs().min() >= 7.0
    err = (out.double() - ref).abs().max().item()
    print(f"long shares, {nodes} nodes, {out_dtype}: max-abs error {err:.3e}")
    assert err <= (2e-4 if out_dtype == torch.float32 else TOL["bf16"])


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("nodes,G,D,scale", [(1, 4, 128, 0.1), (2, 8, 64, -0.2), (9, 8, 64, 0.2), (17, 8, 128, 0.08)])
def test_long_shares_match_plain(nodes, G, D, scale, out_dtype):
    B, Hkv, top = 76, 4, 11000
    gen = torch.Generator().manual_seed(nodes + G + D)
    blocks = -(-top // 16)
    k, v = [torch.randn(blocks, Hkv, 16, D, generator=gen).to(torch.bfloat16).to(DEV) for _ in range(2)]
    lens = [top - 37 * b % 300 for b in range(B)]
    tables = shared_pool(blocks, B, gen)
    start = i32([nodes * b for b in range(B + 1)])
    # the weights' maximum moves late: larger keys in the blocks that come last
    for b in range(0, B, 5):
        k[tables[b, -1].long()] *= 3.0
    mask = plain.tree_masks([nodes] * B, gen).to(DEV)
    q = torch.randn(B * nodes, Hkv * G, D, generator=gen).to(torch.bfloat16).to(DEV)
    out = torch.full((B * nodes, Hkv * G, D), 7.25, dtype=out_dtype, device=DEV)
    want, bound = plain.tree(q, k, v, tables, i32(lens), start, mask, scale, out)
    binding.forge_paged_tree_attention(q, k, v, tables, i32(lens), start, mask, scale, out)
    assert binding.forge_paged_get_device_error() == 0
    off = (out.double() - want).abs()
    assert not off.isnan().any() and (off <= bound).all()


@pytest.mark.parametrize("G,out_dtype", [(1, torch.bfloat16), (1, torch.float32), (8, torch.bfloat16)])
def test_rows_that_see_some_accumulations_only(G, out_dtype):
    """A prompt of 5504 nodes under sparse masks: rows that see nothing at all, nothing before or nothing from position
    5120 on, and infinities on both sides that only some rows see."""
    n, D = 5504, 64
    Hkv = 32 // G
    gen = torch.Generator().manual_seed(G)
    seen = torch.rand(n, n, generator=gen) < 0.004
    seen[5] = False
    seen[6::50, :5120] = False
    seen[7::50, 5120:] = False
    k, v = [torch.randn(n // 16, Hkv, 16, D, generator=gen).to(torch.bfloat16).to(DEV) for _ in range(2)]
    for t in (33, 5300):
        v[t // 16, :, t % 16, 3] = float("inf")
        seen[:, t] = torch.rand(n, generator=gen) < 0.05
    W = -(-n // 64)
    bits = np.zeros((n, 64 * W), dtype=np.uint8)
    bits[:, :n] = seen.numpy()
    mask = torch.from_numpy(np.packbits(bits, axis=1, bitorder="little").view("<i8").copy()).to(DEV)
    q = torch.randn(n, Hkv * G, D, generator=gen).to(torch.bfloat16).to(DEV)
    tables = torch.arange(n // 16, dtype=torch.int32, device=DEV)[None]
    out = torch.full((n, Hkv * G, D), 7.25, dtype=out_dtype, device=DEV)
    binding.forge_paged_tree_attention(q, k, v, tables, i32([n]), i32([0, n]), mask, 0.2, out)
    assert binding.forge_paged_get_device_error() == 0
    seen = seen.to(DEV)
    for g in (0, Hkv - 1):
        h = slice(g * G, (g + 1) * G)
        kk, vv = plain.rows64(k, tables[0], n)[g], plain.rows64(v, tables[0], n)[g]
        ref, _, bound, _ = plain.attend(q[:, h], kk, vv, seen, 0.2)
        got = out[:, h].double()
        fine = ref.isfinite()
        bound = bound + plain.half_step(ref, out_dtype)
        assert ((got - ref).abs()[fine] <= bound[fine]).all()
        assert not fine.all() and not got[~fine].isfinite().any()
    assert (out[5] == 0).all()
