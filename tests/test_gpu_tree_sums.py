"""Sums of the tree attention and the token log probabilities to their last
part: every tile, step and thread has a share of its own that would be missed,
and errors are bounded by the depth of the sums, not by their length."""
import math

import numpy as np
import pytest

import _tree as T
from test_gpu_logprob_range import _check
from test_gpu_tree import HALF

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [T.F32, T.BF16])
@pytest.mark.parametrize("V", [1024, 5003, 129280, 151936, 1048576])
def test_logprobs_of_a_near_uniform_row(dtype, V):
    """A thread's step (32 or 64 tokens) left out or counted twice is above the limit up to 151,936 tokens, a warp's
    part of a step (1,024 or 2,048) at 1,048,576."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.rand((3, V), generator=g, device="cuda") * 0.01
    x = x if dtype == T.F32 else x.bfloat16()
    _check(x, np.array([0, V // 2, V - 1], np.int32), 1.0, 2)


@pytest.mark.parametrize("dtype", [T.F32, T.BF16])
@pytest.mark.parametrize("V,top", [(129280, 0), (70001, 20)])
def test_logprobs_with_half_of_the_mass_in_one_place(dtype, V, top):
    """Row r has half of its probability in piece r of the row: a warp's part of a step, and 40 tokens at a time."""
    import torch
    part = 1024 if dtype == T.F32 else 2048                    # 4 KB
    for size, places in ((part, range(0, V, part)), (40, range(0, V, V // 150))):
        x = torch.zeros((len(places), V), device="cuda")
        for r, a in enumerate(places):
            b = min(V, a + size)
            # (b - a) e^k = V - (b - a): as much as all others; to the quarter, which both types hold
            x[r, a:b] = round(4 * math.log((V - (b - a)) / (b - a))) / 4
        x = x if dtype == T.F32 else x.bfloat16()
        tokens = np.array([min(V - 1, a + size // 2) for a in places], np.int32)
        _check(x, tokens, 1.0, top)


def _limit(dtype, n, ref):
    """Equal weights, values 0 and 1, an output the share of the ones. A lane's weights and values are exact (powers of
    two, kept as two bf16 parts where that is used), the sums of whole numbers times a power of two as well up to 2^24;
    the parts of a sequence are joined with weights 2^0 and divided by the sum: a reciprocal, two products and a sum of
    parts, under 32 roundings of 2^-24; then the output's own rounding."""
    return HALF[dtype] * ref + 32 * 2.0 ** -24


@pytest.mark.parametrize("dtype", [T.F32, T.BF16])
@pytest.mark.parametrize("hq,hkv,d,page,lens,nodes", [
    (10, 10, 128, 16, [1357], [16]), (32, 8, 128, 64, [1288, 5288, 2111], [64, 64, 33]), (8, 2, 64, 16, [40, 700, 127, 128], [64, 9, 1, 1]),
    (10, 10, 128, 16, [336, 5236, 1000, 2500, 777] * 6, [17, 32, 20, 29, 3] * 6), (8, 1, 128, 48, [33011], [13]),
    (16, 2, 64, 16, [30001, 15000], [21, 8])])
def test_attention_counts_every_position(dtype, hq, hkv, d, page, lens, nodes):
    """Queries of zero: equal weights. Value dim c is one for the positions of
    the c-th of d pieces of the sequence, zero for the others: each output is a
    count of a few positions in particular, none of which may be missing."""
    import torch
    rng = np.random.default_rng(len(lens))
    c = T.Cache(rng, lens, nodes, dtype=dtype, layers=1, hkv=hkv, d=d, page=page)
    for s, (n, k) in enumerate(zip(lens, nodes)):
        pos = torch.arange(n + k, device="cuda")
        one = torch.zeros((n + k, 1, d), device="cuda")
        one[pos, 0, pos * d // (n + k)] = 1.0
        one = one.expand(-1, hkv, -1)
        c.kv[c.bt[s].long()[pos // page], 0, :, 1, pos % page] = one.to(c.kv.dtype)
        c.rows[s][:, 0, :, 1] = one.double()
    parents = np.stack([T.rand_parents(rng, k) for k in nodes])
    q = torch.zeros((len(lens), T.N, hq, d), dtype=c.kv.dtype, device="cuda")
    out, err = T.attention(c, 0, q, lens, nodes, parents, 1.0 / math.sqrt(d))
    assert err == 0
    for s, (n, k) in enumerate(zip(lens, nodes)):
        ref, _ = T.ref_attention(c.rows[s], 0, q[s], n, k, parents[s], 1.0)
        off = (out[s, :k].double() - ref).abs()
        assert bool((off <= _limit(dtype, n + k, ref)).all()), (s, float(off.max()))


@pytest.mark.parametrize("dtype", [T.F32, T.BF16])
@pytest.mark.parametrize("G,d", [(1, 64), (3, 128), (8, 64), (16, 128)])
def test_attention_of_one_tile_at_a_time(dtype, G, d):
    """Values that are zero but for 16 positions, somewhere else in each
    sequence, with ordinary queries: the relative error of an output is that of
    its few weights, not of a sum over the sequence."""
    import torch
    rng = np.random.default_rng(G)
    lens, nodes = [1500] * 24, [(7 * i) % 40 + 1 for i in range(24)]
    c = T.Cache(rng, lens, nodes, dtype=dtype, layers=1, hkv=2, d=d, page=16)
    for s, (n, k) in enumerate(zip(lens, nodes)):
        a = (n + k - 16) * s // 23                             # from the first positions to the last nodes
        keep = torch.zeros((n + k, 1, 1), device="cuda")
        keep[a:a + 16] = 1.0
        v = c.rows[s][:, 0, :, 1].abs() * keep                 # (one sign: nothing cancels)
        pos = torch.arange(n + k, device="cuda")
        c.kv[c.bt[s].long()[pos // 16], 0, :, 1, pos % 16] = v.to(c.kv.dtype)
        c.rows[s][:, 0, :, 1] = v
    parents = np.stack([T.rand_parents(rng, k) for k in nodes])
    g = torch.Generator(device="cuda").manual_seed(G)
    q = (torch.randn((24, T.N, 2 * G, d), generator=g, device="cuda") * 0.5).to(c.kv.dtype)
    scale = 1.0 / math.sqrt(d)
    out, err = T.attention(c, 0, q, lens, nodes, parents, scale)
    assert err == 0
    for s, (n, k) in enumerate(zip(lens, nodes)):
        ref, _ = T.ref_attention(c.rows[s], 0, q[s], n, k, parents[s], scale)
        # a score errs by (d + 4) 2^-24 of the sum of its products' sizes, and with it a weight and the weights' sum; the
        # power 2^-22, a weight's two bf16 parts 2^-17; an accumulator takes 128 keys a tile for 13 tiles at most, sums of
        # one sign: a rounding each for the 16 products of an instruction, 8 or 16 instructions a tile, and the joins
        mag = float((torch.einsum("ihgd,jhd->hgij", q[s, :k].double().abs().view(k, 2, G, d), c.rows[s][:, 0, :, 0].abs()) * scale).max())
        e = 2 * ((d + 4) * 2.0 ** -24 * mag + 2.0 ** -22 + 2.0 ** -17 + (13 * 16 + 64) * 2.0 ** -24)
        off = (out[s, :k].double() - ref).abs()
        assert bool((off <= (HALF[dtype] + e) * ref + 1e-30).all()), (s, float((off / ref.clamp(min=1e-30)).max()), e)
