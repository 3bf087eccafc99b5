"""Tree entry points on inputs that they take and that lie at their edges."""
import numpy as np
import pytest

import _tree as T
from test_gpu_tree import HALF, _commit

pytestmark = pytest.mark.gpu


# ---- scores of large magnitude --------------------------------------------------
def _far_cache(rng, lens, nodes, dtype, hkv, d, keys):
    """A cache whose keys are keys[s][position] along dim 0 and zero elsewhere."""
    import torch
    c = T.Cache(rng, lens, nodes, dtype=dtype, layers=1, hkv=hkv, d=d, page=16)
    for s, k in enumerate(keys):
        pos = torch.arange(lens[s] + nodes[s], device="cuda")
        pg = c.bt[s].long()[pos // 16]
        row = torch.zeros((len(k), 1, d), device="cuda")
        row[:, 0, 0] = torch.from_numpy(np.asarray(k, np.float32)).cuda()
        row = row.expand(-1, hkv, -1).to(c.kv.dtype)
        c.kv[pg, 0, :, 0, pos % 16] = row
        c.rows[s][:, 0, :, 0] = row.double()
    return c


def _far_check(c, lens, nodes, parents, G, amps, scale):
    """Queries amps[h % len(amps)] along dim 0, so that heads (lanes of a warp) have scores of different sizes."""
    import torch
    hkv, d = c.hkv, c.d
    q = torch.zeros((len(lens), T.N, hkv * G, d), device="cuda")
    for h in range(hkv * G):
        q[:, :, h, 0] = amps[h % len(amps)]
    q = q.to(c.kv.dtype)
    out, err = T.attention(c, 0, q, lens, nodes, parents, scale)
    assert err == 0
    for s, (n, k) in enumerate(zip(lens, nodes)):
        ref, _ = T.ref_attention(c.rows[s], 0, q[s], n, k, parents[s], scale)
        # products of one term are exact, and so are differences of the scores here: no error of the scores' size
        tol = T.tol(d, n + k, 0.0, float(c.rows[s][:, 0, :, 1].abs().max()))
        err = (out[s, :k].double() - ref).abs()
        assert bool((err <= HALF[c.dtype] * ref.abs() + tol).all()), (s, n, k, float(err.nan_to_num(9e9).max()))


@pytest.mark.parametrize("dtype", [T.F32, T.BF16])
@pytest.mark.parametrize("G,nodes,d", [(1, 12, 64), (2, 28, 128), (3, 40, 64), (8, 64, 128), (1, 20, 128), (6, 33, 64)])
@pytest.mark.parametrize("size", [2.0 ** 10, 2.0 ** 24, 2.0 ** 28, 2.0 ** 31, 2.0 ** 34, 2.0 ** 120])
def test_attention_of_equal_scores_of_any_size(dtype, G, nodes, d, size):
    """All keys alike: every row is the mean of its values, whatever the scores' size and sign."""
    rng = np.random.default_rng(nodes)
    lens, ks = [0, 200, 1500], [nodes, nodes, max(1, nodes - 3)]
    parents = np.stack([T.rand_parents(rng, k) for k in ks])
    c = _far_cache(rng, lens, ks, dtype, 2, d, [np.full(n + k, 1.37 * size ** 0.5) for n, k in zip(lens, ks)])
    a = 1.21 * size ** 0.5                                     # (powers of two would have exact products)
    _far_check(c, lens, ks, parents, G, [a, -a, 1.0 / a, 0.0, -1.0 / a, a / 64], 1.0)


@pytest.mark.parametrize("dtype", [T.F32, T.BF16])
@pytest.mark.parametrize("G,nodes,d", [(1, 12, 64), (2, 28, 128), (3, 40, 64), (8, 64, 128), (1, 20, 128), (6, 33, 64)])
@pytest.mark.parametrize("size", [2.0 ** 26, 2.0 ** 31, 2.0 ** 33, 2.0 ** 60, 2.0 ** 120])
def test_attention_of_scores_far_apart(dtype, G, nodes, d, size):
    """Keys in steps of 1/128 of a large value, up along one sequence, down along
    another, and of both signs in a third: the largest take the whole weight."""
    rng = np.random.default_rng(nodes + 1)
    lens, ks = [900, 900, 700], [nodes, nodes, nodes]
    parents = np.stack([T.rand_parents(rng, k) for k in ks])
    a = size ** 0.5
    ramp = np.floor(np.arange(900 + nodes) / 60) / 128
    keys = [a * (1 + ramp), a * (1 + ramp[::-1]), a * np.where(np.arange(700 + nodes) % 97 == 5, -1.0, 1.0)]
    c = _far_cache(rng, lens, ks, dtype, 2, d, keys)
    _far_check(c, lens, ks, parents, G, [a, -a, 0.0, 1.0 / a, a], 1.0)


# ---- pages of a committed path --------------------------------------------------
@pytest.mark.parametrize("bad", [-1, 10 ** 6])
def test_commit_needs_the_pages_of_rows_that_stay(bad):
    """A path whose rows already lie in place needs its pages as much as one that moves."""
    import torch
    rng = np.random.default_rng(5)
    lens, k = [14, 14, 30, 31], 6
    c = T.Cache(rng, lens, [k] * 4, dtype=T.BF16, layers=2, hkv=2, d=64, page=16, junk=1.0)
    parents = np.tile(np.append(np.arange(-1, k - 1), [-1] * (T.N - k)).astype(np.int32), (4, 1))
    tokens = np.tile(np.arange(T.N, dtype=np.int32), (4, 1))
    target = tokens + 1                                        # a chain, accepted in full: no row moves
    target[3, 0] = 99                                          # the root alone
    c.bt[1, 1] = bad                                           # positions 16 .. 31: nodes 2 and later
    c.bt[2, 2] = bad                                           # positions 32 .. 47: nodes 2 and later
    before = c.kv.clone()
    acc, tok, ln, path, err = _commit(c, tokens, parents, target, lens, [k] * 4)
    assert err == 1
    assert acc.tolist() == [k - 1, -1, -1, 0] and ln.tolist() == [14 + k, 14, 30, 32]
    assert tok.tolist() == [k, -1, -1, 99] and (path[1:3] == -1).all() and path[3, :2].tolist() == [0, -1]
    c.bt[3, 1] = bad                                           # the root's own page
    c.bt[2, 1] = bad
    tokens[0, 2] = 77                                          # ends at position 15: the next page is not asked for
    c.bt[0, 1] = bad
    acc, tok, ln, path, err = _commit(c, tokens, parents, target, lens, [k] * 4)
    assert err == 1 and acc.tolist() == [1, -1, -1, -1] and ln.tolist() == [16, 14, 30, 31]
    assert bool(torch.equal(c.kv, before))


# ---- sizes past 32 bits, long lists -----------------------------------------------
def test_commit_and_copies_past_32_bits():
    """Pages at both ends of a cache of more than 2^32 elements."""
    import torch
    from lossless_speculative_decoding_gb300 import binding as B
    pages, layers, hkv, d, P, k = 3800, 36, 8, 128, 16, 6
    kv = torch.zeros((pages, layers, hkv, 2, P, d), dtype=torch.bfloat16, device="cuda")
    assert kv.numel() > 2 ** 32
    for p in (0, 1, pages - 3, pages - 2, pages - 1):
        kv[p].normal_(generator=torch.Generator(device="cuda").manual_seed(p))
    table = np.array([[pages - 1, pages - 2], [0, pages - 3]], np.int32)
    bt = T.dev(table)
    view = B.make_kv_view(kv, bt, dtype=T.BF16, n_pages=pages, n_layers=layers, n_kv_heads=hkv, page_size=P, head_dim=d, max_pages=2)
    lens = [12, 13]
    parents = np.array([[-1, 0, 0, 0, 3, 4], [-1, 0, 1, 1, 1, 4]], np.int32)
    tokens = np.array([[0, 1, 2, 3, 4, 5], [0, 1, 2, 3, 4, 5]], np.int32)
    target = np.array([[3, 9, 9, 4, 5, 8], [1, 4, 9, 9, 5, 7]], np.int32)
    paths = [T.ref_walk(parents[s], tokens[s], target[s], k) for s in range(2)]
    assert paths == [[0, 3, 4, 5], [0, 1, 4, 5]]
    keep = {p: kv[p].clone() for p in (0, 1, pages - 3, pages - 2, pages - 1)}
    want = {p: v.clone() for p, v in keep.items()}
    for s, path in enumerate(paths):
        for j, i in enumerate(path):
            a, b = lens[s] + i, lens[s] + j
            want[int(table[s, b // P])][:, :, :, b % P] = keep[int(table[s, a // P])][:, :, :, a % P]
    o = [torch.zeros(2, dtype=torch.int32, device="cuda") for _ in range(3)]
    path, err = torch.zeros((2, k), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    B.spec_tree_commit(view, 2, k, T.dev(tokens), T.dev(parents), T.dev([k, k]), T.dev(target), T.dev(lens), o[0], o[1], path, o[2], err, 0)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and o[0].tolist() == [3, 3] and o[2].tolist() == [16, 17]
    for p, v in want.items():
        assert bool(torch.equal(kv[p], v)), p
    B.spec_kv_copy_pages(view, T.dev([pages - 1, 0]), T.dev([2, pages - 4]), 2, err, 0)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and bool(torch.equal(kv[2], want[pages - 1])) and bool(torch.equal(kv[pages - 4], want[0]))
    assert float(kv[3:pages - 4].abs().max()) == 0.0


def test_copies_of_a_list_longer_than_a_grid():
    """More pairs than a grid has rows, most of them padding."""
    import torch
    from lossless_speculative_decoding_gb300 import binding as B
    n, pages = 70001, 40
    kv = torch.randn((pages, 1, 1, 2, 16, 64), device="cuda")
    src, dst = np.full(n, -1, np.int32), np.full(n, -1, np.int32)
    at = np.array([0, 1, 65534, 65535, 65536, 70000])
    src[at], dst[at] = np.arange(6), 20 + np.arange(6)
    want = kv.clone()
    want[20:26] = kv[:6]
    view = B.make_kv_view(kv, None, dtype=T.F32, n_pages=pages, n_layers=1, n_kv_heads=1, page_size=16, head_dim=64, max_pages=0)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.spec_kv_copy_pages(view, T.dev(src), T.dev(dst), n, err, 0)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and bool(torch.equal(kv, want))
