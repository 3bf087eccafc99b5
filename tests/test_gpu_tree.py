"""Tree attention, tree commit and page copies on the GPU against a 64-bit
restatement (tests/_tree.py), at the lengths, trees, head groups and pages
where they can go wrong, and a whole tree step of the operators together.
Unused cache slots hold NaN, rows that must stay hold a marker."""
import math

import numpy as np
import pytest

import _tree as T

pytestmark = pytest.mark.gpu

HALF = {T.F32: 2.0 ** -24, T.BF16: 2.0 ** -8}                  # half a step of the output type


def _q(rng_seed, S, k, hq, d, dtype, sharp=1.0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(rng_seed)
    q = torch.randn((S, k, hq, d), generator=g, device="cuda") * sharp
    return q.to(torch.float32 if dtype == T.F32 else torch.bfloat16)


def _check(c, layer, q, lens, nodes, parents, out, scale):
    for s, (n, k) in enumerate(zip(lens, nodes)):
        if k:
            ref, tol = T.ref_attention(c.rows[s], layer, q[s], n, k, parents[s], scale)
            err = (out[s, :k].double() - ref).abs()
            lim = HALF[c.dtype] * ref.abs() + tol
            assert bool((err <= lim).all()), (s, n, k, float((err / lim).max()))
        assert bool((out[s, k:] == 77.0).all()), "rows past the tree were written"


CASES = [
    # dtype, hq, hkv, d, page, lens, nodes
    (T.F32, 4, 4, 64, 16, [0, 1, 15, 16, 17, 200], [8, 1, 5, 64, 0, 33]),
    (T.F32, 8, 2, 128, 32, [63, 64, 65, 130], [3, 64, 1, 17]),
    (T.F32, 6, 1, 128, 48, [500], [21]),
    (T.BF16, 10, 10, 128, 16, [1357], [16]),
    (T.BF16, 10, 10, 128, 16, [0, 1, 16, 127, 128, 129, 777, 40], [1, 64, 17, 32, 33, 8, 31, 0]),
    (T.BF16, 32, 8, 128, 64, [0, 63, 64, 191, 192, 1000, 2100], [64, 1, 16, 17, 33, 64, 7]),
    (T.BF16, 32, 8, 128, 128, [256, 3001], [64, 21]),
    (T.BF16, 4, 4, 64, 16, [5, 130, 1025, 0], [2, 64, 40, 64]),
    (T.BF16, 16, 2, 64, 48, [95, 96, 97, 700], [64, 16, 4, 33]),
    (T.BF16, 12, 1, 128, 16, [333, 31], [64, 11]),
    (T.BF16, 128, 1, 64, 32, [77, 600], [64, 3]),
    (T.BF16, 10, 10, 128, 16, [3, 900, 2] * 30, [4, 12, 1] * 30),
    (T.BF16, 8, 1, 128, 16, [33011], [13]),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention_matches_64_bits(case):
    dtype, hq, hkv, d, page, lens, nodes = CASES[case]
    rng = np.random.default_rng(100 + case)
    layers = 1 if sum(lens) > 20000 else 2
    c = T.Cache(rng, lens, nodes, dtype=dtype, layers=layers, hkv=hkv, d=d, page=page, seed=case)
    parents = np.stack([T.rand_parents(rng, k, forest=True) for k in nodes])
    q = _q(case, len(lens), T.N, hq, d, dtype, sharp=2.0)
    scale = 1.0 / math.sqrt(d)
    for layer in range(layers):
        out, err = T.attention(c, layer, q, lens, nodes, parents, scale)
        assert err == 0
        _check(c, layer, q, lens, nodes, parents, out, scale)
    again, _ = T.attention(c, layers - 1, q, lens, nodes, parents, scale)
    assert bool((again == out).all()), "the same call, other bits"


@pytest.mark.parametrize("dtype", [T.F32, T.BF16])
@pytest.mark.parametrize("max_nodes", [1, 7, 31])
def test_attention_with_narrow_rows(dtype, max_nodes):
    """max_nodes below 64: rows are max_nodes apart."""
    rng = np.random.default_rng(3)
    lens, nodes = [40, 300, 7], [max_nodes, max(1, max_nodes - 2), 1]
    c = T.Cache(rng, lens, nodes, dtype=dtype, layers=1, hkv=2, d=64, page=16)
    parents = np.stack([T.rand_parents(rng, k)[:max_nodes] for k in nodes])
    q = _q(5, 3, max_nodes, 6, 64, dtype)
    out, err = T.attention(c, 0, q, lens, nodes, parents, 0.125)
    assert err == 0
    _check(c, 0, q, lens, nodes, parents, out, 0.125)


def test_attention_sharp_scores_and_growing_maximum():
    """Keys whose scores grow along the sequence, so that the running maximum
    moves all the way, and a scale that makes the weights nearly one-hot."""
    import torch
    rng = np.random.default_rng(8)
    lens, nodes = [1500, 640], [16, 40]
    c = T.Cache(rng, lens, nodes, dtype=T.BF16, layers=1, hkv=2, d=128, page=16)
    parents = np.stack([T.rand_parents(rng, k) for k in nodes])
    u = torch.randn(128, device="cuda")
    for s in range(2):
        t = lens[s] + nodes[s]
        ramp = torch.linspace(-1.0, 1.0, t, device="cuda")[:, None]
        k = (ramp * u * (1 if s == 0 else -1)).to(torch.bfloat16)
        pos = torch.arange(t, device="cuda")
        pg = c.bt[s].long()[pos // 16]
        c.kv[pg, 0, 0, 0, pos % 16] = k
        c.rows[s][:, 0, 0, 0] = k.double()
    q = _q(9, 2, T.N, 4, 128, T.BF16)
    q[:, :, :2] = (q[:, :, :2] * 0.1 + 3 * u).to(torch.bfloat16)
    out, err = T.attention(c, 0, q, lens, nodes, parents, 0.5)
    assert err == 0
    _check(c, 0, q, lens, nodes, parents, out, 0.5)


def test_attention_offsets_past_32_bits():
    """Pages far apart in a cache of more than 2^32 elements."""
    import torch
    from lossless_speculative_decoding_gb300 import binding as B
    rng = np.random.default_rng(4)
    small = T.Cache(rng, [100, 250], [9, 33], dtype=T.BF16, layers=1, hkv=8, d=128, page=16)
    layers, pages = 36, 3800                                   # 3800 x 1,179,648 elements
    big = torch.empty((pages, layers, 8, 2, 16, 128), dtype=torch.bfloat16, device="cuda")
    assert big.numel() > 2 ** 32
    move = np.sort(rng.permutation(pages)[:small.n_pages]).astype(np.int64)
    move[-1] = pages - 1
    big[torch.from_numpy(move).cuda(), 35] = small.kv[:, 0]
    table = np.where(small.table >= 0, move[small.table], -1).astype(np.int32)
    bt = T.dev(table)
    small.view = B.make_kv_view(big, bt, dtype=T.BF16, n_pages=pages, n_layers=layers, n_kv_heads=8, page_size=16,
                                head_dim=128, max_pages=small.max_pages)
    parents = np.stack([T.rand_parents(rng, k) for k in (9, 33)])
    q = _q(1, 2, T.N, 32, 128, T.BF16)
    out, err = T.attention(small, 35, q, [100, 250], [9, 33], parents, 0.09)
    assert err == 0
    _check(small, 0, q, [100, 250], [9, 33], parents, out, 0.09)


def test_attention_bad_inputs_leave_the_others_alone():
    rng = np.random.default_rng(6)
    lens, nodes = [100, 50, 200, 80, 30], [8, 8, 8, 8, 8]
    c = T.Cache(rng, lens, nodes, dtype=T.BF16, layers=1, hkv=2, d=128, page=16)
    parents = np.stack([T.rand_parents(rng, k) for k in nodes])
    good = parents.copy()
    q = _q(2, 5, T.N, 8, 128, T.BF16)
    bad_lens, bad_nodes = list(lens), list(nodes)
    bad_lens[0], bad_nodes[1] = -1, 65                          # left out
    parents[3, 5], good[3, 5] = 7, -1                           # counts as a root
    c.bt[2, 4], c.bt[4, 1] = c.n_pages, -1
    out, err = T.attention(c, 0, q, bad_lens, bad_nodes, parents, 0.1)
    assert err == 1 | 4 | 16
    assert bool((out[:2] == 77.0).all())
    ref, tol = T.ref_attention(c.rows[3], 0, q[3], 80, 8, good[3], 0.1)
    assert bool(((out[3, :8].double() - ref).abs() <= HALF[T.BF16] * ref.abs() + tol).all())
    out2, err = T.attention(c, 0, q, [c.max_pages * 16 - 7] + lens[1:], nodes, good, 0.1)   # past the block table
    assert err & 4 and bool((out2[0] == 77.0).all())


def test_attention_streams_and_graphs():
    """On another stream, captured, and replayed on new inputs; two graphs
    with a workspace each."""
    import torch
    from lossless_speculative_decoding_gb300 import binding as B
    rng = np.random.default_rng(7)
    lens, nodes = [513, 90, 260], [12, 64, 3]
    c = T.Cache(rng, lens, nodes, dtype=T.BF16, layers=2, hkv=8, d=128, page=16)
    parents = np.stack([T.rand_parents(rng, k) for k in nodes])
    st = torch.cuda.Stream()
    q = [_q(i, 3, T.N, 32, 128, T.BF16) for i in range(2)]
    out = [torch.full_like(q[0], 77.0) for _ in range(2)]
    nb = B.spec_tree_attention_ws_bytes(c.view, 3, T.N, 32)
    ws = [torch.empty(nb, dtype=torch.uint8, device="cuda") for _ in range(2)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    a = (T.dev(lens), T.dev(nodes), T.dev(parents))
    call = lambda i: B.spec_tree_attention(c.view, i, q[i], 3, T.N, 32, *a, 0.09, out[i], ws[i], nb, err, st.cuda_stream)  # noqa: E731
    torch.cuda.synchronize()
    call(0)
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        st.synchronize()
        with torch.cuda.graph(g, stream=st):
            call(i)
        graphs.append(g)
    for seed in (20, 30):
        for i in range(2):
            q[i].copy_(_q(seed + i, 3, T.N, 32, 128, T.BF16))
        torch.cuda.synchronize()
        for i in range(2):
            graphs[i].replay()
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        for i in range(2):
            _check(c, i, q[i], lens, nodes, parents, out[i], 0.09)


# ---- commit ----------------------------------------------------------------
def _commit(c, tokens, parents, target, lens, nodes):
    import torch
    from lossless_speculative_decoding_gb300 import binding as B
    S, m = tokens.shape
    o = [torch.full((S,), -9, dtype=torch.int32, device="cuda") for _ in range(3)]
    path = torch.full((S, m), -9, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.spec_tree_commit(c.view, S, m, T.dev(tokens), T.dev(parents), T.dev(nodes), T.dev(target), T.dev(lens), o[0], o[1],
                       path, o[2], err, 0)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in o] + [path.cpu().numpy(), int(err.item())]


@pytest.mark.parametrize("dtype,layers,hkv,d,page,max_nodes", [(T.F32, 2, 4, 64, 16, 64), (T.BF16, 3, 10, 128, 16, 64),
                                                               (T.BF16, 1, 1, 64, 48, 40), (T.BF16, 12, 8, 128, 64, 33)])
def test_commit_walks_and_moves(dtype, layers, hkv, d, page, max_nodes):
    import torch
    rng = np.random.default_rng(layers * 10 + page)
    S = 9
    lens = [0, 1, 15, 16, 40, 47, 100, 130, 33]
    nodes = [max_nodes, 1, 2, max_nodes, 20, 0, max_nodes, 7, max_nodes - 1]
    c = T.Cache(rng, lens, nodes, dtype=dtype, layers=layers, hkv=hkv, d=d, page=page, junk=5.0)
    parents = np.stack([T.rand_parents(rng, k, forest=True)[:max_nodes] for k in nodes])
    tokens = rng.integers(0, 6, (S, max_nodes)).astype(np.int32)      # few tokens: twins among the children
    target = rng.integers(0, 6, (S, max_nodes)).astype(np.int32)
    # sequence 3: one long chain, all accepted, no row moves; sequence 6: every second node
    parents[3] = np.arange(-1, max_nodes - 1)
    target[3, :-1] = tokens[3, 1:]
    parents[6] = np.maximum(np.arange(max_nodes) - 2, -1)
    parents[6, 2:4] = 0
    target[6, ::2] = np.append(tokens[6, 2::2], 5)[: len(target[6, ::2])]
    before = c.kv.clone()
    acc, tok, ln, path, err = _commit(c, tokens, parents, target, lens, nodes)
    assert err == 0
    want = before.clone()
    deep = 0
    for s, (n, k) in enumerate(zip(lens, nodes)):
        if k == 0:
            assert (acc[s], tok[s], ln[s]) == (-1, -1, n) and (path[s] == -1).all()
            continue
        p = T.ref_walk(parents[s], tokens[s], target[s], k)
        assert acc[s] == len(p) - 1 and tok[s] == target[s, p[-1]] and ln[s] == n + len(p)
        assert path[s].tolist() == p + [-1] * (max_nodes - len(p))
        deep = max(deep, len(p))
        for j, i in enumerate(p):
            src, dst = n + i, n + j
            want[c.table[s, dst // page], :, :, :, dst % page] = before[c.table[s, src // page], :, :, :, src % page]
    assert deep >= max_nodes // 2
    assert bool(torch.equal(c.kv, want))


def test_commit_bad_inputs():
    import torch
    rng = np.random.default_rng(1)
    lens, nodes = [20, 20, 20, -3], [4, 65, 4, 2]
    c = T.Cache(rng, [20, 20, 20, 0], [4, 4, 4, 2], dtype=T.BF16, layers=2, hkv=2, d=64, page=16, junk=1.0)
    parents = np.tile(np.array([-1, 0, 0, 2] + [-1] * 60, np.int32), (4, 1))
    tokens = np.zeros((4, 64), np.int32)
    tokens[:, 2:4] = 7
    target = np.full((4, 64), 9, np.int32)
    target[:, 0] = 7                                                   # accepts node 2, row 2 -> slot n + 1
    parents[0, 3] = 3                                                  # not below 2: raises the bit, is not reached
    c.bt[2, 1] = c.n_pages                                             # the page of positions 16..31
    before = c.kv.clone()
    acc, tok, ln, path, err = _commit(c, tokens, parents, target, lens, nodes)
    assert err == 1 | 4 | 16
    assert acc.tolist() == [1, -1, -1, -1] and tok.tolist() == [9, -1, -1, -1] and ln.tolist() == [22, 20, 20, -3]
    assert (path[1:] == -1).all() and path[0, :3].tolist() == [0, 2, -1]
    want = before.clone()
    pg = c.table[0, 1]
    want[pg, :, :, :, 21 % 16] = before[pg, :, :, :, 22 % 16]
    assert bool(torch.equal(c.kv, want))


# ---- page copies -------------------------------------------------------------
@pytest.mark.parametrize("dtype,layers,hkv,d,page,n", [(T.F32, 2, 4, 64, 16, 5), (T.BF16, 12, 10, 128, 16, 3),
                                                       (T.BF16, 1, 1, 64, 48, 70), (T.BF16, 36, 8, 128, 16, 1)])
def test_copy_pages(dtype, layers, hkv, d, page, n):
    import torch
    from lossless_speculative_decoding_gb300 import binding as B
    rng = np.random.default_rng(n)
    pages = 2 * n + 3
    kv = torch.randn((pages, layers, hkv, 2, page, d), device="cuda")
    kv = kv if dtype == T.F32 else kv.bfloat16()
    ids = rng.permutation(pages)
    dst, src = ids[:n].astype(np.int32), ids[n:][rng.integers(0, pages - n, n)].astype(np.int32)
    view = B.make_kv_view(kv, None, dtype=dtype, n_pages=pages, n_layers=layers, n_kv_heads=hkv, page_size=page, head_dim=d,
                          max_pages=0)
    want = kv.clone()
    want[torch.from_numpy(dst.astype(np.int64)).cuda()] = kv[torch.from_numpy(src.astype(np.int64)).cuda()]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pad = lambda a, v: T.dev(np.concatenate([a, v]))                   # noqa: E731  padded pairs are skipped
    B.spec_kv_copy_pages(view, pad(src, [-1, 0]), pad(dst, [1, -1]), n + 2, err, 0)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and bool(torch.equal(kv, want))
    B.spec_kv_copy_pages(view, T.dev([pages, 0, -2]), T.dev([0, pages + 7, 1]), 3, err, 0)
    torch.cuda.synchronize()
    assert int(err.item()) == 1 and bool(torch.equal(kv, want))


# ---- together ------------------------------------------------------------------
def test_a_tree_step_of_the_operators_together():
    """Two steps of a two-layer attention decoder on trees: attention in every
    layer, logits, target tokens, commit, log probabilities, then a fork whose
    last page is copied, and a step of both branches. The second step has to
    see the cache that plain decoding of the accepted tokens would have."""
    import torch
    from lossless_speculative_decoding_gb300 import binding as B
    rng = np.random.default_rng(12)
    g = torch.Generator(device="cuda").manual_seed(12)
    L, hq, hkv, d, P, V, h = 2, 8, 2, 64, 16, 512, 128
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")         # noqa: E731
    emb, wq = rnd(V, h), rnd(L, h, hq * d) / h ** 0.5
    wkv, wo, wl = rnd(L, h, hkv * 2 * d) / h ** 0.5, rnd(L, hq * d, h) / (hq * d) ** 0.5, rnd(h, V) / h ** 0.5
    n_pages, max_pages = 24, 6
    kv = torch.full((n_pages, L, hkv, 2, P, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    pool = B.spec_pool_create(n_pages, P, 4, max_pages)

    def tables(seqs):
        t = np.full((len(seqs), max_pages), -1, np.int32)
        for i, s in enumerate(seqs):
            row = B.spec_pool_block_table(pool, s)
            t[i, :len(row)] = row
        return t

    def step(seqs, lens, tokens, parents, nodes):
        """A forward over trees: K/V of the nodes into their slots, attention, logits [S, N, V]."""
        t = tables(seqs)
        bt = T.dev(t)
        view = B.make_kv_view(kv, bt, dtype=T.BF16, n_pages=n_pages, n_layers=L, n_kv_heads=hkv, page_size=P, head_dim=d,
                              max_pages=max_pages)
        S, N = tokens.shape
        nb = B.spec_tree_attention_ws_bytes(view, S, N, hq)
        ws, err = torch.empty(nb, dtype=torch.uint8, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        x = emb[torch.from_numpy(tokens.astype(np.int64)).cuda()]
        for layer in range(L):
            q = (x @ wq[layer]).view(S, N, hq, d).bfloat16()
            kvn = (x @ wkv[layer]).view(S, N, hkv, 2, d).bfloat16()
            for s in range(S):
                for i in range(nodes[s]):
                    p = lens[s] + i
                    kv[t[s, p // P], layer, :, :, p % P] = kvn[s, i]
            out = torch.zeros_like(q)
            B.spec_tree_attention(view, layer, q, S, N, hq, T.dev(lens), T.dev(nodes), T.dev(parents), d ** -0.5, out, ws, nb,
                                  err, 0)
            x = x + out.float().view(S, N, hq * d) @ wo[layer]
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        return view, bt, (x @ wl).contiguous()

    def plain(tokens):
        """float64 logits of a token list decoded as a plain sequence (K and V as stored)."""
        x = emb[torch.tensor(tokens, device="cuda")].double()
        n = len(tokens)
        mask = torch.ones((n, n), dtype=torch.bool, device="cuda").triu(1)
        for layer in range(L):
            xf = x.float()
            q = (xf @ wq[layer]).bfloat16().double().view(n, hq, d)
            c = (xf @ wkv[layer]).bfloat16().double().view(n, hkv, 2, d)
            k, v = c[:, :, 0].repeat_interleave(hq // hkv, 1), c[:, :, 1].repeat_interleave(hq // hkv, 1)
            w = torch.softmax((torch.einsum("ihd,jhd->hij", q, k) * d ** -0.5).masked_fill(mask, float("-inf")), -1)
            x = x + torch.einsum("hij,jhd->ihd", w, v).reshape(n, hq * d).bfloat16().double() @ wo[layer].double()
        return x @ wl.double()

    # prompt of 21 tokens, written as a chain-shaped tree
    text = [rng.integers(0, V, 21).tolist()]
    assert B.spec_pool_reserve(pool, 0, 21 + 40) == 0
    chain = np.arange(-1, 20, dtype=np.int32)[None]
    step([0], [0], np.array(text, np.int32), chain, [21])
    lens, seqs = [20], [0]                       # the last token is the next tree's root
    for turn in range(3):
        S = len(seqs)
        N, nodes = 24, [24, 17][:S]
        parents = np.stack([T.rand_parents(rng, k)[:N] for k in nodes])
        tokens = rng.integers(0, V, (S, N)).astype(np.int32)
        for s in range(S):
            assert B.spec_pool_reserve(pool, seqs[s], lens[s] + N) == 0
            tokens[s, 0] = text[s][-1]
            # one path that plain decoding takes, two deep, by nodes that are not next to each other
            p1, p2 = 5, 11
            parents[s, p1], parents[s, p2] = 0, p1
            tokens[s, p1] = int(plain(text[s])[-1].argmax())
            tokens[s, p2] = int(plain(text[s] + [int(tokens[s, p1])])[-1].argmax())
        view, bt, logits = step(seqs, lens, tokens, parents, nodes)
        # every node's logits are those of plain decoding of its path: two layers of results rounded once to bf16
        for s in range(S):
            for i in (0, 5, 11, nodes[s] - 1):
                path = [int(tokens[s, j]) for j in reversed(T.chain_of(parents[s], i))]
                ref = plain(text[s][:-1] + path)[-1]
                assert float((logits[s, i].double() - ref).abs().max()) < 0.02 * float(ref.max() - ref.min())
        target = logits.argmax(-1).int()
        out = [torch.empty(S, dtype=torch.int32, device="cuda") for _ in range(3)]
        path, err = torch.empty((S, N), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        B.spec_tree_commit(view, S, N, T.dev(tokens), T.dev(parents), T.dev(nodes), target, T.dev(lens), out[0], out[1], path,
                           out[2], err, 0)
        f = lambda *s: torch.empty(s, dtype=torch.float32, device="cuda")  # noqa: E731
        lp, ent, rank, ids, top = f(S * N), f(S * N), torch.empty(S * N, dtype=torch.int32, device="cuda"), \
            torch.empty((S * N, 3), dtype=torch.int32, device="cuda"), f(S * N, 3)
        nb = B.spec_token_logprobs_ws_bytes(S * N, V, 3)
        B.spec_token_logprobs(logits, T.F32, V, S * N, V, target, 1.0, 3, lp, ent, rank, ids, top,
                              torch.zeros(nb, dtype=torch.uint8, device="cuda"), nb, 0)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        assert bool((rank == 1).all()) and bool(torch.equal(ids[:, 0], target.reshape(-1)))
        assert bool(torch.equal(lp, top[:, 0]))
        for s in range(S):
            a, p = int(out[0][s]), path[s].tolist()
            assert p[:3] == [0, 5, 11] and a >= 2
            text[s] += [int(tokens[s, i]) for i in p[1:a + 1]] + [int(out[1][s])]
            lens[s] = int(out[2][s])
            assert lens[s] == len(text[s]) - 1
            assert B.spec_pool_commit(pool, seqs[s], lens[s], 0) == 0
        if turn == 0:                            # fork: full pages shared, the last one copied
            full = lens[0] // P
            assert B.spec_pool_share(pool, 0, full, 1) == 0 and B.spec_pool_reserve(pool, 1, lens[0] + 1) == 0
            src, dst = B.spec_pool_block_table(pool, 0)[full:full + 1], B.spec_pool_block_table(pool, 1)[full:full + 1]
            assert src != dst
            B.spec_kv_copy_pages(view, T.dev(src), T.dev(dst), 1, err, 0)
            seqs, lens, text = [0, 1], lens * 2, [text[0], text[0][:-1] + [(text[0][-1] + 1) % V]]
    assert text[0] != text[1]
    B.spec_pool_destroy(pool)


# ---- calls that the entry points allow and nothing above makes -------------------
@pytest.mark.parametrize("dtype,G,hkv,d,page,max_nodes,layers", [
    (T.BF16, 3, 2, 128, 16, 64, 1), (T.BF16, 5, 2, 64, 80, 13, 1), (T.BF16, 7, 1, 128, 144, 64, 2), (T.BF16, 25, 1, 64, 16, 64, 1),
    (T.BF16, 33, 1, 128, 256, 9, 1), (T.BF16, 127, 1, 64, 16, 5, 1), (T.BF16, 128, 1, 128, 32, 64, 1), (T.BF16, 2, 3, 64, 16, 1, 1),
    (T.BF16, 6, 2, 128, 112, 43, 1), (T.F32, 3, 2, 128, 80, 64, 1), (T.F32, 33, 1, 64, 16, 11, 2), (T.F32, 128, 1, 64, 256, 3, 1)])
def test_attention_odd_groups_and_pages(dtype, G, hkv, d, page, max_nodes, layers):
    """Head groups that share no factor with a tile's rows, trees of every width
    up to the widest, pages longer than a tile and not powers of two."""
    rng = np.random.default_rng(G)
    nodes = sorted({1, 2, max_nodes // 2, max_nodes - 1, max_nodes} & set(range(1, max_nodes + 1)))
    lens = [int(rng.integers(0, 700)) for _ in nodes]
    lens[0], lens[-1] = 0, page
    c = T.Cache(rng, lens, nodes, dtype=dtype, layers=layers, hkv=hkv, d=d, page=page, seed=G)
    parents = np.stack([np.resize(T.rand_parents(rng, k, forest=True), max_nodes) for k in nodes])
    q = _q(G, len(lens), max_nodes, G * hkv, d, dtype, sharp=2.0)
    out, err = T.attention(c, layers - 1, q, lens, nodes, parents, 0.11)
    assert err == 0
    _check(c, layers - 1, q, lens, nodes, parents, out, 0.11)


@pytest.mark.parametrize("dtype", [T.F32, T.BF16])
@pytest.mark.parametrize("live", [[], [0], [1029], [3, 4, 300, 301, 302, 640, 999]])
def test_attention_and_commit_of_a_mostly_padded_batch(dtype, live):
    """More sequences than a block has threads, nearly all of them padded."""
    import torch
    rng = np.random.default_rng(9)
    S, k = 1030, 6
    lens, nodes = np.full(S, 5, np.int32), np.zeros(S, np.int32)
    for s in live:
        lens[s], nodes[s] = rng.integers(0, 400), rng.integers(1, k + 1)
    c = T.Cache(rng, np.where(nodes > 0, lens, 0).tolist(), nodes.tolist(), dtype=dtype, layers=1, hkv=2, d=64, page=16)
    if not live:
        c.bt.fill_(-1)
    parents = np.stack([T.rand_parents(rng, int(n))[:k] for n in nodes])
    q = _q(1, S, k, 6, 64, dtype)
    out, err = T.attention(c, 0, q, lens.tolist(), nodes.tolist(), parents, 0.125)
    assert err == 0
    _check(c, 0, q, lens.tolist(), nodes.tolist(), parents, out, 0.125)
    tokens, target = rng.integers(0, 3, (S, k)).astype(np.int32), rng.integers(0, 3, (S, k)).astype(np.int32)
    before = c.kv.clone()
    acc, tok, ln, path, err = _commit(c, tokens, parents, target, lens, nodes)
    assert err == 0
    pad = nodes == 0
    assert (acc[pad] == -1).all() and (ln[pad] == 5).all() and (path[pad] == -1).all()
    for s in live:
        p = T.ref_walk(parents[s], tokens[s], target[s], int(nodes[s]))
        assert acc[s] == len(p) - 1 and ln[s] == lens[s] + len(p)
    if not live:
        assert bool(torch.equal(c.kv.nan_to_num(3.0), before.nan_to_num(3.0)))


@pytest.mark.parametrize("dtype", [T.F32, T.BF16])
def test_attention_in_place(dtype):
    """The result over its own queries: rows in row tiles of several kinds, alone and shared between blocks."""
    rng = np.random.default_rng(2)
    lens, nodes = [1900, 40, 0, 260] * 8, [64, 5, 64, 33] * 8
    c = T.Cache(rng, lens, nodes, dtype=dtype, layers=1, hkv=2, d=128, page=16)
    parents = np.stack([T.rand_parents(rng, k) for k in nodes])
    q = _q(3, len(lens), T.N, 12, 128, dtype)
    out, err = T.attention(c, 0, q, lens, nodes, parents, 0.09)
    assert err == 0
    both = q.clone()
    T.attention(c, 0, both, lens, nodes, parents, 0.09, out=both)
    for s, k in enumerate(nodes):
        assert bool((both[s, :k] == out[s, :k]).all()) and bool((both[s, k:] == q[s, k:]).all())


def test_two_calls_at_once():
    """Attention, and log probabilities, twice at the same time on two streams with a workspace each."""
    import torch
    from lossless_speculative_decoding_gb300 import binding as B
    rng = np.random.default_rng(5)
    lens, nodes = [700, 64, 2100, 5] * 4, [9, 64, 17, 40] * 4
    c = T.Cache(rng, lens, nodes, dtype=T.BF16, layers=2, hkv=4, d=128, page=16)
    parents = np.stack([T.rand_parents(rng, k) for k in nodes])
    S, V = len(lens), 70001
    q = [_q(i, S, T.N, 8, 128, T.BF16) for i in range(2)]
    x = [torch.randn((3, V), device="cuda", generator=torch.Generator(device="cuda").manual_seed(i)) for i in range(2)]
    want = [T.attention(c, i, q[i], lens, nodes, parents, 0.09)[0] for i in range(2)]
    args = (T.dev(lens), T.dev(nodes), T.dev(parents))
    nb, nl = B.spec_tree_attention_ws_bytes(c.view, S, T.N, 8), B.spec_token_logprobs_ws_bytes(3, V, 9)
    ws = [torch.empty(nb, dtype=torch.uint8, device="cuda") for _ in range(2)]
    wl = [torch.zeros(nl, dtype=torch.uint8, device="cuda") for _ in range(2)]
    out = [torch.full_like(q[0], 77.0) for _ in range(2)]
    ids = [torch.zeros((3, 9), dtype=torch.int32, device="cuda") for _ in range(2)]
    top, ent = [torch.zeros((3, 9), device="cuda") for _ in range(2)], [torch.zeros(3, device="cuda") for _ in range(2)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    st = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for turn in range(6):
        for i in range(2):
            B.spec_tree_attention(c.view, i, q[i], S, T.N, 8, *args, 0.09, out[i], ws[i], nb, err, st[i].cuda_stream)
            B.spec_token_logprobs(x[i], T.F32, V, 3, V, None, 1.0, 9, None, ent[i], None, ids[i], top[i], wl[i], nl,
                                  st[i].cuda_stream)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for i in range(2):
        assert bool((out[i] == want[i]).all())
        ref = torch.log_softmax(x[i].double(), -1)
        v, k = ref.sort(dim=-1, descending=True, stable=True)
        assert bool((ids[i] == k[:, :9]).all())
        e = 8 * 8 * 2.0 ** -24 + 2.0 ** -21 + V * 2.0 ** -24              # |x| < 8: as in the log probabilities' own tests
        assert float((top[i].double() - v[:, :9]).abs().max()) <= e + 16 * 2.0 ** -23


def test_a_captured_step_replayed():
    """Attention, commit and log probabilities of a step in one graph; the
    lengths are handed on between replays, so that each replay commits behind
    the one before it."""
    import torch
    from lossless_speculative_decoding_gb300 import binding as B
    rng = np.random.default_rng(15)
    S, k, V = 3, 8, 900
    start = [10, 47, 16]
    c = T.Cache(rng, [n + 40 for n in start], [k] * S, dtype=T.BF16, layers=2, hkv=2, d=64, page=16, junk=0.0)
    parents = np.stack([T.rand_parents(rng, k)[:k] for _ in range(S)])
    q = _q(1, S, k, 8, 64, T.BF16)
    out = torch.full_like(q, 77.0)
    lens, new, nodes, par = T.dev(start), T.dev(start), T.dev([k] * S), T.dev(parents)
    tokens, target = (torch.zeros((S, k), dtype=torch.int32, device="cuda") for _ in range(2))
    acc, tok = (torch.zeros(S, dtype=torch.int32, device="cuda") for _ in range(2))
    path, err = torch.zeros((S, k), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    logits = torch.randn((S * k, V), device="cuda")
    lp = torch.zeros(S * k, device="cuda")
    nb, nl = B.spec_tree_attention_ws_bytes(c.view, S, k, 8), B.spec_token_logprobs_ws_bytes(S * k, V, 0)
    ws, wl = torch.empty(nb, dtype=torch.uint8, device="cuda"), torch.zeros(nl, dtype=torch.uint8, device="cuda")
    st = torch.cuda.Stream()

    def step():
        p = st.cuda_stream
        B.spec_tree_attention(c.view, 1, q, S, k, 8, lens, nodes, par, 0.125, out, ws, nb, err, p)
        B.spec_tree_commit(c.view, S, k, tokens, par, nodes, target, lens, acc, tok, path, new, err, p)
        B.spec_token_logprobs(logits, T.F32, V, S * k, V, target, 1.0, 0, lp, None, None, None, None, wl, nl, p)

    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        step()
    for turn in range(3):
        ids = [rng.integers(0, 3, (S, k)).astype(np.int32) for _ in range(2)]
        tokens.copy_(T.dev(ids[0])), target.copy_(T.dev(ids[1]))
        n = lens.cpu().numpy()
        kv = c.kv.clone()
        g.replay()
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        for s in range(S):
            rows = kv[c.bt[s].long().clamp(min=0)].permute(0, 4, 1, 2, 3, 5).reshape(-1, 2, 2, 2, 64).double()[:n[s] + k]
            ref, tol = T.ref_attention(rows, 1, q[s], int(n[s]), k, parents[s], 0.125)
            assert bool(((out[s].double() - ref).abs() <= HALF[T.BF16] * ref.abs() + tol).all())
            p = T.ref_walk(parents[s], ids[0][s], ids[1][s], k)
            assert int(new[s]) == n[s] + len(p) and path[s].tolist() == p + [-1] * (k - len(p))
            for j, i in enumerate(p):
                a, b = n[s] + i, n[s] + j
                assert bool((c.kv[c.table[s, b // 16], :, :, :, b % 16] == kv[c.table[s, a // 16], :, :, :, a % 16]).all())
        want = torch.log_softmax(logits.double(), -1).gather(1, target.view(-1, 1).long())[:, 0]
        assert float((lp.double() - want).abs().max()) <= 8 * 6 * 2.0 ** -24 + 2.0 ** -21 + V * 2.0 ** -24 + 16 * 2.0 ** -23
        lens.copy_(new)


def test_copy_pages_of_equal_ids_and_one_source():
    import torch
    from lossless_speculative_decoding_gb300 import binding as B
    kv = torch.randn((6, 2, 2, 2, 16, 64), device="cuda")
    want = kv.clone()
    want[[1, 2, 5]] = kv[4]
    view = B.make_kv_view(kv, None, dtype=T.F32, n_pages=6, n_layers=2, n_kv_heads=2, page_size=16, head_dim=64, max_pages=0)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.spec_kv_copy_pages(view, T.dev([4, 3, 4, 4, 4]), T.dev([1, 3, 2, 4, 5]), 5, err, 0)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and bool(torch.equal(kv, want))


@pytest.mark.parametrize("dtype", [T.F32, T.BF16])
@pytest.mark.parametrize("hq,nodes", [(4, 7), (4, 24), (8, 24), (24, 10)])
def test_attention_scores_that_jump(dtype, hq, nodes):
    """Scores that rise by hundreds within a tile, fall again, and rise in other
    places for other rows: the running maximum moves within and between tiles,
    over weights and sums that are already there."""
    import torch
    rng = np.random.default_rng(hq)
    lens, ks = [0, 300, 1111, 40], [nodes, nodes, max(1, nodes // 2), 3]
    c = T.Cache(rng, lens, ks, dtype=dtype, layers=1, hkv=2, d=64, page=16, seed=5)
    parents = np.stack([T.rand_parents(rng, k) for k in ks])
    u = torch.randn((2, 64), device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    td = torch.float32 if dtype == T.F32 else torch.bfloat16
    for s in range(4):
        t = lens[s] + ks[s]
        pos = torch.arange(t, device="cuda")
        step = torch.floor(pos / 23) * ((pos // 200) % 2 * -2 + 1)     # up for 200 keys, down for 200, a step each 23 keys
        k = (step[:, None] * u[0] * 0.2 + (pos % 50)[:, None] * u[1] * 0.05).to(td)
        pg = c.bt[s].long()[pos // 16]
        c.kv[pg, 0, 1, 0, pos % 16] = k
        c.rows[s][:, 0, 1, 0] = k.double()
    q = _q(4, 4, T.N, hq, 64, dtype)
    q[:, :, hq // 2:] = (q[:, :, hq // 2:] * 0.1 + u[0] * 1.5).to(td)
    q[:, 1::3, hq // 2:] = (-u[0] + u[1] * 2).to(td)                   # other rows: the other way
    out, err = T.attention(c, 0, q, lens, ks, parents, 0.5)
    assert err == 0
    _check(c, 0, q, lens, ks, parents, out, 0.5)


def test_attention_of_large_values():
    """Values of 1e35 on some positions and 1e-35 on others: weights near 2^9 times
    them stay in range, and the sums are those of the formula."""
    import torch
    rng = np.random.default_rng(21)
    lens, nodes = [700, 130], [20, 64]
    c = T.Cache(rng, lens, nodes, dtype=T.BF16, layers=1, hkv=2, d=64, page=16, seed=2)
    parents = np.stack([T.rand_parents(rng, k) for k in nodes])
    for s in range(2):
        pos = torch.arange(lens[s] + nodes[s], device="cuda")
        size = torch.where(pos % 7 < 3, 1e35, 1e-35)[:, None, None]
        v = (c.rows[s][:, 0, :, 1] * size).to(torch.bfloat16)
        c.kv[c.bt[s].long()[pos // 16], 0, :, 1, pos % 16] = v
        c.rows[s][:, 0, :, 1] = v.double()
    q = _q(6, 2, T.N, 4, 64, T.BF16, sharp=4.0)
    out, err = T.attention(c, 0, q, lens, nodes, parents, 0.3)
    assert err == 0 and bool(torch.isfinite(out[0, :20].float()).all())
    _check(c, 0, q, lens, nodes, parents, out, 0.3)
