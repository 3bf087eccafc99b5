"""Entry points for chunks of new tokens where sizes, places and order are unusual: offsets past 32 bits, empty
batches, captures, two calls at once, arrays used in place."""
import numpy as np
import pytest

from _chunk import (BF16, F32, Cache, Rows, attention, check_attention, dev, evict, mass, queries, ref_attention, ref_keep,
                    ref_mass, scores)

pytestmark = pytest.mark.gpu


def _cache(lens, new, dtype=BF16, **kw):
    a = dict(layers=1, hkv=2, d=128, page=16)
    a.update(kw)
    return Cache(np.random.default_rng(3), lens, new, dtype=dtype, **a)


# --------------------------------------------------------------------------- offsets past 32 bits
class FarCache:
    """Two sequences whose pages lie at both ends of a pool of more than 2^32 values (the rest is not initialised)."""

    def __init__(self, lens, new, dtype, layers=2, hkv=8, d=128, page=64):
        import torch
        from lossless_speculative_decoding_gb300 import binding as B
        td = torch.float32 if dtype == F32 else torch.bfloat16
        per = layers * hkv * 2 * page * d
        self.n_pages = 2 ** 32 // per + 40
        self.P, self.d, self.hkv, self.layers = page, d, hkv, layers
        self.kv = torch.empty((self.n_pages, layers, hkv, 2, page, d), dtype=td, device="cuda")
        tot = [n + m for n, m in zip(lens, new)]
        need = [-(-t // page) for t in tot]
        self.max_pages = max(need)
        self.table = np.full((len(lens), self.max_pages), -1, np.int32)
        gen = torch.Generator(device="cuda").manual_seed(1)
        self.rows = []
        for s, t in enumerate(tot):
            ids = np.arange(need[s]) * 2 + s                       # sequence by sequence, one at the start, one at the end
            if s % 2 == 0:
                ids = self.n_pages - 1 - ids
            self.table[s, :need[s]] = ids
            r = torch.randn((t, layers, hkv, 2, d), generator=gen, device="cuda").to(td)
            pos = torch.arange(t, device="cuda")
            self.kv[torch.from_numpy(self.table[s].astype(np.int64)).cuda()[pos // page], :, :, :, pos % page] = r
            self.rows.append(r.double())
        self.bt = torch.from_numpy(self.table).cuda()
        self.view = B.make_kv_view(self.kv, self.bt, dtype=dtype, n_pages=self.n_pages, n_layers=layers, n_kv_heads=hkv,
                                   page_size=page, head_dim=d, max_pages=self.max_pages)

    def slots(self, s, n):
        import torch
        pos = torch.arange(n, device="cuda")
        return self.kv[torch.from_numpy(self.table[s].astype(np.int64)).cuda()[pos // self.P], :, :, :, pos % self.P]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("most", [3, 90])
def test_a_cache_of_more_than_2_to_32_values(dtype, most):
    """All four operators on pages at both ends of the pool."""
    import torch
    from lossless_speculative_decoding_gb300 import binding as B
    lens, new = [200, 130], [most, most]
    c = FarCache(lens, new, dtype)
    rows = Rows(new)
    q = queries(rows, 16, 128, dtype, 4)
    out, lse, err = attention(c, 1, q, rows, lens, 0.09)
    assert err == 0
    check_attention(c, 1, q, rows, lens, 0.09, out, lse, one_part=dtype == BF16 and most > 64)
    got, err = mass(c, 1, q, lse, rows, lens, 0.09, most)
    assert err == 0
    for s in range(2):
        w, e = ref_mass(c, s, 1, q[rows.of(s)], lse[rows.of(s)], lens[s], most, 0.09, most)
        assert bool(((got[s, :, :lens[s] + most].double() - w).abs() <= w * e + 1e-37).all())
    before = [c.slots(s, lens[s]).clone() for s in range(2)]
    x = torch.rand((2, 2, 8, 210), device="cuda")
    _, kept, ln, err = evict(c, lens, x, 100, 9)
    assert err == 0 and ln.tolist() == [100, 100]
    for s in range(2):
        now = c.slots(s, 100)
        for layer in range(2):
            for h in range(8):
                keep = ref_keep(x[layer, s, h].cpu().numpy(), lens[s], 100, 9)
                assert np.array_equal(kept[layer, s, h], keep)
                assert torch.equal(now[:, layer, h], before[s][torch.from_numpy(keep).cuda(), layer, h])
    # new rows behind the kept ones
    x = torch.randn((rows.n, 32, 128), device="cuda").to(q.dtype)
    o = torch.zeros((rows.n, 16, 128), device="cuda", dtype=q.dtype)
    e = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.spec_qk_norm_rope(c.view, 1, x, 32 * 128, rows.n, 2, 16, dev(rows.start), dev(rows.new), dev([100, 100]), B.make_rope([]), None,
                        None, None, 0.0, o, e, 0)
    torch.cuda.synchronize()
    assert int(e.item()) == 0 and torch.equal(o[:2 * most], x[:2 * most, :16])
    for s in range(2):
        got = c.slots(s, 100 + most)[100:, 1]
        assert torch.equal(got[:, :, 0], x[rows.of(s), 16:24]) and torch.equal(got[:, :, 1], x[rows.of(s), 24:])


def test_rows_2_to_31_values_apart():
    """qkv rows with a stride past 2^31 values."""
    import torch
    from lossless_speculative_decoding_gb300 import binding as B
    ld = 2 ** 31 + 64
    c = _cache([5], [3])
    wide = torch.empty(2 * ld + 6 * 128, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(wide, (3, 6, 128), (ld, 128, 1))
    x.copy_(torch.randn((3, 6, 128), device="cuda"))
    q = torch.zeros((3, 2, 128), dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.spec_qk_norm_rope(c.view, 0, wide, ld, 3, 1, 2, dev([0]), dev([3]), dev([5]), B.make_rope([]), None, None, None, 0.0, q, err, 0)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and torch.equal(q, x[:, :2])


@pytest.mark.parametrize("most", [4, 70])
def test_rows_past_2_to_31_values(most):
    """Queries, results, lse and mass at the end of arrays of more than 2^31 values."""
    import torch
    lens, new = [50, 7], [most, most]
    c = _cache(lens, new, hkv=4)
    n = 2 ** 31 // (32 * 128) + 2 * most + 5
    q = torch.empty((n, 32, 128), dtype=torch.bfloat16, device="cuda")
    rows = Rows(new)
    rows.start = [n - 2 * most - 1, n - most - 1]
    rows.n = n
    for s in range(2):
        q[rows.of(s)] = torch.randn((most, 32, 128), device="cuda").bfloat16()
    out, lse, err = attention(c, 0, q, rows, lens, 0.09, out=torch.empty_like(q))
    assert err == 0
    for s in range(2):
        o, z, e, ez = ref_attention(c, s, 0, q[rows.of(s)], lens[s], most, 0.09, True)
        assert bool(((out[rows.of(s)].double() - o).abs() <= e + o.abs() * 2.0 ** -8).all())
        assert float((lse[rows.of(s)].double() - z).abs().max()) <= ez
    ld = 2 ** 28 + 1                                               # 2 sequences x 4 heads: the last row starts past 2^31 - 2^28
    got = torch.empty((2, 4, ld), device="cuda")
    got, err = mass(c, 0, q, lse, rows, lens, 0.09, most, out=got, ld=ld)
    assert err == 0
    for s in range(2):
        w, e = ref_mass(c, s, 0, q[rows.of(s)], lse[rows.of(s)], lens[s], most, 0.09, most)
        assert bool(((got[s, :, :lens[s] + most].double() - w).abs() <= w * e + 1e-37).all())


# --------------------------------------------------------------------------- nothing to do
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n_seq", [1, 3, 40, 3000])
@pytest.mark.parametrize("max_new", [1, 500])
def test_batches_of_padded_sequences(dtype, n_seq, max_new):
    """No sequence has tokens (their other sizes may be anything): nothing is written, nothing is reported."""
    import torch
    from lossless_speculative_decoding_gb300 import binding as B
    c = _cache([5], [3], dtype)
    td = c.kv.dtype
    bt = torch.full((n_seq, 4), -1, dtype=torch.int32, device="cuda")
    view = B.make_kv_view(c.kv, bt, dtype=dtype, n_pages=c.n_pages, n_layers=1, n_kv_heads=2, page_size=16, head_dim=128, max_pages=4)
    q = torch.randn((9, 4, 128), device="cuda").to(td)
    zero, junk = dev([0] * n_seq), dev([-5, 10 ** 9, 7] * n_seq)[:n_seq].contiguous()
    out, lse = torch.full_like(q, 77.0), torch.full((9, 4), 77.0, device="cuda")
    nb = B.spec_chunk_attention_ws_bytes(view, n_seq, max_new, 4)
    ws = torch.full((nb,), 0xA5, dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.spec_chunk_attention(view, 0, q, 9, n_seq, max_new, 4, junk, zero, junk, 0.1, out, lse, ws, nb, err, 0)
    m = torch.full((n_seq, 2, 8), 77.0, device="cuda")
    B.spec_attention_mass(view, 0, q, lse, 9, n_seq, max_new, max_new, 4, junk, zero, junk, 0.1, None, m, 8, err, 0)
    x = torch.randn((9, 8, 128), device="cuda").to(td)
    before = c.kv.clone()
    B.spec_qk_norm_rope(view, 0, x, 1024, 9, n_seq, 4, junk, zero, junk, B.make_rope([1.0] * 8), torch.zeros((1, 9), dtype=torch.int32,
                        device="cuda"), None, None, 0.0, out, err, 0)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert bool((out == 77).all()) and bool((lse == 77).all()) and bool((m == 77).all())
    assert torch.equal(c.kv.nan_to_num(5.0), before.nan_to_num(5.0))
    # no positions at all: everything (nothing) is kept
    o, kept, ln, e = evict(Cache(np.random.default_rng(1), [0, 0], [1, 1], dtype=dtype, layers=1, hkv=2, d=64, page=16), [0, 0],
                           torch.ones((1, 2, 2, 4), device="cuda"), 3, 1)
    assert e == 0 and ln.tolist() == [0, 0] and (kept == -1).all() and (o == 77).all()


def test_one_token_alone():
    """The first token of an empty cache: its own value, and the whole weight on itself."""
    import torch
    for dtype in (BF16, F32):
        for most in (1, 300):                                      # (the form for long chunks too)
            c = _cache([0], [1], dtype)
            rows = Rows([1])
            q = queries(rows, 4, 128, dtype, 1)
            out, lse, err = attention(c, 0, q, rows, [0], 0.1, max_new=most)
            assert err == 0
            v = c.rows[0][0, 0, :, 1].repeat_interleave(2, 0).to(q.dtype)
            # the one weight p meets 1 / sum of fp32 weights = 1 / p. fp32: three roundings. bf16: p in 16 bits leaves v its
            # nearest neighbour; p rounded to bf16 is off by 2^-8, and so is the result's rounding
            bound = 3 * 2.0 ** -24 if dtype == F32 else 0 if most == 1 else 2 * 2.0 ** -8 + 2.0 ** -16
            assert bool(((out[0].double() - v.double()).abs() <= v.double().abs() * bound).all())
            m, err = mass(c, 0, q, lse, rows, [0], 0.1, most, max_new=most)
            assert err == 0 and float((m[0, :, 0] - 2).abs().max()) <= 64 * 2.0 ** -24 * (2 + float(lse[0].abs().max()))


# --------------------------------------------------------------------------- captures, streams, arrays in place
def test_a_captured_step_on_two_streams():
    """Two decoders' steps, captured, replayed on two streams at once with a workspace each, give what eager calls on
    one stream give: rotation, attention, mass in place, eviction into a second array."""
    import torch
    from lossless_speculative_decoding_gb300 import binding as B
    lens, new = [90, 33, 150], [1, 70, 4]

    def world(seed):
        c = Cache(np.random.default_rng(seed), lens, new, dtype=BF16, layers=2, hkv=2, d=128, page=16, seed=seed)
        rows = Rows(new)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        t = dict(c=c, rows=rows, x=torch.randn((rows.n, 8, 128), generator=gen, device="cuda").bfloat16())
        t.update(start=dev(rows.start), m=dev(new), n=dev(lens), n2=dev([0] * 3), q=torch.zeros((rows.n, 4, 128), device="cuda").bfloat16())
        t.update(out=torch.zeros_like(t["q"]), z=torch.zeros((rows.n, 4), device="cuda"), err=dev([0]), pos=dev(np.arange(rows.n)[None]))
        t.update(mass=torch.rand((2, 3, 2, 160), generator=gen, device="cuda"), mass2=torch.zeros((2, 3, 2, 160), device="cuda"))
        t.update(kept=torch.zeros((2, 3, 2, 40), dtype=torch.int32, device="cuda"), rope=B.make_rope([0.5 ** i for i in range(64)]))
        t["nb"] = B.spec_chunk_attention_ws_bytes(c.view, 3, 70, 4)
        t["ws"] = torch.empty(t["nb"], dtype=torch.uint8, device="cuda")
        return t

    def step(t, st):
        v, r = t["c"].view, t["rows"]
        for layer in range(2):
            B.spec_qk_norm_rope(v, layer, t["x"], 1024, r.n, 3, 4, t["start"], t["m"], t["n"], t["rope"], t["pos"], None, None, 1e-6,
                                t["q"], t["err"], st)
            B.spec_chunk_attention(v, layer, t["q"], r.n, 3, 70, 4, t["start"], t["m"], t["n"], 0.1, t["out"], t["z"], t["ws"], t["nb"],
                                   t["err"], st)
            B.spec_attention_mass(v, layer, t["q"], t["z"], r.n, 3, 70, 70, 4, t["start"], t["m"], t["n"], 0.1, t["mass"][layer],
                                  t["mass"][layer], 160, t["err"], st)
        B.spec_kv_evict(v, 3, t["n"], t["mass"], 160, 40, 4, t["mass2"], t["kept"], t["n2"], t["err"], st)

    want = [world(s) for s in (1, 2)]
    for t in want:
        step(t, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    got = [world(s) for s in (1, 2)]
    saved = [(t["c"].kv.clone(), t["mass"].clone()) for t in got]
    streams, graphs = [torch.cuda.Stream() for _ in got], []
    torch.cuda.synchronize()
    for t, st in zip(got, streams):
        with torch.cuda.stream(st):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                step(t, st.cuda_stream)
            graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(4):
        for t, (kv, ms) in zip(got, saved):
            t["c"].kv.copy_(kv)
            t["mass"].copy_(ms)
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for k in ("q", "out", "z", "kept", "n2", "err"):
                assert torch.equal(a[k], b[k]), k
            assert torch.equal(a["c"].kv.nan_to_num(5.0), b["c"].kv.nan_to_num(5.0))
            for k in ("mass", "mass2"):
                assert torch.equal(a[k], b[k]), k
            assert int(a["err"].item()) == 0


def test_rotation_for_a_tree():
    """Rows of [sequence][node] with n_nodes as n_new: the nodes' keys and values where the tree attention reads them,
    each node at its depth's position."""
    import torch
    from _tree import N, attention as tree_attention, rand_parents
    from lossless_speculative_decoding_gb300 import binding as B
    rng = np.random.default_rng(1)
    lens, nodes = [40, 7], [9, 30]
    c = Cache(rng, lens, nodes, dtype=F32, layers=1, hkv=2, d=64, page=16)
    parents = np.stack([rand_parents(rng, k) for k in nodes])
    depth = np.zeros((2, N), np.int64)
    for s, k in enumerate(nodes):
        for i in range(1, k):
            depth[s, i] = depth[s, parents[s, i]] + 1
    x = torch.randn((2 * N, 8, 64), device="cuda")
    pos = (np.array(lens)[:, None] + depth).reshape(1, -1).astype(np.int32)
    q = torch.zeros((2 * N, 4, 64), device="cuda")
    err = dev([0])
    freq = 1e4 ** (-np.arange(32) / 32)
    B.spec_qk_norm_rope(c.view, 0, x, 512, 2 * N, 2, 4, dev([0, N]), dev(nodes), dev(lens), B.make_rope(freq), dev(pos), None, None,
                        0.0, q, err, 0)
    torch.cuda.synchronize()
    out, e = tree_attention(c, 0, q.view(2, N, 4, 64), lens, nodes, parents, 0.125)
    assert int(err.item()) == 0 and e == 0
    angle = torch.from_numpy(pos[0][:, None] * freq).cuda()[:, None]
    z = torch.complex(x[:, :6, :32].double(), x[:, :6, 32:].double()) * torch.polar(torch.ones_like(angle), angle)
    z = torch.cat([z.real, z.imag], -1)
    for s, (n, k) in enumerate(zip(lens, nodes)):
        K = torch.cat([c.rows[s][:n, 0, :, 0], z[s * N:s * N + k, 4:]])
        V = torch.cat([c.rows[s][:n, 0, :, 1], x[s * N:s * N + k, 6:].double()])
        qq = z[s * N:s * N + k, :4].view(k, 2, 2, 64)
        t = torch.einsum("ihgd,jhd->hgij", qq, K) * 0.125
        see = np.zeros((k, n + k), bool)
        see[:, :n] = True
        for i in range(k):
            j = i
            while j >= 0:
                see[i, n + j] = True
                j = int(parents[s, j])
        w = torch.softmax(t.masked_fill(~torch.from_numpy(see).cuda(), float("-inf")), -1)
        o = torch.einsum("hgij,jhd->ihgd", w, V).reshape(k, 4, 64)
        assert float((out[s, :k].double() - o).abs().max()) <= 1e-4 * float(V.abs().max())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_mass_with_weights_of_far_apart_rows(dtype):
    """Rows of one unit whose lse lie far apart, sharp and flat ones: each row's weights sum to 1."""
    import torch
    n, m = 300, 40
    c = _cache([n], [m], dtype, hkv=1)
    rows = Rows([m])
    q = queries(rows, 8, 128, dtype, 9, sharp=25.0)
    scale = 128 ** -0.5
    x, mag = scores(c, 0, 0, q[:m], n, m, scale)
    lse = torch.zeros((rows.n, 8), device="cuda")
    lse[:m] = torch.logsumexp(x, -1).permute(2, 0, 1).reshape(m, 8).float()
    assert float(lse[:m].max() - lse[:m].min()) > 30
    got, err = mass(c, 0, q, lse, rows, [n], scale, m)
    w, e = ref_mass(c, 0, 0, q[:m], lse[:m], n, m, scale, m)
    assert err == 0 and bool(((got[0, :, :n + m].double() - w).abs() <= w * e + 1e-30).all())


@pytest.mark.parametrize("hkv", [1, 2])
def test_mass_of_a_prompt_beside_short_chunks(hkv):
    """Units of many tiles of rows and of one to five side by side: what two blocks share, and what one has alone."""
    import torch
    rng = np.random.default_rng(11)
    lens = [2000] + [int(x) for x in rng.integers(3000, 9000, 15)]
    new = [200] + [int(x) for x in rng.integers(1, 80, 15)]
    c = _cache(lens, new, hkv=hkv)
    rows = Rows(new)
    q = queries(rows, 8 * hkv, 128, BF16, 5)
    scale = 128 ** -0.5
    lse = torch.zeros((rows.n, 8 * hkv), device="cuda")
    for s, n in enumerate(lens):
        x, _ = scores(c, s, 0, q[rows.of(s)], n, new[s], scale)
        lse[rows.of(s)] = torch.logsumexp(x, -1).permute(2, 0, 1).reshape(new[s], 8 * hkv).float()
    first, err = mass(c, 0, q, lse, rows, lens, scale, 200)
    assert err == 0
    for s, n in enumerate(lens):
        w, e = ref_mass(c, s, 0, q[rows.of(s)], lse[rows.of(s)], n, new[s], scale, 200)
        assert bool(((first[s, :, :n + new[s]].double() - w).abs() <= w * e + 1e-37).all()), s
    for _ in range(20):
        got, err = mass(c, 0, q, lse, rows, lens, scale, 200)
        assert err == 0 and torch.equal(got, first)
