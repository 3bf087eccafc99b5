"""Entry points for chunks of new tokens against plain implementations in 64 bits."""
import numpy as np
import pytest

from _chunk import (BF16, F32, Cache, Rows, attention, check_attention, dev, evict, mass, queries, ref_keep, ref_mass, scores,
                    slots)

pytestmark = pytest.mark.gpu


def narrow(dtype, rows, G, max_new=None):
    """Weights enter the sum of values with 16 bits or more (the rule that the header states)."""
    most = rows.most if max_new is None else max_new
    return dtype == F32 or (most <= 64 and most * G <= 128)


def build(rng, lens, new, *, dtype, hq, hkv, d, page, layers=2, gap=0, seed=0, sharp=2.0):
    c = Cache(rng, lens, new, dtype=dtype, layers=layers, hkv=hkv, d=d, page=page, seed=seed)
    rows = Rows(new, gap)
    return c, rows, queries(rows, hq, d, dtype, seed + 1, sharp)


# --------------------------------------------------------------------------- attention
SHAPES = [(10, 10, 128), (32, 8, 128), (4, 4, 64), (16, 2, 64), (12, 1, 128), (15, 3, 64), (7, 1, 128), (128, 1, 64)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("page,lens,new", [
    (16, [0, 1, 40, 333], [1, 1, 1, 1]),                                  # single tokens
    (48, [5, 0, 127, 300, 64], [3, 17, 1, 0, 33]),                        # a few, one sequence padded
    (64, [0, 129, 0, 700], [65, 128, 129, 1]),                            # around a tile of keys, mixed with decoding
    (16, [31, 2], [300, 257]),                                            # longer than a row tile
])
def test_attention(dtype, shape, page, lens, new):
    import torch
    hq, hkv, d = SHAPES[shape]
    rng = np.random.default_rng(shape * 10 + page)
    c, rows, q = build(rng, lens, new, dtype=dtype, hq=hq, hkv=hkv, d=d, page=page, gap=1)
    scale = d ** -0.5
    out, lse, err = attention(c, 1, q, rows, lens, scale)
    assert err == 0
    check_attention(c, 1, q, rows, lens, scale, out, lse, one_part=not narrow(dtype, rows, hq // hkv))
    again, lse2, _ = attention(c, 1, q, rows, lens, scale)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    # in place, without lse
    q2 = q.clone()
    attention(c, 1, q2, rows, lens, scale, out=q2, lse=False)
    for s in range(len(lens)):
        assert torch.equal(q2[rows.of(s)], out[rows.of(s)])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("most", [1, 2, 127, 128, 129, 255, 256, 257, 513])
def test_attention_lengths(dtype, most):
    """Every chunk length near a tile's borders, beside a short one, on keys that end in and at a tile."""
    rng = np.random.default_rng(most)
    lens, new = [0, 256 - most if most < 256 else 11, 77], [most, most, 1]
    c, rows, q = build(rng, lens, new, dtype=dtype, hq=4, hkv=2, d=128, page=16, layers=1)
    out, lse, err = attention(c, 0, q, rows, lens, 0.1)
    assert err == 0
    check_attention(c, 0, q, rows, lens, 0.1, out, lse, one_part=not narrow(dtype, rows, 2))


@pytest.mark.parametrize("most", [1, 3, 200])
def test_attention_long_context_is_cut_and_joined(most):
    """One sequence, one kv head: its keys are spread over all blocks."""
    rng = np.random.default_rng(most)
    c, rows, q = build(rng, [20011], [most], dtype=BF16, hq=2, hkv=1, d=128, page=32, layers=1)
    out, lse, err = attention(c, 0, q, rows, [20011], 0.09)
    assert err == 0
    check_attention(c, 0, q, rows, [20011], 0.09, out, lse, one_part=not narrow(BF16, rows, 2))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("most", [1, 130])
def test_attention_many_sequences(dtype, most):
    """More sequences than blocks, most of them padded."""
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 40, 700)
    new = np.where(rng.random(700) < 0.7, 0, rng.integers(1, most + 1, 700))
    c, rows, q = build(rng, lens, new, dtype=dtype, hq=2, hkv=2, d=64, page=16, layers=1)
    out, lse, err = attention(c, 0, q, rows, lens, 0.125)
    assert err == 0
    check_attention(c, 0, q, rows, lens, 0.125, out, lse, one_part=not narrow(dtype, rows, 1))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("most", [2, 150])
@pytest.mark.parametrize("size", [30.0, 3e4, 3e9, 1e15])
def test_attention_scores_of_any_size(dtype, most, size):
    """Scores up to `size`; integers that fp32 holds while it can, so that the largest one is unique in every row: it
    takes all of the weight. (Keys are powers of two in one dim, larger ones later.)"""
    import torch
    d, n = 64, 70
    c = Cache(np.random.default_rng(1), [n], [most], dtype=dtype, layers=1, hkv=1, d=d, page=16)
    T = n + most
    key = torch.zeros((T, d), device="cuda")
    # 2^-x of the largest: with x falling along the row the last visible position wins by at least half its score
    steps = torch.arange(T, device="cuda").float()
    key[:, 0] = torch.where(steps % 7 == 0, -1.0, 1.0) * 2.0 ** torch.floor((steps - T) / 8)
    pg = torch.from_numpy(c.table[0].astype(np.int64)).cuda()
    pos = torch.arange(T, device="cuda")
    c.kv[pg[pos // 16], 0, 0, 0, pos % 16] = key.to(c.kv.dtype)
    c.rows[0][:, 0, 0, 0] = key.double()
    rows = Rows([most])
    q = torch.zeros((rows.n, 2, d), device="cuda", dtype=c.kv.dtype)
    q[:, 0, 0], q[:, 1, 0] = 2.0 ** round(np.log2(size)), -2.0 ** round(np.log2(size))
    out, lse, err = attention(c, 0, q, rows, [n], 1.0)
    assert err == 0 and bool(torch.isfinite(out[:most]).all()) and bool(torch.isfinite(lse[:most]).all())
    x, _ = scores(c, 0, 0, q[:most], n, most, 1.0)
    w = torch.softmax(x, -1)
    o = torch.einsum("hgij,jhd->ihgd", w, c.rows[0][:, 0, :, 1]).reshape(most, 2, d)
    # scores are exact here (one product each); the exponent is off by a rounding of its size where weights are shared
    e = 2.0 ** -8 + 2.0 ** -7 if dtype == BF16 else 0
    tail = (2.0 ** -21 * size) if size < 1e5 else 0     # equal scores share exactly; unequal large ones are worlds apart
    assert float((out[:most].double() - o).abs().max()) <= float(c.rows[0][:, 0, :, 1].abs().max()) * (e + 2 * min(tail, 1) + 1e-5)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_sequences_that_do_not_fit(dtype):
    """Lengths past an array's end are left out and reported, the others are as they would be alone."""
    import torch
    rng = np.random.default_rng(5)
    lens, new = [20, 30, 10, 7, 9, 11], [5, 6, 7, 4, 3, 2]
    c, rows, q = build(rng, lens, new, dtype=dtype, hq=4, hkv=2, d=64, page=16, layers=1)
    want, wl, err = attention(c, 0, q, rows, lens, 0.125)
    assert err == 0
    cap = c.max_pages * 16
    for s, change in [(1, dict(n=-1)), (1, dict(m=-2)), (2, dict(m=8)), (3, dict(r0=-1)), (4, dict(r0=q.shape[0] - 2)),
                      (0, dict(n=cap)), (5, dict(n=2 ** 31 - 1)), (5, dict(r0=2 ** 31 - 1)), (2, dict(m=2 ** 31 - 1)),
                      (2, dict(m=-2 ** 31)), (0, dict(n=-2 ** 31, r0=-2 ** 31))]:
        ll, r2 = list(lens), Rows(new)
        ll[s] = change.get("n", ll[s])
        r2.new[s] = change.get("m", r2.new[s])
        r2.start[s] = change.get("r0", r2.start[s])
        out, lse, err = attention(c, 0, q, r2, ll, 0.125, max_new=7)
        assert err == 4, change
        for i in range(len(lens)):
            if i != s:
                bound = 0.02 if dtype == BF16 else 1e-5      # (another split of the keys)
                assert float((out[rows.of(i)].float() - want[rows.of(i)].float()).abs().max()) <= bound
        assert bool((out[rows.of(s)] == 77).all()) and bool((lse[rows.of(s)] == 77).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("most", [3, 140])
@pytest.mark.parametrize("page_id", [-1, 10 ** 6, -2 ** 31])
def test_attention_bad_page(dtype, most, page_id):
    """A bad page is reported, its sequence's rows come back finite or not, the others are right."""
    rng = np.random.default_rng(6)
    lens, new = [100, 60], [most, most]
    c, rows, q = build(rng, lens, new, dtype=dtype, hq=2, hkv=1, d=64, page=16, layers=1)
    c.bt[0, 2] = page_id
    out, lse, err = attention(c, 0, q, rows, lens, 0.125)
    assert err == 1
    rows1 = Rows(new)
    out[rows.of(0)], lse[rows.of(0)] = 77, 77
    rows1.new[0] = 0
    check_attention(c, 0, q, rows1, lens, 0.125, out, lse, one_part=not narrow(dtype, rows, 2))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("most", [4, 150])
def test_attention_captured_and_replayed(dtype, most):
    """One capture, lengths that change between replays, on a stream of its own."""
    import torch
    from lossless_speculative_decoding_gb300 import binding as B
    rng = np.random.default_rng(8)
    lens, new = [200, 90, 0], [most, 1, most // 2]
    c, rows, q = build(rng, lens, new, dtype=dtype, hq=4, hkv=2, d=128, page=16, layers=1)
    nb = B.spec_chunk_attention_ws_bytes(c.view, 3, most, 4)
    ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    start, mm, nn = dev(rows.start), dev(rows.new), dev(lens)
    out, z, err = torch.empty_like(q), torch.empty((q.shape[0], 4), device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    st = torch.cuda.Stream()

    def call():
        B.spec_chunk_attention(c.view, 0, q, q.shape[0], 3, most, 4, start, mm, nn, 0.1, out, z, ws, nb, err, st.cuda_stream)

    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        call()
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            call()
        for ll, nw in ((lens, new), ([100, 91, 1], [most // 2, 0, 1]), (lens, new)):
            nn.copy_(dev(ll))
            mm.copy_(dev(nw))
            out.fill_(77)
            z.fill_(77)
            g.replay()
            st.synchronize()
            r = Rows(new)
            r.new = nw
            keep = c.rows                                    # (those of the sequence as it is now)
            c.rows = [x[: ll[s] + nw[s]] for s, x in enumerate(keep)]
            check_attention(c, 0, q, r, ll, 0.1, out, z, one_part=not narrow(dtype, rows, 2))
            c.rows = keep
    assert int(err.item()) == 0


# --------------------------------------------------------------------------- norms and rotation
def ref_rope(x, hq, hkv, gammas, eps, angle):
    """float64 rows [n, hq + 2 hkv, d] after norm and rotation; angle [n, half]."""
    import torch
    half = angle.shape[1]
    y = x.double().clone()
    for lo, hi, g in ((0, hq, gammas[0]), (hq, hq + hkv, gammas[1])):
        z = y[:, lo:hi]
        if g is not None:
            z = z / torch.sqrt((z * z).mean(-1, keepdim=True) + eps) * g.double()
        a, b = z[..., :half].clone(), z[..., half:2 * half].clone()
        c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
        z = z.clone()
        z[..., :half], z[..., half:2 * half] = a * c - b * s, b * c + a * s
        y[:, lo:hi] = z
    return y


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("hq,hkv,d,rot,axes,norm,far", [
    (10, 10, 128, 128, 1, True, 0), (32, 8, 128, 128, 3, True, 0), (4, 4, 64, 64, 1, False, 0), (5, 1, 64, 32, 2, True, 0),
    (3, 3, 128, 16, 1, True, 2 ** 31 - 2000), (12, 1, 128, 0, 1, True, 0), (33, 11, 128, 112, 4, False, -2 ** 31),
    (1, 1, 64, 64, 1, True, 65521)])
@pytest.mark.parametrize("lens,new,page,gap", [([37], [1], 16, 0), ([0, 31, 5, 100], [70, 1, 0, 129], 48, 2),
                                              ([3] * 40, [1, 2, 0, 5] * 10, 16, 0)])
def test_rope(dtype, hq, hkv, d, rot, axes, norm, far, lens, new, page, gap):
    import torch
    from lossless_speculative_decoding_gb300 import binding as B
    rng = np.random.default_rng(hq + rot)
    gen = torch.Generator(device="cuda").manual_seed(2)
    td = torch.float32 if dtype == F32 else torch.bfloat16
    c = Cache(rng, lens, new, dtype=dtype, layers=2, hkv=hkv, d=d, page=page)
    rows = Rows(new, gap)
    heads = hq + 2 * hkv
    wide = torch.randn((rows.n, heads + 1, d), generator=gen, device="cuda").mul_(3).to(td)     # rows further apart than long
    x = wide[:, :heads]
    half = rot // 2
    freq = 1e4 ** (-np.arange(half) / max(half, 1))
    axis = rng.integers(0, axes, half)
    pos = (rng.integers(0, 2000, (axes, rows.n)) + far).astype(np.int32)
    gammas = [torch.randn(d, generator=gen, device="cuda") for _ in "qk"] if norm else [None, None]
    if hq == 5:
        gammas[1] = None                                                                        # queries alone
    q = torch.full((rows.n, hq, d), 77.0, device="cuda", dtype=td)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = c.kv.clone()
    B.spec_qk_norm_rope(c.view, 1, x, wide.stride(0), rows.n, len(lens), hq, dev(rows.start), dev(rows.new), dev(lens),
                        B.make_rope(freq, axis=axis, n_axes=axes), dev(pos), gammas[0], gammas[1], 1e-5, q, err, 0)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    angle = torch.from_numpy(pos[axis].T.astype(np.float64) * freq).cuda()
    y = ref_rope(x, hq, hkv, gammas, 1e-5, angle)
    # |x| g: a head's RMS is 1 after the norm, so a normed value is at most sqrt(d) |gamma|; fp32 norm (d + 8 roundings of
    # its sum, halved by the root), rotation (angle 2^-24 of an eighth turn, and 2^-32 of a turn; cos and sin 2^-23) and the
    # products' roundings, against the larger of the pair
    size = y.abs().clone()
    if half:
        pair = torch.maximum(size[..., :half], size[..., half:2 * half]) * 2 ** 0.5
        size[..., :half], size[..., half:2 * half] = pair, pair
    exact = torch.from_numpy(np.abs(pos[axis].T.astype(np.float64)) * freq * 2.0 ** -52).cuda()       # freq's own rounding
    e = size * ((d + 8) * 2.0 ** -25 + 2.0 ** -21)
    if half:
        e[..., :half] += size[..., :half] * exact[:, None]
        e[..., half:2 * half] += size[..., half:2 * half] * exact[:, None]
    if dtype == BF16:
        e = e + y.abs() * 2.0 ** -8
    live = torch.zeros(rows.n, dtype=torch.bool, device="cuda")
    after = c.kv.clone()
    for s, n in enumerate(lens):
        at, m = rows.of(s), rows.new[s]
        if m == 0:
            continue
        live[at] = True
        assert bool(((q[at].double() - y[at, :hq]).abs() <= e[at, :hq]).all()), s
        p = n + torch.arange(m, device="cuda")
        pg = torch.from_numpy(c.table[s].astype(np.int64)).cuda()[p // page]
        got = c.kv[pg, 1, :, :, p % page]                              # [m, hkv, 2, d]
        assert bool(((got[:, :, 0].double() - y[at, hq:hq + hkv]).abs() <= e[at, hq:hq + hkv]).all()), s
        assert torch.equal(got[:, :, 1], x[at, hq + hkv:])
        after[pg, 1, :, :, p % page] = before[pg, 1, :, :, p % page]
    assert bool((q[~live] == 77).all())
    assert torch.equal(after.nan_to_num(5.0), before.nan_to_num(5.0))  # nothing else was written


def test_rope_bad_lengths_and_pages():
    import torch
    from lossless_speculative_decoding_gb300 import binding as B
    lens, new = [20, 17, 6], [30, 4, 2]
    for what, bits in (("page", 1), ("n", 4), ("m", 4), ("r0", 4)):
        c = Cache(np.random.default_rng(1), lens, new, dtype=BF16, layers=1, hkv=2, d=64, page=16)
        rows = Rows(new)
        x = torch.randn((rows.n, 6, 64), device="cuda").bfloat16()
        q = torch.full((rows.n, 2, 64), 77.0, device="cuda", dtype=torch.bfloat16)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        ll, mm, rr = list(lens), list(rows.new), list(rows.start)
        if what == "page":
            c.bt[0, 2] = c.n_pages
        elif what == "n":
            ll[0] = c.max_pages * 16 - 29
        elif what == "m":
            mm[0] = rows.n + 1
        else:
            rr[0] = rows.n - 29
        B.spec_qk_norm_rope(c.view, 0, x, 384, rows.n, 3, 2, dev(rr), dev(mm), dev(ll), B.make_rope([]), None, None, None, 0.0, q,
                            err, 0)
        torch.cuda.synchronize()
        assert int(err.item()) == bits, what
        for s in (1, 2):
            assert torch.equal(q[rows.of(s)], x[rows.of(s), :2])
            assert torch.equal(slots(c, s, lens[s] + new[s])[lens[s]:, 0].transpose(1, 2).reshape(new[s], 4, 64),
                               x[rows.of(s), 2:].double())
        if what == "page":                                             # queries and the slots on good pages are there
            assert torch.equal(q[rows.of(0)], x[rows.of(0), :2])
        else:
            assert bool((q[rows.of(0)] == 77).all())


# --------------------------------------------------------------------------- mass
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("page,lens,new,last", [
    (16, [0, 1, 40, 333], [1, 1, 1, 1], 1),
    (48, [5, 0, 127, 300, 64], [3, 17, 1, 0, 33], 5),
    (64, [0, 129, 0, 700], [65, 128, 129, 1], 1000),
    (16, [31, 2], [300, 257], 32),
])
def test_mass(dtype, shape, page, lens, new, last):
    import torch
    hq, hkv, d = SHAPES[shape]
    rng = np.random.default_rng(shape)
    c, rows, q = build(rng, lens, new, dtype=dtype, hq=hq, hkv=hkv, d=d, page=page, gap=1)
    scale = d ** -0.5
    lse = torch.full((rows.n, hq), float("nan"), device="cuda")
    want, tol = [], []
    for s, n in enumerate(lens):
        m = rows.new[s]
        if m:
            x, _ = scores(c, s, 1, q[rows.of(s)], n, m, scale)
            lse[rows.of(s)] = torch.logsumexp(x, -1).permute(2, 0, 1).reshape(m, hq).float()
            w, e = ref_mass(c, s, 1, q[rows.of(s)], lse[rows.of(s)], n, m, scale, last)
        else:
            w, e = None, 0
        want.append(w)
        tol.append(e)
    ld = max(n + m for n, m in zip(lens, new)) + 3
    before = torch.rand((len(lens), hkv, ld), device="cuda")
    for s, n in enumerate(lens):
        before[s, :, n:] = float("nan")                                # (a new position's weight starts from nothing)
    out, err = mass(c, 1, q, lse, rows, lens, scale, last, before)
    assert err == 0
    for s, n in enumerate(lens):
        m = rows.new[s]
        if m == 0:
            assert bool((out[s] == 77).all())
            continue
        w = want[s].clone()
        w[:, :n] += before[s, :, :n].double()
        # (the addition to what was there rounds once more)
        assert bool(((out[s, :, :n + m].double() - w).abs() <= want[s] * tol[s] + w * 2.0 ** -24 + 1e-37).all()), s
        assert bool((out[s, :, n + m:] == 77).all())
    none, _ = mass(c, 1, q, lse, rows, lens, scale, last)              # no array before, and the same bits
    twice, _ = mass(c, 1, q, lse, rows, lens, scale, last)
    assert torch.equal(none, twice)
    for s, n in enumerate(lens):
        if rows.new[s]:
            assert bool(((none[s, :, :n + rows.new[s]].double() - want[s]).abs() <= want[s] * tol[s] + 1e-37).all())
    same = before.clone()                                              # in place
    mass(c, 1, q, lse, rows, lens, scale, last, same, same)
    for s, n in enumerate(lens):
        if rows.new[s]:
            assert torch.equal(same[s, :, :n + rows.new[s]], out[s, :, :n + rows.new[s]])


def test_mass_of_all_rows_sums_to_their_number():
    """Each counted row's weights sum to 1: 900 tokens x 4 heads on one kv head."""
    import torch
    rng = np.random.default_rng(2)
    c, rows, q = build(rng, [300], [900], dtype=BF16, hq=4, hkv=1, d=128, page=16, layers=1)
    out, lse, _ = attention(c, 0, q, rows, [300], 0.09)
    got, err = mass(c, 0, q, lse, rows, [300], 0.09, 900)
    assert err == 0
    # both sides' scores come from the same products; lse is off by a few 2^-24 of its size and of the sum's terms
    assert abs(float(got[0, 0, :1200].double().sum()) - 3600) <= 3600 * (1200 * 2.0 ** -24 + 64 * 2.0 ** -24 * 20)


def test_mass_bad_lengths_and_pages():
    import torch
    rng = np.random.default_rng(4)
    lens, new = [50, 33, 64], [6, 3, 1]
    c, rows, q = build(rng, lens, new, dtype=BF16, hq=4, hkv=2, d=64, page=16, layers=1)
    lse = torch.zeros((rows.n, 4), device="cuda")
    want, _ = mass(c, 0, q, lse, rows, lens, 0.1, 9)
    got, err = mass(c, 0, q, lse, rows, lens, 0.1, 9, ld=60)           # the third is longer than its mass
    assert err == 4 and bool((got[2] == 77).all())
    assert torch.equal(got[:2, :, :56], want[:2, :, :56])
    c.bt[1, 0] = -7
    got, err = mass(c, 0, q, lse, rows, lens, 0.1, 9)
    assert err == 1 and torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    assert torch.equal(got[1, :, 16:36], want[1, :, 16:36])


# --------------------------------------------------------------------------- eviction
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layers,hkv,d,page", [(2, 3, 128, 16), (1, 1, 64, 48), (3, 2, 64, 64)])
@pytest.mark.parametrize("lens,budget,recent", [
    ([300, 17, 0, 64, 65], 64, 16), ([5, 1, 2], 1, 0), ([5, 3], 1, 1), ([700, 699, 701], 700, 0), ([1500, 40], 1030, 1030),
    ([2100, 4099], 513, 7)])
@pytest.mark.parametrize("kind", ["plain", "ties", "odd"])
def test_evict(dtype, layers, hkv, d, page, lens, budget, recent, kind):
    import torch
    rng = np.random.default_rng(len(lens) + budget)
    c = Cache(rng, lens, [0] * len(lens), dtype=dtype, layers=layers, hkv=hkv, d=d, page=page)
    ld = max(lens) + 2
    x = np.exp(3 * rng.standard_normal((layers, len(lens), hkv, ld))).astype(np.float32)
    if kind == "ties":
        x = np.floor(x).clip(0, 5).astype(np.float32)
    elif kind == "odd":
        with np.errstate(all="ignore"):
            x *= rng.choice([-1, 1, 0, -0.0, np.nan, np.inf, -np.inf, 1e-42, 3e38], x.shape).astype(np.float32)
    old = [slots(c, s, n) for s, n in enumerate(lens)]
    rest = c.kv.clone()
    out, kept, ln, err = evict(c, lens, torch.from_numpy(x).cuda(), budget, recent)
    assert err == 0
    for s, n in enumerate(lens):
        assert ln[s] == min(n, budget)
        now = slots(c, s, n)
        for layer in range(layers):
            for h in range(hkv):
                keep = ref_keep(x[layer, s, h], n, budget, recent) if n > budget else np.arange(n)
                k = len(keep)
                assert np.array_equal(kept[layer, s, h, :k], keep) and (kept[layer, s, h, k:] == -1).all()
                assert np.array_equal(out[layer, s, h, :k], x[layer, s, h, keep], equal_nan=True)
                assert (out[layer, s, h, k:] == 77).all()
                assert torch.equal(now[:k, layer, h], old[s][torch.from_numpy(keep).cuda(), layer, h])
    used = np.unique(np.concatenate([c.table[s, :-(-min(n, budget) // page)] for s, n in enumerate(lens)] + [np.zeros(0, np.int32)]))
    other = np.setdiff1d(np.arange(c.n_pages), used)                   # pages behind the kept slots are as they were
    assert torch.equal(c.kv[other].nan_to_num(5.0), rest[other].nan_to_num(5.0))


def test_evict_bad_lengths_and_pages():
    import torch
    lens = [100, 90, 80]
    for what, bits in (("page", 1), ("neg", 4), ("long", 4), ("ld", 4)):
        c = Cache(np.random.default_rng(1), lens, [0] * 3, dtype=BF16, layers=2, hkv=2, d=64, page=16)
        x = torch.rand((2, 3, 2, 100 if what != "ld" else 95), device="cuda")
        ll = list(lens)
        if what == "page":
            c.bt[0, 6] = c.n_pages                                     # the last page's rows may be kept
        elif what == "neg":
            ll[0] = -5
        elif what == "long":
            ll[0] = c.max_pages * 16 + 1
        before = c.kv.clone()
        out, kept, ln, err = evict(c, ll, x, 50, 10)
        assert err == bits, what
        assert ln.tolist() == [ll[0], 50, 50] and (kept[:, 0] == -1).all() and (out[:, 0] == 77).all()
        mine = c.table[0, :7].astype(np.int64)
        assert torch.equal(c.kv[mine].nan_to_num(5.0), before[mine].nan_to_num(5.0))
        for s in (1, 2):
            for layer in range(2):
                for h in range(2):
                    assert np.array_equal(kept[layer, s, h], ref_keep(x[layer, s, h].cpu().numpy(), lens[s], 50, 10))


# --------------------------------------------------------------------------- together
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_bounded_cache_over_many_steps(dtype):
    """A prompt in chunks, then single tokens, two layers, with eviction to a budget after each step: append, attend,
    count and evict as a decoder calls them, against a plain cache kept in 64 bits beside it."""
    import torch
    from lossless_speculative_decoding_gb300 import binding as B
    td = torch.float32 if dtype == F32 else torch.bfloat16
    L, hq, hkv, d, page, S, budget, recent = 2, 4, 2, 64, 16, 3, 96, 8
    gen = torch.Generator(device="cuda").manual_seed(11)
    c = Cache(np.random.default_rng(1), [0] * S, [304] * S, dtype=dtype, layers=L, hkv=hkv, d=d, page=page)
    ld = 304
    m0, m1 = torch.zeros((L, S, hkv, ld), device="cuda"), torch.zeros((L, S, hkv, ld), device="cuda")
    kept = torch.zeros((L, S, hkv, budget), dtype=torch.int32, device="cuda")
    n0, n1 = dev([0] * S), dev([0] * S)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    freq = 1e4 ** (-np.arange(32) / 32)
    rope, gam = B.make_rope(freq), [torch.rand(d, generator=gen, device="cuda") + 0.5 for _ in "qk"]
    host_n, at_pos = np.zeros(S, int), np.zeros(S, int)
    plain = [[[np.zeros((0, 2, d)) for _ in range(hkv)] for _ in range(S)] for _ in range(L)]
    pmass = [[[np.zeros(0) for _ in range(hkv)] for _ in range(S)] for _ in range(L)]
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    for step, new in enumerate([[150, 20, 1], [1, 1, 1], [4, 0, 150], [1, 1, 1], [1, 60, 1], [1, 1, 1]]):
        rows = Rows(new)
        nb = B.spec_chunk_attention_ws_bytes(c.view, S, rows.most, hq)
        ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
        pos = np.zeros((1, rows.n), np.int32)
        for s in range(S):
            pos[0, rows.of(s)] = at_pos[s] + np.arange(new[s])
        start, mm, pp = dev(rows.start), dev(new), dev(pos)
        for layer in range(L):
            x = torch.randn((rows.n, hq + 2 * hkv, d), generator=gen, device="cuda").to(td)
            q, out = torch.zeros((rows.n, hq, d), device="cuda", dtype=td), torch.zeros((rows.n, hq, d), device="cuda", dtype=td)
            z = torch.zeros((rows.n, hq), device="cuda")
            torch.cuda.synchronize()
            B.spec_qk_norm_rope(c.view, layer, x, x.stride(0), rows.n, S, hq, start, mm, n0, rope, pp, gam[0], gam[1], 1e-6, q,
                                err, st.cuda_stream)
            B.spec_chunk_attention(c.view, layer, q, rows.n, S, rows.most, hq, start, mm, n0, 0.125, out, z, ws, nb, err,
                                   st.cuda_stream)
            B.spec_attention_mass(c.view, layer, q, z, rows.n, S, rows.most, 16, hq, start, mm, n0, 0.125, m0[layer], m0[layer],
                                  ld, err, st.cuda_stream)
            st.synchronize()
            angle = torch.from_numpy(pos[0][:, None] * freq).cuda()
            y = ref_rope(x, hq, hkv, gam, 1e-6, angle)
            for s in range(S):
                if new[s] == 0:
                    continue
                live = slots(c, s, host_n[s] + new[s])[host_n[s]:, layer].cpu().numpy()
                for h in range(hkv):
                    # the new rows as the cache holds them (rounded once from the formulas)
                    e = 2.0 ** -8 if dtype == BF16 else 2.0 ** -18
                    yk = y[rows.of(s), hq + h].cpu().numpy()
                    assert np.abs(live[:, h, 0] - yk).max() <= e * max(1, np.abs(yk).max())
                    plain[layer][s][h] = np.concatenate([plain[layer][s][h], live[:, h]])
                    K, V = (torch.from_numpy(plain[layer][s][h][:, i]).cuda() for i in (0, 1))
                    qd = q[rows.of(s), h * 2:h * 2 + 2].double()
                    t = torch.einsum("igd,jd->gij", qd, K) * 0.125
                    hide = torch.arange(len(K), device="cuda")[None] > host_n[s] + torch.arange(new[s], device="cuda")[:, None]
                    t = t.masked_fill(hide, float("-inf"))
                    w = torch.softmax(t, -1)
                    o = torch.einsum("gij,jd->igd", w, V)
                    got = out[rows.of(s), h * 2:h * 2 + 2].double()
                    vmax = float(V.abs().max())
                    assert float((got - o).abs().max()) <= vmax * ((2 * 2.0 ** -8 if dtype == BF16 else 0) + 2.0 ** -13)
                    pm = np.concatenate([pmass[layer][s][h], np.zeros(new[s])])
                    pmass[layer][s][h] = pm + w[:, -min(16, new[s]):].sum((0, 1)).cpu().numpy()
                    dev_m = m0[layer, s, h, :len(pm)].double().cpu().numpy()
                    assert np.abs(dev_m - pmass[layer][s][h]).max() <= 1e-4
                    pmass[layer][s][h] = dev_m                          # (so that near ties fall the same way)
        # as a program does: the new tokens are held now
        torch.cuda.synchronize()
        n0 += mm
        torch.cuda.synchronize()
        host_n += new
        at_pos += new
        B.spec_kv_evict(c.view, S, n0, m0, ld, budget, recent, m1, kept, n1, err, st.cuda_stream)
        st.synchronize()
        for s in range(S):
            n = host_n[s]
            if n > budget:
                for layer in range(L):
                    for h in range(hkv):
                        keep = ref_keep(pmass[layer][s][h].astype(np.float32), n, budget, recent)
                        assert np.array_equal(kept[layer, s, h].cpu().numpy(), keep)
                        plain[layer][s][h], pmass[layer][s][h] = plain[layer][s][h][keep], pmass[layer][s][h][keep]
                host_n[s] = budget
            now = slots(c, s, host_n[s]).cpu().numpy()
            for layer in range(L):
                for h in range(hkv):
                    assert np.array_equal(now[:, layer, h], plain[layer][s][h])
        m0, m1, n0, n1 = m1, m0, n1, n0
        assert n0.cpu().tolist() == host_n.tolist()
    assert int(err.item()) == 0
