"""Entry points for chunks of new tokens at the ends of their ranges: large factors of a score, many rows, many
sequences, far positions, long caches, many planes."""
import numpy as np
import pytest

from _chunk import (BF16, F32, Cache, Rows, attention, check_attention, dev, evict, mass, queries, ref_keep, ref_mass, slots)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("most", [3, 150])
def test_queries_whose_scaled_values_overflow(dtype, most):
    """scale * q passes the largest float, scale * q.K (up to 8 for each position) does not."""
    import torch
    n, d, scale = 70, 64, 2.0 ** 10
    T = n + most
    c = Cache(np.random.default_rng(1), [n], [most], dtype=dtype, layers=1, hkv=1, d=d, page=16)
    key = torch.zeros((T, d), device="cuda")
    key[:, 0] = 2.0 ** -125 * (1 + torch.arange(T, device="cuda") % 37)      # (whole numbers of 8 bits)
    pos = torch.arange(T, device="cuda")
    c.kv[torch.from_numpy(c.table[0].astype(np.int64)).cuda()[pos // 16], 0, 0, 0, pos % 16] = key.to(c.kv.dtype)
    c.rows[0][:, 0, 0, 0] = key.double()
    rows = Rows([most])
    q = torch.zeros((rows.n, 2, d), device="cuda", dtype=c.kv.dtype)
    q[:, 0, 0], q[:, 1, 0] = 2.0 ** 118, 1.5 * 2.0 ** 117
    out, lse, err = attention(c, 0, q, rows, [n], scale)
    assert err == 0
    check_attention(c, 0, q, rows, [n], scale, out, lse, one_part=dtype == BF16 and most > 64)
    got, err = mass(c, 0, q, lse, rows, [n], scale, most)
    w, e = ref_mass(c, 0, 0, q[:most], lse[:most], n, most, scale, most)
    assert err == 0 and bool(((got[0, :, :T].double() - w).abs() <= w * e + 1e-30).all())


def test_mass_of_65536_rows_in_fp32():
    """Equal weights of many rows: the sum's error does not grow with their number."""
    import torch
    m, G = 4096, 16
    c = Cache(np.random.default_rng(1), [0], [m], dtype=F32, layers=1, hkv=1, d=64, page=64)
    rows = Rows([m])
    q = torch.zeros((rows.n, G, 64), device="cuda")
    lse = torch.full((rows.n, G), 3.0, device="cuda")
    got, err = mass(c, 0, q, lse, rows, [0], 0.125, m)
    assert err == 0
    want = G * torch.arange(m, 0, -1, device="cuda").double() * np.exp(-3.0)
    # 3 log2 e: a rounded constant and a rounded product, 1.5 x 2^-24 of 3 in the exponent; exp2 2 ulp (4 x 2^-24); four
    # weights added at a time and eight threads' sums, 3 + 7 roundings; a compensated sum between, 2; the result, 1
    assert float(((got[0, 0, :m].double() - want).abs() / want).max()) <= (4.5 + 4 + 10 + 2 + 1) * 2.0 ** -24


PI = "3.14159265358979323846264338327950288419716939937510582097494459230781640628620899"


@pytest.mark.parametrize("d", [64, 128])
def test_rotation_angles_at_far_positions(d):
    """Frequencies of either sign, above and far below a turn, at positions up to 2^31: (1, 0) turns to (cos, sin)."""
    import torch
    from decimal import Decimal, localcontext
    from lossless_speculative_decoding_gb300 import binding as B
    rng = np.random.default_rng(d)
    half, m = d // 2, 24
    freq = np.exp(rng.uniform(np.log(1e-9), np.log(50.0), half)) * rng.choice([-1.0, 1.0], half)
    freq[:6] = 1.0, -1.0, -1e-6, 2 * np.pi, -3e-20, 1e6
    pos = rng.integers(-2 ** 31, 2 ** 31, m)
    pos[:4] = 2 ** 31 - 1, -2 ** 31, 0, 1
    c = Cache(rng, [0], [m], dtype=F32, layers=1, hkv=1, d=d, page=16)
    rows = Rows([m])
    x = torch.zeros((rows.n, 3, d), device="cuda")
    x[:, :, :half] = 1.0
    q = torch.zeros((rows.n, 1, d), device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    p = np.zeros((1, rows.n), np.int32)
    p[0, rows.of(0)] = pos
    B.spec_qk_norm_rope(c.view, 0, x, 3 * d, rows.n, 1, 1, dev(rows.start), dev(rows.new), dev([0]), B.make_rope(freq), dev(p), None,
                        None, 0.0, q, err, 0)
    torch.cuda.synchronize()
    with localcontext() as ctx:
        ctx.prec = 70
        angle = np.array([[float(Decimal(int(a)) * Decimal(float(f)) % (2 * Decimal(PI))) for f in freq] for a in pos])
    # the angle is off by 2^-32 of a turn and, an eighth of a turn at most, by its rounding to fp32 (2^-28); sine and cosine
    # by 2 ulp below 1
    e = 2 * np.pi * (2.0 ** -32 + 2.0 ** -28) + 2.0 ** -23
    got = q[rows.of(0), 0].double().cpu().numpy()
    assert int(err.item()) == 0
    assert np.abs(got[:, :half] - np.cos(angle)).max() <= e
    assert np.abs(got[:, half:] - np.sin(angle)).max() <= e


@pytest.mark.parametrize("most,G,n,spread", [(608, 128, 2 ** 25, 1), (3, 64, 2 ** 25, 304), (1, 1, 2 ** 26, 304)])
def test_attention_over_tens_of_millions_of_positions(most, G, n, spread):
    """Segments of 2^18 and 2^19 tiles, each of some 0.3 s, on every block: whole row tiles, row tiles with one group of
    tokens, single tokens; `spread` sequences share the pages of their first n positions. Keys of zeros but for one, values
    of ones but for its: even heads weigh all alike, odd ones take that one."""
    import torch
    from lossless_speculative_decoding_gb300 import binding as B
    P, d, at = 2 ** 14, 64, n - 1000
    m = most if spread == 1 else max(1, most - 1)
    kv = torch.zeros((n // P + spread, 1, 1, 2, P, d), dtype=torch.bfloat16, device="cuda")
    kv[:, :, :, 1] = 1.0
    kv[at // P, 0, 0, 0, at % P, 0], kv[at // P, 0, 0, 1, at % P] = 1.0, 3.0
    bt = torch.empty((spread, n // P + 1), dtype=torch.int32, device="cuda")
    bt[:, :-1] = torch.arange(n // P, device="cuda")
    bt[:, -1] = n // P + torch.arange(spread, device="cuda")
    view = B.make_kv_view(kv, bt, dtype=BF16, n_pages=n // P + spread, n_layers=1, n_kv_heads=1, page_size=P, head_dim=d,
                          max_pages=n // P + 1)
    rows = Rows([m] * spread)
    q = torch.zeros((rows.n, G, d), dtype=torch.bfloat16, device="cuda")
    odd = torch.arange(rows.n * G, device="cuda").view(rows.n, G) % 2 == 1       # (a single head: odd rows)
    q[..., 0] = torch.where(odd, 320.0, 0.0).bfloat16()
    out, lse = torch.full_like(q, 77.0), torch.full((rows.n, G), 77.0, device="cuda")
    nb = B.spec_chunk_attention_ws_bytes(view, spread, most, G)
    ws, err = torch.empty(nb, dtype=torch.uint8, device="cuda"), dev([0])
    B.spec_chunk_attention(view, 0, q, rows.n, spread, most, G, dev(rows.start), dev(rows.new), dev([n] * spread), 0.125, out, lse, ws,
                           nb, err, 0)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    live, odd = spread * m, odd[:spread * m]
    # the others' share of an odd head is 2^26 e^-40 at most, of an even head's value the one's 2 / n; a weight of one bf16
    # part is off by 2^-8, and so is the result's rounding
    want = torch.where(odd, 3.0, 1.0)[..., None]
    assert bool(((out[:live].float() - want).abs() <= want * (2 * 2.0 ** -8 + 2.0 ** -16)).all()) and bool((out[live:] == 77).all())
    seen = n + 1 + torch.arange(live, device="cuda") % m
    z = torch.where(odd, 40.0 + 0 * seen[:, None], torch.log(seen.double())[:, None])
    # sums of equal weights are whole multiples of one; the last of a tile, and each part's, may be rounded: 2^-24 for the
    # segment and 160 parts; the logarithm's own size 40 in fp32 (6 roundings)
    assert float((lse[:live].double() - z).abs().max()) <= 162 * 2.0 ** -24 + 6 * 40 * 2.0 ** -24


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("most", [1, 40])
def test_mass_of_many_sequences(dtype, most):
    """700 sequences, most of them padded, the first live one behind the first 32."""
    import torch
    rng = np.random.default_rng(4)
    lens = rng.integers(0, 600, 700)
    new = np.where(rng.random(700) < 0.7, 0, rng.integers(1, most + 1, 700))
    new[:70] = 0
    c = Cache(rng, lens, new, dtype=dtype, layers=1, hkv=2, d=64, page=16)
    rows = Rows(new)
    q = queries(rows, 4, 64, dtype, 3)
    out, lse, err = attention(c, 0, q, rows, lens, 0.125)
    assert err == 0
    got, err = mass(c, 0, q, lse, rows, lens, 0.125, most)
    assert err == 0
    for s, n in enumerate(lens):
        n, m = int(n), rows.new[s]
        if m:
            w, e = ref_mass(c, s, 0, q[rows.of(s)], lse[rows.of(s)], n, m, 0.125, most)
            assert bool(((got[s, :, :n + m].double() - w).abs() <= w * e + 1e-37).all()), s
        assert bool((got[s, :, n + m if m else 0:] == 77).all()), s


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("most", [1, 40])
def test_rotation_of_many_sequences(dtype, most):
    """700 sequences, most of them padded: rows find their slots (heads copied, none turned)."""
    import torch
    from lossless_speculative_decoding_gb300 import binding as B
    rng = np.random.default_rng(6)
    lens = rng.integers(0, 50, 700)
    new = np.where(rng.random(700) < 0.7, 0, rng.integers(1, most + 1, 700))
    c = Cache(rng, lens, new, dtype=dtype, layers=1, hkv=2, d=64, page=16)
    rows = Rows(new, 1)
    x = torch.randn((rows.n, 6, 64), device="cuda").to(c.kv.dtype)
    q = torch.full((rows.n, 2, 64), 77.0, device="cuda", dtype=c.kv.dtype)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.spec_qk_norm_rope(c.view, 0, x, 384, rows.n, 700, 2, dev(rows.start), dev(rows.new), dev(lens), B.make_rope([]), None, None, None,
                        0.0, q, err, 0)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    live = torch.zeros(rows.n, dtype=torch.bool, device="cuda")
    for s, n in enumerate(lens):
        m = rows.new[s]
        if m:
            at, n = rows.of(s), int(n)
            live[at] = True
            got = slots(c, s, n + m)
            assert torch.equal(got[:n], c.rows[s][:n]), s
            assert torch.equal(got[n:, 0].transpose(1, 2).reshape(m, 4, 64), x[at, 2:].double()), s
    assert torch.equal(q[live], x[live, :2]) and bool((q[~live] == 77).all())


def test_mass_rows_past_2_to_31_values():
    """The last rows of a mass array start past 2^31 values; what was there is read from there."""
    import torch
    lens, new, ld = [50, 7], [4, 70], 2 ** 29
    for dtype in (BF16, F32):
        c = Cache(np.random.default_rng(3), lens, new, dtype=dtype, layers=1, hkv=4, d=128, page=16)
        rows = Rows(new)
        q = queries(rows, 8, 128, dtype, 5)
        out, lse, err = attention(c, 0, q, rows, lens, 0.09)
        assert err == 0
        before, got = torch.empty((2, 4, ld), device="cuda"), torch.empty((2, 4, ld), device="cuda")
        before[..., :200] = torch.rand((2, 4, 200), device="cuda") + 1
        got, err = mass(c, 0, q, lse, rows, lens, 0.09, 70, before, out=got, ld=ld)
        assert err == 0
        for s, n in enumerate(lens):
            w, e = ref_mass(c, s, 0, q[rows.of(s)], lse[rows.of(s)], n, new[s], 0.09, 70)
            y = w.clone()
            y[:, :n] += before[s, :, :n].double()
            assert bool(((got[s, :, :n + new[s]].double() - y).abs() <= w * e + y * 2.0 ** -24 + 1e-37).all()), (dtype, s)
        del before, got


# --------------------------------------------------------------------------- eviction
def check_evict(c, lens, x, budget, recent):
    """Kept positions, their masses and their rows of every plane."""
    import torch
    old = [slots(c, s, n) for s, n in enumerate(lens)]
    out, kept, ln, err = evict(c, lens, torch.from_numpy(x).cuda(), budget, recent)
    assert err == 0 and ln.tolist() == [min(n, budget) for n in lens]
    for s, n in enumerate(lens):
        k = min(n, budget)
        want = np.empty((c.layers, c.hkv, k), np.int64)
        for layer in range(c.layers):
            for h in range(c.hkv):
                want[layer, h] = ref_keep(x[layer, s, h], n, budget, recent) if n > budget else np.arange(n)
        assert np.array_equal(kept[:, s, :, :k], want) and (kept[:, s, :, k:] == -1).all()
        assert np.array_equal(out[:, s, :, :k], np.take_along_axis(x[:, s], want, 2), equal_nan=True)
        assert (out[:, s, :, k:] == 77).all()
        at = torch.from_numpy(want).cuda().permute(2, 0, 1)[..., None, None].expand(-1, -1, -1, 2, c.d)
        assert torch.equal(slots(c, s, k), torch.gather(old[s], 0, at)), s


def masses(rng, shape, kind):
    x = np.exp(3 * rng.standard_normal(shape)).astype(np.float32)
    if kind == "ties":
        x = np.floor(x).clip(0, 5).astype(np.float32)
    elif kind == "nan":
        x[rng.random(shape) < 0.3] = np.nan
    return x


@pytest.mark.parametrize("dtype,d", [(BF16, 64), (BF16, 128), (F32, 64), (F32, 128)])
@pytest.mark.parametrize("kind", ["plain", "ties"])
@pytest.mark.parametrize("lens,budget", [([1500, 701, 40], 700), ([900, 1, 641], 640), ([500, 400, 30], 31)])
def test_evict_many_planes(dtype, d, kind, lens, budget):
    """480 planes: the form for many blocks, in batches of rows that end whole and within one."""
    rng = np.random.default_rng(budget + d)
    c = Cache(rng, lens, [0, 0, 0], dtype=dtype, layers=40, hkv=4, d=d, page=48)
    check_evict(c, lens, masses(rng, (40, 3, 4, max(lens) + 1), kind), budget, 13)


@pytest.mark.parametrize("kind", ["plain", "ties", "nan"])
@pytest.mark.parametrize("budget,recent", [(4001, 100), (8192, 0), (1, 0), (8100, 8100)])
def test_evict_long_sequences(kind, budget, recent):
    """More positions than the selection holds, as many, and fewer."""
    lens = [12011, 8193, 8192, 8191]
    rng = np.random.default_rng(budget)
    c = Cache(rng, lens, [0] * 4, dtype=BF16, layers=1, hkv=2, d=64, page=64)
    check_evict(c, lens, masses(rng, (1, 4, 2, max(lens) + 3), kind), budget, recent)
