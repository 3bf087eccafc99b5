"""Entry points for chunks of new tokens at the ends of their ranges: large factors of a score, many rows, many
sequences, far positions, long caches, many planes."""
import numpy as np
import pytest

from _chunk import BF16, F32, Cache, Rows, attention, check_attention, dev, mass, ref_mass

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
