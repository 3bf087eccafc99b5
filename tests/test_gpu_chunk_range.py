"""Entry points for chunks of new tokens at the ends of their ranges: large factors of a score, many rows, many
sequences, far positions, long caches, many planes."""
import numpy as np
import pytest

from _chunk import BF16, F32, Cache, Rows, attention, check_attention, mass, ref_mass

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
