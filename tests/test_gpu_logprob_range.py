"""Token log probabilities where logits / temperature is large: rows masked
throughout by one finite value, logits at the types' ends, gaps of one step of
the type at large magnitudes, and temperatures from 1e-30 to 1e38."""
import math

import numpy as np
import pytest

import _tree as T
from test_gpu_logprobs import _run

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24                                               # half a step of fp32


def _ref(raw, tokens, temperature, top_n):
    """(logp of the tokens, entropy, rank, ids, logps of the ids, rise) in float64: differences first, so that
    nothing is lost at large magnitudes; raw [R, V] float64 without NaN, +inf or rows of nothing."""
    t = float(np.float32(temperature))
    y = (raw - raw.max(1, keepdims=True)) / t
    e = np.exp(y)
    z = e.sum(1, keepdims=True)
    lp = y - np.log(z)
    ent = np.log(z[:, 0]) - np.where(e > 0, e * np.where(e > 0, y, 0.0), 0.0).sum(1) / z[:, 0]
    order = np.argsort(-raw, axis=1, kind="stable")
    place = np.empty_like(order)
    np.put_along_axis(place, order, np.arange(raw.shape[1])[None], 1)
    R = np.arange(len(raw))
    fin = np.where(np.isfinite(y), -y, 0.0).max()
    return lp[R, tokens], ent, place[R, tokens] + 1, order[:, :top_n], np.take_along_axis(lp, order[:, :top_n], 1), fin


def limits(V, dtype, rise):
    """(log probability, entropy) errors of the kernel's fp32 evaluation, beside a relative 8 EPS of a result.

    A thread adds its values of a step in two chains, then steps, then the lanes of a warp, the warps of a block and the
    blocks of a row as trees of up to five levels: `depth` roundings of a sum of one sign, each EPS. Powers: one for a
    value, one for each step (a new maximum), three for each level of a merge, 2^-22 each. A power's argument y is right
    within 4 EPS |y| (difference, log2 e, 1 / T, product), which enters the sums weighted by the probabilities: sum of
    p |y| <= log2 V; where a maximum rises by r within a step, its values were taken against the one before: EPS r more,
    r < 128. log2 z is within one step of a value of at most log2 V. The entropy's second sum has the same errors,
    times |y|, and each rise r adds EPS r."""
    per = 4 if dtype == T.F32 else 8
    tiles = -(-V // (2048 * per)) + 1
    lg = max(1.0, math.log2(V))
    depth = 4 * per + 2 + 3 * tiles + 3 * 20
    r = min(rise * 1.45, 128.0)
    e = depth * EPS + (1 + tiles + 20) * 2.0 ** -22 + (4 * lg + r) * EPS + lg * 2.0 ** -22
    return e, e * (2 + 2 * lg) + 4 * r * EPS


def _check(x, tokens, temperature, top):
    V = x.shape[1]
    got = _run(x, tokens, temperature, top)
    dtype = T.F32 if str(x.dtype) == "torch.float32" else T.BF16
    lp, ent, rank, ids, tops, rise = _ref(x.double().cpu().numpy(), tokens, temperature, top)
    assert np.array_equal(got[2], rank) and np.array_equal(got[3], ids)
    el, ee = limits(V, dtype, rise)
    for name, a, b, lim in (("logprob", got[0], lp, el), ("top", got[4], tops, el), ("entropy", got[1], ent, ee)):
        with np.errstate(over="ignore"):
            far = b.astype(np.float32) == -np.inf              # past fp32's range
        assert (a[far] == -np.inf).all(), name
        err = np.abs(a[~far].astype(np.float64) - b[~far])
        assert (err <= lim + np.abs(b[~far]) * 8 * EPS).all(), (name, temperature, float(np.nanmax(err)), a[~far][:4], b[~far][:4])


def _rows(rows, dtype):
    import torch
    x = torch.from_numpy(np.stack(rows).astype(np.float32)).cuda()
    return x if dtype == T.F32 else x.bfloat16()


def _ends(dtype):
    import torch
    f = torch.finfo(torch.float32 if dtype == T.F32 else torch.bfloat16)
    return float(f.min), float(f.max)


@pytest.mark.parametrize("dtype", [T.F32, T.BF16])
@pytest.mark.parametrize("V", [7, 1000, 40003, 129280])
def test_logprobs_of_rows_of_one_large_value(dtype, V):
    """Every token masked by the same finite value: equal probabilities, -log V."""
    values = [1e7, -1e7, 1e9, -1e9, 1e10, -1e10, -3e10, 1e30, -1e30, 1e31, -1e31, *_ends(dtype)]
    x = _rows([np.full(V, v) for v in values], dtype)
    tokens = np.arange(len(values), dtype=np.int32) % V
    _check(x, tokens, 1.0, 3)
    _check(x, tokens, 100.0, 3)


@pytest.mark.parametrize("dtype", [T.F32, T.BF16])
@pytest.mark.parametrize("V", [50, 5000, 70001])
def test_logprobs_of_peaks_at_large_magnitudes(dtype, V):
    """One larger token, or one smaller, among equal ones; -inf beside them; two levels; rising rows."""
    rows, low, high = [], *_ends(dtype)
    for v in (1e9, -1e9, 1e10, -1e10, 1e30, -1e30, high / 4, low / 2):
        r = np.full(V, v)
        r[V // 3] = v + abs(v) / 4
        rows.append(r)
        r = np.full(V, v)
        r[V // 2] = v - abs(v) / 4
        rows.append(r)
        r = np.full(V, v)
        r[::3] = -np.inf
        rows.append(r)
        rows.append(v + np.abs(v) / 4 * np.floor(np.arange(V) * 7 / V))        # steps up along the row
    rows.append(np.where(np.arange(V) == V - 1, high, low))
    r = np.full(V, low)
    r[3:9] = 0.25
    rows.append(r)
    x = _rows(rows, dtype)
    rng = np.random.default_rng(V)
    for t in (1.0, 0.01, 300.0):
        tokens = rng.integers(0, V, len(rows)).astype(np.int32)
        tokens[::2] = V // 3
        _check(x, tokens, t, 20)


@pytest.mark.parametrize("dtype", [T.F32, T.BF16])
@pytest.mark.parametrize("masked", [False, True])
def test_logprobs_of_close_values_at_large_magnitudes(dtype, masked):
    """Gaps of a few steps of the type, of the temperature's size: logits / T from 2^5 to 2^24, either side of where
    products and differences part. Masked tokens in some steps and not in others."""
    import torch
    V = 50021
    rng = np.random.default_rng(3)
    td = torch.float32 if dtype == T.F32 else torch.bfloat16
    for v in (1.0, 1.25, 1.9, -1.0, -1.25, -1.9):
        base = torch.full((6, V), v * 2.0 ** 33, dtype=torch.float64).to(td).double()
        gap = torch.finfo(td).eps * 2.0 ** 33                  # one step of the type
        base += torch.from_numpy(rng.integers(-6, 1, (6, V)).astype(np.float64)) * gap * 2
        if masked:
            base[:, V // 2:V // 2 + 9000] = -float("inf")
            base[3, ::17] = -float("inf")
        x = base.to(td).cuda()
        tokens = rng.integers(0, V // 2, 6).astype(np.int32)
        for t in (gap / 2, gap, gap * 3.1, gap * 64):
            _check(x, tokens, t, 4)


@pytest.mark.parametrize("dtype", [T.F32, T.BF16])
@pytest.mark.parametrize("temperature", [1e-38, 1e-30, 1e-9, 1e-6, 1e-3, 1e3, 1e9, 1e30])
def test_logprobs_at_extreme_temperatures(dtype, temperature):
    """Ordinary logits: next to nothing but the largest at one end, equal probabilities at the other."""
    import torch
    V = 30011
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn((5, V), generator=g, device="cuda") * 4
    x[1] = 20.0
    x[2] = -20.0
    x[3, ::2] = -float("inf")
    x = x if dtype == T.F32 else x.bfloat16()
    tokens = np.array([5, 6, 7, 9, int(x[4].float().argmax())], np.int32)
    _check(x, tokens, temperature, 20)


@pytest.mark.parametrize("dtype", [T.F32, T.BF16])
def test_logprobs_of_the_types_ends_at_high_temperature(dtype):
    """Logits of both signs at the type's ends, a temperature that brings them near one."""
    low, high = _ends(dtype)
    rng = np.random.default_rng(11)
    V = 20001
    r = rng.uniform(-1, 1, V) * high
    r[5], r[6] = low, high
    x = _rows([r, np.where(np.arange(V) % 2 == 0, low, high)], dtype)
    for t in (1e38, 2e37, 1e36):
        _check(x, np.array([5, 6], np.int32), t, 5)
