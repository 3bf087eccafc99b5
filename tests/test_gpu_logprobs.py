"""Token log probabilities on the GPU against a 64-bit restatement: odd
vocabularies and row strides, both logit types, ties, masked tokens, rows of
nothing but -inf, NaN and +inf, and rows without a token."""
import numpy as np
import pytest

import _tree as T

pytestmark = pytest.mark.gpu


def _run(x, tokens, temperature, top_n, ld=None, ws=None, stream=0):
    """x: [R, V] tensor (possibly a strided view of rows)."""
    import torch
    from lossless_speculative_decoding_gb300 import binding as B
    R, V = x.shape
    dt = T.F32 if x.dtype == torch.float32 else T.BF16
    f = lambda *s: torch.full(s, 55.0, device="cuda")                   # noqa: E731
    w = lambda *s: torch.full(s, -55, dtype=torch.int32, device="cuda")  # noqa: E731
    lp, ent, rank, ids, top = f(R), f(R), w(R), w(R, top_n), f(R, top_n)
    nb = B.spec_token_logprobs_ws_bytes(R, V, top_n)
    ws = torch.zeros(nb, dtype=torch.uint8, device="cuda") if ws is None else ws
    B.spec_token_logprobs(x, dt, x.stride(0) if R > 1 else V, R, V, T.dev(tokens), temperature, top_n, lp, ent, rank, ids, top,
                          ws, nb, stream)
    torch.cuda.synchronize()
    return [t.cpu().numpy() for t in (lp, ent, rank, ids, top)]


def _ref(x, tokens, temperature, top_n):
    """(logp of all [R, V], entropy, rank, ids, top logps) in float64 numpy."""
    raw = x.double().cpu().numpy()
    it = np.float64(np.float32(1.0) / np.float32(temperature))
    y = raw * it
    key = np.where(np.isnan(raw), -np.inf, raw)
    order = np.argsort(-key, axis=1, kind="stable")
    with np.errstate(invalid="ignore", divide="ignore"):
        m = y.max(1, keepdims=True)
        e = np.exp(y - m)
        z = e.sum(1, keepdims=True)
        lp = y - m - np.log(z)
        ent = np.log(z[:, 0]) - np.where(e > 0, e * (y - m), 0.0).sum(1) / z[:, 0]
    bad = np.isnan(raw).any(1) | (raw == np.inf).any(1) | (key == -np.inf).all(1)
    lp[bad], ent[bad] = np.nan, np.nan
    place = np.empty_like(order)
    np.put_along_axis(place, order, np.arange(raw.shape[1])[None], 1)
    R, t = np.arange(len(raw)), np.asarray(tokens)
    ok = (t >= 0) & (t < raw.shape[1])
    tc = np.where(ok, t, 0)
    return (np.where(ok, lp[R, tc], np.nan), ent, np.where(ok, place[R, tc] + 1, 0), order[:, :top_n],
            np.take_along_axis(lp, order[:, :top_n], 1), float(np.nanmax(np.where(np.isfinite(y), np.abs(y), 0))))


def _compare(got, ref, V):
    lp, ent, rank, ids, top = got
    rlp, rent, rrank, rids, rtop, mag = ref
    assert np.array_equal(rank, rrank) and np.array_equal(ids, rids)
    # fp32: x = logit / T and x - m round at magnitudes up to 2 mag, an exponent's argument is scaled by log2 e once
    # more, the exponential is within 2^-21, and a sum of V terms of one sign within V 2^-24 of itself; log z passes a
    # relative error on as an absolute one, the entropy's second sum multiplies it by at most 2 mag
    e = 8 * mag * 2.0 ** -24 + 2.0 ** -21 + V * 2.0 ** -24
    for a, b, lim in ((lp, rlp, e), (top, rtop, e), (ent, rent, e * (2 + 2 * mag))):
        assert np.array_equal(np.isnan(a), np.isnan(b)) and np.array_equal(np.isinf(a), np.isinf(b))
        ok = np.isfinite(b)
        assert (np.abs(a[ok] - b[ok]) <= lim + np.abs(b[ok]) * 2.0 ** -23).all()


@pytest.mark.parametrize("dtype", [T.F32, T.BF16])
@pytest.mark.parametrize("R,V,top,temp", [(1, 1, 1, 1.0), (3, 2, 2, 0.5), (5, 31, 20, 1.0), (2, 33, 32, 1.3),
                                          (4, 129280, 5, 1.0), (7, 1001, 0, 0.7), (300, 4099, 20, 1.0), (2, 262144, 32, 2.0),
                                          (1, 151936, 1, 1.0), (700, 64, 3, 1.0), (1, 1048576, 7, 1.0), (40, 8193, 32, 0.25)])
def test_logprobs_match_64_bits(dtype, R, V, top, temp):
    import torch
    rng = np.random.default_rng(R * 1000 + V)
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.randn((R, V), generator=g, device="cuda") * torch.linspace(0.1, 6.0, R, device="cuda")[:, None]
    x = x if dtype == T.F32 else x.bfloat16()
    tokens = rng.integers(0, V, R).astype(np.int32)
    tokens[::2] = x.float().argmax(-1).cpu().numpy()[::2]
    if R > 3:
        tokens[1], tokens[3] = -1, V
    _compare(_run(x, tokens, temp, top), _ref(x, tokens, temp, top), V)


@pytest.mark.parametrize("dtype", [T.F32, T.BF16])
@pytest.mark.parametrize("V,ld,off", [(1000, 1007, 1), (4097, 4100, 3), (130, 131, 2), (9001, 9001, 7)])
def test_logprobs_strided_and_unaligned_rows(dtype, V, ld, off):
    """Rows ld apart, from an address with no more than an element's alignment."""
    import torch
    R = 6
    g = torch.Generator(device="cuda").manual_seed(V)
    flat = torch.full((off + R * ld + 9,), float("nan"), device="cuda")
    flat = flat if dtype == T.F32 else flat.bfloat16()
    x = torch.as_strided(flat, (R, V), (ld, 1), off)
    x.copy_(torch.randn((R, V), generator=g, device="cuda"))
    tokens = np.array([0, V - 1, 5, 6, 7, V // 2], np.int32)
    _compare(_run(x, tokens, 1.0, 8), _ref(x, tokens, 1.0, 8), V)


@pytest.mark.parametrize("dtype", [T.F32, T.BF16])
@pytest.mark.parametrize("V", [50, 5000, 40000])
def test_logprobs_ties_masks_and_bad_rows(dtype, V):
    import torch
    rng = np.random.default_rng(V)
    rows = []
    rows.append(np.zeros(V))                                            # all equal: lowest indices, entropy log V
    rows.append(rng.integers(-2, 3, V).astype(float))                   # five values only
    r = rng.standard_normal(V)
    r[rng.random(V) < 0.9] = -np.inf                                    # masked tokens
    r[3] = 1.0
    rows.append(r)
    r = np.full(V, -np.inf)
    r[V - 2] = -7.0                                                     # one token left
    rows.append(r)
    rows.append(np.full(V, -np.inf))                                    # nothing left
    r = rng.standard_normal(V)
    r[[2, V - 1]] = np.nan
    rows.append(r)
    r = rng.standard_normal(V)
    r[V // 2] = np.inf
    rows.append(r)
    r = np.full(V, np.finfo(np.float32).min)                            # masked by the type's lowest value
    r[7] = 0.5
    rows.append(r)
    rows.append(np.arange(V) / 64.0)                                    # rising and falling: every element enters the list
    rows.append(-np.arange(V) / 64.0)
    r = np.zeros(V)
    r[::2] = -0.0                                                       # two zeros, one value
    rows.append(r)
    x = torch.from_numpy(np.stack(rows).astype(np.float32)).cuda()
    x = x if dtype == T.F32 else x.bfloat16()
    for tokens in (np.full(len(rows), 3, np.int32), np.full(len(rows), V - 2, np.int32)):
        got, ref = _run(x, tokens, 1.0, 20), list(_ref(x, tokens, 1.0, 20))
        fin = torch.where(torch.isfinite(x) & (x.abs() < 1e30), x.double().abs(), 0.0)
        ref[5] = float(fin.max())
        low = 7                                                         # its x - m is the lowest value itself: compared apart
        keep = [i for i in range(len(rows)) if i != low]
        _compare([a[keep] for a in got], [a[keep] for a in ref[:5]] + [ref[5]], V)
        assert np.array_equal(got[2], ref[2]) and np.array_equal(got[3], ref[3])
        assert got[4][low, 0] == 0.0 and got[1][low] == 0.0
        assert np.allclose(got[4][low, 1:], ref[4][low, 1:], rtol=2.0 ** -22)


def test_logprobs_outputs_left_out_and_workspace_reused():
    import torch
    from lossless_speculative_decoding_gb300 import binding as B
    R, V = 9, 30011
    g = torch.Generator(device="cuda").manual_seed(0)
    nb = max(B.spec_token_logprobs_ws_bytes(R, V, 4), B.spec_token_logprobs_ws_bytes(2, 129280, 30))
    ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    for seed in range(3):                                               # other shapes in turn on one workspace
        x = torch.randn((R, V), generator=g, device="cuda")
        tokens = np.arange(R, dtype=np.int32) * 100
        _compare(_run(x, tokens, 1.0, 4, ws=ws), _ref(x, tokens, 1.0, 4), V)
        y = torch.randn((2, 129280), generator=g, device="cuda")
        _compare(_run(y, np.array([5, 6], np.int32), 0.8, 30, ws=ws), _ref(y, [5, 6], 0.8, 30), 129280)
    ent = torch.zeros(R, device="cuda")
    B.spec_token_logprobs(x, T.F32, V, R, V, None, 1.0, 0, None, ent, None, None, None, ws, nb, 0)
    torch.cuda.synchronize()
    assert np.allclose(ent.cpu().numpy(), _ref(x, [0] * R, 1.0, 0)[1], rtol=1e-5)
    ids, top = torch.zeros((R, 2), dtype=torch.int32, device="cuda"), torch.zeros((R, 2), device="cuda")
    B.spec_token_logprobs(x, T.F32, V, R, V, None, 1.0, 2, None, None, None, ids, top, ws, nb, 0)
    torch.cuda.synchronize()
    assert np.array_equal(ids.cpu().numpy(), _ref(x, [0] * R, 1.0, 2)[3])


def test_logprobs_captured_and_replayed():
    import torch
    from lossless_speculative_decoding_gb300 import binding as B
    R, V, top = 4, 129280, 5
    x = torch.zeros((R, V), device="cuda")
    tok = torch.zeros(R, dtype=torch.int32, device="cuda")
    lp, ent, tl = torch.zeros(R, device="cuda"), torch.zeros(R, device="cuda"), torch.zeros((R, top), device="cuda")
    rank, ids = torch.zeros(R, dtype=torch.int32, device="cuda"), torch.zeros((R, top), dtype=torch.int32, device="cuda")
    nb = B.spec_token_logprobs_ws_bytes(R, V, top)
    ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    st = torch.cuda.Stream()
    call = lambda: B.spec_token_logprobs(x, T.F32, V, R, V, tok, 1.0, top, lp, ent, rank, ids, tl, ws, nb, st.cuda_stream)  # noqa: E731
    torch.cuda.synchronize()
    call()
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        call()
    for seed in range(2):
        x.copy_(torch.randn((R, V), device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)))
        tok.copy_(x.argmin(-1))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        _compare([t.cpu().numpy() for t in (lp, ent, rank, ids, tl)], _ref(x, tok.cpu().numpy(), 1.0, top), V)
        assert bool((rank == V).all())


@pytest.mark.parametrize("dtype", [T.F32, T.BF16])
@pytest.mark.parametrize("R,V,top", [(65535, 1, 1), (65535, 5, 0), (20000, 9, 4), (305, 16385, 20), (609, 8192, 6)])
def test_logprobs_of_many_short_rows(dtype, R, V, top):
    """More rows than blocks: rows that start and end inside a block's run, with few tokens."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(R)
    x = torch.randn((R, V), generator=g, device="cuda")
    x = x if dtype == T.F32 else x.bfloat16()
    tokens = np.random.default_rng(V).integers(0, V, R).astype(np.int32)
    _compare(_run(x, tokens, 1.0, top), _ref(x, tokens, 1.0, top), V)
