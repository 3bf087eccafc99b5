"""Inputs and 64-bit restatements of the entry points for chunks of new tokens."""
import numpy as np

from _tree import BF16, F32, Cache, dev, tol  # noqa: F401  (shared with the tree tests)


class Rows:
    """Rows of the sequences' tokens in a packed array, a few rows of none between and behind them."""

    def __init__(self, new, gap=0, spare=2):
        self.new = [int(m) for m in new]
        self.start, at = [], gap
        for m in self.new:
            self.start.append(at)
            at += max(m, 0) + gap
        self.n = at + spare
        self.most = max(1, max(self.new))

    def of(self, s):
        return slice(self.start[s], self.start[s] + self.new[s])


def queries(rows, hq, d, dtype, seed, sharp=2.0):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randn((rows.n, hq, d), generator=gen, device="cuda")
    return (q * torch.linspace(0.3, sharp, hq, device="cuda")[:, None]).to(torch.float32 if dtype == F32 else torch.bfloat16)


def attention(c, layer, q, rows, lens, scale, *, out=None, lse=True, stream=0, max_new=None, ws=None):
    """One call on the whole batch; returns (out, lse, error bits)."""
    import torch
    from lossless_speculative_decoding_gb300 import binding as B
    S, hq = len(lens), q.shape[1]
    most = rows.most if max_new is None else max_new
    out = torch.full_like(q, 77.0) if out is None else out
    z = torch.full((q.shape[0], hq), 77.0, device="cuda") if lse else None
    nb = B.spec_chunk_attention_ws_bytes(c.view, S, most, hq)
    ws = torch.full((nb,), 0xA5, dtype=torch.uint8, device="cuda") if ws is None else ws
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.spec_chunk_attention(c.view, layer, q, q.shape[0], S, most, hq, dev(rows.start), dev(rows.new), dev(lens), scale, out, z,
                           ws, nb, err, stream)
    torch.cuda.synchronize()
    return out, z, int(err.item())


def scores(c, s, layer, q, n, m, scale):
    """float64 [hkv, G, m, n + m] with -inf where a token does not look, and the largest sum of a score's magnitudes."""
    import torch
    hkv, d = c.hkv, c.d
    K = c.rows[s][:, layer, :, 0]
    qd = q.double().view(m, hkv, -1, d)
    x = torch.einsum("ihgd,jhd->hgij", qd, K) * scale
    mag = float((torch.einsum("ihgd,jhd->hgij", qd.abs(), K.abs()) * scale).max())
    hide = torch.arange(n + m, device="cuda")[None] > n + torch.arange(m, device="cuda")[:, None]
    return x.masked_fill(hide, float("-inf")), mag


def ref_attention(c, s, layer, q, n, m, scale, one_part=False):
    """float64 output [m, hq, d] and lse [m, hq] of sequence s, and bounds of their errors in an fp32 evaluation.
    one_part: weights enter the sum of values rounded to bf16, 2^-8 each, and their sum does not."""
    import torch
    x, mag = scores(c, s, layer, q, n, m, scale)
    V = c.rows[s][:, layer, :, 1]
    lse = torch.logsumexp(x, -1)
    o = torch.einsum("hgij,jhd->ihgd", torch.exp(x - lse[..., None]), V).reshape(m, -1, c.d)
    e = tol(c.d, n + m, mag, float(V.abs().max()))
    if one_part:
        e += 2.0 ** -8 * float(V.abs().max())
    # the log of a sum with relative error r is off by r; adding the maximum and changing the base round it
    r = (c.d + 4) * 2.0 ** -24 * mag + 2.0 ** -22 + (n + m) * 2.0 ** -24
    return o, lse.permute(2, 0, 1).reshape(m, -1), e, r + 4 * 2.0 ** -24 * float(lse.abs().max() + 1)


def check_attention(c, layer, q, rows, lens, scale, out, lse, one_part):
    """Every row of every sequence against the formulas, the other rows as they were (77)."""
    import torch
    touched = torch.zeros(q.shape[0], dtype=torch.bool, device="cuda")
    for s, n in enumerate(lens):
        m = rows.new[s]
        if m == 0:
            continue
        at = rows.of(s)
        touched[at] = True
        o, z, e, ez = ref_attention(c, s, layer, q[at], int(n), m, scale, one_part)
        bound = e + (o.abs() * 2.0 ** -8 if q.dtype == torch.bfloat16 else 0)     # one rounding of the output
        bad = (out[at].double() - o).abs() - bound
        assert not torch.isnan(out[at]).any() and float(bad.max()) <= 0, (s, n, m, float(bad.max()))
        if lse is not None:
            assert float((lse[at].double() - z).abs().max()) <= ez, (s, n, m)
    assert bool((out[~touched] == 77).all())
    if lse is not None:
        assert bool((lse[~touched] == 77).all())


def ref_mass(c, s, layer, q, lse, n, m, scale, last):
    """float64 sums [hkv, n + m] over the counted tokens, and the relative error bound of an fp32 evaluation."""
    import torch
    x, mag = scores(c, s, layer, q, n, m, scale)
    z = lse.double().view(m, c.hkv, -1).permute(1, 2, 0)
    p = torch.exp(x - z[..., None])
    k = min(m, last)
    G = x.shape[1]
    top = float(z.abs().max())
    # exponents of a size of mag + |lse| in fp32 (score, scale, lse in units of log 2, their difference), the
    # exponential, and a sum of k G terms of one sign
    e = (c.d + 8) * 2.0 ** -24 * mag + 6 * 2.0 ** -24 * (mag + top) + 2.0 ** -22 + k * G * 2.0 ** -24
    return p[:, :, m - k:].sum((1, 2)), e


def mass(c, layer, q, lse, rows, lens, scale, last, before=None, out=None, ld=None, stream=0, max_new=None):
    import torch
    from lossless_speculative_decoding_gb300 import binding as B
    S, hq = len(lens), q.shape[1]
    ld = max(int(n) + m for n, m in zip(lens, rows.new)) + 3 if ld is None else ld
    out = torch.full((S, c.hkv, ld), 77.0, device="cuda") if out is None else out
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.spec_attention_mass(c.view, layer, q, lse, q.shape[0], S, rows.most if max_new is None else max_new, last, hq,
                          dev(rows.start), dev(rows.new), dev(lens), scale, before, out, ld, err, stream)
    torch.cuda.synchronize()
    return out, int(err.item())


def ref_keep(row, n, budget, recent):
    """Positions that a plane keeps: NaN after every number, equal masses by position."""
    x = np.where(np.isnan(row[:n - recent]), -np.inf, row[:n - recent].astype(np.float64))
    nan = np.isnan(row[:n - recent])
    order = np.lexsort((np.arange(n - recent), nan, -x))
    return np.sort(np.concatenate([order[:budget - recent], np.arange(n - recent, n)])).astype(np.int64)


def evict(c, lens, mass_in, budget, recent, stream=0):
    """One call; returns (out_mass, kept, len, error bits) as numpy arrays."""
    import torch
    from lossless_speculative_decoding_gb300 import binding as B
    S, ld = len(lens), mass_in.shape[-1]
    out = torch.full_like(mass_in, 77.0)
    kept = torch.full((c.layers, S, c.hkv, budget), 77, dtype=torch.int32, device="cuda")
    ln = torch.full((S,), 77, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.spec_kv_evict(c.view, S, dev(lens), mass_in, ld, budget, recent, out, kept, ln, err, stream)
    torch.cuda.synchronize()
    return out.cpu().numpy(), kept.cpu().numpy(), ln.cpu().numpy(), int(err.item())


def slots(c, s, n):
    """The cache's content of sequence s's first n slots, float64 [n, layers, hkv, 2, d]."""
    import torch
    pos = torch.arange(n, device="cuda")
    pg = torch.from_numpy(c.table[s].astype(np.int64)).cuda()[pos // c.P]
    return c.kv[pg, :, :, :, pos % c.P].double()
