"""Inputs and a 64-bit restatement of the tree entry points, for their tests."""
import numpy as np

F32, BF16 = 0, 1
N = 64                                                         # SPEC_TREE_MAX_NODES


def rand_parents(rng, k, forest=False):
    p = np.full(N, -1, np.int32)
    for i in range(1, k):
        p[i] = -1 if forest and rng.random() < 0.2 else rng.integers(max(0, i - 6), i)
    return p


def chain_of(parents, i):
    out = [i]
    while 0 <= parents[i] < i:
        i = int(parents[i])
        out.append(i)
    return out


class Cache:
    """A paged cache on the GPU whose unused slots hold `junk`; rows[s] is its
    float64 content [position, layer, kv head, K | V, dim]."""

    def __init__(self, rng, lens, nodes, *, dtype, layers, hkv, d, page, junk=float("nan"), spare=2, seed=0):
        import torch
        from lossless_speculative_decoding_gb300 import binding as B
        self.P, self.dtype, self.d, self.hkv, self.layers = page, dtype, d, hkv, layers
        tot = [n + k for n, k in zip(lens, nodes)]
        need = [-(-t // page) for t in tot]
        self.max_pages = max(need) + 1
        self.n_pages = sum(need) + spare
        ids, at = rng.permutation(self.n_pages), 0
        self.table = np.full((len(lens), self.max_pages), -1, np.int32)
        td = torch.float32 if dtype == F32 else torch.bfloat16
        self.kv = torch.full((self.n_pages, layers, hkv, 2, page, d), junk, dtype=td, device="cuda")
        self.rows = []
        gen = torch.Generator(device="cuda").manual_seed(seed)
        for s, t in enumerate(tot):
            self.table[s, :need[s]] = ids[at:at + need[s]]
            at += need[s]
            r = torch.randn((t, layers, hkv, 2, d), generator=gen, device="cuda").to(td)
            pos = torch.arange(t, device="cuda")
            pg = torch.from_numpy(self.table[s].astype(np.int64)).cuda()[pos // page]
            self.kv[pg, :, :, :, pos % page] = r
            self.rows.append(r.double())
        self.bt = torch.from_numpy(self.table).cuda()
        self.view = B.make_kv_view(self.kv, self.bt, dtype=dtype, n_pages=self.n_pages, n_layers=layers, n_kv_heads=hkv,
                                   page_size=page, head_dim=d, max_pages=self.max_pages)


def ref_attention(rows, layer, q, n, k, parents, scale):
    """float64 [k, hq, d] of one sequence, and the absolute error bound of an
    fp32 evaluation (see tol)."""
    import torch
    hkv, d = rows.shape[2], rows.shape[4]
    G = q.shape[1] // hkv
    hide = torch.ones((k, n + k), dtype=torch.bool)
    hide[:, :n] = False
    for i in range(k):
        for j in chain_of(parents, i):
            hide[i, n + j] = False
    hide = hide.cuda()
    K, V = rows[:, layer, :, 0], rows[:, layer, :, 1]
    qd = q[:k].double().view(k, hkv, G, d)
    x = torch.einsum("ihgd,jhd->hgij", qd, K) * scale
    w = torch.softmax(x.masked_fill(hide, float("-inf")), -1)
    o = torch.einsum("hgij,jhd->ihgd", w, V).reshape(k, hkv * G, d)
    mag = float((torch.einsum("ihgd,jhd->hgij", qd.abs(), K.abs()) * scale).max()) if n + k else 0.0
    return o, tol(d, n + k, mag, float(V.abs().max()))


def tol(d, keys, mag, vmax):
    """Error of an fp32 evaluation, as arithmetic gives it. A score is a sum of
    d products whose magnitudes sum to at most mag: (d + 4) 2^-24 mag with the
    scale's roundings. It enters a weight as a relative error, and so do the
    exponential (2^-22), the weight's own two-part bf16 form where that is
    used (2^-16), and a sum over `keys` terms of one sign (keys 2^-24). The
    output sums weights of total 1 times values below vmax, numerator and
    denominator each with that error, and its own sum adds keys 2^-24."""
    e = (d + 4) * 2.0 ** -24 * mag + 2.0 ** -22 + 2.0 ** -16 + keys * 2.0 ** -24
    return vmax * (2 * e + keys * 2.0 ** -24)


def ref_walk(parents, tokens, target, k):
    path = [0]
    while True:
        below = [c for c in range(path[-1] + 1, k) if parents[c] == path[-1] and tokens[c] == target[path[-1]]]
        if not below:
            return path
        path.append(below[0])


def dev(a, dtype=np.int32):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).cuda()


def attention(c, layer, q, lens, nodes, parents, scale, out=None, stream=0, ws=None, err=None):
    """One call on the whole batch; returns (out, error bits)."""
    import torch
    from lossless_speculative_decoding_gb300 import binding as B
    S, hq = len(lens), q.shape[2]
    out = torch.full_like(q, 77.0) if out is None else out
    nb = B.spec_tree_attention_ws_bytes(c.view, S, q.shape[1], hq)
    ws = torch.full((nb,), 0xA5, dtype=torch.uint8, device="cuda") if ws is None else ws
    err = torch.zeros(1, dtype=torch.int32, device="cuda") if err is None else err
    B.spec_tree_attention(c.view, layer, q, S, q.shape[1], hq, dev(lens), dev(nodes), dev(parents), scale, out, ws, nb, err,
                          stream)
    torch.cuda.synchronize()
    return out, int(err.item())
