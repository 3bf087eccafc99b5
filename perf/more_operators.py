"""Cases of the operators for chunks of new tokens over a paged cache: norms of
queries and keys with the rotation of positions (the new keys and values go
into the cache), attention of the chunk, the attention weight that each cached
position has drawn, and eviction by that weight.

Shapes come from the synthetic model configurations: the 3B-MoE decoder (10
heads of 128, 12 layers), the dense 4B decoder (32 query and 8 key/value heads
of 128, 36 layers) and the tiny fp32 decoder (4 heads of 64). A cache is
[page][layer][kv head][K, V][position in page][dim]; sequence s holds n
positions, and its m new tokens have the slots right after them. The tokens of
all sequences are packed, sequence behind sequence; a few rows behind the last
one belong to none.
"""
import math

import numpy as np
import torch

own = False

F32, BF16 = 0, 1
SPARE_ROWS = 3                             # rows behind the last sequence
MAX_SCORES = 32 * 1021 * 66542             # of the largest attention case, padded to the longest sequence
MAX_MASS_SCORES = 32 * 5288 * 5288         # of the largest count of weights
MAX_CACHE_BYTES = 0.6e9                    # keys and values of one layer
MAX_EVICT_BYTES = 0.6e9                    # the cache of a drawn eviction (the listed ones keep a smaller part of theirs)
MAX_ROW_VALUES = 4623 * 48 * 128           # values of the largest rotation case


# --------------------------------------------------------------------------- cases
def listed():
    rot = dict(op="qk_norm_rope", norm=True, rot=128, theta=1e4, layers=2)
    att = dict(op="chunk_attention", dtype="bf16")
    mas = dict(op="attention_mass", dtype="bf16")
    evi = dict(op="kv_evict", dtype="bf16")
    moe, dense = dict(hq=10, hkv=10, d=128), dict(hq=32, hkv=8, d=128)
    return [
        # the rows of one verify step (the last token and three drafts) enter the cache: a single request, where latency counts
        dict(rot, **moe, name="rope_moe_b1", dtype="bf16", batch=1, page=16, ctx_lo=1357, ctx_hi=1357, new_lo=4, new_hi=4, axes=1),
        # four documents' pages: visual rows with time, height and width, behind short prompts
        dict(rot, **dense, name="rope_dense_pages", dtype="bf16", batch=4, page=16, ctx_lo=0, ctx_hi=301, new_lo=1057,
             new_hi=1257, axes=3, theta=1e6),
        # plain decoding of the 64-sequence workload: one token each, short and long documents side by side
        dict(att, **moe, name="att_moe_b64", batch=64, page=16, ctx_lo=336, ctx_hi=5236, new_lo=1, new_hi=1),
        # chunks of eight prompts beside cached parts of them: ragged, up to 701 tokens
        dict(att, **dense, name="att_dense_chunks", batch=8, page=64, ctx_lo=1288, ctx_hi=5288, new_lo=17, new_hi=701),
        # a whole prompt from an empty cache
        dict(att, **dense, name="att_dense_prompt", batch=1, page=16, ctx_lo=0, ctx_hi=0, new_lo=5288, new_hi=5288),
        # one more chunk of a long document
        dict(att, **dense, name="att_dense_long", batch=1, page=16, ctx_lo=65521, ctx_hi=65521, new_lo=1021, new_hi=1021),
        # the fp32 decoder
        dict(att, name="att_tiny_f32", dtype="f32", hq=4, hkv=4, d=64, batch=4, page=16, ctx_lo=0, ctx_hi=200, new_lo=5,
             new_hi=72),
        # each decoding step adds its weights
        dict(mas, **moe, name="mass_moe_b64", batch=64, page=16, ctx_lo=336, ctx_hi=5236, new_lo=1, new_hi=1, last=1),
        # the last 32 tokens of eight prompts vote
        dict(mas, **dense, name="mass_dense_last", batch=8, page=64, ctx_lo=0, ctx_hi=288, new_lo=1288, new_hi=5288, last=32),
        # every token of a prompt
        dict(mas, **dense, name="mass_dense_prompt", batch=1, page=16, ctx_lo=0, ctx_hi=0, new_lo=5288, new_hi=5288, last=5288),
        # one document, cut to 1,024 positions in 12 layers
        dict(evi, **moe, name="evict_moe_b1", layers=12, batch=1, page=16, ctx_lo=1357, ctx_hi=1357, budget=1024, recent=64),
        # two in 36 layers
        dict(evi, **dense, name="evict_dense_b2", layers=36, batch=2, page=16, ctx_lo=3288, ctx_hi=5288, budget=2048, recent=256),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["qk_norm_rope", "chunk_attention", "chunk_attention", "attention_mass", "kv_evict"])
    hq, hkv, d = rng.choice([(10, 10, 128), (32, 8, 128), (4, 4, 64), (16, 2, 64), (12, 1, 128)])
    page = rng.choice([16, 16, 32, 48, 64, 128])
    dtype = "bf16" if rng.random() < 0.8 else "f32"
    esz = 2 if dtype == "bf16" else 4
    c = dict(op=op, dtype=dtype, hq=hq, hkv=hkv, d=d, page=page)
    pos = hkv * 2 * d * esz                     # bytes of a position in one layer
    if op == "qk_norm_rope":
        total = _log_int(rng, 1, max(1, int(MAX_ROW_VALUES * 2 / esz) // ((hq + 2 * hkv) * d)))
        batch = _log_int(rng, 1, min(64, total))
        hi = total // batch
        lo, top = rng.randint(1, hi), _log_int(rng, 1, 5000)
        while batch * (top + hi) * pos * 2 > MAX_CACHE_BYTES:
            top //= 2
        return dict(c, layers=2, batch=batch, ctx_lo=rng.randint(0, top), ctx_hi=top, new_lo=lo, new_hi=hi,
                    axes=rng.choice([1, 3]), norm=rng.random() < 0.7, rot=rng.choice([d, d, d // 2]), theta=rng.choice([1e4, 1e6]))
    if op == "kv_evict":
        layers, batch = rng.choice([2, 12, 36]), _log_int(rng, 1, 16)
        top = _log_int(rng, 64, 16384)
        while batch > 1 and batch * (top + page) * pos * layers > MAX_EVICT_BYTES:
            batch //= 2
        while (top + page) * pos * layers > MAX_EVICT_BYTES:
            top = top * 3 // 4
        budget = rng.randint(1, top)
        return dict(c, layers=layers, batch=batch, ctx_lo=rng.randint(budget // 2, top), ctx_hi=top, budget=budget,
                    recent=rng.randint(0, min(budget, 512)))
    if dtype == "f32":                          # the fp32 decoder serves short prompts
        batch, hi, top = _log_int(rng, 1, 8), _log_int(rng, 1, 256), _log_int(rng, 1, 1000)
    else:
        batch, hi, top = _log_int(rng, 1, 64), rng.choice([1, _log_int(rng, 1, 4096)]), _log_int(rng, 1, 65536)
    last = rng.choice([32, 1 << 30]) if op == "attention_mass" else 1 << 30
    scores = MAX_MASS_SCORES if op == "attention_mass" else MAX_SCORES
    while batch * (top + hi) * pos > MAX_CACHE_BYTES or batch * hq * min(hi, last) * (top + hi) > scores:
        batch, top, hi = max(1, batch // 2), max(1, top - top // 4), max(1, hi - hi // 8)
    lo = rng.randint(1, hi)
    c.update(batch=batch, ctx_lo=rng.randint(0, top), ctx_hi=top, new_lo=lo, new_hi=hi)
    return dict(c, last=min(hi, last)) if op == "attention_mass" else c


# --------------------------------------------------------------------------- sizes of a case
def _spread(lo, hi, n, step):
    """n whole numbers spread over [lo, hi], both ends among them when n > 1; the case alone decides them."""
    v = lo + np.floor((np.arange(n) * step % 1.0) * (hi - lo + 1)).astype(np.int64)
    v[0] = hi
    if n > 1:
        v[-1] = lo
    return v


def _lengths(case):
    return _spread(case["ctx_lo"], case["ctx_hi"], case["batch"], 0.6180339887498949)


def _new(case):
    if "new_hi" not in case:
        return np.zeros(case["batch"], np.int64)
    return _spread(case["new_lo"], case["new_hi"], case["batch"], 0.4142135623730951)


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _esz(case):
    return 2 if case["dtype"] == "bf16" else 4


def work(case):
    n, m, e = _lengths(case).astype(float), _new(case).astype(float), _esz(case)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "qk_norm_rope":
        rows = float(m.sum())
        return {"bytes": rows * (2.0 * (hq + 2 * hkv) * d * e + 4 * case["axes"]), "flops": 10.0 * rows * (hq + hkv) * d}
    if case["op"] == "chunk_attention":
        return {"bytes": float(((n + m) * hkv * 2 * d * e + m * hq * (2 * d * e + 4)).sum()),
                "flops": 4.0 * d * hq * float((m * n + m * (m + 1) / 2).sum())}
    if case["op"] == "attention_mass":
        c = np.minimum(m, case["last"])         # counted tokens: the last c see n + m - c + 1 .. n + m positions
        return {"bytes": float(((n + m) * hkv * (d * e + 8) + c * hq * (d * e + 4)).sum()),
                "flops": 2.0 * d * hq * float((c * (n + m) - c * (c - 1) / 2).sum())}
    cut = n > case["budget"]
    planes = case["layers"] * hkv
    return {"bytes": float((planes * (4 * n + cut * case["budget"] * (4.0 * d * e) + 8 * np.minimum(n, case["budget"]))).sum()),
            "flops": float((planes * n).sum())}


# --------------------------------------------------------------------------- inputs
def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _cache(case, gen, r, layers):
    """A cache with the sequences' pages in random order, their block table, lengths and rows."""
    n, m, P = _lengths(case), _new(case), case["page"]
    order = r.permutation(len(n))
    n, m = n[order], m[order]
    need = -(-(n + m) // P)
    max_pages = int(need.max()) + 1
    n_pages = int(need.sum()) + 3
    table = np.full((len(n), max_pages), -1, np.int32)
    ids, at = r.permutation(n_pages).astype(np.int32), 0
    for s in range(len(n)):
        table[s, :need[s]] = ids[at:at + need[s]]
        at += need[s]
    kv = torch.empty((n_pages, layers, case["hkv"], 2, P, case["d"]), dtype=_dtype(case), device="cuda")
    kv.normal_(generator=gen)
    start = np.concatenate([[0], np.cumsum(m)])
    return dict(kv=kv, table=_dev(table), cache_len=_dev(n), n_new=_dev(m), row_start=_dev(start[:-1]), n_host=n, m_host=m,
                start_host=start, rows=int(start[-1]) + SPARE_ROWS, err=torch.zeros(1, dtype=torch.int32, device="cuda"))


def _queries(case, s, gen):
    """Queries whose heads differ in how sharply they look."""
    q = torch.empty((s["rows"], case["hq"], case["d"]), dtype=torch.float32, device="cuda")
    q.normal_(generator=gen).mul_(torch.linspace(0.5, 3.0, case["hq"], device="cuda")[:, None])
    s["q"] = q.to(_dtype(case))
    s["scale"] = 1.0 / math.sqrt(case["d"])


def _sections(case):
    """Axis of each rotated pair: time takes the first quarter, height and width what is left."""
    half = case["rot"] // 2
    if case["axes"] == 1:
        return np.zeros(half, np.int64)
    t = half // 4
    return np.concatenate([np.zeros(t, np.int64), np.ones((half - t) // 2, np.int64), np.full(half - t - (half - t) // 2, 2)])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    r = np.random.default_rng(int(seed))
    s = dict(case=case)
    s.update(_cache(case, gen, r, case.get("layers", 1)))
    if case["op"] == "qk_norm_rope":
        heads = case["hq"] + 2 * case["hkv"]
        x = torch.empty((s["rows"], heads, case["d"]), dtype=torch.float32, device="cuda").normal_(generator=gen)
        x.mul_(torch.linspace(0.2, 5.0, heads, device="cuda")[:, None])
        s["qkv"] = x.to(_dtype(case))
        pos = np.zeros((case["axes"], s["rows"]), np.int64)
        for b in range(case["batch"]):
            i = np.arange(s["m_host"][b])
            at = slice(s["start_host"][b], s["start_host"][b + 1])
            if case["axes"] == 1:
                pos[0, at] = s["n_host"][b] + i
            else:                               # a picture 34 patches wide behind the text
                pos[:, at] = s["n_host"][b] + np.stack([0 * i, i // 34, i % 34])
        s["positions"] = _dev(pos)
        half = case["rot"] // 2
        s["freq"] = np.float64(case["theta"]) ** (-np.arange(half) / half)
        s["axis"] = _sections(case)
        s["gamma"] = [None, None]
        if case["norm"]:
            s["gamma"] = [torch.empty(case["d"], dtype=torch.float32, device="cuda").normal_(1.0, 0.2, generator=gen) for _ in "qk"]
        s["eps"] = 1e-6
        s["q"] = torch.zeros((s["rows"], case["hq"], case["d"]), dtype=_dtype(case), device="cuda")
    elif case["op"] == "chunk_attention":
        _queries(case, s, gen)
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros((s["rows"], case["hq"]), dtype=torch.float32, device="cuda")
    elif case["op"] == "attention_mass":
        _queries(case, s, gen)
        s["lse"] = _counted_lse(case, s)
        shape = (case["batch"], case["hkv"], int((s["n_host"] + s["m_host"]).max()) + 5)
        s["mass"] = torch.empty(shape, dtype=torch.float32, device="cuda").exponential_(1.0, generator=gen)
        s["out"] = torch.zeros_like(s["mass"])
    else:
        shape = (case["layers"], case["batch"], case["hkv"], int(s["n_host"].max()) + 5)
        # a few positions draw most of the weight, and some none at all
        x = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(generator=gen).mul_(2.0).exp_()
        s["mass"] = torch.where(torch.rand(shape, generator=gen, device="cuda") < 0.1, 0.0, x)
        s["out_mass"] = torch.zeros_like(s["mass"])
        s["kept"] = torch.full((*shape[:3], case["budget"]), -1, dtype=torch.int32, device="cuda")
        s["len"] = torch.full((case["batch"],), -1, dtype=torch.int32, device="cuda")
    return s


def _counted_lse(case, s):
    """log sum exp of the counted tokens' scores, as the attention before leaves them."""
    lse = torch.zeros((s["rows"], case["hq"]), dtype=torch.float32, device="cuda")
    for b in range(case["batch"]):
        x, at = _scores(case, s, b, torch.float32, case["last"])
        lse[at] = torch.logsumexp(x, -1).permute(2, 0, 1).reshape(-1, case["hq"])
    return lse


def _kept_rows(s, b):
    """The cache's rows of sequence b in one layer's order: pages of its positions, slots in the page."""
    P = s["case"]["page"]
    pos = torch.arange(int(s["n_host"][b] + s["m_host"][b]), device="cuda")
    return s["table"][b].long()[torch.div(pos, P, rounding_mode="floor")], pos % P


def _scores(case, s, b, dtype, last):
    """[kv head, group, counted token, position] scores of sequence b's last tokens, -inf where they do not look, and
    the tokens' rows."""
    n, m = int(s["n_host"][b]), int(s["m_host"][b])
    c, hkv = min(m, last), case["hkv"]
    end = int(s["start_host"][b + 1])
    at = slice(end - c, end)
    page, slot = _kept_rows(s, b)
    key = s["kv"][page, 0, :, 0, slot].to(dtype)                                          # [top, hkv, d]
    q = s["q"][at].to(dtype).view(c, hkv, -1, case["d"])
    x = torch.matmul(q.permute(1, 2, 0, 3), key.permute(1, 2, 0)[:, None]) * s["scale"]
    hide = torch.arange(n + m, device="cuda")[None] > n + m - c + torch.arange(c, device="cuda")[:, None]
    return x.masked_fill_(hide, float("-inf")), at


# --------------------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"qk_norm_rope": _own_rope, "chunk_attention": _own_attention, "attention_mass": _own_mass,
                "kv_evict": _own_evict}[op](state)
    return {"qk_norm_rope": _plain_rope, "chunk_attention": _plain_attention, "attention_mass": _plain_mass,
            "kv_evict": _plain_evict}[op](state)


# ---- plain forms
def _token_rows(s):
    """Sequence and number in its chunk of every row that has one (all rows up to the spare ones, in order)."""
    seq = torch.repeat_interleave(torch.arange(len(s["n_host"]), device="cuda"), s["n_new"].long(),
                                  output_size=s["rows"] - SPARE_ROWS)
    return seq, torch.arange(s["rows"] - SPARE_ROWS, device="cuda") - s["row_start"].long()[seq]


def _plain_rope(s):
    case, P = s["case"], s["case"]["page"]
    hq, hkv, half = case["hq"], case["hkv"], case["rot"] // 2
    rows = s["rows"] - SPARE_ROWS
    seq, i = _token_rows(s)
    pos = s["positions"][:, :rows].double()[torch.from_numpy(s["axis"]).cuda()]           # [half, rows]
    angle = (pos * torch.from_numpy(s["freq"]).cuda()[:, None]).T[:, None]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    x = s["qkv"][:rows].float()

    def turned(x, gamma):
        if gamma is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * gamma
        a, b = x[..., :half], x[..., half:2 * half]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., 2 * half:]], -1).to(_dtype(case))

    s["q"][:rows] = turned(x[:, :hq], s["gamma"][0])
    slot = s["cache_len"].long()[seq] + i
    page = s["table"].long()[seq, torch.div(slot, P, rounding_mode="floor")]
    s["kv"][page, 1, :, 0, slot % P] = turned(x[:, hq:hq + hkv], s["gamma"][1])
    s["kv"][page, 1, :, 1, slot % P] = s["qkv"][:rows, hq + hkv:]
    return dict(q=s["q"], kv=s["kv"])


def _padded(s, x, lengths, most, offset):
    """Rows of x, sequence behind sequence, as [sequence, most, ...]: its rows from `offset` on, the last one repeated."""
    i = torch.minimum(torch.arange(most, device="cuda")[None], (lengths - 1).clamp(min=0)[:, None])
    return x[s["row_start"].long()[:, None] + offset[:, None] + i]


def _padded_scores(s, count, most):
    """[sequence, kv head, group, counted token, position] of each sequence's last `count` tokens."""
    case, P = s["case"], s["case"]["page"]
    n, m = s["cache_len"].long(), s["n_new"].long()
    B, hkv = case["batch"], case["hkv"]
    top = case["ctx_hi"] + case["new_hi"]
    pos = torch.arange(top, device="cuda")
    page = s["table"].long()[:, torch.div(pos, P, rounding_mode="floor").clamp(max=s["table"].shape[1] - 1)].clamp(min=0)
    key = s["kv"][page, 0, :, 0, pos % P].float()                                         # [B, top, hkv, d]
    q = _padded(s, s["q"], count, most, m - count).float().view(B, most, hkv, -1, case["d"])
    x = torch.matmul(q.permute(0, 2, 3, 1, 4), key.permute(0, 2, 3, 1)[:, :, None]).mul_(s["scale"])
    seen = pos[None, None] <= (n + m - count)[:, None, None] + torch.arange(most, device="cuda")[None, :, None]
    return x.masked_fill_(~seen[:, None, None], float("-inf")), page, pos % P


def _plain_attention(s):
    case = s["case"]
    n, m = s["cache_len"].long(), s["n_new"].long()
    B, hkv, most = case["batch"], case["hkv"], case["new_hi"]
    x, page, slot = _padded_scores(s, m, most)
    val = s["kv"][page, 0, :, 1, slot].float()                                            # [B, top, hkv, d]
    top = x.amax(-1, keepdim=True)
    p = x.sub_(top).exp_()
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p.div_(z), val.permute(0, 2, 1, 3)[:, :, None])                      # [B, hkv, G, most, d]
    seq, i = _token_rows(s)
    rows = s["rows"] - SPARE_ROWS
    s["out"][:rows] = o[seq, :, :, i].reshape(rows, case["hq"], case["d"]).to(_dtype(case))
    s["lse"][:rows] = (top + torch.log(z))[..., 0][seq, :, :, i].reshape(rows, case["hq"])
    return dict(out=s["out"], lse=s["lse"])


def _plain_mass(s):
    case = s["case"]
    n, m = s["cache_len"].long(), s["n_new"].long()
    count = m.clamp(max=case["last"])
    most = min(case["new_hi"], case["last"])
    x, _, _ = _padded_scores(s, count, most)
    lse = _padded(s, s["lse"], count, most, m - count).view(case["batch"], most, case["hkv"], -1).permute(0, 2, 3, 1)
    p = x.sub_(lse[..., None]).exp_()
    p.masked_fill_((torch.arange(most, device="cuda") >= count[:, None])[:, None, None, :, None], 0.0)
    s["out"].zero_()
    top = p.shape[-1]
    held = (torch.arange(top, device="cuda") < (n + m)[:, None])[:, None]
    before = torch.where((torch.arange(top, device="cuda") < n[:, None])[:, None], s["mass"][..., :top], 0.0)
    s["out"][..., :top] = torch.where(held, before + p.sum((2, 3)), 0.0)       # (a new position starts from nothing)
    return s["out"]


def _plain_evict(s):
    case, P = s["case"], s["case"]["page"]
    budget, recent = case["budget"], case["recent"]
    n, mass = s["cache_len"].long(), s["mass"]
    width = mass.shape[-1]
    pos = torch.arange(width, device="cuda")
    # a key that orders by weight, then by the lower position; the last positions first of all, those not held last
    key = (mass + 0.0).view(torch.int32).long() * (1 << 20) + (width - pos)
    key = torch.where((pos >= n[:, None] - recent)[:, None], (1 << 60) + pos, key)
    key = torch.where((pos < n[:, None])[:, None], key, -1 - pos)
    ids = torch.topk(key, min(budget, width), -1)[1].sort(-1)[0]                          # [layer, seq, head, budget]
    cut = (n > budget)[:, None, None]
    slot = torch.arange(budget, device="cuda")
    kept = torch.full_like(s["kept"], -1)
    kept[..., :ids.shape[-1]] = ids.int()
    kept = torch.where(cut, kept, torch.where(slot < n[:, None], slot, -1).int()[:, None])
    got = torch.gather(mass, 3, kept.long().clamp(min=0)) * (kept >= 0)
    s["out_mass"].zero_()
    s["out_mass"][..., :min(budget, width)] = got[..., :width]
    table, kv = s["table"].long(), s["kv"]
    for b in torch.nonzero(n > budget)[:, 0].tolist():
        src, dst = kept[:, b].long(), slot                                                # [layer, head, budget]
        layer = torch.arange(case["layers"], device="cuda")[:, None, None]
        head = torch.arange(case["hkv"], device="cuda")[:, None]
        moved = kv[table[b][src // P], layer, head, :, src % P]
        kv[table[b][dst // P][None, None], layer, head, :, (dst % P)[None, None]] = moved
    s["kept"].copy_(kept)
    s["len"].copy_(n.clamp(max=budget))
    return dict(kv=kv, mass=s["out_mass"], kept=s["kept"], len=s["len"])


# ---- the framework's calls
def _binding():
    from lossless_speculative_decoding_gb300 import binding
    return binding


def _view(s):
    if "view" not in s:                # the cache's description, which a program keeps
        case = s["case"]
        s["view"] = _binding().make_kv_view(
            s["kv"], s["table"], dtype=BF16 if case["dtype"] == "bf16" else F32, n_pages=s["kv"].shape[0],
            n_layers=s["kv"].shape[1], n_kv_heads=case["hkv"], page_size=case["page"], head_dim=case["d"],
            max_pages=s["table"].shape[1])
    return s["view"]


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _own_rope(s):
    case, B = s["case"], _binding()
    if "rope" not in s:
        s["rope"] = B.make_rope(s["freq"], axis=s["axis"], n_axes=case["axes"])
    B.spec_qk_norm_rope(_view(s), 1, s["qkv"], s["qkv"].stride(0), s["rows"], case["batch"], case["hq"], s["row_start"],
                        s["n_new"], s["cache_len"], s["rope"], s["positions"], s["gamma"][0], s["gamma"][1], s["eps"],
                        s["q"], s["err"], _stream())
    return dict(q=s["q"], kv=s["kv"])


def _own_attention(s):
    case, B = s["case"], _binding()
    if "ws" not in s:
        s["ws_bytes"] = B.spec_chunk_attention_ws_bytes(_view(s), case["batch"], case["new_hi"], case["hq"])
        s["ws"] = torch.empty(s["ws_bytes"], dtype=torch.uint8, device="cuda")
    B.spec_chunk_attention(_view(s), 0, s["q"], s["rows"], case["batch"], case["new_hi"], case["hq"], s["row_start"],
                           s["n_new"], s["cache_len"], s["scale"], s["out"], s["lse"], s["ws"], s["ws_bytes"], s["err"],
                           _stream())
    return dict(out=s["out"], lse=s["lse"])


def _own_mass(s):
    case, B = s["case"], _binding()
    B.spec_attention_mass(_view(s), 0, s["q"], s["lse"], s["rows"], case["batch"], case["new_hi"], case["last"], case["hq"],
                          s["row_start"], s["n_new"], s["cache_len"], s["scale"], s["mass"], s["out"], s["mass"].shape[-1],
                          s["err"], _stream())
    return s["out"]


def _own_evict(s):
    case, B = s["case"], _binding()
    B.spec_kv_evict(_view(s), case["batch"], s["cache_len"], s["mass"], s["mass"].shape[-1], case["budget"], case["recent"],
                    s["out_mass"], s["kept"], s["len"], s["err"], _stream())
    return dict(kv=s["kv"], mass=s["out_mass"], kept=s["kept"], len=s["len"])


# --------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"qk_norm_rope": _exact_rope, "chunk_attention": _exact_attention, "attention_mass": _exact_mass,
            "kv_evict": _exact_evict}[case["op"]](case, s)


def _exact_rope(case, s):
    """One sequence at a time, the pairs as complex numbers."""
    hq, hkv, half, P = case["hq"], case["hkv"], case["rot"] // 2, case["page"]
    out, kv = s["q"].double(), s["kv"].double()
    for b in range(case["batch"]):
        lo, hi, n = int(s["start_host"][b]), int(s["start_host"][b + 1]), int(s["n_host"][b])
        x = s["qkv"][lo:hi].double()
        turn = torch.stack([s["positions"][int(a), lo:hi].double() * float(f) for a, f in zip(s["axis"], s["freq"])], -1)
        turn = torch.polar(torch.ones_like(turn), turn)[:, None]
        y = []
        for part, gamma in ((x[:, :hq], s["gamma"][0]), (x[:, hq:hq + hkv], s["gamma"][1])):
            if gamma is not None:
                part = part / (part.square().mean(-1, keepdim=True) + s["eps"]).sqrt() * gamma.double()
            z = torch.complex(part[..., :half].contiguous(), part[..., half:2 * half].contiguous()) * turn
            y.append(torch.cat([z.real, z.imag, part[..., 2 * half:]], -1))
        out[lo:hi] = y[0]
        for i in range(n // P, -(-(n + hi - lo) // P)):                                   # page by page
            a, z = max(n, i * P), min(n + hi - lo, (i + 1) * P)
            page = kv[int(s["table"][b, i]), 1]
            page[:, 0, a - i * P:z - i * P] = y[1][a - n:z - n].transpose(0, 1)
            page[:, 1, a - i * P:z - i * P] = x[a - n:z - n, hq + hkv:].transpose(0, 1)
    return dict(q=out, kv=kv)


def _exact_attention(case, s):
    out = s["out"].double()
    lse = s["lse"].double()
    for b in range(case["batch"]):
        x, at = _scores(case, s, b, torch.float64, case["new_hi"])
        page, slot = _kept_rows(s, b)
        val = s["kv"][page, 0, :, 1, slot].double()                                       # [top, hkv, d]
        z = torch.logsumexp(x, -1)
        o = torch.matmul(x.sub_(z[..., None]).exp_(), val.permute(1, 0, 2)[:, None])      # [hkv, G, m, d]
        out[at] = o.permute(2, 0, 1, 3).reshape(-1, case["hq"], case["d"])
        lse[at] = z.permute(2, 0, 1).reshape(-1, case["hq"])
    return dict(out=out, lse=lse)


def _exact_mass(case, s):
    out = torch.zeros(s["mass"].shape, dtype=torch.float64, device="cuda")
    for b in range(case["batch"]):
        x, at = _scores(case, s, b, torch.float64, case["last"])
        lse = s["lse"][at].double().view(x.shape[2], x.shape[0], x.shape[1]).permute(1, 2, 0)
        n, top = int(s["n_host"][b]), x.shape[-1]
        out[b, :, :top] = x.sub_(lse[..., None]).exp_().sum((1, 2))
        out[b, :, :n] += s["mass"][b, :, :n].double()
    return out


def _exact_evict(case, s):
    """One plane at a time; the whole numbers have no exact() value."""
    budget, recent, P = case["budget"], case["recent"], case["page"]
    kv, mass = s["kv"].double(), torch.zeros(s["mass"].shape, dtype=torch.float64, device="cuda")
    host = s["mass"].cpu().numpy()
    table = s["table"].cpu().numpy()
    for layer, b, h in np.ndindex(case["layers"], case["batch"], case["hkv"]):
        n = int(s["n_host"][b])
        keep = np.arange(n)
        if n > budget:
            old = np.argsort(-host[layer, b, h, :n - recent], kind="stable")[:budget - recent]
            keep = np.sort(np.concatenate([old, np.arange(n - recent, n)]))
            i, j = torch.from_numpy(keep).cuda(), np.arange(budget)
            pages = torch.from_numpy(table[b].astype(np.int64)).cuda()
            rows = s["kv"][pages[i // P], layer, h, :, i % P].double()
            j = torch.from_numpy(j).cuda()
            kv[pages[j // P], layer, h, :, j % P] = rows
        mass[layer, b, h, :len(keep)] = torch.from_numpy(host[layer, b, h, keep].astype(np.float64)).cuda()
    return dict(kv=kv, mass=mass, kept=None, len=None)
