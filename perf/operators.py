"""Cases of the tree verify operators: tree attention over a paged cache, the
commit of a verified tree, copies of cache pages, and token log probabilities.

Shapes come from the synthetic model configurations: the 3B-MoE decoder (10
heads of 128, 12 layers, vocabulary 129,280), the dense 4B decoder (32 query
and 8 key/value heads of 128, 36 layers, vocabulary 151,936) and the tiny fp32
decoder (4 heads of 64, 2 layers). A cache is [page][layer][kv head][K, V]
[position in page][dim]; sequence s holds its committed positions first and
its drafted nodes in the slots right after them.
"""
import math

import numpy as np
import torch

own = False

F32, BF16 = 0, 1
MAX_NODES = 64
MAX_ATT_BYTES = 0.9e9                      # keys and values of the largest attention case
MAX_SCORES = 64 * 10 * MAX_NODES * 5268    # its scores
MAX_LOGIT_BYTES = 2 * 1100 * 151936        # of the largest log probability case
MAX_MOVED = 32 * 7 * 36 * 8 * 512          # bytes of the rows that the largest commit moves


# --------------------------------------------------------------------------- cases
def listed():
    att = dict(op="tree_attention")
    com = dict(op="tree_commit")
    cop = dict(op="kv_copy_pages")
    lp = dict(op="token_logprobs")
    return [
        # one page being read, 16 drafted nodes: a single request, where latency counts
        dict(att, name="att_moe_b1", dtype="bf16", batch=1, hq=10, hkv=10, d=128, page=16, ctx_lo=1357, ctx_hi=1357,
             nodes_lo=16, nodes_hi=16),
        # the 64-sequence serving workload: short and long documents side by side, 32 nodes at most
        dict(att, name="att_moe_b64", dtype="bf16", batch=64, hq=10, hkv=10, d=128, page=16, ctx_lo=336, ctx_hi=5236,
             nodes_lo=17, nodes_hi=32),
        # grouped heads and full trees: 64 nodes x 4 query heads share every key
        dict(att, name="att_dense_b8", dtype="bf16", batch=8, hq=32, hkv=8, d=128, page=64, ctx_lo=1288, ctx_hi=5288,
             nodes_lo=64, nodes_hi=64),
        # two long contexts of odd length, a small odd tree
        dict(att, name="att_dense_long", dtype="bf16", batch=2, hq=32, hkv=8, d=128, page=16, ctx_lo=21845,
             ctx_hi=65521, nodes_lo=21, nodes_hi=21),
        # the fp32 decoder
        dict(att, name="att_tiny_f32", dtype="f32", batch=4, hq=4, hkv=4, d=64, page=16, ctx_lo=72, ctx_hi=200,
             nodes_lo=5, nodes_hi=8),
        # one sequence commits a few nodes in all 12 layers
        dict(com, name="commit_moe_b1", dtype="bf16", batch=1, layers=12, hkv=10, d=128, page=16, ctx_lo=1357,
             ctx_hi=1357, nodes_lo=16, nodes_hi=16, acc_lo=3, acc_hi=3, vocab=129280),
        # 32 sequences with deep trees in 36 layers: block drafts accepted far
        dict(com, name="commit_dense_b32", dtype="bf16", batch=32, layers=36, hkv=8, d=128, page=16, ctx_lo=100,
             ctx_hi=401, nodes_lo=40, nodes_hi=64, acc_lo=0, acc_hi=14, vocab=151936),
        # a sequence forked: its last page, partly filled, becomes two
        dict(cop, name="copy_moe_1", dtype="bf16", layers=12, hkv=10, d=128, page=16, pages=40, n=1),
        # 32 sequences forked four ways
        dict(cop, name="copy_dense_96", dtype="bf16", layers=36, hkv=8, d=128, page=16, pages=256, n=96),
        # the rows of one verify step, five alternatives
        dict(lp, name="lp_moe_4", dtype="f32", rows=4, vocab=129280, top=5, temperature=1.0),
        # the rows of the 64-sequence step, twenty alternatives
        dict(lp, name="lp_moe_256", dtype="f32", rows=256, vocab=129280, top=20, temperature=0.7),
        # a prompt's rows scored from 16-bit logits
        dict(lp, name="lp_dense_1100", dtype="bf16", rows=1100, vocab=151936, top=1, temperature=1.0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree_attention", "tree_attention", "tree_commit", "kv_copy_pages", "token_logprobs"])
    if op == "token_logprobs":
        vocab, dtype = rng.choice([129280, 151936, _log_int(rng, 2, 262144)]), rng.choice(["f32", "bf16"])
        most = MAX_LOGIT_BYTES // (vocab * (2 if dtype == "bf16" else 4))
        return dict(op=op, dtype=dtype, rows=_log_int(rng, 1, max(1, min(2048, most))), vocab=vocab, top=rng.randint(0, min(20, vocab)), temperature=rng.choice([1.0, 0.7, 1.3]))
    hq, hkv, d = rng.choice([(10, 10, 128), (32, 8, 128), (4, 4, 64), (16, 2, 64), (12, 1, 128)])
    page = rng.choice([16, 16, 32, 48, 64, 128])
    dtype = "bf16" if rng.random() < 0.8 else "f32"
    esz = 2 if dtype == "bf16" else 4
    if op == "kv_copy_pages":
        layers = rng.choice([2, 12, 36])
        per = layers * hkv * 2 * page * d * esz
        n = _log_int(rng, 1, max(1, min(512, int(2.2e8 // per))))
        return dict(op=op, dtype=dtype, layers=layers, hkv=hkv, d=d, page=page, pages=2 * n + rng.randint(0, 9), n=n)
    hi = rng.randint(1, MAX_NODES)
    lo = rng.randint(1, hi)
    if op == "tree_commit":
        layers = rng.choice([2, 12, 36])
        batch = _log_int(rng, 1, 32)
        top = _log_int(rng, 1, 400)
        acc = rng.randint(0, min(14, max(0, hi - 2)))
        while batch > 1 and batch * (top + 64 + page) * layers * hkv * 2 * d * esz > 2.5e9:
            batch //= 2
        while batch > 1 and batch * acc * layers * hkv * 2 * d * esz > 2 * MAX_MOVED:
            batch //= 2
        return dict(op=op, dtype=dtype, batch=batch, layers=layers, hkv=hkv, d=d, page=page,
                    ctx_lo=rng.randint(0, top), ctx_hi=top, nodes_lo=lo, nodes_hi=hi, acc_lo=rng.randint(0, acc), acc_hi=acc,
                    vocab=rng.choice([1024, 129280, 151936]))
    if dtype == "f32":         # the fp32 decoder serves short prompts
        batch, top, hi = _log_int(rng, 1, 8), _log_int(rng, 1, 1000), min(hi, 32)
        lo = min(lo, hi)
    else:
        batch, top = _log_int(rng, 1, 64), _log_int(rng, 1, 65536)
    while batch * (top + 64) * hkv * 2 * d * esz > MAX_ATT_BYTES or batch * hq * MAX_NODES * (top + 64) > MAX_SCORES:
        batch, top = max(1, batch // 2), max(1, top - top // 4)
    return dict(op=op, dtype=dtype, batch=batch, hq=hq, hkv=hkv, d=d, page=page, ctx_lo=rng.randint(0, top), ctx_hi=top,
                nodes_lo=lo, nodes_hi=hi)


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


def _nodes(case):
    return _spread(case["nodes_lo"], case["nodes_hi"], case["batch"], 0.4142135623730951)


def _accepted(case):
    return np.clip(_spread(case["acc_lo"], case["acc_hi"], case["batch"], 0.7320508075688772), 0,
                   np.maximum(_nodes(case) - 2, 0))


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def work(case):
    esz = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "tree_attention":
        n, k = _lengths(case), _nodes(case)
        kv = float(((n + k) * case["hkv"] * 2 * case["d"] * esz).sum())
        qo = float((k * case["hq"] * case["d"] * 2 * esz).sum())
        return {"bytes": kv + qo + 4.0 * float(k.sum()), "flops": 4.0 * case["d"] * case["hq"] * float((k * (n + 1)).sum())}
    if case["op"] == "tree_commit":
        row = case["layers"] * case["hkv"] * 2 * case["d"] * esz
        return {"bytes": 2.0 * row * float(_accepted(case).sum()) + 12.0 * float(_nodes(case).sum()), "flops": 0.0}
    if case["op"] == "kv_copy_pages":
        return {"bytes": 2.0 * case["n"] * case["layers"] * case["hkv"] * 2 * case["page"] * case["d"] * esz, "flops": 0.0}
    return {"bytes": float(case["rows"]) * (case["vocab"] * esz + 16 + 8 * case["top"]),
            "flops": 6.0 * case["rows"] * case["vocab"]}


# --------------------------------------------------------------------------- inputs
def _random_tree(r, n, chain):
    """Parents of n nodes: node 0 the root, `chain` a path below it, the others under any earlier node, mostly a late one."""
    parents = np.full(MAX_NODES, -1, np.int32)
    for i in range(1, n):
        parents[i] = max(0, i - 1 - int(r.exponential(4.0)))
    last = 0
    for c in chain:
        parents[c] = last
        last = c
    return parents


def _cache(case, gen, r, layers):
    """A cache with the sequences' pages in random order, their block table and lengths."""
    n, k, P = _lengths(case), _nodes(case), case["page"]
    order = r.permutation(len(n))
    n, k = n[order], k[order]
    need = -(-(n + k) // P)
    max_pages = int(need.max()) + 1
    n_pages = int(need.sum()) + 3
    table = np.full((len(n), max_pages), -1, np.int32)
    ids, at = r.permutation(n_pages).astype(np.int32), 0
    for s in range(len(n)):
        table[s, :need[s]] = ids[at:at + need[s]]
        at += need[s]
    kv = torch.empty((n_pages, layers, case["hkv"], 2, P, case["d"]), dtype=_dtype(case), device="cuda")
    kv.normal_(generator=gen)
    return dict(kv=kv, table=_dev(table), cache_len=_dev(n), n_nodes=_dev(k), n_host=n, k_host=k, order=order,
                err=torch.zeros(1, dtype=torch.int32, device="cuda"))


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    r = np.random.default_rng(int(seed))
    s = dict(case=case)
    if case["op"] == "tree_attention":
        s.update(_cache(case, gen, r, 1))
        s["parents"] = _dev(np.stack([_random_tree(r, int(n), ()) for n in s["k_host"]]))
        q = torch.empty((case["batch"], MAX_NODES, case["hq"], case["d"]), dtype=torch.float32, device="cuda")
        # heads differ in how sharply they look
        q.normal_(generator=gen).mul_(torch.linspace(0.5, 3.0, case["hq"], device="cuda")[:, None])
        s["q"] = q.to(_dtype(case))
        s["scale"] = 1.0 / math.sqrt(case["d"])
        s["out"] = torch.zeros_like(s["q"])
    elif case["op"] == "tree_commit":
        s.update(_cache(case, gen, r, case["layers"]))
        acc, V = _accepted(case)[s["order"]], case["vocab"]
        # drafted and target tokens below V - 1: the target after the accepted path is V - 1, which no node drafts
        tokens = r.integers(0, V - 1, (case["batch"], MAX_NODES)).astype(np.int32)
        target = r.integers(0, V - 1, (case["batch"], MAX_NODES)).astype(np.int32)
        parents = np.full((case["batch"], MAX_NODES), -1, np.int32)
        for i in range(case["batch"]):
            k, a = int(s["k_host"][i]), int(acc[i])
            chain = np.sort(r.permutation(max(k - 2, 0))[:a]) + 2
            parents[i] = _random_tree(r, k, [int(c) for c in chain])
            walk = [0] + [int(c) for c in chain]
            for j in range(a):
                target[i, walk[j]] = tokens[i, walk[j + 1]]
            target[i, walk[-1]] = V - 1
        s.update(parents=_dev(parents), tokens=_dev(tokens), target=_dev(target))
        full = lambda *shape: torch.full(shape, -1, dtype=torch.int32, device="cuda")  # noqa: E731
        s.update(accepted=full(case["batch"]), token=full(case["batch"]), length=full(case["batch"]),
                 path=full(case["batch"], MAX_NODES))
    elif case["op"] == "kv_copy_pages":
        kv = torch.empty((case["pages"], case["layers"], case["hkv"], 2, case["page"], case["d"]), dtype=_dtype(case),
                         device="cuda")
        kv.normal_(generator=gen)
        ids = r.permutation(case["pages"])
        # a page may be the source of several copies
        src = ids[case["n"]:][r.integers(0, case["pages"] - case["n"], case["n"])]
        s.update(kv=kv, src=_dev(src), dst=_dev(ids[:case["n"]]), src_i=torch.from_numpy(src).cuda(),
                 dst_i=torch.from_numpy(ids[:case["n"]]).cuda(), err=torch.zeros(1, dtype=torch.int32, device="cuda"))
    else:
        R, V, n = case["rows"], case["vocab"], case["top"]
        x = torch.empty((R, V), dtype=torch.float32, device="cuda").normal_(generator=gen)
        # rows from flat to peaked, as a decoder's are
        x.mul_(torch.linspace(0.5, 4.0, R, device="cuda")[:, None])
        s["logits"] = x.to(_dtype(case))
        s["tokens"] = torch.where(torch.rand(R, generator=gen, device="cuda") < 0.6, s["logits"].argmax(-1),
                                  torch.randint(0, V, (R,), generator=gen, device="cuda")).to(torch.int32)
        f = lambda *shape: torch.empty(shape, dtype=torch.float32, device="cuda")  # noqa: E731
        w = lambda *shape: torch.empty(shape, dtype=torch.int32, device="cuda")  # noqa: E731
        s.update(logprob=f(R), entropy=f(R), rank=w(R), top_ids=w(R, n), top_logprobs=f(R, n))
    return s


# --------------------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"tree_attention": _own_attention, "tree_commit": _own_commit, "kv_copy_pages": _own_copy,
                "token_logprobs": _own_logprobs}[op](state)
    return {"tree_attention": _plain_attention, "tree_commit": _plain_commit, "kv_copy_pages": _plain_copy,
            "token_logprobs": _plain_logprobs}[op](state)


# ---- plain forms
def _ancestors(parents):
    """[n, i, j]: 1 where j is i or above i. With A the child -> parent matrix, sum of A^k = (I - A)^-1: a tree has one
    path from a node to one above it, so the inverse holds zeros and ones."""
    n, N = parents.shape
    eye = torch.eye(N, device=parents.device)
    up = (parents[:, :, None] == torch.arange(N, device=parents.device)).float()
    return torch.linalg.solve_triangular(eye - up, eye.expand(n, N, N), upper=False, unitriangular=True)


def _plain_attention(s):
    case = s["case"]
    kv, P, hq, hkv, d = s["kv"], case["page"], case["hq"], case["hkv"], case["d"]
    n, k = s["cache_len"].long(), s["n_nodes"].long()
    B, top = case["batch"], case["ctx_hi"] + case["nodes_hi"]
    pos = torch.arange(top, device="cuda")
    page = s["table"].long()[:, torch.div(pos, P, rounding_mode="floor")].clamp(min=0)          # [B, top]
    key = kv[page, 0, :, 0, pos % P].permute(0, 2, 1, 3).float()                                  # [B, hkv, top, d]
    val = kv[page, 0, :, 1, pos % P].permute(0, 2, 1, 3).float()
    node = pos[None] - n[:, None]                                                                 # tree index of a slot
    inside = (node < k[:, None])
    val = torch.where(inside[:, None, :, None], val, 0.0)
    anc = _ancestors(s["parents"])
    tree = torch.gather(anc, 2, node.clamp(0, MAX_NODES - 1)[:, None].expand(B, MAX_NODES, top)) > 0
    see = torch.where((node < 0)[:, None], True, tree & inside[:, None])                          # [B, N, top]
    q = s["q"].float().view(B, MAX_NODES, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(B, hkv, -1, d)
    x = torch.matmul(q, key.transpose(2, 3)).mul_(s["scale"]).view(B, hkv, hq // hkv, MAX_NODES, top)
    x.masked_fill_(~see[:, None, None], float("-inf"))
    p = torch.exp(x - x.amax(-1, keepdim=True))
    o = torch.matmul((p / p.sum(-1, keepdim=True)).view(B, hkv, -1, top), val)
    o = o.view(B, hq, MAX_NODES, d).permute(0, 2, 1, 3)
    live = (torch.arange(MAX_NODES, device="cuda") < k[:, None])[:, :, None, None]
    return torch.where(live, o.to(s["q"].dtype), s["out"])


def _plain_commit(s):
    case, P = s["case"], s["case"]["page"]
    n, k, parents, tokens, target = (s[x].long() for x in ("cache_len", "n_nodes", "parents", "tokens", "target"))
    idx = torch.arange(MAX_NODES, device="cuda")
    live = idx < k[:, None]
    ok = live & (parents >= 0) & (tokens == torch.gather(target, 1, parents.clamp(min=0)))
    # of several children that agree, the first one
    twin = (parents[:, :, None] == parents[:, None, :]) & ok[:, None, :] & (idx[None, :] < idx[:, None])
    fine = (ok & ~twin.any(-1)) | ((idx == 0) & live)
    anc = _ancestors(s["parents"])
    taken = live & (torch.matmul(anc, (~fine).float()[:, :, None])[..., 0] == 0)
    path, _ = torch.where(taken, idx, MAX_NODES).sort(-1)
    count = taken.sum(-1)
    path = torch.where(path < MAX_NODES, path, -1)
    token = torch.gather(target, 1, torch.gather(path, 1, (count - 1)[:, None]))[:, 0]
    src = n[:, None] + torch.where(path >= 0, path, 0)
    dst = n[:, None] + torch.where(path >= 0, idx, 0)
    table, kv = s["table"].long(), s["kv"]
    rows = kv[torch.gather(table, 1, src // P), :, :, :, src % P]
    kv[torch.gather(table, 1, dst // P), :, :, :, dst % P] = rows
    return dict(accepted=(count - 1).int(), token=token.int(), path=path.int(), length=(n + count).int(), kv=kv)


def _plain_copy(s):
    s["kv"][s["dst_i"]] = s["kv"][s["src_i"]]
    return s["kv"]


def _plain_logprobs(s):
    case = s["case"]
    V, raw = case["vocab"], s["logits"].float()
    x = raw * (1.0 / case["temperature"])
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    z = e.sum(-1)
    lse = m[:, 0] + torch.log(z)
    t = s["tokens"].long()[:, None]
    idx = torch.arange(V, device="cuda")
    xt = torch.gather(raw, 1, t)
    rank = 1 + ((raw > xt) | ((raw == xt) & (idx < t))).sum(-1)
    entropy = torch.log(z) - torch.where(e > 0, e * (x - m), 0.0).sum(-1) / z
    out = dict(logprob=torch.gather(x, 1, t)[:, 0] - lse, entropy=entropy, rank=rank.int())
    if case["top"]:
        # keys that order by value, then by the lower index (+ 0.0: one zero)
        b = (raw + 0.0).view(torch.int32).long()
        key = torch.where(b < 0, b ^ 0x7FFFFFFF, b) * (1 << 20) + (V - 1 - idx)
        ids = torch.topk(key, case["top"], -1)[1]
        out.update(top_ids=ids.int(), top_logprobs=torch.gather(x, 1, ids) - lse[:, None])
    return out


# ---- the framework's calls
def _binding():
    from lossless_speculative_decoding_gb300 import binding
    return binding


def _view(s):
    case, B = s["case"], _binding()
    return B.make_kv_view(s["kv"], s.get("table"), dtype=BF16 if case["dtype"] == "bf16" else F32,
                          n_pages=s["kv"].shape[0], n_layers=s["kv"].shape[1], n_kv_heads=case["hkv"],
                          page_size=case["page"], head_dim=case["d"], max_pages=s["table"].shape[1] if "table" in s else 0)


def _own_attention(s):
    case, B = s["case"], _binding()
    if "view" not in s:      # the cache's description and the workspace, which a program keeps
        s["view"] = _view(s)
        s["ws_bytes"] = B.spec_tree_attention_ws_bytes(s["view"], case["batch"], MAX_NODES, case["hq"])
        s["ws"] = torch.empty(s["ws_bytes"], dtype=torch.uint8, device="cuda")
    B.spec_tree_attention(s["view"], 0, s["q"], case["batch"], MAX_NODES, case["hq"], s["cache_len"], s["n_nodes"],
                          s["parents"], s["scale"], s["out"], s["ws"], s["ws_bytes"], s["err"],
                          torch.cuda.current_stream().cuda_stream)
    return s["out"]


def _own_commit(s):
    case, B = s["case"], _binding()
    if "view" not in s:
        s["view"] = _view(s)
    B.spec_tree_commit(s["view"], case["batch"], MAX_NODES, s["tokens"], s["parents"], s["n_nodes"], s["target"],
                       s["cache_len"], s["accepted"], s["token"], s["path"], s["length"], s["err"],
                       torch.cuda.current_stream().cuda_stream)
    return {x: s[x] for x in ("accepted", "token", "path", "length", "kv")}


def _own_copy(s):
    case, B = s["case"], _binding()
    if "view" not in s:
        s["view"] = _view(s)
    B.spec_kv_copy_pages(s["view"], s["src"], s["dst"], case["n"], s["err"], torch.cuda.current_stream().cuda_stream)
    return s["kv"]


def _own_logprobs(s):
    case, B = s["case"], _binding()
    R, V, n = case["rows"], case["vocab"], case["top"]
    if "ws" not in s:
        s["ws_bytes"] = B.spec_token_logprobs_ws_bytes(R, V, n)
        s["ws"] = torch.zeros(s["ws_bytes"], dtype=torch.uint8, device="cuda")
    B.spec_token_logprobs(s["logits"], BF16 if case["dtype"] == "bf16" else F32, V, R, V, s["tokens"], case["temperature"],
                          n, s["logprob"], s["entropy"], s["rank"], s["top_ids"], s["top_logprobs"], s["ws"],
                          s["ws_bytes"], torch.cuda.current_stream().cuda_stream)
    out = {x: s[x] for x in ("logprob", "entropy", "rank")}
    return dict(out, top_ids=s["top_ids"], top_logprobs=s["top_logprobs"]) if n else out


# --------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    if case["op"] == "tree_attention":
        return _exact_attention(case, prepare(case, seed))
    if case["op"] == "token_logprobs":
        return _exact_logprobs(case, prepare(case, seed))
    return _exact_moves(case, prepare(case, seed))


def _exact_attention(case, s):
    """One sequence at a time, the keys of every node listed by climbing from it."""
    P, G = case["page"], case["hq"] // case["hkv"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    parents = s["parents"].cpu().numpy()
    for b in range(case["batch"]):
        n, k = int(s["n_host"][b]), int(s["k_host"][b])
        pages = s["table"][b].long()[: -(-(n + k) // P)]
        rows = s["kv"][pages, 0].permute(1, 2, 0, 3, 4).reshape(case["hkv"], 2, -1, case["d"])[:, :, : n + k].double()
        hide = np.ones((k, n + k), bool)
        hide[:, :n] = False
        for i in range(k):
            j = i
            while j >= 0:
                hide[i, n + j] = False
                j = int(parents[b, j])
        hide = torch.from_numpy(hide).cuda()
        q = s["q"][b, :k].double().view(k, case["hkv"], G, case["d"])
        x = torch.einsum("ihgd,hjd->hgij", q, rows[:, 0]) * s["scale"]
        w = torch.softmax(x.masked_fill(hide, float("-inf")), -1)
        out[b, :k] = torch.einsum("hgij,hjd->ihgd", w, rows[:, 1]).reshape(k, case["hq"], case["d"])
    return out


def _exact_logprobs(case, s):
    got = {"logprob": [], "entropy": [], "top_logprobs": []}
    for x, t in zip(s["logits"].split(64), s["tokens"].long().split(64)):
        lp = torch.log_softmax(x.double() / case["temperature"], -1)
        got["logprob"].append(lp[torch.arange(len(t), device="cuda"), t])
        got["entropy"].append(-(lp.exp() * lp).sum(-1))
        got["top_logprobs"].append(lp.sort(-1, descending=True)[0][:, : case["top"]])
    out = dict(logprob=torch.cat(got["logprob"]), entropy=torch.cat(got["entropy"]), rank=None)
    if case["top"]:
        out.update(top_ids=None, top_logprobs=torch.cat(got["top_logprobs"]))
    return out


def _exact_moves(case, s):
    """The cache after a commit or copies, one sequence or page at a time; the whole numbers have no exact() value."""
    kv = s["kv"].double()
    if case["op"] == "kv_copy_pages":
        for a, b in zip(s["src_i"].tolist(), s["dst_i"].tolist()):
            kv[b] = s["kv"][a]
        return kv
    P = case["page"]
    table, parents, tokens, target = (s[x].cpu().numpy() for x in ("table", "parents", "tokens", "target"))
    for b in range(case["batch"]):
        n, k, at, j = int(s["n_host"][b]), int(s["k_host"][b]), 0, 0
        while True:
            below = [c for c in range(1, k) if parents[b, c] == at and tokens[b, c] == target[b, at]]
            if not below:
                break
            at, j = below[0], j + 1
            src, dst = n + at, n + j
            kv[table[b, dst // P], :, :, :, dst % P] = s["kv"][table[b, src // P], :, :, :, src % P].double()
    return dict(accepted=None, token=None, path=None, length=None, kv=kv)
