"""Refusals of the tree entry points, on the host before any CUDA call (the
pointers here are never dereferenced)."""
import pytest

FAKE = 1 << 20


@pytest.fixture(scope="module")
def B():
    from lossless_speculative_decoding_gb300 import build, binding
    build.build()
    return binding


def _view(B, **kw):
    a = dict(dtype=1, n_pages=8, n_layers=2, n_kv_heads=2, page_size=16, head_dim=128, max_pages=4)
    a.update(kw)
    kv, bt = a.pop("kv", FAKE), a.pop("bt", FAKE)
    return B.make_kv_view(kv, bt, **a)


VIEWS = [(dict(kv=0), -1), (dict(kv=FAKE + 8), -1), (dict(dtype=2), -6), (dict(head_dim=96), -6), (dict(page_size=24), -1),
         (dict(page_size=0), -1), (dict(n_pages=0), -1), (dict(n_layers=0), -1), (dict(n_kv_heads=0), -1)]
TABLES = [(dict(bt=0), -1), (dict(max_pages=0), -1), (dict(max_pages=1 << 28), -6)]


def _refused(B, f, args, code):
    with pytest.raises(B.SpecError) as e:
        f(**args)
    assert e.value.code == code, (args, str(e.value))
    assert str(e.value)


def test_attention_refusals(B):
    ok = dict(kv=_view(B), layer=0, q_dev=FAKE, n_seq=2, max_nodes=64, n_q_heads=4, cache_len_dev=FAKE, n_nodes_dev=FAKE,
              parents_dev=FAKE, scale=0.1, out_dev=FAKE, ws_dev=FAKE, ws_bytes=1 << 40, err_dev=FAKE)
    need = B.spec_tree_attention_ws_bytes(ok["kv"], 2, 64, 4)
    assert need > 0
    cases = [(dict(kv=_view(B, **v)), c) for v, c in VIEWS + TABLES]
    cases += [(dict(layer=-1), -1), (dict(layer=2), -1), (dict(n_seq=0), -1), (dict(n_seq=65536), -1), (dict(max_nodes=0), -1),
              (dict(max_nodes=65), -1), (dict(n_q_heads=3), -1), (dict(n_q_heads=0), -1), (dict(n_q_heads=258), -6),
              (dict(scale=0.0), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
              (dict(ws_bytes=need - 1), -1), (dict(ws_dev=FAKE + 4), -1), (dict(q_dev=FAKE + 2), -1),
              (dict(out_dev=FAKE + 8), -1)]
    cases += [({k: None}, -1) for k in ("q_dev", "cache_len_dev", "n_nodes_dev", "parents_dev", "out_dev", "ws_dev", "err_dev")]
    for change, code in cases:
        _refused(B, B.spec_tree_attention, {**ok, **change}, code)
    with pytest.raises(B.SpecError):
        B.spec_tree_attention_ws_bytes(ok["kv"], 2, 65, 4)


def test_commit_refusals(B):
    ok = dict(kv=_view(B), n_seq=2, max_nodes=64, tokens_dev=FAKE, parents_dev=FAKE, n_nodes_dev=FAKE, target_dev=FAKE,
              cache_len_dev=FAKE, out_accepted_dev=FAKE, out_token_dev=FAKE, out_path_dev=FAKE, out_len_dev=FAKE + 64,
              err_dev=FAKE)
    cases = [(dict(kv=_view(B, **v)), c) for v, c in VIEWS + TABLES]
    cases += [(dict(n_seq=0), -1), (dict(n_seq=65536), -1), (dict(max_nodes=0), -1), (dict(max_nodes=65), -1),
              (dict(out_len_dev=FAKE), -1)]
    cases += [({k: None}, -1) for k in ok if k.endswith("_dev")]
    for change, code in cases:
        _refused(B, B.spec_tree_commit, {**ok, **change}, code)


def test_copy_refusals(B):
    ok = dict(kv=_view(B, bt=0, max_pages=0), src_dev=FAKE, dst_dev=FAKE, n=3, err_dev=FAKE)
    cases = [(dict(kv=_view(B, **v)), c) for v, c in VIEWS]
    cases += [(dict(n=-1), -1)] + [({k: None}, -1) for k in ("src_dev", "dst_dev", "err_dev")]
    for change, code in cases:
        _refused(B, B.spec_kv_copy_pages, {**ok, **change}, code)
    B.spec_kv_copy_pages(**{**ok, "n": 0, "src_dev": None, "dst_dev": None})       # nothing to copy


def test_logprobs_refusals(B):
    ok = dict(logits_dev=FAKE, dtype=0, ld=1000, n_rows=4, vocab=1000, tokens_dev=FAKE, temperature=1.0, top_n=5,
              out_logprob_dev=FAKE, out_entropy_dev=FAKE, out_rank_dev=FAKE, out_top_ids_dev=FAKE, out_top_logprobs_dev=FAKE,
              ws_dev=FAKE, ws_bytes=1 << 40)
    need = B.spec_token_logprobs_ws_bytes(4, 1000, 5)
    assert need > 0
    cases = [(dict(logits_dev=None), -1), (dict(ws_dev=None), -1), (dict(tokens_dev=None), -1), (dict(out_top_ids_dev=None), -1),
             (dict(out_top_logprobs_dev=None), -1), (dict(dtype=2), -6), (dict(vocab=1 << 21, ld=1 << 21), -6), (dict(ld=999), -1),
             (dict(n_rows=0), -1), (dict(vocab=0), -1), (dict(top_n=-1), -1), (dict(top_n=33), -1),
             (dict(vocab=4, top_n=5), -1), (dict(temperature=0.0), -1), (dict(temperature=float("nan")), -1),
             (dict(temperature=-1.0), -1), (dict(temperature=float("inf")), -1), (dict(temperature=1e-45), -1),
             (dict(logits_dev=FAKE + 2), -1), (dict(ws_dev=FAKE + 8), -1), (dict(ws_bytes=need - 1), -1)]
    for change, code in cases:
        _refused(B, B.spec_token_logprobs, {**ok, **change}, code)
    for bad in ((0, 10, 1), (1, 0, 0), (1, 10, 11), (1, 10, -1), (1, 100, 33)):
        with pytest.raises(B.SpecError):
            B.spec_token_logprobs_ws_bytes(*bad)


def test_views_past_32_bits_are_refused(B):
    """Planes, a page's rows and positions are counted in 32 bits."""
    ok = dict(layer=0, q_dev=FAKE, n_seq=2, max_nodes=64, n_q_heads=4, cache_len_dev=FAKE, n_nodes_dev=FAKE, parents_dev=FAKE,
              scale=0.1, out_dev=FAKE, ws_dev=FAKE, ws_bytes=1 << 40, err_dev=FAKE)
    for v in (dict(n_pages=1 << 29), dict(page_size=1 << 28), dict(n_layers=1 << 25), dict(max_pages=1 << 27, page_size=16)):
        _refused(B, B.spec_tree_attention, {**ok, "kv": _view(B, **v)}, -6)
    _refused(B, B.spec_tree_attention, {**ok, "kv": _view(B, max_pages=1 << 26, n_kv_heads=16), "n_q_heads": 2048}, -6)
