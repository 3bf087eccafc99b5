"""Refusals of the entry points for chunks of new tokens, on the host before any
CUDA call (the pointers here are never dereferenced)."""
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
    kv, bt = a.pop("kv", 64 << 20), a.pop("bt", FAKE)
    return B.make_kv_view(kv, bt, **a)


VIEWS = [(dict(kv=0), -1), (dict(kv=FAKE + 8), -1), (dict(dtype=2), -6), (dict(head_dim=96), -6), (dict(page_size=24), -1),
         (dict(page_size=0), -1), (dict(n_pages=0), -1), (dict(n_layers=0), -1), (dict(n_kv_heads=0), -1), (dict(bt=0), -1),
         (dict(max_pages=0), -1), (dict(max_pages=1 << 28), -6), (dict(n_pages=1 << 29), -6), (dict(page_size=1 << 28), -6)]


def _refused(B, f, args, code):
    with pytest.raises(B.SpecError) as e:
        f(**args)
    assert e.value.code == code, (args, str(e.value))
    assert str(e.value)


def _all(B, f, ok, cases):
    for change, code in [(dict(kv=_view(B, **v)), c) for v, c in VIEWS] + cases:
        _refused(B, f, {**ok, **change}, code)


INDEX = dict(n_rows=8, n_seq=2, n_q_heads=4, row_start_dev=FAKE, n_new_dev=FAKE, cache_len_dev=FAKE, err_dev=FAKE)
SIZES = [(dict(layer=-1), -1), (dict(layer=2), -1), (dict(n_rows=0), -1), (dict(n_seq=0), -1), (dict(n_seq=65536), -1),
         (dict(n_q_heads=3), -1), (dict(n_q_heads=0), -1)]
SCALES = [(dict(scale=x), -1) for x in (0.0, -1.0, float("nan"), float("inf"), 2.4e38)]


def test_rope_refusals(B):
    rope = B.make_rope([1.0] * 64)
    ok = dict(INDEX, kv=_view(B), layer=0, qkv_dev=FAKE, ld=1024, rope=rope, positions_dev=FAKE, q_gamma_dev=FAKE,
              k_gamma_dev=FAKE, eps=1e-6, q_out_dev=FAKE << 1)

    def rp(**kw):
        r = B.make_rope([1.0] * 32, n_axes=2)
        for k, v in kw.items():
            setattr(r, k, v)
        return dict(rope=r)

    def pair(field, p, v):
        r = B.make_rope([1.0] * 32, n_axes=2)
        getattr(r, field)[p] = v
        return dict(rope=r)

    cases = SIZES + [({k: None}, -1) for k in ("qkv_dev", "row_start_dev", "n_new_dev", "cache_len_dev", "positions_dev",
                                               "q_out_dev", "err_dev")]
    cases += [(dict(ld=1 << 61), -6), (dict(ld=1023), -1), (dict(ld=1016), -1), (dict(ld=1028), -1), (dict(qkv_dev=FAKE + 8), -1),
              (dict(q_out_dev=(FAKE << 1) + 4), -1), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1),
              (rp(dim=-16), -1), (rp(dim=24), -1), (rp(dim=144), -1), (rp(n_axes=0), -1), (rp(n_axes=5), -1),
              (pair("freq", 31, float("nan")), -1), (pair("freq", 0, float("inf")), -1), (pair("axis", 7, 2), -1)]
    # rows of 8 heads x 128 bf16 in 8 rows: 16 KB; queries 8 KB; the cache 8 x 2 x 2 x 2 x 16 x 128 bf16: 256 KB
    cases += [(dict(q_out_dev=FAKE + x), -1) for x in (0, 16, 16384 - 16, 16 - 8192)]
    cases += [(dict(q_out_dev=(64 << 20) + x), -1) for x in (0, 262144 - 16, 16 - 8192)]
    cases += [(dict(qkv_dev=(64 << 20) + x), -1) for x in (0, 262144 - 16, 16 - 16384)]
    _all(B, B.spec_qk_norm_rope, ok, cases)
    with pytest.raises(ValueError):
        B.make_rope([1.0] * 65)
    with pytest.raises(ValueError):
        B.make_rope([1.0] * 8, axis=[0] * 7)


def test_attention_refusals(B):
    ok = dict(INDEX, kv=_view(B), layer=0, q_dev=FAKE, max_new=8, scale=0.1, out_dev=FAKE << 1, out_lse_dev=None, ws_dev=FAKE,
              ws_bytes=1 << 40)
    need = B.spec_chunk_attention_ws_bytes(ok["kv"], 2, 8, 4)
    assert need > 0
    cases = SIZES + SCALES + [({k: None}, -1) for k in ("q_dev", "row_start_dev", "n_new_dev", "cache_len_dev", "out_dev",
                                                        "ws_dev", "err_dev")]
    cases += [(dict(max_new=0), -1), (dict(n_q_heads=258), -6), (dict(ws_bytes=need - 1), -1), (dict(ws_dev=FAKE + 4), -1),
              (dict(q_dev=FAKE + 2), -1), (dict(out_dev=FAKE + 8), -1)]
    # out next to q is fine, over a part of it is not: 8 rows x 4 heads x 128 bf16 = 8 KB
    cases += [(dict(out_dev=FAKE + x), -1) for x in (16, 8192 - 16, -16)]
    # lse, 128 bytes, over a part of either
    cases += [(dict(out_lse_dev=FAKE + x), -1) for x in (0, 8192 - 4, -124)]
    cases += [(dict(out_lse_dev=(FAKE << 1) + x), -1) for x in (0, 8192 - 4, -124)]
    cases += [(dict(kv=_view(B, max_pages=1 << 26, n_kv_heads=256), n_q_heads=256), -6),
              (dict(kv=_view(B, max_pages=1 << 26), n_q_heads=256, max_new=1 << 28), -6)]
    _all(B, B.spec_chunk_attention, ok, cases)
    for bad in ((0, 8, 4), (2, 0, 4), (2, 8, 3)):
        with pytest.raises(B.SpecError):
            B.spec_chunk_attention_ws_bytes(ok["kv"], *bad)


def test_mass_refusals(B):
    ok = dict(INDEX, kv=_view(B), layer=0, q_dev=FAKE, lse_dev=FAKE, max_new=8, last=4, scale=0.1, mass_dev=None,
              out_mass_dev=FAKE << 1, ld=64)
    cases = SIZES + SCALES + [({k: None}, -1) for k in ("q_dev", "lse_dev", "row_start_dev", "n_new_dev", "cache_len_dev",
                                                        "out_mass_dev", "err_dev")]
    cases += [(dict(max_new=0), -1), (dict(last=0), -1), (dict(n_q_heads=258), -6), (dict(ld=0), -1), (dict(ld=1 << 32), -1),
              (dict(q_dev=FAKE + 2), -1), (dict(scale=5e-20), -6), (dict(scale=2e19), -6)]
    # 2 sequences x 2 heads x 64 f32: 1 KB
    cases += [(dict(mass_dev=(FAKE << 1) + x), -1) for x in (4, 1020, -4, -1020)]
    cases += [(dict(out_mass_dev=FAKE + x), -1) for x in (0, 8192 - 4, -1020)]
    cases += [(dict(lse_dev=(FAKE << 1) + x), -1) for x in (0, 1020, -124)]
    _all(B, B.spec_attention_mass, ok, cases)


def test_evict_refusals(B):
    ok = dict(kv=_view(B), n_seq=2, cache_len_dev=FAKE, mass_dev=2 * FAKE, ld=64, budget=32, recent=8, out_mass_dev=3 * FAKE,
              out_kept_dev=4 * FAKE, out_len_dev=5 * FAKE, err_dev=6 * FAKE)
    cases = [({k: None}, -1) for k in ok if k.endswith("_dev")]
    cases += [(dict(n_seq=0), -1), (dict(n_seq=65536), -1), (dict(budget=0), -1), (dict(recent=-1), -1), (dict(recent=33), -1),
              (dict(ld=0), -1), (dict(ld=1 << 32), -1), (dict(budget=(1 << 30) + 1), -6)]
    # masses: 2 layers x 2 sequences x 2 heads x 64 f32 = 2 KB, kept 1 KB, lengths 8 bytes
    cases += [(dict(out_mass_dev=2 * FAKE + x), -1) for x in (0, 2044, -2044)]
    cases += [(dict(out_kept_dev=2 * FAKE + x), -1) for x in (0, 2044, -1020)]
    cases += [(dict(out_kept_dev=3 * FAKE + x), -1) for x in (0, 2044, -1020)]
    cases += [(dict(out_len_dev=FAKE + x), -1) for x in (0, 4, -4)]
    cases += [(dict(out_len_dev=4 * FAKE), -1), (dict(out_len_dev=(64 << 20) + 16), -1)]
    _all(B, B.spec_kv_evict, ok, cases)
    _refused(B, B.spec_kv_evict, dict(ok, kv=_view(B, n_layers=1 << 13, n_kv_heads=1), n_seq=65535), -6)
