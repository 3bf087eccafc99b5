"""Refusals of the tree entry points on the host, before any CUDA call (the
pointers here are never dereferenced)."""
import pytest


@pytest.fixture(scope="module")
def B():
    from lossless_speculative_decoding_gb300 import build, binding
    build.build()
    return binding


def _view(B):
    return B.make_kv_view(1 << 20, 2 << 20, dtype=1, n_pages=8, n_layers=2, n_kv_heads=2, page_size=16, head_dim=128, max_pages=4)


@pytest.mark.parametrize("scale", [3.4e38, 2.4e38])      # log2 e times 2.4e38 is 3.46e38
def test_attention_scales_past_fp32_in_units_of_log2(B, scale):
    """Finite, but not once multiplied by log2 e."""
    with pytest.raises(B.SpecError) as e:
        B.spec_tree_attention(_view(B), 0, 3 << 20, 2, 64, 4, 4 << 20, 5 << 20, 6 << 20, scale, 7 << 20, 8 << 20, 1 << 40,
                              9 << 20)
    assert e.value.code == -1 and "scale" in str(e.value)


OUTS = dict(out_accepted_dev=2, out_token_dev=2, out_path_dev=128, out_len_dev=2)
INS = dict(tokens_dev=128, parents_dev=128, target_dev=128, n_nodes_dev=2, cache_len_dev=2)


@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("other", [*INS, *OUTS])
def test_commit_outputs_that_overlap(B, out, other):
    """The same array, an output's last element on another's first, and the other way round."""
    if out == other:
        return
    size = {**OUTS, **INS}
    base = {k: (16 + i) << 20 for i, k in enumerate(size)}
    for at in (base[other], base[other] - 4 * (size[out] - 1), base[other] + 4 * (size[other] - 1)):
        with pytest.raises(B.SpecError) as e:
            B.spec_tree_commit(kv=_view(B), n_seq=2, max_nodes=64, err_dev=9 << 20, **{**base, out: at})
        assert e.value.code == -1 and "overlap" in str(e.value)
