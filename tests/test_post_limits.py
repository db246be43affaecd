"""Sizes that the post-training entry points refuse on the host, and views that they take."""
import pytest

from top_kl_distill_gb300 import vloss as vl

P = 1 << 20          # never dereferenced


def _refused(fn, *a):
    with pytest.raises(vl.VlossError) as e:
        fn(*a)
    assert fn.__name__ in str(e.value)
    return e.value.status


@pytest.mark.parametrize("K", [(1 << 30) + 1, (1 << 31) - 128, (1 << 31) - 127, (1 << 31) - 1, 1 << 31, 1 << 40])
def test_quantisers_refuse_rows_past_their_indices(K):
    """The product takes K up to 2^30; the quantisers count columns with 32-bit ints."""
    for fn in (vl.vl_quant_fp8_rows, vl.vl_quant_fp8_rows_bf16):
        assert _refused(fn, P, K, 1, K, P, P, 0) == vl.VL_EINVAL
    assert _refused(vl.vl_quant_fp8_blocks_bf16, P, 1, K, P, P, 0) == vl.VL_EINVAL
