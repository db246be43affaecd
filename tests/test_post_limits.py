"""Sizes that the post-training entry points refuse on the host, and views that they take."""
import pytest

from top_kl_distill_gb300 import vloss as vl

P = 1 << 20          # never dereferenced


def _refused(fn, *a, **k):
    with pytest.raises(vl.VlossError) as e:
        fn(*a, **k)
    assert fn.__name__ in str(e.value)
    return e.value.status


@pytest.mark.parametrize("K", [(1 << 30) + 1, (1 << 31) - 128, (1 << 31) - 127, (1 << 31) - 1, 1 << 31, 1 << 40])
def test_quantisers_refuse_rows_past_their_indices(K):
    """The product takes K up to 2^30; the quantisers count columns with 32-bit ints."""
    for fn in (vl.vl_quant_fp8_rows, vl.vl_quant_fp8_rows_bf16):
        assert _refused(fn, P, K, 1, K, P, P, 0) == vl.VL_EINVAL
    assert _refused(vl.vl_quant_fp8_blocks_bf16, P, 1, K, P, P, 0) == vl.VL_EINVAL


def test_rows_that_meet_are_refused():
    """Matrices of one stride that lie between one another's rows may not touch: 8 rows of 24 floats in a
    stride of 48 (192 bytes), the other matrix some bytes further or nearer."""
    for d in (4, 92, 100, 188, -4, -92, -100, -188, 192 + 4, 192 * 7 + 92, -192 * 3 + 100):
        for x, y in ((P, P + d), (P + d, P)):
            assert _refused(vl.vl_layernorm_fwd, x, 48, 8, 24, None, None, 1e-5, y, 48, None, None, 0) == vl.VL_EINVAL
            assert _refused(vl.vl_policy_loss, x, 48, 8, 24, P, P, None, P, P, 0.2, 0.2, 0.0, 1.0, y, 48, P, None, None, None, None,
                            0) == vl.VL_EINVAL
    # of different strides, and of one row
    assert _refused(vl.vl_layernorm_fwd, P, 48, 8, 24, None, None, 1e-5, P + 96, 50, None, None, 0) == vl.VL_EINVAL
    assert _refused(vl.vl_layernorm_fwd, P, 48, 1, 24, None, None, 1e-5, P + 92, 48, None, None, 0) == vl.VL_EINVAL
    # rows of 48 bytes (a bf16 dx) beside rows of 96 (an fp32 dy) in the same 192
    for d in (4, 94, 146, 190):
        assert _refused(vl.vl_layernorm_bwd_bf16, P, 48, P + (1 << 30), 96, 8, 24, None, P, P, P + d, 96, None, None, None, 0,
                        dy_f32=True) == vl.VL_EINVAL
