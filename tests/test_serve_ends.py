"""Argument checks of the serving operators at the ends of their ranges, through
the C ABI without a device."""
from dense_tiled_gemm_fp8_amd import gemm355 as g
from tests.test_serve_host import attention_args, status


def test_attention_scales_whose_binary_logarithm_form_overflows_are_refused():
    """The kernel holds scale * log2(e) in fp32: an infinity from 2.36e38 on,
    and 0 times it, a score of zero, a NaN."""
    for scale in (1.7e38, 2.0 ** 127):
        assert g.gemm355_attention_workspace(attention_args(scale=scale)) == 0
    for scale in (2.0 ** 127 * (1 + 2.0 ** -23), 2.4e38, 2.9e38, 3.0e38, 3.4e38):
        assert status(g.gemm355_attention, attention_args(scale=scale)) == g.EINVAL
