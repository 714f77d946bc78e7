"""Argument checks of the serving operators at the ends of their ranges, through
the C ABI without a device."""
from dense_tiled_gemm_fp8_amd import gemm355 as g
from tests.test_serve_host import X, append_args, attention_args, cache, matrix, status


def test_attention_scales_whose_binary_logarithm_form_overflows_are_refused():
    """The kernel holds scale * log2(e) in fp32: an infinity from 2.36e38 on,
    and 0 times it, a score of zero, a NaN."""
    for scale in (1.7e38, 2.0 ** 127):
        assert g.gemm355_attention_workspace(attention_args(scale=scale)) == 0
    for scale in (2.0 ** 127 * (1 + 2.0 ** -23), 2.4e38, 2.9e38, 3.0e38, 3.4e38):
        assert status(g.gemm355_attention, attention_args(scale=scale)) == g.EINVAL


def test_columns_of_one_buffer_are_told_from_overlapping_rows():
    """Rows of 512 elements in a buffer of 1536: outputs may take the columns
    that no input has, from before or behind it, and no others."""
    wide = dict(ldq=1536, ldo=1536)
    for columns in (512, 1024, 1536 + 512, -512, -1024):
        assert g.gemm355_attention_workspace(attention_args(o=X + 2 * columns, **wide)) == 0
    for columns in (0, 504, 1032, 1536, 1536 + 8, -8, -504, -1032):
        assert status(g.gemm355_attention, attention_args(o=X + 2 * columns, **wide)) == g.EINVAL
        assert status(g.gemm355_kv_append, append_args(q=X, k=X + (1 << 40), q_out=X + 2 * columns, ldq=1536, ldqo=1536)) == g.EINVAL
    # another pitch: rows meet somewhere, or may
    assert status(g.gemm355_attention, attention_args(o=X + 1024, ldq=1536, ldo=1544)) == g.EINVAL
    # rows of 256 elements beside rows of 64: y of 16 bits from column 200 on
    for columns in (200, 248, 328, -56):
        assert status(g.gemm355_w4_gemm, 3, X, matrix(), X + 2 * columns, ldx=384, ldy=384) == g.EINVAL


def test_limits_of_the_header():
    """Both sides of the limits on sizes, by the scratch query where they are
    allowed (which launches nothing)."""
    def tokens(batch, heads, new, **kw):
        return cache(batch=batch, heads=heads, tokens=batch * new, max_new=new, **kw)

    def taken(c, **kw):
        g.gemm355_attention_workspace(attention_args(c, **kw))

    def refused(c, **kw):
        assert status(g.gemm355_attention, attention_args(c, **kw)) == g.EUNSUPPORTED
    far = dict(o=X + (1 << 43), lse=None)
    taken(tokens(8191, 8, 1), q_heads=8, **far)
    refused(tokens(8192, 8, 1), q_heads=8, **far)
    taken(tokens(1, 1, 16 * 65535), q_heads=1, **far)
    refused(tokens(1, 1, 16 * 65535 + 1), q_heads=1, **far)
    refused(tokens(1, 1, 131072), q_heads=8, **far)
    for change in (dict(max_len=(1 << 30) + 1, table_ld=1 << 30), dict(table_ld=(1 << 30) + 1), dict(pages=1 << 31)):
        refused(cache(**change))
        assert status(g.gemm355_kv_append, append_args(cache(**change), rot_len=1 << 31)) == g.EUNSUPPORTED
    refused(cache(), ldq=(1 << 30) + 8)
    # 2 * 8192 workgroups a page, 1024 pages of 64 tokens
    wide = dict(heads=8192, batch=1, tokens=1 << 20, max_len=1 << 20)
    a = append_args(cache(max_new=(1 << 16) - 1, **wide), q=None, q_out=None, rot_dim=0, v=X + (1 << 44))
    assert status(g.gemm355_kv_append, a) == g.EUNSUPPORTED
