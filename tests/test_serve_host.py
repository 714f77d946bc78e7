"""Argument checks of the serving operators through the C ABI: refused before
anything is launched, so they run without a device."""
import pytest

from dense_tiled_gemm_fp8_amd import gemm355 as g

A = 0x100000000000       # addresses far apart, never dereferenced
STEP = 0x10000000000


def status(call, *a, **k):
    with pytest.raises(g.Gemm355Error) as e:
        call(*a, stream=0, **k)
    return e.value.status


def matrix(**kw):
    a = dict(N=64, K=256, codes=A, scales=A + STEP, zeros=None, fmt=g.W4_INT, group=64, ldw=0)
    a.update(kw)
    return g.make_w4_matrix(**a)


@pytest.mark.parametrize("change,want", [
    (dict(N=-1), g.EINVAL), (dict(K=-1), g.EINVAL), (dict(group=48), g.EINVAL), (dict(group=16), g.EINVAL),
    (dict(fmt=2), g.EINVAL), (dict(fmt=-1), g.EINVAL), (dict(fmt=g.W4_MXFP4), g.EINVAL),
    (dict(fmt=g.W4_MXFP4, group=32, zeros=A + 2 * STEP), g.EINVAL),
    (dict(ldw=224), g.EINVAL), (dict(ldw=257), g.EINVAL), (dict(ldw=272), g.EINVAL),
    (dict(codes=None), g.EINVAL), (dict(scales=None), g.EINVAL),
    (dict(codes=A + 8), g.EALIGN), (dict(scales=A + STEP + 1), g.EALIGN),
    (dict(N=(1 << 30) + 1), g.EUNSUPPORTED), (dict(N=1 << 25, K=1 << 20), g.EUNSUPPORTED),
])
def test_w4_matrix_refused(change, want):
    m = matrix(**change)
    x, y = A + 10 * STEP, A + 200 * STEP
    assert status(g.gemm355_w4_gemm, 1, x, m, y) == want
    assert status(g.gemm355_w4_quantize, x, m) == want
    assert status(g.gemm355_w4_dequantize, m, x) == want


def test_w4_calls_refused():
    m, x, y = matrix(), A + 10 * STEP, A + 20 * STEP
    assert status(g.gemm355_w4_gemm, -1, x, m, y) == g.EINVAL
    assert status(g.gemm355_w4_gemm, 1, None, m, y) == g.EINVAL
    assert status(g.gemm355_w4_gemm, 1, x, m, None) == g.EINVAL
    assert status(g.gemm355_w4_gemm, 1, x, m, y, out=2) == g.EINVAL
    assert status(g.gemm355_w4_gemm, 2, x, m, y, ldx=255) == g.EINVAL
    assert status(g.gemm355_w4_gemm, 2, x, m, y, ldy=63) == g.EINVAL
    assert status(g.gemm355_w4_gemm, 1, x + 1, m, y) == g.EALIGN
    assert status(g.gemm355_w4_gemm, 1, x, m, y + 2, out=g.SRC_F32) == g.EALIGN
    assert status(g.gemm355_w4_gemm, (1 << 19) + 1, x, m, y) == g.EUNSUPPORTED
    # y over x, the codes, the scales, the zero points
    assert status(g.gemm355_w4_gemm, 2, x, m, x + 2 * 256 * 2 - 2) == g.EINVAL
    assert status(g.gemm355_w4_gemm, 1, x, m, A + 64 * 128 - 2) == g.EINVAL
    assert status(g.gemm355_w4_gemm, 1, x, m, A + STEP + 64 * 4 * 2 - 2) == g.EINVAL
    assert status(g.gemm355_w4_gemm, 1, x, matrix(zeros=A + 2 * STEP), A + 2 * STEP + 254) == g.EINVAL
    assert status(g.gemm355_w4_quantize, x, m, src=2) == g.EINVAL
    assert status(g.gemm355_w4_quantize, x, m, ld=255) == g.EINVAL
    assert status(g.gemm355_w4_quantize, None, m) == g.EINVAL
    assert status(g.gemm355_w4_quantize, x + 2, m, src=g.SRC_F32) == g.EALIGN
    assert status(g.gemm355_w4_quantize, A, m) == g.EINVAL
    assert status(g.gemm355_w4_dequantize, m, x, dst=-1) == g.EINVAL
    assert status(g.gemm355_w4_dequantize, m, A + STEP) == g.EINVAL


def test_w4_nothing_to_do():
    """Sizes of zero return before any launch (there may be no device)."""
    x, y = A + 10 * STEP, A + 20 * STEP
    g.gemm355_w4_gemm(0, None, matrix(), None, stream=0)
    g.gemm355_w4_gemm(1, x, matrix(N=0, codes=None, scales=None), y, stream=0)
    for m in (matrix(N=0), matrix(K=0), matrix(N=0, K=0, codes=None, scales=None)):
        g.gemm355_w4_quantize(x, m, stream=0)
        g.gemm355_w4_dequantize(m, x, stream=0)


def cache(**kw):
    a = dict(k=A, v=A + STEP, k_scale=A + 2 * STEP, v_scale=A + 3 * STEP, pages=10, heads=2, head_dim=128, page=64,
             table=A + 4 * STEP, lens=A + 5 * STEP, batch=3, max_len=200, q_start=A + 6 * STEP, tokens=5, max_new=4)
    a.update(kw)
    return g.make_kv_cache(**a)


CACHE_REFUSED = [
    (dict(pages=0), g.EINVAL), (dict(heads=0), g.EINVAL), (dict(batch=-1), g.EINVAL), (dict(tokens=-1), g.EINVAL),
    (dict(max_new=0), g.EINVAL), (dict(max_len=-1), g.EINVAL), (dict(table_ld=-1), g.EINVAL),
    (dict(table_ld=3), g.EINVAL), (dict(q_start=None), g.EINVAL),
    (dict(k=None), g.EINVAL), (dict(v=None), g.EINVAL), (dict(k_scale=None), g.EINVAL), (dict(v_scale=None), g.EINVAL),
    (dict(table=None), g.EINVAL), (dict(lens=None), g.EINVAL),
    (dict(head_dim=96), g.EUNSUPPORTED), (dict(head_dim=512), g.EUNSUPPORTED), (dict(page=8), g.EUNSUPPORTED),
    (dict(page=48), g.EUNSUPPORTED), (dict(page=256), g.EUNSUPPORTED), (dict(batch=70000), g.EUNSUPPORTED),
    (dict(pages=1 << 31), g.EUNSUPPORTED),
    (dict(k=A + 8), g.EALIGN), (dict(v=A + STEP + 4), g.EALIGN), (dict(table=A + 4 * STEP + 2), g.EALIGN),
    (dict(lens=A + 5 * STEP + 1), g.EALIGN), (dict(q_start=A + 6 * STEP + 2), g.EALIGN),
]

X = A + 20 * STEP


def append_args(c=None, **kw):
    a = dict(k=X, v=X + STEP, q=X + 2 * STEP, q_out=X + 3 * STEP, q_heads=4, cos=X + 4 * STEP, sin=X + 5 * STEP,
             rot_dim=128, rot_len=200)
    a.update(kw)
    return g.make_kv_append_args(c if c is not None else cache(), **a)


def attention_args(c=None, **kw):
    a = dict(q=X, o=X + STEP, q_heads=4, lse=X + 2 * STEP)
    a.update(kw)
    return g.make_attention_args(c if c is not None else cache(), **a)


@pytest.mark.parametrize("change,want", CACHE_REFUSED)
def test_cache_refused(change, want):
    assert status(g.gemm355_kv_append, append_args(cache(**change))) == want
    assert status(g.gemm355_attention, attention_args(cache(**change))) == want
    with pytest.raises(g.Gemm355Error) as e:
        g.gemm355_attention_workspace(attention_args(cache(**change)))
    assert e.value.status == want


@pytest.mark.parametrize("change,want", [
    (dict(k=None), g.EINVAL), (dict(v=None), g.EINVAL), (dict(q=None), g.EINVAL), (dict(q_out=None), g.EINVAL),
    (dict(k=X + 8), g.EALIGN), (dict(v=X + STEP + 2), g.EALIGN), (dict(q=X + 2 * STEP + 8), g.EALIGN),
    (dict(q_out=X + 3 * STEP + 8), g.EALIGN), (dict(cos=X + 4 * STEP + 2), g.EALIGN),
    (dict(ldk=255), g.EINVAL), (dict(ldk=257), g.EINVAL), (dict(ldv=248), g.EINVAL), (dict(ldq=504), g.EINVAL),
    (dict(ldqo=513), g.EINVAL), (dict(q_heads=0), g.EINVAL),
    (dict(rot_dim=-2), g.EINVAL), (dict(rot_dim=130), g.EINVAL), (dict(rot_dim=7), g.EINVAL),
    (dict(rot_len=199), g.EINVAL), (dict(cos=None), g.EINVAL), (dict(sin=None), g.EINVAL),
    (dict(q_out=X), g.EINVAL), (dict(q_out=X + 2 * STEP + 5 * 512 * 2 - 16), g.EINVAL), (dict(q_out=X + 4 * STEP), g.EINVAL),
    (dict(q_out=A), g.EINVAL), (dict(k=A + STEP), g.EINVAL), (dict(v=A), g.EINVAL), (dict(cos=A), g.EINVAL),
    (dict(q_out=A + 4 * STEP), g.EINVAL),
])
def test_append_refused(change, want):
    assert status(g.gemm355_kv_append, append_args(**change)) == want


@pytest.mark.parametrize("change,want", [
    (dict(q=None), g.EINVAL), (dict(o=None), g.EINVAL), (dict(q=X + 8), g.EALIGN), (dict(o=X + STEP + 8), g.EALIGN),
    (dict(lse=X + 2 * STEP + 2), g.EALIGN), (dict(q_heads=3), g.EINVAL), (dict(q_heads=0), g.EINVAL),
    (dict(ldq=511), g.EINVAL), (dict(ldo=516), g.EINVAL), (dict(window=-1), g.EINVAL), (dict(sinks=-1), g.EINVAL),
    (dict(splits=-1), g.EINVAL), (dict(scale=-1.0), g.EINVAL), (dict(scale=float("nan")), g.EINVAL),
    (dict(scale=float("inf")), g.EINVAL), (dict(o=X + 5 * 512 * 2 - 16), g.EINVAL), (dict(o=A), g.EINVAL),
    (dict(lse=X), g.EINVAL), (dict(lse=X + STEP), g.EINVAL), (dict(lse=A + 5 * STEP), g.EINVAL),
    (dict(workspace=0x7000000000, workspace_bytes=16, splits=4), g.ENOMEM),
    (dict(workspace=0x7000000010, workspace_bytes=1 << 30, splits=4), g.EALIGN),
])
def test_attention_refused(change, want):
    c = cache(max_len=4000) if "workspace" in change else None
    assert status(g.gemm355_attention, attention_args(c, **change)) == want


def test_attention_workspace_sizes():
    one = g.gemm355_attention_workspace(attention_args(cache(max_len=4000), splits=1))
    four = g.gemm355_attention_workspace(attention_args(cache(max_len=4000), splits=4))
    # parts of 16 rows: batch 3, 2 heads, 4 new tokens of 2 query heads each
    assert one == 0 and four == 3 * 2 * 1 * 4 * 16 * (128 + 2) * 4
    # a part is never under 256 tokens, nor outside what a window can see
    assert g.gemm355_attention_workspace(attention_args(cache(max_len=4000), splits=1000)) == four // 4 * 16
    assert g.gemm355_attention_workspace(attention_args(cache(max_len=200), splits=1000)) == 0
    assert g.gemm355_attention_workspace(attention_args(cache(max_len=4000), splits=1000, window=64)) == 0
    with pytest.raises(g.Gemm355Error) as e:
        g._check(g._lib.gemm355_attention_workspace(None, None), "x")
    assert e.value.status == g.EINVAL


def test_null_argument_structs():
    import ctypes
    size = ctypes.c_size_t()
    assert g._lib.gemm355_attention(None, None) == g.EINVAL
    assert g._lib.gemm355_attention_workspace(None, ctypes.byref(size)) == g.EINVAL
    assert g._lib.gemm355_kv_append(None, None) == g.EINVAL
    assert g._lib.gemm355_w4_gemm(1, None, 0, None, None, 0, 0, None) == g.EINVAL
    assert g._lib.gemm355_w4_quantize(None, 0, 0, None, None) == g.EINVAL
    assert g._lib.gemm355_w4_dequantize(None, None, 0, 0, None) == g.EINVAL


def test_empty_steps_do_nothing():
    g.gemm355_kv_append(append_args(cache(tokens=0), k=None, v=None, q=None, q_out=None), stream=0)
    g.gemm355_attention(attention_args(cache(tokens=0), q=None, o=None, lse=None), stream=0)
    empty = cache(batch=0, tokens=0, table=None, lens=None, q_start=None)
    g.gemm355_kv_append(append_args(empty), stream=0)
    g.gemm355_attention(attention_args(empty), stream=0)


def test_w4_quantize_outputs_that_overlap_are_refused():
    x = A + 10 * STEP
    assert status(g.gemm355_w4_quantize, x, matrix(scales=A + 64 * 128 - 2)) == g.EINVAL
    assert status(g.gemm355_w4_quantize, x, matrix(zeros=A + 16)) == g.EINVAL
    assert status(g.gemm355_w4_quantize, x, matrix(zeros=A + STEP + 64 * 4 * 2 - 1)) == g.EINVAL


def test_attention_workspace_over_other_buffers_is_refused():
    for at in (X - 256, X + STEP, X + 2 * STEP, A, A + STEP, A + 4 * STEP, A + 6 * STEP):
        c = cache(max_len=4000)
        assert status(g.gemm355_attention, attention_args(c, workspace=at, workspace_bytes=1 << 30, splits=4)) == g.EINVAL


def test_attention_scratch_past_64_bits_is_refused():
    c = cache(batch=8000, heads=8, max_len=1 << 30, table=1 << 12, table_ld=1 << 23, page=128, tokens=1 << 16, max_new=1 << 12,
              lens=1 << 20, k=A, v=2 * A, pages=10)
    a = attention_args(c, q_heads=8, q=4 * A, o=5 * A, lse=None, splits=1 << 30)
    assert status(g.gemm355_attention, a) == g.EUNSUPPORTED
    with pytest.raises(g.Gemm355Error) as e:
        g.gemm355_attention_workspace(a)
    assert e.value.status == g.EUNSUPPORTED
