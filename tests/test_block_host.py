"""Argument checks of the block-scaled operators through the C ABI: refused before
anything is launched, so they run without a device."""
import math

import pytest

from dense_tiled_gemm_fp8_amd import gemm355 as g
from tests.test_serve_host import A, STEP, status

X, OUT = A + 100 * STEP, A + 200 * STEP


def matrix(at=A, **kw):
    a = dict(rows=300, K=500, codes=at, scales=at + STEP, block_rows=1)
    a.update(kw)
    return g.make_block_matrix(**a)


def weights(at=A + 10 * STEP, **kw):
    a = dict(rows=400, block_rows=128)
    a.update(kw)
    return matrix(at, **a)


def gemm(x=None, w=None, y=OUT, **kw):
    return g.make_block_gemm_args(x or matrix(), w or weights(), y=y, **kw)


def gated(x=None, gate=None, up=None, y=OUT, **kw):
    return g.make_block_gated_args(x or matrix(), gate or weights(), up or weights(A + 20 * STEP), y=y, **kw)


def codes_out(**kw):
    a = dict(rows=300, K=400, codes=OUT, scales=OUT + STEP)
    a.update(kw)
    return g.make_block_matrix(**a)


def norm(**kw):
    a = dict(rows=30, width=256, x=X, residual=X + STEP, sum=X + 2 * STEP, weight=X + 3 * STEP, y=X + 4 * STEP,
             q=codes_out(rows=30, K=256))
    a.update(kw)
    return g.make_rmsnorm_args(**a)


MATRIX = [
    (dict(rows=-1), g.EINVAL), (dict(K=-1), g.EINVAL), (dict(block_rows=0), g.EINVAL), (dict(block_rows=2), g.EINVAL),
    (dict(block_rows=64), g.EINVAL), (dict(block_rows=-128), g.EINVAL),
    (dict(ld=496), g.EINVAL), (dict(ld=500), g.EINVAL), (dict(ld=520), g.EINVAL), (dict(ld=-512), g.EINVAL),
    (dict(codes=None), g.EINVAL), (dict(scales=None), g.EINVAL),
    (dict(codes=A + 8), g.EALIGN), (dict(scales=A + STEP + 2), g.EALIGN),
    (dict(rows=(1 << 26) + 1), g.EUNSUPPORTED), (dict(K=(1 << 22) + 1), g.EUNSUPPORTED),
    (dict(ld=(1 << 22) + 16), g.EUNSUPPORTED), (dict(ld_scale=(1 << 30) + 1), g.EUNSUPPORTED),
]


@pytest.mark.parametrize("change,want", MATRIX)
def test_matrix_refused(change, want):
    m = matrix(**change)
    assert status(g.gemm355_block_quantize, X, m) == want
    assert status(g.gemm355_block_gemm, gemm(x=m)) == want
    assert status(g.gemm355_block_gated, gated(x=m)) == want
    wide = {**dict(block_rows=128), **change}
    assert status(g.gemm355_block_gemm, gemm(w=weights(**wide))) == want
    assert status(g.gemm355_block_gated, gated(gate=weights(**wide))) == want
    assert status(g.gemm355_block_gated, gated(up=weights(**wide))) == want
    with pytest.raises(g.Gemm355Error) as e:
        g.gemm355_block_gemm_workspace(gemm(x=m))
    assert e.value.status == want
    with pytest.raises(g.Gemm355Error) as e:
        g.gemm355_block_gated_workspace(gated(x=m))
    assert e.value.status == want


def test_scale_pitch():
    """At least the rows, or at least the K blocks."""
    assert status(g.gemm355_block_quantize, X, matrix(ld_scale=299)) == g.EINVAL
    assert status(g.gemm355_block_quantize, X, matrix(ld_scale=-1)) == g.EINVAL
    assert status(g.gemm355_block_quantize, X, matrix(block_rows=128, ld_scale=3)) == g.EINVAL
    assert g.gemm355_block_gemm_workspace(gemm(x=matrix(ld_scale=300), w=weights(ld_scale=4))) >= 0


def test_quantize_refused():
    m = matrix()
    assert status(g.gemm355_block_quantize, None, m) == g.EINVAL
    assert status(g.gemm355_block_quantize, X, m, src=2) == g.EINVAL
    assert status(g.gemm355_block_quantize, X, m, src=-1) == g.EINVAL
    assert status(g.gemm355_block_quantize, X, m, ld=499) == g.EINVAL
    assert status(g.gemm355_block_quantize, X + 1, m) == g.EALIGN
    assert status(g.gemm355_block_quantize, X + 2, m, src=g.SRC_F32) == g.EALIGN
    assert status(g.gemm355_block_quantize, X, m, ld=(1 << 30) + 1) == g.EUNSUPPORTED
    # over the codes, over the scales, codes over scales
    assert status(g.gemm355_block_quantize, A + 300 * 512 - 14, m) == g.EINVAL
    assert status(g.gemm355_block_quantize, A + STEP + 4 * 300 * 4 - 2, m) == g.EINVAL
    assert status(g.gemm355_block_quantize, X, matrix(scales=A + 299 * 512 + 508)) == g.EINVAL
    # workgroups: 2^26 / 16 rows of 4 blocks each, 2^26 / 128 of 32
    assert status(g.gemm355_block_quantize, X, matrix(rows=1 << 26, scales=A + (1 << 36))) == g.EUNSUPPORTED
    assert status(g.gemm355_block_quantize, X, matrix(rows=1 << 26, K=4096, scales=A + (1 << 39), block_rows=128)) == g.EUNSUPPORTED


@pytest.mark.parametrize("change,want", [
    (dict(rows=-1), g.EINVAL), (dict(width=-1), g.EINVAL), (dict(x=None), g.EINVAL), (dict(residual=None), g.EINVAL),
    (dict(y=None, q=None), g.EINVAL), (dict(eps=0.0), g.EINVAL), (dict(eps=-1e-5), g.EINVAL), (dict(eps=math.nan), g.EINVAL),
    (dict(eps=math.inf), g.EINVAL), (dict(x_type=2), g.EINVAL), (dict(r_type=-1), g.EINVAL), (dict(w_type=3), g.EINVAL),
    (dict(y_type=2), g.EINVAL), (dict(ldx=255), g.EINVAL), (dict(ldr=255), g.EINVAL), (dict(lds=255), g.EINVAL),
    (dict(ldy=255), g.EINVAL), (dict(x=X + 1), g.EALIGN), (dict(x=X + 2, x_type=g.SRC_F32), g.EALIGN),
    (dict(residual=X + STEP + 1), g.EALIGN), (dict(sum=X + 2 * STEP + 2, r_type=g.SRC_F32), g.EALIGN),
    (dict(weight=X + 3 * STEP + 1), g.EALIGN), (dict(weight=X + 3 * STEP + 2, w_type=g.SRC_F32), g.EALIGN),
    (dict(y=X + 4 * STEP + 1), g.EALIGN), (dict(rows=(1 << 22) + 1), g.EUNSUPPORTED), (dict(width=(1 << 15) + 1), g.EUNSUPPORTED),
    (dict(ldx=(1 << 30) + 1), g.EUNSUPPORTED), (dict(ldy=(1 << 30) + 1), g.EUNSUPPORTED),
    # q of other sizes, of blocks of 128 rows, without codes
    (dict(q=codes_out(rows=29, K=256)), g.EINVAL), (dict(q=codes_out(rows=30, K=255)), g.EINVAL),
    (dict(q=codes_out(rows=30, K=256, block_rows=128)), g.EINVAL), (dict(q=codes_out(rows=30, K=256, codes=None)), g.EINVAL),
    # outputs over inputs by less than whole rows, over each other, over the weight
    (dict(sum=X + 512), g.EINVAL), (dict(y=X + 2), g.EINVAL), (dict(y=X + STEP, ldy=512), g.EINVAL),
    (dict(y=X, y_type=g.SRC_F32), g.EINVAL), (dict(y=X + 2 * STEP), g.EINVAL), (dict(sum=X + 3 * STEP), g.EINVAL),
    (dict(y=X + 3 * STEP + 510), g.EINVAL), (dict(sum=X + STEP, y=X + STEP), g.EINVAL),
    (dict(q=codes_out(rows=30, K=256, codes=X)), g.EINVAL), (dict(q=codes_out(rows=30, K=256, scales=X + STEP)), g.EINVAL),
    (dict(q=codes_out(rows=30, K=256, codes=X + 2 * STEP)), g.EINVAL), (dict(q=codes_out(rows=30, K=256, scales=X + 4 * STEP)), g.EINVAL),
    (dict(q=codes_out(rows=30, K=256, codes=X + 3 * STEP)), g.EINVAL), (dict(q=codes_out(rows=30, K=256, scales=OUT + 30 * 256 - 4)), g.EINVAL),
])
def test_norm_refused(change, want):
    assert status(g.gemm355_rmsnorm, norm(**change)) == want


def test_norm_rows_whose_threads_reach_32_bits():
    # 2^22 rows of 1024 threads are one more than a launch counts
    assert status(g.gemm355_rmsnorm, norm(rows=1 << 22, width=8192)) == g.EUNSUPPORTED


def test_nothing_to_do():
    """Sizes of zero return before any launch (there may be no device)."""
    for m in (matrix(rows=0), matrix(K=0), matrix(rows=0, K=0, codes=None, scales=None)):
        g.gemm355_block_quantize(X, m, stream=0)
    g.gemm355_rmsnorm(norm(rows=0, q=codes_out(rows=0, K=256)), stream=0)
    g.gemm355_rmsnorm(norm(width=0, q=None, x=None, y=None, residual=None, sum=None, weight=None), stream=0)
    for x, w in ((matrix(rows=0), weights()), (matrix(), weights(rows=0))):
        g.gemm355_block_gemm(gemm(x=x, w=w, y=None), stream=0)
        g.gemm355_block_gated(gated(x=x, gate=w, up=w, y=None), stream=0)
        assert g.gemm355_block_gemm_workspace(gemm(x=x, w=w)) == 0


def test_products_refused():
    for args in (dict(y=None), dict(out=2), dict(splits=-1), dict(ldy=399), dict(x=matrix(K=499)), dict(x=matrix(block_rows=128)),
                 dict(w=weights(block_rows=1))):
        assert status(g.gemm355_block_gemm, gemm(**args)) == g.EINVAL
    assert status(g.gemm355_block_gemm, gemm(y=OUT + 1)) == g.EALIGN
    assert status(g.gemm355_block_gemm, gemm(y=OUT + 2, out=g.SRC_F32)) == g.EALIGN
    assert status(g.gemm355_block_gemm, gemm(ldy=(1 << 30) + 1)) == g.EUNSUPPORTED
    assert status(g.gemm355_block_gemm, gemm(x=matrix(rows=(1 << 21) + 1, scales=A + (1 << 36)))) == g.EUNSUPPORTED
    # y over the codes and scales of either matrix
    for at in (A + 300 * 512 - 2, A + STEP + 4 * 300 * 4 - 2, A + 10 * STEP, A + 11 * STEP + 4 * 4 * 4 - 2):
        assert status(g.gemm355_block_gemm, gemm(y=at)) == g.EINVAL
    for args in (dict(y=None), dict(q=codes_out()), dict(act=2), dict(act=-1), dict(out=2), dict(splits=-1), dict(ldy=399),
                 dict(x=matrix(K=499)), dict(gate=weights(K=499)), dict(up=weights(K=499)), dict(up=weights(rows=399)),
                 dict(up=weights(block_rows=1)), dict(gate=weights(block_rows=1)),
                 dict(y=None, q=codes_out(rows=299)), dict(y=None, q=codes_out(K=399)), dict(y=None, q=codes_out(block_rows=128)),
                 dict(y=None, q=codes_out(scales=None)), dict(y=None, q=codes_out(codes=A)),
                 dict(y=None, q=codes_out(scales=A + 21 * STEP)), dict(y=None, q=codes_out(scales=OUT + 300 * 400 - 4)),
                 dict(y=A + 20 * STEP + 4)):
        assert status(g.gemm355_block_gated, gated(**args)) == g.EINVAL, args
        if "act" in args:
            with pytest.raises(g.Gemm355Error):
                g.gemm355_block_gated_workspace(gated(**args))
    assert status(g.gemm355_block_gated, gated(y=None, q=codes_out(codes=OUT + 8))) == g.EALIGN


def test_workspaces_refused():
    """Too small, not aligned, over an input or the output."""
    for make, call, need in ((gemm, g.gemm355_block_gemm, g.gemm355_block_gemm_workspace),
                             (gated, g.gemm355_block_gated, g.gemm355_block_gated_workspace)):
        n = need(make(splits=3))
        assert n > 0 and n % 4 == 0
        far = A + 300 * STEP
        assert status(call, make(splits=3, workspace=far, workspace_bytes=n - 1)) == g.ENOMEM
        assert status(call, make(splits=3, workspace=far + 128, workspace_bytes=n)) == g.EALIGN
        for at in (A, A + STEP, A + 10 * STEP, A + 11 * STEP, OUT):
            assert status(call, make(splits=3, workspace=at, workspace_bytes=n)) == g.EINVAL
    n = g.gemm355_block_gated_workspace(gated(y=None, q=codes_out(), splits=3))
    for at in (OUT, OUT + STEP, A + 20 * STEP):
        assert status(g.gemm355_block_gated, gated(y=None, q=codes_out(), splits=3, workspace=at, workspace_bytes=n)) == g.EINVAL


def test_scratch_limit():
    old = g.gemm355_set_scratch_limit(0)
    try:
        assert status(g.gemm355_block_gemm, gemm(splits=4)) in (g.ENOMEM, g.EHIP)    # EHIP: no device to ask
    finally:
        g.gemm355_set_scratch_limit(old)


def test_limits_of_the_header():
    """Both sides of the limits, by the scratch query where they are allowed."""
    far = A + (1 << 45)
    wide = dict(K=1 << 22, ld=1 << 22)
    w = g.make_block_matrix(128, 1 << 22, A + (1 << 46), A + (1 << 47), block_rows=128)
    assert g.gemm355_block_gemm_workspace(g.make_block_gemm_args(matrix(**wide), w, y=far)) >= 0
    tall = matrix(rows=1 << 21, K=128, scales=A + (1 << 42))
    small = g.make_block_matrix(64, 128, A + (1 << 46), A + (1 << 47), block_rows=128)
    assert g.gemm355_block_gemm_workspace(g.make_block_gemm_args(tall, small, y=far)) == 0
    # 2^21 rows by 2^26 columns: more workgroups than a launch has
    many = g.make_block_matrix(1 << 26, 128, A + (1 << 46), A + (1 << 47), block_rows=128)
    with pytest.raises(g.Gemm355Error) as e:
        g.gemm355_block_gemm_workspace(g.make_block_gemm_args(tall, many, y=A + (1 << 52)))
    assert e.value.status == g.EUNSUPPORTED
    # parts of more than 2^40 bytes
    some = g.make_block_matrix(1 << 17, 4096, A + (1 << 46), A + (1 << 47), block_rows=128)
    x = matrix(rows=1 << 17, K=4096, scales=A + (1 << 42))
    assert g.gemm355_block_gemm_workspace(g.make_block_gemm_args(x, some, y=A + (1 << 52), splits=16)) == 1 << 40
    with pytest.raises(g.Gemm355Error) as e:
        g.gemm355_block_gemm_workspace(g.make_block_gemm_args(x, some, y=A + (1 << 52), splits=17))
    assert e.value.status == g.EUNSUPPORTED


def test_kernels_hold_their_sums_in_registers():
    """Matrix instructions of both kinds, no spills, no accumulation registers (the
    sums go through vector instructions) in any product kernel; no spills in the
    norm's."""
    import re
    from dense_tiled_gemm_fp8_amd import build
    for src, least in (("block.hip", 39), ("norm.hip", 8)):
        bodies = [b for b in re.split(r"\n(?=_ZN4g355\w+:)", open(build.device_asm(src)).read()) if b.startswith("_ZN4g355")]
        assert len(bodies) >= least
        for b in bodies:
            name = b.split(":")[0]
            assert re.search(r"; ScratchSize: 0\b", b), name
            if "finish" in name or src == "norm.hip":
                continue
            assert re.search(r"; NumAgprs: 0\b", b), name
            exact = name.split("EEEv")[0].endswith("1")
            assert ("v_mfma_f32_" in b) and (("_bf16 " in b) if exact else ("f8f6f4" in b)), name


def test_struct_layout_matches_header(tmp_path):
    """ctypes' view of the structures against a C program's."""
    import ctypes
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    classes = (g.gemm355_block_matrix, g.gemm355_rmsnorm_args, g.gemm355_block_gemm_args, g.gemm355_block_gated_args)
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "gemm355.h"', "int main(void) {"]
    for c in classes:
        lines.append('printf("%%zu\\n", sizeof(%s));' % c.__name__)
        lines += ['printf("%%zu\\n", offsetof(%s, %s));' % (c.__name__, f) for f, _ in c._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0; }"]))
    subprocess.check_call(["gcc", "-std=c99", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)])
    got = [int(v) for v in subprocess.check_output([str(exe)]).split()]
    assert got == [v for c in classes for v in [ctypes.sizeof(c)] + [getattr(c, f).offset for f, _ in c._fields_]]
