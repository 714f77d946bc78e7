"""GPU parity of the 4-bit quantiser, dequantiser and product with the oracle
(oracle/w4.py).

Products, |y - ref| <= c * A + half a step of the output type, from the order
of the sums: a group's sum has at most 128 terms, a wavefront adds at most
ceil(K / 128) * (128 / group) group sums, and at most 8 wavefronts are joined.  Each of
those n = min(K, 128) + ng + 8 additions is off by at most 2^-23 (an adder that
truncates) of sums whose magnitude is at most A = sum |x| s (u + z), taken here
as sum |x| s (32 + u + z): the codes enter as u, and z sum x is taken off, which
is one more sum of the same length.  MXFP4 has A = sum |x w| alone.  Products of small whole numbers and
power-of-two scales are exact in every step and compared bit for bit.
"""
import numpy as np
import pytest
import torch

from dense_tiled_gemm_fp8_amd import gemm355 as g
from oracle import w4
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu


def dev(a):
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.copy()).cuda()


def matrix(codes, scales, zeros, fmt, group, ldw=0, fill=0):
    """Device buffers and descriptor; bytes behind K hold `fill`."""
    N, K = codes.shape
    width = ldw or -(-K // 32) * 32
    packed = w4.pack(codes, width)
    behind = w4.pack(np.full((N, width), fill, np.uint8), width)
    packed[:, (K + 1) // 2:] = behind[:, (K + 1) // 2:]
    if K % 2:
        packed[:, K // 2] |= behind[:, K // 2] & 0xF0
    c = dev(packed)
    s = dev(scales) if fmt == "mxfp4" else dev(scales).to(torch.bfloat16)
    z = None if zeros is None else dev(zeros)
    m = g.make_w4_matrix(N, K, c, s, z, fmt=g.W4_MXFP4 if fmt == "mxfp4" else g.W4_INT, group=group, ldw=ldw)
    return m, (c, s, z)


def random_matrix(rng, N, K, fmt, group, zeros):
    ng = -(-K // group)
    codes = rng.integers(0, 16, (N, K)).astype(np.uint8)
    if fmt == "mxfp4":
        return codes, rng.integers(115, 135, (N, ng)).astype(np.uint8), None
    scales = w4.bf16((0.01 * np.exp(rng.standard_normal((N, ng)))).astype(np.float32))
    return codes, scales, rng.integers(0, 16, (N, ng)).astype(np.uint8) if zeros else None


def product(M, xt, m, N, out, ldx=0, ldy=0, fill=7.0):
    y = torch.full((M, ldy or N), fill, dtype=torch.bfloat16 if out == "bf16" else torch.float32, device="cuda")
    g.gemm355_w4_gemm(M, xt, m, y, out=g.SRC_BF16 if out == "bf16" else g.SRC_F32, ldx=ldx, ldy=ldy)
    torch.cuda.synchronize()
    return y


def check(y, x, codes, scales, zeros, fmt, group, out):
    K = codes.shape[1]
    W = w4.values(codes, scales, zeros, fmt, group)
    ref = x @ W.T
    if fmt == "mxfp4":
        A = np.abs(x) @ np.abs(W).T
    else:
        z = np.repeat(zeros, group, 1)[:, :K].astype(float) if zeros is not None else 8.0
        A = np.abs(x) @ (np.repeat(scales, group, 1)[:, :K].astype(float) * (32.0 + codes + z)).T
    n = min(K, 128) + -(-K // group) + 8
    tol = n * 2.0 ** -23 * A + (2.0 ** -8 if out == "bf16" else 2.0 ** -24) * np.abs(ref)
    err = np.abs(y.double().cpu().numpy() - ref)
    assert np.all(err <= tol), "%d outside, worst %.3g of the tolerance" % (int((err > tol).sum()), float((err / tol).max()))


FORMS = [("int", 32, False), ("int", 32, True), ("int", 64, False), ("int", 64, True), ("int", 128, False), ("int", 128, True),
         ("mxfp4", 32, False)]
SHAPES = [(1, 1, 1), (1, 16, 128), (1, 1024, 1024), (2, 17, 33), (3, 250, 776), (4, 64, 4096), (5, 300, 777), (8, 96, 640),
          (13, 1000, 200), (16, 48, 2048), (17, 130, 515), (31, 64, 96), (33, 200, 1000), (64, 128, 512), (65, 40, 384),
          (130, 33, 31), (1, 4099, 260)]


@pytest.mark.parametrize("fmt,group,zeros", FORMS)
def test_w4_gemm_random(fmt, group, zeros):
    rng = np.random.default_rng(group + 10 * zeros + (1000 if fmt == "mxfp4" else 0))
    for M, N, K in SHAPES:
        for out in ("f32", "bf16"):
            say("w4_gemm", fmt, group, zeros, M, N, K, out)
            codes, scales, z = random_matrix(rng, N, K, fmt, group, zeros)
            x = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32)).to(torch.bfloat16)
            m, keep = matrix(codes, scales, z, fmt, group, fill=15)
            y = product(M, x.cuda(), m, N, out)
            check(y, x.double().numpy(), codes, scales, z, fmt, group, out)
            again = product(M, x.cuda(), m, N, out)
            assert torch.equal(y, again)
            del keep


@pytest.mark.parametrize("fmt,group,zeros", FORMS)
@pytest.mark.parametrize("M", (1, 3, 7, 16, 20, 48, 100))
def test_w4_gemm_exact_integers(fmt, group, zeros, M):
    """Whole numbers and powers of two: every sum is exact, so is the result."""
    rng = np.random.default_rng(M)
    for N, K in ((80, 1024), (33, 300), (7, 129)):
        say("w4_gemm exact", fmt, group, zeros, M, N, K)
        codes, scales, z = random_matrix(rng, N, K, fmt, group, zeros)
        scales = rng.integers(126, 129, scales.shape).astype(np.uint8) if fmt == "mxfp4" else \
            np.exp2(rng.integers(-1, 2, scales.shape)).astype(np.float32)
        x = torch.from_numpy(rng.integers(-4, 5, (M, K)).astype(np.float32)).to(torch.bfloat16)
        m, keep = matrix(codes, scales, z, fmt, group)
        y = product(M, x.cuda(), m, N, "f32")
        ref = x.double().numpy() @ w4.values(codes, scales, z, fmt, group).T
        assert np.array_equal(y.double().cpu().numpy(), ref)
        del keep


def test_w4_gemm_strides_and_unaligned_rows():
    """Rows of x with odd and padded strides and an odd start, a padded y whose
    padding stays, and a padded matrix."""
    rng = np.random.default_rng(3)
    for M, N, K, ldx, off, ldy, ldw in ((5, 50, 200, 203, 1, 57, 0), (3, 40, 256, 264, 0, 64, 320), (20, 33, 512, 512, 3, 33, 544),
                                        (2, 16, 136, 136, 4, 20, 160)):
        say("w4_gemm strides", M, N, K, ldx, off, ldy, ldw)
        codes, scales, z = random_matrix(rng, N, K, "int", 64, True)
        flat = torch.from_numpy(rng.standard_normal(off + M * ldx).astype(np.float32)).to(torch.bfloat16)
        x = flat[off:].reshape(M, ldx)[:, :K].double().numpy()
        flat[off:].reshape(M, ldx)[:, K:] = float("nan")
        buf = flat.cuda()
        m, keep = matrix(codes, scales, z, "int", 64, ldw=ldw, fill=15)
        y = product(M, buf.data_ptr() + 2 * off, m, N, "f32", ldx=ldx, ldy=ldy)
        check(y[:, :N], x, codes, scales, z, "int", 64, "f32")
        assert torch.all(y[:, N:] == 7.0)
        del keep


def test_w4_gemm_mxfp4_scale_ends():
    """The whole range of block scales: the smallest, the largest, and the NaN
    code.  Every code is present, so with scales 2^126 and 2^127 a row holds
    values of 4 * 2^126 = 2^128 and more, which are infinities and make the
    row's sum NaN where x is zero."""
    codes = np.tile(np.arange(16, dtype=np.uint8), (6, 2))
    x = torch.zeros(1, 32, dtype=torch.bfloat16)
    x[0, 2] = 1.0                                            # code 2: the value 1
    scales = np.array([[1], [127], [200], [253], [254], [255]], np.uint8)
    m, keep = matrix(codes, scales, None, "mxfp4", 32)
    y = product(1, x.cuda(), m, 6, "f32").cpu().numpy()[0]
    assert np.array_equal(y[:3], np.ldexp(1.0, scales[:3, 0].astype(int) - 127).astype(np.float32)) and np.all(np.isnan(y[3:]))
    back = torch.empty(6, 32, device="cuda")
    g.gemm355_w4_dequantize(m, back, dst=g.SRC_F32)
    with np.errstate(over="ignore"):
        want = w4.values(codes, scales, None, "mxfp4", 32).astype(np.float32)
    assert np.array_equal(back.cpu().numpy(), want, equal_nan=True) and np.isinf(want[3]).any()
    del keep


def test_w4_gemm_k_zero_and_rows_behind():
    m = g.make_w4_matrix(20, 0, group=64)
    y = product(3, None, m, 20, "f32", ldy=24)
    assert torch.all(y[:, :20] == 0) and torch.all(y[:, 20:] == 7.0)
    rng = np.random.default_rng(4)
    codes, scales, z = random_matrix(rng, 24, 64, "int", 64, False)
    m, keep = matrix(codes, scales, z, "int", 64)
    y = torch.full((9, 24), 5.0, device="cuda")
    x = torch.ones(9, 64, dtype=torch.bfloat16, device="cuda")
    g.gemm355_w4_gemm(4, x, m, y, out=g.SRC_F32)
    assert torch.all(y[4:] == 5.0) and not torch.any(y[:4] == 5.0)
    del keep


@pytest.mark.parametrize("fmt,group,zeros", FORMS)
@pytest.mark.parametrize("src", ("f32", "bf16"))
def test_w4_quantize_bit_exact(fmt, group, zeros, src):
    rng = np.random.default_rng(group)
    for N, K, ld, off in ((3, 32, 32, 0), (5, 1000, 1000, 0), (7, 129, 131, 1), (2, 1, 1, 0), (64, 512, 520, 0), (4, 260, 260, 2)):
        say("w4_quantize", fmt, group, zeros, src, N, K, ld, off)
        w = rng.standard_normal((N, ld)).astype(np.float32) * np.exp(rng.standard_normal((N, 1)) * 4).astype(np.float32)
        w[0, :K // 2] = 0.0
        if N > 2:
            w[1] = np.abs(w[1]) + 1e-3                       # one side of zero alone
            w[2] = rng.choice(np.array([-3.5, -0.75, 0.25, 0.5, 1.25, 2.5, 5.0, 7.0], np.float32), ld)   # ties
        if N > 4:
            w[3] *= np.float32(2.0 ** -110)
            w[4] = -0.0
        t = torch.from_numpy(np.concatenate([np.zeros(off, np.float32), w.reshape(-1)]))
        t = t.to(torch.bfloat16) if src == "bf16" else t
        seen = t[off:].reshape(N, ld)[:, :K].float().numpy()
        buf = t.cuda()
        codes, scales, z = w4.quantize(seen, fmt, group, zeros)
        width = -(-K // 32) * 32
        out = torch.full((N, width // 2), 0xAA, dtype=torch.uint8, device="cuda")
        s = torch.zeros(scales.shape, dtype=torch.uint8 if fmt == "mxfp4" else torch.bfloat16, device="cuda")
        zp = torch.full(scales.shape, 99, dtype=torch.uint8, device="cuda") if zeros else None
        m = g.make_w4_matrix(N, K, out, s, zp, fmt=g.W4_MXFP4 if fmt == "mxfp4" else g.W4_INT, group=group)
        g.gemm355_w4_quantize(buf.data_ptr() + off * buf.element_size(), m, src=g.SRC_BF16 if src == "bf16" else g.SRC_F32, ld=ld)
        torch.cuda.synchronize()
        assert np.array_equal(s.float().cpu().numpy().astype(scales.dtype), scales)
        if zeros:
            assert np.array_equal(zp.cpu().numpy(), z)
        nb = (K + 1) // 2
        assert np.array_equal(out.cpu().numpy()[:, :nb], w4.pack(codes, width)[:, :nb])
        tail = -(-K // 8) * 4
        assert torch.all(out[:, tail:] == 0xAA)
        # and back
        vals = w4.values(codes, scales, z, fmt, group)
        for dst, dt in (("f32", torch.float32), ("bf16", torch.bfloat16)):
            back = torch.full((N, ld), 3.0, dtype=dt, device="cuda")
            g.gemm355_w4_dequantize(m, back, dst=g.SRC_BF16 if dst == "bf16" else g.SRC_F32, ld=ld)
            ref = torch.from_numpy(vals.astype(np.float32)).to(dt)
            assert torch.equal(back[:, :K].cpu(), ref) and torch.all(back[:, K:] == 3.0)


def test_dequantized_weights_in_the_dense_product():
    """Quantise, dequantise to bf16, and the tiled product agrees with the
    product over the codes (block-scaled FP4 is exact in bf16)."""
    rng = np.random.default_rng(12)
    N, K, M = 256, 512, 24
    w = torch.from_numpy(rng.standard_normal((N, K)).astype(np.float32)).to(torch.bfloat16).cuda()
    x = torch.from_numpy(rng.integers(-3, 4, (M, K)).astype(np.float32)).to(torch.bfloat16).cuda()
    codes = torch.empty(N, K // 2, dtype=torch.uint8, device="cuda")
    s = torch.empty(N, K // 32, dtype=torch.uint8, device="cuda")
    m = g.make_w4_matrix(N, K, codes, s, fmt=g.W4_MXFP4, group=32)
    g.gemm355_w4_quantize(w, m)
    back = torch.empty_like(w)
    g.gemm355_w4_dequantize(m, back)
    y1 = torch.empty(M, N, device="cuda")
    y2 = torch.empty(M, N, device="cuda")
    g.gemm355_w4_gemm(M, x, m, y1, out=g.SRC_F32)
    g.gemm355_gemm(M, N, K, x, K, back, K, y2, N, g.BF16_F32)
    ref = x.double().cpu() @ back.double().cpu().T
    assert torch.allclose(y1.double().cpu(), ref, rtol=0, atol=1e-4) and torch.allclose(y2.double().cpu(), ref, rtol=0, atol=1e-4)


def test_w4_gemm_streams_and_graph():
    """On a stream other than the current one, and captured: replays follow
    new contents of x and equal the eager result each time."""
    rng = np.random.default_rng(13)
    N, K, M = 500, 1100, 3
    codes, scales, z = random_matrix(rng, N, K, "int", 32, True)
    m, keep = matrix(codes, scales, z, "int", 32)
    x = torch.randn(M, K, device="cuda").to(torch.bfloat16)
    want = product(M, x, m, N, "f32")
    side = torch.cuda.Stream()
    y = torch.zeros(M, N, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    g.gemm355_w4_gemm(M, x, m, y, out=g.SRC_F32, stream=side)
    side.synchronize()
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.gemm355_w4_gemm(M, x, m, y, out=g.SRC_F32)
    for i in range(4):
        x.copy_(torch.randn(M, K, device="cuda"))
        want = product(M, x, m, N, "f32")
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), i
    del keep


def test_default_stream_is_the_current_one():
    """Calls without a stream go to torch's current stream of the current device,
    whichever it is at the call."""
    side = torch.cuda.Stream()
    assert g._stream(None) == torch.cuda.current_stream().cuda_stream
    with torch.cuda.stream(side):
        assert g._stream(None) == side.cuda_stream
    assert g._stream(None) == torch.cuda.current_stream().cuda_stream != side.cuda_stream
