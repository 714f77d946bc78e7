"""GPU parity of the block-scaled operators with the oracle (oracle/block.py).

Codes and scales of the quantiser, and the norm's sum, are compared bit for bit.

Products, |y - ref| <= n * 2^-23 * A + half a step of the output, from the order of
the sums, A = sum |x w|: a block's sum has at most 128 terms, one multiply-add a
block, 8 wavefronts or parts of K at most 256 to join, and the product of the two
scales is rounded: n = min(K, 128) + blocks + joins + 2 roundings, each off by at
most 2^-23 (an adder that truncates) of sums of at most A.  For rows of bf16
the 8-bit instruction cuts each product off at 2^-13 of the largest power of
two in its group of 8: 7 others, each off by less than that, so 7 * 2^-13 * T with T
the sum of the groups' largest |x w|.  (A group is 8 K-values that begin at a
multiple of 8: 1 + 2^-14 at K = 0 and 1 is 1, at K = 0 and 16 it is exact, and of
127 values of 2^-14 beside a 1, 120 arrive.)  Small whole numbers with power-of-two
scales are exact in every step and compared bit for bit.

Gated pairs: h = act(g) u with g and u off by eg and eu as above, |act'| <= 1.13,
and act's own rounding: the exponential of z is off by (|z| + 2) 2^-23 (its
argument's rounding and its own), z of GELU by 5 roundings, quotient and products
by 4 more: (6 |z| + 10) 2^-23 |h| in all.  A result that exp(-z) = infinity makes
0 is under 2^-120 |g u|.

Codes out of computed rows: the value they stand for is off by at most half a step
of E4M3, 2^-4 of it or 2^-10 scales, and by the row's own error; the scale by the
error of the largest / 448 and one rounding.

Norm: the mean of squares is a sum of terms that are not negative: 8 a thread and
octet, 6 and 16 joins, off by (8 + 4 + 22) 2^-24 relative, half of which enters by
the square root; eps, root, division and two products add 6 roundings: 2^-19 bounds
them.
"""
import numpy as np
import pytest
import torch

from dense_tiled_gemm_fp8_amd import gemm355 as g
from oracle import block, w4

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
SRC = {"bf16": g.SRC_BF16, "f32": g.SRC_F32}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a).copy()).cuda()


def r16(n):
    return -(-n // 16) * 16


class Matrix:
    """A matrix on the device; rows `pad` bytes longer than they need be, bytes
    behind K of value `fill`, and scales `spad` floats further apart."""

    def __init__(self, codes, scales, block_rows, pad=0, fill=0x7F, spad=0):
        rows, K = codes.shape
        self.rows, self.K, self.block_rows = rows, K, block_rows
        self.ld = r16(K) + pad
        buf = np.full((rows, self.ld), fill, np.uint8)
        buf[:, :K] = codes
        held = scales.T if block_rows == 1 else scales
        sbuf = np.full((held.shape[0], held.shape[1] + spad), np.nan, np.float32)
        sbuf[:, :held.shape[1]] = held
        self.codes, self.scales = dev(buf), dev(sbuf)
        self.m = g.make_block_matrix(rows, K, self.codes, self.scales, block_rows, ld=self.ld, ld_scale=sbuf.shape[1])

    def host(self):
        torch.cuda.synchronize()
        s = self.scales.cpu().numpy()
        n = self.rows if self.block_rows == 1 else -(-self.K // 128)
        s = s[:, :n]
        return self.codes.cpu().numpy()[:, :self.K], s.T if self.block_rows == 1 else s


def empty(rows, K, block_rows=1, pad=0, spad=0):
    nr, nk = -(-rows // block_rows), -(-K // 128)
    return Matrix(np.full((rows, K), 0x55, np.uint8), np.full((nr, nk), -7.0, np.float32), block_rows, pad, 0x55, spad)


def random_codes(rng, rows, K):
    c = rng.integers(0, 127, (rows, K)).astype(np.uint8)
    return c | (rng.integers(0, 2, (rows, K)) << 7).astype(np.uint8)


def random_matrix(rng, rows, K, block_rows, **kw):
    codes = random_codes(rng, rows, K)
    scales = np.exp(rng.uniform(-6, 0, (-(-rows // block_rows), -(-K // 128)))).astype(np.float32)
    return Matrix(codes, scales, block_rows, **kw), codes, scales


def values(m, codes, scales):
    return block.values(codes, scales, m.block_rows)


# ------------------------------------------------------------------ quantiser

@pytest.mark.parametrize("src", ("bf16", "f32"))
@pytest.mark.parametrize("block_rows", (1, 128))
@pytest.mark.parametrize("rows,K", [(1, 1), (1, 7), (1, 128), (15, 100), (16, 127), (17, 129), (3, 1000), (130, 200), (128, 128),
                                    (257, 777), (64, 2048), (300, 4099)])
def test_quantize(rows, K, block_rows, src):
    rng = np.random.default_rng(rows * 5000 + K)
    x = (rng.standard_normal((rows, K)) * np.exp(rng.uniform(-30, 30, (rows, 1)))).astype(np.float32)
    x[rng.random((rows, K)) < 0.1] = 0.0
    if rows > 2:
        x[1] = 0.0
        x[2] = 2.0 ** -101
    x = w4.bf16(x) if src == "bf16" else x
    for ld, off, pad, spad in ((0, 0, 0, 0), (K + 3, 1, 32, 5)):
        buf = torch.zeros(rows * max(ld, K) + off, dtype=DT[src], device="cuda")
        view = buf[off:].view(rows, max(ld, K))
        view[:, :K] = dev(x).to(DT[src])
        q = empty(rows, K, block_rows, pad, spad)
        g.gemm355_block_quantize(buf[off:], q.m, src=SRC[src], ld=ld)
        codes, scales = q.host()
        want, ws = block.quantize(x, block_rows)
        assert np.array_equal(scales, ws)
        assert np.array_equal(codes, want)
        # nothing behind a row's K values, or behind the scales of a block
        assert bool((q.codes[:, K:] == 0x55).all())
        if spad:
            assert bool(torch.isnan(q.scales[:, -spad:]).all())


def test_quantize_large_and_small_magnitudes():
    """Maxima of 2^-100, of the largest fp32 value, and codes at every border."""
    x = np.zeros((4, 256), np.float32)
    x[0, 3], x[0, 130] = 2.0 ** -100, np.nextafter(np.float32(2.0 ** -100), np.float32(0))
    x[1, :128] = np.float32(3.4028234e38) * np.linspace(-1, 1, 128)
    v = block.decode(np.arange(127, dtype=np.uint8))
    x[2, :127] = v
    x[3, :126] = (v[1:] + v[:-1]) / 2          # ties between neighbours, 448 beside them
    x[3, 126] = 448
    q = empty(4, 256)
    g.gemm355_block_quantize(dev(x), q.m, src=g.SRC_F32)
    codes, scales = q.host()
    want, ws = block.quantize(x, 1)
    assert np.array_equal(scales, ws) and np.array_equal(codes, want)
    assert ws[2, 0] == 1 and np.array_equal(codes[2, :127], np.arange(127))


def test_quantize_of_what_is_not_finite_stays_in_its_block():
    x = np.ones((20, 300), np.float32)
    x[3, 130], x[7, 5] = np.inf, np.nan
    q, clean = empty(20, 300), empty(20, 300)
    g.gemm355_block_quantize(dev(x), q.m, src=g.SRC_F32)
    g.gemm355_block_quantize(dev(np.ones((20, 300))).float(), clean.m, src=g.SRC_F32)
    (a, b), (c, d) = q.host(), clean.host()
    for r in range(20):
        for k in range(3):
            if (r, k) not in ((3, 1), (7, 0)):
                assert np.array_equal(a[r, k * 128:(k + 1) * 128], c[r, k * 128:(k + 1) * 128]) and b[r, k] == d[r, k]


# ------------------------------------------------------------------ norm

def norm_check(rows, width, x_type, r_type, y_type, codes, weight, residual=True, ld=0, seed=0, off=0):
    rng = np.random.default_rng(seed + rows * 100000 + width)
    as_type = lambda a, t: w4.bf16(a.astype(np.float32)) if t == "bf16" else a.astype(np.float32)   # noqa: E731
    x = as_type(rng.standard_normal((rows, width)) * np.exp(rng.uniform(-3, 3, (rows, 1))), x_type)
    r = as_type(rng.standard_normal((rows, width)), r_type) if residual else None
    if rows > 3:
        x[2], x[3] = 0.0, 1e-12
        if residual:
            r[2] = 0.0
    w = as_type(rng.standard_normal(width), weight) if weight else None
    pitch = ld or width

    def rows_of(a, t):
        buf = torch.full((rows * pitch + off,), 7.0, dtype=DT[t], device="cuda")
        if a is not None:
            buf[off:].view(rows, pitch)[:, :width] = dev(a).to(DT[t])
        return buf[off:]

    xd, rd = rows_of(x, x_type), rows_of(r, r_type) if residual else None
    hd, yd = rows_of(None, r_type) if residual else None, rows_of(None, y_type) if y_type else None
    wd = dev(w).to(DT[weight]) if weight else None
    q = empty(rows, width, 1, 16, 2) if codes else None
    eps = 1e-6
    g.gemm355_rmsnorm(g.make_rmsnorm_args(
        rows, width, x=xd, x_type=SRC[x_type], residual=rd, sum=hd, r_type=SRC[r_type], weight=wd, w_type=SRC[weight or "f32"],
        eps=eps, y=yd, y_type=SRC[y_type or "f32"], q=q.m if codes else None, ldx=ld, ldr=ld, lds=ld, ldy=ld))
    torch.cuda.synchronize()
    h = block.norm_input(x, r, r_type)
    if residual:
        got = hd.view(rows, pitch).float().cpu().numpy()
        assert np.array_equal(got[:, :width], h) and np.all(got[:, width:] == 7)
    ref = block.rmsnorm(h, w, eps)
    off_by = 2.0 ** -19 * np.abs(ref) + 1e-37
    if y_type:
        got = yd.view(rows, pitch).float().cpu().numpy()
        assert np.all(got[:, width:] == 7)
        assert np.all(np.abs(got[:, :width] - ref) <= off_by + HALF[y_type] * (np.abs(ref) + off_by))
    if codes:
        check_codes(q, ref, off_by)


def check_codes(q, ref, off_by):
    codes, scales = q.host()
    rows, width = ref.shape
    for k in range(scales.shape[1]):
        at = np.s_[:, k * 128:(k + 1) * 128]
        a, e = np.abs(ref[at]).max(1), off_by[at].max(1)
        s = scales[:, k].astype(float)
        sure = np.abs(a - 2.0 ** -100) > e
        none = a < 2.0 ** -100
        assert np.all((s == 1)[sure & none])
        assert np.all((np.abs(s - a / 448) <= e / 448 + 2.0 ** -24 * (a + e) / 448)[sure & ~none])
        got = block.decode(codes[at]) * s[:, None]
        # x * i: two roundings before the code, a value of the code by one product of 64 bits
        near = np.maximum(2.0 ** -4 * np.abs(ref[at]), 2.0 ** -10 * s[:, None]) * (1 + 2.0 ** -20) + 2 * off_by[at] + e[:, None]
        assert np.all((np.abs(got - ref[at]) <= near)[sure]) and np.all(np.isfinite(got))
    assert bool((q.codes[:, width:] == 0x55).all())


@pytest.mark.parametrize("width", (1, 8, 127, 128, 129, 512, 513, 777, 1024, 2048, 2056, 4096, 4100, 8192, 8200, 16384, 32768))
@pytest.mark.parametrize("rows", (1, 5, 70))
def test_norm_widths(rows, width):
    norm_check(rows, width, "bf16", "bf16", "bf16", True, "bf16")


@pytest.mark.parametrize("x_type", ("bf16", "f32"))
@pytest.mark.parametrize("r_type", ("bf16", "f32"))
@pytest.mark.parametrize("y_type", ("bf16", "f32", None))
@pytest.mark.parametrize("weight", ("bf16", "f32", None))
def test_norm_types(x_type, r_type, y_type, weight):
    norm_check(9, 640, x_type, r_type, y_type, y_type != "f32", weight)


@pytest.mark.parametrize("ld,off", ((1000, 0), (1003, 0), (0, 1), (1008, 8)))
def test_norm_pitch_and_alignment(ld, off):
    norm_check(6, 1000, "bf16", "f32", "bf16", True, "bf16", ld=ld, off=off)


@pytest.mark.parametrize("y_type,codes", (("bf16", False), ("f32", True), (None, True)))
def test_norm_without_residual(y_type, codes):
    norm_check(40, 300, "f32", "bf16", y_type, codes, "f32", residual=False)


def test_norm_without_the_sum():
    """A residual whose sum is not kept."""
    x, r = (torch.randn(7, 3000, device="cuda").bfloat16() for _ in range(2))
    h, a, b = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    g.gemm355_rmsnorm(g.make_rmsnorm_args(7, 3000, x=x, residual=r, sum=h, y=a))
    g.gemm355_rmsnorm(g.make_rmsnorm_args(7, 3000, x=x, residual=r, y=b))
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_norm_in_place():
    """sum over the residual, y over x; then sum over x."""
    rng = np.random.default_rng(3)
    for width in (200, 4096, 9000):
        x, r = (w4.bf16(rng.standard_normal((33, width)).astype(np.float32)) for _ in range(2))
        xd, rd = dev(x).bfloat16(), dev(r).bfloat16()
        h, y = torch.empty_like(xd), torch.empty_like(xd)
        g.gemm355_rmsnorm(g.make_rmsnorm_args(33, width, x=xd, residual=rd, sum=h, y=y))
        a, b = xd.clone(), rd.clone()
        g.gemm355_rmsnorm(g.make_rmsnorm_args(33, width, x=a, residual=b, sum=b, y=a))
        torch.cuda.synchronize()
        assert torch.equal(b, h) and torch.equal(a, y)
        a, b = xd.clone(), rd.clone()
        g.gemm355_rmsnorm(g.make_rmsnorm_args(33, width, x=a, residual=b, sum=a, y=b))
        torch.cuda.synchronize()
        assert torch.equal(a, h) and torch.equal(b, y)


# ------------------------------------------------------------------ products

def joins(splits):
    return 8 + (splits if splits else 256)


def bound(A, K, splits=0):
    return (min(K, 128) + -(-K // 128) + joins(splits) + 2) * 2.0 ** -23 * A


def groups(X, W):
    """T: the sum over 8 K-values each of the largest |x w|."""
    a, b = dev(np.abs(X)), dev(np.abs(W))
    t = torch.zeros(X.shape[0], W.shape[0], dtype=torch.float64, device="cuda")
    for k in range(0, X.shape[1], 8):
        t += (a[:, None, k:k + 8] * b[None, :, k:k + 8]).amax(2)
    return t.cpu().numpy()


def cut(T):
    return 7 * 2.0 ** -13 * T


SHAPES = [(1, 1, 1), (1, 16, 128), (1, 1024, 1024), (2, 17, 33), (3, 250, 776), (5, 300, 777), (8, 96, 640), (15, 129, 100),
          (16, 48, 2048), (17, 130, 515), (33, 200, 1000), (64, 128, 512), (65, 40, 384), (130, 33, 31), (1, 4099, 260),
          (100, 1000, 1500), (129, 257, 255), (256, 256, 256), (300, 520, 1040), (513, 300, 129), (31, 260, 16384)]


def run_gemm(x, w, out, splits=0, ld=0, off=0, ws=None):
    M, N = x.rows, w.rows
    pitch = ld or N
    buf = torch.full((M * pitch + off,), 7.0, dtype=DT[out], device="cuda")
    g.gemm355_block_gemm(g.make_block_gemm_args(x.m, w.m, y=buf[off:], out=SRC[out], ldy=ld, splits=splits, workspace=ws,
                                                workspace_bytes=0 if ws is None else ws.numel()))
    torch.cuda.synchronize()
    assert bool((buf[:off] == 7).all())
    full = buf[off:].view(M, pitch)
    assert bool((full[:, N:] == 7).all())
    return full[:, :N]


@pytest.mark.parametrize("out", ("bf16", "f32"))
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm(M, N, K, out):
    rng = np.random.default_rng(M * 10007 + N * 101 + K)
    x, xc, xs = random_matrix(rng, M, K, 1, pad=16 * (M % 2), spad=M % 3)
    w, wc, ws = random_matrix(rng, N, K, 128, pad=16 * (N % 2), spad=N % 3)
    X, W = values(x, xc, xs), values(w, wc, ws)
    ref, A = X @ W.T, np.abs(X) @ np.abs(W).T
    T = groups(X, W) if out == "bf16" else 0.0
    for splits, ld, off in ((0, 0, 0), (1, N + 5, 1), (3, N + 8 - N % 8, 0)):
        y = run_gemm(x, w, out, splits, ld, off).double().cpu().numpy()
        tol = bound(A, K, splits) + cut(T)
        err = np.abs(y - ref)
        tol = tol + HALF[out] * (np.abs(ref) + tol)
        assert np.all(err <= tol), "splits %d: %d outside, worst %.3g of the tolerance" % (
            splits, int((err > tol).sum()), float((err / np.maximum(tol, 1e-300)).max()))


def whole_matrix(rng, rows, K, block_rows, low, high, **kw):
    """Whole numbers from -4 to 4 and scales of powers of two, another for each block."""
    v = rng.integers(-4, 5, (rows, K))
    codes = torch.from_numpy(v.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    scales = np.exp2(rng.integers(low, high + 1, (-(-rows // block_rows), -(-K // 128)))).astype(np.float32)
    return Matrix(codes, scales, block_rows, **kw), v * block.spread(scales, rows, K, block_rows)


@pytest.mark.parametrize("splits", (0, 1, 2, 7))
@pytest.mark.parametrize("M,N,K", [(1, 300, 2000), (7, 513, 1111), (16, 256, 4096), (40, 400, 1024), (64, 384, 2050), (128, 700, 1300),
                                   (200, 512, 640), (257, 385, 1024), (600, 1030, 515)])
def test_gemm_exact(M, N, K, splits):
    """Products of at most 16 * 2, sums of at most 2^5 K <= 2^17.5, in steps of 2^-6:
    under 2^24 of them, exact whatever the order."""
    rng = np.random.default_rng(M + N + K + splits)
    x, X = whole_matrix(rng, M, K, 1, -3, 0, pad=16)
    w, W = whole_matrix(rng, N, K, 128, -3, 1)
    y = run_gemm(x, w, "f32", splits)
    assert np.array_equal(y.cpu().numpy().astype(np.float64), X @ W.T)


# sizes that each form is chosen for (of 256 compute units) with one matrix and with
# two, for bf16, codes and fp32: rows of 16, 32 and 64 tokens, streams of 128, tiles from
# 128 x 64 to 256 x 256, whole and in parts of K, one unit a workgroup and several
LARGE = [(1, 33, 4329), (1, 533, 4294), (66, 35, 138), (153, 34, 133), (129, 36, 145), (259, 33, 131), (267, 68, 203),
         (291, 33, 139), (296, 34, 2453), (257, 79, 2722), (274, 35, 406), (52, 4097, 268), (33, 5655, 142), (49, 8582, 139),
         (36, 12398, 130), (131, 8812, 310), (137, 8214, 149), (286, 11320, 129), (386, 11371, 131), (925, 10981, 150),
         (700, 6100, 400), (257, 9972, 1229), (2053, 33, 3795), (2101, 33, 5166), (2134, 70, 5722), (1028, 6068, 1301),
         (1319, 5909, 133), (4200, 1100, 130), (1300, 9000, 260), (2100, 8300, 149)]


@pytest.mark.parametrize("M,N,K", LARGE + [(1284, 11057, 145), (257, 10882, 147), (1410, 15694, 131), (569, 11511, 1172)])
def test_gemm_exact_large(M, N, K):
    """As above, and rows of bf16: the exact sums rounded once; rows behind the last
    and columns behind a row's stay as they were."""
    rng = np.random.default_rng(M + N + K)
    x, X = whole_matrix(rng, M, K, 1, -3, 0, pad=16, spad=1)
    w, W = whole_matrix(rng, N, K, 128, -3, 1, pad=32, spad=2)
    ref = dev(X) @ dev(W).T
    for out in ("f32", "bf16"):
        for ld, off in ((0, 0), (N + 3, 1), (N + 8 - N % 8, 0)):
            assert torch.equal(run_gemm(x, w, out, 0, ld, off).double(), ref.to(DT[out]).double()), (out, ld, off)


@pytest.mark.parametrize("kind", ("silu", "gelu"))
@pytest.mark.parametrize("M,N,K", LARGE)
def test_gated_large(M, N, K, kind):
    """Both sums exact (scales of 2^-9 on x keep them near the activation's bend), so
    that the activation's rounding alone is left."""
    rng = np.random.default_rng(M + N + K + 1)
    x, X = whole_matrix(rng, M, K, 1, -9, -8, pad=16)
    (gate, G), (up, U) = (whole_matrix(rng, N, K, 128, -3, 1, spad=2) for _ in range(2))
    gr, ur = ((dev(X) @ dev(B).T).cpu().numpy() for B in (G, U))
    h = block.act(gr, kind) * ur
    off_by = (6 * z_of(gr, kind) + 10) * 2.0 ** -23 * np.abs(h) + 2.0 ** -120 * np.abs(gr * ur) + 1e-37
    for out, ld, off in (("bf16", 0, 0), ("bf16", N + 3, 1), ("f32", N + 8 - N % 8, 0), ("8bit", 0, 0)):
        y = run_gated(x, gate, up, kind, out, 0, ld, off)
        if out == "8bit":
            check_codes(y, h, off_by)
            continue
        err = np.abs(y.double().cpu().numpy() - h)
        assert np.all(err <= off_by + HALF[out] * (np.abs(h) + off_by)), (out, float(err.max()))


@pytest.mark.parametrize("M,N,K,splits", [(385, 10171, 566, 5), (34, 13207, 527, 5), (524, 12721, 2122, 2), (137, 10186, 518, 5),
                                          (33, 6824, 522, 5), (5, 100, 1000, 200), (200, 300, 1000, 256)])
def test_parts_told_large(M, N, K, splits):
    """More units than workgroups run at once, each a part of K; more parts told than
    there are K blocks."""
    rng = np.random.default_rng(M + N + K)
    x, X = whole_matrix(rng, M, K, 1, -3, 0, pad=16)
    w, W = whole_matrix(rng, N, K, 128, -3, 1)
    u, U = whole_matrix(rng, N, K, 128, -3, 1)
    ref, up = dev(X) @ dev(W).T, dev(X) @ dev(U).T
    assert torch.equal(run_gemm(x, w, "f32", splits).double(), ref)
    assert torch.equal(run_gemm(x, w, "bf16", splits), ref.bfloat16())
    q = run_gated(x, w, u, "silu", "8bit", splits)
    one = run_gated(x, w, u, "silu", "8bit", 1)
    assert all(np.array_equal(a, b) for a, b in zip(q.host(), one.host()))
    y = run_gated(x, w, u, "silu", "bf16", splits).double()
    h = ref * torch.sigmoid(ref) * up
    off = (6 * ref.abs() + 10) * 2.0 ** -23 * h.abs() + 2.0 ** -120 * (ref * up).abs() + 1e-37
    assert bool(((y - h).abs() <= off + HALF["bf16"] * (h.abs() + off)).all())


def test_past_32_bit_offsets():
    """A matrix of weights, rows of activations and outputs of more than 2^32 bytes:
    the last rows and columns, bit for bit."""
    N, K = 66000, 65536                                   # 4.3e9 codes
    w = torch.randint(0, 5, (N, K), device="cuda", dtype=torch.uint8)
    w += 0x38                                             # 1, 1.125 .. 1.5
    ws = torch.ones(-(-N // 128), K // 128, device="cuda")
    wm = g.make_block_matrix(N, K, w, ws, block_rows=128)
    x, X = whole_matrix(np.random.default_rng(1), 3, K, 1, 0, 0)
    y = torch.zeros(3, N, device="cuda")
    g.gemm355_block_gemm(g.make_block_gemm_args(x.m, wm, y=y, out=g.SRC_F32))
    torch.cuda.synchronize()
    for n0 in (0, 32768, N - 130):
        part = w[n0:n0 + 130].view(torch.float8_e4m3fn).double()
        ref = dev(X) @ part.T                             # sums of eighths under 2^19: exact
        assert torch.equal(y[:, n0:n0 + 130].double(), ref)
    # the same bytes as activations: 66000 tokens by 40 columns
    xs = torch.ones(K // 128, N, device="cuda")
    xm = g.make_block_matrix(N, K, w, xs)
    v, V = whole_matrix(np.random.default_rng(2), 40, K, 128, 0, 0)
    out = torch.zeros(N, 40, device="cuda")
    g.gemm355_block_gemm(g.make_block_gemm_args(xm, v.m, y=out, out=g.SRC_F32))
    torch.cuda.synchronize()
    for m0 in (0, 32768, N - 130):
        part = w[m0:m0 + 130].view(torch.float8_e4m3fn).double()
        assert torch.equal(out[m0:m0 + 130].double(), part @ dev(V).T)
    del out, y
    # quantised out of bf16 rows of 8.7e9 bytes; a norm over rows of as many
    src = torch.ones(N, K, dtype=torch.bfloat16, device="cuda")
    src[-1] = 3.0
    g.gemm355_block_quantize(src, xm)
    torch.cuda.synchronize()
    assert bool((w[-2:] == 0x7E).all()) and bool((w[0] == 0x7E).all())
    assert float(xs[0, 0]) == float(np.float32(1) / np.float32(448)) and float(xs[-1, -1]) == float(np.float32(3) / np.float32(448))
    rows, width = N * 8, K // 8
    r = torch.full((rows, width), 2.0, dtype=torch.bfloat16, device="cuda")
    g.gemm355_rmsnorm(g.make_rmsnorm_args(rows, width, x=src, residual=r, sum=r, y=src))
    torch.cuda.synchronize()
    assert bool((r[-1] == 5).all()) and bool((r[0] == 3).all()) and bool((src[-1] == 1).all()) and bool((src[0] == 1).all())


def test_gemm_nothing_along_k():
    x, w = Matrix(np.zeros((5, 0), np.uint8), np.zeros((5, 0), np.float32), 1), Matrix(np.zeros((70, 0), np.uint8), np.zeros((1, 0), np.float32), 128)
    for out in ("f32", "bf16"):
        assert not bool(run_gemm(x, w, out).any())


@pytest.mark.parametrize("out", ("bf16", "f32"))
@pytest.mark.parametrize("M,N,K", [(3, 400, 700), (30, 400, 700), (60, 400, 700), (200, 400, 700), (300, 700, 515), (137, 8214, 149),
                                   (131, 8812, 310), (1300, 9000, 260)])
def test_gemm_nan_scales_stay_where_they_are(M, N, K, out):
    """A NaN scale of x reaches its row, one of w its 128 columns, a NaN code its
    row or column, and nothing else changes a bit."""
    rng = np.random.default_rng(9)
    xc, wc = random_codes(rng, M, K), random_codes(rng, N, K)
    xs, ws = np.ones((M, -(-K // 128)), np.float32), np.ones((-(-N // 128), -(-K // 128)), np.float32)
    clean = run_gemm(Matrix(xc, xs, 1), Matrix(wc, ws, 128), out).float().cpu().numpy()
    xs[1, 1], ws[1, 0], xc[2, 600 % K], wc[5, 9] = np.nan, np.nan, 0x7F, 0xFF
    y = run_gemm(Matrix(xc, xs, 1), Matrix(wc, ws, 128), out).float().cpu().numpy()
    bad = np.zeros((M, N), bool)
    bad[1], bad[2], bad[:, 128:256], bad[:, 5] = True, True, True, True
    assert np.array_equal(np.isnan(y), bad)
    assert np.array_equal(y[~bad], clean[~bad])


def z_of(gate, kind):
    return np.abs(gate) if kind == "silu" else 1.6 * np.abs(gate + 0.044715 * gate ** 3)


def run_gated(x, gate, up, kind, out, splits=0, ld=0, off=0):
    M, N = x.rows, gate.rows
    act = g.ACT_SILU if kind == "silu" else g.ACT_GELU_TANH
    if out == "8bit":
        q = empty(M, N, 1, 16, 3)
        g.gemm355_block_gated(g.make_block_gated_args(x.m, gate.m, up.m, act=act, q=q.m, splits=splits))
        torch.cuda.synchronize()
        return q
    pitch = ld or N
    buf = torch.full((M * pitch + off,), 7.0, dtype=DT[out], device="cuda")
    g.gemm355_block_gated(g.make_block_gated_args(x.m, gate.m, up.m, act=act, y=buf[off:], out=SRC[out], ldy=ld, splits=splits))
    torch.cuda.synchronize()
    full = buf[off:].view(M, pitch)
    assert bool((buf[:off] == 7).all()) and bool((full[:, N:] == 7).all())
    return full[:, :N]


@pytest.mark.parametrize("kind", ("silu", "gelu"))
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 16, 128), (1, 1024, 1024), (3, 250, 776), (15, 129, 100), (17, 130, 515),
                                   (64, 128, 512), (65, 40, 384), (100, 1000, 1500), (129, 257, 255), (256, 256, 256), (300, 520, 1040),
                                   (513, 300, 129), (2, 140, 8192)])
def test_gated(M, N, K, kind):
    rng = np.random.default_rng(M * 10007 + N * 101 + K)
    x, xc, xs = random_matrix(rng, M, K, 1, pad=16, spad=1)
    # sums of the size of an activation's range
    parts = []
    for _ in range(2):
        codes = random_codes(rng, N, K)
        scales = (np.exp(rng.uniform(-2, 0, (-(-N // 128), -(-K // 128)))) * 1e-3 / np.sqrt(K)).astype(np.float32)
        parts.append((Matrix(codes, scales, 128, pad=16 * (N % 2)), block.values(codes, scales, 128)))
    X = values(x, xc, xs)
    (gate, G), (up, U) = parts
    gr, ur = X @ G.T, X @ U.T
    Ag, Au = np.abs(X) @ np.abs(G).T, np.abs(X) @ np.abs(U).T
    Tg, Tu = groups(X, G), groups(X, U)
    h = block.act(gr, kind) * ur
    for splits, out, ld, off in ((0, "bf16", 0, 0), (0, "8bit", 0, 0), (1, "f32", N + 3, 1), (3, "bf16", N + 8 - N % 8, 0),
                                 (3, "8bit", 0, 0), (1, "8bit", 0, 0)):
        eg, eu = bound(Ag, K, splits), bound(Au, K, splits)
        if out == "bf16":
            eg, eu = eg + cut(Tg), eu + cut(Tu)
        off_by = (1.13 * eg * (np.abs(ur) + eu) + np.abs(block.act(gr, kind)) * eu
                  + (6 * z_of(gr, kind) + 10) * 2.0 ** -23 * np.abs(h) + 2.0 ** -120 * np.abs(gr * ur) + 1e-37)
        y = run_gated(x, gate, up, kind, out, splits, ld, off)
        if out == "8bit":
            check_codes(y, h, off_by)
            continue
        err = np.abs(y.double().cpu().numpy() - h)
        tol = off_by + HALF[out] * (np.abs(h) + off_by)
        assert np.all(err <= tol), (splits, out, int((err > tol).sum()), float((err / tol).max()))


def test_gated_far_from_zero():
    """Gates of up to +-1000: the activation is g or 0 there, never a NaN."""
    for kind in ("silu", "gelu"):
        v = np.zeros((1, 128))
        v[0, 0] = 1
        codes = torch.from_numpy(v.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        scales = np.array([[1000.0], [-1000.0], [89.0], [-89.0], [0.0]], np.float32)
        x = Matrix(np.repeat(codes, 5, 0), scales, 1)
        one = Matrix(codes, np.ones((1, 1), np.float32), 128)
        y = run_gated(x, one, one, kind, "f32").cpu().numpy()[:, 0]
        assert y[0] == 1e6 and y[1] == 0 and abs(y[2] - 89 * 89) < 1e-2 and abs(y[3]) < 1e-30 and y[4] == 0


# ------------------------------------------------------------------ together, streams, graphs

def test_feed_forward_together():
    """Weights quantised, rows normed into codes, the gated pair into codes, the
    product of those, twice with the residual: against the same steps in 64 bits on
    the values that each step left."""
    rng = np.random.default_rng(11)
    for M in (1, 40, 300):
        D, I, K = 640, 900, 640
        wg, wu, wd = ((rng.standard_normal((n, k)) / np.sqrt(k)).astype(np.float32) for n, k in ((I, K), (I, K), (D, I)))
        mats = []
        for m in (wg, wu, wd):
            q = empty(m.shape[0], m.shape[1], 128)
            g.gemm355_block_quantize(dev(m), q.m, src=g.SRC_F32)
            mats.append(q)
        x, res = dev(rng.standard_normal((M, D)).astype(np.float32)).bfloat16(), dev(rng.standard_normal((M, D)).astype(np.float32)).bfloat16()
        w = dev((1 + 0.1 * rng.standard_normal(D)).astype(np.float32)).bfloat16()
        q, h, y = empty(M, D), empty(M, I), torch.empty(M, D, dtype=torch.bfloat16, device="cuda")
        for _ in range(2):
            h0 = block.norm_input(x.float().cpu().numpy(), res.float().cpu().numpy(), "bf16")
            g.gemm355_rmsnorm(g.make_rmsnorm_args(M, D, x=x, residual=res, sum=res, weight=w, q=q.m))
            g.gemm355_block_gated(g.make_block_gated_args(q.m, mats[0].m, mats[1].m, q=h.m))
            g.gemm355_block_gemm(g.make_block_gemm_args(h.m, mats[2].m, y=y))
            assert np.array_equal(res.float().cpu().numpy(), h0)
            ref = block.rmsnorm(h0, w.float().cpu().numpy(), 1e-5)
            check_codes(q, ref, 2.0 ** -19 * np.abs(ref))
            X = block.values(*q.host(), 1)
            G, U, Wd = (block.values(*m.host(), 128) for m in mats)
            gr, ur = X @ G.T, X @ U.T
            ref = block.act(gr, "silu") * ur
            eg, eu = (bound(np.abs(X) @ np.abs(B).T, K) for B in (G, U))
            check_codes(h, ref, 1.13 * eg * (np.abs(ur) + eu) + np.abs(block.act(gr, "silu")) * eu
                        + (6 * np.abs(gr) + 10) * 2.0 ** -23 * np.abs(ref) + 1e-37)
            H = block.values(*h.host(), 1)
            ref, e = H @ Wd.T, bound(np.abs(H) @ np.abs(Wd).T, I) + cut(groups(H, Wd))
            assert np.all(np.abs(y.double().cpu().numpy() - ref) <= e + HALF["bf16"] * (np.abs(ref) + e))
            x.copy_(y)


def test_same_bits_every_time_and_on_other_streams():
    rng = np.random.default_rng(12)
    for M, N, K in ((1, 1000, 4096), (50, 500, 3000), (300, 400, 2000)):
        x, _, _ = random_matrix(rng, M, K, 1)
        w, _, _ = random_matrix(rng, N, K, 128)
        u, _, _ = random_matrix(rng, N, K, 128)
        for splits in (0, 4):
            first, gated = run_gemm(x, w, "f32", splits), run_gated(x, w, u, "silu", "8bit", splits).host()
            streams = [torch.cuda.Stream() for _ in range(3)]
            outs = [torch.empty(M, N, device="cuda") for _ in streams]
            torch.cuda.synchronize()
            for _ in range(3):
                for st, o in zip(streams, outs):
                    g.gemm355_block_gemm(g.make_block_gemm_args(x.m, w.m, y=o, out=g.SRC_F32, splits=splits), stream=st)
            torch.cuda.synchronize()
            assert all(torch.equal(o, first) for o in outs)
            again = run_gated(x, w, u, "silu", "8bit", splits).host()
            assert all(np.array_equal(a, b) for a, b in zip(again, gated))


def test_captured_layer():
    """The chain captured once and replayed over other inputs gives what the calls
    give; scratch in a capture has to be the caller's."""
    rng = np.random.default_rng(13)
    for M in (1, 20, 150):
        D, I = 512, 768
        gate, up = (random_matrix(rng, I, D, 128)[0] for _ in range(2))
        down, _, _ = random_matrix(rng, D, I, 128)
        x = torch.randn(M, D, device="cuda").bfloat16()
        q, h = empty(M, D), empty(M, I)
        y = torch.empty(M, D, dtype=torch.bfloat16, device="cuda")
        norm = g.make_rmsnorm_args(M, D, x=x, q=q.m)
        ga, ge = (lambda **k: g.make_block_gated_args(q.m, gate.m, up.m, q=h.m, splits=2, **k)), \
                 (lambda **k: g.make_block_gemm_args(h.m, down.m, y=y, splits=2, **k))
        n1, n2 = g.gemm355_block_gated_workspace(ga()), g.gemm355_block_gemm_workspace(ge())
        assert n1 > 0 and n2 > 0
        w1, w2 = (torch.empty(n, dtype=torch.uint8, device="cuda") for n in (n1, n2))
        a1, a2 = ga(workspace=w1, workspace_bytes=n1), ge(workspace=w2, workspace_bytes=n2)

        def layer():
            g.gemm355_rmsnorm(norm)
            g.gemm355_block_gated(a1)
            g.gemm355_block_gemm(a2)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            layer()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            layer()
            for call, args in ((g.gemm355_block_gated, ga()), (g.gemm355_block_gemm, ge())):
                with pytest.raises(g.Gemm355Error) as e:
                    call(args)
                assert e.value.status == g.ENOMEM
        for _ in range(4):
            x.copy_(torch.randn(M, D, device="cuda"))
            graph.replay()
            torch.cuda.synchronize()
            got, codes = y.clone(), h.codes.clone()
            layer()
            torch.cuda.synchronize()
            assert torch.equal(got, y) and torch.equal(codes, h.codes)
