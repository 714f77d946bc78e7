"""GPU tests of the serving operators' forms for larger matrices, longer
sequences and more workgroups than compute units, and of ends of their ranges.
Bounds are those of the files whose helpers this one takes: whole numbers and
powers of two are compared bit for bit, attention by its rounding bound.
"""
import numpy as np
import pytest
import torch

from dense_tiled_gemm_fp8_amd import gemm355 as g
from oracle import w4
from tests.gpu_helpers import say
from tests.test_gpu_kvcache import Case, attend, run_append, verify
from tests.test_gpu_w4 import FORMS, dev, matrix, product, random_matrix

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,group,zeros", FORMS)
@pytest.mark.parametrize("N,K", [(8200, 384), (16400, 256), (48, 8320), (16, 16512)])
def test_w4_gemm_many_rows_and_long_rows(fmt, group, zeros, N, K):
    """Sums stay under 2^24 times the smallest scale: |x| <= 4, |u - z| <= 15,
    scales of 1/2 to 2, K <= 16512: 4 * 15 * 4 * 16512 < 2^22 halves."""
    rng = np.random.default_rng(N + K)
    codes, scales, z = random_matrix(rng, N, K, fmt, group, zeros)
    scales = rng.integers(126, 129, scales.shape).astype(np.uint8) if fmt == "mxfp4" else \
        np.exp2(rng.integers(-1, 2, scales.shape)).astype(np.float32)
    m, keep = matrix(codes, scales, z, fmt, group)
    x = torch.from_numpy(rng.integers(-4, 5, (70, K)).astype(np.float32)).to(torch.bfloat16)
    ref = x.double().numpy() @ w4.values(codes, scales, z, fmt, group).T
    xd = x.cuda()
    for M in (1, 4, 5, 16, 17, 32, 33, 70):
        say("w4_gemm large", fmt, group, zeros, M, N, K)
        y = product(M, xd, m, N, "f32")
        assert np.array_equal(y.double().cpu().numpy(), ref[:M]), M
    del keep


def test_w4_gemm_mxfp4_codes_behind_k_are_not_read_as_infinities():
    """Codes past K of -6 with scales of 2^126 and 2^127, where the row's own
    are small: 0.5 * 2^126 and 2^127."""
    for K in (1, 20, 33, 100, 200):
        codes = np.ones((5, K), np.uint8)
        scales = np.full((5, -(-K // 32)), 253, np.uint8)
        scales[3] = 254
        m, keep = matrix(codes, scales, None, "mxfp4", 32, fill=15)
        x = torch.zeros(2, K, dtype=torch.bfloat16)
        x[0, K - 1], x[1, 0] = 1.0, 0.5
        y = product(2, x.cuda(), m, 5, "f32").double().cpu().numpy()
        assert np.array_equal(y, x.double().numpy() @ w4.values(codes, scales, None, "mxfp4", 32).T), K
        del keep


@pytest.mark.parametrize("K", (32, 128))
def test_w4_mxfp4_smallest_scale(K):
    """Scale byte 0 is 2^-127: values are subnormal in bf16 and fp32."""
    codes = np.tile(np.arange(16, dtype=np.uint8), (4, K // 16))
    scales = np.zeros((4, K // 32), np.uint8)
    m, keep = matrix(codes, scales, None, "mxfp4", 32)
    back = torch.empty(4, K, device="cuda")
    g.gemm355_w4_dequantize(m, back, dst=g.SRC_F32)
    want = w4.values(codes, scales, None, "mxfp4", 32)
    assert np.array_equal(back.double().cpu().numpy(), want)
    x = torch.zeros(3, K, dtype=torch.bfloat16)
    x[0, 2], x[1, 7], x[2, K - 1] = 2.0 ** 100, -2.0 ** 90, 2.0 ** 120
    y = product(3, x.cuda(), m, 4, "f32").double().cpu().numpy()
    assert np.array_equal(y, x.double().numpy() @ want.T)
    del keep


@pytest.mark.parametrize("fmt,group,zeros", FORMS)
@pytest.mark.parametrize("src", (torch.float32, torch.bfloat16))
def test_w4_quantize_large_as_in_pieces(fmt, group, zeros, src):
    """More than 2^20 octets, against the same rows in pieces of 100 (whose bits
    are compared with the oracle elsewhere) and the oracle's last rows."""
    N, K = 2100, 4100
    gen = torch.Generator().manual_seed(group)
    w = (torch.randn(N, K, generator=gen) * torch.exp(torch.randn(N, 1, generator=gen))).to(src).cuda()
    ng, width = -(-K // group), -(-K // 32) * 32
    kind = g.SRC_F32 if src == torch.float32 else g.SRC_BF16

    def buffers():
        return (torch.full((N, width // 2), 0xAA, dtype=torch.uint8, device="cuda"),
                torch.zeros((N, ng), dtype=torch.uint8 if fmt == "mxfp4" else torch.bfloat16, device="cuda"),
                torch.zeros((N, ng), dtype=torch.uint8, device="cuda") if zeros else None)

    def mat(b, lo, hi):
        return g.make_w4_matrix(hi - lo, K, b[0][lo:], b[1][lo:], b[2][lo:] if zeros else None,
                                fmt=g.W4_MXFP4 if fmt == "mxfp4" else g.W4_INT, group=group)
    say("w4_quantize large", fmt, group, zeros, src)
    one, many = buffers(), buffers()
    g.gemm355_w4_quantize(w, mat(one, 0, N), src=kind)
    for lo in range(0, N, 100):
        g.gemm355_w4_quantize(w[lo:], mat(many, lo, lo + 100), src=kind)
    torch.cuda.synchronize()
    assert torch.equal(one[0], many[0]) and torch.equal(one[1], many[1]) and (not zeros or torch.equal(one[2], many[2]))
    codes, scales, z = w4.quantize(w[N - 3:].float().cpu().numpy(), fmt, group, zeros)
    assert np.array_equal(one[0][N - 3:, :(K + 1) // 2].cpu().numpy(), w4.pack(codes, width)[:, :(K + 1) // 2])
    assert np.array_equal(one[1][N - 3:].float().cpu().numpy(), scales.astype(np.float32))
    back, part = (torch.full((N, K + 4), 3.0, dtype=src, device="cuda") for _ in range(2))
    g.gemm355_w4_dequantize(mat(one, 0, N), back, dst=kind, ld=K + 4)
    for lo in range(0, N, 100):
        g.gemm355_w4_dequantize(mat(one, lo, lo + 100), part[lo:], dst=kind, ld=K + 4)
    torch.cuda.synchronize()
    assert torch.equal(back, part)
    ref = torch.from_numpy(w4.values(codes, scales, z, fmt, group).astype(np.float32)).to(src)
    assert torch.equal(back[N - 3:, :K].cpu(), ref) and torch.all(back[:, K:] == 3.0)


@pytest.mark.parametrize("D,page", [(64, 32), (128, 128), (256, 64)])
def test_attention_more_parts_than_one_pass_joins(D, page):
    c = Case(300 + D, [30000, 17000, 900], [2, 1, 1], 2, 1, D, page)
    q = c.rows(2, 2.0)
    for splits in (65, 100):
        say("attention parts", D, splits)
        o, ls = attend(c, q, splits=splits)
        verify(c, q, o, ls)


@pytest.mark.parametrize("D,page,Hq", [(64, 16, 8), (128, 16, 8), (128, 64, 32), (256, 32, 8)])
def test_attention_more_workgroups_than_units(D, page, Hq):
    r = np.random.default_rng(D)
    lens = [int(n) for n in r.integers(0, 300, 40)]
    c = Case(310 + D, lens, [1] * 40, Hq, 8, D, page)
    q = c.rows(Hq, 2.0)
    say("attention workgroups", D, page, Hq)
    for kw in (dict(), dict(window=70, sinks=3)):
        o, ls = attend(c, q, **kw)
        verify(c, q, o, ls, **kw)


@pytest.mark.parametrize("rot", (0, 128, 6))
def test_append_many_tokens_of_a_page(rot):
    """Eight octets a thread: between 65 and 128 new tokens of 128 channels."""
    say("append many", rot)
    c = Case(320, [300, 100, 260, 128], [100, 90, 128, 66], 4, 2, 128, 128)
    run_append(c, rot=rot)


def test_attention_rows_of_nan_and_infinity_stay_alone():
    """Queries that hold a NaN or infinities leave every other row within its
    bound (not its bits: rows of a tile move their references together)."""
    for news, D, splits in (([20, 3], 64, 1), ([1, 1], 128, 0), ([40, 7], 128, 3), ([5, 2], 256, 2)):
        c = Case(330, [700, 90], news, 8, 2, D, 32)
        q = c.rows(8)
        cache = c.upload()
        o, ls = attend(c, q, cache=cache, splits=splits)
        bad = q.clone()
        bad[0, 3, 5] = float("nan")
        bad[c.tokens - 1, 6] = float("inf")
        o2, ls2 = attend(c, bad, cache=cache, splits=splits)
        assert torch.isnan(o2[0, 3]).all() and torch.isnan(ls2[0, 3])
        for r, h in ((0, 3), (c.tokens - 1, 6)):
            o2[r, h], ls2[r, h] = o[r, h], ls[r, h]
        verify(c, q, o2, ls2)


def test_sequences_that_share_pages_they_read():
    c = Case(340, [200, 200, 150], [1, 1, 1], 4, 2, 64, 32)
    c.table[1, :6] = c.table[0, :6]                  # 192 tokens in common, the last page of its own
    q = c.rows(4, 2.0)
    run_append(c)
    o, ls = attend(c, q)
    verify(c, q, o, ls)


def test_steps_without_a_token():
    """max_len 0, no page table: rows that see nothing, nothing appended."""
    dims = dict(pages=2, heads=2, head_dim=64, page=16, table=None, batch=3, max_len=0, tokens=3, max_new=1)
    k = torch.full((2, 2, 16, 64), 5, dtype=torch.uint8, device="cuda")
    v, ks = k.clone(), dev(np.full((2, 2), 120, np.uint8))
    vs, lens = ks.clone(), torch.tensor([0, 7, -3], dtype=torch.int32, device="cuda")
    cache = g.make_kv_cache(k, v, ks, vs, lens=lens, **dims)
    x = torch.ones(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    out, o = torch.full_like(x, 9.0), torch.full_like(x, 9.0)
    lse = torch.full((3, 2), 9.0, device="cuda")
    g.gemm355_kv_append(g.make_kv_append_args(cache, x, x, q=x, q_out=out, q_heads=2))
    g.gemm355_attention(g.make_attention_args(cache, x, o, q_heads=2, lse=lse))
    torch.cuda.synchronize()
    assert torch.all(out == 9.0) and torch.all(o == 0) and torch.all(lse == float("-inf"))
    assert torch.all(k == 5) and torch.all(v == 5) and torch.all(ks == 120) and torch.all(vs == 120)


@pytest.mark.parametrize("window,sinks,splits", [(0, 0, 0), (90, 5, 0), (0, 0, 3), (400, 70, 2)])
@pytest.mark.parametrize("D,page,new", [(64, 16, 80), (128, 64, 80), (256, 32, 140), (64, 128, 262), (128, 16, 262)])
def test_attention_prompt_chunks_of_many_rows(D, page, new, window, sinks, splits):
    """More rows than 16 for each compute unit, at both counts of workgroups;
    lengths that end inside a chunk, rows that the shorter sequence lacks."""
    c = Case(350 + D + new, [700, 301], [new, new - 7], 32, 8, D, page, extra_rows=3)
    c.table[0, 2] = -1                               # a page that nobody holds
    q = c.rows(32, 2.0)
    say("attention prompts", D, page, new, window, sinks, splits)
    kw = dict(window=window, sinks=sinks)
    o, ls = attend(c, q, splits=splits, **kw)
    verify(c, q, o, ls, **kw)
    o2, _ = attend(c, q, splits=splits, **kw)
    assert torch.equal(o.view(torch.int16), o2.view(torch.int16))


@pytest.mark.parametrize("D", (128, 256))
def test_attention_more_workgroups_than_units_of_long_caches(D):
    """A step whose sequences may hold more than 4096 tokens; one does."""
    r = np.random.default_rng(D)
    lens = [4500] + [int(n) for n in r.integers(0, 200, 39)]
    c = Case(400 + D, lens, [1] * 40, 8, 8, D, 64, max_len=5000)
    q = c.rows(8, 2.0)
    o, ls = attend(c, q)
    verify(c, q, o, ls)


@pytest.mark.parametrize("fmt,group,zeros", FORMS)
@pytest.mark.parametrize("N,K", [(8200, 389), (16401, 257), (4097, 1001), (5000, 130), (48, 8321), (33, 16383), (17, 100), (3, 9), (1, 8), (19, 8)])
def test_w4_gemm_any_k_and_row_starts(fmt, group, zeros, N, K):
    """Every count of rows with K of any remainder, rows of x at odd starts and
    strides, NaN behind each and codes behind K; exact, as K <= 16512 above."""
    rng = np.random.default_rng(N + K)
    codes, scales, z = random_matrix(rng, N, K, fmt, group, zeros)
    scales = rng.integers(126, 129, scales.shape).astype(np.uint8) if fmt == "mxfp4" else \
        np.exp2(rng.integers(-1, 2, scales.shape)).astype(np.float32)
    m, keep = matrix(codes, scales, z, fmt, group, fill=15)
    for ldx, off in ((K, 0), (K + 3, 1), (K + 8 - K % 8, 4)):
        flat = torch.full((off + 70 * ldx,), float("nan"), dtype=torch.bfloat16)
        rows = flat[off:].reshape(70, ldx)
        rows[:, :K] = torch.from_numpy(rng.integers(-4, 5, (70, K)).astype(np.float32)).to(torch.bfloat16)
        ref = rows[:, :K].double().numpy() @ w4.values(codes, scales, z, fmt, group).T
        buf = flat.cuda()
        for M in (1, 4, 5, 16, 17, 32, 33, 70):
            say("w4_gemm any", fmt, group, zeros, M, N, K, ldx, off)
            y = product(M, buf.data_ptr() + 2 * off, m, N, "f32", ldx=ldx)
            assert np.array_equal(y.double().cpu().numpy(), ref[:M]), (M, ldx, off)
    del keep


@pytest.mark.parametrize("fmt,group,zeros", FORMS)
def test_w4_gemm_scales_of_nan_stay_in_their_rows(fmt, group, zeros):
    """A last chunk reads more scales than its row has: the next row's, here
    NaN, have no effect.  Rows that begin at every remainder of a dword."""
    rng = np.random.default_rng(11)
    for K in (100, 137, 300, 451):
        codes, scales, z = random_matrix(rng, 40, K, fmt, group, zeros)
        scales = np.full(scales.shape, 127, np.uint8) if fmt == "mxfp4" else np.ones(scales.shape, np.float32)
        clean = [n for n in range(40) if n % 3]
        ref_scales = scales.copy()
        scales[::3] = 255 if fmt == "mxfp4" else np.nan
        m, keep = matrix(codes, scales, z, fmt, group, fill=7)
        x = torch.from_numpy(rng.integers(-4, 5, (3, K)).astype(np.float32)).to(torch.bfloat16)
        y = product(3, x.cuda(), m, 40, "f32").double().cpu().numpy()
        ref = x.double().numpy() @ w4.values(codes, ref_scales, z, fmt, group).T
        assert np.array_equal(y[:, clean], ref[:, clean]) and np.all(np.isnan(y[:, ::3])), K
        del keep


def test_w4_matrix_of_more_than_4_gib_and_2_31_octets():
    """Codes, and the values they stand for, past 32-bit offsets: the last rows
    of a matrix of 2^17 x 2^17 elements and some."""
    N, K = (1 << 17) + 8, 1 << 17
    c = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda")
    s = torch.ones(N, K // 128, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator().manual_seed(1)
    for rows in (slice(0, 3), slice(N - 12, N)):
        c[rows] = torch.randint(0, 256, (c[rows].shape[0], K // 2), generator=gen, dtype=torch.uint8).cuda()
        s[rows] = 0.5
    m = g.make_w4_matrix(N, K, c, s, None, group=128)
    x = torch.zeros(1, K, dtype=torch.bfloat16)
    x[0, ::1025] = 1.0
    y = product(1, x.cuda(), m, N, "f32")
    dense = torch.empty(N, K, dtype=torch.bfloat16, device="cuda")
    g.gemm355_w4_dequantize(m, dense)
    torch.cuda.synchronize()
    for rows in (slice(0, 3), slice(N - 12, N)):
        codes = c[rows].cpu().numpy()
        u = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], K)
        v = (u.astype(np.float32) - 8) * 0.5
        assert np.array_equal(dense[rows].float().cpu().numpy(), v)
        assert np.array_equal(y[0, rows].double().cpu().numpy(), v.astype(np.float64) @ x[0].double().numpy())
    assert torch.all(dense[N // 2] == -8) and torch.all(y[0, N // 2] == -8 * x.double().sum().item())
    c2, s2 = torch.full_like(c, 0x55), torch.zeros_like(s)
    g.gemm355_w4_quantize(dense, g.make_w4_matrix(N, K, c2, s2, None, group=128))
    torch.cuda.synchronize()
    tail = dense[N - 12:].float().cpu().numpy()
    codes, scales, _ = w4.quantize(tail[:, :2048], "int", 128)
    assert np.array_equal(c2[N - 12:, :1024].cpu().numpy(), w4.pack(codes, 2048))
    assert np.array_equal(s2[N - 12:, :16].float().cpu().numpy(), scales)


@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 5)])
@pytest.mark.parametrize("D,page", [(64, 32), (128, 16)])
def test_attention_prompt_chunks_of_most_rows(D, page, window, sinks):
    """More than three workgroups of 32 rows for each compute unit."""
    c = Case(420 + D, [330, 262], [262, 255], 64, 8, D, page)
    q = c.rows(64, 2.0)
    o, ls = attend(c, q, window=window, sinks=sinks)
    verify(c, q, o, ls, window=window, sinks=sinks)
