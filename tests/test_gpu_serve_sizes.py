"""The serving operators at the largest sizes that the header allows, by results
that need no oracle over all of them: whole numbers summed exactly, one visible
token, means of a window, the same step in pieces; and calls from several host
threads at once.
"""
import threading

import pytest
import torch

from dense_tiled_gemm_fp8_amd import gemm355 as g
from tests.gpu_helpers import say
from tests.test_gpu_kvcache import Case, attend

pytestmark = pytest.mark.gpu


def packed(N, K, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (N, -(-K // 32) * 16), generator=gen, device="cuda", dtype=torch.uint8)
    return codes, torch.full((N, -(-K // 128)), 0.5, dtype=torch.bfloat16, device="cuda")


@pytest.mark.parametrize("M,N,K", [(1, 1 << 26, 8), (1 << 19, 3, 40), (1 << 19, 1, 9)])
def test_w4_gemm_most_rows(M, N, K):
    say("w4_gemm most rows", M, N, K)
    codes, scales = packed(N, K, 1)
    x = torch.randint(-4, 5, (M, K), device="cuda").to(torch.bfloat16)
    y = torch.full((M, N), 9.0, device="cuda")
    g.gemm355_w4_gemm(M, x, g.make_w4_matrix(N, K, codes, scales, group=128), y, out=g.SRC_F32)
    want = torch.zeros_like(y)
    for k in range(K):
        w = (codes[:, k // 2] >> (4 * (k % 2)) & 15).float() * 0.5 - 4.0
        want += x[:, k].float()[:, None] * w
    assert torch.equal(y, want)


@pytest.mark.parametrize("K", (1 << 23, (1 << 23) - 5))
def test_w4_gemm_longest_rows(K):
    """1024 elements of x are not zero."""
    say("w4_gemm longest rows", K)
    M, N = 2, 17
    codes, scales = packed(N, K, 2)
    at = torch.randint(0, K, (1024,), device="cuda").unique()
    at[-1] = K - 1
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    x[:, at] = torch.randint(-4, 5, (M, at.numel()), device="cuda").to(torch.bfloat16)
    y = torch.empty(M, N, device="cuda")
    g.gemm355_w4_gemm(M, x, g.make_w4_matrix(N, K, codes, scales, group=128), y, out=g.SRC_F32)
    u = codes[:, at // 2] >> (4 * (at % 2)).to(torch.uint8) & 15
    assert torch.equal(y.double().cpu(), x[:, at].double().cpu() @ (u.double().cpu() * 0.5 - 4.0).T)


@pytest.mark.parametrize("batch,heads", [(65528, 1), (8191, 8)])
def test_most_sequences(batch, heads):
    """One token each, appended and seen alone: attention gives its value back."""
    say("most sequences", batch, heads)
    D, page = 64, 16
    k = torch.full((batch, heads, page, D), 0x7F, dtype=torch.uint8, device="cuda")
    v = torch.full((batch, heads, D, page), 0x7F, dtype=torch.uint8, device="cuda")
    ks, vs = (torch.full((batch, heads), 255, dtype=torch.uint8, device="cuda") for _ in range(2))
    table = torch.randperm(batch, device="cuda").to(torch.int32)
    lens = torch.ones(batch, dtype=torch.int32, device="cuda")
    cache = g.make_kv_cache(k, v, ks, vs, pages=batch, heads=heads, head_dim=D, page=page, table=table, lens=lens, batch=batch,
                            max_len=1, tokens=batch, max_new=1)
    x = torch.randint(-15, 16, (batch, heads, D), device="cuda").to(torch.bfloat16)
    x[..., 0] = 15.0                                         # 15 <= 448 * 2^-4: the scale of every block
    g.gemm355_kv_append(g.make_kv_append_args(cache, x, x))
    o, lse = torch.full_like(x, 9.0), torch.empty(batch, heads, device="cuda")
    g.gemm355_attention(g.make_attention_args(cache, x, o, q_heads=heads, lse=lse))
    assert torch.equal(o, x) and torch.isfinite(lse).all()
    assert torch.all(ks == 127 - 4) and torch.all(vs == 127 - 4)


def test_attention_most_rows_and_append_of_as_many():
    """A prompt of 16 * 65535 tokens with a window of 16 and q = 0: means of 16
    whole numbers, exact.  Its append, against appends of 4096 tokens."""
    T, D, page = 16 * 65535, 64, 128
    pages = -(-T // page)
    say("most rows", T)
    bufs = []
    x = torch.randint(-15, 16, (T, 1, D), device="cuda").to(torch.bfloat16)
    x[..., 0] = 15.0
    for piece in (T, 4096):
        k = torch.zeros(pages, 1, page, D, dtype=torch.uint8, device="cuda")
        v = torch.zeros(pages, 1, D, page, dtype=torch.uint8, device="cuda")
        ks, vs = (torch.zeros(pages, 1, dtype=torch.uint8, device="cuda") for _ in range(2))
        table = torch.arange(pages, dtype=torch.int32, device="cuda")
        for lo in range(0, T, piece):
            n = min(piece, T - lo)
            lens = torch.tensor([lo + n], dtype=torch.int32, device="cuda")
            cache = g.make_kv_cache(k, v, ks, vs, pages=pages, heads=1, head_dim=D, page=page, table=table, lens=lens, batch=1,
                                    max_len=T, tokens=n, max_new=n)
            g.gemm355_kv_append(g.make_kv_append_args(cache, x[lo:], x[lo:]))
            torch.cuda.synchronize()
        bufs.append((k, v, ks, vs))
    assert all(torch.equal(a, b) for a, b in zip(*bufs))
    k, v, ks, vs = bufs[0]
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    cache = g.make_kv_cache(k, v, ks, vs, pages=pages, heads=1, head_dim=D, page=page, table=table, lens=lens, batch=1, max_len=T,
                            tokens=T, max_new=T)
    q, o = torch.zeros_like(x), torch.full_like(x, 9.0)
    g.gemm355_attention(g.make_attention_args(cache, q, o, q_heads=1, window=16))
    sums = torch.cumsum(x[:, 0].double(), 0)
    sums[16:] = sums[16:] - sums[:-16].clone()
    assert torch.equal(o[16:, 0], (sums[16:] / 16).to(torch.bfloat16))
    near = sums[:16] / torch.arange(1, 17, device="cuda")[:, None]
    assert torch.all((o[:16, 0].double() - near).abs() <= 2.0 ** -8 * near.abs() * (1 + 2.0 ** -12))


def test_attention_from_several_threads():
    """Four host threads, a stream and library scratch of its own each."""
    c = Case(800, [3000, 1500], [1, 1], 4, 2, 64, 32)
    q = c.rows(4, 2.0)
    cache = c.upload()
    want, wl = attend(c, q, splits=6, cache=cache)
    qd = q.cuda()
    torch.cuda.synchronize()
    wrong, errors = [], []

    def work():
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for splits in (6, 2, 6, 3, 6):
                    o, ls = torch.zeros_like(want), torch.zeros_like(wl)
                    g.gemm355_attention(g.make_attention_args(cache, qd, o, q_heads=4, lse=ls, splits=splits))
                    stream.synchronize()
                    if splits == 6 and not (torch.equal(o, want) and torch.equal(ls, wl)):
                        wrong.append(splits)
        except Exception as e:                               # noqa: BLE001  (seen by the thread that joins)
            errors.append(e)
    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and not wrong


@pytest.mark.parametrize("fmt", ("int", "mxfp4"))
def test_w4_quantize_and_dequantize_captured(fmt):
    """Replays follow new weights and equal the eager result each time."""
    N, K = 300, 1000
    mx = fmt == "mxfp4"
    ng = -(-K // 32)
    buf = [(torch.zeros(N, -(-K // 32) * 16, dtype=torch.uint8, device="cuda"),
            torch.zeros(N, ng, dtype=torch.uint8 if mx else torch.bfloat16, device="cuda"),
            None if mx else torch.zeros(N, ng, dtype=torch.uint8, device="cuda")) for _ in range(2)]
    m = [g.make_w4_matrix(N, K, *b, fmt=g.W4_MXFP4 if mx else g.W4_INT, group=32) for b in buf]
    w = torch.randn(N, K, device="cuda").to(torch.bfloat16)
    back = [torch.zeros(N, K, device="cuda") for _ in range(2)]

    def step(i):
        g.gemm355_w4_quantize(w, m[i])
        g.gemm355_w4_dequantize(m[i], back[i], dst=g.SRC_F32)
    step(0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(0)
    for _ in range(4):
        w.copy_(torch.randn(N, K, device="cuda"))
        step(1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(back[0], back[1]) and all(a is None or torch.equal(a, b) for a, b in zip(*buf))
