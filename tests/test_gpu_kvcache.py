"""GPU parity of the append to the paged 8-bit cache and of attention over it
with the oracle (oracle/kvcache.py).

Append: codes and scales bit for bit.  Attention, |o - ref| bounded by what is
rounded: the softmax weights to bf16 (2^-8 of each, on W = sum of weights times
|v|), the output (2^-8), scores of D products added in 32 bits, each off by at
most 2^-23 of S = sum |scale q k| for D + 8 additions and the exponential's
argument (which moves a weight by as much, relatively, twice: in the sum and in
the total), the exponential itself (2^-21 relative to each weight with its
argument's rounding), and the sums over n tokens (n 2^-23).
"""
import math

import numpy as np
import pytest
import torch

from dense_tiled_gemm_fp8_amd import gemm355 as g
from oracle import kvcache as ok
from oracle import w4
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu


class Case:
    """A cache with random codes in the tokens held, NaN codes everywhere else,
    and a page table that names nothing valid behind a sequence's last page."""

    def __init__(self, seed, lens, news, Hq, H, D, page, uniform=False, spare=3, extra_rows=0, max_len=None):
        r = self.rng = np.random.default_rng(seed)
        self.lens, self.news, self.Hq, self.H, self.D, self.page = list(lens), list(news), Hq, H, D, page
        B = len(lens)
        self.max_len = max(list(lens) + [1]) if max_len is None else max_len
        cols = -(-self.max_len // page)
        need = [-(-n // page) for n in lens]
        self.pages = sum(need) + spare
        ids = list(r.permutation(self.pages))
        self.table = np.full((B, cols), -7, np.int32)
        self.table[:, 1::2] = 1 << 30
        self.k = np.full((self.pages, H, page, D), 0x7F, np.uint8)
        self.v = np.full((self.pages, H, D, page), 0xFF, np.uint8)
        self.ks = r.integers(118, 122, (self.pages, H)).astype(np.uint8)
        self.vs = r.integers(118, 122, (self.pages, H)).astype(np.uint8)
        for b in range(B):
            for j in range(need[b]):
                at = self.table[b, j] = ids.pop()
                n = min(page, lens[b] - j * page)
                self.k[at, :, :n] = ok.encode(r.standard_normal((H, n, D)) * 100)
                self.v[at, :, :, :n] = ok.encode(r.standard_normal((H, D, n)) * 100)
        self.start = None if uniform else [0] + list(np.cumsum(news))
        self.tokens = sum(news) + extra_rows
        self.max_new = max(list(news) + [1])

    def step(self):
        return ok.Step(self.lens, self.start, self.tokens, self.max_new, self.max_len, self.table, self.page, self.pages)

    def upload(self):
        d = lambda a: torch.from_numpy(np.ascontiguousarray(a).copy()).cuda()  # noqa: E731
        self.d = {n: d(getattr(self, n)) for n in ("k", "v", "ks", "vs", "table")}
        self.d["lens"] = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.d["start"] = None if self.start is None else torch.tensor(self.start, dtype=torch.int32, device="cuda")
        t = self.d
        return g.make_kv_cache(t["k"], t["v"], t["ks"], t["vs"], pages=self.pages, heads=self.H, head_dim=self.D, page=self.page,
                               table=t["table"], lens=t["lens"], batch=len(self.lens), max_len=self.max_len, q_start=t["start"],
                               tokens=self.tokens, max_new=self.max_new)

    def rows(self, heads, scale=1.0):
        return (scale * torch.from_numpy(self.rng.standard_normal((self.tokens, heads, self.D)).astype(np.float32))).to(torch.bfloat16)


def attend(c, q, scale=0.0, window=0, sinks=0, splits=0, lse=True, cache=None, workspace=None, stream=None):
    cache = c.upload() if cache is None else cache
    o = torch.full((c.tokens, c.Hq, c.D), 9.0, dtype=torch.bfloat16, device="cuda")
    ls = torch.full((c.tokens, c.Hq), 9.0, device="cuda") if lse else None
    qd = q.cuda()
    a = g.make_attention_args(cache, qd, o, q_heads=c.Hq, lse=ls, scale=scale, window=window, sinks=sinks, splits=splits,
                              workspace=workspace, workspace_bytes=0 if workspace is None else workspace.numel())
    g.gemm355_attention(a, stream=stream)
    torch.cuda.synchronize()
    return o, ls


def verify(c, q, o, ls, scale=0.0, window=0, sinks=0):
    sc = scale or 1.0 / math.sqrt(c.D)
    ref, rl, W, S = ok.attention(c.step(), c.k, c.v, c.ks, c.vs, q.double().numpy(), sc, window, sinks)
    got, gl = o.double().cpu().numpy(), None if ls is None else ls.double().cpu().numpy()
    owned = ~np.isnan(rl)
    assert np.all(got[~owned] == 9.0) and (gl is None or np.all(gl[~owned] == 9.0))
    n = max(c.lens + [1])
    ds = (c.D + 8) * 2.0 ** -23 * S[..., None]
    tol = (2.0 ** -8 + 2 * ds + 2.0 ** -20 + n * 2.0 ** -23) * W + 2.0 ** -8 * np.abs(ref)
    err = np.abs(got - ref)[owned]
    assert np.all(err <= tol[owned] * (1 + 2.0 ** -8)), "worst %.3g of the tolerance" % float((err / np.maximum(tol[owned], 1e-300)).max())
    if gl is not None:
        fin = owned & np.isfinite(rl)
        assert np.array_equal(gl[owned & ~fin], rl[owned & ~fin])
        lt = ds[..., 0] + (n + 16) * 2.0 ** -23 + 2.0 ** -22 * np.abs(rl)
        assert np.all(np.abs(gl[fin] - rl[fin]) <= lt[fin])


SIZES = [
    # lens, new rows, Hq, H, D, page
    ([1], [1], 1, 1, 64, 16),
    ([15, 16, 17], [1, 1, 1], 8, 8, 64, 16),
    ([63, 64, 65, 0, 1], [1, 1, 1, 1, 1], 4, 2, 128, 16),
    ([700, 3, 129], [1, 1, 1], 10, 2, 128, 32),
    ([500, 40], [4, 40], 6, 2, 64, 64),
    ([300, 0, 77], [33, 0, 7], 4, 4, 128, 128),
    ([90, 5], [3, 2], 8, 1, 256, 32),
    ([70, 2, 0], [7, 5, 3], 5, 1, 64, 16),        # more rows than tokens: rows that see nothing
    ([2100], [2], 16, 2, 128, 64),
    ([260, 257], [130, 1], 2, 1, 256, 128),
]


@pytest.mark.parametrize("splits", (0, 1, 3))
@pytest.mark.parametrize("i", range(len(SIZES)))
def test_attention_sizes(i, splits):
    lens, news, Hq, H, D, page = SIZES[i]
    say("attention", SIZES[i], splits)
    c = Case(i, lens, news, Hq, H, D, page, extra_rows=2)
    q = c.rows(Hq, 2.0)
    o, ls = attend(c, q, splits=splits)
    verify(c, q, o, ls)
    o2, ls2 = attend(c, q, splits=splits)
    assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(ls, ls2)


@pytest.mark.parametrize("splits", (0, 2))
@pytest.mark.parametrize("window,sinks", [(1, 0), (7, 3), (64, 0), (64, 4), (100, 70), (130, 1), (200, 500), (10 ** 12, 4), (33, 64)])
def test_attention_window_and_sinks(window, sinks, splits):
    say("attention window", window, sinks, splits)
    for i, (lens, news, Hq, H, D, page) in enumerate((([600, 65, 1], [1, 1, 1], 4, 2, 64, 32), ([520, 100], [90, 20], 6, 2, 128, 16))):
        c = Case(50 + i, lens, news, Hq, H, D, page)
        q = c.rows(Hq, 2.0)
        o, ls = attend(c, q, window=window, sinks=sinks, splits=splits)
        verify(c, q, o, ls, window=window, sinks=sinks)


def test_attention_scale_no_lse_and_uniform_rows():
    c = Case(60, [130, 70, 9], [2, 2, 2], 4, 2, 64, 16, uniform=True)
    q = c.rows(4)
    o, _ = attend(c, q, scale=0.3, lse=False)
    verify(c, q, o, None, scale=0.3)


def test_attention_large_scores():
    """Scores far from zero on both sides: the running maximum carries them."""
    c = Case(61, [900, 300], [1, 5], 4, 2, 128, 32)
    q = c.rows(4, 60.0)
    for splits in (1, 4):
        o, ls = attend(c, q, splits=splits)
        verify(c, q, o, ls)


def test_attention_bad_pages_and_indices():
    """Page ids outside the cache hide their tokens; lengths and rows out of
    range read as the nearest allowed."""
    c = Case(62, [200, 150, 64], [3, 2, 1], 4, 2, 64, 16)
    c.table[0, 2], c.table[0, 12], c.table[1, 0], c.table[2, :] = -1, c.pages, 1 << 30, -(1 << 31)
    q = c.rows(4, 2.0)
    for splits in (1, 3):
        o, ls = attend(c, q, splits=splits)
        verify(c, q, o, ls)
    c = Case(63, [200, 150, 64], [3, 2, 1], 4, 2, 64, 16)
    c.lens, c.start = [10 ** 9, -5, 64], [-4, 3, 3, 10 ** 9]
    q = c.rows(4, 2.0)
    o, ls = attend(c, q)
    verify(c, q, o, ls)


def test_attention_hidden_nans_stay_hidden():
    """A NaN in a key or value reaches the rows that see it and no other."""
    for new, splits in ((20, 1), (20, 2), (1, 1)):
        c = Case(64, [300, 70], [new, new], 4, 2, 64, 32)
        for t in (295, 299, 40):
            c.v[c.table[0, t // 32], 1, 5, t % 32] = 0x7F
        c.k[c.table[1, 2], 0, 68 % 32, 3] = 0xFF
        q = c.rows(4, 1.0)
        o, ls = attend(c, q, window=100, splits=splits)
        ref, rl, _, _ = ok.attention(c.step(), c.k, c.v, c.ks, c.vs, q.double().numpy(), 0.125, 100, 0)
        got = o.double().cpu().numpy()
        sees = np.isnan(ref)
        assert np.all(np.isnan(got[sees]))
        rows_without = ~sees.any(axis=2)
        assert np.all(np.isfinite(got[rows_without])) and rows_without.any() == (new > 1 or True)
        clean = Case(64, [300, 70], [new, new], 4, 2, 64, 32)
        oc, _ = attend(clean, q, window=100, splits=splits)
        same = torch.from_numpy(rows_without)
        assert torch.equal(o.cpu()[same], oc.cpu()[same])


def test_attention_strides():
    c = Case(65, [100, 30], [3, 2], 4, 2, 64, 16)
    q = c.rows(4, 2.0)
    cache = c.upload()
    wide = torch.full((c.tokens, 3 * 4 * 64 + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + 256] = q.reshape(c.tokens, -1).cuda()
    out = torch.full((c.tokens, 320), 9.0, dtype=torch.bfloat16, device="cuda")
    a = g.make_attention_args(cache, wide.data_ptr() + 16, out, q_heads=4, ldq=wide.shape[1], ldo=320)
    g.gemm355_attention(a)
    torch.cuda.synchronize()
    assert torch.all(out[:, 256:] == 9.0)
    verify(c, q, out[:, :256].reshape(c.tokens, 4, 64), None)


def test_attention_offsets_past_32_bits():
    """A cache of more than 4 GiB, the tokens in its last pages."""
    H, D, page = 2, 128, 128
    pages = (1 << 32) // (H * D * page) + 40
    small = Case(66, [500], [2], 4, H, D, page, spare=0)
    big = {n: torch.empty((pages,) + getattr(small, n).shape[1:], dtype=torch.uint8, device="cuda") for n in ("k", "v", "ks", "vs")}
    ids = [pages - 1, pages - 7, 5, pages - 20]
    for j, at in enumerate(ids):
        src = int(small.table[0, j])
        for n in big:
            big[n][at] = torch.from_numpy(getattr(small, n)[src]).cuda()
    table = torch.tensor([ids], dtype=torch.int32, device="cuda")
    lens = torch.tensor([500], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    cache = g.make_kv_cache(big["k"], big["v"], big["ks"], big["vs"], pages=pages, heads=H, head_dim=D, page=page, table=table,
                            lens=lens, batch=1, max_len=500, q_start=start, tokens=2, max_new=2)
    q = small.rows(4, 2.0)
    xk, xv = small.rows(H), small.rows(H)
    dk, dv = xk.cuda(), xv.cuda()
    g.gemm355_kv_append(g.make_kv_append_args(cache, dk, dv))
    ok.append(small.step(), small.k, small.v, small.ks, small.vs, xk.double().numpy(), xv.double().numpy())
    o, ls = attend(small, q, cache=cache)
    verify(small, q, o, ls)
    for j, at in enumerate(ids):
        src = int(small.table[0, j])
        for n in big:
            assert np.array_equal(big[n][at].cpu().numpy(), getattr(small, n)[src]), (n, j)


def test_attention_workspace_streams_and_graph():
    c = Case(67, [3000, 1500], [1, 1], 4, 2, 64, 32)
    q = c.rows(4, 2.0)
    cache = c.upload()
    want, wl = attend(c, q, splits=6, cache=cache)
    verify(c, q, want, wl)
    a = g.make_attention_args(cache, q.cuda(), want, q_heads=4, splits=6)
    need = g.gemm355_attention_workspace(a)
    assert need > 0
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    got, gl = attend(c, q, splits=6, cache=cache, workspace=ws)
    assert torch.equal(got, want) and torch.equal(gl, wl)
    # two streams at once, library scratch each
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [torch.zeros_like(want) for _ in range(2)]
    qd = q.cuda()
    torch.cuda.synchronize()
    for _ in range(10):
        for s, o in zip((s1, s2), outs):
            g.gemm355_attention(g.make_attention_args(cache, qd, o, q_heads=4, splits=6), stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    # captured: library scratch is refused, a workspace of the caller's replays
    o = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st = torch.cuda.current_stream().cuda_stream
        with pytest.raises(g.Gemm355Error) as e:
            g.gemm355_attention(g.make_attention_args(cache, qd, o, q_heads=4, splits=6), stream=st)
        assert e.value.status == g.ENOMEM
        g.gemm355_attention(g.make_attention_args(cache, qd, o, q_heads=4, splits=6, workspace=ws, workspace_bytes=need), stream=st)
    for i in range(4):
        qd.copy_(2.0 * torch.randn_like(qd, dtype=torch.float32))
        want, _ = attend(c, qd.cpu(), splits=6, cache=cache)
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want), i


def tables(n, half, seed=0):
    angle = np.arange(n)[:, None] * (10000.0 ** (-np.arange(half) / max(half, 1)))[None, :]
    return np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)


def run_append(c, rot=0, interleaved=False, q=True, xk=None, xv=None, pad=0):
    xk = c.rows(c.H) if xk is None else xk
    xv = c.rows(c.H, 3.0) if xv is None else xv
    xq = c.rows(c.Hq)
    cos, sin = tables(c.max_len, rot // 2)
    cache = c.upload()
    ld = c.Hq * c.D + pad
    qo = torch.full((c.tokens, ld), 9.0, dtype=torch.bfloat16, device="cuda")
    keep = [xk.cuda(), xv.cuda(), xq.cuda(), torch.from_numpy(cos).cuda(), torch.from_numpy(sin).cuda()]
    a = g.make_kv_append_args(cache, keep[0], keep[1], q=keep[2] if q else None, q_out=qo if q else None, q_heads=c.Hq,
                              cos=keep[3] if rot else None, sin=keep[4] if rot else None, rot_dim=rot, rot_len=c.max_len,
                              interleaved=interleaved, ldqo=ld)
    g.gemm355_kv_append(a)
    torch.cuda.synchronize()
    ok.append(c.step(), c.k, c.v, c.ks, c.vs, xk.double().numpy(), xv.double().numpy(), cos, sin, rot, interleaved)
    for n in ("ks", "vs", "k", "v"):
        got, ref = c.d[n].cpu().numpy(), getattr(c, n)
        if n in ("k", "v"):      # NaN codes of either sign are one value
            got, ref = np.where(got & 0x7F == 0x7F, 0x7F, got), np.where(ref & 0x7F == 0x7F, 0x7F, ref)
        assert np.array_equal(got, ref), (n, int((got != ref).sum()))
    if q:
        want = torch.full((c.tokens, ld), 9.0, dtype=torch.bfloat16)
        s = c.step()
        for b in range(s.batch):
            for i in range(s.new[b]):
                p = s.len[b] - s.new[b] + i
                if p >= 0:
                    r = ok.rotate(xq[s.row[b] + i].double().numpy(), p, cos, sin, rot, interleaved)
                    want[s.row[b] + i, :c.Hq * c.D] = torch.from_numpy(r).to(torch.bfloat16).reshape(-1)
        assert torch.equal(qo.cpu(), want)
    return cache


@pytest.mark.parametrize("rot_of,interleaved", [(0, False), (1, False), (1, True), (2, False), (2, True), (-6, False), (-6, True)])
@pytest.mark.parametrize("i", range(len(SIZES)))
def test_append_sizes(i, rot_of, interleaved):
    """Every size with no, whole, half and an odd part (6 channels) of the head rotated."""
    lens, news, Hq, H, D, page = SIZES[i]
    say("append", SIZES[i], rot_of, interleaved)
    c = Case(100 + i, lens, news, Hq, H, D, page, extra_rows=2)
    run_append(c, rot=0 if rot_of == 0 else D // rot_of if rot_of > 0 else -rot_of, interleaved=interleaved, pad=8 * (i % 2))


def test_append_scale_growth_and_extremes():
    """Blocks whose scale grows and whose older tokens are written again; zeros,
    infinities, NaN, the largest and smallest magnitudes."""
    for D, page in ((64, 16), (128, 64)):
        c = Case(120, [30, 61, 20, 17, 40, 33], [3, 1, 4, 1, 2, 1], 2, 2, D, page)
        xk, xv = c.rows(2), c.rows(2)
        for x in (xk, xv):
            x[0:3] *= 1000.0
            x[3] *= 1e30
            x[4] = 0.0
            x[5, 0, 1], x[5, 1, 2] = float("inf"), float("-inf")
            x[6, 0, 3] = float("nan")
            x[8] *= 1e-38
            x[9:11] *= 1e-30
            x[11] *= 3e38
        run_append(c, xk=xk, xv=xv)


def test_append_then_grow_token_by_token():
    """A page filled one token a step, and an idempotent second append."""
    c = Case(121, [1], [1], 2, 1, 64, 16, max_len=40, spare=3)
    c.table[0, :3] = [2, 0, 3] if c.pages > 3 else [0, 1, 2]
    for n in range(1, 38):
        c.lens = [n]
        run_append(c, rot=64, xk=c.rows(1, float(2.0 ** (n % 7))), xv=c.rows(1, float(2.0 ** (n % 5))))
    before = [c.d[n].clone() for n in ("k", "v", "ks", "vs")]
    x = c.rows(1).cuda()
    cache = c.upload()
    a = g.make_kv_append_args(cache, x, x)
    g.gemm355_kv_append(a)
    once = [c.d[n].clone() for n in ("k", "v", "ks", "vs")]
    g.gemm355_kv_append(a)
    assert all(torch.equal(c.d[n], o) for n, o in zip(("k", "v", "ks", "vs"), once))
    assert not torch.equal(before[0], once[0])


def test_append_bad_pages_and_indices():
    c = Case(122, [200, 150, 64], [40, 2, 1], 4, 2, 64, 16)
    c.table[0, 11], c.table[1, 9] = -1, c.pages
    run_append(c, rot=64)
    c = Case(123, [200, 150, 64], [3, 2, 1], 4, 2, 64, 16)
    c.lens, c.start = [10 ** 9, -5, 64], [-4, 3, 3, 10 ** 9]
    run_append(c, rot=64)


def test_append_graph_follows_lengths():
    """A captured append replays at the lengths that the device holds then."""
    c = Case(124, [17, 33], [1, 1], 2, 2, 64, 16, max_len=64, spare=6)
    need = [4, 4]
    ids = list(range(c.pages))
    c.table[:] = np.array([ids[:4], ids[4:8]], np.int32)
    cache = c.upload()
    x = c.rows(2).cuda()
    a = g.make_kv_append_args(cache, x, x)
    g.gemm355_kv_append(a)
    torch.cuda.synchronize()
    ok.append(c.step(), c.k, c.v, c.ks, c.vs, x.double().cpu().numpy(), x.double().cpu().numpy())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.gemm355_kv_append(a)
    for i in range(20):
        c.lens = [n + 1 for n in c.lens]
        c.d["lens"].add_(1)
        x.copy_(torch.randn_like(x, dtype=torch.float32) * (i + 1))
        graph.replay()
        torch.cuda.synchronize()
        ok.append(c.step(), c.k, c.v, c.ks, c.vs, x.double().cpu().numpy(), x.double().cpu().numpy())
        for n in ("k", "v", "ks", "vs"):
            got, ref = c.d[n].cpu().numpy(), getattr(c, n)
            if n in "kv":
                got, ref = np.where(got & 0x7F == 0x7F, 0x7F, got), np.where(ref & 0x7F == 0x7F, 0x7F, ref)
            assert np.array_equal(got, ref), (i, n)
    del need


def test_decode_steps_end_to_end():
    """The operators together: weights quantised to 4 bits, projections of a
    step's tokens, append with rotation, windowed attention, output projection;
    a prompt and then single tokens, each stage against the oracle on the
    stage's own inputs."""
    rng = np.random.default_rng(130)
    Hq, H, D, page, model = 4, 2, 64, 16, 256
    group = 64

    def quantised(N, K):
        w = torch.from_numpy((rng.standard_normal((N, K)) / math.sqrt(K)).astype(np.float32)).to(torch.bfloat16).cuda()
        codes = torch.empty(N, K // 2, dtype=torch.uint8, device="cuda")
        s = torch.empty(N, K // group, dtype=torch.bfloat16, device="cuda")
        z = torch.empty(N, K // group, dtype=torch.uint8, device="cuda")
        m = g.make_w4_matrix(N, K, codes, s, z, group=group)
        g.gemm355_w4_quantize(w, m)
        oc, os_, oz = w4.quantize(w.float().cpu().numpy(), "int", group, True)
        assert np.array_equal(codes.cpu().numpy(), w4.pack(oc, K))
        return m, (codes, s, z), w4.values(oc, os_, oz, "int", group)

    qkv, keep1, Wqkv = quantised((Hq + 2 * H) * D, model)
    proj, keep2, Wout = quantised(model, Hq * D)
    c = Case(131, [0, 0], [1, 1], Hq, H, D, page, max_len=96, spare=12)
    c.table[:] = np.array([[5, 0, 7, 1, 9, 3], [2, 11, 4, 10, 6, 8]], np.int32)
    cos, sin = tables(96, D // 2)
    dcos, dsin = torch.from_numpy(cos).cuda(), torch.from_numpy(sin).cuda()
    held = [0, 0]
    for news in ([37, 20], [1, 1], [1, 1], [3, 1]):
        c.news, c.start, c.tokens, c.max_new = news, [0, news[0], sum(news)], sum(news), max(news)
        held = c.lens = [h + n for h, n in zip(held, news)]
        T = c.tokens
        x = torch.from_numpy(rng.standard_normal((T, model)).astype(np.float32)).to(torch.bfloat16)
        row = torch.empty(T, (Hq + 2 * H) * D, dtype=torch.bfloat16, device="cuda")
        g.gemm355_w4_gemm(T, x.cuda(), qkv, row)
        ref = x.double().numpy() @ Wqkv.T
        got = row.double().cpu().numpy()
        assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 1e-4)
        cache = c.upload()
        ld = row.shape[1]
        qr = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
        base = row.data_ptr()
        g.gemm355_kv_append(g.make_kv_append_args(cache, base + 2 * Hq * D, base + 2 * (Hq + H) * D, q=base, q_out=qr, q_heads=Hq,
                                                  cos=dcos, sin=dsin, rot_dim=D, rot_len=96, ldk=ld, ldv=ld, ldq=ld))
        o = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
        g.gemm355_attention(g.make_attention_args(cache, qr, o, q_heads=Hq, window=24, sinks=2))
        y = torch.empty(T, model, dtype=torch.bfloat16, device="cuda")
        g.gemm355_w4_gemm(T, o, proj, y)
        torch.cuda.synchronize()
        parts = got.reshape(T, Hq + 2 * H, D)
        ok.append(c.step(), c.k, c.v, c.ks, c.vs, parts[:, Hq:Hq + H], parts[:, Hq + H:], cos, sin, D)
        for n in ("ks", "vs"):
            assert np.array_equal(c.d[n].cpu().numpy(), getattr(c, n))
        s = c.step()
        for b in range(2):
            for i in range(news[b]):
                p = s.len[b] - news[b] + i
                r = ok.rotate(parts[s.row[b] + i, :Hq], p, cos, sin, D, False)
                assert torch.equal(qr[s.row[b] + i].cpu(), torch.from_numpy(r).to(torch.bfloat16))
        verify(c, qr.cpu(), o, None, window=24, sinks=2)
        ref = o.double().cpu().numpy().reshape(T, -1) @ Wout.T
        assert np.all(np.abs(y.double().cpu().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + 1e-4)
    del keep1, keep2
