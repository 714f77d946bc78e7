"""Attention where every weight is a power of two and every sum a whole number
of halves or more, so that one value lost, cleared or read from the wrong place
shows on axes of any length.

Scores are whole numbers s <= 0 with scale = ln 2 (in binary32 times log2(e)
exactly 1), so weights 2^s are exact in bf16 and their products with values of
few bits and the sums of those are exact in binary32.  What is left is
  equal weights (q = 0): the quotient's two roundings, under 2^-22 of it;
  weights of several sizes: the total, each of whose n / 64 * 17 + 100
    additions a lane makes at most (and each exponential, within one unit in
    the last place) may be off by 2^-23: under 2^-12 of it for n <= 3100;
and the output's rounding, which is monotone: o lies between the roundings of
the quotient brought down and up by that much.  The logarithm of the total: as
much, and 2^-21 of itself for the logarithm and its two roundings.
"""
import math

import numpy as np
import pytest
import torch

from oracle import kvcache as ok
from tests.gpu_helpers import say
from tests.test_gpu_kvcache import Case, attend

pytestmark = pytest.mark.gpu

LN2 = float(np.float32(math.log(2.0)))


def exact_case(seed, lens, news, Hq, H, D, page, steps=0, one_hot=False, **kw):
    """Whole numbers of up to 8 as values, with scales of 1/2 to 2; keys that
    hold -s in one channel (s up to `steps`), of scale 1.  one_hot: a channel
    holds a single token, at the borders of chunks, pages and parts."""
    assert float(np.float32(LN2 * 1.4426950408889634)) == 1.0
    c = Case(seed, lens, news, Hq, H, D, page, **kw)
    r = c.rng
    c.ks[:] = 127
    c.vs[:] = r.integers(126, 129, c.vs.shape)
    c.val, c.low = [], []
    for b, n in enumerate(lens):
        v = r.integers(-8, 9, (n, H, D)).astype(np.float64)
        if one_hot and n:
            edges = [0, n - 1, n // 2] + [e + d for e in range(0, n, 64) for d in (-1, 0)] + [e + d for e in range(0, n, page) for d in (-1, 0)]
            edges = np.array([e for e in dict.fromkeys(edges) if 0 <= e < n])
            v[:] = 0
            for h in range(H):
                v[r.choice(edges, D), h, np.arange(D)] = r.integers(1, 9, D)
        s = r.integers(0, steps + 1, (n, H))
        c.val.append(v)
        c.low.append(s)
        for t in range(0, n, page):
            at, m = c.table[b, t // page], min(page, n - t)
            c.v[at, :, :, :m] = ok.encode(v[t:t + m]).transpose(1, 2, 0)
            key = np.zeros((m, H, D))
            for h in range(H):
                key[np.arange(m), h, (7 * (t + np.arange(m)) + h) % D] = -s[t:t + m, h]
            c.k[at, :, :m] = ok.encode(key).transpose(1, 0, 2)
            c.val[b][t:t + m] = v[t:t + m] * np.ldexp(1.0, c.vs[at].astype(int) - 127)[None, :, None]
    return c


def check(c, factor, o, ls, near, window=0, sinks=0):
    """factor [rows][Hq]: weights are 2^(-factor s)."""
    s = c.step()
    got, gl = o.double().cpu().numpy(), ls.double().cpu().numpy()
    group, seen_rows = c.Hq // c.H, np.zeros(c.tokens, bool)
    for b in range(s.batch):
        n = s.len[b]
        held = np.array([s.page_id(b, t) is not None for t in range(n)], bool)
        for j in range(c.Hq):
            h = j // group
            sums = {}
            for f in np.unique(factor[:, j]):
                w = held * np.exp2(-f * c.low[b][:, h].astype(np.float64))
                sums[f] = (np.concatenate([np.zeros((1, c.D)), np.cumsum(w[:, None] * c.val[b][:, h], 0)]), np.concatenate([[0.0], np.cumsum(w)]))
            for i in range(s.new[b]):
                p, row = s.pos[b] + i, s.row[b] + i
                seen_rows[row] = True
                end = max(p + 1, 0)
                lo = max(end - window, 0) if window else 0
                first = min(sinks, lo)
                V, W = sums[factor[row, j]]
                total = W[end] - W[lo] + W[first]
                if total == 0:
                    assert np.all(got[row, j] == 0) and gl[row, j] == -np.inf
                    continue
                ref = (V[end] - V[lo] + V[first]) / total
                ends = torch.from_numpy(np.stack([ref * (1 - near), ref * (1 + near)])).float().to(torch.bfloat16).double().numpy()
                assert np.all((got[row, j] >= ends.min(0)) & (got[row, j] <= ends.max(0))), (b, j, i)
                want = math.log(total)
                assert abs(gl[row, j] - want) <= near + 2.0 ** -21 * max(1.0, abs(want)), (b, j, i)
    assert np.all(got[~seen_rows] == 9.0)


SHAPES = [
    # lens, new rows, Hq, H, D, page
    ([30000, 17001, 900], [2, 1, 1], 2, 1, 64, 32),
    ([30000, 17001, 900], [2, 1, 1], 2, 1, 128, 128),
    ([30000, 17001, 900], [2, 1, 1], 2, 1, 256, 16),
    ([8000], [1], 8, 2, 128, 64),
    ([1000, 333, 0, 64], [1, 1, 1, 1], 8, 8, 64, 16),
    ([700, 330], [134, 130], 32, 8, 64, 32),          # 32 rows a workgroup, four wavefronts
    ([700, 330], [134, 130], 32, 8, 128, 16),
    ([700, 330], [134, 130], 32, 8, 256, 64),
    ([500, 330], [210, 200], 64, 8, 64, 128),         # and two
    ([500, 330], [210, 200], 64, 8, 128, 32),
]


@pytest.mark.parametrize("one_hot", (False, True))
@pytest.mark.parametrize("splits", (0, 1, 65))
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_attention_means_of_every_token(i, splits, one_hot):
    """q = 0: the mean of the values seen, to the last bit but one."""
    say("attention means", SHAPES[i], splits, one_hot)
    c = exact_case(700 + i, *SHAPES[i], one_hot=one_hot, extra_rows=2)
    q = torch.zeros(c.tokens, c.Hq, c.D, dtype=torch.bfloat16)
    cache = c.upload()
    for kw in (dict(), dict(window=200, sinks=5), dict(window=64), dict(window=1, sinks=70))[:4 if i < 5 else 2]:
        o, ls = attend(c, q, cache=cache, splits=splits, **kw)
        check(c, np.zeros((c.tokens, c.Hq)), o, ls, 2.0 ** -22, **kw)


@pytest.mark.parametrize("splits", (0, 3))
@pytest.mark.parametrize("lens,news,Hq,H,D,page", [([3000, 700], [2, 1], 4, 2, 64, 16), ([3000, 700], [2, 1], 4, 2, 128, 64), ([3000, 700], [2, 1], 8, 2, 256, 32)]
                         + SHAPES[5:])
def test_attention_weights_of_powers_of_two(lens, news, Hq, H, D, page, splits):
    """Weights of 1 down to 2^-6, another factor for each row, pages that nobody
    holds."""
    say("attention powers", lens, news, Hq, H, D, page, splits)
    c = exact_case(720, lens, news, Hq, H, D, page, steps=3, extra_rows=1)
    c.table[0, 2] = -1
    factor = c.rng.integers(0, 3, (c.tokens, Hq))
    q = torch.from_numpy(np.repeat(factor[:, :, None], D, 2).astype(np.float32)).to(torch.bfloat16)
    cache = c.upload()
    for kw in (dict(), dict(window=130, sinks=3)):
        o, ls = attend(c, q, cache=cache, scale=LN2, splits=splits, **kw)
        check(c, factor, o, ls, 2.0 ** -12, **kw)


@pytest.mark.parametrize("new,splits", [(20, 1), (20, 2), (1, 1)])
def test_nan_codes_leave_the_rows_that_do_not_see_them(new, splits):
    """The rows before the tokens that hold a NaN are there, and keep their bits."""
    def case():
        return Case(740, [300, 70], [new, new], 4, 2, 64, 32)
    c, clean = case(), case()
    for t in (295, 299):
        c.v[c.table[0, t // 32], 1, 5, t % 32] = 0x7F
    c.k[c.table[1, 2], 0, 68 % 32, 3] = 0xFF
    q = c.rows(4)
    o, ls = attend(c, q, splits=splits)
    want, wl = attend(clean, q, splits=splits)
    row = np.arange(2 * new)
    first = np.where(row < new, 300 - new + row < 295, 70 - new + row - new < 68)
    assert first.any() == (new > 1) and not first.all()
    heads = np.stack([row >= new, row >= new, row < new, row < new], 1) & ~first[:, None]
    assert np.array_equal(torch.isnan(o).any(2).cpu().numpy(), heads)
    same = torch.from_numpy(~heads)
    assert torch.equal(o.cpu()[same], want.cpu()[same]) and torch.equal(ls.cpu()[same], wl.cpu()[same])


@pytest.mark.parametrize("splits", (0, 3))
@pytest.mark.parametrize("lens,news,Hq,H,D,page", [([3000, 700], [2, 1], 4, 2, 64, 16), ([3000, 700], [2, 1], 4, 2, 128, 64), ([3000, 700], [2, 1], 8, 2, 256, 32)]
                         + SHAPES[5:])
def test_attention_of_equal_values_is_that_value(lens, news, Hq, H, D, page, splits):
    """Random scores, one value a channel: a mean of it, whatever the weights
    were rounded to, as the same weights divide it.  Two sums of at most 3000
    terms, each addition off by 2^-23: under 2^-10, and half a step of bf16 is
    2^-9 at least."""
    say("attention equal values", lens, news, Hq, H, D, page, splits)
    c = Case(760, lens, news, Hq, H, D, page)
    codes = ok.encode(c.rng.standard_normal((len(lens), H, D)) * 100)
    value = np.ldexp(ok.decode(codes), -3)
    c.vs[:] = 124
    for b, n in enumerate(lens):
        for t in range(0, n, page):
            c.v[c.table[b, t // page], :, :, :min(page, n - t)] = codes[b][:, :, None]
    for scale in (1.0, 4.0):
        o, ls = attend(c, c.rows(Hq, scale), splits=splits)
        row = 0
        for b, n in enumerate(news):
            want = torch.from_numpy(np.repeat(value[b], Hq // H, 0)).to(torch.bfloat16)
            assert torch.equal(o[row:row + n].cpu(), want.expand(n, Hq, D)), (scale, b)
            row += n
