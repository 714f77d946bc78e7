"""The ends of the paged 8-bit cache on the GPU: block scales of any byte, held
values past the largest finite one, what hides them, and rows of one tile that
must not feel each other.  Appended bytes are compared with the oracle bit for
bit, attention by the bound of test_gpu_kvcache.py where a row is finite; rows
that see none of what changed are compared with the unchanged cache bit for
bit.
"""
import numpy as np
import pytest
import torch

from dense_tiled_gemm_fp8_amd import gemm355 as g
from oracle import kvcache as ok
from tests.gpu_helpers import say
from tests.test_gpu_kvcache import Case, attend, run_append, verify

pytestmark = pytest.mark.gpu


def free_page_0(c):
    """Gives page 0 to nobody: whoever has it gets a page that is not in use."""
    held = [-(-n // c.page) for n in c.lens]
    used = {int(c.table[b, j]) for b in range(len(c.lens)) for j in range(held[b])}
    spare = next(i for i in range(c.pages) if i not in used)
    for b in range(len(c.lens)):
        for j in range(held[b]):
            if c.table[b, j] == 0:
                c.table[b, j] = spare
                for a in (c.k, c.v, c.ks, c.vs):
                    a[spare] = a[0]
    c.k[0], c.v[0] = 0x7F, 0x7F
    return c


def same_bits(a, b, rows):
    rows = torch.from_numpy(rows)
    return torch.equal(a.cpu().view(torch.int16)[rows], b.cpu().view(torch.int16)[rows])


def positions(c):
    """Sequence and position of each row."""
    s = c.step()
    at = np.full((c.tokens, 2), -1)
    for b in range(s.batch):
        for i in range(s.new[b]):
            at[s.row[b] + i] = b, s.len[b] - s.new[b] + i
    return at


# lens, new rows, Hq, H, D, page: one row, few rows, prompts of both counts of rows a workgroup
FORMS = [([300, 130], [1, 1], 4, 2, 64, 16), ([300, 130], [20, 7], 4, 2, 128, 16), ([300, 130], [20, 3], 4, 2, 256, 16),
         ([400, 330], [134, 130], 32, 8, 64, 32), ([400, 330], [134, 130], 32, 8, 128, 16), ([400, 330], [134, 130], 32, 8, 256, 32)]


@pytest.mark.parametrize("splits", (0, 2))
@pytest.mark.parametrize("i", range(len(FORMS)))
def test_scales_of_hidden_pages_have_no_effect(i, splits):
    """Tokens without a page, where nothing of page 0 may show; pages before the
    window, in a chunk with pages that are seen."""
    lens, news, Hq, H, D, page = FORMS[i]
    say("hidden scales", FORMS[i], splits)
    c = free_page_0(Case(500 + i, lens, news, Hq, H, D, page))
    q = c.rows(Hq, 2.0)
    c.table[0, 3], c.table[0, 5], c.table[1, 1] = -1, c.pages, -(1 << 31)
    for byte in (255, 254):
        c.ks[0], c.vs[0] = byte, byte
        o, ls = attend(c, q, splits=splits)
        verify(c, q, o, ls)
    c = Case(520 + i, lens, news, Hq, H, D, page)
    q = c.rows(Hq, 2.0)
    # the first row's window begins with the last page of a 64-token chunk
    window = next(w for w in range(20, 100) if (lens[0] - news[0] - w + 1) % 64 == 64 - page)
    want, wl = attend(c, q, window=window, splits=splits)
    verify(c, q, want, wl, window=window)
    for b in range(2):
        for j in range(max(0, lens[b] - news[b] - window + 1) // page):
            c.ks[c.table[b, j]], c.vs[c.table[b, j]] = 255, 255
    o, ls = attend(c, q, window=window, splits=splits)
    assert same_bits(o, want, np.arange(c.tokens)) and torch.equal(ls, wl)


@pytest.mark.parametrize("splits", (0, 2))
@pytest.mark.parametrize("which", ("k", "v"))
@pytest.mark.parametrize("i", range(1, len(FORMS)))
def test_a_nan_block_reaches_the_rows_that_see_it_alone(i, which, splits):
    lens, news, Hq, H, D, page = FORMS[i]
    say("NaN block", FORMS[i], which, splits)
    c = Case(540 + i, lens, news, Hq, H, D, page)
    q = c.rows(Hq, 2.0)
    want, wl = attend(c, q, splits=splits)
    p0 = lens[0] - news[0]
    at = -(-(p0 + 3) // page) * page                     # a page that begins between two rows
    if at >= lens[0]:
        at = p0 // page * page
    head = 1
    (c.ks if which == "k" else c.vs)[c.table[0, at // page], head] = 255
    o, ls = attend(c, q, splits=splits)
    pos = positions(c)
    sees = (pos[:, 0] == 0) & (pos[:, 1] >= at)
    assert sees.any()
    group = Hq // H
    mine = slice(head * group, (head + 1) * group)
    other = [j for j in range(Hq) if j // group != head]
    assert torch.isnan(o[torch.from_numpy(sees)][:, mine]).all()
    assert same_bits(o, want, ~sees) and torch.equal(ls.cpu()[torch.from_numpy(~sees)], wl.cpu()[torch.from_numpy(~sees)])
    assert same_bits(o[:, other], want[:, other], np.arange(c.tokens))


@pytest.mark.parametrize("splits", (0, 2))
@pytest.mark.parametrize("i", range(1, len(FORMS)))
def test_values_past_the_largest_reach_the_rows_that_see_them_alone(i, splits):
    """Held values of 2^128 and more: as the append writes them (an infinity, and
    the largest bf16 value, whose code is 2^128), and codes of 2^128 under the
    largest scales.  A value of 2^119 under the same scale is finite, also
    beside the weights of up to 2^8 that it is summed with."""
    lens, news, Hq, H, D, page = FORMS[i]
    mid = news[0] // 2
    t, group = lens[0] - news[0] + mid, Hq // H
    for how in ("inf", "max", 248, 254):
        say("large values", FORMS[i], splits, how)
        c = Case(560 + i, lens, news, Hq, H, D, page)
        q = c.rows(Hq, 2.0)
        at, slot = c.table[0, t // page], t % page
        if isinstance(how, str):
            xv = torch.zeros(c.tokens, H, D, dtype=torch.bfloat16)
            xv[mid, 0, 5] = float("inf") if how == "inf" else torch.finfo(torch.bfloat16).max
            run_append(c, xk=c.rows(H), xv=xv)
            assert c.vs[at, 0] == 247 and ok.decode(c.v[at, 0, 5, slot]) >= 256
        else:
            c.v[at, 0], c.vs[at, 0] = 0, how
            c.v[at, 0, 5, slot] = (262 - how) << 3       # the code of 2^(255 - how)
        o, ls = attend(c, q, splits=splits)
        c.v[at, 0, 5, slot] = 0
        want, wl = attend(c, q, splits=splits)
        verify(c, q, want, wl)
        pos = positions(c)
        sees = (pos[:, 0] == 0) & (pos[:, 1] >= t)
        assert sees.any() and (~sees).any()
        assert not torch.isfinite(o[torch.from_numpy(sees)][:, :group, 5]).any()
        assert same_bits(o, want, ~sees) and torch.equal(ls.cpu()[torch.from_numpy(~sees)], wl.cpu()[torch.from_numpy(~sees)])
        assert same_bits(o[:, group:], want[:, group:], np.arange(c.tokens))
        if not isinstance(how, str):
            c.v[at, 0, 5, slot] = ok.encode(np.float64(2.0 ** (246 - how)))
            o, ls = attend(c, q, splits=splits)
            verify(c, q, o, ls)


@pytest.mark.parametrize("D,page", [(64, 16), (128, 64), (256, 128)])
def test_append_to_pages_of_any_scale(D, page):
    """Every byte a page's scale can have, kept or grown: new codes are those of
    its value (a page of byte 255 stays one, its codes as under 2^128)."""
    for lo in range(0, 256, 64):
        say("append scales", D, page, lo)
        c = Case(580 + lo, [page + 5] * 32, [2] * 32, 2, 2, D, page)
        byte = lo
        for b in range(32):
            for h in range(2):
                c.ks[c.table[b, 1], h], c.vs[c.table[b, 1], h] = byte, 255 - byte
                byte += 1
        xk, xv = c.rows(2), c.rows(2)
        for b in range(32):
            xk[2 * b] *= 2.0 ** float(c.rng.integers(-100, 126))
            xv[2 * b:2 * b + 2] *= 2.0 ** float(c.rng.integers(-100, 126))
        run_append(c, xk=xk, xv=xv)


@pytest.mark.parametrize("splits", (0, 2))
@pytest.mark.parametrize("i", range(len(FORMS)))
def test_rows_of_a_tile_do_not_feel_each_other(i, splits):
    """A NaN, infinities, and scores far above the others' in some rows: the
    others keep their bits, whatever the references of those rows do.  So do the
    rows before a token that changes."""
    lens, news, Hq, H, D, page = FORMS[i]
    say("rows alone", FORMS[i], splits)
    c = Case(600 + i, lens, news, Hq, H, D, page)
    q = c.rows(Hq)
    want, wl = attend(c, q, splits=splits)
    changed = np.zeros((c.tokens, Hq), bool)
    bad = q.clone()
    for n, (r, h) in enumerate(((0, 1), (c.tokens - 1, 2), (c.tokens // 2, 0), (c.tokens // 3, 3))):
        changed[r, h] = True
        bad[r, h] = float("inf") if n == 1 else 100.0 * bad[r, h]
        if n == 0:
            bad[r, h, 5] = float("nan")
    o, ls = attend(c, bad, splits=splits)
    assert same_bits(o, want, ~changed) and torch.equal(ls.cpu()[torch.from_numpy(~changed)], wl.cpu()[torch.from_numpy(~changed)])
    last = lens[0] - 1
    c.k[c.table[0, last // page], :, last % page] = ok.encode(c.rng.standard_normal((H, D)) * 400)
    o, ls = attend(c, q, splits=splits)
    pos = positions(c)
    sees = (pos[:, 0] == 0) & (pos[:, 1] >= last)
    assert same_bits(o, want, ~sees) and torch.equal(ls.cpu()[torch.from_numpy(~sees)], wl.cpu()[torch.from_numpy(~sees)])


@pytest.mark.parametrize("D,page", [(64, 16), (128, 32), (256, 128)])
def test_rows_past_max_new_are_left_out_where_they_are(D, page):
    """More rows than max_new in a sequence: the first of them keep their
    positions, the others are neither read nor written."""
    news = [12, 3, 5]
    for most in (1, 4, 11):
        say("rows past max_new", D, page, most)
        c = Case(620, [90, 40, 7], news, 4, 2, D, page)
        c.max_new = most
        out = torch.cat([torch.arange(n) >= most for n in news])
        q, xk, xv = c.rows(4, 2.0), c.rows(2), c.rows(2, 3.0)
        for x in (q, xk, xv):
            x[out] = float("nan")
        before = [getattr(c, n).copy() for n in ("k", "v")]
        run_append(c, rot=64, q=False, xk=xk, xv=xv)
        for b, n in enumerate(news):
            for t in range(c.lens[b] - n, c.lens[b]):
                at, slot = c.table[b, t // page], t % page
                stays = np.array_equal(c.k[at, :, slot], before[0][at, :, slot]) and np.array_equal(c.v[at, :, :, slot], before[1][at, :, :, slot])
                assert stays == (t >= c.lens[b] - n + most)
        o, ls = attend(c, q)
        assert torch.all(o.cpu()[out] == 9.0) and torch.all(ls.cpu()[out] == 9.0) and not torch.any(o.cpu()[~out] == 9.0)
        verify(c, q, o, ls)


def test_step_in_columns_of_one_buffer():
    """A projection's output, the rotated queries, attention's output and the
    next projection's result side by side in the rows of one buffer."""
    Hq, H, D, page, T, N = 4, 2, 64, 16, 6, 96
    c, d = (Case(640, [50, 33], [4, 2], Hq, H, D, page) for _ in range(2))
    widths = [Hq * D, H * D, H * D, Hq * D, Hq * D, N]
    at = [int(n) for n in np.cumsum([0] + widths)]
    arena = torch.full((T, at[-1] + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    ld = arena.shape[1]
    rows = [c.rows(n) for n in (Hq, H, H)]
    part = [arena[:, a:b] for a, b in zip(at, at[1:])]
    for n in range(3):
        part[n].copy_(rows[n].reshape(T, -1))
    address = [arena.data_ptr() + 2 * n for n in at]
    codes = torch.randint(0, 256, (N, Hq * D // 2), dtype=torch.uint8, device="cuda")
    scales = torch.full((N, Hq * D // 64), 0.125, dtype=torch.bfloat16, device="cuda")
    m = g.make_w4_matrix(N, Hq * D, codes, scales, group=64)
    g.gemm355_kv_append(g.make_kv_append_args(c.upload(), address[1], address[2], q=address[0], q_out=address[3], q_heads=Hq,
                                              ldk=ld, ldv=ld, ldq=ld, ldqo=ld))
    cache = g.make_kv_cache(c.d["k"], c.d["v"], c.d["ks"], c.d["vs"], pages=c.pages, heads=H, head_dim=D, page=page, table=c.d["table"],
                            lens=c.d["lens"], batch=2, max_len=c.max_len, q_start=c.d["start"], tokens=T, max_new=4)
    g.gemm355_attention(g.make_attention_args(cache, address[3], address[4], q_heads=Hq, ldq=ld, ldo=ld))
    g.gemm355_w4_gemm(T, address[4], m, address[5], ldx=ld, ldy=ld)
    torch.cuda.synchronize()
    apart = d.upload()
    x = [r.cuda() for r in rows]
    q, o, y = torch.empty_like(x[0]), torch.empty_like(x[0]), torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    g.gemm355_kv_append(g.make_kv_append_args(apart, x[1], x[2], q=x[0], q_out=q, q_heads=Hq))
    g.gemm355_attention(g.make_attention_args(apart, q, o, q_heads=Hq))
    g.gemm355_w4_gemm(T, o, m, y)
    torch.cuda.synchronize()
    for n, want in zip((0, 1, 2, 3, 4, 5), x + [q, o, y]):
        assert torch.equal(part[n], want.reshape(T, -1)), n
    assert torch.isnan(arena[:, at[-1]:]).all() and all(torch.equal(c.d[n], d.d[n]) for n in ("k", "v", "ks", "vs"))


@pytest.mark.parametrize("i", range(len(FORMS)))
def test_attention_scales_from_end_to_end(i):
    """Scales of 2^-127 to 2^93 for values, to 1 for keys, one size for all or
    mixed.  (Values of bf16's subnormal range may be lost: they are under 1/50
    of the largest of their block, and of these few.)"""
    lens, news, Hq, H, D, page = FORMS[i]
    say("scales", FORMS[i])
    c = Case(660 + i, lens, news, Hq, H, D, page)
    q = c.rows(Hq, 2.0)
    for low, high in ((0, 0), (1, 1), (8, 8), (60, 60), (220, 220), (90, 105)):
        c.vs[:] = c.rng.integers(low, high + 1, c.vs.shape)
        c.ks[:] = c.rng.integers(min(low, 110), min(high, 121) + 1, c.ks.shape)
        o, ls = attend(c, q)
        verify(c, q, o, ls)
