"""Pins for the oracles of the serving operators (oracle/w4.py,
oracle/kvcache.py), against what the definitions and independent libraries fix."""
import numpy as np
import pytest
import torch

from oracle import kvcache, mx, w4


def test_bf16_matches_torch():
    g = np.random.default_rng(1)
    x = np.concatenate([g.standard_normal(50000) * np.exp(g.uniform(-60, 60, 50000)), [0.0, -0.0, 1.00390625, 1.01171875]]).astype(np.float32)
    assert np.array_equal(w4.bf16(x), torch.from_numpy(x).to(torch.bfloat16).float().numpy())


@pytest.mark.parametrize("zeros", (False, True))
@pytest.mark.parametrize("group", (32, 64, 128))
def test_int_round_trip_of_representable_matrices(group, zeros):
    """Values that codes stand for, with the ends of the range present, come
    back as they were."""
    g = np.random.default_rng(group + zeros)
    N, K = 5, 3 * group - 7
    ng = 3
    s = w4.bf16(np.exp2(g.integers(-6, 3, (N, ng))).astype(np.float32) * 1.25)
    z = g.integers(0, 16, (N, ng)).astype(np.uint8) if zeros else None
    u = g.integers(0, 16, (N, K)).astype(np.uint8) if zeros else g.integers(1, 16, (N, K)).astype(np.uint8)
    for i in range(ng):
        u[:, i * group], u[:, i * group + 1] = (0, 15) if zeros else (1, 15)
    w = w4.values(u, s, z, "int", group).astype(np.float32)
    u2, s2, z2 = w4.quantize(w, "int", group, zeros)
    assert np.array_equal(s2, s) and np.array_equal(u2, u)
    if zeros:
        assert np.array_equal(z2, z)


def test_int_error_is_half_a_step():
    g = np.random.default_rng(5)
    w = g.standard_normal((8, 256)).astype(np.float32)
    for zeros in (False, True):
        u, s, z = w4.quantize(w, "int", 64, zeros)
        d = np.abs(w4.values(u, s, z, "int", 64) - w)
        # a scale rounded to 8 bits moves the ends of the range by at most
        # 15 * 2^-8 of a step beyond the half
        assert np.all(d <= np.repeat(s, 64, axis=1) * (0.5 + 15 * 2.0 ** -8 + (0.5 if zeros else 0.0)))


def test_mxfp4_nearest_by_brute_force():
    g = np.random.default_rng(6)
    w = (g.standard_normal((6, 70)) * 3).astype(np.float32)
    w[0, :32] = 0.0
    w[1, :16] = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, 7.9])
    u, e, _ = w4.quantize(w, "mxfp4", 32)
    v = w4.values(u, e, None, "mxfp4", 32)
    table = mx.decode_e2m1(np.arange(16))
    for n in range(6):
        for k in range(70):
            sc = 2.0 ** (int(e[n, k // 32]) - 127)
            near = min(abs(np.clip(w[n, k], -6 * sc, 6 * sc) - t * sc) for t in table)
            assert abs(np.clip(w[n, k], -6 * sc, 6 * sc) - v[n, k]) == near
    assert list(u[1, :8]) == [0, 2, 2, 4, 4, 6, 6, 7] and list(u[1, 8:15]) == [8, 10, 10, 12, 12, 14, 14]
    assert e[0, 0] == 0 and np.all(v[0, :32] == 0)


def test_pack_matches_the_block_scaled_layout():
    u = np.random.default_rng(7).integers(0, 16, (3, 64)).astype(np.uint8)
    assert np.array_equal(mx.unpack_fp4(w4.pack(u, 64)), u)


def test_block_exponent_borders():
    for e in (-100, -3, 0, 5, 119):
        a = np.ldexp(448.0, e)
        assert kvcache.block_exponent(a) == e
        assert kvcache.block_exponent(np.nextafter(a, np.inf)) == e + 1
    assert kvcache.block_exponent(0.0) == -100 and kvcache.block_exponent(np.inf) == 120


def test_attention_against_torch_softmax():
    g = np.random.default_rng(8)
    H, Hq, D, page, pages = 2, 4, 64, 16, 6
    k = kvcache.encode(g.standard_normal((pages, H, page, D)) * 60)
    v = kvcache.encode(g.standard_normal((pages, H, D, page)) * 60)
    ks, vs = np.full((pages, H), 121, np.uint8), np.full((pages, H), 120, np.uint8)
    step = kvcache.Step([40], [0, 3], 3, 3, 64, [[3, 1, 4, 0]], page, pages)
    q = g.standard_normal((3, Hq, D))
    o, lse, _, _ = kvcache.attention(step, k, v, ks, vs, q, 0.125)
    order = [3, 1, 4]
    kk = torch.from_numpy(np.concatenate([kvcache.decode(k[i]) / 64 for i in order], axis=1)[:, :40])
    vv = torch.from_numpy(np.concatenate([kvcache.decode(v[i]).transpose(0, 2, 1) / 128 for i in order], axis=1)[:, :40])
    x = torch.einsum("rhd,htd->rht", torch.from_numpy(q), kk.repeat_interleave(2, 0)) * 0.125
    hidden = torch.arange(40)[None] > torch.arange(37, 40)[:, None]
    x = x.masked_fill(hidden[:, None], -np.inf)
    ref = torch.einsum("rht,htd->rhd", x.softmax(-1), vv.repeat_interleave(2, 0))
    assert np.allclose(o, ref.numpy(), rtol=1e-12, atol=1e-12)
    assert np.allclose(lse, x.logsumexp(-1).numpy(), rtol=1e-12)


def test_append_one_by_one_keeps_the_block_scale_monotone():
    g = np.random.default_rng(9)
    H, D, page = 1, 64, 16
    k = np.full((1, H, page, D), 0x7F, np.uint8)
    v = np.full((1, H, D, page), 0x7F, np.uint8)
    ks, vs = np.full((1, H), 77, np.uint8), np.full((1, H), 77, np.uint8)
    x = g.standard_normal((page, H, D)) * np.exp2(np.arange(page))[:, None, None]
    last = 0
    for t in range(page):
        step = kvcache.Step([t + 1], [0, 1], 1, 1, page, [[0]], page, 1)
        kvcache.append(step, k, v, ks, vs, x[t:t + 1], x[t:t + 1])
        assert ks[0, 0] == vs[0, 0] >= last
        last = ks[0, 0]
        assert np.all(k[0, 0, t + 1:] == 0x7F) and np.all(v[0, 0, :, t + 1:] == 0x7F)
        got = kvcache.decode(k[0, 0, :t + 1]) * 2.0 ** (int(last) - 127)
        assert np.array_equal(got.T, kvcache.decode(v[0, 0, :, :t + 1]) * 2.0 ** (int(last) - 127))
        # each rewriting rounds to nearest again: at most one step of the largest in all
        assert np.max(np.abs(got - x[:t + 1, 0])) <= 32 * 2.0 ** (int(last) - 127)
