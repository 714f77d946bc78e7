"""Pins for the oracle of the block-scaled operators (oracle/block.py), against
what the definitions and independent libraries fix."""
import numpy as np
import torch

from oracle import block


def test_quantize_against_torch_casts():
    """Codes against torch's cast to E4M3, which rounds to nearest even."""
    g = np.random.default_rng(1)
    for rows, K, block_rows in ((1, 1, 1), (3, 300, 1), (130, 200, 128), (128, 128, 128), (257, 129, 128)):
        x = (g.standard_normal((rows, K)) * np.exp(g.uniform(-20, 20, (1, K)))).astype(np.float32)
        codes, scales = block.quantize(x, block_rows)
        assert scales.shape == (-(-rows // block_rows), -(-K // 128))
        for r in range(scales.shape[0]):
            for k in range(scales.shape[1]):
                at = np.s_[r * block_rows:(r + 1) * block_rows, k * 128:(k + 1) * 128]
                a = torch.from_numpy(x[at]).abs().max()
                assert float(a / 448) == float(scales[r, k])
                t = (torch.from_numpy(x[at]) * (448 / a)).clamp(-448, 448).to(torch.float8_e4m3fn)
                assert np.array_equal(t.view(torch.uint8).numpy(), codes[at])


def test_quantize_small_blocks():
    x = np.zeros((2, 260), np.float32)
    x[0, 5] = 2.0 ** -101
    x[1, 128] = -(2.0 ** -100)
    codes, scales = block.quantize(x, 1)
    assert scales[0].tolist() == [1, 1, 1] and scales[1, 0] == 1 and scales[1, 1] == np.float32(2.0 ** -100) / np.float32(448)
    assert not codes[0].any() and codes[1, 128] == 0xFE


def test_round_trip_of_values_that_codes_stand_for():
    """Values of random codes with power-of-two scales and the largest code in
    each block come back as they were."""
    g = np.random.default_rng(2)
    codes = g.integers(0, 127, (256, 384)).astype(np.uint8) | (g.integers(0, 2, (256, 384)) << 7).astype(np.uint8)
    for block_rows in (1, 128):
        scales = np.exp2(g.integers(-8, 9, (256 // block_rows, 3))).astype(np.float32)
        codes[::block_rows, ::128] = 0x7E
        back, s = block.quantize(block.values(codes, scales, block_rows), block_rows)
        assert np.array_equal(s, scales) and np.array_equal(back, codes)


def test_values_element_by_element():
    g = np.random.default_rng(3)
    codes = g.integers(0, 127, (140, 150)).astype(np.uint8)
    for block_rows in (1, 128):
        scales = g.random((-(-140 // block_rows), 2)).astype(np.float32)
        v = block.values(codes, scales, block_rows)
        for r, k in ((0, 0), (127, 127), (128, 128), (139, 149), (5, 128)):
            m = codes[r, k]
            want = (m % 8) / 512 if m < 8 else (1 + m % 8 / 8) * 2.0 ** (int(m) // 8 - 7)
            assert v[r, k] == want * float(scales[r // block_rows, k // 128])


def test_norm_and_activations_against_torch():
    g = np.random.default_rng(4)
    x, r = g.standard_normal((5, 300)).astype(np.float32), g.standard_normal((5, 300)).astype(np.float32)
    w = g.standard_normal(300)
    h = block.norm_input(x, r, "bf16")
    assert np.array_equal(h, (torch.from_numpy(x) + torch.from_numpy(r)).to(torch.bfloat16).float().numpy())
    ref = torch.nn.functional.rms_norm(torch.from_numpy(h).double(), (300,), torch.from_numpy(w), 0.25)
    assert np.allclose(block.rmsnorm(h, w, 0.25), ref.numpy(), rtol=1e-13, atol=0)
    z = torch.linspace(-30, 30, 1001, dtype=torch.float64)
    assert np.allclose(block.act(z.numpy(), "silu"), torch.nn.functional.silu(z).numpy(), rtol=1e-13, atol=1e-300)
    assert np.allclose(block.act(z.numpy(), "gelu"), torch.nn.functional.gelu(z, approximate="tanh").numpy(), rtol=1e-12, atol=1e-15)
