"""Products with 4-bit weights against a bound with nothing to spare in it.

The kernel adds products x u of a group (u the code, without an offset) and
products z x, at most 128 terms each, takes one from the other, scales, adds
ng groups and joins at most 8 wavefronts.  Each of those min(K, 128) + ng + 8
additions, and four roundings of a group's sum on its way, is off by at most
2^-23 (an adder that truncates) of partial sums that stay under
A = sum |x| s (u + z); MXFP4, whose codes are signed values, has A = sum |x w|.
Then the output's rounding: half a step, 2^-24 of the value for fp32 and 2^-8
for bf16.
"""
import numpy as np
import pytest
import torch

from oracle import w4
from tests.gpu_helpers import say
from tests.test_gpu_w4 import FORMS, SHAPES, matrix, product, random_matrix

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,group,zeros", FORMS)
def test_w4_gemm_within_its_own_sums(fmt, group, zeros):
    rng = np.random.default_rng(7 * group + zeros)
    for M, N, K in SHAPES + [(1, 96, 8192), (40, 80, 4100)]:
        for out in ("f32", "bf16"):
            say("w4_gemm bound", fmt, group, zeros, M, N, K, out)
            codes, scales, z = random_matrix(rng, N, K, fmt, group, zeros)
            x = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32)).to(torch.bfloat16)
            m, keep = matrix(codes, scales, z, fmt, group, fill=15)
            y = product(M, x.cuda(), m, N, out).double().cpu().numpy()
            a, W = x.double().numpy(), w4.values(codes, scales, z, fmt, group)
            size = np.abs(W) if fmt == "mxfp4" else \
                np.repeat(scales, group, 1)[:, :K].astype(float) * (codes + (np.repeat(z, group, 1)[:, :K].astype(float) if zeros else 8.0))
            n = min(K, 128) + -(-K // group) + 12
            ref = a @ W.T
            tol = n * 2.0 ** -23 * (np.abs(a) @ size.T) + (2.0 ** -8 if out == "bf16" else 2.0 ** -24) * np.abs(ref)
            assert np.all(np.abs(y - ref) <= tol), (M, N, K, out)
            del keep
