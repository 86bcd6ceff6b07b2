"""Sampling at the edges of its numbers: the smallest temperatures, signalling NaN, random numbers out of range."""
import math

import pytest
import torch

from routed_token_indexer_amd import _lib as M
from test_gpu_sample import both, rows, uniform

pytestmark = pytest.mark.gpu
LEAST = 2.0 ** -149
SMALL = [LEAST, 5 * LEAST, 1e-42, 1e-40, 5.9e-39, 2.0 ** -126, 1.9e-38, 3e-37, 2.0 ** -120, 2.0 ** -119, 1e-35]


def small(T, V, span, seed, dtype=torch.float32, base=0.0):
    """Logits from 0 to -span around base: fp32 is exact there, down to subnormal steps."""
    g = torch.Generator().manual_seed(seed)
    x = base - span * torch.rand(T, V, generator=g, dtype=torch.float64)
    return x.to(dtype).cuda()


@pytest.mark.parametrize("V", [2, 700, 5000, 70001])
@pytest.mark.parametrize("base", [0.0, 1e-36, -3e-38, 1e-12, -2.0 ** -40, 1.0, 3e38])
def test_smallest_temperatures(V, base):
    """Logits that differ by as little as the temperature, and by far more; the same definition down to 2^-149."""
    T = len(SMALL)
    u = uniform(T, V)
    k = [0, 1, 3, 50, V // 2, 0, 7, 0, 2, V, 100]
    p = [1.0, 0.9, 1.0, 0.5, 0.9, 0.3, 0.99, 1.0, 0.7, 0.9, 0.8]
    m = [0.0, 0.0, 0.1, 0.0, 0.01, 0.0, 0.5, 1e-3, 0.0, 0.0, 0.2]
    for span in (40 * LEAST, 1.3e-35, 1e-30):
        x = small(T, V, span, V, base=base)
        both(x, u, t=SMALL, strict=False)
        both(x, u, t=SMALL, p=p, strict=False)
        both(x, u, t=SMALL, k=k, strict=False)
        both(x, u, t=SMALL, k=k, p=p, m=m, strict=False)
    # each row's logits spread by some tens of its own temperature: many tokens in reach
    x = torch.cat([small(1, V, 30.0 * t, i, base=base) for i, t in enumerate(SMALL)])
    both(x, u, t=SMALL, strict=False)
    both(x, u, t=SMALL, p=p, strict=False)
    both(x, u, t=SMALL, k=k, m=m, strict=False)


def test_a_weight_far_below():
    """A logit 1.3e-35 below the largest at a temperature of 1e-40 weighs nothing."""
    x = torch.tensor([[-1.3e-35, 0.0, -1.3e-35]] * 3).cuda()
    got = both(x, [0.0, 0.5, 0.999], t=[1e-40] * 3)
    assert got.tolist() == [1, 1, 1]
    got = both(x, [0.0, 0.5, 0.999], t=[1e-40] * 3, p=[0.9] * 3, k=[2] * 3)
    assert got.tolist() == [1, 1, 1]


def test_smallest_temperatures_of_infinite_and_wide_rows():
    T = len(SMALL)
    x = rows(T, 900, "fp32", 3)
    x[:, 5] = 1e30
    x[:, 6] = -1e30
    both(x, uniform(T, 1), t=SMALL)
    x[:, [17, 300]] = math.inf
    both(x, uniform(T, 2), t=SMALL, p=[0.9] * T)
    x = torch.full((T, 900), -math.inf, device="cuda")
    x[:, 33], x[:, 34], x[:, 800] = -1e-44, -1e38, -1e-41
    both(x, uniform(T, 3), t=SMALL)
    both(x.half(), uniform(T, 4), t=SMALL, k=[2] * T)
    both(x.bfloat16(), uniform(T, 5), t=SMALL, p=[0.99] * T)


@pytest.mark.parametrize("dtype,bits", [("bf16", [0x7f81, -0x7f]), ("fp16", [0x7c01, -0x3ff]), ("fp32", [0x7f800001, -0x7fffff])])
@pytest.mark.parametrize("V", [64, 3001, 70001])
def test_signalling_nan(V, dtype, bits):
    """NaN of every kind is passed over, wherever it stands."""
    x = rows(4, V, dtype, V)
    raw = x.view({"bf16": torch.int16, "fp16": torch.int16, "fp32": torch.int32}[dtype])
    raw[0, ::2], raw[1, 1::3], raw[2, V // 2:], raw[3, :V // 2] = bits[0], bits[1], bits[0], bits[1]
    assert bool(x.isnan().any(1).all())
    u = uniform(4, 1)
    both(x, u, strict=False)
    both(x, u, k=[50, 3, 0, 1], p=[0.9, 1.0, 0.5, 0.9], strict=False)
    both(x, u, t=[0.0] * 4)
    raw[:] = bits[0]
    assert M.sample(x, torch.tensor(u).cuda())[0].tolist() == [-1] * 4


@pytest.mark.parametrize("V", [900, 70001])
def test_random_numbers_out_of_range(V):
    """1 and more pick the last kept token, 0 and less and NaN the first."""
    u = [1.0, 1.5, 2.0 ** 22, 1e10, 1e30, 3.4e38, math.inf, 0.0, -0.0, -1e30, -math.inf, math.nan, -LEAST, LEAST]
    x = torch.zeros(len(u), V).cuda()
    x[:, ::2] = -1.0
    for o in ({}, dict(k=[30] * len(u)), dict(p=[0.5] * len(u)), dict(m=[0.9] * len(u))):
        got = both(x, u, strict=False, **o).tolist()
        assert len(set(got[:7])) == 1 and len(set(got[7:])) == 1 and got[0] > got[7], got
