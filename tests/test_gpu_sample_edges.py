"""Sampling at the edges of its numbers: signalling NaN."""
import pytest
import torch

from routed_token_indexer_amd import _lib as M
from test_gpu_sample import both, rows, uniform

pytestmark = pytest.mark.gpu


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
