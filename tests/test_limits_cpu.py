"""Calls whose launches or scores the device cannot hold are refused before anything is
enqueued (no GPU is needed)."""
import os

import pytest

from test_attend_cpu import B, FAKE, LIB, append, attend, cache, err, selected, shared   # noqa: F401  (B is a fixture)

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libmisa.so not built")


@pytest.mark.parametrize("c,N,o", [
    (dict(heads=4, d=1024, page_stride=1 << 20, token_stride=4096, head_stride=1024), 1 << 24, dict(Hq=0, q=None, q_out=None)),
    (dict(heads=2, d=128), (1 << 31) - 1, dict(Hq=64)),
    (dict(heads=1, d=128, v=None), (1 << 31) - 1, dict(v=None, Hq=15)),
])
def test_appends_of_too_many_tokens(B, c, N, o):   # noqa: F811
    """2^24 workgroups of 256 threads: one token a workgroup, and several."""
    assert append(B, cache(B, **c), N=N, rot=0, **o) == -1 and "grid" in err(B)


@pytest.mark.parametrize("call", [attend, selected, shared])
def test_scales_that_scores_cannot_take(B, call):   # noqa: F811
    """Scores are fp32: a scale that takes ordinary products past 1e8 leaves nothing of their differences."""
    for scale in (1.1e4, 1e6, 1e30):
        assert call(B, cache(B), out=2 * FAKE, scale=scale) == -1 and "scale" in err(B)
