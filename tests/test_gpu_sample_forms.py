"""One workgroup a row and several: the same tokens and the same bits."""
import pytest
import torch

from routed_token_indexer_amd import _lib as M
from test_gpu_sample import rows, uniform

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [65536, 70001, 200003])
def test_a_row_by_itself_and_in_a_batch(V, dtype):
    """A row alone is shared by up to 32 workgroups, in a batch of 129 and more it has one; between, some."""
    T = 129
    assert M.sample_workspace_bytes(T, V) == 0 and M.sample_workspace_bytes(1, V) > 0
    x = rows(T, V, dtype, V, pad=3)
    x[5] = 1.0                                     # more ties than a workgroup lists
    x[6] = (x[6].float() / 4).round().to(x.dtype)
    g = torch.Generator().manual_seed(V)
    dev = lambda t: t.cuda()   # noqa: E731
    u = dev(torch.tensor(uniform(T, V)))
    t = dev(0.5 + torch.rand(T, generator=g))
    k = dev(torch.randint(0, 3000, (T,), generator=g, dtype=torch.int32))
    p = dev(0.3 + 0.8 * torch.rand(T, generator=g))
    m = dev(0.02 * torch.rand(T, generator=g))
    t[7], k[8], p[8], k[5], p[6] = 0.0, 0, 1.0, V // 3, 0.99
    for names in ((), ("top_p",), ("top_k",), ("min_p",), ("temperature", "top_k", "top_p", "min_p")):
        o = {n: v for n, v in dict(temperature=t, top_k=k, top_p=p, min_p=m).items() if n in names}
        whole = M.sample(x, u, want_logprob=True, **o)
        for a, b in ((0, 1), (5, 6), (6, 7), (7, 8), (8, 9), (0, 3), (3, 33), (29, 129), (1, 129)):
            part = M.sample(x[a:b], u[a:b], want_logprob=True, **{n: v[a:b] for n, v in o.items()})
            assert torch.equal(part[0], whole[0][a:b]) and torch.equal(part[1], whole[1][a:b]), (names, a, b)
