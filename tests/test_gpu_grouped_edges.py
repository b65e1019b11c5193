"""Edges of the ragged products and the 4-bit operators: clusters whose CTAs start
unevenly, long waits, tensor scales far from 1, long sums, rows that no expert owns."""

import pytest
import torch

import sparse_moe_transformer_route_b200 as M
from tests._parity import require_gpu

pytestmark = pytest.mark.gpu

BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
NV, MX = M.MOE_NVFP4, M.MOE_MXFP4


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def tensor_scale(amax):
    """max(amax / 2688, 2^-100), rounded once."""
    return torch.clamp((amax.double() / torch.full_like(amax, 2688).double()).float(), min=2.0 ** -100)


def test_tensor_scale_clusters_that_start_unevenly():
    """Groups on clusters of two to eight CTAs of which the last has next to nothing to read
    (so that it is done at once), many clusters, launched while other streams keep the SMs
    busy: a cluster's CTAs need not start together."""
    streams = [torch.cuda.Stream() for _ in range(4)]
    busy = torch.randn(2048, 2048, device="cuda").to(BF)
    cases = []
    for ctas in (2, 3, 5, 8):
        for dt in (BF, F32):
            turn = 4 * 256 * (256 // torch.finfo(dt).bits)  # elements a CTA takes at a time
            x = torch.randn(200, ((ctas - 1) * turn + 32) // 32, 32, device="cuda").to(dt)
            x[:, -1, -1] = torch.arange(10, 210, device="cuda").to(dt)  # in the last CTA's share
            cases.append((x, torch.empty(200, device="cuda")))
    torch.cuda.synchronize()
    for _ in range(20):
        for i, (x, g) in enumerate(cases):
            with torch.cuda.stream(streams[i % 4]):
                busy @ busy
                M.moe_tensor_scale_microscaled(x, g)
    torch.cuda.synchronize()
    for x, g in cases:
        assert torch.equal(g, tensor_scale(x.float().flatten(1).abs().amax(1)))
