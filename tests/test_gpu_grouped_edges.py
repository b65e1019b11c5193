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


def test_a_ragged_group_after_more_than_a_second_of_whole_steps():
    """The weights' gradient on pairs of CTAs. A group whose size is no multiple of 16 needs
    the second CTA's help at its last stage only; here more than a second's work (2 10^15
    operations) on a group that needs none comes before it, and no wait may run out. The
    rows are the same buffer on both sides, so that they fit."""
    rows, tail, width = 1_000_000, 17, 32768
    x = torch.empty(rows + tail, width, dtype=BF, device="cuda").normal_()
    off = torch.tensor([0, rows, rows + tail], dtype=torch.int32, device="cuda")
    sh = M.grouped_shape(rows + tail, 2, width, width, BF)
    ws = M.grouped_workspace(sh)
    dw = torch.full((2, width, width), -77.0, dtype=BF, device="cuda")
    M.moe_grouped_gemm_wgrad(sh, x, x, None, off, dw, ws)
    assert M.moe_get_device_status(ws) == 0
    pick = torch.arange(5, width, 1021, device="cuda")
    for e, (lo, hi) in enumerate(((0, rows), (rows, rows + tail))):
        ref = torch.zeros(len(pick), len(pick), dtype=torch.float64, device="cuda")
        size = torch.zeros_like(ref)
        for at in range(lo, hi, 1 << 16):
            part = x[at:min(at + (1 << 16), hi)][:, pick].double()
            ref += part.t() @ part
            size += part.abs().t() @ part.abs()
        got = dw[e][pick][:, pick].double()
        # parts of 512 rows (32 steps of 17 terms that each may lose 2^-24 of the part's sum of
        # magnitudes), added in fp32 one after the other: half an ulp of at most `size` each
        L = hi - lo
        tol = 2.0 ** -8 * (1 + 2.0 ** -6) * ref.abs() + (17 * 33 + L / 512 + 1) * 2.0 ** -24 * size
        assert ((got - ref).abs() <= tol).all()
    del x, dw
    torch.cuda.empty_cache()
