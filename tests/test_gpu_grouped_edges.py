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


# block scales whose sums below are exact: 1 to 4, 2^-9 to 2^-7, 64 to 256 (E4M3)
BLOCK_SCALES = {"small": [1, 2, 4], "one": [0x38, 0x40, 0x48], "large": [0x68, 0x70, 0x78]}


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("blocks", list(BLOCK_SCALES))
def test_product_with_tensor_scales_far_from_one(blocks, dt):
    """The tensor scales' product leaves fp32's range on either side while the results may
    not. Sums are whole multiples of 21 bits at most, so they are exact, and scales that are
    powers of two leave one rounding (to a subnormal, or to bf16); the last two pairs add
    that of their product and that of the sum's product with it, 2^-24 each."""
    gen = torch.Generator().manual_seed(3)
    rows, n, k = 80, 72, 800
    xc = torch.randint(0, 256, (rows, k // 2), generator=gen).to(U8).cuda()
    wc = torch.randint(0, 256, (2, n, k // 2), generator=gen).to(U8).cuda()
    xc[[0, 50]] = 0  # sums of zero
    s = torch.tensor(BLOCK_SCALES[blocks], dtype=U8)
    xs = s[torch.randint(0, 3, (rows, k // 16), generator=gen)].cuda()
    wsc = s[torch.randint(0, 3, (2, n, k // 16), generator=gen)].cuda()
    sums = torch.empty(rows, n, dtype=torch.float64, device="cuda")
    x, w = torch.empty(rows, k, device="cuda"), torch.empty(2, n, k, device="cuda")
    M.moe_dequantize_microscaled(NV, xc, xs, None, x)
    M.moe_dequantize_microscaled(NV, wc, wsc, None, w)
    off = torch.tensor([0, 33, 80], dtype=torch.int32, device="cuda")
    sums[:33], sums[33:] = x[:33].double() @ w[0].double().t(), x[33:].double() @ w[1].double().t()
    sh = M.grouped_shape(rows, 2, n, k, dt)
    ws = M.grouped_workspace(sh)
    lo, hi = 2.0 ** -100, 2.0 ** 117
    pairs = [(2.0 ** 70, 2.0 ** 70, 2.0 ** 58), (2.0 ** -75, 2.0 ** -75, 2.0 ** -58), (lo, lo, 2.0 ** -30), (hi, hi, 1.0),
             (hi, lo, hi), (lo, hi, lo), (2.0 ** -60, 2.0 ** -68, 2.0 ** -90), (1.0, 2.0 ** -20, 3.0),
             (1.3 * 2.0 ** -64, 1.7 * 2.0 ** -66, 1.9 * 2.0 ** -70), (1.3 * 2.0 ** 64, 1.7 * 2.0 ** 65, 1.1 * 2.0 ** 66)]
    for gx, ga, gb in pairs:
        xg, wg = torch.tensor([gx], device="cuda"), torch.tensor([ga, gb], device="cuda")
        y = torch.full((rows, n), -77.0, dtype=dt, device="cuda")
        M.moe_grouped_gemm_microscaled(sh, NV, xc, xs, xg, None, off, wc, wsc, wg, y, ws)
        assert M.moe_get_device_status(ws) == 0
        ref = sums * xg.double() * wg.double()[[0] * 33 + [1] * 47].unsqueeze(1)
        if (gx, ga, gb) in pairs[:-2] and gb != 3.0:
            assert torch.equal(y, ref.float().to(dt)), (gx, ga, gb)
        else:
            fits = ref.abs() < torch.finfo(dt).max
            tol = (2.0 ** -23 + (2.0 ** -8 if dt == BF else 2.0 ** -24)) * (1 + 2.0 ** -6) * ref.abs() + 2.0 ** -133
            assert ((y.double() - ref).abs() <= tol)[fits].all(), (gx, ga, gb)
            assert torch.isinf(y[ref.abs() > 2.0 ** 129]).all()


# fp32 results of long sums: the tensor core may lose up to an ulp of the running sum a step
# towards zero, over many elements half of one on average; with terms of one sign the sum
# grows evenly, so a part of s steps loses at most s/4 2^-23 of itself in the norm. The parts
# are added to nearest, half an ulp of at most the whole each.
def long_sum_bound(steps, parts):
    return steps / 4 * 2.0 ** -23 + parts * 2.0 ** -24


def relative(got, ref):
    return ((got.double() - ref).norm() / ref.norm()).item()


@pytest.mark.parametrize("fmt", [NV, MX], ids=["nv", "mx"])
@pytest.mark.parametrize("counts,n", [([3], 64), ([40, 70], 256), ([700, 300], 2048)], ids=["few", "rows", "pairs"])
@pytest.mark.parametrize("k", [32768, 16416, 6176])
def test_product_of_long_sums_in_fp32(fmt, counts, n, k):
    """Parts of 8192 terms (128 steps), on every layout of a tile; 16416 ends inside a part."""
    gen = torch.Generator(device="cuda").manual_seed(k)
    total, E, b = sum(counts), len(counts), 16 if fmt == NV else 32

    def operand(*shape):
        v = torch.rand(*shape, generator=gen, device="cuda") + 0.1
        v *= torch.exp2(torch.randint(-6, 7, (*shape[:-1], 1), generator=gen, device="cuda").float())
        codes = torch.empty(*shape[:-1], k // 2, dtype=U8, device="cuda")
        scales = torch.empty(*shape[:-1], k // b, dtype=U8, device="cuda")
        M.moe_quantize_microscaled(fmt, v, None, codes, scales)
        M.moe_dequantize_microscaled(fmt, codes, scales, None, v)
        return codes, scales, v.double()

    xc, xs, x = operand(total, k)
    wc, wsc, w = operand(E, n, k)
    ends = torch.tensor([0] + counts).cumsum(0)
    sh = M.grouped_shape(total, E, n, k, F32)
    ws = M.grouped_workspace(sh)
    cases = [(xs, x, wsc, w, 1.0, 1.0)]
    if fmt == NV:
        cases.append((xs, x, wsc, w, 0.75, 0.6))
        # block scales of 2^-9 on both sides and tensor scales whose product is no fp32 number
        xs1, ws1, x1, w1 = torch.ones_like(xs), torch.ones_like(wsc), x.float(), w.float()
        M.moe_dequantize_microscaled(NV, xc, xs1, None, x1)
        M.moe_dequantize_microscaled(NV, wc, ws1, None, w1)
        cases.append((xs1, x1.double(), ws1, w1.double(), 2.0 ** 66, 2.0 ** 63))
    off = ends.int().cuda()
    for xs, x, wsc, w, gx, gw in cases:
        xg, wg = torch.tensor([gx], device="cuda"), torch.full((E,), gw, device="cuda")
        y = torch.full((total, n), -77.0, device="cuda")
        M.moe_grouped_gemm_microscaled(sh, fmt, xc, xs, xg if fmt == NV else None, None, off, wc, wsc,
                                       wg if fmt == NV else None, y, ws)
        assert M.moe_get_device_status(ws) == 0
        for e in range(E):
            lo, hi = int(ends[e]), int(ends[e + 1])
            ref = x[lo:hi] @ w[e].t() * (xg.double() * wg[e].double())
            got = y[lo:hi]
            # sums of up to 32768 36 2^-18 times 2^129 pass fp32's largest number: those are infinite
            above = ref > torch.finfo(F32).max * (1 + 2.0 ** -18)
            assert torch.isinf(got[above]).all()
            below = ref < torch.finfo(F32).max * (1 - 2.0 ** -18)
            if below.any():  # (and 2^-24 each for the tensor scales' product and for the sum's with it)
                assert relative(got[below], ref[below]) <= long_sum_bound(128, -(-k // 8192)) + 2.0 ** -23


def test_products_of_long_sums_in_fp32():
    """The 16-bit products: parts of 512 terms (32 steps), over the width and over the rows."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    positive = lambda *s: (torch.rand(*s, generator=gen, device="cuda") + 0.1).to(BF)  # noqa: E731
    for rows, n, k in ((130, 264, 8192), (130, 8192, 264), (8200, 264, 256), (8200, 1024, 1024)):
        x, dy, w = positive(rows, k), positive(rows, n), positive(1, n, k)
        off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
        sh = M.grouped_shape(rows, 1, n, k, F32)
        ws = M.grouped_workspace(sh)
        y, dx = torch.empty(rows, n, device="cuda"), torch.empty(rows, k, device="cuda")
        dw = torch.empty(1, n, k, device="cuda")
        M.moe_grouped_gemm(sh, x, None, off, w, y, ws)
        M.moe_grouped_gemm_dgrad(sh, dy, None, off, w, dx, ws)
        M.moe_grouped_gemm_wgrad(sh, dy, x, None, off, dw, ws)
        assert M.moe_get_device_status(ws) == 0
        xd, dyd, wd = x.double(), dy.double(), w[0].double()
        assert relative(y, xd @ wd.t()) <= long_sum_bound(32, -(-k // 512))
        assert relative(dx, dyd @ wd) <= long_sum_bound(32, -(-n // 512))
        assert relative(dw[0], dyd.t() @ xd) <= long_sum_bound(32, -(-rows // 512))


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("how", ["packed", "padded", "gaps", "slack"])
@pytest.mark.parametrize("counts,k", [([1], 32), ([0, 1, 127, 128, 129, 300, 0, 5], 96), ([40] * 64, 2048), ([0, 0], 64),
                                      ([3000, 1, 0, 77], 1056), ([2] * 256, 512)], ids=lambda c: str(c)[:12])
def test_tensor_scale_of_owned_rows(counts, k, how, dt):
    """Bit for bit; rows without an owner hold large numbers and NaN."""
    from tests.test_gpu_ragged import layout
    gs, off, starts, total = layout(counts, how)
    x = torch.full((total, k), 1e30, dtype=dt, device="cuda")
    x[::2] = float("nan")
    amax = torch.zeros(1, device="cuda")
    for i, (s, c) in enumerate(zip(starts, counts)):
        rows = torch.randn(c, k, device="cuda") * 2.0 ** (i % 5)
        if c > 3:
            rows[1, 0], rows[2, k - 1] = float("inf"), float("nan")
        x[s:s + c] = rows.to(dt)
        finite = torch.where(torch.isfinite(x[s:s + c]), x[s:s + c], torch.zeros_like(x[s:s + c]))
        if c:
            amax = torch.maximum(amax, finite.float().abs().max())
    sh = M.grouped_shape(total, len(counts), 8, k)
    ws = M.grouped_workspace(sh)
    g = torch.full((1,), -5.0, device="cuda")
    for _ in range(2):
        M.moe_grouped_tensor_scale_microscaled(sh, x, gs, off, g, ws)
        assert M.moe_get_device_status(ws) == 0
        assert torch.equal(g, tensor_scale(amax))


def test_tensor_scale_of_owned_rows_without_rows_and_with_bad_groups():
    sh, ws = M.grouped_shape(0, 2, 8, 64), M.grouped_workspace()
    g = torch.full((1,), -5.0, device="cuda")
    none = torch.zeros(3, dtype=torch.int32, device="cuda")
    M.moe_grouped_tensor_scale_microscaled(sh, torch.empty(0, 64, device="cuda"), None, none, g, ws)
    assert M.moe_get_device_status(ws) == 0 and g.item() == 2.0 ** -100
    sh = M.grouped_shape(10, 2, 8, 64)
    x = torch.ones(10, 64, device="cuda")
    x[4:] = 9.0
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    for gs, off in ((None, i32(0, 4, 11)), (i32(0, -1, 0), i32(0, 4, 6)), (i32(0, 9, 0), i32(0, 4, 6)), (None, i32(0, 4, 2))):
        M.moe_grouped_tensor_scale_microscaled(sh, x, gs, off, g, ws)
        assert M.moe_get_device_status(ws) == 0x203
        assert torch.equal(g, tensor_scale(torch.ones(1, device="cuda")))


def test_quantised_product_on_a_buffer_with_leftovers():
    """moe_dispatch leaves the rows behind the last group as they were. Whatever an earlier
    step, or nobody, left there: the same tokens give the same product, bit for bit, in a
    call captured once."""
    T, E, top, d, f = 24, 8, 2, 256, 320
    gen = torch.Generator().manual_seed(9)
    cfg = M.config(T, d, E, top, 128)
    P = M.moe_padded_rows(cfg)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    off, gs, perm, inv = i32(E + 1), i32(E + 1), i32(T * top), i32(T * top)
    idx = torch.stack([torch.randperm(E, generator=gen)[:top] for _ in range(T)]).to(torch.int32).cuda()
    x = torch.randn(T, d, generator=gen).to(BF).cuda()
    xp = torch.zeros(P, d, dtype=BF, device="cuda")
    w = (torch.randn(E, f, d, generator=gen) * 0.02).to(BF).cuda()
    wg, wc = torch.empty(E, device="cuda"), torch.empty(E, f, d // 2, dtype=U8, device="cuda")
    wsc = torch.empty(E, f, d // 16, dtype=U8, device="cuda")
    M.moe_tensor_scale_microscaled(w, wg)
    M.moe_quantize_microscaled(NV, w, wg, wc, wsc)
    xg, xc = torch.empty(1, device="cuda"), torch.empty(P, d // 2, dtype=U8, device="cuda")
    xs = torch.empty(P, d // 16, dtype=U8, device="cuda")
    y = torch.zeros(P, f, dtype=BF, device="cuda")
    sh = M.grouped_shape(P, E, f, d)
    ws, lws = M.grouped_workspace(sh), M.workspace(cfg)

    def go():
        M.moe_dispatch(cfg, idx, x, off, perm, inv, gs, xp, lws)
        M.moe_grouped_tensor_scale_microscaled(sh, xp, gs, off, xg, ws)
        M.moe_quantize_microscaled(NV, xp, xg, xc, xs)
        M.moe_grouped_gemm_microscaled(sh, NV, xc, xs, xg, gs, off, wc, wsc, wg, y, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    want = None
    for left in (0.0, 1e30, float("nan"), float("inf"), 3.0):
        xp.fill_(left)
        y.zero_()
        graph.replay()
        assert M.moe_get_device_status(ws) == 0 and M.moe_get_device_status(lws) == 0
        assert torch.equal(xg, tensor_scale(x.float().abs().max().reshape(1)))
        want = y.clone() if want is None else want
        assert torch.equal(y, want) and y[inv.long()].abs().max() > 0
