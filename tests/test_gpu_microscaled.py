"""Microscaled 4-bit values and the products on them against their definition.

Conversions are compared bit for bit: every decision (a block's scale, an element's
code) is a comparison of numbers that fp64 holds exactly or separates, so the
reference below has no rounding of its own. The product's operands are exact; the
tensor core adds 64 products to the fp32 accumulator a step, each of the 65 terms may
lose what lies below 2^-23 of the step's largest, at most S = sum |a||b|: off by at
most 65 (k/64 + 1) 2^-23 S before the tensor scales (a product of two, 2 roundings of
2^-24) and the result's rounding, eps/2 of the value.
"""

import pytest
import torch

import sparse_moe_transformer_route_b200 as M
from tests._parity import require_gpu

pytestmark = pytest.mark.gpu

BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
NV, MX = M.MOE_NVFP4, M.MOE_MXFP4
BLOCK = {NV: 16, MX: 32}
GRID = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
E4M3 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()  # 0 .. 448


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def nearest(v, table):
    """Index of the number in an increasing table nearest to v >= 0 (fp64), ties to the
    even index, capped at the last."""
    hi = torch.searchsorted(table, v.contiguous()).clamp(1, len(table) - 1)
    lo = hi - 1
    mid = (table[lo] + table[hi]) / 2
    up = (v > mid) | ((v == mid) & (lo % 2 == 1))
    return torch.where(up, hi, lo)


def ref_quantize(x, g, fmt):
    """Codes and scale bytes of [G, R, K] on the CPU; g [G] fp64 or None."""
    G, R, K = x.shape
    b = BLOCK[fmt]
    xb = x.cpu().double().reshape(G, R, K // b, b)
    bad = ~torch.isfinite(xb).all(-1)
    xb = torch.where(bad.unsqueeze(-1), torch.zeros_like(xb), xb)
    amax = xb.abs().amax(-1)
    if fmt == MX:
        e = torch.where(amax > 0, torch.frexp(amax).exponent - 3, -127).clamp(-127, 127)
        sbyte = (e + 127).to(U8)
        unit = torch.ldexp(torch.ones_like(amax), e)
        sbyte[bad] = 255
    else:
        gg = (torch.ones(G, dtype=torch.float64) if g is None else g.cpu().double()).reshape(G, 1, 1)
        bad = bad | ~((gg >= 2.0 ** -100) & (gg <= 2.0 ** 117))
        gg = torch.where((gg >= 2.0 ** -100) & (gg <= 2.0 ** 117), gg, torch.ones_like(gg))
        i = nearest(amax / (6 * gg), E4M3)
        sbyte = i.to(U8)
        unit = E4M3[i] * gg
        sbyte[bad] = 127
    u = unit.unsqueeze(-1)
    # a border times the unit has at most 31 bits: comparing x with it is exact
    code = torch.zeros(xb.shape, dtype=torch.int64)
    for j in range(7):
        at = (GRID[j] + GRID[j + 1]) / 2 * u
        code += torch.where(u > 0, (xb.abs() >= at) if j % 2 else (xb.abs() > at), False).long()
    code = code + 8 * torch.signbit(xb).long()
    code[bad] = 0
    return code.reshape(G, R, K), sbyte


def ref_dequantize(code, sbyte, g, fmt, dtype):
    b = BLOCK[fmt]
    G, R, K = code.shape
    v = torch.where(code >= 8, -GRID[code % 8], GRID[code % 8])
    s = sbyte.long()
    if fmt == MX:
        scale = torch.ldexp(torch.ones(s.shape, dtype=torch.float64), (s - 127).clamp(-127, 127))
        scale[s == 255] = float("nan")
    else:
        scale = E4M3[s.clamp(max=126)].clone()
        scale[s == 127] = float("nan")
        if g is not None:
            scale = scale * g.cpu().double().reshape(G, 1, 1)
    out = v.reshape(G, R, K // b, b) * scale.unsqueeze(-1)
    return out.reshape(G, R, K).to(torch.float32).to(dtype)


def unpack(codes):
    c = codes.cpu().long()
    return torch.stack((c & 15, c >> 4), -1).flatten(-2)


def quantize(x, g, fmt):
    G, R, K = x.shape
    codes = torch.full((G, R, K // 2), 0xA5, dtype=U8, device="cuda")
    scales = torch.full((G, R, K // BLOCK[fmt]), 0xA5, dtype=U8, device="cuda")
    M.moe_quantize_microscaled(fmt, x, g, codes, scales)
    return codes, scales


def same(codes, want):
    """Codes agree; which zero a value became does not matter (0 and -0 stand for the same)."""
    got = unpack(codes)
    got, want = torch.where(got == 8, 0, got), torch.where(want == 8, 0, want)
    assert torch.equal(got, want), (got != want).nonzero()[:5].tolist()


def sample(shape, dtype, kind, seed):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=gen)
    if kind == "wide":  # magnitudes over the whole range of the type
        x = x * torch.exp2(torch.randint(-140, 126, shape, generator=gen).float())
        x[..., ::7] = 0
    elif kind == "blocks":  # each block its own magnitude, some blocks zero
        m = torch.exp2(torch.randint(-30, 30, (*shape[:-1], shape[-1] // 16), generator=gen).float())
        m[torch.rand(m.shape, generator=gen) < 0.1] = 0
        x = x * m.repeat_interleave(16, -1)
    elif kind == "ties":  # elements on and next to the borders of a block whose amax is 6 s
        pick = torch.tensor([0., .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6])
        i = torch.randint(0, 15, shape, generator=gen)
        x = pick[i] * torch.sign(x)
        x[..., ::16] = 6.0
        step = torch.randint(-1, 2, shape, generator=gen).float()
        x = x * (1 + step * (2.0 ** -8 if dtype == BF else 2.0 ** -23))
    return x.to(dtype).cuda()


@pytest.mark.parametrize("fmt", [NV, MX], ids=["nv", "mx"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["normal", "wide", "blocks", "ties"])
@pytest.mark.parametrize("shape", [(1, 1, 32), (1, 3, 96), (3, 37, 160), (2, 129, 2048), (70, 5, 64)],
                         ids=lambda s: "x".join(map(str, s)))
def test_quantize_and_back_bit_for_bit(fmt, dtype, kind, shape):
    x = sample(shape, dtype, kind, seed=len(kind) + shape[1])
    tensor_scales = [None]
    if fmt == NV:
        g = torch.empty(shape[0], device="cuda")
        M.moe_tensor_scale_microscaled(x, g)
        amax = x.float().flatten(1).abs().amax(1)
        want = torch.clamp((amax.cpu().double() / 2688).float(), min=2.0 ** -100)
        assert torch.equal(g.cpu(), want)
        tensor_scales += [g, torch.rand(shape[0], device="cuda") * 1e-3 + 1e-4]
    for g in tensor_scales:
        codes, scales = quantize(x, g, fmt)
        want_c, want_s = ref_quantize(x, g, fmt)
        assert torch.equal(scales.cpu(), want_s)
        same(codes, want_c)
        for odt in (BF, F32):
            out = torch.full(shape, 9.0, dtype=odt, device="cuda")
            M.moe_dequantize_microscaled(fmt, codes, scales, g, out)
            assert torch.equal(out.cpu(), ref_dequantize(unpack(codes), scales.cpu(), g, fmt, odt))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_block_scale_borders(dtype):
    """Blocks whose amax puts the scale on and next to every border between E4M3 numbers."""
    mid = (E4M3[:-1] + E4M3[1:]) / 2
    for g in (1.0, 0.37, 2.0 ** -100, 3e20):
        gt = torch.tensor([g], dtype=F32)
        at = (mid * 6 * gt.double()).to(F32)
        near = torch.stack([torch.nextafter(at, torch.tensor(0.)), at, torch.nextafter(at, torch.tensor(float("inf")))])
        x = torch.zeros(1, near.numel(), 32)
        x[0, :, 0] = near.flatten()
        x[0, :, 16] = -near.flatten()
        x[0, :, 5] = near.flatten() / 3
        x = x.to(dtype).cuda()
        codes, scales = quantize(x, gt.cuda(), NV)
        want_c, want_s = ref_quantize(x, gt, NV)
        assert torch.equal(scales.cpu(), want_s)
        same(codes, want_c)


@pytest.mark.parametrize("fmt", [NV, MX], ids=["nv", "mx"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_infinities_nan_and_extremes(fmt, dtype):
    x = torch.randn(1, 8, 96)
    x[0, 0, 3] = float("nan")
    x[0, 1, 40] = float("inf")
    x[0, 2, 95] = -float("inf")
    x[0, 3] = torch.finfo(dtype).max
    x[0, 4] = -torch.finfo(dtype).tiny
    x[0, 5] = 1e-45 if dtype == F32 else 2.0 ** -133
    x[0, 6] = 0
    x = x.to(dtype).cuda()
    g = torch.empty(1, device="cuda")
    M.moe_tensor_scale_microscaled(x, g)
    assert g.item() == (torch.tensor(torch.finfo(dtype).max, dtype=torch.float64) / 2688).float().item()
    for ts in ([None, g] if fmt == NV else [None]):
        codes, scales = quantize(x, ts, fmt)
        want_c, want_s = ref_quantize(x, ts, fmt)
        assert torch.equal(scales.cpu(), want_s)
        same(codes, want_c)
        out = torch.empty(1, 8, 96, device="cuda")
        M.moe_dequantize_microscaled(fmt, codes, scales, ts, out)
        torch.testing.assert_close(out.cpu(), ref_dequantize(unpack(codes), scales.cpu(), ts, fmt, F32), rtol=0, atol=0,
                                   equal_nan=True)
        b = BLOCK[fmt]
        nan = torch.isnan(out[0]).cpu().reshape(8, -1, b).any(-1)
        want = torch.zeros_like(nan)
        want[0, 3 // b] = want[1, 40 // b] = want[2, 95 // b] = True
        assert torch.equal(nan, want)


def test_tensor_scales_out_of_range_read_back_as_nan():
    x = torch.randn(5, 4, 64, device="cuda")
    g = torch.tensor([1.0, 0.0, float("nan"), 2.0 ** 118, -1.0], device="cuda")
    codes, scales = quantize(x, g, NV)
    assert (scales[1:] == 127).all() and (scales[0] != 127).all()
    out = torch.empty_like(x)
    M.moe_dequantize_microscaled(NV, codes, scales, g, out)
    assert torch.isnan(out[1:]).all() and torch.isfinite(out[0]).all()


def test_no_rows_and_two_dimensions():
    x = torch.empty(0, 64, dtype=BF, device="cuda")
    e = torch.empty(0, 32, dtype=U8, device="cuda")
    g = torch.zeros(1, device="cuda")
    M.moe_tensor_scale_microscaled(x, g)
    assert g.item() == 2.0 ** -100
    M.moe_quantize_microscaled(NV, x, g, e, torch.empty(0, 4, dtype=U8, device="cuda"))
    M.moe_dequantize_microscaled(MX, e, torch.empty(0, 2, dtype=U8, device="cuda"), None, x)
    x = torch.randn(3, 64, device="cuda")
    c, s = torch.empty(3, 32, dtype=U8, device="cuda"), torch.empty(3, 4, dtype=U8, device="cuda")
    M.moe_quantize_microscaled(NV, x, None, c, s)
    want_c, want_s = ref_quantize(x.unsqueeze(0), None, NV)
    assert torch.equal(s.cpu(), want_s[0])
    same(c, want_c[0])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("fmt", [NV, MX], ids=["nv", "mx"])
def test_buffers_that_start_at_a_multiple_of_16_only(fmt, dtype):
    """The wide side of a conversion is accessed 32 bytes at a time where it is aligned so."""
    R, K = 37, 96
    skip = 128 // torch.finfo(dtype).bits  # elements of 16 bytes
    held = torch.randn(skip + R * K, device="cuda").to(dtype)
    x = held[skip:].view(1, R, K)
    assert x.data_ptr() % 32 == 16
    g = None
    if fmt == NV:
        g = torch.empty(1, device="cuda")
        M.moe_tensor_scale_microscaled(x, g)
        assert g.item() == max((x.float().abs().max().double() / torch.tensor(2688.0).double()).float().item(), 2.0 ** -100)
    codes, scales = quantize(x, g, fmt)
    want_c, want_s = ref_quantize(x, g, fmt)
    assert torch.equal(scales.cpu(), want_s)
    same(codes, want_c)
    held2 = torch.full((skip + R * K + skip,), 5.0, device="cuda").to(dtype)
    out = held2[skip:-skip].view(1, R, K)
    M.moe_dequantize_microscaled(fmt, codes, scales, g, out)
    assert torch.equal(out.cpu(), ref_dequantize(unpack(codes), scales.cpu(), g, fmt, dtype))
    assert torch.all(held2[:skip] == 5.0) and torch.all(held2[-skip:] == 5.0)


def test_tensor_scale_of_many_sizes():
    """One CTA a group and many; results do not depend on the run."""
    for shape in ((1, 1, 32), (1, 5000, 2048), (300, 2, 32), (70000, 1, 32), (3, 999, 1056)):
        for dt in (BF, F32):
            x = torch.randn(shape, device="cuda").to(dt)
            x[0, 0, 1] = float("inf")
            g = torch.full((shape[0],), -5.0, device="cuda")
            M.moe_tensor_scale_microscaled(x, g)
            amax = torch.where(torch.isfinite(x), x, torch.zeros_like(x)).float().flatten(1).abs().amax(1)
            want = torch.clamp((amax.double() / torch.full_like(amax, 2688).double()).float(), min=2.0 ** -100)
            assert torch.equal(g, want)


# ---------------------------------------------------------------- product


def operands(counts, n, k, fmt, total, seed, scaled=True):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    E = len(counts)
    x = torch.randn(1, total, k, generator=gen, device="cuda")
    w = torch.randn(E, n, k, generator=gen, device="cuda") * 0.05
    xg = wg = None
    if fmt == NV and scaled:
        xg, wg = torch.empty(1, device="cuda"), torch.empty(E, device="cuda")
        M.moe_tensor_scale_microscaled(x, xg)
        M.moe_tensor_scale_microscaled(w, wg)
    xc, xs = quantize(x, xg, fmt)
    wc, wsc = quantize(w, wg, fmt)
    return xc[0], xs[0], xg, wc, wsc, wg


def values(codes, scales, g, fmt):
    out = torch.empty(*codes.shape[:-1], codes.shape[-1] * 2, device="cuda")
    M.moe_dequantize_microscaled(fmt, codes.clone(), scales.clone(), None, out)  # before the tensor scale: exact
    return out.double()


def run_product(counts, n, k, fmt, dt, how="packed", seed=0, scaled=True):
    from tests.test_gpu_ragged import SENTINEL, layout
    gs, off, starts, total = layout(counts, how)
    xc, xs, xg, wc, wsc, wg = operands(counts, n, k, fmt, total, seed, scaled)
    owned = torch.zeros(total, dtype=torch.bool, device="cuda")
    for s, c in zip(starts, counts):
        owned[s:s + c] = True
    xc[~owned] = 0x77
    xs[~owned] = 127 if fmt == NV else 255  # NaN: must not reach a neighbour
    sh = M.grouped_shape(total, len(counts), n, k, dt)
    ws = M.grouped_workspace(sh)
    y = torch.full((total, n), SENTINEL, dtype=dt, device="cuda")
    M.moe_grouped_gemm_microscaled(sh, fmt, xc, xs, xg, gs, off, wc, wsc, wg, y, ws)
    assert M.moe_get_device_status(ws) == 0
    assert torch.all(y[~owned] == SENTINEL)
    for e, (s, c) in enumerate(zip(starts, counts)):
        if c == 0:
            continue
        xe, we = values(xc[s:s + c], xs[s:s + c], None, fmt), values(wc[e], wsc[e], None, fmt)
        alpha = 1.0 if xg is None else xg.double().item() * wg[e].double().item()
        ref, S = xe @ we.t() * alpha, xe.abs() @ we.abs().t() * alpha
        tol = (torch.finfo(dt).eps / 2 * (1 + 2.0 ** -6) + 2.0 ** -22) * ref.abs() + 65 * (k / 64 + 1) * 2.0 ** -23 * S
        bad = ~((y[s:s + c].double() - ref).abs() <= tol + 1e-30)
        assert not bad.any(), f"expert {e}: {int(bad.sum())} of {bad.numel()}, first {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("fmt", [NV, MX], ids=["nv", "mx"])
@pytest.mark.parametrize("how", ["packed", "padded", "gaps", "slack"])
@pytest.mark.parametrize("n,k", [(8, 32), (72, 96), (256, 256), (264, 544), (640, 1056)])
def test_product_matches_64_bits(fmt, how, n, k):
    run_product([0, 1, 127, 128, 129, 300, 0, 5], n, k, fmt, BF if n % 16 else F32, how, seed=n)


@pytest.mark.parametrize("fmt", [NV, MX], ids=["nv", "mx"])
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("counts,n,k", [([1500, 0, 3, 700], 2048, 1024), ([40] * 64, 512, 256), ([3, 200], 264, 4096),
                                        ([1], 2048, 2048), ([900, 900], 1416, 1056)])
def test_product_matches_64_bits_larger(fmt, dt, counts, n, k):
    run_product(counts, n, k, fmt, dt, "gaps", seed=k)


@pytest.mark.parametrize("fmt", [NV, MX], ids=["nv", "mx"])
@pytest.mark.parametrize("n,k,how", [(4096, 2048, "packed"), (4104, 2080, "gaps")])
def test_product_of_large_groups_runs_on_pairs(fmt, n, k, how):
    run_product([700, 1, 650, 0, 1303, 704, 257, 2000], n, k, fmt, BF, how, seed=k)


@pytest.mark.parametrize("fmt", [NV, MX], ids=["nv", "mx"])
@pytest.mark.parametrize("mean,n,k", [(3, 512, 512), (30, 2048, 288), (80, 2048, 1024), (300, 128, 288), (300, 128, 512)])
def test_product_every_kind_of_tile(fmt, mean, n, k):
    g = torch.Generator().manual_seed(mean)
    counts = torch.poisson(torch.full((64,), float(mean)), generator=g).int().tolist()
    run_product(counts, n, k, fmt, BF, "packed", seed=mean)


@pytest.mark.parametrize("fmt", [NV, MX], ids=["nv", "mx"])
def test_product_of_most_experts(fmt):
    g = torch.Generator().manual_seed(6)
    run_product(torch.randint(0, 30, (256,), generator=g).tolist(), 72, 96, fmt, F32)


@pytest.mark.parametrize("k", [4096, 4128])
def test_product_far_rows(k):
    """Codes beyond 2^31 bytes, scales by TMA (4096) and through registers (4128)."""
    n, total = 16, (1 << 20) + 100
    xc = torch.zeros(total, k // 2, dtype=U8, device="cuda")
    xs = torch.zeros(total, k // 32, dtype=U8, device="cuda")
    spans = ((total - 70, 65), (3, 5))
    gs = torch.tensor([total - 70, 3, 0], dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 65, 70], dtype=torch.int32, device="cuda")
    x = torch.randn(1, 70, k, device="cuda")
    c, s = quantize(x, None, MX)
    for at, lo, hi in ((total - 70, 0, 65), (3, 65, 70)):
        xc[at:at + hi - lo], xs[at:at + hi - lo] = c[0, lo:hi], s[0, lo:hi]
    wc, wsc = quantize(torch.randn(2, n, k, device="cuda"), None, MX)
    sh = M.grouped_shape(total, 2, n, k, F32)
    ws = M.grouped_workspace(sh)
    y = torch.zeros(total, n, device="cuda")
    M.moe_grouped_gemm_microscaled(sh, MX, xc, xs, None, gs, off, wc, wsc, None, y, ws)
    assert M.moe_get_device_status(ws) == 0
    for e, (at, m) in enumerate(spans):
        xe, we = values(xc[at:at + m], xs[at:at + m], None, MX), values(wc[e], wsc[e], None, MX)
        ref, S = xe @ we.t(), xe.abs() @ we.abs().t()
        tol = 2.0 ** -24 * ref.abs() + 65 * (k / 64 + 1) * 2.0 ** -23 * S
        assert ((y[at:at + m].double() - ref).abs() <= tol).all()
    assert torch.all(y[8:total - 70] == 0) and torch.all(y[total - 5:] == 0)


@pytest.mark.parametrize("fmt", [NV, MX], ids=["nv", "mx"])
def test_product_is_exact_where_sums_are(fmt):
    """Whole numbers of few bits: every sum is exact, so any misplaced scale or code shows."""
    gen = torch.Generator().manual_seed(0)
    rows, n, k, E = 150, 272, 800, 2
    b = BLOCK[fmt]
    xc = torch.randint(0, 256, (rows, k // 2), generator=gen).to(U8).cuda()
    wc = torch.randint(0, 256, (E, n, k // 2), generator=gen).to(U8).cuda()
    if fmt == NV:  # 1, 2 and 4 in E4M3
        s = torch.tensor([0x38, 0x40, 0x48], dtype=U8)
    else:
        s = torch.tensor([127, 128, 129], dtype=U8)
    xs = s[torch.randint(0, 3, (rows, k // b), generator=gen)].cuda()
    wsc = s[torch.randint(0, 3, (E, n, k // b), generator=gen)].cuda()
    off = torch.tensor([0, 67, 150], dtype=torch.int32, device="cuda")
    sh = M.grouped_shape(rows, E, n, k, F32)
    ws = M.grouped_workspace(sh)
    y = torch.empty(rows, n, device="cuda")
    M.moe_grouped_gemm_microscaled(sh, fmt, xc, xs, None, None, off, wc, wsc, None, y, ws)
    assert M.moe_get_device_status(ws) == 0
    x, w = values(xc, xs, None, fmt), values(wc, wsc, None, fmt)
    # products are multiples of 1/4, at most 36 * 16, sums below 2^19: 21 bits
    assert torch.equal(y[:67].double(), x[:67] @ w[0].t())
    assert torch.equal(y[67:].double(), x[67:] @ w[1].t())


@pytest.mark.parametrize("fmt", [NV, MX], ids=["nv", "mx"])
def test_product_nan_scales_stay_in_their_rows(fmt):
    rows, n, k = 200, 136, 288
    xc, xs, xg, wc, wsc, wg = operands([90, 110], n, k, fmt, rows, 1)
    nan = 127 if fmt == NV else 255
    xs[100, 3] = nan
    wsc[0, 5, 1] = nan
    off = torch.tensor([0, 90, 200], dtype=torch.int32, device="cuda")
    sh = M.grouped_shape(rows, 2, n, k)
    ws = M.grouped_workspace(sh)
    y = torch.zeros(rows, n, dtype=BF, device="cuda")
    M.moe_grouped_gemm_microscaled(sh, fmt, xc, xs, xg, None, off, wc, wsc, wg, y, ws)
    want = torch.zeros(rows, n, dtype=torch.bool, device="cuda")
    want[100] = True
    want[:90, 5] = True
    assert torch.equal(torch.isnan(y), want)


def test_product_bad_group_and_no_rows():
    xc, xs, xg, wc, wsc, wg = operands([5, 5], 64, 64, NV, 10, 1)
    sh = M.grouped_shape(10, 2, 64, 64)
    ws = M.grouped_workspace(sh)
    y = torch.full((10, 64), 3.0, dtype=BF, device="cuda")
    for off, code in (([0, 5, 11], 0x203), ([0, 0, 0], 0)):
        M.moe_grouped_gemm_microscaled(sh, NV, xc, xs, xg, None, torch.tensor(off, dtype=torch.int32, device="cuda"), wc,
                                       wsc, wg, y, ws)
        assert M.moe_get_device_status(ws) == code
        assert torch.all(y[5:] == 3.0)
    sh0 = M.grouped_shape(0, 2, 64, 64)
    M.moe_grouped_gemm_microscaled(sh0, NV, xc[:0], xs[:0], xg, None, torch.zeros(3, dtype=torch.int32, device="cuda"),
                                   wc, wsc, wg, y[:0], ws)


def test_quantised_layer_products_in_a_graph():
    """A layer's gate/up product on 4 bits as it is served: rows quantised and multiplied
    on the device with the sizes a dispatch left there, captured once, replayed on other
    rows. The product must be what the stored operands give; the whole must be near the
    16-bit product: each operand is off by at most half a step of its format, and the
    relative L2 error of a product of two such operands is below the sum of theirs."""
    T, E, top, d, f = 160, 8, 2, 256, 320
    gen = torch.Generator().manual_seed(2)
    cfg = M.config(T, d, E, top, 128)
    P = M.moe_padded_rows(cfg)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    off, gs, perm, inv = i32(E + 1), i32(E + 1), i32(T * top), i32(T * top)
    idx = torch.arange(top, dtype=torch.int32, device="cuda").repeat(T, 1)  # top different experts
    x = torch.zeros(T, d, dtype=BF, device="cuda")
    xp = torch.zeros(P, d, dtype=BF, device="cuda")
    lws = M.workspace(cfg)
    w = (torch.randn(E, f, d, generator=gen) * 0.02).to(BF).cuda()
    wg, wc, wsc = torch.empty(E, device="cuda"), torch.empty(E, f, d // 2, dtype=U8, device="cuda"), torch.empty(
        E, f, d // 16, dtype=U8, device="cuda")
    M.moe_tensor_scale_microscaled(w, wg)
    M.moe_quantize_microscaled(NV, w, wg, wc, wsc)
    xg, xc, xs = torch.empty(1, device="cuda"), torch.empty(P, d // 2, dtype=U8, device="cuda"), torch.empty(
        P, d // 16, dtype=U8, device="cuda")
    y, y16 = torch.zeros(P, f, device="cuda"), torch.zeros(P, f, device="cuda")
    sh = M.grouped_shape(P, E, f, d, F32)
    ws = M.grouped_workspace(sh)

    def go():
        M.moe_dispatch(cfg, idx, x, off, perm, inv, gs, xp, lws)
        M.moe_tensor_scale_microscaled(xp, xg)
        M.moe_quantize_microscaled(NV, xp, xg, xc, xs)
        M.moe_grouped_gemm_microscaled(sh, NV, xc, xs, xg, gs, off, wc, wsc, wg, y, ws)
        M.moe_grouped_gemm(sh, xp, gs, off, w, y16, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for seed in range(3):
        gen = torch.Generator().manual_seed(seed)
        idx.copy_(torch.stack([torch.randperm(E - seed, generator=gen)[:top] for _ in range(T)]).to(torch.int32))
        x.copy_(torch.randn(T, d, generator=gen).to(BF))
        graph.replay()
        assert M.moe_get_device_status(ws) == 0 and M.moe_get_device_status(lws) == 0
        rows, flat = inv.long(), idx.reshape(-1).long()
        xv, wv = values(xc[rows], xs[rows], None, NV), values(wc, wsc, None, NV)
        alpha = (xg.double() * wg.double())[flat].unsqueeze(1)
        ref = torch.einsum("rk,rnk->rn", xv, wv[flat]) * alpha
        S = torch.einsum("rk,rnk->rn", xv.abs(), wv[flat].abs()) * alpha
        tol = 65 * (d / 64 + 1) * 2.0 ** -23 * S + 2.0 ** -21 * ref.abs()
        assert ((y[rows].double() - ref).abs() <= tol).all()
        ex = (xv * xg.double() - xp[rows].double()).norm() / xp[rows].double().norm()
        ew = (wv * wg.double().reshape(-1, 1, 1) - w.double()).norm() / w.double().norm()
        rel = (y[rows] - y16[rows]).norm() / y16[rows].norm()
        # rows and columns of unlike norms: twice the sum of the operands' errors
        assert rel <= 2 * (ex + ew + ex * ew)
