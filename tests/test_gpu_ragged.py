"""The ragged grouped products and their gradients against 64-bit sums.

Tolerances, element by element. Operands are bf16, so products are exact in fp32. The
tensor core adds 16 of them to the accumulator a step; each of the 17 terms may lose
what lies below 2^-24 of the step's largest, which is at most S = sum |a||b| of the
element. A reduction of L terms has L/16 steps, so the sum is off by at most
17 (L/16 + 1) 2^-24 S; parts of 512 terms are then added in fp32, half an ulp each,
at most (L/512 + 1) 2^-24 S. The result's rounding adds eps/2 of the value.
"""

import pytest
import torch

import sparse_moe_transformer_route_b200 as M
from tests._parity import require_gpu

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
BAD_GROUP = 0x203


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def layout(counts, how):
    """(group_start or None, offsets, first rows, rows of the buffer)."""
    off = [0]
    for c in counts:
        off.append(off[-1] + c)
    if how == "packed":
        starts, total, gs = off[:-1], off[-1], None
    elif how == "slack":  # packed, with rows behind the last group
        starts, total, gs = off[:-1], off[-1] + 45, None
    elif how == "padded":
        starts, at = [], 0
        for c in counts:
            starts.append(at)
            at += -(-c // 128) * 128
        total, gs = at + 128, starts + [at]
    else:  # any order, gaps of 3 rows
        starts, at = [0] * len(counts), 3
        for e in reversed(range(len(counts))):
            starts[e] = at
            at += counts[e] + 3
        total, gs = at, starts + [at]
    as_t = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    return (None if gs is None else as_t(gs)), as_t(off), starts, total


def make(counts, n, k, how, seed=0, poison=float("nan")):
    g = torch.Generator(device="cuda").manual_seed(seed)
    gs, off, starts, total = layout(counts, how)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)  # noqa: E731
    x, dy, w = rn(total, k), rn(total, n), rn(len(counts), n, k)
    owned = torch.zeros(total, dtype=torch.bool, device="cuda")
    for s, c in zip(starts, counts):
        owned[s:s + c] = True
    x[~owned] = poison
    dy[~owned] = poison
    return gs, off, starts, total, x, dy, w, owned


def tol(ref, S, L, dtype):
    half = torch.finfo(dtype).eps / 2
    return half * ref.abs() * (1 + 2.0 ** -6) + (17 * (L / 16 + 1) + L / 512 + 1) * 2.0 ** -24 * S + 1e-30


def check(got, ref, S, L, what):
    bad = ~((got.double() - ref).abs() <= tol(ref, S, L, got.dtype))
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first {bad.nonzero()[0].tolist()}"


SENTINEL = -77.0


def run_all(counts, n, k, how, dt, seed=0):
    gs, off, starts, total, x, dy, w, owned = make(counts, n, k, how, seed)
    E = len(counts)
    sh = M.grouped_shape(total, E, n, k, dt)
    ws = M.grouped_workspace(sh)
    y = torch.full((total, n), SENTINEL, dtype=dt, device="cuda")
    dx = torch.full((total, k), SENTINEL, dtype=dt, device="cuda")
    dw = torch.full((E, n, k), SENTINEL, dtype=dt, device="cuda")
    M.moe_grouped_gemm(sh, x, gs, off, w, y, ws)
    M.moe_grouped_gemm_dgrad(sh, dy, gs, off, w, dx, ws)
    M.moe_grouped_gemm_wgrad(sh, dy, x, gs, off, dw, ws)
    assert M.moe_get_device_status(ws) == 0
    assert torch.all(y[~owned] == SENTINEL) and torch.all(dx[~owned] == SENTINEL)
    for e, (s, c) in enumerate(zip(starts, counts)):
        xe, de, we = x[s:s + c].double(), dy[s:s + c].double(), w[e].double()
        check(y[s:s + c], xe @ we.t(), xe.abs() @ we.abs().t(), k, f"y of expert {e}")
        check(dx[s:s + c], de @ we, de.abs() @ we.abs(), n, f"dx of expert {e}")
        check(dw[e], de.t() @ xe, de.abs().t() @ xe.abs(), c, f"dW of expert {e}")


COUNTS = [
    [1],
    [0, 1, 127, 128, 129, 300, 0, 5],
    [0, 0, 0, 17, 0],
    [33, 64, 65, 96, 97, 31, 32],
]
WIDTHS = [(8, 8), (16, 520), (1048, 72), (256, 64), (264, 192), (640, 1024)]


@pytest.mark.parametrize("n,k", WIDTHS)
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{max(c)}")
@pytest.mark.parametrize("how", ["packed", "padded", "gaps", "slack"])
def test_products_match_64_bits(counts, n, k, how):
    run_all(counts, n, k, how, BF if (n + len(counts)) % 16 else F32, seed=n + k)


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("counts,n,k", [
    ([1500, 0, 3, 700], 2048, 1024),    # several row tiles, wide tiles
    ([513, 512, 511, 4097], 264, 256),  # long sums over a group's rows
    ([40] * 64, 512, 256),
    ([3, 200], 4096, 264),              # long sums over the width
    ([2, 5], 64, 8192),
])
def test_products_match_64_bits_larger(counts, n, k, dt):
    run_all(counts, n, k, "gaps", dt, seed=k)


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("how", ["packed", "gaps"])
@pytest.mark.parametrize("n,k", [(2048, 2048), (2056, 1032)])
def test_large_groups_run_on_pairs(n, k, how, dt):
    """Enough rows and columns for 256 x 256 tiles: groups that end anywhere in a tile, in a
    64-row stage of wgrad's reduction and in a 16-row step, among them small and empty ones."""
    run_all([700, 1, 650, 0, 1303, 704, 257, 2000], n, k, how, dt, seed=n)


@pytest.mark.parametrize("mean,n", [(3, 512), (30, 2048), (80, 2048), (300, 128), (140, 384)])
def test_every_kind_of_tile(mean, n):
    """Mean group sizes and widths on both sides of the rule that picks a tile."""
    g = torch.Generator().manual_seed(mean)
    counts = torch.poisson(torch.full((64,), float(mean)), generator=g).int().tolist()
    run_all(counts, n, 136, "packed", BF, seed=mean)


def test_most_experts_with_random_counts():
    g = torch.Generator().manual_seed(5)
    counts = torch.randint(0, 40, (256,), generator=g).tolist()
    run_all(counts, 136, 72, "packed", BF)
    run_all(counts, 136, 72, "packed", F32)


def test_no_rows_at_all():
    for total in (0, 50):
        off = torch.zeros(4, dtype=torch.int32, device="cuda")
        x = torch.full((total, 64), float("nan"), dtype=BF, device="cuda")
        w = torch.randn(3, 64, 64, device="cuda").to(BF)
        y = torch.full((total, 64), SENTINEL, dtype=BF, device="cuda")
        sh = M.grouped_shape(total, 3, 64, 64)
        ws = M.grouped_workspace(sh)
        M.moe_grouped_gemm(sh, x, None, off, w, y, ws)
        M.moe_grouped_gemm_dgrad(sh, x, None, off, w, y, ws)
        dw = torch.full((3, 64, 64), SENTINEL, dtype=BF, device="cuda")
        M.moe_grouped_gemm_wgrad(sh, x, x, None, off, dw, ws)
        assert M.moe_get_device_status(ws) == 0
        assert torch.all(y == SENTINEL) and torch.all(dw == 0)


def test_empty_groups_may_start_anywhere():
    counts, n, k = [4, 0, 6, 0], 64, 64
    gs, off, starts, total, x, dy, w, _ = make(counts, n, k, "gaps")
    gs[1], gs[3] = -7, total + 1000
    sh = M.grouped_shape(total, 4, n, k)
    ws = M.grouped_workspace(sh)
    y = torch.zeros(total, n, dtype=BF, device="cuda")
    dw = torch.full((4, n, k), SENTINEL, dtype=BF, device="cuda")
    M.moe_grouped_gemm(sh, x, gs, off, w, y, ws)
    M.moe_grouped_gemm_wgrad(sh, dy, x, gs, off, dw, ws)
    assert M.moe_get_device_status(ws) == 0
    for e in (0, 2):
        s, c = starts[e], counts[e]
        xe, we = x[s:s + c].double(), w[e].double()
        check(y[s:s + c], xe @ we.t(), xe.abs() @ we.abs().t(), k, f"y of expert {e}")
    assert torch.all(dw[1] == 0) and torch.all(dw[3] == 0)


def test_one_experts_nan_stays_with_it():
    """Groups end inside tiles: a neighbour's NaN rows are loaded and must not count."""
    counts, n, k = [5, 130, 7, 20], 72, 136
    gs, off, starts, total, x, dy, w, _ = make(counts, n, k, "packed")
    bad = slice(starts[1], starts[1] + counts[1])
    x[bad] = float("nan")
    dy[bad] = float("inf")
    w[1] = float("nan")
    sh = M.grouped_shape(total, 4, n, k, F32)
    ws = M.grouped_workspace(sh)
    y, dx = torch.empty(total, n, device="cuda"), torch.empty(total, k, device="cuda")
    dw = torch.empty(4, n, k, device="cuda")
    M.moe_grouped_gemm(sh, x, gs, off, w, y, ws)
    M.moe_grouped_gemm_dgrad(sh, dy, gs, off, w, dx, ws)
    M.moe_grouped_gemm_wgrad(sh, dy, x, gs, off, dw, ws)
    assert M.moe_get_device_status(ws) == 0
    for t in (y, dx):
        assert torch.isnan(t[bad]).all()
        assert torch.isfinite(t[:starts[1]]).all() and torch.isfinite(t[starts[2]:]).all()
    assert torch.isnan(dw[1]).all()
    assert torch.isfinite(dw[[0, 2, 3]]).all()


@pytest.mark.parametrize("how", ["offsets fall", "past the end", "negative start"])
def test_bad_groups_are_recorded_and_left_alone(how):
    counts, n, k = [4, 6, 10], 64, 64
    gs, off, starts, total, x, dy, w, _ = make(counts, n, k, "gaps")
    off2, gs2 = off.clone(), gs.clone()
    if how == "offsets fall":
        off2[2] = off2[1] - 2  # expert 1 has -2 rows; expert 2 now 12
        gs2[2] = 0
        ok = [0]
    elif how == "past the end":
        gs2[1] = total - 5
        ok = [0, 2]
    else:
        gs2[1] = -1
        ok = [0, 2]
    sh = M.grouped_shape(total, 3, n, k)
    ws = M.grouped_workspace(sh)
    y = torch.full((total, n), SENTINEL, dtype=BF, device="cuda")
    dw = torch.full((3, n, k), SENTINEL, dtype=BF, device="cuda")
    M.moe_grouped_gemm(sh, x, gs2, off2, w, y, ws)
    assert M.moe_get_device_status(ws) == BAD_GROUP
    M.moe_grouped_gemm_wgrad(sh, dy, x, gs2, off2, dw, ws)
    assert M.moe_get_device_status(ws) == BAD_GROUP
    assert M.moe_get_device_status(ws) == 0
    if how != "offsets fall":
        assert torch.all(y[starts[1]:starts[1] + 6] == SENTINEL)
    assert torch.all(dw[1] == 0)
    for e in ok:
        s, c = starts[e], counts[e]
        xe, de, we = x[s:s + c].double(), dy[s:s + c].double(), w[e].double()
        check(y[s:s + c], xe @ we.t(), xe.abs() @ we.abs().t(), k, f"y of expert {e}")
        check(dw[e], de.t() @ xe, de.abs().t() @ xe.abs(), c, f"dW of expert {e}")


def test_gradients_against_differences():
    """The product is linear in each operand, so a central difference of <dy, y> along a
    direction is its gradient but for rounding: the two products' sums differ from the
    exact ones by the bound above, and the difference divides that by the step."""
    counts, n, k = [9, 0, 70], 136, 72
    gs, off, starts, total, x, dy, w, owned = make(counts, n, k, "packed", seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    sh = M.grouped_shape(total, 3, n, k, F32)
    ws = M.grouped_workspace(sh)
    dx, dw = torch.empty(total, k, device="cuda"), torch.empty(3, n, k, device="cuda")
    M.moe_grouped_gemm_dgrad(sh, dy, gs, off, w, dx, ws)
    M.moe_grouped_gemm_wgrad(sh, dy, x, gs, off, dw, ws)

    def f(xx, ww):
        y = torch.empty(total, n, device="cuda")
        M.moe_grouped_gemm(sh, xx, gs, off, ww, y, ws)
        return (dy.double() * y.double()).sum()

    # steps that bf16 adds exactly: operands and directions on a grid of 2^-4, at most 4
    q = lambda t: ((t * 16).round() / 16).clamp(-4, 4).to(BF)  # noqa: E731
    x, w = q(x.float()), q(w.float())
    M.moe_grouped_gemm_dgrad(sh, dy, gs, off, w, dx, ws)
    M.moe_grouped_gemm_wgrad(sh, dy, x, gs, off, dw, ws)
    vx = torch.randint(-1, 2, x.shape, generator=g, device="cuda").to(BF)
    vw = torch.randint(-1, 2, w.shape, generator=g, device="cuda").to(BF)
    # (4 + 1) on a grid of 2^-4 needs 7 bits: exact in bf16
    S = 0.0
    for e, (s, c) in enumerate(zip(starts, counts)):
        S += (dy[s:s + c].double().abs() * ((x[s:s + c].double().abs() + 1) @ (w[e].double().abs() + 1).t())).sum().item()
    bound = (17 * (k / 16 + 1) + 2) * 2.0 ** -24 * S
    gx = (f(x + vx, w) - f(x - vx, w)) / 2
    gw = (f(x, w + vw) - f(x, w - vw)) / 2
    Sg = (17 * (max(n, max(counts)) / 16 + 1) + 2) * 2.0 ** -24 * S
    assert abs(gx - (dx.double() * vx.double())[owned].sum()) <= bound + Sg
    assert abs(gw - (dw.double() * vw.double()).sum()) <= bound + Sg


def test_two_streams_share_a_workspace():
    cases = [make([300, 5, 0, 129], 256, 128, "packed", seed=1), make([7, 7, 800, 0], 256, 128, "packed", seed=2)]
    ws = M.grouped_workspace()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [torch.zeros(c[3], 256, device="cuda") for c in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s, y in zip(cases, streams, outs):
            sh = M.grouped_shape(c[3], 4, 256, 128, F32)
            M.moe_grouped_gemm(sh, c[4], c[0], c[1], c[6], y, ws, stream=s)
    torch.cuda.synchronize()
    assert M.moe_get_device_status(ws) == 0
    for c, y, counts in zip(cases, outs, ([300, 5, 0, 129], [7, 7, 800, 0])):
        for e, (s, m) in enumerate(zip(c[2], counts)):
            xe, we = c[4][s:s + m].double(), c[6][e].double()
            check(y[s:s + m], xe @ we.t(), xe.abs() @ we.abs().t(), 128, f"y of expert {e}")


def test_captured_graph_follows_its_inputs():
    """Group sizes live on the device: a captured call serves other sizes on replay, and
    results do not depend on the run."""
    n, k, E, total = 264, 136, 4, 400
    x = torch.zeros(total, k, dtype=BF, device="cuda")
    dy = torch.zeros(total, n, dtype=BF, device="cuda")
    w = torch.randn(E, n, k, device="cuda").to(BF)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    sh = M.grouped_shape(total, E, n, k, F32)
    ws = M.grouped_workspace(sh)
    y, dx = torch.zeros(total, n, device="cuda"), torch.zeros(total, k, device="cuda")
    dw = torch.zeros(E, n, k, device="cuda")

    def go():
        M.moe_grouped_gemm(sh, x, None, off, w, y, ws)
        M.moe_grouped_gemm_dgrad(sh, dy, None, off, w, dx, ws)
        M.moe_grouped_gemm_wgrad(sh, dy, x, None, off, dw, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for seed, counts in enumerate(([100, 100, 100, 100], [0, 390, 1, 0], [0, 0, 0, 0], [13, 129, 2, 128])):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x.copy_(torch.randn(total, k, generator=g, device="cuda"))
        dy.copy_(torch.randn(total, n, generator=g, device="cuda"))
        ends = torch.tensor([0] + counts).cumsum(0)
        off.copy_(ends.to(torch.int32))
        graph.replay()
        first = [t.clone() for t in (y, dx, dw)]
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(first, (y, dx, dw)))
        assert M.moe_get_device_status(ws) == 0
        for e, c in enumerate(counts):
            s = int(ends[e])
            xe, de, we = x[s:s + c].double(), dy[s:s + c].double(), w[e].double()
            check(y[s:s + c], xe @ we.t(), xe.abs() @ we.abs().t(), k, f"y of expert {e}")
            check(dx[s:s + c], de @ we, de.abs() @ we.abs(), n, f"dx of expert {e}")
            check(dw[e], de.t() @ xe, de.abs().t() @ xe.abs(), c, f"dW of expert {e}")


def test_two_graphs_share_a_workspace_and_operands():
    """Two captured calls, replayed on two streams at once."""
    gs, off, starts, total, x, dy, w, _ = make([300, 77, 0, 900], 512, 256, "packed", seed=8)
    sh, shx = M.grouped_shape(total, 4, 512, 256, F32), M.grouped_shape(total, 4, 512, 256, BF)
    ws = M.grouped_workspace(sh)
    dw, dx = torch.zeros(4, 512, 256, device="cuda"), torch.zeros(total, 256, dtype=BF, device="cuda")
    graphs = []
    for call in (lambda: M.moe_grouped_gemm_wgrad(sh, dy, x, gs, off, dw, ws),
                 lambda: M.moe_grouped_gemm_dgrad(shx, dy, gs, off, w, dx, ws)):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        graphs.append((graph, torch.cuda.Stream()))
    want = dw.clone(), dx.clone()
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, stream in graphs:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    assert M.moe_get_device_status(ws) == 0
    assert torch.equal(dw, want[0]) and torch.equal(dx, want[1])
    for e, (s, c) in enumerate(zip(starts, [300, 77, 0, 900])):
        xe, de, we = x[s:s + c].double(), dy[s:s + c].double(), w[e].double()
        check(dx[s:s + c], de @ we, de.abs() @ we.abs(), 512, f"dx of expert {e}")
        check(dw[e], de.t() @ xe, de.abs().t() @ xe.abs(), c, f"dW of expert {e}")


def test_calls_want_the_current_stream_and_device():
    x = torch.zeros(4, 64, dtype=BF, device="cuda")
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    w, y = torch.zeros(1, 64, 64, dtype=BF, device="cuda"), torch.zeros(4, 64, dtype=BF, device="cuda")
    sh = M.grouped_shape(4, 1, 64, 64)
    ws = M.grouped_workspace(sh)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        M.moe_grouped_gemm(sh, x.cpu(), None, off, w, y, ws)
    with pytest.raises(ValueError, match="w must be contiguous"):
        M.moe_grouped_gemm(sh, x, None, off, w.transpose(1, 2), y, ws)
    with pytest.raises(TypeError, match="y must be torch.bfloat16"):
        M.moe_grouped_gemm(sh, x, None, off, w, y.float(), ws)
    with pytest.raises(M.MoeError) as err:
        M.moe_grouped_gemm(sh, x, None, off, w, y, ws[:128])
    assert err.value.status == 3
    if torch.cuda.device_count() > 1:
        with pytest.raises(ValueError, match="current device"):
            M.moe_grouped_gemm(sh, x.to("cuda:1"), None, off, w, y, ws)
        with pytest.raises(ValueError, match="stream"):
            M.moe_grouped_gemm(sh, x, None, off, w, y, ws, stream=torch.cuda.Stream("cuda:1"))


def test_far_rows_of_a_large_buffer():
    """Row offsets beyond 2^31 elements."""
    n, k, total = 8, 4096, (1 << 19) + 100
    x = torch.zeros(total, k, dtype=BF, device="cuda")  # 2^31 + elements
    gs = torch.tensor([total - 70, 3, 0], dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 65, 70], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    for s, c in ((total - 70, 65), (3, 5)):
        x[s:s + c] = torch.randn(c, k, generator=g, device="cuda").to(BF)
    w = torch.randn(2, n, k, generator=g, device="cuda").to(BF)
    sh = M.grouped_shape(total, 2, n, k, F32)
    ws = M.grouped_workspace(sh)
    y = torch.zeros(total, n, device="cuda")
    M.moe_grouped_gemm(sh, x, gs, off, w, y, ws)
    dy = torch.randn(total, n, generator=g, device="cuda").to(BF)
    shx = M.grouped_shape(total, 2, n, k, BF)
    dx = torch.zeros(total, k, dtype=BF, device="cuda")
    M.moe_grouped_gemm_dgrad(shx, dy, gs, off, w, dx, ws)
    assert M.moe_get_device_status(ws) == 0
    for e, (s, c) in enumerate(((total - 70, 65), (3, 5))):
        xe, de, we = x[s:s + c].double(), dy[s:s + c].double(), w[e].double()
        check(y[s:s + c], xe @ we.t(), xe.abs() @ we.abs().t(), k, f"y of expert {e}")
        check(dx[s:s + c], de @ we, de.abs() @ we.abs(), n, f"dx of expert {e}")
    assert torch.all(y[8:total - 70] == 0) and torch.all(dx[total - 5:] == 0)


def test_products_on_dispatched_rows():
    """As a user runs them: moe_dispatch lays the rows out, the products take its offsets
    and group_start as they are."""
    T, E, top, d, f = 200, 8, 2, 256, 384
    g = torch.Generator().manual_seed(1)
    idx = torch.stack([torch.randperm(E - 1, generator=g)[:top] for _ in range(T)]).to(torch.int32).cuda()
    x = torch.randn(T, d, generator=g).to(BF).cuda()
    cfg = M.config(T, d, E, top, 128)
    P = M.moe_padded_rows(cfg)
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    off, gs, perm, inv = i32(E + 1), i32(E + 1), i32(T * top), i32(T * top)
    xp = torch.full((P, d), float("nan"), dtype=BF, device="cuda")
    lws = M.workspace(cfg)
    M.moe_dispatch(cfg, idx, x, off, perm, inv, gs, xp, lws)
    w = torch.randn(E, f, d, generator=g).to(BF).cuda()
    sh = M.grouped_shape(P, E, f, d)
    ws = M.grouped_workspace(sh)
    y = torch.full((P, f), SENTINEL, dtype=BF, device="cuda")
    M.moe_grouped_gemm(sh, xp, gs, off, w, y, ws)
    dx = torch.full((P, d), SENTINEL, dtype=BF, device="cuda")
    M.moe_grouped_gemm_dgrad(sh, y, gs, off, w, dx, ws)
    shw = M.grouped_shape(P, E, f, d, F32)
    dw = torch.empty(E, f, d, device="cuda")
    M.moe_grouped_gemm_wgrad(shw, y, xp, gs, off, dw, ws)
    assert M.moe_get_device_status(ws) == 0 and M.moe_get_device_status(lws) == 0
    flat = idx.reshape(-1).long()
    rows = inv.long()
    xt = x.repeat_interleave(top, 0).double()
    wt = w.double()[flat]
    check(y[rows], torch.einsum("rk,rnk->rn", xt, wt), torch.einsum("rk,rnk->rn", xt.abs(), wt.abs()), d, "y")
    yt = y[rows].double()
    check(dx[rows], torch.einsum("rn,rnk->rk", yt, wt), torch.einsum("rn,rnk->rk", yt.abs(), wt.abs()), f, "dx")
    for e in range(E):
        m = flat == e
        check(dw[e], yt[m].t() @ xt[m], yt[m].abs().t() @ xt[m].abs(), int(m.sum()), f"dW of expert {e}")
    lone = torch.ones(P, dtype=torch.bool, device="cuda")
    lone[rows] = False
    assert torch.all(y[lone] == SENTINEL) and torch.all(dx[lone] == SENTINEL)
