"""The experts' products on the GPU against float64, expert by expert, elementwise within the bounds of dense_reference."""

import pytest
import torch

import dense_reference as R
from test_gpu_dense import Out, guard_ok, rnd

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def N():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mixture_experts_route_amd import native

    return native


def gen_for(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def workspace(N, d, P, backward):
    n = N.moe_experts_workspace_bytes(d, P, backward)
    whole = torch.full((n + 1024,), 0xA5, dtype=torch.uint8, device="cuda")
    N.moe_workspace_init(whole[:n])
    return whole[:n], whole


def stack(gen, E, M, K, dt, scale, pad=0, offset=0, gap=0):
    """[E][M][K] weights; padded: slices of wider rows and longer matrices whose other elements are NaN."""
    v = (torch.randn((E, M, K), generator=gen, device="cuda") * scale).to(dt)
    if not (pad or offset or gap):
        return v
    wide = torch.full((E, M + gap, offset + K + pad), float("nan"), dtype=dt, device="cuda")
    wide[:, :M, offset:offset + K] = v
    return wide[:, :M, offset:offset + K]


def rows_of(counts, lead, tail):
    """offsets on the device, each expert's slice of the rows, and the number of rows."""
    ends = [lead]
    for c in counts:
        ends.append(ends[-1] + c)
    return torch.tensor(ends, dtype=torch.int32, device="cuda"), [slice(a, b) for a, b in zip(ends, ends[1:])], ends[-1] + tail


def check_rows(name, got, refs, slices, lead, tail):
    """Each expert's rows against its reference; the rows of nobody still NaN."""
    for s, ref in zip(slices, refs):
        if s.start < s.stop:
            R.check(f"{name} {s}", got.t[s], ref)
    n = got.t.shape[0]
    assert torch.isnan(got.t[:lead]).all() and torch.isnan(got.t[n - tail:]).all() and got.untouched()


def check_all(N, seed, counts, K, M, dt, act=1, lead=0, tail=0, pad=0, offset=0, gap=0, need=("lin", "gated")):
    gen = gen_for(seed)
    E = len(counts)
    offs, slices, P = rows_of(counts, lead, tail)
    code = N.dtype_code(torch.empty(0, dtype=dt))
    live = [e for e in range(E) if counts[e]]
    x = rnd(gen, (P, K), dt, pad=pad, offset=offset)
    x[:lead], x[P - tail:] = float("nan"), float("nan")  # rows of nobody
    wg, wu = (stack(gen, E, M, K, dt, K ** -0.5, pad, offset, gap) for _ in range(2))
    dy = rnd(gen, (P, M), dt, 0.1, pad, offset)
    dy[:lead], dy[P - tail:] = float("nan"), float("nan")
    zero = (torch.zeros(M, K, dtype=torch.float64, device="cuda"), torch.zeros(M, K, dtype=torch.float64, device="cuda"))
    for gated in (False, True):
        if ("gated" if gated else "lin") not in need:
            continue
        d = N.experts_dims(E, K, M, code, act if gated else 0)
        ws, whole = workspace(N, d, P, False)
        y, g, u = (Out((P, M), dt, pad, offset) for _ in range(3))
        if gated:
            N.moe_experts_gated_forward(d, x, offs, wg, wu, y.t, ws, gate=g.t, up=u.t)
            refs = [R.gated_forward(act, x[slices[e]], wg[e], wu[e], None, None) for e in range(E)]
            for name, out in (("h", y), ("gate", g), ("up", u)):
                check_rows(name, out, [r[name] for r in refs], slices, lead, tail)
            plain = Out((P, M), dt, pad, offset)
            N.moe_experts_gated_forward(d, x, offs, wg, wu, plain.t, ws)
            check_rows("h alone", plain, [r["h"] for r in refs], slices, lead, tail)
        else:
            N.moe_experts_linear_forward(d, x, offs, wg, y.t, ws)
            refs = [R.linear_forward(0, x[slices[e]], wg[e], None, None, dt)["y"] for e in range(E)]
            check_rows("y", y, refs, slices, lead, tail)
        assert N.moe_check_device_error(ws) == 0 and guard_ok(whole)
        ws, whole = workspace(N, d, P, True)
        dx, dws = Out((P, K), dt, pad, offset), [stack(gen, E, M, K, dt, 1.0, pad, offset, gap) for _ in range(2)]
        for t in dws:
            t.fill_(float("nan"))
        if gated:
            N.moe_experts_gated_backward(d, x, offs, wg, wu, g.t, u.t, dy, ws, dx=dx.t, dw_gate=dws[0], dw_up=dws[1])
            refs = {e: R.gated_backward(act, x[slices[e]], wg[e], wu[e], g.t[slices[e]], u.t[slices[e]], dy[slices[e]])
                    for e in live}
        else:
            N.moe_experts_linear_backward(d, x, offs, wg, dy, ws, dx=dx.t, dw=dws[0])
            refs = {e: R.linear_backward(0, x[slices[e]], wg[e], None, dy[slices[e]]) for e in live}
        check_rows("dx", dx, [refs[e]["dx"] if e in refs else None for e in range(E)], slices, lead, tail)
        for m in range(2 if gated else 1):
            for e in range(E):
                R.check(f"dw{m} {e}", dws[m][e], refs[e][f"dw{m}"] if e in refs else zero)
            if gap:
                assert torch.isnan(torch.as_strided(dws[m], (E, gap, K), dws[m].stride(),
                                                    dws[m].storage_offset() + M * dws[m].stride(1))).all()
        # each output alone has the same bits
        one, alone = Out((P, K), dt, pad, offset), torch.empty_like(dws[0])
        if gated:
            N.moe_experts_gated_backward(d, x, offs, wg, wu, g.t, u.t, dy, ws, dx=one.t)
            N.moe_experts_gated_backward(d, x, offs, wg, wu, g.t, u.t, dy, ws, dw_up=alone)
            assert torch.equal(alone, dws[1])
        else:
            N.moe_experts_linear_backward(d, x, offs, wg, dy, ws, dx=one.t)
            N.moe_experts_linear_backward(d, x, offs, wg, dy, ws, dw=alone)
            assert torch.equal(alone, dws[0])
        assert torch.equal(one.t.nan_to_num(9.0), dx.t.nan_to_num(9.0))
        assert N.moe_check_device_error(ws) == 0 and guard_ok(whole)


RAGGED = [0, 1, 2, 15, 16, 17, 0, 63, 64, 65, 33, 0, 127, 128, 129, 7, 255, 257, 0]


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("K,M", [(64, 32), (128, 256), (200, 136), (72, 8), (8, 72), (512, 40)])
def test_ragged_groups(N, K, M, dt):
    check_all(N, K + M, RAGGED, K, M, dt, lead=3, tail=5)


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("K,M", [(1, 1), (7, 5), (65, 33), (100, 130), (131, 64), (64, 131)])
def test_odd_widths(N, K, M, dt):
    check_all(N, K * M, RAGGED, K, M, dt, lead=1, tail=2)


@pytest.mark.parametrize("pad,offset,gap", [(1, 0, 0), (8, 8, 1), (0, 3, 2), (8, 0, 0), (5, 1, 1)])
def test_strides_and_alignments(N, pad, offset, gap):
    check_all(N, 50 + pad, [5, 0, 70, 16, 1], 96, 56, BF16, pad=pad, offset=offset, gap=gap, tail=1)
    check_all(N, 51 + pad, [5, 0, 70, 16, 1], 61, 75, F16, pad=pad, offset=offset, gap=gap, lead=2)


@pytest.mark.parametrize("kernel", range(1, 6))
@pytest.mark.parametrize("K,M", [(192, 320), (256, 100)])
def test_every_kernel(N, kernel, K, M):
    N.moe_debug_force_dense_plan(kernel)
    try:
        check_all(N, kernel, RAGGED + [300, 513], K, M, BF16, act=2, lead=1, tail=1)
        check_all(N, kernel + 9, [0, 3, 0], K, M, F16, act=3)
    finally:
        N.moe_debug_force_dense_plan()


@pytest.mark.parametrize("act", range(6))
def test_every_activation(N, act):
    check_all(N, 60 + act, [20, 0, 33, 5], 128, 64, BF16, act=act, need=("gated",))
    check_all(N, 70 + act, [20, 0, 33, 5], 127, 63, F16, act=act, need=("gated",))


@pytest.mark.parametrize("E", [1, 2, 63, 64, 65, 200, 512, 1000, 1024])
def test_number_of_experts(N, E):
    g = torch.Generator().manual_seed(E)
    counts = torch.randint(0, 4, (E,), generator=g).tolist()
    counts[-1] = 70
    check_all(N, E, counts, 64, 24, BF16, tail=1)


def test_one_row_and_no_rows(N):
    check_all(N, 80, [1], 64, 64, BF16)
    check_all(N, 81, [0, 0, 1], 64, 64, F16)
    check_all(N, 82, [0, 0, 0], 64, 64, BF16, tail=4)  # every row is nobody's
    check_all(N, 83, [0, 0, 0], 63, 61, BF16, lead=4)


def test_many_rows(N):
    """Two million rows of three experts, and the halves of one weight tensor as the gated block's two."""
    check_all(N, 84, [1 << 20, 5, (1 << 20) - 70], 24, 16, BF16, lead=2, tail=3, need=("lin",))
    E, K, M = 5, 96, 40
    counts = [70, 0, 3, 130, 16]
    gen = gen_for(85)
    offs, slices, P = rows_of(counts, 0, 0)
    w = stack(gen, E, 2 * M, K, BF16, K ** -0.5)
    x, dh = rnd(gen, (P, K), BF16), rnd(gen, (P, M), BF16)
    d = N.experts_dims(E, K, M, N.MOE_BF16, 1)
    ws, whole = workspace(N, d, P, True)
    h, g, u, dx, dw = (torch.empty(s, dtype=BF16, device="cuda") for s in ((P, M), (P, M), (P, M), (P, K), (E, 2 * M, K)))
    N.moe_experts_gated_forward(d, x, offs, w[:, :M], w[:, M:], h, ws, gate=g, up=u)
    N.moe_experts_gated_backward(d, x, offs, w[:, :M], w[:, M:], g, u, dh, ws, dx=dx, dw_gate=dw[:, :M], dw_up=dw[:, M:])
    for e in (0, 2, 3, 4):
        s = slices[e]
        R.check("h", h[s], R.gated_forward(1, x[s], w[e, :M], w[e, M:], None, None)["h"])
        ref = R.gated_backward(1, x[s], w[e, :M], w[e, M:], g[s], u[s], dh[s])
        R.check("dx", dx[s], ref["dx"])
        R.check("dw0", dw[e, :M], ref["dw0"])
        R.check("dw1", dw[e, M:], ref["dw1"])
    assert (dw[1] == 0).all() and guard_ok(whole) and N.moe_check_device_error(ws) == 0


def test_bad_offsets_are_reported_and_stay_in_bounds(N):
    E, K, M, P = 4, 64, 40, 50
    gen = gen_for(90)
    x, w, dy = rnd(gen, (P, K), BF16), stack(gen, E, M, K, BF16, 0.1), rnd(gen, (P, M), BF16)
    d = N.experts_dims(E, K, M, N.MOE_BF16, 1)
    dl = N.experts_dims(E, K, M, N.MOE_BF16)
    ws, whole = workspace(N, d, P, True)
    for offs in ([0, 10, 5, 20, 50], [-3, 10, 20, 30, 50], [0, 10, 20, 30, 51], [0, 10, 20, 2 ** 31 - 1, 50],
                 [-2 ** 31, 2 ** 31 - 1, -2 ** 31, 50, 50]):
        o = torch.tensor(offs, dtype=torch.int32, device="cuda")
        y, dx = Out((P, M), BF16), Out((P, K), BF16)
        dw = torch.full((E + 2, M, K), float("nan"), dtype=BF16, device="cuda")
        N.moe_experts_linear_forward(dl, x, o, w, y.t, ws)
        assert N.moe_check_device_error(ws) == N.DERR_ROWS, offs
        N.moe_experts_gated_forward(d, x, o, w, w, y.t, ws)
        assert N.moe_check_device_error(ws) == N.DERR_ROWS, offs
        N.moe_experts_linear_backward(dl, x, o, w, dy, ws, dx=dx.t)
        assert N.moe_check_device_error(ws) == N.DERR_ROWS, offs
        N.moe_experts_linear_backward(dl, x, o, w, dy, ws, dw=dw[1:E + 1])
        assert N.moe_check_device_error(ws) == N.DERR_ROWS, offs
        assert y.untouched() and dx.untouched() and torch.isnan(dw[0]).all() and torch.isnan(dw[-1]).all() and guard_ok(whole)


@pytest.mark.parametrize("kernel", [1, 4])  # the two of 64 rows, which count the most tiles
def test_offsets_that_name_every_row_many_times(N, kernel):
    """2^28 rows, the limit, named by every other of 1024 experts: 2^31 rows of tiles."""
    P, E, K, M = 1 << 28, 1024, 8, 8
    d = N.experts_dims(E, K, M, N.MOE_BF16)
    offs = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offs[1::2] = P
    x, w = torch.ones(P, K, dtype=BF16, device="cuda"), torch.ones(E, M, K, dtype=BF16, device="cuda")
    ws, whole = workspace(N, d, P, True)
    N.moe_debug_force_dense_plan(kernel)
    try:
        y = Out((P, M), BF16)
        N.moe_experts_linear_forward(d, x, offs, w, y.t, ws)
        assert N.moe_check_device_error(ws) == N.DERR_ROWS
        N.moe_experts_linear_backward(d, x, offs, w, x, ws, dx=y.t)
        assert N.moe_check_device_error(ws) == N.DERR_ROWS
        assert torch.isnan(y.buf[0]).all() and torch.isnan(y.buf[-1]).all() and guard_ok(whole)
    finally:
        N.moe_debug_force_dense_plan()


@pytest.mark.parametrize("E,K,M", [(4, 64, 40), (200, 136, 72)])  # dx beside dW in 64- and in 128-square tiles
def test_bad_offsets_of_a_whole_backward_pass(N, E, K, M):
    P = 3 * E
    gen = gen_for(94)
    x, dy, wg, wu = rnd(gen, (P, K), BF16), rnd(gen, (P, M), BF16), *(stack(gen, E, M, K, BF16, 0.1) for _ in range(2))
    d, dl = N.experts_dims(E, K, M, N.MOE_BF16, 1), N.experts_dims(E, K, M, N.MOE_BF16)
    ws, whole = workspace(N, d, P, True)
    good = torch.arange(0, P + 1, 3, dtype=torch.int32, device="cuda")
    for at, value in ((0, -1), (1, -2 ** 31), (2, 2 ** 31 - 1), (E // 2, P + 1), (E, P + 1), (E, 0)):
        offs = good.clone()
        offs[at] = value
        dx, dw = Out((P, K), BF16), torch.full((2, E + 2, M, K), float("nan"), dtype=BF16, device="cuda")
        N.moe_experts_linear_backward(dl, x, offs, wg, dy, ws, dx=dx.t, dw=dw[0, 1:E + 1])
        assert N.moe_check_device_error(ws) == N.DERR_ROWS, (at, value)
        N.moe_experts_gated_backward(d, x, offs, wg, wu, dy, dy, dy, ws, dx=dx.t, dw_gate=dw[0, 1:E + 1], dw_up=dw[1, 1:E + 1])
        assert N.moe_check_device_error(ws) == N.DERR_ROWS, (at, value)
        assert dx.untouched() and torch.isnan(dw[:, 0]).all() and torch.isnan(dw[:, -1]).all() and guard_ok(whole)


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("counts,K,M", [
    ([0, 40, 3, 0, 129, 257, 1, 0] * 2, 1544, 264),  # dx of 13 columns of 128-square tiles
    ([5, 0, 300, 131], 2056, 136),  # of 33 columns of 64-square ones
    ([2] * 260, 136, 392),  # more than a round of tiles: dx alone, then dW
    ([3, 1] * 64, 264, 136),
])
def test_dx_and_dw_together(N, counts, K, M, dt):
    check_all(N, K + M, counts, K, M, dt, lead=2, tail=3)


def test_nan_and_infinity_stay_with_their_expert(N):
    gen = gen_for(91)
    counts, K, M = [40, 3, 70], 128, 96
    offs, slices, P = rows_of(counts, 0, 0)
    x, w = rnd(gen, (P, K), BF16), stack(gen, 3, M, K, BF16, K ** -0.5)
    d = N.experts_dims(3, K, M, N.MOE_BF16)
    ws, _ = workspace(N, d, P, True)
    x[41, 5], w[2, 7, 9] = float("nan"), float("inf")
    y = torch.empty(P, M, dtype=BF16, device="cuda")
    N.moe_experts_linear_forward(d, x, offs, w, y, ws)
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[41], want[43:, 7] = True, True
    assert torch.equal(bad, want)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    N.moe_experts_linear_backward(d, x, offs, w, rnd(gen, (P, M), BF16), ws, dx=dx, dw=dw)
    bad = ~torch.isfinite(dw)
    want = torch.zeros_like(bad)
    want[1, :, 5] = True
    assert torch.equal(bad, want)
    bad = ~torch.isfinite(dx)
    want = torch.zeros_like(bad)
    want[43:, 9] = True
    assert torch.equal(bad, want)


def test_rows_do_not_depend_on_where_they_lie(N):
    """The same expert's rows behind other groups: the same bits."""
    gen = gen_for(92)
    K, M, n = 192, 72, 45
    x, w, dy = rnd(gen, (200, K), BF16), stack(gen, 5, M, K, BF16, K ** -0.5), rnd(gen, (200, M), BF16)
    d = N.experts_dims(5, K, M, N.MOE_BF16)
    ws, _ = workspace(N, d, 200, True)
    seen = []
    for before in (0, 1, 64, 100):
        offs = torch.tensor([0, before, before, before, before + n, 200], dtype=torch.int32, device="cuda")
        xs, dys = x.clone(), dy.clone()
        xs[before:before + n], dys[before:before + n] = x[:n], dy[:n]
        y, dx, dw = torch.empty(200, M, dtype=BF16, device="cuda"), torch.empty_like(x), torch.empty_like(w)
        N.moe_experts_linear_forward(d, xs, offs, w, y, ws)
        N.moe_experts_linear_backward(d, xs, offs, w, dys, ws, dx=dx, dw=dw)
        seen.append((y[before:before + n].clone(), dx[before:before + n].clone(), dw[3].clone()))
    for s in seen[1:]:
        assert all(torch.equal(a, b) for a, b in zip(s, seen[0]))


def test_captured_replayed_and_on_another_stream(N):
    gen = gen_for(93)
    E, K, M, P = 6, 128, 72, 160
    x, dh = rnd(gen, (P, K), BF16), rnd(gen, (P, M), BF16)
    wg, wu = (stack(gen, E, M, K, BF16, K ** -0.5) for _ in range(2))
    d = N.experts_dims(E, K, M, N.MOE_BF16, 1)
    offs = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    ws, _ = workspace(N, d, P, True)

    def outs():
        e = lambda *s: torch.empty(s, dtype=BF16, device="cuda")  # noqa: E731
        return {"h": e(P, M), "g": e(P, M), "u": e(P, M), "dx": e(P, K), "dwg": e(E, M, K), "dwu": e(E, M, K)}

    def step(o):
        N.moe_experts_gated_forward(d, x, offs, wg, wu, o["h"], ws, gate=o["g"], up=o["u"])
        N.moe_experts_gated_backward(d, x, offs, wg, wu, o["g"], o["u"], dh, ws, dx=o["dx"], dw_gate=o["dwg"], dw_up=o["dwu"])

    cap = outs()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(cap)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cap)
    for rep, cuts in enumerate(([0, 10, 10, 80, 81, 150, 160], [0, 0, 0, 0, 0, 0, 160], [0, 64, 65, 100, 120, 140, 160])):
        offs.copy_(torch.tensor(cuts, dtype=torch.int32))  # a replay goes by the offsets that it finds
        x.copy_(rnd(gen, (P, K), BF16))
        eager = outs()
        for v in (*cap.values(), *eager.values()):
            v.fill_(float("nan"))
        step(eager)
        graph.replay()
        torch.cuda.synchronize()
        for n in eager:
            assert torch.equal(eager[n], cap[n]), (rep, n)


def test_more_than_2_31_elements(N):
    """Weights and gradients of 2^31 elements and more: sampled experts."""
    E, K, M = 600, 2048, 2048
    gen = gen_for(94)
    w = torch.empty(E, M, K, dtype=BF16, device="cuda")
    for e in range(0, E, 50):
        w[e:e + 50] = (torch.randn(50, M, K, generator=gen, device="cuda") / 45).to(BF16)
    counts = [0] * E
    for e in (0, 1, 300, 511, 512, 513, 599):
        counts[e] = e % 5 + 1
    offs, slices, P = rows_of(counts, 0, 0)
    x, dy = rnd(gen, (P, K), BF16), rnd(gen, (P, M), BF16, 0.1)
    d = N.experts_dims(E, K, M, N.MOE_BF16)
    ws, _ = workspace(N, d, P, True)
    y, dx, dw = torch.empty(P, M, dtype=BF16, device="cuda"), torch.empty_like(x), torch.empty_like(w)
    N.moe_experts_linear_forward(d, x, offs, w, y, ws)
    N.moe_experts_linear_backward(d, x, offs, w, dy, ws, dx=dx, dw=dw)
    for e in (0, 300, 513, 599):
        s = slices[e]
        R.check("y", y[s], R.linear_forward(0, x[s], w[e], None, None, BF16)["y"])
        ref = R.linear_backward(0, x[s], w[e], None, dy[s])
        R.check("dx", dx[s], ref["dx"])
        R.check("dw", dw[e], ref["dw0"])
    assert (dw[598] == 0).all() and (dw[512].abs().sum() > 0)


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("act,at_low,at_high", [(0, (-1, 1), (1, 1)), (1, (0, 0), (1, 1)), (2, (0, 0), (1, 1)),
                                                (3, (0, 0), (1, 1)), (4, (0, 0), (1, 1)), (5, (0, 0), (0, 0))])
def test_saved_infinities_and_nan_of_the_gated_block(N, act, at_low, at_high, dt):
    """g saved as an infinity: du = dh act(g) and dg = dh u act'(g) are the limits (at_*: the sign of an infinite act, 0: finite;
    act'), zero where dh is, whatever lies beside; a NaN stays in its row and expert."""
    inf = float("inf")
    E, K, M, P = 3, 8, 8, 15
    counts = [5, 4, 6]
    offs, slices, P = rows_of(counts, 0, 0)
    eye = torch.eye(M, dtype=dt, device="cuda").repeat(E, 1, 1)
    x, u = torch.ones(P, K, dtype=dt, device="cuda"), torch.ones(P, M, dtype=dt, device="cuda")
    g = torch.ones(P, M, dtype=dt, device="cuda")
    g[5:9, ::2], g[5:9, 1::2] = -inf, inf  # the second expert's
    dh = torch.ones(P, M, dtype=dt, device="cuda")
    d = N.experts_dims(E, K, M, N.dtype_code(x), act)
    ws, _ = workspace(N, d, P, True)

    def run():
        dx, dwg, dwu = torch.empty_like(x), torch.empty_like(eye), torch.empty_like(eye)
        N.moe_experts_gated_backward(d, x, offs, eye, eye, g, u, dh, ws, dx=dx, dw_gate=dwg, dw_up=dwu)
        assert N.moe_check_device_error(ws) == 0
        return dx, dwg, dwu

    dx, dwg, dwu = run()
    slope = torch.tensor([at_low[1], at_high[1]] * 4, dtype=torch.float64, device="cuda")
    assert torch.equal(dwg[1].double(), (4 * slope)[:, None].expand(M, K))
    sign = torch.tensor([at_low[0], at_high[0]] * 4, device="cuda")
    for j in range(M):
        if sign[j]:
            assert (dwu[1, j] == sign[j].item() * inf).all()
        else:  # act's limit: sigmoid 0 and 1, the others 0 below
            assert (dwu[1, j] == (4.0 if act == 5 and j % 2 else 0.0)).all()
    assert torch.isfinite(dx[:5]).all() and torch.isfinite(dx[9:]).all() and torch.isfinite(dwu[[0, 2]]).all()
    # nothing comes back where dh is zero
    dh[5:9] = 0
    u[5:9] = inf
    dx0, dwg0, dwu0 = run()
    assert (dx0[5:9] == 0).all() and (dwg0[1] == 0).all() and (dwu0[1] == 0).all()
    # a NaN: its row's dx, and its output's row of dW of its expert
    g[10, 3] = float("nan")
    dx1, dwg1, dwu1 = run()
    assert torch.isnan(dx1[10]).all() and torch.isnan(dwu1[2, 3]).all()
    # without an activation, and with relu, act' of a NaN is a number
    assert torch.isnan(dwg1[2, 3]).all() if act not in (0, 4) else torch.isfinite(dwg1[2, 3]).all()
    rows, outs = torch.ones(P, dtype=torch.bool, device="cuda"), torch.ones(E, M, dtype=torch.bool, device="cuda")
    rows[10], outs[2, 3] = False, False
    assert torch.equal(dx1[rows], dx0[rows]) and torch.equal(dwg1[outs], dwg0[outs]) and torch.equal(dwu1[outs], dwu0[outs])


@pytest.mark.parametrize("K,M", [(1 << 20, 24), (24, 1 << 20), ((1 << 20) - 1, 9)])
def test_widest_rows(N, K, M):
    """2^20 inputs or outputs, of whole numbers: every sum is exact in fp32."""
    gen = gen_for(95)
    counts = [5, 0, 70]
    offs, slices, P = rows_of(counts, 1, 1)
    whole = lambda *s: torch.randint(-1, 2, s, generator=gen, device="cuda").to(BF16)  # noqa: E731
    x, w, dy = whole(P, K), whole(3, M, K), whole(P, M)
    d = N.experts_dims(3, K, M, N.MOE_BF16)
    ws, guard = workspace(N, d, P, True)
    y, dx, dw = Out((P, M), BF16), Out((P, K), BF16), torch.empty_like(w)
    N.moe_experts_linear_forward(d, x, offs, w, y.t, ws)
    N.moe_experts_linear_backward(d, x, offs, w, dy, ws, dx=dx.t, dw=dw)
    for e in range(3):
        s = slices[e]
        assert torch.equal(y.t[s], (x[s].double() @ w[e].double().T).to(BF16))
        assert torch.equal(dx.t[s], (dy[s].double() @ w[e].double()).to(BF16))
        assert torch.equal(dw[e], (dy[s].double().T @ x[s].double()).to(BF16))
    assert y.untouched() and dx.untouched() and guard_ok(guard) and N.moe_check_device_error(ws) == 0
