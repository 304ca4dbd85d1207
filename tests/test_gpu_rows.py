"""Rows by expert on the GPU against float64, elementwise within derived bounds.

Bounds (e = 2^-24): a token's sum of k + 1 terms in fp32, each product rounded: 2 (k + 1) e sum|terms|; w dy one product:
e |v|; dw a sum of H products in any order: 2 H e sum|terms|; then the result's own rounding (dense_reference._round)."""

import pytest
import torch

import dense_reference as R
from test_gpu_dense import Out, rnd

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


def layout(gen, T, k, E, pad=1, drop=0.0):
    """perm, inv and the number of rows: pairs sorted by a random expert, groups padded, some pairs dropped."""
    ids = torch.rand(T, E, generator=gen, device="cuda").topk(k, dim=1).indices.flatten()
    kept = torch.rand(T * k, generator=gen, device="cuda") >= drop
    perm, used = [], 0
    for e in range(E):
        mine = torch.nonzero((ids == e) & kept)[:, 0].to(torch.int32)
        fill = -len(mine) % pad
        perm += [mine, torch.full((fill,), -1 - e, dtype=torch.int32, device="cuda")]
        used += len(mine) + fill
    perm = torch.cat(perm + [torch.full((3 if pad > 1 or not used else 0,), -1, dtype=torch.int32, device="cuda")])
    inv = torch.full((T * k,), -1, dtype=torch.int32, device="cuda")
    rows = torch.nonzero(perm >= 0)[:, 0]
    inv[perm[rows].long()] = rows.to(torch.int32)
    return perm, inv.view(T, k)


def workspace(N, d, T):
    ws = torch.full((N.moe_rows_workspace_bytes(d, T),), 0xA5, dtype=torch.uint8, device="cuda")
    N.moe_workspace_init(ws)
    return ws


def taken(rows, inv):
    """rows[inv] in float64, zero where inv is -1."""
    return torch.where(inv[..., None] >= 0, rows.double()[inv.clamp(min=0).long()], 0.0)


def check_all(N, seed, T, k, E, H, dt, f32=False, res=False, pad=1, drop=0.0, slack=0, offset=0):
    gen = gen_for(seed)
    perm, inv = layout(gen, T, k, E, pad, drop)
    P, yt = perm.numel(), F32 if f32 else dt
    d = N.rows_dims(H, k, N.dtype_code(torch.empty(0, dtype=dt)))
    ws = workspace(N, d, T)
    t = (perm.clamp(min=0) // k).long()
    real = perm >= 0
    # dispatch
    x = rnd(gen, (T, H), dt, pad=slack, offset=offset)
    xs, got_inv = Out((P, H), dt, slack, offset), torch.full((T, k), 77, dtype=torch.int32, device="cuda")
    N.moe_dispatch_forward(d, x, T, perm, xs.t, got_inv, ws)
    assert torch.equal(got_inv, inv)
    assert torch.equal(xs.t, torch.where(real[:, None], x[t], torch.zeros((), dtype=dt, device="cuda")))
    assert xs.untouched()
    # rows whose padding ones hold NaN: nobody reads them
    rows = rnd(gen, (P, H), dt, pad=slack, offset=offset)
    rows[~real] = float("nan")
    r = rnd(gen, (T, H), yt, pad=slack, offset=offset) if res else None
    w = torch.rand(T, k, generator=gen, device="cuda")
    at = taken(rows, inv)
    rv = 0.0 if r is None else r.double()
    for name, terms in (("dx", at), ("y", at * w.double()[..., None])):
        y = Out((T, H), yt, slack, offset)
        if name == "dx":
            N.moe_dispatch_backward(d, rows, inv, T, y.t, ws, residual=r)
        else:
            N.moe_combine_forward(d, rows, inv, w, T, y.t, ws, residual=r)
        val = terms.sum(1) + rv
        err = 2 * (k + 1) * R.E * (terms.abs().sum(1) + (0.0 if r is None else r.double().abs()))
        R.check(name, y.t, (val, R._round(val, err, yt)))
        assert y.untouched()
    # combine's gradients, together and each alone
    dy = rnd(gen, (T, H), yt, 0.1, slack, offset)
    dys, dw = Out((P, H), dt, slack, offset), torch.full((T, k), float("nan"), device="cuda")
    N.moe_combine_backward(d, dy, T, perm, inv, w, ws, ys=rows, dys=dys.t, dtopk_w=dw)
    val = torch.where(real[:, None], w.double().flatten()[perm.clamp(min=0).long()][:, None] * dy.double()[t], 0.0)
    R.check("dys", dys.t, (val, R._round(val, R.E * val.abs(), dt)))
    assert dys.untouched()
    prod = at * dy.double()[:, None, :]
    val = prod.sum(2)
    R.check("dw", dw, (val, R._round(val, 2 * H * R.E * prod.abs().sum(2), F32)))
    dys2, dw2 = Out((P, H), dt, slack, offset), torch.full((T * k,), float("nan"), device="cuda")
    N.moe_combine_backward(d, dy, T, perm, inv, w, ws, dys=dys2.t)
    N.moe_combine_backward(d, dy, T, perm, inv, w, ws, ys=rows, dtopk_w=dw2)
    assert torch.equal(dys2.t, dys.t) and torch.equal(dw2.view(T, k), dw)
    assert N.moe_check_device_error(ws) == 0


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("T,k,E,H", [(1, 1, 1, 1), (1, 10, 512, 2048), (3, 2, 4, 7), (8, 10, 16, 64), (17, 3, 5, 129),
                                     (70, 16, 16, 512), (333, 4, 60, 1357), (2100, 7, 9, 40), (2049, 2, 8, 1000)])
def test_against_float64(N, T, k, E, H, dt):
    check_all(N, T + H, T, k, E, H, dt)
    check_all(N, T + H + 1, T, k, E, H, dt, f32=True, res=True)


@pytest.mark.parametrize("k", range(1, 17))
def test_every_top_k(N, k):
    check_all(N, 40 + k, 37, k, 16, 72, BF16, res=True)


@pytest.mark.parametrize("T,k,E,H,pad,drop", [(1, 2, 4, 24, 16, 0.5), (50, 4, 7, 200, 16, 0.3), (300, 2, 33, 1030, 8, 0.1),
                                              (20, 3, 5, 64, 1, 1.0), (1500, 6, 300, 96, 64, 0.2), (9, 1, 2, 3000, 4, 0.5)])
def test_padding_rows_and_dropped_pairs(N, T, k, E, H, pad, drop):
    check_all(N, 7 * T + pad, T, k, E, H, F16, f32=True, res=True, pad=pad, drop=drop)
    check_all(N, 7 * T + pad, T, k, E, H, BF16, pad=pad, drop=drop)


@pytest.mark.parametrize("slack,offset", [(1, 0), (0, 1), (3, 5), (8, 8), (7, 1)])
def test_strides_and_alignments(N, slack, offset):
    check_all(N, 90 + slack, 41, 5, 8, 250, BF16, res=True, pad=4, slack=slack, offset=offset)
    check_all(N, 91 + slack, 41, 5, 8, 61, F16, f32=True, res=True, slack=slack, offset=offset)


def test_values_at_the_limits(N):
    """Infinities and NaN stay in their own token; fp16 sums past 65504 become infinite; weights of zero and negative
    ones count as any other."""
    T, k, H = 4, 2, 16
    d = N.rows_dims(H, k, N.MOE_F16)
    ws = workspace(N, d, T)
    perm = torch.arange(T * k, dtype=torch.int32, device="cuda").flip(0).contiguous()
    inv = torch.empty(T, k, dtype=torch.int32, device="cuda")
    x = torch.ones(T, H, dtype=F16, device="cuda")
    x[0], x[1], x[2] = float("inf"), float("nan"), 60000.0
    xs = torch.empty(T * k, H, dtype=F16, device="cuda")
    N.moe_dispatch_forward(d, x, T, perm, xs, inv, ws)
    assert torch.equal(xs[inv[:, 0].long()].nan_to_num(7.0), x.nan_to_num(7.0))
    w = torch.tensor([[1.0, 1.0], [1.0, 0.0], [1.0, 1.0], [-1.0, 0.25]], device="cuda")
    y = torch.empty(T, H, dtype=F16, device="cuda")
    N.moe_combine_forward(d, xs, inv, w, T, y, ws)
    assert torch.isinf(y[0]).all() and torch.isnan(y[1]).all() and torch.isinf(y[2]).all() and (y[3] == -0.75).all()


@pytest.mark.parametrize("T,H", [(30, 200), (30, 7), (30, 65), (30, 515), (30, 521), (40, 2049), (40, 4099), (2100, 521),
                                 (17000, 515), (17000, 1025), (17000, 131)])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_in_place_on_the_residual(N, T, H, dt):
    """Odd widths too, whose last chunk reaches into the one before it, in another pass or wave."""
    gen = gen_for(5 + H)
    k = 3
    perm, inv = layout(gen, T, k, 4)
    d = N.rows_dims(H, k, N.MOE_BF16)
    ws = workspace(N, d, T)
    rows, w, y = rnd(gen, (T * k, H), BF16), torch.rand(T, k, generator=gen, device="cuda"), rnd(gen, (T, H), dt)
    for call in (lambda out, r: N.moe_combine_forward(d, rows, inv, w, T, out, ws, residual=r),
                 lambda out, r: N.moe_dispatch_backward(d, rows, inv, T, out, ws, residual=r)):
        want, got = torch.empty_like(y), y.clone()
        call(want, y)
        call(got, got)
        assert torch.equal(got, want)


@pytest.mark.parametrize("T", [6, 1200])  # the inverse map in one workgroup, and by all
def test_bad_layouts_are_reported_and_stay_in_bounds(N, T):
    k, H = 2, 40
    gen = gen_for(6)
    perm, inv = layout(gen, T, k, 4)
    P = perm.numel()
    d = N.rows_dims(H, k, N.MOE_BF16)
    ws = workspace(N, d, T)
    x, rows, w = rnd(gen, (T, H), BF16), rnd(gen, (P, H), BF16), torch.rand(T, k, generator=gen, device="cuda")
    for bad in (T * k, 1 << 30, 2 ** 31 - 1):  # a pair that does not exist: a zero row
        p = perm.clone()
        p[1] = bad
        xs, got = Out((P, H), BF16), torch.empty(T, k, dtype=torch.int32, device="cuda")
        N.moe_dispatch_forward(d, x, T, p, xs.t, got, ws)
        assert N.moe_check_device_error(ws) == N.DERR_ROWS and N.moe_check_device_error(ws) == 0
        assert (xs.t[1] == 0).all() and xs.untouched() and got.flatten()[perm[1].long()] == -1
    p = perm.clone()
    p[3] = p[0]  # a pair in two rows: the later one
    xs, got = Out((P, H), BF16), torch.empty(T, k, dtype=torch.int32, device="cuda")
    N.moe_dispatch_forward(d, x, T, p, xs.t, got, ws)
    assert N.moe_check_device_error(ws) == N.DERR_ROWS
    assert got.flatten()[p[0].long()] == 3 and xs.untouched()
    for bad in (P, 2 ** 31 - 1):  # a row that does not exist: an absent pair
        i = inv.clone()
        i[T - 1, 1] = bad
        y = Out((T, H), BF16)
        N.moe_combine_forward(d, rows, i, w, T, y.t, ws)
        assert N.moe_check_device_error(ws) == N.DERR_ROWS and y.untouched()
        val = taken(rows, torch.where(i >= P, -1, i)) * w.double()[..., None]
        R.check("y", y.t, (val.sum(1), R._round(val.sum(1), 6 * R.E * val.abs().sum(1), BF16)))
        dys, dw = Out((P, H), BF16), torch.empty(T, k, device="cuda")
        N.moe_combine_backward(d, x, T, perm, i, w, ws, ys=rows, dys=dys.t, dtopk_w=dw)
        assert N.moe_check_device_error(ws) == N.DERR_ROWS and dys.untouched()
        assert dw[T - 1, 1] == 0 and (dys.t[inv[T - 1, 1].long()] == 0).all()
    i = inv.clone()
    i[0, 0] = i[1, 1]  # two pairs in one row: perm says whose it is
    dys = Out((P, H), BF16)
    N.moe_combine_backward(d, x, T, perm, i, w, ws, dys=dys.t)
    assert N.moe_check_device_error(ws) == N.DERR_ROWS and dys.untouched()
    val = w[1, 1].double() * x[1].double()
    R.check("dys", dys.t[i[1, 1].long()], (val, R._round(val, R.E * val.abs(), BF16)))


def test_equal_calls_give_equal_bits_captured_too(N):
    gen = gen_for(8)
    T, k, H = 300, 10, 264
    perm, inv = layout(gen, T, k, 40, pad=8, drop=0.1)
    P = perm.numel()
    d = N.rows_dims(H, k, N.MOE_BF16)
    ws = workspace(N, d, T)
    x, dy, w = rnd(gen, (T, H), BF16), rnd(gen, (T, H), BF16), torch.rand(T, k, generator=gen, device="cuda")

    def step(o):
        N.moe_dispatch_forward(d, x, T, perm, o["xs"], o["inv"], ws)
        N.moe_combine_forward(d, o["xs"], o["inv"], w, T, o["y"], ws, residual=x)
        N.moe_combine_backward(d, dy, T, perm, o["inv"], w, ws, ys=o["xs"], dys=o["dys"], dtopk_w=o["dw"])
        N.moe_dispatch_backward(d, o["dys"], o["inv"], T, o["dx"], ws, residual=dy)

    def outs():
        e = lambda *s, dt=BF16: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
        return {"xs": e(P, H), "inv": e(T, k, dt=torch.int32), "y": e(T, H), "dys": e(P, H), "dw": e(T, k, dt=F32),
                "dx": e(T, H)}

    cap = outs()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(cap)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(cap)
    for rep in range(4):
        x.copy_(rnd(gen, (T, H), BF16))
        for v in cap.values():
            v.fill_(3)
        eager = outs()
        step(eager)
        g.replay()
        torch.cuda.synchronize()
        for n in eager:
            assert torch.equal(eager[n], cap[n]), (rep, n)


def test_group_tokens_layout(N):
    """The layer's own sort is a layout these calls take: counts, offsets and perm of moe_group_tokens."""
    T, k, E, H = 300, 10, 512, 256
    gen = gen_for(11)
    layer = N.dims(H, 128, E, k)
    ids = torch.rand(T, E, generator=gen, device="cuda").topk(k, dim=1).indices.to(torch.int32).contiguous()
    wl = torch.empty(N.moe_workspace_bytes(layer, T), dtype=torch.uint8, device="cuda")
    N.moe_workspace_init(wl)
    counts, offsets = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (E, E + 1))
    perm, inv = torch.empty(T * k, dtype=torch.int32, device="cuda"), torch.empty(T, k, dtype=torch.int32, device="cuda")
    N.moe_group_tokens(layer, ids, T, counts, offsets, perm, wl)
    d = N.rows_dims(H, k, N.MOE_BF16)
    x, xs = rnd(gen, (T, H), BF16), torch.empty(T * k, H, dtype=BF16, device="cuda")
    N.moe_dispatch_forward(d, x, T, perm, xs, inv, wl)  # on the layer's workspace
    assert N.moe_check_device_error(wl) == 0
    rows = inv.flatten().long()
    assert torch.equal(perm[rows], torch.arange(T * k, dtype=torch.int32, device="cuda"))
    e = ids.flatten().long()
    assert ((rows >= offsets[e]) & (rows < offsets[e + 1])).all()
    assert torch.equal(xs[rows], x.repeat_interleave(k, 0))


def test_more_than_2_31_elements(N):
    """Rows whose element offsets pass 32 bits, at a wide stride: sampled."""
    T, k, H, ld = 66000, 1, 8, 65536
    gen = gen_for(12)
    wide = torch.empty(T, ld, dtype=BF16, device="cuda")
    x, d = wide[:, :H], N.rows_dims(H, k, N.MOE_BF16)
    x.copy_(rnd(gen, (T, H), BF16))
    out = torch.empty(T, ld, dtype=BF16, device="cuda")
    xs = out[:, 8:8 + H]
    ws = workspace(N, d, T)
    perm = torch.arange(T, dtype=torch.int32, device="cuda").flip(0).contiguous()
    inv, w, y = torch.empty_like(perm).view(T, 1), torch.ones(T, 1, device="cuda"), torch.empty(T, H, dtype=F32, device="cuda")
    N.moe_dispatch_forward(d, x, T, perm, xs, inv, ws)
    assert torch.equal(xs, x.flip(0))
    N.moe_combine_forward(d, xs, inv, w, T, y, ws)
    assert torch.equal(y, x.float())
    dys, dw = out[:, :H], torch.empty(T, 1, device="cuda")
    N.moe_combine_backward(d, x, T, perm, inv, w, ws, ys=xs, dys=dys, dtopk_w=dw)
    assert torch.equal(dys, x.flip(0))
    assert N.moe_check_device_error(ws) == 0


def test_most_tokens(N):
    """2^24 tokens, the limit, a pair each, reversed."""
    T, H = 1 << 24, 8
    gen = gen_for(13)
    d = N.rows_dims(H, 1, N.MOE_BF16)
    ws = workspace(N, d, T)
    x = rnd(gen, (T, H), BF16)
    perm = torch.arange(T - 1, -1, -1, dtype=torch.int32, device="cuda")
    perm[5], perm[T - 7] = -1, -1
    xs, inv = torch.empty_like(x), torch.empty(T, 1, dtype=torch.int32, device="cuda")
    N.moe_dispatch_forward(d, x, T, perm, xs, inv, ws)
    want = x.flip(0)
    want[5], want[T - 7] = 0, 0
    assert torch.equal(xs, want) and (inv == -1).sum() == 2 and inv[0, 0] == T - 1
    y, w = torch.empty_like(x), torch.ones(T, 1, device="cuda")
    N.moe_combine_forward(d, xs, inv, w, T, y, ws)
    assert torch.equal(y, want.flip(0))
    dys = torch.full_like(x, 7.0)
    N.moe_combine_backward(d, x, T, perm, inv, w, ws, dys=dys)
    assert torch.equal(dys, want) and N.moe_check_device_error(ws) == 0
    with pytest.raises(N.MoeError) as e:
        N.moe_combine_forward(d, xs, inv, w, T + 1, y, ws)
    assert e.value.code == N.MOE_EINVAL


@pytest.mark.parametrize("T,H", [(30, 7), (30, 65), (30, 521), (2100, 521), (17000, 131)])
def test_in_place_on_the_residual_in_fp16(N, T, H):
    gen = gen_for(15 + H)
    k = 3
    perm, inv = layout(gen, T, k, 4, pad=4, drop=0.2)
    d = N.rows_dims(H, k, N.MOE_F16)
    ws = workspace(N, d, T)
    rows, w, y = rnd(gen, (perm.numel(), H), F16), torch.rand(T, k, generator=gen, device="cuda"), rnd(gen, (T, H), F16)
    for call in (lambda out, r: N.moe_combine_forward(d, rows, inv, w, T, out, ws, residual=r),
                 lambda out, r: N.moe_dispatch_backward(d, rows, inv, T, out, ws, residual=r)):
        want, got = torch.empty_like(y), y.clone()
        call(want, y)
        call(got, got)
        assert torch.equal(got, want)


@pytest.mark.parametrize("H", [1 << 20, (1 << 20) - 3])
def test_widest_rows(N, H):
    check_all(N, 16, 5, 3, 4, H, BF16, f32=True, res=True, pad=2, drop=0.2)
