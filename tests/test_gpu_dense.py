"""The dense operators on the GPU against float64, elementwise within the bounds of dense_reference."""

import pytest
import torch

import dense_reference as R

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
ACTS = range(6)


@pytest.fixture(scope="module")
def N():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mixture_experts_route_amd import native

    return native


def rnd(gen, shape, dt, scale=1.0, pad=0, offset=0):
    """Normal values in a tensor of its own, or (pad, offset > 0) as a slice of wider rows whose other elements
    are NaN: reading them shows in the result."""
    v = (torch.randn(shape, generator=gen, device="cuda") * scale).to(dt)
    if not pad and not offset:
        return v
    rows = shape[0] if len(shape) == 2 else 1
    wide = torch.full((rows, offset + shape[-1] + pad), float("nan"), dtype=dt, device="cuda")
    s = wide[:, offset:offset + shape[-1]]
    s.copy_(v.view(rows, -1))
    return s if len(shape) == 2 else s[0]


class Out:
    """An output of NaNs (never read) inside a larger buffer of NaNs that must stay as they are."""

    def __init__(self, shape, dt, pad=0, offset=0):
        rows, cols = shape if len(shape) == 2 else (1, shape[0])
        self.buf = torch.full((rows + 2, offset + cols + pad), float("nan"), dtype=dt, device="cuda")
        self.rows, self.cols, self.offset = rows, cols, offset
        s = self.buf[1:rows + 1, offset:offset + cols]
        self.t = s if len(shape) == 2 else s[0]

    def untouched(self):
        inside = torch.zeros(self.buf.shape, dtype=torch.bool, device="cuda")
        inside[1:self.rows + 1, self.offset:self.offset + self.cols] = True
        return bool(torch.isnan(self.buf[~inside]).all())


def workspace(N, d, T, backward):
    """Exactly the stated bytes, not cleared beyond the control area, with a guard behind them."""
    n = N.moe_dense_workspace_bytes(d, T, backward)
    whole = torch.full((n + 1024,), 0xA5, dtype=torch.uint8, device="cuda")
    ws = whole[:n]
    N.moe_workspace_init(ws)
    return ws, whole


def guard_ok(whole):
    return bool((whole[-1024:] == 0xA5).all())


def run_linear_forward(N, gen, T, K, M, dt, a, bias=False, res=False, ydt=None, save=False, pad=0, offset=0):
    ydt = ydt or dt
    x = rnd(gen, (T, K), dt, pad=pad, offset=offset)
    w = rnd(gen, (M, K), dt, K ** -0.5, pad=pad, offset=offset)
    b = rnd(gen, (M,), dt, pad=pad, offset=offset) if bias else None
    r = rnd(gen, (T, M), ydt, pad=pad, offset=offset) if res else None
    d = N.dense_dims(K, M, N.dtype_code(x), a)
    ws, whole = workspace(N, d, T, False)
    y, pre = Out((T, M), ydt, pad, offset), Out((T, M), dt, pad, offset)
    N.moe_linear_forward(d, x, T, w, y.t, ws, bias=b, residual=r, pre=pre.t if save else None)
    torch.cuda.synchronize()
    ref = R.linear_forward(a, x, w, b, r, ydt)
    R.check("y", y.t, ref["y"])
    if save:
        R.check("pre", pre.t, ref["pre"])
    else:
        assert torch.isnan(pre.buf).all()
    assert y.untouched() and pre.untouched() and guard_ok(whole)


def run_gated_forward(N, gen, T, K, M, dt, a, bias=False, save=False, pad=0, offset=0, fused=False):
    x = rnd(gen, (T, K), dt, pad=pad, offset=offset)
    if fused:  # the halves of one tensor
        both = rnd(gen, (2 * M, K), dt, K ** -0.5, pad=pad, offset=offset)
        wg, wu = both[:M], both[M:]
    else:
        wg, wu = (rnd(gen, (M, K), dt, K ** -0.5, pad=pad, offset=offset) for _ in range(2))
    bg, bu = (rnd(gen, (M,), dt, pad=pad, offset=offset) if bias else None for _ in range(2))
    d = N.dense_dims(K, M, N.dtype_code(x), a)
    ws, whole = workspace(N, d, T, False)
    h, g, u = (Out((T, M), dt, pad, offset) for _ in range(3))
    N.moe_gated_forward(d, x, T, wg, wu, h.t, ws, gate_bias=bg, up_bias=bu, gate=g.t if save else None,
                        up=u.t if save else None)
    torch.cuda.synchronize()
    ref = R.gated_forward(a, x, wg, wu, bg, bu)
    R.check("h", h.t, ref["h"])
    if save:
        R.check("gate", g.t, ref["gate"])
        R.check("up", u.t, ref["up"])
    assert h.untouched() and g.untouched() and u.untouched() and guard_ok(whole)


def run_linear_backward(N, gen, T, K, M, dt, a, want=("dx", "dw", "db"), pad=0, offset=0):
    x = rnd(gen, (T, K), dt, pad=pad, offset=offset)
    w = rnd(gen, (M, K), dt, K ** -0.5, pad=pad, offset=offset)
    pre = rnd(gen, (T, M), dt, pad=pad, offset=offset) if a else None
    dy = rnd(gen, (T, M), dt, 0.5, pad=pad, offset=offset)
    d = N.dense_dims(K, M, N.dtype_code(x), a)
    ws, whole = workspace(N, d, T, True)
    out = {"dx": Out((T, K), dt, pad, offset), "dw": Out((M, K), dt, pad, offset), "db": Out((M,), dt, pad, offset)}
    t = {k: v.t if k in want else None for k, v in out.items()}
    N.moe_linear_backward(d, x, T, w, dy, ws, pre=pre, dx=t["dx"], dw=t["dw"], dbias=t["db"])
    torch.cuda.synchronize()
    ref = R.linear_backward(a, x, w, pre, dy)
    for k, rk in (("dx", "dx"), ("dw", "dw0"), ("db", "db0")):
        if k in want:
            R.check(k, out[k].t, ref[rk])
        else:
            assert torch.isnan(out[k].buf).all()
    assert all(o.untouched() for o in out.values()) and guard_ok(whole)


def run_gated_backward(N, gen, T, K, M, dt, a, want=("dx", "dwg", "dwu", "dbg", "dbu"), pad=0, offset=0):
    x = rnd(gen, (T, K), dt, pad=pad, offset=offset)
    wg, wu = (rnd(gen, (M, K), dt, K ** -0.5, pad=pad, offset=offset) for _ in range(2))
    g, u, dh = (rnd(gen, (T, M), dt, pad=pad, offset=offset) for _ in range(3))
    d = N.dense_dims(K, M, N.dtype_code(x), a)
    ws, whole = workspace(N, d, T, True)
    out = {"dx": Out((T, K), dt, pad, offset), "dwg": Out((M, K), dt, pad, offset), "dwu": Out((M, K), dt, pad, offset),
           "dbg": Out((M,), dt, pad, offset), "dbu": Out((M,), dt, pad, offset)}
    t = {k: v.t if k in want else None for k, v in out.items()}
    N.moe_gated_backward(d, x, T, wg, wu, g, u, dh, ws, dx=t["dx"], dw_gate=t["dwg"], dw_up=t["dwu"],
                         dgate_bias=t["dbg"], dup_bias=t["dbu"])
    torch.cuda.synchronize()
    ref = R.gated_backward(a, x, wg, wu, g, u, dh)
    for k, rk in (("dx", "dx"), ("dwg", "dw0"), ("dwu", "dw1"), ("dbg", "db0"), ("dbu", "db1")):
        if k in want:
            R.check(k, out[k].t, ref[rk])
        else:
            assert torch.isnan(out[k].buf).all()
    assert all(o.untouched() for o in out.values()) and guard_ok(whole)


# tokens, n_in, n_out: one of everything, below / at / above the vector, step and tile sizes, odd and prime
SHAPES = [(1, 1, 1), (1, 8, 16), (2, 7, 5), (5, 64, 48), (15, 72, 20), (16, 200, 130), (17, 136, 65), (33, 63, 8),
          (64, 256, 128), (65, 264, 257), (128, 128, 128), (129, 1000, 1357), (200, 72, 520), (256, 512, 512),
          (257, 40, 264), (1, 2048, 768), (8, 4096, 1000), (300, 2056, 384)]


def gen_for(*key):
    return torch.Generator(device="cuda").manual_seed(hash(key) % (1 << 31))


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_linear_forward_shapes(N, shape):
    gen = gen_for(1, *shape)
    run_linear_forward(N, gen, *shape, BF16, 1, bias=True, res=True, save=True)
    run_linear_forward(N, gen, *shape, F16, 0, bias=True, res=True, ydt=F32)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gated_forward_shapes(N, shape):
    gen = gen_for(2, *shape)
    run_gated_forward(N, gen, *shape, BF16, 1, save=True, fused=True)
    run_gated_forward(N, gen, *shape, F16, 3, bias=True)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_linear_backward_shapes(N, shape):
    gen = gen_for(3, *shape)
    run_linear_backward(N, gen, *shape, BF16, 0)
    run_linear_backward(N, gen, *shape, F16, 2)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gated_backward_shapes(N, shape):
    gen = gen_for(4, *shape)
    run_gated_backward(N, gen, *shape, BF16, 1)
    run_gated_backward(N, gen, *shape, F16, 2)


@pytest.mark.parametrize("a", ACTS)
@pytest.mark.parametrize("shape", [(6, 96, 40), (150, 192, 136)], ids=str)
def test_every_activation(N, a, shape):
    gen = gen_for(5, a, *shape)
    for dt in (BF16, F16):
        run_linear_forward(N, gen, *shape, dt, a, bias=True, ydt=F32, save=True)
        run_gated_forward(N, gen, *shape, dt, a, bias=True)
        run_linear_backward(N, gen, *shape, dt, a)
        run_gated_backward(N, gen, *shape, dt, a)


@pytest.mark.parametrize("pad,offset", [(8, 8), (3, 0), (1, 1), (0, 5), (2, 4)])
@pytest.mark.parametrize("shape", [(3, 128, 64), (40, 200, 136), (260, 264, 300)], ids=str)
def test_slices_of_wider_rows(N, pad, offset, shape):
    """Strides and addresses of every alignment; nothing between the rows is read into a result or written."""
    gen = gen_for(6, pad, offset, *shape)
    run_linear_forward(N, gen, *shape, BF16, 1, bias=True, res=True, ydt=F32, save=True, pad=pad, offset=offset)
    run_linear_forward(N, gen, *shape, F16, 0, bias=True, res=True, pad=pad, offset=offset)
    run_gated_forward(N, gen, *shape, BF16, 1, bias=True, save=True, pad=pad, offset=offset, fused=True)
    run_linear_backward(N, gen, *shape, F16, 1, pad=pad, offset=offset)
    run_linear_backward(N, gen, *shape, BF16, 0, pad=pad, offset=offset)
    run_gated_backward(N, gen, *shape, BF16, 4, pad=pad, offset=offset)


@pytest.mark.parametrize("step", [8, 3])
@pytest.mark.parametrize("shape", [(5, 128, 64), (90, 200, 136), (300, 520, 264)], ids=str)
def test_every_matrix_its_own_stride(N, shape, step):
    """The gated block with a different row stride for every operand and output, whole 16-byte rows or odd."""
    T, K, M = shape
    gen = gen_for(21, T, step)
    pads = iter(range(step, 20 * step, step))
    x = rnd(gen, (T, K), BF16, pad=next(pads))
    wg, wu = (rnd(gen, (M, K), BF16, K ** -0.5, pad=next(pads)) for _ in range(2))
    dh = rnd(gen, (T, M), BF16, pad=next(pads))
    h, g, u = (Out((T, M), BF16, next(pads)) for _ in range(3))
    dx, dwg, dwu = Out((T, K), BF16, next(pads)), Out((M, K), BF16, next(pads)), Out((M, K), BF16, next(pads))
    d = N.dense_dims(K, M, N.MOE_BF16, N.MOE_ACT_SILU)
    ws, whole = workspace(N, d, T, True)
    N.moe_gated_forward(d, x, T, wg, wu, h.t, ws, gate=g.t, up=u.t)
    N.moe_gated_backward(d, x, T, wg, wu, g.t, u.t, dh, ws, dx=dx.t, dw_gate=dwg.t, dw_up=dwu.t)
    torch.cuda.synchronize()
    ref = R.gated_forward(N.MOE_ACT_SILU, x, wg, wu, None, None)
    for k, o in (("h", h), ("gate", g), ("up", u)):
        R.check(k, o.t, ref[k])
    ref = R.gated_backward(N.MOE_ACT_SILU, x, wg, wu, g.t, u.t, dh)
    for k, o in (("dx", dx), ("dw0", dwg), ("dw1", dwu)):
        R.check(k, o.t, ref[k])
    assert all(o.untouched() for o in (h, g, u, dx, dwg, dwu)) and guard_ok(whole)


@pytest.mark.parametrize("want", [("dx",), ("dw",), ("db",), ("dx", "db"), ("dw", "db")], ids="-".join)
def test_linear_backward_wanted_outputs(N, want):
    for a in (0, 1):
        run_linear_backward(N, gen_for(7, a), 70, 136, 72, BF16, a, want=want)


@pytest.mark.parametrize("want", [("dx",), ("dwg",), ("dwu",), ("dbg",), ("dbu",), ("dx", "dwu", "dbg"),
                                  ("dwg", "dwu")], ids="-".join)
def test_gated_backward_wanted_outputs(N, want):
    run_gated_backward(N, gen_for(8), 70, 136, 72, BF16, 1, want=want)


# long reductions and enough tiles for every kernel; reductions over many tokens
@pytest.mark.parametrize("shape", [(4096, 512, 768), (700, 8192, 256), (3000, 96, 2048), (2100, 1024, 1100),
                                   (20, 8192, 2048), (5, 264, 20011), (1030, 4096, 4096)], ids=str)
def test_large(N, shape):
    gen = gen_for(9, *shape)
    run_linear_forward(N, gen, *shape, BF16, 0, res=True, ydt=F32)
    run_gated_forward(N, gen, *shape, BF16, 1, save=True)
    run_linear_backward(N, gen, *shape, BF16, 0)
    run_gated_backward(N, gen, *shape, F16, 1)


# a few more tiles than fill the chip: those of the last rows share their reductions (both large tiles, each product)
@pytest.mark.parametrize("shape", [(2200, 4104, 4050), (4240, 4104, 4010), (4400, 4104, 2050)], ids=str)
def test_last_tiles_in_parts(N, shape):
    gen = gen_for(23, *shape)
    run_linear_forward(N, gen, *shape, BF16, 2, bias=True, res=True, save=True)
    run_gated_forward(N, gen, *shape, F16, 1, bias=True, save=True)
    run_linear_backward(N, gen, *shape, F16, 0)
    run_gated_backward(N, gen, *shape, BF16, 1)


@pytest.mark.parametrize("splits", [1, 2, 3, 8])
@pytest.mark.parametrize("kernel", [1, 2, 3, 4, 5], ids=["tile64", "tile128", "tile256", "any64", "any128"])
def test_every_kernel_and_split(N, kernel, splits):
    """Each tile kernel at sizes inside, at and past its tile, with the reduction in one piece and in parts (fewer steps
    than parts among them), and the few-token kernel in as many parts."""
    N.moe_debug_force_dense_plan(kernel, splits)
    try:
        for shape in ((20, 64, 40), (64, 320, 64), (130, 1096, 264), (257, 512, 520), (600, 200, 136)):
            gen = gen_for(17, kernel, splits, *shape)
            run_linear_forward(N, gen, *shape, BF16, 1, bias=True, res=True, ydt=F32, save=True)
            run_gated_forward(N, gen, *shape, F16, 1, bias=True, save=True)
            run_linear_backward(N, gen, *shape, F16, 1)
            run_gated_backward(N, gen, *shape, BF16, 3)
        for shape in ((1, 64, 24), (7, 1000, 264), (16, 4160, 40)):
            gen = gen_for(18, kernel, splits, *shape)
            run_linear_forward(N, gen, *shape, BF16, 1, bias=True, res=True, ydt=F32, save=True)
            run_gated_forward(N, gen, *shape, F16, 1, bias=True, save=True)
            run_gated_forward(N, gen, *shape, BF16, 4, bias=True, pad=1, offset=1)
    finally:
        N.moe_debug_force_dense_plan()


def test_residual_in_place(N):
    """y on r exactly: every element is read before it is written."""
    for T, K, M, dt, ydt in ((4, 256, 512, BF16, F32), (300, 512, 264, F16, F16), (40, 96, 33, BF16, BF16)):
        gen = gen_for(10, T)
        x, w = rnd(gen, (T, K), dt), rnd(gen, (M, K), dt, K ** -0.5)
        y = rnd(gen, (T, M), ydt)
        ref = R.linear_forward(0, x, w, None, y.clone(), ydt)
        d = N.dense_dims(K, M, N.dtype_code(x), 0)
        ws, _ = workspace(N, d, T, False)
        N.moe_linear_forward(d, x, T, w, y, ws, residual=y)
        R.check("y", y, ref["y"])


@pytest.mark.parametrize("dt", [BF16, F16], ids=["bf16", "fp16"])
def test_equal_calls_give_equal_bits(N, dt):
    """Twice the same call, and (up to the stated count) a token alone and in any batch."""
    for K, M in ((2048, 768), (256, 4104), (1000, 50), (4096, 520), (2048, 8200)):
        gen = gen_for(11, K)
        x = rnd(gen, (N.MOE_DENSE_ROW_TOKENS, K), dt)
        w, w2 = rnd(gen, (M, K), dt, K ** -0.5), rnd(gen, (M, K), dt, K ** -0.5)
        d = N.dense_dims(K, M, N.dtype_code(x), 1)
        ws, _ = workspace(N, d, 16, False)

        def both(xs):
            t = xs.shape[0]
            y, h = (torch.empty(t, M, dtype=dt, device="cuda") for _ in range(2))
            N.moe_linear_forward(d, xs, t, w, y, ws)
            N.moe_gated_forward(d, xs, t, w, w2, h, ws)
            return y, h

        y16, h16 = both(x)
        for a, b in zip(both(x), (y16, h16)):
            assert torch.equal(a, b)
        for rows in ([0], [15], [3, 4, 5], [9, 2, 11, 0, 1, 7, 8]):
            y, h = both(x[rows].contiguous())
            assert torch.equal(y, y16[rows]) and torch.equal(h, h16[rows])


@pytest.mark.parametrize("T", [6, 300])
def test_infinities_and_nans_stay_in_their_rows(N, T):
    """A token with a NaN or an infinity spoils its own output row only, a weight row its own column only; a NaN
    stays a NaN and an overflowing sum an infinity."""
    K, M = 264, 200
    gen = gen_for(12, T)
    for dt in (BF16, F16):
        x, w, w2 = rnd(gen, (T, K), dt), rnd(gen, (M, K), dt, K ** -0.5), rnd(gen, (M, K), dt, K ** -0.5)
        x[2, 5], x[4, 263] = float("nan"), float("inf")
        w[7, 0] = float("nan")
        d = N.dense_dims(K, M, N.dtype_code(x), 0)
        ws, _ = workspace(N, d, T, False)
        y = torch.empty(T, M, dtype=dt, device="cuda")
        N.moe_linear_forward(d, x, T, w, y, ws)
        bad = torch.zeros(T, M, dtype=torch.bool, device="cuda")
        bad[2], bad[:, 7] = True, True
        assert torch.equal(torch.isnan(y), bad)
        fin = torch.isfinite(y)
        assert not fin[4].any() and torch.isinf(y[4, 8:]).all()
        bad[4] = True
        assert torch.equal(~fin, bad)
        ref = R.linear_forward(0, torch.where(torch.isfinite(x), x, 0), torch.where(torch.isfinite(w), w, 0), None,
                               None, dt)["y"]
        R.check("y", torch.where(bad, ref[0].to(dt), y), ref)
        d = N.dense_dims(K, M, N.dtype_code(x), 1)
        h = torch.empty(T, M, dtype=dt, device="cuda")
        N.moe_gated_forward(d, x, T, w, w2, h, ws)
        assert torch.equal(torch.isfinite(h) | bad, torch.ones_like(bad)) and torch.isnan(h[2]).all()
    # fp16: 70000 rounds to infinity, 65504 + 15 to the largest finite value
    x = torch.zeros(T, 16, dtype=F16, device="cuda")
    x[0, 0], x[1, 0], x[1, 1] = 35000, 32752, 0.25
    w = torch.full((8, 16), 2.0, dtype=F16, device="cuda")
    d = N.dense_dims(16, 8, N.MOE_F16, 0)
    ws, _ = workspace(N, d, T, False)
    y = torch.empty(T, 8, dtype=F16, device="cuda")
    N.moe_linear_forward(d, x, T, w, y, ws)
    assert torch.isinf(y[0]).all() and (y[1] == 65504).all() and (y[2:] == 0).all()


@pytest.mark.parametrize("a", ACTS)
def test_saved_values_far_out_give_the_derivatives_limits(N, a):
    """Pre-activations up to bf16's largest: the derivative is its limit there, 0 or 1 (dx of an identity weight
    is dz itself), and the gated block's factors are the activation's limits.  Beyond |z| = 128 every derivative
    here differs from its limit by less than exp(-128) 129 < 2^-170, so the results are exact, up to sums of
    such remainders (below 2^-100, which the rounding to bf16 may keep)."""
    z = torch.tensor([128.0, 1e3, 1e6, 1e12, 1e15, 1e20, 1e30, 3e38], device="cuda").to(BF16)
    z = torch.cat([z, -z])
    M = z.numel()
    eye = torch.eye(M, device="cuda").to(BF16)
    x = torch.ones(M, M, dtype=BF16, device="cuda")
    d = N.dense_dims(M, M, N.MOE_BF16, a)
    ws, _ = workspace(N, d, M, True)
    dx, dbg, dbu = torch.empty_like(x), torch.empty_like(z), torch.empty_like(z)
    pre = z.repeat(M, 1)
    slope = {0: (1, 1), 5: (0, 0)}.get(a, (1, 0))
    want = torch.tensor(slope, device="cuda").repeat_interleave(M // 2).double().expand(M, M)
    N.moe_linear_backward(d, x, M, eye, x, ws, pre=pre, dx=dx)
    assert ((dx.double() - want).abs() < 2.0 ** -100).all()
    N.moe_gated_backward(d, x, M, eye, torch.zeros_like(eye), pre, x, x, ws, dx=dx, dgate_bias=dbg)
    assert ((dx.double() - want).abs() < 2.0 ** -100).all()
    assert ((dbg.double() - M * want[0]).abs() < 2.0 ** -100).all()
    # du = dh act(z): z, 1 or 0; a row's 1 / M of it, so that the sum over M equal rows stays in range
    N.moe_gated_backward(d, x, M, eye, eye, pre, x, x / M, ws, dup_bias=dbu)
    value = torch.where(z > 0, z.double(), {0: z.double()}.get(a, torch.zeros_like(z).double()))
    if a == 5:
        value = (z > 0).double()
    assert ((dbu.double() - value).abs() <= 2.0 ** -8 * value.abs() + 2.0 ** -100).all()


@pytest.mark.parametrize("T", [3, 100])
def test_subnormal_operands_count(N, T):
    """fp16 values below 2^-14 enter the sums and results exactly."""
    x = torch.zeros(T, 64, dtype=F16, device="cuda")
    x[:, 5], x[:, 40] = 3 * 2.0 ** -24, 2.0 ** -20
    w = torch.ones(32, 64, dtype=F16, device="cuda")
    d = N.dense_dims(64, 32, N.MOE_F16, 0)
    ws, _ = workspace(N, d, T, False)
    y, y16 = torch.empty(T, 32, device="cuda"), torch.empty(T, 32, dtype=F16, device="cuda")
    N.moe_linear_forward(d, x, T, w, y, ws)
    N.moe_linear_forward(d, x, T, w, y16, ws)
    assert (y == 19 * 2.0 ** -24).all() and (y16.double() == 19 * 2.0 ** -24).all()


def test_gradients_match_differences(N):
    """The GPU's gradients against central differences of the float64 forward pass along random directions."""
    T, K, M = 37, 72, 56
    for a in ACTS:
        gen = gen_for(13, a)
        x, wg, wu = rnd(gen, (T, K), BF16), rnd(gen, (M, K), BF16, K ** -0.5), rnd(gen, (M, K), BF16, K ** -0.5)
        dh = rnd(gen, (T, M), BF16)
        xd, gd, ud, dd = (t.double() for t in (x, wg, wu, dh))
        d = N.dense_dims(K, M, N.MOE_BF16, a)
        ws, _ = workspace(N, d, T, True)
        g, u = (xd @ gd.T).to(BF16), (xd @ ud.T).to(BF16)
        dx, dwg, dwu = (torch.empty_like(t) for t in (x, wg, wu))
        N.moe_gated_backward(d, x, T, wg, wu, g, u, dh, ws, dx=dx, dw_gate=dwg, dw_up=dwu)

        def f(xx, ww, vv):
            return (R.act(a, xx @ ww.T) * (xx @ vv.T) * dd).sum()

        for i, grad in enumerate((dx, dwg, dwu)):
            v = torch.randn(grad.shape, generator=gen, device="cuda", dtype=torch.float64)
            eps = 1e-5
            hi = [t + eps * v if j == i else t for j, t in enumerate((xd, gd, ud))]
            lo = [t - eps * v if j == i else t for j, t in enumerate((xd, gd, ud))]
            num = (f(*hi) - f(*lo)) / (2 * eps)
            # relative to the gradient's norm times the direction's: the rounding of g, u (their slopes are at most
            # 2), of dz and of the result are each half a step, 2^-9 of their values: 2^-9 (2 + 2 + 1 + 1) at most
            # when all add up; relu's slope jumps where rounding moves g across 0, which it never does (it keeps signs)
            tol = 6 * R.half_step(BF16) * grad.double().norm() * v.norm()
            assert abs(num - (grad.double() * v).sum()) <= tol


def test_graph_replays_and_streams(N):
    """A step of all four calls captured once and replayed with eager work between; then the same on another stream."""
    T, K, M = 70, 264, 520
    gen = gen_for(14)
    x, wg, wu = rnd(gen, (T, K), BF16), rnd(gen, (M, K), BF16, K ** -0.5), rnd(gen, (M, K), BF16, K ** -0.5)
    wd, r = rnd(gen, (K, M), BF16, M ** -0.5), rnd(gen, (T, K), F32)
    dg, dd = N.dense_dims(K, M, N.MOE_BF16, N.MOE_ACT_SILU), N.dense_dims(M, K, N.MOE_BF16, N.MOE_ACT_NONE)
    n = max(N.moe_dense_workspace_bytes(dg, T, True), N.moe_dense_workspace_bytes(dd, T, True))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    N.moe_workspace_init(ws)

    def buffers():
        e = lambda *s, dt=BF16: torch.zeros(*s, dtype=dt, device="cuda")
        return {"h": e(T, M), "g": e(T, M), "u": e(T, M), "y": e(T, K, dt=F32), "dy": e(T, K), "dh": e(T, M),
                "dwd": e(K, M), "dx": e(T, K), "dwg": e(M, K), "dwu": e(M, K), "dbg": e(M), "dbu": e(M)}

    def step(b):
        N.moe_gated_forward(dg, x, T, wg, wu, b["h"], ws, gate=b["g"], up=b["u"])
        N.moe_linear_forward(dd, b["h"], T, wd, b["y"], ws, residual=r)
        b["dy"].copy_(b["y"])
        N.moe_linear_backward(dd, b["h"], T, wd, b["dy"], ws, dx=b["dh"], dw=b["dwd"])
        N.moe_gated_backward(dg, x, T, wg, wu, b["g"], b["u"], b["dh"], ws, dx=b["dx"], dw_gate=b["dwg"],
                             dw_up=b["dwu"], dgate_bias=b["dbg"], dup_bias=b["dbu"])

    eager, cap = buffers(), buffers()
    step(eager)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cap)
    for rep in range(4):
        x.copy_(rnd(gen, (T, K), BF16))
        step(eager)
        torch.cuda.synchronize()
        for v in cap.values():
            v.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for k in eager:
            assert torch.equal(eager[k], cap[k]), (rep, k)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        step(cap)
    other.synchronize()
    for k in eager:
        assert torch.equal(eager[k], cap[k]), k


def test_dense_shared_expert_on_the_routed_layer(N):
    """The pieces as a model uses them: the routed layer's fp32 output, a dense gated shared expert added onto it
    in place, and the output head's fp32 logits; one workspace for all, one token and a prompt."""
    from layer_fixtures import MODEL, Layer
    from oracle import moe_oracle as O

    dev = torch.device("cuda:0")
    layer = Layer(MODEL, dev, seed=0, layer=1)
    H, F, V = layer.H, 768, 1003
    gen = gen_for(15)
    wg, wu, wd = rnd(gen, (F, H), BF16, H ** -0.5), rnd(gen, (F, H), BF16, H ** -0.5), rnd(gen, (H, F), BF16, F ** -0.5)
    head = rnd(gen, (V, H), BF16, H ** -0.5)
    dims = layer.dims()
    up = N.dense_dims(H, F, N.MOE_BF16, N.MOE_ACT_SILU)
    down, out = N.dense_dims(F, H, N.MOE_BF16), N.dense_dims(H, V, N.MOE_BF16)
    for T in (1, 24):
        x, x64 = layer.x(T, 700 + T, dev)
        n = max(N.moe_workspace_bytes(dims, T), *(N.moe_dense_workspace_bytes(d, T) for d in (up, down, out)))
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        N.moe_workspace_init(ws)
        y = torch.empty(T, H, device=dev)
        h = torch.empty(T, F, dtype=BF16, device=dev)
        logits = torch.empty(T, V, device=dev)
        for _ in range(2):
            N.moe_layer_forward(dims, layer.native_weights(), None, x, T, y, ws)
            routed = y.clone()
            xb = x.view(BF16)
            N.moe_gated_forward(up, xb, T, wg, wu, h, ws)
            N.moe_linear_forward(down, h, T, wd, y, ws, residual=y)
            yb = y.to(BF16)
            N.moe_linear_forward(out, yb, T, head, logits, ws)
            assert N.moe_check_device_error(ws) == 0
            err = O.per_token_rel_err(routed.cpu().numpy(), layer.oracle(x64)["y"])
            assert err.max() <= 2e-3
            R.check("h", h, R.gated_forward(1, xb, wg, wu, None, None)["h"])
            R.check("y", y, R.linear_forward(0, h, wd, None, routed, F32)["y"])
            R.check("logits", logits, R.linear_forward(0, yb, head, None, None, F32)["y"])


def test_binding_refuses_mismatched_tensors(N):
    """Tensors whose shape, type, stride or device does not fit never reach the library, and outputs stay as they are."""
    T, K, M = 4, 64, 32
    x, w = torch.zeros(T, K, dtype=BF16, device="cuda"), torch.zeros(M, K, dtype=BF16, device="cuda")
    y = torch.full((T, M), 7.0, dtype=BF16, device="cuda")
    d = N.dense_dims(K, M, N.MOE_BF16, N.MOE_ACT_SILU)
    ws, _ = workspace(N, d, T, True)
    for bad in (dict(x=x[:3]), dict(x=x.half()), dict(x=x.cpu()), dict(x=torch.zeros(K, T, dtype=BF16, device="cuda").t()),
                dict(w=w[:, :40]), dict(w=w.float()), dict(w=w.cpu()), dict(y=y[:, :31]), dict(y=y.cpu()),
                dict(y=y.half()), dict(ws=ws.cpu()), dict(ws=ws[::2]), dict(ws=ws[:64]), dict(bias=w[0, :31]),
                dict(bias=w[:, 0]), dict(residual=y.float()), dict(pre=y.float()), dict(x=x[:1].expand(T, K))):
        a = dict(x=x, w=w, y=y, ws=ws, bias=None, residual=None, pre=None)
        a.update(bad)
        with pytest.raises(N.MoeError) as e:
            N.moe_linear_forward(d, a["x"], T, a["w"], a["y"], a["ws"], bias=a["bias"], residual=a["residual"], pre=a["pre"])
        assert e.value.code in (N.MOE_EINVAL, N.MOE_EWORKSPACE, N.MOE_EUNSUPPORTED), bad
    for call in (lambda: N.moe_gated_forward(d, x, T, w, w[:16], y, ws),
                 lambda: N.moe_gated_forward(d, x, T, w, w, y, ws, gate=y),
                 lambda: N.moe_linear_backward(d, x, T, w, y, ws, dx=x),
                 lambda: N.moe_linear_backward(d, x, T, w, y, ws, pre=y),
                 lambda: N.moe_gated_backward(d, x, T, w, w, y, y, y[:2], ws, dx=x)):
        with pytest.raises(N.MoeError):
            call()
    torch.cuda.synchronize()
    assert (y == 7.0).all()


def test_more_than_2_31_elements(N):
    """Outputs, inputs and reductions whose element offsets pass 32 bits: sampled rows and columns."""
    T, K, M = 34000, 64, 65536
    gen = gen_for(16)
    x, w = rnd(gen, (T, K), BF16), rnd(gen, (M, K), BF16, K ** -0.5)
    d = N.dense_dims(K, M, N.MOE_BF16, 0)
    ws = torch.empty(N.moe_dense_workspace_bytes(d, T, False), dtype=torch.uint8, device="cuda")
    N.moe_workspace_init(ws)
    y = torch.empty(T, M, dtype=BF16, device="cuda")
    N.moe_linear_forward(d, x, T, w, y, ws)
    rows = torch.tensor([0, 1, 32767, 32768, 33000, 33999], device="cuda")
    R.check("y", y[rows], R.linear_forward(0, x[rows], w, None, None, BF16)["y"])
    # y as the incoming gradient: dx reads rows of it, dW runs down all of it
    ws = torch.empty(N.moe_dense_workspace_bytes(d, T, True), dtype=torch.uint8, device="cuda")
    N.moe_workspace_init(ws)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(M, dtype=BF16, device="cuda")
    N.moe_linear_backward(d, x, T, w, y, ws, dx=dx, dw=dw, dbias=db)
    R.check("dx", dx[rows], R.linear_backward(0, x[rows], w, None, y[rows])["dx"])
    cols = torch.tensor([0, 5, 32768, 65535], device="cuda")
    ref = R.linear_backward(0, x, w[cols], None, y[:, cols].contiguous())
    R.check("dw", dw[cols], ref["dw0"])
    R.check("db", db[cols], ref["db0"])
