"""The dense operators' rules at their edges."""

import math

import pytest
import torch

import dense_reference as R
from test_gpu_dense import ACTS, BF16, F16, F32, Out, gen_for, guard_ok, rnd, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def N():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mixture_experts_route_amd import native

    return native


# (gated, n_in, n_out, forced splits): sums of 16 tokens in as many parts as are asked for would take more than the
# workspace has for them, those of one token would not; the last one chooses its parts itself
@pytest.mark.parametrize("gated,K,M,splits", [(False, 1024, 70000, 8), (True, 1024, 33000, 8), (False, 4096, 200003, 3),
                                              (False, 11264, 131088, 0)])
def test_a_token_has_the_same_bits_where_room_for_parts_is_short(N, gated, K, M, splits):
    gen = gen_for(31, K, M)
    dt = F16 if gated else BF16
    T = N.MOE_DENSE_ROW_TOKENS
    x = rnd(gen, (T, K), dt)
    w = [torch.empty(M, K, dtype=dt, device="cuda").normal_(0, K ** -0.5, generator=gen) for _ in range(1 + gated)]
    d = N.dense_dims(K, M, N.dtype_code(x), N.MOE_ACT_SILU if gated else N.MOE_ACT_NONE)

    def call(xs):
        t = xs.shape[0]
        ws, whole = workspace(N, d, t, False)
        out = [torch.empty(t, M, dtype=dt if gated else F32, device="cuda") for _ in range(3 if gated else 1)]
        if gated:
            N.moe_gated_forward(d, xs, t, *w, out[0], ws, gate=out[1], up=out[2])
        else:
            N.moe_linear_forward(d, xs, t, *w, out[0], ws)
        assert guard_ok(whole)
        return out

    N.moe_debug_force_dense_plan(N.MOE_DENSE_AUTO, splits)
    try:
        full = call(x)
        for rows in ([0], [15], [2, 9, 4], list(range(13))):
            for a, b in zip(call(x[rows].contiguous()), full):
                assert torch.equal(a, b[rows]), rows
    finally:
        N.moe_debug_force_dense_plan()


def limits(N, a):
    """The activation's value and derivative at -infinity and at +infinity."""
    inf = math.inf
    return {N.MOE_ACT_NONE: ((-inf, 1), (inf, 1)), N.MOE_ACT_SIGMOID: ((0, 0), (1, 0))}.get(a, ((0, 0), (inf, 1)))


@pytest.mark.parametrize("dt", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("a", ACTS)
def test_saved_infinities_give_the_limits(N, a, dt):
    """A pre-activation past the operands' type is saved as an infinity: its derivative is the limit there (0 or 1, and
    the activation's value 0, 1 or an infinity), exactly; a gradient or a derivative of zero beside an infinite factor
    gives zero; a NaN stays one."""
    T, M = 5, 8
    z = torch.tensor([-math.inf, math.inf] * 4, device="cuda").to(dt)
    (v0, d0), (v1, d1) = limits(N, a)
    slope = torch.tensor([d0, d1] * 4, device="cuda").double()
    value = torch.tensor([v0, v1] * 4, device="cuda").double()
    eye, ones = torch.eye(M, dtype=dt, device="cuda"), torch.ones(T, M, dtype=dt, device="cuda")
    pre = z.repeat(T, 1)
    d = N.dense_dims(M, M, N.dtype_code(ones), a)
    ws, _ = workspace(N, d, T, True)
    dx, dw, dw2 = torch.empty_like(ones), torch.empty_like(eye), torch.empty_like(eye)
    db, db2 = torch.empty_like(z), torch.empty_like(z)
    # dy = (1, 0, 1, 0, ..) down the tokens: T = 5 has three ones
    dy = ones.clone()
    dy[1::2] = 0
    N.moe_linear_backward(d, ones, T, eye, dy, ws, pre=pre, dx=dx, dw=dw, dbias=db)
    assert torch.equal(dx.double(), dy.double() * slope)
    assert torch.equal(dw.double(), (3 * slope)[:, None].expand(M, M)) and torch.equal(db.double(), 3 * slope)
    N.moe_gated_backward(d, ones, T, eye, eye, pre, ones, dy, ws, dw_gate=dw, dgate_bias=db, dup_bias=db2)
    assert torch.equal(dw.double(), (3 * slope)[:, None].expand(M, M)) and torch.equal(db.double(), 3 * slope)
    assert torch.equal(db2.double(), 3 * value)
    # nothing comes back through either factor where dh is zero
    N.moe_gated_backward(d, ones, T, eye, eye, pre, pre, torch.zeros_like(dy), ws, dx=dx, dw_gate=dw, dw_up=dw2,
                         dgate_bias=db, dup_bias=db2)
    for t in (dx, dw, dw2, db, db2):
        assert (t == 0).all()
    # an infinite up factor: dg is infinite, and zero where the derivative is
    N.moe_gated_backward(d, ones, T, eye, eye, pre, pre, ones, ws, dgate_bias=db)
    assert torch.equal(db.double(), torch.where(slope == 0, 0.0, z.double()))
    # NaN
    bad = torch.full_like(pre, math.nan)
    if a not in (N.MOE_ACT_NONE, N.MOE_ACT_RELU):
        N.moe_linear_backward(d, ones, T, eye, ones, ws, pre=bad, dbias=db)
        assert torch.isnan(db).all()
    N.moe_gated_backward(d, ones, T, eye, eye, bad, ones, ones, ws, dup_bias=db2)
    assert torch.isnan(db2).all()
    N.moe_gated_backward(d, ones, T, eye, eye, ones, bad, ones, ws, dgate_bias=db)
    assert torch.isnan(db).all()


@pytest.mark.parametrize("a", [1, 2, 3, 4], ids=["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("T", [3, 70])
def test_a_finite_forward_has_finite_gradients_past_fp16(N, a, T):
    """z and g of -70000, past fp16: the outputs are finite, and so are the gradients, through the saved -infinity."""
    K, M = 16, 24
    gen = gen_for(33, a, T)
    x, w, w2, dh = rnd(gen, (T, K), F16), rnd(gen, (M, K), F16, 0.25), rnd(gen, (M, K), F16, 0.25), rnd(gen, (T, M), F16)
    x[1], w[:, 0] = 0, 2.0
    x[1, 0] = -35000
    w2[:, 0] = 2.0 ** -8
    d = N.dense_dims(K, M, N.MOE_F16, a)
    ws, _ = workspace(N, d, T, True)
    y = torch.empty(T, M, device="cuda")
    pre, h, g, u = (torch.empty(T, M, dtype=F16, device="cuda") for _ in range(4))
    N.moe_linear_forward(d, x, T, w, y, ws, pre=pre)
    N.moe_gated_forward(d, x, T, w, w2, h, ws, gate=g, up=u)
    assert torch.isfinite(y).all() and torch.isfinite(h).all() and torch.isfinite(u).all()
    assert (pre[1] == -math.inf).all() and (g[1] == -math.inf).all()
    dx, dw, dw2, db, db2 = (torch.empty_like(t) for t in (x, w, w, dh[0], dh[0]))
    low = torch.full_like(pre, -1000.0)  # where every derivative and value here is zero, too
    N.moe_linear_backward(d, x, T, w, dh, ws, pre=pre, dx=dx, dw=dw, dbias=db)
    ref = R.linear_backward(a, x, w, torch.where(torch.isinf(pre), low, pre), dh)
    for name, t, k in (("dx", dx, "dx"), ("dw", dw, "dw0"), ("db", db, "db0")):
        R.check(name, t, ref[k])
    N.moe_gated_backward(d, x, T, w, w2, g, u, dh, ws, dx=dx, dw_gate=dw, dw_up=dw2, dgate_bias=db, dup_bias=db2)
    ref = R.gated_backward(a, x, w, w2, torch.where(torch.isinf(g), low, g), u, dh)
    for name, t, k in (("dx", dx, "dx"), ("dwg", dw, "dw0"), ("dwu", dw2, "dw1"), ("dbg", db, "db0"), ("dbu", db2, "db1")):
        R.check(name, t, ref[k])


@pytest.mark.parametrize("T", [16, 97])
def test_gelu_keeps_its_lower_tail(N, T):
    """Exact gelu and its derivative at z = -9 .. -3, relative to their values.  Bounds in units of E = 2^-24 (fp32's
    half step): the argument z / sqrt 2 is within 2 E, which erfc multiplies by z^2 + 1 at most; erfc itself is within
    16 units in the last place, 32 E; two products, 2 E.  The density's exponent z^2 / 2 is within 3 E of itself; its
    exponential and factors add 6 E."""
    z = (-3 - torch.arange(T, device="cuda", dtype=torch.float64) % 97 / 16).to(BF16)  # exact in bf16
    x, one = z[:, None].contiguous(), torch.ones(8, 1, dtype=BF16, device="cuda")
    d = N.dense_dims(1, 8, N.MOE_BF16, N.MOE_ACT_GELU)
    ws, _ = workspace(N, d, T, True)
    zz = z.double()[:, None].expand(T, 8)
    cdf, pdf = 0.5 * torch.special.erfc(-zz / math.sqrt(2)), torch.exp(-zz * zz / 2) / math.sqrt(2 * math.pi)
    e_cdf, e_pdf = (2 * (zz * zz + 1) + 34) * R.E, (1.5 * zz * zz + 6) * R.E
    value = (zz * cdf, e_cdf * (zz * cdf).abs())
    slope = (cdf + zz * pdf, e_cdf * cdf + e_pdf * (zz * pdf).abs() + R.E * (cdf + zz * pdf).abs())

    def rounded(v, e):  # a result in bf16
        return v, e + R.half_step(BF16) * (v.abs() + e)

    y = torch.empty(T, 8, device="cuda")
    N.moe_linear_forward(d, x, T, one, y, ws)
    R.check("y", y, value)
    h, g, u = (torch.empty(T, 8, dtype=BF16, device="cuda") for _ in range(3))
    N.moe_gated_forward(d, x, T, one, torch.zeros_like(one), h, ws, up_bias=torch.ones(8, dtype=BF16, device="cuda"),
                        gate=g, up=u)
    R.check("h", h, rounded(*value))
    N.moe_gated_forward(d, x, T, one, one, h, ws)  # without saved factors or a bias: h = act(z) z
    R.check("h", h, rounded(value[0] * zz, (value[1] + R.E * value[0].abs()) * zz.abs()))
    # one token's column sums are dz itself: a bias gradient per token
    db, db2 = (torch.empty(T, dtype=BF16, device="cuda") for _ in range(2))
    dt = N.dense_dims(1, T, N.MOE_BF16, N.MOE_ACT_GELU)
    row, ones, wt = z[None, :].contiguous(), torch.ones(1, T, dtype=BF16, device="cuda"), torch.ones(T, 1, dtype=BF16, device="cuda")
    ws, _ = workspace(N, dt, 1, True)
    N.moe_linear_backward(dt, ones[:, :1].contiguous(), 1, wt, ones, ws, pre=row, dbias=db)
    R.check("dz", db, rounded(slope[0][:, 0], slope[1][:, 0]))
    N.moe_gated_backward(dt, ones[:, :1].contiguous(), 1, wt, wt, row, ones, ones, ws, dgate_bias=db, dup_bias=db2)
    R.check("dg", db, rounded(slope[0][:, 0], slope[1][:, 0]))
    R.check("du", db2, rounded(value[0][:, 0], value[1][:, 0]))


@pytest.mark.parametrize("splits", [0, 2, 3, 7])
@pytest.mark.parametrize("kernel", [1, 2, 3], ids=["tile64", "tile128", "tile256"])
def test_weights_of_two_strides_run_the_same_kernels(N, kernel, splits):
    """dx of the gated block with whole 16-byte rows of different strides in Wg and Wu: the tile kernels take them (a kernel
    forced on them runs, unsplit where no parts are asked for), so the bits are those of equal strides; parts that
    begin in either matrix, partial last steps, an odd width."""
    N.moe_debug_force_dense_plan(kernel, splits)
    try:
        for T, K, M, pad_g, pad_u in ((70, 264, 2056, 0, 24), (257, 520, 1000, 56, 8), (40, 261, 4160, 3, 11),
                                      (300, 1000, 72, 0, 8)):
            gen = gen_for(34, T, K, M)
            x, g, u, dh = rnd(gen, (T, K), F16), *(rnd(gen, (T, M), F16) for _ in range(3))
            wg, wu = rnd(gen, (M, K), F16, K ** -0.5, pad=pad_g), rnd(gen, (M, K), F16, K ** -0.5, pad=pad_u)
            same = rnd(gen, (M, K), F16, pad=pad_g)
            same.copy_(wu)
            d = N.dense_dims(K, M, N.MOE_F16, N.MOE_ACT_SILU)
            ws, whole = workspace(N, d, T, True)
            out, want = Out((T, K), F16, 8), Out((T, K), F16, 8)
            N.moe_gated_backward(d, x, T, wg, wu, g, u, dh, ws, dx=out.t)
            N.moe_gated_backward(d, x, T, wg, same, g, u, dh, ws, dx=want.t)
            assert torch.equal(out.t, want.t)
            R.check("dx", out.t, R.gated_backward(N.MOE_ACT_SILU, x, wg, wu, g, u, dh)["dx"])
            assert out.untouched() and guard_ok(whole)
    finally:
        N.moe_debug_force_dense_plan()


def ints(gen, rows, cols, dt, pad=0):
    """Whole numbers -2 .. 2: every product and every sum here is exact in fp32, in any order."""
    t = torch.full((rows, cols + pad), math.nan, dtype=dt, device="cuda")[:, :cols]
    return t.copy_(torch.randint(-2, 3, (rows, cols), generator=gen, device="cuda"))


@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("splits", [0, 3])
@pytest.mark.parametrize("kernel", range(6), ids=["auto", "tile64", "tile128", "tile256", "any64", "any128"])
def test_long_sums_of_whole_numbers_are_exact(N, kernel, splits, pad):
    """Every product at long reductions, where a lost, stale or doubled chunk would hide in the bounds of rounded sums:
    equal to the exact result, and to its rounding where it is stored in 16 bits."""
    N.moe_debug_force_dense_plan(kernel, splits)
    try:
        for dt, short, long in ((BF16, 264, 8256), (F16, 130, 5000)):
            gen = gen_for(35, kernel, splits, pad, short)
            T, K, M = short, long, 392  # sums over K
            x, w, w2 = ints(gen, T, K, dt, pad), ints(gen, M, K, dt, pad), ints(gen, M, K, dt, pad)
            d = N.dense_dims(K, M, N.dtype_code(x), N.MOE_ACT_NONE)
            ws, _ = workspace(N, d, T, False)
            y = Out((T, M), F32)
            h, g, u = (Out((T, M), dt) for _ in range(3))
            N.moe_linear_forward(d, x, T, w, y.t, ws)
            N.moe_gated_forward(d, x, T, w, w2, h.t, ws, gate=g.t, up=u.t)
            zg, zu = x.double() @ w.double().T, x.double() @ w2.double().T
            assert torch.equal(y.t.double(), zg) and torch.equal(g.t, zg.to(dt)) and torch.equal(u.t, zu.to(dt))
            for T, K, M in ((short, 200, long), (long, 200, short)):  # sums over M (dx), over T (dW)
                x, w, w2 = ints(gen, T, K, dt, pad), ints(gen, M, K, dt, pad), ints(gen, M, K, dt, pad)
                g, u, dh = (ints(gen, T, M, dt, pad) for _ in range(3))
                d = N.dense_dims(K, M, N.dtype_code(x), N.MOE_ACT_NONE)
                ws, whole = workspace(N, d, T, True)
                dx, dw, dw2, dx1, dw1 = (Out(s, dt) for s in ((T, K), (M, K), (M, K), (T, K), (M, K)))
                N.moe_gated_backward(d, x, T, w, w2, g, u, dh, ws, dx=dx.t, dw_gate=dw.t, dw_up=dw2.t)
                N.moe_linear_backward(d, x, T, w, dh, ws, dx=dx1.t, dw=dw1.t)
                dg, du = dh.double() * u.double(), dh.double() * g.double()
                for got, want in ((dx, dg @ w.double() + du @ w2.double()), (dw, dg.T @ x.double()), (dw2, du.T @ x.double()),
                                  (dx1, dh.double() @ w.double()), (dw1, dh.double().T @ x.double())):
                    assert torch.equal(got.t, want.to(dt)) and got.untouched()
                assert guard_ok(whole)
    finally:
        N.moe_debug_force_dense_plan()


@pytest.mark.parametrize("kernel,splits,shape", [
    (0, 0, (2200, 4104, 4050)),  # the last tiles in parts
    (0, 0, (333, 1000, 1357)), (1, 0, (300, 4096, 520)), (2, 0, (520, 4096, 520)), (3, 0, (520, 4096, 520)),
    (3, 5, (300, 2056, 2056)), (4, 2, (130, 1001, 264)), (5, 0, (300, 1001, 264))], ids=str)
def test_equal_calls_give_equal_bits_at_any_size(N, kernel, splits, shape):
    """The same four calls three times, outputs and workspace full of something else in between."""
    T, K, M = shape
    gen = gen_for(36, kernel, splits, *shape)
    x, dh = rnd(gen, (T, K), F16), rnd(gen, (T, M), F16)
    w, w2 = (rnd(gen, (M, K), F16, K ** -0.5) for _ in range(2))
    d = N.dense_dims(K, M, N.MOE_F16, N.MOE_ACT_GELU)
    ws, _ = workspace(N, d, T, True)
    nan = lambda *s, dt=F16: torch.full(s, math.nan, dtype=dt, device="cuda")
    N.moe_debug_force_dense_plan(kernel, splits)
    try:
        first = None
        for rep in range(3):
            y, h, g, u, pre = nan(T, M, dt=F32), nan(T, M), nan(T, M), nan(T, M), nan(T, M)
            dx, dw, db, dx2, dwg, dwu = nan(T, K), nan(M, K), nan(M), nan(T, K), nan(M, K), nan(M, K)
            N.moe_linear_forward(d, x, T, w, y, ws, pre=pre)
            N.moe_gated_forward(d, x, T, w, w2, h, ws, gate=g, up=u)
            N.moe_linear_backward(d, x, T, w, dh, ws, pre=pre, dx=dx, dw=dw, dbias=db)
            N.moe_gated_backward(d, x, T, w, w2, g, u, dh, ws, dx=dx2, dw_gate=dwg, dw_up=dwu)
            out = (y, h, g, u, pre, dx, dw, db, dx2, dwg, dwu)
            assert not any(torch.isnan(t).any() for t in out)
            if first is None:
                first = out
            assert all(torch.equal(a, b) for a, b in zip(out, first)), rep
            ws.view(torch.uint8)[4096:].fill_(0xFF)
    finally:
        N.moe_debug_force_dense_plan()


@pytest.mark.parametrize("T", [5, 90])
def test_fp16_dz_past_its_range_is_infinite_and_stays_in_its_row(N, T):
    """dg = dh u act'(g) of finite factors past 65504 becomes an infinity on its way into the products, as stated: its token's
    dx and its output's dWg are not finite, everything else is right; a scaled incoming gradient gives it all."""
    K, M = 40, 72
    gen = gen_for(37, T)
    x, wg, wu = rnd(gen, (T, K), F16), rnd(gen, (M, K), F16, K ** -0.5), rnd(gen, (M, K), F16, K ** -0.5)
    g, u, dh = rnd(gen, (T, M), F16), rnd(gen, (T, M), F16), rnd(gen, (T, M), F16, 0.1)
    g[3, 7], u[3, 7], dh[3, 7] = 4, 250, 300  # dg = 300 250 1.05 = 79000, du = 1178
    d = N.dense_dims(K, M, N.MOE_F16, N.MOE_ACT_SILU)
    ws, _ = workspace(N, d, T, True)
    for scale in (1.0, 2.0 ** -6):
        dy = dh * scale
        dx, dwg, dwu, dbg, dbu = (torch.empty_like(t) for t in (x, wg, wu, g[0], g[0]))
        N.moe_gated_backward(d, x, T, wg, wu, g, u, dy, ws, dx=dx, dw_gate=dwg, dw_up=dwu, dgate_bias=dbg, dup_bias=dbu)
        ref = R.gated_backward(N.MOE_ACT_SILU, x, wg, wu, g, u, dy)
        bad_x, bad_w, bad_b = (torch.zeros_like(t, dtype=torch.bool) for t in (dx, dwg, dbg))
        if scale == 1:
            bad_x[3], bad_w[7], bad_b[7] = True, True, True
        for name, got, bad, k in (("dx", dx, bad_x, "dx"), ("dwg", dwg, bad_w, "dw0"), ("dbg", dbg, bad_b, "db0")):
            assert torch.equal(~torch.isfinite(got), bad), name
            R.check(name, torch.where(bad, ref[k][0].to(F16), got).double().where(~bad, ref[k][0]), ref[k])
        R.check("dwu", dwu, ref["dw1"])
        R.check("dbu", dbu, ref["db1"])
