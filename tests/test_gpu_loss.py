"""The loss over an output head on the GPU against float64, elementwise within the bounds of loss_reference."""

import math

import pytest
import torch

import dense_reference as R
import loss_reference as L
from test_gpu_dense import Out, guard_ok, rnd

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
IGNORE = -100


@pytest.fixture(scope="module")
def N():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mixture_experts_route_amd import native

    return native


def gen_for(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def workspace(N, d, T, backward):
    n = N.moe_loss_workspace_bytes(d, T, backward)
    whole = torch.full((n + 1024,), 0xA5, dtype=torch.uint8, device="cuda")
    N.moe_workspace_init(whole[:n])
    return whole[:n], whole


def inputs(gen, T, K, V, dt, skip=0.1, pad=0, offset=0, sure=True):
    x, w = rnd(gen, (T, K), dt, pad=pad, offset=offset), rnd(gen, (V, K), dt, K ** -0.5, pad, offset)
    targets = torch.randint(0, V, (T,), generator=gen, device="cuda", dtype=torch.int32)
    if sure:  # some tokens are nearly certain of their target
        lean = 8.0 * torch.rand(T, 1, generator=gen, device="cuda")
        x.copy_((x.float() + lean * w[targets.long()].float()).to(dt))
    targets[torch.rand(T, generator=gen, device="cuda") < skip] = IGNORE
    return x, w, targets


def floats(T, n=1):
    return [torch.full((T,), float("nan"), device="cuda") for _ in range(n)]


def check_all(N, seed, T, K, V, dt, skip=0.1, pad=0, offset=0, sure=True):
    gen = gen_for(seed)
    x, w, targets = inputs(gen, T, K, V, dt, skip, pad, offset, sure)
    d = N.loss_dims(K, V, N.dtype_code(x), IGNORE)
    ws, whole = workspace(N, d, T, False)
    loss, lse = floats(T, 2)
    N.moe_loss_forward(d, x, T, w, targets, loss, lse, ws)
    ref = L.forward(x, w, targets, IGNORE)
    R.check("loss", loss, ref["loss"])
    R.check("lse", lse, ref["lse"])
    assert N.moe_check_device_error(ws) == 0 and guard_ok(whole)
    ws, whole = workspace(N, d, T, True)
    dloss = torch.randn(T, generator=gen, device="cuda") / T
    dx, dw = Out((T, K), dt, pad, offset), Out((V, K), dt, pad, offset)
    N.moe_loss_backward(d, x, T, w, targets, loss, lse, dloss, ws, dx=dx.t, dw=dw.t)
    ref = L.backward(x, w, targets, IGNORE, loss, lse, dloss, dt)
    R.check("dx", dx.t, ref["dx"])
    R.check("dw", dw.t, ref["dw"])
    assert dx.untouched() and dw.untouched()
    one, two = Out((T, K), dt, pad, offset), Out((V, K), dt, pad, offset)
    N.moe_loss_backward(d, x, T, w, targets, loss, lse, dloss, ws, dx=one.t)
    N.moe_loss_backward(d, x, T, w, targets, loss, lse, dloss, ws, dw=two.t)
    assert torch.equal(one.t, dx.t) and torch.equal(two.t, dw.t)
    assert N.moe_check_device_error(ws) == 0 and guard_ok(whole)


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("T,K,V", [(1, 8, 1), (1, 64, 2), (2, 8, 7), (5, 64, 64), (3, 128, 65), (16, 64, 129), (17, 200, 1000),
                                   (64, 72, 257), (65, 64, 4099), (300, 136, 513), (129, 512, 2000), (1000, 64, 100)])
def test_against_float64(N, T, K, V, dt):
    check_all(N, T + V, T, K, V, dt)


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("T,K,V", [(1, 1, 1), (3, 7, 5), (33, 65, 130), (130, 61, 1003), (257, 131, 64)])
def test_odd_widths(N, T, K, V, dt):
    check_all(N, T * K, T, K, V, dt)


@pytest.mark.parametrize("dt", [BF16, F16])
def test_odd_widths_of_large_heads(N, dt):
    check_all(N, 25, 5, 129, 140000, dt)  # few tokens: the weights are read as they lie
    check_all(N, 26, 200, 129, 140000, dt)


@pytest.mark.parametrize("pad,offset", [(1, 0), (0, 3), (8, 8), (8, 0), (7, 1)])
def test_strides_and_alignments(N, pad, offset):
    check_all(N, 30 + pad, 70, 64, 300, BF16, pad=pad, offset=offset)
    check_all(N, 31 + pad, 70, 61, 301, F16, pad=pad, offset=offset)


@pytest.mark.parametrize("kernel", range(1, 6))
@pytest.mark.parametrize("splits", [0, 3])
def test_every_kernel(N, kernel, splits):
    N.moe_debug_force_dense_plan(kernel, splits)
    try:
        check_all(N, kernel, 300, 192, 777, BF16)
        check_all(N, kernel + 9, 5, 64, 600, F16)
    finally:
        N.moe_debug_force_dense_plan()


def test_all_and_no_tokens_left_out(N):
    check_all(N, 40, 20, 64, 100, BF16, skip=0.0)
    check_all(N, 41, 20, 64, 100, F16, skip=1.1)


def test_many_tokens_in_several_launches(N):
    check_all(N, 42, 8192 + 5, 64, 200, BF16)


def test_most_tokens(N):
    check_all(N, 50, 1 << 20, 16, 70, BF16)


@pytest.mark.parametrize("dt", [BF16, F16])
def test_vocabulary_in_several_pieces(N, dt):
    check_all(N, 43, 40000, 40, 4000, dt)  # pieces of 2048 and 1952 columns
    check_all(N, 44, 40001, 33, 3077, dt)


def test_fewer_tokens_on_the_workspace_of_more(N):
    """A workspace sized for one count serves those below it, whose pieces of the vocabulary are larger."""
    K, V, many, few = 40, 32768, 4229, 4228
    gen = gen_for(51)
    x, w, targets = inputs(gen, many, K, V, BF16)
    d = N.loss_dims(K, V, N.MOE_BF16, IGNORE)
    got = []
    for size in (few, many):
        ws, whole = workspace(N, d, size, True)
        loss, lse = floats(few, 2)
        N.moe_loss_forward(d, x[:few], few, w, targets[:few], loss, lse, ws)
        dx, dw = torch.empty_like(x[:few]), torch.empty_like(w)
        N.moe_loss_backward(d, x[:few], few, w, targets[:few], loss, lse, torch.ones(few, device="cuda"), ws, dx=dx, dw=dw)
        assert N.moe_check_device_error(ws) == 0 and guard_ok(whole)
        got.append((loss, lse, dx, dw))
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_small_losses_keep_their_digits(N):
    """Targets ahead by up to 40: losses down to 2^-58, each within a relative bound."""
    T, V = 41, 300
    x = torch.zeros(T, 8, dtype=BF16, device="cuda")
    w = torch.zeros(V, 8, dtype=BF16, device="cuda")
    x[:, 0] = torch.arange(T, device="cuda").to(BF16)
    w[7, 0] = 1.0
    targets = torch.full((T,), 7, dtype=torch.int32, device="cuda")
    d = N.loss_dims(8, V, N.MOE_BF16)
    ws, _ = workspace(N, d, T, True)
    loss, lse = floats(T, 2)
    N.moe_loss_forward(d, x, T, w, targets, loss, lse, ws)
    want = torch.log1p((V - 1) * torch.exp(-torch.arange(T, device="cuda", dtype=torch.float64)))
    # the logits are exact; (40 + 4 + 64) roundings of 2 e in the sum, 8 e after it
    assert ((loss.double() - want).abs() <= want * 232 * R.E).all() and loss[40] > 0
    dx = torch.empty_like(x)
    N.moe_loss_backward(d, x, T, w, targets, loss, lse, torch.ones(T, device="cuda"), ws, dx=dx)
    want = torch.expm1(-want)
    assert ((dx[:, 0].double() - want).abs() <= want.abs() * (2 * R.half_step(BF16) + 300 * R.E)).all()


def spread_bounds(x, w, targets, loss, lse, dloss):
    """dx and dW of fp16 with the bounds of loss_reference.backward, but each token's dz rounded relative to its own dloss: brought
    to 2^13 .. 2^15, so that an error of half of fp16's smallest number is 2^-25 / 2^13 of dloss; and x times the token's share s of
    the largest dloss (a power of two: within a factor of two of it) rounded to 2^-25 where the largest |x| is at 2^14 or above, which
    is 2^-39 of it; undone by a share of at least half of dloss's."""
    dz, e = L.dz_of(x, w, targets, IGNORE, loss, lse, dloss)
    live = (targets != IGNORE)[:, None]
    x, w, g = x.double(), w.double(), dloss.double().abs()[:, None]
    r = e + R.half_step(F16) * (dz.abs() + e) + torch.where(live, g * 2.0 ** -38, 0.0)
    dx, dw = dz @ w, dz.T @ x
    e_dx = r @ w.abs() + 2 * w.shape[0] * R.E * ((dz.abs() + r) @ w.abs())
    share = torch.where(live, 2 * g / g[live].max(), 0.0).clamp(max=1.0)
    ex = 2.0 ** -39 * x[live[:, 0]].abs().max() * 4 / share.clamp(min=2.0 ** -60)
    e_dw = r.T @ x.abs() + (dz.abs() + r).T @ torch.where(live, ex, 0.0) + 2 * len(x) * R.E * ((dz.abs() + r).T @ x.abs())
    return {"dx": (dx, R._round(dx, e_dx, F16)), "dw": (dw, R._round(dw, e_dw, F16))}


def check_past_range(name, got, ref):
    """R.check, but fp16's largest number is 65504 and its half step there 16: what is 65520 or more is infinite."""
    val, bound = ref
    inf = torch.isinf(got) & (val.abs() + bound >= 65520) & (torch.sign(got) == torch.sign(val))
    assert inf[val.abs() - bound >= 65520].all()
    R.check(name, torch.where(inf, 0.0, got), (torch.where(inf, 0.0, val), bound))


@pytest.mark.parametrize("T,K,V,pad", [(24, 64, 50000, 0), (24, 61, 20011, 0), (240, 40, 30000, 3), (700, 33, 5001, 0), (9, 2048, 400, 0),
                                       (20000, 1, 40, 0), (400, 300, 900, 5)])
def test_fp16_tokens_of_very_different_weight(N, T, K, V, pad):
    """dloss over twenty-three powers of two: every token's dx keeps its softmax part, relative to its own dloss.  The weights have a
    mean, so that this part is as large as the target's; dloss is large enough for the results to be normal numbers."""
    gen = gen_for(52 + T)
    x = rnd(gen, (T, K), F16, pad=pad)
    w = ((torch.randn(V, K, generator=gen, device="cuda") * 0.3 + 1.0) * K ** -0.5).to(F16)
    targets = torch.randint(0, V, (T,), generator=gen, device="cuda", dtype=torch.int32)
    targets[3::17] = IGNORE
    dloss = (1.0 + torch.rand(T, generator=gen, device="cuda")) * 2.0 ** (14.0 - torch.arange(T, device="cuda") % 24)
    dloss[::2] *= -1
    dloss[3::17] = 1e30
    d = N.loss_dims(K, V, N.MOE_F16, IGNORE)
    ws, whole = workspace(N, d, T, True)
    loss, lse = floats(T, 2)
    N.moe_loss_forward(d, x, T, w, targets, loss, lse, ws)
    dx, dw = Out((T, K), F16, pad), Out((V, K), F16, pad)
    N.moe_loss_backward(d, x, T, w, targets, loss, lse, dloss, ws, dx=dx.t, dw=dw.t)
    ref = spread_bounds(x, w, targets, loss, lse, dloss)
    check_past_range("dx", dx.t, ref["dx"])
    check_past_range("dw", dw.t, ref["dw"])
    one, two = torch.empty_like(dx.t), torch.empty_like(dw.t)
    N.moe_loss_backward(d, x, T, w, targets, loss, lse, dloss, ws, dx=one)
    N.moe_loss_backward(d, x, T, w, targets, loss, lse, dloss, ws, dw=two)
    assert torch.equal(one, dx.t) and torch.equal(two, dw.t) and guard_ok(whole) and N.moe_check_device_error(ws) == 0


def test_targets_out_of_range_are_reported(N):
    T, K, V = 40, 64, 300
    gen = gen_for(45)
    x, w, targets = inputs(gen, T, K, V, BF16, skip=0.0)
    d = N.loss_dims(K, V, N.MOE_BF16, IGNORE)
    ws, _ = workspace(N, d, T, True)
    good = targets.clone()
    for at, bad in ((3, -1), (17, V), (39, 2 ** 31 - 1), (0, -2 ** 31)):
        targets = good.clone()
        targets[at] = bad
        loss, lse = floats(T, 2)
        N.moe_loss_forward(d, x, T, w, targets, loss, lse, ws)
        assert N.moe_check_device_error(ws) == N.DERR_TARGET
        assert torch.isnan(loss[at]) and torch.isnan(lse[at]) and torch.isnan(loss).sum() == 1
        dx, dw = Out((T, K), BF16), Out((V, K), BF16)
        dloss = torch.ones(T, device="cuda")
        N.moe_loss_backward(d, x, T, w, targets, loss, lse, dloss, ws, dx=dx.t, dw=dw.t)
        assert N.moe_check_device_error(ws) == N.DERR_TARGET
        assert (dx.t[at] == 0).all() and dx.untouched() and dw.untouched()
        targets[at], loss[at], lse[at] = IGNORE, 0.0, 0.0
        R.check("dw", dw.t, L.backward(x, w, targets, IGNORE, loss, lse, dloss, BF16)["dw"])


def test_ignore_may_be_any_value(N):
    T, K, V = 30, 64, 50
    gen = gen_for(46)
    x, w, targets = inputs(gen, T, K, V, BF16, skip=0.0)
    targets[4] = -1
    d = N.loss_dims(K, V, N.MOE_BF16, -1)
    ws, _ = workspace(N, d, T, False)
    loss, lse = floats(T, 2)
    N.moe_loss_forward(d, x, T, w, targets, loss, lse, ws)
    assert N.moe_check_device_error(ws) == 0 and loss[4] == 0 and lse[4] == 0
    targets[4], targets[:3] = 3, 7
    d = N.loss_dims(K, V, N.MOE_F16, 7)  # inside the vocabulary: a padding token's id
    ws, _ = workspace(N, d, T, True)
    x, w = x.half(), w.half()
    N.moe_loss_forward(d, x, T, w, targets, loss, lse, ws)
    assert (loss[:3] == 0).all()
    ref = L.forward(x, w, targets, 7)
    R.check("loss", loss, ref["loss"])
    dloss = torch.ones(T, device="cuda")
    dloss[0] = 1e30  # a token that is left out does not count for the scaling either
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    N.moe_loss_backward(d, x, T, w, targets, loss, lse, dloss, ws, dx=dx, dw=dw)
    ref = L.backward(x, w, targets, 7, loss, lse, dloss, F16)
    R.check("dx", dx, ref["dx"])
    R.check("dw", dw, ref["dw"])
    assert N.moe_check_device_error(ws) == 0


def test_infinities_and_nan(N):
    """Limits where logits are infinite; a NaN stays in its token."""
    V, K = 100, 64
    w = torch.zeros(V, K, dtype=BF16, device="cuda")
    w[:, 0], w[5, 1], w[9, 2] = 1.0, float("inf"), float("-inf")
    x = torch.zeros(6, K, dtype=BF16, device="cuda")
    x[0, 0], x[:, 1:3], x[5, 0] = 1.0, 1.0, float("nan")
    targets = torch.tensor([5, 9, 0, 5, IGNORE, 0], dtype=torch.int32, device="cuda")
    d = N.loss_dims(K, V, N.MOE_BF16, IGNORE)
    ws, _ = workspace(N, d, 6, True)
    loss, lse = floats(6, 2)
    N.moe_loss_forward(d, x, 6, w, targets, loss, lse, ws)
    assert loss[0] == 0 and lse[0] == math.inf and loss[3] == 0  # the target's logit alone is infinite
    assert loss[1] == math.inf and loss[2] == math.inf           # another's is
    assert loss[4] == 0 and lse[4] == 0 and torch.isnan(loss[5]) and torch.isnan(lse[5])
    assert N.moe_check_device_error(ws) == 0


def test_equal_calls_give_equal_bits_captured_too(N):
    gen = gen_for(47)
    T, K, V = 200, 128, 1003
    x, w, targets = inputs(gen, T, K, V, F16)
    d = N.loss_dims(K, V, N.MOE_F16, IGNORE)
    ws, _ = workspace(N, d, T, True)
    dloss = torch.full((T,), 1.0 / T, device="cuda")

    def outs():
        return floats(T, 2) + [torch.empty_like(x), torch.empty_like(w)]

    def step(o):
        N.moe_loss_forward(d, x, T, w, targets, o[0], o[1], ws)
        N.moe_loss_backward(d, x, T, w, targets, o[0], o[1], dloss, ws, dx=o[2], dw=o[3])

    cap = outs()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(cap)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cap)
    for rep in range(4):
        nx, _, nt = inputs(gen, T, K, V, F16)
        x.copy_(nx)
        targets.copy_(nt)
        dloss.mul_(3.0)
        eager = outs()
        for v in (*cap, *eager):
            v.fill_(float("nan"))
        step(eager)
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(eager, cap)):
            assert torch.equal(a, b), (rep, i)


def test_large_vocabulary_and_2_31_elements(N):
    """A head of 2^31 elements: a few tokens, sampled columns of dW."""
    T, K, V = 3, 2048, (1 << 20)
    gen = gen_for(48)
    w = torch.empty(V, K, dtype=BF16, device="cuda")
    for i in range(0, V, 1 << 17):
        w[i:i + (1 << 17)] = (torch.randn(1 << 17, K, generator=gen, device="cuda") / 45).to(BF16)
    x = rnd(gen, (T, K), BF16)
    targets = torch.tensor([V - 1, 0, 700000], dtype=torch.int32, device="cuda")
    d = N.loss_dims(K, V, N.MOE_BF16, IGNORE)
    ws, whole = workspace(N, d, T, True)
    loss, lse = floats(T, 2)
    N.moe_loss_forward(d, x, T, w, targets, loss, lse, ws)
    z = torch.cat([x.double() @ w[i:i + (1 << 16)].double().T for i in range(0, V, 1 << 16)], 1)
    want = torch.logsumexp(z, 1)
    bound = 1e-4  # ez = 2 K e sum|terms| < 2 * 2048 * 2^-24 * 0.1, the sum's (24 + 64 + 2048) 2 e; both below
    assert (lse.double() - want).abs().max() < bound and (loss.double() - (want - z.gather(1, targets.long()[:, None])[:, 0])).abs().max() < bound
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    dloss = torch.tensor([1.0, -2.0, 0.5], device="cuda")
    N.moe_loss_backward(d, x, T, w, targets, loss, lse, dloss, ws, dx=dx, dw=dw)
    p = torch.exp(z - lse.double()[:, None])
    p[torch.arange(T), targets.long()] = torch.expm1(-loss.double())
    dz = p * dloss.double()[:, None]
    cols = torch.tensor([0, 1, 65535, 699999, 700000, V - 2, V - 1], device="cuda")
    val = dz[:, cols].T @ x.double()
    mag = dz[:, cols].abs().T @ x.double().abs()
    R.check("dw", dw[cols], (val, R._round(val, mag * (R.half_step(BF16) + bound), BF16)))
    val, mag = torch.zeros(T, K, dtype=torch.float64, device="cuda"), torch.zeros(T, K, dtype=torch.float64, device="cuda")
    for i in range(0, V, 1 << 16):
        val += dz[:, i:i + (1 << 16)] @ w[i:i + (1 << 16)].double()
        mag += dz[:, i:i + (1 << 16)].abs() @ w[i:i + (1 << 16)].double().abs()
    # 2^20 terms in fp32: each wave's chain has at most 2^20 additions, 2 e of what is summed so far, which the bound takes
    # as the sum of magnitudes
    R.check("dx", dx, (val, R._round(val, mag * (R.half_step(BF16) + bound + 2 * V * R.E), BF16)))
    assert guard_ok(whole) and N.moe_check_device_error(ws) == 0


def test_infinities_and_nan_in_the_backward_pass(N):
    """Logits past fp32 from finite operands: the gradients are the limits; a NaN reaches its token's dx and the dW of the columns
    that it has a gradient for, which are all; a token that is left out reaches nothing."""
    V, K, T, g = 100, 64, 6, 0.5
    far = 2.0 ** 65  # its square is infinite in fp32
    w = torch.zeros(V, K, dtype=BF16, device="cuda")
    w[:, 0], w[5, 1], w[9, 2] = 1.0, far, -far
    x = torch.zeros(T, K, dtype=BF16, device="cuda")
    x[:, 0] = 1.0
    x[0, 1], x[1, 1], x[2, 2], x[3, 2], x[4, 1] = far, far, far, far, far
    targets = torch.tensor([5, 7, 7, 9, IGNORE, 0], dtype=torch.int32, device="cuda")
    d = N.loss_dims(K, V, N.MOE_BF16, IGNORE)
    ws, _ = workspace(N, d, T, True)

    def run(x, targets):
        loss, lse = floats(T, 2)
        N.moe_loss_forward(d, x, T, w, targets, loss, lse, ws)
        dx, dw = torch.full_like(x, 7.0), torch.full_like(w, 7.0)
        N.moe_loss_backward(d, x, T, w, targets, loss, lse, torch.full((T,), g, device="cuda"), ws, dx=dx, dw=dw)
        assert N.moe_check_device_error(ws) == 0
        return loss, lse, dx, dw

    # without the token whose gradient is not a number: probabilities that are 0, 1 or one of 99 (98) equal logits
    targets[1] = IGNORE
    loss, lse, dx, dw = run(x, targets)
    assert loss[0] == 0 and lse[0] == math.inf and loss[3] == math.inf and (loss[[1, 4]] == 0).all()
    p = torch.zeros(T, V, dtype=torch.float64, device="cuda")
    p[2], p[3], p[5] = 1 / 99, 1 / 99, 1 / 100  # tokens 2 and 3: z_9 is -infinity
    p[2, 9] = p[3, 9] = 0
    p[2, 7] -= 1
    p[3, 9] -= 1
    p[5, 0] -= 1
    dz = g * p
    # the sum of 99 or 100 exponentials, exp, expm1, a few products: 300 e; dz to bf16; then sums of 100 (6) terms
    r = (R.half_step(BF16) + 300 * R.E) * dz.abs()
    for name, got, a, b in (("dx", dx, dz, w), ("dw", dw, dz.T, x)):
        val, mag = a @ b.double(), a.abs() @ b.double().abs()
        err = (r if name == "dx" else r.T) @ b.double().abs() + 2 * a.shape[1] * R.E * mag
        R.check(name, got, (val, R._round(val, err, BF16)))
    # with it: its dx, and its column of dW, are NaN; its target's column has -g x of it, the others nothing
    targets[1] = 7
    loss, lse, dx1, dw1 = run(x, targets)
    assert loss[1] == math.inf and torch.isnan(dx1[1, 1]) and torch.isnan(dx1[1, 0])
    keep = torch.arange(T, device="cuda") != 1
    assert torch.equal(dx1[keep], dx[keep])
    same = torch.ones(V, dtype=torch.bool, device="cuda")
    same[5] = same[7] = False
    assert torch.equal(dw1[same], dw[same]) and torch.isnan(dw1[5, 0]) and dw1[7, 1] == -g * far
    # a NaN in x
    targets[1], x[5, 3] = IGNORE, math.nan
    loss, lse, dx2, dw2 = run(x, targets)
    assert torch.isnan(loss[5]) and torch.isnan(lse[5]) and torch.isnan(dx2[5]).all()
    assert torch.equal(dx2[:5], dx[:5]) and torch.isnan(dw2[:, 3]).all()


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("T,K,V", [(70, 64, 131072), (9, 40, 300000), (1, 61, 100003)])
def test_the_softmax_part_of_dx_over_a_large_vocabulary(N, T, K, V, dt):
    """Weights with a mean: sum_v p_v w_v is then as large as the target's row, and far beyond the bound, 2 V e (1.6 % of both at
    131072 columns, 3.6 % at 300000) and the roundings of dz; without it no element would be within."""
    gen = gen_for(60 + T)
    x = rnd(gen, (T, K), dt)
    w = ((torch.randn(V, K, generator=gen, device="cuda") * 0.1 + 1.0) * K ** -0.5).to(dt)
    targets = torch.randint(0, V, (T,), generator=gen, device="cuda", dtype=torch.int32)
    d = N.loss_dims(K, V, N.dtype_code(x), IGNORE)
    ws, _ = workspace(N, d, T, True)
    loss, lse = floats(T, 2)
    N.moe_loss_forward(d, x, T, w, targets, loss, lse, ws)
    dx, dloss = torch.empty_like(x), torch.ones(T, device="cuda")
    N.moe_loss_backward(d, x, T, w, targets, loss, lse, dloss, ws, dx=dx)
    val, bound = L.backward(x, w, targets, IGNORE, loss, lse, dloss, dt)["dx"]
    R.check("dx", dx, (val, bound))
    own = torch.expm1(-loss.double())[:, None] * w.double()[targets.long()]
    assert ((own - val).abs() > 4 * bound).all()


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("K", [1 << 20, (1 << 20) - 1])
def test_longest_rows(N, K, dt):
    """2^20 inputs, whole multiples of 2^-7: the logits are exact in fp32 (at most 2^20 terms of one unit), so loss_reference's bounds hold
    with none of their part for the logits."""
    T, V = 5, 70
    gen = gen_for(70)
    x = torch.randint(-1, 2, (T, K), generator=gen, device="cuda").to(dt)
    w = (torch.randint(-1, 2, (V, K), generator=gen, device="cuda") * 2.0 ** -7).to(dt)
    targets = torch.tensor([3, 69, 0, IGNORE, 12], dtype=torch.int32, device="cuda")
    d = N.loss_dims(K, V, N.dtype_code(x), IGNORE)
    ws, whole = workspace(N, d, T, True)
    loss, lse = floats(T, 2)
    N.moe_loss_forward(d, x, T, w, targets, loss, lse, ws)
    z = x.double() @ w.double().T
    live = targets != IGNORE
    at = targets.clamp(min=0).long()[:, None]
    want = torch.where(live, torch.logsumexp(z, 1), 0.0)
    span = z.abs().max()
    # the sum of 70 exponentials of arguments up to 2 span, then a few roundings of lse and of the logits' distance
    bound = 2 * R.E * (2 * span + 4 + 70) + 16 * R.E * span
    assert ((lse.double() - want).abs() <= bound).all()
    assert ((loss.double() - torch.where(live, want - z.gather(1, at)[:, 0], 0.0)).abs() <= bound).all()
    dloss = torch.tensor([1.0, -2.0, 0.5, 1.0, 0.25], device="cuda")
    dx, dw = Out((T, K), dt), Out((V, K), dt)
    N.moe_loss_backward(d, x, T, w, targets, loss, lse, dloss, ws, dx=dx.t, dw=dw.t)
    p = torch.exp(z - lse.double()[:, None]).scatter(1, at, torch.expm1(-loss.double())[:, None])
    dz = torch.where(live[:, None], p * dloss.double()[:, None], 0.0)
    tiny = R.tiny_step(dt) * 2 / (2.0 ** 11 if dt == F16 else 1.0)
    r = dz.abs() * (R.half_step(dt) + 2 * R.E * (4 * span + 20)) + tiny
    for name, got, a, ra, b in (("dx", dx, dz, r, w), ("dw", dw, dz.T, r.T, x)):
        val = a @ b.double()
        err = ra @ b.double().abs() + 2 * a.shape[1] * R.E * ((a.abs() + ra) @ b.double().abs())
        R.check(name, got.t, (val, R._round(val, err, dt)))
        assert got.untouched()
    assert guard_ok(whole) and N.moe_check_device_error(ws) == 0
