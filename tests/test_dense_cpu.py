"""The dense operators' argument checks (host only, no GPU) and their reference formulas (float64)."""

import ctypes

import pytest
import torch

import dense_reference as R

P = 1 << 20  # addresses that are never used: every call here is refused on the host


@pytest.fixture(scope="module")
def N():
    from mixture_experts_route_amd import native

    return native


def lin_fwd(N, d, **kw):
    a = dict(x=P, ldx=64, T=4, w=P, ldw=64, bias=None, res=None, ldr=0, y=P, ldy=32, yd=1, pre=None, ldp=0, ws=P,
             wb=1 << 40)
    a.update(kw)
    return N.raw("moe_linear_forward")(ctypes.byref(d) if d is not None else None, a["x"], a["ldx"], a["T"], a["w"],
                                       a["ldw"], a["bias"], a["res"], a["ldr"], a["y"], a["ldy"], a["yd"], a["pre"],
                                       a["ldp"], a["ws"], a["wb"], None)


def lin_bwd(N, d, **kw):
    a = dict(x=P, ldx=64, T=4, w=P, ldw=64, pre=P, ldp=32, dy=P, ldy=32, dx=P, lddx=64, dw=P, lddw=64, db=P, ws=P,
             wb=1 << 40)
    a.update(kw)
    return N.raw("moe_linear_backward")(ctypes.byref(d), a["x"], a["ldx"], a["T"], a["w"], a["ldw"], a["pre"], a["ldp"],
                                        a["dy"], a["ldy"], a["dx"], a["lddx"], a["dw"], a["lddw"], a["db"], a["ws"],
                                        a["wb"], None)


def gated_fwd(N, d, **kw):
    a = dict(x=P, ldx=64, T=4, wg=P, ldg=64, wu=P, ldu=64, bg=None, bu=None, h=P, ldh=32, g=None, ldpg=0, u=None, ldpu=0,
             ws=P, wb=1 << 40)
    a.update(kw)
    return N.raw("moe_gated_forward")(ctypes.byref(d), a["x"], a["ldx"], a["T"], a["wg"], a["ldg"], a["wu"], a["ldu"],
                                      a["bg"], a["bu"], a["h"], a["ldh"], a["g"], a["ldpg"], a["u"], a["ldpu"], a["ws"],
                                      a["wb"], None)


def gated_bwd(N, d, **kw):
    a = dict(x=P, ldx=64, T=4, wg=P, ldg=64, wu=P, ldu=64, g=P, ldpg=32, u=P, ldpu=32, dh=P, lddh=32, dx=P, lddx=64,
             dwg=P, lddg=64, dwu=P, lddu=64, dbg=None, dbu=None, ws=P, wb=1 << 40)
    a.update(kw)
    return N.raw("moe_gated_backward")(ctypes.byref(d), a["x"], a["ldx"], a["T"], a["wg"], a["ldg"], a["wu"], a["ldu"],
                                       a["g"], a["ldpg"], a["u"], a["ldpu"], a["dh"], a["lddh"], a["dx"], a["lddx"],
                                       a["dwg"], a["lddg"], a["dwu"], a["lddu"], a["dbg"], a["dbu"], a["ws"], a["wb"],
                                       None)


CALLS = [lin_fwd, lin_bwd, gated_fwd, gated_bwd]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("dims,code", [
    ((0, 32, 1, 1), -1), ((64, 0, 1, 1), -1), ((-8, 32, 1, 1), -1),
    (((1 << 20) + 8, 32, 1, 1), -2), ((64, (1 << 20) + 8, 1, 1), -2),
    ((64, 32, 0, 1), -2),                # fp32 operands
    ((64, 32, 3, 1), -2), ((64, 32, 1, 6), -2), ((64, 32, 1, -1), -2),
])
def test_dims_refused(N, call, dims, code):
    d = N.dense_dims(*dims)
    assert call(N, d) == code
    assert N.moe_dense_workspace_bytes(d, 4, True) == 0


@pytest.mark.parametrize("call", CALLS)
def test_tokens_and_workspace_refused(N, call):
    d = N.dense_dims(64, 32, N.MOE_BF16, N.MOE_ACT_SILU)
    assert call(N, d, T=0) == N.MOE_EINVAL
    assert call(N, d, T=-1) == N.MOE_EINVAL
    assert call(N, d, T=(1 << 24) + 1) == N.MOE_EUNSUPPORTED
    assert call(N, d, ws=None) == N.MOE_EWORKSPACE
    assert call(N, d, ws=P + 8) == N.MOE_EWORKSPACE
    need = N.moe_dense_workspace_bytes(d, 4, call in (lin_bwd, gated_bwd))
    assert call(N, d, wb=need - 1) == N.MOE_EWORKSPACE
    assert N.moe_dense_workspace_bytes(d, 0) == 0
    assert N.moe_dense_workspace_bytes(d, (1 << 24) + 1) == 0


def test_workspace_grows_with_tokens(N):
    d = N.dense_dims(2048, 1000, N.MOE_F16, N.MOE_ACT_GELU)
    for backward in (False, True):
        sizes = [N.moe_dense_workspace_bytes(d, t, backward) for t in (1, 16, 17, 64, 300, 4096, 100000)]
        assert sizes == sorted(sizes) and sizes[0] >= 4096


@pytest.mark.parametrize("call,mats", [
    (lin_fwd, [("x", "ldx", 64, 2), ("w", "ldw", 64, 2), ("y", "ldy", 32, 2)]),
    (lin_bwd, [("x", "ldx", 64, 2), ("w", "ldw", 64, 2), ("pre", "ldp", 32, 2), ("dy", "ldy", 32, 2)]),
    (gated_fwd, [("x", "ldx", 64, 2), ("wg", "ldg", 64, 2), ("wu", "ldu", 64, 2), ("h", "ldh", 32, 2)]),
    (gated_bwd, [("x", "ldx", 64, 2), ("wg", "ldg", 64, 2), ("wu", "ldu", 64, 2), ("g", "ldpg", 32, 2),
                 ("u", "ldpu", 32, 2), ("dh", "lddh", 32, 2)]),
])
def test_required_matrices_refused(N, call, mats):
    d = N.dense_dims(64, 32, N.MOE_F16, N.MOE_ACT_RELU)
    kw = dict(yd=N.MOE_F16) if call is lin_fwd else {}
    for p, ld, length, elem in mats:
        assert call(N, d, **{**kw, p: None}) == N.MOE_EINVAL
        assert call(N, d, **{**kw, p: P + 1}) == N.MOE_EINVAL
        assert call(N, d, **{**kw, ld: length - 1}) == N.MOE_EINVAL
        assert call(N, d, **{**kw, ld: -length}) == N.MOE_EINVAL
        assert call(N, d, **{**kw, ld: (1 << 22) + 1}) == N.MOE_EUNSUPPORTED


def test_optional_arguments_refused(N):
    d = N.dense_dims(64, 32, N.MOE_BF16, N.MOE_ACT_SILU)
    assert lin_fwd(N, d, yd=N.MOE_F16) == N.MOE_EUNSUPPORTED   # y is of the operands' type or fp32
    assert lin_fwd(N, d, yd=7) == N.MOE_EUNSUPPORTED
    assert lin_fwd(N, d, yd=N.MOE_F32, y=P + 2) == N.MOE_EINVAL  # fp32 rows on fp32 addresses
    assert lin_fwd(N, d, res=P, ldr=31) == N.MOE_EINVAL
    assert lin_fwd(N, d, pre=P, ldp=31) == N.MOE_EINVAL
    assert lin_fwd(N, d, bias=P + 1) == N.MOE_EINVAL
    assert gated_fwd(N, d, g=P, ldpg=32) == N.MOE_EINVAL       # both pre-activations or neither
    assert gated_fwd(N, d, u=P, ldpu=32) == N.MOE_EINVAL
    assert gated_fwd(N, d, bu=P + 1) == N.MOE_EINVAL
    assert lin_bwd(N, d, dx=None, dw=None, db=None) == N.MOE_EINVAL  # nothing to compute
    assert gated_bwd(N, d, dx=None, dwg=None, dwu=None) == N.MOE_EINVAL
    assert lin_bwd(N, d, lddx=63) == N.MOE_EINVAL
    assert lin_bwd(N, d, lddw=63) == N.MOE_EINVAL
    assert gated_bwd(N, d, lddu=63) == N.MOE_EINVAL
    assert gated_bwd(N, d, dbg=P + 1) == N.MOE_EINVAL


def test_forced_plan_refused(N):
    f = N.raw("moe_debug_force_dense_plan")
    for kernel, splits in ((-1, 0), (6, 0), (0, -1), (0, 9)):
        assert f(kernel, splits) == N.MOE_EINVAL


def test_layer_calls_refuse_fp16(N):
    """MOE_F16 is a dense operand type only: the layer's calls keep refusing it."""
    d = N.dims(2048, 768, 512, 10, 1)
    f = N.raw("moe_route")
    assert f(ctypes.byref(d), P, N.MOE_F16, 1, P, 1, None, P, P, None, P, 1 << 30, None) == N.MOE_EUNSUPPORTED


def test_binding_refuses_mismatched_tensors(N):
    """Host tensors, wrong shapes, types and strides never reach the library."""
    d = N.dense_dims(64, 32, N.MOE_BF16)
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(32, 64, dtype=torch.bfloat16)
    y = torch.zeros(4, 32, dtype=torch.bfloat16)
    ws = torch.zeros(1024, dtype=torch.int32)
    with pytest.raises(N.MoeError) as e:
        N.moe_linear_forward(d, x, 4, w, y, ws)
    assert e.value.code == N.MOE_EINVAL


@pytest.mark.parametrize("a", range(6))
def test_reference_gradients_match_differences(a):
    """The reference's backward formulas against central differences of its forward ones."""
    g = torch.Generator().manual_seed(a)
    T, K, M = 5, 7, 6
    x, wg, wu, dy = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((T, K), (M, K), (M, K), (T, M)))

    def f_lin(x, wg):
        return (R.act(a, x @ wg.T) * dy).sum()

    def f_gated(x, wg, wu):
        return (R.act(a, x @ wg.T) * (x @ wu.T) * dy).sum()

    lin = R.linear_backward(a, x, wg, x @ wg.T, dy)
    gat = R.gated_backward(a, x, wg, wu, x @ wg.T, x @ wu.T, dy)
    eps = 1e-5
    for f, args, grads in ((f_lin, (x, wg), (lin["dx"][0], lin["dw0"][0])),
                           (f_gated, (x, wg, wu), (gat["dx"][0], gat["dw0"][0], gat["dw1"][0]))):
        for i, gr in enumerate(grads):
            v = torch.randn(args[i].shape, generator=g, dtype=torch.float64)
            hi = [t + eps * v if j == i else t for j, t in enumerate(args)]
            lo = [t - eps * v if j == i else t for j, t in enumerate(args)]
            num = (f(*hi) - f(*lo)) / (2 * eps)
            # the truncation error is eps^2 f''' / 6 (f''' of order 1e2 here), the rounding error 2^-52 |f| / eps
            assert abs(num - (gr * v).sum()) <= 1e-7 * (1 + gr.abs().sum())


def test_reference_bound_notices_a_planted_error():
    """The bounds are tight enough to see one misplaced element of a product."""
    g = torch.Generator().manual_seed(9)
    x = torch.randn(9, 40, generator=g).bfloat16()
    w = (torch.randn(11, 40, generator=g) / 40 ** 0.5).bfloat16()
    ref = R.linear_forward(R.SILU, x, w, None, None, torch.bfloat16)["y"]
    good = ref[0].bfloat16()
    R.check("y", good, ref)
    x2 = x.clone()
    x2[:, 39] = 0  # the last element of the reduction lost
    with pytest.raises(AssertionError):
        R.check("y", R.linear_forward(R.SILU, x2, w, None, None, torch.bfloat16)["y"][0].bfloat16(), ref)
