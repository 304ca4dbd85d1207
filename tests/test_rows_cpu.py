"""Argument checks of the rows-by-expert calls (host only, no GPU)."""

import ctypes

import pytest
import torch

P = 1 << 20  # addresses that are never used: every call here is refused on the host


@pytest.fixture(scope="module")
def N():
    from mixture_experts_route_amd import native

    return native


def dispatch_fwd(N, d, **kw):
    a = dict(x=P, ldx=64, T=4, perm=P, rows=8, xs=P, ldxs=64, inv=P, ws=P, wb=1 << 20)
    a.update(kw)
    return N.raw("moe_dispatch_forward")(ctypes.byref(d) if d is not None else None, a["x"], a["ldx"], a["T"], a["perm"],
                                         a["rows"], a["xs"], a["ldxs"], a["inv"], a["ws"], a["wb"], None)


def dispatch_bwd(N, d, **kw):
    a = dict(xs=P, ldxs=64, rows=8, inv=P, T=4, res=None, ldr=0, x=P, ldx=64, yd=1, ws=P, wb=1 << 20)
    a.update(kw)
    return N.raw("moe_dispatch_backward")(ctypes.byref(d) if d is not None else None, a["xs"], a["ldxs"], a["rows"],
                                          a["inv"], a["T"], a["res"], a["ldr"], a["x"], a["ldx"], a["yd"], a["ws"],
                                          a["wb"], None)


def combine_fwd(N, d, **kw):
    a = dict(xs=P, ldxs=64, rows=8, inv=P, w=P, T=4, res=None, ldr=0, x=P, ldx=64, yd=1, ws=P, wb=1 << 20)
    a.update(kw)
    return N.raw("moe_combine_forward")(ctypes.byref(d) if d is not None else None, a["xs"], a["ldxs"], a["rows"],
                                        a["inv"], a["w"], a["T"], a["res"], a["ldr"], a["x"], a["ldx"], a["yd"], a["ws"],
                                        a["wb"], None)


def combine_bwd(N, d, **kw):
    a = dict(x=P, ldx=64, yd=1, T=4, perm=P, inv=P, rows=8, w=P, ys=P, ldys=64, xs=P, ldxs=64, dw=P, ws=P, wb=1 << 20)
    a.update(kw)
    return N.raw("moe_combine_backward")(ctypes.byref(d) if d is not None else None, a["x"], a["ldx"], a["yd"], a["T"],
                                         a["perm"], a["inv"], a["rows"], a["w"], a["ys"], a["ldys"], a["xs"], a["ldxs"],
                                         a["dw"], a["ws"], a["wb"], None)


CALLS = [dispatch_fwd, dispatch_bwd, combine_fwd, combine_bwd]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("dims,code", [
    ((0, 2, 1), -1), ((-64, 2, 1), -1), ((64, 0, 1), -1), ((64, -1, 1), -1),
    (((1 << 20) + 8, 2, 1), -2), ((64, 17, 1), -2), ((64, 2, 0), -2), ((64, 2, 3), -2),
])
def test_dims_refused(N, call, dims, code):
    d = N.rows_dims(*dims)
    assert call(N, d) == code
    assert N.moe_rows_workspace_bytes(d, 4) == 0
    assert call(N, None) == N.MOE_EINVAL


@pytest.mark.parametrize("call", CALLS)
def test_counts_and_workspace_refused(N, call):
    d = N.rows_dims(64, 2, N.MOE_BF16)
    for t, code in ((0, -1), (-1, -1), ((1 << 24) + 1, -2)):
        assert call(N, d, T=t) == code
        assert N.moe_rows_workspace_bytes(d, t) == 0
    for n, code in ((0, -1), (-1, -1), ((1 << 28) + 1, -2)):
        assert call(N, d, rows=n) == code
    need = N.moe_rows_workspace_bytes(d, 4)
    for kw in (dict(ws=None), dict(ws=P + 128), dict(wb=need - 1)):
        assert call(N, d, **kw) == N.MOE_EWORKSPACE


@pytest.mark.parametrize("call,mats,arrays", [
    (dispatch_fwd, ("x", "xs"), ("perm", "inv")), (dispatch_bwd, ("xs", "x"), ("inv",)),
    (combine_fwd, ("xs", "x"), ("inv", "w")), (combine_bwd, ("x", "ys"), ("perm", "inv", "w")),
])
def test_required_arguments_refused(N, call, mats, arrays):
    d = N.rows_dims(64, 2, N.MOE_BF16)
    for p in mats:
        for kw in ({p: None}, {p: P + 1}, {"ld" + p: 63}, {"ld" + p: -64}):
            assert call(N, d, **kw) == N.MOE_EINVAL
        assert call(N, d, **{"ld" + p: (1 << 22) + 1}) == N.MOE_EUNSUPPORTED
    for p in arrays:
        assert call(N, d, **{p: None}) == N.MOE_EINVAL
        assert call(N, d, **{p: P + 2}) == N.MOE_EINVAL


def test_optional_arguments_refused(N):
    d = N.rows_dims(64, 2, N.MOE_BF16)
    for call in (dispatch_bwd, combine_fwd):
        assert call(N, d, yd=N.MOE_F16) == N.MOE_EUNSUPPORTED  # the rows' type or fp32
        assert call(N, d, yd=9) == N.MOE_EUNSUPPORTED
        assert call(N, d, yd=N.MOE_F32, x=P + 2) == N.MOE_EINVAL
        assert call(N, d, res=P, ldr=63) == N.MOE_EINVAL
        assert call(N, d, res=P + 1, ldr=64) == N.MOE_EINVAL
    assert combine_bwd(N, d, yd=N.MOE_F16) == N.MOE_EUNSUPPORTED
    assert combine_bwd(N, d, xs=None, dw=None) == N.MOE_EINVAL  # nothing to compute
    assert combine_bwd(N, d, ldxs=63) == N.MOE_EINVAL
    assert combine_bwd(N, d, dw=P + 2) == N.MOE_EINVAL


def test_binding_refuses_mismatched_tensors(N):
    """Host tensors, wrong shapes and types never reach the library."""
    d = N.rows_dims(64, 2, N.MOE_BF16)
    x, xs = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.bfloat16)
    perm, inv, w = torch.arange(8, dtype=torch.int32), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    ws = torch.zeros(1024, dtype=torch.int32)
    for call in (lambda: N.moe_dispatch_forward(d, x, 4, perm, xs, inv, ws),
                 lambda: N.moe_dispatch_forward(d, x, 4, perm.long(), xs, inv, ws),
                 lambda: N.moe_dispatch_forward(d, x, 4, perm[:7], xs, inv, ws),
                 lambda: N.moe_dispatch_backward(d, xs[:, 0], inv, 4, x, ws),
                 lambda: N.moe_combine_forward(d, xs, inv, w.double(), 4, x, ws),
                 lambda: N.moe_combine_backward(d, x, 4, perm, inv, w, ws, dys=xs[:7])):
        with pytest.raises(N.MoeError) as e:
            call()
        assert e.value.code == N.MOE_EINVAL


@pytest.mark.parametrize("shape", [(), (2, 4), (2, 4, 64), (0,)])
def test_binding_refuses_other_numbers_of_dimensions(N, shape):
    """The arguments that say themselves how many rows there are, a scalar among them."""
    d = N.rows_dims(64, 2, N.MOE_BF16)
    x, xs = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.bfloat16)
    perm, inv, w = torch.arange(8, dtype=torch.int32), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    ws = torch.zeros(1024, dtype=torch.int32)
    rows, pairs = torch.zeros(shape, dtype=torch.bfloat16), torch.zeros(shape, dtype=torch.int32)
    for call in (lambda: N.moe_dispatch_forward(d, x, 4, perm, rows, inv, ws),
                 lambda: N.moe_dispatch_forward(d, x, 4, pairs, xs, inv, ws),
                 lambda: N.moe_dispatch_backward(d, rows, inv, 4, x, ws),
                 lambda: N.moe_combine_forward(d, rows, inv, w, 4, x, ws),
                 lambda: N.moe_combine_backward(d, x, 4, pairs, inv, w, ws, dys=xs)):
        with pytest.raises(N.MoeError) as e:
            call()
        assert e.value.code == N.MOE_EINVAL
