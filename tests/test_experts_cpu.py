"""Argument checks of the experts' products (host only, no GPU)."""

import ctypes

import pytest
import torch

P = 1 << 20  # addresses that are never used: every call here is refused on the host


@pytest.fixture(scope="module")
def N():
    from mixture_experts_route_amd import native

    return native


BASE = dict(xs=P, ldxs=64, rows=8, off=P, w=P, w2=P, ldw=64, sw=64 * 32, ys=P, ldys=32, g=P, u=P, ldg=32, dx=P, lddx=64, dw=P,
            dw2=P, lddw=64, sdw=64 * 32, ws=P, wb=1 << 40)


def call(N, name, d, **kw):
    a = {**BASE, **kw}
    x, w, dw = [a[k] for k in ("xs", "ldxs", "rows", "off")], [a["ldw"], a["sw"]], [a["lddw"], a["sdw"]]
    y, end = [a["ys"], a["ldys"]], [a["ws"], a["wb"], None]
    args = {"linear_forward": [*x, a["w"], *w, *y], "linear_backward": [*x, a["w"], *w, *y, a["dx"], a["lddx"], a["dw"], *dw],
            "gated_forward": [*x, a["w"], a["w2"], *w, *y, a["g"], a["u"], a["ldg"]],
            "gated_backward": [*x, a["w"], a["w2"], *w, a["g"], a["u"], a["ldg"], *y, a["dx"], a["lddx"], a["dw"], a["dw2"],
                               *dw]}[name]
    return N.raw("moe_experts_" + name)(ctypes.byref(d) if d is not None else None, *args, *end)


NAMES = ["linear_forward", "linear_backward", "gated_forward", "gated_backward"]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("dims,code", [
    ((0, 64, 32, 1), -1), ((4, 0, 32, 1), -1), ((4, 64, 0, 1), -1), ((-1, 64, 32, 1), -1), ((1025, 64, 32, 1), -2),
    ((4, (1 << 20) + 8, 32, 1), -2), ((4, 64, (1 << 20) + 8, 1), -2), ((4, 64, 32, 0), -2), ((4, 64, 32, 3), -2),
    ((4, 64, 32, 1, 6), -2), ((4, 64, 32, 1, -1), -2),
])
def test_dims_refused(N, name, dims, code):
    d = N.experts_dims(*dims)
    assert call(N, name, d) == code
    assert N.moe_experts_workspace_bytes(d, 8, True) == 0
    assert call(N, name, None) == N.MOE_EINVAL


@pytest.mark.parametrize("name", NAMES)
def test_rows_and_workspace_refused(N, name):
    d = N.experts_dims(4, 64, 32, N.MOE_BF16)
    for n, code in ((0, -1), (-3, -1), ((1 << 28) + 1, -2)):
        assert call(N, name, d, rows=n) == code
        assert N.moe_experts_workspace_bytes(d, n) == 0
    need = N.moe_experts_workspace_bytes(d, 8, name.endswith("backward"))
    for kw in (dict(ws=None), dict(ws=P + 64), dict(wb=need - 1)):
        assert call(N, name, d, **kw) == N.MOE_EWORKSPACE


def test_linear_has_no_activation(N):
    d = N.experts_dims(4, 64, 32, N.MOE_BF16, N.MOE_ACT_SILU)
    assert call(N, "linear_forward", d) == N.MOE_EUNSUPPORTED
    assert call(N, "linear_backward", d) == N.MOE_EUNSUPPORTED


@pytest.mark.parametrize("name,mats,weights", [
    ("linear_forward", [("xs", 64), ("ys", 32)], ["w"]), ("linear_backward", [("xs", 64), ("ys", 32), ("dx", 64)], ["w"]),
    ("gated_forward", [("xs", 64), ("ys", 32)], ["w", "w2"]),
    ("gated_backward", [("xs", 64), ("ys", 32), ("dx", 64)], ["w", "w2"]),
])
def test_required_arguments_refused(N, name, mats, weights):
    d = N.experts_dims(4, 64, 32, N.MOE_BF16)
    for p, n in mats:
        for kw in ([{p: None}] if p != "dx" else []) + [{p: P + 1}, {"ld" + p: n - 1}, {"ld" + p: -n}]:
            assert call(N, name, d, **kw) == N.MOE_EINVAL
        assert call(N, name, d, **{"ld" + p: (1 << 22) + 1}) == N.MOE_EUNSUPPORTED
    for p in weights:
        assert call(N, name, d, **{p: None}) == N.MOE_EINVAL
        assert call(N, name, d, **{p: P + 1}) == N.MOE_EINVAL
    assert call(N, name, d, ldw=63) == N.MOE_EINVAL
    assert call(N, name, d, sw=64 * 32 - 1) == N.MOE_EINVAL
    assert call(N, name, d, sw=-64 * 32) == N.MOE_EINVAL
    assert call(N, name, d, sw=1 << 45) == N.MOE_EUNSUPPORTED
    assert call(N, name, d, off=None) == N.MOE_EINVAL
    assert call(N, name, d, off=P + 2) == N.MOE_EINVAL


def test_optional_arguments_refused(N):
    d = N.experts_dims(4, 64, 32, N.MOE_F16)
    assert call(N, "gated_forward", d, g=None) == N.MOE_EINVAL  # both or neither
    assert call(N, "gated_forward", d, u=None) == N.MOE_EINVAL
    assert call(N, "gated_forward", d, ldg=31) == N.MOE_EINVAL
    for kw in (dict(g=None), dict(u=None), dict(ldg=31), dict(dx=None, dw=None, dw2=None)):
        assert call(N, "gated_backward", d, **kw) == N.MOE_EINVAL
    assert call(N, "linear_backward", d, dx=None, dw=None) == N.MOE_EINVAL
    for name in ("linear_backward", "gated_backward"):
        for kw in (dict(dw=P + 1), dict(lddw=63), dict(sdw=64 * 32 - 1)):
            assert call(N, name, d, **kw) == N.MOE_EINVAL


def test_workspace_grows_with_rows(N):
    d = N.experts_dims(8, 2048, 1000, N.MOE_F16, N.MOE_ACT_GELU)
    sizes = [N.moe_experts_workspace_bytes(d, n, True) for n in (1, 16, 300, 4096, 100000)]
    assert sizes == sorted(sizes) and N.moe_experts_workspace_bytes(d, 4096) >= 4096


def test_binding_refuses_mismatched_tensors(N):
    """Host tensors, wrong shapes, strides and types never reach the library."""
    bf = torch.bfloat16
    d = N.experts_dims(4, 64, 32, N.MOE_BF16)
    xs, w, ys = torch.zeros(8, 64, dtype=bf), torch.zeros(4, 32, 64, dtype=bf), torch.zeros(8, 32, dtype=bf)
    off, ws = torch.zeros(5, dtype=torch.int32), torch.zeros(1024, dtype=torch.int32)
    f, g = N.moe_experts_linear_forward, N.moe_experts_gated_forward
    for bad in (lambda: f(d, xs, off, w, ys, ws), lambda: f(d, xs, off[:4], w, ys, ws), lambda: f(d, xs, off.long(), w, ys, ws),
                lambda: f(d, xs, off, w[:3], ys, ws), lambda: f(d, xs, off, w.transpose(1, 2), ys, ws),
                lambda: f(d, xs, off, w, ys[:7], ws), lambda: f(d, xs[:, :32], off, w, ys, ws),
                lambda: g(d, xs, off, w, torch.zeros(4, 40, 64, dtype=bf)[:, :32], ys, ws),
                lambda: g(d, xs, off, w, w, ys, ws, gate=ys, up=torch.zeros(8, 40, dtype=bf)[:, :32])):
        with pytest.raises(N.MoeError) as e:
            bad()
        assert e.value.code == N.MOE_EINVAL
