"""Argument checks of the loss over an output head (host only, no GPU), and its reference against differences."""

import ctypes

import pytest
import torch

import loss_reference as L

P = 1 << 20  # addresses that are never used: every call here is refused on the host


@pytest.fixture(scope="module")
def N():
    from mixture_experts_route_amd import native

    return native


def forward(N, d, **kw):
    a = dict(x=P, ldx=64, T=4, w=P, ldw=64, t=P, loss=P, lse=P, ws=P, wb=1 << 40)
    a.update(kw)
    return N.raw("moe_loss_forward")(ctypes.byref(d) if d is not None else None, a["x"], a["ldx"], a["T"], a["w"], a["ldw"],
                                     a["t"], a["loss"], a["lse"], a["ws"], a["wb"], None)


def backward(N, d, **kw):
    a = dict(x=P, ldx=64, T=4, w=P, ldw=64, t=P, loss=P, lse=P, g=P, dx=P, lddx=64, dw=P, lddw=64, ws=P, wb=1 << 40)
    a.update(kw)
    return N.raw("moe_loss_backward")(ctypes.byref(d) if d is not None else None, a["x"], a["ldx"], a["T"], a["w"],
                                      a["ldw"], a["t"], a["loss"], a["lse"], a["g"], a["dx"], a["lddx"], a["dw"],
                                      a["lddw"], a["ws"], a["wb"], None)


CALLS = [forward, backward]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("dims,code", [
    ((0, 32, 1), -1), ((64, 0, 1), -1), ((64, -5, 1), -1), (((1 << 20) + 8, 32, 1), -2), ((64, (1 << 20) + 1, 1), -2),
    ((64, 32, 0), -2), ((64, 32, 3), -2),
])
def test_dims_refused(N, call, dims, code):
    d = N.loss_dims(*dims)
    assert call(N, d) == code
    assert N.moe_loss_workspace_bytes(d, 4, True) == 0
    assert call(N, None) == N.MOE_EINVAL


@pytest.mark.parametrize("call", CALLS)
def test_tokens_and_workspace_refused(N, call):
    d = N.loss_dims(64, 32, N.MOE_BF16)
    for t, code in ((0, -1), (-1, -1), ((1 << 20) + 1, -2)):
        assert call(N, d, T=t) == code
        assert N.moe_loss_workspace_bytes(d, t) == 0
    need = N.moe_loss_workspace_bytes(d, 4, call is backward)
    for kw in (dict(ws=None), dict(ws=P + 64), dict(wb=need - 1)):
        assert call(N, d, **kw) == N.MOE_EWORKSPACE


@pytest.mark.parametrize("call", CALLS)
def test_arguments_refused(N, call):
    d = N.loss_dims(64, 32, N.MOE_F16)
    for p in ("x", "w"):
        for kw in ({p: None}, {p: P + 1}, {"ld" + p: 63}, {"ld" + p: -64}):
            assert call(N, d, **kw) == N.MOE_EINVAL
        assert call(N, d, **{"ld" + p: (1 << 22) + 1}) == N.MOE_EUNSUPPORTED
    for p in ("t", "loss", "lse") + (("g",) if call is backward else ()):
        assert call(N, d, **{p: None}) == N.MOE_EINVAL
        assert call(N, d, **{p: P + 2}) == N.MOE_EINVAL
    if call is backward:
        for kw in (dict(dx=None, dw=None), dict(dx=P + 1), dict(lddx=63), dict(dw=P + 1), dict(lddw=63)):
            assert call(N, d, **kw) == N.MOE_EINVAL


def test_workspace_does_not_hold_the_logits(N):
    d = N.loss_dims(2048, 131072, N.MOE_BF16)
    sizes = [N.moe_loss_workspace_bytes(d, t, True) for t in (1, 16, 300, 4096)]
    assert sizes == sorted(sizes)
    for t in (65536, 1 << 20):  # beside x, dx and the forward's parts, dz of one piece: not the whole
        assert N.moe_loss_workspace_bytes(d, t, True) < t * 131072 * 2 // 8
    assert N.moe_loss_workspace_bytes(d, 65536) < 65536 * 2048 * 2 + (256 << 20)


@pytest.mark.parametrize("K,V", [(2048, 100003), (2048, 32768), (1024, 50304), (33, 3077), (64, 300), (1, 1 << 20)])
@pytest.mark.parametrize("backward", [False, True])
def test_workspace_serves_every_smaller_count(N, K, V, backward):
    """The size for max_tokens is enough for each count up to it: it never falls as tokens are added."""
    d = N.loss_dims(K, V, N.MOE_BF16)
    most = 0
    for t in [*range(1, 16385), *range(16385, (1 << 20) - 300, 997), *range((1 << 20) - 300, (1 << 20) + 1)]:
        n = N.moe_loss_workspace_bytes(d, t, backward)
        assert n >= most, t
        most = n


def test_binding_refuses_mismatched_tensors(N):
    d = N.loss_dims(64, 32, N.MOE_BF16)
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(32, 64, dtype=torch.bfloat16)
    t, f, ws = torch.zeros(4, dtype=torch.int32), torch.zeros(4), torch.zeros(1024, dtype=torch.int32)
    for call in (lambda: N.moe_loss_forward(d, x, 4, w, t, f, f, ws), lambda: N.moe_loss_forward(d, x, 4, w, t.long(), f, f, ws),
                 lambda: N.moe_loss_forward(d, x, 4, w[:31], t, f, f, ws), lambda: N.moe_loss_forward(d, x, 3, w, t, f, f, ws),
                 lambda: N.moe_loss_backward(d, x, 4, w, t, f, f, f[:3], ws, dx=x),
                 lambda: N.moe_loss_backward(d, x, 4, w, t, f, f, f, ws, dx=x.float())):
        with pytest.raises(N.MoeError) as e:
            call()
        assert e.value.code == N.MOE_EINVAL


def test_reference_gradients_match_differences():
    g = torch.Generator().manual_seed(3)
    T, K, V = 5, 6, 9
    x, w = torch.randn(T, K, generator=g, dtype=torch.float64), torch.randn(V, K, generator=g, dtype=torch.float64)
    targets, dloss = torch.tensor([0, 8, -100, 3, 3], dtype=torch.int32), torch.randn(T, generator=g, dtype=torch.float64)
    fwd = L.forward(x, w, targets, -100)
    bwd = L.backward(x, w, targets, -100, fwd["loss"][0], fwd["lse"][0], dloss, torch.bfloat16)
    eps = 1e-5
    for i, gr in enumerate((bwd["dx"][0], bwd["dw"][0])):
        v = torch.randn((x, w)[i].shape, generator=g, dtype=torch.float64)
        hi, lo = ((L.forward(x + s * v, w, targets, -100) if i == 0 else L.forward(x, w + s * v, targets, -100))["loss"][0]
                  for s in (eps, -eps))
        num = ((hi - lo) * dloss).sum() / (2 * eps)
        # truncation eps^2 f''' / 6 (f''' of order 1e2 here), rounding 2^-52 |f| / eps
        assert abs(num - (gr * v).sum()) <= 1e-7 * (1 + gr.abs().sum())
