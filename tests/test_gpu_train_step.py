"""A training step of a routed layer with 16-bit experts under an output head, made of the library's calls as a program makes
them: route, group, dispatch, gated, linear, combine onto the shared expert, loss, and all of it back; one workspace."""

import pytest
import torch

import dense_reference as R
from test_gpu_dense import rnd

pytestmark = pytest.mark.gpu

BF16, F16, F32, F64 = torch.bfloat16, torch.float16, torch.float32, torch.float64


@pytest.fixture(scope="module")
def N():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mixture_experts_route_amd import native

    return native


class Step:
    """The model's weights, the calls' plans, the outputs and the one workspace."""

    def __init__(self, N, T, H, F, E, k, V, seed):
        self.N, self.T, self.k = N, T, k
        g = self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.x, self.router = rnd(g, (T, H), BF16), rnd(g, (E, H), BF16, H ** -0.5)
        self.wg, self.wu = rnd(g, (E * F, H), BF16, H ** -0.5).view(E, F, H), rnd(g, (E * F, H), BF16, H ** -0.5).view(E, F, H)
        self.wd = rnd(g, (E * H, F), BF16, F ** -0.5).view(E, H, F)
        self.sg, self.su, self.sd = rnd(g, (F, H), BF16, H ** -0.5), rnd(g, (F, H), BF16, H ** -0.5), rnd(g, (H, F), BF16, F ** -0.5)
        self.head = rnd(g, (V, H), BF16, H ** -0.5)
        self.targets = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
        self.targets[::7] = -100
        bf = N.MOE_BF16
        self.layer, self.rows = N.dims(H, F, E, k), N.rows_dims(H, k, bf)
        self.up, self.down = N.experts_dims(E, H, F, bf, N.MOE_ACT_SILU), N.experts_dims(E, F, H, bf)
        self.s_up, self.s_down = N.dense_dims(H, F, bf, N.MOE_ACT_SILU), N.dense_dims(F, H, bf)
        self.loss_d = N.loss_dims(H, V, bf)
        P = T * k
        nbytes = max(N.moe_workspace_bytes(self.layer, T), N.moe_rows_workspace_bytes(self.rows, T),
                     N.moe_experts_workspace_bytes(self.up, P, True), N.moe_experts_workspace_bytes(self.down, P, True),
                     N.moe_dense_workspace_bytes(self.s_up, T, True), N.moe_dense_workspace_bytes(self.s_down, T, True),
                     N.moe_loss_workspace_bytes(self.loss_d, T, True))
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        N.moe_workspace_init(self.ws)
        e = lambda *s, dt=BF16: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
        i = lambda *s: e(*s, dt=torch.int32)  # noqa: E731
        self.o = dict(ids=i(T, k), w=e(T, k, dt=F32), counts=i(E), offsets=i(E + 1), perm=i(P), inv=i(T, k), xs=e(P, H),
                      h=e(P, F), g=e(P, F), u=e(P, F), ys=e(P, H), sh=e(T, F), sgate=e(T, F), sup=e(T, F), shared=e(T, H),
                      y=e(T, H), loss=e(T, dt=F32), lse=e(T, dt=F32), dy=e(T, H), dhead=e(V, H), dys=e(P, H),
                      dw=e(T, k, dt=F32), dh=e(P, F), dwd=e(E, H, F), dxs=e(P, H), dwg=e(E, F, H), dwu=e(E, F, H),
                      dsh=e(T, F), dsd=e(H, F), dsx=e(T, H), dsg=e(F, H), dsu=e(F, H), dx=e(T, H))
        self.dloss = (self.targets != -100).float() / (self.targets != -100).sum()

    def run(self):
        N, o, T, ws = self.N, self.o, self.T, self.ws
        N.moe_route(self.layer, self.x, T, self.router, None, o["ids"], o["w"], None, ws)
        N.moe_group_tokens(self.layer, o["ids"], T, o["counts"], o["offsets"], o["perm"], ws)
        N.moe_dispatch_forward(self.rows, self.x, T, o["perm"], o["xs"], o["inv"], ws)
        N.moe_experts_gated_forward(self.up, o["xs"], o["offsets"], self.wg, self.wu, o["h"], ws, gate=o["g"], up=o["u"])
        N.moe_experts_linear_forward(self.down, o["h"], o["offsets"], self.wd, o["ys"], ws)
        N.moe_gated_forward(self.s_up, self.x, T, self.sg, self.su, o["sh"], ws, gate=o["sgate"], up=o["sup"])
        N.moe_linear_forward(self.s_down, o["sh"], T, self.sd, o["shared"], ws)
        N.moe_combine_forward(self.rows, o["ys"], o["inv"], o["w"], T, o["y"], ws, residual=o["shared"])
        N.moe_loss_forward(self.loss_d, o["y"], T, self.head, self.targets, o["loss"], o["lse"], ws)
        N.moe_loss_backward(self.loss_d, o["y"], T, self.head, self.targets, o["loss"], o["lse"], self.dloss, ws,
                            dx=o["dy"], dw=o["dhead"])
        N.moe_combine_backward(self.rows, o["dy"], T, o["perm"], o["inv"], o["w"], ws, ys=o["ys"], dys=o["dys"], dtopk_w=o["dw"])
        N.moe_experts_linear_backward(self.down, o["h"], o["offsets"], self.wd, o["dys"], ws, dx=o["dh"], dw=o["dwd"])
        N.moe_experts_gated_backward(self.up, o["xs"], o["offsets"], self.wg, self.wu, o["g"], o["u"], o["dh"], ws, dx=o["dxs"],
                                     dw_gate=o["dwg"], dw_up=o["dwu"])
        N.moe_linear_backward(self.s_down, o["sh"], T, self.sd, o["dy"], ws, dx=o["dsh"], dw=o["dsd"])
        N.moe_gated_backward(self.s_up, self.x, T, self.sg, self.su, o["sgate"], o["sup"], o["dsh"], ws, dx=o["dsx"],
                             dw_gate=o["dsg"], dw_up=o["dsu"])
        N.moe_dispatch_backward(self.rows, o["dxs"], o["inv"], T, o["dx"], ws, residual=o["dsx"])

    def reference(self):
        """The same model and its gradients by autograd in float64, the routing given."""
        leaf = lambda t: t.double().requires_grad_(True)  # noqa: E731
        p = {n: leaf(getattr(self, n)) for n in ("x", "wg", "wu", "wd", "sg", "su", "sd", "head")}
        p["w"] = leaf(self.o["w"])
        ids = self.o["ids"].long()
        act = torch.nn.functional.silu
        y = (act(p["x"] @ p["sg"].T) * (p["x"] @ p["su"].T)) @ p["sd"].T
        for j in range(self.k):
            wg, wu, wd = (p[n][ids[:, j]] for n in ("wg", "wu", "wd"))  # [T] matrices
            h = act(torch.bmm(wg, p["x"][:, :, None])) * torch.bmm(wu, p["x"][:, :, None])
            y = y + p["w"][:, j:j + 1] * torch.bmm(wd, h)[:, :, 0]
        z = y @ p["head"].T
        live = self.targets != -100
        loss = torch.zeros_like(z[:, 0])
        loss[live] = torch.logsumexp(z[live], 1) - z[live, self.targets[live].long()]
        (loss * self.dloss.double()).sum().backward()
        return loss.detach(), {n: t.grad for n, t in p.items()}


def near(got, want, roundings):
    """Norms within so many bf16 half steps: each intermediate that a value passes through is rounded once, by at most
    2^-9 of itself, and the layer's maps are close to isometries (weights of variance 1 / n_in)."""
    err = (got.double() - want).norm() / want.norm()
    assert err <= roundings * R.half_step(BF16), err


@pytest.mark.parametrize("T,H,F,E,k,V", [(1, 256, 128, 8, 2, 300), (40, 256, 128, 16, 4, 1003), (300, 512, 256, 64, 10, 2000)])
def test_training_step_against_autograd(N, T, H, F, E, k, V):
    s = Step(N, T, H, F, E, k, V, T)
    if T == 1:
        s.targets[0], s.dloss[0] = 5, 1.0
    s.run()
    assert N.moe_check_device_error(s.ws) == 0
    loss, grad = s.reference()
    o = s.o
    # forward h, ys, shared, y; back dy, dys, dh, dg and du, dxs, dx: no value passes more than ten, nor a gradient more than
    # the forward's five beside its own
    near(o["loss"], loss, 8)
    for name, ref in (("dhead", "head"), ("dwd", "wd"), ("dwg", "wg"), ("dwu", "wu"), ("dsd", "sd"), ("dsg", "sg"), ("dsu", "su"),
                      ("dx", "x"), ("dw", "w")):
        near(o[name], grad[ref], 16)


def test_training_step_captured_and_replayed(N):
    """The whole step as one graph, on new inputs and another routing each time, bitwise the eager step."""
    s = Step(N, 120, 256, 128, 32, 6, 500, 77)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for _ in range(4):
        s.x.copy_(rnd(s.gen, tuple(s.x.shape), BF16))
        s.router.copy_(rnd(s.gen, tuple(s.router.shape), BF16, 1 / 16))
        s.run()
        torch.cuda.synchronize()
        eager = {n: t.clone() for n, t in s.o.items()}
        for t in s.o.values():
            t.fill_(1)
        graph.replay()
        torch.cuda.synchronize()
        for n, t in s.o.items():
            assert torch.equal(t, eager[n]), n
        assert N.moe_check_device_error(s.ws) == 0


def test_two_streams_with_a_workspace_each(N):
    """Two steps at once on two streams, each with its own workspace: the bits of each alone."""
    a, b = Step(N, 200, 256, 128, 16, 4, 700, 5), Step(N, 150, 512, 256, 16, 2, 400, 6)
    for s in (a, b):
        s.run()
    torch.cuda.synchronize()
    want = [{n: t.clone() for n, t in s.o.items()} for s in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for s, st in zip((a, b), streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                s.run()
        torch.cuda.synchronize()
        for s, w in zip((a, b), want):
            for n, t in s.o.items():
                assert torch.equal(t, w[n]), n
