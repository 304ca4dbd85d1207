"""The dense operators' rules at their edges."""

import pytest
import torch

from test_gpu_dense import BF16, F16, F32, gen_for, guard_ok, rnd, workspace

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
