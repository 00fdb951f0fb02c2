"""Rotary positions with several axes on the GPU against the 64-bit formula.

Bound of every element: the bf16 rounding 2^-8 |y|, and (|x_a| + |x_b|) times the error of the
fp32 cosine and sine: the angle from the nearest quarter turn is rounded to fp32 twice (2 * 2^-24
of at most pi/4: 9.4e-8), the series left out come to 3e-8, its roundings to 3 * 2^-24 (1.8e-7), the
products to 2 * 2^-24 (1.2e-7): 4.3e-7, and 6e-7 is allowed."""
import numpy as np
import pytest
import torch

from tests import cache_ref as ref

pytestmark = pytest.mark.gpu

ANGLE = 6e-7


def make(rng, B, H, N, d, layout):
    x = torch.from_numpy(rng.standard_normal((B, N, 3, H, d)).astype(np.float32)).to(torch.bfloat16).cuda()
    if layout == "qkv":
        return [x[:, :, i].transpose(1, 2) for i in range(2)]
    if layout == "bnhd":
        return [x[:, :, i].contiguous().transpose(1, 2) for i in range(2)]
    return [x[:, :, i].transpose(1, 2).contiguous() for i in range(2)]


def check(got, x, pos, rope, inverse=False, angle=ANGLE):
    x = x.double().cpu().numpy()
    p = pos.cpu().numpy()
    for b in range(x.shape[0]):
        pb = p if p.ndim == 2 else p[b]
        y = ref.turn(x[b], pb, rope.inv_freq, rope.pair_axis, rope.pairing, -1.0 if inverse else 1.0)
        tol = 2.0 ** -8 * np.abs(y) + angle * ref.partner_size(x[b], len(rope.inv_freq), rope.pairing)
        err = np.abs(got[b].double().cpu().numpy() - y)
        assert (err <= tol).all(), (np.argwhere(err > tol)[:3], err.max())


@pytest.mark.parametrize("pairing", ["interleaved", "half"])
@pytest.mark.parametrize("layout", ["bhnd", "bnhd", "qkv"])
@pytest.mark.parametrize("B,H,N,d,dims", [
    (1, 2, 512, 64, (24, 20, 20)), (2, 5, 77, 128, (44, 42, 42)), (3, 1, 1, 128, (128,)), (1, 7, 33, 64, (32, 32)),
    (1, 3, 65, 128, (16, 16, 16, 16)), (1, 2, 31, 64, (16,)), (2, 9, 130, 128, (0, 48, 16)),
])
def test_rope(B, H, N, d, dims, layout, pairing):
    import top_routed_block_b200 as fv
    rng = np.random.default_rng(B * 1000 + N)
    rope = fv.rope_axes(dims, pairing=pairing)
    pos = torch.from_numpy(rng.integers(-200, 40000, (N, len(dims)) if B != 2 else (B, N, len(dims))).astype(np.int32)).cuda()
    Q, K = make(rng, B, H, N, d, layout)
    q, k = fv.fvattn_rope(Q, K, pos, rope)
    assert q.is_contiguous() and k.is_contiguous()
    check(q, Q, pos, rope)
    check(k, K, pos, rope)
    rest = 2 * len(rope.inv_freq)
    assert torch.equal(q[..., rest:], Q[..., rest:])
    gq, gk = fv.fvattn_rope_bwd(Q, K, pos, rope)
    check(gq, Q, pos, rope, inverse=True)
    check(gk, K, pos, rope, inverse=True)
    one, none = fv.fvattn_rope(Q, None, pos, rope)
    assert none is None and torch.equal(one, q)


def test_rope_far_positions():
    """Angles of positions up to 2^31: the step is rounded to 2^-64 revolutions, 2^31 of which are 1e-9;
    the extended precision of the reference is good to 2^31 2^-64 as well: far inside the 1e-6 allowed."""
    import top_routed_block_b200 as fv
    rng = np.random.default_rng(9)
    rope = fv.rope_axes((64,))
    pos = torch.tensor([[2 ** 31 - 1], [-(2 ** 31)], [2 ** 30 + 12345], [1 << 20], [0], [-1]], dtype=torch.int32).cuda()
    Q, K = make(rng, 1, 2, 6, 64, "bhnd")
    q, _ = fv.fvattn_rope(Q, K, pos, rope)
    check(q, Q, pos, rope, angle=ANGLE + 1e-6)


@pytest.mark.parametrize("pairing", ["interleaved", "half"])
def test_rope_in_place_into_views_and_uneven_heads(pairing):
    import top_routed_block_b200 as fv
    rng = np.random.default_rng(11)
    rope = fv.rope_axes((44, 42, 42), pairing=pairing)
    pos = fv.grid_positions(3, 5, 7)
    Q, _ = make(rng, 2, 8, 105, 128, "bnhd")
    _, K = make(rng, 2, 3, 105, 128, "qkv")
    want = fv.fvattn_rope(Q, K, pos, rope)
    # into a slice of a larger buffer, the rest of which stays
    buf = torch.full((2, 105, 11, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    oq, ok = buf[:, :, :8, 0].transpose(1, 2), buf[:, :, 8:, 1].transpose(1, 2)
    fv.fvattn_rope(Q, K, pos, rope, out_q=oq, out_k=ok)
    assert torch.equal(oq, want[0]) and torch.equal(ok, want[1])
    assert (buf[:, :, :8, 1] == 7).all() and (buf[:, :, 8:, 0] == 7).all()
    fv.fvattn_rope(Q, K, pos, rope, out_q=Q, out_k=K)
    assert torch.equal(Q, want[0]) and torch.equal(K, want[1])


def test_rope_passing_channels_keep_nan_and_infinities():
    import top_routed_block_b200 as fv
    for pairing in ("interleaved", "half"):
        rope = fv.rope_axes((32, 16), pairing=pairing)
        x = torch.randn(1, 1, 4, 128, device="cuda").to(torch.bfloat16)
        x[0, 0, 1, 48:] = float("inf")
        x[0, 0, 2, 49] = float("nan")
        x[0, 0, 3, 0] = float("nan")
        y, _ = fv.fvattn_rope(x, None, fv.grid_positions(1, 2, 2)[:, 1:].contiguous(), rope)
        assert torch.equal(y[..., 48:].view(torch.int16), x[..., 48:].view(torch.int16))
        bad = torch.isnan(y[0, 0, 3])
        assert bad.sum() == 2 and bad[0] and bad[1 if pairing == "interleaved" else 24]
        assert torch.isfinite(y[0, 0, 0]).all() and torch.isfinite(y[0, 0, 1, :48]).all()


def test_rope_on_another_stream_and_in_a_graph():
    import top_routed_block_b200 as fv
    rng = np.random.default_rng(13)
    rope = fv.rope_axes((24, 20, 20))
    pos = fv.grid_positions(2, 8, 9)
    Q, K = make(rng, 1, 3, 144, 64, "bhnd")
    want = fv.fvattn_rope(Q, K, pos, rope)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = fv.fvattn_rope(Q, K, pos, rope, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    outs = [torch.empty_like(Q), torch.empty_like(K)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fv.fvattn_rope(Q, K, pos, rope, out_q=outs[0], out_k=outs[1])
    Q.copy_(torch.randn_like(Q))
    graph.replay()
    want = fv.fvattn_rope(Q, K, pos, rope)
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_rope_angles_that_vanish_or_turn_backwards():
    """A step just below zero revolutions is none (not one short of a whole); negative frequencies turn back."""
    import top_routed_block_b200 as fv
    rng = np.random.default_rng(15)
    pos = torch.arange(40, dtype=torch.int32, device="cuda").view(40, 1)
    Q, _ = make(rng, 1, 2, 40, 64, "bhnd")
    axis = np.zeros(32, np.int32)
    still = fv.RopeAxes(np.full(32, -1e-30), axis)
    assert torch.equal(fv.fvattn_rope(Q, None, pos, still)[0], Q)
    back = fv.RopeAxes(-fv.rope_axes((64,)).inv_freq, axis)
    check(fv.fvattn_rope(Q, None, pos, back)[0], Q, pos, back)


def test_rope_refuses_on_the_gpu():
    import top_routed_block_b200 as fv
    Q = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(8, 1, dtype=torch.int32, device="cuda")
    rope = fv.rope_axes((64,))
    for bad in (Q.float(), Q[..., ::2], Q[0]):
        with pytest.raises(ValueError):
            fv.fvattn_rope(bad, None, pos, rope)
    for p in (pos.long(), pos[:7], pos.cpu(), pos[:, 0]):
        with pytest.raises(ValueError):
            fv.fvattn_rope(Q, None, p, rope)
    with pytest.raises(ValueError):
        fv.fvattn_rope(Q, None, pos, rope._replace(pairing="neither"))
    with pytest.raises(ValueError):
        fv.fvattn_rope(Q, Q[:, :, :4], pos, rope)
    with pytest.raises(fv.FvattnError):   # an axis that is 0 only in 32 bits
        fv.fvattn_rope(Q, None, pos, rope._replace(pair_axis=[1 << 32] * 32))
    with pytest.raises(RuntimeError):     # no single truth value
        fv.fvattn_rope(Q, None, pos, rope, inverse=pos)
    with pytest.raises(fv.FvattnError):
        fv.fvattn_rope(Q, None, pos, rope, out_q=Q[:, :1].expand(1, 2, 8, 64))


def test_training_step_with_positions():
    """rope -> attention -> its gradients -> rope's gradients, against fp64 autograd of the formulas
    (the backward's own bounds: relative Frobenius error 2e-2, and bf16 roundings of Q, K, dQ, dK)."""
    import top_routed_block_b200 as fv
    rng = np.random.default_rng(17)
    B, H, d = 1, 2, 64
    pos = fv.grid_positions(3, 9, 11)
    N = pos.shape[0]
    rope = fv.rope_axes((24, 20, 20))
    x = torch.from_numpy(rng.standard_normal((B, N, 3, H, d)).astype(np.float32)).to(torch.bfloat16).cuda()
    Q, K, V = (x[:, :, i].transpose(1, 2) for i in range(3))
    Vc = V.contiguous()
    plan = fv.FvattnPlan(B, H, N, d, 128)
    O, LSE, st = plan(Q, K, Vc, 1.0, positions=pos, rope=rope)
    plan.check()
    turned = plan.turned
    dO = torch.randn(B, H, N, d, device="cuda").to(torch.bfloat16)
    gq, gk, gv, st = fv.fvattn_sparse_bwd(*plan.turned, Vc, O, LSE, dO, plan.route.row_ptr, plan.route.col_idx, 128)
    fv.check_status(st)
    plan(*turned, Vc, 1.0)
    assert plan.turned is None   # of the last call, which turned nothing
    grad = torch.empty_like(x)
    fv.fvattn_rope_bwd(gq, gk, pos, rope, out_q=grad[:, :, 0].transpose(1, 2), out_k=grad[:, :, 1].transpose(1, 2))
    grad[:, :, 2] = gv.transpose(1, 2)

    leaf = x.double().requires_grad_()
    ang = pos.double()[:, torch.from_numpy(rope.pair_axis).long().cuda()] * torch.from_numpy(rope.inv_freq).cuda()

    def turn(t):
        a, b = t[..., 0::2], t[..., 1::2]
        return torch.stack([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1).flatten(-2)

    q, k, v = (leaf[:, :, i].transpose(1, 2) for i in range(3))
    o = torch.softmax(turn(q) @ turn(k).transpose(-1, -2) / d ** 0.5, -1) @ v
    o.backward(dO.double())
    assert (O.double() - o).abs().max() < 2e-2
    for i in range(3):
        want, got = leaf.grad[:, :, i], grad[:, :, i].double()
        assert (got - want).norm() / want.norm() < 2e-2


def test_rope_offsets_past_32_bits():
    """Tokens 2^22 elements apart: the last ones begin past 2^31 elements."""
    import top_routed_block_b200 as fv
    rng = np.random.default_rng(19)
    N, step = 600, 1 << 22
    x = torch.empty(N * step, dtype=torch.bfloat16, device="cuda").as_strided((1, 2, N, 64), (0, 64, step, 1))
    Q, _ = make(rng, 1, 2, N, 64, "bhnd")
    x.copy_(Q)
    rope = fv.rope_axes((24, 20, 20))
    pos = fv.grid_positions(3, 10, 20)
    want, _ = fv.fvattn_rope(Q, None, pos, rope)
    got, _ = fv.fvattn_rope(x, None, pos, rope)
    assert torch.equal(got, want)
    fv.fvattn_rope(x, None, pos, rope, out_q=x)
    assert torch.equal(x, want)
