"""The per-head norm with rotation, its gradient and the 8-bit activation rows
on the GPU against a plain computation in 64 bits.

Tolerances (u = half a step of the output type relative to the value:
2^-24 fp32, 2^-8 bf16).  The kernel computes in fp32: the mean of squares of
D values and rsqrt are off by a few 2^-24, the products x r w and the two
products of the turn by one 2^-24 each, so an output is within 16 * 2^-24 of
|n_a| + |n_b| (the pair's magnitudes), then rounded once:
    |err| <= u |y| + 16 * 2^-24 * (|n_a| + |n_b|).
dx = r (g w - h m): the two terms are each within 32 * 2^-24 of their
magnitude (m adds a sum of D terms, at most D |g w h|_max):
    |err| <= u |dx| + 32 * 2^-24 * r * (|g w| + |h| mean|g w h|).
dw: each term within 32 * 2^-24 of its magnitude, and rows are summed in
parts of at most R terms one after another: (32 + R) * 2^-24 * sum |g h|
with R <= 64 + rows / 2048."""
import math

import pytest
import torch

from dynamic_block_sparse_pool_b200 import DSAError, ops

pytestmark = pytest.mark.gpu

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
E = 2.0 ** -24


def angles(pos, pairs, theta, D):
    """cos, sin [B, N, 1, D/2] in 64 bits."""
    out = torch.zeros(pos.shape[0], pos.shape[1], D // 2, dtype=torch.float64)
    m = 0
    for a, n in enumerate(pairs):
        for i in range(n):
            out[..., m] = pos[..., a].double().clamp(min=0) * theta ** (-i / n)
            m += 1
    return out.cos()[:, :, None], out.sin()[:, :, None]


def pair_split(x, halves):
    return x.chunk(2, -1) if halves else (x[..., 0::2], x[..., 1::2])


def pair_join(a, b, halves):
    return torch.cat([a, b], -1) if halves else torch.stack([a, b], -1).flatten(-2)


def turn(x, c, s, halves):
    a, b = pair_split(x, halves)
    return pair_join(a * c - b * s, a * s + b * c, halves)


def forward64(x, w, eps, c, s, halves):
    x = x.double().cpu()
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    n = x * r * (1.0 if w is None else w.double().cpu())
    a, b = pair_split(n.abs(), halves)
    return turn(n, c, s, halves).transpose(1, 2), pair_join(a + b, a + b, halves).transpose(1, 2)


def backward64(dy, x, w, eps, c, s, halves):
    x, dy = x.double().cpu(), dy.double().cpu().transpose(1, 2)
    w = torch.ones(x.shape[-1], dtype=torch.float64) if w is None else w.double().cpu()
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    h = x * r
    g = turn(dy, c, -s, halves)
    a, b = pair_split(dy.abs(), halves)
    gm = pair_join(a + b, a + b, halves)  # the magnitudes that the turn mixes
    m = (g * w * h).mean(-1, keepdim=True)
    dx = r * (g * w - h * m)
    mag = r * (gm * w.abs() + h.abs() * (gm * w.abs() * h.abs()).mean(-1, keepdim=True))
    return dx, mag, (g * h).flatten(0, 2).sum(0), (gm * h.abs()).flatten(0, 2).sum(0)


def close(got, ref, mag, dtype, k):
    err = (got.double().cpu() - ref).abs()
    lim = U[dtype] * ref.abs() + k * E * mag + 1e-30
    assert bool((err <= lim).all()), float((err / lim).max())


def inputs(B, N, Hq, Hk, D, dtype, seed, fused=False, scale=1.5):
    g = torch.Generator().manual_seed(seed)
    if fused:
        qkv = (scale * torch.randn(B, N, Hq + 2 * Hk, D, generator=g)).to(dtype).cuda()
        xq, xk = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
    else:
        xq = (scale * torch.randn(B, N, Hq, D, generator=g)).to(dtype).cuda()
        xk = (scale * torch.randn(B, N, Hk, D, generator=g)).to(dtype).cuda()
    wq, wk = ((1 + 0.3 * torch.randn(D, generator=g)).cuda() for _ in range(2))
    dq = torch.randn(B, Hq, N, D, generator=g).to(dtype).cuda()
    dk = torch.randn(B, Hk, N, D, generator=g).to(dtype).cuda()
    return xq, xk, wq, wk, dq, dk


CASES = [
    # B, N, Hq, Hk, D, dtype, fused, halves, grid
    (1, 1, 1, 1, 64, torch.float32, False, False, False),
    (3, 1, 8, 2, 128, torch.bfloat16, False, True, False),
    (2, 37, 5, 3, 64, torch.bfloat16, True, True, False),
    (1, 130, 3, 1, 128, torch.float32, True, False, True),
    (1, 226 + 4 * 6 * 7, 6, 6, 64, torch.bfloat16, True, False, True),
    (2, 1100, 9, 7, 128, torch.bfloat16, False, False, False),  # many tokens: four rows a thread
    (1, 2500, 3, 2, 64, torch.float32, False, True, False),
]


def make_plan(B, N, D, halves, grid, per_batch=True):
    if grid:
        P, T, Y, X = (226, 4, 6, 7) if N == 394 else (4, 3, 6, 7)
        pos = torch.full((1, N, 3), -1, dtype=torch.int32)
        t, y, x = torch.meshgrid(torch.arange(T), torch.arange(Y), torch.arange(X), indexing="ij")
        pos[0, P:] = torch.stack([t.reshape(-1), y.reshape(-1), x.reshape(-1)], 1).int()
        pairs, theta = (D // 2 - 2 * (D // 6), D // 6, D // 6), 256.0
        plan = ops.RopePlan.grid(T, Y, X, D, n_prefix=P, theta=theta)
        assert torch.equal(plan.pos.cpu(), pos)
        return plan, pos, pairs, theta
    pos = (90000 + torch.arange(N)[None] + 1000 * torch.arange(B)[:, None]).int()[..., None]
    pairs, theta = (D // 2 - 3,), 500000.0  # three pairs do not turn
    return ops.RopePlan(pos, pairs, theta=theta, halves=halves), pos, pairs, theta


@pytest.mark.parametrize("B,N,Hq,Hk,D,dtype,fused,halves,grid", CASES)
def test_forward_and_gradient(B, N, Hq, Hk, D, dtype, fused, halves, grid):
    xq, xk, wq, wk, dq, dk = inputs(B, N, Hq, Hk, D, dtype, seed=N + D, fused=fused)
    plan, pos, pairs, theta = make_plan(B, N, D, halves, grid)
    c, s = angles(pos, pairs, theta, D)
    q, k = ops.qk_norm_rope(xq, xk, wq, wk, plan, 1e-6)
    got = ops.qk_norm_rope_bwd(dq, dk, xq, xk, wq, wk, plan, 1e-6)
    again = ops.qk_norm_rope_bwd(dq, dk, xq, xk, wq, wk, plan, 1e-6)
    ops.device_status()
    for y, x, w in ((q, xq, wq), (k, xk, wk)):
        close(y, *forward64(x, w, 1e-6, c, s, halves), dtype, 16)
    rows = B * N * max(Hq, Hk)
    for dy, x, w, dx, dw in ((dq, xq, wq, got[0], got[2]), (dk, xk, wk, got[1], got[3])):
        rx, mx, rw, mw = backward64(dy, x, w, 1e-6, c, s, halves)
        close(dx, rx, mx, dtype, 32)
        close(dw, rw, mw, torch.float32, 32 + 64 + rows / 2048)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_gradient_against_differences():
    B, N, H, D = 1, 3, 2, 64
    xq, xk, wq, wk, dq, dk = inputs(B, N, H, H, D, torch.float32, seed=9)
    plan, pos, pairs, theta = make_plan(B, N, D, True, False)
    c, s = angles(pos, pairs, theta, D)
    dxq, _, dwq, _ = ops.qk_norm_rope_bwd(dq, dk, xq, xk, wq, wk, plan, 1e-6)

    def loss(x, w):
        return float((forward64(x, w, 1e-6, c, s, True)[0] * dq.double().cpu()).sum())

    x64, w64, h = xq.double().cpu(), wq.double().cpu(), 1e-5
    for i in range(0, x64.numel(), 17):  # central differences: h^2 and 1e-16 / h, far below 1e-6
        d = torch.zeros(x64.numel(), dtype=torch.float64)
        d[i] = h
        d = d.view_as(x64)
        diff = (loss(x64 + d, w64) - loss(x64 - d, w64)) / (2 * h)
        assert abs(diff - float(dxq.flatten()[i])) <= 1e-5 * (1 + abs(diff))
    for i in range(0, D, 7):
        d = torch.zeros(D, dtype=torch.float64)
        d[i] = h
        diff = (loss(x64, w64 + d) - loss(x64, w64 - d)) / (2 * h)
        assert abs(diff - float(dwq[i])) <= 1e-5 * (1 + abs(diff))


def test_no_weights_zero_rows_and_large_values():
    # ones for weights; a row of zeros comes out zero; large fp32 rows stay finite
    B, N, H, D = 1, 4, 2, 128
    xq, xk, _, _, dq, dk = inputs(B, N, H, H, D, torch.float32, seed=3)
    xq[0, 1] = 0
    xq[0, 2] *= 1e17
    plan, pos, pairs, theta = make_plan(B, N, D, False, False)
    c, s = angles(pos, pairs, theta, D)
    q, k = ops.qk_norm_rope(xq, xk, None, None, plan, 1e-6)
    dxq = ops.qk_norm_rope_bwd(dq, dk, xq, xk, None, None, plan, 1e-6)[0]
    ops.device_status()
    assert torch.all(q[0, :, 1] == 0)
    close(q, *forward64(xq, None, 1e-6, c, s, False), torch.float32, 16)
    rx, mx, _, _ = backward64(dq, xq, None, 1e-6, c, s, False)
    close(dxq, rx, mx, torch.float32, 32)


def test_strided_gradient_into_a_fused_buffer_and_broadcast_input():
    B, N, H, Hk, D = 2, 21, 4, 2, 64
    xq, xk, wq, wk, dq, dk = inputs(B, N, H, Hk, D, torch.bfloat16, seed=5, fused=True)
    plan = ops.RopePlan(torch.arange(N)[:, None], (D // 2,))
    want = ops.qk_norm_rope_bwd(dq, dk, xq, xk, wq, wk, plan)
    buf = torch.full((B, N, H + 2 * Hk, D), 7.0, device="cuda", dtype=torch.bfloat16)
    got = ops.qk_norm_rope_bwd(dq, dk, xq, xk, wq, wk, plan, dxq=buf[:, :, :H], dxk=buf[:, :, H:H + Hk])
    ops.device_status()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.all(buf[:, :, H + Hk:] == 7.0)  # the values' part is left as it was
    one = xq[:1].expand(B, N, H, D)  # one row of tokens for every batch entry
    assert torch.equal(ops.qk_norm_rope(one, xk, wq, wk, plan)[0][1],
                       ops.qk_norm_rope(xq[:1].contiguous(), xk[:1].contiguous(), wq, wk, plan)[0][0])


def codes64(x):
    """Codes and scales by the same three fp32 operations, in numpy's fp32."""
    import numpy as np
    v = x.float().cpu().numpy()
    amax = np.abs(v).max(-1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore"):
        inv = np.where(amax >= 2.0 ** -119, np.float32(127.0) / amax, np.float32(0)).astype(np.float32)
    scale = np.where(amax >= 2.0 ** -119, amax / np.float32(127.0), np.float32(0)).astype(np.float32)
    return np.rint(v * inv).astype(np.int8), scale[..., 0]


@pytest.mark.parametrize("shape,dtype", [((1, 64), torch.float32), ((3, 5, 128), torch.bfloat16),
                                         ((257, 64), torch.bfloat16), ((2, 1001, 128), torch.float32)])
def test_pack8_codes_are_exact(shape, dtype):
    import numpy as np
    g = torch.Generator().manual_seed(shape[0])
    x = (torch.randn(shape, generator=g) * torch.exp(3 * torch.randn(shape[:-1] + (1,), generator=g))).to(dtype)
    x[..., 0, :] = 0 if len(shape) > 1 and shape[-2] > 1 else x[..., 0, :]
    a = ops.pack8(x.cuda())
    codes, scales = codes64(x)
    assert np.array_equal(a.codes.cpu().numpy(), codes)
    assert np.array_equal(a.scales.cpu().numpy(), scales)
    back = ops.unpack8(a, torch.float32)
    assert torch.equal(back.cpu(), torch.from_numpy(codes.astype(np.float32) * scales[..., None]))
    assert torch.equal(ops.unpack8(a, torch.bfloat16).cpu(), back.cpu().bfloat16())
    # half a step, and three fp32 roundings of values up to amax
    err = (back.double().cpu() - x.double()).abs()
    amax = x.double().abs().amax(-1, keepdim=True)
    assert bool((err <= amax * (0.5 / 127 + 4 * E)).all())


def test_pack8_non_finite_and_tiny_rows():
    x = torch.randn(5, 64)
    x[1, 3] = float("inf")
    x[2, 5] = float("nan")
    x[3] = 2.0 ** -130
    back = ops.unpack8(ops.pack8(x.cuda()), torch.float32).cpu()
    assert torch.isnan(back[1]).all() and torch.isnan(back[2]).all()
    assert torch.all(back[3] == 0) and torch.isfinite(back[[0, 4]]).all()


@pytest.mark.parametrize("D,halves,N,H,Hk", [(64, False, 33, 3, 2), (128, True, 2300, 4, 4)])
def test_8bit_checkpoint_of_a_step(D, halves, N, H, Hk):
    # the forward's saved rows are pack8's; its outputs do not change; the
    # backward and a recomputed forward from the rows are those of the values
    # the rows stand for
    xq, xk, wq, wk, dq, dk = inputs(1, N, H, Hk, D, torch.bfloat16, seed=N, fused=True)
    plan, pos, pairs, theta = make_plan(1, N, D, halves, False)
    c, s = angles(pos, pairs, theta, D)
    q, k, q8, k8 = ops.qk_norm_rope(xq, xk, wq, wk, plan, save8=True)
    q0, k0 = ops.qk_norm_rope(xq, xk, wq, wk, plan)
    assert torch.equal(q, q0) and torch.equal(k, k0)
    for a, x in ((q8, xq), (k8, xk)):
        want = ops.pack8(x.contiguous())
        assert torch.equal(a.codes, want.codes) and torch.equal(a.scales, want.scales)
    vq, vk = ops.unpack8(q8, torch.float32), ops.unpack8(k8, torch.float32)
    rq, rk = ops.qk_norm_rope(q8, k8, wq, wk, plan, dtype=torch.bfloat16)
    got = ops.qk_norm_rope_bwd(dq, dk, q8, k8, wq, wk, plan)
    ops.device_status()
    close(rq, *forward64(vq, wq, 1e-6, c, s, halves), torch.bfloat16, 16)
    close(rk, *forward64(vk, wk, 1e-6, c, s, halves), torch.bfloat16, 16)
    for dy, v, w, dx, dw in ((dq, vq, wq, got[0], got[2]), (dk, vk, wk, got[1], got[3])):
        rx, mx, rw, mw = backward64(dy, v, w, 1e-6, c, s, halves)
        close(dx, rx, mx, torch.bfloat16, 32)
        close(dw, rw, mw, torch.float32, 32 + 64 + N * H / 2048)


def test_position_past_the_table_is_reported():
    N, D = 5, 64
    xq, xk, wq, wk, _, _ = inputs(1, N, 2, 2, D, torch.bfloat16, seed=1)
    plan = ops.RopePlan(torch.arange(N)[:, None], (D // 2,))
    want = ops.qk_norm_rope(xq, xk, wq, wk, plan)[0]
    ops.device_status()
    got = ops.qk_norm_rope(xq, xk, wq, wk, plan.at(torch.tensor([[0], [1], [99], [3], [4]])))[0]
    with pytest.raises(DSAError, match="rotation-position"):
        ops.device_status()
    ops.device_status()
    assert torch.equal(got[:, :, [0, 1, 3, 4]], want[:, :, [0, 1, 3, 4]])
    assert torch.equal(got[:, :, 2], ops.qk_norm_rope(xq, xk, wq, wk, plan.at(torch.full((N, 1), -1)))[0][:, :, 2])


def test_positions_beyond_32_bits_are_reported():
    N, D = 3, 64
    xq, xk, wq, wk, _, _ = inputs(1, N, 2, 2, D, torch.bfloat16, seed=4)
    plan = ops.RopePlan(torch.arange(N)[:, None], (D // 2,))
    got = ops.qk_norm_rope(xq, xk, wq, wk, plan.at(torch.tensor([[0], [2**32 + 1], [-2**40]])))[0]
    with pytest.raises(DSAError, match="rotation-position"):  # not taken for position 1
        ops.device_status()
    still = ops.qk_norm_rope(xq, xk, wq, wk, plan.at(torch.tensor([[0], [-1], [-1]])))[0]
    ops.device_status()
    assert torch.equal(got, still)


def test_captured_and_other_stream():
    N, D = 64, 128
    xq, xk, wq, wk, dq, dk = inputs(1, N, 4, 4, D, torch.bfloat16, seed=2)
    plan = ops.RopePlan(torch.arange(N)[:, None], (D // 2,), halves=True)
    want = ops.qk_norm_rope(xq, xk, wq, wk, plan) + ops.qk_norm_rope_bwd(dq, dk, xq, xk, wq, wk, plan)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        got = ops.qk_norm_rope(xq, xk, wq, wk, plan) + ops.qk_norm_rope_bwd(dq, dk, xq, xk, wq, wk, plan)
    for t in got:
        t.fill_(0)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_offsets_past_32_bits():
    # 2^31 elements and more: the last tokens against the same tokens alone, saved codes among them
    N, H, D, n = 270_000, 64, 128, 1003
    torch.manual_seed(0)
    xq, dq = (torch.empty(1, N, H, D, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    for t in (xq, dq):
        for i in range(0, N, 30_000):
            t[0, i:i + 30_000].normal_()
    dq = dq.view(1, H, N, D)
    xk, dk = xq[:, :, :1], dq[:, :1]
    wq, wk = torch.rand(D, device="cuda") + 0.5, torch.rand(D, device="cuda") + 0.5
    plan = ops.RopePlan((torch.arange(N) % 4096)[:, None], (D // 2,))
    end = plan.at(plan.pos[0, -n:])
    tail = [t[:, -n:].contiguous() for t in (xq, xk)] + [t[:, :, -n:].contiguous() for t in (dq, dk)]
    got = ops.qk_norm_rope(xq, xk, wq, wk, plan, save8=True)
    want = ops.qk_norm_rope(tail[0], tail[1], wq, wk, end, save8=True)
    assert torch.equal(got[0][:, :, -n:], want[0]) and torch.equal(got[1][:, :, -n:], want[1])
    assert torch.equal(got[2].codes[:, -n:], want[2].codes) and torch.equal(got[2].scales[:, -n:], want[2].scales)
    assert torch.equal(ops.unpack8(got[2])[:, -n:], ops.unpack8(want[2]))
    assert torch.equal(ops.pack8(xq).codes[:, -n:], want[2].codes)
    for x8, end8 in (((xq, xk), tail[:2]), (got[2:], want[2:])):
        d = ops.qk_norm_rope_bwd(dq, dk.contiguous(), *x8, wq, wk, plan)
        e = ops.qk_norm_rope_bwd(tail[2], tail[3], *end8, wq, wk, end)
        assert torch.equal(d[0][:, -n:], e[0]) and torch.equal(d[1][:, -n:], e[1])
    ops.device_status()
    del xq, dq, xk, dk, tail, got, want, x8, end8, d, e, t
    torch.cuda.empty_cache()
