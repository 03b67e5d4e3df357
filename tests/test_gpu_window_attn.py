"""The window attention (forward, gradients, single tokens over a cache) on the
GPU against a dense computation in 64 bits.

Tolerances, with u half a step of the type relative to the value (2^-8 bf16,
2^-24 fp32), E = 2^-24, and per row
    eS = scale D E max_u sum_d |q_d k_ud|
the error of a score from its fp32 sum.  A weight exp(s - m) is then off by
eP = 2 eS + 2^-19 relative (the exponentials and the row's reference add a few
2^-22, the sum of n terms n E), and
    o:    u |o| + (2 eP + uP + n E) sum p |v|,  uP = 2^-8 (bf16: P is rounded
          for the second product), 0 (fp32);
    lse:  eP + 2^-22 |lse|.
Gradients, given o and lse as inputs: eW = eP + 2^-22 |lse| for P; the fp32
sums of D terms put eD = 2 D E (sum |do v| + sum |do o|) on dP - delta; so
dS is off by fS = p (eW |dP - delta| + eD) + t |dS| with t = 2 E in fp32; in
bf16 it enters dq as two terms, hi + lo = dS (1 + 2^-8 2^-8): t = 2^-16, and dk
as one term, rounded once: t = uP = 2^-8 (half a step, as P for dv):
    dq:   u |dq| + scale (sum fS |k| + n E sum |dS k|),  dk alike with |q|;
    dv:   u |dv| + (eW + uP + n E) sum p |do|."""
import math

import pytest
import torch

from dynamic_block_sparse_pool_b200 import DSAError, ops

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
U = {torch.float32: E, torch.bfloat16: 2.0 ** -8}
UP = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8}


def visible(Nq, Nk, off, left, right, sink):
    t = off + torch.arange(Nq)[:, None]
    u = torch.arange(Nk)[None]
    ok = torch.ones(Nq, Nk, dtype=torch.bool)
    if right >= 0:
        ok &= u <= t + right
    if left >= 0:
        ok &= (u < sink) | (u >= t - left)
    return ok


def per_head(t, H):
    return t.double().cpu().repeat_interleave(H // t.shape[1], 1)


def dense(q, k, v, ok, scale):
    """o, lse, p and the bounds' ingredients, all [B, H, ...] in 64 bits."""
    H, D = q.shape[1], q.shape[3]
    qd, kd, vd = q.double().cpu(), per_head(k, H), per_head(v, H)
    s = (qd @ kd.transpose(2, 3) * scale).masked_fill(~ok, -math.inf)
    m = s.amax(-1, keepdim=True).clamp(min=-1e300)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    p = p / l.clamp(min=1e-300)
    lse = torch.where(l > 0, m + l.log(), torch.full_like(l, -math.inf))[..., 0]
    es = scale * D * E * (qd.abs() @ kd.abs().transpose(2, 3)).amax(-1, keepdim=True)
    return p @ vd, lse, p, 2 * es + 2.0 ** -19, qd, kd, vd


def inside(got, ref, lim, what):
    err = (got.double().cpu() - ref).abs()
    assert torch.isfinite(got).all(), what
    assert bool((err <= lim + 1e-30).all()), (what, float((err / (lim + 1e-30)).max()))


def make(B, H, Hk, Nq, Nk, D, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    t = lambda h, n: (scale * torch.randn(B, h, n, D, generator=g)).to(dtype).cuda()  # noqa: E731
    return t(H, Nq), t(Hk, Nk), t(Hk, Nk), torch.randn(B, H, Nq, D, generator=g).to(dtype).cuda()


def check_forward(q, k, v, off, left, right, sink, scale=None, got=None):
    D, dt = q.shape[3], q.dtype
    sc = D ** -0.5 if scale is None else scale
    ok = visible(q.shape[2], k.shape[2], off, left, right, sink)
    o, lse, p, ep, _, _, vd = dense(q, k, v, ok, sc)
    if got is None:
        got = ops.window_attn_fwd(q, k, v, left, right, sink, q_offset=off, scale=scale)
        ops.device_status()
    n = ok.sum(-1, keepdim=True)
    inside(got[0], o, U[dt] * o.abs() + (2 * ep + UP[dt] + n * E) * (p @ vd.abs()), "o")
    hidden = ~ok.any(-1)
    gl = got[1].double().cpu()
    assert torch.all(gl[..., hidden] == -math.inf) and torch.all(got[0].cpu()[..., hidden, :] == 0)
    seen = ok.any(-1)
    assert bool(((gl - lse).abs() <= ep[..., 0] + 2.0 ** -22 * lse.abs())[..., seen].all())
    return got


def check_backward(q, k, v, do, off, left, right, sink, scale=None):
    B, H, Nq, D = q.shape
    Hk, Nk, dt = k.shape[1], k.shape[2], q.dtype
    sc = D ** -0.5 if scale is None else scale
    ok = visible(Nq, Nk, off, left, right, sink)
    o64, lse64, p, ep, qd, kd, vd = dense(q, k, v, ok, sc)
    out, lse = o64.to(dt).cuda(), lse64.float().cuda()  # the stored forward, from the oracle
    args = dict(left=left, right=right, sink=sink, q_offset=off, scale=scale)
    got = ops.window_attn_bwd(q, k, v, out, do, lse, **args)
    again = ops.window_attn_bwd(q, k, v, out, do, lse, **args)
    ops.device_status()
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    dd, od = do.double().cpu(), out.double().cpu()
    lse = lse.double().cpu()[..., None]
    p = torch.where(ok, torch.exp((qd @ kd.transpose(2, 3)) * sc - lse.clamp(min=-1e300)), torch.zeros(()).double())
    dp, delta = dd @ vd.transpose(2, 3), (dd * od).sum(-1, keepdim=True)
    ds = p * (dp - delta)
    ew = ep + 2.0 ** -22 * lse.abs().clamp(max=1e30)
    ed = 2 * D * E * (dd.abs() @ vd.abs().transpose(2, 3) + (dd * od).abs().sum(-1, keepdim=True))
    fs = p * (ew * (dp - delta).abs() + ed)
    fsq = fs + (2.0 ** -16 if dt == torch.bfloat16 else 2 * E) * ds.abs()
    fsk = fs + (UP[dt] + 2 * E) * ds.abs()
    grp = lambda x: x.view(B, Hk, H // Hk, *x.shape[2:]).sum(2)  # noqa: E731
    n = ok.sum(-1).max().item()
    m = ok.sum(0).max().item() * (H // Hk)
    dq = sc * ds @ kd
    inside(got[0], dq, U[dt] * dq.abs() + sc * (fsq + n * E * ds.abs()) @ kd.abs(), "dq")
    dk = grp(sc * ds.transpose(2, 3) @ qd)
    inside(got[1], dk, U[dt] * dk.abs() + grp(sc * (fsk + m * E * ds.abs()).transpose(2, 3) @ qd.abs()), "dk")
    dv = grp(p.transpose(2, 3) @ dd)
    inside(got[2], dv, U[dt] * dv.abs() + grp(((ew + UP[dt] + m * E) * p).transpose(2, 3) @ dd.abs()), "dv")
    return got


# B, H, Hk, Nq, Nk, D, off, left, right, sink
MASKS = [
    (1, 1, 1, 1, 1, 64, 0, 0, 0, 0),                 # one token, itself
    (2, 2, 1, 1, 200, 128, 199, 50, 0, 3),           # one query over many keys
    (1, 3, 3, 5, 131, 64, 126, -1, 0, 0),            # plain causal, newest five
    (1, 2, 2, 127, 127, 128, 0, 40, 0, 1),
    (1, 2, 2, 128, 128, 64, 0, -1, -1, 0),           # nothing hidden
    (1, 4, 2, 129, 129, 128, 0, 128, 0, 4),          # one past a tile
    (2, 4, 1, 300, 300, 64, 0, 77, 33, 5),           # uneven window on both sides, shared heads
    (1, 2, 1, 700, 700, 128, 0, 100, 0, 200),        # sinks over two tiles, then a gap
    (1, 1, 1, 640, 640, 64, 0, 0, 0, 0),             # every token sees itself alone
    (1, 2, 2, 400, 900, 128, 500, 130, 60, 7),       # new queries over a longer past
    (1, 2, 2, 300, 260, 64, -40, 90, 0, 2),          # the first 40 queries see nothing
    (1, 2, 2, 300, 200, 64, 150, 20, 0, 0),          # the last queries are past every key
    (1, 1, 1, 300, 200, 128, 150, 20, 0, 150),       # those see the sinks alone
    (1, 1, 1, 200, 500, 64, 0, -1, 250, 0),          # bounded to the right alone
    (1, 1, 1, 520, 520, 64, 0, 64, 10, 100),         # a right bound that hides some sinks
    (1, 5, 5, 1030, 1030, 64, 0, 255, 255, 77),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,H,Hk,Nq,Nk,D,off,left,right,sink", MASKS)
def test_forward(B, H, Hk, Nq, Nk, D, off, left, right, sink, dtype):
    q, k, v, _ = make(B, H, Hk, Nq, Nk, D, dtype, seed=Nq + Nk)
    check_forward(q, k, v, off, left, right, sink)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,H,Hk,Nq,Nk,D,off,left,right,sink", MASKS)
def test_backward(B, H, Hk, Nq, Nk, D, off, left, right, sink, dtype):
    q, k, v, do = make(B, H, Hk, Nq, Nk, D, dtype, seed=Nq + 3 * Nk)
    check_backward(q, k, v, do, off, left, right, sink)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,H,Hk,Nq,Nk,off,left,right,sink", [
    (1, 8, 2, 1100, 1100, 0, 150, 0, 130),   # two tiles with sinks, 36 pairs each, against 8 or 12 of the others
    (1, 8, 1, 1000, 1500, 0, -1, 0, 0),      # 64 pairs down to 8, and the last keys that no query sees
    (2, 6, 1, 700, 1300, 500, -1, -1, 5),    # both kinds in parts, two batches
])
def test_backward_of_key_tiles_in_parts(B, H, Hk, Nq, Nk, off, left, right, sink, D):
    q, k, v, do = make(B, H, Hk, Nq, Nk, D, torch.bfloat16, seed=Nk)
    check_backward(q, k, v, do, off, left, right, sink)


@pytest.mark.parametrize("D", [64, 128])
def test_two_query_tiles_per_item(D):
    # more items than SMs, so each item takes two query tiles; the last one has one
    q, k, v, _ = make(1, 160, 20, 390, 390, D, torch.bfloat16, seed=D)
    check_forward(q, k, v, 0, 140, 0, 3)
    check_forward(q, k, v, 0, 30, 20, 130)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_growing_scores_move_the_reference(dtype):
    # keys whose scores rise by far more than the step from tile to tile, and fall again
    q, k, v, do = make(1, 1, 1, 500, 500, 64, dtype, seed=1)
    q[:] = 0
    q[..., 0] = 4.0
    ramp = torch.cat([torch.arange(250), torch.arange(250, 0, -1)]).float().cuda()
    k[..., 0] = (ramp[None, None] * 2).to(dtype)
    check_forward(q, k, v, 0, -1, -1, 0)
    check_forward(q, k, v, 0, 300, 0, 10)
    check_backward(q, k, v, do, 0, 300, 0, 10)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_hidden_keys_do_not_matter(dtype):
    q, k, v, _ = make(1, 2, 2, 50, 300, 64, dtype, seed=8)
    want = ops.window_attn_fwd(q, k, v, 60, 0, 4, q_offset=200)
    k2 = k.clone()
    k2[:, :, 10:130] = float("nan")
    k2[:, :, 130:140] = float("inf")
    k2[:, :, 255:] = float("-inf")
    got = ops.window_attn_fwd(q, k2, v, 60, 0, 4, q_offset=200)
    ops.device_status()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_gradient_against_differences():
    q, k, v, do = make(1, 2, 1, 9, 9, 64, torch.float32, seed=4)
    ok = visible(9, 9, 0, 3, 1, 1)
    out, lse = ops.window_attn_fwd(q, k, v, 3, 1, 1)
    grads = ops.window_attn_bwd(q, k, v, out, do, lse, 3, 1, 1)
    ops.device_status()
    x = [t.double().cpu() for t in (q, k, v)]

    def loss():
        return float((dense(*x, ok, 64 ** -0.5)[0] * do.double().cpu()).sum())

    h = 1e-5
    for t, g in zip(x, grads):
        flat, gf = t.view(-1), g.double().cpu().view(-1)
        for i in range(0, flat.numel(), 41):
            keep = float(flat[i])
            flat[i] = keep + h
            a = loss()
            flat[i] = keep - h
            b = loss()
            flat[i] = keep
            d = (a - b) / (2 * h)
            assert abs(d - float(gf[i])) <= 1e-5 * (1 + abs(d))


def test_captured_streams_and_a_step_in_a_graph():
    q, k, v, do = make(1, 4, 2, 333, 333, 128, torch.bfloat16, seed=6)
    want_o, want_l = ops.window_attn_fwd(q, k, v, 100, 0, 4)
    want = ops.window_attn_bwd(q, k, v, want_o, do, want_l, 100, 0, 4)
    torch.cuda.synchronize()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        o, l = ops.window_attn_fwd(q, k, v, 100, 0, 4)
        grads = ops.window_attn_bwd(q, k, v, o, do, l, 100, 0, 4)
    o.zero_()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want_o) and torch.equal(l, want_l)
    assert all(torch.equal(a, b) for a, b in zip(grads, want))
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(5):
        for st in streams:
            with torch.cuda.stream(st):
                outs.append(ops.window_attn_fwd(q, k, v, 100, 0, 4)[0])
    torch.cuda.synchronize()
    ops.device_status()
    assert all(torch.equal(a, want_o) for a in outs)


# ---------------------------------------------------------------- cached form

# B, H, Hk, Nq, cap, D, left, sink, lens
CACHES = [
    (1, 1, 1, 1, 1, 64, -1, 0, [1]),
    (3, 4, 4, 1, 50, 128, 10, 2, [50, 1, 0]),
    (2, 8, 1, 1, 300, 64, 100, 4, [300, 97]),
    (2, 10, 2, 3, 700, 128, 200, 50, [700, 2]),        # more new tokens than the second stream holds
    (1, 24, 1, 4, 333, 64, 77, 0, [333]),              # rows over several tiles
    (1, 2, 2, 1, 5000, 128, -1, 0, [4999]),            # a cluster shares one head
    (2, 3, 3, 2, 4100, 64, 4000, 130, [4100, 3000]),
    (1, 2, 1, 1, 2000, 128, 0, 1, [2000]),
    (1, 4, 2, 2, 33000, 128, -1, 0, [32999]),          # large enough for shares through the workspace
    (2, 2, 2, 1, 40000, 64, 30000, 300, [40000, 31]),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,H,Hk,Nq,cap,D,left,sink,lens", CACHES)
@pytest.mark.parametrize("layout", ["heads", "tokens"])
def test_decode(B, H, Hk, Nq, cap, D, left, sink, lens, dtype, layout):
    q, k, v, _ = make(B, H, Hk, Nq, cap, D, dtype, seed=cap)
    if layout == "tokens":  # [B, cap, Hk, D] in memory
        k, v = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (k, v))
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    lse = torch.full((B, H, Nq), 7.0, device="cuda")
    out = ops.window_attn_decode(q, k, v, n, left, sink, lse=lse)
    assert torch.equal(out, ops.window_attn_decode(q, k, v, n, left, sink))
    ops.device_status()
    for b, ln in enumerate(lens):
        one = slice(b, b + 1)
        check_forward(q[one], k[one, :, :ln] if ln else k[one, :, :1], v[one, :, :ln] if ln else v[one, :, :1],
                      ln - Nq if ln else -Nq - 1, left, 0, sink, got=(out[one], lse[one]))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_decode_leaves_hidden_rows_alone(dtype):
    # rows that no query sees -- evicted, or behind the stream's end -- hold NaN
    q, k, v, _ = make(2, 6, 2, 1, 600, 128, dtype, seed=2)
    n = torch.tensor([600, 333], dtype=torch.int32, device="cuda")
    want = ops.window_attn_decode(q, k, v, n, left=100, sink=5)
    for t in (k, v):
        t[:, :, 5:232] = float("nan")
        t[0, :, 232:499] = float("nan")
        t[1, :, 333:] = float("nan")
    got = ops.window_attn_decode(q, k, v, n, left=100, sink=5)
    ops.device_status()
    assert torch.equal(got, want)


def test_decode_bad_lengths_are_reported():
    q, k, v, _ = make(3, 2, 2, 1, 64, 64, torch.bfloat16, seed=3)
    n = torch.tensor([65, 64, -1], dtype=torch.int32, device="cuda")
    out = ops.window_attn_decode(q, k, v, n)
    with pytest.raises(DSAError, match="cached-length"):
        ops.device_status()
    ops.device_status()
    assert torch.all(out[[0, 2]] == 0)
    assert torch.equal(out[1:2], ops.window_attn_decode(q[1:2], k[1:2], v[1:2], n[1:2]))


def test_workspaces_elsewhere_are_refused():
    q, k, v, do = make(1, 2, 1, 40, 40, 64, torch.bfloat16, seed=2)
    out, lse = ops.window_attn_fwd(q, k, v, 8)
    far = torch.empty(1 << 20, dtype=torch.uint8)
    with pytest.raises(ValueError, match="workspace"):
        ops.window_attn_bwd(q, k, v, out, do, lse, 8, workspace=far)
    with pytest.raises(ValueError, match="workspace"):
        ops.window_attn_decode(q, k, v, torch.tensor([40], dtype=torch.int32, device="cuda"), 8, workspace=far)
    with pytest.raises(ValueError, match="32 bits"):
        ops.window_attn_fwd(q, k, v, 2**32)


def test_decode_captured_over_a_growing_cache():
    q, k, v, _ = make(1, 8, 2, 1, 2048, 128, torch.bfloat16, seed=5)
    n = torch.tensor([1000], dtype=torch.int32, device="cuda")
    ops.window_attn_decode(q, k, v, n, 700, 4)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = ops.window_attn_decode(q, k, v, n, 700, 4)
    for ln in (1000, 1001, 2048, 3):
        n.fill_(ln)
        g.replay()
        assert torch.equal(out, ops.window_attn_decode(q, k, v, n, 700, 4))
    ops.device_status()


def test_decode_is_the_forward_of_the_last_tokens():
    q, k, v, _ = make(1, 8, 2, 700, 700, 128, torch.float32, seed=7)
    full, _ = ops.window_attn_fwd(q, k, v, 300, 0, 9)
    n = torch.tensor([700], dtype=torch.int32, device="cuda")
    last = ops.window_attn_decode(q[:, :, -2:].contiguous(), k, v, n, 300, 9)
    ops.device_status()
    assert torch.allclose(last, full[:, :, -2:], rtol=0, atol=2e-5)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
def test_backward_chains_on_two_streams_and_in_a_graph(D, dtype):
    # row terms, gradients in parts and their join: each launch starts while the one before it ends
    q, k, v, do = make(1, 8, 2, 1100, 1100, D, dtype, seed=D)
    out, lse = ops.window_attn_fwd(q, k, v, 150, 0, 130)

    def run():
        return ops.window_attn_bwd(q, k, v, out, do, lse, 150, 0, 130)

    want = run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(6):
        for st in streams:
            with torch.cuda.stream(st):
                got.append(run())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=streams[0]):
        first = run()
        second = run()
    for _ in range(3):
        for t in first + second:
            t.fill_(float("nan"))
        g.replay()
        got.append(run())  # behind the replay, on the current stream
        torch.cuda.synchronize()
        got += [[t.clone() for t in first], [t.clone() for t in second]]
    ops.device_status()
    assert all(torch.equal(a, b) for r in got for a, b in zip(r, want))


def test_decode_chains_on_two_streams_and_in_a_graph():
    # 40 heads of 20,000 keys: shares in a workspace and their join
    q = torch.randn(1, 40, 1, 128, device="cuda", dtype=torch.bfloat16)
    kc, vc = (torch.randn(1, 40, 20000, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    n = torch.tensor([19990], dtype=torch.int32, device="cuda")
    run = lambda: ops.window_attn_decode(q, kc, vc, n, 18000, 500)  # noqa: E731
    want = run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(10):
        for st in streams:
            with torch.cuda.stream(st):
                got.append(run())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=streams[1]):
        first, second = run(), run()
    g.replay()
    torch.cuda.synchronize()
    ops.device_status()
    assert all(torch.equal(a, want) for a in got + [first, second])
    check = ops.window_attn_fwd(q, kc[:, :, :19990].contiguous(), vc[:, :, :19990].contiguous(), 18000, 0, 500)[0]
    # two computations of one value in bf16: weights and output rounded in each, 2^-8 of a value at most
    assert float((check.double() - want.double()).norm() / want.double().norm()) <= 2.0 ** -7


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_offsets_past_32_bits(dtype):
    # 2^31 elements and more in every tensor: the last head against the same head alone
    H, N, D = 34, 500_000, 128
    torch.manual_seed(0)
    q, k, v, do = (torch.empty(1, H, N, D, device="cuda", dtype=dtype) for _ in range(4))
    for t in (q, k, v, do):
        for h in range(H):
            t[0, h].normal_()
    last = [t[:, -1:].clone() for t in (q, k, v, do)]
    mask = dict(left=40, right=3, sink=2)
    out, lse = ops.window_attn_fwd(q, k, v, **mask)
    one, one_lse = ops.window_attn_fwd(*last[:3], **mask)
    assert torch.equal(out[:, -1:], one) and torch.equal(lse[:, -1:], one_lse)
    n = torch.tensor([N - 7], dtype=torch.int32, device="cuda")
    assert torch.equal(ops.window_attn_decode(q[:, :, -1:].contiguous(), k, v, n, 300, 2)[:, -1:],
                       ops.window_attn_decode(last[0][:, :, -1:].contiguous(), last[1], last[2], n, 300, 2))
    got = ops.window_attn_bwd(q, k, v, out, do, lse, **mask)
    want = ops.window_attn_bwd(*last[:3], one, last[3], one_lse, **mask)
    ops.device_status()
    for a, b in zip(got, want):  # the sinks' rows are cut differently: the order of their sums is another
        assert torch.equal(a[:, -1:, 128:], b[:, :, 128:])
    del q, k, v, do, last, out, lse, got, want, one, a, b, t
    torch.cuda.empty_cache()
