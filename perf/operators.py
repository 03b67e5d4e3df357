"""Measured cases of the per-head norm with rotation, the window attention and the 8-bit activation checkpoints.

Every case is one pass through one operator.  `run` computes it in elementary torch operations in 32 bits where `own` is
false, and calls the framework where it is true; `exact` computes it in 64 bits from the definition.

Definitions
  norm and rotation  r = 1 / sqrt(mean(x^2) + eps), n = x * r * w per (token, head) row of D values; pair m of the D/2
                     pairs, (2m, 2m+1) or (m, m + D/2), turns by pos[axis(m)] * theta^(-i/pairs(axis)), i the pair's
                     number within its axis; an axis position below 0 leaves its pairs as they are.  Token-major
                     [B, N, H, D] in, head-major [B, H, N, D] out.
  window attention   key u is visible to the query at position t = offset + i iff u <= t + right and
                     (u < sink or u >= t - left); a negative bound is no bound; softmax over the visible keys.
  8-bit rows         scale = amax / 127, code = round_half_even(x * (127 / amax)), each operation rounded to fp32;
                     the value held is code * scale.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # queries and keys of one video layer, read in place from the fused projection's output
        dict(name="rope_fwd_video", op="rope_fwd", B=1, N=75600, H=40, Hk=40, D=128, dtype="bf16", fused=True,
             grid=True, T=21, Y=45, X=80, prefix=0, halves=False, theta=10000.0, start=0),
        # one new token of each of 16 streams, far into their contexts
        dict(name="rope_fwd_token", op="rope_fwd", B=16, N=1, H=32, Hk=8, D=128, dtype="bf16", fused=False,
             grid=False, T=0, Y=0, X=0, prefix=0, halves=True, theta=500000.0, start=100000),
        # training, with a text prefix that is not rotated
        dict(name="rope_bwd_prefix", op="rope_bwd", B=1, N=17776, H=48, Hk=48, D=64, dtype="bf16", fused=True,
             grid=True, T=13, Y=30, X=45, prefix=226, halves=False, theta=10000.0, start=0),
        # training with 8-bit checkpoints: the forward that writes them and the backward that reads them
        dict(name="rope_step8_video", op="rope_step8", B=1, N=118800, H=24, Hk=24, D=128, dtype="bf16", fused=True,
             grid=True, T=33, Y=45, X=80, prefix=0, halves=False, theta=256.0, start=0),
        # a small odd fp32 activation kept in 8 bits and taken back
        dict(name="act8_small", op="act8", rows=6 * 1001, D=64, dtype="f32"),
        # one layer's values kept in 8 bits and taken back
        dict(name="act8_video", op="act8", rows=40 * 75600, D=128, dtype="bf16"),
        # causal window with four first tokens kept, shared heads
        dict(name="win_fwd_causal", op="win_fwd", B=2, H=32, Hk=8, Nq=8192, Nk=8192, D=128, dtype="bf16",
             left=2047, right=0, sink=4),
        # two frames to either side of every token of a long video
        dict(name="win_fwd_video", op="win_fwd", B=1, H=40, Hk=40, Nq=75600, Nk=75600, D=128, dtype="bf16",
             left=7200, right=7200, sink=0),
        # training with two frames to either side and the whole text prefix in sight
        dict(name="win_bwd_prefix", op="win_bwd", B=1, H=48, Hk=48, Nq=17776, Nk=17776, D=64, dtype="bf16",
             left=2700, right=2700, sink=226),
        # small, odd, fp32, shared heads
        dict(name="win_bwd_small", op="win_bwd", B=1, H=4, Hk=2, Nq=1003, Nk=1003, D=64, dtype="f32",
             left=255, right=0, sink=3),
        # serving: 32 streams of uneven lengths, one new token each, shared heads
        dict(name="decode_batch", op="decode", B=32, H=32, Hk=8, Nq=1, cap=16384, D=128, dtype="bf16",
             left=4095, sink=4),
        # one stream of frames: the first frame and the last eight stay in sight
        dict(name="decode_one", op="decode", B=1, H=40, Hk=40, Nq=1, cap=75600, D=128, dtype="bf16",
             left=28800, sink=3600),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope_fwd", "rope_bwd", "rope_step8", "act8", "win_fwd", "win_bwd", "decode"])
    D = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    Hk = rng.choice([1, 2, 3, 4, 6, 8])
    H = Hk * rng.choice([1, 1, 2, 4, 5, 8])
    B = rng.choice([1, 1, 2, 3])
    if op == "act8":
        return dict(op=op, rows=_log(rng, 1, 2_000_000), D=D, dtype=dtype)
    if op.startswith("rope"):
        if rng.random() < 0.5:
            T, Y, X, prefix = rng.randint(1, 21), rng.randint(1, 45), rng.randint(1, 45), rng.choice([0, 77, 226])
            return dict(op=op, B=1, N=T * Y * X + prefix, H=H, Hk=Hk, D=D, dtype=dtype, fused=rng.random() < 0.5,
                        grid=True, T=T, Y=Y, X=X, prefix=prefix, halves=False, theta=10000.0, start=0)
        return dict(op=op, B=B, N=_log(rng, 1, 30000), H=H, Hk=Hk, D=D, dtype=dtype, fused=rng.random() < 0.5,
                    grid=False, T=0, Y=0, X=0, prefix=0, halves=rng.random() < 0.7, theta=500000.0,
                    start=rng.randint(0, 100000))
    if op == "decode":
        cap = _log(rng, 16, 60000)
        return dict(op=op, B=rng.choice([1, 2, 3, 8, 17]), H=H, Hk=Hk, Nq=rng.choice([1, 1, 1, 2, 4]), cap=cap, D=D,
                    dtype=dtype, left=rng.choice([-1, _log(rng, 16, 20000)]), sink=rng.choice([0, 1, 4, 226]))
    Nq = _log(rng, 100, 12000 if dtype == "bf16" else 4000)
    back = 0 if rng.random() < 0.6 else rng.randint(0, 3000)
    return dict(op=op, B=B, H=H, Hk=Hk, Nq=Nq, Nk=Nq + back, D=D, dtype=dtype, left=_log(rng, 1, 4000),
                right=rng.choice([0, 0, _log(rng, 1, 3000)]), sink=rng.choice([0, 1, 4, 64, 226]))


# ----------------------------------------------------------------------------------------------------------- inputs

def _pairs(case):
    """Rotated pairs of each axis: three axes of a grid, or one axis of plain positions."""
    half = case["D"] // 2
    if not case["grid"]:
        return (half, 0, 0)
    other = half // 3
    return (half - 2 * other, other, other)


def _positions(case):
    """int32 [B or 1, N, 3] on the CPU."""
    B, N = case["B"], case["N"]
    if case["grid"]:
        T, Y, X, P = case["T"], case["Y"], case["X"], case["prefix"]
        t, y, x = torch.meshgrid(torch.arange(T), torch.arange(Y), torch.arange(X), indexing="ij")
        pos = torch.full((1, N, 3), -1, dtype=torch.int32)
        pos[0, P:] = torch.stack([t.reshape(-1), y.reshape(-1), x.reshape(-1)], 1).int()
        return pos
    # every stream of the batch stands somewhere else
    pos = torch.zeros(B, N, 3, dtype=torch.int32)
    pos[..., 0] = case["start"] + torch.arange(N)[None, :] + 37 * torch.arange(B)[:, None]
    return pos


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, shape, dtype, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16 if dtype == torch.bfloat16 else
                       torch.float32).mul_(scale).to(dtype)


def prepare(case, seed):
    g, dt, op, D = _gen(seed), DTYPES.get(case["dtype"]), case["op"], case["D"]
    s = dict(case=case)
    if op.startswith("rope"):
        B, N, H, Hk = case["B"], case["N"], case["H"], case["Hk"]
        if case["fused"]:  # the projection's own output, [B, N, heads of q | k | v, D]
            qkv = _randn(g, (B, N, H + 2 * Hk, D), dt, 1.5)
            s["xq"], s["xk"] = qkv[:, :, :H], qkv[:, :, H:H + Hk]
        else:
            s["xq"], s["xk"] = _randn(g, (B, N, H, D), dt, 1.5), _randn(g, (B, N, Hk, D), dt, 1.5)
        s["wq"] = 1.0 + 0.2 * _randn(g, (D,), torch.float32)
        s["wk"] = 1.0 + 0.2 * _randn(g, (D,), torch.float32)
        s["eps"] = 1e-6
        if op != "rope_fwd":
            s["dq"], s["dk"] = _randn(g, (B, H, N, D), dt), _randn(g, (B, Hk, N, D), dt)
        if own:
            from dynamic_block_sparse_pool_b200 import ops
            s["plan"] = ops.RopePlan(_positions(case), _pairs(case), theta=case["theta"], halves=case["halves"])
        else:
            c, sn = _angles(case)
            s["cos"], s["sin"] = c.float().cuda(), sn.float().cuda()
    elif op == "act8":
        s["x"] = _randn(g, (case["rows"], D), dt, 2.0)
    elif op == "decode":
        B, H, Hk, cap = case["B"], case["H"], case["Hk"], case["cap"]
        s["q"] = _randn(g, (B, H, case["Nq"], D), dt)
        s["k"], s["v"] = _randn(g, (B, Hk, cap, D), dt), _randn(g, (B, Hk, cap, D), dt)
        lens = torch.randint(max(1, cap // 2), cap + 1, (B,), generator=g, device="cuda")
        lens[0] = cap
        s["lens"] = lens.int()
    else:
        B, H, Hk, Nq, Nk = case["B"], case["H"], case["Hk"], case["Nq"], case["Nk"]
        s["q"] = _randn(g, (B, H, Nq, D), dt)
        s["k"], s["v"] = _randn(g, (B, Hk, Nk, D), dt), _randn(g, (B, Hk, Nk, D), dt)
        if op == "win_bwd":  # what the forward left behind
            s["out"], s["lse"] = _window_forward(s)
            s["dout"] = _randn(g, (B, H, Nq, D), dt)
    return s


# ------------------------------------------------------------------------------------------------------ plain forms

def _angles(case):
    """cos and sin [B or 1, N, 1, D/2] in 64 bits (1 and 0 where a pair does not turn)."""
    pos, out = _positions(case).double(), []
    for axis, n in enumerate(_pairs(case)):
        if n:
            f = float(case["theta"]) ** (-torch.arange(n, dtype=torch.float64) / n)
            out.append(pos[..., axis, None].clamp(min=0) * f)
    a = torch.cat(out, -1)[:, :, None, :]
    return torch.cos(a), torch.sin(a)


def _turn(x, cos, sin, halves, back=False):
    if back:
        sin = -sin
    if halves:
        a, b = x.chunk(2, -1)
        return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)


def _norm_turn(x, w, eps, cos, sin, halves):
    x = x.float()
    n = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w
    return _turn(n, cos, sin, halves).transpose(1, 2)


def _norm_turn_grad(dy, x, w, eps, cos, sin, halves):
    x = x.float()
    g = _turn(dy.float().transpose(1, 2), cos, sin, halves, back=True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)
    h = x * r
    gw = g * h
    dw = gw.flatten(0, 2).double().sum(0).float()
    return r * (g * w - h * (gw * w).mean(-1, keepdim=True)), dw


def _codes(x):
    x = x.float()
    amax = x.abs().amax(-1, keepdim=True)
    top = torch.full_like(amax, 127.0)  # a tensor: a plain number would be divided by through its rounded reciprocal
    inv = torch.where(amax > 0, top / amax, torch.zeros_like(amax))
    return torch.round(x * inv), amax / top


def _visible(t, u, c):
    ok = torch.ones(t.shape[0], u.shape[0], dtype=torch.bool, device=t.device)
    if c["right"] >= 0:
        ok &= u[None, :] <= t[:, None] + c["right"]
    if c["left"] >= 0:
        ok &= (u[None, :] < c["sink"]) | (u[None, :] >= t[:, None] - c["left"])
    return ok


def _spans(c, step):
    """Chunks of queries with the positions of the keys that any of them sees: (i0, i1, t, u)."""
    off = c["Nk"] - c["Nq"]
    for i0 in range(0, c["Nq"], step):
        i1 = min(c["Nq"], i0 + step)
        lo = 0 if c["left"] < 0 else max(0, off + i0 - c["left"])
        hi = c["Nk"] if c["right"] < 0 else max(0, min(c["Nk"], off + i1 + c["right"]))
        first = min(c["sink"], lo, hi)
        u = torch.cat([torch.arange(first, device="cuda"), torch.arange(min(lo, hi), hi, device="cuda")])
        yield i0, i1, off + torch.arange(i0, i1, device="cuda"), u, first, min(lo, hi), hi


def _step(c):
    width = c["Nk"] if c["left"] < 0 or c["right"] < 0 else min(c["Nk"], c["left"] + c["right"] + c["sink"] + 1024)
    return max(64, min(1024, int(6e8 / (c["H"] * width))))


def _keys(x, first, lo, hi):
    return torch.cat([x[:, :first], x[:, lo:hi]], 1) if first else x[:, lo:hi]


def _window_forward(s):
    c, q = s["case"], s["q"]
    H, Hk, D = c["H"], c["Hk"], c["D"]
    out = torch.empty_like(q)
    lse = torch.empty(q.shape[:3], device="cuda")
    for b in range(c["B"]):
        k, v = s["k"][b].float(), s["v"][b].float()
        for i0, i1, t, u, first, lo, hi in _spans(c, _step(c)):
            n = i1 - i0
            x = q[b, :, i0:i1].float().reshape(Hk, H // Hk * n, D)
            sc = (x @ _keys(k, first, lo, hi).transpose(1, 2)).view(Hk, H // Hk, n, -1) * D ** -0.5
            sc = sc.masked_fill_(~_visible(t, u, c), -math.inf)
            m = sc.amax(-1, keepdim=True).clamp_(min=-3e38)
            p = sc.sub_(m).exp_()
            l = p.sum(-1, keepdim=True)
            o = (p.view(Hk, H // Hk * n, -1) @ _keys(v, first, lo, hi)).view(Hk, H // Hk, n, D)
            out[b, :, i0:i1] = (o / l.clamp(min=1e-38)).reshape(H, n, D).to(out.dtype)
            lse[b, :, i0:i1] = torch.where(l > 0, m + l.log(), torch.full_like(l, -math.inf)).reshape(H, n)
    return out, lse


def _window_grads(s):
    c, q, k, v = s["case"], s["q"], s["k"], s["v"]
    H, Hk, D = c["H"], c["Hk"], c["D"]
    G, scale = H // Hk, D ** -0.5
    dq = torch.empty_like(q)
    dk, dv = torch.empty_like(k), torch.empty_like(v)
    for b in range(c["B"]):
        kb, vb = k[b].float(), v[b].float()
        ak, av = torch.zeros_like(kb), torch.zeros_like(vb)
        for i0, i1, t, u, first, lo, hi in _spans(c, _step(c)):
            n = i1 - i0
            x, do = (z[b, :, i0:i1].float().reshape(Hk, G * n, D) for z in (q, s["dout"]))
            delta = (do * s["out"][b, :, i0:i1].float().reshape(Hk, G * n, D)).sum(-1, keepdim=True)
            kk, vv = _keys(kb, first, lo, hi), _keys(vb, first, lo, hi)
            p = (x @ kk.transpose(1, 2)).mul_(scale).sub_(s["lse"][b, :, i0:i1].reshape(Hk, G * n, 1)).exp_()
            p = p.view(Hk, G, n, -1).masked_fill_(~_visible(t, u, c), 0.0).view(Hk, G * n, -1)
            ds = (do @ vv.transpose(1, 2)).sub_(delta).mul_(p)
            dq[b, :, i0:i1] = ((ds @ kk) * scale).view(H, n, D).to(dq.dtype)
            gk, gv = (ds.transpose(1, 2) @ x) * scale, p.transpose(1, 2) @ do
            for acc, grad in ((ak, gk), (av, gv)):
                acc[:, :first] += grad[:, :first]
                acc[:, lo:hi] += grad[:, first:]
        dk[b], dv[b] = ak.to(dk.dtype), av.to(dv.dtype)
    return dq, dk, dv


def _decode(s):
    c, q, k, v = s["case"], s["q"], s["k"], s["v"]
    B, H, Hk, Nq, cap, D = c["B"], c["H"], c["Hk"], c["Nq"], c["cap"], c["D"]
    out = torch.empty_like(q)
    u = torch.arange(cap, device="cuda")
    for b in range(B):
        t = s["lens"][b].long() - Nq + torch.arange(Nq, device="cuda")
        x = q[b].float().reshape(Hk, H // Hk * Nq, D)
        sc = (x @ k[b].float().transpose(1, 2)).view(Hk, H // Hk, Nq, cap) * D ** -0.5
        sc = sc.masked_fill_(~_visible(t, u, {**c, "right": 0}), -math.inf)
        p = torch.exp(sc - sc.amax(-1, keepdim=True).clamp(min=-3e38))
        p = p / p.sum(-1, keepdim=True).clamp(min=1e-38)
        out[b] = (p.view(Hk, H // Hk * Nq, cap) @ v[b].float()).view(H, Nq, D).to(out.dtype)
    return out


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        from dynamic_block_sparse_pool_b200 import ops
        if op == "rope_fwd":
            return ops.qk_norm_rope(s["xq"], s["xk"], s["wq"], s["wk"], s["plan"], s["eps"])
        if op == "rope_bwd":
            return ops.qk_norm_rope_bwd(s["dq"], s["dk"], s["xq"], s["xk"], s["wq"], s["wk"], s["plan"], s["eps"])
        if op == "rope_step8":
            q, k, q8, k8 = ops.qk_norm_rope(s["xq"], s["xk"], s["wq"], s["wk"], s["plan"], s["eps"], save8=True)
            return (q, k) + tuple(ops.qk_norm_rope_bwd(s["dq"], s["dk"], q8, k8, s["wq"], s["wk"], s["plan"],
                                                       s["eps"]))
        if op == "act8":
            return ops.unpack8(ops.pack8(s["x"]), s["x"].dtype)
        if op == "decode":
            return ops.window_attn_decode(s["q"], s["k"], s["v"], s["lens"], left=c["left"], sink=c["sink"])
        w = dict(left=c["left"], right=c["right"], sink=c["sink"])
        if op == "win_fwd":
            return ops.window_attn_fwd(s["q"], s["k"], s["v"], **w)
        return ops.window_attn_bwd(s["q"], s["k"], s["v"], s["out"], s["dout"], s["lse"], **w)
    if op == "act8":
        code, scale = _codes(s["x"])
        return (code * scale).to(s["x"].dtype)
    if op == "decode":
        return _decode(s)
    if op == "win_fwd":
        return _window_forward(s)
    if op == "win_bwd":
        return _window_grads(s)
    dt, halves, a = s["xq"].dtype, c["halves"], (s["eps"], s["cos"], s["sin"])
    res = []
    if op != "rope_bwd":
        res += [_norm_turn(s["xq"], s["wq"], *a, halves).to(dt).contiguous(),
                _norm_turn(s["xk"], s["wk"], *a, halves).to(dt).contiguous()]
    if op != "rope_fwd":
        xq, xk = s["xq"], s["xk"]
        if op == "rope_step8":
            xq, xk = (code * scale for code, scale in (_codes(xq), _codes(xk)))
        dxq, dwq = _norm_turn_grad(s["dq"], xq, s["wq"], *a, halves)
        dxk, dwk = _norm_turn_grad(s["dk"], xk, s["wk"], *a, halves)
        res += [dxq.to(dt), dxk.to(dt), dwq, dwk]
    return tuple(res)


# ---------------------------------------------------------------------------------------------------- exact outputs

def _exact_rope(case, s):
    """From complex rotation and the norm's Jacobian, in 64 bits, a few heads at a time."""
    z = torch.polar(torch.ones((), dtype=torch.float64), _exact_angles(case)).cuda()

    def pairs(x):
        if case["halves"]:
            return torch.complex(*x.tensor_split(2, -1))
        return torch.view_as_complex(x.reshape(*x.shape[:-1], -1, 2).contiguous())

    def flat(y):
        if case["halves"]:
            return torch.cat([y.real, y.imag], -1)
        return torch.view_as_real(y).reshape(*y.shape[:-1], -1)

    fwd, dxs, dws = [], [], []
    for x, w, dy in ((s["xq"], s["wq"], s.get("dq")), (s["xk"], s["wk"], s.get("dk"))):
        y, dx, dw = [], [], 0
        for h in range(0, x.shape[2], 4):
            a = x[:, :, h:h + 4].double()
            norm = (a.pow(2).sum(-1, keepdim=True) / case["D"] + s["eps"]).sqrt()
            if case["op"] != "rope_bwd":
                y.append(flat(pairs(a / norm * w.double()) * z).permute(0, 2, 1, 3))
            if case["op"] != "rope_fwd":
                if case["op"] == "rope_step8":  # the codes are defined in fp32 arithmetic
                    top = x[:, :, h:h + 4].float().abs().max(-1, keepdim=True).values
                    full = torch.full_like(top, 127.0)
                    mul = (full / top).nan_to_num(posinf=0.0)
                    a = (x[:, :, h:h + 4].float() * mul).round().double() * (top / full).double()
                    norm = (a.pow(2).sum(-1, keepdim=True) / case["D"] + s["eps"]).sqrt()
                g = flat(pairs(dy[:, h:h + 4].double().permute(0, 2, 1, 3)) * z.conj())
                dw = dw + torch.einsum("bnhd,bnhd->d", g, a / norm)
                gw = g * w.double()
                dx.append(gw / norm - a * (gw * a).sum(-1, keepdim=True) / (case["D"] * norm.pow(3)))
        if y:
            fwd.append(torch.cat(y, 1))
        if dx:
            dxs.append(torch.cat(dx, 2))
            dws.append(dw)
    return tuple(fwd + dxs + dws)


def _exact_angles(case):
    pos = _positions(case)
    cols = []
    for axis, n in enumerate(_pairs(case)):
        for i in range(n):
            p = pos[..., axis].double()
            cols.append(torch.where(p < 0, torch.zeros_like(p), p) * math.pow(case["theta"], -i / n))
    return torch.stack(cols, -1)[:, :, None, :]


def _exact_rows(case, s, b, h, i0, i1, cache_len=None):
    """Scores (64 bits, -inf where hidden) of queries i0..i1 of one head against keys a..z, and those bounds."""
    kv = h * case["Hk"] // case["H"]
    n = cache_len if cache_len is not None else case["Nk"]
    first = n - case["Nq"]
    i = torch.arange(i0, i1, device="cuda") + first
    right = case.get("right", 0)
    a = 0 if case["left"] < 0 or case["sink"] > 0 else max(0, first + i0 - case["left"])
    z = n if right < 0 else min(n, max(a, first + i1 + right))
    j = torch.arange(a, z, device="cuda")
    hidden = torch.zeros(i1 - i0, z - a, dtype=torch.bool, device="cuda")
    if right >= 0:
        hidden |= (j - right)[None] > i[:, None]
    if case["left"] >= 0:
        hidden |= ((j + case["left"])[None] < i[:, None]) & (j >= case["sink"])[None]
    sc = torch.einsum("id,jd->ij", s["q"][b, h, i0:i1].double(), s["k"][b, kv, a:z].double()) / math.sqrt(case["D"])
    return sc.masked_fill(hidden, -math.inf), kv, a, z


def exact(case, seed):
    s = prepare(case, seed)
    op, D = case["op"], case["D"]
    if op == "act8":
        out = []
        for x in s["x"].split(1 << 20):
            top = x.float().abs().max(-1, keepdim=True).values
            full = torch.full_like(top, 127.0)
            mul = (full / top).nan_to_num(posinf=0.0)
            out.append((x.float() * mul).round().double() * (top / full).double())
        return torch.cat(out)
    if op.startswith("rope"):
        return _exact_rope(case, s)
    B, H, Nq = case["B"], case["H"], case["Nq"]
    if op == "decode":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        for b, n in enumerate(s["lens"].tolist()):
            for h in range(H):
                sc, kv, a, z = _exact_rows(case, s, b, h, 0, Nq, n)
                out[b, h] = torch.softmax(sc, -1).nan_to_num(0.0) @ s["v"][b, kv, a:z].double()
        return out
    width = case["Nk"] if min(case["left"], case["right"]) < 0 or case["sink"] else \
        min(case["Nk"], case["left"] + case["right"] + 4096)
    if 4.0 * B * H * Nq * width * D * (1.0 if op == "win_fwd" else 2.5) > 6e13:
        return None  # too long in 64 bits
    if op == "win_fwd":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.zeros(s["q"].shape[:3], dtype=torch.float64, device="cuda")
        for b in range(B):
            for h in range(H):
                for i0 in range(0, Nq, 4096):
                    i1 = min(Nq, i0 + 4096)
                    sc, kv, a, z = _exact_rows(case, s, b, h, i0, i1)
                    lse[b, h, i0:i1] = torch.logsumexp(sc, -1)
                    out[b, h, i0:i1] = torch.softmax(sc, -1).nan_to_num(0.0) @ s["v"][b, kv, a:z].double()
        return out, lse
    grads = [torch.zeros(s[n].shape, dtype=torch.float64, device="cuda") for n in "qkv"]
    for b in range(B):
        for h in range(H):
            for i0 in range(0, Nq, 4096):
                i1 = min(Nq, i0 + 4096)
                sc, kv, a, z = _exact_rows(case, s, b, h, i0, i1)
                do, key = s["dout"][b, h, i0:i1].double(), s["k"][b, kv, a:z].double()
                p = torch.exp(sc - s["lse"][b, h, i0:i1].double()[:, None])
                gp = torch.einsum("id,jd->ij", do, s["v"][b, kv, a:z].double())
                ds = p * (gp - torch.einsum("id,id->i", do, s["out"][b, h, i0:i1].double())[:, None]) / math.sqrt(D)
                grads[0][b, h, i0:i1] = torch.einsum("ij,jd->id", ds, key)
                grads[1][b, kv, a:z] += torch.einsum("ij,id->jd", ds, s["q"][b, h, i0:i1].double())
                grads[2][b, kv, a:z] += torch.einsum("ij,id->jd", p, do)
    return tuple(grads)


# ------------------------------------------------------------------------------------------------------------- work

def _seen(first, Nq, Nk, left, right, sink):
    """Visible (query, key) pairs of one head, and the number of keys that any query sees."""
    t = first + torch.arange(Nq, dtype=torch.int64)
    hi = torch.full_like(t, Nk) if right < 0 else (t + right + 1).clamp(0, Nk)
    lo = torch.zeros_like(t) if left < 0 else (t - left).clamp(min=0)
    lo = torch.minimum(lo, hi)
    pairs = int((hi - lo + torch.minimum(lo, torch.full_like(lo, sink))).sum())
    return pairs, int(hi.max() - lo.min() + min(sink, int(lo.min())))


def work(case):
    op, D = case["op"], case["D"]
    e = 2 if case["dtype"] == "bf16" else 4
    if op == "act8":  # to 8 bits and back: x in, codes and scales out and in, x out
        n = case["rows"] * D
        return dict(bytes=2 * n * e + 2 * n + 8 * case["rows"], flops=5 * n)
    if op.startswith("rope"):
        rows = case["B"] * case["N"] * (case["H"] + case["Hk"])
        n, pos = rows * D, 12 * case["N"] * (1 if case["grid"] else case["B"])
        fwd, bwd = dict(bytes=2 * n * e + pos + 8 * D, flops=8 * n), dict(bytes=3 * n * e + pos + 16 * D, flops=14 * n)
        if op == "rope_fwd":
            return fwd
        if op == "rope_bwd":
            return bwd
        return dict(bytes=fwd["bytes"] + n + 4 * rows + bwd["bytes"] - n * e + n + 4 * rows, flops=24 * n)
    B, H, Hk, Nq = case["B"], case["H"], case["Hk"], case["Nq"]
    if op == "decode":
        # lengths are drawn between half the capacity and all of it
        n = max(1, case["cap"] * 3 // 4) if B > 1 else case["cap"]
        pairs, keys = _seen(n - Nq, Nq, n, case["left"], 0, case["sink"])
        return dict(bytes=e * B * D * (2 * H * Nq + 2 * Hk * keys) + 4 * B, flops=4 * D * B * H * pairs)
    pairs, keys = _seen(case["Nk"] - Nq, Nq, case["Nk"], case["left"], case["right"], case["sink"])
    if op == "win_fwd":
        return dict(bytes=e * B * D * (2 * H * Nq + 2 * Hk * keys) + 4 * B * H * Nq, flops=4 * D * B * H * pairs)
    return dict(bytes=e * B * D * (4 * H * Nq + 2 * Hk * keys + 2 * Hk * case["Nk"]) + 4 * B * H * Nq,
                flops=10 * D * B * H * pairs)
