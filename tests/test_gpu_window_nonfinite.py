"""NaN and infinities in visible places of the window attention: they come out
wherever the softmax over the visible keys would show them, and nowhere that
does not see them.  A gradient may carry them to every row of the tiles (128
rows) that load the row, as a product with a hidden 0 does."""
import math

import pytest
import torch

from dynamic_block_sparse_pool_b200 import ops
from test_gpu_window_attn import make, visible

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
BOTH = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
N, MASK = 700, (90, 20, 3)


def clean(D, dtype, H=4, Hk=2):
    q, k, v, do = make(1, H, Hk, N, N, D, dtype, seed=D)
    k[..., 0] = k[..., 0].abs() + 1  # an infinity there gives scores of +infinity
    q[..., 0] = q[..., 0].abs() + 1
    return q, k, v, do


def gone(t):
    return torch.isnan(t).all(-1).cpu(), torch.isfinite(t).all(-1).cpu()


@BOTH
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("where,value", [("q", NAN), ("k", NAN), ("k", INF), ("v", NAN)])
def test_forward_and_gradients(where, value, D, dtype):
    q, k, v, do = clean(D, dtype)
    ok = visible(N, N, 0, *MASK)
    want_o, want_l = ops.window_attn_fwd(q, k, v, *MASK)
    at, head = 301, 1                                # query head 3 and key head 1
    {"q": q, "k": k, "v": v}[where][0, 3 if where == "q" else head, at, 0] = value
    rows = torch.zeros(N, dtype=torch.bool)          # queries that meet it
    if where == "q":
        rows[at] = True
    else:
        rows = ok[:, at]
    heads = [3] if where == "q" else [2, 3]
    out, lse = ops.window_attn_fwd(q, k, v, *MASK)
    grads = ops.window_attn_bwd(q, k, v, out, do, lse, *MASK)
    ops.device_status()
    for h in range(4):
        if h not in heads:
            assert torch.equal(out[0, h], want_o[0, h]) and torch.equal(lse[0, h], want_l[0, h])
            assert torch.isfinite(grads[0][0, h]).all()
            continue
        if where == "v":                             # one column, and the tiles that load the row
            assert torch.isnan(out[0, h, rows, 0].cpu()).all() and torch.equal(lse[0, h], want_l[0, h])
            assert torch.equal(out[0, h, :, 1:], want_o[0, h, :, 1:])
        else:
            assert torch.isnan(out[0, h, rows].float()).all() and torch.isnan(lse[0, h, rows]).all()
            assert torch.equal(out[0, h, ~rows], want_o[0, h, ~rows]) and torch.equal(lse[0, h, ~rows], want_l[0, h, ~rows])
        all_nan, finite = gone(grads[0][0, h])
        assert all_nan[rows].all(), "dq of the rows that meet it"
        # (a row of k or v reaches every query of the tiles that load it)
        reach = rows if where == "q" else visible_tiles(ok)[:, at // 128].repeat_interleave(128)[:N]
        assert finite[~reach].all(), "dq of the others"
    keys = ok[rows].any(0)                           # keys that those queries see
    near = (visible_tiles(ok)[tiles(rows)]).any(0).repeat_interleave(128)[:N]  # and the tiles they load
    if where == "v":
        near = visible_tiles(ok)[visible_tiles(ok)[:, at // 128]].any(0).repeat_interleave(128)[:N]
    for g, what in ((grads[1], "dk"), (grads[2], "dv")):
        assert torch.isfinite(g[0, 0]).all(), what
        all_nan, finite = gone(g[0, 1])
        assert finite[~near].all(), what
        if what == "dk" or where != "v":
            assert all_nan[keys].all(), what
        else:
            assert finite.all(), what                # dv = P^T dO does not meet v


def tiles(rows):
    return torch.stack([rows[i:i + 128].any() for i in range(0, len(rows), 128)])


def visible_tiles(ok):
    n = math.ceil(ok.shape[0] / 128)
    return torch.stack([torch.stack([ok[128 * i:128 * i + 128, 128 * j:128 * j + 128].any() for j in range(n)])
                        for i in range(n)])
