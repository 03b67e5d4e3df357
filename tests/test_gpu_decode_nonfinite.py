"""NaN and infinities in visible places of the cached window attention: they come
out of every query that sees them, whichever way the keys are shared among
warps and CTAs, and nowhere else."""
import pytest
import torch

from dynamic_block_sparse_pool_b200 import ops
from test_gpu_window_attn import make

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
BOTH = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])


# caches whose keys one CTA, a cluster, and several CTAs through the workspace share
@BOTH
@pytest.mark.parametrize("B,H,Hk,Nq,cap,D", [(40, 8, 4, 1, 300, 64), (2, 4, 2, 1, 3000, 128), (1, 4, 2, 3, 40000, 64),
                                             (1, 2, 1, 1, 200000, 128), (3, 4, 2, 2, 9, 128)])
@pytest.mark.parametrize("where,value", [("q", NAN), ("k", NAN), ("k", INF), ("v", NAN)])
def test_cached(where, value, B, H, Hk, Nq, cap, D, dtype):
    q, k, v, _ = make(B, H, Hk, Nq, cap, D, dtype, seed=cap)
    q[..., 0] = q[..., 0].abs() + 1
    n = torch.full((B,), cap - 1, dtype=torch.int32, device="cuda")
    run = lambda: (lambda l: (ops.window_attn_decode(q, k, v, n, lse=l), l))(torch.zeros(B, H, Nq, device="cuda"))  # noqa: E731
    want, want_l = run()
    G = H // Hk
    at = cap // 2 if cap > 20 else 2                 # a key that every new token sees
    if where == "q":
        q[-1, H - 1, 0, 0] = value
    else:
        (k if where == "k" else v)[-1, Hk - 1, at, 0] = value
    out, lse = run()
    ops.device_status()
    hit = torch.zeros(B, H, Nq, dtype=torch.bool, device="cuda")
    if where == "q":
        hit[-1, H - 1, 0] = True
    else:
        hit[-1, H - G:] = True
    assert torch.equal(out[~hit], want[~hit]) and torch.equal(lse[~hit], want_l[~hit])
    if where == "v":
        assert torch.isnan(out[hit][:, 0]).all() and torch.equal(out[hit][:, 1:], want[hit][:, 1:])
        assert torch.equal(lse, want_l)
    else:
        assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()


@BOTH
def test_cached_queries_without_keys_beside_a_nan(dtype):
    # the second stream holds one token: its two first queries see nothing, whatever they hold
    q, k, v, _ = make(2, 2, 1, 3, 64, 64, dtype, seed=4)
    q[1, :, :2] = NAN
    n = torch.tensor([64, 1], dtype=torch.int32, device="cuda")
    lse = torch.zeros(2, 2, 3, device="cuda")
    out = ops.window_attn_decode(q, k, v, n, lse=lse)
    ops.device_status()
    assert torch.all(out[1, :, :2] == 0) and torch.all(lse[1, :, :2] == -INF)
    assert torch.isfinite(out).all() and torch.isfinite(lse[0]).all() and torch.isfinite(lse[1, :, 2]).all()
