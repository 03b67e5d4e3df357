"""The cached form with more rows of a key head than one grid dimension has
places: 1,024 query heads on one, 128 new tokens, two rows (fp32, D = 128) to a
tile.  A few heads are checked against the dense form in 64 bits."""
import pytest
import torch

from dynamic_block_sparse_pool_b200 import ops
from test_gpu_window_attn import check_forward, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,H,Hk,Nq,D,dtype", [(1, 1024, 1, 128, 128, torch.float32), (2, 2048, 2, 128, 128, torch.float32),
                                               (1, 8192, 1, 128, 64, torch.bfloat16)])
def test_many_row_tiles(B, H, Hk, Nq, D, dtype):
    cap, left, sink = 150, 40, 3
    _, k, v, _ = make(B, Hk, Hk, 1, cap, D, dtype, seed=H)
    q = torch.randn(B, H, Nq, D, device="cuda", generator=torch.Generator("cuda").manual_seed(H)).to(dtype)
    n = torch.tensor([cap, cap - 13][:B], dtype=torch.int32, device="cuda")
    lse = torch.empty(B, H, Nq, device="cuda")
    out = ops.window_attn_decode(q, k, v, n, left, sink, lse=lse)
    ops.device_status()
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    for b, ln in enumerate(n.tolist()):
        for h in (0, 1, H // 2 - 1, H // 2, H - 1):
            kv = h // (H // Hk)
            one, key = (slice(b, b + 1), slice(h, h + 1)), (slice(b, b + 1), slice(kv, kv + 1), slice(0, ln))
            check_forward(q[one], k[key], v[key], ln - Nq, left, 0, sink, got=(out[one], lse[one]))
