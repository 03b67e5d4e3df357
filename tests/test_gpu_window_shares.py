"""Gradients of tiles in several chunks beside tiles in one, where the tiles that
are cut lie among others of their kind: few queries over a longer past, queries
that stand before every key, and windows that are one-sided."""
import pytest
import torch

from test_gpu_window_attn import check_backward, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,H,Hk,Nq,Nk,D,off,left,right,sink", [
    (1, 16, 1, 130, 3000, 64, 2870, 300, 0, 0),     # key tiles near the end alone
    (2, 16, 1, 130, 2000, 128, 1870, 300, 0, 140),  # and those with sinks
    (1, 12, 1, 100, 2500, 64, 1200, 200, 100, 0),   # key tiles in the middle
    (2, 2, 2, 1500, 700, 64, -1300, -1, 0, 0),      # the last queries alone see keys
    (1, 3, 3, 1400, 300, 128, -200, 80, 0, 5),      # query tiles in the middle and the sinks behind
    (1, 4, 2, 700, 700, 64, 0, 0, -1, 100),         # to the right alone
    (1, 8, 2, 900, 900, 128, 0, -1, 0, 0),          # causal
])
def test_backward(B, H, Hk, Nq, Nk, D, off, left, right, sink, dtype):
    q, k, v, do = make(B, H, Hk, Nq, Nk, D, dtype, seed=Nk + D)
    check_backward(q, k, v, do, off, left, right, sink)
