"""Streams that start with a prompt of more tokens than the cached attention takes
in one call, against the whole forward.  Two computations of the same values,
each within the bound of the layer's tests against 64 bits (2^-7 of the
result's 2-norm in bf16, 2^-13 in fp32), so within twice that of each other."""
import pytest
import torch

from dynamic_block_sparse_pool_b200 import ops, window_layer

pytestmark = pytest.mark.gpu

LIMIT = {torch.bfloat16: 2.0 ** -6, torch.float32: 2.0 ** -12}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("steps", [(129, 1), (300, 1, 2), (3, 257, 40)])
@pytest.mark.parametrize("D", [64, 128])
def test_a_prompt_into_a_stream(steps, D, dtype):
    B, H, Hk, N = 2, 6, 2, sum(steps)
    g = torch.Generator().manual_seed(N)
    qkv = torch.randn(B, N, H + 2 * Hk, D, generator=g).to(dtype).cuda()
    wq, wk = ((1 + 0.2 * torch.randn(D, generator=g)).cuda() for _ in range(2))
    pos = torch.stack([torch.arange(N), 900 + torch.arange(N)])[..., None]
    plan = ops.RopePlan(pos, (D // 2,), theta=500000.0)
    m = window_layer.Mask(100, 0, 5)
    want, _ = window_layer.forward(qkv, H, wq, wk, plan, m)
    st = window_layer.Stream(B, H, Hk, N + 3, D, plan, m, wq, wk, dtype=dtype)
    got, at = [], 0
    for n in steps:
        got.append(st.step(qkv[:, at:at + n], pos[:, at:at + n]))
        at += n
        assert st.length == at and st.lens.tolist() == [at, at]
    with pytest.raises(ValueError, match="capacity"):
        st.step(qkv[:, :4], pos[:, :4])
    ops.device_status()
    assert st.length == N and st.lens.tolist() == [N, N]
    err = torch.cat(got, 2).double() - want.double()
    assert float(err.norm() / want.double().norm()) <= LIMIT[dtype]
