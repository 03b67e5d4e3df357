"""The window backward's workspace holds shares of the gradient tiles that several
CTAs work on, and of no others: an SM's chunk of the work (a third of its share
of all tile pairs in fp32, 444 chunks in all) is the least a share stands for,
and a tile's last share may stand for less, so twice 444 shares of each gradient
and a few for the tiles that are not even bound what is needed, whatever the
number of tokens."""
import pytest

from dynamic_block_sparse_pool_b200 import _lib
from dynamic_block_sparse_pool_b200.build import build


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.lib()


def shares(lib, dt, B, H, Hk, Nq, Nk, D, off, left, right, sink):
    n = lib.dsa_window_attn_bwd_workspace_size(dt, B, H, Hk, Nq, Nk, D, off, left, right, sink)
    assert n >= 4 * B * H * Nq
    return n - (4 * B * H * Nq + 15) // 16 * 16


# B, H, Hk, Nq, Nk, D, off, left, right, sink
SHAPES = [
    (1, 1, 1, 100_000, 100_000, 128, 0, 1000, 0, 4),
    (1, 32, 8, 75_600, 75_600, 128, 0, 1023, 0, 4),
    (1, 8, 8, 1_000_000, 1_000_000, 128, 0, 1000, 0, 4),
    (1, 64, 1, 128, 1 << 20, 128, (1 << 20) - 128, 1000, 0, 0),   # few queries over a long past
    (1, 64, 1, 200, 1 << 20, 64, (1 << 20) - 200, 300, 0, 300),
    (2, 2, 2, 1_000_000, 1000, 64, -999_000, 200, 0, 0),          # most queries stand before every key
    (1, 1, 1, 500_000, 500_000, 128, 0, -1, 0, 0),
    (1, 16, 2, 20_000, 20_000, 64, 0, 0, -1, 100),
]


@pytest.mark.parametrize("shape", SHAPES)
def test_fp32_shares_are_those_of_the_tiles_in_chunks(lib, shape):
    D = shape[5]
    assert shares(lib, 0, *shape) <= 3 * 2 * 444 * 64 * D * 4


@pytest.mark.parametrize("shape", SHAPES)
def test_bf16_shares_are_those_of_the_tiles_in_parts(lib, shape):
    # parts of at least eight pairs and at least an SM's share (148 in all), two gradients of 128 rows
    D = shape[5]
    assert shares(lib, 1, *shape) <= 3 * 148 * 2 * 128 * D * 4
