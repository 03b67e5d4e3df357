"""How the window attention's work is cut, on the host: the plans of the library
themselves, at sizes whose tensors no test could hold, and the workspaces that
follow from them."""
import ctypes

import pytest

from dynamic_block_sparse_pool_b200 import _lib
from dynamic_block_sparse_pool_b200.build import build

NO_BOUND = 1 << 29


class Window(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("Nq", "Nk", "off", "left", "right", "sink")]


class BwdChunks(ctypes.Structure):
    _fields_ = [("heads", ctypes.c_int), ("sink_tiles", ctypes.c_int), ("chunks", ctypes.c_int * 2),
                ("counts", ctypes.c_int * 2)]


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.lib()


def bwd_chunks(lib, B, H, Hk, N, left=NO_BOUND, right=NO_BOUND, sink=0):
    f = lib._ZN3dsa10bwd_chunksEiiiRKNS_6WindowE  # dsa::bwd_chunks(int, int, int, const Window&)
    f.restype = BwdChunks
    f.argtypes = [ctypes.c_int] * 3 + [ctypes.POINTER(Window)]
    return f(B, H, Hk, Window(N, N, 0, left, right, sink))


def longest(N, tile, left, right, sink):
    """Query tiles that the key tile sees (square, no offset)."""
    k0, k1 = 128 * tile, min(N, 128 * tile + 128)
    a = max(0, k0 - right)
    b = N if k0 < sink else min(N, k1 + left)
    return max(0, -(-b // 128) - a // 128) if b > a else 0


@pytest.mark.parametrize("B,H,Hk,N,left,right,sink", [
    (1, 1, 1, 73_000_000, NO_BOUND, NO_BOUND, 0),   # 2.2e9 pairs of tiles for each SM
    (1, 1, 1, 1 << 27, NO_BOUND, NO_BOUND, 0),
    (1, 2, 1, 1 << 27, NO_BOUND, 0, 0),
    (3, 16, 4, 1 << 24, NO_BOUND, NO_BOUND, 64),
    (1, 1, 1, 1 << 27, 1000, 0, 4),                 # the tile of the sinks is cut
    (1, 8, 2, 8192, 2047, 0, 4),
    (2, 4, 4, 1003, 255, 0, 3),
])
def test_every_pair_of_tiles_is_in_a_part(lib, B, H, Hk, N, left, right, sink):
    c = bwd_chunks(lib, B, H, Hk, N, left, right, sink)
    tiles, group = -(-N // 128), H // Hk
    assert c.heads == B * Hk and c.sink_tiles == -(-sink // 128)
    picks = {0, 1, tiles // 2, tiles - 1, c.sink_tiles, max(0, c.sink_tiles - 1)}
    for t in (x for x in picks if x < tiles):
        kind = int(t >= c.sink_tiles)
        assert c.chunks[kind] >= 1 and c.counts[kind] >= 1
        assert c.chunks[kind] * c.counts[kind] >= longest(N, t, left, right, sink) * group


# tokens and heads whose share of tile pairs for each SM is small in its low 32 bits
WRAPS = [(102_058_880, 1), (124_990_336, 2), (131_750_144, 3)]


def test_share_beyond_32_bits_asks_for_no_parts(lib):
    # every key tile sees every query: the tiles are alike, and far more than there are SMs
    size = lib.dsa_window_attn_bwd_workspace_size
    for N, heads in WRAPS:
        share = (-(-N // 128)) ** 2 * heads // 148
        assert share >= 1 << 31 and share % (1 << 32) < 600_000   # small once cut to 32 bits
        assert size(1, 1, heads, heads, N, N, 64, 0, -1, -1, 0) == -(-4 * heads * N // 16) * 16

