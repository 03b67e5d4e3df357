"""What the rotation table with a base in 64 bits refuses, without a GPU."""
import ctypes

import pytest

from dynamic_block_sparse_pool_b200 import _lib
from dynamic_block_sparse_pool_b200.build import build

FAKE = 0x10000  # never dereferenced: every call below fails validation first


@pytest.mark.parametrize("bad,what", [
    (dict(positions=0), "positions"), (dict(pairs=0), "pairs"), (dict(pairs=65), "pairs"),
    (dict(positions=1 << 28, pairs=64), "2^30"), (dict(theta=0.0), "theta"), (dict(theta=-1.0), "theta"),
    (dict(theta=float("inf")), "theta"), (dict(theta=float("nan")), "theta"), (dict(theta=None), "theta"),
    (dict(table=None), "null"), (dict(table=FAKE + 4), "aligned")])
def test_table_with_a_64_bit_base(bad, what):
    build()
    lib = _lib.lib()
    a = {**dict(positions=8, pairs=8, theta=1e4, table=FAKE), **bad}
    theta = None if a["theta"] is None else ctypes.byref(ctypes.c_double(a["theta"]))
    assert lib.dsa_rope_table_f64(a["positions"], a["pairs"], theta, a["table"], None) == _lib.DSA_ERR_INVALID_ARG
    assert what in lib.dsa_last_error().decode()
