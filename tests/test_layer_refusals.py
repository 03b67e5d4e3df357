"""What the calls around the attention refuse, without a GPU: every bad argument
returns DSA_ERR_INVALID_ARG with its reason before the device is touched, the
workspace sizes are those of the shapes, and the Python layer checks shapes,
types and devices."""
import ctypes

import pytest
import torch

from dynamic_block_sparse_pool_b200 import _lib, ops, window_layer
from dynamic_block_sparse_pool_b200.build import build

FAKE = 0x10000  # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.lib()


def i64(*v):
    return (ctypes.c_int64 * len(v))(*v)


def i32(*v):
    return (ctypes.c_int32 * len(v))(*v)


def refused(lib, call, what):
    assert call() == _lib.DSA_ERR_INVALID_ARG
    assert what.lower() in lib.dsa_last_error().decode().lower(), lib.dsa_last_error()


ROPE = dict(xq=FAKE, xk=FAKE, xq_scale=None, xk_scale=None, x_strides=(4096, 512, 64, 4096, 512, 64), dt=1, B=2, N=8,
            Hq=4, Hk=2, D=64, wq=FAKE, wk=FAKE, eps=1e-6, table=FAKE, pos=FAKE, per_batch=0, axes=(12, 10, 10, 8, 8, 8),
            halves=0)
BAD_ROPE = [
    (dict(xq=None), "null"), (dict(table=None), "null"), (dict(pos=None), "null"), (dict(dt=2), "dtype"),
    (dict(xq_scale=FAKE), "both"), (dict(B=0), "B and N"), (dict(N=0), "B and N"), (dict(B=1 << 16, N=1 << 16), "B*N"),
    (dict(Hq=0), "Hq"), (dict(Hk=70000), "Hq"), (dict(D=96), "D must"), (dict(eps=-1.0), "eps"),
    (dict(eps=float("nan")), "eps"), (dict(per_batch=2), "0 or 1"), (dict(halves=3), "0 or 1"),
    (dict(axes=(20, 10, 10, 8, 8, 8)), "exceed"), (dict(axes=(-1, 10, 10, 8, 8, 8)), "axis 0"),
    (dict(axes=(12, 10, 10, 8, 0, 8)), "axis 1"), (dict(axes=(32, 0, 0, 1 << 26, 0, 0)), "2^30"),
    (dict(xq=FAKE + 8), "misaligned"), (dict(table=FAKE + 4), "misaligned"),
    (dict(x_strides=(4096, 512, 60, 4096, 512, 64)), "strides"), (dict(x_strides=(4096, 512, 64, -8, 512, 64)), "strides"),
]


def rope_args(a):
    return (a["xq"], a["xk"], a["xq_scale"], a["xk_scale"], i64(*a["x_strides"]), a["dt"], a["B"], a["N"], a["Hq"],
            a["Hk"], a["D"], a["wq"], a["wk"], a["eps"], a["table"], a["pos"], a["per_batch"], i32(*a["axes"]),
            a["halves"])


@pytest.mark.parametrize("bad,what", BAD_ROPE)
def test_norm_rope_refuses(lib, bad, what):
    args = rope_args({**ROPE, **bad})
    refused(lib, lambda: lib.dsa_qk_norm_rope(*args, FAKE, FAKE, None, None, None, None, None), what)
    refused(lib, lambda: lib.dsa_qk_norm_rope_bwd(FAKE, FAKE, *args, FAKE, FAKE, i64(*ROPE["x_strides"]), FAKE, FAKE,
                                                  FAKE, 1 << 30, None), what)


def test_norm_rope_outputs_and_workspace(lib):
    args = rope_args(ROPE)
    refused(lib, lambda: lib.dsa_qk_norm_rope(*args, None, FAKE, None, None, None, None, None), "null q or k")
    refused(lib, lambda: lib.dsa_qk_norm_rope(*args, FAKE + 4, FAKE, None, None, None, None, None), "aligned")
    refused(lib, lambda: lib.dsa_qk_norm_rope(*args, FAKE, FAKE, FAKE, None, None, None, None), "all be")
    refused(lib, lambda: lib.dsa_qk_norm_rope(*args, FAKE, FAKE, FAKE + 4, FAKE, FAKE, FAKE, None), "aligned")
    from8 = rope_args({**ROPE, "xq_scale": FAKE, "xk_scale": FAKE})
    refused(lib, lambda: lib.dsa_qk_norm_rope(*from8, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None), "already")
    need = lib.dsa_qk_norm_rope_bwd_workspace_size(64)
    assert need > 0 and lib.dsa_qk_norm_rope_bwd_workspace_size(128) == 2 * need
    assert lib.dsa_qk_norm_rope_bwd_workspace_size(96) == 0
    st = i64(*ROPE["x_strides"])

    def bwd(dx=FAKE, strides=st, ws=FAKE, n=need):
        return lib.dsa_qk_norm_rope_bwd(FAKE, FAKE, *args, dx, FAKE, strides, FAKE, FAKE, ws, n, None)

    refused(lib, lambda: bwd(n=need - 1), "workspace")
    refused(lib, lambda: bwd(ws=None), "null")
    refused(lib, lambda: bwd(dx=FAKE + 2), "aligned")
    refused(lib, lambda: bwd(strides=i64(1, 512, 64, 4096, 512, 64)), "dx_strides")


@pytest.mark.parametrize("bad,what", [((0, 8, 1e4, FAKE), "positions"), ((8, 0, 1e4, FAKE), "pairs"),
                                      ((8, 65, 1e4, FAKE), "pairs"), ((1 << 28, 64, 1e4, FAKE), "2^30"),
                                      ((8, 8, 0.0, FAKE), "theta"), ((8, 8, float("inf"), FAKE), "theta"),
                                      ((8, 8, 1e4, None), "null"), ((8, 8, 1e4, FAKE + 4), "aligned")])
def test_rope_table_refuses(lib, bad, what):
    refused(lib, lambda: lib.dsa_rope_table(*bad, None), what)


@pytest.mark.parametrize("bad,what", [(dict(x=None), "null"), (dict(dt=7), "dtype"), (dict(rows=0), "rows"),
                                      (dict(rows=(1 << 36) + 1), "rows"), (dict(D=32), "D must"),
                                      (dict(x=FAKE + 8), "aligned"), (dict(codes=FAKE + 4), "aligned"),
                                      (dict(scales=FAKE + 2), "aligned")])
def test_rows8_refuse(lib, bad, what):
    a = {**dict(x=FAKE, dt=1, rows=4, D=64, codes=FAKE, scales=FAKE), **bad}
    refused(lib, lambda: lib.dsa_pack8(a["x"], a["dt"], a["rows"], a["D"], a["codes"], a["scales"], None), what)
    refused(lib, lambda: lib.dsa_unpack8(a["codes"], a["scales"], a["dt"], a["rows"], a["D"], a["x"], None), what)


WIN = dict(q=FAKE, k=FAKE, v=FAKE, dt=1, B=1, H=4, Hk=2, Nq=100, Nk=100, D=64, scale=0.125, off=0, left=10, right=0,
           sink=0)
BAD_WIN = [
    (dict(q=None), "null"), (dict(v=None), "null"), (dict(dt=5), "dtype"), (dict(B=0), "B, H, Hk"),
    (dict(H=3), "multiple"), (dict(Hk=0), "B, H, Hk"), (dict(B=1 << 15), "65535"), (dict(Nq=0), "Nq and Nk"),
    (dict(Nk=(1 << 27) + 1), "Nq and Nk"), (dict(D=80), "D must"), (dict(scale=0.0), "scale"),
    (dict(scale=float("nan")), "scale"), (dict(off=1 << 29), "q_offset"), (dict(off=-(1 << 29)), "q_offset"),
    (dict(sink=-1), "sink"), (dict(q=FAKE + 8), "aligned"),
    (dict(B=1024, H=32, Hk=32, Nq=1 << 27), "tiles"),
]


@pytest.mark.parametrize("bad,what", BAD_WIN)
def test_window_refuses(lib, bad, what):
    a = {**WIN, **bad}
    shape = (a["dt"], a["B"], a["H"], a["Hk"], a["Nq"], a["Nk"], a["D"], a["scale"], a["off"], a["left"], a["right"],
             a["sink"])
    refused(lib, lambda: lib.dsa_window_attn_fwd(a["q"], a["k"], a["v"], *shape, FAKE, None, None), what)
    refused(lib, lambda: lib.dsa_window_attn_bwd(a["q"], a["k"], a["v"], FAKE, FAKE, FAKE, *shape, FAKE, FAKE, FAKE, FAKE,
                                                 1 << 40, None), what)


def test_window_outputs(lib):
    shape = tuple(WIN[n] for n in ("dt", "B", "H", "Hk", "Nq", "Nk", "D", "scale", "off", "left", "right", "sink"))
    refused(lib, lambda: lib.dsa_window_attn_fwd(FAKE, FAKE, FAKE, *shape, None, None, None), "null")
    refused(lib, lambda: lib.dsa_window_attn_fwd(FAKE, FAKE, FAKE, *shape, FAKE + 8, None, None), "aligned")
    refused(lib, lambda: lib.dsa_window_attn_fwd(FAKE, FAKE, FAKE, *shape, FAKE, FAKE + 2, None), "aligned")
    refused(lib, lambda: lib.dsa_window_attn_bwd(FAKE, FAKE, FAKE, FAKE, FAKE, None, *shape, FAKE, FAKE, FAKE, FAKE, 1 << 30,
                                                 None), "null")


def bwd_ws(lib, **kw):
    a = {**WIN, **kw}
    return lib.dsa_window_attn_bwd_workspace_size(a["dt"], a["B"], a["H"], a["Hk"], a["Nq"], a["Nk"], a["D"], a["off"],
                                                  a["left"], a["right"], a["sink"])


def test_workspace_sizes(lib):
    assert bwd_ws(lib) == 4 * 100 * 4                       # delta
    assert bwd_ws(lib, D=32) == 0 and bwd_ws(lib, Nq=0) == 0
    assert bwd_ws(lib, dt=0) >= bwd_ws(lib)                 # fp32: shares where tiles are few
    # 4 query heads, 16 key tiles of which the first sees every query: dK and dV in shares
    assert bwd_ws(lib, dt=0, Nq=1000, Nk=1000, left=200, sink=3) > 4 * 1000 * 4 + 2 * 2 * 1000 * 64 * 4
    # bf16: the shares of the one key tile with sinks (64 query tiles of 4 heads against 17 for the others)
    big = dict(H=16, Hk=4, Nq=8192, Nk=8192, D=128, left=2047)
    assert bwd_ws(lib, **big) == 16 * 8192 * 4
    parts = bwd_ws(lib, **big, sink=4) - 16 * 8192 * 4
    assert parts > 0 and parts % (4 * 2 * 128 * 128 * 4) == 0
    # thousands of tiles: none
    assert bwd_ws(lib, dt=0, H=64, Hk=64, Nq=4096, Nk=4096, left=128) == 64 * 4096 * 4
    need = lib.dsa_window_attn_decode_workspace_size
    assert need(1, 64, 32, 8, 1, 4096, 128, -1, 0) == 0     # heads fill the SMs
    assert need(1, 1, 8, 2, 1, 1000, 128, -1, 0) == 0       # small: a cluster
    assert need(1, 1, 8, 2, 1, 1 << 20, 128, -1, 0) > 0     # long: shares
    assert need(1, 1, 8, 2, 1, 1 << 20, 128, 100, 0) == 0   # but a short window
    assert need(1, 1, 8, 3, 1, 1 << 20, 128, -1, 0) == 0    # bad shape


@pytest.mark.parametrize("bad,what", [
    (dict(q=None), "null"), (dict(lens=None), "null"), (dict(strides=None), "null"), (dict(dt=3), "dtype"),
    (dict(H=5), "multiple"), (dict(Nq=0), "Nq"), (dict(Nq=129), "Nq"), (dict(cap=0), "cap"), (dict(D=256), "D must"),
    (dict(sink=-2), "sink"), (dict(scale=-1.0), "scale"), (dict(q=FAKE + 8), "aligned"), (dict(lens=FAKE + 2), "aligned"),
    (dict(strides=(6400, 6400, 60, 6400, 6400, 64)), "multiples"), (dict(strides=(0, 6400, 64, 12800, 6400, 64)), "overlap"),
    (dict(strides=(12800, 6400, 64, 12800, 6400, 32)), "overlap"),
    (dict(cap=1 << 20, strides=(1 << 30, 1 << 29, 64) * 2), "workspace"),
])
def test_decode_refuses(lib, bad, what):
    a = {**dict(q=FAKE, k=FAKE, v=FAKE, strides=(12800, 6400, 64) * 2, dt=1, B=2, H=4, Hk=2, Nq=1, cap=100, D=64,
                scale=0.125, lens=FAKE, left=-1, sink=0), **bad}
    st = None if a["strides"] is None else i64(*a["strides"])
    refused(lib, lambda: lib.dsa_window_attn_decode(a["q"], a["k"], a["v"], st, a["dt"], a["B"], a["H"], a["Hk"], a["Nq"],
                                                    a["cap"], a["D"], a["scale"], a["lens"], a["left"], a["sink"], FAKE,
                                                    None, None, 0, None), what)


def test_python_checks():
    x = torch.zeros(1, 4, 2, 64)
    with pytest.raises(ValueError):
        ops.pack8(x)                                        # not on a GPU
    with pytest.raises(ValueError):
        ops.window_attn_fwd(x, x, x)
    with pytest.raises(ValueError):
        ops.window_attn_decode(x, x, x, torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        ops.rope_table(0, 4)
    with pytest.raises(ValueError):
        ops.RopePlan(torch.zeros(4, 3, dtype=torch.int32), (), device="cpu")
    with pytest.raises(ValueError):
        ops.RopePlan(torch.zeros(4, 3, dtype=torch.int32), (8, 8), theta=(1e4,), device="cpu")
    with pytest.raises(ValueError, match="rows per token"):
        window_layer._split(torch.zeros(1, 4, 7, 64), 4)
    with pytest.raises(ValueError, match="causal"):
        window_layer.Stream(1, 2, 2, 8, 64, type("P", (), {"table": x}), window_layer.Mask(1, 1, 0))
    with pytest.raises(ValueError, match="CUDA device"):
        ops.rope_table(8, 4, device="cpu")
    for v in (2**31, -2**31 - 1):                           # not cut to 32 bits
        with pytest.raises(ValueError, match="32 bits"):
            ops._check_mask(0, v, 0, 0)
