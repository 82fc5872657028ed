"""Refusals of the attention operators at the C boundary, on the host: no call here passes validation, except the
workspace queries, so nothing touches a GPU."""

import ctypes
import struct

import pytest

import tiled_genome_diffusion_amd as pc
from tiled_genome_diffusion_amd import _lib

F = 4096          # a fake, aligned device address, never dereferenced
MIS = 4104


def sizes(dtype=1, n_kv=2, group=3, len_q=5, len_k=40, heads=4, heads_kv=2, dim=64, scale=0.125, strides=None, **change):
    q, k = (len_q * heads * dim, heads * dim, dim), (len_k * heads_kv * dim, heads_kv * dim, dim)
    s = {"q": q, "k": k, "v": k, "out": q, "dout": q, "dq": q, "dk": k, "dv": k}
    s.update(change)
    return pc._ATTENTION.pack(dtype, n_kv, group, len_q, len_k, heads, heads_kv, dim, scale,
                              *(v for n in ("q", "k", "v", "out", "dout", "dq", "dk", "dv") for v in s[n]))


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def fwd(lib, a, q=F, k=F, v=F, kv_len=None, mask=None, out=F, lse=None, ws=None, n=0):
    return lib.pc_cross_attention(a, q, k, v, kv_len, mask, out, lse, ws, n, None)


def bwd(lib, a, q=F, k=F, v=F, out=F, lse=F, dout=F, kv_len=None, mask=None, dq=F, dk=F, dv=F, ws=F, n=1 << 40):
    return lib.pc_cross_attention_backward(a, q, k, v, out, lse, dout, kv_len, mask, dq, dk, dv, ws, n, None)


def test_struct_sizes_match_the_header():
    assert pc._ATTENTION.size == 40 + 24 * 8 and pc._NORM_SIDE.size == 80 + 12 * 8


@pytest.mark.parametrize("change,status", [
    (dict(dtype=3), -4), (dict(dtype=-1), -4), (dict(dim=4), -2), (dict(dim=60), -2), (dict(dim=136), -2),
    (dict(dim=0), -2), (dict(n_kv=-1), -2), (dict(group=-1), -2), (dict(len_q=-1), -2), (dict(len_k=-1), -2),
    (dict(len_k=(1 << 30) + 1), -2), (dict(heads=0), -2), (dict(heads_kv=0), -2), (dict(heads=5), -2),
    (dict(scale=0.0), -4), (dict(scale=-1.0), -4), (dict(scale=float("nan")), -4), (dict(scale=float("inf")), -4),
    (dict(group=1 << 20, len_q=1 << 11, heads=2, heads_kv=1), -2),            # 2^32 rows share a key head
    (dict(n_kv=1 << 22, heads=1 << 10, heads_kv=1 << 10), -2),                # 2^32 key heads
    (dict(q=(1280, 256, 60)), -2), (dict(k=(5120, 4, 64)), -2), (dict(v=(-5120, 128, 64)), -2),
    (dict(out=(0, 256, 64)), -2), (dict(out=(1280, 192, 64)), -2), (dict(out=(1280, 256, 0)), -2),
    (dict(out=(256, 256, 64)), -2), (dict(q=(1 << 60, 256, 64)), -2),
])
def test_sizes_and_strides(lib, change, status):
    a = sizes(**change)
    n = ctypes.c_int64(-1)
    assert fwd(lib, a) == status and lib.pc_last_error() != b""
    if "out" not in change:      # an input of the gradients: broadcast strides are fine there
        assert bwd(lib, a) == status
    assert lib.pc_cross_attention_workspace(a, 0, ctypes.addressof(n)) == status and n.value == -1


def test_gradients_strides(lib):
    for name in ("dq", "dk", "dv"):
        for bad in ((0, 256, 64), (1 << 20, 256, 32), (1 << 20, -256, 64)):
            assert bwd(lib, sizes(**{name: bad})) == -2
    assert bwd(lib, sizes(dout=(1280, 256, 4))) == -2
    # strides the forward does not use are not looked at
    n = ctypes.c_int64()
    assert lib.pc_cross_attention_workspace(sizes(dq=(0, 0, 0), dk=(-1, 0, 0)), 0, ctypes.addressof(n)) == 0


@pytest.mark.parametrize("args,status", [
    (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(out=None), -1), (dict(q=MIS), -3),
    (dict(k=MIS), -3), (dict(v=MIS), -3), (dict(out=MIS), -3), (dict(lse=MIS), -3), (dict(kv_len=4098), -3)])
def test_pointers_forward(lib, args, status):
    assert fwd(lib, sizes(), **args) == status
    assert lib.pc_cross_attention(None, F, F, F, None, None, F, None, None, 0, None) == -1


@pytest.mark.parametrize("args,status", [
    *((dict([(n, None)]), -1) for n in ("q", "k", "v", "out", "lse", "dout", "dq", "dk", "dv", "ws")),
    *((dict([(n, MIS)]), -3) for n in ("q", "k", "v", "out", "lse", "dout", "dq", "dk", "dv", "ws")),
    (dict(kv_len=4098), -3), (dict(n=100), -2)])
def test_pointers_backward(lib, args, status):
    assert bwd(lib, sizes(), **args) == status


def test_split_needs_its_workspace(lib):
    a = sizes(len_k=4096, len_q=1, group=1)
    n = ctypes.c_int64()
    assert lib.pc_cross_attention_workspace(a, 0, ctypes.addressof(n)) == 0 and n.value > 0
    assert fwd(lib, a) == -1 and fwd(lib, a, ws=F, n=n.value - 1) == -2 and fwd(lib, a, ws=MIS, n=n.value) == -3
    assert lib.pc_cross_attention_workspace(a, 0, None) == -1


def test_axes_without_entries_are_no_ops(lib):
    """No output element: nothing is launched and no pointer is needed."""
    for change in (dict(n_kv=0), dict(group=0), dict(len_q=0)):
        assert fwd(lib, sizes(**change), q=None, k=None, v=None, out=None) == 0
    assert bwd(lib, sizes(n_kv=0), *[None] * 6, None, None, None, None, None, None, 0) == 0
    assert bwd(lib, sizes(group=0, len_k=0), *[None] * 6, None, None, None, None, None, None, 0) == 0


def side(batch=2, len=5, heads=3, x=F, y=F, weight=None, pos=None, pos_b=0, dy=F, dx=F, dw=None, dim=64, sx=None, sy=None,
         sdy=None, sdx=None):
    d = (len * heads * dim, heads * dim, dim)
    return pc._NORM_SIDE.pack(batch, len, heads, x or 0, y or 0, weight or 0, pos or 0, pos_b, dy or 0, dx or 0, dw or 0,
                              *(sx or d), *(sy or d), *(sdy or d), *(sdx or d))


FREQS = struct.pack("32d", *[0.5 ** i for i in range(32)])


def norm(lib, q, k=None, dtype=1, dim=64, rot=64, freqs=FREQS, eps=1e-6):
    return lib.pc_qk_norm_rope(q, k, dtype, dim, rot, freqs, 0, eps, None)


@pytest.mark.parametrize("change,status", [
    (dict(batch=-1), -2), (dict(len=-1), -2), (dict(heads=0), -2), (dict(x=None), -1), (dict(y=None), -1),
    (dict(x=MIS), -3), (dict(y=MIS), -3), (dict(weight=MIS), -3), (dict(pos=4098), -3), (dict(pos=F, pos_b=-1), -2),
    (dict(sx=(960, 192, 60)), -2), (dict(sy=(960, 192, 0)), -2), (dict(sy=(192, 192, 64)), -2),
    (dict(batch=1 << 16, len=1 << 15), -2), (dict(sx=(1920, 384, 128)), -2)])
def test_norm_sides(lib, change, status):
    assert norm(lib, side(**change)) == status     # the last one: in place (x is y) with other strides
    assert norm(lib, None, side(**change)) == status
    assert norm(lib, side(batch=0), side(**change)) == status


def test_norm_parameters(lib):
    s = side()
    assert norm(lib, None) == -1
    assert norm(lib, s, dtype=9) == -4 and norm(lib, s, dim=12) == -2 and norm(lib, s, dim=136) == -2
    assert norm(lib, s, rot=8) == -2 and norm(lib, s, rot=80) == -2 and norm(lib, s, rot=-16) == -2
    assert norm(lib, s, freqs=None) == -1
    assert norm(lib, s, eps=-1.0) == -4 and norm(lib, s, eps=float("inf")) == -4
    for bad in (7.0, -7.0, float("nan"), float("inf")):
        assert norm(lib, s, freqs=struct.pack("32d", *[bad] * 32)) == -4
    assert norm(lib, side(batch=0, x=None, y=None)) == 0        # no element


def test_norm_backward_refusals(lib):
    call = lambda q, ws=F, n=1 << 40: lib.pc_qk_norm_rope_backward(q, None, 1, 64, 64, FREQS, 0, 1e-6, ws, n, None)  # noqa: E731
    assert call(side(dy=None)) == -1 and call(side(dx=None)) == -1 and call(side(dy=MIS)) == -3
    assert call(side(dw=MIS)) == -3 and call(side(sdx=(0, 192, 64))) == -2 and call(side(sdy=(960, 192, 60))) == -2
    n = ctypes.c_int64()
    assert lib.pc_qk_norm_rope_workspace(side(), None, 1, 64, 64, ctypes.addressof(n)) == 0 and n.value > 0
    assert call(side(), None) == -1 and call(side(), F, n.value - 1) == -2 and call(side(), MIS, n.value) == -3
    assert lib.pc_qk_norm_rope_workspace(side(), None, 1, 64, 64, None) == -1
    assert lib.pc_qk_norm_rope_workspace(None, None, 1, 64, 64, ctypes.addressof(n)) == -1
