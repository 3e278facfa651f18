"""Refusals of the int4 and MoE layer entry points, before any HIP call (CPU)."""

import ctypes
import os
import subprocess

import pytest
import torch

from grouped_nf4_expert_amd import gnf4

NULL = ctypes.c_void_p(0)
FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: rejected before any HIP call
OK, INVALID, NOT_DEVICE, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(gnf4.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return gnf4.library()


def test_exported(lib):
    out = subprocess.run(["nm", "-D", "--defined-only", gnf4.LIB_PATH], capture_output=True,
                         text=True, check=True).stdout
    for n in ("gnf4_int4_pack", "gnf4_int4_linear", "gnf4_moe_layer",
              "gnf4_moe_layer_workspace_size"):
        assert f" T {n}\n" in out


def test_int4_pack_arguments(lib):
    def call(**kw):
        a = dict(w=FAKE, wd=0, N=4, K=256, g=64, p=FAKE, s=FAKE, sd=0, z=NULL)
        a.update(kw)
        return lib.gnf4_int4_pack(a["w"], a["wd"], a["N"], a["K"], a["g"], a["p"], a["s"],
                                  a["sd"], a["z"], NULL)
    for kw in (dict(w=NULL), dict(p=NULL), dict(s=NULL), dict(N=0), dict(N=-1), dict(K=0),
               dict(K=96), dict(g=16), dict(g=0), dict(g=-64), dict(wd=2), dict(sd=2),
               dict(w=ctypes.c_void_p(0x1008)), dict(p=ctypes.c_void_p(0x1002)),
               dict(s=ctypes.c_void_p(0x1001)), dict(N=2 ** 62)):
        assert call(**kw) == INVALID, kw
    assert call() == NOT_DEVICE


def test_int4_linear_arguments(lib):
    def call(**kw):
        a = dict(x=FAKE, M=2, p=FAKE, s=FAKE, sd=0, z=NULL, g=64, N=4, K=256, b=NULL, y=FAKE)
        a.update(kw)
        return lib.gnf4_int4_linear(a["x"], a["M"], a["p"], a["s"], a["sd"], a["z"], a["g"],
                                    a["N"], a["K"], a["b"], a["y"], NULL)
    for kw in (dict(x=NULL), dict(p=NULL), dict(s=NULL), dict(y=NULL), dict(M=-1), dict(N=0),
               dict(K=0), dict(K=-64), dict(K=96), dict(g=48), dict(sd=9),
               dict(x=ctypes.c_void_p(0x1008)), dict(p=ctypes.c_void_p(0x1008)),
               dict(y=ctypes.c_void_p(0x1001)), dict(b=ctypes.c_void_p(0x1001)),
               dict(s=ctypes.c_void_p(0x1002), sd=1)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(M=2 ** 20 + 1), dict(N=2 ** 30), dict(K=2 ** 30)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(M=0) == OK
    assert call() == NOT_DEVICE


def test_moe_layer_arguments(lib):
    def call(**kw):
        a = dict(l=FAKE, T=2, E=8, k=2, x=FAKE, gp=FAKE, gs=FAKE, dp=FAKE, ds=FAKE, kind=1, H=128,
                 I=64, r=NULL, o=FAKE, ids=FAKE, w=FAKE, ws=FAKE, n=1 << 30)
        a.update(kw)
        return lib.gnf4_moe_layer(a["l"], a["T"], a["E"], a["k"], a["x"], a["gp"], a["gs"],
                                  a["dp"], a["ds"], a["kind"], a["H"], a["I"], a["r"], a["o"],
                                  a["ids"], a["w"], a["ws"], a["n"], NULL)
    for name in ("l", "x", "gp", "gs", "dp", "ds", "o", "ids", "w"):
        assert call(**{name: NULL}) == INVALID, name
    for kw in (dict(T=-1), dict(E=0), dict(k=0), dict(k=9), dict(H=0), dict(H=96), dict(I=32),
               dict(kind=3), dict(kind=-1), dict(x=ctypes.c_void_p(0x1008)),
               dict(gp=ctypes.c_void_p(0x1004)), dict(dp=ctypes.c_void_p(0x1004)),
               dict(gs=ctypes.c_void_p(0x1002)), dict(o=ctypes.c_void_p(0x1001)),
               dict(r=ctypes.c_void_p(0x1001)), dict(ws=ctypes.c_void_p(0x1004))):
        assert call(**kw) == INVALID, kw
    for kw in (dict(T=65), dict(E=1025), dict(E=64, k=33), dict(H=8256), dict(I=8256)):
        assert call(**kw) == UNSUPPORTED, kw
    need = lib.gnf4_moe_layer_workspace_size(2, 8, 2, 128, 64)
    assert need > 0
    assert call(ws=NULL) == WORKSPACE and call(n=need - 1) == WORKSPACE
    assert call(n=need) == NOT_DEVICE
    assert call(T=0) == OK
    assert lib.gnf4_moe_layer_workspace_size(65, 8, 2, 128, 64) == 0


def test_python_checks():
    x = torch.zeros((2, 128), dtype=torch.bfloat16)
    p = torch.zeros((4, 64), dtype=torch.uint8)
    s = torch.ones((4, 1))
    with pytest.raises(gnf4.Gnf4Error, match="device memory"):
        gnf4.int4_linear(x, p, s)
    with pytest.raises(TypeError):
        gnf4.int4_linear(x.float(), p, s)
    with pytest.raises(TypeError):
        gnf4.int4_linear(x, p, s.half())
    with pytest.raises(ValueError):
        gnf4.int4_linear(x[:, :64].contiguous(), p, s)
    with pytest.raises(ValueError):
        gnf4.int4_linear(x, p, s, zeros=torch.zeros((4, 2), dtype=torch.uint8))
    with pytest.raises(ValueError):
        gnf4.int4_linear(x, p, s, bias=torch.zeros(3, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        gnf4.int4_linear(x, p, s, out=torch.zeros((2, 5), dtype=torch.bfloat16))
    w = torch.zeros((4, 96), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        gnf4.int4_pack(w, 64)
    with pytest.raises(TypeError):
        gnf4.int4_pack(w.half(), 32)
    with pytest.raises(TypeError):
        gnf4.int4_pack(w, 32, scale_dtype=torch.float16)
    with pytest.raises(ValueError):
        gnf4.int4_pack(w[0], 32)
