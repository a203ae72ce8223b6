"""Where the cross attention entry points put the kernels' workspace inside the
caller's: the entry points as they are, over launches that only keep what they
were handed (no GPU needed)."""

import ctypes
import os
import shutil
import subprocess

import pytest

import block_sparse_attention_spark_b200 as spark
from block_sparse_attention_spark_b200 import build
from tests.test_operators_abi import C, FAKE, view

HERE = os.path.dirname(os.path.abspath(__file__))


class Seen(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("many", "bwd", "packed")] + [(n, ctypes.c_uint64) for n in ("ws", "pack_ws")]


@pytest.fixture(scope="module")
def entry(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("fake") / "cross.so")
    cuda = os.path.join(os.path.dirname(os.path.dirname(build.nvcc())), "include")
    subprocess.run([shutil.which("g++"), "-std=c++17", "-O1", "-fPIC", "-shared", "-I" + build.INCLUDE, "-I" + build.CSRC,
                    "-I" + cuda, "-x", "c++", os.path.join(build.CSRC, "cross_api.cu"),
                    os.path.join(HERE, "fake_cross_launch.cpp"), "-o", so], check=True)
    L = ctypes.CDLL(so)
    for name in ("spark_cross_attn", "spark_cross_attn_bwd", "spark_cross_workspace_size"):
        fn = getattr(L, name)
        fn.restype, fn.argtypes = spark._SIGS[name]
    L.fake_set.argtypes = [ctypes.c_size_t, ctypes.c_size_t, ctypes.c_int]
    L.fake_seen.restype = ctypes.POINTER(Seen)
    return L


@pytest.mark.parametrize("kind", ["few", "many", "bwd"])
@pytest.mark.parametrize("own,pack", [(0, 512), (1, 256), (1000, 3328), (4096, 0)])
def test_any_accepted_workspace_gives_the_kernels_an_aligned_one(entry, kind, own, pack):
    L, p = entry, C()
    q, k = view(2, 4, 100, 64), view(2, 2, 70, 64)
    for at in range(0, 512, 16):
        L.fake_set(own, pack, kind == "few")
        ws, size = FAKE + at, L.spark_cross_workspace_size(p, kind == "bwd")
        if kind == "bwd":
            code = L.spark_cross_attn_bwd(p, q, k, k, q, FAKE, q, None, FAKE, q, k, k, ws, size, None)
        else:
            code = L.spark_cross_attn(p, q, k, k, None, FAKE, q, None, ws, size, None)
        assert code == 0
        s = L.fake_seen().contents
        assert (s.many, s.bwd, s.packed) == (kind == "many", kind == "bwd", kind == "many")
        assert ws <= s.ws and s.ws % 256 == 0          # the widest stores take 32 bytes
        end = s.ws + own
        if kind != "few":
            assert s.pack_ws >= end and s.pack_ws % 256 == 0
            end = s.pack_ws + pack
        assert end <= ws + size
