"""The library's own roots and reciprocals (csrc/roots.cuh) on every float32 of
their ranges, against CUDA's correctly rounded ones and float64."""
import ctypes
import struct
import subprocess

import pytest
import torch

pytestmark = pytest.mark.gpu


def bits(x):
    return struct.unpack("I", struct.pack("f", x))[0]


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    from top_routing_dispatch_gb300 import build as B
    so = tmp_path_factory.mktemp("roots") / "roots.so"
    src = __file__.replace("test_gpu_roots.py", "roots.cu")
    subprocess.run([B._nvcc(), *B.ARCH, "-O3", "-std=c++17", "-I", B.CSRC, "-I", B.INCLUDE, "-Xcompiler", "-fPIC",
                    "-shared", "-cudart", "shared", src, "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))

    def run(what, first, last):
        counts = torch.zeros(2, dtype=torch.int64, device="cuda")
        torch.cuda.synchronize()
        assert lib.roots_check(what, ctypes.c_uint(first), ctypes.c_uint(last), ctypes.c_void_p(counts.data_ptr())) == 0
        torch.cuda.synchronize()
        wrong, seen = counts.tolist()
        assert seen == last - first + 1
        return wrong
    return run


LARGEST = 0x7F7FFFFF


def test_square_roots(check):
    assert check(0, bits(2.0 ** -102), LARGEST) == 0


def test_reciprocals(check):
    assert check(1, bits(2.0 ** -126), bits(2.0 ** 126)) == 0


def test_approximate_reciprocals(check):
    assert check(2, bits(2.0 ** -126), bits(2.0 ** 126)) == 0


def test_reciprocal_square_roots(check):
    assert check(3, bits(2.0 ** -126), LARGEST) == 0


def test_the_check_sees_wrong_values(check):
    """Below 2^-102 roots are not all correctly rounded."""
    assert check(0, bits(2.0 ** -126), bits(2.0 ** -110)) > 0
