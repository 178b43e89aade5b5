"""A producer that starts its successor at once and writes late (early_copy.cu)."""
import ctypes as C
import functools
import os
import subprocess
import tempfile

import torch

from bloom_decoder_token_gb300 import _build


@functools.cache
def _lib():
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "early_copy.cu")
    with tempfile.TemporaryDirectory() as d:
        so = os.path.join(d, "early_copy.so")
        subprocess.run([_build.nvcc()] + _build.ARCH + ["-std=c++17", "-Xcompiler", "-fPIC", "-shared", "-o", so, src], check=True)
        lib = C.CDLL(so)
    lib.early_copy.argtypes = [C.c_void_p, C.c_void_p, C.c_int64, C.c_uint64, C.c_void_p]
    return lib


def early_copy(dst, src, us=30):
    """dst's contents become src's, `us` microseconds after the next kernel of the current stream may start."""
    assert dst.is_contiguous() and src.is_contiguous() and dst.dtype is src.dtype and dst.shape == src.shape
    size = dst.numel() * dst.element_size()
    assert size % 4 == 0 and dst.data_ptr() % 4 == 0 and src.data_ptr() % 4 == 0
    stream = torch.cuda.current_stream(dst.device).cuda_stream
    assert _lib().early_copy(dst.data_ptr(), src.data_ptr(), size, us * 1000, stream) == 0
