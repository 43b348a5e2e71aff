"""Sizes that the 4-bit decode's 32-bit counts or its launches cannot hold are
refused with MLA_ERR_UNSUPPORTED before any device work (a call within the limits
fails here for want of a GPU, with another status)."""
import ctypes

import pytest

BIG = 1 << 60
TOP = (1 << 31) - 1


@pytest.fixture(scope="module")
def M():
    from head_latent_attention_10_b200 import build
    build.build()
    import head_latent_attention_10_b200 as M
    M.load_library()
    return M


def decode(M, B=1, mb=1, flags=0, name="mla_decode_int4"):
    lib, d, p = M.load_library(), ctypes.byref(M.dims(16)), ctypes.c_void_p(256)
    cache = (p, p) if name == "mla_decode_int4" else (p,)
    n0 = lib.mla_kernel_launches()
    status = getattr(lib, name)(d, p, *cache, 1, p, mb, p, B, 1, p, None, p, BIG, flags, None)
    assert lib.mla_kernel_launches() == n0 or status == M.MLA_ERR_CUDA
    return status


def test_tiles_of_the_batch_are_counted_in_32_bits(M):
    """The plan adds up ceil(L / 64) + 4 over the sequences, and its last range's end
    is rounded up by less than the ranges there can be (148)."""
    for B, mb in ((64, (1 << 25) - 1), (65, (1 << 25) - 1), (1 << 16, (1 << 15) - 4), (1 << 26, 28), (1 << 26, 32)):
        assert B * (mb + 4) + 148 > TOP and decode(M, B=B, mb=mb) == M.MLA_ERR_UNSUPPORTED, (B, mb)
    for B, mb in ((63, (1 << 25) - 1), (1 << 16, (1 << 15) - 5), (1 << 26, 27)):
        assert B * (mb + 4) + 148 <= TOP and decode(M, B=B, mb=mb) != M.MLA_ERR_UNSUPPORTED, (B, mb)


@pytest.mark.parametrize("name", ["mla_decode", "mla_decode_int4"])
def test_splits_of_the_cuda_core_decode_are_limited(M, name):
    """A split is 1,024 tokens, and splits are its grid's third dimension."""
    most = 65535 * 1024 // 64
    assert decode(M, mb=most + 1, flags=M.MLA_FORCE_SIMPLE, name=name) == M.MLA_ERR_UNSUPPORTED
    assert decode(M, mb=most, flags=M.MLA_FORCE_SIMPLE, name=name) != M.MLA_ERR_UNSUPPORTED
    assert decode(M, mb=most + 1, name=name) != M.MLA_ERR_UNSUPPORTED
