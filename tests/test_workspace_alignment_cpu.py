"""A workspace that is not 16-byte aligned is refused before any device work: the
kernels store and load 16 bytes at a time in it."""
import ctypes

import pytest

BIG = 1 << 40


@pytest.fixture(scope="module")
def M():
    from head_latent_attention_10_b200 import build
    build.build()
    import head_latent_attention_10_b200 as M
    M.load_library()
    return M


def calls(M):
    lib, d, p = M.load_library(), ctypes.byref(M.dims(128)), ctypes.c_void_p(256)
    return {
        "mla_decode": lambda ws, f: lib.mla_decode(d, p, p, 1, p, 1, p, 1, 1, p, None, ws, BIG, f, None),
        "mla_decode_fp8": lambda ws, f: lib.mla_decode_fp8(d, p, p, p, 1, p, 1, p, 1, 1, p, None, ws, BIG, f, None),
        "mla_decode_int4": lambda ws, f: lib.mla_decode_int4(d, p, p, p, 1, p, 1, p, 1, 1, p, None, ws, BIG, f, None),
        "mla_prefill": lambda ws, f: lib.mla_prefill(d, p, p, None, p, p, p, 1, p, 1, p, 1, 4, 64, p, None, ws, BIG, f,
                                                     None),
        "mla_prefill_int4": lambda ws, f: lib.mla_prefill_int4(d, p, p, None, p, p, p, p, 1, p, 1, p, 1, 4, 64, p, None,
                                                               ws, BIG, f, None),
    }


@pytest.mark.parametrize("name, simple", [
    ("mla_decode", 0), ("mla_decode", 1), ("mla_decode_fp8", 0), ("mla_decode_int4", 0), ("mla_decode_int4", 1),
    ("mla_prefill", 0), ("mla_prefill_int4", 0)])
def test_misaligned_workspaces_are_refused(M, name, simple):
    f = M.MLA_FORCE_SIMPLE if simple else 0
    call, n0 = calls(M)[name], M.load_library().mla_kernel_launches()
    for off in (1, 2, 4, 8, 12):
        assert call(ctypes.c_void_p(4096 + off), f) == M.MLA_ERR_INVALID_ARG, off
    assert call(None, f) == M.MLA_ERR_WORKSPACE
    assert M.load_library().mla_kernel_launches() == n0
