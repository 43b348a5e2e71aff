"""Sizes that the prefill's launches or 32-bit indexes cannot hold are refused
with MLA_ERR_UNSUPPORTED before any device work, for either cache (a call within
the limits fails here for want of a GPU, with another status)."""
import ctypes

import pytest

BIG = 1 << 60                     # more workspace than any of these calls could ask for
TILES = 65535                     # 128-row tiles of the expansions at most (their grid's y)


@pytest.fixture(scope="module")
def M():
    from head_latent_attention_10_b200 import build
    build.build()
    import head_latent_attention_10_b200 as M
    M.load_library()
    return M


def status(M, cache, H=16, B=1, s=1, msl=1):
    lib, d, p = M.load_library(), ctypes.byref(M.dims(H)), ctypes.c_void_p(256)
    if cache == "bf16":
        return lib.mla_prefill(d, p, p, None, p, p, p, 1, p, 1, p, B, s, msl, p, None, p, BIG, 0, None)
    return lib.mla_prefill_int4(d, p, p, None, p, p, p, p, 1, p, 1, p, B, s, msl, p, None, p, BIG, 0, None)


@pytest.mark.parametrize("cache", ["bf16", "int4"])
def test_row_tiles_of_the_expansions_are_limited(M, cache):
    n0 = M.load_library().mla_kernel_launches()
    for B, msl in ((TILES + 1, 1), (TILES + 1, 128), (32768, 257), (21846, 300), (1, 128 * TILES + 1),
                   (2, 64 * (TILES + 1) + 1), (1 << 30, 1), (1, (1 << 31) - 1), (1 << 20, (1 << 31) - 1)):
        assert status(M, cache, B=B, msl=msl) == M.MLA_ERR_UNSUPPORTED, (B, msl)
    for B, msl in ((TILES, 1), (TILES, 128), (32767, 256), (21845, 300), (1, 128 * TILES)):
        assert status(M, cache, B=B, msl=msl) != M.MLA_ERR_UNSUPPORTED, (B, msl)
    assert M.load_library().mla_kernel_launches() == n0


def test_workspace_size_of_the_longest_sequence(M):
    """Rounding max_seq_len up to 128 rows passes 2^31: the size still grows with it."""
    lib, d = M.load_library(), ctypes.byref(M.dims(16))
    a, b = (lib.mla_prefill_workspace_size(d, 1, 1, n) for n in ((1 << 31) - 128, (1 << 31) - 1))
    assert b - a == 128 * (576 * 2 + 2 * 16 * 128 * 2)
