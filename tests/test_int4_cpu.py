"""The 4-bit latent cache without a GPU: pins of the oracle's quantizer and
values, and the refusals of the four entry points (C and Python)."""
import ctypes
import os
from fractions import Fraction

import numpy as np
import pytest

import mla_workloads as W
import oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def M():
    from head_latent_attention_10_b200 import build
    build.build()
    import head_latent_attention_10_b200 as M
    M.load_library()
    return M


def value(u, b):
    """(u - 8) (1 + (b & 7) / 8) 2^((b >> 3) - 15), exactly."""
    return (u - 8) * (1 + Fraction(b & 7, 8)) * Fraction(2) ** ((b >> 3) - 15)


def place(i):
    """Byte of a word and shift of the nibble that holds the word's value i."""
    nibble = i // 2 + 4 * (i % 2)
    return nibble // 2, 4 * (nibble % 2)


def test_every_code_and_scale_has_its_value_and_is_a_bf16_value():
    b = np.repeat(np.arange(256, dtype=np.uint8), 1)
    codes = np.zeros((256, 8), np.uint8)            # one group a row: u = 0..15 in place
    for i in range(16):
        byte, sh = place(i % 8)
        codes[:, 4 * (i // 8) + byte] |= np.uint8(i << sh)
    got = oracle.int4_values(codes, b[:, None])
    for r in range(256):
        assert [Fraction(v) for v in got[r]] == [value(u, r) for u in range(16)]
    assert np.array_equal(W.bf16_bits_to_f32(W.f32_to_bf16_bits(got.astype(np.float32))).astype(np.float64), got)


def test_quantizer_against_a_search_over_every_scale_and_code():
    """The scale nearest to amax * (1/7) (even byte on a tie), then the code nearest
    to x / s (even on a tie) among -7..7."""
    rng = np.random.default_rng(11)
    x = rng.standard_normal((60, 32)).astype(np.float32) * np.exp2(rng.integers(-20, 20, (60, 1))).astype(np.float32)
    x[0] = 0.0
    x[1, :16] = 7.0 * (1 + 1 / 16) * (np.arange(16) == 3)      # midway between two scales
    x[2, :16] = np.arange(16) / 2.0 - 3.5                      # halves of the scale 0.5: ties of codes
    x = W.bf16_bits_to_f32(W.f32_to_bf16_bits(x))
    codes, scales = oracle.int4_quantize_rows(x)
    every = [(1 + Fraction(b & 7, 8)) * Fraction(2) ** ((b >> 3) - 15) for b in range(256)]
    for n in range(x.shape[0]):
        for g in range(2):
            v = x[n, 16 * g:16 * g + 16]
            t = Fraction(float(np.abs(v).max() * np.float32(1 / 7)))
            best = min(range(256), key=lambda b: (abs(every[b] - t), b % 2))
            assert scales[n, g] == best
            s = np.float32(float(every[best]))
            for i in range(16):
                q = Fraction(float(v[i] / s))
                want = min(range(-7, 8), key=lambda k: (abs(k - q), k % 2)) + 8
                byte, sh = place(i % 8)
                assert (codes[n, 8 * g + 4 * (i // 8) + byte] >> sh) & 15 == want, (n, g, i)


def test_quantizer_limits():
    """Zero groups, values below and above the scales' range, NaN and infinity
    all give finite values; the error of a group in range is at most half a
    step (the scale rounds by at most 1/16, so no value is clipped by more)."""
    rows = np.zeros((6, 16), np.float32)
    rows[1] = 1e-30
    rows[2, 3] = 3e38
    rows[3, 0], rows[3, 1] = np.inf, -np.inf
    rows[4, 0], rows[4, 5] = np.nan, 2.0
    rows[5] = np.linspace(-3, 3, 16)
    codes, scales = oracle.int4_quantize_rows(rows)
    v = oracle.int4_values(codes, scales)
    top = 7 * 1.875 * 2.0 ** 16
    assert np.all(v[0] == 0) and np.all(v[1] == 0)
    assert v[2, 3] == top and v[3, 0] == top and v[3, 1] == -top
    assert v[4, 0] == 0 and abs(v[4, 5] - 2.0) <= 1 / 7
    s = (1 + (scales[5] & 7) / 8.0) * np.exp2((scales[5] >> 3) - 15.0)
    assert np.max(np.abs(v[5] - rows[5])) <= s[0] / 2 * (1 + 1e-6)


def test_argument_errors_of_the_c_entry_points(M):
    lib = M.load_library()
    d = ctypes.byref(M.dims(128))
    p, odd = ctypes.c_void_p(256), ctypes.c_void_p(264)
    big = 1 << 40
    n0 = lib.mla_kernel_launches()
    INVALID, UNSUP, WS = M.MLA_ERR_INVALID_ARG, M.MLA_ERR_UNSUPPORTED, M.MLA_ERR_WORKSPACE

    def append(T=1, ckv=p, kr=p, codes=p, scales=p, nb=1, mb=1, w=None, eps=0.0, dd=d):
        return lib.mla_append_latent_int4(dd, ckv, kr, T, p, p, p, 1, mb, codes, scales, nb, w, eps, None, None)

    assert append(T=0) == M.MLA_OK and append(T=0, ckv=None, codes=None) == M.MLA_OK
    assert append(dd=None) == INVALID and append(T=-1) == INVALID and append(nb=-1) == INVALID
    assert append(ckv=None) == INVALID and append(scales=None) == INVALID
    assert append(codes=odd) == INVALID and append(scales=odd) == INVALID and append(ckv=odd) == INVALID
    assert append(kr=ctypes.c_void_p(258)) == INVALID
    assert append(w=p, eps=-1.0) == INVALID and append(w=p, eps=float("nan")) == INVALID and append(w=odd) == INVALID
    assert append(T=(1 << 26) + 1) == UNSUP and append(mb=1 << 26) == UNSUP
    assert append(dd=ctypes.byref(M.dims(24))) == UNSUP

    def gather(T=1, codes=p, scales=p, rows=p, mb=1, idx=p, dd=d):
        return lib.mla_gather_latent_int4(dd, codes, scales, 1, idx, p, T, p, 1, mb, rows, None, None)

    assert gather(T=0, codes=None, rows=None) == M.MLA_OK
    assert gather(dd=None) == INVALID and gather(T=-1) == INVALID and gather(mb=-1) == INVALID
    assert gather(idx=None) == INVALID and gather(rows=odd) == INVALID and gather(codes=odd) == INVALID
    assert gather(scales=odd) == INVALID and gather(mb=1 << 26) == UNSUP

    def dec(q=p, B=1, s=1, nb=1, mb=1, codes=p, sc=p, out=p, ws=p, wsb=big, flags=0, dd=d):
        return lib.mla_decode_int4(dd, q, codes, sc, nb, p, mb, p, B, s, out, None, ws, wsb, flags, None)

    for flags in (0, M.MLA_FORCE_SIMPLE):
        assert dec(B=0, q=None, ws=None, flags=flags) == M.MLA_OK
        assert dec(ws=None, flags=flags) == WS and dec(wsb=16, flags=flags) == WS
    assert dec(dd=None) == INVALID and dec(B=-1) == INVALID and dec(s=0) == INVALID
    assert dec(nb=0) == INVALID and dec(mb=0) == INVALID and dec(q=None) == INVALID
    assert dec(q=odd) == INVALID and dec(codes=odd) == INVALID and dec(sc=odd) == INVALID and dec(out=odd) == INVALID
    assert dec(B=1 << 20, s=1 << 10) == UNSUP and dec(mb=1 << 26) == UNSUP
    assert dec(dd=ctypes.byref(M.dims(128, block_size=32))) == UNSUP

    def pre(q=p, B=1, s=4, msl=64, nb=1, mb=1, codes=p, sc=p, ws=p, wsb=big, dd=d):
        return lib.mla_prefill_int4(dd, q, p, None, p, p, codes, sc, nb, p, mb, p, B, s, msl, p, None, ws, wsb, 0, None)

    assert pre(B=0, q=None, ws=None) == M.MLA_OK
    assert pre(dd=None) == INVALID and pre(q=None) == INVALID and pre(q=odd) == INVALID and pre(s=0) == INVALID
    assert pre(s=65) == INVALID and pre(nb=0) == INVALID and pre(mb=0) == INVALID
    assert pre(codes=None) == INVALID and pre(codes=odd) == INVALID and pre(sc=odd) == INVALID
    assert pre(ws=None) == WS and pre(wsb=4096) == WS
    assert pre(B=65536) == UNSUP and pre(msl=(1 << 31) - 1) == UNSUP
    assert lib.mla_kernel_launches() == n0


def test_python_binding_refuses_wrong_shapes_types_and_places(M):
    import torch
    bf, i32, u8 = torch.bfloat16, torch.int32, torch.uint8
    codes, scales = torch.zeros(2, 64, 288, dtype=u8), torch.zeros(2, 64, 36, dtype=u8)
    one, table = torch.zeros(1, dtype=i32), torch.zeros(1, 2, dtype=i32)
    ckv, kr = torch.zeros(1, 512, dtype=bf), torch.zeros(1, 64, dtype=bf)
    d = M.dims(16)
    call = lambda **k: M.mla_append_latent_int4(d, **{**dict(  # noqa: E731
        c_kv=ckv, k_rope=kr, seq_idx=one, pos=one, block_table=table, codes=codes, scales=scales), **k})
    for bad, what in ((dict(scales=scales[:1]), "scales"), (dict(codes=codes.int()), "codes"),
                      (dict(k_rope=kr.float()), "k_rope"), (dict(pos=torch.zeros(2, dtype=i32)), "pos"),
                      (dict(c_kv=ckv[:, :256]), "c_kv"), (dict(block_table=one), "block_table"),
                      (dict(codes=torch.zeros(2, 288, 64, dtype=u8).transpose(1, 2)), "codes"),
                      (dict(kv_norm_weight=torch.zeros(511, dtype=bf)), "kv_norm_weight")):
        with pytest.raises(ValueError, match=what):
            call(**bad)
    with pytest.raises(ValueError, match="current GPU"):        # right in all but its place: the host
        call()
    q, lat = torch.zeros(2, 16, 576, dtype=bf), torch.zeros(2, 16, 512, dtype=bf)
    with pytest.raises(ValueError, match="q_abs"):
        M.mla_decode_int4(d, q, codes, scales, table, one, 1, lat, None, codes)
    with pytest.raises(ValueError, match="block_table"):
        M.mla_decode_int4(d, q, codes, scales, torch.zeros(2, 2, dtype=i32), one, 2, lat, None, codes)
