"""Prefill whose running maxima grow: for eight heads' last query, keys planted along
that query in the second and in the last key tile exceed all before them by more than
the 8 log2 units from which O is rescaled.  Items of 2 to 6 tiles, several to a CTA
(the tiles' parity alternates from item to item).

Tolerances: test_gpu_int4's for the 4-bit cache.  mla_prefill over the same rows
rounds v^C and the weights to bf16, 2^-8 relative each where that tolerance has 2^-11
twice (2^-10), and needs no fixed step for small values."""
import numpy as np
import pytest

import mla_workloads as W
import oracle
from _gpu_setup import assert_parity
from test_gpu_int4 import C, M, floats, plain_prefill, random_cache, run_prefill  # noqa: F401

pytestmark = pytest.mark.gpu


PLANTED = 8          # heads


def plant(codes, scales, d, cfg):
    """The keys, and by how much they raise the maxima (log2 units, of the latents' part
    of the logits: the rotated keys' part has a standard deviation below 2)."""
    qn, wk = oracle.bf16_to_f64(d["q_nope"]), oracle.bf16_to_f64(d["w_uk"])
    grown = []
    for b, L in enumerate(cfg.seq_lens):
        q = [qn[(b + 1) * cfg.s - 1, h] @ wk[h] for h in range(PLANTED)]
        for h in range(PLANTED):
            for j, size in ((130 + h, 4.0), (L - 1 - h, 9.0)):
                row = np.zeros((1, 576), np.float32)
                row[0, :512] = size * q[h] / np.abs(q[h]).max()
                page, slot = d["block_table"][b, j // 64], j % 64
                codes[page, slot], scales[page, slot] = (v[0] for v in oracle.int4_quantize_rows(row))
        pages = d["block_table"][b, :(L + 63) // 64]
        rows = oracle.int4_values(codes[pages], scales[pages]).reshape(-1, 576)[:L, :512]
        for h in range(PLANTED):
            z = rows @ q[h] / np.sqrt(192.0) / np.log(2.0)
            tops = [z[k:k + 128].max() for k in range(0, L, 128)]
            grown += [tops[1] - tops[0], tops[-1] - max(tops[:-1])]
    return np.array(grown)


@pytest.mark.parametrize("cfg", [C("rs_h16", 16, [300, 265, 520, 650, 400] * 6, s=140, seed=90),
                                 C("rs_h128", 128, [300, 520], s=300, seed=91)], ids=lambda c: c.name)
def test_maxima_that_grow_in_later_tiles(M, cfg):  # noqa: F811
    d = W.make_decode_inputs(cfg, with_cache_pages=False)
    codes, scales = random_cache(d, cfg.seed)
    assert plant(codes, scales, d, cfg).min() > 12.0
    got, lse, err, want, want_lse = run_prefill(M, cfg, d, codes, scales, max(cfg.seq_lens))
    assert err == 0
    ref, rlse, tol, tol_lse = plain_prefill(codes, scales, d, cfg)
    assert np.all(np.abs(floats(got) - ref) <= tol), np.max(np.abs(floats(got) - ref) / tol)
    assert np.all(np.abs(lse - rlse) <= tol_lse) and np.all(np.abs(want_lse - rlse) <= tol_lse)
    # and the library's parity bar, which a factor left out or taken twice cannot meet
    for x, what in ((got, "4-bit"), (want, "bf16")):
        assert_parity(floats(x), ref, max_abs=np.inf, what=f"{cfg.name} {what}")
    # the bf16 call: its weights' and v^C's 2^-8 in place of 2^-11, by the same formula
    wide = tol + (2 * 2.0 ** -8 - 2.0 ** -10) * mass(codes, scales, d, cfg)
    assert np.all(np.abs(floats(want) - ref) <= wide), np.max(np.abs(floats(want) - ref) / wide)


def mass(codes, scales, d, cfg):
    """sum_j a_j |v_j| in 64 bits, [B*s][H][128]."""
    f, s, H = oracle.bf16_to_f64, cfg.s, cfg.H
    qr = oracle.rope_rows(f(d["q_rope"]).reshape(-1, 64), np.repeat(d["q_pos"], H)).reshape(cfg.T, H, 64)
    qn, wk, wv, out = f(d["q_nope"]), f(d["w_uk"]), f(d["w_uv"]), np.zeros((cfg.T, H, 128))
    for b, L in enumerate(cfg.seq_lens):
        pages = d["block_table"][b, :(L + 63) // 64]
        rows = oracle.int4_values(codes[pages], scales[pages]).reshape(-1, 576)[:L]
        mine = slice(b * s, b * s + s)
        hide = np.arange(L)[None] > np.arange(L - s, L)[:, None]
        for h in range(H):
            z = (qn[mine, h] @ (rows[:, :512] @ wk[h].T).T + qr[mine, h] @ rows[:, 512:].T) / np.sqrt(192.0)
            z[hide] = -np.inf
            e = np.exp(z - z.max(-1, keepdims=True))
            out[mine, h] = (e / e.sum(-1, keepdims=True)) @ np.abs(rows[:, :512] @ wv[h].T)
    return out
