"""Range of the 4-bit prefill's f16 v^C: its power of two belongs to a sequence and
a head, so large latents of one sequence or large weights of one head cost the
others nothing.  Tolerances are test_gpu_int4's (plain_prefill), whose fixed step
of small v^C is taken from the latents of the row's own sequence and the weights of
its own head."""
import dataclasses

import numpy as np
import pytest

import mla_workloads as W
import oracle
from test_gpu_int4 import C, M, floats, plain_prefill, random_cache, run_prefill  # noqa: F401

pytestmark = pytest.mark.gpu


def rows_of(d, b, L):
    """(page, slot) of sequence b's rows."""
    j = np.arange(L)
    return d["block_table"][b, j // 64], j % 64


def per_sequence_and_head(codes, scales, d, cfg):
    """plain_prefill of every sequence and head for itself."""
    out, tol = np.zeros((2, cfg.T, cfg.H, 128))
    lse, tol_lse = np.zeros((2, cfg.T, cfg.H))
    for b, L in enumerate(cfg.seq_lens):
        mine = slice(b * cfg.s, (b + 1) * cfg.s)
        for h in range(cfg.H):
            one = dataclasses.replace(cfg, B=1, H=1, seq_lens=(L,))
            part = dict(block_table=d["block_table"][b:b + 1], q_pos=d["q_pos"][mine], q_nope=d["q_nope"][mine, h:h + 1],
                        q_rope=d["q_rope"][mine, h:h + 1], w_uk=d["w_uk"][h:h + 1], w_uv=d["w_uv"][h:h + 1])
            o, l, t, tl = plain_prefill(codes, scales, part, one)
            out[mine, h], lse[mine, h], tol[mine, h], tol_lse[mine, h] = o[:, 0], l[:, 0], t[:, 0], tl[:, 0]
    return out, lse, tol, tol_lse


def test_a_huge_sequence_and_a_large_head_leave_the_others_their_bits(M):  # noqa: F811
    cfg = C("pr_bits", 16, [70, 300, 200], s=33, seed=80)
    d = W.make_decode_inputs(cfg, with_cache_pages=False)
    codes, scales = random_cache(d, 80)
    good, lse, err, _, _ = run_prefill(M, cfg, d, codes, scales, 300)
    assert err == 0
    # one row of sequence 1 as the writer stores infinities
    big_c, big_s = codes.copy(), scales.copy()
    page, slot = (x[150] for x in rows_of(d, 1, 300))
    big_c[page, slot, :256], big_s[page, slot, :32] = 0xFF, 255
    got, lse_b, err, _, _ = run_prefill(M, cfg, d, big_c, big_s, 300)
    keep = np.r_[:33, 66:99]
    assert err == 0 and np.array_equal(got[keep], good[keep]) and np.array_equal(lse_b[keep], lse[keep])
    assert not np.array_equal(got[33:66], good[33:66])
    # the weights of head 5 times 2^24
    w = oracle.bf16_to_f64(d["w_uv"])
    w[5] *= 2.0 ** 24
    got, lse_b, err, _, _ = run_prefill(M, cfg, dict(d, w_uv=W.f32_to_bf16_bits(w.astype(np.float32))), codes, scales, 300)
    heads = np.arange(16) != 5
    assert err == 0 and np.array_equal(got[:, heads], good[:, heads]) and np.array_equal(lse_b, lse)
    assert np.array_equal(floats(got[:, 5]), floats(good[:, 5]) * 2.0 ** 24)


@pytest.mark.parametrize("cfg", [C("pr_h16", 16, [40, 300, 129, 260], s=37, seed=81),
                                 C("pr_h48", 48, [333, 190], s=130, seed=82)], ids=lambda c: c.name)
def test_latents_and_weights_of_very_different_size(M, cfg):  # noqa: F811
    """Sequences whose latents are 2^-12 to 2^16 in size and heads whose weights span
    2^-20 to 2^20, against the formula."""
    d = W.make_decode_inputs(cfg, with_cache_pages=False)
    codes, scales = random_cache(d, cfg.seed)
    rng = np.random.default_rng(cfg.seed)
    for b, L in enumerate(cfg.seq_lens):
        page, slot = rows_of(d, b, L)
        scales[page, slot, :32] = rng.integers(0, 10, (L, 32)) + (16, 232)[b % 2]      # 2^-13 .. and 2^14 ..
    w = oracle.bf16_to_f64(d["w_uv"]) * np.exp2(rng.integers(-20, 21, cfg.H))[:, None, None]
    k = oracle.bf16_to_f64(d["w_uk"]) * 2.0 ** -14          # logits of ordinary size over the large latents
    d = dict(d, w_uv=W.f32_to_bf16_bits(w.astype(np.float32)), w_uk=W.f32_to_bf16_bits(k.astype(np.float32)))
    got, lse, err, _, _ = run_prefill(M, cfg, d, codes, scales, max(cfg.seq_lens))
    assert err == 0
    ref, rlse, tol, tol_lse = per_sequence_and_head(codes, scales, d, cfg)
    assert np.all(np.abs(floats(got) - ref) <= tol), np.max(np.abs(floats(got) - ref) / tol)
    assert np.all(np.abs(lse - rlse) <= tol_lse), np.max(np.abs(lse - rlse) / tol_lse)
