"""GPU parity of the 4-bit latent cache: the writer and the row reader bit for
bit against the oracle's quantizer and values, decode against a plain 64-bit
evaluation of the formula on the rows the cache stands for, and prefill against
the same and against the bf16 prefill of those rows, whose error it stays under.

Decode tolerance, element by element.  With a_j the exact weights, c_j the
cached latents and A = sum_j a_j |c_j|: the kernel rounds its weights to bf16
(at most 2^-8 relative each, so 2^-8 A) and the output (2^-8 |out|); a logit is
a sum of 576 products in fp32, off by at most dl = 576 * 2^-23 * scale *
max_j sum |q||row_j| if every addition loses a unit in the last place, which
changes a weight by at most 2 dl relative; the exponentials (2^-22), the sums
of weights and of weighted latents in fp32 (one addition per tile and at most
64 inside one, 2^-23 each) and the merge of partial results stay below 2^-14 A
together at these lengths.  lse: dl, and 2^-16 + 2^-22 |lse| for the exponentials,
the sum and the logarithm.
"""
import numpy as np
import pytest

import mla_workloads as W
import oracle
from _gpu_setup import assert_parity, host_bits, i32, torch_bits

pytestmark = pytest.mark.gpu

SCALE = 1.0 / np.sqrt(192.0)


@pytest.fixture(scope="module")
def M():
    import head_latent_attention_10_b200 as M
    M.load_library()
    return M


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def random_cache(d, seed):
    """Pages of random codes (all 16) and scale bytes (2^-3 .. 2^0); slots no
    token maps to hold 0xFF, the largest value there is."""
    rng = np.random.default_rng(seed)
    nb, N = d["num_blocks"], d["tok_seq"].size
    codes = np.full((nb, 64, 288), 0xFF, np.uint8)
    scales = np.full((nb, 64, 36), 0xFF, np.uint8)
    blk, slot = d["block_table"][d["tok_seq"], d["tok_pos"] // 64], d["tok_pos"] % 64
    codes[blk, slot] = rng.integers(0, 256, (N, 288), dtype=np.uint8)
    scales[blk, slot] = rng.integers(96, 121, (N, 36), dtype=np.uint8)
    return codes, scales


def bf16_cache(codes, scales):
    """The same pages as a bf16 cache (exact)."""
    return W.f32_to_bf16_bits(oracle.int4_values(codes, scales).astype(np.float32))


def plain_decode(codes, scales, d, s, q, seq_lens=None):
    """softmax(scale q . row) c in 64 bits: out [B*s][H][512], lse, and the two
    tolerances of the module's docstring."""
    lens = d["seq_lens"] if seq_lens is None else seq_lens
    T, H, _ = q.shape
    out, tol = np.zeros((T, H, 512)), np.zeros((T, H, 512))
    lse, tol_lse = np.full((T, H), -np.inf), np.zeros((T, H))
    for b, L in enumerate(lens):
        pages = d["block_table"][b, :(L + 63) // 64]
        rows = oracle.int4_values(codes[pages], scales[pages]).reshape(-1, 576)[:L]
        for t in range(s):
            n, r = L - s + t + 1, b * s + t
            if n <= 0:
                continue
            z = SCALE * (q[r] @ rows[:n].T)
            m = z.max(-1, keepdims=True)
            e = np.exp(z - m)
            a = e / e.sum(-1, keepdims=True)
            out[r] = a @ rows[:n, :512]
            lse[r] = m[:, 0] + np.log(e.sum(-1))
            dl = 576 * 2.0 ** -23 * SCALE * (np.abs(q[r]) @ np.abs(rows[:n]).T).max(-1)
            A = a @ np.abs(rows[:n, :512])
            tol[r] = (2.0 ** -8 + 2.0 ** -14 + 2 * dl[:, None]) * A + 2.0 ** -8 * (1 + 2.0 ** -8) * np.abs(out[r])
            tol_lse[r] = dl + 2.0 ** -16 + 2.0 ** -22 * np.abs(lse[r])
    return out, lse, tol, tol_lse


def run_decode(M, cfg, d, codes, scales, q_bits, flags=0, seq_lens=None, table=None, lse=True):
    import torch
    dims = M.dims(cfg.H)
    bt = d["block_table"] if table is None else table
    lat = torch.full((cfg.T, cfg.H, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    out_lse = torch.full((cfg.T, cfg.H), float("nan"), dtype=torch.float32, device="cuda") if lse else None
    ws = torch.full((M.mla_decode_workspace_size(dims, cfg.B, cfg.s, bt.shape[1] * 64),), 0xA5, dtype=torch.uint8,
                    device="cuda")
    M.mla_decode_int4(dims, torch_bits(q_bits), dev(codes), dev(scales), dev(bt),
                      dev(d["seq_lens"] if seq_lens is None else seq_lens), cfg.s, lat, out_lse, ws, flags=flags)
    torch.cuda.synchronize()
    return host_bits(lat), None if out_lse is None else out_lse.cpu().numpy(), M.mla_decode_error(ws)


def floats(bits):
    return W.bf16_bits_to_f32(bits).astype(np.float64)


def C(name, H, lens, s=1, paged=True, seed=0):
    return W.MLAConfig(name, B=len(lens), s=s, H=H, L=0, paged=paged, seed=500 + seed, d_model=2048,
                       seq_lens=tuple(lens))


DECODE = [
    C("one_token", 16, [1]),
    C("h16_ragged", 16, [1000, 65, 1, 64, 63, 129], seed=1),
    C("h48", 48, [700, 191], seed=2),
    C("h64_two_queries", 64, [2, 300, 1500, 3], s=2, seed=3),
    C("h80_three_queries", 80, [3, 190, 640], s=3, seed=4),
    C("h128_ragged", 128, [700, 129, 63, 1, 2], seed=5),
    C("h128_two_queries", 128, [300, 2, 1500], s=2, seed=6),
    C("h16_nine_queries", 16, [9, 200], s=9, seed=7),
    C("h64_many_splits", 64, [2500, 1100], seed=8),
    C("h32_contiguous", 32, [257, 64], paged=False, seed=9),
    C("h16_many_short", 16, list(range(1, 180)), seed=10),
    C("h16_one_long", 16, [9000], seed=11),
    C("h32_two_queries_long", 32, [4200, 2, 3900], s=2, seed=12),
    C("h128_some_pieces", 128, [1700, 1], seed=13),
]


@pytest.mark.parametrize("simple", [True, False], ids=["simple", "tensor_core"])
@pytest.mark.parametrize("cfg", DECODE, ids=lambda c: c.name)
def test_decode_against_the_formula(M, cfg, simple):
    d = W.make_decode_inputs(cfg, with_cache_pages=False)
    codes, scales = random_cache(d, cfg.seed)
    q = W.make_q_abs(cfg)
    got, lse, err = run_decode(M, cfg, d, codes, scales, q, M.MLA_FORCE_SIMPLE if simple else 0)
    assert err == 0
    ref, rlse, tol, tol_lse = plain_decode(codes, scales, d, cfg.s, oracle.bf16_to_f64(q))
    assert np.all(np.abs(floats(got) - ref) <= tol), np.max(np.abs(floats(got) - ref) / np.maximum(tol, 1e-30))
    assert np.all(np.abs(lse - rlse) <= tol_lse), np.max(np.abs(lse - rlse) / tol_lse)
    assert_parity(floats(got), ref, max_abs=np.inf, what=cfg.name)


@pytest.mark.parametrize("simple", [True, False], ids=["simple", "tensor_core"])
def test_decode_of_empty_and_short_sequences(M, simple):
    """Lengths 0 (in the middle and at the end) and below s: rows with no
    visible key are zero with lse = -inf and an error bit; the others are the
    formula's, and a null out_lse is accepted."""
    cfg = C("empty", 32, [200, 0, 70, 1, 0], s=2, seed=20)
    d = W.make_decode_inputs(cfg.with_(seq_lens=(200, 2, 70, 2, 2)), with_cache_pages=False)
    lens = np.array(cfg.seq_lens, np.int32)
    codes, scales = random_cache(d, 20)
    q = W.make_q_abs(cfg)
    flags = M.MLA_FORCE_SIMPLE if simple else 0
    got, lse, err = run_decode(M, cfg, d, codes, scales, q, flags, seq_lens=lens)
    assert err == M.MLA_DEVERR_SEQ_LEN
    ref, rlse, tol, tol_lse = plain_decode(codes, scales, d, 2, oracle.bf16_to_f64(q), lens)
    for r in (2, 3, 6, 8, 9):
        assert np.all(got[r] == 0) and np.all(np.isneginf(lse[r])), r
    see = np.isfinite(rlse)
    assert np.all(np.abs(floats(got) - ref) <= tol) and np.all(np.abs(lse[see] - rlse[see]) <= tol_lse[see])
    again, none, _ = run_decode(M, cfg, d, codes, scales, q, flags, seq_lens=lens, lse=False)
    assert none is None and np.array_equal(again, got)
    # every sequence empty
    got, lse, err = run_decode(M, cfg, d, codes, scales, q, flags, seq_lens=np.zeros(5, np.int32))
    assert np.all(got == 0) and np.all(np.isneginf(lse)) and err == M.MLA_DEVERR_SEQ_LEN


@pytest.mark.parametrize("simple", [True, False], ids=["simple", "tensor_core"])
def test_decode_reports_a_bad_block_and_a_length_past_the_table(M, simple):
    cfg = C("bad", 16, [300, 100], seed=21)
    d = W.make_decode_inputs(cfg, with_cache_pages=False)
    codes, scales = random_cache(d, 21)
    q = W.make_q_abs(cfg)
    flags = M.MLA_FORCE_SIMPLE if simple else 0
    good, _, _ = run_decode(M, cfg, d, codes, scales, q, flags)
    for bad in (d["num_blocks"], -7, 2 ** 31 - 1):
        bt = d["block_table"].copy()
        bt[0, 2] = bad
        got, _, err = run_decode(M, cfg, d, codes, scales, q, flags, table=bt)
        assert err == M.MLA_DEVERR_BLOCK_ID and np.array_equal(got[1], good[1])
    for L in (300 + 5 * 64, -1):
        got, _, err = run_decode(M, cfg, d, codes, scales, q, flags, seq_lens=np.array([L, 100], np.int32))
        assert err & M.MLA_DEVERR_SEQ_LEN and np.array_equal(got[1], good[1])
    with pytest.raises(M.MLAError) as e:
        run_decode(M, cfg, d, codes, scales, q, flags | M.MLA_SYNC_CHECK, seq_lens=np.array([0, 100], np.int32))
    assert e.value.status == M.MLA_ERR_DEVICE


def test_decode_with_large_logits_and_a_maximum_on_the_last_token(M):
    """Queries scaled so that the softmax is close to one-hot, the largest logit
    planted on each sequence's last token: the running maximum jumps on the
    last tile."""
    cfg = C("jump", 128, [900, 64, 130, 65], seed=22)
    d = W.make_decode_inputs(cfg, with_cache_pages=False)
    codes, scales = random_cache(d, 22)
    q = W.f32_to_bf16_bits(8.0 * W.bf16_bits_to_f32(W.make_q_abs(cfg)))
    for b, L in enumerate(cfg.seq_lens):
        pg = d["block_table"][b, (L - 1) // 64]
        row = np.sign(W.bf16_bits_to_f32(q[b, 0])).astype(np.float32)     # along head 0's query
        codes[pg, (L - 1) % 64], scales[pg, (L - 1) % 64] = (v[0] for v in oracle.int4_quantize_rows(row[None] * 2))
    got, lse, err = run_decode(M, cfg, d, codes, scales, q)
    ref, rlse, tol, tol_lse = plain_decode(codes, scales, d, 1, oracle.bf16_to_f64(q))
    assert err == 0 and np.all(np.abs(floats(got) - ref) <= tol) and np.all(np.abs(lse - rlse) <= tol_lse)


def test_decode_bits_do_not_depend_on_page_order_or_on_the_run(M):
    cfg = C("order", 64, [2500, 1100, 60], seed=23)
    d = W.make_decode_inputs(cfg, with_cache_pages=False)
    codes, scales = random_cache(d, 23)
    q = W.make_q_abs(cfg)
    a, la, _ = run_decode(M, cfg, d, codes, scales, q)
    for flags in (0, M.MLA_DEBUG_COMBINE_ALL):
        b, lb, _ = run_decode(M, cfg, d, codes, scales, q, flags)
        assert np.array_equal(a, b) and np.array_equal(la, lb)
    bt = d["block_table"]
    order = bt[bt >= 0]
    ident = np.full_like(bt, -1)
    ident[bt >= 0] = np.arange(order.size)
    c, lc, _ = run_decode(M, cfg, d, codes[order], scales[order], q, table=ident)
    assert np.array_equal(a, c) and np.array_equal(la, lc)


def test_decode_of_full_sized_batches(M):
    """The benchmark's shapes, cut to fewer sequences: 16 heads and 128 heads at
    4,096 tokens, one long context; a sample of rows against the formula."""
    for cfg in (C("v2lite", 16, [4096] * 64, seed=30), C("v2", 128, [4096] * 24, seed=31),
                C("long", 128, [40000, 33333], seed=32)):
        d = W.make_decode_inputs(cfg, with_cache_pages=False)
        codes, scales = random_cache(d, cfg.seed)
        q = W.make_q_abs(cfg)
        got, lse, err = run_decode(M, cfg, d, codes, scales, q)
        assert err == 0
        for b in (0, cfg.B // 2, cfg.B - 1):
            d1 = dict(d, block_table=d["block_table"][b:b + 1], seq_lens=d["seq_lens"][b:b + 1])
            ref, rlse, tol, tol_lse = plain_decode(codes, scales, d1, 1, oracle.bf16_to_f64(q[b:b + 1, ::5]))
            assert np.all(np.abs(floats(got[b:b + 1, ::5]) - ref) <= tol)
            assert np.all(np.abs(lse[b:b + 1, ::5] - rlse) <= tol_lse)


def test_stall_hook_reports_a_timeout(M):
    cfg = C("stall", 128, [700, 129], seed=24)
    d = W.make_decode_inputs(cfg, with_cache_pages=False)
    codes, scales = random_cache(d, 24)
    q = W.make_q_abs(cfg)
    good, _, _ = run_decode(M, cfg, d, codes, scales, q)
    _, _, err = run_decode(M, cfg, d, codes, scales, q, M.MLA_DEBUG_STALL)
    assert err & M.MLA_DEVERR_TIMEOUT
    again, _, err = run_decode(M, cfg, d, codes, scales, q)
    assert err == 0 and np.array_equal(again, good)


# ------------------------------------------------------------ writer, reader
def append(M, dims, rows_c, rows_k, seq, pos, table, nb, fill=0xFF, **kw):
    import torch
    codes = torch.full((nb, 64, 288), fill, dtype=torch.uint8, device="cuda")
    scales = torch.full((nb, 64, 36), fill, dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    M.mla_append_latent_int4(dims, torch_bits(rows_c), torch_bits(rows_k), i32(seq), i32(pos), i32(table), codes,
                             scales, err_word=err, **kw)
    torch.cuda.synchronize()
    return codes.cpu().numpy(), scales.cpu().numpy(), int(err.item())


@pytest.mark.parametrize("norm", [False, True], ids=["copy", "norm"])
@pytest.mark.parametrize("yarn", [0.0, 40.0], ids=["rope", "yarn"])
@pytest.mark.parametrize("lens", [(1,), (300,), (65, 1, 500, 64)], ids=["one", "long", "ragged"])
def test_writer_stores_the_bf16_writers_rows_quantized(M, lens, yarn, norm):
    """Codes and scales equal the oracle quantizer's on the rows that the bf16
    writer stores for the same tokens, bit for bit (positions far out too);
    slots of no token keep their fill."""
    import torch
    cfg = C("writer", 16, lens, seed=len(lens))
    d = W.make_decode_inputs(cfg, with_cache_pages=False)
    kw = {}
    if norm:
        w = W.f32_to_bf16_bits(np.random.default_rng(3).uniform(0.5, 2.0, 512).astype(np.float32))
        kw = dict(kv_norm_weight=torch_bits(w), kv_norm_eps=1e-6)
    far = 100 * 64
    table = np.full((cfg.B, 100 + d["block_table"].shape[1]), -1, np.int32)
    table[:, 100:] = d["block_table"]
    pos = d["tok_pos"] + far
    dims = M.dims(16, rope_scaling=yarn)
    codes, scales, err = append(M, dims, d["c_kv"], d["k_rope"], d["tok_seq"], pos, table, d["num_blocks"], **kw)
    assert err == 0
    bf = torch.full((d["num_blocks"], 64, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    M.mla_append_latent(dims, torch_bits(d["c_kv"]), torch_bits(d["k_rope"]), i32(d["tok_seq"]), i32(pos), i32(table),
                        bf, **kw)
    blk, slot = table[d["tok_seq"], pos // 64], pos % 64
    want_c, want_s = oracle.int4_quantize_rows(floats(host_bits(bf))[blk, slot])
    assert np.array_equal(codes[blk, slot], want_c) and np.array_equal(scales[blk, slot], want_s)
    if not yarn and not norm:       # and the rows are the definition's: rotated in 64 bits, rounded to bf16
        kr = oracle.rope_rows(oracle.bf16_to_f64(d["k_rope"]), pos)
        row = np.concatenate([floats(d["c_kv"]), floats(W.f32_to_bf16_bits(kr.astype(np.float32)))], axis=1)
        assert np.array_equal(oracle.int4_quantize_rows(row)[0], codes[blk, slot])
    free = np.ones((d["num_blocks"], 64), bool)
    free[blk, slot] = False
    assert np.all(codes[free] == 0xFF) and np.all(scales[free] == 0xFF)


def test_writer_on_unusual_values(M):
    """Zero groups, tiny, huge, NaN and infinite values, ties: the oracle's codes
    (at position 0, where the rotation is the identity)."""
    rng = np.random.default_rng(5)
    x = rng.standard_normal((64, 576)).astype(np.float32) * np.exp2(rng.integers(-40, 40, (64, 576))).astype(np.float32)
    x[0], x[1], x[2] = 0.0, 1e-30, 3e38
    x[3, ::7], x[4, ::5], x[5, ::3] = np.nan, np.inf, -np.inf
    x[6] = np.arange(576) % 16 / 2.0 - 3.5
    x[7, 512:] = 0.0
    x[8:] = rng.standard_normal((56, 576))
    with np.errstate(over="ignore", invalid="ignore"):
        bits = W.f32_to_bf16_bits(x)
    bits[3, ::7] = 0x7FC0
    # a NaN or an infinity beside its pair's partner turns both at any position: keys stay finite here
    bits[:6, 512:] = bits[8:14, 512:]
    T = 64
    table = np.arange(T, dtype=np.int32)[:, None]
    codes, scales, err = append(M, M.dims(16), bits[:, :512].copy(), bits[:, 512:].copy(), np.arange(T), np.zeros(T),
                                table, T)
    want_c, want_s = oracle.int4_quantize_rows(W.bf16_bits_to_f32(bits))
    assert err == 0 and np.array_equal(codes[:, 0], want_c) and np.array_equal(scales[:, 0], want_s)


@pytest.mark.parametrize("exp", [-12, 0, 18], ids=["low", "middle", "high"])
def test_writer_rounds_every_quotient(M, exp):
    """For a group's largest value at each of the 128 bf16 mantissas (exponents in
    the scale's range, and where it ends), every bf16 value from 2^-7 of it up, in
    both signs: the oracle's codes, ties among them."""
    top = np.arange(128, dtype=np.int64) + ((127 + exp) << 7)              # bf16 patterns
    below = np.array([np.arange(t - 7 * 128, t + 1) for t in top])         # 128 x 897
    sign = (np.arange(below.size).reshape(below.shape) % 2) << 15
    vals = np.concatenate([below | sign, np.zeros((128, 3), np.int64)], axis=1).reshape(128, 60, 15)
    groups = np.concatenate([np.broadcast_to(top[:, None, None], (128, 60, 1)), vals], axis=2).reshape(-1, 32, 16)
    T = groups.shape[0]
    latent, key = groups.reshape(T, 512).astype(np.uint16), np.zeros((T, 64), np.uint16)
    table = np.arange((T + 63) // 64, dtype=np.int32)[None]
    codes, scales, err = append(M, M.dims(16), latent, key, np.zeros(T), np.arange(T), table, table.size)
    want_c, want_s = oracle.int4_quantize_rows(W.bf16_bits_to_f32(np.concatenate([latent, key], axis=1)))
    assert err == 0 and np.array_equal(codes.reshape(-1, 288)[:T], want_c)
    assert np.array_equal(scales.reshape(-1, 36)[:T], want_s)


def test_writer_and_reader_report_bad_places(M):
    import torch
    rng = np.random.default_rng(6)
    c, k = (W.f32_to_bf16_bits(rng.standard_normal((6, n)).astype(np.float32)) for n in (512, 64))
    table = np.array([[2, 9], [0, -1]], np.int32)      # 3 blocks: entry 9 and -1 are bad
    seq, pos = np.array([0, 0, 1, 1, 2, -1]), np.array([5, 64, 63, 64, 0, 0])
    codes, scales, err = append(M, M.dims(16), c, k, seq, pos, table, 3)
    assert err == M.MLA_DEVERR_BLOCK_ID | M.MLA_DEVERR_SEQ_LEN
    touched = np.zeros((3, 64), bool)
    touched[2, 5] = touched[0, 63] = True
    assert np.array_equal(np.any(codes != 0xFF, axis=2), touched)
    rows = torch.full((8, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    seq, pos = np.array([1, 0, 0, 7, 0, 0, 1, 0]), np.array([63, 5, 64, 0, -1, 128, 63, 5])
    M.mla_gather_latent_int4(M.dims(16), dev(codes), dev(scales), i32(seq), i32(pos), i32(table), rows, err_word=word)
    got = floats(host_bits(rows))
    val = oracle.int4_values(codes, scales)
    assert np.array_equal(got[[0, 1, 6, 7]], np.stack([val[0, 63], val[2, 5], val[0, 63], val[2, 5]]))
    assert np.all(got[2:6] == 0) and int(word.item()) == M.MLA_DEVERR_BLOCK_ID | M.MLA_DEVERR_SEQ_LEN


@pytest.mark.parametrize("T", [1, 3, 72, 1000, 5000])
def test_reader_returns_the_stored_values(M, T):
    """Any order, repeats allowed, every code and scale byte."""
    import torch
    rng = np.random.default_rng(T)
    codes, scales = rng.integers(0, 256, (9, 64, 288), dtype=np.uint8), rng.integers(0, 256, (9, 64, 36), dtype=np.uint8)
    table = rng.permutation(9).astype(np.int32).reshape(3, 3)
    seq, pos = rng.integers(0, 3, T).astype(np.int32), rng.integers(0, 192, T).astype(np.int32)
    rows = torch.full((T + 1, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    M.mla_gather_latent_int4(M.dims(16), dev(codes), dev(scales), i32(seq), i32(pos), i32(table), rows[:T])
    want = oracle.int4_values(codes, scales)[table[seq, pos // 64], pos % 64]
    assert np.array_equal(floats(host_bits(rows[:T])), want) and np.all(floats(host_bits(rows[T:])) == 7.0)


# ------------------------------------------------------------------- prefill
def run_prefill(M, cfg, d, codes, scales, max_len, rotate=True, lens=None):
    import torch
    dims = M.dims(cfg.H)
    out = torch.full((cfg.T, cfg.H, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((cfg.T, cfg.H), float("nan"), dtype=torch.float32, device="cuda")
    ws = torch.empty(M.mla_prefill_workspace_size(dims, cfg.B, cfg.s, max_len), dtype=torch.uint8, device="cuda")
    q_pos = i32(d["q_pos"]) if rotate else None
    args = (torch_bits(d["q_nope"]), torch_bits(d["q_rope"]), q_pos, torch_bits(d["w_uk"]), torch_bits(d["w_uv"]))
    rest = (dev(d["block_table"]), dev(d["seq_lens"] if lens is None else lens), cfg.s, max_len, out, lse, ws)
    M.mla_prefill_int4(dims, *args, dev(codes), dev(scales), *rest)
    got, glse, err = host_bits(out), lse.cpu().numpy(), M.mla_decode_error(ws)
    M.mla_prefill(dims, *args, torch_bits(bf16_cache(codes, scales)), *rest)
    return got, glse, err, host_bits(out), lse.cpu().numpy()


def plain_prefill(codes, scales, d, cfg):
    """The expanded form in 64 bits, out [B*s][H][128] and lse, with tolerances:
    k^C, the rotated q^R and the output are rounded to bf16 (2^-8 relative each),
    v^C and the weights to f16 (2^-11 each) and sums of 512 and 192 products are
    taken in fp32 (2^-23 relative to the sum of magnitudes each addition), so with
    kb, vb the sums of magnitudes in k and v, a logit is off by at most dl = scale
    (2^-8 |q||k| + (512 + 192) 2^-23 |q| kb), which moves a weight by 2 dl.  Below
    f16's normal numbers the step is fixed: a weight times 2^7 is off by 2^-25 (the
    row's largest is 1 or more, so 2^-32 of the sum), and a v^C times 2^-e by 2^-25,
    where 2^(15 + e) is less than 4 times 512 times the largest latent and weight."""
    f, s, H = oracle.bf16_to_f64, cfg.s, cfg.H
    qr = oracle.rope_rows(f(d["q_rope"]).reshape(-1, 64), np.repeat(d["q_pos"], H)).reshape(cfg.T, H, 64)
    qn, wk, wv = f(d["q_nope"]), f(d["w_uk"]), f(d["w_uv"])
    out, tol = np.zeros((cfg.T, H, 128)), np.zeros((cfg.T, H, 128))
    lse, tol_lse = np.zeros((cfg.T, H)), np.zeros((cfg.T, H))
    all_rows = [oracle.int4_values(codes[p], scales[p]).reshape(-1, 576)[:L] for p, L in
                ((d["block_table"][b, :(L + 63) // 64], L) for b, L in enumerate(cfg.seq_lens))]
    low = 2.0 ** -29 * max(np.abs(r[:, :512]).max() for r in all_rows) * np.abs(wv).max()
    for b, L in enumerate(cfg.seq_lens):
        rows = all_rows[b]
        lat, key, mine = rows[:, :512], rows[:, 512:], slice(b * s, b * s + s)
        hide = np.arange(L)[None] > np.arange(L - s, L)[:, None]
        for h in range(H):
            k, v = lat @ wk[h].T, lat @ wv[h].T
            kb, vb = np.abs(lat) @ np.abs(wk[h]).T, np.abs(lat) @ np.abs(wv[h]).T
            z = SCALE * (qn[mine, h] @ k.T + qr[mine, h] @ key.T)
            z[hide] = -np.inf
            m = z.max(-1, keepdims=True)
            e = np.exp(z - m)
            a = e / e.sum(-1, keepdims=True)
            rot = np.abs(qr[mine, h]) @ np.abs(key).T
            dl = SCALE * (2.0 ** -8 * (np.abs(qn[mine, h]) @ np.abs(k).T + rot)
                          + 704 * 2.0 ** -23 * (np.abs(qn[mine, h]) @ kb.T + rot))
            dl[hide] = 0
            dl = dl.max(-1)
            out[mine, h], lse[mine, h] = a @ v, m[:, 0] + np.log(e.sum(-1))
            tol[mine, h] = ((2.0 ** -10 + 2.0 ** -14 + 2 * dl[:, None]) * (a @ np.abs(v)) + 512 * 2.0 ** -23 * (a @ vb)
                            + low + 2.0 ** -32 * np.abs(v).sum(0)
                            + 2.0 ** -8 * (1 + 2.0 ** -7) * np.abs(out[mine, h]))
            tol_lse[mine, h] = dl + 2.0 ** -16 + 2.0 ** -22 * np.abs(lse[mine, h])
    return out, lse, tol, tol_lse


@pytest.mark.parametrize("cfg", [C("p_one", 16, [1]), C("p_ragged", 16, [40, 300, 129], s=37, seed=40),
                                 C("p_chunk", 48, [190, 333], s=130, seed=41), C("p_128", 128, [257], s=200, seed=42)],
                         ids=lambda c: c.name)
def test_prefill_is_the_formula_on_the_stored_rows(M, cfg):
    """Element by element, and within the library's parity bar.  mla_prefill over
    the same rows rounds v^C and the weights to bf16 as well: with many keys its
    error is larger."""
    d = W.make_decode_inputs(cfg, with_cache_pages=False)
    codes, scales = random_cache(d, cfg.seed)
    got, lse, err, want, want_lse = run_prefill(M, cfg, d, codes, scales, max(cfg.seq_lens))
    assert err == 0
    ref, rlse, tol, tol_lse = plain_prefill(codes, scales, d, cfg)
    assert np.all(np.abs(floats(got) - ref) <= tol), np.max(np.abs(floats(got) - ref) / tol)
    assert np.all(np.abs(lse - rlse) <= tol_lse), np.max(np.abs(lse - rlse) / tol_lse)
    assert np.all(np.abs(want_lse - rlse) <= tol_lse)
    _, rel = assert_parity(floats(got), ref, max_abs=np.inf, what=cfg.name)
    _, rel16 = assert_parity(floats(want), ref, max_abs=np.inf, what=cfg.name + " bf16")
    assert min(cfg.seq_lens) < 40 or rel < rel16


def test_prefill_keeps_the_range_of_its_weights(M):
    """v^C is held in f16 under a power of two taken from the operands: weights
    2^n times as large give 2^n times the output, to the bit, and an infinite
    weight of one head leaves the other heads' bits alone."""
    cfg = C("p_range", 16, [70, 200], s=33, seed=44)
    d = W.make_decode_inputs(cfg, with_cache_pages=False)
    codes, scales = random_cache(d, 44)
    good, lse, err, _, _ = run_prefill(M, cfg, d, codes, scales, 200)
    assert err == 0
    for n in (-60, 20, 60):
        w = oracle.bf16_to_f64(d["w_uv"]) * 2.0 ** n
        got, lse_n, err, _, _ = run_prefill(M, cfg, dict(d, w_uv=W.f32_to_bf16_bits(w.astype(np.float32))), codes,
                                            scales, 200)
        assert err == 0 and np.array_equal(floats(got), floats(good) * 2.0 ** n) and np.array_equal(lse, lse_n)
    w = d["w_uv"].copy()
    w[3, 5, 7] = 0x7F80
    got, _, err, _, _ = run_prefill(M, cfg, dict(d, w_uv=w), codes, scales, 200)
    assert err == 0 and not np.isfinite(floats(got)[:, 3, 5]).any()
    keep = np.ones((16, 128), bool)
    keep[3, 5] = False
    assert np.array_equal(got[:, keep], good[:, keep])
    # the largest scale there is in every latent group
    big = scales.copy()
    big[..., :32] = 255
    got, _, err, _, _ = run_prefill(M, cfg, dict(d, q_nope=np.zeros_like(d["q_nope"])), codes, big, 200)
    ref, _, tol, _ = plain_prefill(codes, big, dict(d, q_nope=np.zeros_like(d["q_nope"])), cfg)
    assert err == 0 and np.all(np.abs(floats(got) - ref) <= tol)


def test_prefill_refuses_lengths_it_cannot_hold_and_skips_bad_blocks(M):
    cfg = C("p_bad", 16, [100, 70], s=20, seed=43)
    d = W.make_decode_inputs(cfg, with_cache_pages=False)
    codes, scales = random_cache(d, 43)
    good = run_prefill(M, cfg, d, codes, scales, 100)[0]
    for L in (19, 101, 10 ** 6, -3):
        got, lse, err, _, _ = run_prefill(M, cfg, d, codes, scales, 100, lens=np.array([L, 70], np.int32))
        assert err == M.MLA_DEVERR_SEQ_LEN and np.all(got[:20] == 0) and np.all(np.isneginf(lse[:20]))
        assert np.array_equal(got[20:], good[20:])
    bt = d["block_table"].copy()
    bt[0, 1] = d["num_blocks"]
    got, _, err, _, _ = run_prefill(M, cfg, dict(d, block_table=bt), codes, scales, 100)
    assert err == M.MLA_DEVERR_BLOCK_ID and np.array_equal(got[20:], good[20:])


def test_prefill_of_many_short_and_invalid_sequences(M):
    """More items than SMs, most of one key tile; runs of sequences that are too
    short for the chunk (zero rows) between and around the others, which keep the
    formula's results; and a batch with no valid sequence at all."""
    rng = np.random.default_rng(45)
    lens = rng.integers(3, 190, 300)
    cfg = C("many", 16, lens.tolist(), s=3, seed=45)
    d = W.make_decode_inputs(cfg, with_cache_pages=False)
    codes, scales = random_cache(d, 45)
    ref, rlse, tol, tol_lse = plain_prefill(codes, scales, d, cfg)
    for bad in (np.r_[:120, 150:153, 290:300], np.r_[rng.permutation(300)[:150]], np.r_[1:300], np.r_[:300]):
        now = lens.astype(np.int32)
        now[bad] = rng.integers(-1, 3, bad.size)
        got, lse, err, want, _ = run_prefill(M, cfg, d, codes, scales, int(lens.max()), lens=now)
        dead = np.zeros(300, bool)
        dead[bad] = True
        dead = np.repeat(dead, 3)
        assert err == M.MLA_DEVERR_SEQ_LEN
        assert np.all(got[dead] == 0) and np.all(np.isneginf(lse[dead])) and np.all(want[dead] == 0)
        assert np.all(np.abs(floats(got) - ref)[~dead] <= tol[~dead])
        assert np.all(np.abs(lse - rlse)[~dead] <= tol_lse[~dead])


# --------------------------------------------------------------- all together
def test_a_served_sequence_end_to_end_eager_on_a_stream_and_in_a_graph(M):
    """A prompt is appended and prefilled, then tokens are appended and decoded
    one step at a time; each step is the formula's on the stored rows.  The last
    step, captured in a graph and replayed twice on another stream beside the
    same step run eagerly there, gives the eager step's bits."""
    import torch
    H, P, steps = 16, 150, 3
    cfg = C("served", H, [P + steps] * 2, seed=50)
    d = W.make_decode_inputs(cfg, with_cache_pages=False)
    pre = C("served", H, [P] * 2, s=P, seed=50)
    dp = W.make_decode_inputs(pre, with_cache_pages=False)
    dims, bt = M.dims(H), i32(d["block_table"])
    nb = d["num_blocks"]
    codes = torch.full((nb, 64, 288), 0xFF, dtype=torch.uint8, device="cuda")
    scales = torch.full((nb, 64, 36), 0xFF, dtype=torch.uint8, device="cuda")
    tok = {(int(b), int(p)): i for i, (b, p) in enumerate(zip(d["tok_seq"], d["tok_pos"]))}

    def add(places, stream=None):
        i = [tok[x] for x in places]
        a = (torch_bits(d["c_kv"][i]), torch_bits(d["k_rope"][i]), i32([b for b, _ in places]),
             i32([p for _, p in places]))
        return lambda: M.mla_append_latent_int4(dims, *a, bt, codes, scales)

    add([(b, p) for b in range(2) for p in range(P)])()
    dp["block_table"] = d["block_table"]
    dp["q_pos"] = np.tile(np.arange(P), 2).astype(np.int32)
    host = lambda: (codes.cpu().numpy(), scales.cpu().numpy())  # noqa: E731
    got, _, err, _, _ = run_prefill(M, pre, dp, *host(), P)
    ref, _, tol, _ = plain_prefill(*host(), dp, pre)
    assert err == 0 and np.all(np.abs(floats(got) - ref) <= tol)
    q = W.make_q_abs(cfg)
    lat = torch.empty(2, H, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(2, H, dtype=torch.float32, device="cuda")
    ws = torch.empty(M.mla_decode_workspace_size(dims, 2, 1, bt.shape[1] * 64), dtype=torch.uint8, device="cuda")
    qd, lens = torch_bits(q), torch.empty(2, dtype=torch.int32, device="cuda")

    for t in range(steps):
        lens.fill_(P + t + 1)
        step = add([(0, P + t), (1, P + t)])
        step()
        M.mla_decode_int4(dims, qd, codes, scales, bt, lens, 1, lat, lse, ws)
        torch.cuda.synchronize()
        n = np.full(2, P + t + 1, np.int32)
        ref, rlse, tol, tol_lse = plain_decode(*host(), d, 1, oracle.bf16_to_f64(q), n)
        assert np.all(np.abs(floats(host_bits(lat)) - ref) <= tol)
        assert np.all(np.abs(lse.cpu().numpy() - rlse) <= tol_lse)
    eager, before = host_bits(lat), host()

    side = torch.cuda.Stream()
    lat2, ws2 = torch.empty_like(lat), torch.empty_like(ws)
    lat3 = torch.empty_like(lat)
    rows = torch.empty(2, 576, dtype=torch.bfloat16, device="cuda")
    at = (i32([0, 1]), i32([P + steps - 1] * 2))
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step()
        M.mla_decode_int4(dims, qd, codes, scales, bt, lens, 1, lat2, None, ws)
        M.mla_gather_latent_int4(dims, codes, scales, *at, bt, rows)
    codes[bt[:, (P + steps - 1) // 64].long(), (P + steps - 1) % 64] = 0x11     # the replay writes them again
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(2):
            lat2.fill_(float("nan"))
            g.replay()
            M.mla_decode_int4(dims, qd, codes, scales, bt, lens, 1, lat3, None, ws2)
    torch.cuda.synchronize()
    assert np.array_equal(host_bits(lat2), eager) and np.array_equal(host_bits(lat3), eager)
    after = host()
    assert np.array_equal(after[0], before[0]) and np.array_equal(after[1], before[1])
    blk = d["block_table"][[0, 1], (P + steps - 1) // 64]
    assert np.array_equal(floats(host_bits(rows)), oracle.int4_values(*after)[blk, (P + steps - 1) % 64])


def test_two_decodes_at_once_on_two_streams(M):
    """Calls with workspaces of their own may overlap."""
    import torch
    cfgs = [C("two_a", 128, [900, 300], seed=60), C("two_b", 16, [2000, 17, 640], s=2, seed=61)]
    runs, want = [], []
    for cfg in cfgs:
        d = W.make_decode_inputs(cfg, with_cache_pages=False)
        codes, scales = random_cache(d, cfg.seed)
        q = W.make_q_abs(cfg)
        want.append(run_decode(M, cfg, d, codes, scales, q)[0])
        dims = M.dims(cfg.H)
        ws = torch.empty(M.mla_decode_workspace_size(dims, cfg.B, cfg.s, d["block_table"].shape[1] * 64),
                         dtype=torch.uint8, device="cuda")
        lat = torch.empty(cfg.T, cfg.H, 512, dtype=torch.bfloat16, device="cuda")
        runs.append((dims, torch_bits(q), dev(codes), dev(scales), dev(d["block_table"]), dev(d["seq_lens"]), cfg.s,
                     lat, None, ws))
    streams = [torch.cuda.Stream() for _ in cfgs]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, r in zip(streams, runs):
            with torch.cuda.stream(st):
                M.mla_decode_int4(*r)
    torch.cuda.synchronize()
    for r, w in zip(runs, want):
        assert np.array_equal(host_bits(r[7]), w)


def test_prefill_in_a_graph_and_on_two_streams(M):
    """A captured call takes its operands' range anew at each replay, and two calls
    with workspaces of their own may overlap: the eager calls' bits."""
    import torch
    runs, want = [], []
    for H, lens, q, seed in ((128, [300, 140], 140, 70), (16, [1000, 257, 64], 64, 71)):
        cfg = C("pf", H, lens, s=q, seed=seed)
        d = W.make_decode_inputs(cfg, with_cache_pages=False)
        codes, scales = random_cache(d, seed)
        dims, most = M.dims(H), max(lens)
        want.append(run_prefill(M, cfg, d, codes, scales, most)[0])
        ws = torch.empty(M.mla_prefill_workspace_size(dims, cfg.B, q, most), dtype=torch.uint8, device="cuda")
        out = torch.empty(cfg.T, H, 128, dtype=torch.bfloat16, device="cuda")
        w_uv = torch_bits(d["w_uv"])
        runs.append((dims, torch_bits(d["q_nope"]), torch_bits(d["q_rope"]), i32(d["q_pos"]), torch_bits(d["w_uk"]), w_uv,
                     dev(codes), dev(scales), dev(d["block_table"]), dev(d["seq_lens"]), q, most, out, None, ws))
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(10):
        for st, r in zip(streams, runs):
            with torch.cuda.stream(st):
                M.mla_prefill_int4(*r)
    torch.cuda.synchronize()
    for r, w in zip(runs, want):
        assert np.array_equal(host_bits(r[12]), w)
    r, graph = runs[0], torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.mla_prefill_int4(*r)
    for n in (0, 30, -30, 0):
        scale = 2.0 ** n
        r[5].mul_(scale)
        r[12].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(floats(host_bits(r[12])), floats(want[0]) * scale)
        r[5].mul_(1 / scale)
