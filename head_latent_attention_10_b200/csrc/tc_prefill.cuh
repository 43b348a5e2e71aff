// tc_prefill.cuh -- prefill of a chunk of s new query tokens per sequence in
// the expanded form (sm_100a): every head's keys and values are materialised
// from the cached latents,
//   k_{j,i} = [U^K_i c_j ; k^R_j],  v_{j,i} = U^V_i c_j,
//   o_{t,i} = sum_j softmax_j(q_{t,i} . k_{j,i} * scale) v_{j,i}
// (DeepSeek-V2 paper review, section 2: k^C = W^UK c^KV, v^C = W^UV c^KV;
// section 3: the decoupled RoPE key shared by the heads and the scale
// 1/sqrt(d_h + d_R); DeepSeek-V3 report summary, Method 1:
// k_{t,i} = [k^C_{t,i}; k^R_t]).  Query t of a sequence of L cached tokens
// sits at position L - s + t and sees the keys j <= L - s + t.
//
// With many queries per sequence the expanded form costs fewer flops than the
// absorbed one (2 (192 + 128) per query, key and head against 2 (576 + 512)),
// and the step is bound by the tensor cores: an online-softmax loop on
// tcgen05.  An item is (128-query tile, head i, sequence b), the tile as MMA
// M = 128; it streams 128-key tiles of K = [K^C | k^R] and V^C:
//   S(k) = Q K_k^T    N=128, K=192: 12 MMAs, Q read from TMEM
//   P(k) = exp2(S(k) scale log2 e - m)           one thread per query row
//   O   += P(k) V_k   N=128, K=128: 8 MMAs, P read from TMEM
// One CTA an SM takes items until none is left (the first by its index, more from a
// counter; within a head the longest rows first, so a head's K and V stay in L2).
// A CTA per item started each with 8,400 idle cycles (queries 3,200, the first
// logits 2,000, output 2,600, set-up 600) beside 2,050 a key tile; here the next
// item's queries and tiles are loaded ahead, and its first logits are formed while
// the last item's output is written (916 against 995 us for a call of 4,096 tokens
// x 128 heads).
// TMEM (512 columns): S(t) of the CTA's tile t in buffer t % 2 (columns 0-127,
// 128-255), P(t) written over the first 64 columns of its S buffer, O 256-383, Q
// 384-479 (192 bf16 per row).  With Q and P in TMEM, shared memory holds a 3-slot
// ring of K tiles (K^C 0-63, K^C 64-127, k^R; 48 KB each), in which an item's
// queries, of the same size, take the slot before its first tile until the softmax
// warps have moved them on (read from global memory, a row per thread, they took
// 7,000 cycles), and a 2-slot ring of V tiles (V^C 0-63, 64-127; 32 KB each), 208 KB,
// each ring fed by its own loader warp (0: K, 6: V) so that neither waits behind the
// other.
// Warp 1 keeps the logits one tile ahead: S(t+2) goes into buffer t % 2 once P(t) V
// has completed (S(t+2) overwrites P(t)), so the softmax warps (2-5) find the next
// tile's logits ready when they finish this one; warp 7 issues P(t) V as soon as
// P(t) is written.  Two issuing threads, because a thread's tcgen05.mma issue blocks
// while the tensor pipe is busy, and one thread would hold P(t+1) V back behind
// S(t+2).  Both are chosen by elect.sync: under a `lane == 0` branch the compiler
// takes 76 cycles to issue an MMA, more than its 64 in the pipe.  The causal mask
// applies to the tiles that straddle the diagonal; lazy rescaling as in the decode (O
// is rescaled in TMEM only when the running max grows by more than 8, after
// the previous P V has retired).  Every wait is bounded; no TMA load uses
// cluster multicast.
//
// What bounds a tile: two chains of about 2,000 cycles that take turns.  The softmax
// takes 1,500 a tile (its 128 exponentials a thread 1,024 of them in their pipe); P V
// and the S behind it 1,280 in the tensor pipe and about 600 of waits.  Eight softmax
// warps, two threads to a row, took as long (the exponentials' pipe is the same, and
// the two must exchange maxima).
//
// kHalfV: V^C and P are f16 instead of bf16 (the 4-bit cache's prefill).  The
// latents there are read exactly, and the two roundings to 8 bits of P and V^C
// would be two thirds of the output's squared error (its relative rms 0.0029, so
// 0.0021, of which the output's own rounding to bf16 is 0.0017; the rest is the
// rounding of K^C and the queries).  f16 needs its range kept: V^C is stored times
// 2^-e, with an e of each sequence and head from its largest latent and weight
// magnitudes (prefill_prepare_kernel), so that none overflows whatever the weights,
// and a sequence's outputs do not depend on the others of its batch.  P is formed as
// 2^7 p (p <= 2^8), which leaves weights down to 2^-21 their 11 bits.  Both factors are powers of two and come off in the epilogue.
#pragma once

#include <type_traits>

#include "dec_common.cuh"
#include "k_simple.cuh"
#include "tc_gemm.cuh"

namespace mla {

constexpr int kPfThreads = 256;                        // warps: 0 K loads, 1 S MMAs, 2-5 softmax, 6 V loads, 7 P V MMAs
constexpr int kPfChunk = 128 * 128;                    // [128 rows][64 bf16], 128-byte swizzle: 16 KB
constexpr int kPfKSlots = 3, kPfVSlots = 2;
constexpr int kPfRopeHeads = 16;                       // heads a thread of the set-up rotates one pair of
constexpr int kPfOffK = 0;                             // K slot j: chunks 3j .. 3j+2
constexpr int kPfOffV = kPfKSlots * 3 * kPfChunk;      // V slot j: 2 chunks
constexpr int kPfOffOut = kPfOffV + kPfVSlots * 2 * kPfChunk;   // 212,992: 32 output rows x 128 B of a softmax warp
constexpr int kPfOffBar = kPfOffOut + 4 * 32 * 128;
constexpr int kPfSmem = kPfOffBar + 384 + 1024;        // barriers and the item list, alignment slack
constexpr int kPfList = 8;                             // published items
constexpr int kPfReaders = 7;                          // S, V and P V warps, four softmax warps
constexpr float kPfHalfShift = 7.f;                    // log2 of the factor on f16 P
constexpr uint32_t kPfTmS = 0, kPfTmO = 256, kPfTmQ = 384;   // S/P buffers at 0 and 128

// Tensor maps of one call.  Rows of K^C, V^C and the gathered latents are
// [B * Lpad] long (sequence b at rows b * Lpad ..); outputs are [B][s][H][128]
// with the sequence as the outermost dimension, so a 128-row tile is clipped
// at the end of its own sequence.
struct PrefillMaps {
    CUtensorMap kc;    // K^C   {128, H, B Lpad}, box {64, 1, 128}
    CUtensorMap vc;    // V^C   {128, H, B Lpad}, box {64, 1, 128}
    CUtensorMap kr;    // gathered rows {576, B Lpad, 1}, box {64, 128, 1}, read at x = 512
    CUtensorMap out;   // out   {128, H, s, B}, box {64, 1, 32, 1}
    CUtensorMap qn;    // q_nope {128, H, s, B}, box {64, 1, 128, 1}
    CUtensorMap qr;    // rotated q_rope {64, H, s, B}, box {64, 1, 128, 1}
};

struct PrefillArgs {
    const int32_t *seq_lens;
    int *counter;                 // items taken beyond the first of each CTA (zeroed)
    int s, H, lpad, l_cap;        // l_cap: the largest valid sequence length
    int qtiles, items;            // 128-query tiles of a sequence; times heads and sequences
    float scale_log2;
    float *out_lse;               // [B][s][H] or null
    uint32_t *err;
    const uint32_t *max_lat, *max_w;   // kHalfV: largest magnitudes (bf16 patterns) of a sequence's latents, a head's U^V
    unsigned long long limit_ns;
};

// Number of 128-key tiles the query tile [q0, q0 + 128) of a sequence of L
// tokens sees (0 if the tile holds no query).
__device__ __forceinline__ int prefill_tiles(int q0, int s, int L)
{
    if (q0 >= s) return 0;
    const int last_q = min(q0 + 128, s) - 1;
    return (L - s + last_q) / 128 + 1;
}

__device__ __forceinline__ bool prefill_valid(int L, int s, int l_cap) { return L >= s && L <= l_cap; }

template <bool kHalfV>
__global__ void __launch_bounds__(kPfThreads, 1)
tc_prefill_kernel(const __grid_constant__ PrefillMaps maps, const PrefillArgs a)
{
    extern __shared__ uint8_t pf_smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(pf_smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kPfOffBar);
    uint64_t *k_full = bars;            // [3] K slot loaded (a key tile, or an item's queries)
    uint64_t *k_free = bars + 3;        // [3] S of the slot's tile done, or the queries in TMEM
    uint64_t *v_full = bars + 6;        // [2] V slot loaded
    uint64_t *v_free = bars + 8;        // [2] P V of the slot's tile done
    uint64_t *q_ready = bars + 10;      // Q in TMEM (4 softmax warps)
    uint64_t *s_full = bars + 11;       // [2] S(k) in buffer k % 2
    uint64_t *p_full = bars + 13;       // [2] P(k) in TMEM and O rescaled (4 softmax warps)
    uint64_t *pv_done = bars + 15;      // [2] P(k) V_k done
    uint64_t *done = bars + 17;         // both issuers' last MMAs done (teardown)
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 18);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + 19);
    volatile int *listed = reinterpret_cast<volatile int *>(bars + 20);   // items published
    volatile int *list = reinterpret_cast<volatile int *>(bars + 21);     // [kPfList]
    volatile int *read_to = list + kPfList;                               // [kPfReaders] items each has read

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kPfKSlots; ++i) {
            sm100::mbar_init(&k_full[i], 1);
            sm100::mbar_init(&k_free[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            sm100::mbar_init(&v_full[i], 1);
            sm100::mbar_init(&v_free[i], 1);
            sm100::mbar_init(&p_full[i], 4);
            sm100::mbar_init(&pv_done[i], 1);
        }
        sm100::mbar_init(q_ready, 4);
        sm100::mbar_init(&s_full[0], 1);
        sm100::mbar_init(&s_full[1], 1);
        sm100::mbar_init(done, 2);
        *abort_flag = *listed = 0;
        for (int i = 0; i < kPfReaders; ++i) read_to[i] = 0;
        sm100::fence_mbar_init();
        sm100::prefetch_tensormap(&maps.kc);
        sm100::prefetch_tensormap(&maps.vc);
        sm100::prefetch_tensormap(&maps.kr);
        sm100::prefetch_tensormap(&maps.qn);
        sm100::prefetch_tensormap(&maps.qr);
    }
    if (warp == 1) {
        sm100::tmem_alloc(tmem_slot, 512);
        sm100::tmem_relinquish();
    }
    sm100::tc_fence_before();
    __syncthreads();
    sm100::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const unsigned long long lim = a.limit_ns;
    const unsigned long long drain = lim > 200000000ull ? lim : 200000000ull;
    // launched with programmatic serialization: the expansions' outputs are read only
    // from here on.  (They hold no trigger, so this kernel starts when their last CTAs
    // exit: its launch overlaps them, its set-up hardly.)
    sm100::pdl_wait();

    // An item: 128 queries of one head of one sequence; within a head the longest rows
    // of the causal triangle first.
    struct Item {
        int head, b, q0, L, nk;   // nk: key tiles, 0 if the sequence is invalid; -1: no more items
    };
    auto item_of = [&](int n) -> Item {
        if (n >= a.items) return {0, 0, 0, 0, -1};
        const int hb = n / a.qtiles, q0 = 128 * (a.qtiles - 1 - (n - hb * a.qtiles)), b = hb / a.H;
        const int L = a.seq_lens[b];
        return {hb - b * a.H, b, q0, L, prefill_valid(L, a.s, a.l_cap) ? prefill_tiles(q0, a.s, L) : 0};
    };
    // bounded wait of one thread for a count in shared memory
    auto count_wait = [&](volatile int *cnt, int target) -> bool {
        unsigned long long t0 = 0;
        for (uint32_t i = 1; *cnt < target; ++i) {
            if (i & 255u) continue;
            const unsigned long long now = sm100::globaltimer_ns();
            if (t0 == 0) t0 = now;
            if (*abort_flag) return false;
            if (now - t0 > lim) {
                set_error(a.err, MLA_DEVERR_TIMEOUT);
                *abort_flag = 1;
                return false;
            }
        }
        return true;
    };
    // the CTA's item j, for reader `who`, by one thread
    auto item_at = [&](int j, int who, Item &it) -> bool {
        if (!count_wait(listed, j + 1)) return false;
        it = item_of(list[j % kPfList]);
        __threadfence_block();
        read_to[who] = j + 1;
        return true;
    };

    if (warp == 0) {
        // ------------------------------------ items, queries and K loads
        if (lane == 0) {
            int issued = 0;   // ring entries: an item's queries, then its key tiles
            auto publish = [&](int j, int n) -> bool {
                for (int i = 0; j >= kPfList && i < kPfReaders; ++i)   // the entry it replaces is read
                    if (!count_wait(&read_to[i], j - kPfList + 1)) return false;
                list[j % kPfList] = n;
                __threadfence_block();
                *listed = j + 1;
                return true;
            };
            auto entry = [&]() -> uint8_t * {
                const int sl = issued % kPfKSlots;
                if (issued >= kPfKSlots &&
                    !sm100::mbar_wait(&k_free[sl], ((issued / kPfKSlots) - 1) & 1, abort_flag, a.err, lim))
                    return nullptr;
                sm100::mbar_arrive_expect_tx(&k_full[sl], 3 * kPfChunk);
                ++issued;
                return smem + kPfOffK + 3 * sl * kPfChunk;
            };
            int n = blockIdx.x;
            bool ok = publish(0, n);
            for (int j = 0; ok && n < a.items; ++j) {
                const Item it = item_of(n);
                n = gridDim.x + atomicAdd(a.counter, 1);
                if (!publish(j + 1, n)) break;
                for (int k = -1; ok && k < it.nk && it.nk > 0; ++k) {
                    uint64_t *bar = &k_full[issued % kPfKSlots];
                    uint8_t *dst = entry();
                    if (!(ok = dst != nullptr)) break;
                    if (k < 0) {
                        sm100::tma_load_4d(&maps.qn, bar, dst, 0, it.head, it.q0, it.b);
                        sm100::tma_load_4d(&maps.qn, bar, dst + kPfChunk, 64, it.head, it.q0, it.b);
                        sm100::tma_load_4d(&maps.qr, bar, dst + 2 * kPfChunk, 0, it.head, it.q0, it.b);
                    } else {
                        const int r = it.b * a.lpad + 128 * k;
                        sm100::tma_load_3d(&maps.kc, bar, dst, 0, it.head, r);
                        sm100::tma_load_3d(&maps.kc, bar, dst + kPfChunk, 64, it.head, r);
                        sm100::tma_load_3d(&maps.kr, bar, dst + 2 * kPfChunk, kDc, r, 0);
                    }
                }
            }
            if (*abort_flag) {   // let the copies in flight land before the CTA can exit
                volatile int no_abort = 0;
                for (int g = issued - kPfKSlots < 0 ? 0 : issued - kPfKSlots; g < issued; ++g)
                    sm100::mbar_wait(&k_full[g % kPfKSlots], (g / kPfKSlots) & 1, &no_abort, a.err, drain);
            }
        }
    } else if (warp == 6) {
        // ----------------------------------------------------------- V loads
        if (lane == 0) {
            int t = 0;
            Item it;
            bool ok = true;
            for (int j = 0; ok && (ok = item_at(j, 0, it)) && it.nk >= 0; ++j)
                for (int k = 0; k < it.nk; ++k) {
                    const int sl = t & 1;
                    if (t >= 2 && !(ok = sm100::mbar_wait(&v_free[sl], ((t >> 1) - 1) & 1, abort_flag, a.err, lim))) break;
                    uint8_t *dst = smem + kPfOffV + 2 * sl * kPfChunk;
                    const int r = it.b * a.lpad + 128 * k;
                    sm100::mbar_arrive_expect_tx(&v_full[sl], 2 * kPfChunk);
                    sm100::tma_load_3d(&maps.vc, &v_full[sl], dst, 0, it.head, r);
                    sm100::tma_load_3d(&maps.vc, &v_full[sl], dst + kPfChunk, 64, it.head, r);
                    ++t;
                }
            if (*abort_flag) {
                volatile int no_abort = 0;
                for (int k = t - 2 < 0 ? 0 : t - 2; k < t; ++k)
                    sm100::mbar_wait(&v_full[k & 1], (k >> 1) & 1, &no_abort, a.err, drain);
            }
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------- S MMAs
        if (sm100::elect_one()) {
            const uint32_t idesc_s = sm100::idesc_bf16(128, 128, 0, 0);
            int g = 0, t = 0, q = 0;   // ring entries, tiles, items with tiles
            Item it;
            bool ok = true;
            for (int j = 0; ok && (ok = item_at(j, 1, it)) && it.nk >= 0; ++j) {
                if (it.nk == 0) continue;
                if (!(ok = sm100::mbar_wait(q_ready, q & 1, abort_flag, a.err, lim))) break;
                sm100::mbar_arrive(&k_free[g % kPfKSlots]);   // the queries' slot
                ++g;
                ++q;
                for (int k = 0; k < it.nk; ++k, ++g, ++t) {
                    // S(t) into buffer t % 2, over P(t - 2): that P V must have completed
                    const int sl = g % kPfKSlots;
                    ok = (t < 2 || sm100::mbar_wait(&pv_done[t & 1], ((t >> 1) - 1) & 1, abort_flag, a.err, lim)) &&
                         sm100::mbar_wait(&k_full[sl], (g / kPfKSlots) & 1, abort_flag, a.err, lim);
                    if (!ok) break;
                    sm100::tc_fence_after();
                    const uint32_t ka = sm100::smem_u32(smem + kPfOffK + 3 * sl * kPfChunk);
#pragma unroll
                    for (int step = 0; step < 12; ++step)      // q^C 0-63, q^C 64-127, q^R
                        sm100::umma_ts(tmem + kPfTmS + 128 * (t & 1), tmem + kPfTmQ + 8 * step,
                                       sm100::desc_kmajor(ka + (step >> 2) * kPfChunk + (step & 3) * 32, 128,
                                                          sm100::kSw128),
                                       idesc_s, step > 0);
                    sm100::umma_commit(&s_full[t & 1]);
                    sm100::umma_commit(&k_free[sl]);
                }
            }
            sm100::umma_commit(done);
        }
        __syncwarp();
    } else if (warp == 7) {
        // -------------------------------------------------------- P V MMAs
        if (sm100::elect_one()) {
            const uint32_t idesc_o = kHalfV ? sm100::idesc_f16(128, 128, 0, 1) : sm100::idesc_bf16(128, 128, 0, 1);
            int t = 0;
            Item it;
            bool ok = true;
            for (int j = 0; ok && (ok = item_at(j, 2, it)) && it.nk >= 0; ++j)
                for (int k = 0; k < it.nk; ++k, ++t) {
                    const int pb = t & 1;
                    ok = sm100::mbar_wait(&p_full[pb], (t >> 1) & 1, abort_flag, a.err, lim) &&
                         sm100::mbar_wait(&v_full[pb], (t >> 1) & 1, abort_flag, a.err, lim);
                    if (!ok) break;
                    sm100::tc_fence_after();
                    const uint64_t vd =
                        sm100::desc_mnmajor_sw128(sm100::smem_u32(smem + kPfOffV + 2 * pb * kPfChunk), kPfChunk);
#pragma unroll
                    for (int kq = 0; kq < 8; ++kq)           // 16 keys per MMA: 8 TMEM columns of P
                        sm100::umma_ts(tmem + kPfTmO, tmem + kPfTmS + 128 * pb + 8 * kq,
                                       vd + (uint64_t)((kq * 2048) >> 4), idesc_o, (k > 0 || kq > 0) ? 1u : 0u);
                    sm100::umma_commit(&pv_done[pb]);
                    sm100::umma_commit(&v_free[pb]);
                }
            sm100::umma_commit(done);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------ softmax
        // warp w owns TMEM lane quarter w % 4; thread = query row r
        const int qd = warp & 3;
        const int r = 32 * qd + lane;
        const uint32_t lane_off = (uint32_t)(32 * qd) << 16;
        const uint32_t tm_s = tmem + lane_off + kPfTmS;
        const uint32_t tm_o = tmem + lane_off + kPfTmO, tm_q = tmem + lane_off + kPfTmQ;
        const uint32_t stage = sm100::smem_u32(smem + kPfOffOut) + qd * 32 * 128;
        int g = 0, tile = 0;   // ring entries and tiles so far
        // an item's queries [q^C | rotated q^R] into TMEM (a row: 192 bf16 = 96 columns;
        // rows past the sequence's queries arrive as zeros)
        auto next_item = [&](int j, Item &it) -> bool {
            int n = 0;
            bool ok = true;
            if (lane == 0 && (ok = count_wait(listed, j + 1))) {
                n = list[j % kPfList];
                __threadfence_block();
                read_to[3 + qd] = j + 1;
            }
            if (!__all_sync(0xffffffffu, ok)) return false;
            it = item_of(__shfl_sync(0xffffffffu, n, 0));
            if (it.nk <= 0) return true;
            const int sl = g % kPfKSlots;
            if (!sm100::warp_wait(&k_full[sl], (g / kPfKSlots) & 1, abort_flag, a.err, lim)) return false;
            const uint32_t qs = sm100::smem_u32(smem + kPfOffK + 3 * sl * kPfChunk) + r * 128;
#pragma unroll 1
            for (int c = 0; c < 3; ++c) {
                uint4 v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = ld_shared_v4(qs + c * kPfChunk + ((e ^ (r & 7)) << 4));
                sm100::tmem_st32(tm_q + 32 * c, reinterpret_cast<const uint32_t *>(v));
            }
            sm100::tmem_wait_st();
            sm100::tc_fence_before();
            __syncwarp();
            if (lane == 0) sm100::mbar_arrive(q_ready);
            g += 1 + it.nk;
            return true;
        };
        Item it, nx;
        bool ok = next_item(0, it);
        for (int j = 0; ok && it.nk >= 0; ++j, it = nx) {
            const int t = it.q0 + r;
            const bool has_row = t < a.s;
            const int nvis = has_row ? it.L - a.s + t + 1 : 0;   // keys [0, nvis) visible to row t
            float m_run = -INFINITY, l_run = 0.f;
            for (int k = 0; k < it.nk; ++k, ++tile) {
                const int pb = tile & 1;
                ok = sm100::warp_wait(&s_full[pb], (tile >> 1) & 1, abort_flag, a.err, lim);
                if (!ok) break;
                sm100::tc_fence_after();
                uint32_t x[128];
#pragma unroll
                for (int c = 0; c < 128; c += 32) sm100::tmem_ld32(tm_s + 128 * pb + c, x + c);
                sm100::tmem_wait_ld();
                const int key0 = 128 * k;
                if (key0 + 128 > nvis) {
#pragma unroll
                    for (int c = 0; c < 128; ++c)
                        if (key0 + c >= nvis) x[c] = __float_as_uint(-INFINITY);
                }
                float mx = -INFINITY;
#pragma unroll
                for (int c = 0; c < 128; c += 4)
                    mx = fmaxf(mx, fmaxf(fmaxf(__uint_as_float(x[c]), __uint_as_float(x[c + 1])),
                                         fmaxf(__uint_as_float(x[c + 2]), __uint_as_float(x[c + 3]))));
                const float mt = mx * a.scale_log2;
                const bool grow = (mt != -INFINITY) && (m_run == -INFINITY || mt > m_run + kRescaleThreshold);
                const bool rescale = grow && m_run != -INFINITY;
                const float m_new = grow ? mt : m_run;
                const float corr = rescale ? ex2(m_run - m_new) : 1.f;
                l_run *= corr;
                m_run = m_new;
                float mu = (m_run == -INFINITY) ? 0.f : m_run;
                if (kHalfV) mu -= kPfHalfShift;
                float lsum = 0.f;
#pragma unroll
                for (int c = 0; c < 64; ++c) {
                    const float p0 = ex2(fmaf(__uint_as_float(x[2 * c]), a.scale_log2, -mu));
                    const float p1 = ex2(fmaf(__uint_as_float(x[2 * c + 1]), a.scale_log2, -mu));
                    lsum += p0 + p1;
                    x[c] = kHalfV ? pack_half2(p0, p1) : pack_bf162(p0, p1);
                }
                l_run += lsum;
                // P(k) over the first 64 columns of S(k), already read by this thread
                sm100::tmem_st32(tm_s + 128 * pb, x);
                sm100::tmem_st32(tm_s + 128 * pb + 32, x + 32);
                if (__any_sync(0xffffffffu, rescale)) {
                    // O holds the tiles before k: let P(k-1) V_{k-1} retire, then
                    // scale this thread's row in place
                    ok = sm100::warp_wait(&pv_done[(tile - 1) & 1], ((tile - 1) >> 1) & 1, abort_flag, a.err, lim);
                    if (!ok) break;
                    sm100::tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < 128; c += 32) {
                        uint32_t ov[32];
                        sm100::tmem_ld32(tm_o + c, ov);
                        sm100::tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * corr);
                        sm100::tmem_st32(tm_o + c, ov);
                    }
                }
                sm100::tmem_wait_st();
                sm100::tc_fence_before();
                __syncwarp();
                if (lane == 0) sm100::mbar_arrive(&p_full[pb]);
            }
            // every S of the item has been read: the next item's queries go in now, so
            // that its first logits are formed during this epilogue
            ok = ok && next_item(j + 1, nx);
            if (!ok) break;
            // epilogue: O / l as bf16, 64 columns at a time staged with 128-byte swizzle
            // and stored with TMA by each warp for itself
            if (it.nk > 0) {
                ok = sm100::warp_wait(&pv_done[(tile - 1) & 1], ((tile - 1) >> 1) & 1, abort_flag, a.err, lim);
                if (!ok) break;
                sm100::tc_fence_after();
            }
            const float inv = l_run > 0.f ? 1.f / l_run : 0.f;
            const float vf = kHalfV ? exp2_int(half_exponent(a.max_lat + it.b, a.max_w + it.head)) : 1.f;
            auto o_of = [&](uint32_t x) { return kHalfV ? __uint_as_float(x) * inv * vf : __uint_as_float(x) * inv; };
#pragma unroll 1
            for (int c = 0; c < 128; c += 32) {
                uint32_t ov[32];
                if (it.nk > 0) {
                    sm100::tmem_ld32(tm_o + c, ov);
                    sm100::tmem_wait_ld();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) ov[e] = 0u;
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int unit = ((c & 63) >> 3) + q;        // 16-byte unit of the 128-byte row
                    st_shared_v4(stage + lane * 128 + ((unit ^ (lane & 7)) << 4),
                                 make_uint4(pack_bf162(o_of(ov[8 * q]), o_of(ov[8 * q + 1])),
                                            pack_bf162(o_of(ov[8 * q + 2]), o_of(ov[8 * q + 3])),
                                            pack_bf162(o_of(ov[8 * q + 4]), o_of(ov[8 * q + 5])),
                                            pack_bf162(o_of(ov[8 * q + 6]), o_of(ov[8 * q + 7]))));
                }
                if ((c & 32) == 0) continue;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0 && it.q0 + 32 * qd < a.s) {
                    sm100::tma_store_4d(&maps.out, smem + kPfOffOut + qd * 32 * 128, c & 64, it.head, it.q0 + 32 * qd, it.b);
                    sm100::tma_store_commit();
                    sm100::tma_store_wait_read();
                }
                __syncwarp();
            }
            if (a.out_lse && has_row)
                a.out_lse[((long long)it.b * a.s + t) * a.H + it.head] =
                    l_run > 0.f ? (m_run + __log2f(l_run) - (kHalfV ? kPfHalfShift : 0.f)) * kLn2 : -INFINITY;
            // O is read: the next item's first P V may overwrite it
            sm100::tc_fence_before();
            __syncwarp();
        }
    }

    // ------------------------------------------------------------ teardown
    sm100::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        volatile int no_abort = 0;
        sm100::warp_wait(done, 0, &no_abort, a.err, drain);
        sm100::tc_fence_after();
        sm100::tmem_dealloc(tmem, 512);
    }
}

// The larger of each half's finite magnitudes, as bf16 patterns, over 8 values.
__device__ __forceinline__ uint32_t finite_max(uint4 v)
{
    auto fin = [](uint32_t x) { x &= 0x7FFF7FFFu; return x & __vcmpltu2(x, 0x7F807F80u); };
    return __vmaxu2(__vmaxu2(fin(v.x), fin(v.y)), __vmaxu2(fin(v.z), fin(v.w)));
}

// Prefill set-up, one launch of three kinds of CTAs (PrepareBlocks):
//   - each sequence's cached rows gathered through its block table into rows
//     [b * lpad, b * lpad + lpad) of a contiguous [576]-wide buffer (rows at or past
//     the sequence's length, and every row of an invalid sequence, are zero);
//   - the chunk's RoPE queries rotated to q_pos (copied when q_pos is null), a
//     warp taking one token's 32 pairs of up to 16 heads;
//   - kHalfV: the largest finite magnitudes, as bf16 patterns, of each sequence's
//     gathered latents (max_bits[b]) and of each head's weights w_uv (max_bits[B + i]):
//     maxima, which no order of the atomics changes.  A CTA's rows are one sequence's
//     (lpad is a multiple of 128, and 128 rows are 36 CTAs) and its weights one head's
//     (8 CTAs each).
// Every thread has one piece of work: phases one after the other in each thread
// left the memory waiting for the angles.  Rows: how the cache's rows are read as
// bf16 (Bf16Rows, Int4Rows).
struct PrepareBlocks {
    long long row_units, rope_units, w_units;   // 16-byte units; (token, heads, pair); 16-byte units
    unsigned rows, rope, weights;               // CTAs
    int B;
    PrepareBlocks(int B, int lpad, int s, int H, bool half_v)
        : row_units((long long)B * lpad * (kRow / 8)),
          rope_units((long long)B * s * ((H + kPfRopeHeads - 1) / kPfRopeHeads) * (kDr / 2)),
          w_units(half_v ? (long long)H * kDh * kDc / 8 : 0), rows((unsigned)((row_units + 255) / 256)),
          rope((unsigned)((rope_units + 255) / 256)), weights((unsigned)((w_units + 1023) / 1024)), B(B)
    {
        static_assert(128 * (kRow / 8) % 256 == 0 && kDh * kDc / 8 % 1024 == 0, "a CTA's maximum has one owner");
    }
};

template <class Rows, bool kHalfV>
__global__ void __launch_bounds__(256)
prefill_prepare_kernel(const Rows cache, const PrepareBlocks blocks, int num_blocks,
                       const int32_t *__restrict__ block_table, int max_blocks, const int32_t *__restrict__ seq_lens,
                       int s, int H, int lpad, int l_cap, bf16 *__restrict__ rows, const bf16 *__restrict__ q_rope,
                       const int32_t *__restrict__ q_pos, bf16 *__restrict__ q_rot, const RopeTable rope,
                       const uint4 *__restrict__ w_uv, uint32_t *max_bits, uint32_t *err)
{
    unsigned cta = blockIdx.x;
    uint32_t most = 0;   // kHalfV: bf16 patterns of magnitudes, a pair
    int owner = 0;       // and (of thread 0) whose they are
    const bool weights = cta >= blocks.rows + blocks.rope;
    if (cta < blocks.rows) {
        constexpr int kUnits = kRow / 8;                            // 16-byte units per row
        const long long w = cta * 256ll + threadIdx.x;
        if (w < blocks.row_units) {
            const unsigned row = (unsigned)(w / kUnits);
            const int c = (int)(w % kUnits);
            const int b = (int)(row / lpad), j = (int)(row % lpad);
            const int L = seq_lens[b];
            owner = b;
            const bool valid = prefill_valid(L, s, l_cap);
            if (!valid && j == 0 && c == 0) set_error(err, MLA_DEVERR_SEQ_LEN);
            uint4 v = make_uint4(0, 0, 0, 0);
            if (valid && j < L) {
                const int blk = block_table[(long long)b * max_blocks + j / kBlock];
                if (blk >= 0 && blk < num_blocks)
                    v = cache.unit((long long)blk * kBlock + j % kBlock, c);
                else if (c == 0)
                    set_error(err, MLA_DEVERR_BLOCK_ID);
            }
            reinterpret_cast<uint4 *>(rows + (long long)row * kRow)[c] = v;
            if (kHalfV && c < kDc / 8) most = finite_max(v);
        }
    } else if (!weights) {
        const unsigned hgroups = (H + kPfRopeHeads - 1) / kPfRopeHeads;
        const long long w = (cta - blocks.rows) * 256ll + threadIdx.x;
        if (w < blocks.rope_units) {
            const unsigned g = (unsigned)(w / (kDr / 2));
            const int h0 = (int)(g % hgroups) * kPfRopeHeads;
            rope_heads<std::conditional_t<kHalfV, float, double>>(q_rope, q_pos, g / hgroups, (int)(w % (kDr / 2)), H, rope,
                                                                  q_rot, kDr, 0, h0, min(H, h0 + kPfRopeHeads));
        }
        return;
    } else {
        const unsigned wcta = cta - blocks.rows - blocks.rope;
        const long long w = wcta * 1024ll + threadIdx.x;
        owner = blocks.B + (int)(wcta / (kDh * kDc / 8 / 1024));
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (w + 256 * e < blocks.w_units) most = __vmaxu2(most, finite_max(w_uv[w + 256 * e]));
    }
    if constexpr (kHalfV) {
        __shared__ uint32_t cta_max;
        if (threadIdx.x == 0) cta_max = 0;
        __syncthreads();
        most = __reduce_max_sync(0xffffffffu, max(most & 0xFFFFu, most >> 16));
        if ((threadIdx.x & 31) == 0) atomicMax(&cta_max, most);
        __syncthreads();
        if (threadIdx.x == 0) atomicMax(max_bits + owner, cta_max);
    }
}

}  // namespace mla
