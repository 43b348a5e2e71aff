// tc_decode_int4.cuh -- absorbed-MLA decode over the 4-bit latent cache on
// tcgen05 tensor cores (sm_100a).
//
// What it computes: for every query row (query token t of sequence b, head i)
// softmax_j(scale * q_abs . row_j) weighted sum of the latents c^KV_j, with
// row_j the 576 values that the cache's codes and scales stand for
// (csrc/int4.cuh).  Every value is a bf16 value, so the products are those of
// the bf16 decode: 64 query rows of one sequence (the MMA M dimension) against
// one 64-token page at a time,
//   S(k)  = Q C_k^T            M=64, N=64, K=576 (36 MMAs), Q read from TMEM
//   O    += P(k) C_k[:, 0:512]  M=64, N=2 x 256, K=64 (8 MMAs)
//
// What bounds it: an M=64 MMA runs at half the tensor pipe's rate, 1,154 + 1,012
// cycles of pipe work per page and 64 rows, which at 128 heads is far above the
// page's 20,736 bytes; a full-rate M=128 needs O for 128 rows, all of one SM's TMEM
// (64 rows in each CTA of a cta_group::2 pair, with Q in shared memory, would fit: not
// built).  So the kernel is built to keep that pipe fed:
//   - One elected thread issues every MMA (warp 1), in the order S(k+1), P C(k),
//     S(k+2), ...: between S(k)'s end and P C(k)'s start the pipe has 2,166
//     cycles of other work, and the same between the release of a page's stage
//     and the S that needs it refilled.  Softmax and widening each fit in that
//     time, with three stages.  The thread is chosen by elect.sync: the compiler
//     then moves an MMA's descriptors to uniform registers directly (32 cycles
//     an MMA, the pipe's rate; under an ordinary `lane == 0` branch 76).
//   - Eight converter warps (8-15) read a page's codes and scales from global
//     memory into registers one page ahead, and widen them into the tile layout
//     when its stage is free.  No copy of the codes passes through shared
//     memory, which the three stages fill.  Each register is loaded again in place
//     right after its use and touched a page later: a copy of one in between would
//     wait for its load (293 against 223 us on 128 sequences x 128 heads x 4,096
//     tokens, before the later steps).
//   - Warp 0 walks the range's tile list and publishes {page, sequence, tile}
//     entries in shared memory (and warms L2), so that no other warp holds the
//     walk's state: the loops of all roles together stay small, because the
//     instruction cache is what a warp-specialised loop this wide runs out of.
//
// TMEM (512 columns): a 64-row operand occupies one half of each 32-lane
// quarter (row m at lane 32 (m / 16) + m % 16, plus 16 for the upper half):
//   lanes 0-15:  S(k % 2) (columns 0-127) | Q (128-415, bf16 pairs)
//   lanes 16-31: O (columns 0-511)
// and the softmax warps (4-7) touch it with 16-lane accesses only, two threads
// per row.  P (64 x 64 bf16) goes over the stage's RoPE chunk, which no MMA
// reads once S(k) is done.  Softmax: online, log2 domain, O and the running sum
// rescaled only when the maximum grows by more than 8 (a factor 256); the row
// sum takes the weights before they are rounded to bf16.
//
// Rows past a sequence's end get logit -inf, so weight 0; any pattern a page
// can hold is finite, so their latents add exactly 0 and need no zeroing.
//
// Measured (call, back to back): 128 sequences x 128 heads x 4,096 tokens 203 to 213 us
// by box (146 GFLOP: 88 us at the pipe's full rate, 126 us at M=64; the pipe is active in 70 % of
// the cycles), 64 x 16 heads x 4,096 62 us (87 MB: 13 us), one sequence of 16 heads
// and 256 tokens 15 us.  A tile takes about 2,700 cycles: its 2,166 of MMAs and gaps
// before each group of them.  A sequence's end inside a range takes about 14,000
// cycles, of which the next queries are 4,600 and the output 8,400.
//
// Work split and partial results are the bf16 decode's (plan_range); every cut
// sequence is merged by dec4_combine_kernel.  Every wait is bounded; one that gives
// up sets MLA_DEVERR_TIMEOUT and the CTA unwinds.
#pragma once

#include "dec_common.cuh"
#include "int4.cuh"

namespace mla {

constexpr int kD4Threads = 512;
constexpr int kD4Stages = 3;
constexpr int kD4Chunk = kBlock * 128;            // 64 tokens x 64 columns of bf16
constexpr int kD4Stage = 9 * kD4Chunk;            // 73,728
constexpr int kD4PChunk = 8 * kD4Chunk;           // P goes where the RoPE chunk was
constexpr int kD4OffEpi = kD4Stages * kD4Stage;   // staging: 16 rows x 128 B per softmax warp
constexpr int kD4OffList = kD4OffEpi + 4 * 16 * 128;
constexpr int kD4List = 16;                       // published tile entries
constexpr int kD4OffBar = kD4OffList + kD4List * 16;
constexpr int kD4Smem = kD4OffBar + 256 + 1024;   // + alignment slack
constexpr int kD4MinTiles = 2;                    // pages of the table a range, where there are few
constexpr int kD4Ahead = 6;                       // tiles published ahead of the one being widened
constexpr uint32_t kD4TmO = 16u << 16, kD4TmQ = 128;

struct Dec4Args {
    const bf16 *q_abs;                // [B*s][H][576]
    const uint8_t *codes, *scales;    // [num_blocks][64][288], [num_blocks][64][36]
    const int32_t *block_table, *seq_lens;
    int32_t *plan;                    // written by CTA 0 for the combine
    bf16 *out;
    float *out_lse;
    float *part_o, *part_lse2;        // [2*ranges][s*H][512], [2*ranges][s*H]
    uint32_t *err;
    unsigned long long limit_ns;
    int stall_tile;                   // test hook: this tile of every range is never widened (-1: none)
    float scale_log2;
    int max_blocks, num_blocks, s, H, B, groups;
};

// A published tile: the page (block 0 for a bad table entry), the sequence,
// its tile with flags, and the segment (the walk's count of sequences so far).
struct __align__(16) Dec4Tile {
    int page, seq, tt, seg;
};
constexpr int kD4First = 1 << 30, kD4Last = 1 << 29, kD4Complete = 1 << 28, kD4Tt = (1 << 28) - 1;

// The waits of this kernel poll in a few instructions and come here every 256
// polls: out of line, because the code of a wait that does not end is never run and
// would sit between the loops' own instructions in the instruction cache.  Returns
// the time the wait started (0 before the first call), or ~0 to give up: *abort is
// set, or the limit has passed (then the error bit and *abort are set).
__device__ __noinline__ uint64_t d4_wait_tick(uint64_t t0, volatile int *abort, uint32_t *err, uint64_t limit_ns)
{
    const uint64_t now = sm100::globaltimer_ns();
    if (t0 == 0) return *abort ? ~0ull : now;
    if (*abort) return ~0ull;
    if (now - t0 > limit_ns) {
        set_error(err, MLA_DEVERR_TIMEOUT);
        *abort = 1;
        return ~0ull;
    }
    return t0;
}

// The call's error word cleared (the plan is written whole by plan_range).  A kernel
// rather than a memset, because a memset ends before the next kernel is launched: here
// the decode's set-up overlaps it.
__global__ void __launch_bounds__(32) dec4_clear_kernel(uint32_t *err)
{
    sm100::pdl_trigger();
    sm100::pdl_wait();
    if (threadIdx.x == 0) *err = 0;
}

#define D4_RARE(x) __builtin_expect(!!(x), 0)

__global__ void __launch_bounds__(kD4Threads, 1) tc_decode_int4_kernel(const Dec4Args a)
{
    extern __shared__ uint8_t d4_smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(d4_smem_raw) + 1023) & ~uintptr_t(1023));
    Dec4Tile *list = reinterpret_cast<Dec4Tile *>(smem + kD4OffList);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kD4OffBar);
    uint64_t *cv_full = bars;         // [3] stage widened (8 converter warps)
    uint64_t *kv_empty = bars + 3;    // [3] P C of the stage done
    uint64_t *s_full = bars + 6;      // [2] S(k) in buffer k % 2
    uint64_t *p_full = bars + 10;     // [2] P(k) written and O rescaled (4 softmax warps)
    uint64_t *mma_done = bars + 12;   // the issuer's last MMAs done (teardown)
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 13);
    // counts rather than phases where a follower may be several steps behind
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + 14);
    volatile int *listed = reinterpret_cast<volatile int *>(bars + 15);   // entries published
    volatile int *cvt_at = reinterpret_cast<volatile int *>(bars + 16);   // the tile being widened
    volatile int *q_cnt = reinterpret_cast<volatile int *>(bars + 17);    // 4 per segment whose Q is in TMEM
    int *rplan = reinterpret_cast<int *>(bars + 18);                      // plan_range's out, 6 ints

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = blockIdx.x % a.groups, rng = blockIdx.x / a.groups;
    const int rows_per_seq = a.s * a.H;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kD4Stages; ++i) {
            sm100::mbar_init(&cv_full[i], 8);
            sm100::mbar_init(&kv_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            sm100::mbar_init(&s_full[i], 1);
            sm100::mbar_init(&p_full[i], 4);
        }
        sm100::mbar_init(mma_done, 1);
        *abort_flag = *listed = *cvt_at = *q_cnt = 0;
        sm100::fence_mbar_init();
    }
    if (warp == 1) {
        sm100::tmem_alloc(tmem_slot, 512);
        sm100::tmem_relinquish();
    }
    // lengths, queries and pages may come from the kernel before this one: read
    // after the wait, and through L2
    sm100::pdl_wait();
    if (warp == 2)
        plan_range(a.seq_lens, a.B, a.s, a.max_blocks, gridDim.x / a.groups, rng, blockIdx.x == 0, false, a.plan,
                   nullptr, a.err, rplan);
    sm100::tc_fence_before();
    __syncthreads();
    sm100::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int lo = rplan[0], hi = rplan[1], ntile = hi - lo;
    if (ntile <= 0) {   // no tile for this CTA
        if (warp == 1) sm100::tmem_dealloc(tmem, 512);
        return;
    }
    const unsigned long long lim = a.limit_ns;
    const unsigned long long drain_lim = lim > 200000000ull ? lim : 200000000ull;
    // Bounded waits of one thread: until *cnt >= target, and for a barrier's phase.
    // (A count's wait has no fence: what it covers lies in shared memory and is read
    // with volatile loads, which this thread's accesses stay in order with, and a
    // fence would also wait for the page loads in flight.)
    auto count_wait = [&](volatile int *cnt, int target) -> bool {
        uint64_t t0 = 0;
        for (uint32_t i = 1; *cnt < target; ++i)
            if (D4_RARE((i & 255u) == 0) && (t0 = d4_wait_tick(t0, abort_flag, a.err, lim)) == ~0ull) return false;
        return true;
    };
    auto bar_wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        const uint32_t at = sm100::smem_u32(bar);
        uint64_t t0 = 0;
        for (uint32_t i = 1; !sm100::mbar_test(at, parity); ++i)
            if (D4_RARE((i & 255u) == 0) && (t0 = d4_wait_tick(t0, abort_flag, a.err, lim)) == ~0ull) return false;
        return true;
    };
    // Warp-uniform: every lane polls, one vote (no shuffle through the queue that the
    // warp's stores and loads are in).
    auto phase_wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, bar_wait(bar, parity));
    };
    // the entry of tile k, once it is published (every thread for itself: where
    // lanes must agree, the caller votes before its next warp-wide step)
    auto tile_at = [&](int k, Dec4Tile &t) -> bool {
        if (!count_wait(listed, k + 1)) return false;
        const uint32_t e = sm100::smem_u32(&list[k % kD4List]);
        asm volatile("ld.volatile.shared.v4.s32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(t.page), "=r"(t.seq), "=r"(t.tt), "=r"(t.seg) : "r"(e) : "memory");
        return true;
    };

    if (warp == 0) {
        // ------------------------------------------------------- tile list
        // entry k goes out once tile k - kD4Ahead is being widened; the entry it
        // replaces is 16 tiles back, and no role is more than the three stages
        // behind the converters
        TileIter it;
        it.init(a.seq_lens, a.max_blocks, a.B, lo, hi, rplan[2], rplan[3], rplan[5]);
        for (; it.ok; it.advance()) {
            // (a sleeping poll: nothing waits for the entry yet, and the slots a busy
            // one would take belong to the other warps; it ends with the converters'
            // own bounded waits)
            while (*cvt_at < it.k - kD4Ahead && !*abort_flag) __nanosleep(200);
            if (__any_sync(0xffffffffu, *abort_flag)) break;
            if (lane == 0) {
                int page = __ldcg(a.block_table + (long long)it.seq * a.max_blocks + it.tt);
                if (page < 0 || page >= a.num_blocks) {
                    // never read outside the cache: page 0 stands in; the
                    // sequence's output is then unspecified and the bit says so
                    set_error(a.err, MLA_DEVERR_BLOCK_ID);
                    page = 0;
                }
                sm100::bulk_prefetch_l2(a.codes + (long long)page * (kBlock * kInt4Codes), kBlock * kInt4Codes);
                sm100::bulk_prefetch_l2(a.scales + (long long)page * (kBlock * kInt4Scales), kBlock * kInt4Scales);
                const int fl = (it.first() ? kD4First : 0) | (it.last() ? kD4Last : 0) | (it.complete ? kD4Complete : 0);
                *reinterpret_cast<int4 *>(&list[it.k % kD4List]) = make_int4(page, it.seq, it.tt | fl, it.seg);
                __threadfence_block();
                *listed = it.k + 1;
                if (it.first() && it.k > 0) {
                    const int r0 = group * kGroupRows, nr = min(kGroupRows, rows_per_seq - r0);
                    const char *q0 = reinterpret_cast<const char *>(a.q_abs + ((long long)it.seq * rows_per_seq + r0) * kRow);
                    for (int r = 0; r < nr; r += 8)
                        sm100::bulk_prefetch_l2(q0 + (long long)r * kRow * 2, min(8, nr - r) * kRow * 2);
                }
            }
            __syncwarp();
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMAs
        if (sm100::elect_one()) {
            const uint32_t idesc_s = sm100::idesc_bf16(kGroupRows, kBlock, 0, 0);
            const uint32_t idesc_o = sm100::idesc_bf16(kGroupRows, 256, 0, 1);
            const uint32_t st0 = sm100::smem_u32(smem);
            // S(k)'s buffer is free: P C(k - 2) was issued before it and waited for the
            // softmax of tile k - 2
            auto issue_s = [&](int k, const Dec4Tile &t) -> bool {
                const int st = k % kD4Stages, b = k & 1;
                if (D4_RARE(t.tt & kD4First) && !count_wait(q_cnt, 4 * (t.seg + 1))) return false;
                if (!bar_wait(&cv_full[st], (k / kD4Stages) & 1)) return false;
                sm100::tc_fence_after();
                const uint64_t kd = sm100::desc_kmajor(st0 + st * kD4Stage, 128, sm100::kSw128);
#pragma unroll 1
                for (int c = 0; c < 9; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sm100::umma_ts(tmem + 64 * b, tmem + kD4TmQ + 32 * c + 8 * e,
                                       kd + (uint64_t)((c * kD4Chunk + e * 32) >> 4), idesc_s, c > 0 || e > 0);
                sm100::umma_commit(&s_full[b]);
                return true;
            };
            auto issue_o = [&](int k, uint32_t acc0) -> bool {
                const int st = k % kD4Stages;
                if (!bar_wait(&p_full[k & 1], (k >> 1) & 1)) return false;
                sm100::tc_fence_after();
                const uint64_t vd = sm100::desc_mnmajor_sw128(st0 + st * kD4Stage, kD4Chunk);
                const uint64_t pd = sm100::desc_kmajor(st0 + st * kD4Stage + kD4PChunk, 128, sm100::kSw128);
#pragma unroll 1
                for (int kq = 0; kq < kBlock / 16; ++kq)
#pragma unroll
                    for (int jh = 0; jh < 2; ++jh)
                        sm100::umma_ss(tmem + kD4TmO + 256 * jh, pd + (uint64_t)((kq * 32) >> 4),
                                       vd + (uint64_t)((4 * jh * kD4Chunk + kq * 2048) >> 4), idesc_o, kq > 0 ? 1u : acc0);
                sm100::umma_commit(&kv_empty[st]);
                return true;
            };
            Dec4Tile t, prev;
            prev.tt = 0;
            bool ok = true;
            for (int k = 0; ok && k <= ntile; ++k) {
                bool s_first = true;
                if (k < ntile) {
                    ok = tile_at(k, t);
                    // a new sequence's queries go in behind the last tile's P: that
                    // tile's P C leads
                    s_first = !(t.tt & kD4First) || k == 0;
                    if (ok && s_first) ok = issue_s(k, t);
                }
                if (ok && k > 0) ok = issue_o(k - 1, (prev.tt & kD4First) ? 0u : 1u);
                if (ok && !s_first) ok = issue_s(k, t);
                prev = t;
            }
            sm100::umma_commit(mma_done);
        }
        __syncwarp();
    } else if (warp == 3) {
        // the first segment's queries into L2, ahead of the warps that read them
        if (lane < 8) {
            const int g0 = group * kGroupRows + 8 * lane, nr = min(8, rows_per_seq - g0);
            if (nr > 0)
                sm100::bulk_prefetch_l2(a.q_abs + ((long long)rplan[2] * rows_per_seq + g0) * kRow, nr * kRow * 2);
        }
    } else if (warp >= 8) {
        // ------------------------------------------------ 4-bit -> bf16
        // Thread (r, p) = (ct / 4, ct % 4) takes, of row r and each 128-column
        // pair of chunks c, the 16-byte piece p: 32 values (two scales) in half
        // p & 1 of chunk 2 c + (p >> 1); and of chunk 8 its 8 bytes p.  A quad's
        // loads cover 64 contiguous bytes.  Pieces of the upper chunk store
        // their words in the order 2 3 0 1, so that a quarter warp's 16-byte
        // stores fall on eight different bank groups.
        const int ct = threadIdx.x - 256, r = ct >> 2, p = ct & 3;
        const uint32_t row = sm100::smem_u32(smem) + r * 128 + (p >> 1) * kD4Chunk, sw = r & 7;
        const bool up = p >> 1;
        const uint32_t u = 4 * (p & 1) + (up ? 2 : 0);           // unit of the first word stored
        const uint32_t o0 = ((u ^ sw) << 4), o1 = (((u + 1) ^ sw) << 4), o2 = (((u ^ 2) ^ sw) << 4),
                       o3 = ((((u ^ 2) + 1) ^ sw) << 4);
        const uint32_t sel0 = 0x4440 + 2 * (p & 1), sel1 = sel0 + 1;
        auto src_of = [&](int page) { return a.codes + ((long long)page * kBlock + r) * kInt4Codes; };
        auto words_of = [&](int page) {
            return reinterpret_cast<const uint32_t *>(a.scales + ((long long)page * kBlock + r) * kInt4Scales);
        };
        auto piece = [&](const uint8_t *src, int c) { return __ldcg(reinterpret_cast<const uint4 *>(src + 64 * c) + p); };
        // what this thread holds of the page it will widen next: its pieces, its
        // part of chunk 8, and scale words p, p + 4 and 8 of the row's nine (word
        // j: the four scales of chunk j).  The loop below reloads each register in
        // place and touches it only a page later: a copy or a select on it there
        // would wait for the load
        Dec4Tile t;
        bool ok = __all_sync(0xffffffffu, tile_at(0, t));
        uint4 q[4];
        uint2 c8;
        uint32_t s0, s1, s8;
        if (ok) {
            const uint8_t *src = src_of(t.page);
            const uint32_t *sc = words_of(t.page);
            s0 = __ldcg(sc + p); s1 = __ldcg(sc + 4 + p); s8 = __ldcg(sc + 8);
#pragma unroll
            for (int c = 0; c < 4; ++c) q[c] = piece(src, c);
            c8 = __ldcg(reinterpret_cast<const uint2 *>(src + 256) + p);
        }
        for (int k = 0; ok && k < ntile; ++k) {
            const int st = k % kD4Stages;
            if (ct == 0) *cvt_at = k;
            const bool more = k + 1 < ntile;
            if (more) ok = tile_at(k + 1, t);
            const uint8_t *src = src_of(t.page);
            const uint32_t *sc = words_of(t.page);
            uint32_t n0 = 0, n1 = 0, n8 = 0;
            if (ok && more) { n0 = __ldcg(sc + p); n1 = __ldcg(sc + 4 + p); n8 = __ldcg(sc + 8); }
            if (k >= kD4Stages)   // (whatever this lane's ok: the wait votes)
                ok = phase_wait(&kv_empty[st], ((k / kD4Stages) - 1) & 1) && ok;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (k == a.stall_tile) continue;   // test hook: this tile never becomes full
            uint32_t dst = row + st * kD4Stage;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                // the pair's scale word: word 2 c + (p >> 1) of the row
                const uint32_t w = __shfl_sync(0xffffffffu, c < 2 ? s0 : s1, ((2 * c) & 3) + (p >> 1), 4);
                __nv_bfloat162 a2, am, b2, bm;
                int4_scale2(__byte_perm(w, 0, sel0), a2, am);
                int4_scale2(__byte_perm(w, 0, sel1), b2, bm);
                // words x, y take the first scale, z, w the second; the upper
                // chunk's pieces store z, w first
                const uint4 v = up ? make_uint4(q[c].z, q[c].w, q[c].x, q[c].y) : q[c];
                if (more) q[c] = piece(src, c);
                if (up) {
                    const __nv_bfloat162 t2 = a2, tm = am;
                    a2 = b2; am = bm; b2 = t2; bm = tm;
                }
                st_shared_v4(dst + o0, int4_widen8(v.x, a2, am));
                st_shared_v4(dst + o1, int4_widen8(v.y, a2, am));
                st_shared_v4(dst + o2, int4_widen8(v.z, b2, bm));
                st_shared_v4(dst + o3, int4_widen8(v.w, b2, bm));
                dst += 2 * kD4Chunk;
            }
            {
                __nv_bfloat162 a2, am;
                int4_scale2(__byte_perm(s8, 0, 0x4440 + p), a2, am);
                const uint32_t d8 = dst - (p >> 1) * kD4Chunk;   // chunk 8: units 2 p and 2 p + 1
                st_shared_v4(d8 + (((2 * p) ^ sw) << 4), int4_widen8(c8.x, a2, am));
                st_shared_v4(d8 + (((2 * p + 1) ^ sw) << 4), int4_widen8(c8.y, a2, am));
                if (more) c8 = __ldcg(reinterpret_cast<const uint2 *>(src + 256) + p);
            }
            s0 = n0; s1 = n1; s8 = n8;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) sm100::mbar_arrive(&cv_full[st]);
        }
    } else if (warp >= 4) {
        // -------------------------------------------------------- softmax
        // warp q (0..3) owns group rows [16 q, 16 q + 16): row 16 q + i's logits
        // and Q sit at TMEM lane 32 q + i, its O at lane 32 q + 16 + i; threads i
        // and 16 + i each take half of the row's columns in both
        const int qd = warp & 3;
        const bool srow = lane < 16;
        const int r = 16 * qd + (lane & 15);
        const uint32_t lane_base = tmem + ((uint32_t)(qd * 32) << 16);
        const uint32_t o_base = tmem + ((uint32_t)(qd * 32 + 16) << 16);
        const uint32_t p_row0 = sm100::smem_u32(smem + kD4PChunk) + r * 128;
        const uint32_t pc0 = srow ? 0 : 4;   // first 16-byte chunk of P this thread writes
        const int grow = group * kGroupRows + r;   // index among the sequence's s*H rows
        const bool row_ok = grow < rows_per_seq;
        const int tq = row_ok ? grow / a.H : 0;
        // Q rows of a sequence into TMEM (16-lane stores: the O lanes are left
        // alone): thread i and 16 + i hold half of each 32-column block
        auto write_q = [&](int seq) {
            const uint4 *q4 = reinterpret_cast<const uint4 *>(
                a.q_abs + ((long long)seq * rows_per_seq + (row_ok ? grow : 0)) * kRow) + (srow ? 0 : 4);
#pragma unroll 1
            for (int h = 0; h < 3; ++h) {   // three rounds of 12 loads in flight
                uint4 v[12];
#pragma unroll
                for (int e = 0; e < 12; ++e)
                    v[e] = row_ok ? __ldcg(q4 + 24 * h + 8 * (e >> 2) + (e & 3)) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int j = 0; j < 3; ++j)
                    sm100::tmem_st16x2_16(lane_base + kD4TmQ + 96 * h + 32 * j, reinterpret_cast<const uint32_t *>(v + 4 * j));
            }
            sm100::tmem_wait_st();
            sm100::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                __threadfence_block();
                atomicAdd(const_cast<int *>(q_cnt), 1);
            }
        };
        float m_run = -INFINITY, l_run = 0.f;
        const bool any_row = group * kGroupRows + 16 * qd < rows_per_seq;
        int nvis = 0;
        Dec4Tile t;
        bool ok = __all_sync(0xffffffffu, tile_at(0, t));
        if (ok) write_q(t.seq);
        for (int k = 0; ok && k < ntile; ++k) {
            const int b = k & 1, st = k % kD4Stages;
            if (k > 0) ok = tile_at(k, t);
            if (D4_RARE(ok && (t.tt & kD4First))) {
                m_run = -INFINITY;
                l_run = 0.f;
                // query tq of a sequence of length L sees positions j <= L - s + tq
                nvis = seq_len_clamped(a.seq_lens, t.seq, a.max_blocks) - a.s + tq + 1;
            }
            ok = phase_wait(&s_full[b], (k >> 1) & 1) && ok;   // (whatever this lane's ok: the wait votes)
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (!any_row && !(t.tt & kD4Last)) {   // no row of this quarter is stored: whatever P holds will do
                if (lane == 0) sm100::mbar_arrive(&p_full[b]);
                __syncwarp();
                continue;
            }
            sm100::tc_fence_after();
            float x[32];
            {
                uint32_t sv[32];
                sm100::tmem_ld16x2_32(lane_base + 64u * b, sv);
                sm100::tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 32; ++c) x[c] = __uint_as_float(sv[c]);
            }
            const int left = nvis - (t.tt & kD4Tt) * kBlock - (srow ? 0 : 32);   // visible of these 32 columns
            if (D4_RARE(left < 32)) {
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    if (c >= left) x[c] = -INFINITY;
            }
            float mx = -INFINITY;
#pragma unroll
            for (int c = 0; c < 32; c += 4) mx = fmaxf(mx, fmaxf(fmaxf(x[c], x[c + 1]), fmaxf(x[c + 2], x[c + 3])));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            // both threads of a row take the same decisions: they hold the same max
            const float mt = mx * a.scale_log2;
            const bool grown = (mt != -INFINITY) && (m_run == -INFINITY || mt > m_run + kRescaleThreshold);
            const bool rescale = grown && m_run != -INFINITY;
            const float m_new = grown ? mt : m_run;
            const float corr = rescale ? ex2(m_run - m_new) : (grown ? 0.f : 1.f);
            if (D4_RARE(__any_sync(0xffffffffu, rescale))) {
                // O holds this segment's tiles up to k - 1: let them retire, then
                // scale the O lanes (S(k + 1) may be using the other half)
                ok = phase_wait(&kv_empty[(k - 1) % kD4Stages], ((k - 1) / kD4Stages) & 1);
                if (!ok) break;
                sm100::tc_fence_after();
                const float f = rescale ? corr : 1.f;
#pragma unroll 1
                for (int c = 0; c < 512; c += 64) {
                    uint32_t ov[32];
                    sm100::tmem_ld16x2_32(o_base + c, ov);
                    sm100::tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * f);
                    sm100::tmem_st16x2_32(o_base + c, ov);
                }
                sm100::tmem_wait_st();
                sm100::tc_fence_before();
            }
            m_run = m_new;
            const float mu = (m_run == -INFINITY) ? 0.f : m_run;
            float lsum = 0.f;
            const uint32_t p_row = p_row0 + st * kD4Stage;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                // P row r: 64 bf16, 16-byte chunk c at c ^ (r & 7) (128-byte swizzle);
                // the weights are rounded to bf16 for the MMA, their sum is not
                uint32_t pw[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float p0 = ex2(fmaf(x[8 * q + 2 * e], a.scale_log2, -mu));
                    const float p1 = ex2(fmaf(x[8 * q + 2 * e + 1], a.scale_log2, -mu));
                    pw[e] = pack_bf162(p0, p1);
                    lsum += p0 + p1;
                }
                st_shared_v4(p_row + (((pc0 + q) ^ (r & 7)) << 4), make_uint4(pw[0], pw[1], pw[2], pw[3]));
            }
            l_run = l_run * corr + lsum;   // this lane's share of the row sum
            fence_proxy_async_smem();
            sm100::tc_fence_before();
            __syncwarp();
            if (lane == 0) sm100::mbar_arrive(&p_full[b]);
            if (!(t.tt & kD4Last)) continue;

            // ------------------------------------------- end of a segment
            // every S of this segment has been read: the next sequence's Q goes
            // in now, so that its S overlaps this epilogue
            Dec4Tile nx;
            nx.seq = -1;
            if (k + 1 < ntile) ok = tile_at(k + 1, nx);
            ok = __all_sync(0xffffffffu, ok);
            if (ok && nx.seq >= 0) write_q(nx.seq);
            ok = ok && phase_wait(&kv_empty[st], (k / kD4Stages) & 1);
            if (!ok) break;
            sm100::tc_fence_after();
            const float l_tot = l_run + __shfl_xor_sync(0xffffffffu, l_run, 16);
            const float inv = l_tot > 0.f ? 1.f / l_tot : 0.f;
            const float lse2 = l_tot > 0.f ? m_run + __log2f(l_tot) : -INFINITY;
            const bool complete = t.tt & kD4Complete;
            const long long slot = 2LL * rng + (t.seg == 0 ? 0 : 1);
            // The warp's 16 rows of one 64-column block of O at a time leave
            // through shared memory (16-byte chunks swizzled by row), so that a
            // store instruction writes whole 128-byte lines: bf16 rows of 128 B
            // (complete), or fp32 rows of 256 B in two rounds (partial)
            const uint32_t stg = sm100::smem_u32(smem + kD4OffEpi) + qd * 16 * 128;
            const int lr = lane & 15, r0 = group * kGroupRows + 16 * qd;
            char *base = complete ? reinterpret_cast<char *>(a.out + (long long)t.seq * rows_per_seq * kDc)
                                  : reinterpret_cast<char *>(a.part_o + slot * rows_per_seq * kDc);
            const int rounds = complete ? 1 : 2, eb = complete ? 2 : 4;
#pragma unroll 1
            for (int c = 0; c < 512; c += 64) {
                uint32_t ov[32];
                sm100::tmem_ld16x2_32(o_base + c, ov);
                sm100::tmem_wait_ld();
#pragma unroll 1
                for (int q = 0; q < rounds; ++q) {
                    if (complete) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            auto f = [&](int i) { return __uint_as_float(ov[8 * j + i]) * inv; };
                            st_shared_v4(stg + lr * 128 + (((pc0 + j) ^ (lr & 7)) << 4),
                                         make_uint4(pack_bf162(f(0), f(1)), pack_bf162(f(2), f(3)),
                                                    pack_bf162(f(4), f(5)), pack_bf162(f(6), f(7))));
                        }
                    } else if ((srow ? 0 : 1) == q) {   // round q: columns 32 q .. of the block
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            auto f = [&](int i) { return __float_as_uint(__uint_as_float(ov[4 * j + i]) * inv); };
                            st_shared_v4(stg + lr * 128 + ((j ^ (lr & 7)) << 4), make_uint4(f(0), f(1), f(2), f(3)));
                        }
                    }
                    __syncwarp();
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int i = 4 * e + (lane >> 3), ch = lane & 7;
                        const uint4 v = ld_shared_v4(stg + i * 128 + ((ch ^ (i & 7)) << 4));
                        if (r0 + i < rows_per_seq)
                            *reinterpret_cast<uint4 *>(base + ((long long)(r0 + i) * kDc + c) * eb + 128 * q + 16 * ch) = v;
                    }
                    __syncwarp();
                }
            }
            if (row_ok && srow) {
                if (!complete)
                    a.part_lse2[slot * rows_per_seq + grow] = lse2;
                else if (a.out_lse)
                    a.out_lse[(long long)t.seq * rows_per_seq + grow] = lse2 * kLn2;
            }
            // O is read: the next segment's first P C may overwrite it
            sm100::tc_fence_before();
            __syncwarp();
        }
    }

    // ------------------------------------------------------------ teardown
    sm100::pdl_trigger();   // the combine may start launching
    sm100::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        // every MMA this CTA issued retires before its TMEM is released
        volatile int no_abort = 0;
        sm100::warp_wait(mma_done, 0, &no_abort, a.err, drain_lim);
        sm100::tc_fence_after();
        sm100::tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------ combine
// Sequences cut by range ends are merged by log-sum-exp; sequences one range
// finished are already in place; query rows with no visible key get a zero
// latent and lse = -inf.  Only the sequences plan_range lists are visited.
//   kMode 0: one warp per row, all 512 columns, two pieces' loads in flight.
//   kMode 1, where a sequence may be cut into kD4SomePieces pieces or more and the
//     batch has at most kD4SomeRows rows: one warp per row and 128 columns, eight pieces
//     in flight.  Two sequences of 128 heads x 20,000 tokens (37 pieces): the call
//     takes 41.4 us so, 47.9 with mode 0; 8 x 16 heads x 1,000 (8 pieces) 19.0 against
//     19.6; 32 x 16 heads x 800 (4 pieces) 22.3 against 21.3.
//   kMode 2, where it may be cut into kD4ManyPieces and there are at most kD4FewRows
//     rows: one CTA per row and 128 columns, its eight warps taking the pieces eight by
//     eight in turn; their sums are added in warp order.  One sequence of 16 heads and
//     32,768 tokens (148 pieces): 26.3 us so, 45.1 with mode 1; 4 x 16 heads x 8,000 (37
//     pieces) 24.0 against 27.1; 2 x 128 heads x 5,000 (256 rows) 31.8 against 28.2.
// The weights 2^(lse2_i - max) are kept per warp in shared memory; a warp sums its
// pieces in range order, so the bits do not change from run to run.
constexpr int kD4CombineWarps = 8;
constexpr int kD4SomePieces = 5, kD4SomeRows = 1024;
constexpr int kD4ManyPieces = 28, kD4FewRows = 192;

template <int kMode>
__global__ void __launch_bounds__(32 * kD4CombineWarps)
dec4_combine_kernel(const int32_t *plan, const float *part_o, const float *part_lse2, int B, int s, int H,
                    bf16 *__restrict__ out, float *__restrict__ out_lse)
{
    constexpr bool kParts = kMode > 0, kFew = kMode == 2;
    constexpr int kQuads = kParts ? 1 : 4;    // 128-column quarters of a warp
    constexpr int kAhead = 8 / kQuads;        // pieces in flight
    __shared__ float weight[kD4CombineWarps][kMaxRanges];
    __shared__ float4 sums[kFew ? kD4CombineWarps : 1][32];
    // what the decode kernel wrote is read only after the wait and only through L2
    sm100::pdl_wait();
    const int qv = __ldcg(plan), pw = __ldcg(plan + 3), nlist = __ldcg(plan + 5 + B);
    const int4 *list = reinterpret_cast<const int4 *>(plan + plan_list_off(B));
    const unsigned rows = s * H, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned items = nlist * rows * (kParts ? 4 : 1);
    const unsigned step = kFew ? gridDim.x : gridDim.x * kD4CombineWarps;
    for (unsigned it = kFew ? blockIdx.x : blockIdx.x * kD4CombineWarps + warp; it < items; it += step) {
        const unsigned part = kParts ? it & 3 : 0, line = kParts ? it >> 2 : it;
        const unsigned li = line / rows, row = line - li * rows;
        const int4 seq = __ldcg(list + li);
        const int b = seq.x, va = seq.y, tb = seq.z, L = seq.w;
        const long long orow = (long long)b * rows + row;
        const int col = 128 * part + 4 * lane;   // and, of one warp per row, 128 columns on, ..
        const bool writes = !kFew || warp == 0;
        // the ranges holding the sequence's first and last tiles; the piece in range
        // c0 is that range's first segment only if the range starts with the sequence
        // (slot 2 c0), else its last (2 c0 + 1); every later piece is its range's
        // first segment (slot 2 c)
        const int c0 = tb > 0 ? (va + pw) / qv : 0, c1 = tb > 0 ? (va + pw + tb - 1) / qv : 0;
        const bool visible = L - s + (int)(row / H) + 1 > 0;   // query row / H sees some key
        if (!visible || tb == 0) {   // (the same for every warp of a kFew CTA)
            if (writes) {
#pragma unroll
                for (int e = 0; e < kQuads; ++e)
                    *reinterpret_cast<uint2 *>(out + orow * kDc + col + 128 * e) = make_uint2(0, 0);
                if (part == 0 && lane == 0 && out_lse) out_lse[orow] = -INFINITY;
            }
            continue;
        }
        const int n = c1 - c0 + 1, slot0 = 2 * c0 + (c0 * qv < va ? 1 : 0);
        auto row_of = [&](int i) { return (long long)(i == 0 ? slot0 : 2 * (c0 + i)) * rows + row; };
        float M = -INFINITY;
        for (int i = lane; i < n; i += 32) {
            const float l2 = __ldcg(part_lse2 + row_of(i));
            weight[warp][i] = l2;
            M = fmaxf(M, l2);
        }
        M = warp_max(M);
        float den = 0.f;
        for (int i = lane; i < n; i += 32) {
            const float l2 = weight[warp][i], w = l2 == -INFINITY ? 0.f : exp2f(l2 - M);
            weight[warp][i] = w;
            den += w;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
        __syncwarp();
        float4 acc[kQuads] = {};
        for (int i0 = kFew ? warp * kAhead : 0; i0 < n; i0 += kFew ? kD4CombineWarps * kAhead : kAhead) {
            float4 v[kAhead][kQuads];
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
#pragma unroll
                for (int e = 0; e < kQuads; ++e)
                    v[j][e] = i0 + j < n ? __ldcg(reinterpret_cast<const float4 *>(part_o + row_of(i0 + j) * kDc + col + 128 * e))
                                         : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const float w = i0 + j < n ? weight[warp][i0 + j] : 0.f;
#pragma unroll
                for (int e = 0; e < kQuads; ++e) {
                    acc[e].x = fmaf(w, v[j][e].x, acc[e].x);
                    acc[e].y = fmaf(w, v[j][e].y, acc[e].y);
                    acc[e].z = fmaf(w, v[j][e].z, acc[e].z);
                    acc[e].w = fmaf(w, v[j][e].w, acc[e].w);
                }
            }
        }
        if (kFew) {
            sums[warp][lane] = acc[0];
            __syncthreads();
            if (warp == 0)
                for (int w = 1; w < kD4CombineWarps; ++w) {
                    const float4 x = sums[w][lane];
                    acc[0].x += x.x;
                    acc[0].y += x.y;
                    acc[0].z += x.z;
                    acc[0].w += x.w;
                }
        }
        if (writes) {
            const float inv = den > 0.f ? 1.f / den : 0.f;
#pragma unroll
            for (int e = 0; e < kQuads; ++e)
                *reinterpret_cast<uint2 *>(out + orow * kDc + col + 128 * e) =
                    make_uint2(pack_bf162(acc[e].x * inv, acc[e].y * inv), pack_bf162(acc[e].z * inv, acc[e].w * inv));
            if (part == 0 && lane == 0 && out_lse) out_lse[orow] = den > 0.f ? (M + log2f(den)) * kLn2 : -INFINITY;
        }
        if (kFew)
            __syncthreads();   // the sums are read
        else
            __syncwarp();      // the weights are read
    }
}

}  // namespace mla
