// int4.cuh -- the 4-bit latent cache: its format, the cache writer and the
// row reader.
//
// Format: a token's row [c^KV (512) | k^R (64), rotated] is cut into 36 groups
// of 16 values.  A group has one scale byte b, the scale
//   s = (1 + (b & 7) / 8) 2^((b >> 3) - 15)          (2^-15 .. 1.875 2^16)
// and 16 codes u in 0..15; a code's value is (u - 8) s.
//   codes  [num_blocks][64][288] uint8   (288 B per row, 18,432 B per page)
//   scales [num_blocks][64][36]  uint8   (36 B per row, 2,304 B per page)
// The 8 values v0..v7 of a little-endian 32-bit word of codes are its nibbles
// v0 v2 v4 v6 v1 v3 v5 v7 from the lowest up: a pair (v2p, v2p+1) sits 16 bits
// apart, where a shift and a mask put both into the halves of one register.
//
// Why these widths: u - 8 has 4 significant bits and s has 4, so a value is a
// bf16 value exactly (8 bits).  The cache is 324 B a token (4.5 bits a value)
// against 1152 B in bf16, and every kernel that reads it can use the same bf16
// tensor-core operands as the bf16 cache, with no rounding of its own and no
// scale left to carry into the softmax.  16-value groups keep a large value's
// step away from its neighbours: on N(0,1) rows the stored values' rms error
// is 0.086 with 16-value groups, 0.098 with 32 and 0.108 with 64.  The scale
// format has no zero, infinity or NaN, so every bit pattern a page can hold is
// a finite row: 0 * (whatever lies behind a sequence's end) is 0.
#pragma once

#include "common.cuh"
#include "k_simple.cuh"

namespace mla {

constexpr int kInt4Group = 16;                     // values per scale
constexpr int kInt4Codes = kRow / 2;               // 288 B of codes per row
constexpr int kInt4Scales = kRow / kInt4Group;     // 36 scale bytes per row

// The scale byte of a group: amax * (1/7), both in fp32, rounded to three
// mantissa bits, nearest-even, clamped to the format's range.
__device__ __forceinline__ uint32_t int4_scale_byte(float amax)
{
    const uint32_t u = __float_as_uint(__fmul_rn(amax, 1.f / 7.f));
    const int b = (int)((u + 0x7FFFFu + ((u >> 20) & 1u)) >> 20) - (112 << 3);
    return (uint32_t)min(max(b, 0), 255);
}

__device__ __forceinline__ float int4_scale(uint32_t b) { return __uint_as_float((b << 20) + (112u << 23)); }

// The code of a bf16 x under scale s in the low four bits of the result, above them
// the constant kInt4CodeBits: 8 + x / s rounded to nearest-even, |x| <= 7.5 s; inv_s
// is 1 / s in fp32.  x * inv_s is within 2^-24 of the quotient, relative.  With
// x = X 2^a (X < 256) and s = S 2^b (8 <= S < 16), a quotient below 8 that is not a
// tie k + 1/2 is at least 1/512 away from one (255/512 is), so the sum with 192, which the one
// rounding of the multiply-add takes to a multiple of 2^-16, restores the ties and
// moves nothing across them.  The addition rounds to an integer: 1.5 2^23 + 8 - 192 +
// the sum lies where fp32 has spacing 1.
constexpr uint32_t kInt4CodeBits = 0x4B400000u;   // 1.5 2^23
__device__ __forceinline__ uint32_t int4_code(float x, float inv_s)
{
    return __float_as_uint(__fadd_rn(__fmaf_rn(x, inv_s, 192.f), 12582912.f + 8.f - 192.f));
}

// A pair of bf16 values without NaN: a NaN becomes 0.
__device__ __forceinline__ uint32_t int4_known(uint32_t h)
{
    const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162 *>(&h);
    return h & __heq2_mask(x, x);
}

// A pair limited to +-7 s (7 bits: a bf16 value), where the scale is the format's
// largest: elsewhere no value of the group is beyond 7.5 s.
__device__ __forceinline__ uint32_t int4_limit(uint32_t h, float s)
{
    const __nv_bfloat162 l = __float2bfloat162_rn(7.f * s), x = *reinterpret_cast<const __nv_bfloat162 *>(&h);
    const __nv_bfloat162 y = __hmax2(__hmin2(x, l), __hneg2(l));
    return *reinterpret_cast<const uint32_t *>(&y);
}

__device__ __forceinline__ float int4_low(uint32_t h) { return __uint_as_float(h << 16); }
__device__ __forceinline__ float int4_high(uint32_t h) { return __uint_as_float(h & 0xFFFF0000u); }

// Eight codes (one word) and their scale byte -> 8 bf16 values.  A nibble u
// OR-ed into bits 6..3 of the bf16 pattern of 16.0 is 16 + u, and
// (16 + u) s - 24 s = (u - 8) s in one fused multiply-add; 24 s (2 + 4 bits)
// and the result (4 + 4 bits) are exact, so nothing is rounded.
__device__ __forceinline__ uint4 int4_widen8(uint32_t w, __nv_bfloat162 s2, __nv_bfloat162 m24s2)
{
    auto pair = [&](uint32_t sh) {
        uint32_t v = (sh & 0x00780078u) | 0x41804180u;
        __nv_bfloat162 x = __hfma2(*reinterpret_cast<__nv_bfloat162 *>(&v), s2, m24s2);
        return *reinterpret_cast<uint32_t *>(&x);
    };
    return make_uint4(pair(w << 3), pair(w >> 1), pair(w >> 5), pair(w >> 9));
}

// The scale of byte b in both halves, and -24 times it.
__device__ __forceinline__ void int4_scale2(uint32_t b, __nv_bfloat162 &s2, __nv_bfloat162 &m24s2)
{
    uint32_t v = b * 0x00100010u + 0x38003800u;
    s2 = *reinterpret_cast<__nv_bfloat162 *>(&v);
    m24s2 = __hmul2(s2, __floats2bfloat162_rn(-24.f, -24.f));
}

// Rows of the 4-bit cache as 16-byte units of 8 bf16 values (see Bf16Rows).
struct Int4Rows {
    const uint8_t *codes, *scales;
    __device__ __forceinline__ uint4 unit(long long slot, int c) const
    {
        const uint32_t w = reinterpret_cast<const uint32_t *>(codes + slot * kInt4Codes)[c];
        __nv_bfloat162 s2, m24s2;
        int4_scale2(scales[slot * kInt4Scales + (c >> 1)], s2, m24s2);
        return int4_widen8(w, s2, m24s2);
    }
};

// One warp per token: the token's bf16 row exactly as the bf16 cache writer
// forms it (copy or RMSNorm of the latent, RoPE of the key), then quantized
// per group.  Lane l holds latent values [8l, 8l+8) and [256+8l, 256+8l+8), so
// a latent group is two lanes, and key pair l, so a key group is eight.  A NaN
// is stored as 0.  Tokens whose slot is invalid are skipped with an error bit.
//
// What bounds it: issue (2.9 warp instructions a cycle and SM; the angles in double
// precision are a fifth).  So maxima are taken on bf16 patterns, two at a time, and
// values are quantized with a reciprocal, two fp32 operations each: 65,536 rows take
// 37 us (97 MB, 15 us of traffic), 52 us with a division, two clamps and a NaN test
// per value; 16,384 rows 12.7 against 16.6 us.
__global__ void __launch_bounds__(256)
append_latent_int4_kernel(const bf16 *__restrict__ c_kv, const bf16 *__restrict__ k_rope, int T,
                          const int32_t *__restrict__ seq_idx, const int32_t *__restrict__ pos,
                          const int32_t *__restrict__ block_table, int num_seqs, int max_blocks,
                          uint8_t *__restrict__ codes, uint8_t *__restrict__ scales, int num_blocks,
                          const RopeTable rope, const bf16 *__restrict__ norm_w, float eps, uint32_t *err)
{
    const int warp = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    if (warp >= T) return;
    const int p = pos[warp];
    uint4 v[2];
    __nv_bfloat162 kr;
    latent_row_lanes(c_kv, k_rope, warp, p, lane, rope, norm_w, eps, v[0], v[1], kr);
    const long long slot = cache_slot(block_table, num_seqs, max_blocks, num_blocks, seq_idx[warp], p,
                                      lane == 0 ? err : nullptr);
    if (slot < 0) return;
    uint8_t *crow = codes + slot * kInt4Codes, *srow = scales + slot * kInt4Scales;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        uint32_t h[4] = {int4_known(v[half].x), int4_known(v[half].y), int4_known(v[half].z), int4_known(v[half].w)};
        uint32_t am = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) am = __vmaxu2(am, h[i] & 0x7FFF7FFFu);
        am = __vmaxu2(am, __shfl_xor_sync(0xffffffffu, am, 1));
        const uint32_t b = int4_scale_byte(int4_low(max(am & 0xFFFFu, am >> 16)));
        const float s = int4_scale(b), inv = __frcp_rn(s);
        if (b == 255) {
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = int4_limit(h[i], s);
        }
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w += ((int4_code(int4_low(h[i]), inv) - kInt4CodeBits) << (4 * i)) +
                 ((int4_code(int4_high(h[i]), inv) - kInt4CodeBits) << (16 + 4 * i));
        reinterpret_cast<uint32_t *>(crow)[32 * half + lane] = w;
        if ((lane & 1) == 0) srow[16 * half + (lane >> 1)] = (uint8_t)b;
    }
    uint32_t h = int4_known(*reinterpret_cast<const uint32_t *>(&kr));
    uint32_t am = h & 0x7FFF7FFFu;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) am = __vmaxu2(am, __shfl_xor_sync(0xffffffffu, am, o));
    const uint32_t b = int4_scale_byte(int4_low(max(am & 0xFFFFu, am >> 16)));
    const float s = int4_scale(b), inv = __frcp_rn(s);
    if (b == 255) h = int4_limit(h, s);
    const int i = lane & 3;   // the pair's place in its word
    uint32_t w = ((int4_code(int4_low(h), inv) - kInt4CodeBits) << (4 * i)) +
                 ((int4_code(int4_high(h), inv) - kInt4CodeBits) << (16 + 4 * i));
    w |= __shfl_xor_sync(0xffffffffu, w, 1);
    w |= __shfl_xor_sync(0xffffffffu, w, 2);
    if (i == 0) reinterpret_cast<uint32_t *>(crow + kDc / 2)[lane >> 2] = w;
    if ((lane & 7) == 0) srow[kDc / kInt4Group + (lane >> 3)] = (uint8_t)b;
}

// Rows at T (sequence, position) places, widened to bf16.  Thread = one 8-value
// unit of a row, of four rows, whose loads are in flight together; neighbours'
// 16-byte stores touch.  A place whose slot is invalid gives a row of zeros and an
// error bit.
//
// What bounds it: memory traffic, so loads in flight.  65,536 rows take 20.9 us (97
// MB, 4.7 TB/s), 262,144 rows 73 us (5.3 TB/s); one row a thread at a time 43 and
// 174 us; 8 to 32 rows of a CTA in nine units a thread 20.7 to 29 us, and 2 us more
// on 77 to 4,096 rows, where the CTAs are few.
constexpr int kInt4GatherRows = 4, kInt4GatherThreads = kRow / 8;

__global__ void __launch_bounds__(kInt4GatherThreads)
gather_latent_int4_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales, int num_blocks,
                          const int32_t *__restrict__ seq_idx, const int32_t *__restrict__ pos, int T,
                          const int32_t *__restrict__ block_table, int num_seqs, int max_blocks,
                          bf16 *__restrict__ out, uint32_t *err)
{
    __shared__ long long slots[kInt4GatherRows];
    const long long t0 = (long long)blockIdx.x * kInt4GatherRows;
    const int c = threadIdx.x;
    if (c < kInt4GatherRows)
        slots[c] = t0 + c < T ? cache_slot(block_table, num_seqs, max_blocks, num_blocks, seq_idx[t0 + c], pos[t0 + c],
                                           err) : -1;
    __syncthreads();
    uint32_t w[kInt4GatherRows], b[kInt4GatherRows];
#pragma unroll
    for (int e = 0; e < kInt4GatherRows; ++e) {
        const long long slot = slots[e];
        w[e] = 0x88888888u;   // eight codes of value 0
        b[e] = 0;
        if (slot >= 0) {
            w[e] = reinterpret_cast<const uint32_t *>(codes + slot * kInt4Codes)[c];
            b[e] = scales[slot * kInt4Scales + (c >> 1)];
        }
    }
    uint4 *o = reinterpret_cast<uint4 *>(out + t0 * kRow) + c;
#pragma unroll
    for (int e = 0; e < kInt4GatherRows; ++e) {
        __nv_bfloat162 s2, m24s2;
        int4_scale2(b[e], s2, m24s2);
        if (t0 + e < T) o[e * kInt4GatherThreads] = int4_widen8(w[e], s2, m24s2);
    }
}

}  // namespace mla
