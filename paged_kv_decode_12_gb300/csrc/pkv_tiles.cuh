// pkv_tiles.cuh -- key tiles on the 5th-generation tensor cores, shared by the shared-prefix kernel
// (pkv_shared.cu) and the attention of chunks (pkv_chunk.cu): the layout of a stage, the matrix products of half a
// tile, the conversion of FP8 units, and what makes weights of scores.  Not part of the ABI.
#pragma once

#include "pkv_fp8.cuh"
#include "pkv_tc.cuh"

namespace pkv {
namespace tiles {

using namespace dev;

constexpr int kTilePages = 8;                        // pages of one key tile: 128 tokens
constexpr int kHalf = kTilePages * kPage / 2;        // its halves
constexpr int kRowTile = 128;                        // query rows of one tensor-core tile
constexpr int kStageSize = kTilePages * kStageBytes; // 32 KiB: 8 x (K rows, V rows)
constexpr int kRawSize = kTilePages * kFp8Unit;      // 17 KiB: FP8 units as they lie in the pages
constexpr int kScales = 3 * kTilePages * kPage;      // row scales of a tile: K's, V's, 1 / V's

// Two E4M3 codes as BF16 (exact: 4 significant bits, exponents in range; NaN stays NaN).
__device__ __forceinline__ uint32_t bf16x2_of_f16x2(uint32_t h)
{
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    return pack_bf16x2(f.x, f.y);
}

__device__ __forceinline__ void bf16_of_e4m3x4(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    uint32_t a, b;
    fp8::e4m3x4_to_f16x2(w, a, b);
    lo = bf16x2_of_f16x2(a);
    hi = bf16x2_of_f16x2(b);
}

// One tile of raw units into a stage of the BF16 layout, by 128 threads.
__device__ __forceinline__ void convert_codes(const uint8_t *raw, uint8_t *dst, int t)
{
#pragma unroll
    for (int k = 0; k < 4; ++k) {  // K: 16 codes of a row, two chunks of 8 values
        const int u = t + 128 * k, page = u / 64, row = u % 64 / 4, part = u % 4;
        const uint4 c = *reinterpret_cast<const uint4 *>(raw + page * kFp8Unit + row * kD + part * 16);
        uint4 lo, hi;
        bf16_of_e4m3x4(c.x, lo.x, lo.y);
        bf16_of_e4m3x4(c.y, lo.z, lo.w);
        bf16_of_e4m3x4(c.z, hi.x, hi.y);
        bf16_of_e4m3x4(c.w, hi.z, hi.w);
        *reinterpret_cast<uint4 *>(dst + page * kStageBytes + swz(row, 2 * part)) = lo;
        *reinterpret_cast<uint4 *>(dst + page * kStageBytes + swz(row, 2 * part + 1)) = hi;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {  // V: 8 dims of the tokens 2 pair, 2 pair + 1, codes alternating
        const int u = t + 128 * k, page = u / 64, pair = u % 64 / 8, at = u % 8, chunk = at ^ ((2 * pair) & 7);
        const uint4 c = *reinterpret_cast<const uint4 *>(raw + page * kFp8Unit + fp8::kFp8Tile + pair * 2 * kD + at * 16);
        uint4 even, odd;
        bf16_of_e4m3x4(__byte_perm(c.x, c.y, 0x6420), even.x, even.y);
        bf16_of_e4m3x4(__byte_perm(c.z, c.w, 0x6420), even.z, even.w);
        bf16_of_e4m3x4(__byte_perm(c.x, c.y, 0x7531), odd.x, odd.y);
        bf16_of_e4m3x4(__byte_perm(c.z, c.w, 0x7531), odd.z, odd.w);
        uint8_t *v = dst + page * kStageBytes + kTileBytes;
        *reinterpret_cast<uint4 *>(v + swz(2 * pair, chunk)) = even;
        *reinterpret_cast<uint4 *>(v + swz(2 * pair + 1, chunk)) = odd;
    }
}

// Its row scales, [K (times scale log2 e), V, 1 / V][half][64] in the order of the scores' columns.
__device__ __forceinline__ void convert_scales(const uint8_t *raw, float *scales, float scale_log2, int t)
{
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {  // thread = (page, slot)
        const int page = t / kPage, slot = t % kPage;
        const float f = reinterpret_cast<const float *>(raw + page * kFp8Unit + kFp8UnitCodes)[kv * kPage + slot];
        float *to = scales + slot / 8 * 64 + page * 8 + slot % 8;
        if (kv) {  // (a scale below 2^-100, of rows of nothing, as 2^-100: weights are counted by its inverse)
            const float v = fabsf(f) < 0x1p-100f ? 0x1p-100f : f;
            to[128] = v;
            to[256] = __frcp_rn(v);
        } else {
            to[0] = f * scale_log2;
        }
    }
}

// The matrix products of a key tile, issued by one elected thread of a converged warp.  A key tile goes through in two halves of 64 tokens (slots 0..7 and 8..15 of its 8
// pages), each with scores of its own in tensor memory: while the softmax of one half runs, the
// other half's weights meet the values and its columns take the next tile's scores.
__device__ __forceinline__ void issue_scores(uint32_t k, uint32_t s, uint32_t q, uint64_t *done)
{
    // S[128 x 64] = Q K^T: columns 8 p + i are slot 8 h + i of page p (page stride 4 KiB)
    constexpr uint32_t kIdesc = tc::instr_desc(64, true, false), kHi = tc::smem_desc_hi(kStageBytes);
    const uint32_t lo = tc::smem_desc_lo(k, kStageBytes);
    if (tc::elect()) {
        tc::mma_ts<false>(s, q, lo, kHi, kIdesc);
#pragma unroll
        for (int i = 1; i < kD / 16; ++i)
            tc::mma_ts<true>(s, q + i * 8, lo + i * 2, kHi, kIdesc);
        tc::commit(done);
    }
    __syncwarp();
}

// SUM: L += P times 16 columns beside V (of ones; or, STEP bytes / 16 apart for every 16 rows of P, of anything).
template <bool FIRST, bool SUM, int STEP = 0>
__device__ __forceinline__ void issue_output(uint32_t v, uint32_t o, uint32_t p, uint32_t ones, uint32_t l,
                                             uint64_t *free_stage, int uses, uint64_t *done, uint64_t *last)
{
    // O[128 x 64] += P V: 16 columns of P are 8 slots of two pages
    constexpr uint32_t kIdesc = tc::instr_desc(64, true, true), kHi = tc::smem_desc_hi(kStageBytes);
    const uint32_t lo = tc::smem_desc_lo(v, kStageBytes);
    if (tc::elect()) {
        tc::mma_ts<!FIRST>(o, p, lo, kHi, kIdesc);
#pragma unroll
        for (int i = 1; i < kHalf / 16; ++i)
            tc::mma_ts<true>(o, p + i * 8, lo + i * (2 * kStageBytes / 16), kHi, kIdesc);
        if constexpr (SUM) {  // L[128 x 16] += P 1
            constexpr uint32_t kOnes = tc::instr_desc(16, true, false), kOnesHi = tc::smem_desc_hi(1024);
            const uint32_t one = tc::smem_desc_lo(ones, 1024);
            tc::mma_ts<!FIRST>(l, p, one, kOnesHi, kOnes);
#pragma unroll
            for (int i = 1; i < kHalf / 16; ++i)
                tc::mma_ts<true>(l, p + i * 8, one + i * STEP, kOnesHi, kOnes);
        }
        tc::commit(done);
        if (last)
            tc::commit(last);
        if (free_stage) {
            tc::commit(free_stage);
            if (uses > 1)
                tc::commit(free_stage);
        }
    }
    __syncwarp();
}

// What turns 64 scores into exponents and weights into the second product's operand: one
// factor, or (FP8) a factor and a scale for every column.
struct OneFactor {
    static constexpr bool kSum = false;  // the sum is made by the matrix instruction
    float c;
    __device__ __forceinline__ float2 factor(int) const { return make_float2(c, c); }
    __device__ __forceinline__ float2 weight(int, float2 e) const { return e; }
    __device__ __forceinline__ float2 counted(int, float2 e, uint32_t) const { return e; }
};

struct RowScales {
    static constexpr bool kSum = true;
    const float2 *k, *v, *inverse;  // 32 pairs of columns
    __device__ __forceinline__ float2 factor(int i) const { return k[i]; }
    __device__ __forceinline__ float2 weight(int i, float2 e) const { return tc::mul2(e, v[i]); }
    // The weight that the product holds: what was rounded, without V's scale again.
    __device__ __forceinline__ float2 counted(int i, float2, uint32_t p) const
    {
        return tc::mul2(make_float2(__uint_as_float(p << 16), __uint_as_float(p & 0xffff0000u)), inverse[i]);
    }
};

// Which of a row's 64 scores of half a key tile count; drop() replaces those of pair i of columns
// 32 k .. that do not.
struct EveryColumn {
    __device__ __forceinline__ void drop(int, int, float2 &, float) const {}
};

// The first `pages` pages of the tile.
struct FirstPages {
    int pages;
    __device__ __forceinline__ void drop(int k, int i, float2 &x, float to) const
    {
        if (!(k * 4 + i / 4 < pages))
            x = make_float2(to, to);
    }
};

// 32 scores of one query row (columns 32 k ..) as weights 2^(S c - m): their sum, and the weights
// in pairs rounded to BF16 (half a step, 2^-8) for the second product: what the matrix instruction
// takes beside BF16 values.  Columns that the mask does not keep weigh nothing.  Four chains of
// sums, so that no chain's latency is the time of the whole.
//
// BF16 pages: the softmax's sum is of the weights as rounded, made by the matrix instruction too (L
// += P 1, 16 equal columns), so that the quotient has none of their rounding where few weights make
// it.  256 sequences behind 32768 tokens: error 0.0017 in 94 us, where the sum of the unrounded
// weights, which this function returns, gives 0.0023 in 92, and unpacking the rounded ones took 108.
// FP8 pages: what is rounded is the weight times V's row scale; the sum takes it times the scale's
// inverse (error 0.0017 instead of 0.0023; 72 sequences in 5 groups 32 us instead of 31).
template <class Mask, class Scale>
__device__ __forceinline__ float make_weights(uint32_t ts, int k, const Scale &sc, const Mask &mask, float m,
                                              uint32_t (&pk)[16])
{
    uint32_t w[32];
    tc::ld32(ts + k * 32, w);
    float2 sum[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        sum[i] = make_float2(0.f, 0.f);
    const float2 m2 = make_float2(-m, -m);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float2 x =
            tc::fma2(make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1])), sc.factor(k * 16 + i), m2);
        float2 e = make_float2(ex2_approx(x.x), ex2_approx(x.y));
        mask.drop(k, i, e, 0.f);
        const float2 p = sc.weight(k * 16 + i, e);
        pk[i] = pack_bf16x2(p.x, p.y);
        sum[i % 4] = tc::add2(sum[i % 4], sc.counted(k * 16 + i, e, pk[i]));
    }
    const float2 s = tc::add2(tc::add2(sum[0], sum[1]), tc::add2(sum[2], sum[3]));
    return s.x + s.y;
}

// Their maximum, times the factors.
template <class Mask, class Scale>
__device__ __forceinline__ float max_score(uint32_t ts, int k, const Scale &sc, const Mask &mask)
{
    uint32_t w[32];
    tc::ld32(ts + k * 32, w);
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float2 x = tc::mul2(make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1])), sc.factor(k * 16 + i));
        mask.drop(k, i, x, -INFINITY);
        mx = tc::max3(mx, x.x, x.y);
    }
    return mx;
}

// The reference m of a row's softmax is its first half tile's maximum, and it stays until a
// half tile's weights sum to 2^64 or more: FP32 and BF16 hold 2^127, so m, l and O remain a
// valid log-sum-exp triple that far above m, and no maximum is taken on the way.  (Moving m for
// every score 2^8 above it, as narrower types need, made most half tiles of 32 rows rescale O.)
// O is finite for values up to 2^45: 2^64 times that, over at most 2^18 half tiles.
constexpr float kMostWeight = 18446744073709551616.f;

// An item's first half tile: the row's maximum.  (Not inlined: the loop would pay for its
// registers; 256 sequences behind 32768 tokens 94.5 us instead of 95.1, though 4 behind 512 tokens
// 7.5 instead of 7.2.)
template <class Mask, class Scale>
__device__ __noinline__ float first_reference(uint32_t ts, Scale sc, Mask mask)
{
    return fmaxf(max_score(ts, 0, sc, mask), max_score(ts, 1, sc, mask));
}


}  // namespace tiles
}  // namespace pkv
