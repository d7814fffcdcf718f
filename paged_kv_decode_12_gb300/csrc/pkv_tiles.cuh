// pkv_tiles.cuh -- key tiles on the 5th-generation tensor cores, shared by the shared-prefix kernel
// (pkv_shared.cu) and the attention of chunks (pkv_chunk.cu): the layout of a stage, the matrix products of half a
// tile, the conversion of FP8 units, and how far weights go.  Not part of the ABI.
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

// The matrix products of a key tile, issued by one elected thread of a converged warp.  A key tile goes
// through in two halves of 64 tokens (slots 0..7 and 8..15 of its 8 pages), each with scores of its own
// in tensor memory: while the softmax of one half runs, the other half's weights meet the values and its
// columns take the next tile's scores.
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

// The reference m of a row's softmax is its first half tile's maximum, and it stays until a
// half tile's weights sum to 2^64 or more: FP32 and BF16 hold 2^127, so m, l and O remain a
// valid log-sum-exp triple that far above m, and no maximum is taken on the way.  (Moving m for
// every score 2^8 above it, as narrower types need, made most half tiles of 32 rows rescale O.)
// O is finite for values up to 2^45: 2^64 times that, over at most 2^18 half tiles.
constexpr float kMostWeight = 18446744073709551616.f;

}  // namespace tiles
}  // namespace pkv
