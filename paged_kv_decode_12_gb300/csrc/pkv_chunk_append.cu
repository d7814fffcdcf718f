// pkv_chunk_append.cu -- norms of the query and key heads, rotation and append of a step's new tokens.
//
// A head's row x of 64 values, with weights w and the rotation of its token:
//     y = R(x * w) / sqrt(mean(x^2) + eps),   R: pair (i, i + 32) turned by pos[axis(i)] * theta^(-2i / 64).
// The factor in front is one number a row, so the rotation comes first: the products x * w of two
// BF16 values are exact in FP32, the rotation keeps what cancels (rope_comb's arithmetic), and the
// factor multiplies its sum.  Where the products of the rotation nearly cancel, the error stays
// relative to the small result.  Sum and factor carry a second FP32 part: a value is the FP32 number
// next to the exact one (but for about 2^-40 of it), then rounded to BF16, so that FP8 rows, whose scale
// is their rounded maximum, come out as from 64 bits.
//
// Query rows, which nothing is derived from but their BF16 values, do with one FP32 part: within 2^-20 before
// that rounding, cancellation or not (turn_query_row).
//
// A warp takes a token, or some of its rounds: 8 lanes a head, 4 pairs a lane (8-byte loads, whole sectors), four
// heads at once, 8 rounds for the query and 2 for the keys and values.  A lane's 4 table entries serve all of its
// rounds.
//
// Many tokens are bound by their bytes and, with FP8 pages, by issue: 16384 with norms 41 us (31.5 at the rate of a
// copy), FP8 48 (29).  Without norms 43 and 51: there the query's rotation is in two FP32 parts as well, because its bits
// are those of the other appends.  One token 2.6 us, 1111 7.4: loads behind one another, slot, position, table entry and
// (of a token that several warps share) row; only the table entry's has to wait for one before it.
#include <cuda_bf16.h>

#include "pkv_fp8.cuh"

namespace pkv {
namespace {

using namespace dev;

constexpr int kRowsWarps = 4, kRowsCtas = 8;  // of an SM: 64 registers a thread
constexpr int kAhead = 2;                      // rounds whose loads are on their way (see the launch)
constexpr int kMaxAxes = 3;

struct ChunkAppendArgs {
    uint8_t *slab;
    int num_pages;
    const uint16_t *k, *v, *q;
    int64_t k_stride, v_stride, q_stride;  // elements from a token to the next
    uint16_t *q_out;
    const uint16_t *q_norm, *k_norm;
    float eps;
    const int64_t *slots;
    const int32_t *pos;
    int64_t pos_stride;
    int axis_end[kMaxAxes];  // first pair behind each axis
    int T;
    const float4 *rope;
    int max_pos;
    int32_t *err;
};

// Four consecutive BF16 values.
__device__ __forceinline__ void values4(uint2 w, float (&x)[4])
{
    x[0] = bf16lo(w.x);
    x[1] = bf16hi(w.x);
    x[2] = bf16lo(w.y);
    x[3] = bf16hi(w.y);
}

__device__ __forceinline__ void load4(const uint16_t *p, float (&x)[4]) { values4(*reinterpret_cast<const uint2 *>(p), x); }

// rope_comb with its last sum left in two parts.
__device__ __forceinline__ void rope_parts(float a, float b, float ch, float cl, float sh, float sl, float &hi, float &lo)
{
    const float p = __fmul_rn(a, ch), pe = __fmaf_rn(a, ch, -p);
    const float r = __fmul_rn(b, sh), re = __fmaf_rn(b, sh, -r);
    const float t = __fadd_rn(p, r), bb = __fsub_rn(t, p);
    const float e = __fadd_rn(__fsub_rn(p, __fsub_rn(t, bb)), __fsub_rn(r, bb));
    lo = __fadd_rn(e, __fadd_rn(__fadd_rn(pe, re), __fmaf_rn(a, cl, __fmul_rn(b, sl))));
    hi = t;
}

// 1 / sqrt(mean + eps) of the 64 values that 8 lanes hold, as two FP32 parts.
__device__ __forceinline__ float2 inverse_norm(const float (&x1)[4], const float (&x2)[4], float eps)
{
    // the sum of squares, each exact in FP32, with what its additions drop
    float s = 0.f, c = 0.f;
    const auto add = [&](float v) {
        const float t = __fmaf_rn(v, v, s);
        c = __fadd_rn(c, __fmaf_rn(v, v, __fsub_rn(s, t)));
        s = t;
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        add(x1[i]);
        add(x2[i]);
    }
#pragma unroll
    for (int off = 1; off < 8; off <<= 1) {
        const float s2 = __shfl_xor_sync(kFull, s, off), c2 = __shfl_xor_sync(kFull, c, off);
        const float t = __fadd_rn(s, s2), bb = __fsub_rn(t, s);
        c = __fadd_rn(__fadd_rn(c, c2), __fadd_rn(__fsub_rn(s, __fsub_rn(t, bb)), __fsub_rn(s2, bb)));
        s = t;
    }
    // m = mean + eps (s / 64 is exact)
    const float h = s * (1.f / kD), t = __fadd_rn(h, eps), bb = __fsub_rn(t, h);
    const float e = __fadd_rn(__fadd_rn(__fsub_rn(h, __fsub_rn(t, bb)), __fsub_rn(eps, bb)), c * (1.f / kD));
    // one step of Newton's iteration for 1 / sqrt: r (1 + (1 - m r^2) / 2)
    const float r = rsqrtf(t);
    const float g = __fmul_rn(r, r), ge = __fmaf_rn(r, r, -g);
    const float d = __fsub_rn(__fsub_rn(__fmaf_rn(-t, g, 1.f), __fmul_rn(t, ge)), __fmul_rn(e, g));
    return make_float2(r, r > 0.f ? __fmul_rn(__fmul_rn(0.5f, r), d) : 0.f);
}

// The rotated (and normed) values of a lane's 4 pairs of a row.
template <bool NORM>
__device__ __forceinline__ void turn_row(float (&x1)[4], float (&x2)[4], const float (&w1)[4], const float (&w2)[4], float eps,
                                         const float4 (&cs)[4])
{
    float2 f = make_float2(1.f, 0.f);
    if constexpr (NORM) {
        f = inverse_norm(x1, x2, eps);
        if (!(f.x > 0.f)) {  // (the 8 lanes of a head alike) the squares left FP32's range: once more, scaled down
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x1[i] *= 0x1p-80f;
                x2[i] *= 0x1p-80f;
            }
        }
        if (__any_sync(kFull, !(f.x > 0.f))) {
            const float2 g = inverse_norm(x1, x2, 0.f);
            if (!(f.x > 0.f))
                f = g;
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = NORM ? x1[i] * w1[i] : x1[i], b = NORM ? x2[i] * w2[i] : x2[i];
        if constexpr (NORM) {
            float h1, l1, h2, l2;
            rope_parts(a, -b, cs[i].x, cs[i].z, cs[i].y, cs[i].w, h1, l1);
            rope_parts(b, a, cs[i].x, cs[i].z, cs[i].y, cs[i].w, h2, l2);
            const float p1 = __fmul_rn(h1, f.x), p2 = __fmul_rn(h2, f.x);
            const float r1 = __fadd_rn(__fmaf_rn(h1, f.x, -p1), __fmaf_rn(h1, f.y, __fmul_rn(l1, f.x)));
            const float r2 = __fadd_rn(__fmaf_rn(h2, f.x, -p2), __fmaf_rn(h2, f.y, __fmul_rn(l2, f.x)));
            x1[i] = __fadd_rn(p1, r1);
            x2[i] = __fadd_rn(p2, r2);
        } else {
            rope_rotate_pair(a, b, cs[i], x1[i], x2[i]);
        }
    }
}

// The same of a query row, with norm: rotation by fused multiply-adds whose first product's remainder is kept (Kahan's
// difference of products: what cancels, cancels exactly), sum and factor in FP32.
__device__ __forceinline__ void turn_query_row(float (&x1)[4], float (&x2)[4], const float (&w1)[4], const float (&w2)[4],
                                               float eps, const float4 (&cs)[4])
{
    const auto factor = [&](float e) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            s = fmaf(x1[i], x1[i], fmaf(x2[i], x2[i], s));
#pragma unroll
        for (int off = 1; off < 8; off <<= 1)
            s += __shfl_xor_sync(kFull, s, off);
        return rsqrtf(fmaf(s, 1.f / kD, e));
    };
    float f = factor(eps);
    const bool out = !(f > 0.f);  // (the 8 lanes of a head alike) the squares left FP32's range: once more, scaled down
    if (__any_sync(kFull, out)) {
        if (out) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x1[i] *= 0x1p-80f;
                x2[i] *= 0x1p-80f;
            }
        }
        const float g = factor(0.f);
        if (out)
            f = g;
    }
    const auto turned = [](float a, float b, float ch, float cl, float sh, float sl) {  // a c + b s
        const float p = __fmul_rn(b, sh), e = __fmaf_rn(b, sh, -p);
        return __fadd_rn(__fmaf_rn(a, ch, p), __fmaf_rn(a, cl, __fmaf_rn(b, sl, e)));
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = x1[i] * w1[i], b = x2[i] * w2[i];
        x1[i] = turned(a, -b, cs[i].x, cs[i].z, cs[i].y, cs[i].w) * f;
        x2[i] = turned(b, a, cs[i].x, cs[i].z, cs[i].y, cs[i].w) * f;
    }
}

__device__ __forceinline__ uint2 pack4(const float (&x)[4])
{
    return make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
}

// Row scale of the FP8 row whose BF16 values 8 lanes hold, 8 each.
__device__ __forceinline__ float row_scale8(const float (&x1)[4], const float (&x2)[4])
{
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        m = fmaxf(m, fmaxf(fabsf(x1[i]), fabsf(x2[i])));
#pragma unroll
    for (int off = 1; off < 8; off <<= 1)
        m = fmaxf(m, __shfl_xor_sync(kFull, m, off));
    return fp8::row_scale(m);
}

// E4M3 codes of x / scale, the quotient as FP32 division rounds it: from the rounded reciprocal, one step with
// the remainder gives the rounded quotient (Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990).  (The remainder with its sign turned: one of nothing is then -0 in the step, and a
// quotient of -0 stays one.)  A scale whose reciprocal leaves the range takes the division.
__device__ __forceinline__ uint32_t codes4(const float (&x)[4], float scale, float inv)
{
    float q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float y = __fmul_rn(x[i], inv);
        q[i] = __fmaf_rn(-__fmaf_rn(y, scale, -x[i]), inv, y);
    }
    if (!(scale >= 0x1p-100f && scale <= 0x1p100f)) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            q[i] = __fdiv_rn(x[i], scale);
    }
    return fp8::e4m3x2_of(q[0], q[1]) | fp8::e4m3x2_of(q[2], q[3]) << 16;
}

// One token: `part` of `parts` takes the rounds part, part + parts, ... of 10 (8 of four query heads, 2 of four KV heads).
// WHOLE: one warp takes them all, and the first loads go out before slot, position and table entries are there.
template <bool FP8, bool NORM, bool WHOLE>
__device__ __forceinline__ void token_rows(const ChunkAppendArgs &a, int t, int part_, int parts_)
{
    const int part = WHOLE ? 0 : part_, parts = WHOLE ? 1 : parts_;
    const int lane = threadIdx.x & 31, j = lane & 7, hh = lane >> 3;
    const int64_t at = a.slots[t];
    uint2 ahead[kAhead][2];  // the query's next rounds
    const uint16_t *src_q = a.q + t * a.q_stride + hh * kD + 4 * j;
    const auto load_round = [&](int r, uint2 (&w)[2]) {
        w[0] = *reinterpret_cast<const uint2 *>(src_q + r * 4 * kD);
        w[1] = *reinterpret_cast<const uint2 *>(src_q + r * 4 * kD + kD / 2);
    };
    if (WHOLE && a.q) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            load_round(k, ahead[k]);
    }
    if (at == -1)
        return;  // padding
    if (at < 0 || at >= (int64_t)a.num_pages * kPage) {
        if (lane == 0 && part == 0 && a.err)
            atomicOr(a.err, PKV_DEVERR_PAGE_RANGE);
        return;
    }
    float4 cs[4];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int pair = 4 * j + i, axis = (pair >= a.axis_end[0]) + (pair >= a.axis_end[1]);
        const int p = a.pos[axis * a.pos_stride + t];
        bad |= p < 0 || p >= a.max_pos;
        cs[i] = bad ? make_float4(1.f, 0.f, 0.f, 0.f) : a.rope[(size_t)p * (kD / 2) + pair];
    }
    if (__any_sync(kFull, bad)) {
        if (lane == 0 && part == 0 && a.err)
            atomicOr(a.err, PKV_DEVERR_LENGTH);
        return;
    }
    const int slot = (int)(at % kPage);
    float w1[4] = {1.f, 1.f, 1.f, 1.f}, w2[4] = {1.f, 1.f, 1.f, 1.f};
    if (a.q) {
        if constexpr (NORM) {
            load4(a.q_norm + 4 * j, w1);
            load4(a.q_norm + kD / 2 + 4 * j, w2);
        }
        uint16_t *dst = a.q_out + (size_t)t * kHq * kD + hh * kD + 4 * j;
        const auto round = [&](int r, float (&x1)[4], float (&x2)[4]) {
            if constexpr (NORM)
                turn_query_row(x1, x2, w1, w2, a.eps, cs);
            else
                turn_row<false>(x1, x2, w1, w2, a.eps, cs);
            *reinterpret_cast<uint2 *>(dst + r * 4 * kD) = pack4(x1);
            *reinterpret_cast<uint2 *>(dst + r * 4 * kD + kD / 2) = pack4(x2);
        };
        float x1[4], x2[4];
        if constexpr (WHOLE) {
#pragma unroll
            for (int r = 0; r < kHq / 4; ++r) {
                values4(ahead[r % kAhead][0], x1);
                values4(ahead[r % kAhead][1], x2);
                if (r + kAhead < kHq / 4)
                    load_round(r + kAhead, ahead[r % kAhead]);
                round(r, x1, x2);
            }
        } else {
#pragma unroll 2
            for (int r = part; r < kHq / 4; r += parts) {
                uint2 w[2];
                load_round(r, w);
                values4(w[0], x1);
                values4(w[1], x2);
                round(r, x1, x2);
            }
        }
    }
    if constexpr (NORM) {
        load4(a.k_norm + 4 * j, w1);
        load4(a.k_norm + kD / 2 + 4 * j, w2);
    }
    for (int r = (part + parts - kHq / 4 % parts) % parts; r < kHkv / 4; r += parts) {
        const int h = 4 * r + hh;
        float x1[4], x2[4];
        const uint16_t *src = a.k + t * a.k_stride + h * kD + 4 * j, *val = a.v + t * a.v_stride + h * kD + 4 * j;
        load4(src, x1);
        load4(src + kD / 2, x2);
        const uint2 v1 = *reinterpret_cast<const uint2 *>(val), v2 = *reinterpret_cast<const uint2 *>(val + kD / 2);
        turn_row<NORM>(x1, x2, w1, w2, a.eps, cs);
        if constexpr (!FP8) {
            uint16_t *page = reinterpret_cast<uint16_t *>(a.slab) + (size_t)(at / kPage) * kPageElems;
            uint16_t *dst = page + (h * kPage + slot) * kD + 4 * j;
            *reinterpret_cast<uint2 *>(dst) = pack4(x1);
            *reinterpret_cast<uint2 *>(dst + kD / 2) = pack4(x2);
            dst += kHkv * kPage * kD;
            *reinterpret_cast<uint2 *>(dst) = v1;
            *reinterpret_cast<uint2 *>(dst + kD / 2) = v2;
        } else {
            uint8_t *unit = a.slab + (size_t)(at / kPage) * kFp8PageBytes + (size_t)h * kFp8Unit;
            float *scales = reinterpret_cast<float *>(unit + kFp8UnitCodes);
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // (what is quantized is the BF16 value)
                x1[i] = fp8::bf16_round(x1[i]);
                x2[i] = fp8::bf16_round(x2[i]);
            }
            const float ks = row_scale8(x1, x2), ki = __frcp_rn(ks);
            *reinterpret_cast<uint32_t *>(unit + slot * kD + 4 * j) = codes4(x1, ks, ki);
            *reinterpret_cast<uint32_t *>(unit + slot * kD + kD / 2 + 4 * j) = codes4(x2, ks, ki);
            float y1[4] = {bf16lo(v1.x), bf16hi(v1.x), bf16lo(v1.y), bf16hi(v1.y)};
            float y2[4] = {bf16lo(v2.x), bf16hi(v2.x), bf16lo(v2.y), bf16hi(v2.y)};
            const float vs = row_scale8(y1, y2), vi = __frcp_rn(vs);
            const uint32_t c1 = codes4(y1, vs, vi), c2 = codes4(y2, vs, vi);
            uint8_t *vt = unit + fp8::kFp8Tile;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                vt[fp8::v_code_offset(slot, 4 * j + i)] = (uint8_t)(c1 >> (8 * i));
                vt[fp8::v_code_offset(slot, kD / 2 + 4 * j + i)] = (uint8_t)(c2 >> (8 * i));
            }
            if (j == 0) {
                scales[slot] = ks;
                scales[kPage + slot] = vs;
            }
        }
    }
}

template <bool FP8, bool NORM, bool WHOLE>
__global__ void __launch_bounds__(kRowsWarps * 32, kRowsCtas) chunk_append_kernel(ChunkAppendArgs a, int parts)
{
    grid_dependency_wait();
    allow_dependent_launch();
    const int w = blockIdx.x * kRowsWarps + (threadIdx.x >> 5);
    const int t = w / parts;
    if (t < a.T)
        token_rows<FP8, NORM, WHOLE>(a, t, w - t * parts, parts);
}

// Few tokens are shared by several warps each, so that their rounds overlap: enough of them for 32 warps an SM.  Many
// have a warp each, which loads two rounds ahead (16384 tokens: 41 us, FP8 48, where the loop over its rounds took 52 and
// 60; with four or eight rounds ahead, at more registers and fewer warps, 42 to 47 and 49 to 58).
constexpr int kEnoughWarps = 152 * 32;

template <bool FP8, bool NORM>
int launch_chunk_append(const ChunkAppendArgs &a, cudaStream_t s)
{
    int parts = 1;
    for (const int p : {2, 5, 10})
        if ((int64_t)a.T * parts < kEnoughWarps)
            parts = p;
    const int64_t warps = (int64_t)a.T * parts;
    return launch_kernel(parts == 1 ? chunk_append_kernel<FP8, NORM, true> : chunk_append_kernel<FP8, NORM, false>, dim3((unsigned)((warps + kRowsWarps - 1) / kRowsWarps)),
                         dim3(kRowsWarps * 32), 0, s, true, a, parts);
}

}  // namespace
}  // namespace pkv

extern "C" int pkv_chunk_append(const pkv_pool *pool, const uint16_t *k, int64_t k_stride, const uint16_t *v,
                                int64_t v_stride, const uint16_t *q, int64_t q_stride, uint16_t *q_out,
                                const uint16_t *q_norm, const uint16_t *k_norm, float eps, const int64_t *slots_dev,
                                const int32_t *pos_dev, int64_t pos_stride, const int32_t *axis_pairs, int T,
                                const float *rope_table, int max_pos, int32_t *dev_err_flag, void *cuda_stream)
{
    using namespace pkv;
    if (!pool || !k || !v || !slots_dev || !pos_dev || !rope_table || (q == nullptr) != (q_out == nullptr) ||
        (k_norm == nullptr && q_norm != nullptr) || (q && (q_norm == nullptr) != (k_norm == nullptr)))
        return PKV_ERR_INVALID_ARG;
    if (T < 1 || T > INT32_MAX / 16 || max_pos < 1)
        return PKV_ERR_INVALID_ARG;
    if (k_norm && !(eps > 0.f && eps < INFINITY))
        return PKV_ERR_INVALID_ARG;
    if (k_stride < kHkv * kD || v_stride < kHkv * kD || (q && q_stride < kHq * kD) ||
        ((k_stride | v_stride | (q ? q_stride : 0)) & 3))
        return PKV_ERR_INVALID_ARG;
    if (q == q_out && q && q_stride != kHq * kD)
        return PKV_ERR_INVALID_ARG;  // rows of another stride would be written over unread ones
    if ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) | reinterpret_cast<uintptr_t>(q) |
         reinterpret_cast<uintptr_t>(q_out) | reinterpret_cast<uintptr_t>(q_norm) | reinterpret_cast<uintptr_t>(k_norm)) & 7u)
        return PKV_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(rope_table) & 15u) || (reinterpret_cast<uintptr_t>(slots_dev) & 7u))
        return PKV_ERR_INVALID_ARG;
    ChunkAppendArgs a;
    a.axis_end[0] = a.axis_end[1] = a.axis_end[2] = kD / 2;
    if (axis_pairs) {
        if (axis_pairs[0] < 0 || axis_pairs[1] < 0 || axis_pairs[2] < 0 || pos_stride < T ||
            (int64_t)axis_pairs[0] + axis_pairs[1] + axis_pairs[2] != kD / 2)
            return PKV_ERR_INVALID_ARG;
        a.axis_end[0] = axis_pairs[0];
        a.axis_end[1] = axis_pairs[0] + axis_pairs[1];
    }
    a.slab = reinterpret_cast<uint8_t *>(pool->slab);
    a.num_pages = pool->num_pages;
    a.k = k;
    a.v = v;
    a.q = q;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_stride = q_stride;
    a.q_out = q_out;
    a.q_norm = q_norm;
    a.k_norm = k_norm;
    a.eps = eps;
    a.slots = slots_dev;
    a.pos = pos_dev;
    a.pos_stride = axis_pairs ? pos_stride : 0;
    a.T = T;
    a.rope = reinterpret_cast<const float4 *>(rope_table);
    a.max_pos = max_pos;
    a.err = dev_err_flag;
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    pages_written(pool, s);  // a decode launch behind it may read these pages
    if (pool->kv_format == PKV_KV_FP8)
        return k_norm ? launch_chunk_append<true, true>(a, s) : launch_chunk_append<true, false>(a, s);
    return k_norm ? launch_chunk_append<false, true>(a, s) : launch_chunk_append<false, false>(a, s);
}
