// pkv_step.cuh -- the grid kernels of the decode path as templates: one CTA per
// (sequence, KV head, chunk of pages), with or without the append, over BF16 or FP8
// pages, and over all of a sequence's pages or a selection of them.  pkv_step.cu
// (every page) describes the unit of work; pkv_window.cu, pkv_shared.cu and
// pkv_scored.cu instantiate the kernels for their own selections.
#pragma once

#include <cuda_bf16.h>

#include <algorithm>
#include <climits>
#include <type_traits>

#include "pkv_device.cuh"
#include "pkv_fp8.cuh"

namespace pkv {
namespace {

using namespace dev;

// ------------------------------------------------------------------ page selections

// Which pages a sequence's units go through, in which order, and which of a page's
// tokens they attend to.  A selection makes a list for (sequence b, length L):
//   ok()         false: the sequence is invalid (its outputs are zeros, the flag is set)
//   count()      pages in the list (0: the sequence has one unit without pages)
//   logical(i)   the sequence's page that entry i is, increasing in i
//   before(j)    entries whose page is below j
//   tokens(j)    the tokens of page j attended to
//   kWhole       pages attended to as a whole go through code without a mask; whole(j) says which
//                (256 windows of 4112 FP8 tokens 181 us instead of 187; no faster for whole
//                sequences, whose masks are one comparison)
//   first_slot() partials of the sequence that another kernel writes: they are merged
//                before the units' own
// and says
//   kIdentity    entry i is page i whatever L is: the table is read along with the length
//   kSortable    the list depends on L alone, so that units can be dispatched by size
//   kLateWait    the dependency wait comes before the partials are published instead of
//                before the query rows are read
//   kPublish     units only write their partials, for another kernel to merge; the grid ends
//                after the kernel that it follows, because its first CTA waits for it
//   kLoops       a CTA goes on to chunk c + gridDim.z: the grid need not have a CTA for every
//                chunk of the table's width, which with wide tables and short sequences would
//                be mostly CTAs with nothing to do
//   kFine        scores of FP8 pages for FP32 outputs
// `emit(b, g)` makes what takes the units' scores, `skipped(b, g, j0, jn)` is told of a
// unit that a bad page id keeps from being computed, `finished(b, g, L, M, l, scratch)` is
// called by all threads of the unit that finishes a (sequence, KV head), each with its
// head's softmax statistics; `scratch` is shared memory that the unit has done with.
struct AllPages {
    static constexpr bool kIdentity = true, kSortable = true, kLateWait = false, kPublish = false, kLoops = false,
                          kFine = false;
    __device__ __forceinline__ WholeSequence list(int, int L) const { return {L}; }
    __device__ __forceinline__ EmitNothing emit(int, int) const { return {}; }
    __device__ __forceinline__ void skipped(int, int, int, int) const {}
    __device__ __forceinline__ void finished(int, int, int, float, float, float *) const {}
};

struct StepArgs {
    int num_pages;
    uint16_t *slab;
    const uint16_t *k_new;   // [B][8][64] (APPEND)
    const uint16_t *v_new;   // [B][8][64] (APPEND)
    uint16_t *q;             // [B][32][64], rotated in place (APPEND) or read as given
    const int32_t *bt;       // [B][max_blocks]
    int max_blocks;
    const int32_t *seq_lens; // [B]
    const float4 *rope;      // [max_pos][32] {cos, sin} high then low FP32 parts (APPEND)
    int max_pos;             // APPEND: rope rows; otherwise INT_MAX
    float scale_log2;
    int pages_per_chunk;
    int *counters;           // [B][8], zero between launches
    float2 *part_ml;         // [B][32][max_chunks]
    float *part_o;           // [B][32][max_chunks][64]
    int max_chunks;          // partials per (sequence, head)
    int unit_chunks;         // CTAs per (sequence, KV head) in the grid
    uint16_t *out;           // [B][32][64]
    int32_t *err;
    int sorted;              // units dispatched largest first (PKV_STEP_SORTED)
    int expire_seq;          // testing aid: this sequence's first page waits give up at once (-1: none)
};

constexpr int kMaxSortedBatch = 1024;
static_assert(kMaxPagesPerChunk + 1 + kWarps + 5 <= kWarps * kScratchFloats, "sorted-order scratch");

// Take a ticket: atomic increment with release and acquire semantics at GPU scope.
__device__ __forceinline__ int ticket_acq_rel(int *counter)
{
    int t;
    asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(t) : "l"(counter) : "memory");
    return t;
}

__device__ __forceinline__ uint16_t bf16_bits(float x)
{
    const __nv_bfloat16 h = __float2bfloat16_rn(x);
    return *reinterpret_cast<const uint16_t *>(&h);
}

__device__ __forceinline__ float bf16_value(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }

__device__ __forceinline__ bool length_ok(const StepArgs &a, int L)
{
    return L >= 1 && L <= a.max_blocks * kPage && L <= a.max_pos;
}

// ------------------------------------------------------------------ sorted unit order

// A sequence's work units per KV head: nfull chunks of pages_per_chunk pages and,
// if rem > 0, a last chunk of rem pages; an invalid length has one empty unit.
struct SeqUnits {
    int nfull, rem;
    bool valid;
};

template <class Sel>
__device__ __forceinline__ SeqUnits seq_units(const StepArgs &a, const Sel &sel, int L)
{
    SeqUnits u;
    u.valid = length_ok(a, L);
    if (!u.valid) {
        u.nfull = 0;
        u.rem = 0;
        return u;
    }
    const int ppc = a.pages_per_chunk;
    const int np = sel.list(0, L).count(), nch = (np + ppc - 1) / ppc, rem = np - (nch - 1) * ppc;
    u.nfull = rem == ppc ? nch : nch - 1;
    u.rem = rem == ppc ? 0 : rem;
    return u;
}

// Units of size s of one sequence (s = pages_per_chunk: full chunks; 0 < s < pages_per_chunk:
// a last chunk; s = 0: the empty unit of an invalid length), all KV heads.
__device__ __forceinline__ int units_of_size(const SeqUnits &u, int s, int ppc)
{
    if (!u.valid)
        return s == 0 ? kHkv : 0;
    if (s == ppc)
        return kHkv * u.nfull;
    return (s != 0 && u.rem == s) ? kHkv : 0;
}

// Exclusive prefix sum over the CTA's kThreads threads; `total` receives the sum.
__device__ __forceinline__ int cta_exclusive_scan(int v, int *wsum, int &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(kFull, x, off);
        if (lane >= off)
            x += y;
    }
    if (lane == 31)
        wsum[warp] = x;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const int t = wsum[w];
        before += w < warp ? t : 0;
        total += t;
    }
    __syncthreads();
    return before + x - v;
}

// Sorted dispatch (PKV_STEP_SORTED): the CTA with linear index lin takes the lin-th
// unit in decreasing order of page count (ties by sequence, then chunk, then KV
// head).  The block scheduler places CTAs in index order on whichever SM has room,
// so the largest units are placed first and the small ones fill the gaps (greedy
// largest-first list scheduling), instead of the grid order's mix.  The order only
// decides which CTA computes which unit: every unit's arithmetic and the chunk-order
// merge are unchanged, so results are identical to the unsorted grid.  All threads
// call it (it uses barriers); `scratch` holds kMaxPagesPerChunk + 1 + kWarps + 5 ints.
// Returns false (for the whole CTA) if lin is past the last unit.
template <class Sel>
__device__ bool sorted_unit(const StepArgs &a, const Sel &sel, int B, int lin, int *scratch, int &b, int &g, int &c)
{
    constexpr int kPer = kMaxSortedBatch / kThreads;  // sequences per thread, at most
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ppc = a.pages_per_chunk;
    int *hist = scratch;                            // [ppc + 1] units per size
    int *wsum = scratch + kMaxPagesPerChunk + 1;    // [kWarps]
    int *res = wsum + kWarps;                       // size, rank, b, g, c
    for (int i = tid; i <= ppc; i += kThreads)
        hist[i] = 0;
    // this thread's contiguous run of sequences, read once (one memory round trip)
    const int per = (B + kThreads - 1) / kThreads;
    const int b0 = min(B, tid * per), nb = min(B, b0 + per) - b0;
    SeqUnits u[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        u[i] = seq_units(a, sel, i < nb ? a.seq_lens[b0 + i] : 0);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (i >= nb)
            break;
        if (!u[i].valid) {
            atomicAdd(&hist[0], kHkv);
        } else {
            if (u[i].nfull)
                atomicAdd(&hist[ppc], kHkv * u[i].nfull);
            if (u[i].rem)
                atomicAdd(&hist[u[i].rem], kHkv);
        }
    }
    __syncthreads();
    if (warp == 0) {  // which size bucket holds rank lin, sizes in decreasing order
        constexpr int kBuckets = (kMaxPagesPerChunk + 1 + 31) / 32;
        int cnt[kBuckets];
        int sum = 0;
#pragma unroll
        for (int i = 0; i < kBuckets; ++i) {
            const int k = lane * kBuckets + i;  // k-th largest size, ppc - k
            cnt[i] = k <= ppc ? hist[ppc - k] : 0;
            sum += cnt[i];
        }
        int x = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(kFull, x, off);
            if (lane >= off)
                x += y;
        }
        const int total = __shfl_sync(kFull, x, 31);
        int start = x - sum;
#pragma unroll
        for (int i = 0; i < kBuckets; ++i) {
            if (lin >= start && lin < start + cnt[i]) {
                res[0] = ppc - (lane * kBuckets + i);
                res[1] = lin - start;
            }
            start += cnt[i];
        }
        if (lane == 0 && lin >= total)
            res[0] = -1;
    }
    __syncthreads();
    const int s = res[0], r = res[1];
    if (s < 0)
        return false;
    int mine = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        mine += i < nb ? units_of_size(u[i], s, ppc) : 0;
    int total;
    const int before = cta_exclusive_scan(mine, wsum, total);
    if (r >= before && r < before + mine) {
        int acc = before;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int n = i < nb ? units_of_size(u[i], s, ppc) : 0;
            if (n > 0 && r >= acc && r < acc + n) {
                const int k = r - acc;
                res[2] = b0 + i;
                if (u[i].valid && s == ppc) {  // full chunks 0 .. nfull-1
                    res[3] = k % kHkv;
                    res[4] = k / kHkv;
                } else {                       // the last chunk, or the empty unit of an invalid length
                    res[3] = k;
                    res[4] = u[i].valid ? u[i].nfull : 0;
                }
            }
            acc += n;
        }
    }
    __syncthreads();
    b = res[2];
    g = res[3];
    c = res[4];
    return true;
}

// All kThreads threads: the 4 query rows of group g into q_rot[4][64] (one pair per
// thread) -- rotated to position pos (APPEND), else as given -- and, for the
// sequence's last chunk (APPEND), the new token's rotated key row and its value row
// into new_kv[2][64].
template <bool APPEND>
__device__ __forceinline__ void unit_rows(const StepArgs &a, int b, int g, int pos, bool last_chunk, uint16_t *q_rot,
                                          uint16_t *new_kv)
{
    const int hl = threadIdx.x >> 5, i = threadIdx.x & 31;
    const uint16_t *qrow = a.q + ((size_t)b * kHq + g * kGroup + hl) * kD;
    if (!APPEND) {
        reinterpret_cast<uint32_t *>(q_rot + hl * kD)[i] = reinterpret_cast<const uint32_t *>(qrow)[i];
        return;
    }
    const float4 cs = a.rope[(size_t)pos * (kD / 2) + i];
    float y1, y2;
    rope_rotate_pair(bf16_value(qrow[i]), bf16_value(qrow[i + kD / 2]), cs, y1, y2);
    q_rot[hl * kD + i] = bf16_bits(y1);
    q_rot[hl * kD + i + kD / 2] = bf16_bits(y2);
    if (last_chunk && hl == 0) {
        const uint16_t *krow = a.k_new + ((size_t)b * kHkv + g) * kD;
        rope_rotate_pair(bf16_value(krow[i]), bf16_value(krow[i + kD / 2]), cs, y1, y2);
        new_kv[i] = bf16_bits(y1);
        new_kv[i + kD / 2] = bf16_bits(y2);
    } else if (last_chunk && hl == 1) {
        reinterpret_cast<uint32_t *>(new_kv + kD)[i] =
            reinterpret_cast<const uint32_t *>(a.v_new + ((size_t)b * kHkv + g) * kD)[i];
    }
}

// Threads 0..15: the appended token's K row and V row into their page slot.
__device__ __forceinline__ void store_new_token(const StepArgs &a, int page, int g, int slot, const uint16_t *new_kv)
{
    const int part = threadIdx.x >> 3, ch = threadIdx.x & 7;  // part 0: K row, 1: V row
    uint16_t *row = a.slab + (size_t)page * kPageElems + ((size_t)(part * kHkv + g) * kPage + slot) * kD;
    reinterpret_cast<uint4 *>(row)[ch] = reinterpret_cast<const uint4 *>(new_kv + part * kD)[ch];
}

// The shared-memory copy of the last page carries the slot's previous contents:
// lanes 0..15 overwrite it with the appended token (then the warp syncs).
__device__ __forceinline__ void patch_stage(uint8_t *stage, int slot, const uint16_t *new_kv, int lane)
{
    if (lane < 16) {
        const int part = lane >> 3, ch = lane & 7;
        *reinterpret_cast<uint4 *>(stage + part * kTileBytes + swz(slot, ch)) =
            reinterpret_cast<const uint4 *>(new_kv + part * kD)[ch];
    }
    __syncwarp();
}

// Zeros for the 4 heads of an invalid sequence (one (head, dim pair) per thread).
__device__ __forceinline__ void write_zero_unit(const StepArgs &a, int b, int g)
{
    reinterpret_cast<uint32_t *>(a.out + ((size_t)b * kHq + g * kGroup + (threadIdx.x >> 5)) * kD)[threadIdx.x & 31] =
        0u;
    if (threadIdx.x == 0 && a.err)
        atomicOr(a.err, PKV_DEVERR_LENGTH);
}

// Chunk counts up to which the merging unit holds every partial in registers.
constexpr int kMergeRegs = 8;

// The log-sum-exp merge, in chunk order, of a head's partials (ml_row, and o_col one dim pair).  A partial without
// a maximum counts nothing; where its scores are not numbers, neither are its sums, and they go on.
__device__ __forceinline__ void merge_partials(const float2 *ml_row, const float2 *o_col, int nchunks, float &Mx, float &ls,
                                               float &r0, float &r1)
{
    ls = r0 = r1 = 0.f;
    Mx = -INFINITY;
    if (nchunks <= kMergeRegs) {
        // every partial loaded before the first use: one memory round trip at the end of
        // the sequence's critical path; the arithmetic below is the general loop's
        float2 ml[kMergeRegs], oc[kMergeRegs];
#pragma unroll
        for (int cc = 0; cc < kMergeRegs; ++cc)
            if (cc < nchunks) {
                ml[cc] = __ldcg(ml_row + cc);
                oc[cc] = __ldcg(o_col + cc * (kD / 2));
            }
#pragma unroll
        for (int cc = 0; cc < kMergeRegs; ++cc)
            if (cc < nchunks)
                Mx = fmaxf(Mx, ml[cc].x);
#pragma unroll
        for (int cc = 0; cc < kMergeRegs; ++cc)
            if (cc < nchunks) {
                const float f = (ml[cc].x == -INFINITY) ? 0.f : exp2f(ml[cc].x - Mx);
                ls = fmaf(f, ml[cc].y, ls);
                r0 = fmaf(f, oc[cc].x, r0);
                r1 = fmaf(f, oc[cc].y, r1);
            }
    } else {
#pragma unroll 4
        for (int cc = 0; cc < nchunks; ++cc)
            Mx = fmaxf(Mx, __ldcg(ml_row + cc).x);
#pragma unroll 4
        for (int cc = 0; cc < nchunks; ++cc) {
            const float2 ml = __ldcg(ml_row + cc);
            const float f = (ml.x == -INFINITY) ? 0.f : exp2f(ml.x - Mx);
            const float2 oc = __ldcg(o_col + cc * (kD / 2));
            ls = fmaf(f, ml.y, ls);
            r0 = fmaf(f, oc.x, r0);
            r1 = fmaf(f, oc.y, r1);
        }
    }
}

// The same for many partials: eight at a time are loaded together and joined with what came before,
// one memory round trip for each eight instead of two for each four.
__device__ __forceinline__ void merge_eights(const float2 *ml_row, const float2 *o_col, int n, float &ls, float &r0, float &r1)
{
    float M = -3.402823466e38f;  // (a number, from which a partial without a maximum is infinitely far)
    ls = r0 = r1 = 0.f;
    for (int c0 = 0; c0 < n; c0 += 8) {
        float2 ml[8], oc[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            ml[i] = make_float2(-INFINITY, 0.f);
            oc[i] = make_float2(0.f, 0.f);
            if (c0 + i < n) {
                ml[i] = __ldcg(ml_row + c0 + i);
                oc[i] = __ldcg(o_col + (c0 + i) * (kD / 2));
            }
        }
        float top = M;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            top = fmaxf(top, ml[i].x);
        const float keep = exp2f(M - top);
        ls *= keep;
        r0 *= keep;
        r1 *= keep;
        M = top;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float f = exp2f(ml[i].x - M);
            ls = fmaf(f, ml[i].y, ls);
            r0 = fmaf(f, oc[i].x, r0);
            r1 = fmaf(f, oc[i].y, r1);
        }
    }
}

// Unit epilogue, all threads: combine the warps' states through `state`, then
// write the output (single partial) or publish the chunk partial and take a ticket;
// the unit drawing the last ticket merges every chunk of (b, g) in chunk order, behind
// the `first` partials that another kernel wrote, writes the output (and, WRITE_Q, the
// rotated query rows), and resets the counter.
template <bool WRITE_Q, class Sel, class Warp>
__device__ __forceinline__ void finish_unit(const StepArgs &a, const Sel &sel, Warp &w, float *state, int *ticket,
                                            const uint16_t *q_rot, int b, int g, int c, int nunits, int first, int L)
{
    const int nchunks = first + nunits;
    const int tid = threadIdx.x, warp = tid >> 5;
    __syncthreads();
    w.store_state(state + warp * kStateFloats);
    __syncthreads();
    const int hl = tid >> 5, dp = tid & 31, h = g * kGroup + hl;
    float M, lsum, o0, o1;
    combine_warps(state, hl, dp, M, lsum, o0, o1);
    uint32_t *out_row = reinterpret_cast<uint32_t *>(a.out + ((size_t)b * kHq + h) * kD);
    uint32_t *q_row = reinterpret_cast<uint32_t *>(a.q + ((size_t)b * kHq + h) * kD);
    const uint32_t q_word = reinterpret_cast<const uint32_t *>(q_rot + hl * kD)[dp];
    if (!Sel::kPublish && nchunks == 1) {
        out_row[dp] = finish_pair(o0, o1, lsum);
        sel.finished(b, g, L, M, lsum, state);
        if (WRITE_Q)
            q_row[dp] = q_word;
        if (Sel::kLateWait) {
            grid_dependency_wait();  // this grid ends after the kernel it follows
            allow_dependent_launch();
        }
        return;
    }
    const size_t base = ((size_t)b * kHq + h) * a.max_chunks;
    reinterpret_cast<float2 *>(a.part_o + (base + first + c) * kD)[dp] = make_float2(o0, o1);
    if (dp == 0)
        a.part_ml[base + first + c] = make_float2(M, lsum);
    if (Sel::kPublish)
        return;
    if (Sel::kLateWait) {
        grid_dependency_wait();  // the other kernel's partials
        allow_dependent_launch();
    }
    // publish: the CTA barrier orders every thread's partial stores before thread 0's
    // release-acquire ticket; the acquire side plus the barrier orders the merging
    // unit's loads after every other unit's partial stores
    __syncthreads();
    if (tid == 0)
        *ticket = ticket_acq_rel(&a.counters[b * kHkv + g]);
    __syncthreads();
    if (*ticket != nunits - 1)
        return;
    float ls, r0, r1, Mx = 0.f;
    const float2 *ml_row = a.part_ml + base, *o_col = reinterpret_cast<const float2 *>(a.part_o + base * kD) + dp;
    if constexpr (Sel::kLateWait)
        merge_eights(ml_row, o_col, nchunks, ls, r0, r1);
    else
        merge_partials(ml_row, o_col, nchunks, Mx, ls, r0, r1);
    out_row[dp] = finish_pair(r0, r1, ls);
    sel.finished(b, g, L, Mx, ls, state);
    if (WRITE_Q)
        q_row[dp] = q_word;
    if (tid == 0)
        a.counters[b * kHkv + g] = 0;
}

// ------------------------------------------------------------------ timeline (PKV_TIMELINE builds)

#ifdef PKV_TIMELINE
// Per-CTA timeline of the grid schedule, compiled only into libraries built with
// -DPKV_TIMELINE: globaltimer stamps (ns) at entry, after the unit is known, after
// the dependency wait, after the page loop and at the end, and (SM, sequence, chunk,
// pages) per CTA linear index; CTAs without a unit store SM -1.  Every launch
// overwrites the records of its linear indices.
constexpr int kTimelineMax = 16384;
__device__ unsigned long long g_timeline_stamps[kTimelineMax * 5];
__device__ int g_timeline_meta[kTimelineMax * 4];

__device__ __forceinline__ unsigned long long timeline_now()
{
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

struct Timeline {
    unsigned long long t[4];
    int lin;
    bool rec;
    __device__ __forceinline__ void begin()
    {
        t[0] = timeline_now();
        lin = blockIdx.x + gridDim.x * (blockIdx.y + gridDim.y * blockIdx.z);
        rec = threadIdx.x == 0 && lin < kTimelineMax;
    }
    __device__ __forceinline__ void stamp(int i) { t[i] = timeline_now(); }
    __device__ __forceinline__ void none() const
    {
        if (rec)
            g_timeline_meta[lin * 4] = -1;
    }
    __device__ __forceinline__ void end(int b, int c, int pages) const
    {
        if (!rec)
            return;
        unsigned sm;
        asm volatile("mov.u32 %0, %%smid;" : "=r"(sm));
        for (int i = 0; i < 4; ++i)
            g_timeline_stamps[lin * 5 + i] = t[i];
        g_timeline_stamps[lin * 5 + 4] = timeline_now();
        g_timeline_meta[lin * 4 + 0] = (int)sm;
        g_timeline_meta[lin * 4 + 1] = b;
        g_timeline_meta[lin * 4 + 2] = c;
        g_timeline_meta[lin * 4 + 3] = pages;
    }
};
#else
struct Timeline {  // compiled out
    __device__ __forceinline__ void begin() {}
    __device__ __forceinline__ void stamp(int) {}
    __device__ __forceinline__ void none() const {}
    __device__ __forceinline__ void end(int, int, int) const {}
};
#endif

// ------------------------------------------------------------------ grid schedule

constexpr int kGridExtraBytes = kGroup * kD * 2 + 2 * kD * 2 + 16;  // rotated q rows, new K/V rows, ticket

// All threads, between two units of a CTA: the first one's shared memory is read and its barriers
// (all of whose phases are complete) are free to be initialised again; what threads wrote there
// comes before the next copies.
__device__ __forceinline__ void rearm_barriers(uint64_t *my_bars, int stages, int lane)
{
    fence_proxy_async_smem();
    __syncthreads();
    if (lane == 0)
        for (int s = 0; s < stages; ++s)
            mbar_inval(&my_bars[s]);
    __syncwarp();
}

// One work unit (all threads): chunk c of the nchunks of (sequence b, KV head g).  Lane k of a warp
// holds in `my_page` the warp's k-th table entry if the list is the identity and `prefetched`.
template <class Warp, int STAGES, bool APPEND, class Sel, class List>
__device__ __forceinline__ void decode_unit(const CUtensorMap &tmap, const StepArgs &a, const Sel &sel, const List &list,
                                            SmemLayout<STAGES> &sm, int b, int g, int c, int nchunks, int L, int my_page,
                                            bool prefetched, Timeline &tl)
{
    uint16_t *q_rot = reinterpret_cast<uint16_t *>(sm.extra);  // [4][64] query rows (rotated when APPEND)
    uint16_t *new_kv = q_rot + kGroup * kD;                     // [2][64] rotated key row, value row
    int *ticket = reinterpret_cast<int *>(new_kv + 2 * kD);
    int tid = threadIdx.x;
    if (Sel::kLoops)  // keeps what depends on it from being held in registers across the loop's units
        asm volatile("" : "+r"(tid));
    const int warp = tid >> 5, lane = tid & 31;
    const int npages = (L + kPage - 1) / kPage, j0 = c * a.pages_per_chunk, nlist = list.count();
    const bool last_chunk = c == nchunks - 1;
    const int jn = min(nlist - j0, a.pages_per_chunk);
    const int nmine = warp < jn ? (jn - warp + kWarps - 1) / kWarps : 0;
    if (!prefetched && lane < nmine)
        my_page = a.bt[(size_t)b * a.max_blocks + list.logical(j0 + warp + lane * kWarps)];
    const bool bad = lane < nmine && (my_page < 0 || my_page >= a.num_pages);
    const bool any_bad = __syncthreads_or(bad);  // the new token's page is one of the last chunk's pages

    uint64_t *my_bars = sm.bars + warp * STAGES;
    uint8_t *my_stages = sm.stages + warp * STAGES * kStageBytes;
    const uint64_t policy = l2_evict_first_policy();
    const int nfirst = min(STAGES, nmine);
    const int nearly = any_bad ? 0 : copies_before_wait(list, L, j0, warp, nmine, STAGES);
    if (Sel::kLoops || !any_bad)
        init_warp_barriers<STAGES>(my_bars, lane);
    if (!any_bad) {
        issue_copies<STAGES>(&tmap, my_stages, my_bars, my_page, 0, nearly, g, lane, policy);
    }

    if (!Sel::kLateWait && !Sel::kPublish)
        grid_dependency_wait();  // q, k_new, v_new, recently written pages and every output follow it
    tl.stamp(2);
    if (!any_bad)  // the pages holding positions L - 2 and L - 1
        issue_copies<STAGES>(&tmap, my_stages, my_bars, my_page, nearly, nfirst, g, lane, policy);

    const int pos = L - 1, slot = pos % kPage;
    unit_rows<APPEND>(a, b, g, pos, last_chunk, q_rot, new_kv);
    __syncthreads();
    if (APPEND && last_chunk && !any_bad && tid < 16)
        store_new_token(a, a.bt[(size_t)b * a.max_blocks + npages - 1], g, slot, new_kv);
    if (any_bad) {
        if (tid == 0 && a.err)
            atomicOr(a.err, PKV_DEVERR_PAGE_RANGE);
        sel.skipped(b, g, j0, jn);
    }

    Warp w;
    w.init(q_rot, a.scale_log2, lane, sm.scratch + warp * kScratchFloats);
    if (!any_bad) {
        const auto patch = [&](uint8_t *stage, int j) {
            if (APPEND && last_chunk && j == npages - 1)
                patch_stage(stage, slot, new_kv, lane);
        };
        const uint32_t first_limit = b == a.expire_seq ? 0u : kWaitLimit;
        if (!consume_list<STAGES>(&tmap, my_stages, my_bars, w, my_page, nmine, j0, warp, lane, list, g, policy, patch,
                                  sel.emit(b, g), first_limit) &&
            lane == 0 && a.err)
            atomicOr(a.err, PKV_DEVERR_TIMEOUT);
    }
    tl.stamp(3);
    if (!Sel::kLateWait && !Sel::kPublish)
        allow_dependent_launch();
    // the stages are free now: they hold the combine area
    finish_unit<APPEND>(a, sel, w, reinterpret_cast<float *>(sm.stages), ticket, q_rot, b, g, c, nchunks,
                        list.first_slot(), L);
    tl.end(b, c, jn);
}

// CTAs per SM the register budget of a looping kernel is set for: as many as its ring's shared
// memory lets in (the others have none).
constexpr int loop_ctas_per_sm(bool loops, int stages) { return !loops ? 0 : stages == 2 ? 6 : stages == 3 ? 4 : 3; }

// The end of a publishing kernel's CTA: the first one waits for the kernel before.
template <class Sel>
__device__ __forceinline__ void publish_end()
{
    if constexpr (Sel::kPublish) {
        if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0)
            grid_dependency_wait();
        allow_dependent_launch();
    }
}

template <class Warp, int STAGES, bool APPEND, class Sel>
__device__ __forceinline__ void decode_cta(const CUtensorMap &tmap, const StepArgs &a, const Sel &sel, uint8_t *smem_raw)
{
    SmemLayout<STAGES> sm(smem_raw);
    Timeline tl;
    tl.begin();

    int g = blockIdx.x, b = blockIdx.y, c = blockIdx.z;
    if constexpr (Sel::kSortable) {
        if (a.sorted) {
            const int lin = blockIdx.x + kHkv * (blockIdx.y + gridDim.y * blockIdx.z);
            if (!sorted_unit(a, sel, gridDim.y, lin, reinterpret_cast<int *>(sm.scratch), b, g, c)) {
                tl.none();
                return;
            }
        }
    }
    tl.stamp(1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int j0 = c * a.pages_per_chunk;
    // the length and this chunk's table entries are fetched together (one round trip):
    // entries inside the table row are always readable, whatever the length turns out to be
    const int jcap = min(a.max_blocks - j0, a.pages_per_chunk);
    const int ncap = warp < jcap ? (jcap - warp + kWarps - 1) / kWarps : 0;
    int my_page = 0;
    if (Sel::kIdentity && lane < ncap)
        my_page = a.bt[(size_t)b * a.max_blocks + j0 + warp + lane * kWarps];
    const int L = a.seq_lens[b];
    const auto list = sel.list(b, L);
    if (!length_ok(a, L) || !list.ok()) {
        if (c == 0) {
            if (!Sel::kPublish)
                grid_dependency_wait();
            write_zero_unit(a, b, g);
        }
        tl.none();
        return;
    }
    const int nlist = list.count();
    const int nchunks = Sel::kIdentity ? (nlist + a.pages_per_chunk - 1) / a.pages_per_chunk
                                       : max(1, (nlist + a.pages_per_chunk - 1) / a.pages_per_chunk);
    if (c >= nchunks) {
        tl.none();
        return;
    }
    for (bool first = true;; first = false) {
        decode_unit<Warp, STAGES, APPEND>(tmap, a, sel, list, sm, b, g, c, nchunks, L, my_page, Sel::kIdentity && first, tl);
        if (!Sel::kLoops || (c += gridDim.z) >= nchunks)
            break;
        rearm_barriers(sm.bars + warp * STAGES, STAGES, lane);
    }
}

template <class Warp, int STAGES, bool APPEND, class Sel>
__global__ void __launch_bounds__(kThreads, loop_ctas_per_sm(Sel::kLoops, STAGES))
    decode_step_kernel(const __grid_constant__ CUtensorMap tmap, StepArgs a, Sel sel)
{
    extern __shared__ uint8_t smem_raw[];
    decode_cta<Warp, STAGES, APPEND>(tmap, a, sel, smem_raw);
    publish_end<Sel>();
}

// ------------------------------------------------------------------ FP8 pages, grid schedule

// The fused step over FP8 pages: the same unit, prologue, dependency wait, query
// rotation, ticket and merge as decode_step_kernel, with the FP8 unit copy and the
// Fp8MmaWarp page policy.  The new token's rotated key row and value row are
// quantized once per (sequence, KV head) by the unit of the last chunk -- warp 0 the
// key, warp 1 the value, with the FP8 append's arithmetic -- stored into their page
// slot, and patched into the staged copy of that page.
template <int STAGES>
struct Fp8StepSmem {
    static constexpr int kStagesBytes = kWarps * STAGES * kFp8Unit;
    static constexpr int kBarsBytes = kWarps * STAGES * 8;
    static constexpr int kSortInts = kMaxPagesPerChunk + 1 + kWarps + 5;
    static constexpr int kExtraBytes = kGroup * kD * 2 + 2 * kD * 2 + 2 * kD + 16 + 16 + kSortInts * 4;
    static constexpr int kBytes = 128 + kStagesBytes + kBarsBytes + kExtraBytes;  // incl. alignment slack
    static_assert(kStagesBytes >= kWarps * kStateFloats * 4, "the combine reuses the stages");
    uint8_t *stages;
    uint64_t *bars;
    uint16_t *q_rot;      // [4][64] rotated query rows (BF16)
    uint16_t *new_kv;     // [2][64] rotated key row, value row (BF16)
    uint8_t *new_codes;   // [2][64] their E4M3 codes
    float *new_scales;    // [2] their row scales
    int *ticket;
    int *sort_scratch;

    __device__ __forceinline__ explicit Fp8StepSmem(uint8_t *raw)
    {
        uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 127) & ~uintptr_t(127));
        stages = base;
        bars = reinterpret_cast<uint64_t *>(base + kStagesBytes);
        uint8_t *e = base + kStagesBytes + kBarsBytes;
        q_rot = reinterpret_cast<uint16_t *>(e);
        new_kv = q_rot + kGroup * kD;
        new_codes = reinterpret_cast<uint8_t *>(new_kv + 2 * kD);
        new_scales = reinterpret_cast<float *>(new_codes + 2 * kD);
        ticket = reinterpret_cast<int *>(new_scales + 4);
        sort_scratch = ticket + 4;
    }
};

// A warp writes the new token's rows into a unit (a stage or the page): lanes 0-3 the
// K codes (16 bytes each), every lane two V codes (dims 2 lane, 2 lane + 1) at their
// interleaved positions, lanes 0 and 1 the two scales.
__device__ __forceinline__ void put_new_token_fp8(uint8_t *unit, int slot, const uint8_t *codes, const float *scales,
                                                  int lane)
{
    if (lane < 4)
        *reinterpret_cast<uint4 *>(unit + slot * kD + 16 * lane) = reinterpret_cast<const uint4 *>(codes)[lane];
    uint8_t *vt = unit + fp8::kFp8Tile;
    vt[fp8::v_code_offset(slot, 2 * lane)] = codes[kD + 2 * lane];
    vt[fp8::v_code_offset(slot, 2 * lane + 1)] = codes[kD + 2 * lane + 1];
    if (lane < 2)
        reinterpret_cast<float *>(unit + kFp8UnitCodes)[lane * kPage + slot] = scales[lane];
}

// CTAs per SM the register budget is set for.  The 3-stage ring takes 27.5 KB of shared
// memory per CTA, so seven CTAs fit (at most 72 registers, a few spilled) and keep 7 x 4 x 3
// units of 2176 B in flight per SM; the other rings keep six (80 registers, none spilled).
// (The looping kernels hold more across their units and keep one CTA less.)
constexpr int fp8_ctas_per_sm(int stages) { return stages == 3 ? 7 : 6; }

// decode_unit over FP8 pages.
template <int STAGES, bool APPEND, class Sel, class List>
__device__ __forceinline__ void decode_unit_fp8(const CUtensorMap &tmap, const StepArgs &a, const Sel &sel,
                                                const List &list, Fp8StepSmem<STAGES> &sm, int b, int g, int c, int nchunks,
                                                int L, int my_page, bool prefetched)
{
    int tid = threadIdx.x;
    if (Sel::kLoops)  // keeps what depends on it from being held in registers across the loop's units
        asm volatile("" : "+r"(tid));
    const int warp = tid >> 5, lane = tid & 31;
    const int npages = (L + kPage - 1) / kPage, j0 = c * a.pages_per_chunk, nlist = list.count();
    const bool last_chunk = c == nchunks - 1;
    const int jn = min(nlist - j0, a.pages_per_chunk);
    const int nmine = warp < jn ? (jn - warp + kWarps - 1) / kWarps : 0;
    if (!prefetched && lane < nmine)
        my_page = a.bt[(size_t)b * a.max_blocks + list.logical(j0 + warp + lane * kWarps)];
    const bool bad = lane < nmine && (my_page < 0 || my_page >= a.num_pages);
    const bool any_bad = __syncthreads_or(bad);

    uint64_t *my_bars = sm.bars + warp * STAGES;
    uint8_t *my_stages = sm.stages + warp * STAGES * kFp8Unit;
    const uint64_t policy = l2_evict_first_policy();
    const int nfirst = min(STAGES, nmine);
    const int nearly = any_bad ? 0 : copies_before_wait(list, L, j0, warp, nmine, STAGES);
    const auto issue = [&](int k0, int k1) {
        for (int k = k0; k < k1; ++k) {
            const int pk = __shfl_sync(kFull, my_page, k);
            if (lane == 0)
                fp8::fp8_issue(&tmap, my_stages + k * kFp8Unit, &my_bars[k], g, pk, policy);
        }
    };
    if (Sel::kLoops || !any_bad)
        init_warp_barriers<STAGES>(my_bars, lane);
    if (!any_bad)
        issue(0, nearly);

    if (!Sel::kLateWait && !Sel::kPublish)
        grid_dependency_wait();  // q, k_new, v_new, recently written pages and every output follow it
    if (!any_bad)  // the pages holding positions L - 2 and L - 1
        issue(nearly, nfirst);

    const int pos = L - 1, slot = pos % kPage;
    unit_rows<APPEND>(a, b, g, pos, last_chunk, sm.q_rot, sm.new_kv);
    __syncthreads();
    if (APPEND && last_chunk) {
        if (warp == 0) {  // key row: lane holds dims lane, lane + 32 (rotated, BF16)
            uint32_t c1, c2;
            float sc;
            fp8::quantize_pair(bf16_value(sm.new_kv[lane]), bf16_value(sm.new_kv[lane + kD / 2]), c1, c2, sc);
            sm.new_codes[lane] = (uint8_t)c1;
            sm.new_codes[lane + kD / 2] = (uint8_t)c2;
            if (lane == 0)
                sm.new_scales[0] = sc;
        } else if (warp == 1) {  // value row: lane holds dims 2 lane, 2 lane + 1
            const uint32_t w2 = reinterpret_cast<const uint32_t *>(sm.new_kv + kD)[lane];
            uint32_t c0, c1;
            float sc;
            fp8::quantize_pair(bf16lo(w2), bf16hi(w2), c0, c1, sc);
            reinterpret_cast<uint16_t *>(sm.new_codes + kD)[lane] = (uint16_t)(c0 | (c1 << 8));
            if (lane == 0)
                sm.new_scales[1] = sc;
        }
        __syncthreads();
        if (!any_bad && warp == 0) {
            const int page = a.bt[(size_t)b * a.max_blocks + npages - 1];
            uint8_t *unit = reinterpret_cast<uint8_t *>(a.slab) + (size_t)page * kFp8PageBytes + (size_t)g * kFp8Unit;
            put_new_token_fp8(unit, slot, sm.new_codes, sm.new_scales, lane);
        }
    }
    if (any_bad) {
        if (tid == 0 && a.err)
            atomicOr(a.err, PKV_DEVERR_PAGE_RANGE);
        sel.skipped(b, g, j0, jn);
    }

    fp8::Fp8MmaWarpOf<Sel::kFine> w;
    w.init(sm.q_rot, a.scale_log2, lane);
    if (!any_bad) {
        const uint32_t first_limit = b == a.expire_seq ? 0u : kWaitLimit;
        const auto emit_of = sel.emit(b, g);
        int k = 0;
        for (; k < nmine; ++k) {
            const int s = k % STAGES;
            if (!mbar_wait_warp(&my_bars[s], (uint32_t)((k / STAGES) & 1), k == 0 ? first_limit : kWaitLimit))
                break;
            const int j = list.logical(j0 + warp + k * kWarps);
            uint8_t *stage = my_stages + s * kFp8Unit;
            if (APPEND && last_chunk && j == npages - 1) {  // the copy may predate the new token's store
                put_new_token_fp8(stage, slot, sm.new_codes, sm.new_scales, lane);
                __syncwarp();
            }
            visit_page(w, stage, list, j, emit_of(j));
            __syncwarp();
            if (k + STAGES < nmine) {
                const int pk = __shfl_sync(kFull, my_page, k + STAGES);
                if (lane == 0) {
                    fence_proxy_async_smem();
                    fp8::fp8_issue(&tmap, stage, &my_bars[s], g, pk, policy);
                }
            }
        }
        if (k < nmine) {  // a wait gave up: let the copies in flight land (bounded), flag it
            for (int kk = k; kk < min(nmine, k + STAGES); ++kk)
                (void)mbar_wait_warp(&my_bars[kk % STAGES], (uint32_t)((kk / STAGES) & 1));
            if (lane == 0 && a.err)
                atomicOr(a.err, PKV_DEVERR_TIMEOUT);
        }
    }
    if (!Sel::kLateWait && !Sel::kPublish)
        allow_dependent_launch();
    // the stages are free now: they hold the combine area
    finish_unit<APPEND>(a, sel, w, reinterpret_cast<float *>(sm.stages), sm.ticket, sm.q_rot, b, g, c, nchunks,
                        list.first_slot(), L);
}

template <int STAGES, bool APPEND, class Sel>
__device__ __forceinline__ void decode_cta_fp8(const CUtensorMap &tmap, const StepArgs &a, const Sel &sel, uint8_t *smem_raw)
{
    Fp8StepSmem<STAGES> sm(smem_raw);

    int g = blockIdx.x, b = blockIdx.y, c = blockIdx.z;
    if constexpr (Sel::kSortable) {
        if (a.sorted) {
            const int lin = blockIdx.x + kHkv * (blockIdx.y + gridDim.y * blockIdx.z);
            if (!sorted_unit(a, sel, gridDim.y, lin, sm.sort_scratch, b, g, c))
                return;
        }
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int j0 = c * a.pages_per_chunk;
    const int jcap = min(a.max_blocks - j0, a.pages_per_chunk);
    const int ncap = warp < jcap ? (jcap - warp + kWarps - 1) / kWarps : 0;
    int my_page = 0;
    if (Sel::kIdentity && lane < ncap)
        my_page = a.bt[(size_t)b * a.max_blocks + j0 + warp + lane * kWarps];
    const int L = a.seq_lens[b];
    const auto list = sel.list(b, L);
    if (!length_ok(a, L) || !list.ok()) {
        if (c == 0) {
            if (!Sel::kPublish)
                grid_dependency_wait();
            write_zero_unit(a, b, g);
        }
        return;
    }
    const int nlist = list.count();
    const int nchunks = Sel::kIdentity ? (nlist + a.pages_per_chunk - 1) / a.pages_per_chunk
                                       : max(1, (nlist + a.pages_per_chunk - 1) / a.pages_per_chunk);
    if (c >= nchunks)
        return;
    for (bool first = true;; first = false) {
        decode_unit_fp8<STAGES, APPEND>(tmap, a, sel, list, sm, b, g, c, nchunks, L, my_page, Sel::kIdentity && first);
        if (!Sel::kLoops || (c += gridDim.z) >= nchunks)
            break;
        rearm_barriers(sm.bars + warp * STAGES, STAGES, lane);
    }
}

template <int STAGES, bool APPEND, class Sel>
__global__ void __launch_bounds__(kThreads, fp8_ctas_per_sm(STAGES) - (Sel::kLoops ? 1 : 0))
    decode_step_fp8_kernel(const __grid_constant__ CUtensorMap tmap, StepArgs a, Sel sel)
{
    extern __shared__ uint8_t smem_raw[];
    decode_cta_fp8<STAGES, APPEND>(tmap, a, sel, smem_raw);
    publish_end<Sel>();
}

// ------------------------------------------------------------------ launch

// Ring depth per warp when the options leave it to the library: 3 stages for long
// chunks (4 CTAs per SM for BF16, 7 for FP8), else 2 (6 per SM), the measured best
// for 128-page chunks and for 16- to 32-page chunks of ragged batches respectively.
int default_ring(int pages_per_chunk) { return pages_per_chunk >= 64 ? 3 : 2; }

// Pages per unit where the caller leaves it to the library: as many units as the GPU holds at
// once (6 CTAs on each of 152 SMs), if every list is full, but whole lists before more units than
// that, and at least 8 pages, two a warp.  `spread`: how many times that many units where lists
// are bounded only by the table's width, most of them being much shorter.  Measured (us): a window
// of 2000 tokens, 16 sequences 20 pages 9.7, 32 pages 11.0; a window of 1000, 64 sequences 24
// pages 24.0, 48 pages 21.7, all 65 pages 20.3; a window of 300, 64 sequences 12 pages 11.3, all
// 20 pages 8.0; scored, 64 sequences up to 2048 tokens 36 pages 16.1, 48 pages 17.1, 64 pages 17.5.
inline int default_chunk(int B, int list_pages, int spread)
{
    const int64_t chunks = std::max<int64_t>(1, (int64_t)(152 * 6) * spread / ((int64_t)B * kHkv));
    const int64_t ppc = ((list_pages + chunks - 1) / chunks + kWarps - 1) / kWarps * kWarps;
    return (int)std::min<int64_t>(std::max<int64_t>(ppc, 2 * kWarps), kMaxPagesPerChunk);
}

template <class Warp, int STAGES, bool APPEND, class Sel>
int launch_grid(const CUtensorMap *tmap, const StepArgs &a, const Sel &sel, int B, cudaStream_t s, bool pdl)
{
    auto kernel = decode_step_kernel<Warp, STAGES, APPEND, Sel>;
    constexpr int smem = SmemLayout<STAGES>::kBaseBytes + kGridExtraBytes;
    static PerDeviceOnce attr;
    if (const int st = ensure_smem_attr(attr, kernel, smem); st != PKV_OK)
        return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kHkv, B, a.unit_chunks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attrs[1] = {pdl_attribute()};
    cfg.attrs = attrs;
    cfg.numAttrs = pdl ? 1 : 0;
    return status_from_cuda(cudaLaunchKernelEx(&cfg, kernel, *tmap, a, sel));
}

// FP8 pages: ring depth per warp 2..4 units (2176 B each).
template <int STAGES, bool APPEND, class Sel>
int launch_fp8_grid(const CUtensorMap *tmap, const StepArgs &a, const Sel &sel, int B, cudaStream_t s, bool pdl)
{
    auto kernel = decode_step_fp8_kernel<STAGES, APPEND, Sel>;
    constexpr int smem = Fp8StepSmem<STAGES>::kBytes;
    static PerDeviceOnce attr;
    if (const int st = ensure_smem_attr(attr, kernel, smem); st != PKV_OK)
        return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kHkv, B, a.unit_chunks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attrs[1] = {pdl_attribute()};
    cfg.attrs = attrs;
    cfg.numAttrs = pdl ? 1 : 0;
    return status_from_cuda(cudaLaunchKernelEx(&cfg, kernel, *tmap, a, sel));
}

template <bool APPEND, class Sel>
int launch_fp8_depth(const CUtensorMap *tmap, const StepArgs &a, const Sel &sel, int B, cudaStream_t s, bool pdl,
                     int depth)
{
    switch (depth) {
    case 2: return launch_fp8_grid<2, APPEND>(tmap, a, sel, B, s, pdl);
    case 3: return launch_fp8_grid<3, APPEND>(tmap, a, sel, B, s, pdl);
    default: return launch_fp8_grid<4, APPEND>(tmap, a, sel, B, s, pdl);
    }
}

// Ring depth per warp: 2 stages (36 KB per CTA, 6 CTAs per SM), 3 (4 per SM) or 4 (3 per SM).
template <class Warp, bool APPEND, class Sel>
int launch_grid_depth(const CUtensorMap *tmap, const StepArgs &a, const Sel &sel, int B, cudaStream_t s, bool pdl,
                      int depth)
{
    switch (depth) {
    case 2: return launch_grid<Warp, 2, APPEND>(tmap, a, sel, B, s, pdl);
    case 3: return launch_grid<Warp, 3, APPEND>(tmap, a, sel, B, s, pdl);
    default: return launch_grid<Warp, 4, APPEND>(tmap, a, sel, B, s, pdl);
    }
}

// Option bits every entry point of the grid kernels accepts.
constexpr int kGridOptions = 0xff | PKV_STEP_NO_PDL | PKV_STEP_GRID | PKV_STEP_RING_MASK | PKV_STEP_SORTED |
                             PKV_STEP_TEST_EXPIRE_WAIT;

constexpr int kLoopCtas = 152 * 16;

// The options of a call on `pool` whose lists have at most `list_pages` entries.
template <class Sel>
int check_options(const pkv_pool *pool, int B, int list_pages, int pages_per_chunk, int options)
{
    const int variant = options & 0xff;
    if (variant < PKV_DECODE_DEFAULT || variant > PKV_DECODE_MMA || (options & ~kGridOptions))
        return PKV_ERR_INVALID_ARG;
    if ((options & PKV_STEP_SORTED) && B > kMaxSortedBatch)
        return PKV_ERR_INVALID_ARG;  // the sorted order handles up to 1024 sequences
    const int ring = (options & PKV_STEP_RING_MASK) >> 12;
    if (ring != 0 && (ring < 2 || ring > 4))
        return PKV_ERR_INVALID_ARG;
    if (variant == PKV_DECODE_SIMT && (pool->kv_format == PKV_KV_FP8 || !std::is_same_v<Sel, AllPages>))
        return PKV_ERR_UNSUPPORTED;  // FP8 pages and selections of pages: the MMA policy only
    if ((options & PKV_STEP_SORTED) && !Sel::kSortable)
        return PKV_ERR_UNSUPPORTED;
    if ((list_pages + pages_per_chunk - 1) / pages_per_chunk > 65535)  // the chunk index is gridDim.z
        return PKV_ERR_INVALID_ARG;
    return PKV_OK;
}

// Validates the options, fills the launch-dependent fields of `a` and launches the
// kernel for the pool's format.  `max_blocks` is the table's width, `list_pages` the most
// entries a list of the selection has, `first_slots` the most partials that another
// kernel puts before a sequence's own.  follows: the kernel just before on the stream is
// the call's own and has waited for everything before it.
template <bool APPEND, class Sel>
int launch_fused(const pkv_pool *pool, StepArgs &a, const Sel &sel, int B, int max_blocks, int list_pages,
                 int first_slots, int pages_per_chunk, void *workspace, cudaStream_t s, int options, bool follows = false)
{
    if (const int st = check_options<Sel>(pool, B, list_pages, pages_per_chunk, options); st != PKV_OK)
        return st;
    const int variant = options & 0xff, ring = (options & PKV_STEP_RING_MASK) >> 12;
    const int unit_chunks = (list_pages + pages_per_chunk - 1) / pages_per_chunk;
    const int max_chunks = first_slots + unit_chunks;
    a.unit_chunks = unit_chunks;
    if (Sel::kLoops)  // as many CTAs as fill the GPU about twice
        a.unit_chunks = (int)std::min<int64_t>(unit_chunks, std::max<int64_t>(1, kLoopCtas / ((int64_t)B * kHkv)));
    const CUtensorMap *tmap = pool_tensor_map(pool);
    if (!tmap)
        return PKV_ERR_CUDA;
    const WorkspaceLayout ws = workspace_layout(B, max_chunks);
    char *wsp = static_cast<char *>(workspace);
    a.num_pages = pool->num_pages;
    a.slab = reinterpret_cast<uint16_t *>(pool->slab);
    a.max_blocks = max_blocks;
    a.pages_per_chunk = pages_per_chunk;
    a.counters = wsp ? reinterpret_cast<int *>(wsp) : nullptr;
    a.part_ml = wsp ? reinterpret_cast<float2 *>(wsp + ws.ml_offset()) : nullptr;
    a.part_o = wsp ? reinterpret_cast<float *>(wsp + ws.o_offset()) : nullptr;
    a.max_chunks = max_chunks;
    a.sorted = (options & PKV_STEP_SORTED) ? 1 : 0;
    a.expire_seq = (options & PKV_STEP_TEST_EXPIRE_WAIT) ? 0 : -1;
    const bool wanted = !(options & PKV_STEP_NO_PDL);
    const bool pdl = follows ? wanted : take_pdl_permission(pool, s, wanted);
    // (selections of pages: 2 stages were the fastest or within 1 % of it at every size)
    const int depth = ring ? ring : std::is_same_v<Sel, AllPages> ? default_ring(pages_per_chunk) : 2;
    if (pool->kv_format == PKV_KV_FP8)
        return launch_fp8_depth<APPEND>(tmap, a, sel, B, s, pdl, depth);
    if constexpr (std::is_same_v<Sel, AllPages>) {
        if (variant == PKV_DECODE_SIMT)
            return launch_grid_depth<SimtWarp, APPEND>(tmap, a, sel, B, s, pdl, depth);
    }
    return launch_grid_depth<MmaWarp, APPEND>(tmap, a, sel, B, s, pdl, depth);
}

}  // namespace
}  // namespace pkv
