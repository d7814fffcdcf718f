// pkv_chunk_single.cu -- the attention of chunks for sequences that bring a single token.
//
// The 4 query heads of a KV head are all that meets a sequence's pages, so its bytes are what there is to do, and a
// tensor-core tile of 128 rows would be all but empty.  Four CTAs an SM, each with a run of its own, of four warps
// that take every fourth page of a piece by warp-level products (the decode kernels' policies) and copy their pages
// themselves, so that the next item's are on their way while this one's result is made.  What is cut is joined by the
// part that ends last.
//
// Page products, whose dependent instructions 16 warps an SM hide in part, bound it: 200 sequences of up to 4096 FP8
// tokens take 92.5 us where 63 would do at the rate of a copy (128 by a team of 8 warps beside the tile kernel's, 173
// by one of 24 warps); BF16 125 us of 119.  A call of one short sequence (500 tokens: 10 us) is bound by its
// steps one after the other: the plan, the first piece, the pages, the join of what is cut.
#include <type_traits>

#include "pkv_chunk_run.cuh"
#include "pkv_fp8.cuh"

namespace pkv {
namespace chunk {
namespace {

constexpr int kTeam = kWarps;
constexpr int kTilePages = kPagesOfTile;

template <bool FP8>
struct SingleRun {
    static constexpr int kThreads = (kTeam + 1) * 32, kConsumers = kTeam;
    static constexpr bool kSingles = true;
    static constexpr int kLeast = 20;  // of a CTA's run: shorter ones cost more to join (one sequence of 500 tokens: 11 us, at 36 15)
    // tiles of 8 pages and one KV head, in sixths of the time of one of BF16 pages
    static __device__ __forceinline__ Costs costs() { return {{0, 0, 0, FP8 ? 4 : 6}, {0, 0, 0, 8}}; }
};

struct SingleShared : RunShared {
    uint64_t here[kTeam][8];  // a warp's place holds a page
    uint64_t group;           // times the warps have met
    int last, bad;            // this CTA finished the item last; the last item with a bad page id
    int arrived;              // the other sequences' kernel has handed its wait on
    alignas(16) float states[kTeam][kStateFloats];
    int64_t sums[(kTeam + 1) * 32];
};

template <bool FP8>
struct Team {
    static constexpr int kUnit = FP8 ? kFp8Unit : kStageBytes;
    // A warp's places: what four CTAs an SM have room for.  (BF16 pages: 2 take 126 us where 3 take 132; FP8: with a
    // fifth CTA and 4 places, at fewer registers than the products need, 99 us where 94.)
    static constexpr int kSlots = FP8 ? 5 : 2;
    const CUtensorMap *tmap;
    const ChunkArgs &a;
    SingleShared &sh;
    uint8_t *places;
    int warp, lane;
    int met = 0;
    int copied = 0, seen = 0;       // the warp's pages: on their way or done with, done with
    int begun = -1, first_ids = 0;  // the item whose first pages are on their way, and the ids of its first 32

    __device__ __forceinline__ Team(const CUtensorMap *tmap_, const ChunkArgs &a_, SingleShared &sh_, uint8_t *all)
        : tmap(tmap_), a(a_), sh(sh_), warp(threadIdx.x >> 5), lane(threadIdx.x & 31)
    {
        places = all + warp * kSlots * kUnit;
    }

    // The warps wait for each other; false if that gave up.
    __device__ __forceinline__ bool meet()
    {
        __syncwarp();
        if (lane == 0)
            tc::mbar_arrive(&sh.group);
        return wait_for(&sh.group, met++ & 1, &sh.stop);
    }

    // The warp's pages of a piece: its first page and every fourth from there.
    __device__ __forceinline__ int first_page(const Item &x) const { return x.j0 * kTilePages + warp; }
    __device__ __forceinline__ int own_pages(const Item &x) const
    {
        const int n = min(x.j1 * kTilePages, x.count) - first_page(x);
        return n > 0 ? (n + kTeam - 1) / kTeam : 0;
    }
    __device__ __forceinline__ int own_ids(const Item &x, int from) const  // lane l: the id of the from + l-th
    {
        const int64_t i = first_page(x) + (int64_t)(from + lane) * kTeam;
        return (a.bt + (size_t)x.b * a.max_blocks)[x.page((int)min(i, (int64_t)x.count - 1))];
    }
    __device__ __forceinline__ bool outside(int id) const { return id < 0 || id >= a.num_pages; }
    // The next page on its way (a bad id is replaced by page 0; the item is marked).
    __device__ __forceinline__ void copy_page(int id, int g, uint64_t policy)
    {
        const int n = copied++;
        if (lane == 0) {
            uint64_t *bar = &sh.here[warp][n % kSlots];
            uint8_t *dst = places + n % kSlots * kUnit;
            const int page = outside(id) ? 0 : id;
            fence_proxy_async_smem();
            mbar_arrive_expect_tx(bar, kUnit);
            if (FP8)
                fp8::tma_load_unit(dst, tmap, bar, g, page, policy);
            else
                tma_load_page_head(dst, tmap, bar, g, page, policy);
        }
        __syncwarp();
    }
    __device__ __forceinline__ void begin_pages(const Item &x, int ids, uint64_t policy)
    {
        const int n = min(own_pages(x), kSlots);
        for (int i = 0; i < n; ++i)
            copy_page(__shfl_sync(kFull, ids, i), x.g, policy);
    }

    // Ticket of a cut item, whose partials all threads have written; false if a wait gave up.
    __device__ __forceinline__ bool draw_ticket(const Item &x, bool &last)
    {
        if (!meet())  // (no fences besides: see the tile kernel's)
            return false;
        if (threadIdx.x == 0) {
            int *ticket = &a.tickets[x.first * 2];
            int drawn;
            asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(drawn) : "l"(ticket) : "memory");
            sh.taken[x.me == 0][0] = 1;
            sh.last = drawn == x.parts - 1;
            if (drawn == x.parts - 1)
                *ticket = 0;
        }
        if (!meet())
            return false;
        last = *(volatile int *)&sh.last != 0;
        return true;
    }

    // Partial of part i of an item: its 4 rows.
    static __device__ __forceinline__ size_t part_rows(const Item &x, int i)
    {
        return (size_t)((x.first + i) * 2 + (i == 0 ? 1 : 0)) * kGroup;
    }

    __device__ __forceinline__ bool piece(Feed &feed, const Item &item, uint64_t policy)
    {
        const Item &x = item;
        const int pages = own_pages(x);
        int ids = begun == feed.n ? first_ids : own_ids(x, 0);
        if (begun != feed.n)
            begin_pages(x, ids, policy);
        std::conditional_t<FP8, fp8::Fp8MmaWarp, MmaWarp> w;
        if constexpr (FP8)
            w.init(a.q + x.row, a.scale_log2, lane);
        else
            w.init(a.q + x.row, a.scale_log2, lane, nullptr);
        bool bad = __any_sync(kFull, lane < min(pages, 32) && outside(ids));
        int sent = min(pages, kSlots);  // of them, on their way or done with
        const int p = x.p0, lo = a.window ? max(p + 1 - a.window, 0) : 0;
        for (int k = 0; k < pages; ++k, ++seen) {
            if (a.expire && feed.n == 0)
                *(volatile int *)&sh.stop = 1;  // (and the wait is skipped)
            else if (!wait_for(&sh.here[warp][seen % kSlots], (seen / kSlots) & 1, &sh.stop))
                return false;
            if (a.expire && feed.n == 0)
                return false;
            const uint8_t *page = places + seen % kSlots * kUnit;
            const int i = first_page(x) + k * kTeam;
            if (!x.masked(i / kTilePages)) {
                w.page(page, EveryToken{});
            } else {
                const int first = x.page(i) * kPage;
                const uint32_t upto = p + 1 - first >= kPage ? 0xffffu : (1u << (p + 1 - first)) - 1;
                const uint32_t below = (1u << min(max(lo - first, 0), kPage)) - 1;
                const uint32_t sunk = (1u << min(max(a.sinks - first, 0), kPage)) - 1;
                if (const uint32_t bits = upto & (~below | sunk))
                    w.page(page, TokenSet{bits});
            }
            __syncwarp();
            if (sent < pages) {
                if (sent % 32 == 0) {
                    ids = own_ids(x, sent);
                    bad |= __any_sync(kFull, lane < min(pages - sent, 32) && outside(ids));
                }
                copy_page(__shfl_sync(kFull, ids, sent % 32), x.g, policy);
                ++sent;
            }
        }
        // the next item's pages are on their way while this one's result is made
        if (const Item *y = feed.look(1)) {
            first_ids = own_ids(*y, 0);
            begin_pages(*y, first_ids, policy);
            begun = feed.n + 1;
        }
        if (bad)
            sh.bad = feed.n;
        w.store_state(sh.states[warp]);
        if (!meet())
            return false;
        // (a thread: head `warp`, dims 2 lane and 2 lane + 1)
        float M, l, o0, o1;
        combine_warps(&sh.states[0][0], warp, lane, M, l, o0, o1);
        bad = *(volatile int *)&sh.bad == feed.n;
        if (!meet())  // the states may be written again
            return false;
        if (bad && threadIdx.x == 0 && a.err)
            atomicOr(a.err, PKV_DEVERR_PAGE_RANGE);
        const Item z = x;  // (held in registers from here on only)
        bool write = z.parts == 1;
        if (!write) {
            const size_t at = part_rows(z, z.me) + warp;
            __stcg(reinterpret_cast<float2 *>(a.part_o + at * kD) + lane, make_float2(o0, o1));
            if (lane == 0)
                __stcg(a.part_ml + at, bad ? bad_part() : make_float2(M, l));
            if (!draw_ticket(z, write))
                return false;
            if (write) {
                M = -INFINITY;
                bad = false;
                for (int i = lane; i < z.parts; i += 32) {
                    const float2 ml = __ldcg(a.part_ml + part_rows(z, i) + warp);
                    M = fmaxf(M, ml.x);
                    bad |= is_bad_part(ml.y);
                }
#pragma unroll
                for (int off = 16; off; off >>= 1)
                    M = fmaxf(M, __shfl_xor_sync(kFull, M, off));
                bad = __any_sync(kFull, bad);
                l = o0 = o1 = 0.f;
#pragma unroll 8
                for (int i = 0; i < z.parts; ++i) {
                    const size_t from = part_rows(z, i) + warp;
                    const float2 ml = __ldcg(a.part_ml + from);
                    const float2 v = __ldcg(reinterpret_cast<const float2 *>(a.part_o + from * kD) + lane);
                    const float f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - M);
                    l = fmaf(f, ml.y, l);
                    o0 = fmaf(f, v.x, o0);
                    o1 = fmaf(f, v.y, o1);
                }
            }
        }
        if (write) {
            const float f = inverse_sum(l);
            reinterpret_cast<uint32_t *>(a.out + x.row + warp * kD)[lane] = bad ? 0u : pack_bf16x2(o0 * f, o1 * f);
        }
        return true;
    }

    __device__ __forceinline__ void run()
    {
        const uint64_t policy = l2_evict_first_policy();
        Feed feed(sh);
        for (const Item *x; (x = feed.look()) != nullptr; feed.let_go())
            if (!piece(feed, *x, policy))
                break;
        for (; seen < copied; ++seen)  // (a wait gave up: let the copies in flight land, bounded)
            (void)mbar_wait_warp(&sh.here[warp][seen % kSlots], (seen / kSlots) & 1);
    }
};

template <bool FP8>
__global__ void __launch_bounds__(SingleRun<FP8>::kThreads, kSingleCtas / kSms)
single_kernel(const __grid_constant__ CUtensorMap tmap, const __grid_constant__ ChunkArgs a, bool follows)
{
    using Run = SingleRun<FP8>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *places = smem_raw + (-smem_addr(smem_raw) & 1023u);
    SingleShared &sh = *reinterpret_cast<SingleShared *>(places + kTeam * Team<FP8>::kSlots * Team<FP8>::kUnit);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int w = 0; w < kTeam; ++w)
            for (int i = 0; i < Team<FP8>::kSlots; ++i)
                mbar_init(&sh.here[w][i], 1);
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&sh.item_full[i], 1);
            mbar_init(&sh.item_empty[i], Run::kConsumers);
        }
        mbar_init(&sh.group, kTeam);
        sh.stop = 0;
        sh.bad = -1;
        sh.taken[0][0] = sh.taken[1][0] = 0;
        fence_barrier_init();
        if (follows)
            asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(sh.arrived) : "l"(a.arrived) : "memory");
    }
    if (!follows) {
        grid_dependency_wait();
        allow_dependent_launch();
    }
    __syncthreads();
    if (follows) {  // (see launch_singles)
        if (!sh.arrived)
            grid_dependency_wait();
        asm volatile("fence.proxy.async.global;" ::: "memory");  // (pages are read by copies)
    }
    make_plan<Run>(a, sh);
    __syncthreads();
    if (warp == kTeam)
        pieces<Run>(a, sh, false);
    else
        Team<FP8>(&tmap, a, sh, places).run();
    __syncthreads();
    if (sh.stop && warp == kTeam) {
        pieces<Run>(a, sh, true);
        if ((threadIdx.x & 31) == 0 && a.err)
            atomicOr(a.err, PKV_DEVERR_TIMEOUT);
    }
    if (follows && blockIdx.x == 0) {
        grid_dependency_wait();
        if (threadIdx.x == 0)
            *a.arrived = 0;
    }
}

template <bool FP8>
int launch(const pkv_pool *pool, const ChunkArgs &a, cudaStream_t s, bool pdl, bool follows)
{
    const CUtensorMap *tmap = pool_tensor_map(pool);
    if (!tmap)
        return PKV_ERR_CUDA;
    constexpr int smem = 1024 + kTeam * Team<FP8>::kSlots * Team<FP8>::kUnit + (int)sizeof(SingleShared);
    static_assert((smem + 1024) * (kSingleCtas / kSms) <= 228 * 1024, "shared memory of an SM");
    static PerDeviceOnce attr;
    if (const int st = ensure_smem_attr(attr, single_kernel<FP8>, smem); st != PKV_OK)
        return st;
    return launch_kernel(single_kernel<FP8>, dim3(kSingleCtas), dim3(SingleRun<FP8>::kThreads), smem, s, pdl, *tmap, a, follows);
}

}  // namespace

int launch_singles(const pkv_pool *pool, ChunkArgs a, void *workspace, cudaStream_t s, bool pdl, bool follows)
{
    const SingleWorkspace ws = single_workspace();
    a.tickets = static_cast<int *>(workspace);
    a.part_ml = reinterpret_cast<float2 *>(static_cast<char *>(workspace) + ws.tickets);
    a.part_o = reinterpret_cast<float *>(static_cast<char *>(workspace) + ws.tickets + ws.ml);
    a.refuses = !follows;
    return pool->kv_format == PKV_KV_FP8 ? launch<true>(pool, a, s, pdl, follows) : launch<false>(pool, a, s, pdl, follows);
}

}  // namespace chunk
}  // namespace pkv
