// Pages of a key/value cache, whatever they hold: copies in the caches of all
// layers, and the compaction of a pool.
//
// Compaction.  Live pages are those that a sequence's table names within its
// length; n of them.  Those below n stay, and the k-th live page at or past n
// moves to the k-th free page below n: the fewest moves, none of which reads
// what another writes, so all run at once.  With S(p) the live pages below p,
//   hole p:  k = p - S(p)          mover p:  k = S(p) - S(n)
// A plan kernel of one CTA marks the live pages in a bitmap in shared memory,
// sums it up word by word and lists movers and holes; the move kernel rewrites
// the tables and copies the pages.
//
// Bound: memory where much is copied (64 pages in 64 caches 43 us, 6.2 TB/s, 92 %
// of a copy's rate), the launches where little is.
#include "mmq_internal.h"
#include "sm103_ptx.cuh"

namespace {

using namespace mmq::ptx;
using mmq::up256;

constexpr int kThreads = 256;
constexpr int kFlight = 8;                             // 16-byte loads in flight per thread
constexpr int64_t kChunk = kThreads * kFlight * 16;    // bytes that a CTA copies at a time

struct Caches {
    uint8_t* at[MMQ_PAGES_MAX_CACHES];
};

// A chunk of a page: bytes [first, first + kChunk) of it, as far as it goes.
__device__ __forceinline__ void copy_chunk(uint8_t* cache, int64_t src, int64_t dst, int64_t page_bytes, int64_t first) {
    const uint4* from = reinterpret_cast<const uint4*>(cache + src * page_bytes + first);
    uint4* to = reinterpret_cast<uint4*>(cache + dst * page_bytes + first);
    const int n = int(min(kChunk, page_bytes - first) / 16);
    uint4 v[kFlight];
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
        const int k = i * kThreads + threadIdx.x;
        if (k < n) v[i] = __ldcs(from + k);
    }
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
        const int k = i * kThreads + threadIdx.x;
        if (k < n) __stcs(to + k, v[i]);
    }
}

// -------------------------------------------------------------------- copy
struct CopyArgs {
    const int32_t *src, *dst;
    int64_t pairs, page_bytes, n_pages, chunks;   // chunks of a page
    int* status;
};

__global__ void __launch_bounds__(kThreads) pages_copy_kernel(const __grid_constant__ Caches caches, const CopyArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    uint8_t* const cache = caches.at[blockIdx.y];
    for (int64_t i = blockIdx.x; i < a.pairs * a.chunks; i += gridDim.x) {
        const int64_t pair = i / a.chunks;
        const int64_t src = a.src[pair], dst = a.dst[pair];
        if (src >= a.n_pages || dst >= a.n_pages) {
            if (threadIdx.x == 0) atomicCAS(a.status, 0, MMQ_ERR_ARG);
            continue;
        }
        if (src < 0 || dst < 0 || src == dst) continue;
        copy_chunk(cache, src, dst, a.page_bytes, (i - pair * a.chunks) * kChunk);
    }
}

// ----------------------------------------------------------------- compact
constexpr int kPlanThreads = 1024;

struct Plan {        // in the workspace
    int32_t live, moves, below;   // n, movers, S(n)
};
struct CompactArgs {
    const int32_t *table, *lens;
    int32_t *table_out, *map, *live;
    uint32_t* bits;       // live pages
    int32_t* before;      // live pages below each word of bits
    int32_t *src, *dst;   // the moves
    Plan* plan;
    int64_t n_pages, width, page_bytes, chunks;
    int batch, page_shift, n_caches;
    int* status;
};

// Pages that sequence b holds.
__device__ __forceinline__ int held(const CompactArgs& a, int b, bool tell) {
    const int64_t room = a.width << a.page_shift, len = a.lens[b];
    if (tell && len > room) atomicCAS(a.status, 0, MMQ_ERR_ARG);
    return int((max(int64_t(0), min(len, room)) + (int64_t(1) << a.page_shift) - 1) >> a.page_shift);
}

__global__ void __launch_bounds__(kPlanThreads) pages_plan_kernel(const CompactArgs a) {
    extern __shared__ uint32_t bits[];
    __shared__ int sums[32];
    __shared__ int below;
    griddep_launch_dependents();
    griddep_wait();
    const int words = int((a.n_pages + 31) / 32);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < words; i += kPlanThreads) bits[i] = 0;
    if (threadIdx.x == 0) below = 0;
    __syncthreads();
    // a warp per sequence
    bool bad = false;
    for (int b = warp; b < a.batch; b += kPlanThreads / 32) {
        const int n = held(a, b, lane == 0);
        for (int i = lane; i < n; i += 32) {
            const int32_t id = a.table[int64_t(b) * a.width + i];
            if (id < 0 || id >= a.n_pages) bad = true;
            else atomicOr(&bits[id >> 5], 1u << (id & 31));
        }
    }
    if (bad) atomicCAS(a.status, 0, MMQ_ERR_ARG);
    __syncthreads();
    // sums over the words, each thread a run of them
    const int per = (words + kPlanThreads - 1) / kPlanThreads;
    const int w0 = min(words, int(threadIdx.x) * per), w1 = min(words, w0 + per);
    int mine = 0;
    for (int w = w0; w < w1; ++w) mine += __popc(bits[w]);
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += v;
    }
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    int first = 0, live = 0;
#pragma unroll 8
    for (int w = 0; w < 32; ++w) {
        if (w < warp) first += sums[w];
        live += sums[w];
    }
    first += upto - mine;
    int at = first;
    for (int w = w0; w < w1; ++w) {
        a.bits[w] = bits[w];
        a.before[w] = at;
        if (w == live >> 5) below = at + __popc(bits[w] & ((1u << (live & 31)) - 1u));   // S(n); n = 32 words: see below
        at += __popc(bits[w]);
    }
    __syncthreads();
    const int s_n = (live >> 5) < words ? below : live;   // every page is live
    // the moves
    at = first;
    for (int w = w0; w < w1; ++w) {
        const uint32_t all = bits[w];
        const int page = 32 * w;
        // holes below n, movers from n on
        const uint32_t low = page + 32 <= live ? ~0u : page >= live ? 0u : (1u << (live - page)) - 1u;
        for (uint32_t h = ~all & low; h; h &= h - 1) {
            const int i = __ffs(int(h)) - 1;
            a.dst[page + i - (at + __popc(all & ((1u << i) - 1u)))] = page + i;
        }
        for (uint32_t m = all & ~low; m; m &= m - 1) {
            const int i = __ffs(int(m)) - 1;
            a.src[at + __popc(all & ((1u << i) - 1u)) - s_n] = page + i;
        }
        at += __popc(all);
    }
    if (threadIdx.x == 0) {
        *a.plan = Plan{live, live - s_n, s_n};
        *a.live = live;
    }
}

// Where page p goes, -1 for a page that is free.
__device__ __forceinline__ int32_t target(const CompactArgs& a, const Plan& plan, int32_t p) {
    const uint32_t word = a.bits[p >> 5];
    if (!((word >> (p & 31)) & 1u)) return -1;
    if (p < plan.live) return p;
    return a.dst[a.before[p >> 5] + __popc(word & ((1u << (p & 31)) - 1u)) - plan.below];
}

__global__ void __launch_bounds__(kThreads) pages_move_kernel(const __grid_constant__ Caches caches, const CompactArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    const Plan plan = *a.plan;
    const int64_t threads = int64_t(gridDim.x) * kThreads, me = int64_t(blockIdx.x) * kThreads + threadIdx.x;
    for (int64_t p = me; p < a.n_pages; p += threads) a.map[p] = target(a, plan, int32_t(p));
    for (int64_t i = me; i < a.batch * a.width; i += threads) {
        const int b = int(i / a.width);
        const int32_t id = a.table[i];
        const bool used = i - b * a.width < held(a, b, false) && id >= 0 && id < a.n_pages;
        a.table_out[i] = used ? target(a, plan, id) : -1;
    }
    const int64_t per_cache = int64_t(plan.moves) * a.chunks;
    for (int64_t i = blockIdx.x; i < per_cache * a.n_caches; i += gridDim.x) {
        const int64_t c = i / per_cache, rest = i - c * per_cache, k = rest / a.chunks;
        copy_chunk(caches.at[c], a.src[k], a.dst[k], a.page_bytes, (rest - k * a.chunks) * kChunk);
    }
}

struct Layout {
    size_t bits, before, src, dst, plan, bytes;
};
Layout layout(int64_t n_pages) {
    const size_t words = size_t((n_pages + 31) / 32), moves = size_t(n_pages / 2 + 1);
    Layout l;
    l.bits = 0;
    l.before = l.bits + up256(words * 4);
    l.src = l.before + up256(words * 4);
    l.dst = l.src + up256(moves * 4);
    l.plan = l.dst + up256(moves * 4);
    l.bytes = l.plan + up256(sizeof(Plan));
    return l;
}

}  // namespace

namespace mmq {

cudaError_t launch_pages_copy(const mmq_pages_copy_t& p, int* status, cudaStream_t s) {
    Caches caches = {};
    for (int i = 0; i < p.n_caches; ++i) caches.at[i] = static_cast<uint8_t*>(p.caches[i]);
    const CopyArgs a{p.src, p.dst, p.pairs, p.page_bytes, p.n_pages, (p.page_bytes + kChunk - 1) / kChunk, status};
    const int64_t blocks = a.pairs * a.chunks, most = 1 << 20;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = mmq::launch_config(dim3(unsigned(blocks < most ? blocks : most), unsigned(p.n_caches)),
                                                      dim3(kThreads), 0, s, attr);
    return cudaLaunchKernelEx(&cfg, pages_copy_kernel, caches, a);
}

size_t pages_compact_workspace(const mmq_pages_compact_t& p) { return layout(p.n_pages).bytes; }

cudaError_t launch_pages_compact(const mmq_pages_compact_t& p, void* workspace, int* status, cudaStream_t s) {
    const int nsm = sm_count();
    if (!nsm) return cudaErrorInvalidDevice;
    Caches caches = {};
    for (int i = 0; i < p.n_caches; ++i) caches.at[i] = static_cast<uint8_t*>(p.caches[i]);
    const Layout l = layout(p.n_pages);
    char* const ws = static_cast<char*>(workspace);
    CompactArgs a;
    a.table = p.page_table;
    a.lens = p.lens;
    a.table_out = p.table_out;
    a.map = p.page_map;
    a.live = p.live;
    a.bits = reinterpret_cast<uint32_t*>(ws + l.bits);
    a.before = reinterpret_cast<int32_t*>(ws + l.before);
    a.src = reinterpret_cast<int32_t*>(ws + l.src);
    a.dst = reinterpret_cast<int32_t*>(ws + l.dst);
    a.plan = reinterpret_cast<Plan*>(ws + l.plan);
    a.n_pages = p.n_pages;
    a.width = p.table_width;
    a.page_bytes = p.page_bytes;
    a.chunks = (p.page_bytes + kChunk - 1) / kChunk;
    a.batch = p.batch;
    a.n_caches = p.n_caches;
    a.status = status;
    a.page_shift = 0;
    while ((1 << a.page_shift) < p.page_size) ++a.page_shift;
    const size_t smem = size_t((p.n_pages + 31) / 32) * 4;
    cudaError_t e;
    if ((e = cudaFuncSetAttribute(pages_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, MMQ_PAGES_MAX / 8))) return e;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = mmq::launch_config(dim3(1), dim3(kPlanThreads), smem, s, attr);
    if ((e = cudaLaunchKernelEx(&cfg, pages_plan_kernel, a))) return e;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(unsigned(nsm * 8));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, pages_move_kernel, caches, a);
}

}  // namespace mmq
