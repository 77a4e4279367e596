// What the kernels of the 4-bit cache's attention share: their arguments, the
// sequences as they are after their checks, and how the work is cut up.
//
// Rows are the (new token, head of the group) pairs of one kv head, row r of a
// sequence being token r / group.  R rows make a unit, which needs every step
// of kStep keys that its last row sees.  All units, sequence by sequence, head
// by head, are laid out one after the other, each kIdle long for what it costs
// whatever its length (its rows' loads and stores) and one for each step, and
// cut into runs of equal length.  A cut at a unit's first step or before it is
// moved to the unit's start.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/mmq.h"
#include "kv4.cuh"

namespace mmq {
namespace kv4 {

struct Mark;
struct Kv4Args {
    mmq_kv4_attention_t p;
    float* parts;         // see Mark
    Mark* marks;          // one per run (of a CTA, or a stream of it)
    int* status;
    int inject;
    int page_shift, group;
    int each;             // without q_starts: new tokens of every sequence
    float scale_log2;
    uint32_t low, high;   // masks of codes: 0x000F000F, 0x00F000F0
    int few;              // sequences of up to so many rows are the few-row kernel's, others the tensor-core kernel's
};
// A unit that starts in a run and does not end there: runs up to `last` (-1: no
// such unit) have a part of it.  A run leaves two parts at most, of a unit that
// started before it (0) and of one that does not end in it (1): sums f32
// [run][part][row][dim], and after those (reference, sum of weights) [run][part][row].
struct Mark {
    int last, b, h, tile;
};

// The unit of the sequence's head.
struct Unit {
    int b, h, tile;
};

__device__ __forceinline__ bool finite16(uint32_t bits) { return (bits & 0x7C00u) != 0x7C00u; }   // low half
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// --------------------------------------------------------------- sequences
// The most keys of a sequence: places of keys are 32-bit numbers, the end of a last step and the pages that are looked
// up ahead of it, up to 720 keys past that end, among them.  (As numbers without a sign, so that 2^31 - 1 could be held,
// those comparisons cost the few-row kernel 2 %: 64 sequences of 32k tokens 227 us, and 222.)
constexpr int64_t kMostKeys = (int64_t(1) << 31) - 1024;
struct Sequence {
    int n, len;       // new tokens, tokens
    int64_t start;    // first row of q
};
// Checked: a sequence's rows lie in [0, tokens), its keys in its pages.
__device__ __forceinline__ Sequence sequence(const Kv4Args& a, int b, bool tell) {
    const mmq_kv4_attention_t& p = a.p;
    Sequence s;
    bool bad = false;
    if (p.q_starts) {
        const int64_t lo = p.q_starts[b], hi = p.q_starts[b + 1];
        bad = lo < 0 || hi < lo || hi > p.tokens;
        s.start = lo;
        s.n = bad ? 0 : int(hi - lo);
    } else {
        s.n = a.each;
        s.start = int64_t(b) * s.n;
    }
    const int64_t room = min(p.table_width << a.page_shift, kMostKeys), len = p.lens[b];
    bad = bad || len > room;
    s.len = int(max(int64_t(0), min(len, room)));
    if (tell && bad) atomicCAS(a.status, 0, MMQ_ERR_ARG);
    return s;
}
// Keys that new token j of a sequence sees.
__device__ __forceinline__ int seen(const Sequence& s, int j) { return max(0, s.len - s.n + 1 + j); }

// (A sequence's rows are fewer than 2^31, as the arguments' check has it.)
template <int R>
__device__ __forceinline__ int units(const Sequence& s, int group) {
    return int((uint32_t(s.n) * uint32_t(group) + (R - 1)) / R);
}
// Keys that the unit's last row sees, the most of all.
template <int R>
__device__ __forceinline__ int unit_keys(const Sequence& s, int group, int u) {
    return seen(s, min(s.n - 1, int((uint32_t(u) * R + (R - 1)) / uint32_t(group))));
}
// Steps of kStep keys of one unit, at least one: a unit without keys still has zeros to write.
template <int R, int kStep>
__device__ __forceinline__ int unit_steps(const Sequence& s, int group, int u) {
    return max(1, (unit_keys<R>(s, group, u) + kStep - 1) / kStep);
}
// A unit's length in the layout, and that of one head's units.
template <int R, int kStep, int kIdle>
__device__ __forceinline__ int unit_length(const Sequence& s, int group, int u) {
    return kIdle + unit_steps<R, kStep>(s, group, u);
}
template <int R, int kStep, int kIdle>
__device__ __forceinline__ int64_t head_length(const Sequence& s, int group) {
    int64_t n = 0;
    const int m = units<R>(s, group);
    for (int u = 0; u < m; ++u) n += unit_length<R, kStep, kIdle>(s, group, u);
    return n;
}
// A cut `at` past the start of a sequence whose heads are `each` long: its head and unit, how far it lies in that one,
// and by how much it was moved.
struct Cut {
    int h, u, in, moved;
};
template <int R, int kStep, int kIdle>
__device__ __forceinline__ Cut cut(const Sequence& s, int group, int64_t each, int64_t at) {
    Cut c;
    c.h = int(at / each);
    int64_t in_head = at - c.h * each;
    c.u = 0;
    for (int length; in_head >= (length = unit_length<R, kStep, kIdle>(s, group, c.u)); ++c.u) in_head -= length;
    c.moved = in_head <= kIdle ? int(in_head) : 0;
    c.in = int(in_head) - c.moved;
    return c;
}
// Runs that share a layout of length `total`: the first `longer` of them have one more than the others.
struct Runs {
    int64_t total, each, longer;
    __device__ __forceinline__ Runs(int64_t total, int64_t runs) : total(total), each(total / runs), longer(total - each * runs) {}
    __device__ __forceinline__ int64_t start(int64_t run) const { return min(total, run * each + min(run, longer)); }
    // The run that place `at` lies in.
    __device__ __forceinline__ int64_t of(int64_t at) const {
        const int64_t first = longer * (each + 1);
        return at < first ? at / (each + 1) : longer + (at - first) / each;
    }
};
// An inclusive sum over the threads of a CTA of kWarps warps, and the whole sum; sums: kWarps words of shared memory.
template <int kWarps>
__device__ __forceinline__ int64_t cta_scan(int64_t mine, int64_t* sums, int64_t& total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += v;
    }
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) upto += sums[w];
        total += sums[w];
    }
    return upto;
}

}  // namespace kv4

// The tensor-core kernel (kv4_attention_tc.cu) and its join; two: 256 rows to a unit, not 128.
// Joins what `runs` runs of units of R rows have left (kv4_attention.cu).
cudaError_t launch_kv4_join(const kv4::Kv4Args& a, int R, int runs, cudaStream_t s);
size_t kv4_attention_tc_part_bytes(int head_dim, int nsm);
cudaError_t launch_kv4_attention_tc(const kv4::Kv4Args& a, bool two, int nsm, const cudaLaunchConfig_t& cfg);

}  // namespace mmq
