// A mixture-of-experts FFN on q4_K experts for a few tokens.
//
//   p = softmax(x Wr^T);  the top_k largest of each token (ties: the lower
//   expert);  w = p of those, or p over their sum
//   h = silu(x Wg_e^T) * (x Wu_e^T),  y = h Wd_e^T per chosen expert e
//   out = sum w y (+ residual)
//
// Bound by the experts' weight bytes, each read once.  A q4_K weight is
// d (sc q) - dmin m: sc q (at most 945) and m (at most 63) are exact in fp16,
// so they are the matrix instructions' operands as they are, and an
// activation, f32, goes in as the sum of two fp16 values: per token and 256
// values a power of two 2^e takes the largest to [128, 256), hi = fp16(x 2^-e),
// lo = fp16(x 2^-e - hi), which leaves at most 2^-22 of x or 2^-32 of the
// largest.  hi and lo are two columns of one product, added in f32:
//   sum_k w x = 2^e (d (S_hi + S_lo) - dmin (M_hi + M_lo)),
//   S = sum (sc q) x,  M = sum over the eight 32-value sub-blocks of m X, X the
// sub-block's sum of activations (split in the same way).  So the experts see
// f32 activations (no q8_1 rounding of x or h) at fp16 matrix rates.
//
// Measured: 16 tokens, 64 experts of 4096 x 2048, 6 per token (50 of them
// active): the first product streams 478 MB in 82 us (5.8 TB/s, 86 % of the
// copy rate), the second 239 MB in 42 us, and 35 us go into the router (4), the
// plans and first tiles (8 each), the spread of the CTAs' ends and the combine.
// The instructions that unpack and multiply a tile take 2100 cycles on an SM's
// 16 warps, its bytes 3200 at the copy rate, so a pass is bound by its bytes; an
// expert with more than four tokens takes a pass per four, and each streams its
// weights again: 32 tokens on 8 experts of 4096 x 11008 read 994 + 427 MB from
// DRAM where the weights are 406 + 203 MB, in 296 to 306 us where those need 90
// (the first product at 5.2 TB/s with the issue slots 63 % busy, the second at
// 3.5).  Tried and no faster: an expert's passes side by side, so that all but
// one find the weights in the L2 (310 us); eight tokens a pass; the whole layer
// as one cooperative kernel with barriers (32 tokens 329 us, one token 38
// instead of 30).
#include <cuda_fp16.h>

#include "mmq_internal.h"
#include "sm103_ptx.cuh"
#include "tc_common.cuh"

namespace {

using namespace mmq::ptx;
using namespace mmq::tc;

constexpr int kMaxTokens = MMQ_MOE_MAX_TOKENS;
constexpr int kMaxExperts = MMQ_MOE_MAX_EXPERTS;
constexpr int kMaxPairs = MMQ_MOE_MAX_PAIRS;
constexpr int kBlk = 144;     // bytes of a q4_K super-block
// A warp holds one super-block of a row at a time, a CTA's warps up to 16 (a
// row, or a slice of it), for four tokens.  (Eight tokens at a time halve the
// passes of an expert that many chose, but want twice the registers, so half
// the warps: 32 tokens, 2 of 8 experts each, 150 us instead of 127; 24 tokens,
// 2 of 16: 123 instead of 77.)
constexpr int kWarps = 16, kThreads = 32 * kWarps, kTok = 4;
// A weight tile is 32 rows x one super-block, one TMA box, two per warp in
// flight: 32 boxes per SM.  Streaming 604 MB through such rings with no other
// work takes 92 us (6.5 TB/s) with 32 boxes of 16 or of 32 rows in flight per
// SM, but 127 us with 48 and 154 us with 64.
constexpr int kRows = 32, kStages = 2;
constexpr int kTile = kRows * kBlk;
constexpr int kRedPitch = kRows + 8;   // floats per token: the four lanes of a row on four banks
constexpr int kBatch = 2;              // tiles per team in a batch
constexpr int kLag = 1;                // batches between a warp's own tiles of a batch and its adding the batch up
constexpr int kBuffers = 3;                                // batches of partial sums between the warps
constexpr int kPart = kTok * kRedPitch;                    // floats of one warp's tile
constexpr int kRed = kBatch * kWarps * kPart * 4;          // bytes of one buffer
constexpr int kRing = kWarps * kStages * kTile;
constexpr int kSmemBytes = kRing + kBuffers * kRed + 128;  // + alignment
static_assert(kSmemBytes <= 212 * 1024, "shared memory budget");

// Which tokens go to which expert: pair i = token i / top_k, its i % top_k-th
// expert.  An active expert (one with a token) has its pairs in a row of
// `order`, and one pass over its weights per kTok of them.
struct Plan {
    int active;
    int expert[kMaxExperts];
    int start[kMaxExperts + 1];   // an active expert's pairs: order[start[a]] .. order[start[a + 1] - 1]
    int pass[kMaxExperts + 1];    // passes of the active experts before it
    int order[kMaxPairs];
};

struct MoeArgs {
    mmq_q4K_moe_t p;
    float* logits;       // [tokens][experts]
    float* h;            // first product, rows in the plan's order: h [pairs][ffn], or if its sum is in
                         // parts [gu_slices][pairs][2 ffn] of gate and up, alternating
    float* y;            // second product [down_slices][pairs][model], rows by pair
    int gu_slices, down_slices;
    int* status;
};

// ----------------------------------------------------------------- router
// One CTA: one expert's logits for four tokens, the sum split over its warps
// so that a thread's loads are all in flight at once.
constexpr int kRouterThreads = 256;
__global__ void __launch_bounds__(kRouterThreads) moe_router_kernel(const MoeArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    const mmq_q4K_moe_t& p = a.p;
    __shared__ float part[kRouterThreads / 32][4];
    const int e = blockIdx.x, t0 = blockIdx.y * 4, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float4* w = reinterpret_cast<const float4*>(p.w_router + int64_t(e) * p.model);
    const float4* x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)   // past the last token: the last one again
        x[j] = reinterpret_cast<const float4*>(p.x + int64_t(min(t0 + j, p.tokens - 1)) * p.model);
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    const int n4 = p.model / 4;
#pragma unroll 4
    for (int i = threadIdx.x; i < n4; i += kRouterThreads) {
        const float4 wv = w[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float4 xv = x[j][i];
            acc[j] = fmaf(wv.x, xv.x, fmaf(wv.y, xv.y, fmaf(wv.z, xv.z, fmaf(wv.w, xv.w, acc[j]))));
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], m);
        if (lane == 0) part[warp][j] = acc[j];
    }
    __syncthreads();
    if (threadIdx.x < 4 && t0 + int(threadIdx.x) < p.tokens) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kRouterThreads / 32; ++i) s += part[i][threadIdx.x];
        a.logits[int64_t(t0 + threadIdx.x) * p.experts + e] = s;
    }
}

// One warp: token t's softmax and its top_k experts, best first.  A choice is
// two warp reductions over keys that order the values e^(logit - max), from 0
// to 1 and so by their bits.  A NaN or +Inf among the logits makes the sum and
// with it every softmax value NaN: all keys are equal then, the lowest experts
// are taken, distinct and in range as always, with weights of NaN.
__device__ __forceinline__ void choose(const MoeArgs& a, int t, int lane, int* ids, uint64_t* tokens_of, bool store) {
    const mmq_q4K_moe_t& p = a.p;
    constexpr int kPer = kMaxExperts / 32;
    const int used = (p.experts + 31) / 32;   // of the kPer values per lane
    float v[kPer];
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        if (j >= used) break;
        const int e = lane + 32 * j;
        v[j] = e < p.experts ? a.logits[int64_t(t) * p.experts + e] : -INFINITY;
        top = fmaxf(top, v[j]);
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
    float sum = 0.f;
    uint32_t key[kPer];   // 0: none or taken, 1: NaN, else the value's bits + 2
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        key[j] = 0;
        if (j >= used) break;
        if (lane + 32 * j < p.experts) {
            v[j] = expf(v[j] - top);
            sum += v[j];
            key[j] = __float_as_uint(v[j]) + 2u;
        }
    }
    if (__any_sync(0xffffffffu, sum != sum)) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) key[j] = key[j] ? 1u : 0u;
    }
    float picked = 0.f, mine = 0.f;   // lane i keeps the i-th choice
    int chosen = 0;
    for (int i = 0; i < p.top_k; ++i) {
        uint32_t best = 0;
        int at = kMaxExperts;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            if (j >= used) break;
            if (key[j] > best) {
                best = key[j];
                at = lane + 32 * j;
            }
        }
        const uint32_t most = __reduce_max_sync(0xffffffffu, best);
        at = __reduce_min_sync(0xffffffffu, best == most ? at : kMaxExperts);
        const float value = most > 1u ? __uint_as_float(most - 2u) : __int_as_float(0x7FC00000);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            if (j >= used) break;
            if (lane + 32 * j == at) key[j] = 0;
        }
        picked += value;
        if (lane == i) {
            mine = value;
            chosen = at;
        }
    }
    if (lane < p.top_k) {
        ids[t * p.top_k + lane] = chosen;
        atomicOr(reinterpret_cast<unsigned long long*>(tokens_of + chosen), 1ull << t);
    }
    if (store) {
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
        if (lane < p.top_k) {
            p.ids[t * p.top_k + lane] = chosen;
            p.weights[t * p.top_k + lane] = mine / (p.renormalize ? picked : sum);
        }
    }
}

struct PlanScratch {
    uint64_t tokens_of[kMaxExperts];   // one bit per token of an expert
    int ids[kMaxPairs];
    int totals[3][kMaxExperts / 32];
};

// Fill `plan` (shared memory) from the logits; `store`: also the chosen
// experts and their weights to the caller.
__device__ __forceinline__ void make_plan(const MoeArgs& a, Plan* plan, PlanScratch* z, bool store) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = threadIdx.x;
    static_assert(kMaxExperts <= kThreads && kMaxTokens <= 64, "one thread per expert, one bit per token");
    if (e < kMaxExperts) z->tokens_of[e] = 0;
    __syncthreads();
    for (int t = warp; t < a.p.tokens; t += kThreads / 32) choose(a, t, lane, z->ids, z->tokens_of, store);
    __syncthreads();
    uint64_t mine = e < kMaxExperts ? z->tokens_of[e] : 0;
    const int n = __popcll(mine), passes = (n + kTok - 1) / kTok;
    // prefixes over the experts: of their pairs, their passes, and the active ones
    int pairs = n, pass = passes;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, pairs, m), v = __shfl_up_sync(0xffffffffu, pass, m);
        if (lane >= m) {
            pairs += u;
            pass += v;
        }
    }
    const uint32_t live = __ballot_sync(0xffffffffu, n > 0);
    if (lane == 31 && e < kMaxExperts) {
        z->totals[0][warp] = pairs;
        z->totals[1][warp] = pass;
        z->totals[2][warp] = __popc(live);
    }
    __syncthreads();
    if (e < kMaxExperts) {
        int at = pairs - n, first = pass - passes, rank = __popc(live & ((1u << lane) - 1u));
        for (int w = 0; w < warp; ++w) {
            at += z->totals[0][w];
            first += z->totals[1][w];
            rank += z->totals[2][w];
        }
        if (n > 0) {
            plan->expert[rank] = e;
            plan->start[rank] = at;
            plan->pass[rank] = first;
            for (; mine; mine &= mine - 1) {
                const int t = __ffsll(static_cast<long long>(mine)) - 1;
                int j = 0;
                while (z->ids[t * a.p.top_k + j] != e) ++j;
                plan->order[at++] = t * a.p.top_k + j;
            }
        }
        if (e == kMaxExperts - 1) {
            rank += n > 0;
            plan->active = rank;
            plan->start[rank] = at;
            plan->pass[rank] = first + passes;
        }
    }
    __syncthreads();
}

// --------------------------------------------------------- expert products
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with nothing to add to.
__device__ __forceinline__ void mma16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma1688(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%7,%7,%7,%7};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a0), "r"(a1), "r"(b0), "f"(0.f));
}
__device__ __forceinline__ uint32_t h2u(__half2 v) { return *reinterpret_cast<const uint32_t*>(&v); }
__device__ __forceinline__ __half2 u2h(uint32_t v) { return *reinterpret_cast<const __half2*>(&v); }
__device__ __forceinline__ float silu_times(float gate, float up) { return gate / (1.f + expf(-gate)) * up; }

// One row's part in a lane: lane t of a row's four holds sub-blocks 2t and
// 2t + 1, the low and high nibbles of the row's bytes 32 t .. 32 t + 31.
struct RowScale {
    __half2 s_lo, b_lo, s_hi, b_hi;   // nibbles to sc q: (1024 + q) sc - 1024 sc, (1024 + 16 q) sc / 16 - 64 sc
    uint32_t m;                       // the two minima, fp16
    float d, dmin;
};
// What a lane needs to know of its two sub-blocks' places among the 6-bit
// scales: sub-blocks 0-3 are whole, the low six bits of bytes 0-3 (scales) and
// 4-7 (minima); 4-7 have their low four bits in the nibbles of bytes 8-11 and
// their high two on top of those bytes.
struct Place {
    uint32_t low, high, sel;   // masks of the low and of the high bits; bytes 2 (t & 1) and the next into halfwords
    bool upper;                // sub-blocks 4-7
    __device__ __forceinline__ explicit Place(int t)
        : low(t < 2 ? 0x3F3F3F3Fu : 0x0F0F0F0Fu), high(t < 2 ? 0u : 0x30303030u), sel((t & 1) ? 0x4342u : 0x4140u),
          upper(t >= 2) {}
};
__device__ __forceinline__ RowScale row_scale(const uint4& head, const Place& at) {
    RowScale r;
    const uint32_t scw = ((at.upper ? head.w : head.y) & at.low) | ((head.y >> 2) & at.high);
    const uint32_t mw = ((at.upper ? head.w >> 4 : head.z) & at.low) | ((head.z >> 2) & at.high);
    const __half2 k1024 = u2h(0x64006400u);
    const __half2 sc = __hsub2(u2h(prmt(scw, 0x64646464u, at.sel)), k1024);
    r.m = h2u(__hsub2(u2h(prmt(mw, 0x64646464u, at.sel)), k1024));
    r.s_lo = __low2half2(sc);
    const __half2 hi = __high2half2(sc);
    r.s_hi = __hmul2(hi, u2h(0x2C002C00u));             // / 16
    r.b_lo = __hmul2(r.s_lo, u2h(0xE400E400u));         // * -1024, at most 64512
    r.b_hi = __hmul2(hi, u2h(0xD400D400u));             // * -64
    const float2 f = __half22float2(u2h(head.x));
    r.d = f.x;
    r.dmin = f.y;
    return r;
}
// (a & b) | c in one instruction.
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
// Four nibbles' sc q as two fp16 pairs: elements {0, 2} and {1, 3} of the word.
__device__ __forceinline__ void unpack_lo(uint32_t w, uint32_t w8, const RowScale& r, uint32_t magic, uint32_t& x02,
                                          uint32_t& x13) {
    x02 = h2u(__hfma2(u2h(and_or(w, 0x000F000Fu, magic)), r.s_lo, r.b_lo));
    x13 = h2u(__hfma2(u2h(and_or(w8, 0x000F000Fu, magic)), r.s_lo, r.b_lo));
}
__device__ __forceinline__ void unpack_hi(uint32_t w, uint32_t w8, const RowScale& r, uint32_t magic, uint32_t& x02,
                                          uint32_t& x13) {
    x02 = h2u(__hfma2(u2h(and_or(w, 0x00F000F0u, magic)), r.s_hi, r.b_hi));
    x13 = h2u(__hfma2(u2h(and_or(w8, 0x00F000F0u, magic)), r.s_hi, r.b_hi));
}

// A group of four tokens' activations of one super-block, as the second
// operand of the matrix instructions: column 2 i is token i's hi, 2 i + 1 its
// lo, so lane (column g, t) holds one part of the values of sub-blocks 2t and
// 2t + 1 of token g / 2: step w takes values 4w .. 4w + 3 of both, in the order
// 0, 2, 1, 3 that unpacking the nibbles gives.
struct Act {
    uint32_t b[8][4];
    uint32_t sums;   // the two sub-blocks' sums
    float up;        // token t's 2^e (the lane's column of the result)
};
template <typename Load>   // load(i): values 4 i .. 4 i + 3 of the lane's 64, f32
__device__ __forceinline__ void make_act(Act& act, int lane, Load load) {
    float4 v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = load(i);
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        top = fmaxf(fmaxf(top, fmaxf(fabsf(v[i].x), fabsf(v[i].y))), fmaxf(fabsf(v[i].z), fabsf(v[i].w)));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // 2^e with top 2^-e in [128, 256), e from -126 on
    int e = int(__float_as_uint(top) >> 23) - 127 - 7;
    e = e < -126 ? -126 : e;
    const float down = __uint_as_float(uint32_t(127 - e) << 23);
    const bool is_lo = (lane >> 2) & 1;
    // two values' hi or lo; packed conversions (single ones take the slow pipe)
    auto part = [&](float f, float h) {
        const __half2 hi = __floats2half2_rn(f, h);
        const float2 back = __half22float2(hi);
        const __half2 lo = __floats2half2_rn(f - back.x, h - back.y);
        return is_lo ? h2u(lo) : h2u(hi);
    };
    float sums[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        sums[c] = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            const float4 u = v[8 * c + w];
            const float f[4] = {u.x * down, u.y * down, u.z * down, u.w * down};
            act.b[w][2 * c] = part(f[0], f[2]);
            act.b[w][2 * c + 1] = part(f[1], f[3]);
            sums[c] += (f[0] + f[1]) + (f[2] + f[3]);
        }
    }
    act.sums = part(sums[0], sums[1]);
    act.up = __shfl_sync(0xffffffffu, __uint_as_float(uint32_t(127 + e) << 23), 8 * (lane & 3));
}

// A run of row tiles of one (active expert, slice, pass).
struct Run {
    int a, slice, pass, first, count, left;   // left: tiles the CTA still has, this run's among them
    __device__ __forceinline__ void next(const Plan& plan, int slices, int tiles) {
        left -= count;
        first = 0;
        count = min(tiles, left);
        if (++pass == plan.pass[a + 1] - plan.pass[a]) {
            pass = 0;
            if (++slice == slices) {
                slice = 0;
                ++a;
            }
        }
    }
};

// The shape of one product.
struct Shape {
    int rows, nsb, slices, per, teams, tiles;   // per: super-blocks of a slice and warps of a team
};

// A CTA's share of one product, and where its warps are in it.
struct Product : Shape {
    const CUtensorMap* map;
    int team, ks;  // this warp's team and its super-block of a slice
    Run run;
    Run in;             // the run that lane 0 has issued up to,
    int in_left = 0;    // its tiles that are left for this warp's team,
    int in_x = 0, in_y = 0;   // and the next one's place in the tensor map

    __device__ __forceinline__ Product(const CUtensorMap* m, const Shape& shape, const Plan& plan, int* start_at)
        : Shape(shape), map(m) {
        const int warp = threadIdx.x >> 5;
        team = warp / per;
        ks = warp - team * per;
        // equal consecutive parts of all passes' tiles, the first `more` one longer
        const uint32_t each = uint32_t(slices * tiles), total = uint32_t(plan.pass[plan.active]) * each;
        const uint32_t mine = total / gridDim.x, more = total - mine * gridDim.x;
        const uint32_t i0 = blockIdx.x * mine + min(blockIdx.x, more), i1 = i0 + mine + (blockIdx.x < more ? 1u : 0u);
        const int p0 = int(i0 / each);
        if (int(threadIdx.x) < plan.active && plan.pass[threadIdx.x] <= p0 && p0 < plan.pass[threadIdx.x + 1])
            *start_at = threadIdx.x;
        __syncthreads();
        run.left = int(i1 - i0);
        run.a = run.left > 0 ? *start_at : 0;
        const int passes = plan.pass[run.a + 1] - plan.pass[run.a];
        const int local = run.left > 0 ? int(i0) - plan.pass[run.a] * int(each) : 0, sp = local / tiles;
        run.first = local - sp * tiles;
        run.slice = sp / passes;
        run.pass = sp - run.slice * passes;
        run.count = min(tiles - run.first, run.left);
        in = run;
        if (team >= teams) in.left = 0;
        enter(plan);
    }
    // The next run from `in` on that has a tile for this warp.
    __device__ __forceinline__ void enter(const Plan& plan) {
        for (; in.left > 0; in.next(plan, slices, tiles)) {
            const int sb = in.slice * per + ks;
            if (team >= in.count || sb >= nsb) continue;
            in_left = (in.count - team + teams - 1) / teams;
            in_x = sb * kBlk;
            in_y = plan.expert[in.a] * rows + (in.first + team) * kRows;
            return;
        }
        in_left = 0;
    }
};

struct Layer {
    const MoeArgs& a;
    const Plan& plan;
    AbortFlag abort_flag;
    uint32_t bar0, red_full, red_empty, ring;
    float* red0;
    uint32_t magic;                        // fp16 1024 twice, in a register: one constant per instruction
    int in_stage = 0, out_stage = 0, pending = 0, buffer = 0, turn = 0;
    uint32_t out_phase = 0, red_phase = 0;
    Act act;

    // Lane 0: the warp's next weight tile.
    __device__ __forceinline__ void issue(Product& w) {
        if (w.in_left == 0 || abort_flag.raised()) return;
        const uint32_t bar = bar0 + 8u * uint32_t(in_stage);
        mbar_arrive_expect_tx(bar, kTile);
        tma_load_2d(ring + uint32_t(in_stage * kTile), w.map, bar, w.in_x, w.in_y);
        ++pending;
        if (++in_stage == kStages) in_stage = 0;
        w.in_y += w.teams * kRows;
        if (--w.in_left == 0) {
            w.in.next(plan, w.slices, w.tiles);
            w.enter(plan);
        }
    }
    __device__ __forceinline__ void start(Product& w) {
        if ((threadIdx.x & 31) == 0)
            for (int i = 0; i < kStages; ++i) issue(w);
    }

    // This warp's operand: tokens first .. first + ntok - 1 of the plan's
    // order; `all`: the tokens themselves.
    template <bool kDown>
    __device__ __forceinline__ void fill(const Product& w, int slice, int first, int ntok, bool all) {
        const mmq_q4K_moe_t& p = a.p;
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const int sb = slice * w.per + w.ks, tok = g >> 1, pos = first + tok;
        const bool have = w.team < w.teams && sb < w.nsb && tok < ntok;
        const int64_t col = int64_t(sb) * 256 + 64 * t;
        const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
        if (!kDown || a.gu_slices == 1) {
            const float* x = nullptr;
            if (have)
                x = kDown ? a.h + int64_t(pos) * p.ffn + col
                          : p.x + int64_t(all ? tok : plan.order[pos] / p.top_k) * p.model + col;
            make_act(act, lane, [&](int i) { return have ? reinterpret_cast<const float4*>(x)[i] : zero; });
        } else {
            const int64_t pairs = int64_t(p.tokens) * p.top_k;
            make_act(act, lane, [&](int i) {
                float4 c0 = zero, c1 = zero;
                if (have) {
                    for (int s = 0; s < a.gu_slices; ++s) {
                        const float4* x = reinterpret_cast<const float4*>(a.h + ((s * pairs + pos) * p.ffn + col + 4 * i) * 2);
                        const float4 c = x[0], d = x[1];
                        c0.x += c.x; c0.y += c.y; c0.z += c.z; c0.w += c.w;
                        c1.x += d.x; c1.y += d.y; c1.z += d.z; c1.w += d.w;
                    }
                }
                return make_float4(silu_times(c0.x, c0.y), silu_times(c0.z, c0.w), silu_times(c1.x, c1.y),
                                   silu_times(c1.z, c1.w));
            });
        }
    }

    // The warp's partial sums of the tile at shared address st, to `mine`.
    __device__ __forceinline__ void tile(uint32_t st, float* mine) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const Place place(t);
#pragma unroll 1
        for (int m = 0; m < kRows; m += 16) {
            const uint32_t ra = st + uint32_t((m + g) * kBlk), rb = ra + 8 * kBlk;
            const RowScale r0 = row_scale(lds128(ra), place), r1 = row_scale(lds128(rb), place);
            // The low and the high nibbles apart, since the matrix instructions
            // truncate each step of a sum (9.8e-7 -> 5e-7 of the result for one
            // token).
            float lo[4], hi[4], mn[4];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const uint4 c = lds128(ra + uint32_t(16 + 32 * t + 16 * half));
                const uint4 d = lds128(rb + uint32_t(16 + 32 * t + 16 * half));
                const uint32_t w0[4] = {c.x, c.y, c.z, c.w}, w1[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t x0, x1, x2, x3, y0, y1, y2, y3;
                    const uint32_t p0 = w0[i] >> 8, p1 = w1[i] >> 8;
                    unpack_lo(w0[i], p0, r0, magic, x0, x2);
                    unpack_lo(w1[i], p1, r1, magic, x1, x3);
                    unpack_hi(w0[i], p0, r0, magic, y0, y2);
                    unpack_hi(w1[i], p1, r1, magic, y1, y3);
                    const uint32_t* b = act.b[4 * half + i];
                    if (half + i == 0) {
                        mma16816_first(lo, x0, x1, x2, x3, b[0], b[1]);
                        mma16816_first(hi, y0, y1, y2, y3, b[2], b[3]);
                    } else {
                        mma16816(lo, x0, x1, x2, x3, b[0], b[1]);
                        mma16816(hi, y0, y1, y2, y3, b[2], b[3]);
                    }
                }
            }
            mma1688(mn, r0.m, r1.m, act.sums);
            const float s0 = (lo[0] + hi[0]) + (lo[1] + hi[1]), s1 = (lo[2] + hi[2]) + (lo[3] + hi[3]);
            mine[t * kRedPitch + m + g] = act.up * (r0.d * s0 - r0.dmin * (mn[0] + mn[1]));
            mine[t * kRedPitch + m + g + 8] = act.up * (r1.d * s1 - r1.dmin * (mn[2] + mn[3]));
        }
    }

    // A batch of partial sums to be added up: tiles row_tile .. + tiles - 1
    // (kBatch per team, team by team) for tokens first .. first + ntok - 1 of the
    // plan's order.
    struct Batch {
        const float* red;
        uint32_t full, empty, phase;
        int first, ntok, held, slice, row_tile, tiles;
    };
    // One warp: two rows of one token per lane and step, the team's warps in order.
    template <bool kDown>
    __device__ __forceinline__ bool add(const Product& w, const Batch& d, bool all) {
        const mmq_q4K_moe_t& p = a.p;
        const int lane = threadIdx.x & 31;
        if (!__all_sync(0xffffffffu, wait_bounded(d.full, d.phase, abort_flag, a.status))) return false;
        constexpr int kLanes = kRows / 2;
        const int r = 2 * (lane % kLanes);
        for (int i = 0; i < d.tiles; ++i) {
            const int row = (d.row_tile + i) * kRows + r;
            const int nb = i >= w.teams ? 1 : 0, tm = i - nb * w.teams;
            static_assert(kBatch == 2, "a team's first or second tile");
            for (int tok = lane / kLanes; tok < d.ntok; tok += 32 / kLanes) {
                const int pos = d.first + tok, col = all ? plan.order[pos] / p.top_k : tok;
                const float* from = d.red + (nb * kWarps + tm * w.per) * kPart + col * kRedPitch + r;
                float s0 = 0.f, s1 = 0.f;
#pragma unroll 8
                for (int v = 0; v < d.held; ++v) {
                    const float2 f = *reinterpret_cast<const float2*>(from + v * kPart);
                    s0 += f.x;
                    s1 += f.y;
                }
                const int64_t base = int64_t(d.slice) * p.tokens * p.top_k;
                if (kDown)
                    *reinterpret_cast<float2*>(a.y + (base + plan.order[pos]) * w.rows + row) = make_float2(s0, s1);
                else if (w.slices > 1)
                    *reinterpret_cast<float2*>(a.h + (base + pos) * w.rows + row) = make_float2(s0, s1);
                else
                    a.h[int64_t(pos) * p.ffn + (row >> 1)] = silu_times(s0, s1);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(d.empty);
        return true;
    }

    template <bool kDown>
    __device__ __forceinline__ void go(Product& w) {
        const mmq_q4K_moe_t& p = a.p;
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        // Few tokens in all: every expert gets the columns of all of them
        // (which the matrix instructions have room for anyway), made once.
        const bool all = !kDown && p.tokens <= kTok && w.slices == 1;
        if (all) fill<kDown>(w, 0, 0, p.tokens, true);
        Batch due = {};
        int wait = 0;   // batches until this warp adds `due` up
        for (; w.run.left > 0; w.run.next(plan, w.slices, w.tiles)) {
            const Run& run = w.run;
            const int first = plan.start[run.a] + run.pass * kTok;
            const int ntok = min(kTok, plan.start[run.a + 1] - first);
            const int held = min(w.per, w.nsb - run.slice * w.per);   // super-blocks of this slice
            const bool works = w.team < w.teams && w.ks < held;
            if (!all) fill<kDown>(w, run.slice, first, ntok, false);
            for (int j0 = 0; j0 < run.count; j0 += kBatch * w.teams) {
                float* const red = red0 + buffer * (kRed / 4);
                // The buffer's last batch has been added up (at first: passes at once).
                if (!__all_sync(0xffffffffu, wait_bounded(red_empty + 8u * uint32_t(buffer), red_phase ^ 1u, abort_flag, a.status)))
                    return;
#pragma unroll 1
                for (int nb = 0; nb < kBatch; ++nb) {
                    if (!works || j0 + nb * w.teams + w.team >= run.count) break;
                    if (!__all_sync(0xffffffffu, wait_bounded(bar0 + 8u * uint32_t(out_stage), out_phase, abort_flag, a.status)))
                        return;
                    float* const mine = red + (nb * kWarps + warp) * kPart;
                    const uint32_t st = ring + uint32_t(out_stage * kTile);
                    tile(st, mine);
                    // The stores depend on every load from the stage, so those
                    // are done in every lane: the next copy may land in it.
                    __syncwarp();
                    if (lane == 0) {
                        --pending;
                        issue(w);
                    }
                    if (++out_stage == kStages) {
                        out_stage = 0;
                        out_phase ^= 1u;
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(red_full + 8u * uint32_t(buffer));
                if (turn == warp) {
                    due = {red, red_full + 8u * uint32_t(buffer), red_empty + 8u * uint32_t(buffer), red_phase, first, ntok,
                           held, run.slice, run.first + j0, min(kBatch * w.teams, run.count - j0)};
                    wait = kLag;
                } else if (wait > 0 && --wait == 0) {
                    if (!add<kDown>(w, due, all)) return;
                }
                if (++turn == kWarps) turn = 0;
                if (++buffer == kBuffers) {
                    buffer = 0;
                    red_phase ^= 1u;
                }
            }
        }
        if (wait > 0) add<kDown>(w, due, all);
    }

    // Only after a wait ran out is anything still in flight.
    __device__ __forceinline__ void drain() {
        if ((threadIdx.x & 31) == 0)
            for (; pending > 0; --pending) {
                wait_drain(bar0 + 8u * uint32_t(out_stage), out_phase, a.status);
                if (++out_stage == kStages) {
                    out_stage = 0;
                    out_phase ^= 1u;
                }
            }
    }
};

// One product of all active experts, one CTA per SM.  Activations are
// stationary: a warp keeps the operand of one super-block for four tokens in
// registers and streams weight tiles of it through a ring of its own; the warps
// of a team hold the super-blocks of a row (or of a slice of at most 16 of it),
// so a team reads whole rows.  The partial sums of a batch (two
// tiles per team) meet in shared memory: the warps take turns to add a batch up, in
// a fixed order, and store it, each a batch after its own tiles of it, when
// the others have long finished theirs.  (Adding at once makes every warp
// wait for the one before it, which is late from its own adding: 4950 cycles a
// batch, of them 2100 of products and 200 of waiting for weights.)  The row
// tiles of all passes of all active experts are dealt out in equal consecutive
// parts.
//
// Every CTA makes the plan from the logits.  The second product does so, and
// asks for its first weights, before it waits for the first one's results.
// `inject`, a test hook: 1 more arrival than there will be on the first CTA's
// barriers for full batches.
template <bool kDown>
__global__ void __launch_bounds__(kThreads, 1)
moe_product_kernel(const __grid_constant__ CUtensorMap map, const Shape shape, const MoeArgs a, const int inject) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    __shared__ Plan plan;
    __shared__ PlanScratch scratch;
    __shared__ uint64_t bars[kWarps * kStages + 2 * kBuffers];
    __shared__ uint32_t abort_word;
    __shared__ int start_at;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Layer layer{a, plan, AbortFlag{smem_u32(&abort_word)}, smem_u32(&bars[warp * kStages]),
                    smem_u32(&bars[kWarps * kStages]), smem_u32(&bars[kWarps * kStages + kBuffers]),
                    smem_u32(smem) + uint32_t(warp * kStages * kTile), reinterpret_cast<float*>(smem + kRing)};
    asm volatile("mov.b32 %0, 0x64006400;" : "=r"(layer.magic));
    if (threadIdx.x == 0) {
        layer.abort_flag.set(0u);
        for (int i = 0; i < kBuffers; ++i) {
            mbar_init(layer.red_full + 8u * uint32_t(i), kWarps + (!kDown && blockIdx.x == 0 ? inject : 0));
            mbar_init(layer.red_empty + 8u * uint32_t(i), 1);
        }
        prefetch_tmap(&map);
    }
    if (lane == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(layer.bar0 + 8u * uint32_t(i), 1);
        fence_barrier_init();
    }
    // The logits are complete before the second product starts: the first one
    // lets it be scheduled only after its own wait for the router.
    if (!kDown) griddep_wait();
    griddep_launch_dependents();
    make_plan(a, &plan, &scratch, !kDown && blockIdx.x == 0);
    Product w(&map, shape, plan, &start_at);
    layer.start(w);
    if (kDown) griddep_wait();   // the first product
    layer.go<kDown>(w);
    layer.drain();
}

// out = residual + the sum of the chosen experts' rows
__global__ void __launch_bounds__(128) moe_combine_kernel(const MoeArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    const mmq_q4K_moe_t& p = a.p;
    const int t = blockIdx.y, c = (blockIdx.x * 128 + threadIdx.x) * 4;
    if (c >= p.model) return;
    const int64_t pairs = int64_t(p.tokens) * p.top_k;
    const int64_t at = int64_t(t) * p.model + c;
    float4 r = p.residual ? *reinterpret_cast<const float4*>(p.residual + at) : make_float4(0.f, 0.f, 0.f, 0.f);
    const float* y = a.y + int64_t(t) * p.top_k * p.model + c;
    // the chosen experts in order, the parts of each in order, loads ahead of the sums
    const int n = p.top_k * a.down_slices;
    int k = 0, part = 0;
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
        const float4 v = *reinterpret_cast<const float4*>(y + (part * pairs + k) * p.model);
        const float w = p.weights[t * p.top_k + k];
        r.x = fmaf(w, v.x, r.x); r.y = fmaf(w, v.y, r.y); r.z = fmaf(w, v.z, r.z); r.w = fmaf(w, v.w, r.w);
        if (++part == a.down_slices) {
            part = 0;
            ++k;
        }
    }
    *reinterpret_cast<float4*>(p.out + at) = r;
}

// A kernel of this call that follows another: it may be scheduled before the
// other ends, and waits for it (griddep_wait) before it reads its results.
cudaLaunchConfig_t follow_config(dim3 grid, dim3 block, size_t smem, cudaStream_t s, cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    return cfg;
}

// A row's super-blocks in slices of at most 16.
int slices_of(int inner) { return (inner / 256 + kWarps - 1) / kWarps; }

struct Sizes {
    size_t logits, h, y, bytes;
};
Sizes sizes(const mmq_q4K_moe_t& p) {
    auto up = [](size_t b) { return (b + 255) & ~size_t(255); };
    Sizes z;
    const size_t pairs = size_t(p.tokens) * size_t(p.top_k);
    const int gu = slices_of(p.model);
    z.logits = 0;
    z.h = z.logits + up(size_t(p.tokens) * size_t(p.experts) * 4);
    z.y = z.h + up(pairs * size_t(p.ffn) * 4 * (gu > 1 ? 2 * size_t(gu) : 1));
    z.bytes = z.y + size_t(slices_of(p.ffn)) * pairs * size_t(p.model) * 4;
    return z;
}

template <bool kDown>
cudaError_t launch_product(const MoeArgs& a, int nsm, int inject, cudaStream_t s) {
    const int rows = kDown ? a.p.model : 2 * a.p.ffn;
    Shape shape;
    shape.rows = rows;
    shape.nsb = (kDown ? a.p.ffn : a.p.model) / 256;
    shape.slices = kDown ? a.down_slices : a.gu_slices;
    shape.per = (shape.nsb + shape.slices - 1) / shape.slices;
    shape.teams = kWarps / shape.per;
    shape.tiles = rows / kRows;
    const uint64_t pitch = uint64_t(shape.nsb) * kBlk;
    CUtensorMap map;
    if (!encode_2d(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, kDown ? a.p.w_down : a.p.w_gu, pitch,
                   uint64_t(a.p.experts) * uint64_t(rows), pitch, kBlk, kRows, CU_TENSOR_MAP_SWIZZLE_NONE))
        return cudaErrorInvalidValue;
    cudaError_t e;
    if ((e = cudaFuncSetAttribute(moe_product_kernel<kDown>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes)))
        return e;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = follow_config(dim3(unsigned(nsm)), dim3(kThreads), kSmemBytes, s, attr);
    return cudaLaunchKernelEx(&cfg, moe_product_kernel<kDown>, map, shape, a, inject);
}

}  // namespace

namespace mmq {

size_t q4K_moe_workspace(const mmq_q4K_moe_t& p) { return sizes(p).bytes; }

cudaError_t launch_q4K_moe(const mmq_q4K_moe_t& p, void* workspace, int* status, int inject_timeout, cudaStream_t s) {
    int dev = 0, nsm = 0;
    cudaError_t e;
    if ((e = cudaGetDevice(&dev)) || (e = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev))) return e;
    const Sizes z = sizes(p);
    char* ws = static_cast<char*>(workspace);
    MoeArgs a;
    a.p = p;
    a.logits = reinterpret_cast<float*>(ws + z.logits);
    a.h = reinterpret_cast<float*>(ws + z.h);
    a.y = reinterpret_cast<float*>(ws + z.y);
    a.gu_slices = slices_of(p.model);
    a.down_slices = slices_of(p.ffn);
    a.status = status;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t first = launch_config(dim3(unsigned(p.experts), unsigned((p.tokens + 3) / 4)),
                                                   dim3(kRouterThreads), 0, s, attr);
    if ((e = cudaLaunchKernelEx(&first, moe_router_kernel, a))) return e;
    if ((e = launch_product<false>(a, nsm, inject_timeout, s))) return e;
    if ((e = launch_product<true>(a, nsm, 0, s))) return e;
    cudaLaunchAttribute last_attr[1];
    const cudaLaunchConfig_t last =
        follow_config(dim3(unsigned((p.model / 4 + 127) / 128), unsigned(p.tokens)), dim3(128), 0, s, last_attr);
    return cudaLaunchKernelEx(&last, moe_combine_kernel, a);
}

}  // namespace mmq
