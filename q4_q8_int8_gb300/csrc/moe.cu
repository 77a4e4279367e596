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
constexpr int kWarps = 16, kThreads = kWarps * 32;
constexpr int kBlk = 144;     // bytes of a q4_K super-block
// A weight tile is 32 rows x one super-block, one TMA box, two per warp in
// flight: 32 boxes per SM.  Streaming 604 MB through such rings with no other
// work takes 92 us (6.5 TB/s) with 32 boxes of 16 or of 32 rows in flight per
// SM, but 127 us with 48 and 154 us with 64.
constexpr int kRows = 32, kStages = 2;
constexpr int kTile = kRows * kBlk;

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
    float* logits;   // [tokens][experts]
    float* h;        // first product, rows in the plan's order: h [pairs][ffn], or if its sum is in
                     // parts [gu_slices][pairs][2 ffn] of gate and up, alternating
    float* y;        // second product [down_slices][pairs][model], rows by pair
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
// to 1 and so by their bits; NaN ranks below every number, so the chosen
// experts are always distinct and in range.
__device__ __forceinline__ void choose(const MoeArgs& a, int t, int lane, int* ids, uint64_t* tokens_of, bool store) {
    const mmq_q4K_moe_t& p = a.p;
    constexpr int kPer = kMaxExperts / 32;
    float v[kPer];
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
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
        if (lane + 32 * j < p.experts) {
            v[j] = expf(v[j] - top);
            sum += v[j];
            key[j] = v[j] == v[j] ? __float_as_uint(v[j]) + 2u : 1u;
        }
    }
    float picked = 0.f, mine = 0.f;   // lane i keeps the i-th choice
    int chosen = 0;
    for (int i = 0; i < p.top_k; ++i) {
        uint32_t best = 0;
        int at = kMaxExperts;
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (key[j] > best) {
                best = key[j];
                at = lane + 32 * j;
            }
        const uint32_t most = __reduce_max_sync(0xffffffffu, best);
        at = __reduce_min_sync(0xffffffffu, best == most ? at : kMaxExperts);
        const float value = most > 1u ? __uint_as_float(most - 2u) : __int_as_float(0x7FC00000);
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (lane + 32 * j == at) key[j] = 0;
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
    int totals[3][kWarps];
};

// Fill `plan` (shared memory) from the logits, for passes of `pass_tokens`;
// `store`: also the chosen experts and their weights to the caller.
__device__ void make_plan(const MoeArgs& a, Plan* plan, PlanScratch* z, int pass_tokens, bool store) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = threadIdx.x;
    static_assert(kMaxExperts <= kThreads && kMaxTokens <= 64, "one thread per expert, one bit per token");
    if (e < kMaxExperts) z->tokens_of[e] = 0;
    __syncthreads();
    for (int t = warp; t < a.p.tokens; t += kWarps) choose(a, t, lane, z->ids, z->tokens_of, store);
    __syncthreads();
    uint64_t mine = e < kMaxExperts ? z->tokens_of[e] : 0;
    const int n = __popcll(mine), passes = (n + pass_tokens - 1) / pass_tokens;
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
    if (lane == 31) {
        z->totals[0][warp] = pairs;
        z->totals[1][warp] = pass;
        z->totals[2][warp] = __popc(live);
    }
    __syncthreads();
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
    if (e == kThreads - 1) {
        plan->active = rank;
        plan->start[rank] = at;
        plan->pass[rank] = first;
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
__device__ __forceinline__ void mma1688(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(b0));
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
__device__ __forceinline__ RowScale row_scale(const uint4& head, int t) {
    RowScale r;
    const uint32_t scw = t < 2 ? sc_lo4(head.y) : sc_hi4(head.y, head.w);
    const uint32_t mw = t < 2 ? m_lo4(head.z) : m_hi4(head.z, head.w);
    const uint32_t sel = (t & 1) ? 0x4342u : 0x4140u;   // bytes 2(t & 1), 2(t & 1) + 1 into halfwords
    const __half2 k1024 = u2h(0x64006400u);
    const __half2 sc = __hsub2(u2h(prmt(scw, 0x64646464u, sel)), k1024);
    r.m = h2u(__hsub2(u2h(prmt(mw, 0x64646464u, sel)), k1024));
    r.s_lo = __low2half2(sc);
    r.s_hi = __hmul2(__high2half2(sc), u2h(0x2C002C00u));             // / 16
    r.b_lo = __hmul2(r.s_lo, u2h(0xE400E400u));                       // * -1024, at most 64512
    r.b_hi = __hmul2(__high2half2(sc), u2h(0xD400D400u));             // * -64
    r.d = __half2float(__ushort_as_half(uint16_t(head.x & 0xFFFFu)));
    r.dmin = __half2float(__ushort_as_half(uint16_t(head.x >> 16)));
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
    auto part = [&](float f) {
        const __half hi = __float2half_rn(f);
        return is_lo ? __float2half_rn(f - __half2float(hi)) : hi;
    };
    __half sums[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            const float4 u = v[8 * c + w];
            const float f[4] = {u.x * down, u.y * down, u.z * down, u.w * down};
            act.b[w][2 * c] = h2u(__halves2half2(part(f[0]), part(f[2])));
            act.b[w][2 * c + 1] = h2u(__halves2half2(part(f[1]), part(f[3])));
            s += (f[0] + f[1]) + (f[2] + f[3]);
        }
        sums[c] = part(s);
    }
    act.sums = h2u(__halves2half2(sums[0], sums[1]));
    act.up = __shfl_sync(0xffffffffu, __uint_as_float(uint32_t(127 + e) << 23), 8 * (lane & 3));
}

constexpr int kRedPitch = kRows + 8;   // floats per token: the four lanes of a row on four banks
template <int NG>
struct Smem {
    static constexpr int kBuffers = 5 - NG;                         // batches of partial sums between the warps
    static constexpr int kPart = 4 * NG * kRedPitch;                // floats of one warp's tile
    static constexpr int kRed = kWarps * kPart * 4;                 // bytes of one buffer
    static constexpr int kRing = kWarps * kStages * kTile;
    static constexpr int kBytes = kRing + kBuffers * kRed + 128;    // + alignment
};
static_assert(Smem<2>::kBytes <= 208 * 1024, "shared memory budget");

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

// Both products of the experts.  Activations are stationary: a warp keeps the
// operand of one super-block for 4 NG tokens in registers and streams weight
// tiles of that super-block through a ring of its own; the warps of a team hold the super-blocks of a row (or of a slice of
// at most 16 of it), so a team reads whole rows.  The partial sums of a batch
// (one tile per team) meet in shared memory: the warps take turns to add a
// batch up, in a fixed order, and store it, and none of the others waits for
// that unless it is a few batches ahead.  One CTA per SM; the row tiles of
// all passes of all active experts are dealt out in equal consecutive parts.
template <int NG, bool kDown>
__global__ void __launch_bounds__(kThreads, 1)
moe_expert_kernel(const __grid_constant__ CUtensorMap map, const MoeArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    __shared__ Plan plan;
    __shared__ PlanScratch scratch;
    constexpr int kBuffers = Smem<NG>::kBuffers;
    __shared__ uint64_t bars[kWarps * kStages + 2 * kBuffers];
    __shared__ uint32_t abort_word;
    __shared__ int start_at;
    const mmq_q4K_moe_t& p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const AbortFlag abort_flag{smem_u32(&abort_word)};
    const uint32_t bar0 = smem_u32(&bars[warp * kStages]), red_full = smem_u32(&bars[kWarps * kStages]);
    const uint32_t red_empty = red_full + 8 * kBuffers;
    constexpr int kTok = 4 * NG;
    if (threadIdx.x == 0) {
        abort_flag.set(0u);
        for (int i = 0; i < kBuffers; ++i) {
            mbar_init(red_full + 8u * uint32_t(i), kWarps);
            mbar_init(red_empty + 8u * uint32_t(i), 1);
        }
        prefetch_tmap(&map);
    }
    if (lane == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(bar0 + 8u * uint32_t(i), 1);
        fence_barrier_init();
    }
    // The logits are complete before the second product starts: the first one
    // lets it be scheduled only after its own wait for the router.
    if (!kDown) griddep_wait();
    griddep_launch_dependents();
    make_plan(a, &plan, &scratch, kTok, !kDown && blockIdx.x == 0);

    const int rows = kDown ? p.model : 2 * p.ffn, nsb = (kDown ? p.ffn : p.model) / 256;
    const int slices = kDown ? a.down_slices : a.gu_slices;
    const int per = (nsb + slices - 1) / slices, teams = kWarps / per;
    const int team = warp / per, ks = warp - team * per;
    const int tiles = rows / kRows, each = slices * tiles;   // tiles of a pass
    const uint32_t total = uint32_t(plan.pass[plan.active] * each);
    const int i0 = int(uint64_t(total) * blockIdx.x / gridDim.x), i1 = int(uint64_t(total) * (blockIdx.x + 1) / gridDim.x);
    if (i0 >= i1) return;
    if (int(threadIdx.x) < plan.active) {
        const int p0 = i0 / each;
        if (plan.pass[threadIdx.x] <= p0 && p0 < plan.pass[threadIdx.x + 1]) start_at = threadIdx.x;
    }
    __syncthreads();
    Run run;
    {
        run.a = start_at;
        const int local = i0 - plan.pass[run.a] * each, passes = plan.pass[run.a + 1] - plan.pass[run.a];
        const int sp = local / tiles;
        run.first = local - sp * tiles;
        run.slice = sp / passes;
        run.pass = sp - run.slice * passes;
        run.left = i1 - i0;
        run.count = min(tiles - run.first, run.left);
    }

    // The warp's weight stream: tiles team, team + teams, ... of each run.
    Run in = run;
    int in_tile = team, in_stage = 0, out_stage = 0, pending = 0;
    uint32_t out_phase = 0;
    const uint32_t ring = smem_u32(smem) + uint32_t(warp * kStages * kTile);
    auto settle = [&]() {   // to a run with a tile for this warp
        while (in.left > 0 && (in_tile >= in.count || in.slice * per + ks >= nsb)) {
            in.next(plan, slices, tiles);
            in_tile = team;
        }
    };
    auto issue = [&]() {
        if (in.left <= 0 || abort_flag.raised()) return;
        const uint32_t bar = bar0 + 8u * uint32_t(in_stage);
        mbar_arrive_expect_tx(bar, kTile);
        tma_load_2d(ring + uint32_t(in_stage * kTile), &map, bar, (in.slice * per + ks) * kBlk,
                    plan.expert[in.a] * rows + (in.first + in_tile) * kRows);
        ++pending;
        if (++in_stage == kStages) in_stage = 0;
        in_tile += teams;
        settle();
    };
    if (team >= teams) in.left = 0;
    settle();
    if (lane == 0)
        for (int i = 0; i < kStages; ++i) issue();
    if (kDown) griddep_wait();   // the first product

    float* const red0 = reinterpret_cast<float*>(smem + Smem<NG>::kRing);
    int buffer = 0, turn = 0;
    uint32_t red_phase = 0, magic;   // fp16 1024 twice, kept in a register: one constant per instruction
    asm volatile("mov.b32 %0, 0x64006400;" : "=r"(magic));
    for (; run.left > 0; run.next(plan, slices, tiles)) {
        const int first = plan.start[run.a] + run.pass * kTok;
        const int ntok = min(kTok, plan.start[run.a + 1] - first);
        const int sb = run.slice * per + ks, held = min(per, nsb - run.slice * per);   // super-blocks of this slice
        const bool works = team < teams && sb < nsb;
        Act act[NG];
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            const int tok = 4 * j + (g >> 1), pos = first + tok;
            const bool have = works && tok < ntok;
            const int64_t col = int64_t(sb) * 256 + 64 * t;
            const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
            if (!kDown) {
                const float* x = p.x + (have ? int64_t(plan.order[pos] / p.top_k) * p.model + col : 0);
                make_act(act[j], lane, [&](int i) { return have ? reinterpret_cast<const float4*>(x)[i] : zero; });
            } else if (a.gu_slices == 1) {
                const float* x = a.h + (have ? int64_t(pos) * p.ffn + col : 0);
                make_act(act[j], lane, [&](int i) { return have ? reinterpret_cast<const float4*>(x)[i] : zero; });
            } else {
                const int64_t pairs = int64_t(p.tokens) * p.top_k;
                make_act(act[j], lane, [&](int i) {
                    float4 u = zero, v = zero;
                    if (have) {
                        for (int s = 0; s < a.gu_slices; ++s) {
                            const float4* x =
                                reinterpret_cast<const float4*>(a.h + ((s * pairs + pos) * p.ffn + col + 4 * i) * 2);
                            const float4 c = x[0], d = x[1];
                            u.x += c.x; u.y += c.y; u.z += c.z; u.w += c.w;
                            v.x += d.x; v.y += d.y; v.z += d.z; v.w += d.w;
                        }
                    }
                    return make_float4(silu_times(u.x, u.y), silu_times(u.z, u.w), silu_times(v.x, v.y),
                                       silu_times(v.z, v.w));
                });
            }
        }
        for (int j0 = 0; j0 < run.count; j0 += teams) {
            float* const red = red0 + buffer * (Smem<NG>::kRed / 4);
            // The buffer's last batch has been added up (at first: passes at once).
            if (!__all_sync(0xffffffffu, wait_bounded(red_empty + 8u * uint32_t(buffer), red_phase ^ 1u, abort_flag, a.status)))
                break;
            if (works && j0 + team < run.count) {
                if (!__all_sync(0xffffffffu, wait_bounded(bar0 + 8u * uint32_t(out_stage), out_phase, abort_flag, a.status)))
                    break;
                const uint32_t st = ring + uint32_t(out_stage * kTile);
#pragma unroll 1
                for (int m = 0; m < kRows; m += 16) {
                    const uint32_t ra = st + uint32_t((m + g) * kBlk), rb = ra + 8 * kBlk;
                    const RowScale r0 = row_scale(lds128(ra), t), r1 = row_scale(lds128(rb), t);
                    float lo[NG][4], hi[NG][4];
#pragma unroll
                    for (int j = 0; j < NG; ++j)
#pragma unroll
                        for (int k = 0; k < 4; ++k) lo[j][k] = hi[j][k] = 0.f;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint4 u = lds128(ra + uint32_t(16 + 32 * t + 16 * half));
                        const uint4 v = lds128(rb + uint32_t(16 + 32 * t + 16 * half));
                        const uint32_t w0[4] = {u.x, u.y, u.z, u.w}, w1[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t x0, x1, x2, x3, y0, y1, y2, y3;
                            const uint32_t p0 = w0[i] >> 8, p1 = w1[i] >> 8;
                            unpack_lo(w0[i], p0, r0, magic, x0, x2);
                            unpack_lo(w1[i], p1, r1, magic, x1, x3);
                            unpack_hi(w0[i], p0, r0, magic, y0, y2);
                            unpack_hi(w1[i], p1, r1, magic, y1, y3);
#pragma unroll
                            for (int j = 0; j < NG; ++j) {
                                const uint32_t* b = act[j].b[4 * half + i];
                                mma16816(lo[j], x0, x1, x2, x3, b[0], b[1]);
                                mma16816(hi[j], y0, y1, y2, y3, b[2], b[3]);
                            }
                        }
                    }
                    float* mine = red + warp * Smem<NG>::kPart + t * kRedPitch + m + g;
#pragma unroll
                    for (int j = 0; j < NG; ++j) {
                        float mn[4] = {0.f, 0.f, 0.f, 0.f};
                        mma1688(mn, r0.m, r1.m, act[j].sums);
                        const float s0 = (lo[j][0] + hi[j][0]) + (lo[j][1] + hi[j][1]);
                        const float s1 = (lo[j][2] + hi[j][2]) + (lo[j][3] + hi[j][3]);
                        mine[4 * j * kRedPitch] = act[j].up * (r0.d * s0 - r0.dmin * (mn[0] + mn[1]));
                        mine[4 * j * kRedPitch + 8] = act[j].up * (r1.d * s1 - r1.dmin * (mn[2] + mn[3]));
                    }
                }
                // The stores above depend on every load from the stage, so
                // those are done in every lane: the next copy may land in it.
                __syncwarp();
                if (lane == 0) {
                    --pending;
                    issue();
                }
                if (++out_stage == kStages) {
                    out_stage = 0;
                    out_phase ^= 1u;
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(red_full + 8u * uint32_t(buffer));
            if (turn == warp) {   // this warp adds the batch up: two rows of one token per lane and step
                if (!__all_sync(0xffffffffu, wait_bounded(red_full + 8u * uint32_t(buffer), red_phase, abort_flag, a.status)))
                    break;
                const int batch = min(teams, run.count - j0);
                const int r = 2 * (lane & 15);
                for (int tm = 0; tm < batch; ++tm) {
                    const int row = (run.first + j0 + tm) * kRows + r;
                    for (int tok = lane >> 4; tok < ntok; tok += 2) {
                        const float* from = red + tm * per * Smem<NG>::kPart + tok * kRedPitch + r;
                        float s0 = 0.f, s1 = 0.f;
#pragma unroll 8
                        for (int w = 0; w < held; ++w) {
                            const float2 f = *reinterpret_cast<const float2*>(from + w * Smem<NG>::kPart);
                            s0 += f.x;
                            s1 += f.y;
                        }
                        const int pos = first + tok;
                        const int64_t base = int64_t(run.slice) * p.tokens * p.top_k;
                        if (kDown)
                            *reinterpret_cast<float2*>(a.y + (base + plan.order[pos]) * rows + row) = make_float2(s0, s1);
                        else if (slices > 1)
                            *reinterpret_cast<float2*>(a.h + (base + pos) * rows + row) = make_float2(s0, s1);
                        else
                            a.h[int64_t(pos) * p.ffn + (row >> 1)] = silu_times(s0, s1);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(red_empty + 8u * uint32_t(buffer));
            }
            if (++turn == kWarps) turn = 0;
            if (++buffer == kBuffers) {
                buffer = 0;
                red_phase ^= 1u;
            }
        }
    }
    // Only after a wait ran out is anything still in flight.
    if (lane == 0)
        for (; pending > 0; --pending) {
            wait_drain(bar0 + 8u * uint32_t(out_stage), out_phase, a.status);
            if (++out_stage == kStages) {
                out_stage = 0;
                out_phase ^= 1u;
            }
        }
}

// ---------------------------------------------------------------- combine
__global__ void __launch_bounds__(128) moe_combine_kernel(const MoeArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    const mmq_q4K_moe_t& p = a.p;
    const int t = blockIdx.y, c = (blockIdx.x * 128 + threadIdx.x) * 4;
    if (c >= p.model) return;
    const int64_t pairs = int64_t(p.tokens) * p.top_k;
    const int64_t at = int64_t(t) * p.model + c;
    float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < p.top_k; ++k) {
        const int64_t pair = int64_t(t) * p.top_k + k;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = 0; i < a.down_slices; ++i) {
            const float4 v = *reinterpret_cast<const float4*>(a.y + (i * pairs + pair) * p.model + c);
            s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
        }
        const float w = p.weights[pair];
        r.x = fmaf(w, s.x, r.x); r.y = fmaf(w, s.y, r.y); r.z = fmaf(w, s.z, r.z); r.w = fmaf(w, s.w, r.w);
    }
    if (p.residual) {
        const float4 v = *reinterpret_cast<const float4*>(p.residual + at);
        r.x += v.x; r.y += v.y; r.z += v.z; r.w += v.w;
    }
    *reinterpret_cast<float4*>(p.out + at) = r;
}

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

// A row's super-blocks in slices of at most 16, one per warp of a team.
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

template <int NG, bool kDown>
cudaError_t launch_expert(const MoeArgs& a, int nsm, cudaStream_t s) {
    const int rows = kDown ? a.p.model : 2 * a.p.ffn;
    const uint64_t pitch = uint64_t((kDown ? a.p.ffn : a.p.model) / 256) * kBlk;
    CUtensorMap map;
    if (!encode_2d(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, kDown ? a.p.w_down : a.p.w_gu, pitch,
                   uint64_t(a.p.experts) * uint64_t(rows), pitch, kBlk, kRows, CU_TENSOR_MAP_SWIZZLE_NONE))
        return cudaErrorInvalidValue;
    constexpr int smem = Smem<NG>::kBytes;
    cudaError_t e;
    if ((e = cudaFuncSetAttribute(moe_expert_kernel<NG, kDown>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)))
        return e;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = follow_config(dim3(unsigned(nsm)), dim3(kThreads), smem, s, attr);
    return cudaLaunchKernelEx(&cfg, moe_expert_kernel<NG, kDown>, map, a);
}

}  // namespace

namespace mmq {

size_t q4K_moe_workspace(const mmq_q4K_moe_t& p) { return sizes(p).bytes; }

cudaError_t launch_q4K_moe(const mmq_q4K_moe_t& p, void* workspace, int* status, cudaStream_t s) {
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
    // Four tokens at a time where an expert gets few on average, else eight.
    const bool few = p.tokens <= 4 || p.tokens * p.top_k <= 2 * p.experts;
    if ((e = few ? launch_expert<1, false>(a, nsm, s) : launch_expert<2, false>(a, nsm, s))) return e;
    if ((e = few ? launch_expert<1, true>(a, nsm, s) : launch_expert<2, true>(a, nsm, s))) return e;
    cudaLaunchAttribute last_attr[1];
    const cudaLaunchConfig_t last = follow_config(dim3(unsigned((p.model / 4 + 127) / 128), unsigned(p.tokens)), dim3(128), 0, s, last_attr);
    return cudaLaunchKernelEx(&last, moe_combine_kernel, a);
}

}  // namespace mmq
