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
constexpr int kStages = 4;    // weight tiles (16 rows x one super-block) in flight per warp
constexpr int kTile = 16 * kBlk;

// Which tokens go to which expert: pair i = token i / top_k, its i % top_k-th
// expert; order lists the pairs by expert.
struct Plan {
    int active;                      // experts with a token
    int expert[kMaxExperts];
    int start[kMaxExperts + 1];      // an active expert's pairs: order[start[a]] .. order[start[a + 1] - 1]
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
// One warp: one expert's logits for four tokens.
__global__ void __launch_bounds__(128) moe_router_kernel(const MoeArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    const mmq_q4K_moe_t& p = a.p;
    const int e = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int t0 = blockIdx.y * 4;
    if (e >= p.experts) return;
    const float4* w = reinterpret_cast<const float4*>(p.w_router + int64_t(e) * p.model);
    const float* x = p.x + int64_t(t0) * p.model;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    const int n4 = p.model / 4;
#pragma unroll 4
    for (int i = lane; i < n4; i += 32) {
        const float4 wv = w[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (t0 + j < p.tokens) {
                const float4 xv = reinterpret_cast<const float4*>(x + int64_t(j) * p.model)[i];
                acc[j] = fmaf(wv.x, xv.x, fmaf(wv.y, xv.y, fmaf(wv.z, xv.z, fmaf(wv.w, xv.w, acc[j]))));
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], m);
        if (lane == 0 && t0 + j < p.tokens) a.logits[int64_t(t0 + j) * p.experts + e] = acc[j];
    }
}

// One warp: token t's softmax and its top_k experts.  NaN ranks below every
// number, so the chosen experts are always distinct and in range.
__device__ __forceinline__ void choose(const MoeArgs& a, int t, int lane, int* ids, bool store) {
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
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const bool in = lane + 32 * j < p.experts;
        v[j] = in ? expf(v[j] - top) : 0.f;
        sum += v[j];
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    uint32_t taken = 0;
    float picked = 0.f, mine = 0.f;   // lane i keeps the i-th choice's weight
    for (int i = 0; i < p.top_k; ++i) {
        float best = -2.f, value = 0.f;
        int at = kMaxExperts;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const float key = v[j] == v[j] ? v[j] : -1.f;
            if (lane + 32 * j < p.experts && !((taken >> j) & 1u) && key > best) {
                best = key;
                value = v[j];
                at = lane + 32 * j;
            }
        }
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) {
            const float ob = __shfl_xor_sync(0xffffffffu, best, m), ov = __shfl_xor_sync(0xffffffffu, value, m);
            const int oa = __shfl_xor_sync(0xffffffffu, at, m);
            if (ob > best || (ob == best && oa < at)) {
                best = ob;
                value = ov;
                at = oa;
            }
        }
        if ((at & 31) == lane) taken |= 1u << (at >> 5);
        picked += value;
        if (lane == i) mine = value;
        if (lane == 0) {
            ids[t * p.top_k + i] = at;
            if (store && p.ids) p.ids[t * p.top_k + i] = at;
        }
    }
    if (store && lane < p.top_k) p.weights[t * p.top_k + lane] = mine / (p.renormalize ? picked : sum);
}

// Fill `plan` (shared memory) from the logits; `store`: also the chosen
// experts and their weights to the caller.  scratch: kMaxPairs + 2 * kWarps ints.
__device__ void make_plan(const MoeArgs& a, Plan* plan, int* scratch, bool store) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int* ids = scratch;
    int* totals = scratch + kMaxPairs;
    for (int t = warp; t < a.p.tokens; t += kWarps) choose(a, t, lane, ids, store);
    __syncthreads();
    static_assert(kMaxExperts <= kThreads, "one thread per expert");
    const int e = threadIdx.x, pairs = a.p.tokens * a.p.top_k;
    int n = 0;
    if (e < a.p.experts)
        for (int i = 0; i < pairs; ++i) n += ids[i] == e;
    // exclusive prefixes over the experts: of the pairs, and of the active ones
    int before = n;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, before, m);
        if (lane >= m) before += o;
    }
    const uint32_t live = __ballot_sync(0xffffffffu, n > 0);
    if (lane == 31) {
        totals[warp] = before;
        totals[kWarps + warp] = __popc(live);
    }
    __syncthreads();
    int at = before - n, rank = __popc(live & ((1u << lane) - 1u));
    for (int w = 0; w < warp; ++w) {
        at += totals[w];
        rank += totals[kWarps + w];
    }
    if (n > 0) {
        plan->expert[rank] = e;
        plan->start[rank] = at;
        for (int i = 0; i < pairs; ++i)
            if (ids[i] == e) plan->order[at++] = i;
    }
    if (e == kThreads - 1) {
        plan->active = rank + (n > 0);
        plan->start[rank + (n > 0)] = pairs;
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
// Four nibbles' sc q as two fp16 pairs: elements {0, 2} and {1, 3} of the word.
__device__ __forceinline__ void unpack_lo(uint32_t w, const RowScale& r, uint32_t& x02, uint32_t& x13) {
    x02 = h2u(__hfma2(u2h((w & 0x000F000Fu) | 0x64006400u), r.s_lo, r.b_lo));
    x13 = h2u(__hfma2(u2h(((w >> 8) & 0x000F000Fu) | 0x64006400u), r.s_lo, r.b_lo));
}
__device__ __forceinline__ void unpack_hi(uint32_t w, const RowScale& r, uint32_t& x02, uint32_t& x13) {
    x02 = h2u(__hfma2(u2h((w & 0x00F000F0u) | 0x64006400u), r.s_hi, r.b_hi));
    x13 = h2u(__hfma2(u2h(((w >> 8) & 0x00F000F0u) | 0x64006400u), r.s_hi, r.b_hi));
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
    float top = 0.f;
#pragma unroll 8
    for (int i = 0; i < 16; ++i) {
        const float4 v = load(i);
        top = fmaxf(fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y))), fmaxf(fabsf(v.z), fabsf(v.w)));
    }
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
            const float4 u = load(8 * c + w);
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

constexpr int kRedPitch = 24;   // floats per token: 16 rows, and no two lanes on one bank
template <int NG>
struct Smem {
    static constexpr int kBatch = 2 / NG;                                     // tiles per team and barrier
    static constexpr int kRed = kBatch * kWarps * 4 * NG * kRedPitch * 4;     // one buffer of partial sums
    static constexpr int kRing = kWarps * kStages * kTile;
    static constexpr int kBytes = kRing + 2 * kRed + 128;                     // + alignment
};
static_assert(Smem<1>::kBytes <= 200 * 1024 && Smem<2>::kBytes <= 200 * 1024, "shared memory budget");

// Both products of the experts.  Activations are stationary: a warp keeps the
// operand of one super-block for 4 NG tokens in registers and streams weight
// tiles (16 rows x that super-block, 2304 bytes, one TMA box) through a ring of
// its own; the KS warps of a team hold the KS super-blocks of a row (a slice of
// it, where it has more than 16), so a team reads whole rows, and their partial
// sums of a tile are joined through shared memory, in a fixed order.  One CTA
// per SM; the row tiles of all active experts are dealt out in equal
// consecutive runs, a run being one (expert, slice).
template <int NG, bool kDown>
__global__ void __launch_bounds__(kThreads, 1)
moe_expert_kernel(const __grid_constant__ CUtensorMap map, const MoeArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    __shared__ Plan plan;
    __shared__ int scratch[kMaxPairs + 2 * kWarps];
    __shared__ uint64_t bars[kWarps * kStages];
    __shared__ uint32_t abort_word;
    const mmq_q4K_moe_t& p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const AbortFlag abort_flag{smem_u32(&abort_word)};
    const uint32_t bar0 = smem_u32(&bars[warp * kStages]);
    if (threadIdx.x == 0) abort_flag.set(0u);
    if (lane == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(bar0 + 8u * uint32_t(i), 1);
        fence_barrier_init();
        if (warp == 0) prefetch_tmap(&map);
    }
    // The logits are complete before the second product starts: the first one
    // lets it be scheduled only after its own wait for the router.
    if (!kDown) {
        griddep_wait();
        griddep_launch_dependents();
    } else {
        griddep_launch_dependents();
    }
    make_plan(a, &plan, scratch, !kDown && blockIdx.x == 0);

    const int rows = kDown ? p.model : 2 * p.ffn, nsb = (kDown ? p.ffn : p.model) / 256;
    const int slices = kDown ? a.down_slices : a.gu_slices;
    const int per = (nsb + slices - 1) / slices, teams = kWarps / per;
    const int team = warp / per, ks = warp - team * per;
    const int tiles = rows / 16;
    const int64_t total = int64_t(plan.active) * slices * tiles;
    const int64_t i0 = total * blockIdx.x / gridDim.x, i1 = total * (blockIdx.x + 1) / gridDim.x;
    constexpr int kTok = 4 * NG, kBatch = Smem<NG>::kBatch;

    // Where a warp's weight stream is: a run's tiles team, team + teams, ... ,
    // once per pass over the run's tokens.
    struct Stream {
        int64_t at;          // first tile of the run
        int count, tile;     // tiles of the run, the next one
        int passes, x, y;    // passes left, box coordinates of the run's first tile
    } in;
    auto enter = [&]() {   // the run that starts at tile in.at; skips runs without a tile for this warp
        while (in.at < i1) {
            const int64_t q = in.at / tiles;
            const int first = int(in.at - q * tiles), act = int(q / slices), slice = int(q - int64_t(act) * slices);
            in.count = int(min(int64_t(tiles - first), i1 - in.at));
            in.passes = (plan.start[act + 1] - plan.start[act] + kTok - 1) / kTok;
            in.x = (slice * per + ks) * kBlk;
            in.y = plan.expert[act] * rows + first * 16;
            in.tile = team;
            if (team < in.count && slice * per + ks < nsb) return;
            in.at += in.count;
        }
    };
    in.at = team < teams ? i0 : i1;
    enter();
    const uint32_t ring = smem_u32(smem) + uint32_t(warp * kStages * kTile);
    int in_stage = 0, out_stage = 0, pending = 0;
    uint32_t out_phase = 0;
    auto issue = [&]() {   // lane 0 only
        if (in.at >= i1 || abort_flag.raised()) return;
        mbar_arrive_expect_tx(bar0 + 8u * uint32_t(in_stage), kTile);
        tma_load_2d(ring + uint32_t(in_stage * kTile), &map, bar0 + 8u * uint32_t(in_stage), in.x, in.y + in.tile * 16);
        ++pending;
        if (++in_stage == kStages) in_stage = 0;
        in.tile += teams;
        if (in.tile >= in.count) {
            in.tile = team;
            if (--in.passes == 0) {
                in.at += in.count;
                enter();
            }
        }
    };
    if (lane == 0)
        for (int i = 0; i < kStages; ++i) issue();
    if (kDown) griddep_wait();   // the first product

    float* const red0 = reinterpret_cast<float*>(smem + Smem<NG>::kRing);
    int buffer = 0;
    for (int64_t at = i0; at < i1;) {
        const int64_t q = at / tiles;
        const int first_tile = int(at - q * tiles), act_i = int(q / slices), slice = int(q - int64_t(act_i) * slices);
        const int count = int(min(int64_t(tiles - first_tile), i1 - at));
        const int first = plan.start[act_i], n = plan.start[act_i + 1] - first;
        const int sb = slice * per + ks, held = min(per, nsb - slice * per);   // super-blocks of this slice
        const bool works = team < teams && sb < nsb;
        for (int done = 0; done < n; done += kTok) {
            const int ntok = min(kTok, n - done);
            Act act[NG];
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                const int tok = 4 * j + (g >> 1), pos = first + done + tok;
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
                                const float4* x = reinterpret_cast<const float4*>(
                                    a.h + ((s * pairs + pos) * p.ffn + col + 4 * i) * 2);
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
            for (int j0 = 0; j0 < count; j0 += teams * kBatch) {
                float* const red = red0 + buffer * (Smem<NG>::kRed / 4);
#pragma unroll
                for (int nb = 0; nb < kBatch; ++nb) {
                    const int tile = j0 + nb * teams + team;
                    if (!works || tile >= count) continue;
                    if (!__all_sync(0xffffffffu, wait_bounded(bar0 + 8u * uint32_t(out_stage), out_phase, abort_flag,
                                                              a.status)))
                        continue;
                    const uint32_t st = ring + uint32_t(out_stage * kTile);
                    const uint32_t ra = st + uint32_t(g * kBlk), rb = ra + 8 * kBlk;
                    const RowScale r0 = row_scale(lds128(ra), t), r1 = row_scale(lds128(rb), t);
                    uint32_t w0[8], w1[8];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint4 u = lds128(ra + uint32_t(16 + 32 * t + 16 * i));
                        const uint4 v = lds128(rb + uint32_t(16 + 32 * t + 16 * i));
                        w0[4 * i] = u.x; w0[4 * i + 1] = u.y; w0[4 * i + 2] = u.z; w0[4 * i + 3] = u.w;
                        w1[4 * i] = v.x; w1[4 * i + 1] = v.y; w1[4 * i + 2] = v.z; w1[4 * i + 3] = v.w;
                    }
                    float lo[NG][4], hi[NG][4];
#pragma unroll
                    for (int j = 0; j < NG; ++j)
#pragma unroll
                        for (int k = 0; k < 4; ++k) lo[j][k] = hi[j][k] = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        uint32_t x0, x1, x2, x3, y0, y1, y2, y3;
                        unpack_lo(w0[i], r0, x0, x2);
                        unpack_lo(w1[i], r1, x1, x3);
                        unpack_hi(w0[i], r0, y0, y2);
                        unpack_hi(w1[i], r1, y1, y3);
#pragma unroll
                        for (int j = 0; j < NG; ++j) {
                            mma16816(lo[j], x0, x1, x2, x3, act[j].b[i][0], act[j].b[i][1]);
                            mma16816(hi[j], y0, y1, y2, y3, act[j].b[i][2], act[j].b[i][3]);
                        }
                    }
                    float* mine = red + (nb * kWarps + warp) * (kTok * kRedPitch) + t * kRedPitch + g;
#pragma unroll
                    for (int j = 0; j < NG; ++j) {
                        float mn[4] = {0.f, 0.f, 0.f, 0.f};
                        mma1688(mn, r0.m, r1.m, act[j].sums);
                        const float s0 = (lo[j][0] + hi[j][0]) + (lo[j][1] + hi[j][1]);
                        const float s1 = (lo[j][2] + hi[j][2]) + (lo[j][3] + hi[j][3]);
                        mine[4 * j * kRedPitch] = act[j].up * (r0.d * s0 - r0.dmin * (mn[0] + mn[1]));
                        mine[4 * j * kRedPitch + 8] = act[j].up * (r1.d * s1 - r1.dmin * (mn[2] + mn[3]));
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
                __syncthreads();
                // Join: the tiles of this batch in order, 16 rows each; a
                // buffer is written again only after the next barrier.
                const int batch = min(teams * kBatch, count - j0);
                auto sum = [&](int tile, int tok, int r) {
                    const int nb = tile / teams, tm = tile - nb * teams;
                    const float* from = red + (nb * kWarps + tm * per) * (kTok * kRedPitch) + tok * kRedPitch + r;
                    float s = 0.f;
#pragma unroll 4
                    for (int w = 0; w < held; ++w) s += from[w * (kTok * kRedPitch)];
                    return s;
                };
                const int row0 = (first_tile + j0) * 16, width = batch * 16;
                if (kDown || slices > 1) {
                    for (int i = threadIdx.x; i < width * ntok; i += kThreads) {
                        const int tok = i / width, r = i - tok * width, pos = first + done + tok;
                        float* y = kDown ? a.y + (int64_t(slice) * p.tokens * p.top_k + plan.order[pos]) * p.model
                                         : a.h + (int64_t(slice) * p.tokens * p.top_k + pos) * rows;
                        y[row0 + r] = sum(r >> 4, tok, r & 15);
                    }
                } else {
                    for (int i = threadIdx.x; i < width / 2 * ntok; i += kThreads) {
                        const int tok = i / (width / 2), f = i - tok * (width / 2);
                        const float gate = sum(f >> 3, tok, 2 * f & 15), up = sum(f >> 3, tok, (2 * f & 15) + 1);
                        a.h[int64_t(first + done + tok) * p.ffn + row0 / 2 + f] = silu_times(gate, up);
                    }
                }
                buffer ^= 1;
            }
        }
        at += count;
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
                   uint64_t(a.p.experts) * uint64_t(rows), pitch, kBlk, 16, CU_TENSOR_MAP_SWIZZLE_NONE))
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
    const cudaLaunchConfig_t first = launch_config(dim3(unsigned((p.experts + 3) / 4), unsigned((p.tokens + 3) / 4)),
                                                   dim3(128), 0, s, attr);
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
