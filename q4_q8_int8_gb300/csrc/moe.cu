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
constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kBlk = 144;     // bytes of a q4_K super-block
constexpr int kStages = 4;    // super-blocks per row in flight per warp

// One (super-block, group of four tokens) of activations in shared memory, in
// the order the matrix instructions take them: 8 steps x 32 lanes x 16 bytes,
// then the sub-block sums, 32 lanes x 4 bytes, then the four tokens' 2^e.
constexpr int kAct = 8 * 512 + 128 + 16;

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
    Plan* plan;
    float* h;        // [pairs][ffn], rows in the plan's order
    float* y;        // [slices][pairs][model], rows by pair
    int slices;      // parts of the down product's sum over ffn
    int act_sb;      // super-blocks of activations held at once
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

// Fill `plan` (shared memory) from the logits; block 0 also stores it, the
// chosen experts and their weights.  scratch: kMaxPairs + 2 * kWarps ints.
__device__ void make_plan(const MoeArgs& a, Plan* plan, int* scratch) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int* ids = scratch;
    int* totals = scratch + kMaxPairs;
    for (int t = warp; t < a.p.tokens; t += kWarps) choose(a, t, lane, ids, blockIdx.x == 0);
    __syncthreads();
    static_assert(kMaxExperts == kThreads, "one thread per expert");
    const int e = threadIdx.x, pairs = a.p.tokens * a.p.top_k;
    int n = 0;
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
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma1688(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(b0));
}
__device__ __forceinline__ uint32_t h2u(__half2 v) { return *reinterpret_cast<const uint32_t*>(&v); }
__device__ __forceinline__ __half2 u2h(uint32_t v) { return *reinterpret_cast<const __half2*>(&v); }

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

// One warp: 256 f32 activations of one token into column pair `tok` (0..3) of
// one activation block at shared address `blk`.
__device__ __forceinline__ void put_act(const float* x, uint32_t blk, int tok, int lane) {
    const float4 v[2] = {reinterpret_cast<const float4*>(x)[lane], reinterpret_cast<const float4*>(x)[lane + 32]};
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        top = fmaxf(fmaxf(top, fmaxf(fabsf(v[i].x), fabsf(v[i].y))), fmaxf(fabsf(v[i].z), fabsf(v[i].w)));
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
    // 2^e with top 2^-e in [128, 256), e from -126 on
    int e = int(__float_as_uint(top) >> 23) - 127 - 7;
    e = e < -126 ? -126 : e;
    const float up = __uint_as_float(uint32_t(127 + e) << 23), down = __uint_as_float(uint32_t(127 - e) << 23);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int quad = lane + 32 * i, sub = quad >> 3, w = quad & 7;
        const float f[4] = {v[i].x * down, v[i].y * down, v[i].z * down, v[i].w * down};
        __half hi[4], lo[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            hi[k] = __float2half_rn(f[k]);
            lo[k] = __float2half_rn(f[k] - __half2float(hi[k]));
        }
        const uint32_t at = blk + uint32_t(((w * 8 + 2 * tok) * 4 + (sub >> 1)) * 16 + (sub & 1) * 8);
        const uint32_t h0 = h2u(__halves2half2(hi[0], hi[2])), h1 = h2u(__halves2half2(hi[1], hi[3]));
        const uint32_t l0 = h2u(__halves2half2(lo[0], lo[2])), l1 = h2u(__halves2half2(lo[1], lo[3]));
        asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(h0), "r"(h1) : "memory");
        asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at + 64u), "r"(l0), "r"(l1) : "memory");
        float s = (f[0] + f[1]) + (f[2] + f[3]);
        s += __shfl_xor_sync(0xffffffffu, s, 1);
        s += __shfl_xor_sync(0xffffffffu, s, 2);
        s += __shfl_xor_sync(0xffffffffu, s, 4);
        if (w == 0) {
            const __half sh = __float2half_rn(s), sl = __float2half_rn(s - __half2float(sh));
            const uint32_t xa = blk + 4096u + uint32_t((2 * tok * 4 + (sub >> 1)) * 4 + (sub & 1) * 2);
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(xa), "h"(__half_as_ushort(sh)) : "memory");
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(xa + 16u), "h"(__half_as_ushort(sl)) : "memory");
        }
    }
    if (lane == 0) asm volatile("st.shared.f32 [%0], %1;" ::"r"(blk + 4224u + 4u * uint32_t(tok)), "f"(up) : "memory");
}

__host__ __device__ constexpr int act_bytes(int sb, int ng) { return sb * ng * kAct; }
__host__ __device__ constexpr int ring_bytes(int mt) { return kWarps * kStages * 16 * mt * kBlk; }
__host__ __device__ constexpr int red_pitch(int mt) { return 16 * mt + 4; }
__host__ __device__ constexpr int red_bytes(int ng, int mt) { return kWarps * 4 * ng * red_pitch(mt) * 4; }

// Both products of the experts.  A CTA walks items, (active expert, slice of
// the sum, block of rows), consecutive ones so that the activations it holds
// in shared memory change rarely; a team of KS warps owns 16 MT rows of an
// item, its warps taking every KS-th super-block, and 4 NG tokens at a time.
// Each warp streams its rows' super-blocks through its own cp.async ring,
// which runs on over the items.
template <int NG, int MT, int KS, bool kDown>
__global__ void __launch_bounds__(kThreads) moe_expert_kernel(const MoeArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ Plan plan;
    __shared__ int scratch[kMaxPairs + 2 * kWarps];
    const mmq_q4K_moe_t& p = a.p;
    griddep_launch_dependents();
    griddep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int ks = warp % KS, team = warp / KS;
    constexpr int kRows = 16 * MT, kBlockRows = kRows * (kWarps / KS), kTok = 4 * NG;

    if (!kDown) {
        make_plan(a, &plan, scratch);
        if (blockIdx.x == 0)
            for (int i = threadIdx.x; i < int(sizeof(Plan) / 4); i += kThreads)
                reinterpret_cast<int*>(a.plan)[i] = reinterpret_cast<const int*>(&plan)[i];
    } else {
        for (int i = threadIdx.x; i < int(sizeof(Plan) / 4); i += kThreads)
            reinterpret_cast<int*>(&plan)[i] = reinterpret_cast<const int*>(a.plan)[i];
        __syncthreads();
    }

    const int rows = kDown ? p.model : 2 * p.ffn, inner = kDown ? p.ffn : p.model;
    const int nsb = inner / 256;
    const int64_t pitch = int64_t(nsb) * kBlk;
    const uint8_t* const weights = kDown ? p.w_down : p.w_gu;
    const int blocks = (rows + kBlockRows - 1) / kBlockRows;
    const int slices = kDown ? a.slices : 1;
    const int per = (nsb + slices - 1) / slices;
    const int64_t items = int64_t(plan.active) * slices * blocks;
    const int64_t i0 = items * blockIdx.x / gridDim.x, i1 = items * (blockIdx.x + 1) / gridDim.x;

    const uint32_t act = smem_u32(smem);
    const uint32_t ring = act + uint32_t(act_bytes(a.act_sb, NG)) + uint32_t(warp * kStages * kRows * kBlk);
    float* const red = reinterpret_cast<float*>(smem + act_bytes(a.act_sb, NG) + ring_bytes(MT));

    // A position in this warp's stream: item, pass over its tokens, super-block.
    struct At {
        int64_t item;
        int pass, passes, sb, sb0, sb1;
        const uint8_t* row;   // the team's first row
    };
    auto enter = [&](At& s) {   // item s.item, pass 0
        const int64_t q = s.item / blocks;
        const int act_i = int(q / slices), slice = int(q % slices), block = int(s.item % blocks);
        const int n = plan.start[act_i + 1] - plan.start[act_i];
        s.pass = 0;
        s.passes = (n + kTok - 1) / kTok;
        s.sb0 = slice * per;
        s.sb1 = min(nsb, s.sb0 + per);
        s.sb = s.sb0 + ks;
        s.row = weights + (int64_t(plan.expert[act_i]) * rows + int64_t(block) * kBlockRows + team * kRows) * pitch;
    };
    // Skips to the next position with a super-block for this warp.
    auto settle = [&](At& s) {
        while (s.item < i1 && s.sb >= s.sb1) {
            s.sb = s.sb0 + ks;
            if (++s.pass >= s.passes) {
                if (++s.item < i1) enter(s);
            } else if (s.sb >= s.sb1) {
                s.pass = s.passes;   // this warp has none in this slice
            }
        }
    };
    At in = {i0, 0, 0, 0, 0, 0, nullptr};
    if (i0 < i1) {
        enter(in);
        settle(in);
    }
    int in_stage = 0, out_stage = 0;
    auto issue = [&]() {
        if (in.item < i1) {
            const int left = rows - (int(in.item % blocks) * kBlockRows + team * kRows);
            const uint8_t* src = in.row + int64_t(in.sb) * kBlk;
            const uint32_t dst = ring + uint32_t(in_stage * kRows * kBlk);
#pragma unroll
            for (int j = 0; j < (kRows * 9 + 31) / 32; ++j) {
                const int c = lane + 32 * j, r = c / 9, o = (c - r * 9) * 16;
                if (c < kRows * 9 && r < left) cp_async16(dst + uint32_t(r * kBlk + o), src + r * pitch + o);
            }
            in.sb += KS;
            settle(in);
        }
        cp_async_commit();
        if (++in_stage == kStages) in_stage = 0;
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue();

    int64_t held = -1;   // which activations shared memory holds
    for (int64_t item = i0; item < i1; ++item) {
        const int64_t q = item / blocks;
        const int act_i = int(q / slices), slice = int(q % slices), block = int(item % blocks);
        const int first = plan.start[act_i], n = plan.start[act_i + 1] - first;
        const int sb0 = slice * per, sb1 = min(nsb, sb0 + per);
        const int row0 = block * kBlockRows + team * kRows;
        for (int pass = 0; pass * kTok < n; ++pass) {
            const int ntok = min(kTok, n - pass * kTok), ng = (ntok + 3) / 4;
            float tot[MT][NG][2];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int j = 0; j < NG; ++j) tot[m][j][0] = tot[m][j][1] = 0.f;
            for (int part = sb0; part < sb1; part += a.act_sb) {
                const int end = min(sb1, part + a.act_sb);
                // one token's activations are the same for every expert of the first product
                const int64_t want = (((!kDown && p.tokens == 1) ? 0 : int64_t(act_i)) * (kMaxPairs + 1) + pass) * (int64_t(nsb) + 1) + part;
                if (want != held) {
                    __syncthreads();
                    const int count = (end - part) * ntok;
                    for (int i = warp; i < count; i += kWarps) {
                        const int sb = part + i / ntok, j = i % ntok;
                        const int pos = first + pass * kTok + j;
                        const float* x = kDown ? a.h + int64_t(pos) * p.ffn
                                               : p.x + int64_t(plan.order[pos] / p.top_k) * p.model;
                        put_act(x + sb * 256, act + uint32_t(((sb - part) * NG + j / 4) * kAct), j & 3, lane);
                    }
                    held = want;
                    __syncthreads();
                }
                for (int sb = part + (((ks - (part - sb0)) % KS) + KS) % KS; sb < end; sb += KS) {
                    cp_async_wait<kStages - 2>();
                    __syncwarp();
                    issue();   // into the stage before this one, which every lane has read
                    const uint32_t st = ring + uint32_t(out_stage * kRows * kBlk);
                    const uint32_t ab = act + uint32_t((sb - part) * NG * kAct);
                    if (++out_stage == kStages) out_stage = 0;
                    float acc[MT][NG][4];
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int j = 0; j < NG; ++j)
#pragma unroll
                            for (int k = 0; k < 4; ++k) acc[m][j][k] = 0.f;
                    RowScale r0[MT], r1[MT];
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        r0[m] = row_scale(lds128(st + uint32_t((16 * m + g) * kBlk)), t);
                        r1[m] = row_scale(lds128(st + uint32_t((16 * m + g + 8) * kBlk)), t);
                    }
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t w0[MT][4], w1[MT][4];
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            const uint4 u = lds128(st + uint32_t((16 * m + g) * kBlk + 16 + 32 * t + 16 * half));
                            const uint4 v = lds128(st + uint32_t((16 * m + g + 8) * kBlk + 16 + 32 * t + 16 * half));
                            w0[m][0] = u.x; w0[m][1] = u.y; w0[m][2] = u.z; w0[m][3] = u.w;
                            w1[m][0] = v.x; w1[m][1] = v.y; w1[m][2] = v.z; w1[m][3] = v.w;
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t lo[MT][4], hi[MT][4];
#pragma unroll
                            for (int m = 0; m < MT; ++m) {
                                unpack_lo(w0[m][i], r0[m], lo[m][0], lo[m][2]);
                                unpack_lo(w1[m][i], r1[m], lo[m][1], lo[m][3]);
                                unpack_hi(w0[m][i], r0[m], hi[m][0], hi[m][2]);
                                unpack_hi(w1[m][i], r1[m], hi[m][1], hi[m][3]);
                            }
#pragma unroll
                            for (int j = 0; j < NG; ++j) {
                                if (j < ng) {
                                    const uint4 b = lds128(ab + uint32_t(j * kAct + (4 * half + i) * 512 + lane * 16));
#pragma unroll
                                    for (int m = 0; m < MT; ++m) {
                                        mma16816(acc[m][j], lo[m], b.x, b.y);
                                        mma16816(acc[m][j], hi[m], b.z, b.w);
                                    }
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int j = 0; j < NG; ++j) {
                        if (j < ng) {
                            const uint32_t xs = lds32(ab + uint32_t(j * kAct + 4096 + lane * 4));
                            const float up = __uint_as_float(lds32(ab + uint32_t(j * kAct + 4224 + t * 4)));
#pragma unroll
                            for (int m = 0; m < MT; ++m) {
                                float mn[4] = {0.f, 0.f, 0.f, 0.f};
                                mma1688(mn, r0[m].m, r1[m].m, xs);
                                const float* s = acc[m][j];
                                tot[m][j][0] = fmaf(up, r0[m].d * (s[0] + s[1]) - r0[m].dmin * (mn[0] + mn[1]), tot[m][j][0]);
                                tot[m][j][1] = fmaf(up, r1[m].d * (s[2] + s[3]) - r1[m].dmin * (mn[2] + mn[3]), tot[m][j][1]);
                            }
                        }
                    }
                }
            }
            // Join the team's warps (in their order) and store.
            float* mine = red + warp * kTok * red_pitch(MT);
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int j = 0; j < NG; ++j) {
                    mine[(4 * j + t) * red_pitch(MT) + 16 * m + g] = tot[m][j][0];
                    mine[(4 * j + t) * red_pitch(MT) + 16 * m + g + 8] = tot[m][j][1];
                }
            if (KS == 1) __syncwarp(); else __syncthreads();
            const float* base = red + team * KS * kTok * red_pitch(MT);
            auto sum = [&](int tok, int r) {
                float s = base[tok * red_pitch(MT) + r];
#pragma unroll
                for (int w = 1; w < KS; ++w) s += base[(w * kTok + tok) * red_pitch(MT) + r];
                return s;
            };
            const int me = ks * 32 + lane;
            if (kDown) {
                for (int i = me; i < kRows * ntok; i += KS * 32) {
                    const int tok = i / kRows, r = i % kRows;
                    const int pair = plan.order[first + pass * kTok + tok];
                    if (row0 + r < rows)
                        a.y[(int64_t(slice) * p.tokens * p.top_k + pair) * p.model + row0 + r] = sum(tok, r);
                }
            } else {
                for (int i = me; i < kRows / 2 * ntok; i += KS * 32) {
                    const int tok = i / (kRows / 2), f = i % (kRows / 2);
                    if (row0 + 2 * f < rows) {
                        const float gate = sum(tok, 2 * f), up = sum(tok, 2 * f + 1);
                        a.h[int64_t(first + pass * kTok + tok) * p.ffn + row0 / 2 + f] = gate / (1.f + expf(-gate)) * up;
                    }
                }
            }
            if (KS == 1) __syncwarp(); else __syncthreads();
        }
    }
    cp_async_wait<0>();
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
        for (int i = 0; i < a.slices; ++i) {
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

struct Sizes {
    size_t logits, plan, h, y, bytes;
    int slices;
};
Sizes sizes(const mmq_q4K_moe_t& p) {
    auto up = [](size_t b) { return (b + 255) & ~size_t(255); };
    Sizes z;
    const size_t pairs = size_t(p.tokens) * size_t(p.top_k);
    z.slices = 1;
    z.logits = 0;
    z.plan = z.logits + up(size_t(p.tokens) * size_t(p.experts) * 4);
    z.h = z.plan + up(sizeof(Plan));
    z.y = z.h + up(pairs * size_t(p.ffn) * 4);
    z.bytes = z.y + size_t(z.slices) * pairs * size_t(p.model) * 4;
    return z;
}

template <int NG, int MT, int KS, bool kDown>
cudaError_t launch_expert(MoeArgs a, int nsm, cudaStream_t s) {
    const int nsb = (kDown ? a.p.ffn : a.p.model) / 256;
    a.act_sb = nsb < 16 ? nsb : 16;
    const int smem = act_bytes(a.act_sb, NG) + ring_bytes(MT) + red_bytes(NG, MT);
    cudaError_t e;
    int resident = 0;
    if ((e = cudaFuncSetAttribute(moe_expert_kernel<NG, MT, KS, kDown>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) ||
        (e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&resident, moe_expert_kernel<NG, MT, KS, kDown>, kThreads, smem)))
        return e;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = follow_config(dim3(unsigned(nsm * (resident > 0 ? resident : 1))), dim3(kThreads), smem, s, attr);
    return cudaLaunchKernelEx(&cfg, moe_expert_kernel<NG, MT, KS, kDown>, a);
}

}  // namespace

namespace mmq {

size_t q4K_moe_workspace(const mmq_q4K_moe_t& p) { return sizes(p).bytes; }

cudaError_t launch_q4K_moe(const mmq_q4K_moe_t& p, void* workspace, cudaStream_t s) {
    int dev = 0, nsm = 0;
    cudaError_t e;
    if ((e = cudaGetDevice(&dev)) || (e = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev))) return e;
    const Sizes z = sizes(p);
    char* ws = static_cast<char*>(workspace);
    MoeArgs a;
    a.p = p;
    a.logits = reinterpret_cast<float*>(ws + z.logits);
    a.plan = reinterpret_cast<Plan*>(ws + z.plan);
    a.h = reinterpret_cast<float*>(ws + z.h);
    a.y = reinterpret_cast<float*>(ws + z.y);
    a.slices = z.slices;
    a.act_sb = 0;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t first = launch_config(dim3(unsigned((p.experts + 3) / 4), unsigned((p.tokens + 3) / 4)),
                                                   dim3(128), 0, s, attr);
    if ((e = cudaLaunchKernelEx(&first, moe_router_kernel, a))) return e;
    if ((e = launch_expert<1, 1, 8, false>(a, nsm, s))) return e;
    if ((e = launch_expert<1, 1, 8, true>(a, nsm, s))) return e;
    cudaLaunchAttribute last_attr[1];
    const cudaLaunchConfig_t last = follow_config(dim3(unsigned((p.model / 4 + 127) / 128), unsigned(p.tokens)), dim3(128), 0, s, last_attr);
    return cudaLaunchKernelEx(&last, moe_combine_kernel, a);
}

}  // namespace mmq
