// Query / key head norms, rotary positions and the key / value cache write in
// one pass over the f32 rows a fused q/k/v projection leaves.
//
// Per token t and head h, with x the head's D values (f32):
//   y = x * rsqrt(mean(x^2) + eps) * w       (query and key heads, if w is given)
//   pair j of the first R values: (a, b) -> (a c - b s, a s + b c) with
//   c = cos_table[p][j], s = sin_table[p][j], p the token's position on the
//   axis that pair j belongs to; pairs are (j, j + R/2) or (2j, 2j + 1).
// Query heads go to q, key and value heads to the cache at slots[t], each
// value rounded once, from f32, to the 16-bit type.
//
// Bound by memory: 4 bytes read and 2 written per value, nothing read twice.
// A group of D/8 lanes (rounded up to 8, 16 or 32) owns one head, 8 values
// per lane, held as the two runs of four that rotate with each other, so a
// head is two float4 loads per lane, one shuffle reduction and no shared
// memory.  A thread keeps its lane's cos / sin in registers over its three
// heads of one token, and issues the loads of all of them before it uses any.
//
// Measured at 8192 tokens x 48 heads x 128 (306 MB): 52.5 us, 5.8 TB/s, 86 % of
// the copy rate.  A CTA waits once for its loads and then only stores, so many
// small ones (two warps, 3 heads per lane group) keep more in flight than fewer
// large ones (256 threads: 69.7 us with 3 heads, 79.1 with 4; 64 threads: 57.9
// with 2, 61.5 with 4), and marking both streams as used once leaves the L2 to
// neither (stores unmarked: 56.0 us).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "half_ops.cuh"
#include "mmq_internal.h"
#include "sm103_ptx.cuh"

namespace {

using namespace mmq::ptx;

constexpr int kThreads = 64;
constexpr int kHeads = 3;   // heads in flight per lane group

struct RopeArgs {
    mmq_qk_norm_rope_t p;
    int end[4];    // first pair past each axis's section
    int axes;
    int* status;
};

template <typename T, int L, bool kInter>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const RopeArgs a) {
    constexpr int kGroups = kThreads / L;
    const mmq_qk_norm_rope_t& p = a.p;
    griddep_launch_dependents();
    griddep_wait();
    const int64_t t = blockIdx.x;
    const int D = p.head_dim, half = p.rot / 2;
    const int e = threadIdx.x % L, g = threadIdx.x / L;
    const int h0 = int(blockIdx.y) * kGroups * kHeads + g;
    const int heads = p.heads + 2 * p.kv_heads;
    const bool mine = 8 * e < D;              // lanes past the head's end only take part in the shuffles
    const bool turns = 8 * e < p.rot;         // this lane's 8 values are four rotated pairs
    const int oa = turns && !kInter ? 4 * e : 8 * e;
    const int ob = turns && !kInter ? half + 4 * e : 8 * e + 4;

    float4 xa[kHeads], xb[kHeads];
    const float* row = p.qkv + t * p.ld;
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        const int h = h0 + i * kGroups;
        xa[i] = xb[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (mine && h < heads) {
            xa[i] = __ldcs(reinterpret_cast<const float4*>(row + int64_t(h) * D + oa));
            xb[i] = __ldcs(reinterpret_cast<const float4*>(row + int64_t(h) * D + ob));
        }
    }

    // The token's positions: a position outside the table reads nothing from
    // it, makes the query rows NaN and leaves the cache alone.
    bool ok = true;
    for (int ax = 0; ax < a.axes; ++ax) {
        const int pos = p.positions[int64_t(ax) * p.tokens + t];
        ok = ok && pos >= 0 && pos < p.table_rows;
    }
    const int64_t slot = p.slots[t];
    const bool fits = slot < p.n_slots;
    if ((!ok || !fits) && threadIdx.x == 0 && blockIdx.y == 0) atomicCAS(a.status, 0, MMQ_ERR_ARG);

    float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
    if (!ok) {
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = s[i] = __int_as_float(0x7FC00000);
    } else if (turns) {
        int ax[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = 4 * e + i;
            ax[i] = (j >= a.end[0]) + (j >= a.end[1]) + (j >= a.end[2]);
        }
        if (ax[0] == ax[3]) {
            const int64_t at = int64_t(p.positions[int64_t(ax[0]) * p.tokens + t]) * half + 4 * e;
            const float4 cv = *reinterpret_cast<const float4*>(p.cos_table + at);
            const float4 sv = *reinterpret_cast<const float4*>(p.sin_table + at);
            c[0] = cv.x; c[1] = cv.y; c[2] = cv.z; c[3] = cv.w;
            s[0] = sv.x; s[1] = sv.y; s[2] = sv.z; s[3] = sv.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t at = int64_t(p.positions[int64_t(ax[i]) * p.tokens + t]) * half + 4 * e + i;
                c[i] = p.cos_table[at];
                s[i] = p.sin_table[at];
            }
        }
    }

#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        const int h = h0 + i * kGroups;
        const bool is_q = h < p.heads, is_v = h >= p.heads + p.kv_heads;
        float x[8] = {xa[i].x, xa[i].y, xa[i].z, xa[i].w, xb[i].x, xb[i].y, xb[i].z, xb[i].w};
        const float* w = is_q ? p.q_weight : p.k_weight;
        float ss = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) ss = fmaf(x[k], x[k], ss);
#pragma unroll
        for (int m = L / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        if (h >= heads || !mine) continue;
        if (!is_v && w) {
            const float r = rsqrtf(ss / float(D) + p.eps);
            const float4 wa = *reinterpret_cast<const float4*>(w + oa);
            const float4 wb = *reinterpret_cast<const float4*>(w + ob);
            x[0] *= r * wa.x; x[1] *= r * wa.y; x[2] *= r * wa.z; x[3] *= r * wa.w;
            x[4] *= r * wb.x; x[5] *= r * wb.y; x[6] *= r * wb.z; x[7] *= r * wb.w;
        }
        if (!is_v && (turns || !ok)) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int ia = kInter ? 2 * k : k, ib = kInter ? 2 * k + 1 : k + 4;
                const float u = x[ia], v = x[ib];
                x[ia] = fmaf(u, c[k], -v * s[k]);
                x[ib] = fmaf(u, s[k], v * c[k]);
            }
        }
        T* out;
        if (is_q) {
            out = static_cast<T*>(p.q) + (t * p.heads + h) * D;
        } else {
            if (!ok || !fits || slot < 0) continue;
            out = static_cast<T*>(is_v ? p.v_cache : p.k_cache) +
                  (slot * p.kv_heads + (h - p.heads - (is_v ? p.kv_heads : 0))) * D;
        }
        T* const tag = nullptr;
        __stcs(reinterpret_cast<uint2*>(out + oa), make_uint2(pack16(x[0], x[1], tag), pack16(x[2], x[3], tag)));
        __stcs(reinterpret_cast<uint2*>(out + ob), make_uint2(pack16(x[4], x[5], tag), pack16(x[6], x[7], tag)));
    }
}

template <typename T, int L>
cudaError_t launch(const RopeArgs& a, cudaStream_t s) {
    const int heads = a.p.heads + 2 * a.p.kv_heads;
    const int per = kThreads / L * kHeads;
    const dim3 grid(unsigned(a.p.tokens), unsigned((heads + per - 1) / per));
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = mmq::launch_config(grid, dim3(kThreads), 0, s, attr);
    return a.p.interleaved ? cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<T, L, true>, a)
                           : cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<T, L, false>, a);
}

template <typename T>
cudaError_t launch_dim(const RopeArgs& a, cudaStream_t s) {
    if (a.p.head_dim <= 64) return launch<T, 8>(a, s);
    if (a.p.head_dim <= 128) return launch<T, 16>(a, s);
    return launch<T, 32>(a, s);
}

}  // namespace

namespace mmq {

cudaError_t launch_qk_norm_rope(const mmq_qk_norm_rope_t& p, int* status, cudaStream_t s) {
    RopeArgs a;
    a.p = p;
    a.status = status;
    a.axes = 0;
    int at = 0;
    for (int i = 0; i < 4; ++i) {
        if (p.sections[i]) a.axes = i + 1;
        a.end[i] = (at += p.sections[i]);
    }
    return p.type == MMQ_TYPE_F16 ? launch_dim<__half>(a, s) : launch_dim<__nv_bfloat16>(a, s);
}

}  // namespace mmq
