// Writing keys and values into the 4-bit cache, and expanding them again.
//
// Per block of 32 values x of a token and head, with m the value of largest
// magnitude (the positive one of two):
//   d = float16(bfloat16(-m / 8)), at most 8160 in magnitude
//   code = clamp(rint(x / d), -8, 7) + 8        (8 where d is zero)
// each rounding to nearest even and the quotient's exactly that of x / d.  A
// block with a NaN or an infinity has d = NaN.
//
// A CTA takes 16 tokens of a head, a thread eight values of one token.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv4.cuh"
#include "mmq_internal.h"
#include "sm103_ptx.cuh"

namespace {

using namespace mmq::ptx;
using namespace mmq::kv4;

struct WriteArgs {
    mmq_kv4_write_t p;
    int page_shift;
    int* status;
};
struct ReadArgs {
    mmq_kv4_read_t p;
    int page_shift;
    int* status;
};

// Tile and place in it of a slot of head h.
template <int D, typename Byte>
__device__ __forceinline__ Byte* tile_of(Byte* cache, int64_t slot, int h, int kv_heads, int page_shift) {
    const int64_t page = slot >> page_shift;
    const int64_t tile = (slot & ((int64_t(1) << page_shift) - 1)) >> 4;
    return cache + (((page * kv_heads + h) << (page_shift - 4)) + tile) * tile_bytes(D);
}

// ------------------------------------------------------------------- write
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    float d;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

template <typename T>
__device__ __forceinline__ void load8(const void* base, int64_t at, float (&x)[8]);
template <>
__device__ __forceinline__ void load8<float>(const void* base, int64_t at, float (&x)[8]) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    const float4 a = p[0], b = p[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__half>(const void* base, int64_t at, float (&x)[8]) {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const __half*>(base) + at);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
        x[2 * k] = f.x;
        x[2 * k + 1] = f.y;
    }
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const void* base, int64_t at, float (&x)[8]) {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + at);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        x[2 * k] = __uint_as_float(w[k] << 16);
        x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    }
}

// The scale of a block whose values four neighbouring lanes hold, and this
// lane's eight codes, one per nibble (value k in bits 4k).
__device__ __forceinline__ uint32_t quantize(const float (&x)[8], __half& scale) {
    float most = x[0], least = x[0];
#pragma unroll
    for (int k = 1; k < 8; ++k) {
        most = max_nan(most, x[k]);
        least = min_nan(least, x[k]);
    }
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
        most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, d));
        least = min_nan(least, __shfl_xor_sync(0xffffffffu, least, d));
    }
    const float top = most >= -least ? most : least;   // NaN: least, which is NaN too
    float d = __bfloat162float(__float2bfloat16_rn(__fmul_rn(top, -0.125f)));
    if (fabsf(d) > kTop) d = copysignf(kTop, d);
    if (!(fabsf(top) <= 3.402823466e38f)) d = __int_as_float(0x7FC00000);
    scale = __float2half_rn(d);
    d = __half2float(scale);
    const float inverse = d == 0.f ? 0.f : 1.f / d;
    uint32_t codes = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        // within one of the quotient; then the exact remainder decides, ties to even
        float n = rintf(fminf(fmaxf(x[k] * inverse, -8.f), 7.f));
        const float rest = fmaf(-n, d, x[k]), twice = 2.f * fabsf(rest);
        const bool odd = int(n) & 1;
        if (twice > fabsf(d) || (twice == fabsf(d) && odd)) n += (rest < 0.f) == (d < 0.f) ? 1.f : -1.f;
        n = fminf(fmaxf(n, -8.f), 7.f);
        if (d == 0.f || d != d) n = 0.f;
        codes |= uint32_t(int(n) + 8) << (4 * k);
    }
    return codes;
}

// Bytes x = 0..3 (even lanes) or 4..7 (odd lanes) of the 16 dimensions that
// lanes 2 i and 2 i + 1 hold: the even lane's codes low, the odd lane's high.
__device__ __forceinline__ uint32_t pair_bytes(uint32_t codes, bool odd) {
    const uint32_t other = __shfl_xor_sync(0xffffffffu, codes, 1);
    const uint32_t lo = odd ? other >> 16 : codes & 0xFFFFu, hi = odd ? codes >> 16 : other & 0xFFFFu;
    uint32_t w = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) w |= (((lo >> (4 * k)) & 15u) | (((hi >> (4 * k)) & 15u) << 4)) << (8 * k);
    return w;
}

template <typename T, int D>
__global__ void __launch_bounds__(2 * D) kv4_write_kernel(const WriteArgs a) {
    __shared__ __align__(16) uint8_t tile[tile_bytes(D)];
    __shared__ int64_t first;   // slot of the group's first token
    const mmq_kv4_write_t& p = a.p;
    griddep_launch_dependents();
    griddep_wait();
    constexpr int kLanes = D / 8;   // threads per token
    // Groups of 16 start where the first token's tile does, so that the tokens
    // of one long chunk fill whole tiles.
    const int shift = p.slots[0] < 0 ? 0 : p.slots[0] & 15;
    const int i16 = threadIdx.x / kLanes, e = threadIdx.x % kLanes;
    const int64_t t = int64_t(blockIdx.x) * kTokens - shift + i16;
    const int h = blockIdx.y;
    const bool here = t >= 0 && t < p.tokens;
    const int64_t slot = here ? p.slots[t] : -1;
    const bool good = slot >= 0 && slot < p.n_slots;
    if (slot >= p.n_slots && e == 0 && h == 0) atomicCAS(a.status, 0, MMQ_ERR_ARG);
    float k[8] = {}, v[8] = {};
    if (good) {
        load8<T>(p.k, t * p.k_token_stride + h * p.k_head_stride + 8 * e, k);
        load8<T>(p.v, t * p.v_token_stride + h * p.v_head_stride + 8 * e, v);
    }
    __half ks, vs;
    const bool odd = e & 1;
    const uint32_t kb = pair_bytes(quantize(k, ks), odd), vb = pair_bytes(quantize(v, vs), odd);
    // All 16 tokens of one tile, in order: the tile is put together first.
    if (threadIdx.x == 0) first = slot;
    __syncthreads();
    const bool whole = __syncthreads_and(good && (first & 15) == 0 && slot == first + i16);
    uint8_t* const dst = whole ? tile : good ? tile_of<D>(p.cache, slot, h, p.kv_heads, a.page_shift) : nullptr;
    if (whole || good) {
        const int place = int(slot & 15);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int x = n + (odd ? 4 : 0);
            dst[key_byte(place, e >> 1, x)] = uint8_t(kb >> (8 * n));
            dst[value_byte<D>(place, e >> 1, x)] = uint8_t(vb >> (8 * n));
        }
        if ((e & 3) == 0) {
            *reinterpret_cast<__half*>(dst + key_scale<D>(place, e >> 2)) = ks;
            *reinterpret_cast<__half*>(dst + value_scale<D>(place, e >> 2)) = vs;
        }
    }
    if (!whole) return;
    __syncthreads();
    if (threadIdx.x < tile_bytes(D) / 16) {
        const uint4 w = reinterpret_cast<const uint4*>(tile)[threadIdx.x];
        reinterpret_cast<uint4*>(tile_of<D>(p.cache, slot, h, p.kv_heads, a.page_shift))[threadIdx.x] = w;
    }
}

// -------------------------------------------------------------------- read
__device__ __forceinline__ void store2(__half* at, float x, float y) { *reinterpret_cast<__half2*>(at) = __floats2half2_rn(x, y); }
__device__ __forceinline__ void store2(__nv_bfloat16* at, float x, float y) {
    *reinterpret_cast<__nv_bfloat162*>(at) = __floats2bfloat162_rn(x, y);
}
__device__ __forceinline__ void store2(float* at, float x, float y) { *reinterpret_cast<float2*>(at) = make_float2(x, y); }

template <typename T, int D>
__global__ void __launch_bounds__(2 * D) kv4_read_kernel(const ReadArgs a) {
    const mmq_kv4_read_t& p = a.p;
    griddep_launch_dependents();
    griddep_wait();
    constexpr int kLanes = D / 8;
    const int e = threadIdx.x % kLanes, h = blockIdx.y;
    const int64_t t = int64_t(blockIdx.x) * kTokens + threadIdx.x / kLanes;
    if (t >= p.tokens) return;
    const int64_t slot = p.slots[t];
    const bool good = slot >= 0 && slot < p.n_slots;
    if (slot >= p.n_slots && e == 0 && h == 0) atomicCAS(a.status, 0, MMQ_ERR_ARG);
    float k[8] = {}, v[8] = {};
    if (good) {
        const uint8_t* src = tile_of<D>(p.cache, slot, h, p.kv_heads, a.page_shift);
        const int place = int(slot & 15), nibble = 4 * (e & 1);
        const float ks = __half2float(*reinterpret_cast<const __half*>(src + key_scale<D>(place, e >> 2)));
        const float vs = __half2float(*reinterpret_cast<const __half*>(src + value_scale<D>(place, e >> 2)));
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            k[x] = float(int((src[key_byte(place, e >> 1, x)] >> nibble) & 15) - 8) * ks;
            v[x] = float(int((src[value_byte<D>(place, e >> 1, x)] >> nibble) & 15) - 8) * vs;
        }
    }
    const int64_t at = (t * p.kv_heads + h) * D + 8 * e;
#pragma unroll
    for (int x = 0; x < 8; x += 2) {
        store2(static_cast<T*>(p.k) + at + x, k[x], k[x + 1]);
        store2(static_cast<T*>(p.v) + at + x, v[x], v[x + 1]);
    }
}

int shift_of(int page_size) {
    int s = 0;
    while ((1 << s) < page_size) ++s;
    return s;
}

template <typename T, int D>
cudaError_t write(const WriteArgs& a, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    // one group more than the tokens fill: the first may hold as little as one token
    const dim3 grid(unsigned((a.p.tokens + 15 + kTokens - 1) / kTokens), unsigned(a.p.kv_heads));
    const cudaLaunchConfig_t cfg = mmq::launch_config(grid, dim3(2 * D), 0, s, attr);
    return cudaLaunchKernelEx(&cfg, kv4_write_kernel<T, D>, a);
}
template <typename T, int D>
cudaError_t read(const ReadArgs& a, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    const dim3 grid(unsigned((a.p.tokens + kTokens - 1) / kTokens), unsigned(a.p.kv_heads));
    const cudaLaunchConfig_t cfg = mmq::launch_config(grid, dim3(2 * D), 0, s, attr);
    return cudaLaunchKernelEx(&cfg, kv4_read_kernel<T, D>, a);
}

}  // namespace

namespace mmq {

cudaError_t launch_kv4_write(const mmq_kv4_write_t& p, int* status, cudaStream_t s) {
    const WriteArgs a{p, shift_of(p.page_size), status};
    const bool wide = p.head_dim == 128;
    switch (p.type) {
        case MMQ_TYPE_F16: return wide ? write<__half, 128>(a, s) : write<__half, 64>(a, s);
        case MMQ_TYPE_BF16: return wide ? write<__nv_bfloat16, 128>(a, s) : write<__nv_bfloat16, 64>(a, s);
        default: return wide ? write<float, 128>(a, s) : write<float, 64>(a, s);
    }
}

cudaError_t launch_kv4_read(const mmq_kv4_read_t& p, int* status, cudaStream_t s) {
    const ReadArgs a{p, shift_of(p.page_size), status};
    const bool wide = p.head_dim == 128;
    switch (p.type) {
        case MMQ_TYPE_F16: return wide ? read<__half, 128>(a, s) : read<__half, 64>(a, s);
        case MMQ_TYPE_BF16: return wide ? read<__nv_bfloat16, 128>(a, s) : read<__nv_bfloat16, 64>(a, s);
        default: return wide ? read<float, 128>(a, s) : read<float, 64>(a, s);
    }
}

}  // namespace mmq
