// Writing keys and values into the 4-bit cache, and expanding them again.
//
// Per block of 32 values x of a token and head, with m the value of largest
// magnitude (the positive one of two):
//   d = float16(bfloat16(-m / 8)), at most 8160 in magnitude
//   code = clamp(rint(x / d), -8, 7) + 8        (8 where d is zero)
// each rounding to nearest even and the quotient's exactly that of x / d.  A
// block with a NaN or an infinity has d = NaN.
//
// A warp takes 16 tokens of a head (of two, for D = 64), keys or values: a lane
// what its words of the tile hold, so that it puts whole words together, and
// 32 bytes of a token at a time are one lane's.  Tokens whose tile is not all
// theirs, in order, go byte by byte.
//
// Bound: memory.  32k tokens of 8 heads, D = 128, pages in any order: written
// from float16 in 31 us, read to float16 in 30 us, 5.5 and 5.8 TB/s, 81 and 85 %
// of a copy's rate.  (A thread with eight values of one token, bytes put
// together in shared memory: 45 us for 8192 tokens written and read, now 23,
// and 61 us for the 32k read.)  Few tokens: 3 us, the launch.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

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
    bool aligned;   // k and v to 32 bytes
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

// The lanes of a tile: D / 4 of them, lane 4 i + c with dimensions 16 i to
// 16 i + 15 of the keys of tokens c, c + 4, c + 8, c + 12 and of the values of
// tokens 2 c, 2 c + 1, 2 c + 8, 2 c + 9.  These are 32 contiguous bytes of 16-bit
// values each and all that the lane's eight words of key codes and eight of
// value codes hold.
__device__ __forceinline__ int key_token(int c, int k) { return c + 4 * k; }
__device__ __forceinline__ int value_token(int c, int k) { return 2 * c + (k & 1) + 8 * (k >> 1); }

constexpr int kThreads = 128;

// A lane's place: item (16 tokens of a head, heads fastest) and the token that
// group 0 starts with, at most 0: groups start where the first token's tile
// does, so that the tokens of one long chunk fill whole tiles.
template <int D>
struct Lane {
    static constexpr int kLanes = D / 4;
    int i, c, h;
    int64_t t0;
    __device__ __forceinline__ Lane(const int32_t* slots, int64_t tokens, int kv_heads) {
        const uint32_t item = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;   // below 2^31 and a block's
        i = threadIdx.x % kLanes >> 2;
        c = threadIdx.x & 3;
        h = int(item % uint32_t(kv_heads));
        const int first = slots[0];
        t0 = int64_t(item / uint32_t(kv_heads)) * kTokens - (first < 0 ? 0 : first & 15);
    }
};

// The slot of a token: lane l of the first 16 of an item's holds that of token
// l.  whole: all the warp's items are a tile each, in order.
template <int D>
struct Slots {
    int mine, first;
    bool whole;
    template <typename P>
    __device__ __forceinline__ Slots(const P& p, const Lane<D>& lane, int* status) {
        const int l = threadIdx.x & 15;
        const int64_t t = lane.t0 + l;
        mine = t >= 0 && t < p.tokens ? p.slots[t] : -1;
        if (mine >= p.n_slots) {
            if (lane.h == 0 && blockIdx.y == 0) atomicCAS(status, 0, MMQ_ERR_ARG);
            mine = -1;
        }
        first = __shfl_sync(0xffffffffu, mine, 0, Lane<D>::kLanes);
        whole = __all_sync(0xffffffffu, mine >= 0 && (first & 15) == 0 && mine == first + l);
    }
    __device__ __forceinline__ int of(int l) const { return __shfl_sync(0xffffffffu, mine, l, Lane<D>::kLanes); }
};

// Sixteen values of a token, and what the block's scale needs of them.
template <typename T>
struct Values;
template <typename T>
struct Values16 {
    uint4 u[2];
    __device__ __forceinline__ void load(const void* base, int64_t at, bool here) {
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(base) + at);
#pragma unroll
        for (int k = 0; k < 2; ++k) u[k] = here ? src[k] : make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ uint32_t word(int k) const {
        const uint4& v = u[k >> 2];
        return (k & 3) == 0 ? v.x : (k & 3) == 1 ? v.y : (k & 3) == 2 ? v.z : v.w;
    }
};
template <>
struct Values<__half> : Values16<__half> {
    __device__ __forceinline__ float get(int k) const {
        const uint32_t w = word(k >> 1);
        const __half2 h = *reinterpret_cast<const __half2*>(&w);
        return k & 1 ? __high2float(h) : __low2float(h);
    }
    __device__ __forceinline__ void ends(float& most, float& least) const {
        uint32_t w = word(0);
        __half2 a = *reinterpret_cast<__half2*>(&w), b = a;
#pragma unroll
        for (int k = 1; k < 8; ++k) {
            w = word(k);
            a = __hmax2_nan(a, *reinterpret_cast<__half2*>(&w));
            b = __hmin2_nan(b, *reinterpret_cast<__half2*>(&w));
        }
        most = max_nan(__low2float(a), __high2float(a));
        least = min_nan(__low2float(b), __high2float(b));
    }
};
template <>
struct Values<__nv_bfloat16> : Values16<__nv_bfloat16> {
    __device__ __forceinline__ float get(int k) const {
        return __uint_as_float(k & 1 ? word(k >> 1) & 0xFFFF0000u : word(k >> 1) << 16);
    }
    __device__ __forceinline__ void ends(float& most, float& least) const {
        uint32_t w = word(0);
        __nv_bfloat162 a = *reinterpret_cast<__nv_bfloat162*>(&w), b = a;
#pragma unroll
        for (int k = 1; k < 8; ++k) {
            w = word(k);
            a = __hmax2_nan(a, *reinterpret_cast<__nv_bfloat162*>(&w));
            b = __hmin2_nan(b, *reinterpret_cast<__nv_bfloat162*>(&w));
        }
        most = max_nan(__low2float(a), __high2float(a));
        least = min_nan(__low2float(b), __high2float(b));
    }
};
template <>
struct Values<float> {
    float4 f[4];
    __device__ __forceinline__ void load(const void* base, int64_t at, bool here) {
        const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
#pragma unroll
        for (int k = 0; k < 4; ++k) f[k] = here ? src[k] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __device__ __forceinline__ float get(int k) const {
        const float4& v = f[k >> 2];
        return (k & 3) == 0 ? v.x : (k & 3) == 1 ? v.y : (k & 3) == 2 ? v.z : v.w;
    }
    __device__ __forceinline__ void ends(float& most, float& least) const {
        most = least = get(0);
#pragma unroll
        for (int k = 1; k < 16; ++k) {
            most = max_nan(most, get(k));
            least = min_nan(least, get(k));
        }
    }
};

// code - 8 of x / d as bits whose lowest four are the code and whose others,
// up to the 22nd, are zero.
//
// 16-bit types: a quotient that is no tie (an odd multiple of 1/2) is at least
// 2^-12 from one, x having at most 11 bits, d at most 8, and |x| >= |d| / 2
// there.  x times the rounded 1 / d is off by at most 12.5 * 2^-24.  So the
// product rounded to multiples of 2^-14, which adding 768 does, is the tie where
// the quotient is one and on its side of it where not, and the second sum rounds
// it to an integer, ties to even.
template <typename T>
__device__ __forceinline__ uint32_t code_of(float x, float d, float inverse) {
    const float t = fminf(fmaxf(fmaf(x, inverse, 768.f), 760.f), 775.f);
    return __float_as_uint(t + (12582912.f + 8.f - 768.f));
}
// float: within one of the quotient; then the exact remainder decides.
template <>
__device__ __forceinline__ uint32_t code_of<float>(float x, float d, float inverse) {
    float n = rintf(fminf(fmaxf(x * inverse, -8.f), 7.f));
    const float rest = fmaf(-n, d, x), twice = 2.f * fabsf(rest);
    const bool odd = int(n) & 1;
    if (twice > fabsf(d) || (twice == fabsf(d) && odd)) n += (rest < 0.f) == (d < 0.f) ? 1.f : -1.f;
    return uint32_t(int(fminf(fmaxf(n, -8.f), 7.f)) + 8);
}

// The scale of a block, half of whose values a lane holds, the other half its
// neighbour of i ^ 1, and the lane's codes: byte x the dimensions x (low) and
// x + 8 (high) of its sixteen.
template <typename T>
__device__ __forceinline__ uint2 quantize(const Values<T>& x, __half& scale) {
    float most, least;
    x.ends(most, least);
    most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, 4));
    least = min_nan(least, __shfl_xor_sync(0xffffffffu, least, 4));
    const float top = most >= -least ? most : least;   // NaN: least, which is NaN too
    float d = __bfloat162float(__float2bfloat16_rn(__fmul_rn(top, -0.125f)));
    if (fabsf(d) > kTop) d = copysignf(kTop, d);
    if (!(fabsf(top) <= 3.402823466e38f)) d = __int_as_float(0x7FC00000);
    scale = __float2half_rn(d);
    d = __half2float(scale);
    const bool none = d == 0.f || d != d;
    const float inverse = none ? 0.f : 1.f / d;
    uint32_t w[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        uint32_t b[4];   // the low byte
#pragma unroll
        for (int k = 0; k < 4; ++k)
            b[k] = code_of<T>(x.get(4 * half + k), d, inverse) + 16u * code_of<T>(x.get(4 * half + k + 8), d, inverse);
        w[half] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    }
    return none ? make_uint2(0x88888888u, 0x88888888u) : make_uint2(w[0], w[1]);
}

// Inputs in 16-byte loads: by 32 bytes, as read() stores, 8192 tokens took 12.2 us in place of 10.8.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) kv4_write_kernel(const WriteArgs a) {
    const mmq_kv4_write_t& p = a.p;
    griddep_launch_dependents();
    griddep_wait();
    const Lane<D> lane(p.slots, p.tokens, p.kv_heads);
    const Slots<D> slots(p, lane, a.status);
    const int i = lane.i, c = lane.c;
    const bool keys = blockIdx.y == 0;
    auto token = [&](int n) { return keys ? key_token(c, n) : value_token(c, n); };
    const void* const from = keys ? p.k : p.v;
    const int64_t token_stride = keys ? p.k_token_stride : p.v_token_stride;
    const int64_t column = lane.h * (keys ? p.k_head_stride : p.v_head_stride) + 16 * i;
    Values<T> x[4];
    uint2 b[4];
    __half s[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        const int64_t t = lane.t0 + token(n);
        x[n].load(from, t * token_stride + column, t >= 0 && t < p.tokens);
    }
#pragma unroll
    for (int n = 0; n < 4; ++n) b[n] = quantize<T>(x[n], s[n]);
    if (slots.whole) {
        uint8_t* const dst = tile_of<D>(p.cache, slots.first, lane.h, p.kv_heads, a.page_shift);
        if (keys) {   // word x / 2 of tokens t and t + 8 takes two bytes of each
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int x = 0; x < 8; x += 2) {
                    const uint32_t lo = x < 4 ? b[n].x : b[n].y, hi = x < 4 ? b[n + 2].x : b[n + 2].y;
                    *reinterpret_cast<uint32_t*>(dst + key_byte(key_token(c, n), i, x)) = __byte_perm(lo, hi, x & 2 ? 0x7362 : 0x5140);
                }
            if ((i & 1) == 0) {
#pragma unroll
                for (int n = 0; n < 4; ++n) *reinterpret_cast<__half*>(dst + key_scale<D>(key_token(c, n), i >> 1)) = s[n];
            }
        } else {   // word x takes a byte of each of the four tokens
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                uint32_t w[4];
#pragma unroll
                for (int n = 0; n < 4; ++n) w[n] = x < 4 ? b[n].x : b[n].y;
                const uint32_t sel = uint32_t(x & 3) | uint32_t(4 + (x & 3)) << 4;
                *reinterpret_cast<uint32_t*>(dst + value_byte<D>(2 * c, i, x)) =
                    __byte_perm(__byte_perm(w[0], w[2], sel), __byte_perm(w[1], w[3], sel), 0x5410);
            }
            if ((i & 1) == 0) {
                const __half2 s0 = __halves2half2(s[0], s[1]), s1 = __halves2half2(s[2], s[3]);
                *reinterpret_cast<uint2*>(dst + value_scale<D>(2 * c, i >> 1)) =
                    make_uint2(*reinterpret_cast<const uint32_t*>(&s0), *reinterpret_cast<const uint32_t*>(&s1));
            }
        }
        return;
    }
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        const int slot = slots.of(token(n));
        if (slot < 0) continue;
        uint8_t* const dst = tile_of<D>(p.cache, slot, lane.h, p.kv_heads, a.page_shift);
        const int place = int(slot & 15);
#pragma unroll
        for (int x = 0; x < 8; ++x)
            dst[keys ? key_byte(place, i, x) : value_byte<D>(place, i, x)] = uint8_t((x < 4 ? b[n].x : b[n].y) >> (8 * (x & 3)));
        if ((i & 1) == 0)
            *reinterpret_cast<__half*>(dst + (keys ? key_scale<D>(place, i >> 1) : value_scale<D>(place, i >> 1))) = s[n];
    }
}

// -------------------------------------------------------------------- read
// A pair of codes in the low nibbles of two halves, less 8 and times a scale.
// Exact: 1024 + code and the difference are, and so is the product, by the
// layout's bound on scales.
__device__ __forceinline__ __half2 expand(uint32_t pair, __half2 scale) {
    const uint32_t w = (pair & 0x000F000Fu) | 0x64006400u;
    return __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&w), __float2half2_rn(1032.f)), scale);
}
// 32 bytes, a whole sector, in one store where the address allows it: 32k tokens 30 us, and 37 by two of 16 bytes; 8192 as
// float32 14.5 and 30.5.
__device__ __forceinline__ void store8(void* at, const uint32_t* w, bool aligned) {
    if (aligned) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        static_cast<uint4*>(at)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        static_cast<uint4*>(at)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}
// A token's sixteen values from four words, each with two neighbouring
// dimensions in its halves' low nibbles and those + 8 in the next.
template <typename T>
__device__ __forceinline__ void store16(T* at, const uint32_t (&pairs)[4], __half scale, bool aligned) {
    const __half2 s = __half2half2(scale);
    constexpr int kWords = sizeof(T) / 2;   // of a pair
    uint32_t w[8 * kWords];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const __half2 x = expand(pairs[k & 3] >> (4 * (k >> 2)), s);
        if (std::is_same<T, __half>::value) {
            w[k] = *reinterpret_cast<const uint32_t*>(&x);
        } else {
            const float2 f = __half22float2(x);
            const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
            if (std::is_same<T, float>::value) {
                w[kWords * k] = __float_as_uint(f.x);
                w[kWords * k + kWords - 1] = __float_as_uint(f.y);
            } else {
                w[k] = *reinterpret_cast<const uint32_t*>(&b);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < kWords; ++k) store8(at + 16 / kWords * k, w + 8 * k, aligned);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const ReadArgs a) {
    const mmq_kv4_read_t& p = a.p;
    griddep_launch_dependents();
    griddep_wait();
    const Lane<D> lane(p.slots, p.tokens, p.kv_heads);
    const Slots<D> slots(p, lane, a.status);
    const int i = lane.i, c = lane.c;
    const bool keys = blockIdx.y == 0, aligned = a.aligned;
    auto out = [&](int t) {
        return static_cast<T*>(keys ? p.k : p.v) + ((lane.t0 + t) * p.kv_heads + lane.h) * D + 16 * i;
    };
    if (slots.whole) {
        const uint8_t* const src = tile_of<D>(p.cache, slots.first, lane.h, p.kv_heads, a.page_shift);
        uint32_t w[8];
        if (keys) {
            __half s[4];
#pragma unroll
            for (int x = 0; x < 8; ++x)
                w[x] = *reinterpret_cast<const uint32_t*>(src + key_byte(key_token(c, x >> 2), i, 2 * (x & 3)));
#pragma unroll
            for (int n = 0; n < 4; ++n) s[n] = *reinterpret_cast<const __half*>(src + key_scale<D>(key_token(c, n), i >> 1));
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                uint32_t pairs[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) pairs[x] = w[4 * (n & 1) + x] >> (8 * (n >> 1));
                store16(out(key_token(c, n)), pairs, s[n], aligned);
            }
        } else {
#pragma unroll
            for (int x = 0; x < 8; ++x) w[x] = *reinterpret_cast<const uint32_t*>(src + value_byte<D>(2 * c, i, x));
            const uint2 s = *reinterpret_cast<const uint2*>(src + value_scale<D>(2 * c, i >> 1));
#pragma unroll
            for (int n = 0; n < 4; ++n) {   // token 2 c + n % 2 + 8 (n / 2), byte n / 2 + 2 (n % 2)
                uint32_t pairs[4];
                const uint32_t b = uint32_t((n >> 1) + 2 * (n & 1));
#pragma unroll
                for (int x = 0; x < 4; ++x) pairs[x] = __byte_perm(w[2 * x], w[2 * x + 1], b | (4 + b) << 8);
                const __half2 two = *reinterpret_cast<const __half2*>(n < 2 ? &s.x : &s.y);
                store16(out(value_token(c, n)), pairs, n & 1 ? __high2half(two) : __low2half(two), aligned);
            }
        }
        return;
    }
#pragma unroll 1
    for (int n = 0; n < 4; ++n) {
        const int t = keys ? key_token(c, n) : value_token(c, n);
        const int slot = slots.of(t);
        if (lane.t0 + t < 0 || lane.t0 + t >= p.tokens) continue;
        uint32_t pairs[4] = {0x00880088u, 0x00880088u, 0x00880088u, 0x00880088u};   // zeros
        __half scale = __float2half_rn(0.f);
        if (slot >= 0) {
            const uint8_t* const src = tile_of<D>(p.cache, slot, lane.h, p.kv_heads, a.page_shift);
            const int place = int(slot & 15);
#pragma unroll
            for (int x = 0; x < 8; x += 2)
                pairs[x >> 1] = uint32_t(src[keys ? key_byte(place, i, x) : value_byte<D>(place, i, x)]) |
                                uint32_t(src[keys ? key_byte(place, i, x + 1) : value_byte<D>(place, i, x + 1)]) << 16;
            scale = *reinterpret_cast<const __half*>(src + (keys ? key_scale<D>(place, i >> 1) : value_scale<D>(place, i >> 1)));
        }
        store16(out(t), pairs, scale, aligned);
    }
}

int shift_of(int page_size) {
    int s = 0;
    while ((1 << s) < page_size) ++s;
    return s;
}

template <int D, typename Args>
cudaError_t launch(void (*kernel)(Args), const Args& a, cudaStream_t s) {
    // one group more than the tokens fill: the first may hold as little as one
    const int64_t items = (int64_t(a.p.tokens) + 15 + kTokens - 1) / kTokens * a.p.kv_heads;
    if (items > INT32_MAX) return cudaErrorInvalidValue;
    constexpr int kItems = kThreads / Lane<D>::kLanes;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = mmq::launch_config(dim3(unsigned((items + kItems - 1) / kItems), 2), dim3(kThreads), 0, s, attr);
    return cudaLaunchKernelEx(&cfg, kernel, a);
}
template <typename T, int D>
cudaError_t write(const WriteArgs& a, cudaStream_t s) {
    return launch<D>(kv4_write_kernel<T, D>, a, s);
}
template <typename T, int D>
cudaError_t read(const ReadArgs& a, cudaStream_t s) {
    return launch<D>(kv4_read_kernel<T, D>, a, s);
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
    const bool aligned = (reinterpret_cast<uintptr_t>(p.k) | reinterpret_cast<uintptr_t>(p.v)) % 32 == 0;
    const ReadArgs a{p, shift_of(p.page_size), aligned, status};
    const bool wide = p.head_dim == 128;
    switch (p.type) {
        case MMQ_TYPE_F16: return wide ? read<__half, 128>(a, s) : read<__half, 64>(a, s);
        case MMQ_TYPE_BF16: return wide ? read<__nv_bfloat16, 128>(a, s) : read<__nv_bfloat16, 64>(a, s);
        default: return wide ? read<float, 128>(a, s) : read<float, 64>(a, s);
    }
}

}  // namespace mmq
