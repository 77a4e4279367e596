// The shared prefix's part of shared-prefix attention on the tensor cores.
//
// All rows of one kv head (every token's heads of its group) see the same
// keys, so a key tile is read once for 128 or 256 rows: two products of
// 128 rows x 128 keys x D per tile, S = Q K^T and O += P V with
// P = 2^(S scale log2(e) - m), P rounded to the cache's type, everything else
// f32.  At 2 x 128 rows and D = 128 a 64 KB pair of tiles carries 16.8 MFLOP
// twice over, so with many rows the tensor cores bound it and with few rows the
// key / value bytes.
//
// One CTA per SM:
//   warps 0-3, 4-7  softmax groups 0 and 1, thread = row (its tensor-memory
//                   lane): read S, keep the row's maximum and sum, write P over
//                   S, and now and then scale O
//   warp 8          TMA producer: key and value tiles (128 keys, 128-byte
//                   swizzled panels of 64 values) through a 128 KB ring
//   warps 9, 10     MMA issuers of groups 0 and 1: S = Q K^T, O += P V, P from
//                   tensor memory, taking turns batch by batch
// More than 48 rows: the groups hold two row tiles, of which the second may be
// empty, and share each key tile.  Up to 48: both hold the same rows and take key
// tiles in turn, as two parts (times at prefix_tiles in attention.cu).
// While one group does its softmax (1270 cycles a tile) the tensor cores work
// for the other (16 products of 64 cycles).  The issuing thread is held for the
// whole of its products, so one thread for both groups left the tensor cores
// idle while it did anything else (2050 cycles a batch), and two free ones fell
// into step, both groups at their softmax and then both at their products (1950
// a batch); hence two that pass a turn.
//
// Measured: 1024 rows per kv head x 16384 keys x 8 kv heads, D = 128 (68.7
// GFLOP): 62 us on the 128 CTAs that four parts make, 1.1 PFLOP/s, 59 % of the
// measured bf16 rate.  A pair of tiles takes 2980 cycles of which the products
// are 2048: a group's chain of scores, softmax (1230), hand-over (230) and its
// own products (2 x 512, and the waits between) is what is left to shorten.
// Tried and no faster: half of P handed over early, the maximum of the tile
// before as the reference so that the exponentials need not wait for this
// one's, polling instead of suspended waits.
//
// P is rounded to 16 bits because the second product takes both operands of one
// type.  As the sum of two such values, a second product each, a whole call's
// results have the errors of f32 weights (2.1e-4 instead of 2.9e-4 of the norm
// with an f16 output, whose own rounding is 2.1e-4; 1.65e-3 instead of 2.35e-3 with
// bf16), for 103 -> 125 us here (256 sequences) and 69 -> 78 us (64 sequences x
// 32768 keys): not kept.
//
// The running maximum and sum are the online softmax of Milakov and Gimelshein
// (2018); two groups that alternate between softmax and products, and a maximum
// that may lag, are known from the published work on attention since.  O is only
// scaled when a row's largest score (in units of log2) has grown by more than 8
// since the last time: nothing is lost, since the factor is common to P, the sum
// and O.  P then stays below 2^8, and as fp16 below 2^15: its reference is 7
// under the score, which the rest of fp16's range has room for, so that weights
// of down to 2^-21 of the largest are normal numbers and those below it are off
// by at most 2^-32 of the largest.  (With P at most 2^8 the last was 2^-25, and
// many keys that far under one that takes all were lost.)  Scores past 2^20 have
// a loop of their own, where the reference is the score.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "attention.h"
#include "mmq_internal.h"
#include "sm103_ptx.cuh"
#include "tc_common.cuh"

namespace {

using namespace mmq::ptx;
using namespace mmq::tc;
using mmq::AttnArgs;

constexpr int kKeys = 128, kRows = 128;
constexpr int kThreads = 384, kWarpTma = 8, kWarpMma = 9;   // and kWarpMma + 1
// Registers: 168 per thread at launch (the launcher checks it), of which the
// third warpgroup gives up 80 so that a softmax thread can hold its row of
// 128 scores: 2 x 128 x 208 + 128 x 88 = 384 x 168.
constexpr uint32_t kRegsLaunch = 168, kRegsSoftmax = 208, kRegsOther = 88;
static_assert(256 * kRegsSoftmax + 128 * kRegsOther <= kThreads * kRegsLaunch, "register split");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;   // S_i at 128 i (P_i over its first 64 columns), O_i at 256 + 128 i
constexpr float kGrow = 8.f;
template <typename T>
constexpr float kLift = std::is_same<T, __half>::value ? 7.f : 0.f;   // of P, in units of log2
static_assert(kGrow + kLift<__half> < 16.f, "P within fp16's range");
constexpr float kWide = 0x1p20f;
// What is subtracted from a row's scores, for a largest one of m, or none yet.
template <typename T>
__device__ __forceinline__ float reference(float m) {
    return m == -INFINITY ? 0.f : fabsf(m) < kWide ? m - kLift<T> : m;
}

template <int D>
struct Layout {
    static constexpr int kPanels = D / 64;
    static constexpr int kSlots = 512 / D;                   // 128 KB of tiles in flight: one CTA per SM
    static constexpr int kPanel = kKeys * 128;               // 128 rows of 64 16-bit values
    static constexpr int kTile = kPanels * kPanel;
    static constexpr int kOffQ = 0;                          // two row tiles
    static constexpr int kOffRing = 2 * kTile;
    static constexpr int kOffBar = kOffRing + kSlots * kTile;
    // barriers: full, empty per slot; q_full, s_full, o_full, p_full, turn per group; drain
    static constexpr int kOffMisc = kOffBar + (2 * kSlots + 11) * 8;
    static constexpr int kBytes = kOffMisc + 16 + 1024;
};
static_assert(Layout<128>::kBytes <= 232448, "shared memory budget");

struct Maps {
    CUtensorMap k, v;
};

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack16(float a, float b, __half*) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack16(float a, float b, __nv_bfloat16*) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

template <typename T>
__host__ __device__ constexpr uint32_t idesc_16(int N, bool b_rows_are_k) {
    const uint32_t fmt = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
    return idesc_f16_f32(kRows, N) | (fmt << 7) | (fmt << 10) | (b_rows_are_k ? 1u << 16 : 0u);
}

template <typename T, int D, bool kTwo>
__global__ void __launch_bounds__(kThreads, 1)
attn_prefix_kernel(const __grid_constant__ Maps maps, const AttnArgs a) {
    using L = Layout<D>;
    constexpr int kSlots = L::kSlots;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar0 = sbase + L::kOffBar;
    auto full = [&](int s) { return bar0 + 8u * uint32_t(s); };
    auto empty = [&](int s) { return bar0 + 8u * uint32_t(kSlots + s); };
    auto q_full = [&](int g) { return bar0 + 8u * uint32_t(2 * kSlots + g); };
    auto s_full = [&](int g) { return bar0 + 8u * uint32_t(2 * kSlots + 2 + g); };
    auto o_full = [&](int g) { return bar0 + 8u * uint32_t(2 * kSlots + 4 + g); };
    auto p_full = [&](int g) { return bar0 + 8u * uint32_t(2 * kSlots + 6 + g); };
    auto turn = [&](int g) { return bar0 + 8u * uint32_t(2 * kSlots + 8 + g); };
    const uint32_t drain = bar0 + 8u * uint32_t(2 * kSlots + 10);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffMisc);
    const AbortFlag abort_flag{sbase + L::kOffMisc + 4};
    const mmq_shared_prefix_attention_t& p = a.p;
    int* const status = a.status;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), kTwo ? 2 : 1);
        }
        for (int g = 0; g < 2; ++g) {
            mbar_init(q_full(g), 4);
            mbar_init(s_full(g), 1);
            mbar_init(p_full(g), 4);
            mbar_init(o_full(g), 1);
            mbar_init(turn(g), 1);
        }
        mbar_init(drain, 2);
        abort_flag.set(0u);
        fence_barrier_init();
        prefetch_tmap(&maps.k);
        prefetch_tmap(&maps.v);
    }
    __syncwarp();
    if (warp == kWarpMma) {
        tmem_alloc(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // The suffix kernel may run beside this one (on the SMs this grid leaves
    // free); what it reads is complete once this wait is over.
    griddep_wait();
    griddep_launch_dependents();

    // Items: (row block, kv head, part), parts of one head's keys next to each other.
    const int64_t rows = a.tokens * a.group;
    const int per_unit = kTwo ? 2 * kRows : kRows;
    const int units = int((rows + per_unit - 1) / per_unit);
    const int parts = a.prefix_parts / (kTwo ? 1 : 2);
    const int items = units * p.kv_heads * parts;
    struct Item {
        int h, part, tiles;   // tiles: of 128 keys
        int64_t r0, k0, k1;
    };
    auto get = [&](int i) {
        Item w;
        w.part = i % parts;
        const int u = i / parts;
        w.h = u / units;
        w.r0 = int64_t(u % units) * per_unit;
        w.k0 = w.part * a.part_keys;
        w.k1 = min(w.k0 + a.part_keys, p.prefix);
        w.tiles = int((w.k1 - w.k0 + kKeys - 1) / kKeys);
        return w;
    };

    if (warp >= 8) {
        setmaxnreg_dec<kRegsOther>();
        if (warp == kWarpTma) {
            // ---------------------------------------------------------- producer
            if (lane == 0) {
                Ring<kSlots> r;
                int issued[kSlots] = {};
                uint32_t par[kSlots] = {};
                bool withhold = a.inject && blockIdx.x == 0;
                auto load = [&](const CUtensorMap* map, int h, int64_t key) {
                    if (!wait_bounded(empty(r.slot), r.phase ^ 1u, abort_flag, status)) return false;
                    const uint32_t dst = sbase + uint32_t(L::kOffRing + r.slot * L::kTile);
                    if (!withhold) {
                        mbar_arrive_expect_tx(full(r.slot), uint32_t(L::kTile));
#pragma unroll
                        for (int c = 0; c < L::kPanels; ++c)
                            tma_load_3d(dst + uint32_t(c * L::kPanel), map, full(r.slot), 64 * c, h, int32_t(key));
                        issued[r.slot] = 1;
                        par[r.slot] = r.phase;
                    }
                    withhold = false;
                    r.next();
                    return true;
                };
                for (int i = blockIdx.x; i < items; i += gridDim.x) {
                    const Item w = get(i);
                    const int tiles = w.tiles;
                    auto key = [&](int t) { return w.k0 + int64_t(t) * kKeys; };
                    if (kTwo) {   // K0 V0 K1 V1 ...
                        for (int t = 0; t < tiles; ++t)
                            if (!load(&maps.k, w.h, key(t)) || !load(&maps.v, w.h, key(t))) goto producer_done;
                    } else {      // K0 K1 V0 V1 K2 K3 V2 V3 ..., an odd last tile alone
                        for (int t = 0; t < tiles; t += 2) {
                            const bool two = t + 1 < tiles;
                            if (!load(&maps.k, w.h, key(t)) || (two && !load(&maps.k, w.h, key(t + 1))) ||
                                !load(&maps.v, w.h, key(t)) || (two && !load(&maps.v, w.h, key(t + 1))))
                                goto producer_done;
                        }
                    }
                }
            producer_done:
                for (int s = 0; s < kSlots; ++s)
                    if (issued[s]) wait_drain(full(s), par[s], status);
            }
        } else if (warp < kWarpMma + 2) {
            // ------------------------------------------------------- MMA issuers
            if (lane == 0) {
                const int g = warp - kWarpMma;
                uint32_t q_phase = 0, p_phase = 0, base = 0;   // base: ring position of the item's first tile
                uint32_t t_phase = g == 0 ? 1u : 0u;           // group 0 has the first turn
                constexpr uint32_t kIdQK = idesc_16<T>(kKeys, false), kIdPV = idesc_16<T>(D, true);
                constexpr uint64_t kTileDesc = uint64_t(L::kTile >> 4), kPanelDesc = uint64_t(L::kPanel >> 4);
                const uint64_t dq = smem_desc_sw128(sbase + uint32_t(L::kOffQ + g * L::kTile));
                const uint64_t k_desc = smem_desc_sw128(sbase + uint32_t(L::kOffRing));
                const uint64_t v_desc = smem_desc_mn_sw128(sbase + uint32_t(L::kOffRing), uint32_t(L::kPanel));
                const uint32_t ts = tmem + kColS + 128u * uint32_t(g), to = tmem + kColO + 128u * uint32_t(g);
                auto arrived = [&](uint32_t pos) {
                    return wait_bounded(full(int(pos % kSlots)), (pos / kSlots) & 1u, abort_flag, status);
                };
                for (int i = blockIdx.x; i < items; i += gridDim.x) {
                    const int tiles = get(i).tiles, mine = kTwo ? tiles : (tiles + 1 - g) >> 1;
                    auto k_at = [&](int s) { return base + uint32_t(kTwo ? 2 * s : 4 * s + g); };
                    auto v_at = [&](int s) {
                        return base + uint32_t(kTwo ? 2 * s + 1 : 4 * s + (g == 1 ? 3 : 2 * s + 1 < tiles ? 2 : 1));
                    };
                    // S = Q K^T with K in `slot`, which has arrived
                    auto scores = [&](uint32_t slot, bool pass) {
                        const uint64_t dk = k_desc + slot * kTileDesc;
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint64_t off = uint64_t(kk >> 2) * kPanelDesc + uint64_t((kk & 3) * 2);
                            if (kk == D / 16 - 2 && pass) mbar_arrive(turn(g ^ 1));   // the other thread needs a moment to start
                            mma_f16(ts, dq + off, dk + off, kIdQK, uint32_t(kk > 0));
                        }
                        mma_commit(s_full(g));
                        mma_commit(empty(int(slot)));
                    };
                    if (kTwo || mine > 0) {
                        if (!wait_bounded(q_full(g), q_phase, abort_flag, status)) goto mma_done;
                        q_phase ^= 1u;
                        if (!arrived(k_at(0))) goto mma_done;
                        tc_fence_after();
                        scores(k_at(0) % kSlots, false);
                    }
                    const int rounds = kTwo ? tiles : (tiles + 1) >> 1;   // group 1 may have one tile less
                    for (int s = 0; s < rounds; ++s) {
                        const bool has = s < mine, more = s + 1 < mine;
                        // everything that can be waited for before the turn
                        if (has && (!arrived(v_at(s)) || (more && !arrived(k_at(s + 1))) ||
                                    !wait_bounded(p_full(g), p_phase, abort_flag, status)))
                            goto mma_done;
                        const uint32_t v_slot = v_at(s) % kSlots, k_slot = k_at(s + 1) % kSlots;
                        const uint64_t dv = v_desc + v_slot * kTileDesc;
                        if (!wait_bounded(turn(g), t_phase, abort_flag, status)) goto mma_done;
                        tc_fence_after();
                        t_phase ^= 1u;
                        if (!has) {
                            mbar_arrive(turn(g ^ 1));
                            break;
                        }
                        p_phase ^= 1u;
#pragma unroll
                        for (int kk = 0; kk < kKeys / 16; ++kk)   // 16 keys = 16 rows of 128 bytes
                            mma_f16_ta(to, ts + 8u * uint32_t(kk), dv + uint64_t(kk * 128), kIdPV, uint32_t(s > 0 || kk > 0));
                        if (more) {
                            scores(k_slot, true);
                        } else {
                            mbar_arrive(turn(g ^ 1));
                            mma_commit(o_full(g));
                        }
                        mma_commit(empty(int(v_slot)));
                    }
                    base += uint32_t(2 * tiles);
                }
        mma_done:
                mma_commit(drain);   // everything issued, also after a wait that ran out
                wait_drain(drain, 0u, status);
            }
        }
    } else {
        // ----------------------------------------------------------- softmax
        setmaxnreg_inc<kRegsSoftmax>();
        const int g = warp >> 2;
        const int row = (warp & 3) * 32 + lane;
        const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + kColS + 128u * uint32_t(g), to = tmem + lanes + kColO + 128u * uint32_t(g);
        T* const tag = nullptr;
        uint32_t s_phase = 0, o_phase = 0;
        for (int i = blockIdx.x; i < items; i += gridDim.x) {
            const Item w = get(i);
            const int64_t r = w.r0 + (kTwo ? g * kRows : 0) + row;
            const bool valid = r < rows;
            const int64_t tok = valid ? r / a.group : 0;
            const int head = int(w.h * a.group + (valid ? r - tok * a.group : 0));
            const int mine = kTwo ? w.tiles : (w.tiles + 1 - g) >> 1;
            const int part = kTwo ? w.part : 2 * w.part + g;
            const int64_t at = (int64_t(part) * a.tokens + tok) * p.heads + head;
            // An item of one tile has none for group 1, which does not arrive on q_full for it either: it would wait
            // for nothing here, and be a phase of that barrier ahead before the issuer has seen this one.
            if (!kTwo && mine == 0) {
                if (valid) a.part_ml[at] = make_float2(-INFINITY, 0.f);
                continue;
            }
            // The group's query rows, swizzled (16-byte chunk c of row n at c ^ (n & 7)); zeros past the last row.
            {
                const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + tok * p.q_stride + int64_t(head) * D);
                const uint32_t dst = sbase + uint32_t(L::kOffQ + g * L::kTile + row * 128);
#pragma unroll
                for (int c = 0; c < D / 8; ++c) {
                    const uint4 v = valid ? src[c] : make_uint4(0u, 0u, 0u, 0u);
                    st_shared_v4(dst + uint32_t((c >> 3) * L::kPanel + (((c & 7) ^ (row & 7)) << 4)), v.x, v.y, v.z, v.w);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full(g));
            }
            float m = -INFINITY, l = 0.f;
            bool ok = true, wide = false;
            int n = 0;
            auto scale_o = [&](float f) {   // at rest: the product before this S has completed
                l *= f;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    tmem_ld_32x32b_x32(to + 32u * uint32_t(c), o);
                    tmem_wait_ld(o);
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                    tmem_st_32x32b_x32(to + 32u * uint32_t(c), o);
                }
            };
            for (; n < mine && ok; ++n) {
                ok = __all_sync(0xffffffffu, wait_bounded(s_full(g), s_phase, abort_flag, status));
                if (!ok) break;
                s_phase ^= 1u;
                tc_fence_after();
                uint32_t s[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(ts + 32u * uint32_t(c), s[c]);
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_wait_ld(s[c]);
                const int64_t left = w.k1 - (w.k0 + int64_t(kTwo ? n : 2 * n + g) * kKeys);
                if (left < kKeys) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (32 * c + k >= left) s[c][k] = 0xFF800000u;
                }
                float x0 = __uint_as_float(s[0][0]), x1 = __uint_as_float(s[1][0]), x2 = __uint_as_float(s[2][0]),
                      x3 = __uint_as_float(s[3][0]);
#pragma unroll
                for (int k = 0; k < 32; k += 2) {
                    x0 = max3(x0, __uint_as_float(s[0][k]), __uint_as_float(s[0][k + 1]));
                    x1 = max3(x1, __uint_as_float(s[1][k]), __uint_as_float(s[1][k + 1]));
                    x2 = max3(x2, __uint_as_float(s[2][k]), __uint_as_float(s[2][k + 1]));
                    x3 = max3(x3, __uint_as_float(s[3][k]), __uint_as_float(s[3][k + 1]));
                }
                const float top = fmaxf(fmaxf(x0, x1), fmaxf(x2, x3)) * a.scale_log2;
                if (__any_sync(0xffffffffu, n == 0 || top > m + kGrow)) {
                    const float was = m;
                    wide = __any_sync(0xffffffffu, !(fabsf(fmaxf(m, top)) < kWide));
                    if (wide) break;
                    m = fmaxf(m, top);
                    if (n > 0) scale_o(was == m ? 1.f : ex2(was - m));
                }
                const float base = m - kLift<T>;
                const uint64_t scale2 = pack2(a.scale_log2, a.scale_log2), base2 = pack2(-base, -base);
                uint64_t sum[2] = {0, 0};
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t pk[32];
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        const uint32_t* sc = &s[2 * half + (k >> 4)][2 * (k & 15)];
                        const uint64_t e = ffma2(pack2u(sc[0], sc[1]), scale2, base2);
                        const float u = ex2(lo_f(e)), v = ex2(hi_f(e));
                        sum[k & 1] = fadd2(sum[k & 1], pack2(u, v));
                        pk[k] = pack16(u, v, tag);
                    }
                    tmem_st_32x32b_x32(ts + 32u * uint32_t(half), pk);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full(g));
                sum[0] = fadd2(sum[0], sum[1]);
                l += lo_f(sum[0]) + hi_f(sum[0]);
            }
            // S scale - m in one step, as above, is past zero by what m lost in its rounding, half a unit in its last
            // place: from 2^20 on too much for P's range.  From the first tile where a row of the warp gets there the
            // products are rounded first, as m was, and m is neither lifted nor let behind (nor is a row left out that
            // has no score above -Inf).  No usual call comes here, so short loops over S where it lies.
            for (bool here = true; wide && n < mine; ++n, here = false) {
                if (!here) {
                    ok = __all_sync(0xffffffffu, wait_bounded(s_full(g), s_phase, abort_flag, status));
                    if (!ok) break;
                    s_phase ^= 1u;
                    tc_fence_after();
                }
                const int64_t left = w.k1 - (w.k0 + int64_t(kTwo ? n : 2 * n + g) * kKeys);
                float top = -INFINITY, sum = 0.f;
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    uint32_t x[32];
                    tmem_ld_32x32b_x32(ts + 32u * uint32_t(c), x);
                    tmem_wait_ld(x);
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (32 * c + k < left) top = fmaxf(top, __uint_as_float(x[k]));
                }
                const float was = m;
                m = fmaxf(m, __fmul_rn(top, a.scale_log2));
                const float base = reference<T>(m);
                if (n > 0) scale_o(was == -INFINITY ? 0.f : ex2(reference<T>(was) - base));
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    uint32_t x[32], pk[16];
                    tmem_ld_32x32b_x32(ts + 32u * uint32_t(c), x);
                    tmem_wait_ld(x);
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        const float y = __fmul_rn(__uint_as_float(x[k]), a.scale_log2);
                        x[k] = 32 * c + k < left ? __float_as_uint(ex2(__fsub_rn(y, base))) : 0u;
                        sum += __uint_as_float(x[k]);
                    }
#pragma unroll
                    for (int k = 0; k < 16; ++k) pk[k] = pack16(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1]), tag);
                    tmem_st_32x32b_x16(ts + 16u * uint32_t(c), pk);   // over what has been read
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full(g));
                l += sum;
            }
            // The part's result.
            if (!ok) break;
            ok = __all_sync(0xffffffffu, wait_bounded(o_full(g), o_phase, abort_flag, status));
            if (!ok) break;
            o_phase ^= 1u;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld_32x32b_x32(to + 32u * uint32_t(c), o);
                tmem_wait_ld(o);
                if (valid) {
                    float4* dst = reinterpret_cast<float4*>(a.part_o + at * D + 32 * c);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        dst[k] = make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]),
                                             __uint_as_float(o[4 * k + 2]), __uint_as_float(o[4 * k + 3]));
                }
            }
            tc_fence_before();
            if (valid) a.part_ml[at] = make_float2(m == -INFINITY ? m : reference<T>(m), l);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kWarpMma) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

bool encode_prefix(CUtensorMap* m, const mmq_shared_prefix_attention_t& p, const void* base) {
    auto fn = get_encode();
    if (!fn) return false;
    const cuuint64_t dims[3] = {cuuint64_t(p.head_dim), cuuint64_t(p.kv_heads), cuuint64_t(p.prefix)};
    const cuuint64_t strides[2] = {cuuint64_t(p.prefix_head_stride) * 2, cuuint64_t(p.prefix_token_stride) * 2};
    const cuuint32_t box[3] = {64, 1, kKeys}, estr[3] = {1, 1, 1};
    return fn(m, p.type == MMQ_TYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
              const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D, bool kTwo>
cudaError_t launch(const AttnArgs& a, int nsm, cudaLaunchConfig_t cfg) {
    Maps maps;
    if (!encode_prefix(&maps.k, a.p, a.p.k_prefix) || !encode_prefix(&maps.v, a.p, a.p.v_prefix))
        return cudaErrorInvalidValue;
    cudaError_t e;
    constexpr int smem = Layout<D>::kBytes;
    static const bool registers_ok = [] {   // else the split's increase would wait forever
        cudaFuncAttributes f;
        return cudaFuncGetAttributes(&f, attn_prefix_kernel<T, D, kTwo>) == cudaSuccess && f.numRegs == int(kRegsLaunch);
    }();
    if (!registers_ok) return cudaErrorLaunchOutOfResources;
    if ((e = cudaFuncSetAttribute(attn_prefix_kernel<T, D, kTwo>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)))
        return e;
    const int64_t per = kTwo ? 2 * kRows : kRows;
    const int64_t items = (a.tokens * a.group + per - 1) / per * a.p.kv_heads * (a.prefix_parts / (kTwo ? 1 : 2));
    cfg.gridDim = dim3(unsigned(items < nsm ? items : nsm));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    return cudaLaunchKernelEx(&cfg, attn_prefix_kernel<T, D, kTwo>, maps, a);
}

template <typename T, int D>
cudaError_t launch_rows(const AttnArgs& a, int nsm, const cudaLaunchConfig_t& cfg) {
    return a.prefix_tiles == 2 ? launch<T, D, true>(a, nsm, cfg) : launch<T, D, false>(a, nsm, cfg);
}

}  // namespace

namespace mmq {

cudaError_t launch_attention_prefix(const AttnArgs& a, int nsm, const cudaLaunchConfig_t& cfg) {
    if (a.p.type == MMQ_TYPE_F16)
        return a.p.head_dim == 64 ? launch_rows<__half, 64>(a, nsm, cfg) : launch_rows<__half, 128>(a, nsm, cfg);
    return a.p.head_dim == 64 ? launch_rows<__nv_bfloat16, 64>(a, nsm, cfg) : launch_rows<__nv_bfloat16, 128>(a, nsm, cfg);
}

}  // namespace mmq
