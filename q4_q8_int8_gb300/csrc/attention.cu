// Attention of a batch whose sequences share one prefix: softmax over the
// prefix keys, then each token's own paged suffix, in f32, computed in parts
// and joined by the running maximum and sum:
//   part p of a row:  l_p = sum 2^(s - m_p),  o_p = sum 2^(s - m_p) v,  m_p a
//                     reference near its largest s
//   row:              out = sum_p 2^(m_p - m) o_p / sum_p 2^(m_p - m) l_p,  m = max m_p
// with s = q.k * scale * log2(e).  A row with no key at all (an empty prefix
// and an empty suffix) is zero.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "attention.h"
#include "half_ops.cuh"
#include "mmq_internal.h"
#include "sm103_ptx.cuh"

namespace {

using namespace mmq::ptx;
using mmq::AttnArgs;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// ----------------------------------------------------------------- suffix
// One warp, a CTA of its own: up to 16 rows that see the same keys (a token's
// heads of one kv head, over a part of its suffix).  Bound by the key / value
// bytes: rows are padded to the 16 of one mma.sync tile, keys come 16 at a time
// through a cp.async ring of three (24 KB at 128 dims, nine such warps per SM:
// up to 144 KB in flight), and warps that start, stream and finish on their own
// keep the memory busy where suffixes are short.  Keys past the row's limit are filled with zeros, not
// read, so what the cache holds there cannot matter.  Weights are rounded to
// the cache's type for the second product (their sum is taken in f32 before
// that); as fp16 their reference is 7 (in units of log2) under the largest
// score, so that those down to 2^-21 of the largest are normal numbers, and for
// no score, however it is rounded, more than 8.  Both products accumulate in
// f32.  Measured: 256 suffixes of 1 to 512 tokens, 8 kv heads x 128 (261 MB):
// 50 us, 5.2 TB/s, 77 % of the copy rate (as CTAs of four warps that join in
// shared memory: 66 us).
constexpr int kSlab = 16, kStages = 3;
template <typename T>
constexpr float kLift = std::is_same<T, __half>::value ? 7.f : 0.f;   // of the weights, in units of log2

template <int D>
constexpr int row_smem() {
    return kStages * 2 * kSlab * D * 2;
}
template <int D>
constexpr int row_resident() {   // warps per SM that the launch plans for
    return D == 128 ? 9 : 14;
}

template <typename T, int D, bool kSmallPages>   // small: less than a slab, which else lies on one page
__global__ void __launch_bounds__(32, row_resident<D>()) attn_suffix_kernel(const AttnArgs a) {
    extern __shared__ __align__(128) uint8_t smem[];
    const mmq_shared_prefix_attention_t& p = a.p;
    T* const tag = nullptr;
    if (!a.beside) griddep_wait();
    // Beside a prefix kernel, which was launched (and has seen to it that what
    // precedes the call is complete) but need not have ended: only the last CTA
    // waits for it, at its end, so that this grid's end is also the prefix
    // kernel's for the join.  A wait in every CTA would hold their SMs' room.
    const bool last = a.beside && blockIdx.x == gridDim.x - 1 &&
                      blockIdx.y == gridDim.y - 1 && blockIdx.z == gridDim.z - 1;
    const int lane = threadIdx.x;
    const int h = blockIdx.y, G = a.group;
    const int tiles_per_token = (G + 15) / 16;

    // Rows [r0, r1) and keys [k0, k1) of this warp.
    const int t = int(blockIdx.x) / tiles_per_token, tile = int(blockIdx.x) - t * tiles_per_token;
    const int b = t / p.q_len;
    const int64_t r0 = int64_t(t) * G + tile * 16, r1 = min(r0 + 16, int64_t(t) * G + G);
    const int32_t* pages = p.page_table + b * p.table_width;
    const int64_t room = p.table_width << a.page_shift;
    int64_t len = p.lens[b];
    if (len > room) {
        if (lane == 0) atomicCAS(a.status, 0, MMQ_ERR_ARG);
        len = room;
    }
    len = max(int64_t(0), len - p.q_len + 1 + (t - b * p.q_len));
    const int64_t share = ((len + a.suffix_parts - 1) / a.suffix_parts + 63) & ~int64_t(63);
    const int64_t k0 = min(int64_t(blockIdx.z) * share, len), k1 = min(k0 + share, len);
    const int part = a.prefix_parts + int(blockIdx.z);
    const int64_t part_row = int64_t(part) * a.tokens;
    const int grow = lane >> 2, gcol = lane & 3;
    auto token_head = [&](int64_t r) {   // row r's place among [tokens][heads]
        const int64_t t = r / G;
        return t * p.heads + int64_t(h) * G + (r - t * G);
    };

    if (k0 >= k1) {
        if (lane < 16 && r0 + lane < r1) a.part_ml[part_row * p.heads + token_head(r0 + lane)] = make_float2(-INFINITY, 0.f);
        if (last) griddep_wait();
        return;
    }

    const uint32_t ring = smem_u32(smem);
    constexpr uint32_t kHalfStage = kSlab * D * 2;
    constexpr int kChunks = D / 8;                 // 16-byte chunks of a row
    constexpr int kRowsAtOnce = 32 / kChunks;
    const int slabs = int((k1 - k0 + kSlab - 1) / kSlab);
    bool bad_page = false;

    const T* const keys = static_cast<const T*>(p.k_cache);
    const T* const values = static_cast<const T*>(p.v_cache);
    const int64_t step = int64_t(p.kv_heads) * D;   // from key to key
    const int64_t head = int64_t(h) * D + (lane % kChunks) * 8;
    const int64_t in_page = (int64_t(1) << a.page_shift) - 1;
    int32_t next_id = kSmallPages ? 0 : pages[k0 >> a.page_shift];   // the next slab's page

    // Slab i's rows: kRowsAtOnce rows of 16-byte chunks per instruction, chunk
    // c of row r at c ^ (r & 7) (conflict-free for ldmatrix).
    auto fetch = [&](int i, int stage) {
        const int64_t first = k0 + int64_t(i) * kSlab;
        int left = int(min(k1 - first, int64_t(kSlab)));   // rows to read
        int64_t at = first;                                 // the first row's place in the cache
        if (!kSmallPages) {
            const int32_t id = next_id;
            if (id < 0 || id >= p.n_pages) {
                bad_page = true;
                left = 0;
            }
            at = (int64_t(id) << a.page_shift) + (first & in_page);
            const int64_t then = first + kSlab;
            if (then < k1) next_id = pages[then >> a.page_shift];
        }
        const uint32_t base = ring + uint32_t(stage) * 2 * kHalfStage;
#pragma unroll
        for (int j = 0; j < kSlab / kRowsAtOnce; ++j) {
            const int r = j * kRowsAtOnce + lane / kChunks;
            bool valid = r < left;
            int64_t row = at + r;
            if (kSmallPages && valid) {
                const int32_t id = pages[(first + r) >> a.page_shift];
                if (id < 0 || id >= p.n_pages) {
                    bad_page = true;
                    valid = false;
                }
                row = (int64_t(id) << a.page_shift) + ((first + r) & in_page);
            }
            const int64_t off = row * step + head;
            const uint32_t dst = base + uint32_t(r * D * 2 + (((lane % kChunks) ^ (r & 7)) << 4));
            const T* none = static_cast<const T*>(p.q);   // an invalid row is filled with zeros, nothing is read
            cp_async16(dst, valid ? keys + off : none, valid);
            cp_async16(dst + kHalfStage, valid ? values + off : none, valid);
        }
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) {
        if (s < slabs) fetch(s, s);
        cp_async_commit();
    }

    // Query fragments: rows grow and grow + 8, zero past r1.
    uint32_t qf[D / 16][4];
    {
        const int64_t ra = r0 + grow, rb = ra + 8, ta = ra / G, tb = rb / G;
        const T* qa = static_cast<const T*>(p.q) + ta * p.q_stride + (int64_t(h) * G + (ra - ta * G)) * D;
        const T* qb = static_cast<const T*>(p.q) + tb * p.q_stride + (int64_t(h) * G + (rb - tb * G)) * D;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const int c = kk * 16 + 2 * gcol;
            qf[kk][0] = ra < r1 ? *reinterpret_cast<const uint32_t*>(qa + c) : 0u;
            qf[kk][1] = rb < r1 ? *reinterpret_cast<const uint32_t*>(qb + c) : 0u;
            qf[kk][2] = ra < r1 ? *reinterpret_cast<const uint32_t*>(qa + c + 8) : 0u;
            qf[kk][3] = rb < r1 ? *reinterpret_cast<const uint32_t*>(qb + c + 8) : 0u;
        }
    }

    float o[D / 8][4];
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[n][k] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    const int m = lane >> 3, r7 = lane & 7;
    const uint32_t krow = uint32_t(((m >> 1) * 8 + r7) * D * 2), vrow = uint32_t(((m & 1) * 8 + r7) * D * 2);

    int stage = 0;
    for (int i = 0; i < slabs; ++i) {
        cp_async_wait<kStages - 2>();
        __syncwarp();   // slab i is here, and every lane is done with the stage before it
        if (i + kStages - 1 < slabs) fetch(i + kStages - 1, stage == 0 ? kStages - 1 : stage - 1);
        cp_async_commit();
        const uint32_t kb = ring + uint32_t(stage) * 2 * kHalfStage, vb = kb + kHalfStage;
        float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            uint32_t b[4];
            ldmatrix4(b, kb + krow + uint32_t(((kk * 2 + (m & 1)) ^ r7) << 4));
            mma16816(s0, qf[kk], b[0], b[1], tag);
            mma16816(s1, qf[kk], b[2], b[3], tag);
        }
        float x[8] = {s0[0], s0[1], s1[0], s1[1], s0[2], s0[3], s1[2], s1[3]};
        const int left = int(min(k1 - k0 - int64_t(i) * kSlab, int64_t(kSlab)));
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int key = (k & 2 ? 8 : 0) + 2 * gcol + (k & 1);
            x[k] = key < left ? __fmul_rn(x[k], a.scale_log2) : -INFINITY;
        }
        float t0 = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), t1 = fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7]));
        t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 1));
        t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 1));
        t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 2));
        t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 2));
        const float n0 = fmaxf(m0, t0), n1 = fmaxf(m1, t1);
        if (__any_sync(0xffffffffu, n0 > m0 || n1 > m1)) {
            // (-inf) - (-inf) only where the sums are still zero; m - kLift as it is rounded below
            const float f0 = n0 == -INFINITY ? 1.f : ex2((m0 - kLift<T>) - (n0 - kLift<T>));
            const float f1 = n1 == -INFINITY ? 1.f : ex2((m1 - kLift<T>) - (n1 - kLift<T>));
            l0 *= f0;
            l1 *= f1;
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
                o[n][0] *= f0; o[n][1] *= f0;
                o[n][2] *= f1; o[n][3] *= f1;
            }
            m0 = n0;
            m1 = n1;
        }
        const float b0 = m0 == -INFINITY ? 0.f : m0 - kLift<T>, b1 = m1 == -INFINITY ? 0.f : m1 - kLift<T>;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            x[k] = ex2(x[k] - b0);
            x[k + 4] = ex2(x[k + 4] - b1);
        }
        l0 += (x[0] + x[1]) + (x[2] + x[3]);
        l1 += (x[4] + x[5]) + (x[6] + x[7]);
        const uint32_t pf[4] = {pack16(x[0], x[1], tag), pack16(x[4], x[5], tag), pack16(x[2], x[3], tag),
                                pack16(x[6], x[7], tag)};
#pragma unroll
        for (int dc = 0; dc < D / 16; ++dc) {
            uint32_t b[4];
            ldmatrix4_trans(b, vb + vrow + uint32_t(((dc * 2 + (m >> 1)) ^ r7) << 4));
            mma16816(o[2 * dc], pf, b[0], b[1], tag);
            mma16816(o[2 * dc + 1], pf, b[2], b[3], tag);
        }
        if (++stage == kStages) stage = 0;
    }
    cp_async_wait<0>();
    if (bad_page) atomicCAS(a.status, 0, MMQ_ERR_ARG);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int64_t r = r0 + grow + 8 * half;
        if (r >= r1) continue;
        const int64_t at = part_row * p.heads + token_head(r);
        float* dst = a.part_o + at * D + 2 * gcol;
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
            *reinterpret_cast<float2*>(dst + n * 8) = make_float2(o[n][2 * half], o[n][2 * half + 1]);
        if (gcol == 0) a.part_ml[at] = half ? make_float2(m1 - kLift<T>, l1) : make_float2(m0 - kLift<T>, l0);
    }
    if (last) griddep_wait();
}

// ------------------------------------------------------------------- join
// kWarpsPerRow warps per (token, head).  The parts' (m, l), one part per lane,
// give the maximum and each part's factor; then the parts' sums, the warps
// taking parts in turn with up to eight loads in flight each; parts without
// keys are not read.  Bound by the latency of those three steps where rows are
// few: 34 parts of 128 rows take one warp per row 10.5 us.
constexpr int kJoinWarps = 8;
__device__ __forceinline__ void store_out(void* out, int type, int64_t at, float x, float y) {
    if (type == MMQ_TYPE_F32)
        *reinterpret_cast<float2*>(static_cast<float*>(out) + at) = make_float2(x, y);
    else if (type == MMQ_TYPE_F16)
        *reinterpret_cast<uint32_t*>(static_cast<__half*>(out) + at) = pack16(x, y, static_cast<__half*>(nullptr));
    else
        *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(out) + at) =
            pack16(x, y, static_cast<__nv_bfloat16*>(nullptr));
}

template <int D, int kWarpsPerRow>
__global__ void __launch_bounds__(kJoinWarps * 32) attn_join_kernel(const AttnArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    if (a.suffix_parts == 0) {   // an empty page table: no suffix kernel says that a length is past it
        const int64_t b = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;   // at least one thread per sequence
        if (b < a.p.batch && a.p.lens[b] > 0) atomicCAS(a.status, 0, MMQ_ERR_ARG);
    }
    constexpr int kVec = D / 32;   // values per lane
    __shared__ float sums[kWarpsPerRow > 1 ? kJoinWarps : 1][kVec][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, turn = warp % kWarpsPerRow;
    const int64_t rows = a.tokens * a.p.heads;
    const int64_t row = int64_t(blockIdx.x) * (kJoinWarps / kWarpsPerRow) + warp / kWarpsPerRow;
    const int parts = row < rows ? a.prefix_parts + a.suffix_parts : 0;
    const float2 none = make_float2(-INFINITY, 0.f);
    const float2 ml0 = lane < parts ? a.part_ml[lane * rows + row] : none;
    float m = ml0.x;
    for (int i = lane + 32; i < parts; i += 32) m = fmaxf(m, a.part_ml[i * rows + row].x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    float l = 0.f, acc[kVec] = {};
    for (int first = 0; first < parts; first += 32) {
        const int n = min(32, parts - first);
        const float2 ml = first == 0 ? ml0 : lane < n ? a.part_ml[(first + lane) * rows + row] : none;
        const float mine = ml.y == 0.f ? 0.f : ex2(ml.x - m);   // l = 0: no keys
        l = fmaf(mine, ml.y, l);
        const uint32_t has = __ballot_sync(0xffffffffu, ml.y != 0.f);
        constexpr int kFlight = kWarpsPerRow == 1 ? 4 : 8;
        for (int i0 = turn; i0 < n; i0 += kFlight * kWarpsPerRow) {
            float v[kFlight][kVec];
#pragma unroll
            for (int q = 0; q < kFlight; ++q) {
                const int i = i0 + q * kWarpsPerRow;
                const float* src = a.part_o + (int64_t(first + i) * rows + row) * D + kVec * lane;
#pragma unroll
                for (int k = 0; k < kVec; ++k) v[q][k] = 0.f;
                if (i < n && ((has >> i) & 1u)) {
                    if (kVec == 4) {
                        const float4 u = *reinterpret_cast<const float4*>(src);
                        v[q][0] = u.x; v[q][1] = u.y; v[q][2] = u.z; v[q][kVec - 1] = u.w;
                    } else {
                        const float2 u = *reinterpret_cast<const float2*>(src);
                        v[q][0] = u.x; v[q][kVec - 1] = u.y;
                    }
                }
            }
#pragma unroll
            for (int q = 0; q < kFlight; ++q) {
                const float f = __shfl_sync(0xffffffffu, mine, (i0 + q * kWarpsPerRow) & 31);
#pragma unroll
                for (int k = 0; k < kVec; ++k) acc[k] = fmaf(f, v[q][k], acc[k]);
            }
        }
    }
    if (kWarpsPerRow > 1) {
#pragma unroll
        for (int k = 0; k < kVec; ++k) sums[warp][k][lane] = acc[k];
        __syncthreads();
        if (turn != 0) return;
#pragma unroll
        for (int k = 0; k < kVec; ++k)
#pragma unroll
            for (int w = 1; w < kWarpsPerRow; ++w) acc[k] += sums[warp + w][k][lane];
    }
    if (row >= rows) return;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    const float r = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int k = 0; k < kVec; k += 2)
        store_out(a.p.out, a.p.out_type, row * D + kVec * lane + k, acc[k] * r, acc[k + 1] * r);
}

// A kernel of this call that follows another: it may be scheduled before the
// other ends, and waits for it (griddep_wait) before it touches memory.
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

// Parts for `units` independent pieces of up to `keys` keys each, on `slots`
// resident warps: enough to give every slot a piece, none shorter than `least`.
int split(int64_t units, int64_t keys, int64_t slots, int64_t least) {
    if (keys <= 0) return 0;
    int64_t n = (slots + units - 1) / units;
    const int64_t most = (keys + least - 1) / least;
    if (n > most) n = most;
    if (n > 64) n = 64;
    return int(n < 1 ? 1 : n);
}

// The prefix kernel's row tiles per CTA: two, one of them empty for up to 128
// rows, but for few rows one, the two groups taking key tiles in turn.  (8192
// keys of 8 kv heads x 128: 32 rows 15.2 us with one, 15.7 with two; 64 rows
// 17.6 and 16.9; 128 rows 23.9 and 20.7, where twice as many parts and twice the
// bytes per time cost more than the empty tile; 24 rows, 4096 keys of 32 kv heads x
// 64: 17.1 and 20.2.)
int prefix_tiles(int64_t rows) { return rows <= 48 ? 1 : 2; }

// And its parts: `units` row blocks over `keys` key tiles each.  Estimated in
// units of 1.7 us, the time of a key tile for two row tiles: with one it is half
// of that; every item takes about four more for its queries, first scores and
// results; the kernel writes and the join reads `part` bytes per part, 6.8 MB per
// unit; and the suffix kernel, which follows but starts on the SMs that have no
// item, reads about 140 KB per unit and SM there and 60 KB per SM with all.
// (256 sequences, 1024 rows per kv head x 16384 keys: 122 us with 2 parts, 104 with
// the 3 this gives, 113 with 4.)
int64_t prefix_parts(int tiles, int64_t units, int64_t keys, int64_t nsm, double part, double suffix) {
    int64_t best = 1;
    double least = 1e300;
    for (int64_t n = 1; n <= keys && n <= 64; ++n) {
        const int64_t rounds = (units * n + nsm - 1) / nsm, each = (keys + n - 1) / n;
        const double prefix = double(rounds) * (double(tiles == 2 ? each : (each + 1) / 2) + 4.);
        const double idle = rounds == 1 ? double(nsm - units * n) : 0.;
        const double left = suffix - idle * prefix * 140e3;
        const double cost = prefix + (left > 0. ? left / (double(nsm) * 60e3) : 0.) + part * double(n) / 6.8e6;
        if (cost < least) {
            least = cost;
            best = n;
        }
    }
    return best;
}

void plan(AttnArgs& a, int nsm) {
    const mmq_shared_prefix_attention_t& p = a.p;
    a.tokens = int64_t(p.batch) * p.q_len;
    a.group = p.heads / p.kv_heads;
    a.scale_log2 = p.scale * 1.4426950408889634f;
    a.beside = p.prefix > 0;
    a.page_shift = 0;
    while ((1 << a.page_shift) < p.page_size) ++a.page_shift;
    const int64_t slots = int64_t(nsm) * (p.head_dim == 128 ? row_resident<128>() : row_resident<64>());
    a.prefix_tiles = 0;
    a.prefix_parts = 0;
    a.part_keys = 0;
    if (p.prefix > 0) {
        const int64_t rows = a.tokens * a.group;
        a.prefix_tiles = prefix_tiles(rows);
        const int per_item = a.prefix_tiles == 1 ? 2 : 1;   // parts
        // on average a suffix fills half of its pages
        const double suffix = 2. * double(a.tokens) * double(p.table_width << a.page_shift) * p.kv_heads * p.head_dim;
        const double part = 8. * double(a.tokens) * p.heads * p.head_dim * per_item;   // written and read
        const int64_t n = prefix_parts(a.prefix_tiles, (rows + 128 * a.prefix_tiles - 1) / (128 * a.prefix_tiles) * p.kv_heads,
                                       (p.prefix + 127) / 128, nsm, part, suffix);
        a.part_keys = ((p.prefix + n - 1) / n + 127) / 128 * 128;
        a.prefix_parts = int((p.prefix + a.part_keys - 1) / a.part_keys) * per_item;
    }
    // ragged suffixes: several warps per slot, so that the longest do not end last alone
    a.suffix_parts = split(a.tokens * ((a.group + 15) / 16) * p.kv_heads, p.table_width << a.page_shift, 3 * slots, 64);
}

size_t ml_bytes(const AttnArgs& a) {
    const size_t n = size_t(a.prefix_parts + a.suffix_parts) * size_t(a.tokens) * size_t(a.p.heads) * sizeof(float2);
    return (n + 255) & ~size_t(255);
}

template <typename T, int D>
cudaError_t launch(const AttnArgs& a, int nsm, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    cudaError_t e;
    bool first = true;
    auto config = [&](dim3 grid, dim3 block, size_t smem) {
        const bool f = first;
        first = false;
        return f ? mmq::launch_config(grid, block, smem, s, attr) : follow_config(grid, block, smem, s, attr);
    };
    constexpr int smem = row_smem<D>();
    if (a.prefix_parts) {
        const cudaLaunchConfig_t cfg = config(dim3(1), dim3(1), 0);
        if ((e = mmq::launch_attention_prefix(a, nsm, cfg))) return e;
    }
    if (a.suffix_parts) {
        auto* kernel = a.p.page_size >= kSlab ? attn_suffix_kernel<T, D, false> : attn_suffix_kernel<T, D, true>;
        const dim3 grid(unsigned(a.tokens * ((a.group + 15) / 16)), unsigned(a.p.kv_heads), unsigned(a.suffix_parts));
        const cudaLaunchConfig_t cfg = config(grid, dim3(32), smem);
        if ((e = cudaLaunchKernelEx(&cfg, kernel, a))) return e;
    }
    // Many parts of few rows: the parts of a row over four warps.
    const bool many = a.prefix_parts + a.suffix_parts > 8;
    const int64_t each = many ? kJoinWarps / 4 : kJoinWarps;
    const cudaLaunchConfig_t cfg = config(dim3(unsigned((a.tokens * a.p.heads + each - 1) / each)), dim3(kJoinWarps * 32), 0);
    return many ? cudaLaunchKernelEx(&cfg, attn_join_kernel<D, 4>, a) : cudaLaunchKernelEx(&cfg, attn_join_kernel<D, 1>, a);
}

}  // namespace

namespace mmq {

size_t shared_prefix_attention_workspace(const mmq_shared_prefix_attention_t& p) {
    const int nsm = sm_count();
    if (!nsm) return 0;
    AttnArgs a;
    a.p = p;
    plan(a, nsm);
    const size_t need = ml_bytes(a) + size_t(a.prefix_parts + a.suffix_parts) * size_t(a.tokens) * size_t(p.heads) *
                                          size_t(p.head_dim) * sizeof(float);
    return need ? need : 256;   // no prefix and no page: no parts, but 0 stands for an error
}

cudaError_t launch_shared_prefix_attention(const mmq_shared_prefix_attention_t& p, void* workspace, int* status,
                                           int inject_timeout, cudaStream_t s) {
    const int nsm = sm_count();
    if (!nsm) return cudaErrorInvalidDevice;
    AttnArgs a;
    a.p = p;
    plan(a, nsm);
    a.status = status;
    a.inject = inject_timeout;
    a.part_ml = static_cast<float2*>(workspace);
    a.part_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + ml_bytes(a));
    if (p.type == MMQ_TYPE_F16) return p.head_dim == 64 ? launch<__half, 64>(a, nsm, s) : launch<__half, 128>(a, nsm, s);
    return p.head_dim == 64 ? launch<__nv_bfloat16, 64>(a, nsm, s) : launch<__nv_bfloat16, 128>(a, nsm, s);
}

}  // namespace mmq
