// Attention of a ragged batch over a 4-bit paged cache: few rows per sequence.
//
// With k the codes less 8, d the scales, g the blocks of 32 dimensions of a head:
//   s_t = f sum_g dk_tg sum_{x in g} q'_x k_tx      q' = 2^e q as fp16, f = scale log2(e) 2^-e
//   out = sum_t 2^(s_t - m) dv_t k_t / sum_t 2^(s_t - m)
// in parts joined by their references m and sums, as in attention.cu.
//
// Rows are the (new token, head of the group) pairs of one kv head, R = 8 NT of
// them to a unit, which needs every step of 32 keys (two tiles) that its last
// row sees.  All units' steps, one after the other, are cut into equal runs, one per warp:
// ragged lengths and few long sequences fill the machine alike.  A warp's run
// may hold the end of one unit, some whole ones and the start of another; parts
// of a unit that lie in one CTA join in shared memory, those over several in
// the workspace, joined by a second kernel.
//
// Per tile a warp takes two products on the tensor cores with 16 x 16 blocks of
// codes as the A operand: S^T = K Q^T and O^T = V^T P^T, whose 8 columns are the
// rows, so that a group of up to 8 heads fills a product that would be half
// empty with rows as M.  The cache's bytes are in the A operand's order: a tile
// is one asynchronous bulk copy into the warp's own ring, and a lane's words
// need masks only.
//   Keys: a code masked out of its word is an fp16 subnormal, n 2^-24 (or 2^-20
//   from the upper nibble, for which q' is 2^-4 times smaller), and the block's
//   scale multiplies the f32 sum.  The 8 is taken off in one more product,
//   scales times -8 sum q' of their blocks: a scale, of at most eight
//   significant bits, is a bfloat16, and each f32 sum is three of them.  (By
//   value: float16's bits shifted by three are not, where it is subnormal.)  q'
//   has its row's largest element in [2^13, 2^14): nothing of a bfloat16's or
//   float16's eleven bits is lost down to 2^-23 of it, and of what is smaller no
//   more than 2^-34 of it.
//   Values: (n - 8) d, exact in fp16, because here the scale's index is summed
//   over.  kFine (float16 queries, float32 results): weights are the sum of two
//   fp16 values (22 bits, 2^-25 of the reference at worst), a product each; one
//   alone would double the error of a float16 result.  For a bfloat16 result,
//   rounded eight times as coarsely, one is taken.  The sum of weights is that of
//   the float32 ones either way.
// The reference m of a row starts kLift (in log2) under its first largest score
// and is raised when a score is more than kSpan above it: weights stay below
// 2^14, and what they lose in fp16 is small against the largest.
//
// Bound: a decode step of 64 sequences of up to 32k tokens, 8 heads of keys,
// reads 1.26 GB in 221 us, 5.7 TB/s, 84 % of a copy's rate (float16 results: 251
// us, for their second product).  There the warps' instructions bound it as much
// as memory does: what cut instructions cut time (347 us at first; 250 with
// scales by pairs of tiles, the offset by a product and steps of two tiles; 233
// with fewer stores and pages looked up ahead; the rest by runs of equal time).  Short
// sequences pay for the chain of loads that each unit starts with: 256 of up to
// 512 tokens take 42 us, 12 of them their bytes'.  Four warps to a CTA, three
// CTAs to an SM for eight rows, two for sixteen; a ring of three or four steps
// for each warp.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "half_ops.cuh"
#include "kv4_attention.cuh"
#include "mmq_internal.h"
#include "sm103_ptx.cuh"
#include "tc_common.cuh"

namespace {

using namespace mmq::ptx;
using namespace mmq::kv4;
using mmq::tc::ld_shared_v4;
using mmq::up256;

__device__ __align__(16) const uint8_t zero_tile[tile_bytes(128)] = {};   // of a page that does not exist
constexpr int kWarps = 4;
constexpr int kStep = 2 * kTokens;   // keys that a warp takes at a time
constexpr float kLift = 7.f, kSpan = 14.f;   // a row's reference is 7 (in log2) under its largest score at first, 14 at most
constexpr float kNone = -3.402823466e38f;   // the reference before any score: no score is under it but -Inf
// Steps' time that a unit costs whatever its length: the chain of its first loads takes 5000 to 8000 cycles and its results'
// stores as many, a step 2600.  Units as long as their steps alone: 256 sequences of up to 512 tokens 66 us, and 46; of 3, 7
// and 12 in place of 5: 47, 46 and 45, but 64 sequences of 32k tokens 228, 226 and 229, and 226 by 5.
constexpr int kIdle = 5;
constexpr int kLeast = 2;   // steps to a run, where there are too few for all warps

// mma16816 without an accumulator, and with bfloat16 operands.
__device__ __forceinline__ void mma16816_0(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma16816_bf16_0(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// (v & mask) | bits
__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t mask, uint32_t bits) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(v), "r"(mask), "r"(bits));
    return d;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
    return d;
}

// Two float16 of at most eight significant bits as bfloat16, exactly.
__device__ __forceinline__ uint32_t bf16_of(uint32_t v) {
    const float2 f = __half22float2(u2h(v));
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t*>(&b);
}

// ------------------------------------------------------------------ output
__device__ __forceinline__ void store_value(void* out, int type, int64_t at, float x) {
    if (type == MMQ_TYPE_F32) static_cast<float*>(out)[at] = x;
    else if (type == MMQ_TYPE_F16) static_cast<__half*>(out)[at] = __float2half_rn(x);
    else static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(x);
}

template <int D, int NT>
struct Rows {
    static constexpr int R = 8 * NT;
    static constexpr int kRegs = D / 16 * 4 * NT;         // accumulators per lane
    static constexpr int kPart = kRegs * 32 + 2 * R;      // floats of a part: sums [reg][lane], then m, l [row]
    static constexpr int kCtas = NT == 1 ? 3 : 2;         // per SM
    static constexpr int kStages = D == 128 && NT == 1 ? 3 : 4;   // steps of two tiles
    static constexpr int kRing = kStages * 2 * tile_bytes(D); // a warp's; its last part lies over it
    static constexpr int kOffFirst = kWarps * kRing;      // and its first part here
    static constexpr int kOffBar = kOffFirst + kWarps * kPart * 4;
    static constexpr int kBytes = kOffBar + kWarps * kStages * 8;
    static_assert(kRing >= kPart * 4 && kRing % 16 == 0, "a part fits the ring");
    static_assert(kCtas * (kBytes + 2048) <= 228 * 1024, "shared memory");
};

// Register k = (block i, half of 16 dimensions, column) of lane: its dimension and row.
template <int NT>
__device__ __forceinline__ void element(int k, int lane, int& dim, int& row) {
    const int nt = (k >> 2) % NT, i = (k >> 2) / NT;
    dim = 16 * i + 8 * ((k >> 1) & 1) + (lane >> 2);
    row = 8 * nt + 2 * (lane & 3) + (k & 1);
}

// Where a unit's row goes, in values; -1 past its sequence's last.
template <int D, int R>
__device__ __forceinline__ int64_t out_row(const Kv4Args& a, const Unit& u, const Sequence& s, int row) {
    const int r = u.tile * R + row, j = r / a.group;
    return j < s.n ? ((s.start + j) * a.p.heads + u.h * a.group + (r - j * a.group)) * D : -1;
}

// Parts of one unit, added up by a CTA: a thread has some registers of its lane, all of one row.
template <int D, int NT>
struct Join {
    using W = Rows<D, NT>;
    static constexpr int kMine = W::kRegs / kWarps, kSame = kWarps / 2 / NT;   // warps of the same row
    static_assert(kSame >= 1, "a row per thread");
    float acc[kMine] = {}, m = kNone, l = 0.f;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = warp & 1, nt = (warp >> 1) % NT, rest = (warp >> 1) / NT;
    const int row = 8 * nt + 2 * (lane & 3) + col;

    __device__ __forceinline__ int reg(int i) const {   // as element() has it
        const int c = rest + kSame * i;
        return 4 * ((c >> 1) * NT + nt) + 2 * (c & 1) + col;
    }
    __device__ __forceinline__ void add(const float* part) {
        const float pm = part[W::kRegs * 32 + row], pl = part[W::kRegs * 32 + W::R + row];
        if (pl == 0.f) return;   // no key
        const float top = fmaxf(m, pm);
        const float mine = ex2(m - top), its = ex2(pm - top);
        m = top;
        l = l * mine + pl * its;
#pragma unroll
        for (int i = 0; i < kMine; ++i) acc[i] = acc[i] * mine + part[reg(i) * 32 + lane] * its;
    }
    __device__ __forceinline__ void finish(const Kv4Args& a, const Unit& u, const Sequence& s) const {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int64_t out = out_row<D, W::R>(a, u, s, row);
        if (out < 0) return;
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            int dim, same;
            element<NT>(reg(i), lane, dim, same);
            store_value(a.p.out, a.p.out_type, out + dim, acc[i] * inv);
        }
    }
    __device__ __forceinline__ void keep(const Kv4Args& a, int64_t part) const {
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            int dim, same;
            element<NT>(reg(i), lane, dim, same);
            a.parts[(part * W::R + row) * D + dim] = acc[i];
        }
        if (lane < 4 && rest == 0)
            reinterpret_cast<float2*>(a.parts + int64_t(gridDim.x) * 2 * W::R * D)[part * W::R + row] = make_float2(m, l);
    }
};

// ------------------------------------------------------------------ kernel
// kFine: weights as two fp16 values, for a result that shows it.
template <typename T, int D, int NT, bool kFine>
__global__ void __launch_bounds__(kWarps * 32, Rows<D, NT>::kCtas) kv4_rows_kernel(const Kv4Args a) {
    using W = Rows<D, NT>;
    constexpr int R = W::R, kStages = W::kStages, kGroups = D / 32;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ struct {
        int64_t total[kWarps];
        int64_t first[kWarps + 1];      // where each warp's run starts, and the next CTA's first
        int b[kWarps + 1];              // the sequence it lies in
        int64_t offset[kWarps + 1];     // and its place there
        // the parts of each warp, its first and its last: the unit's name or -1, whether it starts and ends there
        int64_t name[2 * kWarps];
        int whole[2 * kWarps];          // bit 0: starts, bit 1: ends
        Unit unit[2 * kWarps];
        uint32_t aborted;
    } sh;
    static_assert(sizeof(sh) <= 1024, "counted in Rows");
    const mmq_kv4_attention_t& p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r8 = lane >> 2, c4 = lane & 3;
    const AbortFlag abort_flag{smem_u32(&sh.aborted)};
    const uint32_t ring = smem_u32(smem) + uint32_t(warp * W::kRing);
    const uint32_t bars = smem_u32(smem) + uint32_t(W::kOffBar + warp * kStages * 8);

    if (lane == 0)
        for (int i = 0; i < kStages; ++i) mbar_init(bars + 8u * uint32_t(i), 2);
    if (threadIdx.x == 0) sh.aborted = 0;
    if (threadIdx.x < 2 * kWarps) sh.name[threadIdx.x] = -1;
    fence_barrier_init();
    griddep_launch_dependents();
    griddep_wait();

    // ---- who does what: a scan over the sequences
    const int per = (p.batch + kWarps * 32 - 1) / (kWarps * 32);
    const int b0 = min(p.batch, int(threadIdx.x) * per), b1 = min(p.batch, b0 + per);
    auto length_of = [&](const Sequence& s) {   // of one head
        return int64_t(s.n) * a.group > a.few ? 0 : head_length<R, kStep, kIdle>(s, a.group);
    };
    int64_t mine = 0, total;
    for (int b = b0; b < b1; ++b) mine += length_of(sequence(a, b, blockIdx.x == 0)) * p.kv_heads;
    const int64_t x1 = cta_scan<kWarps>(mine, sh.total, total), x0 = x1 - mine;
    const Runs runs(total, max(int64_t(1), min(int64_t(gridDim.x) * kWarps, total / kLeast)));
    for (int w = 0; w <= kWarps; ++w) {
        const int64_t at = runs.start(int64_t(blockIdx.x) * kWarps + w);
        if (threadIdx.x == 0 && at >= total) sh.first[w] = total;
        if (x0 <= at && at < x1) {   // of one thread
            int64_t x = x0;
            for (int b = b0; b < b1; ++b) {
                const Sequence s = sequence(a, b, false);
                const int64_t each = length_of(s);
                if (at < x + each * p.kv_heads) {
                    const int moved = cut<R, kStep, kIdle>(s, a.group, each, at - x).moved;
                    sh.first[w] = at - moved;
                    sh.b[w] = b;
                    sh.offset[w] = at - moved - x;
                    break;
                }
                x += each * p.kv_heads;
            }
        }
    }
    __syncthreads();

    // ---- this warp's run
    int64_t at = sh.first[warp];
    const int64_t end = sh.first[warp + 1];
    int b = at < end ? sh.b[warp] : 0;
    int64_t offset = at < end ? sh.offset[warp] : 0;
    auto part_at = [&](int slot) {
        return reinterpret_cast<float*>(smem + (slot & 1 ? (slot >> 1) * W::kRing : W::kOffFirst + (slot >> 1) * W::kPart * 4));
    };
    int stage = 0, fill = 0, flying = 0;   // the ring's next step to take, to fill, and those under way
    uint32_t phase = 0;
    const bool inject = a.inject && at == 0 && end > 0;   // test hook: the first copies never come
    bool withheld = inject;
    bool ok = true, bad_page = false;
    // The masks are kernel arguments so that they stay in registers: an instruction takes one constant, the other bits.
    const uint32_t low = a.low, high = a.high;   // 0x000F000F, 0x00F000F0
    float o[W::kRegs / 4][4];
    float m[NT][2], l[NT][2];      // of rows 2 c, 2 c + 1

    while (at < end && ok) {
        const Sequence s = sequence(a, b, false);
        const int64_t each = length_of(s);
        if (offset >= each * p.kv_heads) {   // also a sequence without rows
            ++b;
            offset = 0;
            continue;
        }
        const Cut from = cut<R, kStep, kIdle>(s, a.group, each, offset);   // not moved: it has been, or is a unit's start
        const Unit u{b, from.h, from.u};
        const int length = unit_length<R, kStep, kIdle>(s, a.group, u.tile), upto = int(min(int64_t(length), from.in + (end - at)));
        const int t0 = max(0, from.in - kIdle), t1 = upto - kIdle;
        const int64_t name = at - from.in;   // the unit's place
        const int row0 = u.tile * R;   // first row of the unit

        const int most = min(unit_keys<R>(s, a.group, u.tile), t1 * kStep);   // that the unit's last row sees of these
        const int least = min(seen(s, row0 / a.group), t1 * kStep);           // and its first
        const int last = min(t1, (most + kStep - 1) / kStep);   // steps with a key
        // Copies, of two tiles a step.  Lanes 2 i and 2 i + 1 have the places of step i of the next 16 and issue its copies.
        const int32_t* const table = p.page_table + int64_t(b) * p.table_width;
        const int tile_shift = a.page_shift - 4;
        const uint8_t* src = zero_tile;
        int next = t0;
        int32_t ahead = -1;            // the page of this lane's tile of the 16 steps after those
        auto page_of = [&](int step) {
            const int tile = 2 * step + lane;
            return tile * kTokens < most ? table[tile >> tile_shift] : -1;
        };
        auto fetch = [&]() {
            const int i = (next - t0) & 15;
            if (i == 0) {
                const int tile = 2 * next + lane;
                const int32_t id = next == t0 ? page_of(next) : ahead;
                const bool good = id >= 0 && id < p.n_pages;
                src = zero_tile;
                if (good)
                    src = p.cache + (((int64_t(id) * p.kv_heads + u.h) << tile_shift) + (tile & ((1 << tile_shift) - 1))) * tile_bytes(D);
                bad_page |= !good && tile * kTokens < most;
            } else if (i == 8) {
                ahead = page_of(next + 8);
            }
            const uint32_t bar = bars + 8u * uint32_t(fill), dst = ring + uint32_t(fill * 2 * tile_bytes(D)) + uint32_t(lane & 1) * tile_bytes(D);
            if (lane >> 1 == i && !withheld) {
                mbar_arrive_expect_tx(bar, tile_bytes(D));
                bulk_load(dst, src, tile_bytes(D), bar);
            }
            withheld = false;
            fill = fill + 1 == kStages ? 0 : fill + 1;
            ++flying;
            ++next;
        };
        // Queries: lane's row is r8 (of each eight), its dimensions 2 c, 2 c + 1 and those + 8 of every 16.  On their way
        // beside the pages' numbers.
        uint32_t raw[NT][D / 16][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = row0 + 8 * nt + r8, j = row / a.group;
            const bool has = j < s.n;
            const T* src = static_cast<const T*>(p.q) + (s.start + (has ? j : 0)) * p.q_stride +
                           (int64_t(u.h) * a.group + (has ? row - j * a.group : 0)) * D + 2 * c4;
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k) raw[nt][i][k] = has ? *reinterpret_cast<const uint32_t*>(src + 16 * i + 8 * k) : 0u;
        }
        for (int i = 0; i < kStages - 1 && next < last; ++i) fetch();

        uint32_t qf[NT][D / 16][2];
        uint32_t qs[NT][2];            // -8 sum q' of each block, as an operand
        float f[NT][2];
        int see[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int j = (row0 + 8 * nt + r8) / a.group;
            const bool has = j < s.n;
            float x[D / 16][4];
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                const uint32_t lo = raw[nt][i][0], hi = raw[nt][i][1];
                if (std::is_same<T, __half>::value) {
                    const float2 u0 = __half22float2(u2h(lo)), u1 = __half22float2(u2h(hi));
                    x[i][0] = u0.x; x[i][1] = u0.y; x[i][2] = u1.x; x[i][3] = u1.y;
                } else {
                    x[i][0] = __uint_as_float(lo << 16); x[i][1] = __uint_as_float(lo & 0xFFFF0000u);
                    x[i][2] = __uint_as_float(hi << 16); x[i][3] = __uint_as_float(hi & 0xFFFF0000u);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) top = fmaxf(top, fabsf(x[i][k]));
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // top in [2^e, 2^(e+1)) -> [2^13, 2^14); a row of zeros or tiny values as if it had 2^-100
            const int e = max(-100, int((__float_as_uint(top) >> 23) & 0xFF) - 127);
            const float up = __uint_as_float(uint32_t(127 + 13 - e) << 23);
            float sum[kGroups];
#pragma unroll
            for (int g = 0; g < kGroups; ++g) sum[g] = 0.f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                const __half2 v0 = __floats2half2_rn(x[i][0] * up, x[i][1] * up);
                const __half2 v1 = __floats2half2_rn(x[i][2] * up * 0.0625f, x[i][3] * up * 0.0625f);
                qf[nt][i][0] = h2u(v0);
                qf[nt][i][1] = h2u(v1);
                const float2 w0 = __half22float2(v0), w1 = __half22float2(v1);
                sum[i / 2] += (w0.x + w0.y) + 16.f * (w1.x + w1.y);
            }
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 1);
                sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 2);
                sum[g] *= -8.f * 0x1p-24f;
            }
            // As three bfloat16 each, in the order in which take() has the scales: of 16 places, lane c has 2 c, 2 c + 1
            // (first word) and those + 8 (second), the scales of blocks 2 c, 2 c + 1 modulo their number.
            uint32_t part[3][kGroups / 2];
#pragma unroll
            for (int k = 0; k < 3; ++k)
#pragma unroll
                for (int g = 0; g < kGroups; g += 2) {
                    const __nv_bfloat162 v = __floats2bfloat162_rn(sum[g], sum[g + 1]);
                    sum[g] -= __low2float(v);
                    sum[g + 1] -= __high2float(v);
                    part[k][g / 2] = *reinterpret_cast<const uint32_t*>(&v);
                }
            if (D == 128) {
                const uint32_t one = c4 & 1 ? part[0][kGroups / 2 - 1] : part[0][0], two = c4 & 1 ? part[1][kGroups / 2 - 1] : part[1][0];
                qs[nt][0] = c4 & 2 ? two : one;
                qs[nt][1] = c4 & 2 ? 0u : c4 & 1 ? part[2][kGroups / 2 - 1] : part[2][0];
            } else {
                qs[nt][0] = c4 == 0 ? part[0][0] : c4 == 1 ? part[1][0] : c4 == 2 ? part[2][0] : 0u;
                qs[nt][1] = 0u;
            }
            // The products carry 2^-24 from the codes.  Held below infinity: all scores of the row are too large by
            // then for it to matter, but zeros stay zeros.
            const float mine_f = fminf(a.scale_log2 * __uint_as_float(uint32_t(127 + e - 13) << 23) * 0x1p24f, 3.4e38f);
            const int mine_see = has ? min(seen(s, j), t1 * kStep) : 0;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int from = (2 * c4 + k) * 4;
                f[nt][k] = __shfl_sync(0xffffffffu, mine_f, from);
                see[nt][k] = __shfl_sync(0xffffffffu, mine_see, from);
                m[nt][k] = kNone;
                l[nt][k] = 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < W::kRegs / 4; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) o[i][k] = 0.f;

        // One step; kRagged: not all rows see all of it.
        auto take = [&](int t, auto ragged) {
            constexpr bool kRagged = decltype(ragged)::value;
            const uint32_t base = ring + uint32_t(stage * 2 * tile_bytes(D));
            stage = stage + 1 == kStages ? 0 : stage + 1;
            phase ^= stage == 0 ? 1u : 0u;
            --flying;
            if (next < last) fetch();   // into the step's before this one, whose words the products have taken

            // ---- scores of tokens r8, r8 + 8 of each tile against rows 2 c, 2 c + 1
            float y[2][NT][4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t at = base + uint32_t(j * tile_bytes(D));
                uint32_t kw[D / 16], ks[kGroups];   // ks: blocks of token r8, then of r8 + 8, two to a word
#pragma unroll
                for (int i = 0; i < D / 64; ++i) {
                    const uint4 w = ld_shared_v4(at + uint32_t(512 * i + 16 * lane));
                    kw[4 * i] = w.x; kw[4 * i + 1] = w.y; kw[4 * i + 2] = w.z; kw[4 * i + 3] = w.w;
                }
                const uint32_t from = at + uint32_t(key_scales(D) + r8 * (D / 8));
                if (D == 128) {
                    const uint4 w = ld_shared_v4(from);
                    ks[0] = w.x; ks[1] = w.y; ks[kGroups / 2] = w.z; ks[kGroups - 1] = w.w;
                } else {
                    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(ks[0]), "=r"(ks[1]) : "r"(from) : "memory");
                }
                // What the codes' 8 takes off: the scales, as bfloat16, times the blocks' sums.
                {
                    const uint32_t w0 = D == 128 && (c4 & 1) ? ks[kGroups / 2 - 1] : ks[0];
                    const uint32_t w1 = D == 128 && (c4 & 1) ? ks[kGroups - 1] : ks[kGroups / 2];
                    const uint32_t d0 = bf16_of(w0), d1 = bf16_of(w1);
                    const uint32_t A[4] = {d0, d1, d0, d1};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma16816_bf16_0(y[j][nt], A, qs[nt][0], qs[nt][1]);
                }
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    float acc[NT][4];
#pragma unroll
                    for (int i = 2 * g; i < 2 * g + 2; ++i) {
                        const uint32_t w8 = kw[i] >> 8;
                        const uint32_t A[4] = {kw[i] & low, w8 & low, kw[i] & high, w8 & high};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            if (i % 2 == 0) mma16816_0(acc[nt], A, qf[nt][i][0], qf[nt][i][1]);
                            else mma16816(acc[nt], A, qf[nt][i][0], qf[nt][i][1]);
                        }
                    }
                    const float2 lo = __half22float2(u2h(ks[g / 2])), hi = __half22float2(u2h(ks[kGroups / 2 + g / 2]));
                    const float d0 = g & 1 ? lo.y : lo.x, d1 = g & 1 ? hi.y : hi.x;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int k = 0; k < 4; ++k) y[j][nt][k] = fmaf(k & 2 ? d1 : d0, acc[nt][k], y[j][nt][k]);
                }
            }
            bool rises = false;
            float top[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        y[j][nt][k] = __fmul_rn(y[j][nt][k], f[nt][k & 1]);
                        if (kRagged && t * kStep + kTokens * j + r8 + (k & 2 ? 8 : 0) >= see[nt][k & 1]) y[j][nt][k] = -INFINITY;
                    }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    top[nt][k] = fmaxf(fmaxf(y[0][nt][k], y[0][nt][k + 2]), fmaxf(y[1][nt][k], y[1][nt][k + 2]));
                    rises |= top[nt][k] - m[nt][k] > kSpan;   // exact where it matters, however large they are
                }
            }
            if (__any_sync(0xffffffffu, rises)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float now = fmaxf(top[nt][k], __shfl_xor_sync(0xffffffffu, top[nt][k], 4));
                        now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, 8));
                        now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, 16));
                        now = fmaxf(m[nt][k], now - kLift);
                        const float by = ex2(m[nt][k] - now);
                        m[nt][k] = now;
                        l[nt][k] *= by;
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {
                            o[i * NT + nt][k] *= by;
                            o[i * NT + nt][k + 2] *= by;
                        }
                    }
            }
            // ---- weights, as the B operand: tokens 2 c, 2 c + 1 and those + 8 of row r8
            uint32_t hi[2][NT][2], lo[2][NT][2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float* const x = y[j][nt];
#pragma unroll
                    for (int k = 0; k < 4; ++k) x[k] = ex2(__fsub_rn(x[k], m[nt][k & 1]));
                    l[nt][0] += x[0] + x[2];
                    l[nt][1] += x[1] + x[3];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const __half2 v = __floats2half2_rn(x[2 * k], x[2 * k + 1]);
                        const float2 back = __half22float2(v);
                        hi[j][nt][k] = transpose8x8(h2u(v));
                        if (kFine) {
                            const __half2 rest = __floats2half2_rn(x[2 * k] - back.x, x[2 * k + 1] - back.y);
                            lo[j][nt][k] = transpose8x8(h2u(rest));
                        }
                    }
                }

            // ---- values
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t at = base + uint32_t(j * tile_bytes(D));
                uint32_t vs[kGroups][2];   // scales of tokens 2 c, 2 c + 1 and those + 8
#pragma unroll
                for (int g = 0; g < kGroups; g += 2) {
                    const uint4 w = ld_shared_v4(at + uint32_t(value_scales(D) + c4 * (D / 4) + 8 * g));
                    vs[g][0] = w.x; vs[g][1] = w.y; vs[g + 1][0] = w.z; vs[g + 1][1] = w.w;
                }
                const int first = t * kStep + kTokens * j;
                uint32_t off[kGroups];   // ragged steps: tokens whose scale is no number, as bits
                bool any_off = false;
                if (kRagged) {
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) {
                        off[g] = 0;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int token = 2 * c4 + (k & 1) + (k & 2 ? 8 : 0);
                            const uint32_t bits = k & 1 ? vs[g][k >> 1] >> 16 : vs[g][k >> 1] & 0xFFFFu;
                            const bool past = first + token >= most;
                            if (past || !finite16(bits)) vs[g][k >> 1] &= k & 1 ? 0x0000FFFFu : 0xFFFF0000u;
                            if (!past && !finite16(bits)) off[g] |= 1u << token;
                        }
                        off[g] |= __shfl_xor_sync(0xffffffffu, off[g], 1);
                        off[g] |= __shfl_xor_sync(0xffffffffu, off[g], 2);
                        any_off |= off[g] != 0;
                    }
                }
                const __half2 bias_lo = __float2half2_rn(1032.f), bias_hi = __float2half2_rn(72.f);
#pragma unroll
                for (int i4 = 0; i4 < D / 64; ++i4) {
                    const uint4 v = ld_shared_v4(at + uint32_t(value_codes(D) + 512 * i4 + 16 * lane));
                    const uint32_t word[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int i = 4 * i4; i < 4 * i4 + 4; ++i) {
                        const uint32_t w = word[i % 4], w8 = w >> 8;
                        const __half2 d0 = u2h(vs[i / 2][0]), d1 = u2h(vs[i / 2][1]);
                        const uint32_t A[4] = {h2u(__hmul2(__hsub2(u2h(and_or(w, low, 0x64006400u)), bias_lo), d0)),
                                               h2u(__hmul2(__hsub2(u2h(and_or(w, high, 0x54005400u)), bias_hi), d0)),
                                               h2u(__hmul2(__hsub2(u2h(and_or(w8, low, 0x64006400u)), bias_lo), d1)),
                                               h2u(__hmul2(__hsub2(u2h(and_or(w8, high, 0x54005400u)), bias_hi), d1))};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            if (kFine) mma16816(o[i * NT + nt], A, lo[j][nt][0], lo[j][nt][1]);
                            mma16816(o[i * NT + nt], A, hi[j][nt][0], hi[j][nt][1]);
                        }
                    }
                }
                if (kRagged && any_off) {   // such a token's block is no number for the rows that see it, and only for them
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int n = min(16, max(0, see[nt][k] - first));
                            const uint32_t sees = (1u << n) - 1u;
#pragma unroll
                            for (int i = 0; i < D / 16; ++i)
                                if (off[i / 2] & sees) o[i * NT + nt][k] = o[i * NT + nt][k + 2] = __int_as_float(0x7FC00000);
                        }
                }
            }
        };
        for (int t = t0; t < last; ++t) {
            ok = __all_sync(0xffffffffu, wait_bounded(bars + 8u * uint32_t(stage), phase, abort_flag, a.status));
            if (!ok) break;
            if (t * kStep + kStep > least) take(t, std::true_type{});
            else take(t, std::false_type{});
        }
        if (!ok) break;

#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[nt][k] += __shfl_xor_sync(0xffffffffu, l[nt][k], d);

        at += upto - from.in;
        offset += upto - from.in;
        const bool starts = t0 == 0, ends = upto == length;
        if (starts && ends) {
            float inv[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int k = 0; k < 2; ++k) inv[nt][k] = l[nt][k] == 0.f ? 0.f : 1.f / l[nt][k];
            for (int nt = 0; nt < NT; ++nt) {
                if (p.out_type == MMQ_TYPE_F32) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int64_t out = out_row<D, R>(a, u, s, 8 * nt + 2 * c4 + k);
                        if (out < 0) continue;
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {
                            static_cast<float*>(p.out)[out + 16 * i + r8] = o[i * NT + nt][k] * inv[nt][k];
                            static_cast<float*>(p.out)[out + 16 * i + 8 + r8] = o[i * NT + nt][k + 2] * inv[nt][k];
                        }
                    }
                    continue;
                }
                // 8 x 8 blocks turned round: row r8, dimensions 2 c, 2 c + 1
                const int64_t out = out_row<D, R>(a, u, s, 8 * nt + r8);
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const float x = o[i * NT + nt][2 * half] * inv[nt][0], y = o[i * NT + nt][2 * half + 1] * inv[nt][1];
                        uint32_t w;
                        if (std::is_same<T, __half>::value) {
                            w = h2u(__floats2half2_rn(x, y));
                        } else {
                            const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
                            w = *reinterpret_cast<const uint32_t*>(&v);
                        }
                        w = transpose8x8(w);
                        if (out >= 0) *reinterpret_cast<uint32_t*>(static_cast<T*>(p.out) + out + 16 * i + 8 * half + 2 * c4) = w;
                    }
            }
            continue;
        }
        // A part of a unit: the warp's last, or its first.
        const int slot = 2 * warp + (at == end ? 1 : 0);
        float* const part = part_at(slot);
#pragma unroll
        for (int k = 0; k < W::kRegs; ++k) part[k * 32 + lane] = o[k >> 2][k & 3];
        if (r8 == 0)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    part[W::kRegs * 32 + 8 * nt + 2 * c4 + k] = m[nt][k];
                    part[W::kRegs * 32 + R + 8 * nt + 2 * c4 + k] = l[nt][k];
                }
        if (lane == 0) {
            sh.name[slot] = name;
            sh.whole[slot] = (starts ? 1 : 0) | (ends ? 2 : 0);
            sh.unit[slot] = u;
        }
    }
    if (bad_page) atomicCAS(a.status, 0, MMQ_ERR_ARG);
    // After a wait that ran out: the copies still in flight.
    for (bool never = inject; flying > 0; --flying, never = false) {
        if (!never) wait_drain(bars + 8u * uint32_t(stage), phase, a.status);
        stage = stage + 1 == kStages ? 0 : stage + 1;
        phase ^= stage == 0 ? 1u : 0u;
    }
    __syncthreads();

    // ---- units of several warps: joined, finished or left for the join over CTAs
    Mark mark{-1, 0, 0, 0};
    if (!abort_flag.raised()) {
        for (int i = 0; i < 2 * kWarps;) {
            if (sh.name[i] < 0) {
                ++i;
                continue;
            }
            const int64_t name = sh.name[i];
            int upto = i + 1, ends = sh.whole[i] & 2;
            for (int j = i + 1; j < 2 * kWarps; ++j)
                if (sh.name[j] == name) {
                    upto = j + 1;
                    ends = sh.whole[j] & 2;
                } else if (sh.name[j] >= 0) {
                    break;
                }
            const bool starts = sh.whole[i] & 1;
            const Unit u = sh.unit[i];
            Join<D, NT> join;
            for (int j = i; j < upto; ++j)
                if (sh.name[j] >= 0) join.add(part_at(j));
            if (starts && ends) {
                join.finish(a, u, sequence(a, u.b, false));
            } else {
                join.keep(a, int64_t(blockIdx.x) * 2 + (starts ? 1 : 0));
                if (starts) {
                    const int64_t end = name + unit_length<R, kStep, kIdle>(sequence(a, u.b, false), a.group, u.tile);
                    mark = Mark{int(runs.of(end - 1) / kWarps), u.b, u.h, u.tile};
                }
            }
            i = upto;
        }
    }
    if (threadIdx.x == 0) a.marks[blockIdx.x] = mark;
}

// Units of several runs: blocks (i, *) join the one that starts in run i and does not end there.  kShare: a block per
// row, whose warps share the row's parts (one sequence of 32k tokens has 57 of them); else a warp per row, eight rows.
constexpr int kJoinRows = 8;
template <int D, bool kShare>
__global__ void __launch_bounds__(kJoinRows * 32) kv4_join_kernel(const Kv4Args a, int R) {
    constexpr int kVec = D / 32, kFlight = 4;
    __shared__ float sums[kShare ? kJoinRows : 1][D + 1];
    griddep_launch_dependents();
    griddep_wait();
    const Mark mark = a.marks[blockIdx.x];
    if (mark.last < 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Sequence s = sequence(a, mark.b, false);
    const float2* const mls = reinterpret_cast<const float2*>(a.parts + int64_t(gridDim.x) * 2 * R * D);
    const int parts = mark.last - int(blockIdx.x) + 1;
    auto at = [&](int k) { return (k == 0 ? int64_t(blockIdx.x) * 2 + 1 : (int64_t(blockIdx.x) + k) * 2) * R; };   // of row 0
    // Row `row`'s parts first, first + step, ...: their weighted sum, from the row's reference on
    auto gather = [&](int row, int first, int step, float (&acc)[kVec], float& l) {
        float m = kNone;
        for (int k = lane; k < parts; k += 32) {
            const float2 ml = mls[at(k) + row];
            if (ml.y != 0.f) m = fmaxf(m, ml.x);   // else no key
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        l = 0.f;
#pragma unroll
        for (int k = 0; k < kVec; ++k) acc[k] = 0.f;
        for (int k0 = first; k0 < parts; k0 += kFlight * step) {
            float v[kFlight][kVec];
            float2 ml[kFlight];
#pragma unroll
            for (int f = 0; f < kFlight; ++f) {
                const int k = k0 + f * step;
                ml[f] = make_float2(kNone, 0.f);
#pragma unroll
                for (int c = 0; c < kVec; ++c) v[f][c] = 0.f;
                if (k < parts) {
                    ml[f] = mls[at(k) + row];
#pragma unroll
                    for (int c = 0; c < kVec; c += 2) {
                        const float2 u = *reinterpret_cast<const float2*>(a.parts + (at(k) + row) * D + kVec * lane + c);
                        v[f][c] = u.x;
                        v[f][c + 1] = u.y;
                    }
                }
            }
#pragma unroll
            for (int f = 0; f < kFlight; ++f) {
                if (ml[f].y == 0.f) continue;
                const float by = ex2(ml[f].x - m);
                l = fmaf(by, ml[f].y, l);
#pragma unroll
                for (int c = 0; c < kVec; ++c) acc[c] = fmaf(by, v[f][c], acc[c]);
            }
        }
    };
    auto store = [&](int row, const float (&acc)[kVec], float l) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int64_t r = int64_t(mark.tile) * R + row, j = r / a.group;
        const int64_t out = ((s.start + j) * a.p.heads + mark.h * a.group + (r - j * a.group)) * D + kVec * lane;
#pragma unroll
        for (int c = 0; c < kVec; ++c) store_value(a.p.out, a.p.out_type, out + c, acc[c] * inv);
    };
    const int64_t rows = int64_t(s.n) * a.group - int64_t(mark.tile) * R;   // of the unit, from its first on
    float acc[kVec], l;
    const int row = kShare ? int(blockIdx.y) : int(blockIdx.y) * kJoinRows + warp;
    if (row >= rows) return;   // the whole block, if it shares
    gather(row, kShare ? warp : 0, kShare ? kJoinRows : 1, acc, l);
    if (kShare) {
#pragma unroll
        for (int c = 0; c < kVec; ++c) sums[warp][kVec * lane + c] = acc[c];
        if (lane == 0) sums[warp][D] = l;
        __syncthreads();
        if (warp) return;
        for (int w = 1; w < kJoinRows; ++w) {
            l += sums[w][D];
#pragma unroll
            for (int c = 0; c < kVec; ++c) acc[c] += sums[w][kVec * lane + c];
        }
    }
    store(row, acc, l);
}

// A ragged batch of more than eight tokens a sequence on average, which is taken to hold chunks, and single tokens beside.
bool mixed(const mmq_kv4_attention_t& p) { return p.q_starts && p.tokens > int64_t(8) * p.batch; }

// Eight rows to a unit where a sequence has no more on average, else sixteen.  33 sequences of 5001 tokens, four heads of
// keys: seven rows 27 us, and 31 by units of sixteen; 14 rows 37 by twice as many units of eight, and 33.  64 sequences of
// 32k tokens: four rows 221 and 308, sixteen 424 and 310.  Beside chunks the others are taken to have one token: 60 of 4096
// tokens, four rows, and two chunks of 500: 105 and 116.
bool narrow(const mmq_kv4_attention_t& p) {
    const int64_t group = p.heads / p.kv_heads;
    return p.tokens * group <= int64_t(8) * p.batch || (mixed(p) && group <= 8);
}

template <int D, int NT>
size_t part_bytes(int nsm) {
    return up256(size_t(nsm) * Rows<D, NT>::kCtas * 2 * Rows<D, NT>::R * (D + 2) * 4);
}
size_t part_bytes(const mmq_kv4_attention_t& p, int nsm) {
    if (p.head_dim == 64) return narrow(p) ? part_bytes<64, 1>(nsm) : part_bytes<64, 2>(nsm);
    return narrow(p) ? part_bytes<128, 1>(nsm) : part_bytes<128, 2>(nsm);
}

template <typename T, int D, int NT>
cudaError_t launch(const Kv4Args& a, int nsm, cudaStream_t s) {
    using W = Rows<D, NT>;
    const bool fine = std::is_same<T, __half>::value || a.p.out_type == MMQ_TYPE_F32;
    auto* kernel = fine ? kv4_rows_kernel<T, D, NT, true> : kv4_rows_kernel<T, D, NT, std::is_same<T, __half>::value>;
    cudaError_t e;
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, W::kBytes))) return e;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = mmq::launch_config(dim3(unsigned(nsm * W::kCtas)), dim3(kWarps * 32), W::kBytes, s, attr);
    if ((e = cudaLaunchKernelEx(&cfg, kernel, a))) return e;
    return mmq::launch_kv4_join(a, W::R, nsm * W::kCtas, s);
}
template <typename T, int D>
cudaError_t launch(const Kv4Args& a, int nsm, cudaStream_t s) {
    return narrow(a.p) ? launch<T, D, 1>(a, nsm, s) : launch<T, D, 2>(a, nsm, s);
}

}  // namespace

namespace {

struct Forms {
    bool few, many, two;   // which kernels a call may need; two: units of 256 rows
    int most_few;          // a sequence of up to so many rows is the few-row kernel's
};
Forms forms(const mmq_kv4_attention_t& p) {
    const int64_t group = p.heads / p.kv_heads, rows = p.tokens * group;   // of all sequences
    const int64_t most = p.q_starts ? rows : rows / p.batch;               // of one, at most
    // 33 sequences of 5001 tokens, four heads of keys, alike: 21 rows 47 us by two units of sixteen and 54 by the other
    // kernel, 28 rows 48 and 56, 35 rows 60 and 54.  A ragged batch costs the time of two kernels where it has rows for
    // both: 48 sequences of 8192 tokens, one to eight new ones, four rows each, 143 us cut at 16 rows, 136 at 24, 123 at 40
    // (and 170 by the other kernel alone); 33 of 5001, one to five, seven rows each, 68, 68, 60 (and 62).  So where the
    // average tells that most are few, the cut is high.  Around that border (one to eleven or twelve new ones, four rows
    // each, 24 or 26 on average) little depends on it: of 8192 tokens 145 us cut at 16 and 141 at 40, of 2000 tokens 74
    // and 77.
    const bool mostly_few = rows <= int64_t(24) * p.batch;
    const int most_few = p.q_starts ? mostly_few ? 40 : 16 : 24;
    // 256 rows: chunks of 2047 tokens 556 us, and 924 by units of 128; 64 tokens of 8 sequences, 256 rows each, 57 and 85.
    // Up to 128 rows: 128 rows 89 us, and 90 by a unit of 256 that is half empty; 35 rows 54 and 65.  Two chunks of 500
    // tokens beside 60 single ones: 105 and 131.
    const bool two = rows > int64_t(128) * p.batch || mixed(p);
    return Forms{p.q_starts || most <= most_few, most > most_few, two, most_few};
}
size_t all_part_bytes(const mmq_kv4_attention_t& p, int nsm) {
    const Forms f = forms(p);
    const size_t few = f.few ? part_bytes(p, nsm) : 0, many = f.many ? up256(mmq::kv4_attention_tc_part_bytes(p.head_dim, nsm)) : 0;
    return few > many ? few : many;
}
constexpr int kMostRuns = 3;   // marks per SM, of either kernel

}  // namespace

namespace mmq {

cudaError_t launch_kv4_join(const Kv4Args& a, int R, int runs, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // it waits for the kernel before it
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.stream = s;
    // Many parts to a unit (its share of the runs), so that a warp alone would take them one after the other: one sequence
    // of 32k tokens 25 us, and 34 by a warp per row.  Else a warp per row is the faster: 33 sequences of one to five
    // tokens 64 us shared and 60 not, 64 of 32k tokens 224 and 222.
    const bool share = R <= 16 && int64_t(a.p.batch) * a.p.kv_heads * 4 <= runs;
    cfg.gridDim = dim3(unsigned(runs), unsigned(share ? R : R / kJoinRows));
    cfg.blockDim = dim3(kJoinRows * 32);
    if (a.p.head_dim == 64)
        return share ? cudaLaunchKernelEx(&cfg, kv4_join_kernel<64, true>, a, R) : cudaLaunchKernelEx(&cfg, kv4_join_kernel<64, false>, a, R);
    return share ? cudaLaunchKernelEx(&cfg, kv4_join_kernel<128, true>, a, R) : cudaLaunchKernelEx(&cfg, kv4_join_kernel<128, false>, a, R);
}

size_t kv4_attention_workspace(const mmq_kv4_attention_t& p) {
    const int nsm = sm_count();
    return nsm ? all_part_bytes(p, nsm) + up256(size_t(nsm) * kMostRuns * sizeof(Mark)) : 0;
}

cudaError_t launch_kv4_attention(const mmq_kv4_attention_t& p, void* workspace, int* status, int inject_timeout,
                                 cudaStream_t s) {
    const int nsm = sm_count();
    if (!nsm) return cudaErrorInvalidDevice;
    Kv4Args a;
    a.p = p;
    a.parts = static_cast<float*>(workspace);
    a.marks = reinterpret_cast<Mark*>(static_cast<char*>(workspace) + all_part_bytes(p, nsm));
    a.status = status;
    a.inject = inject_timeout;
    a.page_shift = 0;
    while ((1 << a.page_shift) < p.page_size) ++a.page_shift;
    a.group = p.heads / p.kv_heads;
    a.each = p.batch ? int(p.tokens / p.batch) : 0;
    a.scale_log2 = p.scale * 1.4426950408889634f;
    a.low = 0x000F000Fu;
    a.high = 0x00F000F0u;
    const Forms f = forms(p);
    a.few = f.most_few;
    if (f.few) {
        cudaError_t e;
        if (p.type == MMQ_TYPE_F16) e = p.head_dim == 64 ? launch<__half, 64>(a, nsm, s) : launch<__half, 128>(a, nsm, s);
        else e = p.head_dim == 64 ? launch<__nv_bfloat16, 64>(a, nsm, s) : launch<__nv_bfloat16, 128>(a, nsm, s);
        if (e || !f.many) return e;
    }
    cudaLaunchAttribute attr[1];
    return launch_kv4_attention_tc(a, f.two, nsm, mmq::launch_config(dim3(1), dim3(1), 0, s, attr));
}

}  // namespace mmq
