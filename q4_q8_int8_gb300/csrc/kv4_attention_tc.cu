// Attention over a 4-bit paged cache on the tensor cores: sequences with many
// rows (a chunk of a prompt, or a speculative step of a wide group).
//
// A unit is 128 or 256 rows of one sequence's kv head.  Per tile of 64 keys it
// takes two products of 128 rows x 64 keys x D for each 128 rows, S = Q K^T and
// O += P V with P = 2^(S f - m) as fp16, the rest f32; the keys and values, (code
// - 8) * scale, are exact in fp16, so that P's rounding is the only one beside the
// result's.  A 16-bit result takes one fp16 value per weight, which a float16 one
// shows (its error 2.9e-4 of the norm, 2.1e-4 its own rounding); a float32 result
// takes two (kFine: 22 bits, what is left of P over the other half of S, with a
// product of its own; 653 us in place of 513 for the chunks below).  Q is fp16: a bfloat16 row with its largest element in [2^13,
// 2^14), of which fp16 loses nothing down to 2^-28 of it, and 2^-e in f.
//
// One CTA per SM:
//   warps 0-3, 4-7  softmax groups 0 and 1, thread = row (its tensor-memory
//                   lane): read S, keep the row's maximum and sum, write P over
//                   S, now and then scale O
//   warps 8-11      expand raw keys to operand tiles (128-byte swizzle), [key][dimension]
//   warps 12-15     and raw values, transposed, [dimension][key]
//   warp 16         fetches raw tiles: one to four bulk copies for 64 keys, by the page's size
//   warps 17, 18    MMA issuers of groups 0 and 1
//   warp 19         tells the others which pieces of units their run has
// Runs of equal length of all units' key tiles are the CTAs' work, as in the
// few-row kernel; the parts of units that lie in several runs are joined by a
// second kernel.  kTwo: 256 rows to a unit, both groups share each key tile,
// expanded once.  Else 128 rows, and each group has a run of its own.
//
// S has two buffers: a group's softmax works on one tile while the next one's
// product is made.  What is expanded goes to a slot each for keys and for
// values, so that the two are not tied to one another.
//
// Bound: neither rate.  Chunks of up to 3 x 2047 tokens over up to 12k (32 heads, 8
// of keys, D = 128) take 519 us, 1160 TFLOP/s, 61 % of the products' measured
// rate.  A tile's chain, scores to softmax to product, is longer than the
// products of both groups; with the exponentials or the expansion left out it
// was hardly faster: what the roles wait for one another bounds it.  Few rows (33
// sequences, 35 rows, 5001 tokens: 54 us) pay for the expansion of every key
// with products that are a quarter full.  What steps gave, on three chunks of 2047
// tokens each, which take 554 us with all of them: products issued by lane 0 in
// place of an elected thread, 649 us and 582.  Tiles of 128
// keys with one buffer of scores: 706 us and 704, and 87 and 70 for the few rows,
// before that; keys and values expanded by one warpgroup: 706 and 693 then.  Two
// raw slots: the same as three.  The maximum of a tile's first half beside the
// load of its second, 577 us and 556; its weights beside the maximum, 553 and 559,
// but 70.7 and 69.8 for 64 rows of 16 sequences.
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
using namespace mmq::tc;
using namespace mmq::kv4;

constexpr int kKeys = 64, kRows = 128;   // keys of a tile
constexpr int kThreads = 640;
constexpr int kWarpExpand = 8, kWarpFetch = 16, kWarpMma = 17;   // and kWarpMma + 1; four expand keys, four values
// Registers: 96 per thread at launch (the launcher checks it): 256 x 144 + 256 x 64 + 128 x 64 = 640 x 96.
constexpr uint32_t kRegsLaunch = 96, kRegsSoftmax = 144, kRegsExpand = 64, kRegsOther = 64;
static_assert(256 * kRegsSoftmax + 256 * kRegsExpand + 128 * kRegsOther <= kThreads * kRegsLaunch, "register split");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;   // S_g at 128 g and 64 on, in turn (P over its first 32 columns), O_g at 256 + 128 g
constexpr float kGrow = 8.f, kLift = 7.f;    // P at most 2^15
constexpr float kNone = -3.402823466e38f;    // the maximum before any score
constexpr float kWide = 0x1p20f;
__device__ __forceinline__ float reference(float m) { return fabsf(m) < kWide ? m - kLift : m; }

__device__ __align__(16) const uint8_t zero_tiles[kKeys / kTokens * tile_bytes(128)] = {};   // of a page that does not exist

// Tiles' time that a unit costs whatever its length.  256 rows, chunks of 512 tokens: 291 us with 5, 288 with 8, 290 and 292
// with 10 and 12 (371 with none and 335 with 8, before products were issued as they are now).  128 rows, 33 sequences of 35
// rows: 54 to 56 with 3 to 6 (70 with none and 61 with 4, before).
__host__ __device__ constexpr int idle(int R) { return R > kRows ? 8 : 4; }

// Where a run starts in the layout and where the next does, and in it: place t of unit u of head h of sequence b.
struct Start {
    int64_t first, end;
    int b, h, u, t;
};

// A run's units one after the other, each with the places [t, t1) that the run has of it.
template <int R>
struct Walk {
    const Kv4Args& a;
    int64_t left, name;   // length after this piece; the unit's place
    Sequence s;
    int b, h, u, t, t1, length;

    __device__ __forceinline__ Walk(const Kv4Args& args, const Start& from) : a(args) {
        left = from.end - from.first;
        b = from.b;
        h = from.h;
        u = from.u;
        t = t1 = from.t;
        name = from.first - from.t;
        if (left > 0) {
            s = sequence(a, b, false);
            begin(from.t);
        }
    }
    __device__ __forceinline__ bool valid() const { return t < t1; }
    __device__ __forceinline__ int first_tile() const { return max(0, t - idle(R)); }
    __device__ __forceinline__ int end_tile() const { return t1 - idle(R); }
    __device__ __forceinline__ bool starts() const { return t == 0; }
    __device__ __forceinline__ bool ends() const { return t1 == length; }
    __device__ __forceinline__ int most() const { return unit_keys<R>(s, a.group, u); }     // keys that its last row sees
    __device__ __forceinline__ int least() const { return seen(s, u * R / a.group); }       // and its first
    __device__ __forceinline__ void begin(int from) {
        length = unit_length<R, kKeys, idle(R)>(s, a.group, u);
        t = from;
        t1 = int(min(int64_t(length), from + left));
        left -= t1 - t;
    }
    __device__ __forceinline__ void next() {   // the next piece
        t = t1;
        if (left == 0) return;
        name += length;
        if (++u == units<R>(s, a.group)) {
            u = 0;
            if (++h == a.p.kv_heads) {
                h = 0;
                do s = sequence(a, ++b, false);
                while (int64_t(s.n) * a.group <= a.few);
            }
        }
        begin(0);
    }
};

// What the roles are told of a piece: tiles [t0, t1) of a unit; none: the run's end.
struct Piece {
    int64_t start;                   // the sequence's first row of q
    int b, h, u, t0, t1, starts, ends;
    int last;                        // the run that the unit ends in
    int n, len, most, least;         // of the sequence; keys that the unit's last and first row see
};
constexpr int kPieces = 4;           // told ahead

template <int D, bool kTwo>
struct Layout {
    static constexpr int kStreams = kTwo ? 1 : 2;
    static constexpr int kTile = kKeys * D * 2;              // of keys or values as fp16
    static constexpr int kQ = kRows * D * 2;
    static constexpr int kSlots = 1024 / D;
    static constexpr int kBufs = kSlots / 2 / kStreams;      // per stream, of keys and of values
    static constexpr int kRaw = kKeys / kTokens * tile_bytes(D);   // a tile's keys and values in 4 bits
    static constexpr int kRawSlots = 384 / D;
    static constexpr int kOffQ = 0;
    static constexpr int kOffSlots = 2 * kQ;
    static constexpr int kOffRaw = kOffSlots + kSlots * kTile;
    static constexpr int kOffSums = kOffRaw + kRawSlots * kRaw;
    static constexpr int kOffStart = kOffSums + (kThreads / 32) * 8;
    static constexpr int kOffPieces = kOffStart + 2 * int(sizeof(Start));
    static constexpr int kOffBar = kOffPieces + 2 * kPieces * int(sizeof(Piece));
    // barriers: raw_full, raw_empty; full, empty per slot; q_full per group, o_done, s_full, p_full per group and
    // buffer; drain; told, done per piece
    static constexpr int kOffMisc = kOffBar + (2 * kRawSlots + 2 * kSlots + 15 + 4 * kPieces) * 8;
    static constexpr int kBytes = kOffMisc + 32 + 1024;
    static constexpr int kR = kTwo ? 2 * kRows : kRows;      // rows of a unit
};
static_assert(Layout<128, true>::kBytes <= 232448 && Layout<128, false>::kBytes <= 232448, "shared memory budget");

__device__ __forceinline__ uint32_t pack16(float a, float b) { return h2u(__floats2half2_rn(a, b)); }
// What pack16 left of them.
__device__ __forceinline__ uint32_t rest16(float a, float b, uint32_t packed) {
    const float2 back = __half22float2(u2h(packed));
    return pack16(a - back.x, b - back.y);
}
// Two codes in the lower nibbles, or the upper ones, of v's bytes 0 and 2, less 8, times the scales.
__device__ __forceinline__ uint32_t expand_low(uint32_t v, uint32_t scales) {
    uint32_t d;
    asm("lop3.b32 %0, %1, 0x000F000F, 0x64006400, 0xEA;" : "=r"(d) : "r"(v));
    return h2u(__hmul2(__hsub2(u2h(d), __float2half2_rn(1032.f)), u2h(scales)));
}
__device__ __forceinline__ uint32_t expand_high(uint32_t v, uint32_t scales) {
    uint32_t d;
    asm("lop3.b32 %0, %1, 0x00F000F0, 0x54005400, 0xEA;" : "=r"(d) : "r"(v));
    return h2u(__hmul2(__hsub2(u2h(d), __float2half2_rn(72.f)), u2h(scales)));
}
// One thread of the warp, always the same one.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}
template <int N>
__device__ __forceinline__ void ld_shared_words(uint32_t addr, uint32_t* w) {
    if (N == 2) asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr) : "memory");
    else w[0] = ld_shared_u32(addr);
}

// kFine: weights as two fp16 values, for a float32 result.
template <typename T, int D, bool kTwo, bool kFine>
__global__ void __launch_bounds__(kThreads, 1) kv4_tc_kernel(const Kv4Args a) {
    using L = Layout<D, kTwo>;
    constexpr int kSlots = L::kSlots, kRawSlots = L::kRawSlots, kStreams = L::kStreams, kBufs = L::kBufs, kR = L::kR;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar0 = sbase + L::kOffBar;
    auto raw_full = [&](int s) { return bar0 + 8u * uint32_t(s); };
    auto raw_empty = [&](int s) { return bar0 + 8u * uint32_t(kRawSlots + s); };
    auto full = [&](int s) { return bar0 + 8u * uint32_t(2 * kRawSlots + s); };
    auto empty = [&](int s) { return bar0 + 8u * uint32_t(2 * kRawSlots + kSlots + s); };
    const uint32_t bar1 = bar0 + 8u * uint32_t(2 * kRawSlots + 2 * kSlots);
    auto q_full = [&](int g) { return bar1 + 8u * uint32_t(g); };
    auto o_done = [&](int g, uint32_t no) { return bar1 + 8u * (2u + 2u * uint32_t(g) + (no & 1u)); };
    auto s_full = [&](int g, uint32_t no) { return bar1 + 8u * (6u + 2u * uint32_t(g) + (no & 1u)); };
    auto p_full = [&](int g, uint32_t no) { return bar1 + 8u * (10u + 2u * uint32_t(g) + (no & 1u)); };
    const uint32_t drain = bar1 + 8u * 14u;
    auto told = [&](int st, uint32_t i) { return bar1 + 8u * (15u + uint32_t(st * kPieces) + i % kPieces); };
    auto done_with = [&](int st, uint32_t i) { return told(st, i) + 8u * 2u * kPieces; };
    Piece* const pieces = reinterpret_cast<Piece*>(smem + L::kOffPieces);
    auto piece_at = [&](int st, uint32_t i) -> Piece& { return pieces[st * kPieces + int(i % kPieces)]; };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffMisc);
    const AbortFlag abort_flag{sbase + L::kOffMisc + 4};
    const AbortFlag no_number{sbase + L::kOffMisc + 8};   // a value scale that is none was met where not all rows see it
    Start* const from = reinterpret_cast<Start*>(smem + L::kOffStart);   // of each stream's run
    int64_t* const sums = reinterpret_cast<int64_t*>(smem + L::kOffSums);
    const mmq_kv4_attention_t& p = a.p;
    int* const status = a.status;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kRawSlots; ++s) {
            mbar_init(raw_full(s), 1);
            mbar_init(raw_empty(s), 8);
        }
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(full(s), 4);
            mbar_init(empty(s), kTwo ? 2 : 1);
        }
        for (int g = 0; g < 2; ++g) {
            mbar_init(q_full(g), 4);
            for (uint32_t i = 0; i < 2; ++i) {
                mbar_init(o_done(g, i), 1);
                mbar_init(s_full(g, i), 1);
                mbar_init(p_full(g, i), 4);
            }
        }
        mbar_init(drain, 2);
        for (int st = 0; st < kStreams; ++st)
            for (int i = 0; i < kPieces; ++i) {
                mbar_init(told(st, i), 1);
                mbar_init(done_with(st, i), kTwo ? 1 + 8 + 2 + 8 : 1 + 8 + 1 + 4);   // fetch, expand, MMA, softmax
            }
        abort_flag.set(0u);
        no_number.set(0u);
        fence_barrier_init();
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
    griddep_launch_dependents();
    griddep_wait();

    // ---- who does what
    const int per = (p.batch + kThreads - 1) / kThreads;
    const int b0 = min(p.batch, int(threadIdx.x) * per), b1 = min(p.batch, b0 + per);
    auto length_of = [&](const Sequence& s) {   // of one head
        return int64_t(s.n) * a.group <= a.few ? 0 : head_length<kR, kKeys, idle(kR)>(s, a.group);
    };
    int64_t mine = 0, total;
    for (int b = b0; b < b1; ++b) mine += length_of(sequence(a, b, blockIdx.x == 0)) * p.kv_heads;
    const int64_t x1 = cta_scan<kThreads / 32>(mine, sums, total), x0 = x1 - mine;
    const Runs runs(total, max(int64_t(1), min(int64_t(gridDim.x) * kStreams, total)));
    if (threadIdx.x < kStreams) a.marks[blockIdx.x + threadIdx.x * gridDim.x] = Mark{-1, 0, 0, 0};

#pragma unroll 1
    for (int i = 0; i < 2 * kStreams; ++i) {   // where each stream's run starts and where the next one does
        const int st = i >> 1;
        const int64_t at = runs.start(blockIdx.x + int64_t(st) * gridDim.x + (i & 1));
        int64_t& place = i & 1 ? from[st].end : from[st].first;
        if (threadIdx.x == 0 && at >= total) place = total;
        if (x0 <= at && at < x1) {   // of one thread
            int64_t x = x0;
            for (int b = b0; b < b1; ++b) {
                const Sequence s = sequence(a, b, false);
                const int64_t each = length_of(s);
                if (at < x + each * p.kv_heads) {
                    const Cut c = cut<kR, kKeys, idle(kR)>(s, a.group, each, at - x);
                    place = at - c.moved;
                    if ((i & 1) == 0) {
                        from[st].b = b;
                        from[st].h = c.h;
                        from[st].u = c.u;
                        from[st].t = c.in;
                    }
                    break;
                }
                x += each * p.kv_heads;
            }
        }
    }
    __syncthreads();
    auto slot_of = [&](int st, int kind, uint32_t no) { return (st * 2 + kind) * kBufs + int(no % kBufs); };
    auto phase_of = [&](uint32_t no) { return (no / kBufs) & 1u; };

    // Piece i of stream st, once it is told; false after a wait that ran out.
    auto await_piece = [&](int st, uint32_t i) { return wait_bounded(told(st, i), (i / kPieces) & 1u, abort_flag, status); };
    // A warp's way through the streams' tiles, a tile of each per step.  (No arrays: they would lie in local memory.)
    struct Place {
        uint32_t piece = 0, no = 0;   // pieces and tiles before
        int t = 0;
        bool live = false;
    };
    Place one, two;
    uint32_t raw_no = 0;              // raw tiles before this step
    auto load = [&](int st, Place& at) {   // the next piece
        if (!__all_sync(0xffffffffu, await_piece(st, at.piece))) return false;
        const Piece& q = piece_at(st, at.piece);
        at.live = q.t0 < q.t1;
        at.t = q.t0;
        return true;
    };
    auto begin = [&]() { return load(0, one) && (kTwo || load(1, two)); };
    auto advance = [&](int st, Place& at) {
        if (!at.live) return true;
        ++at.no;
        if (++at.t < piece_at(st, at.piece).t1) return true;
        __syncwarp();
        if (lane == 0) mbar_arrive(done_with(st, at.piece));
        ++at.piece;
        return load(st, at);
    };
    auto step = [&]() {
        raw_no += uint32_t(one.live) + uint32_t(two.live);
        return advance(0, one) && (kTwo || advance(1, two));
    };
    auto more = [&]() { return one.live || two.live; };
    auto raw_of = [&](int st) { return raw_no + (st ? uint32_t(one.live) : 0u); };   // of stream st in this step
    auto raw_slot = [&](uint32_t i) { return int(i % uint32_t(kRawSlots)); };
    auto raw_phase = [&](uint32_t i) { return (i / uint32_t(kRawSlots)) & 1u; };
    if (warp >= kWarpExpand && warp < kWarpFetch) {
        // ------------------------------------------------------------ expand
        setmaxnreg_dec<kRegsExpand>();
        // Thread: tile of 16 tokens (one per warp), a row of eight in it (tokens r, r + 8 of keys, dimensions r, r + 8 of
        // 16 of values), and a quarter of the dimensions.  A block of 16's four words there give four 16-byte chunks: the
        // lower nibbles, the upper, and both after a shift by 8.
        constexpr int kJ = D / 64;   // blocks of 16 dimensions
        const bool values = warp >= kWarpExpand + 4;
        const uint32_t scratch = sbase + uint32_t(L::kOffMisc + 16 + 4 * (warp & 3));
        const int tile = warp & 3, r = lane & 7, part = lane >> 3;
        const int block32 = D == 128 ? part : part >> 1;
        const uint32_t half = uint32_t(tile * tile_bytes(D) + (values ? value_codes(D) : 0));
        const uint32_t words = half + uint32_t(r * 64) + (D == 128 ? (part >> 1) * 512u + (part & 1) * 8u : part * 4u);
        const uint32_t scales = half + uint32_t(8 * D) + (values ? uint32_t(block32 * 8) : uint32_t(r * (D / 8) + 4 * (block32 >> 1)));
        // Keys: blocks along the row, shift by 8 rows.  Values: blocks by 16 rows, upper nibbles 8 rows on.
        const uint32_t row0 = values ? uint32_t((16 * part * kJ + r) * 128)
                                     : uint32_t((D == 128 ? (part >> 1) * kKeys * 128 : 0) + (tile * 16 + r) * 128);
        auto expand = [&](int st, const Place& place) {
            const Piece& q = piece_at(st, place.piece);
            const int t = place.t;
            const uint32_t raw = raw_of(st);
            const int slot = slot_of(st, values, place.no), raw_at_slot = raw_slot(raw);
            if (!__all_sync(0xffffffffu, wait_bounded(raw_full(raw_at_slot), raw_phase(raw), abort_flag, status))) return false;
            const uint32_t raw_at = sbase + uint32_t(L::kOffRaw + raw_at_slot * L::kRaw);
            const uint32_t to = sbase + uint32_t(L::kOffSlots + slot * L::kTile) + row0;
            uint32_t w[4][kJ], sc[4][2];   // sc: of the lower and the upper tokens, for each word
            // Word c of rows r is at 64 r + 16 c: lane r takes them from r / 2 on, so that eight lanes hit all banks.
#pragma unroll
            for (int c = 0; c < 4; ++c) ld_shared_words<kJ>(raw_at + words + ((16u * c + 8u * uint32_t(r & 6)) & 48u), w[c]);
            if (values) {
#pragma unroll
                for (int c = 0; c < 4; ++c)   // tokens 2 c, 2 c + 1 and those + 8
                    ld_shared_words<2>(raw_at + scales + uint32_t(c * (D / 4)), sc[c]);
                if (t * kKeys + kKeys > q.least) {
                    // tokens that some rows of the unit do not see: what is no number must not reach those, and what
                    // lies past the last must reach none
                    const int left = q.most - (t * kKeys + tile * 16);
                    bool none = false;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const bool past = 2 * c + (k & 1) + (k & 2 ? 8 : 0) >= left;
                            uint32_t& v = sc[c][k >> 1];
                            const bool good = finite16(k & 1 ? v >> 16 : v);
                            if (past || !good) v &= k & 1 ? 0x0000FFFFu : 0xFFFF0000u;
                            none |= !past && !good;
                        }
                    if (none) no_number.set(1u);
                }
            } else {
                // tokens r and r + 8: two blocks of 32 to a word
                const uint32_t lo = ld_shared_u32(raw_at + scales), hi = ld_shared_u32(raw_at + scales + uint32_t(D / 16));
                const uint32_t sel = block32 & 1 ? 0x3232u : 0x1010u;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    sc[c][0] = prmt(lo, 0u, sel);
                    sc[c][1] = prmt(hi, 0u, sel);
                }
            }
            // all loads are back (each is in the sum) before the raw slot is handed on
            loads_done(scratch, sc[0][0] ^ sc[0][1] ^ sc[1][0] ^ sc[2][0] ^ sc[3][0] ^ w[0][0] ^ w[1][0] ^ w[2][0] ^ w[3][0]);
            __syncwarp();
            if (lane == 0) mbar_arrive(raw_empty(raw_at_slot));
            if (!__all_sync(0xffffffffu, wait_bounded(empty(slot), phase_of(place.no) ^ 1u, abort_flag, status))) return false;
            // words back in order: w[c] is word c + r / 2
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
                const uint32_t a0 = w[0][j], a1 = w[1][j], a2 = w[2][j], a3 = w[3][j];
                const bool one = r & 2, two = r & 4;
                const uint32_t b0 = one ? a3 : a0, b1 = one ? a0 : a1, b2 = one ? a1 : a2, b3 = one ? a2 : a3;
                w[0][j] = two ? b2 : b0;
                w[1][j] = two ? b3 : b1;
                w[2][j] = two ? b0 : b2;
                w[3][j] = two ? b1 : b3;
            }
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
                const int chunk = 2 * (values ? tile : (part * kJ + j) & 3);
                const uint32_t at = to + (values ? uint32_t(j * 2048) : 0u);
                const uint32_t x0 = uint32_t(chunk ^ r) << 4, x1 = uint32_t((chunk + 1) ^ r) << 4;
                const uint32_t y1 = values ? 1024u + x0 : x1, y2 = values ? x1 : 1024u + x0;
                st_shared_v4(at + x0, expand_low(w[0][j], sc[0][0]), expand_low(w[1][j], sc[1][0]), expand_low(w[2][j], sc[2][0]), expand_low(w[3][j], sc[3][0]));
                st_shared_v4(at + y1, expand_high(w[0][j], sc[0][0]), expand_high(w[1][j], sc[1][0]), expand_high(w[2][j], sc[2][0]), expand_high(w[3][j], sc[3][0]));
#pragma unroll
                for (int c = 0; c < 4; ++c) w[c][j] >>= 8;
                st_shared_v4(at + y2, expand_low(w[0][j], sc[0][1]), expand_low(w[1][j], sc[1][1]), expand_low(w[2][j], sc[2][1]), expand_low(w[3][j], sc[3][1]));
                st_shared_v4(at + 1024u + x1, expand_high(w[0][j], sc[0][1]), expand_high(w[1][j], sc[1][1]), expand_high(w[2][j], sc[2][1]), expand_high(w[3][j], sc[3][1]));
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(full(slot));
            return true;
        };
        bool ok = begin();
        while (ok && more()) {
#pragma unroll 1
            for (int st = 0; st < kStreams && ok; ++st) {
                const Place& place = !kTwo && st ? two : one;
                const Place copy = place;
                if (copy.live) ok = expand(st, copy);
            }
            ok = ok && step();
        }
    } else if (warp >= kWarpFetch) {
        setmaxnreg_dec<kRegsOther>();
        if (warp == kWarpFetch) {
            // ------------------------------------------------------ raw tiles
            uint32_t issued = 0, parity = 0;   // slots with a copy, the parity of its arrival
            bool withhold = false;   // test hook: the first copy never comes
            for (int st = 0; st < kStreams; ++st) withhold |= a.inject && from[st].first == 0 && from[st].end > 0;
            const int tile_shift = a.page_shift - 4;
            constexpr int kOf = kKeys / kTokens;   // tiles of 16
            // A copy takes as many of a key tile's tiles of 16 as lie on one page, up to all; lane i issues the i-th.
            const int of_page = min(kOf, 1 << tile_shift), copies = kOf / of_page;
            const uint32_t bytes = uint32_t(of_page * tile_bytes(D)), into = uint32_t(lane) * bytes;
            // The page of this lane's copy, looked up a step ahead; what lies past the unit's keys is no page.
            auto page_of = [&](int st, const Place& at) {
                if (!at.live) return -1;
                const Piece& q = piece_at(st, at.piece);
                const int tile = kOf * at.t + of_page * lane;
                return lane < copies && tile * kTokens < q.most ? p.page_table[int64_t(q.b) * p.table_width + (tile >> tile_shift)] : -1;
            };
            auto place_of = [&](int st, const Place& at, int32_t id) -> const uint8_t* {
                const Piece& q = piece_at(st, at.piece);
                const int tile = kOf * at.t + of_page * lane;
                if (id >= 0 && id < p.n_pages)
                    return p.cache + (((int64_t(id) * p.kv_heads + q.h) << tile_shift) + (tile & ((1 << tile_shift) - 1))) * tile_bytes(D);
                if (lane < copies && tile * kTokens < q.most) atomicCAS(status, 0, MMQ_ERR_ARG);
                return zero_tiles;
            };
            auto copy = [&](const uint8_t* src, uint32_t i) {
                const int slot = raw_slot(i);
                if (!__all_sync(0xffffffffu, wait_bounded(raw_empty(slot), raw_phase(i) ^ 1u, abort_flag, status))) return false;
                if (!withhold) {
                    if (lane == 0) mbar_arrive_expect_tx(raw_full(slot), uint32_t(L::kRaw));
                    __syncwarp();
                    if (lane < copies) bulk_load(sbase + uint32_t(L::kOffRaw + slot * L::kRaw) + into, src, bytes, raw_full(slot));
                    issued |= 1u << slot;
                    parity = (parity & ~(1u << slot)) | (raw_phase(i) << slot);
                }
                withhold = false;
                return true;
            };
            bool ok = begin();
            int32_t id0 = ok ? page_of(0, one) : -1, id1 = ok && !kTwo ? page_of(1, two) : -1;
            while (ok && more()) {
                const uint8_t* src0 = one.live ? place_of(0, one, id0) : zero_tiles;
                const uint8_t* src1 = two.live ? place_of(1, two, id1) : zero_tiles;
                const bool has0 = one.live, has1 = two.live;
                const uint32_t raw0 = raw_of(0), raw1 = raw_of(1);
                ok = step();
                if (ok) {
                    id0 = page_of(0, one);
                    if (!kTwo) id1 = page_of(1, two);
                }
                // (a piece that has been stepped past is not looked at again)
                ok = (!has0 || copy(src0, raw0)) && (!has1 || copy(src1, raw1)) && ok;
            }
            // copies still in flight, also after a wait that ran out
            if (lane == 0)
                for (int s = 0; s < kRawSlots; ++s)
                    if ((issued >> s) & 1u) wait_drain(raw_full(s), (parity >> s) & 1u, status);
        } else if (warp <= kWarpMma + 1) {
            // ---------------------------------------------------- MMA issuers
            if (elect_one()) {
                const int g = warp - kWarpMma, st = kTwo ? 0 : g;
                constexpr uint32_t kIdQK = idesc_f16_f32(kRows, kKeys), kIdPV = idesc_f16_f32(kRows, D);
                // Descriptors by their lower words, which hold the address; the upper is the same for all.
                constexpr uint32_t kTileDesc = uint32_t(L::kTile >> 4);
                const uint32_t dq = uint32_t(smem_desc_sw128(sbase + uint32_t(L::kOffQ + g * L::kQ)));
                const uint32_t slots = uint32_t(smem_desc_sw128(sbase + uint32_t(L::kOffSlots)));
                auto desc = [](uint32_t low) { return (smem_desc_sw128(0) >> 32 << 32) | low; };
                const uint32_t ts = tmem + kColS + 128u * uint32_t(g), to = tmem + kColO + 128u * uint32_t(g);
                auto arrived = [&](int kind, uint32_t no) {
                    return wait_bounded(full(slot_of(st, kind, no)), phase_of(no), abort_flag, status);
                };
                // A tile's, opaque so that the loop does not keep one for every product: this thread has few registers.
                auto described = [](uint32_t d) {
                    asm volatile("" : "+r"(d));
                    return d;
                };
                uint32_t no = 0;   // tiles so far, the buffer of S in turn
                // S = Q K^T with tile i of keys, once it is there
                auto scores = [&](uint32_t i) {
                    if (!arrived(0, i)) return false;
                    tc_fence_after();
                    const int slot = slot_of(st, 0, i);
                    const uint32_t dk = described(slots + uint32_t(slot) * kTileDesc), dq_now = described(dq);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        mma_f16(ts + 64u * (i & 1u), desc(dq_now + uint32_t((kk >> 2) * (kRows * 128 >> 4) + (kk & 3) * 2)),
                                desc(dk + uint32_t((kk >> 2) * (kKeys * 128 >> 4) + (kk & 3) * 2)), kIdQK, uint32_t(kk > 0));
                    mma_commit(s_full(g, i));
                    mma_commit(empty(slot));
                    return true;
                };
                uint32_t q_phase = 0;
                bool ok = true;
                for (uint32_t i = 0; ok; ++i) {
                    ok = await_piece(st, i);
                    const int tiles = piece_at(st, i).t1 - piece_at(st, i).t0;
                    if (!ok || tiles == 0) break;
                    mbar_arrive(done_with(st, i));
                    ok = wait_bounded(q_full(g), q_phase, abort_flag, status) && scores(no) && (tiles == 1 || scores(no + 1));
                    q_phase ^= 1u;
                    for (int s = 0; s < tiles && ok; ++s, ++no) {
                        ok = arrived(1, no) && wait_bounded(p_full(g, no), (no >> 1) & 1u, abort_flag, status);
                        if (!ok) break;
                        tc_fence_after();
                        const int slot = slot_of(st, 1, no);
                        const uint32_t dv = described(slots + uint32_t(slot) * kTileDesc);
#pragma unroll
                        for (int kk = 0; kk < kKeys / 16; ++kk)
                            mma_f16_ta(to, ts + 64u * (no & 1u) + 8u * uint32_t(kk), desc(dv + uint32_t(kk * 2)), kIdPV, uint32_t(s > 0 || kk > 0));
                        if constexpr (kFine) {
#pragma unroll
                            for (int kk = 0; kk < kKeys / 16; ++kk)
                                mma_f16_ta(to, ts + 64u * (no & 1u) + 32u + 8u * uint32_t(kk), desc(dv + uint32_t(kk * 2)), kIdPV, 1u);
                        }
                        mma_commit(o_done(g, no));
                        mma_commit(empty(slot));
                        if (s + 2 < tiles) ok = scores(no + 2);
                    }
                }
                mma_commit(drain);   // everything issued, also after a wait that ran out
                wait_drain(drain, 0u, status);
            }
        } else if (lane < kStreams) {
            // ---------------------------------------------- the runs' pieces
            Walk<kR> q(a, from[lane]);
            for (uint32_t i = 0;; ++i) {
                Piece& to = piece_at(lane, i);
                // Until a whole piece is done, which may have millions of tiles: 1 us each, 20 are granted.
                const uint64_t limit = kWaitLimitNs + (i < kPieces ? 0 : uint64_t(to.t1 - to.t0) * 20000);
                if (!wait_bounded(done_with(lane, i), ((i / kPieces) & 1u) ^ 1u, abort_flag, status, limit)) break;
                to.t0 = to.t1 = 0;
                if (q.valid()) {
                    to.t0 = q.first_tile();
                    to.t1 = q.end_tile();
                    to.start = q.s.start;
                    to.last = int(runs.of(q.name + q.length - 1));
                    to.b = q.b;
                    to.h = q.h;
                    to.u = q.u;
                    to.starts = q.starts();
                    to.ends = q.ends();
                    to.n = q.s.n;
                    to.len = q.s.len;
                    to.most = q.most();
                    to.least = q.least();
                }
                mbar_arrive(told(lane, i));
                if (!q.valid()) break;
                q.next();
            }
        }
    } else {
        // ---------------------------------------------------------- softmax
        setmaxnreg_inc<kRegsSoftmax>();
        const int g = warp >> 2, st = kTwo ? 0 : g;
        const int row = (warp & 3) * 32 + lane;
        const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
        const uint32_t ts0 = tmem + lanes + kColS + 128u * uint32_t(g), to = tmem + lanes + kColO + 128u * uint32_t(g);
        uint32_t no = 0;   // tiles so far
        bool ok = true;
        for (uint32_t piece_no = 0;; ++piece_no) {
            ok = __all_sync(0xffffffffu, await_piece(st, piece_no));
            const Piece& q = piece_at(st, piece_no);
            const int tiles = q.t1 - q.t0;
            if (!ok || tiles == 0) break;
            int left;   // keys that the row sees from the next tile on
            float scale = a.scale_log2;
            // The group's query rows, swizzled (16-byte chunk c of row n at c ^ (n & 7)); zeros past the last row.  Of 256
            // rows a warp takes kLanes lanes to a row, each lane one chunk of each of kTurns rows, and the results go out
            // the same way; of at most 128, which are few as a rule, each thread takes its own row.  Own rows for the many:
            // 70 -> 80 us (64 tokens of 8 sequences), 390 -> 409 (4096 of 2); together for the few: 21 rows of 33
            // sequences 63 -> 70, 35 rows 70 -> 77.
            constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes, kTurns = 32 / kAtOnce;
            const int in_row = lane % kLanes, of_turn = lane / kLanes;
            const uint32_t q_rows = sbase + uint32_t(L::kOffQ + g * L::kQ + (in_row >> 3) * (kRows * 128) + (warp & 3) * 32 * 128);
            auto q_chunk = [&](int r) { return q_rows + uint32_t(r * 128 + (((in_row & 7) ^ (r & 7)) << 4)); };
            {
                const int r = q.u * kR + (kTwo ? g * kRows : 0) + row, j = r / a.group, head = q.h * a.group + r - j * a.group;
                const bool valid = j < q.n;
                left = (valid ? max(0, q.len - q.n + 1 + j) : 0x7FFFFFFF) - q.t0 * kKeys;
                if constexpr (kTwo) {
                    const int64_t at = valid ? (q.start + j) * p.q_stride + int64_t(head) * D : -1;
                    const uint32_t some = __ballot_sync(0xffffffffu, valid);
                    uint4 v[kTurns];
#pragma unroll
                    for (int i = 0; i < kTurns; ++i) {
                        const int64_t from_row = __shfl_sync(0xffffffffu, at, i * kAtOnce + of_turn);
                        v[i] = make_uint4(0u, 0u, 0u, 0u);
                        if (from_row >= 0) v[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + from_row + 8 * in_row);
                    }
                    if (std::is_same<T, __nv_bfloat16>::value && some) {
                        int e[kTurns];
#pragma unroll
                        for (int i = 0; i < kTurns; ++i) {
                            uint32_t top = 0;   // magnitudes order as integers; NaN's as the largest
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const uint32_t w = k == 0 ? v[i].x : k == 1 ? v[i].y : k == 2 ? v[i].z : v[i].w;
                                top = max(top, max((w << 16) & 0x7FFF0000u, w & 0x7FFF0000u));
                            }
                            // top in [2^e, 2^(e+1)) -> [2^13, 2^14); a row of zeros or tiny values as if it had 2^-100
                            e[i] = max(-100, int(top >> 23) - 127);
                        }
#pragma unroll
                        for (int d = 1; d < kLanes; d <<= 1) {
#pragma unroll
                            for (int i = 0; i < kTurns; ++i) e[i] = max(e[i], __shfl_xor_sync(0xffffffffu, e[i], d));
                        }
#pragma unroll
                        for (int i = 0; i < kTurns; ++i) {
                            const float up = __uint_as_float(uint32_t(127 + 13 - e[i]) << 23);
                            uint32_t* const w[4] = {&v[i].x, &v[i].y, &v[i].z, &v[i].w};
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                *w[k] = pack16(__uint_as_float(*w[k] << 16) * up, __uint_as_float(*w[k] & 0xFFFF0000u) * up);
                            const int of_mine = __shfl_sync(0xffffffffu, e[i], lane % kAtOnce * kLanes);
                            if (lane / kAtOnce == i) scale = fminf(a.scale_log2 * __uint_as_float(uint32_t(127 + of_mine - 13) << 23), 3.4e38f);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < kTurns; ++i) st_shared_v4(q_chunk(i * kAtOnce + of_turn), v[i].x, v[i].y, v[i].z, v[i].w);
                } else {
                    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + (valid ? (q.start + j) * p.q_stride + int64_t(head) * D : 0));
                    const uint32_t dst = sbase + uint32_t(L::kOffQ + g * L::kQ + row * 128);
                    uint4 v[D / 8];
#pragma unroll
                    for (int c = 0; c < D / 8; ++c) v[c] = valid ? src[c] : make_uint4(0u, 0u, 0u, 0u);
                    if (std::is_same<T, __nv_bfloat16>::value) {
                        uint32_t top = 0;   // magnitudes order as integers; NaN's as the largest
#pragma unroll
                        for (int c = 0; c < D / 8; ++c) {
                            const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
                            for (int k = 0; k < 4; ++k) top = max(top, max((w[k] << 16) & 0x7FFF0000u, w[k] & 0x7FFF0000u));
                        }
                        // top in [2^e, 2^(e+1)) -> [2^13, 2^14); a row of zeros or tiny values as if it had 2^-100
                        const int e = max(-100, int(top >> 23) - 127);
                        const float up = __uint_as_float(uint32_t(127 + 13 - e) << 23);
                        scale = fminf(scale * __uint_as_float(uint32_t(127 + e - 13) << 23), 3.4e38f);
#pragma unroll
                        for (int c = 0; c < D / 8; ++c) {
                            uint32_t* const w[4] = {&v[c].x, &v[c].y, &v[c].z, &v[c].w};
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                *w[k] = pack16(__uint_as_float(*w[k] << 16) * up, __uint_as_float(*w[k] & 0xFFFF0000u) * up);
                        }
                    }
#pragma unroll
                    for (int c = 0; c < D / 8; ++c)
                        st_shared_v4(dst + uint32_t((c >> 3) * (kRows * 128) + (((c & 7) ^ (row & 7)) << 4)), v[c].x, v[c].y, v[c].z, v[c].w);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full(g));
            }
            float m = kNone, l = 0.f;
            bool wide = false;
            int n = 0;
            // The product of the tile before; the one before that has come with the last scores, so that o_done, one for
            // every other tile, is never two phases off.
            auto await_product = [&]() {
                ok = __all_sync(0xffffffffu, wait_bounded(o_done(g, no - 1), ((no - 1) >> 1) & 1u, abort_flag, status));
                tc_fence_after();
            };
            auto scale_o = [&](float f) {   // O at rest
                await_product();
                if (!ok) return;
                l *= f;
#pragma unroll 1
                for (int c = 0; c < D / 16; ++c) {   // few registers beside the scores
                    uint32_t o[16];
                    tmem_ld_32x32b_x16(to + 16u * uint32_t(c), o);
                    tmem_wait_ld(o);
#pragma unroll
                    for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                    tmem_st_32x32b_x16(to + 16u * uint32_t(c), o);
                }
            };
            for (; n < tiles; ++n, ++no) {
                ok = __all_sync(0xffffffffu, wait_bounded(s_full(g, no), (no >> 1) & 1u, abort_flag, status));
                if (!ok) break;
                tc_fence_after();
                const uint32_t ts = ts0 + 64u * (no & 1u);
                uint32_t s[2][32];
#pragma unroll
                for (int c = 0; c < 2; ++c) tmem_ld_32x32b_x32(ts + 32u * uint32_t(c), s[c]);
#pragma unroll
                for (int c = 0; c < 2; ++c) tmem_wait_ld(s[c]);
                if (left < kKeys) {
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (32 * c + k >= left) s[c][k] = 0xFF800000u;
                }
                float x0 = __uint_as_float(s[0][0]), x1 = __uint_as_float(s[0][1]), x2 = __uint_as_float(s[1][0]),
                      x3 = __uint_as_float(s[1][1]);
#pragma unroll
                for (int k = 0; k < 32; k += 4) {
                    x0 = max3(x0, __uint_as_float(s[0][k]), __uint_as_float(s[0][k + 1]));
                    x1 = max3(x1, __uint_as_float(s[0][k + 2]), __uint_as_float(s[0][k + 3]));
                    x2 = max3(x2, __uint_as_float(s[1][k]), __uint_as_float(s[1][k + 1]));
                    x3 = max3(x3, __uint_as_float(s[1][k + 2]), __uint_as_float(s[1][k + 3]));
                }
                const float top = fmaxf(fmaxf(x0, x1), fmaxf(x2, x3)) * scale;
                const bool rises = top > m + kGrow;
                if (__any_sync(0xffffffffu, rises)) {
                    const float was = m, now = fmaxf(m, top);   // of every row, also one that rises by less than kGrow
                    wide = __any_sync(0xffffffffu, now != m && !(fabsf(now) < kWide));
                    if (wide) break;
                    m = now;
                    if (n > 0) scale_o(ex2(was - m));
                    if (!ok) break;
                }
                const float base = m - kLift;
                const uint64_t scale2 = pack2(scale, scale), base2 = pack2(-base, -base);
                uint64_t sum[2] = {0, 0};
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t pk[16], rest[kFine ? 16 : 1];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const uint64_t e = ffma2(pack2u(s[c][2 * k], s[c][2 * k + 1]), scale2, base2);
                        const float u = ex2(lo_f(e)), v = ex2(hi_f(e));
                        sum[k & 1] = fadd2(sum[k & 1], pack2(u, v));
                        pk[k] = pack16(u, v);
                        if constexpr (kFine) rest[k] = rest16(u, v, pk[k]);
                    }
                    tmem_st_32x32b_x16(ts + 16u * uint32_t(c), pk);
                    if constexpr (kFine) tmem_st_32x32b_x16(ts + 32u + 16u * uint32_t(c), rest);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full(g, no));
                sum[0] = fadd2(sum[0], sum[1]);
                l += lo_f(sum[0]) + hi_f(sum[0]);
                left -= kKeys;
            }
            // S scale - m in one step, as above, is past zero by what m lost in its rounding, half a unit in its
            // last place: from 2^20 on too much for P's range.  From the first tile where a row of the warp gets
            // there the products are rounded first, as m was, and m is neither lifted nor let behind.  No usual
            // call comes here, so short loops over S where it lies.
            for (bool here = true; ok && wide && n < tiles; ++n, ++no, here = false) {
                if (!here) {
                    ok = __all_sync(0xffffffffu, wait_bounded(s_full(g, no), (no >> 1) & 1u, abort_flag, status));
                    if (!ok) break;
                    tc_fence_after();
                }
                const uint32_t ts = ts0 + 64u * (no & 1u);
                float top = -INFINITY, sum = 0.f;
#pragma unroll 1
                for (int c = 0; c < 2; ++c) {
                    uint32_t x[32];
                    tmem_ld_32x32b_x32(ts + 32u * uint32_t(c), x);
                    tmem_wait_ld(x);
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (32 * c + k < left) top = fmaxf(top, __uint_as_float(x[k]));
                }
                const float was = m;
                m = fmaxf(m, __fmul_rn(top, scale));
                const float base = reference(m);
                if (n > 0) scale_o(ex2(reference(was) - base));
                if (!ok) break;
                uint32_t second[kFine ? 32 : 1];   // the rests of the first half's weights go over the second half
                if constexpr (kFine) {
                    tmem_ld_32x32b_x32(ts + 32u, second);
                    tmem_wait_ld(second);
                }
#pragma unroll 1
                for (int c = 0; c < 2; ++c) {
                    uint32_t x[32], pk[16];
                    if (!kFine || c == 0) {
                        tmem_ld_32x32b_x32(ts + 32u * uint32_t(c), x);
                        tmem_wait_ld(x);
                    }
                    if constexpr (kFine) {
                        if (c == 1) {
#pragma unroll
                            for (int k = 0; k < 32; ++k) x[k] = second[k];
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        const float y = __fmul_rn(__uint_as_float(x[k]), scale);
                        x[k] = 32 * c + k < left ? __float_as_uint(ex2(__fsub_rn(y, base))) : 0u;
                        sum += __uint_as_float(x[k]);
                    }
#pragma unroll
                    for (int k = 0; k < 16; ++k) pk[k] = pack16(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1]));
                    tmem_st_32x32b_x16(ts + 16u * uint32_t(c), pk);   // over what has been read
                    if constexpr (kFine) {
#pragma unroll
                        for (int k = 0; k < 16; ++k) pk[k] = rest16(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1]), pk[k]);
                        tmem_st_32x32b_x16(ts + 32u + 16u * uint32_t(c), pk);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full(g, no));
                l += sum;
                left -= kKeys;
            }
            if (!ok) break;
            await_product();
            if (!ok) break;
            tc_fence_after();
            const int r = q.u * kR + (kTwo ? g * kRows : 0) + row, j = r / a.group, head = q.h * a.group + r - j * a.group;
            const bool valid = j < q.n, done = q.starts && q.ends;
            // Where a value scale is no number and not all rows see its token: the rows that do, block by block.
            uint32_t none = 0;
            if (no_number.raised() && valid) {
                const int tile_shift = a.page_shift - 4, see = max(0, q.len - q.n + 1 + j);
                for (int key = max(q.t0, q.least / kKeys) * kKeys; key < min(see, q.t1 * kKeys); ++key) {
                    const int32_t id = p.page_table[int64_t(q.b) * p.table_width + (key >> a.page_shift)];
                    if (id < 0 || id >= p.n_pages) continue;
                    const uint8_t* at = p.cache + (((int64_t(id) * p.kv_heads + q.h) << tile_shift) +
                                                   ((key >> 4) & ((1 << tile_shift) - 1))) * tile_bytes(D);
                    for (int b = 0; b < D / 32; ++b)
                        if (!finite16(*reinterpret_cast<const uint16_t*>(at + value_scale<D>(key & 15, b)))) none |= 1u << b;
                }
            }
            const float factor = done ? l == 0.f ? 0.f : 1.f / l : 1.f;
            const int64_t run = blockIdx.x + int64_t(st) * gridDim.x;
            const int64_t at = (run * 2 + (q.starts ? 1 : 0)) * kR + (r - q.u * kR);   // a part's row
            const int64_t out = !valid ? -1 : done ? ((q.start + j) * p.heads + head) * D : at * D;
            const bool narrow = done && p.out_type != MMQ_TYPE_F32;
            float* const out32 = done ? static_cast<float*>(p.out) : a.parts;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld_32x32b_x32(to + 32u * uint32_t(c), o);
                tmem_wait_ld(o);
                const float by = (none >> c) & 1u ? __int_as_float(0x7FC00000) : factor;
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * by);
                if (narrow) {
                    uint32_t pk[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const float u = __uint_as_float(o[2 * k]), v = __uint_as_float(o[2 * k + 1]);
                        if (std::is_same<T, __half>::value) {
                            pk[k] = pack16(u, v);
                        } else {
                            const __nv_bfloat162 w = __floats2bfloat162_rn(u, v);
                            pk[k] = *reinterpret_cast<const uint32_t*>(&w);
                        }
                    }
                    if constexpr (kTwo) {   // through the queries' place, which is free now
                        const uint32_t mine = sbase + uint32_t(L::kOffQ + g * L::kQ + (c >> 1) * (kRows * 128) + row * 128);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            st_shared_v4(mine + uint32_t(((4 * (c & 1) + k) ^ (row & 7)) << 4), pk[4 * k], pk[4 * k + 1], pk[4 * k + 2], pk[4 * k + 3]);
                    } else if (valid) {
                        uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + out + 32 * c);
#pragma unroll
                        for (int k = 0; k < 4; ++k) dst[k] = make_uint4(pk[4 * k], pk[4 * k + 1], pk[4 * k + 2], pk[4 * k + 3]);
                    }
                } else if constexpr (kTwo) {
                    const uint32_t rows = sbase + uint32_t(L::kOffQ + g * L::kQ + (warp & 3) * 32 * 128);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        st_shared_v4(rows + uint32_t(lane * 128 + ((k ^ (lane & 7)) << 4)), o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int of = 4 * k + (lane >> 3);
                        const int64_t to_row = __shfl_sync(0xffffffffu, out, of);
                        const uint4 v = ld_shared_v4(rows + uint32_t(of * 128 + (((lane ^ of) & 7) << 4)));
                        if (to_row >= 0) *reinterpret_cast<uint4*>(out32 + to_row + 32 * c + 4 * (lane & 7)) = v;
                    }
                    __syncwarp();
                } else if (valid) {
                    uint4* dst = reinterpret_cast<uint4*>(out32 + out + 32 * c);
#pragma unroll
                    for (int k = 0; k < 8; ++k) dst[k] = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                }
            }
            if (kTwo && narrow) {
                __syncwarp();
#pragma unroll
                for (int i = 0; i < kTurns; ++i) {
                    const int64_t to_row = __shfl_sync(0xffffffffu, out, i * kAtOnce + of_turn);
                    const uint4 v = ld_shared_v4(q_chunk(i * kAtOnce + of_turn));
                    if (to_row >= 0) *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + to_row + 8 * in_row) = v;
                }
                __syncwarp();
            }
            tc_fence_before();
            if (!done && q.starts && row == 0 && (g == 0 || !kTwo)) a.marks[run] = Mark{q.last, q.b, q.h, q.u};
            if (!done && valid)
                reinterpret_cast<float2*>(a.parts + int64_t(gridDim.x) * kStreams * 2 * kR * D)[at] = make_float2(reference(m), l);
            __syncwarp();
            if (lane == 0) mbar_arrive(done_with(st, piece_no));
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

template <typename T, int D, bool kTwo, bool kFine>
cudaError_t launch(const Kv4Args& a, int nsm, cudaLaunchConfig_t cfg) {
    using L = Layout<D, kTwo>;
    auto* const kernel = kv4_tc_kernel<T, D, kTwo, kFine>;
    static const bool registers_ok = [] {   // else the split's increase would wait forever
        cudaFuncAttributes f;
        return cudaFuncGetAttributes(&f, kv4_tc_kernel<T, D, kTwo, kFine>) == cudaSuccess && f.numRegs == int(kRegsLaunch);
    }();
    if (!registers_ok) return cudaErrorLaunchOutOfResources;
    cudaError_t e;
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes))) return e;
    cfg.gridDim = dim3(unsigned(nsm));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = L::kBytes;
    if ((e = cudaLaunchKernelEx(&cfg, kernel, a))) return e;
    return mmq::launch_kv4_join(a, L::kR, nsm * L::kStreams, cfg.stream);
}
template <typename T, int D>
cudaError_t launch(const Kv4Args& a, bool two, int nsm, const cudaLaunchConfig_t& cfg) {
    if (a.p.out_type == MMQ_TYPE_F32)
        return two ? launch<T, D, true, true>(a, nsm, cfg) : launch<T, D, false, true>(a, nsm, cfg);
    return two ? launch<T, D, true, false>(a, nsm, cfg) : launch<T, D, false, false>(a, nsm, cfg);
}

}  // namespace

namespace mmq {

// Parts of 2 x nsm x 256 rows either way (two runs of 128 rows per CTA, or one of 256).
size_t kv4_attention_tc_part_bytes(int head_dim, int nsm) { return size_t(nsm) * 2 * 256 * size_t(head_dim + 2) * 4; }

cudaError_t launch_kv4_attention_tc(const kv4::Kv4Args& a, bool two, int nsm, const cudaLaunchConfig_t& cfg) {
    if (a.p.type == MMQ_TYPE_F16)
        return a.p.head_dim == 64 ? launch<__half, 64>(a, two, nsm, cfg) : launch<__half, 128>(a, two, nsm, cfg);
    return a.p.head_dim == 64 ? launch<__nv_bfloat16, 64>(a, two, nsm, cfg) : launch<__nv_bfloat16, 128>(a, two, nsm, cfg);
}

}  // namespace mmq
