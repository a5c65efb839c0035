// arkv_prefix_attn: decode attention of many branches to the prefixes they share,
// joined with each branch's own part.
//
// The queries of a prefix's branches that meet the same key head are the rows of one
// matrix (row = branch x query of the group, tiles of 128 rows), so the prefix is read
// once for all of them and both products run on the tensor cores:
//   S[128 rows][64 tokens] = Q K^T,   O[128 rows][D] += P V,   P = 2^(S c - m).
//
// Work.  A unit is (prefix, key head, one or two tiles of rows); its tiles of 64 tokens are
// the bf16 and the FP8 tiles of the prefix row.  The tiles of all units form one list, cut
// into equal runs, one a CTA and one CTA an SM (with shares of a unit's bf16 and FP8 tiles in
// proportion: an FP8 tile has twice the arithmetic per byte).  A run that crosses units is
// several segments, each with a partial (max, sum, unnormalised o) in the workspace.  In the
// list every unit begins with kSegCost empty places, about what the start of another segment
// costs, so that the run that holds them has that many tiles less.
// prefix_join_kernel joins the partials and the branch's own part.
//
// A CTA.  Warp 0 walks the run, streams K and V by TMA through a ring of slots (a slot is a
// tile's K or its V) and hands the segments to the others through shared memory.  Warps 1 and
// 2 issue the products, warp 3 fetches FP8 scales.  Two warpgroups do the softmax, each with
// its own two S (and P) and O in tensor memory and its own state, so that neither waits for
// the other.  Two more rewrite FP8 tiles in place as bf16 (exact: 4 or 3 significant bits),
// one the K tiles, one the V tiles.  With one tile of rows the softmax warpgroups take the
// token tiles in turn and their two O are added at the end of the segment; with two each has
// its rows, and a token tile is loaded and converted once for both.  Either way a softmax job
// is one S, and the jobs alternate.
// P takes the place of S.  The K scale of an FP8 token multiplies its logit, its V scale is
// folded into P.
// The softmax reference m starts as zero and moves only when a logit exceeds it by 2^32 (or
// the first tile's are all as far below: float32 and bf16 have the range), so O is hardly
// ever rescaled and a job needs no maximum before its exponentials.  P is the sum of two bf16
// parts (16 bits, as arkv_decode_attn holds it), which take all of S's place; each is multiplied
// with V.  One part alone would be as coarse as o's own rounding, and show beside it whatever the
// number of tokens.  The sum is of the unrounded values.
//
// Bound.  HBM for one tile of rows, the tensor cores for two (floors of a prefix of
// 23701 bf16 and 18900 FP8 tokens, 8 key heads of 128: 21.2 us for 128 rows, 26.8 us for 256).
// Measured with the join: 59.6 and 92.1 us; 23.5 us for 5921 + 4739 tokens and 128 rows
// (floor 5.3).  What takes the time is the issue of the softmax and the conversion, two warps of
// each on every scheduler: 64 tokens take an SM 1.3 us with one tile of rows and 2.1 us with two,
// and no pipe is busy for more than 37% of that.  About 11 us of every call are start, end of the
// segment, and the join.
//
// Every wait is bounded: one that runs out raises ARKV_STATUS_TIMEOUT and a flag that
// ends every role, copies and products in flight are given a last bounded wait, tensor
// memory is freed and the call ends.
#include <math.h>
#include <mutex>
#include <type_traits>

#include <cudaTypedefs.h>

#include "arkv_internal.cuh"
#include "prefix_join.h"
#include "tc.cuh"

namespace arkv {

namespace {

using namespace tc;

constexpr float kNegInf = -INFINITY;
constexpr float kNoLogit = -32768.f;   // the reference of a row whose logits so far are all -inf: any rise from it is exact enough
constexpr unsigned kFull = 0xffffffffu;
constexpr int kRows = 128;            // query rows of a tile
constexpr int kTok = 64;              // tokens of a tile
constexpr int kWarps = 20;            // 4 of single roles, 2 x 4 softmax, 2 x 4 conversion
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxCtas = 192;         // of one call
constexpr int kSegCost = 5;           // a segment's start and end, in tiles (4 to 7 measure alike, 2 is 4% slower)
constexpr int kSpinLimit = 1 << 20;   // polls of one wait

struct RowInfo {
    int n16, n8, T16, T8, b0, nb, mt;   // live slots, tiles, first branch, branches, units
};

// This CTA's run of the list: [v, v_end); the row that holds place v, its first place, the
// units before it.
struct Sched {
    int v, v_end, base, row, units;
    RowInfo r;
};

// A segment: tiles [i16, e16) of the row's bf16 tiles, then those from i8 on of its FP8 tiles, n in
// all.
enum : int { kSegFirst = 1, kSegLast = 2, kSegTwo = 4, kSegEnd = 8 };
struct Seg {
    int row, n16, n8, n, i16, e16, i8;
    int branch, rows0, rows1;   // first branch; live rows of the two tiles of rows
    int slot, flags;            // place of its partial; first, last of its unit, two tiles of rows, no segment
};

// ------------------------------------------------------------------ shared memory
// TWO: room for two tiles of queries (else one, and a tile of tokens more in the ring).
template <int D, bool TWO>
struct Smem {
    static constexpr int kSlots = TWO ? 10 : 12;            // five or six tiles
    static constexpr int kSegs = 2;                         // segments on their way from the scheduler
    static constexpr int kSlot = kTok * D * 2;              // a K or V tile in bf16
    static constexpr int kRegion = kTok * 128;              // 64 dimensions of it (128-byte rows, swizzled)
    static constexpr int kRaw = D == 64 ? kSlot / 2 : 0;    // where in its slot an FP8 tile lands
    static constexpr int kQ = 0;
    static constexpr int kQTile = kRows * D * 2;
    static constexpr int kRing = (TWO ? 2 : 1) * kQTile;
    static constexpr int kScale = kRing + kSlots * kSlot;   // float [kScales][2][kTok]: K and V scales
    static constexpr int kScales = 4;                       // tiles of scales, fewer than the ring has
    static constexpr int kBars = kScale + kScales * 2 * kTok * 4;
    // mbarriers.  K is in the even slots, V in the odd ones.  A slot's load completes on kFullB,
    // or on kRawB (K) or kRawB + kSlots (V) if the tile has to be converted first (kConvB tells
    // when): each barrier then has one reader that sees every one of its phases, whichever kinds
    // of tile come in between.
    static constexpr int kFullB = 0, kEmptyB = kSlots, kConvB = 2 * kSlots, kRawB = 3 * kSlots, kQFull = 5 * kSlots,
                         kQEmpty = kQFull + 1, kSFull = kQEmpty + 1, kPFull = kSFull + 4,
                         kScFree = kPFull + 4, kOFull = kScFree + kScales, kXch = kOFull + 1, kEpi = kXch + 1,
                         kFin = kEpi + 1, kCvt = kFin + 2, kSegFull = kCvt + 2, kSegEmpty = kSegFull + kSegs,
                         kNumBars = kSegEmpty + kSegs;
    static constexpr int kMisc = kBars + ((kNumBars * 8 + 15) & ~15);   // tensor-memory base, abort flag
    static constexpr int kSeg = kMisc + 16;                             // Seg [kSegs]
    static constexpr int kBytes = kSeg + kSegs * 64;
    static_assert(kScales < kSlots / 2, "see load_scales");
    static_assert(sizeof(Seg) <= 64 && kBytes <= 232448, "shared memory of one CTA");
};

// tensor-memory columns: two S (and P) of each of the two softmax warpgroups, then their O
constexpr uint32_t kTmemCols = 512;
__host__ __device__ constexpr uint32_t tmem_s(int wg, int buf) { return (uint32_t)(2 * wg + buf) * kTok; }
template <int D>
__host__ __device__ constexpr uint32_t tmem_o(int wg) { return 4 * kTok + (uint32_t)wg * D; }

// ------------------------------------------------------------------ schedule
struct AttnArgs {
    CUtensorMap tm_q;                       // [branches][hkv][G][D] bf16, boxes of 128 / G branches x G x 64
    CUtensorMap tm_k16, tm_v16, tm_k8, tm_v8;   // [R * cap][D], boxes of 128 tokens
    PrefixParams p;
    float4* part_o;      // [slots][row_tiles][D / 4][128 rows]: a warp's rows side by side
    float2* part_ml;     // [slots][row_tiles][128]
    int4* join;          // [branches][hkv]: first and last slot with a partial, row in it (none: last < first)
    unsigned div_hkv, div_unit, div_ctas;   // divisors hkv, branches of a unit, CTAs (see divided)
    int slots;
    int per_tile;        // branches of one tile of rows
    int row_tiles;       // tiles of rows of a unit, at most
};

// x / d for x d < 2^32, with m = floor(2^32 / d) + 1 made by the host (d = 1: m = 0).
__device__ __forceinline__ int divided(int x, unsigned m) { return m ? (int)__umulhi((unsigned)x, m) : x; }

__device__ __forceinline__ RowInfo row_info(const AttnArgs& a, int row) {
    const LayerDims& d = a.p.d;
    RowInfo r;
    const int pre = divided(row, a.div_hkv);
    r.n16 = __ldg(a.p.c.n_bf16 + row);
    r.n8 = __ldg(a.p.c.n_fp8 + row);
    int b0 = 0, b1 = a.p.branches;
    if (a.p.branch_start) {
        const int s0 = __ldg(a.p.branch_start + pre), s1 = __ldg(a.p.branch_start + pre + 1);
        b0 = min(max(s0, 0), b1);
        b1 = min(max(s1, b0), b1);
    }
    r.b0 = b0;
    r.nb = b1 - b0;
    r.mt = divided(r.nb + a.row_tiles * a.per_tile - 1, a.div_unit);
    r.n16 = min(max(r.n16, 0), d.cap_o);   // clamped to the capacities
    r.n8 = min(max(r.n8, 0), d.cap_q);
    r.T16 = (r.n16 + kTok - 1) / kTok;
    r.T8 = (r.n8 + kTok - 1) / kTok;
    return r;
}
// Places a unit of this row takes in the list.
__device__ __forceinline__ int unit_len(const RowInfo& r) { return r.T16 + r.T8 > 0 ? r.T16 + r.T8 + kSegCost : 0; }

// Run c of P CTAs over V places begins at c V / P (V = q P + r, so the product stays small).
struct Runs {
    int P, q, r;
    unsigned m;
    __device__ __forceinline__ Runs(int V, int ctas, unsigned div_ctas) : P(ctas), m(div_ctas) {
        if (V < ctas) {   // a place each
            P = V;
            q = 1;
            r = 0;
        } else {
            q = divided(V, m);   // one too many at most: V may be past 2^32 / ctas
            if (q * P > V) --q;
            r = V - q * P;
        }
    }
    __device__ __forceinline__ int begin(int c) const { return c * q + divided(c * r, m); }
};

struct Tile {
    int fp8, idx, valid;   // kind, place in its row's segment of the cache, live tokens
};

// The tiles of a segment in order: the bf16 tiles first.  (Alternating the two kinds makes the
// softmax warps fetch their code anew all the time.)
struct Tiles {
    int n, i16, e16, i8, n16, n8;
    __device__ __forceinline__ explicit Tiles(const Seg& s)   // (a whole warp)
        : n(uniform(s.n)), i16(uniform(s.i16)), e16(uniform(s.e16)), i8(uniform(s.i8)), n16(uniform(s.n16)),
          n8(uniform(s.n8)) {}
    __device__ __forceinline__ Tile next() {
        Tile x;
        x.fp8 = i16 >= e16;
        x.idx = x.fp8 ? i8++ : i16++;
        x.valid = min(kTok, (x.fp8 ? n8 : n16) - x.idx * kTok);
        return x;
    }
};

// ------------------------------------------------------------------ helpers
struct Ctx {
    uint32_t bars;
    volatile int* abort_flag;
    int32_t* status;
    __device__ __forceinline__ uint32_t bar(int i) const { return bars + 8u * i; }
    // A bounded wait for a phase; false if it ran out or the CTA is giving up.
    __device__ __forceinline__ bool wait(int i, uint32_t parity) const {
        const uint32_t b = bar(i);
        for (int k = 0; k < kSpinLimit; ++k) {
            if (mbar_try_wait(b, parity)) return true;
            if ((k & 31) == 31 && *abort_flag) return false;
        }
        *abort_flag = 1;
        atomicOr(status, ARKV_STATUS_TIMEOUT);
        return false;
    }
    // The same for a whole warp, with one outcome.
    __device__ __forceinline__ bool warp_wait(int i, uint32_t parity) const { return __all_sync(kFull, wait(i, parity)); }
};

// One arrival for a warp, after all its lanes (n: counted n times).
__device__ __forceinline__ void warp_arrive(uint32_t bar, uint32_t n = 1) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive_n(bar, n);
}

// Segment number `seg` from the scheduler, to a warp; false at the end of the run.
template <int D, bool TWO>
__device__ __forceinline__ bool warp_segment(const Ctx& cx, const char* smem, int seg, Seg& out) {
    using L = Smem<D, TWO>;
    const int z = seg % L::kSegs;
    if (!cx.warp_wait(L::kSegFull + z, (seg / L::kSegs) & 1)) return false;
    out = *reinterpret_cast<const Seg*>(smem + L::kSeg + z * 64);
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(cx.bar(L::kSegEmpty + z));
    return !(out.flags & kSegEnd);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
// Four FP8 codes (low byte first) -> two bf16x2 words, exact (NaN and infinities too).
template <int FMT>
__device__ __forceinline__ void fp8x4_to_bf16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    uint32_t h0, h1;   // f16 pairs
    if constexpr (FMT == ARKV_FMT_E5M2) {
        h0 = __byte_perm(w, 0u, 0x1404);   // E5M2 is the upper byte of the f16
        h1 = __byte_perm(w, 0u, 0x3424);
    } else {
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n}"
            : "=r"(h0), "=r"(h1)
            : "r"(w));
    }
    const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&h0));
    const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&h1));
    lo = pack_bf16(f0.x, f0.y);
    hi = pack_bf16(f1.x, f1.y);
}
// 16-byte chunk c of row r in rows of 128 (64) bytes under the 128-byte (64-byte) swizzle.
__device__ __forceinline__ uint32_t sw128(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }
__device__ __forceinline__ uint32_t sw64(int r, int c) { return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4)); }

// ------------------------------------------------------------------ products (one thread)
// Softmax job x of a segment belongs to warpgroup x & 1 and its S number (x >> 1) & 1: token
// tile x with one tile of rows, token tile x / 2 with two.  One warp issues the S, another the
// P V (one lane each), so that neither product waits behind the other's operands; S of job x
// follows the completion of P V of job x - 4, which read P from the same place.  (With one warp
// for both, polling for whichever was ready, a tile of 64 took 0.5 us more: it shares its
// scheduler with four busy warps, and its instructions were what a tile waited for.)
template <int D, bool TWO>
__device__ void multiply_qk(const Ctx& cx, const char* gsmem, uint32_t smem, uint32_t tmem) {
    using L = Smem<D, TWO>;
    constexpr uint32_t kIdQK = idesc_bf16(kRows, kTok, false);
    int j = 0;                     // tiles so far
    uint32_t full = 0, conv = 0;   // parity of each slot's next phase
    const bool leader = elect_one();
    const uint64_t q_desc = desc_sw128(smem + L::kQ, 16, 1024);
    Seg w{};
    for (int seg = 0; warp_segment<D, TWO>(cx, gsmem, seg, w); ++seg) {
        Tiles tiles(w);
        const bool two = TWO && (uniform(w.flags) & kSegTwo);
        const int sh = two ? 1 : 0, n = tiles.n, jobs = n << sh;
        if (!cx.warp_wait(L::kQFull, seg & 1) || (seg > 0 && !cx.warp_wait(L::kEpi, (seg - 1) & 1))) return;
#pragma unroll 1
        for (int x = 0; x < jobs; ++x) {
            const int b = x & 1, t = x >> sh, e = 2 * (j + t), s = e % L::kSlots;
            if (!two || b == 0) {
                const int before = t - (two ? 2 : 4);   // the tile whose P V frees this S
                const int ev = 2 * (j + before) + 1;
                if (before >= 0 && !cx.warp_wait(L::kEmptyB + ev % L::kSlots, (ev / L::kSlots) & 1)) return;
                const bool c = tiles.next().fp8;
                if (!cx.warp_wait((c ? L::kConvB : L::kFullB) + s, ((c ? conv : full) >> s) & 1u)) return;
                if (c) conv ^= 1u << s;
                else full ^= 1u << s;
            }
            fence_after();
            const uint64_t k_desc = desc_sw128(smem + L::kRing + s * L::kSlot, 16, 1024);
            const uint64_t qd = q_desc + (uint64_t)(two ? b * (L::kQTile >> 4) : 0);
            const uint32_t to = tmem + tmem_s(b, (x >> 1) & 1);
            if (leader) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    mma_ss(to, qd + (uint64_t)((k >> 2) * (kRows * 128 >> 4) + (k & 3) * 2),
                           k_desc + (uint64_t)((k >> 2) * (L::kRegion >> 4) + (k & 3) * 2), kIdQK, k > 0);
                commit(cx.bar(L::kSFull + (x & 3)));
                if (!two || b == 1) commit(cx.bar(L::kEmptyB + s));
                if (x + 1 == jobs) commit(cx.bar(L::kQEmpty));
            }
            __syncwarp();
        }
        j += n;
    }
}

template <int D, bool TWO>
__device__ void multiply_pv(const Ctx& cx, const char* gsmem, uint32_t smem, uint32_t tmem) {
    using L = Smem<D, TWO>;
    constexpr uint32_t kIdPV = idesc_bf16(kRows, D, true);
    int j = 0;                     // tiles so far
    uint32_t full = 0, conv = 0;   // parity of each slot's next phase
    int f = 0;                     // FP8 tiles so far
    bool fp8 = false;
    uint32_t p_ph = 0;             // parity of the next P of each of the four S
    const bool leader = elect_one();
    Seg w{};
    for (int seg = 0; warp_segment<D, TWO>(cx, gsmem, seg, w); ++seg) {
        Tiles tiles(w);
        const bool two = TWO && (uniform(w.flags) & kSegTwo);
        const int sh = two ? 1 : 0, n = tiles.n, jobs = n << sh;
#pragma unroll 1
        for (int x = 0; x < jobs; ++x) {
            const int b = x & 1, z = x & 3, e = 2 * (j + (x >> sh)) + 1, s = e % L::kSlots;
            if (!two || b == 0) {
                const Tile t = tiles.next();
                const bool c = t.fp8 || t.valid < kTok;
                fp8 = t.fp8;
                f += fp8;
                if (!cx.warp_wait((c ? L::kConvB : L::kFullB) + s, ((c ? conv : full) >> s) & 1u)) return;
                if (c) conv ^= 1u << s;
                else full ^= 1u << s;
            }
            if (!cx.warp_wait(L::kPFull + z, (p_ph >> z) & 1u)) return;
            p_ph ^= 1u << z;
            fence_after();
            const uint64_t v_desc = desc_sw128(smem + L::kRing + s * L::kSlot, L::kRegion, 1024);
            const uint32_t to = tmem + tmem_o<D>(b), from = tmem + tmem_s(b, (x >> 1) & 1);
            const bool add = x >= 2;   // each warpgroup's first product of the segment starts its O
            if (leader) {
#pragma unroll
                for (int k = 0; k < 2 * kTok / 16; ++k)   // the upper parts, then the lower ones
                    mma_ts(to, from + 8 * k, v_desc + (uint64_t)(k % (kTok / 16) * 128), kIdPV, add || k > 0);
                if (!two || b == 1) commit(cx.bar(L::kEmptyB + s));
                if (fp8 && (!two || b == 1)) commit(cx.bar(L::kScFree + (f - 1) % L::kScales));
                if (x + 1 == jobs) commit(cx.bar(L::kOFull));
            }
            __syncwarp();
        }
        j += n;
    }
}

// Waits until every product of this warp has completed (before tensor memory is freed).
template <int D, bool TWO>
__device__ __forceinline__ void drain(const Ctx& cx, int which) {
    using L = Smem<D, TWO>;
    if (elect_one()) commit(cx.bar(L::kFin + which));
    __syncwarp();
    for (int z = 0; z < kSpinLimit && !mbar_try_wait(cx.bar(L::kFin + which), 0); ++z) {
    }
}

// ------------------------------------------------------------------ FP8 scales (one warp)
// The K and V scales of every FP8 tile, by asynchronous copies up to kScales tiles ahead of the
// softmax (which waits a latency of HBM for them otherwise).  They count among the arrivals that
// let S = Q K^T of the tile begin, and the completion of its P V frees their place: a wait that
// need not wait costs a softmax warp 0.13 us all the same.
// Past the end of the row the last token's: what P = 0 meets has to be finite.
template <int D, bool TWO>
__device__ void load_scales(const AttnArgs& a, const Ctx& cx, char* smem) {
    using L = Smem<D, TWO>;
    const int lane = threadIdx.x & 31;
    const uint32_t to = smem_u32(smem + L::kScale) + 4 * lane;
    int f = 0, j = 0, last = 0;   // FP8 tiles, tiles so far; the last FP8 tile
    bool ok = true;
    Seg w{};
    for (int seg = 0; ok && warp_segment<D, TWO>(cx, smem, seg, w); ++seg) {
        const float* sk = a.p.c.sk + (size_t)w.row * a.p.d.cap_q;
        const float* sv = a.p.c.sv + (size_t)w.row * a.p.d.cap_q;
        Tiles tiles(w);
#pragma unroll 1
        for (int i = 0; i < tiles.n; ++i) {
            const Tile t = tiles.next();
            if (!t.fp8) continue;
            const int z = f % L::kScales, use = f / L::kScales;
            ok = use == 0 || cx.warp_wait(L::kScFree + z, (use - 1) & 1);   // its last readers
            if (!ok) break;
            // The slot's barrier has to be done with the FP8 tile that had the slot before.  In a run
            // of FP8 tiles that one is more than kScales back, so the wait above shows it; after bf16
            // tiles (of a new segment) every FP8 tile so far has to be done.
            if (f > 0 && j + i > last + 1)
                ok = cx.warp_wait(L::kScFree + (f - 1) % L::kScales, ((f - 1) / L::kScales) & 1);
            if (!ok) break;
#pragma unroll
            for (int c = 0; c < 2 * kTok; c += 32) {
                const int tok = min(t.idx * kTok + (c & (kTok - 1)) + lane, w.n8 - 1);
                cp_async4(to + 4 * (2 * z * kTok + c), (c < kTok ? sk : sv) + tok);
            }
            cp_async_arrive(cx.bar(L::kConvB + 2 * (j + i) % L::kSlots));
            last = j + i;
            ++f;
        }
        j += tiles.n;
    }
    cp_async_wait_all();   // (also when it gives up)
}

// ------------------------------------------------------------------ FP8 -> bf16 (128 threads, two a token)
// kv = 0: the K tiles, 1: the V tiles, whose rows past the segment end become zero in either
// format (stale bits must not meet P = 0).
template <int D, int FMT, bool TWO>
__device__ void convert(const Ctx& cx, char* smem, int ct, int kv) {
    using L = Smem<D, TWO>;
    const int row = ct >> 1, h = ct & 1;   // token of the tile, half of its dimensions
    int cvt = 0, j = 0;          // uses of the read-before-write barrier (D = 64); tiles so far
    uint32_t raw_ph = 0;         // parity of each slot's next phase (of the K or V loads to convert)
    Seg w{};
    for (int seg = 0; warp_segment<D, TWO>(cx, smem, seg, w); ++seg) {
        Tiles tiles(w);
#pragma unroll 1
        for (const int end = j + tiles.n; j < end; ++j) {
            const Tile cur = tiles.next();
            const bool tail = kv == 1 && !cur.fp8 && cur.valid < kTok;
            if (!cur.fp8 && !tail) continue;
            const int s = (2 * j + kv) % L::kSlots;
            if (!cx.warp_wait(L::kRawB + kv * L::kSlots + s, (raw_ph >> s) & 1u)) return;
            raw_ph ^= 1u << s;
            char* slot = smem + L::kRing + s * L::kSlot;
            const bool zero = kv == 1 && row >= cur.valid;
            if (!tail) {
                // D / 2 codes a thread.  A 128-byte row's codes lie where its lower half goes: both
                // threads of the row (one warp) read before either writes; rows of 64 codes grow
                // over other rows' codes, so all threads do.  The upper half goes through its
                // 16-byte chunks in another order, which keeps the two halves' banks apart.  (The
                // loop is short code, see softmax_job.)
                constexpr int N = D / 32;
                uint4 raw[N];
#pragma unroll
                for (int c = 0; c < N; ++c) {
                    const int at = D == 128 ? 4 * h + (c ^ (2 * h)) : 2 * h + c;
                    raw[c] = *reinterpret_cast<const uint4*>(slot + L::kRaw + (D == 128 ? sw128(row, at) : sw64(row, at)));
                    if (zero) raw[c] = make_uint4(0u, 0u, 0u, 0u);
                }
                if constexpr (D == 64) {
                    warp_arrive(cx.bar(L::kCvt + kv));
                    if (!cx.warp_wait(L::kCvt + kv, cvt++ & 1)) return;
                } else {
                    __syncwarp();
                }
                char* reg = slot + (D == 128 ? h * L::kRegion : 0);
                auto put = [&](const uint4& w, int c) {
                    uint4 lo, hi;
                    fp8x4_to_bf16<FMT>(w.x, lo.x, lo.y);
                    fp8x4_to_bf16<FMT>(w.y, lo.z, lo.w);
                    fp8x4_to_bf16<FMT>(w.z, hi.x, hi.y);
                    fp8x4_to_bf16<FMT>(w.w, hi.z, hi.w);
                    const int to = D == 128 ? 2 * (c ^ (2 * h)) : 4 * h + 2 * c;
                    *reinterpret_cast<uint4*>(reg + sw128(row, to)) = lo;
                    *reinterpret_cast<uint4*>(reg + sw128(row, to + 1)) = hi;
                };
#pragma unroll 1
                for (int c = 0; c < N; ++c) {
                    put(raw[0], c);
#pragma unroll
                    for (int i = 0; i + 1 < N; ++i) raw[i] = raw[i + 1];
                }
            } else if (zero) {
#pragma unroll 1
                for (int c = h; c < D / 8; c += 2)
                    *reinterpret_cast<uint4*>(slot + (c >> 3) * L::kRegion + row * 128 + ((c & 7) << 4)) =
                        make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async();
            warp_arrive(cx.bar(L::kConvB + s));
        }
    }
}

// ------------------------------------------------------------------ softmax (128 threads)
// A warp owns 32 rows (tensor-memory lanes).  S is read in the matrix layout: lane t holds of
// rows t / 4 + 8 k (k = 0..3) the columns 2 (t % 4), 2 (t % 4) + 1 of every 8, so that the
// per-column FP8 scales are read once for two rows (a lane a row, every lane reads every
// scale, and the shared memory's bandwidth sets the time).
// State of a lane's rows in log2 units (logit * log2(e) / sqrt(D)): the reference m of P
// and O (the same in the four lanes of a row), the largest logit top and the sum l of
// 2^(x - m), both of this lane's columns alone.
struct Rows {
    float m[4], top[4], l[4];
};

__device__ __forceinline__ void swap2(float& x, float& y) {
    const float t = x;
    x = y;
    y = t;
}
// Over the four lanes of a row.
__device__ __forceinline__ float quad_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(kFull, x, 1));
    return fmaxf(x, __shfl_xor_sync(kFull, x, 2));
}
__device__ __forceinline__ float quad_sum(float x) {
    x += __shfl_xor_sync(kFull, x, 1);
    return x + __shfl_xor_sync(kFull, x, 2);
}
// From the matrix layout to a lane a row: the value of row `lane`.
__device__ __forceinline__ float row_value(const float (&x)[4]) {
    const int lane = threadIdx.x & 31, src = 4 * (lane & 7);
    const float y0 = __shfl_sync(kFull, x[0], src), y1 = __shfl_sync(kFull, x[1], src);
    const float y2 = __shfl_sync(kFull, x[2], src), y3 = __shfl_sync(kFull, x[3], src);
    return lane < 16 ? (lane < 8 ? y0 : y1) : (lane < 24 ? y2 : y3);
}

// The reference of some of the warp's rows moves by a whole number of log2 units, so that O,
// weighed with the old one, is rescaled exactly, by ff for the row of this lane.
template <int D>
__device__ __noinline__ void rescale(uint32_t o, float ff) {
#pragma unroll 1
    for (int i = 0; i < D; i += 16) {
        float x[16];
        tmem_ld16(o + i, x);
        wait_ld(x);
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] *= ff;
        tmem_st16(o + i, x);
    }
    wait_st();
}

// One job: S at column s of the warp's lanes becomes P, 16 rows at a time by one piece of code
// (32 rows at once are twice the instructions, which with the conversion's do not fit the cache
// nearest to the schedulers).
// A half is run again when its reference turns out wrong: too low, or, in a segment's first
// job, which starts from zero, too high.  O (column o) then has to be idle: the product of the
// job before has completed when it frees its V, entry pv.  False if that took too long.
template <int D, bool FP8, bool TWO>
__device__ __forceinline__ bool softmax_job(const Ctx& cx, int pv, uint32_t s, uint32_t o, bool first, int valid,
                                            const float* sk, const float* sv, float c2, Rows& r) {
    const float2 cc = make_float2(c2, c2);
    const int col = 2 * (threadIdx.x & 3);
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
        bool begin = first;
        for (;;) {
            // row k of the half, columns 8 g + col and the next: va[4 g + 2 k ..]
            float va[32];
            tmem_ld_16x256b_x8(s + half * (16u << 16), va);
            wait_ld(va);
            if (FP8) {
#pragma unroll
                for (int g = 0; g < 8; ++g) {
                    const float2 ks = *reinterpret_cast<const float2*>(sk + 8 * g + col);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float* v = va + 4 * g + 2 * k;
                        const float2 x = mul2(make_float2(v[0], v[1]), ks);
                        v[0] = x.x;
                        v[1] = x.y;
                    }
                }
            }
            if (valid < kTok) {   // columns that are no tokens
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (8 * (i / 4) + col + (i & 1) >= valid) va[i] = kNegInf;
            }
            float mx[2];
            float2 l[2];
            uint32_t pa[16], pl[16];   // P of the two rows: [2 g + k], its upper and lower parts
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                mx[k] = kNegInf;
                l[k] = make_float2(0.f, 0.f);
            }
#pragma unroll
            for (int g = 0; g < 8; ++g) {
                float2 vs = make_float2(1.f, 1.f);
                if (FP8) vs = *reinterpret_cast<const float2*>(sv + 8 * g + col);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float* v = va + 4 * g + 2 * k;
                    const float2 x = make_float2(v[0], v[1]);
                    mx[k] = fmaxf(fmaxf(mx[k], x.x), x.y);
                    const float2 m2 = make_float2(-r.m[k], -r.m[k]);
                    float2 p = fma2(x, cc, m2);
                    p = make_float2(ex2(p.x), ex2(p.y));
                    l[k] = add2(l[k], p);
                    if (FP8) p = mul2(p, vs);
                    const uint32_t hi = pack_bf16(p.x, p.y);
                    pa[2 * g + k] = hi;
                    pl[2 * g + k] = pack_bf16(p.x - bf16_lo(hi), p.y - bf16_hi(hi));
                }
            }
            bool move = false, low = false;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                mx[k] *= c2;
                r.top[k] = fmaxf(r.top[k], mx[k]);
                move |= mx[k] > r.m[k] + 32.f;
                if (begin) low |= quad_max(mx[k]) < -32.f;
            }
            if (!__any_sync(kFull, move || low)) {
#pragma unroll
                for (int k = 0; k < 2; ++k) r.l[k] += l[k].x + l[k].y;
                tmem_st_16x128b_x8(s + half * (16u << 16), pa);   // over S, which has been read
                tmem_st_16x128b_x8(s + kTok / 2 + half * (16u << 16), pl);
                break;
            }
            float f[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float t = quad_max(mx[k]);
                if (begin) {
                    // (each row for itself; without any weight so far, below what a later logit has)
                    r.m[k] = t == kNegInf ? kNoLogit : fabsf(t) > 32.f ? t : 0.f;
                } else {
                    const float up = fmaxf(ceilf(t - r.m[k]), 0.f);
                    f[k] = ex2(-up);
                    r.m[k] += up;
                    r.l[k] *= f[k];
                }
            }
            if (!begin) {
                if (!cx.warp_wait(Smem<D, TWO>::kEmptyB + pv % Smem<D, TWO>::kSlots, (pv / Smem<D, TWO>::kSlots) & 1)) {
                    wait_st();
                    return false;
                }
                fence_after();
                const int lane = threadIdx.x & 31, src = 4 * (lane & 7);
                const float f0 = __shfl_sync(kFull, f[0], src), f1 = __shfl_sync(kFull, f[1], src);
                rescale<D>(o, lane >> 4 == half ? (lane & 8 ? f1 : f0) : 1.f);
            }
            begin = false;
        }
        // the other half's turn
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            swap2(r.m[k], r.m[k + 2]);
            swap2(r.top[k], r.top[k + 2]);
            swap2(r.l[k], r.l[k + 2]);
        }
    }
    wait_st();
    return true;
}

template <int D, bool TWO>
__device__ void softmax(const AttnArgs& a, const Ctx& cx, char* smem, uint32_t tmem, int b) {
    using L = Smem<D, TWO>;
    const LayerDims& d = a.p.d;
    const int quad = (threadIdx.x >> 5) & 3, row = quad * 32 + (threadIdx.x & 31);
    const uint32_t lane = tmem + ((uint32_t)(quad * 32) << 16), s = lane + tmem_s(b, 0), o = lane + tmem_o<D>(b);
    const float c2 = (float)(a.p.inv_sqrt_d * 1.4426950408889634);
    int f = 0, xch = 0, j = 0;      // FP8 tiles, exchanges and tiles so far
    uint32_t s_ph = 0;              // parity of the next of each of its two S
    for (int seg = 0;; ++seg) {
        // (what the end of the segment needs stays in shared memory until then)
        const Seg& w = *reinterpret_cast<const Seg*>(smem + L::kSeg + seg % L::kSegs * 64);
        if (!cx.warp_wait(L::kSegFull + seg % L::kSegs, (seg / L::kSegs) & 1) || (w.flags & kSegEnd)) return;
        const bool two = TWO && (w.flags & kSegTwo);
        Tiles tiles(w);
        const int n = tiles.n;
        Rows r;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            r.m[k] = 0.f;
            r.top[k] = kNegInf;
            r.l[k] = 0.f;
        }
        bool first = true;
#pragma unroll 1
        for (int x = 0; x < n; ++x) {
            const Tile t = tiles.next();
            const int z = f % L::kScales;
            f += t.fp8;
            if (!two && (x & 1) != b) continue;
            const int buf = (two ? x : x >> 1) & 1;
            if (!cx.warp_wait(L::kSFull + b + 2 * buf, (s_ph >> buf) & 1u)) return;
            s_ph ^= 1u << buf;
            fence_after();
            const int pv = 2 * (j + x - (two ? 1 : 2)) + 1;   // the V of this warpgroup's job before
            if (t.fp8) {
                const float* sk = reinterpret_cast<const float*>(smem + L::kScale) + 2 * z * kTok;
                if (!softmax_job<D, true, TWO>(cx, pv, s + buf * kTok, o, first, t.valid, sk, sk + kTok, c2, r)) return;
            } else {
                if (!softmax_job<D, false, TWO>(cx, pv, s + buf * kTok, o, first, t.valid, nullptr, nullptr, c2, r)) return;
            }
            first = false;
            fence_before();
            warp_arrive(cx.bar(L::kPFull + b + 2 * buf));
        }
        j += n;
        // The segment's partial, a lane a row from here.  With one tile of rows both warpgroups
        // hold half of the tokens: each gets the other's state (through S, idle by then) and adds
        // half of the columns.
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            r.top[k] = quad_max(r.top[k]);
            r.l[k] = quad_sum(r.l[k]);
        }
        const float m = row_value(r.m), my_top = row_value(r.top), my_l = row_value(r.l);
        if (!cx.warp_wait(L::kOFull, seg & 1)) return;
        fence_after();
        float y[4] = {0.f, kNegInf, 0.f, 0.f};
        if (!two) {
            tmem_st4(s, m, my_top, my_l, 0.f);
            wait_st();
            fence_before();
            warp_arrive(cx.bar(L::kXch));
            if (!cx.warp_wait(L::kXch, xch++ & 1)) return;
            fence_after();
            tmem_ld4(lane + tmem_s(b ^ 1, 0), y);
            wait_ld(y);
        }
        const bool mine = two || n > b, theirs = !two && n > (b ^ 1);   // who had a tile
        const float top = fmaxf(my_top, y[1]);   // a warpgroup without one has -inf
        // raw units for the join; what the rounding of the maximum moves goes into the weights
        const float M = top == kNegInf ? kNegInf : top / c2, at = top == kNegInf ? 0.f : M * c2;
        const float lo = top == kNegInf ? 0.f : fmaf(M, c2, -at);
        const float w_mine = ex2(m - at - lo), w_theirs = theirs ? ex2(y[0] - at - lo) : 0.f;
        const float sum = (mine ? my_l * w_mine : 0.f) + (theirs ? y[2] * w_theirs : 0.f);
        const int rt = two ? b : 0;
        const bool live = row < (rt ? w.rows1 : w.rows0) && w.slot < a.slots;
        const size_t at_slot = (size_t)w.slot * a.row_tiles + rt;
        if (live && (two || b == 0)) {
            a.part_ml[at_slot * kRows + row] = make_float2(M, sum);
            // the branch's slots, from its unit's first and last segment
            const int br = row / d.G;
            int4* to = a.join + (size_t)(w.branch + rt * a.per_tile + br) * d.hkv + w.row % d.hkv;
            if (row == br * d.G) {
                if (w.flags & kSegFirst) {
                    to->x = w.slot;
                    to->z = rt * kRows + row;
                }
                if (w.flags & kSegLast) to->y = w.slot;
            }
        }
        float4* out = a.part_o + at_slot * (D / 4) * kRows + row;
        const int c_begin = two ? 0 : b * (D / 2), c_end = two ? D : c_begin + D / 2;
#pragma unroll 1
        for (int c = c_begin; c < c_end; c += 16) {
            float u[16], v[16];
            tmem_ld16(o + c, u);   // (a warpgroup without a tile reads what it does not use)
            tmem_ld16(lane + tmem_o<D>(b ^ 1) + c, v);
            wait_ld(u, v);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                u[i] = mine ? u[i] * w_mine : 0.f;
                if (theirs) u[i] = fmaf(v[i], w_theirs, u[i]);
            }
            if (live) {
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                    __stcg(out + (size_t)((c + i) / 4) * kRows, make_float4(u[i], u[i + 1], u[i + 2], u[i + 3]));
            }
        }
        fence_before();
        warp_arrive(cx.bar(L::kEpi));
        warp_arrive(cx.bar(L::kSegEmpty + seg % L::kSegs));
    }
}

// ------------------------------------------------------------------ scheduler and producer (one warp)
// Inclusive scan of (x, y) over a warp.
__device__ __forceinline__ int2 warp_scan(int2 v) {
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int px = __shfl_up_sync(kFull, v.x, m), py = __shfl_up_sync(kFull, v.y, m);
        if ((threadIdx.x & 31) >= m) {
            v.x += px;
            v.y += py;
        }
    }
    return v;
}

// This CTA's run.  Lane l owns rows [l per, (l + 1) per): a scan of their places gives the
// list's length and, with it, the lane and then the row that hold the run's first place.
__device__ __forceinline__ Sched find_run(const AttnArgs& a) {
    const int lane = threadIdx.x & 31, R = a.p.d.R;
    const int per = (R + 31) / 32, r0 = min(R, lane * per), r1 = min(R, r0 + per);
    int2 x = make_int2(0, 0);
    RowInfo i{};
#pragma unroll 4
    for (int r = r0; r < r1; ++r) {
        i = row_info(a, r);
        x.x += i.mt * unit_len(i);
        x.y += i.mt;
    }
    const int2 s = warp_scan(x);
    const int V = __shfl_sync(kFull, s.x, 31);
    int at = s.x - x.x, units = s.y - x.y;
    Sched out{};
    const Runs runs(V, gridDim.x, a.div_ctas);
    if ((int)blockIdx.x >= runs.P) return out;
    const int v = runs.begin(blockIdx.x), v_end = runs.begin(blockIdx.x + 1);
    const bool here = v >= at && v < at + x.x;
    const int src = __ffs(__ballot_sync(kFull, here)) - 1;
    int row = r0;
    if (here && per > 1) {
        for (;; ++row) {
            i = row_info(a, row);
            const int n = i.mt * unit_len(i);
            if (v < at + n) break;
            at += n;
            units += i.mt;
        }
    }
    out.v = v;
    out.v_end = v_end;
    out.row = __shfl_sync(kFull, row, src);
    out.base = __shfl_sync(kFull, at, src);
    out.units = __shfl_sync(kFull, units, src);
    out.r.n16 = __shfl_sync(kFull, i.n16, src);
    out.r.n8 = __shfl_sync(kFull, i.n8, src);
    out.r.T16 = (out.r.n16 + kTok - 1) / kTok;
    out.r.T8 = (out.r.n8 + kTok - 1) / kTok;
    out.r.b0 = __shfl_sync(kFull, i.b0, src);
    out.r.nb = __shfl_sync(kFull, i.nb, src);
    out.r.mt = __shfl_sync(kFull, i.mt, src);
    return out;
}

// Walks the run (one warp, one lane of which issues): loads every segment's tiles and queries, and publishes the
// segment once its first loads are on their way (the other roles need it, and their code,
// only when those land).
template <int D, bool TWO>
__device__ void produce(const AttnArgs& a, const Ctx& cx, char* gsmem, uint32_t smem, Sched s) {
    using L = Smem<D, TWO>;
    const LayerDims& d = a.p.d;
    const int per_unit = a.row_tiles * a.per_tile;
    int seg = 0, e = 0, m = 0;              // segments and entries so far; place of the unit in its row
    int queries = 0;                        // loads of a segment's queries so far
    uint32_t ph[3] = {0, 0, 0}, last[3] = {0, 0, 0};   // by barrier (full, raw K, raw V): parity of each slot's next
                                                       // phase, the slots whose last load it has
    RowInfo r = s.r;
    int T = r.T16 + r.T8;
    if (r.mt > 1) {
        m = (s.v - s.base) / (T + kSegCost);
        s.base += m * (T + kSegCost);
    }
    Seg x{};
    const bool leader = elect_one();
    auto load = [&](const Tile& t, bool v) {
        const int z = e % L::kSlots;
        if (e >= L::kSlots && !cx.warp_wait(L::kEmptyB + z, ((e / L::kSlots) & 1) ^ 1)) return false;
        const int kind = t.fp8 || (v && t.valid < kTok) ? (v ? 2 : 1) : 0;
        const uint32_t dst = smem + L::kRing + z * L::kSlot;
        const uint32_t bar = cx.bar((kind == 0 ? L::kFullB : kind == 1 ? L::kRawB : L::kRawB + L::kSlots) + z);
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            if (i == kind) ph[i] ^= 1u << z;
            last[i] = i == kind ? last[i] | (1u << z) : last[i] & ~(1u << z);
        }
        const int y = x.row * (t.fp8 ? d.cap_q : d.cap_o) + t.idx * kTok;
        if (leader) {
            if (t.fp8) {
                mbar_expect_tx(bar, kTok * D);
                tma_load_2d(dst + L::kRaw, v ? &a.tm_v8 : &a.tm_k8, 0, y, bar);
            } else {
                mbar_expect_tx(bar, L::kSlot);
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                    tma_load_2d(dst + c * L::kRegion, v ? &a.tm_v16 : &a.tm_k16, 64 * c, y, bar);
            }
        }
        __syncwarp();
        ++e;
        return true;
    };
    bool ok = true, waited = !a.p.early_start;
    for (;;) {
        // the next segment
        bool any = false;
        int t0 = 0, t1 = 0;   // the run's tiles of the unit
        while (ok && !any && s.v < s.v_end) {
            while (s.v >= s.base + T + kSegCost) {   // the unit that holds place v
                s.base += T + kSegCost;
                if (++m >= r.mt) {
                    do {
                        s.units += r.mt;
                        if (++s.row >= d.R) {
                            s.v = s.v_end;   // (counts that changed during the call)
                            break;
                        }
                        r = row_info(a, s.row);
                        T = r.T16 + r.T8;
                    } while (T == 0 || r.mt == 0);
                    m = 0;
                }
                if (s.v >= s.v_end) break;
            }
            if (s.v >= s.v_end) break;
            t0 = max(s.v - s.base - kSegCost, 0);
            t1 = min(s.v_end - s.base - kSegCost, T);
            s.v = min(s.base + kSegCost + T, s.v_end);
            any = t0 < t1;
        }
        const int z = seg % L::kSegs;
        Seg* out = reinterpret_cast<Seg*>(gsmem + L::kSeg + z * 64);
        if (!any) {
            if (!ok || (seg >= L::kSegs && !cx.warp_wait(L::kSegEmpty + z, ((seg / L::kSegs) & 1) ^ 1))) break;
            if (leader) {
                out->flags = kSegEnd;
                mbar_arrive(cx.bar(L::kSegFull + z));
            }
            break;
        }
        // a share of the bf16 and of the FP8 tiles in proportion: of t tiles, floor(t T8 / T) are FP8
        auto fp8_of = [&](int t) { return T < 65536 ? (int)((unsigned)t * r.T8 / (unsigned)T) : (int)((long long)t * r.T8 / T); };
        const int f0 = t0 == 0 ? 0 : fp8_of(t0), f1 = t1 == T ? r.T8 : fp8_of(t1);
        x.n = t1 - t0;
        x.i16 = t0 - f0;
        x.e16 = t1 - f1;
        x.i8 = f0;
        x.row = s.row;
        x.n16 = r.n16;
        x.n8 = r.n8;
        const int left = r.nb - m * per_unit;
        x.branch = r.b0 + m * per_unit;
        x.flags = (t0 == 0 ? kSegFirst : 0) | (t1 == T ? kSegLast : 0) |
                  (a.row_tiles > 1 && left > a.per_tile ? kSegTwo : 0);
        // The segment's queries follow its first tiles: an early-started call fills its whole
        // ring before the wait for the previous kernel, and a later segment's queries wait
        // until the products of the one before have read theirs, which its first tile need not.
        Tiles tiles(x);
        const int n = x.n, ahead = min(n, seg == 0 && a.p.early_start ? L::kSlots / 2 : 1);
#pragma unroll 1
        for (int j = 0; ok && j < n; ++j) {
            const Tile t = tiles.next();
            ok = load(t, false) && load(t, true);
            if (!ok || j != ahead - 1) continue;
            if (!waited) {
                pdl_wait();
                waited = true;
            }
            if (seg > 0 && !(ok = cx.warp_wait(L::kQEmpty, (seg - 1) & 1))) continue;
            const int count = TWO && (x.flags & kSegTwo) ? 2 : 1, head = x.row - divided(x.row, a.div_hkv) * d.hkv;
            if (leader) {
                mbar_expect_tx(cx.bar(L::kQFull), count * a.per_tile * d.G * D * 2);
#pragma unroll 1
                for (int q = 0; q < count; ++q)
#pragma unroll
                    for (int c = 0; c < D / 64; ++c)
                        tma_load_4d(smem + L::kQ + q * L::kQTile + c * kRows * 128, &a.tm_q, 64 * c, 0, head,
                                    x.branch + q * a.per_tile, cx.bar(L::kQFull));
            }
            __syncwarp();
            ++queries;
            if (seg >= L::kSegs && !(ok = cx.warp_wait(L::kSegEmpty + z, ((seg / L::kSegs) & 1) ^ 1))) continue;
            x.rows0 = min(left, a.per_tile) * d.G;
            x.rows1 = max(min(left - a.per_tile, a.per_tile), 0) * d.G;
            x.slot = blockIdx.x + s.units + m;
            if (leader) {
                *out = x;
                mbar_arrive(cx.bar(L::kSegFull + z));
            }
            __syncwarp();
            ++seg;
        }
    }
    if (!waited) pdl_wait();
    // copies in flight land before the CTA ends, also when it gives up
#pragma unroll
    for (int i = 0; i < 3; ++i)
#pragma unroll 1
        for (int z = 0; z < L::kSlots; ++z)
            if ((last[i] >> z) & 1u)
                for (int k = 0; k < kSpinLimit && !mbar_try_wait(cx.bar((i == 0 ? L::kFullB : i == 1 ? L::kRawB : L::kRawB + L::kSlots) + z),
                                                                 ((ph[i] >> z) & 1u) ^ 1u); ++k) {
                }
    if (queries > 0)
        for (int k = 0; k < kSpinLimit && !mbar_try_wait(cx.bar(L::kQFull), (queries - 1) & 1); ++k) {
        }
}

// Tells the join which branches have no prefix token (a CTA's share of the branches).
// (Out of line, so that it does not lie between the loops that run all the time: a 42601-token
// prefix with 32 branches takes 63.9 us so and 65.5 inlined, but with 64 branches 97.9 and 94.8.)
__device__ __noinline__ void no_prefix(const AttnArgs& a) {
    const LayerDims& d = a.p.d;
    for (int b = blockIdx.x * 32 + (threadIdx.x & 31); b < a.p.branches; b += gridDim.x * 32) {
        int pre = 0;
        bool has = true;
        if (a.p.branch_start) {   // the last prefix that starts at or before b
            int hi = d.batch;
            while (hi - pre > 1) {
                const int mid = (pre + hi) / 2;
                if (__ldg(a.p.branch_start + mid) <= b) pre = mid;
                else hi = mid;
            }
            has = __ldg(a.p.branch_start + pre) <= b && b < __ldg(a.p.branch_start + pre + 1);
        }
        for (int g = 0; g < d.hkv; ++g) {
            const int row = pre * d.hkv + g;
            if (!has || (__ldg(a.p.c.n_bf16 + row) <= 0 && __ldg(a.p.c.n_fp8 + row) <= 0))
                a.join[(size_t)b * d.hkv + g] = make_int4(0, -1, 0, 0);
        }
    }
}

template <int D, int FMT, bool TWO>
__global__ void __launch_bounds__(kThreads, 1) prefix_attn_kernel(const __grid_constant__ AttnArgs a) {
    using L = Smem<D, TWO>;
    extern __shared__ __align__(1024) char smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_launch_dependents();
    const uint32_t base = smem_u32(smem);
    if (base & 1023) {   // the swizzled tiles need it; the CTA's shared memory starts there
        pdl_wait();
        if (tid == 0) atomicOr(a.p.c.status, ARKV_STATUS_TIMEOUT);
        return;
    }
    int* misc = reinterpret_cast<int*>(smem + L::kMisc);
    Ctx cx{base + L::kBars, misc + 1, a.p.c.status};
    // what needs nothing of the previous kernel comes before the wait for it
    if (warp == 2) tmem_alloc(base + L::kMisc, kTmemCols);
    if (tid < L::kNumBars) {
        const int i = tid;
        auto among = [&](int at, int count) { return i >= at && i < at + count; };
        int n = 1;                                                    // arrivals of a phase
        if (among(L::kConvB, L::kSlots) || among(L::kPFull, 4) || among(L::kCvt, 2)) n = 4;   // the warps of a group
        if (among(L::kXch, 1) || among(L::kEpi, 1)) n = 8;     // of two
        if (among(L::kConvB, L::kSlots) && (i - L::kConvB) % 2 == 0) n = 4 + 32;   // and the lanes that fetch scales
        if (among(L::kSegEmpty, L::kSegs)) n = 19;                    // the warps that read it
        mbar_init(cx.bar(i), n);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async();
    }
    // Rows of the query tiles that no copy fills (groups of 3: 126 and 127) are zero: their logits
    // would move references and have jobs run again (27.7 us against 26.8 for 5 prefixes of 3900
    // tokens on average, 4 key heads, 23 branches).
    for (int i = tid; i < (TWO ? 2 : 1) * (D / 64) * 128 / 16 * (kRows - a.per_tile * a.p.d.G); i += kThreads) {
        const int n = 8 * (kRows - a.per_tile * a.p.d.G);   // 16-byte pieces of 64 dimensions' rows
        *reinterpret_cast<uint4*>(smem + L::kQ + (i / n + 1) * (kRows * 128) - (i % n + 1) * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async();
    if (warp == 3 && lane == 0) {
        misc[1] = 0;
        prefetch_map(&a.tm_q); prefetch_map(&a.tm_k16); prefetch_map(&a.tm_v16); prefetch_map(&a.tm_k8);
        prefetch_map(&a.tm_v8);
    }
    if (warp == 0) {   // (a prefetch reads nothing that the kernel uses)
        const int r = min(lane, a.p.d.R - 1);
        prefetch_l2(a.p.c.n_bf16 + r);
        prefetch_l2(a.p.c.n_fp8 + r);
        if (a.p.branch_start) prefetch_l2(a.p.branch_start + divided(r, a.div_hkv));
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(misc);
    // Registers go to the softmax warpgroups: 80 + 2 x 56 + 2 x 144 = the 5 x 96 at launch.  Bounded
    // waits start when the previous kernel has finished.
    if (warp < 4) {
        set_regs<80, false>();
        if (warp == 0) {
            if (!a.p.early_start) pdl_wait();
            const Sched sched = find_run(a);
            produce<D, TWO>(a, cx, smem, base, sched);
        } else if (warp == 3) {
            pdl_wait();   // the workspace is the previous call's until it has finished
            no_prefix(a);   // while the first segment is on its way (at the end the CTA waits for it)
            load_scales<D, TWO>(a, cx, smem);
        } else if (warp == 1) {
            pdl_wait();
            multiply_qk<D, TWO>(cx, smem, base, uniform(tmem));
            drain<D, TWO>(cx, 0);
        } else if (warp == 2) {
            pdl_wait();
            multiply_pv<D, TWO>(cx, smem, base, uniform(tmem));
            drain<D, TWO>(cx, 1);
        }
    } else if (warp < 12) {
        set_regs<144, true>();
        pdl_wait();
        softmax<D, TWO>(a, cx, smem, tmem, (warp - 4) >> 2);
    } else {
        set_regs<56, false>();
        pdl_wait();
        convert<D, FMT, TWO>(cx, smem, tid & 127, (warp - 12) >> 2);
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    if (warp == 2) {
        fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ------------------------------------------------------------------ join
// One block per (branch, key head): thread = (4 dimensions, query of the group), four times:
// each quarter of the block takes every fourth partial, its loads all in flight at once; the
// quarters and the own part are joined in float32 in a fixed order, and o rounded to bf16.
// Differences of two maxima are small where a weight counts, so float32 keeps them.
template <int D>
__global__ void __launch_bounds__(4 * D) prefix_join_kernel(const __grid_constant__ AttnArgs a) {
    constexpr int kBatch = 5;
    __shared__ float2 sm_ml[4][4];
    __shared__ float4 sm_o[4][D];
    const LayerDims& d = a.p.d;
    const int tid = threadIdx.x % D, part = threadIdx.x / D, jq = tid & 3, c4 = tid >> 2;
    const int b = divided(blockIdx.x, a.div_hkv), g = blockIdx.x - b * d.hkv;
    const float c2 = (float)(a.p.inv_sqrt_d * 1.4426950408889634);
    const size_t mi = (size_t)blockIdx.x * 4 + jq, at = (((size_t)b * d.hq + g * d.G + jq) * D) / 4 + c4;
    pdl_wait();
    // Only now may the next kernel start: what came before the attention kernel is then complete
    // and visible to whatever that kernel reads ahead of its own wait.
    pdl_launch_dependents();
    const int4 info = __ldcg(a.join + blockIdx.x);
    const JoinSpan span = join_span(info.x, info.y, info.z, a.slots, a.row_tiles, kRows, d.G);
    float M = kNegInf, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (part == 0 && a.p.ml_own && jq < d.G) {
        const float2 own = a.p.ml_own[mi];
        const float4 o = reinterpret_cast<const float4*>(a.p.o_own)[at];
        if (own.y != 0.f) {   // L = 0: no own tokens
            M = own.x;
            L = own.y;
            acc = make_float4(L * o.x, L * o.y, L * o.z, L * o.w);
        }
    }
    const int last = jq < d.G ? span.last : -1;
    for (int c = span.first + part; c <= last; c += 4 * kBatch) {
        float2 ml[kBatch];
        float4 x[kBatch];
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            ml[q] = make_float2(kNegInf, 0.f);
            if (c + 4 * q <= last) {
                const size_t s = (size_t)(c + 4 * q) * a.row_tiles + span.row / kRows;
                ml[q] = __ldcg(a.part_ml + s * kRows + span.row % kRows + jq);
                x[q] = __ldcg(a.part_o + (s * (D / 4) + c4) * kRows + span.row % kRows + jq);
            }
        }
        float mb = M;
#pragma unroll
        for (int q = 0; q < kBatch; ++q) mb = fmaxf(mb, ml[q].y != 0.f ? ml[q].x : kNegInf);
        const float f = M == mb ? 1.f : ex2((M - mb) * c2);
        M = mb;
        L *= f;
        acc.x *= f; acc.y *= f; acc.z *= f; acc.w *= f;
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            if (ml[q].y == 0.f) continue;   // no weight (a NaN goes through)
            const float w = ml[q].x == M ? 1.f : ex2((ml[q].x - M) * c2);
            L = fmaf(ml[q].y, w, L);
            acc.x = fmaf(x[q].x, w, acc.x); acc.y = fmaf(x[q].y, w, acc.y);
            acc.z = fmaf(x[q].z, w, acc.z); acc.w = fmaf(x[q].w, w, acc.w);
        }
    }
    sm_o[part][tid] = acc;
    if (c4 == 0) sm_ml[part][jq] = make_float2(M, L);
    __syncthreads();
    if (part != 0 || jq >= d.G) return;
#pragma unroll
    for (int q = 1; q < 4; ++q) M = fmaxf(M, sm_ml[q][jq].y != 0.f ? sm_ml[q][jq].x : kNegInf);
    L = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const float2 ml = sm_ml[q][jq];
        if (ml.y == 0.f) continue;
        const float w = ml.x == M ? 1.f : ex2((ml.x - M) * c2);
        const float4 x = sm_o[q][tid];
        L = fmaf(ml.y, w, L);
        acc.x = fmaf(x.x, w, acc.x); acc.y = fmaf(x.y, w, acc.y);
        acc.z = fmaf(x.z, w, acc.z); acc.w = fmaf(x.w, w, acc.w);
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    reinterpret_cast<uint2*>(a.p.o)[at] =
        make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    if (c4 == 0 && a.p.ml) a.p.ml[mi] = make_float2(M, L);
}

// ------------------------------------------------------------------ host
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    });
    return fn;
}

bool make_map(CUtensorMap* m, const void* base, bool fp8, int D, long long rows) {
    auto fn = encode_fn();
    if (!fn) return false;
    const int eb = fp8 ? 1 : 2;
    cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)(D * eb)};
    cuuint32_t box[2] = {(cuuint32_t)(fp8 ? D : 64), kTok};
    cuuint32_t es[2] = {1, 1};
    return fn(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims,
              strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              fp8 && D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_q_map(CUtensorMap* m, const void* base, const LayerDims& d, int branches, int per_tile) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[4] = {(cuuint64_t)d.D, (cuuint64_t)d.G, (cuuint64_t)d.hkv, (cuuint64_t)branches};
    cuuint64_t strides[3] = {(cuuint64_t)d.D * 2, (cuuint64_t)d.G * d.D * 2, (cuuint64_t)d.hq * d.D * 2};
    cuuint32_t box[4] = {64, (cuuint32_t)d.G, 1, (cuuint32_t)per_tile};
    cuuint32_t es[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct PrefixWs {
    size_t part_o, part_ml, join, total;
    long long slots, units, places;
    int per_tile, row_tiles;
};

// A segment's partial goes to slot (CTA + unit): along the list each next segment raises one
// of the two, so the slots differ, and there are at most CTAs + units of them.  places: the
// longest the list can get.
PrefixWs ws_layout(const LayerDims& d, int branches) {
    PrefixWs w{};
    w.per_tile = kRows / d.G;
    w.row_tiles = branches > w.per_tile ? 2 : 1;
    w.units = (long long)d.hkv * (d.batch + branches / (w.row_tiles * w.per_tile));
    w.places = w.units * (((long long)d.cap_o + kTok - 1) / kTok + ((long long)d.cap_q + kTok - 1) / kTok + kSegCost);
    w.slots = kMaxCtas + w.units;
    auto al = [](size_t x) { return (x + 255) & ~(size_t)255; };
    const size_t rows = (size_t)w.slots * w.row_tiles * kRows;
    size_t off = 0;
    w.join = off;    off = al(off + sizeof(int4) * (size_t)branches * d.hkv);
    w.part_ml = off; off = al(off + sizeof(float2) * rows);
    w.part_o = off;  off = al(off + sizeof(float) * rows * d.D);
    w.total = off;
    return w;
}

}  // namespace

// Whether the kernels' 32-bit places, rows and divisions hold for these sizes.
bool prefix_sizes_fit(const LayerDims& d, int branches) {
    const PrefixWs w = ws_layout(d, branches);
    const long long blocks = (long long)branches * d.hkv, rows = (long long)d.batch * d.hkv;
    const long long per_unit = (long long)w.row_tiles * w.per_tile;
    return w.places <= 0x7fffffff && blocks <= 0x7fffffff && blocks * d.hkv <= 0xffffffffll && rows * d.hkv <= 0xffffffffll &&
           (branches + per_unit) * per_unit <= 0xffffffffll && rows * d.cap_o <= 0x7fffffff - 256 &&
           rows * d.cap_q <= 0x7fffffff - 256;
}
size_t prefix_ws_bytes(const LayerDims& d, int branches) { return ws_layout(d, branches).total; }

cudaError_t launch_prefix_attn(const PrefixParams& p, void* ws, cudaStream_t s) {
    const LayerDims& d = p.d;
    const PrefixWs w = ws_layout(d, p.branches);
    const long long blocks = (long long)p.branches * d.hkv;
    const long long per_unit = (long long)w.row_tiles * w.per_tile;
    AttnArgs a{};
    a.p = p;
    a.slots = (int)w.slots;
    a.per_tile = w.per_tile;
    a.row_tiles = w.row_tiles;
    a.join = reinterpret_cast<int4*>((char*)ws + w.join);
    a.part_ml = reinterpret_cast<float2*>((char*)ws + w.part_ml);
    a.part_o = reinterpret_cast<float4*>((char*)ws + w.part_o);
    const long long r16 = (long long)d.R * d.cap_o, r8 = (long long)d.R * d.cap_q;
    if (!make_q_map(&a.tm_q, p.q, d, p.branches, w.per_tile) || !make_map(&a.tm_k16, p.c.k16, false, d.D, r16) ||
        !make_map(&a.tm_v16, p.c.v16, false, d.D, r16) || !make_map(&a.tm_k8, p.c.k8, true, d.D, r8) ||
        !make_map(&a.tm_v8, p.c.v8, true, d.D, r8))
        return cudaErrorInvalidValue;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    long long ctas = sms < kMaxCtas ? sms : kMaxCtas;   // one an SM
    if (ctas > w.places) ctas = w.places;
    auto divisor = [](long long x) { return x == 1 ? 0u : (unsigned)(0x100000000ll / x + 1); };
    a.div_hkv = divisor(d.hkv);
    a.div_unit = divisor(per_unit);
    a.div_ctas = divisor(ctas);
    static unsigned char done[8][64], done_join[8][64];
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t lc{};
    lc.stream = s;
    lc.attrs = attr;
    lc.numAttrs = 1;
    auto go = [&](auto kernel, auto join, int which, int bytes) {
        // both with the largest shared-memory carveout: an SM runs them side by side only if it
        // need not change its split between them
        cudaError_t err = allow_max_dyn_smem(kernel, done[which]);
        if (err == cudaSuccess) err = allow_max_dyn_smem(join, done_join[which]);
        if (err != cudaSuccess) return err;
        lc.gridDim = dim3((unsigned)ctas);
        lc.blockDim = dim3(kThreads);
        lc.dynamicSmemBytes = (size_t)bytes;
        if ((err = cudaLaunchKernelEx(&lc, kernel, a)) != cudaSuccess) return err;
        lc.gridDim = dim3((unsigned)blocks);
        lc.blockDim = dim3(4 * (unsigned)d.D);
        lc.dynamicSmemBytes = 0;
        return cudaLaunchKernelEx(&lc, join, a);
    };
    auto pick = [&](auto dim, auto fmt, auto two, int which) {
        constexpr int D = decltype(dim)::value, F = decltype(fmt)::value;
        constexpr bool T = decltype(two)::value;
        return go(prefix_attn_kernel<D, F, T>, prefix_join_kernel<D>, which, Smem<D, T>::kBytes);
    };
    using std::integral_constant;
    auto with = [&](auto dim, auto fmt, int which) {
        if (w.row_tiles == 2) return pick(dim, fmt, std::true_type{}, which + 4);
        return pick(dim, fmt, std::false_type{}, which);
    };
    const integral_constant<int, 128> d128{};
    const integral_constant<int, 64> d64{};
    const integral_constant<int, ARKV_FMT_E4M3> e4m3{};
    const integral_constant<int, ARKV_FMT_E5M2> e5m2{};
    const bool e5 = d.fmt == ARKV_FMT_E5M2;
    if (d.D == 128) e = e5 ? with(d128, e5m2, 0) : with(d128, e4m3, 1);
    else e = e5 ? with(d64, e5m2, 2) : with(d64, e4m3, 3);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace arkv
