// arkv_prefix_attn: decode attention of many branches to the prefixes they share,
// joined with each branch's own part.
//
// The queries of a prefix's branches that meet the same key head are the rows of one
// matrix (row = branch x query of the group, tiles of 128 rows), so the prefix is read
// once for all of them and both products run on the tensor cores:
//   S[128 rows][128 tokens] = Q K^T,   O[128 rows][D] += P V,   P = 2^(S c - m).
//
// Work.  A unit is (prefix, key head, one or two tiles of rows); its tiles of 128 tokens
// are the bf16 and the FP8 tiles of the prefix row, interleaved evenly, because an FP8
// tile has twice the arithmetic per byte.  The tiles of all units form one list, cut into
// equal runs, one a CTA and one CTA an SM; a run that crosses units is several segments,
// each with a partial (max, sum, unnormalised o) in the workspace.  In the list every unit
// begins with kSegCost empty places, about what the start of another segment costs, so
// that the run that holds them has that many tiles less.
// prefix_join_kernel joins the partials and the branch's own part.
//
// A CTA: warp 0 streams K and V by TMA through a ring of slots (a slot is a tile's K or
// its V), warp 1 issues the products, two warpgroups do the softmax (thread = row =
// tensor-memory lane), each with its own S, P and O in tensor memory and its own state, so
// that neither waits for the other, and two warpgroups rewrite FP8 tiles in place as bf16
// (exact: 4 or 3 significant bits), one K, one V.  With one tile of rows the softmax
// warpgroups take the token tiles in turn and their two O are added at the end of the
// segment; with two each has its rows, and a token tile is loaded and converted once for
// both.  Either way a softmax job is one S, and the jobs alternate.
// P takes the place of S.  The K scale of an FP8 token enters the exponent's factor, its V
// scale is folded into P.  The softmax reference m moves only when a logit exceeds it by
// 2^8, so O is seldom rescaled.  P is rounded to bf16 once, the rounding that o itself
// gets; the sum is of the unrounded values.
// The loops over a tile's columns are not unrolled past 32: a short call runs each piece of
// code once or twice, and fetching it cost more than the arithmetic.
// Every wait is bounded: one that runs out raises ARKV_STATUS_TIMEOUT and a flag that
// ends every role, copies and products in flight are given a last bounded wait, tensor
// memory is freed and the call ends.
#include <math.h>
#include <mutex>

#include <cudaTypedefs.h>

#include "arkv_internal.cuh"
#include "tc.cuh"

namespace arkv {

namespace {

using namespace tc;

constexpr float kNegInf = -INFINITY;
constexpr unsigned kFull = 0xffffffffu;
constexpr int kRows = 128;            // query rows of a tile
constexpr int kTok = 128;             // tokens of a tile
constexpr int kWarps = 20;            // 4 of single roles, 2 x 4 softmax, 2 x 4 conversion
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxCtas = 192;         // of one call
constexpr int kSegCost = 3;           // a segment's start and end, in tiles
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

// ------------------------------------------------------------------ shared memory
template <int D>
struct Smem {
    static constexpr int kSlots = 5;
    static constexpr int kSlot = kTok * D * 2;              // a K or V tile in bf16
    static constexpr int kRegion = kTok * 128;              // 64 dimensions of it (128-byte rows, swizzled)
    static constexpr int kRaw = D == 64 ? kSlot / 2 : 0;    // where in its slot an FP8 tile lands
    static constexpr int kQ = 0;                            // two tiles of queries
    static constexpr int kQTile = kRows * D * 2;
    static constexpr int kRing = 2 * kQTile;
    static constexpr int kScale = kRing + kSlots * kSlot;   // float [2][2][kTok]: K (log2 units) and V scales
    static constexpr int kBars = kScale + 2 * 2 * kTok * 4;
    // mbarriers.  A slot's load completes on kFullB, or on kRawB (K) or kRawB + kSlots (V) if
    // the tile has to be converted first (kConvB tells when): each barrier then has one
    // reader that sees every one of its phases, whichever kinds of tile come in between.
    static constexpr int kFullB = 0, kEmptyB = kSlots, kConvB = 2 * kSlots, kRawB = 3 * kSlots, kQFull = 5 * kSlots,
                         kQEmpty = kQFull + 1, kSFull = kQEmpty + 1, kPFull = kSFull + 2, kScFull = kPFull + 2,
                         kScFree = kScFull + 2, kOFull = kScFree + 2, kXch = kOFull + 1, kEpi = kXch + 1,
                         kFin = kEpi + 1, kCvt = kFin + 1, kNumBars = kCvt + 2;
    static constexpr int kMisc = kBars + ((kNumBars * 8 + 15) & ~15);   // tensor-memory base, abort flag
    static constexpr int kSched = kMisc + 16;
    static constexpr int kSums = kSched + 64;                           // int2 [kWarps]: the scan's warp sums
    static constexpr int kBytes = kSums + kWarps * 8;
    static_assert(sizeof(Sched) <= 64 && kBytes <= 232448, "shared memory of one CTA");
};

// tensor-memory columns: S (and P) of the two warpgroups, then their O
constexpr uint32_t kTmemCols = 512;
__host__ __device__ constexpr uint32_t tmem_s(int b) { return (uint32_t)b * kTok; }
template <int D>
__host__ __device__ constexpr uint32_t tmem_o(int b) { return 2 * kTok + (uint32_t)b * D; }

// ------------------------------------------------------------------ schedule
struct AttnArgs {
    CUtensorMap tm_q;                       // [branches][hkv][G][D] bf16, boxes of 128 / G branches x G x 64
    CUtensorMap tm_k16, tm_v16, tm_k8, tm_v8;   // [R * cap][D], boxes of 128 tokens
    PrefixParams p;
    float4* part_o;      // [slots][row_tiles][D / 4][128 rows]: a warp's rows side by side
    float2* part_ml;     // [slots][row_tiles][128]
    int2* unit_slots;    // [R][row_units]: the first and last slot with a partial of a unit
    int row_units;       // units of a row, at most
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
    int fp8, idx, valid;   // kind, place in its segment, live tokens
};

// Walks a CTA's run: segments (the run's tiles of one unit), then their tiles.
struct Walk {
    const AttnArgs& a;
    int v, v_end, base;         // next place, end of the run, first place of the unit
    int row, m, unit0;          // the unit: row, place in it; units before the row
    RowInfo r;
    int T, i, i_end, err, f8;   // tiles of the unit; next tile and end of the segment; the interleave

    __device__ __forceinline__ Walk(const AttnArgs& args, const Sched& s)
        : a(args), v(s.v), v_end(s.v_end), base(s.base), row(s.row), m(0), unit0(s.units), r(s.r), T(r.T16 + r.T8), i(0),
          i_end(0), err(0), f8(0) {
        if (r.mt > 1) {
            m = (v - base) / (T + kSegCost);
            base += m * (T + kSegCost);
        }
    }
    __device__ __forceinline__ bool segment() {
        while (v < v_end) {
            while (v >= base + T + kSegCost) {
                base += T + kSegCost;
                if (++m >= r.mt) {
                    do {
                        unit0 += r.mt;
                        if (++row >= a.p.d.R) return false;
                        r = row_info(a, row);
                        T = r.T16 + r.T8;
                    } while (T == 0 || r.mt == 0);
                    m = 0;
                }
            }
            i = max(v - base - kSegCost, 0);
            i_end = min(v_end - base - kSegCost, T);
            v = min(base + kSegCost + T, v_end);
            if (i < i_end) {   // after i tiles, floor(i T8 / T) are FP8
                if (T < 65536) {
                    const unsigned w = (unsigned)i * r.T8;
                    f8 = w / (unsigned)T;
                    err = w - f8 * T;
                } else {
                    const long long w = (long long)i * r.T8;
                    f8 = (int)(w / T);
                    err = (int)(w - (long long)f8 * T);
                }
                return true;
            }
        }
        return false;
    }
    __device__ __forceinline__ Tile tile() {
        Tile x;
        err += r.T8;
        x.fp8 = err >= T;
        if (x.fp8) {
            err -= T;
            x.idx = f8++;
            x.valid = min(kTok, r.n8 - x.idx * kTok);
        } else {
            x.idx = i - f8;
            x.valid = min(kTok, r.n16 - x.idx * kTok);
        }
        ++i;
        return x;
    }
    __device__ __forceinline__ int first_branch() const { return m * a.row_tiles * a.per_tile; }   // of the prefix's
    __device__ __forceinline__ bool two() const { return r.nb - first_branch() > a.per_tile; }     // tiles of rows
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

// ------------------------------------------------------------------ producer (one thread)
template <int D>
__device__ void produce(const AttnArgs& a, const Ctx& cx, uint32_t smem, Walk w) {
    using L = Smem<D>;
    const LayerDims& d = a.p.d;
    int e = 0, seg = 0;
    uint32_t ph[3] = {0, 0, 0}, last[3] = {0, 0, 0};   // by barrier (full, raw K, raw V): parity of each slot's next
                                                       // phase, the slots whose last load it has
    bool ok = true, waited = !a.p.early_start;
    auto load = [&](const Tile& x, bool v) {
        const int s = e % L::kSlots;
        if (e >= L::kSlots && !cx.wait(L::kEmptyB + s, ((e / L::kSlots) & 1) ^ 1)) return false;
        const bool conv = x.fp8 || (v && x.valid < kTok);
        const int kind = conv ? (v ? 2 : 1) : 0;
        const uint32_t dst = smem + L::kRing + s * L::kSlot;
        const uint32_t bar = cx.bar((kind == 0 ? L::kFullB : kind == 1 ? L::kRawB : L::kRawB + L::kSlots) + s);
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            if (i == kind) ph[i] ^= 1u << s;
            last[i] = i == kind ? last[i] | (1u << s) : last[i] & ~(1u << s);
        }
        if (x.fp8) {
            mbar_expect_tx(bar, kTok * D);
            tma_load_2d(dst + L::kRaw, v ? &a.tm_v8 : &a.tm_k8, 0, w.row * d.cap_q + x.idx * kTok, bar);
        } else {
            mbar_expect_tx(bar, L::kSlot);
            const int y = w.row * d.cap_o + x.idx * kTok;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) tma_load_2d(dst + c * L::kRegion, v ? &a.tm_v16 : &a.tm_k16, 64 * c, y, bar);
        }
        ++e;
        return true;
    };
    while (ok && w.segment()) {
        // The segment's queries follow its first tiles: an early-started call fills its whole
        // ring before the wait for the previous kernel, and a later segment's queries wait
        // until the products of the one before have read theirs, which its first tile need not.
        const int n = w.i_end - w.i, ahead = min(n, seg == 0 && a.p.early_start ? L::kSlots / 2 : 1);
        for (int j = 0; ok && j < n; ++j) {
            const Tile x = w.tile();
            ok = load(x, false) && load(x, true);
            if (!ok || j != ahead - 1) continue;
            if (!waited) {
                pdl_wait();
                waited = true;
            }
            if (seg > 0 && !(ok = cx.wait(L::kQEmpty, (seg - 1) & 1))) continue;
            const int tiles = w.two() ? 2 : 1, b0 = w.r.b0 + w.first_branch();
            mbar_expect_tx(cx.bar(L::kQFull), tiles * a.per_tile * d.G * D * 2);
            for (int t = 0; t < tiles; ++t)
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                    tma_load_4d(smem + L::kQ + t * L::kQTile + c * L::kRegion, &a.tm_q, 64 * c, 0, w.row % d.hkv,
                                b0 + t * a.per_tile, cx.bar(L::kQFull));
            ++seg;
        }
    }
    // copies in flight land before the CTA ends, also when it gives up
#pragma unroll
    for (int i = 0; i < 3; ++i)
        for (int s = 0; s < L::kSlots; ++s)
            if ((last[i] >> s) & 1u)
                for (int z = 0; z < kSpinLimit && !mbar_try_wait(cx.bar((i == 0 ? L::kFullB : i == 1 ? L::kRawB : L::kRawB + L::kSlots) + s),
                                                                 ((ph[i] >> s) & 1u) ^ 1u); ++z) {
                }
    if (seg > 0)
        for (int z = 0; z < kSpinLimit && !mbar_try_wait(cx.bar(L::kQFull), (seg - 1) & 1); ++z) {
        }
}

// ------------------------------------------------------------------ products (one thread)
// Softmax job x of a segment belongs to warpgroup x & 1: token tile x with one tile of
// rows, token tile x / 2 with two.  S of job x + 1 is issued before P V of job x, and so
// after that of job x - 1, which read P from the same place.
template <int D>
__device__ void multiply(const AttnArgs& a, const Ctx& cx, uint32_t smem, uint32_t tmem, Walk w) {
    using L = Smem<D>;
    constexpr uint32_t kIdQK = idesc_bf16(kRows, kTok, false), kIdPV = idesc_bf16(kRows, D, true);
    int j = 0, seg = 0;            // tiles and segments so far
    uint32_t full = 0, conv = 0;   // parity of each slot's next phase
    uint32_t p_ph = 0;             // parity of each warpgroup's next P
    bool ok = true;
    const uint64_t q_desc = desc_sw128(smem + L::kQ, 16, 1024);
    auto ready = [&](int e, bool converted) {   // entry e has landed (and been converted)
        const int s = e % L::kSlots;
        uint32_t& ph = converted ? conv : full;
        const bool r = cx.wait((converted ? L::kConvB : L::kFullB) + s, (ph >> s) & 1u);
        ph ^= 1u << s;
        return r;
    };
    while (ok && w.segment()) {
        const bool two = w.two();
        const int sh = two ? 1 : 0, n = w.i_end - w.i, jobs = n << sh;
        ok = cx.wait(L::kQFull, seg & 1) && (seg == 0 || cx.wait(L::kEpi, (seg - 1) & 1));
        uint32_t conv_v = 0;       // by job & 1: its V tile is converted
        Tile t{};
        for (int x = 0; ok && x <= jobs; ++x) {
            if (x < jobs) {        // S of job x
                const int b = x & 1, e = 2 * (j + (x >> sh)), s = e % L::kSlots;
                const bool opens = !two || b == 0, closes = !two || b == 1;   // the tile's first, last job
                if (opens) {
                    t = w.tile();
                    if (!(ok = ready(e, t.fp8))) break;
                    fence_after();
                }
                conv_v = (conv_v & ~(1u << b)) | ((uint32_t)(t.fp8 || t.valid < kTok) << b);
                const uint64_t k_desc = desc_sw128(smem + L::kRing + s * L::kSlot, 16, 1024);
                const uint64_t qd = q_desc + (uint64_t)(two ? b * (L::kQTile >> 4) : 0);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint64_t o = (uint64_t)((k >> 2) * (L::kRegion >> 4) + (k & 3) * 2);
                    mma_ss(tmem + tmem_s(b), qd + o, k_desc + o, kIdQK, k > 0);
                }
                commit(cx.bar(L::kSFull + b));
                if (closes) commit(cx.bar(L::kEmptyB + s));
                if (x + 1 == jobs) commit(cx.bar(L::kQEmpty));
            }
            if (x > 0) {           // P V of job x - 1
                const int y = x - 1, b = y & 1, e = 2 * (j + (y >> sh)) + 1, s = e % L::kSlots;
                const bool opens = !two || b == 0, closes = !two || b == 1;
                if (!(ok = cx.wait(L::kPFull + b, (p_ph >> b) & 1u) && (!opens || ready(e, (conv_v >> b) & 1u)))) break;
                p_ph ^= 1u << b;
                fence_after();
                const uint64_t v_desc = desc_sw128(smem + L::kRing + s * L::kSlot, L::kRegion, 1024);
                const bool add = y >= 2;   // each warpgroup's first product of the segment starts its O
#pragma unroll
                for (int k = 0; k < kTok / 16; ++k)
                    mma_ts(tmem + tmem_o<D>(b), tmem + tmem_s(b) + 8 * k, v_desc + (uint64_t)(k * 128), kIdPV,
                           add || k > 0);
                if (closes) commit(cx.bar(L::kEmptyB + s));
                if (x == jobs) commit(cx.bar(L::kOFull));
            }
        }
        j += n;
        ++seg;
    }
    // every product has completed before tensor memory is freed
    commit(cx.bar(L::kFin));
    for (int z = 0; z < kSpinLimit && !mbar_try_wait(cx.bar(L::kFin), 0); ++z) {
    }
}

// ------------------------------------------------------------------ FP8 -> bf16 (128 threads, one a token)
// KV = 0: the K tiles and the scales, 1: the V tiles, whose rows past the segment end
// become zero in either format (stale bits must not meet P = 0).
template <int D, int FMT, int KV>
__device__ void convert(const AttnArgs& a, const Ctx& cx, char* smem, int ct, Walk w) {
    using L = Smem<D>;
    const LayerDims& d = a.p.d;
    const float c2 = (float)(a.p.inv_sqrt_d * 1.4426950408889634);
    float* scales = reinterpret_cast<float*>(smem + L::kScale);
    int cvt = 0, f = 0;      // uses of the read-before-write barrier (D = 64); FP8 tiles so far
    uint32_t raw_ph = 0;     // parity of each slot's next phase (of the K or V loads to convert)
    auto next = [&](Tile& x) {
        if (w.i == w.i_end && !w.segment()) return false;
        x = w.tile();
        return true;
    };
    auto load_scales = [&](const Tile& x, int row, float& sk, float& sv) {
        sk = 1.f;            // past the segment end: a masked column
        sv = 0.f;
        if (KV == 0 && x.fp8 && ct < x.valid) {
            const size_t at = (size_t)row * d.cap_q + x.idx * kTok + ct;
            sk = __ldg(a.p.c.sk + at) * c2;
            sv = __ldg(a.p.c.sv + at);
        }
    };
    Tile cur{}, ahead{};
    float sk, sv, sk1 = 0.f, sv1 = 0.f;
    if (!next(cur)) return;
    load_scales(cur, w.row, sk, sv);
#pragma unroll 1
    for (int j = 0;; ++j) {
        const bool more = next(ahead);   // the next tile's scales are loaded one tile early
        if (more) load_scales(ahead, w.row, sk1, sv1);
        const int s = (2 * j + KV) % L::kSlots;
        const bool tail = KV == 1 && !cur.fp8 && cur.valid < kTok;
        if (cur.fp8 || tail) {
            if (KV == 0) {
                const int z = f & 1, use = f >> 1;
                if (use > 0 && !cx.warp_wait(L::kScFree + z, (use - 1) & 1)) return;   // their last readers
                scales[(2 * z) * kTok + ct] = sk;
                scales[(2 * z + 1) * kTok + ct] = sv;
                mbar_arrive(cx.bar(L::kScFull + z));
                ++f;
            }
            if (!cx.warp_wait(L::kRawB + KV * L::kSlots + s, (raw_ph >> s) & 1u)) return;
            raw_ph ^= 1u << s;
            char* slot = smem + L::kRing + s * L::kSlot;
            const bool zero = KV == 1 && ct >= cur.valid;
            if (!tail) {
                // 64 dimensions at a time, the upper half of a 128-byte row first: the codes lie
                // where the lower half goes
#pragma unroll 1
                for (int h = D / 64 - 1; h >= 0; --h) {
                    uint4 raw[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        raw[c] = *reinterpret_cast<const uint4*>(
                            slot + L::kRaw + (D == 128 ? sw128(ct, 4 * h + c) : sw64(ct, c)));
                        if (zero) raw[c] = make_uint4(0u, 0u, 0u, 0u);
                    }
                    if constexpr (D == 64) {   // rows grow over other threads' codes (D = 128: over their own alone)
                        mbar_arrive(cx.bar(L::kCvt + KV));
                        if (!cx.warp_wait(L::kCvt + KV, cvt++ & 1)) return;
                    }
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint4 lo, hi;
                        fp8x4_to_bf16<FMT>(raw[c].x, lo.x, lo.y);
                        fp8x4_to_bf16<FMT>(raw[c].y, lo.z, lo.w);
                        fp8x4_to_bf16<FMT>(raw[c].z, hi.x, hi.y);
                        fp8x4_to_bf16<FMT>(raw[c].w, hi.z, hi.w);
                        char* reg = slot + h * L::kRegion;
                        *reinterpret_cast<uint4*>(reg + sw128(ct, 2 * c)) = lo;
                        *reinterpret_cast<uint4*>(reg + sw128(ct, 2 * c + 1)) = hi;
                    }
                }
            } else if (zero) {
#pragma unroll
                for (int c = 0; c < D / 8; ++c)
                    *reinterpret_cast<uint4*>(slot + (c >> 3) * L::kRegion + ct * 128 + ((c & 7) << 4)) =
                        make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async();
            mbar_arrive(cx.bar(L::kConvB + s));
        }
        if (!more) return;
        cur = ahead;
        sk = sk1;
        sv = sv1;
    }
}

// ------------------------------------------------------------------ softmax (128 threads, one a row)
// Row state in log2 units (logit * log2(e) / sqrt(D)): the reference m of P and O, the
// largest logit top, the sum l of 2^(x - m).
struct Row {
    float m, top, l;
};

// Sixteen columns of S: those from `valid` on are no tokens; times their K scales (FP8).
template <bool FP8>
__device__ __forceinline__ void logits16(float (&v)[16], int valid, const float* sk) {
    float4 k[4];
    if (FP8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) k[i] = reinterpret_cast<const float4*>(sk)[i];
    }
    wait_ld(v);
    if (valid < 16) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (i >= valid) v[i] = kNegInf;
    }
    if (FP8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = mul2(make_float2(v[4 * i], v[4 * i + 1]), make_float2(k[i].x, k[i].y));
            const float2 y = mul2(make_float2(v[4 * i + 2], v[4 * i + 3]), make_float2(k[i].z, k[i].w));
            v[4 * i] = x.x; v[4 * i + 1] = x.y; v[4 * i + 2] = y.x; v[4 * i + 3] = y.y;
        }
    }
}

// One job: S at column s of this thread's lane becomes P.  O (column o) is idle while it
// lasts: the product into S came after the last one into O.  S is read twice, 16 columns at
// a time.
template <int D, bool FP8>
__device__ __forceinline__ void softmax_job(uint32_t s, uint32_t o, bool first, int valid, const float* sk,
                                            const float* sv, float c2, Row& r) {
    float v[16];
    float mx[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll 1
    for (int c = 0; c < kTok; c += 16) {
        tmem_ld16(s + c, v);
        logits16<FP8>(v, valid - c, sk + c);
#pragma unroll
        for (int i = 0; i < 16; i += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e) mx[e] = fmaxf(fmaxf(mx[e], v[i + e]), v[i + 4 + e]);
    }
    float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
    if (!FP8) top *= c2;
    r.top = fmaxf(r.top, top);
    if (first) {
        r.m = top == kNegInf ? 0.f : top;
    } else {
        const bool move = top > r.m + 8.f;
        if (__any_sync(kFull, move)) {
            const float f = move ? ex2(r.m - top) : 1.f;
            r.l *= f;
            if (move) r.m = top;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                float x[32];
                tmem_ld32(o + c, x);
                wait_ld(x);
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] *= f;
                tmem_st32(o + c, x);
            }
        }
    }
    const float2 m2 = make_float2(-r.m, -r.m), cc = FP8 ? make_float2(1.f, 1.f) : make_float2(c2, c2);
    float2 l = make_float2(0.f, 0.f);
#pragma unroll 1
    for (int c = 0; c < kTok; c += 16) {
        tmem_ld16(s + c, v);
        logits16<FP8>(v, valid - c, sk + c);
        uint32_t pk[8];
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            float4 f = make_float4(1.f, 1.f, 1.f, 1.f);
            if (FP8) f = *reinterpret_cast<const float4*>(sv + c + i);
            float2 a = FP8 ? add2(make_float2(v[i], v[i + 1]), m2) : fma2(make_float2(v[i], v[i + 1]), cc, m2);
            float2 b = FP8 ? add2(make_float2(v[i + 2], v[i + 3]), m2) : fma2(make_float2(v[i + 2], v[i + 3]), cc, m2);
            a = make_float2(ex2(a.x), ex2(a.y));
            b = make_float2(ex2(b.x), ex2(b.y));
            l = add2(l, add2(a, b));
            if (FP8) {
                a = mul2(a, make_float2(f.x, f.y));
                b = mul2(b, make_float2(f.z, f.w));
            }
            pk[i / 2] = pack_bf16(a.x, a.y);
            pk[i / 2 + 1] = pack_bf16(b.x, b.y);
        }
        tmem_st8(s + c / 2, pk);   // over columns of S that have been read
    }
    r.l += l.x + l.y;
    wait_st();
}

template <int D>
__device__ void softmax(const AttnArgs& a, const Ctx& cx, char* smem, uint32_t tmem, int b, Walk w, int cta) {
    using L = Smem<D>;
    const LayerDims& d = a.p.d;
    const int quad = (threadIdx.x >> 5) & 3, row = quad * 32 + (threadIdx.x & 31);
    const uint32_t lane = tmem + ((uint32_t)(quad * 32) << 16), s = lane + tmem_s(b), o = lane + tmem_o<D>(b);
    const float c2 = (float)(a.p.inv_sqrt_d * 1.4426950408889634);
    int seg = 0, f = 0, xch = 0;   // segments, FP8 tiles and exchanges so far
    uint32_t s_ph = 0;         // parity of this warpgroup's next S
    while (w.segment()) {
        const bool two = w.two();
        const int i0 = w.i, n = w.i_end - i0;
        Row r{0.f, kNegInf, 0.f};
        bool first = true;
#pragma unroll 1
        for (int x = 0; x < n; ++x) {
            const Tile t = w.tile();
            const int z = f & 1, use = (f >> 1) & 1;
            f += t.fp8;
            if (!two && (x & 1) != b) continue;
            if (!cx.warp_wait(L::kSFull + b, s_ph)) return;
            s_ph ^= 1u;
            fence_after();
            if (t.fp8) {
                if (!cx.warp_wait(L::kScFull + z, use)) return;   // complete: K came after the scales
                const float* sk = reinterpret_cast<const float*>(smem + L::kScale) + 2 * z * kTok;
                softmax_job<D, true>(s, o, first, t.valid, sk, sk + kTok, c2, r);
            } else {
                softmax_job<D, false>(s, o, first, t.valid, nullptr, nullptr, c2, r);
            }
            first = false;
            fence_before();
            mbar_arrive(cx.bar(L::kPFull + b));
            if (t.fp8) mbar_arrive_n(cx.bar(L::kScFree + z), two ? 1 : 2);   // 256 in all, whoever read them
        }
        if (!cx.warp_wait(L::kOFull, seg & 1)) return;
        fence_after();
        // The segment's partial.  With one tile of rows both warpgroups hold half of the tokens:
        // each gets the other's state (through S, idle now) and adds half of the columns.
        float y[4] = {0.f, kNegInf, 0.f, 0.f};
        if (!two) {
            tmem_st4(s, r.m, r.top, r.l, 0.f);
            wait_st();
            fence_before();
            mbar_arrive(cx.bar(L::kXch));
            if (!cx.warp_wait(L::kXch, xch++ & 1)) return;
            fence_after();
            tmem_ld4(lane + tmem_s(b ^ 1), y);
            wait_ld(y);
        }
        const bool mine = two || n > b, theirs = !two && n > (b ^ 1);   // who had a tile
        const float top = fmaxf(r.top, y[1]);   // a warpgroup without one has -inf
        // raw units for the join; what the rounding of the maximum moves goes into the weights
        const float M = top == kNegInf ? kNegInf : top / c2, at = top == kNegInf ? 0.f : M * c2;
        const float lo = top == kNegInf ? 0.f : fmaf(M, c2, -at);
        const float w_mine = ex2(r.m - at - lo), w_theirs = theirs ? ex2(y[0] - at - lo) : 0.f;
        const float sum = (mine ? r.l * w_mine : 0.f) + (theirs ? y[2] * w_theirs : 0.f);
        const int slot = cta + w.unit0 + w.m, rt = two ? b : 0;
        const int rows = min(a.per_tile, w.r.nb - w.first_branch() - rt * a.per_tile) * d.G;
        const bool live = row < rows && slot < a.slots;
        if (b == 0 && row == 0) {   // the unit's slots, from its first and its last segment
            int2* us = a.unit_slots + (size_t)w.row * a.row_units + w.m;
            if (i0 == 0) us->x = slot;
            if (w.i_end == w.T) us->y = slot;
        }
        const size_t at_slot = (size_t)slot * a.row_tiles + rt;
        if (live && (two || b == 0)) a.part_ml[at_slot * kRows + row] = make_float2(M, sum);
        float4* out = a.part_o + at_slot * (D / 4) * kRows + row;
        const int c_begin = two ? 0 : b * (D / 2), c_end = two ? D : c_begin + D / 2;
#pragma unroll 1
        for (int c = c_begin; c < c_end; c += 32) {
            float u[32], v[32];
            if (mine) {
                tmem_ld32(o + c, u);
                wait_ld(u);
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) u[i] = mine ? u[i] * w_mine : 0.f;
            if (theirs) {
                tmem_ld32(lane + tmem_o<D>(b ^ 1) + c, v);
                wait_ld(v);
#pragma unroll
                for (int i = 0; i < 32; ++i) u[i] = fmaf(v[i], w_theirs, u[i]);
            }
            if (live) {
#pragma unroll
                for (int i = 0; i < 32; i += 4)
                    __stcg(out + (size_t)((c + i) / 4) * kRows, make_float4(u[i], u[i + 1], u[i + 2], u[i + 3]));
            }
        }
        fence_before();
        mbar_arrive(cx.bar(L::kEpi));
        ++seg;
    }
}

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

// This CTA's run, up to 32 rows: every warp for itself, a lane a row.
__device__ __forceinline__ Sched schedule_warp(const AttnArgs& a) {
    const int lane = threadIdx.x & 31;
    RowInfo i{};
    if (lane < a.p.d.R) i = row_info(a, lane);
    const int n = i.mt * unit_len(i);
    const int2 s = warp_scan(make_int2(n, i.mt));
    const int V = __shfl_sync(kFull, s.x, 31), at = s.x - n;
    Sched out{};
    const Runs runs(V, gridDim.x, a.div_ctas);
    if ((int)blockIdx.x >= runs.P) return out;
    out.v = runs.begin(blockIdx.x);
    out.v_end = runs.begin(blockIdx.x + 1);
    const int src = __ffs(__ballot_sync(kFull, out.v >= at && out.v < at + n)) - 1;
    out.row = src;
    out.base = __shfl_sync(kFull, at, src);
    out.units = __shfl_sync(kFull, s.y - i.mt, src);
    out.r.n16 = __shfl_sync(kFull, i.n16, src);
    out.r.n8 = __shfl_sync(kFull, i.n8, src);
    out.r.T16 = (out.r.n16 + kTok - 1) / kTok;
    out.r.T8 = (out.r.n8 + kTok - 1) / kTok;
    out.r.b0 = __shfl_sync(kFull, i.b0, src);
    out.r.nb = __shfl_sync(kFull, i.nb, src);
    out.r.mt = __shfl_sync(kFull, i.mt, src);
    return out;
}

// The same for any number: a block scan over the rows (threads own contiguous ones), then the
// thread whose rows hold the run's first place hands over where that is.
template <int D>
__device__ __noinline__ void schedule_block(const AttnArgs& a, char* smem) {
    using L = Smem<D>;
    Sched* out = reinterpret_cast<Sched*>(smem + L::kSched);
    int2* sums = reinterpret_cast<int2*>(smem + L::kSums);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, R = a.p.d.R;
    const int per = (R + kThreads - 1) / kThreads, r0 = min(R, tid * per), r1 = min(R, r0 + per);
    int2 x = make_int2(0, 0);
    for (int r = r0; r < r1; ++r) {
        const RowInfo i = row_info(a, r);
        x.x += i.mt * unit_len(i);
        x.y += i.mt;
    }
    const int2 s = warp_scan(x);
    if (lane == 31) sums[warp] = s;
    if (tid == 0) *out = Sched{};
    __syncthreads();
    int V = 0, at = s.x - x.x, units = s.y - x.y;
    for (int i = 0; i < kWarps; ++i) {
        const int2 z = sums[i];
        V += z.x;
        if (i < warp) {
            at += z.x;
            units += z.y;
        }
    }
    const Runs runs(V, gridDim.x, a.div_ctas);
    if ((int)blockIdx.x < runs.P) {
        const int v0 = runs.begin(blockIdx.x);
        for (int r = r0; r < r1 && at <= v0; ++r) {
            const RowInfo i = row_info(a, r);
            const int n = i.mt * unit_len(i);
            if (v0 < at + n) *out = Sched{v0, runs.begin(blockIdx.x + 1), at, r, units, i};
            at += n;
            units += i.mt;
        }
    }
    __syncthreads();
}

template <int D, int FMT>
__global__ void __launch_bounds__(kThreads, 1) prefix_attn_kernel(const __grid_constant__ AttnArgs a) {
    using L = Smem<D>;
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
        int n = 1;
        if ((i >= L::kConvB && i < L::kConvB + L::kSlots) || (i >= L::kPFull && i < L::kPFull + 2) ||
            (i >= L::kScFull && i < L::kScFull + 2) || i >= L::kCvt)
            n = 128;
        if (i == L::kXch || i == L::kEpi || (i >= L::kScFree && i < L::kScFree + 2)) n = 256;
        mbar_init(cx.bar(i), n);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async();
    }
    if (warp == 3 && lane == 0) {
        misc[1] = 0;
        prefetch_map(&a.tm_q); prefetch_map(&a.tm_k16); prefetch_map(&a.tm_v16); prefetch_map(&a.tm_k8);
        prefetch_map(&a.tm_v8);
    }
    // (a prefetch reads nothing that the kernel uses)
    if (warp == 0) {
        const int r = min(lane, a.p.d.R - 1);
        prefetch_l2(a.p.c.n_bf16 + r);
        prefetch_l2(a.p.c.n_fp8 + r);
        if (a.p.branch_start) prefetch_l2(a.p.branch_start + divided(r, a.div_hkv));
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(misc);
    if (!a.p.early_start) pdl_wait();
    Sched sched;
    if (a.p.d.R <= 32) {
        sched = schedule_warp(a);
    } else {
        schedule_block<D>(a, smem);
        sched = *reinterpret_cast<const Sched*>(smem + L::kSched);
    }
    if (sched.v < sched.v_end) {   // the same for the whole CTA
        // registers go to the softmax warpgroups: 80 + 2 x 72 + 2 x 128 = the 5 x 96 at launch
        if (warp < 4) set_regs<80, false>();
        if (warp == 0) {
            if (lane == 0) produce<D>(a, cx, base, Walk(a, sched));
        } else if (warp == 1) {
            if (lane == 0) {
                pdl_wait();   // bounded waits start when the previous kernel has finished
                multiply<D>(a, cx, base, tmem, Walk(a, sched));
            }
        } else if (warp >= 16) {
            set_regs<72, false>();
            pdl_wait();
            convert<D, FMT, 1>(a, cx, smem, tid - 512, Walk(a, sched));
        } else if (warp >= 12) {
            set_regs<72, false>();
            pdl_wait();
            convert<D, FMT, 0>(a, cx, smem, tid - 384, Walk(a, sched));
        } else if (warp >= 4) {
            set_regs<128, true>();
            pdl_wait();
            softmax<D>(a, cx, smem, tmem, (warp - 4) >> 2, Walk(a, sched), blockIdx.x);
        }
    }
    if (blockIdx.x == 0 && warp == 3) pdl_wait();   // the grid outlasts the previous kernel even with nothing to do
    __syncwarp();
    fence_before();
    __syncthreads();
    if (warp == 2) {
        fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ------------------------------------------------------------------ join
// One block per (branch, key head): thread = (4 dimensions, query of the group).  The partials
// of the row in CTA order and the own part, joined in float32; o is rounded to bf16.  The
// loads of a batch of partials are all in flight at once.
template <int D>
__global__ void __launch_bounds__(D) prefix_join_kernel(const __grid_constant__ AttnArgs a) {
    constexpr int kBatch = 10;
    const LayerDims& d = a.p.d;
    const int jq = threadIdx.x & 3, c4 = threadIdx.x >> 2;
    const int b = divided(blockIdx.x, a.div_hkv), g = blockIdx.x - b * d.hkv;
    pdl_launch_dependents();
    pdl_wait();
    if (jq >= d.G) return;
    const size_t mi = (size_t)blockIdx.x * 4 + jq, at = (((size_t)b * d.hq + g * d.G + jq) * D) / 4 + c4;
    float2 own = make_float2(kNegInf, 0.f);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.p.ml_own) {
        own = a.p.ml_own[mi];
        acc = reinterpret_cast<const float4*>(a.p.o_own)[at];
    }
    int pre = 0, b0 = 0;
    bool has = true;
    if (a.p.branch_start) {   // the last prefix that starts at or before b
        int hi = d.batch;
        while (hi - pre > 1) {
            const int mid = (pre + hi) / 2;
            if (__ldg(a.p.branch_start + mid) <= b) pre = mid;
            else hi = mid;
        }
        b0 = __ldg(a.p.branch_start + pre);
        has = b0 <= b && b < __ldg(a.p.branch_start + pre + 1);
        b0 = max(b0, 0);
    }
    const int row = pre * d.hkv + g, m = divided(b - b0, a.div_unit);
    const int in_unit = b - b0 - m * a.row_tiles * a.per_tile, rt = in_unit >= a.per_tile;
    const int rr = (in_unit - rt * a.per_tile) * d.G + jq;
    int2 slots = make_int2(0, -1);
    if (has) {
        slots = __ldcg(a.unit_slots + (size_t)row * a.row_units + min(m, a.row_units - 1));
        if (min(__ldg(a.p.c.n_bf16 + row), d.cap_o) <= 0 && min(__ldg(a.p.c.n_fp8 + row), d.cap_q) <= 0) slots.y = -1;
        slots.x = max(slots.x, 0);
        slots.y = min(slots.y, a.slots - 1);
    }
    const float c2 = (float)(a.p.inv_sqrt_d * 1.4426950408889634);
    float M = own.y != 0.f ? own.x : kNegInf, L = own.y;   // L = 0: no own tokens
    acc = own.y != 0.f ? make_float4(L * acc.x, L * acc.y, L * acc.z, L * acc.w) : make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = slots.x; c <= slots.y; c += kBatch) {
        float2 ml[kBatch];
        float4 x[kBatch];
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            ml[q] = make_float2(kNegInf, 0.f);
            if (c + q <= slots.y) {
                const size_t s = (size_t)(c + q) * a.row_tiles + rt;
                ml[q] = __ldcg(a.part_ml + s * kRows + rr);
                x[q] = __ldcg(a.part_o + (s * (D / 4) + c4) * kRows + rr);
            }
        }
        float mb = M;
#pragma unroll
        for (int q = 0; q < kBatch; ++q) mb = fmaxf(mb, ml[q].y != 0.f ? ml[q].x : kNegInf);
        // differences are small where a weight counts, so float32 keeps them
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
    size_t part_o, part_ml, unit_slots, total;
    long long slots, units, places;
    int per_tile, row_tiles, row_units;
};

// A segment's partial goes to slot (CTA + unit): along the list each next segment raises one
// of the two, so the slots differ, and there are at most CTAs + units of them.  places: the
// longest the list can get.
PrefixWs ws_layout(const LayerDims& d, int branches) {
    PrefixWs w{};
    w.per_tile = kRows / d.G;
    w.row_tiles = branches > w.per_tile ? 2 : 1;
    w.row_units = (branches + w.row_tiles * w.per_tile - 1) / (w.row_tiles * w.per_tile);
    w.units = (long long)d.hkv * (d.batch + branches / (w.row_tiles * w.per_tile));
    w.places = w.units * (((long long)d.cap_o + kTok - 1) / kTok + ((long long)d.cap_q + kTok - 1) / kTok + kSegCost);
    w.slots = kMaxCtas + w.units;
    auto al = [](size_t x) { return (x + 255) & ~(size_t)255; };
    const size_t rows = (size_t)w.slots * w.row_tiles * kRows;
    size_t off = 0;
    w.unit_slots = off; off = al(off + sizeof(int2) * (size_t)d.R * w.row_units);
    w.part_ml = off; off = al(off + sizeof(float2) * rows);
    w.part_o = off;  off = al(off + sizeof(float) * rows * d.D);
    w.total = off;
    return w;
}

}  // namespace

size_t prefix_ws_bytes(const LayerDims& d, int branches) { return ws_layout(d, branches).total; }

cudaError_t launch_prefix_attn(const PrefixParams& p, void* ws, cudaStream_t s) {
    const LayerDims& d = p.d;
    const PrefixWs w = ws_layout(d, p.branches);
    const long long blocks = (long long)p.branches * d.hkv;
    const long long per_unit = (long long)w.row_tiles * w.per_tile;
    if (w.places > 0x7fffffff || blocks * d.hkv > 0xffffffffll || (long long)d.R * d.hkv > 0xffffffffll ||
        (p.branches + per_unit) * per_unit > 0xffffffffll)
        return cudaErrorInvalidValue;
    AttnArgs a{};
    a.p = p;
    a.slots = (int)w.slots;
    a.per_tile = w.per_tile;
    a.row_tiles = w.row_tiles;
    a.unit_slots = reinterpret_cast<int2*>((char*)ws + w.unit_slots);
    a.row_units = w.row_units;
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
    static unsigned char done[4][64], done_join[4][64];
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
        lc.blockDim = dim3((unsigned)d.D);
        lc.dynamicSmemBytes = 0;
        return cudaLaunchKernelEx(&lc, join, a);
    };
    if (d.D == 128)
        e = d.fmt == ARKV_FMT_E5M2
                ? go(prefix_attn_kernel<128, ARKV_FMT_E5M2>, prefix_join_kernel<128>, 0, Smem<128>::kBytes)
                : go(prefix_attn_kernel<128, ARKV_FMT_E4M3>, prefix_join_kernel<128>, 1, Smem<128>::kBytes);
    else
        e = d.fmt == ARKV_FMT_E5M2 ? go(prefix_attn_kernel<64, ARKV_FMT_E5M2>, prefix_join_kernel<64>, 2, Smem<64>::kBytes)
                                   : go(prefix_attn_kernel<64, ARKV_FMT_E4M3>, prefix_join_kernel<64>, 3, Smem<64>::kBytes);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace arkv
