// arkv_prefix_attn: decode attention of many branches to the prefixes they share,
// joined with each branch's own part.
//
// The queries of a prefix's branches that meet the same key head are the rows of one
// matrix (row = branch x query of the group, 128 rows a tile), so the prefix is read
// once for all of them and both products run on the tensor cores:
//   S[128 rows][128 tokens] = Q K^T,   O[128 rows][D] += P V,   P = 2^(S c - m).
//
// Work.  A unit is (prefix, key head, tile of rows); its tiles of 128 tokens are the
// bf16 and the FP8 tiles of the prefix row, interleaved evenly, because an FP8 tile has
// twice the arithmetic per byte.  The tiles of all units form one list, cut into equal
// runs, one a CTA and one CTA an SM; a run that crosses units is several segments, each
// with a partial (max, sum, unnormalised o) of its own in the workspace.
// prefix_join_kernel joins the partials and the branch's own part.
//
// A CTA: warp 0 streams K and V by TMA through a ring of slots (a slot is a tile's K or
// its V), warp 1 issues the products, two warpgroups take the tiles in turn (softmax;
// thread = row = tensor-memory lane), each with its own S, P and O in tensor memory and
// its own softmax state, so that neither waits for the other, and one warpgroup rewrites
// FP8 tiles in place as bf16 (exact: 4 or 3 significant bits).  P takes the place of S.
// The K scale of an FP8 token enters the exponent's factor, its V scale is folded into P.
// The softmax reference m moves only when a logit exceeds it by 2^8, so O is seldom
// rescaled.  P is rounded to bf16 once, the rounding that o itself gets; the sum is of
// the unrounded values.
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
constexpr int kRows = 128;            // query rows of a unit
constexpr int kTok = 128;             // tokens of a tile
constexpr int kThreads = 512;
constexpr int kMaxCtas = 192;         // of one call
constexpr int kSpinLimit = 1 << 20;   // polls of one wait

// ------------------------------------------------------------------ shared memory
template <int D>
struct Smem {
    static constexpr int kSlots = 6;                        // three tiles in flight
    static constexpr int kSlot = kTok * D * 2;              // a K or V tile in bf16
    static constexpr int kRegion = kTok * 128;              // 64 dimensions of it (128-byte rows, swizzled)
    static constexpr int kRaw = D == 64 ? kSlot / 2 : 0;    // where in its slot an FP8 tile lands
    static constexpr int kQ = 0;
    static constexpr int kRing = kRows * D * 2;
    static constexpr int kScale = kRing + kSlots * kSlot;   // float [2][2][kTok]: K (log2 units) and V scales
    static constexpr int kBars = kScale + 2 * 2 * kTok * 4;
    // mbarriers.  A slot's load completes on kFullB, or on kRawB if the tile has to be
    // converted first (kConvB tells when): each barrier then has one reader that sees every
    // one of its phases, whichever kinds of tile come in between.
    static constexpr int kFullB = 0, kEmptyB = kSlots, kRawB = 2 * kSlots, kConvB = 3 * kSlots, kQFull = 4 * kSlots,
                         kQEmpty = kQFull + 1, kSFull = kQEmpty + 1, kPFull = kSFull + 2, kScFull = kPFull + 2,
                         kScFree = kScFull + 2, kOFull = kScFree + 2, kXch = kOFull + 1, kEpi = kXch + 1,
                         kFin = kEpi + 1, kCvt = kFin + 1, kNumBars = kCvt + 1;
    static constexpr int kMisc = kBars + ((kNumBars * 8 + 15) & ~15);   // tensor-memory base, abort flag
    static constexpr int kSched = kMisc + 16;                           // this CTA's run
    static constexpr int kSums = kSched + 32;                           // longlong2 [16]: the scan's warp sums
    static constexpr int kBytes = kSums + 16 * 16;
    static_assert(kBytes <= 232448, "shared memory of one CTA");
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
    float* part_o;       // [slots][128][D]
    float2* part_ml;     // [slots][128]
    longlong2* starts;   // [R + 1]: tiles and units before each row
    int slots;
    int per_tile;        // branches of one unit
};

struct RowInfo {
    int n16, n8, T16, T8, b0, nb, mt;   // live slots, tiles, first branch, branches, units
};

__device__ __forceinline__ RowInfo row_info(const AttnArgs& a, int row) {
    const LayerDims& d = a.p.d;
    RowInfo r;
    const int pre = row / d.hkv;
    int b0 = 0, b1 = a.p.branches;
    if (a.p.branch_start) {
        b0 = min(max(__ldg(a.p.branch_start + pre), 0), b1);
        b1 = min(max(__ldg(a.p.branch_start + pre + 1), b0), b1);
    }
    r.b0 = b0;
    r.nb = b1 - b0;
    r.mt = (r.nb + a.per_tile - 1) / a.per_tile;
    r.n16 = min(max(__ldg(a.p.c.n_bf16 + row), 0), d.cap_o);   // clamped to the capacities
    r.n8 = min(max(__ldg(a.p.c.n_fp8 + row), 0), d.cap_q);
    r.T16 = (r.n16 + kTok - 1) / kTok;
    r.T8 = (r.n8 + kTok - 1) / kTok;
    return r;
}

// Run of CTA c of P over T tiles: [c T / P, (c + 1) T / P); the CTA of tile t.
__device__ __forceinline__ long long run_begin(long long T, int P, int c) { return T * c / P; }
__device__ __forceinline__ int run_of(long long T, int P, long long t) { return (int)(((t + 1) * P + T - 1) / T) - 1; }

struct Sched {
    long long t, t_end, base;   // this CTA's run; tiles before `row`
    int row, units;             // the row that holds tile t; units before it
};

struct Tile {
    int fp8, idx, valid;   // kind, place in its segment, live tokens
};

// Walks a CTA's run: segments (the run's part of one unit), then their tiles.
struct Walk {
    const AttnArgs& a;
    long long t, t_end, base;   // next tile, end of the run, first tile of the unit
    int row, m, unit0;          // the unit: row, tile of rows; units before the row
    RowInfo r;
    int T, i, i_end, err, f8;   // tiles of the unit; next tile and end of the segment; the interleave

    __device__ __forceinline__ Walk(const AttnArgs& args, const Sched& s)
        : a(args), t(s.t), t_end(s.t_end), base(s.base), row(s.row), m(0), unit0(s.units), r(row_info(args, s.row)),
          T(r.T16 + r.T8), i(0), i_end(0), err(0), f8(0) {
        if (T > 0) {
            m = (int)((t - base) / T);
            base += (long long)m * T;
        }
    }
    __device__ __forceinline__ bool segment() {
        if (t >= t_end) return false;
        while (t >= base + T) {
            base += T;
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
        i = (int)(t - base);
        i_end = (int)min((long long)T, t_end - base);
        const long long w = (long long)i * r.T8;   // after i tiles, floor(i T8 / T) are FP8
        f8 = (int)(w / T);
        err = (int)(w - (long long)f8 * T);
        t = base + i_end;
        return true;
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
    uint32_t full = 0, raw = 0, last = 0;   // parity of each slot's next phase; which barrier its last load is on
    bool ok = true, waited = !a.p.early_start;
    auto load = [&](const Tile& x, bool v) {
        const int s = e % L::kSlots;
        if (e >= L::kSlots && !cx.wait(L::kEmptyB + s, ((e / L::kSlots) & 1) ^ 1)) return false;
        const bool conv = x.fp8 || (v && x.valid < kTok);
        const uint32_t dst = smem + L::kRing + s * L::kSlot, bar = cx.bar((conv ? L::kRawB : L::kFullB) + s);
        if (conv) {
            raw ^= 1u << s;
            last |= 1u << s;
        } else {
            full ^= 1u << s;
            last &= ~(1u << s);
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
            mbar_expect_tx(cx.bar(L::kQFull), a.per_tile * d.G * D * 2);
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
                tma_load_4d(smem + L::kQ + c * L::kRegion, &a.tm_q, 64 * c, 0, w.row % d.hkv, w.r.b0 + w.m * a.per_tile,
                            cx.bar(L::kQFull));
            ++seg;
        }
    }
    // copies in flight land before the CTA ends, also when it gives up
    for (int s = 0; s < min(e, L::kSlots); ++s) {
        const bool r = (last >> s) & 1u;
        const uint32_t par = (((r ? raw : full) >> s) & 1u) ^ 1u;
        for (int z = 0; z < kSpinLimit && !mbar_try_wait(cx.bar((r ? L::kRawB : L::kFullB) + s), par); ++z) {
        }
    }
    if (seg > 0)
        for (int z = 0; z < kSpinLimit && !mbar_try_wait(cx.bar(L::kQFull), (seg - 1) & 1); ++z) {
        }
}

// ------------------------------------------------------------------ products (one thread)
template <int D>
__device__ void multiply(const AttnArgs& a, const Ctx& cx, uint32_t smem, uint32_t tmem, Walk w) {
    using L = Smem<D>;
    constexpr uint32_t kIdQK = idesc_bf16(kRows, kTok, false), kIdPV = idesc_bf16(kRows, D, true);
    int j = 0, seg = 0;        // tiles and segments so far
    uint32_t full = 0, conv = 0;   // parity of each slot's next phase
    bool ok = true;
    const uint64_t q_desc = desc_sw128(smem + L::kQ, 16, 1024);
    auto ready = [&](int e, bool converted) {   // entry e has landed (and been converted)
        const int s = e % L::kSlots;
        uint32_t& ph = converted ? conv : full;
        const bool r = cx.wait((converted ? L::kConvB : L::kFullB) + s, (ph >> s) & 1u);
        ph ^= 1u << s;
        return r;
    };
    auto qk = [&](const Tile& x, int jj, bool last) {
        const int e = 2 * jj, s = e % L::kSlots, b = jj & 1;
        if (!ready(e, x.fp8)) return false;
        fence_after();
        const uint64_t k_desc = desc_sw128(smem + L::kRing + s * L::kSlot, 16, 1024);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            const uint64_t o = (uint64_t)((k >> 2) * (L::kRegion >> 4) + (k & 3) * 2);
            mma_ss(tmem + tmem_s(b), q_desc + o, k_desc + o, kIdQK, k > 0);
        }
        commit(cx.bar(L::kSFull + b));
        commit(cx.bar(L::kEmptyB + s));
        if (last) commit(cx.bar(L::kQEmpty));
        return true;
    };
    while (ok && w.segment()) {
        const int n = w.i_end - w.i;
        ok = cx.wait(L::kQFull, seg & 1) && (seg == 0 || cx.wait(L::kEpi, (seg - 1) & 1));
        if (!ok) break;
        Tile cur = w.tile();
        ok = qk(cur, j, n == 1);
        bool started[2] = {false, false};
        for (int x = 0; ok && x < n; ++x, ++j) {
            Tile next = cur;
            if (x + 1 < n) {
                next = w.tile();
                if (!(ok = qk(next, j + 1, x + 2 == n))) break;
            }
            const int e = 2 * j + 1, s = e % L::kSlots, b = j & 1;
            if (!(ok = cx.wait(L::kPFull + b, (j >> 1) & 1) && ready(e, cur.fp8 || cur.valid < kTok))) break;
            fence_after();
            const uint64_t v_desc = desc_sw128(smem + L::kRing + s * L::kSlot, L::kRegion, 1024);
#pragma unroll
            for (int k = 0; k < kTok / 16; ++k)
                mma_ts(tmem + tmem_o<D>(b), tmem + tmem_s(b) + 8 * k, v_desc + (uint64_t)(k * 128), kIdPV,
                       started[b] || k > 0);
            started[b] = true;
            commit(cx.bar(L::kEmptyB + s));
            if (x + 1 == n) commit(cx.bar(L::kOFull));
            cur = next;
        }
        ++seg;
    }
    // every product has completed before tensor memory is freed
    commit(cx.bar(L::kFin));
    for (int z = 0; z < kSpinLimit && !mbar_try_wait(cx.bar(L::kFin), 0); ++z) {
    }
}

// ------------------------------------------------------------------ FP8 -> bf16 (128 threads, one a token)
template <int D, int FMT>
__device__ void convert(const AttnArgs& a, const Ctx& cx, char* smem, int ct, Walk w) {
    using L = Smem<D>;
    const LayerDims& d = a.p.d;
    const float c2 = (float)(a.p.inv_sqrt_d * 1.4426950408889634);
    float* scales = reinterpret_cast<float*>(smem + L::kScale);
    int cvt = 0;   // uses of the read-before-write barrier (D = 64)
    uint32_t raw_ph = 0;             // parity of each slot's next phase
    int uses[2] = {0, 0};            // FP8 tiles through each scale buffer
    auto landed = [&](int s) {
        const bool r = cx.warp_wait(L::kRawB + s, (raw_ph >> s) & 1u);
        raw_ph ^= 1u << s;
        return r;
    };
    auto rewrite = [&](int s, bool zero) {
        char* slot = smem + L::kRing + s * L::kSlot;
        uint4 raw[D / 16];
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
            raw[c] = *reinterpret_cast<const uint4*>(slot + L::kRaw + (D == 128 ? sw128(ct, c) : sw64(ct, c)));
        if (zero) {
#pragma unroll
            for (int c = 0; c < D / 16; ++c) raw[c] = make_uint4(0u, 0u, 0u, 0u);
        }
        if constexpr (D == 64) {   // rows grow over other threads' codes (D = 128: over their own alone)
            mbar_arrive(cx.bar(L::kCvt));
            if (!cx.warp_wait(L::kCvt, cvt++ & 1)) return false;
        }
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
            uint4 lo, hi;
            fp8x4_to_bf16<FMT>(raw[c].x, lo.x, lo.y);
            fp8x4_to_bf16<FMT>(raw[c].y, lo.z, lo.w);
            fp8x4_to_bf16<FMT>(raw[c].z, hi.x, hi.y);
            fp8x4_to_bf16<FMT>(raw[c].w, hi.z, hi.w);
            char* reg = slot + (c >> 2) * L::kRegion;
            *reinterpret_cast<uint4*>(reg + sw128(ct, 2 * (c & 3))) = lo;
            *reinterpret_cast<uint4*>(reg + sw128(ct, 2 * (c & 3) + 1)) = hi;
        }
        fence_proxy_async();
        mbar_arrive(cx.bar(L::kConvB + s));
        return true;
    };
    auto load_scales = [&](const Tile& x, int row, float& sk, float& sv) {
        sk = sv = 0.f;   // zero past the segment end, where stale bits must not enter
        if (x.fp8 && ct < x.valid) {
            const size_t at = (size_t)row * d.cap_q + x.idx * kTok + ct;
            sk = __ldg(a.p.c.sk + at);
            sv = __ldg(a.p.c.sv + at);
        }
    };
    auto next = [&](Tile& x) {
        if (w.i == w.i_end && !w.segment()) return false;
        x = w.tile();
        return true;
    };
    Tile cur{}, ahead{};
    float sk, sv, sk1 = 0.f, sv1 = 0.f;
    if (!next(cur)) return;
    load_scales(cur, w.row, sk, sv);
    for (int j = 0;; ++j) {
        const bool more = next(ahead);   // the next tile's scales are loaded one tile early
        if (more) load_scales(ahead, w.row, sk1, sv1);
        const int b = j & 1, ks = (2 * j) % L::kSlots, vs = (2 * j + 1) % L::kSlots;
        if (cur.fp8) {
            if (uses[b] > 0 && !cx.warp_wait(L::kScFree + b, (uses[b] - 1) & 1)) return;   // their last readers
            ++uses[b];
            scales[(2 * b) * kTok + ct] = sk * c2;
            scales[(2 * b + 1) * kTok + ct] = sv;
            mbar_arrive(cx.bar(L::kScFull + b));
            if (!landed(ks) || !rewrite(ks, false)) return;
            if (!landed(vs) || !rewrite(vs, ct >= cur.valid)) return;
        } else if (cur.valid < kTok) {   // stale V rows past the end must not meet P = 0
            if (!landed(vs)) return;
            if (ct >= cur.valid) {
#pragma unroll
                for (int c = 0; c < D / 8; ++c)
                    *reinterpret_cast<uint4*>(smem + L::kRing + vs * L::kSlot + (c >> 3) * L::kRegion + ct * 128 +
                                              ((c & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async();
            mbar_arrive(cx.bar(L::kConvB + vs));
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

// One tile of this thread's row: S at column s of its lane becomes P.  TAIL: only the first
// `valid` columns are tokens.
template <int D, bool FP8, bool TAIL>
__device__ __forceinline__ void softmax_tile(uint32_t s, uint32_t o, bool first, int valid, const float* sk,
                                             const float* sv, float c2, Row& r) {
    float v[32];
    float mx = kNegInf;
#pragma unroll
    for (int c = 0; c < kTok / 32; ++c) {
        tmem_ld32(s + 32 * c, v);
        wait_ld(v);
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            float4 k = make_float4(1.f, 1.f, 1.f, 1.f);
            if (FP8) k = *reinterpret_cast<const float4*>(sk + 32 * c + i);
            const float kk[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                float x = FP8 ? v[i + u] * kk[u] : v[i + u];
                if (TAIL && 32 * c + i + u >= valid) x = kNegInf;
                mx = fmaxf(mx, x);
            }
        }
    }
    if (!FP8) mx *= c2;
    r.top = first ? mx : fmaxf(r.top, mx);
    if (first) {
        r.m = mx == kNegInf ? 0.f : mx;
        r.l = 0.f;
    } else {
        const bool move = mx > r.m + 8.f;
        if (__any_sync(kFull, move)) {   // O is idle: the product into S came after the last one into O
            const float f = move ? ex2(r.m - mx) : 1.f;
            r.l *= f;
            if (move) r.m = mx;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                tmem_ld32(o + 32 * c, v);
                wait_ld(v);
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] *= f;
                tmem_st32(o + 32 * c, v);
            }
        }
    }
    const float m = r.m;
    float l0 = 0.f, l1 = 0.f;
#pragma unroll
    for (int c = 0; c < kTok / 32; ++c) {
        tmem_ld32(s + 32 * c, v);
        wait_ld(v);
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            float4 k = make_float4(c2, c2, c2, c2), f = make_float4(1.f, 1.f, 1.f, 1.f);
            if (FP8) {
                k = *reinterpret_cast<const float4*>(sk + 32 * c + i);
                f = *reinterpret_cast<const float4*>(sv + 32 * c + i);
            }
            const float kk[4] = {k.x, k.y, k.z, k.w}, ff[4] = {f.x, f.y, f.z, f.w};
            float p[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                p[u] = ex2(fmaf(v[i + u], kk[u], -m));
                if (TAIL && 32 * c + i + u >= valid) p[u] = 0.f;
            }
            l0 += p[0] + p[2];
            l1 += p[1] + p[3];
            if (FP8) {
#pragma unroll
                for (int u = 0; u < 4; ++u) p[u] *= ff[u];
            }
            pk[i / 2] = pack_bf16(p[0], p[1]);
            pk[i / 2 + 1] = pack_bf16(p[2], p[3]);
        }
        tmem_st16(s + 16 * c, pk);   // over columns of S that have been read
    }
    r.l += l0 + l1;
    wait_st();
}

template <int D>
__device__ void softmax(const AttnArgs& a, const Ctx& cx, char* smem, uint32_t tmem, int b, Walk w, int cta) {
    using L = Smem<D>;
    const LayerDims& d = a.p.d;
    const int quad = (threadIdx.x >> 5) & 3, row = quad * 32 + (threadIdx.x & 31);
    const uint32_t lane = tmem + ((uint32_t)(quad * 32) << 16), s = lane + tmem_s(b), o = lane + tmem_o<D>(b);
    const float c2 = (float)(a.p.inv_sqrt_d * 1.4426950408889634);
    const float* sk = reinterpret_cast<const float*>(smem + L::kScale) + 2 * b * kTok;
    const float* sv = sk + kTok;
    int j = 0, seg = 0, scales = 0;
    while (w.segment()) {
        const int n = w.i_end - w.i, j0 = j;
        Row r{0.f, kNegInf, 0.f};
        bool first = true;
        for (int x = 0; x < n; ++x, ++j) {
            const Tile t = w.tile();
            if ((j & 1) != b) continue;
            if (t.fp8 && !cx.warp_wait(L::kScFull + b, scales++ & 1)) return;
            if (!cx.warp_wait(L::kSFull + b, (j >> 1) & 1)) return;
            fence_after();
            if (t.valid == kTok) {
                if (t.fp8) softmax_tile<D, true, false>(s, o, first, kTok, sk, sv, c2, r);
                else softmax_tile<D, false, false>(s, o, first, kTok, sk, sv, c2, r);
            } else {
                if (t.fp8) softmax_tile<D, true, true>(s, o, first, t.valid, sk, sv, c2, r);
                else softmax_tile<D, false, true>(s, o, first, t.valid, sk, sv, c2, r);
            }
            first = false;
            fence_before();
            mbar_arrive(cx.bar(L::kPFull + b));
            if (t.fp8) mbar_arrive(cx.bar(L::kScFree + b));
        }
        // the segment's partial: both warpgroups' O under one reference, half the columns each
        if (!cx.warp_wait(L::kOFull, seg & 1)) return;
        fence_after();
        tmem_st4(s, r.m, r.top, r.l, 0.f);   // S and P are idle: the state goes to the other warpgroup through them
        wait_st();
        fence_before();
        mbar_arrive(cx.bar(L::kXch));
        if (!cx.warp_wait(L::kXch, seg & 1)) return;
        fence_after();
        float y[4];
        tmem_ld4(lane + tmem_s(b ^ 1), y);
        wait_ld(y);
        const bool mine = n > 1 || (j0 & 1) == b, theirs = n > 1 || (j0 & 1) != b;   // who had a tile
        const float top = fmaxf(r.top, y[1]);   // a warpgroup without one has -inf
        // raw units for the join; what the rounding of the maximum moves goes into the weights
        const double c2d = a.p.inv_sqrt_d * 1.4426950408889634;
        const float M = top == kNegInf ? kNegInf : top / c2;
        const double at = top == kNegInf ? 0.0 : (double)M * c2d;
        const float w_mine = mine ? exp2f((float)((double)r.m - at)) : 0.f;
        const float w_theirs = theirs ? exp2f((float)((double)y[0] - at)) : 0.f;
        const float sum = (mine ? r.l * w_mine : 0.f) + (theirs ? y[2] * w_theirs : 0.f);
        const int slot = cta + w.unit0 + w.m;
        const int rows = min(a.per_tile, w.r.nb - w.m * a.per_tile) * d.G;
        const bool live = row < rows && slot < a.slots;
        if (live && b == 0) a.part_ml[(size_t)slot * kRows + row] = make_float2(M, sum);
        float* out = a.part_o + ((size_t)slot * kRows + row) * D + b * (D / 2);
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            float u[32], v[32];
            const uint32_t col = b * (D / 2) + 32 * c;
            if (mine) {
                tmem_ld32(o + col, u);
                wait_ld(u);
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) u[i] = mine ? u[i] * w_mine : 0.f;
            if (theirs) {
                tmem_ld32(lane + tmem_o<D>(b ^ 1) + col, v);
                wait_ld(v);
#pragma unroll
                for (int i = 0; i < 32; ++i) u[i] = fmaf(v[i], w_theirs, u[i]);
            }
            if (live) {
#pragma unroll
                for (int i = 0; i < 32; i += 4)
                    *reinterpret_cast<float4*>(out + 32 * c + i) = make_float4(u[i], u[i + 1], u[i + 2], u[i + 3]);
            }
        }
        fence_before();
        mbar_arrive(cx.bar(L::kEpi));
        ++seg;
    }
}

// Tiles and units before every row, for the join (one warp).
__device__ void write_starts(const AttnArgs& a) {
    const int lane = threadIdx.x & 31;
    long long t = 0, u = 0;
    for (int r0 = 0; r0 < a.p.d.R; r0 += 32) {
        long long x = 0, y = 0;
        if (r0 + lane < a.p.d.R) {
            const RowInfo r = row_info(a, r0 + lane);
            x = (long long)r.mt * (r.T16 + r.T8);
            y = r.mt;
        }
        long long sx = x, sy = y;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const long long px = __shfl_up_sync(kFull, sx, m), py = __shfl_up_sync(kFull, sy, m);
            if (lane >= m) {
                sx += px;
                sy += py;
            }
        }
        if (r0 + lane < a.p.d.R) a.starts[r0 + lane] = make_longlong2(t + sx - x, u + sy - y);
        t += __shfl_sync(kFull, sx, 31);
        u += __shfl_sync(kFull, sy, 31);
    }
    if (lane == 0) a.starts[a.p.d.R] = make_longlong2(t, u);
}

// This CTA's run: a block scan of the rows' tiles (threads own contiguous rows), then the
// thread whose rows hold the run's first tile hands over where that is.
template <int D>
__device__ __forceinline__ Sched schedule(const AttnArgs& a, char* smem) {
    using L = Smem<D>;
    Sched* out = reinterpret_cast<Sched*>(smem + L::kSched);
    longlong2* sums = reinterpret_cast<longlong2*>(smem + L::kSums);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, R = a.p.d.R;
    const int per = (R + kThreads - 1) / kThreads, r0 = min(R, tid * per), r1 = min(R, r0 + per);
    long long x = 0, y = 0;
    for (int r = r0; r < r1; ++r) {
        const RowInfo i = row_info(a, r);
        x += (long long)i.mt * (i.T16 + i.T8);
        y += i.mt;
    }
    long long sx = x, sy = y;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const long long px = __shfl_up_sync(kFull, sx, m), py = __shfl_up_sync(kFull, sy, m);
        if (lane >= m) {
            sx += px;
            sy += py;
        }
    }
    if (lane == 31) sums[warp] = make_longlong2(sx, sy);
    if (tid == 0) *out = Sched{0, 0, 0, 0, 0};
    __syncthreads();
    long long T = 0, tx = sx - x, ty = sy - y;
    for (int i = 0; i < kThreads / 32; ++i) {
        const longlong2 z = sums[i];
        T += z.x;
        if (i < warp) {
            tx += z.x;
            ty += z.y;
        }
    }
    const int P = (int)min((long long)gridDim.x, T);
    if ((int)blockIdx.x < P) {
        const long long t0 = run_begin(T, P, blockIdx.x), t1 = run_begin(T, P, blockIdx.x + 1);
        for (int r = r0; r < r1; ++r) {
            const RowInfo i = row_info(a, r);
            const long long n = (long long)i.mt * (i.T16 + i.T8);
            if (t0 >= tx && t0 < tx + n) *out = Sched{t0, t1, tx, r, (int)ty};
            tx += n;
            ty += i.mt;
        }
    }
    __syncthreads();
    return *out;
}

template <int D, int FMT>
__global__ void __launch_bounds__(kThreads, 1) prefix_attn_kernel(const __grid_constant__ AttnArgs a) {
    using L = Smem<D>;
    extern __shared__ __align__(1024) char smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_launch_dependents();
    if (tid == 0) {
        prefetch_map(&a.tm_q); prefetch_map(&a.tm_k16); prefetch_map(&a.tm_v16); prefetch_map(&a.tm_k8);
        prefetch_map(&a.tm_v8);
    }
    if (!a.p.early_start) pdl_wait();
    const uint32_t base = smem_u32(smem);
    if (base & 1023) {   // the swizzled tiles need it; the CTA's shared memory starts there
        if (tid == 0) atomicOr(a.p.c.status, ARKV_STATUS_TIMEOUT);
        pdl_wait();
        return;
    }
    int* misc = reinterpret_cast<int*>(smem + L::kMisc);
    Ctx cx{base + L::kBars, misc + 1, a.p.c.status};
    if (tid == 0) {
        for (int i = 0; i < L::kNumBars; ++i) {
            int n = 1;
            if ((i >= L::kConvB && i < L::kConvB + L::kSlots) || i == L::kPFull || i == L::kPFull + 1 || i == L::kScFull ||
                i == L::kScFull + 1 || i == L::kScFree || i == L::kScFree + 1 || i == L::kCvt)
                n = 128;
            if (i == L::kXch || i == L::kEpi) n = 256;
            mbar_init(cx.bar(i), n);
        }
        misc[1] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async();
    }
    const Sched sched = schedule<D>(a, smem);
    const bool busy = sched.t < sched.t_end;   // the same for the whole CTA
    if (busy && warp == 2) tmem_alloc(base + L::kMisc, kTmemCols);
    __syncthreads();
    if (blockIdx.x == 0 && warp == 3) {   // the workspace is the previous call's until it has finished
        pdl_wait();
        write_starts(a);
    }
    if (!busy) return;
    fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(misc);
    if (warp == 0) {
        if (lane == 0) produce<D>(a, cx, base, Walk(a, sched));
    } else if (warp == 1) {
        if (lane == 0) {
            pdl_wait();   // bounded waits start when the previous kernel has finished
            multiply<D>(a, cx, base, tmem, Walk(a, sched));
        }
    } else if (warp >= 12) {
        pdl_wait();
        convert<D, FMT>(a, cx, smem, tid - 384, Walk(a, sched));
    } else if (warp >= 4) {
        pdl_wait();
        softmax<D>(a, cx, smem, tmem, (warp - 4) >> 2, Walk(a, sched), blockIdx.x);
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
// One warp per (branch, query head): the partials of its row in CTA order and the own part,
// (M, L, o) joined in float32, o rounded to bf16.  The partials' loads of a batch are all in
// flight at once.
template <int D>
__global__ void __launch_bounds__(128) prefix_join_kernel(const __grid_constant__ AttnArgs a, int ctas) {
    constexpr int VEC = D / 32, kBatch = 8;
    const LayerDims& d = a.p.d;
    const int lane = threadIdx.x & 31;
    const long long item = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    pdl_launch_dependents();
    pdl_wait();
    if (item >= (long long)a.p.branches * d.hq) return;
    const int b = (int)(item / d.hq), h = (int)(item % d.hq), g = h / d.G, jq = h % d.G;
    int pre = 0, b0 = 0;
    bool has = true;
    if (a.p.branch_start) {   // the last prefix that starts at or before b
        int lo = 0, hi = d.batch;   // starts[lo] <= b < starts[hi], sentinels at both ends
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (a.p.branch_start[mid] <= b) lo = mid;
            else hi = mid;
        }
        pre = lo;
        const int s = a.p.branch_start[pre];
        has = s <= b && b < a.p.branch_start[pre + 1];
        b0 = max(s, 0);
    }
    const size_t mi = ((size_t)b * d.hkv + g) * 4 + jq;
    const size_t at = (size_t)item * D + VEC * lane;
    float M = kNegInf, L = 0.f, acc[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
    if (a.p.ml_own) {
        const float2 own = a.p.ml_own[mi];
        if (own.y != 0.f) {
            M = own.x;
            L = own.y;
#pragma unroll
            for (int e = 0; e < VEC; ++e) acc[e] = own.y * a.p.o_own[at + e];
        }
    }
    if (has) {
        const int row = pre * d.hkv + g;
        const long long T = a.starts[d.R].x;
        const longlong2 st = a.starts[row];
        const RowInfo r = row_info(a, row);
        const int m = (b - b0) / a.per_tile, tiles = r.T16 + r.T8;
        if (tiles > 0) {
            const long long t0 = st.x + (long long)m * tiles;
            const int P = (int)min((long long)ctas, T), c0 = run_of(T, P, t0), c1 = run_of(T, P, t0 + tiles - 1);
            const int unit = (int)st.y + m, rr = (b - b0 - m * a.per_tile) * d.G + jq;
            for (int c = c0; c <= c1; c += kBatch) {
                const int cnt = min(kBatch, c1 - c + 1);
                auto slot = [&](int q) { return min(c + q + unit, a.slots - 1); };
                float2 ml = make_float2(kNegInf, 0.f);
                if (lane < cnt) ml = __ldcg(a.part_ml + (size_t)slot(lane) * kRows + rr);
                float v[kBatch][VEC];
#pragma unroll
                for (int q = 0; q < kBatch; ++q) {
                    const float* src = a.part_o + ((size_t)slot(q) * kRows + rr) * D + VEC * lane;
#pragma unroll
                    for (int e = 0; e < VEC; e += 2) {
                        const float2 x = q < cnt ? __ldcg(reinterpret_cast<const float2*>(src + e)) : make_float2(0.f, 0.f);
                        v[q][e] = x.x;
                        v[q][e + 1] = x.y;
                    }
                }
                float mb = ml.y != 0.f ? ml.x : kNegInf;
#pragma unroll
                for (int k = 16; k >= 1; k >>= 1) mb = fmaxf(mb, __shfl_xor_sync(kFull, mb, k));
                if (mb > M) {
                    const float f = M == kNegInf ? 0.f : exp_scaled(M, mb, a.p.inv_sqrt_d);
                    L *= f;
#pragma unroll
                    for (int e = 0; e < VEC; ++e) acc[e] *= f;
                    M = mb;
                }
                // a partial without weight has l = 0; a NaN sum goes through
                const float wl = ml.y == 0.f ? 0.f : (ml.x == M ? 1.f : exp_scaled(ml.x, M, a.p.inv_sqrt_d));
                float part = ml.y * wl;
#pragma unroll
                for (int k = 16; k >= 1; k >>= 1) part += __shfl_xor_sync(kFull, part, k);
                L += part;
#pragma unroll
                for (int q = 0; q < kBatch; ++q) {
                    const float f = __shfl_sync(kFull, wl, q);
                    if (q < cnt && f != 0.f) {
#pragma unroll
                        for (int e = 0; e < VEC; ++e) acc[e] = fmaf(v[q][e], f, acc[e]);
                    }
                }
            }
        }
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    uint32_t out[VEC / 2];
#pragma unroll
    for (int e = 0; e < VEC; e += 2) out[e / 2] = pack_bf16(acc[e] * inv, acc[e + 1] * inv);
    if constexpr (VEC == 4) *reinterpret_cast<uint2*>(a.p.o + at) = make_uint2(out[0], out[1]);
    else *reinterpret_cast<uint32_t*>(a.p.o + at) = out[0];
    if (lane == 0 && a.p.ml) a.p.ml[mi] = make_float2(M, L);
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
    size_t part_o, part_ml, starts, total;
    int slots, per_tile;
};

// A segment's partial goes to slot (CTA + unit): along the list of tiles each next segment
// raises one of the two, so the slots differ, and there are at most CTAs + units of them.
PrefixWs ws_layout(const LayerDims& d, int branches) {
    PrefixWs w{};
    w.per_tile = kRows / d.G;
    const long long units = (long long)d.hkv * (d.batch + branches / w.per_tile);
    w.slots = (int)(kMaxCtas + units);
    auto al = [](size_t x) { return (x + 255) & ~(size_t)255; };
    size_t off = 0;
    w.starts = off;  off = al(off + sizeof(longlong2) * ((size_t)d.R + 1));
    w.part_ml = off; off = al(off + sizeof(float2) * kRows * (size_t)w.slots);
    w.part_o = off;  off = al(off + sizeof(float) * kRows * (size_t)d.D * w.slots);
    w.total = off;
    return w;
}

}  // namespace

size_t prefix_ws_bytes(const LayerDims& d, int branches) { return ws_layout(d, branches).total; }

cudaError_t launch_prefix_attn(const PrefixParams& p, void* ws, cudaStream_t s) {
    const LayerDims& d = p.d;
    const PrefixWs w = ws_layout(d, p.branches);
    AttnArgs a{};
    a.p = p;
    a.slots = w.slots;
    a.per_tile = w.per_tile;
    a.starts = reinterpret_cast<longlong2*>((char*)ws + w.starts);
    a.part_ml = reinterpret_cast<float2*>((char*)ws + w.part_ml);
    a.part_o = reinterpret_cast<float*>((char*)ws + w.part_o);
    const long long r16 = (long long)d.R * d.cap_o, r8 = (long long)d.R * d.cap_q;
    if (!make_q_map(&a.tm_q, p.q, d, p.branches, w.per_tile) || !make_map(&a.tm_k16, p.c.k16, false, d.D, r16) ||
        !make_map(&a.tm_v16, p.c.v16, false, d.D, r16) || !make_map(&a.tm_k8, p.c.k8, true, d.D, r8) ||
        !make_map(&a.tm_v8, p.c.v8, true, d.D, r8))
        return cudaErrorInvalidValue;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    // one CTA an SM, at most one a tile of the fullest prefixes
    const long long most = (w.slots - kMaxCtas) * (((long long)d.cap_o + kTok - 1) / kTok + (d.cap_q + kTok - 1) / kTok);
    long long ctas = sms < kMaxCtas ? sms : kMaxCtas;
    if (ctas > most) ctas = most;
    static unsigned char done[4][64];
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t lc{};
    lc.stream = s;
    lc.attrs = attr;
    lc.numAttrs = 1;
    auto go = [&](auto kernel, auto join, int which, int bytes) {
        cudaError_t err = allow_max_dyn_smem(kernel, done[which]);
        if (err != cudaSuccess) return err;
        lc.gridDim = dim3((unsigned)ctas);
        lc.blockDim = dim3(kThreads);
        lc.dynamicSmemBytes = (size_t)bytes;
        if ((err = cudaLaunchKernelEx(&lc, kernel, a)) != cudaSuccess) return err;
        lc.gridDim = dim3((unsigned)(((long long)p.branches * d.hq + 3) / 4));
        lc.blockDim = dim3(128);
        lc.dynamicSmemBytes = 0;
        return cudaLaunchKernelEx(&lc, join, a, (int)ctas);
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
