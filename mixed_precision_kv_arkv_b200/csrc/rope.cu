// arkv_qk_norm_rope: per-head RMS norm of queries and keys, rotation by position and the
// head-major layouts of the decode and prefill calls, from the rows of a fused projection.
//
// With inv = 1 / sqrt(mean(x^2) + eps) and partner p(a) = b, p(b) = a of every rotated pair,
//   y_i = inv (x_i w_i cos f_i + x_p(i) w_p(i) (-+ sin f_i)),
// so a thread keeps two factors for each of its 8 dimensions (cos and sin with the weights
// folded in) and reuses them for all the heads of its token that it takes.
//
// A group of D / 8 threads takes a head, 16 bytes a thread; a block's groups are dealt to its
// tokens, and each group takes every n-th head of its token, four loads in flight.  The
// arithmetic is on packed pairs.  Sines and cosines are computed
// once a token and pair, into shared memory: the angle in turns as a 64-bit fraction,
// position * round(freq / 2 pi * 2^64) modulo 2^64, is exact for any position.
//
// Bound: HBM, every projection row read and every output written once.  8192 tokens of 48
// heads of 128: 201.9 MB, floor 31.2 us at 6461.5 GB/s; 42.5 us measured (4.8 TB/s; the
// loads' and shuffles' latencies at 32 warps an SM and half of the issue slots are what is left).
#include "arkv_internal.cuh"
#include "tc.cuh"

namespace arkv {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;   // heads of a group in flight
constexpr int kMaxTokens = 16;

enum { kHalf = 0, kInterleaved = 1, kOdd = 2 };   // pairs (i, i + rot / 2), whole vectors apart; (2i, 2i + 1); any rot

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Position (an integer) times freq radians, sine and cosine: float32 of the exact angle.
__device__ __forceinline__ float2 turn(int64_t pos, double freq) {
    const double t = freq * 0.15915494309189533577;   // turns per position
    const uint64_t frac = (uint64_t)((t - floor(t)) * 18446744073709551616.0);
    const int64_t at = (int64_t)((uint64_t)pos * frac);   // of a turn, in [-1/2, 1/2)
    float s, c;
    sincospif((float)(int)(at >> 32) * 4.656612873077393e-10f, &s, &c);   // 2^-31: half turns
    return make_float2(c, s);
}

template <int D, int MODE>
__global__ void __launch_bounds__(kThreads, 4) qk_norm_rope_kernel(const __grid_constant__ RopeParams p, int tokens) {
    constexpr int kGroup = D / 8, kGroups = kThreads / kGroup;
    __shared__ __align__(16) float2 sm_turn[kMaxTokens][D / 2];
    const LayerDims& d = p.d;
    const int tid = threadIdx.x, gl = tid % kGroup, group = tid / kGroup;
    const int half = p.rot / 2, total = d.batch * p.n_tok;
    const int row0 = blockIdx.x * tokens;
    tc::pdl_wait();
    tc::pdl_launch_dependents();
    for (int i = tid; i < tokens * half; i += kThreads) {
        const int t = i / half, j = i - t * half, row = row0 + t;
        if ((unsigned)row >= (unsigned)total) break;
        const int b = row / p.n_tok;
        sm_turn[t][j] = turn((p.pos0 ? (int64_t)p.pos0[b] : 0) + p.step + (row - b * p.n_tok), p.freq[j]);
    }
    __syncthreads();
    const int per = kGroups / tokens;               // groups of a token in this block
    const int lt = group / per, row = row0 + lt;
    const int stride = per * gridDim.y, first = (group - lt * per) + per * blockIdx.y;
    const int b = row / p.n_tok, t = row - b * p.n_tok;   // (past the end only when not `in`)
    const bool in = lt < tokens && (unsigned)row < (unsigned)total;
    const int len = in ? (p.length ? min(max(p.length[b], 0), p.n_tok) : p.n_tok) : 0;
    if (!in || t >= len) return;           // whole groups; the shuffles stay within a group
    const unsigned mask = (kGroup == 32 ? 0xffffffffu : ((1u << kGroup) - 1u) << ((tid & 31) / kGroup * kGroup));
    const uint16_t* x_row = p.qkv + (int64_t)row * p.qkv_stride;
    const int heads = d.hq + d.hkv, dim0 = 8 * gl;
    int partner = gl;                               // the thread that holds the partners of these dimensions
    if (MODE == kHalf && dim0 < p.rot) partner = dim0 < half ? gl + half / 8 : gl - half / 8;

    // factors of this thread's dimensions for queries, then keys: pairs of dimensions
    float2 fc[4], fs[4];
    auto partner_dim = [&](int i) {
        if (i >= p.rot) return i;
        if (MODE == kInterleaved) return i ^ 1;
        return i < half ? i + half : i - half;
    };
    auto factors = [&](const uint16_t* w) {
        float c[8], v[8], wo[8], wp[8];
        const bool rotated = dim0 < p.rot;
        if (MODE == kHalf) {   // whole vectors: pairs j0 .. j0 + 7, partners dim0 +- half ..
            const int j0 = dim0 < half ? dim0 : dim0 - half;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4 cs = rotated ? *reinterpret_cast<const float4*>(&sm_turn[lt][j0 + 2 * e])
                                          : make_float4(1.f, 0.f, 1.f, 0.f);
                c[2 * e] = cs.x; c[2 * e + 1] = cs.z;
                v[2 * e] = dim0 < half ? -cs.y : cs.y; v[2 * e + 1] = dim0 < half ? -cs.w : cs.w;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = dim0 + e;
                const bool in = i < p.rot;
                const float2 cs = in ? sm_turn[lt][MODE == kInterleaved ? i >> 1 : (i < half ? i : i - half)] : make_float2(1.f, 0.f);
                c[e] = cs.x;
                v[e] = (MODE == kInterleaved ? !(e & 1) : i < half) ? -cs.y : cs.y;
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) wo[e] = wp[e] = 1.f;
        if (w) {
            if (MODE == kHalf && (reinterpret_cast<uintptr_t>(w) & 15) == 0) {
                const uint4 a = *reinterpret_cast<const uint4*>(w + dim0);
                const uint4 q = *reinterpret_cast<const uint4*>(w + (rotated ? partner_dim(dim0) : dim0));
                const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, qw[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    wo[2 * e] = bf16_lo(aw[e]); wo[2 * e + 1] = bf16_hi(aw[e]);
                    if (rotated) {   // (else the factor of no partner has to be zero, whatever the weight)
                        wp[2 * e] = bf16_lo(qw[e]);
                        wp[2 * e + 1] = bf16_hi(qw[e]);
                    }
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    wo[e] = bf16_to_f32(w[dim0 + e]);
                    if (dim0 + e < p.rot) wp[e] = bf16_to_f32(w[partner_dim(dim0 + e)]);
                }
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            fc[e] = make_float2(c[2 * e] * wo[2 * e], c[2 * e + 1] * wo[2 * e + 1]);
            fs[e] = make_float2(v[2 * e] * wp[2 * e], v[2 * e + 1] * wp[2 * e + 1]);
        }
    };
    // Heads first, first + stride, .. below hi: head h goes to out + (h - h_base) * step, and to
    // obs + (h - h_base) * obs_step (a query of the last positions).
    auto run = [&](int h, int hi, const uint16_t* w, uint16_t* out, int64_t step, uint16_t* obs, int64_t obs_step) {
        const uint4* src = reinterpret_cast<const uint4*>(x_row + (int64_t)h * D + dim0);
        const int src_step = stride * (D / 8);
        auto one = [&](const uint4& raw, int hh, int u) {
            const uint32_t r[4] = {raw.x, raw.y, raw.z, raw.w};
            float2 x[4], y[4];
            float2 ss = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = make_float2(bf16_lo(r[e]), bf16_hi(r[e]));
            float inv = 1.f;
            if (w) {
#pragma unroll
                for (int e = 0; e < 4; ++e) ss = tc::fma2(x[e], x[e], ss);
                float t = ss.x + ss.y;
#pragma unroll
                for (int m = kGroup / 2; m >= 1; m >>= 1) t += __shfl_xor_sync(mask, t, m);
                inv = rsqrtf(fmaf(t, 1.f / D, p.eps));
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float2 z;
                if (MODE == kInterleaved) {
                    z = dim0 + 2 * e < p.rot ? make_float2(x[e].y, x[e].x) : make_float2(0.f, 0.f);
                } else if (MODE == kHalf) {
                    uint32_t o = __shfl_sync(mask, r[e], partner, kGroup);
                    if (dim0 >= p.rot) o = 0u;   // not rotated: rot is a multiple of 16 here
                    z = make_float2(bf16_lo(o), bf16_hi(o));
                } else {
                    const int i = dim0 + 2 * e;
                    const uint16_t* from = x_row + (int64_t)hh * D;
                    z.x = i < p.rot ? bf16_to_f32(from[partner_dim(i)]) : 0.f;
                    z.y = i + 1 < p.rot ? bf16_to_f32(from[partner_dim(i + 1)]) : 0.f;
                }
                y[e] = tc::fma2(x[e], fc[e], tc::mul2(z, fs[e]));
                if (w) y[e] = tc::mul2(y[e], make_float2(inv, inv));
            }
            const uint4 v = make_uint4(pack2(y[0].x, y[0].y), pack2(y[1].x, y[1].y), pack2(y[2].x, y[2].y), pack2(y[3].x, y[3].y));
            if (out) *reinterpret_cast<uint4*>(out + u * step) = v;
            if (obs) *reinterpret_cast<uint4*>(obs + u * obs_step) = v;
        };
        for (; h + (kUnroll - 1) * stride < hi; h += kUnroll * stride) {
            uint4 raw[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) raw[u] = __ldcs(src + u * src_step);
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) one(raw[u], h + u * stride, u);
            src += kUnroll * src_step;
            if (out) out += kUnroll * step;
            if (obs) obs += kUnroll * obs_step;
        }
        for (; h < hi; h += stride) {
            one(__ldcs(src), h, 0);
            src += src_step;
            if (out) out += step;
            if (obs) obs += obs_step;
        }
    };
    auto begin = [&](int from) {   // this group's first head at or after `from`
        const int k = from <= first ? 0 : (from - first + stride - 1) / stride;
        return first + k * stride;
    };
    const int64_t head_step = (int64_t)p.n_stride * D, at = (int64_t)t * D + dim0;
    const int o = t - (len - d.n_obs);
    if (p.q || (p.q_obs && o >= 0)) {
        const int h = begin(0);
        factors(p.q_weight);
        run(h, d.hq, p.q_weight, p.q ? p.q + ((int64_t)b * d.hq + h) * head_step + at : nullptr, stride * head_step,
            p.q_obs && o >= 0 ? p.q_obs + (((int64_t)b * d.hq + h) * d.n_obs + o) * D + dim0 : nullptr,
            (int64_t)stride * d.n_obs * D);
    }
    {
        const int h = begin(d.hq);
        factors(p.k_weight);
        run(h, heads, p.k_weight, p.k + ((int64_t)b * d.hkv + h - d.hq) * head_step + at, stride * head_step, nullptr, 0);
    }
    int h = begin(heads);   // values: a copy
    const uint4* src = reinterpret_cast<const uint4*>(x_row + (int64_t)h * D + dim0);
    uint16_t* out = p.v + ((int64_t)b * d.hkv + h - heads) * head_step + at;
    for (; h < heads + d.hkv; h += kUnroll * stride) {
        uint4 raw[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (h + u * stride < heads + d.hkv) raw[u] = __ldcs(src + u * stride * (D / 8));
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (h + u * stride < heads + d.hkv) *reinterpret_cast<uint4*>(out + u * stride * head_step) = raw[u];
        src += kUnroll * stride * (D / 8);
        out += kUnroll * stride * head_step;
    }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeParams& p, cudaStream_t s) {
    const LayerDims& d = p.d;
    const long long total = (long long)d.batch * p.n_tok;
    const int groups = kThreads / (d.D / 8);
    // (148: a B200's SMs.)  A group's start (its factors) is shared by all the heads it takes, so a block takes as many
    // tokens as leave a group 48 heads, or two blocks an SM (8192 tokens of 48 heads: 2 tokens a
    // block 67 us, 4 54, 8 45, 16 44; 6964 of 12 heads of 64: 4 tokens 15, 16 10.8).  A call of
    // few tokens gives each a block, or several (at most a head a group), up to two an SM.
    const int heads = d.hq + 2 * d.hkv;
    int tokens = 1;
    while (tokens < kMaxTokens && heads * tokens < groups * 48 && total >= 2ll * 148 * tokens) tokens *= 2;
    // Calls of one wave (four blocks an SM) give every block the same number of tokens instead, so
    // that no SM has a block more than another, if that leaves a group 7 heads or more (48 heads of
    // 128: 4096 tokens 30.4 -> 23.1 us, 1500 tokens 15.7 -> 14.6, but 800 tokens 9.7 -> 10.1).
    // That ends at 16 tokens a block, 9472 tokens; the waves of longer calls are uneven (9472 tokens
    // 45.7 us, 9500 61.5, 12000 68.2, 16384 81.4, 32768 154.4 with a floor of 124.6).
    const long long wave = 4 * 148, even = (total + wave - 1) / wave;
    if (even <= kMaxTokens && even * heads >= 7 * groups) tokens = (int)even;
    const int per = groups / tokens;
    long long split = 1;
    while (tokens == 1 && total * split < 2 * 148 && split * per < heads) ++split;
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3((unsigned)((total + tokens - 1) / tokens), (unsigned)split);
    lc.blockDim = dim3(kThreads);
    lc.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    auto go = [&](auto kernel) { return cudaLaunchKernelEx(&lc, kernel, p, tokens); };
    // kHalf shuffles whole vectors of partners; kOdd, for pairs (i, i + rot / 2) that straddle vectors, loads
    // each partner again (8192 tokens of 48 heads of 128: 42.4 us with rot 128, 42.1 with 112, 67.0
    // with 116, interleaved 38.1).
    const int mode = p.interleaved ? kInterleaved : (p.rot / 2) % 8 == 0 ? kHalf : kOdd;
    cudaError_t e;
    if (d.D == 128)
        e = mode == kHalf ? go(qk_norm_rope_kernel<128, kHalf>)
                          : mode == kInterleaved ? go(qk_norm_rope_kernel<128, kInterleaved>) : go(qk_norm_rope_kernel<128, kOdd>);
    else
        e = mode == kHalf ? go(qk_norm_rope_kernel<64, kHalf>)
                          : mode == kInterleaved ? go(qk_norm_rope_kernel<64, kInterleaved>) : go(qk_norm_rope_kernel<64, kOdd>);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace arkv
