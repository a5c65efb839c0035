// arkv_qk_norm_rope: per-head RMS norm of queries and keys, rotation by position and the
// head-major layouts of the decode and prefill calls, from the rows of a fused projection.
//
// With inv = 1 / sqrt(mean(x^2) + eps) and partner p(a) = b, p(b) = a of every rotated pair,
//   y_i = inv (x_i w_i cos f_i + x_p(i) w_p(i) (-+ sin f_i)),
// so a thread keeps two factors for each of its 8 dimensions (cos and sin with the weights
// folded in) and reuses them for all the heads of its token that it takes.
//
// A group of D / 8 threads takes a head, 16 bytes a thread; a block's groups are dealt to 4
// tokens (1 when there are few, so that a decode step still fills the GPU), and each group
// takes every n-th head of its token, four loads in flight.  Sines and cosines are computed
// once a token and pair, into shared memory: the angle in turns as a 64-bit fraction,
// position * round(freq / 2 pi * 2^64) modulo 2^64, is exact for any position.
//
// Bound: HBM, every projection row read and every output written once.  8192 tokens of 48
// heads of 128: 201.9 MB, floor 31.2 us at 6461.5 GB/s; MEASURED_LINE
#include "arkv_internal.cuh"
#include "tc.cuh"

namespace arkv {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;   // heads of a group in flight

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
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const __grid_constant__ RopeParams p, int tokens) {
    constexpr int kGroup = D / 8, kGroups = kThreads / kGroup;
    __shared__ float2 sm_turn[4][D / 2];
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
    const bool in = (unsigned)row < (unsigned)total;
    const int len = in ? (p.length ? min(max(p.length[b], 0), p.n_tok) : p.n_tok) : 0;
    if (!in || t >= len) return;           // whole groups; the shuffles stay within a group
    const unsigned mask = (kGroup == 32 ? 0xffffffffu : ((1u << kGroup) - 1u) << ((tid & 31) / kGroup * kGroup));
    const uint16_t* x_row = p.qkv + (int64_t)row * p.qkv_stride;
    const int heads = d.hq + d.hkv, dim0 = 8 * gl;
    int partner = gl;                               // the thread that holds the partners of these dimensions
    if (MODE == kHalf && dim0 < p.rot) partner = dim0 < half ? gl + half / 8 : gl - half / 8;

    // factors of this thread's dimensions for queries (kind 0), then keys (1)
    float fc[8], fs[8];
    auto partner_dim = [&](int i) {
        if (i >= p.rot) return i;
        if (MODE == kInterleaved) return i ^ 1;
        return i < half ? i + half : i - half;
    };
    auto factors = [&](const uint16_t* w) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = dim0 + e;
            float c = 1.f, s = 0.f;
            if (i < p.rot) {
                const int j = MODE == kInterleaved ? i >> 1 : (i < half ? i : i - half);
                const float2 cs = sm_turn[lt][j];
                const bool a = MODE == kInterleaved ? !(e & 1) : i < half;
                c = cs.x;
                s = a ? -cs.y : cs.y;
            }
            fc[e] = w ? c * bf16_to_f32(w[i]) : c;
            fs[e] = w ? s * bf16_to_f32(w[partner_dim(i)]) : s;
        }
    };
    auto head_out = [&](int h, const uint4& y) {
        const int64_t at = ((int64_t)t) * D + dim0;
        if (h < d.hq) {
            if (p.q) *reinterpret_cast<uint4*>(p.q + ((int64_t)b * d.hq + h) * p.n_stride * D + at) = y;
            const int o = t - (len - d.n_obs);
            if (p.q_obs && o >= 0)
                *reinterpret_cast<uint4*>(p.q_obs + (((int64_t)b * d.hq + h) * d.n_obs + o) * D + dim0) = y;
        } else {
            const int kv = h - d.hq, g = kv < d.hkv ? kv : kv - d.hkv;
            *reinterpret_cast<uint4*>((kv < d.hkv ? p.k : p.v) + ((int64_t)b * d.hkv + g) * p.n_stride * D + at) = y;
        }
    };
    // heads [lo, hi) of one kind, kUnroll at a time
    auto run = [&](int lo, int hi, bool norm) {
        for (int h0 = lo; h0 < hi; h0 += kUnroll * stride) {
            uint4 raw[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int h = h0 + u * stride;
                raw[u] = h < hi ? __ldcs(reinterpret_cast<const uint4*>(x_row + (int64_t)h * D + dim0)) : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int h = h0 + u * stride;
                if (h >= hi) break;
                const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
                float x[8], y[8];
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[2 * e] = bf16_lo(w[e]);
                    x[2 * e + 1] = bf16_hi(w[e]);
                    ss = fmaf(x[2 * e], x[2 * e], fmaf(x[2 * e + 1], x[2 * e + 1], ss));
                }
                float inv = 1.f;
                if (norm) {
#pragma unroll
                    for (int m = kGroup / 2; m >= 1; m >>= 1) ss += __shfl_xor_sync(mask, ss, m);
                    inv = rsqrtf(ss * (1.f / D) + p.eps);
                }
                if (MODE == kInterleaved) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        y[e] = inv * fmaf(x[e], fc[e], dim0 + e < p.rot ? x[e ^ 1] * fs[e] : 0.f);
                } else {
                    float z[8];
                    if (MODE == kHalf) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t o = __shfl_sync(mask, w[e], partner, kGroup);
                            if (dim0 >= p.rot) o = 0u;   // not rotated: rot is a multiple of 16 here
                            z[2 * e] = bf16_lo(o);
                            z[2 * e + 1] = bf16_hi(o);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            z[e] = dim0 + e < p.rot ? bf16_to_f32(x_row[(int64_t)h * D + partner_dim(dim0 + e)]) : 0.f;
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = inv * fmaf(x[e], fc[e], z[e] * fs[e]);
                }
                head_out(h, make_uint4(pack2(y[0], y[1]), pack2(y[2], y[3]), pack2(y[4], y[5]), pack2(y[6], y[7])));
            }
        }
    };
    auto begin = [&](int from) {   // this group's first head at or after `from`
        const int k = from <= first ? 0 : (from - first + stride - 1) / stride;
        return first + k * stride;
    };
    if (p.q || (p.q_obs && t >= len - d.n_obs)) {
        factors(p.q_weight);
        run(begin(0), d.hq, p.q_weight != nullptr);
    }
    factors(p.k_weight);
    run(begin(d.hq), heads, p.k_weight != nullptr);
    for (int h0 = begin(heads); h0 < heads + d.hkv; h0 += kUnroll * stride) {   // values: a copy
        uint4 raw[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (h0 + u * stride < heads + d.hkv)
                raw[u] = __ldcs(reinterpret_cast<const uint4*>(x_row + (int64_t)(h0 + u * stride) * D + dim0));
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (h0 + u * stride < heads + d.hkv) head_out(h0 + u * stride, raw[u]);
    }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeParams& p, cudaStream_t s) {
    const LayerDims& d = p.d;
    const long long total = (long long)d.batch * p.n_tok;
    const int groups = kThreads / (d.D / 8);
    // 4 tokens a block share the block's start; with fewer than about four blocks an SM that
    // way, a token gets the whole block, or several (a head a group and no more).
    // ROPE_SPLIT_NOTE
    const int tokens = total >= 4 * 4 * 148 ? 4 : 1;
    const int per = groups / tokens, heads = d.hq + 2 * d.hkv;
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
