// arkv_qk_norm_rope: per-head RMS norm of queries and keys, rotation by position and
// the head-major layouts of the decode and prefill calls, from the rows of a fused
// projection.
//
// y = x / sqrt(mean(x^2) + eps) * w, then (y_a, y_b) turned by position * freq.  One
// warp per (token, head), the head's values in shared memory so that any pairing of
// dimensions can be read back.
#include "arkv_internal.cuh"

namespace arkv {

namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ uint16_t f32_to_bf16(float x) {
    const __nv_bfloat16 h = __float2bfloat16_rn(x);
    return *reinterpret_cast<const uint16_t*>(&h);
}

__global__ void __launch_bounds__(32 * kWarps) qk_norm_rope_kernel(const RopeParams p) {
    __shared__ float sm[kWarps][128];
    const LayerDims& d = p.d;
    const int D = d.D, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int heads = d.hq + 2 * d.hkv;
    const int64_t item = (int64_t)blockIdx.x * kWarps + warp;
    if (item >= (int64_t)d.batch * p.n_tok * heads) return;
    const int head = (int)(item % heads);
    const int64_t row = item / heads;
    const int b = (int)(row / p.n_tok), t = (int)(row % p.n_tok);
    const int len = p.length ? min(max(p.length[b], 0), p.n_tok) : p.n_tok;
    if (t >= len) return;
    const uint16_t* x = p.qkv + row * p.qkv_stride + (int64_t)head * D;
    const bool is_q = head < d.hq, is_v = head >= d.hq + d.hkv;
    uint16_t* out = nullptr;
    uint16_t* obs = nullptr;
    if (is_q) {
        if (p.q) out = p.q + (((int64_t)b * d.hq + head) * p.n_stride + t) * D;
        const int i = t - (len - d.n_obs);
        if (p.q_obs && i >= 0) obs = p.q_obs + (((int64_t)b * d.hq + head) * d.n_obs + i) * D;
    } else {
        uint16_t* base = is_v ? p.v : p.k;
        out = base + (((int64_t)b * d.hkv + (head - d.hq) % d.hkv) * p.n_stride + t) * D;
    }
    if (is_v) {
        for (int i = lane; i < D; i += 32) out[i] = x[i];
        return;
    }
    const uint16_t* w = is_q ? p.q_weight : p.k_weight;
    float ss = 0.f;
    for (int i = lane; i < D; i += 32) {
        const float v = bf16_to_f32(x[i]);
        sm[warp][i] = v;
        ss = fmaf(v, v, ss);
    }
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
    if (w) {
        const float inv = 1.f / sqrtf(ss / (float)D + p.eps);
        for (int i = lane; i < D; i += 32) sm[warp][i] = sm[warp][i] * inv * bf16_to_f32(w[i]);
    }
    __syncwarp();
    const double pos = (double)((p.pos0 ? (int64_t)p.pos0[b] : 0) + p.step + t);
    const int half = p.rot / 2;
    for (int i = lane; i < D; i += 32) {
        float y = sm[warp][i];
        if (i < p.rot) {
            const int j = p.interleaved ? i >> 1 : (i < half ? i : i - half);
            const bool first = p.interleaved ? !(i & 1) : i < half;
            const float other = sm[warp][p.interleaved ? i ^ 1 : (first ? i + half : i - half)];
            double s, c;
            sincos(pos * p.freq[j], &s, &c);
            y = first ? y * (float)c - other * (float)s : other * (float)s + y * (float)c;
        }
        const uint16_t o = f32_to_bf16(y);
        if (out) out[i] = o;
        if (obs) obs[i] = o;
    }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeParams& p, cudaStream_t s) {
    const int64_t items = (int64_t)p.d.batch * p.n_tok * (p.d.hq + 2 * p.d.hkv);
    const int64_t blocks = (items + kWarps - 1) / kWarps;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    qk_norm_rope_kernel<<<(unsigned)blocks, 32 * kWarps, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace arkv
