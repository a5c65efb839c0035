// arkv_prefix_attn: decode attention of many branches to the prefixes they share,
// joined with each branch's own part.
//
// One CTA per (branch, query head): its warps take the live slots of the prefix row
// round robin, each with an online softmax in float32; the warps and the branch's own
// (o, M, L) are joined in shared memory.
#include "arkv_internal.cuh"

namespace arkv {

namespace {

constexpr int kWarps = 8;
constexpr float kNegInf = -INFINITY;

__device__ __forceinline__ float fp8_value(uint8_t c, int fmt) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(c, fmt == ARKV_FMT_E5M2 ? __NV_E5M2 : __NV_E4M3);
    return __half2float(__half(h));
}

template <int D>
__global__ void __launch_bounds__(32 * kWarps) prefix_attn_kernel(const PrefixParams p) {
    constexpr int VEC = D / 32;
    __shared__ float sm_o[kWarps][D], sm_m[kWarps], sm_l[kWarps];
    const LayerDims& d = p.d;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = blockIdx.x, h = blockIdx.y, g = h / d.G;
    int pre = -1;
    if (!p.branch_start) pre = 0;
    else
        for (int i = 0; i < d.batch; ++i)
            if (b >= p.branch_start[i] && b < p.branch_start[i + 1]) pre = i;
    const int row = max(pre, 0) * d.hkv + g;
    const int n16 = pre < 0 ? 0 : min(max(p.c.n_bf16[row], 0), d.cap_o);
    const int n8 = pre < 0 ? 0 : min(max(p.c.n_fp8[row], 0), d.cap_q);
    const size_t at = ((size_t)b * d.hq + h) * D;
    float q[VEC], o[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        q[e] = bf16_to_f32(p.q[at + VEC * lane + e]);
        o[e] = 0.f;
    }
    float m = kNegInf, l = 0.f;
    for (int i = warp; i < n16 + n8; i += kWarps) {
        float k[VEC], v[VEC], sk = 1.f, sv = 1.f;
        if (i < n16) {
            const size_t s = ((size_t)row * d.cap_o + i) * D + VEC * lane;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                k[e] = bf16_to_f32(p.c.k16[s + e]);
                v[e] = bf16_to_f32(p.c.v16[s + e]);
            }
        } else {
            const size_t slot = (size_t)row * d.cap_q + (i - n16), s = slot * D + VEC * lane;
            sk = p.c.sk[slot];
            sv = p.c.sv[slot];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                k[e] = fp8_value(p.c.k8[s + e], d.fmt);
                v[e] = fp8_value(p.c.v8[s + e], d.fmt);
            }
        }
        float raw = 0.f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) raw = fmaf(q[e], k[e], raw);
#pragma unroll
        for (int x = 16; x >= 1; x >>= 1) raw += __shfl_xor_sync(0xffffffffu, raw, x);
        raw *= sk;
        if (raw > m) {
            const float f = m == kNegInf ? 0.f : exp_scaled(m, raw, p.inv_sqrt_d);
            l *= f;
#pragma unroll
            for (int e = 0; e < VEC; ++e) o[e] *= f;
            m = raw;
        }
        const float w = raw == kNegInf ? 0.f : exp_scaled(raw, m, p.inv_sqrt_d);   // a NaN goes through
        l += w;
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = fmaf(w * sv, v[e], o[e]);
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) sm_o[warp][VEC * lane + e] = o[e];
    if (lane == 0) {
        sm_m[warp] = m;
        sm_l[warp] = l;
    }
    __syncthreads();
    if (warp != 0) return;
    const size_t mi = ((size_t)b * d.hkv + g) * 4 + h % d.G;
    float M = kNegInf, L = 0.f, acc[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
    const float2 mo = p.ml_own ? p.ml_own[mi] : make_float2(kNegInf, 0.f);
    if (mo.y != 0.f) M = mo.x;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_l[w] != 0.f ? sm_m[w] : kNegInf);
    if (mo.y != 0.f) {
        L = mo.y * exp_scaled(mo.x, M, p.inv_sqrt_d);
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] = L * p.o_own[at + VEC * lane + e];
    }
    for (int w = 0; w < kWarps; ++w) {
        if (sm_l[w] == 0.f) continue;
        const float f = exp_scaled(sm_m[w], M, p.inv_sqrt_d);
        L = fmaf(sm_l[w], f, L);
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] = fmaf(sm_o[w][VEC * lane + e], f, acc[e]);
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        const __nv_bfloat16 x = __float2bfloat16_rn(acc[e] * inv);
        p.o[at + VEC * lane + e] = *reinterpret_cast<const uint16_t*>(&x);
    }
    if (lane == 0 && p.ml) p.ml[mi] = make_float2(M, L);
}

}  // namespace

size_t prefix_ws_bytes(const LayerDims&, int) { return 256; }

cudaError_t launch_prefix_attn(const PrefixParams& p, cudaStream_t s) {
    const dim3 grid((unsigned)p.branches, (unsigned)p.d.hq);
    if (p.d.hq > 65535) return cudaErrorInvalidValue;
    if (p.d.D == 128) prefix_attn_kernel<128><<<grid, 32 * kWarps, 0, s>>>(p);
    else prefix_attn_kernel<64><<<grid, 32 * kWarps, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace arkv
