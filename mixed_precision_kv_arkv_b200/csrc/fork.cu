// arkv_cache_fork: copies, forks and frees the sequences of a packed cache (live
// slots, counts and score state), slot by slot in place.
#include "arkv_internal.cuh"

namespace arkv {

namespace {

// What becomes of destination sequence b: its source, or kSkip (kept, or refused),
// or kFree.
constexpr int kFree = ARKV_SEQ_FREE, kSkip = ARKV_SEQ_KEEP;

__device__ __forceinline__ bool keeps_state(const ForkParams& p, int s) {
    if (!p.in_place) return true;
    const int m = p.src_seq[s];
    return m == s || m == ARKV_SEQ_KEEP;
}

__device__ __forceinline__ int fork_source(const ForkParams& p, int b, bool* bad) {
    const int s = p.src_seq[b];
    *bad = false;
    if (s == ARKV_SEQ_FREE || s == ARKV_SEQ_KEEP) return s;
    if (s < 0 || s >= p.src_batch) {
        *bad = true;
        return kSkip;
    }
    if (p.in_place && s == b) return kSkip;
    if (!keeps_state(p, s)) {
        *bad = true;
        return kSkip;
    }
    return s;
}

template <class T>
__device__ __forceinline__ void copy_row(T* dst, const T* src, size_t n) {
    for (size_t i = threadIdx.x + (size_t)blockIdx.x * blockDim.x; i < n; i += (size_t)gridDim.x * blockDim.x)
        dst[i] = src[i];
}

__global__ void __launch_bounds__(256) cache_fork_kernel(const ForkParams p) {
    const int row = blockIdx.y, b = row / p.hkv, g = row % p.hkv;
    bool bad;
    const int s = fork_source(p, b, &bad);
    const bool first = blockIdx.x == 0 && threadIdx.x == 0;
    if (first && bad) atomicOr(p.dst.status, ARKV_STATUS_BAD_FORK);
    if (s == kSkip) return;
    if (s == kFree) {
        if (first) p.dst.n_bf16[row] = p.dst.n_fp8[row] = 0;
        return;
    }
    const size_t r = row, q = (size_t)s * p.hkv + g, D = p.D;
    const int m16 = min(max(p.src.n_bf16[q], 0), p.src_cap_o), m8 = min(max(p.src.n_fp8[q], 0), p.src_cap_q);
    const int n16 = min(m16, p.dst_cap_o), n8 = min(m8, p.dst_cap_q);
    if (first) {
        p.dst.n_bf16[row] = n16;
        p.dst.n_fp8[row] = n8;
        const int lost = (n16 < m16 ? ARKV_STATUS_BF16_FULL : 0) | (n8 < m8 ? ARKV_STATUS_FP8_FULL : 0);
        if (lost) atomicOr(p.dst.status, lost);
    }
    const size_t do_ = r * p.dst_cap_o, so = q * p.src_cap_o, dq = r * p.dst_cap_q, sq = q * p.src_cap_q;
    copy_row((uint4*)(p.dst.k16 + do_ * D), (const uint4*)(p.src.k16 + so * D), n16 * D / 8);
    copy_row((uint4*)(p.dst.v16 + do_ * D), (const uint4*)(p.src.v16 + so * D), n16 * D / 8);
    copy_row(p.dst.pos16 + do_, p.src.pos16 + so, n16);
    copy_row(p.dst.mu16 + do_, p.src.mu16 + so, n16);
    copy_row(p.dst.m2_16 + do_, p.src.m2_16 + so, n16);
    copy_row((uint4*)(p.dst.k8 + dq * D), (const uint4*)(p.src.k8 + sq * D), n8 * D / 16);
    copy_row((uint4*)(p.dst.v8 + dq * D), (const uint4*)(p.src.v8 + sq * D), n8 * D / 16);
    copy_row(p.dst.sk + dq, p.src.sk + sq, n8);
    copy_row(p.dst.sv + dq, p.src.sv + sq, n8);
    copy_row(p.dst.pos8 + dq, p.src.pos8 + sq, n8);
    copy_row(p.dst.mu8 + dq, p.src.mu8 + sq, n8);
    copy_row(p.dst.m2_8 + dq, p.src.m2_8 + sq, n8);
}

}  // namespace

cudaError_t launch_cache_fork(const ForkParams& p, cudaStream_t s) {
    const long long rows = (long long)p.dst_batch * p.hkv;
    if (rows > 65535) return cudaErrorInvalidValue;
    const int cap = p.dst_cap_o > p.dst_cap_q ? p.dst_cap_o : p.dst_cap_q;
    int x = (cap + 255) / 256;
    cache_fork_kernel<<<dim3(x < 1 ? 1 : x, (unsigned)rows), 256, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace arkv
