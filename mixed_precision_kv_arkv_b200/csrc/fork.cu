// arkv_cache_fork: copies, forks and frees the sequences of a packed cache (live slots,
// counts and score state), slot by slot in place.
//
// A block owns one 16 KB piece of a source row's K or V codes (or 512 slots of its scales,
// positions and score state), reads it once into registers and writes it to every
// destination of that source, so that a prompt forked n times is read once.
//
// Bound: HBM, each source's live bytes read once and written once a destination.  One 32K
// prompt (35.97 MB of live slots) to 16 sequences: 611.4 MB, floor 94.6 us at 6461.5 GB/s;
// 115 us measured
// (5.3 TB/s, of which 15/16 are writes).
#include "arkv_internal.cuh"

namespace arkv {

namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 4;                                 // 16-byte vectors of a piece, a thread
constexpr int kPiece = kThreads * kVecs * 16;
constexpr int kSlotsPer = 512;                           // slots of a piece of the small arrays
constexpr int kList = 512;                               // destinations handled at a time

// Whether sequence s still holds its state when the call is over.
__device__ __forceinline__ bool keeps_state(const ForkParams& p, int s) {
    if (!p.in_place) return true;
    const int m = p.src_seq[s];
    return m == s || m == ARKV_SEQ_KEEP;
}

struct Pieces {
    int k16, k8, s16, s8;   // pieces of a row: bf16 K (and V), FP8 K (and V), small arrays of either segment
    __host__ __device__ int total() const { return 2 * k16 + 2 * k8 + s16 + s8; }
};

// n elements of a small array from src (starting at `from`) to every listed destination row.
template <class T>
__device__ __forceinline__ void copy_small(T* dst, const T* src, int cap_dst, int from, int n, const int* list, int count,
                                           int hkv, int g) {
    constexpr int kPer = kSlotsPer / kThreads;
    T v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int k = from + threadIdx.x + i * kThreads;
        if (k < n) v[i] = src[k];
    }
    for (int c = 0; c < count; ++c) {
        T* to = dst + (size_t)(list[c] * hkv + g) * cap_dst;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int k = from + threadIdx.x + i * kThreads;
            if (k < n) to[k] = v[i];
        }
    }
}

// `per_row` blocks share the pieces of a source row round robin.
__global__ void __launch_bounds__(kThreads, 4) cache_fork_kernel(const __grid_constant__ ForkParams p, Pieces pc, int per_row) {
    __shared__ int list[kList];
    __shared__ int count;
    const int tid = threadIdx.x, pieces = pc.total();
    const int row = blockIdx.x / per_row, s = row / p.hkv, g = row - s * p.hkv, first = blockIdx.x - row * per_row;
    const size_t D = p.D;
    if (blockIdx.x == 0) {   // what has no source: freed sequences, and refused ones
        for (int b = tid; b < p.dst_batch; b += kThreads) {
            const int m = p.src_seq[b];
            if (m == ARKV_SEQ_FREE)
                for (int i = 0; i < p.hkv; ++i) p.dst.n_bf16[b * p.hkv + i] = p.dst.n_fp8[b * p.hkv + i] = 0;
            else if (m != ARKV_SEQ_KEEP && (m < 0 || m >= p.src_batch || (m != b && !keeps_state(p, m))))
                atomicOr(p.dst.status, ARKV_STATUS_BAD_FORK);
        }
    }
    if (!keeps_state(p, s)) return;
    const int m16 = min(max(p.src.n_bf16[row], 0), p.src_cap_o), m8 = min(max(p.src.n_fp8[row], 0), p.src_cap_q);
    const int n16 = min(m16, p.dst_cap_o), n8 = min(m8, p.dst_cap_q);
    for (int b0 = 0; b0 < p.dst_batch; b0 += kList) {
        __syncthreads();
        if (tid == 0) count = 0;
        __syncthreads();
        for (int b = b0 + tid; b < min(b0 + kList, p.dst_batch); b += kThreads)
            if (p.src_seq[b] == s && !(p.in_place && b == s)) list[atomicAdd(&count, 1)] = b;
        __syncthreads();
        const int n = count;
        if (n == 0) continue;
        if (first == 0)
            for (int c = tid; c < n; c += kThreads) {
                const int to = list[c] * p.hkv + g;
                p.dst.n_bf16[to] = n16;
                p.dst.n_fp8[to] = n8;
                const int lost = (n16 < m16 ? ARKV_STATUS_BF16_FULL : 0) | (n8 < m8 ? ARKV_STATUS_FP8_FULL : 0);
                if (lost) atomicOr(p.dst.status, lost);
            }
        for (int at_piece = first; at_piece < pieces; at_piece += per_row) {
            int piece = at_piece, kind;   // which array, and which piece of it
            if (piece < 2 * pc.k16) kind = piece & 1, piece >>= 1;
            else if ((piece -= 2 * pc.k16) < 2 * pc.k8) kind = 2 + (piece & 1), piece >>= 1;
            else if ((piece -= 2 * pc.k8) < pc.s16) kind = 4;
            else kind = 5, piece -= pc.s16;
            if (kind < 4) {
                const bool b16 = kind < 2;
                const size_t bytes = b16 ? n16 * D * 2 : n8 * D, from = (size_t)piece * kPiece;
                if (from >= bytes) continue;
                const size_t src_row = b16 ? p.src_cap_o * D * 2 : p.src_cap_q * D;
                const size_t dst_row = b16 ? p.dst_cap_o * D * 2 : p.dst_cap_q * D;
                const char* src = (const char*)(kind == 0 ? (const void*)p.src.k16 : kind == 1 ? (const void*)p.src.v16
                                                : kind == 2 ? (const void*)p.src.k8 : (const void*)p.src.v8) + row * src_row + from;
                char* dst = (char*)(kind == 0 ? (void*)p.dst.k16 : kind == 1 ? (void*)p.dst.v16
                                    : kind == 2 ? (void*)p.dst.k8 : (void*)p.dst.v8) + from;
                const int left = (int)min(bytes - from, (size_t)kPiece);
                uint4 v[kVecs];
#pragma unroll
                for (int i = 0; i < kVecs; ++i)
                    if ((tid + i * kThreads) * 16 < left) v[i] = __ldcs(reinterpret_cast<const uint4*>(src) + tid + i * kThreads);
                for (int c = 0; c < n; ++c) {
                    uint4* to = reinterpret_cast<uint4*>(dst + (size_t)(list[c] * p.hkv + g) * dst_row) + tid;
#pragma unroll
                    for (int i = 0; i < kVecs; ++i)
                        if ((tid + i * kThreads) * 16 < left) __stcs(to + i * kThreads, v[i]);
                }
                continue;
            }
            const int k0 = piece * kSlotsPer;
            const size_t so = (size_t)row * p.src_cap_o, sq = (size_t)row * p.src_cap_q;
            if (kind == 4 && k0 < n16) {
                copy_small(p.dst.pos16, p.src.pos16 + so, p.dst_cap_o, k0, n16, list, n, p.hkv, g);
                copy_small(p.dst.mu16, p.src.mu16 + so, p.dst_cap_o, k0, n16, list, n, p.hkv, g);
                copy_small(p.dst.m2_16, p.src.m2_16 + so, p.dst_cap_o, k0, n16, list, n, p.hkv, g);
            } else if (kind == 5 && k0 < n8) {
                copy_small(p.dst.pos8, p.src.pos8 + sq, p.dst_cap_q, k0, n8, list, n, p.hkv, g);
                copy_small(p.dst.sk, p.src.sk + sq, p.dst_cap_q, k0, n8, list, n, p.hkv, g);
                copy_small(p.dst.sv, p.src.sv + sq, p.dst_cap_q, k0, n8, list, n, p.hkv, g);
                copy_small(p.dst.mu8, p.src.mu8 + sq, p.dst_cap_q, k0, n8, list, n, p.hkv, g);
                copy_small(p.dst.m2_8, p.src.m2_8 + sq, p.dst_cap_q, k0, n8, list, n, p.hkv, g);
            }
        }
    }
}

}  // namespace

cudaError_t launch_cache_fork(const ForkParams& p, cudaStream_t s) {
    auto up = [](long long x, long long y) { return (int)((x + y - 1) / y); };
    const int cap_o = p.src_cap_o < p.dst_cap_o ? p.src_cap_o : p.dst_cap_o;
    const int cap_q = p.src_cap_q < p.dst_cap_q ? p.src_cap_q : p.dst_cap_q;
    Pieces pc;
    pc.k16 = up((long long)cap_o * p.D * 2, kPiece);
    pc.k8 = up((long long)cap_q * p.D, kPiece);
    pc.s16 = up(cap_o, kSlotsPer);
    pc.s8 = up(cap_q, kSlotsPer);
    // A block a piece, but no more than about eight waves of a B200's 148 SMs: rows that nobody copies (most of
    // them, when a few sequences of a large batch move) cost their blocks all the same (8 of 32
    // sequences replaced: 49.6 us with a block a piece, 26.6 us so).
    const long long rows = (long long)p.src_batch * p.hkv, most = (8ll * 4 * 148 + rows - 1) / rows;
    const int per_row = (int)(pc.total() < most ? pc.total() : most);
    const long long blocks = rows * per_row;
    cache_fork_kernel<<<(unsigned)blocks, kThreads, 0, s>>>(p, pc, per_row);
    return cudaGetLastError();
}

}  // namespace arkv
