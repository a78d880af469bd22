// Balance loss of the hard selection: what its kernels share.
#pragma once

#include "common.cuh"

namespace pdssm {

constexpr int kBalMaxK = 32, kBalMaxD = 256;

struct BalParams {
    int B, H, K, D;
    int64_t L, rows;                    // rows = B L
    const void *u;
    const float *W;
    const int32_t *k;
    const int32_t *lengths;
    const int64_t *steps;               // in front of the lengths, of more than kBalWarpB sequences
    float inv_tau;
    const int32_t *counts;
    const float *g_loss;
    void *g_u;
    int slices;                         // of the steps
    int heads, groups, gslices, vec;    // fp32: heads per group, groups, their slices for g_u,
                                        // 16-byte accesses
    float *part;                        // per slice: sums of p [H][K], of g_W [H][K][D], or of
                                        // g_u [rows][D]
    int32_t *part_n;                    // per slice: counts [H][K]
};

__device__ __forceinline__ int64_t bal_len(const BalParams &p, int b) {
    if (!p.lengths) return p.L;
    const int64_t n = p.lengths[b];
    return n < 0 ? 0 : (n > p.L ? p.L : n);
}

// steps in front of the lengths, for a whole warp: of more sequences than a
// warp has lanes, they have been counted before (k_bal_steps)
constexpr int kBalWarpB = 32;
__device__ __forceinline__ int64_t bal_steps(const BalParams &p) {
    if (!p.lengths) return p.rows;
    if (p.steps) return *p.steps;
    const int lane = threadIdx.x % 32;
    int64_t n = lane < p.B ? bal_len(p, lane) : 0;
#pragma unroll
    for (int d = 16; d; d >>= 1) n += __shfl_xor_sync(kFull, n, d);
    return n;
}

// counts / T of one entry, less 1 / K: the probabilities' sum is 1, so the
// gradients are of f_k - sum p f whatever is taken from every f alike, and of a
// selection that is nearly even the difference is what counts (2 entries, 30000
// steps, fp32: g_W off by 2.2e-5 of its norm with f itself, by less than a tenth
// of that so)
__device__ __forceinline__ float bal_excess(int32_t count, int K, int64_t steps) {
    // an exact whole number, rounded once, and the same factor for every entry
    return steps > 0 ? (float)(count * (int64_t)K - steps) * (1.f / ((float)K * (float)steps)) : 0.f;
}

__device__ __forceinline__ bool bal_live(const BalParams &p, int64_t row) {
    if (row >= p.rows) return false;
    if (!p.lengths) return true;
    const uint32_t b = (uint32_t)row / (uint32_t)p.L;       // B L < 2^31
    return (int64_t)((uint32_t)row - b * (uint32_t)p.L) < bal_len(p, (int)b);
}

// Plan of the tensor-core kernels (bf16 u): groups of heads whose weights, as
// three bf16 parts, lie in shared memory.
struct BalTcPlan {
    int KT;                             // entries of a head, rounded up to a power of two
    int N;                              // entries of a group (heads per group * KT): 64 or 128
    int Dp;                             // D rounded up to 64
    int groups, slices, tiles;          // slices of the 128-row tiles per group
    size_t w_bytes;                     // bytes of one group's parts
};
BalTcPlan bal_tc_plan(const pdssm_dims &d);
size_t bal_tc_extra(const BalTcPlan &pl);   // scratch behind the partial sums
// what: 0 sums and counts, 1 g_u, 2 g_W partials (slices of [H][K][D])
cudaError_t launch_bal_tc(const BalParams &p, const BalTcPlan &pl, int what, void *w_parts,
                          cudaStream_t st);
cudaError_t launch_bal_tc_prep(const BalParams &p, const BalTcPlan &pl, void *w_parts,
                               cudaStream_t st);

}  // namespace pdssm
