// Products of shared-memory tiles on the CUDA cores: 16 x 16 threads, each with
// a TM x TN tile of the result in registers.
#pragma once

namespace pdssm {

// Where a thread's i-th row or column of a tile lies: in pairs, so that an
// operand whose rows run along the product's k is read by 8-byte loads, or
// strided, for operands that run across it.
__device__ __forceinline__ int pairs(int t, int i) { return 2 * t + (i & 1) + 32 * (i >> 1); }
__device__ __forceinline__ int strided(int t, int i) { return t + 16 * i; }

// Operands of a product, four values of k at a time:
// Along: element (i, k) at [idx(i)][k], one 16-byte load per row
template <int T, bool PAIRS>
struct Along {
    const float *p;
    int ld, t;
    __device__ __forceinline__ void load(float (&v)[T][4], int k) const {
#pragma unroll
        for (int i = 0; i < T; ++i) {
            const float4 x = *reinterpret_cast<const float4 *>(
                p + (PAIRS ? pairs(t, i) : strided(t, i)) * ld + k);
            v[i][0] = x.x; v[i][1] = x.y; v[i][2] = x.z; v[i][3] = x.w;
        }
    }
};
// Along, rows strided and off the 16-byte grid: two 8-byte loads per row
template <int T>
struct Along2 {
    const float *p;
    int ld, t;
    __device__ __forceinline__ void load(float (&v)[T][4], int k) const {
#pragma unroll
        for (int i = 0; i < T; ++i) {
            const float2 *at = reinterpret_cast<const float2 *>(p + strided(t, i) * ld + k);
            const float2 x = at[0], y = at[1];
            v[i][0] = x.x; v[i][1] = x.y; v[i][2] = y.x; v[i][3] = y.y;
        }
    }
};
// Across: element (i, k) at [k][idx(i)], one 8-byte load per pair and k
template <int T>
struct Across {
    const float *p;
    int ld, t;
    __device__ __forceinline__ void load(float (&v)[T][4], int k) const {
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int i = 0; i < T; i += 2) {
                const float2 x =
                    *reinterpret_cast<const float2 *>(p + (k + q) * ld + pairs(t, i));
                v[i][q] = x.x;
                v[i + 1][q] = x.y;
            }
    }
};

// acc[i][j] += sum_k a(i, k) b(j, k), K a multiple of 4
template <int TM, int TN, class FA, class FB>
__device__ __forceinline__ void tile_mm(float (&acc)[TM][TN], int K, const FA &a, const FB &b) {
#pragma unroll 2
    for (int k = 0; k < K; k += 4) {
        float av[TM][4], bv[TN][4];
        a.load(av, k);
        b.load(bv, k);
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) acc[i][j] = fmaf(av[i][q], bv[j][q], acc[i][j]);
    }
}

template <int TM, int TN>
__device__ __forceinline__ void zero(float (&acc)[TM][TN]) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = 0.f;
}

}  // namespace pdssm
