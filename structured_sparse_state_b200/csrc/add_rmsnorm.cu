// Residual addition and root-mean-square norm, forward (16-, 32- or 8-bit
// output) and backward.
//
//     s = x + residual,  rstd = (mean(s^2) + eps)^(-1/2),  out = s rstd w
//     g_s = rstd (g w - hat mean(g w hat)) + g_res,  hat = s rstd
//     g_w = sum over rows of g hat
//
// Bound: HBM, every operand once.  A row stays in the registers of TPR
// threads (at most 32 values each), so nothing is read twice; sums of squares
// and products go through warp shuffles and, above one warp, shared memory.
// The backward's CTAs are persistent: each thread owns the same columns of
// every row it sees and sums its share of g_w in registers; a CTA's sums go to
// scratch and a second kernel adds the CTAs in order, so the result does not
// depend on timing.  Of the measured copy rate the forward reaches 0.94 (65536 x
// 1024 bf16, 87 us) and 0.93 (16384 x 2048, fp32 stream, 67 us), the backward
// 0.87 (16384 x 2048, fp32 stream, 83 us) and 0.72 (65536 x 1024 bf16, 114 us).
#include <cuda_fp8.h>

#include <initializer_list>

#include "common.cuh"

namespace pdssm {
namespace {

// The types are uniform over a launch: one branch per 16-byte access keeps the
// kernels few, and these kernels wait for memory, not for issue slots.
template <int V>
__device__ __forceinline__ void load_vec(float (&v)[V], const void *p, int64_t at, int dt) {
    if constexpr (V == 8) {
        if (dt == PDSSM_F32) {
            const float4 *q = reinterpret_cast<const float4 *>((const float *)p + at);
            const float4 a = q[0], b = q[1];
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
            const uint4 a = *reinterpret_cast<const uint4 *>((const __nv_bfloat16 *)p + at);
            const unsigned w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    } else if constexpr (V == 2) {
        if (dt == PDSSM_F32) {
            const float2 a = *reinterpret_cast<const float2 *>((const float *)p + at);
            v[0] = a.x; v[1] = a.y;
        } else {
            const unsigned w = *reinterpret_cast<const unsigned *>((const __nv_bfloat16 *)p + at);
            v[0] = __uint_as_float(w << 16);
            v[1] = __uint_as_float(w & 0xffff0000u);
        }
    } else {
        v[0] = dt == PDSSM_F32 ? ((const float *)p)[at]
                               : __bfloat162float(((const __nv_bfloat16 *)p)[at]);
    }
}

__device__ __forceinline__ unsigned pack_bf16(float a, float b) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const unsigned *>(&t);
}

template <int V>
__device__ __forceinline__ void store_vec(const float (&v)[V], void *p, int64_t at, int dt) {
    if constexpr (V == 8) {
        if (dt == PDSSM_F32) {
            float4 *q = reinterpret_cast<float4 *>((float *)p + at);
            q[0] = make_float4(v[0], v[1], v[2], v[3]);
            q[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else if (dt == PDSSM_BF16) {
            *reinterpret_cast<uint4 *>((__nv_bfloat16 *)p + at) =
                make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                           pack_bf16(v[6], v[7]));
        } else {
            // round to nearest, saturating; the row's scale keeps values within 448
            unsigned w[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const unsigned t = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i], v[2 * i + 1]),
                                                            __NV_SATFINITE, __NV_E4M3);
                w[i / 2] |= t << (16 * (i % 2));
            }
            *reinterpret_cast<uint2 *>((unsigned char *)p + at) = make_uint2(w[0], w[1]);
        }
    } else if constexpr (V == 2) {
        if (dt == PDSSM_F32)
            *reinterpret_cast<float2 *>((float *)p + at) = make_float2(v[0], v[1]);
        else
            *reinterpret_cast<unsigned *>((__nv_bfloat16 *)p + at) = pack_bf16(v[0], v[1]);
    } else {
        if (dt == PDSSM_F32)
            ((float *)p)[at] = v[0];
        else if (dt == PDSSM_BF16)
            ((__nv_bfloat16 *)p)[at] = __float2bfloat16_rn(v[0]);
        else
            ((unsigned char *)p)[at] = __nv_cvt_float_to_fp8(v[0], __NV_SATFINITE, __NV_E4M3);
    }
}

// A NaN must reach the row's scale: max that keeps it.
__device__ __forceinline__ float max_nan(float a, float b) {
    return (a > b || a != a) ? a : b;
}

struct AddOp {
    __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
struct MaxOp {
    __device__ __forceinline__ float operator()(float a, float b) const { return max_nan(a, b); }
};

// Reduction over the TPR threads of a row (TPR = 32, or the whole CTA); `red`
// holds one value per warp and is free again after the call's last barrier.
template <int TPR, class OP>
__device__ __forceinline__ float row_reduce(float v, float *red, OP op) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v = op(v, __shfl_xor_sync(kFull, v, d));
    if constexpr (TPR > 32) {
        __syncthreads();
        if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int w = 1; w < TPR / 32; ++w) v = op(v, red[w]);
    }
    return v;
}

// The sums alone, of NR rows, with one barrier: the caller alternates between
// two buffers, so that a buffer is written again only after the next call's
// barrier.
template <int TPR, int NR>
__device__ __forceinline__ void row_sums_once(float (&v)[NR], float *red) {
#pragma unroll
    for (int k = 0; k < NR; ++k) {
#pragma unroll
        for (int d = 16; d; d >>= 1) v[k] += __shfl_xor_sync(kFull, v[k], d);
        if (TPR > 32 && threadIdx.x % 32 == 0) red[k * (TPR / 32) + threadIdx.x / 32] = v[k];
    }
    if constexpr (TPR > 32) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < NR; ++k) {
            v[k] = red[k * (TPR / 32)];
#pragma unroll
            for (int w = 1; w < TPR / 32; ++w) v[k] += red[k * (TPR / 32) + w];
        }
    }
}

struct NormParams {
    int64_t rows;
    int D;
    const void *x, *residual, *weight;
    void *out, *res_out;
    float *rstd, *scale;
    int x_dt, res_dt, w_dt, out_dt;
    float eps;
};

constexpr int kRowValues = 32;      // most values of a row per thread

// TPR = 32: a warp per row, 4 rows per CTA; else a CTA per row.  A thread takes
// pieces of V values.  SHIFT: rows of a width that is no multiple of 8, whose
// first pieces start before the row, so that every piece lies on its 8 values;
// the row's first and last pieces go value by value (2020 rows of 4143 bf16
// values: 30 us, all values by themselves 95).
template <int TPR, int V, bool SHIFT>
__global__ void __launch_bounds__(TPR == 32 ? 128 : TPR, TPR == 128 && V == 8 ? 8 : 0) k_add_rmsnorm(NormParams p) {
    constexpr int NV = kRowValues / V;
    __shared__ float red[32];
    const int lane = TPR == 32 ? threadIdx.x % 32 : threadIdx.x;
    const int64_t row = TPR == 32 ? (int64_t)blockIdx.x * 4 + threadIdx.x / 32 : blockIdx.x;
    if (row >= p.rows) return;          // TPR = 32 only, where no barrier follows
    const int64_t base = row * p.D;
    const int shift = SHIFT ? (int)(base & 7) : 0;
    auto col_of = [&](int i) { return (i * TPR + lane) * V - shift; };
    auto whole = [&](int col) { return !SHIFT || (col >= 0 && col + V <= p.D); };
    auto load = [&](float (&v)[V], const void *src, int64_t from, int col, int dt) {
        if (whole(col)) {
            load_vec<V>(v, src, from + col, dt);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float one[1] = {0.f};
                if (col + j >= 0 && col + j < p.D) load_vec<1>(one, src, from + col + j, dt);
                v[j] = one[0];
            }
        }
    };
    auto store = [&](const float (&v)[V], void *dst, int col, int dt) {
        if (whole(col)) {
            store_vec<V>(v, dst, base + col, dt);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float one[1] = {v[j]};
                if (col + j >= 0 && col + j < p.D) store_vec<1>(one, dst, base + col + j, dt);
            }
        }
    };
    float s[NV][V];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (col_of(i) < p.D) load(s[i], p.x, base, col_of(i), p.x_dt);
    if (p.residual) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (col_of(i) >= p.D) continue;
            float r[V];
            load(r, p.residual, base, col_of(i), p.res_dt);
#pragma unroll
            for (int j = 0; j < V; ++j) s[i][j] += r[j];
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (col_of(i) >= p.D) continue;
        if (p.res_dt == PDSSM_BF16) {   // the norm is of the rounded sum
#pragma unroll
            for (int j = 0; j < V; ++j) s[i][j] = __bfloat162float(__float2bfloat16_rn(s[i][j]));
        }
#pragma unroll
        for (int j = 0; j < V; ++j) sum = fmaf(s[i][j], s[i][j], sum);
    }
    sum = row_reduce<TPR>(sum, red, AddOp());
    const float rstd = 1.f / sqrtf(sum / (float)p.D + p.eps);
    if (p.rstd && lane == 0) p.rstd[row] = rstd;
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int col = col_of(i);
        if (col >= p.D) continue;
        if (p.res_out) store(s[i], p.res_out, col, p.res_dt);
        float w[V];
        if constexpr (SHIFT) {
            const bool f32 = p.w_dt == PDSSM_F32;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = min(max(col + j, 0), p.D - 1);
                w[j] = f32 ? __ldg((const float *)p.weight + c)
                           : __bfloat162float(((const __nv_bfloat16 *)p.weight)[c]);
            }
        } else {
            load_vec<V>(w, p.weight, col, p.w_dt);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            s[i][j] = s[i][j] * rstd * w[j];
            if (SHIFT && (col + j < 0 || col + j >= p.D)) s[i][j] = 0.f;    // no part of the row
            top = max_nan(top, fabsf(s[i][j]));
        }
        if (p.out_dt != PDSSM_E4M3) store(s[i], p.out, col, p.out_dt);
    }
    if (p.out_dt != PDSSM_E4M3) return;
    top = row_reduce<TPR>(top, red, MaxOp());
    float scale = top / 448.f;
    if (scale == 0.f) scale = 1.f;
    if (lane == 0) p.scale[row] = scale;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (col_of(i) >= p.D) continue;
#pragma unroll
        for (int j = 0; j < V; ++j) s[i][j] = s[i][j] / scale;
        store(s[i], p.out, col_of(i), p.out_dt);
    }
}

struct NormBwdParams {
    int64_t rows;
    int D, ctas;
    const void *g_out, *s, *weight, *g_res;
    const float *rstd;
    void *g_x;
    float *part;                // [ctas][D]
    int g_dt, res_dt, w_dt;
};

constexpr int kBwdValues = 16;      // values per thread: of one row, or of two

// TPR = 32: 4 warps per CTA, a row per warp at a time; else a row per CTA, or
// NR rows of at most kBwdValues / NR values per thread (65536 rows of 1024 in
// bf16: one row, too little in flight, 161 us; two 144, and with the next rows
// prefetched 111).  The weights are read again for every row (from L1): held in
// registers they would cost a CTA per SM.
template <int TPR, int V, int GD, int RD, int NR>
__global__ void __launch_bounds__(TPR == 32 ? 128 : TPR, TPR <= 128 ? 5 : TPR == 256 ? 2 : 1)
    k_add_rmsnorm_bwd(NormBwdParams p) {
    constexpr int NV = kBwdValues / NR / V;
    constexpr int RPC = TPR == 32 ? 4 : NR;
    __shared__ float red[64];
    __shared__ float comb[TPR == 32 ? 4 * 32 * kBwdValues : 1];
    const int lane = TPR == 32 ? threadIdx.x % 32 : threadIdx.x;
    const int sub = TPR == 32 ? threadIdx.x / 32 : 0;
    float gw[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) gw[i][j] = 0.f;
    int turn = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * RPC + sub; row0 < p.rows;
         row0 += (int64_t)gridDim.x * RPC) {
        float g[NR][NV][V], h[NR][NV][V], r[NR][NV][V], rstd[NR], dot[NR];
        auto each = [&](auto &&f) {         // f(k, i, col) of the values there are
#pragma unroll
            for (int k = 0; k < NR; ++k)
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int col = (i * TPR + lane) * V;
                    if (col < p.D && (NR == 1 || row0 + k < p.rows)) f(k, i, col);
                }
        };
#pragma unroll
        for (int k = 0; k < NR; ++k) {
            rstd[k] = NR == 1 || row0 + k < p.rows ? p.rstd[row0 + k] : 0.f;
            dot[k] = 0.f;
        }
        each([&](int k, int i, int col) {
            load_vec<V>(g[k][i], p.g_out, (row0 + k) * p.D + col, GD);
            load_vec<V>(h[k][i], p.s, (row0 + k) * p.D + col, RD);
        });
        if (p.g_res)
            each([&](int k, int i, int col) {
                load_vec<V>(r[k][i], p.g_res, (row0 + k) * p.D + col, RD);
            });
        // the next turn's rows on their way to L2
        const int64_t next = row0 + (int64_t)gridDim.x * RPC;
        if (next < p.rows) {
            const int64_t n = NR == 1 ? p.D : imin64(NR, p.rows - next) * p.D;
            auto ahead = [&](const void *t, int size) {
                const char *at = (const char *)t + next * p.D * size;
                for (int64_t o = lane * 128; o < n * size; o += TPR * 128)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(at + o));
            };
            ahead(p.g_out, GD == PDSSM_F32 ? 4 : 2);
            ahead(p.s, RD == PDSSM_F32 ? 4 : 2);
            if (p.g_res) ahead(p.g_res, RD == PDSSM_F32 ? 4 : 2);
        }
        each([&](int k, int i, int col) {
            float w[V];
            load_vec<V>(w, p.weight, col, p.w_dt);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                h[k][i][j] *= rstd[k];
                gw[i][j] = fmaf(g[k][i][j], h[k][i][j], gw[i][j]);
                g[k][i][j] *= w[j];
                dot[k] = fmaf(g[k][i][j], h[k][i][j], dot[k]);
            }
        });
        // rows take the two halves of `red` in turn: one barrier per turn
        row_sums_once<TPR, NR>(dot, red + 32 * (turn ^= 1));
        each([&](int k, int i, int col) {
            const float mean = dot[k] / (float)p.D;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                g[k][i][j] = (g[k][i][j] - h[k][i][j] * mean) * rstd[k];
                if (p.g_res) g[k][i][j] += r[k][i][j];
            }
            store_vec<V>(g[k][i], p.g_x, (row0 + k) * p.D + col, RD);
        });
    }
    if constexpr (TPR == 32) {          // the CTA's four warps hold the same columns
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j)
                comb[(sub * 32 + lane) * kBwdValues + i * V + j] = gw[i][j];
        __syncthreads();
        if (sub) return;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j)
                for (int q = 1; q < 4; ++q)
                    gw[i][j] += comb[(q * 32 + lane) * kBwdValues + i * V + j];
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int col = (i * TPR + lane) * V;
        if (col >= p.D) continue;
#pragma unroll
        for (int j = 0; j < V; ++j) p.part[(int64_t)blockIdx.x * p.D + col + j] = gw[i][j];
    }
}

// g_w: the CTAs' sums in order, 32 columns per CTA, 32 partial sums per column
__global__ void __launch_bounds__(1024) k_rmsnorm_gw(const float *part, int ctas, int D,
                                                     float *g_w) {
    __shared__ float sm[32][33];
    const int col = blockIdx.x * 32 + threadIdx.x % 32, sub = threadIdx.x / 32;
    float s = 0.f;
    if (col < D)
        for (int c = sub; c < ctas; c += 32) s += part[(int64_t)c * D + col];
    sm[sub][threadIdx.x % 32] = s;
    __syncthreads();
    s = sm[threadIdx.x % 32][sub];
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(kFull, s, d);
    if (threadIdx.x % 32 == 0 && blockIdx.x * 32 + sub < D) g_w[blockIdx.x * 32 + sub] = s;
}

constexpr int kMaxD = 16384;

// CTAs of the backward: enough to fill the GPU (about 16 warps per SM), no
// more than rows
int bwd_tpr(int64_t D) {
    return D <= 32 * kBwdValues ? 32 : D <= 128 * kBwdValues ? 128 : D <= 256 * kBwdValues ? 256
           : D <= 512 * kBwdValues ? 512 : 1024;
}
// rows of a CTA at once
int bwd_rows(int64_t D) { return bwd_tpr(D) == 128 && D <= 64 * kBwdValues ? 2 : 1; }
int64_t bwd_ctas(int64_t rows, int64_t D) {
    const int tpr = bwd_tpr(D);
    const int rpc = tpr == 32 ? 4 : bwd_rows(D);
    const int per_sm = tpr <= 128 ? 5 : tpr == 256 ? 2 : 1;     // as many as are resident
    const int64_t n = (rows + rpc - 1) / rpc, most = 148 * per_sm;
    return n < most ? (n > 0 ? n : 1) : most;
}

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
// values per access: eight where rows and pointers lie on 16 bytes, two on 8
int width_of(int64_t D, std::initializer_list<const void *> ptrs) {
    int v = D % 8 == 0 ? 8 : D % 2 == 0 ? 2 : 1;
    for (const void *q : ptrs) {
        if (!aligned(q, 8)) return 1;
        if (!aligned(q, 16) && v == 8) v = 2;
    }
    return v;
}
bool wide(int dt) { return dt == PDSSM_F32 || dt == PDSSM_BF16; }

template <int V, bool SHIFT>
cudaError_t run_fwd(const NormParams &p, cudaStream_t st) {
    const unsigned rows = (unsigned)p.rows;
    const int width = p.D + (SHIFT ? 7 : 0);
    if (width <= 32 * kRowValues)
        k_add_rmsnorm<32, V, SHIFT><<<(rows + 3) / 4, 128, 0, st>>>(p);
    else if (width <= 128 * kRowValues)
        k_add_rmsnorm<128, V, SHIFT><<<rows, 128, 0, st>>>(p);
    else if (width <= 256 * kRowValues)
        k_add_rmsnorm<256, V, SHIFT><<<rows, 256, 0, st>>>(p);
    else
        k_add_rmsnorm<512, V, SHIFT><<<rows, 512, 0, st>>>(p);
    return cudaGetLastError();
}

// Types as template arguments here: with the branch of load_vec the row's
// registers cost a quarter of the resident CTAs (108 us against 96 at 16384 x
// 2048, fp32 stream).
template <int V, int GD, int RD>
cudaError_t run_bwd_t(const NormBwdParams &p, cudaStream_t st) {
    switch (bwd_tpr(p.D)) {
        case 32: k_add_rmsnorm_bwd<32, V, GD, RD, 1><<<p.ctas, 128, 0, st>>>(p); break;
        case 128:
            if (bwd_rows(p.D) == 2)
                k_add_rmsnorm_bwd<128, V, GD, RD, 2><<<p.ctas, 128, 0, st>>>(p);
            else
                k_add_rmsnorm_bwd<128, V, GD, RD, 1><<<p.ctas, 128, 0, st>>>(p);
            break;
        case 256: k_add_rmsnorm_bwd<256, V, GD, RD, 1><<<p.ctas, 256, 0, st>>>(p); break;
        case 512: k_add_rmsnorm_bwd<512, V, GD, RD, 1><<<p.ctas, 512, 0, st>>>(p); break;
        default: k_add_rmsnorm_bwd<1024, V, GD, RD, 1><<<p.ctas, 1024, 0, st>>>(p); break;
    }
    return cudaGetLastError();
}

template <int V>
cudaError_t run_bwd(const NormBwdParams &p, cudaStream_t st) {
    if (p.g_dt == PDSSM_F32)
        return p.res_dt == PDSSM_F32 ? run_bwd_t<V, PDSSM_F32, PDSSM_F32>(p, st)
                                     : run_bwd_t<V, PDSSM_F32, PDSSM_BF16>(p, st);
    return p.res_dt == PDSSM_F32 ? run_bwd_t<V, PDSSM_BF16, PDSSM_F32>(p, st)
                                 : run_bwd_t<V, PDSSM_BF16, PDSSM_BF16>(p, st);
}

pdssm_status check_sizes(int64_t rows, int64_t D) {
    if (rows < 0 || D < 1) return arg_fail(PDSSM_ERR_INVALID_ARG, "need rows >= 0 and D >= 1");
    if (D > kMaxD) return arg_fail(PDSSM_ERR_UNSUPPORTED, "D > 16384");
    if (rows > 0x7fffffff) return arg_fail(PDSSM_ERR_UNSUPPORTED, "rows >= 2^31");
    return PDSSM_OK;
}

}  // namespace
}  // namespace pdssm

using namespace pdssm;

extern "C" {

pdssm_status pdssm_add_rmsnorm_fwd(int64_t rows, int64_t D, const void *x, pdssm_dtype x_dtype,
                                   const void *residual, pdssm_dtype res_dtype,
                                   const void *weight, pdssm_dtype w_dtype, float eps, void *out,
                                   pdssm_dtype out_dtype, void *res_out, float *rstd, float *scale,
                                   void *stream) {
    pdssm_status st = check_sizes(rows, D);
    if (st != PDSSM_OK) return st;
    if (!wide(x_dtype) || !wide(res_dtype) || !wide(w_dtype) ||
        (!wide(out_dtype) && out_dtype != PDSSM_E4M3))
        return arg_fail(PDSSM_ERR_INVALID_ARG, "unknown dtype");
    if (!(eps >= 0.f) || eps > 3.0e38f)
        return arg_fail(PDSSM_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if ((out_dtype == PDSSM_E4M3) != (scale != nullptr) && rows > 0)
        return arg_fail(PDSSM_ERR_INVALID_ARG, "scale goes with an 8-bit output, and only with it");
    if (rows == 0) return PDSSM_OK;
    if (!x || !weight || !out) return arg_fail(PDSSM_ERR_INVALID_ARG, "NULL tensor pointer");
    NormParams p{rows, (int)D, x, residual, weight, out, res_out, rstd, scale,
                 x_dtype, res_dtype, w_dtype, out_dtype, eps};
    bool grid = true;
    for (const void *q : {x, residual, (const void *)res_out, (const void *)out}) grid = grid && aligned(q, 16);
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e = grid && D % 8 == 0 && aligned(weight, 16) ? run_fwd<8, false>(p, s)
                    : grid && D + 7 <= kMaxD                  ? run_fwd<8, true>(p, s)
                                                              : run_fwd<1, false>(p, s);
    return e == cudaSuccess ? PDSSM_OK : cuda_fail(e, "add + norm");
}

size_t pdssm_add_rmsnorm_scratch_bytes(int64_t rows, int64_t D) {
    if (check_sizes(rows, D) != PDSSM_OK) return 0;
    return align256((size_t)bwd_ctas(rows, D) * (size_t)D * 4);
}

pdssm_status pdssm_add_rmsnorm_bwd(int64_t rows, int64_t D, const void *g_out, pdssm_dtype g_dtype,
                                   const void *res_out, pdssm_dtype res_dtype, const void *weight,
                                   pdssm_dtype w_dtype, const float *rstd, const void *g_res,
                                   void *g_x, float *g_weight, void *scratch, size_t scratch_bytes,
                                   void *stream) {
    pdssm_status st = check_sizes(rows, D);
    if (st != PDSSM_OK) return st;
    if (!wide(g_dtype) || !wide(res_dtype) || !wide(w_dtype))
        return arg_fail(PDSSM_ERR_INVALID_ARG, "unknown dtype");
    if (!g_weight) return arg_fail(PDSSM_ERR_INVALID_ARG, "NULL g_weight");
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (rows == 0) {
        e = cudaMemsetAsync(g_weight, 0, (size_t)D * 4, s);
        return e == cudaSuccess ? PDSSM_OK : cuda_fail(e, "g_weight of no rows");
    }
    if (!g_out || !res_out || !weight || !rstd || !g_x)
        return arg_fail(PDSSM_ERR_INVALID_ARG, "NULL tensor pointer");
    if (!scratch || !aligned(scratch, 256))
        return arg_fail(PDSSM_ERR_INVALID_ARG, "scratch NULL or not 256-byte aligned");
    if (scratch_bytes < pdssm_add_rmsnorm_scratch_bytes(rows, D))
        return arg_fail(PDSSM_ERR_WORKSPACE, "scratch too small");
    NormBwdParams p{rows, (int)D, (int)bwd_ctas(rows, D), g_out, res_out, weight, g_res, rstd, g_x,
                    (float *)scratch, g_dtype, res_dtype, w_dtype};
    const int v = width_of(D, {g_out, res_out, weight, g_res, g_x});
    e = v == 8 ? run_bwd<8>(p, s) : v == 2 ? run_bwd<2>(p, s) : run_bwd<1>(p, s);
    if (e != cudaSuccess) return cuda_fail(e, "add + norm backward");
    k_rmsnorm_gw<<<(unsigned)((D + 31) / 32), 1024, 0, s>>>(p.part, p.ctas, (int)D, g_weight);
    e = cudaGetLastError();
    return e == cudaSuccess ? PDSSM_OK : cuda_fail(e, "weight gradient");
}

}  // extern "C"
