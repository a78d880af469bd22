// Decay scan (linear attention with a decay for each head): shared
// parameters, addressing and the chunk's decay sums.
//
//     S_t = a_t S_{t-1} + b_t x_t^T,   y_t = S_t^T c_t,   a_t = exp(log_a_t)
//
// in chunks of C steps: with G_i the sum of log_a over the chunk's steps
// 0..i and S0 the state at its start,
//     y_i = e^{G_i} S0^T c_i + sum_{j<=i} e^{G_i-G_j} (c_i . b_j) x_j
//     S_C = e^{G_C} S0 + sum_j e^{G_C-G_j} b_j x_j^T
// Every exponent that is used is a sum of log_a over a range of steps, so a
// decaying state never divides by a small number.
//
// A sequence's chunks are dealt to `nseg` segments when there are too few
// (batch, head) pairs to fill the GPU: a first kernel runs the state alone
// over each segment from zero, a second joins the segments, and the main
// kernel runs each segment from its true start.
#pragma once

#include "common.cuh"

namespace pdssm {

constexpr int kDecaySMs = 148;          // B200; the segment rule is fixed so that ws sizes are too
constexpr int kDecayMaxW = 128;         // widest N or P
constexpr double kDecayFloor = -200.0;  // exp(-200) is 0 in fp32
constexpr double kLog2e = 1.4426950408889634;

struct DecayParams {
    int B, H, G, rep;                   // rep = H / G heads share one c and b
    int N, P;
    int64_t L;
    int64_t key_t, key_h, key_b;        // element strides of c, b by step, group, batch
    int64_t val_t, val_h, val_b;        // of x, y
    int64_t okey_t, okey_h, okey_b;     // of g_c, g_b
    int64_t oval_t, oval_h, oval_b;     // of y, g_x
    int64_t la_t, la_h, la_b;           // of log_a
    int64_t gla_t, gla_h, gla_b;        // of the per-step g_log_a buffer
    const void *c, *b, *x;
    const float *log_a;
    const float *h0;
    const int32_t *lengths;
    void *y;
    float *h_last;
    const void *g_y;
    const float *g_hlast;
    void *g_c, *g_b, *g_x;              // g_c, g_b: fp32 [B][H][L][N] partials when rep > 1
    float *g_la, *g_h0;
    float *seg_state;                   // [B*H][nseg][N][P]: per segment, local then incoming
    float *seg_decay;                   // [B*H][nseg]
    float *carry;                       // [B*H][nchunks][N][P]: state at every chunk's start
    int *status;                        // the workspace's status word
    int nseg, seg_chunks, nchunks, pslices;
    int vec, ovec;                      // inputs' rows and pointers allow 16-byte accesses; results'
                                        // (2: y by 32 bytes)
    int hold;                           // self-test: the tensor-core forward makes no copies
};

// One step's log decay in base 2, floored (a NaN passes).
__device__ __forceinline__ double decay_log2(float la) {
    double v = (double)la;
    v = v < kDecayFloor ? kDecayFloor : v;
    return v * kLog2e;
}

__device__ __forceinline__ double shfl_up_d(double v, int d) {
    return __shfl_up_sync(kFull, v, d);
}

// Inclusive sums of the C steps' log decays (base 2), by one warp, held as
// hi + lo floats: a difference of two sums then has the error of the
// difference, not of the sums (a chunk may cumulate 64 * 200).
// la(t) gives step t's log decay (0 behind the sequence's end).
template <int C, class LA>
__device__ __forceinline__ void decay_sums(LA la, float2 *G, int lane) {
    double carry = 0.0;
#pragma unroll
    for (int base = 0; base < C; base += 32) {
        double v = decay_log2(la(base + lane));
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const double o = shfl_up_d(v, d);
            if (lane >= d) v += o;
        }
        v += carry;
        carry = __shfl_sync(kFull, v, 31);
        const float hi = (float)v;
        G[base + lane] = make_float2(hi, (float)(v - (double)hi));
    }
}

// 2^(a - b) of two sums
__device__ __forceinline__ float decay_between(float2 a, float2 b) {
    return exp2f((a.x - b.x) + (a.y - b.y));
}
__device__ __forceinline__ float decay_from_start(float2 a) { return exp2f(a.x + a.y); }

// End of sequence b, in steps.
__device__ __forceinline__ int64_t decay_len(const DecayParams &p, int b) {
    if (!p.lengths) return p.L;
    const int64_t n = p.lengths[b];
    return n < 0 ? 0 : (n > p.L ? p.L : n);
}

template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}

// bf16 rows of a width that is not whole 16 bytes, and their padded copy.
struct DecayPad {
    const void *src;
    void *dst;
    int64_t rows;
    int width;
};

// launchers (each returns the launch's error)
cudaError_t launch_decay_join(const DecayParams &p, const float *first, bool reverse,
                              cudaStream_t st);
cudaError_t launch_decay_sum_heads(const DecayParams &p, pdssm_dtype dt, const float *part_c,
                                   const float *part_b, void *g_c, void *g_b, cudaStream_t st);
cudaError_t launch_decay_pad(const DecayPad *t, int count, cudaStream_t st);
cudaError_t launch_decay_unpad(const void *padded, void *out, int64_t rows, int width, cudaStream_t st);
cudaError_t launch_decay_sum_steps(const DecayParams &p, const float *part, float *g_log_a,
                                   cudaStream_t st);
cudaError_t launch_decay_fwd_gen(const DecayParams &p, cudaStream_t st);
cudaError_t launch_decay_bwd_gen(const DecayParams &p, cudaStream_t st);
cudaError_t launch_decay_fwd_tc(const DecayParams &p, cudaStream_t st);
cudaError_t launch_decay_seg_rev_tc(const DecayParams &p, cudaStream_t st);
cudaError_t launch_decay_bwd_mma(const DecayParams &p, cudaStream_t st);
bool decay_tc_copies();                 // the driver's tensor maps are at hand
cudaError_t launch_decay_step(const DecayParams &p, pdssm_dtype dt, float *state, int64_t n_slots,
                              const int32_t *slots, cudaStream_t st);

// Chunk and segments of one direction, from the sizes alone.
struct DecayPlan {
    int chunk, nchunks, nseg, seg_chunks, pslices;
};
DecayPlan decay_plan(const pdssm_decay_dims &d, bool tc, bool adjoint);

}  // namespace pdssm
