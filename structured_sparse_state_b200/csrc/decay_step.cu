// One step of the decay scan for single tokens:
//     S = a S + b x^T,  y = S^T c      per (batch row, head), S in a slot.
//
// Bound: HBM, one read and one write of the fp32 state (2 * 4 * N * P bytes
// per head against 2 N + 2 P narrow inputs).  One CTA per (row, head): a
// group of P / 4 threads takes a state row by 16-byte loads, the groups take
// rows in turn, and y is summed over the groups in shared memory in a fixed
// order.  All of a CTA's loads are issued before the first is used.
#include "decay.cuh"

namespace pdssm {
namespace {

constexpr int kStepThreads = 128;

// VW floats per access; RPT state rows of one thread in flight
template <typename T, int VW, int RPT>
__global__ void __launch_bounds__(kStepThreads) k_decay_step(DecayParams p, float *state,
                                                             int64_t n_slots,
                                                             const int32_t *slots) {
    __shared__ float sk[2 * kDecayMaxW];
    __shared__ float sx[kDecayMaxW];
    __shared__ float sy[kStepThreads * VW];
    const int h = blockIdx.x % p.H;
    const int64_t row = blockIdx.x / p.H;
    const int tid = threadIdx.x;
    const int64_t slot = slots ? (int64_t)slots[row] : row;
    const int64_t koff = (row * p.G + h / p.rep) * p.N, voff = (row * p.H + h) * p.P;
    T *y = (T *)p.y + voff;

    // a slot outside the pool, or one that an earlier row uses: an empty row
    bool bad = slot < 0 || slot >= n_slots;
    if (slots) {
        int64_t r = 0;
        if (((uintptr_t)slots & 15) == 0) {         // four at a time
            const int4 *s4 = reinterpret_cast<const int4 *>(slots);
            for (int64_t q = tid; q < row / 4; q += kStepThreads) {
                const int4 v = __ldg(s4 + q);
                bad |= v.x == (int)slot || v.y == (int)slot || v.z == (int)slot || v.w == (int)slot;
            }
            r = row / 4 * 4;
        }
        for (r += tid; r < row; r += kStepThreads) bad |= slots[r] == (int32_t)slot;
    }
    if (__syncthreads_or(bad)) {
        for (int q = tid; q < p.P; q += kStepThreads) y[q] = from_f<T>(0.f);
        return;
    }
    const float la = p.log_a[row * p.la_b + h * p.la_h];
    const float a = expf(la < (float)kDecayFloor ? (float)kDecayFloor : la);
    for (int n = tid; n < p.N; n += kStepThreads) {
        sk[n] = to_f<T>(((const T *)p.b)[koff + n]);
        sk[kDecayMaxW + n] = to_f<T>(((const T *)p.c)[koff + n]);
    }
    for (int q = tid; q < p.P; q += kStepThreads) sx[q] = to_f<T>(((const T *)p.x)[voff + q]);
    __syncthreads();

    const int cols = p.P / VW;                  // accesses per state row
    const int groups = kStepThreads / cols;     // state rows at once
    const int g = tid / cols, q = (tid % cols) * VW;
    float acc[VW];
#pragma unroll
    for (int v = 0; v < VW; ++v) acc[v] = 0.f;
    if (g < groups) {
        float *S = state + (slot * p.H + h) * p.N * p.P + q;
        for (int n0 = g; n0 < p.N; n0 += groups * RPT) {
            float s[RPT][VW];
#pragma unroll
            for (int r = 0; r < RPT; ++r) {
                const int n = n0 + r * groups;
                if (n >= p.N) continue;
                if constexpr (VW == 4) {
                    const float4 t = *reinterpret_cast<const float4 *>(S + (int64_t)n * p.P);
                    s[r][0] = t.x; s[r][1] = t.y; s[r][2] = t.z; s[r][3] = t.w;
                } else {
                    s[r][0] = S[(int64_t)n * p.P];
                }
            }
#pragma unroll
            for (int r = 0; r < RPT; ++r) {
                const int n = n0 + r * groups;
                if (n >= p.N) continue;
                const float bn = sk[n], cn = sk[kDecayMaxW + n];
#pragma unroll
                for (int v = 0; v < VW; ++v) {
                    s[r][v] = fmaf(a, s[r][v], bn * sx[q + v]);
                    acc[v] = fmaf(cn, s[r][v], acc[v]);
                }
                if constexpr (VW == 4)
                    *reinterpret_cast<float4 *>(S + (int64_t)n * p.P) =
                        make_float4(s[r][0], s[r][1], s[r][2], s[r][3]);
                else
                    S[(int64_t)n * p.P] = s[r][0];
            }
        }
#pragma unroll
        for (int v = 0; v < VW; ++v) sy[g * p.P + q + v] = acc[v];
    }
    __syncthreads();
    for (int o = tid; o < p.P; o += kStepThreads) {
        float s = 0.f;
        for (int r = 0; r < groups; ++r) s += sy[r * p.P + o];
        y[o] = from_f<T>(s);
    }
}

template <typename T>
cudaError_t go(const DecayParams &p, float *state, int64_t n_slots, const int32_t *slots,
               cudaStream_t st) {
    const unsigned grid = (unsigned)((int64_t)p.B * p.H);
    if (p.vec)
        k_decay_step<T, 4, 8><<<grid, kStepThreads, 0, st>>>(p, state, n_slots, slots);
    else
        k_decay_step<T, 1, 8><<<grid, kStepThreads, 0, st>>>(p, state, n_slots, slots);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decay_step(const DecayParams &p, pdssm_dtype dt, float *state, int64_t n_slots,
                              const int32_t *slots, cudaStream_t st) {
    return dt == PDSSM_BF16 ? go<__nv_bfloat16>(p, state, n_slots, slots, st)
                            : go<float>(p, state, n_slots, slots, st);
}

}  // namespace pdssm
