// One step of the decay scan for single tokens:
//     S = a S + b x^T,  y = S^T c      per (batch row, head), S in a slot.
//
// Bound: HBM, one read and one write of the fp32 state (2 * 4 * N * P bytes
// per head against 2 N + 2 P narrow inputs).  One CTA per batch row and a few
// heads (as many as hold 4096 values): a group of P / 4 threads takes a state
// row by 16-byte loads, each head has its share of the groups, which take the
// head's rows in turn, and y is summed over them in shared memory in a fixed
// order.  The first loads of the state and of the small inputs are issued as
// soon as the slot is known, ahead of the search for it in earlier rows.
// Loads and stores of the state are marked as streaming and a thread keeps
// four rows in flight: 256 rows of 16 heads of 64 x 64 (134 MB) take 28.7 us,
// 4.8 TB/s; eight rows in flight 30.8, without the marks 32 to 37.
#include "decay.cuh"

namespace pdssm {
namespace {

constexpr int kStepThreads = 128;
constexpr int kStepIn = 512;            // entries of b, of c and of x in a CTA

// VW floats per access; RPT state rows of one thread in flight
template <typename T, int VW, int RPT>
__global__ void __launch_bounds__(kStepThreads) k_decay_step(DecayParams p, float *state,
                                                             int64_t n_slots,
                                                             const int32_t *slots, int hpc) {
    __shared__ float sb[kStepIn], sc[kStepIn], sx[kStepIn];
    __shared__ float sy[kStepThreads * VW];
    const int hgroups = (p.H + hpc - 1) / hpc;
    const int h0 = blockIdx.x % hgroups * hpc, nh = min(hpc, p.H - h0);
    const int64_t row = blockIdx.x / hgroups;
    const int tid = threadIdx.x;
    const int64_t slot = slots ? (int64_t)slots[row] : row;
    bool bad = slot < 0 || slot >= n_slots;

    const int cols = p.P / VW;                      // accesses per state row
    const int groups = kStepThreads / cols / hpc;   // rows of a head at once
    const int hg = tid / cols / groups, h = h0 + hg;
    const int g = tid / cols % groups, q = (tid % cols) * VW;
    const bool on = hg < nh;
    float *S = state + (slot * p.H + h) * p.N * p.P + q;
    float s[RPT][VW];
    auto load = [&](int n0) {
#pragma unroll
        for (int r = 0; r < RPT; ++r) {
            const int n = n0 + r * groups;
            if (n >= p.N) continue;
            if constexpr (VW == 4) {
                const float4 t = __ldcs(reinterpret_cast<const float4 *>(S + (int64_t)n * p.P));
                s[r][0] = t.x; s[r][1] = t.y; s[r][2] = t.z; s[r][3] = t.w;
            } else {
                s[r][0] = S[(int64_t)n * p.P];
            }
        }
    };
    if (on && !bad) load(g);

    float a = 0.f;
    if (on) {
        const float la = p.log_a[row * p.la_b + h * p.la_h];
        a = expf(la < (float)kDecayFloor ? (float)kDecayFloor : la);
    }
    for (int i = tid; i < nh * p.N; i += kStepThreads) {
        const int64_t o = (row * p.G + (h0 + i / p.N) / p.rep) * p.N + i % p.N;
        sb[i] = to_f<T>(((const T *)p.b)[o]);
        sc[i] = to_f<T>(((const T *)p.c)[o]);
    }
    const int64_t voff = (row * p.H + h0) * p.P;
    for (int i = tid; i < nh * p.P; i += kStepThreads) sx[i] = to_f<T>(((const T *)p.x)[voff + i]);

    // a slot outside the pool, or one that an earlier row uses: an empty row
    if (slots) {
        int64_t r = 0;
        if (((uintptr_t)slots & 15) == 0) {         // four at a time
            const int4 *s4 = reinterpret_cast<const int4 *>(slots);
            for (int64_t i = tid; i < row / 4; i += kStepThreads) {
                const int4 v = __ldg(s4 + i);
                bad |= v.x == (int)slot || v.y == (int)slot || v.z == (int)slot || v.w == (int)slot;
            }
            r = row / 4 * 4;
        }
        for (r += tid; r < row; r += kStepThreads) bad |= slots[r] == (int32_t)slot;
    }
    T *y = (T *)p.y + voff;
    if (__syncthreads_or(bad)) {
        for (int i = tid; i < nh * p.P; i += kStepThreads) y[i] = from_f<T>(0.f);
        return;
    }
    if (on) {
        const float *bh = sb + hg * p.N, *ch = sc + hg * p.N;
        float acc[VW], xv[VW];
#pragma unroll
        for (int v = 0; v < VW; ++v) acc[v] = 0.f, xv[v] = sx[hg * p.P + q + v];
        for (int n0 = g; n0 < p.N; n0 += groups * RPT) {
            if (n0 > g) load(n0);
#pragma unroll
            for (int r = 0; r < RPT; ++r) {
                const int n = n0 + r * groups;
                if (n >= p.N) continue;
                const float bn = bh[n], cn = ch[n];
#pragma unroll
                for (int v = 0; v < VW; ++v) {
                    s[r][v] = fmaf(a, s[r][v], bn * xv[v]);
                    acc[v] = fmaf(cn, s[r][v], acc[v]);
                }
                if constexpr (VW == 4)
                    __stcs(reinterpret_cast<float4 *>(S + (int64_t)n * p.P),
                           make_float4(s[r][0], s[r][1], s[r][2], s[r][3]));
                else
                    S[(int64_t)n * p.P] = s[r][0];
            }
        }
#pragma unroll
        for (int v = 0; v < VW; ++v) sy[(hg * groups + g) * p.P + q + v] = acc[v];
    }
    __syncthreads();
    for (int o = tid; o < nh * p.P; o += kStepThreads) {
        const float *part = sy + o / p.P * groups * p.P + o % p.P;
        float t = 0.f;
        for (int r = 0; r < groups; ++r) t += part[r * p.P];
        y[o] = from_f<T>(t);
    }
}

template <typename T>
cudaError_t go(const DecayParams &p, float *state, int64_t n_slots, const int32_t *slots,
               cudaStream_t st) {
    // heads of a CTA: 4096 state values, at least one group of threads each
    const int w = p.N > p.P ? p.N : p.P, groups = kStepThreads / (p.P / (p.vec ? 4 : 1));
    int hpc = 4096 / (p.N * p.P);
    hpc = hpc < groups ? hpc : groups;
    hpc = hpc < kStepIn / w ? hpc : kStepIn / w;
    hpc = hpc < p.H ? hpc : p.H;
    hpc = hpc < 1 ? 1 : hpc;
    const unsigned grid = (unsigned)((int64_t)p.B * ((p.H + hpc - 1) / hpc));
    if (p.vec)
        k_decay_step<T, 4, 4><<<grid, kStepThreads, 0, st>>>(p, state, n_slots, slots, hpc);
    else
        k_decay_step<T, 1, 8><<<grid, kStepThreads, 0, st>>>(p, state, n_slots, slots, hpc);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decay_step(const DecayParams &p, pdssm_dtype dt, float *state, int64_t n_slots,
                              const int32_t *slots, cudaStream_t st) {
    return dt == PDSSM_BF16 ? go<__nv_bfloat16>(p, state, n_slots, slots, st)
                            : go<float>(p, state, n_slots, slots, st);
}

}  // namespace pdssm
