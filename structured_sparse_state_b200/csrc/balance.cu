// Balance loss of the hard selection, counts of every dictionary entry, and
// the loss's gradients to the selection input and weights.
//
//     p_t = softmax(inv_tau W u_t),  f_k = counts_k / T,  m_k = mean_t p_t[k]
//     loss = K sum_k f_k m_k
//     g_l_t[k] = g_loss K inv_tau / T p_t[k] (f_k - sum_k' p_t[k'] f_k')
//     g_W = sum_t g_l_t u_t^T,  g_u_t = W^T g_l_t
//
// The logits are recomputed where they are needed: they are H K values per
// step against D_in inputs, so writing them would move more bytes than u.
// Sums over steps go per CTA to scratch and are added in order by a second
// kernel.  bf16 u runs on the tensor cores (balance_tc.cu); fp32 u here, on
// the CUDA cores.
#include "balance.cuh"
#include "launch.cuh"

namespace pdssm {
namespace {

constexpr int kBalThreads = 256;
constexpr int kBalRows = 64;            // steps per tile (four threads per step)

// CTA work over one tile of kBalRows steps: u tile in shared memory (odd row
// length), one head's weights, logits and softmax weights.
template <int KT>
struct Tile {
    float *su, *sW, *sp;                // [64][D|1], [KT][D|1], [64][KT + 1]
    int ld;
    __device__ __forceinline__ Tile(float *sm, int D) {
        ld = D | 1;
        su = sm;
        sW = su + kBalRows * ld;
        sp = sW + KT * ld;
    }
    // a warp per row, its lanes along the row
    __device__ __forceinline__ void load_u(const BalParams &p, int64_t r0) {
        const float *u = (const float *)p.u;
        const int lane = threadIdx.x % 32;
#pragma unroll 4
        for (int r = threadIdx.x / 32; r < kBalRows; r += kBalThreads / 32) {
            const bool live = bal_live(p, r0 + r);
            for (int q = lane; q < p.D; q += 32)
                su[r * ld + q] = live ? u[(r0 + r) * p.D + q] : 0.f;
        }
    }
    __device__ __forceinline__ void load_W(const BalParams &p, int h) {
        const int lane = threadIdx.x % 32;
#pragma unroll 4
        for (int r = threadIdx.x / 32; r < KT; r += kBalThreads / 32)
            for (int q = lane; q < p.D; q += 32)
                sW[r * ld + q] = r < p.K ? p.W[((int64_t)h * p.K + r) * p.D + q] : 0.f;
    }
    // sp = softmax weights of the tile's live rows, zero elsewhere; four
    // threads per row
    __device__ __forceinline__ void softmax(const BalParams &p, int64_t r0) {
        const int r = threadIdx.x / 4, sub = threadIdx.x % 4;
        constexpr int KP = KT / 4;
        float l[KP];
#pragma unroll
        for (int i = 0; i < KP; ++i) l[i] = 0.f;
#pragma unroll 8
        for (int q = 0; q < p.D; ++q) {
            const float uv = su[r * ld + q];
#pragma unroll
            for (int i = 0; i < KP; ++i) l[i] = fmaf(sW[(sub + 4 * i) * ld + q], uv, l[i]);
        }
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < KP; ++i) {
            l[i] = sub + 4 * i < p.K ? l[i] * p.inv_tau : -INFINITY;
            m = fmaxf(m, l[i]);
        }
        m = fmaxf(m, __shfl_xor_sync(kFull, m, 1));
        m = fmaxf(m, __shfl_xor_sync(kFull, m, 2));
        float z = 0.f;
#pragma unroll
        for (int i = 0; i < KP; ++i) {
            l[i] = sub + 4 * i < p.K ? expf(l[i] - m) : 0.f;
            z += l[i];
        }
        z += __shfl_xor_sync(kFull, z, 1);
        z += __shfl_xor_sync(kFull, z, 2);
        const bool live = bal_live(p, r0 + r);
        const float inv = 1.f / z;
#pragma unroll
        for (int i = 0; i < KP; ++i) sp[r * (KT + 1) + sub + 4 * i] = live ? l[i] * inv : 0.f;
    }
    // sp = gradients of the logits, from the softmax weights (same threads)
    __device__ __forceinline__ void grads(const BalParams &p, const float *f, float by) {
        const int r = threadIdx.x / 4, sub = threadIdx.x % 4;
        constexpr int KP = KT / 4;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < KP; ++i) s = fmaf(sp[r * (KT + 1) + sub + 4 * i], f[sub + 4 * i], s);
        s += __shfl_xor_sync(kFull, s, 1);
        s += __shfl_xor_sync(kFull, s, 2);
#pragma unroll
        for (int i = 0; i < KP; ++i) {
            float *v = &sp[r * (KT + 1) + sub + 4 * i];
            *v = by * *v * (f[sub + 4 * i] - s);
        }
    }
};

template <int KT>
constexpr size_t bal_smem(int D) {
    return (size_t)((kBalRows + KT) * (D | 1) + kBalRows * (KT + 1)) * 4;
}

// Sums of p and counts over one slice of the steps of one head.
template <int KT>
__global__ void __launch_bounds__(kBalThreads) k_bal_sums(BalParams p) {
    extern __shared__ float sm[];
    __shared__ int scount[KT];
    const int h = blockIdx.x % p.H, slice = blockIdx.x / p.H;
    Tile<KT> t(sm, p.D);
    t.load_W(p, h);
    if (threadIdx.x < KT) scount[threadIdx.x] = 0;
    float sum = 0.f;                    // column threadIdx.x % KT, rows threadIdx.x / KT ...
    constexpr int RG = kBalThreads / KT;
    for (int64_t r0 = (int64_t)slice * kBalRows; r0 < p.rows; r0 += (int64_t)p.slices * kBalRows) {
        __syncthreads();
        t.load_u(p, r0);
        __syncthreads();
        t.softmax(p, r0);
        if (threadIdx.x < kBalRows && bal_live(p, r0 + threadIdx.x)) {
            const int64_t r = r0 + threadIdx.x, b = r / p.L;
            const int kk = p.k[(b * p.H + h) * p.L + r % p.L];
            if (kk >= 0 && kk < p.K) atomicAdd(&scount[kk], 1);     // integers: any order
        }
        __syncthreads();
        for (int r = threadIdx.x / KT; r < kBalRows; r += RG)
            sum += t.sp[r * (KT + 1) + threadIdx.x % KT];
    }
    __syncthreads();
    t.sp[threadIdx.x] = sum;
    __syncthreads();
    if (threadIdx.x < p.K) {
        float s = 0.f;
        for (int g = 0; g < RG; ++g) s += t.sp[g * KT + threadIdx.x];
        const int64_t at = ((int64_t)slice * p.H + h) * p.K + threadIdx.x;
        p.part[at] = s;
        p.part_n[at] = scount[threadIdx.x];
    }
}

// counts, probs and loss of one head from the slices' sums
__global__ void k_bal_loss(BalParams p, float *loss, int32_t *counts, float *probs) {
    const int h = blockIdx.x, k = threadIdx.x;
    const int64_t T = bal_steps(p);
    const double inv = T > 0 ? 1.0 / (double)T : 0.0;
    double s = 0.0;
    int n = 0;
    if (k < p.K)
        for (int q = 0; q < p.slices; ++q) {
            const int64_t at = ((int64_t)q * p.H + h) * p.K + k;
            s += (double)p.part[at];
            n += p.part_n[at];
        }
    if (k < p.K) {
        counts[h * p.K + k] = n;
        probs[h * p.K + k] = (float)(s * inv);
    }
    double v = k < p.K ? s * inv * ((double)n * inv) : 0.0;
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
    if (k == 0) loss[h] = (float)(v * p.K);
}

// g_u of one tile of steps over heads h0 .. h1 - 1: thread (ty, tx) owns rows
// ty + 16 i and columns tx + 16 j.  A head takes about 10 us, most of it the
// latency of its phases, so where the tiles do not fill the GPU the heads are
// split over CTAs too, whose sums k_bal_gu_sum adds in order (one step, 16
// heads of 32 entries: GUSPLIT us for the whole loss and its gradients, by one
// CTA 190).
template <int KT>
__global__ void __launch_bounds__(kBalThreads) k_bal_gu(BalParams p) {
    extern __shared__ float sm[];
    __shared__ float f[KT];
    Tile<KT> t(sm, p.D);
    const int64_t r0 = (int64_t)(blockIdx.x / p.hslices) * kBalRows;
    const int hs = blockIdx.x % p.hslices;
    const int h0 = (int)((int64_t)p.H * hs / p.hslices), h1 = (int)((int64_t)p.H * (hs + 1) / p.hslices);
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    const int64_t steps = bal_steps(p);
    const float inv = steps > 0 ? 1.f / (float)steps : 0.f;
    float acc[4][kBalMaxD / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < kBalMaxD / 16; ++j) acc[i][j] = 0.f;
    t.load_u(p, r0);
    for (int h = h0; h < h1; ++h) {
        __syncthreads();
        t.load_W(p, h);
        if (threadIdx.x < KT)
            f[threadIdx.x] = threadIdx.x < p.K ? (float)p.counts[h * p.K + threadIdx.x] * inv : 0.f;
        __syncthreads();
        t.softmax(p, r0);
        t.grads(p, f, p.g_loss[h] * ((float)p.K * p.inv_tau) * inv);
        __syncthreads();
        for (int k = 0; k < KT; ++k) {
            float g[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) g[i] = t.sp[(ty + 16 * i) * (KT + 1) + k];
#pragma unroll
            for (int j = 0; j < kBalMaxD / 16; ++j) {
                const int q = tx + 16 * j;
                if (q >= p.D) break;
                const float w = t.sW[k * t.ld + q];
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i][j] = fmaf(g[i], w, acc[i][j]);
            }
        }
    }
    float *gu = p.hslices > 1 ? p.part + hs * p.rows * p.D : (float *)p.g_u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = r0 + ty + 16 * i;
        if (r >= p.rows) continue;
#pragma unroll
        for (int j = 0; j < kBalMaxD / 16; ++j) {
            const int q = tx + 16 * j;
            if (q >= p.D) break;
            gu[r * p.D + q] = acc[i][j];
        }
    }
}

__global__ void k_bal_gu_sum(BalParams p) {
    const int64_t n = p.rows * p.D;
    for (int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; e < n;
         e += (int64_t)gridDim.x * blockDim.x) {
        float s = 0.f;
        for (int q = 0; q < p.hslices; ++q) s += p.part[q * n + e];
        ((float *)p.g_u)[e] = s;
    }
}

// g_W of one head over one slice of the steps
template <int KT>
__global__ void __launch_bounds__(kBalThreads) k_bal_gw(BalParams p) {
    extern __shared__ float sm[];
    __shared__ float f[KT];
    Tile<KT> t(sm, p.D);
    const int h = blockIdx.x % p.H, slice = blockIdx.x / p.H;
    const int64_t steps = bal_steps(p);
    const float inv = steps > 0 ? 1.f / (float)steps : 0.f;
    constexpr int KP = KT / 8;          // thread (kr, c): entries kr + 8 i, columns c + 32 j
    const int kr = threadIdx.x / 32, c = threadIdx.x % 32;
    float acc[KP][kBalMaxD / 32];
#pragma unroll
    for (int i = 0; i < KP; ++i)
#pragma unroll
        for (int j = 0; j < kBalMaxD / 32; ++j) acc[i][j] = 0.f;
    t.load_W(p, h);
    if (threadIdx.x < KT)
        f[threadIdx.x] = threadIdx.x < p.K ? (float)p.counts[h * p.K + threadIdx.x] * inv : 0.f;
    const float by = p.g_loss[h] * ((float)p.K * p.inv_tau) * inv;
    for (int64_t r0 = (int64_t)slice * kBalRows; r0 < p.rows; r0 += (int64_t)p.slices * kBalRows) {
        __syncthreads();
        t.load_u(p, r0);
        __syncthreads();
        t.softmax(p, r0);
        t.grads(p, f, by);
        __syncthreads();
        for (int r = 0; r < kBalRows; ++r) {
            float g[KP];
#pragma unroll
            for (int i = 0; i < KP; ++i) g[i] = t.sp[r * (KT + 1) + kr + 8 * i];
#pragma unroll
            for (int j = 0; j < kBalMaxD / 32; ++j) {
                if (c + 32 * j >= p.D) break;
                const float uv = t.su[r * t.ld + c + 32 * j];
#pragma unroll
                for (int i = 0; i < KP; ++i) acc[i][j] = fmaf(g[i], uv, acc[i][j]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < KP; ++i)
#pragma unroll
        for (int j = 0; j < kBalMaxD / 32; ++j)
            if (kr + 8 * i < p.K && c + 32 * j < p.D)
                p.part[(((int64_t)slice * p.H + h) * p.K + kr + 8 * i) * p.D + c + 32 * j] =
                    acc[i][j];
}

// g_W: the slices' sums in order
__global__ void k_bal_gw_sum(BalParams p, float *g_W) {
    const int64_t n = (int64_t)p.H * p.K * p.D;
    const int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (e >= n) return;
    float s = 0.f;
    for (int q = 0; q < p.slices; ++q) s += p.part[q * n + e];
    g_W[e] = s;
}

// slices of the steps per head: fill the GPU, at least one tile each
int bal_slices(int64_t rows, int64_t H) {
    const int64_t tiles = (rows + kBalRows - 1) / kBalRows;
    int64_t n = (148 * 4 + H - 1) / H;
    if (n > tiles) n = tiles;
    return (int)(n < 1 ? 1 : n);
}

// slices of the heads for fp32 g_u: as many as the GPU takes beside the tiles
int bal_hslices(int64_t rows, int64_t H) {
    const int64_t tiles = (rows + kBalRows - 1) / kBalRows;
    const int64_t n = tiles > 0 ? 148 / tiles : 1;
    return (int)(n < 1 ? 1 : n > H ? H : n);
}

template <void (*KERN)(BalParams)>
cudaError_t launch(int64_t grid, size_t smem, cudaStream_t st, const BalParams &p) {
    static std::atomic<int> set[kLimitDevices];
    const cudaError_t e = allow_smem((const void *)KERN, (int)smem, set);
    if (e != cudaSuccess) return e;
    KERN<<<dim3((unsigned)grid), kBalThreads, smem, st>>>(p);
    return cudaGetLastError();
}

template <int KT>
cudaError_t run(const BalParams &p, int what, cudaStream_t st) {
    const size_t smem = bal_smem<KT>(p.D);
    if (what == 0) return launch<k_bal_sums<KT>>((int64_t)p.H * p.slices, smem, st, p);
    if (what == 1) {
        const int64_t tiles = (p.rows + kBalRows - 1) / kBalRows;
        const cudaError_t e = launch<k_bal_gu<KT>>(tiles * p.hslices, smem, st, p);
        if (e != cudaSuccess || p.hslices == 1) return e;
        k_bal_gu_sum<<<(unsigned)((p.rows * p.D + 255) / 256), 256, 0, st>>>(p);
        return cudaGetLastError();
    }
    return launch<k_bal_gw<KT>>((int64_t)p.H * p.slices, smem, st, p);
}

cudaError_t run_k(const BalParams &p, int what, cudaStream_t st) {
    if (p.K <= 8) return run<8>(p, what, st);
    if (p.K <= 16) return run<16>(p, what, st);
    return run<32>(p, what, st);
}

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

pdssm_status check_bal(const pdssm_dims *d) {
    if (!d) return arg_fail(PDSSM_ERR_INVALID_ARG, "dims is NULL");
    if (d->B < 1 || d->H < 1 || d->L < 0 || d->K < 1 || d->D_in < 1)
        return arg_fail(PDSSM_ERR_INVALID_ARG, "need B, H, K, D_in >= 1 and L >= 0");
    if (d->K > kBalMaxK || d->D_in > kBalMaxD)
        return arg_fail(PDSSM_ERR_UNSUPPORTED, "K > 32 or D_in > 256");
    const int64_t most = 0x7fffffff;
    if (d->B > most || d->L > most || d->B * d->L > most || d->H > 65536 ||
        d->B * d->L > ((int64_t)1 << 40) / d->H)
        return arg_fail(PDSSM_ERR_UNSUPPORTED, "B*L >= 2^31 or H too large");
    return PDSSM_OK;
}

// partial sums of g_W, or of p with the counts
size_t bal_partials(const pdssm_dims &d, int slices) {
    return align256((size_t)slices * (size_t)(d.H * d.K) * (size_t)(d.D_in > 2 ? d.D_in : 2) * 4);
}

size_t bal_scratch(const pdssm_dims &d) {
    const BalTcPlan pl = bal_tc_plan(d);
    const size_t a = bal_partials(d, bal_slices(d.B * d.L, d.H));
    const size_t b = bal_partials(d, pl.slices) + bal_tc_extra(pl);
    const int hs = bal_hslices(d.B * d.L, d.H);
    const size_t c = hs > 1 ? (size_t)hs * (size_t)(d.B * d.L * d.D_in) * 4 : 0;
    return a > b ? (a > c ? a : c) : (b > c ? b : c);
}

pdssm_status bal_common(const pdssm_dims *d, const void *u, pdssm_dtype dt, const float *W,
                        float inv_tau, const int32_t *lengths, void *scratch, size_t bytes,
                        BalParams *p) {
    pdssm_status st = check_bal(d);
    if (st != PDSSM_OK) return st;
    if (dt != PDSSM_F32 && dt != PDSSM_BF16)
        return arg_fail(PDSSM_ERR_INVALID_ARG, "unknown dtype");
    if (!(inv_tau > 0.f) || inv_tau > 3.0e38f)
        return arg_fail(PDSSM_ERR_INVALID_ARG, "inv_tau must be positive and finite");
    if (!W || (d->L > 0 && !u)) return arg_fail(PDSSM_ERR_INVALID_ARG, "NULL u or W_sel");
    if (!scratch || !aligned(scratch, 256))
        return arg_fail(PDSSM_ERR_INVALID_ARG, "scratch NULL or not 256-byte aligned");
    if (bytes < bal_scratch(*d)) return arg_fail(PDSSM_ERR_WORKSPACE, "scratch too small");
    BalParams q{};
    q.B = (int)d->B; q.H = (int)d->H; q.K = (int)d->K; q.D = (int)d->D_in;
    q.L = d->L; q.rows = d->B * d->L;
    q.u = u; q.W = W; q.lengths = lengths; q.inv_tau = inv_tau;
    q.slices = dt == PDSSM_BF16 ? bal_tc_plan(*d).slices : bal_slices(q.rows, d->H);
    q.hslices = bal_hslices(q.rows, d->H);
    q.part = (float *)scratch;
    q.part_n = (int32_t *)(q.part + (int64_t)q.slices * q.H * q.K);
    *p = q;
    return PDSSM_OK;
}

// fp32 on the CUDA cores, bf16 on the tensor cores (which keep W's parts
// behind the partial sums in scratch)
cudaError_t run_any(const pdssm_dims &d, const BalParams &p, pdssm_dtype dt, int what,
                    cudaStream_t st) {
    if (dt != PDSSM_BF16) return run_k(p, what, st);
    const BalTcPlan pl = bal_tc_plan(d);
    unsigned char *parts = reinterpret_cast<unsigned char *>(p.part) + bal_partials(d, pl.slices);
    if (what == 0 || what == 1 || !p.g_u) {
        const cudaError_t e = launch_bal_tc_prep(p, pl, parts, st);
        if (e != cudaSuccess) return e;
    }
    return launch_bal_tc(p, pl, what, parts, st);
}

}  // namespace
}  // namespace pdssm

using namespace pdssm;

extern "C" {

size_t pdssm_select_balance_scratch_bytes(const pdssm_dims *dims) {
    if (check_bal(dims) != PDSSM_OK) return 0;
    return bal_scratch(*dims);
}

pdssm_status pdssm_select_balance_fwd(const pdssm_dims *dims, const void *u, pdssm_dtype u_dtype,
                                      const float *W_sel, const int32_t *k, float inv_tau,
                                      const int32_t *lengths, float *loss, int32_t *counts,
                                      float *probs, void *scratch, size_t scratch_bytes,
                                      void *stream) {
    BalParams p;
    pdssm_status st = bal_common(dims, u, u_dtype, W_sel, inv_tau, lengths, scratch, scratch_bytes, &p);
    if (st != PDSSM_OK) return st;
    if (!loss || !counts || !probs || (dims->L > 0 && !k))
        return arg_fail(PDSSM_ERR_INVALID_ARG, "NULL k, loss, counts or probs");
    p.k = k;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e = run_any(*dims, p, u_dtype, 0, s);
    if (e != cudaSuccess) return cuda_fail(e, "balance sums");
    k_bal_loss<<<p.H, 32, 0, s>>>(p, loss, counts, probs);
    e = cudaGetLastError();
    return e == cudaSuccess ? PDSSM_OK : cuda_fail(e, "balance loss");
}

pdssm_status pdssm_select_balance_bwd(const pdssm_dims *dims, const void *u, pdssm_dtype u_dtype,
                                      const float *W_sel, const int32_t *counts, float inv_tau,
                                      const int32_t *lengths, const float *g_loss, void *g_u,
                                      float *g_W, void *scratch, size_t scratch_bytes,
                                      void *stream) {
    BalParams p;
    pdssm_status st = bal_common(dims, u, u_dtype, W_sel, inv_tau, lengths, scratch, scratch_bytes, &p);
    if (st != PDSSM_OK) return st;
    if (!counts || !g_loss) return arg_fail(PDSSM_ERR_INVALID_ARG, "NULL counts or g_loss");
    p.counts = counts;
    p.g_loss = g_loss;
    p.g_u = g_u;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (g_u && p.rows > 0) {
        e = run_any(*dims, p, u_dtype, 1, s);
        if (e != cudaSuccess) return cuda_fail(e, "balance g_u");
    }
    if (g_W) {
        e = run_any(*dims, p, u_dtype, 2, s);
        if (e != cudaSuccess) return cuda_fail(e, "balance g_W");
        const int64_t n = (int64_t)p.H * p.K * p.D;
        k_bal_gw_sum<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(p, g_W);
        e = cudaGetLastError();
        if (e != cudaSuccess) return cuda_fail(e, "balance g_W sum");
    }
    return PDSSM_OK;
}

}  // extern "C"
