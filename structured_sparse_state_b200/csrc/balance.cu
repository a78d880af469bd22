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
#include "tile_mm.cuh"

namespace pdssm {
namespace {

constexpr int kBalThreads = 256;        // 16 x 16
constexpr int kBalRows = 64;            // steps per tile

// Entries per group (whole heads): 64, or 32 where all the heads have no more
// (4 x 9607 steps, 8 heads of 4, D = 256: 212 us, with 64 314; 16 heads of 16:
// 1029 us, with 64 937).
int bal_cols(int H, int K) { return H * K <= 32 ? 32 : 64; }
int bal_heads(int H, int K) { return bal_cols(H, K) / K; }
int bal_groups(int H, int K) {
    const int n = bal_heads(H, K);
    return (H + n - 1) / n;
}

// A CTA's work on one tile of steps and one group of heads in fp32: u and W
// rows in shared memory, the logits (then softmax weights, then gradients) of
// 64 steps x EC entries beside them.  Per 4 of D a thread reads eight 16-byte
// pieces for 64 multiply-adds (EC = 32: six for 32), which leaves the logits to
// the FFMA units, not to shared memory.  8 x 4096 steps, 16 heads of 16, D = 128:
// loss and gradients in 378 us, 28 TFLOP/s; the softmax and the barriers around
// it, and the 16-byte rows of the other products, keep it below the units' 70.
template <int EC>
struct Tile {
    static constexpr int kLdP = EC + 2;
    float *su, *sW, *sp;                // [64][ld], [EC][ld], [64][kLdP]
    int *live;                          // [64]
    int ld, Dp;
    __device__ __forceinline__ Tile(float *sm, int D) {
        Dp = (D + 7) / 8 * 8;
        ld = Dp + 4;                    // an odd number of 16-byte pieces
        su = sm;
        sW = su + kBalRows * ld;
        sp = sW + EC * ld;
        live = reinterpret_cast<int *>(sp + kBalRows * kLdP);
    }
    // rows of D values, on their way to shared memory; zero where on(r) is false
    template <int ROWS, class ON>
    __device__ __forceinline__ void load(float *dst, const float *src, int D, bool vec, ON on) const {
        const uint32_t to = smem_u32(dst);
        if (vec) {
            const int pieces = Dp / 4;
            for (int i = threadIdx.x; i < ROWS * pieces; i += kBalThreads) {
                const int r = i / pieces, q = 4 * (i - r * pieces);
                const bool in = q < D && on(r);
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + 4u * (r * ld + q)),
                             "l"(in ? src + (int64_t)r * D + q : src), "r"(in ? 16 : 0)
                             : "memory");
            }
        } else {
            for (int i = threadIdx.x; i < ROWS * Dp; i += kBalThreads) {
                const int r = i / Dp, q = i - r * Dp;
                const bool in = q < D && on(r);
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to + 4u * (r * ld + q)),
                             "l"(in ? src + (int64_t)r * D + q : src), "r"(in ? 4 : 0)
                             : "memory");
            }
        }
    }
    __device__ __forceinline__ void load_u(const BalParams &p, int64_t r0) const {
        if (threadIdx.x < kBalRows) live[threadIdx.x] = bal_live(p, r0 + threadIdx.x);
        load<kBalRows>(su, (const float *)p.u + r0 * p.D, p.D, p.vec, [&](int r) { return bal_live(p, r0 + r); });
    }
    __device__ __forceinline__ void load_W(const BalParams &p, int e0, int ne) const {
        load<EC>(sW, p.W + (int64_t)e0 * p.D, p.D, p.vec, [&](int r) { return r < ne; });
    }
    __device__ __forceinline__ void landed() const {
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
    }
    // sp = inv_tau u W^T; a barrier follows
    __device__ __forceinline__ void logits(const BalParams &p) const {
        const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
        float acc[4][EC / 16];
        zero(acc);
        tile_mm(acc, Dp, Along<4, false>{su, ld, ty}, Along<EC / 16, false>{sW, ld, tx});
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < EC / 16; ++j)
                sp[strided(ty, i) * kLdP + strided(tx, j)] = acc[i][j] * p.inv_tau;
        __syncthreads();
    }
    // per (step, head): sp = softmax weights, zero behind the lengths; with GRAD
    // the logits' gradients instead.  A barrier follows.
    template <bool GRAD>
    __device__ __forceinline__ void softmax(const BalParams &p, int nh, const float *f,
                                            const float *by) const {
        for (int i = threadIdx.x; i < kBalRows * nh; i += kBalThreads) {
            const int r = i % kBalRows, hh = i / kBalRows;
            float *x = sp + r * kLdP + hh * p.K;
            const float *fh = f + hh * p.K;
            float m = x[0];
            for (int k = 1; k < p.K; ++k) m = fmaxf(m, x[k]);
            float z = 0.f, s = 0.f;
            for (int k = 0; k < p.K; ++k) {
                const float v = expf(x[k] - m);
                x[k] = v;
                z += v;
                if (GRAD) s = fmaf(v, fh[k], s);
            }
            const float inv = 1.f / z;
            for (int k = 0; k < p.K; ++k)
                x[k] = !live[r] ? 0.f : GRAD ? by[hh] * (x[k] * inv) * (fh[k] - s * inv) : x[k] * inv;
        }
        __syncthreads();
    }
};

size_t bal_smem(int D, int cols) {
    return (size_t)((kBalRows + cols) * ((D + 7) / 8 * 8 + 4) + kBalRows * (cols + 2) + kBalRows) * 4;
}

// Sums of p and counts over one slice of the steps of one group of heads.
template <int EC>
__global__ void __launch_bounds__(kBalThreads) k_bal_sums(BalParams p) {
    extern __shared__ float sm[];
    __shared__ int scount[EC];
    const Tile<EC> t(sm, p.D);
    const int group = blockIdx.x % p.groups, slice = blockIdx.x / p.groups;
    const int h0 = group * p.heads, nh = min(p.heads, p.H - h0), e0 = h0 * p.K, ne = nh * p.K;
    constexpr int RG = kBalThreads / EC;
    const int col = threadIdx.x % EC, rg = threadIdx.x / EC;
    t.load_W(p, e0, ne);
    if (threadIdx.x < EC) scount[threadIdx.x] = 0;
    float sum = 0.f;                    // column col, rows rg, rg + RG, ..
    for (int64_t r0 = (int64_t)slice * kBalRows; r0 < p.rows; r0 += (int64_t)p.slices * kBalRows) {
        __syncthreads();
        t.load_u(p, r0);
        t.landed();
        t.logits(p);
        t.template softmax<false>(p, nh, nullptr, nullptr);
        for (int i = threadIdx.x; i < kBalRows * nh; i += kBalThreads) {
            const int hh = i / kBalRows;
            const uint32_t r = (uint32_t)r0 + i % kBalRows;
            if (!t.live[i % kBalRows]) continue;
            const uint32_t b = r / (uint32_t)p.L;
            const int kk = p.k[((int64_t)b * p.H + h0 + hh) * p.L + (r - b * (uint32_t)p.L)];
            if (kk >= 0 && kk < p.K) atomicAdd(&scount[hh * p.K + kk], 1);      // integers: any order
        }
#pragma unroll
        for (int r = 0; r < kBalRows / RG; ++r) sum += t.sp[(RG * r + rg) * t.kLdP + col];
    }
    t.landed();                         // also where there was no tile
    t.sp[threadIdx.x] = sum;
    __syncthreads();
    if (threadIdx.x < ne) {
        const int64_t at = (int64_t)slice * p.H * p.K + e0 + threadIdx.x;
        float total = 0.f;
        for (int q = 0; q < RG; ++q) total += t.sp[q * EC + col];
        p.part[at] = total;
        p.part_n[at] = scount[threadIdx.x];
    }
}

// Steps in front of the lengths, once for all the kernels that divide by them
// (every thread added up all the lengths by itself before: 16 heads of 16, D =
// 128, 4096 sequences of up to 32 steps, loss and gradients: fp32 6118 -> 1409 us,
// bf16 414 -> 216).
constexpr int kStepThreads = 1024;
__global__ void __launch_bounds__(kStepThreads) k_bal_steps(BalParams p, int64_t *steps) {
    __shared__ int64_t sums[kStepThreads / 32];
    int64_t n = 0;
#pragma unroll 8
    for (int b = threadIdx.x; b < p.B; b += kStepThreads) n += bal_len(p, b);
#pragma unroll
    for (int d = 16; d; d >>= 1) n += __shfl_xor_sync(kFull, n, d);
    if (threadIdx.x % 32 == 0) sums[threadIdx.x / 32] = n;
    __syncthreads();
    if (threadIdx.x) return;
    for (int w = 1; w < kStepThreads / 32; ++w) n += sums[w];
    *steps = n;
}

// counts, probs and loss of one head from the slices' sums: a warp takes every
// kSumWays-th slice, and the warps' sums are added in order
constexpr int kSumWays = 8;
__global__ void __launch_bounds__(32 * kSumWays) k_bal_loss(BalParams p, float *loss, int32_t *counts,
                                                            float *probs) {
    __shared__ double sums[kSumWays][32];
    __shared__ int ns[kSumWays][32];
    const int h = blockIdx.x, k = threadIdx.x % 32, way = threadIdx.x / 32;
    double s = 0.0;
    int n = 0;
    if (k < p.K)
        for (int q = way; q < p.slices; q += kSumWays) {
            const int64_t at = ((int64_t)q * p.H + h) * p.K + k;
            s += (double)p.part[at];
            n += p.part_n[at];
        }
    sums[way][k] = s;
    ns[way][k] = n;
    __syncthreads();
    if (way) return;
    for (int w = 1; w < kSumWays; ++w) {
        s += sums[w][k];
        n += ns[w][k];
    }
    const int64_t T = bal_steps(p);
    const double inv = T > 0 ? 1.0 / (double)T : 0.0;
    if (k < p.K) {
        counts[h * p.K + k] = n;
        probs[h * p.K + k] = (float)(s * inv);
    }
    double v = k < p.K ? s * inv * ((double)n * inv) : 0.0;
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
    if (k == 0) loss[h] = (float)(v * p.K);
}

// what the gradients of a group need: its entries' excess counts / T, and per
// head the factor
__device__ __forceinline__ void bal_factors(const BalParams &p, int h0, int nh, float *f, float *by) {
    const int64_t steps = bal_steps(p);
    const float inv = steps > 0 ? 1.f / (float)steps : 0.f;
    const int i = threadIdx.x;
    if (i < nh * p.K) f[i] = bal_excess(p.counts[h0 * p.K + i], p.K, steps);
    if (i < nh) by[i] = p.g_loss[h0 + i] * ((float)p.K * p.inv_tau) * inv;
}

// g_u of one tile of steps over a slice of the groups: thread (ty, tx) owns rows
// ty + 16 i and pairs of columns, D <= DT.  A group takes about 10 us, so
// where the tiles do not fill the GPU the groups are split over CTAs too, and
// k_bal_gu_sum adds their sums in order.
template <int EC, int DT>
__global__ void __launch_bounds__(kBalThreads) k_bal_gu(BalParams p) {
    extern __shared__ float sm[];
    __shared__ float f[EC], by[EC];
    const Tile<EC> t(sm, p.D);
    const int gs = blockIdx.x % p.gslices;
    const int64_t r0 = (int64_t)(blockIdx.x / p.gslices) * kBalRows;
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    float acc[4][DT / 16];
    zero(acc);
    t.load_u(p, r0);
    for (int group = gs; group < p.groups; group += p.gslices) {
        const int h0 = group * p.heads, nh = min(p.heads, p.H - h0);
        __syncthreads();
        t.load_W(p, h0 * p.K, nh * p.K);
        bal_factors(p, h0, nh, f, by);
        t.landed();
        t.logits(p);
        t.template softmax<true>(p, nh, f, by);
        // entries behind the group's have zero weights, and logits that are zero
        tile_mm(acc, EC, Along2<4>{t.sp, t.kLdP, ty}, Across<DT / 16>{t.sW, t.ld, tx});
    }
    float *gu = p.gslices > 1 ? p.part + gs * p.rows * p.D : (float *)p.g_u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = r0 + strided(ty, i);
        if (r >= p.rows) continue;
#pragma unroll
        for (int j = 0; j < DT / 16; j += 2) {
            const int q = pairs(tx, j);
            float *at = gu + r * p.D + q;
            if (p.vec) {
                if (q < p.D) *reinterpret_cast<float2 *>(at) = make_float2(acc[i][j], acc[i][j + 1]);
            } else {
                if (q < p.D) at[0] = acc[i][j];
                if (q + 1 < p.D) at[1] = acc[i][j + 1];
            }
        }
    }
}

__global__ void k_bal_gu_sum(BalParams p) {
    const int64_t n = p.rows * p.D;
    for (int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; e < n;
         e += (int64_t)gridDim.x * blockDim.x) {
        float s = 0.f;
        for (int q = 0; q < p.gslices; ++q) s += p.part[q * n + e];
        ((float *)p.g_u)[e] = s;
    }
}

// g_W of one group over one slice of the steps
template <int EC, int DT>
__global__ void __launch_bounds__(kBalThreads) k_bal_gw(BalParams p) {
    extern __shared__ float sm[];
    __shared__ float f[EC], by[EC];
    const Tile<EC> t(sm, p.D);
    const int group = blockIdx.x % p.groups, slice = blockIdx.x / p.groups;
    const int h0 = group * p.heads, nh = min(p.heads, p.H - h0), ne = nh * p.K;
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    float acc[EC / 16][DT / 16];
    zero(acc);
    t.load_W(p, h0 * p.K, ne);
    bal_factors(p, h0, nh, f, by);
    for (int64_t r0 = (int64_t)slice * kBalRows; r0 < p.rows; r0 += (int64_t)p.slices * kBalRows) {
        __syncthreads();
        t.load_u(p, r0);
        t.landed();
        t.logits(p);
        t.template softmax<true>(p, nh, f, by);
        tile_mm(acc, kBalRows, Across<EC / 16>{t.sp, t.kLdP, ty}, Across<DT / 16>{t.su, t.ld, tx});
    }
    t.landed();                         // also where there was no tile
#pragma unroll
    for (int i = 0; i < EC / 16; ++i) {
        const int e = pairs(ty, i);
        if (e >= ne) continue;
        float *out = p.part + ((int64_t)slice * p.H * p.K + h0 * p.K + e) * p.D;
#pragma unroll
        for (int j = 0; j < DT / 16; ++j)
            if (pairs(tx, j) < p.D) out[pairs(tx, j)] = acc[i][j];
    }
}

// g_W: the slices' sums, likewise
__global__ void __launch_bounds__(32 * kSumWays) k_bal_gw_sum(BalParams p, float *g_W) {
    __shared__ float sums[kSumWays][32];
    const int64_t n = (int64_t)p.H * p.K * p.D;
    const int lane = threadIdx.x % 32, way = threadIdx.x / 32;
    const int64_t e = (int64_t)blockIdx.x * 32 + lane;
    float s = 0.f;
    if (e < n)
        for (int q = way; q < p.slices; q += kSumWays) s += p.part[q * n + e];
    sums[way][lane] = s;
    __syncthreads();
    if (way || e >= n) return;
    for (int w = 1; w < kSumWays; ++w) s += sums[w][lane];
    g_W[e] = s;
}

// slices of the steps per group: two CTAs per SM, at least one tile each
int bal_slices(int64_t rows, int groups) {
    const int64_t tiles = (rows + kBalRows - 1) / kBalRows;
    int64_t n = (148 * 2 + groups - 1) / groups;
    if (n > tiles) n = tiles;
    return (int)(n < 1 ? 1 : n);
}

// slices of the groups for g_u: as many as the GPU takes beside the tiles
int bal_gslices(int64_t rows, int groups) {
    const int64_t tiles = (rows + kBalRows - 1) / kBalRows;
    const int64_t n = tiles > 0 ? 148 / tiles : 1;
    return (int)(n < 1 ? 1 : n > groups ? groups : n);
}

template <int EC, void (*KERN)(BalParams)>
cudaError_t launch(int64_t grid, cudaStream_t st, const BalParams &p) {
    static std::atomic<int> set[kLimitDevices];
    const cudaError_t e = allow_smem((const void *)KERN, (int)bal_smem(kBalMaxD, EC), set);
    if (e != cudaSuccess) return e;
    KERN<<<dim3((unsigned)grid), kBalThreads, bal_smem(p.D, EC), st>>>(p);
    return cudaGetLastError();
}

template <int EC, int DT>
cudaError_t run_grads(const BalParams &p, int what, cudaStream_t st) {
    if (what == 2) return launch<EC, k_bal_gw<EC, DT>>((int64_t)p.groups * p.slices, st, p);
    const int64_t tiles = (p.rows + kBalRows - 1) / kBalRows;
    const cudaError_t e = launch<EC, k_bal_gu<EC, DT>>(tiles * p.gslices, st, p);
    if (e != cudaSuccess || p.gslices == 1) return e;
    k_bal_gu_sum<<<(unsigned)((p.rows * p.D + 255) / 256), 256, 0, st>>>(p);
    return cudaGetLastError();
}

template <int EC>
cudaError_t run_cols(const BalParams &p, int what, cudaStream_t st) {
    if (what == 0) return launch<EC, k_bal_sums<EC>>((int64_t)p.groups * p.slices, st, p);
    if (p.D <= 64) return run_grads<EC, 64>(p, what, st);
    if (p.D <= 128) return run_grads<EC, 128>(p, what, st);
    return run_grads<EC, 256>(p, what, st);
}

cudaError_t run_f32(const BalParams &p, int what, cudaStream_t st) {
    return bal_cols(p.H, p.K) == 32 ? run_cols<32>(p, what, st) : run_cols<64>(p, what, st);
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

constexpr size_t kBalHead = 256;        // scratch in front of the partial sums: the steps

// partial sums of g_W, or of p with the counts
size_t bal_partials(const pdssm_dims &d, int slices) {
    return align256((size_t)slices * (size_t)(d.H * d.K) * (size_t)(d.D_in > 2 ? d.D_in : 2) * 4);
}

size_t bal_scratch(const pdssm_dims &d) {
    const BalTcPlan pl = bal_tc_plan(d);
    const size_t a = bal_partials(d, bal_slices(d.B * d.L, bal_groups((int)d.H, (int)d.K)));
    const size_t b = bal_partials(d, pl.slices) + bal_tc_extra(pl);
    const int hs = bal_gslices(d.B * d.L, bal_groups((int)d.H, (int)d.K));
    const size_t c = hs > 1 ? (size_t)hs * (size_t)(d.B * d.L * d.D_in) * 4 : 0;
    return kBalHead + (a > b ? (a > c ? a : c) : (b > c ? b : c));
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
    q.slices = dt == PDSSM_BF16 ? bal_tc_plan(*d).slices : bal_slices(q.rows, bal_groups(q.H, q.K));
    q.heads = bal_heads(q.H, q.K);
    q.groups = bal_groups(q.H, q.K);
    q.gslices = bal_gslices(q.rows, q.groups);
    q.vec = q.D % 4 == 0 && aligned(u, 16) && aligned(W, 16);
    q.steps = lengths && d->B > kBalWarpB ? (const int64_t *)scratch : nullptr;
    q.part = (float *)((unsigned char *)scratch + kBalHead);
    q.part_n = (int32_t *)(q.part + (int64_t)q.slices * q.H * q.K);
    *p = q;
    return PDSSM_OK;
}

cudaError_t count_steps(const BalParams &p, cudaStream_t st) {
    if (!p.steps) return cudaSuccess;
    k_bal_steps<<<1, kStepThreads, 0, st>>>(p, const_cast<int64_t *>(p.steps));
    return cudaGetLastError();
}

// fp32 on the CUDA cores, bf16 on the tensor cores (which keep W's parts
// behind the partial sums in scratch)
cudaError_t run_any(const pdssm_dims &d, const BalParams &p, pdssm_dtype dt, int what,
                    cudaStream_t st) {
    if (dt != PDSSM_BF16) return run_f32(p, what, st);
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
    cudaError_t e = count_steps(p, s);
    if (e == cudaSuccess) e = run_any(*dims, p, u_dtype, 0, s);
    if (e != cudaSuccess) return cuda_fail(e, "balance sums");
    k_bal_loss<<<p.H, 32 * kSumWays, 0, s>>>(p, loss, counts, probs);
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
    p.vec = p.vec && aligned(g_u, 16);
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e = count_steps(p, s);
    if (e != cudaSuccess) return cuda_fail(e, "balance steps");
    if (g_u && p.rows > 0) {
        e = run_any(*dims, p, u_dtype, 1, s);
        if (e != cudaSuccess) return cuda_fail(e, "balance g_u");
    }
    if (g_W) {
        e = run_any(*dims, p, u_dtype, 2, s);
        if (e != cudaSuccess) return cuda_fail(e, "balance g_W");
        const int64_t n = (int64_t)p.H * p.K * p.D;
        k_bal_gw_sum<<<(unsigned)((n + 31) / 32), 32 * kSumWays, 0, s>>>(p, g_W);
        e = cudaGetLastError();
        if (e != cudaSuccess) return cuda_fail(e, "balance g_W sum");
    }
    return PDSSM_OK;
}

}  // extern "C"
