// Adjoint of the decay scan for bf16 inputs: chunks of 64 steps in reverse,
// warp-level bf16 products (m16n8k16, fp32 accumulation).
//
// With S0 the state at the chunk's start (the forward left it), R = dl/dS at
// its end, e_i = e^{G_i}, w_j = e^{G_C - G_j}, D_ij = e^{G_i - G_j} (j <= i):
//     P = D (c b^T),  Q = D (g_y x^T)
//     g_c = e (g_y S0^T) + Q b          g_b = w (x R^T) + Q^T c
//     g_x = w (b R) + P^T g_y           R' = e^{G_C} R + (e c)^T g_y
//     g_log_a[t] = sum_{j<t<=i} P_ij (g_y_i . x_j) + sum_{i>=t} c_i . e_i (S0 g_y_i)
//                  + sum_{j<t} b_j . w_j (R x_j) + e^{G_C} <S0, R>
// R stays in fp32 registers.  Where a result is fp32 (R', and g_log_a through
// the state parts of g_c and g_b) the operand that is not bf16 by itself is
// split into three bf16 parts (24 bits); P, Q and the R that g_x reads are
// rounded to bf16 once.  g_x, g_c and g_b are bf16 themselves, which alone puts
// them 1.66e-3 of their norm off; with these roundings g_x is 2.35e-3 off, g_c
// and g_b 1.86e-3.
//
// tcgen05 is not used here: a chunk has nine 64-wide products whose results
// are all rescaled, masked or summed by rows and columns before the next one,
// and accumulators in registers take that without a round trip.  Bound: no one
// unit; of a chunk's time the warp-level tensor pipe takes 27 %, shared-memory
// wavefronts 56 %, instruction issue 43 %, in phases that barriers separate.
// 32 heads x 16384 steps of 64 x 64: 373 us (107 kflop per step, 150 TFLOP/s).
#include "decay.cuh"
#include "launch.cuh"
#include "tile_bf16.cuh"

namespace pdssm {
namespace {

constexpr int kC = 64;                      // steps of a chunk
constexpr uint32_t kTile = 64 * 128;        // 64 rows of 64 bf16, 128-byte swizzle

// Per chunk, double-buffered: its decays (made a chunk ahead) and what
// g_log_a adds up (taken a chunk later).  WC: column groups of the warps.
template <int WC>
struct Sums {
    float2 G[kC];           // cumulated, base 2, hi + lo
    float e[kC], w[kC];     // e_i, w_j
    float row[WC][kC];      // pair sums by row, per column group
    float col[4][kC];       // by column, per row block
    float u[WC][kC], v[WC][kC];
    float dot[4 * WC];
};

// NT and PT: N and P in units of 64.  Above 64 x 64 R's parts take the place of
// S0's once those have been read, and as one CTA fits an SM it has twice the
// warps (64 heads x 2048 steps forward and backward, 128 x 128: 510 us, with
// eight 554).
template <int NT, int PT>
struct Smem {
    static constexpr bool kShare = NT * PT > 1;
    // warps of the products: 4 by rows times WC by columns; then one for decays and
    // g_log_a
    static constexpr int kWC = kShare ? 4 : 2, kWarps = 4 * kWC, kTh = 32 * kWarps, kAll = kTh + 32;
    static constexpr uint32_t kState = NT * PT * kTile;             // one part
    static constexpr uint32_t kc = 0, kb = NT * kTile, kx = 2 * NT * kTile, kg = kx + PT * kTile;
    static constexpr uint32_t kS = kg + PT * kTile, kR = kShare ? kS : kS + 3 * kState;
    static constexpr uint32_t kP = kR + 3 * kState, kQ = kP + kTile;
    static constexpr uint32_t kF = kQ + kTile;                      // floats below
    static constexpr uint32_t kTotal = kF + 2 * sizeof(Sums<kWC>);
};

__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a));
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a));
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Fragment addresses in a tile; `l` is the lane.
// A (16 x 16 at row m0, k-step ks) of rows stored [m][k]
__device__ __forceinline__ uint32_t at_a(uint32_t t, int m0, int ks, int l) {
    return t + piece(m0 + (l & 15), 2 * ks + (l >> 4));
}
// A of columns stored [k][m]
__device__ __forceinline__ uint32_t at_at(uint32_t t, int m0, int ks, int l) {
    return t + piece(16 * ks + (l & 7) + ((l >> 4) << 3), m0 / 8 + ((l >> 3) & 1));
}
// B (k-step ks, columns n0..n0+15) stored [n][k]
__device__ __forceinline__ uint32_t at_b(uint32_t t, int n0, int ks, int l) {
    return t + piece(n0 + (l & 7) + ((l >> 4) << 3), 2 * ks + ((l >> 3) & 1));
}
// B stored [k][n]
__device__ __forceinline__ uint32_t at_bt(uint32_t t, int n0, int ks, int l) {
    return t + piece(16 * ks + (l & 15), n0 / 8 + (l >> 4));
}

// three bf16 parts of a pair
__device__ __forceinline__ void split3(float a, float b, uint32_t (&o)[3]) {
    o[0] = pack2(a, b);
    a -= lo_of(o[0]);
    b -= hi_of(o[0]);
    o[1] = pack2(a, b);
    a -= lo_of(o[1]);
    b -= hi_of(o[1]);
    o[2] = pack2(a, b);
}

__device__ __forceinline__ void sts32(uint32_t a, uint32_t v) {
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ float quad_sum(float v) {
    v += __shfl_xor_sync(kFull, v, 1);
    return v + __shfl_xor_sync(kFull, v, 2);
}

// Barrier of the product warps.
template <int TH>
__device__ __forceinline__ void sync_products() {
    asm volatile("bar.sync 1, %0;" ::"n"(TH) : "memory");
}

template <int NT, int PT>
__global__ void __launch_bounds__(Smem<NT, PT>::kAll, NT * PT > 1 ? 1 : 2) k_decay_bwd_mma(DecayParams p) {
    using SM = Smem<NT, PT>;
    constexpr int kTh = SM::kTh, WC = SM::kWC, F = 8 / WC;     // F: 8-column pieces of a warp
    using Sums = Sums<WC>;
    extern __shared__ __align__(128) unsigned char sm_raw[];
    const uint32_t sm = smem_u32(sm_raw);
    Sums *sums = reinterpret_cast<Sums *>(sm_raw + SM::kF);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int wr = warp & 3, wc = warp >> 2;    // 16 rows and 8 F columns of each product
    const int g = lane >> 2, q2 = (lane & 3) * 2;
    const int m0 = 16 * wr, n0 = 8 * F * wc;

    const int seg = blockIdx.x % p.nseg;
    const int64_t bh = blockIdx.x / p.nseg;
    const int b = (int)(bh / p.H), h = (int)(bh % p.H);
    const int64_t len = decay_len(p, b);
    const int64_t koff = b * p.key_b + (h / p.rep) * p.key_h, voff = b * p.val_b + h * p.val_h;
    typedef __nv_bfloat16 T;
    const T *c = (const T *)p.c + koff, *bb = (const T *)p.b + koff;
    const T *x = (const T *)p.x + voff, *gy = (const T *)p.g_y + voff;
    T *gx = (T *)p.g_x + b * p.oval_b + h * p.oval_h;
    const float *la = p.log_a + b * p.la_b + h * p.la_h;
    float *gla = p.g_la + b * p.gla_b + h * p.gla_h;
    const int64_t okoff = b * p.okey_b + (h / p.rep) * p.okey_h;
    const bool part = p.rep > 1;        // gradients of shared keys: fp32 [B][H][L][N] partials
    const int64_t poff = bh * p.L * p.N, np = (int64_t)p.N * p.P;

    const int c0 = seg * p.seg_chunks, c1 = min(c0 + p.seg_chunks, p.nchunks);

    if (warp == SM::kWarps) {
        // ---- decays of the next chunk and g_log_a of the last one, while the
        // product warps work on this one
        auto decays = [&](int ch) {
            const int64_t t0 = (int64_t)ch * kC;
            if (ch < c0 || t0 >= len) return;
            Sums &s = sums[ch & 1];
            decay_sums<kC>([&](int t) { return t0 + t < len ? la[(t0 + t) * p.la_t] : 0.f; }, s.G, lane);
            __syncwarp();
            const float2 end = s.G[kC - 1];
#pragma unroll
            for (int i = 0; i < kC; i += 32) {
                s.e[i + lane] = decay_from_start(s.G[i + lane]);
                s.w[i + lane] = decay_between(end, s.G[i + lane]);
            }
        };
        // g_log_a[t] = sum_{i>=t} (row_i + u_i - col_i) + sum_{j<t} v_j + e^{G_C} <S0, R>
        auto gradient = [&](int ch) {
            const int64_t t0 = (int64_t)ch * kC;
            if (ch >= c1 || t0 >= len) return;
            const Sums &s = sums[ch & 1];
            double through = 0.0;
            for (int w = 0; w < SM::kWarps; ++w) through += (double)s.dot[w];
            through *= (double)s.e[kC - 1];
            double before = 0.0, total = 0.0, inc[2], pre[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int t = q * 32 + lane;
                double a = 0.0, v = 0.0;
#pragma unroll
                for (int w = 0; w < WC; ++w) {
                    a += (double)s.row[w][t] + (double)s.u[w][t];
                    v += (double)s.v[w][t];
                }
                a -= (double)s.col[0][t] + (double)s.col[1][t] + (double)s.col[2][t] + (double)s.col[3][t];
                const double a0 = a, v0 = v;
#pragma unroll
                for (int d = 1; d < 32; d *= 2) {
                    const double oa = shfl_up_d(a, d), ov = shfl_up_d(v, d);
                    if (lane >= d) {
                        a += oa;
                        v += ov;
                    }
                }
                inc[q] = total + a - a0;
                pre[q] = before + v - v0;
                total += __shfl_sync(kFull, a, 31);
                before += __shfl_sync(kFull, v, 31);
            }
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int64_t t = t0 + q * 32 + lane;
                if (t < p.L)    // a floored decay is a constant
                    gla[t * p.gla_t] = t < len && !(la[t * p.la_t] <= (float)kDecayFloor)
                                           ? (float)(total - inc[q] + pre[q] + through)
                                           : 0.f;
            }
        };
        decays(c1 - 1);
        for (int ch = c1 - 1; ch >= c0; --ch) {
            __syncthreads();
            gradient(ch + 1);
            __syncwarp();
            decays(ch - 1);
        }
        __syncthreads();
        gradient(c0);
        return;
    }

    // R: per 64 x 64 rows m0 + g (+ 8), columns n0 + 8 f + q2 (+ 1)
    float R[NT][PT][F][4];
    auto each = [&](auto &&f) {         // f(nt, pt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int pt = 0; pt < PT; ++pt) f(nt, pt);
    };
    {
        const float *in = p.nseg > 1 ? p.seg_state + (bh * p.nseg + seg) * np
                                     : (p.g_hlast ? p.g_hlast + bh * np : nullptr);
        each([&](int nt, int pt) {
#pragma unroll
            for (int f = 0; f < F; ++f)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int n = 64 * nt + m0 + g + 8 * (e >> 1), q = 64 * pt + n0 + 8 * f + q2 + (e & 1);
                    R[nt][pt][f][e] = in && n < p.N && q < p.P ? in[(int64_t)n * p.P + q] : 0.f;
                }
        });
    }
    // blocks above the diagonal of P and Q stay zero
    for (int e = tid; e < 2 * 512; e += kTh)
        *reinterpret_cast<uint4 *>(sm_raw + SM::kP + 16 * e) = make_uint4(0, 0, 0, 0);

    auto store_key = [&](void *out, int64_t t, int q, float v0, float v1) {     // columns q, q + 1
        if (t >= p.L) return;
        if (t >= len) v0 = v1 = 0.f;
        if (part) {
            float *o = (float *)out + poff + t * p.N + q;
            if (q < p.N) o[0] = v0;
            if (q + 1 < p.N) o[1] = v1;
        } else {
            T *o = (T *)out + okoff + t * p.okey_t + q;
            if (p.ovec) {
                if (q < p.N) *reinterpret_cast<uint32_t *>(o) = pack2(v0, v1);
            } else {
                if (q < p.N) o[0] = __float2bfloat16_rn(v0);
                if (q + 1 < p.N) o[1] = __float2bfloat16_rn(v1);
            }
        }
    };

    for (int ch = c1 - 1; ch >= c0; --ch) {
        const int64_t t0 = (int64_t)ch * kC;
        __syncthreads();                // the last chunk's tiles have been read; decays are in
        Sums &sw = sums[ch & 1];
        if (t0 >= len) {                // behind the end: zero gradients, R stays
            constexpr int W = 64 * (NT > PT ? NT : PT);
            for (int e = tid; e < kC * W; e += kTh) {
                const int64_t t = t0 + e / W;
                const int q = e % W;
                if (t >= p.L) continue;
                if (q < p.P) gx[t * p.oval_t + q] = __float2bfloat16_rn(0.f);
                if (q < p.N) {
                    if (part) {
                        ((float *)p.g_c)[poff + t * p.N + q] = 0.f;
                        ((float *)p.g_b)[poff + t * p.N + q] = 0.f;
                    } else {
                        ((T *)p.g_c)[okoff + t * p.okey_t + q] = __float2bfloat16_rn(0.f);
                        ((T *)p.g_b)[okoff + t * p.okey_t + q] = __float2bfloat16_rn(0.f);
                    }
                }
                if (q == 0) gla[t * p.gla_t] = 0.f;
            }
            continue;
        }
        // ---- tiles: zero behind the end and behind the widths
        if (p.vec) {
#pragma unroll
            for (int i = 0; i < 512 / kTh; ++i) {
                const int e = tid + i * kTh, r = e >> 3, q = e & 7;
                const bool on = t0 + r < len;
                const int64_t t = on ? t0 + r : t0;
                auto cp = [&](uint32_t tile, const T *src, bool in) {
                    const int n = on && in ? 16 : 0;
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sm + tile + piece(r, q)),
                                 "l"(src), "r"(n)
                                 : "memory");
                };
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const bool in = 64 * j + 8 * q < p.N;
                    const int64_t at = t * p.key_t + (in ? 64 * j + 8 * q : 0);
                    cp(SM::kc + j * kTile, c + at, in);
                    cp(SM::kb + j * kTile, bb + at, in);
                }
#pragma unroll
                for (int j = 0; j < PT; ++j) {
                    const bool in = 64 * j + 8 * q < p.P;
                    const int64_t at = t * p.val_t + (in ? 64 * j + 8 * q : 0);
                    cp(SM::kx + j * kTile, x + at, in);
                    cp(SM::kg + j * kTile, gy + at, in);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        } else {
            for (int e = tid; e < kC * 32; e += kTh) {
                const int r = e >> 5, q = (e & 31) * 2;
                const int64_t t = t0 + r;
                auto cp = [&](uint32_t tile, const T *src, int64_t stride, int width) {
                    uint32_t w = 0;
                    if (t < len) {
                        const unsigned short *s = reinterpret_cast<const unsigned short *>(src + t * stride) + q;
                        if (q < width) w = s[0];
                        if (q + 1 < width) w |= (uint32_t)s[1] << 16;
                    }
                    sts32(sm + tile + piece(r, q / 8) + (q & 7) * 2, w);
                };
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    cp(SM::kc + j * kTile, c + 64 * j, p.key_t, p.N - 64 * j);
                    cp(SM::kb + j * kTile, bb + 64 * j, p.key_t, p.N - 64 * j);
                }
#pragma unroll
                for (int j = 0; j < PT; ++j) {
                    cp(SM::kx + j * kTile, x + 64 * j, p.val_t, p.P - 64 * j);
                    cp(SM::kg + j * kTile, gy + 64 * j, p.val_t, p.P - 64 * j);
                }
            }
        }
        // the next chunk's rows and state on their way to L2
        if (ch > c0) {
            const int64_t tn = t0 - kC + (tid & 63);
            const void *at = tid < 64    ? (const void *)(c + tn * p.key_t)
                             : tid < 128 ? (const void *)(bb + tn * p.key_t)
                             : tid < 192 ? (const void *)(x + tn * p.val_t)
                                         : (const void *)(gy + tn * p.val_t);
            if (tid < 256) asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
#pragma unroll
            for (int j = tid; j < NT * PT * 128; j += kTh)
                if (ch > 1 && j * 32 < np)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(p.carry + (bh * p.nchunks + ch - 1) * np + j * 32));
        }
        // ---- parts of S0 and R, and <S0, R>
        {
            const float *S0 = ch > 0 ? p.carry + (bh * p.nchunks + ch) * np
                                     : (p.h0 ? p.h0 + bh * np : nullptr);
            float dot = 0.f;
            const bool even = p.P % 2 == 0 && ((uintptr_t)S0 & 7) == 0;
            each([&](int nt, int pt) {
                float S[F][4];
#pragma unroll
                for (int f = 0; f < F; ++f)
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        const int n = 64 * nt + m0 + g + 4 * e, q = 64 * pt + n0 + 8 * f + q2;
                        const bool in = S0 && n < p.N;
                        const float *at = S0 + (int64_t)n * p.P + q;
                        if (even) {
                            const float2 v = in && q < p.P ? *reinterpret_cast<const float2 *>(at) : make_float2(0.f, 0.f);
                            S[f][e] = v.x;
                            S[f][e + 1] = v.y;
                        } else {
                            S[f][e] = in && q < p.P ? at[0] : 0.f;
                            S[f][e + 1] = in && q + 1 < p.P ? at[1] : 0.f;
                        }
                    }
#pragma unroll
                for (int f = 0; f < F; ++f)
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        const float(&r)[4] = R[nt][pt][f];
                        const uint32_t at = sm + (nt * PT + pt) * kTile + piece(m0 + g + 4 * e, n0 / 8 + f) + q2 * 2;
                        uint32_t o[3];
                        dot = fmaf(S[f][e], r[e], dot);
                        dot = fmaf(S[f][e + 1], r[e + 1], dot);
                        split3(S[f][e], S[f][e + 1], o);
#pragma unroll
                        for (int k = 0; k < 3; ++k) sts32(at + SM::kS + k * SM::kState, o[k]);
                        if (!SM::kShare) {
                            split3(r[e], r[e + 1], o);
#pragma unroll
                            for (int k = 0; k < 3; ++k) sts32(at + SM::kR + k * SM::kState, o[k]);
                        }
                    }
            });
#pragma unroll
            for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(kFull, dot, d);
            if (lane == 0) sw.dot[warp] = dot;
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        sync_products<kTh>();
        const float aend = sw.e[kC - 1];

        // ---- P and Q of rows m0.., the 16-column blocks k = wc, wc + WC, .. <= wr
        {
            // rows' operands: kept over the blocks, or fetched for each (registers)
            uint32_t ca[4][4], ga[4][4];
            if (!SM::kShare) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {
                    ldm4(ca[ks], at_a(sm + SM::kc, m0, ks, lane));
                    ldm4(ga[ks], at_a(sm + SM::kg, m0, ks, lane));
                }
            }
            const float2 gr0 = sw.G[m0 + g], gr1 = sw.G[m0 + g + 8];
            float row0 = 0.f, row1 = 0.f;
#pragma unroll 1
            for (int k = wc; k < 4; k += WC) {
                float *col = sw.col[wr] + 16 * k;
                if (k > wr) {
                    if (lane < 16) col[lane] = 0.f;
                    continue;
                }
                float s[2][4], v[2][4];
#pragma unroll
                for (int f = 0; f < 2; ++f)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[f][e] = v[f][e] = 0.f;
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {
                    uint32_t f[4];
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        if (SM::kShare) ldm4(ca[ks], at_a(sm + SM::kc + j * kTile, m0, ks, lane));
                        ldm4(f, at_b(sm + SM::kb + j * kTile, 16 * k, ks, lane));
                        mma(s[0], ca[ks], f[0], f[1]);
                        mma(s[1], ca[ks], f[2], f[3]);
                    }
#pragma unroll
                    for (int j = 0; j < PT; ++j) {
                        if (SM::kShare) ldm4(ga[ks], at_a(sm + SM::kg + j * kTile, m0, ks, lane));
                        ldm4(f, at_b(sm + SM::kx + j * kTile, 16 * k, ks, lane));
                        mma(v[0], ga[ks], f[0], f[1]);
                        mma(v[1], ga[ks], f[2], f[3]);
                    }
                }
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    const int j = 16 * k + 8 * f + q2;
                    const float2 gj0 = sw.G[j], gj1 = sw.G[j + 1];
                    float pv[4], qv[4], ev[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int i = m0 + g + 8 * (e >> 1), jj = j + (e & 1);
                        const float d = decay_between(e < 2 ? gr0 : gr1, e & 1 ? gj1 : gj0);
                        pv[e] = jj <= i ? s[f][e] * d : 0.f;
                        qv[e] = jj <= i ? v[f][e] * d : 0.f;
                        ev[e] = jj < i ? pv[e] * v[f][e] : 0.f;
                    }
                    row0 += ev[0] + ev[1];
                    row1 += ev[2] + ev[3];
                    float c0s = ev[0] + ev[2], c1s = ev[1] + ev[3];
#pragma unroll
                    for (int d = 4; d < 32; d *= 2) {
                        c0s += __shfl_xor_sync(kFull, c0s, d);
                        c1s += __shfl_xor_sync(kFull, c1s, d);
                    }
                    if (g == 0) {
                        col[8 * f + q2] = c0s;
                        col[8 * f + q2 + 1] = c1s;
                    }
                    const uint32_t a0 = sm + piece(m0 + g, 2 * k + f) + q2 * 2,
                                   a1 = sm + piece(m0 + g + 8, 2 * k + f) + q2 * 2;
                    sts32(a0 + SM::kP, pack2(pv[0], pv[1]));
                    sts32(a1 + SM::kP, pack2(pv[2], pv[3]));
                    sts32(a0 + SM::kQ, pack2(qv[0], qv[1]));
                    sts32(a1 + SM::kQ, pack2(qv[2], qv[3]));
                }
                __syncwarp();
            }
            row0 = quad_sum(row0);
            row1 = quad_sum(row1);
            if ((lane & 3) == 0) {
                sw.row[wc][m0 + g] = row0;
                sw.row[wc][m0 + g + 8] = row1;
            }
        }
        sync_products<kTh>();

        float acc[F][4];
        auto zero = [&]() {
#pragma unroll
            for (int f = 0; f < F; ++f)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[f][e] = 0.f;
        };
        // rows times the transpose of a [n][k] operand in three parts
        auto by_parts = [&](uint32_t rows, uint32_t parts) {
            uint32_t a[4][4];
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) ldm4(a[ks], at_a(rows, m0, ks, lane));
#pragma unroll
            for (int k = 2; k >= 0; --k)        // the small parts first: additions truncate
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {
#pragma unroll
                    for (int f = 0; f < F; f += 2) {
                        uint32_t b[4];
                        ldm4(b, at_b(parts + k * SM::kState, n0 + 8 * f, ks, lane));
                        mma(acc[f], a[ks], b[0], b[1]);
                        mma(acc[f + 1], a[ks], b[2], b[3]);
                    }
                }
        };
        // acc *= by row factors; the rows' products with a tile's rows
        auto scale_rows = [&](float f0, float f1) {
#pragma unroll
            for (int f = 0; f < F; ++f) {
                acc[f][0] *= f0;
                acc[f][1] *= f0;
                acc[f][2] *= f1;
                acc[f][3] *= f1;
            }
        };
        float d0, d1;
        auto row_dots = [&](uint32_t tile) {
#pragma unroll
            for (int f = 0; f < F; ++f) {
                const uint32_t w0 = lds_u32(sm + tile + piece(m0 + g, n0 / 8 + f) + q2 * 2),
                               w1 = lds_u32(sm + tile + piece(m0 + g + 8, n0 / 8 + f) + q2 * 2);
                d0 = fmaf(acc[f][0], lo_of(w0), fmaf(acc[f][1], hi_of(w0), d0));
                d1 = fmaf(acc[f][2], lo_of(w1), fmaf(acc[f][3], hi_of(w1), d1));
            }
        };
        auto leave_dots = [&](float (&out)[WC][kC]) {
            d0 = quad_sum(d0);
            d1 = quad_sum(d1);
            if ((lane & 3) == 0) {
                out[wc][m0 + g] = d0;
                out[wc][m0 + g + 8] = d1;
            }
            __syncwarp();
        };
        auto add_pairs = [&](const uint32_t (&a)[4], uint32_t tile, int ks) {
#pragma unroll
            for (int f = 0; f < F; f += 2) {
                uint32_t b[4];
                ldm4t(b, at_bt(tile, n0 + 8 * f, ks, lane));
                mma(acc[f], a, b[0], b[1]);
                mma(acc[f + 1], a, b[2], b[3]);
            }
        };
        const int64_t tr0 = t0 + m0 + g, tr1 = tr0 + 8;

        // ---- g_c
        d0 = d1 = 0.f;
#pragma unroll 1
        for (int nt = 0; nt < NT; ++nt) {
            zero();
#pragma unroll 1
            for (int pt = 0; pt < PT; ++pt)
                by_parts(sm + SM::kg + pt * kTile, sm + SM::kS + (nt * PT + pt) * kTile);
            scale_rows(sw.e[m0 + g], sw.e[m0 + g + 8]);
            row_dots(SM::kc + nt * kTile);
#pragma unroll 1
            for (int ks = 0; ks <= wr; ++ks) {
                uint32_t a[4];
                ldm4(a, at_a(sm + SM::kQ, m0, ks, lane));
                add_pairs(a, sm + SM::kb + nt * kTile, ks);
            }
#pragma unroll
            for (int f = 0; f < F; ++f) {
                store_key(p.g_c, tr0, 64 * nt + n0 + 8 * f + q2, acc[f][0], acc[f][1]);
                store_key(p.g_c, tr1, 64 * nt + n0 + 8 * f + q2, acc[f][2], acc[f][3]);
            }
            __syncwarp();               // rows behind the end part ways; products are the whole warp's
        }
        leave_dots(sw.u);
        if (SM::kShare) {
            sync_products<kTh>();            // S0's parts have been read
            each([&](int nt, int pt) {
#pragma unroll
                for (int f = 0; f < F; ++f)
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        const float(&r)[4] = R[nt][pt][f];
                        const uint32_t at = sm + SM::kR + (nt * PT + pt) * kTile +
                                            piece(m0 + g + 4 * e, n0 / 8 + f) + q2 * 2;
                        uint32_t o[3];
                        split3(r[e], r[e + 1], o);
#pragma unroll
                        for (int k = 0; k < 3; ++k) sts32(at + k * SM::kState, o[k]);
                    }
            });
            sync_products<kTh>();
        }
        // ---- g_b
        const float w0 = sw.w[m0 + g], w1 = sw.w[m0 + g + 8];
        d0 = d1 = 0.f;
#pragma unroll 1
        for (int nt = 0; nt < NT; ++nt) {
            zero();
#pragma unroll 1
            for (int pt = 0; pt < PT; ++pt)
                by_parts(sm + SM::kx + pt * kTile, sm + SM::kR + (nt * PT + pt) * kTile);
            scale_rows(w0, w1);
            row_dots(SM::kb + nt * kTile);
#pragma unroll 1
            for (int ks = wr; ks < 4; ++ks) {
                uint32_t a[4];
                ldm4t(a, at_at(sm + SM::kQ, m0, ks, lane));
                add_pairs(a, sm + SM::kc + nt * kTile, ks);
            }
#pragma unroll
            for (int f = 0; f < F; ++f) {
                store_key(p.g_b, tr0, 64 * nt + n0 + 8 * f + q2, acc[f][0], acc[f][1]);
                store_key(p.g_b, tr1, 64 * nt + n0 + 8 * f + q2, acc[f][2], acc[f][3]);
            }
            __syncwarp();
        }
        leave_dots(sw.v);
        // ---- g_x
#pragma unroll 1
        for (int pt = 0; pt < PT; ++pt) {
            zero();
#pragma unroll 1
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {
                    uint32_t a[4];
                    ldm4(a, at_a(sm + SM::kb + nt * kTile, m0, ks, lane));
                    add_pairs(a, sm + SM::kR + (nt * PT + pt) * kTile, ks);
                }
            scale_rows(w0, w1);
#pragma unroll 1
            for (int ks = wr; ks < 4; ++ks) {
                uint32_t a[4];
                ldm4t(a, at_at(sm + SM::kP, m0, ks, lane));
                add_pairs(a, sm + SM::kg + pt * kTile, ks);
            }
#pragma unroll
            for (int f = 0; f < F; ++f) {
                const int q = 64 * pt + n0 + 8 * f + q2;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int64_t t = e ? tr1 : tr0;
                    if (t >= p.L) continue;
                    const float v0 = t < len ? acc[f][2 * e] : 0.f, v1 = t < len ? acc[f][2 * e + 1] : 0.f;
                    T *o = gx + t * p.oval_t + q;
                    if (p.ovec) {
                        if (q < p.P) *reinterpret_cast<uint32_t *>(o) = pack2(v0, v1);
                    } else {
                        if (q < p.P) o[0] = __float2bfloat16_rn(v0);
                        if (q + 1 < p.P) o[1] = __float2bfloat16_rn(v1);
                    }
                }
            }
            __syncwarp();
        }
        // ---- R: the chunk's part from zero, then one fp32 multiply-add (a product's
        // own additions truncate, which would pile up over a long memory)
        each([&](int nt, int pt) {
            zero();
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                uint32_t a[4], parts[3][4], fb[F / 2][4];
                ldm4t(a, at_at(sm + SM::kc + nt * kTile, m0, ks, lane));
#pragma unroll
                for (int f = 0; f < F / 2; ++f)
                    ldm4t(fb[f], at_bt(sm + SM::kg + pt * kTile, n0 + 16 * f, ks, lane));
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 w = *reinterpret_cast<const float2 *>(sw.e + 16 * ks + 8 * (e >> 1) + q2);
                    uint32_t o[3];
                    split3(lo_of(a[e]) * w.x, hi_of(a[e]) * w.y, o);
#pragma unroll
                    for (int k = 0; k < 3; ++k) parts[k][e] = o[k];
                }
#pragma unroll
                for (int k = 0; k < 3; ++k)
#pragma unroll
                    for (int f = 0; f < F / 2; ++f) {
                        mma(acc[2 * f], parts[k], fb[f][0], fb[f][1]);
                        mma(acc[2 * f + 1], parts[k], fb[f][2], fb[f][3]);
                    }
            }
#pragma unroll
            for (int f = 0; f < F; ++f)
#pragma unroll
                for (int e = 0; e < 4; ++e) R[nt][pt][f][e] = fmaf(aend, R[nt][pt][f][e], acc[f][e]);
        });
    }
    __syncthreads();                    // for the last chunk's g_log_a
    if (p.g_h0 && seg == 0) {
        float *out = p.g_h0 + bh * np;
        each([&](int nt, int pt) {
#pragma unroll
            for (int f = 0; f < F; ++f)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int n = 64 * nt + m0 + g + 8 * (e >> 1), q = 64 * pt + n0 + 8 * f + q2 + (e & 1);
                    if (n < p.N && q < p.P) out[(int64_t)n * p.P + q] = R[nt][pt][f][e];
                }
        });
    }
}

template <int NT, int PT>
cudaError_t go(const DecayParams &p, cudaStream_t st) {
    static std::atomic<int> set[kLimitDevices];
    constexpr int smem = (int)Smem<NT, PT>::kTotal;
    const cudaError_t e = allow_smem((const void *)k_decay_bwd_mma<NT, PT>, smem, set);
    if (e != cudaSuccess) return e;
    k_decay_bwd_mma<NT, PT><<<dim3((unsigned)((int64_t)p.B * p.H * p.nseg)), Smem<NT, PT>::kAll, smem, st>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decay_bwd_mma(const DecayParams &p, cudaStream_t st) {
    if (p.nseg > 1) {
        // the segments in the tensor-core kernel's chunks of 128 steps
        DecayParams s = p;
        s.nchunks = (int)((p.L + 127) / 128);
        s.seg_chunks = p.seg_chunks / 2;
        s.pslices = (p.P + 63) / 64;
        cudaError_t e = launch_decay_seg_rev_tc(s, st);
        if (e != cudaSuccess) return e;
        e = launch_decay_join(p, p.g_hlast, true, st);
        if (e != cudaSuccess) return e;
    }
    if (p.N <= 64) return p.P <= 64 ? go<1, 1>(p, st) : go<1, 2>(p, st);
    return p.P <= 64 ? go<2, 1>(p, st) : go<2, 2>(p, st);
}

}  // namespace pdssm
