// Decay scan of fp32 inputs on the CUDA cores, any width, and the small kernels
// of both paths.  One CTA of 256 threads (16 x 16) per segment of a (batch, head);
// a chunk's operands sit in shared memory as fp32 rows of width + 4 floats, and
// each thread owns a TM x TN tile of a product's result.
//
// Bound: shared-memory bandwidth.  Both orientations of a product are read by
// 16- or 8-byte loads (see Along and Across): about half of the wavefronts and
// a third of the instructions of 4-byte loads.  64 heads x 1024 steps of 64 x
// 64: forward 144 us, forward and adjoint 506 us.
#include "decay.cuh"
#include "launch.cuh"
#include "tile_mm.cuh"

namespace pdssm {
namespace {

constexpr int kThreads = 256;
constexpr int kC = 32;                  // steps of a chunk

// Rows t0..t0+C-1 of a [step][width] tensor on their way to shared rows of
// WT + 4 floats; zero behind `len` and behind the width.  A chunk's rows are
// fetched while the chunk before it is worked on (their latency, a
// microsecond, is a third of a short chunk's time).
template <int C, int WT>
struct Rows {
    static constexpr int kN = C * WT / kThreads;
    float v[kN];
    __device__ __forceinline__ void fetch(const float *src, int64_t stride, int width, int64_t t0,
                                          int64_t len) {
        const int n = threadIdx.x % WT;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int64_t t = t0 + (i * kThreads + threadIdx.x) / WT;
            v[i] = n < width && t < len ? src[t * stride + n] : 0.f;
        }
    }
    __device__ __forceinline__ void put(float *dst) const {
#pragma unroll
        for (int i = 0; i < kN; ++i)
            dst[(i * kThreads + threadIdx.x) / WT * (WT + 4) + threadIdx.x % WT] = v[i];
    }
};

struct Head {
    int bh, b, h;
    int64_t len;
    const float *la;
    __device__ __forceinline__ float log_a(const DecayParams &p, int64_t t) const {
        return t < len ? la[t * p.la_t] : 0.f;
    }
};

__device__ __forceinline__ Head head_of(const DecayParams &p, int64_t bh) {
    Head hd;
    hd.bh = (int)bh;
    hd.b = (int)(bh / p.H);
    hd.h = (int)(bh % p.H);
    hd.len = decay_len(p, hd.b);
    hd.la = p.log_a + hd.b * p.la_b + hd.h * p.la_h;
    return hd;
}

// A chunk's log decays, fetched likewise, by the first warp.
template <int C>
struct Steps {
    float v[C / 32];
    __device__ __forceinline__ void fetch(const DecayParams &p, const Head &hd, int64_t t0) {
        if (threadIdx.x < 32)
#pragma unroll
            for (int i = 0; i < C / 32; ++i) v[i] = hd.log_a(p, t0 + 32 * i + threadIdx.x);
    }
    __device__ __forceinline__ void sums(float2 *G) const {
        if (threadIdx.x < 32)
            decay_sums<C>([&](int t) { return v[t / 32]; }, G, threadIdx.x);
    }
};

// The state alone over one segment from zero.  Forward (REV = false): rows u
// = b, v = x, weights e^{G_C - G_t}, chunks in order.  Reverse: u = c, v =
// g_y, weights e^{G_t}, chunks in reverse.
template <int C, int NT, int PT, bool REV>
__global__ void __launch_bounds__(kThreads) k_decay_seg_gen(DecayParams p) {
    extern __shared__ float sm[];
    constexpr int LN = NT + 4, LP = PT + 4, TN = NT / 16, TP = PT / 16;
    float *su = sm, *sv = su + C * LN;
    float2 *sG = reinterpret_cast<float2 *>(sv + C * LP);
    const int seg = blockIdx.x % p.nseg;
    const Head hd = head_of(p, blockIdx.x / p.nseg);
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    const float *u = (const float *)(REV ? p.c : p.b) + hd.b * p.key_b + (hd.h / p.rep) * p.key_h;
    const float *v = (const float *)(REV ? p.g_y : p.x) + hd.b * p.val_b + hd.h * p.val_h;
    float S[TN][TP];
    zero(S);
    double total = 0.0;
    const int c0 = seg * p.seg_chunks, c1 = min(c0 + p.seg_chunks, p.nchunks);
    Rows<C, NT> ru;
    Rows<C, PT> rv;
    Steps<C> rl;
    auto fetch = [&](int i) {
        const int64_t t0 = i < c1 ? (int64_t)(REV ? c1 - 1 - (i - c0) : i) * C : hd.len;
        ru.fetch(u, p.key_t, p.N, t0, hd.len);
        rv.fetch(v, p.val_t, p.P, t0, hd.len);
        rl.fetch(p, hd, t0);
    };
    fetch(c0);
    for (int i = c0; i < c1; ++i) {
        const int64_t t0 = (int64_t)(REV ? c1 - 1 - (i - c0) : i) * C;
        if (t0 >= hd.len) {             // behind the end: nothing is added, nothing decays
            fetch(i + 1);
            continue;
        }
        ru.put(su);
        rv.put(sv);
        rl.sums(sG);
        fetch(i + 1);
        __syncthreads();
        const float2 end = sG[C - 1];
        total += (double)end.x + (double)end.y;
        for (int e = threadIdx.x; e < C * NT; e += kThreads) {
            const int t = e / NT;
            const float w = REV ? decay_from_start(sG[t]) : decay_between(end, sG[t]);
            su[t * LN + e % NT] *= w;
        }
        __syncthreads();
        const float a = decay_from_start(end);
#pragma unroll
        for (int m = 0; m < TN; ++m)
#pragma unroll
            for (int n = 0; n < TP; ++n) S[m][n] *= a;
        tile_mm(S, C, Across<TN>{su, LN, ty}, Across<TP>{sv, LP, tx});
        __syncthreads();
    }
    float *out = p.seg_state + ((int64_t)hd.bh * p.nseg + seg) * p.N * p.P;
#pragma unroll
    for (int m = 0; m < TN; ++m)
#pragma unroll
        for (int n = 0; n < TP; ++n) {
            const int r = pairs(ty, m), q = pairs(tx, n);
            if (r < p.N && q < p.P) out[r * p.P + q] = S[m][n];
        }
    if (threadIdx.x == 0) p.seg_decay[(int64_t)hd.bh * p.nseg + seg] = exp2f((float)total);
}

template <int C, int NT, int PT>
__global__ void __launch_bounds__(kThreads) k_decay_fwd_gen(DecayParams p) {
    constexpr int PS = PT < 64 ? PT : 64;
    constexpr int LD = NT + 4, LP = PS + 4, LC = C + 4;
    constexpr int TM = C / 16, TN = NT / 16, TP = PS / 16;
    extern __shared__ float sm[];
    float *sc = sm, *sb = sc + C * LD, *sx = sb + C * LD, *sS = sx + C * LP, *sP = sS + NT * LP;
    float2 *sG = reinterpret_cast<float2 *>(sP + C * LC);
    const int seg = blockIdx.x % p.nseg;
    const int ps = (blockIdx.x / p.nseg) % p.pslices;
    const Head hd = head_of(p, blockIdx.x / p.nseg / p.pslices);
    const int p0 = ps * PS, pw = min(PS, p.P - p0);
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    const int64_t koff = hd.b * p.key_b + (hd.h / p.rep) * p.key_h;
    const int64_t voff = hd.b * p.val_b + hd.h * p.val_h + p0;
    const float *c = (const float *)p.c + koff, *b = (const float *)p.b + koff, *x = (const float *)p.x + voff;
    float *y = (float *)p.y + voff;
    const int64_t np = (int64_t)p.N * p.P;
    // these kernels have no bounded waits: the workspace's status is good
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;

    // the segment's incoming state
    const float *in = p.nseg > 1 ? p.seg_state + ((int64_t)hd.bh * p.nseg + seg) * np
                                 : (p.h0 ? p.h0 + (int64_t)hd.bh * np : nullptr);
    for (int e = threadIdx.x; e < NT * PS; e += kThreads) {
        const int n = e / PS, q = e % PS;
        sS[n * LP + q] = (in && n < p.N && q < pw) ? in[(int64_t)n * p.P + p0 + q] : 0.f;
    }
    const int c0 = seg * p.seg_chunks, c1 = min(c0 + p.seg_chunks, p.nchunks);
    Rows<C, NT> rc, rb;
    Rows<C, PS> rx;
    Steps<C> rl;
    auto fetch = [&](int i) {
        const int64_t t0 = i < c1 ? (int64_t)i * C : hd.len;
        rc.fetch(c, p.key_t, p.N, t0, hd.len);
        rb.fetch(b, p.key_t, p.N, t0, hd.len);
        rx.fetch(x, p.val_t, pw, t0, hd.len);
        rl.fetch(p, hd, t0);
    };
    fetch(c0);
    for (int i = c0; i < c1; ++i) {
        const int64_t t0 = (int64_t)i * C;
        __syncthreads();
        if (t0 < hd.len) {
            rc.put(sc);
            rb.put(sb);
            rx.put(sx);
            rl.sums(sG);
            fetch(i + 1);
        }
        if (p.carry && i > 0) {
            float *out = p.carry + ((int64_t)hd.bh * p.nchunks + i) * np + p0;
            for (int e = threadIdx.x; e < NT * PS; e += kThreads) {
                const int n = e / PS, q = e % PS;
                if (n < p.N && q < pw) out[(int64_t)n * p.P + q] = sS[n * LP + q];
            }
        }
        if (t0 >= hd.len) {             // behind the end: y is zero, the state stays
            for (int e = threadIdx.x; e < C * PS; e += kThreads) {
                const int64_t t = t0 + e / PS;
                if (t < p.L && e % PS < pw) y[t * p.val_t + e % PS] = 0.f;
            }
            continue;
        }
        __syncthreads();
        const float2 end = sG[C - 1];
        {
            float acc[TM][TM];
            zero(acc);
            tile_mm(acc, NT, Along<TM, true>{sc, LD, ty}, Along<TM, false>{sb, LD, tx});
#pragma unroll
            for (int m = 0; m < TM; ++m)
#pragma unroll
                for (int n = 0; n < TM; ++n) {
                    const int r = pairs(ty, m), q = strided(tx, n);
                    sP[r * LC + q] = q <= r ? acc[m][n] * decay_between(sG[r], sG[q]) : 0.f;
                }
        }
        __syncthreads();
        {
            float acc[TM][TP];
            zero(acc);
            tile_mm(acc, NT, Along<TM, true>{sc, LD, ty}, Across<TP>{sS, LP, tx});
#pragma unroll
            for (int m = 0; m < TM; ++m) {
                const float e = decay_from_start(sG[pairs(ty, m)]);
#pragma unroll
                for (int n = 0; n < TP; ++n) acc[m][n] *= e;
            }
            tile_mm(acc, C, Along<TM, true>{sP, LC, ty}, Across<TP>{sx, LP, tx});
#pragma unroll
            for (int m = 0; m < TM; ++m) {
                const int64_t t = t0 + pairs(ty, m);
#pragma unroll
                for (int n = 0; n < TP; ++n)
                    if (t < p.L && pairs(tx, n) < pw)
                        y[t * p.val_t + pairs(tx, n)] = t < hd.len ? acc[m][n] : 0.f;
            }
        }
        for (int e = threadIdx.x; e < C * NT; e += kThreads)
            sb[(e / NT) * LD + e % NT] *= decay_between(end, sG[e / NT]);
        __syncthreads();
        {
            float acc[TN][TP];
            zero(acc);
            tile_mm(acc, C, Across<TN>{sb, LD, ty}, Across<TP>{sx, LP, tx});
            const float a = decay_from_start(end);
#pragma unroll
            for (int m = 0; m < TN; ++m)
#pragma unroll
                for (int n = 0; n < TP; ++n) {
                    float *s = &sS[pairs(ty, m) * LP + pairs(tx, n)];
                    *s = fmaf(a, *s, acc[m][n]);
                }
        }
    }
    __syncthreads();
    if (p.h_last && seg == p.nseg - 1) {
        float *out = p.h_last + (int64_t)hd.bh * np + p0;
        for (int e = threadIdx.x; e < NT * PS; e += kThreads) {
            const int n = e / PS, q = e % PS;
            if (n < p.N && q < pw) out[(int64_t)n * p.P + q] = sS[n * LP + q];
        }
    }
}

// Adjoint of one segment's chunks in reverse; sR is dl/dS at the chunk's end.
template <int C, int NT, int PT>
__global__ void __launch_bounds__(kThreads) k_decay_bwd_gen(DecayParams p) {
    constexpr int LN = NT + 4, LP = PT + 4, LC = C + 4, TM = C / 16, TN = NT / 16, TP = PT / 16;
    extern __shared__ float sm[];
    float *sc = sm, *sb = sc + C * LN, *sx = sb + C * LN, *sg = sx + C * LP, *sR = sg + C * LP;
    float *sS = sR + NT * LP, *sP = sS + NT * LP, *sQ = sP + C * LC;
    float *sfrom = sQ + C * LC, *sto = sfrom + C;       // per step: pairs' and states' sums
    float *sred = sto + C;                              // 16 x C + 32
    float2 *sG = reinterpret_cast<float2 *>(sred + 16 * C + 32);
    const int seg = blockIdx.x % p.nseg;
    const Head hd = head_of(p, blockIdx.x / p.nseg);
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    const int64_t koff = hd.b * p.key_b + (hd.h / p.rep) * p.key_h;
    const int64_t voff = hd.b * p.val_b + hd.h * p.val_h;
    const float *c = (const float *)p.c + koff, *b = (const float *)p.b + koff;
    const float *x = (const float *)p.x + voff, *gy = (const float *)p.g_y + voff;
    float *gx = (float *)p.g_x + voff;
    const int64_t np = (int64_t)p.N * p.P;
    float *gla = p.g_la + hd.b * p.gla_b + hd.h * p.gla_h;
    // gradients of shared keys go to fp32 [B][H][L][N] partials
    const bool part = p.rep > 1;
    const int64_t poff = (int64_t)hd.bh * p.L * p.N;

    const float *in = p.nseg > 1 ? p.seg_state + ((int64_t)hd.bh * p.nseg + seg) * np
                                 : (p.g_hlast ? p.g_hlast + (int64_t)hd.bh * np : nullptr);
    for (int e = threadIdx.x; e < NT * PT; e += kThreads) {
        const int n = e / PT, q = e % PT;
        sR[n * LP + q] = (in && n < p.N && q < p.P) ? in[(int64_t)n * p.P + q] : 0.f;
    }
    const int c0 = seg * p.seg_chunks, c1 = min(c0 + p.seg_chunks, p.nchunks);
    Rows<C, NT> rc, rb;
    Rows<C, PT> rx, rg;
    Steps<C> rl;
    auto fetch = [&](int i) {
        const int64_t t0 = i >= c0 ? (int64_t)i * C : hd.len;
        rc.fetch(c, p.key_t, p.N, t0, hd.len);
        rb.fetch(b, p.key_t, p.N, t0, hd.len);
        rx.fetch(x, p.val_t, p.P, t0, hd.len);
        rg.fetch(gy, p.val_t, p.P, t0, hd.len);
        rl.fetch(p, hd, t0);
    };
    constexpr bool kAhead = NT + PT <= 192; // wider rows would not fit the registers
    if (kAhead) fetch(c1 - 1);
    for (int i = c1 - 1; i >= c0; --i) {
        const int64_t t0 = (int64_t)i * C;
        __syncthreads();
        const bool live = t0 < hd.len;
        if (!kAhead && live) fetch(i);
        if (live) {
            rc.put(sc);
            rb.put(sb);
            rx.put(sx);
            rg.put(sg);
            const float *S0 = i > 0 ? p.carry + ((int64_t)hd.bh * p.nchunks + i) * np
                                    : (p.h0 ? p.h0 + (int64_t)hd.bh * np : nullptr);
#pragma unroll 4
            for (int e = threadIdx.x; e < NT * PT; e += kThreads) {
                const int n = e / PT, q = e % PT;
                sS[n * LP + q] = S0 && n < p.N && q < p.P ? S0[(int64_t)n * p.P + q] : 0.f;
            }
            rl.sums(sG);
        }
        if (kAhead) fetch(i - 1);
        if (!live) {                    // behind the end: zero gradients, the state's stays
            constexpr int W = NT > PT ? NT : PT;
            for (int e = threadIdx.x; e < C * W; e += kThreads) {
                const int64_t t = t0 + e / W;
                const int q = e % W;
                if (t >= p.L) continue;
                if (q < p.P) gx[t * p.val_t + q] = 0.f;
                if (q < p.N) {
                    if (part) {
                        ((float *)p.g_c)[poff + t * p.N + q] = 0.f;
                        ((float *)p.g_b)[poff + t * p.N + q] = 0.f;
                    } else {
                        ((float *)p.g_c)[koff + t * p.key_t + q] = 0.f;
                        ((float *)p.g_b)[koff + t * p.key_t + q] = 0.f;
                    }
                }
                if (q == 0) gla[t * p.gla_t] = 0.f;
            }
            continue;
        }
        __syncthreads();
        const float2 end = sG[C - 1];
        const float aend = decay_from_start(end);
        // decayed scores P and Q, and the pair products' row and column sums
        {
            float s[TM][TM], v[TM][TM];
            zero(s);
            zero(v);
            tile_mm(s, NT, Along<TM, true>{sc, LN, ty}, Along<TM, false>{sb, LN, tx});
            tile_mm(v, PT, Along<TM, true>{sg, LP, ty}, Along<TM, false>{sx, LP, tx});
            float col[TM];
#pragma unroll
            for (int n = 0; n < TM; ++n) col[n] = 0.f;
#pragma unroll
            for (int m = 0; m < TM; ++m) {
                float row = 0.f;
#pragma unroll
                for (int n = 0; n < TM; ++n) {
                    const int r = pairs(ty, m), q = strided(tx, n);
                    const float d = q <= r ? decay_between(sG[r], sG[q]) : 0.f;
                    const float pv = q <= r ? s[m][n] * d : 0.f, qv = q <= r ? v[m][n] * d : 0.f;
                    sP[r * LC + q] = pv;
                    sQ[r * LC + q] = qv;
                    const float e = q < r ? pv * v[m][n] : 0.f;
                    row += e;
                    col[n] += e;
                }
                // the 16 threads of a row are half a warp
#pragma unroll
                for (int d = 8; d; d >>= 1) row += __shfl_xor_sync(kFull, row, d);
                if (tx == 0) sfrom[pairs(ty, m)] = row;
            }
#pragma unroll
            for (int n = 0; n < TM; ++n) sred[ty * C + strided(tx, n)] = col[n];
        }
        __syncthreads();
        for (int t = threadIdx.x; t < C; t += kThreads) {
            float s = 0.f;
            for (int r = 0; r < 16; ++r) s += sred[r * C + t];
            sto[t] = s;                 // sum over i > t of the pairs (i, t)
        }
        __syncthreads();
        // g_c: state part (kept for g_log_a), then the pairs
        float uc[TM], vb[TM];
        {
            float acc[TM][TN];
            zero(acc);
            tile_mm(acc, PT, Along<TM, true>{sg, LP, ty}, Along<TN, true>{sS, LP, tx});
#pragma unroll
            for (int m = 0; m < TM; ++m) {
                const float e = decay_from_start(sG[pairs(ty, m)]);
                uc[m] = 0.f;
#pragma unroll
                for (int n = 0; n < TN; ++n) {
                    acc[m][n] *= e;
                    uc[m] = fmaf(acc[m][n], sc[pairs(ty, m) * LN + pairs(tx, n)], uc[m]);
                }
            }
            tile_mm(acc, C, Along<TM, true>{sQ, LC, ty}, Across<TN>{sb, LN, tx});
#pragma unroll
            for (int m = 0; m < TM; ++m) {
                const int64_t t = t0 + pairs(ty, m);
#pragma unroll
                for (int n = 0; n < TN; ++n) {
                    const int q = pairs(tx, n);
                    if (t >= p.L || q >= p.N) continue;
                    const float v = t < hd.len ? acc[m][n] : 0.f;
                    if (part)
                        ((float *)p.g_c)[poff + t * p.N + q] = v;
                    else
                        ((float *)p.g_c)[koff + t * p.key_t + q] = v;
                }
            }
        }
        // g_b
        {
            float acc[TM][TN];
            zero(acc);
            tile_mm(acc, PT, Along<TM, true>{sx, LP, ty}, Along<TN, true>{sR, LP, tx});
#pragma unroll
            for (int m = 0; m < TM; ++m) {
                const float w = decay_between(end, sG[pairs(ty, m)]);
                vb[m] = 0.f;
#pragma unroll
                for (int n = 0; n < TN; ++n) {
                    acc[m][n] *= w;
                    vb[m] = fmaf(acc[m][n], sb[pairs(ty, m) * LN + pairs(tx, n)], vb[m]);
                }
            }
            tile_mm(acc, C, Across<TM>{sQ, LC, ty}, Across<TN>{sc, LN, tx});
#pragma unroll
            for (int m = 0; m < TM; ++m) {
                const int64_t t = t0 + pairs(ty, m);
#pragma unroll
                for (int n = 0; n < TN; ++n) {
                    const int q = pairs(tx, n);
                    if (t >= p.L || q >= p.N) continue;
                    const float v = t < hd.len ? acc[m][n] : 0.f;
                    if (part)
                        ((float *)p.g_b)[poff + t * p.N + q] = v;
                    else
                        ((float *)p.g_b)[koff + t * p.key_t + q] = v;
                }
            }
        }
        // g_x
        {
            float acc[TM][TP];
            zero(acc);
            tile_mm(acc, NT, Along<TM, true>{sb, LN, ty}, Across<TP>{sR, LP, tx});
#pragma unroll
            for (int m = 0; m < TM; ++m) {
                const float w = decay_between(end, sG[pairs(ty, m)]);
#pragma unroll
                for (int n = 0; n < TP; ++n) acc[m][n] *= w;
            }
            tile_mm(acc, C, Across<TM>{sP, LC, ty}, Across<TP>{sg, LP, tx});
#pragma unroll
            for (int m = 0; m < TM; ++m) {
                const int64_t t = t0 + pairs(ty, m);
#pragma unroll
                for (int n = 0; n < TP; ++n)
                    if (t < p.L && pairs(tx, n) < p.P)
                        gx[t * p.val_t + pairs(tx, n)] = t < hd.len ? acc[m][n] : 0.f;
            }
        }
        // e^{G_C} <S0, R>, the row sums u_i + R_i and v_j
        float dot = 0.f;
        for (int e = threadIdx.x; e < NT * PT; e += kThreads)
            dot = fmaf(sS[(e / PT) * LP + e % PT], sR[(e / PT) * LP + e % PT], dot);
#pragma unroll
        for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(kFull, dot, d);
#pragma unroll
        for (int m = 0; m < TM; ++m)
#pragma unroll
            for (int d = 8; d; d >>= 1) {
                uc[m] += __shfl_xor_sync(kFull, uc[m], d);
                vb[m] += __shfl_xor_sync(kFull, vb[m], d);
            }
        __syncthreads();                // sR and the column sums have been read
        if (threadIdx.x % 32 == 0) sred[16 * C + threadIdx.x / 32] = dot;
        if (tx == 0)
#pragma unroll
            for (int m = 0; m < TM; ++m) {
                sred[pairs(ty, m)] = uc[m];
                sred[C + pairs(ty, m)] = vb[m];
            }
        for (int e = threadIdx.x; e < C * NT; e += kThreads)
            sc[(e / NT) * LN + e % NT] *= decay_from_start(sG[e / NT]);
        __syncthreads();
        if (threadIdx.x < 32) {
            // g_log_a[t] = sum_{i>=t} (row_i + u_i - col_i) + sum_{j<t} v_j + e^{G_C} <S0, R>
            const int lane = threadIdx.x;
            double through = 0.0;
            for (int w = 0; w < kThreads / 32; ++w) through += (double)sred[16 * C + w];
            through *= (double)aend;
            double before = 0.0, total = 0.0;
            double inc[C / 32], pre[C / 32];
#pragma unroll
            for (int q = 0; q < C / 32; ++q) {
                const int t = q * 32 + lane;
                double a = (double)sfrom[t] + (double)sred[t] - (double)sto[t];
                double v = (double)sred[C + t];
                const double a0 = a, v0 = v;
#pragma unroll
                for (int d = 1; d < 32; d *= 2) {
                    const double oa = shfl_up_d(a, d), ov = shfl_up_d(v, d);
                    if (lane >= d) {
                        a += oa;
                        v += ov;
                    }
                }
                inc[q] = total + a - a0;        // sum over i < t
                pre[q] = before + v - v0;
                total += __shfl_sync(kFull, a, 31);
                before += __shfl_sync(kFull, v, 31);
            }
#pragma unroll
            for (int q = 0; q < C / 32; ++q) {
                const int64_t t = t0 + q * 32 + lane;
                if (t < p.L)
                    // a floored decay is a constant: its gradient is zero, and
                    // not what rounding leaves of the cancelled pairs
                    gla[t * p.gla_t] = t < hd.len && !(hd.log_a(p, t) <= (float)kDecayFloor)
                                           ? (float)(total - inc[q] + pre[q] + through)
                                           : 0.f;
            }
        }
        {
            float acc[TN][TP];
            zero(acc);
            tile_mm(acc, C, Across<TN>{sc, LN, ty}, Across<TP>{sg, LP, tx});
#pragma unroll
            for (int m = 0; m < TN; ++m)
#pragma unroll
                for (int n = 0; n < TP; ++n) {
                    float *s = &sR[pairs(ty, m) * LP + pairs(tx, n)];
                    *s = fmaf(aend, *s, acc[m][n]);
                }
        }
    }
    __syncthreads();
    if (p.g_h0 && seg == 0) {
        float *out = p.g_h0 + (int64_t)hd.bh * np;
        for (int e = threadIdx.x; e < NT * PT; e += kThreads) {
            const int n = e / PT, q = e % PT;
            if (n < p.N && q < p.P) out[(int64_t)n * p.P + q] = sR[n * LP + q];
        }
    }
}

// Joins the segments: seg_state[s] becomes the state that enters segment s
// (from its left, or, reversed, its right), starting from `first`.
__global__ void k_decay_join(DecayParams p, const float *first, int reverse) {
    const int64_t np = (int64_t)p.N * p.P;
    const int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (e >= (int64_t)p.B * p.H * np) return;
    const int64_t bh = e / np, i = e % np;
    float s = first ? first[e] : 0.f;
    // the loads of several segments on their way at once
    constexpr int kAhead = 8;
    for (int q0 = 0; q0 < p.nseg; q0 += kAhead) {
        float loc[kAhead], a[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int q = q0 + k, seg = reverse ? p.nseg - 1 - q : q;
            loc[k] = q < p.nseg ? p.seg_state[(bh * p.nseg + seg) * np + i] : 0.f;
            a[k] = q < p.nseg ? p.seg_decay[bh * p.nseg + seg] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int q = q0 + k, seg = reverse ? p.nseg - 1 - q : q;
            if (q >= p.nseg) break;
            p.seg_state[(bh * p.nseg + seg) * np + i] = s;
            s = fmaf(a[k], s, loc[k]);
        }
    }
}

// g_c, g_b of shared keys: the sum over their heads, in head order.
template <typename T>
__global__ void k_decay_sum_heads(DecayParams p, const float *part_c, const float *part_b, T *g_c,
                                  T *g_b) {
    const int64_t n = (int64_t)p.B * p.G * p.L * p.N;
    for (int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; e < n;
         e += (int64_t)gridDim.x * blockDim.x) {
        const int64_t j = e % p.N, t = e / p.N % p.L, g = e / p.N / p.L % p.G,
                      b = e / p.N / p.L / p.G;
        const int64_t from = ((b * p.H + g * p.rep) * p.L + t) * p.N + j;
        float sc = 0.f, sb = 0.f;
        for (int r = 0; r < p.rep; ++r) {
            sc += part_c[from + (int64_t)r * p.L * p.N];
            sb += part_b[from + (int64_t)r * p.L * p.N];
        }
        const int64_t to = b * p.okey_b + g * p.okey_h + t * p.okey_t + j;
        g_c[to] = from_f<T>(sc);
        g_b[to] = from_f<T>(sb);
    }
}

// g_log_a of a per-head decay: the sum over (b, t), one CTA per head, in fp64
// (steps of opposite sign cancel over a long sequence).
__global__ void __launch_bounds__(1024) k_decay_sum_steps(DecayParams p, const float *part,
                                                          float *g_log_a) {
    __shared__ double red[32];
    const int h = blockIdx.x;
    double s = 0.0;
    for (int b = 0; b < p.B; ++b) {
        const float *row = part + ((int64_t)b * p.H + h) * p.L;
#pragma unroll 4
        for (int64_t t = threadIdx.x; t < p.L; t += blockDim.x) s += (double)row[t];
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(kFull, s, d);
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        double t = 0.0;
        for (int w = 0; w < (int)blockDim.x / 32; ++w) t += red[w];
        g_log_a[h] = (float)t;
    }
}

// Rows to rows of whole 16 bytes, zero behind the width.  A thread makes 16
// bytes.
__global__ void k_decay_pad(DecayPad t0, DecayPad t1, DecayPad t2) {
    const DecayPad &t = blockIdx.y == 0 ? t0 : blockIdx.y == 1 ? t1 : t2;
    const int q8 = (t.width + 7) / 8;
    const int64_t n = t.rows * q8;
    for (int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; e < n;
         e += (int64_t)gridDim.x * blockDim.x) {
        const int64_t row = e / q8;
        const int q = 8 * (int)(e - row * q8);
        const unsigned short *src = (const unsigned short *)t.src + row * t.width + q;
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (q + j < t.width) w[j / 2] |= (uint32_t)__ldg(src + j) << (16 * (j % 2));
        reinterpret_cast<uint4 *>(t.dst)[e] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// and back.  A thread makes 8 values, 16 bytes where the result's address and
// end allow it.
__global__ void k_decay_unpad(const unsigned short *padded, unsigned short *out, int64_t rows, int width,
                              int vec) {
    const int w8 = (width + 7) / 8 * 8;
    const int64_t n = rows * width;
    for (int64_t e = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * 8; e < n;
         e += (int64_t)gridDim.x * blockDim.x * 8) {
        const int64_t row = e / width;
        int col = (int)(e - row * width);
        const unsigned short *src = padded + row * w8;
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (e + j < n) w[j / 2] |= (uint32_t)__ldg(src + col) << (16 * (j % 2));
            if (++col == width) {
                col = 0;
                src += w8;
            }
        }
        if (vec && e + 8 <= n) {
            *reinterpret_cast<uint4 *>(out + e) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (e + j < n) out[e + j] = (unsigned short)(w[j / 2] >> (16 * (j % 2)));
        }
    }
}

template <void (*KERN)(DecayParams)>
cudaError_t launch(int64_t grid, size_t smem, cudaStream_t st, const DecayParams &p) {
    static std::atomic<int> set[kLimitDevices];
    const cudaError_t e = allow_smem((const void *)KERN, (int)smem, set);
    if (e != cudaSuccess) return e;
    KERN<<<dim3((unsigned)grid), kThreads, smem, st>>>(p);
    return cudaGetLastError();
}

template <int NT, int PT, bool REV>
cudaError_t seg_gen(const DecayParams &p, cudaStream_t st) {
    const size_t smem = (size_t)(kC * (NT + PT + 8) + 2 * kC) * 4;
    return launch<k_decay_seg_gen<kC, NT, PT, REV>>((int64_t)p.B * p.H * p.nseg, smem, st, p);
}

template <int NT, int PT>
struct Fwd {
    static cudaError_t run(const DecayParams &p, cudaStream_t st) {
        constexpr int PS = PT < 64 ? PT : 64;
        if (p.nseg > 1) {
            cudaError_t e = seg_gen<NT, PT, false>(p, st);
            if (e != cudaSuccess) return e;
            e = launch_decay_join(p, p.h0, false, st);
            if (e != cudaSuccess) return e;
        }
        const size_t smem =
            (size_t)(2 * kC * (NT + 4) + (kC + NT) * (PS + 4) + kC * (kC + 4) + 2 * kC) * 4;
        return launch<k_decay_fwd_gen<kC, NT, PT>>((int64_t)p.B * p.H * p.nseg * p.pslices, smem, st, p);
    }
};

template <int NT, int PT>
struct Bwd {
    static cudaError_t run(const DecayParams &p, cudaStream_t st) {
        if (p.nseg > 1) {
            cudaError_t e = seg_gen<NT, PT, true>(p, st);
            if (e != cudaSuccess) return e;
            e = launch_decay_join(p, p.g_hlast, true, st);
            if (e != cudaSuccess) return e;
        }
        const size_t smem = (size_t)(2 * kC * (NT + PT + 8) + 2 * NT * (PT + 4) + 2 * kC * (kC + 4) +
                                     2 * kC + 16 * kC + 32 + 2 * kC) * 4;
        return launch<k_decay_bwd_gen<kC, NT, PT>>((int64_t)p.B * p.H * p.nseg, smem, st, p);
    }
};

// the widths in shared memory: N and P rounded up to 32, 64 or 128 each
template <template <int, int> class WHAT, int NT>
cudaError_t by_p(const DecayParams &p, cudaStream_t st) {
    if (p.P <= 32) return WHAT<NT, 32>::run(p, st);
    if (p.P <= 64) return WHAT<NT, 64>::run(p, st);
    return WHAT<NT, 128>::run(p, st);
}
template <template <int, int> class WHAT>
cudaError_t by_widths(const DecayParams &p, cudaStream_t st) {
    if (p.N <= 32) return by_p<WHAT, 32>(p, st);
    if (p.N <= 64) return by_p<WHAT, 64>(p, st);
    return by_p<WHAT, 128>(p, st);
}

}  // namespace

cudaError_t launch_decay_join(const DecayParams &p, const float *first, bool reverse,
                              cudaStream_t st) {
    const int64_t n = (int64_t)p.B * p.H * p.N * p.P;
    k_decay_join<<<dim3((unsigned)((n + 127) / 128)), 128, 0, st>>>(p, first, reverse ? 1 : 0);
    return cudaGetLastError();
}

cudaError_t launch_decay_sum_heads(const DecayParams &p, pdssm_dtype dt, const float *part_c,
                                   const float *part_b, void *g_c, void *g_b, cudaStream_t st) {
    const int64_t n = (int64_t)p.B * p.G * p.L * p.N;
    const unsigned grid = (unsigned)imin64((n + 255) / 256, (int64_t)kDecaySMs * 16);
    if (dt == PDSSM_BF16)
        k_decay_sum_heads<__nv_bfloat16><<<grid, 256, 0, st>>>(
            p, part_c, part_b, (__nv_bfloat16 *)g_c, (__nv_bfloat16 *)g_b);
    else
        k_decay_sum_heads<float><<<grid, 256, 0, st>>>(p, part_c, part_b, (float *)g_c,
                                                       (float *)g_b);
    return cudaGetLastError();
}

cudaError_t launch_decay_pad(const DecayPad *t, int count, cudaStream_t st) {
    if (count < 1) return cudaSuccess;
    int64_t most = 0;
    for (int i = 0; i < count; ++i) {
        const int64_t n = t[i].rows * ((t[i].width + 7) / 8);
        most = n > most ? n : most;
    }
    const dim3 grid((unsigned)imin64((most + 255) / 256, (int64_t)kDecaySMs * 32), (unsigned)count);
    k_decay_pad<<<grid, 256, 0, st>>>(t[0], t[count > 1 ? 1 : 0], t[count > 2 ? 2 : 0]);
    return cudaGetLastError();
}

cudaError_t launch_decay_unpad(const void *padded, void *out, int64_t rows, int width, cudaStream_t st) {
    const int64_t n = (rows * width + 7) / 8;
    k_decay_unpad<<<dim3((unsigned)imin64((n + 255) / 256, (int64_t)kDecaySMs * 32)), 256, 0, st>>>(
        (const unsigned short *)padded, (unsigned short *)out, rows, width, ((uintptr_t)out & 15) == 0);
    return cudaGetLastError();
}

cudaError_t launch_decay_sum_steps(const DecayParams &p, const float *part, float *g_log_a,
                                   cudaStream_t st) {
    k_decay_sum_steps<<<p.H, 1024, 0, st>>>(p, part, g_log_a);
    return cudaGetLastError();
}

cudaError_t launch_decay_fwd_gen(const DecayParams &p, cudaStream_t st) {
    return by_widths<Fwd>(p, st);
}

cudaError_t launch_decay_bwd_gen(const DecayParams &p, cudaStream_t st) {
    return by_widths<Bwd>(p, st);
}

}  // namespace pdssm
