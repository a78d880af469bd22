// Balance loss of the hard selection for bf16 u on the tensor cores (tcgen05).
//
// A group is as many heads as fill N = 128 entries (64 above D = 128; a head
// takes K entries rounded up to a power of two).  Its weights lie in shared
// memory as three bf16 parts (8 + 8 + 8 bits of fp32), so that the logits
//     L = u W^T            128 rows x N, K = D, three products
// have fp32 accuracy (u is bf16 by itself; g_u takes two parts); the small parts
// are multiplied first, since a product's additions truncate the sum so far.
// Sixteen warps (N = 64: eight) take a finished L from TMEM, a row and 32 of its
// columns per thread: softmax per head, then
//   sums    column sums of p over the rows, in registers over the CTA's tiles;
//           counts by shared-memory atomics (integers)
//   g_u     G, the logits' gradients, back to TMEM as bf16, and
//           g_u += G W  (K = N; W's first two parts: G's rounding to bf16 is
//           then the only one besides g_u's own: 2.35e-3 of its norm off, by its
//           own rounding alone 1.66e-3), over the groups
//   g_W     G as three bf16 parts to shared memory (two, then the largest), and
//           g_W += G^T u  (K = 128 rows), a tile's in TMEM, the CTA's tiles'
//           added up in registers (a product's own additions truncate: over
//           a CTA's 14 tiles that cost 5.6e-6 of g_W's norm)
// L is double-buffered: the next tile's products run under this one's softmax.
//
// Bound: the chain of a tile through the roles (copy, logits, softmax, second
// product); the products alone take a third of the time, and leaving two of the
// three parts out of the logits saves 20 % of the sums, 4 % of g_W.  u is read
// once per group (from L2 after the first).  8 x 16384 steps, 16 heads of 16
// entries, D = 128: sums 36 us, g_u 56, g_W 86 (one issuing thread and eight
// softmax warps: 40, 70, 93).
#include <string.h>

#include "balance.cuh"
#include "launch.cuh"
#include "tile_bf16.cuh"
#include "umma.cuh"

namespace pdssm {
namespace {

enum { kSums = 0, kGu = 1, kGw = 2 };
// W's parts that a kernel takes: the loss, the probabilities and g_W are fp32;
// g_u is bf16, and 16 bits of W move its logits by 1e-5 of them at most
__host__ __device__ constexpr int parts_of(int mode) { return mode == kGu ? 2 : 3; }
// softmax warps of a group of N entries: 4 by rows times N / 32 by entries
__host__ __device__ constexpr int epi_of(int N) { return N / 8; }
constexpr int kRows = 128;

enum { kUFull, kWFull, kLFull, kGReady, kGHalf, kGThird, kDone, kGuFull, kGuFree, kBars };

struct TcP {
    BalParams p;
    BalTcPlan pl;
    const unsigned char *parts;                 // [groups][3][Dp/64][N][128 bytes], swizzled
    const float *freq;                          // excess counts / T [groups * N], then per head the
                                                // factor g_loss K inv_tau / T
    int vec;
    int nslot, ustages;                         // of W, of u
    uint32_t o_u, o_g, o_tab, o_bar;            // shared-memory offsets (weights at 0)
};

// Softmax of the heads in 32 columns, logits in units of log2 e / tau applied
// here; columns of absent entries (k >= K) get 0.
template <int KT>
__device__ __forceinline__ void softmax32(float (&v)[32], int K, float scale, bool live) {
#pragma unroll
    for (int h = 0; h < 32 / KT; ++h) {
        float *x = v + h * KT;
        float m = x[0];
#pragma unroll
        for (int k = 1; k < KT; ++k)
            if (k < K) m = fmaxf(m, x[k]);
        float z = 0.f;
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            x[k] = k < K ? ex2((x[k] - m) * scale) : 0.f;
            z += x[k];
        }
        const float inv = live ? 1.f / z : 0.f;
#pragma unroll
        for (int k = 0; k < KT; ++k) x[k] = live ? x[k] * inv : 0.f;
    }
}

// and two that issue products (a thread takes 100 to 200 cycles for each), one
// for copies
__host__ __device__ constexpr int threads_of(int N) { return (epi_of(N) + 3) * 32; }

template <int KT, int MODE, int N>
__global__ void __launch_bounds__(threads_of(N), 1)
    k_bal_tc(const __grid_constant__ CUtensorMap umap, const TcP t) {
    constexpr int kEpi = epi_of(N), kTh = threads_of(N);
    constexpr int kBlocks = N / 32;                             // of 32 entries
    const BalParams &p = t.p;
    const BalTcPlan &pl = t.pl;
    extern __shared__ unsigned char sm_raw[];
    const uint32_t sm = (smem_u32(sm_raw) + 1023u) & ~1023u;
    unsigned char *smg = sm_raw + (sm - smem_u32(sm_raw));
    __shared__ uint32_t tmem_slot;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int Dp = pl.Dp, atoms = Dp / 64;
    const uint32_t ubytes = (uint32_t)kRows * Dp * 2, wpart = (uint32_t)N * Dp * 2;
    constexpr int kParts = parts_of(MODE);
    const uint32_t wslotb = kParts * wpart;
    auto bar = [&](int which, int i) { return sm + t.o_bar + 8u * (uint32_t)(4 * which + (i & 3)); };
    bool ok = true;
    auto wait = [&](int which, int i) {
        return ok = ok && mbar_wait_hot(bar(which, i), (uint32_t)((i >> 2) & 1));
    };
    auto wait_warp = [&](int which, int i) { return ok = __all_sync(kFull, wait(which, i)); };

    // an item is a tile and a group: the CTA's group and every slices-th tile,
    // or (g_u) every group of every gridDim-th tile
    const int group0 = MODE == kGu ? 0 : blockIdx.x % pl.groups;
    const int ng = MODE == kGu ? pl.groups : 1;
    const int tile0 = MODE == kGu ? blockIdx.x : blockIdx.x / pl.groups;
    const int tstep = MODE == kGu ? gridDim.x : pl.slices;
    const int ntiles = tile0 < pl.tiles ? (pl.tiles - tile0 + tstep - 1) / tstep : 0;
    const int items = ntiles * ng;
    auto row0 = [&](int tile) { return (int64_t)(tile0 + tile * tstep) * kRows; };
    // W's slot of an item: resident when the groups fit, else a ring
    const bool resident = ng <= t.nslot;
    auto wslot = [&](int i) { return resident ? i % ng : i % t.nslot; };
    auto wait_w = [&](int i) {
        const int use = resident ? 0 : i / t.nslot;
        return ok = ok && mbar_wait_hot(bar(kWFull, wslot(i)), (uint32_t)(use & 1));
    };
    auto wait_u = [&](int tile) {
        return ok = ok && mbar_wait_hot(bar(kUFull, tile % t.ustages), (uint32_t)((tile / t.ustages) & 1));
    };

    if (tid == 0) {
        for (int s = 0; s < 4; ++s) {
            mbar_init(bar(kUFull, s), t.vec ? 1 : 32);
            mbar_init(bar(kWFull, s), 1);
            mbar_init(bar(kLFull, s), 1);
            mbar_init(bar(kGReady, s), 32 * kEpi);
            mbar_init(bar(kGHalf, s), 1);
            mbar_init(bar(kGThird, s), 32 * kEpi);
            mbar_init(bar(kDone, s), 1);
            mbar_init(bar(kGuFull, s), 1);
            mbar_init(bar(kGuFree, s), 32 * kEpi);
        }
        fence_mbar_init();
    }
    if (warp == kEpi) tmem_alloc(smem_u32(&tmem_slot), 512);
    int *cnt = reinterpret_cast<int *>(smg + t.o_tab);          // sums: [N]
    if (MODE == kSums)
        for (int e = tid; e < N; e += kTh) cnt[e] = 0;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    // TMEM: L 2 x 128 columns (g_u: G as bf16 in the first half of each 32),
    // then g_u or g_W, Dp columns
    auto tL = [&](int i) { return tmem + (uint32_t)(i & 1) * 128; };
    const uint32_t tAcc = tmem + 256;

    const float scale = p.inv_tau * 1.4426950408889634f;
    const int quad = warp & 3, block = warp >> 2, r = quad * 32 + lane;
    const int col0 = 32 * block;                                // this thread's entries
    const uint32_t tlane = (uint32_t)(quad * 32) << 16;

    if (warp < kEpi) {
        // sums: this thread's entries; g_W: one entry and a quarter of d (a group of
        // 64 entries lies in the lanes twice, so their second half takes others)
        constexpr int kAcc = MODE == kGu ? 1 : MODE == kGw && N == 64 ? 64 : 32;
        float acc[kAcc];
#pragma unroll
        for (int q = 0; q < kAcc; ++q) acc[q] = 0.f;
        const int we = N > 64 ? r : r & 63;
        const int wn = Dp / 4;
        const int wd = (N > 64 ? block : block * 2 + (r >> 6)) * wn;
        auto take = [&]() {         // the finished tile's g_W
            if constexpr (MODE == kGw) {
                tc_fence_after();
#pragma unroll
                for (int q = 0; q < kAcc / 16; ++q) {
                    if (16 * q >= wn) break;
                    uint32_t raw[16];
                    tmem_ld16_raw(tAcc + wd + 16 * q + tlane, raw);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e) acc[16 * q + e] += __uint_as_float(raw[e]);
                }
            }
        };
        for (int i = 0; i < items; ++i) {
            const int tile = i / ng, gi = i % ng;
            const int c0 = (group0 + gi) * N + col0;            // first entry of this thread
            const int64_t row = row0(tile) + r;
            const bool live = bal_live(p, row);
            // the selections of this thread's heads: on their way while the
            // products run
            constexpr int kHeads = MODE == kSums ? 32 / KT : 1;
            int sel[kHeads];
            if (MODE == kSums) {
                const uint32_t b = (uint32_t)row / (uint32_t)p.L, s = (uint32_t)row - b * (uint32_t)p.L;
                const int32_t *kr = p.k + ((int64_t)b * p.H + c0 / KT) * p.L + s;
#pragma unroll
                for (int h = 0; h < kHeads; ++h)
                    sel[h] = live && c0 / KT + h < p.H ? kr[(int64_t)h * p.L] : -1;
            }
            if (!wait_warp(kLFull, i)) break;
            tc_fence_after();
            if (MODE == kGw) {
                // the last tile's g_W is there, and the parts of its G have been read
                if (i > 0) {
                    if (!wait_warp(kDone, i - 1)) break;
                    take();
                }
                if (!live) {        // behind an end: u must not meet a zero gradient as a NaN
                    const uint32_t ut = sm + t.o_u + (uint32_t)(tile % t.ustages) * ubytes;
                    for (int a = block; a < atoms; a += kBlocks)
                        for (int q = 0; q < 8; ++q) sts128(ut + a * (kRows * 128) + piece(r, q), 0, 0, 0, 0);
                }
                __syncwarp();       // the loads below are the whole warp's
            }
            uint32_t third[MODE == kGw ? 16 : 1];
            {
                uint32_t raw[32];
                float v[32];
                tmem_ld32(tL(i) + col0 + tlane, raw);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(raw[e]);
                softmax32<KT>(v, p.K, scale, live);
                if constexpr (MODE == kSums) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) acc[e] += v[e];
                } else {
                    const float4 *tf = reinterpret_cast<const float4 *>(t.freq + c0);
                    const int heads = pl.groups * N / KT;
                    float fq[32];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float4 a = __ldg(tf + e);
                        fq[4 * e] = a.x;
                        fq[4 * e + 1] = a.y;
                        fq[4 * e + 2] = a.z;
                        fq[4 * e + 3] = a.w;
                    }
#pragma unroll
                    for (int h = 0; h < 32 / KT; ++h) {
                        const float by = __ldg(t.freq + heads * KT + c0 / KT + h);
                        float dot = 0.f;
#pragma unroll
                        for (int k = 0; k < KT; ++k) dot = fmaf(v[h * KT + k], fq[h * KT + k], dot);
#pragma unroll
                        for (int k = 0; k < KT; ++k)
                            v[h * KT + k] = by * v[h * KT + k] * (fq[h * KT + k] - dot);
                    }
                    if constexpr (MODE == kGu) {
                        uint32_t o[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = pack2(v[2 * e], v[2 * e + 1]);
                        tmem_st16(tL(i) + col0 + tlane, o);
                    } else {
                        // piece e of this row: entries col0 + 8 e
                        const uint32_t gt = sm + t.o_g;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t p1[4], p2[4];      // parts 1 and 2; the first goes last
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                float a = v[8 * e + 2 * k], b = v[8 * e + 2 * k + 1];
                                const uint32_t w = pack2(a, b);
                                third[4 * e + k] = w;
                                a -= lo_of(w);
                                b -= hi_of(w);
                                p1[k] = pack2(a, b);
                                p2[k] = pack2(a - lo_of(p1[k]), b - hi_of(p1[k]));
                            }
                            const int col = col0 + 8 * e;
                            const uint32_t at = gt + (uint32_t)(col / 64) * (kRows * 128) + piece(r, (col & 63) / 8);
                            sts128(at, p1[0], p1[1], p1[2], p1[3]);
                            sts128(at + (uint32_t)kRows * N * 2, p2[0], p2[1], p2[2], p2[3]);
                        }
                    }
                }
            }
            if (MODE == kSums) {
#pragma unroll
                for (int h = 0; h < kHeads; ++h)
                    if (sel[h] >= 0 && sel[h] < p.K)
                        atomicAdd(&cnt[col0 + h * KT + sel[h]], 1);
            }
            if (MODE == kGu) tmem_wait_st();
            if (MODE == kGw) fence_proxy_async_smem();
            tc_fence_before();
            mbar_arrive(bar(kGReady, i));
            if constexpr (MODE == kGw) {
                if (!wait_warp(kGHalf, i)) break;       // part 1's buffer has been read
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int col = col0 + 8 * e;
                    sts128(sm + t.o_g + (uint32_t)(col / 64) * (kRows * 128) + piece(r, (col & 63) / 8),
                           third[4 * e], third[4 * e + 1], third[4 * e + 2], third[4 * e + 3]);
                }
                fence_proxy_async_smem();
                mbar_arrive(bar(kGThird, i));
            }
            if (MODE == kGu && gi == ng - 1) {
                if (!wait_warp(kGuFull, tile)) break;
                tc_fence_after();
                __nv_bfloat16 *out = (__nv_bfloat16 *)p.g_u + row * p.D;
                const int dcols = Dp / kBlocks;
#pragma unroll 1
                for (int q = 0; q < dcols; q += 16) {
                    uint32_t raw[16];
                    float v[16];
                    tmem_ld16_raw(tAcc + block * dcols + q + tlane, raw);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] = live ? __uint_as_float(raw[e]) : 0.f;
                    const int col = block * dcols + q;
                    if (row < p.rows) {
                        if (t.vec) {
#pragma unroll
                            for (int e = 0; e < 16; e += 8)
                                if (col + e < p.D)
                                    *reinterpret_cast<uint4 *>(out + col + e) =
                                        make_uint4(pack2(v[e], v[e + 1]), pack2(v[e + 2], v[e + 3]),
                                                   pack2(v[e + 4], v[e + 5]), pack2(v[e + 6], v[e + 7]));
                        } else {
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                if (col + e < p.D) out[col + e] = __float2bfloat16_rn(v[e]);
                        }
                    }
                    __syncwarp();   // rows behind the last part ways: together again for the next load
                }
                tc_fence_before();
                mbar_arrive(bar(kGuFree, tile));
            }
        }
        if constexpr (MODE == kGw) {
            // g_W of the group over the CTA's tiles
            if (items > 0 && wait_warp(kDone, items - 1)) take();
            const int c = group0 * N + we, h = c / KT, k = c % KT;
            const int slice = blockIdx.x / pl.groups;
            const bool mine = h < p.H && k < p.K;
            float *out = p.part + (((int64_t)slice * p.H + h) * p.K + k) * p.D + wd;
#pragma unroll
            for (int e = 0; e < kAcc; ++e)
                if (mine && e < wn && wd + e < p.D) out[e] = acc[e];
        }
        if constexpr (MODE == kSums) {
            // column sums over the warp's rows
            float *red = reinterpret_cast<float *>(smg + t.o_g);        // [kEpi][32]
#pragma unroll
            for (int q = 0; q < 32; ++q) {
                float s = acc[q];
#pragma unroll
                for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(kFull, s, d);
                if (lane == 0) red[warp * 32 + q] = s;
            }
        }
    } else if (warp == kEpi || (MODE == kSums && warp == kEpi + 1)) {
        // ---- products: logits.  Sums: the two warps take items in turn, each with its
        // stage of u; with one stage (whose phases a warp must see one by one) the
        // first takes all
        const bool two = MODE == kSums && t.ustages > 1;
        if (lane == 0 && (two || warp == kEpi)) {
            const uint32_t idL = umma_idesc_bf16(N);
            const uint32_t w0 = umma_lo(sm, 16), u0 = umma_lo(sm + t.o_u, 16);
            int last = -1;
            for (int i = warp - kEpi; i < items; i += two ? 2 : 1) {
                const int tile = i / ng;
                // L's buffer: its columns have been read (g_u: its G has gone into the
                // second product).  Ahead of the wait for u: then every earlier copy has
                // landed, also those that the other warp waited for.
                if (i >= 2 && !wait(MODE == kGu ? kDone : kGReady, i - 2)) break;
                if (!wait_u(tile) || !wait_w(i)) break;
                tc_fence_after();
                const uint32_t ub = u0 + (uint32_t)(tile % t.ustages) * umma_step(ubytes);
                const uint32_t wb = w0 + (uint32_t)wslot(i) * umma_step(wslotb);
#pragma unroll 1
                for (int part = kParts - 1; part >= 0; --part)      // the small ones first
#pragma unroll 1
                    for (int a = 0; a < atoms; ++a) {
                        const uint32_t ar = ub + a * umma_step(kRows * 128);
                        const uint32_t br = wb + part * umma_step(wpart) + a * umma_step((uint32_t)N * 128);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            umma_ss(tL(i), ar + k * umma_step(32), br + k * umma_step(32), idL,
                                    part < kParts - 1 || a > 0 || k > 0);
                    }
                umma_commit(bar(kLFull, i));
                last = i;
            }
            if (last >= 0 && ok) wait(kLFull, last);    // nothing is in flight when the CTA ends
        }
        __syncwarp();
    } else if (warp == kEpi + 1) {
        // ---- products: what an item's G goes into
        if (lane == 0) {
            const uint32_t idU = umma_idesc_bf16(Dp, false, true), idW = umma_idesc_bf16(Dp, true, true);
            const uint32_t wmn0 = umma_lo(sm, (uint32_t)N * 128), umn0 = umma_lo(sm + t.o_u, kRows * 128);
            // the two 64-entry blocks of G (one: the same rows twice)
            const uint32_t g0 = umma_lo(sm + t.o_g, N > 64 ? kRows * 128 : 0);
            for (int j = 0; j < items; ++j) {
                const int tile = j / ng, gi = j % ng;
                if (!wait(kGReady, j)) break;
                if (MODE == kGu) {
                    if (gi == 0 && tile > 0 && !wait(kGuFree, tile - 1)) break;
                    tc_fence_after();
                    const uint32_t wb = wmn0 + (uint32_t)wslot(j) * umma_step(wslotb);
#pragma unroll 1
                    for (int part = 0; part < 2; ++part) {
                        // a block's 32 entries lie packed in its first 16 columns
#pragma unroll
                        for (int kb = 0; kb < kBlocks; ++kb) {
                            const uint32_t ar = tL(j) + kb * 32;
                            const uint32_t br = wb + part * umma_step(wpart) + kb * 2 * umma_step(2048);
                            umma_ts(tAcc, ar, br, idU, gi > 0 || part > 0 || kb > 0);
                            umma_ts(tAcc, ar + 8, br + umma_step(2048), idU, true);
                        }
                    }
                    if (gi == ng - 1) umma_commit(bar(kGuFull, tile));
                } else {
                    const uint32_t ub = umn0 + (uint32_t)(tile % t.ustages) * umma_step(ubytes);
#pragma unroll 1
                    for (int part = 0; part < 3; ++part) {      // parts 2, 1, 0 of G
                        if (part == 2) {
                            umma_commit(bar(kGHalf, j));
                            if (!wait(kGThird, j)) break;
                        }
                        tc_fence_after();
                        const uint32_t ar = g0 + (part == 0 ? umma_step((uint32_t)kRows * N * 2) : 0u);
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            umma_ss(tAcc, ar + k * umma_step(2048), ub + k * umma_step(2048), idW,
                                    part > 0 || k > 0);
                    }
                }
                if (!ok) break;
                umma_commit(bar(kDone, j));
            }
            if (items > 0 && ok) wait(kDone, items - 1);
        }
        __syncwarp();
    } else {
        // ---- copies: W's parts as they lie, u by tensor map or plain loads
        for (int i = 0; i < items && ok; ++i) {
            const int tile = i / ng, gi = i % ng;
            if (lane == 0) {
                const bool load = resident ? i < ng : true;
                if (load) {
                    if (!resident && i >= t.nslot) wait(kDone, i - t.nslot);
                    if (ok) {
                        const uint32_t wb = bar(kWFull, wslot(i));
                        const uint32_t bytes = wslotb;
                        mbar_expect_tx(wb, bytes);
                        const unsigned char *src = t.parts + (size_t)(group0 + gi) * pl.w_bytes;
                        for (uint32_t o = 0; o < bytes; o += 16384)
                            bulk_g2s(sm + (uint32_t)wslot(i) * bytes + o, src + o, min(16384u, bytes - o), wb);
                    }
                }
            }
            ok = __shfl_sync(kFull, (int)ok, 0) != 0;
            if (!ok) break;
            if (gi) continue;
            // a stage of u is free once its last reader is done
            if (tile >= t.ustages) {
                const int last = (tile - t.ustages) * ng + ng - 1;
                if (!wait_warp(MODE == kGw ? kDone : kLFull, last)) break;
            }
            const uint32_t ut = sm + t.o_u + (uint32_t)(tile % t.ustages) * ubytes;
            const uint32_t ub = bar(kUFull, tile % t.ustages);
            if (t.vec) {
                if (lane == 0) {
                    mbar_expect_tx(ub, ubytes);
                    for (int a = 0; a < atoms; ++a)
                        asm volatile(
                            "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
                            "[%0], [%1, {%2, %3}], [%4];" ::"r"(ut + a * (kRows * 128)),
                            "l"(reinterpret_cast<uint64_t>(&umap)), "r"(64 * a), "r"((int)row0(tile)), "r"(ub)
                            : "memory");
                }
                __syncwarp();
            } else {
                const unsigned short *u = reinterpret_cast<const unsigned short *>(p.u);
                for (int e = lane; e < kRows * atoms * 8; e += 32) {
                    const int rr = e / (atoms * 8), q = e % (atoms * 8);
                    const int64_t row = row0(tile) + rr;
                    uint32_t w[4] = {0, 0, 0, 0};
                    if (row < p.rows)
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (8 * q + j < p.D) w[j / 2] |= (uint32_t)u[row * p.D + 8 * q + j] << (16 * (j % 2));
                    sts128(ut + (q / 8) * (kRows * 128) + piece(rr, q % 8), w[0], w[1], w[2], w[3]);
                }
                fence_proxy_async_smem();
                mbar_arrive(ub);
            }
        }
    }
    tc_fence_before();
    const bool failed = __syncthreads_or(!ok);
    if (failed) {
        // a wait gave up: let copies and products in flight land, for a
        // millisecond at most, before the CTA ends
        const uint64_t s = global_ns();
        for (int it = 0; it < (1 << 20) && global_ns() - s < 1000000u; ++it) __nanosleep(1000);
        __syncthreads();
    }
    tc_fence_after();
    if (warp == kEpi) tmem_dealloc(tmem, 512);
    // a wait that gave up must not pass for a result
    const float nan = __int_as_float(0x7fffffff);
    if (MODE == kSums) {
        const float *red = reinterpret_cast<const float *>(smg + t.o_g);
        const int slice = blockIdx.x / pl.groups;
        for (int e = tid; e < N; e += kTh) {
            const int c = group0 * N + e, h = c / KT, k = c % KT;
            if (h >= p.H || k >= p.K) continue;
            const int w = e / 32 * 4, col = e % 32;
            const float s = (red[w * 32 + col] + red[(w + 1) * 32 + col]) +
                            (red[(w + 2) * 32 + col] + red[(w + 3) * 32 + col]);
            const int64_t at = ((int64_t)slice * p.H + h) * p.K + k;
            p.part[at] = failed ? nan : s;
            p.part_n[at] = cnt[e];
        }
    } else if (failed) {
        if (MODE == kGw) {
            for (int e = tid; e < N * p.D; e += kTh) {
                const int c = group0 * N + e / p.D, h = c / KT, k = c % KT;
                if (h < p.H && k < p.K)
                    p.part[(((int64_t)(blockIdx.x / pl.groups) * p.H + h) * p.K + k) * p.D + e % p.D] = nan;
            }
        } else {
            for (int tile = 0; tile < ntiles; ++tile)
                for (int64_t e = tid; e < (int64_t)kRows * p.D; e += kTh)
                    if (row0(tile) + e / p.D < p.rows)
                        ((__nv_bfloat16 *)p.g_u)[row0(tile) * p.D + e] = __float2bfloat16_rn(nan);
        }
    }
}

// W's three bf16 parts, per group in the shared-memory image of a K-major
// operand: [3][Dp / 64][N rows][128 bytes], 128-byte swizzle.
// With counts (backward) also the table of their excess and the heads' factors.
__global__ void k_bal_parts(BalParams p, BalTcPlan pl, unsigned char *parts, float *freq) {
    const int64_t n = (int64_t)pl.groups * pl.N * (pl.Dp / 2);
    const int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (e >= n) return;                 // n is a multiple of 2048: whole CTAs
    const int d = (int)(e % (pl.Dp / 2)) * 2;
    const int64_t c = e / (pl.Dp / 2);
    const int h = (int)(c / pl.KT), k = (int)(c % pl.KT);
    const int g = (int)(c / pl.N), row = (int)(c % pl.N);
    // d = 0 falls on a warp's first thread, since Dp / 2 is a multiple of 32
    if (p.counts && __shfl_sync(kFull, d, 0) == 0) {
        const int64_t steps = bal_steps(p);
        const float inv = steps > 0 ? 1.f / (float)steps : 0.f;
        if (d == 0) freq[c] = h < p.H && k < p.K ? bal_excess(p.counts[h * p.K + k], p.K, steps) : 0.f;
        if (d == 0 && k == 0)
            freq[(int64_t)pl.groups * pl.N + h] =
                h < p.H ? p.g_loss[h] * ((float)p.K * p.inv_tau) * inv : 0.f;
    }
    float a = 0.f, b = 0.f;
    if (h < p.H && k < p.K) {
        const float *w = p.W + ((int64_t)h * p.K + k) * p.D;
        if (d < p.D) a = w[d];
        if (d + 1 < p.D) b = w[d + 1];
    }
    unsigned char *out = parts + (size_t)g * pl.w_bytes + (size_t)(d / 64) * pl.N * 128 +
                         piece(row, (d & 63) / 8) + (d & 7) * 2;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const uint32_t w = pack2(a, b);
        a -= lo_of(w);
        b -= hi_of(w);
        *reinterpret_cast<uint32_t *>(out + (size_t)i * pl.N * pl.Dp * 2) = w;
    }
}

template <int KT, int MODE, int N>
cudaError_t go(const BalParams &p, const BalTcPlan &pl, const void *parts, cudaStream_t st) {
    TcP t;
    memset(&t, 0, sizeof(t));
    t.p = p;
    t.pl = pl;
    t.parts = (const unsigned char *)parts;
    t.freq = reinterpret_cast<const float *>(t.parts + (size_t)pl.groups * pl.w_bytes);
    const uint32_t u = (uint32_t)kRows * pl.Dp * 2, slot = parts_of(MODE) * (uint32_t)pl.N * pl.Dp * 2;
    t.nslot = 1;
    t.ustages = pl.Dp > 128 ? 1 : 2;
    if (MODE == kGu) {
        // as many groups' weights as fit (at most four slots); two stages of u where
        // they fit too and a tile has at most three groups (a barrier's slots
        // come round after four)
        const uint32_t room = 227 * 1024 - 2048;
        t.nslot = pl.groups < 4 ? pl.groups : 4;
        while (t.nslot > 1 && t.nslot * slot + u > room) --t.nslot;
        t.ustages = pl.groups <= 3 && t.nslot * slot + 2 * u <= room ? 2 : 1;
    }
    uint32_t o = t.nslot * slot;
    t.o_u = o; o += t.ustages * u;
    t.o_g = o; o += MODE == kGw ? 2u * kRows * pl.N * 2 : MODE == kSums ? epi_of(N) * 32 * 4 : 0;
    t.o_tab = o; o += MODE == kSums ? pl.N * 4 : 0;
    t.o_bar = o; o += 32 * kBars;
    const int smem = (int)o + 1024;
    t.vec = p.D % 8 == 0 && ((uintptr_t)p.u % 16) == 0 && ((uintptr_t)p.g_u % 16) == 0 &&
            p.rows > 0 && tensor_map_encoder() != nullptr;
    CUtensorMap map;
    memset(&map, 0, sizeof(map));
    if (t.vec) {
        const cuuint64_t gdim[2] = {(cuuint64_t)p.D, (cuuint64_t)p.rows};
        const cuuint64_t gstride[1] = {(cuuint64_t)p.D * 2};
        const cuuint32_t box[2] = {64u, (cuuint32_t)kRows};
        const cuuint32_t es[2] = {1, 1};
        if (tensor_map_encoder()(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(p.u), gdim,
                                 gstride, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                 CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                                 CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    auto kern = k_bal_tc<KT, MODE, N>;
    static std::atomic<int> set[kLimitDevices];
    const cudaError_t e = allow_smem((const void *)kern, smem, set);
    if (e != cudaSuccess) return e;
    const int grid = MODE == kGu ? (pl.tiles < 148 ? pl.tiles : 148) : pl.groups * pl.slices;
    kern<<<grid, threads_of(N), smem, st>>>(map, t);
    return cudaGetLastError();
}

template <int KT, int N>
cudaError_t go_n(const BalParams &p, const BalTcPlan &pl, int what, const void *parts, cudaStream_t st) {
    if (what == kSums) return go<KT, kSums, N>(p, pl, parts, st);
    if (what == kGu) return go<KT, kGu, N>(p, pl, parts, st);
    return go<KT, kGw, N>(p, pl, parts, st);
}

template <int KT>
cudaError_t go_k(const BalParams &p, const BalTcPlan &pl, int what, const void *parts, cudaStream_t st) {
    return pl.N == 128 ? go_n<KT, 128>(p, pl, what, parts, st) : go_n<KT, 64>(p, pl, what, parts, st);
}

}  // namespace

BalTcPlan bal_tc_plan(const pdssm_dims &d) {
    BalTcPlan pl{};
    pl.KT = 2;
    while (pl.KT < d.K) pl.KT *= 2;
    pl.Dp = (int)((d.D_in + 63) / 64 * 64);
    pl.N = pl.Dp <= 128 ? 128 : 64;     // three parts of a group: at most 96 KB
    pl.groups = (int)((d.H * pl.KT + pl.N - 1) / pl.N);
    pl.tiles = (int)((d.B * d.L + kRows - 1) / kRows);
    int s = 148 / pl.groups;
    if (s > pl.tiles) s = pl.tiles;
    pl.slices = s < 1 ? 1 : s;
    pl.w_bytes = (size_t)3 * pl.N * pl.Dp * 2;
    return pl;
}

size_t bal_tc_extra(const BalTcPlan &pl) {
    return (size_t)pl.groups * pl.w_bytes + align256((size_t)pl.groups * pl.N * 8);
}

cudaError_t launch_bal_tc_prep(const BalParams &p, const BalTcPlan &pl, void *parts, cudaStream_t st) {
    const int64_t n = (int64_t)pl.groups * pl.N * (pl.Dp / 2);
    unsigned char *w = (unsigned char *)parts;
    k_bal_parts<<<dim3((unsigned)((n + 255) / 256)), 256, 0, st>>>(
        p, pl, w, reinterpret_cast<float *>(w + (size_t)pl.groups * pl.w_bytes));
    return cudaGetLastError();
}

cudaError_t launch_bal_tc(const BalParams &p, const BalTcPlan &pl, int what, void *parts,
                          cudaStream_t st) {
    switch (pl.KT) {
        case 2: return go_k<2>(p, pl, what, parts, st);
        case 4: return go_k<4>(p, pl, what, parts, st);
        case 8: return go_k<8>(p, pl, what, parts, st);
        case 16: return go_k<16>(p, pl, what, parts, st);
        default: return go_k<32>(p, pl, what, parts, st);
    }
}

}  // namespace pdssm
