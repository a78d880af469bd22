// Decay scan of bf16 inputs on the tensor cores (tcgen05): the forward, and
// the state alone over a segment (forward and reverse) for the join.
//
// A CTA runs one segment of one (batch, head) and 64 columns of the state, in
// chunks of 128 steps (M = 128).  Per chunk, with G_i the cumulated log
// decays and S0 the state at the chunk's start:
//     1. Sc = c b^T                            128 x 128, K = N
//     2. P  = Sc * e^{G_i - G_j}, j <= i, as bf16 back into Sc's columns
//     3. Y  = P x                              128 x 64, K = 128, P from TMEM
//     4. Yi = c S0                             128 x 64, K = N
//     5. y  = Y + e^{G_i} Yi
//     6. S  = e^{G_C} S0 + sum_j (e^{G_C - G_j} b_j) x_j^T; for the adjoint, whose
//        chunks are 64 steps, in two halves, each one's state written out
// The state is an fp32 register of one of 128 threads per row and is decayed
// there; only product 6 adds to it.  Its decayed operand is split into three
// bf16 parts (8 + 8 + 8 bits), so that the state keeps fp32 accuracy (two
// parts were measured at 2.4e-6 of the state's norm, three at 2e-7); the other
// operand is exact.  P and the copy of S0 that product 4 reads are rounded to
// bf16 once each: y is bf16 itself, so they add a rounding of its own size.
//
// N <= 64 (STK): the split operand is b, its rows twice to fill M = 128.
// N <= 128: the split operand is x, and M = N = 128.
//
// Decays: within a 32 x 32 diagonal block each pair's exponential; a block to
// its left as e^{G_i - G_e} e^{G_e - G_j}, e the last step of j's block: both
// factors are at most 1 for a decaying state, so neither over- nor underflows
// where the product does not.
//
// Warps: 0-3 and 4-7 take chunks in turn (steps 2 and 5), 8-15 hold the state
// (32 columns each), 16-23 build the split operand, 24-27 issue the products
// (scores; Yi and Y; two for the state: one thread would hold each of them back
// by the others' waits, and takes about 100 cycles per product), 28 makes the
// copies, 29 and 30 compute the decays in turn.  Accumulators and (N <= 64)
// split parts are double-buffered, c and b tiles three deep (N <= 64; the
// scores of chunk i + 1 run ahead of the rest of chunk i, so two stages would
// expose each copy's latency), all handed over by mbarriers.
//
// Bound: shared memory.  A chunk of 64 x 64 moves 330 KB through it (products'
// operands 210, split parts 64, copies 48), 2600 of the 4200 cycles that a chunk
// takes, and the tensor pipe is busy for 1900; the rest is the hand-overs
// between the roles.  128 heads x 16384 steps: 329 us among other calls (3.3
// TB/s), 290 repeated by itself; the state alone 2500 cycles a chunk for 1900 of
// shared memory.
#include <string.h>

#include "decay.cuh"
#include "launch.cuh"
#include "tile_bf16.cuh"
#include "umma.cuh"

namespace pdssm {
namespace {

constexpr int kC = 128;                 // steps per chunk
// warps by role
constexpr int kState = 8, kBuild = 16, kScores = 24, kOutputs = 25, kStates = 26, kProducer = 28,
              kDecay = 29;
constexpr int kTcTh = 31 * 32;
constexpr int kLoaders = 32;            // threads of plain loads (the producer's warp)
constexpr uint32_t kTile = kC * 128;    // 128 rows of 64 bf16

// forward; the state alone; the state alone in reverse; forward that leaves
// the state at every 64 steps for the adjoint
enum { kFwd = 0, kSegFwd = 1, kSegRev = 2, kFwdCarry = 3 };

// Decays of one chunk in shared memory.
struct __align__(16) Decays {
    float2 G[kC];           // cumulated, base 2, hi + lo
    float start[kC];        // e^{G_t}
    float weight[kC];       // of the state's update: to the end of the chunk (kFwdCarry: of t's
                            // half of it; in reverse: from its start)
    float col[kC];          // e^{G_e - G_t}, e = last step of t's block of 32
    float row[3][kC];       // e^{G_t - G_e}, e = last step of block 0..2 (t behind it)
    float half[2], all[2];  // decay over each half; over the chunk (and padding)
};

// Sets of decays.  The state gives one back a whole chunk after the operand's
// builders; with two sets the decays, the operand and its products of a chunk
// stood in one line behind that (training step of 32 heads x 16384, 64 x 64:
// 603 us with two, 597 with four).
constexpr int kNDec = 4;

// Barriers: four slots of each kind (chunk i: slot i & 3, phase i >> 2, so
// that no role can be a whole round of a slot behind), and the rings' own.
enum {
    kFullCB, kFullX, kScFull, kPReady, kPlReady, kDFull, kS0Ready, kYFull, kYFree,
    kDecReady, kDecFree, kPlRead, kPlLate, kYiFull, kNumBars
};

// Shared memory.  The state alone needs no c (in reverse no b) and no S0, so it
// has deeper rings.
template <bool STK, bool SEG>
struct Smem {
    static constexpr int kNCB = SEG ? (STK ? 4 : 2) : (STK ? 3 : 2);    // stages of c and b
    static constexpr int kNX = SEG ? 3 : 2;             // stages of x
    static constexpr int kNPL = SEG ? (STK ? 3 : 2) : (STK ? 2 : 1);    // sets of split parts
    // parts of a set: STK's part 2 takes b's place; the wide forward has room for
    // two, and its part 0 follows when part 2 has been read
    static constexpr bool kLate = !STK && !SEG;
    static constexpr int kParts = STK || kLate ? 2 : 3;
    static constexpr uint32_t kKey = STK ? kTile : 2 * kTile;   // one c or b tile
    static constexpr uint32_t kB = SEG ? 0 : kKey;      // b (in reverse c) behind the stage's c
    static constexpr uint32_t kStage = kB + kKey;
    static constexpr uint32_t kC0 = 0;                  // [kNCB]
    static constexpr uint32_t kX = kC0 + kNCB * kStage; // [kNX]
    static constexpr uint32_t kPl = kX + kNX * kTile;   // [kNPL][kParts]
    static constexpr uint32_t kS0 = kPl + kNPL * kParts * kTile;
    static constexpr uint32_t kDec = kS0 + (SEG ? 0 : kTile);
    static constexpr uint32_t kBar = kDec + kNDec * sizeof(Decays);
    static constexpr uint32_t kTotal = kBar + 32 * kNumBars + 1024;     // + alignment
};

struct TcParams {
    DecayParams d;
    int first;              // this launch clears the status word
};

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(a));
    return v;
}

// What a wait that gave up left must not pass for a result: NaN in `n` rows of
// y, and in `count` states one behind another (a CTA's columns of each).  Out of
// line, since the place of the roles' code moves the time by several percent.
__device__ __noinline__ void spoil_rows(__nv_bfloat16 *y, int64_t stride, int64_t n, int width) {
    for (int64_t t = threadIdx.x / 32; t < n; t += kTcTh / 32)
        for (int q = threadIdx.x % 32; q < width; q += 32)
            y[t * stride + q] = __ushort_as_bfloat16(0x7fff);
}
__device__ __noinline__ void spoil_states(float *s, int count, int N, int P, int width) {
    for (int i = 0; i < count; ++i, s += (int64_t)N * P)
        for (int e = threadIdx.x; e < N * width; e += kTcTh)
            s[(int64_t)(e / width) * P + e % width] = __int_as_float(0x7fffffff);
}

template <bool STK, int MODE>
__global__ void __launch_bounds__(kTcTh, 1)
    k_decay_tc(const __grid_constant__ CUtensorMap cmap, const __grid_constant__ CUtensorMap bmap,
               const __grid_constant__ CUtensorMap xmap, const TcParams tp) {
    constexpr bool FWD = MODE == kFwd || MODE == kFwdCarry;
    constexpr bool HALVES = MODE == kFwdCarry;
    using SM = Smem<STK, !FWD>;
    const DecayParams &p = tp.d;
    extern __shared__ unsigned char sm_raw[];
    const uint32_t sm = (smem_u32(sm_raw) + 1023u) & ~1023u;
    unsigned char *smg = sm_raw + (sm - smem_u32(sm_raw));
    Decays *dec = reinterpret_cast<Decays *>(smg + SM::kDec);
    __shared__ uint32_t tmem_slot;
    __shared__ double totals[2];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto bar = [&](int which, int i) { return sm + SM::kBar + 8u * (uint32_t)(4 * which + (i & 3)); };
    auto bar_cb = [&](int i) { return sm + SM::kBar + 8u * (uint32_t)(4 * kFullCB + i % SM::kNCB); };
    auto bar_x = [&](int i) { return sm + SM::kBar + 8u * (uint32_t)(4 * kFullX + i % SM::kNX); };

    const int seg = blockIdx.x % p.nseg;
    const int ps = (blockIdx.x / p.nseg) % p.pslices;
    const int64_t bh = blockIdx.x / p.nseg / p.pslices;
    const int b = (int)(bh / p.H), h = (int)(bh % p.H), g = h / p.rep;
    const int p0 = ps * 64, pw = min(64, p.P - p0);
    const int64_t len = decay_len(p, b);
    const int c0 = seg * p.seg_chunks, c1 = min(c0 + p.seg_chunks, p.nchunks);
    // chunks with a live step: n of them, first .. first + n - 1 (reverse: from
    // the last one down)
    const int live_end = (int)((len + kC - 1) / kC);
    const int n = max(0, min(c1, live_end) - c0);
    auto chunk_t0 = [&](int i) {
        return (int64_t)(MODE == kSegRev ? c0 + n - 1 - i : c0 + i) * kC;
    };

    if (tid == 0) {
        if (tp.first && blockIdx.x == 0) *p.status = 0;
        // a tile lands by one copy's bytes, or by the loader threads
        const uint32_t loaders = p.vec ? 1 : kLoaders;
        for (int s = 0; s < 4; ++s) {
            mbar_init(bar(kFullCB, s), loaders);
            mbar_init(bar(kFullX, s), loaders);
            mbar_init(bar(kScFull, s), 1);
            mbar_init(bar(kPReady, s), 128);
            mbar_init(bar(kPlReady, s), 256);
            mbar_init(bar(kPlRead, s), HALVES ? 2 : 1);
            mbar_init(bar(kYiFull, s), 1);
            mbar_init(bar(kPlLate, s), 256);
            mbar_init(bar(kDFull, s), HALVES ? 2 : 1);
            mbar_init(bar(kS0Ready, s), 256);
            mbar_init(bar(kYFull, s), 1);
            mbar_init(bar(kYFree, s), 128);
            mbar_init(bar(kDecReady, s), 32);
            mbar_init(bar(kDecFree, s), FWD ? 640 : 512);
        }
        fence_mbar_init();
    }
    if (warp == kScores) tmem_alloc(smem_u32(&tmem_slot), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    // TMEM columns of buffer i & 1: Sc 128 (P in its first 64, Y in its last 64,
    // Yi 64), and what the chunk adds to the state, 64 (with HALVES buffer 0 is the
    // first half's and 1 the second's of every chunk)
    auto tcol = [&](int i, int col) { return tmem + (uint32_t)((i & 1) * 256 + col); };

    // Bounded waits of one thread, or of a whole warp (which then agrees on the
    // outcome, as the warp-wide TMEM accesses need).  After the first that
    // gives up, a role waits for nothing more and leaves its loop.
    bool ok = true;
    auto wait_at = [&](uint32_t at, int phase) {
        if (ok && !mbar_wait_hot(at, (uint32_t)(phase & 1))) {
            ok = false;
            flag_status(p.status, kStTimeout);
        }
        return ok;
    };
    auto wait = [&](int which, int i) { return wait_at(bar(which, i), i >> 2); };
    auto wait_cb = [&](int i) { return wait_at(bar_cb(i), i / SM::kNCB); };
    auto wait_x = [&](int i) { return wait_at(bar_x(i), i / SM::kNX); };
    auto wait_warp = [&](int which, int i) { return ok = __all_sync(kFull, wait(which, i)); };
    auto wait_cb_warp = [&](int i) { return ok = __all_sync(kFull, wait_cb(i)); };
    auto wait_x_warp = [&](int i) { return ok = __all_sync(kFull, wait_x(i)); };

    if (warp < 8) {
        if (FWD) {
            // ---- decayed scores and y: row r of chunks i = warp / 4, + 2, ...
            const int r = tid & 127, quad = warp & 3;
            const uint32_t tlane = (uint32_t)(quad * 32) << 16;
            __nv_bfloat16 *y = (__nv_bfloat16 *)p.y + b * p.oval_b + h * p.oval_h + p0;
            for (int i = warp >> 2; i < n; i += 2) {
                const Decays &dc = dec[i & (kNDec - 1)];
                if (!wait_warp(kDecReady, i) || !wait_warp(kScFull, i)) break;
                tc_fence_after();
                const float es = dc.start[r];
                // 16 columns at a time; the loops stay rolled: six roles share each
                // scheduler's instruction cache
#pragma unroll 1
                for (int c = 0; c < 8; ++c) {
                    uint32_t o[8];
                    const int J = c >> 1;
                    if (J <= quad) {
                        uint32_t v[16];
                        tmem_ld16_raw(tcol(i, 16 * c) + tlane, v);
                        tmem_wait_ld();
                        if (J < quad) {
                            const float rf = dc.row[J][r];
                            const float4 *cf = reinterpret_cast<const float4 *>(dc.col + 16 * c);
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const float4 f = cf[q];
                                o[2 * q] = pack2(__uint_as_float(v[4 * q]) * (f.x * rf),
                                                 __uint_as_float(v[4 * q + 1]) * (f.y * rf));
                                o[2 * q + 1] = pack2(__uint_as_float(v[4 * q + 2]) * (f.z * rf),
                                                     __uint_as_float(v[4 * q + 3]) * (f.w * rf));
                            }
                        } else {
                            const float2 gr = dc.G[r];
                            const float4 *gc = reinterpret_cast<const float4 *>(dc.G + 16 * c);
                            const int past = r - 16 * c;        // columns up to here count
#pragma unroll
                            for (int q = 0; q < 8; ++q) {
                                const float4 g = gc[q];
                                const float e0 = ex2((gr.x - g.x) + (gr.y - g.y));
                                const float e1 = ex2((gr.x - g.z) + (gr.y - g.w));
                                o[q] = pack2(2 * q <= past ? __uint_as_float(v[2 * q]) * e0 : 0.f,
                                             2 * q < past ? __uint_as_float(v[2 * q + 1]) * e1 : 0.f);
                            }
                        }
                    } else {
#pragma unroll
                        for (int q = 0; q < 8; ++q) o[q] = 0;
                    }
                    tmem_st8(tcol(i, 8 * c) + tlane, o);
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(bar(kPReady, i));
                mbar_arrive(bar(kDecFree, i));

                if (!wait_warp(kYFull, i)) break;       // Y, and Yi before it
                tc_fence_after();
                const int64_t t = chunk_t0(i) + r;
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {
                    uint32_t u[16], w[16], o[8];
                    tmem_ld16_raw(tcol(i, 64 + 16 * q) + tlane, u);
                    tmem_ld16_raw(tcol(i, 128 + 16 * q) + tlane, w);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float y0 = fmaf(es, __uint_as_float(w[2 * e]), __uint_as_float(u[2 * e]));
                        const float y1 =
                            fmaf(es, __uint_as_float(w[2 * e + 1]), __uint_as_float(u[2 * e + 1]));
                        o[e] = t < len ? pack2(y0, y1) : 0u;
                    }
                    if (q == 3) {
                        tc_fence_before();
                        mbar_arrive(bar(kYFree, i));
                    }
                    const int left = pw - 16 * q;               // columns left
                    if (t < p.L && left > 0) {
                        __nv_bfloat16 *row = y + t * p.oval_t + 16 * q;
                        if (p.ovec == 2 && left > 8) {
                            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(row),
                                         "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]),
                                         "r"(o[6]), "r"(o[7])
                                         : "memory");
                        } else if (p.ovec) {                    // rows in eights
                            *reinterpret_cast<uint4 *>(row) = make_uint4(o[0], o[1], o[2], o[3]);
                            if (left > 8)
                                *reinterpret_cast<uint4 *>(row + 8) = make_uint4(o[4], o[5], o[6], o[7]);
                        } else {
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                if (e < left)
                                    reinterpret_cast<unsigned short *>(row)[e] =
                                        (unsigned short)(o[e / 2] >> (16 * (e % 2)));
                        }
                    }
                    __syncwarp();       // rows behind the end part ways: together again for the next load
                }
            }
        }
    } else if (warp < kBuild) {
        // ---- the state: a row and kCols columns per thread (STK: the accumulators'
        // rows 64.. repeat 0..63, so their lanes take other columns)
        constexpr int kCols = STK ? 16 : 32;
        const int quad = warp & 3, lr = quad * 32 + lane;
        const int r = STK ? (lr & 63) : lr;                 // row of N
        const int q0 = ((warp - kState) >> 2) * 32 + (STK ? (quad >> 1) * 16 : 0);
        const uint32_t tlane = (uint32_t)(quad * 32) << 16;
        const int64_t np = (int64_t)p.N * p.P;
        const int left = r < p.N ? pw - q0 : 0;             // columns of this thread
        const int64_t at = (int64_t)r * p.P + p0 + q0;
        float S[kCols];
        {
            const float *in = nullptr;
            if (FWD)
                in = p.nseg > 1 ? p.seg_state + (bh * p.nseg + seg) * np
                                : (p.h0 ? p.h0 + bh * np : nullptr);
#pragma unroll
            for (int q = 0; q < kCols; ++q) S[q] = in && q < left ? in[at + q] : 0.f;
        }
        // this thread's part of the state; a caller's buffer may start anywhere
        auto leave = [&](float *out) {
            const bool wide = p.P % 4 == 0 && ((uintptr_t)out & 15) == 0;
            out += at;
#pragma unroll
            for (int q = 0; q < kCols; q += 4) {
                if (wide) {
                    if (q < left)
                        *reinterpret_cast<float4 *>(out + q) = make_float4(S[q], S[q + 1], S[q + 2], S[q + 3]);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (q + e < left) out[q + e] = S[q + e];
                }
            }
        };
        auto put_S0 = [&](int i) {
#pragma unroll
            for (int q = 0; q < kCols / 8; ++q)
                sts128(sm + SM::kS0 + piece(r, q0 / 8 + q), pack2(S[8 * q], S[8 * q + 1]),
                       pack2(S[8 * q + 2], S[8 * q + 3]), pack2(S[8 * q + 4], S[8 * q + 5]),
                       pack2(S[8 * q + 6], S[8 * q + 7]));
            fence_proxy_async_smem();
            tc_fence_before();
            mbar_arrive(bar(kS0Ready, i));
        };
        // kFwdCarry: the state at the start of the sequence's 64-step chunk ch
        const int chunks64 = (int)((p.L + 63) / 64);
        auto carry = [&](int ch) {
            if (ch > 0 && ch < chunks64) leave(p.carry + (bh * chunks64 + ch) * np);
        };
        if (FWD && n > 0) put_S0(0);
        for (int i = 0; i < n; ++i) {
            if (!wait_warp(kDecReady, i)) break;
            const float a[2] = {HALVES ? dec[i & (kNDec - 1)].half[0] : dec[i & (kNDec - 1)].all[0], dec[i & (kNDec - 1)].half[1]};
            mbar_arrive(bar(kDecFree, i));
            if (HALVES) carry(2 * (c0 + i));
            if (!wait_warp(kDFull, i)) break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < (HALVES ? 2 : 1); ++k) {
                if (k == 1) carry(2 * (c0 + i) + 1);
                __syncwarp();                               // the loads below are the whole warp's
#pragma unroll
                for (int q = 0; q < kCols; q += 16) {
                    uint32_t v[16];
                    tmem_ld16_raw(tcol(HALVES ? k : i, 192 + q0 + q) + tlane, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e) S[q + e] = fmaf(a[k], S[q + e], __uint_as_float(v[e]));
                }
            }
            if (FWD) {
                if (i + 1 == n) break;
                if (!wait_warp(kYiFull, i)) break;          // S0 has been read
                put_S0(i + 1);
            } else {
                tc_fence_before();
                mbar_arrive(bar(kS0Ready, i));              // the accumulators are free
            }
        }
        if (!FWD)
            leave(p.seg_state + (bh * p.nseg + seg) * np);
        else if (p.h_last && seg == p.nseg - 1)
            leave(p.h_last + bh * np);
    } else if (warp < kScores) {
        // ---- the three parts of each chunk's decayed operand: row r = step t0 + r,
        // four of its eight pieces
        const int r = tid & 127, h0 = ((warp - kBuild) >> 2) * 4;
        for (int i = 0; i < n; ++i) {
            if (!wait_warp(kDecReady, i)) break;
            const float w = dec[i & (kNDec - 1)].weight[r];
            mbar_arrive(bar(kDecFree, i));
            const bool on = chunk_t0(i) + r < len;
            if (!wait_cb_warp(i)) break;
            if ((!STK || chunk_t0(i) + kC > len) && !wait_x_warp(i)) break;
            // the tiles change (part 2, rows behind the end) and are given back only
            // once the scores have read them
            if (FWD && !wait_warp(kScFull, i)) break;
            if (i >= SM::kNPL && !wait_warp(kDFull, i - SM::kNPL)) break;
            const uint32_t keys = sm + SM::kC0 + (uint32_t)(i % SM::kNCB) * SM::kStage;
            const uint32_t bt = keys + SM::kB, xt = sm + SM::kX + (uint32_t)(i % SM::kNX) * kTile;
            if (!on) {      // behind the end: whatever lies there must not meet a zero weight
#pragma unroll
                for (int q = h0; q < h0 + 4; ++q) {
                    sts128(xt + piece(r, q), 0, 0, 0, 0);
                    sts128(bt + piece(r, q), 0, 0, 0, 0);
                    if (!STK) sts128(bt + kTile + piece(r, q), 0, 0, 0, 0);
                }
            }
            const uint32_t src = STK ? bt : xt;
            const uint32_t dst = sm + SM::kPl + (uint32_t)(i % SM::kNPL) * SM::kParts * kTile;
            // where parts 0, 1 and 2 go
            const uint32_t d0 = dst, d1 = dst + kTile, d2 = STK ? bt : SM::kLate ? dst : dst + 2 * kTile;
            uint32_t late[SM::kLate ? 16 : 1];
#pragma unroll (SM::kLate ? 4 : 2)
            for (int k = 0; k < 4; ++k) {
                const int q = h0 + k;
                const uint4 u = lds128(src + piece(r, q));
                const uint32_t in[4] = {u.x, u.y, u.z, u.w};
                uint32_t p1[4], p2[4], p3[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float v0 = lo_of(in[e]) * w, v1 = hi_of(in[e]) * w;
                    p1[e] = pack2(v0, v1);
                    v0 -= lo_of(p1[e]);
                    v1 -= hi_of(p1[e]);
                    p2[e] = pack2(v0, v1);
                    v0 -= lo_of(p2[e]);
                    v1 -= hi_of(p2[e]);
                    p3[e] = pack2(v0, v1);
                }
                const uint32_t at = piece(r, q);
                if constexpr (SM::kLate) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) late[4 * k + e] = p1[e];
                } else {
                    sts128(d0 + at, p1[0], p1[1], p1[2], p1[3]);
                }
                sts128(d1 + at, p2[0], p2[1], p2[2], p2[3]);
                sts128(d2 + at, p3[0], p3[1], p3[2], p3[3]);
            }
            fence_proxy_async_smem();
            mbar_arrive(bar(kPlReady, i));
            if constexpr (SM::kLate) {
                if (!wait_warp(kPlRead, i)) break;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    sts128(d0 + piece(r, h0 + k), late[4 * k], late[4 * k + 1], late[4 * k + 2],
                           late[4 * k + 3]);
                fence_proxy_async_smem();
                mbar_arrive(bar(kPlLate, i));
            }
        }
    } else if (warp == kScores) {
        // ---- products: the scores
        if (lane == 0 && FWD) {
            constexpr uint32_t kIdSc = umma_idesc_bf16(128);
            const uint32_t key0 = umma_lo(sm + SM::kC0, kTile);
            for (int i = 0; i < n; ++i) {
                if (!wait_cb(i) || (i >= 2 && !wait(kYFree, i - 2))) break;
                tc_fence_after();
                const uint32_t ct = key0 + (uint32_t)(i % SM::kNCB) * umma_step(SM::kStage);
                const uint32_t bt = ct + umma_step(SM::kB), dS = tcol(i, 0);
#pragma unroll
                for (int k = 0; k < (STK ? 4 : 8); ++k) {
                    const uint32_t off = (k >> 2) * umma_step(kTile) + (k & 3) * umma_step(32);
                    umma_ss(dS, ct + off, bt + off, kIdSc, k > 0);
                }
                umma_commit(bar(kScFull, i));
            }
            if (n > 0 && ok) wait(kScFull, n - 1);  // nothing is in flight when the CTA ends
        }
        __syncwarp();
    } else if (warp == kOutputs) {
        // ---- products: Yi and Y
        if (lane == 0 && FWD) {
            constexpr uint32_t kIdY = umma_idesc_bf16(64, false, true);
            const uint32_t key0 = umma_lo(sm + SM::kC0, kTile), x0 = umma_lo(sm + SM::kX, 0),
                           s0 = umma_lo(sm + SM::kS0, 0);
            for (int i = 0; i < n; ++i) {
                if (!wait_cb(i) || !wait(kS0Ready, i) || (i >= 2 && !wait(kYFree, i - 2))) break;
                tc_fence_after();
                const uint32_t ct = key0 + (uint32_t)(i % SM::kNCB) * umma_step(SM::kStage);
                const uint32_t dYi = tcol(i, 128);
#pragma unroll
                for (int k = 0; k < (STK ? 4 : 8); ++k)
                    umma_ss(dYi, ct + (k >> 2) * umma_step(kTile) + (k & 3) * umma_step(32),
                            s0 + k * umma_step(2048), kIdY, k > 0);
                umma_commit(bar(kYiFull, i));
                if (!wait(kPReady, i) || !wait_x(i) || !wait(kPlReady, i)) break;
                tc_fence_after();
                const uint32_t dY = tcol(i, 64), pa = tcol(i, 0);
                const uint32_t xr = x0 + (uint32_t)(i % SM::kNX) * umma_step(kTile);
#pragma unroll
                for (int k = 0; k < 8; ++k) umma_ts(dY, pa + 8 * k, xr + k * umma_step(2048), kIdY, k > 0);
                umma_commit(bar(kYFull, i));
            }
            if (n > 0) wait(kYiFull, n - 1) && wait(kYFull, n - 1);
        }
        __syncwarp();
    } else if (warp == kStates || warp == kStates + 1) {
        // ---- products: what the chunk adds to the state; the two warps take chunks in
        // turn, or (HALVES) a half of each chunk
        const int w = warp - kStates;
        if (lane == 0) {
            constexpr uint32_t kIdD = umma_idesc_bf16(64, true, true);
            constexpr uint32_t kRow16 = umma_step(2048);    // 16 rows of a tile
            constexpr int kSteps = HALVES ? 4 : 8;
            const uint32_t key0 = umma_lo(sm + SM::kC0, kTile) + (HALVES ? w * 4 * kRow16 : 0),
                           x0 = umma_lo(sm + SM::kX, 0) + (HALVES ? w * 4 * kRow16 : 0),
                           pl0 = umma_lo(sm + SM::kPl, kTile) + (HALVES ? w * 4 * kRow16 : 0);
            int last = -1;
            for (int i = HALVES ? 0 : w; i < n; i += HALVES ? 1 : 2) {
                const uint32_t bt = key0 + (uint32_t)(i % SM::kNCB) * umma_step(SM::kStage) +
                                    umma_step(SM::kB);
                const uint32_t xr = x0 + (uint32_t)(i % SM::kNX) * umma_step(kTile);
                // the accumulators are free: the state took chunk i - 2's (HALVES: i - 1's)
                // before it left S0 of the chunk behind (the state alone: before it said so)
                const int taken = HALVES ? i : FWD ? i - 1 : i - 2;
                if (!wait_cb(i) || (taken > 0 - !FWD && !wait(kS0Ready, taken))) break;
                if (!wait(kPlReady, i) || !wait_x(i)) break;
                tc_fence_after();
                const uint32_t dD = tcol(HALVES ? w : i, 192);
                const uint32_t pl = pl0 + (uint32_t)(i % SM::kNPL) * umma_step(SM::kParts * kTile);
                // STK: the parts' 64 columns twice as the 128 rows (leading offset 0;
                // part 2 lies in b's place)
#pragma unroll 1
                for (int part = 2; part >= 0; --part) {     // the small ones first
                    if (SM::kLate && part == 0) {       // in part 2's buffer, once that has been read
                        umma_commit(bar(kPlRead, i));
                        if (!wait(kPlLate, i)) break;
                        tc_fence_after();
                    }
                    const uint32_t ar = STK ? (part < 2 ? pl + part * umma_step(kTile) : bt) - umma_lo(0, kTile) : bt;
                    const uint32_t br = STK ? xr : pl + (SM::kLate && part == 2 ? 0 : part) * umma_step(kTile);
#pragma unroll
                    for (int k = 0; k < kSteps; ++k)
                        umma_ss(dD, ar + k * kRow16, br + k * kRow16, kIdD, k > 0 || part < 2);
                }
                if (!ok) break;
                umma_commit(bar(kDFull, i));
                last = i;
            }
            if (last >= 0 && ok) wait(kDFull, last);    // nothing is in flight when the CTA ends
        }
        __syncwarp();
    } else if (warp >= kDecay) {
        // ---- decays: the two warps take chunks in turn, four consecutive steps per
        // lane
        const float *la = p.log_a + b * p.la_b + h * p.la_h;
        double total = 0.0;
        float nx[4];
        auto fetch = [&](int i) {
            const int64_t t0 = chunk_t0(i) + 4 * lane;
#pragma unroll
            for (int q = 0; q < 4; ++q) nx[q] = i < n && t0 + q < len ? la[(t0 + q) * p.la_t] : 0.f;
        };
        fetch(warp - kDecay);
        for (int i = warp - kDecay; i < n; i += 2) {
            double v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = decay_log2(nx[q]) + (q ? v[q ? q - 1 : 0] : 0.0);
            fetch(i + 2);
            double s = v[3];
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const double o = shfl_up_d(s, d);
                if (lane >= d) s += o;
            }
            total += __shfl_sync(kFull, s, 31);
            s -= v[3];
            float2 G[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const double c = s + v[q];
                const float hi = (float)c;
                G[q] = make_float2(hi, (float)(c - (double)hi));
            }
            if (i >= kNDec && !wait_warp(kDecFree, i - kNDec)) break;
            Decays &dc = dec[i & (kNDec - 1)];
            float4 *gs = reinterpret_cast<float4 *>(dc.G + 4 * lane);
            gs[0] = make_float4(G[0].x, G[0].y, G[1].x, G[1].y);
            gs[1] = make_float4(G[2].x, G[2].y, G[3].x, G[3].y);
            __syncwarp();
            const float2 mid = dc.G[kC / 2 - 1], end = dc.G[kC - 1];
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
                const int t = 32 * q + lane;
                const float2 g = dc.G[t];
                const float es = ex2(g.x + g.y);
                dc.start[t] = es;
                const float2 to = HALVES && q < 2 ? mid : end;
                dc.weight[t] = MODE == kSegRev ? es : ex2((to.x - g.x) + (to.y - g.y));
                if (FWD) {
                    const float2 own = dc.G[32 * q + 31];
                    dc.col[t] = ex2((own.x - g.x) + (own.y - g.y));
#pragma unroll 1
                    for (int e = 0; e < q; ++e) {
                        const float2 b = dc.G[32 * e + 31];
                        dc.row[e][t] = ex2((g.x - b.x) + (g.y - b.y));
                    }
                }
            }
            if (lane == 0) {
                dc.all[0] = ex2(end.x + end.y);
                dc.half[0] = ex2(mid.x + mid.y);
                dc.half[1] = ex2((end.x - mid.x) + (end.y - mid.y));
            }
            mbar_arrive(bar(kDecReady, i));
        }
        if (!FWD && lane == 0) totals[warp - kDecay] = total;
    } else if (p.vec) {
        // ---- copies
        if (warp == kProducer && lane == 0 && !p.hold) {
            int i = 0;
            for (; i < n && ok; ++i) {
                const int t0 = (int)chunk_t0(i);
                if (i >= SM::kNCB && (!wait(kDFull, i - SM::kNCB) || (FWD && !wait(kYiFull, i - SM::kNCB))))
                    break;
                const uint32_t keys = sm + SM::kC0 + (uint32_t)(i % SM::kNCB) * SM::kStage;
                const uint32_t cb = bar_cb(i);
                const int subs = STK ? 1 : 2;
                mbar_expect_tx(cb, (uint32_t)(FWD ? 2 : 1) * SM::kKey);
                for (int q = 0; q < subs; ++q) {
                    // the state alone needs one key tensor: b, or c in reverse
                    if (FWD) tma_load_4d(keys + q * kTile, &cmap, 64 * q, t0, g, b, cb);
                    tma_load_4d(keys + SM::kB + q * kTile, MODE == kSegRev ? &cmap : &bmap, 64 * q, t0,
                                g, b, cb);
                }
                if (i >= SM::kNX && (!wait(kDFull, i - SM::kNX) || (FWD && !wait(kYFull, i - SM::kNX)))) break;
                const uint32_t xb = bar_x(i);
                mbar_expect_tx(xb, kTile);
                tma_load_4d(sm + SM::kX + (uint32_t)(i % SM::kNX) * kTile, &xmap, p0, t0, h, b, xb);
            }
        }
        __syncwarp();
    } else {
        // ---- the same tiles by plain loads of one warp: odd widths, odd
        // addresses
        const int l = lane;
        const __nv_bfloat16 *kc = (const __nv_bfloat16 *)p.c + b * p.key_b + g * p.key_h;
        const __nv_bfloat16 *kb = (const __nv_bfloat16 *)(MODE == kSegRev ? p.c : p.b) + b * p.key_b +
                                  g * p.key_h;
        const __nv_bfloat16 *vx = (const __nv_bfloat16 *)(MODE == kSegRev ? p.g_y : p.x) + b * p.val_b +
                                  h * p.val_h + p0;
        auto copy = [&](uint32_t dst, const __nv_bfloat16 *src, int64_t stride, int width, int64_t t0) {
            for (int e = l; e < kC * 8; e += kLoaders) {
                const int r = e / 8, q = e % 8;
                uint32_t w[4] = {0, 0, 0, 0};
                if (t0 + r < len) {
                    const unsigned short *s =
                        reinterpret_cast<const unsigned short *>(src + (t0 + r) * stride) + 8 * q;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (8 * q + j < width) w[j / 2] |= (uint32_t)s[j] << (16 * (j % 2));
                }
                sts128(dst + piece(r, q), w[0], w[1], w[2], w[3]);
            }
        };
        for (int i = 0; i < n && ok; ++i) {
            const int64_t t0 = chunk_t0(i);
            if (i >= SM::kNCB && (!wait_warp(kDFull, i - SM::kNCB) || (FWD && !wait_warp(kYiFull, i - SM::kNCB))))
                break;
            const uint32_t keys = sm + SM::kC0 + (uint32_t)(i % SM::kNCB) * SM::kStage;
            for (int q = 0; q < (STK ? 1 : 2); ++q) {
                if (FWD)
                    copy(keys + q * kTile, kc + 64 * q, p.key_t, p.N - 64 * q, t0);
                copy(keys + SM::kB + q * kTile, kb + 64 * q, p.key_t, p.N - 64 * q, t0);
            }
            fence_proxy_async_smem();
            mbar_arrive(bar_cb(i));
            if (i >= SM::kNX && (!wait_warp(kDFull, i - SM::kNX) ||
                                  (FWD && !wait_warp(kYFull, i - SM::kNX))))
                break;
            copy(sm + SM::kX + (uint32_t)(i % SM::kNX) * kTile, vx, p.val_t, pw, t0);
            fence_proxy_async_smem();
            mbar_arrive(bar_x(i));
        }
    }
    tc_fence_before();
    const bool failed = __syncthreads_or(!ok);
    if (failed) {
        // a wait gave up (the status word says so): let copies and products in
        // flight land, for a millisecond at most, before the CTA ends
        const uint64_t t = global_ns();
        for (int it = 0; it < (1 << 20) && global_ns() - t < 1000000u; ++it) __nanosleep(1000);
        __syncthreads();
    }
    tc_fence_after();
    if (warp == kScores) tmem_dealloc(tmem, 512);
    if (!FWD && ps == 0 && tid == 0)
        p.seg_decay[bh * p.nseg + seg] = exp2f((float)(totals[0] + totals[1]));
    if (FWD) {
        // rows of the segment's chunks behind the sequence's end
        __nv_bfloat16 *y = (__nv_bfloat16 *)p.y + b * p.oval_b + h * p.oval_h + p0;
        const int64_t t_end = imin64((int64_t)c1 * kC, p.L);
        for (int64_t t = (int64_t)(c0 + n) * kC + warp; t < t_end; t += kTcTh / 32)
            for (int q = lane; q < pw; q += 32) y[t * p.oval_t + q] = __float2bfloat16_rn(0.f);
        if (failed)
            spoil_rows(y + (int64_t)c0 * kC * p.oval_t, p.oval_t, min((int64_t)n * kC, t_end - (int64_t)c0 * kC), pw);
    }
    if (failed) {
        const int64_t np = (int64_t)p.N * p.P;
        if (!FWD) spoil_states(p.seg_state + (bh * p.nseg + seg) * np + p0, 1, p.N, p.P, pw);
        if (FWD && p.h_last && seg == p.nseg - 1) spoil_states(p.h_last + bh * np + p0, 1, p.N, p.P, pw);
        if (HALVES) {
            const int chunks64 = (int)((p.L + 63) / 64), ch = max(2 * c0, 1);
            spoil_states(p.carry + (bh * chunks64 + ch) * np + p0, min(2 * c1, chunks64) - ch, p.N, p.P, pw);
        }
    }
}

bool encode_map(CUtensorMap *m, const void *ptr, int width, int heads, const DecayParams &p,
                int64_t st, int64_t sh, int64_t sb) {
    const cuuint64_t dim[4] = {(cuuint64_t)width, (cuuint64_t)p.L, (cuuint64_t)heads, (cuuint64_t)p.B};
    const cuuint64_t stride[3] = {(cuuint64_t)st * 2, (cuuint64_t)sh * 2, (cuuint64_t)sb * 2};
    const cuuint32_t box[4] = {64, kC, 1, 1};
    const cuuint32_t es[4] = {1, 1, 1, 1};
    return tensor_map_encoder()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(ptr), dim,
                                stride, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool STK, int MODE>
cudaError_t go(const DecayParams &p, bool first, cudaStream_t st) {
    CUtensorMap cm, bm, xm;
    memset(&cm, 0, sizeof(cm));
    memset(&bm, 0, sizeof(bm));
    memset(&xm, 0, sizeof(xm));
    const void *x = MODE == kSegRev ? p.g_y : p.x;
    if (p.vec) {
        if (!encode_map(&cm, p.c, p.N, p.G, p, p.key_t, p.key_h, p.key_b) ||
            !encode_map(&bm, p.b, p.N, p.G, p, p.key_t, p.key_h, p.key_b) ||
            !encode_map(&xm, x, p.P, p.H, p, p.val_t, p.val_h, p.val_b))
            return cudaErrorInvalidValue;
    }
    auto kern = k_decay_tc<STK, MODE>;
    const int smem = (int)Smem<STK, MODE == kSegFwd || MODE == kSegRev>::kTotal;
    static std::atomic<int> set[kLimitDevices];
    const cudaError_t e = allow_smem((const void *)kern, smem, set);
    if (e != cudaSuccess) return e;
    const int64_t grid = (int64_t)p.B * p.H * p.nseg * p.pslices;
    kern<<<dim3((unsigned)grid), kTcTh, smem, st>>>(cm, bm, xm, TcParams{p, first ? 1 : 0});
    return cudaGetLastError();
}

template <bool STK>
cudaError_t fwd_tc(const DecayParams &p, cudaStream_t st) {
    if (p.nseg > 1) {
        cudaError_t e = go<STK, kSegFwd>(p, true, st);
        if (e != cudaSuccess) return e;
        e = launch_decay_join(p, p.h0, false, st);
        if (e != cudaSuccess) return e;
    }
    return p.carry ? go<STK, kFwdCarry>(p, p.nseg <= 1, st) : go<STK, kFwd>(p, p.nseg <= 1, st);
}

}  // namespace

bool decay_tc_copies() { return tensor_map_encoder() != nullptr; }

cudaError_t launch_decay_fwd_tc(const DecayParams &p, cudaStream_t st) {
    return p.N <= 64 ? fwd_tc<true>(p, st) : fwd_tc<false>(p, st);
}

cudaError_t launch_decay_seg_rev_tc(const DecayParams &p, cudaStream_t st) {
    return p.N <= 64 ? go<true, kSegRev>(p, false, st) : go<false, kSegRev>(p, false, st);
}

}  // namespace pdssm
