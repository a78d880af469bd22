// C ABI of the decay scan: argument checks, workspace, launch sequence.
#include <string.h>

#include <initializer_list>

#include "decay.cuh"

using namespace pdssm;

namespace pdssm {

// Chunks and segments from the sizes alone, so that workspace sizes follow.
// Segments fill the GPU when the (batch, head, 64 columns) units do not: one
// CTA of the tensor-core forward fits an SM, two of its adjoint (above 64 x 64
// one), about three of the others.  Each segment costs a second read of b and x (the adjoint: of
// c and g_y).  A segment has at least four chunks of the tensor-core kernels
// (whose start-up is worth about one), one of the others: a training step of
// 8 heads x 1501 steps, 64 x 48 fp32, took 222 us with segments of at least
// four, 127 with two.
DecayPlan decay_plan(const pdssm_decay_dims &d, bool tc, bool adjoint) {
    DecayPlan pl{};
    pl.chunk = tc ? (adjoint ? 64 : 128) : 32;
    pl.nchunks = (int)((d.L + pl.chunk - 1) / pl.chunk);
    pl.pslices = adjoint ? 1 : (int)((d.P + 63) / 64);
    const int64_t units = d.B * d.H * pl.pslices;
    int64_t nseg = (int64_t)kDecaySMs * (tc ? (adjoint && d.N <= 64 && d.P <= 64 ? 2 : 1) : 3) / units;
    if (tc && nseg > pl.nchunks / 4) nseg = pl.nchunks / 4;
    if (nseg > pl.nchunks) nseg = pl.nchunks;
    if (nseg < 1) nseg = 1;
    pl.seg_chunks = (int)((pl.nchunks + nseg - 1) / nseg);
    if (tc && adjoint) pl.seg_chunks = (pl.seg_chunks + 1) / 2 * 2;     // whole chunks of 128
    if (pl.seg_chunks < 1) pl.seg_chunks = 1;
    pl.nseg = pl.nchunks > 0 ? (pl.nchunks + pl.seg_chunks - 1) / pl.seg_chunks : 1;
    return pl;
}

}  // namespace pdssm

namespace {

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

pdssm_status check_dims(const pdssm_decay_dims *d, pdssm_dtype dt, bool step) {
    if (!d) return arg_fail(PDSSM_ERR_INVALID_ARG, "dims is NULL");
    if (dt != PDSSM_F32 && dt != PDSSM_BF16)
        return arg_fail(PDSSM_ERR_INVALID_ARG, "dtype must be fp32 or bf16");
    if (d->B < 1 || d->H < 1 || d->G < 1 || d->N < 1 || d->P < 1 || (!step && d->L < 0))
        return arg_fail(PDSSM_ERR_INVALID_ARG, "need B, H, G, N, P >= 1 and L >= 0");
    if (d->H % d->G) return arg_fail(PDSSM_ERR_INVALID_ARG, "H must be a multiple of G");
    if (d->N > kDecayMaxW || d->P > kDecayMaxW)
        return arg_fail(PDSSM_ERR_UNSUPPORTED, "N > 128 or P > 128");
    const int64_t big = (int64_t)1 << 24;
    if (d->B > big || d->H > big || d->B * d->H > big)
        return arg_fail(PDSSM_ERR_UNSUPPORTED, "B*H > 2^24");
    if (!step && (d->L > ((int64_t)1 << 31) || d->B * d->H * d->L > ((int64_t)1 << 40)))
        return arg_fail(PDSSM_ERR_UNSUPPORTED, "L or B*H*L too large");
    return PDSSM_OK;
}

// bf16 runs on the tensor cores, fp32 on the CUDA cores.
bool on_tc(pdssm_dtype dt) { return dt == PDSSM_BF16; }

struct DecayWs {
    size_t seg_state, seg_decay, carry, part_c, part_b, part_la;
    size_t pad_c, pad_b, pad_x, pad_v, total;   // padded rows; pad_v: y, or g_y
};

DecayWs ws_of(const pdssm_decay_dims &d, pdssm_dtype dt, bool for_bwd) {
    DecayWs w{};
    const DecayPlan f = decay_plan(d, on_tc(dt), false), r = decay_plan(d, on_tc(dt), true);
    const size_t np = (size_t)(d.N * d.P) * 4, bh = (size_t)(d.B * d.H);
    const size_t nseg = (size_t)(for_bwd && r.nseg > f.nseg ? r.nseg : f.nseg);
    size_t o = 256;     // the status word's block
    w.seg_state = o; o = align256(o + bh * nseg * np);
    w.seg_decay = o; o = align256(o + bh * nseg * 4);
    if (for_bwd) {
        w.carry = o; o = align256(o + bh * (size_t)r.nchunks * np);
        if (d.G < d.H) {
            const size_t keys = bh * (size_t)(d.L * d.N) * 4;
            w.part_c = o; o = align256(o + keys);
            w.part_b = o; o = align256(o + keys);
        }
        w.part_la = o; o = align256(o + bh * (size_t)d.L * 4);
    }
    if (on_tc(dt) && d.N % 8) {
        const size_t keys = (size_t)(d.B * d.G * d.L) * (size_t)((d.N + 7) / 8 * 16);
        w.pad_c = o; o = align256(o + keys);
        w.pad_b = o; o = align256(o + keys);
    }
    if (on_tc(dt) && d.P % 8) {
        const size_t vals = bh * (size_t)d.L * (size_t)((d.P + 7) / 8 * 16);
        w.pad_x = o; o = align256(o + vals);
        w.pad_v = o; o = align256(o + vals);
    }
    w.total = o;
    return w;
}

void set_strides(DecayParams &p, const pdssm_decay_dims &d, pdssm_layout lay, bool per_step) {
    p.B = (int)d.B; p.H = (int)d.H; p.G = (int)d.G; p.rep = (int)(d.H / d.G);
    p.N = (int)d.N; p.P = (int)d.P; p.L = d.L;
    if (lay == PDSSM_BHL) {
        p.key_t = d.N; p.key_h = d.L * d.N;
        p.val_t = d.P; p.val_h = d.L * d.P;
        p.la_t = 1; p.la_h = d.L;
    } else {
        p.key_t = d.G * d.N; p.key_h = d.N;
        p.val_t = d.H * d.P; p.val_h = d.P;
        p.la_t = d.H; p.la_h = 1;
    }
    p.key_b = d.G * d.L * d.N;
    p.val_b = d.H * d.L * d.P;
    p.okey_t = p.key_t; p.okey_h = p.key_h; p.okey_b = p.key_b;
    p.oval_t = p.val_t; p.oval_h = p.val_h; p.oval_b = p.val_b;
    p.la_b = d.H * d.L;
    p.gla_t = p.la_t; p.gla_h = p.la_h; p.gla_b = p.la_b;
    if (!per_step) {
        p.la_t = 0; p.la_h = 1; p.la_b = 0;
        p.gla_t = 1; p.gla_h = d.L; p.gla_b = d.H * d.L;     // partials [B][H][L]
    }
}

bool all_aligned(std::initializer_list<const void *> ptrs, size_t a) {
    for (const void *q : ptrs)
        if (!aligned(q, a)) return false;
    return true;
}

// Inputs for the tensor-core kernels: rows whose width is not a multiple of 8
// are copied to padded ones, and y is made in such rows too: 64 heads x 8192
// steps of 31 x 31 take 188 us, by one warp's 2-byte loads and the epilogue's
// 2-byte stores 284.  The adjoint takes the copies that the forward left, and
// needs g_y's.  Tensors off the 16-byte grid keep the plain accesses.
cudaError_t set_inputs(DecayParams &p, const DecayWs &w, unsigned char *base, bool adjoint,
                       cudaStream_t st) {
    const bool keys = p.N % 8 != 0, vals = p.P % 8 != 0;
    const int n8 = (p.N + 7) / 8 * 8, p8 = (p.P + 7) / 8 * 8;
    const int64_t key_rows = p.B * p.L * p.G, val_rows = p.B * p.L * p.H;
    DecayPad t[3];
    int n = 0;
    auto pad = [&](const void *&src, size_t at, int64_t rows, int width, bool made) {
        if (!made) t[n++] = DecayPad{src, base + at, rows, width};
        src = base + at;
    };
    if (keys) {
        pad(p.c, w.pad_c, key_rows, p.N, adjoint);
        pad(p.b, w.pad_b, key_rows, p.N, adjoint);
        p.key_t = p.key_t / p.N * n8; p.key_h = p.key_h / p.N * n8; p.key_b = p.key_b / p.N * n8;
    }
    if (vals) {
        pad(p.x, w.pad_x, val_rows, p.P, adjoint);
        if (adjoint) pad(p.g_y, w.pad_v, val_rows, p.P, false);
        p.val_t = p.val_t / p.P * p8; p.val_h = p.val_h / p.P * p8; p.val_b = p.val_b / p.P * p8;
    }
    p.vec = decay_tc_copies() && all_aligned({p.c, p.b, p.x, adjoint ? p.g_y : p.x}, 16);
    return launch_decay_pad(t, n, st);
}

void set_plan(DecayParams &p, const DecayPlan &pl, const DecayWs &w, unsigned char *base) {
    p.status = reinterpret_cast<int *>(base);
    p.nseg = pl.nseg; p.seg_chunks = pl.seg_chunks; p.nchunks = pl.nchunks; p.pslices = pl.pslices;
    p.seg_state = reinterpret_cast<float *>(base + w.seg_state);
    p.seg_decay = reinterpret_cast<float *>(base + w.seg_decay);
}

pdssm_status check_scan(const pdssm_decay_dims *d, pdssm_dtype dt, pdssm_layout lay,
                        const float *log_a, const void *ws, size_t ws_bytes, bool for_bwd,
                        DecayWs *w) {
    pdssm_status st = check_dims(d, dt, false);
    if (st != PDSSM_OK) return st;
    if (lay != PDSSM_BHL && lay != PDSSM_BLH)
        return arg_fail(PDSSM_ERR_INVALID_ARG, "unknown layout");
    if (d->L > 0 && !log_a) return arg_fail(PDSSM_ERR_INVALID_ARG, "NULL log_a");
    if (!ws) return arg_fail(PDSSM_ERR_INVALID_ARG, "NULL workspace");
    if (!aligned(ws, 256)) return arg_fail(PDSSM_ERR_INVALID_ARG, "ws not 256-byte aligned");
    *w = ws_of(*d, dt, for_bwd);
    if (ws_bytes < w->total) return arg_fail(PDSSM_ERR_WORKSPACE, "workspace too small");
    return PDSSM_OK;
}

}  // namespace

extern "C" {

size_t pdssm_decay_workspace_bytes(const pdssm_decay_dims *dims, pdssm_dtype dtype, int for_bwd) {
    if (check_dims(dims, dtype, false) != PDSSM_OK) return 0;
    return ws_of(*dims, dtype, for_bwd != 0).total;
}

pdssm_status pdssm_decay_scan_fwd(const pdssm_decay_dims *dims, const void *c, const void *b,
                                  const void *x, pdssm_dtype dtype, pdssm_layout layout,
                                  const float *log_a, int log_a_per_step, const float *h0,
                                  const int32_t *lengths, void *y, float *h_last, int for_bwd,
                                  void *ws, size_t ws_bytes, void *stream) {
    DecayWs w;
    pdssm_status st = check_scan(dims, dtype, layout, log_a, ws, ws_bytes, for_bwd != 0, &w);
    if (st != PDSSM_OK) return st;
    if (dims->L > 0 && (!c || !b || !x || !y))
        return arg_fail(PDSSM_ERR_INVALID_ARG, "NULL tensor pointer");
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (dims->L == 0) {
        e = cudaMemsetAsync(ws, 0, sizeof(int), s);     // the status word
        if (e != cudaSuccess) return cuda_fail(e, "status for L = 0");
        if (h_last && h_last != h0) {
            const size_t bytes = (size_t)(dims->B * dims->H * dims->N * dims->P) * 4;
            e = h0 ? cudaMemcpyAsync(h_last, h0, bytes, cudaMemcpyDeviceToDevice, s)
                   : cudaMemsetAsync(h_last, 0, bytes, s);
            if (e != cudaSuccess) return cuda_fail(e, "h_last for L = 0");
        }
        return PDSSM_OK;
    }
    DecayParams p;
    memset(&p, 0, sizeof(p));
    unsigned char *base = reinterpret_cast<unsigned char *>(ws);
    set_strides(p, *dims, layout, log_a_per_step != 0);
    set_plan(p, decay_plan(*dims, on_tc(dtype), false), w, base);
    p.c = c; p.b = b; p.x = x; p.log_a = log_a; p.h0 = h0; p.lengths = lengths;
    p.y = y; p.h_last = h_last;
    if (for_bwd) p.carry = reinterpret_cast<float *>(base + w.carry);
    if (on_tc(dtype)) {
        e = set_inputs(p, w, base, false, s);
        if (p.P % 8) {                  // y in rows like x's
            p.y = base + w.pad_v;
            p.oval_t = p.val_t; p.oval_h = p.val_h; p.oval_b = p.val_b;
        }
        p.ovec = (p.P + 7) / 8 % 2 == 0 && aligned(p.y, 32) ? 2 : aligned(p.y, 16);
        if (e == cudaSuccess) e = launch_decay_fwd_tc(p, s);
        if (e == cudaSuccess && p.P % 8)
            e = launch_decay_unpad(p.y, y, p.B * p.L * p.H, p.P, s);
    } else {
        e = launch_decay_fwd_gen(p, s);
    }
    return e == cudaSuccess ? PDSSM_OK : cuda_fail(e, "decay scan");
}

pdssm_status pdssm_decay_wait_selftest(const pdssm_decay_dims *dims, const float *log_a, void *y,
                                       float *h_last, int for_bwd, void *ws, size_t ws_bytes,
                                       void *stream) {
    DecayWs w;
    pdssm_status st = check_scan(dims, PDSSM_BF16, PDSSM_BHL, log_a, ws, ws_bytes, for_bwd != 0, &w);
    if (st != PDSSM_OK) return st;
    if (!y || !h_last || !log_a) return arg_fail(PDSSM_ERR_INVALID_ARG, "NULL tensor pointer");
    if (!aligned(y, 16) || dims->L < 1 || dims->G != dims->H || dims->N != dims->P || dims->N % 8)
        return arg_fail(PDSSM_ERR_INVALID_ARG, "need L >= 1, G = H, N = P in eights and y on 16 bytes");
    if (!decay_tc_copies()) return arg_fail(PDSSM_ERR_UNSUPPORTED, "no tensor maps");
    DecayParams p;
    memset(&p, 0, sizeof(p));
    unsigned char *base = reinterpret_cast<unsigned char *>(ws);
    set_strides(p, *dims, PDSSM_BHL, true);
    set_plan(p, decay_plan(*dims, true, false), w, base);
    p.c = p.b = p.x = y;                // named by the tensor maps, never copied
    p.log_a = log_a; p.y = y; p.h_last = h_last;
    if (for_bwd) p.carry = reinterpret_cast<float *>(base + w.carry);
    p.vec = p.ovec = p.hold = 1;
    const cudaError_t e = launch_decay_fwd_tc(p, (cudaStream_t)stream);
    return e == cudaSuccess ? PDSSM_OK : cuda_fail(e, "decay wait self-test");
}

pdssm_status pdssm_decay_scan_bwd(const pdssm_decay_dims *dims, const void *c, const void *b,
                                  const void *x, pdssm_dtype dtype, pdssm_layout layout,
                                  const float *log_a, int log_a_per_step, const float *h0,
                                  const int32_t *lengths, const void *g_y, const float *g_hlast,
                                  void *g_c, void *g_b, void *g_x, float *g_log_a, float *g_h0,
                                  void *ws, size_t ws_bytes, void *stream) {
    DecayWs w;
    pdssm_status st = check_scan(dims, dtype, layout, log_a, ws, ws_bytes, true, &w);
    if (st != PDSSM_OK) return st;
    if (dims->L > 0 && (!c || !b || !x || !g_y || !g_c || !g_b || !g_x))
        return arg_fail(PDSSM_ERR_INVALID_ARG, "NULL tensor pointer");
    if (!g_log_a && (dims->L > 0 || !log_a_per_step))
        return arg_fail(PDSSM_ERR_INVALID_ARG, "NULL g_log_a");
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (dims->L == 0) {
        if (g_h0 && g_h0 != g_hlast) {
            const size_t bytes = (size_t)(dims->B * dims->H * dims->N * dims->P) * 4;
            e = g_hlast ? cudaMemcpyAsync(g_h0, g_hlast, bytes, cudaMemcpyDeviceToDevice, s)
                        : cudaMemsetAsync(g_h0, 0, bytes, s);
            if (e != cudaSuccess) return cuda_fail(e, "g_h0 for L = 0");
        }
        if (!log_a_per_step) {
            e = cudaMemsetAsync(g_log_a, 0, (size_t)dims->H * 4, s);
            if (e != cudaSuccess) return cuda_fail(e, "g_log_a for L = 0");
        }
        return PDSSM_OK;
    }
    DecayParams p;
    memset(&p, 0, sizeof(p));
    unsigned char *base = reinterpret_cast<unsigned char *>(ws);
    set_strides(p, *dims, layout, log_a_per_step != 0);
    set_plan(p, decay_plan(*dims, on_tc(dtype), true), w, base);
    p.c = c; p.b = b; p.x = x; p.log_a = log_a; p.h0 = h0; p.lengths = lengths;
    p.g_y = g_y; p.g_hlast = g_hlast; p.g_h0 = g_h0;
    p.carry = reinterpret_cast<float *>(base + w.carry);
    const bool shared = p.rep > 1;
    float *part_c = reinterpret_cast<float *>(base + w.part_c);
    float *part_b = reinterpret_cast<float *>(base + w.part_b);
    float *part_la = reinterpret_cast<float *>(base + w.part_la);
    p.g_c = shared ? (void *)part_c : g_c;
    p.g_b = shared ? (void *)part_b : g_b;
    p.g_x = g_x;
    p.g_la = log_a_per_step ? g_log_a : part_la;
    if (on_tc(dtype)) {
        p.ovec = p.N % 2 == 0 && p.P % 2 == 0 && all_aligned({g_c, g_b, g_x}, 4);
        e = set_inputs(p, w, base, true, s);
        if (e == cudaSuccess) e = launch_decay_bwd_mma(p, s);
    } else {
        e = launch_decay_bwd_gen(p, s);
    }
    if (e != cudaSuccess) return cuda_fail(e, "decay scan adjoint");
    if (shared) {
        e = launch_decay_sum_heads(p, dtype, part_c, part_b, g_c, g_b, s);
        if (e != cudaSuccess) return cuda_fail(e, "shared keys' gradients");
    }
    if (!log_a_per_step) {
        e = launch_decay_sum_steps(p, part_la, g_log_a, s);
        if (e != cudaSuccess) return cuda_fail(e, "per-head decays' gradient");
    }
    return PDSSM_OK;
}

pdssm_status pdssm_decay_step(const pdssm_decay_dims *dims, const void *c, const void *b,
                              const void *x, pdssm_dtype dtype, const float *log_a,
                              int log_a_per_step, float *state, int64_t n_slots,
                              const int32_t *slots, void *y, void *stream) {
    pdssm_status st = check_dims(dims, dtype, true);
    if (st != PDSSM_OK) return st;
    if (!c || !b || !x || !log_a || !y) return arg_fail(PDSSM_ERR_INVALID_ARG, "NULL tensor pointer");
    if (n_slots < 0 || n_slots > 0x7fffffff)
        return arg_fail(PDSSM_ERR_INVALID_ARG, "n_slots must lie in [0, 2^31)");
    if (!state && n_slots > 0) return arg_fail(PDSSM_ERR_INVALID_ARG, "NULL state");
    if (!slots && n_slots < dims->B)
        return arg_fail(PDSSM_ERR_INVALID_ARG, "without slots, n_slots must be >= B");
    DecayParams p;
    memset(&p, 0, sizeof(p));
    pdssm_decay_dims d = *dims;
    d.L = 1;
    set_strides(p, d, PDSSM_BHL, log_a_per_step != 0);
    p.c = c; p.b = b; p.x = x; p.log_a = log_a; p.y = y;
    p.vec = d.P % 4 == 0 && aligned(state, 16);
    cudaError_t e = launch_decay_step(p, dtype, state, n_slots, slots, (cudaStream_t)stream);
    return e == cudaSuccess ? PDSSM_OK : cuda_fail(e, "decay step");
}

}  // extern "C"
