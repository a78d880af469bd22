// Native half of the block operators' binding (blocks.py): checks tensors,
// allocates outputs and calls the C ABI.  These calls are short (a decoded
// token's norm or step runs for 3 microseconds), so the host's part decides
// how fast they follow one another: 5.5 microseconds a call of the step here,
// 12.6 through ctypes.
//
// A wrong argument raises ValueError, a status of the library PdssmError.
// Every tensor of a call lies on one CUDA device, which need not be the
// current one; work goes to that device's current stream.
#include <torch/csrc/utils/pybind.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <optional>
#include <tuple>

#include "../../include/pdssm.h"

namespace {

namespace py = pybind11;
using at::IntArrayRef;
using at::ScalarType;
using at::Tensor;
using MaybeT = std::optional<Tensor>;

constexpr auto kF32 = at::kFloat, kI32 = at::kInt, kU8 = at::kByte;

[[noreturn]] void refuse(const std::string &why) { throw py::value_error(why); }

std::string text(IntArrayRef s) {
    std::string o = "(";
    for (size_t i = 0; i < s.size(); ++i) o += (i ? ", " : "") + std::to_string(s[i]);
    return o + ")";
}

// One call: its device, and the checks of its tensors.
struct Call {
    const char *what;
    int dev;
    c10::cuda::OptionalCUDAGuard guard;
    Call(const char *what, const Tensor &first, const char *name) : what(what) {
        if (!first.defined() || !first.is_cuda())
            refuse(std::string(name) + " must be a CUDA tensor (no CPU path)");
        dev = first.get_device();
        guard.set_index((c10::DeviceIndex)dev);
    }
    void *stream() const { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }

    void *plain(const Tensor &t, const char *name) const {
        if (!t.defined() || !t.is_cuda())
            refuse(std::string(name) + " must be a CUDA tensor (no CPU path)");
        if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
        if (t.get_device() != dev)
            refuse(std::string(name) + " is on " + t.device().str() + ", expected cuda:" + std::to_string(dev));
        return t.data_ptr();
    }
    void *arg(const Tensor &t, const char *name, ScalarType type) const {
        void *p = plain(t, name);
        if (t.scalar_type() != type)
            refuse(std::string(name) + " has dtype " + c10::toString(t.scalar_type()) + ", expected " +
                   c10::toString(type));
        return p;
    }
    void *arg(const Tensor &t, const char *name, ScalarType type, IntArrayRef shape) const {
        void *p = arg(t, name, type);
        if (t.sizes() != shape)
            refuse(std::string(name) + " has shape " + text(t.sizes()) + ", expected " + text(shape));
        return p;
    }
    template <class... A>
    void *opt(const MaybeT &t, A &&...a) const {
        return t.has_value() ? arg(*t, std::forward<A>(a)...) : nullptr;
    }
    // fp32 or bf16, of any shape
    pdssm_dtype wide(const Tensor &t, const char *name) const {
        plain(t, name);
        if (t.scalar_type() == at::kFloat) return PDSSM_F32;
        if (t.scalar_type() == at::kBFloat16) return PDSSM_BF16;
        refuse(std::string(name) + " has dtype " + c10::toString(t.scalar_type()) + ", expected Float or BFloat16");
    }
    Tensor fresh(IntArrayRef shape, ScalarType type) const {
        return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, (c10::DeviceIndex)dev));
    }
    // a caller's output buffer, checked, or a new one
    Tensor out(const MaybeT &t, const char *name, ScalarType type, IntArrayRef shape) const {
        if (!t.has_value()) return fresh(shape, type);
        arg(*t, name, type, shape);
        return *t;
    }
    void check(pdssm_status st) const {
        if (st == PDSSM_OK) return;
        py::object cls = py::module_::import("structured_sparse_state_b200").attr("PdssmError");
        py::object e = cls((int)st, what);
        PyErr_SetObject(cls.ptr(), e.ptr());
        throw py::error_already_set();
    }
};

pdssm_dtype code(ScalarType t) {
    return t == at::kBFloat16 ? PDSSM_BF16 : t == at::kFloat8_e4m3fn ? PDSSM_E4M3 : PDSSM_F32;
}

float *f32(const Tensor &t) { return static_cast<float *>(t.data_ptr()); }

// ---------------------------------------------------------------------------
// decay scan
// ---------------------------------------------------------------------------
struct Scan {
    pdssm_decay_dims d;
    pdssm_layout layout;
    pdssm_dtype dt;
    int per_step;
    void *c, *b, *x;
    float *log_a;
    int64_t state[4];
    Scan(const Call &k, const Tensor &tc, const Tensor &tb, const Tensor &tx, const Tensor &la, bool blh) {
        dt = k.wide(tx, "x");
        if (tx.dim() != 4 || tc.dim() != 4) refuse("x and c must have four dimensions");
        layout = blh ? PDSSM_BLH : PDSSM_BHL;
        const int h = blh ? 2 : 1, l = blh ? 1 : 2;
        d = {tx.size(0), tx.size(h), tc.size(h), tx.size(l), tc.size(3), tx.size(3)};
        int64_t keys[4] = {d.B, 0, 0, d.N}, gate[3] = {d.B, 0, 0};
        keys[h] = d.G;
        keys[l] = d.L;
        gate[h] = d.H;
        gate[l] = d.L;
        c = k.arg(tc, "c", tx.scalar_type(), keys);
        b = k.arg(tb, "b", tx.scalar_type(), keys);
        x = tx.data_ptr();
        if (d.G == 0 || d.H % d.G)
            refuse(std::to_string(d.H) + " heads cannot share " + std::to_string(d.G) + " groups of c and b");
        per_step = la.dim() != 1;
        log_a = static_cast<float *>(per_step ? k.arg(la, "log_a", kF32, gate)
                                              : k.arg(la, "log_a", kF32, {d.H}));
        state[0] = d.B; state[1] = d.H; state[2] = d.N; state[3] = d.P;
    }
};

std::tuple<Tensor, Tensor, Tensor> decay_scan_fwd(const Tensor &c, const Tensor &b, const Tensor &x,
                                                  const Tensor &log_a, const MaybeT &h0,
                                                  const MaybeT &lengths, bool blh, bool for_bwd,
                                                  const MaybeT &ws_in, const MaybeT &y_in,
                                                  const MaybeT &h_in) {
    Call k("pdssm_decay_scan_fwd", x, "x");
    Scan s(k, c, b, x, log_a, blh);
    auto *ph0 = static_cast<float *>(k.opt(h0, "h0", kF32, s.state));
    auto *pn = static_cast<int32_t *>(k.opt(lengths, "lengths", kI32, IntArrayRef{s.d.B}));
    // sizes outside the limits need 0 bytes: the call itself then says which
    size_t n = ws_in.has_value() ? 0 : pdssm_decay_workspace_bytes(&s.d, s.dt, for_bwd);
    Tensor ws = ws_in.has_value() ? *ws_in : k.fresh({(int64_t)(n ? n : 256)}, kU8);
    void *pws = k.arg(ws, "ws", kU8);
    Tensor y = k.out(y_in, "y", x.scalar_type(), x.sizes());
    Tensor h = k.out(h_in, "h_last", kF32, s.state);
    k.check(pdssm_decay_scan_fwd(&s.d, s.c, s.b, s.x, s.dt, s.layout, s.log_a, s.per_step, ph0, pn,
                                 y.data_ptr(), f32(h), for_bwd, pws, (size_t)ws.numel(), k.stream()));
    return {y, h, ws};
}

std::tuple<Tensor, Tensor, Tensor, Tensor, Tensor> decay_scan_bwd(
    const Tensor &c, const Tensor &b, const Tensor &x, const Tensor &log_a, const MaybeT &h0,
    const Tensor &g_y, const Tensor &ws, const MaybeT &g_hlast, const MaybeT &lengths, bool blh,
    const MaybeT &gc_in, const MaybeT &gb_in, const MaybeT &gx_in, const MaybeT &gla_in,
    const MaybeT &gh0_in) {
    Call k("pdssm_decay_scan_bwd", x, "x");
    Scan s(k, c, b, x, log_a, blh);
    auto *ph0 = static_cast<float *>(k.opt(h0, "h0", kF32, s.state));
    auto *pgh = static_cast<float *>(k.opt(g_hlast, "g_hlast", kF32, s.state));
    auto *pn = static_cast<int32_t *>(k.opt(lengths, "lengths", kI32, IntArrayRef{s.d.B}));
    void *pgy = k.arg(g_y, "g_y", x.scalar_type(), x.sizes());
    void *pws = k.arg(ws, "ws", kU8);
    Tensor gc = k.out(gc_in, "g_c", x.scalar_type(), c.sizes());
    Tensor gb = k.out(gb_in, "g_b", x.scalar_type(), c.sizes());
    Tensor gx = k.out(gx_in, "g_x", x.scalar_type(), x.sizes());
    Tensor gla = k.out(gla_in, "g_log_a", kF32, log_a.sizes());
    Tensor gh0 = k.out(gh0_in, "g_h0", kF32, s.state);
    k.check(pdssm_decay_scan_bwd(&s.d, s.c, s.b, s.x, s.dt, s.layout, s.log_a, s.per_step, ph0, pn, pgy,
                                 pgh, gc.data_ptr(), gb.data_ptr(), gx.data_ptr(), f32(gla), f32(gh0), pws,
                                 (size_t)ws.numel(), k.stream()));
    return {gc, gb, gx, gla, gh0};
}

Tensor decay_step(const Tensor &c, const Tensor &b, const Tensor &x, const Tensor &log_a,
                  const Tensor &state, const MaybeT &slots, const MaybeT &y_in) {
    Call k("pdssm_decay_step", x, "x");
    const pdssm_dtype dt = k.wide(x, "x");
    if (x.dim() != 3 || c.dim() != 3) refuse("x and c must have three dimensions");
    pdssm_decay_dims d = {x.size(0), x.size(1), c.size(1), 1, c.size(2), x.size(2)};
    void *pc = k.arg(c, "c", x.scalar_type(), {d.B, d.G, d.N});
    void *pb = k.arg(b, "b", x.scalar_type(), {d.B, d.G, d.N});
    if (d.G == 0 || d.H % d.G)
        refuse(std::to_string(d.H) + " heads cannot share " + std::to_string(d.G) + " groups of c and b");
    const int per_step = log_a.dim() != 1;
    void *pla = per_step ? k.arg(log_a, "log_a", kF32, {d.B, d.H}) : k.arg(log_a, "log_a", kF32, {d.H});
    const int64_t n = state.dim() ? state.size(0) : 0;
    void *ps = k.arg(state, "state", kF32, {n, d.H, d.N, d.P});
    auto *pslots = static_cast<int32_t *>(k.opt(slots, "slots", kI32, IntArrayRef{d.B}));
    Tensor y = k.out(y_in, "y", x.scalar_type(), x.sizes());
    k.check(pdssm_decay_step(&d, pc, pb, x.data_ptr(), dt, static_cast<float *>(pla), per_step,
                             static_cast<float *>(ps), n, pslots, y.data_ptr(), k.stream()));
    return y;
}

// ---------------------------------------------------------------------------
// residual addition and root-mean-square norm
// ---------------------------------------------------------------------------
std::tuple<Tensor, Tensor, Tensor, MaybeT> add_rmsnorm_fwd(const Tensor &x, const MaybeT &residual,
                                                           const Tensor &weight, double eps,
                                                           std::optional<ScalarType> out_type,
                                                           const MaybeT &out_in, const MaybeT &res_in,
                                                           const MaybeT &rstd_in, const MaybeT &scale_in) {
    Call k("pdssm_add_rmsnorm_fwd", x, "x");
    const pdssm_dtype xt = k.wide(x, "x");
    if (x.dim() < 1) refuse("x must have at least one dimension");
    const int64_t D = x.size(-1);
    const IntArrayRef lead = x.sizes().slice(0, x.dim() - 1);
    int64_t rows = 1;
    for (int64_t n : lead) rows *= n;
    const void *pr = nullptr;
    ScalarType rt = x.scalar_type();
    if (residual.has_value()) {
        k.wide(*residual, "residual");
        rt = residual->scalar_type();
        pr = k.arg(*residual, "residual", rt, x.sizes());
    }
    const pdssm_dtype wt = k.wide(weight, "weight");
    k.arg(weight, "weight", weight.scalar_type(), {D});
    const ScalarType ot = out_type.value_or(x.scalar_type());
    if (ot != at::kFloat && ot != at::kBFloat16 && ot != at::kFloat8_e4m3fn)
        refuse(std::string("out_dtype ") + c10::toString(ot) + ", expected Float, BFloat16 or Float8_e4m3fn");
    Tensor out = k.out(out_in, "out", ot, x.sizes());
    Tensor res = k.out(res_in, "res_out", rt, x.sizes());
    Tensor rstd = k.out(rstd_in, "rstd", kF32, lead);
    MaybeT scale;
    if (ot == at::kFloat8_e4m3fn)
        scale = k.out(scale_in, "scale", kF32, lead);
    else if (scale_in.has_value())
        refuse("scale goes with an 8-bit output only");
    k.check(pdssm_add_rmsnorm_fwd(rows, D, x.data_ptr(), xt, pr, code(rt), weight.data_ptr(), wt, (float)eps,
                                  out.data_ptr(), code(ot), res.data_ptr(), f32(rstd),
                                  scale.has_value() ? f32(*scale) : nullptr, k.stream()));
    return {out, res, rstd, scale};
}

std::tuple<Tensor, Tensor> add_rmsnorm_bwd(const Tensor &g_out, const Tensor &res_out,
                                           const Tensor &weight, const Tensor &rstd, const MaybeT &g_res,
                                           const MaybeT &gx_in, const MaybeT &gw_in,
                                           const MaybeT &scratch_in) {
    Call k("pdssm_add_rmsnorm_bwd", res_out, "res_out");
    const pdssm_dtype rt = k.wide(res_out, "res_out");
    if (res_out.dim() < 1) refuse("res_out must have at least one dimension");
    const int64_t D = res_out.size(-1);
    const pdssm_dtype gt = k.wide(g_out, "g_out");
    k.arg(g_out, "g_out", g_out.scalar_type(), res_out.sizes());
    const pdssm_dtype wt = k.wide(weight, "weight");
    k.arg(weight, "weight", weight.scalar_type(), {D});
    k.arg(rstd, "rstd", kF32, res_out.sizes().slice(0, res_out.dim() - 1));
    void *pr = k.opt(g_res, "g_res", res_out.scalar_type(), res_out.sizes());
    const int64_t rows = rstd.numel();
    Tensor gx = k.out(gx_in, "g_x", res_out.scalar_type(), res_out.sizes());
    Tensor gw = k.out(gw_in, "g_weight", kF32, {D});
    const size_t n = scratch_in.has_value() ? 0 : pdssm_add_rmsnorm_scratch_bytes(rows, D);
    Tensor scratch = scratch_in.has_value() ? *scratch_in : k.fresh({(int64_t)(n ? n : 256)}, kU8);
    k.arg(scratch, "scratch", kU8);
    k.check(pdssm_add_rmsnorm_bwd(rows, D, g_out.data_ptr(), gt, res_out.data_ptr(), rt, weight.data_ptr(), wt,
                                  f32(rstd), pr, gx.data_ptr(), f32(gw), scratch.data_ptr(),
                                  (size_t)scratch.numel(), k.stream()));
    return {gx, gw};
}

// ---------------------------------------------------------------------------
// balance of the hard selection
// ---------------------------------------------------------------------------
struct Balance {
    pdssm_dims d;
    pdssm_dtype dt;
    const float *W;
    const int32_t *lengths;
    Balance(const Call &k, const Tensor &u, const Tensor &W_sel, const MaybeT &n) {
        dt = k.wide(u, "u");
        if (u.dim() != 3) refuse("u must be [B, L, D_in]");
        W = static_cast<float *>(k.arg(W_sel, "W_sel", kF32));
        if (W_sel.dim() != 3 || W_sel.size(2) != u.size(2)) refuse("W_sel must be [H, K, D_in]");
        d = {u.size(0), W_sel.size(0), u.size(1), 0, W_sel.size(1), u.size(2)};
        lengths = static_cast<int32_t *>(k.opt(n, "lengths", kI32, IntArrayRef{d.B}));
    }
    Tensor scratch(const Call &k, const MaybeT &given) const {
        if (given.has_value()) {
            k.arg(*given, "scratch", kU8);
            return *given;
        }
        const size_t n = pdssm_select_balance_scratch_bytes(&d);
        return k.fresh({(int64_t)(n ? n : 256)}, kU8);
    }
};

std::tuple<Tensor, Tensor, Tensor> select_balance_fwd(const Tensor &u, const Tensor &W_sel, const Tensor &sel,
                                                      double inv_tau, const MaybeT &lengths,
                                                      const MaybeT &scratch_in) {
    Call k("pdssm_select_balance_fwd", u, "u");
    Balance s(k, u, W_sel, lengths);
    auto *pk = static_cast<int32_t *>(k.arg(sel, "k", kI32, {s.d.B, s.d.H, s.d.L}));
    Tensor loss = k.fresh({s.d.H}, kF32), counts = k.fresh({s.d.H, s.d.K}, kI32),
           probs = k.fresh({s.d.H, s.d.K}, kF32), scratch = s.scratch(k, scratch_in);
    k.check(pdssm_select_balance_fwd(&s.d, u.data_ptr(), s.dt, s.W, pk, (float)inv_tau, s.lengths, f32(loss),
                                     static_cast<int32_t *>(counts.data_ptr()), f32(probs), scratch.data_ptr(),
                                     (size_t)scratch.numel(), k.stream()));
    return {loss, counts, probs};
}

std::tuple<Tensor, Tensor> select_balance_bwd(const Tensor &u, const Tensor &W_sel, const Tensor &counts,
                                              const Tensor &g_loss, double inv_tau, const MaybeT &lengths,
                                              const MaybeT &scratch_in) {
    Call k("pdssm_select_balance_bwd", u, "u");
    Balance s(k, u, W_sel, lengths);
    auto *pk = static_cast<int32_t *>(k.arg(counts, "counts", kI32, {s.d.H, s.d.K}));
    auto *pg = static_cast<float *>(k.arg(g_loss, "g_loss", kF32, {s.d.H}));
    Tensor gu = k.fresh(u.sizes(), u.scalar_type()), gw = k.fresh(W_sel.sizes(), kF32),
           scratch = s.scratch(k, scratch_in);
    k.check(pdssm_select_balance_bwd(&s.d, u.data_ptr(), s.dt, s.W, pk, (float)inv_tau, s.lengths, pg,
                                     gu.data_ptr(), f32(gw), scratch.data_ptr(), (size_t)scratch.numel(),
                                     k.stream()));
    return {gu, gw};
}

}  // namespace

PYBIND11_MODULE(_blocks, m) {
    m.doc() = "Checks and calls of the block operators (used by blocks.py).";
    m.def("decay_scan_fwd", &decay_scan_fwd);
    m.def("decay_scan_bwd", &decay_scan_bwd);
    m.def("decay_step", &decay_step);
    m.def("add_rmsnorm_fwd", &add_rmsnorm_fwd);
    m.def("add_rmsnorm_bwd", &add_rmsnorm_bwd);
    m.def("select_balance_fwd", &select_balance_fwd);
    m.def("select_balance_bwd", &select_balance_bwd);
}
