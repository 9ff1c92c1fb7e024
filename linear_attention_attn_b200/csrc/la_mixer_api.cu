// la_mixer_api.cu -- C entry points of the operators around the token mixers: argument checks,
// workspace sizes, and what a call without tokens leaves behind.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include "la_mixer.cuh"

namespace la {
namespace {

la_status refuse(la_status s, const char *fmt, ...) {
    char buf[400];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    set_error("%s", buf);
    return s;
}

#define LA_TRY(x)                     \
    do {                              \
        la_status _rc = (x);          \
        if (_rc != LA_OK) return _rc; \
    } while (0)

bool known(la_dtype dt) { return dt == LA_F32 || dt == LA_F16 || dt == LA_BF16; }

la_status check_ws(size_t need, const void *ws, size_t bytes) {
    if (need == 0) return LA_OK;
    if (!ws) return refuse(LA_ERR_WORKSPACE, "workspace is NULL but %zu bytes are needed", need);
    if ((uintptr_t)ws & 255) return refuse(LA_ERR_ALIGNMENT, "workspace is not 256-byte aligned");
    if (bytes < need) return refuse(LA_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", bytes, need);
    return LA_OK;
}

// The tensors of one call: presence, alignment to an element, and that no output overlaps another
// tensor of the call.  in() gives the input's bit; in_place is the inputs that an output may be,
// exactly (another input at the same address is an overlap: it may be read after the output is written).
class Tensors {
public:
    explicit Tensors(bool no_tokens) : no_tokens_(no_tokens) {}
    unsigned in(const char *name, const void *p, double count, size_t elem, bool optional = false) {
        return add(name, p, count, elem, optional, false, 0);
    }
    void out(const char *name, const void *p, double count, size_t elem, bool optional = false, unsigned in_place = 0) {
        add(name, p, count, elem, optional, true, in_place);
    }
    // Presence and alignment, then the workspace (`need` bytes, if any), then the overlaps, the
    // workspace's among them.
    la_status check(size_t need = 0, const void *ws = nullptr, size_t ws_bytes = 0) {
        if (status_ != LA_OK) return refuse(status_, "%s %s", bad_, status_ == LA_ERR_INVALID_ARG ? "is NULL" : "is not aligned to its element size");
        LA_TRY(check_ws(need, ws, ws_bytes));
        if (need) out("workspace", ws, (double)need, 1);
        for (int i = 0; i < n_; ++i) {
            if (!t_[i].out) continue;
            for (int j = 0; j < n_; ++j) {
                if (j == i || (t_[j].out && j < i)) continue;
                if (t_[i].p == t_[j].p && (t_[i].in_place >> j & 1) && t_[i].bytes == t_[j].bytes) continue;
                if (t_[i].p < t_[j].p + t_[j].bytes && t_[j].p < t_[i].p + t_[i].bytes)
                    return refuse(LA_ERR_INVALID_ARG, "%s overlaps %s", t_[i].name, t_[j].name);
            }
        }
        return LA_OK;
    }

private:
    struct Tensor {
        const char *name;
        uintptr_t p, bytes;
        bool out;
        unsigned in_place;
    };
    unsigned add(const char *name, const void *p, double count, size_t elem, bool optional, bool out, unsigned in_place) {
        if (!p) {
            if (!optional && !(no_tokens_ && count == 0) && status_ == LA_OK) {
                status_ = LA_ERR_INVALID_ARG;
                bad_ = name;
            }
            return 0;
        }
        if (((uintptr_t)p & (elem - 1)) && status_ == LA_OK) {
            status_ = LA_ERR_ALIGNMENT;
            bad_ = name;
        }
        if (!(count > 0)) return 0;
        t_[n_] = Tensor{name, (uintptr_t)p, (uintptr_t)(count * elem), out, in_place};
        return 1u << n_++;
    }
    Tensor t_[24];
    int n_ = 0;
    bool no_tokens_;
    la_status status_ = LA_OK;
    const char *bad_ = "";
};

// Sizes of a [B,T,C] call: counts stay far inside 63 bits and every grid inside 2^31 blocks.
la_status check_btc(int B, int T, int C, la_dtype dt) {
    if (B < 1 || C < 1 || T < 0) return refuse(LA_ERR_INVALID_ARG, "B and C must be >= 1 and T >= 0");
    if (!known(dt)) return refuse(LA_ERR_UNSUPPORTED, "unknown dtype %d", (int)dt);
    if (C > (1 << 20) || T > (1 << 30) || (double)B * C >= 2147483648.0 || (double)B * T * C >= 1099511627776.0)
        return refuse(LA_ERR_UNSUPPORTED, "tensor too large (C <= 2^20, T <= 2^30, B*C < 2^31, B*T*C < 2^40)");
    return LA_OK;
}

la_status check_scan(int B, int T, int C, int G, int N, la_dtype dt) {
    LA_TRY(check_btc(B, T, C, dt));
    if (G < 1 || C % G) return refuse(LA_ERR_INVALID_ARG, "C=%d is not a multiple of G=%d", C, G);
    if (N < 1 || N > 64) return refuse(LA_ERR_UNSUPPORTED, "N must be in [1, 64] (got %d)", N);
    if ((double)B * T * G * N >= 34359738368.0 || (double)B * C * N >= 2147483648.0)
        return refuse(LA_ERR_UNSUPPORTED, "tensor too large (B*T*G*N < 2^35, B*C*N < 2^31)");
    return LA_OK;
}

la_status check_norm(int B, int T, int C, int G, la_dtype dt, la_activation act) {
    LA_TRY(check_btc(B, T, C, dt));
    if (G < 1 || C % G) return refuse(LA_ERR_INVALID_ARG, "C=%d is not a multiple of G=%d", C, G);
    if (act != LA_ACT_NONE && act != LA_ACT_SILU) return refuse(LA_ERR_UNSUPPORTED, "unknown activation %d", (int)act);
    return LA_OK;
}

la_status check_conv(int B, int T, int C, int W, la_dtype dt, la_activation act) {
    LA_TRY(check_btc(B, T, C, dt));
    if (W < 2 || W > 8) return refuse(LA_ERR_UNSUPPORTED, "W must be in [2, 8] (got %d)", W);
    if (act != LA_ACT_NONE && act != LA_ACT_SILU) return refuse(LA_ERR_UNSUPPORTED, "unknown activation %d", (int)act);
    return LA_OK;
}

size_t need_for(la_op op, int B, int T, int C, int G, int N, la_dtype dt) {
    switch (op) {
    case LA_OP_SHORT_CONV_BWD: return T == 0 ? 0 : conv_bwd_workspace(B, T, C, N, dt);
    case LA_OP_SELECTIVE_SCAN_FWD: return T == 0 ? 0 : scan_fwd_workspace(B, T, C, G, N);
    case LA_OP_SELECTIVE_SCAN_BWD: return T == 0 ? 0 : scan_bwd_workspace(B, T, C, G, N);
    case LA_OP_GROUP_NORM_FWD: return T == 0 ? 0 : norm_fwd_workspace(B, T, C, G, dt);
    case LA_OP_GROUP_NORM_BWD: return T == 0 ? 0 : norm_bwd_workspace(B, T, C, G, dt);
    default: return 0;
    }
}

// A state (or gradient) that passes a call without tokens: `out` becomes `in`, or zeros.
la_status pass_on(void *out, const void *in, size_t bytes, cudaStream_t st) {
    if (!out || out == in) return LA_OK;
    const cudaError_t e = in ? cudaMemcpyAsync(out, in, bytes, cudaMemcpyDeviceToDevice, st)
                             : cudaMemsetAsync(out, 0, bytes, st);
    return e == cudaSuccess ? LA_OK : cuda_fail(e, "passing on a state");
}

la_status rotary_entry(float sign, const void *q, const void *k, void *oq, void *ok, const float *freqs,
                       const long long *positions, int per_batch, long long start, la_rotary_layout layout,
                       float magnitude, int B, int H, int Hk, int T, int D, int R, la_dtype dt, void *stream) {
    const bool two = k || ok;
    if (B < 1 || H < 1 || T < 0 || (two && Hk < 1))
        return refuse(LA_ERR_INVALID_ARG, "B, H (and Hk) must be >= 1 and T >= 0");
    if (!known(dt)) return refuse(LA_ERR_UNSUPPORTED, "unknown dtype %d", (int)dt);
    if (layout != LA_ROTARY_HALF && layout != LA_ROTARY_INTERLEAVED)
        return refuse(LA_ERR_UNSUPPORTED, "unknown rotary layout %d", (int)layout);
    if (R < 2 || (R & 1) || R > D) return refuse(LA_ERR_INVALID_ARG, "R must be even and in [2, D] (R=%d, D=%d)", R, D);
    if (D > 1024) return refuse(LA_ERR_UNSUPPORTED, "D must be <= 1024 (got %d)", D);
    if (!isfinite(magnitude)) return refuse(LA_ERR_INVALID_ARG, "magnitude must be finite");
    if (per_batch != 0 && per_batch != 1) return refuse(LA_ERR_INVALID_ARG, "positions_per_batch must be 0 or 1");
    if (!two) Hk = 0;
    if ((double)H + Hk > 65535 || (double)B * T * D >= 137438953472.0 || (double)B * ((double)H + Hk) * T * D >= 1e15)
        return refuse(LA_ERR_UNSUPPORTED, "tensor too large (H + Hk <= 65535, B*T*D < 2^37)");
    const double n = (double)B * T * D;
    const size_t es = elem_bytes(dt);
    Tensors t(T == 0);
    const unsigned q_bit = t.in(sign > 0 ? "q" : "doq", q, n * H, es);
    const unsigned k_bit = two ? t.in(sign > 0 ? "k" : "dok", k, n * Hk, es) : 0;
    t.in("freqs", freqs, R / 2, 4);
    t.in("positions", positions, (double)T * (per_batch ? B : 1), 8, true);
    t.out(sign > 0 ? "oq" : "dq", oq, n * H, es, false, q_bit);
    if (two) t.out(sign > 0 ? "ok" : "dk", ok, n * Hk, es, false, k_bit);
    LA_TRY(t.check());
    if (T == 0) return LA_OK;
    return rotary(RotaryArgs{q, k, oq, ok, freqs, positions, start, per_batch, B, H, Hk, T, D, R,
                             layout == LA_ROTARY_INTERLEAVED, magnitude, sign, dt},
                  (cudaStream_t)stream);
}

la_status conv_fwd_entry(const void *x, const float *w, const float *bias, const void *state_in, void *y,
                         void *state_out, const int *lengths, la_activation act, int B, int T, int C, int W,
                         la_dtype dt, bool step, void *stream) {
    LA_TRY(check_conv(B, T, C, W, dt, act));
    const size_t es = elem_bytes(dt);
    const double n = (double)B * T * C, st = (double)B * (W - 1) * C;
    Tensors t(T == 0);
    t.in("x", x, n, es);
    t.in("w", w, (double)C * W, 4);
    t.in("bias", bias, C, 4, true);
    const unsigned state = t.in("state_in", state_in, st, es, !step);
    t.in("lengths", lengths, B, 4, true);
    t.out("y", y, n, es);
    t.out("state_out", state_out, st, es, !step, state);
    LA_TRY(t.check());
    if (T == 0) return pass_on(state_out, state_in, (size_t)st * es, (cudaStream_t)stream);
    ConvArgs a = {};
    a.x = x; a.w = w; a.bias = bias; a.state_in = state_in; a.y = y; a.state_out = state_out; a.lengths = lengths;
    a.silu = act == LA_ACT_SILU; a.B = B; a.T = T; a.C = C; a.W = W; a.dt = dt;
    return conv_fwd(a, (cudaStream_t)stream);
}

la_status scan_fwd_entry(bool step, const void *x, const void *dt, const float *A, const void *Bm, const void *Cm,
                         const float *D, const void *z, const float *dt_bias, const float *state_in, void *y,
                         float *state_out, const int *lengths, int softplus, int B, int T, int C, int G, int N,
                         la_dtype dtype, void *ws, size_t ws_bytes, void *stream) {
    LA_TRY(check_scan(B, T, C, G, N, dtype));
    if (step && B > 262140) return refuse(LA_ERR_UNSUPPORTED, "B must be <= 262140 for a step (got %d)", B);
    const size_t es = elem_bytes(dtype);
    const double n = (double)B * T * C, bc = (double)B * T * G * N, st = (double)B * C * N;
    Tensors t(T == 0);
    t.in("x", x, n, es);
    t.in("dt", dt, n, es);
    t.in("A", A, (double)C * N, 4);
    t.in("Bm", Bm, bc, es);
    t.in("Cm", Cm, bc, es);
    t.in("D", D, C, 4, true);
    t.in("z", z, n, es, true);
    t.in("dt_bias", dt_bias, C, 4, true);
    const unsigned state = t.in("state_in", state_in, st, 4, !step);
    t.in("lengths", lengths, B, 4, true);
    t.out("y", y, n, es);
    t.out("state_out", state_out, st, 4, !step, state);
    const size_t need = step ? 0 : need_for(LA_OP_SELECTIVE_SCAN_FWD, B, T, C, G, N, dtype);
    LA_TRY(t.check(need, ws, ws_bytes));
    if (T == 0) return pass_on(state_out, state_in, (size_t)st * 4, (cudaStream_t)stream);
    ScanArgs a = {};
    a.x = x; a.dt_in = dt; a.A = A; a.Bm = Bm; a.Cm = Cm; a.D = D; a.z = z; a.dt_bias = dt_bias;
    a.state_in = state_in; a.y = y; a.state_out = state_out; a.lengths = lengths; a.softplus = softplus != 0;
    a.B = B; a.T = T; a.C = C; a.G = G; a.N = N; a.dt = dtype; a.ws = ws;
    return step ? scan_step(a, (cudaStream_t)stream) : scan_fwd(a, (cudaStream_t)stream);
}

}  // namespace
}  // namespace la

using namespace la;

extern "C" {

size_t la_mixer_workspace_size(la_op op, int B, int T, int C, int G, int N, la_dtype dtype) {
    la_status ok = LA_ERR_UNSUPPORTED;
    if (op == LA_OP_SHORT_CONV_BWD) ok = check_conv(B, T, C, N, dtype, LA_ACT_NONE);
    else if (op == LA_OP_SELECTIVE_SCAN_FWD || op == LA_OP_SELECTIVE_SCAN_BWD) ok = check_scan(B, T, C, G, N, dtype);
    else if (op == LA_OP_GROUP_NORM_FWD || op == LA_OP_GROUP_NORM_BWD) ok = check_norm(B, T, C, G, dtype, LA_ACT_NONE);
    return ok == LA_OK ? need_for(op, B, T, C, G, N, dtype) : 0;
}

la_status la_rotary_fwd(const void *q, const void *k, void *oq, void *ok, const float *freqs,
                        const long long *positions, int positions_per_batch, long long start,
                        la_rotary_layout layout, float magnitude, int B, int H, int Hk, int T, int D, int R,
                        la_dtype dtype, void *stream) {
    return rotary_entry(1.f, q, k, oq, ok, freqs, positions, positions_per_batch, start, layout, magnitude, B, H, Hk,
                        T, D, R, dtype, stream);
}

la_status la_rotary_bwd(const void *doq, const void *dok, void *dq, void *dk, const float *freqs,
                        const long long *positions, int positions_per_batch, long long start,
                        la_rotary_layout layout, float magnitude, int B, int H, int Hk, int T, int D, int R,
                        la_dtype dtype, void *stream) {
    return rotary_entry(-1.f, doq, dok, dq, dk, freqs, positions, positions_per_batch, start, layout, magnitude, B, H,
                        Hk, T, D, R, dtype, stream);
}

la_status la_rotary_frequencies(float *freqs, int R, double base, la_rotary_scaling scaling, double factor,
                                double original_length, double beta_fast, double beta_slow) {
    if (!freqs) return refuse(LA_ERR_INVALID_ARG, "freqs is NULL");
    if (R < 2 || (R & 1)) return refuse(LA_ERR_INVALID_ARG, "R must be even and >= 2 (got %d)", R);
    if (!(base > 0) || !isfinite(base)) return refuse(LA_ERR_INVALID_ARG, "base must be positive and finite");
    if (scaling != LA_ROTARY_SCALE_NONE && scaling != LA_ROTARY_SCALE_LINEAR && scaling != LA_ROTARY_SCALE_NTK &&
        scaling != LA_ROTARY_SCALE_BY_PARTS)
        return refuse(LA_ERR_UNSUPPORTED, "unknown rotary scaling %d", (int)scaling);
    if (scaling != LA_ROTARY_SCALE_NONE && (!(factor >= 1) || !isfinite(factor)))
        return refuse(LA_ERR_INVALID_ARG, "factor must be finite and >= 1");
    if (scaling == LA_ROTARY_SCALE_NTK && R == 2)
        return refuse(LA_ERR_INVALID_ARG, "the NTK scaling needs R > 2");
    if (scaling == LA_ROTARY_SCALE_BY_PARTS &&
        (!(original_length > 0) || !isfinite(original_length) || !(beta_slow >= 0) || !(beta_fast > beta_slow) ||
         !isfinite(beta_fast)))
        return refuse(LA_ERR_INVALID_ARG, "scaling by parts needs original_length > 0 and beta_fast > beta_slow >= 0");
    if (scaling == LA_ROTARY_SCALE_NTK) base *= pow(factor, R / (R - 2.0));
    for (int i = 0; i < R / 2; ++i) {
        double f = pow(base, -2.0 * i / R);
        if (scaling == LA_ROTARY_SCALE_LINEAR) f /= factor;
        if (scaling == LA_ROTARY_SCALE_BY_PARTS) {
            const double turns = original_length * f / 6.283185307179586477;
            double keep = (turns - beta_slow) / (beta_fast - beta_slow);
            keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
            f = f * keep + f / factor * (1 - keep);
        }
        freqs[i] = (float)f;
    }
    return LA_OK;
}

la_status la_short_conv_fwd(const void *x, const float *w, const float *bias, const void *state_in, void *y,
                            void *state_out, const int *lengths, la_activation act, int B, int T, int C, int W,
                            la_dtype dtype, void *stream) {
    return conv_fwd_entry(x, w, bias, state_in, y, state_out, lengths, act, B, T, C, W, dtype, false, stream);
}

la_status la_short_conv_step(const void *x, const float *w, const float *bias, const void *state_in, void *y,
                             void *state_out, la_activation act, int B, int C, int W, la_dtype dtype, void *stream) {
    return conv_fwd_entry(x, w, bias, state_in, y, state_out, nullptr, act, B, 1, C, W, dtype, true, stream);
}

la_status la_short_conv_bwd(const void *x, const float *w, const float *bias, const void *state_in, const void *dy,
                            const void *dstate_in, void *dx, float *dw, float *dbias, void *dstate_out,
                            const int *lengths, la_activation act, int B, int T, int C, int W, la_dtype dtype,
                            void *workspace, size_t workspace_bytes, void *stream) {
    LA_TRY(check_conv(B, T, C, W, dtype, act));
    const size_t es = elem_bytes(dtype);
    const double n = (double)B * T * C, st = (double)B * (W - 1) * C;
    const size_t need = need_for(LA_OP_SHORT_CONV_BWD, B, T, C, 1, W, dtype);
    Tensors t(T == 0);
    t.in("x", x, n, es);
    t.in("w", w, (double)C * W, 4);
    t.in("bias", bias, C, 4, true);
    t.in("state_in", state_in, st, es, true);
    t.in("dy", dy, n, es);
    t.in("dstate_in", dstate_in, st, es, true);
    t.in("lengths", lengths, B, 4, true);
    t.out("dx", dx, n, es);
    t.out("dw", dw, (double)C * W, 4);
    t.out("dbias", dbias, C, 4, true);
    t.out("dstate_out", dstate_out, st, es, true);
    LA_TRY(t.check(need, workspace, workspace_bytes));
    cudaStream_t s = (cudaStream_t)stream;
    if (T == 0) {
        LA_TRY(pass_on(dw, nullptr, (size_t)C * W * 4, s));
        LA_TRY(pass_on(dbias, nullptr, (size_t)C * 4, s));
        return pass_on(dstate_out, dstate_in, (size_t)st * es, s);
    }
    ConvArgs a = {};
    a.x = x; a.dy = dy; a.state_in = state_in; a.dstate_in = dstate_in; a.w = w; a.bias = bias; a.lengths = lengths;
    a.dx = dx; a.dstate_out = dstate_out; a.dw = dw; a.dbias = dbias;
    a.B = B; a.T = T; a.C = C; a.W = W; a.silu = act == LA_ACT_SILU; a.dt = dtype; a.ws = workspace;
    return conv_bwd(a, s);
}

la_status la_selective_scan_fwd(const void *x, const void *dt, const float *A, const void *Bm, const void *Cm,
                                const float *D, const void *z, const float *dt_bias, const float *state_in, void *y,
                                float *state_out, const int *lengths, int softplus, int B, int T, int C, int G, int N,
                                la_dtype dtype, void *workspace, size_t workspace_bytes, void *stream) {
    return scan_fwd_entry(false, x, dt, A, Bm, Cm, D, z, dt_bias, state_in, y, state_out, lengths, softplus, B, T, C, G,
                          N, dtype, workspace, workspace_bytes, stream);
}

la_status la_selective_scan_step(const void *x, const void *dt, const float *A, const void *Bm, const void *Cm,
                                 const float *D, const void *z, const float *dt_bias, const float *state_in, void *y,
                                 float *state_out, int softplus, int B, int C, int G, int N, la_dtype dtype,
                                 void *stream) {
    return scan_fwd_entry(true, x, dt, A, Bm, Cm, D, z, dt_bias, state_in, y, state_out, nullptr, softplus, B, 1, C, G,
                          N, dtype, nullptr, 0, stream);
}

la_status la_selective_scan_bwd(const void *x, const void *dt, const float *A, const void *Bm, const void *Cm,
                                const float *D, const void *z, const float *dt_bias, const float *state_in,
                                const void *dy, const float *dstate_in, void *dx, void *ddt, float *dA, void *dBm,
                                void *dCm, float *dD, void *dz, float *ddt_bias, float *dstate_out,
                                const int *lengths, int softplus, int B, int T, int C, int G, int N, la_dtype dtype,
                                void *workspace, size_t workspace_bytes, void *stream) {
    LA_TRY(check_scan(B, T, C, G, N, dtype));
    if (!z != !dz && T > 0) return refuse(LA_ERR_INVALID_ARG, "z and dz must be given together");
    const size_t es = elem_bytes(dtype);
    const double n = (double)B * T * C, bc = (double)B * T * G * N, st = (double)B * C * N;
    const size_t need = need_for(LA_OP_SELECTIVE_SCAN_BWD, B, T, C, G, N, dtype);
    Tensors t(T == 0);
    t.in("x", x, n, es);
    t.in("dt", dt, n, es);
    t.in("A", A, (double)C * N, 4);
    t.in("Bm", Bm, bc, es);
    t.in("Cm", Cm, bc, es);
    t.in("D", D, C, 4, true);
    t.in("z", z, n, es, true);
    t.in("dt_bias", dt_bias, C, 4, true);
    t.in("state_in", state_in, st, 4, true);
    t.in("dy", dy, n, es);
    t.in("dstate_in", dstate_in, st, 4, true);
    t.in("lengths", lengths, B, 4, true);
    t.out("dx", dx, n, es);
    t.out("ddt", ddt, n, es);
    t.out("dA", dA, (double)C * N, 4);
    t.out("dBm", dBm, bc, es);
    t.out("dCm", dCm, bc, es);
    t.out("dD", dD, C, 4, true);
    t.out("dz", dz, n, es, true);
    t.out("ddt_bias", ddt_bias, C, 4, true);
    t.out("dstate_out", dstate_out, st, 4, true);
    LA_TRY(t.check(need, workspace, workspace_bytes));
    cudaStream_t s = (cudaStream_t)stream;
    if (T == 0) {
        LA_TRY(pass_on(dA, nullptr, (size_t)C * N * 4, s));
        LA_TRY(pass_on(dD, nullptr, (size_t)C * 4, s));
        LA_TRY(pass_on(ddt_bias, nullptr, (size_t)C * 4, s));
        return pass_on(dstate_out, dstate_in, (size_t)st * 4, s);
    }
    ScanArgs a = {};
    a.x = x; a.dt_in = dt; a.A = A; a.Bm = Bm; a.Cm = Cm; a.D = D; a.z = z; a.dt_bias = dt_bias;
    a.state_in = state_in; a.dy = dy; a.dstate_in = dstate_in; a.lengths = lengths;
    a.dx = dx; a.ddt = ddt; a.dA = dA; a.dBm = dBm; a.dCm = dCm; a.dD = dD; a.dz = dz; a.ddt_bias = ddt_bias;
    a.dstate_out = dstate_out; a.softplus = softplus != 0;
    a.B = B; a.T = T; a.C = C; a.G = G; a.N = N; a.dt = dtype; a.ws = workspace;
    return scan_bwd(a, s);
}

la_status la_group_norm_fwd(const void *x, const float *gamma, const float *beta, void *y, float *mean, float *rstd,
                            float eps, la_activation act, int B, int T, int C, int G, la_dtype dtype,
                            void *workspace, size_t workspace_bytes, void *stream) {
    LA_TRY(check_norm(B, T, C, G, dtype, act));
    if (!(eps > 0.f) || !isfinite(eps)) return refuse(LA_ERR_INVALID_ARG, "eps must be finite and > 0");
    const size_t es = elem_bytes(dtype);
    const double n = (double)B * T * C, bg = (double)B * G;
    const size_t need = need_for(LA_OP_GROUP_NORM_FWD, B, T, C, G, 1, dtype);
    Tensors t(T == 0);
    const unsigned x_bit = t.in("x", x, n, es);
    t.in("gamma", gamma, C, 4, true);
    t.in("beta", beta, C, 4, true);
    t.out("y", y, n, es, false, x_bit);
    t.out("mean", mean, bg, 4, true);
    t.out("rstd", rstd, bg, 4, true);
    LA_TRY(t.check(need, workspace, workspace_bytes));
    cudaStream_t s = (cudaStream_t)stream;
    if (T == 0) {
        LA_TRY(pass_on(mean, nullptr, (size_t)bg * 4, s));
        return pass_on(rstd, nullptr, (size_t)bg * 4, s);
    }
    NormArgs a = {};
    a.x = x; a.gamma = gamma; a.beta = beta; a.y = y; a.mean = mean; a.rstd = rstd;
    a.B = B; a.T = T; a.C = C; a.G = G; a.silu = act == LA_ACT_SILU; a.eps = eps; a.dt = dtype; a.ws = workspace;
    return norm_fwd(a, s);
}

la_status la_group_norm_bwd(const void *x, const void *dy, const float *mean, const float *rstd, const float *gamma,
                            const float *beta, void *dx, float *dgamma, float *dbeta, la_activation act, int B, int T,
                            int C, int G, la_dtype dtype, void *workspace, size_t workspace_bytes, void *stream) {
    LA_TRY(check_norm(B, T, C, G, dtype, act));
    const size_t es = elem_bytes(dtype);
    const double n = (double)B * T * C, bg = (double)B * G;
    const size_t need = need_for(LA_OP_GROUP_NORM_BWD, B, T, C, G, 1, dtype);
    Tensors t(T == 0);
    // every element of x and dy is read by the thread that writes it in dx, and the sums are done by
    // then: dx may be dy, also where dy is x
    const unsigned x_bit = t.in("x", x, n, es), dy_bit = t.in("dy", dy, n, es);
    t.in("mean", mean, bg, 4);
    t.in("rstd", rstd, bg, 4);
    t.in("gamma", gamma, C, 4, true);
    t.in("beta", beta, C, 4, true);
    t.out("dx", dx, n, es, false, dy_bit | (x == dy ? x_bit : 0));
    t.out("dgamma", dgamma, C, 4, true);
    t.out("dbeta", dbeta, C, 4, true);
    LA_TRY(t.check(need, workspace, workspace_bytes));
    cudaStream_t s = (cudaStream_t)stream;
    if (T == 0) {
        LA_TRY(pass_on(dgamma, nullptr, (size_t)C * 4, s));
        return pass_on(dbeta, nullptr, (size_t)C * 4, s);
    }
    NormArgs a = {};
    a.x = x; a.dy = dy; a.mean_in = mean; a.rstd_in = rstd; a.gamma = gamma; a.beta = beta; a.dx = dx;
    a.dgamma = dgamma; a.dbeta = dbeta;
    a.B = B; a.T = T; a.C = C; a.G = G; a.silu = act == LA_ACT_SILU; a.dt = dtype; a.ws = workspace;
    return norm_bwd(a, s);
}

}  // extern "C"
