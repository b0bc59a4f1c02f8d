// C ABI of the sequence operators: argument validation and launch. Declarations and the
// contract of every entry point: include/sequence_ops.h.
#include <initializer_list>

#include "kernels.hpp"
#include "runtime.hpp"

namespace {

using namespace c2d;

constexpr long long kMaxTokens = 1ll << 30;
// Channels of a token, and inputs or outputs of a product: the kernels round them up to whole
// blocks and tiles in 32 bits.
constexpr int kMaxWidth = 1 << 30;

// Memory that a call reads or writes.
struct Extent {
    const char *name;
    const void *p;
    long long bytes;
};

struct Rows {
    const char *name;
    const void *p;
    long long batch, token, width;  // elements
};

// Sequence geometry common to the prompt and single-token calls.
struct Shape {
    const char *op;
    long long tokens;
    int nseq, dtype;
    bool packed, step;
    long long rows() const { return step ? nseq : packed ? tokens : tokens * nseq; }
};

int check_shape(Shape *s, const int *offsets, const int *slots, int state_rows) {
    if (!dtype_bytes(s->dtype)) return set_error(CONV2D_EINVAL, "%s: unknown dtype %d", s->op, s->dtype);
    if (s->nseq < 0 || s->tokens < 0 || state_rows < 0)
        return set_error(CONV2D_EINVAL, "%s: sizes must not be negative (nseq=%d tokens=%lld state_rows=%d)", s->op,
                         s->nseq, s->tokens, state_rows);
    if (s->step && (offsets || s->tokens != 1))
        return set_error(CONV2D_EINVAL, "%s: takes one token of each sequence and no offsets", s->op);
    s->packed = offsets != nullptr;
    if (((uintptr_t)offsets | (uintptr_t)slots) % 4)
        return set_error(CONV2D_EINVAL, "%s: offsets and slots must be 4-byte aligned", s->op);
    if (s->nseq > kMaxTokens || s->tokens > kMaxTokens || s->rows() > kMaxTokens)
        return set_error(CONV2D_EUNSUPPORTED, "%s: more than 2^30 tokens are not supported", s->op);
    return CONV2D_OK;
}

// The bytes from the first to the last value of the rows; negative: refused, error set.
long long rows_bytes(const Shape &s, const Rows &r) {
    const int eb = dtype_bytes(s.dtype);
    if (!r.p && s.rows() > 0) return set_error(CONV2D_EINVAL, "%s: %s must not be null", s.op, r.name);
    if ((uintptr_t)r.p % eb) return set_error(CONV2D_EINVAL, "%s: %s is not aligned to its type", s.op, r.name);
    if (r.token < 0 || r.batch < 0) return set_error(CONV2D_EINVAL, "%s: %s has a negative stride", s.op, r.name);
    const __int128 b = s.step ? s.nseq : s.packed ? 1 : s.nseq, t = s.step ? 1 : s.tokens;
    if (b == 0 || t == 0) return 0;
    const __int128 last = (b - 1) * (s.step ? r.token : r.batch) + (t - 1) * r.token + r.width;
    if (last > (__int128)1 << 45) return set_error(CONV2D_EINVAL, "%s: %s reaches too far", s.op, r.name);
    return (long long)last * eb;
}

// Whether no two rows share memory, as those of an output must not.
bool rows_disjoint(const Shape &s, const Rows &r) {
    if (s.rows() == 0) return true;
    if (s.step || s.packed) return s.rows() <= 1 || r.token >= r.width;
    if (s.tokens > 1 && r.token < r.width) return false;
    if (s.nseq > 1 && r.batch < r.width) return false;
    if (s.tokens <= 1 || s.nseq <= 1) return true;
    return r.batch >= (__int128)(s.tokens - 1) * r.token + r.width ||
           r.token >= (__int128)(s.nseq - 1) * r.batch + r.width;
}

int check_no_overlap(const char *op, const Extent &out, std::initializer_list<Extent> others) {
    for (const Extent &e : others)
        if (overlap(out.p, out.bytes, e.p, e.bytes))
            return set_error(CONV2D_EINVAL, "%s: %s overlaps %s", op, out.name, e.name);
    return CONV2D_OK;
}

long long state_bytes(const char *op, const void *state, int rows, long long per_row, int eb) {
    if (!state) return 0;
    if ((uintptr_t)state % eb) return set_error(CONV2D_EINVAL, "%s: state is not aligned to its type", op);
    const __int128 n = (__int128)rows * per_row;
    if (n > (__int128)1 << 45) return set_error(CONV2D_EINVAL, "%s: state reaches too far", op);
    return (long long)n * eb;
}

bool aligned_floats(std::initializer_list<const float *> ps) {
    for (const float *p : ps)
        if ((uintptr_t)p % 4) return false;
    return true;
}

int check_act(const char *op, int act, const float *alpha, int flags) {
    const int code = act & 0xff;
    if (code > CONV2D_ACT_PRELU || (act & ~(0xff | flags)))
        return set_error(CONV2D_EINVAL, "%s: unknown activation flags 0x%x", op, act);
    if (code == CONV2D_ACT_PRELU && !alpha) return set_error(CONV2D_EINVAL, "%s: PRELU needs alpha", op);
    return CONV2D_OK;
}

int too_wide(const char *op) {
    return set_error(CONV2D_EUNSUPPORTED, "%s: more than 2^30 channels, inputs or outputs are not supported", op);
}

// The status of a call whose kernels were launched with `e`.
int launched(const char *op, hipError_t e) {
    if (e == hipErrorInvalidConfiguration)  // from launch_blocks
        return set_error(CONV2D_EUNSUPPORTED, "%s: 2^32 threads or more, too many for one launch", op);
    return e == hipSuccess ? set_ok() : hip_fail(e, op);
}

int run_conv(const causal_conv1d_args *args, bool step, void *stream) {
    const char *op = step ? "causal_conv1d_step" : "causal_conv1d";
    if (!args) return set_error(CONV2D_EINVAL, "%s: args must not be null", op);
    const causal_conv1d_args &a = *args;
    Shape s{op, a.tokens, a.nseq, a.dtype, false, step};
    int rc = check_shape(&s, a.offsets, a.slots, a.state_rows);
    if (rc) return rc;
    if (a.channels <= 0) return set_error(CONV2D_EINVAL, "%s: channels must be positive (got %d)", op, a.channels);
    if (a.channels > kMaxWidth) return too_wide(op);
    if (a.width < 2 || a.width > 4) return set_error(CONV2D_EINVAL, "%s: width must be 2, 3 or 4 (got %d)", op, a.width);
    rc = check_act(op, a.act, a.alpha, 0);
    if (rc) return rc;
    const int eb = dtype_bytes(a.dtype);
    if (!a.w) return set_error(CONV2D_EINVAL, "%s: w must not be null", op);
    if ((uintptr_t)a.w % eb || !aligned_floats({a.bias, a.alpha}))
        return set_error(CONV2D_EINVAL, "%s: w, bias or alpha is not aligned to its type", op);
    if (s.nseq == 0) return set_ok();
    const Rows x{"x", a.x, a.x_batch, a.x_token, a.channels}, y{"y", a.y, a.y_batch, a.y_token, a.channels};
    const long long xb = rows_bytes(s, x), yb = rows_bytes(s, y);
    if (xb < 0 || yb < 0) return (int)(xb < 0 ? xb : yb);
    if (!rows_disjoint(s, y)) return set_error(CONV2D_EINVAL, "%s: rows of y overlap each other", op);
    const long long sb = state_bytes(op, a.state, a.state_rows, (long long)(a.width - 1) * a.channels, eb);
    if (sb < 0) return (int)sb;
    const Extent ex{"x", a.x, xb}, ey{"y", a.y, yb}, es{"state", a.state, sb};
    const Extent ew{"w", a.w, (long long)a.channels * a.width * eb}, eB{"bias", a.bias, 4ll * a.channels};
    const Extent ea{"alpha", a.act == CONV2D_ACT_PRELU ? a.alpha : nullptr, 4ll * a.channels};
    const Extent eo{"offsets", a.offsets, 4ll * (a.nseq + 1ll)}, el{"slots", a.slots, 4ll * a.nseq};
    rc = check_no_overlap(op, ey, {ex, es, ew, eB, ea, eo, el});
    if (!rc) rc = check_no_overlap(op, es, {ex, ew, eB, ea, eo, el});
    if (rc) return rc;
    const int V = 16 / eb;
    const bool vec = a.channels % V == 0 && aligned16(a.x) && aligned16(a.y) && aligned16(a.w) && aligned16(a.state) &&
                     a.x_token % V == 0 && a.y_token % V == 0 &&
                     (s.packed || step || (a.x_batch % V == 0 && a.y_batch % V == 0));
    return launched(op, launch_causal_conv(a, vec, step, static_cast<hipStream_t>(stream)));
}

// Validates a scan's arguments.
int check_scan(const selective_scan_args *args, const char *op, bool step) {
    if (!args) return set_error(CONV2D_EINVAL, "%s: args must not be null", op);
    const selective_scan_args &a = *args;
    Shape s{op, a.tokens, a.nseq, a.dtype, false, step};
    int rc = check_shape(&s, a.offsets, a.slots, a.state_rows);
    if (rc) return rc;
    if (a.channels <= 0 || a.groups <= 0 || a.channels % a.groups)
        return set_error(CONV2D_EINVAL, "%s: channels must be a positive multiple of groups (got %d and %d)", op,
                         a.channels, a.groups);
    if (a.channels > kMaxWidth) return too_wide(op);
    if (a.states < 1 || a.states > 256)
        return set_error(CONV2D_EINVAL, "%s: states must be 1 to 256 (got %d)", op, a.states);
    if (a.longest < 0) return set_error(CONV2D_EINVAL, "%s: longest must not be negative", op);
    if (!a.a) return set_error(CONV2D_EINVAL, "%s: a must not be null", op);
    if (!aligned_floats({a.a, a.skip, a.dt_bias}))
        return set_error(CONV2D_EINVAL, "%s: a, skip or dt_bias is not aligned to its type", op);
    if (s.nseq == 0) return CONV2D_OK;
    const long long gn = (long long)a.groups * a.states;
    const Rows rows[] = {{"u", a.u, a.u_batch, a.u_token, a.channels}, {"dt", a.dt, a.dt_batch, a.dt_token, a.channels},
                         {"b", a.b, a.b_batch, a.b_token, gn},         {"c", a.c, a.c_batch, a.c_token, gn},
                         {"y", a.y, a.y_batch, a.y_token, a.channels}, {"gate", a.gate, a.gate_batch, a.gate_token, a.channels}};
    Extent in[6];
    for (int i = 0; i < 6; i++) {
        const long long n = i == 5 && !a.gate ? 0 : rows_bytes(s, rows[i]);
        if (n < 0) return (int)n;
        in[i] = Extent{rows[i].name, rows[i].p, n};
    }
    const Extent ey = in[4];
    if (!rows_disjoint(s, rows[4])) return set_error(CONV2D_EINVAL, "%s: rows of y overlap each other", op);
    const long long per_row = (long long)a.channels * a.states;
    const long long sb = state_bytes(op, a.state, a.state_rows, per_row, 4);
    if (sb < 0) return (int)sb;
    const Extent es{"state", a.state, sb}, ea{"a", a.a, per_row * 4}, ek{"skip", a.skip, 4ll * a.channels};
    const Extent eb{"dt_bias", a.dt_bias, 4ll * a.channels};
    const Extent eo{"offsets", a.offsets, 4ll * (a.nseq + 1ll)}, el{"slots", a.slots, 4ll * a.nseq};
    rc = check_no_overlap(op, ey, {in[0], in[1], in[2], in[3], in[5], es, ea, ek, eb, eo, el});
    if (!rc) rc = check_no_overlap(op, es, {in[0], in[1], in[2], in[3], in[5], ea, ek, eb, eo, el});
    return rc;
}

int run_scan(const selective_scan_args *args, bool step, void *stream) {
    const char *op = step ? "selective_scan_step" : "selective_scan";
    const int rc = check_scan(args, op, step);
    if (rc) return rc;
    if (args->nseq == 0) return set_ok();
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const Workspace ws = step ? Workspace{} : current_ws();
    return launched(op, step ? launch_scan_token(*args, st) : launch_scan(*args, ws.p, ws.bytes, st));
}

int check_w4(const char *op, int out_features, int in_features, int group) {
    if (out_features <= 0 || in_features <= 0)
        return set_error(CONV2D_EINVAL, "%s: sizes must be positive (out %d, in %d)", op, out_features, in_features);
    if (group != 32 && group != 64 && group != 128)
        return set_error(CONV2D_EINVAL, "%s: group must be 32, 64 or 128 (got %d)", op, group);
    if (out_features > kMaxWidth || in_features > kMaxWidth) return too_wide(op);
    if ((long long)out_features * in_features > 1ll << 40)
        return set_error(CONV2D_EUNSUPPORTED, "%s: more than 2^40 weights are not supported", op);
    return CONV2D_OK;
}

bool type16(int dtype) { return dtype == CONV2D_DTYPE_BF16 || dtype == CONV2D_DTYPE_F16; }

}  // namespace

extern "C" {

int causal_conv1d(const causal_conv1d_args *args, void *stream) { return run_conv(args, false, stream); }
int causal_conv1d_step(const causal_conv1d_args *args, void *stream) { return run_conv(args, true, stream); }
int selective_scan(const selective_scan_args *args, void *stream) { return run_scan(args, false, stream); }

int selective_scan_workspace_size(const selective_scan_args *args, size_t *bytes) {
    const char *op = "selective_scan_workspace_size";
    if (!bytes) return set_error(CONV2D_EINVAL, "%s: bytes must not be null", op);
    const int rc = check_scan(args, op, false);
    if (rc) return rc;
    *bytes = args->nseq ? scan_workspace(*args) : 0;
    return set_ok();
}

int selective_scan_step(const selective_scan_args *args, void *stream) { return run_scan(args, true, stream); }

int matvec_w4_packed_bytes(int out_features, int in_features, int group, int has_zeros, size_t *bytes) {
    const char *op = "matvec_w4_packed_bytes";
    if (!bytes) return set_error(CONV2D_EINVAL, "%s: bytes must not be null", op);
    const int rc = check_w4(op, out_features, in_features, group);
    if (rc) return rc;
    *bytes = w4_packed_bytes(out_features, in_features, group, has_zeros != 0);
    return set_ok();
}

int matvec_w4_pack(const void *codes, const void *scales, const void *zeros, void *packed, int out_features,
                   int in_features, int group, int dtype, void *stream) {
    const char *op = "matvec_w4_pack";
    if (!codes || !scales || !packed) return set_error(CONV2D_EINVAL, "%s: codes, scales and packed must not be null", op);
    const int rc = check_w4(op, out_features, in_features, group);
    if (rc) return rc;
    if (!type16(dtype)) return set_error(CONV2D_EINVAL, "%s: scales are bf16 or f16 (got dtype %d)", op, dtype);
    if (!aligned16(packed) || (uintptr_t)scales % 2)
        return set_error(CONV2D_EINVAL, "%s: packed must be 16-byte and scales 2-byte aligned", op);
    const long long groups = (in_features + group - 1ll) / group, n = out_features;
    const long long bytes = (long long)w4_packed_bytes(out_features, in_features, group, zeros != nullptr);
    if (overlap(packed, bytes, codes, n * ((in_features + 1ll) / 2)) || overlap(packed, bytes, scales, 2 * n * groups) ||
        overlap(packed, bytes, zeros, n * groups))
        return set_error(CONV2D_EINVAL, "%s: packed overlaps an input", op);
    const hipError_t e = launch_w4_pack(codes, scales, zeros, packed, out_features, in_features, group, dtype,
                                        static_cast<hipStream_t>(stream));
    return e == hipSuccess ? set_ok() : hip_fail(e, op);
}

int matvec_w4(const matvec_w4_args *args, void *stream) {
    const char *op = "matvec_w4";
    if (!args) return set_error(CONV2D_EINVAL, "%s: args must not be null", op);
    const matvec_w4_args &a = *args;
    int rc = check_w4(op, a.out_features, a.in_features, a.group);
    if (!rc) rc = check_act(op, a.act, a.alpha, CONV2D_RES_BEFORE_ACT);
    if (rc) return rc;
    if (!type16(a.dtype)) return set_error(CONV2D_EINVAL, "%s: x is bf16 or f16 (got dtype %d)", op, a.dtype);
    Shape s{op, 1, a.rows, a.dtype, false, true};
    rc = check_shape(&s, nullptr, nullptr, 0);
    if (rc) return rc;
    if (!a.packed || !aligned16(a.packed))
        return set_error(CONV2D_EINVAL, "%s: packed must not be null and 16-byte aligned", op);
    if (!aligned_floats({a.bias, a.alpha}))
        return set_error(CONV2D_EINVAL, "%s: bias or alpha is not aligned to its type", op);
    if (a.rows == 0) return set_ok();
    const Rows x{"x", a.x, 0, a.x_row, a.in_features}, y{"y", a.y, 0, a.y_row, a.out_features};
    const Rows r{"residual", a.residual, 0, a.residual_row, a.out_features};
    const long long xb = rows_bytes(s, x), yb = rows_bytes(s, y), rb = a.residual ? rows_bytes(s, r) : 0;
    if (xb < 0 || yb < 0 || rb < 0) return (int)(xb < 0 ? xb : yb < 0 ? yb : rb);
    if (!rows_disjoint(s, y)) return set_error(CONV2D_EINVAL, "%s: rows of y overlap each other", op);
    const long long pb = (long long)w4_packed_bytes(a.out_features, a.in_features, a.group, a.has_zeros != 0);
    rc = check_no_overlap(op, Extent{"y", a.y, yb},
                          {Extent{"x", a.x, xb}, Extent{"residual", a.residual, rb}, Extent{"packed", a.packed, pb},
                           Extent{"bias", a.bias, 4ll * a.out_features},
                           Extent{"alpha", (a.act & 0xff) == CONV2D_ACT_PRELU ? a.alpha : nullptr, 4ll * a.out_features}});
    if (rc) return rc;
    return launched(op, launch_matvec_w4(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
