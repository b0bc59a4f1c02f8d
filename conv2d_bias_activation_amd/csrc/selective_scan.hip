// Selective state space scan over channel-last token rows, for prompts and single tokens.
#include "kernels.hpp"
#include "seq_common.hpp"

namespace c2d {

namespace {

constexpr int kBlock = 256;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

// log(1 + exp(x)) = max(x, 0) + log(1 + t), t = exp(-|x|). The step sizes of a scan are often
// 1e-3 and less, where log(1 + t) takes its relative precision from the bits of t that the
// sum w = 1 + t rounds away: they are t - (w - 1), exactly, and log(1 + t) is log(w) plus
// those over w, which is 1 to within what they matter. (Measured over t from 2^-22 to 1: the
// hardware's log2 is within 1.2e-7 of the exact value, relatively, down to w = 1 + 2^-22.)
__device__ __forceinline__ float softplus(float x) {
    const float t = __builtin_amdgcn_exp2f(-fabsf(x) * kLog2e);
    const float w = 1.0f + t;
    const float lost = t - (w - 1.0f);
    return fmaxf(x, 0.0f) + fmaf(__builtin_amdgcn_logf(w), kLn2, lost);
}

// Lane i of a channel's `lanes` lanes holds the states i, i + lanes, ...: S of them.
template <typename T, int S>
__global__ __launch_bounds__(kBlock) void scan_kernel(const selective_scan_args a, int lanes, int cblocks) {
    const int cl = threadIdx.x % lanes;
    const int ch = (int)(blockIdx.x % cblocks) * (kBlock / lanes) + threadIdx.x / lanes;
    const int c = ch < a.channels ? ch : a.channels - 1;  // idle lanes follow for the sums across lanes
    const int seq = blockIdx.x / cblocks;
    long long row0[6] = {seq * a.u_batch, seq * a.dt_batch, seq * a.b_batch,
                         seq * a.c_batch, seq * a.gate_batch, seq * a.y_batch};
    int len = (int)a.tokens;
    if (a.offsets) {
        const int start = clamped_offset(a.offsets, seq, (int)a.tokens);
        const int end = clamped_offset(a.offsets, seq + 1, (int)a.tokens);
        len = end > start ? end - start : 0;
        const long long t[6] = {a.u_token, a.dt_token, a.b_token, a.c_token, a.gate_token, a.y_token};
        for (int i = 0; i < 6; i++) row0[i] = start * t[i];
    }
    const int g = c / (a.channels / a.groups);
    const T *u = (const T *)a.u + row0[0] + c, *dt = (const T *)a.dt + row0[1] + c;
    const T *b = (const T *)a.b + row0[2] + (long long)g * a.states, *cc = (const T *)a.c + row0[3] + (long long)g * a.states;
    const T *gate = a.gate ? (const T *)a.gate + row0[4] + c : nullptr;
    T *y = (T *)a.y + row0[5] + c;
    const int row = state_row(a.state, a.slots, seq, a.state_rows);
    float *state = row < 0 ? nullptr : a.state + ((long long)row * a.channels + c) * a.states;
    float h[S], A[S];
    for (int i = 0; i < S; i++) {
        const int n = cl + i * lanes;
        A[i] = n < a.states ? a.a[(long long)c * a.states + n] * kLog2e : 0.0f;
        h[i] = n < a.states && state && !a.fresh ? state[n] : 0.0f;
    }
    const float bias = a.dt_bias ? a.dt_bias[c] : 0.0f, skip = a.skip ? a.skip[c] : 0.0f;
    for (int t = 0; t < len; t++) {
        const float x = to_f32(u[t * a.u_token]);
        float d = to_f32(dt[t * a.dt_token]) + bias;
        if (a.softplus) d = softplus(d);
        float sum = 0.0f;
        for (int i = 0; i < S; i++) {
            const int n = cl + i * lanes;
            if (n >= a.states) break;
            h[i] = fmaf(__builtin_amdgcn_exp2f(d * A[i]), h[i], d * x * to_f32(b[t * a.b_token + n]));
            sum = fmaf(h[i], to_f32(cc[t * a.c_token + n]), sum);
        }
        for (int o = 1; o < lanes; o *= 2) sum += __shfl_xor(sum, o);
        sum = fmaf(skip, x, sum);
        if (gate) sum *= activate_c<CONV2D_ACT_SILU>(to_f32(gate[t * a.gate_token]), 0.0f);
        if (cl == 0 && ch < a.channels) y[t * a.y_token] = round_fp32<T>(sum);
    }
    if (state && ch < a.channels)
        for (int i = 0; i < S; i++)
            if (cl + i * lanes < a.states) state[cl + i * lanes] = h[i];
}

template <typename T> hipError_t launch_t(const selective_scan_args &a, hipStream_t st) {
    int lanes = 1;
    while (lanes < a.states && lanes < 64) lanes *= 2;
    const int cblocks = (a.channels + kBlock / lanes - 1) / (kBlock / lanes);
    const dim3 grid((unsigned)((long long)cblocks * a.nseq));
    if (a.states <= 64) return launch_kernel(scan_kernel<T, 1>, grid, dim3(kBlock), 0, st, a, lanes, cblocks);
    return launch_kernel(scan_kernel<T, 4>, grid, dim3(kBlock), 0, st, a, lanes, cblocks);
}

}  // namespace

hipError_t launch_scan(const selective_scan_args &a, bool step, hipStream_t st) {
    selective_scan_args s = a;
    if (step) {  // rows are sequences of one token
        s.u_batch = a.u_token, s.dt_batch = a.dt_token, s.b_batch = a.b_token, s.c_batch = a.c_token;
        s.gate_batch = a.gate_token, s.y_batch = a.y_token;
        s.tokens = 1;
    }
    switch (a.dtype) {
    case CONV2D_DTYPE_F32:
        return launch_t<float>(s, st);
    case CONV2D_DTYPE_BF16:
        return launch_t<bf16>(s, st);
    default:
        return launch_t<f16>(s, st);
    }
}

}  // namespace c2d
