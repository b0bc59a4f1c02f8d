// Selective state space scan over channel-last token rows, for prompts and single tokens.
#include "kernels.hpp"
#include "seq_common.hpp"

namespace c2d {

namespace {

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

// ---------------------------------------------------------------------------- prompts

// What a launch adds to the arguments: how the work is cut.
struct ScanCut {
    int shift;    // chunks of 1 << shift tokens
    int items;    // chunk numbers in all (find_run), or nseq * chunks
    int chunks;   // unpacked: chunks of a sequence
    int cblocks;  // 64-channel blocks of a group
    float *ws;    // split sequences: a record per item, see Record
};

// Record of a chunk of a split sequence, left by the first pass for the second: the sum of
// its step sizes [channels], then its end state [states][channels], from a zero start state
// (the first chunk: from the sequence's own). The last chunk's end state is of no use to
// another chunk; its place takes the sequence's start state, which the second pass could
// not read from the state row any more, where another workgroup leaves the final one.
__device__ __forceinline__ float *record(const selective_scan_args &a, const ScanCut &k, int item) {
    return k.ws + (long long)item * (a.states + 1) * a.channels;
}

// A workgroup takes 64 channels (one a lane) of one chunk of a sequence. Its NW waves share the
// states of those channels, NS a lane, so that few channels still make many waves, and walk
// the chunk in tiles of TT tokens:
//   1. all threads turn the tile's u and dt into d and d * u, and b and c into fp32, in LDS
//      (the next tile's values are on their way from HBM meanwhile);
//   2. each wave runs its states over the tile: per state and token one exp2 (two issue
//      slots), two products and two multiply-adds, and leaves its part of y in LDS;
//   3. all threads add the NW parts, the skip and the gate, and store y.
// Past the chunk's end d = d * u = 0, which keeps the states as they are.
// Bound by the vector ALU: 6 N issue slots a token and channel and about 36 for the step
// size, gate and conversions, against 4 values moved.
template <typename T, int NS, int NW, bool FIRST>
__global__ __launch_bounds__(64 * NW) void scan_prompt_kernel(const selective_scan_args a, const ScanCut k) {
    constexpr int TT = NW == 16 ? 8 : 16;
    constexpr int NP = NS * NW;                  // states with their padding
    constexpr int EPT = (TT + NW - 1) / NW;      // tile tokens of a thread
    constexpr int BCE = TT * NP * 2 / (64 * NW);  // b and c values of a thread
    __shared__ float2 s_d[TT][64];               // d, d * u
    __shared__ __attribute__((aligned(16))) float s_bc[2][TT][NP];
    __shared__ float s_y[FIRST ? 1 : NW][FIRST ? 1 : TT][64];

    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int blocks = k.cblocks * a.groups;
    const int cb = blockIdx.x % blocks, item = blockIdx.x / blocks;
    const int per = a.channels / a.groups, g = cb / k.cblocks;
    const int in_group = (cb % k.cblocks) * 64 + lane;
    const bool on = in_group < per;
    const int c = on ? g * per + in_group : a.channels - 1;

    SeqRun r;
    long long start = 0;
    if (a.offsets) {
        if (!find_run(a.offsets, a.nseq, (int)a.tokens, k.shift, item, &r)) return;
        start = r.start;
    } else {
        r.seq = item / k.chunks;
        r.first = (item - r.seq * k.chunks) << k.shift;
        r.len = (int)a.tokens;
    }
    const int chunk = r.first >> k.shift;
    const int last = r.len > 0 ? (r.len - 1) >> k.shift : 0;
    if (FIRST && chunk == last) return;
    const long long lead = a.offsets ? 0 : r.seq;
    const T *u = (const T *)a.u + lead * a.u_batch + start * a.u_token + c;
    const T *dt = (const T *)a.dt + lead * a.dt_batch + start * a.dt_token + c;
    const T *bp = (const T *)a.b + lead * a.b_batch + start * a.b_token + (long long)g * a.states;
    const T *cp = (const T *)a.c + lead * a.c_batch + start * a.c_token + (long long)g * a.states;
    const T *gate = a.gate ? (const T *)a.gate + lead * a.gate_batch + start * a.gate_token + c : nullptr;
    T *y = (T *)a.y + lead * a.y_batch + start * a.y_token + c;

    const int row = state_row(a.state, a.slots, r.seq, a.state_rows);
    float *state = row < 0 ? nullptr : a.state + ((long long)row * a.channels + c) * a.states;
    float h[NS], A[NS];
#pragma unroll
    for (int i = 0; i < NS; i++) {
        const int n = wave * NS + i;
        A[i] = n < a.states ? a.a[(long long)c * a.states + n] * kLog2e : 0.0f;
        h[i] = 0.0f;
        if (n < a.states && chunk == 0 && (FIRST || last == 0) && state && !a.fresh) h[i] = state[n];
    }
    if (FIRST && chunk == 0) {
        float *p = record(a, k, item + last) + a.channels + c;
#pragma unroll
        for (int i = 0; i < NS; i++)
            if (on && wave * NS + i < a.states) p[(long long)(wave * NS + i) * a.channels] = h[i];
    }
    if (!FIRST && last > 0) {
        // the start state: chunk 0's end state decayed through the chunks after it
        const float *p = record(a, k, chunk ? item - chunk : item + last) + c;
#pragma unroll
        for (int i = 0; i < NS; i++)
            if (wave * NS + i < a.states) h[i] = p[(long long)(wave * NS + i + 1) * a.channels];
#pragma unroll 4
        for (int j = 1; j < chunk; j++) {
            const float *q = record(a, k, item - chunk + j) + c;
            const float sum = q[0];
#pragma unroll
            for (int i = 0; i < NS; i++)
                if (wave * NS + i < a.states)
                    h[i] = fmaf(__builtin_amdgcn_exp2f(sum * A[i]), h[i], q[(long long)(wave * NS + i + 1) * a.channels]);
        }
    }
    const float bias = a.dt_bias ? a.dt_bias[c] : 0.0f, skip = a.skip ? a.skip[c] : 0.0f;
    const int waves = (a.states + NS - 1) / NS;  // waves with states
    float dsum = 0.0f;

    const int end = r.len < r.first + (1 << k.shift) ? r.len : r.first + (1 << k.shift);
    T nu[EPT], nd[EPT], ng[EPT], nbc[BCE];
    auto fetch = [&](int t0) {
#pragma unroll
        for (int e = 0; e < EPT; e++) {
            const int t = t0 + e * NW + wave;
            if (e * NW + wave < TT && t < end) {
                nu[e] = u[t * a.u_token];
                nd[e] = dt[t * a.dt_token];
                if (!FIRST && gate) ng[e] = gate[t * a.gate_token];
            }
        }
#pragma unroll
        for (int e = 0; e < BCE; e++) {
            const int i = e * 64 * NW + threadIdx.x;
            const int n = i % NP, t = t0 + i / NP % TT;
            nbc[e] = (T)0.0f;
            if (n < a.states && t < end && (!FIRST || i < TT * NP))
                nbc[e] = (i < TT * NP ? bp + t * a.b_token : cp + t * a.c_token)[n];
        }
    };
    fetch(r.first);
    for (int t0 = r.first; t0 < end; t0 += TT) {
        float x[EPT], z[EPT];
#pragma unroll
        for (int e = 0; e < EPT; e++) {
            const int tt = e * NW + wave;
            if (tt < TT) {
                const bool in = t0 + tt < end;
                x[e] = in ? to_f32(nu[e]) : 0.0f;
                z[e] = in && !FIRST && gate ? to_f32(ng[e]) : 0.0f;
                float d = in ? to_f32(nd[e]) + bias : 0.0f;
                if (a.softplus && in) d = softplus(d);
                s_d[tt][lane] = float2{d, d * x[e]};
            }
        }
#pragma unroll
        for (int e = 0; e < BCE; e++) {
            const int i = e * 64 * NW + threadIdx.x;
            (&s_bc[0][0][0])[i] = to_f32(nbc[e]);
        }
        fetch(t0 + TT);
        __syncthreads();
        if (wave < waves) {
#pragma unroll
            for (int t = 0; t < TT; t++) {
                const float2 d = s_d[t][lane];
                if (FIRST) dsum += d.x;
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < NS; i++) {
                    const float add = d.y * s_bc[0][t][wave * NS + i];
                    h[i] = fmaf(__builtin_amdgcn_exp2f(d.x * A[i]), h[i], add);
                    if (!FIRST) sum = fmaf(h[i], s_bc[1][t][wave * NS + i], sum);
                }
                if (!FIRST) s_y[wave][t][lane] = sum;
            }
        }
        __syncthreads();
        if (!FIRST) {
#pragma unroll
            for (int e = 0; e < EPT; e++) {
                const int tt = e * NW + wave;
                if (tt < TT && t0 + tt < end) {
                    float sum = skip * x[e];
                    for (int w = 0; w < waves; w++) sum += s_y[w][tt][lane];
                    if (gate) sum *= activate_c<CONV2D_ACT_SILU>(z[e], 0.0f);
                    if (on) y[(t0 + tt) * a.y_token] = round_fp32<T>(sum);
                }
            }
        }
    }

    if (!on || wave >= waves) return;
    if (FIRST) {
        float *p = record(a, k, item) + c;
        if (wave == 0) p[0] = dsum;
#pragma unroll
        for (int i = 0; i < NS; i++)
            if (wave * NS + i < a.states) p[(long long)(wave * NS + i + 1) * a.channels] = h[i];
    } else if (state && chunk == last) {
#pragma unroll
        for (int i = 0; i < NS; i++)
            if (wave * NS + i < a.states) state[wave * NS + i] = h[i];
    }
}

template <typename T, int NS, int NW> hipError_t launch_prompt(const selective_scan_args &a, const ScanCut &k, hipStream_t st) {
    const dim3 grid((unsigned)((long long)k.items * k.cblocks * a.groups)), block(64 * NW);
    if (k.ws) {
        const hipError_t e = launch_kernel(scan_prompt_kernel<T, NS, NW, true>, grid, block, 0, st, a, k);
        if (e != hipSuccess) return e;
    }
    return launch_kernel(scan_prompt_kernel<T, NS, NW, false>, grid, block, 0, st, a, k);
}

template <typename T> hipError_t launch_prompt_t(const selective_scan_args &a, const ScanCut &k, hipStream_t st) {
    if (a.states <= 4) return launch_prompt<T, 4, 1>(a, k, st);
    if (a.states <= 8) return launch_prompt<T, 4, 2>(a, k, st);
    if (a.states <= 16) return launch_prompt<T, 4, 4>(a, k, st);
    if (a.states <= 32) return launch_prompt<T, 4, 8>(a, k, st);
    if (a.states <= 64) return launch_prompt<T, 4, 16>(a, k, st);
    if (a.states <= 128) return launch_prompt<T, 8, 16>(a, k, st);
    return launch_prompt<T, 16, 16>(a, k, st);
}

// Waves of the kernel that launch_prompt_t picks.
int waves_of(int states) {
    int w = 1;
    while (w < 16 && w * 4 < states) w *= 2;
    return w;
}

// ---------------------------------------------------------------------------- single tokens

constexpr int kBlock = 256;

// Lane i of a channel's `lanes` lanes holds the states i, i + lanes, ...: S of them.
template <typename T, int S>
__global__ __launch_bounds__(kBlock) void scan_token_kernel(const selective_scan_args a, int lanes, int cblocks) {
    const int cl = threadIdx.x % lanes;
    const int ch = (int)(blockIdx.x % cblocks) * (kBlock / lanes) + threadIdx.x / lanes;
    const int c = ch < a.channels ? ch : a.channels - 1;  // idle lanes follow for the sums across lanes
    const long long seq = blockIdx.x / cblocks;
    const int g = c / (a.channels / a.groups);
    const T *b = (const T *)a.b + seq * a.b_token + (long long)g * a.states;
    const T *cc = (const T *)a.c + seq * a.c_token + (long long)g * a.states;
    const int row = state_row(a.state, a.slots, (int)seq, a.state_rows);
    float *state = row < 0 ? nullptr : a.state + ((long long)row * a.channels + c) * a.states;
    const float x = to_f32(((const T *)a.u)[seq * a.u_token + c]);
    float d = to_f32(((const T *)a.dt)[seq * a.dt_token + c]) + (a.dt_bias ? a.dt_bias[c] : 0.0f);
    if (a.softplus) d = softplus(d);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < S; i++) {
        const int n = cl + i * lanes;
        if (n < a.states) {
            const float A = a.a[(long long)c * a.states + n] * kLog2e;
            float h = state && !a.fresh ? state[n] : 0.0f;
            h = fmaf(__builtin_amdgcn_exp2f(d * A), h, d * x * to_f32(b[n]));
            sum = fmaf(h, to_f32(cc[n]), sum);
            if (state && ch < a.channels) state[n] = h;
        }
    }
    for (int o = 1; o < lanes; o *= 2) sum += __shfl_xor(sum, o);
    if (cl != 0 || ch >= a.channels) return;
    if (a.skip) sum = fmaf(a.skip[c], x, sum);
    if (a.gate) sum *= activate_c<CONV2D_ACT_SILU>(to_f32(((const T *)a.gate)[seq * a.gate_token + c]), 0.0f);
    ((T *)a.y)[seq * a.y_token + c] = round_fp32<T>(sum);
}

template <typename T> hipError_t launch_token_t(const selective_scan_args &a, hipStream_t st) {
    int lanes = 1;
    while (lanes < a.states && lanes < 64) lanes *= 2;
    const int cblocks = (a.channels + kBlock / lanes - 1) / (kBlock / lanes);
    const dim3 grid((unsigned)((long long)cblocks * a.nseq));
    if (a.states <= 64) return launch_kernel(scan_token_kernel<T, 1>, grid, dim3(kBlock), 0, st, a, lanes, cblocks);
    return launch_kernel(scan_token_kernel<T, 4>, grid, dim3(kBlock), 0, st, a, lanes, cblocks);
}

// How a prompt call is cut for a workspace of ws_bytes. A sequence left whole is walked by
// one workgroup for each 64 channels, so its length is a time; a split one is read twice (the
// first pass for the chunks' end states), 1.8 times the work, but fills the card.
ScanCut cut_prompt(const selective_scan_args &a, size_t ws_bytes, size_t *want) {
    ScanCut k{};
    const int per = a.channels / a.groups;
    k.cblocks = (per + 63) / 64;
    const long long waves = (long long)k.cblocks * a.groups * waves_of(a.states);
    const long long total = a.offsets ? a.tokens : a.tokens * a.nseq;
    const long long mean = total / a.nseq;
    long long longest = a.offsets ? (a.longest ? a.longest : 2 * mean) : a.tokens;
    if (longest > a.tokens) longest = a.tokens;
    k.shift = 30;
    // tokens a wave walks one after the other, whole and split over 1024 SIMDs
    const long long whole = longest, even = total * waves / 1024;
    if (longest > 256 && whole > even * 18 / 10 + 128) {
        int shift = 6;
        while ((total >> shift) * waves > 4096 || (longest >> shift) >= 64) shift++;
        if ((longest >> shift) >= 1) {
            const long long items = a.offsets ? (a.tokens >> shift) + a.nseq
                                              : ((a.tokens + (1ll << shift) - 1) >> shift) * a.nseq;
            const size_t need = (size_t)items * (a.states + 1) * a.channels * sizeof(float);
            *want = need;
            if (need <= ws_bytes) k.shift = shift;
        }
    }
    k.chunks = a.offsets ? 0 : (int)((a.tokens + (1ll << k.shift) - 1) >> k.shift);
    if (!a.offsets && k.chunks == 0) k.chunks = 1;  // empty sequences still have a state
    k.items = a.offsets ? (int)((a.tokens >> k.shift) + a.nseq) : k.chunks * a.nseq;
    return k;
}

}  // namespace

size_t scan_workspace(const selective_scan_args &a) {
    size_t want = 0;
    cut_prompt(a, 0, &want);
    return want;
}

hipError_t launch_scan(const selective_scan_args &a, void *ws, size_t ws_bytes, hipStream_t st) {
    size_t want = 0;
    ScanCut k = cut_prompt(a, ws ? ws_bytes : 0, &want);
    k.ws = k.shift < 30 ? static_cast<float *>(ws) : nullptr;
    switch (a.dtype) {
    case CONV2D_DTYPE_F32:
        return launch_prompt_t<float>(a, k, st);
    case CONV2D_DTYPE_BF16:
        return launch_prompt_t<bf16>(a, k, st);
    default:
        return launch_prompt_t<f16>(a, k, st);
    }
}

hipError_t launch_scan_token(const selective_scan_args &a, hipStream_t st) {
    switch (a.dtype) {
    case CONV2D_DTYPE_F32:
        return launch_token_t<float>(a, st);
    case CONV2D_DTYPE_BF16:
        return launch_token_t<bf16>(a, st);
    default:
        return launch_token_t<f16>(a, st);
    }
}

}  // namespace c2d
