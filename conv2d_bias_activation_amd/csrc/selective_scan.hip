// Selective state space scan over channel-last token rows, for prompts and single tokens.
#include <algorithm>

#include "kernels.hpp"
#include "runtime.hpp"
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

// A log2(e), for exp(d A) = exp2(d (A log2(e))). A finite A stays finite, so that a step of zero
// keeps the state: one past 2.36e38 counts as that.
__device__ __forceinline__ float rate_base2(float A) {
    const float r = A * kLog2e;
    return __builtin_isinf(r) && !__builtin_isinf(A) ? __builtin_copysignf(__FLT_MAX__, A) : r;
}

// ---------------------------------------------------------------------------- prompts

// What a launch adds to the arguments: how the work is cut.
struct ScanCut {
    int run;      // tokens of a chunk
    int items;    // chunk numbers in all (find_run), or nseq * chunks
    int chunks;   // unpacked: chunks of a sequence
    int cblocks;  // 64-channel blocks of a group
    bool vec;     // states a multiple of four, a and the state 16-byte aligned
    bool ranked;  // whole packed sequences: the longest first
    float *ws;    // split sequences: a record per item, see Record
};

// Record of a chunk of a split sequence, left by the first pass for the second: half the sum of
// its step sizes [channels], then its end state [states][channels], from a zero start state
// (the first chunk: from the sequence's own). The last chunk's end state is of no use to
// another chunk; its place takes the sequence's start state, which the second pass could
// not read from the state row any more, where another workgroup leaves the final one.
__device__ __forceinline__ float *record(const selective_scan_args &a, const ScanCut &k, int item) {
    return k.ws + (long long)item * (a.states + 1) * a.channels;
}

constexpr int kMaxRanked = 256;

// The sequence that stands at place `rank` when the longest come first (ties by number), so
// that the workgroups that start last are short (cut_prompt says when).
// key: room for a sequence's length and number each.
__device__ __forceinline__ int by_length(const int *offsets, int nseq, int tokens, int rank, uint64_t *key, int &found) {
    for (int i = threadIdx.x; i < nseq; i += blockDim.x) {
        const int len = clamped_offset(offsets, i + 1, tokens) - clamped_offset(offsets, i, tokens);
        key[i] = (uint64_t)max(len, 0) << 32 | (uint32_t)(nseq - i);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nseq; i += blockDim.x) {
        const uint64_t mine = key[i];
        int before = 0;
        for (int j = 0; j < nseq; j++) before += key[j] > mine;
        if (before == rank) found = i;
    }
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(found);
}

// NS states from n on of a row of `states`, zeros behind its end.
template <int NS> __device__ __forceinline__ void load_states(const float *row, int n, int states, bool vec, float *v) {
    if (vec) {
#pragma unroll
        for (int i = 0; i < NS; i += 4) {
            const Pack<float, 4> p = n + i < states ? load_pack<float, 4>(row + n + i) : Pack<float, 4>{};
#pragma unroll
            for (int j = 0; j < 4; j++) v[i + j] = p.v[j];
        }
    } else {
#pragma unroll
        for (int i = 0; i < NS; i++) v[i] = n + i < states ? row[n + i] : 0.0f;
    }
}

// A workgroup takes 64 channels (one a lane) of one chunk of a sequence. Its NW waves share the
// states of those channels, NS a lane, so that few channels still make many waves, and walk
// the chunk in tiles of TT tokens:
//   1. all threads turn the tile's u and dt into d and d * u, and b and c into fp32, in LDS
//      (the next tile's values are on their way from HBM meanwhile);
//   2. each wave runs its states over the tile: per state and token one exp2 (two issue
//      slots), two products and two multiply-adds, and leaves its part of y in LDS;
//   3. all threads add the NW parts, the skip and the gate, and store y.
// The last tile stops at the chunk's end: a token of no step would not do there, as 0 * A is NaN
// for an infinite A.
// Bound by the vector ALU: 6 N issue slots of four cycles a token and channel, and about 38 for
// the step size, gate, conversions and sums (some 26 of them the formula's own), against 4
// values moved. Measured, bf16, 16 states, cards 4 % apart: 16384 ragged tokens x 4096 channels 256
// to 267 us, the ALUs 93 % busy; one sequence of 32768 x 1024, in two passes, 236 us (86 %). Four
// states a lane on four waves are faster than eight on two (267 and 381 us, 237 and 303): more
// waves hide the latencies.
// The bounds on a SIMD's waves: for 9 to 32 states five, as registers for six spill to memory
// (267 and 276 us); for up to 8 four, as five spill (24 sequences of 16384 tokens x 4096 in all, 4
// states: 376 and 559 us; 8 states 300 and 298). From 33 states on one workgroup of 16 waves fills
// a CU, by its LDS up to 64 states and by its registers past that.
template <typename T, int NS, int NW, bool FIRST>
__global__ __launch_bounds__(64 * NW, NW <= 2 ? 4 : NW <= 8 ? 5 : NS == 4 ? 8 : 4) void scan_prompt_kernel(
    const selective_scan_args a, const ScanCut k) {
    // tokens of a tile; eight where sixteen would leave fewer waves resident for want of LDS
    constexpr int TT = NS * NW > 64 || NW <= 2 ? 8 : 16;
    constexpr int NP = NS * NW;                   // states with their padding
    constexpr int EPT = (TT + NW - 1) / NW;       // tile tokens of a thread
    constexpr bool kEven = TT % NW == 0;          // all waves have as many
    constexpr int BCE = TT * NP * 2 / (64 * NW);  // b and c values of a thread, b's first
    __shared__ int s_seq;
    __shared__ float2 s_d[TT][64];               // d, d * u
    __shared__ __attribute__((aligned(16))) float s_bc[2][TT][NP];
    __shared__ __attribute__((aligned(16))) float s_y[FIRST ? 1 : NW][FIRST ? 1 : TT][64];
    static_assert(FIRST || sizeof(s_y) >= kMaxRanked * sizeof(uint64_t));

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
        if (!FIRST && k.ranked) {
            const int s = by_length(a.offsets, a.nseq, (int)a.tokens, item, reinterpret_cast<uint64_t *>(s_y), s_seq);
            r.seq = s;
            r.start = clamped_offset(a.offsets, s, (int)a.tokens);
            const int e = clamped_offset(a.offsets, s + 1, (int)a.tokens);
            r.len = e > r.start ? e - r.start : 0;
            r.first = 0;
        } else if (!find_run(a.offsets, a.nseq, (int)a.tokens, k.run, item, &r)) {
            return;
        }
        start = r.start;
    } else {
        r.seq = item / k.chunks;
        r.first = (item - r.seq * k.chunks) * k.run;
        r.len = (int)a.tokens;
    }
    const int chunk = r.first / k.run;
    const int last = r.len > 0 ? (r.len - 1) / k.run : 0;
    if (FIRST && chunk == last) return;
    const long long lead = a.offsets ? 0 : r.seq;
    const T *u = (const T *)a.u + lead * a.u_batch + start * a.u_token;
    const T *dt = (const T *)a.dt + lead * a.dt_batch + start * a.dt_token;
    const T *bp = (const T *)a.b + lead * a.b_batch + start * a.b_token + (long long)g * a.states;
    const T *cp = (const T *)a.c + lead * a.c_batch + start * a.c_token + (long long)g * a.states;
    const bool gated = !FIRST && a.gate;
    // without a gate its loads, never used, go to u
    const T *gate = gated ? (const T *)a.gate + lead * a.gate_batch + start * a.gate_token : u;
    const long long gate_token = gated ? a.gate_token : a.u_token;
    T *y = (T *)a.y + lead * a.y_batch + start * a.y_token;

    const int row = state_row(a.state, a.slots, r.seq, a.state_rows);
    float *state = row < 0 ? nullptr : a.state + ((long long)row * a.channels + c) * a.states;
    float h[NS], A[NS];
    const bool starts = chunk == 0 && (FIRST || last == 0) && state && !a.fresh;
    load_states<NS>(a.a + (long long)c * a.states, wave * NS, a.states, k.vec, A);
    if (starts) load_states<NS>(state, wave * NS, a.states, k.vec, h);
#pragma unroll
    for (int i = 0; i < NS; i++) {
        A[i] = rate_base2(A[i]);
        if (!starts) h[i] = 0.0f;
    }
    if (FIRST && chunk == 0) {
        float *p = record(a, k, item + last) + a.channels + c;
#pragma unroll
        for (int i = 0; i < NS; i++)
            if (on && wave * NS + i < a.states) p[(long long)(wave * NS + i) * a.channels] = h[i];
    }
    const float bias = a.dt_bias ? a.dt_bias[c] : 0.0f, skip = a.skip ? a.skip[c] : 0.0f;
    const int waves = (a.states + NS - 1) / NS;  // waves with states; the others' part of y is 0
    if (!FIRST && wave >= waves) {
#pragma unroll
        for (int t = 0; t < TT; t++) s_y[wave][t][lane] = 0.0f;
    }
    float dsum = 0.0f;

    const int end = min(r.len, r.first + k.run);
    T nu[EPT], nd[EPT], ng[EPT], nbc[BCE];  // the next tile
    // Offsets of its first row of this wave, and of the lane's rows of b and c: they move on by
    // a tile with each fetch. Rows past the end are the last one again.
    const int first = r.first + wave, past = end - 1;
    long long ou = first * a.u_token, od = first * a.dt_token, og = first * gate_token, ob[BCE];
#pragma unroll
    for (int e = 0; e < BCE; e++) {
        const int i = e * 64 * NW + threadIdx.x;
        ob[e] = (r.first + i / NP % TT) * (i < TT * NP ? a.b_token : a.c_token);
    }
    auto fetch = [&](int t0) {
#pragma unroll
        for (int e = 0; e < EPT; e++) {
            const bool in = t0 + e * NW + wave < end;
            nu[e] = (u + (in ? ou + e * NW * a.u_token : past * a.u_token))[(unsigned)c];
            nd[e] = (dt + (in ? od + e * NW * a.dt_token : past * a.dt_token))[(unsigned)c];
            if (!FIRST) ng[e] = (gate + (in ? og + e * NW * gate_token : past * gate_token))[(unsigned)c];
        }
        ou += TT * a.u_token, od += TT * a.dt_token, og += TT * gate_token;
#pragma unroll
        for (int e = 0; e < BCE; e++) {
            const int i = e * 64 * NW + threadIdx.x;
            const int n = min(i % NP, a.states - 1);
            const bool in = t0 + i / NP % TT < end;
            const long long token = i < TT * NP ? a.b_token : a.c_token;
            if (!FIRST || i < TT * NP) nbc[e] = ((i < TT * NP ? bp : cp) + (in ? ob[e] : past * token))[(unsigned)n];
            ob[e] += TT * token;
        }
    };
    if (end > r.first) fetch(r.first);  // on its way with the records
    if (!FIRST && last > 0) {
        // the start state: chunk 0's end state decayed through the chunks after it, kAhead
        // records on their way at once
        constexpr int kAhead = NS == 16 ? 2 : NS == 8 || NW == 8 ? 4 : 8;
        const long long stride = (long long)(a.states + 1) * a.channels;
        unsigned at[NS];  // states past the end take the last one's and are cleared behind
#pragma unroll
        for (int i = 0; i < NS; i++) at[i] = (unsigned)(min(wave * NS + i, a.states - 1) + 1) * a.channels + c;
        const float *p = record(a, k, chunk ? item - chunk : item + last);
#pragma unroll
        for (int i = 0; i < NS; i++) h[i] = p[at[i]];
        for (int j = 1; j < chunk; j += kAhead) {
            float sum[kAhead], add[kAhead][NS];
#pragma unroll
            for (int m = 0; m < kAhead; m++) {
                const float *q = p + min(j + m, chunk - 1) * stride;
                sum[m] = q[(unsigned)c];
#pragma unroll
                for (int i = 0; i < NS; i++) add[m][i] = q[at[i]];
            }
#pragma unroll
            for (int m = 0; m < kAhead; m++)
                if (j + m < chunk) {
#pragma unroll
                    for (int i = 0; i < NS; i++) {
                        // A chunk's decay in two equal factors: rates or steps of the other sign may
                        // make it pass fp32's range while the state, zero or tiny, does not.
                        const float e = __builtin_amdgcn_exp2f(fminf(sum[m] * A[i], 127.0f));
                        h[i] = fmaf(e, e * h[i], add[m][i]);
                    }
                }
        }
#pragma unroll
        for (int i = 0; i < NS; i++)
            if (wave * NS + i >= a.states) h[i] = 0.0f;
    }
    auto tile = [&](int t0, auto full) {
        constexpr bool kFull = decltype(full)::value;
        float x[EPT], z[EPT], d[EPT];
#pragma unroll
        for (int e = 0; e < EPT; e++) {
            x[e] = to_f32(nu[e]);
            d[e] = to_f32(nd[e]) + bias;
            z[e] = to_f32(ng[e]);
        }
        if (a.softplus) {
#pragma unroll
            for (int e = 0; e < EPT; e++) d[e] = softplus(d[e]);
        }
#pragma unroll
        for (int e = 0; e < EPT; e++) {
            const int tt = e * NW + wave;
            if (kEven || tt < TT) s_d[tt][lane] = float2{d[e], d[e] * x[e]};
            if (FIRST && (kEven || tt < TT) && (kFull || t0 + tt < end)) dsum += d[e];
        }
#pragma unroll
        for (int e = 0; e < BCE; e++) {
            const int i = e * 64 * NW + threadIdx.x;
            if (!FIRST || i < TT * NP) (&s_bc[0][0][0])[i] = i % NP < a.states ? to_f32(nbc[e]) : 0.0f;
        }
        fetch(t0 + TT);
        __syncthreads();
        if (wave < waves) {
#pragma unroll
            for (int t = 0; t < TT; t++) {
                if (!kFull && t0 + t >= end) break;
                const float2 v = s_d[t][lane];
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < NS; i++) {
                    const float add = v.y * s_bc[0][t][wave * NS + i];
                    h[i] = fmaf(__builtin_amdgcn_exp2f(v.x * A[i]), h[i], add);
                    if (!FIRST) sum = fmaf(h[i], s_bc[1][t][wave * NS + i], sum);
                }
                if (!FIRST) s_y[wave][t][lane] = sum;
            }
        }
        __syncthreads();
        if (FIRST) return;
        float v[EPT];
#pragma unroll
        for (int e = 0; e < EPT; e++) {
            v[e] = skip * x[e];
#pragma unroll
            for (int w = 0; w < NW; w++)
                if (kEven || e * NW + wave < TT) v[e] += s_y[w][e * NW + wave][lane];
        }
        if (gated) {
#pragma unroll
            for (int e = 0; e < EPT; e++) v[e] *= activate_c<CONV2D_ACT_SILU>(z[e], 0.0f);
        }
#pragma unroll
        for (int e = 0; e < EPT; e++) {
            const int tt = e * NW + wave;
            if (on && (kEven || tt < TT) && (kFull || t0 + tt < end))
                (y + (t0 + tt) * a.y_token)[(unsigned)c] = round_fp32<T>(v[e]);
        }
    };
    int t0 = r.first;
    for (; t0 + TT <= end; t0 += TT) tile(t0, std::true_type{});
    if (t0 < end) tile(t0, std::false_type{});

    if (FIRST) {  // the chunk's step sizes: a part in each wave
        float *part = &s_d[0][0].x;  // free after the last tile
        __syncthreads();
        part[threadIdx.x] = dsum;
        __syncthreads();
        dsum = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; w++) dsum += part[w * 64 + lane];
    }
    if (!on || wave >= waves) return;
    if (FIRST) {
        float *p = record(a, k, item) + c;
        if (wave == 0) p[0] = 0.5f * dsum;
#pragma unroll
        for (int i = 0; i < NS; i++)
            if (wave * NS + i < a.states) p[(long long)(wave * NS + i + 1) * a.channels] = h[i];
    } else if (state && chunk == last) {
        if (k.vec) {
#pragma unroll
            for (int i = 0; i < NS; i += 4)
                if (wave * NS + i < a.states)
                    store_pack<float, 4>(state + wave * NS + i, Pack<float, 4>{{h[i], h[i + 1], h[i + 2], h[i + 3]}});
        } else {
#pragma unroll
            for (int i = 0; i < NS; i++)
                if (wave * NS + i < a.states) state[wave * NS + i] = h[i];
        }
    }
}

template <typename T, int NS, int NW> hipError_t launch_prompt(const selective_scan_args &a, const ScanCut &k, hipStream_t st) {
    const long long blocks = (long long)k.items * k.cblocks * a.groups;
    if (k.ws) {
        const hipError_t e = launch_blocks(scan_prompt_kernel<T, NS, NW, true>, blocks, 64 * NW, st, a, k);
        if (e != hipSuccess) return e;
    }
    return launch_blocks(scan_prompt_kernel<T, NS, NW, false>, blocks, 64 * NW, st, a, k);
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

// One token of each sequence. A channel's states lie on `lanes` lanes (a power of two), VEC
// neighbouring ones a lane, so that a wave reads and writes its state as whole cache lines;
// with VEC = 1 (unaligned rows, or states not a multiple of four) a lane takes up to S,
// `lanes` apart. A workgroup takes the same channels of ROWS sequences: a is read once for
// them and their states are on their way together. Bound by the state's bytes (8 a state and
// token), or by the launch for few rows.
template <typename T, int VEC, int S, int ROWS>
__global__ __launch_bounds__(kBlock) void scan_token_kernel(const selective_scan_args a, int lanes, int cblocks) {
    const int cl = threadIdx.x % lanes;
    const int ch = (int)(blockIdx.x % cblocks) * (kBlock / lanes) + threadIdx.x / lanes;
    const bool on = ch < a.channels;
    const int c = on ? ch : a.channels - 1;  // idle lanes follow for the sums across lanes
    const int g = c / (a.channels / a.groups);
    const int first = (int)(blockIdx.x / cblocks) * ROWS;

    float A[S][VEC];
    int at[S];
    bool has[S];
#pragma unroll
    for (int i = 0; i < S; i++) {
        const int n = (cl + i * lanes) * VEC;
        has[i] = n < a.states;
        at[i] = has[i] ? n : 0;
        const Pack<float, VEC> v = load_pack<float, VEC>(a.a + (long long)c * a.states + at[i]);
#pragma unroll
        for (int j = 0; j < VEC; j++) A[i][j] = rate_base2(v.v[j]);
    }
    const float bias = a.dt_bias ? a.dt_bias[c] : 0.0f, skip = a.skip ? a.skip[c] : 0.0f;

    float *state[ROWS];
    Pack<float, VEC> h[ROWS][S];
    Pack<T, VEC> b[ROWS][S], cc[ROWS][S];
    T u[ROWS], dt[ROWS], gate[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; r++) {
        const long long seq = min(first + r, a.nseq - 1);
        const int row = state_row(a.state, a.slots, (int)seq, a.state_rows);
        state[r] = row < 0 ? nullptr : a.state + ((long long)row * a.channels + c) * a.states;
        u[r] = ((const T *)a.u)[seq * a.u_token + c];
        dt[r] = ((const T *)a.dt)[seq * a.dt_token + c];
        if (a.gate) gate[r] = ((const T *)a.gate)[seq * a.gate_token + c];
#pragma unroll
        for (int i = 0; i < S; i++) {
            b[r][i] = load_pack<T, VEC>((const T *)a.b + seq * a.b_token + (long long)g * a.states + at[i]);
            cc[r][i] = load_pack<T, VEC>((const T *)a.c + seq * a.c_token + (long long)g * a.states + at[i]);
            h[r][i] = Pack<float, VEC>{};
            if (state[r] && !a.fresh) h[r][i] = load_pack<float, VEC>(state[r] + at[i]);
        }
    }
#pragma unroll
    for (int r = 0; r < ROWS; r++) {
        if (first + r >= a.nseq) break;
        const float x = to_f32(u[r]);
        float d = to_f32(dt[r]) + bias;
        if (a.softplus) d = softplus(d);
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < S; i++) {
            if (!has[i]) continue;
#pragma unroll
            for (int j = 0; j < VEC; j++) {
                h[r][i].v[j] = fmaf(__builtin_amdgcn_exp2f(d * A[i][j]), h[r][i].v[j], d * x * to_f32(b[r][i].v[j]));
                sum = fmaf(h[r][i].v[j], to_f32(cc[r][i].v[j]), sum);
            }
            if (state[r] && on) store_pack<float, VEC>(state[r] + at[i], h[r][i]);
        }
        for (int o = 1; o < lanes; o *= 2) sum += __shfl_xor(sum, o);
        sum = fmaf(skip, x, sum);
        if (a.gate) sum *= activate_c<CONV2D_ACT_SILU>(to_f32(gate[r]), 0.0f);
        if (cl == 0 && on) ((T *)a.y)[(long long)(first + r) * a.y_token + c] = round_fp32<T>(sum);
    }
}

template <typename T, int VEC, int S> hipError_t launch_token(const selective_scan_args &a, hipStream_t st) {
    int lanes = 1;
    while (lanes * VEC < a.states && lanes < 64) lanes *= 2;
    const int cblocks = (a.channels + kBlock / lanes - 1) / (kBlock / lanes);
    const long long blocks = (long long)cblocks * a.nseq;
    // two sequences a workgroup where that leaves the card full (512 sequences x 4096 channels x
    // 16 states: 59.4 us, 4.8 TB/s; one: 63.1, four: 59.9, eight: 71.0), else one
    if (S == 1 && blocks >= 4096)
        return launch_blocks(scan_token_kernel<T, VEC, S, 2>, cblocks * ((a.nseq + 1ll) / 2), kBlock, st, a, lanes, cblocks);
    return launch_blocks(scan_token_kernel<T, VEC, S, 1>, blocks, kBlock, st, a, lanes, cblocks);
}

template <typename T> hipError_t launch_token_t(const selective_scan_args &a, hipStream_t st) {
    const bool vec = a.states % 4 == 0 && a.b_token % 4 == 0 && a.c_token % 4 == 0 && aligned16(a.a) && aligned16(a.state) &&
                     (uintptr_t)a.b % (4 * sizeof(T)) == 0 && (uintptr_t)a.c % (4 * sizeof(T)) == 0;
    if (vec) return launch_token<T, 4, 1>(a, st);
    if (a.states <= 64) return launch_token<T, 1, 1>(a, st);
    return launch_token<T, 1, 4>(a, st);
}

constexpr int kWhole = 0x7fffffff;  // run of a call that is not split: more than any sequence has
constexpr int kMaxChunks = 96;

// How a prompt call is cut for a workspace of ws_bytes. A sequence left whole is walked by
// one workgroup for each 64 channels, so its length is a time; a split one is read twice (the
// first pass for the chunks' end states), 1.8 times the work, but fills the card. Whole and
// split, us: 50 tokens x 512 channels x 16 states 11.0 and 12.5, 64: 12.1 and 12.8, 72: 13.5 and 12.6,
// 100: 16.9 and 12.8; of 4 states 50: 14.9 and 14.3, 64: 17.1 and 14.6.
// More chunks fill the card, but each reads the records before it: 32768 tokens x 1024 in 64
// chunks 247 us, in 94 237.
ScanCut cut_prompt(const selective_scan_args &a, size_t ws_bytes, size_t *want) {
    ScanCut k{};
    const int per = a.channels / a.groups;
    k.cblocks = (per + 63) / 64;
    const long long waves = (long long)k.cblocks * a.groups * waves_of(a.states);
    const long long total = a.offsets ? a.tokens : a.tokens * a.nseq;
    const long long mean = total / a.nseq;
    long long longest = a.offsets ? (a.longest ? a.longest : 2 * mean) : a.tokens;
    if (longest > a.tokens) longest = a.tokens;
    k.run = kWhole;
    k.vec = a.states % 4 == 0 && aligned16(a.a) && aligned16(a.state);
    // tokens a wave walks one after the other, whole and split over 1024 SIMDs
    const long long even = total * waves / 1024;
    if (longest > 48 && longest > even * 18 / 10 + 24) {
        // Chunks for five waves a SIMD, which is what the kernel of 9 to 32 states keeps (the others
        // four: a quarter of their workgroups start late), in whole tiles; as a chunk reads
        // the records of those before it, two tiles at least where there would be over 32
        // chunks (1000 tokens x 512 channels: 22.7 us in chunks of 16, 19.2 of 32; 400 tokens:
        // 15.5 and 16.8)
        const long long least = longest > 512 ? 16 : 0;
        const long long run = std::max({total * waves / (5 * 1024), longest / kMaxChunks, least}) / 16 * 16 + 16;
        if (run < longest) {
            const long long items = a.offsets ? a.tokens / run + a.nseq : (a.tokens + run - 1) / run * a.nseq;
            *want = (size_t)items * (a.states + 1) * a.channels * sizeof(float);
            if ((a.states + 1ll) * a.channels > 1ll << 31) *want = 0;  // 32-bit offsets within a record
            if (*want && *want <= ws_bytes) k.run = (int)run;
        }
    }
    // The order of lengths costs each workgroup a look at all of them, which long sequences earn
    // back. Ordered and not, us, 16 states: 24 sequences of a mean of 683 tokens x 4096 channels 256
    // and 297; 64 of 128 x 2048 71.4 and 92.0; 128 of 32 x 512 17.9 and 21.2, of 16 15.8 and 14.3; 256 of
    // 128 x 2048 285 and 276, of 16 x 2048 88 and 68; 64 states, 256 of 128 x 512 288 and 339, of 16 112
    // and 101.
    k.ranked = a.offsets && k.run == kWhole && a.nseq <= kMaxRanked && 4 * a.tokens >= (long long)a.nseq * a.nseq;
    k.chunks = a.offsets ? 0 : (int)std::max((a.tokens + k.run - 1) / k.run, 1ll);  // empty sequences have a state
    k.items = a.offsets ? (int)(a.tokens / k.run + a.nseq) : k.chunks * a.nseq;
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
    k.ws = k.run < kWhole ? static_cast<float *>(ws) : nullptr;
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
