// Gated linear recurrence over channel-last token rows, for prompts and single tokens, and its
// gradient (gfx950 only).
//
//     h_t = f_t h_{t-1} + b_t,   f = sigmoid(forget + bias),   b = (1 - f) x or x,   y = h silu(gate)
//
// A run of tokens maps the state before it to the state behind it as h -> A h + B, A the product
// of its f and B what it ends in from zero; runs compose, so the waves of a workgroup take
// neighbouring tokens of a tile, exchange their (A, B) in LDS and then know where each starts.
// The gradient carried towards the first token, c_t = f_t g_t with g_t = e_t + c_{t+1} and e the
// part of h_t's gradient that comes from y_t, is the same scan backwards: c -> A c + D.
#include <algorithm>
#include <type_traits>

#include "kernels.hpp"
#include "runtime.hpp"
#include "seq_common.hpp"

namespace c2d {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;

// keep = sigmoid(z) and take = 1 - sigmoid(z) for z = forget + bias, which is added before anything else, as the two may
// cancel. With u = 2^-24, exp2's argument is off by up to 1.5 u |z| and its value by two roundings, so keep is off by
// u ((2.5 |z| + 2) take + 3) of itself, the sum's rounding counted, and take by u ((2.5 |z| + 2) keep + 4). The
// reciprocal gives no numbers below the smallest normal one: keep is 0 for z under some -87.3, and take, whose product would be 0
// or not a number, is 1 there. A z that is not a number makes both one.
__device__ __forceinline__ void gates(float z, float &keep, float &take) {
    const float t = __builtin_amdgcn_exp2f(-kLog2e * z);
    keep = __builtin_amdgcn_rcpf(1.0f + t);
    take = keep == 0.0f ? 1.0f : t * keep;
}

constexpr int kTW = 8;          // neighbouring tokens of a wave
constexpr int kNW = 8;          // waves of a workgroup
constexpr int kTile = kTW * kNW;
constexpr int kWhole = 1 << 30;  // run of a call that is not split; whole tiles

// How a prompt call is cut.
struct RecCut {
    int run;      // tokens of a chunk, whole tiles
    int items;    // chunk numbers in all (find_run), or nseq * chunks
    int chunks;   // unpacked: chunks of a sequence
    int cblocks;  // blocks of 64 VEC channels
    int ranked;   // whole packed sequences: how many stand side by side on the card, else 0
    int near;     // blocks of channels of the same tokens stand on one XCD
    float *rec;   // split sequences: records of the chunks, [item][fields][channels]
    float *tile;  // gradient: [tile number][2][channels]
    float *bias;  // gradient: sums of grad_forget, [item][channels]
};

// Records of a split sequence's chunks, left by the first pass for the second.
//   kA: product of f; 0 in the chunks from which the scan starts (see kB and kD)
//   kB: end state, from zero; chunk 0: from the sequence's own start state. The last chunk's
//       end state is of no use to another chunk; its place takes the sequence's start state
//       (forward) or the gradient of its final state (backward), which the second pass
//       cannot read from the state row any more, where another workgroup leaves the new one
//   kD: gradient: carry at the chunk's first token, from zero; last chunk: from the final one
enum { kA, kB, kD };

// The workgroup's chunk number and its block of channels. Workgroups go to the XCDs in turn; with `near` eight
// numbers at a time are given out, one to each XCD, with all their blocks, which share cache lines.
struct Slot {
    int item, cblock;
};
__device__ __forceinline__ Slot slot_of(const RecCut &k) {
    const int b = blockIdx.x, even = k.near ? k.items / 8 * 8 : 0;
    if (b >= even * k.cblocks) return {b / k.cblocks, b % k.cblocks};
    const int j = b / 8;
    return {j / k.cblocks * 8 + b % 8, j % k.cblocks};
}

// Where a workgroup stands.
struct Place {
    int chunk, last, item, end;  // number in the sequence, the last one's, in the call; end token
    long long lead, start;       // batch entry; first row of the sequence
    SeqRun r;
};

template <typename Args> __device__ __forceinline__ bool place_of(const Args &a, const RecCut &k, int item, Place &p) {
    p.item = item;
    p.start = 0;
    if (a.offsets) {
        if (!find_run(a.offsets, a.nseq, (int)a.tokens, k.run, item, &p.r)) return false;
        p.start = p.r.start;
    } else {
        p.r.seq = item / k.chunks;
        p.r.first = (item - p.r.seq * k.chunks) * k.run;
        p.r.len = (int)a.tokens;
        p.r.start = 0;
    }
    p.lead = a.offsets ? 0 : p.r.seq;
    p.chunk = p.r.first / k.run;
    p.last = p.r.len > 0 ? (p.r.len - 1) / k.run : 0;
    p.end = min(p.r.len, p.r.first + k.run);
    return true;
}

constexpr int kMaxRanked = 256;

// The sequence at place `at` of whole packed ones. The first `side` of them have a CU each for every block
// of channels, the next `side` share those CUs, and so on: the longest come first, and every other
// row of `side` runs backwards, so that long ones share with short ones. In this order and in
// that of their numbers, bf16, us: 16 ragged sequences of 32768 tokens x 4096 in all 238 and 276, 32 of
// 32000 x 2048 123 and 154, 64 of 8192 x 2048 34 and 36; 200 of 28000 x 1024 61 and 54. key: room for
// kMaxRanked.
__device__ __forceinline__ int by_length(const int *offsets, int nseq, int tokens, int at, int side, uint64_t *key, int &found) {
    for (int i = threadIdx.x; i < nseq; i += blockDim.x) {
        const int len = clamped_offset(offsets, i + 1, tokens) - clamped_offset(offsets, i, tokens);
        key[i] = (uint64_t)max(len, 0) << 32 | (uint32_t)(nseq - i);  // ties by number
    }
    __syncthreads();
    const int row = at / side, first = row * side, last = min(first + side, nseq) - 1;
    const int rank = row % 2 ? last - (at - first) : at;
    for (int i = threadIdx.x; i < nseq; i += blockDim.x) {
        const uint64_t mine = key[i];
        int before = 0;
        for (int j = 0; j < nseq; j++) before += key[j] > mine;
        if (before == rank) found = i;
    }
    __syncthreads();
    const int seq = __builtin_amdgcn_readfirstlane(found);
    __syncthreads();  // the keys' room is free again
    return seq;
}

template <typename T> __device__ __forceinline__ const T *rows(const void *p, const Place &w, long long batch, long long token) {
    return static_cast<const T *>(p) + w.lead * batch + w.start * token;
}
template <typename T> __device__ __forceinline__ T *rows(void *p, const Place &w, long long batch, long long token) {
    return static_cast<T *>(p) + w.lead * batch + w.start * token;
}

template <int VEC> using Floats = Pack<float, VEC>;

// A lane's channels: c to c + VEC - 1, of which it owns the last `own` (0: it only follows). The last
// lane of an odd number of channels takes the last two and owns one.
struct Channels {
    int c, own;
};
template <int VEC> __device__ __forceinline__ Channels channels_of(int ch, int channels) {
    if (ch + VEC <= channels) return {ch, VEC};
    return {channels - VEC, ch < channels ? channels - ch : 0};
}

// Rows need not be aligned to more than their type.
template <typename T, int VEC> __device__ __forceinline__ Pack<T, VEC> get(const T *p) {
    Pack<T, VEC> v;
    __builtin_memcpy(&v, p, sizeof v);
    return v;
}
template <typename T, int VEC> __device__ __forceinline__ void put(T *p, const Pack<T, VEC> &v, int own = VEC) {
    static_assert(VEC <= 2);
    if (own == VEC)
        __builtin_memcpy(p, &v, sizeof v);
    else if (VEC == 2 && own == 1)
        p[VEC - 1] = v.v[VEC - 1];
}

// Whether every lane of a wave owns all its channels.
template <int VEC> __device__ __forceinline__ bool all_own(int own) { return __all(own == VEC); }

// kTW tokens from t on of token rows, the last row again from `end` on.
template <typename T, int VEC>
__device__ __forceinline__ void fetch(Pack<T, VEC> (&v)[kTW], const T *p, long long token, int t, int end, int c) {
#pragma unroll
    for (int i = 0; i < kTW; i++) v[i] = get<T, VEC>(p + min(t + i, end - 1) * token + (unsigned)c);
}

// Composite of the records from lo on and before hi (towards later tokens, or earlier ones), the
// waves taking parts of them.
template <int VEC, bool BACK>
__device__ __forceinline__ Floats<VEC> fold(const float *rec, long long stride, int channels, int lo, int hi, int c, int wave,
                                            int lane, float2 (*s)[VEC][64]) {
    const int per = (hi - lo + kNW - 1) / kNW, first = min(lo + wave * per, hi), n = min(per, hi - first);
    float A[VEC], B[VEC];
#pragma unroll
    for (int v = 0; v < VEC; v++) A[v] = 1.0f, B[v] = 0.0f;
    for (int j0 = 0; j0 < n; j0 += 4) {
        Floats<VEC> ra[4], rb[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int j = min(j0 + i, n - 1);
            const float *p = rec + (BACK ? first + n - 1 - j : first + j) * stride + c;
            ra[i] = get<float, VEC>(p + kA * (long long)channels);
            rb[i] = get<float, VEC>(p + (BACK ? kD : kB) * (long long)channels);
        }
#pragma unroll
        for (int i = 0; i < 4; i++) {
            if (j0 + i >= n) break;
#pragma unroll
            for (int v = 0; v < VEC; v++) {
                B[v] = fmaf(ra[i].v[v], B[v], rb[i].v[v]);
                A[v] *= ra[i].v[v];
            }
        }
    }
#pragma unroll
    for (int v = 0; v < VEC; v++) s[wave][v][lane] = float2{A[v], B[v]};
    __syncthreads();
    Floats<VEC> out{};
#pragma unroll
    for (int w = 0; w < kNW; w++)
#pragma unroll
        for (int v = 0; v < VEC; v++) {
            const float2 m = s[BACK ? kNW - 1 - w : w][v][lane];
            out.v[v] = fmaf(m.x, out.v[v], m.y);
        }
    __syncthreads();
    return out;
}

// ---------------------------------------------------------------------------- prompts

// The first pass over split sequences, which leaves the chunks' records. A wave takes an eighth of
// the chunk and needs the others at the end only: no barriers, and tokens that nobody writes for.
// Bound by HBM: 65536 x 1024 bf16 in 50 to 52 us, 5.2 to 5.4 TB/s, the vector ALU 52 % busy.
template <typename T, int VEC, bool COUPLED>
__global__ __launch_bounds__(64 * kNW) void rec_first_kernel(const gated_recurrence_args a, const RecCut k) {
    __shared__ float2 s_run[kNW][VEC][64];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const auto [item, cblock] = slot_of(k);
    const auto [c, own] = channels_of<VEC>((cblock * 64 + lane) * VEC, a.channels);
    Place p;
    if (!place_of(a, k, item, p) || p.chunk == p.last) return;  // so the chunk is a whole run
    const T *x = rows<T>(a.x, p, a.x_batch, a.x_token), *forget = rows<T>(a.forget, p, a.forget_batch, a.forget_token);
    const long long stride = 2ll * a.channels;
    Floats<VEC> h{};
    if (p.chunk == 0 && wave == 0) {
        const int row = state_row(a.state, a.slots, p.r.seq, a.state_rows);
        if (row >= 0 && !a.fresh) h = get<float, VEC>(a.state + (long long)row * a.channels + c);
        put<float, VEC>(k.rec + (item + p.last) * stride + kB * (long long)a.channels + c, h, own);
    }
    float bias[VEC] = {};
#pragma unroll
    for (int v = 0; v < VEC; v++) bias[v] = a.forget_bias ? a.forget_bias[c + v] : 0.0f;
    float At[VEC], Bt[VEC];
#pragma unroll
    for (int v = 0; v < VEC; v++) At[v] = 1.0f, Bt[v] = 0.0f;
    const int part = (k.run + kNW * kTW - 1) / (kNW * kTW) * kTW, t0 = p.r.first + wave * part, t1 = min(t0 + part, p.end);
    Pack<T, VEC> nx[kTW], nf[kTW];
    if (t0 < t1) {
        fetch<T, VEC>(nf, forget, a.forget_token, t0, t1, c);
        fetch<T, VEC>(nx, x, a.x_token, t0, t1, c);
    }
    for (int t = t0; t < t1; t += kTW) {
        float f[kTW][VEC], b[kTW][VEC];
#pragma unroll
        for (int i = 0; i < kTW; i++)
#pragma unroll
            for (int v = 0; v < VEC; v++) {
                float take;
                gates(to_f32(nf[i].v[v]) + bias[v], f[i][v], take);
                b[i][v] = COUPLED ? to_f32(nx[i].v[v]) * take : to_f32(nx[i].v[v]);
            }
        if (t + kTW < t1) {
            fetch<T, VEC>(nf, forget, a.forget_token, t + kTW, t1, c);
            fetch<T, VEC>(nx, x, a.x_token, t + kTW, t1, c);
        }
#pragma unroll
        for (int i = 0; i < kTW; i++)
#pragma unroll
            for (int v = 0; v < VEC; v++) {
                Bt[v] = fmaf(f[i][v], Bt[v], b[i][v]);
                At[v] *= f[i][v];
            }
    }
#pragma unroll
    for (int v = 0; v < VEC; v++) s_run[wave][v][lane] = float2{At[v], Bt[v]};
    __syncthreads();
    if (wave != 0) return;
    Floats<VEC> decay;
#pragma unroll
    for (int v = 0; v < VEC; v++) decay.v[v] = p.chunk == 0 ? 0.0f : 1.0f;
#pragma unroll
    for (int w = 0; w < kNW; w++)
#pragma unroll
        for (int v = 0; v < VEC; v++) {
            const float2 m = s_run[w][v][lane];
            h.v[v] = fmaf(m.x, h.v[v], m.y);
            decay.v[v] *= m.x;
        }
    float *q = k.rec + item * stride + c;
    put<float, VEC>(q + kA * (long long)a.channels, decay, own);
    put<float, VEC>(q + kB * (long long)a.channels, h, own);
}

// The pass that writes y and the states. The eight waves of a tile take eight tokens each, so that a
// workgroup's loads and stores stand side by side and the next tile's are on their way over the one
// barrier of a tile (its LDS buffer alternates). Bound by HBM: 65536 x 1024 bf16 in 103 to 111 us behind the
// first pass, 4.8 to 5.2 TB/s; the vector ALU is 54 % busy, whence one exponential and one reciprocal a gate.
// Two workgroups a CU, for which registers are held to 128. Whole sequences need no first pass: 32768
// tokens x 4096 in ragged sequences 227 to 230 us, 4.7 TB/s, with fewer workgroups towards the end.
template <typename T, int VEC, bool COUPLED, bool GATED>
__global__ __launch_bounds__(64 * kNW, 4) void rec_prompt_kernel(const gated_recurrence_args a, const RecCut k) {
    __shared__ float2 s_run[2][kNW][VEC][64];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    // the second pass takes the chunks that the first read last first: they may still be cached
    __shared__ int s_found;
    const auto [place, cblock] = slot_of(k);
    const int item = k.ranked ? by_length(a.offsets, a.nseq, (int)a.tokens, place, k.ranked, reinterpret_cast<uint64_t *>(s_run), s_found)
                              : k.items - 1 - place;
    const auto [c, own] = channels_of<VEC>((cblock * 64 + lane) * VEC, a.channels);
    Place p;
    if (!place_of(a, k, item, p)) return;

    const T *x = rows<T>(a.x, p, a.x_batch, a.x_token), *forget = rows<T>(a.forget, p, a.forget_batch, a.forget_token);
    const T *gate = GATED ? rows<T>(a.gate, p, a.gate_batch, a.gate_token) : nullptr;
    T *y = rows<T>(a.y, p, a.y_batch, a.y_token);
    const int row = state_row(a.state, a.slots, p.r.seq, a.state_rows);
    float *state = row < 0 ? nullptr : a.state + (long long)row * a.channels + c;
    const long long stride = 2ll * a.channels;

    Floats<VEC> bias{}, h{};
    if (a.forget_bias) bias = get<float, VEC>(a.forget_bias + c);
    if (p.last == 0 && state && !a.fresh) h = get<float, VEC>(state);

    Pack<T, VEC> nx[kTW], nf[kTW], ng[kTW];
    auto next = [&](int t0) {
        const int t = t0 + wave * kTW;
        fetch<T, VEC>(nx, x, a.x_token, t, p.end, c);
        fetch<T, VEC>(nf, forget, a.forget_token, t, p.end, c);
        if (GATED) fetch<T, VEC>(ng, gate, a.gate_token, t, p.end, c);
    };
    if (p.end > p.r.first) next(p.r.first);
    if (p.last > 0) {
        const float *rec = k.rec + (item - p.chunk) * stride;
        if (p.chunk == 0)
            h = get<float, VEC>(rec + p.last * stride + kB * (long long)a.channels + c);
        else
            h = fold<VEC, false>(rec, stride, a.channels, 0, p.chunk, c, wave, lane, s_run[0]);
    }

    int buf = 0;
    auto tile = [&](int t0, auto full) {
        constexpr bool kFull = decltype(full)::value;
        const int t = t0 + wave * kTW;
        float f[kTW][VEC], b[kTW][VEC], A[VEC], B[VEC];
        Pack<T, VEC> g[kTW];
#pragma unroll
        for (int v = 0; v < VEC; v++) A[v] = 1.0f, B[v] = 0.0f;
#pragma unroll
        for (int i = 0; i < kTW; i++) {
#pragma unroll
            for (int v = 0; v < VEC; v++) {
                float take;
                gates(to_f32(nf[i].v[v]) + bias.v[v], f[i][v], take);
                b[i][v] = COUPLED ? to_f32(nx[i].v[v]) * take : to_f32(nx[i].v[v]);
                if (!kFull && t + i >= p.end) f[i][v] = 1.0f, b[i][v] = 0.0f;
                B[v] = fmaf(f[i][v], B[v], b[i][v]);
                A[v] *= f[i][v];
            }
            if (GATED) g[i] = ng[i];
        }
        if (t0 + kTile < p.end) next(t0 + kTile);
#pragma unroll
        for (int v = 0; v < VEC; v++) s_run[buf][wave][v][lane] = float2{A[v], B[v]};
        __syncthreads();
        float from[VEC];  // the wave's start state
#pragma unroll
        for (int w = 0; w < kNW; w++)
#pragma unroll
            for (int v = 0; v < VEC; v++) {
                if (w == wave) from[v] = h.v[v];
                const float2 m = s_run[buf][w][v][lane];
                h.v[v] = fmaf(m.x, h.v[v], m.y);
            }
        buf ^= 1;
#pragma unroll
        for (int i = 0; i < kTW; i++) {
            Pack<T, VEC> out;
#pragma unroll
            for (int v = 0; v < VEC; v++) {
                from[v] = fmaf(f[i][v], from[v], b[i][v]);
                const float z = GATED ? activate_c<CONV2D_ACT_SILU>(to_f32(g[i].v[v]), 0.0f) : 1.0f;
                out.v[v] = round_fp32<T>(GATED ? from[v] * z : from[v]);
            }
            if (kFull)
                put<T, VEC>(y + (t + i) * a.y_token + (unsigned)c, out);
            else if (t + i < p.end)
                put<T, VEC>(y + (t + i) * a.y_token + (unsigned)c, out, own);
        }
    };
    int t0 = p.r.first;
    if (all_own<VEC>(own))
        for (; t0 + kTile <= p.end; t0 += kTile) tile(t0, std::true_type{});
    for (; t0 < p.end; t0 += kTile) tile(t0, std::false_type{});
    if (wave == 0 && state && p.chunk == p.last) put<float, VEC>(state, h, own);
}

// ---------------------------------------------------------------------------- gradient

// The first pass of the gradient walks forwards: it leaves, for each tile, the state before it as
// an affine map of the state before the chunk, and, for split sequences, the chunks' records. A map
// of 8 bytes for 64 tokens spares the second pass a walk of its own. HBM: 8 x 4096 x 2048 bf16 in 125 us,
// 4.3 TB/s, the vector ALU 47 % busy. (A wave with an eighth of the chunk to itself, without the tile's
// barrier, as in rec_first_kernel: 3 to 5 % slower for the whole call, whose second pass starts where
// the workgroups' last tiles may still be cached.)
template <typename T, int VEC, bool GATED, bool SPLIT>
__global__ __launch_bounds__(64 * kNW) void rec_back_first_kernel(const gated_recurrence_backward_args a, const RecCut k) {
    __shared__ float4 s_run[2][kNW][VEC][64];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    __shared__ int s_found;
    auto [item, cblock] = slot_of(k);
    if (k.ranked) item = by_length(a.offsets, a.nseq, (int)a.tokens, item, k.ranked, reinterpret_cast<uint64_t *>(s_run), s_found);
    const auto [c, own] = channels_of<VEC>((cblock * 64 + lane) * VEC, a.channels);
    Place p;
    if (!place_of(a, k, item, p)) return;
    const bool split = p.last > 0;

    const T *x = rows<T>(a.x, p, a.x_batch, a.x_token), *forget = rows<T>(a.forget, p, a.forget_batch, a.forget_token);
    const T *gate = GATED ? rows<T>(a.gate, p, a.gate_batch, a.gate_token) : nullptr;
    const T *grad = rows<T>(a.grad, p, a.grad_batch, a.grad_token);
    const long long tiles = a.offsets ? 0 : (a.tokens + kTile - 1) / kTile;
    float *tile = k.tile + (a.offsets ? p.start / kTile + p.r.seq : p.r.seq * tiles) * 2 * a.channels + c;

    Floats<VEC> bias{}, h{}, carry{};
    if (a.forget_bias) bias = get<float, VEC>(a.forget_bias + c);
    if (p.chunk == 0) {
        const int row = state_row(a.state, a.slots, p.r.seq, a.state_rows);
        if (row >= 0) h = get<float, VEC>(a.state + (long long)row * a.channels + c);
    }
    if (split && p.chunk == p.last) {
        const int row = state_row(a.grad_state, a.slots, p.r.seq, a.state_rows);
        if (row >= 0) carry = get<float, VEC>(a.grad_state + (long long)row * a.channels + c);
    }
    Pack<T, VEC> nx[kTW], nf[kTW], ng[kTW], ne[kTW];
    auto next = [&](int t0) {
        const int t = t0 + wave * kTW;
        fetch<T, VEC>(nx, x, a.x_token, t, p.end, c);
        fetch<T, VEC>(nf, forget, a.forget_token, t, p.end, c);
        if (SPLIT) {
            fetch<T, VEC>(ne, grad, a.grad_token, t, p.end, c);
            if constexpr (GATED) fetch<T, VEC>(ng, gate, a.gate_token, t, p.end, c);
        }
    };
    if (p.end > p.r.first) next(p.r.first);
    float decay[VEC], D[VEC];  // of the chunk so far
#pragma unroll
    for (int v = 0; v < VEC; v++) decay[v] = 1.0f, D[v] = 0.0f;

    int buf = 0;
    for (int t0 = p.r.first; t0 < p.end; t0 += kTile) {
        if (wave == 0) {
            float *q = tile + (t0 / kTile) * 2ll * a.channels;
            Floats<VEC> A;
#pragma unroll
            for (int v = 0; v < VEC; v++) A.v[v] = p.chunk == 0 ? 0.0f : decay[v];
            put<float, VEC>(q, A, own);
            put<float, VEC>(q + a.channels, h, own);
        }
        const int t = t0 + wave * kTW;
        float A[VEC], B[VEC], E[VEC];
#pragma unroll
        for (int v = 0; v < VEC; v++) A[v] = 1.0f, B[v] = 0.0f, E[v] = 0.0f;
#pragma unroll
        for (int i = 0; i < kTW; i++) {
#pragma unroll
            for (int v = 0; v < VEC; v++) {
                float f, take;
                gates(to_f32(nf[i].v[v]) + bias.v[v], f, take);
                float b = to_f32(nx[i].v[v]) * (a.coupled ? take : 1.0f);
                if (t + i >= p.end) f = 1.0f, b = 0.0f;
                B[v] = fmaf(f, B[v], b);
                A[v] *= f;
                if (SPLIT) {
                    float e = to_f32(ne[i].v[v]);
                    if constexpr (GATED) e *= activate_c<CONV2D_ACT_SILU>(to_f32(ng[i].v[v]), 0.0f);
                    if (t + i >= p.end) e = 0.0f;
                    E[v] = fmaf(A[v], e, E[v]);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if (t0 + kTile < p.end) next(t0 + kTile);
#pragma unroll
        for (int v = 0; v < VEC; v++) s_run[buf][wave][v][lane] = float4{A[v], B[v], E[v], 0.0f};
        __syncthreads();
        const auto *runs = s_run[buf];
        buf ^= 1;
        if (wave != 0) continue;
#pragma unroll
        for (int w = 0; w < kNW; w++)
#pragma unroll
            for (int v = 0; v < VEC; v++) {
                const float4 m = runs[w][v][lane];
                h.v[v] = fmaf(m.x, h.v[v], m.y);
                D[v] = fmaf(decay[v], m.z, D[v]);
                decay[v] *= m.x;
            }
    }
    if (!split || wave != 0) return;
    float *q = k.rec + item * 3ll * a.channels + c;
    Floats<VEC> A, B, E;
    const bool last = p.chunk == p.last;
#pragma unroll
    for (int v = 0; v < VEC; v++) {
        A.v[v] = p.chunk == 0 || last ? 0.0f : decay[v];
        B.v[v] = last ? carry.v[v] : h.v[v];
        E.v[v] = last ? fmaf(decay[v], carry.v[v], D[v]) : D[v];
    }
    put<float, VEC>(q + kA * (long long)a.channels, A, own);
    put<float, VEC>(q + kB * (long long)a.channels, B, own);
    put<float, VEC>(q + kD * (long long)a.channels, E, own);
}

// The second pass walks backwards over the tiles and writes the gradients: the states before each
// token again from the tile's, and the carry against them, both composed over the waves from the
// same LDS records. Four inputs on their way and four values a token kept take 250 registers in f16, so one
// workgroup a CU, and in gated bf16 256 and 12 to 24 bytes a lane spilled. Forms without the spill are no faster: with the
// records of one direction read before the other's (231 registers) 8 x 4096 x 2048 takes 311 us, not 309, 64 ragged
// sequences of 16000 x 1500 148, not 141; with x unpacked again for each use (251) 310 and 141.
// HBM: 8 x 4096 x 2048 bf16 in 178 to 182 us, 5.2 TB/s, the vector ALU 56 % busy. WHOLE: the channels
// fill their blocks, which all waves would ask otherwise (a gradient of 8 x 4096 x 2048 in 313 us, not 323); else the
// waves whose lanes all own theirs still store without a look at each (8 x 4096 x 2112 352 us, not 392).
template <typename T, int VEC, bool WHOLE, bool GATED>
__global__ __launch_bounds__(64 * kNW) void rec_back_kernel(const gated_recurrence_backward_args a, const RecCut k) {
    __shared__ float4 s_run[2][kNW][VEC][64];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    __shared__ int s_found;
    const auto [place, cblock] = slot_of(k);
    const int item = k.ranked ? by_length(a.offsets, a.nseq, (int)a.tokens, place, k.ranked, reinterpret_cast<uint64_t *>(s_run), s_found)
                              : k.items - 1 - place;
    const auto [c, own] = channels_of<VEC>((cblock * 64 + lane) * VEC, a.channels);
    const bool whole = WHOLE || all_own<VEC>(own);
    float sum[VEC];
#pragma unroll
    for (int v = 0; v < VEC; v++) sum[v] = 0.0f;
    Place p;
    if (!place_of(a, k, item, p)) {
        if (k.bias && wave == 0) put<float, VEC>(k.bias + item * (long long)a.channels + c, Floats<VEC>{}, own);
        return;
    }
    const T *x = rows<T>(a.x, p, a.x_batch, a.x_token), *forget = rows<T>(a.forget, p, a.forget_batch, a.forget_token);
    const T *gate = GATED ? rows<T>(a.gate, p, a.gate_batch, a.gate_token) : nullptr;
    const T *grad = rows<T>(a.grad, p, a.grad_batch, a.grad_token);
    T *gx = rows<T>(a.grad_x, p, a.grad_x_batch, a.grad_x_token);
    T *gf = rows<T>(a.grad_forget, p, a.grad_forget_batch, a.grad_forget_token);
    T *gg = GATED ? rows<T>(a.grad_gate, p, a.grad_gate_batch, a.grad_gate_token) : nullptr;
    const long long tiles = a.offsets ? 0 : (a.tokens + kTile - 1) / kTile;
    const float *tile = k.tile + (a.offsets ? p.start / kTile + p.r.seq : p.r.seq * tiles) * 2 * a.channels + c;
    const int row = state_row(a.grad_state, a.slots, p.r.seq, a.state_rows);
    float *grad_state = row < 0 ? nullptr : a.grad_state + (long long)row * a.channels + c;

    Floats<VEC> bias{}, before{}, carry{};  // state before the chunk, gradient carried into the tile
    if (a.forget_bias) bias = get<float, VEC>(a.forget_bias + c);

    Pack<T, VEC> nx[kTW], nf[kTW], ng[kTW], ne[kTW];
    Floats<VEC> na, nb;
    auto next = [&](int t0) {
        const int t = t0 + wave * kTW;
        const float *q = tile + (t0 / kTile) * 2ll * a.channels;
        na = get<float, VEC>(q);
        nb = get<float, VEC>(q + a.channels);
        fetch<T, VEC>(nx, x, a.x_token, t, p.end, c);
        fetch<T, VEC>(nf, forget, a.forget_token, t, p.end, c);
        fetch<T, VEC>(ne, grad, a.grad_token, t, p.end, c);
        if constexpr (GATED) fetch<T, VEC>(ng, gate, a.gate_token, t, p.end, c);
    };
    const int final = p.end > p.r.first ? p.r.first + (p.end - 1 - p.r.first) / kTile * kTile : p.r.first - kTile;
    if (final >= p.r.first) next(final);
    if (p.last > 0) {
        const float *rec = k.rec + (item - p.chunk) * 3ll * a.channels;
        float2(*s)[VEC][64] = reinterpret_cast<float2(*)[VEC][64]>(s_run);
        if (p.chunk > 0) before = fold<VEC, false>(rec, 3ll * a.channels, a.channels, 0, p.chunk, c, wave, lane, s);
        if (p.chunk < p.last)
            carry = fold<VEC, true>(rec, 3ll * a.channels, a.channels, p.chunk + 1, p.last + 1, c, wave, lane, s);
        else
            carry = get<float, VEC>(rec + p.last * 3ll * a.channels + kB * (long long)a.channels + c);
    } else if (grad_state) {
        carry = get<float, VEC>(grad_state);
    }

    int buf = 0;
    for (int t0 = final; t0 >= p.r.first; t0 -= kTile) {
        const int t = t0 + wave * kTW;
        float xs[kTW][VEC], f[kTW][VEC], take[kTW][VEC], e[kTW][VEC], dz[kTW][VEC], A[VEC], B[VEC], D[VEC];
        float start[VEC];
#pragma unroll
        for (int v = 0; v < VEC; v++) {
            A[v] = 1.0f, B[v] = 0.0f, D[v] = 0.0f;
            start[v] = fmaf(na.v[v], before.v[v], nb.v[v]);
        }
#pragma unroll
        for (int i = 0; i < kTW; i++) {
#pragma unroll
            for (int v = 0; v < VEC; v++) {
                xs[i][v] = to_f32(nx[i].v[v]);
                gates(to_f32(nf[i].v[v]) + bias.v[v], f[i][v], take[i][v]);
                e[i][v] = to_f32(ne[i].v[v]);
                dz[i][v] = 0.0f;
                if constexpr (GATED) {
                    const float g = to_f32(ng[i].v[v]);
                    float up, down;
                    gates(g, up, down);
                    dz[i][v] = e[i][v] * up * fmaf(g, down, 1.0f);
                    e[i][v] *= g * up;
                }
                if (t + i >= p.end) f[i][v] = 1.0f, xs[i][v] = 0.0f, e[i][v] = 0.0f;
                const float b = xs[i][v] * (a.coupled ? take[i][v] : 1.0f);
                B[v] = fmaf(f[i][v], B[v], b);
                D[v] = fmaf(A[v] * f[i][v], e[i][v], D[v]);
                A[v] *= f[i][v];
            }
            __builtin_amdgcn_sched_barrier(0);  // token by token, as their loads arrive
        }
        if (t0 > p.r.first) next(t0 - kTile);
#pragma unroll
        for (int v = 0; v < VEC; v++) s_run[buf][wave][v][lane] = float4{A[v], B[v], D[v], 0.0f};
        __syncthreads();
        float h[VEC], cin[VEC];  // state before the wave's tokens, carry behind them
#pragma unroll
        for (int w = 0; w < kNW; w++)
#pragma unroll
            for (int v = 0; v < VEC; v++) {
                if (w == wave) h[v] = start[v];
                const float4 m = s_run[buf][w][v][lane];
                start[v] = fmaf(m.x, start[v], m.y);
            }
#pragma unroll
        for (int w = kNW - 1; w >= 0; w--)
#pragma unroll
            for (int v = 0; v < VEC; v++) {
                if (w == wave) cin[v] = carry.v[v];
                const float4 m = s_run[buf][w][v][lane];
                carry.v[v] = fmaf(m.x, carry.v[v], m.z);
            }
        float prev[kTW][VEC];  // states before each token
#pragma unroll
        for (int i = 0; i < kTW; i++)
#pragma unroll
            for (int v = 0; v < VEC; v++) {
                prev[i][v] = h[v];
                h[v] = fmaf(f[i][v], h[v], xs[i][v] * (a.coupled ? take[i][v] : 1.0f));
                dz[i][v] *= h[v];
            }
#pragma unroll
        for (int i = kTW - 1; i >= 0; i--) {
            Pack<T, VEC> ox, of, og;
#pragma unroll
            for (int v = 0; v < VEC; v++) {
                const float g = e[i][v] + cin[v];
                const float d = g * f[i][v] * take[i][v] * (a.coupled ? prev[i][v] - xs[i][v] : prev[i][v]);
                ox.v[v] = round_fp32<T>(a.coupled ? g * take[i][v] : g);
                of.v[v] = round_fp32<T>(d);
                og.v[v] = round_fp32<T>(dz[i][v]);
                cin[v] = g * f[i][v];
                if (t + i < p.end) sum[v] += d;
            }
            if (t + i < p.end) {
                T *px = gx + (t + i) * a.grad_x_token + (unsigned)c, *pf = gf + (t + i) * a.grad_forget_token + (unsigned)c, *pg;
                if constexpr (GATED) pg = gg + (t + i) * a.grad_gate_token + (unsigned)c;
                if (whole) {
                    put<T, VEC>(px, ox);
                    put<T, VEC>(pf, of);
                    if constexpr (GATED) put<T, VEC>(pg, og);
                } else {
                    put<T, VEC>(px, ox, own);
                    put<T, VEC>(pf, of, own);
                    if constexpr (GATED) put<T, VEC>(pg, og, own);
                }
            }
        }
        buf ^= 1;
    }
    if (k.bias) {
        __syncthreads();
#pragma unroll
        for (int v = 0; v < VEC; v++) s_run[0][wave][v][lane].x = sum[v];
        __syncthreads();
        if (wave == 0) {
            Floats<VEC> total{};
#pragma unroll
            for (int w = 0; w < kNW; w++)
#pragma unroll
                for (int v = 0; v < VEC; v++) total.v[v] += s_run[0][w][v][lane].x;
            put<float, VEC>(k.bias + item * (long long)a.channels + c, total, own);
        }
    }
    if (wave == 0 && grad_state && p.chunk == 0) put<float, VEC>(grad_state, carry, own);
}

// Sums of `items` rows of partial sums, in a fixed order. 1.5 to 4.6 us, of which most is the launch and the
// first access. Sums by atomics in the second pass would have no order; a ticket, with the last workgroup of a block of
// channels adding the rows, would have this one and no launch (not built).
__global__ __launch_bounds__(1024) void rec_bias_kernel(const float *part, float *out, int items, int channels) {
    __shared__ float s[16][64];
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int c = blockIdx.x * 64 + lane, at = min(c, channels - 1);
    float sum = 0.0f;
    for (int i = wave; i < items; i += 16) sum += part[i * (long long)channels + at];
    s[wave][lane] = sum;
    __syncthreads();
    if (wave || c >= channels) return;
    sum = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; w++) sum += s[w][lane];
    out[c] = sum;
}

// ---------------------------------------------------------------------------- single tokens

constexpr int kBlock = 256;

// One token of each sequence, VEC channels a thread, a row of threads for each sequence. Bound by
// latency (1 x 2048: 2.6 us) and, with many sequences, by HBM and the last-level cache (512 x 4096 f16 6.8
// us, 4.9 TB/s).
template <typename T, int VEC>
__global__ __launch_bounds__(kBlock) void rec_token_kernel(const gated_recurrence_args a, int cblocks) {
    const int c = ((int)(blockIdx.x % cblocks) * kBlock + threadIdx.x) * VEC;
    const long long seq = blockIdx.x / cblocks;
    if (c >= a.channels) return;
    const int row = state_row(a.state, a.slots, (int)seq, a.state_rows);
    float *state = row < 0 ? nullptr : a.state + (long long)row * a.channels + c;
    const Pack<T, VEC> x = load_pack<T, VEC>((const T *)a.x + seq * a.x_token + c);
    const Pack<T, VEC> z = load_pack<T, VEC>((const T *)a.forget + seq * a.forget_token + c);
    Pack<T, VEC> gate{}, y;
    Floats<VEC> bias{}, h{};
    if (a.gate) gate = load_pack<T, VEC>((const T *)a.gate + seq * a.gate_token + c);
    if (a.forget_bias) bias = load_pack<float, VEC>(a.forget_bias + c);
    if (state && !a.fresh) h = load_pack<float, VEC>(state);
#pragma unroll
    for (int v = 0; v < VEC; v++) {
        float keep, take;
        gates(to_f32(z.v[v]) + bias.v[v], keep, take);
        h.v[v] = fmaf(keep, h.v[v], to_f32(x.v[v]) * (a.coupled ? take : 1.0f));
        y.v[v] = round_fp32<T>(a.gate ? h.v[v] * activate_c<CONV2D_ACT_SILU>(to_f32(gate.v[v]), 0.0f) : h.v[v]);
    }
    if (state) store_pack<float, VEC>(state, h);
    store_pack<T, VEC>((T *)a.y + seq * a.y_token + c, y);
}

template <typename T, int VEC> hipError_t launch_token(const gated_recurrence_args &a, hipStream_t st) {
    const int cblocks = (a.channels + kBlock * VEC - 1) / (kBlock * VEC);
    return launch_blocks(rec_token_kernel<T, VEC>, (long long)cblocks * a.nseq, kBlock, st, a, cblocks);
}

// ---------------------------------------------------------------------------- host

// What a call costs whole and split, in us: fixed, a tile of a sequence left whole (one after the
// other), and the values moved for each that the call takes in or gives out, whole and split (a second
// pass finds a few of its values cached).
struct Costs {
    double fixed_whole, fixed_split, tile_us, moved_whole, moved_split;
    bool share;  // workgroups share CUs (the gradient's hold one each)
};
// Measured, bf16, us whole / split:
//   sequences x tokens x channels   prompt             gradient
//   1 x 256 x 1024                   9.8 /   8.4       25 /  14
//   1 x 4096 x 1024                  148 /  16         376 /  30
//   32 x 512 x 2048                   46 /  68         128 / 170
//   12 x 1000 x 1280                  43 /  39         105 /  74
//   8 x 4096 x 2048                  174 / 138         464 / 312
//   8 x 4096 x 2176                  177 / 163         452 / 342
//   16 x 2048 x 2176                 156 / 156         406 / 353
//   16 x 2048 x 4096, ragged         253 / 330         620 / 666
//   64 x 250 x 1500, ragged           52 /  75         141 / 198
//   40 x 1000 x 2112, ragged         159 / 205         387 / 530
//   32 x 1000 x 1000, ragged         124 /  86         322 / 236
//   1 x 65536 x 1024                2590 / 157        6510 / 331
constexpr Costs kPrompt{3.0, 9.0, 2.2, 4.0, 4.7, true}, kGradient{8.0, 17.0, 5.8, 9.0, 10.3, false};

constexpr int kWorkgroups = 256;        // that the card runs at full speed side by side: one for each CU
constexpr int kRaggedWorkgroups = 768;  // of a split call whose sequences are not as long as each other, which evens them out
// (8 x 1000 x 2048, ragged, into 256, 384, 512, 768, 1024 workgroups, us: prompt 54.2, 44.5, 44.6, 38.6,
// 42.3, gradient 100, 94.0, 91.9, 84.5, 95.8)

// How long that many equal workgroups take, in the time of one among kWorkgroups: those of a last
// round that does not fill the card are faster, but not by as much as they are fewer.
double rounds(long long groups) {
    if (groups <= kWorkgroups) return 1.0;
    const double rest = (double)(groups % kWorkgroups) / kWorkgroups;
    return (double)(groups / kWorkgroups) + (rest > 0.0 ? 0.6 + 0.4 * rest : 0.0);
}

// The tiles of a chunk that equal sequences of `tiles` tiles, each in `wide` blocks of channels, are
// best split into: nearly whole rounds of workgroups, few chunks. By its factor over a full card's time the call
// takes longer. Into 2, 3, 4, 5, 6 chunks a sequence, us:
//   8 x 4096 x 2176 (272 to 816 workgroups)     prompt 187, 159, 169, 157, 161   gradient 483, 365, 401, 346, 368
//   16 x 4096 x 1024 (256 to 768)                      133, 166, 138, 159, 145            308, 378, 303, 348, 321
//   3 x 2048 x 4096 (192 to 576)                        63,  62,  58,  55,  60            135, 158, 131, 121, 125
long long best_run(long long tiles, long long wide, double *factor) {
    constexpr double kStart = 0.35;  // tiles' time that a workgroup takes to start
    const double full = (double)(tiles * wide) / kWorkgroups;
    long long run = tiles;
    double least = 0.0;
    for (int full_rounds = 1; full_rounds <= 8; full_rounds++) {
        const long long c = std::min(std::max(full_rounds * kWorkgroups / wide, 2ll), tiles);
        const long long r = (tiles + c - 1) / c, groups = (tiles + r - 1) / r * wide;
        const double time = rounds(groups) * (double)r + kStart * (double)((groups + kWorkgroups - 1) / kWorkgroups);
        if (full_rounds == 1 || time < least) run = r, least = time;
    }
    *factor = least / (full + kStart);
    return run;
}

// How a call is cut. A sequence left whole is walked by one workgroup for each 64 VEC channels, so its
// length is a time; a split one is read twice.
template <typename Args> RecCut cut(const Args &a, int vec, const Costs &costs, bool may_split) {
    RecCut k{};
    k.cblocks = (a.channels + 64 * vec - 1) / (64 * vec);
    const bool ragged = a.offsets && a.nseq > 1;
    const long long total = a.offsets ? a.tokens : a.tokens * a.nseq;
    long long longest = a.offsets ? (a.longest ? a.longest : 2 * (total / std::max(a.nseq, 1))) : a.tokens;
    if (longest > a.tokens) longest = a.tokens;
    const long long tiles = (longest + kTile - 1) / kTile, wide = (long long)a.nseq * k.cblocks;
    k.run = kWhole;
    // us to move one value of each token and channel at 4.7 TB/s
    const double value_us = (double)total * a.channels * dtype_bytes(a.dtype) / 4.7e6;
    // ragged sequences and waits for other workgroups' loads make a walk longer than its tiles alone
    const double walk = 1.3 * costs.tile_us * (double)tiles * (ragged ? 1.0 : rounds(wide));
    const double whole = costs.fixed_whole + std::max(walk, costs.moved_whole * value_us);
    if (may_split && wide && whole > costs.fixed_split + costs.moved_split * value_us) {
        // ragged: a sequence's last chunk is as short as it comes
        double factor = 1.1 + 0.5 * (double)wide / kRaggedWorkgroups;
        const long long run = ragged ? std::max((total * k.cblocks + kRaggedWorkgroups * kTile - 1) / (kRaggedWorkgroups * kTile), 1ll)
                                     : best_run(tiles, wide, &factor);
        if (run < tiles && whole > costs.fixed_split + costs.moved_split * value_us * factor) k.run = (int)(run * kTile);
    }
    k.chunks = a.offsets ? 0 : (int)std::max((a.tokens + k.run - 1) / k.run, 1ll);
    k.items = a.offsets ? (int)(a.tokens / k.run + a.nseq) : k.chunks * a.nseq;
    // Rows that do not start on cache lines share them between blocks of channels. On one XCD and on any, us,
    // prompt / gradient: 5 x 3000 x 1500 60 / 132 and 68 / 144, 8 x 4096 x 2050 161 / 406 and 183 / 432, 32 ragged
    // sequences of 32000 x 1000 84 / 236 and 93 / 243. Rows on lines: 8 x 4096 x 2048 130 / 309 and 131 / 306; few ragged
    // chunks fill the XCDs unevenly (6 sequences of 20000 x 2560 133 / 309 and 116 / 266), and small calls have little
    // to share (1 x 999 x 250 13 / 18 and 10 / 16). The other rows are taken to stand as x and forget do.
    const uintptr_t lines = (uintptr_t)a.x | (uintptr_t)a.forget | (uintptr_t)(a.x_token * dtype_bytes(a.dtype)) |
                            (uintptr_t)(a.forget_token * dtype_bytes(a.dtype));
    k.near = lines % 128 != 0 && value_us > 1.0 && (!ragged || k.items >= 64);
    // the order costs each workgroup a look at all lengths, which long sequences earn back
    if (a.offsets && k.run == kWhole && k.items == a.nseq && a.nseq <= kMaxRanked && wide > kWorkgroups &&
        a.tokens >= 2ll * a.nseq * a.nseq)
        k.ranked = costs.share ? std::max(kWorkgroups / k.cblocks, 1) : kMaxRanked;
    return k;
}

// The channels of a lane, and the cut of a call with them: two of 16 bits, four bytes of a row, but one
// where tiles of two would not make a workgroup for each CU (us: 1 x 77 x 512 8.1 and 6.3, 1 x 1024 x 1024
// 10.3 and 8.7, its gradient 18.2 and 14.7; 1 x 4096 x 1024 15.3 and 19.6).
template <typename Args> RecCut plan(const Args &a, const Costs &costs, bool may_split, int *vec) {
    const long long total = a.offsets ? a.tokens : a.tokens * a.nseq;
    *vec = a.dtype == CONV2D_DTYPE_F32 || a.channels == 1 || total * ((a.channels + 127) / 128) < (long long)kWorkgroups * kTile ? 1 : 2;
    return cut(a, *vec, costs, may_split);
}

size_t record_bytes(const RecCut &k, int fields, int channels) {
    return k.run < kWhole ? ((size_t)k.items * fields * channels * 4 + 255) / 256 * 256 : 0;
}

// Calls f with the two as integral constants.
template <typename F> hipError_t by_form(bool first, bool gated, F f) {
    if (first) return gated ? f(std::true_type{}, std::true_type{}) : f(std::true_type{}, std::false_type{});
    return gated ? f(std::false_type{}, std::true_type{}) : f(std::false_type{}, std::false_type{});
}

template <typename T, int VEC> hipError_t launch_prompt(const gated_recurrence_args &a, const RecCut &k, hipStream_t st) {
    const long long blocks = (long long)k.items * k.cblocks;
    return by_form(a.coupled, a.gate, [&](auto coupled, auto gated) {
        constexpr bool C = decltype(coupled)::value, G = decltype(gated)::value;
        hipError_t e = hipSuccess;
        if (k.rec) e = launch_blocks(rec_first_kernel<T, VEC, C>, blocks, 64 * kNW, st, a, k);
        return e != hipSuccess ? e : launch_blocks(rec_prompt_kernel<T, VEC, C, G>, blocks, 64 * kNW, st, a, k);
    });
}

template <typename T, int VEC> hipError_t launch_back(const gated_recurrence_backward_args &a, const RecCut &k, hipStream_t st) {
    const long long blocks = (long long)k.items * k.cblocks, bias_blocks = (a.channels + 63) / 64;
    if (a.grad_forget_bias && bias_blocks > 0xffffffffll / 1024) return hipErrorInvalidConfiguration;  // before any launch
    hipError_t e = hipSuccess;
    if (blocks) {
        if (!k.rec)
            e = launch_blocks(rec_back_first_kernel<T, VEC, false, false>, blocks, 64 * kNW, st, a, k);
        else if (a.gate)
            e = launch_blocks(rec_back_first_kernel<T, VEC, true, true>, blocks, 64 * kNW, st, a, k);
        else
            e = launch_blocks(rec_back_first_kernel<T, VEC, false, true>, blocks, 64 * kNW, st, a, k);
        if (e == hipSuccess)
            e = by_form(a.channels % (64 * VEC) == 0, a.gate, [&](auto whole, auto gated) {
                return launch_blocks(rec_back_kernel<T, VEC, decltype(whole)::value, decltype(gated)::value>, blocks, 64 * kNW, st, a, k);
            });
    }
    if (e == hipSuccess && a.grad_forget_bias)
        e = launch_blocks(rec_bias_kernel, bias_blocks, 1024, st, k.bias, a.grad_forget_bias, k.items, a.channels);
    return e;
}

struct BackLayout {
    RecCut k;
    int vec;
    size_t rec, tile, bias, bytes;
};

BackLayout back_layout(const gated_recurrence_backward_args &a) {
    BackLayout l{};
    l.k = plan(a, kGradient, true, &l.vec);
    if (a.nseq == 0) {  // no chunks: only a bias gradient of zeros is written
        l.k.items = 0;
        return l;
    }
    l.rec = record_bytes(l.k, 3, a.channels);
    const long long tiles = a.offsets ? a.tokens / kTile + a.nseq : (a.tokens + kTile - 1) / kTile * a.nseq;
    l.tile = ((size_t)tiles * 2 * a.channels * 4 + 255) / 256 * 256;
    l.bias = a.grad_forget_bias ? (size_t)l.k.items * a.channels * 4 : 0;
    l.bytes = l.rec + l.tile + l.bias;
    return l;
}

}  // namespace

size_t recurrence_workspace(const gated_recurrence_args &a) {
    int vec;
    return record_bytes(plan(a, kPrompt, true, &vec), 2, a.channels);
}

hipError_t launch_recurrence(const gated_recurrence_args &a, void *ws, size_t ws_bytes, hipStream_t st) {
    int vec;
    RecCut k = plan(a, kPrompt, true, &vec);
    const size_t want = record_bytes(k, 2, a.channels);
    if (want && ws && want <= ws_bytes)
        k.rec = static_cast<float *>(ws);
    else
        k = plan(a, kPrompt, false, &vec);
    if (a.dtype == CONV2D_DTYPE_F32) return launch_prompt<float, 1>(a, k, st);
    if (a.dtype == CONV2D_DTYPE_BF16) return vec == 2 ? launch_prompt<bf16, 2>(a, k, st) : launch_prompt<bf16, 1>(a, k, st);
    return vec == 2 ? launch_prompt<f16, 2>(a, k, st) : launch_prompt<f16, 1>(a, k, st);
}

hipError_t launch_recurrence_token(const gated_recurrence_args &a, hipStream_t st) {
    const int vec = a.dtype == CONV2D_DTYPE_F32 ? 4 : 8;
    const bool whole = a.channels % vec == 0 && aligned16(a.x) && aligned16(a.forget) && aligned16(a.gate) && aligned16(a.y) &&
                       a.x_token % vec == 0 && a.forget_token % vec == 0 && (!a.gate || a.gate_token % vec == 0) &&
                       a.y_token % vec == 0 && aligned16(a.forget_bias) && aligned16(a.state);
    if (a.dtype == CONV2D_DTYPE_F32) return whole ? launch_token<float, 4>(a, st) : launch_token<float, 1>(a, st);
    if (a.dtype == CONV2D_DTYPE_BF16) return whole ? launch_token<bf16, 8>(a, st) : launch_token<bf16, 1>(a, st);
    return whole ? launch_token<f16, 8>(a, st) : launch_token<f16, 1>(a, st);
}

size_t recurrence_backward_workspace(const gated_recurrence_backward_args &a) { return back_layout(a).bytes; }

hipError_t launch_recurrence_backward(const gated_recurrence_backward_args &a, void *ws, hipStream_t st) {
    BackLayout l = back_layout(a);
    char *p = static_cast<char *>(ws);
    if (l.rec) l.k.rec = reinterpret_cast<float *>(p);
    l.k.tile = reinterpret_cast<float *>(p + l.rec);
    if (a.grad_forget_bias) l.k.bias = reinterpret_cast<float *>(p + l.rec + l.tile);
    const int vec = l.vec;
    if (a.dtype == CONV2D_DTYPE_F32) return launch_back<float, 1>(a, l.k, st);
    if (a.dtype == CONV2D_DTYPE_BF16) return vec == 2 ? launch_back<bf16, 2>(a, l.k, st) : launch_back<bf16, 1>(a, l.k, st);
    return vec == 2 ? launch_back<f16, 2>(a, l.k, st) : launch_back<f16, 1>(a, l.k, st);
}

}  // namespace c2d
