// Short causal depthwise convolution over channel-last token rows: bias, activation and the
// carried state (the last width - 1 inputs) in one pass.
//
// Two to four products a value against four to eight bytes moved: bound by HBM. A thread owns
// one 16-byte vector of channels and walks kRun tokens of one sequence, the last width - 1
// inputs in registers, so each input is read once but for the width - 1 rows before a run.
#include "kernels.hpp"
#include "seq_common.hpp"

namespace c2d {

namespace {

constexpr int kBlock = 256;

template <int VEC> __device__ __forceinline__ void activate_all(int act, float *v, const float *alpha) {
    if (act == CONV2D_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < VEC; i++) v[i] = activate_c<CONV2D_ACT_SILU>(v[i], 0.0f);
    } else if (act != CONV2D_ACT_NONE) {
#pragma unroll
        for (int i = 0; i < VEC; i++) v[i] = activate(act, v[i], alpha[i]);
    }
}

template <typename T, int VEC, int W> struct ConvWeights {
    float w[W][VEC], bias[VEC], alpha[VEC];

    __device__ __forceinline__ void load(const causal_conv1d_args &a, int c) {
        const T *wp = static_cast<const T *>(a.w) + (long long)c * W;
        Pack<T, VEC> raw[W];  // [VEC][W] values
#pragma unroll
        for (int j = 0; j < W; j++) raw[j] = load_pack<T, VEC>(wp + j * VEC);
#pragma unroll
        for (int i = 0; i < VEC; i++)
#pragma unroll
            for (int j = 0; j < W; j++) w[j][i] = to_f32(raw[(i * W + j) / VEC].v[(i * W + j) % VEC]);
#pragma unroll
        for (int i = 0; i < VEC; i++) {
            bias[i] = a.bias ? a.bias[c + i] : 0.0f;
            alpha[i] = a.act == CONV2D_ACT_PRELU ? a.alpha[c + i] : 0.0f;
        }
    }

    // y of the token whose input is `now`; `past` holds the W - 1 before it, the oldest first,
    // and moves on by one.
    __device__ __forceinline__ Pack<T, VEC> step(int act, Pack<T, VEC> *past, const Pack<T, VEC> &now) const {
        float v[VEC];
#pragma unroll
        for (int i = 0; i < VEC; i++) {
            v[i] = bias[i];
#pragma unroll
            for (int j = 0; j < W - 1; j++) v[i] = fmaf(w[j][i], to_f32(past[j].v[i]), v[i]);
            v[i] = fmaf(w[W - 1][i], to_f32(now.v[i]), v[i]);
        }
        activate_all<VEC>(act, v, alpha);
        Pack<T, VEC> y;
#pragma unroll
        for (int i = 0; i < VEC; i++) y.v[i] = round_fp32<T>(v[i]);
#pragma unroll
        for (int j = 0; j + 1 < W - 1; j++) past[j] = past[j + 1];
        past[W - 2] = now;
        return y;
    }
};

// Block: tx threads along the channels, kBlock / tx runs. The first run of a sequence is the
// only one that reads its state, and rewrites it from the sequence's last inputs when its own
// outputs are done, so that the state may be updated in place.
template <typename T, int VEC, int W, int kRun>
__global__ __launch_bounds__(kBlock) void causal_conv_kernel(const causal_conv1d_args a, int tx, int cblocks, int items,
                                                             int runs) {
    constexpr int kBatch = kRun < 8 ? kRun : 8;  // loads a thread has in flight
    // long runs: neighbouring runs on one XCD, whose L2 then holds the rows that both read
    const int block = kRun == 32 ? xcd_remap(blockIdx.x, gridDim.x) : blockIdx.x;
    const int cb = block % cblocks;
    const int item = __builtin_amdgcn_readfirstlane((block / cblocks) * (kBlock / tx) + (int)threadIdx.x / tx);
    const int c = (cb * tx + (int)threadIdx.x % tx) * VEC;
    if (item >= items || c >= a.channels) return;

    SeqRun r;
    const T *x = static_cast<const T *>(a.x);
    T *y = static_cast<T *>(a.y);
    if (a.offsets) {
        if (!find_run(a.offsets, a.nseq, (int)a.tokens, kRun, item, &r)) return;
        x += (long long)r.start * a.x_token;
        y += (long long)r.start * a.y_token;
    } else {
        r.seq = item / runs;
        r.first = (item - r.seq * runs) * kRun;
        r.len = (int)a.tokens;
        x += (long long)r.seq * a.x_batch;
        y += (long long)r.seq * a.y_batch;
    }
    x += c;
    y += c;
    const int row = state_row(a.state, a.slots, r.seq, a.state_rows);
    T *state = row < 0 ? nullptr : static_cast<T *>(a.state) + (long long)row * (W - 1) * a.channels + c;

    Pack<T, VEC> past[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; j++) {
        const int t = r.first - (W - 1) + j;
        past[j] = Pack<T, VEC>{};
        if (t >= 0)
            past[j] = load_pack<T, VEC>(x + (long long)t * a.x_token);
        else if (state && !a.fresh)
            past[j] = load_pack<T, VEC>(state + (long long)(W - 1 + t) * a.channels);
    }
    // The first run of a sequence leaves the state: entry j is the input W - 1 - j places before
    // the sequence's end, an old entry further on (j + len) where the sequence is shorter
    // than that.
    Pack<T, VEC> kept[W - 1];
    if (r.first == 0 && state) {
#pragma unroll
        for (int j = 0; j < W - 1; j++) {
            const int t = r.len - (W - 1) + j;
            kept[j] = Pack<T, VEC>{};
            if (t >= 0)
                kept[j] = load_pack<T, VEC>(x + (long long)t * a.x_token);
            else if (!a.fresh)
                kept[j] = load_pack<T, VEC>(state + (long long)(W - 1 + t) * a.channels);
        }
    }
    ConvWeights<T, VEC, W> k;
    k.load(a, c);

    const int end = r.len < r.first + kRun ? r.len : r.first + kRun;
    for (int t0 = r.first; t0 < end; t0 += kBatch) {
        Pack<T, VEC> now[kBatch];
        if (t0 + kBatch <= end) {
#pragma unroll
            for (int i = 0; i < kBatch; i++) now[i] = load_pack<T, VEC>(x + (long long)(t0 + i) * a.x_token);
#pragma unroll
            for (int i = 0; i < kBatch; i++)
                store_pack<T, VEC>(y + (long long)(t0 + i) * a.y_token, k.step(a.act, past, now[i]));
        } else {
#pragma unroll
            for (int i = 0; i < kBatch; i++)
                if (t0 + i < end) now[i] = load_pack<T, VEC>(x + (long long)(t0 + i) * a.x_token);
#pragma unroll
            for (int i = 0; i < kBatch; i++)
                if (t0 + i < end)
                    store_pack<T, VEC>(y + (long long)(t0 + i) * a.y_token, k.step(a.act, past, now[i]));
        }
    }

    if (r.first == 0 && state) {
#pragma unroll
        for (int j = 0; j < W - 1; j++) store_pack<T, VEC>(state + (long long)j * a.channels, kept[j]);
    }
}

// One token of each sequence: a thread reads its channels' state, writes it moved on by one
// and y. Bound by the state's bytes, and by the launch for few rows (1 x 2048, bf16: 4.0 us of
// kernel; 384 x 4096, f16, width 3: 7.9 us, 2.4 TB/s, less than the host takes for a call).
template <typename T, int VEC, int W>
__global__ __launch_bounds__(kBlock) void causal_conv_step_kernel(const causal_conv1d_args a, int cblocks) {
    const int cb = blockIdx.x % cblocks, seq = blockIdx.x / cblocks;
    const int c = (cb * kBlock + (int)threadIdx.x) * VEC;
    if (c >= a.channels) return;
    const int row = state_row(a.state, a.slots, seq, a.state_rows);
    T *state = row < 0 ? nullptr : static_cast<T *>(a.state) + (long long)row * (W - 1) * a.channels + c;
    Pack<T, VEC> past[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; j++) {
        past[j] = Pack<T, VEC>{};
        if (state && !a.fresh) past[j] = load_pack<T, VEC>(state + (long long)j * a.channels);
    }
    const Pack<T, VEC> now = load_pack<T, VEC>(static_cast<const T *>(a.x) + (long long)seq * a.x_token + c);
    ConvWeights<T, VEC, W> k;
    k.load(a, c);
    store_pack<T, VEC>(static_cast<T *>(a.y) + (long long)seq * a.y_token + c, k.step(a.act, past, now));
    if (state) {
#pragma unroll
        for (int j = 0; j < W - 1; j++) store_pack<T, VEC>(state + (long long)j * a.channels, past[j]);
    }
}

template <typename T, int VEC, int W, int kRun> hipError_t launch_prompt(const causal_conv1d_args &a, int nvec, hipStream_t st) {
    const int tx = nvec <= 64 ? 64 : nvec <= 128 ? 128 : kBlock;  // whole waves share a run
    const int cblocks = (nvec + tx - 1) / tx;
    const int runs = (int)((a.tokens + kRun - 1) / kRun);
    const long long items = a.offsets ? a.tokens / kRun + a.nseq : (long long)(runs ? runs : 1) * a.nseq;
    const long long blocks = (items + kBlock / tx - 1) / (kBlock / tx) * cblocks;
    return launch_blocks(causal_conv_kernel<T, VEC, W, kRun>, blocks, kBlock, st, a, tx, cblocks, (int)items,
                         runs ? runs : 1);
}

template <typename T, int VEC, int W> hipError_t launch_w(const causal_conv1d_args &a, bool step, hipStream_t st) {
    const int nvec = (a.channels + VEC - 1) / VEC;
    if (step) {
        const int cblocks = (nvec + kBlock - 1) / kBlock;
        return launch_blocks(causal_conv_step_kernel<T, VEC, W>, (long long)cblocks * a.nseq, kBlock, st, a, cblocks);
    }
    // Short runs make many threads and a short walk for each; long ones read fewer rows twice
    // and load the weights less often. Times in us of runs of 4, 16 and 32 (bf16, width 4):
    // 77 x 512: 5.2, 9.1, -; 2000 x 1024: 6.3, 10.2, 15.0; 4000 x 4096: 23.4, 18.6, 23.4;
    // 16384 x 2048: 46.0, 36.4, 39.2; 32768 x 4096: 177, 121, 111 (4.8 TB/s).
    const long long vectors = (a.offsets ? a.tokens : a.tokens * a.nseq) * nvec;
    if (vectors < 600000) return launch_prompt<T, VEC, W, 4>(a, nvec, st);
    if (vectors < 8000000) return launch_prompt<T, VEC, W, 16>(a, nvec, st);
    return launch_prompt<T, VEC, W, 32>(a, nvec, st);
}

template <typename T> hipError_t launch_t(const causal_conv1d_args &a, bool vec, bool step, hipStream_t st) {
    constexpr int V = 16 / (int)sizeof(T);
    switch (a.width) {
    case 2:
        return vec ? launch_w<T, V, 2>(a, step, st) : launch_w<T, 1, 2>(a, step, st);
    case 3:
        return vec ? launch_w<T, V, 3>(a, step, st) : launch_w<T, 1, 3>(a, step, st);
    default:
        return vec ? launch_w<T, V, 4>(a, step, st) : launch_w<T, 1, 4>(a, step, st);
    }
}

}  // namespace

hipError_t launch_causal_conv(const causal_conv1d_args &a, bool vec, bool step, hipStream_t st) {
    switch (a.dtype) {
    case CONV2D_DTYPE_F32:
        return launch_t<float>(a, vec, step, st);
    case CONV2D_DTYPE_BF16:
        return launch_t<bf16>(a, vec, step, st);
    default:
        return launch_t<f16>(a, vec, step, st);
    }
}

}  // namespace c2d
