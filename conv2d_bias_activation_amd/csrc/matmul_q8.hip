// Products of token rows with weights, both as 8-bit integers with a scale for each row (gfx950
// only), and the quantizer that makes such rows.
//
// Packed rows, of activations and weights alike: tiles of 16 rows x 64 values, all value blocks of
// a row tile in a row, then the scales. A tile is 64 records of 16 bytes, record l the values
// 16 (l / 16) .. + 15 of row l % 16: what lane l of a 16x16x64 matrix instruction takes. Rows and
// values past the end are 0. With both operands in this order every load moves whole kilobytes, to
// registers or to LDS, and odd sizes end in zeros that need no test in the loops.
#include <type_traits>
#include <utility>

#include "igemm_common.hpp"
#include "kernels.hpp"
#include "runtime.hpp"
#include "seq_common.hpp"

namespace c2d {

namespace {

typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

constexpr int kRows = 16, kVals = 64, kTileBytes = kRows * kVals;

__host__ __device__ inline int row_tiles(int rows) { return (rows + kRows - 1) / kRows; }
__host__ __device__ inline int val_blocks(int n) { return (n + kVals - 1) / kVals; }
__host__ __device__ inline long long tile_bytes(int rows, int n) {
    return (long long)row_tiles(rows) * val_blocks(n) * kTileBytes;
}
__host__ __device__ inline const float *scales_of(const void *packed, int rows, int n) {
    return reinterpret_cast<const float *>(static_cast<const char *>(packed) + tile_bytes(rows, n));
}
__host__ __device__ inline float *scales_of(void *packed, int rows, int n) {
    return reinterpret_cast<float *>(static_cast<char *>(packed) + tile_bytes(rows, n));
}

// Where 16-value group g of a row stands, in records.
__device__ __forceinline__ long long record_at(int row, int g, int blocks) {
    return ((long long)(row / kRows) * blocks + g / 4) * 64 + g % 4 * 16 + row % kRows;
}

// ---------------------------------------------------------------------------- rows

// The scale of a row whose largest magnitude has the bits `amax`: a 127th of it, at least the
// smallest normal number; NaN for a row with an infinity or a NaN.
__device__ __forceinline__ float row_scale(uint32_t amax) {
    if (amax >= 0x7f800000u) return __builtin_nanf("");
    return fmaxf(__builtin_bit_cast(float, amax) / 127.0f, 0x1p-126f);
}

// x / s rounded to the nearest whole number, ties to even, exactly; r = 1 / s. The product with r
// may end on the wrong side of the border of two codes; the remainder x - q s, which fp32 holds
// exactly, tells. A scale of NaN gives 0.
__device__ __forceinline__ int code_of(float x, float s, float r) {
    float q = rintf(x * r);
    const float d = fmaf(-q, s, x), twice = 2.0f * fabsf(d);
    const int odd = (int)q & 1;
    if (twice > s || (twice == s && odd)) q += __builtin_copysignf(1.0f, d);
    return s == s ? (int)q : 0;
}

// 16 values of a row from k on, zeros from n on; rows need not be aligned.
template <typename T> __device__ __forceinline__ void load16(const T *row, int k, int n, Pack<T, 16> &v) {
    if (k + 16 <= n) {
        __builtin_memcpy(&v, row + k, sizeof v);
    } else {  // all on their way together: the last value stands in for those behind it
#pragma unroll
        for (int e = 0; e < 16; e++) v.v[e] = row[min(k + e, n - 1)];
#pragma unroll
        for (int e = 0; e < 16; e++)
            if (k + e >= n) v.v[e] = from_f32<T>(0.0f);
    }
}

// The largest magnitude of the values so far, as the bits of an fp32 number: those of an infinity
// or a NaN are larger than any finite one's. 16-bit values are compared as they are, two at once.
template <typename T> struct Most {
    u16x2 pair = {0, 0};
    __device__ __forceinline__ void take(const Pack<T, 16> &v) {
        uint32_t w[8];
        __builtin_memcpy(w, &v, sizeof w);
#pragma unroll
        for (int i = 0; i < 8; i++) pair = __builtin_elementwise_max(pair, __builtin_bit_cast(u16x2, w[i] & 0x7fff7fffu));
    }
    __device__ __forceinline__ void take(T v) {
        const uint16_t b = __builtin_bit_cast(uint16_t, v) & 0x7fffu;
        pair[0] = max(pair[0], b);
    }
    __device__ __forceinline__ uint32_t bits() const {
        return __builtin_bit_cast(uint32_t, to_f32(__builtin_bit_cast(T, max(pair[0], pair[1]))));
    }
};
template <> struct Most<float> {
    uint32_t most = 0;
    __device__ __forceinline__ void take(float v) { most = max(most, __builtin_bit_cast(uint32_t, v) & 0x7fffffffu); }
    __device__ __forceinline__ void take(const Pack<float, 16> &v) {
#pragma unroll
        for (int e = 0; e < 16; e++) take(v.v[e]);
    }
    __device__ __forceinline__ uint32_t bits() const { return most; }
};

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
    for (int o = 1; o < 64; o *= 2) v = max(v, (uint32_t)__shfl_xor((int)v, o));
    return v;
}

// 16 codes. Added to 1.5 * 2^23, x r is rounded to a whole number that stands in the last byte of
// the sum; it is the code unless its remainder reaches half a scale, which one of some 10^5 does,
// by r's rounding or in a tie. Only a group with one takes the long way.
template <typename T> __device__ __forceinline__ u32x4 codes16(const Pack<T, 16> &v, float s, float r) {
    constexpr float kShift = 12582912.0f;
    uint32_t b[16];
    float off = 0.0f;
#pragma unroll
    for (int e = 0; e < 16; e++) {
        const float x = to_f32(v.v[e]), t = fmaf(x, r, kShift);
        b[e] = __builtin_bit_cast(uint32_t, t);
        off = fmaxf(off, fabsf(fmaf(kShift - t, s, x)));
    }
    if (!(2.0f * off < s)) {
#pragma unroll
        for (int e = 0; e < 16; e++) b[e] = (uint32_t)code_of(to_f32(v.v[e]), s, r);
    }
    u32x4 out;
#pragma unroll
    for (int i = 0; i < 4; i++) {  // the last bytes of four words
        const uint32_t lo = __builtin_amdgcn_perm(b[4 * i + 1], b[4 * i], 0x0c0c0400u);
        const uint32_t hi = __builtin_amdgcn_perm(b[4 * i + 3], b[4 * i + 2], 0x04000c0cu);
        out[i] = lo | hi;
    }
    return out;
}

// WPR waves a row, so that few rows still make many waves, and ROWS neighbouring rows a workgroup,
// whose 16-byte records make whole runs of 64 or 128 bytes. NR groups of 16 values of a lane stay
// in registers between the maximum and the codes; a longer row is read again. The values behind
// the last whole group go to a lane each. 4096 x 4096 bf16 in 13.2 to 15.5 us (50 MB, 3.2 to 3.8 TB/s, the vector ALU 28 %
// busy with some 14 instructions a value: neither is full, and what bounds it is not established); 37 x 4010 in 4 us, a
// launch and two latencies.
template <typename T, int WPR, int ROWS, int NR>
__global__ __launch_bounds__(64 * WPR * ROWS) void quantize_kernel(const T *x, long long x_row, void *packed, int rows, int n) {
    __shared__ uint32_t s_most[WPR * ROWS];
    constexpr int TR = 64 * WPR;  // threads of a row
    const int lane = threadIdx.x % TR, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int row = blockIdx.x * ROWS + wave / WPR, blocks = val_blocks(n), groups = blocks * 4, full = n / 16, tail = n % 16;
    u32x4 *out = static_cast<u32x4 *>(packed);
    float *scales = scales_of(packed, rows, n);
    const bool real = row < rows;  // the others stand behind the last row in its tile
    const T *p = x + (real ? row : 0) * x_row;
    Pack<T, 16> kept[NR];
    T last = from_f32<T>(0.0f);
    if (real && lane < tail) last = p[full * 16 + lane];
#pragma unroll
    for (int i = 0; i < NR; i++)
        if (real && i * TR + lane < full) __builtin_memcpy(&kept[i], p + (i * TR + lane) * 16, sizeof kept[i]);
    Most<T> most;
    most.take(last);
#pragma unroll
    for (int i = 0; i < NR; i++)
        if (real && i * TR + lane < full) most.take(kept[i]);
    for (int g = NR * TR + lane; real && g < full; g += TR) {
        Pack<T, 16> v;
        __builtin_memcpy(&v, p + g * 16, sizeof v);
        most.take(v);
    }
    uint32_t m = wave_max(most.bits());
    if constexpr (WPR > 1) {
        if (threadIdx.x % 64 == 0) s_most[wave] = m;
        __syncthreads();
        m = 0;
#pragma unroll
        for (int i = 0; i < WPR; i++) m = max(m, s_most[wave / WPR * WPR + i]);
    }
    if (!real) {
        for (int g = lane; g < groups; g += TR) out[record_at(row, g, blocks)] = u32x4{};
        if (lane == 0) scales[row] = 0.0f;
        return;
    }
    const float s = row_scale(m), r = 1.0f / s;
    if (lane == 0) scales[row] = s;
#pragma unroll
    for (int i = 0; i < NR; i++)
        if (i * TR + lane < full) out[record_at(row, i * TR + lane, blocks)] = codes16(kept[i], s, r);
    for (int g = NR * TR + lane; g < full; g += TR) {
        Pack<T, 16> v;
        __builtin_memcpy(&v, p + g * 16, sizeof v);
        out[record_at(row, g, blocks)] = codes16(v, s, r);
    }
    if (tail && lane < 16) reinterpret_cast<int8_t *>(out + record_at(row, full, blocks))[lane] = (int8_t)code_of(to_f32(last), s, r);
    const int behind = full + (tail ? 1 : 0) + lane;
    if (behind < groups) out[record_at(row, behind, blocks)] = u32x4{};
}

// Codes and scales as they come, [rows, n] and [rows], to packed rows and back.
__global__ __launch_bounds__(256) void q8_pack_kernel(const int8_t *codes, const float *scales, void *packed, int rows, int n) {
    const int blocks = val_blocks(n), padded = row_tiles(rows) * kRows;
    const long long records = (long long)padded * blocks * 4;
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < records; i += gridDim.x * 256ll) {
        const int l = i % 64;
        const long long tile = i / 64;
        const int row = (int)(tile / blocks) * kRows + l % 16, k = (int)(tile % blocks) * kVals + l / 16 * 16;
        u32x4 w{};
        if (row < rows) {
            const int8_t *p = codes + (long long)row * n + k;
            if (k + 16 <= n) {
                __builtin_memcpy(&w, p, 16);
            } else {
                for (int e = 0; k + e < n; e++) w[e / 4] |= (uint32_t)(uint8_t)p[e] << 8 * (e % 4);
            }
        }
        static_cast<u32x4 *>(packed)[i] = w;
    }
    float *ps = scales_of(packed, rows, n);
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < padded; i += gridDim.x * 256ll) ps[i] = i < rows ? scales[i] : 0.0f;
}

__global__ __launch_bounds__(256) void q8_unpack_kernel(const void *packed, int8_t *codes, float *scales, int rows, int n) {
    const int blocks = val_blocks(n);
    const long long records = (long long)row_tiles(rows) * kRows * blocks * 4;
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < records; i += gridDim.x * 256ll) {
        const int l = i % 64;
        const long long tile = i / 64;
        const int row = (int)(tile / blocks) * kRows + l % 16, k = (int)(tile % blocks) * kVals + l / 16 * 16;
        if (row >= rows) continue;
        const u32x4 w = static_cast<const u32x4 *>(packed)[i];
        int8_t *p = codes + (long long)row * n + k;
        if (k + 16 <= n) {
            __builtin_memcpy(p, &w, 16);
        } else {
            for (int e = 0; k + e < n; e++) p[e] = (int8_t)(w[e / 4] >> 8 * (e % 4));
        }
    }
    const float *ps = scales_of(packed, rows, n);
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < rows; i += gridDim.x * 256ll) scales[i] = ps[i];
}

// ---------------------------------------------------------------------------- products

// What a product kernel needs, passed by value.
struct Q8Args {
    const u32x4 *x, *w;           // tiles
    const float *sx, *sw;         // scales
    const float *bias, *alpha;    // may be null
    const void *residual;         // may be null
    void *y;
    long long residual_row, y_row;
    int rows, outs, blocks;       // blocks: value blocks of a row
    int act, before;
};

// sum * a * b + bias for the scales a and b. Scales of ordinary sizes are multiplied first; of others the
// smaller one is applied first, so that nothing overflows or loses bits on the way that the
// product itself does not (scales of quantized rows are normal numbers). Every kernel does the same.
__device__ __forceinline__ bool ordinary(float a) { return fabsf(a) >= 0x1p-60f && fabsf(a) <= 0x1p60f; }
__device__ __forceinline__ float affine(int sum, float a, float b, float bias) {
    if (ordinary(a) && ordinary(b)) return fmaf((float)sum, a * b, bias);
    const bool less = fabsf(a) < fabsf(b);
    return (float)sum * (less ? a : b) * (less ? b : a) + bias;
}

// What the epilogue of conv2d_fused does behind the bias.
__device__ __forceinline__ float behind_bias(float v, float alpha, float r, bool has_res, int act, bool before) {
    return epilogue(v, 0.0f, alpha, r, has_res, act, before);
}

// A few rows: a workgroup computes 16 NT outputs of 16 MT rows, straight from memory; its W waves
// take the value blocks in turn and add up in LDS. The weights are read once for 16 MT rows and bound it
// where they come from HBM: 64 x 4010 -> 8192 in 13.0 us, 2.5 TB/s; 8 x 2048 -> 4096 in 3.6 us, which is a launch and
// two latencies.
template <typename T, int NT, int MT, int W>
__global__ __launch_bounds__(64 * W) void q8_few_kernel(const Q8Args a, int nblocks) {
    __shared__ i32x4 s_sum[W][NT * MT][64];
    constexpr int U = 4;  // value blocks on their way together
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int ntiles = row_tiles(a.outs), mtiles = row_tiles(a.rows);
    const int n0 = (int)(blockIdx.x % nblocks) * NT, m0 = (int)(blockIdx.x / nblocks) * MT;
    const u32x4 *w[NT], *x[MT];  // tiles past the last: that again, never stored
#pragma unroll
    for (int n = 0; n < NT; n++) w[n] = a.w + (long long)min(n0 + n, ntiles - 1) * a.blocks * 64 + lane;
#pragma unroll
    for (int m = 0; m < MT; m++) x[m] = a.x + (long long)min(m0 + m, mtiles - 1) * a.blocks * 64 + lane;
    // What this thread's outputs need beside their sums, on its way with the first blocks: value r
    // of lane l of tile (n, m) is row 4 (l / 16) + r, output l % 16.
    constexpr int OUTS = NT * MT * 256, PER = (OUTS + 64 * W - 1) / (64 * W);
    int row[PER], o[PER];
    float sx[PER], sw[PER], bias[PER], alpha[PER], res[PER];
    bool on[PER];
#pragma unroll
    for (int j = 0; j < PER; j++) {
        const int i = threadIdx.x + j * 64 * W, l = i % 64, r = i / 64 % 4, t = i / 256;
        row[j] = (m0 + t % MT) * 16 + l / 16 * 4 + r, o[j] = (n0 + t / MT) * 16 + l % 16;
        on[j] = i < OUTS && row[j] < a.rows && o[j] < a.outs;
        if (!on[j]) continue;
        sx[j] = a.sx[row[j]], sw[j] = a.sw[o[j]];
        bias[j] = a.bias ? a.bias[o[j]] : 0.0f;
        alpha[j] = a.act == CONV2D_ACT_PRELU ? a.alpha[o[j]] : 0.0f;
        res[j] = a.residual ? to_f32(static_cast<const T *>(a.residual)[row[j] * a.residual_row + o[j]]) : 0.0f;
    }
    i32x4 acc[NT][MT] = {};
    for (int k0 = wave; k0 < a.blocks; k0 += U * W) {
        u32x4 wv[U][NT], xv[U][MT];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const bool in = k0 + u * W < a.blocks;
            const int k = in ? k0 + u * W : k0;
#pragma unroll
            for (int n = 0; n < NT; n++) wv[u][n] = w[n][k * 64];
#pragma unroll
            for (int m = 0; m < MT; m++) xv[u][m] = x[m][k * 64];
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            if (k0 + u * W >= a.blocks) break;
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int m = 0; m < MT; m++)
                    acc[n][m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, xv[u][m]),
                                                                      __builtin_bit_cast(i32x4, wv[u][n]), acc[n][m], 0, 0, 0);
        }
    }
#pragma unroll
    for (int n = 0; n < NT; n++)
#pragma unroll
        for (int m = 0; m < MT; m++) s_sum[wave][n * MT + m][lane] = acc[n][m];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < PER; j++) {
        if (!on[j]) continue;
        const int i = threadIdx.x + j * 64 * W, l = i % 64, r = i / 64 % 4, t = i / 256;
        int sum = 0;
#pragma unroll
        for (int v = 0; v < W; v++) sum += s_sum[v][t][l][r];
        const float v = behind_bias(affine(sum, sx[j], sw[j], bias[j]), alpha[j], res[j], a.residual != nullptr, a.act, a.before != 0);
        static_cast<T *>(a.y)[row[j] * a.y_row + o[j]] = round_fp32<T>(v);
    }
}

constexpr int kDirectWaves = 8, kDirectInputs = kDirectWaves * 64 * 16;  // a group of 16 values a thread

// Up to R rows that are not quantized yet, of at most kDirectInputs values: each workgroup does
// that for itself, from L2, which costs less than a launch before this one, and keeps the codes
// in LDS. The rest is as in q8_few_kernel; the first weights are on their way meanwhile. 1 x 2048 -> 4096
// in 3.9 us; with a launch of its own for the rows the call took 11.0 us, not 7.3.
template <typename T, int R, int NT>
__global__ __launch_bounds__(64 * kDirectWaves) void q8_direct_kernel(const Q8Args a, const T *xs, long long x_row, int inputs) {
    constexpr int W = kDirectWaves, U = 4, OUTS = NT * 16 * R;
    static_assert(OUTS <= 64 * W, "an output a thread");
    __shared__ u32x4 s_codes[R][W * 64];
    __shared__ uint32_t s_most[R][W];
    __shared__ int s_sum[W][NT][R][16];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int n0 = blockIdx.x * NT, ntiles = row_tiles(a.outs);
    const u32x4 *w[NT];
#pragma unroll
    for (int n = 0; n < NT; n++) w[n] = a.w + (long long)min(n0 + n, ntiles - 1) * a.blocks * 64 + lane;
    Pack<T, 16> v[R];
    const int k = threadIdx.x * 16;
#pragma unroll
    for (int r = 0; r < R; r++) {
        v[r] = Pack<T, 16>{};
        if (r < a.rows && k < inputs) load16(xs + r * x_row, k, inputs, v[r]);
    }
    u32x4 wv[U][NT];
    auto fetch = [&](int k0) {
#pragma unroll
        for (int u = 0; u < U; u++)
#pragma unroll
            for (int n = 0; n < NT; n++) wv[u][n] = w[n][min(k0 + u * W, a.blocks - 1) * 64];
    };
    fetch(wave);
    // the thread's output, and what it needs beside the sum
    const int row = threadIdx.x / (16 * NT), o = n0 * 16 + threadIdx.x % (16 * NT);
    const bool on = threadIdx.x < OUTS && row < a.rows && o < a.outs;
    float sw = 0.0f, bias = 0.0f, alpha = 0.0f, res = 0.0f;
    if (on) {
        sw = a.sw[o];
        if (a.bias) bias = a.bias[o];
        if (a.act == CONV2D_ACT_PRELU) alpha = a.alpha[o];
        if (a.residual) res = to_f32(static_cast<const T *>(a.residual)[row * a.residual_row + o]);
    }
#pragma unroll
    for (int r = 0; r < R; r++) {
        Most<T> most;
        most.take(v[r]);
        const uint32_t m = wave_max(most.bits());
        if (lane == 0) s_most[r][wave] = m;
    }
    __syncthreads();
    float sx = 0.0f;
#pragma unroll
    for (int r = 0; r < R; r++) {
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < W; i++) most = max(most, s_most[r][i]);
        const float s = row_scale(most);
        if (row == r) sx = s;
        s_codes[r][threadIdx.x] = codes16(v[r], s, 1.0f / s);
    }
    __syncthreads();
    i32x4 acc[NT] = {};
    for (int k0 = wave; k0 < a.blocks; k0 += U * W) {
        if (k0 != wave) fetch(k0);
#pragma unroll
        for (int u = 0; u < U; u++) {
            if (k0 + u * W >= a.blocks) break;
            const u32x4 x = lane % 16 < R ? s_codes[lane % 16 < R ? lane % 16 : 0][(k0 + u * W) * 4 + lane / 16] : u32x4{};
#pragma unroll
            for (int n = 0; n < NT; n++)
                acc[n] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, x), __builtin_bit_cast(i32x4, wv[u][n]),
                                                               acc[n], 0, 0, 0);
        }
    }
    if (lane < 16) {  // rows 0 to 3 of the 16
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int r = 0; r < R; r++) s_sum[wave][n][r][lane] = acc[n][r];
    }
    __syncthreads();
    if (!on) return;
    int sum = 0;
#pragma unroll
    for (int i = 0; i < W; i++) sum += s_sum[i][threadIdx.x / 16 % NT][row][threadIdx.x % 16];
    const float f = behind_bias(affine(sum, sx, sw, bias), alpha, res, a.residual != nullptr, a.act, a.before != 0);
    static_cast<T *>(a.y)[row * a.y_row + o] = round_fp32<T>(f);
}

template <int N> __device__ __forceinline__ void q8_wait_vmcnt() {
    static_assert(N >= 0 && N < 64, "vmcnt has 6 bits");
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}

// Workgroup barrier behind this wave's LDS accesses.
__device__ __forceinline__ void q8_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// What this wave wrote to LDS is there for its other lanes.
__device__ __forceinline__ void q8_wave_lds() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);
    __builtin_amdgcn_wave_barrier();
    asm volatile("" ::: "memory");
}

// Many rows: BM rows x BN outputs a workgroup, WM x WN waves of 32x32 blocks, steps of one value
// block through a ring of NS stages in LDS, loaded directly from memory.
// 4096 x 4096 -> 16384 in 248 to 284 us (2100 TOP/s at 262), 8192 x 8192 -> 8192 in 457 (2400): under such a load the clock
// falls to 1.7 GHz, and the matrix units are 59 to 66 % busy at it. What they miss is the start of a
// workgroup and the end of its tile, some 11 us of 130 at 4096 inputs (one workgroup a CU: its
// registers hold 256 x 256 sums). 333 x 2048 -> 4096 in 9.9 us on 64 x 64 tiles: 5 us are the launch and the first and
// last steps, the rest the 256 KB that each workgroup brings into LDS.
template <typename T, int BM, int BN, int WM, int WN, int NS, int KS>
__global__ __launch_bounds__(64 * WM * WN) void q8_tile_kernel(const Q8Args a, int tiles_m, int tiles_n) {
    constexpr int NW = WM * WN, FM = BM / (32 * WM), FN = BN / (32 * WN);
    constexpr int BLOCK = (BM + BN) * kVals, STAGE = KS * BLOCK, CH = (BM + BN) / 16, LPW = CH / NW;
    static_assert(CH % NW == 0 && NS >= 3, "whole loads a wave");
    constexpr int LD = 32 * FN + 4;  // stride of the epilogue's rows, in sums
    constexpr int SLICES = NW * 32 * LD * 4;
    __shared__ float s_sx[BM];
    __shared__ __attribute__((aligned(1024))) char lds[NS * STAGE > SLICES ? NS * STAGE : SLICES];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int wm = wave % WM, wn = wave / WM;
    const int g = xcd_remap(blockIdx.x, tiles_m * tiles_n);
    const int tm = g % tiles_m, tn = g / tiles_m;
    const int mtiles = row_tiles(a.rows), ntiles = row_tiles(a.outs), KB = a.blocks;

    // This wave's loads of a stage: row tile `d * NW + wave` of the rows, then of the weights, as
    // buffers of the row tile's value blocks.
    i32x4 src[LPW];
#pragma unroll
    for (int d = 0; d < LPW; d++) {
        const int ch = d * NW + wave;
        const bool isx = ch < BM / 16;
        const int t = isx ? min(tm * (BM / 16) + ch, mtiles - 1) : min(tn * (BN / 16) + ch - BM / 16, ntiles - 1);
        src[d] = rsrc_words(reinterpret_cast<const char *>(isx ? a.x : a.w) + (long long)t * KB * kTileBytes, KB * kTileBytes);
#pragma unroll
        for (int i = 0; i < 4; i++) src[d][i] = __builtin_amdgcn_readfirstlane(src[d][i]);
    }
    // What the epilogue needs beside the sums, on its way before the first stage: VE neighbouring
    // outputs a lane, LPR lanes a row, RP rows a pass.
    constexpr int VE = 16 / sizeof(T), LPR = 32 * FN / VE, RP = 64 / LPR;
    const int o0 = tn * BN + wn * 32 * FN + lane % LPR * VE;
    float sw[VE], bias[VE], alpha[VE];
#pragma unroll
    for (int e = 0; e < VE; e++) {
        const int o = min(o0 + e, a.outs - 1);
        sw[e] = a.sw[o];
        bias[e] = a.bias ? a.bias[o] : 0.0f;
        alpha[e] = a.act == CONV2D_ACT_PRELU ? a.alpha[o] : 0.0f;
    }
    for (int i = threadIdx.x; i < BM; i += 64 * NW) s_sx[i] = a.sx[min(tm * BM + i, a.rows - 1)];

    const uint32_t base = lds_addr(lds);
    auto issue = [&](int kb, int d0, int d1) {
#pragma unroll
        for (int s = 0; s < KS; s++)  // blocks past the last are past the buffer: zeros
#pragma unroll
            for (int d = d0; d < d1; d++)
                dma_b128(src[d], (uint32_t)((kb * KS + s) * kTileBytes + lane * 16),
                         base + kb % NS * STAGE + s * BLOCK + (d * NW + wave) * kTileBytes);
    };

    i32x16 acc[FM][FN] = {};
    const int at = (lane % 32 / 16) * kTileBytes + lane / 32 * 256 + lane % 16 * 16;
    if constexpr (KS == 1) {
#pragma unroll
        for (int s = 0; s < NS - 1; s++) issue(s, 0, LPW);
        i32x4 xf[2][FM], wf[2][FN];
        // Operand f of half h of step kb from LDS: the weights', then the rows'.
        auto read = [&](int kb, int h, int f0, int f1) {
            const char *st = lds + kb % NS * STAGE + h * 512 + at;
#pragma unroll
            for (int f = f0; f < f1; f++) {
                if (f < FN)
                    wf[h][f] = *reinterpret_cast<const i32x4 *>(st + BM * kVals + (wn * FN + f) * 2 * kTileBytes);
                else if (f < FN + FM)
                    xf[h][f - FN] = *reinterpret_cast<const i32x4 *>(st + (wm * FM + f - FN) * 2 * kTileBytes);
            }
        };
        // The products of half h of step kb, with the operands of the next half read, and the step
        // NS - 1 ahead loaded, between them: the order is kept as written, as the compiler would read
        // the operands last and wait for them.
        constexpr int RG = (FM + FN + FM - 1) / FM, DG = (LPW + FM - 1) / FM;
        auto half = [&](int kb, auto hc) {
            constexpr int h = decltype(hc)::value;
#pragma unroll
            for (int m = 0; m < FM; m++) {
                if constexpr (h == 1) issue(kb + NS - 1, m * DG, min((m + 1) * DG, LPW));
                // all reads in the first half of the products
                read(kb + h, 1 - h, m * 2 * RG, (m + 1) * 2 * RG);
#pragma unroll
                for (int n = 0; n < FN; n++) acc[m][n] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[h][n], xf[h][m], acc[m][n], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        // The barrier that hands out the next stage stands between a step's halves.
        q8_wait_vmcnt<(NS - 2) * LPW>();
        q8_barrier();
        read(0, 0, 0, FM + FN);
        for (int kb = 0; kb < KB; kb++) {
            half(kb, std::integral_constant<int, 0>{});
            q8_wait_vmcnt<(NS - 3) * LPW>();
            q8_barrier();
            half(kb, std::integral_constant<int, 1>{});
        }
    } else {
        // Small tiles: the operands of a whole step are read while those of the step before are
        // multiplied, so that a step waits for one barrier and for no read. A stage is free for
        // its next load once it has been read, at the barrier of the step that multiplies it.
        constexpr int H = 2 * KS;
        const int steps = (KB + KS - 1) / KS;
        i32x4 xf[2][H][FM], wf[2][H][FN];
#pragma unroll
        for (int s = 0; s < NS; s++) issue(s, 0, LPW);
        auto read = [&](int kb, auto pc) {
            constexpr int p = decltype(pc)::value;
            const char *st = lds + kb % NS * STAGE + at;
#pragma unroll
            for (int h = 0; h < H; h++) {
#pragma unroll
                for (int n = 0; n < FN; n++)
                    wf[p][h][n] = *reinterpret_cast<const i32x4 *>(st + h / 2 * BLOCK + h % 2 * 512 + BM * kVals + (wn * FN + n) * 2 * kTileBytes);
#pragma unroll
                for (int m = 0; m < FM; m++)
                    xf[p][h][m] = *reinterpret_cast<const i32x4 *>(st + h / 2 * BLOCK + h % 2 * 512 + (wm * FM + m) * 2 * kTileBytes);
            }
        };
        auto multiply = [&](auto pc) {
            constexpr int p = decltype(pc)::value;
#pragma unroll
            for (int h = 0; h < H; h++)
#pragma unroll
                for (int m = 0; m < FM; m++)
#pragma unroll
                    for (int n = 0; n < FN; n++)
                        acc[m][n] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[p][h][n], xf[p][h][m], acc[m][n], 0, 0, 0);
        };
        const std::integral_constant<int, 0> even;
        const std::integral_constant<int, 1> odd;
        q8_wait_vmcnt<(NS - 1) * KS * LPW>();
        q8_barrier();
        read(0, even);
        for (int kb = 0; kb < steps; kb += 2) {  // a step past the last multiplies zeros
            q8_wait_vmcnt<(NS - 2) * KS * LPW>();
            q8_barrier();
            issue(kb + NS, 0, LPW);
            read(kb + 1, odd);
            __builtin_amdgcn_sched_barrier(0);
            multiply(even);
            __builtin_amdgcn_sched_barrier(0);
            q8_wait_vmcnt<(NS - 2) * KS * LPW>();
            q8_barrier();
            issue(kb + 1 + NS, 0, LPW);
            read(kb + 2, even);
            __builtin_amdgcn_sched_barrier(0);
            multiply(odd);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    q8_wait_vmcnt<0>();
    q8_barrier();

    // 32 rows of the wave's outputs at a time through LDS, so that a lane finishes neighbouring
    // outputs of a row. Value i of lane l of a block: output 8 (i / 4) + 4 (l / 32) +
    // i % 4, row l % 32.
    int *slice = reinterpret_cast<int *>(lds) + wave * 32 * LD;
    const T *res = static_cast<const T *>(a.residual);
    T *y = static_cast<T *>(a.y);
    const bool whole = o0 + VE <= a.outs;  // rows need not be aligned
    bool plain = true;
#pragma unroll
    for (int e = 0; e < VE; e++) plain &= ordinary(sw[e]);
    auto finish_rows = [&](int row0, auto act) {
#pragma unroll 2
        for (int p = 0; p < 32 / RP; p++) {
            const int row = row0 + p * RP + lane / LPR;
            if (row >= a.rows || o0 >= a.outs) continue;
            const float sx = s_sx[row - tm * BM];
            Pack<T, VE> r{}, out;
            if (res) {
                if (whole) {
                    __builtin_memcpy(&r, res + row * a.residual_row + o0, sizeof r);
                } else {
#pragma unroll
                    for (int e = 0; e < VE; e++)
                        if (o0 + e < a.outs) r.v[e] = res[row * a.residual_row + o0 + e];
                }
            }
            const int *q = slice + (p * RP + lane / LPR) * LD + lane % LPR * VE;
            float v[VE];
            if (plain && ordinary(sx)) {
#pragma unroll
                for (int e = 0; e < VE; e++) v[e] = fmaf((float)q[e], sx * sw[e], bias[e]);
            } else {
#pragma unroll
                for (int e = 0; e < VE; e++) v[e] = affine(q[e], sx, sw[e], bias[e]);
            }
#pragma unroll
            for (int e = 0; e < VE; e++) {
                const float add = to_f32(r.v[e]);
                if (res && a.before) v[e] += add;
                v[e] = activate_c<decltype(act)::value>(v[e], alpha[e]);
                if (res && !a.before) v[e] += add;
                out.v[e] = round_fp32<T>(v[e]);
            }
            if (whole) {
                __builtin_memcpy(y + row * a.y_row + o0, &out, sizeof out);
            } else {
#pragma unroll
                for (int e = 0; e < VE; e++)
                    if (o0 + e < a.outs) y[row * a.y_row + o0 + e] = out.v[e];
            }
        }
    };
    auto part = [&](auto mc) {
        constexpr int m = decltype(mc)::value;
#pragma unroll
        for (int n = 0; n < FN; n++)
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<i32x4 *>(slice + lane % 32 * LD + n * 32 + i * 2 + lane / 32 * 4) =
                    i32x4{acc[m][n][i], acc[m][n][i + 1], acc[m][n][i + 2], acc[m][n][i + 3]};
        q8_wave_lds();
        const int row0 = tm * BM + (wm * FM + m) * 32;
        switch (a.act) {
        case CONV2D_ACT_RELU: finish_rows(row0, std::integral_constant<int, CONV2D_ACT_RELU>{}); break;
        case CONV2D_ACT_SILU: finish_rows(row0, std::integral_constant<int, CONV2D_ACT_SILU>{}); break;
        case CONV2D_ACT_PRELU: finish_rows(row0, std::integral_constant<int, CONV2D_ACT_PRELU>{}); break;
        default: finish_rows(row0, std::integral_constant<int, CONV2D_ACT_NONE>{});
        }
        q8_wave_lds();
    };
    // one after the other by number: the sums stay in registers
    [&]<int... M>(std::integer_sequence<int, M...>) { (part(std::integral_constant<int, M>{}), ...); }(std::make_integer_sequence<int, FM>{});
}

template <typename T, int NT, int MT, int W> hipError_t few(const Q8Args &a, hipStream_t st) {
    const int nblocks = (row_tiles(a.outs) + NT - 1) / NT;
    const long long mblocks = (row_tiles(a.rows) + MT - 1) / MT;
    return launch_blocks(q8_few_kernel<T, NT, MT, W>, nblocks * mblocks, 64 * W, st, a, nblocks);
}

template <typename T, int BM, int BN, int WM, int WN, int NS, int KS> hipError_t tiled(const Q8Args &a, hipStream_t st) {
    const long long tm = (a.rows + BM - 1ll) / BM, tn = (a.outs + BN - 1ll) / BN;
    if (tm * tn > 0x7fffffff) return hipErrorInvalidConfiguration;
    return launch_blocks(q8_tile_kernel<T, BM, BN, WM, WN, NS, KS>, tm * tn, 64 * WM * WN, st, a, (int)tm, (int)tn);
}

template <typename T, int R, int NT> hipError_t direct(const Q8Args &a, const void *x, long long x_row, int inputs, hipStream_t st) {
    return launch_blocks(q8_direct_kernel<T, R, NT>, (row_tiles(a.outs) + NT - 1) / NT, 64 * kDirectWaves, st, a,
                         static_cast<const T *>(x), x_row, inputs);
}

// Products of the rows of a that the call quantizes, without a launch for that.
template <typename T> hipError_t launch_direct(const Q8Args &p, const matmul_q8_args &a, hipStream_t st) {
    if (a.rows == 1)
        return row_tiles(a.out_features) >= 1024 ? direct<T, 1, 2>(p, a.x, a.x_row, a.in_features, st)
                                                 : direct<T, 1, 1>(p, a.x, a.x_row, a.in_features, st);
    return row_tiles(a.out_features) >= 1024 ? direct<T, 4, 2>(p, a.x, a.x_row, a.in_features, st)
                                             : direct<T, 4, 1>(p, a.x, a.x_row, a.in_features, st);
}

// Which kernel and tile. A few-rows kernel, whose operands come straight from memory, for rows and outputs that make at most two
// of its workgroups a CU; from there on tiles, through LDS. Times in us, weights not in the caches, few-rows kernels by their
// NT, MT, W, tiles by rows x outputs; the last column has the workgroups of 2,2,8:
//   rows x inputs -> outputs    1,1,8  2,1,8  2,2,8  64x64 128x128
//       8 x  2048 ->  4096        3.6    4.2    4.7    6.5   10.0
//       8 x  8192 -> 16384       27.1   23.5   24.3   25.1   47.4
//      32 x  2048 ->  4096        4.0    4.2    5.0    7.1   11.6
//      33 x  2048 ->  8192                      7.2    7.9            512
//      64 x  4010 ->  8192                     13.0   14.4            512
//      20 x  4010 -> 16384                     15.2   16.4            512
//     128 x  2048 ->  4096        7.6    6.4    6.2    7.2   14.2     512
//      90 x  4010 ->  6000                     13.6   12.7            564
//      33 x  2048 -> 10007                     10.1    8.7            626
//      37 x  4010 -> 10007                     16.5   14.2            626
//      48 x  8192 -> 10007                     28.8   24.0            626
//      33 x  4010 -> 13000                     20.0   15.1            814
//     256 x  2048 ->  4096       12.9   10.4    9.0    8.2   14.4    1024
// Among the tiles the one is taken whose workgroups, spread over the 256 CUs, take the least time
// by what a step of 64 inputs of one takes where the card is full: 64x64 0.11 us, 128x128 0.30,
// 128x256 0.55, 256x256 0.87. Larger tiles read each operand less often; smaller ones
// make more workgroups. (2048 x 4096 -> 4096: 128x128 41.3 us, 128x256 40.5, 256x256 53.7; 1024 x 2048
// -> 4096: 64x64 21, 128x128 17.5; 4096 x 4096 -> 16384: 128x128 362, 128x256 334, 256x256
// 262.) 64x64 tiles with three stages of the ring, for three workgroups a CU, where there are more of them than CUs,
// else with four (256 x 2048 -> 4096 8.2 and 7.8 us, 333 x 2048 -> 4096 9.9 and 10.4, 1000 x 2048 -> 2048 10.5 and 11.0).
template <typename T> hipError_t launch_product(const Q8Args &a, hipStream_t st) {
    const long long n = row_tiles(a.outs), m = row_tiles(a.rows);
    if (m == 1) return n >= 1024 ? few<T, 2, 1, 8>(a, st) : few<T, 1, 1, 8>(a, st);
    if (n * m <= 512) return few<T, 1, 1, 8>(a, st);
    if ((n + 1) / 2 * ((m + 1) / 2) <= 512) return few<T, 2, 2, 8>(a, st);
    const struct { int bm, bn, step; } tiles[] = {{64, 64, 11}, {128, 128, 30}, {128, 256, 55}, {256, 256, 87}};
    int best = 0;
    long long least = 0, groups = 0;
    for (int i = 0; i < 4; i++) {
        const long long blocks = ((a.rows + tiles[i].bm - 1ll) / tiles[i].bm) * ((a.outs + tiles[i].bn - 1ll) / tiles[i].bn);
        const long long time = (blocks + 255) / 256 * tiles[i].step;
        if (i == 0 || time < least) best = i, least = time, groups = blocks;
    }
    switch (best) {
    case 0: return groups > 256 ? tiled<T, 64, 64, 2, 2, 3, 2>(a, st) : tiled<T, 64, 64, 2, 2, 4, 2>(a, st);
    case 1: return tiled<T, 128, 128, 2, 2, 4, 1>(a, st);
    case 2: return tiled<T, 128, 256, 2, 4, 6, 1>(a, st);
    default: return tiled<T, 256, 256, 2, 4, 4, 1>(a, st);
    }
}

template <typename T> hipError_t quantize(const void *x, long long x_row, void *packed, int rows, int n, hipStream_t st) {
    const int tiles = row_tiles(rows);
    const T *p = static_cast<const T *>(x);
    if (n <= 2048) return launch_blocks(quantize_kernel<T, 1, 8, 2>, tiles * 2, 512, st, p, x_row, packed, rows, n);
    return launch_blocks(quantize_kernel<T, 4, 4, 2>, tiles * 4ll, 1024, st, p, x_row, packed, rows, n);
}

}  // namespace

size_t q8_bytes(int rows, int in_features) { return (size_t)tile_bytes(rows, in_features) + (size_t)row_tiles(rows) * kRows * 4; }

hipError_t launch_quantize_rows(const quantize_rows_args &a, hipStream_t st) {
    if (a.dtype == CONV2D_DTYPE_F32) return quantize<float>(a.x, a.x_row, a.packed, a.rows, a.in_features, st);
    if (a.dtype == CONV2D_DTYPE_BF16) return quantize<bf16>(a.x, a.x_row, a.packed, a.rows, a.in_features, st);
    return quantize<f16>(a.x, a.x_row, a.packed, a.rows, a.in_features, st);
}

hipError_t launch_q8_pack(const void *codes, const float *scales, void *packed, int rows, int in_features, hipStream_t st) {
    const long long blocks = tile_bytes(rows, in_features) / 16 / 256 + 1;
    return launch_kernel(q8_pack_kernel, dim3((unsigned)(blocks < 8192 ? blocks : 8192)), dim3(256), 0, st,
                         static_cast<const int8_t *>(codes), scales, packed, rows, in_features);
}

hipError_t launch_q8_unpack(const void *packed, void *codes, float *scales, int rows, int in_features, hipStream_t st) {
    const long long blocks = tile_bytes(rows, in_features) / 16 / 256 + 1;
    return launch_kernel(q8_unpack_kernel, dim3((unsigned)(blocks < 8192 ? blocks : 8192)), dim3(256), 0, st, packed,
                         static_cast<int8_t *>(codes), scales, rows, in_features);
}

bool q8_in_one(const matmul_q8_args &a) { return a.x && a.rows <= 4 && a.in_features <= kDirectInputs; }

hipError_t launch_matmul_q8(const matmul_q8_args &a, void *ws, hipStream_t st) {
    const bool one = q8_in_one(a);
    const void *x = a.x_packed;
    if (!x && !one) {
        const quantize_rows_args q{a.x, ws, a.x_row, a.rows, a.in_features, a.dtype};
        const hipError_t e = launch_quantize_rows(q, st);
        if (e != hipSuccess) return e;
        x = ws;
    }
    const Q8Args p{static_cast<const u32x4 *>(x), static_cast<const u32x4 *>(a.weights),
                   one ? nullptr : scales_of(x, a.rows, a.in_features), scales_of(a.weights, a.out_features, a.in_features),
                   a.bias, a.alpha, a.residual, a.y, a.residual_row, a.y_row, a.rows, a.out_features,
                   val_blocks(a.in_features), a.act & 0xff, (a.act & CONV2D_RES_BEFORE_ACT) != 0};
    switch (a.dtype) {
    case CONV2D_DTYPE_F32:
        return one ? launch_direct<float>(p, a, st) : launch_product<float>(p, st);
    case CONV2D_DTYPE_BF16:
        return one ? launch_direct<bf16>(p, a, st) : launch_product<bf16>(p, st);
    default:
        return one ? launch_direct<f16>(p, a, st) : launch_product<f16>(p, st);
    }
}

}  // namespace c2d
