// Products of token rows with weights, both as 8-bit integers with a scale for each row (gfx950
// only), and the quantizer that makes such rows.
//
// Packed rows, of activations and weights alike: tiles of 16 rows x 64 values, all value blocks of
// a row tile in a row, then the scales. A tile is 64 records of 16 bytes, record l the values
// 16 (l / 16) .. + 15 of row l % 16: what lane l of a 16x16x64 matrix instruction takes. Rows and
// values past the end are 0. With both operands in this order every load moves whole kilobytes, to
// registers or to LDS, and odd sizes end in zeros that need no test in the loops.
#include "igemm_common.hpp"
#include "kernels.hpp"
#include "runtime.hpp"
#include "seq_common.hpp"

namespace c2d {

namespace {

typedef int i32x16 __attribute__((ext_vector_type(16)));

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

// 16 values of a row from k on as fp32, zeros from n on; rows need not be aligned.
template <typename T> __device__ __forceinline__ void load16(const T *row, int k, int n, Pack<T, 16> &v) {
    if (k + 16 <= n) {
        __builtin_memcpy(&v, row + k, sizeof v);
    } else {
#pragma unroll
        for (int e = 0; e < 16; e++) v.v[e] = k + e < n ? row[k + e] : from_f32<T>(0.0f);
    }
}

template <typename T> __device__ __forceinline__ uint32_t magnitude(const Pack<T, 16> &v, uint32_t most) {
#pragma unroll
    for (int e = 0; e < 16; e++) most = max(most, __builtin_bit_cast(uint32_t, to_f32(v.v[e])) & 0x7fffffffu);
    return most;
}

template <typename T> __device__ __forceinline__ u32x4 codes16(const Pack<T, 16> &v, float s, float r) {
    u32x4 out;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < 4; e++) w |= ((uint32_t)code_of(to_f32(v.v[4 * i + e]), s, r) & 255u) << 8 * e;
        out[i] = w;
    }
    return out;
}

// One row a wave, 16 rows (a row tile) a workgroup, so that the 16-byte records of a kilobyte
// meet in one L2. NR records of a lane stay in registers between the maximum and the codes; a
// longer row is read again.
template <typename T, int NR>
__global__ __launch_bounds__(1024) void quantize_kernel(const T *x, long long x_row, void *packed, int rows, int n) {
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int row = blockIdx.x * kRows + wave, blocks = val_blocks(n), groups = blocks * 4;
    u32x4 *out = static_cast<u32x4 *>(packed);
    float *scales = scales_of(packed, rows, n);
    if (row >= rows) {
        for (int g = lane; g < groups; g += 64) out[record_at(row, g, blocks)] = u32x4{};
        if (lane == 0) scales[row] = 0.0f;
        return;
    }
    const T *p = x + row * x_row;
    Pack<T, 16> kept[NR];
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < NR; i++)
        if (i * 1024 < n) load16(p, (i * 64 + lane) * 16, n, kept[i]);
#pragma unroll
    for (int i = 0; i < NR; i++)
        if (i * 1024 < n) most = magnitude(kept[i], most);
    for (int g = NR * 64 + lane; g < groups; g += 64) {
        Pack<T, 16> v;
        load16(p, g * 16, n, v);
        most = magnitude(v, most);
    }
#pragma unroll
    for (int o = 1; o < 64; o *= 2) most = max(most, (uint32_t)__shfl_xor((int)most, o));
    const float s = row_scale(most), r = 1.0f / s;
    if (lane == 0) scales[row] = s;
#pragma unroll
    for (int i = 0; i < NR; i++)
        if (i * 64 + lane < groups) out[record_at(row, i * 64 + lane, blocks)] = codes16(kept[i], s, r);
    for (int g = NR * 64 + lane; g < groups; g += 64) {
        Pack<T, 16> v;
        load16(p, g * 16, n, v);
        out[record_at(row, g, blocks)] = codes16(v, s, r);
    }
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

// sum * sx * sw, the smaller scale first: nothing overflows or loses bits on the way that the
// product itself does not (scales of quantized rows are normal numbers).
__device__ __forceinline__ float scaled(int sum, float a, float b) {
    const bool less = fabsf(a) < fabsf(b);
    return (float)sum * (less ? a : b) * (less ? b : a);
}

template <typename T> __device__ __forceinline__ T finish(const Q8Args &a, int sum, int row, int o) {
    const float res = a.residual ? to_f32(static_cast<const T *>(a.residual)[row * a.residual_row + o]) : 0.0f;
    const float v = epilogue(scaled(sum, a.sx[row], a.sw[o]), a.bias ? a.bias[o] : 0.0f,
                             a.act == CONV2D_ACT_PRELU ? a.alpha[o] : 0.0f, res, a.residual != nullptr, a.act, a.before != 0);
    return round_fp32<T>(v);
}

// A few rows: a workgroup computes 16 NT outputs of 16 MT rows, straight from memory; its W waves
// take the value blocks in turn and add up in LDS.
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
    for (int i = threadIdx.x; i < NT * MT * 256; i += 64 * W) {
        // value r of lane l of tile (n, m): row 4 (l / 16) + r, output l % 16
        const int l = i % 64, r = i / 64 % 4, t = i / 256;
        const int row = (m0 + t % MT) * 16 + l / 16 * 4 + r, o = (n0 + t / MT) * 16 + l % 16;
        if (row >= a.rows || o >= a.outs) continue;
        int sum = 0;
#pragma unroll
        for (int v = 0; v < W; v++) sum += s_sum[v][t][l][r];
        static_cast<T *>(a.y)[row * a.y_row + o] = finish<T>(a, sum, row, o);
    }
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

// Many rows: BM rows x BN outputs a workgroup, WM x WN waves of 32x32 blocks, steps of one value
// block through a ring of NS stages in LDS, loaded directly from memory.
template <typename T, int BM, int BN, int WM, int WN, int NS>
__global__ __launch_bounds__(64 * WM * WN) void q8_tile_kernel(const Q8Args a, int tiles_m, int tiles_n) {
    constexpr int NW = WM * WN, FM = BM / (32 * WM), FN = BN / (32 * WN);
    constexpr int STAGE = (BM + BN) * kVals, CH = (BM + BN) / 16, LPW = CH / NW;
    static_assert(CH % NW == 0 && NS >= 3, "whole loads a wave");
    __shared__ __attribute__((aligned(1024))) char lds[NS * STAGE];
    static_assert(NW * 32 * 36 * 4 <= NS * STAGE, "the epilogue's slices fit");
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int wm = wave % WM, wn = wave / WM;
    const int g = xcd_remap(blockIdx.x, tiles_m * tiles_n);
    const int tm = g % tiles_m, tn = g / tiles_m;
    const int mtiles = row_tiles(a.rows), ntiles = row_tiles(a.outs), KB = a.blocks;

    // This wave's loads of a stage: row tile `d * NW + wave` of the rows, then of the weights, as
    // buffers of the row tile's value blocks.
    const char *src[LPW];
#pragma unroll
    for (int d = 0; d < LPW; d++) {
        const int ch = d * NW + wave;
        const bool isx = ch < BM / 16;
        const int t = isx ? min(tm * (BM / 16) + ch, mtiles - 1) : min(tn * (BN / 16) + ch - BM / 16, ntiles - 1);
        src[d] = reinterpret_cast<const char *>(isx ? a.x : a.w) + (long long)t * KB * kTileBytes;
    }
    const uint32_t base = lds_addr(lds);
    auto issue = [&](int kb) {
        const int k = min(kb, KB - 1);
#pragma unroll
        for (int d = 0; d < LPW; d++)
            dma_b128(rsrc_words(src[d], KB * kTileBytes), (uint32_t)(k * kTileBytes + lane * 16),
                     base + kb % NS * STAGE + (d * NW + wave) * kTileBytes);
    };
#pragma unroll
    for (int s = 0; s < NS - 1; s++) issue(s);

    i32x16 acc[FM][FN] = {};
    const int at = (lane % 32 / 16) * kTileBytes + lane / 32 * 256 + lane % 16 * 16;
    for (int kb = 0; kb < KB; kb++) {
        q8_wait_vmcnt<(NS - 2) * LPW>();
        q8_barrier();
        issue(kb + NS - 1);
        const char *st = lds + kb % NS * STAGE;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            i32x4 xf[FM], wf[FN];
#pragma unroll
            for (int m = 0; m < FM; m++) xf[m] = *reinterpret_cast<const i32x4 *>(st + (wm * FM + m) * 2 * kTileBytes + h * 512 + at);
#pragma unroll
            for (int n = 0; n < FN; n++)
                wf[n] = *reinterpret_cast<const i32x4 *>(st + BM * kVals + (wn * FN + n) * 2 * kTileBytes + h * 512 + at);
#pragma unroll
            for (int m = 0; m < FM; m++)
#pragma unroll
                for (int n = 0; n < FN; n++) acc[m][n] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[n], xf[m], acc[m][n], 0, 0, 0);
        }
    }
    q8_wait_vmcnt<0>();
    q8_barrier();

    // Block by block through LDS, so that a lane stores neighbouring outputs of one row.
    // Value i of lane l: output 8 (i / 4) + 4 (l / 32) + i % 4, row l % 32.
    int *slice = reinterpret_cast<int *>(lds) + wave * 32 * 36;
#pragma unroll
    for (int m = 0; m < FM; m++)
#pragma unroll
        for (int n = 0; n < FN; n++) {
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<i32x4 *>(slice + lane % 32 * 36 + i * 2 + lane / 32 * 4) =
                    i32x4{acc[m][n][i], acc[m][n][i + 1], acc[m][n][i + 2], acc[m][n][i + 3]};
            __builtin_amdgcn_s_waitcnt(0xC07F);
            __builtin_amdgcn_wave_barrier();
            for (int i = lane; i < 32 * 32; i += 64) {
                const int row = tm * BM + (wm * FM + m) * 32 + i / 32, o = tn * BN + (wn * FN + n) * 32 + i % 32;
                if (row < a.rows && o < a.outs)
                    static_cast<T *>(a.y)[row * a.y_row + o] = finish<T>(a, slice[i / 32 * 36 + i % 32], row, o);
            }
            __builtin_amdgcn_s_waitcnt(0xC07F);
            __builtin_amdgcn_wave_barrier();
        }
}

template <typename T, int NT, int MT, int W> hipError_t few(const Q8Args &a, hipStream_t st) {
    const int nblocks = (row_tiles(a.outs) + NT - 1) / NT;
    const long long mblocks = (row_tiles(a.rows) + MT - 1) / MT;
    return launch_blocks(q8_few_kernel<T, NT, MT, W>, nblocks * mblocks, 64 * W, st, a, nblocks);
}

template <typename T, int BM, int BN, int WM, int WN, int NS> hipError_t tiled(const Q8Args &a, hipStream_t st) {
    const long long tm = (a.rows + BM - 1ll) / BM, tn = (a.outs + BN - 1ll) / BN;
    if (tm * tn > 0x7fffffff) return hipErrorInvalidConfiguration;
    return launch_blocks(q8_tile_kernel<T, BM, BN, WM, WN, NS>, tm * tn, 64 * WM * WN, st, a, (int)tm, (int)tn);
}

template <typename T> hipError_t launch_product(const Q8Args &a, hipStream_t st) {
    if (a.rows <= 16) return few<T, 1, 1, 8>(a, st);
    if (a.rows <= 64) return few<T, 2, 2, 8>(a, st);
    if (a.rows <= 1024) return tiled<T, 64, 64, 2, 2, 4>(a, st);
    return tiled<T, 256, 256, 2, 2, 4>(a, st);
}

template <typename T> hipError_t quantize(const void *x, long long x_row, void *packed, int rows, int n, hipStream_t st) {
    const int tiles = row_tiles(rows);
    const T *p = static_cast<const T *>(x);
    if (n <= 2048) return launch_blocks(quantize_kernel<T, 2>, tiles, 1024, st, p, x_row, packed, rows, n);
    return launch_blocks(quantize_kernel<T, sizeof(T) == 4 ? 4 : 8>, tiles, 1024, st, p, x_row, packed, rows, n);
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

hipError_t launch_matmul_q8(const matmul_q8_args &a, void *ws, hipStream_t st) {
    const void *x = a.x_packed;
    if (!x) {
        const quantize_rows_args q{a.x, ws, a.x_row, a.rows, a.in_features, a.dtype};
        const hipError_t e = launch_quantize_rows(q, st);
        if (e != hipSuccess) return e;
        x = ws;
    }
    const Q8Args p{static_cast<const u32x4 *>(x), static_cast<const u32x4 *>(a.weights), scales_of(x, a.rows, a.in_features),
                   scales_of(a.weights, a.out_features, a.in_features), a.bias, a.alpha, a.residual, a.y, a.residual_row, a.y_row,
                   a.rows, a.out_features, val_blocks(a.in_features), a.act & 0xff, (a.act & CONV2D_RES_BEFORE_ACT) != 0};
    if (a.dtype == CONV2D_DTYPE_F32) return launch_product<float>(p, st);
    if (a.dtype == CONV2D_DTYPE_BF16) return launch_product<bf16>(p, st);
    return launch_product<f16>(p, st);
}

}  // namespace c2d
