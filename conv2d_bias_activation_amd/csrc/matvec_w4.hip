// Products of a few token rows with 4-bit weights (gfx950 only).
//
// Packed weights: tiles of 16 outputs x 128 inputs, all input blocks of an output tile in a
// row. A tile is 64 records of 16 bytes, record l for output l % 16 and the inputs with
// (k / 8) % 4 == l / 16: dword j holds k = 32 j + 8 (l / 16) + i, i = 0 .. 7, the code of i at
// bits 16 (i % 2) + 4 (i / 2), so that one mask takes two neighbouring codes into the halves
// of a register. Behind all tiles come the scales, [tile][input block][output][128 / group],
// then the zero points in the same order, one byte each. Outputs and inputs past the end have
// code 0 and scale 0.
#include "kernels.hpp"
#include "seq_common.hpp"

namespace c2d {

namespace {

constexpr int kTileN = 16, kTileK = 128, kTileBytes = kTileN * kTileK / 2;

__global__ __launch_bounds__(256) void w4_pack_kernel(const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros,
                                                      uint32_t *packed, int N, int K, int group) {
    const int nt = (N + kTileN - 1) / kTileN, kb = (K + kTileK - 1) / kTileK, per = kTileK / group;
    const int groups = (K + group - 1) / group, bytes = (K + 1) / 2;
    const long long words = (long long)nt * kb * (kTileBytes / 4);
    const long long nscale = (long long)nt * kb * kTileN * per;
    uint16_t *ps = reinterpret_cast<uint16_t *>(packed + words);
    uint8_t *pz = reinterpret_cast<uint8_t *>(ps + nscale);
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < words; i += gridDim.x * 256ll) {
        const int j = i % 4, l = i / 4 % 64;
        const long long tile = i / 256;
        const int n = (int)(tile / kb) * kTileN + l % 16;
        const int k0 = (int)(tile % kb) * kTileK + 32 * j + 8 * (l / 16);
        uint32_t q = 0;  // the codes in the order of their inputs
        if (n < N && k0 + 8 <= K) {
            __builtin_memcpy(&q, codes + (long long)n * bytes + k0 / 2, 4);
        } else if (n < N) {
            for (int e = 0; k0 + e < K; e++) q |= (codes[(long long)n * bytes + (k0 + e) / 2] >> (4 * (e % 2)) & 15u) << 4 * e;
        }
        uint32_t w = 0;
        for (int e = 0; e < 8; e++) w |= (q >> 4 * e & 15u) << (16 * (e % 2) + 4 * (e / 2));
        packed[i] = w;
    }
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < nscale; i += gridDim.x * 256ll) {
        const long long tile = i / (kTileN * per);
        const int n = (int)(tile / kb) * kTileN + (int)(i / per % kTileN);
        const int g = (int)(tile % kb) * per + (int)(i % per);
        const bool in = n < N && g < groups;
        ps[i] = in ? scales[(long long)n * groups + g] : 0;
        if (zeros) pz[i] = in ? zeros[(long long)n * groups + g] & 15u : 0;
    }
}

template <typename T> struct Frag;
template <> struct Frag<bf16> {
    typedef bf16 v8 __attribute__((ext_vector_type(8)));
    // Everything that meets x is 2^-12 of its value, so that the sums of a group, with its offset
    // of up to 31 a code, stay in range for any finite x; the products of even the smallest x
    // are still exact in fp32, as multiples of 2^-145.
    static constexpr float kUnit = 4096.0f;
    static constexpr uint32_t kOnes = 0x39803980u;
    // 16 + q for the codes of pair p: q in the upper four mantissa bits of 16
    static __device__ __forceinline__ uint32_t pair(uint32_t w, int p) {
        return ((p == 0 ? w << 3 : w >> (4 * p - 3)) & 0x00780078u) | 0x3b803b80u;
    }
    static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
    }
};
template <> struct Frag<f16> {
    typedef f16 v8 __attribute__((ext_vector_type(8)));
    static constexpr float kUnit = 1.0f;
    static constexpr uint32_t kOnes = 0x3c003c00u;
    static __device__ __forceinline__ uint32_t pair(uint32_t w, int p) {
        return ((p < 2 ? w << (6 - 4 * p) : w >> (4 * p - 6)) & 0x03c003c0u) | 0x4c004c00u;
    }
    static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
    }
};

// Eight values of a row from k on, zeros from K on; rows need not be aligned. Where the eight
// reach past the row's end its last eight are loaded and moved down.
template <typename T> __device__ __forceinline__ u32x4 load_row8(const T *row, int k, int K) {
    uint64_t lo = 0, hi = 0;
    if (K < 8) {
#pragma unroll
        for (int e = 0; e < 7; e++) {
            const uint64_t h = k + e < K ? __builtin_bit_cast(uint16_t, row[k + e]) : 0;
            (e < 4 ? lo : hi) |= h << 16 * (e % 4);
        }
    } else {
        const int at = min(k, K - 8), bits = 16 * min(k - at, 8);
        u32x4 v;
        __builtin_memcpy(&v, row + at, 16);
        lo = (uint64_t)v[1] << 32 | v[0];
        hi = (uint64_t)v[3] << 32 | v[2];
        if (bits >= 64) {
            lo = bits < 128 ? hi >> (bits - 64) : 0;
            hi = 0;
        } else if (bits) {
            lo = lo >> bits | hi << (64 - bits);
            hi >>= bits;
        }
    }
    return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

// What a wave needs of one input block.
template <int NT, int MT, int PER> struct Block {
    u32x4 codes[NT], x[MT][4];
    Pack<uint16_t, PER> scale[NT];
    Pack<uint8_t, PER> zero[NT];
};

// A workgroup computes 16 NT outputs of 16 MT rows; its W waves take the input blocks in
// turn, so that together they read whole runs of packed weights, and add up in LDS at the
// end, in a fixed order.
//
// The matrix cores take x as the A operand and the codes, as the exact 16-bit values 16 + q, as
// B: two instructions for two codes, and no multiplication with scales before the sum. With S
// the sum of the same inputs (x times ones), a group's part of an output is
// scale * (sum of x (16 + q) - (16 + zero) S), in fp32. Its rounding error is a few 2^-24 of
// scale * (sum of |x|) * (47 + zero), five times what the codes without the offset would have
// (little beside y's own rounding but where a row's products cancel). Bound by the bytes
// of the packed weights where there are many (16 rows, 8192 -> 32768: 38 us, 3.9 TB/s), else by
// the latency of a wave's few blocks (1 row, 2048 -> 4096: 3.8 us of kernel).
template <typename T, int NT, int MT, int W, int PER, bool ZEROS>
__global__ __launch_bounds__(64 * W) void matvec_w4_kernel(const matvec_w4_args a, const u32x4 *packed, const uint16_t *scales,
                                                           const uint8_t *zeros, int nblocks) {
    __shared__ f32x4 s_sum[W][NT * MT][64];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int KB = (a.in_features + kTileK - 1) / kTileK, tiles = (a.out_features + kTileN - 1) / kTileN;
    const int tile0 = (int)(blockIdx.x % nblocks) * NT, row0 = (int)(blockIdx.x / nblocks) * 16 * MT;

    const T *row[MT];  // the lane's rows of x (past the last one: that again, never stored)
#pragma unroll
    for (int m = 0; m < MT; m++)
        row[m] = static_cast<const T *>(a.x) + min(row0 + 16 * m + lane % 16, a.rows - 1) * a.x_row;
    long long at[NT];  // first input block of the lane's tiles
#pragma unroll
    for (int n = 0; n < NT; n++) at[n] = (long long)min(tile0 + n, tiles - 1) * KB;

    auto load = [&](int kb, Block<NT, MT, PER> &b) {
#pragma unroll
        for (int n = 0; n < NT; n++) {
            b.codes[n] = packed[(at[n] + kb) * 64 + lane];
            const long long g = ((at[n] + kb) * kTileN + lane % 16) * PER;
            b.scale[n] = load_pack<uint16_t, PER>(scales + g);
            if (ZEROS) b.zero[n] = load_pack<uint8_t, PER>(zeros + g);
        }
        const int k = kb * kTileK + lane / 16 * 8;
        if ((kb + 1) * kTileK <= a.in_features) {
#pragma unroll
            for (int m = 0; m < MT; m++)
#pragma unroll
                for (int j = 0; j < 4; j++) __builtin_memcpy(&b.x[m][j], row[m] + k + 32 * j, 16);
        } else {
#pragma unroll
            for (int m = 0; m < MT; m++)
#pragma unroll
                for (int j = 0; j < 4; j++) b.x[m][j] = load_row8(row[m], k + 32 * j, a.in_features);
        }
    };

    f32x4 out[NT][MT] = {};
    const u32x4 ones = {Frag<T>::kOnes, Frag<T>::kOnes, Frag<T>::kOnes, Frag<T>::kOnes};
    auto multiply = [&](const Block<NT, MT, PER> &b) {
#pragma unroll
        for (int g = 0; g < PER; g++) {
            f32x4 acc[NT][MT] = {}, sum[MT] = {};
#pragma unroll
            for (int j = g * 4 / PER; j < (g + 1) * 4 / PER; j++) {
#pragma unroll
                for (int m = 0; m < MT; m++) sum[m] = Frag<T>::mfma(b.x[m][j], ones, sum[m]);
#pragma unroll
                for (int n = 0; n < NT; n++) {
                    u32x4 q;
#pragma unroll
                    for (int p = 0; p < 4; p++) q[p] = Frag<T>::pair(b.codes[n][j], p);
#pragma unroll
                    for (int m = 0; m < MT; m++) acc[n][m] = Frag<T>::mfma(b.x[m][j], q, acc[n][m]);
                }
            }
#pragma unroll
            for (int n = 0; n < NT; n++) {
                const float s = to_f32(__builtin_bit_cast(T, b.scale[n].v[g]));
                const float z = ZEROS ? -16.0f - (float)b.zero[n].v[g] : -24.0f;
#pragma unroll
                for (int m = 0; m < MT; m++)
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        out[n][m][i] = fmaf(s, fmaf(z, sum[m][i], acc[n][m][i]), out[n][m][i]);
            }
        }
    };
    if (wave < KB) {
        // One block on its way while another is multiplied. With four tiles, whose waves have
        // many blocks each, loading the last one again is cheaper than a branch around it (16
        // rows, 8192 -> 32768, groups of 64: 37.8 and 40.3 us); with fewer it is not (5 rows,
        // 4010 -> 10007: 12.2 and 11.1 us).
        constexpr bool kAgain = NT == 4;
        Block<NT, MT, PER> even, odd;
        load(wave, even);
        for (int kb = wave; kb < KB; kb += 2 * W) {
            if (kAgain || kb + W < KB) load(min(kb + W, KB - 1), odd);
            multiply(even);
            if (kb + W >= KB) break;
            if (kAgain || kb + 2 * W < KB) load(min(kb + 2 * W, KB - 1), even);
            multiply(odd);
        }
    }

#pragma unroll
    for (int n = 0; n < NT; n++)
#pragma unroll
        for (int m = 0; m < MT; m++) s_sum[wave][n * MT + m][lane] = out[n][m];
    __syncthreads();
    const int act = a.act & 0xff;
    for (int i = threadIdx.x; i < NT * MT * 256; i += 64 * W) {
        // value r of lane l of tile (n, m): row 4 (l / 16) + r, output l % 16
        const int l = i % 64, r = i / 64 % 4, t = i / 256;
        const int m = row0 + 16 * (t % MT) + l / 16 * 4 + r, n = (tile0 + t / MT) * kTileN + l % 16;
        if (m >= a.rows || n >= a.out_features) continue;
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < W; w++) sum += s_sum[w][t][l][r];
        const float res = a.residual ? to_f32(static_cast<const T *>(a.residual)[m * a.residual_row + n]) : 0.0f;
        const float v = epilogue(sum * Frag<T>::kUnit, a.bias ? a.bias[n] : 0.0f, act == CONV2D_ACT_PRELU ? a.alpha[n] : 0.0f, res,
                                 a.residual != nullptr, act, (a.act & CONV2D_RES_BEFORE_ACT) != 0);
        static_cast<T *>(a.y)[m * a.y_row + n] = round_fp32<T>(v);
    }
}

long long tiles(int N, int K) { return (long long)((N + kTileN - 1) / kTileN) * ((K + kTileK - 1) / kTileK); }

template <typename T, int NT, int MT, int W, int PER, bool ZEROS> hipError_t launch(const matvec_w4_args &a, hipStream_t st) {
    const long long nt = tiles(a.out_features, a.in_features);
    const char *p = static_cast<const char *>(a.packed);
    const uint16_t *scales = reinterpret_cast<const uint16_t *>(p + nt * kTileBytes);
    const uint8_t *zeros = reinterpret_cast<const uint8_t *>(scales + nt * kTileN * PER);
    const int nblocks = ((a.out_features + kTileN - 1) / kTileN + NT - 1) / NT;
    const long long mblocks = (a.rows + 16 * MT - 1) / (16 * MT);
    return launch_blocks(matvec_w4_kernel<T, NT, MT, W, PER, ZEROS>, nblocks * mblocks, 64 * W, st, a,
                         static_cast<const u32x4 *>(a.packed), scales, zeros, nblocks);
}

// Output tiles (NT) and waves (W) of a workgroup. More tiles read x less often, which counts
// from some eight rows on; fewer give more workgroups; more waves halve the blocks that each
// reads one after the other, and make the sum in LDS longer. Times in us, 1 row / 16 rows,
// groups of 128, weights not in cache:
//   outputs x inputs   NT=4 W=4    NT=4 W=8    NT=2 W=8    NT=1 W=16   NT=1 W=8    NT=1 W=4
//   32768 x 8192      33.2 / 37.6 33.6 / 39.6 31.9 / 46.3 47.5 / 87.6 40.4 / 73.5 40.8 / 70.9
//   16384 x 4096      12.4 / 13.0 10.5 / 11.5 10.3 / 14.4 14.3 / 28.5 11.4 / 22.5 10.9 / 21.0
//    8192 x 8192      18.8 / 19.0 13.8 / 15.7 10.1 / 13.4 11.8 / 23.3 10.6 / 20.8 13.0 / 19.5
//    4096 x 4096      10.9 / 11.5  8.1 /  9.7  5.9 /  8.3  5.1 /  8.9  5.2 /  7.9  6.8 /  8.1
//    2048 x 8192      17.4 / 17.9 12.3 / 14.5  8.6 / 12.0  6.5 / 12.4  7.3 / 11.4 10.3 / 12.1
//    4096 x 1024       5.1 /  5.8  4.5 /  5.6  3.4 /  4.7  3.3 /  4.6  3.1 /  4.5  3.1 /  4.0
// Past 16 rows the weights are read and decoded again for every 32 (one plan; not tuned). That
// and the library's 1x1 convolution on 16-bit weights, us at 32 / 64 / 128 rows, groups of 64: 2048
// -> 4096 8.1 / 8.2 / 14.3 and 15.4 / 15.6 / 15.8; 4096 -> 4096 12.0 / 12.3 / 22.5 and 17.1 / 17.8 / 22.0;
// 2048 -> 16384 15.7 / 27.9 / 52.1 and 21.8 / 22.5 / 26.9; 8192 -> 32768 77 / 152 / 296 and 168 / 176 / 197.
template <typename T, int PER, bool ZEROS> hipError_t launch_per(const matvec_w4_args &a, hipStream_t st) {
    const int n = (a.out_features + kTileN - 1) / kTileN, kb = (a.in_features + kTileK - 1) / kTileK;
    if (a.rows > 16) return launch<T, 2, 2, 8, PER, ZEROS>(a, st);
    const bool many = a.rows > 8;
    if (n >= 2048 && many) return launch<T, 4, 1, 4, PER, ZEROS>(a, st);
    if (n >= 1024 && many) return launch<T, 4, 1, 8, PER, ZEROS>(a, st);
    if (n >= 512) return launch<T, 2, 1, 8, PER, ZEROS>(a, st);
    if (kb <= 8) return launch<T, 1, 1, 4, PER, ZEROS>(a, st);
    if (kb >= 32 && !many) return launch<T, 1, 1, 16, PER, ZEROS>(a, st);
    return launch<T, 1, 1, 8, PER, ZEROS>(a, st);
}

template <typename T, int PER> hipError_t launch_z(const matvec_w4_args &a, hipStream_t st) {
    return a.has_zeros ? launch_per<T, PER, true>(a, st) : launch_per<T, PER, false>(a, st);
}

template <typename T> hipError_t launch_t(const matvec_w4_args &a, hipStream_t st) {
    return a.group == 32 ? launch_z<T, 4>(a, st) : a.group == 64 ? launch_z<T, 2>(a, st) : launch_z<T, 1>(a, st);
}

}  // namespace

size_t w4_packed_bytes(int out_features, int in_features, int group, bool zeros) {
    const size_t per_tile = kTileBytes + (size_t)kTileN * (kTileK / group) * (zeros ? 3 : 2);
    return (size_t)tiles(out_features, in_features) * per_tile;
}

hipError_t launch_w4_pack(const void *codes, const void *scales, const void *zeros, void *packed, int out_features,
                          int in_features, int group, int dtype, hipStream_t st) {
    (void)dtype;  // scales move as 16-bit patterns
    const long long words = tiles(out_features, in_features) * (kTileBytes / 4);
    const long long blocks = (words + 255) / 256;
    return launch_kernel(w4_pack_kernel, dim3((unsigned)(blocks < 8192 ? blocks : 8192)), dim3(256), 0, st,
                         static_cast<const uint8_t *>(codes), static_cast<const uint16_t *>(scales),
                         static_cast<const uint8_t *>(zeros), static_cast<uint32_t *>(packed), out_features, in_features,
                         group);
}

hipError_t launch_matvec_w4(const matvec_w4_args &a, hipStream_t st) {
    return a.dtype == CONV2D_DTYPE_BF16 ? launch_t<bf16>(a, st) : launch_t<f16>(a, st);
}

}  // namespace c2d
