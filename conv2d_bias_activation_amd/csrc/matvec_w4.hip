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
        uint32_t w = 0;
        for (int e = 0; e < 8; e++) {
            const int k = k0 + e;
            if (n < N && k < K) {
                const uint32_t q = codes[(long long)n * bytes + k / 2] >> (4 * (k % 2)) & 15u;
                w |= q << (16 * (e % 2) + 4 * (e / 2));
            }
        }
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

// One wave for 16 outputs of one row: each lane sums its record's inputs.
template <typename T>
__global__ __launch_bounds__(64) void matvec_w4_kernel(const matvec_w4_args a, const uint32_t *packed, const T *scales,
                                                       const uint8_t *zeros) {
    const int kb = (a.in_features + kTileK - 1) / kTileK, per = kTileK / a.group;
    const int l = threadIdx.x, tiles = (a.out_features + kTileN - 1) / kTileN;
    const int tile = blockIdx.x % tiles, r = blockIdx.x / tiles;
    const int n = tile * kTileN + l % 16;
    const T *x = static_cast<const T *>(a.x) + r * a.x_row;
    float sum = 0.0f;
    for (int b = 0; b < kb; b++) {
        const long long at = (long long)tile * kb + b;
        for (int j = 0; j < 4; j++) {
            const uint32_t w = packed[at * 256 + l * 4 + j];
            const long long g = (at * kTileN + l % 16) * per + 32 * j / a.group;
            const float s = to_f32(scales[g]), z = zeros ? (float)zeros[g] : 8.0f;
            float part = 0.0f;
            for (int e = 0; e < 8; e++) {
                const int k = b * kTileK + 32 * j + 8 * (l / 16) + e;
                const float q = (float)(w >> (16 * (e % 2) + 4 * (e / 2)) & 15u);
                if (k < a.in_features) part = fmaf(to_f32(x[k]), q - z, part);
            }
            sum = fmaf(part, s, sum);
        }
    }
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    if (l >= 16 || n >= a.out_features) return;
    const float res = a.residual ? to_f32(static_cast<const T *>(a.residual)[r * a.residual_row + n]) : 0.0f;
    const int act = a.act & 0xff;
    const float v = epilogue(sum, a.bias ? a.bias[n] : 0.0f, act == CONV2D_ACT_PRELU ? a.alpha[n] : 0.0f, res,
                             a.residual != nullptr, act, (a.act & CONV2D_RES_BEFORE_ACT) != 0);
    static_cast<T *>(a.y)[r * a.y_row + n] = round_fp32<T>(v);
}

long long tiles(int N, int K) { return (long long)((N + kTileN - 1) / kTileN) * ((K + kTileK - 1) / kTileK); }

template <typename T> hipError_t launch_t(const matvec_w4_args &a, hipStream_t st) {
    const long long nt = tiles(a.out_features, a.in_features);
    const char *p = static_cast<const char *>(a.packed);
    const T *scales = reinterpret_cast<const T *>(p + nt * kTileBytes);
    const uint8_t *zeros = reinterpret_cast<const uint8_t *>(scales + nt * kTileN * (kTileK / a.group));
    return launch_kernel(matvec_w4_kernel<T>, dim3((unsigned)((long long)((a.out_features + kTileN - 1) / kTileN) * a.rows)),
                         dim3(64), 0, st, a, static_cast<const uint32_t *>(a.packed), scales,
                         a.has_zeros ? zeros : nullptr);
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
