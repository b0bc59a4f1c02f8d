// Shared device helpers of the sequence operators (gfx950 only).
#pragma once

#include "common.hpp"
#include "../../include/sequence_ops.h"

namespace c2d {

// VEC consecutive values of the storage type, moved by one load or store (16 bytes in the
// vector paths).
template <typename T, int VEC> struct alignas(sizeof(T) * VEC) Pack {
    T v[VEC];
};

template <typename T, int VEC> __device__ __forceinline__ Pack<T, VEC> load_pack(const T *p) {
    return *reinterpret_cast<const Pack<T, VEC> *>(p);
}

template <typename T, int VEC> __device__ __forceinline__ void store_pack(T *p, const Pack<T, VEC> &v) {
    *reinterpret_cast<Pack<T, VEC> *>(p) = v;
}

// One run of at most `run` tokens of one sequence.
struct SeqRun {
    int seq;
    int start;  // first token row of the sequence (packed), or 0
    int len;    // tokens of the sequence
    int first;  // first token of the run within the sequence
};

__device__ __forceinline__ int clamped_offset(const int *offsets, int i, int tokens) {
    const int v = offsets[i];
    return v < 0 ? 0 : (v > tokens ? tokens : v);
}

// Runs of packed sequences are numbered so that sequence s owns the numbers from
// offsets[s] / run + s up to offsets[s + 1] / run + s: at least ceil(len / run) of them, at
// least one, and tokens / run + nseq in all, which the host knows without reading the
// offsets. False for a number that no tokens belong to; the first run of an empty sequence
// counts, for its state.
__device__ __forceinline__ bool find_run(const int *offsets, int nseq, int tokens, int run, int item, SeqRun *r) {
    int lo = 0, hi = nseq - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (clamped_offset(offsets, mid, tokens) / run + mid <= item)
            lo = mid;
        else
            hi = mid - 1;
    }
    const int start = clamped_offset(offsets, lo, tokens);
    const int end = clamped_offset(offsets, lo + 1, tokens);
    const long long first = (long long)(item - start / run - lo) * run;
    r->seq = lo;
    r->start = start;
    r->len = end > start ? end - start : 0;
    if (first < 0 || (first > 0 && first >= r->len)) return false;
    r->first = (int)first;
    return true;
}

// State row of sequence seq, or -1 for none.
__device__ __forceinline__ int state_row(const void *state, const int *slots, int seq, int rows) {
    const int s = slots ? slots[seq] : seq;
    return state && s >= 0 && s < rows ? s : -1;
}

}  // namespace c2d
