// select.cuh -- order-preserving keys and the block-wide radix descent that
// the cache eviction and the sampler share.
#pragma once

#include <stdint.h>

namespace spectra {

// Unsigned key with the order of the floats (-0 reads as +0); NaN gets the
// lowest key, below -infinity.
__device__ __forceinline__ uint32_t float_key(float x) {
    if (!(x == x)) return 0u;
    const uint32_t b = __float_as_uint(x + 0.0f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
constexpr uint32_t kKeyNegInf = 0x007FFFFFu;  // float_key(-infinity)

// The float of a key that float_key made (not of NaN's).
__device__ __forceinline__ float key_float(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

// The key's digits, most significant first: 11 + 11 + 10 bits.
constexpr int kDigits = 3;
constexpr int kBins = 2048;
__device__ __forceinline__ int digit_shift(int d) { return d == 0 ? 21 : (d == 1 ? 10 : 0); }
__device__ __forceinline__ uint32_t digit_mask(int d) { return d == 2 ? 1023u : 2047u; }
// Whether key agrees with prefix in the digits above digit d.
__device__ __forceinline__ bool digit_in(uint32_t key, uint32_t prefix, int d) {
    return d == 0 || (key >> (d == 1 ? 21 : 10)) == (prefix >> (d == 1 ? 21 : 10));
}

// Sum of the 32 lanes below this one.
template <class T>
__device__ __forceinline__ T warp_exclusive(T v, int lane) {
    T s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += u;
    }
    return s - v;
}

// Exclusive sum over the block's threads (a multiple of 32, at most 1024), in
// thread order; *total gets the whole.  `part` is shared, 33 values; a barrier
// must lie between two uses.
template <class T>
__device__ __forceinline__ T block_exclusive(T v, T *part, T *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    const T before = warp_exclusive(v, lane);
    if (lane == 31) part[warp] = before + v;
    __syncthreads();
    if (warp == 0) {
        const T w = lane < nw ? part[lane] : T(0);
        const T e = warp_exclusive(w, lane);
        part[lane] = e;
        if (lane == 31) part[32] = e + w;
    }
    __syncthreads();
    *total = part[32];
    return part[warp] + before;
}

// Walks a histogram from its largest bin down and finds the bin in which the
// running sum first reaches `need` (1 <= need <= the histogram's sum): *bin,
// and in *above the sum of the bins over it.  All of the block's threads call
// it (a barrier before it must have completed the histogram); scratch: shared.
template <class T>
__device__ void find_bin_from_top(const T *hist, T need, T *part, int *bin, T *above) {
    const int nt = blockDim.x, per = (kBins + nt - 1) / nt;
    const int first = kBins - 1 - (int)threadIdx.x * per;  // this thread's largest bin
    T own = 0;
    for (int i = 0; i < per; ++i)
        if (first - i >= 0) own += hist[first - i];
    T total;
    T run = block_exclusive(own, part, &total);
    if (run < need && need <= run + own) {
        for (int i = 0; i < per && first - i >= 0; ++i) {
            const T h = hist[first - i];
            if (need <= run + h) {
                *bin = first - i;
                *above = run;
                break;
            }
            run += h;
        }
    }
    __syncthreads();
}

}  // namespace spectra
