// pool.cuh -- addressing of the paged 4-bit KV pool (layout in spectra.h).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "spectra.h"

namespace spectra {

// What the kernels need of a spectra_kv_pool (page_size is a power of two).
struct PoolView {
    uint32_t *kc;        // K code words, slot*4G + w*G + g
    uint16_t *ks;
    uint32_t *kz;
    uint16_t *vc;        // V code halfwords, slot*8G + e*G + g
    uint16_t *vs;
    uint32_t *vz;
    float *mass;
    int H, G, lp, n_pages;  // heads, groups of 32 channels, log2(page size), pages

    static PoolView of(const spectra_kv_pool &p) {
        PoolView v;
        v.kc = reinterpret_cast<uint32_t *>(p.k_codes);
        v.ks = p.k_scales;
        v.kz = p.k_zeros;
        v.vc = reinterpret_cast<uint16_t *>(p.v_codes);
        v.vs = p.v_scales;
        v.vz = p.v_zeros;
        v.mass = p.mass;
        v.H = p.n_heads;
        v.G = p.head_dim / 32;
        v.lp = 0;
        while ((1 << v.lp) < p.page_size) ++v.lp;
        v.n_pages = p.n_pages;
        return v;
    }
    // Slot of head h at token slot ts = page * page_size + r.
    __device__ __forceinline__ int64_t slot(int32_t ts, int h) const {
        return (((int64_t)(ts >> lp) * H + h) << lp) + (ts & ((1 << lp) - 1));
    }
    // Token slot of position t of a sequence with this page table row; -1 for
    // a page outside the pool.
    __device__ __forceinline__ int32_t token_slot(const int32_t *pages, int t) const {
        const int32_t p = pages[t >> lp];
        return (uint32_t)p < (uint32_t)n_pages ? (p << lp) + (t & ((1 << lp) - 1)) : -1;
    }
    __host__ __device__ int64_t token_slots() const { return (int64_t)n_pages << lp; }
};

}  // namespace spectra
