// pool.cu -- the paged Group-32 4-bit KV pool: append, read back, evict
// (sm_100a).
//
// Method: "SPECTRA: Sparse-Precision Exact Channel Tensor Reconstruction
// Architecture" (Dev.to abstract), abstract paragraph: microscaled Group-32
// 4-bit key-value caching keeps long contexts resident.  Many sequences share
// one pool of pages; a page holds page_size positions of every head.  The
// codec is the weight quantiser (quant.cuh) per token and head.
#include "internal.cuh"
#include "pool.cuh"
#include "select.cuh"

namespace spectra {
namespace {

// bit 0: a non-finite value was appended; bit 1: a group's scale overflowed
// FP16; bit 2: a slot or page outside the pool.
__device__ unsigned int g_pool_error;

// One thread quantises 8 channels: the four threads of a group share its
// minimum and maximum, a head's 4G threads lie in one warp (32 / 4G heads per
// warp).  Item = (token, K or V, head), heads innermost, so a warp reads
// contiguous rows.
//
// The quantiser is quant.cuh's, bit for bit, with the scale's quotient in
// double and the codes' in single precision: rint(v / S) only depends on how
// v / S compares with k + 1/2.  For v != (k + 1/2) S, 2v - (2k+1)S is a
// multiple of the smaller of S's and 2v's last place; S has 11 significant
// bits and v has 8, so the quotient is at least 2^-12 from the tie.  It is at
// most 15 * 2^8 in magnitude (two different BF16 values near v differ by
// 2^-8 |v| or more, and S is their difference over 15), where a correctly
// rounded FP32 quotient is off by at most 2^-13; so it lies on the same side,
// and exact ties are exact in FP32.  (A subnormal S = j 2^-24 doubles both
// the bound on the quotient and the distance.)
__global__ void __launch_bounds__(256) pool_append_kernel(PoolView p, const uint16_t *__restrict__ k,
                                                          const uint16_t *__restrict__ v, int64_t k_stride,
                                                          int64_t v_stride, const int32_t *__restrict__ slots,
                                                          int64_t n_items) {
    const int G = p.G, tph = 4 * G, hpw = 32 / tph;  // threads per head, heads per warp
    const int lane = threadIdx.x & 31;
    const int sub = lane / tph, in = lane - sub * tph;
    const int64_t warp = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int64_t item = warp * hpw + sub;  // (token * 2 + which) * H + h
    bool live = sub < hpw && item < n_items;
    int h = 0, which = 0, g = in >> 2, part = in & 3;
    int32_t ts = -1;
    uint4 raw = make_uint4(0u, 0u, 0u, 0u);
    if (live) {
        const int64_t tw = item / p.H;
        h = (int)(item - tw * p.H);
        which = (int)(tw & 1);
        const int64_t tok = tw >> 1;
        ts = slots[tok];
        if (ts >= p.token_slots()) {
            if (in == 0) atomicOr(&g_pool_error, 4u);
            ts = -1;
        }
        const uint16_t *src = which ? v + tok * v_stride : k + tok * k_stride;
        raw = *reinterpret_cast<const uint4 *>(src + (int64_t)h * 32 * G + 8 * in);
    }
    live = live && ts >= 0;
    const uint32_t r4[4] = {raw.x, raw.y, raw.z, raw.w};
    float x[8];
    bool bad = false;
    float lo = 0.f, hi = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t b = i & 1 ? r4[i >> 1] & 0xFFFF0000u : r4[i >> 1] << 16;
        bad |= (b & 0x7F800000u) == 0x7F800000u;
        x[i] = __uint_as_float(b) + 0.0f;  // -0 reads as +0
        lo = i == 0 ? x[i] : fminf(lo, x[i]);
        hi = i == 0 ? x[i] : fmaxf(hi, x[i]);
    }
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        bad |= (bool)__shfl_xor_sync(0xffffffffu, (int)bad, o);
    }
    const double q15 = __ddiv_rn(__dsub_rn((double)hi, (double)lo), 15.0);
    unsigned short sbits;
    asm("cvt.rn.f16.f64 %0, %1;" : "=h"(sbits) : "d"(q15));
    unsigned int flags = 0;
    if (bad) flags = 1u;
    else if ((sbits & 0x7FFFu) == 0x7C00u) flags = 2u;
    if (flags) sbits = 0;  // the group is stored as zeros
    const float S = __half2float(__ushort_as_half(sbits));
    uint32_t z = 0, word = 0;
    if (S != 0.f) {
        const float zf = fminf(fmaxf(rintf(__fdiv_rn(-lo, S)), 0.f), 15.f);
        z = (uint32_t)zf;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float c = fminf(fmaxf(rintf(__fdiv_rn(x[i], S)) + zf, 0.f), 15.f);
            word |= (uint32_t)c << (4 * i);
        }
    }
    // the head's zero word: nibble g from the first thread of group g
    uint32_t zw = 0;
    const int base = sub < hpw ? sub * tph : 0;
    for (int j = 0; j < G; ++j) zw |= __shfl_sync(0xffffffffu, z, base + 4 * j) << (4 * j);
    if (!live) return;
    if (flags && part == 0) atomicOr(&g_pool_error, flags);
    const int64_t slot = p.slot(ts, h);
    if (which == 0) {
        p.kc[slot * 4 * G + part * G + g] = word;
        if (part == 0) p.ks[slot * G + g] = sbits;
        if (in == 0) p.kz[slot] = zw;
        if (in == 1 && p.mass) p.mass[slot] = 0.f;
    } else {
        uint16_t *c = p.vc + slot * 8 * G + (2 * part) * G + g;
        c[0] = (uint16_t)word;
        c[G] = (uint16_t)(word >> 16);
        if (part == 0) p.vs[slot * G + g] = sbits;
        if (in == 0) p.vz[slot] = zw;
    }
}

// Token slots dequantised: one thread per 8 channels of (token, head).
template <bool BF16>
__global__ void __launch_bounds__(256) pool_read_kernel(PoolView p, const int32_t *__restrict__ slots,
                                                        int64_t n_threads, void *__restrict__ k_out,
                                                        void *__restrict__ v_out) {
    const int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (e >= n_threads) return;
    const int G = p.G, per = p.H * 4 * G;
    const int64_t tok = e / per;
    const int in = (int)(e - tok * per);
    const int h = in / (4 * G), gp = in - h * 4 * G, g = gp >> 2, part = gp & 3;
    int32_t ts = slots[tok];
    if (ts >= p.token_slots()) {
        if (in == 0) atomicOr(&g_pool_error, 4u);
        ts = -1;
    }
    const int64_t slot = ts >= 0 ? p.slot(ts, h) : 0;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        void *out = which ? v_out : k_out;
        if (!out) continue;
        float x[8];
        if (ts >= 0) {
            uint32_t word;
            if (which == 0) {
                word = p.kc[slot * 4 * G + part * G + g];
            } else {
                const uint16_t *c = p.vc + slot * 8 * G + (2 * part) * G + g;
                word = (uint32_t)c[0] | ((uint32_t)c[G] << 16);
            }
            const float s = __half2float(__ushort_as_half((which ? p.vs : p.ks)[slot * G + g]));
            const int z = (int)(((which ? p.vz : p.kz)[slot] >> (4 * g)) & 15u);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = (float)((int)((word >> (4 * i)) & 15u) - z) * s;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = 0.f;
        }
        if (BF16) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&b);
            }
            reinterpret_cast<uint4 *>(out)[e] = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            float4 *o = reinterpret_cast<float4 *>(out) + 2 * e;
            o[0] = make_float4(x[0], x[1], x[2], x[3]);
            o[1] = make_float4(x[4], x[5], x[6], x[7]);
        }
    }
}

// ---- eviction ----
// Two launches: select (one CTA per sequence and head) finds the smallest
// kept key and, per chunk of positions, the number of kept positions before
// it; move (one CTA per chunk) copies the chunk's kept entries to their
// places in the fresh pages.
constexpr int kSelThreads = 1024;
constexpr int kMoveChunk = 256;  // positions per chunk (= threads of a move CTA)

struct EvictArgs {
    PoolView p;
    const int32_t *pages;
    const int32_t *dst_pages;
    const int32_t *lengths;
    int32_t *new_lengths;
    int max_pages, dst_max_pages, budget, recent, nch;  // nch: chunks of the longest sequence
    uint32_t *thr;   // [seq][head]: smallest kept key
    int *ties;       // [seq][head]: kept positions with that key, the first ones
    int2 *before;    // [seq][head][nch]: (keys above thr, keys equal to it) before the chunk
};

// n entries, of which the last `recent` always stay and `need` of the `old`
// ones before them do.
struct EvictPlan {
    int n, kept, old, need;
};

__device__ __forceinline__ EvictPlan evict_plan(const EvictArgs &a, int b) {
    EvictPlan e;
    e.n = a.lengths[b];
    if (e.n < 0 || (int64_t)e.n > ((int64_t)a.max_pages << a.p.lp)) {
        if (threadIdx.x == 0) atomicOr(&g_pool_error, 4u);
        e.n = 0;
    }
    e.kept = min(e.n, a.budget);
    const int rec = min(a.recent, e.kept);
    e.old = e.n - rec;
    e.need = e.kept - rec;
    return e;
}

__device__ __forceinline__ uint32_t evict_key(const EvictArgs &a, const int32_t *pages, int h, int t) {
    const int32_t ts = a.p.token_slot(pages, t);
    return ts < 0 ? 0u : float_key(a.p.mass[a.p.slot(ts, h)]);
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(EvictArgs a) {
    __shared__ int hist[kBins];
    __shared__ int part[33];
    __shared__ int s_bin, s_above;
    const int b = blockIdx.y, h = blockIdx.x, tid = threadIdx.x;
    const EvictPlan e = evict_plan(a, b);
    const int32_t *pages = a.pages + (int64_t)b * a.max_pages;
    if (h == 0 && tid == 0) a.new_lengths[b] = e.kept;
    const int64_t bh = (int64_t)b * a.p.H + h;
    if (e.need == e.old) return;  // everything stays
    uint32_t prefix = 0;
    int need = e.need;
    if (need > 0) {
        for (int d = 0; d < kDigits; ++d) {
            for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
            __syncthreads();
            for (int t = tid; t < e.old; t += kSelThreads) {
                const uint32_t key = evict_key(a, pages, h, t);
                if (digit_in(key, prefix, d)) atomicAdd(&hist[(key >> digit_shift(d)) & digit_mask(d)], 1);
            }
            __syncthreads();
            find_bin_from_top(hist, need, part, &s_bin, &s_above);
            prefix |= (uint32_t)s_bin << digit_shift(d);
            need -= s_above;
            __syncthreads();
        }
    } else {
        prefix = 0xFFFFFFFFu;  // no float has this key
    }
    if (tid == 0) {
        a.thr[bh] = prefix;
        a.ties[bh] = need;
    }
    // chunk totals, a warp per chunk, then their running sums
    int2 *before = a.before + bh * a.nch;
    const int warp = tid >> 5, lane = tid & 31;
    const int nch = (e.n + kMoveChunk - 1) / kMoveChunk;
    for (int c = warp; c < nch; c += kSelThreads / 32) {
        int gt = 0, eq = 0;
        for (int i = 0; i < kMoveChunk; i += 32) {
            const int t = c * kMoveChunk + i + lane;
            const uint32_t key = t < e.old ? evict_key(a, pages, h, t) : 0u;
            gt += __popc(__ballot_sync(0xffffffffu, t < e.old && key > prefix));
            eq += __popc(__ballot_sync(0xffffffffu, t < e.old && key == prefix));
        }
        if (lane == 0) before[c] = make_int2(gt, eq);
    }
    __syncthreads();
    int carry_gt = 0, carry_eq = 0;
    for (int c0 = 0; c0 < nch; c0 += kSelThreads) {
        const int c = c0 + tid;
        const int2 v = c < nch ? before[c] : make_int2(0, 0);
        int tg, te;
        const int g = block_exclusive(v.x, part, &tg);
        __syncthreads();
        const int q = block_exclusive(v.y, part, &te);
        __syncthreads();
        if (c < nch) before[c] = make_int2(carry_gt + g, carry_eq + q);
        carry_gt += tg;
        carry_eq += te;
    }
}

__global__ void __launch_bounds__(kMoveChunk) evict_move_kernel(EvictArgs a) {
    __shared__ int part[33];
    __shared__ int64_t s_src[kMoveChunk], s_dst[kMoveChunk];
    const int b = blockIdx.z, h = blockIdx.y, c = blockIdx.x, tid = threadIdx.x;
    const EvictPlan e = evict_plan(a, b);
    const int t = c * kMoveChunk + tid;
    if (c * kMoveChunk >= e.n) return;
    const int32_t *pages = a.pages + (int64_t)b * a.max_pages;
    const int64_t bh = (int64_t)b * a.p.H + h;
    int32_t ts = -1;
    if (t < e.n) ts = a.p.token_slot(pages, t);
    int at = -1;  // place among the kept
    if (e.need == e.old) {
        if (t < e.n) at = t;
    } else {
        const uint32_t thr = a.thr[bh];
        const int ties = a.ties[bh];
        const int2 before = a.before[bh * a.nch + c];
        const bool old = t < e.old;
        const uint32_t key = old && ts >= 0 ? float_key(a.p.mass[a.p.slot(ts, h)]) : 0u;
        int total;
        const int eq = before.y + block_exclusive((int)(old && key == thr), part, &total);
        __syncthreads();
        const bool keep = t < e.n && (!old || key > thr || (key == thr && eq < ties));
        const int rank = block_exclusive((int)keep, part, &total);
        // kept before the chunk: keys above the threshold, the first ties, and
        // (in the last chunks) entries past `old`
        const int past = max(0, c * kMoveChunk - e.old);
        if (keep) at = before.x + min(before.y, ties) + past + rank;
    }
    int64_t src = -1, dst = -1;
    if (at >= 0) {
        const int32_t td = a.p.token_slot(a.dst_pages + (int64_t)b * a.dst_max_pages, at);
        if (ts < 0 || td < 0) {
            atomicOr(&g_pool_error, 4u);
        } else {
            src = a.p.slot(ts, h);
            dst = a.p.slot(td, h);
        }
    }
    s_src[tid] = src;
    s_dst[tid] = dst;
    if (src >= 0) {
        a.p.kz[dst] = a.p.kz[src];
        a.p.vz[dst] = a.p.vz[src];
        a.p.mass[dst] = a.p.mass[src];
    }
    __syncthreads();
    // code records (G 16-byte pieces of K and of V) and scales, neighbouring
    // threads on neighbouring pieces of an entry
    const int G = a.p.G;
    uint4 *kc = reinterpret_cast<uint4 *>(a.p.kc), *vc = reinterpret_cast<uint4 *>(a.p.vc);
    for (int i = tid; i < kMoveChunk * G; i += kMoveChunk) {
        const int s = i / G, g = i - s * G;
        const int64_t from = s_src[s], to = s_dst[s];
        if (from >= 0) {
            kc[to * G + g] = kc[from * G + g];
            vc[to * G + g] = vc[from * G + g];
            a.p.ks[to * G + g] = a.p.ks[from * G + g];
            a.p.vs[to * G + g] = a.p.vs[from * G + g];
        }
    }
}

int64_t evict_chunks(int64_t positions) { return cdiv(positions, kMoveChunk); }

}  // namespace

spectra_status launch_pool_append(const spectra_kv_pool &pool, const uint16_t *k, const uint16_t *v,
                                  int n_tok, int64_t k_stride, int64_t v_stride, const int32_t *slots,
                                  cudaStream_t s) {
    const PoolView p = PoolView::of(pool);
    const int64_t items = (int64_t)n_tok * 2 * p.H;
    const int64_t warps = cdiv(items, 32 / (4 * p.G));
    pool_append_kernel<<<(unsigned)cdiv(warps * 32, 256), 256, 0, s>>>(p, k, v, k_stride, v_stride, slots, items);
    return cudaGetLastError() == cudaSuccess ? SPECTRA_OK : SPECTRA_ERR_CUDA;
}

spectra_status launch_pool_read(const spectra_kv_pool &pool, const int32_t *slots, int n, void *k_out,
                                void *v_out, bool bf16, cudaStream_t s) {
    const PoolView p = PoolView::of(pool);
    const int64_t threads = (int64_t)n * p.H * 4 * p.G;
    const unsigned grid = (unsigned)cdiv(threads, 256);
    if (bf16) pool_read_kernel<true><<<grid, 256, 0, s>>>(p, slots, threads, k_out, v_out);
    else pool_read_kernel<false><<<grid, 256, 0, s>>>(p, slots, threads, k_out, v_out);
    return cudaGetLastError() == cudaSuccess ? SPECTRA_OK : SPECTRA_ERR_CUDA;
}

size_t evict_workspace_bytes(int n_seq, int n_heads, int64_t positions) {
    const size_t bh = (size_t)n_seq * n_heads;
    return bh * 8 + bh * (size_t)evict_chunks(positions) * sizeof(int2) + 8;
}

spectra_status launch_evict(const spectra_kv_pool &pool, const int32_t *pages, int max_pages,
                            const int32_t *lengths, int n_seq, const int32_t *dst_pages,
                            int dst_max_pages, int budget, int recent, int32_t *new_lengths, void *ws,
                            cudaStream_t s) {
    EvictArgs a;
    a.p = PoolView::of(pool);
    a.pages = pages;
    a.dst_pages = dst_pages;
    a.lengths = lengths;
    a.new_lengths = new_lengths;
    a.max_pages = max_pages;
    a.dst_max_pages = dst_max_pages;
    a.budget = budget;
    a.recent = recent;
    a.nch = (int)evict_chunks((int64_t)max_pages << a.p.lp);
    const size_t bh = (size_t)n_seq * a.p.H;
    a.before = static_cast<int2 *>(ws);
    a.thr = reinterpret_cast<uint32_t *>(a.before + bh * a.nch);
    a.ties = reinterpret_cast<int *>(a.thr + bh);
    evict_select_kernel<<<dim3((unsigned)a.p.H, (unsigned)n_seq), kSelThreads, 0, s>>>(a);
    if (cudaGetLastError() != cudaSuccess) return SPECTRA_ERR_CUDA;
    evict_move_kernel<<<dim3((unsigned)a.nch, (unsigned)a.p.H, (unsigned)n_seq), kMoveChunk, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? SPECTRA_OK : SPECTRA_ERR_CUDA;
}

spectra_status pool_device_error(unsigned int *bits, cudaStream_t s) {
    unsigned int v = 0;
    if (cudaMemcpyFromSymbolAsync(&v, g_pool_error, sizeof v, 0, cudaMemcpyDeviceToHost, s) != cudaSuccess)
        return SPECTRA_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return SPECTRA_ERR_CUDA;
    *bits = v;
    if (v != 0) {
        const unsigned int zero = 0;
        if (cudaMemcpyToSymbolAsync(g_pool_error, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, s) != cudaSuccess ||
            cudaStreamSynchronize(s) != cudaSuccess)
            return SPECTRA_ERR_CUDA;
    }
    return SPECTRA_OK;
}

}  // namespace spectra
