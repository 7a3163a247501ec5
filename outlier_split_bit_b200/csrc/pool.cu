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

// N words to or from p, in the widest pieces that N words lie aligned for.
template <int N>
__device__ __forceinline__ void store_words(uint32_t *p, const uint32_t (&r)[N]) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) *reinterpret_cast<uint4 *>(p + i) = make_uint4(r[i], r[i + 1], r[i + 2], r[i + 3]);
    } else if constexpr (N % 2 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 2) *reinterpret_cast<uint2 *>(p + i) = make_uint2(r[i], r[i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) p[i] = r[i];
    }
}
template <int N>
__device__ __forceinline__ void read_words(uint32_t (&r)[N], const uint32_t *p) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p + i);
            r[i] = v.x; r[i + 1] = v.y; r[i + 2] = v.z; r[i + 3] = v.w;
        }
    } else if constexpr (N % 2 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const uint2 v = *reinterpret_cast<const uint2 *>(p + i);
            r[i] = v.x; r[i + 1] = v.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) r[i] = p[i];
    }
}

// bit 0: a non-finite value was appended; bit 1: a group's scale overflowed
// FP16; bit 2: a slot or page outside the pool.
__device__ unsigned int g_pool_error;

// Four threads hold one vector (a token's K or V of one head): thread w the
// channels 32g + 8w .. +7 of every group g, so its codes are the pool's word w
// of every group, G words that lie together (V: halfwords 2w and 2w + 1, the
// same bytes).
//
// A group's minimum and maximum take two shuffles; its scale and zero point
// are found by one of the four threads (group g by thread g % 4) and handed
// round.  The arithmetic is quant.cuh's, bit for bit, without its divisions:
//
// Scale, RN16((hi - lo) / 15): where hi - lo is exact in FP32 (d, checked by
// taking it apart again), the FP32 quotient q = RN(d / 15) rounds to FP16 as
// d / 15 does.  It would not only if q fell on a midpoint of FP16 that d / 15
// is not on; but a midpoint m has 12 bits, 15 m is a multiple of d's last
// place u (or of a larger power of two), so |d / 15 - m| >= u / 15, and that
// is more than q's half step, u / 16 at most.  Otherwise the double quotient
// is taken.
//
// Codes, rint(v / S): q = v * (1 / S) in FP32 is off by 2^-18 at most where |q|
// is 32 or less; beyond, where it may reach 15 * 2^9 (two different BF16 values
// near v differ by 2^-8 |v| or more, and S is 1/15 of that, or half of it where S
// is subnormal), the code is 0 or 15 either way.  A true quotient
// that is not k + 1/2 lies 2^-12 or more from it: 2v - (2k+1)S is a multiple of
// the smaller of S's last place (2^-10 of S or more, or S / j for a subnormal
// S = j 2^-24) and 2v's (2^-8 of S or more, near a tie).  So 2q within 2^-12 of
// a whole number means that 2v / S is that number, or near an even one, where
// it makes no difference; q is set to it, and rounding half to even gives the
// double quotient's result.
//
// Measured (B200): 8192 tokens of 8 heads of 128, K and V, 33.5 MB read and 10.5
// written, 13 us, 3.4 TB/s, bound by the codec's instructions (minima and maxima in
// FP32 instead of BF16 pairs: 16 us); one token of 2 heads 2.3 us, its launch.
constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: a float sum with it is a whole number

__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t x) { return *reinterpret_cast<const __nv_bfloat162 *>(&x); }

__device__ __forceinline__ uint32_t group_scale(float lo, float hi, float *zero_out, unsigned int *flags) {
    const bool bad = !(isfinite(lo) && isfinite(hi));
    const float d = hi - lo;
    unsigned short s;
    if (hi - d == lo && d + lo == hi && d < 3e38f) {
        s = __half_as_ushort(__float2half_rn(__fdiv_rn(d, 15.f)));
    } else {
        const double q15 = __ddiv_rn(__dsub_rn((double)hi, (double)lo), 15.0);
        asm("cvt.rn.f16.f64 %0, %1;" : "=h"(s) : "d"(q15));
    }
    if (bad) {
        *flags |= 1u;
        s = 0;  // the group is stored as zeros
    } else if ((s & 0x7FFFu) == 0x7C00u) {
        *flags |= 2u;
        s = 0;
    }
    const float S = __half2float(__ushort_as_half(s));
    float z = 0.f;
    if (S != 0.f) z = fminf(fmaxf(rintf(__fdiv_rn(-lo, S)), 0.f), 15.f);
    *zero_out = z;
    return s;
}

template <int G>
__global__ void __launch_bounds__(256) pool_append_kernel(PoolView p, const uint16_t *__restrict__ k,
                                                          const uint16_t *__restrict__ v, int64_t k_stride,
                                                          int64_t v_stride, const int32_t *__restrict__ slots,
                                                          uint32_t n_vectors) {
    const uint32_t i = (blockIdx.x * 256u + threadIdx.x) >> 2;  // token * H + head
    const int w = threadIdx.x & 3, lane = threadIdx.x & 31, which = blockIdx.y;
    const bool in = i < n_vectors;
    const uint32_t tok = in ? i / (uint32_t)p.H : 0, h = in ? i - tok * (uint32_t)p.H : 0;
    int32_t ts = in ? slots[tok] : -1;
    if (ts >= p.token_slots()) {
        atomicOr(&g_pool_error, 4u);
        ts = -1;
    }
    const uint16_t *src = (which ? v + tok * v_stride : k + tok * k_stride) + h * 32 * G + 8 * w;
    uint4 raw[G];
#pragma unroll
    for (int g = 0; g < G; ++g)
        raw[g] = ts >= 0 ? __ldg(reinterpret_cast<const uint4 *>(src + 32 * g)) : make_uint4(0u, 0u, 0u, 0u);
    // minimum and maximum in BF16 pairs (of the two zeros either may come out,
    // which makes no difference below); a NaN stays one
    float lo[G], hi[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const uint32_t r4[4] = {raw[g].x, raw[g].y, raw[g].z, raw[g].w};
        __nv_bfloat162 l = as_bf162(r4[0]), u = l;
#pragma unroll
        for (int j = 1; j < 4; ++j) {
            l = __hmin2_nan(l, as_bf162(r4[j]));
            u = __hmax2_nan(u, as_bf162(r4[j]));
        }
        // the two halves, then the four threads: minimum in the lower half, maximum in the upper
        __nv_bfloat162 both = __halves2bfloat162(__hmin_nan(__low2bfloat16(l), __high2bfloat16(l)),
                                                 __hmax_nan(__low2bfloat16(u), __high2bfloat16(u)));
#pragma unroll
        for (int o = 1; o <= 2; o <<= 1) {
            const uint32_t mine = *reinterpret_cast<const uint32_t *>(&both);
            const __nv_bfloat162 other = as_bf162(__shfl_xor_sync(0xffffffffu, mine, o));
            both = __halves2bfloat162(__hmin_nan(__low2bfloat16(both), __low2bfloat16(other)),
                                      __hmax_nan(__high2bfloat16(both), __high2bfloat16(other)));
        }
        lo[g] = __low2float(both);
        hi[g] = __high2float(both);
    }
    constexpr int kOwn = (G + 3) / 4;  // groups of a thread's own: w, w + 4
    float own_z[kOwn];
    uint32_t own_s[kOwn];
    unsigned int flags = 0;
#pragma unroll
    for (int e = 0; e < kOwn; ++e) {
        float l = lo[4 * e], u = hi[4 * e];
#pragma unroll
        for (int j = 1; j < 4; ++j)
            if (4 * e + j < G && w == j) {
                l = lo[4 * e + j];
                u = hi[4 * e + j];
            }
        own_s[e] = group_scale(l, u, &own_z[e], &flags);
    }
    if (flags && ts >= 0) atomicOr(&g_pool_error, flags);
    uint32_t word[G], sc[G], zw = 0;
#pragma unroll
    for (int g = 0; g < G; ++g) {
        sc[g] = __shfl_sync(0xffffffffu, own_s[g / 4], (lane & ~3) + (g & 3));
        const int z = (int)__shfl_sync(0xffffffffu, own_z[g / 4], (lane & ~3) + (g & 3));
        zw |= (uint32_t)z << (4 * g);
        const float S = __half2float(__ushort_as_half((unsigned short)sc[g]));
        const float r2 = S != 0.f ? __fdiv_rn(2.f, S) : 0.f;  // 0: codes 0 below (z is 0, and every q)
        const uint32_t r4[4] = {raw[g].x, raw[g].y, raw[g].z, raw[g].w};
        uint32_t c8 = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float x = __uint_as_float(j & 1 ? r4[j >> 1] & 0xFFFF0000u : r4[j >> 1] << 16);
            const float q2 = x * r2;
            const float near = (q2 + kMagic) - kMagic;
            const float q = (fabsf(q2 - near) < 0x1p-12f ? near : q2) * 0.5f;
            const int c = __float_as_int(q + kMagic) - __float_as_int(kMagic) + z;
            c8 |= (uint32_t)min(max(c, 0), 15) << (4 * j);
        }
        word[g] = sc[g] ? c8 : 0u;  // (a bad group's values are NaN here)
    }
    if (ts < 0) return;
    const int64_t slot = p.slot(ts, (int)h);
    if (which) {
        // halfwords 2w and 2w + 1 of every group: G and G of them
        uint32_t v16[G];
#pragma unroll
        for (int e = 0; e < 2 * G; ++e) {
            const uint32_t half = e < G ? word[e] & 0xFFFFu : word[e - G] >> 16;
            if (e & 1) v16[e / 2] |= half << 16;
            else v16[e / 2] = half;
        }
        store_words<G>(reinterpret_cast<uint32_t *>(p.vc + slot * 8 * G + 2 * w * G), v16);
    } else {
        store_words<G>(p.kc + slot * 4 * G + w * G, word);
    }
    if (w == 0) {
        uint16_t *s = (which ? p.vs : p.ks) + slot * G;
        if constexpr (G % 2 == 0) {
            uint32_t pair[G / 2];
#pragma unroll
            for (int g = 0; g < G; g += 2) pair[g / 2] = sc[g] | sc[g + 1] << 16;
            store_words<G / 2>(reinterpret_cast<uint32_t *>(s), pair);
        } else {
#pragma unroll
            for (int g = 0; g < G; ++g) s[g] = (uint16_t)sc[g];
        }
    }
    if (w == 1) (which ? p.vz : p.kz)[slot] = zw;
    if (w == 2 && which == 0 && p.mass) p.mass[slot] = 0.f;
}

// Token slots dequantised, four threads to a vector as above.  Bound by the
// writes: 36000 tokens of 8 heads of 128 to BF16 in 32 us, 44 MB of records read
// and 147 written; to FP32 in 77 us, 295 written.
template <int G, bool BF16>
__global__ void __launch_bounds__(256) pool_read_kernel(PoolView p, const int32_t *__restrict__ slots,
                                                        uint32_t n_vectors, void *__restrict__ k_out,
                                                        void *__restrict__ v_out) {
    const uint32_t i = (blockIdx.x * 256u + threadIdx.x) >> 2;
    const int w = threadIdx.x & 3, which = blockIdx.y;
    void *out = which ? v_out : k_out;
    if (i >= n_vectors || !out) return;
    const uint32_t tok = i / (uint32_t)p.H, h = i - tok * (uint32_t)p.H;
    int32_t ts = slots[tok];
    if (ts >= p.token_slots()) {
        atomicOr(&g_pool_error, 4u);
        ts = -1;
    }
    uint32_t word[G], s[G], zw = 0;
#pragma unroll
    for (int g = 0; g < G; ++g) word[g] = s[g] = 0;
    if (ts >= 0) {
        const int64_t slot = p.slot(ts, (int)h);
        zw = (which ? p.vz : p.kz)[slot];
        const uint16_t *sp = (which ? p.vs : p.ks) + slot * G;
        if constexpr (G % 2 == 0) {
            uint32_t pair[G / 2];
            read_words<G / 2>(pair, reinterpret_cast<const uint32_t *>(sp));
#pragma unroll
            for (int g = 0; g < G; ++g) s[g] = g & 1 ? pair[g / 2] >> 16 : pair[g / 2] & 0xFFFFu;
        } else {
#pragma unroll
            for (int g = 0; g < G; ++g) s[g] = sp[g];
        }
        if (which) {
            uint32_t v16[G];
            read_words<G>(v16, reinterpret_cast<const uint32_t *>(p.vc + slot * 8 * G + 2 * w * G));
#pragma unroll
            for (int e = 0; e < 2 * G; ++e) {
                const uint32_t half = e & 1 ? v16[e / 2] >> 16 : v16[e / 2] & 0xFFFFu;
                if (e < G) word[e] = half;
                else word[e - G] |= half << 16;
            }
        } else {
            read_words<G>(word, p.kc + slot * 4 * G + w * G);
        }
    }
    const int64_t at = (int64_t)i * 32 * G + 8 * w;
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const float S = __half2float(__ushort_as_half((unsigned short)s[g]));
        const float z = (float)((zw >> (4 * g)) & 15u);
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = ((float)((word[g] >> (4 * j)) & 15u) - z) * S;
        if (BF16) {
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[j]) : "f"(x[2 * j + 1]), "f"(x[2 * j]));
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + at + 32 * g) = make_uint4(o[0], o[1], o[2], o[3]);
        } else {
            float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(out) + at + 32 * g);
            o[0] = make_float4(x[0], x[1], x[2], x[3]);
            o[1] = make_float4(x[4], x[5], x[6], x[7]);
        }
    }
}

// ---- eviction ----
// Two launches: select (one CTA per sequence and head) finds the smallest kept
// key and lists the kept positions; move (launched as a programmatic dependent)
// copies their entries to the fresh pages, an entry's pieces by neighbouring
// threads.  Select reads every weight once, through the page table with eight
// look-ups in flight per thread, and keeps the keys in shared memory (of the first
// kKeys positions; what lies past them is read again in each pass).
//
// The smallest kept key is found by counting in 2048 bins over the keys' range
// (from the smallest positive one: zeros, of positions that no query has seen,
// would stretch it over all exponents), then in the bin it lies in; a bin of at
// most kSelList keys is ranked all pairs.  Few keys share a bin, so the counters'
// atomics seldom meet (with the key's upper 11 bits as the bin, and three passes: 53
// us where this takes 50).
//
// Measured (B200): 1 sequence of 8192 positions, 2 heads of 128, 2048 kept: 15 us,
// latency (select's chain of look-ups, passes and barriers is 10 of them).  24 of
// 5000, 8 heads, 1500 kept: 38 us; move takes 22 of them for 90 MB read (45 of
// entries: an entry's scales, zero points and weight fill 36 of the 160 bytes in
// their sectors) and 45 MB written, 6.1 TB/s, select the rest.  Without the list,
// move looking at every position's weight again: 50 us.
constexpr int kKeys = 55296;  // 216 KB of an SM's 227
constexpr int kLookUps = 8;
constexpr int kSelList = 256;
constexpr int kBinBits = 11;               // of kBins
constexpr uint32_t kZeroKey = 0x80000000u;  // float_key(0)
constexpr int kMoveThreads = 256;
constexpr int kMoveChunk = 128;            // kept entries of a move CTA

struct EvictArgs {
    PoolView p;
    const int32_t *pages;
    const int32_t *dst_pages;
    const int32_t *lengths;
    int32_t *new_lengths;
    int max_pages, dst_max_pages, budget, recent, room;
    int32_t *list;   // [seq][head][room]: the kept ones of the `old` positions, in order
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

template <int T>
__global__ void __launch_bounds__(T) evict_select_kernel(EvictArgs a) {
    extern __shared__ uint32_t keys[];
    __shared__ int hist[kBins];
    __shared__ int part[33];
    __shared__ int s_bin, s_above, s_listed, s_ties;
    __shared__ int2 s_counts[T / 32];
    __shared__ uint32_t list[kSelList], s_min, s_max, s_over_zero, s_thr;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int b = blockIdx.y, h = blockIdx.x, tid = threadIdx.x;
    const EvictPlan e = evict_plan(a, b);
    const int32_t *pages = a.pages + (int64_t)b * a.max_pages;
    if (h == 0 && tid == 0) a.new_lengths[b] = e.kept;
    const int64_t bh = (int64_t)b * a.p.H + h;
    if (e.need == e.old) return;  // everything stays
    const int cached = min(e.old, kKeys);
    if (tid == 0) {
        s_min = s_over_zero = 0xFFFFFFFFu;
        s_max = 0;
    }
    __syncthreads();
    uint32_t least = 0xFFFFFFFFu, most = 0, over_zero = 0xFFFFFFFFu;
    auto seen = [&](uint32_t key) {
        least = min(least, key);
        most = max(most, key);
        if (key > kZeroKey) over_zero = min(over_zero, key);
    };
    for (int t0 = tid; t0 < cached; t0 += kLookUps * T) {
        int32_t ts[kLookUps];
        float m[kLookUps];
#pragma unroll
        for (int j = 0; j < kLookUps; ++j) {
            const int t = t0 + j * T;
            ts[j] = t < cached ? a.p.token_slot(pages, t) : -1;
        }
#pragma unroll
        for (int j = 0; j < kLookUps; ++j) m[j] = ts[j] >= 0 ? a.p.mass[a.p.slot(ts[j], h)] : 0.f;
#pragma unroll
        for (int j = 0; j < kLookUps; ++j)
            if (t0 + j * T < cached) {
                const uint32_t key = ts[j] >= 0 ? float_key(m[j]) : 0u;
                keys[t0 + j * T] = key;
                seen(key);
            }
    }
    auto key_at = [&](int t) { return t < cached ? keys[t] : evict_key(a, pages, h, t); };
    uint32_t thr = 0xFFFFFFFFu;  // no float has this key
    int need = e.need;  // (of the threshold's own, in the end: the first ones stay)
    if (need > 0) {
        least = __reduce_min_sync(0xffffffffu, least);
        most = __reduce_max_sync(0xffffffffu, most);
        over_zero = __reduce_min_sync(0xffffffffu, over_zero);
        if ((tid & 31) == 0) {
            atomicMin(&s_min, least);
            atomicMax(&s_max, most);
            atomicMin(&s_over_zero, over_zero);
        }
        __syncthreads();
        // the threshold lies in [lo, hi]; bins of 2^shift keys from base to top,
        // what lies under base in the first, over top in the last
        const bool all = cached == e.old;
        uint32_t lo = all ? s_min : 0, hi = all ? s_max : 0xFFFFFFFFu, top = s_max, base = min(s_over_zero, top);
        // (the first bins, then 32 bits of a key, 11 at a time: 4 passes at most)
        for (int pass = 0; lo < hi && pass < 5; ++pass) {
            const int shift = max(0, 32 - kBinBits - __clz(top - base));
            const uint32_t last = (top - base) >> shift;
            for (int i = tid; i < kBins; i += T) hist[i] = 0;
            if (tid == 0) s_listed = 0;
            __syncthreads();
#pragma unroll 4
            for (int t = tid; t < e.old; t += T) {
                const uint32_t key = key_at(t);
                if (lo <= key && key <= hi) atomicAdd(&hist[key > base ? min((key - base) >> shift, last) : 0], 1);
            }
            __syncthreads();
            find_bin_from_top(hist, need, part, &s_bin, &s_above);
            const uint32_t bin = (uint32_t)s_bin;
            const int in_bin = hist[bin];
            need -= s_above;
            if (bin != last) hi = base + ((bin + 1) << shift) - 1;
            if (bin != 0) lo = base + (bin << shift);
            base = lo;
            top = hi;
            if (in_bin <= kSelList) {
                for (int t = tid; t < e.old; t += T) {
                    const uint32_t key = key_at(t);
                    if (lo <= key && key <= hi) {
                        const int at = atomicAdd(&s_listed, 1);
                        if (at < kSelList) list[at] = key;  // always, unless the weights change meanwhile
                    }
                }
                __syncthreads();
                if (tid < in_bin) {
                    const uint32_t key = list[tid];
                    int over = 0, equal = 0;
#pragma unroll 8
                    for (int i = 0; i < in_bin; ++i) {
                        over += list[i] > key;
                        equal += list[i] == key;
                    }
                    if (over < need && need <= over + equal) {  // (equal keys write the same)
                        s_thr = key;
                        s_ties = need - over;
                    }
                }
                __syncthreads();
                lo = hi = s_thr;
                need = s_ties;
            }
            __syncthreads();
        }
        thr = lo;
    } else {
        return;  // the recent ones alone
    }
    // the list: a warp takes a part of the positions, counts its keys over the
    // threshold and at it, and after the warps before it writes its own
    int32_t *list_out = a.list + bh * a.room;
    const int warp = tid >> 5, lane = tid & 31;
    const int per = (e.old + T - 1) / T * 32;
    const int t0 = warp * per, t1 = min(e.old, t0 + per);
    int over = 0, equal = 0;
#pragma unroll 4
    for (int t = t0; t < t1; t += 32) {
        const uint32_t key = t + lane < t1 ? key_at(t + lane) : 0u;
        over += __popc(__ballot_sync(0xffffffffu, t + lane < t1 && key > thr));
        equal += __popc(__ballot_sync(0xffffffffu, t + lane < t1 && key == thr));
    }
    if (lane == 0) s_counts[warp] = make_int2(over, equal);
    __syncthreads();
    const int2 all_counts = lane < T / 32 ? s_counts[lane] : make_int2(0, 0);
    over = __shfl_sync(0xffffffffu, warp_exclusive(all_counts.x, lane), warp);
    equal = __shfl_sync(0xffffffffu, warp_exclusive(all_counts.y, lane), warp);
    const uint32_t below = (1u << lane) - 1;
#pragma unroll 4
    for (int t = t0; t < t1; t += 32) {
        const bool in = t + lane < t1;
        const uint32_t key = in ? key_at(t + lane) : 0u;
        const uint32_t gt = __ballot_sync(0xffffffffu, in && key > thr), eq = __ballot_sync(0xffffffffu, in && key == thr);
        const int ties = equal + __popc(eq & below);
        const bool keep = in && (key > thr || (key == thr && ties < need));
        // (a place over the list's end: the weights were changed meanwhile)
        const int place = over + __popc(gt & below) + min(ties, need);
        if (keep && place < e.need) list_out[place] = t + lane;
        over += __popc(gt);
        equal += __popc(eq);
    }
}

template <int G>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(EvictArgs a) {
    __shared__ int64_t s_src[kMoveChunk], s_dst[kMoveChunk];
    const int b = blockIdx.z, h = blockIdx.y, tid = threadIdx.x;
    const EvictPlan e = evict_plan(a, b);
    const int32_t *src_pages = a.pages + (int64_t)b * a.max_pages, *dst_pages = a.dst_pages + (int64_t)b * a.dst_max_pages;
    const int32_t *list = a.list + ((int64_t)b * a.p.H + h) * a.room;
    for (int r0 = blockIdx.x * kMoveChunk; r0 < e.kept; r0 += gridDim.x * kMoveChunk) {
    const int rank = r0 + tid, total = min(kMoveChunk, e.kept - r0);
    const int32_t td = tid < total ? a.p.token_slot(dst_pages, rank) : -1;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // select's lists; nothing was written before
    if (tid < total) {
        int t = rank;  // everything stays
        if (e.need != e.old) t = rank < e.need ? list[rank] : e.old + rank - e.need;
        const int32_t ts = (uint32_t)t < (uint32_t)e.n ? a.p.token_slot(src_pages, t) : -1;
        int64_t src = -1, dst = -1;
        if (ts < 0 || td < 0) {
            atomicOr(&g_pool_error, 4u);
        } else {
            src = a.p.slot(ts, h);
            dst = a.p.slot(td, h);
            a.p.kz[dst] = a.p.kz[src];
            a.p.vz[dst] = a.p.vz[src];
            a.p.mass[dst] = a.p.mass[src];
        }
        s_src[tid] = src;
        s_dst[tid] = dst;
    }
    __syncthreads();
    // code records, G 16-byte pieces of K and of V, and scales: neighbouring
    // threads on neighbouring pieces of an entry
    uint4 *kc = reinterpret_cast<uint4 *>(a.p.kc), *vc = reinterpret_cast<uint4 *>(a.p.vc);
#pragma unroll 2
    for (int i = tid; i < total * G; i += kMoveThreads) {
        const int s = i / G, g = i - s * G;
        const int64_t from = s_src[s] * G + g, to = s_dst[s] * G + g;
        if (to >= 0) {
            const uint4 x = kc[from], y = vc[from];
            const uint16_t u = a.p.ks[from], v = a.p.vs[from];
            kc[to] = x;
            vc[to] = y;
            a.p.ks[to] = u;
            a.p.vs[to] = v;
        }
    }
    __syncthreads();
    }
    // a CTA without entries waits too: this grid's end stands for select's, whose
    // lengths the next kernel of the stream may read
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

}  // namespace

// The kernels' G, from the pool's head_dim.
#define SPECTRA_POOL_GROUPS(G_, CALL)    \
    switch (G_) {                        \
        case 1: CALL(1); break;          \
        case 2: CALL(2); break;          \
        case 3: CALL(3); break;          \
        case 4: CALL(4); break;          \
        case 5: CALL(5); break;          \
        case 6: CALL(6); break;          \
        case 7: CALL(7); break;          \
        default: CALL(8); break;         \
    }

spectra_status launch_pool_append(const spectra_kv_pool &pool, const uint16_t *k, const uint16_t *v,
                                  int n_tok, int64_t k_stride, int64_t v_stride, const int32_t *slots,
                                  cudaStream_t s) {
    const PoolView p = PoolView::of(pool);
    const uint32_t n = (uint32_t)n_tok * (uint32_t)p.H;
    const dim3 grid((unsigned)cdiv((int64_t)n * 4, 256), 2);
#define SPECTRA_CALL(G) pool_append_kernel<G><<<grid, 256, 0, s>>>(p, k, v, k_stride, v_stride, slots, n)
    SPECTRA_POOL_GROUPS(p.G, SPECTRA_CALL)
#undef SPECTRA_CALL
    return cudaGetLastError() == cudaSuccess ? SPECTRA_OK : SPECTRA_ERR_CUDA;
}

spectra_status launch_pool_read(const spectra_kv_pool &pool, const int32_t *slots, int n_tok, void *k_out,
                                void *v_out, bool bf16, cudaStream_t s) {
    const PoolView p = PoolView::of(pool);
    const uint32_t n = (uint32_t)n_tok * (uint32_t)p.H;
    const dim3 grid((unsigned)cdiv((int64_t)n * 4, 256), 2);
#define SPECTRA_CALL(G)                                                                         \
    if (bf16) pool_read_kernel<G, true><<<grid, 256, 0, s>>>(p, slots, n, k_out, v_out);        \
    else pool_read_kernel<G, false><<<grid, 256, 0, s>>>(p, slots, n, k_out, v_out)
    SPECTRA_POOL_GROUPS(p.G, SPECTRA_CALL)
#undef SPECTRA_CALL
    return cudaGetLastError() == cudaSuccess ? SPECTRA_OK : SPECTRA_ERR_CUDA;
}

size_t evict_workspace_bytes(int n_seq, int n_heads, int64_t positions, int budget) {
    return (size_t)n_seq * n_heads * (size_t)(positions < budget ? positions : budget) * 4 + 16;
}

spectra_status launch_evict(const spectra_kv_pool &pool, const int32_t *pages, int max_pages,
                            const int32_t *lengths, int n_seq, const int32_t *dst_pages,
                            int dst_max_pages, int budget, int recent, int32_t *new_lengths, void *ws,
                            cudaStream_t s, const DeviceInfo &dev) {
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
    const int64_t longest = (int64_t)max_pages << a.p.lp;
    a.room = (int)(longest < budget ? longest : budget);
    a.list = static_cast<int32_t *>(ws);
    const size_t smem = (size_t)(longest < kKeys ? longest : kKeys) * 4;
    // Threads: one row's chain of passes is shorter with more; with more rows than
    // SMs, smaller CTAs share an SM where their keys leave room (24 sequences of 5000,
    // 8 heads: 43 us with 1024, 38 with 512; 1 of 8192: 14.9 and 17.7).
    const dim3 grid((unsigned)a.p.H, (unsigned)n_seq);
    if ((int64_t)n_seq * a.p.H <= dev.sm_count || smem > 100 * 1024) {
        static std::atomic<uint64_t> ready{0};
        if (allow_smem((const void *)evict_select_kernel<1024>, kKeys * 4, dev, &ready) != cudaSuccess)
            return SPECTRA_ERR_CUDA;
        evict_select_kernel<1024><<<grid, 1024, smem, s>>>(a);
    } else {
        static std::atomic<uint64_t> ready{0};
        if (allow_smem((const void *)evict_select_kernel<512>, kKeys * 4, dev, &ready) != cudaSuccess)
            return SPECTRA_ERR_CUDA;
        evict_select_kernel<512><<<grid, 512, smem, s>>>(a);
    }
    if (cudaGetLastError() != cudaSuccess) return SPECTRA_ERR_CUDA;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    // a few waves of CTAs at most, however large the budget is
    const int64_t chunks = cdiv(a.room, kMoveChunk), per_head = cdiv((int64_t)dev.sm_count * 32, (int64_t)n_seq * a.p.H);
    cfg.gridDim = dim3((unsigned)(per_head < chunks ? per_head : chunks), (unsigned)a.p.H, (unsigned)n_seq);
    cfg.blockDim = dim3(kMoveThreads, 1, 1);
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    cudaError_t err;
#define SPECTRA_CALL(G) err = cudaLaunchKernelEx(&cfg, evict_move_kernel<G>, a)
    SPECTRA_POOL_GROUPS(a.p.G, SPECTRA_CALL)
#undef SPECTRA_CALL
    return err == cudaSuccess ? SPECTRA_OK : SPECTRA_ERR_CUDA;
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
