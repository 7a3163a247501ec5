// sample.cu -- token choice from the LM head's logits (sm_100a).
//
// Per row: w_i = exp((x_i - max) / T); the tokens left after top-k (largest
// value first, ties to the lower index), top-p (a token stays while the
// weight before it, in that order, is under p of the whole) and min-p
// (w_i >= min_p) share the whole again; the choice is the first token, in
// index order, whose running sum passes u of it.
//
// No sort: top-k and top-p keep the keys above a threshold and the first few
// ties of it, and a radix descent over the order-preserving key (three digits
// of 11, 11 and 10 bits) finds the threshold, by counts for top-k and by
// weight for top-p.  Weights are 64-bit fixed point, w * 2^44 rounded from a
// double exponential: integer sums do not depend on their order, so the
// histograms may use atomics and the row repeats bit for bit; a row of up to
// 2^19 tokens cannot overflow, and a token lighter than 2^-45 of the heaviest
// has weight 0.
#include "internal.cuh"
#include "select.cuh"

namespace spectra {
namespace {

// bit 0: a NaN logit; bit 1: a row with nothing to choose from.
__device__ unsigned int g_sample_error;

typedef unsigned long long u64;
constexpr int kThreads = 1024;
constexpr int kFix = 44;
constexpr int kMaxVocab = 1 << 19;
constexpr int kChunks = kMaxVocab / kThreads;  // chunks of one position per thread

struct SampleArgs {
    const float *x;
    const float *u, *temperature, *top_p, *min_p;
    const int32_t *top_k;
    int32_t *ids;
    float *logp;
    int64_t stride;
    int vocab;
};

// floor(f * n) for 0 <= f < 1 (f in steps of 2^-64, which holds every f from
// 2^-40 up exactly); *rest: whether anything was cut off.
__device__ __forceinline__ u64 fraction_of(float f, u64 n, bool *rest) {
    const u64 fx = (u64)((double)f * 18446744073709551616.0);
    *rest = fx * n != 0;
    return __umul64hi(fx, n);
}

__global__ void __launch_bounds__(kThreads) sample_kernel(SampleArgs a) {
    __shared__ u64 hist[kBins];
    __shared__ u64 part[33];
    __shared__ int s_bin, s_pick;
    __shared__ u64 s_above;
    __shared__ float s_max;
    __shared__ u64 sums[kChunks];
    const int row = blockIdx.x, tid = threadIdx.x, V = a.vocab;
    const int lane = tid & 31, warp = tid >> 5;
    const float *x = a.x + (int64_t)row * a.stride;

    // the largest logit, and whether one is NaN
    float mx = -INFINITY;
    bool nan = false;
    for (int i = tid; i < V; i += kThreads) {
        nan |= !(x[i] == x[i]);
        mx = fmaxf(mx, x[i]);
    }
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (nan) atomicOr(&g_sample_error, 1u);
    if (tid == 0) s_pick = V;
    if (lane == 0) part[warp] = float_key(mx);
    __syncthreads();
    if (tid == 0) {
        u64 m = 0;
        for (int i = 0; i < kThreads / 32; ++i) m = part[i] > m ? part[i] : m;
        s_max = key_float((uint32_t)m);
    }
    __syncthreads();
    mx = s_max;
    if (mx == -INFINITY) {
        if (tid == 0) {
            a.ids[row] = -1;
            if (a.logp) a.logp[row] = -INFINITY;
            atomicOr(&g_sample_error, 2u);
        }
        return;
    }
    const float temp = a.temperature ? a.temperature[row] : 1.f;
    if (!(temp > 0.f)) {  // greedy: the first of the largest
        for (int i = tid; i < V; i += kThreads)
            if (x[i] == mx) atomicMin(&s_pick, i);
        __syncthreads();
        if (tid == 0) {
            a.ids[row] = s_pick;
            if (a.logp) a.logp[row] = 0.f;
        }
        return;
    }
    const double t64 = (double)temp, m64 = (double)mx;
    auto weight = [&](float v) -> double {
        if (v == mx) return 1.0;
        return v == v ? exp(((double)v - m64) / t64) : 0.0;
    };
    auto fixed = [&](double w) -> u64 { return (u64)__double2ll_rn(w * (double)(1ll << kFix)); };

    // the smallest kept key, and how many of its ties stay
    uint32_t thr = 0;
    int ties = V;
    const int k = a.top_k ? a.top_k[row] : 0;
    if (k > 0 && k < V) {
        uint32_t prefix = 0;
        u64 need = (u64)k;
        for (int d = 0; d < kDigits; ++d) {
            for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
            __syncthreads();
            for (int i = tid; i < V; i += kThreads) {
                const uint32_t key = float_key(x[i]);
                if (digit_in(key, prefix, d)) atomicAdd(&hist[(key >> digit_shift(d)) & digit_mask(d)], 1ull);
            }
            __syncthreads();
            find_bin_from_top(hist, need, part, &s_bin, &s_above);
            prefix |= (uint32_t)s_bin << digit_shift(d);
            need -= s_above;
            __syncthreads();
        }
        thr = prefix;
        ties = (int)need;
    }
    const float p = a.top_p ? a.top_p[row] : 1.f;
    if (p < 1.f) {
        // the whole of the top-k set: keys above thr, and `ties` of thr's
        uint32_t prefix = 0;
        u64 need = 0, tie_w = 0;
        if (thr > kKeyNegInf) tie_w = fixed(weight(key_float(thr)));
        for (int d = 0; d < kDigits; ++d) {
            for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
            __syncthreads();
            u64 own = 0;
            for (int i = tid; i < V; i += kThreads) {
                const uint32_t key = float_key(x[i]);
                if (key <= kKeyNegInf || key <= thr || !digit_in(key, prefix, d)) continue;
                const u64 q = fixed(weight(x[i]));
                own += q;
                atomicAdd(&hist[(key >> digit_shift(d)) & digit_mask(d)], q);
            }
            if (tid == 0 && thr > kKeyNegInf && digit_in(thr, prefix, d))
                atomicAdd(&hist[(thr >> digit_shift(d)) & digit_mask(d)], tie_w * (u64)ties);
            __syncthreads();
            if (d == 0) {
                u64 total;
                block_exclusive(own, part, &total);
                if (thr > kKeyNegInf) total += tie_w * (u64)ties;
                bool rest = false;
                // kept while before < p * whole: the last kept one is where the
                // running sum reaches ceil(p * whole); the heaviest always stays
                need = p > 0.f ? fraction_of(p, total, &rest) : 0;
                need += rest;
                if (need == 0) need = 1;
                __syncthreads();
            }
            find_bin_from_top(hist, need, part, &s_bin, &s_above);
            prefix |= (uint32_t)s_bin << digit_shift(d);
            need -= s_above;
            __syncthreads();
        }
        const u64 w = fixed(weight(key_float(prefix)));
        const u64 m = (need + w - 1) / w;
        if (prefix == thr) ties = min(ties, (int)m);
        else ties = (int)min(m, (u64)V);
        thr = prefix;
    }
    // the kept weight of each chunk of positions, in index order; ties of thr
    // count from the lowest index
    const double least = a.min_p ? fmin((double)a.min_p[row], 1.0) : 0.0;
    const int nch = (V + kThreads - 1) / kThreads;
    int tie_base = 0;
    auto kept = [&](int i, int *tie_total) -> u64 {
        const float v = i < V ? x[i] : -INFINITY;
        const uint32_t key = i < V ? float_key(v) : 0u;
        const bool tie = i < V && key == thr;
        int rank = 0;
        *tie_total = 0;
        if (__syncthreads_or(tie)) {
            rank = block_exclusive((int)tie, reinterpret_cast<int *>(part), tie_total);
            __syncthreads();
        }
        if (key <= kKeyNegInf || !(key > thr || (tie && tie_base + rank < ties))) return 0;
        const double w = weight(v);
        return w >= least ? fixed(w) : 0;
    };
    u64 total = 0;
    for (int c = 0; c < nch; ++c) {
        int nt;
        const u64 q = kept(c * kThreads + tid, &nt);
        tie_base += nt;
        u64 sum;
        block_exclusive(q, part, &sum);
        __syncthreads();
        if (tid == 0) sums[c] = sum;
        total += sum;
    }
    __syncthreads();
    float u = a.u[row];
    u = u == u ? fminf(fmaxf(u, 0.f), 0.99999994f) : 0.f;
    bool rest;
    const u64 target = fraction_of(u, total, &rest);  // the first running sum over it
    u64 run = 0;
    int c = 0;
    for (; c < nch - 1; ++c) {
        if (run + sums[c] > target) break;
        run += sums[c];
    }
    // ties before this chunk
    tie_base = 0;
    {
        int own = 0;
        for (int i = tid; i < c * kThreads; i += kThreads) own += float_key(x[i]) == thr;
        int all;
        block_exclusive(own, reinterpret_cast<int *>(part), &all);
        __syncthreads();
        tie_base = all;
    }
    int nt;
    const u64 q = kept(c * kThreads + tid, &nt);
    u64 sum;
    const u64 before = run + block_exclusive(q, part, &sum);
    if (q > 0 && before <= target && target < before + q) {
        const int i = c * kThreads + tid;
        a.ids[row] = i;
        const double e = x[i] == mx ? 0.0 : ((double)x[i] - m64) / t64;
        if (a.logp) a.logp[row] = (float)(e - log((double)total / (double)(1ll << kFix)));
    }
}

}  // namespace

int sample_max_vocab() { return kMaxVocab; }

spectra_status launch_sample(const float *logits, int rows, int vocab, int64_t stride, const float *u,
                             const float *temperature, const int32_t *top_k, const float *top_p,
                             const float *min_p, int32_t *ids, float *logp, cudaStream_t s) {
    SampleArgs a;
    a.x = logits;
    a.u = u;
    a.temperature = temperature;
    a.top_p = top_p;
    a.min_p = min_p;
    a.top_k = top_k;
    a.ids = ids;
    a.logp = logp;
    a.stride = stride;
    a.vocab = vocab;
    sample_kernel<<<(unsigned)rows, kThreads, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? SPECTRA_OK : SPECTRA_ERR_CUDA;
}

spectra_status sample_device_error(unsigned int *bits, cudaStream_t s) {
    unsigned int v = 0;
    if (cudaMemcpyFromSymbolAsync(&v, g_sample_error, sizeof v, 0, cudaMemcpyDeviceToHost, s) != cudaSuccess)
        return SPECTRA_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return SPECTRA_ERR_CUDA;
    *bits = v;
    if (v != 0) {
        const unsigned int zero = 0;
        if (cudaMemcpyToSymbolAsync(g_sample_error, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, s) != cudaSuccess ||
            cudaStreamSynchronize(s) != cudaSuccess)
            return SPECTRA_ERR_CUDA;
    }
    return SPECTRA_OK;
}

}  // namespace spectra
