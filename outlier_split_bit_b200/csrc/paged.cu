// paged.cu -- attention of a batch of sequences over the paged 4-bit KV pool
// (sm_100a).
//
// Method: "SPECTRA: Sparse-Precision Exact Channel Tensor Reconstruction
// Architecture" (Dev.to abstract), abstract paragraph: microscaled Group-32
// 4-bit key-value caching keeps long contexts resident.
//
// For query j of a sequence of length n with m new tokens, at position
// pos = n - m + j, and query head i over KV head h = i / grp:
//   s_t = f(scale * q . k_t) - slope_i * (pos - t),  f(x) = cap * tanh(x / cap),
//   over the t with 0 <= pos - t (and pos - t < window, with a window),
//   out = sum_t softmax(s)_t v_t,  lse = log sum_t exp(s_t),
//   mass[h][t] += sum over the group's heads and the tokens of softmax(s)_t.
#include "internal.cuh"
#include "pool.cuh"

namespace spectra {
namespace {

// bit 2: a page outside the pool, a length or a row range out of bounds.
__device__ unsigned int g_paged_error;

struct PagedArgs {
    PoolView p;
    const int32_t *pages;
    const int32_t *lengths;
    const int32_t *q_start;
    const uint16_t *q;
    const float *slopes;
    void *out;
    float *lse;
    int max_pages, n_seq, n_rows, max_q, Hq, grp, window;
    float scale, cap;
    bool bf16;
};

// A sequence's length and rows; nothing for values out of bounds.
struct Sequence {
    int n, row0, m;
};
__device__ __forceinline__ Sequence sequence_of(const PagedArgs &a, int b) {
    Sequence s;
    s.n = a.lengths[b];
    s.row0 = a.q_start ? a.q_start[b] : b;
    const int row1 = a.q_start ? a.q_start[b + 1] : b + 1;
    s.m = row1 - s.row0;
    bool bad = false;
    if (s.n < 0 || (int64_t)s.n > ((int64_t)a.max_pages << a.p.lp)) {
        s.n = 0;
        bad = true;
    }
    if (s.row0 < 0 || row1 > a.n_rows || s.m < 0 || s.m > a.max_q) {
        s.m = 0;
        bad = true;
    }
    if (bad && threadIdx.x == 0) atomicOr(&g_paged_error, 4u);
    return s;
}

constexpr int kThreads = 128;

__device__ __forceinline__ float score(const PagedArgs &a, float dot, float slope, int gap) {
    float s = dot * a.scale;
    if (a.cap > 0.f) s = a.cap * tanhf(s / a.cap);
    return s - slope * (float)gap;
}

__device__ __forceinline__ float k_dot(const PagedArgs &a, int64_t slot, const uint16_t *q) {
    const int G = a.p.G;
    float dot = 0.f;
    const uint32_t zw = a.p.kz[slot];
    for (int g = 0; g < G; ++g) {
        float part = 0.f;
        const int z = (int)((zw >> (4 * g)) & 15u);
        for (int w = 0; w < 4; ++w) {
            const uint32_t word = a.p.kc[slot * 4 * G + w * G + g];
            for (int i = 0; i < 8; ++i)
                part = fmaf((float)((int)((word >> (4 * i)) & 15u) - z),
                            __uint_as_float((uint32_t)q[32 * g + 8 * w + i] << 16), part);
        }
        dot = fmaf(__half2float(__ushort_as_half(a.p.ks[slot * G + g])), part, dot);
    }
    return dot;
}

// One CTA per sequence, query row and query head; a thread per position for
// the scores, a thread per channel for the weighted sum.
__global__ void __launch_bounds__(kThreads) paged_attention_kernel(PagedArgs a) {
    __shared__ float w[kThreads];
    __shared__ int64_t at[kThreads];
    __shared__ float red[kThreads / 32];
    const int i = blockIdx.x, j = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, D = 32 * a.p.G;
    const Sequence s = sequence_of(a, b);
    if (j >= s.m) return;
    const int h = i / a.grp, pos = s.n - s.m + j;
    const int first = a.window > 0 ? max(0, pos - a.window + 1) : 0;
    const int64_t row = (int64_t)(s.row0 + j) * a.Hq + i;
    const uint16_t *q = a.q + row * D;
    const float slope = a.slopes ? a.slopes[i] : 0.f;
    const int32_t *pages = a.pages + (int64_t)b * a.max_pages;
    float m = -INFINITY, l = 0.f, acc[2] = {0.f, 0.f};
    for (int t0 = first; t0 <= pos; t0 += kThreads) {
        const int t = t0 + tid;
        float x = -INFINITY;
        int64_t slot = -1;
        if (t <= pos) {
            const int32_t ts = a.p.token_slot(pages, t);
            if (ts < 0) {
                atomicOr(&g_paged_error, 4u);
            } else {
                slot = a.p.slot(ts, h);
                x = score(a, k_dot(a, slot, q), slope, pos - t);
            }
        }
        float mx = x;
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        __syncthreads();
        if ((tid & 31) == 0) red[tid >> 5] = mx;
        __syncthreads();
        mx = m;
        for (int k = 0; k < kThreads / 32; ++k) mx = fmaxf(mx, red[k]);
        const float old = mx == -INFINITY ? 1.f : expf(m - mx);
        m = mx;
        w[tid] = x == -INFINITY ? 0.f : expf(x - m);
        at[tid] = slot;
        __syncthreads();
        l *= old;
        for (int k = 0; k < kThreads; ++k) l += w[k];
        for (int e = 0; e < 2; ++e) {
            const int d = tid + e * kThreads;
            acc[e] *= old;
            if (d >= D) continue;
            const int g = d >> 5, hw = (d & 31) >> 2, sh = 4 * (d & 3);
            for (int k = 0; k < kThreads; ++k) {
                if (at[k] < 0) continue;
                const uint32_t word = a.p.vc[at[k] * 8 * a.p.G + hw * a.p.G + g];
                const int z = (int)((a.p.vz[at[k]] >> (4 * g)) & 15u);
                const float v = (float)((int)((word >> sh) & 15u) - z) *
                                __half2float(__ushort_as_half(a.p.vs[at[k] * a.p.G + g]));
                acc[e] = fmaf(w[k], v, acc[e]);
            }
        }
    }
    for (int e = 0; e < 2; ++e) {
        const int d = tid + e * kThreads;
        if (d >= D) continue;
        const float v = l > 0.f ? acc[e] / l : 0.f;
        if (a.bf16) reinterpret_cast<__nv_bfloat16 *>(a.out)[row * D + d] = __float2bfloat16_rn(v);
        else reinterpret_cast<float *>(a.out)[row * D + d] = v;
    }
    if (tid == 0 && a.lse) a.lse[row] = l > 0.f ? m + logf(l) : -INFINITY;
}

// The accumulated weights: a thread per position of one head.
__global__ void __launch_bounds__(kThreads) paged_mass_kernel(PagedArgs a) {
    const int h = blockIdx.y, b = blockIdx.z;
    const Sequence s = sequence_of(a, b);
    const int t = blockIdx.x * kThreads + threadIdx.x;
    if (t >= s.n || s.m == 0) return;
    const int D = 32 * a.p.G;
    const int32_t ts = a.p.token_slot(a.pages + (int64_t)b * a.max_pages, t);
    if (ts < 0) return;
    const int64_t slot = a.p.slot(ts, h);
    float sum = 0.f;
    for (int j = 0; j < s.m; ++j) {
        const int gap = s.n - s.m + j - t;
        if (gap < 0 || (a.window > 0 && gap >= a.window)) continue;
        for (int i = h * a.grp; i < (h + 1) * a.grp; ++i) {
            const int64_t row = (int64_t)(s.row0 + j) * a.Hq + i;
            const float x = score(a, k_dot(a, slot, a.q + row * D), a.slopes ? a.slopes[i] : 0.f, gap);
            sum += expf(x - a.lse[row]);
        }
    }
    a.p.mass[slot] += sum;
}

}  // namespace

size_t paged_workspace_bytes(int n_rows, int n_q_heads, int head_dim) {
    (void)head_dim;
    return ((size_t)n_rows * n_q_heads * 4 + 15) / 16 * 16;
}

spectra_status launch_paged_attention(const spectra_kv_pool &pool, const spectra_paged_query &x, void *ws,
                                      cudaStream_t s, const DeviceInfo &) {
    PagedArgs a;
    a.p = PoolView::of(pool);
    a.pages = x.pages;
    a.lengths = x.lengths;
    a.q_start = x.q_start;
    a.q = x.q;
    a.slopes = x.slopes;
    a.out = x.out;
    a.lse = x.lse ? x.lse : (x.update_mass ? static_cast<float *>(ws) : nullptr);
    a.max_pages = x.max_pages;
    a.n_seq = x.n_seq;
    a.n_rows = x.n_rows;
    a.max_q = x.max_q;
    a.Hq = x.n_q_heads;
    a.grp = x.n_q_heads / pool.n_heads;
    a.window = x.window;
    a.scale = x.scale;
    a.cap = x.softcap;
    a.bf16 = x.out_dtype == SPECTRA_BF16;
    paged_attention_kernel<<<dim3((unsigned)a.Hq, (unsigned)a.max_q, (unsigned)a.n_seq), kThreads, 0, s>>>(a);
    if (cudaGetLastError() != cudaSuccess) return SPECTRA_ERR_CUDA;
    if (x.update_mass) {
        const int64_t positions = (int64_t)x.max_pages << a.p.lp;
        paged_mass_kernel<<<dim3((unsigned)cdiv(positions, kThreads), (unsigned)a.p.H, (unsigned)a.n_seq), kThreads,
                            0, s>>>(a);
        if (cudaGetLastError() != cudaSuccess) return SPECTRA_ERR_CUDA;
    }
    return SPECTRA_OK;
}

spectra_status paged_device_error(unsigned int *bits, cudaStream_t s) {
    unsigned int v = 0;
    if (cudaMemcpyFromSymbolAsync(&v, g_paged_error, sizeof v, 0, cudaMemcpyDeviceToHost, s) != cudaSuccess)
        return SPECTRA_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return SPECTRA_ERR_CUDA;
    *bits = v;
    if (v != 0) {
        const unsigned int zero = 0;
        if (cudaMemcpyToSymbolAsync(g_paged_error, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, s) != cudaSuccess ||
            cudaStreamSynchronize(s) != cudaSuccess)
            return SPECTRA_ERR_CUDA;
    }
    return SPECTRA_OK;
}

}  // namespace spectra
