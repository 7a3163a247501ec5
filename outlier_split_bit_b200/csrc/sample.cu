// sample.cu -- token choice from the LM head's logits (sm_100a).
//
// Per row: w_i = exp((x_i - max) / T); the tokens left after top-k (largest
// value first, ties to the lower index), top-p (a token stays while the
// weight before it, in that order, is under p of the whole) and min-p
// (w_i >= min_p) share the whole again; the choice is the first token, in
// index order, whose running sum passes u of it.
//
// No sort of the row: top-k and top-p keep the values above a threshold and
// the first few ties of it, and the threshold is found by counting.  A
// histogram over 2048 equal steps of the distance to the maximum (31.5 T in
// all: what lies further has weight 0), by counts for top-k and by weight for
// top-p, finds the threshold's step; the few tokens in it are gathered and
// ranked against one another.  A step that holds too many of them (equal
// logits, say) is divided by the digits of the order-preserving key instead.
// Where what a row keeps fits a list of 512 (a small top-k, a min-p that leaves few)
// it is gathered whole and the row ends in one CTA of the cluster.
//
// Weights are 64-bit fixed point, w * 2^44 rounded from a double: integer sums
// do not depend on their order, so the histograms use atomics and the row
// repeats bit for bit; a row of up to 2^19 tokens cannot overflow, and a token
// lighter than 2^-45 of the heaviest has weight 0.
//
// A row is a cluster of 1 to 8 CTAs, as many as keep the rows' clusters in one
// wave; a CTA takes a contiguous part of the row, reads it from memory once
// (the maximum) and from L2 after that, and exchanges maxima, histograms and
// sums with its cluster through distributed shared memory.
//
// Measured (B200): 1 row of 131072 logits, top-k 50 then top-p: 16 us, a chain of
// passes, cluster barriers and remote reads (histogram and its search 6, the list's
// end 3), where the row's bytes would take 0.1.  64 rows of 131071, top-p and
// min-p: 57 us against 5 for the bytes: every weight in reach is an exponential in
// FP64 (some 12 FP64 instructions) and two shared atomics, of which the one and
// the other take about half.  By counts alone (top-k 50): 25 us.  Without filters 37 us
// (1 row 16), greedy 10 (1 row 5.5).
#include <cooperative_groups.h>

#include <utility>

#include "internal.cuh"
#include "select.cuh"

namespace spectra {
namespace {

namespace cg = cooperative_groups;

// bit 0: a NaN logit; bit 1: a row with nothing to choose from.
__device__ unsigned int g_sample_error;

typedef unsigned long long u64;
constexpr int kThreads = 1024;
constexpr int kFix = 44;
constexpr int kMaxVocab = 1 << 19;
constexpr int kSegment = 512;                     // tokens of a warp's running sum
constexpr int kMaxSegments = kMaxVocab / kSegment;
constexpr int kList = 512;                        // tokens that are ranked against one another, all pairs
constexpr float kReach = 31.5f;                   // exp(-31.5) < 2^-45
constexpr int kTable = 32;
constexpr int kMaxRanks = 8;

// Constants of the exponential, in the kernel's parameters (as operands they
// cost no instruction there).
struct Exp {
    double to_steps = 46.166241308446828384;      // 32 / ln 2
    double step = -0.021660849392498290195;       // -ln(2) / 32
    double round = 6755399441055744.0;            // 1.5 * 2^52
    double two52 = 4503599627370496.0;
    double taylor[6] = {1.0, 1.0, 1.0 / 2, 1.0 / 6, 1.0 / 24, 1.0 / 120};
};

struct SampleArgs {
    Exp exp;
    const float *x;
    const float *u, *temperature, *top_p, *min_p;
    const int32_t *top_k;
    int32_t *ids;
    float *logp;
    int64_t stride;
    int vocab, per_cta;  // per_cta: tokens of a CTA, a multiple of kSegment
};

struct Smem {
    uint32_t lo[kBins + 32], hi[kBins + 32];  // this CTA's histogram, low and high words (behind it: what does not count)
    u64 merged[kBins];               // this CTA's share of the bins, over the cluster
    u64 comp[kList], q[kList];       // gathered tokens: (key, ~index), weight
    u64 seg[kMaxSegments];
    int seg_ties[kMaxSegments];
    double table[kTable];            // 2^(i / 32)
    float queue[kThreads / 32][64];
    u64 part[33];
    u64 found_above, total, cta_mass;
    int found_bin, n_list[2], cta_ties, pick;  // n_list: of this gathering and the next, in turn
    float cta_max;
    uint32_t thr;
    int ties;
};

// floor(f * n) for 0 <= f < 1 (f in steps of 2^-64, which holds every f from
// 2^-40 up exactly); *rest: whether anything was cut off.
__device__ __forceinline__ u64 fraction_of(float f, u64 n, bool *rest) {
    const u64 fx = (u64)((double)f * 18446744073709551616.0);
    *rest = fx * n != 0;
    return __umul64hi(fx, n);
}

// A row's weights.  exp(z) = 2^(n/32) * exp(t), n the nearest whole number to
// 32 z / ln 2, |t| <= ln(2) / 64: the Taylor polynomial of degree 5 is within
// t^6 / 720 < 2^-48 of it; the powers of two come from a table of 32 and the
// exponent field.
struct Weights {
    float mx;
    double m64, inv_t;
    const double *table;
    const Exp *c;
    __device__ __forceinline__ double exponent(float v) const { return v == mx ? 0.0 : ((double)v - m64) * inv_t; }
    // w * 2^shift for -40 <= z <= 0
    __device__ __forceinline__ double scaled(double z, int shift) const {
        const double nr = fma(z, c->to_steps, c->round);  // the round constant makes the sum a whole number
        const int n = __double2loint(nr);
        const double t = fma(nr - c->round, c->step, z);
        double p = fma(t, c->taylor[5], c->taylor[4]);
        p = fma(p, t, c->taylor[3]);
        p = fma(p, t, c->taylor[2]);
        p = fma(p, t, 1.0);
        p = fma(p, t, 1.0);
        return table[n & (kTable - 1)] * p * __hiloint2double((1023 + shift + (n >> 5)) << 20, 0);
    }
    __device__ __forceinline__ u64 rounded(double x) const {
        return (u64)__double_as_longlong(x + c->two52) & 0xFFFFFFFFFFFFFull;
    }
    // The weight in fixed point: of a value within the reach,
    __device__ __forceinline__ u64 fixed_near(float v) const { return rounded(scaled(exponent(v), kFix)); }
    // of any value (0 beyond the reach), and 0 for a weight under `least`.
    __device__ __forceinline__ u64 fixed(float v, double least) const {
        const double x = scaled(fmax(exponent(v), -32.0), kFix);  // 0.2 at -32 (and for a NaN): rounds to 0
        return x >= least * (double)(1ll << kFix) ? rounded(x) : 0;
    }
    __device__ __forceinline__ double weight(float v) const {
        const double z = exponent(v);
        return z >= -40.0 ? scaled(z, 0) : 0.0;
    }
};

__device__ __forceinline__ void add_to(Smem &s, int bin, u64 q) {
    const uint32_t l = (uint32_t)q;
    const uint32_t old = atomicAdd(&s.lo[bin], l);
    atomicAdd(&s.hi[bin], (uint32_t)(q >> 32) + (old + l < old));
}

// Over the cluster's histograms (filled, not yet synchronised), from bin 0 up:
// the bin in which the running sum reaches need (1 <= need), and the sum before
// it; *total: of all bins.  Returns false where the total is under need.
__device__ bool cluster_find(cg::cluster_group &cl, Smem &s, u64 need, bool ceil_of_p, float p, int *bin, u64 *above,
                             u64 *total, u64 *need_out) {
    const int tid = threadIdx.x, ranks = (int)cl.num_blocks(), rank = (int)cl.block_rank(), n = kBins / ranks;
    cl.sync();
    u64 own = 0;
    for (int i = tid; i < n; i += kThreads) {
        uint32_t lo[kMaxRanks], hi[kMaxRanks];  // all loads in flight at once
#pragma unroll
        for (int r = 0; r < kMaxRanks; ++r) {
            lo[r] = hi[r] = 0;
            if (r < ranks) {
                const Smem *o = cl.map_shared_rank(&s, r);
                lo[r] = o->lo[rank * n + i];
                hi[r] = o->hi[rank * n + i];
            }
        }
        u64 v = 0;
#pragma unroll
        for (int r = 0; r < kMaxRanks; ++r) v += (u64)lo[r] + ((u64)hi[r] << 32);
        s.merged[i] = v;
        own += v;
    }
    u64 sum;
    block_exclusive(own, s.part, &sum);
    if (tid == 0) s.total = sum;
    cl.sync();
    u64 totals[kMaxRanks], all = 0;
#pragma unroll
    for (int r = 0; r < kMaxRanks; ++r) totals[r] = r < ranks ? cl.map_shared_rank(&s, r)->total : 0;
#pragma unroll
    for (int r = 0; r < kMaxRanks; ++r) all += totals[r];
    *total = all;
    if (ceil_of_p) {
        // a token stays while the sum before it is under p of the whole: the
        // last one is where the sum reaches that, rounded up; the first stays
        bool rest = false;
        need = p > 0.f ? fraction_of(p, all, &rest) : 0;
        need += rest;
        if (need == 0) need = 1;
    }
    *need_out = need;
    const bool ok = need <= all;
    if (ok) {
        u64 run = 0;
        int at = 0;
#pragma unroll
        for (int r = 0; r < kMaxRanks - 1; ++r)
            if (at == r && r < ranks - 1 && need > run + totals[r]) {
                run += totals[r];
                ++at;
            }
        const Smem *o = cl.map_shared_rank(&s, at);
        // n <= 2 * kThreads bins of that share, two neighbours per thread
        const u64 v0 = 2 * tid < n ? o->merged[2 * tid] : 0, v1 = 2 * tid + 1 < n ? o->merged[2 * tid + 1] : 0;
        u64 t;
        const u64 before = run + block_exclusive(v0 + v1, s.part, &t);
        if (before < need && need <= before + v0 + v1) {
            const bool second = need > before + v0;
            s.found_bin = at * n + 2 * tid + second;
            s.found_above = before + (second ? v0 : 0);
        }
    }
    __syncthreads();  // (what others still read here is written after the cluster's next barrier)
    *bin = s.found_bin;
    *above = s.found_above;
    __syncthreads();
    return ok;
}

__device__ __forceinline__ void clear_bins(Smem &s) {
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += kThreads) s.lo[i] = s.hi[i] = 0;
    __syncthreads();
}

// The bin of key digit d, largest digit first.
__device__ __forceinline__ int digit_bin(uint32_t key, int d) {
    return kBins - 1 - (int)((key >> digit_shift(d)) & digit_mask(d));
}

// f(logit, index) for the CTA's tokens, eight loads in flight per thread.
constexpr int kBatch = 8;
template <class F>
__device__ __forceinline__ void for_each(const float *x, int i0, int i1, const F &f) {
    int i = i0 + (int)threadIdx.x;
    const float *at = x + i;
    for (; i + (kBatch - 1) * kThreads < i1; i += kBatch * kThreads, at += kBatch * kThreads) {
        float v[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) v[j] = __ldg(at + j * kThreads);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) f(v[j], i + j * kThreads);
    }
#pragma unroll 1
    for (; i < i1; i += kThreads, at += kThreads) f(__ldg(at), i);
}

__global__ void __launch_bounds__(kThreads, 1) sample_kernel(const __grid_constant__ SampleArgs a) {
    extern __shared__ __align__(16) unsigned char raw[];
    Smem &s = *reinterpret_cast<Smem *>(raw);
    cg::cluster_group cl = cg::this_cluster();
    const int ranks = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const int row = blockIdx.x / ranks, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int i0 = min(a.vocab, rank * a.per_cta), i1 = min(a.vocab, i0 + a.per_cta);
    const float *x = a.x + (int64_t)row * a.stride;
    const float temp = a.temperature ? a.temperature[row] : 1.f;

    // the largest logit, and whether one is NaN
    float mx = -INFINITY;
    bool nan = false;
    for_each(x, i0, i1, [&](float v, int) {
        nan |= !(v == v);
        mx = fmaxf(mx, v);
    });
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (nan) atomicOr(&g_sample_error, 1u);
    if (tid < kTable) s.table[tid] = exp2((double)tid / kTable);
    if (tid == 0) {
        s.pick = a.vocab;
        s.n_list[0] = s.n_list[1] = 0;
    }
    if (lane == 0) s.part[warp] = float_key(mx);
    __syncthreads();
    if (tid == 0) {
        u64 m = 0;
        for (int i = 0; i < kThreads / 32; ++i) m = s.part[i] > m ? s.part[i] : m;
        s.cta_max = key_float((uint32_t)m);
    }
    cl.sync();
    mx = -INFINITY;
#pragma unroll
    for (int r = 0; r < kMaxRanks; ++r)
        if (r < ranks) mx = fmaxf(mx, cl.map_shared_rank(&s, r)->cta_max);
    if (mx == -INFINITY) {
        if (rank == 0 && tid == 0) {
            a.ids[row] = -1;
            if (a.logp) a.logp[row] = -INFINITY;
            atomicOr(&g_sample_error, 2u);
        }
        cl.sync();
        return;
    }
    if (!(temp > 0.f)) {  // greedy: the first of the largest
        for_each(x, i0, i1, [&](float v, int i) {
            if (v == mx) atomicMin(&s.pick, i);
        });
        cl.sync();
        if (rank == 0 && tid == 0) {
            int best = a.vocab;
            for (int r = 0; r < ranks; ++r) best = min(best, cl.map_shared_rank(&s, r)->pick);
            a.ids[row] = best;
            if (a.logp) a.logp[row] = 0.f;
        }
        cl.sync();
        return;
    }
    Weights w;
    w.mx = mx;
    w.m64 = (double)mx;
    w.inv_t = 1.0 / (double)temp;
    w.table = s.table;
    w.c = &a.exp;
    // half the distance to the maximum in steps: of logits of 1e38 and both signs the
    // distance itself may not be finite (at a temperature of that size)
    const float half_mx = 0.5f * mx, inv_step = 2.f * kBins / (kReach * temp);
    // the step of a value below the maximum, kBins or more beyond the reach
    // (subtraction, product and truncation keep the order of the values)
    auto step_of = [&](float v) -> int {
        return v == mx ? 0 : (int)fminf(fmaf(v, -0.5f, half_mx) * inv_step, (float)kBins);  // (fminf drops a NaN)
    };

    uint32_t thr = 0;  // the smallest kept key,
    int ties = a.vocab;  // and how many of its tokens stay (the first ones)
    // Gathers the tokens for which take(v) into rank 0's list, as far as there
    // is room, and returns their number.  (The next gathering's counter is
    // cleared here; a barrier of the cluster lies between the two.)
    int gathering = 0;
    auto gather = [&](auto take) -> int {
        Smem *to = cl.map_shared_rank(&s, 0);
        int *count = &to->n_list[gathering & 1];
        for_each(x, i0, i1, [&](float v, int i) {
            if (take(v)) {
                const int at = atomicAdd(count, 1);
                if (at < kList) to->comp[at] = ((u64)float_key(v) << 32) | (0xFFFFFFFFu - (uint32_t)i);
            }
        });
        cl.sync();
        const int n = *count;
        ++gathering;
        if (rank == 0) {
            if (tid == 0) s.n_list[gathering & 1] = 0;
            if (n <= kList && tid < n) s.q[tid] = w.fixed(key_float((uint32_t)(s.comp[tid] >> 32)), 0.0);
        }
        __syncthreads();
        return n;
    };
    // Finds the threshold within step `bin`: the `need`-th token of it, or the
    // token at which its weight reaches `need`.  tie_w, tie_n: the weight and
    // number of thr's own tokens (top-p after top-k), which lie last.
    auto resolve = [&](int bin, u64 need, bool by_weight, u64 tie_w) {
        const uint32_t from = thr;
        // a look at the value first, with room for roundings
        const float width = kReach * temp / kBins, room = 1e-3f * width + 1e-6f * (fabsf(mx) + kReach * temp);
        const float upper = mx - (float)bin * width + room, lower = mx - (float)(bin + 1) * width - room;
        const bool look = mx < INFINITY && upper < INFINITY && lower > -INFINITY;
        auto member = [&](float v) { return step_of(v) == bin && (from == 0 || float_key(v) > from); };
        const int n = gather([&](float v) { return (!look || (v <= upper && v >= lower)) && member(v); });
        if (n <= kList) {
            if (rank == 0) {
                if (tid == 0) {
                    s.thr = from;  // unless one of the list is it
                    s.ties = -1;
                }
                __syncthreads();
                u64 listed = 0;
                if (tid < n) {
                    const u64 mine = s.comp[tid], own = by_weight ? s.q[tid] : 1;
                    u64 before = 0;
                    int same = 1;
#pragma unroll 8
                    for (int j = 0; j < n; ++j) {
                        const u64 c = s.comp[j], q = by_weight ? s.q[j] : 1;
                        before += c > mine ? q : 0;
                        same += c > mine && (uint32_t)(c >> 32) == (uint32_t)(mine >> 32);
                    }
                    listed = own;
                    if (before < need && need <= before + own) {
                        s.thr = (uint32_t)(mine >> 32);
                        s.ties = same;
                    }
                }
                u64 sum;
                block_exclusive(listed, s.part, &sum);
                if (tid == 0) {
                    if (s.ties < 0) {  // the threshold stays, with fewer ties
                        const u64 m = tie_w ? (need - sum + tie_w - 1) / tie_w : 0;
                        s.ties = (int)min(m, (u64)ties);
                    }
                }
            }
            cl.sync();
            const Smem *o = cl.map_shared_rank(&s, 0);
            thr = o->thr;
            ties = o->ties;  // (written again, if at all, two barriers later)
            return;
        }
        uint32_t prefix = 0;
        for (int d = 0; d < kDigits; ++d) {
            clear_bins(s);
            for_each(x, i0, i1, [&](float v, int) {
                const uint32_t key = float_key(v);
                if (member(v) && digit_in(key, prefix, d)) add_to(s, digit_bin(key, d), by_weight ? w.fixed_near(v) : 1);
            });
            if (rank == 0 && tid == 0 && tie_w && step_of(key_float(from)) == bin && digit_in(from, prefix, d))
                add_to(s, digit_bin(from, d), tie_w * (u64)ties);
            int b;
            u64 above, total, unused;
            cluster_find(cl, s, need, false, 0.f, &b, &above, &total, &unused);
            prefix |= (uint32_t)(kBins - 1 - b) << digit_shift(d);
            need -= above;
        }
        const u64 each = by_weight ? w.fixed(key_float(prefix), 0.0) : 1;
        const u64 m = each ? (need + each - 1) / each : 0;
        ties = prefix == from ? (int)min(m, (u64)ties) : (int)min(m, (u64)a.vocab);
        thr = prefix;
    };

    const int k = a.top_k ? a.top_k[row] : 0;
    const float p = a.top_p ? a.top_p[row] : 1.f;
    const float min_p = a.min_p ? a.min_p[row] : 0.f;
    const double least = min_p > 0.f ? fmin((double)min_p, 1.0) : 0.0;  // (a NaN: off)
    float u = a.u[row];
    u = u == u ? fminf(fmaxf(u, 0.f), 0.99999994f) : 0.f;
    auto choose = [&](int i, u64 total) {
        a.ids[row] = i;
        if (a.logp) a.logp[row] = (float)(w.exponent(x[i]) - log((double)total / (double)(1ll << kFix)));
    };
    // what lies at or under `least_v` has no weight or fails min-p (with room
    // for the rounding of the bound)
    float least_v = -INFINITY;
    if (mx < INFINITY) {
        float reach = kReach + 1.f;
        if (least > 0.0) reach = fminf(reach, (float)(-log(least)) + 1e-3f);
        least_v = mx - reach * temp - 1e-6f * fabsf(mx);
    }
    // The end of a row whose kept tokens are all in rank 0's list of n (and no
    // better ones outside it): rank 0 keeps the `most` best of them, then those
    // before which, in order of value, less than `need` lies (0: top-p of the
    // list's own whole), then min-p's, and chooses.
    auto finish = [&](int n, int most, u64 need) {
        const u64 mine = tid < n ? s.comp[tid] : 0;
        u64 before = 0, own = 0;
        if (tid < n) {
            int place = 0;
#pragma unroll 8
            for (int j = 0; j < n; ++j) {
                const u64 q = s.q[j];
                const bool better = s.comp[j] > mine;
                place += better;
                before += better ? q : 0;
            }
            if (place < most) own = s.q[tid];
        }
        u64 whole;
        block_exclusive(own, s.part, &whole);
        if (need == 0) {
            need = whole;
            if (p < 1.f) {
                bool rest = false;
                need = p > 0.f ? fraction_of(p, whole, &rest) : 0;
                need += rest;
                if (need == 0) need = 1;
            }
        }
        if (own && !(before < need && w.weight(key_float((uint32_t)(mine >> 32))) >= least)) own = 0;
        __syncthreads();
        if (tid < n) s.q[tid] = own;
        u64 left;
        block_exclusive(own, s.part, &left);
        bool rest;
        const u64 target = fraction_of(u, left, &rest);
        if (own) {
            u64 run = 0;
#pragma unroll 8
            for (int j = 0; j < n; ++j) {
                const u64 q = s.q[j];
                run += (uint32_t)s.comp[j] > (uint32_t)mine ? q : 0;  // ~index
            }
            if (run <= target && target < run + own) choose((int)(0xFFFFFFFFu - (uint32_t)mine), left);
        }
    };
    // The row's end in rank 0's list: the other CTAs have read its counter, which
    // lies in rank 0's memory, when they arrive at the barrier, and rank 0 leaves
    // only after that.  It arrives before its own work, so nobody waits for that.
    auto end_row = [&](int n, int most, u64 need) {
        auto read = cl.barrier_arrive();
        if (rank == 0) finish(n, most, need);
        cl.barrier_wait(std::move(read));
    };
    if (k > 0 && k < a.vocab) {
        clear_bins(s);
        for_each(x, i0, i1, [&](float v, int) {
            const int b = step_of(v);
            atomicAdd(&s.lo[b < kBins ? b : kBins + lane], 1u);
        });
        int bin;
        u64 above, total, unused;
        if (cluster_find(cl, s, (u64)k, false, 0.f, &bin, &above, &total, &unused)) {
            // how many tokens the step holds (the bins are cleared after the next barrier)
            u64 members = 0;
#pragma unroll
            for (int r = 0; r < kMaxRanks; ++r)
                if (r < ranks) members += cl.map_shared_rank(&s, r)->lo[bin];
            if (above + members <= kList) {
                const int n = gather([&](float v) { return step_of(v) <= bin; });
                return end_row(n, k, 0);
            }
            resolve(bin, (u64)k - above, false, 0);
        }
    }
    if (p < 1.f) {
        // the whole of the top-k set: keys above thr, and `ties` of thr's
        const u64 tie_w = thr > kKeyNegInf ? w.fixed(key_float(thr), 0.0) : 0;
        clear_bins(s);
        for_each(x, i0, i1, [&](float v, int) {
            const int b = step_of(v);
            add_to(s, b < kBins && (thr == 0 || float_key(v) > thr) ? b : kBins + lane, w.fixed_near(v));
        });
        if (rank == 0 && tid == 0 && tie_w) add_to(s, step_of(key_float(thr)), tie_w * (u64)ties);
        int bin;
        u64 above, total, need;
        cluster_find(cl, s, 0, true, p, &bin, &above, &total, &need);
        if (thr == 0 && (double)total <= 2.0 * kList * (double)(1ll << kFix) * least) {
            // min-p is likely to leave few (total / least at most, and those that
            // pass it weigh more than that): what passes it and lies over the
            // threshold's step or in it holds all that stays, and all that is better
            const int n = gather([&](float v) { return v > least_v && step_of(v) <= bin; });
            if (n <= kList) return end_row(n, kList, need);
            cl.sync();  // (the count was read; the list starts anew)
        }
        resolve(bin, need - above, true, tie_w);
    } else if (least > 0.0 && thr == 0) {
        const int n = gather([&](float v) { return v > least_v; });
        if (n <= kList) return end_row(n, kList, 0);
    }

    // the kept weight of each segment in index order, thr's ties counted apart
    const int segs = (i1 - i0 + kSegment - 1) / kSegment;
    const u64 tie_q = thr > kKeyNegInf ? w.fixed(key_float(thr), least) : 0;
    const float thr_v = thr > kKeyNegInf ? key_float(thr) : -INFINITY;
    const float cut = fmaxf(thr_v, least_v);  // what lies at or under it is not kept, but for thr's ties
    auto over = [&](float v) { return v > cut; };
    if (tid == 0) {
        s.cta_mass = 0;
        s.cta_ties = 0;
    }
    __syncthreads();
    float *queue = s.queue[warp];
    for (int g = warp; g < segs; g += kThreads / 32) {
        u64 m = 0;
        int t = 0, waiting = 0;
        // kept tokens queue up, so that their weights are taken 32 at a time
        for (int j = 0; j < kSegment; j += 32 * kBatch) {
            float v[kBatch];
            const int i = i0 + g * kSegment + j + lane;
#pragma unroll
            for (int c = 0; c < kBatch; ++c) v[c] = i + 32 * c < i1 ? __ldg(x + i + 32 * c) : __int_as_float(0x7FC00000);
#pragma unroll
            for (int c = 0; c < kBatch; ++c) {
                const bool keep = over(v[c]);
                t += v[c] == thr_v;
                const unsigned who = __ballot_sync(0xffffffffu, keep);
                if (who == 0) continue;
                if (keep) queue[waiting + __popc(who & ((1u << lane) - 1))] = v[c];
                waiting += __popc(who);
                __syncwarp();
                if (waiting >= 32) {
                    m += w.fixed(queue[lane], least);
                    waiting -= 32;
                    const float last = queue[32 + lane];
                    __syncwarp();
                    queue[lane] = last;
                    __syncwarp();
                }
            }
        }
        if (lane < waiting) m += w.fixed(queue[lane], least);
        __syncwarp();
        for (int o = 16; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
        t = __reduce_add_sync(0xffffffffu, t);
        if (lane == 0) {
            s.seg[g] = m;
            s.seg_ties[g] = t;
            atomicAdd(&s.cta_mass, m);
            atomicAdd(&s.cta_ties, t);
        }
    }
    cl.sync();
    u64 total = 0, run = 0, mine = 0;
    int ties_run = 0, ties_all = 0;
    for (int r = 0; r < ranks; ++r) {
        const Smem *o = cl.map_shared_rank(&s, r);
        const u64 m = o->cta_mass + tie_q * (u64)max(0, min(ties - ties_all, o->cta_ties));
        if (r == rank) {
            run = total;
            ties_run = ties_all;
            mine = m;
        }
        total += m;
        ties_all += o->cta_ties;
    }
    cl.sync();  // nobody reads another CTA's memory from here on
    bool rest;
    const u64 target = fraction_of(u, total, &rest);  // the first running sum over it
    if (!(run <= target && target < run + mine)) return;
    // this CTA holds it: its segment, then its token
    int all;
    const int st = tid < segs ? s.seg_ties[tid] : 0;
    const int tie_before = ties_run + block_exclusive(st, reinterpret_cast<int *>(s.part), &all);
    __syncthreads();
    const u64 sm = tid < segs ? s.seg[tid] + tie_q * (u64)max(0, min(ties - tie_before, st)) : 0;
    u64 sum;
    const u64 before = run + block_exclusive(sm, s.part, &sum);
    if (before <= target && target < before + sm) {
        s.found_bin = tid;
        s.found_above = before;
        s.cta_ties = tie_before;
    }
    __syncthreads();
    const int i = i0 + s.found_bin * kSegment + tid;
    const bool in = tid < kSegment && i < i1;
    const float v = in ? x[i] : -INFINITY;
    const bool tie = in && v == thr_v;
    const int tie_rank = s.cta_ties + block_exclusive((int)tie, reinterpret_cast<int *>(s.part), &all);
    __syncthreads();
    u64 q = 0;
    if (in) q = tie ? (tie_rank < ties ? tie_q : 0) : (over(v) ? w.fixed(v, least) : 0);
    const u64 at = s.found_above + block_exclusive(q, s.part, &sum);
    if (q && at <= target && target < at + q) choose(i, total);
}

}  // namespace

int sample_max_vocab() { return kMaxVocab; }

spectra_status launch_sample(const float *logits, int rows, int vocab, int64_t stride, const float *u,
                             const float *temperature, const int32_t *top_k, const float *top_p,
                             const float *min_p, int32_t *ids, float *logp, cudaStream_t s,
                             const DeviceInfo &dev) {
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
    // as many CTAs a row as keep one wave, each with 4096 tokens or more
    int ranks = 1;
    while (ranks < kMaxRanks && (int64_t)rows * ranks * 2 <= dev.sm_count && vocab >= 2 * ranks * 4096) ranks *= 2;
    a.per_cta = (int)(cdiv(vocab, (int64_t)ranks * kSegment) * kSegment);
    static std::atomic<uint64_t> ready{0};
    cudaError_t e = allow_smem((const void *)sample_kernel, (int)sizeof(Smem), dev, &ready);
    if (e != cudaSuccess) return SPECTRA_ERR_CUDA;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)ranks;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)rows * ranks, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = sizeof(Smem);
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, sample_kernel, a);
    return e == cudaSuccess ? SPECTRA_OK : SPECTRA_ERR_CUDA;
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
