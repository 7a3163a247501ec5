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
//
// One pass over K and V.  A KV head's queries (tokens x group heads) are the
// columns of a tile of 8 * NT; a warp takes 16 positions (a unit) at a time, one
// or two units a step, and multiplies them on the tensor cores, m16n8k16 with
// FP32 accumulation:
//   scores: A = 16 positions x 16 channels of K, B = q, as FP16 after a power of
//     two that brings its row's largest value to 2^14 (BF16 has fewer bits, so
//     only values under 2^-28 of the largest lose any).  The product sums are
//     exact up to FP32 accumulation, and each group's is multiplied by its scale
//     in FP32;
//   weighted sum: A = 16 channels x 16 positions of V, B = the weights in FP16,
//     scaled so that they lie under 2^15.
// The codes enter in one of two forms:
//   as they stand (8 columns: decode): a nibble masked in place is an FP16
//     subnormal, one instruction for two codes.  K's zero points take one FP32
//     multiply-add per group, z times the query's own sum over the group; V's a
//     product of their own, and V's scale goes into the weight: w * s rounded to
//     FP16.  For that the scales are multiplied with a power of two that brings the
//     largest of the warp's first step to 2^-3 .. 2 (none where it lies there), and
//     the sums with its inverse: a product under FP16's normal range is then off by
//     2^-25 where the largest weight times the largest scale is 2^4 or more, 2^-29 of
//     it.  (Without the power, values of 1e-5 lost 0.2 % of the largest output, and
//     many light weights beside a heavy one far more.)  Where scales grow so far
//     that a product passes FP16's range, which is seen in the sums, the item is
//     run again with the power that the largest of all its scales wants.
//     The tensor core lines an instruction's products up at their exponents, of which
//     a subnormal's counts as 2^-14 (by its results), and cuts off 24 bits under the
//     largest: 2^-14 of a code's step times the largest query value (K), or times the
//     unit's largest weight (V).  For K that shows where a query value is a thousand times the
//     others (one of 3000 beside ones of 1: outputs off by 4.6e-5, in FP32
//     arithmetic 1.5e-5; of 300 both 1e-6), for V it is under a BF16 output's step;
//   less the zero point (16 columns and more, and V for an FP32 output): a nibble
//     or-ed under 0x6400 is 1024 + c, or 1024 + 16c where it stands, and one
//     half-precision instruction takes it to c - z, exactly.  V is dequantised to
//     (c - z) * s with one rounding; dearer per code, but done once for all
//     columns, where the other form's work on weights and zero points is per
//     column.  A V beyond FP16's range turns the output non-finite, which is
//     reported.
// For a BF16 output the FP16 roundings are enough: 2^-11 each, an eighth of the
// output's own, and for a weight under FP16's normal range 2^-25, which is 2^-32
// of the largest.  For an FP32 output what the two roundings left goes in as
// well, as two more products (V's remainder is exact; of the weights 2^-22 is
// lost, or 2^-32 of the largest; of values under 2^-14 2^-38, as above), and each unit's sum is added to the accumulator
// in FP32: the tensor core cuts its sums off (error at 8192 positions 1.4e-6 of
// the largest output, with the separate addition 2.4e-7).
//
// The scores' accumulator layout (positions in rows) is transposed into the
// weights' operand layout inside the warp (movmatrix on FP16 pairs).  Which lane
// holds which channel or position is free as long as both operands agree, so the
// pool's words are laid out to be read with one load per position: lane (g, t) =
// (lane / 4, lane % 4) reads K's word t of every group of positions g', g' + 8
// and V's halfword g of every group of positions t, t + 4, t + 8, t + 12.
//
// The running maximum is only a reference: it moves when a weight would pass
// 2^15 (2^14 where V's scale is multiplied in), and then to 2^7 for the largest, so most units need no reduction over
// the lanes and no rescaling.
//
// Each warp copies its own units into a ring of three steps in shared memory,
// asynchronously and without the block's barriers, which only an item's end has.
//
// Work split: the tiles (64 positions, or 128 where a step takes two units) of
// every (sequence, head, column tile) make one list, cut into equal runs, one per
// CTA, from the lengths on the device; so ragged batches balance and the host
// need not know the lengths.  A run's first and last piece may be part of a longer
// item; such pieces go to the workspace (at most two per CTA) and a second
// kernel, launched as a programmatic dependent, joins them in order.  Every order
// is fixed, so results repeat bit for bit.
//
// Measured (B200, in a graph; positions of a batch, Hq / H heads, D channels):
//   16 sequences of 20000 to 65536 positions, 32 / 8, 128, one new token: 862 MB in
//     191 us, 4.5 TB/s, against 134 us at the rate of a copy (over a second and
//     more of such calls 195 to 205 us: the clock falls to the power limit).  The ring
//     alone, without the arithmetic, runs at 6.05 TB/s.  No pipe is full (189 MB of
//     such sequences: integer 48 %, matrix 27 %, half of the issue slots): a warp waits
//     on its own chain from code to operand, product and weight, at 1.8 GHz; how
//     the time over the copy divides between the chain and the clock is open;
//   1 sequence of 8192, 12 / 2, 128: 10.4 us; of 300: 9.2 us, which is the two
//     launches, the run search, the ring's first fill and the join.
// Tried and no faster: 4 to 6 CTAs an SM with one unit a step, 4 ring steps, the
// queries' operands in shared memory for 8 columns, 16 columns a tile where 32 fit.
// The power of V's scales: found at each step 217 us instead of 202 in a loop of the
// first case, multiplied in always (also by 1) 184 instead of 178 on a like pool; so
// it is found once per item and the loop exists twice, with it and without.
#include <type_traits>

#include "internal.cuh"
#include "pool.cuh"
#include "select.cuh"

namespace spectra {
namespace {

// bit 1: a non-finite output; bit 2: a page outside the pool, a length or a row range out of bounds.
__device__ unsigned int g_paged_error;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kUnit = 16;                // positions of a warp's step
// Positions of a CTA's step (a tile of the list), U units per warp.
template <int U>
constexpr int kTile = kUnit * kWarps * U;
constexpr int kMaxCtas = 148 * 4;        // runs, at most: a wave
constexpr int kMinPositions = 128;       // of a run, at least (fewer pieces to join)
// The reference lies kRefBelow under the maximum (base 2) when it is set, and
// moves when a score is kRefRoom over it (kRefRoomRaw for weights that are
// multiplied with V's scales, brought under 2).
constexpr float kRefBelow = 7.f, kRefRoom = 15.f, kRefRoomRaw = 14.f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct PagedArgs {
    PoolView p;
    const int32_t *pages;
    const int32_t *lengths;
    const int32_t *q_start;
    const uint16_t *q;
    const float *slopes;
    void *out;
    float *lse;
    float2 *ws_row;  // [rows][query heads]: store_lse's, for the accumulated weights (null without them)
    float *ws_acc;   // [2 * runs][columns][D]
    float2 *ws_ml;   // [2 * runs][columns]: reference, sum
    int4 *ws_item;   // [runs]: an item cut at the run's end: (last run, first row, columns, head); last run -1: none
    int max_pages, n_seq, n_rows, max_q, Hq, grp, window;
    float scale, cap;
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
    if (s.row0 < 0 || row1 > a.n_rows || row1 < s.row0 || s.m > a.max_q) {
        s.m = 0;
        bad = true;
    }
    if (bad) atomicOr(&g_paged_error, 4u);
    return s;
}

// Tiles of one item of a sequence in the list: from the one with the first
// visible position, and before them as many as make 256 positions, which stand
// for the time an item takes whatever its length.  (Without them the runs of
// short items came last: 48 sequences of 1 to 6000 positions took 68 us; with
// 128, 256, 384 and 768 positions 60, 51, 51 and 55 us.)  Every column tile lists the
// whole sequence's tiles, those after its own last row's position too, which cost
// nothing when their run comes to them: of a whole prompt half the list is empty,
// and the runs over the last column tiles set the time.
template <int U>
constexpr int kItemCost = 256 / kTile<U>;
struct Tiles {
    int first, count;
};
template <int U>
__device__ __forceinline__ Tiles tiles_of(const PagedArgs &a, const Sequence &s) {
    const int64_t lo = a.window > 0 ? (int64_t)s.n - s.m - a.window + 1 : 0;
    Tiles t;
    t.first = lo > 0 ? (int)(lo / kTile<U>) : 0;
    t.count = max(0, (s.n + kTile<U> - 1) / kTile<U> - t.first) + kItemCost<U>;
    return t;
}

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same from zero.
__device__ __forceinline__ void mma_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// (hi, lo) rounded to BF16, lo in the lower half.
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    uint32_t y;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
    return y;
}
__device__ __forceinline__ uint32_t f16_pair(float lo, float hi) {
    uint32_t y;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
    return y;
}
__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<const __half2 *>(&x); }
__device__ __forceinline__ uint32_t as_bits(__half2 x) { return *reinterpret_cast<const uint32_t *>(&x); }

// (w & MASK) | magic in one instruction, the magic number in a register.
template <uint32_t MASK>
__device__ __forceinline__ uint32_t masked_or(uint32_t w, uint32_t magic) {
    uint32_t y;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(y) : "r"(w), "n"(MASK), "r"(magic));
    return y;
}

// The codes of word w as they stand: nibble j of both halfwords is the FP16
// subnormal c * 2^-24 (j = 0, 2) or 16 c * 2^-24 (j = 1, 3).  Products and sums
// with them are as exact as with any other number; what is multiplied with the
// odd ones is divided by 16, and 2^24 and the zero point are seen to later.
__device__ __forceinline__ void raw_codes(uint32_t w, uint32_t (&x)[4]) {
    const uint32_t w8 = w >> 8;
    x[0] = w & 0x000F000Fu;
    x[1] = w & 0x00F000F0u;
    x[2] = w8 & 0x000F000Fu;
    x[3] = w8 & 0x00F000F0u;
}
constexpr float kRaw = 16777216.f;  // 2^24

// The bits of 2^p in FP16, -24 <= p <= 15 (16: infinity), and its exponent of x > 0.
__device__ __forceinline__ uint32_t half_pow2(int p) { return p >= -14 ? (uint32_t)(p + 15) << 10 : 1u << (24 + p); }
__device__ __forceinline__ int half_exponent(uint32_t x) { return x >= 0x400u ? (int)(x >> 10) - 15 : 7 - __clz(x); }
// 2^p in FP32, -126 <= p <= 127.
__device__ __forceinline__ float pow2(int p) { return __uint_as_float((uint32_t)(p + 127) << 23); }

// A group's zero points of two rows (or one, twice), as the FP16 pairs that
// take 1024 + c and (1024 + 16c) / 16 to c - z.  zp: the rows' zero halfwords
// side by side, four groups each, shifted down by 8 for groups 2 and 3; odd:
// the group's lowest bit.
struct ZeroPair {
    __half2 a, b;  // -(1024 + z), -(64 + z)
    __device__ __forceinline__ ZeroPair(uint32_t zp, bool odd) {
        if (!odd) {
            a = as_half2(masked_or<0x000F000Fu>(zp, 0xE400E400u));
            b = __hadd2(a, __float2half2_rn(960.f));
        } else {
            const __half2 y = as_half2(masked_or<0x00F000F0u>(zp, 0xE400E400u));  // -(1024 + 16z)
            b = __hmul2(y, __float2half2_rn(0.0625f));
            a = __hfma2(y, __float2half2_rn(0.0625f), __float2half2_rn(-960.f));
        }
    }
    // Nibble j of both halfwords of w, less the zero points, j = 0 .. 3.
    __device__ __forceinline__ void codes(uint32_t w, __half2 (&x)[4]) const {
        const uint32_t w8 = w >> 8;
        const __half2 sixteenth = __float2half2_rn(0.0625f);
        x[0] = __hadd2(as_half2(masked_or<0x000F000Fu>(w, 0x64006400u)), a);
        x[1] = __hfma2(as_half2(masked_or<0x00F000F0u>(w, 0x64006400u)), sixteenth, b);
        x[2] = __hadd2(as_half2(masked_or<0x000F000Fu>(w8, 0x64006400u)), a);
        x[3] = __hfma2(as_half2(masked_or<0x00F000F0u>(w8, 0x64006400u)), sixteenth, b);
    }
};

// Row r of a unit's 16 (as the tensor core counts them) is its position
// unit_position(r): rows 2t, 2t+1, 2t+8, 2t+9 are t, t+4, t+8, t+12.
__device__ __forceinline__ int unit_position(int r) { return (r & 8) | ((r & 1) << 2) | ((r & 7) >> 1); }

// A place in shared memory, read once: left to itself the compiler reads some
// of a stage's data again.
struct Shared {
    uint32_t at;
    __device__ __forceinline__ Shared operator+(uint32_t bytes) const { return {at + bytes}; }
    __device__ __forceinline__ uint4 get16() const {
        uint4 v;
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
        return v;
    }
    __device__ __forceinline__ uint2 get8() const {
        uint2 v;
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
        return v;
    }
    __device__ __forceinline__ uint32_t get4() const {
        uint32_t v;
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at));
        return v;
    }
    __device__ __forceinline__ uint32_t get2() const {
        uint16_t v;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at));
        return v;
    }
};

// N 32-bit words, or N halfwords in (N + 1) / 2 words, with the widest loads
// that their alignment (the size's own) allows.
template <int N>
__device__ __forceinline__ void load_words(uint32_t (&r)[N], Shared p) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint4 v = (p + 4 * i).get16();
            r[i] = v.x; r[i + 1] = v.y; r[i + 2] = v.z; r[i + 3] = v.w;
        }
    } else if constexpr (N % 2 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const uint2 v = (p + 4 * i).get8();
            r[i] = v.x; r[i + 1] = v.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) r[i] = (p + 4 * i).get4();
    }
}
template <int N>
__device__ __forceinline__ void load_halfwords(uint32_t (&r)[(N + 1) / 2], Shared p) {
    if constexpr (N % 2 == 0) {
        load_words<N / 2>(r, p);
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 2) r[i / 2] = (p + 2 * i).get2() | (i + 1 < N ? (p + 2 * i + 2).get2() << 16 : 0u);
    }
}
__device__ __forceinline__ float half_of(uint32_t w, int which) {
    return which ? __high2float(as_half2(w)) : __low2float(as_half2(w));
}

// A unit's 16 slots lie together in each of the pool's six arrays; a warp
// copies them (or K's three) into its stage in shared memory, 16 bytes a lane
// and copy, asynchronously, at these places.
template <int G, bool V>
struct Stage {
    static constexpr int kCodes = 256 * G, kScales = 32 * G, kZeros = 64;  // bytes per unit
    static constexpr int kc = 0, vc = kc + kCodes, ks = vc + (V ? kCodes : 0), vs = ks + kScales,
                         kz = vs + (V ? kScales : 0), vz = kz + kZeros, kBytes = vz + (V ? kZeros : 0);
    static constexpr int kSmall = (V ? 2 : 1) * (2 * G + 4);  // 16-byte pieces of the scales and zero words
    static constexpr int kPer = (kSmall + 31) / 32;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// What a lane copies of every unit.
template <int G, bool V>
struct Copier {
    using S = Stage<G, V>;
    const char *kc, *vc, *small[S::kPer];
    uint32_t stride[S::kPer], to[S::kPer];
    __device__ __forceinline__ Copier(const PoolView &p, int lane) {
        kc = reinterpret_cast<const char *>(p.kc) + 16 * lane;
        vc = reinterpret_cast<const char *>(p.vc) + 16 * lane;
#pragma unroll
        for (int j = 0; j < S::kPer; ++j) {
            int m = min(lane + 32 * j, S::kSmall - 1);  // lanes past the last piece copy it again
            const char *from;
            uint32_t at;
            if (m < 2 * G) {
                from = reinterpret_cast<const char *>(p.ks);
                stride[j] = S::kScales;
                at = S::ks;
            } else if (V && (m -= 2 * G) < 2 * G) {
                from = reinterpret_cast<const char *>(p.vs);
                stride[j] = S::kScales;
                at = S::vs;
            } else if ((m -= 2 * G) < 4) {
                from = reinterpret_cast<const char *>(p.kz);
                stride[j] = S::kZeros;
                at = S::kz;
            } else {
                m -= 4;
                from = reinterpret_cast<const char *>(p.vz);
                stride[j] = S::kZeros;
                at = S::vz;
            }
            small[j] = from + 16 * m;
            to[j] = at + 16 * m;
        }
    }
    __device__ __forceinline__ void copy(uint32_t dst, uint32_t unit, int lane) const {
        const char *k = kc + (uint64_t)unit * S::kCodes, *v = vc + (uint64_t)unit * S::kCodes;
#pragma unroll
        for (int c = 0; c < 16 * G; c += 32)
            if (c + 32 <= 16 * G || lane < 16 * G - c) {
                copy16(dst + S::kc + 16 * (c + lane), k + 16 * c);
                if (V) copy16(dst + S::vc + 16 * (c + lane), v + 16 * c);
            }
#pragma unroll
        for (int j = 0; j < S::kPer; ++j) copy16(dst + to[j], small[j] + (uint64_t)unit * stride[j]);
    }
};

// Byte offsets of a lane's own data within a unit's six arrays.  (Hidden from
// the compiler's arithmetic: it would recompute them for every unit.)
template <int G>
struct LaneOffsets {
    uint32_t kc, ks, kz, vc, vs, vz;
    __device__ __forceinline__ explicit LaneOffsets(int lane) {
        const int g = lane >> 2, t = lane & 3, up = unit_position(g);
        kc = (up * 4 * G + t * G) * 4;
        ks = up * G * 2;
        kz = up * 4;
        vc = (t * 8 * G + g * G) * 2;
        vs = t * G * 2;
        vz = t * 4;
        asm volatile("" : "+r"(kc), "+r"(ks), "+r"(kz), "+r"(vc), "+r"(vs), "+r"(vz));
    }
};

// One unit's K for this lane: rows lane/4 and lane/4 + 8.
template <int G>
struct KUnit {
    uint32_t w[2][G];
    uint32_t s[2][(G + 1) / 2];
    uint32_t z[2];
    // From the lane's places in a stage.
    __device__ __forceinline__ void load(Shared kc, Shared ks, Shared kz) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {  // unit_position(g + 8) = unit_position(g) + 8
            load_words<G>(w[r], kc + r * 8 * 16 * G);
            load_halfwords<G>(s[r], ks + r * 8 * 2 * G);
            z[r] = (kz + r * 8 * 4).get4();
        }
    }
    // The A operands of group gr from the codes as they stand, k-steps 0 and 1;
    // and row r's zero points of groups gr (even) and gr + 1, z * 2^-24 and
    // 16 z * 2^-24.
    __device__ __forceinline__ void raw_operands(int gr, uint32_t (&a0)[4], uint32_t (&a1)[4]) const {
        uint32_t x[2][4];
#pragma unroll
        for (int r = 0; r < 2; ++r) raw_codes(w[r][gr], x[r]);
        a0[0] = x[0][0]; a0[1] = x[1][0]; a0[2] = x[0][1]; a0[3] = x[1][1];
        a1[0] = x[0][2]; a1[1] = x[1][2]; a1[2] = x[0][3]; a1[3] = x[1][3];
    }
    __device__ __forceinline__ uint32_t raw_zeros(int r, int gr) const {
        return (__byte_perm(z[r], 0, gr < 4 ? 0x1010 : 0x3232) >> (gr & 2 ? 8 : 0)) & 0x00F0000Fu;
    }
    // The A operands of group gr less the zero points, k-steps 0 and 1.
    __device__ __forceinline__ void operands(int gr, uint32_t (&a0)[4], uint32_t (&a1)[4]) const {
        __half2 x[2][4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const uint32_t zp = __byte_perm(z[r], 0, gr < 4 ? 0x1010 : 0x3232) >> (gr & 2 ? 8 : 0);
            ZeroPair(zp, gr & 1).codes(w[r][gr], x[r]);
        }
        a0[0] = as_bits(x[0][0]); a0[1] = as_bits(x[1][0]); a0[2] = as_bits(x[0][1]); a0[3] = as_bits(x[1][1]);
        a1[0] = as_bits(x[0][2]); a1[1] = as_bits(x[1][2]); a1[2] = as_bits(x[0][3]); a1[3] = as_bits(x[1][3]);
    }
};

// One unit's V for this lane: positions t, t + 4, t + 8, t + 12 (t = lane % 4),
// channels 4g .. 4g + 3 of every group (g = lane / 4).
template <int G>
struct VUnit {
    static constexpr int W = (G + 1) / 2;
    uint32_t w[4][W];
    uint32_t s[4][W];
    uint32_t z[4];
    __device__ __forceinline__ void load(Shared vc, Shared vs, Shared vz) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            load_halfwords<G>(w[i], vc + i * 4 * 16 * G);
            load_halfwords<G>(s[i], vs + i * 4 * 2 * G);
            z[i] = (vz + i * 4 * 4).get4();
        }
    }
    // `left` positions belong to the sequence; entries past them may hold
    // anything, so their scales become 0.
    __device__ __forceinline__ void cut_off(int left, int lane) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if ((lane & 3) + 4 * i >= left)
#pragma unroll
                for (int k = 0; k < W; ++k) s[i][k] = 0u;
    }
    // The A operands of group gr from the codes as they stand, channels (4g, 4g +
    // 1) and (4g + 2, 4g + 3); and minus the zero points in the same form (the
    // same for both).
    __device__ __forceinline__ void raw_operands(int gr, uint32_t (&a0)[4], uint32_t (&a1)[4], uint32_t (&az)[4]) const {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            uint32_t x[4];
            raw_codes(__byte_perm(w[2 * r][gr / 2], w[2 * r + 1][gr / 2], gr & 1 ? 0x7632u : 0x5410u), x);
            a0[2 * r] = x[0]; a0[2 * r + 1] = x[1];
            a1[2 * r] = x[2]; a1[2 * r + 1] = x[3];
            const uint32_t zp = __byte_perm(z[2 * r], z[2 * r + 1], gr < 4 ? 0x5410u : 0x7632u) >> (gr & 2 ? 8 : 0);
            az[2 * r] = masked_or<0x000F000Fu>(gr & 1 ? zp >> 4 : zp, 0x80008000u);
            az[2 * r + 1] = masked_or<0x00F000F0u>(gr & 1 ? zp : zp << 4, 0x80008000u);
        }
    }
    // The scales times 2^pow, -17 <= pow <= 22.
    __device__ __forceinline__ void scale_by(int pow) {
        const uint32_t by = half_pow2(min(pow, 15)) * 0x10001u;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < W; ++k) s[i][k] = as_bits(__hmul2(as_half2(s[i][k]), as_half2(by)));
        if (pow > 15) {
            const uint32_t more = half_pow2(pow - 15) * 0x10001u;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int k = 0; k < W; ++k) s[i][k] = as_bits(__hmul2(as_half2(s[i][k]), as_half2(more)));
        }
    }
    // The scales of group gr at two of the lane's four positions.
    __device__ __forceinline__ __half2 scale_pair(int gr, int r) const {
        return as_half2(__byte_perm(s[2 * r][gr / 2], s[2 * r + 1][gr / 2], gr & 1 ? 0x7632u : 0x5410u));
    }
    // The A operands of group gr, channels (4g, 4g + 1) and (4g + 2, 4g + 3):
    // (c - z) * s rounded to FP16, and (EXACT) in l0, l1 what that left, which is
    // exact: the product has 15 bits at most and its last one is 2^-24 or more.
    template <bool EXACT>
    __device__ __forceinline__ void operands(int gr, uint32_t (&a0)[4], uint32_t (&a1)[4], uint32_t (&l0)[4],
                                             uint32_t (&l1)[4]) const {
        const uint32_t pick = gr & 1 ? 0x7632u : 0x5410u;
        uint32_t x[2][4], rest[2][4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const uint32_t c = __byte_perm(w[2 * r][gr / 2], w[2 * r + 1][gr / 2], pick);
            const uint32_t zp = __byte_perm(z[2 * r], z[2 * r + 1], gr < 4 ? 0x5410u : 0x7632u);
            __half2 v[4];
            ZeroPair(zp >> (gr & 2 ? 8 : 0), gr & 1).codes(c, v);
            const __half2 sc = as_half2(__byte_perm(s[2 * r][gr / 2], s[2 * r + 1][gr / 2], pick));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __half2 y = __hmul2(v[j], sc);
                x[r][j] = as_bits(y);
                if constexpr (EXACT) rest[r][j] = as_bits(__hfma2(v[j], sc, __hneg2(y)));
            }
        }
        a0[0] = x[0][0]; a0[1] = x[0][1]; a0[2] = x[1][0]; a0[3] = x[1][1];
        a1[0] = x[0][2]; a1[1] = x[0][3]; a1[2] = x[1][2]; a1[3] = x[1][3];
        if constexpr (EXACT) {
            l0[0] = rest[0][0]; l0[1] = rest[0][1]; l0[2] = rest[1][0]; l0[3] = rest[1][1];
            l1[0] = rest[0][2]; l1[1] = rest[0][3]; l1[2] = rest[1][2]; l1[3] = rest[1][3];
        }
    }
};

// One query vector's operands: group gr of the lane's 8 channels (t = lane %
// 4), pairs (q0, q4), (q1, q5) of k-step 0 and (q2, q6), (q3, q7) of k-step 1,
// the order in which ZeroPair::codes takes a word's nibbles.  `back` undoes the
// row's power of two.  Rows lie on groups of 4 lanes; all lanes of the warp call
// it (q is null for a column without a query).
// RAW, for codes as they stand: q1, q3, q5, q7 divided by 16; and in `zero` minus
// the group's sum of the query, as the zero points' form wants it (an odd
// group's divided by 16).
template <int G, bool RAW>
__device__ __forceinline__ void query_operands(const uint16_t *q, int t, uint4 (&f)[G], float &back,
                                               float (&zero)[RAW ? G : 1]) {
    uint32_t top = 0;
#pragma unroll
    for (int gr = 0; gr < G; ++gr) {
        f[gr] = q ? *reinterpret_cast<const uint4 *>(q + 32 * gr + 8 * t) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t w[4] = {f[gr].x, f[gr].y, f[gr].z, f[gr].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max(top, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
    }
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const uint32_t e = max(top >> 7, 16u);  // the largest value's exponent field (2^-111 or less: as 2^-111)
    const float up = __uint_as_float((268u - e) << 23);
    back = e == 255u ? __int_as_float(0x7FC00000) : __uint_as_float((e - 14u) << 23);  // NaN: q is not finite
#pragma unroll
    for (int gr = 0; gr < G; ++gr) {
        const uint32_t w[4] = {f[gr].x, f[gr].y, f[gr].z, f[gr].w};
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16) * up;
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u) * up;
        }
        constexpr float odd = RAW ? 0.0625f : 1.f;
        f[gr] = make_uint4(f16_pair(v[0], v[4]), f16_pair(v[1] * odd, v[5] * odd), f16_pair(v[2], v[6]),
                           f16_pair(v[3] * odd, v[7] * odd));
        if constexpr (RAW) {
            const float even = half_of(f[gr].x, 0) + half_of(f[gr].x, 1) + half_of(f[gr].z, 0) + half_of(f[gr].z, 1);
            const float odds = half_of(f[gr].y, 0) + half_of(f[gr].y, 1) + half_of(f[gr].w, 0) + half_of(f[gr].w, 1);
            float sum = -fmaf(16.f, odds, even);
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            zero[gr] = gr & 1 ? sum * 0.0625f : sum;
        }
    }
}

// tanh to a relative 1.5 * 2^-22: a score is the cap times it, so an absolute error
// would grow with the cap.  Under kTanhNear y + y^3 p(y^2), p of degree 4 fitted to
// the least relative error (4.1e-9; 1.3 * 2^-24 with its roundings); over it 1 - 2 /
// (exp(2y) + 1), where the exponential's 2^-22 and the reciprocal's 2^-23 count by
// 0.35 and 0.45 of 0.55 or more.  Scores are mostly well under their cap, so a warp's step takes the second
// form only where one of its values wants it.
constexpr float kTanhNear = 0.625f;
__device__ __forceinline__ float tanh_near(float y) {
    const float u = y * y;
    float p = fmaf(u, -0.00571703365f, 0.0206505762f);
    p = fmaf(p, u, -0.0537434943f);
    p = fmaf(p, u, 0.133314912f);
    p = fmaf(p, u, -0.333332839f);
    return fmaf(p, u * y, y);
}
__device__ __forceinline__ float tanh_any(float y) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(ex2(2.f * kLog2e * fabsf(y)) + 1.f));
    return fabsf(y) < kTanhNear ? tanh_near(y) : copysignf(fmaf(-2.f, r, 1.f), y);
}

// What turns a product sum (its factor taken in) into a score in base 2.
struct Score {
    float mul, cap;  // without a cap: s = mul * dot; with: cap * tanh(mul * dot)
    bool capped;
    __device__ __forceinline__ explicit Score(const PagedArgs &a) {
        // (a cap over 2^100 changes no score under 2^88, and its product with log2 e
        // might not be finite)
        capped = a.cap > 0.f && a.cap < 0x1p100f;
        mul = capped ? a.scale / a.cap : a.scale * kLog2e;
        cap = a.cap * kLog2e;
    }
    // Caps a step's values, N of this lane's.
    template <int N>
    __device__ __forceinline__ void cap_all(float (&y)[N]) const {
        bool near = true;
#pragma unroll
        for (int i = 0; i < N; ++i) near = near && fabsf(y[i]) < kTanhNear;
        if (__all_sync(0xffffffffu, near)) {
#pragma unroll
            for (int i = 0; i < N; ++i) y[i] = cap * tanh_near(y[i]);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) y[i] = cap * tanh_any(y[i]);
        }
    }
};

// (No pool has 2^31 units: they would be 4 TB and more.)
constexpr uint32_t kNoUnit = 0xFFFFFFFFu, kSpecial = 0x80000000u;
// The unit of the pool that holds positions t0 .. t0 + 15 of head h; kNoUnit
// for a page outside the pool.  (Units number under 2^31.)
__device__ __forceinline__ uint32_t unit_of(const PoolView &p, int32_t page, int t0, int h) {
    if ((uint32_t)page >= (uint32_t)p.n_pages) {
        atomicOr(&g_paged_error, 4u);
        return kNoUnit;
    }
    return (((uint32_t)page * (uint32_t)p.H + (uint32_t)h) << (p.lp - 4)) + ((uint32_t)(t0 & ((1 << p.lp) - 1)) >> 4);
}

constexpr int kStages = 3;

// The bits of the largest scale of V, without its sign (a pool's own are positive),
// over a warp's units (U at a time, from t0) with positions from `lo` on and before
// t_end, of a length of n positions.
template <int G, int U>
__device__ __forceinline__ uint32_t largest_scale(const PoolView &p, const int32_t *pages, int h, int t0, int lo,
                                                  int t_end, int n) {
    uint32_t most = 0;
    for (int f = threadIdx.x & 31;; f += 32) {
        const int t = t0 + f / U * kTile<U> + f % U * kUnit;
        if (t >= t_end) break;
        if (t + kUnit <= lo) continue;
        const uint32_t unit = unit_of(p, pages[t >> p.lp], t, h);
        if (unit == kNoUnit) continue;
        const uint16_t *at = p.vs + (uint64_t)unit * kUnit * G;
        const int count = min(kUnit, n - t) * G;  // (of what lies behind them nothing counts)
#pragma unroll 4
        for (int k = 0; k < 2 * G; ++k) {
            const uint4 w4 = reinterpret_cast<const uint4 *>(at)[k];
            const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (8 * k + 2 * e < count) most = max(most, w[e] & 0x7FFFu);
                if (8 * k + 2 * e + 1 < count) most = max(most, w[e] >> 16 & 0x7FFFu);
            }
        }
    }
    return __reduce_max_sync(0xffffffffu, most);
}

// A warp's way through its units of one item, U at a step: unit j of step i is
// the positions t0 + i * kTile<U> + 16 j .. + 15.  Copies run kStages - 1 steps
// ahead, a group each.  The bookkeeping is done 32 units at a time: a lane finds
// one unit's place in the pool; the top bit marks a unit with positions that some
// column does not see, or none does (one past the end, a page outside the pool).
template <int G, bool V, int U>
struct UnitRing {
    using S = Stage<G, V>;
    const PoolView &p;
    const Copier<G, V> &copier;
    const int32_t *pages;
    uint32_t first;  // the ring's address
    int h, t0, t_end, pos_lo, pos_hi, window, lane;
    int steps;
    uint32_t units = 0, before = 0;              // the units looked up last, and the 32 before those
    uint32_t marks = 0, at = 0, done = 0;        // marks: bit i is that of the unit fetched i ago

    __device__ __forceinline__ int position(int f) const { return t0 + f / U * kTile<U> + f % U * kUnit; }
    __device__ __forceinline__ void look_up(int f) {
        const int t = position(f + lane);
        before = units;
        units = kNoUnit;
        // (a unit wholly behind the window may lie on a page that was freed)
        if (t < t_end && !(window > 0 && t + kUnit - 1 <= pos_lo - window)) {
            const uint32_t unit = unit_of(p, pages[t >> p.lp], t, h);
            if (unit != kNoUnit) {
                units = unit;
                if (t + kUnit - 1 > pos_lo || (window > 0 && t <= pos_hi - window)) units |= kSpecial;
            }
        }
    }
    __device__ __forceinline__ void fetch(int step, uint32_t dst) {
        if (step < steps) {
            if ((step * U & 31) == 0) look_up(step * U);
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const uint32_t unit = __shfl_sync(0xffffffffu, units, step * U + j);
                // unit 0 in the place of one that is not there
                copier.copy(dst + j * S::kBytes, unit == kNoUnit ? 0u : unit & ~kSpecial, lane);
                marks = __funnelshift_l(unit, marks, 1);
            }
        } else {
            marks <<= U;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    __device__ __forceinline__ void start() {
        steps = t0 < t_end ? (t_end - t0 + kTile<U> - 1) / kTile<U> : 0;
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) fetch(i, first + i * U * S::kBytes);
        at = first;
        done = first + (kStages - 1) * U * S::kBytes;
    }
    // Step i's stage, once every lane's copies of it have landed.
    __device__ __forceinline__ Shared next(int i) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
        __syncwarp();  // and nobody reads the last step's stage any more
        fetch(i + kStages - 1, done);
        done = at;
        at = at == first + (kStages - 1) * U * S::kBytes ? first : at + U * S::kBytes;
        return {done};
    }
    __device__ __forceinline__ bool marked() const { return marks & (((1u << U) - 1) << ((kStages - 1) * U)); }
    // Unit j of step i (the last that `next` gave): its place in the pool, or kNoUnit.
    __device__ __forceinline__ uint32_t unit(int i, int j) const {
        const int f = i * U + j;
        const uint32_t u = __shfl_sync(0xffffffffu, looked_ahead(i) ? before : units, f);
        return u == kNoUnit ? u : u & ~kSpecial;
    }
    // The bits of the largest scale of V, without its sign, of step 0's entries, whose stage is waited
    // for (vs: LaneOffsets), of a length of n positions.
    __device__ __forceinline__ uint32_t first_scales(int n, uint32_t vs) const {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
        __syncwarp();
        auto size = [](uint32_t x) { return __habs2(as_half2(x)); };
        if (__all_sync(0xffffffffu, lane >= U || !(units & kSpecial))) {  // whole units: 8 scales a lane
            const int piece = min(lane, U * 2 * G - 1), j = piece / (2 * G);
            const uint4 w = (Shared{first} + j * S::kBytes + S::vs + 16 * (piece - j * 2 * G)).get16();
            const uint32_t b = as_bits(__hmax2(__hmax2(size(w.x), size(w.y)), __hmax2(size(w.z), size(w.w))));
            return __reduce_max_sync(0xffffffffu, max(b & 0xFFFFu, b >> 16));
        }
        uint32_t most = 0;
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int left = unit(0, j) == kNoUnit ? 0 : n - position(j);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t w[(G + 1) / 2];
                load_halfwords<G>(w, Shared{first} + j * S::kBytes + S::vs + vs + i * 4 * 2 * G);
                if ((lane & 3) + 4 * i < left)
#pragma unroll
                    for (int k = 0; k < (G + 1) / 2; ++k) most = max(most, max(w[k] & 0x7FFFu, w[k] >> 16 & 0x7FFFu));
            }
        }
        return __reduce_max_sync(0xffffffffu, most);
    }
    // Whether the units of a later step have been looked up since step i's.
    __device__ __forceinline__ bool looked_ahead(int i) const {
        return ((i * U ^ min(i + kStages - 1, steps - 1) * U) & ~31) != 0;
    }
};

// This CTA's run of the tile list and where it starts: sequence b, `off` tiles
// into it.
struct Run {
    int64_t cur, end, total;
    int64_t off;
    int b, runs;
};

// a / b, with the short division where it will do.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    if ((uint64_t)(a | b) >> 32 == 0) return (int64_t)((uint32_t)a / (uint32_t)b);
    return a / b;
}

// per_seq(b): tiles of sequence b in the list.
template <class F>
__device__ __forceinline__ Run find_run(const F &per_seq, int n_seq, int run, int max_runs, int min_tiles, int64_t *part,
                                        int64_t *found) {
    const int tid = threadIdx.x, per = (n_seq + kThreads - 1) / kThreads;
    const int b0 = min(n_seq, tid * per), b1 = min(n_seq, b0 + per);
    int64_t own = 0;
    for (int b = b0; b < b1; ++b) own += per_seq(b);
    Run r;
    int64_t before = block_exclusive(own, part, &r.total);
    const int64_t want = (r.total + min_tiles - 1) / min_tiles;
    r.runs = (int)(want < max_runs ? want : max_runs);
    if (run >= r.runs) {
        r.cur = r.end = r.off = 0;
        r.b = 0;
        return r;
    }
    r.cur = quotient(run * r.total, r.runs);
    r.end = quotient((run + 1) * r.total, r.runs);
    if (before <= r.cur && r.cur < before + own) {
        for (int b = b0;; ++b) {
            const int64_t n = per_seq(b);
            if (r.cur < before + n) {
                found[0] = b;
                found[1] = r.cur - before;
                break;
            }
            before += n;
        }
    }
    __syncthreads();
    r.b = (int)found[0];
    r.off = found[1];
    return r;
}

// The run that holds tile t of the list.
__device__ __forceinline__ int run_of(int64_t t, const Run &r) {
    return (int)quotient((t + 1) * r.runs - 1, r.total);
}

// Four channels of an output row: the weighted sum over the sum of weights.
template <bool EXACT>
__device__ __forceinline__ void store_out(const PagedArgs &a, int64_t at, float4 v, float l) {
    const float r = l > 0.f ? 1.f / l : 0.f;
    v = make_float4(v.x * r, v.y * r, v.z * r, v.w * r);
    if (EXACT) {
        *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at) = v;
    } else {
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + at) =
            make_uint2(bf16_pair(v.x, v.y), bf16_pair(v.z, v.w));
    }
    if (!(isfinite(v.x) && isfinite(v.y) && isfinite(v.z) && isfinite(v.w))) atomicOr(&g_paged_error, 2u);
}

// A row's lse from its reference and sum (base 2).  The accumulated weights take the
// two apart, reference and inverse sum, so that a score and the reference, both of
// them large perhaps, are subtracted before anything is rounded to their size.
// A row that saw nothing, or whose query is not finite (l is NaN then, and so is its
// lse): infinity and 0, which make every weight 0.
__device__ __forceinline__ void store_lse(const PagedArgs &a, int64_t row, float m, float l) {
    if (a.lse) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    if (a.ws_row) a.ws_row[row] = l > 0.f ? make_float2(m, 1.f / l) : make_float2(INFINITY, 0.f);
}

// Units of a step: two where the accumulators leave the registers for it (the
// loop's own work is done once for both, and their instructions interleave).
template <int G, int NT>
constexpr int units_per_step() {
    return G * NT <= 4 ? 2 : 1;
}
// (Three CTAs an SM where two would have registers to spare: under the bound FP32
// decode keeps 312 bytes a thread in local memory at D = 256 and 108 at 224, BF16
// decode 156 and 64, the other forms 60 or less, but 116 at D = 32 with 32 columns; the
// join of few pieces 8 to 104.)
template <int G, int NT>
constexpr int min_ctas() {
    return G * NT <= 8 ? 3 : 2;
}

// Shared memory: the warps' stages, which the exchange of the warps' sums
// takes over at an item's end; then the queries' operands of several n-tiles.
template <int G, int U>
constexpr int ring_bytes() {
    constexpr int ring = kWarps * kStages * U * Stage<G, true>::kBytes, xch = kWarps * 8 * (32 * G + 4) * 4;
    return ring > xch ? ring : xch;
}

template <int G, int NT, bool EXACT>
__global__ void __launch_bounds__(kThreads, min_ctas<G, NT>()) paged_attention_kernel(const PagedArgs a) {
    constexpr int U = units_per_step<G, NT>();
    // codes as they stand: of K, and of V (whose zero points take a product of
    // their own, dearer for many columns than subtracting them once)
    constexpr bool kRawK = NT == 1, kRawV = NT == 1 && !EXACT;
    constexpr int D = 32 * G, C = 8 * NT, kRow = D + 4;  // kRow: a padded column of the exchange buffer
    extern __shared__ __align__(16) unsigned char smem[];
    float *xch = reinterpret_cast<float *>(smem);                      // [kWarps][8][kRow]
    uint4 *qs = reinterpret_cast<uint4 *>(smem + ring_bytes<G, U>());  // NT > 1: [NT][G][32]
    __shared__ float2 s_ml[kWarps][C];
    __shared__ float s_back[C];
    __shared__ float2 s_col[kWarps][C];  // a column's position and slope (each warp its own copy)
    __shared__ int64_t s_part[33], s_found[2];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    const PoolView &p = a.p;
    const Copier<G, true> copier(p, lane);
    const LaneOffsets<G> lo(lane);
    using S = Stage<G, true>;
    const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(smem) + warp * kStages * U * S::kBytes;
    const Score score(a);
    const bool shaped = score.capped || a.slopes;  // scores are more than a multiple of the products

    // the join may be launched: it waits for this grid's end before it reads
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    auto per_seq = [&](int b) -> int64_t {
        const Sequence s = sequence_of(a, b);
        return s.m == 0 ? 0 : (int64_t)p.H * ((s.m * a.grp + C - 1) / C) * tiles_of<U>(a, s).count;
    };
    Run run = find_run(per_seq, a.n_seq, blockIdx.x, gridDim.x, kMinPositions / kTile<U>, s_part, s_found);
    int4 cut = make_int4(-1, 0, 0, 0);
    int b = run.b;
    while (run.cur < run.end) {
        const Sequence s = sequence_of(a, b);
        const Tiles tiles = tiles_of<U>(a, s);
        const int ncols = s.m * a.grp, n_ct = (ncols + C - 1) / C;
        if (s.m == 0 || run.off >= (int64_t)p.H * n_ct * tiles.count) {
            ++b;
            run.off = 0;
            continue;
        }
        const int item = (int)quotient(run.off, tiles.count);
        const int ta = (int)(run.off - (int64_t)item * tiles.count);
        const int tb = (int)min((int64_t)tiles.count, ta + (run.end - run.cur));
        const int h = item / n_ct, c0 = (item - h * n_ct) * C;
        const int cols = min(C, ncols - c0);
        const int pos_lo = s.n - s.m + c0 / a.grp, pos_hi = s.n - s.m + (c0 + cols - 1) / a.grp;
        const int vis_lo = a.window > 0 ? max(0, pos_lo - a.window + 1) : 0;  // the first position any column sees
        // this warp's units: tiles first + ta .. first + tb - 1 that any column sees
        const int32_t *pages = a.pages + (int64_t)b * a.max_pages;
        const int t_end = min((tiles.first + tb - kItemCost<U>) * kTile<U>, min(s.n, pos_hi + 1));
        int t0 = (tiles.first + max(0, ta - kItemCost<U>)) * kTile<U> + warp * (U * kUnit);
        while (t0 + U * kUnit <= vis_lo) t0 += kTile<U>;
        uint4 qf[G];
        float mul[NT][2], qz[kRawK ? G : 1][2];
        float ref[NT][2], limit[NT][2], sum[NT][2], o[NT][G][2][4];
        // V's scales go into the products times 2^v_pow, which brings the first step's
        // largest to 2^-3 .. 2; where scales grow so far that a product passes FP16's
        // range, the item is run again, with the largest of all.
#pragma unroll 1
        for (bool again = false;; again = true) {
        UnitRing<G, true, U> ring{p, copier, pages, ring_at, h, t0, t_end, pos_lo, pos_hi, a.window, lane};
        ring.start();  // the first units are on their way while the queries are prepared
        if (!again) {
        if (lane < C) {
            const int c = c0 + min(lane, cols - 1);
            s_col[warp][lane] = make_float2(__int_as_float(s.n - s.m + c / a.grp),
                                            a.slopes ? a.slopes[h * a.grp + c % a.grp] * kLog2e : 0.f);
        }
        __syncwarp();
        // queries: column g of every n-tile (zeros past the last column); mul
        // is what this lane's columns' products are multiplied with
        auto query_row = [&](int nt) -> const uint16_t * {
            const int c = c0 + 8 * nt + g;
            return 8 * nt + g < cols
                       ? a.q + ((int64_t)(s.row0 + c / a.grp) * a.Hq + h * a.grp + c % a.grp) * D : nullptr;
        };
        if constexpr (NT == 1) {
            float back, zero[G];
            query_operands<G, true>(query_row(0), t4, qf, back, zero);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                mul[0][e] = score.mul * __shfl_sync(0xffffffffu, back, 4 * (2 * t4 + e));
#pragma unroll
                for (int gr = 0; gr < G; ++gr) qz[gr][e] = __shfl_sync(0xffffffffu, zero[gr], 4 * (2 * t4 + e));
            }
        } else {
            for (int nt = warp; nt < NT; nt += kWarps) {
                float back, none[1];
                query_operands<G, false>(query_row(nt), t4, qf, back, none);
#pragma unroll
                for (int gr = 0; gr < G; ++gr) qs[(nt * G + gr) * 32 + lane] = qf[gr];
                if (t4 == 0) s_back[8 * nt + g] = back;
            }
            __syncthreads();
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) mul[nt][e] = score.mul * s_back[8 * nt + 2 * t4 + e];
        }
        }
        // ref: what weights are relative to; limit: the score that moves it
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            ref[nt][0] = ref[nt][1] = 0.f;
            limit[nt][0] = limit[nt][1] = -INFINITY;
            sum[nt][0] = sum[nt][1] = 0.f;
#pragma unroll
            for (int gr = 0; gr < G; ++gr)
#pragma unroll
                for (int i = 0; i < 8; ++i) o[nt][gr][i >> 2][i & 3] = 0.f;
        }

        int v_pow = 0;
        if constexpr (kRawV) {
            uint32_t most = again || ring.steps == 0 ? 0u : ring.first_scales(s.n, lo.vs);
            if (most == 0) most = largest_scale<G, U>(p, pages, h, t0, vis_lo, t_end, s.n);
            if (most > 0) {
                const int e = half_exponent(most);
                v_pow = e >= -3 && e <= 0 ? 0 : -2 - e;
            }
        }
        auto units = [&](auto scaled) {
        for (int i = 0; i < ring.steps; ++i) {
            const Shared here = ring.next(i);
            float x[U][NT][4];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const Shared at = here + j * S::kBytes;
                KUnit<G> ku;
                ku.load(at + S::kc + lo.kc, at + S::ks + lo.ks, at + S::kz + lo.kz);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[j][nt][e] = 0.f;
#pragma unroll
                for (int gr = 0; gr < G; ++gr) {
                    uint32_t a0[4], a1[4];
                    if constexpr (kRawK) ku.raw_operands(gr, a0, a1);
                    else ku.operands(gr, a0, a1);
                    const float s0 = half_of(ku.s[0][gr / 2], gr & 1), s1 = half_of(ku.s[1][gr / 2], gr & 1);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        uint4 q4;
                        if constexpr (NT == 1) q4 = qf[gr];
                        else q4 = qs[(nt * G + gr) * 32 + lane];
                        float d[4];
                        mma_first(d, a0, q4.x, q4.y);
                        mma(d, a1, q4.z, q4.w);
                        if constexpr (kRawK) {
                            const float z0 = half_of(ku.raw_zeros(0, gr), gr & 1), z1 = half_of(ku.raw_zeros(1, gr), gr & 1);
                            d[0] = fmaf(z0, qz[gr][0], d[0]);
                            d[1] = fmaf(z0, qz[gr][1], d[1]);
                            d[2] = fmaf(z1, qz[gr][0], d[2]);
                            d[3] = fmaf(z1, qz[gr][1], d[3]);
                        }
                        x[j][nt][0] = fmaf(d[0], s0, x[j][nt][0]);
                        x[j][nt][1] = fmaf(d[1], s0, x[j][nt][1]);
                        x[j][nt][2] = fmaf(d[2], s1, x[j][nt][2]);
                        x[j][nt][3] = fmaf(d[3], s1, x[j][nt][3]);
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[j][nt][e] = (kRawK ? x[j][nt][e] * kRaw : x[j][nt][e]) * mul[nt][e & 1];
            }
            if (shaped) {
                if (score.capped) score.cap_all(reinterpret_cast<float(&)[U * NT * 4]>(x));
#pragma unroll
                for (int j = 0; j < U; ++j)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float2 col = s_col[warp][8 * nt + 2 * t4 + e];
                            const int gap = __float_as_int(col.x) - (t0 + i * kTile<U> + j * kUnit) - unit_position(g);
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                x[j][nt][2 * r + e] = fmaf(-col.y, (float)(gap - 8 * r), x[j][nt][2 * r + e]);
                            }
                        }
            }
            const bool marked = ring.marked();
            if (marked) {
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    const int t = t0 + i * kTile<U> + j * kUnit;
                    const bool gone = ring.unit(i, j) == kNoUnit;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int pos = __float_as_int(s_col[warp][8 * nt + 2 * t4 + e].x);
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                const int gap = pos - t - unit_position(g) - 8 * r;
                                if (gone || gap < 0 || (a.window > 0 && gap >= a.window)) x[j][nt][2 * r + e] = -INFINITY;
                            }
                        }
                }
            }
            bool up = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float m = fmaxf(x[0][nt][e], x[0][nt][2 + e]);
                    if (U > 1) m = fmaxf(m, fmaxf(x[U - 1][nt][e], x[U - 1][nt][2 + e]));
                    up |= m > limit[nt][e];
                }
            if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float m = fmaxf(x[0][nt][e], x[0][nt][2 + e]);
                        if (U > 1) m = fmaxf(m, fmaxf(x[U - 1][nt][e], x[U - 1][nt][2 + e]));
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
                        // a column that saw nothing yet keeps its zeros
                        const bool first = limit[nt][e] == -INFINITY;
                        const float under = m - kRefBelow;
                        const float to = m == -INFINITY ? ref[nt][e] : (first ? under : fmaxf(under, ref[nt][e]));
                        const float f = first ? 1.f : ex2(ref[nt][e] - to);
                        // (rounded down: up, at scores past 2^24, a weight would leave FP16's range)
                        if (m > -INFINITY) limit[nt][e] = __fadd_rd(to, kRawV ? kRefRoomRaw : kRefRoom);
                        ref[nt][e] = to;
                        sum[nt][e] *= f;
#pragma unroll
                        for (int gr = 0; gr < G; ++gr) {
                            o[nt][gr][0][e] *= f;
                            o[nt][gr][0][2 + e] *= f;
                            o[nt][gr][1][e] *= f;
                            o[nt][gr][1][2 + e] *= f;
                        }
                    }
            }
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const Shared at = here + j * S::kBytes;
                VUnit<G> vu;
                vu.load(at + S::vc + lo.vc, at + S::vs + lo.vs, at + S::vz + lo.vz);
                if (marked) {
                    const int t = t0 + i * kTile<U> + j * kUnit;
                    vu.cut_off(ring.unit(i, j) == kNoUnit ? 0 : s.n - t, lane);
                }
                if constexpr (decltype(scaled)::value) vu.scale_by(v_pow);
                // the weights as B operands: b, and (EXACT) what its rounding left
                uint32_t b[NT][2];
                [[maybe_unused]] uint32_t rest[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float w0 = ex2(x[j][nt][2 * r] - ref[nt][0]), w1 = ex2(x[j][nt][2 * r + 1] - ref[nt][1]);
                        sum[nt][0] += w0;
                        sum[nt][1] += w1;
                        const uint32_t h2 = f16_pair(w0, w1);
                        b[nt][r] = transpose8x8(h2);
                        if constexpr (EXACT)
                            rest[nt][r] = transpose8x8(f16_pair(w0 - half_of(h2, 0), w1 - half_of(h2, 1)));
                    }
#pragma unroll
                for (int gr = 0; gr < G; ++gr) {
                    uint32_t a0[4], a1[4], l0[4], l1[4];
                    if constexpr (kRawV) {
                        vu.raw_operands(gr, a0, a1, l0);
                        const uint32_t b0 = as_bits(__hmul2(as_half2(b[0][0]), vu.scale_pair(gr, 0)));
                        const uint32_t b1 = as_bits(__hmul2(as_half2(b[0][1]), vu.scale_pair(gr, 1)));
                        mma(o[0][gr][0], a0, b0, b1);
                        mma(o[0][gr][1], a1, b0, b1);
                        mma(o[0][gr][0], l0, b0, b1);
                        mma(o[0][gr][1], l0, b0, b1);
                        continue;
                    }
                    vu.template operands<EXACT>(gr, a0, a1, l0, l1);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        if constexpr (EXACT) {
                            // summed apart and added in FP32: the tensor core cuts
                            // its sums off, which would add up over a long context
                            float d0[4], d1[4];
                            mma_first(d0, l0, b[nt][0], b[nt][1]);
                            mma_first(d1, l1, b[nt][0], b[nt][1]);
                            mma(d0, a0, rest[nt][0], rest[nt][1]);
                            mma(d1, a1, rest[nt][0], rest[nt][1]);
                            mma(d0, a0, b[nt][0], b[nt][1]);
                            mma(d1, a1, b[nt][0], b[nt][1]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                o[nt][gr][0][e] += d0[e];
                                o[nt][gr][1][e] += d1[e];
                            }
                        } else {
                            mma(o[nt][gr][0], a0, b[nt][0], b[nt][1]);
                            mma(o[nt][gr][1], a1, b[nt][0], b[nt][1]);
                        }
                    }
                }
            }
        }
        };
        if (kRawV && v_pow != 0) units(std::integral_constant<bool, kRawV>());
        else units(std::false_type());
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        if constexpr (kRawV) {
            float odd = 0.f;  // NaN if a sum is not finite (though its query is)
#pragma unroll
            for (int gr = 0; gr < G; ++gr)
#pragma unroll
                for (int e = 0; e < 8; ++e) odd = fmaf(mul[0][e & 1] == mul[0][e & 1] ? o[0][gr][e >> 2][e & 3] : 0.f, 0.f, odd);
            if (!again && __any_sync(0xffffffffu, odd != 0.f)) continue;
            const float f = kRaw * pow2(-v_pow);
#pragma unroll
            for (int gr = 0; gr < G; ++gr)
#pragma unroll
                for (int e = 0; e < 8; ++e) o[0][gr][e >> 2][e & 3] *= e & 2 ? f * 0.0625f : f;  // rows g + 8: odd codes
        }
        break;
        }
        // the exchange buffer takes the ring's place
        __syncthreads();

        // join the four warps; a whole item is written out, a piece of one kept
        const bool whole = ta == 0 && tb == tiles.count;
        const int64_t slot = 2 * (int64_t)blockIdx.x + (ta > 0 ? 0 : 1);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) sum[nt][e] += __shfl_xor_sync(0xffffffffu, sum[nt][e], d);
                if (g == 0)
                    s_ml[warp][8 * nt + 2 * t4 + e] =
                        make_float2(limit[nt][e] == -INFINITY ? -INFINITY : ref[nt][e], sum[nt][e]);
            }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if (8 * nt >= cols) break;
#pragma unroll
            for (int gr = 0; gr < G; ++gr)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    *reinterpret_cast<float4 *>(xch + (warp * 8 + 2 * t4 + e) * kRow + 32 * gr + 4 * g) =
                        make_float4(o[nt][gr][0][e], o[nt][gr][0][2 + e], o[nt][gr][1][e], o[nt][gr][1][2 + e]);
            __syncthreads();
            for (int i = tid; i < min(8, cols - 8 * nt) * (D / 4); i += kThreads) {
                const int cl = i / (D / 4), d = 4 * (i - cl * (D / 4)), c = 8 * nt + cl;
                float m = -INFINITY, l = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s_ml[w][c].x);
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float f = s_ml[w][c].x == -INFINITY ? 0.f : ex2(s_ml[w][c].x - m);
                    const float4 u = *reinterpret_cast<const float4 *>(xch + (w * 8 + cl) * kRow + d);
                    l = fmaf(f, s_ml[w][c].y, l);
                    v.x = fmaf(f, u.x, v.x);
                    v.y = fmaf(f, u.y, v.y);
                    v.z = fmaf(f, u.z, v.z);
                    v.w = fmaf(f, u.w, v.w);
                }
                if (whole) {
                    const int64_t row = (int64_t)(s.row0 + (c0 + c) / a.grp) * a.Hq + h * a.grp + (c0 + c) % a.grp;
                    store_out<EXACT>(a, row * D + d, v, l);
                    if (d == 0) store_lse(a, row, m, l);
                } else {
                    *reinterpret_cast<float4 *>(a.ws_acc + (slot * C + c) * D + d) = v;
                    if (d == 0) a.ws_ml[slot * C + c] = make_float2(m, l);
                }
            }
            __syncthreads();
        }
        if (ta == 0 && !whole) {
            cut.x = run_of(run.cur + tiles.count - 1, run);
            cut.y = s.row0;
            cut.z = c0 | (cols << 24);
            cut.w = h;
        }
        run.cur += tb - ta;
        run.off += tb - ta;
    }
    if (tid == 0) a.ws_item[blockIdx.x] = cut;
}

// Joins the pieces of the item that was cut at the end of run blockIdx.x: piece 0
// in that run's second place, the others in the first place of the following runs.
// Of few pieces (a batch: most items lie in one run or two) each thread joins four
// channels of a column, with all its loads in flight; of many (a long sequence) a
// CTA takes a column, its threads the pieces side by side, and the first loads of
// the sums do not wait for the weights.  LONG: for few items in many runs, the
// second form alone (a smaller kernel starts sooner: 1 sequence of 300 positions
// takes 1.3 us less than with both).  Bound by its launch and the trips to L2.
constexpr int kJoinThreads = 128, kFewPieces = 4;
template <int G, int NT, bool EXACT, bool LONG>
__global__ void __launch_bounds__(kJoinThreads, LONG ? 7 : 8) paged_join_kernel(const PagedArgs a) {
    constexpr int D = 32 * G, C = 8 * NT, Q = D / 4, kSplit = kJoinThreads / Q;  // Q threads per piece, kSplit pieces at once
    constexpr int kAhead = 8, kW = kJoinThreads / 32;
    __shared__ float4 s_v[kJoinThreads];
    __shared__ float s_f[kMaxCtas], s_m[kW], s_l[kW];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 cut = a.ws_item[blockIdx.x];
    const int c0 = cut.z & 0xFFFFFF, cols = cut.z >> 24;
    if (cut.x < 0) return;
    const int np = cut.x - (int)blockIdx.x + 1;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto finish = [&](int c, int d, const float4 &v, float m, float l) {
        const int h = cut.w;
        const int64_t row = (int64_t)(cut.y + (c0 + c) / a.grp) * a.Hq + h * a.grp + (c0 + c) % a.grp;
        store_out<EXACT>(a, row * D + d, v, l);
        if (d == 0) store_lse(a, row, m, l);
    };
    if (!LONG && np <= kFewPieces) {
        for (int i = blockIdx.y * kJoinThreads + tid; i < cols * Q; i += gridDim.y * kJoinThreads) {
            const int c = i / Q, d = 4 * (i - c * Q);
            float2 x[kFewPieces];
            float4 u[kFewPieces];
            float m = -INFINITY, l = 0.f;
#pragma unroll
            for (int k = 0; k < kFewPieces; ++k) {
                const int64_t at = (2 * ((int64_t)blockIdx.x + k) + (k == 0)) * C + c;
                x[k] = k < np ? a.ws_ml[at] : make_float2(-INFINITY, 0.f);
                u[k] = k < np ? *reinterpret_cast<const float4 *>(a.ws_acc + at * D + d) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int k = 0; k < kFewPieces; ++k) m = fmaxf(m, x[k].x);
            const float mm = m == -INFINITY ? 0.f : m;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < kFewPieces; ++k) {
                const float f = ex2(x[k].x - mm);
                l = fmaf(f, x[k].y, l);
                v.x = fmaf(f, u[k].x, v.x);
                v.y = fmaf(f, u[k].y, v.y);
                v.z = fmaf(f, u[k].z, v.z);
                v.w = fmaf(f, u[k].w, v.w);
            }
            finish(c, d, v, m, l);
        }
        return;
    }
    // (a turn's shared values are last read before the next turn's second barrier)
    for (int c = blockIdx.y; c < cols; c += gridDim.y) {
    auto at = [&](int i) -> int64_t { return (2 * ((int64_t)blockIdx.x + i) + (i == 0)) * C + c; };
    const int part = tid / Q, d = 4 * (tid - part * Q);
    const bool summing = part < kSplit;
    // the first pieces' sums are on their way while the weights are found
    float4 ahead[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
        const int i = part + j * kSplit;
        if (summing && i < np) ahead[j] = *reinterpret_cast<const float4 *>(a.ws_acc + at(i) * D + d);
    }
    constexpr int kOwn = (kMaxCtas + kJoinThreads - 1) / kJoinThreads;
    float2 own[kOwn];
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
        const int i = tid + j * kJoinThreads;
        own[j] = i < np ? a.ws_ml[at(i)] : make_float2(-INFINITY, 0.f);
        m = fmaxf(m, own[j].x);
    }
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) s_m[warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kW; ++w) m = fmaxf(m, s_m[w]);
    const float mm = m == -INFINITY ? 0.f : m;
    float l = 0.f;
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
        const int i = tid + j * kJoinThreads;
        const float f = ex2(own[j].x - mm);
        if (i < np) s_f[i] = f;
        l = fmaf(f, own[j].y, l);
    }
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) s_l[warp] = l;
    __syncthreads();
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](int i, const float4 &u) {
        const float f = s_f[i];
        v.x = fmaf(f, u.x, v.x);
        v.y = fmaf(f, u.y, v.y);
        v.z = fmaf(f, u.z, v.z);
        v.w = fmaf(f, u.w, v.w);
    };
    if (summing) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (part + j * kSplit < np) add(part + j * kSplit, ahead[j]);
#pragma unroll 8
        for (int i = part + kAhead * kSplit; i < np; i += kSplit)
            add(i, *reinterpret_cast<const float4 *>(a.ws_acc + at(i) * D + d));
    }
    s_v[tid] = v;
    __syncthreads();
    if (tid < Q) {
        l = 0.f;
#pragma unroll
        for (int w = 0; w < kW; ++w) l += s_l[w];
#pragma unroll
        for (int k = 1; k < kSplit; ++k) {
            const float4 u = s_v[k * Q + tid];
            v.x += u.x;
            v.y += u.y;
            v.z += u.z;
            v.w += u.w;
        }
        finish(c, d, v, m, l);
    }
    if (LONG) break;  // a CTA for every column
    }
}

// The accumulated weights, a second pass over K alone with the rows' sums (a
// weight needs the whole row's): a warp per unit, 8 columns at a time.  A position's
// sum over the columns is formed in one warp, in order; it is added to the mass
// atomically, for the pages that several sequences share.  (Where they do, the
// order of those additions, and so the last bit, may differ from run to run.)
// Keeping the first pass's scores instead would move fewer bytes up to 8 query heads
// per KV head (8 bytes a head and position, written and read, against K's D / 2 + D /
// 16 + 4 = 76 at D = 128), and would spare the products; it is not built.  With more
// columns the pass walks K once per 8 of them.
// Measured with the attention before it: 48 sequences of 1 to 6000 positions, 32 /
// 8 heads of 128 channels, 189 MB in 85 us, 33 of them this pass; 12 of 40 to 7001 with 16
// tokens (8 walks) 162 us, 83 more than without; a prompt of 2048 tokens (1024 walks)
// 2.2 ms, 1.8 of them this pass.
template <int G>
__global__ void __launch_bounds__(kThreads, G <= 4 ? 4 : 3) paged_mass_kernel(const PagedArgs a) {
    constexpr int D = 32 * G, U = units_per_step<G, 1>();
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ int64_t s_part[33], s_found[2];
    using S = Stage<G, false>;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    const PoolView &p = a.p;
    const Copier<G, false> copier(p, lane);
    const LaneOffsets<G> lo(lane);
    const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(smem) + warp * kStages * U * S::kBytes;
    const Score score(a);
    const bool shaped = score.capped || a.slopes;
    auto per_seq = [&](int b) -> int64_t {
        const Sequence s = sequence_of(a, b);
        return s.m == 0 || s.n == 0 ? 0 : (int64_t)p.H * tiles_of<U>(a, s).count;
    };
    Run run = find_run(per_seq, a.n_seq, blockIdx.x, gridDim.x, kMinPositions / kTile<U>, s_part, s_found);
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the rows' sums
    int b = run.b;
    while (run.cur < run.end) {
        const Sequence s = sequence_of(a, b);
        const Tiles tiles = tiles_of<U>(a, s);
        if (s.m == 0 || s.n == 0 || run.off >= (int64_t)p.H * tiles.count) {
            ++b;
            run.off = 0;
            continue;
        }
        const int h = (int)quotient(run.off, tiles.count);
        const int ta = (int)(run.off - (int64_t)h * tiles.count);
        const int tb = (int)min((int64_t)tiles.count, ta + (run.end - run.cur));
        const int32_t *pages = a.pages + (int64_t)b * a.max_pages;
        const int ncols = s.m * a.grp;
        for (int c0 = 0; c0 < ncols; c0 += 8) {
            const int cols = min(8, ncols - c0);
            const int pos_lo = s.n - s.m + c0 / a.grp, pos_hi = s.n - s.m + (c0 + cols - 1) / a.grp;
            const int vis_lo = a.window > 0 ? max(0, pos_lo - a.window + 1) : 0;
            const int t_end = min((tiles.first + tb - kItemCost<U>) * kTile<U>, min(s.n, pos_hi + 1));
            int t0 = (tiles.first + max(0, ta - kItemCost<U>)) * kTile<U> + warp * (U * kUnit);
            while (t0 + U * kUnit <= vis_lo) t0 += kTile<U>;
            UnitRing<G, false, U> ring{p, copier, pages, ring_at, h, t0, t_end, pos_lo, pos_hi, a.window, lane};
            __syncwarp();  // every lane has read the ring's last unit of the columns before
            ring.start();
            float ref[2], inv[2], slope[2];
            int pos[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                // a column past the last, or one that saw nothing: weight 0
                const int c = c0 + min(2 * t4 + e, cols - 1);
                const float2 v = a.ws_row[(int64_t)(s.row0 + c / a.grp) * a.Hq + h * a.grp + c % a.grp];
                ref[e] = 2 * t4 + e < cols ? v.x : INFINITY;
                inv[e] = 2 * t4 + e < cols ? v.y : 0.f;
                pos[e] = s.n - s.m + c / a.grp;
                slope[e] = a.slopes ? a.slopes[h * a.grp + c % a.grp] * kLog2e : 0.f;
            }
            uint4 qf[G];
            // (a query whose weights are 0 all the same reads as zeros: its products may be NaN)
            const int64_t at_q = (int64_t)(s.row0 + (c0 + g) / a.grp) * a.Hq + h * a.grp + (c0 + g) % a.grp;
            float back, mul[2], zero[G], qz[G][2];
            query_operands<G, true>(g < cols && a.ws_row[at_q].y != 0.f ? a.q + at_q * D : nullptr, t4, qf, back, zero);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                mul[e] = score.mul * __shfl_sync(0xffffffffu, back, 4 * (2 * t4 + e));
#pragma unroll
                for (int gr = 0; gr < G; ++gr) qz[gr][e] = __shfl_sync(0xffffffffu, zero[gr], 4 * (2 * t4 + e));
            }
            for (int i = 0; i < ring.steps; ++i) {
                const Shared here = ring.next(i);
                const bool marked = ring.marked();
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    const Shared at = here + j * S::kBytes;
                    const int t = t0 + i * kTile<U> + j * kUnit;
                    KUnit<G> ku;
                    ku.load(at + S::kc + lo.kc, at + S::ks + lo.ks, at + S::kz + lo.kz);
                    float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int gr = 0; gr < G; ++gr) {
                        uint32_t a0[4], a1[4];
                        ku.raw_operands(gr, a0, a1);
                        const float s0 = half_of(ku.s[0][gr / 2], gr & 1), s1 = half_of(ku.s[1][gr / 2], gr & 1);
                        const float z0 = half_of(ku.raw_zeros(0, gr), gr & 1), z1 = half_of(ku.raw_zeros(1, gr), gr & 1);
                        float d[4];
                        mma_first(d, a0, qf[gr].x, qf[gr].y);
                        mma(d, a1, qf[gr].z, qf[gr].w);
                        d[0] = fmaf(z0, qz[gr][0], d[0]);
                        d[1] = fmaf(z0, qz[gr][1], d[1]);
                        d[2] = fmaf(z1, qz[gr][0], d[2]);
                        d[3] = fmaf(z1, qz[gr][1], d[3]);
                        x[0] = fmaf(d[0], s0, x[0]);
                        x[1] = fmaf(d[1], s0, x[1]);
                        x[2] = fmaf(d[2], s1, x[2]);
                        x[3] = fmaf(d[3], s1, x[3]);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = x[e] * kRaw * mul[e & 1];
                    if (shaped) {
                        if (score.capped) score.cap_all(x);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int gap = pos[e & 1] - t - unit_position(g) - 4 * (e & 2);
                            x[e] = fmaf(-slope[e & 1], (float)gap, x[e]);
                        }
                    }
                    if (marked) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int gap = pos[e & 1] - t - unit_position(g) - 4 * (e & 2);
                            if (gap < 0 || (a.window > 0 && gap >= a.window)) x[e] = -INFINITY;
                        }
                    }
                    const uint32_t unit = ring.unit(i, j);
                    float w[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        w[r] = fmaf(ex2(x[2 * r] - ref[0]), inv[0], ex2(x[2 * r + 1] - ref[1]) * inv[1]);
                        w[r] += __shfl_xor_sync(0xffffffffu, w[r], 1);
                        w[r] += __shfl_xor_sync(0xffffffffu, w[r], 2);
                    }
                    // lanes t4 = 0 and 1 add the rows g and g + 8 (an entry past the
                    // sequence is left alone: its weight is 0, its mass may be anything)
                    const int u = unit_position(g) + 8 * t4;
                    if (t4 < 2 && t + u < s.n && unit != kNoUnit) {
                        atomicAdd(p.mass + (uint64_t)unit * kUnit + u, t4 ? w[1] : w[0]);
                    }
                }
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        run.cur += tb - ta;
        run.off += tb - ta;
    }
}

// ---- host ----

// n-tiles of 8 columns: as few as hold a KV head's queries, up to 4, and up to
// 128 accumulator registers a thread.
int n_tiles(int G, int64_t cols) {
    const int most = G <= 4 ? 4 : 2;
    return cols <= 8 ? 1 : (cols <= 16 || most == 2 ? 2 : 4);
}

size_t ceil16(size_t n) { return (n + 15) / 16 * 16; }

struct Workspace {
    size_t acc, ml, item, row, total;
    Workspace(int G, int C, int64_t n_rows, int Hq) {
        acc = 0;
        ml = acc + (size_t)2 * kMaxCtas * C * 32 * G * sizeof(float);
        item = ml + (size_t)2 * kMaxCtas * C * sizeof(float2);
        row = item + kMaxCtas * sizeof(int4);
        total = row + ceil16((size_t)n_rows * Hq * sizeof(float2));
    }
};

template <class... A>
cudaError_t launch(void (*kernel)(A...), dim3 grid, int threads, size_t smem, bool dependent, cudaStream_t s,
                   const PagedArgs &a) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = dependent ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int G, int NT, bool EXACT>
cudaError_t run_attention(const PagedArgs &a, const DeviceInfo &dev, bool mass, cudaStream_t s) {
    constexpr int C = 8 * NT;
    const size_t smem = ring_bytes<G, units_per_step<G, NT>()>() + (NT > 1 ? NT * G * 512 : 0);
    static std::atomic<uint64_t> ready{0};
    cudaError_t e = allow_smem((const void *)paged_attention_kernel<G, NT, EXACT>, (int)smem, dev, &ready);
    if (e != cudaSuccess) return e;
    // runs: one wave, and no more than the tables' width allows tiles for
    const int64_t cols = (int64_t)a.max_q * a.grp, n_ct = (cols + C - 1) / C;
    const int64_t positions = (int64_t)a.max_pages << a.p.lp, heads = (int64_t)a.n_seq * a.p.H;
    auto runs = [&](int64_t items, int per_sm, int U) {
        const int64_t most = (int64_t)dev.sm_count * per_sm < kMaxCtas ? (int64_t)dev.sm_count * per_sm : kMaxCtas;
        const int64_t each = cdiv((cdiv(positions, kUnit * kWarps * U) + 256 / (kUnit * kWarps * U)) * kUnit * kWarps * U, kMinPositions);
        if (items >= most || each >= most) return (unsigned)most;
        return (unsigned)(items * each < most ? items * each : most);
    };
    const unsigned grid = runs(heads * n_ct, min_ctas<G, NT>(), units_per_step<G, NT>());
    e = launch(paged_attention_kernel<G, NT, EXACT>, dim3(grid), kThreads, smem, false, s, a);
    if (e != cudaSuccess) return e;
    // the join's CTAs for a run's cut item: one a column where few items make many
    // runs (an item in four at least, on the average), else fewer (12 sequences of 16
    // tokens, 32 columns a tile: 78 us with 10 CTAs, 83 with 32)
    const int64_t item_cols = cols < C ? cols : C;
    if (heads * n_ct * 4 <= grid) {
        e = launch(paged_join_kernel<G, NT, EXACT, true>, dim3(grid, (unsigned)item_cols), kJoinThreads, 0, true, s, a);
    } else {
        const unsigned y = (unsigned)(item_cols < 2 * NT + 2 ? item_cols : 2 * NT + 2);
        e = launch(paged_join_kernel<G, NT, EXACT, false>, dim3(grid, y), kJoinThreads, 0, true, s, a);
    }
    if (e != cudaSuccess || !mass) return e;
    constexpr int mass_smem = kWarps * kStages * units_per_step<G, 1>() * Stage<G, false>::kBytes;
    static_assert(mass_smem <= 46 * 1024, "fits without asking for more");
    return launch(paged_mass_kernel<G>, dim3(runs(heads, G <= 4 ? 4 : 3, units_per_step<G, 1>())), kThreads, mass_smem, true, s,
                  a);
}

template <int G, bool EXACT>
cudaError_t run_attention_g(const PagedArgs &a, const DeviceInfo &dev, bool mass, cudaStream_t s) {
    switch (n_tiles(G, (int64_t)a.max_q * a.grp)) {
        case 1: return run_attention<G, 1, EXACT>(a, dev, mass, s);
        case 2: return run_attention<G, 2, EXACT>(a, dev, mass, s);
        default:
            if constexpr (G <= 4) return run_attention<G, 4, EXACT>(a, dev, mass, s);
            return cudaErrorInvalidValue;
    }
}

template <int G>
cudaError_t run_attention_g(const PagedArgs &a, const DeviceInfo &dev, bool exact, bool mass, cudaStream_t s) {
    return exact ? run_attention_g<G, true>(a, dev, mass, s) : run_attention_g<G, false>(a, dev, mass, s);
}

}  // namespace

size_t paged_workspace_bytes(int n_rows, int n_q_heads, int n_kv_heads, int head_dim) {
    const int G = head_dim / 32;
    return Workspace(G, 8 * n_tiles(G, (int64_t)n_rows * (n_q_heads / n_kv_heads)), n_rows, n_q_heads).total;
}

spectra_status launch_paged_attention(const spectra_kv_pool &pool, const spectra_paged_query &x, void *ws,
                                      cudaStream_t s, const DeviceInfo &dev) {
    PagedArgs a;
    a.p = PoolView::of(pool);
    a.pages = x.pages;
    a.lengths = x.lengths;
    a.q_start = x.q_start;
    a.q = x.q;
    a.slopes = x.slopes;
    a.out = x.out;
    a.max_pages = x.max_pages;
    a.n_seq = x.n_seq;
    a.n_rows = x.n_rows;
    a.max_q = x.max_q < x.n_rows ? x.max_q : x.n_rows;
    a.Hq = x.n_q_heads;
    a.grp = x.n_q_heads / pool.n_heads;
    a.window = x.window < (1 << 30) ? x.window : 1 << 30;  // positions number 2^30 at most
    a.scale = x.scale;
    a.cap = x.softcap;
    const Workspace w(a.p.G, 8 * n_tiles(a.p.G, (int64_t)a.max_q * a.grp), x.n_rows, x.n_q_heads);
    char *base = static_cast<char *>(ws);
    a.ws_acc = reinterpret_cast<float *>(base + w.acc);
    a.ws_ml = reinterpret_cast<float2 *>(base + w.ml);
    a.ws_item = reinterpret_cast<int4 *>(base + w.item);
    a.lse = x.lse;
    a.ws_row = x.update_mass ? reinterpret_cast<float2 *>(base + w.row) : nullptr;
    cudaError_t e = cudaErrorInvalidValue;
    const bool mass = x.update_mass != 0, exact = x.out_dtype == SPECTRA_F32;
    switch (a.p.G) {
        case 1: e = run_attention_g<1>(a, dev, exact, mass, s); break;
        case 2: e = run_attention_g<2>(a, dev, exact, mass, s); break;
        case 3: e = run_attention_g<3>(a, dev, exact, mass, s); break;
        case 4: e = run_attention_g<4>(a, dev, exact, mass, s); break;
        case 5: e = run_attention_g<5>(a, dev, exact, mass, s); break;
        case 6: e = run_attention_g<6>(a, dev, exact, mass, s); break;
        case 7: e = run_attention_g<7>(a, dev, exact, mass, s); break;
        case 8: e = run_attention_g<8>(a, dev, exact, mass, s); break;
    }
    return e == cudaSuccess ? SPECTRA_OK : SPECTRA_ERR_CUDA;
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
