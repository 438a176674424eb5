// sv_sample.cu -- drawing a token of each row after temperature, top-k, top-p and min-p,
// from a given random number (spec_verify_sample).
//
// A token is where a sum of weights passes u times their total, so with V tokens there are V
// borders, some 1e-5 apart or less, and which side of one a draw falls on must not depend on
// how the sum was formed.  Weights exp((z - m) / T) are therefore formed as pairs of 32-bit
// numbers (to 2^-33.6 of themselves; the 64-bit units of this GPU are too few), turned
// into whole numbers of 2^-44 (to 0.54 of one), and added as such: sums are exact and have no
// order.
//
// A cluster of CTAs has a row, each a slice of it in shared memory.  What is kept is always a
// run of the order (logit falling, id rising), so it is given by its last member: a cut
// (value, id).
//   small top-k, few tokens, or min-p alone  the k-th largest of the warps' few largest lane
//       maxima is a floor that at least k tokens reach; those that do (some 1.2 k) are listed by
//       one CTA, which cuts them by k, mass and min-p and draws.  In a list of up to 512 each
//       token adds up those before it, which needs no order; a longer one is sorted.
//   larger top-k  the cut is found by narrowing: a pass counts the tokens at and above seven
//       pivots of the interval that holds it, until the interval has few tokens (listed as
//       above) or one value (whose tokens are counted by id).
//   top-p  a histogram of rough masses over the distance from the largest, and one inside the
//       interval that it leaves, then one pass of exact masses, above the interval, in it and in
//       all, and a list of what is in it.  (If the interval was wrong, or has too many: narrowing
//       by exact masses.)
//   then a pass adds up what is kept, warp by warp in the order of ids, and the warp in whose
//       part the sum passes u times the total goes through it again.
// A pass is bound by the instructions of the weights, some 35 an element.  Nothing is done in
// 64-bit floating point: a warp's instruction of it takes 16 cycles, and a logarithm by all
// threads took 12 us.
#include <cooperative_groups.h>

#include <atomic>

#include "sv_internal.cuh"
#include "sv_paged.cuh"

namespace sv {
namespace {

namespace cg = cooperative_groups;

constexpr int kSThreads = 512, kSWarps = kSThreads / 32;
constexpr int kSCluster = 8;      // CTAs a row at most
// Tokens of a list: what one CTA sorts, and (kShort) what needs no order.  us for 4 rows of 32000 and a top-k of 50 / 100 /
// 200 / 400 / 1000 (lists of 1.2 k): 9.8 / 10.5 / 14.1 / 29.7 / 35.7; in an order from 257 tokens on 9.8 / 10.5 / 14.1 / 21.4 /
// 35.7, from 129 on 17.7 for 200, always 14.0 / 15.5 / 17.8 / 21.5 / 35.7: lists of 257 to 512 would be better off in order.
// A list of 1024 at most: 52.3 for 1000; rows of up to as many tokens are one list (2000 tokens, top-p: 39.6, where the
// histograms take 16.4).
constexpr int kList = 2048;
constexpr int kPer = kList / kSThreads;
constexpr int kPivots = 7;
constexpr int kFix = 44;          // weights are whole numbers of 2^-44: sums of 2^18 of them stay below 2^62
constexpr int kHalfFix = kFix / 2;
constexpr int kTops = 8;          // lanes of a warp that the floor may rank
constexpr int kShort = kSThreads;  // tokens of a list that needs no order

struct Cut {  // kept: x > v, and x == v up to id
    float v;
    int id;
};
struct Slot {  // what a CTA tells the others
    long long mass[kPivots + 1];
    int count[kPivots + 1];
    uint32_t bins[kSThreads];
    long long warp[kSWarps];
    alignas(16) int tops[kSWarps][kTops];  // of each warp its largest lane maxima (ord), falling
    int n, id;
    Cut cut;
};
constexpr int kTable = 1024;  // entries of 2^(i / 1024), in two parts
struct alignas(16) SampleTable {
    float v[2 * kTable];
};
constexpr SampleTable make_table() {
    SampleTable t{};
    for (int i = 0; i < kTable; ++i) {
        const double x = 0.69314718055994530942 * i / kTable;
        double y = 1.0, term = 1.0;
        for (int k = 1; k < 20; ++k) y += term = term * x / k;
        t.v[2 * i] = (float)y;
        t.v[2 * i + 1] = (float)(y - (double)t.v[2 * i]);
    }
    return t;
}
__device__ const SampleTable g_table = make_table();
constexpr int kBins = kSThreads, kCopies = 4;  // of a histogram, and copies of it
struct Pair16 {
    uint64_t key;
    unsigned long long mass;
};
struct SampleSmem {
    union {
        uint64_t list[kList];
        struct {
            uint64_t list_start[kShort];
            Pair16 pairs[kShort];
        };
        uint32_t bins[kBins][kCopies];
    };
    SampleTable tab;
    Slot slot[2];
    long long sum_mass[kPivots + 1];  // of the cluster
    int sum_count[kPivots + 1];
    long long wmass[kSWarps][kPivots + 1];
    int wcount[kSWarps][kPivots + 1];
    long long keep[kSWarps];  // of each warp the mass above the interval of top-p
    float wbin[kSWarps], edge;
    long long total, before;
    int n_list, place, edges[2];
};

// values in their order as whole numbers (both zeros are 0)
__device__ __forceinline__ int ord(float x) {
    const int b = __float_as_int(x);
    return b >= 0 ? b : -(b & 0x7FFFFFFF);
}
__device__ __forceinline__ float of_ord(int o) { return o >= 0 ? __int_as_float(o) : __int_as_float(-o | 0x80000000); }
// falling by value, then rising by id
__device__ __forceinline__ uint64_t list_key(float x, int id) {
    return (uint64_t)((uint32_t)ord(x) ^ 0x80000000u) << 32 | (0xFFFFFFFFu - (uint32_t)id);
}
__device__ __forceinline__ float key_value(uint64_t k) { return of_ord((int)((uint32_t)(k >> 32) ^ 0x80000000u)); }
__device__ __forceinline__ int key_id(uint64_t k) { return (int)(0xFFFFFFFFu - (uint32_t)k); }
__device__ __forceinline__ bool kept(Cut c, float x, int id) { return x > c.v || (x == c.v && id <= c.id); }

struct Weight {
    float m, c_hi, c_lo;  // the row's largest logit; log2(e) / T in two parts
    const float2* tab;
};
// Rounds to whole numbers by adding 1.5 * 2^23: they are then the sum's low bits, from this on.
constexpr float kMagic = 12582912.0f;
constexpr int kMagicBits = 0x4B400000;

// exp((x - m) / T) * 2^44 as hi * 2^22 + lo, each rounded by kMagic (returned with it)
__device__ __forceinline__ void weigh(const Weight& w, float x, int& hi, int& lo) {
    // x - m and its error
    const float d = __fsub_rn(x, w.m), bv = __fsub_rn(d, x), av = __fsub_rn(d, bv);
    const float e = __fadd_rn(__fsub_rn(x, av), -__fadd_rn(w.m, bv));
    // times log2(e) / T: p + q
    const float p = __fmul_rn(d, w.c_hi);
    float q = __fmaf_rn(d, w.c_hi, -p);
    q = __fmaf_rn(d, w.c_lo, q);
    q = __fmaf_rn(e, w.c_hi, q);
    if (!(p > -60.0f)) {  // below half of 2^-44
        hi = lo = kMagicBits;
        return;
    }
    // 2^p = 2^(j / 1024) 2^f: f in [-2^-11, 2^-11]
    const float js = __fadd_rn(p, 12288.0f);  // 1.5 * 2^13: steps of 1/1024
    const int j = __float_as_int(js) - 0x46400000;
    const float f = __fsub_rn(p, __fsub_rn(js, 12288.0f));
    // 2^(f + q) - 1 by its series to f^3 and f q: |f| <= 2^-11 and |q| < 2^-17, so what is left out is below 2^-40
    // where a weight is above 2^-16.  (Without f q weights were off by up to 2^-31: q is half a step of p at most.)
    // Five roundings of 2^-36 remain: f's factor twice, f's product, g and, of a table's entry, k.
    constexpr float kLn2 = 0.69314718f, kLn2Sq = 0.24022651f, kLn2Cb = 0.05550411f;  // ln 2, its square / 2, cube / 6
    float g = __fmaf_rn(f, kLn2Cb, kLn2Sq);
    g = __fmaf_rn(f, g, kLn2);
    g = __fmaf_rn(q, __fmaf_rn(f, 2.0f * kLn2Sq, kLn2), __fmul_rn(f, g));
    const float2 b = w.tab[j & (kTable - 1)];
    const float k = __fmaf_rn(b.x, g, b.y);
    const float h = __fadd_rn(b.x, k), l = __fsub_rn(k, __fsub_rn(h, b.x));
    const float scale = __int_as_float(((j >> 10) + kHalfFix + 127) << 23);
    // the whole number nearest to the upper part, then what is missing, 2^22 times as large
    const float u = __fmul_rn(h, scale), r = __fadd_rn(u, kMagic);
    hi = __float_as_int(r);
    const float rest = __fmaf_rn(l, scale, __fsub_rn(u, __fsub_rn(r, kMagic)));
    lo = __float_as_int(__fmaf_rn(rest, (float)(1 << kHalfFix), kMagic));
}
__device__ __forceinline__ long long fixed(int hi, int lo) {
    return ((long long)(hi - kMagicBits) << kHalfFix) + (lo - kMagicBits);
}
__device__ __forceinline__ long long weight(const Weight& w, float x) {
    int hi, lo;
    weigh(w, x, hi, lo);
    return fixed(hi, lo);
}

// floor(x * 2^bits) of a number in [0, 1], and the same rounded up
__device__ __forceinline__ unsigned long long scaled(float x, int bits, bool up = false) {
    const int b = __float_as_int(x), e = max(b >> 23, 1) - 150 + bits;
    const unsigned long long f = (b & 0x7FFFFF) | (b >> 23 ? 0x800000 : 0);
    if (e >= 0) return f << e;
    return e <= -25 ? (up && f ? 1 : 0) : (f + (up ? (1ull << -e) - 1 : 0)) >> -e;
}
// a / b rounded to nearest (to within 2^-40 of a step's half)
__device__ __forceinline__ float ratio(long long a, long long b) {
    const float ah = __ll2float_rn(a), bh = __ll2float_rn(b);
    const float al = __ll2float_rn(a - (long long)ah), bl = __ll2float_rn(b - (long long)bh);
    const float q = __fdiv_rn(ah, bh);
    const float r = __fmaf_rn(-q, bl, __fadd_rn(__fmaf_rn(-q, bh, ah), al));
    return __fadd_rn(q, __fdiv_rn(r, bh));
}

template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(uint4 r, float (&x)[4]) {
        x[0] = __uint_as_float(r.x), x[1] = __uint_as_float(r.y), x[2] = __uint_as_float(r.z), x[3] = __uint_as_float(r.w);
    }
    static constexpr uint32_t kLowest = 0xFF800000u;  // -inf (all of a word)
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(uint4 r, float (&x)[8]) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
    static constexpr uint32_t kLowest = 0xFF80FF80u;
};

__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

template <typename T>
struct SampleRow {
    static constexpr int VEC = Vec<T>::N;
    const sv_sample_args& a;
    SampleSmem& s;
    const uint4* slice;
    cg::cluster_group cl;
    int C, rank, t, lane, warp;
    int v0, v1, id0;  // the warp's vectors; the id of the slice's first element
    int turn;         // exchanges so far
    Weight w;

    __device__ Slot& mine() { return s.slot[turn & 1]; }
    // what every CTA wrote to mine() is there for all; slots are used in turn, so that nobody writes
    // to one that another still reads
    __device__ void exchange() {
        if (C > 1)
            cl.sync();
        else
            __syncthreads();
        ++turn;
    }
    __device__ const Slot* of(int r) {
        Slot* p = &s.slot[(turn - 1) & 1];
        return C > 1 ? cl.map_shared_rank(p, r) : p;
    }
    template <typename F>
    __device__ void each(F f) {
        for (int v = v0 + lane; v < v1; v += 32) {
            float x[VEC];
            Vec<T>::unpack(slice[v], x);
#pragma unroll
            for (int k = 0; k < VEC; ++k) f(x[k], id0 + v * VEC + k);
        }
    }

    // Sorts the n entries of the list (falling); entries up to the next power of two are 0.
    __device__ int sort(int n) {
        int n2 = 32;
        while (n2 < n) n2 <<= 1;
        for (int i = n + t; i < n2; i += kSThreads) s.list[i] = 0;
        __syncthreads();
        for (int k = 2; k <= n2; k <<= 1)
            for (int j = k >> 1; j > 0; j >>= 1) {
                for (int i = t; i < n2 / 2; i += kSThreads) {
                    const int x = ((i & ~(j - 1)) << 1) | (i & (j - 1)), y = x | j;
                    const uint64_t p = s.list[x], q = s.list[y];
                    if ((p < q) == ((x & k) == 0)) s.list[x] = q, s.list[y] = p;
                }
                __syncthreads();
            }
        return n2;
    }
    // before[i]: the sum of val over the entries before entry kPer * t + i; returns the sum of all
    __device__ long long scan(const long long (&val)[kPer], long long (&before)[kPer]) {
        long long own = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) own += val[i];
        long long x = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if (lane >= o) x += y;
        }
        __syncthreads();
        if (lane == 31) s.wmass[warp][0] = x;
        __syncthreads();
        long long base = x - own, total = 0;
        for (int i = 0; i < kSWarps; ++i) {
            const long long y = s.wmass[i][0];
            if (i < warp) base += y;
            total += y;
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            before[i] = base;
            base += val[i];
        }
        return total;
    }
    __device__ int count_of(int own) {  // over the CTA
        own = __reduce_add_sync(0xFFFFFFFFu, own);
        __syncthreads();
        if (lane == 0) s.wcount[warp][0] = own;
        __syncthreads();
        int n = 0;
        for (int i = 0; i < kSWarps; ++i) n += s.wcount[i][0];
        return n;
    }

    // The tokens that f takes, of all CTAs, in the list of the cluster's first (unsorted); how many, to all.
    // Above kList there is no list.
    template <typename F>
    __device__ int gather(F f) {
        if (t == 0) s.n_list = 0;
        __syncthreads();
        each([&](float x, int id) {
            if (f(x, id)) {
                const int at = atomicAdd(&s.n_list, 1);
                if (at < kList) s.list[at] = list_key(x, id);
            }
        });
        __syncthreads();
        if (t == 0) mine().n = s.n_list;
        exchange();
        int n = 0, at = 0;
#pragma unroll
        for (int r = 0; r < kSCluster; ++r) {  // (unrolled, so that the others' memory is waited for once)
            const int c = r < C ? of(r)->n : 0;
            if (r < rank) at += c;
            n += c;
        }
        if (C > 1) {
            if (n <= kList && rank > 0) {
                uint64_t* dst = cl.map_shared_rank(s.list, 0) + at;
                for (int i = t; i < s.n_list; i += kSThreads) dst[i] = s.list[i];
            }
            cl.sync();
        } else {
            __syncthreads();
        }
        return n;
    }

    // ceil(P S) for the comparison of whole numbers with it (at least 1: the likeliest is kept), floor(u S)
    static __device__ long long mass_target(float P, long long S) {
        const unsigned long long p = scaled(P, 64);
        return max((long long)(__umul64hi(p, (unsigned long long)S) + (p * (unsigned long long)S != 0)), 1ll);
    }
    static __device__ long long share_of(float u, long long S) {
        return (long long)__umul64hi(scaled(u, 64), (unsigned long long)S);
    }
    __device__ long long sum_of(long long own) {  // over the CTA
        own = warp_sum(own);
        __syncthreads();
        if (lane == 0) s.wmass[warp][0] = own;
        __syncthreads();
        long long n = 0;
#pragma unroll
        for (int i = 0; i < kSWarps; ++i) n += s.wmass[i][0];
        return n;
    }

    // A short list (n <= kShort), token by token: G neighbouring threads have entry e.  Of the
    // entries with a greater key their number (low 10 bits) and mass (above).
    struct Entry {
        int e, G;
        bool first;  // of the G threads
        uint64_t key;
        long long w;
    };
    __device__ Entry entry(int n) {
        int size = 16;
        while (size < n) size <<= 1;
        Entry x;
        x.G = kSThreads / size;
        x.e = t / x.G;
        x.first = t % x.G == 0;
        x.key = 0;
        x.w = 0;
        return x;
    }
    __device__ Entry listed(int n) {
        Entry x = entry(n);
        if (x.e < n) {
            x.key = s.list[x.e];
            x.w = weight(w, key_value(x.key));
            if (x.first) s.pairs[x.e] = Pair16{x.key, (unsigned long long)x.w << 10 | 1};
        }
        __syncthreads();
        return x;
    }
    __device__ unsigned long long above(const Entry& x, int n) {
        unsigned long long sum = 0;
        if (x.e < n)
#pragma unroll 4
            for (int f = t % x.G; f < n; f += x.G) {
                const Pair16 p = s.pairs[f];
                if (p.key > x.key) sum += p.mass;
            }
        for (int o = 1; o < x.G; o <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        return sum;
    }

    // Draws from the list's n entries: top-k, top-p and min-p (a weight of `least`), then by id.  By one CTA.
    __device__ void draw_from_list(int n, int K, float P, long long least, float u, int32_t* token, float* prob) {
        if (n <= kShort) {
            const Entry x = listed(n);
            const unsigned long long a = above(x, n);
            const int place = (int)(a & 1023);
            const bool in = x.e < n && place < K;
            const long long S = sum_of(in && x.first ? x.w : 0);
            const long long target = P < 1.0f ? mass_target(P, S) : 0x7FFFFFFFFFFFFFFFll;
            // what is kept comes first in the order (by number: weights of neighbouring logits may be off by more than
            // their distance)
            const int kept_n = count_of(in && x.first && (long long)(a >> 10) < target && x.w >= least);
            // again, by ids (the low half of a key falls with them)
            if (x.e < n && x.first && place < kept_n) s.pairs[place] = Pair16{x.key & 0xFFFFFFFFu, (unsigned long long)x.w};
            __syncthreads();
            Entry y = entry(kept_n);
            if (y.e < kept_n) {
                y.key = s.pairs[y.e].key;
                y.w = (long long)s.pairs[y.e].mass;
            }
            const long long kept_mass = sum_of(y.first ? y.w : 0);
            const long long before = (long long)above(y, kept_n), v = share_of(u, kept_mass);
            if (y.e < kept_n && y.first && before <= v && before + y.w > v) {
                *token = key_id(y.key);
                if (prob) *prob = ratio(y.w, kept_mass);
            }
            return;
        }
        sort(n);
        if (K < n) n = K;
        long long val[kPer], before[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = t * kPer + i;
            val[i] = e < n ? weight(w, key_value(s.list[e])) : 0;
        }
        const long long S = scan(val, before);
        const long long target = P < 1.0f ? mass_target(P, S) : 0x7FFFFFFFFFFFFFFFll;
        int keep = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = t * kPer + i;
            keep += e < n && before[i] < target && val[i] >= least;
        }
        n = count_of(keep);
        // in the order of ids
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = t * kPer + i;
            if (e < n) {
                const uint64_t k = s.list[e];
                s.list[e] = ~((uint64_t)(uint32_t)key_id(k) << 32 | (uint32_t)(k >> 32));
            }
        }
        __syncthreads();
        sort(n);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = t * kPer + i;
            val[i] = e < n ? weight(w, key_value(~s.list[e] << 32)) : 0;
        }
        const long long kept_mass = scan(val, before);
        const long long v = share_of(u, kept_mass);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (before[i] <= v && before[i] + val[i] > v) {
                *token = (int)(~s.list[t * kPer + i] >> 32);
                if (prob) *prob = ratio(val[i], kept_mass);
            }
    }

    // The cut behind the first `number` of the list's n entries in their order, or (number 0) behind those that
    // have less than `target` mass before them, `done` of it not in the list; to all.
    __device__ Cut cut_in_list(int n, int number, long long done, long long target) {
        if (rank == 0) {
            if (n <= kShort) {
                const Entry x = listed(n);
                const unsigned long long a = above(x, n);
                if (number == 0)
                    number = count_of(x.e < n && x.first && done + (long long)(a >> 10) < target);
                if (x.e < n && x.first && (int)(a & 1023) == max(number, 1) - 1)
                    mine().cut = Cut{key_value(x.key), key_id(x.key)};
            } else {
                sort(n);
                if (number == 0) {
                    long long val[kPer], before[kPer];
#pragma unroll
                    for (int i = 0; i < kPer; ++i) {
                        const int e = t * kPer + i;
                        val[i] = e < n ? weight(w, key_value(s.list[e])) : 0;
                    }
                    scan(val, before);
#pragma unroll
                    for (int i = 0; i < kPer; ++i) number += t * kPer + i < n && done + before[i] < target;
                    number = count_of(number);
                }
                if (t == 0) {
                    const uint64_t k = s.list[max(number, 1) - 1];
                    mine().cut = Cut{key_value(k), key_id(k)};
                }
            }
        }
        exchange();
        return of(0)->cut;
    }

    // One pass of narrowing: of the members of `cut` in [lo, hi), mass and number at and above each
    // pivot; entry kPivots: of all of them.  Summed over the cluster.
    template <bool MASS, int USED = kPivots>
    __device__ void pass(Cut cut, float lo, float hi, const float (&p)[kPivots], long long (&mass)[kPivots + 1],
                         int (&count)[kPivots + 1]) {
        int h[kPivots + 1], l[kPivots + 1], n[kPivots + 1];
#pragma unroll
        for (int j = 0; j <= kPivots; ++j) h[j] = l[j] = n[j] = 0;
        each([&](float x, int id) {
            if (x >= lo && x < hi && kept(cut, x, id)) {
                int wh = 0, wl = 0;
                if (MASS) weigh(w, x, wh, wl);
                wh -= kMagicBits, wl -= kMagicBits;
#pragma unroll
                for (int j = 0; j <= kPivots; ++j)
                    if (j == kPivots || (j < USED && x >= p[j])) {
                        if (MASS) h[j] += wh, l[j] += wl;
                        ++n[j];
                    }
            }
        });
#pragma unroll
        for (int j = 0; j <= kPivots; ++j) {
            if (j >= USED && j < kPivots) continue;
            const int c = __reduce_add_sync(0xFFFFFFFFu, n[j]);
            if (lane == 0) s.wcount[warp][j] = c;
            if (MASS) {
                const long long m = warp_sum(((long long)(uint32_t)h[j] << kHalfFix) + l[j]);
                if (lane == 0) s.wmass[warp][j] = m;
            }
        }
        __syncthreads();
        if (t <= kPivots) {
            long long m = 0;
            int c = 0;
            for (int i = 0; i < kSWarps; ++i) {
                c += s.wcount[i][t];
                if (MASS) m += s.wmass[i][t];
            }
            mine().count[t] = c;
            mine().mass[t] = m;
        }
        exchange();
        if (t <= kPivots) {
            int c[kSCluster];
            long long m[kSCluster];
#pragma unroll
            for (int r = 0; r < kSCluster; ++r) {
                c[r] = r < C ? of(r)->count[t] : 0;
                m[r] = MASS && r < C ? of(r)->mass[t] : 0;
            }
#pragma unroll
            for (int r = 1; r < kSCluster; ++r) c[0] += c[r], m[0] += m[r];
            s.sum_count[t] = c[0], s.sum_mass[t] = m[0];
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j <= kPivots; ++j) mass[j] = s.sum_mass[j], count[j] = s.sum_count[j];
    }

    // The warp in whose part the running sum of f over ids first passes `over` (or share * the total of
    // all, where over < 0): its place in the cluster, the sum before it and the total, in s; nobody: -1.
    // ready: of each warp's sum a part that is known.
    template <typename F>
    __device__ void locate(F f, long long over, float share, long long ready = 0) {
        long long own = 0;
        each([&](float x, int id) { own += f(x, id); });
        own = warp_sum(own) + ready;
        if (lane == 0) mine().warp[warp] = own;
        exchange();
        if (warp == 0) {
            constexpr int PER = kSCluster * kSWarps / 32;
            long long part[PER], sum = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int at = lane * PER + i;
                part[i] = at < C * kSWarps ? of(at / kSWarps)->warp[at % kSWarps] : 0;
                sum += part[i];
            }
            long long x = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xFFFFFFFFu, x, o);
                if (lane >= o) x += y;
            }
            const long long total = __shfl_sync(0xFFFFFFFFu, x, 31);
            const long long v = over >= 0 ? over : share_of(share, total);
            if (lane == 0) s.place = -1, s.total = total;
            __syncwarp();
            long long before = x - sum;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                if (before <= v && before + part[i] > v) s.place = lane * PER + i, s.before = before - v;
                before += part[i];
            }
        }
        __syncthreads();
    }
    // by that warp: the first element at which the running sum passes; found(x, id) by one lane
    template <typename F, typename G>
    __device__ void search(F f, G found) {
        if (s.place != rank * kSWarps + warp) return;
        long long run = s.before;  // less what is to be passed: the first sum above 0
        for (int v = v0; v < v1; v += 32) {
            float x[VEC];
            long long own = 0;
            const bool in = v + lane < v1;
            if (in) {
                Vec<T>::unpack(slice[v + lane], x);
#pragma unroll
                for (int k = 0; k < VEC; ++k) own += f(x[k], id0 + (v + lane) * VEC + k);
            }
            long long upto = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
                if (lane >= o) upto += y;
            }
            const unsigned past = __ballot_sync(0xFFFFFFFFu, run + upto > 0);
            if (past) {
                if (lane == __ffs(past) - 1) {
                    long long at = run + upto - own;
#pragma unroll
                    for (int k = 0; k < VEC; ++k) {
                        const int id = id0 + (v + lane) * VEC + k;
                        const long long y = f(x[k], id);
                        if (at <= 0 && at + y > 0) found(x[k], id);
                        at += y;
                    }
                }
                return;
            }
            run += __shfl_sync(0xFFFFFFFFu, upto, 31);
        }
    }

    __device__ float first_pivot(int j, float temp) {  // by distance from the largest
        constexpr float kFirst[kPivots] = {16.0f, 12.0f, 9.0f, 7.0f, 5.0f, 3.0f, 1.5f};
        return w.m - kFirst[j] * temp;
    }
    // The cut of the K largest members (MASS false), or of the shortest run with P of the members' mass.
    template <bool MASS>
    __device__ Cut narrow(Cut cut, int K, float P, float temp) {
        // kept: all members from hi on, with mass (number) `above`, which is not enough; lo is
        float lo = -3.402823466e38f, hi = of_ord(ord(w.m) + 1);
        long long above = 0, target = K;
        for (int round = 0;; ++round) {
            float p[kPivots];
#pragma unroll
            for (int j = 0; j < kPivots; ++j) {
                const float x = (float)(j + 1) / (kPivots + 1);
                // by distance from the largest; then by value and by the order of floats in turn: one converges
                // quickly on smooth rows, the other in 11 passes on any
                p[j] = round == 0 ? first_pivot(j, temp)
                       : round & 1 ? lo * (1.0f - x) + hi * x
                                   : of_ord((int)(ord(lo) + ((long long)ord(hi) - ord(lo)) * (j + 1) / (kPivots + 1)));
                p[j] = fminf(fmaxf(p[j], lo), hi);
            }
            long long mass[kPivots + 1];
            int count[kPivots + 1];
            pass<MASS>(cut, lo, hi, p, mass, count);
            if (round == 0) {
                if (MASS)
                    target = mass_target(P, mass[kPivots]);
                else if (count[kPivots] <= K)  // (masked tokens are not members)
                    return cut;
            }
            int in = count[kPivots];
            long long more = 0;
#pragma unroll
            for (int j = kPivots - 1, go = 1; j >= 0; --j) {
                if (!go) continue;
                const long long sum = MASS ? mass[j] : count[j];
                if (above + sum < target) {
                    hi = p[j];
                    more = sum;
                    in = count[kPivots] - count[j];
                } else {
                    lo = p[j];
                    in = count[j] - (count[kPivots] - in);
                    go = 0;
                }
            }
            above += more;
            if (in <= kList || ord(hi) - ord(lo) == 1) {
                Cut res;
                if (in <= kList) {
                    const int n = gather([&](float x, int id) { return x >= lo && x < hi && kept(cut, x, id); });
                    res = cut_in_list(n, MASS ? 0 : (int)(target - above), above, target);
                } else {
                    // one value: its first `keep` by id
                    const long long each_one = MASS ? weight(w, lo) : 1;
                    const long long keep = (target - above + each_one - 1) / max(each_one, 1ll);
                    auto one = [&](float x, int id) -> long long { return x == lo && kept(cut, x, id); };
                    locate(one, keep - 1, 0.0f);
                    const int at = s.place;
                    search(one, [&](float, int id) { mine().id = id; });
                    exchange();
                    res = Cut{lo, at < 0 ? 0x7FFFFFFF : of(at / kSWarps)->id};
                }
                return res;
            }
        }
    }

    // A histogram of rough masses of the members, over p = log2 of their weights: bin i has those with
    // from - (i + 1) * width < p <= from - i * width, the last all below as well (`open`); those above
    // `from` are in none.  Masses count in 2^-13 of the bin's upper end (rounded to 2^-14 of it: 2^18 of them fit).
    // Bin t's mass comes back to thread t, the same in all CTAs.
    __device__ float histogram(Cut cut, float from, float width, bool open) {
        for (int i = t; i < kBins * kCopies; i += kSThreads) (&s.bins[0][0])[i] = 0;
        __syncthreads();
        const float per = 1.0f / width;
        each([&](float x, int id) {
            const float p = (x - w.m) * w.c_hi;
            float i = (from - p) * per;
            if (i >= 0.0f && (open || i < (float)kBins) && kept(cut, x, id)) {
                i = floorf(fminf(i, kBins - 1.0f));
                float y;
                asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(p - (from - i * width)));
                atomicAdd(&s.bins[(int)i][lane & (kCopies - 1)], (uint32_t)__float2int_rn(y * 8192.0f));
            }
        });
        __syncthreads();
        const uint4 four = *reinterpret_cast<const uint4*>(s.bins[t]);
        mine().bins[t] = four.x + four.y + four.z + four.w;
        exchange();
        float sum = 0.0f;
#pragma unroll
        for (int r = 0; r < kSCluster; ++r) sum += r < C ? (float)of(r)->bins[t] : 0.0f;
        float y;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(from - t * width));
        return sum * y * (1.0f / 8192.0f);
    }
    // The first bin (of thread t: `mass`) up to which P of all is reached perhaps, and that up to which it is for
    // certain (kBins: none); the mass before the former, and of all bins.  `before`: what lies before them;
    // all: the whole mass (0: that of the bins).
    __device__ void crossing(float mass, float before, float P, float all, int& first, int& last, float& lead, float& total) {
        float x = mass;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float y = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if (lane >= o) x += y;
        }
        __syncthreads();
        if (lane == 31) s.wbin[warp] = x;
        if (t < 2) s.edges[t] = kBins;
        if (t == 0) s.edge = 0.0f;
        __syncthreads();
        float base = before;
        total = 0.0f;
        for (int i = 0; i < kSWarps; ++i) {
            if (i < warp) base += s.wbin[i];
            total += s.wbin[i];
        }
        const float S = all > 0.0f ? all : total, need = P * S, room = S * (1.0f / 8192);
        const float upto = base + x;
        if (upto >= need - room) atomicMin(&s.edges[0], t);
        if (upto > need + room) atomicMin(&s.edges[1], t);
        __syncthreads();
        first = s.edges[0], last = s.edges[1];
        if (t == first) s.edge = upto - mass;
        __syncthreads();
        lead = s.edge;
    }

    // The cut of the shortest run with P of the members' mass.  inner: where the interval ends, above which all
    // is kept (its mass by warps is in s.keep); infinite: they are not known.
    __device__ Cut nucleus(Cut cut, float P, float temp, float& inner) {
        // the interval as p = log2 of weights, from `top` down to `bottom`
        int first, last;
        float lead, all, rest;
        constexpr float kWidth = 1.0f / 16;
        crossing(histogram(cut, 0.0f, kWidth, true), 0.0f, P, 0.0f, first, last, lead, all);
        float top = -kWidth * first, bottom = last >= kBins - 1 ? -INFINITY : -kWidth * (last + 1);
        if (first < kBins && last < kBins - 1) {
            const float width = (top - bottom) / kBins;
            crossing(histogram(cut, top, width, false), lead, P, all, first, last, lead, rest);
            if (last < kBins) bottom = top - width * (last + 1);
            if (first < kBins) top = top - width * first;
        }
        // as values, a little wider
        const float slack = 1e-6f * fabsf(w.m);
        const float hi = top == 0.0f ? of_ord(ord(w.m) + 1) : w.m + top / w.c_hi * (1.0f - 1e-6f) + slack;
        const float lo = bottom == -INFINITY ? -3.402823466e38f : w.m + bottom / w.c_hi * (1.0f + 1e-6f) - slack;
        const float p[kPivots] = {lo, hi, hi, hi, hi, hi, hi};
        long long mass[kPivots + 1];
        int count[kPivots + 1];
        pass<true, 2>(cut, -3.402823466e38f, INFINITY, p, mass, count);
        const long long target = mass_target(P, mass[kPivots]);
        inner = INFINITY;
        if (mass[1] >= target || mass[0] < target || count[0] - count[1] > kList) return narrow<true>(cut, 0, P, temp);
        if (lane == 0) s.keep[warp] = s.wmass[warp][1];
        inner = hi;
        const int n = gather([&](float x, int id) { return x >= lo && x < hi && kept(cut, x, id); });
        return cut_in_list(n, 0, mass[1], target);
    }
};

template <typename T>
__global__ void __launch_bounds__(kSThreads, 2)
    sample_kernel(const __grid_constant__ sv_sample_args a, int C, int slice_elems) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    SampleSmem& s = *reinterpret_cast<SampleSmem*>(smem_raw);
    uint4* slice = reinterpret_cast<uint4*>(smem_raw + align_up(sizeof(SampleSmem), 16));
    constexpr int VEC = Vec<T>::N;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int64_t row = blockIdx.x / C;
    const int rank = (int)(blockIdx.x % C), b = (int)(row / a.N), i = (int)(row % a.N), V = (int)a.V;
    // the row's settings (the same answer in every CTA of the cluster)
    const float Tm = a.temperature ? a.temperature[b] : 1.0f;
    int K = a.top_k ? a.top_k[b] : 0;
    const float P = a.top_p ? a.top_p[b] : 1.0f, M = a.min_p ? a.min_p[b] : 0.0f;
    const float u = a.uniforms[(int64_t)b * a.uniform_stride + i];
    uint32_t bad = 0;
    if (!(Tm >= 0.0f) || isinf(Tm)) bad |= SV_ROW_BAD_TEMPERATURE;
    if (K < 0) bad |= SV_ROW_BAD_TOP_K;
    if (!(P > 0.0f) || P > 1.0f) bad |= SV_ROW_BAD_TOP_P;
    if (!(M >= 0.0f) || M > 1.0f) bad |= SV_ROW_BAD_MIN_P;
    if (!(u >= 0.0f) || u >= 1.0f) bad |= SV_ROW_BAD_UNIFORM;
    int32_t* token = a.tokens + row;
    float* prob = a.probs ? a.probs + row : nullptr;
    auto refuse = [&](uint32_t why) {
        if (rank == 0 && t == 0) {
            *token = -1;
            if (prob) *prob = NAN;
            if (a.row_status) atomicOr(a.row_status + b, why);
        }
    };
    if (bad) {
        refuse(bad);
        return;
    }
    if (K == 0 || K > V) K = V;

    // ---- the CTA's slice to shared memory, its vectors where they lie in the row
    const int first = min(rank * slice_elems, V), n = min(slice_elems, V - first);
    const T* src = (const T*)a.logits + (int64_t)b * a.stride_b + (int64_t)i * a.stride_n + first;
    const int pad = (int)((uintptr_t)src / sizeof(T) % VEC);  // elements of the first vector before the slice
    const uint4* vec = reinterpret_cast<const uint4*>(src - pad);
    const int nv = n > 0 ? (pad + n + VEC - 1) / VEC : 0;
    const int v0 = (int)((int64_t)nv * warp / kSWarps), v1 = (int)((int64_t)nv * (warp + 1) / kSWarps);
    float top = -INFINITY;
    for (int v = v0 + lane; v < v1; v += 128) {
        uint4 r[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int x = v + 32 * k;
            if (x >= v1) continue;
            if (x * VEC >= pad && (x + 1) * VEC <= pad + n) {
                r[k] = ld_stream16(vec + x);
            } else {  // the row's ends: what is not of it is -inf
                uint32_t q[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    q[y] = Vec<T>::kLowest;
#pragma unroll
                    for (int z = 0; z < VEC / 4; ++z) {
                        const int e = x * VEC + y * (VEC / 4) + z - pad;
                        if (e < 0 || e >= n) continue;
                        if constexpr (VEC == 8) {
                            const uint32_t w = reinterpret_cast<const unsigned short*>(src)[e];
                            q[y] = z ? (q[y] & 0xFFFFu) | w << 16 : (q[y] & 0xFFFF0000u) | w;
                        } else {
                            q[y] = reinterpret_cast<const uint32_t*>(src)[e];
                        }
                    }
                }
                r[k] = make_uint4(q[0], q[1], q[2], q[3]);
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (v + 32 * k >= v1) continue;
            slice[v + 32 * k] = r[k];
            float x[VEC];
            Vec<T>::unpack(r[k], x);
#pragma unroll
            for (int y = 0; y < VEC; ++y) top = max_nan(top, x[y]);
        }
    }
    for (int k = t; k < kTable / 2; k += kSThreads)
        reinterpret_cast<float4*>(s.tab.v)[k] = __ldg(reinterpret_cast<const float4*>(g_table.v) + k);
    SampleRow<T> r{a, s, slice, cg::this_cluster(), C, rank, t, lane, warp, v0, v1, first - pad, 0, {}};

    // ---- the largest of the row and, of each warp, its largest lane maxima: one more than would do
    const int warps = C * kSWarps, j = min((K + warps - 1) / warps + 1, kTops);
    const bool ranked = K < V && warps * j >= K;
    const bool poison = __any_sync(0xFFFFFFFFu, !(top < INFINITY));
    int o = ord(top);
    for (int k = 0; k < (ranked ? j : 1); ++k) {
        const int most = __reduce_max_sync(0xFFFFFFFFu, o);
        const unsigned who = __ballot_sync(0xFFFFFFFFu, o == most);
        if (lane == __ffs(who) - 1) o = ord(-INFINITY);
        if (lane == 0) r.mine().tops[warp][k] = most;
    }
    if (poison && lane == 0) r.mine().tops[warp][0] = 0x7FFFFFFF;  // (no float's)
    r.exchange();
    constexpr int PER = kSCluster * kSWarps * kTops / kSThreads;
    int v[PER], most = ord(-INFINITY);
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        // the largest of every warp, then their second largest, ... (C is a power of two)
        const int at = t + k * kSThreads, y = at & (warps - 1), of = at / kSWarps >> (__ffs(C) - 1);
        v[k] = of < (ranked ? j : 1) ? r.of(y / kSWarps)->tops[y % kSWarps][of] : (int)0x80000000;
    }
#pragma unroll
    for (int k = 0; k < PER; ++k) most = max(most, v[k]);
    most = __reduce_max_sync(0xFFFFFFFFu, most);
    if (lane == 0) s.wcount[warp][0] = most;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kSWarps; ++k) most = max(most, s.wcount[k][0]);
    const bool any = most == 0x7FFFFFFF;
    const float m = of_ord(most);
    uint32_t floor_bits = 0;  // the K-th largest of the warps' maxima, to 16 bits
    if (ranked)
        for (int bit = 31; bit >= 16; --bit) {
            const uint32_t x = floor_bits | 1u << bit;
            int n = 0;
#pragma unroll
            for (int k = 0; k < PER; ++k)
                if (k * kSThreads < warps * j) n += __syncthreads_count(((uint32_t)v[k] ^ 0x80000000u) >= x);
            if (n >= K) floor_bits = x;
        }
    if (any || m == -INFINITY) {
        refuse(SV_ROW_NONFINITE);
    } else if (Tm == 0.0f) {
        // ---- greedy: the first of the largest
        int least = 0x7FFFFFFF;
        r.each([&](float x, int id) {
            if (x == m) least = min(least, id);
        });
        least = __reduce_min_sync(0xFFFFFFFFu, least);
        if (lane == 0) s.wcount[warp][3] = least;
        __syncthreads();
        if (t == 0) {
            for (int k = 0; k < kSWarps; ++k) least = min(least, s.wcount[k][3]);
            r.mine().id = least;
        }
        r.exchange();
        if (rank == 0 && t == 0) {
            for (int k = 0; k < C; ++k) least = min(least, r.of(k)->id);
            *token = least;
            if (prob) *prob = 1.0f;
        }
    } else {
        constexpr float kLog2e = (float)1.4426950408889634074, kLog2eLo = (float)(1.4426950408889634074 - (double)kLog2e);
        const float temp = fmaxf(Tm, 1e-30f), c = __fdiv_rn(kLog2e, temp);
        r.w = Weight{m, c, __fdiv_rn(__fadd_rn(__fmaf_rn(-c, temp, kLog2e), kLog2eLo), temp), reinterpret_cast<const float2*>(s.tab.v)};
        // min-p: the least weight, and a value below which no weight is as large
        long long least = (long long)scaled(M, kFix, true);
        float from = -INFINITY;
        if (M > 0.0f) {
            const float x = temp * logf(M);
            from = m + x - 1e-5f * (fabsf(x) + fabsf(m));
        }
        const bool alone = K == V && P >= 1.0f;  // nothing but min-p
        int listed = kList + 1;
        if (ranked || V <= kList || (alone && M > 0.0f)) {
            const float low = ranked ? of_ord(max((int)(floor_bits ^ 0x80000000u), ord(-INFINITY))) : alone ? from : -INFINITY;
            listed = r.gather([&](float x, int) { return x >= low && x > -INFINITY; });
            if (listed <= kList) {
                // (nobody reads another's shared memory any more)
                if (rank == 0) r.draw_from_list(listed, K, P, least, u, token, prob);
                return;
            }
        }
        Cut cut{-INFINITY, -1};
        if (K < V) cut = r.template narrow<false>(cut, K, P, temp);
        float inner = INFINITY;
        if (P < 1.0f) cut = r.nucleus(cut, P, temp, inner);
        // Of what is kept, what min-p takes is known by weight, unless the cut's own is enough: then it takes nothing.
        // (Looked at one by one, a token above the cut may be below `least` all the same, since weights of neighbouring
        // logits may be out of order by their rounding; both passes have to count it then.)
        // (Settings that say so cost no registers; a second test in `mass` took 9.3 us for 4 rows of 32000 where this takes 9.0.)
        const bool known = inner < INFINITY && weight(r.w, cut.v) >= least;
        if (known) from = -INFINITY, least = 0;
        auto mass = [&](float x, int id) -> long long {
            if (!(x >= from) || !kept(cut, x, id)) return 0;
            const long long y = weight(r.w, x);
            return y >= least ? y : 0;
        };
        if (known)  // what lies above the interval has been added up
            r.locate([&](float x, int id) -> long long { return x < inner && kept(cut, x, id) ? weight(r.w, x) : 0; }, -1, u,
                     s.keep[warp]);
        else
            r.locate(mass, -1, u);
        const long long total = s.total;
        r.search(mass, [&](float x, int id) {
            *token = id;
            if (prob) *prob = ratio(weight(r.w, x), total);
        });
    }
    if (C > 1) r.cl.sync();  // nobody leaves while its shared memory may be read
}

template <typename T>
cudaError_t launch_sample(const sv_sample_args& a, int C, int slice_elems, cudaStream_t st) {
    const size_t bytes = align_up(sizeof(SampleSmem), 16) + ((size_t)slice_elems + Vec<T>::N) * sizeof(T) + 16;
    static std::atomic<uint64_t> ready{0};  // devices whose kernel has its shared memory
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(ready.load() >> dev & 1)) {
        e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready.fetch_or(1ull << dev);
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {(unsigned)C, 1, 1};
    cfg.gridDim = dim3((unsigned)(a.B * a.N * C));
    cfg.blockDim = dim3(kSThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, sample_kernel<T>, a, C, slice_elems);
}

}  // namespace
}  // namespace sv

extern "C" int spec_verify_sample(const sv_sample_args* args, void* stream) {
    using namespace sv;
    if (!args || args->struct_size != sizeof(sv_sample_args)) return SV_EINVAL;
    const sv_sample_args& a = *args;
    if (a.dtype != SV_F32 && a.dtype != SV_BF16) return SV_EUNSUPPORTED;
    if (a.B < 0 || a.N < 1 || a.V < 1) return SV_EINVAL;
    if (a.V > SV_MAX_VOCAB || a.B > SV_MAX_BATCH || (double)a.B * a.N * kSCluster > 2147483647.0) return SV_ETOO_LARGE;
    if (a.B == 0) return SV_OK;
    const int es = a.dtype == SV_F32 ? 4 : 2;
    if (!a.logits || !a.uniforms || !a.tokens || a.stride_b < 0 || a.stride_n < 0 || a.uniform_stride < 0) return SV_EINVAL;
    if ((uintptr_t)a.logits % es || (((uintptr_t)a.uniforms | (uintptr_t)a.tokens | (uintptr_t)a.probs) & 3u)) return SV_EINVAL;
    // CTAs a row: slices of at most 80 KB, so that two CTAs have room on an SM (one's loads run while
    // the other computes), and more while the rows leave SMs empty and a slice keeps 2048 tokens.
    // us with 1 / 2 / 4 / 8 (the rule's: *; bf16, top-k 50 or 200 and top-p; nuclei: fp32, top-p alone):
    //    4 x 8000                  9.1 /  9.8* /  9.6 /      32 x 32000             11.7 / 11.0 / 10.4* / 12.4
    //    4 x 32000                11.0 / 10.6 /  9.8 / 10.0* 32 x 32000 bf16 nuclei 42.7 / 31.4 / 25.2* / 25.4
    //  256 x 32000                15.3* / 25.1 / 39.6 /      256 x 128256              - / 74.2 / 67.0* / 103.1
    //  192 x 151936 nuclei           - /    - / 227.6 / 208.1*
    int C = 1;
    while (C < kSCluster && ((a.V + C - 1) / C * es > 80 * 1024 || (a.B * a.N * C * 2 <= 152 && a.V / (2 * C) >= 2048))) C *= 2;
    const int slice = (int)(((a.V + C - 1) / C + 7) / 8 * 8);
    const cudaError_t e = a.dtype == SV_F32 ? launch_sample<float>(a, C, slice, (cudaStream_t)stream)
                                            : launch_sample<__nv_bfloat16>(a, C, slice, (cudaStream_t)stream);
    return e == cudaSuccess ? SV_OK : SV_ECUDA;
}
