// sv_sample.cu -- drawing a token of each row after temperature, top-k, top-p and min-p,
// from a given random number (spec_verify_sample).
//
// A token is where a sum of weights passes u times their total, so with V tokens there are V
// borders, some 1e-5 apart or less, and which side of one a draw falls on must not depend on
// how the sum was formed.  Weights exp((z - m) / T) are therefore formed as pairs of 32-bit
// numbers (to about 2^-40 of themselves; the 64-bit units of this GPU are too few), turned
// into whole numbers of 2^-44, and added as such: sums are exact and have no order.
//
// A cluster of CTAs has a row, each a slice of it in shared memory.  What is kept is always a
// run of the order (logit falling, id rising), so it is given by its last member: a cut
// (value, id).
//   top-k up to 128 a CTA, or few tokens  every warp's j-th largest lane maximum is a floor
//       that at least k tokens reach; those that do (a few times k) are listed, and one CTA
//       sorts them, cuts them by k, mass and min-p and draws.
//   otherwise  the cut is found by narrowing: a pass counts or weighs the tokens at and above
//       seven pivots of the interval that holds it, in 3 bits a pass, until the interval has few
//       tokens (listed and sorted as above) or one value (whose tokens are counted by id).
//       Then a pass adds up what is kept, warp by warp in the order of ids, and the warp in
//       whose part the sum passes u times the total goes through it again.
// A pass is bound by the instructions of the weights, some 45 an element.
#include <cooperative_groups.h>

#include <atomic>

#include "sv_internal.cuh"
#include "sv_paged.cuh"

namespace sv {
namespace {

namespace cg = cooperative_groups;

constexpr int kSThreads = 512, kSWarps = kSThreads / 32;
constexpr int kSCluster = 8;      // CTAs a row at most
constexpr int kList = 2048;       // tokens that one CTA sorts
constexpr int kPer = kList / kSThreads;
constexpr int kPivots = 7;
constexpr int kFix = 44;          // weights are whole numbers of 2^-44: sums of 2^18 of them stay below 2^62
constexpr int kHalfFix = kFix / 2;
constexpr int kFloorRank = 8;     // lanes of a warp that the floor may rank

struct Cut {  // kept: x > v, and x == v up to id
    float v;
    int id;
};
struct Slot {  // what a CTA tells the others
    long long mass[kPivots + 1];
    int count[kPivots + 1];
    long long warp[kSWarps];
    float top, floor;
    int bad, n, id;
    Cut cut;
};
struct SampleSmem {
    uint64_t list[kList];
    float2 tab[64];  // 2^(i / 64) in two parts
    Slot slot[2];
    long long wmass[kSWarps][kPivots + 1];
    int wcount[kSWarps][kPivots + 1];
    long long total, before;
    int n_list, place, r;
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
    // 2^p = 2^(j / 64) 2^f: f in [-1/128, 1/128]
    const float js = __fadd_rn(p, 196608.0f);  // 1.5 * 2^17: steps of 1/64
    const int j = __float_as_int(js) - 0x48400000;
    const float f = __fsub_rn(p, __fsub_rn(js, 196608.0f));
    // (f + q) ln 2 = t + s
    constexpr float kLn2 = (float)0.69314718055994530942, kLn2Lo = (float)(0.69314718055994530942 - (double)kLn2);
    const float t = __fmul_rn(f, kLn2);
    float s = __fmaf_rn(f, kLn2, -t);
    s = __fmaf_rn(f, kLn2Lo, s);
    s = __fmaf_rn(q, kLn2, s);
    // exp(t + s) - 1 - t: the series to t^5 (t is below 2^-7.5)
    float g = __fmaf_rn(t, 1.0f / 120.0f, 1.0f / 24.0f);
    g = __fmaf_rn(t, g, 1.0f / 6.0f);
    g = __fmaf_rn(t, g, 0.5f);
    g = __fmul_rn(__fmul_rn(t, t), g);
    g = __fadd_rn(g, __fmaf_rn(t, s, s));
    const float2 b = w.tab[j & 63];
    // b (1 + t + g): the parts below 1 first, then their sum and what it leaves
    const float a = __fmul_rn(b.x, t), ae = __fmaf_rn(b.x, t, -a), bg = __fmul_rn(b.x, g);
    const float k = __fadd_rn(a, bg), ke = __fsub_rn(bg, __fsub_rn(k, a));
    const float h = __fadd_rn(b.x, k);
    float l = __fsub_rn(k, __fsub_rn(h, b.x));
    l = __fadd_rn(l, __fadd_rn(ae, ke));
    l = __fmaf_rn(b.y, __fadd_rn(1.0f, t), l);
    const float scale = __int_as_float(((j >> 6) + kHalfFix + 127) << 23);
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
        int n = 0, counts[kSCluster];
        for (int r = 0; r < C; ++r) n += counts[r] = of(r)->n;
        if (C > 1) {
            if (n <= kList && rank == 0) {
                int at = counts[0];
                for (int r = 1; r < C; ++r) {
                    const uint64_t* src = cl.map_shared_rank(s.list, r);
                    for (int i = t; i < counts[r]; i += kSThreads) s.list[at + i] = src[i];
                    at += counts[r];
                }
            }
            cl.sync();  // the others' lists may be written again
        } else {
            __syncthreads();
        }
        return n;
    }

    // ceil(P S) for the comparison of whole numbers with it
    static __device__ long long mass_target(float P, long long S) { return (long long)ceil((double)P * (double)S); }

    // Draws from the list's n entries, sorted: top-k, top-p and min-p (x >= least), then by id.  By one CTA.
    __device__ void draw_from_list(int n, int K, float P, float least, float u, int32_t* token, float* prob) {
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
            keep += e < n && before[i] < target && key_value(s.list[e]) >= least;
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
        const long long v = (long long)floor((double)u * (double)kept_mass);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (before[i] <= v && before[i] + val[i] > v) {
                *token = (int)(~s.list[t * kPer + i] >> 32);
                if (prob) *prob = (float)((double)val[i] / (double)kept_mass);
            }
    }

    // One pass of narrowing: of the members of `cut` in [lo, hi), mass and number at and above each
    // pivot; entry kPivots: of all of them.  Summed over the cluster.
    template <bool MASS>
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
                    if (j == kPivots || x >= p[j]) {
                        if (MASS) h[j] += wh, l[j] += wl;
                        ++n[j];
                    }
            }
        });
#pragma unroll
        for (int j = 0; j <= kPivots; ++j) {
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
#pragma unroll
        for (int j = 0; j <= kPivots; ++j) mass[j] = 0, count[j] = 0;
        for (int r = 0; r < C; ++r) {
            const Slot* q = of(r);
#pragma unroll
            for (int j = 0; j <= kPivots; ++j) {
                count[j] += q->count[j];
                if (MASS) mass[j] += q->mass[j];
            }
        }
    }

    // The warp in whose part the running sum of f over ids first passes `over` (or share * the total of
    // all, where over < 0): its place in the cluster, the sum before it and the total, in s; nobody: -1.
    template <typename F>
    __device__ void locate(F f, long long over, double share) {
        long long own = 0;
        each([&](float x, int id) { own += f(x, id); });
        own = warp_sum(own);
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
            const long long v = over >= 0 ? over : (long long)floor(share * (double)total);
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
                constexpr float kFirst[kPivots] = {16.0f, 12.0f, 9.0f, 7.0f, 5.0f, 3.0f, 1.5f};
                const float x = (float)(j + 1) / (kPivots + 1);
                // by distance from the largest; then by value and by the order of floats in turn: one converges
                // quickly on smooth rows, the other in 11 passes on any
                p[j] = round == 0 ? w.m - kFirst[j] * temp
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
                    if (rank == 0) {
                        sort(n);
                        int keep = 0;
                        if (MASS) {
                            long long val[kPer], before[kPer];
#pragma unroll
                            for (int i = 0; i < kPer; ++i) {
                                const int e = t * kPer + i;
                                val[i] = e < n ? weight(w, key_value(s.list[e])) : 0;
                            }
                            scan(val, before);
#pragma unroll
                            for (int i = 0; i < kPer; ++i) keep += t * kPer + i < n && above + before[i] < target;
                            keep = count_of(keep);
                        } else {
                            keep = (int)(target - above);
                        }
                        if (t == 0) {
                            const uint64_t k = s.list[max(keep, 1) - 1];
                            mine().cut = Cut{key_value(k), key_id(k)};
                        }
                    }
                    exchange();
                    res = of(0)->cut;
                } else {
                    // one value: its first `keep` by id
                    const long long each_one = MASS ? weight(w, lo) : 1;
                    const long long keep = (target - above + each_one - 1) / max(each_one, 1ll);
                    auto one = [&](float x, int id) -> long long { return x == lo && kept(cut, x, id); };
                    locate(one, keep - 1, 0.0);
                    const int at = s.place;
                    search(one, [&](float, int id) { mine().id = id; });
                    exchange();
                    res = Cut{lo, at < 0 ? 0x7FFFFFFF : of(at / kSWarps)->id};
                }
                return res;
            }
        }
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
    if (t < 64) {
        const double d = exp2(t / 64.0);
        s.tab[t] = make_float2((float)d, (float)(d - (double)(float)d));
    }
    SampleRow<T> r{a, s, slice, cg::this_cluster(), C, rank, t, lane, warp, v0, v1, first - pad, 0, {}};

    // ---- the largest, and a floor that at least K tokens reach
    const int j = (K + C * kSWarps - 1) / (C * kSWarps);  // of each warp
    const bool ranked = K < V && j <= kFloorRank;
    const bool poison = __any_sync(0xFFFFFFFFu, !(top < INFINITY));
    int o = ord(top);
    const float wtop = of_ord(__reduce_max_sync(0xFFFFFFFFu, o));
    float wfloor = -INFINITY;
    if (ranked) {
        int least = 0;
        for (int k = 0; k < j; ++k) {
            least = __reduce_max_sync(0xFFFFFFFFu, o);
            const unsigned who = __ballot_sync(0xFFFFFFFFu, o == least);
            if (lane == __ffs(who) - 1) o = (int)0x80000000;
        }
        wfloor = of_ord(max(least, ord(-INFINITY)));
    }
    if (lane == 0) {
        s.wcount[warp][0] = poison;
        s.wcount[warp][1] = __float_as_int(wtop);
        s.wcount[warp][2] = __float_as_int(wfloor);
    }
    __syncthreads();
    if (t == 0) {
        int any = 0;
        float hi = -INFINITY, lo = INFINITY;
        for (int k = 0; k < kSWarps; ++k) {
            any |= s.wcount[k][0];
            hi = fmaxf(hi, __int_as_float(s.wcount[k][1]));
            lo = fminf(lo, __int_as_float(s.wcount[k][2]));
        }
        Slot& q = r.mine();
        q.bad = any, q.top = hi, q.floor = lo;
    }
    r.exchange();
    int any = 0;
    float m = -INFINITY, floor_at = INFINITY;
    for (int k = 0; k < C; ++k) {
        const Slot* q = r.of(k);
        any |= q->bad;
        m = fmaxf(m, q->top);
        floor_at = fminf(floor_at, q->floor);
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
        const double c = 1.4426950408889634 / (double)fmaxf(Tm, 1e-30f);
        r.w = Weight{m, (float)c, (float)(c - (double)(float)c), s.tab};
        // min-p: the least value that is likely enough
        float least = -INFINITY;
        if (M > 0.0f) {
            const double x = (double)m + (double)Tm * log((double)M);
            least = fminf(__double2float_ru(x), m);
        }
        const bool alone = K == V && P >= 1.0f;  // nothing but min-p
        int listed = kList + 1;
        if (ranked || V <= kList || (alone && M > 0.0f)) {
            const float from = ranked ? floor_at : alone ? least : -INFINITY;
            listed = r.gather([&](float x, int) { return x >= from && x > -INFINITY; });
            if (listed <= kList && rank == 0) r.draw_from_list(listed, K, P, least, u, token, prob);
        }
        if (listed > kList) {
            Cut cut{-INFINITY, -1};
            if (K < V) cut = r.template narrow<false>(cut, K, P, Tm);
            if (P < 1.0f) cut = r.template narrow<true>(cut, K, P, Tm);
            if (least > cut.v) cut = Cut{least, 0x7FFFFFFF};
            auto mass = [&](float x, int id) -> long long { return kept(cut, x, id) ? weight(r.w, x) : 0; };
            r.locate(mass, -1, (double)u);
            const long long total = s.total;
            r.search(mass, [&](float x, int id) {
                *token = id;
                if (prob) *prob = (float)((double)weight(r.w, x) / (double)total);
            });
        }
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
    // the other computes), and more while the rows leave SMs empty and a slice keeps 2048 tokens
    int C = 1;
    while (C < kSCluster && ((a.V + C - 1) / C * es > 80 * 1024 || (a.B * a.N * C * 2 <= 152 && a.V / (2 * C) >= 2048))) C *= 2;
    const int slice = (int)(((a.V + C - 1) / C + 7) / 8 * 8);
    const cudaError_t e = a.dtype == SV_F32 ? launch_sample<float>(a, C, slice, (cudaStream_t)stream)
                                            : launch_sample<__nv_bfloat16>(a, C, slice, (cudaStream_t)stream);
    return e == cudaSuccess ? SV_OK : SV_ECUDA;
}
