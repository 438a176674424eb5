// sv_attend_rows.cu -- attention of a few query rows a cache head over a long cache:
// single tokens and verification rounds.
//
// Each key and value is read once for 16 or 32 query rows, 4 to 8 multiply-adds a byte
// and row: the call is bound by reading the cache.  So the design is about loads in
// flight.  The eight warps of a CTA work alone: a warp takes every eighth block of 16
// keys, with its own ring of blocks that it fills itself by asynchronous 16-byte copies
// (192 KB in flight a CTA), its own running maximum and sum (one pass over the keys) and
// its own output in registers; no barrier stands between it and its next block.  The
// ring runs on over the borders of units.  At the end of a unit the eight results are
// joined in shared memory.
//
// Scores and outputs use the warp-wide 16x8x16 matrix instructions: 16 rows of them are
// what a decode step fills, and they take under a third of the time that the bytes take.
#include "sv_attend.cuh"

namespace sv {
namespace {

constexpr int kAWarps = 8;
constexpr int kAThreads = 32 * kAWarps;
constexpr int kBlk = 16;  // keys of a block
static_assert(kBlk * kAWarps == kKeyTile, "a step of the CTA is one block a warp");

template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// shared memory: a row of D elements is D / 8 16-byte chunks, chunk c of row r at place
// c ^ (r & 7): the eight rows of a matrix load fall on different banks
template <int D>
__device__ __forceinline__ uint32_t sw(int r, int c) {
    return (uint32_t)(r * (D * 2) + ((c ^ (r & 7)) << 4));
}

template <int D>
struct RowsCfg {
    static constexpr int kStageBytes = 2 * kBlk * D * 2;           // a block's keys and values
    static constexpr int kStages = 24576 / kStageBytes;            // 24 KB a warp
    static constexpr int kRing = kAWarps * kStages * kStageBytes;  // 192 KB
    static constexpr int kJoinCols = 64;
    static constexpr int kJoin = kAWarps * 16 * kJoinCols * 4;     // 32 KB
};

// MT: tiles of 16 query rows
template <typename T, int D, int MT>
__global__ void __launch_bounds__(kAThreads, 1) attend_rows_kernel(const __grid_constant__ AttendArgs p) {
    using C = RowsCfg<D>;
    constexpr int RM = 16 * MT;
    constexpr int CH = D / 8;  // 16-byte chunks of a row
    extern __shared__ __align__(1024) unsigned char smem[];
    float* s_join = reinterpret_cast<float*>(smem + C::kRing);
    __shared__ float s_m[kAWarps][RM], s_l[kAWarps][RM];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int g = lane >> 2, q4 = lane & 3;
    grid_dependents_go();
    fill_idle_rows<T, kAThreads>(p);
    Part part;
    find_part<RM, kAThreads>(p, part, reinterpret_cast<int*>(s_join));
    if (part.todo == 0) return;

    unsigned char* ring = smem + warp * (C::kStages * C::kStageBytes);
    const uint32_t ring_s = (uint32_t)__cvta_generic_to_shared(ring);
    const int page_size = (int)p.a.cache.page_size;

    // the filling side: unit, tile in it, tiles left.  One block is in reach of a unit's
    // rows if it holds a key that a row of the tile sees.
    Unit fu = part.u;
    int ft = part.tile, fleft = part.todo;
    uint32_t bad_pages = 0;  // bit s: the block in stage s lies on a bad page
    auto fill = [&](int stage) {
        if (fleft > 0) {
            const int kb = ft * kAWarps + warp;  // block index
            const int k0 = kb * kBlk;
            int lo, hi;
            tile_keys<RM>(p, fu.past, fu.n, fu.rt, lo, hi);
            bad_pages &= ~(1u << stage);
            if (k0 <= hi && k0 + kBlk > lo) {
                const int index = page_of(p, k0);
                const int page = p.a.cache.page_table[fu.b * p.a.cache.page_table_stride + index];
                if (page < 0 || page >= p.a.cache.pages) {
                    bad_pages |= 1u << stage;
                    if (lane == 0 && p.a.row_status) atomicOr(p.a.row_status + fu.b, SV_ROW_BAD_PAGE);
                } else {
                    const int64_t in_page = k0 - index * page_size;
                    const T* k = (const T*)p.a.cache.k_pages + page * p.a.cache.k_stride_page +
                                 fu.h * p.a.cache.k_stride_head + in_page * p.a.cache.k_stride_slot;
                    const T* v = (const T*)p.a.cache.v_pages + page * p.a.cache.v_stride_page +
                                 fu.h * p.a.cache.v_stride_head + in_page * p.a.cache.v_stride_slot;
                    const uint32_t ks = ring_s + stage * C::kStageBytes, vs = ks + kBlk * D * 2;
#pragma unroll
                    for (int x = lane; x < kBlk * CH; x += 32) {
                        const int r = x / CH, c = x % CH;
                        cp_async16(ks + sw<D>(r, c), k + r * p.a.cache.k_stride_slot + c * 8);
                        cp_async16(vs + sw<D>(r, c), v + r * p.a.cache.v_stride_slot + c * 8);
                    }
                }
            }
            --fleft;
            if (++ft == fu.t1 && fleft > 0) {
                next_unit<RM>(p, fu);
                ft = fu.t0;
            }
        }
        cp_commit();
    };
#pragma unroll
    for (int s = 0; s < C::kStages - 1; ++s) fill(s);

    Unit u = part.u;
    int tile = part.tile;
    int left = part.todo, stage = 0;
    bool first_unit = true;
    while (left > 0) {
        const int rows = min(RM, u.n * p.group - u.rt * RM), r00 = u.rt * RM;
        const int i_first = by_group(p, r00);
        int lo, hi;
        tile_keys<RM>(p, u.past, u.n, u.rt, lo, hi);
        const int end = min(u.t1, tile + left);
        const bool from_start = tile == u.t0, to_end = end == u.t1;

        // query fragments: row g (and g + 8) of a tile, columns 2 q4 (and + 8) of a 16-wide step
        uint32_t qf[MT][D / 16][4];
        int qpos[MT][2];  // a row's own position: the last key it sees
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = m * 16 + g + e * 8;
                qpos[m][e] = r < rows ? u.past + by_group(p, r00 + r) : -1;
                const T* q = q_row<T>(p, u.b, u.h, r00 + min(r, rows - 1));
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
#pragma unroll
                    for (int f = 0; f < 2; ++f)
                        qf[m][k][e + 2 * f] = __ldg(reinterpret_cast<const uint32_t*>(q + k * 16 + f * 8 + q4 * 2));
            }
        float o[MT][D / 8][4];
        float mx[MT][2], sum[MT][2];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
#pragma unroll
            for (int d = 0; d < D / 8; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[m][d][e] = 0.0f;
            mx[m][0] = mx[m][1] = -INFINITY;
            sum[m][0] = sum[m][1] = 0.0f;
        }
        bool poisoned = false;

        for (; tile < end; ++tile, --left) {
            cp_wait<C::kStages - 2>();
            __syncwarp();
            // every lane is through with the stage before this one: fill it again
            fill(stage == 0 ? C::kStages - 1 : stage - 1);
            const uint32_t ks = ring_s + stage * C::kStageBytes, vs = ks + kBlk * D * 2;
            const int k0 = (tile * kAWarps + warp) * kBlk;
            const bool reach = k0 <= hi && k0 + kBlk > lo;
            const bool bad = bad_pages >> stage & 1u;
            poisoned |= bad;
            if (reach && !bad) {
                // values at positions that no row sees may be anything, and 0 * NaN is NaN
                const int vlo = lo - k0, vhi = u.past + u.n - k0;  // valid rows of the block
                if (vlo > 0 || vhi < kBlk) {
                    for (int x = lane; x < kBlk * CH; x += 32) {
                        const int r = x / CH;
                        if (r < vlo || r >= vhi)
                            *reinterpret_cast<uint4*>(ring + stage * C::kStageBytes + kBlk * D * 2 +
                                                      sw<D>(r, x % CH)) = make_uint4(0, 0, 0, 0);
                    }
                    __syncwarp();
                }
                float s[MT][2][4];
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[m][n][e] = 0.0f;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    uint32_t kf[4];  // keys 0..7: (k lo, k hi), keys 8..15: (k lo, k hi)
                    const int r = (lane & 7) + ((lane >> 4) << 3), c = 2 * k + ((lane >> 3) & 1);
                    ldsm4(kf, ks + sw<D>(r, c));
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        mma16816<T>(s[m][0], qf[m][k], kf[0], kf[1]);
                        mma16816<T>(s[m][1], qf[m][k], kf[2], kf[3]);
                    }
                }
                const bool all = k0 + kBlk - 1 <= u.past + i_first &&
                                 (p.a.window <= 0 || k0 > (int64_t)hi - p.a.window);
                uint32_t pf[MT][4];
#pragma unroll
                for (int m = 0; m < MT; ++m) {
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float x = s[m][n][e] * p.qscale;
                            if (!all) {
                                const int j = k0 + n * 8 + q4 * 2 + (e & 1), at = qpos[m][e >> 1];
                                if (j > at || (p.a.window > 0 && j <= at - p.a.window)) x = -INFINITY;
                            }
                            s[m][n][e] = x;
                        }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float v = fmaxf(fmaxf(s[m][0][2 * e], s[m][0][2 * e + 1]),
                                        fmaxf(s[m][1][2 * e], s[m][1][2 * e + 1]));
                        v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 1));
                        v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 2));
                        const float now = fmaxf(mx[m][e], v);
                        const float ref = now == -INFINITY ? 0.0f : now;  // nothing seen yet: weights 0
                        const float shrink = fast_exp2(mx[m][e] - ref);
                        mx[m][e] = now;
                        float add = 0.0f;
#pragma unroll
                        for (int n = 0; n < 2; ++n)
#pragma unroll
                            for (int f = 0; f < 2; ++f) {
                                const float w = fast_exp2(s[m][n][2 * e + f] - ref);
                                s[m][n][2 * e + f] = w;
                                add += w;
                            }
                        sum[m][e] = sum[m][e] * shrink + add;
                        if (__any_sync(0xFFFFFFFFu, shrink != 1.0f)) {
#pragma unroll
                            for (int d = 0; d < D / 8; ++d) {
                                o[m][d][2 * e] *= shrink;
                                o[m][d][2 * e + 1] *= shrink;
                            }
                        }
                    }
                    // weights in [0, 1] enter the product in 16 bits, as the values do
                    pf[m][0] = Pair<T>::pack(s[m][0][0], s[m][0][1]);
                    pf[m][1] = Pair<T>::pack(s[m][0][2], s[m][0][3]);
                    pf[m][2] = Pair<T>::pack(s[m][1][0], s[m][1][1]);
                    pf[m][3] = Pair<T>::pack(s[m][1][2], s[m][1][3]);
                }
#pragma unroll
                for (int d = 0; d < D / 16; ++d) {
                    uint32_t vf[4];
                    const int r = (lane & 7) + (((lane >> 3) & 1) << 3), c = 2 * d + (lane >> 4);
                    ldsm4t(vf, vs + sw<D>(r, c));
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        mma16816<T>(o[m][2 * d], pf[m], vf[0], vf[1]);
                        mma16816<T>(o[m][2 * d + 1], pf[m], vf[2], vf[3]);
                    }
                }
            }
            stage = stage + 1 == C::kStages ? 0 : stage + 1;
        }

        // join the warps: common maximum, then the sums in the warps' order
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l = sum[m][e];
                l += __shfl_xor_sync(0xFFFFFFFFu, l, 1);
                l += __shfl_xor_sync(0xFFFFFFFFu, l, 2);
                if (poisoned) l = NAN;
                if (q4 == 0) {
                    s_m[warp][m * 16 + g + e * 8] = mx[m][e];
                    s_l[warp][m * 16 + g + e * 8] = l;
                }
            }
        __syncthreads();
        const bool whole = from_start && to_end;
        const int place = 2 * blockIdx.x + (first_unit ? 0 : 1);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            float f[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float top = -INFINITY;
#pragma unroll
                for (int w = 0; w < kAWarps; ++w) top = fmaxf(top, s_m[w][m * 16 + g + e * 8]);
                f[e] = mx[m][e] == -INFINITY ? 0.0f : fast_exp2(mx[m][e] - top);
            }
#pragma unroll
            for (int half = 0; half < D / C::kJoinCols; ++half) {
#pragma unroll
                for (int d = 0; d < C::kJoinCols / 8; ++d) {
                    const int dd = half * (C::kJoinCols / 8) + d;
                    float* j0 = s_join + (warp * 16 + g) * C::kJoinCols + d * 8 + q4 * 2;
                    float* j1 = j0 + 8 * C::kJoinCols;
                    *reinterpret_cast<float2*>(j0) = make_float2(o[m][dd][0] * f[0], o[m][dd][1] * f[0]);
                    *reinterpret_cast<float2*>(j1) = make_float2(o[m][dd][2] * f[1], o[m][dd][3] * f[1]);
                }
                __syncthreads();
                // 16 rows x 64 columns: 4 columns a thread
                const int r = t >> 4, c = (t & 15) * 4, rr = m * 16 + r;
                float4 acc = make_float4(0, 0, 0, 0);
                float top = -INFINITY, l = 0.0f;
#pragma unroll
                for (int w = 0; w < kAWarps; ++w) top = fmaxf(top, s_m[w][rr]);
#pragma unroll
                for (int w = 0; w < kAWarps; ++w) {
                    const float4 x = *reinterpret_cast<const float4*>(s_join + (w * 16 + r) * C::kJoinCols + c);
                    acc.x += x.x;
                    acc.y += x.y;
                    acc.z += x.z;
                    acc.w += x.w;
                    l += s_l[w][rr] * (s_m[w][rr] == -INFINITY ? (s_l[w][rr] == 0.0f ? 0.0f : 1.0f)
                                                              : fast_exp2(s_m[w][rr] - top));
                }
                if (rr < rows) {
                    if (whole) {
                        const float inv = 1.0f / l;
                        uint2 pk = make_uint2(Pair<T>::pack(acc.x * inv, acc.y * inv),
                                              Pair<T>::pack(acc.z * inv, acc.w * inv));
                        *reinterpret_cast<uint2*>(out_row<T>(p, u.b, u.h, r00 + rr) + half * C::kJoinCols + c) = pk;
                    } else {
                        *reinterpret_cast<float4*>(p.part_o + ((int64_t)place * RM + rr) * D + half * C::kJoinCols +
                                                   c) = acc;
                        if (half == 0 && c == 0)
                            *reinterpret_cast<float2*>(p.part_ml + ((int64_t)place * RM + rr) * 2) =
                                make_float2(top, l);
                    }
                }
                __syncthreads();
            }
        }
        first_unit = false;
        if (left > 0) {
            next_unit<RM>(p, u);
            tile = u.t0;
        }
    }
    cp_wait<0>();
}

// A unit that was cut: the partial results of the CTAs that worked on it, in order.  Block
// c looks at the unit in which CTA c began; the first CTA that began inside a unit joins it.
constexpr int kJoinThreads = 256;
constexpr int kJoinCols = 16;
__device__ __forceinline__ bool join_unit(const AttendArgs& p, Cut& k) {
    grid_dependency_wait();
    k = p.cut[blockIdx.x];
    const long long c = blockIdx.x;
    if (k.ctas == 0 || c == 0) return false;
    return k.per * c + min(c, (long long)k.more) != k.base && k.per * (c - 1) + min(c - 1, (long long)k.more) <= k.base;
}
// calls f(place) for the unit's partial results in order
template <typename F>
__device__ __forceinline__ void join_each(const Cut& k, F f) {
#pragma unroll 4
    for (int c = blockIdx.x - 1; c < k.ctas; ++c) {
        const long long from = k.per * c + min(c, k.more);  // a CTA's first tile
        if (from >= k.end) break;
        f((int64_t)(2 * c + (from >= k.base ? 0 : 1)));
    }
}
// adds (m, l, x) to the running (top, sum, acc)
template <int N>
__device__ __forceinline__ void join_add(float& top, float& sum, float (&acc)[N], float m, float l, const float (&x)[N]) {
    if (m == -INFINITY) {
        sum += l;  // 0, or the NaN of a bad page or a wait that ran out
        return;
    }
    const float now = fmaxf(top, m);
    const float fa = fast_exp2(top - now), fb = fast_exp2(m - now);
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = acc[i] * fa + x[i] * fb;
    sum = sum * fa + l * fb;
    top = now;
}

// results by rows: a warp a row
template <typename T, int D, int RM>
__global__ void __launch_bounds__(kJoinThreads) attend_join_kernel(const __grid_constant__ AttendArgs p) {
    constexpr int PER = D / 32;  // columns a lane
    Cut k;
    if (!join_unit(p, k)) return;
    const int lane = threadIdx.x & 31;
    const int r = blockIdx.y * (kJoinThreads / 32) + (threadIdx.x >> 5);
    if (r >= k.n * p.group - k.rt * RM) return;
    float top = -INFINITY, l = 0.0f, acc[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] = 0.0f;
    join_each(k, [&](int64_t place) {
        const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + (place * RM + r) * 2);
        const float* src = p.part_o + (place * RM + r) * D + lane * PER;
        float x[PER];
        if constexpr (PER == 4) {
            const float4 y = *reinterpret_cast<const float4*>(src);
            x[0] = y.x, x[1] = y.y, x[2] = y.z, x[3] = y.w;
        } else {
            const float2 y = *reinterpret_cast<const float2*>(src);
            x[0] = y.x, x[1] = y.y;
        }
        join_add(top, l, acc, ml.x, ml.y, x);
    });
    const float inv = 1.0f / l;
    uint32_t w[PER / 2];
#pragma unroll
    for (int i = 0; i < PER / 2; ++i) w[i] = Pair<T>::pack(acc[2 * i] * inv, acc[2 * i + 1] * inv);
    T* dst = out_row<T>(p, k.b, k.h, k.rt * RM + r) + lane * PER;
    if constexpr (PER == 4)
        *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    else
        *reinterpret_cast<uint32_t*>(dst) = w[0];
}

// results by columns: a thread has kJoinCols columns of a row, a warp 32 rows
template <typename T, int D, int RM>
__global__ void __launch_bounds__(kJoinThreads) attend_join_columns_kernel(const __grid_constant__ AttendArgs p) {
    static_assert(RM == kJoinThreads, "a thread a row");
    Cut k;
    if (!join_unit(p, k)) return;
    const int r = threadIdx.x, c0 = blockIdx.y * kJoinCols;
    if (r >= k.n * p.group - k.rt * RM) return;
    float top = -INFINITY, l = 0.0f, acc[kJoinCols];
#pragma unroll
    for (int i = 0; i < kJoinCols; ++i) acc[i] = 0.0f;
    join_each(k, [&](int64_t place) {
        const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + (place * RM + r) * 2);
        float x[kJoinCols];
#pragma unroll
        for (int i = 0; i < kJoinCols; ++i) x[i] = p.part_o[(place * D + c0 + i) * RM + r];
        join_add(top, l, acc, ml.x, ml.y, x);
    });
    const float inv = 1.0f / l;
    uint32_t w[kJoinCols / 2];
#pragma unroll
    for (int i = 0; i < kJoinCols / 2; ++i) w[i] = Pair<T>::pack(acc[2 * i] * inv, acc[2 * i + 1] * inv);
    uint4* dst = reinterpret_cast<uint4*>(out_row<T>(p, k.b, k.h, k.rt * RM + r) + c0);
    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

template <typename T, int D, int MT>
cudaError_t launch_rows(const AttendArgs& p, cudaStream_t s) {
    using C = RowsCfg<D>;
    constexpr int bytes = C::kRing + C::kJoin;
    const cudaError_t e = cudaFuncSetAttribute(attend_rows_kernel<T, D, MT>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    attend_rows_kernel<T, D, MT><<<p.ctas, kAThreads, bytes, s>>>(p);
    return cudaGetLastError();
}
template <typename T, int D, int RM>
cudaError_t launch_join(const AttendArgs& p, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if constexpr (RM == kJoinThreads) {
        cfg.gridDim = dim3((unsigned)p.ctas, D / kJoinCols);
        return cudaLaunchKernelEx(&cfg, attend_join_columns_kernel<T, D, RM>, p);
    } else {
        cfg.gridDim = dim3((unsigned)p.ctas, RM / (kJoinThreads / 32));
        return cudaLaunchKernelEx(&cfg, attend_join_kernel<T, D, RM>, p);
    }
}

}  // namespace

cudaError_t launch_attend_rows(int dtype, int dim, int mt, const AttendArgs& p, cudaStream_t s) {
    if (dtype == SV_BF16) {
        if (dim == 64) return mt == 1 ? launch_rows<__nv_bfloat16, 64, 1>(p, s) : launch_rows<__nv_bfloat16, 64, 2>(p, s);
        return mt == 1 ? launch_rows<__nv_bfloat16, 128, 1>(p, s) : launch_rows<__nv_bfloat16, 128, 2>(p, s);
    }
    if (dim == 64) return mt == 1 ? launch_rows<__half, 64, 1>(p, s) : launch_rows<__half, 64, 2>(p, s);
    return mt == 1 ? launch_rows<__half, 128, 1>(p, s) : launch_rows<__half, 128, 2>(p, s);
}

template <typename T, int D>
cudaError_t join_of(int rm, const AttendArgs& p, cudaStream_t s) {
    return rm == 16 ? launch_join<T, D, 16>(p, s) : rm == 32 ? launch_join<T, D, 32>(p, s) : launch_join<T, D, 256>(p, s);
}

cudaError_t launch_attend_join(int dtype, int dim, int rm, const AttendArgs& p, cudaStream_t s) {
    if (dtype == SV_BF16)
        return dim == 64 ? join_of<__nv_bfloat16, 64>(rm, p, s) : join_of<__nv_bfloat16, 128>(rm, p, s);
    return dim == 64 ? join_of<__half, 64>(rm, p, s) : join_of<__half, 128>(rm, p, s);
}

}  // namespace sv
