// sv_attend_rows.cu -- attention of a few query rows a cache head over a long cache:
// single tokens and verification rounds; and the join of units that were cut.
//
// Each key and value is read once for up to 32 query rows, 2 multiply-adds a byte and
// row: the call is bound by reading the cache.  Three warps of a CTA do nothing but load:
// they look the pages up, 32 blocks of 16 keys at a time, and keep a ring of 144 KB of
// blocks in flight by TMA.  (One such warp takes some 700 cycles a block, twice what the
// memory does.)  Twelve warps compute.  A block belongs to a group of MT
// warps, one for each 16 rows, and blocks go round the 12 / MT groups, so that no barrier
// stands between a warp and its next block: each has its own running maximum and sum (one
// pass over the keys) and its own output in registers.  The ring runs on over the borders
// of units; at the end of a unit the groups' results are joined in shared memory.
//
// 64 sequences of 1.5-8k keys, 8 tokens each (32 / 8 heads of 128, bf16): 234 us, 5.5 TB/s
// of keys and values, 0.82 of the copy rate; the rest is the units' ends and the start.
// (Warps that filled their own rings by 16-byte copies spent 885 instructions on a block,
// half of them on addresses, and reached 3.7 TB/s; with one loading warp it was 3.4 TB/s.)
//
// Scores and outputs use the warp-wide 16x8x16 matrix instructions: 16 rows of them are
// what a decode step fills.
#include <atomic>

#include "sv_async.cuh"
#include "sv_attend.cuh"

namespace sv {
namespace {

constexpr int kAWarps = 12;  // that compute
constexpr int kLoaders = 3;  // warps that load; up to 16 in all, four a scheduler, leave 128 registers a thread
constexpr int kACompute = 32 * kAWarps;
constexpr int kAThreads = kACompute + 32 * kLoaders;
constexpr int kBlk = 16;  // keys of a block
constexpr int kTileBlks = kKeyTile / kBlk;

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
// a block in shared memory: D / 64 parts of 16 rows x 128 bytes, as TMA writes them; 16-byte
// chunk c of a row at place c ^ (row & 7) of its part, so that the eight rows of a matrix
// load fall on different banks
__device__ __forceinline__ uint32_t blk_at(int r, int c) {
    return (uint32_t)((c >> 3) * (kBlk * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}
// query rows of D elements, swizzled likewise
template <int D>
__device__ __forceinline__ uint32_t q_at(int r, int c) {
    return (uint32_t)(r * (D * 2) + ((c ^ (r & 7)) << 4));
}
__device__ __forceinline__ void compute_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kACompute) : "memory"); }

template <int D, int MT>
struct RowsCfg {
    static constexpr int kHalfBytes = kBlk * D * 2;       // a block's keys, or its values
    static constexpr int kBlkBytes = 2 * kHalfBytes;
    // 144 KB (192 KB for MT = 1).  A stage belongs to one group and one loading warp for
    // good: a phase parity only tells a barrier's last two phases apart, so nobody may wait
    // for a phase of a stage whose phase before was not its own to see.
    static constexpr int kStages = D == 64 ? 36 : MT == 1 ? 24 : 18;
    static_assert(kStages % (kAWarps / MT) == 0 && kStages % kLoaders == 0, "stages change hands");
    static constexpr int kRing = kStages * kBlkBytes;
    static constexpr int kQBytes = 16 * MT * D * 2;
    static constexpr int kJoinCols = 32;
    static constexpr int kJoin = kAWarps * 16 * kJoinCols * 4;  // 24 KB
    static constexpr int kSmem = kRing + kQBytes + kJoin + 1024;  // and room to align
};

// MT: tiles of 16 query rows
template <typename T, int D, int MT>
__global__ void __launch_bounds__(kAThreads, 1)
    attend_rows_kernel(const __grid_constant__ AttendArgs p, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap) {
    using C = RowsCfg<D, MT>;
    constexpr int RM = 16 * MT;
    constexpr int GROUPS = kAWarps / MT;
    constexpr int CH = D / 8;  // 16-byte chunks of a row
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint64_t s_full[C::kStages], s_empty[C::kStages];
    __shared__ uint8_t s_bad[C::kStages];  // the block in the stage lies on a bad page
    __shared__ int s_dead;
    __shared__ float s_m[GROUPS][RM], s_l[GROUPS][RM];  // per group: reference and sum
    __shared__ float2 s_ml[RM];                         // of all
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    grid_dependents_go();
    const uint32_t ring_s = (smem_u32(smem_raw) + 1023u) & ~1023u;
    unsigned char* ring = smem_raw + (ring_s - smem_u32(smem_raw));
    unsigned char* s_q = ring + C::kRing;
    const uint32_t q_s = ring_s + C::kRing;
    float* s_join = reinterpret_cast<float*>(ring + C::kRing + C::kQBytes);
    if (t == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            bar_init(&s_full[s], 1);
            bar_init(&s_empty[s], MT);
        }
        s_dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
    }
    grid_dependency_wait();
    fill_idle_rows<T, D, kAThreads>(p);
    Part part;
    find_part<RM, kAThreads>(p, part, reinterpret_cast<int*>(s_join));
    __syncthreads();
    if (part.todo == 0) return;
    volatile int* dead = &s_dead;
    const unsigned long long limit = p.wait_ns;

    if (warp >= kAWarps) {
        // ---------------------------------------------------------------- loads
        // every kLoaders-th block of the CTA's part
        const uint32_t mine = warp - kAWarps;
        Unit u = part.u;
        int tile = part.tile, left = part.todo;
        uint32_t seq = 0, done = 0;  // blocks counted through; the end of those issued
        bool alive = true;
        while (alive && left > 0) {
            const int end = min(u.t1, tile + left);
            int lo, hi;
            tile_keys<RM>(p, u.past, u.n, u.rt, lo, hi);
            const int32_t* pages = p.a.cache.page_table + u.b * p.a.cache.page_table_stride;
            for (int b0 = tile * kTileBlks; alive && b0 < end * kTileBlks; b0 += 32) {
                // a lane a block: its page, and the row of it (no visible key: -1, bad: -2)
                const int k0 = (b0 + lane) * kBlk;
                int page = -1, in_page = 0;
                if (b0 + lane < end * kTileBlks && k0 <= hi && k0 + kBlk > lo) {
                    const int i = page_of(p, k0);
                    page = pages[i];
                    in_page = k0 - i * (int)p.a.cache.page_size;
                    if (page < 0 || page >= p.a.cache.pages) {
                        page = -2;
                        if (p.a.row_status) atomicOr(p.a.row_status + u.b, SV_ROW_BAD_PAGE);
                    }
                }
                const uint32_t n = min(32, end * kTileBlks - b0);
                for (uint32_t i = (mine + kLoaders - seq % kLoaders) % kLoaders; i < n; i += kLoaders) {
                    const int pg = __shfl_sync(0xFFFFFFFFu, page, i), at = __shfl_sync(0xFFFFFFFFu, in_page, i);
                    const uint32_t stage = (seq + i) % C::kStages;
                    alive = bar_wait(&s_empty[stage], ((seq + i) / C::kStages & 1u) ^ 1u, limit, dead);
                    if (!alive) break;
                    if (lane == 0) {
                        s_bad[stage] = pg == -2;
                        if (pg >= 0)
                            bar_expect(&s_full[stage], C::kBlkBytes);
                        else
                            bar_arrive(&s_full[stage]);
                    }
                    __syncwarp();
                    if (pg >= 0 && lane < 2)
                        tma_box(ring_s + stage * C::kBlkBytes + lane * C::kHalfBytes, lane ? &vmap : &kmap, at, u.h, pg,
                                &s_full[stage]);
                    done = seq + i + 1;
                }
                seq += n;
            }
            left -= end - tile;
            if (left > 0) {
                next_unit<RM>(p, u);
                tile = u.t0;
            }
        }
        // copies still in flight end before the CTA does (whoever gave up)
        const unsigned long long t0 = now_ns();
        for (uint32_t i = done < C::kStages ? 0 : done - C::kStages; i < done; ++i)
            if (i % kLoaders == mine)
                while (!bar_try(&s_full[i % C::kStages], (i / C::kStages) & 1u) && now_ns() - t0 < kWaitLimitNs) {}
    } else {
        // -------------------------------------------------------------- products
        const int grp = warp / MT, m = warp % MT;
        const int g = lane >> 2, q4 = lane & 3;
        Unit u = part.u;
        int tile = part.tile, left = part.todo;
        uint32_t first_blk = 0;  // the unit's first block, counted through the CTA's part
        bool first_unit = true, alive = true;

        // a unit's query rows: the thread's pieces, then to shared memory
        constexpr int QP = (RM * CH + kACompute - 1) / kACompute;
        uint4 qv[QP];
        auto fetch_q = [&](const Unit& w) {
#pragma unroll
            for (int i = 0; i < QP; ++i) {
                const int x = t + i * kACompute, r = x / CH;
                if (x < RM * CH)
                    qv[i] = __ldg(reinterpret_cast<const uint4*>(
                                      q_row<T>(p, w.b, w.h, min(w.rt * RM + r, w.n * p.group - 1))) + x % CH);
            }
        };
        auto place_q = [&]() {
#pragma unroll
            for (int i = 0; i < QP; ++i) {
                const int x = t + i * kACompute;
                if (x < RM * CH) *reinterpret_cast<uint4*>(s_q + q_at<D>(x / CH, x % CH)) = qv[i];
            }
            compute_sync();
        };
        fetch_q(u);
        place_q();
        while (left > 0) {
            const int r00 = u.rt * RM, rows = min(RM, u.n * p.group - r00);
            int lo, hi;
            tile_keys<RM>(p, u.past, u.n, u.rt, lo, hi);
            const int end = min(u.t1, tile + left);
            const bool whole = tile == u.t0 && end == u.t1;
            // the warp's rows g and g + 8: their positions, the last keys that they see
            const int r0 = m * 16 + g;
            const int pos[2] = {u.past + by_group(p, r00 + min(r0, rows - 1)),
                                u.past + by_group(p, r00 + min(r0 + 8, rows - 1))};
            const int pos_first = u.past + by_group(p, r00);
            float o[D / 8][4];
            float ref[2] = {-INFINITY, -INFINITY}, sum[2] = {0.0f, 0.0f};
#pragma unroll
            for (int d = 0; d < D / 8; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[d][e] = 0.0f;
            bool poisoned = false;
            const uint32_t nblk = (uint32_t)(end - tile) * kTileBlks;
            // this group's blocks: those whose count is grp modulo GROUPS
            for (uint32_t i = (grp + GROUPS - first_blk % GROUPS) % GROUPS; alive && i < nblk; i += GROUPS) {
                const uint32_t seq = first_blk + i, stage = seq % C::kStages;
                alive = bar_wait(&s_full[stage], (seq / C::kStages) & 1u, limit, dead);
                if (!alive) break;
                const int k0 = (tile * kTileBlks + (int)i) * kBlk;
                const bool bad = s_bad[stage];
                poisoned |= bad;
                if (!bad && m * 16 < rows && k0 <= hi && k0 + kBlk > lo) {
                    const uint32_t ks = ring_s + stage * C::kBlkBytes, vs = ks + C::kHalfBytes;
                    // values at positions that no row sees may be anything, and 0 * NaN is NaN
                    // (each warp of the group writes these zeros, before it reads)
                    const int vlo = lo - k0, vhi = u.past + u.n - k0;  // valid rows of the block
                    if (vlo > 0 || vhi < kBlk) {
                        for (int x = lane; x < kBlk * CH; x += 32) {
                            const int r = x / CH;
                            if (r < vlo || r >= vhi)
                                *reinterpret_cast<uint4*>(ring + stage * C::kBlkBytes + C::kHalfBytes +
                                                          blk_at(r, x % CH)) = make_uint4(0, 0, 0, 0);
                        }
                        fence_async_smem();
                        __syncwarp();
                    }
                    float s[2][4];
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[n][e] = 0.0f;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        uint32_t qf[4], kf[4];  // keys 0..7: (k lo, k hi), keys 8..15: (k lo, k hi)
                        ldsm4(qf, q_s + q_at<D>(m * 16 + (lane & 15), 2 * k + (lane >> 4)));
                        ldsm4(kf, ks + blk_at((lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)));
                        mma16816<T>(s[0], qf, kf[0], kf[1]);
                        mma16816<T>(s[1], qf, kf[2], kf[3]);
                    }
                    const bool all = k0 + kBlk - 1 <= pos_first &&
                                     (p.a.window <= 0 || k0 > (int64_t)hi - p.a.window);
                    if (!all) {
#pragma unroll
                        for (int n = 0; n < 2; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int j = k0 + n * 8 + q4 * 2 + (e & 1), at = pos[e >> 1];
                                if (j > at || (p.a.window > 0 && j <= at - p.a.window)) s[n][e] = -INFINITY;
                            }
                    }
                    float top[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float v = fmaxf(fmaxf(s[0][2 * e], s[0][2 * e + 1]), fmaxf(s[1][2 * e], s[1][2 * e + 1]));
                        v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 1));
                        top[e] = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 2)) * p.qscale;
                    }
                    // the reference of the weights is only raised when a row outgrows it by 2^8
                    if (__any_sync(0xFFFFFFFFu, top[0] > ref[0] + 8.0f || top[1] > ref[1] + 8.0f)) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float now = fmaxf(ref[e], top[e]);
                            const float f = now == -INFINITY ? 1.0f : fast_exp2(ref[e] - now);
                            ref[e] = now;
                            sum[e] *= f;
#pragma unroll
                            for (int d = 0; d < D / 8; ++d) {
                                o[d][2 * e] *= f;
                                o[d][2 * e + 1] *= f;
                            }
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float base = weight_base<T>(ref[e]);
#pragma unroll
                        for (int n = 0; n < 2; ++n)
#pragma unroll
                            for (int f = 0; f < 2; ++f) {
                                const float w = fast_exp2(fmaf(s[n][2 * e + f], p.qscale, -base));
                                s[n][2 * e + f] = w;
                                sum[e] += w;
                            }
                    }
                    // weights enter the product in 16 bits, as the values do
                    const uint32_t pf[4] = {Pair<T>::pack(s[0][0], s[0][1]), Pair<T>::pack(s[0][2], s[0][3]),
                                            Pair<T>::pack(s[1][0], s[1][1]), Pair<T>::pack(s[1][2], s[1][3])};
#pragma unroll
                    for (int d = 0; d < D / 16; ++d) {
                        uint32_t vf[4];
                        ldsm4t(vf, vs + blk_at((lane & 7) + (((lane >> 3) & 1) << 3), 2 * d + (lane >> 4)));
                        mma16816<T>(o[2 * d], pf, vf[0], vf[1]);
                        mma16816<T>(o[2 * d + 1], pf, vf[2], vf[3]);
                    }
                }
                __syncwarp();
                if (lane == 0) bar_arrive(&s_empty[stage]);
            }
            if (!alive && lane == 0 && p.a.row_status) atomicOr(p.a.row_status + u.b, SV_ROW_INTERNAL);
            first_blk += nblk;
            left -= end - tile;
            Unit next = u;
            if (left > 0) {
                next_unit<RM>(p, next);
                fetch_q(next);
            }

            // join the groups: common maximum, then the sums in the groups' order
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l = sum[e];
                l += __shfl_xor_sync(0xFFFFFFFFu, l, 1);
                l += __shfl_xor_sync(0xFFFFFFFFu, l, 2);
                if (q4 == 0) {
                    s_m[grp][r0 + e * 8] = ref[e];
                    s_l[grp][r0 + e * 8] = poisoned || !alive ? NAN : l;
                }
            }
            compute_sync();
            const int place = 2 * blockIdx.x + (first_unit ? 0 : 1);
            float f[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float top = -INFINITY;
#pragma unroll
                for (int w = 0; w < GROUPS; ++w) top = fmaxf(top, s_m[w][r0 + e * 8]);
                f[e] = ref[e] == -INFINITY ? 0.0f : fast_exp2(ref[e] - top);
            }
            if (t < RM) {
                float top = -INFINITY, l = 0.0f;
#pragma unroll
                for (int w = 0; w < GROUPS; ++w) top = fmaxf(top, s_m[w][t]);
#pragma unroll
                for (int w = 0; w < GROUPS; ++w) {
                    const float mw = s_m[w][t], lw = s_l[w][t];
                    l += lw != lw ? lw : mw == -INFINITY ? 0.0f : lw * fast_exp2(mw - top);
                }
                s_ml[t] = make_float2(top, l);
                if (!whole && t < rows)
                    *reinterpret_cast<float2*>(p.part_ml + ((int64_t)place * RM + t) * 2) = make_float2(top, l);
            }
#pragma unroll
            for (int c0 = 0; c0 < D; c0 += C::kJoinCols) {
#pragma unroll
                for (int d = 0; d < C::kJoinCols / 8; ++d) {
                    float* j0 = s_join + (warp * 16 + g) * C::kJoinCols + ((d * 8 + q4 * 2) ^ ((g & 3) << 3));
                    float* j1 = j0 + 8 * C::kJoinCols;
                    const int dd = c0 / 8 + d;
                    *reinterpret_cast<float2*>(j0) = make_float2(o[dd][0] * f[0], o[dd][1] * f[0]);
                    *reinterpret_cast<float2*>(j1) = make_float2(o[dd][2] * f[1], o[dd][3] * f[1]);
                }
                compute_sync();
                for (int x = t; x < RM * (C::kJoinCols / 4); x += kACompute) {
                    const int r = x / (C::kJoinCols / 4), c = x % (C::kJoinCols / 4) * 4;
                    if (r >= rows) continue;
                    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                    for (int w = 0; w < GROUPS; ++w) {
                        const float4 y = *reinterpret_cast<const float4*>(
                            s_join + ((w * MT + (r >> 4)) * 16 + (r & 15)) * C::kJoinCols + (c ^ ((r & 3) << 3)));
                        acc.x += y.x;
                        acc.y += y.y;
                        acc.z += y.z;
                        acc.w += y.w;
                    }
                    if (whole) {
                        const float inv = 1.0f / s_ml[r].y;
                        *reinterpret_cast<uint2*>(out_row<T>(p, u.b, u.h, r00 + r) + c0 + c) = make_uint2(
                            Pair<T>::pack(acc.x * inv, acc.y * inv), Pair<T>::pack(acc.z * inv, acc.w * inv));
                    } else {
                        *reinterpret_cast<float4*>(p.part_o + ((int64_t)place * RM + r) * D + c0 + c) = acc;
                    }
                }
                compute_sync();
            }
            first_unit = false;
            if (left > 0) {
                place_q();
                u = next;
                tile = u.t0;
            }
        }
    }
}

// A unit that was cut: the partial results of the CTAs that worked on it, joined in order.
// Blocks (c, ...) look at the unit in which CTA c began; the first CTA that began inside a
// unit joins it.  Of a long axis there are many partial results to a row: PG warps take
// every PG-th each, and their sums meet in shared memory.
__device__ __forceinline__ bool join_unit(const AttendArgs& p, Cut& k) {
    grid_dependents_go();
    grid_dependency_wait();
    k = p.cut[blockIdx.x];
    const long long c = blockIdx.x;
    if (k.ctas == 0 || c == 0) return false;
    return k.per * c + min(c, (long long)k.more) != k.base && k.per * (c - 1) + min(c - 1, (long long)k.more) <= k.base;
}
// calls f(place) for the unit's partial results g, g + PG, ...
template <int PG, typename F>
__device__ __forceinline__ void join_each(const Cut& k, int g, F f) {
#pragma unroll 4
    for (int c = (int)blockIdx.x - 1 + g; c < k.ctas; c += PG) {
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

// results by rows: a warp has all columns of a row; a block kJoinRows rows
constexpr int kJoinRows = 4, kJoinGroups = 4;
template <typename T, int D, int RM>
__global__ void __launch_bounds__(32 * kJoinRows * kJoinGroups)
    attend_join_kernel(const __grid_constant__ AttendArgs p) {
    constexpr int PER = D / 32;  // columns a lane
    __shared__ float s_x[kJoinRows][kJoinGroups][D];
    __shared__ float2 s_ml[kJoinRows][kJoinGroups];
    Cut k;
    if (!join_unit(p, k)) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int j = warp / kJoinGroups, g = warp % kJoinGroups, r = blockIdx.y * kJoinRows + j;
    const bool live = r < k.n * p.group - k.rt * RM;
    float top = -INFINITY, l = 0.0f, acc[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] = 0.0f;
    auto add = [&](const float2 ml, const float* src) {
        float x[PER];
        if constexpr (PER == 4) {
            const float4 y = *reinterpret_cast<const float4*>(src);
            x[0] = y.x, x[1] = y.y, x[2] = y.z, x[3] = y.w;
        } else {
            const float2 y = *reinterpret_cast<const float2*>(src);
            x[0] = y.x, x[1] = y.y;
        }
        join_add(top, l, acc, ml.x, ml.y, x);
    };
    if (live)
        join_each<kJoinGroups>(k, g, [&](int64_t place) {
            add(*reinterpret_cast<const float2*>(p.part_ml + (place * RM + r) * 2),
                p.part_o + (place * RM + r) * D + lane * PER);
        });
#pragma unroll
    for (int i = 0; i < PER; ++i) s_x[j][g][lane * PER + i] = acc[i];
    if (lane == 0) s_ml[j][g] = make_float2(top, l);
    __syncthreads();
    if (g != 0 || !live) return;
#pragma unroll
    for (int o = 1; o < kJoinGroups; ++o) add(s_ml[j][o], &s_x[j][o][lane * PER]);
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

// results by columns: a warp has kJoinCols columns of 32 rows; a block CG such sets
constexpr int kJoinCols = 16;
template <int D, int RM>
struct JoinCfg {
    static constexpr int PG = RM == 128 ? 4 : 1;  // units of 128 rows have long axes
    static constexpr int CG = PG == 4 ? 2 : D / kJoinCols;
    static constexpr int kThreads = 32 * PG * CG;
    static constexpr int kBlocks = (RM / 32) * (D / (CG * kJoinCols));
};
template <typename T, int D, int RM>
__global__ void __launch_bounds__(JoinCfg<D, RM>::kThreads)
    attend_join_columns_kernel(const __grid_constant__ AttendArgs p) {
    using C = JoinCfg<D, RM>;
    __shared__ float s_x[C::PG][C::CG][kJoinCols][32];
    __shared__ float2 s_ml[C::PG][C::CG][32];
    Cut k;
    if (!join_unit(p, k)) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = warp % C::PG, cg = warp / C::PG;
    const int r = blockIdx.y % (RM / 32) * 32 + lane;
    const int c0 = (blockIdx.y / (RM / 32) * C::CG + cg) * kJoinCols;
    const bool live = r < k.n * p.group - k.rt * RM;
    float top = -INFINITY, l = 0.0f, acc[kJoinCols];
#pragma unroll
    for (int i = 0; i < kJoinCols; ++i) acc[i] = 0.0f;
    if (live)
        join_each<C::PG>(k, g, [&](int64_t place) {
            const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + (place * RM + r) * 2);
            float x[kJoinCols];
#pragma unroll
            for (int i = 0; i < kJoinCols; ++i) x[i] = p.part_o[(place * D + c0 + i) * RM + r];
            join_add(top, l, acc, ml.x, ml.y, x);
        });
    if constexpr (C::PG > 1) {
#pragma unroll
        for (int i = 0; i < kJoinCols; ++i) s_x[g][cg][i][lane] = acc[i];
        s_ml[g][cg][lane] = make_float2(top, l);
        __syncthreads();
        if (g != 0) return;
#pragma unroll
        for (int o = 1; o < C::PG; ++o) {
            float x[kJoinCols];
#pragma unroll
            for (int i = 0; i < kJoinCols; ++i) x[i] = s_x[o][cg][i][lane];
            join_add(top, l, acc, s_ml[o][cg][lane].x, s_ml[o][cg][lane].y, x);
        }
    }
    if (!live) return;
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
    constexpr int bytes = RowsCfg<D, MT>::kSmem;
    CUtensorMap km, vm;
    if (!encode_pages(&km, &vm, p, kBlk, D / 64)) return cudaErrorInvalidValue;
    static std::atomic<uint64_t> ready{0};  // devices whose kernel has its shared memory
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(ready.load() >> dev & 1)) {
        e = cudaFuncSetAttribute(attend_rows_kernel<T, D, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready.fetch_or(1ull << dev);
    }
    return launch_early(attend_rows_kernel<T, D, MT>, dim3((unsigned)p.ctas), dim3(kAThreads), bytes, s, p, km, vm);
}
template <typename T, int D, int RM>
cudaError_t launch_join(const AttendArgs& p, cudaStream_t s) {
    if constexpr (RM >= 128) {
        using C = JoinCfg<D, RM>;
        return launch_early(attend_join_columns_kernel<T, D, RM>, dim3((unsigned)p.ctas, C::kBlocks), dim3(C::kThreads), 0,
                            s, p);
    } else {
        return launch_early(attend_join_kernel<T, D, RM>, dim3((unsigned)p.ctas, RM / kJoinRows),
                            dim3(32 * kJoinRows * kJoinGroups), 0, s, p);
    }
}

template <typename T, int D>
cudaError_t rows_of(int mt, const AttendArgs& p, cudaStream_t s) {
    return mt == 1 ? launch_rows<T, D, 1>(p, s) : launch_rows<T, D, 2>(p, s);
}
template <typename T, int D>
cudaError_t join_of(int rm, const AttendArgs& p, cudaStream_t s) {
    return rm == 16 ? launch_join<T, D, 16>(p, s) : rm == 32 ? launch_join<T, D, 32>(p, s)
         : rm == 128 ? launch_join<T, D, 128>(p, s) : launch_join<T, D, 256>(p, s);
}

}  // namespace

cudaError_t launch_attend_rows(int dtype, int dim, int mt, const AttendArgs& p, cudaStream_t s) {
    if (dtype == SV_BF16)
        return dim == 64 ? rows_of<__nv_bfloat16, 64>(mt, p, s) : rows_of<__nv_bfloat16, 128>(mt, p, s);
    return dim == 64 ? rows_of<__half, 64>(mt, p, s) : rows_of<__half, 128>(mt, p, s);
}

cudaError_t launch_attend_join(int dtype, int dim, int rm, const AttendArgs& p, cudaStream_t s) {
    if (dtype == SV_BF16)
        return dim == 64 ? join_of<__nv_bfloat16, 64>(rm, p, s) : join_of<__nv_bfloat16, 128>(rm, p, s);
    return dim == 64 ? join_of<__half, 64>(rm, p, s) : join_of<__half, 128>(rm, p, s);
}

}  // namespace sv
