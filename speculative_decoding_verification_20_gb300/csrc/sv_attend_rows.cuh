// sv_attend_rows.cuh -- attention of a few query rows a cache head over a long cache:
// single tokens and verification rounds.
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
// Over a cache held in 8 bits (E8) a block is 32 keys, as many bytes.  Codes become fp16 on the
// way from shared memory to the products, which is exact.  A matrix load gives a lane four
// neighbouring codes of a key, where the product of 16 elements wants two and two: queries lie
// in shared memory with their elements in that order.  Of values a lane gets two neighbouring
// codes of two keys: even and odd columns of 16 become a product each.  The keys' scales
// multiply the scores; the values' scales multiply the weights, relative to the largest met so
// far (vref), which is raised as the maximum is.  The call above then takes 226 us, 2.9 TB/s: a
// block takes a warp some 700 instructions, and both warps of a group convert the same codes.
//
// Scores and outputs use the warp-wide 16x8x16 matrix instructions: 16 rows of them are
// what a decode step fills.
#pragma once

#include <atomic>
#include <type_traits>

#include "sv_async.cuh"
#include "sv_attend.cuh"

namespace sv {
namespace {

constexpr int kAWarps = 12;  // that compute
constexpr int kLoaders = 3;  // warps that load; up to 16 in all, four a scheduler, leave 128 registers a thread
constexpr int kACompute = 32 * kAWarps;
constexpr int kAThreads = kACompute + 32 * kLoaders;
constexpr int kLook = 16;  // keys whose page (and scale) is looked up at once

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
    return (uint32_t)((c >> 3) * (16 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}
// E8: rows of D codes, swizzled likewise
template <int D>
__device__ __forceinline__ uint32_t code_at(int r, int c) {
    return (uint32_t)(r * D + ((c ^ (D == 64 ? r >> 1 & 3 : r & 7)) << 4));
}
// query rows of D elements, swizzled likewise
template <int D>
__device__ __forceinline__ uint32_t q_at(int r, int c) {
    return (uint32_t)(r * (D * 2) + ((c ^ (r & 7)) << 4));
}
__device__ __forceinline__ void compute_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kACompute) : "memory"); }

template <int D, int MT, bool E8>
struct RowsCfg {
    static constexpr int kBlk = E8 ? 32 : 16;             // keys of a block
    static constexpr int kTileBlks = kKeyTile / kBlk;
    static constexpr int kHalfBytes = 16 * D * 2;         // a block's keys, or its values
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
template <typename T, int D, int MT, bool SINKS, bool E8>
__global__ void __launch_bounds__(kAThreads, 1)
    attend_rows_kernel(const __grid_constant__ AttendArgs p, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap) {
    using C = RowsCfg<D, MT, E8>;
    using P = typename std::conditional<E8, __half, T>::type;  // of the products
    constexpr int kBlk = C::kBlk, kTileBlks = C::kTileBlks;
    constexpr int RM = 16 * MT;
    constexpr int GROUPS = kAWarps / MT;
    constexpr int CH = D / 8;  // 16-byte chunks of a row
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint64_t s_full[C::kStages], s_empty[C::kStages];
    __shared__ uint8_t s_bad[C::kStages];  // the block in the stage lies on a bad page
    __shared__ int s_dead;
    __shared__ float s_m[GROUPS][RM], s_l[GROUPS][RM];  // per group: reference and sum
    __shared__ float2 s_ml[RM];                         // of all
    __shared__ float s_ks[E8 ? C::kStages : 1][2], s_vs[E8 ? C::kStages : 1][2];  // E8: scales of the block's halves
    __shared__ float s_qf[E8 ? RM : 1];                                          // what a row's scores are multiplied by
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
    find_part<RM, kAThreads, SINKS>(p, part, reinterpret_cast<int*>(s_join));
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
            constexpr int kLooks = kBlk / kLook, kAhead = 32 / kLooks;  // look-ups a block, blocks in one go
            for (int b0 = tile * kTileBlks; alive && b0 < end * kTileBlks; b0 += kAhead) {
                // a lane a look-up: its page, and the row of it (no visible key: -1, bad: -2)
                const int blk = b0 + lane / kLooks;
                const int k0 = blk * kBlk + lane % kLooks * kLook - (SINKS && blk < u.w0 * kTileBlks ? u.t0 * kKeyTile : 0);
                int page = -1, in_page = 0;
                float ks = 1.0f, vs = 0.0f;
                if (blk < end * kTileBlks && any_visible<SINKS>(p, k0, kLook, lo, hi)) {
                    const int i = page_of(p, k0);
                    page = pages[i];
                    in_page = k0 - i * (int)p.a.cache.page_size;
                    if (page < 0 || page >= p.a.cache.pages) {
                        page = -2;
                        if (p.a.row_status) atomicOr(p.a.row_status + u.b, SV_ROW_BAD_PAGE);
                    } else if (E8) {
                        ks = key_scale(p, u.h, page, in_page);
                        vs = value_scale(p, u.h, page, in_page);
                    }
                }
                const uint32_t n = min(kAhead, end * kTileBlks - b0);
                for (uint32_t i = (mine + kLoaders - seq % kLoaders) % kLoaders; i < n; i += kLoaders) {
                    // E8: lanes 0 and 1 (of values: 2 and 3) have the block's two look-ups
                    const int from = E8 ? 2 * i + (lane & 1) : i;
                    const int pg = __shfl_sync(0xFFFFFFFFu, page, from), at = __shfl_sync(0xFFFFFFFFu, in_page, from);
                    const uint32_t stage = (seq + i) % C::kStages;
                    alive = bar_wait(&s_empty[stage], ((seq + i) / C::kStages & 1u) ^ 1u, limit, dead);
                    if (!alive) break;
                    if constexpr (E8) {
                        const float fk = __shfl_sync(0xFFFFFFFFu, ks, from), fv = __shfl_sync(0xFFFFFFFFu, vs, from);
                        const uint32_t bad = __ballot_sync(0xFFFFFFFFu, pg == -2) & 3u;
                        const uint32_t there = __ballot_sync(0xFFFFFFFFu, pg >= 0) & 3u;
                        if (lane < 2) {
                            s_ks[stage][lane] = fk;
                            s_vs[stage][lane] = fv;
                        }
                        __syncwarp();
                        if (lane == 0) {
                            s_bad[stage] = bad != 0;
                            if (there)
                                bar_expect(&s_full[stage], __popc(there) * 2 * kLook * D);
                            else
                                bar_arrive(&s_full[stage]);
                        }
                        __syncwarp();
                        if (pg >= 0 && lane < 4)
                            tma_codes(ring_s + stage * C::kBlkBytes + (lane >> 1) * C::kHalfBytes + (lane & 1) * kLook * D,
                                      lane >> 1 ? &vmap : &kmap, at, u.h, pg, &s_full[stage]);
                    } else {
                        if (lane == 0) {
                            s_bad[stage] = pg == -2;
                            if (pg >= 0)
                                bar_expect(&s_full[stage], C::kBlkBytes);
                            else
                                bar_arrive(&s_full[stage]);
                        }
                        __syncwarp();
                        if (pg >= 0 && lane < 2)
                            tma_box(ring_s + stage * C::kBlkBytes + lane * C::kHalfBytes, lane ? &vmap : &kmap, at, u.h,
                                    pg, &s_full[stage]);
                    }
                    done = seq + i + 1;
                }
                seq += n;
            }
            left -= end - tile;
            if (left > 0) {
                next_unit<RM, SINKS>(p, u);
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
                if constexpr (E8) {
                    // a row's pieces lie in CH neighbouring lanes
                    uint32_t w[4] = {qv[i].x, qv[i].y, qv[i].z, qv[i].w};
                    if constexpr (!std::is_same<T, __half>::value) {
                        float2 f[4];
                        float top = 0.0f;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            f[j] = Pair<T>::unpack(x < RM * CH ? w[j] : 0u);
                            if (isfinite(f[j].x)) top = fmaxf(top, fabsf(f[j].x));
                            if (isfinite(f[j].y)) top = fmaxf(top, fabsf(f[j].y));
                        }
#pragma unroll
                        for (int o = 1; o < CH; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                        const int lift = row_lift(top);
                        const float up = __int_as_float(lift);
#pragma unroll
                        for (int j = 0; j < 4; ++j) w[j] = Pair<__half>::pack(f[j].x * up, f[j].y * up);
                        if (x < RM * CH && x % CH == 0) s_qf[x / CH] = p.qscale * __int_as_float((254 << 23) - lift);
                    } else if (x < RM * CH && x % CH == 0) {
                        s_qf[x / CH] = p.qscale;
                    }
                    // elements 4 j, 4 j + 1 of 16 first, then 4 j + 2, 4 j + 3
                    if (x < RM * CH) {
                        const int r = x / CH, c = x % CH & ~1, odd = x % CH & 1;
                        *reinterpret_cast<uint2*>(s_q + q_at<D>(r, c) + odd * 8) = make_uint2(w[0], w[2]);
                        *reinterpret_cast<uint2*>(s_q + q_at<D>(r, c + 1) + odd * 8) = make_uint2(w[1], w[3]);
                    }
                } else {
                    if (x < RM * CH) *reinterpret_cast<uint4*>(s_q + q_at<D>(x / CH, x % CH)) = qv[i];
                }
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
            float vref = E8 ? kLeastScale : 1.0f, vinv = 1.0f / vref;
            const float qf[2] = {E8 ? s_qf[r0] : p.qscale, E8 ? s_qf[r0 + 8] : p.qscale};
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
                const int blk = tile * kTileBlks + (int)i;
                const int k0 = blk * kBlk - (SINKS && blk < u.w0 * kTileBlks ? u.t0 * kKeyTile : 0);
                const bool bad = s_bad[stage];
                poisoned |= bad;
                if (!bad && m * 16 < rows && any_visible<SINKS>(p, k0, kBlk, lo, hi)) {
                    const uint32_t ks = ring_s + stage * C::kBlkBytes, vs = ks + C::kHalfBytes;
                    // values at positions that no row sees may be anything, and 0 * NaN is NaN
                    // (each warp of the group writes these zeros, before it reads)
                    // valid rows of the block: [vlo, vhi), and the sinks below vsink
                    const int vlo = lo - k0, vhi = hi + 1 - k0, vsink = sinks_of<SINKS>(p) - k0;
                    if (vlo > 0 || vhi < kBlk) {
                        constexpr int PC = E8 ? D / 16 : CH;  // 16-byte pieces of a row
                        for (int x = lane; x < kBlk * PC; x += 32) {
                            const int r = x / PC;
                            if ((r < vlo && (!SINKS || r >= vsink)) || r >= vhi)
                                *reinterpret_cast<uint4*>(ring + stage * C::kBlkBytes + C::kHalfBytes +
                                                          (E8 ? code_at<D>(r, x % PC) : blk_at(r, x % PC))) =
                                    make_uint4(0, 0, 0, 0);
                        }
                        fence_async_smem();
                        __syncwarp();
                    }
                    constexpr int NT = kBlk / 8;  // scores of 8 keys each
                    float s[NT][4];
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[n][e] = 0.0f;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        uint32_t qf4[4], kf[4];
                        ldsm4(qf4, q_s + q_at<D>(m * 16 + (lane & 15), 2 * k + (lane >> 4)));
                        if constexpr (E8) {  // 16 codes of keys 0..7, 8..15, 16..23, 24..31
                            ldsm4(kf, ks + code_at<D>(lane, k));
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                uint32_t b0, b1;
                                codes_half(kf[n], b0, b1);
                                mma16816<P>(s[n], qf4, b0, b1);
                            }
                        } else {  // keys 0..7: (k lo, k hi), keys 8..15: (k lo, k hi)
                            ldsm4(kf, ks + blk_at((lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)));
                            mma16816<P>(s[0], qf4, kf[0], kf[1]);
                            mma16816<P>(s[1], qf4, kf[2], kf[3]);
                        }
                    }
                    const bool all = k0 + kBlk - 1 <= pos_first &&
                                     (p.a.window <= 0 || k0 > (int64_t)hi - p.a.window ||
                                      (SINKS && k0 + kBlk <= p.sinks));
                    if (!all) {
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int j = k0 + n * 8 + q4 * 2 + (e & 1), at = pos[e >> 1];
                                if (j > at || (p.a.window > 0 && j <= at - p.a.window && (!SINKS || j >= p.sinks)))
                                    s[n][e] = -INFINITY;
                            }
                    }
                    // what scores are multiplied by (E8: by halves of the block)
                    float qk[2][NT / 2], vw[NT / 2];
#pragma unroll
                    for (int y = 0; y < NT / 2; ++y) {
                        if constexpr (E8) vw[y] = s_vs[stage][y];
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            qk[e][y] = E8 ? score_factor(qf[e], s_ks[stage][y]) : p.qscale;
                    }
                    float top[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float v = -INFINITY;
#pragma unroll
                        for (int y = 0; y < NT / 2; ++y) {
                            const float w = fmaxf(fmaxf(s[2 * y][2 * e], s[2 * y][2 * e + 1]),
                                                  fmaxf(s[2 * y + 1][2 * e], s[2 * y + 1][2 * e + 1]));
                            v = E8 ? fmaxf(v, w * qk[e][y]) : w;
                        }
                        v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 1));
                        v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 2));
                        top[e] = E8 ? v : v * p.qscale;
                    }
                    // the reference of the weights is only raised when a row outgrows it by 2^8
                    bool raise = top[0] > ref[0] + 8.0f || top[1] > ref[1] + 8.0f;
                    float vtop = vref;
                    if constexpr (E8) {
                        vtop = fmaxf(vref, fmaxf(vw[0], vw[1]));
                        raise |= vtop > vref;
                    }
                    if (__any_sync(0xFFFFFFFFu, raise)) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float now = fmaxf(ref[e], top[e]);
                            float f = now == -INFINITY ? 1.0f : fast_exp2(ref[e] - now);
                            ref[e] = now;
                            sum[e] *= f;
                            if constexpr (E8) f *= vref / vtop;
#pragma unroll
                            for (int d = 0; d < D / 8; ++d) {
                                o[d][2 * e] *= f;
                                o[d][2 * e + 1] *= f;
                            }
                        }
                        if (E8 && vtop > vref) {
                            vref = vtop;
                            vinv = 1.0f / vtop;
                        }
                    }
                    if constexpr (E8) {
                        vw[0] *= vinv;
                        vw[1] *= vinv;
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float base = weight_base<P>(ref[e]);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int f = 0; f < 2; ++f) {
                                const float w = fast_exp2(fmaf(s[n][2 * e + f], qk[e][n / 2], -base));
                                s[n][2 * e + f] = E8 ? w * vw[n / 2] : w;
                                sum[e] += w;
                            }
                    }
                    // weights enter the product in 16 bits, as the values do
                    uint32_t pf[NT / 2][4];
#pragma unroll
                    for (int y = 0; y < NT / 2; ++y) {
                        pf[y][0] = Pair<P>::pack(s[2 * y][0], s[2 * y][1]), pf[y][1] = Pair<P>::pack(s[2 * y][2], s[2 * y][3]);
                        pf[y][2] = Pair<P>::pack(s[2 * y + 1][0], s[2 * y + 1][1]);
                        pf[y][3] = Pair<P>::pack(s[2 * y + 1][2], s[2 * y + 1][3]);
                    }
#pragma unroll
                    for (int d = 0; d < D / 16; ++d) {
                        uint32_t vf[4];
                        if constexpr (E8) {
                            // columns 2 g, 2 g + 1 of keys 2 q4, 2 q4 + 1 (of eight): by columns, then to fp16
                            ldsm4t(vf, vs + code_at<D>(lane, d));
                            uint32_t even[4], odd[4];
#pragma unroll
                            for (int x = 0; x < 4; ++x) codes_half(__byte_perm(vf[x], 0, 0x3120), even[x], odd[x]);
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                mma16816<P>(o[2 * d], pf[y], even[2 * y], even[2 * y + 1]);
                                mma16816<P>(o[2 * d + 1], pf[y], odd[2 * y], odd[2 * y + 1]);
                            }
                        } else {
                            ldsm4t(vf, vs + blk_at((lane & 7) + (((lane >> 3) & 1) << 3), 2 * d + (lane >> 4)));
                            mma16816<P>(o[2 * d], pf[0], vf[0], vf[1]);
                            mma16816<P>(o[2 * d + 1], pf[0], vf[2], vf[3]);
                        }
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
                next_unit<RM, SINKS>(p, next);
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
                if constexpr (E8) f[e] *= vref;
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
                if constexpr (E8) {  // even and odd columns of 16: a lane has four neighbours
#pragma unroll
                    for (int d = 0; d < C::kJoinCols / 16; ++d) {
                        float* j0 = s_join + (warp * 16 + g) * C::kJoinCols + ((d * 16 + q4 * 4) ^ ((g & 3) << 3));
                        const int dd = c0 / 8 + 2 * d;
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            *reinterpret_cast<float4*>(j0 + e * 8 * C::kJoinCols) =
                                make_float4(o[dd][2 * e] * f[e], o[dd + 1][2 * e] * f[e], o[dd][2 * e + 1] * f[e],
                                            o[dd + 1][2 * e + 1] * f[e]);
                    }
                } else {
#pragma unroll
                    for (int d = 0; d < C::kJoinCols / 8; ++d) {
                        float* j0 = s_join + (warp * 16 + g) * C::kJoinCols + ((d * 8 + q4 * 2) ^ ((g & 3) << 3));
                        float* j1 = j0 + 8 * C::kJoinCols;
                        const int dd = c0 / 8 + d;
                        *reinterpret_cast<float2*>(j0) = make_float2(o[dd][0] * f[0], o[dd][1] * f[0]);
                        *reinterpret_cast<float2*>(j1) = make_float2(o[dd][2] * f[1], o[dd][3] * f[1]);
                    }
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

template <typename T, int D, int MT, bool SINKS, bool E8>
cudaError_t launch_rows(const AttendArgs& p, cudaStream_t s) {
    constexpr int bytes = RowsCfg<D, MT, E8>::kSmem;
    CUtensorMap km, vm;
    if (!(E8 ? encode_codes(&km, &vm, p, kLook) : encode_pages(&km, &vm, p, kLook, D / 64))) return cudaErrorInvalidValue;
    static std::atomic<uint64_t> ready{0};  // devices whose kernel has its shared memory
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(ready.load() >> dev & 1)) {
        e = cudaFuncSetAttribute(attend_rows_kernel<T, D, MT, SINKS, E8>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready.fetch_or(1ull << dev);
    }
    return launch_early(attend_rows_kernel<T, D, MT, SINKS, E8>, dim3((unsigned)p.ctas), dim3(kAThreads), bytes, s, p, km, vm);
}
template <typename T, int D, bool SINKS, bool E8>
cudaError_t rows_of(int mt, const AttendArgs& p, cudaStream_t s) {
    return mt == 1 ? launch_rows<T, D, 1, SINKS, E8>(p, s) : launch_rows<T, D, 2, SINKS, E8>(p, s);
}
template <bool SINKS, bool E8>
cudaError_t rows_of_type(int dtype, int dim, int mt, const AttendArgs& p, cudaStream_t s) {
    if (dtype == SV_BF16)
        return dim == 64 ? rows_of<__nv_bfloat16, 64, SINKS, E8>(mt, p, s) : rows_of<__nv_bfloat16, 128, SINKS, E8>(mt, p, s);
    return dim == 64 ? rows_of<__half, 64, SINKS, E8>(mt, p, s) : rows_of<__half, 128, SINKS, E8>(mt, p, s);
}

}  // namespace
}  // namespace sv
