// sv_attend_tiles.cu -- attention of many query rows a cache head: chunks of a prompt, and
// rounds whose group fills a tile.
//
// Here the products bound the call, so they run on the tensor cores' own memory
// (tcgen05): a unit is 256 query rows, two tiles of 128 that share every key tile of 128
// keys.  Twelve warps, one job each:
//   warps 0-3, 4-7  the softmax of one row tile each, a thread a row: scores from tensor
//                   memory, weights to shared memory, output rows at the end; and the
//                   queries of the next unit, fetched behind the last scores of this one
//   warps 8, 10     issue the products of one row tile each: S = Q K^T and O += P V, operands
//                   in shared memory
//   warp 9          loads keys and values by TMA, page by page, into a ring
// The scores are read by the time half of the weights are there; then the next S is issued,
// so that it is done when the softmax ends, and the output's product needs the tensor cores
// only while the next softmax looks for its maximum.  The output stays in tensor memory
// over all keys; the running maximum it refers to is only raised when a row's scores
// outgrow it by 2^8, so that rescaling the output is rare.  Weights of up to 2^8 lose
// nothing in the 16-bit types' relative step (fp16: see kLift), and sums are 32-bit.
//
// Up to 128 rows (SPLIT) the loads bound the call, and the room goes to the ring: the
// weights lie over their scores in tensor memory, and warp 11 loads the queries, a unit
// ahead of the products: 3900 cycles for 128 rows of 128, where a unit of one key tile
// takes more than 10000 (128 sequences x 8 tokens behind 100, 64 / 8 heads: seven units a CTA,
// 47 us).
//
// Pages become boxes of gcd(page_size, 128) keys x 64 elements.  A box with no visible
// key, or on a bad page, is loaded from past the last page, where TMA gives zeros: its
// scores are masked, and its values add nothing.  Rows of a box past the sequence's end
// are zeroed in shared memory before their product, since they may hold anything.
//
// Two chunks of 2048 tokens behind 4-6k keys (32 / 8 heads of 128, bf16): 305-308 us, 1300
// TFLOP/s, 0.68 of the measured rate.  What bounds it is the softmax: some 2900 cycles for
// two tiles of 128 x 128 (2600 with heads of 64), of which the exponential unit fills 1024
// and the tiles' products 2080; it waits for nothing else.  The start and the units' ends
// are a tenth.  Tried and slower: weights over the scores for these units too (337 us: the
// next S waits for the output's product), room for the weights of 64 keys and one more stage
// (308 us, and 403 with the next S ahead of the output's product), two threads a row (451: the
// output's product then stands between one softmax and the next), and before that steps of
// 64 keys (365 us of then 331) and registers moved from the other warps to the softmax (340: the warps
// that issue products then spill).
//
// Every wait has a limit.  When one runs out, the CTA writes NaN for what is left of its
// part, sets SV_ROW_INTERNAL, lets its copies and products finish (with a limit) and ends.
#include <atomic>
#include <type_traits>

#include "sv_async.cuh"
#include "sv_attend.cuh"

namespace sv {
namespace {

constexpr int kTThreads = 384;
constexpr int kBadSlots = 16;  // units that the loader can be ahead by, and more

template <int D, bool SPLIT>
struct TilesCfg {
    static constexpr int kTileBytes = kKeyTile * D * 2;
    static constexpr int kQBytes = 256 * D * 2;
    static constexpr int kWBytes = SPLIT ? 0 : 2 * 128 * kKeyTile * 2;  // weights of the two tiles
    static constexpr int kStages = D == 64 ? 8 : SPLIT ? 5 : 3;
    static constexpr int kHalves = D / 64;                // 128-byte columns of a tile
    static constexpr int kHalfBytes = kKeyTile * 128;     // 128 rows of one
    static constexpr int kSmem = kQBytes + kWBytes + kStages * kTileBytes + 1024;  // and room to align
    // tensor memory columns: scores (SPLIT: and weights) of the two tiles, then their outputs
    static constexpr int kS = 0, kO = 256;
};

struct TilesArgs {
    AttendArgs p;
    int box;  // keys of a box
};

// ---- tensor memory and products -------------------------------------------
// Descriptors of swizzled operands in shared memory, groups of 8 rows (1024 bytes) apart:
// the low word has the address (in 16 bytes) and, for values, which are read across
// (64 contiguous elements of N, then the next block of 64), the distance of the blocks.
// The high word is the same for all.
constexpr uint32_t kDescHigh = 64u | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_keys(uint32_t addr) { return (addr >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_values(uint32_t addr, uint32_t block_bytes) {
    return (addr >> 4) | ((block_bytes >> 4) << 16);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n.reg .pred p;\n.reg .b64 da, db;\nsetp.ne.u32 p, %5, 0;\nmov.b64 da, {%1, %4};\nmov.b64 db, {%2, %4};\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(kDescHigh), "r"((uint32_t)add)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n.reg .pred p;\n.reg .b64 db;\nsetp.ne.u32 p, %5, 0;\nmov.b64 db, {%2, %4};\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(kDescHigh), "r"((uint32_t)add)
        : "memory");
}
// one lane of the warp, the same each time; the products are issued from code that the
// compiler can see to be uniform (descriptors in uniform registers)
__device__ __forceinline__ bool elect() {
    uint32_t one;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xFFFFFFFF;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
    return one;
}
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xFFFFFFFFu, x, 0); }
// (a warp that gives up says so before it arrives anywhere)
__device__ __forceinline__ bool none_gave_up(volatile int* dead) { return !__any_sync(0xFFFFFFFFu, *dead); }
// two 32-bit operations in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n.reg .b64 a, b, c, d;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nmov.b64 c, {%6, %7};\n"
        "fma.rn.f32x2 d, a, b, c;\nmov.b64 {%0, %1}, d;\n}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n.reg .b64 a, b, d;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nadd.rn.f32x2 d, a, b;\n"
        "mov.b64 {%0, %1}, d;\n}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ void mma_commit(uint64_t* b) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(b))
                 : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

#define SV_R8(a, i) "=r"(a[i]), "=r"(a[i + 1]), "=r"(a[i + 2]), "=r"(a[i + 3]), "=r"(a[i + 4]), "=r"(a[i + 5]), \
                    "=r"(a[i + 6]), "=r"(a[i + 7])
#define SV_RW8(a, i) "+r"(a[i]), "+r"(a[i + 1]), "+r"(a[i + 2]), "+r"(a[i + 3]), "+r"(a[i + 4]), "+r"(a[i + 5]), \
                     "+r"(a[i + 6]), "+r"(a[i + 7])
#define SV_I8(a, i) "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3]), "r"(a[i + 4]), "r"(a[i + 5]), \
                    "r"(a[i + 6]), "r"(a[i + 7])
// 16 columns of the thread's row; the values are there when this returns
__device__ __forceinline__ void tmem_load16(uint32_t addr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : SV_R8(r, 0), SV_R8(r, 8)
        : "r"(addr)
        : "memory");
}
// 64 columns, not waited for
__device__ __forceinline__ void tmem_start64(uint32_t addr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];"
        : SV_R8(r, 0), SV_R8(r, 8), SV_R8(r, 16), SV_R8(r, 24), SV_R8(r, 32), SV_R8(r, 40), SV_R8(r, 48), SV_R8(r, 56)
        : "r"(addr)
        : "memory");
}
// waits for the loads so far; the registers pass through it, so that nothing reads them before
__device__ __forceinline__ void tmem_wait64(uint32_t* r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : SV_RW8(r, 0), SV_RW8(r, 8), SV_RW8(r, 16), SV_RW8(r, 24), SV_RW8(r, 32), SV_RW8(r, 40), SV_RW8(r, 48),
                   SV_RW8(r, 56)::"memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            addr),
        SV_I8(r, 0), SV_I8(r, 8)
        : "memory");
}
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// the instruction descriptor: fp32 results, T operands, n columns, B read across its rows
// (values) or along them (keys), 128 rows
template <typename T>
__device__ constexpr uint32_t idesc(int n, bool b_across) {
    const uint32_t f = sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
    return (1u << 4) | (f << 7) | (f << 10) | (b_across ? 1u << 16 : 0u) | ((uint32_t)(n / 8) << 17) | (8u << 24);
}

// SPLIT: a unit is one tile of 128 rows, and the two halves of the CTA take its key tiles
// in turn, each with its own maximum, sum and output; the first half joins them.
template <typename T, int D, bool SPLIT>
__global__ void __launch_bounds__(kTThreads, 1)
    attend_tiles_kernel(const __grid_constant__ TilesArgs ta, const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap) {
    using C = TilesCfg<D, SPLIT>;
    constexpr int RM = SPLIT ? 128 : 256;
    constexpr int STEP = SPLIT ? 2 : 1;  // key tiles from one of a half's to the next
    const AttendArgs& p = ta.p;
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint64_t s_full[C::kStages], s_empty[C::kStages];  // ring of key and value tiles
    __shared__ uint64_t s_q[2], s_scores[2], s_weights[2][2], s_out[2];  // per half (weights: in two parts)
    __shared__ uint64_t s_q_free[2];  // per place of the queries
    __shared__ uint64_t s_last, s_second, s_joined;
    __shared__ float2 s_ml[SPLIT ? 128 : 1];  // the second half's maximum and sum
    __shared__ uint32_t s_tmem;
    __shared__ int s_dead;
    __shared__ int s_bad[kBadSlots];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    grid_dependents_go();
    // swizzled tiles start on 1024-byte boundaries
    const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
    unsigned char* smem_p = smem_raw + (smem - smem_u32(smem_raw));
    const uint32_t q_s = smem, w_s = smem + C::kQBytes, ring_s = w_s + C::kWBytes;
    if (t == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            bar_init(&s_full[s], 1);
            bar_init(&s_empty[s], 2);  // both halves, whether or not they read the stage
        }
        for (int x = 0; x < 2; ++x) {
            bar_init(&s_q[x], SPLIT ? 1 : 128);
            bar_init(&s_q_free[x], 2);
            bar_init(&s_scores[x], 1);
            bar_init(&s_weights[x][0], 128);
            bar_init(&s_weights[x][1], 128);
            bar_init(&s_out[x], 1);
        }
        bar_init(&s_last, 2);
        bar_init(&s_second, 128);
        bar_init(&s_joined, 128);
        s_dead = 0;
        for (int i = 0; i < kBadSlots; ++i) s_bad[i] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
    }
    grid_dependency_wait();
    // (tensor memory is taken only now: the kernel before this one may need it to end)
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fill_idle_rows<T, D, kTThreads>(p);
    Part part;
    find_part<RM, kTThreads>(p, part, reinterpret_cast<int*>(smem_p));
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = s_tmem;
    volatile int* dead = &s_dead;
    const unsigned long long limit = p.wait_ns;

    if (part.todo == 0) {
        // nothing to do
    } else if (warp < 8) {
        // ---------------------------------------------------------------- softmax
        const int x = warp >> 2;              // half of the CTA
        const int row = t & 127;              // row of its tile
        const int x0 = SPLIT ? 0 : x * 128;   // the tile's first row in the unit
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + C::kS + x * 128 + lanes, tO = tmem + C::kO + x * D + lanes;
        Unit u = part.u;
        int first = part.tile, left = part.todo, index = 0;
        uint32_t n_scores = 0, n_out = 0;  // phases seen
        bool alive = true;
        // !SPLIT: the warp's 32 query rows of a unit, into shared memory as the products read them.  (There is one
        // place for them: one warp for all 256 rows took 5000 cycles a half between two units; here a unit's rows
        // come while its predecessor ends.)
        bool q_there = false;
        auto load_q = [&](const Unit& w) {
            constexpr int RC = D / 8, RS = 32 / RC;  // 16-byte pieces of a row, rows a step
            const int c = lane % RC, r0 = (warp & 3) * 32, count = w.n * p.group;
            const uint32_t dst = q_s + x * 128 * D * 2 + (c >> 3) * C::kHalfBytes;
#pragma unroll 4
            for (int i = r0 + lane / RC; i < r0 + 32; i += RS) {  // (rows past the last are computed and dropped)
                const T* src = q_row<T>(p, w.b, w.h, min(w.rt * RM + x0 + i, count - 1)) + c * 8;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + i * 128 + (((c & 7) ^ (i & 7)) << 4)),
                             "l"(src)
                             : "memory");
            }
            q_there = true;
        };
        auto hand_q = [&]() {
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_async_smem();
            bar_arrive(&s_q[x]);
        };

        while (left > 0) {
            const int rows = u.n * p.group, r = u.rt * RM + x0 + row;
            const int end = min(u.t1, first + left);
            const bool whole = first == u.t0 && end == u.t1;
            left -= end - first;
            Unit next = u;
            bool ahead = false;  // next is the next unit
            if (SPLIT || u.rt * RM + x0 < rows) {  // the tile has rows
                if (!SPLIT && !q_there) {
                    load_q(u);
                    hand_q();
                }
                q_there = false;
                const int start = first + (SPLIT ? x : 0);
                const int pos = u.past + by_group(p, min(r, rows - 1));
                // of the warp's rows: the least and the greatest position; or there is none
                const int wr0 = r - lane;
                const int pos0 = u.past + by_group(p, min(wr0, rows - 1));
                const int pos1 = u.past + by_group(p, min(wr0 + 31, rows - 1));
                float ref = -INFINITY, sum = 0.0f;
                // The first half has to be through with what the second left of the unit before.
                // Warps that gave up a wait still arrive, here and on s_second, for every unit that
                // is left, so after these two waits a warp looks whether one has: a phase of theirs
                // alone may be over before the others have done their part of it.
                if (SPLIT && x == 1 && index > 0)
                    alive = alive && bar_wait(&s_joined, (index - 1) & 1, limit, dead) && none_gave_up(dead);
                for (int tile = start; alive && tile < end; tile += STEP) {
                    alive = bar_wait(&s_scores[x], n_scores & 1, limit, dead);
                    if (!alive) break;
                    ++n_scores;
                    fence_after();
                    if (!SPLIT && tile + 1 == end && left > 0) {  // the unit's last scores: its queries are read
                        next_unit<RM>(p, next);
                        ahead = true;
                        if (next.rt * RM + x0 < next.n * p.group) load_q(next);
                    }
                    if (wr0 >= rows) {  // no rows: their lanes' products go nowhere
                        // (not SPLIT: these scores can be there before the others' weights of the
                        // tile before, whose phase this warp must not enter twice)
                        if (!SPLIT && tile != start) alive = bar_wait(&s_out[x], n_out++ & 1, limit, dead);
                        fence_before();
                        bar_arrive(&s_weights[x][0]);
                        bar_arrive(&s_weights[x][1]);
                        continue;
                    }
                    // The scores of 128 keys, as two halves.  The second is read for the maximum, and
                    // again when the first has become weights: held through, it costs spills.
                    float s0[64], s1[64];
                    uint32_t *w0 = reinterpret_cast<uint32_t*>(s0), *w1 = reinterpret_cast<uint32_t*>(s1);
                    tmem_start64(tS + 64, w1);
                    tmem_start64(tS, w0);
                    tmem_wait64(w1);
                    tmem_wait64(w0);
                    const int k0 = tile * kKeyTile;
                    const bool cut = k0 + kKeyTile - 1 > pos0 || (p.a.window > 0 && k0 <= (int64_t)pos1 - p.a.window);
                    // visible: keys [seen0, seen1] of the tile
                    const int seen0 = p.a.window > 0 ? (int)max((int64_t)pos - p.a.window + 1 - k0, (int64_t)0) : 0;
                    const int seen1 = pos - k0;
                    if (cut) {
#pragma unroll
                        for (int j = 0; j < 64; ++j) {
                            if (j < seen0 || j > seen1) s0[j] = -INFINITY;
                            if (j + 64 < seen0 || j + 64 > seen1) s1[j] = -INFINITY;
                        }
                    }
                    float top[4] = {s0[0], s0[1], s1[0], s1[1]};
#pragma unroll
                    for (int j = 2; j < 62; j += 4) {
                        top[0] = max3(top[0], s0[j], s0[j + 1]);
                        top[1] = max3(top[1], s0[j + 2], s0[j + 3]);
                        top[2] = max3(top[2], s1[j], s1[j + 1]);
                        top[3] = max3(top[3], s1[j + 2], s1[j + 3]);
                    }
                    top[0] = max3(top[0], s0[62], s0[63]);
                    top[2] = max3(top[2], s1[62], s1[63]);
                    const float m = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * p.qscale;
                    // The product before this one has read its weights.  (SPLIT: it is through when these
                    // scores are there, for their commit covers what its thread issued before; s_out
                    // has one phase a unit.)
                    if (!SPLIT && tile != start) {
                        alive = bar_wait(&s_out[x], n_out++ & 1, limit, dead);
                        if (!alive) break;
                        fence_after();
                    }
                    if (tile == start) {
                        ref = m;
                    } else if (__any_sync(0xFFFFFFFFu, m > ref + 8.0f)) {
                        // raise the reference; the output so far shrinks by as much
                        const float now = fmaxf(ref, m);
                        const float f = now == -INFINITY ? 1.0f : fast_exp2(ref - now);
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) {
                            float o[16];
                            tmem_load16(tO + c, reinterpret_cast<uint32_t*>(o));
#pragma unroll
                            for (int j = 0; j < 16; ++j) o[j] *= f;
                            tmem_store16(tO + c, reinterpret_cast<const uint32_t*>(o));
                        }
                        if (!SPLIT) tmem_store_wait();
                        sum *= f;
                        ref = now;
                    }
                    const float base = weight_base<T>(ref);
                    const float2 qs = make_float2(p.qscale, p.qscale), mb = make_float2(-base, -base);
                    float2 add[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
                    auto weigh = [&](const float* v, int c) {  // 32 keys, the c-th such set of the tile
                        uint32_t w[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            float2 e = fma2(make_float2(v[2 * j], v[2 * j + 1]), qs, mb);
                            e.x = fast_exp2(e.x);
                            e.y = fast_exp2(e.y);
                            add[j & 1] = add2(add[j & 1], e);
                            w[j] = Pair<T>::pack(e.x, e.y);  // 16 bits into the product, as the values
                        }
                        if constexpr (SPLIT) {
                            tmem_store16(tS + c * 16, w);
                        } else {
                            unsigned char* dst =
                                smem_p + C::kQBytes + x * (C::kWBytes / 2) + (c >> 1) * (128 * 128) + row * 128;
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                *reinterpret_cast<uint4*>(dst + ((((c & 1) * 4 + j) ^ (row & 7)) << 4)) =
                                    make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
                        }
                    };
                    auto handed = [&](uint64_t* bar) {  // the weights so far are where their product reads them
                        if constexpr (SPLIT)
                            tmem_store_wait();
                        else
                            fence_async_smem();
                        fence_before();
                        bar_arrive(bar);
                    };
                    weigh(s0, 0);
                    tmem_start64(tS + 64, w1);
                    weigh(s0 + 32, 1);
                    tmem_wait64(w1);
                    handed(&s_weights[x][0]);  // their product can start, and the scores may be written over
                    if (cut) {
#pragma unroll
                        for (int j = 0; j < 64; ++j)
                            if (j + 64 < seen0 || j + 64 > seen1) s1[j] = -INFINITY;
                    }
                    weigh(s1, 2);
                    weigh(s1 + 32, 3);
                    handed(&s_weights[x][1]);
                    add[0] = add2(add[0], add[1]);
                    sum += add[0].x + add[0].y;
                }
                if (q_there) hand_q();
                if (left > 0 && !ahead) next_unit<RM>(p, next);
                if (alive && start < end) alive = bar_wait(&s_out[x], n_out++ & 1, limit, dead);
                if (SPLIT && x == 1) {
                    if (alive) s_ml[row] = make_float2(ref, sum);  // (else the unit before may be read from it yet)
                    fence_before();
                    bar_arrive(&s_second);
                } else {
                    float f0 = 1.0f, f1 = 0.0f;  // of the two halves' outputs
                    if (SPLIT) {
                        alive = alive && bar_wait(&s_second, index & 1, limit, dead) && none_gave_up(dead);
                        if (alive) {
                            const float2 ml = s_ml[row];
                            const float now = fmaxf(ref, ml.x);
                            f0 = ref == -INFINITY ? 0.0f : fast_exp2(ref - now);
                            f1 = ml.x == -INFINITY ? 0.0f : fast_exp2(ml.x - now);
                            ref = now;
                            sum = sum * f0 + ml.y * f1;
                        }
                    }
                    fence_after();
                    const bool bad = !alive || s_bad[index % kBadSlots];
                    const int place = 2 * blockIdx.x + (index == 0 ? 0 : 1);
                    // partial results lie by columns, so that a warp's stores are whole lines
                    float* part_o = p.part_o + (int64_t)place * RM * D + x0 + row;
                    const float l = bad ? NAN : sum;
                    const float inv = 1.0f / l;
                    T* dst = r < rows ? out_row<T>(p, u.b, u.h, r) : nullptr;
                    if (!whole && r < rows)
                        *reinterpret_cast<float2*>(p.part_ml + ((int64_t)place * RM + x0 + row) * 2) =
                            make_float2(alive ? ref : -INFINITY, l);
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        float o[16];
                        __syncwarp();  // tensor memory is read by whole warps
                        if (alive) {
                            tmem_load16(tO + c, reinterpret_cast<uint32_t*>(o));
                            if (SPLIT) {
                                if (end - first > 1) {
                                    float o1[16];
                                    tmem_load16(tO + D + c, reinterpret_cast<uint32_t*>(o1));
#pragma unroll
                                    for (int j = 0; j < 16; ++j) o[j] = o[j] * f0 + o1[j] * f1;
                                }
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < 16; ++j) o[j] = 0.0f;
                        }
                        if (r < rows) {
                            if (whole) {
#pragma unroll
                                for (int j = 0; j < 16; j += 8)
                                    *reinterpret_cast<uint4*>(dst + c + j) =
                                        make_uint4(Pair<T>::pack(o[j] * inv, o[j + 1] * inv),
                                                   Pair<T>::pack(o[j + 2] * inv, o[j + 3] * inv),
                                                   Pair<T>::pack(o[j + 4] * inv, o[j + 5] * inv),
                                                   Pair<T>::pack(o[j + 6] * inv, o[j + 7] * inv));
                            } else {
#pragma unroll
                                for (int j = 0; j < 16; ++j) part_o[(int64_t)(c + j) * RM] = o[j];
                            }
                        }
                    }
                    fence_before();
                    if (SPLIT) bar_arrive(&s_joined);
                }
            } else if (left > 0) {
                next_unit<RM>(p, next);
            }
            if (!alive && lane == 0 && p.a.row_status) atomicOr(p.a.row_status + u.b, SV_ROW_INTERNAL);
            u = next;
            first = u.t0;
            ++index;
        }
    } else {
        if (warp == 8 || warp == 10) {
            // ------------------------------------------------------------ products
            // of one half each.  (One warp for both left the tensor cores idle between its
            // batches: they take in only a few products ahead, and each hand-over costs a
            // few hundred cycles.)
            constexpr uint32_t i_s = idesc<T>(kKeyTile, false), i_o = idesc<T>(D, true);
            const int x = uniform(warp == 8 ? 0 : 1);
            Unit u = part.u;
            int first = part.tile, left = part.todo, index = 0;
            // Places of the ring, counted through: keys and values of one tile, then the next.
            // Every half waits for every place in order and gives it back, read or not: a
            // phase parity only tells a barrier's last two phases apart, so that a half that
            // skipped the other's places could run a lap ahead of them and pass too early.
            uint32_t at = 0, stage = 0, turn = 0;
            uint32_t n_w = 0, n_q = 0;
            bool alive = true;
            const uint32_t tS = uniform(tmem) + C::kS + x * 128, tO = uniform(tmem) + C::kO + x * D;
            auto next_place = [&]() {
                ++at;
                if (++stage == C::kStages) {
                    stage = 0;
                    turn ^= 1;
                }
            };
            // waits up to place i; gives back those before it
            auto reach = [&](uint32_t i) -> bool {
                while (at != i) {
                    if (!bar_wait(&s_full[stage], turn, limit, dead)) return false;
                    if (lane == 0) bar_arrive(&s_empty[stage]);
                    next_place();
                }
                return bar_wait(&s_full[stage], turn, limit, dead);
            };
            // S of the keys in the place that was reached; the unit's last frees its queries' place
            auto scores = [&](uint32_t q_desc, bool last, int place) {
                const uint32_t b = uniform(desc_keys(ring_s + stage * C::kTileBytes));
                fence_after();
                if (elect()) {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t off = ((k / 4) * C::kHalfBytes + (k % 4) * 32) >> 4;
                        mma_ss(tS, q_desc + off, b + off, i_s, k > 0);
                    }
                    mma_commit(&s_scores[x]);
                    mma_commit(&s_empty[stage]);
                    if (SPLIT && last) mma_commit(&s_q_free[place]);
                }
                __syncwarp();
                next_place();
            };
            while (alive && left > 0) {
                const int end = min(u.t1, first + left);
                const uint32_t last = at + 2 * (end - first);  // the place after the unit's
                const int q_place = SPLIT ? index & 1 : x;
                if (SPLIT || u.rt * RM + x * 128 < u.n * p.group) {
                    const int start = first + (SPLIT ? x : 0);
                    int lo, hi;
                    tile_keys<RM>(p, u.past, u.n, u.rt, lo, hi);
                    const int vend = u.past + u.n;
                    const uint32_t q_desc = uniform(desc_keys(q_s + q_place * 128 * D * 2));
                    uint32_t i = at + 2 * (start - first);
                    // SPLIT: a half waits for the queries of every unit, also of one whose single
                    // tile is the other's, and frees their place only then.  So nobody frees a place
                    // twice while the other half has yet to read it, and nobody is a phase of s_q
                    // ahead: a parity only tells a barrier's last two phases apart.  The place is
                    // written again when both have freed it, so the unit's count gives the phase.
                    alive = bar_wait(&s_q[q_place], (SPLIT ? index >> 1 : (int)n_q++) & 1, limit, dead);
                    if (start < end) {
                        alive = alive && reach(i);
                        if (alive) scores(q_desc, start + STEP >= end, q_place);
                    } else if (SPLIT && alive && lane == 0) {
                        bar_arrive(&s_q_free[q_place]);
                    }
                    for (int tile = start; alive && tile < end; tile += STEP, i += 2 * STEP) {
                        const bool more = tile + STEP < end;
                        if (!SPLIT) {
                            // the next scores, as soon as these are read: they are there when the
                            // softmax ends
                            if (more) alive = bar_wait(&s_full[stage], turn, limit, dead);
                            alive = alive && bar_wait(&s_weights[x][0], n_w & 1, limit, dead);
                            if (alive && more) scores(q_desc, tile + 2 >= end, q_place);
                            alive = alive && bar_wait(&s_full[stage], turn, limit, dead);
                        } else {
                            alive = reach(i + 1);
                        }
                        if (!alive) break;
                        const uint32_t vstage = stage, vs = ring_s + stage * C::kTileBytes;
                        next_place();
                        // rows of a box outside the visible keys: what they hold times 0 must be
                        // 0 (both tiles' warps write these zeros, each before its product)
                        const int k0 = tile * kKeyTile;
                        if (k0 < lo || k0 + kKeyTile > vend) {
                            const int z0 = max(0, min(kKeyTile, lo - k0)), z1 = max(0, min(kKeyTile, vend - k0));
                            const int from = z0 & ~(ta.box - 1), to = (z1 + ta.box - 1) & ~(ta.box - 1);
                            constexpr int RC = D / 8;  // 16-byte pieces of a row
                            for (int j = lane; j < (z0 - from + to - z1) * RC; j += 32) {
                                const int zr = j / RC, c = j % RC;
                                const int rr = zr < z0 - from ? from + zr : z1 + zr - (z0 - from);
                                *reinterpret_cast<uint4*>(smem_p + (vs - smem) + (c / 8) * C::kHalfBytes + rr * 128 +
                                                          ((c & 7) << 4)) = make_uint4(0, 0, 0, 0);
                            }
                            fence_async_smem();
                            __syncwarp();
                        }
                        const uint32_t v_desc = uniform(desc_values(vs, C::kHalfBytes));
                        const uint32_t w_desc = uniform(desc_keys(w_s + x * (C::kWBytes / 2)));
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            if (SPLIT || half) alive = alive && bar_wait(&s_weights[x][half], n_w & 1, limit, dead);
                            if (!alive) break;
                            fence_after();
                            if (elect()) {
#pragma unroll
                                for (int k = half * 4; k < half * 4 + 4; ++k) {
                                    const uint32_t b = v_desc + k * (16 * 128 >> 4);
                                    const bool add = tile > start || k > 0;
                                    if constexpr (SPLIT)
                                        mma_ts(tO, tS + k * 8, b, i_o, add);
                                    else
                                        mma_ss(tO, w_desc + (((k / 4) * (128 * 128) + (k % 4) * 32) >> 4), b, i_o, add);
                                }
                                if (half) {
                                    if (!SPLIT || !more) mma_commit(&s_out[x]);
                                    mma_commit(&s_empty[vstage]);
                                }
                            }
                            __syncwarp();
                        }
                        if (!alive) break;
                        ++n_w;
                        if (SPLIT && more) {
                            alive = reach(i + 2 * STEP);
                            if (alive) scores(q_desc, tile + 2 * STEP >= end, q_place);
                        }
                    }
                }
                while (alive && at != last) {  // what is left of the unit is the other half's
                    alive = bar_wait(&s_full[stage], turn, limit, dead);
                    if (alive && lane == 0) bar_arrive(&s_empty[stage]);
                    if (alive) next_place();
                }
                left -= end - first;
                ++index;
                if (alive && left > 0) {
                    next_unit<RM>(p, u);
                    first = u.t0;
                }
            }
            // products still in flight end before tensor memory is given back
            if (elect()) mma_commit(&s_last);
            __syncwarp();
            const unsigned long long t0 = now_ns();
            while (!bar_try(&s_last, 0) && now_ns() - t0 < kWaitLimitNs) {}
        } else if (warp == 9) {
            // ------------------------------------------------------------ loads
            Unit u = part.u;
            int tile = part.tile, left = part.todo, index = 0;
            uint32_t stage = 0, turn = 0;
            const int per = kKeyTile / ta.box;
            const bool loads = lane < per * C::kHalves;
            const int box = lane / C::kHalves, half = lane % C::kHalves;
            const int no_page = (int)p.a.cache.pages;  // past the last: zeros
            bool alive = true;
            int issued = 0;
            auto put = [&](const CUtensorMap* map, int h, int page, int in_page) {
                alive = alive && bar_wait(&s_empty[stage], turn ^ 1, limit, dead);
                if (!alive) return;
                if (lane == 0) bar_expect(&s_full[stage], C::kTileBytes);
                __syncwarp();
                if (loads)
                    tma_part(ring_s + stage * C::kTileBytes + half * C::kHalfBytes + box * ta.box * 128, map, half,
                             in_page, h, page, &s_full[stage]);
                ++issued;
                if (++stage == C::kStages) {
                    stage = 0;
                    turn ^= 1;
                }
            };
            // the lane's box of a tile: page id (bad and invisible ones: no_page)
            auto find = [&](const Unit& w, int tl, int& page, int& in_page) -> bool {
                int lo, hi;
                tile_keys<RM>(p, w.past, w.n, w.rt, lo, hi);
                const int k = tl * kKeyTile + box * ta.box;
                page = no_page;
                in_page = 0;
                if (!loads || k > hi || k + ta.box <= lo) return false;
                const int i = page_of(p, k);
                page = p.a.cache.page_table[w.b * p.a.cache.page_table_stride + i];
                in_page = k - i * (int)p.a.cache.page_size;
                if (page < 0 || page >= no_page) {
                    page = no_page;
                    return true;
                }
                return false;
            };
            auto mark = [&](bool bad) {  // a tile with a bad page
                if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) {
                    *(volatile int*)&s_bad[index % kBadSlots] = 1;
                    if (p.a.row_status) atomicOr(p.a.row_status + u.b, SV_ROW_BAD_PAGE);
                    __threadfence_block();
                }
            };
            int page, in_page;
            bool bad = find(u, tile, page, in_page);
            while (alive && left > 0) {
                const int end = min(u.t1, tile + left);
                left -= end - tile;
                if (lane == 0) s_bad[index % kBadSlots] = 0;
                __syncwarp();
                Unit next = u;
                if (left > 0) next_unit<RM>(p, next);
                // the next tiles' pages are looked up while this one's copies run
                int page1 = no_page, in_page1 = 0;
                bool bad1 = false;
                if (!SPLIT) {  // keys are one tile ahead of the values
                    mark(bad);
                    put(&kmap, u.h, page, in_page);
                    if (tile + 1 < end) bad1 = find(u, tile + 1, page1, in_page1);
                }
                for (; alive && tile < end; ++tile) {
                    int page2 = no_page, in_page2 = 0;
                    bool bad2 = false;
                    if (!SPLIT && tile + 1 < end) {
                        mark(bad1);
                        put(&kmap, u.h, page1, in_page1);
                    }
                    if (SPLIT) {
                        mark(bad);
                        put(&kmap, u.h, page, in_page);
                    }
                    const int ahead = tile + (SPLIT ? 1 : 2);
                    if (ahead < end)
                        bad2 = find(u, ahead, page2, in_page2);
                    else if (left > 0 && tile + 1 == end)
                        bad2 = find(next, next.t0, page2, in_page2);
                    put(&vmap, u.h, page, in_page);
                    if (!SPLIT && tile + 1 < end) {
                        page = page1, in_page = in_page1;
                        page1 = page2, in_page1 = in_page2, bad1 = bad2;
                    } else {
                        page = page2, in_page = in_page2, bad = bad2;
                    }
                }
                ++index;
                u = next;
                tile = u.t0;
            }
            // copies still in flight end before the CTA does (whoever gave up)
            const unsigned long long t0 = now_ns();
            const int n = min(issued, C::kStages);
            for (int i = 0; i < n; ++i) {
                stage = stage == 0 ? C::kStages - 1 : stage - 1;
                if (stage == C::kStages - 1) turn ^= 1;
                while (!bar_try(&s_full[stage], turn) && now_ns() - t0 < kWaitLimitNs) {}
            }
        } else if (SPLIT) {
            // ---------------------------------------------------------- queries
            // A unit's 128 rows into shared memory, swizzled as the products read them, in two
            // places in turn.  A place is free when the last scores of what it held are through.
            Unit u = part.u;
            int first = part.tile, left = part.todo, index = 0;
            uint32_t n_free[2] = {0, 0};
            bool alive = true;
            constexpr int RC = D / 8, RS = 32 / RC;  // 16-byte pieces of a row, rows a step
            const int c = lane % RC, sub = lane / RC;
            while (alive && left > 0) {
                const int rows = u.n * p.group;
                const int r0 = u.rt * RM, place = index & 1;
                if (n_free[place]++ > 0) alive = bar_wait(&s_q_free[place], n_free[place] & 1, limit, dead);
                if (!alive) break;
                const uint32_t dst = q_s + place * 128 * D * 2 + (c >> 3) * C::kHalfBytes;
#pragma unroll 4
                for (int i = sub; i < 128; i += RS) {  // (rows past the last are computed and dropped)
                    const T* src = q_row<T>(p, u.b, u.h, min(r0 + i, rows - 1)) + c * 8;
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                     dst + i * 128 + (((c & 7) ^ (i & 7)) << 4)),
                                 "l"(src)
                                 : "memory");
                }
                asm volatile("cp.async.wait_all;" ::: "memory");
                fence_async_smem();
                __syncwarp();
                if (lane == 0) bar_arrive(&s_q[place]);
                const int end = min(u.t1, first + left);
                left -= end - first;
                ++index;
                if (left > 0) {
                    next_unit<RM>(p, u);
                    first = u.t0;
                }
            }
        }
    }
    __syncthreads();
    if (warp == 8) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

template <typename T, int D, bool SPLIT>
cudaError_t launch_tiles(const AttendArgs& p, cudaStream_t s) {
    constexpr int bytes = TilesCfg<D, SPLIT>::kSmem;
    TilesArgs ta;
    ta.p = p;
    ta.box = 16;
    while (ta.box < kKeyTile && p.a.cache.page_size % (2 * ta.box) == 0) ta.box *= 2;
    CUtensorMap km, vm;
    if (!encode_pages(&km, &vm, p, ta.box, 1)) return cudaErrorInvalidValue;
    // once a device: room in shared memory
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(ready.load() >> dev & 1)) {
        e = cudaFuncSetAttribute(attend_tiles_kernel<T, D, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready.fetch_or(1ull << dev);
    }
    return launch_early(attend_tiles_kernel<T, D, SPLIT>, dim3((unsigned)p.ctas), dim3(kTThreads), bytes, s, ta, km, vm);
}

template <typename T>
cudaError_t tiles_of(int dim, int rm, const AttendArgs& p, cudaStream_t s) {
    if (rm == 128) return dim == 64 ? launch_tiles<T, 64, true>(p, s) : launch_tiles<T, 128, true>(p, s);
    return dim == 64 ? launch_tiles<T, 64, false>(p, s) : launch_tiles<T, 128, false>(p, s);
}

}  // namespace

cudaError_t launch_attend_tiles(int dtype, int dim, int rm, const AttendArgs& p, cudaStream_t s) {
    return dtype == SV_BF16 ? tiles_of<__nv_bfloat16>(dim, rm, p, s) : tiles_of<__half>(dim, rm, p, s);
}

}  // namespace sv
