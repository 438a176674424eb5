// sv_attend.cuh -- how the attention kernels share out a batch among their CTAs.
//
// The work is a list of units (sequence, cache head, tile of RM query rows), each a run
// of tiles of kKeyTile keys.  Query rows of one cache head are its group's heads of
// every new token, token-major: row r is token r / group, head r % group of the group,
// so that one read of a key serves all of them.  The list, flattened to key tiles, is cut
// into equal parts, one per CTA, whatever the lengths; a unit that is cut gets one partial
// result from each CTA that works on it (running maximum, sum and unnormalised output),
// and the join kernel adds them in order.  A CTA has at most two such units, its first
// and its last, so the partials need two places a CTA.
//
// With a window, the first `sinks` positions stay visible.  A unit's key tiles are then
// those that hold them and, apart from these, those of the window; the tiles are numbered
// through, so that the division knows nothing of the gap: key_tile() gives a number's place.
// Kernels without sinks are compiled apart (SINKS false): the few instructions more cost a
// prompt's chunk 13% (307 to 350 us), since its softmax has no register and no issue slot to
// spare, and a round of 64 sequences 6%.
#pragma once

#include <cuda.h>

#include <type_traits>
#include <utility>

#include "sv_internal.cuh"
#include "sv_paged.cuh"

namespace sv {

constexpr int kKeyTile = 128;  // keys a CTA takes per step
constexpr int kMaxCtas = 152;  // one CTA per SM; also sizes the workspace

// a CTA's first unit and its place in the list
struct Cut {
    long long base, end;  // the unit's tiles of the list
    long long per;        // tiles a CTA; the first `more` CTAs have one tile more
    int more, ctas;       // CTAs with work (0: this one has none)
    int b, h, rt, n;
};

struct AttendArgs {
    sv_attention_args a;
    int group;           // query heads per cache head
    uint32_t group_inv;  // 2^32 / group, rounded up (0: group is 1)
    int page_shift;      // log2 of page_size, or -1
    int max_row_tiles;   // row tiles of a sequence with all N new tokens
    float qscale;        // scale * log2(e): scores are kept as powers of two
    int sinks;           // first positions that the window does not hide (0 without a window)
    int sink_tiles;      // key tiles that hold them
    sv_cache_scales sc;  // of a cache held in 8 bits (k: null for 16 bits)
    int ctas;            // CTAs that share the work (at most kMaxCtas)
    int64_t capacity;    // positions that the page table addresses
    unsigned long long wait_ns;  // limit of a wait
    Cut* cut;            // [ctas] each CTA's first unit, for the join
    float* part_o;       // [2 * ctas][RM][dim]
    float* part_ml;      // [2 * ctas][RM][2] running maximum (in log2 units) and sum
};
// r / group by a product: exact for r < 2^26 and groups up to 64, since the error of
// group_inv, below group / 2^32 relative to it, then stays below 1 / group
constexpr int64_t kMaxRows = 1 << 26;

#ifdef __CUDACC__

// a unit, and its key tiles [t0, t1): those below w0 are the sinks', the first of the row
struct Unit {
    int b, h, rt;
    int past, n;
    int t0, t1, w0;
};
// the place in the sequence of a unit's key tile
template <bool SINKS>
__device__ __forceinline__ int key_tile(const Unit& u, int tile) {
    return SINKS && tile < u.w0 ? tile - u.t0 : tile;
}
// the first positions that a window leaves in sight
template <bool SINKS>
__device__ __forceinline__ int sinks_of(const AttendArgs& p) {
    return SINKS ? p.sinks : 0;
}

__device__ __forceinline__ int by_group(const AttendArgs& p, int r) {
    return p.group_inv ? (int)__umulhi((uint32_t)r, p.group_inv) : r;
}
__device__ __forceinline__ int page_of(const AttendArgs& p, int key) {
    return p.page_shift >= 0 ? key >> p.page_shift : key / (int)p.a.cache.page_size;
}
// the visible keys [lo, hi] of a tile of rows, and the sinks below lo
template <int RM>
__device__ __forceinline__ void tile_keys(const AttendArgs& p, int past, int n, int rt, int& lo, int& hi) {
    const int r0 = rt * RM, r1 = min(r0 + RM, n * p.group) - 1;
    lo = p.a.window > 0 ? (int)max((int64_t)0, past + by_group(p, r0) + 1 - p.a.window) : 0;
    hi = past + by_group(p, r1);
}
template <int RM, bool SINKS>
__device__ __forceinline__ int tile_count(const AttendArgs& p, int past, int n, int rt) {
    int lo, hi;
    tile_keys<RM>(p, past, n, rt, lo, hi);
    return hi / kKeyTile + 1 - lo / kKeyTile + (SINKS ? min(p.sink_tiles, lo / kKeyTile) : 0);
}
template <int RM, bool SINKS>
__device__ __forceinline__ void unit_tiles(const AttendArgs& p, Unit& u) {
    int lo, hi;
    tile_keys<RM>(p, u.past, u.n, u.rt, lo, hi);
    u.w0 = lo / kKeyTile;
    u.t0 = SINKS ? u.w0 - min(p.sink_tiles, u.w0) : u.w0;
    u.t1 = hi / kKeyTile + 1;
}
// whether any row of the tile sees one of `len` keys from k0 on
template <bool SINKS>
__device__ __forceinline__ bool any_visible(const AttendArgs& p, int k0, int len, int lo, int hi) {
    return k0 <= hi && (k0 + len > lo || (SINKS && k0 < p.sinks));
}
template <int RM>
__device__ __forceinline__ int row_tiles(const AttendArgs& p, int n) {
    return (n * p.group + RM - 1) / RM;
}

// The CTA's part of the list: its first unit, the tile in it to begin with, and how
// many tiles to do in all.  Every thread of the CTA calls this and gets the same
// answer, and the first unit is left for the join.  s_tiles: NT words of shared memory.
struct Part {
    int todo;
    int tile;  // in u
    Unit u;
};
template <int RM, int NT, bool SINKS>
__device__ void find_part(const AttendArgs& p, Part& part, int* s_tiles) {
    __shared__ long long s_warp[NT / 32];
    __shared__ long long s_before;
    __shared__ int s_seq;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, B = (int)p.a.B, c = blockIdx.x;
    const int Hkv = (int)p.a.kv_heads;
    // key tiles of one head of sequence b, by a thread alone or by a warp
    auto alone = [&](const SeqLens s) -> int {
        int n = 0;
        for (int rt = row_tiles<RM>(p, s.n); rt-- > 0;) n += tile_count<RM, SINKS>(p, s.past, s.n, rt);
        return n;
    };
    auto by_warp = [&](const SeqLens s) -> int {
        int n = 0;
        for (int rt = lane; rt < row_tiles<RM>(p, s.n); rt += 32) n += tile_count<RM, SINKS>(p, s.past, s.n, rt);
        return warp_sum(n);
    };
    auto lens = [&](int b) -> SeqLens { return seq_lens(p.a.cache, b, (int)p.a.N, p.capacity); };
    auto scan = [&](long long own) -> long long {  // inclusive, over the warp
        long long x = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if (lane >= o) x += y;
        }
        return x;
    };
    // the CTA's share of `total` tiles
    long long begin = 0, per = 0;
    int more = 0, ctas = 0;
    auto share = [&](long long total) -> bool {
        ctas = total < p.ctas ? (int)total : p.ctas;
        part.todo = 0;
        if (c >= ctas) {
            if (t == 0) p.cut[c].ctas = 0;
            return false;
        }
        per = total >> 31 ? total / ctas : (long long)((uint32_t)total / (uint32_t)ctas);
        more = (int)(total - per * ctas);
        begin = per * c + min(c, more);
        part.todo = (int)per + (c < more ? 1 : 0);
        return true;
    };
    int seq = 0, per_head = 0;
    long long before_seq = 0;
    const bool many_rows = p.max_row_tiles > 4;
    SeqLens s;  // of the first unit's sequence
    if (many_rows ? B * ((p.max_row_tiles + 31) / 32) <= 16 : B <= 32) {
        // a small batch: every warp by itself, with no barrier
        // (a lane a sequence: the lengths of all come in one wait)
        const SeqLens held = lens(min(lane, B - 1));
        auto of = [&](int b) -> SeqLens {
            SeqLens x = held;
            x.past = __shfl_sync(0xFFFFFFFFu, held.past, b);
            x.n = __shfl_sync(0xFFFFFFFFu, held.n, b);
            return x;
        };
        int mine = 0;
        if (many_rows) {
            for (int b = 0; b < B; ++b) {
                const int n = by_warp(of(b));
                if (lane == b) mine = n;
            }
        } else {
            mine = alone(held);  // by every lane: the warp stays together for the scan
            if (lane >= B) mine = 0;
        }
        __syncwarp();
        const long long own = (long long)mine * Hkv, upto = scan(own);
        if (!share(__shfl_sync(0xFFFFFFFFu, upto, 31))) return;
        seq = __ffs(__ballot_sync(0xFFFFFFFFu, upto > begin)) - 1;
        before_seq = __shfl_sync(0xFFFFFFFFu, upto - own, seq);
        per_head = __shfl_sync(0xFFFFFFFFu, mine, seq);
        s = of(seq);
    } else {
        auto head_tiles = [&](int b0) -> int {  // of sequence b0 + t
            if (!many_rows) return b0 + t < B ? alone(lens(b0 + t)) : 0;
            __syncthreads();
            for (int i = warp; i < NT && b0 + i < B; i += NT / 32) {
                const int n = by_warp(lens(b0 + i));
                if (lane == 0) s_tiles[i] = n;
            }
            __syncthreads();
            return b0 + t < B ? s_tiles[t] : 0;
        };
        long long total = 0;
        int mine = 0;
        for (int b0 = 0; b0 < B; b0 += NT) {
            mine = head_tiles(b0);
            total += (long long)mine * Hkv;
        }
        total = warp_sum(total);
        if (lane == 0) s_warp[warp] = total;
        __syncthreads();
        total = 0;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) total += s_warp[w];
        __syncthreads();
        if (!share(total)) return;
        long long base = 0;
        for (int b0 = 0; b0 < B; b0 += NT) {
            if (B > NT) mine = head_tiles(b0);
            const long long own = (long long)mine * Hkv, x = scan(own);
            if (lane == 31) s_warp[warp] = x;
            __syncthreads();
            long long before = base + x - own;
            for (int w = 0; w < warp; ++w) before += s_warp[w];
            if (begin >= before && begin < before + own) {
                s_seq = b0 + t;
                s_before = before;
                s_tiles[0] = mine;
            }
            for (int w = 0; w < NT / 32; ++w) base += s_warp[w];
            __syncthreads();
            if (base > begin) break;
        }
        seq = s_seq;
        before_seq = s_before;
        per_head = s_tiles[0];
        s = lens(seq);
    }
    // then the head and the row tile
    Unit& u = part.u;
    u.b = seq;
    u.past = s.past;
    u.n = s.n;
    const long long off = begin - before_seq;
    u.h = off >> 31 ? (int)(off / per_head) : (int)((uint32_t)off / (uint32_t)per_head);
    int at = (int)(off - (long long)u.h * per_head);
    for (int rt0 = 0;; rt0 += 32) {  // (at < per_head: a row tile holds it)
        const int n = rt0 + lane < row_tiles<RM>(p, s.n) ? tile_count<RM, SINKS>(p, s.past, s.n, rt0 + lane) : 0;
        int x = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if (lane >= o) x += y;
        }
        const unsigned past_it = __ballot_sync(0xFFFFFFFFu, x > at);
        if (past_it) {
            const int l = __ffs(past_it) - 1;
            u.rt = rt0 + l;
            at -= __shfl_sync(0xFFFFFFFFu, x - n, l);
            break;
        }
        at -= __shfl_sync(0xFFFFFFFFu, x, 31);
        if (rt0 + 32 >= row_tiles<RM>(p, s.n)) break;
    }
    unit_tiles<RM, SINKS>(p, u);
    part.tile = u.t0 + at;
    if (t == 0) p.cut[c] = Cut{begin - at, begin - at + (u.t1 - u.t0), per, more, ctas, u.b, u.h, u.rt, u.n};
}

// the unit after u (there is one: the caller counts tiles)
template <int RM, bool SINKS>
__device__ __forceinline__ void next_unit(const AttendArgs& p, Unit& u) {
    if (++u.rt == row_tiles<RM>(p, u.n)) {
        u.rt = 0;
        if (++u.h == p.a.kv_heads) {
            u.h = 0;
            do {
                ++u.b;
                const SeqLens s = seq_lens(p.a.cache, u.b, (int)p.a.N, p.capacity);
                u.past = s.past;
                u.n = s.n;
            } while (u.n == 0 && u.b + 1 < p.a.B);
        }
    }
    unit_tiles<RM, SINKS>(p, u);
}

// Rows that no unit covers: zeros past a sequence's new tokens, NaN for a sequence whose
// lengths are bad.  A sequence's rows are shared by the CTAs c, c + B, ..., a warp a token.
template <typename T, int D, int NT>
__device__ void fill_idle_rows(const AttendArgs& p) {
    constexpr int VECS = D / 8;
    const int B = (int)p.a.B, ctas = (int)gridDim.x, lane = threadIdx.x & 31;
    const int parts = max(1, ctas / B), part = (int)blockIdx.x / B;
    if (part >= parts) return;
    for (int b = (int)blockIdx.x % B; b < B; b += ctas) {
        const SeqLens s = seq_lens(p.a.cache, b, (int)p.a.N, p.capacity);
        if (s.bad && part == 0 && threadIdx.x == 0 && p.a.row_status)
            atomicOr(p.a.row_status + b, SV_ROW_BAD_LENGTH);
        const uint32_t w = s.bad ? Pair<T>::pack(NAN, NAN) : 0u;
        for (int i = s.n + part * (NT / 32) + (int)threadIdx.x / 32; i < p.a.N; i += parts * (NT / 32)) {
            T* o = (T*)p.a.out + (int64_t)b * p.a.o_stride_b + (int64_t)i * p.a.o_stride_n;
            for (int x = lane; x < (int)p.a.q_heads * VECS; x += 32)
                *reinterpret_cast<uint4*>(o + (int64_t)(x / VECS) * p.a.o_stride_h + x % VECS * 8) =
                    make_uint4(w, w, w, w);
        }
    }
}

template <typename T>
__device__ __forceinline__ T* out_row(const AttendArgs& p, int b, int h, int r) {
    const int i = by_group(p, r);
    return (T*)p.a.out + (int64_t)b * p.a.o_stride_b + (int64_t)i * p.a.o_stride_n +
           (int64_t)(h * p.group + r - i * p.group) * p.a.o_stride_h;
}
template <typename T>
__device__ __forceinline__ const T* q_row(const AttendArgs& p, int b, int h, int r) {
    const int i = by_group(p, r);
    return (const T*)p.a.q + (int64_t)b * p.a.q_stride_b + (int64_t)i * p.a.q_stride_n +
           (int64_t)(h * p.group + r - i * p.group) * p.a.q_stride_h;
}

// Weights are 2^(score - reference + lift): at most 2^8, times 2^7 in fp16.  Its steps become
// coarse below 2^-14 and end at 2^-24, and the many small weights of a long row beside a large
// one add up: without the lift 16000 weights of 2^-25.2 came to nothing in the product with
// the values while their sum had them.  A weight is off by at most 2^-11 of itself or
// by 2^-32 of the row's largest.  The factor falls out of output / sum.
template <typename T>
constexpr float kLift = std::is_same<T, __half>::value ? 7.0f : 0.0f;
// what a row's scores are reduced by (nothing visible yet: weights 0)
template <typename T>
__device__ __forceinline__ float weight_base(float ref) {
    return ref == -INFINITY ? 0.0f : ref - kLift<T>;
}

// Cache held in 8 bits.  Four codes as two pairs in fp16 (exact):
__device__ __forceinline__ void codes_half(uint32_t w, uint32_t& b0, uint32_t& b1) {
    asm("{\n.reg .b16 lo, hi;\nmov.b32 {lo, hi}, %2;\ncvt.rn.f16x2.e4m3x2 %0, lo;\ncvt.rn.f16x2.e4m3x2 %1, hi;\n}\n"
        : "=r"(b0), "=r"(b1)
        : "r"(w));
}
// the scales of a block of positions:
__device__ __forceinline__ float key_scale(const AttendArgs& p, int h, int page, int in_page) {
    return p.sc.k[page * p.sc.k_stride_page + h * p.sc.k_stride_head + in_page / SV_SCALE_BLOCK];
}
__device__ __forceinline__ float value_scale(const AttendArgs& p, int h, int page, int in_page) {
    return p.sc.v[page * p.sc.v_stride_page + h * p.sc.v_stride_head + in_page / SV_SCALE_BLOCK];
}
// What scores are multiplied by: not 0, which would make NaN of a masked one (-inf); a NaN stays
__device__ __forceinline__ float score_factor(float row, float scale) {
    const float f = row * scale;
    return f < 1.17549435e-38f ? 1.17549435e-38f : f;
}
// The least that scales of values are held against, so that a block of zeros divides by something.
constexpr float kLeastScale = 7.88860905e-31f;  // 2^-100
// The codes are exact in fp16, so the products are formed in it.  A row of bf16 queries is brought
// into its range by a power of two, given as the exponent bits of a float (those of its inverse
// are (254 << 23) - them): its largest element goes to [2^14, 2^15), its sums stay below 2^31.
__device__ __forceinline__ int row_lift(float largest) {
    const int e = (__float_as_int(largest) >> 23) - 127;  // (0 and subnormal: as the smallest normal)
    return min(127 + 14 - e, 253) << 23;
}

__device__ __forceinline__ float fast_exp2(float x) {  // 2^x; 2^-inf = 0
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

#endif  // __CUDACC__

// tensor maps of the pages, a head's rows in parts of 64 elements (128 bytes, swizzled):
// boxes of `box` rows and `parts` parts
bool encode_pages(CUtensorMap* keys, CUtensorMap* values, const AttendArgs& p, int box, int parts);
// of a cache held in 8 bits: boxes of `box` whole rows of a head, swizzled
bool encode_codes(CUtensorMap* keys, CUtensorMap* values, const AttendArgs& p, int box);

// Launch whose start may overlap with the end of the kernel before it on the stream; the
// kernels wait for that one with grid_dependency_wait() before they read anything.
template <typename... P, typename... A>
inline cudaError_t launch_early(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, A&&... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

// the two kernels' launchers (RM rows a tile) and the join of the cut units
// (compiled apart: plain calls, those with sinks, and those over a cache held in 8 bits)
cudaError_t launch_attend_rows(int dtype, int dim, int mt, const AttendArgs& p, cudaStream_t s);
cudaError_t launch_attend_rows_sinks(int dtype, int dim, int mt, const AttendArgs& p, cudaStream_t s);
cudaError_t launch_attend_rows_8bit(int dtype, int dim, int mt, const AttendArgs& p, cudaStream_t s);
cudaError_t launch_attend_tiles(int dtype, int dim, int rm, const AttendArgs& p, cudaStream_t s);
cudaError_t launch_attend_tiles_sinks(int dtype, int dim, int rm, const AttendArgs& p, cudaStream_t s);
cudaError_t launch_attend_tiles_8bit(int dtype, int dim, int rm, const AttendArgs& p, cudaStream_t s);
cudaError_t launch_attend_join(int dtype, int dim, int rm, const AttendArgs& p, cudaStream_t s);

}  // namespace sv
