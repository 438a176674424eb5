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
#pragma once

#include "sv_internal.cuh"
#include "sv_paged.cuh"

namespace sv {

constexpr int kKeyTile = 128;  // keys a CTA takes per step
constexpr int kMaxCtas = 152;  // one CTA per SM; also sizes the workspace

// a CTA's first unit and its place in the list
struct Cut {
    long long total;       // tiles in the list (0: the CTA has none)
    long long base, end;   // the unit's tiles of the list
    int b, h, rt, past, n;
};

struct AttendArgs {
    sv_attention_args a;
    int group;      // query heads per cache head
    float qscale;   // scale * log2(e): scores are kept as powers of two
    int ctas;       // CTAs that share the work (at most kMaxCtas)
    int64_t capacity;   // positions that the page table addresses
    struct Cut* cut;    // [ctas] each CTA's first unit, for the join
    float* part_o;      // [2 * ctas][RM][dim]
    float* part_ml;     // [2 * ctas][RM][2] running maximum (in log2 units) and sum
};

#ifdef __CUDACC__

// a unit, and its key tiles [t0, t1)
struct Unit {
    int b, h, rt;
    int past, n;
    int t0, t1;
};

template <int RM>
__device__ __forceinline__ void unit_tiles(const AttendArgs& p, Unit& u) {
    const int rows = u.n * p.group;
    const int r0 = u.rt * RM, r1 = min(r0 + RM, rows) - 1;
    const int lo = p.a.window > 0 ? (int)max((int64_t)0, u.past + r0 / p.group + 1 - p.a.window) : 0;
    const int hi = u.past + r1 / p.group;  // last visible key
    u.t0 = lo / kKeyTile;
    u.t1 = hi / kKeyTile + 1;
}

// key tiles of one head of sequence b
template <int RM>
__device__ __forceinline__ long long head_tiles(const AttendArgs& p, int past, int n) {
    const int nrt = (n * p.group + RM - 1) / RM;
    long long c = 0;
    Unit u;
    u.past = past;
    u.n = n;
    for (u.rt = 0; u.rt < nrt; ++u.rt) {
        unit_tiles<RM>(p, u);
        c += u.t1 - u.t0;
    }
    return c;
}

template <int RM>
__device__ __forceinline__ long long seq_tiles(const AttendArgs& p, int b) {
    const SeqLens s = seq_lens(p.a.cache, b, (int)p.a.N, p.capacity);
    return head_tiles<RM>(p, s.past, s.n) * p.a.kv_heads;
}

// The CTA's part of the list: its first unit, the tile in it to begin with, and how
// many tiles to do in all.  Every thread of the CTA calls this and gets the same
// answer, and the first unit is left for the join.
struct Part {
    long long begin, total;  // the CTA's first tile of the list, tiles in the list
    long long base;          // list index of the first unit's first tile
    int todo;
    Unit u;
};
template <int RM, int NT>
__device__ void find_part(const AttendArgs& p, Part& part) {
    __shared__ long long s_warp[NT / 32];
    __shared__ long long s_before;
    __shared__ int s_seq;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, B = (int)p.a.B;
    long long total = 0, mine = 0;
    for (int b0 = 0; b0 < B; b0 += NT) {
        mine = b0 + t < B ? seq_tiles<RM>(p, b0 + t) : 0;
        total += mine;
    }
    total = warp_sum(total);
    if (lane == 0) s_warp[warp] = total;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) total += s_warp[w];
    __syncthreads();
    part.total = total;
    const long long ctas = min((long long)p.ctas, total);
    const int c = blockIdx.x;
    part.todo = 0;
    if (c >= ctas) {
        if (t == 0) p.cut[c].total = 0;
        return;
    }
    part.begin = total * c / ctas;
    part.todo = (int)(total * (c + 1) / ctas - part.begin);
    long long base = 0;
    for (int b0 = 0; b0 < B; b0 += NT) {
        if (B > NT) mine = b0 + t < B ? seq_tiles<RM>(p, b0 + t) : 0;
        long long x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) s_warp[warp] = x;
        __syncthreads();
        long long before = base + x - mine;
        for (int w = 0; w < warp; ++w) before += s_warp[w];
        if (part.begin >= before && part.begin < before + mine) {
            s_seq = b0 + t;
            s_before = before;
        }
        for (int w = 0; w < NT / 32; ++w) base += s_warp[w];
        __syncthreads();
        if (base > part.begin) break;
    }
    // then the head and the row tile
    Unit& u = part.u;
    u.b = s_seq;
    const SeqLens s = seq_lens(p.a.cache, u.b, (int)p.a.N, p.capacity);
    u.past = s.past;
    u.n = s.n;
    const long long per_head = head_tiles<RM>(p, s.past, s.n);
    long long at = part.begin - s_before;
    u.h = (int)(at / per_head);
    at -= u.h * per_head;
    part.base = s_before + u.h * per_head;
    for (u.rt = 0;; ++u.rt) {
        unit_tiles<RM>(p, u);
        if (at < u.t1 - u.t0) break;
        at -= u.t1 - u.t0;
        part.base += u.t1 - u.t0;
    }
    if (t == 0) p.cut[c] = Cut{total, part.base, part.base + (u.t1 - u.t0), u.b, u.h, u.rt, u.past, u.n};
}

// the unit after u (there is one: the caller counts tiles)
template <int RM>
__device__ __forceinline__ void next_unit(const AttendArgs& p, Unit& u) {
    const int nrt = (u.n * p.group + RM - 1) / RM;
    if (++u.rt == nrt) {
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
    unit_tiles<RM>(p, u);
}

// rows that no unit covers: zeros past a sequence's new tokens, NaN for a sequence
// whose lengths are bad
template <typename T, int NT>
__device__ void fill_idle_rows(const AttendArgs& p) {
    const int vecs = (int)p.a.dim / 8, Hq = (int)p.a.q_heads;
    for (int b = blockIdx.x; b < p.a.B; b += gridDim.x) {
        const SeqLens s = seq_lens(p.a.cache, b, (int)p.a.N, p.capacity);
        if (s.bad && threadIdx.x == 0 && p.a.row_status) atomicOr(p.a.row_status + b, SV_ROW_BAD_LENGTH);
        const uint32_t w = s.bad ? Pair<T>::pack(NAN, NAN) : 0u;
        const int64_t idle = (int64_t)(p.a.N - s.n) * Hq * vecs;
        for (int64_t x = threadIdx.x; x < idle; x += NT) {
            const int64_t row = x / vecs;
            T* o = (T*)p.a.out + b * p.a.o_stride_b + (s.n + row / Hq) * p.a.o_stride_n +
                   (row % Hq) * p.a.o_stride_h + (x % vecs) * 8;
            *reinterpret_cast<uint4*>(o) = make_uint4(w, w, w, w);
        }
    }
}

template <typename T>
__device__ __forceinline__ T* out_row(const AttendArgs& p, const Unit& u, int r) {
    return (T*)p.a.out + (int64_t)u.b * p.a.o_stride_b + (int64_t)(r / p.group) * p.a.o_stride_n +
           (int64_t)(u.h * p.group + r % p.group) * p.a.o_stride_h;
}
template <typename T>
__device__ __forceinline__ const T* q_row(const AttendArgs& p, const Unit& u, int r) {
    return (const T*)p.a.q + (int64_t)u.b * p.a.q_stride_b + (int64_t)(r / p.group) * p.a.q_stride_n +
           (int64_t)(u.h * p.group + r % p.group) * p.a.q_stride_h;
}

__device__ __forceinline__ float fast_exp2(float x) {  // 2^x; 2^-inf = 0
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

#endif  // __CUDACC__

// the two kernels' launchers (RM rows a tile) and the join of the cut units
cudaError_t launch_attend_rows(int dtype, int dim, int mt, const AttendArgs& p, cudaStream_t s);
cudaError_t launch_attend_tiles(int dtype, int dim, const AttendArgs& p, unsigned long long wait_ns, cudaStream_t s);
cudaError_t launch_attend_join(int dtype, int dim, int rm, const AttendArgs& p, cudaStream_t s);

}  // namespace sv
