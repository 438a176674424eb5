// sv_attend_join.cu -- the join of the attention's units that were cut.
#include "sv_attend.cuh"

namespace sv {
namespace {

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
cudaError_t join_of(int rm, const AttendArgs& p, cudaStream_t s) {
    return rm == 16 ? launch_join<T, D, 16>(p, s) : rm == 32 ? launch_join<T, D, 32>(p, s)
         : rm == 128 ? launch_join<T, D, 128>(p, s) : launch_join<T, D, 256>(p, s);
}

}  // namespace

cudaError_t launch_attend_join(int dtype, int dim, int rm, const AttendArgs& p, cudaStream_t s) {
    if (dtype == SV_BF16)
        return dim == 64 ? join_of<__nv_bfloat16, 64>(rm, p, s) : join_of<__nv_bfloat16, 128>(rm, p, s);
    return dim == 64 ? join_of<__half, 64>(rm, p, s) : join_of<__half, 128>(rm, p, s);
}

}  // namespace sv
