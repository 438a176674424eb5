// sv_logits.cu -- penalties, biases and grammar masks on logits, and the token
// history that the penalties read (declared in include/spec_verify_target.h).
//
// The work on a logit is a handful of operations; what bounds the call is reading and
// writing [B, N, V] once.  Everything else is kept small beside that: which tokens
// were seen and produced are bit planes (V / 8 bytes a sequence each), so a count is
// only fetched where the bit says that there is one, and a vector of logits that the
// mask hides as a whole is not read.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "spec_verify_target.h"
#include "sv_internal.cuh"

namespace sv {
namespace {

constexpr int kLThreads = 256;
constexpr int kLWarps = kLThreads / 32;
// biases of one chunk that each warp can hold; a chunk with more re-reads the list
constexpr int kLBiasCap = 64;

// VEC bits of a bit plane from token e0 on (e0 may be negative or run past the
// end; those bits are 0)
template <int VEC>
__device__ __forceinline__ uint32_t plane_bits(const uint32_t* __restrict__ p, int e0, int V) {
    const int i = e0 >> 5, sh = e0 & 31, last = (V - 1) >> 5;
    const uint32_t lo = (i >= 0 && i <= last) ? __ldg(p + i) : 0u;
    uint32_t w = lo >> sh;
    if (sh + VEC > 32) {
        const uint32_t hi = (i + 1 >= 0 && i + 1 <= last) ? __ldg(p + i + 1) : 0u;
        w = __funnelshift_r(lo, hi, sh);
    }
    return w & ((1u << VEC) - 1u);
}

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <typename T, int VEC>
__device__ __forceinline__ void unpack(const uint4& r, float (&z)[VEC]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            z[2 * i] = __uint_as_float(w[i] << 16);
            z[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = __uint_as_float(w[i]);
    }
}
template <typename T, int VEC>
__device__ __forceinline__ uint4 pack(const float (&z)[VEC]) {
    uint32_t w[4];
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(z[2 * i], z[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(z[i]);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return x < lo ? lo : x > hi ? hi : x; }

// One CTA adjusts a chunk of kLThreads * U vectors of one row.  Tokens that the
// draft prefix or the bias list name ("special") are marked in a bit map of the
// chunk first, so that the plain tokens of a vector never look at either list.
template <typename T, int U>
__global__ void __launch_bounds__(kLThreads) logits_kernel(sv_logits_args a, int chunks) {
    constexpr int VEC = 16 / (int)sizeof(T);
    constexpr int CHUNK = kLThreads * U * VEC;
    __shared__ uint32_t s_special[CHUNK / 32];
    __shared__ int s_bias_at[kLWarps][kLBiasCap];
    __shared__ float s_bias_val[kLWarps][kLBiasCap];
    __shared__ int s_bias_n[kLWarps];
    __shared__ int s_draft[SV_MAX_GAMMA];

    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int64_t row = blockIdx.x / (unsigned)chunks;
    const int chunk = (int)(blockIdx.x % (unsigned)chunks);
    const int V = (int)a.V, b = (int)(row / a.N), i = (int)(row % a.N);
    const T* in = (const T*)a.logits + b * a.logits_stride_b + i * a.logits_stride_n;
    T* out = (T*)a.out + b * a.out_stride_b + i * a.out_stride_n;
    // vectors lie on 16-byte boundaries of the row's memory: vector j covers the
    // tokens j * VEC - skew and on
    const int skew = (int)(((uintptr_t)in & 15u) / sizeof(T));
    const bool vec = (((uintptr_t)in ^ (uintptr_t)out) & 15u) == 0;
    const int first = chunk * CHUNK - skew;
    if (first >= V) return;

    // the sequence's parameters; bad ones give NaN rows
    uint32_t bad = 0;
    int64_t slot = b;
    if (a.seen) {
        if (a.slot_of) slot = a.slot_of[b];
        if (slot < 0 || slot >= a.slots) bad |= SV_ROW_BAD_SLOT;
    }
    const float rep = a.repetition ? a.repetition[b] : 1.0f;
    const float freq = a.frequency ? a.frequency[b] : 0.0f;
    const float pres = a.presence ? a.presence[b] : 0.0f;
    if (!(rep > 0.0f) || isinf(rep) || !isfinite(freq) || !isfinite(pres)) bad |= SV_ROW_BAD_PENALTY;
    if (bad) {
        if (t == 0 && chunk == 0 && a.row_status) atomicOr(a.row_status + b, bad);
        for (int e = max(first, 0) + t; e < min(first + CHUNK, V); e += kLThreads) store1(out + e, NAN);
        return;
    }
    const uint32_t* seen = a.seen ? a.seen + slot * a.words : nullptr;
    const uint32_t* produced = a.seen ? a.produced + slot * a.words : nullptr;
    const int32_t* counts = a.seen ? a.counts + slot * a.V : nullptr;
    const uint32_t* mask = a.mask ? a.mask + b * a.mask_stride_b + i * a.mask_stride_n : nullptr;

    const int nprefix = a.draft_tokens ? (int)min((int64_t)i, a.draft_len) : 0;
    int blo = 0, bhi = 0;
    if (a.bias_ids) {
        blo = clampi(a.bias_offsets[b], 0, (int)a.bias_total);
        bhi = clampi(a.bias_offsets[b + 1], blo, (int)a.bias_total);
    }
    const bool special = nprefix > 0 || bhi > blo;

    // masks, then the logits that they leave
    uint32_t ok[U];
    uint4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int e0 = first + (u * kLThreads + t) * VEC;
        ok[u] = mask ? plane_bits<VEC>(mask, e0, V) : ((1u << VEC) - 1u);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int e0 = first + (u * kLThreads + t) * VEC;
        raw[u] = make_uint4(0, 0, 0, 0);
        if (ok[u] && e0 >= 0 && e0 + VEC <= V && vec) raw[u] = *reinterpret_cast<const uint4*>(in + e0);
    }
    uint32_t was[U], made[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int e0 = first + (u * kLThreads + t) * VEC;
        was[u] = seen ? plane_bits<VEC>(seen, e0, V) & ok[u] : 0u;
        made[u] = was[u] ? plane_bits<VEC>(produced, e0, V) & ok[u] : 0u;
    }

    bool overflow = false;
    if (special) {
        for (int w = t; w < CHUNK / 32; w += kLThreads) s_special[w] = 0u;
        __syncthreads();
        if (t < nprefix) {
            const int x = a.draft_tokens[b * a.draft_stride + t];
            s_draft[t] = x;
            const int at = x - first;
            if (x >= 0 && x < V && at >= 0 && at < CHUNK) atomicOr(&s_special[at >> 5], 1u << (at & 31));
        }
        // each warp takes a contiguous part of the bias list and keeps its order
        const int per = (bhi - blo + kLWarps - 1) / kLWarps;
        const int lo = blo + warp * per, hi = min(lo + per, bhi);
        int n = 0;
        for (int j0 = lo; j0 < hi; j0 += 32) {
            const int j = j0 + lane;
            const int x = j < hi ? a.bias_ids[j] : -1;
            const int at = x - first;
            const bool hit = x >= 0 && x < V && at >= 0 && at < CHUNK;
            const unsigned m = __ballot_sync(0xFFFFFFFFu, hit);
            if (hit) {
                atomicOr(&s_special[at >> 5], 1u << (at & 31));
                const int k = n + __popc(m & ((1u << lane) - 1u));
                if (k < kLBiasCap) {
                    s_bias_at[warp][k] = at;
                    s_bias_val[warp][k] = a.bias_values[j];
                }
            }
            n += __popc(m);
        }
        if (lane == 0) s_bias_n[warp] = n;
        overflow = __syncthreads_or(n > kLBiasCap);
    }

#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int at0 = (u * kLThreads + t) * VEC, e0 = first + at0;
        if (e0 >= V || e0 + VEC <= 0) continue;
        const bool whole = e0 >= 0 && e0 + VEC <= V && vec;
        float z[VEC];
        unpack<T, VEC>(raw[u], z);
        if (!whole) {
#pragma unroll
            for (int v = 0; v < VEC; ++v)
                if (e0 + v >= 0 && e0 + v < V && (ok[u] >> v & 1u)) z[v] = load1(in + e0 + v);
        }
        uint32_t spec = 0;
        if (special) spec = (s_special[at0 >> 5] >> (at0 & 31)) & ((1u << VEC) - 1u) & ok[u];
        if (was[u] | spec) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                if (!((was[u] | spec) >> v & 1u)) continue;
                int n = (made[u] >> v & 1u) ? counts[e0 + v] : 0;
                bool hit = was[u] >> v & 1u;
                if (spec >> v & 1u) {
                    int own = 0;
                    for (int j = 0; j < nprefix; ++j) own += s_draft[j] == e0 + v;
                    n += own;
                    hit |= own > 0;
                }
                float x = z[v];
                if (hit) {
                    x = x > 0.0f ? x / rep : x * rep;
                    x -= freq * (float)n;
                    if (n > 0) x -= pres;
                }
                if (spec >> v & 1u) {
                    float add = 0.0f;
                    if (!overflow) {
                        for (int w = 0; w < kLWarps; ++w)
                            for (int j = 0; j < s_bias_n[w]; ++j)
                                if (s_bias_at[w][j] == at0 + v) add += s_bias_val[w][j];
                    } else {
                        for (int j = blo; j < bhi; ++j)
                            if (a.bias_ids[j] == e0 + v) add += a.bias_values[j];
                    }
                    x += add;
                }
                z[v] = x;
            }
        }
#pragma unroll
        for (int v = 0; v < VEC; ++v)
            if (!(ok[u] >> v & 1u)) z[v] = -INFINITY;
        if (whole) {
            *reinterpret_cast<uint4*>(out + e0) = pack<T, VEC>(z);
        } else {
#pragma unroll
            for (int v = 0; v < VEC; ++v)
                if (e0 + v >= 0 && e0 + v < V) store1(out + e0 + v, z[v]);
        }
    }
}

__global__ void history_clear_kernel(sv_history_args a) {
    const int b = blockIdx.y;
    const int64_t slot = a.slot_of ? a.slot_of[b] : b;
    if (slot < 0 || slot >= a.slots) return;
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    const int64_t t = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    for (int64_t i = t; i < a.V; i += step) a.counts[slot * a.V + i] = 0;
    for (int64_t i = t; i < a.words; i += step) {
        a.seen[slot * a.words + i] = 0u;
        a.produced[slot * a.words + i] = 0u;
    }
}

// integer atomics only: the result does not depend on their order
__global__ void history_add_kernel(sv_history_args a) {
    const int b = blockIdx.y;
    const int64_t slot = a.slot_of ? a.slot_of[b] : b;
    if (slot < 0 || slot >= a.slots) return;
    const int L = (int)a.L;
    const int total = a.total_lens ? clampi(a.total_lens[b], 0, L) : L;
    const int prompt = a.prompt_lens ? clampi(a.prompt_lens[b], 0, total) : 0;
    for (int j = blockIdx.x * blockDim.x + threadIdx.x; j < total; j += gridDim.x * blockDim.x) {
        const int x = a.tokens[b * a.tokens_stride + j];
        if (x < 0 || x >= a.V) continue;
        atomicOr(a.seen + slot * a.words + (x >> 5), 1u << (x & 31));
        if (j >= prompt) {
            atomicOr(a.produced + slot * a.words + (x >> 5), 1u << (x & 31));
            atomicAdd(a.counts + slot * a.V + x, 1);
        }
    }
}

template <typename T, int U>
cudaError_t launch_logits(const sv_logits_args& a, cudaStream_t s) {
    constexpr int VEC = 16 / (int)sizeof(T);
    // a row that starts off a 16-byte boundary needs up to one vector more
    const int64_t nvec = (a.V + VEC - 1) / VEC + (VEC > 1 ? 1 : 0);
    const bool aligned = ((uintptr_t)a.logits & 15u) == 0 && (a.logits_stride_b * sizeof(T)) % 16 == 0 &&
                         (a.logits_stride_n * sizeof(T)) % 16 == 0;
    const int64_t need = aligned ? (a.V + VEC - 1) / VEC : nvec;
    const int64_t chunks = (need + kLThreads * U - 1) / (kLThreads * U);
    logits_kernel<T, U><<<(unsigned)(a.B * a.N * chunks), kLThreads, 0, s>>>(a, (int)chunks);
    return cudaGetLastError();
}

}  // namespace
}  // namespace sv

extern "C" int spec_verify_history_add(const sv_history_args* args, void* stream) {
    if (!args || args->struct_size != sizeof(sv_history_args)) return SV_EINVAL;
    const sv_history_args& a = *args;
    if (a.B < 0 || a.L < 0 || a.V < 1 || a.slots < 0 || a.words < (a.V + 31) / 32 || a.tokens_stride < 0)
        return SV_EINVAL;
    if (a.B > 65535 || a.V > SV_MAX_VOCAB || a.L > 0x7FFFFFFF) return SV_ETOO_LARGE;
    if (!a.slot_of && a.B > a.slots) return SV_EINVAL;
    if (a.B == 0) return SV_OK;
    if (!a.seen || !a.produced || !a.counts || (!a.tokens && a.L > 0)) return SV_EINVAL;
    cudaStream_t s = (cudaStream_t)stream;
    if (a.clear) {
        sv::history_clear_kernel<<<dim3((unsigned)((a.V + 4095) / 4096), (unsigned)a.B), 256, 0, s>>>(a);
        if (cudaGetLastError() != cudaSuccess) return SV_ECUDA;
    }
    if (a.L > 0) {
        const unsigned gx = (unsigned)((a.L + 1023) / 1024 < 64 ? (a.L + 1023) / 1024 : 64);
        sv::history_add_kernel<<<dim3(gx, (unsigned)a.B), 256, 0, s>>>(a);
        if (cudaGetLastError() != cudaSuccess) return SV_ECUDA;
    }
    return SV_OK;
}

extern "C" int spec_verify_process_logits(const sv_logits_args* args, void* stream) {
    if (!args || args->struct_size != sizeof(sv_logits_args)) return SV_EINVAL;
    const sv_logits_args& a = *args;
    if (a.dtype != SV_F32 && a.dtype != SV_BF16) return SV_EUNSUPPORTED;
    if (a.B < 0 || a.N < 1 || a.V < 1) return SV_EINVAL;
    if (a.B > SV_MAX_BATCH || a.N > SV_MAX_POSITIONS || a.V > SV_MAX_VOCAB) return SV_ETOO_LARGE;
    if (a.B == 0) return SV_OK;
    const size_t es = a.dtype == SV_BF16 ? 2 : 4;
    if (!a.logits || !a.out || ((uintptr_t)a.logits % es) || ((uintptr_t)a.out % es)) return SV_EINVAL;
    if (a.logits_stride_b < 0 || a.logits_stride_n < 0 || a.out_stride_b < 0 || a.out_stride_n < 0) return SV_EINVAL;
    // two output rows on the same memory would race
    if (a.N > 1 && a.out_stride_n < a.V) return SV_EINVAL;
    if (a.B > 1 && a.out_stride_b < a.V) return SV_EINVAL;
    if (a.seen && (!a.produced || !a.counts || a.slots < 0 || a.words < (a.V + 31) / 32)) return SV_EINVAL;
    if (a.seen && !a.slot_of && a.B > a.slots) return SV_EINVAL;
    if (a.draft_tokens && (a.draft_len < 0 || a.draft_stride < 0)) return SV_EINVAL;
    if (a.bias_ids && (!a.bias_values || !a.bias_offsets || a.bias_total < 0 || a.bias_total > 0x7FFFFFFF))
        return SV_EINVAL;
    if (a.mask && (a.mask_stride_b < 0 || a.mask_stride_n < 0)) return SV_EINVAL;
    const int64_t chunks = (a.V + 1) / (sv::kLThreads * (16 / (int)es)) + 2;  // an upper bound
    if (a.B * a.N * chunks > 0x7FFFFFFF) return SV_ETOO_LARGE;
    cudaStream_t s = (cudaStream_t)stream;
    // 64 bytes a thread where that still leaves every SM several CTAs, else 16
    const bool wide = a.B * a.N * ((a.V * (int64_t)es + 16383) / 16384) >= 2048;
    cudaError_t e;
    if (a.dtype == SV_BF16)
        e = wide ? sv::launch_logits<__nv_bfloat16, 4>(a, s) : sv::launch_logits<__nv_bfloat16, 1>(a, s);
    else
        e = wide ? sv::launch_logits<float, 4>(a, s) : sv::launch_logits<float, 1>(a, s);
    return e == cudaSuccess ? SV_OK : SV_ECUDA;
}
