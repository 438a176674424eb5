// sv_logits.cu -- penalties, biases and grammar masks on logits, and the token
// history that the penalties read (declared in include/spec_verify_target.h).
//
// The work on a logit is a handful of operations; what bounds the call is reading and
// writing [B, N, V] once.  Everything else is kept small beside that: which tokens
// were seen is a bit plane (V / 8 bytes a sequence), so a count is only fetched where
// the bit says so, and a vector of logits that the mask hides as a whole is not read.
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

// 32 bits of a bit plane from token e0 on (e0 may be negative or run past V; those bits
// are 0, whatever the plane's last word holds there: the listed tokens come from here)
__device__ __forceinline__ uint32_t plane_word(const uint32_t* __restrict__ p, int e0, int V) {
    const int i = e0 >> 5, sh = e0 & 31, last = (V - 1) >> 5;
    uint32_t w = (i >= 0 && i <= last) ? __ldg(p + i) : 0u;
    if (sh) {
        const uint32_t hi = (i + 1 >= 0 && i + 1 <= last) ? __ldg(p + i + 1) : 0u;
        w = __funnelshift_r(w, hi, sh);
    }
    if (e0 + 32 > V) w = e0 < V ? w & (0xFFFFFFFFu >> (e0 + 32 - V)) : 0u;
    return w;
}

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// -inf where the bit of a vector's element is 0.  bf16: bits 2i and 2i + 1 are spread to
// bits 0 and 16, and a product makes each a 16-bit mask.
__device__ __forceinline__ uint4 hide(uint4 r, uint32_t ok, const __nv_bfloat16*) {
    uint32_t w[4] = {r.x, r.y, r.z, r.w};
    const uint32_t spread = ok | (ok << 15);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t keep = ((spread >> (2 * i)) & 0x00010001u) * 0xFFFFu;
        w[i] = (w[i] & keep) | (0xFF80FF80u & ~keep);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 hide(uint4 r, uint32_t ok, const float*) {
    const uint32_t lowest = 0xFF800000u;
    return make_uint4(ok & 1u ? r.x : lowest, ok & 2u ? r.y : lowest, ok & 4u ? r.z : lowest, ok & 8u ? r.w : lowest);
}

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return x < lo ? lo : x > hi ? hi : x; }

// One CTA adjusts a chunk of WORDS * 32 tokens of one row, in two passes.  The first
// copies the chunk with the mask applied: nearly all of the tokens need no more than
// that.  The tokens that do (in the history, the draft prefix or the bias list) are
// gathered into a list from their bit planes, one word of 32 tokens a thread, and the
// second pass takes them one a thread, reading the logit again.  Left to the threads of
// the first pass, the few such tokens of a row cost each of their warps the whole
// arithmetic: that form took 886 us for [256, 8, 128256] bf16; this one takes 177 us (6.2
// TB/s of logits, counting those that the masks spare).  A CTA is a chain of short waits
// (parameters, bit planes, logits, listed tokens), so eight of them share an SM: at 32
// registers a thread it takes 180 us, at 40 registers 211 us.
template <typename T, int WORDS>
__global__ void __launch_bounds__(kLThreads, 8) logits_kernel(sv_logits_args a, int chunks) {
    constexpr int VEC = 16 / (int)sizeof(T);
    constexpr int CHUNK = WORDS * 32;
    constexpr int U = CHUNK / (kLThreads * VEC);
    static_assert(U * kLThreads * VEC == CHUNK && WORDS <= kLThreads, "whole vectors for every thread");
    __shared__ uint32_t s_ok[WORDS], s_seen[WORDS], s_special[WORDS];
    __shared__ uint16_t s_list[CHUNK];
    __shared__ int s_count;
    __shared__ int s_bias_at[kLWarps][kLBiasCap];
    __shared__ float s_bias_val[kLWarps][kLBiasCap];
    __shared__ int s_bias_n[kLWarps];
    __shared__ int s_draft[SV_MAX_GAMMA];

    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const unsigned row = blockIdx.x / (unsigned)chunks, chunk = blockIdx.x - row * (unsigned)chunks;
    const int V = (int)a.V, b = (int)(row / (unsigned)a.N), i = (int)(row - (unsigned)b * (unsigned)a.N);
    const T* in = (const T*)a.logits + b * a.logits_stride_b + i * a.logits_stride_n;
    T* out = (T*)a.out + b * a.out_stride_b + i * a.out_stride_n;
    // vectors lie on 16-byte boundaries of the row's memory: the chunk begins up to a
    // vector before its place
    const int skew = (int)(((uintptr_t)in & 15u) / sizeof(T));
    const bool vec = (((uintptr_t)in ^ (uintptr_t)out) & 15u) == 0;
    const int first = (int)chunk * CHUNK - skew;
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
    const uint32_t* mask = a.mask ? a.mask + b * a.mask_stride_b + i * a.mask_stride_n : nullptr;
    const int nprefix = a.draft_tokens ? (int)min((int64_t)i, a.draft_len) : 0;
    int blo = 0, bhi = 0;
    if (a.bias_ids) {
        blo = clampi(a.bias_offsets[b], 0, (int)a.bias_total);
        bhi = clampi(a.bias_offsets[b + 1], blo, (int)a.bias_total);
    }
    const bool special = nprefix > 0 || bhi > blo;
    // each warp takes a contiguous part of the bias list and keeps its order; what it needs
    // first is asked for before the barrier
    const int bias_per = (bhi - blo + kLWarps - 1) / kLWarps;
    const int bias_lo = blo + warp * bias_per, bias_hi = min(bias_lo + bias_per, bhi);
    int bias_x = bias_lo + lane < bias_hi ? a.bias_ids[bias_lo + lane] : -1;
    const int draft_x = t < nprefix ? a.draft_tokens[b * a.draft_stride + t] : -1;

    if (t < WORDS) {
        s_ok[t] = mask ? plane_word(mask, first + 32 * t, V) : 0xFFFFFFFFu;
        s_seen[t] = a.seen ? plane_word(a.seen + slot * a.words, first + 32 * t, V) : 0u;
        s_special[t] = 0u;
    }
    if (t == 0) s_count = 0;
    __syncthreads();

    // the tokens that need more
    bool overflow = false;
    if (special) {
        if (t < nprefix) {
            s_draft[t] = draft_x;
            const int at = draft_x - first;
            if (draft_x >= 0 && draft_x < V && at >= 0 && at < CHUNK) atomicOr(&s_special[at >> 5], 1u << (at & 31));
        }
        int n = 0;
        for (int j0 = bias_lo; j0 < bias_hi; j0 += 32) {
            const int j = j0 + lane;
            if (j0 != bias_lo) bias_x = j < bias_hi ? a.bias_ids[j] : -1;
            const int at = bias_x - first;
            const bool hit = bias_x >= 0 && bias_x < V && at >= 0 && at < CHUNK;
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
    if (special || a.seen) {
        // (the list's order differs from run to run; what is done to a token does not depend on it)
        if (t < WORDS) {
            uint32_t w = (s_seen[t] | s_special[t]) & s_ok[t];
            if (w) {
                int k = atomicAdd(&s_count, __popc(w));
                for (; w; w &= w - 1) s_list[k++] = (uint16_t)(32 * t + __ffs(w) - 1);
            }
        }
    }

    // the copy; a vector that the mask hides whole is not read
    if (vec && first >= 0 && first + CHUNK <= V) {
        const uint4* src = reinterpret_cast<const uint4*>(in + first) + t;
        uint4* dst = reinterpret_cast<uint4*>(out + first) + t;
        uint4 raw[U];
        uint32_t m[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = (u * kLThreads + t) * VEC;
            m[u] = (s_ok[at >> 5] >> (at & 31)) & ((1u << VEC) - 1u);
            raw[u] = make_uint4(0, 0, 0, 0);
            if (m[u]) raw[u] = src[u * kLThreads];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) dst[u * kLThreads] = hide(raw[u], m[u], in);
    } else {
#pragma unroll 1
        for (int u = 0; u < U; ++u) {
            const int at = (u * kLThreads + t) * VEC, e0 = first + at;
            const uint32_t m = (s_ok[at >> 5] >> (at & 31)) & ((1u << VEC) - 1u);
            if (vec && e0 >= 0 && e0 + VEC <= V) {
                uint4 raw = make_uint4(0, 0, 0, 0);
                if (m) raw = *reinterpret_cast<const uint4*>(in + e0);
                *reinterpret_cast<uint4*>(out + e0) = hide(raw, m, in);
                continue;
            }
#pragma unroll 1
            for (int v = 0; v < VEC; ++v) {
                const int e = e0 + v;
                if (e >= 0 && e < V) {
                    if (m >> v & 1u)
                        out[e] = in[e];
                    else
                        store1(out + e, -INFINITY);
                }
            }
        }
    }
    if (!special && !a.seen) return;
    __syncthreads();  // the list; and the copies of these logits, which the next stores replace

    const int32_t* counts = a.seen ? a.counts + slot * a.V : nullptr;
    for (int k = t; k < s_count; k += kLThreads) {
        const int at = s_list[k], e = first + at;
        float x = load1(in + e);  // unchanged by the copy, in place too
        bool hit = s_seen[at >> 5] >> (at & 31) & 1u;
        int n = hit ? counts[e] : 0;
        const bool sp = s_special[at >> 5] >> (at & 31) & 1u;
        if (sp) {
            int own = 0;
            for (int j = 0; j < nprefix; ++j) own += s_draft[j] == e;
            n += own;
            hit |= own > 0;
        }
        if (hit) {
            x = x > 0.0f ? x / rep : x * rep;
            x -= freq * (float)n;
            if (n > 0) x -= pres;
        }
        if (sp) {
            float add = 0.0f;
            if (!overflow) {
                for (int w = 0; w < kLWarps; ++w)
                    for (int j = 0; j < s_bias_n[w]; ++j)
                        if (s_bias_at[w][j] == at) add += s_bias_val[w][j];
            } else {
                for (int j = blo; j < bhi; ++j)
                    if (a.bias_ids[j] == e) add += a.bias_values[j];
            }
            x += add;
        }
        store1(out + e, x);
    }
}

__global__ void history_clear_kernel(sv_history_args a) {
    const int b = blockIdx.y;
    const int64_t slot = a.slot_of ? a.slot_of[b] : b;
    if (slot < 0 || slot >= a.slots) return;
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    const int64_t t = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    for (int64_t i = t; i < a.V; i += step) a.counts[slot * a.V + i] = 0;
    for (int64_t i = t; i < a.words; i += step) a.seen[slot * a.words + i] = 0u;
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
        if (j >= prompt) atomicAdd(a.counts + slot * a.V + x, 1);
    }
}

template <typename T, int WORDS>
cudaError_t launch_logits(const sv_logits_args& a, cudaStream_t s) {
    constexpr int64_t VEC = 16 / (int)sizeof(T), CHUNK = WORDS * 32;
    // a row that starts off a 16-byte boundary begins up to VEC - 1 tokens before its first chunk
    const bool aligned = ((uintptr_t)a.logits & 15u) == 0 && (a.logits_stride_b * sizeof(T)) % 16 == 0 &&
                         (a.logits_stride_n * sizeof(T)) % 16 == 0;
    const int64_t chunks = (a.V + (aligned ? 0 : VEC - 1) + CHUNK - 1) / CHUNK;
    logits_kernel<T, WORDS><<<(unsigned)(a.B * a.N * chunks), kLThreads, 0, s>>>(a, (int)chunks);
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
    if (!a.seen || !a.counts || (!a.tokens && a.L > 0)) return SV_EINVAL;
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
    if (a.seen && (!a.counts || a.slots < 0 || a.words < (a.V + 31) / 32)) return SV_EINVAL;
    if (a.seen && !a.slot_of && a.B > a.slots) return SV_EINVAL;
    if (a.draft_tokens && (a.draft_len < 0 || a.draft_stride < 0)) return SV_EINVAL;
    if (a.bias_ids && (!a.bias_values || !a.bias_offsets || a.bias_total < 0 || a.bias_total > 0x7FFFFFFF))
        return SV_EINVAL;
    if (a.mask && (a.mask_stride_b < 0 || a.mask_stride_n < 0)) return SV_EINVAL;
    if (a.B * a.N * ((a.V + 7) / 2048 + 1) > 0x7FFFFFFF) return SV_ETOO_LARGE;
    cudaStream_t s = (cudaStream_t)stream;
    // 16 KB of logits a CTA where that makes two CTAs a SM or more, else 4 or 8 KB: 64 rows of
    // 128256 bf16 logits (1024 CTAs of 16 KB) take 9.9 us by 16 KB and 16.9 us by 4 KB, 8 rows
    // (128 CTAs) 7.1 and 5.9 us; at 256 CTAs either may win
    const bool wide = a.B * a.N * ((a.V * (int64_t)es + 16383) / 16384) >= 304;
    cudaError_t e;
    if (a.dtype == SV_BF16)
        e = wide ? sv::launch_logits<__nv_bfloat16, 256>(a, s) : sv::launch_logits<__nv_bfloat16, 64>(a, s);
    else
        e = wide ? sv::launch_logits<float, 128>(a, s) : sv::launch_logits<float, 64>(a, s);
    return e == cudaSuccess ? SV_OK : SV_ECUDA;
}
