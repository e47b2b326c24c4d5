// Training of the top-k router for gfx950 (MI355X): the balance loss of each
// sequence's tokens over the experts, the counts, and the gradient of the logits
// from it and from the chosen experts' weights.
//
//   f_e = count_e E / (k n),  P_e = mean p_e,  lse = logsumexp(l)
//   loss = 1/S sum_s (alpha sum_e f_e P_e + z mean lse^2)
//   softmax: p = e^l / sum e^l,      dl = p (c - sum c p)              c_e = alpha f_e / (S n)
//   sigmoid: p = s / sum s,          dl = s (1 - s) / (sum s) (c - sum c p)
//   and 2 z / (S n) lse e^l / sum e^l from the last term
//   weights w_j = scale v_j (/ sum v), v the softmax or the sigmoid of the chosen:
//   dL/dv_j = scale dw_j, or scale (dw_j - sum dw v / sum v) / sum v
//
// A wave has a token, its lanes the experts lane, lane + 64, ...; a row of logits
// is read once by each of the two passes.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "gfg.h"
#include "gfg_device.h"
#include "gfg_internal.h"

namespace gfg {
namespace {

constexpr int64_t kMostChunks = 1024;          // token ranges of the loss, a workgroup each

struct RouterArgs {
    const void* logits;
    const int32_t *ids, *offsets;
    int64_t T;
    int E, k, S, score;
    int per;                 // tokens of a range
    float* sums;             // [ranges + S - 1 pieces][2 E + 2]: p, counts, lse^2, tokens
    unsigned* arrived;
    float* losses;           // one of each finishing workgroup
    float *loss, *factors;
    int32_t* counts;
    float alpha, z;
};

__device__ __forceinline__ float add(float a, float b) { return a + b; }

// A token's logits, NaN as -infinity.
template <typename L, int NE>
__device__ __forceinline__ void load_logits(float (&l)[NE], const L* row, int E, int lane) {
#pragma unroll
    for (int j = 0; j < NE; ++j) {
        const int e = lane + 64 * j;
        const float v = e < E ? float(row[e]) : -INFINITY;
        l[j] = v != v ? -INFINITY : v;
    }
}

// Its softmax in `e` (zeros if every expert is masked): e^(l - top) * inv; returns logsumexp.
template <int NE>
__device__ __forceinline__ float softmax_of(const float (&l)[NE], float (&e)[NE], float& top, float& inv) {
    top = l[0];
#pragma unroll
    for (int j = 1; j < NE; ++j) top = fmaxf(top, l[j]);
    top = wave_reduce(top, [](float a, float b) { return fmaxf(a, b); });
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < NE; ++j) {
        e[j] = l[j] == top ? 1.0f : __expf(l[j] - top);        // (infinity less itself)
        if (l[j] == -INFINITY) e[j] = 0.0f;
        sum += e[j];
    }
    sum = wave_reduce(sum, add);
    inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
    for (int j = 0; j < NE; ++j) e[j] *= inv;
    return sum > 0.0f ? top + __logf(sum) : 0.0f;
}

// Sigmoid and its derivative s (1 - s), without cancellation.
__device__ __forceinline__ float sigmoid(float l, float* slope) {
    const float e = __expf(-fabsf(l)), r = 1.0f / (1.0f + e);
    *slope = e * r * r;
    return l >= 0.0f ? r : e * r;
}

// The last sequence s with offsets[s] <= t (0 where there is none).
__device__ __forceinline__ int sequence_of(const int32_t* offsets, int S, int64_t t) {
    int lo = 0, hi = S;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (offsets[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

// A workgroup's range of tokens, piece by piece of the sequences in it.  Piece
// (range r, sequence s) is number r + s: both only rise from one piece to the
// next, so no two share one.
template <typename L, int NE>
__global__ __launch_bounds__(256) void balance_sums_kernel(RouterArgs p) {
    __shared__ int count[64 * NE];
    __shared__ float total[64 * NE];
    __shared__ float zsum[4];
    __shared__ int tokens[4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t begin = int64_t(blockIdx.x) * p.per, end = begin + p.per < p.T ? begin + p.per : p.T;
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.arrived = 0u;
    int s = p.offsets ? sequence_of(p.offsets, p.S, begin) : 0;
    for (int64_t at = begin; at < end;) {
        // the sequence's tokens in the range; those before the first one's start or
        // past the last one's end are in none
        int64_t stop = end, first = 0, last = p.T;
        if (p.offsets) {
            while (s + 1 < p.S && p.offsets[s + 1] <= at) ++s;
            first = p.offsets[s];
            last = p.offsets[s + 1];
            if (s + 1 < p.S && last > at && last < end) stop = last;
        }
        for (int e = threadIdx.x; e < 64 * NE; e += 256) count[e] = 0;
        __syncthreads();
        float sum[NE] = {}, z = 0.0f;
        int n = 0;
        for (int64_t t = at + wave; t < stop; t += 4) {
            if (t < first || t >= last) continue;
            const int id = lane < p.k ? p.ids[t * p.k + lane] : -1;
            const bool chosen = id >= 0 && id < p.E;
            if (!__any(chosen)) continue;
            if (chosen) atomicAdd(&count[id], 1);
            float l[NE], e[NE], top, scale;
            load_logits(l, static_cast<const L*>(p.logits) + t * p.E, p.E, lane);
            if (p.score == GFG_SCORE_SOFTMAX || p.z != 0.0f) {
                const float lse = softmax_of(l, e, top, scale);
                if (p.z != 0.0f) z += lse * lse;
            }
            if (p.score == GFG_SCORE_SIGMOID) {
                float all = 0.0f, slope;
#pragma unroll
                for (int j = 0; j < NE; ++j) {
                    e[j] = sigmoid(l[j], &slope);
                    all += e[j];
                }
                all = wave_reduce(all, add);
                const float inv = all > 0.0f ? 1.0f / all : 0.0f;
#pragma unroll
                for (int j = 0; j < NE; ++j) e[j] *= inv;
            }
#pragma unroll
            for (int j = 0; j < NE; ++j) sum[j] += e[j];
            ++n;
        }
        // the waves' sums in order
        if (lane == 0) {
            zsum[wave] = z;
            tokens[wave] = n;
        }
        for (int w = 0; w < 4; ++w) {
            if (wave == w) {
#pragma unroll
                for (int j = 0; j < NE; ++j) total[lane + 64 * j] = w ? total[lane + 64 * j] + sum[j] : sum[j];
            }
            __syncthreads();
        }
        float* const out = p.sums + (int64_t(blockIdx.x) + s) * (2 * p.E + 2);
        for (int e = threadIdx.x; e < p.E; e += 256) {
            out[e] = total[e];
            out[p.E + e] = __int_as_float(count[e]);
        }
        if (threadIdx.x == 0) {
            out[2 * p.E] = (zsum[0] + zsum[1]) + (zsum[2] + zsum[3]);
            out[2 * p.E + 1] = __int_as_float(tokens[0] + tokens[1] + tokens[2] + tokens[3]);
        }
        __syncthreads();                       // count and total are reused
        at = stop;
        ++s;
    }
}

// Workgroup (eb, s): experts 16 eb .. +15 of sequence s over its pieces, 16 lanes
// an expert, in a fixed order; the last workgroup to finish adds the losses up,
// in order.
__global__ __launch_bounds__(256) void balance_finish_kernel(RouterArgs p) {
    __shared__ float fpart[16][17];
    __shared__ int ipart[16][17];
    __shared__ float zpart[256];
    __shared__ int npart[256];
    __shared__ bool is_last;
    const int l = threadIdx.x & 15, g = threadIdx.x >> 4, e = int(blockIdx.x) * 16 + l, s = int(blockIdx.y);
    int64_t from = 0, to = p.T;
    if (p.offsets) {
        from = p.offsets[s];
        to = p.offsets[s + 1];
        from = from < 0 ? 0 : from;
        to = to > p.T ? p.T : to;
    }
    const int64_t stride = 2 * p.E + 2;
    const int64_t r0 = from < to ? from / p.per : 0, r1 = from < to ? (to - 1) / p.per + 1 : 0;
    float P = 0.0f, zs = 0.0f;
    int c = 0, n = 0;
    if (e < p.E)
        for (int64_t r = r0 + g; r < r1; r += 16) {
            const float* const piece = p.sums + (r + s) * stride;
            P += piece[e];
            c += __float_as_int(piece[p.E + e]);
        }
    for (int64_t r = r0 + threadIdx.x; r < r1; r += 256) {
        const float* const piece = p.sums + (r + s) * stride;
        zs += piece[2 * p.E];
        n += __float_as_int(piece[2 * p.E + 1]);
    }
    fpart[g][l] = P;
    ipart[g][l] = c;
    zpart[threadIdx.x] = zs;
    npart[threadIdx.x] = n;
    __syncthreads();
    for (int w = 128; w >= 1; w >>= 1) {
        if (int(threadIdx.x) < w) {
            zpart[threadIdx.x] += zpart[threadIdx.x + w];
            npart[threadIdx.x] += npart[threadIdx.x + w];
        }
        __syncthreads();
    }
    n = npart[0];
    const float rn = n > 0 ? 1.0f / float(n) : 0.0f, rs = 1.0f / float(p.S);
    float part = 0.0f;
    if (g == 0 && e < p.E) {
        P = 0.0f;
        c = 0;
#pragma unroll
        for (int w = 0; w < 16; ++w) {
            P += fpart[w][l];
            c += ipart[w][l];
        }
        const float factor = p.alpha * rs * rn * (float(c) * (float(p.E) / float(p.k)) * rn);
        p.counts[int64_t(s) * p.E + e] = c;
        p.factors[int64_t(s) * (p.E + 1) + e] = factor;
        part = factor * P;
    }
    if (g == 0) {
#pragma unroll
        for (int w = 8; w >= 1; w >>= 1) part += __shfl_xor(part, w, 16);
    }
    if (threadIdx.x == 0) {
        if (blockIdx.x == 0) {
            p.factors[int64_t(s) * (p.E + 1) + p.E] = 2.0f * p.z * rs * rn;
            if (p.z != 0.0f) part += p.z * rs * rn * zpart[0];
        }
        const unsigned of = gridDim.x * gridDim.y, me = blockIdx.y * gridDim.x + blockIdx.x;
        __hip_atomic_store(&p.losses[me], part, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __threadfence();
        is_last = __hip_atomic_fetch_add(p.arrived, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == of - 1;
    }
    __syncthreads();
    if (!is_last) return;
    __threadfence();
    const int of = int(gridDim.x * gridDim.y);
    float t = 0.0f;
    for (int i = threadIdx.x; i < of; i += 256) t += __hip_atomic_load(&p.losses[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    zpart[threadIdx.x] = t;
    __syncthreads();
    for (int w = 128; w >= 1; w >>= 1) {
        if (int(threadIdx.x) < w) zpart[threadIdx.x] += zpart[threadIdx.x + w];
        __syncthreads();
    }
    if (threadIdx.x == 0) *p.loss = zpart[0];
}

struct RouterBack {
    const void* logits;
    const int32_t *ids, *offsets;
    const float *dweights, *factors, *dloss;
    void* dlogits;
    int64_t T;
    int E, k, S, score, renorm;
    float scale;
};

template <typename L, int NE>
__global__ __launch_bounds__(256) void router_backward_kernel(RouterBack p) {
    const int lane = threadIdx.x & 63;
    for (int64_t t = int64_t(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); t < p.T; t += int64_t(gridDim.x) * 4) {
        const int id = lane < p.k ? p.ids[t * p.k + lane] : -1;
        const bool chosen = id >= 0 && id < p.E;
        const L* const row = static_cast<const L*>(p.logits) + t * p.E;
        float l[NE], e[NE], slope[NE], d[NE], top, one;
        load_logits(l, row, p.E, lane);
        const float lse = softmax_of(l, e, top, one);  // e: the softmax
#pragma unroll
        for (int j = 0; j < NE; ++j) d[j] = 0.0f;
        const bool sigmoids = p.score == GFG_SCORE_SIGMOID;
        float all = 0.0f;                              // of the sigmoids
        float v[NE];                                   // the scores
#pragma unroll
        for (int j = 0; j < NE; ++j) {
            v[j] = e[j];
            if (sigmoids) {
                v[j] = sigmoid(l[j], &slope[j]);
                all += v[j];
            }
        }
        // ---- the loss
        if (p.factors) {
            int s = 0;
            bool in = true;
            if (p.offsets) {
                s = sequence_of(p.offsets, p.S, t);
                in = t >= p.offsets[s] && t < p.offsets[s + 1];
            }
            if (in && __any(chosen)) {
                const float* const f = p.factors + int64_t(s) * (p.E + 1);
                const float up = *p.dloss, zf = f[p.E] != 0.0f ? f[p.E] * lse : 0.0f;
                float inv = 1.0f;
                if (sigmoids) {
                    all = wave_reduce(all, add);
                    inv = all > 0.0f ? 1.0f / all : 0.0f;
                }
                float c[NE], dot = 0.0f;
#pragma unroll
                for (int j = 0; j < NE; ++j) {
                    c[j] = lane + 64 * j < p.E ? f[lane + 64 * j] : 0.0f;
                    dot += c[j] * v[j] * inv;
                }
                dot = wave_reduce(dot, add);
#pragma unroll
                for (int j = 0; j < NE; ++j)
                    d[j] = up * ((sigmoids ? slope[j] * inv : e[j]) * (c[j] - dot) + (zf != 0.0f ? zf * e[j] : 0.0f));
            }
        }
        // ---- the weights
        if (p.dweights) {
            float dw = chosen ? p.dweights[t * p.k + lane] * p.scale : 0.0f;
            // this lane's choice and its score
            float lc = chosen ? float(row[id]) : -INFINITY;
            if (lc != lc) lc = -INFINITY;
            float ds, sc;
            if (sigmoids) {
                sc = sigmoid(lc, &ds);
            } else {
                sc = lc == -INFINITY ? 0.0f : lc == top ? one : __expf(lc - top) * one;
            }
            if (p.renorm) {
                const float total = wave_reduce(chosen ? sc : 0.0f, add);
                const float inv = total > 0.0f ? 1.0f / total : 0.0f;
                const float mean = wave_reduce(chosen ? dw * sc * inv : 0.0f, add);
                dw = chosen ? (dw - mean) * inv : 0.0f;
            }
            // softmax: v (g - sum g v); sigmoid: g times its slope
            const float dot = sigmoids ? 0.0f : wave_reduce(chosen ? dw * sc : 0.0f, add);
            const float g = dw;
#pragma unroll
            for (int j = 0; j < NE; ++j)
                if (!sigmoids) d[j] -= e[j] * dot;
            for (int q = 0; q < p.k; ++q) {
                const int i = __builtin_amdgcn_readlane(id, q);
                const float gq = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(g), q));
                if (i < 0 || i >= p.E) continue;
#pragma unroll
                for (int j = 0; j < NE; ++j)
                    if (i == lane + 64 * j) d[j] += gq * (sigmoids ? slope[j] : e[j]);
            }
        }
        L* const out = static_cast<L*>(p.dlogits) + t * p.E;
#pragma unroll
        for (int j = 0; j < NE; ++j)
            if (lane + 64 * j < p.E) out[lane + 64 * j] = L(d[j]);
    }
}

template <typename F>
void by_experts(int64_t E, F f) {
    if (E <= 64) f(std::integral_constant<int, 1>{});
    else if (E <= 128) f(std::integral_constant<int, 2>{});
    else if (E <= 256) f(std::integral_constant<int, 4>{});
    else if (E <= 512) f(std::integral_constant<int, 8>{});
    else f(std::integral_constant<int, 16>{});
}
template <typename F>
void by_type(int32_t dtype, F f) {
    if (dtype == GFG_IN_F32) f(float{});
    else if (dtype == GFG_IN_BF16) f(__bf16{});
    else f(_Float16{});
}

int64_t tokens_a_range(int64_t T) {
    const int64_t n = (T + kMostChunks - 1) / kMostChunks;
    return n < 16 ? 16 : n;
}
int64_t ranges(int64_t T) { return T > 0 ? (T + tokens_a_range(T) - 1) / tokens_a_range(T) : 0; }
int64_t piece_bytes(int64_t T, int64_t E, int64_t S) { return (ranges(T) + S) * (2 * E + 2) * 4; }
int64_t finishers(int64_t E, int64_t S) { return (E + 15) / 16 * S; }

int launched() {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(GFG_EHIP, "kernel launch failed: %s", hipGetErrorString(e));
    return GFG_OK;
}

int check_router(const char* fn, int32_t in_dtype, int64_t T, int64_t E, int64_t k, int64_t S, int32_t score, const int32_t* offsets) {
    if (in_dtype != GFG_IN_F32 && in_dtype != GFG_IN_BF16 && in_dtype != GFG_IN_F16)
        return fail(GFG_EINVAL, "%s: in_dtype %d is not a GFG_IN_* value", fn, in_dtype);
    if (score != GFG_SCORE_SOFTMAX && score != GFG_SCORE_SIGMOID)
        return fail(GFG_EINVAL, "%s: score %d is not a GFG_SCORE_* value", fn, score);
    if (T < 0 || E <= 0 || k <= 0 || S <= 0)
        return fail(GFG_EINVAL, "%s: bad sizes T=%lld E=%lld k=%lld S=%lld", fn, (long long)T, (long long)E, (long long)k, (long long)S);
    if (T >= int64_t(1) << 31 || E > 1024 || k > 64 || S > 65535)
        return fail(GFG_EUNSUPPORTED, "%s: T=%lld E=%lld k=%lld S=%lld; at most 2^31 - 1, 1024, 64, 65535", fn, (long long)T, (long long)E,
                    (long long)k, (long long)S);
    if (!offsets && S != 1) return fail(GFG_EINVAL, "%s: S=%lld sequences without seq_offsets", fn, (long long)S);
    return GFG_OK;
}

bool misaligned(const void* p, uintptr_t by) { return reinterpret_cast<uintptr_t>(p) % by != 0; }

}  // namespace
}  // namespace gfg

using namespace gfg;

extern "C" int64_t moe_balance_workspace_bytes(int64_t T, int64_t E, int64_t S) {
    return T >= 0 && E > 0 && S > 0 ? 16 + piece_bytes(T, E, S) + finishers(E, S) * 4 : 0;
}

extern "C" int moe_balance_loss(const void* logits, int32_t in_dtype, const int32_t* ids, const int32_t* seq_offsets, float* loss,
                                int32_t* counts, float* factors, int64_t T, int64_t E, int64_t k, int64_t S, int32_t score,
                                float alpha, float z, void* workspace, int64_t workspace_bytes, void* stream) {
    clear_error();
    const char* fn = "moe_balance_loss";
    if (int rc = check_router(fn, in_dtype, T, E, k, S, score, seq_offsets)) return rc;
    if (!loss || !counts || !factors || (T > 0 && (!logits || !ids))) return fail(GFG_EINVAL, "%s: null pointer argument", fn);
    if (misaligned(logits, in_dtype == GFG_IN_F32 ? 4 : 2) || misaligned(ids, 4) || misaligned(seq_offsets, 4) || misaligned(loss, 4) ||
        misaligned(counts, 4) || misaligned(factors, 4))
        return fail(GFG_EINVAL, "%s: a pointer is not aligned to its elements", fn);
    if (!workspace || misaligned(workspace, 16))
        return fail(GFG_EINVAL, "%s: workspace must be a 16-byte aligned device pointer", fn);
    if (workspace_bytes < moe_balance_workspace_bytes(T, E, S))
        return fail(GFG_EINVAL, "%s: workspace of %lld bytes, %lld are needed", fn, (long long)workspace_bytes,
                    (long long)moe_balance_workspace_bytes(T, E, S));
    uint8_t* const ws = static_cast<uint8_t*>(workspace);
    RouterArgs a{};
    a.logits = logits;
    a.ids = ids;
    a.offsets = seq_offsets;
    a.T = T;
    a.E = int(E);
    a.k = int(k);
    a.S = int(S);
    a.score = score;
    a.per = int(tokens_a_range(T));
    a.arrived = reinterpret_cast<unsigned*>(ws);
    a.sums = reinterpret_cast<float*>(ws + 16);
    a.losses = reinterpret_cast<float*>(ws + 16 + piece_bytes(T, E, S));
    a.loss = loss;
    a.factors = factors;
    a.counts = counts;
    a.alpha = alpha;
    a.z = z;
    hipStream_t s = static_cast<hipStream_t>(stream);
    // (a range more than there are: without tokens one workgroup still clears `arrived`)
    const unsigned grid = unsigned(T > 0 ? ranges(T) : 1);
    by_experts(E, [&](auto n) {
        by_type(in_dtype, [&](auto l) {
            hipLaunchKernelGGL((balance_sums_kernel<decltype(l), decltype(n)::value>), dim3(grid), dim3(256), 0, s, a);
        });
    });
    if (int rc = launched()) return rc;
    hipLaunchKernelGGL(balance_finish_kernel, dim3(unsigned((E + 15) / 16), unsigned(S)), dim3(256), 0, s, a);
    return launched();
}

extern "C" int moe_router_backward(const void* logits, int32_t in_dtype, const int32_t* ids, const float* dweights,
                                   const float* factors, const float* dloss, const int32_t* seq_offsets, void* dlogits, int64_t T,
                                   int64_t E, int64_t k, int64_t S, int32_t score, int32_t renormalize, float scale, void* stream) {
    clear_error();
    const char* fn = "moe_router_backward";
    if (int rc = check_router(fn, in_dtype, T, E, k, S, score, seq_offsets)) return rc;
    if (!factors != !dloss) return fail(GFG_EINVAL, "%s: factors and dloss do not go together", fn);
    if (T == 0) return GFG_OK;
    if (!factors && !dweights) return fail(GFG_EINVAL, "%s: neither the loss's nor the weights' gradient is given", fn);
    if (!logits || !ids || !dlogits) return fail(GFG_EINVAL, "%s: null pointer argument", fn);
    const uintptr_t size = in_dtype == GFG_IN_F32 ? 4 : 2;
    if (misaligned(logits, size) || misaligned(dlogits, size) || misaligned(ids, 4) || misaligned(seq_offsets, 4) ||
        misaligned(dweights, 4) || misaligned(factors, 4) || misaligned(dloss, 4))
        return fail(GFG_EINVAL, "%s: a pointer is not aligned to its elements", fn);
    const RouterBack a{logits, ids, seq_offsets, dweights, factors, dloss, dlogits, T, int(E), int(k), int(S), score, renormalize, scale};
    const int64_t wgs = (T + 3) / 4, most = int64_t(1) << 22;
    by_experts(E, [&](auto n) {
        by_type(in_dtype, [&](auto l) {
            hipLaunchKernelGGL((router_backward_kernel<decltype(l), decltype(n)::value>), dim3(unsigned(wgs < most ? wgs : most)), dim3(256), 0,
                               static_cast<hipStream_t>(stream), a);
        });
    });
    return launched();
}
