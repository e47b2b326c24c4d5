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
//   (sums of scores below 2^-30 go a way of their own, on which 1 / sum stays in range)
//
// LPT lanes share a token, NE neighbouring experts each (LPT also reaches k, so a
// lane has at most one of the token's choices), and a wave has 64 / LPT tokens;
// a row of logits is read once by each of the two passes.  32768 tokens of 385, nine
// choices, sigmoid, bf16: the loss 11 us and 7.5 for the sum over its 519 pieces, the
// gradient 25, at 2.2 TB/s of memory traffic.  Vector instructions (exp, reciprocals,
// reductions) fill two thirds of both: the gradient's 10 thousand a SIMD keep it busy
// for 42 thousand of some 62 thousand cycles; LDS is active for 12 thousand a CU, of
// which 5.5 are bank conflicts of the choices' array; the rest is waiting.  Few tokens
// take a launch each (77 of 64: 4.2 and 3.2 us).
#include <hip/hip_runtime.h>

#include <cstdint>

#include "gfg.h"
#include "gfg_device.h"
#include "gfg_internal.h"

namespace gfg {
namespace {

constexpr int64_t kMostChunks = 512;          // token ranges of the loss, a workgroup each

struct RouterArgs {
    const void* logits;
    const int32_t *ids, *offsets;
    int64_t T;
    int E, k, S, score;
    int per;                 // tokens of a range
    bool alone;              // one range of one sequence: its workgroup also finishes
    float* sums;             // [ranges + S - 1 pieces][2 E + 2]: p, counts, lse^2, tokens
    unsigned* arrived;
    float* losses;           // one of each finishing workgroup
    float *loss, *factors;
    int32_t* counts;
    float alpha, z;
};

// A lane's NE experts: those from `col` on, of which the ones from `skip` on are
// its own.  Past the last whole NE of E a lane takes the row's last ones, some of
// which (or all) are another lane's, so every load is one whole vector inside the
// row, by every lane, and no branch stands between the loads.  TINY: fewer than
// NE experts, loaded one by one, the last of them in place of those past it.
template <typename T, int NE>
struct Vec { typedef T type __attribute__((ext_vector_type(NE), aligned(sizeof(T)))); };

template <int NE, bool TINY>
struct Lane {
    int col, skip, E;
    __device__ __forceinline__ Lane(int l, int E) : E(E) {
        col = TINY ? NE * l : min(NE * l, E - NE);
        skip = min(NE * l - col, NE);
    }
    __device__ __forceinline__ bool own(int j) const { return TINY ? col + j < E : j >= skip; }
    template <typename T>
    __device__ __forceinline__ typename Vec<T, NE>::type load(const T* row) const {
        if constexpr (!TINY) return *reinterpret_cast<const typename Vec<T, NE>::type*>(row + col);
        typename Vec<T, NE>::type v;
#pragma unroll
        for (int j = 0; j < NE; ++j) v[j] = row[min(col + j, E - 1)];
        return v;
    }
    template <typename T>
    __device__ __forceinline__ void store(T* row, const float (&v)[NE]) const {
        if (!TINY && skip == 0) {
            typename Vec<T, NE>::type w;
#pragma unroll
            for (int j = 0; j < NE; ++j) w[j] = T(v[j]);
            *reinterpret_cast<typename Vec<T, NE>::type*>(row + col) = w;
        } else if (skip < NE) {
#pragma unroll
            for (int j = 0; j < NE; ++j)
                if (own(j)) row[col + j] = T(v[j]);
        }
    }
    // where expert `id` lies in an array of the lanes' NE elements each
    __device__ __forceinline__ int place(int id) const {
        const int tail = TINY ? 0 : E & (NE - 1);
        return tail && id >= E - tail ? id + NE - tail : id;
    }
    // a token's logits: NaN (the larger of a NaN and a number is the number) and another lane's as -infinity
    template <typename T>
    __device__ __forceinline__ void get(float (&f)[NE], T v) const {
#pragma unroll
        for (int j = 0; j < NE; ++j) f[j] = own(j) ? fmaxf(float(v[j]), -INFINITY) : -INFINITY;
    }
};

// Reductions over the LPT lanes of a token: exchanges inside quads, between the
// quads of 8 lanes and the halves of 16 (DPP), then between rows of 16.
template <int LPT, typename Op>
__device__ __forceinline__ float group_reduce(float v, Op op) {
    auto with = [&](auto ctrl) { return __int_as_float(dpp<decltype(ctrl)::value>(__float_as_int(v))); };
    if constexpr (LPT == 64) return wave_reduce(v, op);
    if constexpr (LPT >= 2) v = op(v, with(std::integral_constant<int, 0xB1>{}));       // quad_perm 1,0,3,2
    if constexpr (LPT >= 4) v = op(v, with(std::integral_constant<int, 0x4E>{}));       // quad_perm 2,3,0,1
    if constexpr (LPT >= 8) v = op(v, with(std::integral_constant<int, 0x141>{}));      // row_half_mirror
    if constexpr (LPT >= 16) v = op(v, with(std::integral_constant<int, 0x140>{}));     // row_mirror
    if constexpr (LPT >= 32) v = op(v, __int_as_float(__builtin_amdgcn_ds_swizzle(__float_as_int(v), 0x401F)));   // lane ^ 16
    return v;
}
template <int LPT>
__device__ __forceinline__ float group_sum(float v) { return group_reduce<LPT>(v, [](float a, float b) { return a + b; }); }
template <int LPT>
__device__ __forceinline__ bool group_any(bool b, int lane) {
    const uint64_t all = __ballot(b);
    if constexpr (LPT == 64) return all != 0;
    else return ((all >> (lane & ~(LPT - 1))) & ((uint64_t(1) << LPT) - 1)) != 0;
}
// The first of the token's lanes with b (where there is none, any).
template <int LPT>
__device__ __forceinline__ int first_of(bool b, int lane) {
    const int base = lane & ~(LPT - 1);
    const uint64_t mine = (__ballot(b) >> base) << base;
    return mine ? int(__builtin_ctzll(mine)) : lane;
}

// 1 / v to one unit of the last place; 0 for 0.
__device__ __forceinline__ float reciprocal(float v) { return v > 0.0f ? __builtin_amdgcn_rcpf(v) : 0.0f; }

// A token's softmax in `e` (zeros if every expert is masked): e^(l - top) * inv; returns logsumexp.
template <int LPT, int NE>
__device__ __forceinline__ float softmax_of(const float (&l)[NE], float (&e)[NE], float& top, float& inv) {
    top = l[0];
#pragma unroll
    for (int j = 1; j < NE; ++j) top = fmaxf(top, l[j]);
    top = group_reduce<LPT>(top, [](float a, float b) { return fmaxf(a, b); });
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < NE; ++j) {
        e[j] = l[j] == top ? 1.0f : __expf(l[j] - top);        // (infinity less itself)
        if (l[j] == -INFINITY) e[j] = 0.0f;
        sum += e[j];
    }
    sum = group_sum<LPT>(sum);
    inv = reciprocal(sum);
#pragma unroll
    for (int j = 0; j < NE; ++j) e[j] *= inv;
    return sum > 0.0f ? top + __logf(sum) : 0.0f;
}

// Sigmoid s, and its derivative s (1 - s) = (e^-l s) s without cancellation; both
// 0 for a masked expert.  (The hardware reciprocal is within one unit of the last
// place, and 0 for infinity.)
__device__ __forceinline__ float sigmoid(float l, float* slope) {
    const float e = __expf(-l), s = __builtin_amdgcn_rcpf(1.0f + e);
    *slope = fminf(e, 0x1p126f) * s * s;
    return s;
}

// p[i] of data that the kernel does not write; UNIFORM: i is the same for a wave,
// and the load goes through the scalar cache.
template <bool UNIFORM, typename T>
__device__ __forceinline__ T read(const T* p, int i) {
    if constexpr (UNIFORM) return ((const __attribute__((address_space(4))) T*)p)[__builtin_amdgcn_readfirstlane(i)];
    else return p[i];
}

// The last sequence s with offsets[s] <= t (0 where there is none).
template <bool UNIFORM>
__device__ __forceinline__ int sequence_of(const int32_t* offsets, int S, int t) {
    if constexpr (UNIFORM) t = __builtin_amdgcn_readfirstlane(t);
    int lo = 0, hi = S;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (read<UNIFORM>(offsets, mid) <= t) lo = mid;
        else hi = mid;
    }
    if constexpr (UNIFORM) return __builtin_amdgcn_readfirstlane(lo);
    return lo;
}

// The factor of an expert with that count among 1 / rn tokens.
__device__ __forceinline__ float factor_of(const RouterArgs& p, int count, float rn) {
    return p.alpha * (1.0f / float(p.S)) * rn * (float(count) * (float(p.E) / float(p.k)) * rn);
}

// A workgroup's range of tokens, piece by piece of the sequences in it.  Piece
// (range r, sequence s) is number r + s: both only rise from one piece to the
// next, so no two share one.
constexpr int SUMS_THREADS = 512;

template <typename L, int LPT, int NE, bool TINY, int SCORE>
__global__ __launch_bounds__(SUMS_THREADS) void balance_sums_kernel(RouterArgs p) {
    constexpr int WAVES = SUMS_THREADS / 64, TPW = 64 / LPT;       // tokens a wave has at a time
    __shared__ int count[LPT * NE];
    __shared__ float total[WAVES][LPT * NE];
    __shared__ float zsum[WAVES];
    __shared__ int tokens[WAVES];
    const int lane = threadIdx.x & 63, l = lane & (LPT - 1), slot = lane / LPT;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Lane<NE, TINY> my(l, p.E);
    const int64_t begin = int64_t(blockIdx.x) * p.per, end = begin + p.per < p.T ? begin + p.per : p.T;
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.arrived = 0u;
    float factored = 0.0f;                     // sum of this thread's factors times P (alone)
    int s = p.offsets ? sequence_of<true>(p.offsets, p.S, int(begin)) : 0;
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
        for (int e = threadIdx.x; e < LPT * NE; e += SUMS_THREADS) count[e] = 0;
        __syncthreads();
        float sum[NE] = {}, z = 0.0f;
        int n = 0;
        typename Vec<L, NE>::type now, next;
        int id, next_id;
        // (a token past the piece is read as its last one, and does not count)
        auto load = [&](typename Vec<L, NE>::type& v, int& i, int64_t t) {
            t = t < stop ? t : stop - 1;
            v = my.load(static_cast<const L*>(p.logits) + t * p.E);
            i = p.ids[t * p.k + min(l, p.k - 1)];
        };
        load(now, id, at + wave * TPW + slot);
        for (int64_t t0 = at + wave * TPW; t0 < stop; t0 += WAVES * TPW) {
            const int64_t t = t0 + slot;
            load(next, next_id, t + WAVES * TPW);
            const bool chosen = l < p.k && id >= 0 && id < p.E && t >= first && t < last && t < stop;
            const bool counts = group_any<LPT>(chosen, lane);
            if (chosen) atomicAdd(&count[id], 1);
            float lg[NE], e[NE], top, inv = 1.0f;
            my.get(lg, now);
            if (SCORE == GFG_SCORE_SOFTMAX || p.z != 0.0f) {
                const float lse = softmax_of<LPT>(lg, e, top, inv);
                if (p.z != 0.0f && counts && l == 0) z += lse * lse;
                inv = 1.0f;
            }
            if constexpr (SCORE == GFG_SCORE_SIGMOID) {
                float all = 0.0f, slope;
#pragma unroll
                for (int j = 0; j < NE; ++j) {
                    e[j] = sigmoid(lg[j], &slope);
                    all += e[j];
                }
                all = group_sum<LPT>(all);
                inv = reciprocal(all);
            }
            if (counts) {
#pragma unroll
                for (int j = 0; j < NE; ++j) sum[j] += e[j] * inv;
                n += l == 0;
            }
            now = next;
            id = next_id;
        }
        // the lanes' sums of an expert in a fixed order: a wave's slots, then the waves
        z = wave_reduce(z, [](float a, float b) { return a + b; });
        n = wave_reduce(n, [](int a, int b) { return a + b; });
        if (lane == 0) {
            zsum[wave] = z;
            tokens[wave] = n;
        }
#pragma unroll
        for (int j = 0; j < NE; ++j) {
#pragma unroll
            for (int x = LPT; x < 64; x <<= 1) sum[j] += __shfl_xor(sum[j], x, 64);
            if (slot == 0) total[wave][NE * l + j] = sum[j];     // (another lane's are 0)
        }
        __syncthreads();
        float zz = 0.0f;
        int nn = 0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            zz += zsum[w];
            nn += tokens[w];
        }
        const float rn = nn > 0 ? 1.0f / float(nn) : 0.0f;
        float* const out = p.sums + (int64_t(blockIdx.x) + s) * (2 * p.E + 2);
        for (int e = threadIdx.x; e < p.E; e += SUMS_THREADS) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) v += total[w][my.place(e)];
            if (p.alone) {
                const float factor = factor_of(p, count[e], rn);
                p.counts[e] = count[e];
                p.factors[e] = factor;
                factored += factor * v;
            } else {
                out[e] = v;
                out[p.E + e] = __int_as_float(count[e]);
            }
        }
        if (threadIdx.x == 0 && p.alone) {
            p.factors[p.E] = 2.0f * p.z * rn;
            if (p.z != 0.0f) factored += p.z * rn * zz;
        } else if (threadIdx.x == 0) {
            out[2 * p.E] = zz;
            out[2 * p.E + 1] = __int_as_float(nn);
        }
        __syncthreads();                       // count, total, zsum and tokens are reused
        at = stop;
        ++s;
    }
    if (!p.alone) return;
    factored = wave_reduce(factored, [](float a, float b) { return a + b; });
    if (lane == 0) zsum[wave] = factored;
    __syncthreads();
    if (threadIdx.x) return;
    float loss = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) loss += zsum[w];
    *p.loss = loss;
}

// Workgroup (eb, s): experts 32 eb .. +31 of sequence s over its pieces, 32 lanes
// an expert, in a fixed order; the last workgroup to finish adds the losses up,
// in order.
__global__ __launch_bounds__(1024) void balance_finish_kernel(RouterArgs p) {
    __shared__ float fpart[32][33];
    __shared__ int ipart[32][33];
    __shared__ float zpart[16];
    __shared__ int npart[16];
    __shared__ bool is_last;
    const int l = threadIdx.x & 31, g = threadIdx.x >> 5, e = int(blockIdx.x) * 32 + l, s = int(blockIdx.y);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
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
        for (int64_t r = r0 + g; r < r1; r += 32) {
            const float* const piece = p.sums + (r + s) * stride;
            P += piece[e];
            c += __float_as_int(piece[p.E + e]);
        }
    for (int64_t r = r0 + threadIdx.x; r < r1; r += 1024) {
        const float* const piece = p.sums + (r + s) * stride;
        zs += piece[2 * p.E];
        n += __float_as_int(piece[2 * p.E + 1]);
    }
    fpart[g][l] = P;
    ipart[g][l] = c;
    zs = wave_reduce(zs, [](float a, float b) { return a + b; });
    n = wave_reduce(n, [](int a, int b) { return a + b; });
    if (lane == 0) {
        zpart[wave] = zs;
        npart[wave] = n;
    }
    __syncthreads();
    n = 0;
    zs = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
        n += npart[w];
        zs += zpart[w];
    }
    const float rn = n > 0 ? 1.0f / float(n) : 0.0f, rs = 1.0f / float(p.S);
    float part = 0.0f;
    if (g == 0 && e < p.E) {
        P = 0.0f;
        c = 0;
#pragma unroll
        for (int w = 0; w < 32; ++w) {
            P += fpart[w][l];
            c += ipart[w][l];
        }
        const float factor = factor_of(p, c, rn);
        p.counts[int64_t(s) * p.E + e] = c;
        p.factors[int64_t(s) * (p.E + 1) + e] = factor;
        part = factor * P;
    }
    if (wave == 0) part = wave_reduce(part, [](float a, float b) { return a + b; });     // (0 in its upper half)
    if (threadIdx.x == 0) {
        if (blockIdx.x == 0) {
            p.factors[int64_t(s) * (p.E + 1) + p.E] = 2.0f * p.z * rs * rn;
            if (p.z != 0.0f) part += p.z * rs * rn * zs;
        }
        const unsigned of = gridDim.x * gridDim.y, me = blockIdx.y * gridDim.x + blockIdx.x;
        if (of == 1) {
            *p.loss = part;
        } else {
            __hip_atomic_store(&p.losses[me], part, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __threadfence();
            is_last = __hip_atomic_fetch_add(p.arrived, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == of - 1;
        }
    }
    if (gridDim.x * gridDim.y == 1) return;
    __syncthreads();
    if (!is_last || wave) return;
    __threadfence();
    const int of = int(gridDim.x * gridDim.y);
    float t = 0.0f;
    for (int i = lane; i < of; i += 64) t += __hip_atomic_load(&p.losses[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    t = wave_reduce(t, [](float a, float b) { return a + b; });
    if (lane == 0) *p.loss = t;
}

constexpr float kSmall = 0x1p-30f;            // sums of scores below it

struct RouterBack {
    const void* logits;
    const int32_t *ids, *offsets;
    const float *dweights, *factors, *dloss;
    void* dlogits;
    int64_t T;
    int E, k, S, score, renorm;
    float scale;
};

template <typename L, int LPT, int NE, bool TINY, int SCORE>
__global__ __launch_bounds__(256) void router_backward_kernel(RouterBack p) {
    constexpr int TPW = 64 / LPT;
    constexpr bool SIGMOID = SCORE == GFG_SCORE_SIGMOID;
    typedef float v4 __attribute__((ext_vector_type(4)));
    __shared__ __attribute__((aligned(16))) float scatter_smem[4][TPW][LPT * NE];
    const int lane = threadIdx.x & 63, l = lane & (LPT - 1), slot = lane / LPT;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    GFG_LDS float* const scatter = (GFG_LDS float*)scatter_smem + (wave * TPW + slot) * (LPT * NE);
    auto lds_done = [] { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); };     // (a wave's own; LDS operations keep their order)
    const Lane<NE, TINY> my(l, p.E);
    typename Vec<L, NE>::type now, next;
    int id, next_id;
    float dw_in, next_dw;
    // (a token past the last is read as the last, and not stored; without dweights
    // the ids are read in their place, and not used)
    const float* const dws = p.dweights ? p.dweights : reinterpret_cast<const float*>(p.ids);
    auto load = [&](typename Vec<L, NE>::type& v, int& i, float& dw, int64_t t) {
        t = t < p.T ? t : p.T - 1;
        v = my.load(static_cast<const L*>(p.logits) + t * p.E);
        const int64_t at = t * p.k + min(l, p.k - 1);
        i = p.ids[at];
        dw = dws[at];
    };
    const float up = p.dloss ? *p.dloss : 0.0f;
    const int64_t step = int64_t(gridDim.x) * (4 * TPW);
    int64_t mine = int64_t(blockIdx.x) * (4 * TPW) + wave * TPW + slot;
    load(now, id, dw_in, mine);
    for (int64_t first = int64_t(blockIdx.x) * (4 * TPW); first < p.T; first += step, mine += step) {
        load(next, next_id, next_dw, mine + step);
        const int64_t t = mine < p.T ? mine : p.T - 1;
        const bool chosen = l < p.k && id >= 0 && id < p.E;
        dw_in = chosen && p.dweights ? dw_in * p.scale : 0.0f;
        const int place = chosen ? my.place(id) : 0;
        // the loss's factors of the token's sequence
        typename Vec<float, NE>::type c = {};
        float zf = 0.0f;
        bool counts = false;
        if (p.factors) {
            int s = 0;
            counts = group_any<LPT>(chosen, lane);
            if (p.offsets) {
                s = sequence_of<LPT == 64>(p.offsets, p.S, int(t));
                counts = counts && t >= read<LPT == 64>(p.offsets, s) && t < read<LPT == 64>(p.offsets, s + 1);
            }
            const float* const f = p.factors + int64_t(s) * (p.E + 1);
            c = my.load(f);
            zf = read<LPT == 64>(f, p.E);
        }
        float lg[NE], e[NE], v[NE], slope[NE], d[NE], top = 0.0f, one = 0.0f, lse = 0.0f;
        my.get(lg, now);
        float lc = -INFINITY;                                  // the logit of this lane's choice
        if (p.dweights) {
#pragma unroll
            for (int j = 0; j < NE; j += 4) *reinterpret_cast<GFG_LDS v4*>(scatter + NE * l + j) = v4{lg[j], lg[j + 1], lg[j + 2], lg[j + 3]};
            lds_done();
            if (chosen) lc = scatter[place];
            lds_done();
        }
        if (!SIGMOID || zf != 0.0f) lse = softmax_of<LPT>(lg, e, top, one);        // e: the softmax
        float sc, ds = 0.0f;                                   // the choice's score, and its slope
        if constexpr (SIGMOID) sc = sigmoid(lc, &ds);
        else sc = lc == -INFINITY ? 0.0f : lc == top ? one : __expf(lc - top) * one;
        sc = chosen ? sc : 0.0f;
        // all that is summed over the token's lanes
        float all = 0.0f, dot = 0.0f;
#pragma unroll
        for (int j = 0; j < NE; ++j) {
            v[j] = SIGMOID ? sigmoid(lg[j], &slope[j]) : e[j];
            all += v[j];
            dot += c[j] * v[j];
        }
        float g = dw_in, of_softmax = 0.0f;
        if (p.dweights) {
            if (p.renorm) {
                float total = group_sum<LPT>(sc);
                if (total < kSmall) {
                    // shares of small scores are ordinary numbers: they come from scores relative to
                    // the largest choice's (sigmoids this small are e^l to fp32's last place, and so
                    // is their slope).  Scores that moe_topk holds as zero, whose weights are zero,
                    // stay out.
                    const float most = group_reduce<LPT>(lc, [](float a, float b) { return fmaxf(a, b); });
                    const bool held = lc > (SIGMOID ? -88.7f : fmaxf(top - 103.0f, -INFINITY));
                    sc = held ? __expf(lc - most) : 0.0f;
                    ds = sc;
                    total = group_sum<LPT>(sc);
                }
                // dw less the first choice's, which changes nothing but that equal ones, a
                // single one above all, give 0 and not the rest of two roundings
                const int first_choice = first_of<LPT>(chosen, lane);
                const float less = chosen ? dw_in - __shfl(dw_in, first_choice, 64) : 0.0f, inv = reciprocal(total);
                g = (less - group_sum<LPT>(less * sc) * inv) * inv;
            } else if (!SIGMOID) {
                of_softmax = group_sum<LPT>(dw_in * sc);       // (renormalized, this sum is 0)
            }
            g = chosen ? g * (SIGMOID ? ds : sc) : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < NE; ++j) d[j] = SIGMOID ? 0.0f : -(e[j] * of_softmax);
        if (p.factors) {
            float inv = 1.0f;
            dot = group_sum<LPT>(dot);
            if constexpr (SIGMOID) {
                all = group_sum<LPT>(all);
                inv = reciprocal(all);
                dot *= inv;
                if (all < kSmall) {
                    // (factors times sigmoids may lie below fp32's range, and dloss / sum above it)
                    dot = 0.0f;
#pragma unroll
                    for (int j = 0; j < NE; ++j) {
                        dot += c[j] * (v[j] * inv);
                        slope[j] *= inv;
                    }
                    dot = group_sum<LPT>(dot);
                    inv = 1.0f;
                }
            }
            if (counts) {
                const float scale = up * inv;
#pragma unroll
                for (int j = 0; j < NE; ++j) d[j] += scale * (SIGMOID ? slope[j] : e[j]) * (c[j] - dot);
                if (zf != 0.0f) {
                    const float zl = up * zf * lse;
#pragma unroll
                    for (int j = 0; j < NE; ++j) d[j] += zl * e[j];
                }
            }
        }
        // ---- the weights' part goes to the lanes that have its experts, through LDS
        if (p.dweights) {
            // a choice that stands twice is found by its place in the list, and added up in the list's order
            GFG_LDS int* const places = (GFG_LDS int*)scatter;
            if (chosen) places[place] = l;
            lds_done();
            const bool twice = chosen && places[place] != l;
            bool writes = chosen;
            lds_done();
            if (__any(twice)) {
                float sum = 0.0f;
                bool last = true;
                for (int q = 0; q < p.k; ++q) {
                    const int iq = __shfl(id, q, LPT);
                    const float gq = __shfl(g, q, LPT);
                    if (iq == id) {
                        sum += gq;
                        last = q <= l;
                    }
                }
                g = sum;
                writes = chosen && last;
            }
#pragma unroll
            for (int j = 0; j < NE; j += 4) *reinterpret_cast<GFG_LDS v4*>(scatter + NE * l + j) = v4{0.0f, 0.0f, 0.0f, 0.0f};
            lds_done();
            if (writes) scatter[place] = g;
            lds_done();
#pragma unroll
            for (int j = 0; j < NE; j += 4) {
                const v4 w = *reinterpret_cast<GFG_LDS v4*>(scatter + NE * l + j);
#pragma unroll
                for (int i = 0; i < 4; ++i) d[j + i] += w[i];
            }
            lds_done();
        }
        now = next;
        id = next_id;
        dw_in = next_dw;
        if (mine < p.T) my.store(static_cast<L*>(p.dlogits) + t * p.E, d);
    }
}

// Lanes a token and experts a lane.
template <int T, int N, bool S> struct Split {
    static constexpr int LPT = T, NE = N;
    static constexpr bool TINY = S;
};
template <typename F>
void by_split(int64_t E, int64_t k, F f) {
    const int64_t lanes = (E + 7) / 8 > k ? (E + 7) / 8 : k;
    if (E < 8 && lanes <= 8) f(Split<8, 8, true>{});
    else if (E < 8) f(Split<64, 8, true>{});
    else if (lanes <= 8) f(Split<8, 8, false>{});
    else if (lanes <= 16) f(Split<16, 8, false>{});
    else if (lanes <= 32) f(Split<32, 8, false>{});
    else if (lanes <= 64) f(Split<64, 8, false>{});
    else f(Split<64, 16, false>{});
}
template <typename F>
void by_type(int32_t dtype, F f) {
    if (dtype == GFG_IN_F32) f(float{});
    else if (dtype == GFG_IN_BF16) f(__bf16{});
    else f(_Float16{});
}

// Tokens that a workgroup of the loss has lanes for.
int64_t tokens_at_a_time(int64_t E) {
    int64_t lanes = 8;
    while (lanes < 64 && lanes * 8 < E) lanes *= 2;
    return SUMS_THREADS / lanes;
}
// Tokens of a workgroup's range: at least as many as it has lanes for,
// and up to four times as many where one range then has them all, which saves the
// second launch (E = 64: 64 tokens 4.2 us, 256 6.2, 257 in two launches 8.5).
int64_t tokens_a_range(int64_t T, int64_t E) {
    const int64_t n = (T + kMostChunks - 1) / kMostChunks, least = tokens_at_a_time(E);
    if (T > least && T <= 4 * least) return T;
    return n < least ? least : n;
}
int64_t ranges(int64_t T, int64_t E) { return T > 0 ? (T + tokens_a_range(T, E) - 1) / tokens_a_range(T, E) : 0; }
// The workspace holds as many pieces as T tokens or fewer ever have.
int64_t most_ranges(int64_t T, int64_t E) {
    const int64_t n = (T + tokens_at_a_time(E) - 1) / tokens_at_a_time(E);
    return n < kMostChunks ? n : kMostChunks;
}
int64_t piece_bytes(int64_t T, int64_t E, int64_t S) { return (most_ranges(T, E) + S) * (2 * E + 2) * 4; }
int64_t finishers(int64_t E, int64_t S) { return (E + 31) / 32 * S; }

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
    a.per = int(tokens_a_range(T, E));
    a.alone = ranges(T, E) == 1 && S == 1;
    a.arrived = reinterpret_cast<unsigned*>(ws);
    a.sums = reinterpret_cast<float*>(ws + 16);
    a.losses = reinterpret_cast<float*>(ws + 16 + piece_bytes(T, E, S));
    a.loss = loss;
    a.factors = factors;
    a.counts = counts;
    a.alpha = alpha;
    a.z = z;
    hipStream_t s = static_cast<hipStream_t>(stream);
    // (without tokens one workgroup still clears `arrived`)
    const unsigned grid = unsigned(T > 0 ? ranges(T, E) : 1);
    by_split(E, k, [&](auto n) {
        constexpr int LPT = decltype(n)::LPT, NE = decltype(n)::NE;
        constexpr bool TINY = decltype(n)::TINY;
        by_type(in_dtype, [&](auto l) {
            auto* kernel = score == GFG_SCORE_SOFTMAX ? balance_sums_kernel<decltype(l), LPT, NE, TINY, GFG_SCORE_SOFTMAX>
                                                      : balance_sums_kernel<decltype(l), LPT, NE, TINY, GFG_SCORE_SIGMOID>;
            hipLaunchKernelGGL(kernel, dim3(grid), dim3(SUMS_THREADS), 0, s, a);
        });
    });
    if (int rc = launched()) return rc;
    if (a.alone) return GFG_OK;
    hipLaunchKernelGGL(balance_finish_kernel, dim3(unsigned((E + 31) / 32), unsigned(S)), dim3(1024), 0, s, a);
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
    by_split(E, k, [&](auto n) {
        constexpr int LPT = decltype(n)::LPT, NE = decltype(n)::NE;
        constexpr bool TINY = decltype(n)::TINY;
        const int64_t wgs = (T + 4 * (64 / LPT) - 1) / (4 * (64 / LPT)), most = 2048;     // 8 a CU, each of which walks tokens
        by_type(in_dtype, [&](auto l) {
            auto* kernel = score == GFG_SCORE_SOFTMAX ? router_backward_kernel<decltype(l), LPT, NE, TINY, GFG_SCORE_SOFTMAX>
                                                      : router_backward_kernel<decltype(l), LPT, NE, TINY, GFG_SCORE_SIGMOID>;
            hipLaunchKernelGGL(kernel, dim3(unsigned(wgs < most ? wgs : most)), dim3(256), 0, static_cast<hipStream_t>(stream), a);
        });
    });
    return launched();
}
