// A mixture-of-experts layer for a few tokens, and its top-k router, for
// gfx950 (MI355X).
//
// Router.  For each token the k experts of the largest logits (ties to the
// lowest index) and their weights: the softmax over all experts, or the
// sigmoid of each, optionally divided by the sum over the chosen ones.
//
// Layer.  For a pair (t, j) with expert e = ids[t, j]:
//
//   g | u = W1[e] x[t],  h = silu(g) * u,  out[t] = sum_j w[t, j] * W2[e] h
//
// With few tokens the weights of the chosen experts are the whole cost: they
// are read once and everything else is small beside them.  So the tokens stay
// in 16 bits (rounding them to 8 would save nothing), the 8-bit weights are
// widened in registers (exactly: E4M3 and int8 fit bf16 and f16), and the
// products run on 16x16x32 MFMAs whose 16 rows are weight rows and whose 16
// columns are tokens.  Two launches: the experts' hidden rows, and the
// weighted sum of their down projections.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "gfg.h"
#include "gfg_device.h"
#include "gfg_internal.h"

namespace gfg {
namespace {

// ------------------------------------------------------------------ router
constexpr int kMaxExperts = 1024;

__device__ __forceinline__ float as_f32(float v) { return v; }
__device__ __forceinline__ float as_f32(__bf16 v) { return float(v); }
__device__ __forceinline__ float as_f32(_Float16 v) { return float(v); }

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int w = 32; w >= 1; w >>= 1) v = fmaxf(v, __shfl_xor(v, w, 64));
    return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int w = 32; w >= 1; w >>= 1) v += __shfl_xor(v, w, 64);
    return v;
}
__device__ __forceinline__ int wave_min(int v) {
#pragma unroll
    for (int w = 32; w >= 1; w >>= 1) v = min(v, __shfl_xor(v, w, 64));
    return v;
}

// One wave a token; lane l holds experts l, l + 64, ... (EPL of them).  A round
// takes the largest remaining selection value and, among its holders, the
// lowest index; lane j keeps the result of round j.
template <typename T, int EPL>
__global__ __launch_bounds__(256) void moe_topk_kernel(const T* __restrict__ logits, const float* __restrict__ bias,
                                                       int32_t* __restrict__ ids, float* __restrict__ weights,
                                                       int64_t tokens, int E, int k, bool sigmoid, bool renorm,
                                                       float scale) {
    const int lane = threadIdx.x & 63;
    const int64_t t = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6);
    if (t >= tokens) return;
    const float ninf = -__builtin_inff();
    const T* row = logits + t * E;
    float l[EPL], s[EPL];
    float m = ninf;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = lane + 64 * i;
        const float v = e < E ? as_f32(row[e]) : ninf;
        l[i] = v == v ? v : ninf;              // a NaN never runs
        m = fmaxf(m, l[i]);
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) s[i] = l[i];
    m = wave_max(m);
    float total = 1.0f;
    // exp(l - m) with the difference of two infinities taken as zero
    auto expo = [&](float v) { return v == m ? 1.0f : expf(v - m); };
    auto sig = [](float v) { return 1.0f / (1.0f + expf(-v)); };
    if (!sigmoid) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) sum += l[i] > ninf ? expo(l[i]) : 0.0f;
        total = wave_sum(sum);
    }
    if (bias) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = lane + 64 * i;
            if (l[i] > ninf) s[i] = (sigmoid ? sig(l[i]) : expo(l[i]) / total) + bias[e];
        }
    }
    int mine = -1;
    for (int j = 0; j < k; ++j) {
        float best = ninf;
        int at = 0x7FFFFFFF;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (s[i] > best) { best = s[i]; at = lane + 64 * i; }
        const float top = wave_max(best);
        const int e = wave_min(best == top ? at : 0x7FFFFFFF);
        if (e == 0x7FFFFFFF) break;            // nothing above -infinity is left
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (e == lane + 64 * i) s[i] = ninf;
        if (lane == j) mine = e;
    }
    float w = 0.0f;
    if (mine >= 0) {
        const float v = as_f32(row[mine]);
        w = sigmoid ? sig(v) : expo(v) / total;
    }
    if (renorm) {
        const float sum = wave_sum(w);
        w = sum > 0.0f ? w / sum : 0.0f;
    }
    if (lane < k) {
        ids[t * k + lane] = mine;
        weights[t * k + lane] = w * scale;
    }
}

template <typename T>
void launch_topk(const void* logits, const float* bias, int32_t* ids, float* weights, int64_t tokens, int E, int k,
                 bool sigmoid, bool renorm, float scale, hipStream_t s) {
    const dim3 grid(unsigned((tokens + 3) / 4));
    const T* l = static_cast<const T*>(logits);
#define GFG_TOPK(EPL)                                                                                              \
    hipLaunchKernelGGL((moe_topk_kernel<T, EPL>), grid, dim3(256), 0, s, l, bias, ids, weights, tokens, E, k, sigmoid, \
                       renorm, scale)
    if (E <= 64) GFG_TOPK(1);
    else if (E <= 128) GFG_TOPK(2);
    else if (E <= 256) GFG_TOPK(4);
    else if (E <= 512) GFG_TOPK(8);
    else GFG_TOPK(16);
#undef GFG_TOPK
}

// ------------------------------------------------------------------ layer
constexpr int NT_THREADS = 256, NW = 4;
constexpr int kMaxPairs = 1024;
constexpr int kUnitRows = 64;                  // pairs of one expert that share a pass over its weights
constexpr uint32_t kOutside = 0x80000000u;     // past every buffer window used here (all below 2^30 bytes)

typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));

enum Weight { FP8 = 0, INT8 = 1 };

struct MoeParams {
    const void* x;           // [T][H] bf16 or f16
    const int32_t* ids;      // [T][k]
    const float* weights;    // [T][k]
    const uint8_t* w1;       // [E][2I][H]
    const void* s1;          // FP8: [E][2I/128][H/128] bytes; INT8: [E][2I] float
    const uint8_t* w2;       // [E][H][I]
    const void* s2;          // FP8: [E][H/128][I/128] bytes; INT8: [E][H] float
    uint8_t* h;              // [T*k][2][I] bf16: the hidden rows as high and low halves
    void* out;               // [T][H]
    int T, k, E, H, I;
    int ks;                  // down projection: waves that split an expert's I
};

template <typename A> struct Vec;
template <> struct Vec<__bf16> { typedef bf8 v8; };
template <> struct Vec<_Float16> { typedef h8 v8; };

__device__ __forceinline__ v4f mma(bf8 a, bf8 b, v4f c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
__device__ __forceinline__ v4f mma(h8 a, h8 b, v4f c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }

// Eight weight codes as eight 16-bit floats, exactly: E4M3 has 4 significant
// bits and exponents from -9 to 8, an int8 has at most 8 significant bits.
template <int W, typename A>
__device__ __forceinline__ typename Vec<A>::v8 widen(uint32_t lo, uint32_t hi) {
    typename Vec<A>::v8 o;
#pragma unroll
    for (int d = 0; d < 2; ++d) {
        const uint32_t c = d ? hi : lo;
        if constexpr (W == FP8) {
            if constexpr (__is_same(A, __bf16)) {
                const bf2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, false);
                const bf2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, true);
                o[4 * d] = a[0]; o[4 * d + 1] = a[1]; o[4 * d + 2] = b[0]; o[4 * d + 3] = b[1];
            } else {
                const h2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c, 1.0f, false);
                const h2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c, 1.0f, true);
                o[4 * d] = a[0]; o[4 * d + 1] = a[1]; o[4 * d + 2] = b[0]; o[4 * d + 3] = b[1];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) o[4 * d + i] = A(float(int8_t(c >> (8 * i))));
        }
    }
    return o;
}

// E8M0 byte b as 2^(b - 127): 255 is NaN, and 0 (2^-127) a subnormal.
__device__ __forceinline__ float e8m0(uint32_t b) {
    return __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7FC00000u : b << 23);
}

// The pairs of every expert, side by side: list[] holds the pair indices
// (t * k + j) expert by expert, unit[] the stretches of at most kUnitRows of
// them: expert | first << 10 | (rows - 1) << 20.  Ids outside [0, E) are in no
// unit.  Every workgroup builds its own copy, so the copies have to agree on
// which pairs a unit holds: an expert of one unit may list its pairs in the
// order of the LDS atomics (a pair's sums never mix with another's), an expert
// of several lists them in their own order.
struct Routing {
    int16_t list[kMaxPairs];
    int16_t expert[kMaxPairs];
    uint32_t unit[kMaxPairs];
    int cnt[kMaxExperts];
    int tmp[NW];
    int units, most;         // units, and the largest unit's rows
};

__device__ __forceinline__ void build_routing(GFG_LDS Routing* r, const int32_t* ids, int P, int E) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    constexpr int PPT = kMaxPairs / NT_THREADS, EPT = kMaxExperts / NT_THREADS;
    int e[PPT], slot[PPT];
#pragma unroll
    for (int i = 0; i < PPT; ++i) {
        const int p = tid + i * NT_THREADS;
        e[i] = p < P ? ids[p] : -1;
    }
    if (tid == 0) r->most = 0;
#pragma unroll
    for (int i = 0; i < EPT; ++i) r->cnt[tid * EPT + i] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PPT; ++i) {
        slot[i] = -1;
        if (e[i] < 0 || e[i] >= E) e[i] = -1;
        r->expert[tid + i * NT_THREADS] = int16_t(e[i]);
        if (e[i] >= 0) slot[i] = __hip_atomic_fetch_add(&r->cnt[e[i]], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PPT; ++i)
        if (slot[i] >= 0 && r->cnt[e[i]] > kUnitRows) {
            const int p = tid + i * NT_THREADS;
            int before = 0;
            for (int q = 0; q < p; ++q) before += int(r->expert[q]) == e[i];
            slot[i] = before;
        }
    int c[EPT], mine = 0;                      // pairs | units << 16 of this thread's experts
    int most = 0;
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
        c[i] = r->cnt[tid * EPT + i];
        most = max(most, c[i]);
        mine += c[i] | ((c[i] + kUnitRows - 1) / kUnitRows) << 16;
    }
    int x = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int y = __shfl_up(x, d, 64);
        if (lane >= d) x += y;
    }
    if (lane == 63) r->tmp[wave] = x;
    __hip_atomic_fetch_max(&r->most, min(most, kUnitRows), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    __syncthreads();
    int before = x - mine;
#pragma unroll
    for (int w = 0; w < NW; ++w)
        if (w < wave) before += r->tmp[w];
    int first = before & 0xFFFF, u = before >> 16;
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
        const int ex = tid * EPT + i;
        r->cnt[ex] = first;
        for (int done = 0; done < c[i]; done += kUnitRows)
            r->unit[u++] = uint32_t(ex) | uint32_t(first + done) << 10 | uint32_t(min(c[i] - done, kUnitRows) - 1) << 20;
        first += c[i];
    }
    if (tid == NT_THREADS - 1) r->units = u;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PPT; ++i)
        if (slot[i] >= 0) r->list[r->cnt[e[i]] + slot[i]] = int16_t(tid + i * NT_THREADS);
    __syncthreads();
}

struct Unit { int e, first, rows; };
__device__ __forceinline__ Unit unit_of(const GFG_LDS Routing* r, int u) {
    const uint32_t w = __builtin_amdgcn_readfirstlane(r->unit[u]);
    return Unit{int(w & 0x3FF), int((w >> 10) & 0x3FF), int(w >> 20) + 1};
}

__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0);
}

// ---- hidden rows: h = silu(g) * u for 16 columns of I and one unit.
//
// A tile is the 16 gate rows and the 16 up rows of those columns.  The four
// waves split H; a lane reads 16 bytes of a weight row (K chunk 16 lq of a
// 64-byte half) and the token's elements of the same chunk, so the MFMA's K
// order is a permutation that both operands share.
template <int NT> constexpr int kUpDepth = NT == 1 ? 4 : NT == 2 ? 3 : 2;

template <int W, int NT>
struct UpStage {
    u32x4 w[2][2];           // [gate, up][64-byte half]
    u32x4 x[NT][2][2];       // [token tile][half][8 elements]
    uint32_t s[2];           // E8M0 bytes
};

template <int W, typename A, int NT>
__device__ __forceinline__ void up_tile(const MoeParams& p, const GFG_LDS Routing* r, GFG_LDS v4f* red, Unit un, int it) {
    typedef typename Vec<A>::v8 v8;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, lq = lane >> 4;
    const int KB = p.H / 128;
    const int kb0 = wave * KB / NW, kb1 = (wave + 1) * KB / NW;
    const uint8_t* const base = p.w1 + (int64_t(un.e) * 2 * p.I + it * 16) * p.H;
    const __amdgpu_buffer_rsrc_t rw[2] = {make_rsrc(base, 16u * uint32_t(p.H)),
                                          make_rsrc(base + int64_t(p.I) * p.H, 16u * uint32_t(p.H))};
    const auto rx = make_rsrc(p.x, uint32_t(p.T) * uint32_t(p.H) * 2u);
    const int sb = p.I / 128;                  // 128-row scale blocks of the gate half
    const uint8_t* const sbase = static_cast<const uint8_t*>(p.s1) + (int64_t(un.e) * 2 * sb + it / 8) * KB;
    const __amdgpu_buffer_rsrc_t rs[2] = {make_rsrc(sbase, uint32_t(KB)), make_rsrc(sbase + int64_t(sb) * KB, uint32_t(KB))};
    const uint32_t woff = uint32_t(l16) * uint32_t(p.H) + uint32_t(lq * 16);
    uint32_t xoff[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int i = 16 * t + l16;
        xoff[t] = i < un.rows ? uint32_t(r->list[un.first + i] / p.k) * uint32_t(p.H) * 2u + uint32_t(lq * 32) : kOutside;
    }
    constexpr int D = kUpDepth<NT>;
    UpStage<W, NT> st[D];
    auto load = [&](UpStage<W, NT>& s, int kb) {
        const bool in = kb < kb1;
        const uint32_t ko = in ? uint32_t(kb) * 128u : 0x40000000u;
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
            for (int j = 0; j < 2; ++j) s.w[f][j] = load16(rw[f], woff + ko + 64u * j);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    s.x[t][j][q] = load16(rx, xoff[t] + (in ? uint32_t(kb) * 256u : 0x40000000u) + 128u * j + 16u * q);
        if constexpr (W == FP8) {
#pragma unroll
            for (int f = 0; f < 2; ++f)
                s.s[f] = __builtin_amdgcn_raw_buffer_load_b8(rs[f], in ? uint32_t(kb) : kOutside, 0, 0);
        }
    };
    v4f acc[2][NT] = {};
    auto consume = [&](const UpStage<W, NT>& s) {
        v4f part[2][NT];
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
            for (int t = 0; t < NT; ++t) part[f][t] = W == FP8 ? v4f{} : acc[f][t];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    const v8 a = widen<W, A>(s.w[f][j][2 * q], s.w[f][j][2 * q + 1]);
#pragma unroll
                    for (int t = 0; t < NT; ++t) part[f][t] = mma(a, __builtin_bit_cast(v8, s.x[t][j][q]), part[f][t]);
                }
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if constexpr (W == FP8) {
                    const float sc = e8m0(s.s[f]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[f][t][i] = fmaf(part[f][t][i], sc, acc[f][t][i]);
                } else {
                    acc[f][t] = part[f][t];
                }
            }
    };
#pragma unroll
    for (int d = 0; d < D; ++d) {
        load(st[d], kb0 + d);
        __builtin_amdgcn_sched_barrier(0);
    }
    // the barriers keep the order as written: consume a block, load the one
    // that takes its registers, D blocks ahead
    for (int kb = kb0; kb < kb1; kb += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (kb + d < kb1) consume(st[d]);
            __builtin_amdgcn_sched_barrier(0);
            load(st[d], kb + d + D);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    // the waves' sums meet in LDS; wave t finishes token tile t
    __syncthreads();                           // the previous tile's sums have been read
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int t = 0; t < NT; ++t) red[((wave * 2 + f) * NT + t) * 64 + lane] = acc[f][t];
    __syncthreads();
    const int i = 16 * wave + l16;
    if (wave >= NT || i >= un.rows) return;
    v4f g = {}, u = {};
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        g += red[((w * 2) * NT + wave) * 64 + lane];
        u += red[((w * 2 + 1) * NT + wave) * 64 + lane];
    }
    const int col = it * 16 + lq * 4;
    if constexpr (W == INT8) {
        const float* sc = static_cast<const float*>(p.s1) + int64_t(un.e) * 2 * p.I + col;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            g[c] *= sc[c];
            u[c] *= sc[p.I + c];
        }
    }
    // h in two bf16 halves, high and low: 16 significant bits with fp32's
    // range, so that the only rounding to 16 bits is the output's
    typedef __bf16 b4 __attribute__((ext_vector_type(4)));
    b4 hi, lo;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const float v = g[c] / (1.0f + expf(-g[c])) * u[c];
        hi[c] = __bf16(v);
        const float rest = v - float(hi[c]);
        lo[c] = __bf16(rest == rest ? rest : 0.0f);   // an infinite v has no low half
    }
    uint8_t* const row = p.h + int64_t(r->list[un.first + i]) * 4 * p.I + col * 2;
    *reinterpret_cast<b4*>(row) = hi;
    *reinterpret_cast<b4*>(row + 2 * p.I) = lo;
}

template <int W, typename A>
__global__ __launch_bounds__(NT_THREADS, 2) void moe_up_kernel(MoeParams p) {
    __shared__ Routing routing;
    __shared__ v4f red_mem[NW * 2 * 4 * 64];
    GFG_LDS Routing* const r = (GFG_LDS Routing*)&routing;
    GFG_LDS v4f* const red = (GFG_LDS v4f*)red_mem;
    build_routing(r, p.ids, p.T * p.k, p.E);
    const int IT = p.I / 16;
    const int items = __builtin_amdgcn_readfirstlane(r->units) * IT;
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const int u = item / IT, it = item - u * IT;
        const Unit un = unit_of(r, u);
        if (un.rows <= 16) up_tile<W, A, 1>(p, r, red, un, it);
        else if (un.rows <= 32) up_tile<W, A, 2>(p, r, red, un, it);
        else up_tile<W, A, 4>(p, r, red, un, it);
    }
}

// ---- down projection: 16 output columns (rows of W2) for all tokens.
//
// A workgroup walks all units; wave w takes units (w / ks), + NW / ks, ... and
// part w % ks of their I.  Every (part, pair) sum goes to its own place in
// LDS, and the tokens' weighted sums are taken from there in the order of j:
// no atomics, and the result does not depend on the routing's list order.
template <int NT> constexpr int kDownDepth = NT == 1 ? 4 : NT == 2 ? 2 : 1;

template <int NT>
struct DownStage {
    u32x4 w[2];              // [64-byte half]
    u32x4 h[NT][2][2][2];    // [pair tile][high, low][half][8 elements]
    uint32_t s;
    int unit;                // the unit this block belongs to, or -1
    bool last;               // its last block of this wave's part
};

template <int W, int NT>
__device__ __forceinline__ void down_tile(const MoeParams& p, const GFG_LDS Routing* r, GFG_LDS v4f* y, int tile) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, lq = lane >> 4;
    const int KB = p.I / 128, P = p.T * p.k;
    const int part = wave % p.ks, stride = NW / p.ks;
    const int kb0 = part * KB / p.ks, kb1 = (part + 1) * KB / p.ks;     // never empty: ks <= KB
    const int units = __builtin_amdgcn_readfirstlane(r->units);
    const auto rh = make_rsrc(p.h, uint32_t(P) * 4u * uint32_t(p.I));
    const uint32_t woff = uint32_t(l16) * uint32_t(p.I) + uint32_t(lq * 16);
    // the cursor of the loads, one unit's block after the other
    int cu = wave / p.ks, ck = kb0;
    Unit un{};
    uint32_t hoff[NT];
    __amdgpu_buffer_rsrc_t rw = make_rsrc(p.w2, 0), rs = make_rsrc(p.w2, 0);
#pragma unroll
    for (int t = 0; t < NT; ++t) hoff[t] = kOutside;
    // past the last unit the windows are empty: the loads stay in the stream,
    // so that the compiler's waits count the same on every path, and touch nothing
    auto enter = [&]() {
        if (cu >= units) {
            rw = make_rsrc(p.w2, 0);
            rs = make_rsrc(p.w2, 0);
#pragma unroll
            for (int t = 0; t < NT; ++t) hoff[t] = kOutside;
            return;
        }
        un = unit_of(r, cu);
        rw = make_rsrc(p.w2 + (int64_t(un.e) * p.H + tile * 16) * p.I, 16u * uint32_t(p.I));
        rs = make_rsrc(static_cast<const uint8_t*>(p.s2) + (int64_t(un.e) * (p.H / 128) + tile / 8) * KB, uint32_t(KB));
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int i = 16 * t + l16;
            hoff[t] = i < un.rows ? uint32_t(r->list[un.first + i]) * 4u * uint32_t(p.I) + uint32_t(lq * 32) : kOutside;
        }
    };
    enter();
    constexpr int D = kDownDepth<NT>;
    DownStage<NT> st[D];
    auto load = [&](DownStage<NT>& s) {
        s.unit = cu < units ? cu : -1;
#pragma unroll
        for (int j = 0; j < 2; ++j) s.w[j] = load16(rw, woff + uint32_t(ck) * 128u + 64u * j);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int pl = 0; pl < 2; ++pl)
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        s.h[t][pl][j][q] = load16(rh, hoff[t] + uint32_t(pl) * 2u * uint32_t(p.I) + uint32_t(ck) * 256u + 128u * j + 16u * q);
        if constexpr (W == FP8) s.s = __builtin_amdgcn_raw_buffer_load_b8(rs, uint32_t(ck), 0, 0);
        s.last = ++ck == kb1;
        if (s.last) {
            ck = kb0;
            cu += stride;
            enter();
        }
    };
    v4f acc[NT] = {};
    auto consume = [&](const DownStage<NT>& s) {
        v4f sum[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) sum[t] = W == FP8 ? v4f{} : acc[t];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const bf8 a = widen<W, __bf16>(s.w[j][2 * q], s.w[j][2 * q + 1]);
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int pl = 0; pl < 2; ++pl) sum[t] = mma(a, __builtin_bit_cast(bf8, s.h[t][pl][j][q]), sum[t]);
            }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if constexpr (W == FP8) {
                const float sc = e8m0(s.s);
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[t][i] = fmaf(sum[t][i], sc, acc[t][i]);
            } else {
                acc[t] = sum[t];
            }
        }
        if (s.last) {
            const Unit of = unit_of(r, s.unit);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int i = 16 * t + l16;
                if (i < of.rows) y[(part * P + r->list[of.first + i]) * 4 + lq] = acc[t];
                acc[t] = v4f{};
            }
        }
    };
#pragma unroll
    for (int d = 0; d < D; ++d) {
        load(st[d]);
        __builtin_amdgcn_sched_barrier(0);
    }
    while (st[0].unit >= 0) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (st[d].unit >= 0) consume(st[d]);
            __builtin_amdgcn_sched_barrier(0);
            load(st[d]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
}

template <int W, typename OutT>
__global__ __launch_bounds__(NT_THREADS, 2) void moe_down_kernel(MoeParams p) {
    __shared__ Routing routing;
    extern __shared__ v4f y_mem[];             // [ks][T * k][16 columns]
    GFG_LDS Routing* const r = (GFG_LDS Routing*)&routing;
    GFG_LDS v4f* const y = (GFG_LDS v4f*)y_mem;
    const int P = p.T * p.k;
    build_routing(r, p.ids, P, p.E);
    const int most = __builtin_amdgcn_readfirstlane(r->most);
    typedef OutT o4 __attribute__((ext_vector_type(4)));
    for (int tile = blockIdx.x; tile < p.H / 16; tile += gridDim.x) {
        if (most <= 16) down_tile<W, 1>(p, r, y, tile);
        else if (most <= 32) down_tile<W, 2>(p, r, y, tile);
        else down_tile<W, 4>(p, r, y, tile);
        __syncthreads();
        for (int i = threadIdx.x; i < p.T * 4; i += NT_THREADS) {
            const int t = i >> 2, quad = i & 3, col = tile * 16 + quad * 4;
            v4f sum = {};
            for (int j = 0; j < p.k; ++j) {
                const int e = p.ids[t * p.k + j];
                if (e < 0 || e >= p.E) continue;
                v4f v = {};
                for (int s = 0; s < p.ks; ++s) v += y[(s * P + t * p.k + j) * 4 + quad];
                if constexpr (W == INT8) {
                    const float* sc = static_cast<const float*>(p.s2) + int64_t(e) * p.H + col;
#pragma unroll
                    for (int c = 0; c < 4; ++c) v[c] *= sc[c];
                }
                const float w = p.weights[t * p.k + j];
#pragma unroll
                for (int c = 0; c < 4; ++c) sum[c] = fmaf(w, v[c], sum[c]);
            }
            *reinterpret_cast<o4*>(static_cast<OutT*>(p.out) + int64_t(t) * p.H + col) =
                o4{OutT(sum[0]), OutT(sum[1]), OutT(sum[2]), OutT(sum[3])};
        }
        __syncthreads();
    }
}

template <int W, typename A>
int launch_layer(const MoeParams& p, hipStream_t s) {
    int cus = 0;
    if (int rc = device_cus(&cus)) return rc;
    const int P = p.T * p.k;
    const int64_t up_items = int64_t(P < p.E ? P : p.E) * (p.I / 16) + int64_t(P / kUnitRows) * (p.I / 16);
    const int up_grid = int(up_items < 2 * cus ? up_items : 2 * cus);
    hipLaunchKernelGGL((moe_up_kernel<W, A>), dim3(up_grid), dim3(NT_THREADS), 0, s, p);
    const int tiles = p.H / 16, down_grid = tiles < 2 * cus ? tiles : 2 * cus;
    hipLaunchKernelGGL((moe_down_kernel<W, A>), dim3(down_grid), dim3(NT_THREADS), unsigned(p.ks * P * 64), s, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(GFG_EHIP, "kernel launch failed: %s", hipGetErrorString(e));
    return GFG_OK;
}

int64_t workspace_bytes(int64_t T, int64_t k, int64_t I) { return T > 0 && k > 0 && I > 0 ? T * k * I * 4 : 0; }

int layer(const char* fn, int weight, const void* x, int32_t x_dtype, const int32_t* ids, const float* weights,
          const void* w1, const void* s1, const void* w2, const void* s2, void* out, int64_t T, int64_t k, int64_t E,
          int64_t H, int64_t I, void* workspace, int64_t bytes, void* stream) {
    clear_error();
    if (x_dtype != GFG_OUT_BF16 && x_dtype != GFG_OUT_F16)
        return fail(GFG_EINVAL, "%s: dtype %d is not GFG_OUT_BF16 or GFG_OUT_F16", fn, x_dtype);
    if (T < 0 || k <= 0 || E <= 0 || H <= 0 || I <= 0)
        return fail(GFG_EINVAL, "%s: bad sizes T=%lld k=%lld E=%lld H=%lld I=%lld", fn, (long long)T, (long long)k,
                    (long long)E, (long long)H, (long long)I);
    if (E > kMaxExperts || T > kMaxPairs || k > kMaxPairs || T * k > kMaxPairs)
        return fail(GFG_EUNSUPPORTED, "%s: E=%lld above %d or T*k=%lld above %d", fn, (long long)E, kMaxExperts,
                    (long long)(T * k), kMaxPairs);
    if (H % 128 || I % 128 || H > 65536 || I > 65536)
        return fail(GFG_EUNSUPPORTED, "%s: H=%lld and I=%lld must be multiples of 128 up to 65536", fn, (long long)H, (long long)I);
    if (T == 0) return GFG_OK;
    if (!x || !ids || !weights || !w1 || !s1 || !w2 || !s2 || !out) return fail(GFG_EINVAL, "%s: null pointer argument", fn);
    if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(w1) | reinterpret_cast<uintptr_t>(w2) |
         reinterpret_cast<uintptr_t>(out)) % 16 ||
        (reinterpret_cast<uintptr_t>(ids) | reinterpret_cast<uintptr_t>(weights)) % 4 ||
        (weight == INT8 && (reinterpret_cast<uintptr_t>(s1) | reinterpret_cast<uintptr_t>(s2)) % 4))
        return fail(GFG_EINVAL, "%s: x, w1, w2 and out must be 16-byte aligned, the other operands to their element", fn);
    if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16)
        return fail(GFG_EINVAL, "%s: workspace must be a 16-byte aligned device pointer", fn);
    if (bytes < workspace_bytes(T, k, I))
        return fail(GFG_EINVAL, "%s: workspace of %lld bytes, %lld are needed", fn, (long long)bytes,
                    (long long)workspace_bytes(T, k, I));
    MoeParams p{x, ids, weights, static_cast<const uint8_t*>(w1), s1, static_cast<const uint8_t*>(w2), s2,
                static_cast<uint8_t*>(workspace), out, int(T), int(k), int(E), int(H), int(I), 1};
    while (p.ks < NW && p.ks * 2 <= I / 128 && p.ks * 2 * T * k <= 512) p.ks *= 2;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (weight == FP8) return x_dtype == GFG_OUT_BF16 ? launch_layer<FP8, __bf16>(p, s) : launch_layer<FP8, _Float16>(p, s);
    return x_dtype == GFG_OUT_BF16 ? launch_layer<INT8, __bf16>(p, s) : launch_layer<INT8, _Float16>(p, s);
}

}  // namespace
}  // namespace gfg

using namespace gfg;

extern "C" int moe_topk(const void* logits, int32_t in_dtype, const float* bias, int32_t* ids, float* weights, int64_t T,
                        int64_t E, int64_t k, int32_t score, int32_t renormalize, float scale, void* stream) {
    clear_error();
    const char* fn = "moe_topk";
    if (in_dtype != GFG_IN_F32 && in_dtype != GFG_IN_BF16 && in_dtype != GFG_IN_F16)
        return fail(GFG_EINVAL, "%s: in_dtype %d is not a GFG_IN_* value", fn, in_dtype);
    if (score != GFG_SCORE_SOFTMAX && score != GFG_SCORE_SIGMOID)
        return fail(GFG_EINVAL, "%s: score %d is not a GFG_SCORE_* value", fn, score);
    if (T < 0 || E <= 0 || k <= 0 || k > E)
        return fail(GFG_EINVAL, "%s: bad sizes T=%lld E=%lld k=%lld", fn, (long long)T, (long long)E, (long long)k);
    if (E > kMaxExperts || k > 64 || T >= int64_t(1) << 31)
        return fail(GFG_EUNSUPPORTED, "%s: E=%lld above %d, k=%lld above 64 or T=%lld of 2^31 or more", fn, (long long)E,
                    kMaxExperts, (long long)k, (long long)T);
    if (T == 0) return GFG_OK;
    if (!logits || !ids || !weights) return fail(GFG_EINVAL, "%s: null pointer argument", fn);
    const uintptr_t align = in_dtype == GFG_IN_F32 ? 4 : 2;
    if (reinterpret_cast<uintptr_t>(logits) % align ||
        (reinterpret_cast<uintptr_t>(ids) | reinterpret_cast<uintptr_t>(weights) | reinterpret_cast<uintptr_t>(bias)) % 4)
        return fail(GFG_EINVAL, "%s: every operand must be aligned to its element", fn);
    hipStream_t s = static_cast<hipStream_t>(stream);
    const bool sg = score == GFG_SCORE_SIGMOID, rn = renormalize != 0;
    if (in_dtype == GFG_IN_F32) launch_topk<float>(logits, bias, ids, weights, T, int(E), int(k), sg, rn, scale, s);
    else if (in_dtype == GFG_IN_BF16) launch_topk<__bf16>(logits, bias, ids, weights, T, int(E), int(k), sg, rn, scale, s);
    else launch_topk<_Float16>(logits, bias, ids, weights, T, int(E), int(k), sg, rn, scale, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(GFG_EHIP, "%s: kernel launch failed: %s", fn, hipGetErrorString(e));
    return GFG_OK;
}

extern "C" int64_t moe_layer_workspace_bytes(int64_t T, int64_t k, int64_t I) { return workspace_bytes(T, k, I); }

extern "C" int moe_fp8_layer(const void* x, int32_t dtype, const int32_t* topk_ids, const float* topk_weights,
                             const void* w1, const uint8_t* w1_scale, const void* w2, const uint8_t* w2_scale, void* out,
                             int64_t T, int64_t k, int64_t E, int64_t H, int64_t I, void* workspace,
                             int64_t workspace_bytes, void* stream) {
    return layer("moe_fp8_layer", FP8, x, dtype, topk_ids, topk_weights, w1, w1_scale, w2, w2_scale, out, T, k, E, H, I,
                 workspace, workspace_bytes, stream);
}

extern "C" int moe_int8_layer(const void* x, int32_t dtype, const int32_t* topk_ids, const float* topk_weights,
                              const int8_t* w1, const float* w1_scale, const int8_t* w2, const float* w2_scale, void* out,
                              int64_t T, int64_t k, int64_t E, int64_t H, int64_t I, void* workspace,
                              int64_t workspace_bytes, void* stream) {
    return layer("moe_int8_layer", INT8, x, dtype, topk_ids, topk_weights, w1, w1_scale, w2, w2_scale, out, T, k, E, H, I,
                 workspace, workspace_bytes, stream);
}
