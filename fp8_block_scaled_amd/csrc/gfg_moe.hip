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
#include <cstdlib>

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
constexpr int kUnitRows = 32;                  // most pairs of one expert that share a pass over its weights
constexpr int kMaxDepth = 6;                   // LDS stages of a wave's ring
constexpr uint32_t kOutside = 0x80000000u;     // past every buffer window used here (all below 2^30 bytes)

typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf4 __attribute__((ext_vector_type(4)));
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
    int ring;                // bytes of each wave's ring
    int unit_rows;           // 4, 8, 16 or 32: most pairs of a unit
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
// (t * k + j) expert by expert, unit[] the stretches of at most unit_rows of
// them: expert | first << 10 | (rows - 1) << 20.  Ids outside [0, E) are in no
// unit.  Every workgroup builds its own copy, so the copies have to agree on
// which pairs a unit holds: an expert of one unit may list its pairs in the
// order of the LDS atomics (a pair's sums never mix with another's), an expert
// of several lists them in their own order.
struct Routing {
    int16_t list[kMaxPairs];
    uint32_t unit[kMaxPairs];
    int tmp[NW];
    int units, most;         // units, and the largest unit's rows
};
constexpr int kBuildBytes = kMaxExperts * 4 + kMaxPairs * 2;    // scratch of the build

__device__ __forceinline__ void build_routing(GFG_LDS Routing* r, GFG_LDS uint8_t* scratch, const int32_t* ids, int P, int E,
                                              int unit_rows) {
    GFG_LDS int* const cnt = reinterpret_cast<GFG_LDS int*>(scratch);                    // [kMaxExperts]
    GFG_LDS int16_t* const expert = reinterpret_cast<GFG_LDS int16_t*>(cnt + kMaxExperts);   // [kMaxPairs]
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
    for (int i = 0; i < EPT; ++i) cnt[tid * EPT + i] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PPT; ++i) {
        slot[i] = -1;
        if (e[i] < 0 || e[i] >= E) e[i] = -1;
        expert[tid + i * NT_THREADS] = int16_t(e[i]);
        if (e[i] >= 0) slot[i] = __hip_atomic_fetch_add(&cnt[e[i]], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PPT; ++i)
        if (slot[i] >= 0 && cnt[e[i]] > unit_rows) {
            const int p = tid + i * NT_THREADS;
            int before = 0;
            for (int q = 0; q < p; ++q) before += int(expert[q]) == e[i];
            slot[i] = before;
        }
    int c[EPT], mine = 0;                      // pairs | units << 16 of this thread's experts
    int most = 0;
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
        c[i] = cnt[tid * EPT + i];
        most = max(most, c[i]);
        mine += c[i] | ((c[i] + unit_rows - 1) / unit_rows) << 16;
    }
    int x = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int y = __shfl_up(x, d, 64);
        if (lane >= d) x += y;
    }
    if (lane == 63) r->tmp[wave] = x;
    __hip_atomic_fetch_max(&r->most, min(most, unit_rows), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    __syncthreads();
    int before = x - mine;
#pragma unroll
    for (int w = 0; w < NW; ++w)
        if (w < wave) before += r->tmp[w];
    int first = before & 0xFFFF, u = before >> 16;
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
        const int ex = tid * EPT + i;
        cnt[ex] = first;
        for (int done = 0; done < c[i]; done += unit_rows)
            r->unit[u++] = uint32_t(ex) | uint32_t(first + done) << 10 | uint32_t(min(c[i] - done, unit_rows) - 1) << 20;
        first += c[i];
    }
    if (tid == NT_THREADS - 1) r->units = u;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PPT; ++i)
        if (slot[i] >= 0) r->list[cnt[e[i]] + slot[i]] = int16_t(tid + i * NT_THREADS);
    __syncthreads();
}

struct Unit { int e, first, rows; };
__device__ __forceinline__ Unit unit_of(const GFG_LDS Routing* r, int u) {
    const uint32_t w = __builtin_amdgcn_readfirstlane(r->unit[u]);
    return Unit{int(w & 0x3FF), int((w >> 10) & 0x3FF), int(w >> 20) + 1};
}

// ---- what both kernels share: a wave's ring.
//
// A wave streams 128-byte blocks of 16 or 32 weight rows, with the tokens' (or
// hidden rows') elements of the same columns, through its own ring of LDS
// stages filled by direct-to-LDS loads, up to kMaxDepth stages ahead and across
// the ends of experts and tiles; no barrier stands between a load and its
// MFMAs.  Whole 128-byte lines by adjacent lanes: loaded straight into MFMA
// fragments, adjacent lanes are adjacent rows, and the load path passes a
// quarter of its 64 bytes a cycle.  The fragments are read from LDS in inline
// assembly, each group together with its wait: the stage index is a run-time
// value, so the compiler, which cannot tell the stages apart, would make its
// own LDS reads wait for every load in flight.

// Wait until at most (depth - 1) * PER vector-memory operations are in flight:
// the stage loaded depth - 1 stages ago has landed.  (The counter has six bits:
// callers keep (depth - 1) * PER at most 63.)
template <int PER>
__device__ __forceinline__ void wait_stage(int depth) {
#define GFG_AHEAD(D) ((D) * PER < 63 ? (D) * PER : 63)
    switch (depth) {
        case 1: GFG_WAITCNT(0, 15); break;
        case 2: GFG_WAITCNT(GFG_AHEAD(1), 15); break;
        case 3: GFG_WAITCNT(GFG_AHEAD(2), 15); break;
        case 4: GFG_WAITCNT(GFG_AHEAD(3), 15); break;
        case 5: GFG_WAITCNT(GFG_AHEAD(4), 15); break;
        default: GFG_WAITCNT(GFG_AHEAD(5), 15); break;
    }
#undef GFG_AHEAD
}

__device__ __forceinline__ void dma(__amdgpu_buffer_rsrc_t r, GFG_LDS uint8_t* dst, uint32_t off) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (GFG_LDS void*)dst, 16, off, 0, 0, 0);
}

// Elements 4 q .. 4 q + 3 of the 16 floats at p (wave-uniform, 4-byte aligned),
// through the scalar cache: a vector load here would be younger than the loads
// in flight, and waiting for it would wait for all of them.
__device__ __forceinline__ v4f quad_of(const float* p, int q) {
    typedef const __attribute__((address_space(4))) float sfloat_t;
    sfloat_t* const s = reinterpret_cast<sfloat_t*>(reinterpret_cast<uintptr_t>(uniform_ptr(reinterpret_cast<const uint8_t*>(p))));
    v4f o;
#pragma unroll
    for (int c = 0; c < 4; ++c) o[c] = q == 0 ? s[c] : q == 1 ? s[4 + c] : q == 2 ? s[8 + c] : s[12 + c];
    return o;
}

// Token (or hidden) rows staged for a block: the most that any unit has,
// rounded up to one of these.  A 16-column MFMA with fewer rows repeats them;
// the columns past a unit's rows are never stored.
template <int NR> constexpr int kTiles = NR <= 16 ? 1 : NR / 16;

// Four fragments of one 16-column tile at the addresses a[0..3] plus OFS.
template <int OFS>
__device__ __forceinline__ void read4(u32x4 (&f)[4], const uint32_t (&a)[4]) {
    asm volatile(
        "ds_read_b128 %0, %4 offset:%c8\n\tds_read_b128 %1, %5 offset:%c8\n\t"
        "ds_read_b128 %2, %6 offset:%c8\n\tds_read_b128 %3, %7 offset:%c8\n\ts_waitcnt lgkmcnt(0)"
        : "=&v"(f[0]), "=&v"(f[1]), "=&v"(f[2]), "=&v"(f[3])
        : "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3]), "i"(OFS)
        : "memory");
}

// Weight rows (two 64-byte halves at w0, w1; GATE_UP: and 16 rows further on)
// and four fragments of a tile, with one wait.
template <int OFS>
__device__ __forceinline__ void read_weights(u32x4 (&w)[2], u32x4 (&f)[4], uint32_t w0, uint32_t w1, const uint32_t (&a)[4]) {
    asm volatile(
        "ds_read_b128 %0, %6\n\tds_read_b128 %2, %8 offset:%c12\n\tds_read_b128 %3, %9 offset:%c12\n\tds_read_b128 %1, %7\n\t"
        "ds_read_b128 %4, %10 offset:%c12\n\tds_read_b128 %5, %11 offset:%c12\n\ts_waitcnt lgkmcnt(0)"
        : "=&v"(w[0]), "=&v"(w[1]), "=&v"(f[0]), "=&v"(f[1]), "=&v"(f[2]), "=&v"(f[3])
        : "v"(w0), "v"(w1), "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3]), "i"(OFS)
        : "memory");
}
template <int OFS>
__device__ __forceinline__ void read_weights(u32x4 (&w)[4], u32x4 (&f)[4], uint32_t w0, uint32_t w1, const uint32_t (&a)[4]) {
    asm volatile(
        "ds_read_b128 %0, %8\n\tds_read_b128 %1, %9\n\tds_read_b128 %2, %8 offset:2048\n\tds_read_b128 %3, %9 offset:2048\n\t"
        "ds_read_b128 %4, %10 offset:%c14\n\tds_read_b128 %5, %11 offset:%c14\n\tds_read_b128 %6, %12 offset:%c14\n\t"
        "ds_read_b128 %7, %13 offset:%c14\n\ts_waitcnt lgkmcnt(0)"
        : "=&v"(w[0]), "=&v"(w[1]), "=&v"(w[2]), "=&v"(w[3]), "=&v"(f[0]), "=&v"(f[1]), "=&v"(f[2]), "=&v"(f[3])
        : "v"(w0), "v"(w1), "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3]), "i"(OFS)
        : "memory");
}

__device__ __forceinline__ uint32_t lds_addr(GFG_LDS uint8_t* p) { return uint32_t(reinterpret_cast<uintptr_t>(p)); }

// ---- hidden rows: h = silu(g) * u.
//
// A work item is 16 columns of I for one unit: the 16 gate rows and the 16 up
// rows of W1.  The four waves split H: wave w takes blocks w, w + 4, ...  LDS
// stage: 32 weight rows of 128 bytes, 16-byte chunks XOR-swizzled by row & 7,
// then NR token rows of 256 bytes, chunks XOR-swizzled by row & 15.  Weight
// chunk c of a row (16 k's) meets the token chunks 2 c and 2 c + 1: the MFMA's
// k order is a permutation that both operands share.
template <int W, typename A, int NR>
__device__ __forceinline__ void up_items(const MoeParams& p, const GFG_LDS Routing* r, GFG_LDS uint8_t* ring, GFG_LDS v4f* red) {
    typedef typename Vec<A>::v8 v8;
    constexpr int NT = kTiles<NR>, XL = NR / 4, PER = 4 + XL, STAGE = PER * 1024;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, lq = lane >> 4;
    const int KB = p.H / 128, IT = p.I / 16;
    const int items = __builtin_amdgcn_readfirstlane(r->units) * IT;
    const int depth = min(p.ring / STAGE, kMaxDepth);
    ring += wave * p.ring;
    const auto rx = make_rsrc(p.x, uint32_t(p.T) * uint32_t(p.H) * 2u);

    // ---- the loads' cursor: item, block, stage
    const uint32_t woff = uint32_t(lane >> 3) * uint32_t(p.H) + uint32_t(((lane & 7) ^ (lane >> 3)) * 16);
    uint32_t xoff[XL];
    __amdgpu_buffer_rsrc_t rg = make_rsrc(p.w1, 0), ru = make_rsrc(p.w1, 0);
    int li = wave < KB ? int(blockIdx.x) : items, lk = wave, ls = 0;
    // past the last item the windows are empty: the loads stay in the stream,
    // so that every wait counts alike, and touch nothing
    auto enter = [&]() {
        uint32_t window = 0;
        const uint8_t* base = p.w1;
        Unit un{0, 0, 0};
        if (li < items) {
            const int u = li / IT, it = li - u * IT;
            un = unit_of(r, u);
            base += (int64_t(un.e) * 2 * p.I + it * 16) * p.H;
            window = 16u * uint32_t(p.H);
        }
        rg = make_rsrc(base, window);
        ru = make_rsrc(base + int64_t(p.I) * p.H, window);
#pragma unroll
        for (int j = 0; j < XL; ++j) {
            const int row = 4 * j + (lane >> 4);
            xoff[j] = row < un.rows ? uint32_t(r->list[un.first + row] / p.k) * uint32_t(p.H) * 2u + uint32_t(((lane & 15) ^ (row & 15)) * 16)
                                    : kOutside;
        }
    };
    enter();
    auto issue = [&]() {
        GFG_LDS uint8_t* const dst = ring + ls * STAGE;
        const uint32_t kw = uint32_t(lk) * 128u, kx = uint32_t(lk) * 256u;
#pragma unroll
        for (int j = 0; j < 4; ++j) dma(j < 2 ? rg : ru, dst + j * 1024, woff + kw + uint32_t(8 * (j & 1)) * uint32_t(p.H));
#pragma unroll
        for (int j = 0; j < XL; ++j) dma(rx, dst + (4 + j) * 1024, xoff[j] + kx);
        ls = ls + 1 == depth ? 0 : ls + 1;
        lk += NW;
        if (lk >= KB) {
            lk = wave;
            li += gridDim.x;
            enter();
        }
    };
    for (int d = 0; d < depth; ++d) issue();

    // fragment addresses in stage 0
    const uint32_t w0 = lds_addr(ring) + uint32_t(l16 * 128 + ((lq ^ (l16 & 7)) << 4)), w1 = w0 ^ 64u;
    const int xr = l16 & (NR - 1) & 15;
    const uint32_t x0 = lds_addr(ring) + 4096u + uint32_t(xr * 256) + uint32_t(((2 * lq) ^ xr) << 4);
    int cs = 0;
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const int u = item / IT, it = item - u * IT;
        const Unit un = unit_of(r, u);
        const int sb = p.I / 128;              // 128-row scale blocks of the gate half
        const uint8_t* const sg = uniform_ptr(static_cast<const uint8_t*>(p.s1) + (int64_t(un.e) * 2 * sb + it / 8) * KB);
        const uint8_t* const su = uniform_ptr(sg + int64_t(sb) * KB);
        v4f acc[2][NT] = {};
        for (int kb = wave; kb < KB; kb += NW) {
            int bg = 0, bu = 0;
            if constexpr (W == FP8) {
                bg = load_scale_word(sg, kb);
                bu = load_scale_word(su, kb);
            }
            __builtin_amdgcn_sched_barrier(0);
            wait_stage<PER>(depth);
            const uint32_t so = uint32_t(cs * STAGE);
            const uint32_t xa[4] = {x0 + so, (x0 ^ 16u) + so, (x0 ^ 128u) + so, (x0 ^ 144u) + so};   // [64-byte half][8 elements]
            u32x4 w[4], x[NT][4];
            read_weights<0>(w, x[0], w0 + so, w1 + so, xa);
            if constexpr (NT > 1) read4<4096>(x[1], xa);
            __builtin_amdgcn_sched_barrier(0);
            issue();                           // into the stage just read
            __builtin_amdgcn_sched_barrier(0);
            cs = cs + 1 == depth ? 0 : cs + 1;
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
                        const v8 a = widen<W, A>(w[2 * f + j][2 * q], w[2 * f + j][2 * q + 1]);
#pragma unroll
                        for (int t = 0; t < NT; ++t) part[f][t] = mma(a, __builtin_bit_cast(v8, x[t][2 * j + q]), part[f][t]);
                    }
            const float sc[2] = {e8m0(uint32_t(scale_byte(bg, sg, kb))), e8m0(uint32_t(scale_byte(bu, su, kb)))};
#pragma unroll
            for (int f = 0; f < 2; ++f)
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    if constexpr (W == FP8) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[f][t][i] = fmaf(part[f][t][i], sc[f], acc[f][t][i]);
                    } else {
                        acc[f][t] = part[f][t];
                    }
                }
        }
        // the waves' sums meet in LDS; wave t finishes token tile t
        GFG_WAITCNT(63, 0);
        __builtin_amdgcn_s_barrier();          // the previous item's sums have been read
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
            for (int t = 0; t < NT; ++t) red[((wave * 2 + f) * NT + t) * 64 + lane] = acc[f][t];
        GFG_WAITCNT(63, 0);
        __builtin_amdgcn_s_barrier();
        const int i = 16 * wave + l16;
        if (wave >= NT || i >= un.rows) continue;
        v4f g = {}, v = {};
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            g += red[((w * 2) * NT + wave) * 64 + lane];
            v += red[((w * 2 + 1) * NT + wave) * 64 + lane];
        }
        const int col = it * 16 + lq * 4;
        if constexpr (W == INT8) {
            const float* sc = static_cast<const float*>(p.s1) + int64_t(un.e) * 2 * p.I + it * 16;
            const v4f cg = quad_of(sc, lq), cu = quad_of(sc + p.I, lq);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                g[c] *= cg[c];
                v[c] *= cu[c];
            }
        }
        // h in two bf16 halves, high and low: 16 significant bits with fp32's
        // range, so that the only rounding to 16 bits is the output's
        bf4 hi, lo;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float h = g[c] / (1.0f + expf(-g[c])) * v[c];
            hi[c] = __bf16(h);
            const float rest = h - float(hi[c]);
            lo[c] = __bf16(rest == rest ? rest : 0.0f);   // an infinite h has no low half
        }
        uint8_t* const row = p.h + int64_t(r->list[un.first + i]) * 4 * p.I + col * 2;
        *reinterpret_cast<bf4*>(row) = hi;
        *reinterpret_cast<bf4*>(row + 2 * p.I) = lo;
    }
}

template <int W, typename A>
__global__ __launch_bounds__(NT_THREADS) void moe_up_kernel(MoeParams p) {
    __shared__ Routing routing;
    __shared__ v4f red_mem[NW * 2 * kTiles<kUnitRows> * 64];
    extern __shared__ __attribute__((aligned(1024))) uint8_t ring_mem[];      // [NW][ring]
    GFG_LDS Routing* const r = (GFG_LDS Routing*)&routing;
    GFG_LDS v4f* const red = (GFG_LDS v4f*)red_mem;
    GFG_LDS uint8_t* const ring = (GFG_LDS uint8_t*)ring_mem;
    build_routing(r, ring, p.ids, p.T * p.k, p.E, p.unit_rows);
    const int most = __builtin_amdgcn_readfirstlane(r->most);
    if (most <= 4) up_items<W, A, 4>(p, r, ring, red);
    else if (most <= 8) up_items<W, A, 8>(p, r, ring, red);
    else if (most <= 16) up_items<W, A, 16>(p, r, ring, red);
    else up_items<W, A, 32>(p, r, ring, red);
    GFG_WAITCNT(0, 0);                         // the last loads land before the workgroup ends
}

// ---- down projection: 16 output columns (rows of W2) for all tokens.
//
// A workgroup walks all units; wave w takes units (w / ks), + NW / ks, ... and
// of their I the blocks w % ks, + ks, ...  Every (part, pair) sum goes to its
// own place in LDS, and the tokens' weighted sums are taken from there in the
// order of j: no atomics, and the result does not depend on the routing's list
// order.  LDS stage: 16 weight rows of 128 bytes, then the high halves of NR
// hidden rows of 256 bytes, then their low halves.
template <int W, int NR>
__device__ __forceinline__ void down_tile(const MoeParams& p, const GFG_LDS Routing* r, GFG_LDS uint8_t* ring, uint32_t y, int tile) {
    constexpr int NT = kTiles<NR>, HL = NR / 4, PER = 2 + 2 * HL, STAGE = PER * 1024;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, lq = lane >> 4;
    const int KB = p.I / 128, P = p.T * p.k;
    const int part = wave % p.ks, stride = NW / p.ks;
    const int units = __builtin_amdgcn_readfirstlane(r->units);
    const int depth = min(min(p.ring / STAGE, kMaxDepth), 63 / PER + 1);
    ring += wave * p.ring;
    const auto rh = make_rsrc(p.h, uint32_t(P) * 4u * uint32_t(p.I));

    const uint32_t woff = uint32_t(lane >> 3) * uint32_t(p.I) + uint32_t(((lane & 7) ^ (lane >> 3)) * 16);
    uint32_t hoff[HL];
    __amdgpu_buffer_rsrc_t rw = make_rsrc(p.w2, 0);
    int lu = wave / p.ks, lk = part, ls = 0;
    auto enter = [&]() {
        uint32_t window = 0;
        const uint8_t* base = p.w2;
        Unit un{0, 0, 0};
        if (lu < units) {
            un = unit_of(r, lu);
            base += (int64_t(un.e) * p.H + tile * 16) * p.I;
            window = 16u * uint32_t(p.I);
        }
        rw = make_rsrc(base, window);
#pragma unroll
        for (int j = 0; j < HL; ++j) {
            const int row = 4 * j + (lane >> 4);
            hoff[j] = row < un.rows ? uint32_t(r->list[un.first + row]) * 4u * uint32_t(p.I) + uint32_t(((lane & 15) ^ (row & 15)) * 16)
                                    : kOutside;
        }
    };
    enter();
    auto issue = [&]() {
        GFG_LDS uint8_t* const dst = ring + ls * STAGE;
        const uint32_t kw = uint32_t(lk) * 128u, kh = uint32_t(lk) * 256u;
#pragma unroll
        for (int j = 0; j < 2; ++j) dma(rw, dst + j * 1024, woff + kw + uint32_t(8 * j) * uint32_t(p.I));
#pragma unroll
        for (int pl = 0; pl < 2; ++pl)
#pragma unroll
            for (int j = 0; j < HL; ++j) dma(rh, dst + (2 + pl * HL + j) * 1024, hoff[j] + kh + uint32_t(pl) * 2u * uint32_t(p.I));
        ls = ls + 1 == depth ? 0 : ls + 1;
        lk += p.ks;
        if (lk >= KB) {
            lk = part;
            lu += stride;
            enter();
        }
    };
    for (int d = 0; d < depth; ++d) issue();

    const uint32_t w0 = lds_addr(ring) + uint32_t(l16 * 128 + ((lq ^ (l16 & 7)) << 4)), w1 = w0 ^ 64u;
    const int hr = l16 & (NR - 1) & 15;
    const uint32_t h0 = lds_addr(ring) + 2048u + uint32_t(hr * 256) + uint32_t(((2 * lq) ^ hr) << 4);
    int cs = 0;
    for (int u = wave / p.ks; u < units; u += stride) {
        const Unit un = unit_of(r, u);
        const uint8_t* const srow = uniform_ptr(static_cast<const uint8_t*>(p.s2) + (int64_t(un.e) * (p.H / 128) + tile / 8) * KB);
        v4f acc[NT] = {};
        for (int kb = part; kb < KB; kb += p.ks) {
            int b = 0;
            if constexpr (W == FP8) b = load_scale_word(srow, kb);
            __builtin_amdgcn_sched_barrier(0);
            wait_stage<PER>(depth);
            const uint32_t so = uint32_t(cs * STAGE);
            const uint32_t ha[4] = {h0 + so, (h0 ^ 16u) + so, (h0 ^ 128u) + so, (h0 ^ 144u) + so};   // [64-byte half][8 elements]
            u32x4 w[2], h[NT][2][4];           // [tile][high, low][half, 8 elements]
            read_weights<0>(w, h[0][0], w0 + so, w1 + so, ha);
            read4<HL * 1024>(h[0][1], ha);
            if constexpr (NT > 1) {
                read4<4096>(h[1][0], ha);
                read4<HL * 1024 + 4096>(h[1][1], ha);
            }
            __builtin_amdgcn_sched_barrier(0);
            issue();                           // into the stage just read
            __builtin_amdgcn_sched_barrier(0);
            cs = cs + 1 == depth ? 0 : cs + 1;
            v4f sum[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) sum[t] = W == FP8 ? v4f{} : acc[t];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const bf8 a = widen<W, __bf16>(w[j][2 * q], w[j][2 * q + 1]);
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int pl = 0; pl < 2; ++pl) sum[t] = mma(a, __builtin_bit_cast(bf8, h[t][pl][2 * j + q]), sum[t]);
                }
            const float sc = e8m0(uint32_t(scale_byte(b, srow, kb)));
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if constexpr (W == FP8) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[t][i] = fmaf(sum[t][i], sc, acc[t][i]);
                } else {
                    acc[t] = sum[t];
                }
            }
        }
        // (in assembly for the same reason as the reads: no wait for the loads in flight)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int i = 16 * t + l16;
            if (i < un.rows) {
                const uint32_t at = y + uint32_t((part * P + r->list[un.first + i]) * 64 + lq * 16);
                asm volatile("ds_write_b128 %0, %1" : : "v"(at), "v"(acc[t]) : "memory");
            }
        }
    }
}

template <int W, typename OutT>
__global__ __launch_bounds__(NT_THREADS) void moe_down_kernel(MoeParams p) {
    __shared__ Routing routing;
    extern __shared__ __attribute__((aligned(1024))) uint8_t ring_mem[];      // [NW][ring], then sums [ks][T * k][16 columns]
    GFG_LDS Routing* const r = (GFG_LDS Routing*)&routing;
    GFG_LDS uint8_t* const ring = (GFG_LDS uint8_t*)ring_mem;
    GFG_LDS v4f* const y = (GFG_LDS v4f*)(ring + NW * p.ring);
    const int P = p.T * p.k;
    build_routing(r, ring, p.ids, P, p.E, p.unit_rows);
    const int most = __builtin_amdgcn_readfirstlane(r->most);
    typedef OutT o4 __attribute__((ext_vector_type(4)));
    for (int tile = blockIdx.x; tile < p.H / 16; tile += gridDim.x) {
        const uint32_t ya = lds_addr((GFG_LDS uint8_t*)y);
        if (most <= 4) down_tile<W, 4>(p, r, ring, ya, tile);
        else if (most <= 8) down_tile<W, 8>(p, r, ring, ya, tile);
        else if (most <= 16) down_tile<W, 16>(p, r, ring, ya, tile);
        else down_tile<W, 32>(p, r, ring, ya, tile);
        GFG_WAITCNT(0, 0);                     // the last loads have landed, the sums are written
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
int launch_layer(MoeParams p, hipStream_t s) {
    int cus = 0;
    if (int rc = device_cus(&cus)) return rc;
    const int P = p.T * p.k;
    static const char* v1 = getenv("MOE_UP"); static const char* v2 = getenv("MOE_DN");
    const int r1 = v1 ? atoi(v1) : 14, r2 = v2 ? atoi(v2) : 14;
    p.ring = r1 * 1024;
    p.unit_rows = p.T <= 4 ? 4 : p.T <= 8 ? 8 : p.T <= 16 ? 16 : 32;
    const int64_t up_items = int64_t(P < p.E ? P : p.E) * (p.I / 16) + int64_t(P / p.unit_rows) * (p.I / 16);
    const int per = r1 > 16 ? 1 : 2, per2 = r2 > 16 ? 1 : 2;
    const int up_grid = int(up_items < per * cus ? up_items : per * cus);
    hipLaunchKernelGGL((moe_up_kernel<W, A>), dim3(up_grid), dim3(NT_THREADS), unsigned(NW * p.ring), s, p);
    const int tiles = p.H / 16, down_grid = tiles < per2 * cus ? tiles : per2 * cus;
    p.ring = r2 * 1024;
    if (p.unit_rows == 32 && p.ring < 18 * 1024) p.ring = 18 * 1024;
    hipLaunchKernelGGL((moe_down_kernel<W, A>), dim3(down_grid), dim3(NT_THREADS), unsigned(NW * p.ring + p.ks * P * 64), s, p);
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
                static_cast<uint8_t*>(workspace), out, int(T), int(k), int(E), int(H), int(I), 0, kUnitRows, 1};
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
