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
// weighted sum of their down projections; where the experts' items are shared
// out over the CUs (shared_down), that sum is a launch of its own.  Measured in a
// trace, us up / down (/ sum): one token, k = 9, E = 385, H = 7168, I = 512, FP8: 18 /
// 11 (99 MB); 32 tokens of it: 246-274 / 135-148 (2.25 GB, 5.0-5.6 TB/s); 100 tokens,
// k = 2, E = 8, H = 4096, I = 1792, FP8: 35-37 / 19-22 / 4.5 (178 MB); 5 tokens, k = 6,
// E = 64, H = 2048, I = 1408, int8: 31-33 / 20 / 4.5 (216 MB).
#include <hip/hip_runtime.h>

#include <cstdint>
#include <cmath>

#include "gfg.h"
#include "gfg_device.h"
#include "gfg_internal.h"

namespace gfg {
namespace {

// ------------------------------------------------------------------ router
constexpr int kMaxExperts = 1024;
constexpr int64_t kMostWorkgroups = 1 << 20;   // of the router; each walks on where there are more tokens

__device__ __forceinline__ float as_f32(float v) { return v; }
__device__ __forceinline__ float as_f32(__bf16 v) { return float(v); }
__device__ __forceinline__ float as_f32(_Float16 v) { return float(v); }

__device__ __forceinline__ float wave_max(float v) { return wave_reduce(v, [](float a, float b) { return fmaxf(a, b); }); }
__device__ __forceinline__ float wave_sum(float v) { return wave_reduce(v, [](float a, float b) { return a + b; }); }
__device__ __forceinline__ int wave_min(int v) { return wave_reduce(v, [](int a, int b) { return min(a, b); }); }

// One wave a token; lane l holds experts l, l + 64, ... (EPL of them).  A round
// takes the largest remaining selection value and, among its holders, the
// lowest index; lane j keeps the result of round j.  The rounds are a chain of
// wave reductions, which stay in registers (DPP rotations; through LDS they cost
// twice as much): 3.8 us for one token of 256 experts, k = 8, of which 2.5 are the
// launch; 8.3-9.2 us for 4096 tokens of 385 in fp32, k = 9 (6.6 MB: 0.7-0.8 TB/s),
// bound by those chains.
template <typename T, int EPL>
__device__ __forceinline__ void topk_row(const T* __restrict__ row, const float* __restrict__ bias, int32_t* __restrict__ ids,
                                         float* __restrict__ weights, int lane, int E, int k, bool sigmoid, bool renorm,
                                         float scale) {
    const float ninf = -__builtin_inff();
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
    float logit = ninf;
    for (int j = 0; j < k; ++j) {
        float best = ninf, held = ninf;
        int at = 0x7FFFFFFF;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (s[i] > best) { best = s[i]; held = l[i]; at = lane + 64 * i; }
        const float top = wave_max(best);
        if (top == ninf) break;                // nothing above -infinity is left
        const uint64_t holders = __ballot(best == top);
        const int e = __popcll(holders) == 1 ? __builtin_amdgcn_readlane(at, __builtin_ctzll(holders))
                                             : wave_min(best == top ? at : 0x7FFFFFFF);
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (e == lane + 64 * i) s[i] = ninf;
        const float v = __uint_as_float(uint32_t(__builtin_amdgcn_readlane(int(__float_as_uint(held)), e & 63)));
        if (lane == j) { mine = e; logit = v; }
    }
    float w = 0.0f;
    if (mine >= 0) {
        w = sigmoid ? sig(logit) : expo(logit) / total;
    }
    if (renorm) {
        const float sum = wave_sum(w);
        w = sum > 0.0f ? w / sum : 0.0f;
    }
    if (lane < k) {
        ids[lane] = mine;
        weights[lane] = w * scale;
    }
}

template <typename T, int EPL>
__global__ __launch_bounds__(256) void moe_topk_kernel(const T* __restrict__ logits, const float* __restrict__ bias,
                                                       int32_t* __restrict__ ids, float* __restrict__ weights,
                                                       int64_t tokens, int E, int k, bool sigmoid, bool renorm,
                                                       float scale) {
    const int lane = threadIdx.x & 63;
    for (int64_t t = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6); t < tokens; t += int64_t(gridDim.x) * 4)
        topk_row<T, EPL>(logits + t * E, bias, ids + t * k, weights + t * k, lane, E, k, sigmoid, renorm, scale);
}

template <typename T>
void launch_topk(const void* logits, const float* bias, int32_t* ids, float* weights, int64_t tokens, int E, int k,
                 bool sigmoid, bool renorm, float scale, hipStream_t s) {
    const int64_t wgs = (tokens + 3) / 4;
    const dim3 grid(unsigned(wgs < kMostWorkgroups ? wgs : kMostWorkgroups));
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
constexpr int kWaves = 8;
constexpr int kMaxPairs = 1024;
constexpr int kSmallPairs = 32;                // up to these the routing is built by a wave alone
constexpr int kScaleBytes = 512;               // scales of a stage (see below)
constexpr int kMaxDim = 252 * 128;             // H and I: the words of a scale row fit a wave's lanes
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
    float* y;                // [T*k][H]: the pairs' outputs, where they are summed by a launch of their own
    void* out;               // [T][H]
    int T, k, E, H, I;
    int ring;                // bytes of each wave's ring
    int resident;            // bytes of the rows that stay in LDS, in whole loads; 0: they go through the ring
    int ks_most;             // down projection: most waves that may split an expert's I
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
// (t * k + j) expert by expert, unit[] the stretches of at most `rows` of
// them: expert | first << 10 | (rows - 1) << 20.  Ids outside [0, E) are in no
// unit.  Every workgroup builds its own copy, so the copies have to agree on
// which pairs a unit holds: an expert of one unit may list its pairs in the
// order of the LDS atomics (a pair's sums never mix with another's), an expert
// of several lists them in their own order.
struct Routing {
    int16_t list[kMaxPairs];
    uint32_t unit[kMaxPairs];
    int tmp[8];
    int total[6];            // units if they had at most 2, 4, 8, 16, 32, 64 pairs
    int units;
};
constexpr int kBuildBytes = kMaxExperts * 4 + kMaxPairs * 2;    // scratch of the build

// Units of at most LO .. HI pairs (powers of two): the largest size that leaves
// room for two stages in the ring reads an expert's weights the fewest times;
// of the sizes that make hardly more units (1/64), the smallest stages the
// fewest rows that do not exist.  A stage: `fixed` KB of weights, `per4` KB for
// every four rows.
template <int LO, int HI>
__device__ __forceinline__ int choose_rows(const int (&total)[6], int fixed, int per4, int ring) {
    int rows = LO, fewest = 0;
#pragma unroll
    for (int i = 5; i >= 0; --i) {
        const int r = 2 << i;
        if (r < LO || r > HI || (r > LO && 2 * ((fixed + per4 * r / 4) * 1024 + kScaleBytes) > ring)) continue;
        if (fewest == 0) fewest = total[i] + total[i] / 64;
        if (total[i] <= fewest) rows = r;
    }
    return rows;
}

// Up to kSmallPairs pairs: lane p of every wave holds pair p, and no barrier
// but the last is needed.  choose(total) gives the unit size, which is returned.
template <typename Choose>
__device__ __forceinline__ int build_small(GFG_LDS Routing* r, const int32_t* ids, int P, int E, Choose choose) {
    const int lane = threadIdx.x & 63;
    int e = lane < P ? ids[lane] : -1;
    const bool live = e >= 0 && e < E;
    if (!live) e = -1;
    uint64_t same = 0;                         // the pairs of this lane's expert
    for (int q = 0; q < P; ++q) {
        const uint64_t m = __ballot(__builtin_amdgcn_readlane(e, q) == e);
        same = lane == q ? m : same;
    }
    const int lead = __builtin_ctzll(same | 1ull << 63), count = __popcll(same);
    const int before = __popcll(same & ((1ull << lane) - 1));
    int total[6];
#pragma unroll
    for (int i = 0; i < 6; ++i) total[i] = __popcll(__ballot(live && (before & ((2 << i) - 1)) == 0));
    const int rows = choose(total);
    // pairs | units << 16 of the experts whose first pair lies before this lane
    const int own = live && lane == lead ? count | ((count + rows - 1) / rows) << 16 : 0;
    int x = own;
#pragma unroll
    for (int d = 1; d < kSmallPairs; d <<= 1) {
        const int y = __shfl_up(x, d, 64);
        if (lane >= d) x += y;
    }
    const int base = __shfl(x - own, lead, 64);
    const int units = __shfl(x, kSmallPairs - 1, 64) >> 16;
    if (threadIdx.x < 64) {
        const int first = base & 0xFFFF;
        if (live) r->list[first + before] = int16_t(lane);
        if (live && before % rows == 0)
            r->unit[(base >> 16) + before / rows] =
                uint32_t(e) | uint32_t(first + before) << 10 | uint32_t(min(count - before, rows) - 1) << 20;
        if (lane == 0) r->units = units;
    }
    __syncthreads();
    return rows;
}

template <typename Choose>
__device__ __forceinline__ int build_routing(GFG_LDS Routing* r, GFG_LDS uint8_t* scratch, const int32_t* ids, int P, int E,
                                             Choose choose) {
    if (P <= kSmallPairs) return build_small(r, ids, P, E, choose);
    GFG_LDS int* const cnt = reinterpret_cast<GFG_LDS int*>(scratch);                    // [kMaxExperts]
    GFG_LDS int16_t* const expert = reinterpret_cast<GFG_LDS int16_t*>(cnt + kMaxExperts);   // [kMaxPairs]
    constexpr int THREADS = kWaves * 64, PPT = kMaxPairs / THREADS, EPT = kMaxExperts / THREADS;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int e[PPT], slot[PPT];
#pragma unroll
    for (int i = 0; i < PPT; ++i) {
        const int p = tid + i * THREADS;
        e[i] = p < P ? ids[p] : -1;
    }
    if (tid < 6) r->total[tid] = 0;
#pragma unroll
    for (int i = 0; i < EPT; ++i) cnt[tid * EPT + i] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PPT; ++i) {
        slot[i] = -1;
        if (e[i] < 0 || e[i] >= E) e[i] = -1;
        expert[tid + i * THREADS] = int16_t(e[i]);
        if (e[i] >= 0) slot[i] = __hip_atomic_fetch_add(&cnt[e[i]], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    }
    __syncthreads();
    int c[EPT];
    int sums[6] = {};                          // units of at most 2, 4, ... 64 pairs
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
        c[i] = cnt[tid * EPT + i];
#pragma unroll
        for (int z = 0; z < 6; ++z) sums[z] += (c[i] + (2 << z) - 1) >> (1 + z);
    }
    if (sums[5]) {
#pragma unroll
        for (int z = 0; z < 6; ++z)
            __hip_atomic_fetch_add(&r->total[z], sums[z], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    }
    __syncthreads();
    int total[6];
#pragma unroll
    for (int z = 0; z < 6; ++z) total[z] = __builtin_amdgcn_readfirstlane(r->total[z]);
    const int rows = choose(total);
#pragma unroll
    for (int i = 0; i < PPT; ++i)
        if (slot[i] >= 0 && cnt[e[i]] > rows) {
            const int p = tid + i * THREADS;
            int before = 0;                    // earlier pairs of the expert, eight at a time
            for (int q = 0; q < p; q += 8) {
                const u32x4 v = *reinterpret_cast<GFG_LDS u32x4*>(expert + q);
#pragma unroll
                for (int c = 0; c < 8; ++c) before += q + c < p && int(v[c >> 1] >> (16 * (c & 1)) & 0xFFFF) == e[i];
            }
            slot[i] = before;
        }
    int mine = 0;                              // pairs | units << 16 of this thread's experts
#pragma unroll
    for (int i = 0; i < EPT; ++i) mine += c[i] | ((c[i] + rows - 1) / rows) << 16;
    int x = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int y = __shfl_up(x, d, 64);
        if (lane >= d) x += y;
    }
    if (lane == 63) r->tmp[wave] = x;
    __syncthreads();
    int before = x - mine;
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
        if (w < wave) before += r->tmp[w];
    int first = before & 0xFFFF, u = before >> 16;
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
        const int ex = tid * EPT + i;
        cnt[ex] = first;
        for (int done = 0; done < c[i]; done += rows)
            r->unit[u++] = uint32_t(ex) | uint32_t(first + done) << 10 | uint32_t(min(c[i] - done, rows) - 1) << 20;
        first += c[i];
    }
    if (tid == THREADS - 1) r->units = u;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PPT; ++i)
        if (slot[i] >= 0) r->list[cnt[e[i]] + slot[i]] = int16_t(tid + i * THREADS);
    __syncthreads();
    return rows;
}

struct Unit { int e, first, rows; };
__device__ __forceinline__ Unit unit_of(const GFG_LDS Routing* r, int u) {
    const uint32_t w = __builtin_amdgcn_readfirstlane(r->unit[u]);
    return Unit{int(w & 0x3FF), int((w >> 10) & 0x3FF), int(w >> 20) + 1};
}

// ---- what both kernels share: a wave's ring.
//
// A wave streams 128-byte blocks of 16 or 32 weight rows through its own ring
// of LDS stages filled by direct-to-LDS loads, up to kMaxDepth stages ahead
// and across the ends of experts and tiles; no barrier stands between a load
// and its MFMAs.  Whole 128-byte lines by adjacent lanes: loaded straight into
// MFMA fragments, adjacent lanes are adjacent rows, and a load takes four times
// as long.  What bounds the kernels: HBM where the launch is long (32 tokens, k = 9,
// E = 385, H = 7168, I = 512: 5.6 TB/s up and 5.1 down by the traffic counters).  The
// short ones reach 3.0-4.4 TB/s and 12-19 GB/s into each CU, with the matrix pipes 2-11%
// busy and half of the waves' time spent waiting for memory: some 5 us of
// launch, routing and the first loads' way (an up launch of 16 items takes 7.5 us),
// then the latency of each wave's chain of stages.  So what goes beside the weights
// is kept small: the tokens' rows stay in LDS for the whole launch where they are
// small, else the stage holds only as many of them as units have; an expert's
// scales come once for a unit.
//
// The fragments are read from LDS in inline assembly, each group together with
// its wait: the stage index is a run-time value, so the compiler, which cannot
// tell the stages apart, would make its own LDS reads wait for every load in
// flight.

// Wait until at most (depth - 1) * PER vector-memory operations are in flight:
// the stage loaded depth - 1 stages ago has landed.  (Loads beside the PER of a
// stage only make the wait stricter.)
template <int PER>
__device__ __forceinline__ void wait_stage(int depth) {
#define GFG_AHEAD(D) ((D) * PER < 63 ? (D) * PER : 63)
    switch (depth) {
        case 1: GFG_WAITCNT(0, 15); break;
        case 2: GFG_WAITCNT(GFG_AHEAD(1), 15); break;
        case 3: GFG_WAITCNT(GFG_AHEAD(2), 15); break;
        case 4: GFG_WAITCNT(GFG_AHEAD(3), 15); break;
        case 5: GFG_WAITCNT(GFG_AHEAD(4), 15); break;
        case 6: GFG_WAITCNT(GFG_AHEAD(5), 15); break;
        default: GFG_WAITCNT(GFG_AHEAD(6), 15); break;
    }
#undef GFG_AHEAD
}

__device__ __forceinline__ void dma(__amdgpu_buffer_rsrc_t r, GFG_LDS uint8_t* dst, uint32_t off) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (GFG_LDS void*)dst, 16, off, 0, 0, 0);
}
__device__ __forceinline__ void dma4(__amdgpu_buffer_rsrc_t r, GFG_LDS uint8_t* dst, uint32_t off) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (GFG_LDS void*)dst, 4, off, 0, 0, 0);
}
__device__ __forceinline__ uint32_t lds_addr(GFG_LDS uint8_t* p) { return uint32_t(reinterpret_cast<uintptr_t>(p)); }

// Scales.  A unit's first stage also carries them, behind its rows.  FP8: the
// aligned words of the whole scale row (all K blocks of a 128-row block), one a
// lane, read into a register and picked by lane when their block comes.  INT8:
// a float for each output channel.
//
// A window over the whole scale tensor that starts on a word; `shift` is what
// that adds to the tensor's byte offsets.  (An aligned word that holds a byte
// of an allocation lies in that byte's page.)
__device__ __forceinline__ __amdgpu_buffer_rsrc_t scale_rsrc(const void* s, uint32_t bytes, uint32_t* shift) {
    const uintptr_t v = reinterpret_cast<uintptr_t>(s);
    *shift = uint32_t(v & 3);
    return make_rsrc(reinterpret_cast<const void*>(v & ~uintptr_t(3)), (bytes + *shift + 3) & ~3u);
}
// The scale of block kb of the row that starts at byte offset `row`, from the
// row's words (lane i: word i).
__device__ __forceinline__ float picked_scale(uint32_t words, uint32_t row, int kb) {
    const uint32_t at = row + uint32_t(kb);
    const uint32_t w = uint32_t(__builtin_amdgcn_readlane(int(words), int((at >> 2) - (row >> 2))));
    return e8m0((w >> (8 * (at & 3))) & 0xFF);
}
__device__ __forceinline__ uint32_t read_word(uint32_t at) {
    uint32_t v;
    asm volatile("ds_read_b32 %0, %1\n\ts_waitcnt lgkmcnt(0)" : "=&v"(v) : "v"(at) : "memory");
    return v;
}
__device__ __forceinline__ v4f read_quad(uint32_t at) {
    v4f v;
    asm volatile("ds_read_b128 %0, %1\n\ts_waitcnt lgkmcnt(0)" : "=&v"(v) : "v"(at) : "memory");
    return v;
}

// 16 or 32 weight rows (their 64-byte halves at w0 and w1) and the four
// fragments of the 16 columns beside them, with one wait.
__device__ __forceinline__ void read_block(u32x4 (&w)[2], u32x4 (&f)[4], uint32_t w0, uint32_t w1, const uint32_t (&a)[4]) {
    asm volatile(
        "ds_read_b128 %0, %6\n\tds_read_b128 %1, %7\n\tds_read_b128 %2, %8\n\tds_read_b128 %3, %9\n\t"
        "ds_read_b128 %4, %10\n\tds_read_b128 %5, %11\n\ts_waitcnt lgkmcnt(0)"
        : "=&v"(w[0]), "=&v"(w[1]), "=&v"(f[0]), "=&v"(f[1]), "=&v"(f[2]), "=&v"(f[3])
        : "v"(w0), "v"(w1), "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3])
        : "memory");
}
__device__ __forceinline__ void read_block(u32x4 (&w)[4], u32x4 (&f)[4], uint32_t w0, uint32_t w1, const uint32_t (&a)[4]) {
    asm volatile(
        "ds_read_b128 %0, %8\n\tds_read_b128 %1, %9\n\tds_read_b128 %2, %8 offset:2048\n\tds_read_b128 %3, %9 offset:2048\n\t"
        "ds_read_b128 %4, %10\n\tds_read_b128 %5, %11\n\tds_read_b128 %6, %12\n\tds_read_b128 %7, %13\n\ts_waitcnt lgkmcnt(0)"
        : "=&v"(w[0]), "=&v"(w[1]), "=&v"(w[2]), "=&v"(w[3]), "=&v"(f[0]), "=&v"(f[1]), "=&v"(f[2]), "=&v"(f[3])
        : "v"(w0), "v"(w1), "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3])
        : "memory");
}

// Four more fragments, OFS bytes further on.
template <int OFS>
__device__ __forceinline__ void read4(u32x4 (&f)[4], const uint32_t (&a)[4]) {
    asm volatile(
        "ds_read_b128 %0, %4 offset:%c8\n\tds_read_b128 %1, %5 offset:%c8\n\t"
        "ds_read_b128 %2, %6 offset:%c8\n\tds_read_b128 %3, %7 offset:%c8\n\ts_waitcnt lgkmcnt(0)"
        : "=&v"(f[0]), "=&v"(f[1]), "=&v"(f[2]), "=&v"(f[3])
        : "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3]), "i"(OFS)
        : "memory");
}

// Token rows of `bytes` (a multiple of 256) that stay in LDS, as they lie in
// memory, loaded by all waves; 16-byte chunks XOR-swizzled by row & 15.
__device__ __forceinline__ void load_resident(GFG_LDS uint8_t* dst, __amdgpu_buffer_rsrc_t r, int bytes, int total) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (int at = wave * 1024; at < total; at += kWaves * 1024) {
        const int b = at + lane * 16;
        dma(r, dst + at, uint32_t(b ^ (((b / bytes) & 15) << 4)));
    }
}

// h = silu(g) * u for four columns of a pair, in two bf16 halves, high and low:
// 16 significant bits with fp32's range, so that the only rounding to 16 bits
// is the output's.  (The sums over them are of raw codes, before their scales.)  A finite h above the largest bf16 keeps that as its high
// half and the rest as its low one; a NaN or an infinity has no low half.
__device__ __forceinline__ void store_hidden(const MoeParams& p, int pair, int col, const v4f& g, const v4f& u) {
    constexpr float kTop = 0x1.FEp127f;        // the largest bf16
    bf4 hi, lo;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const float h = g[c] / (1.0f + expf(-g[c])) * u[c];
        const bool finite = fabsf(h) < __builtin_inff();
        hi[c] = __bf16(finite ? fminf(fmaxf(h, -kTop), kTop) : h);
        lo[c] = __bf16(finite ? h - float(hi[c]) : 0.0f);
    }
    uint8_t* const row = p.h + int64_t(pair) * 4 * p.I + col * 2;
    *reinterpret_cast<bf4*>(row) = hi;
    *reinterpret_cast<bf4*>(row + 2 * p.I) = lo;
}

// ---- hidden rows: h = silu(g) * u.
//
// A work item is 16 columns of I for one unit: the 16 gate rows and the 16 up
// rows of W1, a fragment each.  The eight waves split H: wave w takes blocks w,
// w + 8, ...  LDS stage: 32 weight rows of 128 bytes, 16-byte chunks
// XOR-swizzled by row & 7, then (unless they are resident) NR token rows of 256
// bytes, chunks XOR-swizzled by row & 15.
// Weight chunk c of a row (16 k's) meets the token chunks 2 c and 2 c + 1: the
// MFMA's k order is a permutation that both operands share.  A unit has at most
// NR rows; the MFMA's other columns repeat them, and their sums are not stored.
template <int W, typename A, int NR, bool RES>
__device__ __forceinline__ void up_items(const MoeParams& p, const GFG_LDS Routing* r, GFG_LDS uint8_t* ring, GFG_LDS uint8_t* rows_mem,
                                         GFG_LDS v4f* red) {
    typedef typename Vec<A>::v8 v8;
    constexpr int C = 16, F = 2, WL = 4, XL = RES ? 0 : NR / 4, PER = WL + XL, STAGE = PER * 1024 + kScaleBytes;
    constexpr bool TWICE = NR <= 8;            // the waves' sums have room for two items
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, lq = lane >> 4;
    const int KB = p.H / 128, IT = p.I / C;
    const int items = __builtin_amdgcn_readfirstlane(r->units) * IT;
    const int depth = min(min(p.ring / STAGE, kMaxDepth), 63 / PER);
    ring += wave * p.ring;
    const auto rx = make_rsrc(p.x, uint32_t(p.T) * uint32_t(p.H) * 2u);

    // ---- the loads' cursor: item, block, stage
    const uint32_t woff = uint32_t(lane >> 3) * uint32_t(p.H) + uint32_t(((lane & 7) ^ (lane >> 3)) * 16);
    uint32_t xoff[XL ? XL : 1], soff[2] = {0, 0};
    uint32_t shift;
    const int sb = p.I / 128;                  // 128-row scale blocks of the gate half
    const auto rs = scale_rsrc(p.s1, W == FP8 ? uint32_t(p.E) * 2u * uint32_t(sb) * uint32_t(KB) : uint32_t(p.E) * 8u * uint32_t(p.I), &shift);
    __amdgpu_buffer_rsrc_t rg = make_rsrc(p.w1, 0), ru = make_rsrc(p.w1, 0);
    int li = wave < KB ? int(blockIdx.x) : items, lk = wave, ls = 0;
    bool fresh = true;                         // the next block is its item's first
    // past the last item the windows are empty: the loads stay in the stream,
    // so that every wait counts alike, and touch nothing
    auto enter = [&]() {
        uint32_t window = 0;
        const uint8_t* base = p.w1;
        Unit un{0, 0, 0};
        if (li < items) {
            const int u = li / IT, it = li - u * IT;
            un = unit_of(r, u);
            base += (int64_t(un.e) * 2 * p.I + it * C) * p.H;
            window = uint32_t(C) * uint32_t(p.H);
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                if constexpr (W == FP8)
                    soff[f] = ((uint32_t(un.e * 2 * sb + it * C / 128 + f * sb) * uint32_t(KB) + shift) & ~3u) + 4u * uint32_t(lane);
                else
                    soff[f] = lane < C ? uint32_t((un.e * 2 + f) * p.I + it * C + lane) * 4u : kOutside;
            }
        } else {
            soff[0] = soff[1] = kOutside;
        }
        rg = make_rsrc(base, window);
        ru = make_rsrc(base + int64_t(p.I) * p.H, window);
#pragma unroll
        for (int j = 0; j < XL; ++j) {
            const int row = 4 * j + (lane >> 4);
            xoff[j] = row < un.rows ? uint32_t(r->list[un.first + row] / p.k) * uint32_t(p.H) * 2u + uint32_t(((lane & 15) ^ (row & 15)) * 16)
                                    : kOutside;
        }
        fresh = true;
    };
    enter();
    auto issue = [&]() {
        GFG_LDS uint8_t* const dst = ring + ls * STAGE;
        const uint32_t kw = uint32_t(lk) * 128u, kx = uint32_t(lk) * 256u;
        if (fresh) {
            dma4(rs, dst + PER * 1024, soff[0]);
            dma4(rs, dst + PER * 1024 + 256, soff[1]);
            fresh = false;
        }
#pragma unroll
        for (int j = 0; j < WL; ++j)
            dma(j < WL / 2 ? rg : ru, dst + j * 1024, woff + kw + uint32_t(8 * (j % (WL / 2))) * uint32_t(p.H));
#pragma unroll
        for (int j = 0; j < XL; ++j) dma(rx, dst + (WL + j) * 1024, xoff[j] + kx);
        ls = ls + 1 == depth ? 0 : ls + 1;
        lk += kWaves;
        if (lk >= KB) {
            lk = wave;
            li += gridDim.x;
            enter();
        }
    };
    for (int d = 0; d < depth; ++d) issue();
    if constexpr (RES) {                       // the resident rows, loaded before the stages, have landed
        wait_stage<PER>(depth + 1);
        lds_barrier();
    }

    // fragment addresses in stage 0
    const uint32_t w0 = lds_addr(ring) + uint32_t(l16 * 128 + ((lq ^ (l16 & 7)) << 4)), w1 = w0 ^ 64u;
    const int xr = l16 & (NR - 1);
    const uint32_t x0 = lds_addr(ring) + uint32_t(WL * 1024 + xr * 256) + uint32_t(((2 * lq) ^ xr) << 4);
    int cs = 0, done = 0;
    for (int item = blockIdx.x; item < items; item += gridDim.x, ++done) {
        const int u = item / IT, it = item - u * IT;
        const Unit un = unit_of(r, u);
        // byte offsets of the item's gate and up scale rows
        const uint32_t sg = uint32_t(un.e * 2 * sb + it * C / 128) * uint32_t(KB) + shift, su = sg + uint32_t(sb) * uint32_t(KB);
        uint32_t wg = 0, wu = 0;               // FP8: their words
        v4f cg = {}, cu = {};                  // INT8: the channels' scales
        uint32_t xres = 0;                     // resident: this column's token row
        if constexpr (RES) {
            const int tok = r->list[un.first + min(xr, un.rows - 1)] / p.k;
            xres = lds_addr(rows_mem) + uint32_t(tok) * uint32_t(p.H) * 2u + uint32_t(((2 * lq) ^ (tok & 15)) << 4);
        }
        v4f acc[F] = {};
        // FP8: a block's sums take its scales when the next block's fragments
        // have been read, so that its MFMAs run under those reads
        v4f part[F] = {};
        float sc[2] = {0.0f, 0.0f};
        auto apply = [&]() {
#pragma unroll
            for (int f = 0; f < F; ++f)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[f][i] = fmaf(part[f][i], sc[f], acc[f][i]);
        };
        for (int kb = wave; kb < KB; kb += kWaves) {
            __builtin_amdgcn_sched_barrier(0);
            wait_stage<PER>(depth);
            const uint32_t so = uint32_t(cs * STAGE);
            const uint32_t xb = RES ? xres + uint32_t(kb) * 256u : x0 + so;
            const uint32_t xa[4] = {xb, xb ^ 16u, xb ^ 128u, xb ^ 144u};    // [64-byte half][8 elements]
            u32x4 w[WL], x[4];
            if (kb == wave) {                  // the item's scales
                const uint32_t sa = lds_addr(ring) + so + PER * 1024u;
                if constexpr (W == FP8) {
                    wg = read_word(sa + uint32_t(lane * 4));
                    wu = read_word(sa + 256u + uint32_t(lane * 4));
                } else {                       // lanes of the finishing step's rows: see there
                    cg = read_quad(sa + uint32_t(lq * 16));
                    cu = read_quad(sa + 256u + uint32_t(lq * 16));
                }
            }
            read_block(w, x, w0 + so, w1 + so, xa);
            __builtin_amdgcn_sched_barrier(0);
            issue();                           // into the stage just read
            __builtin_amdgcn_sched_barrier(0);
            cs = cs + 1 == depth ? 0 : cs + 1;
            if constexpr (W == FP8) {
                apply();
                sc[0] = picked_scale(wg, sg, kb);
                sc[1] = picked_scale(wu, su, kb);
#pragma unroll
                for (int f = 0; f < F; ++f) part[f] = v4f{};
            }
            v4f(&to)[F] = W == FP8 ? part : acc;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int f = 0; f < F; ++f) {
                        const v8 a = widen<W, A>(w[2 * f + j][2 * q], w[2 * f + j][2 * q + 1]);
                        to[f] = mma(a, __builtin_bit_cast(v8, x[2 * j + q]), to[f]);
                    }
        }
        if constexpr (W == FP8) apply();
        // The waves' sums meet in LDS, and the waves with blocks finish items in turn; the
        // sums of two items have room where units are small, so one barrier an
        // item is enough (a wave that passes it has finished the item before
        // the last).  Fragment f, column l16 of row quad lq: place lq * NR + l16.
        const int last = done % min(KB, kWaves), mine = wave - (wave > last);
        GFG_LDS v4f* const sums = red + (TWICE && (done & 1) ? (kWaves - 1) * F * 4 * NR : 0);
        if (!TWICE) lds_barrier();
        if (wave != last && l16 < NR) {
#pragma unroll
            for (int f = 0; f < F; ++f) sums[(mine * F + f) * 4 * NR + lq * NR + l16] = acc[f];
        }
        lds_barrier();
        if (wave != last) continue;
        const int lr = l16 & (NR - 1);
#pragma unroll
        for (int w = 0; w < kWaves - 1; ++w)
#pragma unroll
            for (int f = 0; f < F; ++f) acc[f] += sums[(w * F + f) * 4 * NR + lq * NR + lr];
        v4f g = acc[0], v = acc[1];
        if constexpr (W == INT8) {
            g *= cg;
            v *= cu;
        }
        if (l16 < un.rows) store_hidden(p, r->list[un.first + l16], it * C + lq * 4, g, v);
    }
}

// ---- experts with many rows: the waves share them.
//
// Where units are large, staging their rows for every 16 columns costs more
// than the weights.  Here a work item is 128 weight rows for one unit of up to
// 32 or 64 rows: each of the eight waves has 16 of the weight rows, and all of
// them read the unit's rows from one LDS stage.  One barrier a block: a wave that passes it has
// seen every wave finish the block before, whose stage the new loads go to.
// The items run on without a break, as above.
//
// UP: the weight rows are 64 gate and 64 up rows, eight of each to a wave, so
// that gate and up meet in a wave.  DOWN: 128 rows of W2; sums go to y.
// Units of 64 rows where that saves a round of items over the workgroups: a few
// experts with slightly more than 32 rows would otherwise cost a second pass
// over their weights (us a layer, units by the rule and of 32 alone: 100 tokens,
// k = 2, E = 8, H = 4096, I = 1792: 63.7, 69.9; 130 tokens: 66.6, 89.5; of 64 alone: 48
// tokens with one or two rows an expert 97.1, by the rule 93.3).  (Smaller stages
// leave room for one more of them.)  Units of 8, two MFMA halves in one, measured
// no faster.
__device__ __forceinline__ int shared_rows(const int (&total)[6], int tiles) {
    const int grid = int(gridDim.x);
    return (total[5] * tiles + grid - 1) / grid < (total[4] * tiles + grid - 1) / grid ? 64 : 32;
}

constexpr int shared_stage(int rows, bool up) { return 16 * 1024 + rows * 256 * (up ? 1 : 2) + kScaleBytes; }
constexpr int shared_depth(int rows, bool up) { return rows == 32 ? (up ? 5 : 4) : (up ? 4 : 3); }
constexpr int kSharedLds = 3 * shared_stage(64, false);    // the largest ring of the down projection
static_assert(4 * shared_stage(32, false) <= kSharedLds, "the rings of either unit size fit");

template <int W, typename A, int NR, bool UP>
__device__ __forceinline__ void shared_items(const MoeParams& p, const GFG_LDS Routing* r, GFG_LDS uint8_t* ring) {
    typedef typename Vec<A>::v8 v8;
    constexpr int HALVES = UP ? 1 : 2, RL = NR / 32, NT = NR / 16, S = shared_depth(NR, UP), PER = 2 + HALVES * RL;
    constexpr int ROWS_AT = 16 * 1024, STAGE = shared_stage(NR, UP), SCALES_AT = STAGE - kScaleBytes;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, lq = lane >> 4;
    const int K = UP ? p.H : p.I, N = UP ? 2 * p.I : p.H;      // the weight matrix of an expert is [N][K]
    const int KB = K / 128, IT = N / 128;
    const int items = __builtin_amdgcn_readfirstlane(r->units) * IT;
    const uint8_t* const weights = UP ? p.w1 : p.w2;
    const auto rx = UP ? make_rsrc(p.x, uint32_t(p.T) * uint32_t(p.H) * 2u) : make_rsrc(p.h, uint32_t(p.T * p.k) * 4u * uint32_t(p.I));
    uint32_t shift;
    const auto rs = scale_rsrc(UP ? p.s1 : p.s2,
                               W == FP8 ? uint32_t(p.E) * uint32_t(N / 128) * uint32_t(KB) : uint32_t(p.E) * uint32_t(N) * 4u, &shift);
    // (UP: blocks it / 2 of the gate and of the up half; DOWN: block it)
    auto scale_row = [&](int e, int it, int f) {
        return uint32_t(e * (N / 128) + (UP ? it / 2 + f * (p.I / 128) : it)) * uint32_t(KB) + shift;
    };

    const uint32_t woff = uint32_t(lane >> 3) * uint32_t(K) + uint32_t(((lane & 7) ^ (lane >> 3)) * 16);
    uint32_t xoff[RL], soff[2] = {0, 0};       // rows 32 j + 4 wave + (lane >> 4) of the unit's
    __amdgpu_buffer_rsrc_t rw[2] = {make_rsrc(weights, 0), make_rsrc(weights, 0)};
    int li = blockIdx.x, lk = 0, ls = 0;
    auto enter = [&]() {
        uint32_t window = 0;
        const uint8_t* base = weights;
        Unit un{0, 0, 0};
        if (li < items) {
            const int u = li / IT, it = li - u * IT;
            un = unit_of(r, u);
            base += (int64_t(un.e) * N + (UP ? it * 64 + wave * 8 : it * 128 + wave * 16)) * K;
            window = 8u * uint32_t(K);
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                if constexpr (W == FP8)
                    soff[f] = (UP || f == 0) ? (scale_row(un.e, it, f) & ~3u) + 4u * uint32_t(lane) : kOutside;
                else
                    soff[f] = uint32_t(un.e * N + (UP ? f * p.I + it * 64 : it * 128 + f * 64) + lane) * 4u;
            }
        } else {
            soff[0] = soff[1] = kOutside;
        }
        rw[0] = make_rsrc(base, window);
        rw[1] = make_rsrc(base + int64_t(UP ? p.I : 8) * K, window);
#pragma unroll
        for (int j = 0; j < RL; ++j) {
            const int row = 32 * j + 4 * wave + (lane >> 4);
            xoff[j] = kOutside;
            if (row < un.rows) {
                const int pair = r->list[un.first + row];
                xoff[j] = (UP ? uint32_t(pair / p.k) * 2u : uint32_t(pair) * 4u) * uint32_t(K) + uint32_t(((lane & 15) ^ (row & 15)) * 16);
            }
        }
    };
    enter();
    auto issue = [&]() {
        GFG_LDS uint8_t* const dst = ring + ls * STAGE;
        const uint32_t kw = uint32_t(lk) * 128u, kx = uint32_t(lk) * 256u;
        if (lk == 0 && wave == 0) {            // the item's scales, for all waves
            dma4(rs, dst + SCALES_AT, soff[0]);
            dma4(rs, dst + SCALES_AT + 256, soff[1]);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) dma(rw[j], dst + wave * 2048 + j * 1024, woff + kw);
#pragma unroll
        for (int f = 0; f < HALVES; ++f)       // the low halves' chunks swizzled by 8 more
#pragma unroll
            for (int j = 0; j < RL; ++j)
                dma(rx, dst + ROWS_AT + f * NR * 256 + j * 8192 + wave * 1024, (xoff[j] ^ uint32_t(f * 128)) + kx + uint32_t(f) * 2u * uint32_t(K));
        ls = ls + 1 == S ? 0 : ls + 1;
        if (++lk == KB) {
            lk = 0;
            li += gridDim.x;
            enter();
        }
    };
#pragma unroll
    for (int d = 0; d < S - 1; ++d) issue();

    const uint32_t base = lds_addr(ring);
    const uint32_t w0 = base + uint32_t(wave * 2048 + l16 * 128 + ((lq ^ (l16 & 7)) << 4)), w1 = w0 ^ 64u;
    const uint32_t x0 = base + uint32_t(ROWS_AT + l16 * 256) + uint32_t(((2 * lq) ^ l16) << 4);
    int cs = 0;
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const int u = item / IT, it = item - u * IT;
        const Unit un = unit_of(r, u);
        const int tiles = (un.rows + 15) / 16;
        uint32_t words[2] = {0, 0};
        v4f channel = {};                      // INT8: the scales of this lane's rows
        v4f acc[NT] = {}, part[NT] = {};       // [16 rows of the unit]
        float sc = 0.0f;                       // FP8: the scale of this lane's rows in the last block
        auto apply = [&]() {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[t][i] = fmaf(part[t][i], sc, acc[t][i]);
        };
        for (int kb = 0; kb < KB; ++kb) {
            __builtin_amdgcn_sched_barrier(0);
            GFG_WAITCNT((S - 2) * PER, 15);
            lds_barrier();
            __builtin_amdgcn_sched_barrier(0);
            const uint32_t so = uint32_t(cs * STAGE);
            cs = cs + 1 == S ? 0 : cs + 1;
            issue();                           // into the stage read a block ago
            __builtin_amdgcn_sched_barrier(0);
            if (kb == 0) {
                const uint32_t sa = base + so + SCALES_AT;
                if constexpr (W == FP8) {
                    words[0] = read_word(sa + uint32_t(lane * 4));
                    words[1] = read_word(sa + 256u + uint32_t(lane * 4));
                } else {
                    channel = read_quad(sa + uint32_t(UP ? (lq >> 1) * 256 + (wave * 8 + (lq & 1) * 4) * 4 : (wave * 16 + lq * 4) * 4));
                }
            }
            const uint32_t xb = x0 + so, xa[4] = {xb, xb ^ 16u, xb ^ 128u, xb ^ 144u};     // [64-byte half][8 elements]
            const uint32_t xl[4] = {xa[2], xa[3], xa[0], xa[1]};                           // ... of the low halves
            u32x4 w[2], x[HALVES][4];
            read_block(w, x[0], w0 + so, w1 + so, xa);
            if constexpr (!UP) read4<NR * 256>(x[HALVES - 1], xl);
            if constexpr (W == FP8) {
                apply();
                sc = picked_scale(words[0], scale_row(un.e, it, 0), kb);
                if constexpr (UP) {
                    const float su = picked_scale(words[1], scale_row(un.e, it, 1), kb);
                    sc = lq < 2 ? sc : su;
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) part[t] = v4f{};
            }
            v4f(&to)[NT] = W == FP8 ? part : acc;
            v8 a[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) a[c] = widen<W, A>(w[c >> 1][2 * (c & 1)], w[c >> 1][2 * (c & 1) + 1]);
            auto multiply = [&](v4f& sum) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int f = 0; f < HALVES; ++f) sum = mma(a[c], __builtin_bit_cast(v8, x[f][c]), sum);
            };
            multiply(to[0]);
            if (tiles > 1) {
                read4<4096>(x[0], xa);
                if constexpr (!UP) read4<NR * 256 + 4096>(x[HALVES - 1], xl);
                multiply(to[1]);
            }
            if constexpr (NT > 2) {
                if (tiles > 2) {
                    read4<8192>(x[0], xa);
                    if constexpr (!UP) read4<NR * 256 + 8192>(x[HALVES - 1], xl);
                    multiply(to[NT - 2]);
                }
                if (tiles > 3) {
                    read4<12288>(x[0], xa);
                    if constexpr (!UP) read4<NR * 256 + 12288>(x[HALVES - 1], xl);
                    multiply(to[NT - 1]);
                }
            }
        }
        if constexpr (W == FP8) apply();
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            v4f v = acc[t];
            if constexpr (W == INT8) v *= channel;
            const bool live = 16 * t + l16 < un.rows;
            const int pair = r->list[un.first + min(16 * t + l16, un.rows - 1)];
            if constexpr (UP) {                // quads 0, 1 hold the gate rows, quads 2, 3 the up rows
                v4f up;
#pragma unroll
                for (int i = 0; i < 4; ++i) up[i] = __shfl_xor(v[i], 32, 64);
                if (live && lq < 2) store_hidden(p, pair, it * 64 + wave * 8 + lq * 4, v, up);
            } else {
                if (live) *reinterpret_cast<v4f*>(p.y + int64_t(pair) * p.H + it * 128 + wave * 16 + lq * 4) = v;
            }
        }
    }
    GFG_WAITCNT(0, 0);                         // the last loads land before the workgroup ends
}

template <int W, typename A, bool RES>
__global__ __launch_bounds__(kWaves * 64) void moe_up_kernel(MoeParams p) {
    __shared__ Routing routing;
    __shared__ v4f red_mem[(kWaves - 1) * 2 * 64];
    extern __shared__ __attribute__((aligned(256))) uint8_t ring_mem[];       // [waves][ring], then the resident rows
    GFG_LDS Routing* const r = (GFG_LDS Routing*)&routing;
    GFG_LDS v4f* const red = (GFG_LDS v4f*)red_mem;
    GFG_LDS uint8_t* const ring = (GFG_LDS uint8_t*)ring_mem;
    GFG_LDS uint8_t* const rows_mem = ring + kWaves * p.ring;
    if constexpr (RES) {
        load_resident(rows_mem, make_rsrc(p.x, uint32_t(p.T) * uint32_t(p.H) * 2u), p.H * 2, p.resident);
        const int rows = build_routing(r, ring, p.ids, p.T * p.k, p.E,
                                       [&](const int (&total)[6]) { return choose_rows<4, 8>(total, 4, 0, p.ring); });
        if (rows <= 4) up_items<W, A, 4, true>(p, r, ring, rows_mem, red);
        else up_items<W, A, 8, true>(p, r, ring, rows_mem, red);
    } else {
        const int rows = build_routing(r, ring, p.ids, p.T * p.k, p.E, [&](const int (&total)[6]) {
            const int few = choose_rows<4, 16>(total, 4, 1, p.ring), rows = shared_rows(total, p.I / 64);
            // KB a block of K for 16 columns: streamed, and shared; the latter's
            // coarser items have to fill the launch too.  Measured, us a layer,
            // shared and streamed: 100 tokens, k = 2, E = 8, H = 4096, I = 1792: 63.6,
            // 72.4; 200 tokens 72.3, 104; 64 tokens, k = 6, E = 64, H = 2048, I = 1408: 125,
            // 136; the rule streams 48 tokens with one or two rows an expert,
            // H = 4096, I = 1024: 102, 93.1; 4 tokens, k = 9, E = 385: 94.6, 75.5.  Near
            // its threshold it shares where streaming is faster: 30 tokens of the
            // first layer 59.7, 56.1; 40 tokens, k = 4, E = 32, H = 3584, I = 768: 79.3,
            // 74.6.
            const int units = total[rows == 32 ? 4 : 5];
            const int streamed = total[few == 4 ? 1 : few == 8 ? 2 : 3] * (4 + few / 4), shared = units * 6;
            return shared * 10 < streamed * 9 && units * (p.I / 64) * 4 >= int(gridDim.x) * 3 ? rows : few;
        });
        if (rows == 64) shared_items<W, A, 64, true>(p, r, ring);
        else if (rows == 32) shared_items<W, A, 32, true>(p, r, ring);
        else if (rows <= 4) up_items<W, A, 4, false>(p, r, ring, rows_mem, red);
        else if (rows <= 8) up_items<W, A, 8, false>(p, r, ring, rows_mem, red);
        else up_items<W, A, 16, false>(p, r, ring, rows_mem, red);
    }
    GFG_WAITCNT(0, 0);                         // the last loads land before the workgroup ends
}

// ---- down projection: 16 RT output columns (rows of W2) for all tokens.
//
// A workgroup walks all units; ks waves share one: wave w takes the units
// w / ks, + 8 / ks, ... and of their I the blocks w % ks, + ks, ...  Every
// (part, pair) sum goes to its own place in LDS, and the tokens' weighted sums
// are taken from there in the order of j: no atomics, and the result does not
// depend on the routing's list order.  LDS stage: 16 RT weight rows of 128
// bytes, then (unless they are resident) the high halves of NR hidden rows of
// 256 bytes, then their low halves (chunks XOR-swizzled by the row, those of
// the low halves by 8 more).  A unit has at most 8 rows, so one MFMA takes both
// halves: the high ones in columns 0..7, the low ones in columns 8..15.
template <int W, int NR, int RT>
__device__ __forceinline__ void down_tile(const MoeParams& p, const GFG_LDS Routing* r, GFG_LDS uint8_t* ring, uint32_t y, int ks,
                                          int tile) {
    constexpr int HL = NR / 2, WL = 2 * RT, PER = WL + HL, STAGE = PER * 1024 + kScaleBytes;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, lq = lane >> 4;
    const int KB = p.I / 128, P = p.T * p.k;
    const int part = wave % ks, stride = kWaves / ks;
    const int units = __builtin_amdgcn_readfirstlane(r->units);
    const int depth = min(min(p.ring / STAGE, kMaxDepth), 63 / PER);
    ring += wave * p.ring;
    const auto rh = make_rsrc(p.h, uint32_t(P) * 4u * uint32_t(p.I));

    const uint32_t woff = uint32_t(lane >> 3) * uint32_t(p.I) + uint32_t(((lane & 7) ^ (lane >> 3)) * 16);
    uint32_t hoff[HL], soff = 0, shift;
    const auto rs = scale_rsrc(p.s2, W == FP8 ? uint32_t(p.E) * uint32_t(p.H / 128) * uint32_t(KB) : uint32_t(p.E) * uint32_t(p.H) * 4u, &shift);
    __amdgpu_buffer_rsrc_t rw = make_rsrc(p.w2, 0);
    int lu = wave / ks, lk = part, ls = 0;
    bool fresh = true;
    auto enter = [&]() {
        uint32_t window = 0;
        const uint8_t* base = p.w2;
        Unit un{0, 0, 0};
        if (lu < units) {
            un = unit_of(r, lu);
            base += (int64_t(un.e) * p.H + tile * 16 * RT) * p.I;
            window = 16u * RT * uint32_t(p.I);
            if constexpr (W == FP8)
                soff = ((uint32_t(un.e * (p.H / 128) + tile * RT / 8) * uint32_t(KB) + shift) & ~3u) + 4u * uint32_t(lane);
            else
                soff = lane < 16 * RT ? uint32_t(un.e * p.H + tile * RT * 16 + lane) * 4u : kOutside;
        } else {
            soff = kOutside;
        }
        rw = make_rsrc(base, window);
        // staged row 4 j + (lane >> 4): the high halves of the unit's rows, then the low ones
#pragma unroll
        for (int j = 0; j < HL; ++j) {
            const int at = 4 * j + (lane >> 4), row = at & (NR - 1), low = at / NR;
            hoff[j] = row < un.rows ? uint32_t(r->list[un.first + row]) * 4u * uint32_t(p.I) + uint32_t(low) * 2u * uint32_t(p.I) +
                                          uint32_t(((lane & 15) ^ row ^ (8 * low)) * 16)
                                    : kOutside;
        }
        fresh = true;
    };
    enter();
    auto issue = [&]() {
        GFG_LDS uint8_t* const dst = ring + ls * STAGE;
        const uint32_t kw = uint32_t(lk) * 128u, kh = uint32_t(lk) * 256u;
        if (fresh) {
            dma4(rs, dst + PER * 1024, soff);
            fresh = false;
        }
#pragma unroll
        for (int j = 0; j < WL; ++j) dma(rw, dst + j * 1024, woff + kw + uint32_t(8 * j) * uint32_t(p.I));
#pragma unroll
        for (int j = 0; j < HL; ++j) dma(rh, dst + (WL + j) * 1024, hoff[j] + kh);
        ls = ls + 1 == depth ? 0 : ls + 1;
        lk += ks;
        if (lk >= KB) {
            lk = part;
            lu += stride;
            enter();
        }
    };
    for (int d = 0; d < depth; ++d) issue();

    const uint32_t w0 = lds_addr(ring) + uint32_t(l16 * 128 + ((lq ^ (l16 & 7)) << 4)), w1 = w0 ^ 64u;
    const int low = l16 >> 3, hr = l16 & (NR - 1);             // the half and the row of this lane's column
    const uint32_t h0 = lds_addr(ring) + uint32_t(WL * 1024 + (low * NR + hr) * 256) + uint32_t(((2 * lq) ^ hr ^ (8 * low)) << 4);
    int cs = 0;
    for (int u = wave / ks; u < units; u += stride) {
        const Unit un = unit_of(r, u);
        const uint32_t srow = uint32_t(un.e * (p.H / 128) + tile * RT / 8) * uint32_t(KB) + shift;
        uint32_t words = 0;                    // FP8: the scale row's words
        v4f channel[RT] = {};                  // INT8: the channels' scales
        v4f acc[RT] = {};
        v4f sum[RT] = {};                      // FP8: the last block's sums, before its scale
        float sc = 0.0f;
        auto apply = [&]() {
#pragma unroll
            for (int f = 0; f < RT; ++f)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[f][i] = fmaf(sum[f][i], sc, acc[f][i]);
        };
        for (int kb = part; kb < KB; kb += ks) {
            __builtin_amdgcn_sched_barrier(0);
            wait_stage<PER>(depth);
            const uint32_t so = uint32_t(cs * STAGE);
            const uint32_t hb = h0 + so;
            const uint32_t ha[4] = {hb, hb ^ 16u, hb ^ 128u, hb ^ 144u};    // [64-byte half][8 elements]
            u32x4 w[WL], h[4];
            if (kb == part) {                  // the unit's scales
                const uint32_t sa = lds_addr(ring) + so + PER * 1024u;
                if constexpr (W == FP8) {
                    words = read_word(sa + uint32_t(lane * 4));
                } else {
#pragma unroll
                    for (int f = 0; f < RT; ++f) channel[f] = read_quad(sa + uint32_t(64 * f + lq * 16));
                }
            }
            read_block(w, h, w0 + so, w1 + so, ha);
            __builtin_amdgcn_sched_barrier(0);
            issue();                           // into the stage just read
            __builtin_amdgcn_sched_barrier(0);
            cs = cs + 1 == depth ? 0 : cs + 1;
            if constexpr (W == FP8) {
                apply();
                sc = picked_scale(words, srow, kb);
#pragma unroll
                for (int f = 0; f < RT; ++f) sum[f] = v4f{};
            }
            v4f(&to)[RT] = W == FP8 ? sum : acc;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int f = 0; f < RT; ++f) {
                        const bf8 a = widen<W, __bf16>(w[2 * f + j][2 * q], w[2 * f + j][2 * q + 1]);
                        to[f] = mma(a, __builtin_bit_cast(bf8, h[2 * j + q]), to[f]);
                    }
        }
        if constexpr (W == FP8) apply();
#pragma unroll
        for (int f = 0; f < RT; ++f) {
            v4f v = acc[f];                    // column c takes its low half from column c + 8
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] += __uint_as_float(uint32_t(__builtin_amdgcn_update_dpp(0, int(__float_as_uint(v[i])), 0x128, 0xF, 0xF, false)));
            if constexpr (W == INT8) v *= channel[f];
            if (l16 < un.rows) {
                // (in assembly for the same reason as the reads: no wait for the loads in flight)
                const uint32_t at = y + uint32_t(((part * P + r->list[un.first + l16]) * RT + f) * 64 + lq * 16);
                asm volatile("ds_write_b128 %0, %1" : : "v"(at), "v"(v) : "memory");
            }
        }
    }
}

template <int W, typename OutT, int RT>
__global__ __launch_bounds__(kWaves * 64) void moe_down_kernel(MoeParams p) {
    constexpr int THREADS = kWaves * 64;
    __shared__ Routing routing;
    __shared__ float wt[kMaxPairs];            // the pairs' weights
    __shared__ uint64_t live[kMaxPairs / 64];  // bit p: pair p has an expert here
    // [waves][ring], then the sums [ks][T * k][16 RT columns]
    extern __shared__ __attribute__((aligned(256))) uint8_t ring_mem[];
    GFG_LDS Routing* const r = (GFG_LDS Routing*)&routing;
    GFG_LDS uint8_t* const ring = (GFG_LDS uint8_t*)ring_mem;
    GFG_LDS v4f* const y = (GFG_LDS v4f*)(ring + kWaves * p.ring);
    const int P = p.T * p.k;
    for (int i = threadIdx.x; i < (P + 63) / 64 * 64; i += THREADS) {
        const int e = i < P ? p.ids[i] : -1;
        const uint64_t m = __ballot(e >= 0 && e < p.E);
        if ((i & 63) == 0) live[i / 64] = m;
        if (i < P) wt[i] = p.weights[i];
    }
    const int rows = build_routing(r, ring, p.ids, P, p.E, [&](const int (&total)[6]) { return choose_rows<2, 8>(total, 2 * RT, 2, p.ring); });
    const int units = __builtin_amdgcn_readfirstlane(r->units), KB = p.I / 128;
    // the waves that share a unit: the split with the shortest longest walk, in
    // blocks of I; entering a unit costs about three.  Measured, us a layer of one
    // token, unsplit and split as far as there is room: H = 7168, k = 9, I = 512: 29.2,
    // 31.6 (by the rule unsplit); k = 2, I = 2048: 24.9, 24.5 (by the rule split in
    // four: 23.8); H = 2048, k = 6, I = 1408: 24.8, 27.7.
    constexpr int kEnter = 3;
    int ks = 1, best = (units + kWaves - 1) / kWaves * (KB + kEnter);
    for (int c = 2; c <= p.ks_most; c *= 2) {
        const int walk = (units * c + kWaves - 1) / kWaves * ((KB + c - 1) / c + kEnter);
        if (walk < best) {
            best = walk;
            ks = c;
        }
    }
    const uint32_t ya = lds_addr((GFG_LDS uint8_t*)y);
    typedef OutT o4 __attribute__((ext_vector_type(4)));
    for (int tile = blockIdx.x; tile < p.H / (16 * RT); tile += gridDim.x) {
        if (rows <= 2) down_tile<W, 2, RT>(p, r, ring, ya, ks, tile);
        else if (rows <= 4) down_tile<W, 4, RT>(p, r, ring, ya, ks, tile);
        else down_tile<W, 8, RT>(p, r, ring, ya, ks, tile);
        GFG_WAITCNT(0, 0);                     // the last loads have landed, the sums are written
        __syncthreads();
        for (int i = threadIdx.x; i < p.T * 4 * RT; i += THREADS) {
            const int t = i / (4 * RT), quad = i % (4 * RT);
            v4f sum = {};
            for (int j = 0; j < p.k; ++j) {
                const int pair = t * p.k + j;
                if (!((live[pair / 64] >> (pair % 64)) & 1)) continue;
                v4f v = y[pair * 4 * RT + quad];
                for (int s = 1; s < ks; ++s) v += y[(s * P + pair) * 4 * RT + quad];
                const float w = wt[pair];
#pragma unroll
                for (int c = 0; c < 4; ++c) sum[c] = fmaf(w, v[c], sum[c]);
            }
            *reinterpret_cast<o4*>(static_cast<OutT*>(p.out) + int64_t(t) * p.H + (tile * RT * 16 + quad * 4)) =
                o4{OutT(sum[0]), OutT(sum[1]), OutT(sum[2]), OutT(sum[3])};
        }
        __syncthreads();
    }
}

// The down projection by shared items, and the sums over a token's pairs.
// (384 items, 128 x 1408 each, 1.5 rounds: 20.5 us, 3.4-3.8 TB/s of weights.)
template <int W>
__global__ __launch_bounds__(kWaves * 64) void moe_down_shared_kernel(MoeParams p) {
    __shared__ Routing routing;
    extern __shared__ __attribute__((aligned(256))) uint8_t ring_mem[];       // the stages
    GFG_LDS Routing* const r = (GFG_LDS Routing*)&routing;
    GFG_LDS uint8_t* const ring = (GFG_LDS uint8_t*)ring_mem;
    const int rows = build_routing(r, ring, p.ids, p.T * p.k, p.E, [&](const int (&total)[6]) { return shared_rows(total, p.H / 128); });
    if (rows == 32) shared_items<W, __bf16, 32, false>(p, r, ring);
    else shared_items<W, __bf16, 64, false>(p, r, ring);
}

// Four columns of a token a thread.  The pairs' sums, ids and weights are loaded
// eight pairs at a time, also the sums of pairs without an expert (whose places
// hold anything), and only then picked, so that no load waits for another.
template <typename OutT>
__global__ __launch_bounds__(256) void moe_combine_kernel(MoeParams p) {
    const int t = blockIdx.y, col = (int(blockIdx.x) * 256 + int(threadIdx.x)) * 4;
    if (col >= p.H) return;
    const float* const y = p.y + int64_t(t) * p.k * p.H + col;
    v4f sum = {};
    for (int j0 = 0; j0 < p.k; j0 += 8) {
        v4f v[8];
        int e[8];
        float w[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const int j = min(j0 + c, p.k - 1);
            v[c] = *reinterpret_cast<const v4f*>(y + int64_t(j) * p.H);
            e[c] = p.ids[t * p.k + j];
            w[c] = p.weights[t * p.k + j];
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const bool live = j0 + c < p.k && e[c] >= 0 && e[c] < p.E;
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[i] = live ? fmaf(w[c], v[c][i], sum[i]) : sum[i];
        }
    }
    typedef OutT o4 __attribute__((ext_vector_type(4)));
    *reinterpret_cast<o4*>(static_cast<OutT*>(p.out) + int64_t(t) * p.H + col) = o4{OutT(sum[0]), OutT(sum[1]), OutT(sum[2]), OutT(sum[3])};
}

constexpr int kLds = 160 * 1024;

// Whether the down projection goes by shared items and a launch that combines
// them, from the KB that the busiest CU would read either way if the pairs
// spread evenly over min(T * k, E) experts.  (The second launch counts as 180 KB.)
// Walking all units for 16 or 32 columns leaves CUs idle where H is small and reads
// the rows again for every 16 columns where experts have many.  Measured, us a
// layer, walked and shared: 5 tokens, k = 6, E = 64, H = 2048, I = 1408: 62.9, 58.1; 12
// tokens of it 104, 91.9; 100 tokens, k = 2, E = 8, H = 4096, I = 1792: 83.5, 63.8; but
// one token, k = 9, E = 385, H = 7168, I = 512: 29.6, 31.6; 32 tokens of it 390, 397.
// Near the threshold it walks where sharing is faster: 30 tokens, k = 2, E = 8
// 59.8, 53.4; 40 tokens, k = 4, E = 32, H = 3584, I = 768: 79.3, 73.1.  Pairs of other
// ranks' experts are counted too, since the ids are device data: a rank with an
// eighth of them (48 tokens, k = 8, E = 48, H = 4096, I = 1024) shares, 93.3, where
// walking takes 91.3.
bool shared_down(const MoeParams& p, int cus, int rt) {
    const float P = float(p.T) * float(p.k), experts = P < float(p.E) ? P : float(p.E), rows = P / experts;
    const float split8 = ceilf(rows / 8), split32 = ceilf(rows / 32), blocks = float(p.I / 128);
    const float walked = ceilf(float(p.H / (16 * rt)) / float(cus)) * experts * split8 * blocks * (2.0f * float(rt) + 0.5f * rows / split8);
    const float shared = ceilf(experts * split32 * float(p.H / 128) / float(cus)) * blocks * (16.0f + 0.5f * rows / split32);
    return shared + 180.0f < 0.7f * walked;
}

template <int W, typename A>
int launch_layer(MoeParams p, hipStream_t s) {
    int cus = 0;
    if (int rc = device_cus(&cus)) return rc;
    // what a grid limit leaves of the CUs: the kernels walk their items by the grid they get
    if (const int lim = grid_limit(); lim > 0 && lim < cus) cus = lim;
    const int P = p.T * p.k;
    const dim3 block(kWaves * 64);
    // one workgroup a CU: what its LDS has left after the fixed parts and the
    // resident rows goes to the rings.  (Us a layer, rows resident and in the stages:
    // one token, k = 9, H = 7168, I = 512: 29.4, 30.4; k = 2, I = 2048: 23.8, 24.4; H = 4096,
    // k = 3, I = 1536: 21.8, 22.5; two tokens of H = 7168, 28 KB: 43.1, 43.4; but one of
    // H = 2048, k = 6, I = 1408: 25.2, 24.9; 12 of H = 2048, 48 KB: 91.0, 91.8, no more
    // than runs differ, so larger rows leave the LDS to the rings.)
    const int64_t up_items = (int64_t(P < p.E ? P : p.E) + P / 4) * (p.I / 16);
    const int up_grid = int(up_items < cus ? up_items : cus);
    const int x_bytes = p.T * p.H * 2;
    p.resident = x_bytes <= 32 * 1024 ? (x_bytes + 1023) & ~1023 : 0;
    p.ring = ((kLds - int(sizeof(Routing)) - (kWaves - 1) * 2048 - 512 - p.resident) / kWaves) & ~255;
    const unsigned up_lds = unsigned(kWaves * p.ring + p.resident);
    if (p.resident) hipLaunchKernelGGL((moe_up_kernel<W, A, true>), dim3(up_grid), block, up_lds, s, p);
    else hipLaunchKernelGGL((moe_up_kernel<W, A, false>), dim3(up_grid), block, up_lds, s, p);
    // 32 columns a workgroup of the down projection where they fill three quarters of
    // the CUs and the sums stay small (us a layer, 32 and 16 columns: one token, k = 9,
    // H = 7168, I = 512, 224 tiles: 29.6, 33.6; k = 2, I = 2048: 23.9, 27.0; with H = 4096,
    // 128 tiles, k = 2, E = 8, I = 1792: 10 tokens 49.8, 44.6, but 30 tokens 54.3, 59.8)
    const int rt = p.H % 32 == 0 && p.H / 32 >= cus * 3 / 4 && P * 128 <= 40 * 1024 ? 2 : 1;
    if (shared_down(p, cus, rt)) {
        const int items = ((P < p.E ? P : p.E) + P / 32) * (p.H / 128);
        hipLaunchKernelGGL((moe_down_shared_kernel<W>), dim3(items < cus ? items : cus), block, kSharedLds, s, p);
        hipLaunchKernelGGL((moe_combine_kernel<A>), dim3((p.H + 1023) / 1024, p.T), dim3(256), 0, s, p);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return fail(GFG_EHIP, "kernel launch failed: %s", hipGetErrorString(e));
        return GFG_OK;
    }
    while (p.ks_most < kWaves && p.ks_most * 2 <= p.I / 128 && p.ks_most * 2 * P * 64 * rt <= 24 * 1024) p.ks_most *= 2;
    const int y_bytes = p.ks_most * P * 64 * rt;
    const int tiles = p.H / (16 * rt), down_grid = tiles < cus ? tiles : cus;
    p.ring = ((kLds - int(sizeof(Routing)) - kMaxPairs * 4 - 512 - y_bytes) / kWaves) & ~255;
    const unsigned lds = unsigned(kWaves * p.ring + y_bytes);
    if (rt == 2) hipLaunchKernelGGL((moe_down_kernel<W, A, 2>), dim3(down_grid), block, lds, s, p);
    else hipLaunchKernelGGL((moe_down_kernel<W, A, 1>), dim3(down_grid), block, lds, s, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(GFG_EHIP, "kernel launch failed: %s", hipGetErrorString(e));
    return GFG_OK;
}

int64_t workspace_bytes(int64_t T, int64_t k, int64_t H, int64_t I) { return T > 0 && k > 0 && H > 0 && I > 0 ? T * k * (H + I) * 4 : 0; }

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
        return fail(GFG_EUNSUPPORTED, "%s: E=%lld above %d, or T=%lld times k=%lld above %d", fn, (long long)E, kMaxExperts,
                    (long long)T, (long long)k, kMaxPairs);
    if (H % 128 || I % 128 || H > kMaxDim || I > kMaxDim)
        return fail(GFG_EUNSUPPORTED, "%s: H=%lld and I=%lld must be multiples of 128 up to %d", fn, (long long)H, (long long)I, kMaxDim);
    if (T == 0) return GFG_OK;
    if (!x || !ids || !weights || !w1 || !s1 || !w2 || !s2 || !out) return fail(GFG_EINVAL, "%s: null pointer argument", fn);
    if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(w1) | reinterpret_cast<uintptr_t>(w2) |
         reinterpret_cast<uintptr_t>(out)) % 16 ||
        (reinterpret_cast<uintptr_t>(ids) | reinterpret_cast<uintptr_t>(weights)) % 4 ||
        (weight == INT8 && (reinterpret_cast<uintptr_t>(s1) | reinterpret_cast<uintptr_t>(s2)) % 4))
        return fail(GFG_EINVAL, "%s: x, w1, w2 and out must be 16-byte aligned, the other operands to their element", fn);
    if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16)
        return fail(GFG_EINVAL, "%s: workspace must be a 16-byte aligned device pointer", fn);
    if (bytes < workspace_bytes(T, k, H, I))
        return fail(GFG_EINVAL, "%s: workspace of %lld bytes, %lld are needed", fn, (long long)bytes,
                    (long long)workspace_bytes(T, k, H, I));
    MoeParams p{x, ids, weights, static_cast<const uint8_t*>(w1), s1, static_cast<const uint8_t*>(w2), s2,
                static_cast<uint8_t*>(workspace), reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + T * k * I * 4), out, int(T), int(k), int(E), int(H), int(I), 0, 0, 1};
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

extern "C" int64_t moe_layer_workspace_bytes(int64_t T, int64_t k, int64_t H, int64_t I) { return workspace_bytes(T, k, H, I); }

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
