// The FP8 (E4M3) linear layer with one power-of-two scale per 128 channels of a
// token and per 128 x 128 block of the weight, and its gradients, for gfx950
// (MI355X).
//
//   Q(v)      per block: t = the smallest integer with 448 * 2^t >= max|v| (0
//             for zeros), codes E4M3(v / 2^t), value code * 2^t
//   y  = Q(x) W^T + b         x in blocks of 1 x 128 along K
//   dx = Q(dy) W              dy in blocks of 1 x 128 along N; the product of
//                             dy and the transposed weight, whose 128 x 128
//                             blocks are the same blocks
//   dW = Q(dy^T) Q(x^T)^T     both in blocks of 128 tokens, for the sum runs
//                             over tokens
//   db = sum of dy over the tokens, in fp32
//
// The products run on v_mfma_scale_f32_16x16x128_f8f6f4, whose 128 k are one
// scale block, so the E8M0 bytes are its scale operands and a sum over K is a
// chain of fp32 accumulations.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "gfg.h"
#include "gfg_device.h"
#include "gfg_fp8_linear.h"
#include "gfg_fp8_quant.h"
#include "gfg_internal.h"

namespace gfg {
namespace {

constexpr int QB = 128;                        // elements of a scale block
constexpr uint32_t kOutside = 0x80000000u;     // past every buffer window used here (all below 2^31 bytes)

// The largest of 16 neighbouring lanes' magnitudes.
template <typename T>
__device__ __forceinline__ uint32_t row_largest(uint32_t m) {
    m = larger<T>(m, uint32_t(dpp<0x128>(int(m))));        // rotations by 8, 4, 2, 1
    m = larger<T>(m, uint32_t(dpp<0x124>(int(m))));
    m = larger<T>(m, uint32_t(dpp<0x122>(int(m))));
    return larger<T>(m, uint32_t(dpp<0x121>(int(m))));
}

// ------------------------------------------------------------------ token quantizer
// x [R][C] -> q [R][C], scale [ceil(C/128)][ld]: 16 lanes share a block, a
// workgroup takes 16 U rows of one column of blocks, so that its scale bytes
// are neighbours.  C a multiple of 16.  Bound by HBM: 4096 x 16384 bf16, 201 MB in 33
// us, 6.1 TB/s; 4096 x 2304 7.4 us.
template <typename T, int U>
__global__ __launch_bounds__(256) void quant_rows_kernel(const T* __restrict__ x, uint8_t* __restrict__ q,
                                                         uint8_t* __restrict__ scale, int64_t R, int C, int64_t ld) {
    const int CB = (C + QB - 1) / QB;
    const int kb = int(blockIdx.x % unsigned(CB));
    const int64_t r0 = int64_t(blockIdx.x / unsigned(CB)) * (16 * U) + (threadIdx.x >> 4);
    const int col = kb * QB + int(threadIdx.x & 15) * 8;
    Eight<T> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        v[u] = Eight<T>{};
        if (r0 + 16 * u < R && col < C) v[u] = load8(x + (r0 + 16 * u) * C + col);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t r = r0 + 16 * u;
        const uint32_t byte = scale_byte_of(as_f32<T>(row_largest<T>(largest(v[u]))));
        if (r >= R) continue;
        if (col < C) *reinterpret_cast<u32x2*>(q + r * C + col) = encode(v[u], byte);
        if ((threadIdx.x & 15) == 0) scale[kb * ld + r] = uint8_t(byte);
    }
}

// ------------------------------------------------------------------ tile quantizer
// One 128 x 128 tile of x [R][C] a workgroup, read once, for what needs it in
// both orientations: codes along the rows (q, scale [CB][ld]), codes along the
// columns, transposed (qt [C][ldt], scale_t [RB][ld_t]), and the columns' sums
// (sums [RB][C]); each one only where its pointer is given.  BLOCK: one scale
// for the whole tile in place of both (scale [RB][CB], scale_t [CB][RB]), G
// matrices one after the other.  Thread (g, l) holds rows 8 g .. +7 and columns
// 8 l .. +7, so a column's eight codes are one 8-byte word of the transposed
// tile in LDS, whose words are XOR-swizzled by the column's l.  Bound by HBM: a weight
// of 7168 x 2304 f32 in both orientations, 99 MB in 19 us, 5.2 TB/s; dy (4096 x 7168, both
// ways and sums) and x (4096 x 2304, transposed), bf16, 148 MB in 28 us, 5.3 TB/s.
struct TileJob {
    const void* x;
    uint8_t *q, *scale;
    int64_t ld;
    uint8_t* qt;
    int64_t ldt, store_t;    // row stride of qt, and how many of a row's bytes are written
    uint8_t* scale_t;
    int64_t ld_t;
    float* sums;
    int64_t R;
    int C;
    unsigned tiles;
};

// Two rows' values of column i in one word (of 16 bits each).
template <typename T>
__device__ __forceinline__ uint32_t pair_of(const Eight<T>& a, const Eight<T>& b, int i) {
    return __builtin_amdgcn_perm(b.w[i >> 1], a.w[i >> 1], (i & 1) ? 0x07060302u : 0x05040100u);
}

template <typename T, bool BLOCK>
__device__ __forceinline__ void quant_tile(TileJob p, unsigned item0) {
    constexpr int PER = sizeof(T) == 4 ? 8 : 4;            // words of eight magnitudes
    __shared__ __attribute__((aligned(16))) uint8_t tile[QB * QB];
    __shared__ uint32_t top[16][16 * PER];
    __shared__ float part[16][QB];
    __shared__ uint32_t bytes[QB];
    const int l = threadIdx.x & 15, g = threadIdx.x >> 4;
    const T* x = static_cast<const T*>(p.x);
    const int CB = (p.C + QB - 1) / QB;
    const int64_t RB = (p.R + QB - 1) / QB;
    int64_t item = item0;
    if (BLOCK) {
        const int64_t per = RB * CB, gi = item / per;
        item -= gi * per;
        x += gi * p.R * p.C;
        p.q += gi * p.R * p.C;
        p.scale += gi * per;
        if (p.qt) {
            p.qt += gi * p.R * p.C;
            p.scale_t += gi * per;
        }
    }
    const int cb = int(item % CB);
    const int64_t rb = item / CB, r0 = rb * QB + 8 * g;
    const int col = cb * QB + 8 * l;
    Eight<T> v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        v[u] = Eight<T>{};
        if (r0 + u < p.R && col < p.C) v[u] = load8(x + (r0 + u) * p.C + col);
    }
    uint32_t block_byte = 0;
    if (BLOCK) {
        uint32_t m = 0;
#pragma unroll
        for (int u = 0; u < 8; ++u) m = larger<T>(m, largest(v[u]));
        uint32_t whole = as_f32<T>(m);
        whole = wave_reduce(whole, [](uint32_t a, uint32_t b) { return max(a, b); });
        if ((threadIdx.x & 63) == 0) top[0][threadIdx.x >> 6] = whole;
        lds_barrier();
        block_byte = scale_byte_of(max(max(top[0][0], top[0][1]), max(top[0][2], top[0][3])));
        if (threadIdx.x == 0) {
            p.scale[rb * CB + cb] = uint8_t(block_byte);
            if (p.qt) p.scale_t[cb * RB + rb] = uint8_t(block_byte);
        }
    }
    // ---- along the columns: magnitudes, and sums of eight rows a thread
    if (!BLOCK && p.qt) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            uint32_t m = 0;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                uint32_t w = v[u].w[i & 3];
                if constexpr (sizeof(T) == 4) w = i < 4 ? v[u].w[i & 3] : v[u].w2[i & 3];
                m = larger<T>(m, magnitudes<T>(w));
            }
            top[g][PER * l + i] = m;
        }
    }
    if (!BLOCK && p.sums) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float t = 0.0f;
#pragma unroll
            for (int u = 0; u < 8; ++u) t += v[u].at(i);
            part[g][8 * l + i] = t;
        }
    }
    // ---- along the rows
    if (p.q) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            uint32_t byte = block_byte;
            if (!BLOCK) {
                byte = scale_byte_of(as_f32<T>(row_largest<T>(largest(v[u]))));
                if (l == 0 && r0 + u < p.R) p.scale[cb * p.ld + r0 + u] = uint8_t(byte);
            }
            if (r0 + u < p.R && col < p.C) *reinterpret_cast<u32x2*>(p.q + (r0 + u) * p.C + col) = encode(v[u], byte);
        }
    }
    if (!p.qt && !p.sums) return;
    if (!BLOCK) {
        lds_barrier();
        const int c = threadIdx.x;
        if (c < QB) {
            if (p.qt) {
                const int word = sizeof(T) == 4 ? c : c >> 1;
                uint32_t m = 0;
#pragma unroll
                for (int w = 0; w < 16; ++w) m = larger<T>(m, top[w][word]);
                const uint32_t byte = scale_byte_of(as_f32<T>(m, c & 1));
                bytes[c] = byte;
                if (cb * QB + c < p.C) p.scale_t[rb * p.ld_t + cb * QB + c] = uint8_t(byte);
            }
            if (p.sums && cb * QB + c < p.C) {
                float t = 0.0f;
#pragma unroll
                for (int w = 0; w < 16; ++w) t += part[w][c];
                p.sums[rb * p.C + cb * QB + c] = t;
            }
        }
        if (!p.qt) return;
        lds_barrier();
    }
    if (!p.qt) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t byte = BLOCK ? block_byte : bytes[8 * l + i], none = none_of(byte);
        const float scale = scale_of(byte);
        u32x2 o;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if constexpr (sizeof(T) == 4)
                o[h] = four(v[4 * h].at(i), v[4 * h + 1].at(i), v[4 * h + 2].at(i), v[4 * h + 3].at(i), scale);
            else
                o[h] = two<T, true>(two<T, false>(0u, pair_of(v[4 * h], v[4 * h + 1], i), scale), pair_of(v[4 * h + 2], v[4 * h + 3], i), scale);
            o[h] = or_nan(o[h], none);
        }
        *reinterpret_cast<u32x2*>(tile + (8 * l + i) * QB + ((g ^ l) << 3)) = o;
    }
    lds_barrier();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int c = 32 * j + int(threadIdx.x >> 3), ch = threadIdx.x & 7, key = c >> 3;
        const u32x4 w = *reinterpret_cast<const u32x4*>(tile + c * QB + ((ch ^ (key >> 1)) << 4));
        const u32x4 o = (key & 1) ? u32x4{w[2], w[3], w[0], w[1]} : w;
        if (cb * QB + c < p.C && rb * QB + 16 * ch < p.store_t)
            *reinterpret_cast<u32x4*>(p.qt + (cb * QB + c) * p.ldt + rb * QB + 16 * ch) = o;
    }
}

template <typename T, bool BLOCK>
__global__ __launch_bounds__(256) void quant_tile_kernel(TileJob p) {
    quant_tile<T, BLOCK>(p, blockIdx.x);
}

// Two tensors in one launch (dy and x of a backward pass).
template <typename T>
__global__ __launch_bounds__(256) void quant_tiles_kernel(TileJob a, TileJob b) {
    const bool second = blockIdx.x >= a.tiles;
    quant_tile<T, false>(second ? b : a, second ? blockIdx.x - a.tiles : blockIdx.x);
}

// A job's columns 16 block .. +15, in a fixed order: THREADS / 16 lanes of partial
// sums a column, then those.
constexpr int kSumColumns = 16;
template <int THREADS>
__device__ __forceinline__ void column_sums(const SumJob& p, unsigned block) {
    constexpr int LANES = THREADS / kSumColumns;
    __shared__ float part[LANES][kSumColumns + 1];
    const int l = threadIdx.x % kSumColumns, g = threadIdx.x / kSumColumns, c = int(block) * kSumColumns + l;
    float t = 0.0f;
    if (c < p.C)
        for (int64_t r = g; r < p.RB; r += LANES) t += p.sums[r * p.C + c];
    part[g][l] = t;
    __syncthreads();
    if (g || c >= p.C) return;
    t = 0.0f;
#pragma unroll
    for (int w = 0; w < LANES; ++w) t += part[w][l];
    p.out[c] = p.accumulate ? p.out[c] + t : t;
}
__global__ __launch_bounds__(256) void column_sums_kernel(SumJob p) { column_sums<256>(p, blockIdx.x); }

template <typename T>
__global__ __launch_bounds__(256) void zero_kernel(T* __restrict__ p, int64_t n) {
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256) p[i] = T(0.0f);
}

// ------------------------------------------------------------------ tiled product
// N bytes at any address
template <int N> struct Bytes;
template <> struct Bytes<1> { typedef uint8_t type; };
template <> struct Bytes<2> { typedef uint16_t type __attribute__((aligned(1))); };
template <> struct Bytes<4> { typedef uint32_t type __attribute__((aligned(1))); };

__device__ __forceinline__ v8i join(u32x4 l, u32x4 h) {
    return __builtin_bit_cast(v8i, __builtin_shufflevector(l, h, 0, 1, 2, 3, 4, 5, 6, 7));
}

// The product of one 16 x 16 block and 128 k; the scale bytes SB of sb and SA
// of sa (they have to be constants of the instruction).
template <int SB, int SA>
__device__ __forceinline__ v4f mfma_at(const v8i& b, const v8i& a, const v4f& c, int sb, int sa) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, c, 0, 0, SB, sb, SA, sa);
}
template <int SB>
__device__ __forceinline__ v4f mfma_sa(const v8i& b, const v8i& a, const v4f& c, int sb, int y, int sa) {
    switch (y) {
        case 0: return mfma_at<SB, 0>(b, a, c, sb, sa);
        case 1: return mfma_at<SB, 1>(b, a, c, sb, sa);
        case 2: return mfma_at<SB, 2>(b, a, c, sb, sa);
        default: return mfma_at<SB, 3>(b, a, c, sb, sa);
    }
}
__device__ __forceinline__ v4f mfma(const v8i& b, const v8i& a, const v4f& c, int x, int sb, int y, int sa) {
    switch (x) {
        case 0: return mfma_sa<0>(b, a, c, sb, y, sa);
        case 1: return mfma_sa<1>(b, a, c, sb, y, sa);
        case 2: return mfma_sa<2>(b, a, c, sb, y, sa);
        default: return mfma_sa<3>(b, a, c, sb, y, sa);
    }
}

// Rows of a tile of RB fragments: fragment f of lane l16 is row RB l16 + f, so
// that a lane's RB scale bytes are neighbours (one load).  LDS row R holds tile
// row R ^ ((R >> r) & 1), r = log2 RB (R itself for RB = 1), and its 16-byte
// chunk c the logical chunk c ^ ((R >> r) & 7): the 16 rows of a fragment then
// lie in both halves of the banks and in all chunks.
template <int RB> struct Rows {
    static constexpr int r = RB == 4 ? 2 : RB == 2 ? 1 : 0;
    __device__ static __forceinline__ int key(int R) { return (R >> r) & 7; }
    __device__ static __forceinline__ int swap(int R) { return RB == 1 ? R : R ^ ((R >> r) & 1); }
};

// Where a lane's RB scale bytes of one operand's rows lie: at `at` in a row of
// `total` bytes, with `shift` to bring them down where the load had to start
// lower to end inside the row (total >= RB).
struct ScaleAt { uint32_t at; int shift; };
template <int RB>
__device__ __forceinline__ ScaleAt scale_at(int64_t row, int64_t total) {
    const int64_t at = row < total - RB ? row : total - RB;
    const int64_t by = row - at;
    return ScaleAt{uint32_t(at), int(by < RB ? 8 * by : 8 * RB)};
}
template <int RB>
__device__ __forceinline__ int scale_bytes(uint32_t raw, const ScaleAt& s) {
    return int(s.shift >= 32 ? 0u : raw >> s.shift);
}

// Columns n .. n + CNT - 1 of a row.
template <int CNT, typename OutT>
__device__ __forceinline__ void store_row(OutT* row, int n, int N, const float (&v)[CNT], int accumulate) {
    typedef OutT vec __attribute__((ext_vector_type(CNT), aligned(sizeof(OutT))));     // (rows start anywhere where N is odd)
    const bool add = sizeof(OutT) == 4 && accumulate;
    if (n + CNT <= N) {
        vec o;
#pragma unroll
        for (int i = 0; i < CNT; ++i) o[i] = OutT(v[i]);
        if (add) o += *reinterpret_cast<const vec*>(row + n);
        *reinterpret_cast<vec*>(row + n) = o;
    } else {
#pragma unroll
        for (int i = 0; i < CNT; ++i)
            if (n + i < N) row[n + i] = add ? OutT(row[n + i] + OutT(v[i])) : OutT(v[i]);
    }
}

// The bias of columns n .. n + CNT - 1; without one -0, which changes nothing, not even a zero's sign.
template <int CNT>
__device__ __forceinline__ void load_bias(float (&v)[CNT], const F8Params& p, int n) {
#pragma unroll
    for (int i = 0; i < CNT; ++i) v[i] = -0.0f;
    if (p.bias) {
#pragma unroll
        for (int i = 0; i < CNT; ++i) v[i] = p.bias[min(n + i, p.N - 1)];
    }
}

// TM x TN output tiles, WM x WN waves, K in steps of 128 through four LDS
// stages (three of 256 x 128) filled by direct-to-LDS loads: all but one are in
// flight while that is consumed, and a step has one barrier (a wave that passes it has seen every
// wave finish the previous step, whose buffer the new loads go to).  Rows past
// an operand's end and chunks past K lie outside the buffer window, where the
// hardware returns zeros; zeros add nothing whatever their scale (which is a
// clamped one of the operand's own).
template <int TM, int TN, int WM, int WN, bool BROW, typename OutT>
__device__ __forceinline__ void ring_tile(const F8Params& p, unsigned w) {
    constexpr int WAVES = WM * WN, BYTES = (TM + TN) * QB, S = 4 * BYTES <= 128 * 1024 ? 4 : 3;
    constexpr int PER = BYTES / 1024 / WAVES, A_LOADS = TM / 8 / WAVES;
    constexpr int RB = TM / WM / 16, CB = TN / WN / 16;
    constexpr int OPS = PER + 1 + (BROW ? 1 : 0);      // vector-memory operations of a wave and stage
    static_assert(BYTES % (1024 * WAVES) == 0 && TM % (8 * WAVES) == 0 && WAVES % 4 == 0 && TN <= QB, "stage shape");
    // an array for each stage: the compiler then knows that reading one need
    // not wait for the loads into another
    __shared__ __attribute__((aligned(1024))) uint8_t s0[BYTES], s1[BYTES], s2[BYTES], s3[S > 3 ? BYTES : 1024];
    GFG_LDS uint8_t* const buf[4] = {(GFG_LDS uint8_t*)s0, (GFG_LDS uint8_t*)s1, (GFG_LDS uint8_t*)s2, (GFG_LDS uint8_t*)s3};
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, lq = lane >> 4;
    // tiles in ranges, one for each XCD (the hardware deals workgroup w to XCD
    // w % num_xcd), row tiles first, so that a B panel stays in one L2
    const unsigned nx = unsigned(p.num_xcd), x = w % nx, per = p.tiles / nx, rem = p.tiles % nx;
    const unsigned item = x * per + min(x, rem) + w / nx;
    const int mt = int(item % unsigned(p.m_tiles)), n0 = int(item / unsigned(p.m_tiles)) * TN;
    const int64_t row0 = int64_t(mt) * TM;
    const int lim = int(p.rows - row0 < TM ? p.rows - row0 : TM), ncols = min(TN, p.N - n0);
    const auto ra = make_rsrc(p.a + row0 * p.K, uint32_t(lim) * uint32_t(p.K));
    const auto rb = make_rsrc(p.b + int64_t(n0) * p.K, uint32_t(ncols) * uint32_t(p.K));
    const int wm = (wave / WN) * (TM / WM), wn = (wave % WN) * (TN / WN);

    // load j of a wave: LDS rows 8 (WAVES j + wave) .. +7 of the stage (A's TM
    // rows, then B's); lane i writes physical chunk i & 7 of row i >> 3 of them
    const int R = 8 * wave + (lane >> 3);
    const int ka = ((lane & 7) ^ Rows<RB>::key(R)) * 16, kbo = ((lane & 7) ^ Rows<CB>::key(R)) * 16;
    const uint32_t src_a = uint32_t(Rows<RB>::swap(R)) * uint32_t(p.K) + uint32_t(ka);
    const uint32_t src_b = uint32_t(Rows<CB>::swap(R)) * uint32_t(p.K) + uint32_t(kbo);
    const ScaleAt at_a = scale_at<RB>(row0 + wm + RB * l16, p.rows);
    const ScaleAt at_b = BROW ? scale_at<CB>(n0 + wn + CB * l16, p.N) : ScaleAt{};
    const uint8_t* const sb_row = uniform_ptr(p.b_scale + (BROW ? 0 : int64_t(n0 / QB) * p.KB));
    uint32_t sa[S], sb[S];
    auto issue = [&](int j, int kb) {
        const int ks = min(kb, p.KB - 1);
        __builtin_amdgcn_sched_barrier(0);         // (the waits count what was issued after a stage's loads)
        sa[j] = *reinterpret_cast<const typename Bytes<RB>::type*>(p.a_scale + ks * p.ld_a + at_a.at);
        if (BROW) sb[j] = *reinterpret_cast<const typename Bytes<CB>::type*>(p.b_scale + ks * p.ld_b + at_b.at);
        else sb[j] = uint32_t(load_scale_word(sb_row, ks));
        const uint32_t oa = kb * QB + ka < p.K ? src_a + uint32_t(kb) * QB : kOutside;
        const uint32_t ob = kb * QB + kbo < p.K ? src_b + uint32_t(kb) * QB : kOutside;
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int jr = i < A_LOADS ? i : i - A_LOADS;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(i < A_LOADS ? ra : rb, (GFG_LDS void*)(buf[j] + (WAVES * i + wave) * 1024), 16,
                                                     (i < A_LOADS ? oa : ob) + uint32_t(8 * WAVES * jr) * uint32_t(p.K), 0, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    auto frag = [&](GFG_LDS uint8_t* src, int row, int key) {
        auto part = [&](int c) { return *reinterpret_cast<GFG_LDS u32x4*>(src + row * QB + ((c ^ key) << 4)); };
        return join(part(lq), part(lq + 4));
    };
    v4f acc[RB][CB] = {};                          // [row fragment][column fragment]
#pragma unroll
    for (int j = 0; j < S - 1; ++j) issue(j, j);
    auto step = [&](int j, int kb, auto ops) {
        __builtin_amdgcn_sched_barrier(0);
        GFG_WAITCNT((S - 2) * decltype(ops)::value, 15);
        lds_barrier();
        __builtin_amdgcn_sched_barrier(0);
        const int a_bytes = scale_bytes<RB>(sa[j], at_a);
        const int b_bytes = BROW ? scale_bytes<CB>(sb[j], at_b) : scale_byte(int(sb[j]), sb_row, kb);
        issue((j + S - 1) % S, kb + S - 1);        // a stage past K loads zeros
        __builtin_amdgcn_sched_barrier(0);
        v8i af[RB], bf[CB];
#pragma unroll
        for (int f = 0; f < RB; ++f) {
            const int row = Rows<RB>::swap(wm + RB * l16 + f);
            af[f] = frag(buf[j], row, Rows<RB>::key(row));
        }
#pragma unroll
        for (int f = 0; f < CB; ++f) {
            const int row = Rows<CB>::swap(wn + CB * l16 + f);
            bf[f] = frag(buf[j] + TM * QB, row, Rows<CB>::key(row));
        }
#pragma unroll
        for (int y = 0; y < RB; ++y)
#pragma unroll
            for (int c = 0; c < CB; ++c) acc[y][c] = mfma(bf[c], af[y], acc[y][c], BROW ? c : 0, b_bytes, y, a_bytes);
    };
    // whole rounds of the ring, then the rest: a loop with one way out, in which
    // every path to a stage's reads passes the same loads, so that the compiler's
    // own waits stay exact.  (The rest's own scale loads are of use to nobody and
    // not issued, so its waits count the direct-to-LDS loads alone.)
    constexpr std::integral_constant<int, OPS> all{};
    constexpr std::integral_constant<int, PER> least{};
    int kb = 0;
    for (; kb + S <= p.KB; kb += S) {
#pragma unroll
        for (int j = 0; j < S; ++j) step(j, kb + j, all);
    }
    if (kb < p.KB) {
        step(0, kb, least);
        if (kb + 1 < p.KB) {
            step(1, kb + 1, least);
            if constexpr (S > 3)
                if (kb + 2 < p.KB) step(2, kb + 2, least);
        }
    }
    GFG_WAITCNT(0, 15);                            // the last loads land before the workgroup ends

    // acc[y][c][i] of lane (l16, lq): row RB l16 + y, column CB (4 lq + i) + c
    OutT* const d = static_cast<OutT*>(p.d);
    const int n = n0 + wn + 4 * CB * lq;
    float bias[4 * CB];
    load_bias(bias, p, n);
#pragma unroll
    for (int y = 0; y < RB; ++y) {
        const int r = wm + RB * l16 + y;
        if (r >= lim) continue;
        float v[4 * CB];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < CB; ++c) v[CB * i + c] = acc[y][c][i] + bias[CB * i + c];
        store_row<4 * CB>(d + (row0 + r) * p.N, n, p.N, v, p.accumulate);
    }
}

// The tiles of a workgroup: one, or, under a grid limit, every gridDim.x-th.
template <typename Tile>
__device__ __forceinline__ void walk(unsigned tiles, Tile tile) {
    for (unsigned w = blockIdx.x;;) {
        tile(w);
        w += gridDim.x;
        if (w >= tiles) return;
        __syncthreads();                           // every wave is done with the tile's LDS
    }
}

template <int TM, int TN, int WM, int WN, bool BROW, typename OutT>
__global__ __launch_bounds__(WM * WN * 64) void fp8_ring_kernel(F8Params p) {
    if (blockIdx.x >= p.tiles) return column_sums<WM * WN * 64>(p.sums, blockIdx.x - p.tiles);
    walk(p.tiles, [&](unsigned w) { ring_tile<TM, TN, WM, WN, BROW, OutT>(p, w); });
}

// ------------------------------------------------------------------ streamed product
//
// 16 RB x 16 CB output tiles whose NW waves split K: wave w takes the 128-byte
// units w, w + NW, ... of the tile's rows through its own ring of D LDS stages,
// filled by direct-to-LDS loads.  No barrier stands between a load and its
// MFMAs, every byte of the tile's rows enters the CU once and leaves the LDS
// once; the waves' sums meet in LDS at the end, in wave order.
template <int RB, int CB> constexpr int kUnit = 16 * (RB + CB) * QB;     // bytes of a wave's stage: A's rows, then B's

// s0 .. s3: a stage of every wave each (NW * kUnit bytes; the last two with D = 4).
template <int RB, int CB, int NW, int D, bool BROW, typename OutT>
__device__ __forceinline__ void stream_tile(const F8Params& p, unsigned w, uint8_t* s0, uint8_t* s1, uint8_t* s2, uint8_t* s3) {
    constexpr int TM = 16 * RB, TN = 16 * CB;
    constexpr int UNIT = kUnit<RB, CB>;
    constexpr int PER = UNIT / 1024;               // loads per stage
    constexpr int OPS = PER + 1 + (BROW ? 1 : 0);
    static_assert((D == 2 || D == 4) && OPS * D < 64, "ring depth");
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, lq = lane >> 4;
    GFG_LDS uint8_t* const ring[4] = {(GFG_LDS uint8_t*)s0 + wave * UNIT, (GFG_LDS uint8_t*)s1 + wave * UNIT,
                                      (GFG_LDS uint8_t*)s2 + (D > 2 ? wave * UNIT : 0), (GFG_LDS uint8_t*)s3 + (D > 2 ? wave * UNIT : 0)};
    const unsigned nx = unsigned(p.num_xcd), x = w % nx, per = p.tiles / nx, rem = p.tiles % nx;
    const unsigned item = x * per + min(x, rem) + w / nx;
    const int mt = int(item % unsigned(p.m_tiles)), n0 = int(item / unsigned(p.m_tiles)) * TN;
    const int64_t row0 = int64_t(mt) * TM;
    const int lim = int(p.rows - row0 < TM ? p.rows - row0 : TM), ncols = min(TN, p.N - n0);
    const auto ra = make_rsrc(p.a + row0 * p.K, uint32_t(lim) * uint32_t(p.K));
    const auto rb = make_rsrc(p.b + int64_t(n0) * p.K, uint32_t(ncols) * uint32_t(p.K));

    // load i: LDS rows 8 i .. +7 of the stage; lane l writes physical chunk
    // l & 7 of row l >> 3 of them
    const ScaleAt at_a = scale_at<RB>(row0 + RB * l16, p.rows);
    const ScaleAt at_b = BROW ? scale_at<CB>(n0 + CB * l16, p.N) : ScaleAt{};
    const uint8_t* const sb_row = uniform_ptr(p.b_scale + (BROW ? 0 : int64_t(n0 / QB) * p.KB));
    uint32_t sa[D], sb[D];
    auto load = [&](int d, int kb) {
        const int ks = min(kb, p.KB - 1);
        __builtin_amdgcn_sched_barrier(0);
        sa[d] = *reinterpret_cast<const typename Bytes<RB>::type*>(p.a_scale + ks * p.ld_a + at_a.at);
        if (BROW) sb[d] = *reinterpret_cast<const typename Bytes<CB>::type*>(p.b_scale + ks * p.ld_b + at_b.at);
        else sb[d] = uint32_t(load_scale_word(sb_row, ks));
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const bool of_a = i < TM / 8;
            const int R = 8 * (of_a ? i : i - TM / 8) + (lane >> 3);
            const int k = kb * QB + ((lane & 7) ^ (of_a ? Rows<RB>::key(R) : Rows<CB>::key(R))) * 16;
            const int row = of_a ? Rows<RB>::swap(R) : Rows<CB>::swap(R);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(of_a ? ra : rb, (GFG_LDS void*)(ring[d] + i * 1024), 16,
                                                     k < p.K ? uint32_t(row) * uint32_t(p.K) + uint32_t(k) : kOutside, 0, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    v4f acc[RB][CB] = {};
    auto frag = [&](GFG_LDS uint8_t* src, int row, int key) {
        auto part = [&](int c) { return *reinterpret_cast<GFG_LDS u32x4*>(src + row * QB + ((c ^ key) << 4)); };
        return join(part(lq), part(lq + 4));
    };
    // consume a unit, then load the one that takes its place, D units ahead
    auto step = [&](int d, int kb, auto ops) {
        __builtin_amdgcn_sched_barrier(0);
        GFG_WAITCNT((D - 1) * decltype(ops)::value, 15);
        __builtin_amdgcn_sched_barrier(0);
        const int a_bytes = scale_bytes<RB>(sa[d], at_a);
        const int b_bytes = BROW ? scale_bytes<CB>(sb[d], at_b) : scale_byte(int(sb[d]), sb_row, kb);
        v8i af[RB], bf[CB];
#pragma unroll
        for (int f = 0; f < RB; ++f) {
            const int row = Rows<RB>::swap(RB * l16 + f);
            af[f] = frag(ring[d], row, Rows<RB>::key(row));
        }
#pragma unroll
        for (int f = 0; f < CB; ++f) {
            const int row = Rows<CB>::swap(CB * l16 + f);
            bf[f] = frag(ring[d] + TM * QB, row, Rows<CB>::key(row));
        }
#pragma unroll
        for (int y = 0; y < RB; ++y)
#pragma unroll
            for (int c = 0; c < CB; ++c) acc[y][c] = mfma(bf[c], af[y], acc[y][c], BROW ? c : 0, b_bytes, y, a_bytes);
        load(d, kb + D * NW);                      // past K: zeros
    };
    constexpr std::integral_constant<int, OPS> all{};
    constexpr std::integral_constant<int, PER> least{};
#pragma unroll
    for (int d = 0; d < D; ++d) load(d, wave + d * NW);
    int kb = wave;                                 // (rounds as above)
    for (; kb + (D - 1) * NW < p.KB; kb += D * NW) {
#pragma unroll
        for (int d = 0; d < D; ++d) step(d, kb + d * NW, all);
    }
    if (kb < p.KB) {
        step(0, kb, least);
        if constexpr (D > 2) {
            if (kb + NW < p.KB) {
                step(1, kb + NW, least);
                if (kb + 2 * NW < p.KB) step(2, kb + 2 * NW, least);
            }
        }
    }
    GFG_WAITCNT(0, 15);                            // the last loads land before the workgroup ends
    // a wave's sums go where its first stage was
    static_assert(RB * CB * 1024 <= UNIT, "the sums fit a stage");
    auto sums = [&](int v, int i) -> GFG_LDS v4f& { return reinterpret_cast<GFG_LDS v4f*>((GFG_LDS uint8_t*)s0 + v * UNIT)[i * 64 + lane]; };
#pragma unroll
    for (int y = 0; y < RB; ++y)
#pragma unroll
        for (int c = 0; c < CB; ++c) sums(wave, y * CB + c) = acc[y][c];
    __syncthreads();
    // wave y sums and stores the rows of fragment y
    static_assert(RB <= NW, "a wave for each row fragment");
    if (wave >= RB) return;
    const int r = RB * l16 + wave, n = n0 + 4 * CB * lq;
    if (r >= lim) return;
    float v[4 * CB], bias[4 * CB];
    load_bias(bias, p, n);
#pragma unroll
    for (int c = 0; c < CB; ++c) {
        v4f t = sums(0, wave * CB + c);
#pragma unroll
        for (int u = 1; u < NW; ++u) t += sums(u, wave * CB + c);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[CB * i + c] = t[i] + bias[CB * i + c];
    }
    store_row<4 * CB>(static_cast<OutT*>(p.d) + (row0 + r) * p.N, n, p.N, v, p.accumulate);
}

template <int RB, int CB, int NW, int D, bool BROW, typename OutT>
__global__ __launch_bounds__(NW * 64) void fp8_stream_kernel(F8Params p) {
    // an array for each stage: the compiler then knows that reading one need
    // not wait for the loads into another
    constexpr int BYTES = NW * kUnit<RB, CB>;
    __shared__ __attribute__((aligned(1024))) uint8_t s0[BYTES], s1[BYTES], s2[D > 2 ? BYTES : 1024], s3[D > 2 ? BYTES : 1024];
    if (blockIdx.x >= p.tiles) return column_sums<NW * 64>(p.sums, blockIdx.x - p.tiles);
    walk(p.tiles, [&](unsigned w) { stream_tile<RB, CB, NW, D, BROW, OutT>(p, w, s0, s1, s2, s3); });
}

// ------------------------------------------------------------------ a few tokens, quantized on the way
//
// Tiles of 16 RB rows of x in 32 or 16 bits, one launch: a block's scale needs its
// 128 channels alone, so a wave quantizes each unit of K that it takes itself, in
// registers, where lane (l16, lq) loads what it needs of its rows RB l16 .. for the
// matrix instruction (the 16-byte chunks lq and lq + 4 of the unit's codes); the
// block's maximum crosses the four lanes of a row.  The weights come as in the
// streamed product, 16 CB columns a workgroup.
// Lanes l16, 16 + l16, 32 + l16, 48 + l16 all get the largest of their four values.
template <typename T>
__device__ __forceinline__ uint32_t largest_of_rows(uint32_t v) {
    auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = larger<T>(uint32_t(a[0]), uint32_t(a[1]));
    auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return larger<T>(uint32_t(b[0]), uint32_t(b[1]));
}

template <typename X, int RB, int CB, int NW, int D, typename OutT>
__global__ __launch_bounds__(NW * 64) void fp8_few_kernel(const X* __restrict__ xs, F8Params p) {
    constexpr int TM = 16 * RB, TN = 16 * CB, UNIT = TN * QB, PER = UNIT / 1024;
    constexpr int XL = RB * 4 * (sizeof(X) / 2), OPS = PER + XL;   // vector-memory operations of a stage
    static_assert((D == 2 || D == 4) && OPS * (D - 1) < 63, "ring depth");
    constexpr int SUMS = RB * CB * 1024;                           // bytes of a wave's sums
    constexpr int STAGE = UNIT > SUMS ? UNIT : SUMS;
    __shared__ __attribute__((aligned(1024))) uint8_t s0[NW * STAGE], s1[NW * UNIT];
    __shared__ __attribute__((aligned(1024))) uint8_t s2[D > 2 ? NW * UNIT : 1024], s3[D > 2 ? NW * UNIT : 1024];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, lq = lane >> 4;
    GFG_LDS uint8_t* const ring[4] = {(GFG_LDS uint8_t*)s0 + wave * STAGE, (GFG_LDS uint8_t*)s1 + wave * UNIT,
                                      (GFG_LDS uint8_t*)s2 + (D > 2 ? wave * UNIT : 0), (GFG_LDS uint8_t*)s3 + (D > 2 ? wave * UNIT : 0)};
    const int mt = int(blockIdx.x % unsigned(p.m_tiles)), n0 = int(blockIdx.x / unsigned(p.m_tiles)) * TN, ncols = min(TN, p.N - n0);
    const int M = int(p.rows), row0 = mt * TM, lim = min(TM, M - row0);
    const auto rx = make_rsrc(xs + int64_t(row0) * p.K, uint32_t(lim) * uint32_t(p.K) * uint32_t(sizeof(X)));
    const auto rb = make_rsrc(p.b + int64_t(n0) * p.K, uint32_t(ncols) * uint32_t(p.K));
    const uint8_t* const sb_row = uniform_ptr(p.b_scale + int64_t(n0 / QB) * p.KB);
    Eight<X> x[D][RB][4];
    uint32_t sb[D];
    auto load = [&](int d, int kb) {
        __builtin_amdgcn_sched_barrier(0);
        sb[d] = uint32_t(load_scale_word(sb_row, min(kb, p.KB - 1)));
#pragma unroll
        for (int f = 0; f < RB; ++f)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // (rows past M repeat the last one and are not stored)
                const int k = kb * QB + 64 * h + 16 * lq;
                const uint32_t at = k < p.K ? (uint32_t(min(RB * l16 + f, lim - 1)) * uint32_t(p.K) + uint32_t(k)) * uint32_t(sizeof(X)) : kOutside;
                x[d][f][2 * h] = load8<X>(rx, at);
                x[d][f][2 * h + 1] = load8<X>(rx, at + 8 * sizeof(X));
            }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int R = 8 * i + (lane >> 3);
            const int k = kb * QB + ((lane & 7) ^ Rows<CB>::key(R)) * 16;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (GFG_LDS void*)(ring[d] + i * 1024), 16,
                                                     k < p.K ? uint32_t(Rows<CB>::swap(R)) * uint32_t(p.K) + uint32_t(k) : kOutside, 0, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    v4f acc[RB][CB] = {};
    auto step = [&](int d, int kb, auto ops) {
        __builtin_amdgcn_sched_barrier(0);
        GFG_WAITCNT((D - 1) * decltype(ops)::value, 15);
        __builtin_amdgcn_sched_barrier(0);
        v8i bf[CB];
#pragma unroll
        for (int c = 0; c < CB; ++c) {
            const int row = Rows<CB>::swap(CB * l16 + c), key = Rows<CB>::key(row);
            auto part = [&](int ch) { return *reinterpret_cast<GFG_LDS u32x4*>(ring[d] + row * QB + ((ch ^ key) << 4)); };
            bf[c] = join(part(lq), part(lq + 4));
        }
        const int b_byte = scale_byte(int(sb[d]), sb_row, kb);
#pragma unroll
        for (int f = 0; f < RB; ++f) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) m = larger<X>(m, largest(x[d][f][i]));
            const uint32_t a_byte = scale_byte_of(as_f32<X>(largest_of_rows<X>(m)));
            v8i af;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const u32x2 w = encode(x[d][f][i], a_byte);
                af[2 * i] = int(w[0]);
                af[2 * i + 1] = int(w[1]);
            }
#pragma unroll
            for (int c = 0; c < CB; ++c) acc[f][c] = mfma_at<0, 0>(bf[c], af, acc[f][c], b_byte, int(a_byte));
        }
        load(d, kb + D * NW);                      // past K: zeros
    };
    constexpr std::integral_constant<int, OPS> all{};
    constexpr std::integral_constant<int, PER> least{};
#pragma unroll
    for (int d = 0; d < D; ++d) load(d, wave + d * NW);
    int kb = wave;                                 // (rounds as above)
    for (; kb + (D - 1) * NW < p.KB; kb += D * NW) {
#pragma unroll
        for (int d = 0; d < D; ++d) step(d, kb + d * NW, all);
    }
    if (kb < p.KB) {
        step(0, kb, least);
        if constexpr (D > 2) {
            if (kb + NW < p.KB) {
                step(1, kb + NW, least);
                if (kb + 2 * NW < p.KB) step(2, kb + 2 * NW, least);
            }
        }
    }
    GFG_WAITCNT(0, 15);                            // the last loads land before the workgroup ends
    // a wave's sums go where its first stage was; wave f sums and stores the rows of fragment f
    auto sums = [&](int v, int i) -> GFG_LDS v4f& { return reinterpret_cast<GFG_LDS v4f*>((GFG_LDS uint8_t*)s0 + v * STAGE)[i * 64 + lane]; };
#pragma unroll
    for (int f = 0; f < RB; ++f)
#pragma unroll
        for (int c = 0; c < CB; ++c) sums(wave, f * CB + c) = acc[f][c];
    __syncthreads();
    static_assert(RB <= NW, "a wave for each row fragment");
    const int r = RB * l16 + wave;
    if (wave >= RB || r >= lim) return;
    const int n = n0 + 4 * CB * lq;
    float v[4 * CB], bias[4 * CB];
    load_bias(bias, p, n);
#pragma unroll
    for (int c = 0; c < CB; ++c) {
        v4f t = sums(0, wave * CB + c);
#pragma unroll
        for (int u = 1; u < NW; ++u) t += sums(u, wave * CB + c);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[CB * i + c] = t[i] + bias[CB * i + c];
    }
    store_row<4 * CB>(static_cast<OutT*>(p.d) + int64_t(row0 + r) * p.N, n, p.N, v, 0);
}

// The products of a small backward pass and its bias gradient in one launch: the
// tiles of dx, then those of dW, then the columns.  Up to four tiles a CU (the whole
// pass with its quantizers, us, tokens x N x K, one launch and three: 16 x 512 x 512
// 9.1, 12.9; 300 x 528 x 1040, 891 tiles, 12.8, 16.0; 1024 x 512 x 512, 768 tiles, 14.4,
// 16.2; but 2048 x 256 x 512, 1152 tiles, 17.0, 16.0; 1024 x 1024 x 1024, 2048 tiles,
// 23.5, 20.0).  A workgroup has one tile of its own shape, so not under a grid limit
// or a set shape; the gradient of one token has too few rows for these tiles.
template <typename OutX, typename OutW>
__global__ __launch_bounds__(256) void fp8_backward_kernel(F8Params dx, F8Params dw) {
    constexpr int BYTES = 4 * kUnit<2, 2>;
    __shared__ __attribute__((aligned(1024))) uint8_t s0[BYTES], s1[BYTES], none[1024];
    const unsigned w = blockIdx.x;
    if (w < dx.tiles) stream_tile<2, 2, 4, 2, false, OutX>(dx, w, s0, s1, none, none);
    else if (w < dx.tiles + dw.tiles) stream_tile<2, 2, 4, 2, true, OutW>(dw, w - dx.tiles, s0, s1, none, none);
    else column_sums<256>(dx.sums, w - dx.tiles - dw.tiles);
}

// Workgroups of a launch over p.tiles tiles: one for each, or as many as the
// grid limit allows, which is rounded up to whole slots on every XCD.
unsigned workgroups(const F8Params& p) {
    const int lim = grid_limit();
    const unsigned nx = unsigned(p.num_xcd), most = lim > 0 ? (unsigned(lim) + nx - 1) / nx * nx : p.tiles;
    return p.tiles < most ? p.tiles : most;
}

int launched() {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(GFG_EHIP, "kernel launch failed: %s", hipGetErrorString(e));
    return GFG_OK;
}

template <int TM, int TN, int WM, int WN, bool BROW>
int launch_ring(F8Params p, int out_dtype, hipStream_t s) {
    p.m_tiles = int((p.rows + TM - 1) / TM);
    const int64_t tiles = int64_t(p.m_tiles) * ((p.N + TN - 1) / TN);
    if ((tiles + p.sum_groups) * (WM * WN * 64) >= int64_t(1) << 32) return fail(GFG_EUNSUPPORTED, "the output has too many tiles for one launch");
    p.tiles = unsigned(tiles);
    const dim3 grid(workgroups(p) + p.sum_groups), block(WM * WN * 64);
    if (out_dtype == GFG_OUT_BF16)
        hipLaunchKernelGGL((fp8_ring_kernel<TM, TN, WM, WN, BROW, __bf16>), grid, block, 0, s, p);
    else if (out_dtype == GFG_OUT_F16)
        hipLaunchKernelGGL((fp8_ring_kernel<TM, TN, WM, WN, BROW, _Float16>), grid, block, 0, s, p);
    else if constexpr (BROW)
        hipLaunchKernelGGL((fp8_ring_kernel<TM, TN, WM, WN, BROW, float>), grid, block, 0, s, p);
    return launched();
}

template <int RB, int CB, int NW, int D, bool BROW>
int launch_stream(F8Params p, int out_dtype, hipStream_t s) {
    p.m_tiles = int((p.rows + 16 * RB - 1) / (16 * RB));
    const int64_t tiles = int64_t(p.m_tiles) * ((p.N + 16 * CB - 1) / (16 * CB));
    if ((tiles + p.sum_groups) * (NW * 64) >= int64_t(1) << 32) return fail(GFG_EUNSUPPORTED, "the output has too many tiles for one launch");
    p.tiles = unsigned(tiles);
    const dim3 grid(workgroups(p) + p.sum_groups), block(NW * 64);
    if (out_dtype == GFG_OUT_BF16)
        hipLaunchKernelGGL((fp8_stream_kernel<RB, CB, NW, D, BROW, __bf16>), grid, block, 0, s, p);
    else if (out_dtype == GFG_OUT_F16)
        hipLaunchKernelGGL((fp8_stream_kernel<RB, CB, NW, D, BROW, _Float16>), grid, block, 0, s, p);
    else if constexpr (BROW)
        hipLaunchKernelGGL((fp8_stream_kernel<RB, CB, NW, D, BROW, float>), grid, block, 0, s, p);
    return launched();
}

// The tile by how many of each size there are, asked in this order (M x N x K, us, the
// product alone, cold weights, the chosen tile first):
//  * more tiles of 128 x 128 than CUs, but not of 256 x 128: those (1783 x 3777 x 14672:
//    141, 256 x 256 186; 2048 x 4096 x 7168: 55, 75; 2200 x 2048 x 4096: 30, 45; 4000 x
//    2000 x 528: 12.2, 17.5);
//  * more of both: 256 x 256 (4096 x 4096 x 16384: 205-240, 128 x
//    128 346-370; 4096 x 7168 x 2304: 70, 110; 7168 x 2304 x 4096 with a scale a row of
//    both: 62, 97); also for few rows of an output so wide, from 4 rows and 32769 columns
//    on, where it is the slower one (16 x 33024 x 7168: 77, streamed 53; 32: 78, 55; 64:
//    78, 70; 128: 78, 83; 16 x 129280 x 7168: 177, 174);
//  * up to 16 rows: streamed, 16 x 16 on eight waves where those do not outnumber
//    the CUs (1 x 2048 x 7168: 6.7, 16 x 32 8.0; 16 x 2048 x 16384: 12.5, 16.0; 1 x
//    4096 x 4096: 6.0, 6.3), else 16 x 32 (1 x 7168 x 2304: 5.8);
//  * up to 32 rows: 32 x 32, streamed (32 x 4096 x 4096: 8.0);
//  * more tiles of 64 x 64 than two a CU, which is what fits: 128 x 128 (1100 x 1900 x
//    7168: 29, 64 x 64 37; 1664 x 1792 x 2304: 13.0, 15.8; but 1408 x 1408 x 7168, 484
//    of them: 30, 26; 100 x 16000 x 4096: 20.1, 18.2);
//  * up to two tiles of 32 x 32 a CU: those, streamed (300 x 1500 x 2304: 6.8, 64 x 64
//    7.7; 128 x 2048 x 7168: 7.9, 16.6; but 400 x 1500 x 2304, 611 of them: 8.8, 7.7);
//  * else 64 x 64 (512 x 2048 x 7168: 18.3; 512 x 4096 x 4096: 18.9).
// Where a CU has one tile, what it takes in sets the time: 64 x 64 of 512 x 2048 x 7168
// 917 KB in 18.3 us, 50 GB/s with 48 KB in flight, 12% of the matrix pipes; 32 x 32 of
// 128 x 2048 x 7168 459 KB in 7.9, 58.
// A tile's lane loads the scale bytes of its RB (CB) neighbouring rows at once,
// so an operand has to have that many rows: up to 16 rows of A go to RB = 1,
// and the gradient of a weight has at least 16 of both.
int64_t tiles_of(const F8Params& p, int64_t tm, int64_t tn) { return (p.rows + tm - 1) / tm * ((p.N + tn - 1) / tn); }
bool tall(const F8Params& p, int cus) {
    return tile_shape_choice() == GFG_TILE_AUTO && tiles_of(p, 128, 128) > cus && tiles_of(p, 256, 128) <= cus;
}
// Whether the product runs on the 256 x 256 tiles, which its workgroups walk.
bool walks(const F8Params& p, int out_dtype, int cus) {
    const int choice = tile_shape_choice();
    return fp8_256_fits(p, out_dtype) && (choice == GFG_TILE_256x256 || (choice == GFG_TILE_AUTO && tiles_of(p, 128, 128) > cus && !tall(p, cus)));
}

template <bool BROW>
int launch_product(const char* fn, const F8Params& p, int out_dtype, hipStream_t s) {
    int cus = 0;
    if (int rc = device_cus(&cus)) return rc;
    if (tile_shape_choice() == GFG_TILE_256x256 && !fp8_256_fits(p, out_dtype) && p.rows >= 4 && p.N >= 4)
        return fail(GFG_EUNSUPPORTED, "%s: the 256 x 256 tile's offsets do not reach over N=%d", fn, p.N);
    auto tiles = [&](int64_t tm, int64_t tn) { return tiles_of(p, tm, tn); };
    if (tall(p, cus)) return launch_ring<256, 128, 4, 2, BROW>(p, out_dtype, s);
    if (walks(p, out_dtype, cus)) return launch_fp8_256(p, BROW, out_dtype, s);
    if constexpr (!BROW)
        if (p.rows <= 16) {
            if (p.N <= 16 * cus) return launch_stream<1, 1, 8, 4, false>(p, out_dtype, s);
            return launch_stream<1, 2, 4, 4, false>(p, out_dtype, s);
        }
    if (p.rows <= 32) return launch_stream<2, 2, 4, 2, BROW>(p, out_dtype, s);
    if (tiles(64, 64) > 2 * cus) return launch_ring<128, 128, 2, 4, BROW>(p, out_dtype, s);
    if (tiles(32, 32) <= 2 * cus) return launch_stream<2, 2, 4, 2, BROW>(p, out_dtype, s);
    return launch_ring<64, 64, 2, 2, BROW>(p, out_dtype, s);
}

F8Params product(const void* a, const uint8_t* a_scale, int64_t ld_a, const void* b, const uint8_t* b_scale, int64_t ld_b,
                 const float* bias, void* d, int64_t M, int64_t N, int64_t K) {
    F8Params p{};
    p.a = static_cast<const uint8_t*>(a);
    p.a_scale = a_scale;
    p.b = static_cast<const uint8_t*>(b);
    p.b_scale = b_scale;
    p.bias = bias;
    p.d = d;
    p.rows = M;
    p.ld_a = ld_a;
    p.ld_b = ld_b;
    p.N = int(N);
    p.K = int(K);
    p.KB = int((K + QB - 1) / QB);
    p.group_m = locality_group_m();
    p.num_xcd = locality_num_xcd();
    return p;
}

template <typename T>
int launch_quant_rows(const void* x, uint8_t* q, uint8_t* scale, int64_t R, int64_t C, int64_t ld, hipStream_t s) {
    const int64_t CB = (C + QB - 1) / QB;
    if (R <= 16) {
        hipLaunchKernelGGL((quant_rows_kernel<T, 1>), dim3(unsigned(CB)), dim3(256), 0, s, static_cast<const T*>(x), q, scale, R, int(C), ld);
    } else {
        const int64_t wgs = (R + 63) / 64 * CB;    // (below 2^31: R * CB is)
        hipLaunchKernelGGL((quant_rows_kernel<T, 4>), dim3(unsigned(wgs)), dim3(256), 0, s, static_cast<const T*>(x), q, scale, R, int(C), ld);
    }
    return launched();
}

int quantize_rows(const void* x, int32_t in_dtype, uint8_t* q, uint8_t* scale, int64_t R, int64_t C, int64_t ld, hipStream_t s) {
    if (in_dtype == GFG_IN_F32) return launch_quant_rows<float>(x, q, scale, R, C, ld, s);
    if (in_dtype == GFG_IN_BF16) return launch_quant_rows<__bf16>(x, q, scale, R, C, ld, s);
    return launch_quant_rows<_Float16>(x, q, scale, R, C, ld, s);
}

// What goes this way (cold weights, us in a graph, one launch and two): rows whose
// elements every workgroup can load again for less than a launch.
//  * up to 16 rows: 1 x 7168 x 2304 6.5, 7.8; 16 x 7168 x 2304 7.2, 8.1; 16 x 2048 x
//    7168 11.1, 11.5; 4 x 2048 x 16384 14.0, 16.2; but 16 x 2048 x 16384 20.3, 18.5;
//    16 x 300 x 16384 18.9, 12.8;
//  * more rows, in tiles of 32 x 32, with up to ten units of K in 16 bits and five in 32
//    (a lane's loads are 16 bytes of a row each, which costs more than the launch soon):
//    bf16 77 x 1003 x 1072 6.1, 6.7; 300 x 528 x 1040 6.1, 6.9; 512 x 512 x 512 4.5, 6.1;
//    77 x 1003 of 8, 10, 11, 12 and 14 units 5.7, 6.3; 6.5, 6.8; 6.9, 6.9; 6.8, 6.9; 7.3,
//    7.3; 300 x 528 of 10, 12 and 14 6.6, 6.9; 7.1, 7.2; 7.8, 7.7; 32 x 7168 x 2304 10.0,
//    8.8; f32 128 x 512 of 4, 5 and 6 units 4.6, 5.6; 5.5, 5.9; 5.9, 5.9;
//    and up to two tiles a CU: 128 x 4096 x 512 6.4, 7.3, but 256 x 4096 x 512 10.6, 7.0.
// A workgroup has one tile of its own shape, so not under a grid limit or a set shape.
bool few(const F8Params& p, int size, int cus) {
    if (grid_limit() != 0 || tile_shape_choice() != GFG_TILE_AUTO) return false;
    if (p.rows <= 16) return p.rows * p.K <= 1 << 17;
    return p.KB <= (size == 2 ? 10 : 5) && (p.rows + 31) / 32 * ((p.N + 31) / 32) <= 2 * cus;
}

template <typename X, int RB, int CB, int NW, int D>
int launch_few_on(const void* x, F8Params p, int out_dtype, hipStream_t s) {
    p.m_tiles = int((p.rows + 16 * RB - 1) / (16 * RB));
    const dim3 grid(unsigned((p.N + 16 * CB - 1) / (16 * CB) * p.m_tiles)), block(NW * 64);
    if (out_dtype == GFG_OUT_BF16)
        hipLaunchKernelGGL((fp8_few_kernel<X, RB, CB, NW, D, __bf16>), grid, block, 0, s, static_cast<const X*>(x), p);
    else
        hipLaunchKernelGGL((fp8_few_kernel<X, RB, CB, NW, D, _Float16>), grid, block, 0, s, static_cast<const X*>(x), p);
    return launched();
}

// Up to 16 rows: 16 columns a workgroup on eight waves where those do not outnumber
// the CUs, else 32 on four (16 and 32: 1 x 2048 x 7168 8.0, 9.4; 1 x 4096 x 4096 7.0,
// 7.3; 1 x 7168 x 2304 7.1, 6.5; 1 x 28672 x 4096 32.2, 27.7).
template <typename X>
int launch_few(const void* x, const F8Params& p, int cus, int out_dtype, hipStream_t s) {
    if (p.rows > 16) return launch_few_on<X, 2, 2, 4, sizeof(X) == 4 ? 2 : 4>(x, p, out_dtype, s);
    if (p.N <= 16 * cus) return launch_few_on<X, 1, 1, 8, 4>(x, p, out_dtype, s);
    return launch_few_on<X, 1, 2, 4, 4>(x, p, out_dtype, s);
}

// Tiles of 32 x 32 of a product, which are set in it.
int64_t few_tiles(F8Params* p) {
    p->m_tiles = int((p->rows + 31) / 32);
    const int64_t tiles = int64_t(p->m_tiles) * ((p->N + 31) / 32);
    p->tiles = unsigned(tiles < (1 << 30) ? tiles : 1 << 30);
    return tiles;
}

int launch_pair(const F8Params& dx, const F8Params& dw, int dx_dtype, int dw_dtype, hipStream_t s) {
    auto go = [&](auto* kernel) { hipLaunchKernelGGL(kernel, dim3(dx.tiles + dw.tiles + dx.sum_groups), dim3(256), 0, s, dx, dw); };
    auto with = [&](auto x) {
        typedef decltype(x) X;
        if (dw_dtype == GFG_OUT_BF16) go(fp8_backward_kernel<X, __bf16>);
        else if (dw_dtype == GFG_OUT_F16) go(fp8_backward_kernel<X, _Float16>);
        else go(fp8_backward_kernel<X, float>);
    };
    if (dx_dtype == GFG_OUT_BF16) with(__bf16{});
    else with(_Float16{});
    return launched();
}

TileJob job(const void* x, int64_t R, int64_t C, int64_t G) {
    TileJob p{};
    p.x = x;
    p.R = R;
    p.C = int(C);
    p.tiles = unsigned((R + QB - 1) / QB * ((C + QB - 1) / QB) * G);
    return p;
}

template <typename F>
int by_type(int32_t in_dtype, F f) {
    if (in_dtype == GFG_IN_F32) f(float{});
    else if (in_dtype == GFG_IN_BF16) f(__bf16{});
    else f(_Float16{});
    return launched();
}

// ------------------------------------------------------------------ argument checks
constexpr int64_t kMaxK = int64_t(1) << 22;            // 256 rows of K stay below 2^31 bytes
constexpr int64_t kMaxN = int64_t(1) << 28;
constexpr int64_t kMaxRows = int64_t(65535) * 128;

bool misaligned(const void* p, uintptr_t by) { return reinterpret_cast<uintptr_t>(p) % by != 0; }

int check_in(const char* fn, int32_t in_dtype) {
    if (in_dtype != GFG_IN_F32 && in_dtype != GFG_IN_BF16 && in_dtype != GFG_IN_F16)
        return fail(GFG_EINVAL, "%s: in_dtype %d is not a GFG_IN_* value", fn, in_dtype);
    return GFG_OK;
}

// Sizes of a product of M rows; M = 0 passes.
int check_sizes(const char* fn, int64_t M, int64_t N, int64_t K) {
    if (M < 0 || N <= 0 || K <= 0)
        return fail(GFG_EINVAL, "%s: bad sizes M=%lld N=%lld K=%lld", fn, (long long)M, (long long)N, (long long)K);
    if (K % 16 || K > kMaxK)
        return fail(GFG_EUNSUPPORTED, "%s: K=%lld must be a multiple of 16 and at most %lld", fn, (long long)K, (long long)kMaxK);
    if (N > kMaxN) return fail(GFG_EUNSUPPORTED, "%s: N=%lld above 2^28", fn, (long long)N);
    if (M > kMaxRows) return fail(GFG_EUNSUPPORTED, "%s: M=%lld above %lld", fn, (long long)M, (long long)kMaxRows);
    if ((M + 3) * ((K + QB - 1) / QB) >= int64_t(1) << 31)
        return fail(GFG_EUNSUPPORTED, "%s: M=%lld rows of %lld scales are 2^31 bytes or more", fn, (long long)M, (long long)((K + QB - 1) / QB));
    return GFG_OK;
}

int check_out(const char* fn, int32_t out_dtype) {
    if (out_dtype != GFG_OUT_BF16 && out_dtype != GFG_OUT_F16)
        return fail(GFG_EINVAL, "%s: out_dtype %d is not GFG_OUT_BF16 or GFG_OUT_F16", fn, out_dtype);
    return GFG_OK;
}

int check_operands(const char* fn, const void* a, const void* b, const void* b_scale, const void* bias, const void* d) {
    if (!a || !b || !b_scale || !d) return fail(GFG_EINVAL, "%s: null pointer argument", fn);
    if (misaligned(a, 16) || misaligned(b, 16) || misaligned(bias, 4) || misaligned(d, 8))
        return fail(GFG_EINVAL, "%s: the operands must be 16-byte aligned, the output 8-byte, the bias 4-byte", fn);
    return GFG_OK;
}

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

int check_workspace(const char* fn, const void* workspace, int64_t have, int64_t need) {
    if (!workspace || misaligned(workspace, 16))
        return fail(GFG_EINVAL, "%s: workspace must be a 16-byte aligned device pointer", fn);
    if (have < need)
        return fail(GFG_EINVAL, "%s: workspace of %lld bytes, %lld are needed", fn, (long long)have, (long long)need);
    return GFG_OK;
}

// The backward workspace: dy along N with its scales, dy and x along the tokens
// (padded to whole blocks) with theirs, and the parts of the bias's gradient.
struct BackwardSpace {
    int64_t Mp, MB, ldm, ldn, ldk, q, qs, yt, yts, xt, xts, sums, bytes;
    BackwardSpace(int64_t M, int64_t N, int64_t K) {
        Mp = up(M, QB);
        MB = Mp / QB;
        ldm = up(M, 4);
        ldn = up(N, 4);
        ldk = up(K, 4);
        int64_t at = 0;
        auto take = [&](int64_t n) {
            const int64_t v = at;
            at += up(n, 16);
            return v;
        };
        q = take(M * N);
        qs = take((N + QB - 1) / QB * ldm);
        yt = take(N * Mp);
        yts = take(MB * ldn);
        xt = take(K * Mp);
        xts = take(MB * ldk);
        sums = take(MB * N * 4);
        bytes = at;
    }
};

template <typename T>
void zero(T* p, int64_t n, hipStream_t s) {
    const int64_t wgs = (n + 255) / 256;
    hipLaunchKernelGGL((zero_kernel<T>), dim3(unsigned(wgs < 2048 ? wgs : 2048)), dim3(256), 0, s, p, n);
}

}  // namespace
}  // namespace gfg

using namespace gfg;

extern "C" int fp8_quantize_weight_device(const void* w, int32_t in_dtype, int32_t G, int64_t N, int64_t K, uint8_t* q,
                                          uint8_t* scale, uint8_t* q_t, uint8_t* scale_t, void* stream) {
    clear_error();
    const char* fn = "fp8_quantize_weight_device";
    if (int rc = check_in(fn, in_dtype)) return rc;
    if (G <= 0 || G > 65535) return fail(GFG_EINVAL, "%s: G=%d outside [1, 65535]", fn, G);
    if (int rc = check_sizes(fn, 1, N, K)) return rc;
    if ((N + QB - 1) / QB * ((K + QB - 1) / QB) * G >= int64_t(1) << 24)
        return fail(GFG_EUNSUPPORTED, "%s: 2^24 blocks of 128 x 128 or more", fn);
    if (!w || !q || !scale || (!q_t != !scale_t)) return fail(GFG_EINVAL, "%s: null pointer argument", fn);
    if (misaligned(w, 16) || misaligned(q, 16) || misaligned(q_t, 16))
        return fail(GFG_EINVAL, "%s: w, q and q_t must be 16-byte aligned", fn);
    if (q_t && N % 16) return fail(GFG_EUNSUPPORTED, "%s: N=%lld must be a multiple of 16 for the transposed codes", fn, (long long)N);
    TileJob p = job(w, N, K, G);
    p.q = q;
    p.scale = scale;
    p.qt = q_t;
    p.ldt = p.store_t = N;
    p.scale_t = scale_t;
    return by_type(in_dtype, [&](auto t) {
        hipLaunchKernelGGL((quant_tile_kernel<decltype(t), true>), dim3(p.tiles), dim3(256), 0, static_cast<hipStream_t>(stream), p);
    });
}

extern "C" int fp8_gemm(const void* a, const uint8_t* a_scale, int64_t a_scale_ld, const void* b, const uint8_t* b_scale,
                        const float* bias, void* d, int64_t M, int64_t N, int64_t K, int32_t out_dtype, void* stream) {
    clear_error();
    const char* fn = "fp8_gemm";
    if (int rc = check_out(fn, out_dtype)) return rc;
    if (int rc = check_sizes(fn, M, N, K)) return rc;
    if (M == 0) return GFG_OK;
    if (a_scale_ld < M) return fail(GFG_EINVAL, "%s: a_scale_ld=%lld is below M=%lld", fn, (long long)a_scale_ld, (long long)M);
    if (int rc = check_operands(fn, a, b, b_scale, bias, d)) return rc;
    if (!a_scale) return fail(GFG_EINVAL, "%s: null pointer argument", fn);
    return launch_product<false>(fn, product(a, a_scale, a_scale_ld, b, b_scale, 0, bias, d, M, N, K), out_dtype, static_cast<hipStream_t>(stream));
}

extern "C" int64_t fp8_linear_workspace_bytes(int64_t M, int64_t K) {
    return M > 0 && K > 0 ? M * up(K, 16) + (K + QB - 1) / QB * up(M, 4) : 0;
}

extern "C" int fp8_linear(const void* x, int32_t in_dtype, const void* b, const uint8_t* b_scale, const float* bias, void* d,
                          int64_t M, int64_t N, int64_t K, int32_t out_dtype, void* workspace, int64_t workspace_bytes, void* stream) {
    clear_error();
    const char* fn = "fp8_linear";
    if (int rc = check_in(fn, in_dtype)) return rc;
    if (int rc = check_out(fn, out_dtype)) return rc;
    if (int rc = check_sizes(fn, M, N, K)) return rc;
    if (M == 0) return GFG_OK;
    if ((M + 63) / 64 * ((K + QB - 1) / QB) >= int64_t(1) << 24)
        return fail(GFG_EUNSUPPORTED, "%s: x has 2^37 elements or more", fn);
    if (int rc = check_operands(fn, x, b, b_scale, bias, d)) return rc;
    if (int rc = check_workspace(fn, workspace, workspace_bytes, fp8_linear_workspace_bytes(M, K))) return rc;
    hipStream_t s = static_cast<hipStream_t>(stream);
    uint8_t *q = static_cast<uint8_t*>(workspace), *scale = q + M * K;
    int cus = 0;
    if (int rc = device_cus(&cus)) return rc;
    if (const F8Params p = product(nullptr, nullptr, 0, b, b_scale, 0, bias, d, M, N, K);
        few(p, in_dtype == GFG_IN_F32 ? 4 : 2, cus)) {
        if (in_dtype == GFG_IN_F32) return launch_few<float>(x, p, cus, out_dtype, s);
        if (in_dtype == GFG_IN_BF16) return launch_few<__bf16>(x, p, cus, out_dtype, s);
        return launch_few<_Float16>(x, p, cus, out_dtype, s);
    }
    const int64_t ld = up(M, 4);
    if (int rc = quantize_rows(x, in_dtype, q, scale, M, K, ld, s)) return rc;
    return launch_product<false>(fn, product(q, scale, ld, b, b_scale, 0, bias, d, M, N, K), out_dtype, s);
}

extern "C" int64_t fp8_linear_backward_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    return M > 0 && N > 0 && K > 0 ? BackwardSpace(M, N, K).bytes : 0;
}

extern "C" int fp8_linear_backward(const void* dy, const void* x, int32_t in_dtype, const void* b_t, const uint8_t* b_t_scale,
                                   void* dx, void* dw, float* dbias, int64_t M, int64_t N, int64_t K, int32_t dx_dtype,
                                   int32_t dw_dtype, int32_t accumulate, void* workspace, int64_t workspace_bytes, void* stream) {
    clear_error();
    const char* fn = "fp8_linear_backward";
    if (int rc = check_in(fn, in_dtype)) return rc;
    if (dx)
        if (int rc = check_out(fn, dx_dtype)) return rc;
    if (dw && dw_dtype != GFG_OUT_F32)
        if (int rc = check_out(fn, dw_dtype)) return rc;
    if (dw && accumulate && dw_dtype != GFG_OUT_F32)
        return fail(GFG_EINVAL, "%s: a gradient that is added to has to be GFG_OUT_F32", fn);
    if (int rc = check_sizes(fn, M, N, K)) return rc;
    if (N % 16 || N > kMaxK)
        return fail(GFG_EUNSUPPORTED, "%s: N=%lld must be a multiple of 16 and at most %lld", fn, (long long)N, (long long)kMaxK);
    if (M > kMaxK) return fail(GFG_EUNSUPPORTED, "%s: M=%lld above %lld", fn, (long long)M, (long long)kMaxK);
    const int64_t MB = (M + QB - 1) / QB;
    if (MB * ((N + K + 2 * QB) / QB) >= int64_t(1) << 24)
        return fail(GFG_EUNSUPPORTED, "%s: dy and x (M=%lld, N=%lld, K=%lld) are 2^24 tiles of 128 x 128 or more", fn, (long long)M, (long long)N, (long long)K);
    if (!dx && !dw && !dbias) return fail(GFG_EINVAL, "%s: dx, dw and dbias are all null", fn);
    if (misaligned(dx, 8) || misaligned(dw, 8) || misaligned(dbias, 4))
        return fail(GFG_EINVAL, "%s: dx and dw must be 8-byte aligned, dbias 4-byte", fn);
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (M == 0) {                                  // the sums over no tokens
        if (accumulate || (!dw && !dbias)) return GFG_OK;
        if (dw && dw_dtype == GFG_OUT_F32) zero(static_cast<float*>(dw), N * K, s);
        else if (dw) zero(static_cast<_Float16*>(dw), N * K, s);       // (bf16 and f16 zeros are the same bits)
        if (dbias) zero(dbias, N, s);
        return launched();
    }
    if (!dy || (dw && !x) || (dx && (!b_t || !b_t_scale))) return fail(GFG_EINVAL, "%s: null pointer argument", fn);
    if (misaligned(dy, 16) || misaligned(x, 16) || misaligned(b_t, 16))
        return fail(GFG_EINVAL, "%s: dy, x and b_t must be 16-byte aligned", fn);
    const BackwardSpace at(M, N, K);
    if (int rc = check_workspace(fn, workspace, workspace_bytes, at.bytes)) return rc;
    uint8_t* const ws = static_cast<uint8_t*>(workspace);
    float* const sums = reinterpret_cast<float*>(ws + at.sums);
    TileJob a = job(dy, M, N, 1), b = job(x, M, K, 1);
    if (dx) {
        a.q = ws + at.q;
        a.scale = ws + at.qs;
        a.ld = at.ldm;
    }
    if (dw) {
        a.qt = ws + at.yt;
        b.qt = ws + at.xt;
        a.ldt = a.store_t = b.ldt = b.store_t = at.Mp;
        a.scale_t = ws + at.yts;
        b.scale_t = ws + at.xts;
        a.ld_t = at.ldn;
        b.ld_t = at.ldk;
    } else {
        b.tiles = 0;
    }
    a.sums = dbias ? sums : nullptr;
    if (int rc = by_type(in_dtype, [&](auto t) {
            hipLaunchKernelGGL((quant_tiles_kernel<decltype(t)>), dim3(a.tiles + b.tiles), dim3(256), 0, s, a, b);
        }))
        return rc;
    F8Params px = product(ws + at.q, ws + at.qs, at.ldm, b_t, b_t_scale, 0, nullptr, dx, M, K, N);
    F8Params pw = product(ws + at.yt, ws + at.yts, at.ldn, ws + at.xt, ws + at.xts, at.ldk, nullptr, dw, N, K, at.Mp);
    pw.accumulate = accumulate;
    int cus = 0;
    if (int rc = device_cus(&cus)) return rc;
    // the bias gradient: workgroups behind the first product's, or a launch of its own
    // where that walks its tiles (all on 256 x 256 tiles, or under a grid limit)
    const SumJob db{sums, dbias, at.MB, int(N), accumulate};
    const unsigned db_groups = dbias ? unsigned((N + kSumColumns - 1) / kSumColumns) : 0u;
    if (F8Params& first = dx ? px : pw; dbias && (dx || dw) && grid_limit() == 0 && !walks(first, dx ? dx_dtype : dw_dtype, cus)) {
        first.sums = db;
        first.sum_groups = db_groups;
    } else if (dbias) {
        hipLaunchKernelGGL(column_sums_kernel, dim3(db_groups), dim3(256), 0, s, db);
        if (int rc = launched()) return rc;
    }
    if (dx && dw && M >= 2 && grid_limit() == 0 && tile_shape_choice() == GFG_TILE_AUTO && few_tiles(&px) + few_tiles(&pw) <= 4 * cus)
        return launch_pair(px, pw, dx_dtype, dw_dtype, s);
    if (dx)
        if (int rc = launch_product<false>(fn, px, dx_dtype, s)) return rc;
    return dw ? launch_product<true>(fn, pw, dw_dtype, s) : GFG_OK;
}
