// Between two blocks of a network, for gfx950 (MI355X): the norm after a block,
// its gate, the residual sum and the norm before the next block in one pass, the
// last one's rows in 16 bits or as the FP8 operand of the next product, and the
// gradients.
//
//   u = y ry wp,  out = alpha r + g u,  z = out ro w       ry = rstd(y), ro = rstd(out)
//   backward, zh = out ro, yh = y ry, h = dz w:
//   G = dout + ro (h - zh mean(h zh)),  dr = alpha G,  du = g G
//   dy = ry (wp du - yh mean(wp du yh))
//   dw = sum dz zh,  dwp = sum du yh,  dg = sum G u
//
// The second mean needs G, but not in full: sum wp g yh G is
// sum wp g yh (dout + ro h) - ro mean(h zh) sum wp g yh zh, so one round of
// reductions a row serves both means.  A channel's dwp and dg are one sum over
// the rows, S = sum G yh (with a token's gate inside: sum g G yh), times g or wp.
//
// A row's lanes hold it in registers (two chunks of 8 elements a lane, four above
// 16384) between the sums and the outputs, so it is read once (but by the backward pass
// above 8192, which reads it again): both passes are bound by HBM, or by a launch and one
// row's chain of load, sum and store.
//   forward, 4096 x 7168 bf16 with an f32 residual: 354 MB in 69 us, 5.1 TB/s (a large
//   copy: 5.06); the FP8 rows of 512 x 7168 9 us; one row 4.2 us
//   backward, 8192 x 4096 bf16: 421 MB in 79-82 us, 5.2 TB/s, and the column sums 7 us;
//   333 x 2049 f16 9.8 and 3.0 us
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "gfg.h"
#include "gfg_device.h"
#include "gfg_fp8_quant.h"
#include "gfg_internal.h"

namespace gfg {
namespace {

constexpr int64_t kMaxH = 32768;               // 1024 lanes of 4 chunks of 8 elements

// Eight neighbouring elements at any address of their type.
template <typename T>
struct Row8 {
    typedef T vec __attribute__((ext_vector_type(8), aligned(sizeof(T))));
    vec v;
    __device__ __forceinline__ void load(const T* p) { v = *reinterpret_cast<const vec*>(p); }
    __device__ __forceinline__ float at(int i) const { return float(v[i]); }
};

// A lane's chunk of a row: columns col .. col + 7, of which those from `skip` on
// are its own.  Past the last whole chunk of the row a lane takes the row's last
// eight columns, some of which (or all: skip 8) are another lane's, so every load
// is one whole vector inside the row, by every lane: no branch stands between
// the loads, and the waits for them stay exact.
struct Chunk { int col, skip; };
__device__ __forceinline__ Chunk chunk_of(int c, int H) {
    const int col = min(8 * c, H - 8);
    return Chunk{col, min(8 * c - col, 8)};
}

// The chunk, of which the compiler knows no load before this one: what it held
// instead would be spilled.
__device__ __forceinline__ Chunk again(Chunk c) {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" : "+v"(c.col));
    return c;
}

// Column i of a chunk where it is the lane's own, else 0.
__device__ __forceinline__ float own(const Chunk& c, int i, float v) { return i >= c.skip ? v : 0.0f; }

template <typename T>
__device__ __forceinline__ void store8(T* row, const Chunk& c, const float (&f)[8]) {
    typedef T vec __attribute__((ext_vector_type(8), aligned(sizeof(T))));
    if (c.skip == 0) {
        vec t;
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = T(f[i]);
        *reinterpret_cast<vec*>(row + c.col) = t;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i >= c.skip) row[c.col + i] = T(f[i]);
    }
}

// Sums of N values over the TPR threads that share a row, R rows a workgroup;
// `turn` alternates between two buffers, so one barrier is enough.  Every thread
// of the workgroup is here.
template <int TPR, int R, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], GFG_LDS float* part, int& turn) {
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = wave_reduce(v[n], [](float a, float b) { return a + b; });
    if constexpr (TPR > 64) {
        constexpr int W = TPR / 64;
        GFG_LDS float* const p = part + turn * (N * W * R) + (threadIdx.x / TPR) * (N * W);
        turn ^= 1;
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int n = 0; n < N; ++n) p[n * W + (threadIdx.x % TPR >> 6)] = v[n];
        }
        lds_barrier();
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float t = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) t += p[n * W + w];
            v[n] = t;
        }
    }
}

struct NormArgs {
    const void *y, *residual;
    const float *weight, *post, *gate;
    int gate_kind;
    float alpha, eps;
    void *out, *normed;
    uint8_t *q, *scale;
    int64_t scale_ld;
    float* stats;
    int64_t M;
    int H;
};

// TPR lanes share a row, a workgroup holds 256 / TPR rows at a time, or one.
template <int TPR> constexpr int kThreads = TPR < 256 ? 256 : TPR;
template <int TPR> constexpr int kRows = kThreads<TPR> / TPR;

// A row of `weights`, 1 where there are none, on a lane's own columns; 0 on the others.
template <int CH>
__device__ __forceinline__ void load_weights(float (&f)[CH][8], const float* weights, const Chunk (&c)[CH]) {
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        Row8<float> v;
        if (weights) v.load(weights + c[j].col);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[j][i] = own(c[j], i, weights ? v.v[i] : 1.0f);
    }
}

// The weights of a lane's columns, post weight times a channel's gate and weight, from
// the registers that hold them for all rows, or from memory once more.
template <int CH, bool HELD>
struct Weights {
    const float *post, *gate, *weight;
    float k[HELD ? CH : 1][8], w[HELD ? CH : 1][8];
    __device__ __forceinline__ Weights(const float* post, const float* gate, const float* weight, const Chunk (&c)[CH])
        : post(post), gate(gate), weight(weight) {
        if constexpr (HELD) {
            load_weights(k, post, c);
            if (gate) {
                float g[CH][8];
                load_weights(g, gate, c);
#pragma unroll
                for (int j = 0; j < CH; ++j)
#pragma unroll
                    for (int i = 0; i < 8; ++i) k[j][i] *= g[j][i];
            }
            load_weights(w, weight, c);
        }
    }
    __device__ __forceinline__ void get_k(float (&f)[8], int j, const Chunk& c) const {
        if constexpr (HELD) {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = k[j][i];
        } else {
            float g[1][8], h[1][8];
            load_weights(h, post, {c});
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = h[0][i];
            if (!gate) return;
            load_weights(g, gate, {c});
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] *= g[0][i];
        }
    }
    __device__ __forceinline__ void get_w(float (&f)[8], int j, const Chunk& c) const {
        float h[1][8];
        if constexpr (!HELD) load_weights(h, weight, {c});
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = HELD ? w[HELD ? j : 0][i] : h[0][i];
    }
};

// AHEAD: the next row is loaded while one is computed.  HELD: the weights stay in
// registers (not with four chunks a lane: 1024 x 32768 bf16 56 us, HELD 102).
template <typename Y, typename R, int TPR, int CH, bool AHEAD, bool HELD>
__global__ __launch_bounds__(kThreads<TPR>) void residual_norm_kernel(NormArgs p) {
    constexpr int ROWS = kRows<TPR>;
    __shared__ float part_smem[2 * kThreads<TPR> / 64];
    GFG_LDS float* const part = (GFG_LDS float*)part_smem;
    const int lane = threadIdx.x % TPR, in = threadIdx.x / TPR;
    Chunk c[CH];
#pragma unroll
    for (int j = 0; j < CH; ++j) c[j] = chunk_of(lane + j * TPR, p.H);
    const bool has_y = p.y != nullptr;
    // without y its loads go to the residual's rows, which are at least as long, and are not used
    const Y* const ys = static_cast<const Y*>(has_y ? p.y : p.residual);
    const R* const rs = static_cast<const R*>(p.residual);
    Row8<Y> y[CH], ny[CH];
    Row8<R> r[CH], nr[CH];
    auto load = [&](Row8<Y> (&a)[CH], Row8<R> (&b)[CH], int64_t m) {
        m = m < p.M ? m : p.M - 1;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            a[j].load(ys + m * p.H + c[j].col);
            b[j].load(rs + m * p.H + c[j].col);
        }
    };
    const int64_t step = int64_t(gridDim.x) * ROWS;
    int64_t m = int64_t(blockIdx.x) * ROWS + in;
    load(y, r, m);
    const Weights<CH, HELD> weights(p.post, p.gate_kind == GFG_GATE_CHANNEL ? p.gate : nullptr, p.weight, c);
    int turn = 0;
    // (every thread takes part in the sums of its workgroup's rows, also past the last row)
    for (int64_t base = int64_t(blockIdx.x) * ROWS; base < p.M; base += step, m += step) {
        if constexpr (AHEAD) load(ny, nr, m + step);
        const bool valid = m < p.M;
        float ry = 1.0f;
        if (p.post && has_y) {
            float s[1] = {0.0f};
#pragma unroll
            for (int j = 0; j < CH; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float v = own(c[j], i, y[j].at(i));
                    s[0] += v * v;
                }
            row_sums<TPR, ROWS>(s, part, turn);
            ry = rsqrtf(s[0] / float(p.H) + p.eps);
        }
        const float scale = ry * (p.gate_kind == GFG_GATE_TOKEN ? p.gate[valid ? m : p.M - 1] : 1.0f);
        float o[CH][8], s[1] = {0.0f};
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            float k[8];
            weights.get_k(k, j, HELD ? c[j] : again(c[j]));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                o[j][i] = p.alpha * r[j].at(i) + (has_y ? y[j].at(i) * scale * k[i] : 0.0f);
                const float v = own(c[j], i, o[j][i]);
                s[0] += v * v;
            }
            if (p.out && valid) store8(static_cast<R*>(p.out) + m * p.H, c[j], o[j]);
        }
        if (p.weight) {
            row_sums<TPR, ROWS>(s, part, turn);
            const float ro = rsqrtf(s[0] / float(p.H) + p.eps);
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                float z[8], w[8];
                weights.get_w(w, j, HELD ? c[j] : again(c[j]));
#pragma unroll
                for (int i = 0; i < 8; ++i) z[i] = o[j][i] * ro * w[i];
                if (p.normed && valid) store8(static_cast<Y*>(p.normed) + m * p.H, c[j], z);
                if (p.q) {
                    // 16 neighbouring lanes hold a block of 128 channels (z is 0 outside a lane's own)
                    uint32_t ab = 0;
#pragma unroll
                    for (int i = 0; i < 8; ++i) ab = max(ab, __float_as_uint(z[i]) & 0x7FFFFFFFu);
                    if (c[j].skip) ab = 0;                 // (0 times an infinity is NaN)
                    ab = max(ab, uint32_t(dpp<0x128>(int(ab))));
                    ab = max(ab, uint32_t(dpp<0x124>(int(ab))));
                    ab = max(ab, uint32_t(dpp<0x122>(int(ab))));
                    ab = max(ab, uint32_t(dpp<0x121>(int(ab))));
                    const uint32_t byte = scale_byte_of(ab), none = none_of(byte);
                    const float by = scale_of(byte);
                    const u32x2 code = {or_nan(four(z[0], z[1], z[2], z[3], by), none), or_nan(four(z[4], z[5], z[6], z[7], by), none)};
                    if (valid && !c[j].skip) {
                        *reinterpret_cast<u32x2*>(p.q + m * p.H + c[j].col) = code;
                        if ((c[j].col & 127) == 0) p.scale[(c[j].col >> 7) * p.scale_ld + m] = uint8_t(byte);
                    }
                }
            }
            if (p.stats && valid && lane == 0) p.stats[p.M + m] = ro;
        }
        if (p.stats && valid && lane == 0) p.stats[m] = ry;
        if constexpr (AHEAD) {
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                y[j] = ny[j];
                r[j] = nr[j];
            }
        } else {
            load(y, r, m + step);
        }
    }
}

struct BackArgs {
    const void *dout, *dnormed, *out, *y;
    const float *stats, *weight, *post, *gate;
    int gate_kind;
    float alpha;
    void *dresidual, *dy;
    float* dgate;            // a token gate's
    float* sums;             // [workgroups][2][H]: dz zh, then S; null where no sum is wanted
    int64_t M;
    int H;
};

// HELD: a row and the weights stay in registers, and the next row is loaded while
// one is computed; otherwise (rows above 8192, whose 1024 lanes have 128 registers each)
// both passes read them, a chunk at a time (1024 rows bf16, us, otherwise and HELD: 12288
// 62, 161; 16384 73, 171; 32768 412, 1077).
template <typename Y, typename R, int TPR, int CH, bool HELD>
__global__ __launch_bounds__(kThreads<TPR>) void residual_norm_backward_kernel(BackArgs p) {
    constexpr int ROWS = kRows<TPR>;
    __shared__ float part_smem[6 * kThreads<TPR> / 64];
    __shared__ float join_smem[ROWS > 1 ? 2 * CH * 8 * TPR : 1];
    // four chunks a lane: the sums S lie in LDS, each lane's own (128 KB; 1024 x 32768
    // bf16 240 us, in registers 412)
    constexpr bool IN_LDS = CH == 4;
    typedef float v4 __attribute__((ext_vector_type(4)));
    __shared__ __attribute__((aligned(16))) v4 s_smem[IN_LDS ? 2 * CH * TPR : 1];
    GFG_LDS v4* const s_lds = (GFG_LDS v4*)s_smem + threadIdx.x;
    GFG_LDS float* const part = (GFG_LDS float*)part_smem;
    const int lane = threadIdx.x % TPR, in = threadIdx.x / TPR;
    Chunk c[CH];
#pragma unroll
    for (int j = 0; j < CH; ++j) c[j] = chunk_of(lane + j * TPR, p.H);
    const bool norm = p.dnormed && p.weight, post = p.post && p.y, has_y = p.y != nullptr, has_dout = p.dout != nullptr;
    // what is not there is read from a tensor that is, of at least its length, and not used
    const R* const louts = static_cast<const R*>(has_dout ? p.dout : p.out);
    const R* const outs = static_cast<const R*>(norm ? p.out : louts);
    const Y* const dzs = static_cast<const Y*>(norm ? p.dnormed : has_y ? p.y : static_cast<const void*>(louts));
    const Y* const ys = static_cast<const Y*>(has_y ? p.y : static_cast<const void*>(dzs));
    struct Part {
        Row8<R> dout, out;
        Row8<Y> dz, y;
    };
    auto part_of = [&](int64_t m, const Chunk& c) {
        const int64_t at = (m < p.M ? m : p.M - 1) * p.H + c.col;
        Part v;
        v.out.load(outs + at);
        v.dz.load(dzs + at);
        v.dout.load(louts + at);
        v.y.load(ys + at);
        return v;
    };
    Part a[HELD ? CH : 1], b[HELD ? CH : 1];
    auto load = [&](Part (&v)[HELD ? CH : 1], int64_t m) {
        if constexpr (HELD) {
#pragma unroll
            for (int j = 0; j < CH; ++j) v[j] = part_of(m, c[j]);
        }
    };
    const int64_t step = int64_t(gridDim.x) * ROWS;
    int64_t m = int64_t(blockIdx.x) * ROWS + in;
    load(a, m);
    const Weights<CH, HELD> weights(post ? p.post : nullptr, p.gate_kind == GFG_GATE_CHANNEL ? p.gate : nullptr, norm ? p.weight : nullptr, c);
    float sw[CH][8] = {}, sp[IN_LDS ? 1 : CH][8] = {};
    if constexpr (IN_LDS) {
#pragma unroll
        for (int j = 0; j < 2 * CH; ++j) s_lds[j * TPR] = v4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    int turn = 0;
    // (every thread takes part in the sums of its workgroup's rows, also past the last row)
    for (int64_t base = int64_t(blockIdx.x) * ROWS; base < p.M; base += step, m += step) {
        load(b, m + step);
        const bool valid = m < p.M;
        const int64_t at = valid ? m : p.M - 1;
        const float ry = post ? p.stats[at] : 1.0f, ro = norm ? p.stats[p.M + at] : 0.0f;
        const float token_gate = p.gate_kind == GFG_GATE_TOKEN ? p.gate[at] : 1.0f;
        auto zh = [&](const Part& v, int i) { return norm ? v.out.at(i) * ro : 0.0f; };
        auto yh = [&](const Part& v, int i) { return has_y ? v.y.at(i) * ry : 0.0f; };
        auto h = [&](const Part& v, int i, const float (&w)[8]) { return norm ? v.dz.at(i) * w[i] : 0.0f; };
        auto dout = [&](const Part& v, int i) { return has_dout ? v.dout.at(i) : 0.0f; };
        auto take = [&](int j, float (&k)[8], float (&w)[8]) {
            const Chunk now = HELD ? c[j] : again(c[j]);
            weights.get_k(k, j, now);
            weights.get_w(w, j, now);
            if constexpr (HELD) return a[j];
            else return part_of(m, now);
        };
        // A = sum h zh, B = sum k yh (dout + ro h), C = sum k yh zh (w and k are 0 outside a lane's own)
        float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            float k[8], w[8];
            const Part x = take(j, k, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float v = yh(x, i) * k[i], z = zh(x, i), t = h(x, i, w);
                s[0] += t * z;
                s[1] += v * (dout(x, i) + ro * t);
                s[2] += v * z;
            }
        }
        row_sums<TPR, ROWS>(s, part, turn);
        const float mean_h = s[0] / float(p.H);
        const float row = s[1] - ro * mean_h * s[2];          // sum k yh G
        const float mean_y = token_gate * row / float(p.H);
        if (valid) {
            if (p.gate_kind == GFG_GATE_TOKEN && p.dgate && lane == 0) p.dgate[m] = row;
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                float dr[8], dy[8], k[8], w[8];
                const Part x = take(j, k, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float z = zh(x, i), yv = yh(x, i);
                    const float G = dout(x, i) + ro * (h(x, i, w) - z * mean_h);
                    const float gG = token_gate * G;
                    dr[i] = p.alpha * G;
                    dy[i] = post ? ry * (k[i] * gG - yv * mean_y) : k[i] * gG;
                    sw[j][i] += (norm ? x.dz.at(i) : 0.0f) * z;
                    if constexpr (IN_LDS) sp[0][i] = gG * yv;
                    else sp[j][i] += gG * yv;
                }
                if constexpr (IN_LDS) {
                    s_lds[2 * j * TPR] += v4{sp[0][0], sp[0][1], sp[0][2], sp[0][3]};
                    s_lds[(2 * j + 1) * TPR] += v4{sp[0][4], sp[0][5], sp[0][6], sp[0][7]};
                }
                if (p.dresidual) store8(static_cast<R*>(p.dresidual) + m * p.H, c[j], dr);
                if (p.dy) store8(static_cast<Y*>(p.dy) + m * p.H, c[j], dy);
            }
        }
        if constexpr (HELD) {
#pragma unroll
            for (int j = 0; j < CH; ++j) a[j] = b[j];
        }
    }
    if (!p.sums) return;
    if constexpr (ROWS > 1) {                  // the rows' lanes, in order
        GFG_LDS float* const sum = (GFG_LDS float*)join_smem;      // [2][CH * 8][TPR]
        for (int n = 0; n < ROWS; ++n) {
            if (in == n) {
#pragma unroll
                for (int j = 0; j < CH; ++j)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        GFG_LDS float* const at = sum + (j * 8 + i) * TPR + lane;
                        if (n > 0) {
                            sw[j][i] += at[0];
                            sp[j][i] += at[TPR * CH * 8];
                        }
                        at[0] = sw[j][i];
                        at[TPR * CH * 8] = sp[j][i];
                    }
            }
            lds_barrier();
        }
        if (in != ROWS - 1) return;
    }
    float* const o = p.sums + int64_t(blockIdx.x) * 2 * p.H;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        store8(o, c[j], sw[j]);
        if constexpr (IN_LDS) {
            const v4 a = s_lds[2 * j * TPR], b = s_lds[(2 * j + 1) * TPR];
            const float f[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
            store8(o + p.H, c[j], f);
        } else {
            store8(o + p.H, c[j], sp[j]);
        }
    }
}

// The sums over the workgroups' rows, in a fixed order: 32 channels a workgroup,
// 32 lanes each; blockIdx.y 0: dweight, 1: S, for the other two.
__global__ __launch_bounds__(1024) void norm_sums_kernel(const float* __restrict__ sums, int P, int H, const float* post,
                                                         const float* gate, int gate_kind, float* dweight, float* dpost,
                                                         float* dgate, int accumulate) {
    __shared__ float part[32][33];
    const int l = threadIdx.x & 31, g = threadIdx.x >> 5, c = int(blockIdx.x) * 32 + l;
    float t = 0.0f;
    if (c < H)
        for (int r = g; r < P; r += 32) t += sums[(int64_t(r) * 2 + blockIdx.y) * H + c];
    part[g][l] = t;
    __syncthreads();
    if (g || c >= H) return;
    t = 0.0f;
#pragma unroll
    for (int w = 0; w < 32; ++w) t += part[w][l];
    auto put = [&](float* p, float v) {
        if (p) p[c] = accumulate ? p[c] + v : v;
    };
    if (blockIdx.y == 0) {
        put(dweight, t);
        return;
    }
    // (without rows the factors are not read)
    put(dpost, P > 0 && gate_kind == GFG_GATE_CHANNEL ? gate[c] * t : t);
    if (gate_kind == GFG_GATE_CHANNEL) put(dgate, P > 0 && post ? post[c] * t : t);
}

// Lanes a row, and chunks that a lane holds.
template <int T, int C> struct Width { static constexpr int TPR = T, CH = C; };
template <typename F>
void by_width(int64_t H, F f) {
    if (H <= 1024) f(Width<64, 2>{});
    else if (H <= 2048) f(Width<128, 2>{});
    else if (H <= 4096) f(Width<256, 2>{});
    else if (H <= 8192) f(Width<512, 2>{});
    else if (H <= 16384) f(Width<1024, 2>{});
    else f(Width<1024, 4>{});
}
template <typename F>
void by_type(int32_t dtype, int32_t residual_dtype, F f) {
    if (dtype == GFG_IN_F32) f(float{}, float{});
    else if (dtype == GFG_IN_BF16 && residual_dtype == GFG_IN_BF16) f(__bf16{}, __bf16{});
    else if (dtype == GFG_IN_BF16) f(__bf16{}, float{});
    else if (residual_dtype == GFG_IN_F16) f(_Float16{}, _Float16{});
    else f(_Float16{}, float{});
}

// Workgroups of a pass over M rows: at most `waves` waves in all, as many as the
// registers leave room for on 256 CUs, one a CU at least, each of which then walks
// rows.  (The whole GPU's CUs and not those that there are: the size of a workspace is
// asked for without one, and must not change.)
constexpr int64_t kForwardWaves = 4096, kBackwardWaves = 2048;
struct Grid { int64_t turns, most; };          // times a workgroup's rows that there are, and workgroups
Grid grid_of(int64_t M, int64_t H, int64_t waves) {
    int64_t rows = 1, most = 1;
    by_width(H, [&](auto w) {
        rows = kRows<decltype(w)::TPR>;
        most = std::max<int64_t>(waves * 64 / kThreads<decltype(w)::TPR>, 256);
    });
    return Grid{(M + rows - 1) / rows, most};
}
int64_t forward_groups(int64_t M, int64_t H) {
    const Grid g = grid_of(M, H, kForwardWaves);
    return g.turns < g.most ? g.turns : g.most;
}
// Backward, each workgroup also writes sums that are read again: up to five turns a
// CU one workgroup a CU, and all of them as many turns (both launches, us, 512 and
// 256 workgroups at most: 512 x 4096 20.4, 17.1; 478 x 3033 21.1, 16.9; 1264 x 3791
// 26.1, 25.5; but 2048 x 4096, eight turns, 29.1, 31.6).
int64_t backward_groups(int64_t M, int64_t H) {
    const Grid g = grid_of(M, H, kBackwardWaves);
    const int64_t most = g.turns <= 5 * 256 && g.most > 256 ? 256 : g.most, each = (g.turns + most - 1) / most;
    return (g.turns + each - 1) / each;
}
// The workspace holds as many workgroups' sums as M rows or fewer ever take.
int64_t backward_bytes(int64_t M, int64_t H) {
    const Grid g = grid_of(M, H, kBackwardWaves);
    return std::min(g.turns, g.most) * 2 * H * 4;
}

int launched() {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(GFG_EHIP, "kernel launch failed: %s", hipGetErrorString(e));
    return GFG_OK;
}

int check_norm(const char* fn, int64_t M, int64_t H, int32_t dtype, int32_t residual_dtype, const float* gate, int32_t gate_kind) {
    if (dtype != GFG_IN_F32 && dtype != GFG_IN_BF16 && dtype != GFG_IN_F16)
        return fail(GFG_EINVAL, "%s: dtype %d is not a GFG_IN_* value", fn, dtype);
    if (residual_dtype != dtype && residual_dtype != GFG_IN_F32)
        return fail(GFG_EINVAL, "%s: residual_dtype %d is neither dtype nor GFG_IN_F32", fn, residual_dtype);
    if (gate_kind != GFG_GATE_NONE && gate_kind != GFG_GATE_CHANNEL && gate_kind != GFG_GATE_TOKEN)
        return fail(GFG_EINVAL, "%s: gate_kind %d is not a GFG_GATE_* value", fn, gate_kind);
    if (M < 0 || H <= 0) return fail(GFG_EINVAL, "%s: bad sizes M=%lld H=%lld", fn, (long long)M, (long long)H);
    if (H < 8 || H > kMaxH) return fail(GFG_EUNSUPPORTED, "%s: H=%lld outside [8, %lld]", fn, (long long)H, (long long)kMaxH);
    if (M >= int64_t(1) << 31) return fail(GFG_EUNSUPPORTED, "%s: M=%lld is 2^31 or more", fn, (long long)M);
    if (M > 0 && (gate_kind != GFG_GATE_NONE) != (gate != nullptr))
        return fail(GFG_EINVAL, "%s: gate and gate_kind do not go together", fn);
    return GFG_OK;
}

bool misaligned(const void* p, uintptr_t by) { return reinterpret_cast<uintptr_t>(p) % by != 0; }
uintptr_t size_of(int32_t dtype) { return dtype == GFG_IN_F32 ? 4 : 2; }

int forward(const char* fn, NormArgs a, int32_t dtype, int32_t residual_dtype, void* stream) {
    if (!a.residual) return fail(GFG_EINVAL, "%s: null pointer argument", fn);
    if (!(a.eps >= 0.0f)) return fail(GFG_EINVAL, "%s: eps must not be negative", fn);
    if (!a.out && !a.normed && !a.q) return fail(GFG_EINVAL, "%s: neither out nor the normed rows are wanted", fn);
    if (misaligned(a.y, size_of(dtype)) || misaligned(a.normed, size_of(dtype)) || misaligned(a.residual, size_of(residual_dtype)) ||
        misaligned(a.out, size_of(residual_dtype)) || misaligned(a.q, 8) || misaligned(a.weight, 4) || misaligned(a.post, 4) ||
        misaligned(a.gate, 4) || misaligned(a.stats, 4))
        return fail(GFG_EINVAL, "%s: a pointer is not aligned to its elements (q: 8 bytes)", fn);
    by_width(a.H, [&](auto width) {
        constexpr int TPR = decltype(width)::TPR, CH = decltype(width)::CH;
        const dim3 grid(unsigned(forward_groups(a.M, a.H))), block(kThreads<TPR>);
        by_type(dtype, residual_dtype, [&](auto y, auto r) {
            hipLaunchKernelGGL((residual_norm_kernel<decltype(y), decltype(r), TPR, CH, (CH == 2), (CH == 2)>), grid, block, 0, static_cast<hipStream_t>(stream), a);
        });
    });
    return launched();
}

}  // namespace
}  // namespace gfg

using namespace gfg;

extern "C" int residual_norm(const void* y, const void* residual, const float* weight, const float* post_weight,
                             const float* gate, int32_t gate_kind, float alpha, float eps, void* out, void* normed,
                             float* stats, int64_t M, int64_t H, int32_t dtype, int32_t residual_dtype, void* stream) {
    clear_error();
    const char* fn = "residual_norm";
    if (int rc = check_norm(fn, M, H, dtype, residual_dtype, gate, gate_kind)) return rc;
    if (M == 0) return GFG_OK;
    if (!weight != !normed) return fail(GFG_EINVAL, "%s: weight and normed do not go together", fn);
    return forward(fn, NormArgs{y, residual, weight, post_weight, gate, gate_kind, alpha, eps, out, normed, nullptr, nullptr, 0, stats, M, int(H)},
                   dtype, residual_dtype, stream);
}

extern "C" int residual_norm_fp8(const void* y, const void* residual, const float* weight, const float* post_weight,
                                 const float* gate, int32_t gate_kind, float alpha, float eps, void* out, uint8_t* q,
                                 uint8_t* scale, int64_t scale_ld, float* stats, int64_t M, int64_t H, int32_t dtype,
                                 int32_t residual_dtype, void* stream) {
    clear_error();
    const char* fn = "residual_norm_fp8";
    if (int rc = check_norm(fn, M, H, dtype, residual_dtype, gate, gate_kind)) return rc;
    if (H % 16) return fail(GFG_EUNSUPPORTED, "%s: H=%lld must be a multiple of 16", fn, (long long)H);
    if (M == 0) return GFG_OK;
    if (!weight || !q || !scale) return fail(GFG_EINVAL, "%s: null pointer argument", fn);
    if (scale_ld < M) return fail(GFG_EINVAL, "%s: scale_ld=%lld is below M=%lld", fn, (long long)scale_ld, (long long)M);
    return forward(fn, NormArgs{y, residual, weight, post_weight, gate, gate_kind, alpha, eps, out, nullptr, q, scale, scale_ld, stats, M, int(H)},
                   dtype, residual_dtype, stream);
}

extern "C" int64_t residual_norm_backward_workspace_bytes(int64_t M, int64_t H) {
    return M > 0 && H > 0 ? backward_bytes(M, H) : 0;
}

extern "C" int residual_norm_backward(const void* dout, const void* dnormed, const void* out, const void* y, const float* stats,
                                      const float* weight, const float* post_weight, const float* gate, int32_t gate_kind,
                                      float alpha, void* dresidual, void* dy, float* dweight, float* dpost_weight, float* dgate,
                                      int32_t accumulate, int64_t M, int64_t H, int32_t dtype, int32_t residual_dtype,
                                      void* workspace, int64_t workspace_bytes, void* stream) {
    clear_error();
    const char* fn = "residual_norm_backward";
    if (int rc = check_norm(fn, M, H, dtype, residual_dtype, gate, gate_kind)) return rc;
    if (dgate && gate_kind == GFG_GATE_NONE) return fail(GFG_EINVAL, "%s: dgate without a gate", fn);
    if (dweight && !weight && M > 0) return fail(GFG_EINVAL, "%s: dweight without weight", fn);
    if (dpost_weight && !post_weight && M > 0) return fail(GFG_EINVAL, "%s: dpost_weight without post_weight", fn);
    if (!dresidual && !dy && !dweight && !dpost_weight && !dgate) return fail(GFG_EINVAL, "%s: no gradient is wanted", fn);
    const bool sums = dweight || dpost_weight || (dgate && gate_kind == GFG_GATE_CHANNEL);
    if (M > 0) {
        if (!dout && !dnormed) return fail(GFG_EINVAL, "%s: dout and dnormed are both null", fn);
        if ((dy || dpost_weight || dgate) && !y) return fail(GFG_EINVAL, "%s: null pointer argument", fn);
        if (dnormed && (!weight || !out)) return fail(GFG_EINVAL, "%s: dnormed needs weight and out", fn);
        if (!stats && ((dnormed && weight) || (y && post_weight))) return fail(GFG_EINVAL, "%s: null pointer argument", fn);
        const uintptr_t ys = size_of(dtype), rs = size_of(residual_dtype);
        if (misaligned(dout, rs) || misaligned(out, rs) || misaligned(dresidual, rs) || misaligned(dnormed, ys) || misaligned(y, ys) ||
            misaligned(dy, ys) || misaligned(stats, 4) || misaligned(weight, 4) || misaligned(post_weight, 4) || misaligned(gate, 4))
            return fail(GFG_EINVAL, "%s: a pointer is not aligned to its elements", fn);
    }
    if (misaligned(dweight, 4) || misaligned(dpost_weight, 4) || misaligned(dgate, 4))
        return fail(GFG_EINVAL, "%s: a pointer is not aligned to its elements", fn);
    if (M > 0 && sums) {
        if (!workspace || misaligned(workspace, 16))
            return fail(GFG_EINVAL, "%s: workspace must be a 16-byte aligned device pointer", fn);
        if (workspace_bytes < residual_norm_backward_workspace_bytes(M, H))
            return fail(GFG_EINVAL, "%s: workspace of %lld bytes, %lld are needed", fn, (long long)workspace_bytes,
                        (long long)residual_norm_backward_workspace_bytes(M, H));
    }
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int64_t P = M > 0 ? backward_groups(M, H) : 0;
    if (M > 0) {
        const BackArgs a{dout, dnormed, out, y, stats, weight, post_weight, gate, gate_kind, alpha, dresidual, dy, dgate,
                         sums ? static_cast<float*>(workspace) : nullptr, M, int(H)};
        by_width(H, [&](auto width) {
            constexpr int TPR = decltype(width)::TPR, CH = decltype(width)::CH;
            by_type(dtype, residual_dtype, [&](auto yt, auto rt) {
                hipLaunchKernelGGL((residual_norm_backward_kernel<decltype(yt), decltype(rt), TPR, CH, (TPR < 1024)>), dim3(unsigned(P)),
                                   dim3(kThreads<TPR>), 0, s, a);
            });
        });
        if (int rc = launched()) return rc;
    }
    if (!sums || (M == 0 && accumulate)) return GFG_OK;
    hipLaunchKernelGGL(norm_sums_kernel, dim3(unsigned((H + 31) / 32), 2), dim3(1024), 0, s, static_cast<const float*>(workspace), int(P), int(H),
                       post_weight, gate, gate_kind, dweight, dpost_weight, dgate, accumulate);
    return launched();
}
