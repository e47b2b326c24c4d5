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
#include <hip/hip_runtime.h>

#include <cstdint>

#include "gfg.h"
#include "gfg_device.h"
#include "gfg_internal.h"

namespace gfg {
namespace {

constexpr int CH = 4;                          // chunks of 8 elements that a lane holds of a row
constexpr int64_t kMaxH = 32768;               // 1024 lanes of them
constexpr int64_t kMostGroups = 512;           // workgroups of the backward pass: rows of partial sums

typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

// Eight elements at any address of their type, the first n of them (zeros past those).
template <typename T>
struct Row8 {
    typedef T vec __attribute__((ext_vector_type(8), aligned(sizeof(T))));
    T v[8];
    __device__ __forceinline__ void load(const T* p, int n) {
        if (n >= 8) {
            const vec t = *reinterpret_cast<const vec*>(p);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = t[i];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : T(0.0f);
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = T(0.0f);
    }
    __device__ __forceinline__ float at(int i) const { return float(v[i]); }
};
template <typename T>
__device__ __forceinline__ void store8(T* p, int n, const float (&f)[8]) {
    typedef T vec __attribute__((ext_vector_type(8), aligned(sizeof(T))));
    if (n >= 8) {
        vec t;
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = T(f[i]);
        *reinterpret_cast<vec*>(p) = t;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = T(f[i]);
    }
}

// Sums of N values over the TPR threads that share a row; `turn` alternates
// between two buffers, so one barrier is enough.
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], GFG_LDS float* part, int& turn) {
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = wave_reduce(v[n], [](float a, float b) { return a + b; });
    if constexpr (TPR > 64) {
        constexpr int W = TPR / 64;
        GFG_LDS float* const p = part + turn * (N * W);
        turn ^= 1;
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int n = 0; n < N; ++n) p[n * W + (threadIdx.x >> 6)] = v[n];
        }
        __syncthreads();
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

template <int TPR> constexpr int kRows = TPR == 64 ? 4 : 1;       // rows a workgroup holds at a time
template <int TPR> constexpr int kThreads = TPR == 64 ? 256 : TPR;

// The E8M0 byte of a block with largest magnitude bits `ab`, and 2^-t (0 for a
// block that has none): t the smallest integer with 448 * 2^t >= max, at least -127.
__device__ __forceinline__ uint32_t block_scale(uint32_t ab, float* inv) {
    if (ab >= 0x7F800000u) {
        *inv = 0.0f;
        return 255u;
    }
    int e = int(ab >> 23) - 127;
    uint32_t mant = ab & 0x7FFFFFu;
    if (e == -127) {
        const int lz = __builtin_clz(mant | 1u) - 8;
        mant = (mant << lz) & 0x7FFFFFu;
        e = -126 - lz;
    }
    int t = mant <= 0x600000u ? e - 8 : e - 7;
    t = ab == 0 ? 0 : t < -127 ? -127 : t;
    *inv = __builtin_ldexpf(1.0f, -t);
    return uint32_t(t + 127);
}

template <typename Y, typename R, int TPR>
__global__ __launch_bounds__(kThreads<TPR>) void residual_norm_kernel(NormArgs p) {
    __shared__ float part_smem[TPR > 64 ? 2 * TPR / 64 : 1];
    GFG_LDS float* const part = (GFG_LDS float*)part_smem;
    const int lane = threadIdx.x % TPR, chunks = (p.H + 7) / 8;
    int turn = 0;
    for (int64_t m = int64_t(blockIdx.x) * kRows<TPR> + threadIdx.x / TPR; m < p.M; m += int64_t(gridDim.x) * kRows<TPR>) {
        Row8<Y> y[CH];
        Row8<R> r[CH];
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int c = lane + j * TPR, n = p.H - 8 * c;
            y[j].zero();
            r[j].zero();
            if (c < chunks) {
                if (p.y) y[j].load(static_cast<const Y*>(p.y) + m * p.H + 8 * c, n);
                r[j].load(static_cast<const R*>(p.residual) + m * p.H + 8 * c, n);
            }
        }
        float ry = 1.0f;
        if (p.post && p.y) {
            float s[1] = {0.0f};
#pragma unroll
            for (int j = 0; j < CH; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) s[0] += y[j].at(i) * y[j].at(i);
            row_sums<TPR>(s, part, turn);
            ry = rsqrtf(s[0] / float(p.H) + p.eps);
        }
        const float token_gate = p.gate_kind == GFG_GATE_TOKEN ? p.gate[m] : 1.0f;
        float o[CH][8], s[1] = {0.0f};
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int c = lane + j * TPR, n = p.H - 8 * c;
            Row8<float> wp, g;
            wp.zero();
            g.zero();
            if (c < chunks) {
                if (p.post) wp.load(p.post + 8 * c, n);
                if (p.gate_kind == GFG_GATE_CHANNEL) g.load(p.gate + 8 * c, n);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float u = y[j].at(i);
                if (p.post) u = u * ry * wp.v[i];
                u *= p.gate_kind == GFG_GATE_CHANNEL ? g.v[i] : token_gate;
                o[j][i] = p.alpha * r[j].at(i) + u;
                s[0] += o[j][i] * o[j][i];
            }
            if (c < chunks && p.out) store8(static_cast<R*>(p.out) + m * p.H + 8 * c, n, o[j]);
        }
        float ro = 1.0f;
        if (p.weight) {
            row_sums<TPR>(s, part, turn);
            ro = rsqrtf(s[0] / float(p.H) + p.eps);
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                const int c = lane + j * TPR, n = p.H - 8 * c;
                Row8<float> w;
                w.zero();
                if (c < chunks) w.load(p.weight + 8 * c, n);
                float z[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) z[i] = o[j][i] * ro * w.v[i];
                if (p.normed && c < chunks) store8(static_cast<Y*>(p.normed) + m * p.H + 8 * c, n, z);
                if (p.q) {
                    // 16 neighbouring lanes hold a block of 128 channels
                    uint32_t ab = 0;
#pragma unroll
                    for (int i = 0; i < 8; ++i) ab = max(ab, __float_as_uint(z[i]) & 0x7FFFFFFFu);
                    ab = max(ab, uint32_t(dpp<0x128>(int(ab))));
                    ab = max(ab, uint32_t(dpp<0x124>(int(ab))));
                    ab = max(ab, uint32_t(dpp<0x122>(int(ab))));
                    ab = max(ab, uint32_t(dpp<0x121>(int(ab))));
                    float inv;
                    const uint32_t byte = block_scale(ab, &inv);
                    u32x2 code = {0x7F7F7F7Fu, 0x7F7F7F7Fu};
                    if (inv != 0.0f) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(z[4 * h] * inv, z[4 * h + 1] * inv, 0, false);
                            code[h] = uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(z[4 * h + 2] * inv, z[4 * h + 3] * inv, lo, true));
                        }
                    }
                    if (c < chunks) {
                        *reinterpret_cast<u32x2*>(p.q + m * p.H + 8 * c) = code;
                        if ((c & 15) == 0) p.scale[(c >> 4) * p.scale_ld + m] = uint8_t(byte);
                    }
                }
            }
        }
        if (p.stats && lane == 0) {
            p.stats[m] = ry;
            if (p.weight) p.stats[p.M + m] = ro;
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

template <typename Y, typename R, int TPR>
__global__ __launch_bounds__(kThreads<TPR>) void residual_norm_backward_kernel(BackArgs p) {
    __shared__ float part_smem[TPR > 64 ? 6 * TPR / 64 : 1];
    __shared__ float join_smem[TPR == 64 ? 2 * 64 * CH * 8 : 1];
    GFG_LDS float* const part = (GFG_LDS float*)part_smem;
    const int lane = threadIdx.x % TPR, chunks = (p.H + 7) / 8;
    const bool norm = p.dnormed && p.weight, post = p.post && p.y;
    int turn = 0;
    float sw[CH][8] = {}, sp[CH][8] = {};
    for (int64_t m = int64_t(blockIdx.x) * kRows<TPR> + threadIdx.x / TPR; m < p.M; m += int64_t(gridDim.x) * kRows<TPR>) {
        Row8<R> dout[CH], out[CH];
        Row8<Y> dz[CH], y[CH];
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int c = lane + j * TPR, n = p.H - 8 * c;
            dout[j].zero();
            out[j].zero();
            dz[j].zero();
            y[j].zero();
            if (c < chunks) {
                const int64_t at = m * p.H + 8 * c;
                if (p.dout) dout[j].load(static_cast<const R*>(p.dout) + at, n);
                if (norm) {
                    out[j].load(static_cast<const R*>(p.out) + at, n);
                    dz[j].load(static_cast<const Y*>(p.dnormed) + at, n);
                }
                if (p.y) y[j].load(static_cast<const Y*>(p.y) + at, n);
            }
        }
        const float ry = post ? p.stats[m] : 1.0f, ro = norm ? p.stats[p.M + m] : 0.0f;
        const float token_gate = p.gate_kind == GFG_GATE_TOKEN ? p.gate[m] : 1.0f;
        // A = sum h zh, B = sum wp g yh (dout + ro h), C = sum wp g yh zh (a token's g left out)
        float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int c = lane + j * TPR, n = p.H - 8 * c;
            Row8<float> w, wp, g;
            w.zero();
            wp.zero();
            g.zero();
            if (c < chunks) {
                if (norm) w.load(p.weight + 8 * c, n);
                if (post) wp.load(p.post + 8 * c, n);
                if (p.gate_kind == GFG_GATE_CHANNEL) g.load(p.gate + 8 * c, n);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float h = dz[j].at(i) * w.v[i], zh = out[j].at(i) * ro;
                float v = y[j].at(i) * ry;
                if (post) v *= wp.v[i];
                if (p.gate_kind == GFG_GATE_CHANNEL) v *= g.v[i];
                s[0] += h * zh;
                s[1] += v * (dout[j].at(i) + ro * h);
                s[2] += v * zh;
            }
        }
        row_sums<TPR>(s, part, turn);
        const float mean_h = s[0] / float(p.H);
        const float row = s[1] - ro * mean_h * s[2];          // sum wp g yh G
        if (p.gate_kind == GFG_GATE_TOKEN && p.dgate && lane == 0) p.dgate[m] = row;
        const float mean_y = token_gate * row / float(p.H);
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int c = lane + j * TPR, n = p.H - 8 * c;
            if (c >= chunks) continue;
            Row8<float> w, wp, g;
            w.zero();
            wp.zero();
            g.zero();
            if (norm) w.load(p.weight + 8 * c, n);
            if (post) wp.load(p.post + 8 * c, n);
            if (p.gate_kind == GFG_GATE_CHANNEL) g.load(p.gate + 8 * c, n);
            float dr[8], dy[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float zh = out[j].at(i) * ro, yh = y[j].at(i) * ry;
                const float G = dout[j].at(i) + ro * (dz[j].at(i) * w.v[i] - zh * mean_h);
                const float du = (p.gate_kind == GFG_GATE_CHANNEL ? g.v[i] : token_gate) * G;
                dr[i] = p.alpha * G;
                dy[i] = post ? ry * (wp.v[i] * du - yh * mean_y) : du;
                sw[j][i] += dz[j].at(i) * zh;
                sp[j][i] += token_gate * G * yh;
            }
            if (p.dresidual) store8(static_cast<R*>(p.dresidual) + m * p.H + 8 * c, n, dr);
            if (p.dy) store8(static_cast<Y*>(p.dy) + m * p.H + 8 * c, n, dy);
        }
    }
    if (!p.sums) return;
    float* const o = p.sums + int64_t(blockIdx.x) * 2 * p.H;
    if constexpr (TPR == 64) {                 // the four rows' waves, in order
        GFG_LDS float* const sum = (GFG_LDS float*)join_smem;      // [2][CH * 8][64]
        const int wave = threadIdx.x >> 6;
        for (int w = 0; w < 4; ++w) {
            if (wave == w) {
#pragma unroll
                for (int j = 0; j < CH; ++j)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        GFG_LDS float* const at = sum + (j * 8 + i) * 64 + lane;
                        if (w > 0) {
                            sw[j][i] += at[0];
                            sp[j][i] += at[64 * CH * 8];
                        }
                        at[0] = sw[j][i];
                        at[64 * CH * 8] = sp[j][i];
                    }
            }
            __syncthreads();
        }
        if (wave != 3) return;
    }
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int c = lane + j * TPR, n = p.H - 8 * c;
        if (c < chunks) {
            store8(o + 8 * c, n, sw[j]);
            store8(o + p.H + 8 * c, n, sp[j]);
        }
    }
}

// The sums over the workgroups' rows, in a fixed order: 16 lanes a channel.
__global__ __launch_bounds__(256) void norm_sums_kernel(const float* __restrict__ sums, int64_t P, int H, const float* post,
                                                        const float* gate, int gate_kind, float* dweight, float* dpost,
                                                        float* dgate, int accumulate) {
    __shared__ float part[2][16][17];
    const int l = threadIdx.x & 15, g = threadIdx.x >> 4, c = int(blockIdx.x) * 16 + l;
    float a = 0.0f, b = 0.0f;
    if (c < H)
        for (int64_t r = g; r < P; r += 16) {
            a += sums[r * 2 * H + c];
            b += sums[r * 2 * H + H + c];
        }
    part[0][g][l] = a;
    part[1][g][l] = b;
    __syncthreads();
    if (g || c >= H) return;
    a = b = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
        a += part[0][w][l];
        b += part[1][w][l];
    }
    auto put = [&](float* p, float v) {
        if (p) p[c] = accumulate ? p[c] + v : v;
    };
    put(dweight, a);
    // (without rows the factors are not read)
    put(dpost, P > 0 && gate_kind == GFG_GATE_CHANNEL ? gate[c] * b : b);
    if (gate_kind == GFG_GATE_CHANNEL) put(dgate, P > 0 && post ? post[c] * b : b);
}

// Lanes a row: enough for its chunks, CH each.
template <typename F>
void by_width(int64_t H, F f) {
    if (H <= 64 * 8 * CH) f(std::integral_constant<int, 64>{});
    else if (H <= 128 * 8 * CH) f(std::integral_constant<int, 128>{});
    else if (H <= 256 * 8 * CH) f(std::integral_constant<int, 256>{});
    else if (H <= 512 * 8 * CH) f(std::integral_constant<int, 512>{});
    else f(std::integral_constant<int, 1024>{});
}
template <typename F>
void by_type(int32_t dtype, int32_t residual_dtype, F f) {
    if (dtype == GFG_IN_F32) f(float{}, float{});
    else if (dtype == GFG_IN_BF16 && residual_dtype == GFG_IN_BF16) f(__bf16{}, __bf16{});
    else if (dtype == GFG_IN_BF16) f(__bf16{}, float{});
    else if (residual_dtype == GFG_IN_F16) f(_Float16{}, _Float16{});
    else f(_Float16{}, float{});
}

int64_t groups(int64_t M, int64_t H) {
    const int64_t rows = H <= 64 * 8 * CH ? 4 : 1, n = (M + rows - 1) / rows;
    return n < kMostGroups ? n : kMostGroups;
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
    if (H > kMaxH) return fail(GFG_EUNSUPPORTED, "%s: H=%lld above %lld", fn, (long long)H, (long long)kMaxH);
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
    by_width(a.H, [&](auto lanes) {
        constexpr int TPR = decltype(lanes)::value;
        const int64_t wgs = (a.M + kRows<TPR> - 1) / kRows<TPR>, most = int64_t(1) << 21;
        const dim3 grid(unsigned(wgs < most ? wgs : most)), block(kThreads<TPR>);
        by_type(dtype, residual_dtype, [&](auto y, auto r) {
            hipLaunchKernelGGL((residual_norm_kernel<decltype(y), decltype(r), TPR>), grid, block, 0, static_cast<hipStream_t>(stream), a);
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
    return M > 0 && H > 0 ? groups(M, H) * 2 * H * 4 : 0;
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
    const int64_t P = M > 0 ? groups(M, H) : 0;
    if (M > 0) {
        const BackArgs a{dout, dnormed, out, y, stats, weight, post_weight, gate, gate_kind, alpha, dresidual, dy, dgate,
                         sums ? static_cast<float*>(workspace) : nullptr, M, int(H)};
        by_width(H, [&](auto lanes) {
            constexpr int TPR = decltype(lanes)::value;
            by_type(dtype, residual_dtype, [&](auto yt, auto rt) {
                hipLaunchKernelGGL((residual_norm_backward_kernel<decltype(yt), decltype(rt), TPR>), dim3(unsigned(P)), dim3(kThreads<TPR>), 0, s, a);
            });
        });
        if (int rc = launched()) return rc;
    }
    if (!sums || (M == 0 && accumulate)) return GFG_OK;
    hipLaunchKernelGGL(norm_sums_kernel, dim3(unsigned((H + 15) / 16)), dim3(256), 0, s, static_cast<const float*>(workspace), P, int(H),
                       post_weight, gate, gate_kind, dweight, dpost_weight, dgate, accumulate);
    return launched();
}
