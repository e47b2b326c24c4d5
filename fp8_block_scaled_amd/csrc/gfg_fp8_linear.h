// The dense FP8 (E4M3) product of the linear layer: what its kernels share.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

namespace gfg {

// out[c] (+)= the sum over the row blocks of sums [RB][C].
struct SumJob {
    const float* sums;
    float* out;
    int64_t RB;
    int C, accumulate;
};

// One product d[m, n] = sum_k a[m, k] b[n, k] (+ bias[n]), both operands E4M3
// with K fastest, one E8M0 byte per row of `a` and 128 k, and either one per
// 128 x 128 block of `b` or one per row of `b` and 128 k.
struct F8Params {
    const uint8_t* a;        // [M][K]
    const uint8_t* a_scale;  // [KB][ld_a]
    const uint8_t* b;        // [N][K]
    const uint8_t* b_scale;  // blocks: [ceil(N/128)][KB] ; rows: [KB][ld_b]
    const float* bias;       // [N] or null
    void* d;                 // [M][N]
    int64_t rows;            // M
    int64_t ld_a, ld_b;
    int N, K, KB;            // KB = ceil(K / 128)
    int accumulate;          // d += (32-bit d only)
    int group_m, num_xcd;
    int m_tiles;             // tiles along M of the kernel's height
    unsigned tiles;
    unsigned sum_groups;     // workgroups behind the tiles' that take `sums` (0: none)
    SumJob sums;
};

// The kernel on 256 x 256 tiles (gfg_fp8_dense256.hip): whether its 32-bit
// offsets reach, and the launch.
bool fp8_256_fits(const F8Params& p, int out_dtype);
int launch_fp8_256(const F8Params& p, bool brow, int out_dtype, hipStream_t s);

}  // namespace gfg
