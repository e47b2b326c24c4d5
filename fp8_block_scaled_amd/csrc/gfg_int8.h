// Types and parameters shared by the int8 product kernels (gfx950).
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "gfg_device.h"

namespace gfg {

typedef int v4i __attribute__((ext_vector_type(4)));

enum I8Layout { DENSE = 0, CONTIG = 1, MASKED = 2 };

// Arguments of one int8 product launch.
struct I8Params {
    const uint8_t* a;        // [rows][K] (masked: [G][rows][K])
    const float* a_scale;    // [rows] (masked: [G][rows])
    const uint8_t* b;        // [G][N][K]
    const float* b_scale;    // [G][N]
    const float* bias;       // [N] or null (dense)
    const int32_t* meta;     // grouped_layout or masked_m
    void* d;                 // [rows][N] (masked: [G][rows][N])
    int64_t rows;            // masked: rows per group
    int N, K, G;
    int m_tiles;             // row tiles of the kernel's tile height, over all groups (the 256 x 256 kernel: of 128 rows)
    int tiles_per_group;     // masked: row tiles per group (not the 256 x 256 kernel)
    unsigned tiles;          // output tiles of the launch (not the 256 x 256 kernel)
    int group_m, num_xcd;    // tile order of the 256 x 256 kernel
};

// The 256 x 256-tile kernel (gfg_int8_gemm256.hip).  The caller has
// checked: N at most 2^22, and for the grouped layouts at most 4096 tiles of
// 128 rows.
int launch_int8_256(const I8Params& p, int layout, int out_dtype, hipStream_t s);

}  // namespace gfg
