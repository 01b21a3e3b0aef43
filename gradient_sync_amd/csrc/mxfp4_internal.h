// Internal declarations of the 4-bit block-scaled (e2m1 with a power-of-two
// scale per 32 values) kernels: quantisation, expansion and product.
#pragma once

#include "dps_internal.h"

namespace dps {

// A quantised [rows, cols] matrix, blocks of 32 along the columns.
//   codes : rows of 64 * ceil(cols / 128) bytes; column j's code in bits
//           4 (j % 2) .. + 3 of byte j / 2; codes past cols are zero.
//   scales: one byte per block (exponent + 127; 255: the block is NaN), in
//           256-byte tiles of 16 rows x 16 blocks, tiles of one row group
//           consecutive. Within a tile the byte of row i, block b is at
//           (16 (b % 4) + i) * 4 + b / 4: lane 16 (b % 4) + i of a wave gets
//           its bytes for four consecutive 16x16x128 matrix instructions in
//           one 32-bit load.
__host__ __device__ inline long long mx_pitch(long long cols) { return (cols + 127) / 128 * 64; }
__host__ __device__ inline long long mx_scale_tiles(long long cols) { return (cols + 511) / 512; }
__host__ __device__ inline long long mx_scale_at(long long row, int block, long long tiles)
{
    return ((row >> 4) * tiles + (block >> 4)) * 256 + (((block & 3) << 4) + (int)(row & 15)) * 4 +
           ((block >> 2) & 3);
}

struct MxQuantParams {
    const char *src;
    long long rows, cols, ld;       // ld in elements
    unsigned char *codes, *scales;      // of src, or NULL
    unsigned char *codes_t, *scales_t;  // of its transpose, or NULL
};
hipError_t launch_mxfp4_quantize(const MxQuantParams &p, int dt, hipStream_t stream);

struct MxExpandParams {
    const unsigned char *codes, *scales;
    char *dst;
    long long rows, cols, ld;
};
hipError_t launch_mxfp4_dequantize(const MxExpandParams &p, int dt, hipStream_t stream);

// c[m, n] = a[m, k] . b[n, k]^T
struct MxGemmParams {
    const unsigned char *a, *a_scales;
    const unsigned char *b, *b_scales;
    char *c;
    const char *x;                  // few rows: a as plain values, quantised on the way (a unused)
    long long ldx;
    long long m, n, k;
    int accumulate;                 // add to c (fp32)
};
constexpr int kMxFewRows = 16;      // rows up to which x may be taken as it is
// whether a product of m rows of plain values quantises them inside
bool mx_quantize_inside(long long m, long long n, long long k);
// x_dt < 0: a is given as codes
hipError_t launch_mxfp4_gemm(const MxGemmParams &p, int c_dt, int x_dt, hipStream_t stream);

}  // namespace dps
