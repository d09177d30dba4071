// mx_fp4.cuh -- what the translation units of the microscaled 4-bit operators share.
//
// Numbers: e2m1, two to a byte, the lower column in the low nibble; a scale for each block
// of a row's columns: e8m0 for 32, or e4m3 for 16 and one fp32 factor of the tensor.
#pragma once

#include "mx_common.cuh"
#include "mx_internal.h"
#include "mx_moe.h"

namespace mx {
namespace fp4 {

constexpr int kStageCols = 256;  // columns of one ring stage: 128 bytes of a row

struct QuantArgs {
    const void *x;  // [rows][cols]
    int64_t ldx;
    int rows, cols, bf16;
    int vx, vq;     // pieces of x, of q may be moved as vectors
    uint8_t *q, *scales;  // scales [ceil(cols / 256)][rows][256 / block]
    int64_t ldq;
    const float *tensor_scale;  // e4m3; nullable
};
cudaError_t launch_quantize(int block, const QuantArgs &a, int sms, cudaStream_t s);

struct GemmArgs {
    CUtensorMap wm, xm;      // packed bytes of the weights [E][N][K / 2] and of the rows
    int rows, K, N, E;
    const int32_t *offsets;  // [E + 1] first row of each matrix's group, nullable: one group of all rows
    const uint8_t *sx, *sw;  // scales of the rows [stage][rows][256 / block], of the weights as packed
    const float *tx, *tw;    // factors of the rows and of each matrix, nullable
    void *out;
    int64_t ldo;
    int out_bf16, out_vec;
    unsigned *err;
    int stages, cl;          // ring depth, cluster size (split of the inner dimension)
};

// One row (mx_fp4_gemv.cu), which lies in shared memory; the rule that takes it ends at 6144 columns.
struct GemvArgs {
    int K, N;
    const uint8_t *q, *sx;   // the row, its scales
    const uint8_t *w, *sw;   // the matrix, its scales as packed
    int64_t ldw;
    const float *tx, *tw;    // nullable
    void *out;
    int out_bf16;
};
cudaError_t launch_gemv(int block, const GemvArgs &a, cudaStream_t s);

struct PackArgs {
    const uint8_t *scales;  // [count][rows][nb], row pitch ld
    int64_t ld;
    int rows, nb, count, block;
    uint8_t *out;           // [count][tiles of 128 rows][stages][512-byte pieces]
};
cudaError_t launch_pack(const PackArgs &a, cudaStream_t s);

// What a sum is multiplied by, one after the other, for the factors tx and tw: their product where that is a normal
// number, so that a large factor meets the small one and not the sum; else both are above 1, or both below, and one after the
// other leaves fp32's range only where the result does.
struct Factors {
    float a, b;
};
__device__ __forceinline__ Factors factors_of(float tx, float tw)
{
    const float both = tx * tw;
    return both >= 0x1p-126f && both < INFINITY ? Factors{both, 1.0f} : Factors{tx, tw};
}

__host__ __device__ constexpr int stages_of(int cols) { return (cols + kStageCols - 1) / kStageCols; }
__host__ __device__ constexpr int atoms_of(int block) { return 64 / block; }  // pieces of 128 rows in a stage

// Token tiles of launch_gemm: 16, 32, 64, 128, 224.
cudaError_t launch_gemm(int block, int nt, const GemmArgs &a, int grid, cudaStream_t s);
size_t gemm_smem(int block, int nt, int stages);
constexpr int box_rows(int nt) { return nt < 32 ? nt : 32; }  // token rows of one copy

}  // namespace fp4
}  // namespace mx
