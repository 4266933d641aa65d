// Internal declarations of the microscaled 4-bit matrices: quantization by rows
// and by columns, dequantization and the product (gfx950 only).
#pragma once

#include "common.h"

namespace i8mp {

constexpr int kMxBlock = 32;    // elements under one scale
constexpr int kMxPad = 128;     // rows are padded with zeros to whole multiples: 64 bytes of codes, 4 scales

// A [rows x k] matrix of E2M1 codes, two a byte, and one E8M0 scale a block.
struct Mx4 {
    uint8_t* codes; int64_t ldc;    // bytes; 16-byte aligned, ldc a multiple of 16
    uint8_t* scales; int64_t lds;   // bytes; 4-byte aligned, lds a multiple of 4
    int64_t rows, k;
    __host__ __device__ int64_t kp() const { return (k + kMxPad - 1) / kMxPad * kMxPad; }
};

struct MxQuantArgs {
    const half_bits* x;             // [m x k], or with `columns` [q.k x q.rows]: its transpose is quantized
    int64_t ldx;
    bool bf16;
    bool columns;
    Mx4 q;
    Mx4 rows;                       // with `columns`, where its codes are given: x quantized by rows beside it
    // set by the launcher
    bool aligned, runs;             // by columns: x can be read in whole words; each XCD gets a run of workgroups
    bool few;                       // by rows: a lane takes one row
    int32_t lane_shift;             // and lanes along a row
    uint32_t block0, blocks_x, blocks_y;  // first workgroup, workgroups along a row of them and rows
};
constexpr int kMxJobs = 4;
struct MxQuantJobs {
    MxQuantArgs job[kMxJobs];
    int32_t count;
};

struct MxDequantArgs {
    Mx4 q;
    int32_t out_dtype;
    void* out; int64_t ldout;
};

struct MxGemmArgs {
    Mx4 a, b;                       // out [a.rows x b.rows] = a . b^T + bias
    const void* bias;               // nullable, [b.rows] of out's type
    int32_t out_dtype;
    void* out; int64_t ldout;
    const half_bits* x; int64_t ldx;  // launch_mx4_decode: if given, a's 16-bit form, quantized on the way
    float* part;                    // workspace of mx4_gemm_workspace() bytes
    // set by the launcher: the sums over k in so many parts of so many stages, each with an output of its own
    int32_t parts, part_stages;
    int64_t part_bytes;
    bool past;                      // out passes the last-level cache by
};

// Up to kMxJobs matrices of one type, in one launch; empty ones are passed over.
hipError_t launch_mx4_quantize(const MxQuantArgs* args, int count, hipStream_t stream);
// whether a matrix that is wanted by rows and by columns is better quantized by one job (MxQuantArgs::rows) than by two
bool mx4_quantize_both(int64_t rows, int64_t cols);
hipError_t launch_mx4_dequantize(const MxDequantArgs& a, hipStream_t stream);
// workspace of a product of these sizes (0: none needed)
size_t mx4_gemm_workspace(int64_t m, int64_t n, int64_t k);
hipError_t launch_mx4_gemm(const MxGemmArgs& g, hipStream_t stream);
// Two products whose outputs are of one 16-bit type.
hipError_t launch_mx4_gemm_pair(const MxGemmArgs& a, const MxGemmArgs& b, hipStream_t stream);
// The product of a few rows, where mx4_decode_fits: the weights streamed through the matrix cores.  x in place of a's
// codes (and of out's type) where mx4_decode_quantizes.
constexpr int kMxDecodeRows = 16;
bool mx4_decode_fits(int64_t m, int64_t k);
bool mx4_decode_quantizes(int64_t m, int64_t k);
hipError_t launch_mx4_decode(const MxGemmArgs& g, hipStream_t stream);

}  // namespace i8mp
