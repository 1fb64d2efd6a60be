// Tables and launch interface of the operators of a layer in 8 bits:
// quantisation, 8-bit weights, the root-mean-square norm and the product.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "adamw.hpp"   // element types

namespace shampoo {

constexpr int kBlock8 = 128;         // values under one scale
enum : int { F8_E4M3 = 0, F8_E5M2 = 1 };
// Sources of the quantising kernels: the element types, then 8-bit matrices.
enum : int { SRC_E4M3 = 3, SRC_E5M2 = 4 };

// A matrix of floating-point values; pitch in elements.
struct Wide {
    uint64_t ptr;
    int64_t pitch;
};
// An 8-bit matrix: codes, and words of four exponent bytes for each group of
// four blocks along a row and each row.
struct Mat8 {
    uint64_t codes, scales;          // codes 0: absent
    int64_t pitch;                   // bytes from row to row
    int64_t spitch;                  // words from group to group
};

// One matrix (or one tile list entry's matrix) to be quantised.
struct QuantJob {
    Wide x;                          // wide source
    Mat8 src;                        // or an 8-bit one
    Mat8 rows, cols;                 // outputs: the matrix, its transpose
    int64_t nrows, ncols;            // of the source
};
// The matrix and the 128 x 128 tile of one workgroup of the weights' kernel.
struct QuantTile {
    int32_t job, pad_;
    int32_t row, col;                // in tiles
};
constexpr int kWeightBatch = 400;    // addresses per launch of the binding kernel (3.2 KB of
                                     // kernel arguments)
struct AddrBatch {
    uint64_t a[kWeightBatch];
};

struct NormFwdArgs {
    Wide x, res, total, out;         // ptr 0: absent
    Mat8 out8;
    const void* w;
    float* rstd;
    int64_t rows, dim;
    double eps;
    int32_t w_type, out_type;
};

struct NormBwdArgs {
    Wide g, z, add, dz;
    const void* w;
    const float* rstd;
    float* dw;                       // or null
    float* partials;                 // slots x dim
    int64_t rows, dim;
    int32_t w_type, accumulate, slots;
};

struct Mul8Args {
    Mat8 a, b;
    Wide c;
    float* partials;                 // splits x M x N, or null
    int64_t m, n, k;
    int32_t c_type, accumulate;
    int32_t fa, fb;                  // formats
    int32_t splits, blocks_per_split;
};

hipError_t launch_quantize(int src, int fmt_rows, int fmt_cols, const QuantJob& j, hipStream_t s);
hipError_t launch_weights8(int src, const QuantJob* jobs, const QuantTile* tiles, int ntiles, hipStream_t s);
hipError_t launch_weights8_bind(QuantJob* jobs, int first, int n, const AddrBatch& b, hipStream_t s);
// Whether the rows are fewer than a launch takes.
bool norm_fwd_fits(int64_t rows, int64_t dim);
hipError_t launch_norm_fwd(int xt, int rt, const NormFwdArgs& a, hipStream_t s);
int norm_bwd_slots(int64_t rows, int64_t dim);
hipError_t launch_norm_bwd(int gt, int zt, const NormBwdArgs& a, hipStream_t s);

// How a product is cut up: the kernel's tile and the parts of its k.
struct Mul8Plan {
    int32_t kind;
    int32_t splits, blocks_per_split;
};
Mul8Plan plan_mul8(int64_t m, int64_t n, int64_t k, int type);
size_t mul8_workspace(const Mul8Plan& p, int64_t m, int64_t n);
// Whether a launch takes that many tiles.
bool mul8_fits(const Mul8Plan& p, int64_t m, int64_t n);
hipError_t launch_mul8(const Mul8Plan& p, const Mul8Args& a, hipStream_t s);

}  // namespace shampoo
