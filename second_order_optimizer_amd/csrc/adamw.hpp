// Tables and launch interface of the first-order operators (the AdamW step
// over many tensors and the global gradient norm).
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

namespace shampoo {

constexpr int kRun = 256;            // elements of one run: the unit of a tensor's state, and
                                     // of one scale of 8-bit moments
constexpr int kBindBatch = 200;      // pointer pairs per launch of the pointer-table kernel
                                     // (3.2 KB of kernel arguments)

enum : int { DT_F32 = 0, DT_BF16 = 1, DT_F16 = 2 };

// One tensor of an AdamW plan.
struct AdamwTensor {
    uint64_t p_ptr, g_ptr;   // weights and gradient (0: no gradient, the tensor is left as it is)
    int64_t numel;
    int64_t state_run;       // first run in the moments' region (fp32 or 8-bit)
    int64_t rem_run;         // first run in the remainders' region (bf16 weights)
    double lr_scale, weight_decay;
    int32_t id, pad_;        // index in the plan's list
};

// Up to kTileRuns runs of one tensor, the work of one workgroup of four waves.
constexpr int kTileRuns = 8;
struct AdamwTile {
    int32_t tensor, pad_;    // index into the tensor table
    int64_t run0;            // first run within the tensor
};

// The step counter and what follows from it.  Every workgroup has its own
// copy, which it reads first and advances last, so that one launch is the
// whole step, replayed launches count on, and no workgroup waits for another.
struct AdamwClock {
    int64_t t;               // steps done
    int64_t k;               // steps that the corrections count: t, or the tensor's own
    double b1k, b2k;         // beta^(k + 1)
    double inv1;             // 1 / (1 - beta1^(k + 1))
    float inv_root2;         // 1 / sqrt(1 - beta2^(k + 1))
    int32_t pad_[5];
};
static_assert(sizeof(AdamwClock) == 64, "one clock per 64 bytes");

// Device record of the gradient norm (same layout as the public one).
struct ClipRecord {
    float norm, coef;
    int32_t nonfinite, pad_;
};

struct AdamwArgs {
    const AdamwTensor* tensors;
    const AdamwTile* tiles;
    AdamwClock* clocks;      // one per workgroup of this launch
    const ClipRecord* clip;  // or null
    const float* lr_dev;     // or null: lr
    double lr;
    double beta1, beta2;
    float b1, c1, b2, c2, eps;   // beta1, 1 - beta1, beta2, 1 - beta2, eps
    uint32_t seed_mixed;
    int32_t ntiles;
    int32_t stream_past;         // the step touches more than the caches hold
    int32_t per_tensor;          // the corrections count a tensor's own steps
    float *m, *v;                // fp32 moments
    unsigned char *m8, *s8;      // 8-bit moments: e4m3 of m and sqrt(v)
    float *m_scale, *s_scale;
    int16_t* rem;
};

struct PtrBatch {
    uint64_t a[kBindBatch], b[kBindBatch];
};

// One gradient of a norm plan.
struct NormTensor {
    uint64_t g_ptr, out_ptr;  // 0: absent
    int64_t numel;
    int32_t dtype, pad_;
};
struct NormTile {
    int32_t tensor, pad_;
    int64_t first;            // first element of the tile
};
constexpr int kNormWaves = 8;    // waves of a workgroup of the norm
constexpr int kNormGroups = 16;   // groups that a large grid counts its workgroups in
constexpr int kNormPiece = 1024;  // elements that a wave has in flight together; a tile is some

struct NormArgs {
    const NormTensor* tensors;
    const NormTile* tiles;
    int32_t ntiles, pieces;   // pieces of a tile
    double* partials;         // one per workgroup
    int32_t* tickets;         // kNormGroups + 1 counts, 128 bytes apart
    int32_t stream_past, pad_; // the gradients are more than the caches hold
    ClipRecord* record;
    double max_norm, grad_scale;
};

// 32 bits mixed by two rounds of shift-xor and odd multiplication.
__host__ __device__ inline uint32_t mix32_rest(uint32_t x) {   // after the first shift-xor
    x *= 0xFD63ED5Bu;
    x ^= x >> 15;
    x *= 0x7BC73A83u;
    x ^= x >> 16;
    return x;
}
__host__ __device__ inline uint32_t mix32(uint32_t x) { return mix32_rest(x ^ (x >> 16)); }

int norm_grid(int64_t ntiles);

hipError_t launch_adamw(int param, int grad, bool bits8, const AdamwArgs& a, hipStream_t s);
// which: 1 the step count, 2 the corrections' count and factors
hipError_t launch_adamw_clock(AdamwClock* clocks, int n, const AdamwClock& c, int which, hipStream_t s);
hipError_t launch_adamw_bind(AdamwTensor* tensors, int first, int n, const PtrBatch& b, int which,
                             hipStream_t s);
hipError_t launch_norm(const NormArgs& a, hipStream_t s);
hipError_t launch_clip(const NormArgs& a, hipStream_t s);
hipError_t launch_norm_bind(NormTensor* tensors, int first, int n, const PtrBatch& b,
                            hipStream_t s);

}  // namespace shampoo
