// The 8-bit linear layer's operators: parameters of their kernels, and the
// host's checks and launch rules (plain C++, no HIP).
#pragma once

#include "tp_internal.hpp"

namespace tp {

constexpr int kOpBlock = 128;                 // numbers that share a scale
constexpr int64_t kOpMaxRows = int64_t(1) << 31;
constexpr int64_t kOpMaxCols = int64_t(1) << 24;
constexpr int64_t kOpMaxStride = int64_t(1) << 36;
constexpr int kOpCus = 256;                   // compute units of the device

TP_HD constexpr int64_t op_ceil(int64_t a, int64_t b) { return (a + b - 1) / b; }
TP_HD constexpr int type_bytes(int type)
{
    return type == TP_FP32 ? 4 : type == TP_BF16 || type == TP_FP16 ? 2 : 1;
}

// ---------------------------------------------------------------- row kernels
// The norm and its gradient: a workgroup holds a row in registers, kRowUnits
// units of 8 elements a lane at most (or one, where rows are few and a row is
// spread over more lanes), and walks over rows.
constexpr int kRowUnits = 4;
constexpr int kRowMaxWaves = 16;
// Waves of a workgroup at most: with kRowUnits units a lane needs more than
// the 128 registers that 16 waves leave it.
TP_HD constexpr int row_max_waves(int units) { return units == 1 ? kRowMaxWaves : 8; }
constexpr int kRowRedBytes = 2 * kRowMaxWaves * 4;   // two sets of the waves' sums
constexpr int kRowCutBytes = 256;             // a wave's dwords of a unit cut by the row's end

// LDS of one wave: `tensors` rows' units and cut units.
TP_HD constexpr int row_wave_lds(int tensors, int units, int bytes)
{
    return tensors * (units * 64 * 8 * bytes + kRowCutBytes);
}

// Tensors that a wave has places for. With one unit a lane the weight has its
// own, so that it and the first row are waited for together; otherwise it
// passes through the first tensor's before any row does.
TP_HD constexpr int row_places(int tensors, int units) { return units == 1 ? tensors + 1 : tensors; }

// Partial sums of the weight's gradient: rows of whole runs of 512, a wave's
// units.
constexpr int kPartialRun = 512;
TP_HD constexpr int64_t partial_pitch(int64_t cols) { return op_ceil(cols, kPartialRun) * kPartialRun; }

// Loads non-temporal and stores written through to memory; loads or both with
// the caches' ordinary policy.
enum RowPolicy : int { kRowPast = 0, kRowStoresPast = 1, kRowCached = 2 };

struct RowPlan {
    int units;       // units a lane holds: 1 or kRowUnits; 0: the row does not fit, it is read twice
    int waves;
    int lds_bytes;
    int64_t grid;
};

struct NormParams {
    const void *x, *r, *w;
    void *sum, *out;
    float *scale, *rstd;
    int64_t x_stride, r_stride, sum_stride, out_stride;   // bytes
    int64_t rows;
    int32_t cols;
    float eps;
};

struct NormGradParams {
    const void *dy, *x, *ds, *w;
    const float *rstd;
    void *dx;
    float *dw;
    float *partial;          // `groups` rows of partial_pitch(cols) sums
    int64_t dy_stride, x_stride, ds_stride, dx_stride;    // bytes
    int64_t rows;
    int32_t cols;
    int32_t groups;
};

struct QuantParams {
    const void *x;
    uint8_t *q, *qt;
    float *scale, *scale_t;
    int64_t x_stride, q_stride, qt_stride;                // bytes
    int64_t rows, cols;
    int32_t square;
    int32_t across;          // blocks of 128 columns
    int32_t cached;          // loads with the caches' ordinary policy
};

struct MatmulParams {
    const uint8_t *a, *b;
    const float *sa, *sb;
    void *out;
    float *partial;          // `splits` products of m x n, or null
    int64_t a_stride, b_stride, out_stride;               // bytes
    int64_t m, n;
    int32_t k, blocks;       // blocks: ceil(k / 128)
    int32_t out_type;
    int32_t splits;          // workgroups that share a tile's sum
    int32_t tiles_m, tiles_n;
};

// Whether the product's blocks are summed in fp32 (through fp16 instructions)
// rather than by the 8-bit instructions, which keep fewer bits.
TP_HD constexpr bool matmul_wide(int out_type) { return out_type != TP_BF16; }

// How the product is cut; see matmul_plan.
enum MatmulShape : int32_t { kMatmulSkinny = 0, kMatmul128 = 1, kMatmul128x256 = 2, kMatmul256 = 3, kMatmul64 = 4 };

// Stages of LDS that the operands' blocks pass through.
TP_HD constexpr int matmul_stages(int shape)
{
    // (64 x 64 with a fourth stage: 1 to 3 % slower)
    return shape == kMatmul64 || shape == kMatmul128x256 ? 3 : 2;
}

// LDS of a workgroup: the stages, two sets of four blocks' scales, and a place
// for loads of nothing; of the few-rows kernel, each wave's slots and scales.
constexpr int kSkinnyWaves = 8;
TP_HD constexpr int matmul_tile_lds(int tile_m, int tile_n, int stages)
{
    return (tile_m + tile_n) * (stages * kOpBlock + 2 * 16) + 1024;
}
TP_HD constexpr int matmul_skinny_lds(int tile_m, int slots)
{
    return kSkinnyWaves * (tile_m + 16) * (slots * kOpBlock + 2 * 16);
}

struct MatmulPlan {
    int shape;               // MatmulShape
    int tile_m, tile_n;
    int waves;               // of a workgroup
    int stages;              // of LDS; slots of each wave of the few-rows kernel
    int lds_bytes;
    int splits;
    int64_t grid;            // workgroups
    int64_t partial_bytes;
};

constexpr int kQuantLdsBytes = 20992;         // of a workgroup of the quantiser

RowPlan norm_plan(int64_t rows, int64_t cols, int type, bool residual);
RowPlan norm_grad_plan(int64_t rows, int64_t cols, int type, bool more);
// The RowPolicy of a call.
int norm_policy(const NormParams &p, int type, int out_type);
int norm_grad_policy(const NormGradParams &p, int type);
bool quantize_cached(const QuantParams &p, int type);
// Rows of partial sums of dw: the workgroups of the kernel that makes them.
// The same with and without the second gradient, so that one workspace fits.
int64_t norm_grad_groups(int64_t rows, int64_t cols, int type);
MatmulPlan matmul_plan(int64_t m, int64_t n, int64_t k, int out_type);

int plan_rms_norm(uintptr_t x, int64_t x_stride, uintptr_t r, int64_t r_stride, uintptr_t w,
                  int64_t rows, int64_t cols, int type, float eps, uintptr_t sum,
                  int64_t sum_stride, uintptr_t out, int64_t out_stride, int out_type,
                  uintptr_t scale, uintptr_t rstd, tp_plan *plan);
int plan_rms_norm_backward(uintptr_t dy, int64_t dy_stride, uintptr_t x, int64_t x_stride,
                           uintptr_t w, uintptr_t rstd, uintptr_t ds, int64_t ds_stride,
                           int64_t rows, int64_t cols, int type, uintptr_t dx, int64_t dx_stride,
                           uintptr_t dw, uintptr_t workspace, int64_t workspace_bytes,
                           tp_plan *plan);
int plan_block_quantize(uintptr_t x, int64_t x_stride, int64_t rows, int64_t cols, int type,
                        int square, int out_type, uintptr_t q, int64_t q_stride, uintptr_t scale,
                        uintptr_t qt, int64_t qt_stride, uintptr_t scale_t, tp_plan *plan);
int plan_block_matmul(uintptr_t a, int64_t a_stride, int a_type, uintptr_t sa, uintptr_t b,
                      int64_t b_stride, int b_type, uintptr_t sb, int b_square, int64_t m,
                      int64_t n, int64_t k, uintptr_t out, int64_t out_stride, int out_type,
                      uintptr_t workspace, int64_t workspace_bytes, tp_plan *plan);

int64_t rms_norm_backward_workspace(int64_t rows, int64_t cols, int type);
int64_t block_matmul_workspace(int64_t m, int64_t n, int64_t k, int out_type);

// Launchers: each returns a hipError_t value.
int launch_rms_norm(const NormParams &p, int type, int out_type, void *stream);
int launch_rms_norm_backward(const NormGradParams &p, int type, void *stream);
int launch_block_quantize(const QuantParams &p, int type, int out_type, void *stream);
// One entry for each pair of operand types, each a compilation of its own.
int launch_matmul_e4m3_e4m3(const MatmulPlan &plan, const MatmulParams &p, int square, void *stream);
int launch_matmul_e4m3_e5m2(const MatmulPlan &plan, const MatmulParams &p, int square, void *stream);
int launch_matmul_e5m2_e4m3(const MatmulPlan &plan, const MatmulParams &p, int square, void *stream);
int launch_matmul_e5m2_e5m2(const MatmulPlan &plan, const MatmulParams &p, int square, void *stream);
int launch_block_matmul(const MatmulParams &p, int a_type, int b_type, int square, void *stream);

}  // namespace tp
