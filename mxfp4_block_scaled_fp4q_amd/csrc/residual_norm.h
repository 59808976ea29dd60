// Operands of the residual norms, as the host hands them to the kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp4q {

constexpr int kPostNone = 2;  // FP4Q_NO_NORM

// Group g of the gate holds rows g * gate_rows .. ; without a gate, gate_rows
// is the number of rows.  *_bf16: the operand's type, fp32 otherwise.
struct ResidualNorm {
    int64_t rows, cols, gate_rows;
    const void *x, *b, *gate, *post_weight, *post_bias, *weight, *bias;
    int64_t ldx, ldb, ldg;
    int x_bf16, b_bf16, gate_bf16, w_bf16, y_bf16;
    int post, rms;  // kind of the norm behind the block (kPostNone), whether the other is an RMS norm
    float x_scale, branch_scale, eps;
    void *xo, *y;
    int64_t ldxo, ldy;
    uint8_t *codes, *scales;
    float *post_mean, *post_rstd, *mean, *rstd;
};
struct ResidualNormGrad {
    int64_t rows, cols, gate_rows;
    const void *dy, *dxo, *xo, *b, *gate, *post_weight, *post_bias, *weight;
    int64_t lddy, lddxo, ldxo, ldb, ldg;
    int dy_bf16, x_bf16, b_bf16, gate_bf16, w_bf16;
    int post, rms;
    float x_scale, branch_scale;
    const float *post_mean, *post_rstd, *mean, *rstd;
    void *dx, *db;
    int64_t lddx, lddb;
    float *dpost_weight, *dpost_bias, *dgate, *dweight, *dbias;
};

hipError_t launch_residual_norm(const ResidualNorm& a, hipStream_t s);
size_t residual_norm_grad_workspace_bytes(int64_t rows, int64_t cols, int64_t gate_rows);
hipError_t launch_residual_norm_grad(const ResidualNormGrad& a, void* ws, hipStream_t s);

}  // namespace fp4q
