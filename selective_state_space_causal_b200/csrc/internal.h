// internal.h -- launchers behind the C ABI (host side, C++ only).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ssm {

enum class DType { F32 = 0, BF16 = 1 };

struct ConvArgs {
    const void *x;
    void *xc;
    const float *w;
    const float *bias;
    int64_t tok, D;
    int K;
    const int32_t *cu;  // nullptr: dense rows of tok / S
    int64_t S;
    const void *state_in;
    void *state_out;
    int apply_silu;
    DType x_dtype, state_dtype;
    bool vec;  // 16-byte vector path allowed (alignment checked by the caller)
};

struct ScanArgs {
    const void *u, *delta;
    const float *A;
    const void *B, *C;
    const float *Dskip;
    const void *z;
    const float *dt_bias;
    int delta_softplus;
    const float *h0;
    const int32_t *cu;
    int64_t S;
    void *y;
    float *h_final;
    int64_t tok, D;
    int N;
    DType dtype;
    int32_t *order;  // nullptr: sequences in index order; else S entries of scratch
    bool vec;
    // the state before every 8th token of each sequence, for the backward
    // pass, or nullptr; *ckpt_written reports whether the kernel that ran wrote
    // them (the pipelined kernel does, the other schedules do not)
    float *ckpt = nullptr;
    bool *ckpt_written = nullptr;
};

struct DecodeArgs {
    void *conv_state;
    float *ssm_state;
    const void *x, *dt, *B, *C, *z;
    const float *conv_w, *conv_b, *A, *Dskip, *dt_bias;
    int delta_softplus;
    const int32_t *idx;
    int64_t n_slots;
    void *y;
    int64_t Bt, D;
    int N, K;
    DType dtype, conv_dtype;
};

// The scan with one decay per head; strides are elements between tokens.
struct HeadScanArgs {
    const void *u, *delta;
    const float *A;
    const void *B, *C;
    int64_t u_stride, delta_stride, bc_stride;
    const float *Dskip, *dt_bias;
    int delta_softplus;
    const float *h0;
    const int32_t *cu;
    int64_t S;
    int64_t tok, H, P, G, N;
    DType dtype;
    void *workspace;
    // forward
    void *y = nullptr;
    float *h_final = nullptr;
    // backward
    const void *dy = nullptr;
    const float *dh_final = nullptr;
    void *du = nullptr, *ddelta = nullptr, *dB = nullptr, *dC = nullptr;
    float *dA = nullptr, *dDskip = nullptr, *ddt_bias = nullptr, *dh0 = nullptr;
};

struct HeadStepArgs {
    float *state;
    const void *x, *dt, *B, *C;
    int64_t x_stride, dt_stride, bc_stride;
    const float *A, *Dskip, *dt_bias;
    int delta_softplus;
    const int32_t *idx;
    int64_t n_slots;
    void *y;
    int64_t Bt, H, P, G, N;
    DType dtype;
};

// Norms around a mixer block. Gated: x and z with row strides, groups of
// `group` columns. Residual: r = residual + alpha * x_scale * x, group = D.
struct NormArgs {
    bool gated;
    const void *x, *z, *residual;
    int64_t x_stride, z_stride;
    const float *weight, *x_scale;
    float alpha, eps;
    int norm_before_gate;
    void *y, *residual_out;
    int64_t tok, D, group;
    DType dtype, res_dtype;
    // backward (x_res: the residual stream that the forward stored)
    const void *dy = nullptr, *x_res = nullptr, *dres_out = nullptr;
    void *dx = nullptr, *dz = nullptr, *dres = nullptr;
    float *dweight = nullptr, *dscale = nullptr;
    float *partials = nullptr;
};

size_t head_scan_workspace_bytes(int64_t tok, int64_t H, int64_t P, int64_t G, int64_t N, int64_t S,
                                 DType dtype);
size_t head_scan_bwd_workspace_bytes(int64_t tok, int64_t H, int64_t P, int64_t G, int64_t N,
                                     int64_t S, DType dtype);
cudaError_t launch_head_scan(const HeadScanArgs &a, cudaStream_t stream, int *launches);
cudaError_t launch_head_scan_bwd(const HeadScanArgs &a, cudaStream_t stream, int *launches);
cudaError_t launch_head_step(const HeadStepArgs &a, cudaStream_t stream, int *launches);
size_t norm_bwd_workspace_bytes(int64_t tok, int64_t D);
cudaError_t launch_norm_fwd(const NormArgs &a, cudaStream_t stream, int *launches);
cudaError_t launch_norm_bwd(const NormArgs &a, cudaStream_t stream, int *launches);

// Each returns cudaSuccess or the launch error.
cudaError_t launch_conv1d(const ConvArgs &a, cudaStream_t stream, int *launches);
cudaError_t launch_scan(const ScanArgs &a, cudaStream_t stream, int *launches);
cudaError_t launch_decode(const DecodeArgs &a, cudaStream_t stream, int *launches);

}  // namespace ssm
