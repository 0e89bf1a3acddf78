// head_step.cu -- one decode token per row for the scan with one decay per head.
//
//   S = exp(d A) S + d x B^T (P x N, in place at the row's slot), y = S C + Dskip x.
//
// Bound by memory: the state is read and written once, 8 bytes per entry, against
// five flops. One CTA has one row's head; LR lanes share a state row (4 entries
// each), and a lane issues the loads of up to 8 state rows before it uses the first.
// Measured on a B200: 256 rows of 128 heads of 64 x 128 (2.15 GB) 365 us, 5.9 TB/s or 90%
// of a copy's rate (382 us from call to call); one row of 24 heads 5 us, a launch's latency.
#include "head_scan.cuh"

namespace ssm {
namespace {

template <typename T>
struct StepArgs {
    float *state;
    const T *x, *dt, *B, *C;
    int64_t x_stride, dt_stride, bc_stride;
    const float *A, *Dskip, *dt_bias;
    int softplus;
    const int32_t *idx;
    int64_t n_slots;
    T *y;
    int H, P, G, N;
};

template <typename T, int LR, bool VEC>
__global__ void __launch_bounds__(256) head_step_kernel(StepArgs<T> a)
{
    constexpr int RPW = 32 / LR;      // state rows of a warp at a time
    constexpr int RPB = 8 * RPW;      // and of the CTA
    constexpr int U = 8;              // state rows of a lane in flight
    const int64_t b = blockIdx.x / a.H;
    const int h = (int)(blockIdx.x % a.H);
    const int64_t slot = a.idx ? (int64_t)a.idx[b] : b;
    if (slot < 0 || slot >= a.n_slots) return;
    const int g = h / (a.H / a.G), P = a.P, N = a.N;
    const int l = threadIdx.x % LR, r0 = (threadIdx.x / 32) * RPW + (threadIdx.x % 32) / LR;
    const float d = head_step(to_f32(a.dt[b * a.dt_stride + h]) + (a.dt_bias ? a.dt_bias[h] : 0.0f),
                              a.softplus);
    const float lg = d * a.A[h];
    const float da = expf(lg < kHeadMinLog ? kHeadMinLog : lg);
    const float skip = a.Dskip ? a.Dskip[h] : 0.0f;
    float Bv[4], Cv[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int n = VEC ? 4 * l + e : l + LR * e;
        const int64_t at = b * a.bc_stride + (int64_t)g * N + n;
        Bv[e] = n < N ? to_f32(a.B[at]) : 0.0f;
        Cv[e] = n < N ? to_f32(a.C[at]) : 0.0f;
    }
    float *st = a.state + (slot * a.H + h) * (int64_t)P * N;
    const T *x = a.x + b * a.x_stride + (int64_t)h * P;
    T *y = a.y + (b * a.H + h) * (int64_t)P;
    for (int p0 = 0; p0 < P; p0 += RPB * U) {
        float v[U][4], xv[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int p = p0 + r0 + RPB * i;
            const bool in = p < P;
            if (VEC) {
                float4 q = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (in && 4 * l < N) q = __ldcs(reinterpret_cast<const float4 *>(st + (int64_t)p * N) + l);
                v[i][0] = q.x; v[i][1] = q.y; v[i][2] = q.z; v[i][3] = q.w;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[i][e] = in && l + LR * e < N ? st[(int64_t)p * N + l + LR * e] : 0.0f;
            }
            xv[i] = in ? to_f32(x[p]) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int p = p0 + r0 + RPB * i;
            if (p0 + RPB * i >= P) break;  // the same for the whole CTA
            const float w = d * xv[i];
            float s = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[i][e] = fmaf(da, v[i][e], w * Bv[e]);
                s = fmaf(v[i][e], Cv[e], s);
            }
#pragma unroll
            for (int o = LR / 2; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (p < P) {
                if (VEC) {
                    if (4 * l < N)
                        __stcs(reinterpret_cast<float4 *>(st + (int64_t)p * N) + l,
                               make_float4(v[i][0], v[i][1], v[i][2], v[i][3]));
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (l + LR * e < N) st[(int64_t)p * N + l + LR * e] = v[i][e];
                }
                if (l == 0) y[p] = from_f32<T>(fmaf(skip, xv[i], s));
            }
        }
    }
}

template <typename T>
cudaError_t launch(const HeadStepArgs &a, cudaStream_t stream, int *launches)
{
    StepArgs<T> k{a.state, static_cast<const T *>(a.x), static_cast<const T *>(a.dt),
                  static_cast<const T *>(a.B), static_cast<const T *>(a.C), a.x_stride, a.dt_stride,
                  a.bc_stride, a.A, a.Dskip, a.dt_bias, a.delta_softplus, a.idx, a.n_slots,
                  static_cast<T *>(a.y), (int)a.H, (int)a.P, (int)a.G, (int)a.N};
    const bool vec = a.N % 4 == 0 && reinterpret_cast<uintptr_t>(a.state) % 16 == 0;
    const unsigned grid = (unsigned)(a.Bt * a.H);
#define SSM_STEP(LR)                                                                     \
    (vec ? head_step_kernel<T, LR, true><<<grid, 256, 0, stream>>>(k)                    \
         : head_step_kernel<T, LR, false><<<grid, 256, 0, stream>>>(k))
    if (a.N <= 16) SSM_STEP(4);
    else if (a.N <= 32) SSM_STEP(8);
    else if (a.N <= 64) SSM_STEP(16);
    else SSM_STEP(32);
#undef SSM_STEP
    ++*launches;
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_head_step(const HeadStepArgs &a, cudaStream_t stream, int *launches)
{
    if (a.Bt == 0) return cudaSuccess;
    return a.dtype == DType::BF16 ? launch<__nv_bfloat16>(a, stream, launches)
                                  : launch<float>(a, stream, launches);
}

}  // namespace ssm
