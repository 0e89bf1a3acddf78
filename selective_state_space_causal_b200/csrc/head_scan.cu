// head_scan.cu -- the scan with one decay per head in fp32, token by token, its backward,
// and the choice between these kernels and the tensor-core ones (bf16).
//
// head_recurrent_kernel walks a sequence with a 32-row tile of one head's state
// in registers (the forward, or the reverse walk of the state's gradient);
// head_bwd_chunk_kernel takes every chunk's start state and end gradient and
// gives the chunk's gradients in the matrix form
//   G = C B^T, L_ts = exp(c_t - c_s) (t >= s), M = G L d_s, dM = dy u^T,
//   du = M^T dy + d_s e^{cQ-c_s} dS B_s + D dy,
//   dC = sum_h (dM L d) B + e^{c_t} S0^T dy,  dB = sum_h (dM L d)^T C + d_s e^{cQ-c_s} dS^T u,
// with c the running sum of d_t A inside the chunk.
#include "head_mma.cuh"

namespace ssm {
namespace {

constexpr int kQ = 32;   // tokens per chunk
constexpr int kPT = 64;  // state rows at a time in the backward
constexpr int kBwdT = 512;

struct RecArgs {
    const float *x;  // u, or dy in the reverse walk
    const float *B, *C, *delta;
    int64_t x_stride, bc_stride, delta_stride;
    const float *A, *Dskip, *dt_bias;
    int softplus;
    const float *init;  // h0 or dh_final
    const int32_t *cu;
    int64_t S, tok;
    int H, P, G, N;
    float *y;       // forward output
    float *marks;   // state before each chunk in walking order, or nullptr
    float *final_;  // h_final or dh0, or nullptr
    bool vec;       // B and C in vectors of four
};

// Walks of a state: the forward with outputs, the backward's reverse walk of the state's
// gradient, and its forward walk, which only leaves the states before the chunks.
enum Walk { kOutputs, kReverse, kStates };

// LR lanes share a state row, each with NV float4 of its columns; a lane has RL rows: 32
// rows a CTA. With 64 rows (four lanes a row) too few warps hide a token's chain: 16384
// tokens of 24 heads of 64 x 128 in 8 sequences take 919 us (1295 with 64 rows), 17 tokens
// 10 us (15); with 880 tiles of 64 rows, enough of them, the two are within 6%. 16 rows a
// CTA load B and C too often (1244 us). Bound by the latency of a token: its loads from
// shared memory, its multiply-adds and the three steps of its sum.
template <int NV, int LR, int RL, Walk WALK>
__global__ void __launch_bounds__(128) head_recurrent_kernel(RecArgs a)
{
    constexpr bool REV = WALK == kReverse, OUT = WALK == kOutputs;
    constexpr int NP = NV * 4 * LR, RS = 128 / LR, kPT = RS * RL;  // rows a lane apart, rows of the CTA
    __shared__ __align__(16) float sB[kQ][NP], sC[kQ][NP];
    __shared__ float sx[kQ][kPT + 1], sa[kQ], sd[kQ];
    const int tid = threadIdx.x, j = tid % LR, pr = tid / LR;
    const int64_t s = blockIdx.y;
    const int np = (a.P + kPT - 1) / kPT;
    const int h = blockIdx.x / np, p0 = (blockIdx.x % np) * kPT;
    const int g = h / (a.H / a.G);
    const int rows = min(kPT, a.P - p0);
    int64_t lo, hi;
    seq_bounds(a.cu, a.S, a.tok, s, lo, hi);
    const int nchunk = (int)((hi - lo + kQ - 1) / kQ);
    const int64_t base = lo / kQ + s;
    const float Ah = a.A[h], bias = a.dt_bias ? a.dt_bias[h] : 0.0f;
    const float skip = a.Dskip ? a.Dskip[h] : 0.0f;
    const int64_t state_at = ((s * a.H + h) * a.P + p0) * (int64_t)a.N;

    f32x2 st[RL][NV * 2];
    auto four = [&](int r, int i, float (&v)[4]) {
        upk2(st[r][2 * i], v[0], v[1]);
        upk2(st[r][2 * i + 1], v[2], v[3]);
    };
#pragma unroll
    for (int r = 0; r < RL; ++r)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int p = pr + RS * r, n = 4 * (j + LR * i) + e;
                v[e] = (a.init && p < rows && n < a.N) ? a.init[state_at + (int64_t)p * a.N + n] : 0.0f;
            }
            st[r][2 * i] = pk2(v[0], v[1]);
            st[r][2 * i + 1] = pk2(v[2], v[3]);
        }

    for (int kk = 0; kk < nchunk; ++kk) {
        const int k = REV ? nchunk - 1 - kk : kk;
        const int64_t t0 = lo + (int64_t)k * kQ;
        const int len = (int)min((int64_t)kQ, hi - t0);
        if (a.marks) {
            float *m = a.marks + (((base + k) * a.H + h) * a.P + p0) * (int64_t)a.N;
#pragma unroll
            for (int r = 0; r < RL; ++r)
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int p = pr + RS * r, n = 4 * (j + LR * i);
                    float v[4];
                    four(r, i, v);
                    if (p >= rows) continue;
                    if (a.N % 4 == 0) {
                        if (n < a.N)
                            *reinterpret_cast<float4 *>(m + (int64_t)p * a.N + n) = make_float4(v[0], v[1], v[2], v[3]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (n + e < a.N) m[(int64_t)p * a.N + n + e] = v[e];
                    }
                }
        }
        __syncthreads();
        if (a.vec) {
#pragma unroll 4
            for (int i = tid; i < len * (NP / 4); i += 128) {
                const int t = i / (NP / 4), n = i % (NP / 4) * 4;
                const int64_t at = (t0 + t) * a.bc_stride + (int64_t)g * a.N + n;
                const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (!REV) *reinterpret_cast<float4 *>(&sB[t][n]) = n < a.N ? *reinterpret_cast<const float4 *>(a.B + at) : zero;
                if (REV || OUT) *reinterpret_cast<float4 *>(&sC[t][n]) = n < a.N ? *reinterpret_cast<const float4 *>(a.C + at) : zero;
            }
        }
        for (int i = tid; !a.vec && i < len * NP; i += 128) {
            const int t = i / NP, n = i % NP;
            const int64_t at = (t0 + t) * a.bc_stride + (int64_t)g * a.N + n;
            if (!REV) sB[t][n] = n < a.N ? a.B[at] : 0.0f;
            if (REV || OUT) sC[t][n] = n < a.N ? a.C[at] : 0.0f;
        }
#pragma unroll 4
        for (int i = tid; i < len * kPT; i += 128) {
            const int t = i / kPT, p = i % kPT;
            sx[t][p] = p < rows ? a.x[(t0 + t) * a.x_stride + (int64_t)h * a.P + p0 + p] : 0.0f;
        }
        if (tid < len) {
            const float d = head_step(a.delta[(t0 + tid) * a.delta_stride + h] + bias, a.softplus);
            const float lg = d * Ah;
            sd[tid] = d;
            sa[tid] = expf(lg < kHeadMinLog ? kHeadMinLog : lg);
        }
        __syncthreads();
#pragma unroll 2
        for (int tt = 0; tt < len; ++tt) {
            const int t = REV ? len - 1 - tt : tt;
            const float at = sa[t];
            float x[RL], y[RL];
            f32x2 w[RL], y2[RL];
            const f32x2 at2 = pk2(at, at);
#pragma unroll
            for (int r = 0; r < RL; ++r) {
                x[r] = sx[t][pr + RS * r];
                const float v = REV ? x[r] : sd[t] * x[r];
                w[r] = pk2(v, v);
                y2[r] = pk2(0.0f, 0.0f);
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float4 c, b;
                if (REV || OUT) c = *reinterpret_cast<const float4 *>(&sC[t][4 * (j + LR * i)]);
                if (!REV) b = *reinterpret_cast<const float4 *>(&sB[t][4 * (j + LR * i)]);
                if (REV) b = c;
                if (!OUT) c = b;
                const f32x2 cv[2] = {pk2(c.x, c.y), pk2(c.z, c.w)};
                const f32x2 bv[2] = {pk2(b.x, b.y), pk2(b.z, b.w)};
#pragma unroll
                for (int r = 0; r < RL; ++r)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        f32x2 &v = st[r][i * 2 + e];
                        if (REV) {
                            v = mul2(at2, fma2(w[r], bv[e], v));
                        } else {
                            v = fma2(at2, v, mul2(w[r], bv[e]));
                            if (OUT) y2[r] = fma2(v, cv[e], y2[r]);
                        }
                    }
            }
#pragma unroll
            for (int r = 0; r < RL; ++r) {
                float lo2, hi2;
                upk2(y2[r], lo2, hi2);
                y[r] = lo2 + hi2;
            }
            if (OUT) {
#pragma unroll
                for (int r = 0; r < RL; ++r) {
#pragma unroll
                    for (int o = 1; o < LR; o <<= 1) y[r] += __shfl_xor_sync(0xffffffffu, y[r], o);
                    // only this lane group reads row t of these columns
                    if (j == 0) sx[t][pr + RS * r] = fmaf(skip, x[r], y[r]);
                }
            }
        }
        if (OUT) {
            __syncthreads();
            for (int i = tid; i < len * kPT; i += 128) {
                const int t = i / kPT, p = i % kPT;
                if (p < rows)
                    a.y[((t0 + t) * a.H + h) * (int64_t)a.P + p0 + p] = sx[t][p];
            }
        }
    }
    if (a.final_) {
#pragma unroll
        for (int r = 0; r < RL; ++r)
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float v[4];
                four(r, i, v);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int p = pr + RS * r, n = 4 * (j + LR * i) + e;
                    if (p < rows && n < a.N) a.final_[state_at + (int64_t)p * a.N + n] = v[e];
                }
            }
    }
}

// out(i, j) = sum_k fa(i, k) fb(k, j) for i < M, j < N, by `count` threads from `first` on,
// 4 x 4 values each.
template <typename FA, typename FB, typename FO>
__device__ __forceinline__ void small_gemm(int first, int count, int M, int N, int K, FA fa, FB fb, FO out)
{
    const int mt = (M + 3) / 4, nt = (N + 3) / 4;
    const int me = (int)threadIdx.x - first;
    if (me < 0 || me >= count) return;
    for (int x = me; x < mt * nt; x += count) {
        const int i0 = x / nt * 4, j0 = x % nt;  // columns j0 + nt * r: neighbours in a warp are adjacent
        float acc[4][4] = {};
        int ir[4], jr[4];  // rows and columns that do not exist repeat the last one
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            ir[r] = min(i0 + r, M - 1);
            jr[r] = min(j0 + nt * r, N - 1);
        }
#pragma unroll 4
        for (int k = 0; k < K; ++k) {
            float av[4], bv[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) av[r] = fa(ir[r], k);
#pragma unroll
            for (int r = 0; r < 4; ++r) bv[r] = fb(k, jr[r]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[i][r] = fmaf(av[i], bv[r], acc[i][r]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (i0 + i < M && j0 + nt * r < N) out(i0 + i, j0 + nt * r, acc[i][r]);
    }
}

struct ChunkBwdArgs {
    const float *u, *B, *C, *delta, *dy;
    int64_t u_stride, bc_stride, delta_stride;
    const float *A, *Dskip, *dt_bias;
    int softplus;
    const int32_t *cu;
    int64_t S, tok;
    int H, P, G, N;
    const float *S0, *dS;  // per chunk: start state, gradient of the end state
    float *du, *ddelta, *dB, *dC;
    float *part;  // (slot, H, 3): this chunk's share of dA, ddt_bias, dDskip
};

// head_bwd_chunk_kernel has a chunk of one group and takes its heads in turn; products that
// do not wait for one another share the 512 threads. Its reads of shared memory bound it
// (eight for 16 multiply-adds): 3.1 ms for 16384 tokens of 24 heads of 64 x 128.
// Shared floats of it; row strides are odd so that walks down a
// column hit different banks.
int chunk_bwd_floats(int N)
{
    const int ns = N | 1;
    return 2 * kQ + 4 * kQ * ns + 2 * kPT * ns + 4 * kQ * (kPT + 1) + 3 * kQ * (kQ + 1) + 5 * kQ + 64;
}

__global__ void __launch_bounds__(kBwdT) head_bwd_chunk_kernel(ChunkBwdArgs a)
{
    extern __shared__ __align__(16) float smem[];
    const int tid = threadIdx.x, N = a.N, ns = N | 1, ps = kPT + 1, qs = kQ + 1;
    double *c = reinterpret_cast<double *>(smem);
    float *sB = smem + 2 * kQ, *sC = sB + kQ * ns, *sdB = sC + kQ * ns, *sdC = sdB + kQ * ns;
    float *S0 = sdC + kQ * ns, *dS = S0 + kPT * ns, *U = dS + kPT * ns, *Y = U + kQ * ps;
    float *V = Y + kQ * ps, *W = V + kQ * ps, *Gm = W + kQ * ps, *M = Gm + kQ * qs, *X = M + kQ * qs;
    float *d = X + kQ * qs, *raw = d + kQ, *row = raw + kQ, *col = row + kQ, *own = col + kQ;
    float *red = own + kQ;

    const int64_t slot = blockIdx.x;
    const int g = blockIdx.y, hpg = a.H / a.G;
    const ChunkRef ck = find_chunk(a.cu, a.S, a.tok, kQ, slot);
    const int len = ck.len;
    if (len == 0) {
        for (int i = tid; i < hpg * 3; i += kBwdT) a.part[(slot * a.H + g * hpg) * 3 + i] = 0.0f;
        return;
    }
    for (int i = tid; i < kQ * N; i += kBwdT) {
        const int t = i / N, n = i % N;
        const int64_t at = (ck.start + t) * a.bc_stride + (int64_t)g * N + n;
        sB[t * ns + n] = t < len ? a.B[at] : 0.0f;
        sC[t * ns + n] = t < len ? a.C[at] : 0.0f;
        sdB[t * ns + n] = 0.0f;
        sdC[t * ns + n] = 0.0f;
    }
    __syncthreads();
    small_gemm(0, kBwdT, kQ, kQ, N, [&](int t, int n) { return sC[t * ns + n]; },
               [&](int n, int s) { return sB[s * ns + n]; },
               [&](int t, int s, float v) { Gm[t * qs + s] = v; });

    for (int hh = 0; hh < hpg; ++hh) {
        const int h = g * hpg + hh;
        const float Ah = a.A[h], skip = a.Dskip ? a.Dskip[h] : 0.0f;
        __syncthreads();
        if (tid < 32) {
            const float bias = a.dt_bias ? a.dt_bias[h] : 0.0f;
            const float rw = tid < len ? (a.delta[(ck.start + tid) * a.delta_stride + h]) + bias : 0.0f;
            const float dt = tid < len ? head_step(rw, a.softplus) : 0.0f;
            float lg = dt * Ah;
            lg = lg < kHeadMinLog ? kHeadMinLog : lg;
            double run = tid < len ? (double)lg : 0.0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double v = __shfl_up_sync(0xffffffffu, run, o);
                if (tid >= o) run += v;
            }
            c[tid] = run;
            d[tid] = dt;
            raw[tid] = rw;
            row[tid] = 0.0f;
            col[tid] = 0.0f;
            own[tid] = 0.0f;
        }
        if (tid < 64) red[tid] = 0.0f;
        float dskip = 0.0f, dot_state = 0.0f;
        for (int p0 = 0; p0 < a.P; p0 += kPT) {
            const int rows = min(kPT, a.P - p0);
            __syncthreads();
#pragma unroll
            for (int i = tid; i < kQ * kPT; i += kBwdT) {
                const int t = i / kPT, p = i % kPT;
                const bool in = t < len && p < rows;
                const int64_t tk = ck.start + t;
                const float uv = in ? a.u[tk * a.u_stride + (int64_t)h * a.P + p0 + p] : 0.0f;
                const float yv = in ? a.dy[(tk * a.H + h) * a.P + p0 + p] : 0.0f;
                U[t * ps + p] = uv;
                Y[t * ps + p] = yv;
                dskip = fmaf(uv, yv, dskip);
            }
            const float eQ = expf((float)c[len - 1]);
            const int64_t sat = ((slot * a.H + h) * a.P + p0) * (int64_t)N;
#pragma unroll 8
            for (int i = tid; i < kPT * N; i += kBwdT) {
                const int p = i / N, n = i % N;
                const float s0 = p < rows ? a.S0[sat + i] : 0.0f, ds = p < rows ? a.dS[sat + i] : 0.0f;
                S0[p * ns + n] = s0;
                dS[p * ns + n] = ds;
                dot_state = fmaf(eQ * s0, ds, dot_state);
            }
            __syncthreads();
            // M and dM, V[s, p] = dS B_s (for du and J) and W[t, p] = S0 C_t (for I) at once
            small_gemm(0, 64, kQ, kQ, kPT, [&](int t, int p) { return Y[t * ps + p]; },
                       [&](int p, int s) { return U[s * ps + p]; },
                       [&](int t, int s, float v) {
                           const float L = t >= s ? expf((float)(c[t] - c[s])) : 0.0f;
                           M[t * qs + s] = Gm[t * qs + s] * L;   // without d_s
                           X[t * qs + s] = v * L;
                       });
            small_gemm(64, 128, kQ, kPT, N, [&](int s, int n) { return sB[s * ns + n]; },
                       [&](int n, int p) { return dS[p * ns + n]; },
                       [&](int s, int p, float v) { V[s * ps + p] = v; });
            small_gemm(192, 128, kQ, kPT, N, [&](int t, int n) { return sC[t * ns + n]; },
                       [&](int n, int p) { return S0[p * ns + n]; },
                       [&](int t, int p, float v) { W[t * ps + p] = v; });
            __syncthreads();
            if (tid < 32) {  // row and column sums of dM G L, the diagonal apart
                float r = 0.0f, k = 0.0f;
                for (int i = 0; i < kQ; ++i) {
                    if (i == tid) continue;
                    r = fmaf(X[tid * qs + i] * Gm[tid * qs + i], d[i], r);
                    k = fmaf(X[i * qs + tid], Gm[i * qs + tid], k);
                }
                float jv = 0.0f, iv = 0.0f;
                for (int p = 0; p < kPT; ++p) {
                    jv = fmaf(U[tid * ps + p], V[tid * ps + p], jv);
                    iv = fmaf(Y[tid * ps + p], W[tid * ps + p], iv);
                }
                jv *= expf((float)(c[len - 1] - c[tid]));
                row[tid] += r + iv * expf((float)c[tid]);
                col[tid] += k;
                own[tid] += X[tid * qs + tid] * Gm[tid * qs + tid] + (tid < len ? jv : 0.0f);
                red[tid] += tid < len ? d[tid] * jv : 0.0f;
            }
            small_gemm(32, 128, kQ, kPT, kQ, [&](int s, int t) { return M[t * qs + s]; },
                       [&](int t, int p) { return Y[t * ps + p]; },
                       [&](int s, int p, float v) {
                           if (s < len && p < rows) {
                               const float w = expf((float)(c[len - 1] - c[s]));
                               const float o = fmaf(d[s], v + w * V[s * ps + p], skip * Y[s * ps + p]);
                               a.du[((ck.start + s) * a.H + h) * (int64_t)a.P + p0 + p] = o;
                           }
                       });
            // both terms of an entry of dC, and of dB, are one thread's
            small_gemm(160, 176, kQ, N, kQ, [&](int t, int s) { return X[t * qs + s] * d[s]; },
                       [&](int s, int n) { return sB[s * ns + n]; },
                       [&](int t, int n, float v) { sdC[t * ns + n] += v; });
            small_gemm(160, 176, kQ, N, kPT, [&](int t, int p) { return Y[t * ps + p]; },
                       [&](int p, int n) { return S0[p * ns + n]; },
                       [&](int t, int n, float v) { sdC[t * ns + n] += expf((float)c[t]) * v; });
            small_gemm(336, 176, kQ, N, kQ, [&](int s, int t) { return X[t * qs + s] * d[s]; },
                       [&](int t, int n) { return sC[t * ns + n]; },
                       [&](int s, int n, float v) { sdB[s * ns + n] += v; });
            small_gemm(336, 176, kQ, N, kPT, [&](int s, int p) { return U[s * ps + p]; },
                       [&](int p, int n) { return dS[p * ns + n]; },
                       [&](int s, int n, float v) {
                           sdB[s * ns + n] += d[s] * expf((float)(c[len - 1] - c[s])) * v;
                       });
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            dskip += __shfl_xor_sync(0xffffffffu, dskip, o);
            dot_state += __shfl_xor_sync(0xffffffffu, dot_state, o);
        }
        __syncthreads();
        if ((tid & 31) == 0) {
            red[32 + tid / 32] = dskip;
            red[48 + tid / 32] = dot_state;
        }
        __syncthreads();
        if (tid < 32) {
            // gradient of log a_r, from what passes through token r: outputs at or after
            // it from inputs before it (W_ts, s < r <= t: a suffix sum of rows less
            // columns, without the diagonal, which would cancel only up to rounding), from
            // the start state (I), and the end state's share of inputs before it (J) and
            // of the start state
            double X = 0.0;
            float ds = 0.0f;
            for (int i = 0; i < kBwdT / 32; ++i) {
                X += red[48 + i];
                ds += red[32 + i];
            }
            double dg = tid < len ? (double)row[tid] - (double)d[tid] * col[tid] : 0.0;
            double before = red[tid];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double v = __shfl_down_sync(0xffffffffu, dg, o);
                const double w = __shfl_up_sync(0xffffffffu, before, o);
                if (tid + o < 32) dg += v;
                if (tid >= o) before += w;
            }
            before = __shfl_up_sync(0xffffffffu, before, 1);
            dg += X + (tid ? before : 0.0);
            float pa = 0.0f, pb = 0.0f;
            if (tid < len) {
                const float gv = (col[tid] + own[tid] + Ah * (float)dg) * head_step_grad(raw[tid], a.softplus);
                a.ddelta[(ck.start + tid) * a.H + h] = gv;
                pa = d[tid] * (float)dg;
                pb = gv;
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                pa += __shfl_xor_sync(0xffffffffu, pa, o);
                pb += __shfl_xor_sync(0xffffffffu, pb, o);
            }
            if (tid == 0) {
                float *q = a.part + (slot * a.H + h) * 3;
                q[0] = pa;
                q[1] = pb;
                q[2] = ds;
            }
        }
    }
    __syncthreads();
    for (int i = tid; i < len * N; i += kBwdT) {
        const int t = i / N, n = i % N;
        const int64_t at = ((ck.start + t) * a.G + g) * (int64_t)N + n;
        a.dB[at] = sdB[t * ns + n];
        a.dC[at] = sdC[t * ns + n];
    }
}

// One block per head: sums of the chunks' shares of dA, ddt_bias and dDskip, in a fixed order.
__global__ void __launch_bounds__(256) head_reduce_kernel(const float *part, int64_t slots, int H,
                                                          float *dA, float *dbias, float *dskip)
{
    __shared__ double sm[3][8];
    const int h = blockIdx.x;
    double v[3] = {0.0, 0.0, 0.0};
    for (int64_t s = threadIdx.x; s < slots; s += 256)
        for (int i = 0; i < 3; ++i) v[i] += part[(s * H + h) * 3 + i];
    for (int i = 0; i < 3; ++i) {
        for (int o = 16; o; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        if ((threadIdx.x & 31) == 0) sm[i][threadIdx.x / 32] = v[i];
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 0; i < 3; ++i)
            for (int w = 1; w < 8; ++w) sm[i][0] += sm[i][w];
        dA[h] = (float)sm[0][0];
        if (dbias) dbias[h] = (float)sm[1][0];
        if (dskip) dskip[h] = (float)sm[2][0];
    }
}

RecArgs rec_args(const HeadScanArgs &a, bool rev)
{
    RecArgs r;
    r.x = static_cast<const float *>(rev ? a.dy : a.u);
    r.x_stride = rev ? a.H * a.P : a.u_stride;
    r.B = static_cast<const float *>(a.B);
    r.C = static_cast<const float *>(a.C);
    r.delta = static_cast<const float *>(a.delta);
    r.bc_stride = a.bc_stride;
    r.delta_stride = a.delta_stride;
    r.A = a.A;
    r.Dskip = a.Dskip;
    r.dt_bias = a.dt_bias;
    r.softplus = a.delta_softplus;
    r.init = rev ? a.dh_final : a.h0;
    r.cu = a.cu;
    r.S = a.S;
    r.tok = a.tok;
    r.H = (int)a.H;
    r.P = (int)a.P;
    r.G = (int)a.G;
    r.N = (int)a.N;
    r.y = nullptr;
    r.marks = nullptr;
    r.final_ = nullptr;
    r.vec = a.N % 4 == 0 && a.bc_stride % 4 == 0 && reinterpret_cast<uintptr_t>(a.B) % 16 == 0 &&
            reinterpret_cast<uintptr_t>(a.C) % 16 == 0;
    return r;
}

template <int NV, int LR, int RL, Walk WALK>
void recurrent(const RecArgs &r, cudaStream_t stream)
{
    constexpr int rows = 128 / LR * RL;
    const dim3 grid((unsigned)(r.H * ((r.P + rows - 1) / rows)), (unsigned)r.S);
    head_recurrent_kernel<NV, LR, RL, WALK><<<grid, 128, 0, stream>>>(r);
}

template <Walk WALK>
cudaError_t launch_recurrent(const RecArgs &r, cudaStream_t stream, int *launches)
{
    if (r.N <= 16) recurrent<1, 4, 2, WALK>(r, stream);
    else if (r.N <= 32) recurrent<1, 8, 2, WALK>(r, stream);
    else if (r.N <= 64) recurrent<2, 8, 2, WALK>(r, stream);
    else recurrent<4, 8, 2, WALK>(r, stream);
    ++*launches;
    return cudaGetLastError();
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

cudaError_t fwd(const HeadScanArgs &a, cudaStream_t stream, int *launches)
{
    RecArgs r = rec_args(a, false);
    r.y = static_cast<float *>(a.y);
    r.final_ = a.h_final;
    return launch_recurrent<kOutputs>(r, stream, launches);
}

cudaError_t bwd(const HeadScanArgs &a, cudaStream_t stream, int *launches)
{
    const int64_t slots = head_slots(a.tok, a.S, kQ);
    const size_t state = align256((size_t)slots * a.H * a.P * a.N * 4);
    char *ws = static_cast<char *>(a.workspace);
    float *S0 = reinterpret_cast<float *>(ws), *dS = reinterpret_cast<float *>(ws + state);
    float *part = reinterpret_cast<float *>(ws + 2 * state);
    RecArgs r = rec_args(a, false);
    r.marks = S0;
    if (cudaError_t e = launch_recurrent<kStates>(r, stream, launches); e != cudaSuccess) return e;
    r = rec_args(a, true);
    r.marks = dS;
    r.final_ = a.dh0;
    if (cudaError_t e = launch_recurrent<kReverse>(r, stream, launches); e != cudaSuccess) return e;
    ChunkBwdArgs b;
    b.u = static_cast<const float *>(a.u);
    b.B = static_cast<const float *>(a.B);
    b.C = static_cast<const float *>(a.C);
    b.delta = static_cast<const float *>(a.delta);
    b.dy = static_cast<const float *>(a.dy);
    b.u_stride = a.u_stride;
    b.bc_stride = a.bc_stride;
    b.delta_stride = a.delta_stride;
    b.A = a.A;
    b.Dskip = a.Dskip;
    b.dt_bias = a.dt_bias;
    b.softplus = a.delta_softplus;
    b.cu = a.cu;
    b.S = a.S;
    b.tok = a.tok;
    b.H = (int)a.H;
    b.P = (int)a.P;
    b.G = (int)a.G;
    b.N = (int)a.N;
    b.S0 = S0;
    b.dS = dS;
    b.du = static_cast<float *>(a.du);
    b.ddelta = static_cast<float *>(a.ddelta);
    b.dB = static_cast<float *>(a.dB);
    b.dC = static_cast<float *>(a.dC);
    b.part = part;
    const int bytes = chunk_bwd_floats(b.N) * 4;
    if (cudaError_t e = cudaFuncSetAttribute(head_bwd_chunk_kernel,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        e != cudaSuccess)
        return e;
    head_bwd_chunk_kernel<<<dim3((unsigned)slots, (unsigned)a.G), kBwdT, bytes, stream>>>(b);
    ++*launches;
    if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
    return launch_head_reduce(part, slots, b.H, a.dA, a.ddt_bias, a.dDskip, stream, launches);
}

}  // namespace

cudaError_t launch_head_reduce(const float *part, int64_t slots, int H, float *dA, float *dbias,
                               float *dskip, cudaStream_t stream, int *launches)
{
    head_reduce_kernel<<<(unsigned)H, 256, 0, stream>>>(part, slots, H, dA, dbias, dskip);
    ++*launches;
    return cudaGetLastError();
}

size_t head_scan_workspace_bytes(int64_t tok, int64_t H, int64_t P, int64_t G, int64_t N, int64_t S,
                                 DType dtype)
{
    if (dtype != DType::BF16) return 0;
    HeadScanArgs a{};
    a.S = S; a.tok = tok; a.H = H; a.P = P; a.G = G; a.N = N;
    return hm::forward_bytes(hm::dims_of(a));
}

size_t head_scan_bwd_workspace_bytes(int64_t tok, int64_t H, int64_t P, int64_t G, int64_t N,
                                     int64_t S, DType dtype)
{
    if (dtype == DType::BF16) {
        HeadScanArgs a{};
        a.S = S; a.tok = tok; a.H = H; a.P = P; a.G = G; a.N = N;
        return hm::backward_bytes(hm::dims_of(a));
    }
    const int64_t slots = head_slots(tok, S, kQ);
    return 2 * align256((size_t)slots * H * P * N * 4) + align256((size_t)slots * H * 3 * 4);
}

cudaError_t launch_head_scan(const HeadScanArgs &a, cudaStream_t stream, int *launches)
{
    return a.dtype == DType::BF16 ? hm::launch_forward(a, stream, launches)
                                  : fwd(a, stream, launches);
}

cudaError_t launch_head_scan_bwd(const HeadScanArgs &a, cudaStream_t stream, int *launches)
{
    return a.dtype == DType::BF16 ? hm::launch_backward(a, stream, launches)
                                  : bwd(a, stream, launches);
}

}  // namespace ssm
