// norms.cu -- RMS norms around a mixer block, fused with the gate and the residual.
//
//   gated (after the block):  v = x silu(z), y = v rstd(v) w  per group of columns,
//                             or, with the norm before the gate, y = x rstd(x) w silu(z)
//   residual (before it):     r = residual + alpha x_scale x (as stored), y = r rstd(r) w
//
// Backward, with vh = v rstd, dh = dy w (times the gate when it comes after the norm):
//   dv = rstd (dh - vh mean(dh vh)),  dw = sum over rows of dy vh (times the gate).
//
// All four move each byte once: every input is read once and every output written
// once, because a team of threads (a warp for groups up to 64 vectors, a block sized to
// the row beyond) keeps its row in registers between the sums and the scaling. The
// backward keeps the row as it was loaded, computes from it twice, and loads the next
// row before it waits for this one's sums; the weights and their gradients' sums stay in
// registers over all rows of a block (weights read per row: 5% slower in the first line
// below). Rows that are not 16-byte aligned, or longer than the registers hold, go to
// kernels that read the row twice (the second time from cache).
//
// Measured on a B200, bf16, 16384 rows, of a copy's 6534 GB/s (the weight gradients' sum over
// partial rows takes 7 us more):
//   gate then norm, 5120 wide      forward 102 us (4.9 TB/s, 76%), backward 235 us (3.6 TB/s, 55%)
//   residual in fp32, 2560 wide    forward  81 us (6.2 TB/s, 95%), backward 152 us (5.0 TB/s, 76%, with
//                                  a learned scale)
// The forward with a gate and both backwards are held by what a row waits for: its loads,
// one sum over the block, its stores, with 20 warps an SM in flight (registers), and by
// the exponentials and reciprocals of the gate, taken twice an element in the backward.
#include "common.cuh"
#include "internal.h"

namespace ssm {
namespace {

constexpr int kParts = 1184;  // most partial rows of a weight gradient (8 per SM of 148)

struct Args {
    const void *x, *z, *residual, *dy, *xres, *dro;
    int64_t xs, zs;
    const float *w, *scale;
    float alpha, eps;
    void *y, *ro, *dx, *dz, *dres;
    float *part;
    int64_t tok;
    int D, group;
    bool has_dw, has_ds;
};

__device__ __forceinline__ float sigmoid_of(float z, float) { return 1.0f / (1.0f + expf(-z)); }
__device__ __forceinline__ float sigmoid_of(float z, __nv_bfloat16)
{
    return __fdividef(1.0f, 1.0f + __expf(-z));  // inf in the denominator gives 0
}

// Sums of a team's values in every thread of it: a warp, or (WARP false) the block. A
// block's calls take the two halves of sm in turn, so one barrier a call is enough.
template <bool WARP>
__device__ __forceinline__ float2 team_sum(float2 v, float2 (*sm)[32], int turn)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    if (WARP) return v;
    float2 *buf = sm[turn & 1];
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x / 32] = v;
    __syncthreads();
    v = make_float2(0.0f, 0.0f);
    for (int i = 0; i < (int)blockDim.x / 32; ++i) {
        v.x += buf[i].x;
        v.y += buf[i].y;
    }
    return v;
}

// V elements as 32-bit words, moved 16 (or 8) bytes at a time.
template <typename E, int V>
struct Raw {
    static constexpr int W = V * sizeof(E) / 4;
    uint32_t w[W];
    template <typename F>
    __device__ __forceinline__ void load(const E *p, F get)
    {
        if constexpr (W == 2) {
            const uint2 v = get(reinterpret_cast<const uint2 *>(p));
            w[0] = v.x; w[1] = v.y;
        } else {
#pragma unroll
            for (int i = 0; i < W / 4; ++i) {
                const uint4 v = get(reinterpret_cast<const uint4 *>(p) + i);
                w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
            }
        }
    }
    __device__ __forceinline__ void load(const E *p)
    {
        load(p, [](auto q) { return __ldcs(q); });  // read once
    }
    __device__ __forceinline__ float operator[](int i) const
    {
        if (sizeof(E) == 4) return __uint_as_float(w[i]);
        return __uint_as_float(i % 2 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    }
};

template <typename T, int V>
__device__ __forceinline__ void load_f(const T *p, float (&v)[V])
{
    Raw<T, V> r;
    r.load(p, [](auto q) { return __ldg(q); });
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = r[i];
}

// read-write data (a residual stream updated in place): no read-only cache
template <typename T, int V>
__device__ __forceinline__ void load_rw(const T *p, float (&v)[V])
{
    Raw<T, V> r;
    r.load(p, [](auto q) { return *q; });
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = r[i];
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <typename T, int V>
__device__ __forceinline__ void store_f(T *p, const float (&v)[V])
{
    constexpr int W = V * sizeof(T) / 4;
    uint32_t w[W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
        if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(v[i]);
        else w[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
    }
    if constexpr (W == 2) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int i = 0; i < W / 4; ++i)
            reinterpret_cast<uint4 *>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
}

// Elements per vector: 16 bytes of the widest tensor of a row. Beside an fp32 stream bf16
// goes 8 bytes at a time: two 16-byte halves of fp32 32 bytes apart cost twice the
// cache's time.
template <typename T, typename R> struct VecOf { static constexpr int v = sizeof(T) == 2 && sizeof(R) == 2 ? 8 : 4; };

// MODE 0: x only; 1: gate then norm; 2: norm then gate; 3: residual.
template <typename T, typename R, int MODE, bool WARP, int K>
__global__ void __launch_bounds__(WARP ? 256 : 512) norm_fwd_kernel(Args a)
{
    constexpr int V = VecOf<T, R>::v;
    __shared__ float2 sm[2][32];
    const int TEAM = WARP ? 32 : blockDim.x;
    const int l = WARP ? threadIdx.x % 32 : threadIdx.x;
    const int64_t row = WARP ? (int64_t)blockIdx.x * 8 + threadIdx.x / 32 : blockIdx.x;
    if (WARP && row >= a.tok) return;  // a block always has a row
    const int gs = a.group, c0 = blockIdx.y * gs;
    const T *x = static_cast<const T *>(a.x) + row * a.xs + c0;
    const T *z = MODE == 1 || MODE == 2 ? static_cast<const T *>(a.z) + row * a.zs + c0 : nullptr;
    const R *res = MODE == 3 && a.residual ? static_cast<const R *>(a.residual) + row * a.D : nullptr;
    R *ro = MODE == 3 && a.ro ? static_cast<R *>(a.ro) + row * a.D : nullptr;
    float v[K][V], gate[MODE == 2 ? K : 1][V], ss = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (l + TEAM * k) * V;
        if (c >= gs) {
#pragma unroll
            for (int i = 0; i < V; ++i) v[k][i] = 0.0f;
            continue;
        }
        load_f<T, V>(x + c, v[k]);
        if (MODE == 1 || MODE == 2) {
            float zv[V];
            load_f<T, V>(z + c, zv);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float gv = zv[i] * sigmoid_of(zv[i], T());
                if (MODE == 1) v[k][i] *= gv;
                else gate[k][i] = gv;
            }
        }
        if (MODE == 3) {
            float rv[V] = {}, sc[V];
            if (res) load_rw<R, V>(res + c, rv);
            if (a.scale) load_f<float, V>(a.scale + c, sc);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float s = a.scale ? a.alpha * sc[i] : a.alpha;
                // the norm is of the stream as it is stored, which the backward reads
                v[k][i] = to_f32(from_f32<R>(fmaf(s, v[k][i], rv[i])));
            }
            if (ro) store_f<R, V>(ro + c, v[k]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) ss = fmaf(v[k][i], v[k][i], ss);
    }
    const float rstd = 1.0f / sqrtf(team_sum<WARP>(make_float2(ss, 0.0f), sm, 0).x / (float)gs + a.eps);
    T *y = static_cast<T *>(a.y) + row * a.D + c0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (l + TEAM * k) * V;
        if (c >= gs) continue;
        float wv[V];
        if (a.w) load_f<float, V>(a.w + c0 + c, wv);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            v[k][i] *= rstd;
            if (a.w) v[k][i] *= wv[i];
            if (MODE == 2) v[k][i] *= gate[k][i];
        }
        store_f<T, V>(y + c, v[k]);
    }
}

// Teams walk rows with a stride; thread l keeps the weight-gradient sums of its columns.
template <typename T, typename R, int MODE, bool WARP, int K, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) norm_bwd_kernel(Args a)
{
    constexpr int V = VecOf<T, R>::v;
    __shared__ float2 sm[2][32];
    const int TEAM = WARP ? 32 : blockDim.x;
    const int l = WARP ? threadIdx.x % 32 : threadIdx.x;
    const int64_t team = WARP ? (int64_t)blockIdx.x * 8 + threadIdx.x / 32 : blockIdx.x;
    const int64_t teams = (int64_t)gridDim.x * (WARP ? 8 : 1);
    const int gs = a.group, c0 = blockIdx.y * gs;
    struct Row {
        Raw<T, V> x, dy;                     // x of MODE 3 only for its scale's gradient
        Raw<T, V> z;
        Raw<R, V> r, g;                      // MODE 3: the stream and its incoming gradient
    };
    Row cur[K];
    auto load = [&](int64_t row, int k, Row &to) {
        const int c = (l + TEAM * k) * V;
        if (row >= a.tok || c >= gs) return;
        const int64_t at = row * a.D + c0 + c;
        to.dy.load(static_cast<const T *>(a.dy) + at);
        if (MODE != 3 || a.has_ds) to.x.load(static_cast<const T *>(a.x) + row * a.xs + c0 + c);
        if (MODE == 1 || MODE == 2) to.z.load(static_cast<const T *>(a.z) + row * a.zs + c0 + c);
        if (MODE == 3) {
            to.r.load(static_cast<const R *>(a.xres) + at);
            if (a.dro) to.g.load(static_cast<const R *>(a.dro) + at);
        }
    };
    float dw[K][V] = {}, ds[MODE == 3 ? K : 1][V] = {};
#pragma unroll
    for (int k = 0; k < K; ++k) load(team, k, cur[k]);
    float weight[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (l + TEAM * k) * V;
#pragma unroll
        for (int i = 0; i < V; ++i) weight[k][i] = 1.0f;
        if (a.w && c < gs) load_f<float, V>(a.w + c0 + c, weight[k]);
    }
    int turn = 0;
    for (int64_t row = team; row < a.tok; row += teams, ++turn) {
        Row next[K];
#pragma unroll
        for (int k = 0; k < K; ++k) load(row + teams, k, next[k]);
        float ss = 0.0f, dot = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (l + TEAM * k) * V;
            if (c >= gs) continue;
            const float (&wv)[V] = weight[k];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float v = MODE == 3 ? cur[k].r[i] : cur[k].x[i], q = cur[k].dy[i];
                if (MODE == 1 || MODE == 2) {
                    const float zv = cur[k].z[i], gv = zv * sigmoid_of(zv, T());
                    if (MODE == 1) v *= gv;
                    else q *= gv;
                }
                ss = fmaf(v, v, ss);
                dot = fmaf(q * wv[i], v, dot);
            }
        }
        const float2 both = team_sum<WARP>(make_float2(ss, dot), sm, turn);
        const float rstd = 1.0f / sqrtf(both.x / (float)gs + a.eps);
        const float m = both.y * rstd * rstd / (float)gs;  // mean(dh vh) rstd, for vh = v rstd
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (l + TEAM * k) * V;
            if (c >= gs) continue;
            const int64_t at = row * a.D + c0 + c;
            float o1[V], o2[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float w = weight[k][i], yv = cur[k].dy[i];
                if (MODE == 0) {
                    const float v = cur[k].x[i];
                    dw[k][i] = fmaf(yv, v * rstd, dw[k][i]);
                    o1[i] = rstd * (yv * w - v * m);
                } else if (MODE == 3) {
                    const float v = cur[k].r[i];
                    dw[k][i] = fmaf(yv, v * rstd, dw[k][i]);
                    o1[i] = rstd * (yv * w - v * m) + (a.dro ? cur[k].g[i] : 0.0f);
                    if (a.has_ds) ds[k][i] = fmaf(a.alpha * o1[i], cur[k].x[i], ds[k][i]);
                } else {
                    const float xv = cur[k].x[i], zv = cur[k].z[i], sg = sigmoid_of(zv, T());
                    const float gv = zv * sg, dsilu = sg * fmaf(zv, 1.0f - sg, 1.0f);
                    const float v = MODE == 1 ? xv * gv : xv, q = MODE == 1 ? yv : yv * gv;
                    dw[k][i] = fmaf(q, v * rstd, dw[k][i]);
                    const float dv = rstd * (q * w - v * m);
                    o1[i] = MODE == 1 ? dv * gv : dv;
                    o2[i] = (MODE == 1 ? dv * xv : yv * (xv * rstd) * w) * dsilu;
                }
            }
            if (MODE == 3) {
                if (a.dres) store_f<R, V>(static_cast<R *>(a.dres) + at, o1);
                if (a.dx) {
                    float sc[V];
                    if (a.scale) load_f<float, V>(a.scale + c, sc);
#pragma unroll
                    for (int i = 0; i < V; ++i) o2[i] = o1[i] * (a.scale ? a.alpha * sc[i] : a.alpha);
                    store_f<T, V>(static_cast<T *>(a.dx) + at, o2);
                }
            } else {
                store_f<T, V>(static_cast<T *>(a.dx) + at, o1);
                if (MODE != 0 && a.dz) store_f<T, V>(static_cast<T *>(a.dz) + at, o2);
            }
            cur[k] = next[k];
        }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (l + TEAM * k) * V;
        if (c >= gs) continue;
        if (a.has_dw) store_f<float, V>(a.part + team * a.D + c0 + c, dw[k]);
        if (MODE == 3 && a.has_ds) store_f<float, V>(a.part + (teams + team) * a.D + c0 + c, ds[MODE == 3 ? k : 0]);
    }
}

// Any size and alignment: a block per row (and group), elements one by one, the row read twice.
template <typename T, typename R, int MODE>
__device__ __forceinline__ float normed(const Args &a, int64_t row, int c0, int c, float &gate)
{
    float v;
    gate = 1.0f;
    if (MODE == 3) {
        v = to_f32(static_cast<const R *>(a.xres)[row * a.D + c]);
    } else {
        v = to_f32(static_cast<const T *>(a.x)[row * a.xs + c0 + c]);
        if (MODE != 0) {
            const float zv = to_f32(static_cast<const T *>(a.z)[row * a.zs + c0 + c]);
            gate = zv * sigmoid_of(zv, T());
            if (MODE == 1) v *= gate;
        }
    }
    return v;
}

template <typename T, typename R, int MODE>
__global__ void __launch_bounds__(256) norm_fwd_any_kernel(Args a)
{
    __shared__ float2 sm[2][32];
    const int64_t row = blockIdx.x;
    const int gs = a.group, c0 = blockIdx.y * gs;
    const T *x = static_cast<const T *>(a.x) + row * a.xs + c0;
    const R *res = MODE == 3 && a.residual ? static_cast<const R *>(a.residual) + row * a.D : nullptr;
    R *ro = MODE == 3 && a.ro ? static_cast<R *>(a.ro) + row * a.D : nullptr;
    T *y = static_cast<T *>(a.y) + row * a.D + c0;
    // a stream updated in place is not read again after it was written
    auto stream = [&](int c) {
        if (res == ro && res && ro) return to_f32(ro[c]);
        const float s = a.scale ? a.alpha * a.scale[c] : a.alpha;
        return to_f32(from_f32<R>(fmaf(s, to_f32(x[c]), res ? to_f32(res[c]) : 0.0f)));
    };
    float ss = 0.0f, gate;
    for (int c = threadIdx.x; c < gs; c += 256) {
        float v;
        if (MODE == 3) {
            const float s = a.scale ? a.alpha * a.scale[c] : a.alpha;
            const R r = from_f32<R>(fmaf(s, to_f32(x[c]), res ? to_f32(res[c]) : 0.0f));
            if (ro) ro[c] = r;
            v = to_f32(r);
        } else {
            v = normed<T, R, MODE>(a, row, c0, c, gate);
        }
        ss = fmaf(v, v, ss);
    }
    const float rstd = 1.0f / sqrtf(team_sum<false>(make_float2(ss, 0.0f), sm, 0).x / (float)gs + a.eps);
    for (int c = threadIdx.x; c < gs; c += 256) {
        gate = 1.0f;
        float v = MODE == 3 ? stream(c) : normed<T, R, MODE>(a, row, c0, c, gate);
        v *= rstd;
        if (a.w) v *= a.w[c0 + c];
        if (MODE == 2) v *= gate;
        y[c] = from_f32<T>(v);
    }
}

// Thread c sums over its block's rows into the block's partial row in memory.
template <typename T, typename R, int MODE>
__global__ void __launch_bounds__(256) norm_bwd_any_kernel(Args a)
{
    __shared__ float2 sm[2][32];
    const int gs = a.group, c0 = blockIdx.y * gs;
    const int64_t team = blockIdx.x, teams = gridDim.x;
    float *pw = a.part + team * a.D + c0, *ps = a.part + (teams + team) * a.D + c0;
    for (int c = threadIdx.x; c < gs; c += 256) {
        if (a.has_dw) pw[c] = 0.0f;
        if (a.has_ds) ps[c] = 0.0f;
    }
    int turn = 0;
    for (int64_t row = team; row < a.tok; row += teams, ++turn) {
        const T *dyp = static_cast<const T *>(a.dy) + row * a.D + c0;
        float ss = 0.0f, dot = 0.0f, gate;
        for (int c = threadIdx.x; c < gs; c += 256) {
            const float v = normed<T, R, MODE>(a, row, c0, c, gate);
            float q = to_f32(dyp[c]) * (a.w ? a.w[c0 + c] : 1.0f);
            if (MODE == 2) q *= gate;
            ss = fmaf(v, v, ss);
            dot = fmaf(q, v, dot);
        }
        const float2 both = team_sum<false>(make_float2(ss, dot), sm, turn);
        const float rstd = 1.0f / sqrtf(both.x / (float)gs + a.eps);
        const float m = both.y * rstd * rstd / (float)gs;
        for (int c = threadIdx.x; c < gs; c += 256) {
            const float v = normed<T, R, MODE>(a, row, c0, c, gate);
            const float w = a.w ? a.w[c0 + c] : 1.0f, dyv = to_f32(dyp[c]);
            const float q = MODE == 2 ? dyv * gate : dyv;
            if (a.has_dw) pw[c] = fmaf(q, v * rstd, pw[c]);
            float dv = rstd * (q * w - v * m);
            const int64_t at = row * a.D + c0 + c;
            if (MODE == 3) {
                if (a.dro) dv += to_f32(static_cast<const R *>(a.dro)[at]);
                const float s = a.scale ? a.alpha * a.scale[c] : a.alpha;
                if (a.has_ds)
                    ps[c] = fmaf(a.alpha * dv, to_f32(static_cast<const T *>(a.x)[row * a.xs + c]), ps[c]);
                if (a.dres) static_cast<R *>(a.dres)[at] = from_f32<R>(dv);
                if (a.dx) static_cast<T *>(a.dx)[at] = from_f32<T>(s * dv);
            } else if (MODE == 0) {
                static_cast<T *>(a.dx)[at] = from_f32<T>(dv);
            } else {
                const float xv = to_f32(static_cast<const T *>(a.x)[row * a.xs + c0 + c]);
                const float zv = to_f32(static_cast<const T *>(a.z)[row * a.zs + c0 + c]);
                const float sg = sigmoid_of(zv, T());
                const float dsilu = sg * fmaf(zv, 1.0f - sg, 1.0f);
                static_cast<T *>(a.dx)[at] = from_f32<T>(MODE == 1 ? dv * (zv * sg) : dv);
                if (a.dz)
                    static_cast<T *>(a.dz)[at] =
                        from_f32<T>((MODE == 1 ? dv * xv : dyv * (xv * rstd) * w) * dsilu);
            }
        }
    }
}

// Sums over partial rows, in a fixed order: 32 columns by 32 strides of rows a block.
__global__ void __launch_bounds__(1024) norm_reduce_kernel(const float *part, int parts, int D, float *dw, float *ds)
{
    if (blockIdx.y) part += (int64_t)parts * D;  // the second plane is the scale's
    float *out = blockIdx.y ? ds : dw;
    if (!out) return;
    __shared__ double sm[32][32];
    const int lane = threadIdx.x % 32, c = blockIdx.x * 32 + lane, r0 = threadIdx.x / 32;
    double s = 0.0;
    if (c < D)
#pragma unroll 4
        for (int r = r0; r < parts; r += 32) s += part[(int64_t)r * D + c];
    sm[r0][lane] = s;
    __syncthreads();
    if (r0 == 0 && c < D) {
#pragma unroll 8
        for (int i = 1; i < 32; ++i) s += sm[i][lane];
        out[c] = (float)s;
    }
}

bool al16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Threads of a block that has K vectors of a row in each.
unsigned block_of(int nv, int K) { return (unsigned)(((nv + K - 1) / K + 31) / 32 * 32); }

template <typename T, typename R, int MODE>
cudaError_t fwd(const NormArgs &n, const Args &a, bool vec, cudaStream_t st)
{
    constexpr int V = VecOf<T, R>::v;
    const unsigned groups = (unsigned)(n.D / n.group);
    const int nv = (int)(n.group / V);
    const dim3 warps((unsigned)((n.tok + 7) / 8), groups), rows((unsigned)n.tok, groups);
    if (!vec || nv > 2048) norm_fwd_any_kernel<T, R, MODE><<<rows, 256, 0, st>>>(a);
    else if (nv <= 32) norm_fwd_kernel<T, R, MODE, true, 1><<<warps, 256, 0, st>>>(a);
    else if (nv <= 64) norm_fwd_kernel<T, R, MODE, true, 2><<<warps, 256, 0, st>>>(a);
    else if (nv <= 256) norm_fwd_kernel<T, R, MODE, false, 1><<<rows, block_of(nv, 1), 0, st>>>(a);
    else if (nv <= 1024) norm_fwd_kernel<T, R, MODE, false, 2><<<rows, block_of(nv, 2), 0, st>>>(a);
    else norm_fwd_kernel<T, R, MODE, false, 4><<<rows, block_of(nv, 4), 0, st>>>(a);
    return cudaGetLastError();
}

// Blocks of a kernel that fit the GPU at once: a backward block walks rows until none is
// left, so one more wave of blocks would run almost alone.
int resident(const void *kernel, int threads)
{
    int dev = 0, sms = 148, per = 1;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, 0) != cudaSuccess || per < 1) per = 1;
    return per * sms;
}

// What a block is, by the vectors of a row (or group). To 320 one a thread and three blocks an
// SM, to 640 two and two blocks, to 1024 two in a block of 512, then four. Backward of 16384 rows
// in us, the weights' sum with it, as chosen and with the next size of thread or block:
//   gated bf16     1024 wide 57 (two a thread, blocks to 320: 62; to 512: 55), 2560 133 (125; 125),
//                  4096 209 (one a thread, blocks to 512: 197; two, to 512: 182), 5120 240 (two, to
//                  512: 338), 6144 340 (four: 553), 8192 391 (594), 16384 1217
//   gated fp32     1024 86 (two, to 512: 94), 2048 188 (182), 4096 397 (465), 8192 958
//   fp32 stream    1024 68 (63; 66), 1280 92 (80; 88), 2048 133 (127), 2560 156 (238), 4096 281
//                  (440), 8192 942
// The steps at 640 and 1024 are worth a third; inside the first two ranges the neighbours are
// within 15%, to either side. Four vectors a thread run out of registers: 3.0 times the bytes'
// time where the others take 1.5 to 2.2.
// With a warp a row (to 64 vectors) each warp has a partial row, so kParts allows one block of
// eight warps an SM: 131072 rows of 512 182 us (bytes 103), of 256 105 (51). A group of 64
// columns has work for 8 of a warp's 32 lanes: 16384 x 5120 in groups of 64 821 us (bytes 128).
template <typename T, typename R, int MODE>
cudaError_t bwd(const NormArgs &n, const Args &a, bool vec, cudaStream_t st, int *parts)
{
    constexpr int V = VecOf<T, R>::v;
    const int64_t groups = n.D / n.group;
    const int nv = (int)(n.group / V);
    const bool warp = vec && nv <= 64;
    void (*kernel)(Args);
    int threads = 256;
    if (!vec || nv > 2048) {
        kernel = norm_bwd_any_kernel<T, R, MODE>;
    } else if (nv <= 32) {
        kernel = norm_bwd_kernel<T, R, MODE, true, 1, 256, 2>;
    } else if (nv <= 64) {
        kernel = norm_bwd_kernel<T, R, MODE, true, 2, 256, 2>;
    } else if (nv <= 320) {
        kernel = norm_bwd_kernel<T, R, MODE, false, 1, 320, 3>;
        threads = (int)block_of(nv, 1);
    } else if (nv <= 640) {
        kernel = norm_bwd_kernel<T, R, MODE, false, 2, 320, 2>;
        threads = (int)block_of(nv, 2);
    } else if (nv <= 1024) {
        kernel = norm_bwd_kernel<T, R, MODE, false, 2, 512, 1>;
        threads = (int)block_of(nv, 2);
    } else {
        kernel = norm_bwd_kernel<T, R, MODE, false, 4, 512, 1>;
        threads = (int)block_of(nv, 4);
    }
    // at most one wave of blocks over all groups, and no more partial rows than the workspace has
    int64_t blocks = warp ? (n.tok + 7) / 8 : n.tok, most = resident((const void *)kernel, threads) / groups;
    if (most > kParts / (warp ? 8 : 1)) most = kParts / (warp ? 8 : 1);
    if (most < 1) most = 1;
    if (blocks > most) blocks = most;
    *parts = (int)(warp ? blocks * 8 : blocks);
    kernel<<<dim3((unsigned)blocks, (unsigned)groups), threads, 0, st>>>(a);
    return cudaGetLastError();
}

Args common(const NormArgs &n)
{
    Args a;
    a.x = n.x; a.z = n.z; a.residual = n.residual;
    a.dy = n.dy; a.xres = n.x_res; a.dro = n.dres_out;
    a.xs = n.x_stride; a.zs = n.z_stride;
    a.w = n.weight; a.scale = n.x_scale;
    a.alpha = n.alpha; a.eps = n.eps;
    a.y = n.y; a.ro = n.residual_out; a.dx = n.dx; a.dz = n.dz; a.dres = n.dres;
    a.part = n.partials;
    a.tok = n.tok; a.D = (int)n.D; a.group = (int)n.group;
    a.has_dw = n.dweight != nullptr;
    a.has_ds = n.dscale != nullptr;
    return a;
}

// Every pointer 16-byte aligned, strides and the group multiples of a vector.
bool vectors(const NormArgs &n, int V)
{
    const void *ps[] = {n.x, n.z, n.residual, n.weight, n.x_scale, n.y, n.residual_out,
                        n.dy, n.x_res, n.dres_out, n.dx, n.dz, n.dres};
    for (const void *p : ps)
        if (!al16(p)) return false;
    return n.group % V == 0 && n.x_stride % V == 0 && (!n.z || n.z_stride % V == 0);
}

template <typename F>
cudaError_t by_type(const NormArgs &n, F f)
{
    using bf = __nv_bfloat16;
    const bool b = n.dtype == DType::BF16, rb = n.res_dtype == DType::BF16;
    if (n.gated) return b ? f(bf(), bf()) : f(float(), float());
    if (b) return rb ? f(bf(), bf()) : f(bf(), float());
    return f(float(), float());
}

}  // namespace

size_t norm_bwd_workspace_bytes(int64_t tok, int64_t D)
{
    (void)tok;
    return (size_t)2 * kParts * D * sizeof(float);
}

cudaError_t launch_norm_fwd(const NormArgs &n, cudaStream_t st, int *launches)
{
    if (n.tok == 0) return cudaSuccess;
    const Args a = common(n);
    ++*launches;
    return by_type(n, [&](auto t, auto r) {
        using T = decltype(t);
        using R = decltype(r);
        const bool vec = vectors(n, VecOf<T, R>::v);
        if (!n.gated) return fwd<T, R, 3>(n, a, vec, st);
        if (!n.z) return fwd<T, R, 0>(n, a, vec, st);
        return n.norm_before_gate ? fwd<T, R, 2>(n, a, vec, st) : fwd<T, R, 1>(n, a, vec, st);
    });
}

cudaError_t launch_norm_bwd(const NormArgs &n, cudaStream_t st, int *launches)
{
    const Args a = common(n);
    int parts = 0;
    if (n.tok > 0) {
        ++*launches;
        const cudaError_t e = by_type(n, [&](auto t, auto r) {
            using T = decltype(t);
            using R = decltype(r);
            const bool vec = vectors(n, VecOf<T, R>::v);
            if (!n.gated) return bwd<T, R, 3>(n, a, vec, st, &parts);
            if (!n.z) return bwd<T, R, 0>(n, a, vec, st, &parts);
            return n.norm_before_gate ? bwd<T, R, 2>(n, a, vec, st, &parts)
                                      : bwd<T, R, 1>(n, a, vec, st, &parts);
        });
        if (e != cudaSuccess) return e;
    }
    const unsigned blocks = (unsigned)((n.D + 31) / 32);
    if (!n.dweight && !n.dscale) return cudaSuccess;
    norm_reduce_kernel<<<dim3(blocks, n.dscale ? 2 : 1), 1024, 0, st>>>(n.partials, parts, (int)n.D,
                                                                       n.dweight, n.dscale);
    ++*launches;
    return cudaGetLastError();
}

}  // namespace ssm
