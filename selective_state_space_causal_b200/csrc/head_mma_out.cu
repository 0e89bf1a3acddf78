// head_mma_out.cu -- outputs of the bf16 scan with one decay per head (tensor cores).
//
// One CTA has a chunk (128 tokens) of one group and some of its panels. It makes
// G = C B^T once (it stays in tensor memory), and for every panel
//   y = M u + e^{c_t} (C S0^T) + D u,   M_ts = G_ts e^{c_t - c_s} d_s  (t >= s).
// Two warpgroups take panels in turn, each with its own buffers, so one's matrix
// instructions run beside the other's arithmetic; the next panel's u and S0 are
// loaded meanwhile. M is rounded to bf16 once, goes to tensor memory and is the left
// operand from there.
//
// e^{c_t - c_s} needs no exponential per pair below the diagonal blocks: for t in the
// 32-token block i and s in an earlier one it is e^{c_t - r_i} e^{r_i - c_s}, r_i the
// running sum before block i, and both factors are at most one. Inside a diagonal
// block the exponent is a difference of two 32-bit pairs.
#include "head_mma.cuh"

namespace ssm {
namespace hm {

__device__ int g_out_status;

namespace {

struct OutArgs {
    Dims z;
    const bf16 *u, *B, *C;
    int64_t u_stride, bc_stride;
    const float *Dskip;
    const double *c;
    const float *d;
    const bf16 *marks;
    bf16 *y;
    int per;  // panels of a CTA
    bool u_vec, bc_vec, y_vec;
};

struct WgTables {
    double c[kC];
    float col[3][kC];  // d_s e^{r_i - c_s}, i = 1..3, s < 32 i
    float d[kC];
    float hi[kC], lo[kC];  // c_s - r_{block of s}
};

template <int NPAD>
constexpr int out_smem()
{
    return 1024 + 2 * (NPAD / 64) * umma::kPanel + 4 * (umma::kPanel + 64 * NPAD * 2) + 2 * (int)sizeof(WgTables);
}

template <int NPAD>
__global__ void __launch_bounds__(256) head_out_kernel(OutArgs a)
{
    constexpr int BP = NPAD / 64;
    constexpr uint32_t S0P = 64 * 128;                          // bytes of a 64-row panel
    constexpr uint32_t STAGE = umma::kPanel + BP * S0P;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t gbar, wbar[2];
    __shared__ uint32_t tmem_slot;
    const Dims &z = a.z;
    const int tid = threadIdx.x, warp = tid / 32, wg = tid / 128, t = tid % 128;
    const int64_t slot = blockIdx.x;
    const int nb = (z.npan + a.per - 1) / a.per;
    const int g = blockIdx.y / nb, pb = blockIdx.y % nb * a.per, pe = min(pb + a.per, z.npan);
    const ChunkRef ck = find_chunk(z.cu, z.S, z.tok, kC, slot);
    if (ck.len == 0) return;
    const int len = ck.len;

    const uint32_t base = (saddr(raw) + 1023) & ~1023u;
    const uint32_t sC = base, sB = sC + BP * umma::kPanel;
    const uint32_t sW = sB + BP * umma::kPanel + wg * 2 * STAGE;  // this warpgroup's two stages
    WgTables &tb = *reinterpret_cast<WgTables *>(
        raw + (sB + BP * umma::kPanel + 4 * STAGE - saddr(raw)) + wg * sizeof(WgTables));
    if (tid == 0) {
        mbar_init(&gbar);
        mbar_init(&wbar[0]);
        mbar_init(&wbar[1]);
    }
    if (warp == 0) umma::alloc(&tmem_slot, 512);

    load_tile<NPAD, 256>(sC, a.C + ck.start * a.bc_stride + (int64_t)g * z.N, a.bc_stride, len, z.N, a.bc_vec, tid);
    load_tile<NPAD, 256>(sB, a.B + ck.start * a.bc_stride + (int64_t)g * z.N, a.bc_stride, len, z.N, a.bc_vec, tid);
    umma::cp_commit();
    double cr = 0.0;
    float dr = 0.0f;
    auto load = [&](int pi, int stage) {  // u and S0 of a panel; its tables into registers
        const PanelRef p = panel_of(z, g, pi);
        const uint32_t at = sW + stage * STAGE;
        load_tile<64, 128>(at, a.u + ck.start * a.u_stride + (int64_t)p.h * z.P + p.p0, a.u_stride, len,
                           p.rows, a.u_vec, t);
        const bf16 *m = a.marks + (slot * z.G * z.npan + g * z.npan + pi) * kMark<NPAD>;
#pragma unroll
        for (int i = 0; i < 64 * NPAD / 8 / 128; ++i) {
            const int x = t + 128 * i, r = x % 64, c = x / 64;  // state row, piece of its columns
            umma::cp16(at + umma::kPanel + (c / 8) * S0P + umma::piece(r, c % 8), m + (int64_t)x * 8, true);
        }
        umma::cp_commit();
        const int64_t k = (slot * z.H + p.h) * kC + t;
        cr = a.c[k];
        dr = a.d[k];
    };
    const int p0 = pb + wg;
    if (p0 < pe) load(p0, 0);
    else umma::cp_commit();
    umma::cp_wait<1>();
    fence_proxy_async();
    umma::fence_before();
    __syncthreads();
    umma::fence_after();
    const uint32_t tm = tmem_slot;
    const uint32_t tM = tm + 128 + wg * 192, tYa = tM + 64, tYb = tM + 128;
    if (tid == 0) {
#pragma unroll
        for (int k = 0; k < NPAD / 16; ++k)
            umma::mma(tm, umma::desc_k(sC + (k / 4) * umma::kPanel, k % 4),
                      umma::desc_k(sB + (k / 4) * umma::kPanel, k % 4), umma::idesc(128, false, false), k > 0);
        umma::commit(&gbar);
    }
    __syncwarp();
    const int wi = warp & 3;  // this warp's 32-token block of rows
    {  // the blocks above the diagonal stay zero for every panel
        uint32_t zero[16] = {};
        for (int j = wi + 1; j < 4; ++j) umma::st16(umma::lanes(tM, warp) + 16 * j, zero);
        umma::wait_st();
    }
    bool failed = false;
    mbar_wait(&gbar, 0, failed, &g_out_status, 1);
    umma::fence_after();

    int it = 0;
    for (int pi = p0; pi < pe; pi += 2, ++it) {
        const PanelRef p = panel_of(z, g, pi);
        const uint32_t su = sW + (it & 1) * STAGE, ss = su + umma::kPanel;
        const double cm = cr;
        const float dm = dr;
        tb.c[t] = cm;
        tb.d[t] = dm;
        if (pi + 2 < pe) {
            load(pi + 2, (it + 1) & 1);
            umma::cp_wait<1>();
        } else {
            umma::cp_wait<0>();
        }
        fence_proxy_async();
        umma::fence_before();
        bar_sync(1 + wg, 128);
        umma::fence_after();
        if (t == 0) {
#pragma unroll
            for (int k = 0; k < NPAD / 16; ++k)
                umma::mma(tYb, umma::desc_k(sC + (k / 4) * umma::kPanel, k % 4),
                          umma::desc_k(ss + (k / 4) * S0P, k % 4), umma::idesc(64, false, false), k > 0);
        }
        __syncwarp();
        const double r1 = tb.c[31], r2 = tb.c[63], r3 = tb.c[95];
        const double ri = wi == 0 ? 0.0 : wi == 1 ? r1 : wi == 2 ? r2 : r3;
        if (wi < 1) tb.col[0][t] = dm * ex2_approx((float)(r1 - cm));
        if (wi < 2) tb.col[1][t] = dm * ex2_approx((float)(r2 - cm));
        if (wi < 3) tb.col[2][t] = dm * ex2_approx((float)(r3 - cm));
        const float hi = (float)(cm - ri), lo = (float)((cm - ri) - (double)hi);
        tb.hi[t] = hi;
        tb.lo[t] = lo;
        bar_sync(1 + wg, 128);
        const float rowf = ex2_approx(hi);
        for (int j = 0; j < wi; ++j) {
            uint32_t v[32], w[16];
            umma::ld32(umma::lanes(tm, warp) + 32 * j, v);
            const float4 *cf = reinterpret_cast<const float4 *>(&tb.col[wi - 1][32 * j]);
            umma::wait_ld();
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const float4 f = cf[q];
                w[2 * q] = umma::pack(__uint_as_float(v[4 * q]) * (f.x * rowf),
                                      __uint_as_float(v[4 * q + 1]) * (f.y * rowf));
                w[2 * q + 1] = umma::pack(__uint_as_float(v[4 * q + 2]) * (f.z * rowf),
                                          __uint_as_float(v[4 * q + 3]) * (f.w * rowf));
            }
            umma::st16(umma::lanes(tM, warp) + 16 * j, w);
        }
        {
            uint32_t v[32], w[16];
            umma::ld32(umma::lanes(tm, warp) + 32 * wi, v);
            umma::wait_ld();
            const int own = t & 31;
#pragma unroll
            for (int s = 0; s < 32; s += 2) {
                float m[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int sg = 32 * wi + s + e;
                    const float x = (hi - tb.hi[sg]) + (lo - tb.lo[sg]);
                    m[e] = s + e <= own ? __uint_as_float(v[s + e]) * (ex2_approx(x) * tb.d[sg]) : 0.0f;
                }
                w[s / 2] = umma::pack(m[0], m[1]);
            }
            umma::st16(umma::lanes(tM, warp) + 16 * wi, w);
        }
        umma::wait_st();
        umma::fence_before();
        bar_sync(1 + wg, 128);
        if (t == 0) {
            umma::fence_after();
#pragma unroll
            for (int k = 0; k < 8; ++k)
                umma::mma_ta(tYa, tM + 8 * k, umma::desc_mn(su, k, 0), umma::idesc(64, false, true), k > 0);
            umma::commit(&wbar[wg]);
        }
        __syncwarp();
        mbar_wait(&wbar[wg], it & 1, failed, &g_out_status, 1);
        umma::fence_after();
        const float ec = ex2_approx((float)cm), skip = a.Dskip ? a.Dskip[p.h] : 0.0f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t va[32], vb[32];
            umma::ld32(umma::lanes(tYa, warp) + 32 * j, va);
            umma::ld32(umma::lanes(tYb, warp) + 32 * j, vb);
            umma::wait_ld();
#pragma unroll
            for (int q = 0; q < 4; ++q) {  // y takes u's place in shared memory
                const uint32_t at = su + umma::piece(t, 4 * j + q);
                const uint4 uv = lds16(at);
                const uint32_t in[4] = {uv.x, uv.y, uv.z, uv.w};
                uint32_t out[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int x = 8 * q + 2 * i;
                    const float y0 = fmaf(ec, __uint_as_float(vb[x]), __uint_as_float(va[x]));
                    const float y1 = fmaf(ec, __uint_as_float(vb[x + 1]), __uint_as_float(va[x + 1]));
                    out[i] = umma::pack(fmaf(skip, umma::lo_f(in[i]), y0), fmaf(skip, umma::hi_f(in[i]), y1));
                }
                sts16(at, make_uint4(out[0], out[1], out[2], out[3]));
            }
        }
        umma::fence_before();
        bar_sync(1 + wg, 128);
        bf16 *yo = a.y + (ck.start * z.H + p.h) * (int64_t)z.P + p.p0;
        const int64_t ys = (int64_t)z.H * z.P;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = 16 * i + t / 8, c = t % 8, n = min(8, p.rows - 8 * c);
            if (r >= len || n <= 0) continue;
            const uint4 v = lds16(su + umma::piece(r, c));
            if (a.y_vec) {
                *reinterpret_cast<uint4 *>(yo + r * ys + 8 * c) = v;
            } else {
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < n)
                        reinterpret_cast<unsigned short *>(yo + r * ys + 8 * c)[e] =
                            (unsigned short)(w[e / 2] >> (16 * (e & 1)));
            }
        }
        bar_sync(1 + wg, 128);  // the stage and the tables are free
    }
    umma::fence_before();
    __syncthreads();
    if (warp == 0) umma::dealloc(tm, 512);
}

template <int NPAD>
cudaError_t out(const OutArgs &a, int64_t slots, cudaStream_t st)
{
    constexpr int bytes = out_smem<NPAD>();
    if (cudaError_t e = cudaFuncSetAttribute(head_out_kernel<NPAD>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        e != cudaSuccess)
        return e;
    const dim3 grid((unsigned)slots, (unsigned)(a.z.G * ((a.z.npan + a.per - 1) / a.per)));
    head_out_kernel<NPAD><<<grid, 256, bytes, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

// Workspace of the forward: tables, segment states, marks.
Layout forward_layout(const Dims &z, int planes, int64_t span, bool split)
{
    const int64_t slots = head_slots(z.tok, z.S, kC), segs = split ? head_slots(z.tok, z.S, span) : 0;
    const int npad = z.N > 64 ? 128 : 64;
    const size_t panel = (size_t)z.G * z.npan * 64 * npad;
    Layout l;
    l.c = 0;
    l.d = l.c + up256((size_t)slots * z.H * kC * 8);
    l.seg = l.d + up256((size_t)slots * z.H * kC * 4);
    l.segdec = l.seg + up256((size_t)segs * panel * 4);
    l.marks = l.segdec + up256((size_t)segs * z.H * 8);
    l.total = l.marks + up256((size_t)slots * panel * 2 * planes);
    return l;
}

cudaError_t launch_forward(const HeadScanArgs &a, cudaStream_t st, int *launches)
{
    const Dims z = dims_of(a);
    bool split;
    const int64_t span = segment_span(z, &split);
    const Layout l = forward_layout(z, 1, span, split);
    char *ws = static_cast<char *>(a.workspace);
    double *c = reinterpret_cast<double *>(ws + l.c);
    float *d = reinterpret_cast<float *>(ws + l.d);
    bf16 *marks = reinterpret_cast<bf16 *>(ws + l.marks);
    if (cudaError_t e = launch_tables(a, z, c, d, st, launches); e != cudaSuccess) return e;
    const bool bc_vec = vec16(a.B, a.bc_stride, a.N) && vec16(a.C, a.bc_stride, a.N);
    const bool u_vec = vec16(a.u, a.u_stride, a.P);
    StateArgs s{z, static_cast<const bf16 *>(a.u), a.u_stride, static_cast<const bf16 *>(a.B), a.bc_stride,
                c, d, a.h0, a.h_final, marks, span, reinterpret_cast<float *>(ws + l.seg),
                reinterpret_cast<double *>(ws + l.segdec), u_vec, bc_vec};
    if (cudaError_t e = launch_states(s, false, 1, split, st, launches); e != cudaSuccess) return e;
    if (a.tok == 0) return cudaSuccess;
    const int64_t slots = head_slots(z.tok, z.S, kC);
    // G is made once per CTA: as many panels a CTA as leave about four CTAs an SM
    int64_t per = slots * z.G * z.npan / (148 * 4);
    per = per < 2 ? 2 : per > 24 ? 24 : per;
    if (per > z.npan) per = z.npan;
    OutArgs o{z, static_cast<const bf16 *>(a.u), static_cast<const bf16 *>(a.B), static_cast<const bf16 *>(a.C),
              a.u_stride, a.bc_stride, a.Dskip, c, d, marks, static_cast<bf16 *>(a.y), (int)per, u_vec, bc_vec,
              vec16(a.y, a.P, a.P)};
    ++*launches;
    return z.N > 64 ? out<128>(o, slots, st) : out<64>(o, slots, st);
}

size_t forward_bytes(const Dims &z)
{
    bool split;
    const int64_t span = segment_span(z, &split);
    return forward_layout(z, 1, span, split).total;
}

}  // namespace hm

int read_head_out_status(bool clear)
{
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, hm::g_out_status, sizeof(v)) != cudaSuccess) return -1;
    if (clear && v) {
        const int zero = 0;
        if (cudaMemcpyToSymbol(hm::g_out_status, &zero, sizeof(zero)) != cudaSuccess) return -1;
    }
    return v;
}

}  // namespace ssm
