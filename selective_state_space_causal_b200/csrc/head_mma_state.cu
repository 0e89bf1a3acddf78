// head_mma_state.cu -- chunk tables and chunk states of the bf16 scan with one decay
// per head (tensor cores).
//
// State of a chunk's end from its start:  S' = e^{cQ} S + sum_t w_t x_t b_t^T, with
//   forward  x = u, b = B, w_t = d_t e^{cQ - c_t};   reverse  x = dy, b = C, w_t = e^{c_t}.
// The sum over a chunk is one 128 x N x 128 product for two panels: D[p, n], A = (w x)^T
// with rows p (both panels), B = b. w x is split into three bf16 planes (24 bits), so the
// state keeps fp32 accuracy; b is bf16 as given. The products of different chunks are
// independent: only S' = e S + delta runs chunk after chunk, in registers, while the
// next product is under way.
#include "head_mma.cuh"

namespace ssm {
namespace hm {

__device__ int g_status;

namespace {

// One block per (chunk slot, 32 heads).
__global__ void __launch_bounds__(256) head_table_kernel(Dims z, const bf16 *delta, int64_t stride,
                                                         const float *A, const float *bias,
                                                         int softplus, double *c, float *d)
{
    __shared__ float sd[kC][33];
    const int64_t slot = blockIdx.x;
    const int h0 = blockIdx.y * 32, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const ChunkRef ck = find_chunk(z.cu, z.S, z.tok, kC, slot);
    if (ck.len == 0) return;
    const int h = h0 + lane;
    const float bs = bias && h < z.H ? bias[h] : 0.0f;
#pragma unroll
    for (int t = warp; t < kC; t += 8) {
        float v = 0.0f;
        if (t < ck.len && h < z.H) v = head_step(to_f32(delta[(ck.start + t) * stride + h]) + bs, softplus);
        sd[t][lane] = v;
    }
    __syncthreads();
    for (int i = warp; i < 32 && h0 + i < z.H; i += 8) {
        const float Ah = A[h0 + i];
        double run[4], sum = 0.0;
        float dv[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int t = 4 * lane + j;
            dv[j] = sd[t][i];
            float g = dv[j] * Ah;
            g = g < kHeadMinLog ? kHeadMinLog : g;
            sum += t < ck.len ? (double)g * kLog2eD : 0.0;
            run[j] = sum;
        }
        double pre = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double v = __shfl_up_sync(0xffffffffu, pre, o);
            if (lane >= o) pre += v;
        }
        pre -= sum;
        const int64_t at = (slot * z.H + h0 + i) * kC + 4 * lane;
#pragma unroll
        for (int j = 0; j < 4; ++j) run[j] += pre;
        *reinterpret_cast<double2 *>(c + at) = make_double2(run[0], run[1]);
        *reinterpret_cast<double2 *>(c + at + 2) = make_double2(run[2], run[3]);
        *reinterpret_cast<float4 *>(d + at) = make_float4(dv[0], dv[1], dv[2], dv[3]);
    }
}

// Splits 8 bf16 times w into three planes: the sum of the planes is w x to 24 bits.
__device__ __forceinline__ void split3(uint4 x, float w, uint4 &hi, uint4 &mid, uint4 &lo)
{
    const uint32_t in[4] = {x.x, x.y, x.z, x.w};
    uint32_t a[4], b[4], c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float v0 = w * umma::lo_f(in[i]), v1 = w * umma::hi_f(in[i]);
        a[i] = umma::pack(v0, v1);
        const float r0 = v0 - umma::lo_f(a[i]), r1 = v1 - umma::hi_f(a[i]);
        b[i] = umma::pack(r0, r1);
        c[i] = umma::pack(r0 - umma::lo_f(b[i]), r1 - umma::hi_f(b[i]));
    }
    hi = make_uint4(a[0], a[1], a[2], a[3]);
    mid = make_uint4(b[0], b[1], b[2], b[3]);
    lo = make_uint4(c[0], c[1], c[2], c[3]);
}

template <int NPAD>
constexpr int state_smem()
{
    return 1024 + 6 * umma::kPanel + 2 * (NPAD / 64) * umma::kPanel + 2 * 2 * kC * 4 + 32;
}

// One CTA has two panels of one group and walks a segment's chunks. SEGMENT 0: a whole
// sequence; 1: first pass of a split walk (from zero, only the end state); 2: second
// pass (from the start states that head_join_kernel made).
template <int NPAD, bool REV, int PLANES, int SEGMENT>
__global__ void __launch_bounds__(256) head_state_kernel(StateArgs a)
{
    constexpr int COLS = NPAD / 2;  // state columns of a thread
    constexpr int BP = NPAD / 64;   // panels of a b tile
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t bar;
    __shared__ uint32_t tmem_slot;
    const Dims &z = a.z;
    const int tid = threadIdx.x, warp = tid / 32, wg = tid / 128, wt = tid % 128;
    const int64_t slot = blockIdx.x;
    const int pairs = (z.npan + 1) / 2, g = blockIdx.y / pairs, pair = blockIdx.y % pairs;
    const ChunkRef sg = find_chunk(z.cu, z.S, z.tok, a.span, slot);
    if (sg.len == 0 && (sg.k != 0 || SEGMENT != 0)) return;
    const int nchunk = (sg.len + kC - 1) / kC;
    int64_t lo, hi;
    seq_bounds(z.cu, z.S, z.tok, sg.seq, lo, hi);
    const int64_t first = lo / kC + sg.seq + (int64_t)sg.k * (a.span / kC);  // first chunk's slot

    const uint32_t base = (saddr(raw) + 1023) & ~1023u;
    const uint32_t sx = base, sb = base + 6 * umma::kPanel;
    float *weights = reinterpret_cast<float *>(raw + (sb + 2 * BP * umma::kPanel - saddr(raw)));
    float *decays = weights + 2 * 2 * kC;
    if (tid == 0) mbar_init(&bar);
    if (warp == 0) umma::alloc(&tmem_slot, NPAD == 128 ? 256 : 128);
    umma::fence_before();
    __syncthreads();
    umma::fence_after();
    const uint32_t tm = tmem_slot;

    // conversion side: this warpgroup's panel; state side: row wt (of both panels), COLS columns
    const int xi = 2 * pair + wg, si = 2 * pair + wt / 64;
    const bool has_x = xi < z.npan, has_s = si < z.npan;
    const PanelRef xp = panel_of(z, g, min(xi, z.npan - 1)), sp = panel_of(z, g, min(si, z.npan - 1));
    const int p = wt % 64, n0 = wg * COLS;
    const bool row_in = has_s && p < sp.rows;
    const bf16 *bsrc = a.b + (int64_t)g * z.N;
    const bf16 *xsrc = a.x + (int64_t)xp.h * z.P + xp.p0;

    float st[COLS];
    {
        const float *src = nullptr;
        if (SEGMENT == 0 && a.init && row_in)
            src = a.init + (((int64_t)sg.seq * z.H + sp.h) * z.P + sp.p0 + p) * z.N;
        const float4 *sgp = nullptr;
        if (SEGMENT == 2 && has_s)
            sgp = reinterpret_cast<const float4 *>(
                      a.seg + (slot * z.G * z.npan + g * z.npan + si) * 64 * NPAD) + (n0 / 4) * 64 + p;
#pragma unroll
        for (int i = 0; i < COLS / 4; ++i) {
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (sgp) v = sgp[i * 64];
            st[4 * i] = v.x; st[4 * i + 1] = v.y; st[4 * i + 2] = v.z; st[4 * i + 3] = v.w;
            if (src)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (n0 + 4 * i + e < z.N) st[4 * i + e] = src[n0 + 4 * i + e];
        }
    }

    uint4 xr[8];
    double cn = 0.0, cq = 0.0;
    float dn = 0.0f;
    auto chunk_at = [&](int kk) { return REV ? nchunk - 1 - kk : kk; };
    auto load = [&](int kk) {
        const int k = chunk_at(kk);
        const int64_t t0 = sg.start + (int64_t)k * kC;
        const int len = (int)min((int64_t)kC, sg.start + sg.len - t0);
        load_tile<NPAD, 256>(sb + (kk & 1) * BP * umma::kPanel, bsrc + t0 * a.b_stride, a.b_stride, len,
                             z.N, a.b_vec, tid);
        umma::cp_commit();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = 16 * i + wt / 8, c = wt % 8;
            const int n = has_x && r < len ? min(8, xp.rows - 8 * c) : 0;
            const bf16 *q = xsrc + (t0 + r) * a.x_stride + 8 * c;
            xr[i] = n <= 0 ? make_uint4(0, 0, 0, 0) : a.x_vec ? ldg16(q) : read8(q, n);
        }
        const int64_t at = ((first + k) * z.H + xp.h) * kC;
        cn = a.c[at + wt];
        cq = a.c[at + kC - 1];
        dn = a.d[at + wt];
    };
    auto set_weights = [&](int kk) {
        weights[(kk & 1) * 256 + tid] =
            REV ? ex2_approx((float)cn) : dn * ex2_approx((float)(cq - cn));
        // four deep: a slow warp may still be at chunk kk - 2
        if (wt == 0) decays[(kk & 3) * 2 + wg] = ex2_approx((float)cq);
    };
    auto step = [&](int kk) {  // st = decay st + product of chunk kk
        const float e = decays[(kk & 3) * 2 + wt / 64];
#pragma unroll
        for (int j = 0; j < COLS / 32; ++j) {
            uint32_t v[32];
            umma::ld32(umma::lanes(tm + (kk & 1) * NPAD + n0 + 32 * j, warp), v);
            umma::wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i)
                st[32 * j + i] = fmaf(e, st[32 * j + i], __uint_as_float(v[i]));
        }
    };
    auto mark = [&](int kk) {
        if (SEGMENT == 1 || !has_s) return;
        bf16 *m = a.marks + ((first + chunk_at(kk)) * z.G * z.npan + g * z.npan + si) * PLANES * kMark<NPAD>;
        uint4 *q = reinterpret_cast<uint4 *>(m) + (n0 / 8) * 64 + p;
#pragma unroll
        for (int j = 0; j < COLS / 8; ++j) {
            uint32_t w[PLANES][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float v0 = st[8 * j + 2 * i], v1 = st[8 * j + 2 * i + 1];
#pragma unroll
                for (int s = 0; s < PLANES; ++s) {
                    w[s][i] = umma::pack(v0, v1);
                    v0 -= umma::lo_f(w[s][i]);
                    v1 -= umma::hi_f(w[s][i]);
                }
            }
#pragma unroll
            for (int s = 0; s < PLANES; ++s)
                q[(s * (NPAD / 8) + j) * 64] = make_uint4(w[s][0], w[s][1], w[s][2], w[s][3]);
        }
    };

    bool failed = false;
    if (nchunk > 0) {
        load(0);
        set_weights(0);
    }
    __syncthreads();
    for (int kk = 0; kk < nchunk; ++kk) {
        if (kk > 0) mbar_wait(&bar, (kk - 1) & 1, failed, &g_status, 1);
        umma::fence_after();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = 16 * i + wt / 8, c = wt % 8;
            uint4 hi4, mid4, lo4;
            split3(xr[i], weights[(kk & 1) * 256 + wg * 128 + r], hi4, mid4, lo4);
            const uint32_t at = sx + wg * umma::kPanel + umma::piece(r, c);
            sts16(at, hi4);
            sts16(at + 2 * umma::kPanel, mid4);
            sts16(at + 4 * umma::kPanel, lo4);
        }
        if (kk + 1 < nchunk) {
            load(kk + 1);
            umma::cp_wait<1>();
        } else {
            umma::cp_wait<0>();
        }
        fence_proxy_async();
        umma::fence_before();
        __syncthreads();
        if (tid == 0) {
            umma::fence_after();
            const uint32_t bt = sb + (kk & 1) * BP * umma::kPanel;
            for (int s = 0; s < 3; ++s)
#pragma unroll
                for (int k16 = 0; k16 < 8; ++k16)
                    umma::mma(tm + (kk & 1) * NPAD,
                              umma::desc_mn(sx + 2 * s * umma::kPanel, k16, umma::kPanel),
                              umma::desc_mn(bt, k16, umma::kPanel), umma::idesc(NPAD, true, true),
                              s + k16 > 0);
            umma::commit(&bar);
        }
        __syncwarp();
        if (kk > 0) step(kk - 1);
        mark(kk);
        if (kk + 1 < nchunk) set_weights(kk + 1);
        umma::fence_before();
        __syncthreads();
    }
    if (nchunk > 0) {
        mbar_wait(&bar, (nchunk - 1) & 1, failed, &g_status, 1);
        umma::fence_after();
        step(nchunk - 1);
    }
    if (SEGMENT == 0 && a.final_ && row_in) {
        float *dst = a.final_ + (((int64_t)sg.seq * z.H + sp.h) * z.P + sp.p0 + p) * z.N;
        const bool v4 = z.N % 4 == 0 && reinterpret_cast<uintptr_t>(a.final_) % 16 == 0;
#pragma unroll
        for (int i = 0; i < COLS / 4; ++i) {
            const int n = n0 + 4 * i;
            if (v4 && n < z.N)
                *reinterpret_cast<float4 *>(dst + n) =
                    make_float4(st[4 * i], st[4 * i + 1], st[4 * i + 2], st[4 * i + 3]);
            else
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (n + e < z.N) dst[n + e] = st[4 * i + e];
        }
    }
    if (SEGMENT == 1 && has_s) {
        float4 *q = reinterpret_cast<float4 *>(
                        a.seg + (slot * z.G * z.npan + g * z.npan + si) * 64 * NPAD) + (n0 / 4) * 64 + p;
#pragma unroll
        for (int i = 0; i < COLS / 4; ++i)
            q[i * 64] = make_float4(st[4 * i], st[4 * i + 1], st[4 * i + 2], st[4 * i + 3]);
        if (wg == 0 && p == 0) {
            double t = 0.0;
            for (int k = 0; k < nchunk; ++k) t += a.c[((first + k) * z.H + sp.h) * kC + kC - 1];
            a.segdec[slot * z.H + sp.h] = t;
        }
    }
    umma::fence_before();
    __syncthreads();
    if (warp == 0) umma::dealloc(tm, NPAD == 128 ? 256 : 128);
}

// One block per (sequence, panel): turns the segments' end states from zero into their
// start states, and leaves the sequence's final state.
template <int NPAD, bool REV>
__global__ void __launch_bounds__(256) head_join_kernel(StateArgs a)
{
    const Dims &z = a.z;
    const int64_t s = blockIdx.x;
    const int g = blockIdx.y / z.npan, pi = blockIdx.y % z.npan;
    const PanelRef pr = panel_of(z, g, pi);
    int64_t lo, hi;
    seq_bounds(z.cu, z.S, z.tok, s, lo, hi);
    const int nseg = (int)((hi - lo + a.span - 1) / a.span);
    const int64_t base = lo / a.span + s;
    for (int x = threadIdx.x; x < 16 * NPAD; x += 256) {
        const int n = x / 64 * 4, p = x % 64;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float *e = &v.x;
        const int64_t at = ((s * z.H + pr.h) * z.P + pr.p0 + p) * z.N + n;
        if (a.init && p < pr.rows)
            for (int i = 0; i < 4; ++i)
                if (n + i < z.N) e[i] = a.init[at + i];
        for (int k = 0; k < nseg; ++k) {
            const int64_t slot = base + (REV ? nseg - 1 - k : k);
            float4 *q = reinterpret_cast<float4 *>(a.seg + (slot * z.G * z.npan + g * z.npan + pi) * 64 * NPAD) + x;
            const float4 end = *q;
            const float dec = ex2_approx((float)a.segdec[slot * z.H + pr.h]);
            *q = v;
            v.x = fmaf(dec, v.x, end.x);
            v.y = fmaf(dec, v.y, end.y);
            v.z = fmaf(dec, v.z, end.z);
            v.w = fmaf(dec, v.w, end.w);
        }
        if (a.final_ && p < pr.rows)
            for (int i = 0; i < 4; ++i)
                if (n + i < z.N) a.final_[at + i] = e[i];
    }
}

template <int NPAD, bool REV, int PLANES, int SEGMENT>
cudaError_t launch_walk(const StateArgs &a, cudaStream_t st, int *launches)
{
    constexpr int bytes = state_smem<NPAD>();
    if (cudaError_t e = cudaFuncSetAttribute(head_state_kernel<NPAD, REV, PLANES, SEGMENT>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        e != cudaSuccess)
        return e;
    const dim3 grid((unsigned)head_slots(a.z.tok, a.z.S, a.span), (unsigned)(a.z.G * ((a.z.npan + 1) / 2)));
    head_state_kernel<NPAD, REV, PLANES, SEGMENT><<<grid, 256, bytes, st>>>(a);
    ++*launches;
    return cudaGetLastError();
}

template <int NPAD, bool REV, int PLANES>
cudaError_t states(const StateArgs &a, bool split, cudaStream_t st, int *launches)
{
    if (!split) return launch_walk<NPAD, REV, PLANES, 0>(a, st, launches);
    if (cudaError_t e = launch_walk<NPAD, REV, PLANES, 1>(a, st, launches); e != cudaSuccess) return e;
    head_join_kernel<NPAD, REV><<<dim3((unsigned)a.z.S, (unsigned)(a.z.G * a.z.npan)), 256, 0, st>>>(a);
    ++*launches;
    if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
    return launch_walk<NPAD, REV, PLANES, 2>(a, st, launches);
}

}  // namespace

Dims dims_of(const HeadScanArgs &a)
{
    Dims z;
    z.cu = a.cu;
    z.S = a.S;
    z.tok = a.tok;
    z.H = (int)a.H;
    z.P = (int)a.P;
    z.G = (int)a.G;
    z.N = (int)a.N;
    z.np = (z.P + 63) / 64;
    z.npan = z.H / z.G * z.np;
    return z;
}

// A split walk reads its inputs twice, so it pays once it more than doubles the CTAs at
// work: below a third of the SMs.
int64_t segment_span(const Dims &z, bool *split)
{
    const int64_t walks = z.S * z.G * ((z.npan + 1) / 2);
    const int64_t chunks = (z.tok + kC - 1) / kC;
    *split = false;
    if (walks * 3 > 148 || chunks < 8 * z.S) return (int64_t)1 << 31;
    int64_t seg = (chunks * walks / z.S + 147) / 148;  // chunks a segment, for at most one CTA an SM
    if (seg < 2) seg = 2;
    *split = true;
    return seg * kC;
}

cudaError_t launch_tables(const HeadScanArgs &a, const Dims &z, double *c, float *d,
                          cudaStream_t stream, int *launches)
{
    const dim3 grid((unsigned)head_slots(z.tok, z.S, kC), (unsigned)((z.H + 31) / 32));
    head_table_kernel<<<grid, 256, 0, stream>>>(z, static_cast<const bf16 *>(a.delta), a.delta_stride,
                                                a.A, a.dt_bias, a.delta_softplus, c, d);
    ++*launches;
    return cudaGetLastError();
}

cudaError_t launch_states(const StateArgs &a, bool rev, int planes, bool split, cudaStream_t st,
                          int *launches)
{
    const bool wide = a.z.N > 64;
    if (planes == 1)
        return wide ? states<128, false, 1>(a, split, st, launches)
                    : states<64, false, 1>(a, split, st, launches);
    if (rev) return wide ? states<128, true, 2>(a, split, st, launches)
                         : states<64, true, 2>(a, split, st, launches);
    return wide ? states<128, false, 2>(a, split, st, launches)
                : states<64, false, 2>(a, split, st, launches);
}

}  // namespace hm

int read_head_state_status(bool clear)
{
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, hm::g_status, sizeof(v)) != cudaSuccess) return -1;
    if (clear && v) {
        const int zero = 0;
        if (cudaMemcpyToSymbol(hm::g_status, &zero, sizeof(zero)) != cudaSuccess) return -1;
    }
    return v;
}

}  // namespace ssm
