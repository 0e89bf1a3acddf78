// head_mma_out.cu -- outputs of the bf16 scan with one decay per head (tensor cores).
//
// One CTA has a chunk (128 tokens) of one group and some of its panels. It makes
// G = C B^T once (it stays in tensor memory), and for every panel
//   y = M u + e^{c_t} (C S0^T) + D u,   M_ts = G_ts e^{c_t - c_s} d_s  (t >= s).
// Two teams of eight warps take panels in turn, each with its own buffers, a warp that
// issues the matrix instructions and one that copies the next panel's u, S0 and tables
// in and y out. M is rounded to bf16 once, goes to tensor memory and is the left
// operand from there. Eight warps a panel, two threads a row: what bounds the arithmetic
// is the latency of a warp's own chain, so more and shorter chains win.
//
// e^{c_t - c_s} needs no exponential per pair below the diagonal blocks: for t in the
// 32-token block i and s in an earlier one it is e^{c_t - r_i} e^{r_i - c_s}, r_i the
// running sum before block i, and both factors are at most one.
//
// Measured on a B200, 65536 tokens, 80 heads of 64 x 128: 441 us for 2.15 GB (u, y, the
// states before the chunks, tables), 4.9 TB/s or 75% of a copy's rate; 20% of the matrix
// rate. Bound by a team's chain of waits (tables and u in, M, product, y out) at two teams
// an SM, which shared memory allows. Roles instead of teams (16 warps for M, 8 for y) took
// 548 us.
#include <type_traits>

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
    const float *tab;
    const bf16 *marks;
    bf16 *y;
    int per;  // panels of a CTA
    bool y_vec;
};

constexpr int kTeamWarps = 8, kTeams = 2;
constexpr int kOutIssuer = kTeams * kTeamWarps, kOutLoader = kOutIssuer + kTeams;
constexpr int kOutThreads = (kOutLoader + kTeams) * 32;

// A stage: u (y takes its place), S0, tables.
template <int NPAD>
constexpr uint32_t out_stage()
{
    return (umma::kPanel + 64 * NPAD * 2 + kTabOut * 4 + 1023) / 1024 * 1024;
}
template <int NPAD>
constexpr int out_smem()
{
    return 1024 + 2 * (NPAD / 64) * umma::kPanel + 2 * kTeams * out_stage<NPAD>();
}

template <int NPAD, bool VEC>
__global__ void __launch_bounds__(kOutThreads) head_out_kernel(OutArgs a, const __grid_constant__ CUtensorMap umap,
                                                               const __grid_constant__ CUtensorMap ymap)
{
    constexpr int BP = NPAD / 64;
    constexpr uint32_t STAGE = out_stage<NPAD>(), S0B = 64 * NPAD * 2;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t gbar, landed[kTeams][2], stored[kTeams][2], ready[kTeams], done[kTeams];
    __shared__ uint32_t tmem_slot;
    const Dims &z = a.z;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int64_t slot = blockIdx.x;
    const int nb = (z.npan + a.per - 1) / a.per;
    const int g = blockIdx.y / nb, pb = blockIdx.y % nb * a.per, pe = min(pb + a.per, z.npan);
    const ChunkRef ck = find_chunk(z.cu, z.S, z.tok, kC, slot);
    if (ck.len == 0) return;
    const int len = ck.len;
    // a whole chunk's y goes out as tiles; the tail of a sequence must not cover the next
    const bool tiles = VEC && a.y_vec && len == kC;

    const uint32_t sC = (saddr(raw) + 1023) & ~1023u, sB = sC + BP * umma::kPanel;
    const int team = warp < kOutIssuer ? warp / kTeamWarps : (warp - kOutIssuer) % kTeams, x = tid % 256;
    const uint32_t sW = sB + BP * umma::kPanel + team * 2 * STAGE;  // this team's two stages
    if (tid == 0) {
        mbar_init_n(&gbar, 1);
        for (int i = 0; i < kTeams; ++i) {
            for (int j = 0; j < 2; ++j) {
                mbar_init_n(&landed[i][j], 1);
                mbar_init_n(&stored[i][j], kTeamWarps);
            }
            mbar_init_n(&ready[i], kTeamWarps);
            mbar_init_n(&done[i], 1);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) umma::alloc(&tmem_slot, 512);
    if (warp < kOutIssuer) {
        load_tile<NPAD, 512, VEC>(sC, a.C + ck.start * a.bc_stride + (int64_t)g * z.N, a.bc_stride, len, z.N, tid);
        load_tile<NPAD, 512, VEC>(sB, a.B + ck.start * a.bc_stride + (int64_t)g * z.N, a.bc_stride, len, z.N, tid);
        umma::cp_commit();
        umma::cp_wait<0>();
        fence_proxy_async();
    }
    umma::fence_before();
    __syncthreads();
    umma::fence_after();
    constexpr uint32_t tm = umma::kWhole;
    const uint32_t tM = tm + 128 + team * 192, tYa = tM + 64, tYb = tM + 128;
    const int p0 = pb + team, count = p0 < pe ? (pe - p0 + kTeams - 1) / kTeams : 0;
    unsigned tries = umma::kTries;
    auto wait = [&](uint64_t *bar, uint32_t parity) { umma::wait(bar, parity & 1, tries, &g_out_status); };

    if (warp >= kOutLoader) {
        for (int it = 0; it < count + 2; ++it) {
            const uint32_t su = sW + (it & 1) * STAGE;
            if (it >= 2 && it - 2 < count) {
                wait(&stored[team][it & 1], (it >> 1) - 1);
                if (tiles) {
                    const PanelRef p = panel_of(z, g, p0 + kTeams * (it - 2));
                    if (lane == 0) {
                        umma::tma_store_3d(&ymap, su, p.p0, p.h, (int)ck.start);
                        bulk_commit();
                        bulk_wait_read<0>();
                    }
                    __syncwarp();
                }
            }
            if (it >= count) continue;
            const PanelRef p = panel_of(z, g, p0 + kTeams * it);
            if (!VEC) {
                load_tile_warp<64>(su, a.u + ck.start * a.u_stride + (int64_t)p.h * z.P + p.p0, a.u_stride, len,
                                   p.rows, lane);
                fence_proxy_async();
            }
            __syncwarp();
            if (lane == 0) {
                uint64_t *bar = &landed[team][it & 1];
                mbar_expect_tx(bar, S0B + kTabOut * 4 + (VEC ? umma::kPanel : 0));
                if (VEC) umma::tma_3d(su, &umap, bar, p.p0, p.h, (int)ck.start);
                umma::bulk_load(su + umma::kPanel,
                                a.marks + (slot * z.G * z.npan + g * z.npan + p0 + kTeams * it) * kMark<NPAD>, S0B, bar);
                umma::bulk_load(su + umma::kPanel + S0B, a.tab + (slot * z.H + p.h) * kTab, kTabOut * 4, bar);
            }
            __syncwarp();
        }
        if (lane == 0) bulk_wait<0>();
        __syncwarp();
    } else if (warp >= kOutIssuer) {
        if (umma::elect()) {
            const uint64_t c0 = umma::desc_k(sC, 0), b0 = umma::desc_k(sB, 0);
            auto c_at = [](int k) { return (uint32_t)(k / 4 * umma::kPanel + k % 4 * 32); };
            if (team == 0) {
#pragma unroll
                for (int k = 0; k < NPAD / 16; ++k)
                    umma::mma(tm, umma::moved(c0, c_at(k)), umma::moved(b0, c_at(k)), umma::idesc(128, false, false),
                              k > 0);
                umma::commit(&gbar);
            }
            const uint64_t u0 = umma::desc_mn(sW, 0, 0), s0 = umma::plain_k(sW + umma::kPanel, 0, 64);
            auto run = [&](auto which) {  // the team's columns, known when compiling
                constexpr uint32_t m = tm + 128 + decltype(which)::value * 192, ya = m + 64, yb = m + 128;
                for (int it = 0; it < count; ++it) {
                    const uint32_t at = (it & 1) * STAGE;
                    const uint64_t u = umma::moved(u0, at), s = umma::moved(s0, at);
                    wait(&landed[team][it & 1], it >> 1);
                    if (it > 0) wait(&stored[team][(it - 1) & 1], (it - 1) >> 1);  // both accumulators were read
                    umma::fence_after();
#pragma unroll
                    for (int k = 0; k < NPAD / 16; ++k)
                        umma::mma(yb, umma::moved(c0, c_at(k)), umma::moved(s, k * 2048), umma::idesc(64, false, false),
                                  k > 0);
                    wait(&ready[team], it);
                    umma::fence_after();
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        umma::mma_ta(ya, m + 8 * k, umma::moved(u, k * 2048), umma::idesc(64, false, true), k > 0);
                    umma::commit(&done[team]);
                }
            };
            if (team == 0) run(std::integral_constant<uint32_t, 0>());
            else run(std::integral_constant<uint32_t, 1>());
        }
        __syncwarp();
    } else {
        // row t of the chunk, one of two 16-column halves of every 32
        const int wi = warp & 3, t = wi * 32 + lane, half = (warp >> 2) & 1;
        const uint32_t rM = umma::lanes(tM, warp) + 8 * half, rG = umma::lanes(tm, warp) + 16 * half;
        {  // the blocks above the diagonal stay zero for every panel
            const uint32_t zero[8] = {};
            for (int j = wi + 1; j < 4; ++j) umma::st8(rM + 16 * j, zero);
            umma::wait_st();
        }
        wait(&gbar, 0);
        umma::fence_after();
        const int own = lane - 16 * half;  // columns of a diagonal block up to this one count
        for (int it = 0; it < count; ++it) {
            const PanelRef p = panel_of(z, g, p0 + kTeams * it);
            const uint32_t su = sW + (it & 1) * STAGE;
            const float *tb = reinterpret_cast<const float *>(raw + (su + umma::kPanel + S0B - saddr(raw)));
            const float skip = a.Dskip ? a.Dskip[p.h] : 0.0f;
            uint32_t v[16];
            umma::ld16(rG, v);
            wait(&landed[team][it & 1], it >> 1);
            if (VEC && len < kC) {
                zero_tail(su, 1, len, x, 256);
                fence_proxy_async();
            }
            const float lt = tb[kTabL + t], ec = tb[kTabEc + t];
            const float rf = ex2_approx(lt);
            const f32x2 row2 = pk2(rf, rf);
            for (int j = 0; j < wi; ++j) {
                uint32_t cur[16], w[8];
                umma::wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) cur[i] = v[i];
                umma::ld16(rG + 32 * (j + 1), v);
                const float4 *cf = reinterpret_cast<const float4 *>(tb + col_at(wi) + 32 * j + 16 * half);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float4 f = cf[q];
                    float m0, m1, m2, m3;
                    upk2(mul2(mul2(pk2(f.x, f.y), row2),
                              pk2(__uint_as_float(cur[4 * q]), __uint_as_float(cur[4 * q + 1]))), m0, m1);
                    upk2(mul2(mul2(pk2(f.z, f.w), row2),
                              pk2(__uint_as_float(cur[4 * q + 2]), __uint_as_float(cur[4 * q + 3]))), m2, m3);
                    w[2 * q] = umma::pack(m0, m1);
                    w[2 * q + 1] = umma::pack(m2, m3);
                }
                umma::st8(rM + 16 * j, w);
            }
            {
                uint32_t w[8];
                const float4 *dl = reinterpret_cast<const float4 *>(tb + kTabL + 32 * wi + 16 * half);
                const float4 *dd = reinterpret_cast<const float4 *>(tb + kTabD + 32 * wi + 16 * half);
                umma::wait_ld();
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float4 l4 = dl[q], d4 = dd[q];
                    const float ls[4] = {l4.x, l4.y, l4.z, l4.w}, ds[4] = {d4.x, d4.y, d4.z, d4.w};
                    float m[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        m[e] = 4 * q + e <= own
                                   ? __uint_as_float(v[4 * q + e]) * (ex2_approx(lt - ls[e]) * ds[e]) : 0.0f;
                    w[2 * q] = umma::pack(m[0], m[1]);
                    w[2 * q + 1] = umma::pack(m[2], m[3]);
                }
                umma::st8(rM + 16 * wi, w);
            }
            umma::wait_st();
            umma::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ready[team]);
            wait(&done[team], it);
            umma::fence_after();
            {
                uint32_t va[2][16], vb[2][16];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    umma::ld16(umma::lanes(tYa, warp) + 32 * half + 16 * j, va[j]);
                    umma::ld16(umma::lanes(tYb, warp) + 32 * half + 16 * j, vb[j]);
                }
                umma::wait_ld();
#pragma unroll
                for (int j = 0; j < 4; ++j) {  // y takes u's place in shared memory
                    const uint32_t at = su + umma::piece(t, 4 * half + j);
                    const uint4 uv = lds16(at);
                    const uint32_t in[4] = {uv.x, uv.y, uv.z, uv.w};
                    uint32_t o[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int n = 8 * (j & 1) + 2 * i;
                        const float y0 = fmaf(ec, __uint_as_float(vb[j / 2][n]), __uint_as_float(va[j / 2][n]));
                        const float y1 = fmaf(ec, __uint_as_float(vb[j / 2][n + 1]), __uint_as_float(va[j / 2][n + 1]));
                        o[i] = umma::pack(fmaf(skip, umma::lo_f(in[i]), y0), fmaf(skip, umma::hi_f(in[i]), y1));
                    }
                    sts16(at, make_uint4(o[0], o[1], o[2], o[3]));
                }
            }
            umma::fence_before();
            if (!tiles) {
                bar_sync(1 + team, 256);
                const int r0 = x / 8, c = x % 8, n = min(8, p.rows - 8 * c);
                bf16 *yo = a.y + ((ck.start + r0) * z.H + p.h) * (int64_t)z.P + p.p0 + 8 * c;
                for (int i = 0; i < 4; ++i) {
                    if (r0 + 32 * i < len && n > 0) {
                        const uint4 o = lds16(su + umma::piece(r0 + 32 * i, c));
                        if (VEC && a.y_vec) {
                            *reinterpret_cast<uint4 *>(yo) = o;
                        } else {
                            const uint32_t w[4] = {o.x, o.y, o.z, o.w};
                            for (int e = 0; e < n; ++e)
                                reinterpret_cast<unsigned short *>(yo)[e] =
                                    (unsigned short)((e < 4 ? (e < 2 ? w[0] : w[1]) : (e < 6 ? w[2] : w[3])) >> (16 * (e & 1)));
                        }
                    }
                    yo += 32 * (int64_t)z.H * z.P;
                }
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&stored[team][it & 1]);
        }
    }
    umma::fence_before();
    __syncthreads();
    if (warp == 0) umma::dealloc(tm, 512);
}

template <int NPAD, bool VEC>
cudaError_t out(const OutArgs &a, int64_t slots, cudaStream_t st)
{
    constexpr int bytes = out_smem<NPAD>();
    if (cudaError_t e = cudaFuncSetAttribute(head_out_kernel<NPAD, VEC>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        e != cudaSuccess)
        return e;
    const dim3 grid((unsigned)slots, (unsigned)(a.z.G * ((a.z.npan + a.per - 1) / a.per)));
    CUtensorMap umap{}, ymap{};
    if (VEC && (!umma::encode_3d(&umap, a.u, a.z.tok, a.z.H, a.z.P, a.u_stride) ||
                (a.y_vec && !umma::encode_3d(&ymap, a.y, a.z.tok, a.z.H, a.z.P, (int64_t)a.z.H * a.z.P))))
        return cudaErrorInvalidValue;
    head_out_kernel<NPAD, VEC><<<grid, kOutThreads, bytes, st>>>(a, umap, ymap);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_forward(const HeadScanArgs &a, cudaStream_t st, int *launches)
{
    const Dims z = dims_of(a);
    const Plan plan = plan_of(z, lengths_known(z));
    const Layout l = layout_of(z, 1, plan);
    char *ws = static_cast<char *>(a.workspace);
    float *tab = reinterpret_cast<float *>(ws + l.tab);
    bf16 *marks = reinterpret_cast<bf16 *>(ws + l.marks);
    int64_t *span = reinterpret_cast<int64_t *>(ws + l.span);
    if (cudaError_t e = launch_tables(a, z, tab, false, plan, span, st, launches); e != cudaSuccess) return e;
    const bool vec = vec16(a.B, a.bc_stride, a.N) && vec16(a.C, a.bc_stride, a.N) && vec16(a.u, a.u_stride, a.P);
    StateArgs s{z, static_cast<const bf16 *>(a.u), a.u_stride, static_cast<const bf16 *>(a.B), a.bc_stride,
                tab, a.h0, a.h_final, marks, reinterpret_cast<float *>(ws + l.seg),
                reinterpret_cast<float *>(ws + l.segdec),
                a.cu && a.S > 1 ? reinterpret_cast<int32_t *>(ws + l.order) : nullptr, span};
    if (cudaError_t e = launch_states(s, false, 1, plan, vec, st, launches); e != cudaSuccess) return e;
    if (a.tok == 0) return cudaSuccess;
    const int64_t slots = head_slots(z.tok, z.S, kC);
    // G is made once per CTA, a start worth about two panels
    const int64_t per = units_of_cta(slots * z.G, z.npan, 2.0);
    OutArgs o{z, static_cast<const bf16 *>(a.u), static_cast<const bf16 *>(a.B), static_cast<const bf16 *>(a.C),
              a.u_stride, a.bc_stride, a.Dskip, tab, marks, static_cast<bf16 *>(a.y), (int)per, vec16(a.y, a.P, a.P)};
    ++*launches;
    if (z.N > 64) return vec ? out<128, true>(o, slots, st) : out<128, false>(o, slots, st);
    return vec ? out<64, true>(o, slots, st) : out<64, false>(o, slots, st);
}

size_t forward_bytes(const Dims &z)
{
    // asked for without cu_seqlens: room for the walk of dense rows and of packed ones
    const size_t dense = layout_of(z, 1, plan_of(z, true)).total, packed = layout_of(z, 1, plan_of(z, false)).total;
    return dense > packed ? dense : packed;
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
