// head_mma_bwd.cu -- backward of the bf16 scan with one decay per head (tensor cores).
//
// With every chunk's start state S0 and end-state gradient dS in the workspace (two bf16
// planes each), chunks are independent. Per chunk and panel, rows s, columns t:
//   G^T = B C^T, dM^T = u dy^T, L = e^{c_t - c_s} (t >= s), M^T = G^T L d_s,
//   V = B dS, Yi = C S0,
//   du = M^T dy + d_s e^{cQ-c_s} V + D dy,   dG^T = dM^T L d_s  (summed over panels),
//   K_s = sum_t dM G L, R_t = sum_s dM G L d_s, J_s = e^{cQ-c_s} u.V, I_t = e^{c_t} dy.Yi,
// from which one warp per CTA makes ddelta and the chunk's shares of dA and ddt_bias.
// head_bwd_kernel does this; head_bwd_bc_kernel then makes
//   dC = sum over panels of e^{c_t} dy S0 + dG B,   dB = the same of w_s u dS + dG^T C.
//
// What gradients of the decays are made of is never rounded to bf16: G and dM come from
// the exact bf16 inputs, V and Yi from two planes of the states (17 bits), and the sums
// are fp32. Rounded to bf16 once: M as a left operand (of du), the states that dB and dC
// take in from other chunks.
//
// Measured on a B200, 32768 tokens, 80 heads of 64 x 128: head_bwd_kernel 614 us (2.6 GB:
// u, dy, du, four planes of states: 4.2 TB/s, 65% of a copy's rate; issue slots 60% used,
// the matrix pipe 23%), head_bwd_bc_kernel 238 us (1.5 GB, 6.3 TB/s, 96%). The first is
// bound by its 16 compute warps' instructions and their latency, and was held by the
// instruction cache before: 119 KB of code took 860 us, 75 KB takes 614.
#include <type_traits>

#include "head_mma.cuh"

namespace ssm {
namespace hm {

__device__ int g_bwd_status;

namespace {

struct BwdArgs {
    Dims z;
    const bf16 *u, *dy, *B, *C, *delta;
    int64_t u_stride, bc_stride, delta_stride;
    const float *A, *Dskip, *dt_bias;
    int softplus;
    const float *tab;
    const bf16 *S0, *dS;  // marks, two planes
    bf16 *du, *ddelta, *dB, *dC;
    bf16 *dg;     // (slot, group, range, 2 planes) 128 x 128 tiles of dG^T as they lie in shared memory
    float *part;  // (slot, head, 3)
    int per, ranges;  // panels of a CTA (whole heads), CTAs of a chunk and group
    bool du_vec;
};

constexpr int kWork = 16;  // compute warps
constexpr int kBIssuer = kWork, kBLoader = kWork + 1, kBFinish = kWork + 2;
constexpr int kFinish = 2, kBwdThreads = (kBFinish + kFinish) * 32;

// Sums over a panel that one warp finishes; two buffers.
struct Sums {
    float r[4][kC];   // R from each 32-row block
    float k[4][kC];   // K from each column group
    float i[4][kC], j[4][kC];
    float own[kC];    // the diagonal of dM G
    float skip[kWork], dot[kWork];
};

template <int NPAD>
constexpr int bwd_smem()
{
    return 1024 + 2 * (NPAD / 64) * umma::kPanel + 4 * umma::kPanel + 4 * 64 * NPAD * 2 + 2 * kTab * 4 +
           2 * (int)sizeof(Sums);
}

// Tensor memory.
constexpr uint32_t kG = 0, kDm = 128, kMt = 256, kDu = 320, kV = 384, kYi = 448;

// Sums of 8 values over the 32 lanes of a warp: lane l returns value l % 8's.
__device__ __forceinline__ float reduce8(const float (&v)[8], int lane)
{
    float a[4], b[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool up = lane & 4;
        const float keep = up ? v[i + 4] : v[i], give = up ? v[i] : v[i + 4];
        a[i] = keep + __shfl_xor_sync(0xffffffffu, give, 4);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const bool up = lane & 2;
        const float keep = up ? a[i + 2] : a[i], give = up ? a[i] : a[i + 2];
        b[i] = keep + __shfl_xor_sync(0xffffffffu, give, 2);
    }
    const bool up = lane & 1;
    float c = (up ? b[1] : b[0]) + __shfl_xor_sync(0xffffffffu, up ? b[0] : b[1], 1);
    c += __shfl_xor_sync(0xffffffffu, c, 8);
    return c + __shfl_xor_sync(0xffffffffu, c, 16);
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A panel of u or dy by one warp, with zeros behind the sequence's end.
template <bool VEC>
__device__ __forceinline__ void load_rows(uint32_t dst, const bf16 *src, int64_t stride, int len, int cols, int lane)
{
    if (VEC) load_tile<64, 32, true>(dst, src, stride, len, cols, lane);
    else load_tile_warp<64>(dst, src, stride, len, cols, lane);
}

template <int NPAD, bool VEC>
__global__ void __launch_bounds__(kBwdThreads) head_bwd_kernel(BwdArgs a, const __grid_constant__ CUtensorMap umap,
                                                               const __grid_constant__ CUtensorMap ymap,
                                                               const __grid_constant__ CUtensorMap dumap)
{
    constexpr int BP = NPAD / 64;
    constexpr uint32_t PLANE = 64 * NPAD * 2;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t gbar, ud[2], ss, ss_free, dm, vy, mt, du, epi[2], fin[2];
    __shared__ uint32_t tmem_slot;
    const Dims &z = a.z;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int64_t slot = blockIdx.x;
    const int g = blockIdx.y / a.ranges, range = blockIdx.y % a.ranges;
    const int pb = range * a.per, pe = min(pb + a.per, z.npan), count = pe - pb;
    const ChunkRef ck = find_chunk(z.cu, z.S, z.tok, kC, slot);
    if (ck.len == 0) {  // the sums over chunks read every slot
        for (int i = tid; i < count / z.np * 3; i += kBwdThreads)
            a.part[(slot * z.H + panel_of(z, g, pb).h) * 3 + i] = 0.0f;
        return;
    }
    const int len = ck.len;
    const bool whole = VEC && len == kC;      // u and dy come as tiles
    const bool tiles = whole && a.du_vec;     // and du goes as tiles

    const uint32_t sC = (saddr(raw) + 1023) & ~1023u, sB = sC + BP * umma::kPanel;
    const uint32_t sUD = sB + BP * umma::kPanel, sS = sUD + 4 * umma::kPanel, sT = sS + 4 * PLANE;
    Sums *sums = reinterpret_cast<Sums *>(raw + (sT + 2 * kTab * 4 - saddr(raw)));
    if (tid == 0) {
        mbar_init_n(&gbar, 1);
        mbar_init_n(&ss, 1);
        mbar_init_n(&ss_free, kWork / 2 + 1);
        mbar_init_n(&dm, 1);
        mbar_init_n(&vy, 1);
        mbar_init_n(&mt, kWork);
        mbar_init_n(&du, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init_n(&ud[i], 1);
            mbar_init_n(&epi[i], kWork);
            mbar_init_n(&fin[i], kFinish);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) umma::alloc(&tmem_slot, 512);
    if (warp < kWork) {
        load_tile<NPAD, 512, VEC>(sC, a.C + ck.start * a.bc_stride + (int64_t)g * z.N, a.bc_stride, len, z.N, tid);
        load_tile<NPAD, 512, VEC>(sB, a.B + ck.start * a.bc_stride + (int64_t)g * z.N, a.bc_stride, len, z.N, tid);
        umma::cp_commit();
        umma::cp_wait<0>();
        fence_proxy_async();
    }
    umma::fence_before();
    __syncthreads();
    umma::fence_after();
    unsigned tries = umma::kTries;
    auto wait = [&](uint64_t *bar, uint32_t parity) { umma::wait(bar, parity & 1, tries, &g_bwd_status); };
    const int64_t mark0 = (slot * z.G * z.npan + g * z.npan + pb) * 2 * kMark<NPAD>;  // both planes of a panel

    if (warp == kBLoader) {
        for (int it = 0; it < count + 2; ++it) {
            const uint32_t su = sUD + (it & 1) * 2 * umma::kPanel;
            if (it >= 2 && it - 2 < count) {
                wait(&epi[it & 1], (it >> 1) - 1);
                if (tiles) {
                    const PanelRef p = panel_of(z, g, pb + it - 2);
                    if (lane == 0) {
                        umma::tma_store_3d(&dumap, su, p.p0, p.h, (int)ck.start);
                        bulk_commit();
                        bulk_wait_read<0>();
                    }
                    __syncwarp();
                }
            }
            if (it >= count) continue;
            const PanelRef p = panel_of(z, g, pb + it);
            if (!whole) {
                load_rows<VEC>(su, a.u + ck.start * a.u_stride + (int64_t)p.h * z.P + p.p0, a.u_stride, len, p.rows, lane);
                load_rows<VEC>(su + umma::kPanel, a.dy + (ck.start * z.H + p.h) * (int64_t)z.P + p.p0,
                               (int64_t)z.H * z.P, len, p.rows, lane);
                umma::cp_commit();
                umma::cp_wait<0>();
                fence_proxy_async();
            }
            __syncwarp();
            if (lane == 0) {
                uint64_t *bar = &ud[it & 1];
                mbar_expect_tx(bar, kTab * 4 + (whole ? 2 * umma::kPanel : 0));
                if (whole) {
                    umma::tma_3d(su, &umap, bar, p.p0, p.h, (int)ck.start);
                    umma::tma_3d(su + umma::kPanel, &ymap, bar, p.p0, p.h, (int)ck.start);
                }
                umma::bulk_load(sT + (it & 1) * kTab * 4, a.tab + (slot * z.H + p.h) * kTab, kTab * 4, bar);
            }
            __syncwarp();
            if (it > 0) wait(&ss_free, it - 1);
            if (lane == 0) {
                mbar_expect_tx(&ss, 4 * PLANE);
                umma::bulk_load(sS, a.S0 + mark0 + it * 2 * kMark<NPAD>, 2 * PLANE, &ss);
                umma::bulk_load(sS + 2 * PLANE, a.dS + mark0 + it * 2 * kMark<NPAD>, 2 * PLANE, &ss);
            }
            __syncwarp();
        }
        if (lane == 0) bulk_wait<0>();
        __syncwarp();
    } else if (warp == kBIssuer) {
        if (umma::elect()) {
            const uint64_t c0 = umma::desc_k(sC, 0), b0 = umma::desc_k(sB, 0);
            auto at = [](int k) { return (uint32_t)(k / 4 * umma::kPanel + k % 4 * 32); };
#pragma unroll
            for (int k = 0; k < NPAD / 16; ++k)
                umma::mma(kG, umma::moved(b0, at(k)), umma::moved(c0, at(k)), umma::idesc(128, false, false), k > 0);
            umma::commit(&gbar);
            const uint64_t u0 = umma::desc_k(sUD, 0), y0 = umma::desc_k(sUD + umma::kPanel, 0);
            const uint64_t ym = umma::desc_mn(sUD + umma::kPanel, 0, 0);
            const uint64_t s0 = umma::plain_k(sS, 0, 64), ds0 = umma::plain_k(sS + 2 * PLANE, 0, 64);
            auto issue_dm = [&](int it) {
                const uint32_t o = (it & 1) * 2 * umma::kPanel;
                wait(&ud[it & 1], it >> 1);
                umma::fence_after();
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    umma::mma(kDm, umma::moved(u0, o + k * 32), umma::moved(y0, o + k * 32),
                              umma::idesc(128, false, false), k > 0);
                umma::commit(&dm);
            };
            issue_dm(0);
            for (int it = 0; it < count; ++it) {
                const uint32_t o = (it & 1) * 2 * umma::kPanel;
                wait(&ss, it);
                if (it > 0) wait(&epi[(it - 1) & 1], (it - 1) >> 1);  // V, Yi and du were read
                umma::fence_after();
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int k = 0; k < NPAD / 16; ++k)
                        umma::mma(kV, umma::moved(b0, at(k)), umma::moved(ds0, s * PLANE + k * 2048),
                                  umma::idesc(64, false, false), s + k > 0);
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int k = 0; k < NPAD / 16; ++k)
                        umma::mma(kYi, umma::moved(c0, at(k)), umma::moved(s0, s * PLANE + k * 2048),
                                  umma::idesc(64, false, false), s + k > 0);
                umma::commit(&vy);
                umma::commit(&ss_free);
                wait(&mt, it);
                umma::fence_after();
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    umma::mma_ta(kDu, kMt + 8 * k, umma::moved(ym, o + k * 2048), umma::idesc(64, false, true), k > 0);
                umma::commit(&du);
                if (it + 1 < count) issue_dm(it + 1);
            }
        }
        __syncwarp();
    } else if (warp >= kBFinish) {
        // two warps, heads in turn: tokens 4 lane .. 4 lane + 3, sums over a head's panels,
        // then the head's gradients. A barrier tells phases apart by parity only, so a warp
        // may skip none of a buffer's: both wait for every panel's sums and free them,
        // whichever of them reads them. (Heads of one panel could do without, as a warp's
        // panels are then all those of one buffer: 1565 us instead of 1569 for a whole call.)
        float R[4], K[4], I[4], J[4], own[4], dsk = 0.0f, dot = 0.0f;
        auto add4 = [&](float (&v)[4], const float *q) {
            const float4 x = *reinterpret_cast<const float4 *>(q + 4 * lane);
            v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
        };
        for (int it = 0; it < count; ++it) {
            if (it / z.np % kFinish != warp - kBFinish) {  // the other warp's head
                wait(&epi[it & 1], it >> 1);
                __syncwarp();
                if (lane == 0) mbar_arrive(&fin[it & 1]);
                continue;
            }
            const PanelRef p = panel_of(z, g, pb + it);
            const bool start = p.p0 == 0, end = p.p0 + 64 >= z.P;
            const float *tb = a.tab + (slot * z.H + p.h) * kTab;
            // what the end needs from memory is on its way during the wait
            const float bias = a.dt_bias ? a.dt_bias[p.h] : 0.0f, Ah = a.A[p.h], last = tb[kTabEc + kC - 1];
            const float4 d4 = *reinterpret_cast<const float4 *>(tb + kTabD + 4 * lane);
            const float4 e4 = *reinterpret_cast<const float4 *>(tb + kTabEc + 4 * lane);
            const float4 w4 = *reinterpret_cast<const float4 *>(tb + kTabWn + 4 * lane);
            float raw4[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = 4 * lane + e;
                raw4[e] = t < len ? to_f32(a.delta[(ck.start + t) * a.delta_stride + p.h]) + bias : 0.0f;
            }
            if (start) {
#pragma unroll
                for (int e = 0; e < 4; ++e) R[e] = K[e] = I[e] = J[e] = own[e] = 0.0f;
                dsk = dot = 0.0f;
            }
            wait(&epi[it & 1], it >> 1);
            const Sums &s = sums[it & 1];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (q <= lane / 8) add4(R, s.r[q]);  // later blocks hold no row before these tokens
                add4(K, s.k[q]);
                add4(I, s.i[q]);
                add4(J, s.j[q]);
            }
            add4(own, s.own);
            dsk += lane < kWork ? s.skip[lane] : 0.0f;
            dot += lane < kWork ? s.dot[lane] : 0.0f;
            __syncwarp();
            if (lane == 0) mbar_arrive(&fin[it & 1]);
            if (!end) continue;
            const float d[4] = {d4.x, d4.y, d4.z, d4.w}, ec[4] = {e4.x, e4.y, e4.z, e4.w};
            const float wn[4] = {w4.x, w4.y, w4.z, w4.w};
            const float X = warp_sum(dot) * last;
            // gradient of log a_r from what passes through token r: outputs at or after it
            // from inputs before it (a suffix sum of rows less columns, the diagonal left
            // out since it would cancel only up to rounding), from the start state, and the
            // end state's share of inputs before it and of the start state
            double after[4], before[4], sa = 0.0, sb = 0.0;
#pragma unroll
            for (int e = 3; e >= 0; --e) {
                sa += (double)R[e] + (double)ec[e] * I[e] - (double)d[e] * K[e];
                after[e] = sa;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                before[e] = sb;
                J[e] *= wn[e];
                sb += (double)d[e] * J[e];
            }
            double ta = sa, tp = sb;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double x = __shfl_down_sync(0xffffffffu, ta, o), y = __shfl_up_sync(0xffffffffu, tp, o);
                if (lane + o < 32) ta += x;
                if (lane >= o) tp += y;
            }
            ta -= sa;
            tp -= sb;
            float pa = 0.0f, pbias = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = 4 * lane + e;
                const float dg = (float)(after[e] + ta + before[e] + tp + X);
                const float gv = (K[e] + own[e] + J[e] + Ah * dg) * head_step_grad(raw4[e], a.softplus);
                if (t < len) {
                    a.ddelta[(ck.start + t) * z.H + p.h] = __float2bfloat16_rn(gv);
                    pa = fmaf(d[e], dg, pa);
                    pbias += gv;
                }
            }
            pa = warp_sum(pa);
            pbias = warp_sum(pbias);
            dsk = warp_sum(dsk);
            if (lane == 0) {
                float *q = a.part + (slot * z.H + p.h) * 3;
                q[0] = pa;
                q[1] = pbias;
                q[2] = dsk;
            }
        }
    } else {
        // row s of the chunk (in the epilogue also row t), columns 8 cg .. of every 32
        const int wi = warp & 3, cg = warp >> 2, row = wi * 32 + lane;
        const uint32_t me = (uint32_t)wi << 21;
        {  // M^T is zero for t in blocks before s's, for every panel
            const uint32_t zero[4] = {};
            for (int j = 0; j < wi; ++j)
                umma::st4(kMt + me + 16 * j + 4 * cg, zero);
            umma::wait_st();
        }
        wait(&gbar, 0);
        umma::fence_after();
        // A warp's lanes of tensor memory and its scheduler both go by warp % 4, and later
        // rows have fewer columns t >= s: the warps of the last two blocks of rows take
        // <S0, dS> as well, 5 of 8 pieces by the last's.
        constexpr int DOTS = PLANE / 16;
        const int dot0 = (wi == 3 ? 0 : DOTS * 5 / 8) + cg * 32 + lane, dot1 = wi == 3 ? DOTS * 5 / 8 : DOTS;
        if (wi < 2 && lane == 0) sums[0].dot[warp] = sums[1].dot[warp] = 0.0f;
        float dg[4][8];  // of blocks wi, wi + 1 ..
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int c = 0; c < 8; ++c) dg[j][c] = 0.0f;
        for (int it = 0; it < count; ++it) {
            const PanelRef p = panel_of(z, g, pb + it);
            const uint32_t su = sUD + (it & 1) * 2 * umma::kPanel, sy = su + umma::kPanel;
            const float *tb = reinterpret_cast<const float *>(raw + (sT + (it & 1) * kTab * 4 - saddr(raw)));
            Sums &s = sums[it & 1];
            const float skip = a.Dskip ? a.Dskip[p.h] : 0.0f;
            float dot = 0.0f;
            if (wi >= 2) {  // <S0, dS> of this panel
                wait(&ss, it);
                for (int i = dot0; i < dot1; i += 128) {
                    const uint32_t o = sS + i * 16;
                    const uint4 ah = lds16(o), al = lds16(o + PLANE), bh = lds16(o + 2 * PLANE), bl = lds16(o + 3 * PLANE);
                    const uint32_t A4[4] = {ah.x, ah.y, ah.z, ah.w}, a4[4] = {al.x, al.y, al.z, al.w};
                    const uint32_t B4[4] = {bh.x, bh.y, bh.z, bh.w}, b4[4] = {bl.x, bl.y, bl.z, bl.w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        dot = fmaf(umma::lo_f(A4[q]) + umma::lo_f(a4[q]), umma::lo_f(B4[q]) + umma::lo_f(b4[q]), dot);
                        dot = fmaf(umma::hi_f(A4[q]) + umma::hi_f(a4[q]), umma::hi_f(B4[q]) + umma::hi_f(b4[q]), dot);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&ss_free);
                dot = warp_sum(dot);
            }
            if (it >= 2) wait(&fin[it & 1], (it >> 1) - 1);

            wait(&ud[it & 1], it >> 1);
            const float ds = tb[kTabD + row], ls = tb[kTabL + row], lls = tb[kTabLl + row];
            wait(&dm, it);
            umma::fence_after();
            float own = 0.0f;
            const f32x2 d2 = pk2(ds, ds);
            f32x2 k2 = pk2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = wi + i;  // counted from the diagonal: its code exists once
                if (j > 3) break;
                uint32_t gv[8], mv[8], w[4];
                umma::ld8(kG + me + 32 * j + 8 * cg, gv);
                umma::ld8(kDm + me + 32 * j + 8 * cg, mv);
                float L[8];
                if (i > 0) {
                    const float rn = tb[col_at(j) + row];
                    const f32x2 r2 = pk2(rn, rn);
                    const float4 ea = *reinterpret_cast<const float4 *>(tb + kTabEl + 32 * j + 8 * cg);
                    const float4 eb = *reinterpret_cast<const float4 *>(tb + kTabEl + 32 * j + 8 * cg + 4);
                    upk2(mul2(pk2(ea.x, ea.y), r2), L[0], L[1]);
                    upk2(mul2(pk2(ea.z, ea.w), r2), L[2], L[3]);
                    upk2(mul2(pk2(eb.x, eb.y), r2), L[4], L[5]);
                    upk2(mul2(pk2(eb.z, eb.w), r2), L[6], L[7]);
                } else {
                    const float4 la = *reinterpret_cast<const float4 *>(tb + kTabL + 32 * j + 8 * cg);
                    const float4 lb = *reinterpret_cast<const float4 *>(tb + kTabL + 32 * j + 8 * cg + 4);
                    const float4 ra = *reinterpret_cast<const float4 *>(tb + kTabLl + 32 * j + 8 * cg);
                    const float4 rb = *reinterpret_cast<const float4 *>(tb + kTabLl + 32 * j + 8 * cg + 4);
                    const float lt[8] = {la.x, la.y, la.z, la.w, lb.x, lb.y, lb.z, lb.w};
                    const float lr[8] = {ra.x, ra.y, ra.z, ra.w, rb.x, rb.y, rb.z, rb.w};
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        L[c] = 8 * cg + c >= lane ? ex2_approx((lt[c] - ls) + (lr[c] - lls)) : 0.0f;
                }
                umma::wait_ld();
                float wd[8];
#pragma unroll
                for (int c = 0; c < 8; c += 2) {
                    const f32x2 l2 = pk2(L[c], L[c + 1]);
                    const f32x2 g2 = pk2(__uint_as_float(gv[c]), __uint_as_float(gv[c + 1]));
                    const f32x2 m2 = pk2(__uint_as_float(mv[c]), __uint_as_float(mv[c + 1]));
                    const f32x2 gl = mul2(g2, l2), xl = mul2(m2, l2);
                    f32x2 acc = fma2(xl, d2, pk2(dg[i][c], dg[i][c + 1]));
                    upk2(acc, dg[i][c], dg[i][c + 1]);
                    float m0, m1, w0, w1;
                    upk2(mul2(gl, d2), m0, m1);
                    w[c / 2] = umma::pack(m0, m1);
                    f32x2 wl = mul2(m2, gl);
                    if (i == 0) {  // the diagonal apart
                        upk2(wl, w0, w1);
                        const bool q0 = 8 * cg + c == lane, q1 = 8 * cg + c + 1 == lane;
                        own = q0 ? w0 : q1 ? w1 : own;
                        wl = pk2(q0 ? 0.0f : w0, q1 ? 0.0f : w1);
                    }
                    k2 = add2(k2, wl);
                    upk2(mul2(wl, d2), wd[c], wd[c + 1]);
                }
                umma::st4(kMt + me + 16 * j + 4 * cg, w);
                const float r = reduce8(wd, lane);
                if (lane < 8) s.r[wi][32 * j + 8 * cg + lane] = r;
            }
            umma::wait_st();
            umma::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&mt);
            float k0, k1;
            upk2(k2, k0, k1);
            s.k[cg][row] = k0 + k1;
            if (lane / 8 == cg) s.own[row] = own;

            // columns 16 cg .. of the panel: du of row s, and the dots of rows s and t
            const float wf = tb[kTabWf + row];
            wait(&vy, it);
            umma::fence_after();
            float iv = 0.0f, jv = 0.0f, sk = 0.0f;
            const uint32_t at0 = umma::piece(row, 2 * cg), at1 = umma::piece(row, 2 * cg + 1);
            const uint4 ua = lds16(su + at0), ub = lds16(su + at1), ya = lds16(sy + at0), yb = lds16(sy + at1);
            const uint32_t uu[8] = {ua.x, ua.y, ua.z, ua.w, ub.x, ub.y, ub.z, ub.w};
            const uint32_t yy[8] = {ya.x, ya.y, ya.z, ya.w, yb.x, yb.y, yb.z, yb.w};
            float o[16];
            {
                uint32_t v[16];
                umma::ld16(kV + me + 16 * cg, v);
                umma::wait_ld();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float u0 = umma::lo_f(uu[i]), u1 = umma::hi_f(uu[i]);
                    const float y0 = umma::lo_f(yy[i]), y1 = umma::hi_f(yy[i]);
                    jv = fmaf(u0, __uint_as_float(v[2 * i]), jv);
                    jv = fmaf(u1, __uint_as_float(v[2 * i + 1]), jv);
                    sk = fmaf(u0, y0, sk);
                    sk = fmaf(u1, y1, sk);
                    o[2 * i] = fmaf(wf, __uint_as_float(v[2 * i]), skip * y0);
                    o[2 * i + 1] = fmaf(wf, __uint_as_float(v[2 * i + 1]), skip * y1);
                }
                umma::ld16(kYi + me + 16 * cg, v);
                umma::wait_ld();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    iv = fmaf(umma::lo_f(yy[i]), __uint_as_float(v[2 * i]), iv);
                    iv = fmaf(umma::hi_f(yy[i]), __uint_as_float(v[2 * i + 1]), iv);
                }
                s.i[cg][row] = iv;
                s.j[cg][row] = jv;
                sk = warp_sum(sk);
                if (lane == 0) {
                    s.skip[warp] = sk;
                    if (wi >= 2) s.dot[warp] = dot;
                }
                wait(&du, it);
                umma::fence_after();
                umma::ld16(kDu + me + 16 * cg, v);
                umma::wait_ld();
                uint32_t q[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    q[i] = umma::pack(o[2 * i] + __uint_as_float(v[2 * i]), o[2 * i + 1] + __uint_as_float(v[2 * i + 1]));
                sts16(su + at0, make_uint4(q[0], q[1], q[2], q[3]));  // du takes u's place
                sts16(su + at1, make_uint4(q[4], q[5], q[6], q[7]));
            }
            umma::fence_before();
            if (!tiles) {
                bar_sync(1, kWork * 32);
                const int r0 = tid / 8, c = tid % 8, n = min(8, p.rows - 8 * c);
                bf16 *uo = a.du + ((ck.start + r0) * z.H + p.h) * (int64_t)z.P + p.p0 + 8 * c;
                for (int i = 0; i < 2; ++i) {
                    if (r0 + 64 * i < len && n > 0) {
                        const uint4 v = lds16(su + umma::piece(r0 + 64 * i, c));
                        if (VEC && a.du_vec) {
                            *reinterpret_cast<uint4 *>(uo) = v;
                        } else {
                            for (int e = 0; e < n; ++e)
                                reinterpret_cast<unsigned short *>(uo)[e] = (unsigned short)(
                                    (e < 4 ? (e < 2 ? v.x : v.y) : (e < 6 ? v.z : v.w)) >> (16 * (e & 1)));
                        }
                    }
                    uo += 64 * (int64_t)z.H * z.P;
                }
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&epi[it & 1]);
        }
        // dG^T of the panels in two planes, as the next kernel's left operands
        char *tile = reinterpret_cast<char *>(a.dg + ((slot * z.G + g) * a.ranges + range) * (int64_t)(2 * kC * kC));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = 4 * ((wi + j) & 3) + cg;  // blocks before the diagonal are zeros
            char *to = tile + (c / 8) * umma::kPanel + umma::piece(row, c % 8);
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                hi[i] = umma::pack(dg[j][2 * i], dg[j][2 * i + 1]);
                lo[i] = umma::pack(dg[j][2 * i] - umma::lo_f(hi[i]), dg[j][2 * i + 1] - umma::hi_f(hi[i]));
            }
            *reinterpret_cast<uint4 *>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(to + 2 * umma::kPanel) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
    }
    umma::fence_before();
    __syncthreads();
    if (warp == 0) umma::dealloc(tmem_slot, 512);
}

constexpr int kBcStages = 3, kBcThreads = (kWork + 2) * 32;
template <int NPAD>
constexpr uint32_t bc_stage()
{
    return 2 * umma::kPanel + 2 * 64 * NPAD * 2 + 1024;
}
template <int NPAD>
constexpr int bc_smem()
{
    return 1024 + kBcStages * bc_stage<NPAD>();
}

// dB and dC of a chunk and group: one CTA over all its panels, so that the sums over the
// heads that share B and C stay in registers, 64 a thread.
template <int NPAD, bool VEC>
__global__ void __launch_bounds__(kBcThreads) head_bwd_bc_kernel(BwdArgs a, const __grid_constant__ CUtensorMap umap,
                                                                 const __grid_constant__ CUtensorMap ymap)
{
    constexpr int BP = NPAD / 64, COLS = NPAD / 4;
    constexpr uint32_t PLANE = 64 * NPAD * 2, STAGE = bc_stage<NPAD>();
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t landed[kBcStages], used[kBcStages], summed[2], taken[2], last_in, last_out;
    __shared__ uint32_t tmem_slot;
    const Dims &z = a.z;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int64_t slot = blockIdx.x;
    const int g = blockIdx.y, count = z.npan;
    const ChunkRef ck = find_chunk(z.cu, z.S, z.tok, kC, slot);
    if (ck.len == 0) return;
    const int len = ck.len;
    const uint32_t stages = (saddr(raw) + 1023) & ~1023u;
    if (tid == 0) {
        for (int i = 0; i < kBcStages; ++i) {
            mbar_init_n(&landed[i], 1);
            mbar_init_n(&used[i], kWork + 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init_n(&summed[i], 1);
            mbar_init_n(&taken[i], kWork);
        }
        mbar_init_n(&last_in, kWork);
        mbar_init_n(&last_out, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) umma::alloc(&tmem_slot, 512);
    umma::fence_before();
    __syncthreads();
    umma::fence_after();
    unsigned tries = umma::kTries;
    auto wait = [&](uint64_t *bar, uint32_t parity) { umma::wait(bar, parity & 1, tries, &g_bwd_status); };

    if (warp == kWork + 1) {  // loader
        for (int it = 0; it < count; ++it) {
            const int st = it % kBcStages;
            const uint32_t su = stages + st * STAGE, sm = su + 2 * umma::kPanel;
            const PanelRef p = panel_of(z, g, it);
            if (it >= kBcStages) wait(&used[st], it / kBcStages - 1);
            if (!VEC) {
                load_tile_warp<64>(su, a.u + ck.start * a.u_stride + (int64_t)p.h * z.P + p.p0, a.u_stride, len, p.rows, lane);
                load_tile_warp<64>(su + umma::kPanel, a.dy + (ck.start * z.H + p.h) * (int64_t)z.P + p.p0,
                                   (int64_t)z.H * z.P, len, p.rows, lane);
                fence_proxy_async();
            }
            __syncwarp();
            if (lane == 0) {
                uint64_t *bar = &landed[st];
                const int64_t mark = (slot * z.G * z.npan + g * z.npan + it) * 2 * kMark<NPAD>;
                const float *tb = a.tab + (slot * z.H + p.h) * kTab;
                mbar_expect_tx(bar, 2 * PLANE + 1024 + (VEC ? 2 * umma::kPanel : 0));
                if (VEC) {  // rows behind the sequence only reach rows of dB and dC that are not stored
                    umma::tma_3d(su, &umap, bar, p.p0, p.h, (int)ck.start);
                    umma::tma_3d(su + umma::kPanel, &ymap, bar, p.p0, p.h, (int)ck.start);
                }
                umma::bulk_load(sm, a.S0 + mark, PLANE, bar);
                umma::bulk_load(sm + PLANE, a.dS + mark, PLANE, bar);
                umma::bulk_load(sm + 2 * PLANE, tb + kTabEc, 512, bar);
                umma::bulk_load(sm + 2 * PLANE + 512, tb + kTabWf, 512, bar);
            }
            __syncwarp();
        }
    } else if (warp == kWork) {  // issuer
        if (umma::elect()) {
            const uint64_t u0 = umma::desc_k(stages, 0), y0 = umma::desc_k(stages + umma::kPanel, 0);
            const uint64_t s0 = umma::plain_mn(stages + 2 * umma::kPanel, 0, 64);
            int st = 0, round = 0;
            auto panel = [&](int it, auto buf) {
                constexpr uint32_t x = decltype(buf)::value * 256, y = x + 128;
                const uint32_t o = st * STAGE;
                wait(&landed[st], round);
                if (it >= 2) wait(&taken[decltype(buf)::value], (it >> 1) - 1);
                umma::fence_after();
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    umma::mma(x, umma::moved(y0, o + k * 32), umma::moved(s0, o + k * 256),
                              umma::idesc(NPAD, false, true), k > 0);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    umma::mma(y, umma::moved(u0, o + k * 32), umma::moved(s0, o + PLANE + k * 256),
                              umma::idesc(NPAD, false, true), k > 0);
                umma::commit(&summed[decltype(buf)::value]);
                umma::commit(&used[st]);
                if (++st == kBcStages) {
                    st = 0;
                    ++round;
                }
            };
            for (int it = 0; it < count; it += 2) {
                panel(it, std::integral_constant<uint32_t, 0>());
                if (it + 1 < count) panel(it + 1, std::integral_constant<uint32_t, 1>());
            }
            // dC += dG B, dB += dG^T C: both from the tile of dG^T
            const uint64_t cm = umma::desc_mn(stages, 0, umma::kPanel);
            const uint64_t bm = umma::desc_mn(stages + BP * umma::kPanel, 0, umma::kPanel);
            const uint64_t gk = umma::desc_k(stages + STAGE, 0), gm = umma::desc_mn(stages + STAGE, 0, umma::kPanel);
            for (int r = 0; r < 2 * a.ranges; ++r) {
                wait(&last_in, r);
                umma::fence_after();
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    umma::mma(0, umma::moved(gm, k * 2048), umma::moved(bm, k * 2048), umma::idesc(NPAD, true, true),
                              r + k > 0);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    umma::mma(128, umma::moved(gk, k / 4 * umma::kPanel + k % 4 * 32), umma::moved(cm, k * 2048),
                              umma::idesc(NPAD, false, true), r + k > 0);
                umma::commit(&last_out);
            }
        }
        __syncwarp();
    } else {
        const int wi = warp & 3, n0 = (warp >> 2) * COLS, row = wi * 32 + lane;
        const uint32_t me = (uint32_t)wi << 21;
        float dc[COLS], db[COLS];
#pragma unroll
        for (int i = 0; i < COLS; ++i) dc[i] = db[i] = 0.0f;
        auto add = [&](uint32_t col, float f, float (&acc)[COLS]) {
#pragma unroll
            for (int j = 0; j < COLS / 16; ++j) {
                uint32_t v[16];
                umma::ld16(col + me + n0 + 16 * j, v);
                umma::wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[16 * j + i] = fmaf(f, __uint_as_float(v[i]), acc[16 * j + i]);
            }
        };
        for (int it = 0; it < count; ++it) {
            const int st = it % kBcStages;
            const float *f = reinterpret_cast<const float *>(
                raw + (stages + st * STAGE + 2 * umma::kPanel + 2 * PLANE - saddr(raw)));
            wait(&landed[st], it / kBcStages);
            const float ec = f[row], wf = f[kC + row];
            __syncwarp();
            if (lane == 0) mbar_arrive(&used[st]);
            wait(&summed[it & 1], it >> 1);
            umma::fence_after();
            add((it & 1) * 256, ec, dc);
            add((it & 1) * 256 + 128, wf, db);
            umma::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&taken[it & 1]);
        }
        // every product is done, so the stages are free: C and B, then the tiles of dG^T
        load_tile<NPAD, 512, VEC>(stages, a.C + ck.start * a.bc_stride + (int64_t)g * z.N, a.bc_stride, len, z.N, tid);
        load_tile<NPAD, 512, VEC>(stages + BP * umma::kPanel, a.B + ck.start * a.bc_stride + (int64_t)g * z.N,
                                  a.bc_stride, len, z.N, tid);
        for (int r = 0; r < 2 * a.ranges; ++r) {
            const bf16 *tile = a.dg + ((slot * z.G + g) * a.ranges * 2 + r) * (int64_t)kC * kC;
            if (r > 0) wait(&last_out, r - 1);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                umma::cp16(stages + STAGE + (tid + 512 * i) * 16, tile + (tid + 512 * i) * 8, true);
            umma::cp_commit();
            umma::cp_wait<0>();
            fence_proxy_async();
            umma::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&last_in);
        }
        wait(&last_out, 2 * a.ranges - 1);
        umma::fence_after();
        add(0, 1.0f, dc);
        add(128, 1.0f, db);
        if (row < len) {
            const int64_t at = ((ck.start + row) * z.G + g) * (int64_t)z.N + n0;
            bf16 *pc = a.dC + at, *pb = a.dB + at;
            const bool v16 = z.N % 8 == 0 && reinterpret_cast<uintptr_t>(a.dC) % 16 == 0 &&
                             reinterpret_cast<uintptr_t>(a.dB) % 16 == 0;
#pragma unroll
            for (int j = 0; j < COLS / 8; ++j) {
                const int n = z.N - n0 - 8 * j;  // columns left
                if (v16 && n >= 8) {
                    *reinterpret_cast<uint4 *>(pc + 8 * j) =
                        make_uint4(umma::pack(dc[8 * j], dc[8 * j + 1]), umma::pack(dc[8 * j + 2], dc[8 * j + 3]),
                                   umma::pack(dc[8 * j + 4], dc[8 * j + 5]), umma::pack(dc[8 * j + 6], dc[8 * j + 7]));
                    *reinterpret_cast<uint4 *>(pb + 8 * j) =
                        make_uint4(umma::pack(db[8 * j], db[8 * j + 1]), umma::pack(db[8 * j + 2], db[8 * j + 3]),
                                   umma::pack(db[8 * j + 4], db[8 * j + 5]), umma::pack(db[8 * j + 6], db[8 * j + 7]));
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (e < n) {
                            pc[8 * j + e] = __float2bfloat16_rn(dc[8 * j + e]);
                            pb[8 * j + e] = __float2bfloat16_rn(db[8 * j + e]);
                        }
                }
            }
        }
    }
    umma::fence_before();
    __syncthreads();
    if (warp == 0) umma::dealloc(tmem_slot, 512);
}

template <int NPAD, bool VEC>
cudaError_t chunks(const BwdArgs &a, int64_t slots, cudaStream_t st, int *launches)
{
    CUtensorMap umap{}, ymap{}, dumap{};
    const int64_t row = (int64_t)a.z.H * a.z.P;
    if (VEC && (!umma::encode_3d(&umap, a.u, a.z.tok, a.z.H, a.z.P, a.u_stride) ||
                !umma::encode_3d(&ymap, a.dy, a.z.tok, a.z.H, a.z.P, row) ||
                (a.du_vec && !umma::encode_3d(&dumap, a.du, a.z.tok, a.z.H, a.z.P, row))))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(head_bwd_kernel<NPAD, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         bwd_smem<NPAD>());
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(head_bwd_bc_kernel<NPAD, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 bc_smem<NPAD>());
    if (e != cudaSuccess) return e;
    head_bwd_kernel<NPAD, VEC><<<dim3((unsigned)slots, (unsigned)(a.z.G * a.ranges)), kBwdThreads, bwd_smem<NPAD>(), st>>>(
        a, umap, ymap, dumap);
    ++*launches;
    if (e = cudaGetLastError(); e != cudaSuccess) return e;
    head_bwd_bc_kernel<NPAD, VEC><<<dim3((unsigned)slots, (unsigned)a.z.G), kBcThreads, bc_smem<NPAD>(), st>>>(a, umap, ymap);
    ++*launches;
    return cudaGetLastError();
}

struct BwdLayout {
    Layout walk;
    size_t dS, dg, part, total;
    int per, ranges;
    Plan plan;
};

BwdLayout bwd_layout(const Dims &z, bool known)
{
    BwdLayout l;
    l.plan = plan_of(z, known);
    l.walk = layout_of(z, 2, l.plan);
    const int64_t slots = head_slots(z.tok, z.S, kC);
    const size_t marks = l.walk.order - l.walk.marks;
    // whole heads per CTA; G^T and the rounded dG^T are shared by a CTA's panels: a start and
    // an end worth about two panels
    l.per = (int)units_of_cta(slots * z.G, z.H / z.G, 2.0 / z.np) * z.np;
    l.ranges = (z.npan + l.per - 1) / l.per;
    l.dS = l.walk.total;
    l.dg = l.dS + marks;
    l.part = l.dg + up256((size_t)slots * z.G * l.ranges * kC * kC * 4);
    l.total = l.part + up256((size_t)slots * z.H * 3 * 4);
    return l;
}

}  // namespace

size_t backward_bytes(const Dims &z)
{
    const size_t dense = bwd_layout(z, true).total, packed = bwd_layout(z, false).total;
    return dense > packed ? dense : packed;
}

cudaError_t launch_backward(const HeadScanArgs &a, cudaStream_t st, int *launches)
{
    const Dims z = dims_of(a);
    const BwdLayout l = bwd_layout(z, lengths_known(z));
    char *ws = static_cast<char *>(a.workspace);
    float *tab = reinterpret_cast<float *>(ws + l.walk.tab);
    bf16 *S0 = reinterpret_cast<bf16 *>(ws + l.walk.marks), *dS = reinterpret_cast<bf16 *>(ws + l.dS);
    float *seg = reinterpret_cast<float *>(ws + l.walk.seg), *segdec = reinterpret_cast<float *>(ws + l.walk.segdec);
    int64_t *span = reinterpret_cast<int64_t *>(ws + l.walk.span);
    int32_t *order = a.cu && a.S > 1 ? reinterpret_cast<int32_t *>(ws + l.walk.order) : nullptr;
    float *part = reinterpret_cast<float *>(ws + l.part);
    if (cudaError_t e = launch_tables(a, z, tab, true, l.plan, span, st, launches); e != cudaSuccess) return e;
    const int64_t row = a.H * a.P;
    const bool bc_vec = vec16(a.B, a.bc_stride, a.N) && vec16(a.C, a.bc_stride, a.N);
    const bool vec = bc_vec && vec16(a.u, a.u_stride, a.P) && vec16(a.dy, row, a.P);
    const bf16 *u = static_cast<const bf16 *>(a.u), *dy = static_cast<const bf16 *>(a.dy);
    const bf16 *B = static_cast<const bf16 *>(a.B), *C = static_cast<const bf16 *>(a.C);
    StateArgs s{z, u, a.u_stride, B, a.bc_stride, tab, a.h0, nullptr, S0, seg, segdec, order, span};
    if (cudaError_t e = launch_states(s, false, 2, l.plan, vec, st, launches); e != cudaSuccess) return e;
    StateArgs r{z, dy, row, C, a.bc_stride, tab, a.dh_final, a.dh0, dS, seg, segdec, order, span};
    if (cudaError_t e = launch_states(r, true, 2, l.plan, vec, st, launches); e != cudaSuccess) return e;
    const int64_t slots = head_slots(z.tok, z.S, kC);
    BwdArgs b{z, u, dy, B, C, static_cast<const bf16 *>(a.delta), a.u_stride, a.bc_stride, a.delta_stride,
              a.A, a.Dskip, a.dt_bias, a.delta_softplus, tab, S0, dS, static_cast<bf16 *>(a.du),
              static_cast<bf16 *>(a.ddelta), static_cast<bf16 *>(a.dB), static_cast<bf16 *>(a.dC),
              reinterpret_cast<bf16 *>(ws + l.dg), part, l.per, l.ranges, vec16(a.du, row, a.P)};
    if (a.tok > 0) {
        cudaError_t e;
        if (z.N > 64) e = vec ? chunks<128, true>(b, slots, st, launches) : chunks<128, false>(b, slots, st, launches);
        else e = vec ? chunks<64, true>(b, slots, st, launches) : chunks<64, false>(b, slots, st, launches);
        if (e != cudaSuccess) return e;
    }
    return launch_head_reduce(part, a.tok > 0 ? slots : 0, z.H, a.dA, a.ddt_bias, a.dDskip, st, launches);
}

}  // namespace hm

int read_head_bwd_status(bool clear)
{
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, hm::g_bwd_status, sizeof(v)) != cudaSuccess) return -1;
    if (clear && v) {
        const int zero = 0;
        if (cudaMemcpyToSymbol(hm::g_bwd_status, &zero, sizeof(zero)) != cudaSuccess) return -1;
    }
    return v;
}

}  // namespace ssm
