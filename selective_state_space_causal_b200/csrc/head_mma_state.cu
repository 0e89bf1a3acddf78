// head_mma_state.cu -- chunk tables and chunk states of the bf16 scan with one decay
// per head (tensor cores).
//
// State of a chunk's end from its start:  S' = e^{cQ} S + sum_t w_t x_t b_t^T, with
//   forward  x = u, b = B, w_t = d_t e^{cQ - c_t};   reverse  x = dy, b = C, w_t = e^{c_t}.
// The sum over a chunk is one 128 x N x 128 product for two panels: D[p, n], A = (w x)^T
// with rows p (both panels), B = b. w x is split into three bf16 planes (24 bits), so the
// state keeps fp32 accuracy; b is bf16 as given. The products of different chunks are
// independent: only S' = e S + delta runs chunk after chunk, in registers, while the
// next products are under way.
//
// Measured on a B200, 80 heads of 64 x 128 in one group: 65536 tokens in 43 sequences, one
// plane of marks, 369 us (1.34 GB of x, marks and tables: 3.6 TB/s, 56% of a copy's rate;
// 24% of the matrix rate for the one product the mathematics needs in three planes);
// 32768 tokens in 21 sequences, two planes, 258 us forward and 283 us reverse (1.06 GB, 4.1
// TB/s). Bound by the converters' latency (below), not by memory: without the marks'
// stores the last two would take 233 and 257 us, with a split that costs nothing 263 and
// 278. Marks sent by bulk copies instead of the threads' own stores: 5% slower.
#include <type_traits>

#include "head_mma.cuh"

namespace ssm {

cudaError_t launch_seq_order(const int32_t *cu, int64_t S, int64_t tok, int32_t *order, cudaStream_t stream);

namespace hm {

__device__ int g_status;

namespace {

constexpr int kTabHeads = 8;

// 2^x with the argument's rounding to fp32 made good: at x = -20 it alone is 1e-6.
__device__ __forceinline__ float exp2_of(double x)
{
    const float h = (float)x, r = ex2_approx(h);
    return fmaf(r, (float)(x - (double)h) * 0.6931471806f, r);
}

// One block per (chunk slot, kTabHeads heads), a warp per head. Sums and their differences are 64-bit. Bound by
// the latency of a block's few steps and its special functions: 58 us for 65536 tokens of 80
// heads (0.2 GB), 9 us for 16384 of 24 (18 with 32 heads a block).
__global__ void __launch_bounds__(256) head_table_kernel(Dims z, const bf16 *delta, int64_t stride,
                                                         const float *A, const float *bias,
                                                         int softplus, bool backward, float *tab,
                                                         Plan plan, int64_t *span)
{
    __shared__ float sd[kC][kTabHeads + 1];
    const int64_t slot = blockIdx.x;
    const int h0 = blockIdx.y * kTabHeads, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    if (plan.mode == Plan::kAsk && blockIdx.x + blockIdx.y == 0) {
        // the walks are cut only if the longest sequence would outlast two passes of pieces
        __shared__ int longest;
        if (tid == 0) longest = 0;
        __syncthreads();
        int most = 0;
        for (int64_t s = tid; s < z.S; s += 256) {
            int64_t lo, hi;
            seq_bounds(z.cu, z.S, z.tok, s, lo, hi);
            most = max(most, (int)((hi - lo + kC - 1) / kC));
        }
        atomicMax(&longest, most);
        __syncthreads();
        if (tid == 0) *span = longest > plan.limit ? plan.span : kNoSpan;
    }
    const ChunkRef ck = find_chunk(z.cu, z.S, z.tok, kC, slot);
    if (ck.len == 0) return;
    const int hl = tid % kTabHeads, h = h0 + hl;
    const float bs = bias && h < z.H ? bias[h] : 0.0f;
#pragma unroll
    for (int t = tid / kTabHeads; t < kC; t += 256 / kTabHeads) {
        float v = 0.0f;
        if (t < ck.len && h < z.H) v = head_step(to_f32(delta[(ck.start + t) * stride + h]) + bs, softplus);
        sd[t][hl] = v;
    }
    __syncthreads();
    for (int i = warp; i < kTabHeads && h0 + i < z.H; i += 8) {
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
        const double last = __shfl_sync(0xffffffffu, pre, 31);
        const double r1 = __shfl_sync(0xffffffffu, pre, 7), r2 = __shfl_sync(0xffffffffu, pre, 15),
                     r3 = __shfl_sync(0xffffffffu, pre, 23);
        pre -= sum;
        const int blk = lane / 8;
        const double r = blk == 0 ? 0.0 : blk == 1 ? r1 : blk == 2 ? r2 : r3;
        float lv[4], ll[4], ev[4], wv[4], wn[4], el[4], c1[4], c2[4], c3[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const double c = pre + run[j];
            lv[j] = (float)(c - r);
            ev[j] = exp2_of(c);
            wn[j] = exp2_of(last - c);
            wv[j] = dv[j] * wn[j];
            if (backward) {
                ll[j] = (float)(c - r - (double)lv[j]);
                el[j] = exp2_of(c - r);
                c1[j] = exp2_of(r1 - c);
                c2[j] = exp2_of(r2 - c);
                c3[j] = exp2_of(r3 - c);
            } else {  // factors of M, which is rounded to bf16
                c1[j] = dv[j] * ex2_approx((float)(r1 - c));
                c2[j] = dv[j] * ex2_approx((float)(r2 - c));
                c3[j] = dv[j] * ex2_approx((float)(r3 - c));
            }
        }
        float *q = tab + (slot * z.H + h0 + i) * kTab;
        auto put = [&](int at, const float (&v)[4]) {
            *reinterpret_cast<float4 *>(q + at + 4 * lane) = make_float4(v[0], v[1], v[2], v[3]);
        };
        put(kTabD, dv);
        put(kTabL, lv);
        put(kTabEc, ev);
        put(kTabWf, wv);
        if (backward) {
            put(kTabWn, wn);
            put(kTabEl, el);
            put(kTabLl, ll);
        }
        if (blk < 1) put(col_at(1), c1);
        if (blk < 2) put(col_at(2), c2);
        if (blk < 3) put(col_at(3), c3);
    }
}

// Two neighbouring tokens' w x as three pairs of bf16 that add up to it exactly: each
// takes the top 8 bits that are left (24 in all), by truncation.
__device__ __forceinline__ void split3(uint32_t x, f32x2 w, uint32_t &hi, uint32_t &mid, uint32_t &lo)
{
    const f32x2 minus = pk2(-1.0f, -1.0f);
    f32x2 v = mul2(pk2(umma::lo_f(x), umma::hi_f(x)), w);
    float v0, v1;
    upk2(v, v0, v1);
    hi = __byte_perm(__float_as_uint(v0), __float_as_uint(v1), 0x7632);
    v = fma2(pk2(umma::hi_f(__float_as_uint(v0)), umma::hi_f(__float_as_uint(v1))), minus, v);
    upk2(v, v0, v1);
    mid = __byte_perm(__float_as_uint(v0), __float_as_uint(v1), 0x7632);
    v = fma2(pk2(umma::hi_f(__float_as_uint(v0)), umma::hi_f(__float_as_uint(v1))), minus, v);
    upk2(v, v0, v1);
    lo = __byte_perm(__float_as_uint(v0), __float_as_uint(v1), 0x7632);
}

constexpr int kGroups = 3, kConvWarps = 4 * kGroups, kStateWarps = 16;
constexpr int kIssuer = kConvWarps + kStateWarps, kLoader = kIssuer + 1;
constexpr int kStateThreads = (kLoader + 1) * 32;
constexpr int kStages = 3;

// A stage: two x panels, the b tile, weights of the two panels' heads.
template <int NPAD>
constexpr uint32_t state_stage()
{
    return (2 + NPAD / 64) * umma::kPanel + 1024;
}
template <int NPAD>
constexpr int state_smem()
{
    return 1024 + kStages * state_stage<NPAD>();
}

// The segment behind a slot; whole sequences need no search.
__device__ __forceinline__ ChunkRef segment_of(const Dims &z, int64_t span, int64_t slot)
{
    if (span <= z.tok) return find_chunk(z.cu, z.S, z.tok, span, slot);
    ChunkRef r;
    int64_t lo, hi;
    r.seq = (int)min(slot, z.S - 1);
    r.k = (int)(slot - r.seq);
    seq_bounds(z.cu, z.S, z.tok, r.seq, lo, hi);
    r.start = lo;
    r.len = r.k == 0 ? (int)(hi - lo) : 0;
    r.last = true;
    return r;
}

// One CTA has two panels of one group and walks a segment's chunks. The warps have
// roles, so that loads, conversion, matrix instructions and state updates of
// neighbouring chunks run at the same time (with all warps in step, each phase's
// latency was exposed: 5500 clocks a chunk against 1536 of matrix instructions):
//   loader     copies x, b and weights of the next chunks into one of three stages
//   converters make w x as three planes in tensor memory, transposed on the way, 32
//              tokens at a time, three groups of four warps in turn: 2000 clocks a step,
//              so 3000 a chunk; a fourth group does not fit in the registers. (Planes in
//              shared memory cost it 384 KB of traffic a chunk against 192 KB.)
//   issuer     multiplies into one of two tensor-memory buffers
//   state      keep the state in registers, write it before each chunk, add the product
// A walk may be cut into segments that run side by side, in two passes: `first` makes every
// segment's end state from zero (but the walk's last one's) and a copy of the initial
// state, then each segment starts from that and the ends before it, joined in order: S =
// decay S + end.
template <int NPAD, bool REV, int PLANES, bool VEC>
__global__ void __launch_bounds__(kStateThreads) head_state_kernel(StateArgs a, const __grid_constant__ CUtensorMap xmap,
                                                                   const __grid_constant__ CUtensorMap bmap)
{
    constexpr int COLS = NPAD / 4;  // state columns of a thread
    constexpr int BP = NPAD / 64;   // panels of a b tile
    constexpr uint32_t STAGE = state_stage<NPAD>();
    extern __shared__ uint8_t raw[];
    // landed / used: a stage; made / eaten: 32 tokens' planes; summed / taken: a product
    __shared__ uint64_t landed[kStages], used[kStages], made[4], eaten[4], summed[2], taken[2];
    __shared__ uint32_t tmem_slot;
    const Dims &z = a.z;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    // whole sequences go longest first: a long one started last would run almost alone
    const int64_t slot = a.order ? a.order[blockIdx.y] : blockIdx.y, span = a.asked ? *a.asked : a.span;
    const int per_group = (z.npan + 1) / 2;
    const int g = blockIdx.x / per_group, pan0 = blockIdx.x % per_group * 2;
    const int np = min(2, z.npan - pan0);  // panels of this CTA
    const ChunkRef sg = segment_of(z, span, slot);
    if (sg.len == 0 && sg.k != 0) return;
    const int nchunk = (sg.len + kC - 1) / kC;
    int64_t lo, hi;
    seq_bounds(z.cu, z.S, z.tok, sg.seq, lo, hi);
    const int64_t first = lo / kC + sg.seq + (int64_t)sg.k * (span / kC);  // first chunk's slot
    const int nseg = max(1, (int)((hi - lo + span - 1) / span));
    const int before = REV ? nseg - 1 - sg.k : sg.k;  // segments walked before this one
    if (a.first && before == nseg - 1) {
        // This segment's end is not asked for: its place keeps the walk's initial state,
        // whose own memory `final_` may be, for all segments of the second pass.
        const int entries = 64 * (NPAD / 4);
        for (int i = tid; nseg > 1 && a.init && i < np * entries; i += kStateThreads) {
            const int q = i / entries, n = i % entries / 64 * 4, p = i % 64;
            const PanelRef sp = panel_of(z, g, pan0 + q);
            const float *src = a.init + (((int64_t)sg.seq * z.H + sp.h) * z.P + sp.p0 + p) * z.N;
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = p < sp.rows && n + e < z.N ? src[n + e] : 0.0f;
            reinterpret_cast<float4 *>(a.seg + (slot * z.G * z.npan + g * z.npan + pan0) * 64 * NPAD)[i] =
                make_float4(v[0], v[1], v[2], v[3]);
        }
        return;
    }

    const uint32_t stages = (saddr(raw) + 1023) & ~1023u;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init_n(&landed[i], 1);
            mbar_init_n(&used[i], 4 * 4 + 1);  // four warps for each 32 tokens, and the products
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init_n(&made[i], 4);
            mbar_init_n(&eaten[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init_n(&summed[i], 1);
            mbar_init_n(&taken[i], kStateWarps);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) umma::alloc(&tmem_slot, 512);
    umma::fence_before();
    __syncthreads();
    umma::fence_after();
    constexpr uint32_t tm = umma::kWhole, planes = tm + 256;  // two products, then 4 x 3 planes of 16 columns
    unsigned tries = umma::kTries;
    auto chunk_at = [&](int kk) { return REV ? nchunk - 1 - kk : kk; };
    auto len_of = [&](int k) { return min(kC, sg.len - k * kC); };
    auto wait = [&](uint64_t *bar, uint32_t parity) { umma::wait(bar, parity & 1, tries, &g_status); };

    if (warp == kLoader) {
        const PanelRef q0 = panel_of(z, g, pan0), q1 = panel_of(z, g, pan0 + np - 1);
        for (int kk = 0; kk < nchunk; ++kk) {
            const int k = chunk_at(kk), sg_i = kk % kStages;
            const int64_t t0 = sg.start + (int64_t)k * kC;
            const uint32_t sx = stages + sg_i * STAGE, sb = sx + 2 * umma::kPanel, sw = sb + BP * umma::kPanel;
            uint64_t *bar = &landed[sg_i];
            if (kk >= kStages) wait(&used[sg_i], kk / kStages - 1);
            if (!VEC) {
                const int len = len_of(k);
                load_tile_warp<64>(sx, a.x + t0 * a.x_stride + (int64_t)q0.h * z.P + q0.p0, a.x_stride, len, q0.rows, lane);
                if (np > 1)
                    load_tile_warp<64>(sx + umma::kPanel, a.x + t0 * a.x_stride + (int64_t)q1.h * z.P + q1.p0,
                                       a.x_stride, len, q1.rows, lane);
                load_tile_warp<NPAD>(sb, a.b + t0 * a.b_stride + (int64_t)g * z.N, a.b_stride, len, z.N, lane);
                fence_proxy_async();
            }
            __syncwarp();
            if (umma::elect()) {
                const float *w0 = a.tab + ((first + k) * z.H + q0.h) * kTab + (REV ? kTabEc : kTabWf);
                const float *w1 = a.tab + ((first + k) * z.H + q1.h) * kTab + (REV ? kTabEc : kTabWf);
                mbar_expect_tx(bar, 1024 + (VEC ? (np + BP) * umma::kPanel : 0));
                umma::bulk_load(sw, w0, 512, bar);
                umma::bulk_load(sw + 512, w1, 512, bar);
                if (VEC) {
                    umma::tma_3d(sx, &xmap, bar, q0.p0, q0.h, (int)t0);
                    if (np > 1) umma::tma_3d(sx + umma::kPanel, &xmap, bar, q1.p0, q1.h, (int)t0);
                    for (int i = 0; i < BP; ++i) umma::tma_3d(sb + i * umma::kPanel, &bmap, bar, 64 * i, g, (int)t0);
                }
            }
            __syncwarp();
        }
    } else if (warp == kIssuer) {
        if (umma::elect()) {
            const uint64_t b0 = umma::desc_mn(stages + 2 * umma::kPanel, 0, umma::kPanel);
            int st = 0, round = 0;
            auto chunk = [&](int kk, auto buf) {
                constexpr uint32_t d = tm + decltype(buf)::value * NPAD;
                const uint64_t b = umma::moved(b0, st * STAGE);
                wait(&landed[st], round);
                if (kk >= 2) wait(&taken[decltype(buf)::value], (kk >> 1) - 1);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    wait(&made[q], kk);
                    umma::fence_after();
#pragma unroll
                    for (int s = 0; s < 3; ++s)
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            umma::mma_ta(d, planes + (3 * q + s) * 16 + 8 * k, umma::moved(b, (2 * q + k) * 2048),
                                         umma::idesc(NPAD, false, true), q + s + k > 0);
                    umma::commit(&eaten[q]);
                }
                umma::commit(&summed[decltype(buf)::value]);
                umma::commit(&used[st]);
                if (++st == kStages) {
                    st = 0;
                    ++round;
                }
            };
            for (int kk = 0; kk < nchunk; kk += 2) {
                chunk(kk, std::integral_constant<uint32_t, 0>());
                if (kk + 1 < nchunk) chunk(kk + 1, std::integral_constant<uint32_t, 1>());
            }
        }
        __syncwarp();
    } else if (warp < kConvWarps) {
        // 32 tokens at a time; this warp has state rows 32 (warp % 4) .. of the two panels
        const int grp = warp / 4, w4 = warp % 4, cp = w4 / 2;
        const bool has_x = cp < np;  // without a second panel its half of the product is never read
        const uint32_t rows = (uint32_t)w4 << 21;
        // the tiles of ldsm_t: tokens 0-7, rows 0-7; the same tokens, rows 8-15; tokens 8-15
        const int tt = lane % 8 + (lane / 16) * 8, pc = (w4 & 1) * 4 + (lane / 8) % 2;
        for (int j = grp; j < 4 * nchunk; j += kGroups) {
            const int kk = j / 4, q = j % 4, st = kk % kStages;
            const int len = len_of(chunk_at(kk)) - 32 * q;  // tokens left from here
            const uint32_t sx = stages + st * STAGE, sb = sx + 2 * umma::kPanel;
            const float2 *w = reinterpret_cast<const float2 *>(
                raw + (sb + BP * umma::kPanel + cp * 512 + q * 128 - saddr(raw))) + lane % 4;
            wait(&landed[st], kk / kStages);
            // loads first: a wait takes some 250 clocks even if there is nothing to wait for
            uint32_t x[2][8], v[3][8];
#pragma unroll
            for (int ph = 0; ph < 2; ++ph)  // 16 state rows
#pragma unroll
                for (int th = 0; th < 2; ++th)  // 16 tokens
                    umma::ldsm_t(sx + cp * umma::kPanel + umma::piece(32 * q + 16 * th + tt, pc + 2 * ph),
                                 x[ph][4 * th], x[ph][4 * th + 1], x[ph][4 * th + 2], x[ph][4 * th + 3]);
            f32x2 wt[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 v = w[4 * i];  // tokens 8 i + 2 (lane % 4) and + 1
                wt[i] = pk2(v.x, v.y);
            }
            if (len < 32) {  // tokens behind the sequence: b's rows become zeros (x's do below)
                for (int i = tid % 128; i < 32 * BP * 8; i += 128) {
                    const int r = i / (BP * 8), c = i % (BP * 8);
                    if (r >= len)
                        sts16(sb + (c / 8) * umma::kPanel + umma::piece(32 * q + r, c % 8), make_uint4(0, 0, 0, 0));
                }
                fence_proxy_async();
            }
            if (kk > 0) wait(&eaten[q], kk - 1);
            umma::fence_after();
#pragma unroll
            for (int ph = 0; ph < 2 && has_x; ++ph) {
                if (len < 32) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int t = 8 * (i / 2) + 2 * (lane % 4);
                        const uint32_t keep = (t < len ? 0xFFFFu : 0u) | (t + 1 < len ? 0xFFFF0000u : 0u);
                        x[ph][i] &= keep;
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) split3(x[ph][i], wt[i / 2], v[0][i], v[1][i], v[2][i]);
#pragma unroll
                for (int s = 0; s < 3; ++s)
                    umma::st_tiles(planes + rows + ((uint32_t)ph << 20) + (3 * q + s) * 16, v[s]);
            }
            umma::wait_st();
            umma::fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&made[q]);
                mbar_arrive(&used[st]);
            }
        }
    } else {
        // row sr of the two panels, columns n0 ..
        const int sw = warp - kConvWarps, sr = (sw & 3) * 32 + lane, n0 = (sw / 4) * COLS;
        const int si = pan0 + sr / 64, p = sr % 64;
        const bool has_s = sr / 64 < np;
        const PanelRef sp = panel_of(z, g, min(si, z.npan - 1));
        const bool row_in = has_s && p < sp.rows;
        const int64_t dir = REV ? -1 : 1, c0 = first + chunk_at(0);
        const float *dec = a.tab + (c0 * z.H + sp.h) * kTab + kTabEc + kC - 1;
        const int64_t dec_step = dir * z.H * kTab;

        auto seg_at = [&](int64_t sl) {
            return reinterpret_cast<float4 *>(a.seg + (sl * z.G * z.npan + g * z.npan + si) * 64 * NPAD) + (n0 / 4) * 64 + p;
        };
        float st[COLS];
        {
            const float *src = nullptr;
            if (!a.first && a.init && row_in && nseg == 1)
                src = a.init + (((int64_t)sg.seq * z.H + sp.h) * z.P + sp.p0 + p) * z.N;
#pragma unroll
            for (int i = 0; i < COLS; ++i) st[i] = src && n0 + i < z.N ? src[n0 + i] : 0.0f;
            if (!a.first && a.init && has_s && nseg > 1) {
                const float4 *q = seg_at(slot - sg.k + (REV ? 0 : nseg - 1));
#pragma unroll
                for (int i = 0; i < COLS / 4; ++i) {
                    const float4 v = q[i * 64];
                    st[4 * i] = v.x; st[4 * i + 1] = v.y; st[4 * i + 2] = v.z; st[4 * i + 3] = v.w;
                }
            }
            for (int j = 0; j < (a.first ? 0 : before) && has_s; ++j) {
                const int64_t other = slot - sg.k + (REV ? nseg - 1 - j : j);
                const float4 *q = seg_at(other);
                const float d = a.segdec[other * z.H + sp.h];
#pragma unroll
                for (int i = 0; i < COLS / 4; ++i) {
                    const float4 v = q[i * 64];
                    st[4 * i] = fmaf(d, st[4 * i], v.x);
                    st[4 * i + 1] = fmaf(d, st[4 * i + 1], v.y);
                    st[4 * i + 2] = fmaf(d, st[4 * i + 2], v.z);
                    st[4 * i + 3] = fmaf(d, st[4 * i + 3], v.w);
                }
            }
        }
        uint4 *mk = reinterpret_cast<uint4 *>(
                        a.marks + (c0 * z.G * z.npan + g * z.npan + si) * PLANES * kMark<NPAD>) + (n0 / 8) * 64 + p;
        const int64_t mk_step = dir * z.G * z.npan * PLANES * kMark<NPAD> / 8;
        const bool marking = !a.first && has_s;
        float e = nchunk > 0 ? *dec : 1.0f;
        for (int kk = 0; kk < nchunk; ++kk) {
            if (marking) {
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
                        mk[(s * (NPAD / 8) + j) * 64] = make_uint4(w[s][0], w[s][1], w[s][2], w[s][3]);
                }
                mk += mk_step;
            }
            const float now = e;
            if (kk + 1 < nchunk) {
                dec += dec_step;
                e = *dec;
            }
            wait(&summed[kk & 1], kk >> 1);
            umma::fence_after();
#pragma unroll
            for (int j = 0; j < COLS / 16 && has_s; ++j) {
                uint32_t v[16];
                umma::ld16(umma::lanes(tm + (kk & 1) * NPAD + n0 + 16 * j, warp), v);
                umma::wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    st[16 * j + i] = fmaf(now, st[16 * j + i], __uint_as_float(v[i]));
            }
            umma::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&taken[kk & 1]);
        }
        if (!a.first && before == nseg - 1 && a.final_ && row_in) {
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
                    for (int x = 0; x < 4; ++x)
                        if (n + x < z.N) dst[n + x] = st[4 * i + x];
            }
        }
        if (a.first && has_s) {
            float4 *q = seg_at(slot);
#pragma unroll
            for (int i = 0; i < COLS / 4; ++i)
                q[i * 64] = make_float4(st[4 * i], st[4 * i + 1], st[4 * i + 2], st[4 * i + 3]);
            if (n0 == 0 && p == 0) {
                float t = 1.0f;
                for (int k = 0; k < nchunk; ++k) t *= a.tab[((first + k) * z.H + sp.h) * kTab + kTabEc + kC - 1];
                a.segdec[slot * z.H + sp.h] = t;
            }
        }
    }
    umma::fence_before();
    __syncthreads();
    if (warp == 0) umma::dealloc(tm, 512);
}

template <int NPAD, bool REV, int PLANES, bool VEC>
cudaError_t launch_walk(const StateArgs &a, cudaStream_t st, int *launches)
{
    constexpr int bytes = state_smem<NPAD>();
    if (cudaError_t e = cudaFuncSetAttribute(head_state_kernel<NPAD, REV, PLANES, VEC>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        e != cudaSuccess)
        return e;
    const dim3 grid((unsigned)(a.z.G * ((a.z.npan + 1) / 2)),
                    (unsigned)head_slots(a.z.tok, a.z.S, a.span));
    CUtensorMap xmap{}, bmap{};
    if (VEC && a.z.tok > 0 &&
        (!umma::encode_3d(&xmap, a.x, a.z.tok, a.z.H, a.z.P, a.x_stride) ||
         !umma::encode_3d(&bmap, a.b, a.z.tok, a.z.G, a.z.N, a.b_stride)))
        return cudaErrorInvalidValue;
    head_state_kernel<NPAD, REV, PLANES, VEC><<<grid, kStateThreads, bytes, st>>>(a, xmap, bmap);
    ++*launches;
    return cudaGetLastError();
}

template <int NPAD, bool REV, int PLANES>
cudaError_t states(StateArgs a, const Plan &plan, bool vec, cudaStream_t st, int *launches)
{
    auto walk = [&](bool first) {
        a.first = first;
        return vec ? launch_walk<NPAD, REV, PLANES, true>(a, st, launches)
                   : launch_walk<NPAD, REV, PLANES, false>(a, st, launches);
    };
    a.span = plan.mode == Plan::kWhole ? kNoSpan : plan.span;
    if (plan.mode != Plan::kAsk) a.asked = nullptr;
    if (plan.mode != Plan::kWhole) {
        a.order = nullptr;
        if (cudaError_t e = walk(true); e != cudaSuccess) return e;
    } else if (a.order) {
        if (cudaError_t e = launch_seq_order(a.z.cu, a.z.S, a.z.tok, a.order, st); e != cudaSuccess) return e;
        ++*launches;
    }
    return walk(false);
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

// A cut walk reads its inputs twice, so with W chunks for every SM it takes about 2 W, one
// that is not takes as long as the longest sequence. 8 x 12 walks (H = 24) of 134 chunks,
// measured: the longest 54, 124 us whole and 85 us cut at 11; all of 16, 45 us whole and
// 8 us more for the first pass that finds nothing to do. Whole forward calls in us, heads of
// 64 x 128, whole / cut, the rule's choice second to none by more than 4%:
//   24 heads  one sequence of 512 43 / 47, 1024 51 / 49, 2048 68 / 51, 8192 160 / 74, 65536 1053
//             / 377; four of 4096 125 / 111; 9000 among 3 shorter ones 201 / 150
//   32 heads  four of 4096 139 / 160;   48 heads  two of 8192 215 / 180 to 203
//   64 heads  one of 8192 191 / 145, two 238 / 256;   128 heads in 8 groups  one of 8192 252 / 258
//   80 heads  one of 32768 707 / 571, 30000 among 3 shorter ones 694 / 569
// Where the lengths are only known on the device, the table kernel decides.
Plan plan_of(const Dims &z, bool known)
{
    Plan p;
    const int64_t walks = z.G * ((z.npan + 1) / 2);  // of one sequence
    const int64_t longest = (z.tok / z.S + kC - 1) / kC;
    const int64_t chunks = known ? longest * z.S : z.tok / kC + z.S;
    const int64_t load = (chunks * walks + 147) / 148;
    p.limit = (int)(load * 11 / 5 + 4);
    p.span = (load < 4 ? 4 : load) * kC;
    if (known) p.mode = longest > p.limit ? Plan::kCut : Plan::kWhole;
    // with two walks an SM the longest sequence first does as well; and no sequence is
    // longer than all chunks together
    else p.mode = walks * z.S >= 2 * 148 || z.tok / kC + 1 <= p.limit ? Plan::kWhole : Plan::kAsk;
    return p;
}

cudaError_t launch_tables(const HeadScanArgs &a, const Dims &z, float *tab, bool backward,
                          const Plan &plan, int64_t *span, cudaStream_t stream, int *launches)
{
    const dim3 grid((unsigned)head_slots(z.tok, z.S, kC), (unsigned)((z.H + kTabHeads - 1) / kTabHeads));
    head_table_kernel<<<grid, 256, 0, stream>>>(z, static_cast<const bf16 *>(a.delta), a.delta_stride,
                                                a.A, a.dt_bias, a.delta_softplus, backward, tab,
                                                plan, span);
    ++*launches;
    return cudaGetLastError();
}

cudaError_t launch_states(const StateArgs &a, bool rev, int planes, const Plan &plan, bool vec,
                          cudaStream_t st, int *launches)
{
    const bool wide = a.z.N > 64;
    if (planes == 1)
        return wide ? states<128, false, 1>(a, plan, vec, st, launches)
                    : states<64, false, 1>(a, plan, vec, st, launches);
    if (rev) return wide ? states<128, true, 2>(a, plan, vec, st, launches)
                         : states<64, true, 2>(a, plan, vec, st, launches);
    return wide ? states<128, false, 2>(a, plan, vec, st, launches)
                : states<64, false, 2>(a, plan, vec, st, launches);
}

Layout layout_of(const Dims &z, int planes, const Plan &plan)
{
    const int64_t slots = head_slots(z.tok, z.S, kC);
    const int64_t segs = plan.mode == Plan::kWhole ? 0 : head_slots(z.tok, z.S, plan.span);
    const int npad = z.N > 64 ? 128 : 64;
    const size_t panel = (size_t)z.G * z.npan * 64 * npad;
    Layout l;
    l.tab = 0;
    l.seg = l.tab + up256((size_t)slots * z.H * kTab * 4);
    l.segdec = l.seg + up256((size_t)segs * panel * 4);
    l.marks = l.segdec + up256((size_t)segs * z.H * 4);
    l.order = l.marks + up256((size_t)slots * panel * 2 * planes);
    l.span = l.order + up256(z.S > 1 ? (size_t)z.S * 4 : 0);
    l.total = l.span + 256;
    return l;
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
