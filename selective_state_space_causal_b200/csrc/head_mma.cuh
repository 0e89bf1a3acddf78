// head_mma.cuh -- the bf16 scan with one decay per head on the tensor cores: chunk
// tables and states, shared by the forward and the backward.
//
// Chunks have 128 tokens, the M of the matrix instructions. A state is worked on in
// panels of 64 rows (head, 64 of its P rows); rows and columns beyond P and N are
// zeros. Workspace tables hold what a chunk's decays are needed as, per (chunk slot,
// head) and token t: with c_t the running sum of d_t A log2(e) inside the chunk, made in
// 64 bits because it reaches hundreds and small differences of it are used, and r_i
// its value before 32-token block i,
//   d      d_t                      l      c_t - r_{block of t}
//   ec     2^{c_t}                  wf     d_t 2^{c_127 - c_t}
//   col    2^{r_i - c_t} for blocks i = 1..3 and t < 32 i (192 values); times d_t in
//          the forward's tables
//   wn, el 2^{c_127 - c_t} and 2^{l_t}, for the backward;  ll  what rounding l left
#pragma once

#include "head_scan.cuh"
#include "umma.cuh"

namespace ssm {
namespace hm {

constexpr int kC = 128;  // tokens per chunk
constexpr double kLog2eD = 1.4426950408889634;

using bf16 = __nv_bfloat16;

struct Dims {
    const int32_t *cu;
    int64_t S, tok;
    int H, P, G, N;
    int np;    // panels per head
    int npan;  // panels per group
};

// Panel `pi` of group g: its head and first state row.
struct PanelRef {
    int h, p0, rows;
};
__device__ __forceinline__ PanelRef panel_of(const Dims &z, int g, int pi)
{
    PanelRef r;
    r.h = g * (z.H / z.G) + pi / z.np;
    r.p0 = (pi % z.np) * 64;
    r.rows = min(64, z.P - r.p0);
    return r;
}

// Tables of one (chunk slot, head), in floats.
constexpr int kTabD = 0, kTabL = kC, kTabEc = 2 * kC, kTabCol = 3 * kC, kTabWf = 3 * kC + 192;
constexpr int kTabWn = kTabWf + kC, kTabEl = kTabWn + kC, kTabLl = kTabEl + kC;
constexpr int kTab = 7 * kC + 192;
constexpr int kTabOut = kTabWf;  // what the outputs need comes first
__host__ __device__ constexpr int col_at(int i) { return kTabCol + (i == 1 ? 0 : i == 2 ? 32 : 96); }

// Eight bf16 of a row as 16 bytes, elements from `n` on as zeros.
__device__ __forceinline__ uint4 read8(const bf16 *p, int n)
{
    const unsigned short *q = reinterpret_cast<const unsigned short *>(p);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = 2 * i < n ? q[2 * i] : 0, hi = 2 * i + 1 < n ? q[2 * i + 1] : 0;
        w[i] = lo | hi << 16;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void sts16(uint32_t addr, uint4 v)
{
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};"
                 :: "r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

// Tokens [0, len) of a slice with `cols` columns as panels of 128 rows x 64, zeros
// elsewhere. VEC: rows are 16-byte aligned and `cols` a multiple of 8.
template <int COLS, int THREADS, bool VEC>
__device__ __forceinline__ void load_tile(uint32_t dst, const bf16 *src, int64_t stride, int len,
                                          int cols, int tid)
{
    constexpr int PIECES = COLS / 8, ROWS = THREADS / PIECES;  // rows of one pass
    static_assert(THREADS % PIECES == 0 && kC % ROWS == 0, "whole passes");
    const int r0 = tid / PIECES, c = tid % PIECES;
    const int n = min(8, cols - 8 * c);
    const bf16 *q = src + r0 * stride + 8 * c;
    const int64_t step = ROWS * stride;
    const uint32_t at = dst + (c / 8) * umma::kPanel;
#pragma unroll 8
    for (int i = 0; i < kC / ROWS; ++i) {
        const int r = r0 + ROWS * i;
        const bool in = r < len && n > 0;
        const uint32_t to = at + umma::piece(r, c % 8);
        if (VEC) umma::cp16(to, in ? q : src, in);
        else sts16(to, in ? read8(q, n) : make_uint4(0, 0, 0, 0));
        q += step;
    }
}

// The same by one warp, without copies in flight afterwards.
template <int COLS>
__device__ __forceinline__ void load_tile_warp(uint32_t dst, const bf16 *src, int64_t stride, int len,
                                               int cols, int lane)
{
    constexpr int PIECES = COLS / 8, BATCH = 4;  // loads of a batch are all under way before a store
    const uintptr_t at = reinterpret_cast<uintptr_t>(src) | (uintptr_t)stride * 2;  // what all rows are aligned to
    const int unit = at % 16 == 0 ? 16 : at % 4 == 0 ? 4 : 2;
    for (int i0 = lane; i0 < kC * PIECES; i0 += 32 * BATCH) {
        uint4 v[BATCH];
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            const int r = (i0 + 32 * j) / PIECES, c = (i0 + 32 * j) % PIECES, n = min(8, cols - 8 * c);
            const bf16 *q = src + r * stride + 8 * c;
            if (r >= len || n <= 0) v[j] = make_uint4(0, 0, 0, 0);
            else if (n == 8 && unit == 16) v[j] = *reinterpret_cast<const uint4 *>(q);
            else if (n == 8 && unit == 4) {
                const uint32_t *w = reinterpret_cast<const uint32_t *>(q);
                v[j] = make_uint4(w[0], w[1], w[2], w[3]);
            } else v[j] = read8(q, n);
        }
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            const int r = (i0 + 32 * j) / PIECES, c = (i0 + 32 * j) % PIECES;
            sts16(dst + (c / 8) * umma::kPanel + umma::piece(r, c % 8), v[j]);
        }
    }
}

// Rows [len, 128) of `panels` panels become zeros (a tile copy brought the next sequence's).
__device__ __forceinline__ void zero_tail(uint32_t dst, int panels, int len, int tid, int threads)
{
    const int n = (kC - len) * 8;
    for (int i = tid; i < n * panels; i += threads)
        sts16(dst + (i / n) * umma::kPanel + len * 128 + (i % n) * 16, make_uint4(0, 0, 0, 0));
}

__device__ __forceinline__ void bar_sync(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" :: "r"(id), "r"(threads) : "memory");
}

// A state mark: per panel and plane, NPAD / 8 pieces x 64 rows x 8 bf16: a thread per
// row writes whole lines, and a plain copy of it is a matrix operand without swizzle.
template <int NPAD>
constexpr int64_t kMark = (int64_t)64 * NPAD;  // elements of one plane

// Scratch that one call needs, carved from the workspace in this order.
struct Layout {
    size_t tab, seg, segdec, marks, order, span, total;
};

inline size_t up256(size_t v) { return (v + 255) / 256 * 256; }

struct StateArgs {
    Dims z;
    const bf16 *x;  // u, or dy in the reverse walk
    int64_t x_stride;
    const bf16 *b;  // B, or C in the reverse walk
    int64_t b_stride;
    const float *tab;
    const float *init;  // (S, H, P, N) or nullptr
    float *final_;      // (S, H, P, N) or nullptr
    bf16 *marks;        // state before each chunk in walking order
    float *seg;         // (segment slot, panel, NPAD / 4, 64, 4): segments' end states from zero
    float *segdec;      // (segment slot, head): a segment's decay
    int32_t *order;     // room for the sequences' order, or nullptr
    const int64_t *asked;  // where the table kernel left the span, for Plan::kAsk
    int64_t span = 0;   // tokens of a segment (a multiple of kC)
    bool first = false; // the first of a cut walk's two passes
};

// How sequences are walked: whole, cut into segments of `span` tokens, or cut if the
// longest has more than `limit` chunks, which the device finds out.
struct Plan {
    enum Mode { kWhole, kCut, kAsk } mode;
    int64_t span;
    int limit;
};
constexpr int64_t kNoSpan = (int64_t)1 << 31;  // longer than any sequence
// `known`: the lengths are those of dense rows. A workspace has room for either plan, since
// its size is asked for without cu_seqlens.
Plan plan_of(const Dims &z, bool known);
inline bool lengths_known(const Dims &z) { return !z.cu; }

// Steps and running decays of every chunk.
cudaError_t launch_tables(const HeadScanArgs &a, const Dims &z, float *tab, bool backward,
                          const Plan &plan, int64_t *span, cudaStream_t stream, int *launches);
// The states before every chunk (forward) or the gradients of the states after every
// chunk (reverse), `planes` bf16 planes each.
cudaError_t launch_states(const StateArgs &a, bool rev, int planes, const Plan &plan, bool vec,
                          cudaStream_t stream, int *launches);
// Workspace of the tables and of one walk's segments and marks.
Layout layout_of(const Dims &z, int planes, const Plan &plan);
Dims dims_of(const HeadScanArgs &a);

cudaError_t launch_backward(const HeadScanArgs &a, cudaStream_t stream, int *launches);
size_t backward_bytes(const Dims &z);
cudaError_t launch_forward(const HeadScanArgs &a, cudaStream_t stream, int *launches);
size_t forward_bytes(const Dims &z);

inline bool vec16(const void *p, int64_t stride, int64_t width)
{
    // a tile copy's strides end at 2^40 bytes
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride % 8 == 0 && width % 8 == 0 &&
           stride < ((int64_t)1 << 38);
}

}  // namespace hm

// How many of `units` (panels or heads) one CTA takes when `ctas` CTAs could take all of
// theirs: the fewest whole waves over 148 SMs, a CTA's start counted as `start` units. At most
// 16 waves are tried: a start is a small part of a CTA's time by then. Outputs of 136 chunks
// of 24 panels: 39 us with all panels in a CTA, 58 with five; of 555 chunks of 80 panels 441
// us with all, 471 with 20.
inline int64_t units_of_cta(int64_t ctas, int64_t units, double start)
{
    int64_t best = units;
    double cost = -1.0;
    for (int64_t waves = 1; waves <= 16; ++waves) {
        int64_t r = ctas > 0 ? waves * 148 / ctas : units;
        r = r < 1 ? 1 : r > units ? units : r;
        const int64_t per = (units + r - 1) / r, ranges = (units + per - 1) / per;
        const double c = (double)((ctas * ranges + 147) / 148) * ((double)per + start);
        if (cost < 0.0 || c < cost) {
            cost = c;
            best = per;
        }
        if (r == units) break;
    }
    return best;
}

// Sums of the chunks' shares (slot, head, 3) of dA, ddt_bias and dDskip, in a fixed order.
cudaError_t launch_head_reduce(const float *part, int64_t slots, int H, float *dA, float *dbias,
                               float *dskip, cudaStream_t stream, int *launches);
}  // namespace ssm
