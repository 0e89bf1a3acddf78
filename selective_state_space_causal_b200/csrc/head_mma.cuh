// head_mma.cuh -- the bf16 scan with one decay per head on the tensor cores: chunk
// tables and states, shared by the forward and the backward.
//
// Chunks have 128 tokens, the M of the matrix instructions. A state is worked on in
// panels of 64 rows (head, 64 of its P rows); rows and columns beyond P and N are
// zeros. Workspace tables hold, per (chunk slot, head), the steps d_t and the running
// sum of d_t A log2(e) inside the chunk, the latter in 64 bits: it reaches hundreds,
// and what is used are small differences of it.
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

// One 16-byte piece (n of its 8 elements inside the tensor) into shared memory; vec:
// sources are 16-byte aligned and n is 0 or 8.
__device__ __forceinline__ void load_piece(uint32_t dst, const bf16 *src, int n, bool vec)
{
    if (vec) umma::cp16(dst, src, n > 0);
    else sts16(dst, n > 0 ? read8(src, n) : make_uint4(0, 0, 0, 0));
}

// Tokens [t0, t0 + len) of a (tok, cols) slice as panels of 128 rows x 64, zeros elsewhere.
template <int COLS, int THREADS>
__device__ __forceinline__ void load_tile(uint32_t dst, const bf16 *src, int64_t stride, int len,
                                          int cols, bool vec, int tid)
{
    constexpr int PIECES = COLS / 8;
    static_assert(kC * PIECES % THREADS == 0, "whole passes");
#pragma unroll
    for (int i = 0; i < kC * PIECES / THREADS; ++i) {
        const int x = tid + THREADS * i, r = x / PIECES, c = x % PIECES;
        const int n = r < len ? min(8, cols - 8 * c) : 0;
        load_piece(dst + (c / 8) * umma::kPanel + umma::piece(r, c % 8),
                   n > 0 ? src + r * stride + 8 * c : src, n, vec);
    }
}

__device__ __forceinline__ void bar_sync(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" :: "r"(id), "r"(threads) : "memory");
}

// A state mark: per panel and plane, NPAD / 8 pieces x 64 rows x 8 bf16, so that both
// a thread per row (writing) and a copy piece by piece (reading) touch whole lines.
template <int NPAD>
constexpr int64_t kMark = (int64_t)64 * NPAD;  // elements of one plane

// Scratch that one call needs, carved from the workspace in this order.
struct Layout {
    size_t c, d, seg, segdec, marks, total;
};

inline size_t up256(size_t v) { return (v + 255) / 256 * 256; }

struct StateArgs {
    Dims z;
    const bf16 *x;  // u, or dy in the reverse walk
    int64_t x_stride;
    const bf16 *b;  // B, or C in the reverse walk
    int64_t b_stride;
    const double *c;
    const float *d;
    const float *init;  // (S, H, P, N) or nullptr
    float *final_;      // (S, H, P, N) or nullptr
    bf16 *marks;        // state before each chunk in walking order
    int64_t span;       // tokens of a segment (a multiple of kC)
    float *seg;         // split walks: (segment slot, panel, NPAD / 4, 64, 4) end, then start states
    double *segdec;     // (segment slot, head): the segment's decay, log2
    bool x_vec, b_vec;
};

// Steps and running decays of every chunk.
cudaError_t launch_tables(const HeadScanArgs &a, const Dims &z, double *c, float *d,
                          cudaStream_t stream, int *launches);
// The states before every chunk (forward) or the gradients of the states after every
// chunk (reverse), `planes` bf16 planes each.
cudaError_t launch_states(const StateArgs &a, bool rev, int planes, bool split, cudaStream_t stream,
                          int *launches);
Dims dims_of(const HeadScanArgs &a);
// Tokens per segment of the walk, and whether walks are split.
int64_t segment_span(const Dims &z, bool *split);

cudaError_t launch_forward(const HeadScanArgs &a, cudaStream_t stream, int *launches);
size_t forward_bytes(const Dims &z);

inline bool vec16(const void *p, int64_t stride, int64_t width)
{
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride % 8 == 0 && width % 8 == 0;
}

}  // namespace hm
}  // namespace ssm
