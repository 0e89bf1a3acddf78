// umma.cuh -- tcgen05 matrix instructions on bf16 tiles in shared and tensor memory.
//
// Operand tiles are panels of R rows x 64 bf16, 128 bytes a row, rows in order, the
// 16-byte pieces of row r permuted by piece ^ (r & 7) (the 128-byte swizzle), each
// panel 1024-byte aligned. The same panel serves both ways:
//   K-major   rows are the operand's M (or N) index, the 64 columns its K index;
//   MN-major  rows are the K index, the 64 columns the M (or N) index; 128 columns
//             are two panels, one `panel` stride apart.
// Accumulators are 128 lanes x N fp32 columns of tensor memory, one row a lane.
#pragma once

#include <cuda_bf16.h>

#include "tma.cuh"

namespace ssm {
namespace umma {

constexpr uint32_t kPanel = 128 * 128;  // bytes of a 128-row panel

// Byte offset of 16-byte piece `c` of row r in a panel.
__device__ __forceinline__ uint32_t piece(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

// Shared-memory descriptor: 128-byte swizzle, strides in bytes.
__device__ __forceinline__ uint64_t desc(uint32_t addr, uint32_t lead, uint32_t stride)
{
    return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)(lead >> 4) << 16) |
           ((uint64_t)(stride >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// K-major: 8 rows (1024 bytes) from one group to the next; a step of 16 along K is 32 bytes.
__device__ __forceinline__ uint64_t desc_k(uint32_t panel, int k16)
{
    return desc(panel + k16 * 32, 16, 1024);
}
// MN-major: 8 rows along K are 1024 bytes, the next 64 columns one panel away; 16 rows a step.
__device__ __forceinline__ uint64_t desc_mn(uint32_t panel, int k16, uint32_t next)
{
    return desc(panel + k16 * 2048, next, 1024);
}

// Tiles without swizzle, as the state marks are kept: pieces of 8 bf16, [piece][row][8],
// `rows` rows. K-major when the pieces run along K, MN-major when the rows do.
__device__ __forceinline__ uint64_t desc_plain(uint32_t addr, uint32_t lead, uint32_t stride)
{
    return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)(lead >> 4) << 16) |
           ((uint64_t)(stride >> 4) << 32) | ((uint64_t)1 << 46);
}
__device__ __forceinline__ uint64_t plain_k(uint32_t tile, int k16, int rows)
{
    return desc_plain(tile + k16 * 32 * rows, 16 * rows, 128);
}
__device__ __forceinline__ uint64_t plain_mn(uint32_t tile, int k16, int rows)
{
    return desc_plain(tile + k16 * 256, 128, 16 * rows);
}

// A descriptor moved on by `bytes`: cheap enough to be an immediate, where building each
// descriptor anew costs an issuing thread more than the instruction itself.
__device__ __forceinline__ constexpr uint64_t moved(uint64_t d, uint32_t bytes) { return d + (bytes >> 4); }

// Instruction descriptor: bf16 x bf16 -> fp32, M = 128.
__device__ __forceinline__ constexpr uint32_t idesc(int N, bool a_mn, bool b_mn)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) |
           ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
}

// True in one lane of a converged warp. The matrix instructions of a warp are issued
// under it: the compiler then knows that one thread runs them and keeps descriptors in
// uniform registers, which a test of the thread index does not tell it (100 clocks an
// instruction instead of the 32 to 64 that the tensor core takes).
__device__ __forceinline__ bool elect()
{
    uint32_t r;
    asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n"
                 : "=r"(r) :: "memory");
    return r != 0;
}

// D (+)= A B, operands in shared memory. One thread.
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool add)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n"
        :: "r"(d), "l"(a), "l"(b), "r"(id), "r"(add ? 1u : 0u) : "memory");
}

// The same with A in tensor memory: row a lane, two bf16 of K a column.
__device__ __forceinline__ void mma_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t id, bool add)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n"
        :: "r"(d), "r"(a), "l"(b), "r"(id), "r"(add ? 1u : 0u) : "memory");
}

// The barrier completes once every matrix instruction this thread issued before has.
__device__ __forceinline__ void commit(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                 :: "r"(saddr(bar)) : "memory");
}

// A CTA that allocates all 512 columns gets them from column 0: with addresses known when
// compiling, an issuing thread needs no registers moved to the uniform file.
constexpr uint32_t kWhole = 0;

// One warp: allocate / free `cols` (a power of two >= 32) columns of tensor memory.
__device__ __forceinline__ void alloc(uint32_t *slot, uint32_t cols)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(saddr(slot)), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void dealloc(uint32_t addr, uint32_t cols)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(addr), "r"(cols));
}

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// mbar_wait for barriers that matrix instructions complete: these waits are short and
// on the critical path, so they poll with the hardware's own suspend time. At most 2^22
// tries, then bit 0 of *status is set and each later wait of this thread tries once. The
// count of tries is hidden from the compiler, which otherwise makes a second copy of
// the code behind a wait for the case that it failed: the instruction cache feels it.
constexpr unsigned kTries = 1u << 22;
__device__ __forceinline__ void wait(uint64_t *bar, uint32_t parity, unsigned &tries, int *status)
{
#pragma unroll 1
    for (unsigned i = 0; i < tries; ++i) {
        uint32_t done;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
            " selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(done) : "r"(saddr(bar)), "r"(parity) : "memory");
        if (done) return;
    }
    asm volatile("mov.u32 %0, 1;" : "=r"(tries));
    atomicOr(status, 1);
}

// Address of this warp's lanes: a warp reaches lanes 32 (warp % 4) .. + 31.
__device__ __forceinline__ uint32_t lanes(uint32_t base, int warp) { return base + ((uint32_t)(warp & 3) << 21); }

// 16 or 8 columns of this thread's lane. The values are there after wait_ld.
__device__ __forceinline__ void ld16(uint32_t addr, uint32_t (&v)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(addr));
}

__device__ __forceinline__ void ld8(uint32_t addr, uint32_t (&v)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(addr));
}

__device__ __forceinline__ void st4(uint32_t addr, const uint32_t (&v)[4])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};"
                 :: "r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}

__device__ __forceinline__ void st8(uint32_t addr, const uint32_t (&v)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 :: "r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// 16 lanes (from the address's lane) x 16 columns, as four 8 x 8 bf16 tiles read by
// ldsm_t leave them: registers 2 q, 2 q + 1 hold lanes l / 4 and l / 4 + 8, column 4 q + l % 4.
__device__ __forceinline__ void st_tiles(uint32_t addr, const uint32_t (&v)[8])
{
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 :: "r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
// Four 8 x 8 bf16 tiles, transposed: lane l of tile i gives the address of the tile's row
// l % 8 (lanes 8 i ..), and gets column l / 4, rows 2 (l % 4) and + 1.
__device__ __forceinline__ void ldsm_t(uint32_t addr, uint32_t &a, uint32_t &b, uint32_t &c, uint32_t &d)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(addr) : "memory");
}

// Two fp32 to a bf16 pair, lo in the low half.
__device__ __forceinline__ uint32_t pack(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float lo_f(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_f(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// 16 bytes global -> shared; without `in`, zeros and no read.
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool in)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 :: "r"(dst), "l"(src), "r"(in ? 16u : 0u) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait()
{
    asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory");
}

// 3-D tile load / store; a store's completion is tracked by bulk groups.
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap *map, uint64_t *bar, int x, int y, int z)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];"
        :: "r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(saddr(bar)) : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, uint32_t src, int x, int y, int z)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];"
                 :: "l"(map), "r"(src), "r"(x), "r"(y), "r"(z) : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
        :: "r"(dst), "l"(src), "r"(bytes), "r"(saddr(bar)) : "memory");
}

// (tokens, groups, width) bf16 with a token stride, in boxes of 128 tokens x 64 columns
// of one group, 128-byte swizzle; columns beyond `width` and tokens beyond the last read
// as zeros and are not stored. Base 16-byte aligned, stride and width multiples of 8.
inline bool encode_3d(CUtensorMap *map, const void *base, int64_t tokens, int64_t groups, int64_t width,
                      int64_t stride)
{
    auto fn = tensor_map_encoder();
    if (!fn || tokens < 1) return false;
    cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)groups, (cuuint64_t)tokens};
    cuuint64_t strides[2] = {(cuuint64_t)width * 2, (cuuint64_t)stride * 2};
    cuuint32_t box[3] = {64, 1, 128};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace umma
}  // namespace ssm
