// head_scan.cuh -- shared pieces of the scan with one decay per head.
//
// Per head h of group g = h / (H / G), with a P x N state:
//   d_t = softplus(delta_t + bias),  S_t = exp(d_t A) S_{t-1} + d_t u_t B_t^T,
//   y_t = S_t C_t + Dskip u_t.
// The sequences are cut into chunks of Q tokens counted from each sequence's own
// start, so a chunk never crosses a boundary. Chunk k of sequence s has slot
// floor(start_s / Q) + s + k: slots of different chunks differ, there are at most
// tok / Q + S of them, and a kernel with one CTA per slot needs no host copy of
// cu_seqlens (some slots stay idle).
#pragma once

#include "common.cuh"
#include "internal.h"

namespace ssm {

constexpr float kHeadMinLog = -208.0f;  // exp of it is 0 in fp32: a stronger decay is the same decay

struct ChunkRef {
    int64_t start;  // first token
    int seq, k;     // sequence, chunk number in it
    int len;        // tokens, 0: idle slot
    bool last;      // the sequence's last chunk
};

__device__ __forceinline__ void seq_bounds(const int32_t *cu, int64_t S, int64_t tok, int64_t s,
                                           int64_t &lo, int64_t &hi)
{
    if (cu) {
        lo = s == 0 ? 0 : clamp_off(cu[s], tok);
        hi = clamp_off(cu[s + 1], tok);
    } else {
        const int64_t L = tok / S;
        lo = s * L;
        hi = lo + L;
    }
    if (hi < lo) hi = lo;
}

// The chunk behind a slot; `span` tokens per chunk. Slot bases increase strictly
// with s for valid cu_seqlens; an invalid array gives some chunk inside [0, tok].
__device__ __forceinline__ ChunkRef find_chunk(const int32_t *cu, int64_t S, int64_t tok,
                                               int64_t span, int64_t slot)
{
    int64_t lo = 0, hi = S - 1;
    if (cu) {
        while (lo < hi) {
            const int64_t mid = (lo + hi + 1) >> 1;
            if (clamp_off(cu[mid], tok) / span + mid <= slot) lo = mid;
            else hi = mid - 1;
        }
    } else {
        const int64_t L = tok / S;
        while (lo < hi) {
            const int64_t mid = (lo + hi + 1) >> 1;
            if (mid * L / span + mid <= slot) lo = mid;
            else hi = mid - 1;
        }
    }
    ChunkRef r;
    int64_t a, b;
    seq_bounds(cu, S, tok, lo, a, b);
    const int64_t k = slot - (a / span + lo);
    const int64_t at = a + k * span;
    r.seq = (int)lo;
    r.k = (int)k;
    r.start = at;
    r.len = (k < 0 || at >= b) ? 0 : (int)(b - at < span ? b - at : span);
    r.last = at + span >= b;
    return r;
}

__host__ __device__ __forceinline__ int64_t head_slots(int64_t tok, int64_t S, int64_t span)
{
    return tok / span + S;
}

// softplus to about one fp32 ulp: its relative error becomes an absolute error of
// the decay's exponent, so the faster forms of the per-channel scan lose too much.
__device__ __forceinline__ float softplus_exact(float v)
{
    return fmaxf(v, 0.0f) + log1pf(expf(-fabsf(v)));
}

__device__ __forceinline__ float head_step(float raw, int softplus)
{
    return softplus ? softplus_exact(raw) : raw;
}

// d(head_step)/d(raw)
__device__ __forceinline__ float head_step_grad(float raw, int softplus)
{
    return softplus ? 1.0f / (1.0f + expf(-raw)) : 1.0f;
}

}  // namespace ssm
