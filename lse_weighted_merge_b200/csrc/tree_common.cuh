// tree_common.cuh -- what the tree attention's two kernels share: parameters,
// the shards, and conversions of e4m3 codes.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

#include "attn_common.cuh"

namespace lsem {
namespace attn {

struct TreeParams {
    const char *q, *k, *v, *kd, *vd;
    const float *ks, *vs;
    const int64_t* tree;
    const int32_t *kv_len, *draft_len;
    int64_t q_b, q_t, q_h;                          // byte strides
    int64_t k_b, k_h, k_l, v_b, v_h, v_l;
    int64_t kd_b, kd_h, kd_t, vd_b, vd_h, vd_t;
    int64_t ks_b, ks_h, ks_l, vs_b, vs_h, vs_l;     // element strides
    int64_t tree_b;
    int T, Hq, G, L, R, shards;
    int row_tiles;      // wide kernel: of 256 rows
    int r0;             // shard of the launch's first block
    int fold;           // the last cached shard has the drafts too
    int join;           // po and pl hold one shard's partials, which the launch merges with its own shard
    int out_dtype;
    float scale_log2;   // scale * log2(e)
    float* po;          // partials [B, T, Hq, shards, D], or NULL:
    float* pl;          // [B, T, Hq, shards]
    char* out;          // the result [B, T, Hq, D]
    float* out_lse;     // [B, T, Hq]
};

// The kernel for more than 16 query rows per (sequence, KV head) (tree_wide.cu):
// launches `shards` shards of p from p.r0 on; fp8: the cache is e4m3 (the shard of
// the drafts, p.R, is 16-bit and of a launch of its own).
cudaError_t launch_tree_wide(const TreeParams& p, int dtype, bool fp8, int shards, int out_dtype, int B, int Hkv, int D,
                             bool pdl, cudaStream_t stream);

// cudaFuncSetAttribute(max dynamic shared memory) once per (kernel, device).
cudaError_t allow_smem(const void* fn, int bytes);

namespace {

// Longest key index of a row: nothing beyond it is read.
struct Shard {
    int b, hk, r, lo, hi, live;   // live: drafts of the sequence (rows t >= live are dead)
    bool drafts;
    const char *kb, *vb;
};

__device__ __forceinline__ Shard shard_of(const TreeParams& p, int r, int hk, int b) {
    Shard x;
    x.b = b;
    x.hk = hk;
    x.r = r;
    x.live = p.draft_len ? min(max(__ldcg(p.draft_len + b), 0), p.T) : p.T;
    x.drafts = r == p.R;
    if (x.drafts) {
        x.lo = 0;
        x.hi = x.live;
        x.kb = p.kd + b * p.kd_b + hk * p.kd_h;
        x.vb = p.vd + b * p.vd_b + hk * p.vd_h;
    } else {
        const int len = p.kv_len ? min(max(__ldcg(p.kv_len + b), 0), p.L) : p.L;
        const int per = (int)(((int64_t)len + p.R - 1) / p.R);
        x.lo = (int)min((int64_t)len, (int64_t)r * per);
        x.hi = (int)min((int64_t)len, (int64_t)x.lo + per);
        x.kb = p.k + b * p.k_b + hk * p.k_h;
        x.vb = p.v + b * p.v_b + hk * p.v_h;
    }
    return x;
}

// The address of query row `row` of (b, hk).
__device__ __forceinline__ const char* q_row(const TreeParams& p, int b, int hk, int row) {
    const int t = row / p.G;
    return p.q + b * p.q_b + t * p.q_t + (int64_t)(hk * p.G + row - t * p.G) * p.q_h;
}

// Two e4m3 codes (in the low or high half of c) as two f16.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t c) {
    uint32_t h;
    asm("{\n.reg .b16 lo, hi;\nmov.b32 {lo, hi}, %1;\ncvt.rn.f16x2.e4m3x2 %0, lo;\n}" : "=r"(h) : "r"(c));
    return h;
}
__device__ __forceinline__ uint32_t e4m3x2_f16x2_hi(uint32_t c) {
    uint32_t h;
    asm("{\n.reg .b16 lo, hi;\nmov.b32 {lo, hi}, %1;\ncvt.rn.f16x2.e4m3x2 %0, hi;\n}" : "=r"(h) : "r"(c));
    return h;
}
// 4-byte global -> shared copy; `bytes` = 0 writes zeros without reading.
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// The power of two at or below x (of its bits): 2^floor(log2 x), x > 0.
__device__ __forceinline__ float pow2_below(float x) {
    return __uint_as_float(min(max(__float_as_uint(x) & 0x7f800000u, 0x00800000u), 0x7e800000u));
}
// 1 / r of a power of two in [2^-126, 2^126].
__device__ __forceinline__ float pow2_inverse(float r) {
    return __uint_as_float(0x7f000000u - __float_as_uint(r));
}

// Infinities and NaN among the 8 elements of the 16-byte chunk become 0; whether there were any.
template <typename T>
__device__ __forceinline__ bool scrub16(uint32_t (&c)[4]) {
    constexpr uint32_t kExp = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if ((c[i] & kExp) == kExp) c[i] &= 0xffff0000u, bad = true;
        if ((c[i] >> 16 & kExp) == kExp) c[i] &= 0x0000ffffu, bad = true;
    }
    return bad;
}

}  // namespace
}  // namespace attn
}  // namespace lsem
