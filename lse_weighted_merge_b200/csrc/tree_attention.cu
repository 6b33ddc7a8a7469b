// tree_attention.cu -- attention of T query tokens per sequence over a KV
// cache (16-bit, or e4m3 with a scale per token and head) and over the T
// tokens' own keys, which a mask selects (a tree of drafted tokens).
//
// The work is cut as the merge likes it: the cached keys of a (sequence, KV
// head) into R shards.  The drafts' keys are one more shard (rows16 kernel, or an
// e4m3 cache) or a tile of the last one (tree_wide.cu).  Every shard gives (o, lse)
// partials in fp32 and the LSE merge combines them; a lone shard writes the result
// itself.
//
// The query rows of a (sequence, KV head) are the T * G pairs (token, head of
// the group), row = t * G + g: all of them read the same keys.
//
// rows16 kernel, up to 16 rows: one CTA per shard, 4 warps, each with the key tiles w, w + 4,
// ... of the shard in a private ring filled by cp.async, an online softmax in
// log2 units, mma.sync m16n8k16; the warps' states merge in shared memory.
//   * 16-bit tiles: ldmatrix from XOR-swizzled rows (as decode_attention.cu).
//   * e4m3 tiles stay 8 bits in shared memory and become f16 pairs in
//     registers (exact: e4m3 is a subset of f16), so both products are f16
//     products whatever the query's type.  The order of the inner index of a
//     product is free as long as both operands agree, which lets every thread
//     read 16 consecutive bytes: thread t of a quad holds bytes 16t..16t+15 of
//     a key's 64-byte block for 4 steps of Q K^T, and keys 4t..4t+3 at 16 (or
//     8) consecutive d for P V.
//     q is scaled per row by a power of two to at most 2^15 (f16 holds what is
//     left exactly, down to 2^-39 of the row's largest element).  A key's scale
//     multiplies its score.  A value's scale s multiplies its weight p before
//     the rounding to f16, times a power of two per row (the row's gain) that keeps
//     the largest p * s seen so far, of a value that is not all zeros, at 2^4 or
//     more.  So what counts is a key's part in the result, not its scale: a row
//     of zeros (whose scale is 1) or a large value of little weight takes no
//     precision from the others.  Scales within 2^100 of each other are held.
//   * Up to 8 rows (a decode step, mostly) leave the products' rows 8 to 15 empty;
//     nothing but the products is then done for them.
// Measured on B200, 64 sequences of 4096 e4m3 tokens, 32 heads over 8, D = 128:
// 98 to 103 us by GPU, 5.4 to 5.7 TB/s, 82 to 87 % of the measured copy rate (95 us
// where the keys of the call before are partly in L2 still).  Bound by the instructions
// per key (codes to f16, products that use 4 of 16 rows) and their latencies: two warps
// per scheduler use 37 % of the issue slots.  The gains cost 1 us of that.  Other forms:
// tests in full tiles too 106, three CTAs per SM with two stages each 112 (512 CTAs leave
// a tail), scaling o in every tile and all rows' softmax 119.  One sequence, 16 shards:
// 10.2 to 13 us by machine with the merge, latency.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>
#include <mutex>
#include <type_traits>

#include "attn_common.cuh"
#include "kv_plan.h"
#include "lse_merge.h"
#include "plan.h"
#include "tree_common.cuh"

namespace lsem {
namespace attn {
namespace {

constexpr int kRowWarps = 4;
constexpr int kRowStages = 3;
constexpr int kRowCtas = 2;     // per SM

// The running state of a warp's online softmax: rows g and g + 8, log2 units.
template <int D>
struct RowState {
    float m0, m1;
    float l0, l1;
    float o[D / 8][4];
    __device__ __forceinline__ void reset() {
        m0 = m1 = -INFINITY;
        l0 = l1 = 0.f;
#pragma unroll
        for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    }
};

// The reference of a row's weights lies kLow below the maximum when it is set, and
// is moved when a score lies kHigh above it (the o of all rows is scaled then, so it
// is done seldom).  With f16 weights 2^7 .. 2^14 is the largest one's range: those
// down to 2^-21 of it at least keep f16's 11 bits, and times a value's scale below 2
// they stay below f16's 65504.  bf16 has fp32's range.
template <typename TM>
struct Reference {
    static constexpr bool kHalf = std::is_same<TM, __half>::value;
    static constexpr float kLow = kHalf ? 7.f : 0.f, kHigh = kHalf ? 14.f : 30.f;
};
__device__ __forceinline__ float ex2(float x) {   // results below 2^-126 are 0
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 2^e; below 2^-126: 0.
__device__ __forceinline__ float pow2_of(int e) { return e < -126 ? 0.f : __uint_as_float((uint32_t)(min(e, 127) + 127) << 23); }
__device__ __forceinline__ int exponent(float x) { return (int)(__float_as_uint(x) >> 23) - 127; }

// e4m3: the powers of two by which the weights of rows g and g + 8, times their values'
// scales, are multiplied before they are rounded: o is that much larger.  As large as
// can be until the row has met a value.  top: the largest exponent of a scale so far.
constexpr float kTopGain = 8.507059e37f;   // 2^126
struct Gain {
    float a = kTopGain, b = kTopGain;
    int top = -128;
};

// Fold the tile's scores (C layout, log2 units, -inf where not seen) into the
// running sums: on return sc holds the weights exp2(s - reference).  A row without
// any key so far keeps m = -inf, sums 0.  kRows8: there are no rows g + 8.  kGain (an
// e4m3 cache): where the reference rises by 2^k, the gain does in place of o falling, so
// that o stays relative to its largest parts.  Returns, for the whole warp, whether a
// score lies more than high0 (rows g) or high1 above its reference.
template <typename TM, int D, int NJ, bool kRows8, bool kGain>
__device__ __forceinline__ bool softmax_step(float (&sc)[NJ][4], RowState<D>& w, Gain& gain, float high0, float high1) {
    using Ref = Reference<TM>;
    float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        mx0 = fmaxf(mx0, fmaxf(sc[j][0], sc[j][1]));
        if (!kRows8) mx1 = fmaxf(mx1, fmaxf(sc[j][2], sc[j][3]));
    }
    bool move = mx0 - w.m0 > high0;   // (of any lane of the row: NaN, no key, is false)
    if (!kRows8) move = move || mx1 - w.m1 > high1;
    move = __any_sync(kFull, move);
    if (move) {
        auto raise = [](float mx, float& m, float& l, float& up) {
            mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
            if (!(mx - m > Ref::kHigh)) return 1.f;
            const float next = mx - Ref::kLow;
            if (kGain) {
                const float by = ceilf(next - m);   // infinite at first
                if (!(by <= 252.f)) {
                    m = next;
                    l *= 0.f;
                    up = kTopGain;
                    return 0.f;
                }
                const int k = (int)by, e = exponent(up) + k;
                m += by;
                l *= pow2_of(-k);
                up = pow2_of(min(e, 126));
                return e > 126 ? pow2_of(126 - e) : 1.f;
            }
            const float a = ex2(m - next);   // 0 at first
            m = next;
            l *= a;
            return a;
        };
        const float a0 = raise(mx0, w.m0, w.l0, gain.a);
        float a1 = 1.f;
        if (!kRows8) a1 = raise(mx1, w.m1, w.l1, gain.b);
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
            w.o[n][0] *= a0;
            w.o[n][1] *= a0;
            if (!kRows8) w.o[n][2] *= a1, w.o[n][3] *= a1;
        }
    }
    const float r0 = w.m0 == -INFINITY ? 0.f : w.m0, r1 = w.m1 == -INFINITY ? 0.f : w.m1;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        sc[j][0] = ex2(sc[j][0] - r0);
        sc[j][1] = ex2(sc[j][1] - r0);
        w.l0 += sc[j][0] + sc[j][1];
        if (!kRows8) {
            sc[j][2] = ex2(sc[j][2] - r1);
            sc[j][3] = ex2(sc[j][3] - r1);
            w.l1 += sc[j][2] + sc[j][3];
        }
    }
    return move;
}

// ------------------------------------------------------------ 16-bit tiles

// Tiles of 16 keys, K then V, rows of 2 * D bytes swizzled by tile_off.
template <typename T, int D, bool kRows8>
struct Tiles16 {
    static constexpr int TK = 16;
    static constexpr int kBytes = 2 * TK * D * 2;
    static constexpr int kVOff = TK * D * 2;

    __device__ static void issue(const TreeParams& p, const Shard& x, int key0, uint32_t st, int lane) {
        constexpr int CPR = D / 8;
        const int64_t kl = x.drafts ? p.kd_t : p.k_l, vl = x.drafts ? p.vd_t : p.v_l;
#pragma unroll 4
        for (int c = lane; c < TK * CPR; c += 32) {
            const int row = c / CPR, ch = c - row * CPR;
            const bool ok = key0 + row < x.hi;
            const int64_t key = ok ? key0 + row : x.lo;
            cp_async16(st + tile_off<D>(row, ch), x.kb + key * kl + ch * 16, ok ? 16 : 0);
            cp_async16(st + kVOff + tile_off<D>(row, ch), x.vb + key * vl + ch * 16, ok ? 16 : 0);
        }
    }

    struct Query {
        uint32_t a[D / 16][4];
        float scale0, scale1;
    };
    __device__ static void load_q(const TreeParams& p, const Shard& x, const char* r0, const char* r1,
                                  int t, Query& q) {
        q.scale0 = q.scale1 = p.scale_log2;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            const int c0 = (ks * 16 + 2 * t) * 2;
            q.a[ks][0] = r0 ? *reinterpret_cast<const uint32_t*>(r0 + c0) : 0u;
            q.a[ks][1] = r1 ? *reinterpret_cast<const uint32_t*>(r1 + c0) : 0u;
            q.a[ks][2] = r0 ? *reinterpret_cast<const uint32_t*>(r0 + c0 + 16) : 0u;
            q.a[ks][3] = r1 ? *reinterpret_cast<const uint32_t*>(r1 + c0 + 16) : 0u;
        }
    }

    // words: the draft masks of rows g and g + 8 (all ones over a cache).
    __device__ static void attend(const TreeParams& p, const Shard& x, unsigned char* st_p, uint32_t st,
                                  const Query& q, int key0, uint64_t word0, uint64_t word1, int lane,
                                  RowState<D>& w, Gain& gain) {
        const int t = lane & 3;
        float sc[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j) sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            const int mi = lane >> 3, rr = lane & 7;
            uint32_t bf[4];
            ldsm_x4(st + tile_off<D>((mi >> 1) * 8 + rr, 2 * ks + (mi & 1)), bf);
            Mma<T>::run(sc[0], q.a[ks], bf[0], bf[1]);
            Mma<T>::run(sc[1], q.a[ks], bf[2], bf[3]);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int key = key0 + 8 * j + 2 * t + e;
                bool ok0 = key < x.hi, ok1 = ok0;
                if (x.drafts) {
                    ok0 = ok0 && (word0 >> (key & 63) & 1);
                    ok1 = ok1 && (word1 >> (key & 63) & 1);
                }
                sc[j][e] = ok0 ? sc[j][e] * q.scale0 : -INFINITY;
                if (!kRows8) sc[j][e + 2] = ok1 ? sc[j][e + 2] * q.scale1 : -INFINITY;
            }
        softmax_step<T, D, 2, kRows8, false>(sc, w, gain, Reference<T>::kHigh, Reference<T>::kHigh);
        uint32_t pa[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            pa[2 * j] = Mma<T>::pack(sc[j][0], sc[j][1]);
            pa[2 * j + 1] = kRows8 ? 0u : Mma<T>::pack(sc[j][2], sc[j][3]);
        }
        bool bad = false;
        if (x.drafts) {
            // a value that is no number meets rows that do not see its key with
            // weight 0, and 0 * NaN is NaN: take such elements out of the product
#pragma unroll 1
            for (int c = lane; c < TK * D / 8; c += 32) {
                uint4* at = reinterpret_cast<uint4*>(st_p + kVOff + c * 16);
                const uint4 u = *at;
                uint32_t e[4] = {u.x, u.y, u.z, u.w};
                if (scrub16<T>(e)) {
                    *at = make_uint4(e[0], e[1], e[2], e[3]);
                    bad = true;
                }
            }
            bad = __any_sync(kFull, bad);
            __syncwarp();
        }
#pragma unroll
        for (int np = 0; np < D / 16; ++np) {
            const int mi = lane >> 3, rr = lane & 7;
            uint32_t bf[4];
            ldsm_x4_t(st + kVOff + tile_off<D>((mi & 1) * 8 + rr, 2 * np + (mi >> 1)), bf);
            Mma<T>::run(w.o[2 * np], pa, bf[0], bf[1]);
            Mma<T>::run(w.o[2 * np + 1], pa, bf[2], bf[3]);
        }
        if (bad) {   // ... and give them to the rows that do see them
#pragma unroll 1
            for (int key = key0; key < min(key0 + TK, x.hi); ++key) {
                const char* row = x.vb + key * p.vd_t;
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const T raw = *reinterpret_cast<const T*>(row + (8 * n + 2 * t + e) * 2);
                        const float f = (float)raw;
                        if (!(fabsf(f) <= 3.402823466e38f)) {
                            if (word0 >> (key & 63) & 1) w.o[n][e] += f;
                            if (word1 >> (key & 63) & 1) w.o[n][e + 2] += f;
                        }
                    }
            }
        }
    }
    // The d of element e (0, 1) of accumulator n.
    __device__ static int column(int n, int e, int t) { return 8 * n + 2 * t + e; }
};

// -------------------------------------------------------------- e4m3 tiles

// Tiles of 32 keys: K codes, V codes, K scales, V scales.
template <typename T, int D, bool kRows8>
struct Tiles8 {
    static constexpr int TK = 32;
    static constexpr int kVOff = TK * D;
    static constexpr int kSOff = 2 * TK * D;
    static constexpr int kBytes = 2 * TK * D + 2 * TK * 4;
    static constexpr int CPR = D / 16;   // 16-byte chunks per row

    // Swizzles that spread what a quarter warp reads over all banks.  K: rows
    // g, chunks t (+4).  V: rows 4t + i (i fixed), chunk g, or half a chunk at D = 64.
    __device__ static uint32_t k_off(int row, int ch) {
        return (uint32_t)(row * D + (D == 128 ? (ch ^ (row & 1) << 2) : ch) * 16);
    }
    __device__ static uint32_t v_off(int row, int ch) {
        if (D == 128) return (uint32_t)(row * D + (ch ^ (row >> 2 & 3) << 1) * 16);
        return (uint32_t)((row ^ (row >> 2 & 1)) * D + (ch ^ (row >> 3 & 1) << 1) * 16);
    }

    __device__ static void issue(const TreeParams& p, const Shard& x, int key0, uint32_t st, int lane) {
        const char* kp = x.kb + (key0 + lane / CPR) * p.k_l + lane % CPR * 16;
        const char* vp = x.vb + (key0 + lane / CPR) * p.v_l + lane % CPR * 16;
        if (key0 + TK <= x.hi) {   // (all but a shard's last tile)
#pragma unroll
            for (int i = 0; i < TK * CPR / 32; ++i) {
                const int row = lane / CPR + i * (32 / CPR), ch = lane % CPR;
                cp_async16(st + k_off(row, ch), kp, 16);
                cp_async16(st + kVOff + v_off(row, ch), vp, 16);
                kp += (32 / CPR) * p.k_l;
                vp += (32 / CPR) * p.v_l;
            }
        } else {
#pragma unroll 2
            for (int i = 0; i < TK * CPR / 32; ++i) {
                const int row = lane / CPR + i * (32 / CPR), ch = lane % CPR;
                const bool ok = key0 + row < x.hi;
                cp_async16(st + k_off(row, ch), ok ? kp : x.kb, ok ? 16 : 0);
                cp_async16(st + kVOff + v_off(row, ch), ok ? vp : x.vb, ok ? 16 : 0);
                kp += (32 / CPR) * p.k_l;
                vp += (32 / CPR) * p.v_l;
            }
        }
        const bool ok = key0 + lane < x.hi;
        const int64_t key = ok ? key0 + lane : x.lo;
        cp_async4(st + kSOff + lane * 4, p.ks + x.b * p.ks_b + x.hk * p.ks_h + key * p.ks_l, ok ? 4 : 0);
        cp_async4(st + kSOff + TK * 4 + lane * 4, p.vs + x.b * p.vs_b + x.hk * p.vs_h + key * p.vs_l, ok ? 4 : 0);
    }

    struct Query {
        uint32_t a[D / 16][4];
        float scale0, scale1;
    };
    // Steps 4 * blk + i of thread t: columns 64 * blk + 16 * t + 4 * i + {0, 1 | 2, 3}.
    __device__ static void load_row(const char* row, int t, int half, uint32_t (&a)[D / 16][4], float& scale) {
        float f[D / 64][16];
        float big = 0.f;
#pragma unroll
        for (int blk = 0; blk < D / 64; ++blk) {
            uint4 u[2] = {};
            if (row) {
                u[0] = *reinterpret_cast<const uint4*>(row + (64 * blk + 16 * t) * 2);
                u[1] = *reinterpret_cast<const uint4*>(row + (64 * blk + 16 * t) * 2 + 16);
            }
            T e[16];
            memcpy(e, u, 32);
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                f[blk][c] = (float)e[c];
                big = fmaxf(big, fabsf(f[blk][c]));
            }
        }
        big = fmaxf(big, __shfl_xor_sync(kFull, big, 1));
        big = fmaxf(big, __shfl_xor_sync(kFull, big, 2));
        // 2^(14 - e), e the exponent of the largest element, held to [-100, 126]
        const float top = fminf(fmaxf(pow2_below(big), 7.888609e-31f), 8.507059e37f);
        const float up = 16384.f * pow2_inverse(top);
        scale *= top * (1.f / 16384.f);
#pragma unroll
        for (int blk = 0; blk < D / 64; ++blk)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[4 * blk + i][half] = Mma<__half>::pack(f[blk][4 * i] * up, f[blk][4 * i + 1] * up);
                a[4 * blk + i][half + 2] = Mma<__half>::pack(f[blk][4 * i + 2] * up, f[blk][4 * i + 3] * up);
            }
    }
    __device__ static void load_q(const TreeParams& p, const Shard& x, const char* r0, const char* r1,
                                  int t, Query& q) {
        q.scale0 = q.scale1 = p.scale_log2;
        load_row(r0, t, 0, q.a, q.scale0);
        load_row(r1, t, 1, q.a, q.scale1);
    }

    // Column 2t + e of score tile 2 * kk + h is key 16 * kk + 4t + 2h + e.
    __device__ static void attend(const TreeParams& p, const Shard& x, unsigned char* st_p, uint32_t st,
                                  const Query& q, int key0, uint64_t, uint64_t, int lane,
                                  RowState<D>& w, Gain& gain) {
        constexpr int NJ = TK / 8;
        const int g = lane >> 2, t = lane & 3;
        float sc[NJ][4];
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
            const int row = 16 * (j >> 1) + 4 * (g >> 1) + 2 * (j & 1) + (g & 1);
#pragma unroll
            for (int blk = 0; blk < D / 64; ++blk) {
                const uint4 u = *reinterpret_cast<const uint4*>(st_p + k_off(row, 4 * blk + t));
                const uint32_t c[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    Mma<__half>::run(sc[j], q.a[4 * blk + i], e4m3x2_f16x2(c[i]), e4m3x2_f16x2_hi(c[i]));
            }
        }
        const float* ks = reinterpret_cast<const float*>(st_p + kSOff);
        float* vs = reinterpret_cast<float*>(st_p + kSOff) + TK;
#pragma unroll
        for (int kk = 0; kk < TK / 16; ++kk) {
            const float4 s4 = *reinterpret_cast<const float4*>(ks + 16 * kk + 4 * t);
            const float s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float* c = sc[2 * kk + h];
                    c[e] *= s[2 * h + e] * q.scale0;
                    if (!kRows8) c[e + 2] *= s[2 * h + e] * q.scale1;
                }
        }
        if (key0 + TK > x.hi) {
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (key0 + 16 * (j >> 1) + 4 * t + 2 * (j & 1) + e >= x.hi) sc[j][e] = sc[j][e + 2] = -INFINITY;
        }
        // A weight times its value's scale and the gain stays below 2^16 where the row's
        // largest score and the tile's largest scale say so.
        using Ref = Reference<__half>;
        const int top = exponent(__uint_as_float(__reduce_max_sync(kFull, __float_as_uint(vs[lane]))));
        const float high0 = fminf(Ref::kHigh, 14.99f - (float)(top + exponent(gain.a)));
        const float high1 = fminf(Ref::kHigh, 14.99f - (float)(top + exponent(gain.b)));
        const bool near = softmax_step<__half, D, NJ, kRows8, true>(sc, w, gain, high0, high1) || top > gain.top;
        const bool first = gain.top == -128;
        gain.top = max(gain.top, top);
        if (near) {
            // Values that are all zeros do not count.
            uint32_t code = 0;
#pragma unroll
            for (int i = 0; i < CPR; ++i) {   // (from another chunk in each lane: other banks)
                const uint4 y = *reinterpret_cast<const uint4*>(st_p + kVOff + v_off(lane, (lane + i) % CPR));
                code |= y.x | y.y | y.z | y.w;
            }
            const float mine = vs[lane];
            const bool none = (code & 0x7f7f7f7fu) == 0;
            const int low = exponent(__uint_as_float(__reduce_min_sync(kFull, __float_as_uint(mine) - 1) + 1));   // (not absent keys' 0)
            if (first && !__any_sync(kFull, none && mine != 0.f) && top - low <= 3 && top > -127 && top < 127) {
                // The largest weight is 2^7 here, the largest product 2^4 to 2^8 at this gain:
                // good enough, and 1 us less for one sequence's call than the steps below.
                gain.a = gain.b = pow2_of(-top);
            } else {
                // A row whose largest product is too large lowers its gain.
                if (none) vs[lane] = 0.f;
                __syncwarp();
                float mx0 = 0.f, mx1 = 0.f;   // the largest products, times 2^-15
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float s = vs[16 * (j >> 1) + 4 * t + 2 * (j & 1) + e] * 3.0517578e-05f;
                        mx0 = fmaxf(mx0, sc[j][e] * s);
                        if (!kRows8) mx1 = fmaxf(mx1, sc[j][e + 2] * s);
                    }
                // (a scale times the gain stays finite: a weight of 0 times it is 0)
                const float most = pow2_of(min(100 - gain.top, 126));
                auto lower = [most](float mx, float& up) {
                    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
                    float next = up;
                    // (65504 = 1.999 * 2^15; the largest product becomes 2^7 to 2^8)
                    if (mx * up > 1.9989f) next = fmaxf(pow2_inverse(pow2_below(mx)) * 0.00390625f, 1.17549435e-38f);
                    next = fminf(next, most);
                    const float down = next * pow2_inverse(up);
                    up = next;
                    return down;
                };
                const float d0 = lower(mx0, gain.a);
                float d1 = 1.f;
                if (!kRows8) d1 = lower(mx1, gain.b);
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    w.o[n][0] *= d0;
                    w.o[n][1] *= d0;
                    if (!kRows8) w.o[n][2] *= d1, w.o[n][3] *= d1;
                }
            }
        }
#pragma unroll
        for (int kk = 0; kk < TK / 16; ++kk) {
            const float4 s4 = *reinterpret_cast<const float4*>(vs + 16 * kk + 4 * t);
            const float s[4] = {s4.x, s4.y, s4.z, s4.w};
            uint32_t pa[4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float* c = sc[2 * kk + h];
                pa[2 * h] = Mma<__half>::pack(c[0] * (s[2 * h] * gain.a), c[1] * (s[2 * h + 1] * gain.a));
                pa[2 * h + 1] = 0u;
                if (!kRows8) pa[2 * h + 1] = Mma<__half>::pack(c[2] * (s[2 * h] * gain.b), c[3] * (s[2 * h + 1] * gain.b));
            }
            // keys 4t .. 4t + 3 of this step at D / 8 consecutive d from g * D / 8
            uint32_t u[4][D / 32];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const unsigned char* at = st_p + kVOff;
                if constexpr (D == 128) {
                    const uint4 y = *reinterpret_cast<const uint4*>(at + v_off(16 * kk + 4 * t + i, g));
                    u[i][0] = y.x, u[i][1] = y.y, u[i][2] = y.z, u[i][3] = y.w;
                } else {
                    const uint2 y = *reinterpret_cast<const uint2*>(at + v_off(16 * kk + 4 * t + i, g >> 1) + (g & 1) * 8);
                    u[i][0] = y.x, u[i][1] = y.y;
                }
            }
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                const uint32_t p0 = __byte_perm(u[0][c], u[1][c], 0x5140), p1 = __byte_perm(u[0][c], u[1][c], 0x7362);
                const uint32_t r0 = __byte_perm(u[2][c], u[3][c], 0x5140), r1 = __byte_perm(u[2][c], u[3][c], 0x7362);
                Mma<__half>::run(w.o[4 * c], pa, e4m3x2_f16x2(p0), e4m3x2_f16x2(r0));
                Mma<__half>::run(w.o[4 * c + 1], pa, e4m3x2_f16x2_hi(p0), e4m3x2_f16x2_hi(r0));
                Mma<__half>::run(w.o[4 * c + 2], pa, e4m3x2_f16x2(p1), e4m3x2_f16x2(r1));
                Mma<__half>::run(w.o[4 * c + 3], pa, e4m3x2_f16x2_hi(p1), e4m3x2_f16x2_hi(r1));
            }
        }
    }
    // Column 2t + e of accumulator n: block 2t + e of D / 8 consecutive d, place n in it.
    __device__ static int column(int n, int e, int t) { return (2 * t + e) * (D / 8) + n; }
};

// ------------------------------------------------------------ rows16 kernel

// One warp's share of a shard: tiles warp, warp + kRowWarps, ...
template <typename Tiles, int D>
__device__ __forceinline__ void attend_shard(const TreeParams& p, const Shard& x, int rows, int warp,
                                             int lane, unsigned char* ring, RowState<D>& w) {
    constexpr int TK = Tiles::TK, S = kRowStages;
    const uint32_t ring_u = smem_u32(ring);
    const int g = lane >> 2, t = lane & 3;
    w.reset();
    Gain gain;
    const int ntiles = (x.hi - x.lo + TK - 1) / TK;
    const int mine = ntiles > warp ? (ntiles - warp + kRowWarps - 1) / kRowWarps : 0;
#pragma unroll
    for (int s = 0; s < S - 1; ++s) {
        if (s < mine) Tiles::issue(p, x, x.lo + (warp + s * kRowWarps) * TK, ring_u + s * Tiles::kBytes, lane);
        cp_commit();
    }
    const char* r0 = g < rows ? q_row(p, x.b, x.hk, g) : nullptr;
    const char* r1 = g + 8 < rows ? q_row(p, x.b, x.hk, g + 8) : nullptr;
    typename Tiles::Query q;
    Tiles::load_q(p, x, r0, r1, t, q);
    uint64_t word0 = ~0ull, word1 = ~0ull;
    if (x.drafts) {
        word0 = r0 ? (uint64_t)p.tree[x.b * p.tree_b + g / p.G] : 0;
        word1 = r1 ? (uint64_t)p.tree[x.b * p.tree_b + (g + 8) / p.G] : 0;
    }
    for (int i = 0; i < mine; ++i) {
        if (i + S - 1 < mine)
            Tiles::issue(p, x, x.lo + (warp + (i + S - 1) * kRowWarps) * TK,
                         ring_u + ((i + S - 1) % S) * Tiles::kBytes, lane);
        cp_commit();
        cp_wait<S - 1>();
        __syncwarp();
        Tiles::attend(p, x, ring + (i % S) * Tiles::kBytes, ring_u + (i % S) * Tiles::kBytes, q,
                      x.lo + (warp + i * kRowWarps) * TK, word0, word1, lane, w, gain);
        __syncwarp();
    }
    cp_wait<0>();
    w.l0 += __shfl_xor_sync(kFull, w.l0, 1);
    w.l0 += __shfl_xor_sync(kFull, w.l0, 2);
    w.l1 += __shfl_xor_sync(kFull, w.l1, 1);
    w.l1 += __shfl_xor_sync(kFull, w.l1, 2);
    if (Tiles::TK == 32) {
        const float down0 = pow2_inverse(gain.a), down1 = pow2_inverse(gain.b);
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
            w.o[n][0] *= down0;
            w.o[n][1] *= down0;
            w.o[n][2] *= down1;
            w.o[n][3] *= down1;
        }
    }
}

// Warp states in shared memory: m [warps][16], l [warps][16], o [warps][16][D].
template <typename Tiles, int D>
__device__ __forceinline__ void store_state(float* st, int warp, int lane, const RowState<D>& w) {
    const int g = lane >> 2, t = lane & 3;
    float* st_o = st + 2 * kRowWarps * 16;
    if (t == 0) {
        st[warp * 16 + g] = w.m0;
        st[warp * 16 + g + 8] = w.m1;
        st[(kRowWarps + warp) * 16 + g] = w.l0;
        st[(kRowWarps + warp) * 16 + g + 8] = w.l1;
    }
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            st_o[(warp * 16 + g) * D + Tiles::column(n, e, t)] = w.o[n][e];
            st_o[(warp * 16 + g + 8) * D + Tiles::column(n, e, t)] = w.o[n][e + 2];
        }
}

// grid (shards, Hkv, B)
template <typename T, int D, bool kFp8, bool kRows8, typename TOut>
__global__ void __launch_bounds__(kRowWarps * 32, kRowCtas) tree_rows16_kernel(const TreeParams p) {
    extern __shared__ __align__(128) unsigned char smem[];
    using Cache = typename std::conditional<kFp8, Tiles8<T, D, kRows8>, Tiles16<T, D, kRows8>>::type;
    using Draft = Tiles16<T, D, kRows8>;
    constexpr int kRing = kRowStages * (Cache::kBytes > Draft::kBytes ? Cache::kBytes : Draft::kBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rows = p.T * p.G;
    pdl_wait();
    pdl_release();
    Shard x = shard_of(p, blockIdx.x, blockIdx.y, blockIdx.z);
    if (x.live == 0) x.hi = x.lo;   // dead rows only
    RowState<D> w;
    unsigned char* ring = smem + warp * kRing;
    float* st = reinterpret_cast<float*>(smem);
    if (kFp8 && !x.drafts) {
        attend_shard<Cache, D>(p, x, rows, warp, lane, ring, w);
        __syncthreads();
        store_state<Cache, D>(st, warp, lane, w);
    } else {
        attend_shard<Draft, D>(p, x, rows, warp, lane, ring, w);
        __syncthreads();
        store_state<Draft, D>(st, warp, lane, w);
    }
    __syncthreads();
    const float* st_o = st + 2 * kRowWarps * 16;
    for (int idx = threadIdx.x; idx < 16 * D; idx += kRowWarps * 32) {
        const int i = idx / D, d = idx - i * D;   // row i
        if (i >= rows) break;
        const int t = i / p.G;
        float M = -INFINITY;
#pragma unroll
        for (int v = 0; v < kRowWarps; ++v) M = fmaxf(M, st[v * 16 + i]);
        float den = 0.f, num = 0.f;
        if (t < x.live) {
            // a warp that saw no key has sums 0 (NaN, where all its scores were)
#pragma unroll
            for (int v = 0; v < kRowWarps; ++v) {
                const float mv = st[v * 16 + i];
                const float e = mv == -INFINITY ? 1.f : exp2f(mv - M);
                den += e * st[(kRowWarps + v) * 16 + i];
                num += e * st_o[(v * 16 + i) * D + d];
            }
        }
        const bool any = den != 0.f;   // NaN where a score was
        const float o = any ? num / den : 0.f;
        const float lse = any ? (M + log2f(den)) * kLn2 : -INFINITY;
        const int64_t at = ((int64_t)x.b * p.T + t) * p.Hq + x.hk * p.G + (i - t * p.G);
        if (p.po) {
            p.po[(at * p.shards + x.r) * D + d] = o;
            if (d == 0) p.pl[at * p.shards + x.r] = lse;
        } else {
            store_out<TOut>(p.out + (at * D + d) * (int64_t)sizeof(TOut), o);
            if (d == 0) p.out_lse[at] = lse;
        }
    }
}

// -------------------------------------------------------------------- merge

// The LSE merge of a row's shards.  D / 4 lanes hold a row, 4 elements each; kWide
// gives a row to the whole block, whose groups of lanes take every 4th (D = 64: 8th)
// shard and join through shared memory, else to one group.  The loads of kBatch
// shards are in flight before any is used, folded into a running (max, weight sum,
// weighted sum).  (lse_merge gives -inf as the lse of a row one of whose partials is
// NaN; here that is NaN.)
// Few rows with many shards are bound by latency: 32 rows of 16 shards and 4096 keys
// (one decode step of one sequence) take 12.8 us with a group per row.
template <typename TOut, int D, bool kWide>
__global__ void __launch_bounds__(128) tree_merge_kernel(const float* po, const float* pl, int shards, uint32_t rows,
                                                         char* out, float* out_lse) {
    constexpr int kLanes = D / 4, kGroups = 128 / kLanes, kBatch = 8;
    const int group = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
    const uint32_t row = kWide ? blockIdx.x : blockIdx.x * kGroups + group;
    if (row >= rows) return;
    const int first = kWide ? group : 0, step = kWide ? kGroups : 1;
    const float* o = po + (int64_t)row * shards * D + lane * 4;
    const float* l = pl + (int64_t)row * shards;
    pdl_wait();
    pdl_release();
    float mx = -INFINITY, den = 0.f;
    float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = first; s0 < shards; s0 += kBatch * step) {
        float lv[kBatch];
        float4 ov[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int s = s0 + u * step;
            const bool in = s < shards;
            lv[u] = in ? __ldcg(l + s) : -INFINITY;
            ov[u] = in ? __ldcg(reinterpret_cast<const float4*>(o + (int64_t)s * D)) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float top = mx;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) top = fmaxf(top, lv[u]);
        const float ref = top == -INFINITY ? 0.f : top;
        const float down = expf(mx - ref);   // 0 while nothing was seen
        den *= down;
        num.x *= down, num.y *= down, num.z *= down, num.w *= down;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const float e = expf(lv[u] - ref);
            den += e;
            num.x = fmaf(e, ov[u].x, num.x);
            num.y = fmaf(e, ov[u].y, num.y);
            num.z = fmaf(e, ov[u].z, num.z);
            num.w = fmaf(e, ov[u].w, num.w);
        }
        mx = top;
    }
    if constexpr (kWide) {
        __shared__ float4 other[128];
        __shared__ float2 state[kGroups];
        other[threadIdx.x] = num;
        if (lane == 0) state[group] = make_float2(mx, den);
        __syncthreads();
        if (group > 0) return;
        float top = -INFINITY;
#pragma unroll
        for (int g = 0; g < kGroups; ++g) top = fmaxf(top, state[g].x);
        const float ref = top == -INFINITY ? 0.f : top;
        den = 0.f;
        num = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {   // (a group that saw no key has sums 0, or NaN)
            const float e = state[g].x == -INFINITY ? 1.f : expf(state[g].x - ref);
            const float4 v = other[g * kLanes + lane];
            den = fmaf(e, state[g].y, den);
            num.x = fmaf(e, v.x, num.x);
            num.y = fmaf(e, v.y, num.y);
            num.z = fmaf(e, v.z, num.z);
            num.w = fmaf(e, v.w, num.w);
        }
        mx = top;
    }
    const bool any = den != 0.f;   // NaN where a partial is
    const float inv = any ? 1.f / den : 0.f;
    const float f[4] = {num.x * inv, num.y * inv, num.z * inv, num.w * inv};
    char* at = out + ((int64_t)row * D + lane * 4) * (int64_t)sizeof(TOut);
    if constexpr (sizeof(TOut) == 4) {
        *reinterpret_cast<float4*>(at) = make_float4(f[0], f[1], f[2], f[3]);
    } else {
        *reinterpret_cast<uint2*>(at) = make_uint2(Mma<TOut>::pack(f[0], f[1]), Mma<TOut>::pack(f[2], f[3]));
    }
    if (lane == 0) out_lse[row] = any ? mx + logf(den) : -INFINITY;
}

using MergeFn = void (*)(const float*, const float*, int, uint32_t, char*, float*);
template <typename TOut>
MergeFn pick_merge_d(int D, bool wide) {
    if (D == 64) return wide ? tree_merge_kernel<TOut, 64, true> : tree_merge_kernel<TOut, 64, false>;
    return wide ? tree_merge_kernel<TOut, 128, true> : tree_merge_kernel<TOut, 128, false>;
}
MergeFn pick_merge(int out_dtype, int D, bool wide) {
    switch (out_dtype) {
        case LSE_MERGE_F32: return pick_merge_d<float>(D, wide);
        case LSE_MERGE_F16: return pick_merge_d<__half>(D, wide);
        default: return pick_merge_d<__nv_bfloat16>(D, wide);
    }
}

// ------------------------------------------------------------------- launch

struct TreeKernel {
    void (*fn)(TreeParams);
    int smem;
};

template <typename T, int D, bool kFp8, bool kRows8, typename TOut>
TreeKernel rows16() {
    constexpr int ring8 = kFp8 ? Tiles8<T, D, kRows8>::kBytes : 0, ring16 = Tiles16<T, D, kRows8>::kBytes;
    constexpr int ring = kRowWarps * kRowStages * (ring8 > ring16 ? ring8 : ring16);
    constexpr int states = kRowWarps * 16 * (D + 2) * 4;
    return TreeKernel{tree_rows16_kernel<T, D, kFp8, kRows8, TOut>, ring > states ? ring : states};
}
template <typename T, int D, bool kFp8, bool kRows8>
TreeKernel pick_out(int out_dtype) {
    switch (out_dtype) {
        case LSE_MERGE_F32: return rows16<T, D, kFp8, kRows8, float>();
        case LSE_MERGE_F16: return rows16<T, D, kFp8, kRows8, __half>();
        default: return rows16<T, D, kFp8, kRows8, __nv_bfloat16>();
    }
}
template <typename T, int D>
TreeKernel pick_rows(bool fp8, bool rows8, int out_dtype) {
    if (rows8) return fp8 ? pick_out<T, D, true, true>(out_dtype) : pick_out<T, D, false, true>(out_dtype);
    return fp8 ? pick_out<T, D, true, false>(out_dtype) : pick_out<T, D, false, false>(out_dtype);
}
template <typename T>
TreeKernel pick_tree(int D, bool fp8, bool rows8, int out_dtype) {
    return D == 64 ? pick_rows<T, 64>(fp8, rows8, out_dtype) : pick_rows<T, 128>(fp8, rows8, out_dtype);
}

std::mutex g_tree_mu;
struct TreeAttr {
    const void* fn;
    int dev;
};
TreeAttr g_tree_done[256];
int g_tree_n = 0;

}  // namespace

cudaError_t allow_smem(const void* fn, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lk(g_tree_mu);
    for (int i = 0; i < g_tree_n; ++i)
        if (g_tree_done[i].fn == fn && g_tree_done[i].dev == dev) return cudaSuccess;
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && g_tree_n < 256) g_tree_done[g_tree_n++] = TreeAttr{fn, dev};
    return e;
}

namespace {

int launch_tree(const lse_merge_tree_args* args, cudaStream_t stream) {
    if (!args) return LSE_MERGE_ENULL;
    const lse_merge_tree_args& a = *args;
    TreePlan pl;
    const int rc = make_tree_plan(a, &pl);
    if (rc != LSE_MERGE_OK) return rc;
    const bool fp8 = a.cache_dtype == LSE_MERGE_E4M3, drafts = a.k_draft != nullptr;
    const int64_t ce = fp8 ? 1 : 2;
    TreeParams p{};
    p.q = static_cast<const char*>(a.q);
    p.k = static_cast<const char*>(a.k);
    p.v = static_cast<const char*>(a.v);
    p.ks = a.k_scale;
    p.vs = a.v_scale;
    p.kv_len = a.kv_len;
    p.draft_len = a.draft_len;
    p.q_b = a.q_b * 2, p.q_t = a.q_t * 2, p.q_h = a.q_h * 2;
    p.k_b = a.k_b * ce, p.k_h = a.k_h * ce, p.k_l = a.k_l * ce;
    p.v_b = a.v_b * ce, p.v_h = a.v_h * ce, p.v_l = a.v_l * ce;
    p.ks_b = a.ks_b, p.ks_h = a.ks_h, p.ks_l = a.ks_l;
    p.vs_b = a.vs_b, p.vs_h = a.vs_h, p.vs_l = a.vs_l;
    if (drafts) {
        p.kd = static_cast<const char*>(a.k_draft);
        p.vd = static_cast<const char*>(a.v_draft);
        p.tree = a.tree;
        p.kd_b = a.kd_b * 2, p.kd_h = a.kd_h * 2, p.kd_t = a.kd_t * 2;
        p.vd_b = a.vd_b * 2, p.vd_h = a.vd_h * 2, p.vd_t = a.vd_t * 2;
        p.tree_b = a.tree_b;
    }
    p.T = a.T, p.Hq = a.Hq, p.G = pl.G, p.L = a.L, p.R = a.R;
    // More than 16 rows take the wide kernel.  The drafts of a 16-bit cache are
    // then with its last shard; those of an 8-bit one, whose products are of
    // another type, are a shard of an earlier launch, which a lone shard of the
    // cache merges with itself.
    const bool wide = pl.rows > 16;
    p.fold = wide && !fp8 && drafts;
    p.join = wide && fp8 && drafts && a.R == 1;
    p.shards = p.fold ? a.R : p.join ? 1 : pl.shards;
    p.scale_log2 = a.scale * kLog2e;
    if (p.shards > 1 || p.join) {
        p.po = static_cast<float*>(a.workspace);
        p.pl = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + pl.ws_l_off);
    }
    if (p.shards == 1) {
        p.out = static_cast<char*>(a.out_o);
        p.out_lse = a.out_lse;
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = kPdl ? 1 : 0;
    cudaError_t e = cudaSuccess;
    if (wide) {
        if (fp8 && drafts) {
            TreeParams d = p;
            d.r0 = a.R;
            d.join = 0;
            e = launch_tree_wide(d, a.dtype, false, 1, a.out_dtype, a.B, a.Hkv, a.D, kPdl != 0, stream);
        }
        if (e == cudaSuccess)
            e = launch_tree_wide(p, a.dtype, fp8, a.R, a.out_dtype, a.B, a.Hkv, a.D, kPdl != 0, stream);
    } else {
        const TreeKernel k = a.dtype == LSE_MERGE_F16 ? pick_tree<__half>(a.D, fp8, pl.rows <= 8, a.out_dtype)
                                                      : pick_tree<__nv_bfloat16>(a.D, fp8, pl.rows <= 8, a.out_dtype);
        e = allow_smem((const void*)k.fn, k.smem);
        if (e == cudaSuccess) {
            cfg.gridDim = dim3((unsigned)p.shards, (unsigned)a.Hkv, (unsigned)a.B);
            cfg.blockDim = dim3(kRowWarps * 32);
            cfg.dynamicSmemBytes = (size_t)k.smem;
            e = cudaLaunchKernelEx(&cfg, k.fn, p);
        }
    }
    if (e == cudaSuccess && p.shards > 1) {
        // a block per row, whose groups share the shards, for more than 4 of them
        const bool spread = p.shards > 4;
        const uint32_t rows = (uint32_t)a.B * a.T * a.Hq, per = spread ? 1u : 128u / (uint32_t)(a.D / 4);
        cfg.gridDim = dim3((rows + per - 1) / per);
        cfg.blockDim = dim3(128);
        cfg.dynamicSmemBytes = 0;
        e = cudaLaunchKernelEx(&cfg, pick_merge(a.out_dtype, a.D, spread), (const float*)p.po, (const float*)p.pl, p.shards,
                               rows, static_cast<char*>(a.out_o), a.out_lse);
    }
    if (e != cudaSuccess) {
        set_last_cuda_error((int)e);
        (void)cudaGetLastError();
        return LSE_MERGE_ELAUNCH;
    }
    return LSE_MERGE_OK;
}

}  // namespace
}  // namespace attn
}  // namespace lsem

extern "C" {

int lse_merge_tree_attention(const lse_merge_tree_args* args, lse_merge_stream_t stream) {
    return lsem::attn::launch_tree(args, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
