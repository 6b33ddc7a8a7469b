// tree_wide.cu -- the tree attention for more than 16 query rows per (sequence,
// KV head): both products on the 5th-generation tensor cores (tcgen05).
//
// One CTA has up to 256 query rows of a (sequence, KV head) and one shard of its
// cached keys, in tiles of 128 keys.  Two streams of products run against each
// other, so that one is in the tensor cores while the other is in its softmax:
//   * more than 128 rows: stream s has the rows 128 s .. 128 s + 127, both read
//     every key tile;
//   * up to 128 rows: both streams have the same rows, stream s the key tiles
//     s, s + 2, ...; their states are merged at the end, in shared memory.
// Warps 0-3 and 4-7 are the softmax of stream 0 and 1 (thread = query row = TMEM
// lane; one thread of each also issues the stream's products), warps 8-15 bring
// the tiles:
//   S = Q K^T   128 x 128, Q and K in shared memory (K-major, 128-byte swizzle)
//   O += P V    128 x D, P in TMEM over S (16 bits, half its columns), V in shared
//               memory as it lies in the cache (its D is the fast index: MN-major)
// TMEM: S0 | S1 | O0 | O1.  The order "QK of tile i + 1 after PV of tile i" of
// each stream makes S complete imply O complete, so a softmax thread may scale
// its row of O when it has seen S.  It does so only where the running maximum has
// grown by 2^kHigh over the reference: the reference lies kLow .. kHigh below the
// maximum, and what it is drops out at the end.
//
// 16-bit tiles come by cp.async into the swizzled layout.  e4m3 tiles come by
// cp.async as they are, each thread converts the 16-byte chunks that it fetched
// itself to f16 (exact) and stores them swizzled; q is scaled per row by a power
// of two, a key's scale multiplies its score and a value's scale its weight,
// relative to a power of two near the largest scale so far (as in the rows16
// kernel).  Keys past the shard's end are zeros, so that no value there, whatever
// it is, meets a weight of 0.
//
// The exponentials (16 per clock and SM) and the tensor cores (128 x 128 x 256
// multiply-adds per tile at 4096 per clock) bound it alike: 1024 clocks per tile
// of 128 rows and 128 keys each.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "device_common.cuh"
#include "lse_merge.h"
#include "plan.h"
#include "tree_common.cuh"

namespace lsem {
namespace attn {
namespace {

constexpr int kLoadWarps = 8;
constexpr int kThreads = (8 + kLoadWarps) * 32;
// Registers per thread of the softmax and of the loading warps: together what the
// block is launched with, 65536.
constexpr int kSoftRegs = 184, kLoadRegs = 72;
static_assert(256 * kSoftRegs + kLoadWarps * 32 * kLoadRegs <= 65536 && kThreads * 128 == 65536, "registers");
constexpr int kTK = 128;                    // keys per tile
constexpr int64_t kGiveUpClocks = 4000000000;  // longest wait for another warp, about 2 s

// CTAs of which a wait ran out (their rows are NaN).
__device__ unsigned g_gave_up;

// ------------------------------------------------------------ PTX

__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}
__device__ __forceinline__ void arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Barrier of the softmax warps.
__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
// Wait for phase `parity`; once a wait has run out, none waits any more.  (By the
// SM's clock: a read of the global timer takes about as long as a tile's softmax.)
__device__ __forceinline__ void wait(uint32_t bar, uint32_t parity, volatile int* dead) {
    if (try_wait(bar, parity)) return;
    const int64_t t0 = clock64();
    while (*dead == 0) {
        for (int i = 0; i < 16; ++i)
            if (try_wait(bar, parity)) return;
        if (clock64() - t0 > kGiveUpClocks) *dead = 1;
    }
}

__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
        "r"((uint32_t)add)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
        "r"((uint32_t)add)
        : "memory");
}
#define LSEM_OP32(c, u) \
    c(u[0]), c(u[1]), c(u[2]), c(u[3]), c(u[4]), c(u[5]), c(u[6]), c(u[7]), c(u[8]), c(u[9]), c(u[10]), c(u[11]), \
        c(u[12]), c(u[13]), c(u[14]), c(u[15]), c(u[16]), c(u[17]), c(u[18]), c(u[19]), c(u[20]), c(u[21]), c(u[22]), \
        c(u[23]), c(u[24]), c(u[25]), c(u[26]), c(u[27]), c(u[28]), c(u[29]), c(u[30]), c(u[31])
// 32 columns of the thread's lane; the values are there after tm_wait32.
__device__ __forceinline__ void tm_get32(uint32_t at, float (&f)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : LSEM_OP32("=f", f)
        : "r"(at)
        : "memory");
}
// (the operands keep every use of the values behind it)
__device__ __forceinline__ void tm_wait32(float (&f)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : LSEM_OP32("+f", f)::"memory");
}
__device__ __forceinline__ void tm_ld32(uint32_t at, float (&f)[32]) {
    tm_get32(at, f);
    tm_wait32(f);
}
__device__ __forceinline__ void tm_put32(uint32_t at, const float (&f)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(at),
        LSEM_OP32("f", f)
        : "memory");
}
// One thread of the (converged) warp, in a form that lets the branch be uniform.
__device__ __forceinline__ bool elect() {
    uint32_t yes;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(yes));
    return yes != 0;
}
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ float ex2(float x) {   // results below 2^-126 are 0
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Descriptor of a shared-memory operand at byte address `at`: 128-byte swizzle,
// groups of 8 rows of 128 bytes 1024 bytes apart.  With the fast index along the
// inner dimension of the product that is all; with it along M or N (V), blocks of
// 64 elements are `block` bytes apart.
__device__ __forceinline__ uint64_t smem_desc(uint32_t at, uint32_t block) {
    return (uint64_t)((at & 0x3ffffu) >> 4) | (uint64_t)(block >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
           1ull << 46 | 2ull << 61;
}
// kind::f16: fp32 accumulators, both operands of type T, M = 128.
template <typename T>
__device__ constexpr uint32_t instr_desc(int n, bool b_mn) {
    const uint32_t t = std::is_same<T, __half>::value ? 0u : 1u;
    return 1u << 4 | t << 7 | t << 10 | (uint32_t)b_mn << 16 | (uint32_t)(n >> 3) << 17 | (128u >> 4) << 24;
}

// ------------------------------------------------------------ layout

template <int D>
struct Lay {
    static constexpr int kTile = kTK * D * 2;       // a tile of 16-bit rows
    static constexpr int kBlock = kTK * 128;        // 64 columns of it
    static constexpr int kRaw = kTK * D;            // a tile of codes
    static constexpr int kCtrl = 7 * kTile;
    static constexpr int kBytes = kCtrl + 256 + 5 * 512;
    // byte offset of 16-byte chunk ch of row
    __device__ static uint32_t at(int row, int ch) {
        return (uint32_t)((ch >> 3) * kBlock + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
    }
};

// Barriers, 8 bytes each, at the control block.
enum { kQFull = 0, kKFull = 1, kKEmpty = 4, kVFull = 7, kVEmpty = 10, kSFull = 13, kPFull = 15, kOFull = 17, kStart = 19, kBars = 20 };

struct Ctrl {
    uint64_t bar[kBars];
    uint32_t tmem;
    int dead;
    int bad;            // a value of the drafts is no number
    // e4m3, known with a tile's keys: the power of two that these were scaled by
    // (0: their scores still need the scales), the reference of the values' scales,
    // and whether the tile's values are relative to it already
    float kref[3], vref[3];
    int vplain[3];
};
static_assert(sizeof(Ctrl) <= 256, "control block");

// How a CTA's tiles are laid out in time: the same for all roles.
struct WidePlan {
    bool two;        // two row tiles
    int n;           // key tiles
    int cached;      // of them over the cache; the last may be the drafts
    __device__ __forceinline__ int count(int s) const { return two ? n : (n + 1 - s) >> 1; }
    __device__ __forceinline__ int tile(int s, int i) const { return two ? i : 2 * i + s; }
};

struct Ring {
    int n, slot;
    uint32_t phase;
    __device__ __forceinline__ void next() {
        if (++slot == n) slot = 0, phase ^= 1;
    }
};

// ------------------------------------------------------------ loaders

// The keys of tile j: [key0, key0 + count) of the cache, or the drafts.
struct Keys {
    const char *k, *v;
    int64_t kl, vl;
    int key0, count;
    bool drafts;
};
__device__ __forceinline__ Keys keys_of(const TreeParams& p, const Shard& x, const WidePlan& pl, int j) {
    Keys t;
    t.drafts = j >= pl.cached;
    if (t.drafts) {
        t.k = p.kd + x.b * p.kd_b + x.hk * p.kd_h;
        t.v = p.vd + x.b * p.vd_b + x.hk * p.vd_h;
        t.kl = p.kd_t, t.vl = p.vd_t;
        t.key0 = 0, t.count = x.live;
    } else {
        t.k = x.kb, t.v = x.vb;
        t.kl = p.k_l, t.vl = p.v_l;
        t.key0 = x.lo + j * kTK;
        t.count = min(kTK, x.hi - t.key0);
    }
    return t;
}

// Brings the keys and values of tiles still to come into L2, kTilesAhead before
// they are fetched: one thread per row, threads 0-127 keys, 128-255 values.
constexpr int kTilesAhead = 4;
struct Prefetch {
    const char *at, *scale;
    int64_t step, scale_step;
    int key, hi;
    __device__ __forceinline__ Prefetch(const TreeParams& p, const Shard& x, int tid, bool fp8) {
        const bool value = tid >= kTK;
        key = x.lo + (tid & (kTK - 1));
        hi = x.hi;
        at = (value ? x.vb : x.kb) + key * (value ? p.v_l : p.k_l);
        step = kTK * (value ? p.v_l : p.k_l);
        scale = nullptr;
        scale_step = 0;
        if (fp8) {
            scale = reinterpret_cast<const char*>(value ? p.vs + x.b * p.vs_b + x.hk * p.vs_h + key * p.vs_l
                                                        : p.ks + x.b * p.ks_b + x.hk * p.ks_h + key * p.ks_l);
            scale_step = 4 * kTK * (value ? p.vs_l : p.ks_l);
        }
    }
    template <int kRowBytes, bool kScale>
    __device__ __forceinline__ void next() {
        if (key < hi) {
#pragma unroll
            for (int b = 0; b < kRowBytes; b += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(at + b));
            if (kScale) asm volatile("prefetch.global.L2 [%0];" ::"l"(scale));
        }
        at += step;
        if (kScale) scale += scale_step;
        key += kTK;
    }
};

// The loaders bring K0, V0, K1, V1, ...
template <typename T, int D>
__device__ __forceinline__ void load16(const TreeParams& p, const Shard& x, const WidePlan& pl, unsigned char* smem,
                                       uint32_t smem_u, Ctrl* ctrl, uint32_t bars, int tid) {
    using L = Lay<D>;
    constexpr int CPR = D / 8, kRows = kLoadWarps * 32 / CPR, kPending = 3;
    const int ch = tid % CPR, row0 = tid / CPR, items = 2 * pl.n;
    Ring kr{pl.two ? 2 : 3, 0, 1}, vr{3, 0, 1};
    Prefetch pf(p, x, tid, false);
    for (int i = 0; i < kTilesAhead; ++i) pf.next<2 * D, false>();
    uint32_t pend[kPending];   // full barriers of the items in flight, oldest first
    int np = 0;
#pragma unroll
    for (int i = 0; i < kPending; ++i) pend[i] = 0;
    auto signal = [&](int keep) {   // complete and announce all but the newest `keep` items
        if (np <= keep) return;
        if (keep == 0) cp_wait<0>();
        if (keep == kPending - 1) cp_wait<kPending - 1>();
        fence_async();
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kPending; ++i)
            if (i < np - keep && (tid & 31) == 0) arrive(pend[i]);
        if (keep) pend[0] = pend[1], pend[1] = pend[2];
        np = keep;
    };
    for (int i = 0; i < items; ++i) {
        const int j = i >> 1;
        const bool value = i & 1;
        if (!value) pf.next<2 * D, false>();
        Ring& r = value ? vr : kr;
        const uint32_t empty = bars + 8 * ((value ? kVEmpty : kKEmpty) + r.slot);
        if (!__all_sync(kFull, try_wait(empty, r.phase))) {
            signal(0);
            wait(empty, r.phase, &ctrl->dead);
        }
        const Keys t = keys_of(p, x, pl, j);
        const int slot = value ? 4 + r.slot : r.slot < 2 ? 2 + r.slot : 1;
        const uint32_t dst = smem_u + slot * L::kTile;
        const char* src = (value ? t.v : t.k) + ch * 16;
        const int64_t stride = value ? t.vl : t.kl;
        if (value && t.drafts) {
            // 0 * NaN is NaN: what is no number leaves the product, and comes
            // back at the end for the rows that see it
            bool bad = false;
            for (int row = row0; row < kTK; row += kRows) {
                uint4 u = make_uint4(0, 0, 0, 0);
                if (row < t.count) u = *reinterpret_cast<const uint4*>(src + row * stride);
                uint32_t c[4] = {u.x, u.y, u.z, u.w};
                bad |= scrub16<T>(c);
                *reinterpret_cast<uint4*>(smem + slot * L::kTile + L::at(row, ch)) = make_uint4(c[0], c[1], c[2], c[3]);
            }
            if (bad) ctrl->bad = 1;
        } else {
            const char* at = src + (t.key0 + row0) * stride;
#pragma unroll
            for (int row = row0; row < kTK; row += kRows) {
                const bool ok = row < t.count;
                cp_async16(dst + L::at(row, ch), ok ? at : src, ok ? 16 : 0);
                at += kRows * stride;
            }
        }
        cp_commit();
        const uint32_t full = bars + 8 * ((value ? kVFull : kKFull) + r.slot);
        if (np == 0) pend[0] = full;
        if (np == 1) pend[1] = full;
        if (np == 2) pend[2] = full;
        ++np;
        if (np == kPending) signal(kPending - 1);
        r.next();
    }
    signal(0);
}

template <int D>
__device__ __forceinline__ void load8(const TreeParams& p, const Shard& x, const WidePlan& pl, unsigned char* smem,
                                      uint32_t smem_u, Ctrl* ctrl, uint32_t bars, float* ks, float* vs, int tid) {
    using L = Lay<D>;
    constexpr int kWarpRows = 512 / D;                  // a warp's 32 chunks of 16 codes
    constexpr int kStep = kLoadWarps * kWarpRows, N = kTK / kStep;
    const int lane = tid & 31, warp = tid >> 5, ahead = pl.two ? 1 : 2;
    const int row0 = warp * kWarpRows + lane * 16 / D, col = lane * 16 % D;
    // Codes come as they are into 2 or 4 raw tiles: two behind the tiles, two where
    // the second tile of queries would be.  A warp converts what it fetched.
    auto raw = [&](int value, int j) -> uint32_t {
        return (uint32_t)(((j & (ahead - 1)) ? L::kTile : 6 * L::kTile) + value * L::kRaw + warp * 512);
    };
    struct Source {
        const char *base, *at;
        int64_t step;
        int key;
    };
    auto fetch = [&](Source& f, uint32_t dst) {
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const bool ok = f.key < x.hi;
            cp_async16(smem_u + dst + u * kLoadWarps * 512 + lane * 16, ok ? f.at : f.base, ok ? 16 : 0);
            f.at += f.step;
            f.key += kStep;
        }
        cp_commit();
    };
    // A tile's scales, lane l keys l, l + 32, l + 64, l + 96 (0: no key), brought a
    // tile ahead by every warp for itself.
    struct Scales {
        const float* src;
        int64_t stride;
        int key;
        float v[4];
        __device__ __forceinline__ void next(int hi) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = key + 32 * e < hi ? src[(key + 32 * e) * stride] : 0.f;
            key += kTK;
        }
        // The largest and smallest, and whether all are powers of two.
        __device__ __forceinline__ bool survey(float& big, float& small) const {
            uint32_t hi = 0, lo = ~0u, frac = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t b = __float_as_uint(v[e]);
                hi = max(hi, b);
                lo = min(lo, b - 1);   // 0 becomes the largest
                frac |= b;
            }
            big = __uint_as_float(__reduce_max_sync(kFull, hi));
            small = __uint_as_float(__reduce_min_sync(kFull, lo) + 1);
            return (__reduce_or_sync(kFull, frac) & 0x807fffffu) == 0;
        }
    };
    // mul: the rows are multiplied by their scales times inv
    auto convert = [&](unsigned char* tile, uint32_t from, bool mul, const Scales& sc, float inv) {
        const unsigned char* src = smem + from + lane * 8;
        uint2 c[2 * N];
#pragma unroll
        for (int u = 0; u < 2 * N; ++u)
            c[u] = *reinterpret_cast<const uint2*>(src + (u >> 1) * kLoadWarps * 512 + (u & 1) * 256);
#pragma unroll
        for (int u = 0; u < 2 * N; ++u) {
            const int within = warp * kWarpRows + (u & 1) * (256 / D) + lane * 8 / D;   // below kStep
            uint32_t h[4] = {e4m3x2_f16x2(c[u].x), e4m3x2_f16x2_hi(c[u].x), e4m3x2_f16x2(c[u].y), e4m3x2_f16x2_hi(c[u].y)};
            if (mul) {
                const float mine = D == 128 ? sc.v[u >> 1] : warp & 4 ? sc.v[(u & 2) + 1] : sc.v[u & 2];
                const float f = __shfl_sync(kFull, mine, within & 31) * inv;
                const uint32_t f2 = Mma<__half>::pack(f, f);
#pragma unroll
                for (int e = 0; e < 4; ++e) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(h[e]) : "r"(f2));
            }
            *reinterpret_cast<uint4*>(tile + L::at((u >> 1) * kStep + within, lane & (D / 8 - 1))) =
                make_uint4(h[0], h[1], h[2], h[3]);
        }
        fence_async();
        __syncwarp();
    };
    auto landed = [&]() {   // the oldest tile's codes, for the whole warp
        if (pl.two)
            cp_wait<1>();
        else
            cp_wait<3>();
        __syncwarp();
    };
    Source k{x.kb + col, x.kb + (x.lo + row0) * p.k_l + col, kStep * p.k_l, x.lo + row0};
    Source v{x.vb + col, x.vb + (x.lo + row0) * p.v_l + col, kStep * p.v_l, x.lo + row0};
    Prefetch pf(p, x, tid, true);
    for (int i = 0; i < kTilesAhead; ++i) pf.next<D, true>();
    for (int j = 0; j < ahead; ++j) {
        fetch(k, raw(0, j));
        fetch(v, raw(1, j));
    }
    Ring kr{2, 0, 1}, vr{2, 0, 1};
    float run = 1.17549435e-38f;   // the reference of the values' scales
    Scales sk{p.ks + x.b * p.ks_b + x.hk * p.ks_h, p.ks_l, x.lo + lane, {}};
    Scales sv{p.vs + x.b * p.vs_b + x.hk * p.vs_h, p.vs_l, x.lo + lane, {}};
    sk.next(x.hi);
    sv.next(x.hi);
    int kslot = 0;
    // the first warp keeps the scales that are not in the tile
    auto keep = [&](float* at, const Scales& sc) {
        if (warp != 0) return;
#pragma unroll
        for (int e = 0; e < 4; ++e) at[lane + 32 * e] = sc.v[e];
    };
    for (int j = 0; j < pl.n; ++j) {
        pf.next<D, true>();
        // f16 has codes * 2^-15 .. 1 exactly: scales that are powers of two go into the tile
        float kbig, vbig, small;
        bool kplain = sk.survey(kbig, small);
        kplain = kplain && small >= kbig * 3.0517578e-05f && kbig >= 1.17549435e-38f && kbig <= 8.507059e37f;
        bool vplain = sv.survey(vbig, small);
        run = fmaxf(run, pow2_below(vbig));
        vplain = vplain && small >= run * 3.0517578e-05f && small >= 1.17549435e-38f && vbig <= run;
        landed();
        wait(bars + 8 * (kKEmpty + kr.slot), kr.phase, &ctrl->dead);
        convert(smem + (2 + kr.slot) * L::kTile, raw(0, j), kplain, sk, pow2_inverse(pow2_below(kbig)));
        // (the place of three tiles ago: the values of two tiles ago would not be
        // in if that tile's softmax were not over)
        if (!kplain) keep(ks + kslot * kTK, sk);
        if (tid == 0) ctrl->kref[kslot] = kplain ? kbig : 0.f, ctrl->vref[kslot] = run, ctrl->vplain[kslot] = vplain;
        __syncwarp();
        if (lane == 0) arrive(bars + 8 * (kKFull + kr.slot));
        kr.next();
        if (++kslot == 3) kslot = 0;
        sk.next(x.hi);
        fetch(k, raw(0, j));
        landed();
        wait(bars + 8 * (kVEmpty + vr.slot), vr.phase, &ctrl->dead);
        convert(smem + (4 + vr.slot) * L::kTile, raw(1, j), vplain, sv, pow2_inverse(run));
        if (!vplain) keep(vs + vr.slot * kTK, sv);
        __syncwarp();
        if (lane == 0) arrive(bars + 8 * (kVFull + vr.slot));
        vr.next();
        sv.next(x.hi);
        fetch(v, raw(1, j));
    }
    cp_wait<0>();
}

// ------------------------------------------------------------ products

// What one thread issues for stream s: S of its tile i, and O += P V of it.
template <typename TM, int D, bool kFp8>
struct Products {
    using L = Lay<D>;
    static constexpr uint32_t kIdQK = instr_desc<TM>(kTK, false), kIdPV = instr_desc<TM>(D, true);
    const WidePlan& pl;
    uint32_t smem_u, tmem, bars;
    Ctrl* ctrl;
    int s;

    __device__ __forceinline__ void qk(int i) const {
        const int j = pl.tile(s, i), nk = kFp8 || pl.two ? 2 : 3, slot = j % nk;
        const uint64_t q = smem_desc(smem_u + (pl.two ? s : 0) * L::kTile, 16);
        const uint64_t k = smem_desc(smem_u + (slot < 2 ? 2 + slot : 1) * L::kTile, 16);
        wait(bars + 8 * (kKFull + slot), (uint32_t)(j / nk) & 1u, &ctrl->dead);
        tc_after();
#pragma unroll
        for (int u = 0; u < D / 16; ++u) {   // (descriptors count in 16 bytes)
            const uint32_t off = ((u >> 2) * L::kBlock + (u & 3) * 32) >> 4;
            mma_ss(tmem + s * kTK, q + off, k + off, kIdQK, u > 0);
        }
        tc_commit(bars + 8 * (kSFull + s));
        tc_commit(bars + 8 * (kKEmpty + slot));
    }
    __device__ __forceinline__ void pv(int i) const {
        const int j = pl.tile(s, i), nv = kFp8 ? 2 : 3, slot = j % nv;
        const uint64_t v = smem_desc(smem_u + (4 + slot) * L::kTile, L::kBlock);
        wait(bars + 8 * (kVFull + slot), (uint32_t)(j / nv) & 1u, &ctrl->dead);
        wait(bars + 8 * (kPFull + s), (uint32_t)i & 1u, &ctrl->dead);
        tc_after();
#pragma unroll
        for (int u = 0; u < kTK / 16; ++u)
            mma_ts(tmem + 2 * kTK + s * D, tmem + s * kTK + u * 8, v + (u * 2048 >> 4), kIdPV, i > 0 || u > 0);
        tc_commit(bars + 8 * (kVEmpty + slot));
        if (i == pl.count(s) - 1) tc_commit(bars + 8 * (kOFull + s));
    }
};

// ------------------------------------------------------------ queries

// Query row -> row `row` of the tile at `tile` (or nowhere); e4m3: scaled to at
// most 2^15 in f16, the inverse times `scale`.  A negative scale changes q's sign.
template <typename T, int D, bool kFp8>
__device__ __forceinline__ void load_query(const char* src, unsigned char* tile, int row, bool flip, float& scale) {
    constexpr int CPR = D / 8;
    const uint32_t sign = flip ? 0x80008000u : 0u;
    float up = 1.f;
    if constexpr (kFp8) {
        float big = 0.f;
        if (src) {
#pragma unroll 4
            for (int c = 0; c < CPR; ++c) {
                float f[8];
                Elem<T>::unpack(*reinterpret_cast<const uint4*>(src + c * 16), f);
#pragma unroll
                for (int e = 0; e < 8; ++e) big = fmaxf(big, fabsf(f[e]));
            }
        }
        const float top = fminf(fmaxf(pow2_below(big), 7.888609e-31f), 8.507059e37f);
        up = 16384.f * pow2_inverse(top);
        scale *= top * (1.f / 16384.f);
    }
    if (!tile) return;
#pragma unroll 4
    for (int c = 0; c < CPR; ++c) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (src) u = *reinterpret_cast<const uint4*>(src + c * 16);
        if constexpr (kFp8) {
            float f[8];
            Elem<T>::unpack(u, f);
            u = make_uint4(Mma<__half>::pack(f[0] * up, f[1] * up), Mma<__half>::pack(f[2] * up, f[3] * up),
                           Mma<__half>::pack(f[4] * up, f[5] * up), Mma<__half>::pack(f[6] * up, f[7] * up));
        }
        *reinterpret_cast<uint4*>(tile + Lay<D>::at(row, c)) =
            make_uint4(u.x ^ sign, u.y ^ sign, u.z ^ sign, u.w ^ sign);
    }
}

// ------------------------------------------------------------ softmax

// A row's running state: reference (log2 units), sum of weights, by how much the
// reference is to rise before the next tile, and e4m3: the values' scale that O is
// relative to.
struct RowSum {
    float m, l, rise, vref;
};
// Weights are watched as the largest sum of 4 of them.  A new reference lies
// kLow below the maximum.  Past kSoft it rises for the next tile, by a power of
// two that leaves the sum at 2^kBase to 2^(kBase + 1), the largest weight at a
// quarter of that or more: f16 weights then stay between 2^7 (which keeps 2^-24 of
// the largest at f16's 11 bits) and f16's 65504, a value's scale below 2 included.
// Past kHard the tile's weights are made again.
template <typename TM>
struct Bounds {
    static constexpr bool kHalf = std::is_same<TM, __half>::value;
    static constexpr float kLow = kHalf ? 7.f : 0.f, kSoft = kHalf ? 2048.f : 1.0995116e12f;
    static constexpr float kHard = kHalf ? 32000.f : 1e30f;
    static constexpr int kBase = kHalf ? 9 : 2;
};

// A tile's scores: where, what multiplies them, which of them the row sees.
struct Scores {
    uint32_t at;
    float scale;             // of the row (and of all keys of the tile)
    const float4 *k4, *v4;   // e4m3 whose scales are not in the tiles: the keys' (or NULL), the values' (or NULL)
    float vinv;              // what the values' are multiplied by
    uint64_t see0, see1;
};

// Replace the tile's scores by the scaled ones, -inf where not seen: for tiles with
// a mask or with scales key by key, and where the scores are so large that a fused
// difference from the reference could lie far from that of the rounded scores.
template <bool kFp8>
__device__ __forceinline__ void scale_scores(Scores& x) {
#pragma unroll 1
    for (int c = 0; c < kTK; c += 32) {
        float f[32];
        tm_ld32(x.at + c, f);
        const uint32_t see = (uint32_t)((c < 64 ? x.see0 : x.see1) >> (c & 63));
#pragma unroll
        for (int u = 0; u < 32; u += 4) {
            float k[4] = {x.scale, x.scale, x.scale, x.scale};
            if (kFp8 && x.k4) {
                const float4 s = x.k4[(c + u) / 4];
                k[0] *= s.x, k[1] *= s.y, k[2] *= s.z, k[3] *= s.w;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) f[u + e] = see >> (u + e) & 1 ? f[u + e] * k[e] : -INFINITY;
        }
        tm_put32(x.at + c, f);
    }
    tm_wait_st();
    x.scale = 1.f;
}

// The largest score, scaled.
__device__ __forceinline__ float softmax_top(const Scores& x) {
    float top = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < kTK; c += 32) {
        float f[32];
        tm_ld32(x.at + c, f);
#pragma unroll
        for (int u = 0; u < 32; u += 4) top = fmaxf(fmaxf(top, fmaxf(f[u], f[u + 1])), fmaxf(f[u + 2], f[u + 3]));
    }
    return top == -INFINITY ? top : top * x.scale;
}

// Weights relative to ref, as 16-bit pairs, and their sums: `sum` of all, `top` the
// largest of 4.  kValue: the weights are multiplied by the values' scales.
template <typename TM, bool kValue>
__device__ __forceinline__ void weights32(const Scores& x, int c, float (&f)[32], uint64_t scale2, uint64_t ref2,
                                          uint64_t (&sum)[4], float& top, uint32_t* w) {
    // in steps over all 32, so that each step's latencies overlap
    uint64_t a[16], t[4];
#pragma unroll
    for (int u = 0; u < 16; ++u) {
        a[u] = ref2;
        fma2(a[u], pack2f(f[2 * u], f[2 * u + 1]), scale2);
    }
#pragma unroll
    for (int u = 0; u < 16; ++u) {
        float e0, e1;
        unpack2f(a[u], e0, e1);
        a[u] = pack2f(ex2(e0), ex2(e1));
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        t[u] = a[u];
#pragma unroll
        for (int h = 4; h < 16; h += 4) asm("add.rn.f32x2 %0, %0, %1;" : "+l"(t[u]) : "l"(a[u + h]));
        float t0, t1;
        unpack2f(t[u], t0, t1);
        top = fmaxf(top, fmaxf(t0, t1));
        asm("add.rn.f32x2 %0, %0, %1;" : "+l"(sum[u]) : "l"(t[u]));
    }
    if (kValue) {
#pragma unroll
        for (int u = 0; u < 16; u += 2) {
            const float4 v = x.v4[c / 4 + u / 2];
            mul2(a[u], pack2f(v.x * x.vinv, v.y * x.vinv));
            mul2(a[u + 1], pack2f(v.z * x.vinv, v.w * x.vinv));
        }
    }
#pragma unroll
    for (int u = 0; u < 16; ++u) {
        float e0, e1;
        unpack2f(a[u], e0, e1);
        w[u] = Mma<TM>::pack(e0, e1);
    }
}
template <typename TM, bool kValue>
__device__ __forceinline__ float softmax_pass(const Scores& x, float ref, float& top, uint32_t* w) {
    const uint64_t scale2 = pack2f(x.scale, x.scale), ref2 = pack2f(-ref, -ref);
    uint64_t sum[4] = {0, 0, 0, 0};
    float fa[32], fb[32];
    top = 0.f;
    tm_get32(x.at, fa);
#pragma unroll
    for (int c = 0; c < kTK; c += 64) {
        tm_wait32(fa);
        tm_get32(x.at + c + 32, fb);
        weights32<TM, kValue>(x, c, fa, scale2, ref2, sum, top, w + c / 2);
        tm_wait32(fb);
        if (c == 0) tm_get32(x.at + 64, fa);
        weights32<TM, kValue>(x, c + 32, fb, scale2, ref2, sum, top, w + c / 2 + 16);
    }
    float s[8];
#pragma unroll
    for (int u = 0; u < 4; ++u) unpack2f(sum[u], s[2 * u], s[2 * u + 1]);
    return ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
}

// S of one tile -> P over it.  The weights are taken relative to the reference
// that the earlier tiles left, in one pass over S; where they turn out too large
// (hardly ever) or the row has no reference yet, the maximum is looked up, the
// reference moves and the pass is made again.
template <typename TM, int D, bool kFp8>
__device__ __forceinline__ void softmax_tile(Scores x, uint32_t tO, float vref, bool scaled, bool first, RowSum& st) {
    using Bd = Bounds<TM>;
    uint32_t w[kTK / 2];
    float l, top, down = 1.f;
    if (st.rise > 0.f) st.m += st.rise, down = ex2(-st.rise);
    if (scaled) scale_scores<kFp8>(x);
    bool move = st.m == -INFINITY, moved = false;
    for (;;) {
        if (__any_sync(kFull, move)) {
            const float next = softmax_top(x) - Bd::kLow;
            if (move && next != -INFINITY) {
                down *= ex2(st.m - next);   // 0 at first
                st.m = next;
            }
            moved = moved || move;   // once: past 2^26 the reference has no finer steps
        }
        const float ref = st.m == -INFINITY ? 0.f : st.m;
        if (!scaled && __any_sync(kFull, fabsf(ref) > 4194304.f)) {
            scale_scores<kFp8>(x);
            scaled = true;
        }
        if (kFp8 && x.v4)
            l = softmax_pass<TM, true>(x, ref, top, w);
        else
            l = softmax_pass<TM, false>(x, ref, top, w);
        move = top > Bd::kHard && !moved;
        if (!__any_sync(kFull, move)) break;
    }
    st.rise = top > Bd::kSoft ? (float)((int)(__float_as_uint(top) >> 23) - 127 - Bd::kBase) : 0.f;
    st.l = st.l * down + l;
    if constexpr (kFp8) {
        down *= st.vref * pow2_inverse(vref);
        st.vref = vref;
    }
    if (!first && __any_sync(kFull, down != 1.f)) {
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
            float f[32];
            tm_ld32(tO + c, f);
#pragma unroll
            for (int e = 0; e < 32; ++e) f[e] *= down;
            tm_put32(tO + c, f);
        }
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        float f[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(w[32 * c + e]);
        tm_put32(x.at + 32 * c, f);
    }
    tm_wait_st();
}

// ------------------------------------------------------------ kernel

template <typename T, int D, bool kFp8>
__global__ void __launch_bounds__(kThreads, 1) tree_wide_kernel(const TreeParams p) {
    using L = Lay<D>;
    using TM = typename std::conditional<kFp8, __half, T>::type;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t smem_u = smem_u32(smem);
    Ctrl* ctrl = reinterpret_cast<Ctrl*>(smem + L::kCtrl);
    const uint32_t bars = smem_u + L::kCtrl;
    const int tid = threadIdx.x, warp = __shfl_sync(kFull, tid >> 5, 0), lane = tid & 31;

    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&ctrl->tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    pdl_wait();
    pdl_release();

    const int r = blockIdx.x / p.row_tiles, row0 = (blockIdx.x - r * p.row_tiles) * 256, rows = p.T * p.G;
    Shard x = shard_of(p, r, blockIdx.y, blockIdx.z);
    WidePlan pl;
    const int last_row = min(rows, x.live * p.G);   // rows from here on are dead
    pl.two = last_row - row0 > 128;
    pl.cached = last_row > row0 ? (x.hi - x.lo + kTK - 1) / kTK : 0;
    pl.n = pl.cached + (p.fold && r == p.R - 1 && last_row > row0 ? 1 : 0);
    // the scales' rings: keys' by tile, values' by slot
    float* ks = reinterpret_cast<float*>(smem + L::kCtrl + 256);
    float* vs = ks + 3 * kTK;
    if (tid == 0) {
        auto init = [&](int b, int n) {
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bars + 8 * b), "r"(n) : "memory");
        };
        const int users = pl.two ? 2 : 1;   // streams that read a tile
        init(kQFull, 8);
        for (int i = 0; i < 3; ++i) {
            init(kKFull + i, kLoadWarps), init(kKEmpty + i, users);
            init(kVFull + i, kLoadWarps), init(kVEmpty + i, users);
        }
        for (int s = 0; s < 2; ++s) init(kSFull + s, 1), init(kPFull + s, 4), init(kOFull + s, 1);
        init(kStart, 4);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        ctrl->dead = (smem_u & 1023u) != 0;   // the swizzle's atoms are 1024 bytes
        ctrl->bad = 0;
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = ctrl->tmem;

    const int s = warp >> 2 & 1;                        // softmax warps: the stream
    const int row = row0 + (pl.two ? 128 * s : 0) + (tid & 127);
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // the warp's lanes of TMEM
    RowSum st{-INFINITY, 0.f, 0.f, 1.17549435e-38f};
    uint64_t word = 0;

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLoadRegs));
        if constexpr (kFp8)
            load8<D>(p, x, pl, smem, smem_u, ctrl, bars, ks, vs, tid - 256);
        else
            load16<T, D>(p, x, pl, smem, smem_u, ctrl, bars, tid - 256);
        return;
    }
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    {
        float scale = fabsf(p.scale_log2);
        if (pl.n > 0) {
            const char* src = row < last_row ? q_row(p, x.b, x.hk, row) : nullptr;
            load_query<T, D, kFp8>(src, pl.two || s == 0 ? smem + (pl.two ? s : 0) * L::kTile : nullptr, tid & 127,
                                   p.scale_log2 < 0.f, scale);
            if (p.fold && src) word = (uint64_t)p.tree[x.b * p.tree_b + row / p.G];
        }
        fence_async();
        __syncwarp();
        if (lane == 0) arrive(bars + 8 * kQFull);
        const bool idle = row - lane >= last_row;   // no live row in the warp
        const uint32_t tS = tmem + lanes + s * kTK, tO = tmem + lanes + 2 * kTK + s * D;
        const Products<TM, D, kFp8> products{pl, smem_u, tmem, bars, ctrl, s};
        const bool issues = (warp & 3) == 0;
        const int count = pl.count(s);
        Ring vr{2, pl.two ? 0 : s, 0};
        int kslot = pl.two ? 0 : s;
        if (issues && count > 0 && elect()) {
            wait(bars + 8 * kQFull, 0, &ctrl->dead);
            if (s == 1) wait(bars + 8 * kStart, 0, &ctrl->dead);
            products.qk(0);
        }
        __syncwarp();
        for (int i = 0; i < count; ++i) {
            const int j = pl.tile(s, i);
            const int nkeys = j < pl.cached ? min(kTK, x.hi - x.lo - j * kTK) : x.live;
            const bool masked = nkeys < kTK;
            // the keys of the tile that the row sees (a masked tile's)
            uint64_t see0 = nkeys >= 64 ? ~0ull : (1ull << nkeys) - 1;
            uint64_t see1 = nkeys >= 128 ? ~0ull : nkeys > 64 ? (1ull << (nkeys - 64)) - 1 : 0;
            if (j >= pl.cached) see0 &= word;
            wait(bars + 8 * (kSFull + s), (uint32_t)i & 1u, &ctrl->dead);
            tc_after();
            if (!idle) {
                Scores sc{tS, scale, nullptr, nullptr, 0.f, see0, see1};
                float vref = 1.f;
                bool scaled = masked;
                if constexpr (kFp8) {
                    const float kref = ctrl->kref[kslot];
                    vref = ctrl->vref[kslot];
                    if (kref != 0.f)
                        sc.scale *= kref;
                    else
                        sc.k4 = reinterpret_cast<const float4*>(ks + kslot * kTK);
                    if (!ctrl->vplain[kslot]) {
                        wait(bars + 8 * (kVFull + vr.slot), vr.phase, &ctrl->dead);   // the values' scales
                        sc.v4 = reinterpret_cast<const float4*>(vs + vr.slot * kTK);
                        sc.vinv = pow2_inverse(vref);
                    }
                    scaled = scaled || sc.k4;
                    __syncwarp();
                }
                softmax_tile<TM, D, kFp8>(sc, tO, vref, scaled, i == 0, st);
            }
            tc_before();
            __syncwarp();
            if (lane == 0) {
                arrive(bars + 8 * (kPFull + s));
                if (s == 0 && i == 0) arrive(bars + 8 * kStart);
            }
            if (issues && elect()) {
                products.pv(i);
                if (i + 1 < count) products.qk(i + 1);
            }
            __syncwarp();
            // ring places of the stream's next tile
            vr.next();
            if (!pl.two) vr.next();
            kslot += pl.two ? 1 : 2;
            if (kslot >= 3) kslot -= 3;
        }
        if (count > 0) wait(bars + 8 * (kOFull + s), 0, &ctrl->dead);
        if (ctrl->dead) {   // what was issued has to be complete before TMEM is freed
            const int64_t t0 = clock64();
            while (count > 0 && !try_wait(bars + 8 * (kOFull + s), 0) && clock64() - t0 < kGiveUpClocks) {
            }
        }
        tc_after();
    }
    soft_sync();

    // ---- the end: rows of one stream, or of both merged through shared memory
    float* other = reinterpret_cast<float*>(smem);   // [D][128] of stream 1, then m, l, vref
    const uint32_t tO = tmem + lanes + 2 * kTK + s * D;
    if (!pl.two && warp >= 4 && pl.count(1) > 0) {
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
            float f[32];
            tm_ld32(tO + c * 32, f);
#pragma unroll
            for (int u = 0; u < 32; ++u) other[(c * 32 + u) * 128 + (tid & 127)] = f[u];
        }
        other[D * 128 + (tid & 127)] = st.m;
        other[(D + 1) * 128 + (tid & 127)] = st.l;
        other[(D + 2) * 128 + (tid & 127)] = st.vref;
    }
    soft_sync();
    const bool dead = ctrl->dead != 0;
    {
        // with one row tile, stream 1 has the second one's rows here: all dead
        const int row = row0 + 128 * s + (tid & 127);
        const bool join = !pl.two && s == 0 && pl.count(1) > 0;
        float a0 = 1.f, a1 = 0.f, M = st.m, den = st.l;
        if (join) {
            const float m1 = other[D * 128 + tid], l1 = other[(D + 1) * 128 + tid];
            M = fmaxf(st.m, m1);
            const float ref = M == -INFINITY ? 0.f : M;
            a0 = st.m == -INFINITY ? 1.f : ex2(st.m - ref);   // (a stream that saw no key has sums 0, or NaN)
            a1 = m1 == -INFINITY ? 1.f : ex2(m1 - ref);
            den = a0 * st.l + a1 * l1;
            if (kFp8) a1 *= other[(D + 2) * 128 + tid];
        }
        if (kFp8) a0 *= st.vref;
        if (pl.n == 0) den = 0.f;
        bool any = den != 0.f;   // NaN where a score was
        if (row >= last_row) any = false;
        float inv = any ? 1.f / den : 0.f;
        float lse = any ? (M + log2f(den)) * kLn2 : -INFINITY;
        if (dead) any = true, inv = lse = __uint_as_float(0x7fc00000u);
        if (dead && tid == 0) atomicAdd(&g_gave_up, 1u);
        const bool bad = ctrl->bad != 0 && pl.n > pl.cached;
        const int t = row / p.G;
        const int64_t at = ((int64_t)x.b * p.T + t) * p.Hq + x.hk * p.G + (row - t * p.G);
        const bool store = row < rows;
        char* dst;
        int kind = p.out_dtype;
        if (p.po) {
            dst = reinterpret_cast<char*>(p.po + (at * p.shards + r) * D);
            kind = LSE_MERGE_F32;
            if (store) p.pl[at * p.shards + r] = lse;
        } else {
            dst = p.out + at * D * (int64_t)(kind == LSE_MERGE_F32 ? 4 : 2);
            if (store) p.out_lse[at] = lse;
        }
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
            float f[32];
            __syncwarp();
            if (pl.n > 0) {
                tm_ld32(tO + c * 32, f);
            } else {
#pragma unroll
                for (int u = 0; u < 32; ++u) f[u] = 0.f;
            }
            if (!store) continue;
#pragma unroll
            for (int u = 0; u < 32; ++u) f[u] *= a0;
            if (join) {
#pragma unroll
                for (int u = 0; u < 32; ++u) f[u] = fmaf(a1, other[(c * 32 + u) * 128 + tid], f[u]);
            }
            if (bad) {
                const char* v = p.vd + x.b * p.vd_b + x.hk * p.vd_h;
                for (int key = 0; key < x.live; ++key) {
                    if (!(word >> key & 1)) continue;
#pragma unroll
                    for (int u = 0; u < 32; ++u) {
                        const float e = (float)*reinterpret_cast<const T*>(v + key * p.vd_t + (c * 32 + u) * 2);
                        if (!(fabsf(e) <= 3.402823466e38f)) f[u] += e;
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < 32; ++u) f[u] = any ? f[u] * inv : 0.f;
            if (kind == LSE_MERGE_F32) {
                float4* o = reinterpret_cast<float4*>(dst + c * 128);
#pragma unroll
                for (int u = 0; u < 8; ++u) o[u] = make_float4(f[4 * u], f[4 * u + 1], f[4 * u + 2], f[4 * u + 3]);
            } else {
                uint4* o = reinterpret_cast<uint4*>(dst + c * 64);
                const bool half = kind == LSE_MERGE_F16;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float a = f[8 * u + 2 * e], b = f[8 * u + 2 * e + 1];
                        w[e] = half ? Mma<__half>::pack(a, b) : Mma<__nv_bfloat16>::pack(a, b);
                    }
                    o[u] = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
        }
    }
    tc_before();
    soft_sync();
    tc_after();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

using WideFn = void (*)(TreeParams);
template <typename T>
WideFn pick(int D, bool fp8) {
    if (D == 64) return fp8 ? tree_wide_kernel<T, 64, true> : tree_wide_kernel<T, 64, false>;
    return fp8 ? tree_wide_kernel<T, 128, true> : tree_wide_kernel<T, 128, false>;
}

}  // namespace

cudaError_t launch_tree_wide(const TreeParams& p, int dtype, bool fp8, int out_dtype, int B, int Hkv, int D, bool pdl,
                             cudaStream_t stream) {
    const WideFn fn = dtype == LSE_MERGE_F16 ? pick<__half>(D, fp8) : pick<__nv_bfloat16>(D, fp8);
    const int smem = D == 64 ? Lay<64>::kBytes : Lay<128>::kBytes;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(fn), smem);
    if (e != cudaSuccess) return e;
    TreeParams q = p;
    q.row_tiles = (p.T * p.G + 255) / 256;
    q.out_dtype = out_dtype;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(q.row_tiles * p.R), (unsigned)Hkv, (unsigned)B);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, fn, q);
}

}  // namespace attn
}  // namespace lsem

extern "C" {

int lse_merge_tree_status(uint32_t* gave_up) {
    if (!gave_up) return LSE_MERGE_ENULL;
    const cudaError_t e = cudaMemcpyFromSymbol(gave_up, lsem::attn::g_gave_up, sizeof *gave_up);
    if (e == cudaSuccess) return LSE_MERGE_OK;
    lsem::set_last_cuda_error((int)e);
    (void)cudaGetLastError();
    return LSE_MERGE_ECUDA;
}

}  // extern "C"
