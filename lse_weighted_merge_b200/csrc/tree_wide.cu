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
// lane), warps 8-15 bring the tiles, one thread of warps 16 and 17 each issues the
// products of a stream, in halves of a tile:
//   S = Q K^T   128 x 64, Q and K in shared memory (K-major, 128-byte swizzle)
//   O += P V    128 x D, P in TMEM over S (16 bits, half its columns), V in shared
//               memory as it lies in the cache (its D is the fast index: MN-major)
// TMEM: S0 | S1 (two buffers of 64 columns each) | O0 | O1.  While a softmax warp is
// in one half, the other buffer's S is made.  Weights are relative to a reference
// that lies below the row's maximum and hardly ever moves; where it does, the
// thread waits for the stream's last P V and scales its row of O.
//
// 16-bit tiles come by cp.async into the swizzled layout; the drafts are a tile of
// the last shard, the only one with a mask row by row.  e4m3 tiles come by cp.async
// as they are; each warp converts what it fetched to f16 (exact) and stores it
// swizzled.  q is scaled per row by a power of two.  Scales that are powers of two
// (as lse_merge_kv_quantize writes them) and near each other go into the f16 tiles,
// exactly; others multiply scores and weights one by one.  The values' scales are
// relative to a unit that changes where a tile's scales do not fit it; values that are
// all zeros (whose scale is 1) do not count.  Weights of a tile whose values' scales lie
// far apart are rounded with their scales, relative to the largest such product, so that
// a large value of little weight takes no precision from the others.  (Values up to
// 2^70 apart in one call are held.)  The drafts of an e4m3 cache, whose
// products are of another type, are a launch of their own; a lone cached shard
// joins their partial.  Weights are rounded to the tiles' type (a tensor core product
// takes one type: f16 for e4m3 and f16 caches, bf16 for a bf16 one), their sums are
// of the unrounded ones.  Keys past the shard's end are zeros, so that no value
// there, whatever it is, meets a weight of 0.
//
// Measured on B200, 16 trees of 64 drafts, 32 heads over 8, D = 128, 8192 e4m3 tokens:
// 226 to 228 us, 603 to 609 TFLOP/s (the rows16 kernel: 913; scales that are no powers
// of two: 337; a row of zeros of another size every 50 tokens: 267); 16 trees of 16
// over 4096 bf16 tokens: 58 to 66 us, 4.2 to 4.6 TB/s (186). The exponentials (16 per
// clock and SM) and the tensor cores bound a tile of 128 rows and 128 keys at 1024
// clocks alike; a softmax warp takes about 2500 clocks for a half, of which the
// exponentials are 512: its own chain of barrier, TMEM load, weights, TMEM store and
// barrier, not a unit, is what is left (no unit is busy more than 30 % of the time).
// Taking the exponentials out saves 19 %, the products 7 %, the conversion 5 %. Two
// threads per row (16 softmax warps) gave 236 us, halves of 128 keys with one buffer
// 207 instead of 199 for the cached part, a prefetch into L2 four tiles ahead nothing.
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
constexpr int kThreads = (8 + kLoadWarps + 4) * 32;
// Registers per thread of the softmax, loading and issuing warps: together at most
// what the block is launched with.
constexpr int kSoftRegs = 144, kLoadRegs = 80, kIssueRegs = 32, kLaunchRegs = 96;
static_assert(256 * kSoftRegs + kLoadWarps * 32 * kLoadRegs + 128 * kIssueRegs <= kThreads * kLaunchRegs &&
              kThreads * kLaunchRegs <= 65536 && kThreads * (kLaunchRegs + 8) > 65536, "registers");
constexpr int kTK = 128;                    // keys per tile
constexpr int kHK = 64;                     // keys per step of a stream: half a tile
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
__device__ __forceinline__ float4 lds4(uint32_t at) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ float2 lds2(uint32_t at) {
    float2 v;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
    return v;
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
    static constexpr int kScales = kCtrl + 384;     // rings of scales, behind the control block
    static constexpr int kBytes = kScales + 5 * 512;
    // byte offset of 16-byte chunk ch of row
    __device__ static uint32_t at(int row, int ch) {
        return (uint32_t)((ch >> 3) * kBlock + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
    }
};

// Barriers, 8 bytes each, at the control block: S, P and the end of a P V by stream
// and half, the end of all products by stream.  A wait names a phase by its parity, so
// it must never be made while the phase before is still open: whoever waits for P V of
// a half knows from S of that half or the next, issued behind them, that the P V of
// two halves before, the barrier's phase before, is complete.
enum { kQFull = 0, kKFull = 1, kKEmpty = 4, kVFull = 7, kVEmpty = 10, kSFull = 13, kPFull = 17, kODone = 21, kEnd = 25, kBars = 27 };

struct Ctrl {
    uint64_t bar[kBars];
    uint32_t tmem;
    int dead;
    int bad;            // a value of the drafts is no number
    // e4m3, known with a tile's keys: the power of two that the values are relative to,
    // the Values they are, and the power of two that the keys were scaled by (0: their
    // scores still need the scales); by tile, these three
    float4 tile[3];
};
static_assert(sizeof(Ctrl) <= 384, "control block");

// e4m3: the values of a tile are codes times scale / unit, or codes whose scales (at most
// 2 units) multiply the weights, or all zeros.
enum Values { kScaled = 0, kCodes = 1, kZeros = 2 };
// The scales that go into the tile are powers of two in [unit * kFloor, unit * kCeil]: f16
// has codes times these exactly, and weights alone, rounded to f16, are precise enough.
constexpr float kFloor = 0.00390625f, kCeil = 128.f;

// How a CTA's tiles are laid out in time: the same for all roles.
struct WidePlan {
    bool two;        // two row tiles
    int n;           // key tiles
    int cached;      // of them over the cache; the last may be the drafts
    int len, live;   // keys of the shard, drafts
    __device__ __forceinline__ int count(int s) const { return two ? n : (n + 1 - s) >> 1; }
    __device__ __forceinline__ int tile(int s, int i) const { return two ? i : 2 * i + s; }
    __device__ __forceinline__ int keys(int j) const { return j < cached ? min(kTK, len - j * kTK) : live; }
};

// The halves of a stream's tiles, without those that have no key.
struct Halves {
    const WidePlan& pl;
    int s, i, half, seq;
    __device__ __forceinline__ Halves(const WidePlan& pl_, int s_) : pl(pl_), s(s_), i(0), half(0), seq(0) {}
    __device__ __forceinline__ bool more() const { return i < pl.count(s); }
    __device__ __forceinline__ int tile() const { return pl.tile(s, i); }
    __device__ __forceinline__ bool ends_tile() const { return half == 1 || pl.keys(tile()) <= kHK; }
    __device__ __forceinline__ void next() {
        if (ends_tile())
            ++i, half = 0;
        else
            half = 1;
        ++seq;
    }
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

// The loaders bring K0, V0, K1, V1, ...
template <typename T, int D>
__device__ __forceinline__ void load16(const TreeParams& p, const Shard& x, const WidePlan& pl, unsigned char* smem,
                                       uint32_t smem_u, Ctrl* ctrl, uint32_t bars, int tid) {
    using L = Lay<D>;
    constexpr int CPR = D / 8, kRows = kLoadWarps * 32 / CPR, kPending = 3;
    const int ch = tid % CPR, row0 = tid / CPR, items = 2 * pl.n;
    Ring kr{pl.two ? 2 : 3, 0, 1}, vr{3, 0, 1};
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
                if (row < t.count) u = __ldcg(reinterpret_cast<const uint4*>(src + row * stride));
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
    // (nothing past the end is fetched: the merge of the streams reuses the space)
    auto fetch = [&](Source& f, uint32_t dst, bool more) {
#pragma unroll
        for (int u = 0; more && u < N; ++u) {
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
            const float* at = src;
            if (key + 96 < hi) {
#pragma unroll
                for (int e = 0; e < 4; ++e, at += 32 * stride) v[e] = __ldcg(at);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e, at += 32 * stride) v[e] = key + 32 * e < hi ? __ldcg(at) : 0.f;
            }
            src = at;
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
            return __all_sync(kFull, (frac & 0x807fffffu) == 0);
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
    for (int j = 0; j < ahead; ++j) {
        fetch(k, raw(0, j), j < pl.n);
        fetch(v, raw(1, j), j < pl.n);
    }
    Ring kr{2, 0, 1}, vr{2, 0, 1};
    float base = 0.f, unit = 1.f;   // what scaled values are relative to, this tile's
    Scales sk{p.ks + x.b * p.ks_b + x.hk * p.ks_h + (x.lo + lane) * p.ks_l, p.ks_l, x.lo + lane, {}};
    Scales sv{p.vs + x.b * p.vs_b + x.hk * p.vs_h + (x.lo + lane) * p.vs_l, p.vs_l, x.lo + lane, {}};
    sk.next(x.hi);
    sv.next(x.hi);
    int kslot = 0;
    // the first warp keeps the scales that are not in the tile
    auto keep = [&](float* at, const Scales& sc, float inv) {
        if (warp != 0) return;
#pragma unroll
        for (int e = 0; e < 4; ++e) at[lane + 32 * e] = sc.v[e] * inv;
    };
    for (int j = 0; j < pl.n; ++j) {
        // f16 has codes * 2^-15 .. 1 exactly: scales that are powers of two go into the tile
        float kbig, vbig, small;
        bool kplain = sk.survey(kbig, small);
        kplain = kplain && small >= kbig * 3.0517578e-05f && kbig >= 1.17549435e-38f && kbig <= 8.507059e37f;
        bool pow2 = sv.survey(vbig, small);
        auto fits = [&]() { return pow2 && small >= base * kFloor && vbig <= base * kCeil; };
        auto compact = [&]() { return pow2 && small >= vbig * kFloor && vbig >= 7.7037198e-34f && vbig <= 1.2980742e33f; };
        int form = kScaled;
        if (vbig == 0.f || !fits()) {
            // Values that are all zeros do not count: of those whose scales stand out (in the
            // first tile, those of 1 as well, which lse_merge_kv_quantize gives them), every
            // warp looks at the codes (for itself: it happens seldom).
            const float low = base * kFloor, high = fminf(base != 0.f ? base * kCeil : 0.999f, small / kFloor);
            if (vbig > high || small < low) {
#pragma unroll 1
                for (int e = 0; e < 4; ++e) {
                    float mine = sv.v[0];
                    if (mine > high || (mine < low && mine != 0.f)) {
                        const char* at = x.vb + (int64_t)(x.lo + j * kTK + lane + 32 * e) * p.v_l;
                        uint32_t code = 0;
#pragma unroll
                        for (int c = 0; c < D / 16; ++c) {
                            const uint4 y = __ldcg(reinterpret_cast<const uint4*>(at) + c);
                            code |= y.x | y.y | y.z | y.w;
                        }
                        if ((code & 0x7f7f7f7fu) == 0) mine = 0.f;
                    }
                    sv.v[0] = sv.v[1], sv.v[1] = sv.v[2], sv.v[2] = sv.v[3], sv.v[3] = mine;
                }
                __syncwarp();
                pow2 = sv.survey(vbig, small);
            }
            if (vbig == 0.f)
                form = kZeros;
            else if (!fits()) {
                if (compact())
                    base = vbig;
                else
                    form = kCodes;
            }
        }
        if (form == kScaled) unit = base;
        if (form == kCodes && !(vbig < 2.f * unit && vbig >= 0.0625f * unit)) unit = pow2_below(vbig);
        landed();
        wait(bars + 8 * (kKEmpty + kr.slot), kr.phase, &ctrl->dead);
        convert(smem + (2 + kr.slot) * L::kTile, raw(0, j), kplain, sk, pow2_inverse(pow2_below(kbig)));
        // (the place of three tiles ago: the values of two tiles ago would not be
        // in if that tile's softmax were not over)
        if (!kplain) keep(ks + kslot * kTK, sk, 1.f);
        if (tid == 0) ctrl->tile[kslot] = make_float4(unit, (float)form, kplain ? kbig : 0.f, 0.f);
        __syncwarp();
        if (lane == 0) arrive(bars + 8 * (kKFull + kr.slot));
        kr.next();
        if (++kslot == 3) kslot = 0;
        sk.next(x.hi);
        fetch(k, raw(0, j), j + ahead < pl.n);
        landed();
        wait(bars + 8 * (kVEmpty + vr.slot), vr.phase, &ctrl->dead);
        convert(smem + (4 + vr.slot) * L::kTile, raw(1, j), form == kScaled, sv, pow2_inverse(unit));
        if (form == kCodes) keep(vs + vr.slot * kTK, sv, pow2_inverse(unit));
        __syncwarp();
        if (lane == 0) arrive(bars + 8 * (kVFull + vr.slot));
        vr.next();
        sv.next(x.hi);
        fetch(v, raw(1, j), j + ahead < pl.n);
    }
    cp_wait<0>();
}

// ------------------------------------------------------------ products

// All products of stream s, issued by one thread.  S and P are two buffers of 64
// columns: Q K^T of a half is issued two halves ahead of its P V, behind the P V that
// frees its buffer.
template <typename TM, int D, bool kFp8>
__device__ __forceinline__ void issue(const WidePlan& pl, int s, uint32_t smem_u, uint32_t tmem, Ctrl* ctrl,
                                      uint32_t bars) {
    using L = Lay<D>;
    constexpr uint32_t kIdQK = instr_desc<TM>(kHK, false), kIdPV = instr_desc<TM>(D, true);
    const int nk = kFp8 || pl.two ? 2 : 3, nv = kFp8 ? 2 : 3;
    const uint64_t q = smem_desc(smem_u + (pl.two ? s : 0) * L::kTile, 16);
    const uint32_t tS = tmem + s * kTK, tO = tmem + 2 * kTK + s * D;
    auto qk = [&](const Halves& h) {
        const int j = h.tile(), slot = j % nk;
        const uint64_t k = smem_desc(smem_u + (slot < 2 ? 2 + slot : 1) * L::kTile + h.half * kHK * 128, 16);
        wait(bars + 8 * (kKFull + slot), (uint32_t)(j / nk) & 1u, &ctrl->dead);
        tc_after();
#pragma unroll
        for (int u = 0; u < D / 16; ++u) {   // (descriptors count in 16 bytes)
            const uint32_t off = ((u >> 2) * L::kBlock + (u & 3) * 32) >> 4;
            mma_ss(tS + (h.seq & 1) * kHK, q + off, k + off, kIdQK, u > 0);
        }
        tc_commit(bars + 8 * (kSFull + 2 * s + (h.seq & 1)));
        if (h.ends_tile()) tc_commit(bars + 8 * (kKEmpty + slot));
    };
    auto pv = [&](const Halves& h) {
        const int j = h.tile(), slot = j % nv;
        const uint64_t v = smem_desc(smem_u + (4 + slot) * L::kTile + h.half * kHK * 128, L::kBlock);
        wait(bars + 8 * (kVFull + slot), (uint32_t)(j / nv) & 1u, &ctrl->dead);
        wait(bars + 8 * (kPFull + 2 * s + (h.seq & 1)), (uint32_t)(h.seq >> 1) & 1u, &ctrl->dead);
        tc_after();
#pragma unroll
        for (int u = 0; u < kHK / 16; ++u)
            mma_ts(tO, tS + (h.seq & 1) * kHK + u * 8, v + (u * 2048 >> 4), kIdPV, h.seq > 0 || u > 0);
        tc_commit(bars + 8 * (kODone + 2 * s + (h.seq & 1)));
        if (h.ends_tile()) tc_commit(bars + 8 * (kVEmpty + slot));
    };
    Halves a(pl, s), b(pl, s);   // of Q K^T and of P V
    wait(bars + 8 * kQFull, 0, &ctrl->dead);
    for (int e = 0; e < 2 && a.more(); ++e, a.next()) qk(a);
    for (; b.more(); b.next()) {
        pv(b);
        if (a.more()) {
            qk(a);
            a.next();
        }
    }
    if (b.seq > 0) tc_commit(bars + 8 * (kEnd + s));   // behind all of the stream's products
}

// ------------------------------------------------------------ queries

// The warp's 32 query rows (lane's own at `src`, NULL: zeros) -> rows row0 .. row0 + 31
// of the tile (or nowhere); e4m3: scaled to at most 2^15 in f16, the inverse times the
// lane's `scale`.  A negative scale changes q's sign.  D / 8 lanes bring a row.
template <typename T, int D, bool kFp8>
__device__ __forceinline__ void load_queries(const char* src, unsigned char* tile, int row0, int lane, bool flip,
                                             float& scale) {
    constexpr int kLanes = D / 8, kRows = 32 / kLanes, N = 32 / kRows;
    const uint32_t sign = flip ? 0x80008000u : 0u;
    const int sub = lane / kLanes, ch = lane % kLanes;
    // 8 loads in flight: straight code that runs once per block costs more in
    // instruction fetches than a second round trip
#pragma unroll 1
    for (int b = 0; b < N; b += 8) {
        uint4 u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint64_t at = __shfl_sync(kFull, (uint64_t)src, (b + i) * kRows + sub);
            u[i] = make_uint4(0, 0, 0, 0);
            if (at) u[i] = __ldcg(reinterpret_cast<const uint4*>(at + ch * 16));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (kFp8) {
                float f[8], big = 0.f;
                Elem<T>::unpack(u[i], f);
#pragma unroll
                for (int e = 0; e < 8; ++e) big = fmaxf(big, fabsf(f[e]));
#pragma unroll
                for (int o = kLanes / 2; o; o >>= 1) big = fmaxf(big, __shfl_xor_sync(kFull, big, o));
                const float top = fminf(fmaxf(pow2_below(big), 7.888609e-31f), 8.507059e37f);
                const float up = 16384.f * pow2_inverse(top);
                u[i] = make_uint4(Mma<__half>::pack(f[0] * up, f[1] * up), Mma<__half>::pack(f[2] * up, f[3] * up),
                                  Mma<__half>::pack(f[4] * up, f[5] * up), Mma<__half>::pack(f[6] * up, f[7] * up));
                const float mine = __shfl_sync(kFull, top, lane % kRows * kLanes);
                if (lane / kRows == b + i) scale *= mine * (1.f / 16384.f);
            }
            if (tile)
                *reinterpret_cast<uint4*>(tile + Lay<D>::at(row0 + (b + i) * kRows + sub, ch)) =
                    make_uint4(u[i].x ^ sign, u[i].y ^ sign, u[i].z ^ sign, u[i].w ^ sign);
        }
    }
}

// ------------------------------------------------------------ softmax

// A row's running state: reference (log2 units), sum of weights, and e4m3: the gain of
// O, which is the sum of weight * scale * code * gain (0: none yet), and the largest
// weight * scale * gain so far.  The gain is 1 / unit of the tile: weights go into the
// product as they are, or times scale / unit.  Only where the latter are all below 2^3,
// so far and in this half, is it larger.  O is scaled where the gain changes.
struct RowSum {
    float m, l, gain, peak;
};
constexpr float kMostPeak = 3.0948501e26f;   // 2^88: O, up to 2^36 times that, stays finite
// Weights are watched as the largest sum of 4 of them.  A row's first reference
// lies kLow below its maximum.  Where the sum is past kHigh the reference rises by
// a power of two that leaves it at 2^kBase to 2^(kBase + 1), the largest weight at
// a quarter of that or more.  f16 weights so stay between 2^7 (which keeps 2^-21 of
// the largest at f16's 11 bits) and f16's 65504, a value's scale below 2 included.
template <typename TM>
struct Bounds {
    static constexpr bool kHalf = std::is_same<TM, __half>::value;
    static constexpr float kLow = kHalf ? 7.f : 0.f, kHigh = kHalf ? 32000.f : 1.0995116e12f;
    static constexpr int kBase = kHalf ? 9 : 2;
};

// The scores of a half tile: where, what multiplies them, which of them the row sees.
struct Scores {
    uint32_t at;
    float scale;             // of the row (and of all keys of the tile)
    bool each;               // not all are seen, or their scales differ
    // e4m3, shared-memory addresses: the scales of keys and of values that are not in the
    // tiles (or 0), and the tile's unit and Values
    uint32_t k4, v4, values;
    uint64_t see;
};

// Replace the scores by the scaled ones, -inf where not seen.
template <bool kFp8>
__device__ __forceinline__ void scale_scores(Scores& x) {
#pragma unroll 1
    for (int c = 0; c < kHK; c += 32) {
        float f[32];
        tm_ld32(x.at + c, f);
        const uint32_t see = (uint32_t)(x.see >> c);
#pragma unroll
        for (int u = 0; u < 32; u += 4) {
            float k[4] = {x.scale, x.scale, x.scale, x.scale};
            if (kFp8 && x.k4) {
                const float4 s = lds4(x.k4 + (c + u) * 4);
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
__device__ __forceinline__ float largest_score(const Scores& x) {
    float top = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < kHK; c += 32) {
        float f[32];
        tm_ld32(x.at + c, f);
#pragma unroll
        for (int u = 0; u < 32; u += 4) top = fmaxf(fmaxf(top, fmaxf(f[u], f[u + 1])), fmaxf(f[u + 2], f[u + 3]));
    }
    return top == -INFINITY ? top : top * x.scale;
}

// Scores -> weights relative to ref, with their sum l and the largest sum of 4, top.
__device__ __forceinline__ void weigh(float (&f)[64], float scale, float ref, float& l, float& top) {
    const uint64_t scale2 = pack2f(scale, scale), ref2 = pack2f(-ref, -ref);
    uint64_t sum[4] = {0, 0, 0, 0};
    top = 0.f;
    // in steps over 32, so that each step's latencies overlap
#pragma unroll
    for (int c = 0; c < 64; c += 32) {
#pragma unroll
        for (int u = c; u < c + 32; u += 2) {
            uint64_t a = ref2;
            fma2(a, pack2f(f[u], f[u + 1]), scale2);
            unpack2f(a, f[u], f[u + 1]);
        }
#pragma unroll
        for (int u = c; u < c + 32; ++u) f[u] = ex2(f[u]);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            uint64_t t = pack2f(f[c + 2 * u], f[c + 2 * u + 1]);
#pragma unroll
            for (int h = 8; h < 32; h += 8)
                asm("add.rn.f32x2 %0, %0, %1;" : "+l"(t) : "l"(pack2f(f[c + h + 2 * u], f[c + h + 2 * u + 1])));
            float t0, t1;
            unpack2f(t, t0, t1);
            top = fmaxf(top, fmaxf(t0, t1));
            asm("add.rn.f32x2 %0, %0, %1;" : "+l"(sum[u]) : "l"(t));
        }
    }
    float s[8];
#pragma unroll
    for (int u = 0; u < 4; ++u) unpack2f(sum[u], s[2 * u], s[2 * u + 1]);
    l = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
}

// S of a half tile -> P over it: one pass, made again with a higher reference in the
// few halves where weights leave their range.  `ready`: all rows of the warp have a
// reference.  The rare steps are short loops over TMEM, so that the instructions of
// all halves stay near.
template <typename TM, int D, bool kFp8>
__device__ __forceinline__ void softmax_half(Scores x, uint32_t tO, uint32_t o_done, int seq,
                                             volatile int* dead, bool& ready, RowSum& st) {
    using Bd = Bounds<TM>;
    float f[64], l, top, down = 1.f;
    float (&fa)[32] = *reinterpret_cast<float (*)[32]>(f), (&fb)[32] = *reinterpret_cast<float (*)[32]>(f + 32);
    if (x.each) scale_scores<kFp8>(x);
    if (!ready) {
        const float mx = largest_score(x);
        if (st.m == -INFINITY && mx != -INFINITY) st.m = mx - Bd::kLow;   // (its sums are 0 so far)
        ready = !__any_sync(kFull, st.m == -INFINITY);
    }
    for (int tries = 0;; ++tries) {
        tm_get32(x.at, fa);
        tm_get32(x.at + 32, fb);
        tm_wait32(fa);
        tm_wait32(fb);
        const float ref = st.m == -INFINITY ? 0.f : st.m;
        weigh(f, x.scale, ref, l, top);
        // where scores are so large that a fused difference could lie far from that of
        // the rounded scores, which the reference is made from, they are rounded first
        const bool large = !x.each && fabsf(ref) > 4194304.f;
        if (!__any_sync(kFull, top > Bd::kHigh || large) || tries == 3) break;
        if (__any_sync(kFull, large)) {
            scale_scores<kFp8>(x);
            x.each = true;
            continue;
        }
        float next = ref;
        if (top > Bd::kHigh)   // (past 2^24 the reference has steps above 1: by one at least)
            next += fmaxf((float)((int)(__float_as_uint(top) >> 23) - 127 - Bd::kBase), fabsf(ref) * 1.8e-7f);
        if (__any_sync(kFull, top == INFINITY)) {
            const float mx = largest_score(x);
            if (top == INFINITY) next = mx - Bd::kLow;
        }
        if (next != ref) {
            const float a = ex2(ref - next);
            down *= a;
            st.l *= a;
            st.m = next;
        }
    }
    if constexpr (kFp8) {
        const float2 values = lds2(x.values);   // (once more: registers are scarce)
        const float g = pow2_inverse(values.x);
        float most = top;
        if (x.v4) {
            most = 0.f;
#pragma unroll
            for (int u = 0; u < 64; u += 4) {
                const float4 v = lds4(x.v4 + u * 4);
                f[u] *= v.x, f[u + 1] *= v.y, f[u + 2] *= v.z, f[u + 3] *= v.w;
                most = fmaxf(fmaxf(most, fmaxf(f[u], f[u + 1])), fmaxf(f[u + 2], f[u + 3]));
            }
        }
        if (x.v4 || !__all_sync(kFull, st.gain == g)) {
            const float old = st.gain == 0.f ? g : st.gain;
            const float was = st.peak * down * (g * pow2_inverse(old));   // what O's largest part is at gain g
            float more = 1.f;
            if (values.y == (float)kZeros) {
                most = 0.f;
            } else if (was <= kMostPeak) {
                const float row = fmaxf(was, most);
                if (x.v4 && row < 8.f && row > 0.f)   // (at most 2^80, and the gain at most 2^120)
                    more = fminf(512.f * pow2_inverse(pow2_below(row)), fminf(1.2089258e24f, 1.3292280e36f * values.x));
                st.gain = g * more;
                down *= st.gain * pow2_inverse(old);
            } else {   // next to nothing beside what O has: left out
                more = 0.f;
            }
            most *= more;
            if (__any_sync(kFull, more != 1.f)) {
                tm_put32(x.at, fa);
                tm_put32(x.at + 32, fb);
#pragma unroll 1
                for (int c = 0; c < kHK; c += 32) {
                    tm_wait_st();
                    tm_ld32(x.at + c, fa);
#pragma unroll
                    for (int u = 0; u < 32; ++u) fa[u] *= more;
                    tm_put32(x.at + c, fa);
                }
                tm_wait_st();
                tm_get32(x.at, fa);
                tm_get32(x.at + 32, fb);
                tm_wait32(fa);
                tm_wait32(fb);
            }
        }
        st.peak = fmaxf(st.peak * down, most);
    }
#pragma unroll
    for (int u = 0; u < 32; ++u) f[u] = __uint_as_float(Mma<TM>::pack(f[2 * u], f[2 * u + 1]));
    tm_put32(x.at, fa);
    st.l += l;
    if (__any_sync(kFull, down != 1.f) && seq > 0) {
        wait(o_done + 8 * ((seq - 1) & 1), (uint32_t)((seq - 1) >> 1) & 1u, dead);   // P V of the half before is in
        tc_after();
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
            tm_ld32(tO + c, fa);
#pragma unroll
            for (int u = 0; u < 32; ++u) fa[u] *= down;
            tm_put32(tO + c, fa);
        }
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
    // The launch before a joining one is that of the drafts, and its blocks wait for
    // what precedes it before they let this one start: only their partials are still
    // to come, and are waited for at the end.
    if (!p.join) pdl_wait();
    pdl_release();

    const int block = blockIdx.x / p.row_tiles, row0 = (blockIdx.x - block * p.row_tiles) * 256, rows = p.T * p.G;
    const int r = p.r0 + block;
    const Shard x = shard_of(p, r, blockIdx.y, blockIdx.z);
    WidePlan pl;
    const int last_row = min(rows, x.live * p.G);   // rows from here on are dead
    pl.two = last_row - row0 > 128;
    pl.cached = last_row > row0 && !x.drafts ? (x.hi - x.lo + kTK - 1) / kTK : 0;
    pl.n = pl.cached + (last_row > row0 && (x.drafts || (p.fold && r == p.R - 1)) ? 1 : 0);
    pl.len = x.hi - x.lo, pl.live = x.live;
    // the scales' rings: keys' by tile, values' by slot
    float* ks = reinterpret_cast<float*>(smem + L::kScales);
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
        for (int i = 0; i < 4; ++i) init(kSFull + i, 1), init(kPFull + i, 4);
        for (int i = 0; i < 4; ++i) init(kODone + i, 1);
        for (int s = 0; s < 2; ++s) init(kEnd + s, 1);
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
    RowSum st{-INFINITY, 0.f, 0.f, 0.f};
    uint64_t word = 0;

    if (warp >= 8 + kLoadWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
        if (warp < 10 + kLoadWarps && elect()) issue<TM, D, kFp8>(pl, warp - 8 - kLoadWarps, smem_u, tmem, ctrl, bars);
        return;
    }
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
            load_queries<T, D, kFp8>(src, pl.two || s == 0 ? smem + (pl.two ? s : 0) * L::kTile : nullptr,
                                     (warp & 3) * 32, lane, p.scale_log2 < 0.f, scale);
            if (!kFp8 && (p.fold || x.drafts) && src) word = (uint64_t)__ldcg(p.tree + x.b * p.tree_b + row / p.G);
        }
        fence_async();
        __syncwarp();
        if (lane == 0) arrive(bars + 8 * kQFull);
        const bool idle = row - lane >= last_row;   // no live row in the warp
        const uint32_t tS = tmem + lanes + s * kTK, tO = tmem + lanes + 2 * kTK + s * D;
        const int count = pl.count(s), step = pl.two ? 1 : 2;
        const uint32_t s_full = bars + 8 * (kSFull + 2 * s), p_full = bars + 8 * (kPFull + 2 * s);
        int seq = 0, kslot = pl.two ? 0 : s;
        bool ready = false;   // all rows of the warp have a reference
        for (int i = 0; i < count; ++i) {
            const int j = pl.tile(s, i), keys = pl.keys(j);
            float tile_scale = scale;
#pragma unroll 1
            for (int half = 0; half * kHK < keys; ++half, ++seq) {
                const int buf = seq & 1;
                wait(s_full + 8 * buf, (uint32_t)(seq >> 1) & 1u, &ctrl->dead);
                tc_after();
                if (!idle) {
                    float4 info = make_float4(0.f, 0.f, 1.f, 0.f);
                    if constexpr (kFp8) {
                        info = lds4(smem_u32(&ctrl->tile[kslot]));
                        tile_scale = scale * info.z;
                    }
                    const int left = keys - half * kHK;
                    Scores sc{tS + buf * kHK, tile_scale, left < kHK || (!kFp8 && j >= pl.cached), 0, 0, smem_u32(&ctrl->tile[kslot]), ~0ull};
                    if (sc.each) {
                        if (left < kHK) sc.see = (1ull << left) - 1;
                        if (!kFp8 && j >= pl.cached) sc.see &= word;
                    }
                    if (kFp8 && info.z == 0.f) {
                        sc.scale = scale;
                        sc.k4 = smem_u32(ks + kslot * kTK + half * kHK);
                        sc.each = true;
                    }
                    if (kFp8 && info.y == (float)kCodes) {
                        wait(bars + 8 * (kVFull + j % 2), (uint32_t)(j / 2) & 1u, &ctrl->dead);   // their scales
                        sc.v4 = smem_u32(vs + j % 2 * kTK + half * kHK);
                        __syncwarp();
                    }
                    softmax_half<TM, D, kFp8>(sc, tO, bars + 8 * (kODone + 2 * s), seq, &ctrl->dead, ready, st);
                }
                tc_before();
                __syncwarp();
                if (lane == 0) arrive(p_full + 8 * buf);
            }
            kslot += step;
            if (kslot >= 3) kslot -= 3;
        }
        if (seq > 0) wait(bars + 8 * (kEnd + s), 0, &ctrl->dead);
        if (ctrl->dead) {   // what was issued has to be complete before TMEM is freed
            const int64_t t0 = clock64();
            while (seq > 0 && !try_wait(bars + 8 * (kEnd + s), 0) && clock64() - t0 < kGiveUpClocks) {
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
        other[(D + 2) * 128 + (tid & 127)] = st.gain;
    }
    soft_sync();
    const bool dead = ctrl->dead != 0;
    if (p.join) pdl_wait();
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
            const float gain = other[(D + 2) * 128 + tid];
            if (kFp8 && gain != 0.f) a1 /= gain;
        }
        if (kFp8 && st.gain != 0.f) a0 /= st.gain;
        if (pl.n == 0) den = 0.f;
        bool any = den != 0.f;   // NaN where a score was
        if (row >= last_row) any = false;
        float inv = any ? 1.f / den : 0.f;
        float lse = any ? (M + log2f(den)) * kLn2 : -INFINITY;
        if (dead) any = true, inv = lse = __uint_as_float(0x7fc00000u);
        if (dead && tid == 0) atomicAdd(&g_gave_up, 1u);
        const bool bad = !kFp8 && ctrl->bad != 0 && pl.n > pl.cached;
        const int t = row / p.G;
        const int64_t at = ((int64_t)x.b * p.T + t) * p.Hq + x.hk * p.G + (row - t * p.G);
        const bool store = row < rows;
        char* dst;
        int kind = p.out_dtype;
        // the drafts' shard, written by an earlier launch, joins the only other one here
        const float* joined = nullptr;
        float b0 = 1.f, b1 = 0.f;
        if (p.join && store) {
            joined = p.po + at * D;
            const float l1 = __ldcg(p.pl + at);
            const float mx = fmaxf(lse, l1), ref = mx == -INFINITY ? 0.f : mx;
            const float e0 = expf(lse - ref), e1 = expf(l1 - ref), total = e0 + e1;
            const bool seen = total != 0.f;   // NaN where a score was
            b0 = seen ? e0 / total : 0.f;
            b1 = seen ? e1 / total : 0.f;
            lse = seen ? mx + logf(total) : -INFINITY;
        }
        if (p.po && !p.join) {
            const int64_t place = p.shards > 1 ? at * p.shards + r : at;
            dst = reinterpret_cast<char*>(p.po + place * D);
            kind = LSE_MERGE_F32;
            if (store) p.pl[place] = lse;
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
            if (joined) {
#pragma unroll
                for (int u = 0; u < 32; u += 4) {
                    const float4 o = __ldcg(reinterpret_cast<const float4*>(joined + c * 32 + u));
                    f[u] = f[u] * b0 + o.x * b1, f[u + 1] = f[u + 1] * b0 + o.y * b1;
                    f[u + 2] = f[u + 2] * b0 + o.z * b1, f[u + 3] = f[u + 3] * b0 + o.w * b1;
                }
            }
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

cudaError_t launch_tree_wide(const TreeParams& p, int dtype, bool fp8, int shards, int out_dtype, int B, int Hkv, int D,
                             bool pdl, cudaStream_t stream) {
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
    cfg.gridDim = dim3((unsigned)(q.row_tiles * shards), (unsigned)Hkv, (unsigned)B);
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
