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
// lane; one thread of each also issues the stream's products), warps 8-11 bring
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

constexpr int kThreads = 12 * 32;
constexpr int kTK = 128;                    // keys per tile
constexpr uint64_t kGiveUpNs = 2000000000;  // longest wait for another warp

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
// Wait for phase `parity`; once a wait has run out, none waits any more.
__device__ __forceinline__ void wait(uint32_t bar, uint32_t parity, volatile int* dead) {
    if (try_wait(bar, parity)) return;
    const uint64_t t0 = global_ns();
    while (*dead == 0) {
        for (int i = 0; i < 16; ++i)
            if (try_wait(bar, parity)) return;
        if (global_ns() - t0 > kGiveUpNs) *dead = 1;
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
enum { kQFull = 0, kKFull = 1, kKEmpty = 4, kVFull = 7, kVEmpty = 10, kSFull = 13, kPFull = 15, kOFull = 17, kBars = 19 };

struct Ctrl {
    uint64_t bar[kBars];
    uint32_t tmem;
    int dead;
    int bad;            // a value of the drafts is no number
    float vref[2];      // of the weights, by value slot
    float top[2][4];
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

// Item i of the loaders' order K0, K1, V0, K2, V1, ..., V(n-1): tile and kind.
__device__ __forceinline__ void item_of(int i, int n, int& j, bool& value) {
    if (i == 0) {
        j = 0, value = false;
    } else if (i == 2 * n - 1) {
        j = n - 1, value = true;
    } else {
        j = (i + 1) >> 1, value = !(i & 1);
        if (value) j -= 1;
    }
}

template <typename T, int D>
__device__ __forceinline__ void load16(const TreeParams& p, const Shard& x, const WidePlan& pl, unsigned char* smem,
                                       uint32_t smem_u, Ctrl* ctrl, uint32_t bars, int tid) {
    using L = Lay<D>;
    constexpr int CPR = D / 8, kRows = 128 / CPR, kPending = 3;
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
        int j;
        bool value;
        item_of(i, pl.n, j, value);
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
#pragma unroll 4
            for (int row = row0; row < kTK; row += kRows) {
                const bool ok = row < t.count;
                cp_async16(dst + L::at(row, ch), src + (t.key0 + (ok ? row : 0)) * stride, ok ? 16 : 0);
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
    constexpr int CPR = D / 16, N = kTK * CPR / 128, kRows = 128 / CPR;
    const int ch = tid % CPR, row0 = tid / CPR, items = 2 * pl.n, raws = pl.two ? 2 : 3, nks = pl.two ? 3 : 4;
    const int lane = tid & 31, warp = tid >> 5;
    Ring kr{2, 0, 1}, vr{2, 0, 1};
    float run = 1.17549435e-38f;   // the reference of the values' scales
    // raw slots 0 and 1 behind the tiles, 2 where the second tile of queries would be
    auto raw = [&](int i) -> uint32_t { return (uint32_t)(i < 2 ? 6 * L::kTile + i * L::kRaw : L::kTile) + tid * 16; };
    auto fetch = [&](int i, int slot) {
        if (i < items) {
            int j;
            bool value;
            item_of(i, pl.n, j, value);
            const Keys t = keys_of(p, x, pl, j);
            const char* src = (value ? t.v : t.k) + ch * 16;
            const int64_t stride = value ? t.vl : t.kl;
            const uint32_t dst = smem_u + raw(slot);
#pragma unroll
            for (int u = 0; u < N; ++u) {
                const int row = row0 + u * kRows;
                const bool ok = row < t.count;
                cp_async16(dst + u * 2048, src + (t.key0 + (ok ? row : 0)) * stride, ok ? 16 : 0);
            }
        }
        cp_commit();
    };
    const float* ksrc = p.ks + x.b * p.ks_b + x.hk * p.ks_h;
    const float* vsrc = p.vs + x.b * p.vs_b + x.hk * p.vs_h;
    auto scale_at = [&](const float* src, int64_t stride, int j) -> float {   // of key tid of tile j
        const int key = x.lo + j * kTK + tid;
        return j < pl.n && key < x.hi ? src[key * stride] : 0.f;
    };
    int rs = 0, item = 0;
    // the next item's codes -> f16 in place `r` of its ring
    auto convert = [&](bool value, Ring& r) {
        unsigned char* tile = smem + (value ? 4 + r.slot : 2 + r.slot) * L::kTile;
        const unsigned char* src = smem + raw(rs);
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const uint4 c = *reinterpret_cast<const uint4*>(src + u * 2048);
            const uint4 lo = make_uint4(e4m3x2_f16x2(c.x), e4m3x2_f16x2_hi(c.x), e4m3x2_f16x2(c.y), e4m3x2_f16x2_hi(c.y));
            const uint4 hi = make_uint4(e4m3x2_f16x2(c.z), e4m3x2_f16x2_hi(c.z), e4m3x2_f16x2(c.w), e4m3x2_f16x2_hi(c.w));
            const int row = row0 + u * kRows;
            // lanes of the upper half of a row store their two chunks the other
            // way round: 8 neighbours then hit 8 different groups of banks
            const int odd = ch >> 2 & 1;
            *reinterpret_cast<uint4*>(tile + L::at(row, 2 * ch + odd)) = odd ? hi : lo;
            *reinterpret_cast<uint4*>(tile + L::at(row, 2 * ch + 1 - odd)) = odd ? lo : hi;
        }
        fence_async();
        __syncwarp();
        if (lane == 0) arrive(bars + 8 * ((value ? kVFull : kKFull) + r.slot));
        r.next();
        fetch(item + raws, rs);
        ++item;
        if (++rs == raws) rs = 0;
    };
    auto landed = [&]() {
        if (pl.two)
            cp_wait<1>();
        else
            cp_wait<2>();
    };
    for (int i = 0; i < raws; ++i) fetch(i, i);
    // the scales come a whole tile ahead
    float ksc = scale_at(ksrc, p.ks_l, 0), vsc = scale_at(vsrc, p.vs_l, 0);
    for (int j = -1; j < pl.n; ++j) {
        if (j + 1 < pl.n) {
            landed();
            wait(bars + 8 * (kKEmpty + kr.slot), kr.phase, &ctrl->dead);
            ks[(j + 1) % nks * kTK + tid] = ksc;
            ksc = scale_at(ksrc, p.ks_l, j + 2);
            convert(false, kr);
        }
        if (j >= 0) {
            landed();
            wait(bars + 8 * (kVEmpty + vr.slot), vr.phase, &ctrl->dead);
            const uint32_t top = __reduce_max_sync(kFull, __float_as_uint(vsc));
            if (lane == 0) ctrl->top[j & 1][warp] = __uint_as_float(top);
            asm volatile("bar.sync 2, 128;" ::: "memory");
            const float* tp = ctrl->top[j & 1];
            run = fmaxf(run, pow2_below(fmaxf(fmaxf(tp[0], tp[1]), fmaxf(tp[2], tp[3]))));
            vs[vr.slot * kTK + tid] = vsc * pow2_inverse(run);
            if (tid == 0) ctrl->vref[vr.slot] = run;
            vsc = scale_at(vsrc, p.vs_l, j + 1);
            convert(true, vr);
        }
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
        wait(bars + 8 * (kKFull + slot), (uint32_t)(j / nk) & 1u, &ctrl->dead);
        tc_after();
        const uint32_t q = smem_u + (pl.two ? s : 0) * L::kTile;
        const uint32_t k = smem_u + (slot < 2 ? 2 + slot : 1) * L::kTile;
#pragma unroll
        for (int u = 0; u < D / 16; ++u) {
            const uint32_t off = (u >> 2) * L::kBlock + (u & 3) * 32;
            mma_ss(tmem + s * kTK, smem_desc(q + off, 16), smem_desc(k + off, 16), kIdQK, u > 0);
        }
        tc_commit(bars + 8 * (kKEmpty + slot));
        tc_commit(bars + 8 * (kSFull + s));
    }
    __device__ __forceinline__ void pv(int i) const {
        const int j = pl.tile(s, i), nv = kFp8 ? 2 : 3, slot = j % nv;
        wait(bars + 8 * (kVFull + slot), (uint32_t)(j / nv) & 1u, &ctrl->dead);
        wait(bars + 8 * (kPFull + s), (uint32_t)i & 1u, &ctrl->dead);
        tc_after();
        const uint32_t v = smem_u + (4 + slot) * L::kTile;
#pragma unroll
        for (int u = 0; u < kTK / 16; ++u)
            mma_ts(tmem + 2 * kTK + s * D, tmem + s * kTK + u * 8, smem_desc(v + u * 2048, L::kBlock), kIdPV,
                   i > 0 || u > 0);
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

// A row's running state: reference (log2 units, kLow .. kHigh below the maximum),
// sum of weights, and e4m3: the values' scale that O is relative to.
struct RowSum {
    float m, l, vref;
};
template <typename TM>
constexpr float kLow = std::is_same<TM, __half>::value ? 7.f : 0.f;
template <typename TM>
constexpr float kHigh = std::is_same<TM, __half>::value ? 14.f : 8.f;

// The weights of 32 scores f, their sum and the largest exponent.  kCareful: a
// mask, and the scaled score rounded before the reference is subtracted (a fused
// difference of numbers past 2^22 could lie far from that of the rounded ones,
// which the reference is made from).
template <typename TM, bool kFp8, bool kCareful>
__device__ __forceinline__ void weights32(const float (&f)[32], const float4* k4, const float4* v4, uint64_t scale2,
                                          uint64_t ref2, uint32_t see, uint64_t& sum, float& top, uint32_t* w) {
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        uint64_t k2[2] = {scale2, scale2};
        if constexpr (kFp8) {
            const float4 k = k4[u];
            k2[0] = pack2f(k.x, k.y), k2[1] = pack2f(k.z, k.w);
            mul2(k2[0], scale2);
            mul2(k2[1], scale2);
        }
        uint64_t e2[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint64_t a;
            float e0, e1;
            if constexpr (kCareful) {
                a = pack2f(f[4 * u + 2 * h], f[4 * u + 2 * h + 1]);
                mul2(a, k2[h]);
                asm("add.rn.f32x2 %0, %0, %1;" : "+l"(a) : "l"(ref2));
            } else {
                a = ref2;
                fma2(a, pack2f(f[4 * u + 2 * h], f[4 * u + 2 * h + 1]), k2[h]);
            }
            unpack2f(a, e0, e1);
            if (kCareful) {
                e0 = see >> (4 * u + 2 * h) & 1 ? e0 : -INFINITY;
                e1 = see >> (4 * u + 2 * h + 1) & 1 ? e1 : -INFINITY;
            }
            top = fmaxf(top, fmaxf(e0, e1));
            e2[h] = pack2f(ex2(e0), ex2(e1));
            asm("add.rn.f32x2 %0, %0, %1;" : "+l"(sum) : "l"(e2[h]));
        }
        if constexpr (kFp8) {
            const float4 v = v4[u];
            mul2(e2[0], pack2f(v.x, v.y));
            mul2(e2[1], pack2f(v.z, v.w));
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float e0, e1;
            unpack2f(e2[h], e0, e1);
            w[2 * u + h] = Mma<TM>::pack(e0, e1);
        }
    }
}

// S of one tile (at tS) -> P over it.  The weights are taken relative to the
// reference that the earlier tiles left, in one pass over S; where the tile's
// maximum turns out to lie kHigh above it (always in a row's first tile, hardly
// ever later) the reference moves and the pass is made again.
template <typename TM, bool kFp8, bool kCareful>
__device__ __forceinline__ void softmax_pass(uint32_t tS, const float4* k4, const float4* v4, float scale, float ref,
                                             uint64_t see0, uint64_t see1, float& l, float& top, uint32_t* w) {
    const uint64_t scale2 = pack2f(scale, scale), ref2 = pack2f(-ref, -ref);
    uint64_t sum = 0;
    float fa[32], fb[32];
    tm_get32(tS, fa);
#pragma unroll
    for (int c = 0; c < 4; c += 2) {
        tm_wait32(fa);
        tm_get32(tS + 32 * c + 32, fb);
        weights32<TM, kFp8, kCareful>(fa, k4 + 8 * c, v4 + 8 * c, scale2, ref2, (uint32_t)(c ? see1 : see0), sum, top,
                                      w + 16 * c);
        tm_wait32(fb);
        if (c == 0) tm_get32(tS + 64, fa);
        weights32<TM, kFp8, kCareful>(fb, k4 + 8 * c + 8, v4 + 8 * c + 8, scale2, ref2,
                                      (uint32_t)((c ? see1 : see0) >> 32), sum, top, w + 16 * c + 16);
    }
    float s0, s1;
    unpack2f(sum, s0, s1);
    l = s0 + s1;
}

template <typename TM, int D, bool kFp8>
__device__ __forceinline__ void softmax_tile(uint32_t tS, uint32_t tO, const float4* k4, const float4* v4, float vref,
                                             float scale, bool masked, uint64_t see0, uint64_t see1, bool first,
                                             RowSum& st) {
    uint32_t w[kTK / 2];
    float down = 1.f, l;
    for (;;) {
        const float ref = st.m == -INFINITY ? 0.f : st.m;
        float top = -INFINITY;
        if (masked || __any_sync(kFull, fabsf(ref) > 4194304.f))
            softmax_pass<TM, kFp8, true>(tS, k4, v4, scale, ref, see0, see1, l, top, w);
        else
            softmax_pass<TM, kFp8, false>(tS, k4, v4, scale, ref, see0, see1, l, top, w);
        const float next = top + ref - kLow<TM>;
        const bool move = st.m == -INFINITY ? top != -INFINITY : top > kHigh<TM> && next != st.m;
        if (!__any_sync(kFull, move)) break;
        if (move) {
            down *= ex2(st.m - next);   // 0 at first
            st.m = next;
        }
    }
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
        tm_put32(tS + 32 * c, f);
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
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (warp == 8) {
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
    float* ks = reinterpret_cast<float*>(pl.two ? smem + L::kCtrl + 256 : smem + L::kTile + L::kRaw);
    float* vs = ks + (pl.two ? 3 : 4) * kTK;
    if (tid == 0) {
        auto init = [&](int b, int n) {
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bars + 8 * b), "r"(n) : "memory");
        };
        const int users = pl.two ? 2 : 1;   // streams that read a tile
        init(kQFull, 8);
        for (int i = 0; i < 3; ++i) {
            init(kKFull + i, 4), init(kKEmpty + i, users);
            init(kVFull + i, 4), init(kVEmpty + i, users);
        }
        for (int s = 0; s < 2; ++s) init(kSFull + s, 1), init(kPFull + s, 4), init(kOFull + s, 1);
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
    RowSum st{-INFINITY, 0.f, 1.17549435e-38f};
    uint64_t word = 0;

    if (warp >= 8) {
        if constexpr (kFp8)
            load8<D>(p, x, pl, smem, smem_u, ctrl, bars, ks, vs, tid - 256);
        else
            load16<T, D>(p, x, pl, smem, smem_u, ctrl, bars, tid - 256);
    } else {
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
        const bool issues = (warp & 3) == 0 && lane == 0;
        const int count = pl.count(s);
        Ring vr{2, pl.two ? 0 : s, 0};
        int kslot = pl.two ? 0 : s;
        if (issues && count > 0) {
            wait(bars + 8 * kQFull, 0, &ctrl->dead);
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
                const float4* k4 = reinterpret_cast<const float4*>(ks + kslot * kTK);
                const float4* v4 = reinterpret_cast<const float4*>(vs + vr.slot * kTK);
                float vref = 1.f;
                if constexpr (kFp8) {
                    wait(bars + 8 * (kVFull + vr.slot), vr.phase, &ctrl->dead);   // the values' scales
                    vref = ctrl->vref[vr.slot];
                    __syncwarp();
                }
                softmax_tile<TM, D, kFp8>(tS, tO, k4, v4, vref, scale, masked, see0, see1, i == 0, st);
            }
            tc_before();
            __syncwarp();
            if (lane == 0) arrive(bars + 8 * (kPFull + s));
            if (issues) {
                products.pv(i);
                if (i + 1 < count) products.qk(i + 1);
            }
            __syncwarp();
            // ring places of the stream's next tile
            vr.next();
            if (!pl.two) vr.next();
            kslot += pl.two ? 1 : 2;
            if (kslot >= (pl.two ? 3 : 4)) kslot -= pl.two ? 3 : 4;
        }
        if (count > 0) wait(bars + 8 * (kOFull + s), 0, &ctrl->dead);
        if (ctrl->dead) {   // what was issued has to be complete before TMEM is freed
            const uint64_t t0 = global_ns();
            while (count > 0 && !try_wait(bars + 8 * (kOFull + s), 0) && global_ns() - t0 < kGiveUpNs) {
            }
        }
        tc_after();
    }
    __syncthreads();

    // ---- the end: rows of one stream, or of both merged through shared memory
    float* other = reinterpret_cast<float*>(smem);   // [D][128] of stream 1, then m, l, vref
    const uint32_t tO = tmem + lanes + 2 * kTK + s * D;
    if (!pl.two && warp >= 4 && warp < 8 && pl.count(1) > 0) {
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
    __syncthreads();
    const bool dead = ctrl->dead != 0;
    if (warp < 8) {
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
    __syncthreads();
    tc_after();
    if (warp == 8)
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
