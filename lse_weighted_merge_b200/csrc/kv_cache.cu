// kv_cache.cu -- an 8-bit KV cache: rows quantised as they are written, and
// read back.
//
// A row is the D elements of one token's key (or value) in one head.  Written:
// a = max |x| over its finite elements, scale = 2^e with e the smallest integer
// >= -126 such that a <= 448 * 2^e (448 is e4m3's largest value), codes =
// x / scale to the nearest e4m3.  The scale is a power of two, so the division
// is a product without a rounding and the only rounding is the one to e4m3
// (half a step, 2^-4 of the value); e4m3 is a floating type, so a scale that
// is up to twice the smallest possible one costs range at the bottom (2^-9 of
// 448 either way), not precision.  e is read off the bits of a: 448 = 1.75 * 2^8,
// so e = exponent(a) - 8, and one more where the mantissa is above 1.75.
//
// Both kernels are bound by memory, with 16 elements of a row per lane.  Writing
// 16 x 4096 tokens of 8 heads, D = 128, bf16, takes 66 to 71 us by GPU (5.8 to 6.1
// TB/s, 88 to 92 % of the measured copy rate).  With tests for infinities on every
// element it was bound by the compares (98 us): the maximum is taken over the
// magnitudes' bits, two 16-bit ones per instruction, and shows infinities and NaN
// by itself.  Four rows per group of lanes took 168 us (registers).  Reading them
// back: 62 us, the measured copy rate (8 codes per lane: 71 to 75; loads that stay
// in L1: 81).  Few rows are bound by the launch: 3.3 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>
#include <type_traits>

#include "device_common.cuh"
#include "kv_plan.h"
#include "lse_merge.h"
#include "plan.h"

namespace lsem {
namespace kv {
namespace {

struct KvParams {
    char* cache[2];        // k, v codes
    float* scale[2];
    char* x[2];            // k, v rows, read (quantize) or written (dequantize)
    const int32_t *start, *count, *select;
    int64_t c_b[2], c_h[2], c_l[2];   // byte strides of the caches
    int64_t s_b[2], s_h[2], s_l[2];   // element strides of the scales
    int64_t x_b[2], x_h[2], x_t[2];   // byte strides of the rows
    uint64_t div0, div1;              // constants of the divisions by n0 and n1
    uint32_t n0, n1, rows;            // rows = B * n1 * n0, (n1, n0) = (Hkv, T) or (T, Hkv)
    int heads_inner;                  // n0 is Hkv
    int L, T, S;
};

// Row i's sequence, head and token.
__device__ __forceinline__ void row_of(const KvParams& p, uint32_t i, int& b, int& h, int& j) {
    const uint32_t q0 = fastdiv(i, p.div0, p.n0), r0 = i - q0 * p.n0;
    const uint32_t q1 = fastdiv(q0, p.div1, p.n1), r1 = q0 - q1 * p.n1;
    b = (int)q1;
    h = (int)(p.heads_inner ? r0 : r1);
    j = (int)(p.heads_inner ? r1 : r0);
}

// Two codes from two fp32 values, |x| <= 448 or NaN (lo in the low byte).
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two codes as fp32 (exact).
__device__ __forceinline__ float2 from_e4m3x2(uint32_t c) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
    __half2 v;
    memcpy(&v, &h, 4);
    return __half22float2(v);
}

// 16 bytes, not kept in L1; volatile, so that it stays behind pdl_wait().
__device__ __forceinline__ uint4 ld16(const char* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
__device__ __forceinline__ uint2 ld8(const char* p) {
    uint2 v;
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}
// 16 elements of a row per lane, as two runs of 8 that lie D / 2 apart (so that a
// load of all lanes is contiguous).
template <typename T>
struct Run;
template <>
struct Run<float> {
    uint4 u[4];
    __device__ __forceinline__ void load(const char* p, int apart) {
        u[0] = ld16(p), u[1] = ld16(p + 16), u[2] = ld16(p + apart), u[3] = ld16(p + apart + 16);
    }
    // Bits of the largest magnitude (as integers: infinities and NaN are largest).
    __device__ __forceinline__ uint32_t top() const {
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            m = max(max(max(m, u[k].x & 0x7fffffffu), max(u[k].y & 0x7fffffffu, u[k].z & 0x7fffffffu)), u[k].w & 0x7fffffffu);
        return m;
    }
    __device__ static uint32_t join(uint32_t a, uint32_t b) { return max(a, b); }
    __device__ static uint32_t bits(uint32_t m) { return m; }
    __device__ __forceinline__ void get(float (&f)[16]) const {
#pragma unroll
        for (int k = 0; k < 4; ++k) Elem<float>::unpack(u[k], f + 4 * k);
    }
};
// 16-bit types: two magnitudes per 32-bit word.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <typename T>
struct Run16 {
    uint4 u[2];
    __device__ __forceinline__ void load(const char* p, int apart) { u[0] = ld16(p), u[1] = ld16(p + apart); }
    __device__ __forceinline__ uint32_t top() const {
        constexpr uint32_t kAbs = 0x7fff7fffu;
        const uint32_t a = max_u16x2(max_u16x2(u[0].x & kAbs, u[0].y & kAbs), max_u16x2(u[0].z & kAbs, u[0].w & kAbs));
        const uint32_t b = max_u16x2(max_u16x2(u[1].x & kAbs, u[1].y & kAbs), max_u16x2(u[1].z & kAbs, u[1].w & kAbs));
        return max_u16x2(a, b);
    }
    __device__ static uint32_t join(uint32_t a, uint32_t b) { return max_u16x2(a, b); }
    // fp32 bits of the larger of the two.
    __device__ static uint32_t bits(uint32_t m) {
        float f[2];
        Run16::unpack(max(m & 0xffffu, m >> 16), f);
        return __float_as_uint(f[0]);
    }
    __device__ static void unpack(uint32_t w, float* f) {
        if constexpr (std::is_same<T, __half>::value)
            unpack_f16x2(w, f);
        else
            unpack_bf16x2(w, f);
    }
    __device__ __forceinline__ void get(float (&f)[16]) const {
#pragma unroll
        for (int k = 0; k < 2; ++k) Elem<T>::unpack(u[k], f + 8 * k);
    }
};
template <>
struct Run<__half> : Run16<__half> {};
template <>
struct Run<__nv_bfloat16> : Run16<__nv_bfloat16> {};

// D / 16 lanes per row.  The maximum is taken over the magnitudes' bits, which is
// also how a row with elements that are no numbers is noticed: it takes a path of
// its own, and the others test nothing.
template <typename T, int D>
__global__ void __launch_bounds__(256) kv_quantize_kernel(const KvParams p) {
    constexpr int kLanes = D / 16, E = (int)sizeof(T);
    pdl_wait();
    pdl_release();
    const uint32_t i = blockIdx.x * (256u / kLanes) + threadIdx.x / kLanes;   // (threads may pass 32 bits, rows do not)
    const int lane = threadIdx.x % kLanes;
    if (i >= p.rows) return;   // whole groups of lanes: the shuffles below stay within one
    int b, h, j;
    row_of(p, i, b, h, j);
    const int pos = (int)min((int64_t)p.start[b] + j, (int64_t)INT32_MAX);
    const bool there = pos >= 0 && pos < p.L && (!p.count || j < p.count[b]);
    const int src = there && p.select ? p.select[(int64_t)b * p.T + j] : j;
    if (!there || src < 0 || src >= p.S) return;
    const unsigned group = ((1u << kLanes) - 1u) << ((threadIdx.x & 31) / kLanes * kLanes);
    Run<T> x[2];
#pragma unroll
    for (int s = 0; s < 2; ++s)
        x[s].load(p.x[s] + b * p.x_b[s] + h * p.x_h[s] + src * p.x_t[s] + lane * 8 * E, D / 2 * E);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        uint32_t m = x[s].top();
#pragma unroll
        for (int o = kLanes / 2; o; o >>= 1) m = Run<T>::join(m, __shfl_xor_sync(group, m, o));
        uint32_t bits = Run<T>::bits(m);
        float f[16];
        x[s].get(f);
        if (bits >= 0x7f800000u) {
            float a = 0.f;
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const float v = fabsf(f[k]);
                const bool fin = v <= 3.402823466e38f;
                f[k] = fin ? f[k] : __uint_as_float(0x7fc00000u);
                a = fin ? fmaxf(a, v) : a;
            }
#pragma unroll
            for (int o = kLanes / 2; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(group, a, o));
            bits = __float_as_uint(a);
        }
        int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u);
        e = max(e, -126);
        if (bits == 0) e = 0;
        const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
        char* to = p.cache[s] + b * p.c_b[s] + h * p.c_h[s] + pos * p.c_l[s] + lane * 8;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float* g = f + 8 * r;
            uint2 w;
            w.x = to_e4m3x2(g[0] * inv, g[1] * inv) | to_e4m3x2(g[2] * inv, g[3] * inv) << 16;
            w.y = to_e4m3x2(g[4] * inv, g[5] * inv) | to_e4m3x2(g[6] * inv, g[7] * inv) << 16;
            *reinterpret_cast<uint2*>(to + r * (D / 2)) = w;
        }
        if (lane == 0)
            p.scale[s][b * p.s_b[s] + h * p.s_h[s] + pos * p.s_l[s]] = __uint_as_float((uint32_t)(127 + e) << 23);
    }
}

// D / 16 lanes per row, the same two runs.
template <typename T, int D>
__global__ void __launch_bounds__(256) kv_dequantize_kernel(const KvParams p) {
    constexpr int kLanes = D / 16, E = (int)sizeof(T);
    pdl_wait();
    pdl_release();
    const uint32_t i = blockIdx.x * (256u / kLanes) + threadIdx.x / kLanes;   // (threads may pass 32 bits, rows do not)
    const int lane = threadIdx.x % kLanes;
    if (i >= p.rows) return;
    int b, h, j;
    row_of(p, i, b, h, j);
    const int pos = (int)min((int64_t)p.start[b] + j, (int64_t)INT32_MAX);
    const bool there = pos >= 0 && pos < p.L && (!p.count || j < p.count[b]);
    uint2 w[2][2] = {};
    float sc[2] = {0.f, 0.f};
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        if (there) {
            const char* from = p.cache[s] + b * p.c_b[s] + h * p.c_h[s] + pos * p.c_l[s] + lane * 8;
            w[s][0] = ld8(from);
            w[s][1] = ld8(from + D / 2);
            sc[s] = p.scale[s][b * p.s_b[s] + h * p.s_h[s] + pos * p.s_l[s]];
        }
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        char* to = p.x[s] + b * p.x_b[s] + h * p.x_h[s] + j * p.x_t[s] + lane * 8 * E;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float f[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 v = from_e4m3x2((k < 2 ? w[s][r].x : w[s][r].y) >> (16 * (k & 1)) & 0xffffu);
                f[2 * k] = v.x * sc[s];
                f[2 * k + 1] = v.y * sc[s];
            }
            store_vec<T, 8>(to + r * (D / 2) * E, f);
        }
    }
}

using KvFn = void (*)(KvParams);

template <typename T>
KvFn pick_d(bool write, int D) {
    if (write) return D == 64 ? kv_quantize_kernel<T, 64> : kv_quantize_kernel<T, 128>;
    return D == 64 ? kv_dequantize_kernel<T, 64> : kv_dequantize_kernel<T, 128>;
}
KvFn pick(bool write, int dtype, int D) {
    switch (dtype) {
        case LSE_MERGE_F32: return pick_d<float>(write, D);
        case LSE_MERGE_F16: return pick_d<__half>(write, D);
        default: return pick_d<__nv_bfloat16>(write, D);
    }
}

int launch(const lse_merge_kv_args* args, bool write, cudaStream_t stream) {
    if (!args) return LSE_MERGE_ENULL;
    const lse_merge_kv_args& a = *args;
    const int rc = check_kv_args(a, write);
    if (rc != LSE_MERGE_OK) return rc;
    const int e = elem_bytes(a.dtype);
    KvParams p{};
    p.cache[0] = static_cast<char*>(a.k_cache);
    p.cache[1] = static_cast<char*>(a.v_cache);
    p.scale[0] = a.k_scale;
    p.scale[1] = a.v_scale;
    p.x[0] = static_cast<char*>(a.k);
    p.x[1] = static_cast<char*>(a.v);
    p.start = a.start;
    p.count = a.count;
    p.select = a.select;
    p.c_b[0] = a.k_b, p.c_h[0] = a.k_h, p.c_l[0] = a.k_l;
    p.c_b[1] = a.v_b, p.c_h[1] = a.v_h, p.c_l[1] = a.v_l;
    p.s_b[0] = a.ks_b, p.s_h[0] = a.ks_h, p.s_l[0] = a.ks_l;
    p.s_b[1] = a.vs_b, p.s_h[1] = a.vs_h, p.s_l[1] = a.vs_l;
    p.x_b[0] = a.kx_b * e, p.x_h[0] = a.kx_h * e, p.x_t[0] = a.kx_t * e;
    p.x_b[1] = a.vx_b * e, p.x_h[1] = a.vx_h * e, p.x_t[1] = a.vx_t * e;
    p.L = a.L;
    p.T = a.T;
    p.S = a.S;
    // neighbouring groups of lanes take the rows that are neighbours in the
    // cache: tokens of a head, or heads of a token
    p.heads_inner = a.k_h < a.k_l;
    p.n0 = (uint32_t)(p.heads_inner ? a.Hkv : a.T);
    p.n1 = (uint32_t)(p.heads_inner ? a.T : a.Hkv);
    p.div0 = fastdiv_c(p.n0);
    p.div1 = fastdiv_c(p.n1);
    p.rows = (uint32_t)a.B * p.n0 * p.n1;
    const uint32_t per = 256u / (uint32_t)(a.D / 16);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((p.rows + per - 1) / per);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = kPdl ? 1 : 0;
    const cudaError_t err = cudaLaunchKernelEx(&cfg, pick(write, a.dtype, a.D), p);
    if (err != cudaSuccess) {
        set_last_cuda_error((int)err);
        (void)cudaGetLastError();
        return LSE_MERGE_ELAUNCH;
    }
    return LSE_MERGE_OK;
}

}  // namespace
}  // namespace kv
}  // namespace lsem

extern "C" {

int lse_merge_kv_quantize(const lse_merge_kv_args* args, lse_merge_stream_t stream) {
    return lsem::kv::launch(args, true, reinterpret_cast<cudaStream_t>(stream));
}

int lse_merge_kv_dequantize(const lse_merge_kv_args* args, lse_merge_stream_t stream) {
    return lsem::kv::launch(args, false, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
