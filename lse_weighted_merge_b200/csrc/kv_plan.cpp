// kv_plan.cpp -- validation and geometry of the 8-bit cache's calls and of the
// attention over a cache and drafts.
#include "kv_plan.h"

#include <cstdint>

#include "plan.h"

namespace lsem {

namespace {

using i128 = __int128;

// Byte interval [lo, hi) of a buffer.
struct Span {
    uintptr_t lo;
    i128 hi;
};

bool overlap(const Span& a, const Span& b) { return (i128)a.lo < b.hi && (i128)b.lo < a.hi; }
bool aligned(const void* p, int a) { return ((uintptr_t)p % (uintptr_t)a) == 0; }

// One dimension of a strided tensor.
struct Dim {
    int64_t n, stride;
};

// Bytes from the first to past the last element of a tensor of rows of `row`
// contiguous elements; -1 for an extent past 2^62.
i128 span_bytes(const Dim (&d)[3], int64_t row, int elem) {
    i128 last = row;
    for (const Dim& x : d) last += (i128)(x.n - 1) * x.stride;
    last *= elem;
    return last > ((i128)1 << 62) ? (i128)-1 : last;
}

// Whether every element has an address of its own: by ascending stride, each
// dimension steps over all that the smaller ones reach.
bool distinct(const Dim (&d)[3], int64_t row) {
    Dim s[3] = {d[0], d[1], d[2]};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (s[j].stride < s[i].stride) {
                const Dim t = s[i];
                s[i] = s[j];
                s[j] = t;
            }
    i128 reach = row;
    for (const Dim& x : s) {
        if (x.n == 1) continue;
        if ((i128)x.stride < reach) return false;
        reach += (i128)(x.n - 1) * x.stride;
    }
    return true;
}

bool any_negative(const int64_t* s, int n) {
    for (int i = 0; i < n; ++i)
        if (s[i] < 0) return true;
    return false;
}

// The byte strides of a 16-byte accessed tensor are whole 16-byte multiples.
bool strides16(const int64_t* s, int n, int elem) {
    for (int i = 0; i < n; ++i)
        if ((s[i] % 16) * elem % 16 != 0) return false;
    return true;
}

Span span_of(const void* p, i128 bytes) { return Span{(uintptr_t)p, (i128)(uintptr_t)p + bytes}; }

// Fill sp[0..n-1] from pointers and byte counts; false for an extent that does not fit.
bool spans(Span* sp, const void* const* p, const i128* bytes, int n) {
    for (int i = 0; i < n; ++i) {
        if (bytes[i] < 0) return false;
        sp[i] = span_of(p[i], p[i] ? bytes[i] : 0);
    }
    return true;
}

// Whether a written span overlaps a read one or another written one (NULL
// pointers have empty spans at 0, which overlap nothing).
bool written_overlap(const Span* wr, int nw, const Span* rd, int nr) {
    for (int i = 0; i < nw; ++i) {
        for (int j = i + 1; j < nw; ++j)
            if (overlap(wr[i], wr[j])) return true;
        for (int j = 0; j < nr; ++j)
            if (overlap(wr[i], rd[j])) return true;
    }
    return false;
}

}  // namespace

int check_kv_args(const lse_merge_kv_args& a, bool write) {
    const int e = elem_bytes(a.dtype);
    if (e == 0) return LSE_MERGE_EDTYPE;
    if (a.B < 1 || a.Hkv < 1 || a.L < 1 || a.D < 1 || a.T < 1 || a.S < 1) return LSE_MERGE_EDIMS;
    if (!a.k_cache || !a.v_cache || !a.k_scale || !a.v_scale || !a.k || !a.v || !a.start)
        return LSE_MERGE_ENULL;
    if (!a.select && a.S != a.T) return LSE_MERGE_EDIMS;
    if (!write && a.select) return LSE_MERGE_EUNSUP;
    if (any_negative(&a.k_b, 18)) return LSE_MERGE_ESTRIDE;
    if (a.D != 64 && a.D != 128) return LSE_MERGE_EUNSUP;
    // row and token indexes of the kernels fit 31 bits
    if ((i128)a.B * a.Hkv * a.T > ((i128)1 << 30)) return LSE_MERGE_EDIMS;
    if (!aligned(a.k_cache, 16) || !aligned(a.v_cache, 16) || !aligned(a.k, 16) ||
        !aligned(a.v, 16) || !aligned(a.k_scale, 4) || !aligned(a.v_scale, 4) ||
        !aligned(a.start, 4) || !aligned(a.count, 4) || !aligned(a.select, 4))
        return LSE_MERGE_EALIGN;
    if (!strides16(&a.k_b, 6, 1) || !strides16(&a.kx_b, 6, e)) return LSE_MERGE_EALIGN;
    const Dim kc[3] = {{a.B, a.k_b}, {a.Hkv, a.k_h}, {a.L, a.k_l}};
    const Dim vc[3] = {{a.B, a.v_b}, {a.Hkv, a.v_h}, {a.L, a.v_l}};
    const Dim ks[3] = {{a.B, a.ks_b}, {a.Hkv, a.ks_h}, {a.L, a.ks_l}};
    const Dim vs[3] = {{a.B, a.vs_b}, {a.Hkv, a.vs_h}, {a.L, a.vs_l}};
    const Dim kx[3] = {{a.B, a.kx_b}, {a.Hkv, a.kx_h}, {a.S, a.kx_t}};
    const Dim vx[3] = {{a.B, a.vx_b}, {a.Hkv, a.vx_h}, {a.S, a.vx_t}};
    const void* pc[4] = {a.k_cache, a.v_cache, a.k_scale, a.v_scale};
    const i128 bc[4] = {span_bytes(kc, a.D, 1), span_bytes(vc, a.D, 1), span_bytes(ks, 1, 4),
                        span_bytes(vs, 1, 4)};
    const void* px[2] = {a.k, a.v};
    const i128 bx[2] = {span_bytes(kx, a.D, e), span_bytes(vx, a.D, e)};
    const void* pi[3] = {a.start, a.count, a.select};
    const i128 bi[3] = {(i128)a.B * 4, (i128)a.B * 4, (i128)a.B * a.T * 4};
    Span c[4], x[2], in[3];
    if (!spans(c, pc, bc, 4) || !spans(x, px, bx, 2) || !spans(in, pi, bi, 3)) return LSE_MERGE_EDIMS;
    // What is written overlaps nothing that is read.  Tensors of one side may
    // interleave (keys and values in one buffer); only equal ones are refused.
    for (int i = 0; i < 3; ++i)
        for (int j = 0; j < 4; ++j) {
            if (j < 2 && !write && overlap(in[i], x[j])) return LSE_MERGE_EALIAS;
            if (write && overlap(in[i], c[j])) return LSE_MERGE_EALIAS;
        }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 2; ++j)
            if (overlap(c[i], x[j])) return LSE_MERGE_EALIAS;
    if (write) {
        if (!distinct(kc, a.D) || !distinct(vc, a.D) || !distinct(ks, 1) || !distinct(vs, 1))
            return LSE_MERGE_ESTRIDE;
        if (a.k_cache == a.v_cache || a.k_scale == a.v_scale) return LSE_MERGE_EALIAS;
        for (int i = 0; i < 2; ++i)
            for (int j = 2; j < 4; ++j)
                if (overlap(c[i], c[j])) return LSE_MERGE_EALIAS;
    } else {
        if (!distinct(kx, a.D) || !distinct(vx, a.D)) return LSE_MERGE_ESTRIDE;
        if (a.k == a.v) return LSE_MERGE_EALIAS;
    }
    return LSE_MERGE_OK;
}

int tree_workspace(int B, int T, int Hq, int D, int R, bool drafts, TreePlan* plan) {
    if (B < 1 || T < 1 || Hq < 1 || D < 1 || R < 1) return LSE_MERGE_EDIMS;
    plan->shards = R + (drafts ? 1 : 0);
    plan->ws_l_off = plan->ws_bytes = 0;
    if (plan->shards > 1) {
        const i128 rows = (i128)B * T * Hq * plan->shards;
        const i128 l_off = (rows * D * 4 + 255) / 256 * 256;
        const i128 total = l_off + rows * 4;
        if (total > ((i128)1 << 62)) return LSE_MERGE_EDIMS;
        plan->ws_l_off = (int64_t)l_off;
        plan->ws_bytes = (int64_t)total;
    }
    return LSE_MERGE_OK;
}

// Shards of the cached keys: the R with the least modelled time on `sms` SMs.  Up to
// 16 query rows per KV head (rows16 kernel, two CTAs per SM, steps of 128 keys): a
// CTA's start and end take about as long as 5.5 steps, two CTAs on an SM take 1.35
// times as long as one, each shard adds to the merge.  (Measured for one sequence of
// 4096 e4m3 tokens, 8 KV heads: R = 1, 4, 8, 16, 32, 64 in 38.7, 16.8, 12.5, 10.8,
// 12.4, 20.8 us.)  More rows (wide kernel, one CTA per SM, tiles of 128 keys): start
// and end take about 3 tiles' time.  (4096 bf16 tokens under 20 rows: R = 1, 4, 8,
// 16, 32 in 54.6, 23.6, 17.5, 15.2, 22.9 us.)
int tree_default_splits(int B, int T, int Hq, int Hkv, int L, int D, int sms) {
    if (B < 1 || T < 1 || Hq < 1 || Hkv < 1 || L < 1 || D < 1 || sms < 1) return 1;
    const int64_t rows = (int64_t)T * (Hq / Hkv);
    int R = 1;
    if (rows > 16) {
        const int64_t units = (int64_t)B * Hkv * ((rows + 255) / 256), tiles = ((int64_t)L + 127) / 128;
        int64_t best = -1;
        for (int r = 1; r <= 64 && r <= tiles; ++r) {
            const int64_t cost = (units * r + sms - 1) / sms * ((tiles + r - 1) / r + 3);
            if (best < 0 || cost < best) best = cost, R = r;
        }
        return R;
    }
    const int64_t units = (int64_t)B * Hkv, steps = ((int64_t)L + 127) / 128;
    double best = -1;
    for (int r = 1; r <= 64 && r <= steps; ++r) {
        const int64_t ctas = units * r, waves = (ctas + 2 * (int64_t)sms - 1) / (2 * (int64_t)sms);
        const double each = 5.5 + (double)((steps + r - 1) / r);
        const double cost = (double)waves * each * (ctas > sms ? 1.35 : 1.0) + 0.04 * r;
        if (best < 0 || cost < best) best = cost, R = r;
    }
    return R;
}

int make_tree_plan(const lse_merge_tree_args& a, TreePlan* plan) {
    const int e = elem_bytes(a.dtype), ob = elem_bytes(a.out_dtype);
    const bool fp8 = a.cache_dtype == LSE_MERGE_E4M3, drafts = a.k_draft != nullptr;
    const int ce = fp8 ? 1 : e;
    if (e == 0 || ob == 0) return LSE_MERGE_EDTYPE;
    if (!fp8 && elem_bytes(a.cache_dtype) == 0) return LSE_MERGE_EDTYPE;
    if (a.B < 1 || a.T < 1 || a.Hq < 1 || a.Hkv < 1 || a.L < 1 || a.D < 1 || a.R < 1)
        return LSE_MERGE_EDIMS;
    if (!a.q || !a.k || !a.v || !a.out_o || !a.out_lse || !plan) return LSE_MERGE_ENULL;
    if (fp8 && (!a.k_scale || !a.v_scale)) return LSE_MERGE_ENULL;
    if (drafts && (!a.v_draft || !a.tree)) return LSE_MERGE_ENULL;
    if (any_negative(&a.q_b, 9)) return LSE_MERGE_ESTRIDE;
    if (fp8 && any_negative(&a.ks_b, 6)) return LSE_MERGE_ESTRIDE;
    if (drafts && any_negative(&a.kd_b, 7)) return LSE_MERGE_ESTRIDE;
    if (a.dtype == LSE_MERGE_F32 || (!fp8 && a.cache_dtype != a.dtype)) return LSE_MERGE_EUNSUP;
    if (a.D != 64 && a.D != 128) return LSE_MERGE_EUNSUP;
    if (a.Hq % a.Hkv != 0 || a.Hq / a.Hkv > 16 || a.T > LSE_MERGE_TREE_MAX_T) return LSE_MERGE_EUNSUP;
    if (a.B > 65535 || a.Hkv > 65535 || a.R > 65535) return LSE_MERGE_EDIMS;
    // 32-bit key indexes run past a shard's end, by up to 351 (the wide kernel's scales,
    // brought a tile ahead)
    if (a.L > INT32_MAX - 1024) return LSE_MERGE_EDIMS;
    // row indexes of the merge fit 30 bits
    if ((i128)a.B * a.T * a.Hq > ((i128)1 << 30)) return LSE_MERGE_EDIMS;
    // times log2(e) it stays finite (NaN fails too)
    if (!(a.scale <= 2.3e38f && a.scale >= -2.3e38f)) return LSE_MERGE_EDIMS;
    if (!aligned(a.q, 16) || !aligned(a.k, 16) || !aligned(a.v, 16) || !aligned(a.out_o, 16) ||
        !aligned(a.out_lse, 4) || !aligned(a.kv_len, 4) || !aligned(a.draft_len, 4))
        return LSE_MERGE_EALIGN;
    if (!strides16(&a.q_b, 3, e) || !strides16(&a.k_b, 6, ce)) return LSE_MERGE_EALIGN;
    if (fp8 && (!aligned(a.k_scale, 4) || !aligned(a.v_scale, 4))) return LSE_MERGE_EALIGN;
    if (drafts && (!aligned(a.k_draft, 16) || !aligned(a.v_draft, 16) || !aligned(a.tree, 8) ||
                   !strides16(&a.kd_b, 6, e)))
        return LSE_MERGE_EALIGN;
    TreePlan p{};
    p.G = a.Hq / a.Hkv;
    p.rows = a.T * p.G;
    const int rc = tree_workspace(a.B, a.T, a.Hq, a.D, a.R, drafts, &p);
    if (rc != LSE_MERGE_OK) return rc;
    if (p.ws_bytes) {
        if (!a.workspace) return LSE_MERGE_ENULL;
        if (!aligned(a.workspace, 16)) return LSE_MERGE_EALIGN;
        if (a.workspace_bytes < p.ws_bytes) return LSE_MERGE_EDIMS;
    }
    const Dim qd[3] = {{a.B, a.q_b}, {a.T, a.q_t}, {a.Hq, a.q_h}};
    const Dim kc[3] = {{a.B, a.k_b}, {a.Hkv, a.k_h}, {a.L, a.k_l}};
    const Dim vc[3] = {{a.B, a.v_b}, {a.Hkv, a.v_h}, {a.L, a.v_l}};
    const Dim ks[3] = {{a.B, a.ks_b}, {a.Hkv, a.ks_h}, {a.L, a.ks_l}};
    const Dim vs[3] = {{a.B, a.vs_b}, {a.Hkv, a.vs_h}, {a.L, a.vs_l}};
    const Dim kd[3] = {{a.B, a.kd_b}, {a.Hkv, a.kd_h}, {a.T, a.kd_t}};
    const Dim vd[3] = {{a.B, a.vd_b}, {a.Hkv, a.vd_h}, {a.T, a.vd_t}};
    const Dim tr[3] = {{a.B, a.tree_b}, {1, 0}, {1, 0}};
    const i128 rows = (i128)a.B * a.T * a.Hq;
    const void* pr[10] = {a.q, a.k, a.v, fp8 ? a.k_scale : nullptr, fp8 ? a.v_scale : nullptr,
                          a.k_draft, drafts ? a.v_draft : nullptr, drafts ? a.tree : nullptr,
                          a.kv_len, a.draft_len};
    const i128 br[10] = {span_bytes(qd, a.D, e), span_bytes(kc, a.D, ce), span_bytes(vc, a.D, ce),
                         fp8 ? span_bytes(ks, 1, 4) : 0, fp8 ? span_bytes(vs, 1, 4) : 0,
                         drafts ? span_bytes(kd, a.D, e) : 0, drafts ? span_bytes(vd, a.D, e) : 0,
                         drafts ? span_bytes(tr, a.T, 8) : 0, (i128)a.B * 4, (i128)a.B * 4};
    const void* pw[3] = {a.out_o, a.out_lse, p.ws_bytes ? a.workspace : nullptr};
    const i128 bw[3] = {rows * a.D * ob, rows * 4, p.ws_bytes};
    Span rd[10], wr[3];
    if (!spans(rd, pr, br, 10) || !spans(wr, pw, bw, 3)) return LSE_MERGE_EDIMS;
    if (written_overlap(wr, 3, rd, 10)) return LSE_MERGE_EALIAS;
    *plan = p;
    return LSE_MERGE_OK;
}

}  // namespace lsem

extern "C" {

int lse_merge_tree_workspace_bytes(int B, int T, int Hq, int D, int R, int drafts, int64_t* bytes) {
    if (!bytes) return LSE_MERGE_ENULL;
    lsem::TreePlan p{};
    const int rc = lsem::tree_workspace(B, T, Hq, D, R, drafts != 0, &p);
    if (rc == LSE_MERGE_OK) *bytes = p.ws_bytes;
    return rc;
}

int lse_merge_tree_default_splits(int B, int T, int Hq, int Hkv, int L, int D, int sms) {
    return lsem::tree_default_splits(B, T, Hq, Hkv, L, D, sms);
}

}  // extern "C"
