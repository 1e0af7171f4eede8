// attn_api.cpp -- C ABI of the grouped-attention entry points: argument checks on the
// host, then dispatch.  A call that fails a check enqueues nothing.
#include <hip/hip_runtime.h>
#include <math.h>

#include "../../include/gdn.h"
#include "api_checks.h"
#include "attn.h"

namespace {

using namespace gdn_checks;

// Memory of a tensor: rows of `row` bytes, `step` bytes from one to the next (one row of all
// bytes where it is contiguous).
struct Rows {
    uintptr_t at;
    unsigned long long count, row, step;
};

Rows rows(const void *p, long long count, long long row, long long step) {
    if (!p || count <= 0 || row <= 0) return {0, 0, 0, 0};
    if (step == row) return {reinterpret_cast<uintptr_t>(p), 1, (unsigned long long)(count * row), 0};
    return {reinterpret_cast<uintptr_t>(p), (unsigned long long)count, (unsigned long long)row, (unsigned long long)step};
}
Rows block(const void *p, unsigned long long bytes) { return rows(p, 1, (long long)bytes, (long long)bytes); }

// Slices of one larger tensor (equal steps, rows that miss each other) are apart; else any
// overlap of the ranges counts.
bool meet(const Rows &a, const Rows &b) {
    if (!a.count || !b.count) return false;
    const uintptr_t ae = a.at + (a.count - 1) * a.step + a.row, be = b.at + (b.count - 1) * b.step + b.row;
    if (a.at >= be || b.at >= ae) return false;
    const unsigned long long step = a.count > 1 ? a.step : b.step;
    if (step == 0 || (a.count > 1 && b.count > 1 && a.step != b.step)) return true;
    if (a.row > step || b.row > step) return true;
    const unsigned long long d = b.at >= a.at ? (b.at - a.at) % step : (step - (a.at - b.at) % step) % step;
    return d < a.row || d + b.row > step;
}

template <int NO, int NI> bool apart(const Rows (&out)[NO], const Rows (&in)[NI]) {
    for (int i = 0; i < NO; ++i) {
        for (int j = 0; j < NI; ++j)
            if (meet(out[i], in[j])) return false;
        for (int j = 0; j < i; ++j)
            if (meet(out[i], out[j])) return false;
    }
    return true;
}

bool dtype_ok(gdn_dtype t) { return t == GDN_F32 || t == GDN_BF16; }
bool scale_ok(float s) { return s > 0.f && isfinite(s * gdn::LOG2E); }

// Elements from token to token: the heads of a token at least, and whole 16-byte pieces.
bool stride_ok(long long s, int H, int D, long long es) { return s >= (long long)H * D && s * es % 16 == 0; }
constexpr long long STRIDES = 1LL << 21;   // and at most so many (GDN_ENOTSUP beyond): 24 bits of bytes

gdn_status prologue_sizes(int T, int Hq, int Hk, int D, int R, gdn_dtype dtype)
{
    if (!dtype_ok(dtype) || T < 0 || Hq < 0 || Hk < 0 || D <= 0 || R < 0 || R > D) return GDN_EINVAL;
    if (prod(T, (long long)Hq + Hk, D, 4) < 0) return GDN_EINVAL;
    if ((D != 64 && D != 128) || R % 16 != 0) return GDN_ENOTSUP;
    if (Hq > (1 << 15) || Hk > (1 << 15) || T >= (1 << 24)) return GDN_ENOTSUP;
    return GDN_OK;
}

gdn_status attn_sizes(int B, int Tq, int Tk, int Hq, int Hk, int D, gdn_dtype dtype)
{
    if (!dtype_ok(dtype) || B < 0 || Tq < 0 || Tk < 0 || Hq <= 0 || Hk <= 0 || D <= 0 || Hq % Hk != 0) return GDN_EINVAL;
    if (prod(Tq, Hq, D, 4) < 0 || prod(Tk, Hk, D, 4) < 0) return GDN_EINVAL;
    if ((D != 64 && D != 128) || Hq / Hk > 64 || Hq > (1 << 14)) return GDN_ENOTSUP;
    // rows of a key head (token, head) in 30 bits, those of all heads in 28; grids: workgroups * threads < 2^32
    // (64 threads for four keys where dk and dv of many are added up)
    const bool bf16 = dtype == GDN_BF16;
    const int G = Hq / Hk;
    if (((long long)Tq + Tk) * G >= (1LL << 30) || prod(Tq, Hq) >= (1LL << 28) || prod(Tk, Hk) >= (1LL << 26)) return GDN_ENOTSUP;
    if (B >= (1 << 24)) return GDN_ENOTSUP;
    const gdn::AttnFwdPlan f = gdn::attn_fwd_plan(bf16, B, Tq, Tk, Hk, G);
    const gdn::AttnBwdPlan b = gdn::attn_bwd_plan(bf16, B, Tq, Tk, Hk, G);
    if (f.tiles * Hk >= (1LL << 24) || b.qtiles * Hk * b.kp >= (1LL << 24)) return GDN_ENOTSUP;
    return GDN_OK;
}

gdn_status cache_sizes(int N, int Hk, int D, int pages, int page, int width)
{
    if (N < 0 || Hk <= 0 || D <= 0 || pages < 0 || page <= 0 || width < 0) return GDN_EINVAL;
    if (prod(pages, page, Hk, D) < 0) return GDN_EINVAL;
    if ((D != 64 && D != 128) || page % 16 != 0 || page >= 16 << 15 || Hk > (1 << 15)) return GDN_ENOTSUP;
    // 31 bits for blocks of the cache and table entries, 30 for a sequence's tokens
    if (prod(pages, page / 16, Hk) > 0x7fffffffLL || prod(N, width) > 0x7fffffffLL || prod(width, page) > (1LL << 30)) return GDN_ENOTSUP;
    if (N >= (1 << 22)) return GDN_ENOTSUP;
    return GDN_OK;
}

bool all_aligned(std::initializer_list<const void *> ps, unsigned to) {
    for (const void *p : ps)
        if (p && !aligned(p, to)) return false;
    return true;
}

hipStream_t stream_of(void *s) { return static_cast<hipStream_t>(s); }
gdn_status status_of(hipError_t e) { return e == hipSuccess ? GDN_OK : GDN_EHIP; }

} // namespace

extern "C" {

gdn_status gdn_attn_prologue(const void *q_raw, const void *k_raw, const float *w_q, const float *w_k,
                             const float *inv_freq, const int *pos, void *q, void *k, int T, int Hq, int Hk, int D,
                             int R, long long q_stride, long long k_stride, float eps, gdn_dtype dtype, void *stream)
{
    const gdn_status st = prologue_sizes(T, Hq, Hk, D, R, dtype);
    if (st == GDN_EINVAL) return st;
    const long long es = dtype == GDN_BF16 ? 2 : 4;
    if (!(eps >= 0.f) || !isfinite(eps) || !stride_ok(q_stride, Hq, D, es) || !stride_ok(k_stride, Hk, D, es)) return GDN_EINVAL;
    if (T > 0 && Hq > 0 && (!q_raw || !w_q || !q)) return GDN_EINVAL;
    if (T > 0 && Hk > 0 && (!k_raw || !w_k || !k)) return GDN_EINVAL;
    if (T > 0 && R > 0 && (!inv_freq || !pos)) return GDN_EINVAL;
    if (!all_aligned({q_raw, k_raw, w_q, w_k, q, k}, 16) || !all_aligned({inv_freq, pos}, 4)) return GDN_EINVAL;
    const Rows in[] = {rows(q_raw, T, Hq * (long long)D * es, q_stride * es), rows(k_raw, T, Hk * (long long)D * es, k_stride * es),
                       block(w_q, D * 4), block(w_k, D * 4), block(inv_freq, R * 2), block(pos, T * 4LL)};
    const Rows out[] = {block(q, prod(T, Hq, D, es)), block(k, prod(T, Hk, D, es))};
    if (!apart(out, in)) return GDN_EINVAL;
    if (st != GDN_OK) return st;
    if (q_stride > STRIDES || k_stride > STRIDES) return GDN_ENOTSUP;
    if (T == 0 || Hq + Hk == 0) return GDN_OK;
    gdn::AttnPrologueArgs a = {};
    a.q_raw = q_raw; a.k_raw = k_raw; a.w_q = w_q; a.w_k = w_k; a.inv_freq = inv_freq; a.pos = pos; a.q = q; a.k = k;
    a.q_stride = q_stride; a.k_stride = k_stride; a.eps = eps; a.T = T; a.Hq = Hq; a.Hk = Hk; a.R = R;
    return status_of(gdn::attn_prologue_launch(dtype == GDN_BF16, D, a, stream_of(stream)));
}

gdn_status gdn_attn_prologue_bwd_workspace_size(int T, int Hq, int Hk, int D, int R, gdn_dtype dtype, size_t *bytes)
{
    if (!bytes) return GDN_EINVAL;
    const gdn_status st = prologue_sizes(T, Hq, Hk, D, R, dtype);
    if (st != GDN_OK) return st;
    *bytes = (size_t)gdn::attn_prologue_bwd_workspace(T, Hq, D);
    return GDN_OK;
}

gdn_status gdn_attn_prologue_bwd(const void *q_raw, const void *k_raw, const float *w_q, const float *w_k,
                                 const float *inv_freq, const int *pos, const void *d_q, const void *d_k, void *dq_raw,
                                 void *dk_raw, float *dw_q, float *dw_k, void *workspace, size_t workspace_bytes, int T,
                                 int Hq, int Hk, int D, int R, long long q_stride, long long k_stride,
                                 long long dq_stride, long long dk_stride, float eps, gdn_dtype dtype, void *stream)
{
    const gdn_status st = prologue_sizes(T, Hq, Hk, D, R, dtype);
    if (st == GDN_EINVAL) return st;
    const long long es = dtype == GDN_BF16 ? 2 : 4, qrow = Hq * (long long)D * es, krow = Hk * (long long)D * es;
    if (!(eps >= 0.f) || !isfinite(eps)) return GDN_EINVAL;
    for (long long s : {q_stride, dq_stride})
        if (!stride_ok(s, Hq, D, es)) return GDN_EINVAL;
    for (long long s : {k_stride, dk_stride})
        if (!stride_ok(s, Hk, D, es)) return GDN_EINVAL;
    if (!dw_q || !dw_k) return GDN_EINVAL;
    if (T > 0 && Hq > 0 && (!q_raw || !w_q || !d_q || !dq_raw)) return GDN_EINVAL;
    if (T > 0 && Hk > 0 && (!k_raw || !w_k || !d_k || !dk_raw)) return GDN_EINVAL;
    if (T > 0 && R > 0 && (!inv_freq || !pos)) return GDN_EINVAL;
    if (!all_aligned({q_raw, k_raw, w_q, w_k, d_q, d_k, dq_raw, dk_raw}, 16) || !all_aligned({inv_freq, pos, dw_q, dw_k}, 4) ||
        !all_aligned({workspace}, 256))
        return GDN_EINVAL;
    const unsigned long long need = st == GDN_OK ? gdn::attn_prologue_bwd_workspace(T, Hq, D) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need)) return GDN_EINVAL;
    const Rows in[] = {rows(q_raw, T, qrow, q_stride * es), rows(k_raw, T, krow, k_stride * es), block(w_q, D * 4), block(w_k, D * 4),
                       block(inv_freq, R * 2), block(pos, T * 4LL), block(d_q, T * qrow), block(d_k, T * krow)};
    const Rows out[] = {rows(dq_raw, T, qrow, dq_stride * es), rows(dk_raw, T, krow, dk_stride * es), block(dw_q, D * 4),
                        block(dw_k, D * 4), block(workspace, need)};
    if (!apart(out, in)) return GDN_EINVAL;
    if (st != GDN_OK) return st;
    for (long long s : {q_stride, k_stride, dq_stride, dk_stride})
        if (s > STRIDES) return GDN_ENOTSUP;
    gdn::AttnPrologueArgs a = {};
    a.q_raw = q_raw; a.k_raw = k_raw; a.w_q = w_q; a.w_k = w_k; a.inv_freq = inv_freq; a.pos = pos;
    a.q = const_cast<void *>(d_q); a.k = const_cast<void *>(d_k); a.dq_raw = dq_raw; a.dk_raw = dk_raw;
    a.dw_q = dw_q; a.dw_k = dw_k; a.ws = (float *)workspace;
    a.q_stride = q_stride; a.k_stride = k_stride; a.dq_stride = dq_stride; a.dk_stride = dk_stride;
    a.eps = eps; a.T = T; a.Hq = Hq; a.Hk = Hk; a.R = R;
    return status_of(gdn::attn_prologue_bwd_launch(dtype == GDN_BF16, D, a, stream_of(stream)));
}

gdn_status gdn_attn_fwd_workspace_size(int B, int Tq, int Tk, int Hq, int Hk, int D, gdn_dtype dtype, size_t *bytes)
{
    if (!bytes) return GDN_EINVAL;
    const gdn_status st = attn_sizes(B, Tq, Tk, Hq, Hk, D, dtype);
    if (st != GDN_OK) return st;
    *bytes = B > 0 ? (size_t)gdn::attn_fwd_workspace(dtype == GDN_BF16, B, Tq, Tk, Hk, Hq / Hk, D) : 0;
    return GDN_OK;
}

gdn_status gdn_attn_fwd(const void *q, const void *k, const void *v, const int *cu_q, const int *cu_k, void *o, float *lse,
                        void *workspace, size_t workspace_bytes, int B, int Tq, int Tk, int Hq, int Hk, int D,
                        long long q_stride, long long k_stride, long long v_stride, float scale, gdn_dtype dtype,
                        void *stream)
{
    const gdn_status st = attn_sizes(B, Tq, Tk, Hq, Hk, D, dtype);
    if (st == GDN_EINVAL) return st;
    const bool bf16 = dtype == GDN_BF16;
    const long long es = bf16 ? 2 : 4, qrow = Hq * (long long)D * es, krow = Hk * (long long)D * es;
    if (!scale_ok(scale) || (!cu_k && Tq != Tk)) return GDN_EINVAL;
    if (!stride_ok(q_stride, Hq, D, es) || !stride_ok(k_stride, Hk, D, es) || !stride_ok(v_stride, Hk, D, es)) return GDN_EINVAL;
    const bool live = B > 0 && Tq > 0;
    if (live && (!q || !o || !cu_q)) return GDN_EINVAL;
    if (live && Tk > 0 && (!k || !v)) return GDN_EINVAL;
    if (!all_aligned({q, k, v, o}, 16) || !all_aligned({cu_q, cu_k, lse}, 4) || !all_aligned({workspace}, 256)) return GDN_EINVAL;
    const unsigned long long need = st == GDN_OK && live ? gdn::attn_fwd_workspace(bf16, B, Tq, Tk, Hk, Hq / Hk, D) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need)) return GDN_EINVAL;
    const Rows in[] = {rows(q, Tq, qrow, q_stride * es), rows(k, Tk, krow, k_stride * es), rows(v, Tk, krow, v_stride * es),
                       block(cu_q, (B + 1LL) * 4), block(cu_k, (B + 1LL) * 4)};
    const Rows out[] = {block(o, Tq * qrow), block(lse, prod(Tq, Hq, 4)), block(workspace, need)};
    if (!apart(out, in)) return GDN_EINVAL;
    if (st != GDN_OK) return st;
    if (q_stride > STRIDES || k_stride > STRIDES || v_stride > STRIDES) return GDN_ENOTSUP;
    if (!live) return GDN_OK;
    gdn::AttnArgs a = {};
    a.q = q; a.k = k; a.v = v; a.cu_q = cu_q; a.cu_k = cu_k; a.o = o; a.lse = lse; a.ws = workspace;
    a.qs = q_stride; a.ks = k_stride; a.vs = v_stride; a.scale = scale; a.B = B; a.Tq = Tq; a.Tk = Tk; a.Hk = Hk; a.G = Hq / Hk;
    return status_of(gdn::attn_fwd_launch(bf16, D, a, stream_of(stream)));
}

gdn_status gdn_attn_bwd_workspace_size(int B, int Tq, int Tk, int Hq, int Hk, int D, gdn_dtype dtype, size_t *bytes)
{
    if (!bytes) return GDN_EINVAL;
    const gdn_status st = attn_sizes(B, Tq, Tk, Hq, Hk, D, dtype);
    if (st != GDN_OK) return st;
    *bytes = B > 0 ? (size_t)gdn::attn_bwd_workspace(dtype == GDN_BF16, B, Tq, Tk, Hk, Hq / Hk, D) : 0;
    return GDN_OK;
}

gdn_status gdn_attn_bwd(const void *q, const void *k, const void *v, const int *cu_q, const int *cu_k, const void *o,
                        const float *lse, const void *d_o, void *dq, void *dk, void *dv, void *workspace,
                        size_t workspace_bytes, int B, int Tq, int Tk, int Hq, int Hk, int D, long long q_stride,
                        long long k_stride, long long v_stride, long long dq_stride, long long dk_stride,
                        long long dv_stride, float scale, gdn_dtype dtype, void *stream)
{
    const gdn_status st = attn_sizes(B, Tq, Tk, Hq, Hk, D, dtype);
    if (st == GDN_EINVAL) return st;
    const bool bf16 = dtype == GDN_BF16;
    const long long es = bf16 ? 2 : 4, qrow = Hq * (long long)D * es, krow = Hk * (long long)D * es;
    if (!scale_ok(scale) || (!cu_k && Tq != Tk)) return GDN_EINVAL;
    for (long long s : {q_stride, dq_stride})
        if (!stride_ok(s, Hq, D, es)) return GDN_EINVAL;
    for (long long s : {k_stride, v_stride, dk_stride, dv_stride})
        if (!stride_ok(s, Hk, D, es)) return GDN_EINVAL;
    if (B > 0 && Tq + (long long)Tk > 0 && !cu_q) return GDN_EINVAL;
    if (B > 0 && Tq > 0 && (!q || !o || !lse || !d_o || !dq)) return GDN_EINVAL;
    if (B > 0 && Tk > 0 && (!k || !v || !dk || !dv)) return GDN_EINVAL;
    if (!all_aligned({q, k, v, o, d_o, dq, dk, dv}, 16) || !all_aligned({cu_q, cu_k, lse}, 4) || !all_aligned({workspace}, 256))
        return GDN_EINVAL;
    const unsigned long long need = st == GDN_OK && B > 0 ? gdn::attn_bwd_workspace(bf16, B, Tq, Tk, Hk, Hq / Hk, D) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need)) return GDN_EINVAL;
    const Rows in[] = {rows(q, Tq, qrow, q_stride * es), rows(k, Tk, krow, k_stride * es), rows(v, Tk, krow, v_stride * es),
                       block(cu_q, (B + 1LL) * 4), block(cu_k, (B + 1LL) * 4), block(o, Tq * qrow), block(lse, prod(Tq, Hq, 4)),
                       block(d_o, Tq * qrow)};
    const Rows out[] = {rows(dq, Tq, qrow, dq_stride * es), rows(dk, Tk, krow, dk_stride * es), rows(dv, Tk, krow, dv_stride * es),
                        block(workspace, need)};
    if (!apart(out, in)) return GDN_EINVAL;
    if (st != GDN_OK) return st;
    for (long long s : {q_stride, k_stride, v_stride, dq_stride, dk_stride, dv_stride})
        if (s > STRIDES) return GDN_ENOTSUP;
    if (B == 0 || Tq + (long long)Tk == 0) return GDN_OK;
    gdn::AttnArgs a = {};
    a.q = q; a.k = k; a.v = v; a.cu_q = cu_q; a.cu_k = cu_k; a.o = const_cast<void *>(o); a.lse = const_cast<float *>(lse);
    a.d_o = d_o; a.dq = dq; a.dk = dk; a.dv = dv; a.ws = workspace;
    a.qs = q_stride; a.ks = k_stride; a.vs = v_stride; a.dqs = dq_stride; a.dks = dk_stride; a.dvs = dv_stride;
    a.scale = scale; a.B = B; a.Tq = Tq; a.Tk = Tk; a.Hk = Hk; a.G = Hq / Hk;
    return status_of(gdn::attn_bwd_launch(bf16, D, a, stream_of(stream)));
}

gdn_status gdn_attn_append(const void *k, const void *v, const int *cu, void *k_cache, void *v_cache, float *k_scale,
                           float *v_scale, const int *table, const int *lens, int N, int T, int Hk, int D, int pages,
                           int page, int width, long long k_stride, long long v_stride, gdn_dtype dtype, void *stream)
{
    if (!dtype_ok(dtype) || T < 0) return GDN_EINVAL;
    const gdn_status st = cache_sizes(N, Hk, D, pages, page, width);
    if (st == GDN_EINVAL) return st;
    const long long es = dtype == GDN_BF16 ? 2 : 4, row = Hk * (long long)D * es;
    if ((!cu && T != N) || !stride_ok(k_stride, Hk, D, es) || !stride_ok(v_stride, Hk, D, es) || prod(T, row) < 0) return GDN_EINVAL;
    const bool live = N > 0 && T > 0 && pages > 0 && width > 0;
    if (live && (!k || !v || !k_cache || !v_cache || !k_scale || !v_scale || !table || !lens)) return GDN_EINVAL;
    if (!all_aligned({k, v, k_cache, v_cache}, 16) || !all_aligned({cu, k_scale, v_scale, table, lens}, 4)) return GDN_EINVAL;
    const unsigned long long cache = prod(pages, page, Hk, D), scales = prod(pages, page / 16, Hk, 4);
    const Rows in[] = {rows(k, T, row, k_stride * es), rows(v, T, row, v_stride * es), block(cu, (N + 1LL) * 4),
                       block(table, prod(N, width, 4)), block(lens, N * 4LL)};
    const Rows out[] = {block(k_cache, cache), block(v_cache, cache), block(k_scale, scales), block(v_scale, scales)};
    if (!apart(out, in)) return GDN_EINVAL;
    if (st != GDN_OK) return st;
    if (k_stride > STRIDES || v_stride > STRIDES || T / 16 + 2LL * N >= (1LL << 24)) return GDN_ENOTSUP;
    if (!live) return GDN_OK;
    gdn::AttnCacheArgs a = {};
    a.k = k; a.v = v; a.cu = cu; a.k_cache = k_cache; a.v_cache = v_cache; a.k_scale = k_scale; a.v_scale = v_scale;
    a.table = table; a.lens = lens; a.ks = k_stride; a.vs = v_stride; a.N = N; a.T = T; a.Hk = Hk;
    a.pages = pages; a.page = page; a.width = width;
    return status_of(gdn::attn_append_launch(dtype == GDN_BF16, D, a, stream_of(stream)));
}

gdn_status gdn_attn_step_workspace_size(int N, int Hq, int Hk, int D, int page, int width, size_t *bytes)
{
    if (!bytes || Hq <= 0 || Hk <= 0 || Hq % Hk != 0) return GDN_EINVAL;
    const gdn_status st = cache_sizes(N, Hk, D, 0, page, width);
    if (st != GDN_OK) return st;
    if (Hq / Hk > 64 || prod(N, Hq) >= (1LL << 23)) return GDN_ENOTSUP;
    *bytes = (size_t)gdn::attn_step_workspace(N, Hk, Hq / Hk, D, page, width);
    return GDN_OK;
}

gdn_status gdn_attn_step(const void *q, const void *k_cache, const void *v_cache, const float *k_scale,
                         const float *v_scale, const int *table, const int *lens, void *o, float *lse, void *workspace,
                         size_t workspace_bytes, int N, int Hq, int Hk, int D, int pages, int page, int width, float scale,
                         gdn_dtype dtype, void *stream)
{
    if (!dtype_ok(dtype) || Hq <= 0 || !scale_ok(scale)) return GDN_EINVAL;
    gdn_status st = cache_sizes(N, Hk, D, pages, page, width);
    if (st == GDN_EINVAL || Hq % Hk != 0) return GDN_EINVAL;
    // the grid: a workgroup of 256 threads for each 16 heads, and those that share the tiles
    if (Hq / Hk > 64 || prod(N, Hq) >= (1LL << 23)) st = GDN_ENOTSUP;
    const long long es = dtype == GDN_BF16 ? 2 : 4, bytes = prod(N, Hq, D, es);
    if (bytes < 0) return GDN_EINVAL;
    if (N > 0 && (!q || !lens || !o || (width > 0 && !table))) return GDN_EINVAL;
    if (N > 0 && pages > 0 && width > 0 && (!k_cache || !v_cache || !k_scale || !v_scale)) return GDN_EINVAL;
    if (!all_aligned({q, k_cache, v_cache, o}, 16) || !all_aligned({k_scale, v_scale, table, lens, lse}, 4) || !all_aligned({workspace}, 256))
        return GDN_EINVAL;
    const unsigned long long need = st == GDN_OK ? gdn::attn_step_workspace(N, Hk, Hq / Hk, D, page, width) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need)) return GDN_EINVAL;
    const unsigned long long cache = prod(pages, page, Hk, D), scales = prod(pages, page / 16, Hk, 4);
    const Rows in[] = {block(q, bytes), block(k_cache, cache), block(v_cache, cache), block(k_scale, scales), block(v_scale, scales),
                       block(table, prod(N, width, 4)), block(lens, N * 4LL)};
    const Rows out[] = {block(o, bytes), block(lse, prod(N, Hq, 4)), block(workspace, need)};
    if (!apart(out, in)) return GDN_EINVAL;
    if (st != GDN_OK) return st;
    if (N == 0) return GDN_OK;
    gdn::AttnCacheArgs a = {};
    a.q = q; a.k_cache = const_cast<void *>(k_cache); a.v_cache = const_cast<void *>(v_cache);
    a.k_scale = const_cast<float *>(k_scale); a.v_scale = const_cast<float *>(v_scale); a.table = table; a.lens = lens;
    a.o = o; a.lse = lse; a.ws = workspace; a.qs = Hq * (long long)D; a.scale = scale; a.N = N; a.Hk = Hk; a.G = Hq / Hk;
    a.pages = pages; a.page = page; a.width = width;
    return status_of(gdn::attn_step_launch(dtype == GDN_BF16, D, a, stream_of(stream)));
}

} // extern "C"
