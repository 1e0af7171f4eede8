// latent_api.cpp -- C ABI of the latent-attention entry points: argument checks on
// the host, then dispatch.  A call that fails a check enqueues nothing.
#include <hip/hip_runtime.h>
#include <math.h>

#include "../../include/gdn.h"
#include "api_checks.h"
#include "latent.h"

namespace {

using namespace gdn_checks;

bool overlaps_any(Range out, const Range *in, int n) {
    for (int i = 0; i < n; ++i)
        if (overlap(out, in[i])) return true;
    return false;
}

template <int NO, int NI> bool outputs_clear(const Range (&out)[NO], const Range (&in)[NI]) {
    for (int i = 0; i < NO; ++i) {
        if (overlaps_any(out[i], in, NI)) return false;
        if (overlaps_any(out[i], out, i)) return false;
    }
    return true;
}

// The kernels take exponentials to the base 2, of scores times scale log2(e).
bool scale_ok(float s) { return s > 0.f && isfinite(s * gdn::LOG2E); }

// Sizes of the expanded form: EINVAL for negative or overflowing ones, ENOTSUP for
// those without a kernel.
gdn_status expanded_sizes(int B, int Tq, int Tk, int H, int dn, int dr, int dv, gdn_dtype dtype)
{
    if (dtype != GDN_F32 && dtype != GDN_BF16) return GDN_EINVAL;
    if (B < 0 || Tq < 0 || Tk < 0 || H < 0 || dn <= 0 || dr <= 0 || dv <= 0 || Tq > Tk) return GDN_EINVAL;
    if (prod(B, Tk, H, 4LL * ((long long)dn + dr + dv)) < 0) return GDN_EINVAL;
    if ((dn != 64 && dn != 128) || (dv != 64 && dv != 128) || dr != gdn::LATENT_ROPE) return GDN_ENOTSUP;
    // grids: workgroups * 256 threads < 2^32 (16 rows of B Tk a workgroup)
    const long long rows = prod(B, H, Tq), tiles = prod(B, H, ((long long)Tk + 63) / 64);
    // a lane's offset within the 32 rows that one copy covers: 32 bits
    if (H > (1 << 15)) return GDN_ENOTSUP;
    if (rows >= (1LL << 28) || tiles >= (1LL << 24) || prod(B, Tk) >= (1LL << 27)) return GDN_ENOTSUP;
    return GDN_OK;
}

// The same for the backward, whose key-owning kernel has 512 threads a workgroup.
gdn_status backward_sizes(int B, int Tq, int Tk, int H, int dn, int dr, int dv, gdn_dtype dtype)
{
    const gdn_status st = expanded_sizes(B, Tq, Tk, H, dn, dr, dv, dtype);
    if (st != GDN_OK) return st;
    const long long own = dtype == GDN_BF16 ? 128 : 64;
    return prod(B, H, (Tk + own - 1) / own) < (1LL << 23) ? GDN_OK : GDN_ENOTSUP;
}

gdn_status absorbed_sizes(int N, int M, int H, int r, int dr, gdn_dtype dtype)
{
    if (dtype != GDN_F32 && dtype != GDN_BF16) return GDN_EINVAL;
    if (N < 0 || M < 0 || H < 0 || r <= 0 || dr <= 0) return GDN_EINVAL;
    if (prod(N, M, H, 4LL * ((long long)r + dr)) < 0) return GDN_EINVAL;
    if ((r != 256 && r != 512) || dr != gdn::LATENT_ROPE || M > 64) return GDN_ENOTSUP;
    // the join kernel's grid: a workgroup of 256 threads a row
    if (prod(M, H) > (1LL << 20) || prod(N, M, H) >= (1LL << 24)) return GDN_ENOTSUP;
    return GDN_OK;
}

gdn_status absorbed(const void *q, const void *draft, const long long *tree, bool drafts, const void *cache,
                    const int *table, const int *lens, void *o, float *lse, void *ws, size_t ws_bytes, int N,
                    int M, int H, int r, int dr, int pages, int page, int width, float scale, gdn_dtype dtype,
                    void *stream)
{
    const gdn_status st = absorbed_sizes(N, M, H, r, dr, dtype);
    if (st == GDN_EINVAL) return st;
    if (pages < 0 || page <= 0 || width < 0 || !scale_ok(scale)) return GDN_EINVAL;
    const long long es = dtype == GDN_BF16 ? 2 : 4, D = (long long)r + dr;
    const long long rows = prod(N, M, H), slots = prod(pages, page), entries = prod(N, width);
    const long long ncache = prod(pages, page, D * es), ndraft = drafts ? prod(N, M, D * es) : 0;
    if (ncache < 0 || ndraft < 0) return GDN_EINVAL;
    if (rows > 0) {
        if (!q || !lens || !o || (drafts && !draft)) return GDN_EINVAL;
        if (width > 0 && !table) return GDN_EINVAL;
        if (slots > 0 && width > 0 && !cache) return GDN_EINVAL;
    }
    for (const void *p : {q, draft, cache, (const void *)o})
        if (p && !aligned16(p)) return GDN_EINVAL;
    for (const void *p : {(const void *)table, (const void *)lens, (const void *)lse})
        if (p && !aligned(p, 4)) return GDN_EINVAL;
    if (tree && !aligned(tree, 8)) return GDN_EINVAL;
    if (ws && !aligned(ws, 256)) return GDN_EINVAL;
    const bool bf16 = dtype == GDN_BF16;
    const unsigned long long need = st == GDN_OK && rows > 0 ? gdn::latent_step_workspace(bf16, N, M, H, r) : 0;
    if (need > 0 && (!ws || ws_bytes < need)) return GDN_EINVAL;
    const Range in[] = {range(q, rows * D * es), range(draft, draft ? ndraft : 0), range(tree, tree ? prod(N, M, 8) : 0),
                        range(cache, cache ? ncache : 0), range(table, table ? entries * 4 : 0), range(lens, (long long)N * 4)};
    const Range out[] = {range(o, o ? rows * r * es : 0), range(lse, lse ? rows * 4 : 0), range(ws, need)};
    if (!outputs_clear(out, in)) return GDN_EINVAL;
    if (st != GDN_OK) return st;
    // 32-bit slots, table entries, tokens a sequence and tiles of the whole batch
    if (slots > 0x7fffffffLL || entries > 0x7fffffffLL || prod(width, page) > (1LL << 30)) return GDN_ENOTSUP;
    if (prod(N, (prod(width, page) + M + 31) / 32) > 0x7fffffffLL) return GDN_ENOTSUP;
    if (rows == 0) return GDN_OK;
    gdn::LatentStepArgs a = {};
    a.q = q; a.draft = draft; a.tree = tree; a.cache = cache; a.table = table; a.lens = lens;
    a.o = o; a.lse = lse; a.ws = ws; a.scale = scale; a.N = N; a.M = M; a.H = H; a.drafts = drafts ? M : 0;
    a.pages = pages; a.page = page; a.width = width;
    const hipError_t e = gdn::latent_step_launch(bf16, r, a, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? GDN_OK : GDN_EHIP;
}

} // namespace

extern "C" {

gdn_status gdn_latent_fwd_workspace_size(int B, int Tq, int Tk, int H, int dn, int dr, int dv, gdn_dtype dtype,
                                         size_t *bytes)
{
    if (!bytes) return GDN_EINVAL;
    const gdn_status st = expanded_sizes(B, Tq, Tk, H, dn, dr, dv, dtype);
    if (st != GDN_OK) return st;
    *bytes = (size_t)gdn::latent_fwd_workspace(dtype == GDN_BF16, B, Tq, Tk, H, dv);
    return GDN_OK;
}

gdn_status gdn_latent_fwd(const void *q, const void *kv, const void *k_rope, const int *lens, void *o, float *lse,
                          void *workspace, size_t workspace_bytes, int B, int Tq, int Tk, int H, int dn, int dr,
                          int dv, float scale, gdn_dtype dtype, void *stream)
{
    const gdn_status st = expanded_sizes(B, Tq, Tk, H, dn, dr, dv, dtype);
    if (st == GDN_EINVAL) return st;
    if (!scale_ok(scale)) return GDN_EINVAL;
    const long long es = dtype == GDN_BF16 ? 2 : 4, qrows = prod(B, Tq, H), krows = prod(B, Tk, H), ks = prod(B, Tk);
    if (qrows > 0 && (!q || !kv || !k_rope || !o)) return GDN_EINVAL;
    for (const void *p : {q, kv, k_rope, (const void *)o})
        if (p && !aligned16(p)) return GDN_EINVAL;
    for (const void *p : {(const void *)lens, (const void *)lse})
        if (p && !aligned(p, 4)) return GDN_EINVAL;
    if (workspace && !aligned(workspace, 256)) return GDN_EINVAL;
    const unsigned long long need =
        st == GDN_OK ? gdn::latent_fwd_workspace(dtype == GDN_BF16, B, Tq, Tk, H, dv) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need)) return GDN_EINVAL;
    const Range in[] = {range(q, qrows * (dn + dr) * es), range(kv, krows * (dn + dv) * es), range(k_rope, ks * dr * es),
                        range(lens, lens ? (long long)B * 4 : 0)};
    const Range out[] = {range(o, qrows * dv * es), range(lse, lse ? qrows * 4 : 0), range(workspace, need)};
    if (!outputs_clear(out, in)) return GDN_EINVAL;
    if (st != GDN_OK) return st;
    if (qrows == 0) return GDN_OK;
    gdn::LatentFwdArgs a = {};
    a.q = q; a.kv = kv; a.k_rope = k_rope; a.lens = lens; a.o = o; a.lse = lse; a.ws = need ? workspace : nullptr;
    a.scale = scale; a.B = B; a.Tq = Tq; a.Tk = Tk; a.H = H;
    const hipError_t e = gdn::latent_fwd_launch(dtype == GDN_BF16, dn, dv, a, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? GDN_OK : GDN_EHIP;
}

gdn_status gdn_latent_bwd_workspace_size(int B, int Tq, int Tk, int H, int dn, int dr, int dv, gdn_dtype dtype,
                                         size_t *bytes)
{
    if (!bytes) return GDN_EINVAL;
    const gdn_status st = backward_sizes(B, Tq, Tk, H, dn, dr, dv, dtype);
    if (st != GDN_OK) return st;
    *bytes = (size_t)gdn::latent_bwd_workspace(dtype == GDN_BF16, B, Tq, Tk, H, dn, dv);
    return GDN_OK;
}

gdn_status gdn_latent_bwd(const void *q, const void *kv, const void *k_rope, const int *lens, const void *o,
                          const float *lse, const void *d_o, void *dq, void *dkv, void *dk_rope, void *workspace,
                          size_t workspace_bytes, int B, int Tq, int Tk, int H, int dn, int dr, int dv, float scale,
                          gdn_dtype dtype, void *stream)
{
    const gdn_status st = backward_sizes(B, Tq, Tk, H, dn, dr, dv, dtype);
    if (st == GDN_EINVAL) return st;
    if (!scale_ok(scale)) return GDN_EINVAL;
    const long long es = dtype == GDN_BF16 ? 2 : 4, qrows = prod(B, Tq, H), krows = prod(B, Tk, H), ks = prod(B, Tk);
    if (qrows > 0 && (!q || !o || !lse || !d_o || !dq)) return GDN_EINVAL;
    if (krows > 0 && (!kv || !k_rope || !dkv)) return GDN_EINVAL;
    if (ks > 0 && !dk_rope) return GDN_EINVAL;
    for (const void *p : {q, kv, k_rope, o, d_o, (const void *)dq, (const void *)dkv, (const void *)dk_rope})
        if (p && !aligned16(p)) return GDN_EINVAL;
    for (const void *p : {(const void *)lens, (const void *)lse})
        if (p && !aligned(p, 4)) return GDN_EINVAL;
    if (workspace && !aligned(workspace, 256)) return GDN_EINVAL;
    const unsigned long long need = st == GDN_OK ? gdn::latent_bwd_workspace(dtype == GDN_BF16, B, Tq, Tk, H, dn, dv) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need)) return GDN_EINVAL;
    const Range in[] = {range(q, qrows * (dn + dr) * es), range(kv, krows * (dn + dv) * es), range(k_rope, ks * dr * es),
                        range(lens, lens ? (long long)B * 4 : 0), range(o, qrows * dv * es), range(lse, qrows * 4),
                        range(d_o, qrows * dv * es)};
    const Range out[] = {range(dq, qrows * (dn + dr) * es), range(dkv, krows * (dn + dv) * es),
                         range(dk_rope, ks * dr * es), range(workspace, need)};
    if (!outputs_clear(out, in)) return GDN_EINVAL;
    if (st != GDN_OK) return st;
    if (ks == 0) return GDN_OK;
    gdn::LatentBwdArgs a = {};
    a.q = q; a.kv = kv; a.k_rope = k_rope; a.lens = lens; a.o = o; a.lse = lse; a.d_o = d_o;
    a.dq = dq; a.dkv = dkv; a.dk_rope = dk_rope; a.ws = workspace; a.scale = scale;
    a.B = B; a.Tq = Tq; a.Tk = Tk; a.H = H;
    const hipError_t e = gdn::latent_bwd_launch(dtype == GDN_BF16, dn, dv, a, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? GDN_OK : GDN_EHIP;
}

gdn_status gdn_latent_steps_workspace_size(int N, int M, int H, int r, int dr, gdn_dtype dtype, size_t *bytes)
{
    if (!bytes) return GDN_EINVAL;
    const gdn_status st = absorbed_sizes(N, M, H, r, dr, dtype);
    if (st != GDN_OK) return st;
    *bytes = prod(N, M, H) > 0 ? (size_t)gdn::latent_step_workspace(dtype == GDN_BF16, N, M, H, r) : 0;
    return GDN_OK;
}

gdn_status gdn_latent_step(const void *q, const void *cache, const int *table, const int *lens, void *o, float *lse,
                           void *workspace, size_t workspace_bytes, int N, int H, int r, int dr, int pages, int page,
                           int width, float scale, gdn_dtype dtype, void *stream)
{
    return absorbed(q, nullptr, nullptr, false, cache, table, lens, o, lse, workspace, workspace_bytes, N, 1, H, r, dr,
                    pages, page, width, scale, dtype, stream);
}

gdn_status gdn_latent_steps(const void *q, const void *draft, const long long *tree, const void *cache,
                            const int *table, const int *lens, void *o, float *lse, void *workspace,
                            size_t workspace_bytes, int N, int M, int H, int r, int dr, int pages, int page, int width,
                            float scale, gdn_dtype dtype, void *stream)
{
    return absorbed(q, draft, tree, true, cache, table, lens, o, lse, workspace, workspace_bytes, N, M, H, r, dr, pages,
                    page, width, scale, dtype, stream);
}

} // extern "C"
