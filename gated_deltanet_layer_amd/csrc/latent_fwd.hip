// latent_fwd.hip -- expanded latent attention, causal forward (gfx950).
//
//   s_ij = scale (q_i^nope . k_j^nope + q_i^rope . k_j^rope),  j <= p_i = Tk - Tq + i
//   o_i = sum_j softmax_j(s_ij) v_j,   lse_i = log sum_j exp s_ij
//
// A workgroup of four waves owns RT = 64 NR query rows of one head and walks
// the key tiles once, keeping the running maximum and sum of every row.  Scores
// are computed transposed (keys on the accumulator's rows, query rows on its
// lanes): a lane then holds four consecutive keys of one query row, so the
// softmax needs two cross-lane steps a tile, and the weights feed the second
// product (o^T = V^T P^T) as its B operand straight from the registers.
//
// Bound by the matrix cores: 8192 rows of 16 heads, bf16, dn = dv = 128 in 301-350 us,
// 0.98-1.14 PFLOP/s, which is what a library product of 8192^3 reaches on the same card
// (1.11; its clock falls with the power that the matrix cores draw: they are busy for
// half of the cycles).  Two tiles of 64 keys stand in LDS (80 KB at 128, two workgroups a
// unit), 32 rows a wave, so that a key operand read from LDS serves two products.  Small
// calls are a chain of latencies: 333 rows of 16 heads 13 us, six tiles one after the
// other.
#include "latent.h"

namespace gdn {

template <typename T, int DN, int DV, int NR> struct FwdCfg {   // NR: 16-row groups a wave
    static constexpr int NW = 4;
    static constexpr int RT = 16 * NR * NW;                // query rows a workgroup
    static constexpr int KT = sizeof(T) == 2 ? 64 : 32;    // keys a tile
    static constexpr int DK = DN + LATENT_ROPE;
    static constexpr int ES = (int)sizeof(T), NCPR = DN * ES / 16, RCPR = LATENT_ROPE * ES / 16, VCPR = DV * ES / 16;
    // a tile: [KT][DN] keys, [KT][64] rotary keys, [KT][DV] values
    static constexpr int OFF_R = KT * NCPR * 16, OFF_V = OFF_R + KT * RCPR * 16, BUF = OFF_V + KT * VCPR * 16;
};

// How a call is cut: 16-row groups a wave, and pieces of the keys.
struct FwdPlan {
    int nr, pieces, keys;   // keys a piece, whole tiles
};

// Rows: two groups a wave (each key operand serves two products) once that gives
// every compute unit a workgroup; below that, one (333 rows, 16 heads: 13.5 us from
// 14.4).  Keys: where there is less than two workgroups a unit and a row has eight
// tiles or more, in pieces of four tiles or more; the longest row of a causal call is
// otherwise its time (bf16, one row of 16 heads over 8192 keys 246 us, in pieces 36; 64
// rows of 8 heads over 4096: 111, 25; fp32, 4 heads of 2048: 211, 77; from 512
// workgroups on pieces cost more than they give: 2 x 16 heads of 2048 64, 70).  Pieces
// to fill the units twice, of bf16 four where there is a workgroup a unit already
// (causal rows differ).  fp32 has tiles of half the keys and four times the time: half
// as many again, as half the pieces of causal rows are empty (4 heads of 2048 77 us,
// 97 without), and from a workgroup a unit on about 16 tiles a piece (8 heads of 3000
// 223 us, in four pieces 293; 16 of 1021 in three 48, in four 52).
inline FwdPlan fwd_plan(bool bf16, int B, int Tq, int Tk, int H)
{
    const long bh = (long)B * H;
    const int kt = bf16 ? 64 : 32, nt = (Tk + kt - 1) / kt;
    FwdPlan p = {bf16 && bh * ((Tq + 127) / 128) >= 256 ? 2 : 1, 1, nt * kt};
    const long wgs = bh * ((Tq + 64 * p.nr - 1) / (64 * p.nr));
    if (wgs > 0 && wgs < 512 && nt >= 8) {
        const long fill = bf16 ? 512 : 768, many = bf16 ? 4 : nt < 52 ? 3 : (nt + 12) / 16;
        long n = wgs < 256 ? (fill + wgs - 1) / wgs : many;
        if (n > nt / 4) n = nt / 4;
        if (n > 32) n = 32;
        const int each = (int)((nt + n - 1) / n);
        p.keys = each * kt;
        p.pieces = (nt + each - 1) / each;
    }
    return p;
}

// Workspace of a call in pieces: float o[pieces][rows][DV], then float lse (base 2)
// [pieces][rows], rows = B Tq H.
template <typename T, int DN, int DV, int NR, bool CUT>
__global__ __launch_bounds__(256, 2) void latent_fwd_kernel(LatentFwdArgs a, int ntiles, FwdPlan plan)
{
    typedef FwdCfg<T, DN, DV, NR> C;
    constexpr int KT = C::KT, DK = C::DK, NKB = DK / 32, NS = KT / 16, NCB = DV / 16;
    extern __shared__ char lds[];
    const int BH = a.B * a.H;
    const int bh = blockIdx.x % BH, piece = CUT ? blockIdx.x / BH % plan.pieces : 0;
    const int tile = ntiles - 1 - (int)(blockIdx.x / BH / (CUT ? plan.pieces : 1));   // longest rows first
    const int b = bh / a.H, h = bh % a.H;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r16 = lane_r16(), gq = lane_gq();
    const int off = a.Tk - a.Tq, n = live_len(a.lens, b, a.Tk);
    const int q0 = tile * C::RT, w0 = q0 + wave * 16 * NR;   // first row of the workgroup, of the wave
    const long qs = (long)a.H * DK, kvs = (long)a.H * (DN + DV), os = (long)a.H * DV;
    const T *q = (const T *)a.q + ((long)b * a.Tq * a.H + h) * DK;
    const T *kv = (const T *)a.kv + ((long)b * a.Tk * a.H + h) * (DN + DV);
    const T *kr = (const T *)a.k_rope + (long)b * a.Tk * LATENT_ROPE;
    const float c = a.scale * LOG2E;

    int pos[NR];   // position of this lane's rows; -1: the row sees nothing
    Frag<T> qf[NR][NKB];
#pragma unroll
    for (int g = 0; g < NR; ++g) {
        const int row = w0 + 16 * g + r16;
        const bool live = row < a.Tq && off + row < n;
        pos[g] = live ? off + row : -1;
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb)
            qf[g][kb] = live ? load_frag<T>(q + row * qs + 32 * kb + 8 * gq) : zero_frag<T>();
    }
    f32x4 acc[NCB][NR];
    float m[NR], l[NR];
#pragma unroll
    for (int g = 0; g < NR; ++g) {
        m[g] = -INFINITY;
        l[g] = 0.f;
#pragma unroll
        for (int cb = 0; cb < NCB; ++cb) acc[cb][g] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    // keys that any row of the workgroup, of this wave, may see
    const int last = min(n, off + min(q0 + C::RT, a.Tq));
    const int all = (off + q0 < n) ? (last + KT - 1) / KT : 0;
    const int j0 = CUT ? piece * plan.keys / KT : 0, nt = CUT ? min(all, j0 + plan.keys / KT) : all;
    const int wlast = min(n, off + min(w0 + 16 * NR, a.Tq)), wfull = off + w0 + 1;
    auto load = [&](int j) {
        char *buf = lds + (j & 1) * C::BUF;
        load_rows<C::NCPR, KT>(buf, (const char *)kv, kvs * C::ES, j * KT, n);
        load_rows<C::RCPR, KT>(buf + C::OFF_R, (const char *)kr, LATENT_ROPE * C::ES, j * KT, n);
        load_rows<C::VCPR, KT>(buf + C::OFF_V, (const char *)(kv + DN), kvs * C::ES, j * KT, n);
    };
    const int nb = row_base<T, C::NCPR>(r16), rb = row_base<T, C::RCPR>(r16), vb = col_base<T, C::VCPR>(4 * gq);
    if (nt > j0) load(j0);
    for (int j = j0; j < nt; ++j) {
        const char *kt = lds + (j & 1) * C::BUF, *vt = kt + C::OFF_V;
        const int k0 = j * KT;
        wait_vm<0>();
        lds_barrier();
        if (j + 1 < nt) load(j + 1);
        if (k0 >= wlast || off + w0 >= n) continue;   // nothing for this wave in the tile
        f32x4 s[NS][NR];
#pragma unroll
        for (int t = 0; t < NS; ++t) {
#pragma unroll
            for (int g = 0; g < NR; ++g) s[t][g] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb) {
                const Frag<T> kf = kb < DN / 32
                    ? row_frag<T>(kt + 16 * t * C::NCPR * 16, nb, kb)
                    : row_frag<T>(kt + C::OFF_R + 16 * t * C::RCPR * 16, rb, kb - DN / 32);
#pragma unroll
                for (int g = 0; g < NR; ++g) s[t][g] = mma(s[t][g], kf, qf[g][kb]);
            }
        }
        if (sizeof(T) == 2) pipeline<4, NS * NKB, NS * NKB * NR, 1, NR>();
        if (k0 + KT > wfull || k0 + KT > n) {   // the tile reaches past some row's last key
#pragma unroll
            for (int t = 0; t < NS; ++t)
#pragma unroll
                for (int g = 0; g < NR; ++g)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (k0 + 16 * t + 4 * gq + e > pos[g]) s[t][g][e] = -INFINITY;
        }
#pragma unroll
        for (int g = 0; g < NR; ++g) {
            float mx = -INFINITY;
#pragma unroll
            for (int t = 0; t < NS; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) mx = fmaxf(mx, s[t][g][e]);
            mx = rows_max(mx);
            const bool up = (mx - m[g]) * c > RAISE;   // false while both are -inf
            if (__any(up)) {
                const float mn = up ? mx : m[g];
                const float al = up ? exp2_hw((m[g] - mn) * c) : 1.f;
                m[g] = mn;
                l[g] *= al;
#pragma unroll
                for (int cb = 0; cb < NCB; ++cb) acc[cb][g] *= al;
            }
            const float mb = m[g] == -INFINITY ? 0.f : m[g] * c;
#pragma unroll
            for (int t = 0; t < NS; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float p = exp2_hw(__builtin_fmaf(s[t][g][e], c, -mb));
                    s[t][g][e] = p;
                    l[g] += p;
                }
        }
        // weights rounded to the storage type for the matrix cores (half a step
        // each, as the output itself); their sum is the unrounded one
#pragma unroll
        for (int t = 0; t < NS; t += 2) {
            Frag<T> pf[NR];
#pragma unroll
            for (int g = 0; g < NR; ++g) pf[g] = reg_frag<T>(s[t][g], s[t + 1][g]);
#pragma unroll
            for (int cb = 0; cb < NCB; ++cb) {
                const Frag<T> vf = col_frag<T, C::VCPR>(vt + 16 * t * C::VCPR * 16, vb, cb);
#pragma unroll
                for (int g = 0; g < NR; ++g) acc[cb][g] = mma(acc[cb][g], vf, pf[g]);
            }
        }
        if (sizeof(T) == 2) pipeline<4, NS * NCB, NS / 2 * NCB * NR, 2, NR>();
    }
    T *o = (T *)a.o + ((long)b * a.Tq * a.H + h) * DV;
    const long rows = (long)a.B * a.Tq * a.H;
    float *po = (float *)a.ws + piece * rows * DV + ((long)b * a.Tq * a.H + h) * DV;
    float *pl = (float *)a.ws + plan.pieces * rows * DV + piece * rows;
#pragma unroll
    for (int g = 0; g < NR; ++g) {
        const int row = w0 + 16 * g + r16;
        const float ls = rows_sum(l[g]);
        // a row of a piece may see none of its keys: its sum is 0 (and a NaN where scores are)
        const bool seen = pos[g] >= (CUT ? j0 * KT : 0) && (!CUT || ls != 0.f);
        const float inv = seen ? 1.f / ls : 0.f;
        if (row >= a.Tq) continue;
        if (seen || !CUT) {
#pragma unroll
            for (int cb = 0; cb < NCB; ++cb) {
                const f32x4 v = seen ? acc[cb][g] * inv : f32x4{0.f, 0.f, 0.f, 0.f};
                if (CUT) store4(po + row * os + 16 * cb + 4 * gq, v);
                else store4(o + row * os + 16 * cb + 4 * gq, v);
            }
        }
        const float lg = seen ? m[g] * c + __builtin_amdgcn_logf(ls) : -INFINITY;
        const long at = ((long)b * a.Tq + row) * a.H + h;
        if (gq == 0) {
            if (CUT) pl[at] = lg;
            else if (a.lse) a.lse[at] = lg * LN2;
        }
    }
}

// Joins the pieces of every row; DV / 4 lanes a row.
template <typename T, int DV>
__global__ __launch_bounds__(256) void latent_fwd_join_kernel(LatentFwdArgs a, int pieces)
{
    constexpr int LPR = DV / 4;
    const long rows = (long)a.B * a.Tq * a.H, row = (long)blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
    const int at = threadIdx.x % LPR * 4;
    if (row >= rows) return;
    const float *po = (const float *)a.ws, *pl = po + pieces * rows * DV;
    float top = -INFINITY, ls = 0.f;
    for (int i = 0; i < pieces; ++i) top = fmaxf(top, pl[i * rows + row]);
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    for (int i = 0; i < pieces; ++i) {
        const float lg = pl[i * rows + row];
        if (lg == -INFINITY) continue;   // nothing was written
        const float f = exp2_hw(lg - top);
        ls += f;
        sum += f * *reinterpret_cast<const f32x4 *>(po + (i * rows + row) * DV + at);
    }
    store4((T *)a.o + row * DV + at, ls != 0.f ? sum * (1.f / ls) : sum);
    if (a.lse && at == 0) a.lse[row] = ls != 0.f ? (top + __builtin_amdgcn_logf(ls)) * LN2 : -INFINITY;
}

template <typename T, int DN, int DV, int NR, bool CUT>
static hipError_t fwd_enqueue(const LatentFwdArgs &a, const FwdPlan &plan, hipStream_t st)
{
    typedef FwdCfg<T, DN, DV, NR> C;
    const int ntiles = (a.Tq + C::RT - 1) / C::RT;
    auto k = latent_fwd_kernel<T, DN, DV, NR, CUT>;
    const hipError_t e = hipFuncSetAttribute((const void *)k, hipFuncAttributeMaxDynamicSharedMemorySize, 2 * C::BUF);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k, dim3((unsigned)((long)ntiles * a.B * a.H * plan.pieces)), dim3(256), 2 * C::BUF, st, a, ntiles, plan);
    if (CUT) {
        const long rows = (long)a.B * a.Tq * a.H, per = 256 / (DV / 4);
        hipLaunchKernelGGL((latent_fwd_join_kernel<T, DV>), dim3((unsigned)((rows + per - 1) / per)), dim3(256), 0, st, a, plan.pieces);
    }
    return hipGetLastError();
}

template <typename T, int DN, int DV> static hipError_t fwd_launch(const LatentFwdArgs &a, hipStream_t st)
{
    constexpr bool BF = sizeof(T) == 2;
    const FwdPlan plan = fwd_plan(BF, a.B, a.Tq, a.Tk, a.H);
    if constexpr (BF) {
        if (plan.nr == 2)
            return plan.pieces > 1 ? fwd_enqueue<T, DN, DV, 2, true>(a, plan, st) : fwd_enqueue<T, DN, DV, 2, false>(a, plan, st);
    }
    return plan.pieces > 1 ? fwd_enqueue<T, DN, DV, 1, true>(a, plan, st) : fwd_enqueue<T, DN, DV, 1, false>(a, plan, st);
}

hipError_t latent_fwd_launch(bool bf16, int dn, int dv, const LatentFwdArgs &a, hipStream_t st)
{
    if (bf16) {
        if (dn == 128) return dv == 128 ? fwd_launch<__bf16, 128, 128>(a, st) : fwd_launch<__bf16, 128, 64>(a, st);
        return dv == 128 ? fwd_launch<__bf16, 64, 128>(a, st) : fwd_launch<__bf16, 64, 64>(a, st);
    }
    if (dn == 128) return dv == 128 ? fwd_launch<float, 128, 128>(a, st) : fwd_launch<float, 128, 64>(a, st);
    return dv == 128 ? fwd_launch<float, 64, 128>(a, st) : fwd_launch<float, 64, 64>(a, st);
}

unsigned long long latent_fwd_workspace(bool bf16, int B, int Tq, int Tk, int H, int dv)
{
    const FwdPlan plan = fwd_plan(bf16, B, Tq, Tk, H);
    return plan.pieces > 1 ? (unsigned long long)plan.pieces * B * Tq * H * (dv + 1) * 4 : 0;
}

} // namespace gdn
