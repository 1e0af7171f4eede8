// attn_bwd.hip -- gradients of the packed grouped attention (gfx950).
//
//   P_ij = exp(s_ij - lse_i),  D_i = do_i . o_i,  dS_ij = scale P_ij (do_i . v_j - D_i)
//   dv_j = sum_i P_ij do_i,  dk_j = sum_i dS_ij q_i,  dq_i = sum_j dS_ij k_j
//
// A row that sees one key (position 0) has P = 1 and dS = 0, as D = dP; from a rounded lse and o
// there would be a residue in place of the zero, so both kernels leave its dS out.
//
// The sums of dk and dv run over the rows of all G query heads that share the key head: rows
// (token, head) in one run, as in the forward's tiles.  No atomics, so results do not depend
// on the order in which workgroups run: one kernel owns query rows and walks their keys (dq),
// one owns keys and walks the rows that see them (dk, dv); the scores are computed in both.
// What walks by keys is shared by a fixed number of workgroups, what walks by few query rows is
// cut into pieces; the sums of what is cut a third kernel adds up in order.
//
// Seven products for the five of the formulas, bound by the matrix cores: 8192 packed tokens (one
// sequence of 4999 among seven) of 16 over 4 heads of 128, bf16, take 432 to 440 us; in a trace
// dq 191 (0.93 PFLOP/s over its three products), dk and dv 246 (0.96 over four), the sums 16.
#include "attn.h"

namespace gdn {

// Workspace: float D[Tq][Hq]; where dq is cut, float dq[kp][Tq][Hq][D]; long prefix[B + 1],
// the rows that the owners of keys walk by before each sequence, then for each share of them
// its first and last piece, float dkv[slot][2 D] (dk, then dv), slot = min(OWN, Tk) keys.
struct AttnBwdWs {
    long dq, prefix, dkv, bytes;
    int rows;
    __host__ __device__ AttnBwdWs(const AttnBwdPlan &p, int B, int Tq, int Tk, int Hk, int G, int d, int own) {
        const long qr = (long)Tq * Hk * G;
        rows = Tk < own ? Tk : own;
        dq = (qr * 4 + 255) & ~255L;
        prefix = dq + (p.kp > 1 ? p.kp * qr * d * 4 : 0);
        dkv = prefix + (((long)(B + 1) * 8 + 255) & ~255L);
        bytes = dkv + 2L * p.shares * rows * 2 * d * 4;
    }
};

// This lane's share of a row's do . o (the four 16-lane rows hold its columns).
template <typename T> __device__ __forceinline__ float frag_dot(const Frag<T> &x, const Frag<T> &y) {
    float s = 0.f;
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int e = 0; e < 8; ++e) s += (float)x.v[e] * (float)y.v[e];
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) s += x.lo[e] * y.lo[e] + x.hi[e] * y.hi[e];
    }
    return s;
}

// P from wave to wave: fp32 as it is, beside bf16 operands as fp16 of P 2^12 (half the
// room).  P <= 1, so nothing overflows, and down to P = 2^-26 it is off by 2^-11 of itself,
// an eighth of what dS, which it becomes, is rounded by; below, by 2^-37.  The exponential
// gives the power of two along, which comes out of dk and dv at the end.
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
template <typename T> __device__ __forceinline__ constexpr float hand_bits() { return sizeof(T) == 2 ? 12.f : 0.f; }
template <typename T> __device__ __forceinline__ void hand_over(char *to, f32x4 p) {
    if constexpr (sizeof(T) == 2) {
        f16x4 h;
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = (_Float16)p[e];
        *reinterpret_cast<f16x4 *>(to) = h;
    } else {
        *reinterpret_cast<f32x4 *>(to) = p;
    }
}
template <typename T> __device__ __forceinline__ f32x4 take_over(const char *from) {
    if constexpr (sizeof(T) == 2) {
        const f16x4 h = *reinterpret_cast<const f16x4 *>(from);
        return f32x4{(float)h[0], (float)h[1], (float)h[2], (float)h[3]};
    } else {
        return *reinterpret_cast<const f32x4 *>(from);
    }
}

template <typename T, int D> struct AttnBwdCfg {
    static constexpr int OWN = attn_own(sizeof(T) == 2), ST = attn_walk(sizeof(T) == 2), NG = OWN / 64;
    static constexpr int ES = (int)sizeof(T), CPR = D * ES / 16;
    static constexpr int OFF_V = ST * CPR * 16, BUF = 2 * OFF_V;   // a tile: [ST][D] of k or q, [ST][D] of v or do
    static constexpr int ROWS = 2 * ST * 4;                        // lse and D of the tile's rows
    static constexpr int HP = 64 * 4 * (ES == 2 ? 2 : 4);          // four values of P of each lane
    static constexpr int HAND = 2 * ST / 16 * NG * HP;             // P of two tiles, one pair of waves
    static constexpr int KV_LDS = 3 * (BUF + ROWS) + 4 * HAND;
    static_assert(KV_LDS <= 160 * 1024, "LDS");
};

constexpr int OWN_COST = 2;   // what a change of owners takes, in rows for each of its keys (see Share)

// Owners of OWN keys of a sequence, and the rows that walk by: all that see one of the keys.
// Those are the last of the sequence: row r of a key head is token r / G, head r % G.
template <int OWN> struct KeyTiles {
    static constexpr int extra = OWN_COST * OWN;
    int lq, lk, g;
    __device__ __forceinline__ KeyTiles(const Seq &s, int g) : lq(s.lq), lk(s.lk), g(g) {}
    __device__ __forceinline__ int count() const { return (lk + OWN - 1) / OWN; }
    __device__ __forceinline__ int first() const { return 0; }
    __device__ __forceinline__ int walk(int i) const { return min(lq, lk - i * OWN) * g; }
    __device__ __forceinline__ long before(int i) const {
        const int f = lq > lk ? 0 : min(i, (lk - lq) / OWN + 1);   // owners that all rows see
        return ((long)f * lq + (long)(i - f) * lk - OWN * ((long)i * (i - 1) - (long)f * (f - 1)) / 2) * g + (lq > 0 ? (long)i * extra : 0);
    }
    __device__ __forceinline__ long all() const { return before(count()); }
};

constexpr int BWD_LEAST = 2;   // tiles of a share

// dk and dv.  Four pairs of waves; a pair owns 16 NG keys.  The first of the pair
// computes the scores and P and adds up dv^T (k and dv in its registers), the second
// takes P over, computes dP and dS and adds up dk^T (v and dk in its registers): the
// same number of products for both, and of q and do each reads from LDS one along
// the rows and the other across them, where one wave for both would not have the
// registers for 32 keys, and with 16 keys would read twice as much.  The second is
// one tile of query rows behind, so neither waits for the other inside a tile.
// Scores have query rows on the accumulator's rows: P and dS feed the gradient
// products as B operands straight from the registers, and P changes hands between
// equal lanes.  The workgroups take equal runs of all tiles that walk by (whole owners of keys
// leave the longest sequence's first ones as the call's time: 954 us for what is 618 in
// shares); 32 keys a wave and 64 query rows a tile fill the LDS of a unit, so one workgroup.
template <typename T, int D>
__global__ __launch_bounds__(512, 1) void attn_bwd_kv_kernel(AttnArgs a, AttnBwdPlan plan)
{
    typedef AttnBwdCfg<T, D> C;
    constexpr int NG = C::NG, ST = C::ST, NKB = D / 32, NC = D / 16, OWN = C::OWN;
    constexpr int NS = ST / 16;
    extern __shared__ char lds[];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r16 = lane_r16(), gq = lane_gq();
    const int pair = wave & 3, lane = threadIdx.x & 63, Hq = a.Hk * a.G;
    const bool isv = wave < 4;   // the first of the pair
    const AttnBwdWs lay(plan, a.B, a.Tq, a.Tk, a.Hk, a.G, D, OWN);
    // shares of one head, which walk by the same rows, on one XCD
    const int share = blockIdx.x % 8 * (plan.shares / 8) + blockIdx.x / 8;
    auto make = [&](const Seq &s) { return KeyTiles<OWN>(s, a.G); };
    Share sh;
    if (!share_begin<ST>(a, make, share, plan.shares, BWD_LEAST, (long *)((char *)a.ws + lay.prefix), sh) || !share_next<ST>(a, make, sh)) return;
    const float c = a.scale * LOG2E;
    float *stat = (float *)(lds + 3 * C::BUF);                  // [3][2][ST]: lse and D of the rows
    char *hand = lds + 3 * (C::BUF + C::ROWS) + pair * C::HAND; // [2][ST / 16 NG][64 lanes]: P of a tile, four values a lane
    const int rb = row_base<T, C::CPR>(r16), cb = col_base<T, C::CPR>(4 * gq);
    int count = 0;   // tiles so far: which of three buffers, and of two places for P

    // Copies of tile j of a run into its buffer: rows r0 .. of the packed (token, head) rows
    // that see the owner's keys, r0 in token t0 of the sequence at head g0.  A row is at
    // token (g0 + row) / G behind t0: all offsets of a tile in 24-bit products from scalar
    // addresses (64-bit ones a lane took as long as the tile's scores).
    auto first_row = [&](const Run &r) { return max(0, r.t * OWN - (r.s.lk - r.s.lq)) * a.G; };
    auto load = [&](const Run &r, int j, int buf) {
        const int r0 = first_row(r) + (r.j + j) * ST, left = min(r.s.lq * a.G, first_row(r) + r.end * ST) - r0;
        const int t0 = uniform(quotient(r0, a.g_mul, a.g_shift)), g0 = r0 - t0 * a.G;
        constexpr int RP = 512 / C::CPR;
        static_assert(ST % RP == 0 && RP % 16 == 0, "");
        const int row = threadIdx.x / C::CPR, ch = ((threadIdx.x % C::CPR) ^ swz<C::CPR>(row)) * 16;
        const char *to = lds + uniform(buf * C::BUF + wave * 1024);
        const long tok = (long)r.s.q0 + t0, head = (long)tok * Hq + r.h * a.G;
        const char *q = uniform((const T *)a.q + tok * a.qs + r.h * a.G * D), *d_o = uniform((const T *)a.d_o + head * D);
        const unsigned qst = (unsigned)a.qs * C::ES, ost = Hq * D * C::ES;
#pragma unroll
        for (int i = 0; i < ST / RP; ++i) {
            const int x = g0 + i * RP + row, t = (int)(__umul24(x, a.g_mul16) >> 16), g = x - t * a.G;
            const unsigned in = g * (D * C::ES) + ch, oq = __umul24(t, qst) + in, od = __umul24(t, ost) + in;
            if (left >= ST) {
                copy16u(q, oq, to + i * 512 * 16);
                copy16u(d_o, od, to + C::OFF_V + i * 512 * 16);
            } else {
                const bool is = i * RP + row < left;
                copy16(is ? q + oq : (const char *)latent_zero, to + i * 512 * 16);
                copy16(is ? d_o + od : (const char *)latent_zero, to + C::OFF_V + i * 512 * 16);
            }
        }
        if (wave < 2 && lane < ST) {   // lse by the first wave, D by the second
            const int x = g0 + lane, t = (int)(__umul24(x, a.g_mul16) >> 16);
            const float *src = (wave ? (const float *)a.ws : a.lse) + head + t * Hq + (x - t * a.G);
            copy4(lane < left ? (const void *)src : (const void *)latent_zero, (char *)(stat + uniform((buf * 2 + wave) * ST)));
        }
    };
    load(sh.r, 0, 0);
    for (bool more = true; more;) {   // one owner, or what the share has of its walk
        const Run cur = sh.r;
        const Seq sq = cur.s;
        const int off = sq.lk - sq.lq, n = sq.lk, h = cur.h;
        const int k0 = cur.t * OWN, w0 = k0 + pair * 16 * NG;
        const int qfirst = first_row(cur) + cur.j * ST, nt = cur.end - cur.j, qn = min(sq.lq * a.G, qfirst + nt * ST);
        // before tile j: it is there, and P of tile j - 1 is whole
        auto sync = [&](int j) {
            if (j < nt) wait_vm<0>();
            lds_barrier();
            if (j + 1 < nt) load(cur, j + 1, uniform((count + j + 1) % 3));   // over tile j - 2
        };
        // first row that sees key j: its token is j - off
        auto sees = [&](int j) { return (j - off) * a.G; };
        auto seen = [&](int r) { return r + ST - 1 >= sees(w0) && w0 < n; };   // whether a row of the tile sees a key of the wave
        // rows of one key at the run's begin: the first that walk by the first owner
        const int single = cur.t == 0 && off <= 0 ? a.G - cur.j * ST : 0;
        const T *x = isv ? (const T *)a.k + sq.k0 * a.ks + h * D : (const T *)a.v + sq.k0 * a.vs + h * D;
        const long xs = isv ? a.ks : a.vs;
        Frag<T> xf[NG][NKB];   // k for the first of the pair, v for the second
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const int key = w0 + 16 * g + r16;
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb) xf[g][kb] = key < n ? load_frag<T>(x + key * xs + 32 * kb + 8 * gq) : zero_frag<T>();
        }
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb) landed<T>(xf[g][kb]);
        f32x4 acc[NC][NG];   // dv^T, dk^T
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int i = 0; i < NC; ++i) acc[i][g] = f32x4{0.f, 0.f, 0.f, 0.f};

        if (isv) {
#pragma unroll 1
            for (int j = 0; j <= nt; ++j) {
                sync(j);
                if (j == nt) break;
                const char *qt = lds + (count + j) % 3 * C::BUF, *dt = qt + C::OFF_V;
                const float *st = stat + (count + j) % 3 * 2 * ST;
                char *to = hand + ((count + j) & 1) * (C::HAND / 2) + lane * (C::HP / 64);
                const int r0 = qfirst + j * ST;
                if (!seen(r0)) continue;
                f32x4 s[NS][NG];
#pragma unroll
                for (int u = 0; u < NS; ++u) {
#pragma unroll
                    for (int g = 0; g < NG; ++g) s[u][g] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int kb = 0; kb < NKB; ++kb) {
                        const Frag<T> f = row_frag<T>(qt + 16 * u * C::CPR * 16, rb, kb);
#pragma unroll
                        for (int g = 0; g < NG; ++g) s[u][g] = mma(s[u][g], f, xf[g][kb]);
                    }
                }
                if (sizeof(T) == 2) pipeline<6, NS * NKB, NS * NKB * NG, 1, NG>();
                GDN_SCHED_FENCE();
#pragma unroll
                for (int u = 0; u < NS; ++u) {
                    const f32x4 ls = *reinterpret_cast<const f32x4 *>(st + 16 * u + 4 * gq) * LOG2E - hand_bits<T>();
#pragma unroll
                    for (int g = 0; g < NG; ++g)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[u][g][e] = exp2_hw(__builtin_fmaf(s[u][g][e], c, -ls[e]));
                }
                if (r0 < sees(w0 + 16 * NG - 1) || r0 + ST > qn) {
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        const int lim = sees(w0 + 16 * g + r16) - r0 - 4 * gq, end = qn - r0 - 4 * gq;
#pragma unroll
                        for (int u = 0; u < NS; ++u)
#pragma unroll
                            for (int e = 0; e < 4; ++e) s[u][g][e] = ((16 * u + e < lim) | (16 * u + e >= end)) ? 0.f : s[u][g][e];
                    }
                }
#pragma unroll
                for (int u = 0; u < NS; ++u)
#pragma unroll
                    for (int g = 0; g < NG; ++g) hand_over<T>(to + (u * NG + g) * C::HP, s[u][g]);
                // P (and below dS) rounded to the storage type for the matrix cores: half
                // a step each, as the gradients themselves
#pragma unroll
                for (int u = 0; u < NS; u += 2) {
                    Frag<T> pf[NG];
#pragma unroll
                    for (int g = 0; g < NG; ++g) pf[g] = reg_frag<T>(s[u][g], s[u + 1][g]);
#pragma unroll
                    for (int v = 0; v < NC; ++v) {
                        const Frag<T> f = col_frag<T, C::CPR>(dt + 16 * u * C::CPR * 16, cb, v);
#pragma unroll
                        for (int g = 0; g < NG; ++g) acc[v][g] = mma(acc[v][g], f, pf[g]);
                    }
                }
                if (sizeof(T) == 2) pipeline<6, NS * NC, NS / 2 * NC * NG, 2, NG>();
            }
        } else {
#pragma unroll 1
            for (int j = 0; j <= nt; ++j) {
                sync(j);
                if (j == 0) continue;
                const int k = count + j - 1;
                const char *qt = lds + k % 3 * C::BUF, *dt = qt + C::OFF_V;
                const float *st = stat + (k % 3 * 2 + 1) * ST;
                const char *from = hand + (k & 1) * (C::HAND / 2) + lane * (C::HP / 64);
                if (!seen(qfirst + (j - 1) * ST)) continue;
                f32x4 dp[NS][NG];
#pragma unroll
                for (int u = 0; u < NS; ++u) {
#pragma unroll
                    for (int g = 0; g < NG; ++g) dp[u][g] = -*reinterpret_cast<const f32x4 *>(st + 16 * u + 4 * gq);   // D
#pragma unroll
                    for (int v = 0; v < NKB; ++v) {
                        const Frag<T> f = row_frag<T>(dt + 16 * u * C::CPR * 16, rb, v);
#pragma unroll
                        for (int g = 0; g < NG; ++g) dp[u][g] = mma(dp[u][g], f, xf[g][v]);
                    }
                }
                if (sizeof(T) == 2) pipeline<6, NS * NKB, NS * NKB * NG, 1, NG>();
                GDN_SCHED_FENCE();
#pragma unroll
                for (int u = 0; u < NS; ++u) {
#pragma unroll
                    for (int g = 0; g < NG; ++g) dp[u][g] *= take_over<T>(from + (u * NG + g) * C::HP);
                }
                if ((j - 1) * ST < single) {
                    const int end = single - (j - 1) * ST - 4 * gq;
#pragma unroll
                    for (int u = 0; u < NS; ++u)
#pragma unroll
                        for (int g = 0; g < NG; ++g)
#pragma unroll
                            for (int e = 0; e < 4; ++e) dp[u][g][e] = 16 * u + e < end ? 0.f : dp[u][g][e];
                }
#pragma unroll
                for (int u = 0; u < NS; u += 2) {
                    Frag<T> sf[NG];
#pragma unroll
                    for (int g = 0; g < NG; ++g) sf[g] = reg_frag<T>(dp[u][g], dp[u + 1][g]);
#pragma unroll
                    for (int v = 0; v < NC; ++v) {
                        const Frag<T> f = col_frag<T, C::CPR>(qt + 16 * u * C::CPR * 16, cb, v);
#pragma unroll
                        for (int g = 0; g < NG; ++g) acc[v][g] = mma(acc[v][g], f, sf[g]);
                    }
                }
                if (sizeof(T) == 2) pipeline<6, NS * NC, NS / 2 * NC * NG, 2, NG>();
            }
        }
        count = uniform(count + nt);
        more = share_next<ST>(a, make, sh);
        if (more) load(sh.r, 0, uniform(count % 3));   // over the tile before the last
        const bool whole = cur.j == 0 && cur.end == cur.n;
        const float by = (isv ? 1.f : a.scale) * exp2_hw(-hand_bits<T>());
        T *out = isv ? (T *)a.dv + sq.k0 * a.dvs + h * D : (T *)a.dk + sq.k0 * a.dks + h * D;
        const long outs = isv ? a.dvs : a.dks;
        float *sum = (float *)((char *)a.ws + lay.dkv) + (share * 2 + (cur.j == 0)) * (long)lay.rows * 2 * D + (isv ? D : 0);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const int key = w0 + 16 * g + r16;
            if (key >= n) continue;
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const f32x4 v = acc[i][g] * by;
                if (whole) store4(out + key * outs + 16 * i + 4 * gq, v);
                else store4(sum + (key - k0) * 2 * D + 16 * i + 4 * gq, v);
            }
        }
    }
}

// dq, and D for the kernel above, which is launched after this one.  A wave owns 16
// NG rows, q and do of them in registers; scores are transposed as in the forward pass,
// and dS^T feeds dq^T = K^T dS^T from the registers.
// Two workgroups a unit hide each other's waits: row tiles stay whole in large calls (in
// shares, as above, the join costs more: 333 rows 48 us, whole 41).  The first key tile is
// under way before the rows' operands (one sequence of 128 31 us for all three kernels from 32).
template <typename T, int D, bool CUT>
__global__ __launch_bounds__(256, 2) void attn_bwd_q_kernel(AttnArgs a, AttnBwdPlan plan)
{
    typedef AttnBwdCfg<T, D> C;
    constexpr int NG = C::NG, ST = C::ST, NKB = D / 32, NC = D / 16;
    constexpr bool BF = sizeof(T) == 2;
    extern __shared__ char lds[];
    const int h = blockIdx.x % a.Hk, piece = CUT ? blockIdx.x / a.Hk % plan.kp : 0, per = plan.tokens;
    const int pieces = CUT ? plan.kp : 1;
    const Item it = find_tile(a, per, blockIdx.x / a.Hk / pieces, gridDim.x / a.Hk / pieces);
    if (it.b < 0) return;
    const Seq sq = seq_of(a, it.b);
    const AttnTiles tl(per, sq);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r16 = lane_r16(), gq = lane_gq();
    const int off = tl.off, n = sq.lk, Hq = a.Hk * a.G, t0 = uniform(it.i) * per, lr0 = wave * 16 * NG;
    const int nlive = min(per, sq.lq - t0) * a.G;
    const T *k = (const T *)a.k + sq.k0 * a.ks + h * D, *v = (const T *)a.v + sq.k0 * a.vs + h * D;
    const float c = a.scale * LOG2E;

    const int all = uniform((tl.walk(it.i) + ST - 1) / ST);
    const int j0 = CUT ? piece * (plan.kstep / ST) : 0, nt = CUT && piece + 1 < plan.kp ? min(all, j0 + plan.kstep / ST) : all;
    if (CUT && piece > 0 && nt <= j0) return;   // the last kernel knows which pieces there are
    auto load = [&](int j) {
        char *to = lds + (j & 1) * C::BUF;
        load_tile<C::CPR, ST>(to, (const char *)k, a.ks * C::ES, j * ST, n, threadIdx.x);
        load_tile<C::CPR, ST>(to + C::OFF_V, (const char *)v, a.vs * C::ES, j * ST, n, threadIdx.x);
    };
    // Of few keys, D needs all of them first (below); two tiles then stay where they are.
    const bool few = BF && all <= 2;
    if (few ? all > 0 : nt > j0) load(few ? 0 : j0);

    int pos[NG];
    long row[NG];   // of [Tq Hq]
    float ls[NG], dd[NG];
    Frag<T> qf[NG][NKB], of[NG][NKB];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        const int lr = lr0 + 16 * g + r16, i = quotient(lr, a.g_mul, a.g_shift), tok = t0 + i, head = h * a.G + lr - i * a.G;
        const bool live = lr < nlive && off + tok >= 0;
        pos[g] = live ? off + tok : -1;
        row[g] = (sq.q0 + (long)tok) * Hq + head;
        const T *q = (const T *)a.q + (sq.q0 + (long)tok) * a.qs + head * D;
        const T *d_o = (const T *)a.d_o + row[g] * D, *o = (const T *)a.o + row[g] * D;
        ls[g] = live ? a.lse[row[g]] * LOG2E : 0.f;
        float dot = 0.f;
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb) {
            qf[g][kb] = live ? load_frag<T>(q + 32 * kb + 8 * gq) : zero_frag<T>();
            of[g][kb] = live ? load_frag<T>(d_o + 32 * kb + 8 * gq) : zero_frag<T>();
            if (live) dot += frag_dot<T>(of[g][kb], load_frag<T>(o + 32 * kb + 8 * gq));
        }
        dd[g] = rows_sum(dot);
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        asm volatile("" : "+v"(ls[g]));
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb) {
            landed<T>(qf[g][kb]);
            landed<T>(of[g][kb]);
        }
    }
    f32x4 dq[NC][NG];
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int i = 0; i < NC; ++i) dq[i][g] = f32x4{0.f, 0.f, 0.f, 0.f};

    // keys that some, that all of the wave's rows see
    const int wend = min(lr0 + 16 * NG, nlive) - 1;
    const int wlast = wend < lr0 ? 0 : off + t0 + quotient(max(wend, 0), a.g_mul, a.g_shift) + 1;
    const int wfull = off + t0 + quotient(lr0, a.g_mul, a.g_shift) + 1;
    const int rb = row_base<T, C::CPR>(r16), cb = col_base<T, C::CPR>(4 * gq);
    // of 32 keys (block t of tile j): P, and dP in the same layout
    auto products = [&](int j, int t, f32x4 (&s)[2][NG], f32x4 (&dp)[2][NG]) {
        const char *kt = lds + (j & 1) * C::BUF, *vt = kt + C::OFF_V;
        const int k0 = j * ST, rbl = pin(rb);
        const bool part = k0 + ST > wfull;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                s[u][g] = f32x4{0.f, 0.f, 0.f, 0.f};
                dp[u][g] = s[u][g];
            }
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb) {
                const Frag<T> f = row_frag<T>(kt + (32 * t + 16 * u) * C::CPR * 16, rbl, kb);
#pragma unroll
                for (int g = 0; g < NG; ++g) s[u][g] = mma(s[u][g], f, qf[g][kb]);
            }
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb) {
                const Frag<T> f = row_frag<T>(vt + (32 * t + 16 * u) * C::CPR * 16, rbl, kb);
#pragma unroll
                for (int g = 0; g < NG; ++g) dp[u][g] = mma(dp[u][g], f, of[g][kb]);
            }
            if (BF) pipeline<4, 2 * NKB, 2 * NKB * NG, 1, NG>();
            GDN_SCHED_FENCE();
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[u][g][e] = exp2_hw(__builtin_fmaf(s[u][g][e], c, -ls[g]));
            if (part) {
#pragma unroll
                for (int g = 0; g < NG; ++g)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        s[u][g][e] = k0 + 32 * t + 16 * u + 4 * gq + e > pos[g] ? 0.f : s[u][g][e];
            }
        }
    };
    if (few) {
        // The first rows, of few keys: o, rounded to bf16, is as large as v there, and the
        // error that its rounding leaves in D, the same for all keys of a row, would be as
        // large as the rounding of dS.  They have D from P and dP themselves.  The others
        // have do . o, where that error is small as long as a row's weights are spread over
        // its n keys (1 / sqrt(n) as large), and is not where one key takes most of them.
        float sum[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) sum[g] = 0.f;
        for (int j = 0; j < all; ++j) {
            wait_vm<0>();
            lds_barrier();
            if (j + 1 < all) load(j + 1);
#pragma unroll 1
            for (int t = 0; t < ST / 32; ++t) {
                f32x4 s[2][NG], dp[2][NG];
                products(j, t, s, dp);
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int g = 0; g < NG; ++g)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sum[g] += s[u][g][e] * dp[u][g][e];
            }
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) dd[g] = rows_sum(sum[g]);
    }
    if (piece == 0 && gq == 0) {
#pragma unroll
        for (int g = 0; g < NG; ++g)   // also of rows that see nothing: they stand in walked tiles
            if (lr0 + 16 * g + r16 < nlive) ((float *)a.ws)[row[g]] = dd[g];
    }
    for (int j = j0; j < nt; ++j) {
        const char *kt = lds + (j & 1) * C::BUF;
        if (!few) {
            wait_vm<0>();
            lds_barrier();
            if (j + 1 < nt) load(j + 1);
        }
        if (j * ST >= wlast) continue;
#pragma unroll 1
        for (int t = 0; t < ST / 32; ++t) {
            f32x4 s[2][NG], dp[2][NG];
            products(j, t, s, dp);
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int g = 0; g < NG; ++g) dp[u][g] = s[u][g] * (dp[u][g] - dd[g]);
            const int cbl = pin(cb);
            Frag<T> sf[NG];
#pragma unroll
            for (int g = 0; g < NG; ++g) sf[g] = reg_frag<T>(dp[0][g], dp[1][g]);
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const Frag<T> f = col_frag<T, C::CPR>(kt + 32 * t * C::CPR * 16, cbl, i);
#pragma unroll
                for (int g = 0; g < NG; ++g) dq[i][g] = mma(dq[i][g], f, sf[g]);
            }
            if (BF) pipeline<4, 2 * NC, NC * NG, 2, NG>();
        }
    }
    float *sum = (float *)((char *)a.ws + AttnBwdWs(plan, a.B, a.Tq, a.Tk, a.Hk, a.G, D, C::OWN).dq) + (long)piece * a.Tq * Hq * D;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        const int lr = lr0 + 16 * g + r16, i = quotient(lr, a.g_mul, a.g_shift);
        if (lr >= nlive) continue;
        T *out = (T *)a.dq + (sq.q0 + (long)(t0 + i)) * a.dqs + (h * a.G + lr - i * a.G) * D;
#pragma unroll
        for (int e = 0; e < NC; ++e) {
            const f32x4 x = pos[g] > 0 ? dq[e][g] * a.scale : f32x4{0.f, 0.f, 0.f, 0.f};   // at 0: one key, dS = 0
            if (CUT) store4(sum + row[g] * D + 16 * e + 4 * gq, x);
            else store4(out + 16 * e + 4 * gq, x);
        }
    }
}

// The sums over pieces and shares, in order: of dq by the first ndq workgroups (D / 4 lanes a
// row), of dk and dv by the others (2 D / 4 lanes take `run` tokens of a head, one after the
// other), which also write the keys that no row sees.  A piece counts for the rows that its
// workgroup has worked on.
template <typename T, int D> __global__ __launch_bounds__(256) void attn_bwd_sum_kernel(AttnArgs a, AttnBwdPlan plan, int ndq, int run)
{
    typedef AttnBwdCfg<T, D> C;
    constexpr int LPR = D / 4;
    const AttnBwdWs lay(plan, a.B, a.Tq, a.Tk, a.Hk, a.G, D, C::OWN);
    if ((int)blockIdx.x < ndq) {
        const unsigned id = blockIdx.x * 256 + threadIdx.x, row = id / LPR, H = a.Hk * a.G;   // the grid has less than 2^32 threads
        if (row >= a.Tq * H) return;
        const int token = (int)(row / H), head = (int)row - token * (int)H, col = (int)(id % LPR) * 4;
        const Seq s = seq_lane(a, seq_at(a.cu_q, a.B, a.Tq, token));
        const int i = token - s.q0;
        if (i < 0 || i >= s.lq) return;   // of no sequence
        // the owner of the row walks the keys up to its last row's position; piece 0 always writes
        const int end = min(plan.kp, max(1, (AttnTiles(plan.tokens, s).walk(i / plan.tokens) + plan.kstep - 1) / plan.kstep));
        const float *part = (const float *)((const char *)a.ws + lay.dq) + (long)row * D + col;
        f32x4 x = {0.f, 0.f, 0.f, 0.f};
        for (int p = 0; p < end; ++p) x += *reinterpret_cast<const f32x4 *>(part + p * (long)a.Tq * H * D);
        store4((T *)a.dq + token * a.dqs + head * D + col, x);
        return;
    }
    const unsigned id = (blockIdx.x - ndq) * 256 + threadIdx.x, group = id / (2 * LPR);
    const int first = (int)(group / (unsigned)a.Hk), head = (int)group - first * a.Hk, col = (int)(id % (2 * LPR)) * 4;
    const long *prefix = (const long *)((const char *)a.ws + lay.prefix);
    const float *parts = (const float *)((const char *)a.ws + lay.dkv) + col;
    Seq s = {0, 0, 0, 0};
    int own = 0, end = 0, wf = 0, wl = -1;   // tokens of one owner, and its shares
    for (int token = first * run; token < min(a.Tk, (first + 1) * run); ++token) {
        if (token >= end) {
            const int b = seq_at(a.cu_k ? a.cu_k : a.cu_q, a.B, a.Tk, token);
            s = seq_lane(a, b);
            const int i = token - s.k0;
            if (i < 0 || i >= s.lk) continue;   // of no sequence
            const KeyTiles<C::OWN> owners(s, a.G);
            const int t = i / C::OWN;
            own = s.k0 + t * C::OWN;
            end = min(own + C::OWN, s.k0 + s.lk);
            wf = 0, wl = -1;
            if (s.lq > 0)
                share_range<C::ST>(prefix[b] + head * owners.all() + owners.before(t), owners, t, share_each<C::ST>(prefix[a.B], plan.shares, BWD_LEAST), wf, wl);
        }
        if (s.lq > 0 && wf == wl) continue;   // written by its one workgroup
        f32x4 x = {0.f, 0.f, 0.f, 0.f};
        const float *part = parts + (token - own) * 2 * D;
#pragma unroll 4
        for (int w = wf; w <= wl; ++w) x += *reinterpret_cast<const f32x4 *>(part + (w * 2 + (w == wf)) * (long)lay.rows * 2 * D);
        store4(col < D ? (T *)a.dk + token * a.dks + head * D + col : (T *)a.dv + token * a.dvs + head * D + col - D, x);
    }
}

template <typename T, int D> static hipError_t bwd_launch(AttnArgs a, hipStream_t st)
{
    typedef AttnBwdCfg<T, D> C;
    const AttnBwdPlan plan = attn_bwd_plan(sizeof(T) == 2, a.B, a.Tq, a.Tk, a.Hk, a.G);
    divisor(a.G, a.g_mul, a.g_shift);
    a.g_mul16 = (65536 + a.G - 1) / a.G;
    auto kkv = attn_bwd_kv_kernel<T, D>;
    auto kq = plan.kp > 1 ? attn_bwd_q_kernel<T, D, true> : attn_bwd_q_kernel<T, D, false>;
    hipError_t e = hipFuncSetAttribute((const void *)kkv, hipFuncAttributeMaxDynamicSharedMemorySize, C::KV_LDS);
    if (e != hipSuccess) return e;
    static_assert(2 * C::BUF <= 64 * 1024, "more dynamic LDS has to be asked for");
    if (plan.qtiles > 0) hipLaunchKernelGGL(kq, dim3((unsigned)(plan.qtiles * a.Hk * plan.kp)), dim3(256), 2 * C::BUF, st, a, plan);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (a.Tk > 0) hipLaunchKernelGGL(kkv, dim3((unsigned)plan.shares), dim3(512), C::KV_LDS, st, a, plan);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    // Four tokens for one search of their owner and its shares, where that leaves 4096 runs (16 of
    // 512, 32 over 8 heads of 64, 137 us, one by one 143; 333 rows over 4 heads 35 us, 29).
    const int run = (long)a.Tk * a.Hk >= 4 * 4096 ? 4 : 1;
    auto groups = [](long values) { return (int)((values + 1023) / 1024); };
    const int ndq = plan.kp > 1 ? groups((long)a.Tq * a.Hk * a.G * D) : 0, ndkv = groups((long)((a.Tk + run - 1) / run) * a.Hk * 2 * D);
    if (ndq + ndkv > 0) hipLaunchKernelGGL((attn_bwd_sum_kernel<T, D>), dim3(ndq + ndkv), dim3(256), 0, st, a, plan, ndq, run);
    return hipGetLastError();
}

hipError_t attn_bwd_launch(bool bf16, int D, const AttnArgs &a, hipStream_t st)
{
    if (bf16) return D == 128 ? bwd_launch<__bf16, 128>(a, st) : bwd_launch<__bf16, 64>(a, st);
    return D == 128 ? bwd_launch<float, 128>(a, st) : bwd_launch<float, 64>(a, st);
}

unsigned long long attn_bwd_workspace(bool bf16, int B, int Tq, int Tk, int Hk, int G, int D)
{
    return (unsigned long long)AttnBwdWs(attn_bwd_plan(bf16, B, Tq, Tk, Hk, G), B, Tq, Tk, Hk, G, D, attn_own(bf16)).bytes;
}

} // namespace gdn
