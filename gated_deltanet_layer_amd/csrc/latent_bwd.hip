// latent_bwd.hip -- gradients of the expanded latent attention (gfx950).
//
//   P_ij = exp(s_ij - lse_i),  D_i = do_i . o_i,  dS_ij = scale P_ij (do_i . v_j - D_i)
//   dv_j = sum_i P_ij do_i,  dk_j = sum_i dS_ij q_i,  dq_i = sum_j dS_ij k_j
//   dk_rope_j = sum over heads of the rotary part of dk_j
//
// No atomics, so results do not depend on the order in which workgroups run:
// one kernel owns key rows and walks the query rows that see them (dk, dv), one
// owns query rows and walks their keys (dq); the scores are computed in both.
// The rotary part of dk is written per head in fp32 and added over the heads in
// order by a last kernel, with the pieces of what was cut.
//
// Bound by the matrix cores, with seven products where atomics would do with five: 8192
// rows of 16 heads, bf16, dn = dv = 128 in 1155-1270 us (dq 480-520, dk and dv 640-700),
// 1.0 PFLOP/s over the seven, about a library product's rate on the same card (1.11;
// matrix cores 51 and 42 % busy).  Padded batches of some 1500 rows (4 x 16 heads, 70 +
// 100 us) are bound by each workgroup's own chain (loads of its operands, blocks one
// after the other, its stores), which at one workgroup a unit nothing hides.
#include "latent.h"

namespace gdn {

// Workspace, all float: D[B][Tq][H]; dk_rope[qp][B][Tk][H][64]; where there are pieces,
// dq[kp][B][Tq][H][DK] and dkv[qp][B][Tk][H][DN + DV].
struct BwdWs {
    long rope, dq, dkv, bytes;
    __host__ __device__ BwdWs(const BwdPlan &p, int B, int Tq, int Tk, int H, int dn, int dv) {
        const long qr = (long)B * Tq * H, kr = (long)B * Tk * H;
        rope = (qr * 4 + 255) & ~255L;
        dq = rope + p.qp * kr * LATENT_ROPE * 4;
        dkv = dq + (p.kp > 1 ? p.kp * qr * (dn + LATENT_ROPE) * 4 : 0);
        bytes = dkv + (p.qp > 1 ? p.qp * kr * (dn + dv) * 4 : 0);
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
// room, which lets the waves meet once a tile of 64 rows instead of 32: 4 x 16 heads of
// 1531, 64 / 128, 156 us from 168; at 128 / 128 the same).  P <= 1, so nothing overflows,
// and down to P = 2^-26 it is off by 2^-11 of itself, an eighth of what dS, which it
// becomes, is rounded by; below, by 2^-37.  The power of two comes out of dk at the end.
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
template <typename T> __device__ __forceinline__ constexpr float hand_scale() { return sizeof(T) == 2 ? 1.f / 4096.f : 1.f; }
template <typename T> __device__ __forceinline__ void hand_over(char *to, f32x4 p) {
    if constexpr (sizeof(T) == 2) {
        f16x4 h;
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = (_Float16)(p[e] * 4096.f);
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

template <typename T, int DN, int DV> struct BwdCfg {
    static constexpr int NG = sizeof(T) == 2 ? 2 : 1;      // 16-row groups a wave owns
    static constexpr int OWN = 64 * NG;                    // rows a workgroup owns (keys or queries)
    static constexpr int ST = sizeof(T) == 2 ? 64 : 32;    // rows a tile that walks by
    static constexpr int DK = DN + LATENT_ROPE;
    static constexpr int ES = (int)sizeof(T), NCPR = DN * ES / 16, RCPR = LATENT_ROPE * ES / 16, VCPR = DV * ES / 16;
    // a tile: [ST][DN] and [ST][64] of the rows' two key parts, [ST][DV]
    static constexpr int OFF_R = ST * NCPR * 16, OFF_V = OFF_R + ST * RCPR * 16, BUF = OFF_V + ST * VCPR * 16;
    static constexpr int ROWS = 2 * ST * 4;                // lse and D of the tile's rows
    static constexpr int HP = 64 * 4 * (ES == 2 ? 2 : 4);  // four values of P of each lane
    static constexpr int HAND = 2 * ST / 16 * NG * HP;     // P of two tiles, one pair of waves
    static constexpr int KV_LDS = 3 * (BUF + ROWS) + 4 * HAND;
    static_assert(KV_LDS <= 160 * 1024, "LDS");
};

// dk and dv.  Four pairs of waves; a pair owns 16 NG keys.  The first of the pair
// computes the scores and P and adds up dv^T (k and dv in its registers), the second
// takes P over, computes dP and dS and adds up dk^T (v and dk in its registers): the
// same number of products for both, and of q and do each reads from LDS one along
// the rows and the other across them, where one wave for both would not have the
// registers for 32 keys, and with 16 keys would read twice as much.  The second is
// one tile of query rows behind, so neither waits for the other inside a tile.
// Scores have query rows on the accumulator's rows: P and dS feed the gradient
// products as B operands straight from the registers, and P changes hands between
// equal lanes.
template <typename T, int DN, int DV, bool CUT>
__global__ __launch_bounds__(512, 1) void latent_bwd_kv_kernel(LatentBwdArgs a, BwdPlan plan)
{
    typedef BwdCfg<T, DN, DV> C;
    constexpr int NG = C::NG, ST = C::ST, DK = C::DK, NKB = DK / 32, NVB = DV / 32, NKC = DK / 16, NVC = DV / 16;
    constexpr int BPT = ST / 32;   // blocks a tile
    extern __shared__ char lds[];
    const int BH = a.B * a.H;
    const int bh = blockIdx.x % BH, piece = CUT ? blockIdx.x / BH % plan.qp : 0;
    const int tile = blockIdx.x / BH / (CUT ? plan.qp : 1);   // the first keys are seen by most rows
    const int b = bh / a.H, h = bh % a.H;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r16 = lane_r16(), gq = lane_gq();
    const int pair = wave & 3, lane = threadIdx.x & 63;
    const int off = a.Tk - a.Tq, n = live_len(a.lens, b, a.Tk);
    const int k0 = tile * C::OWN, w0 = k0 + pair * 16 * NG;
    const long qs = (long)a.H * DK, kvs = (long)a.H * (DN + DV), os = (long)a.H * DV;
    const T *q = (const T *)a.q + ((long)b * a.Tq * a.H + h) * DK;
    const T *d_o = (const T *)a.d_o + ((long)b * a.Tq * a.H + h) * DV;
    const T *kv = (const T *)a.kv + ((long)b * a.Tk * a.H + h) * (DN + DV);
    const T *kr = (const T *)a.k_rope + (long)b * a.Tk * LATENT_ROPE;
    const float *lse = a.lse + (long)b * a.Tq * a.H + h, *Dw = (const float *)a.ws + (long)b * a.Tq * a.H + h;
    const float c = a.scale * LOG2E;
    float *stat = (float *)(lds + 3 * C::BUF);                  // [3][2][ST]: lse and D of the rows
    char *hand = lds + 3 * (C::BUF + C::ROWS) + pair * C::HAND; // [2][ST / 16 NG][64 lanes]: P of a tile, four values a lane

    // query rows that are no padding and see the workgroup's first key (of the piece)
    const int qn = min(min(a.Tq, n - off), CUT ? (piece + 1) * plan.qstep : a.Tq);
    const int qfirst = max(CUT ? piece * plan.qstep : 0, max(0, k0 - off) / ST * ST);
    const int nt = k0 < n && qfirst < qn ? (qn - qfirst + ST - 1) / ST : 0;
    auto load = [&](int j) {
        const int r0 = qfirst + j * ST, buf = __builtin_amdgcn_readfirstlane(j % 3);
        char *to = lds + buf * C::BUF;
        load_rows<C::NCPR, ST, 512>(to, (const char *)q, qs * C::ES, r0, qn);
        load_rows<C::RCPR, ST, 512>(to + C::OFF_R, (const char *)(q + DN), qs * C::ES, r0, qn);
        load_rows<C::VCPR, ST, 512>(to + C::OFF_V, (const char *)d_o, os * C::ES, r0, qn);
        if (wave < 2 && lane < ST) {   // lse by the first wave, D by the second
            const int r = r0 + lane;
            const void *src = r >= qn ? (const void *)latent_zero : (wave ? Dw : lse) + (long)r * a.H;
            copy4(src, (char *)(stat + (buf * 2 + wave) * ST));
        }
    };
    // before tile j: it is there, and P of tile j - 1 is whole
    auto sync = [&](int j) {
        if (j < nt) wait_vm<0>();
        lds_barrier();
        if (j + 1 < nt) load(j + 1);   // over tile j - 2
    };
    auto seen = [&](int i) {   // whether a row of block i sees a key of the wave
        return off + qfirst + i * 32 + 31 >= w0 && w0 < n;
    };
    const BwdWs lay(plan, a.B, a.Tq, a.Tk, a.H, DN, DV);
    if (CUT && nt == 0) return;   // the last kernel knows which pieces there are
    if (nt > 0) load(0);

    if (wave < 4) {
        const int nb = row_base<T, C::NCPR>(r16), rb = row_base<T, C::RCPR>(r16), vc = col_base<T, C::VCPR>(4 * gq);
        Frag<T> kf[NG][NKB];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const int key = w0 + 16 * g + r16;
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb) {
                const int col = 32 * kb + 8 * gq;
                const T *p = 32 * kb < DN ? kv + key * kvs + col : kr + (long)key * LATENT_ROPE + (col - DN);
                kf[g][kb] = key < n ? load_frag<T>(p) : zero_frag<T>();
            }
        }
        f32x4 dv[NVC][NG];
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int i = 0; i < NVC; ++i) dv[i][g] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int j = 0; j <= nt; ++j) {
            sync(j);
            if (j == nt) break;
            const char *qt = lds + j % 3 * C::BUF, *dt = qt + C::OFF_V;
            const float *st = stat + j % 3 * 2 * ST;
            char *to = hand + (j & 1) * (C::HAND / 2) + lane * (C::HP / 64);
#pragma unroll 1
            for (int t = 0; t < BPT; ++t) {
                if (!seen(j * BPT + t)) continue;
                const int r0 = qfirst + j * ST + t * 32;
                const bool part = off + r0 < w0 + 16 * NG - 1 || r0 + 32 > qn;
                f32x4 s[2][NG];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
#pragma unroll
                    for (int g = 0; g < NG; ++g) s[u][g] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int kb = 0; kb < NKB; ++kb) {
                        const Frag<T> f = kb < DN / 32
                            ? row_frag<T>(qt + (32 * t + 16 * u) * C::NCPR * 16, nb, kb)
                            : row_frag<T>(qt + C::OFF_R + (32 * t + 16 * u) * C::RCPR * 16, rb, kb - DN / 32);
#pragma unroll
                        for (int g = 0; g < NG; ++g) s[u][g] = mma(s[u][g], f, kf[g][kb]);
                    }
                    const int row = 16 * u + 4 * gq;
                    const f32x4 ls = *reinterpret_cast<const f32x4 *>(st + 32 * t + row) * LOG2E;
#pragma unroll
                    for (int g = 0; g < NG; ++g)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[u][g][e] = exp2_hw(__builtin_fmaf(s[u][g][e], c, -ls[e]));
                    if (part) {
#pragma unroll
                        for (int g = 0; g < NG; ++g)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const bool hide = (off + r0 + row + e < w0 + 16 * g + r16) | (r0 + row + e >= qn);
                                s[u][g][e] = hide ? 0.f : s[u][g][e];
                            }
                    }
#pragma unroll
                    for (int g = 0; g < NG; ++g) hand_over<T>(to + ((2 * t + u) * NG + g) * C::HP, s[u][g]);
                }
                // P (and below dS) rounded to the storage type for the matrix cores: half
                // a step each, as the gradients themselves
                Frag<T> pf[NG];
#pragma unroll
                for (int g = 0; g < NG; ++g) pf[g] = reg_frag<T>(s[0][g], s[1][g]);
#pragma unroll
                for (int v = 0; v < NVC; ++v) {
                    const Frag<T> f = col_frag<T, C::VCPR>(dt + 32 * t * C::VCPR * 16, vc, v);
#pragma unroll
                    for (int g = 0; g < NG; ++g) dv[v][g] = mma(dv[v][g], f, pf[g]);
                }
            }
        }
        T *dkv = (T *)a.dkv + ((long)b * a.Tk * a.H + h) * (DN + DV) + DN;
        float *part = (float *)((char *)a.ws + lay.dkv) + ((piece * (long)a.B + b) * a.Tk * a.H + h) * (DN + DV) + DN;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const int key = w0 + 16 * g + r16;
            if (key >= a.Tk) continue;
#pragma unroll
            for (int v = 0; v < NVC; ++v) {
                if (CUT) store4(part + key * kvs + 16 * v + 4 * gq, dv[v][g]);
                else store4(dkv + key * kvs + 16 * v + 4 * gq, dv[v][g]);
            }
        }
    } else {
        const int vb = row_base<T, C::VCPR>(r16), nc = col_base<T, C::NCPR>(4 * gq), rc = col_base<T, C::RCPR>(4 * gq);
        Frag<T> vf[NG][NVB];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const int key = w0 + 16 * g + r16;
#pragma unroll
            for (int v = 0; v < NVB; ++v)
                vf[g][v] = key < n ? load_frag<T>(kv + key * kvs + DN + 32 * v + 8 * gq) : zero_frag<T>();
        }
        f32x4 dk[NKC][NG];
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int i = 0; i < NKC; ++i) dk[i][g] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int j = 0; j <= nt; ++j) {
            sync(j);
            if (j == 0) continue;
            const int k = j - 1;
            const char *qt = lds + k % 3 * C::BUF, *dt = qt + C::OFF_V;
            const float *st = stat + (k % 3 * 2 + 1) * ST;
            const char *from = hand + (k & 1) * (C::HAND / 2) + lane * (C::HP / 64);
#pragma unroll 1
            for (int t = 0; t < BPT; ++t) {
                if (!seen(k * BPT + t)) continue;
                f32x4 dp[2][NG];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
#pragma unroll
                    for (int g = 0; g < NG; ++g) dp[u][g] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int v = 0; v < NVB; ++v) {
                        const Frag<T> f = row_frag<T>(dt + (32 * t + 16 * u) * C::VCPR * 16, vb, v);
#pragma unroll
                        for (int g = 0; g < NG; ++g) dp[u][g] = mma(dp[u][g], f, vf[g][v]);
                    }
                    const f32x4 dd = *reinterpret_cast<const f32x4 *>(st + 32 * t + 16 * u + 4 * gq);
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        const f32x4 p = take_over<T>(from + ((2 * t + u) * NG + g) * C::HP);
#pragma unroll
                        for (int e = 0; e < 4; ++e) dp[u][g][e] = p[e] * (dp[u][g][e] - dd[e]);
                    }
                }
                Frag<T> sf[NG];
#pragma unroll
                for (int g = 0; g < NG; ++g) sf[g] = reg_frag<T>(dp[0][g], dp[1][g]);
#pragma unroll
                for (int v = 0; v < NKC; ++v) {
                    const Frag<T> f = v < DN / 16 ? col_frag<T, C::NCPR>(qt + 32 * t * C::NCPR * 16, nc, v)
                                                  : col_frag<T, C::RCPR>(qt + C::OFF_R + 32 * t * C::RCPR * 16, rc, v - DN / 16);
#pragma unroll
                    for (int g = 0; g < NG; ++g) dk[v][g] = mma(dk[v][g], f, sf[g]);
                }
            }
        }
        T *dkv = (T *)a.dkv + ((long)b * a.Tk * a.H + h) * (DN + DV);
        float *rope = (float *)((char *)a.ws + lay.rope);
        float *part = (float *)((char *)a.ws + lay.dkv) + ((piece * (long)a.B + b) * a.Tk * a.H + h) * (DN + DV);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const int key = w0 + 16 * g + r16;
            if (key >= a.Tk) continue;
#pragma unroll
            for (int i = 0; i < NKC; ++i) {
                const f32x4 v = dk[i][g] * (a.scale * hand_scale<T>());
                if (16 * i >= DN)
                    store4(rope + (((piece * (long)a.B + b) * a.Tk + key) * a.H + h) * LATENT_ROPE + (16 * i - DN) + 4 * gq, v);
                else if (CUT) store4(part + key * kvs + 16 * i + 4 * gq, v);
                else store4(dkv + key * kvs + 16 * i + 4 * gq, v);
            }
        }
    }
}

// dq, and D for the kernel above, which is launched after this one.  A wave owns 16
// NG query rows, q and do of them in registers; scores are transposed as in the
// forward pass, and dS^T feeds dq^T = K^T dS^T from the registers.
template <typename T, int DN, int DV, bool CUT>
__global__ __launch_bounds__(256, 2) void latent_bwd_q_kernel(LatentBwdArgs a, int ntiles, BwdPlan plan)
{
    typedef BwdCfg<T, DN, DV> C;
    constexpr int NG = C::NG, ST = C::ST, DK = C::DK, NKB = DK / 32, NVB = DV / 32, NKC = DK / 16;
    constexpr bool BF = sizeof(T) == 2;
    extern __shared__ char lds[];
    const int BH = a.B * a.H;
    const int bh = blockIdx.x % BH, piece = CUT ? blockIdx.x / BH % plan.kp : 0;
    const int tile = ntiles - 1 - (int)(blockIdx.x / BH / (CUT ? plan.kp : 1));   // longest rows first
    const int b = bh / a.H, h = bh % a.H;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r16 = lane_r16(), gq = lane_gq();
    const int off = a.Tk - a.Tq, n = live_len(a.lens, b, a.Tk);
    const int q0 = tile * C::OWN, w0 = q0 + wave * 16 * NG;
    const long qs = (long)a.H * DK, kvs = (long)a.H * (DN + DV), os = (long)a.H * DV;
    const T *q = (const T *)a.q + ((long)b * a.Tq * a.H + h) * DK;
    const T *d_o = (const T *)a.d_o + ((long)b * a.Tq * a.H + h) * DV;
    const T *kv = (const T *)a.kv + ((long)b * a.Tk * a.H + h) * (DN + DV);
    const T *kr = (const T *)a.k_rope + (long)b * a.Tk * LATENT_ROPE;
    const T *o = (const T *)a.o + ((long)b * a.Tq * a.H + h) * DV;
    const float *lse = a.lse + (long)b * a.Tq * a.H + h;
    float *Dw = (float *)a.ws + (long)b * a.Tq * a.H + h;
    const float c = a.scale * LOG2E;

    int pos[NG];
    float ls[NG], dd[NG];
    Frag<T> qf[NG][NKB], of[NG][NVB];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        const int row = w0 + 16 * g + r16;
        const bool live = row < a.Tq && off + row < n;
        pos[g] = live ? off + row : -1;
        ls[g] = live ? lse[(long)row * a.H] * LOG2E : 0.f;
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb)
            qf[g][kb] = live ? load_frag<T>(q + row * qs + 32 * kb + 8 * gq) : zero_frag<T>();
#pragma unroll
        for (int v = 0; v < NVB; ++v)
            of[g][v] = live ? load_frag<T>(d_o + row * os + 32 * v + 8 * gq) : zero_frag<T>();
        float dot = 0.f;
#pragma unroll
        for (int v = 0; v < NVB; ++v)
            if (live) dot += frag_dot<T>(of[g][v], load_frag<T>(o + row * os + 32 * v + 8 * gq));
        dd[g] = rows_sum(dot);
    }
    f32x4 dq[NKC][NG];
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int i = 0; i < NKC; ++i) dq[i][g] = f32x4{0.f, 0.f, 0.f, 0.f};

    const int last = min(n, off + min(q0 + C::OWN, a.Tq));
    const int all = (off + q0 < n) ? (last + ST - 1) / ST : 0;
    const int j0 = CUT ? piece * plan.kstep / ST : 0, nt = CUT ? min(all, j0 + plan.kstep / ST) : all;
    if (CUT && piece > 0 && nt <= j0) return;   // the last kernel knows which pieces there are
    const int wlast = min(n, off + min(w0 + 16 * NG, a.Tq)), wfull = off + w0 + 1;
    auto load = [&](int j) {
        char *to = lds + (j & 1) * C::BUF;
        load_rows<C::NCPR, ST>(to, (const char *)kv, kvs * C::ES, j * ST, n);
        load_rows<C::RCPR, ST>(to + C::OFF_R, (const char *)kr, LATENT_ROPE * C::ES, j * ST, n);
        load_rows<C::VCPR, ST>(to + C::OFF_V, (const char *)(kv + DN), kvs * C::ES, j * ST, n);
    };
    const int nb = row_base<T, C::NCPR>(r16), rb = row_base<T, C::RCPR>(r16), vb = row_base<T, C::VCPR>(r16);
    const int nc = col_base<T, C::NCPR>(4 * gq), rc = col_base<T, C::RCPR>(4 * gq);
    // of 32 keys (block t of tile j): P, and dP in the same layout
    auto products = [&](int j, int t, f32x4 (&s)[2][NG], f32x4 (&dp)[2][NG]) {
        const char *kt = lds + (j & 1) * C::BUF, *vt = kt + C::OFF_V;
        const int k0 = j * ST;
        const bool part = k0 + ST > wfull || k0 + ST > n;
        const int nbl = pin(nb), rbl = pin(rb), vbl = pin(vb);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                s[u][g] = f32x4{0.f, 0.f, 0.f, 0.f};
                dp[u][g] = s[u][g];
            }
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb) {
                const Frag<T> f = kb < DN / 32
                    ? row_frag<T>(kt + (32 * t + 16 * u) * C::NCPR * 16, nbl, kb)
                    : row_frag<T>(kt + C::OFF_R + (32 * t + 16 * u) * C::RCPR * 16, rbl, kb - DN / 32);
#pragma unroll
                for (int g = 0; g < NG; ++g) s[u][g] = mma(s[u][g], f, qf[g][kb]);
            }
#pragma unroll
            for (int v = 0; v < NVB; ++v) {
                const Frag<T> f = row_frag<T>(vt + (32 * t + 16 * u) * C::VCPR * 16, vbl, v);
#pragma unroll
                for (int g = 0; g < NG; ++g) dp[u][g] = mma(dp[u][g], f, of[g][v]);
            }
            if (BF) pipeline<4, NKB + NVB, (NKB + NVB) * NG, 1, NG>();
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
    if (BF && all <= 2) {
        // The first rows, of few keys: o, rounded to bf16, is as large as v there, and
        // the error that its rounding leaves in D, the same for all keys of a row, would
        // be as large as the rounding of dS (a sixth more error in dq over 30 rows).  They
        // have D from P and dP themselves.  The others have do . o, where that error is
        // small as long as a row's weights are spread over its n keys (1 / sqrt(n) as
        // large), and is not where one key takes most of them: 600 rows of 4 heads, scores
        // of a standard deviation of 1, 4, 8 and 64, errors of dq relative to its norm
        // 2.3e-3, 3.2e-3, 4.4e-3 and 7.1e-3 (the formulas in fp32: 1.7e-3; here it
        // would take one more pass over the keys).
        float sum[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) sum[g] = 0.f;
        for (int j = 0; j < all; ++j) {
            if (j == 0) load(0);
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
        lds_barrier();
#pragma unroll
        for (int g = 0; g < NG; ++g) dd[g] = rows_sum(sum[g]);
    }
    if (piece == 0 && gq == 0) {
#pragma unroll
        for (int g = 0; g < NG; ++g)
            if (pos[g] >= 0) Dw[(long)(w0 + 16 * g + r16) * a.H] = dd[g];
    }
    if (nt > j0) load(j0);
    for (int j = j0; j < nt; ++j) {
        const char *kt = lds + (j & 1) * C::BUF;
        const int k0 = j * ST;
        wait_vm<0>();
        lds_barrier();
        if (j + 1 < nt) load(j + 1);
        if (k0 >= wlast || off + w0 >= n) continue;
#pragma unroll 1
        for (int t = 0; t < ST / 32; ++t) {
            f32x4 s[2][NG], dp[2][NG];
            products(j, t, s, dp);
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int g = 0; g < NG; ++g) dp[u][g] = s[u][g] * (dp[u][g] - dd[g]);
            const int ncl = pin(nc), rcl = pin(rc);
            Frag<T> sf[NG];
#pragma unroll
            for (int g = 0; g < NG; ++g) sf[g] = reg_frag<T>(dp[0][g], dp[1][g]);
#pragma unroll
            for (int i = 0; i < NKC; ++i) {
                const Frag<T> f = i < DN / 16 ? col_frag<T, C::NCPR>(kt + 32 * t * C::NCPR * 16, ncl, i)
                                              : col_frag<T, C::RCPR>(kt + C::OFF_R + 32 * t * C::RCPR * 16, rcl, i - DN / 16);
#pragma unroll
                for (int g = 0; g < NG; ++g) dq[i][g] = mma(dq[i][g], f, sf[g]);
            }
            if (BF) pipeline<4, 2 * NKC, NKC * NG, 2, NG>();
        }
    }
    T *dqp = (T *)a.dq + ((long)b * a.Tq * a.H + h) * DK;
    float *sum = (float *)((char *)a.ws + BwdWs(plan, a.B, a.Tq, a.Tk, a.H, DN, DV).dq) + ((piece * (long)a.B + b) * a.Tq * a.H + h) * DK;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        const int row = w0 + 16 * g + r16;
        if (row >= a.Tq) continue;
#pragma unroll
        for (int i = 0; i < NKC; ++i) {
            const f32x4 v = pos[g] >= 0 ? dq[i][g] * a.scale : f32x4{0.f, 0.f, 0.f, 0.f};
            if (CUT) store4(sum + row * qs + 16 * i + 4 * gq, v);
            else store4(dqp + row * qs + 16 * i + 4 * gq, v);
        }
    }
}

// dk_rope[b][t], the sum over pieces and heads, and where there are pieces the sums of
// dq and dkv over them; all in order.  The first nr workgroups take 16 rows of dk_rope
// each, the next ones 4 x 256 values of dq, the others of dkv.  A piece counts for the
// rows that its workgroup has worked on.
template <typename T, int DN, int DV>
__global__ __launch_bounds__(256) void latent_bwd_sum_kernel(LatentBwdArgs a, BwdPlan plan, int nr, int ndq)
{
    typedef BwdCfg<T, DN, DV> C;
    const BwdWs lay(plan, a.B, a.Tq, a.Tk, a.H, DN, DV);
    const int off = a.Tk - a.Tq;
    // pieces of the query rows that the owner of key t walks: [first, end)
    auto walked = [&](int b, int t, int &first, int &end) {
        const int n = live_len(a.lens, b, a.Tk), k0 = t / C::OWN * C::OWN, qn = min(a.Tq, n - off);
        const int q0 = max(0, k0 - off) / C::ST * C::ST;
        const bool any = k0 < n && q0 < qn;
        first = any ? q0 / plan.qstep : 0;
        end = any ? (qn - 1) / plan.qstep + 1 : 0;
    };
    if ((int)blockIdx.x < nr) {
        const long krows = (long)a.B * a.Tk, row = (long)blockIdx.x * 16 + threadIdx.x / 16;
        const int at = (threadIdx.x & 15) * 4;
        if (row >= krows) return;
        int first = 0, end = 1;
        if (plan.qp > 1) walked((int)(row / a.Tk), (int)(row % a.Tk), first, end);
        const float *part = (const float *)((const char *)a.ws + lay.rope);
        f32x4 s = {0.f, 0.f, 0.f, 0.f};
        for (int p = first; p < end; ++p)
#pragma unroll 4
            for (int h = 0; h < a.H; ++h)
                s += *reinterpret_cast<const f32x4 *>(part + ((p * krows + row) * a.H + h) * LATENT_ROPE + at);
        store4((T *)a.dk_rope + row * LATENT_ROPE + at, s);
        return;
    }
    const bool isq = (int)blockIdx.x < nr + ndq;
    const int W = isq ? C::DK : DN + DV, T_ = isq ? a.Tq : a.Tk;
    const long at = ((long)(blockIdx.x - nr - (isq ? 0 : ndq)) * 256 + threadIdx.x) * 4, size = (long)a.B * T_ * a.H * W;
    if (at >= size) return;
    const int b = (int)(at / W / a.H / T_), t = (int)(at / W / a.H % T_);
    int first = 0, end;
    if (isq) {   // the owner of row t walks the keys up to its last row's position
        const int n = live_len(a.lens, b, a.Tk), q0 = t / C::OWN * C::OWN;
        const int last = min(n, off + min(q0 + C::OWN, a.Tq));
        end = off + q0 < n ? (last - 1) / plan.kstep + 1 : 1;   // piece 0 always writes
    } else {
        walked(b, t, first, end);
    }
    const float *part = (const float *)((const char *)a.ws + (isq ? lay.dq : lay.dkv)) + at;
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
    for (int p = first; p < end; ++p) s += *reinterpret_cast<const f32x4 *>(part + p * size);
    store4((T *)(isq ? a.dq : a.dkv) + at, s);
}

static hipError_t allow_lds(const void *kernel, int bytes) {
    return hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <typename T, int DN, int DV>
static hipError_t bwd_launch(const LatentBwdArgs &a, hipStream_t st)
{
    typedef BwdCfg<T, DN, DV> C;
    const BwdPlan plan = bwd_plan(sizeof(T) == 2, a.B, a.Tq, a.Tk, a.H);
    const long BH = (long)a.B * a.H, krows = (long)a.B * a.Tk;
    const int nq = (a.Tq + C::OWN - 1) / C::OWN, nk = (a.Tk + C::OWN - 1) / C::OWN;
    auto kkv = plan.qp > 1 ? latent_bwd_kv_kernel<T, DN, DV, true> : latent_bwd_kv_kernel<T, DN, DV, false>;
    auto kq = plan.kp > 1 ? latent_bwd_q_kernel<T, DN, DV, true> : latent_bwd_q_kernel<T, DN, DV, false>;
    hipError_t e = allow_lds((const void *)kkv, C::KV_LDS);
    if (e == hipSuccess) e = allow_lds((const void *)kq, 2 * C::BUF);
    if (e != hipSuccess) return e;
    if (BH * nq > 0) hipLaunchKernelGGL(kq, dim3((unsigned)(BH * nq * plan.kp)), dim3(256), 2 * C::BUF, st, a, nq, plan);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (BH * nk > 0) hipLaunchKernelGGL(kkv, dim3((unsigned)(BH * nk * plan.qp)), dim3(512), C::KV_LDS, st, a, plan);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    auto groups = [](long values) { return (int)((values + 1023) / 1024); };
    const int nr = (int)((krows + 15) / 16), ndq = plan.kp > 1 ? groups(BH * a.Tq * C::DK) : 0;
    const int ndkv = plan.qp > 1 ? groups(BH * a.Tk * (DN + DV)) : 0;
    if (krows > 0)
        hipLaunchKernelGGL((latent_bwd_sum_kernel<T, DN, DV>), dim3(nr + ndq + ndkv), dim3(256), 0, st, a, plan, nr, ndq);
    return hipGetLastError();
}

hipError_t latent_bwd_launch(bool bf16, int dn, int dv, const LatentBwdArgs &a, hipStream_t st)
{
    if (bf16) {
        if (dn == 128) return dv == 128 ? bwd_launch<__bf16, 128, 128>(a, st) : bwd_launch<__bf16, 128, 64>(a, st);
        return dv == 128 ? bwd_launch<__bf16, 64, 128>(a, st) : bwd_launch<__bf16, 64, 64>(a, st);
    }
    if (dn == 128) return dv == 128 ? bwd_launch<float, 128, 128>(a, st) : bwd_launch<float, 128, 64>(a, st);
    return dv == 128 ? bwd_launch<float, 64, 128>(a, st) : bwd_launch<float, 64, 64>(a, st);
}

unsigned long long latent_bwd_workspace(bool bf16, int B, int Tq, int Tk, int H, int dn, int dv)
{
    return (unsigned long long)BwdWs(bwd_plan(bf16, B, Tq, Tk, H), B, Tq, Tk, H, dn, dv).bytes;
}

} // namespace gdn
