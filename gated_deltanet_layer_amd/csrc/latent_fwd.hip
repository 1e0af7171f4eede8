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

// Workspace of a call that is cut.  Pieces: float o[pieces][B Tq H][DV], float
// lse[pieces][B Tq H] (base 2).  Shares: int prefix[B + 1], the key tiles before each
// sequence, then for each share its first and last piece of a row tile, float o[slot][DV],
// and float lse[slot] of each, slot = min(RT, Tq) rows.
struct FwdWs {
    long o, lse, bytes, rows;
    __host__ __device__ FwdWs(const FwdPlan &p, int B, int Tq, int H, int dv) {
        const int rt = 64 * p.nr;
        rows = p.shares ? (Tq < rt ? Tq : rt) : (long)B * Tq * H;
        o = p.shares ? ((long)(B + 1) * 4 + 255) & ~255L : 0;
        const long all = rows * (p.shares ? 2 * p.shares : p.pieces);
        lse = o + all * dv * 4;
        bytes = lse + all * 4;
    }
};

// The key tiles of a causal call.  Row tile t of a sequence of n keys has those up to its
// last row's position: ceil(off / KT) + (t + 1) RT / KT of them, the last live one up to n.
template <int RT, int KT> struct FwdTiles {
    static __device__ __forceinline__ int of(const LatentFwdArgs &a, int n, int t) {
        const int off = a.Tk - a.Tq, end = off + min((t + 1) * RT, a.Tq);
        return t * RT < a.Tq && off + t * RT < n ? (min(n, end) + KT - 1) / KT : 0;
    }
    static __device__ __forceinline__ int before(const LatentFwdArgs &a, int t) {   // row tile t, a live one
        return t * ((a.Tk - a.Tq + KT - 1) / KT) + (RT / KT) * (t * (t + 1) / 2);
    }
    static __device__ __forceinline__ int all(const LatentFwdArgs &a, int n) {   // of one head
        const int off = a.Tk - a.Tq;
        if (n <= off) return 0;
        const int t = (n - off - 1) / RT;
        return before(a, t) + of(a, n, t);
    }
};

// Key tile j of the nkt of row tile t, head h of sequence b, which has n keys.
struct FwdPos {
    int b, h, t, j, nkt, n;
};

// The tile after p; called only while one is left.
template <int RT, int KT> __device__ __forceinline__ FwdPos fwd_after(const LatentFwdArgs &a, FwdPos p)
{
    if (++p.j < p.nkt) return p;
    p.j = 0;
    p.nkt = FwdTiles<RT, KT>::of(a, p.n, ++p.t);
    if (p.nkt == 0) {
        p.t = 0;
        if (++p.h == a.H) {
            p.h = 0;
            do p.n = live_len(a.lens, ++p.b, a.Tk);
            while (p.n <= a.Tk - a.Tq && p.b + 1 < a.B);
        }
        p.nkt = FwdTiles<RT, KT>::of(a, p.n, 0);
    }
    return p;
}

// Sums of a value of each lane over the lanes up to it.
__device__ __forceinline__ int lanes_scan(int x)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(x, d, 64);
        if ((int)(threadIdx.x & 63) >= d) x += v;
    }
    return x;
}

// Tiles of a share: all of the call's over the shares, rounded up.
__device__ __forceinline__ int fwd_each(int total) { return max(1, (total + FWD_SHARES - 1) / FWD_SHARES); }

// This workgroup's share, its first key tile and the number of them; 0 if it has none.
// Every wave adds up all sequences on its own; the first share leaves the tiles before
// each for the join.
template <int RT, int KT> __device__ __forceinline__ int fwd_share(const LatentFwdArgs &a, int share, FwdPos &cur)
{
    typedef FwdTiles<RT, KT> Tiles;
    const int lane = threadIdx.x & 63;
    int *prefix = (int *)a.ws;
    auto of = [&](int b) { return b < a.B ? a.H * Tiles::all(a, live_len(a.lens, b, a.Tk)) : 0; };
    int total = 0;
    for (int b = 0; b < a.B; b += 64) {
        const int mine = of(b + lane), incl = lanes_scan(mine);
        if (share == 0 && b + lane < a.B) prefix[b + lane] = total + incl - mine;
        total += __builtin_amdgcn_readlane(incl, 63);
    }
    if (share == 0 && lane == 0) prefix[a.B] = total;
    const int each = fwd_each(total), g0 = share * each;
    if (g0 >= total) return 0;
    int at = cur.b = 0;
    for (int b = 0; b < a.B; b += 64) {
        const int mine = of(b + lane), incl = lanes_scan(mine), sum = __builtin_amdgcn_readlane(incl, 63);
        if (g0 < at + sum) {
            const int l = __builtin_ctzll(__ballot(g0 < at + incl));
            cur.b = b + l;
            at += __builtin_amdgcn_readlane(incl - mine, l);
            break;
        }
        at += sum;
    }
    cur.n = __builtin_amdgcn_readfirstlane(live_len(a.lens, cur.b, a.Tk));
    const unsigned one = Tiles::all(a, cur.n), r = g0 - at;
    cur.h = (int)(r / one);
    const int x = (int)(r % one);
    // the row tile: before(t) <= x < before(t + 1)
    const float c = (a.Tk - a.Tq + KT - 1) / KT + .5f * (RT / KT);
    int t = max(0, (int)((sqrtf(c * c + 2.f * (RT / KT) * (float)x) - c) / (RT / KT)) - 1);
    while (t * RT + RT < a.Tq && Tiles::before(a, t + 1) <= x) ++t;
    while (t > 0 && Tiles::before(a, t) > x) --t;
    cur.t = __builtin_amdgcn_readfirstlane(t);
    cur.j = __builtin_amdgcn_readfirstlane(x - Tiles::before(a, t));
    cur.nkt = Tiles::of(a, cur.n, cur.t);
    return min(each, total - g0);
}

enum { WHOLE, PIECES, SHARES };   // how a call is cut

template <typename T, int DN, int DV, int NR, int CUT>
__global__ __launch_bounds__(256, 2) void latent_fwd_kernel(LatentFwdArgs a, int ntiles, FwdPlan plan)
{
    typedef FwdCfg<T, DN, DV, NR> C;
    constexpr int KT = C::KT, RT = C::RT, DK = C::DK, NKB = DK / 32, NS = KT / 16, NCB = DV / 16;
    extern __shared__ char lds[];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r16 = lane_r16(), gq = lane_gq();
    const int off = a.Tk - a.Tq;
    const long qs = (long)a.H * DK, kvs = (long)a.H * (DN + DV), os = (long)a.H * DV;
    const float c = a.scale * LOG2E;
    const FwdWs lay(plan, a.B, a.Tq, a.H, DV);
    FwdPos cur, nxt;
    int share = 0, left;   // key tiles to go
    if constexpr (CUT == SHARES) {
        // the shares of one head, which read the same keys, on one XCD
        share = blockIdx.x % 8 * (FWD_SHARES / 8) + blockIdx.x / 8;
        left = fwd_share<RT, KT>(a, share, cur);
        if (left == 0) return;
    } else {
        const int BH = a.B * a.H, bh = blockIdx.x % BH, piece = CUT == PIECES ? blockIdx.x / BH % plan.pieces : 0;
        cur.b = bh / a.H;
        cur.h = bh % a.H;
        cur.t = ntiles - 1 - (int)(blockIdx.x / BH / (CUT == PIECES ? plan.pieces : 1));   // longest rows first
        cur.n = live_len(a.lens, cur.b, a.Tk);
        cur.nkt = FwdTiles<RT, KT>::of(a, cur.n, cur.t);
        cur.j = piece * plan.each;
        left = min(plan.each, cur.nkt - cur.j);
        if (CUT == PIECES && left <= 0) return;   // the join knows which pieces there are
    }
    auto load = [&](const FwdPos &p, int buffer) {
        char *buf = lds + buffer * C::BUF;
        const T *kv = (const T *)a.kv + ((long)p.b * a.Tk * a.H + p.h) * (DN + DV);
        const T *kr = (const T *)a.k_rope + (long)p.b * a.Tk * LATENT_ROPE;
        load_rows<C::NCPR, KT>(buf, (const char *)kv, kvs * C::ES, p.j * KT, p.n);
        load_rows<C::RCPR, KT>(buf + C::OFF_R, (const char *)kr, LATENT_ROPE * C::ES, p.j * KT, p.n);
        load_rows<C::VCPR, KT>(buf + C::OFF_V, (const char *)(kv + DN), kvs * C::ES, p.j * KT, p.n);
    };
    const int nb = row_base<T, C::NCPR>(r16), rb = row_base<T, C::RCPR>(r16), vb = col_base<T, C::VCPR>(4 * gq);
    if (left > 0) load(cur, 0);
    int buffer = 0;
    for (;;) {   // one row tile, or what the share has of it
        const int n = cur.n, w0 = cur.t * RT + wave * 16 * NR;   // first row of the wave
        const int j0 = cur.j;
        const T *q = (const T *)a.q + ((long)cur.b * a.Tq * a.H + cur.h) * DK;
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

        const int wlast = min(n, off + min(w0 + 16 * NR, a.Tq)), wfull = off + w0 + 1;   // keys that some, that all of its rows see
        bool more = left > 0;   // false: a row tile of padding
        while (more) {
            const char *kt = lds + buffer * C::BUF, *vt = kt + C::OFF_V;
            const int k0 = cur.j * KT;
            wait_vm<0>();
            lds_barrier();
            buffer ^= 1;
            if (--left > 0) {
                if constexpr (CUT == SHARES) {
                    nxt = fwd_after<RT, KT>(a, cur);
                } else {
                    nxt = cur;
                    ++nxt.j;
                }
                load(nxt, buffer);
            }
            more = left > 0 && (CUT != SHARES || cur.j + 1 < cur.nkt);
            if (more) cur.j = nxt.j;
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
        const bool whole = !CUT || (j0 == 0 && cur.j + 1 >= cur.nkt);
        T *o = (T *)a.o + ((long)cur.b * a.Tq * a.H + cur.h) * DV;
        // where a part of the row tile goes: its number, its first row there, the step from row to row
        const long part = CUT == SHARES ? share * 2 + (j0 == 0) : j0 / plan.each, step = CUT == SHARES ? 1 : a.H;
        const long r0 = part * lay.rows + (CUT == SHARES ? 0 : ((long)cur.b * a.Tq + cur.t * RT) * a.H + cur.h);
        float *po = (float *)((char *)a.ws + lay.o) + r0 * DV, *pl = (float *)((char *)a.ws + lay.lse) + r0;
#pragma unroll
        for (int g = 0; g < NR; ++g) {
            const int row = w0 + 16 * g + r16, lr = row - cur.t * RT;
            const float ls = rows_sum(l[g]);
            // of part of the keys a row may see none: its sum is 0 (and a NaN where scores are)
            const bool seen = pos[g] >= 0 && (!CUT || ls != 0.f);
            const float inv = seen ? 1.f / ls : 0.f, lg = seen ? m[g] * c + __builtin_amdgcn_logf(ls) : -INFINITY;
            if (row >= a.Tq) continue;
            if (whole) {
#pragma unroll
                for (int cb = 0; cb < NCB; ++cb)
                    store4(o + row * os + 16 * cb + 4 * gq, seen ? acc[cb][g] * inv : f32x4{0.f, 0.f, 0.f, 0.f});
                if (gq == 0 && a.lse) a.lse[((long)cur.b * a.Tq + row) * a.H + cur.h] = lg * LN2;
            } else {
                if (seen) {
#pragma unroll
                    for (int cb = 0; cb < NCB; ++cb) store4(po + lr * step * DV + 16 * cb + 4 * gq, acc[cb][g] * inv);
                }
                if (gq == 0) pl[lr * step] = lg;
            }
        }
        if (CUT != SHARES || left == 0) break;
        cur = nxt;
    }
}

// Joins the rows that several workgroups worked on and writes those of row tiles without a
// key; DV / 4 lanes a row.
template <typename T, int DN, int DV, int NR, int CUT>
__global__ __launch_bounds__(256) void latent_fwd_join_kernel(LatentFwdArgs a, FwdPlan plan)
{
    typedef FwdCfg<T, DN, DV, NR> C;
    typedef FwdTiles<C::RT, C::KT> Tiles;
    constexpr int LPR = DV / 4;
    const unsigned of = a.Tq * a.H, r = blockIdx.x * (256 / LPR) + threadIdx.x / LPR;   // the rows of sequence b
    const int at = threadIdx.x % LPR * 4, b = blockIdx.y;
    if (r >= of) return;
    const int i = (int)(r / a.H), h = (int)(r - i * a.H), t = i / C::RT, lr = i % C::RT;
    const long row = (long)b * of + r;
    const int n = live_len(a.lens, b, a.Tk), k = Tiles::of(a, n, t);
    int wf = 0, wl = -1;   // shares, or pieces of the row tile
    if (CUT == PIECES) {
        wl = (k + plan.each - 1) / plan.each - 1;
    } else if (k > 0) {
        const int *prefix = (const int *)a.ws;
        const int c0 = prefix[b] + h * Tiles::all(a, n) + Tiles::before(a, t), each = fwd_each(prefix[a.B]);
        const float inv = 1.f / (float)each;
        auto share = [&](int c) {   // c / each, below FWD_SHARES: the product is off by less than 1
            const int q = (int)((float)c * inv), left = c - q * each;
            return q + (left >= each) - (left < 0);
        };
        wf = share(c0);
        wl = share(c0 + k - 1);
    }
    if (wf == wl) return;   // written by its one workgroup
    const FwdWs lay(plan, a.B, a.Tq, a.H, DV);
    const float *po = (const float *)((const char *)a.ws + lay.o), *pl = (const float *)((const char *)a.ws + lay.lse);
    auto place = [&](int w) {   // of share wf its last part, of the others the first
        return CUT == SHARES ? (w * 2 + (w == wf)) * lay.rows + lr : w * lay.rows + row;
    };
    float top = -INFINITY, ls = 0.f;
    for (int w = wf; w <= wl; ++w) top = fmaxf(top, pl[place(w)]);
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
    for (int w = wf; w <= wl; ++w) {
        const float lg = pl[place(w)];
        const f32x4 v = *reinterpret_cast<const f32x4 *>(po + place(w) * DV + at);
        const float f = exp2_hw(lg - top);
        if (lg == -INFINITY) continue;   // v was never written
        ls += f;
        sum += f * v;
    }
    store4((T *)a.o + row * DV + at, ls != 0.f ? sum * (1.f / ls) : sum);
    if (a.lse && at == 0) a.lse[row] = ls != 0.f ? (top + __builtin_amdgcn_logf(ls)) * LN2 : -INFINITY;
}

template <typename T, int DN, int DV, int NR, int CUT>
static hipError_t fwd_enqueue(const LatentFwdArgs &a, const FwdPlan &plan, hipStream_t st)
{
    typedef FwdCfg<T, DN, DV, NR> C;
    const int ntiles = (a.Tq + C::RT - 1) / C::RT;
    auto k = latent_fwd_kernel<T, DN, DV, NR, CUT>;
    const hipError_t e = hipFuncSetAttribute((const void *)k, hipFuncAttributeMaxDynamicSharedMemorySize, 2 * C::BUF);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k, dim3((unsigned)(plan.shares ? plan.shares : (long)ntiles * a.B * a.H * plan.pieces)), dim3(256), 2 * C::BUF, st, a, ntiles, plan);
    if constexpr (CUT != WHOLE) {
        const long rows = (long)a.Tq * a.H, per = 256 / (DV / 4);
        hipLaunchKernelGGL((latent_fwd_join_kernel<T, DN, DV, NR, CUT>), dim3((unsigned)((rows + per - 1) / per), a.B), dim3(256), 0, st, a, plan);
    }
    return hipGetLastError();
}

template <typename T, int DN, int DV, int NR> static hipError_t fwd_cut(const LatentFwdArgs &a, const FwdPlan &plan, hipStream_t st)
{
    if (plan.shares > 0) return fwd_enqueue<T, DN, DV, NR, SHARES>(a, plan, st);
    return plan.pieces > 1 ? fwd_enqueue<T, DN, DV, NR, PIECES>(a, plan, st) : fwd_enqueue<T, DN, DV, NR, WHOLE>(a, plan, st);
}

template <typename T, int DN, int DV> static hipError_t fwd_launch(const LatentFwdArgs &a, hipStream_t st)
{
    constexpr bool BF = sizeof(T) == 2;
    const FwdPlan plan = fwd_plan(BF, a.B, a.Tq, a.Tk, a.H);
    if constexpr (BF) {
        if (plan.nr == 2) return fwd_cut<T, DN, DV, 2>(a, plan, st);
    }
    return fwd_cut<T, DN, DV, 1>(a, plan, st);
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
    return plan.shares > 0 || plan.pieces > 1 ? (unsigned long long)FwdWs(plan, B, Tq, H, dv).bytes : 0;
}

} // namespace gdn
