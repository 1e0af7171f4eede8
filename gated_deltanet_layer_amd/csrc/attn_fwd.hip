// attn_fwd.hip -- causal attention of grouped heads over packed sequences (gfx950).
//
//   s_ij = scale q_i . k_j,  j <= p_i = lk - lq + i        (within one sequence)
//   o_i = sum_j softmax_j(s_ij) v_j,   lse_i = log sum_j exp s_ij
//
// The G query heads that share a key head are rows of one tile (row r: token r / G, head
// r % G), so a tile of 64 or 128 rows covers few tokens: keys are read once for all heads,
// little of the diagonal's tiles is masked, and short sequences still fill a tile.
//
// A workgroup of four waves owns a row tile of one key head and walks the key tiles once,
// keeping the running maximum and sum of every row.  Scores are computed transposed (keys
// on the accumulator's rows, query rows on its lanes): a lane holds four consecutive keys of
// one row, the softmax needs two cross-lane steps a tile, and the weights feed the second
// product (o^T = V^T P^T) as its B operand straight from the registers.
//
// Long rows are bound by the matrix cores and the exponentials that stand between their
// products: 8192 packed tokens (one sequence of 4999 among seven) of 32 over 8 heads of 128, bf16,
// take 250 to 290 us (0.82 to 0.94 PFLOP/s of the visible half; a library product reaches 1.34),
// in which the matrix cores are busy for 43 % of the cycles.  Without its exponentials the
// kernel takes 0.93 of that, without its reads of keys 0.86, without its copies 0.89: no one of
// them bounds it alone.  Short rows are bound by latency, a key tile after the other, some 1 us
// each in bf16.
#include "attn.h"

namespace gdn {

template <typename T, int D, int NR> struct AttnFwdCfg {   // NR: 16-row groups a wave
    static constexpr int RT = 64 * NR;                     // rows a workgroup
    static constexpr int KT = sizeof(T) == 2 ? 64 : 32;    // keys a tile
    static constexpr int ES = (int)sizeof(T), CPR = D * ES / 16;
    static constexpr int OFF_V = KT * CPR * 16, BUF = 2 * OFF_V;   // a tile: [KT][D] keys, [KT][D] values
};

// Workspace of a call in shares: long prefix[B + 1], the keys (of row tiles) before each
// sequence, then for each share its first and last piece of a row tile, float o[slot][D],
// and float lse[slot] of each, slot = RT rows.
struct AttnFwdWs {
    long o, lse, bytes;
    __host__ __device__ AttnFwdWs(int B, int rt, int d) {
        o = ((long)(B + 1) * 8 + 255) & ~255L;
        lse = o + 2L * ATTN_SHARES * rt * d * 4;
        bytes = lse + 2L * ATTN_SHARES * rt * 4;
    }
};

constexpr int FWD_LEAST = 4;   // key tiles of a share
// Rows, at most, that are joined by a workgroup each, not by D / 4 lanes: few rows have many
// parts (32 over 4 heads of 128, one token of 20000 keys 24 us from 52; 32 over 8, 64 tokens 53
// from 55; with 128 tokens it would be 85 from 79).
constexpr int FWD_JOIN = 2048;

// KS: groups of four waves that take the key tiles of a row tile in turn, each with buffers of
// its own, and put their sums together at the end: two for calls that leave compute units idle.
enum { WHOLE, HALVES, SHARED };
template <typename T, int D, int NR, int FORM>
__global__ __launch_bounds__(FORM == HALVES ? 512 : 256, FORM == HALVES ? 1 : 2) void attn_fwd_kernel(AttnArgs a, int per)
{
    typedef AttnFwdCfg<T, D, NR> C;
    constexpr int KT = C::KT, RT = C::RT, NKB = D / 32, NS = KT / 16, NCB = D / 16, KS = FORM == HALVES ? 2 : 1;
    constexpr bool SHARES = FORM == SHARED;
    extern __shared__ char all_lds[];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) & 3, r16 = lane_r16(), gq = lane_gq();
    const int half = KS > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 8) : 0, tid = threadIdx.x & 255;
    char *lds = all_lds + half * 2 * C::BUF;
    const float c = a.scale * LOG2E;
    const int share = SHARES ? blockIdx.x % 8 * (ATTN_SHARES / 8) + blockIdx.x / 8 : 0;   // a head's on one XCD
    auto make = [&](const Seq &s) { return AttnTiles(per, s); };
    Share sh;
    Run cur;
    bool any = true;
    if constexpr (SHARES) {
        if (!share_begin<KT>(a, make, share, ATTN_SHARES, FWD_LEAST, (long *)a.ws, sh) || !share_next<KT>(a, make, sh)) return;
        cur = sh.r;
    } else {
        cur.h = blockIdx.x % a.Hk;
        const Item it = find_tile(a, per, blockIdx.x / a.Hk, gridDim.x / a.Hk);
        if (it.b < 0) return;
        cur.b = it.b;
        cur.t = uniform(it.i);
        cur.s = seq_of(a, it.b);
        cur.j = 0;
        cur.n = cur.end = uniform((make(cur.s).walk(cur.t) + KT - 1) / KT);
        if (half > 0 && cur.end < 2) return;   // nothing to take
        any = cur.end > half;
    }
    auto load = [&](const Run &r, int j, int buffer) {
        char *buf = lds + buffer * C::BUF;
        const T *k = (const T *)a.k + r.s.k0 * a.ks + r.h * D, *v = (const T *)a.v + r.s.k0 * a.vs + r.h * D;
        load_tile<C::CPR, KT>(buf, (const char *)k, a.ks * C::ES, j * KT, r.s.lk, tid);
        load_tile<C::CPR, KT>(buf + C::OFF_V, (const char *)v, a.vs * C::ES, j * KT, r.s.lk, tid);
    };
    const int kb0 = row_base<T, C::CPR>(r16), vb = col_base<T, C::CPR>(4 * gq);
    if (any) load(cur, cur.j + half, 0);
    int buffer = 0;
    bool more = false;
    for (;;) {   // one row tile, or what the share has of it
        const int off = cur.s.lk - cur.s.lq, lr0 = wave * 16 * NR;   // first row of the wave
        const int nlive = min(per, cur.s.lq - cur.t * per) * a.G;    // rows of the tile
        int pos[NR];   // position of this lane's rows; -1: the row sees nothing, or is none
        int tok[NR], head[NR];
        Frag<T> qf[NR][NKB];
#pragma unroll
        for (int g = 0; g < NR; ++g) {
            const int lr = lr0 + 16 * g + r16, i = quotient(lr, a.g_mul, a.g_shift);
            tok[g] = cur.t * per + i;
            head[g] = cur.h * a.G + lr - i * a.G;
            const bool live = lr < nlive && off + tok[g] >= 0;
            pos[g] = live ? off + tok[g] : -1;
            const T *q = (const T *)a.q + (cur.s.q0 + (long)tok[g]) * a.qs + head[g] * D;
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb) qf[g][kb] = live ? load_frag<T>(q + 32 * kb + 8 * gq) : zero_frag<T>();
        }
#pragma unroll
        for (int g = 0; g < NR; ++g)
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb) landed<T>(qf[g][kb]);
        f32x4 acc[NCB][NR];
        float m[NR], l[NR];
#pragma unroll
        for (int g = 0; g < NR; ++g) {
            m[g] = -INFINITY;
            l[g] = 0.f;
#pragma unroll
            for (int cb = 0; cb < NCB; ++cb) acc[cb][g] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
        // keys that some, that all of the wave's rows see
        const int wend = min(lr0 + 16 * NR, nlive) - 1;
        const int wlast = wend < lr0 ? 0 : off + cur.t * per + quotient(max(wend, 0), a.g_mul, a.g_shift) + 1;
        const int wfull = off + cur.t * per + quotient(lr0, a.g_mul, a.g_shift) + 1;
        for (int j = cur.j + half; j < cur.end + half; j += KS) {   // as many times in both halves
            const char *kt = lds + buffer * C::BUF, *vt = kt + C::OFF_V;
            const int k0 = j * KT;
            wait_vm<0>();
            lds_barrier();
            buffer ^= 1;
            if (j + KS < cur.end) {
                load(cur, j + KS, buffer);
            } else if (SHARES) {
                more = share_next<KT>(a, make, sh);
                if (more) load(sh.r, sh.r.j, buffer);
            }
            if (k0 >= wlast || (KS > 1 && j >= cur.end)) continue;   // nothing for this wave in the tile
            f32x4 s[NS][NR];
#pragma unroll
            for (int t = 0; t < NS; ++t) {
#pragma unroll
                for (int g = 0; g < NR; ++g) s[t][g] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int kb = 0; kb < NKB; ++kb) {
                    const Frag<T> kf = row_frag<T>(kt + 16 * t * C::CPR * 16, kb0, kb);
#pragma unroll
                    for (int g = 0; g < NR; ++g) s[t][g] = mma(s[t][g], kf, qf[g][kb]);
                }
            }
            if (sizeof(T) == 2) pipeline<4, NS * NKB, NS * NKB * NR, 1, NR>();
            if (k0 + KT > wfull) {   // the tile reaches past some row's last key
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
            // weights rounded to the storage type for the matrix cores (half a step each,
            // as the output itself); their sum is the unrounded one
#pragma unroll
            for (int t = 0; t < NS; t += 2) {
                Frag<T> pf[NR];
#pragma unroll
                for (int g = 0; g < NR; ++g) pf[g] = reg_frag<T>(s[t][g], s[t + 1][g]);
#pragma unroll
                for (int cb = 0; cb < NCB; ++cb) {
                    const Frag<T> vf = col_frag<T, C::CPR>(vt + 16 * t * C::CPR * 16, vb, cb);
#pragma unroll
                    for (int g = 0; g < NR; ++g) acc[cb][g] = mma(acc[cb][g], vf, pf[g]);
                }
            }
            if (sizeof(T) == 2) pipeline<4, NS * NCB, NS / 2 * NCB * NR, 2, NR>();
        }
        if (KS > 1 && cur.end > 1) {   // the second half's maxima and sums, through LDS, to the first
            lds_barrier();
            f32x4 *to = (f32x4 *)all_lds + wave * (NCB * NR + 1) * 64 + (threadIdx.x & 63);
            static_assert(4 * (NCB * NR + 1) * 64 * 16 <= 4 * C::BUF && NR <= 2, "");
            if (half > 0) {
                f32x4 ml = {m[0], l[0], m[NR - 1], l[NR - 1]};
                to[0] = ml;
#pragma unroll
                for (int cb = 0; cb < NCB; ++cb)
#pragma unroll
                    for (int g = 0; g < NR; ++g) to[(1 + cb * NR + g) * 64] = acc[cb][g];
            }
            lds_barrier();
            if (half > 0) return;
            const f32x4 ml = to[0];
#pragma unroll
            for (int g = 0; g < NR; ++g) {
                const float m1 = ml[2 * g], mn = fmaxf(m[g], m1);
                const float f0 = m[g] == -INFINITY ? 0.f : exp2_hw((m[g] - mn) * c), f1 = m1 == -INFINITY ? 0.f : exp2_hw((m1 - mn) * c);
                m[g] = mn;
                l[g] = l[g] * f0 + ml[2 * g + 1] * f1;
#pragma unroll
                for (int cb = 0; cb < NCB; ++cb) acc[cb][g] = acc[cb][g] * f0 + to[(1 + cb * NR + g) * 64] * f1;
            }
        }
        const bool whole = !SHARES || (cur.j == 0 && cur.end == cur.n);
        const AttnFwdWs lay(a.B, RT, D);
        const long slot = (share * 2 + (cur.j == 0)) * (long)RT;
        float *po = (float *)((char *)a.ws + lay.o) + slot * D, *pl = (float *)((char *)a.ws + lay.lse) + slot;
#pragma unroll
        for (int g = 0; g < NR; ++g) {
            const int lr = lr0 + 16 * g + r16;
            const float ls = rows_sum(l[g]);
            // of part of the keys a row may see none: its sum is 0 (and a NaN where scores are)
            const bool seen = pos[g] >= 0 && (!SHARES || ls != 0.f);
            const float inv = seen ? 1.f / ls : 0.f, lg = seen ? m[g] * c + __builtin_amdgcn_logf(ls) : -INFINITY;
            if (lr >= nlive) continue;
            if (whole) {
                const long row = (cur.s.q0 + (long)tok[g]) * (a.Hk * a.G) + head[g];
#pragma unroll
                for (int cb = 0; cb < NCB; ++cb)
                    store4((T *)a.o + row * D + 16 * cb + 4 * gq, seen ? acc[cb][g] * inv : f32x4{0.f, 0.f, 0.f, 0.f});
                if (gq == 0 && a.lse) a.lse[row] = lg * LN2;
            } else {
                if (seen) {
#pragma unroll
                    for (int cb = 0; cb < NCB; ++cb) store4(po + lr * D + 16 * cb + 4 * gq, acc[cb][g] * inv);
                }
                if (gq == 0) pl[lr] = lg;
            }
        }
        if (!SHARES || !more) break;
        cur = sh.r;
    }
}

// Joins the rows that several shares worked on and writes those that see no key: GR groups of
// D / 4 lanes a row.
template <typename T, int D, int NR, int GR> __global__ __launch_bounds__(256) void attn_fwd_join_kernel(AttnArgs a, int per)
{
    typedef AttnFwdCfg<T, D, NR> C;
    constexpr int LPR = D / 4, KT = C::KT, ROWS = 256 / LPR / GR;   // rows of a workgroup
    const int Hq = a.Hk * a.G, at = threadIdx.x % LPR * 4;
    const long row = (long)blockIdx.x * ROWS + (ROWS > 1 ? threadIdx.x / LPR : 0);
    if (row >= (long)a.Tq * Hq) return;
    const int token = (int)(row / Hq), head = (int)(row - (long)token * Hq);
    const int b = seq_at(a.cu_q, a.B, a.Tq, token);
    const Seq s = seq_lane(a, b);
    const int i = token - s.q0;
    if (i < 0 || i >= s.lq) return;   // of no sequence
    const AttnTiles tl(per, s);
    const int t = i / per, lr = (i - t * per) * a.G + head % a.G, keys = tl.walk(t);
    int wf = 0, wl = -1;
    if (keys > 0) {
        const long *prefix = (const long *)a.ws;
        share_range<KT>(prefix[b] + head / a.G * tl.all() + tl.before(t), tl, t, share_each<KT>(prefix[a.B], ATTN_SHARES, FWD_LEAST), wf, wl);
    }
    if (wf == wl) return;   // written by its one workgroup
    const AttnFwdWs lay(a.B, C::RT, D);
    f32x4 sum;
    float lg;
    if (!join_parts<D, GR>((const float *)((const char *)a.ws + lay.o), (const float *)((const char *)a.ws + lay.lse), wl - wf + 1,
                           [&](int p) { return ((wf + p) * 2 + (p == 0)) * (long)C::RT + lr; }, sum, lg))   // of share wf its last part
        return;
    store4((T *)a.o + row * D + at, sum);
    if (a.lse && at == 0) a.lse[row] = lg * LN2;
}

template <typename T, int D, int NR, int FORM> static hipError_t fwd_enqueue(const AttnArgs &a, const AttnFwdPlan &plan, hipStream_t st)
{
    typedef AttnFwdCfg<T, D, NR> C;
    constexpr int KS = FORM == HALVES ? 2 : 1, BYTES = KS * 2 * C::BUF;
    auto k = attn_fwd_kernel<T, D, NR, FORM>;
    if (BYTES > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute((const void *)k, hipFuncAttributeMaxDynamicSharedMemorySize, BYTES);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(k, dim3((unsigned)(FORM == SHARED ? plan.shares : plan.tiles * a.Hk)), dim3(KS * 256), BYTES, st, a, plan.tokens);
    if (FORM == SHARED) {
        const long rows = (long)a.Tq * a.Hk * a.G;
        constexpr int EACH = 1024 / D;
        if (rows <= FWD_JOIN) hipLaunchKernelGGL((attn_fwd_join_kernel<T, D, NR, EACH>), dim3((unsigned)rows), dim3(256), 0, st, a, plan.tokens);
        else hipLaunchKernelGGL((attn_fwd_join_kernel<T, D, NR, 1>), dim3((unsigned)((rows + EACH - 1) / EACH)), dim3(256), 0, st, a, plan.tokens);
    }
    return hipGetLastError();
}

template <typename T, int D> static hipError_t fwd_launch(AttnArgs a, hipStream_t st)
{
    const AttnFwdPlan plan = attn_fwd_plan(sizeof(T) == 2, a.B, a.Tq, a.Tk, a.Hk, a.G);
    divisor(a.G, a.g_mul, a.g_shift);
    if constexpr (sizeof(T) == 2) {
        if (plan.nr == 2) return plan.shares ? fwd_enqueue<T, D, 2, SHARED>(a, plan, st) : fwd_enqueue<T, D, 2, WHOLE>(a, plan, st);
    }
    if (plan.shares) return fwd_enqueue<T, D, 1, SHARED>(a, plan, st);
    return plan.halves ? fwd_enqueue<T, D, 1, HALVES>(a, plan, st) : fwd_enqueue<T, D, 1, WHOLE>(a, plan, st);
}

hipError_t attn_fwd_launch(bool bf16, int D, const AttnArgs &a, hipStream_t st)
{
    if (bf16) return D == 128 ? fwd_launch<__bf16, 128>(a, st) : fwd_launch<__bf16, 64>(a, st);
    return D == 128 ? fwd_launch<float, 128>(a, st) : fwd_launch<float, 64>(a, st);
}

unsigned long long attn_fwd_workspace(bool bf16, int B, int Tq, int Tk, int Hk, int G, int D)
{
    const AttnFwdPlan plan = attn_fwd_plan(bf16, B, Tq, Tk, Hk, G);
    return plan.shares ? (unsigned long long)AttnFwdWs(B, 64 * plan.nr, D).bytes : 0;
}

} // namespace gdn
