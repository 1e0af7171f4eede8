// latent_step.hip -- absorbed latent attention over a paged cache (gfx950): one
// token a sequence, or M drafted tokens (a tree) a sequence.
//
//   row_j = [c_j (r) | k_j^rope (64)], j over the len_n cached tokens, then the drafts
//   s_ij = scale q_i . row_j,   o_i = sum_j softmax_j(s_ij) c_j
//
// All M * H query rows of a sequence read the same cache rows.  A workgroup
// takes RT of the rows and a run of key tiles; each tile is copied once into LDS and serves as keys (all columns) and as values (the first r).
// In the first product the waves split the tile's keys, in the second the r
// output columns, so the tile is read from LDS twice (three times at RT = 64, where two waves share
// each slab of keys: the queries of 64 rows do not fit one wave's registers).
//
// The runs are equal shares of all key tiles of the batch, whatever the lengths:
// the workgroups add up the tiles of all sequences on their own and each takes
// its share, which may begin and end inside a sequence.  Such pieces go to the
// workspace (normalised, with their log-sum-exp) and a second kernel joins them.
#include "latent.h"

namespace gdn {

constexpr int STEP_CUS = 256;   // one workgroup a compute unit: two tiles fill its LDS

// SPLIT: the waves divide each tile's keys for the scores and the output columns for
// the second product, every wave for all 16 G rows.  Otherwise every wave owns 16 G
// rows and takes all keys and columns for them.
template <typename T, int R, bool SPLIT, int G, int NW> struct StepCfg {
    static constexpr int NTHR = 64 * NW, D = R + LATENT_ROPE;
    static constexpr int RT = SPLIT ? 16 * G : 16 * G * NW;
    static constexpr int KT = sizeof(T) == 2 ? 64 : 32;
    static constexpr int NS = KT / 16;                      // 16-key slabs
    static constexpr int CB = SPLIT ? R / 16 / NW : R / 16; // 16-column blocks of the output a wave
    static constexpr int ES = (int)sizeof(T), CPR = R * ES / 16, RCPR = LATENT_ROPE * ES / 16;
    static constexpr int OFF_R = KT * CPR * 16;             // a tile: [KT][R] latents, [KT][64] rotary keys
    static constexpr int TILE = OFF_R + KT * RCPR * 16;
    static constexpr int PF = 64 * 8 * ES;                  // an operand of weights: 16 rows, 32 keys
    static constexpr int OFF_P = 2 * TILE;                  // [G][KT / 32] of them
    static constexpr int OFF_MX = OFF_P + (SPLIT ? G * KT / 32 * PF : 0);   // [NS][RT] maxima, then sums
    static constexpr int OFF_KV = OFF_MX + (SPLIT ? NS * RT * 4 : 0);     // [2][KT] bytes: key is there
    static constexpr int OFF_SCAN = OFF_KV + 2 * KT;        // [NW + 2] ints
    static constexpr int BYTES = OFF_SCAN + (NW + 2) * 4;
    static_assert(BYTES <= 160 * 1024 && (!SPLIT || NS <= NW), "");
};

// Rows of a workgroup.  fp32 has registers for 16.
__host__ __device__ inline int step_rt(bool bf16, int rows)
{
    return !bf16 || rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
}

// Workgroups that may share the key tiles of one row tile.
__host__ __device__ inline int step_shares(int ntile) {
    int g = STEP_CUS / (ntile < 1 ? 1 : ntile);
    if (g >= 8) g &= ~7;   // the row tiles of one share land on one XCD
    return g < 1 ? 1 : g;
}

// Workspace: int prefix[N + 1] tiles before each sequence, then for each share, its
// first and last piece and each row tile: float o[RT][R], float lse[RT] (base 2).
struct StepWs {
    long part, bytes;
    __host__ __device__ StepWs(int N, int ntile, int rt, int r) {
        part = ((long)(N + 1) * 4 + 255) & ~255L;
        bytes = part + (long)step_shares(ntile) * 2 * ntile * rt * (r + 1) * 4;
    }
};

__device__ __forceinline__ int step_len(const LatentStepArgs &a, int n) {
    const int cap = (int)min((long)a.width * a.page, 0x7fffffffL);
    const int v = a.lens[n];
    return v < 0 ? 0 : v > cap ? cap : v;
}
__device__ __forceinline__ int step_tiles(int len, int drafts, int kt) { return (len + drafts + kt - 1) / kt; }

// A key tile: tile t of the nkt of sequence n, whose cached length is len.
struct StepPos {
    int n, t, len, nkt;
};

template <typename T, int R, bool SPLIT, int G, int NW>
__global__ __launch_bounds__(64 * NW, 1) void latent_step_kernel(LatentStepArgs a, int ntile, int max_shares)
{
    typedef StepCfg<T, R, SPLIT, G, NW> C;
    constexpr int D = C::D, KT = C::KT, RT = C::RT, NKB = D / 32, NS = C::NS, CPR = C::CPR, CB = C::CB;
    extern __shared__ char lds[];
    const int share = blockIdx.x % max_shares, rt = blockIdx.x / max_shares;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), r16 = lane_r16(), gq = lane_gq();
    const int rows = a.M * a.H;
    const float c = a.scale * LOG2E;
    const StepWs lay(a.N, ntile, RT, R);
    int *prefix = (int *)a.ws;
    float *part = (float *)((char *)a.ws + lay.part);

    // tiles before each sequence: every thread adds up a run of sequences, then a scan
    int *scan = (int *)(lds + C::OFF_SCAN);
    const int per = (a.N + C::NTHR - 1) / C::NTHR, s0 = min(a.N, tid * per), s1 = min(a.N, s0 + per);
    int mine = 0;
    for (int n = s0; n < s1; ++n) mine += step_tiles(step_len(a, n), a.drafts, KT);
    int incl = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(incl, d, 64);
        if (lane >= d) incl += v;
    }
    if (lane == 63) scan[wave] = incl;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        if (w < wave) incl += scan[w];
        total += scan[w];
    }
    total = __builtin_amdgcn_readfirstlane(total);
    const int shares = min(max_shares, total);   // none without a tile
    if (share == 0 && rt == 0) {
        int at = incl - mine;
        for (int n = s0; n < s1; ++n) {
            prefix[n] = at;
            at += step_tiles(step_len(a, n), a.drafts, KT);
        }
        if (tid == 0) prefix[a.N] = total;
    }
    if (share >= shares) return;
    const int g0 = (int)((long)share * total / shares), g1 = (int)((long)(share + 1) * total / shares);
    if (g0 >= incl - mine && g0 < incl) {
        int at = incl - mine;
        for (int n = s0; n < s1; ++n) {
            const int t = step_tiles(step_len(a, n), a.drafts, KT);
            if (g0 >= at && g0 < at + t) {
                scan[NW] = n;
                scan[NW + 1] = g0 - at;
            }
            at += t;
        }
    }
    __syncthreads();

    StepPos cur, nxt;
    cur.n = __builtin_amdgcn_readfirstlane(scan[NW]);
    cur.t = __builtin_amdgcn_readfirstlane(scan[NW + 1]);
    cur.len = __builtin_amdgcn_readfirstlane(step_len(a, cur.n));
    cur.nkt = step_tiles(cur.len, a.drafts, KT);
    auto after = [&](StepPos p) {   // called only while a tile is left
        if (++p.t == p.nkt) {
            p.t = 0;
            do {
                ++p.n;
                p.len = __builtin_amdgcn_readfirstlane(step_len(a, p.n));
                p.nkt = step_tiles(p.len, a.drafts, KT);
            } while (p.nkt == 0 && p.n + 1 < a.N);
        }
        return p;
    };
    // The wave copies WR rows of a tile; its lanes look up one each (lanes beyond
    // WR repeat them): page() the page of the lane's row, a tile ahead of its use,
    // load_tile() the copies into buffer `buf`.
    constexpr int WR = KT / NW;
    const int krow = wave * WR + (lane & (WR - 1));
    auto page = [&](const StepPos &p) {
        const int key = p.t * KT + krow;
        return key < p.len ? a.table[(long)p.n * a.width + key / a.page] : -1;
    };
    auto load_tile = [&](const StepPos &p, int id, int buf) {
        const int key = p.t * KT + krow;
        const char *src = (const char *)latent_zero;
        bool there = false;
        if (key < p.len) {
            there = id >= 0 && id < a.pages;   // any other page holds nothing
            if (there) src = (const char *)a.cache + ((long)id * a.page + key % a.page) * (D * C::ES);
        } else if (key - p.len < a.drafts) {
            there = true;
            src = (const char *)a.draft + ((long)p.n * a.M + (key - p.len)) * (D * C::ES);
        }
        if (lane < WR) lds[C::OFF_KV + buf * KT + krow] = there;
        const int lo = (int)(uintptr_t)src, hi = (int)((uintptr_t)src >> 32);
        auto row_ptr = [&](int row) {   // of a row that differs by lane
            return (const char *)(((uintptr_t)(unsigned)__shfl(hi, row, 64) << 32) | (unsigned)__shfl(lo, row, 64));
        };
        char *dst = lds + buf * C::TILE + wave * WR * CPR * 16;
        if constexpr (CPR >= 64) {   // a row is whole instructions: its address is uniform
#pragma unroll
            for (int i = 0; i < WR; ++i) {
                const unsigned rlo = (unsigned)__builtin_amdgcn_readlane(lo, i), rhi = (unsigned)__builtin_amdgcn_readlane(hi, i);
                const char *q = (const char *)(((uintptr_t)rhi << 32) | rlo);
#pragma unroll
                for (int k = 0; k < CPR / 64; ++k)
                    g2lds16s(q, (unsigned)((k * 64 + (lane ^ swz<CPR>(wave * WR + i))) * 16), dst + (i * CPR / 64 + k) * 1024);
            }
        } else {
#pragma unroll
            for (int i = 0; i < WR * CPR / 64; ++i) {
                const int row = i * (64 / CPR) + lane / CPR;
                g2lds16(row_ptr(row) + ((lane % CPR) ^ swz<CPR>(wave * WR + row)) * 16, dst + i * 1024);
            }
        }
        char *rdst = lds + buf * C::TILE + C::OFF_R + wave * WR * C::RCPR * 16;
#pragma unroll
        for (int i = 0; i < WR * C::RCPR / 64; ++i) {
            const int row = i * (64 / C::RCPR) + lane / C::RCPR, ch = (lane % C::RCPR) ^ swz<C::RCPR>(wave * WR + row);
            const char *q = row_ptr(row);   // a row that is not there: the first of the zeros
            g2lds16(__shfl((int)there, row, 64) ? q + R * C::ES + ch * 16 : q, rdst + i * 1024);
        }
    };

    // lane parts of the LDS addresses; first product: this wave's slab of keys (SPLIT)
    const int slab = SPLIT ? wave : 0, row0 = SPLIT ? 0 : wave * 16 * G;
    const int nb = row_base<T, CPR>(16 * slab + r16), rb = row_base<T, C::RCPR>(16 * slab + r16);
    // second product: this wave's first 16-column block, as a part inside 256 bytes
    // and whole ones
    constexpr int PC = 16 / C::ES;
    static_assert(CB % PC == 0 || PC % CB == 0, "");
    const int col0 = SPLIT ? wave * CB : 0;
    const int vb = col_base<T, CPR>(4 * gq) ^ (col0 % PC * 16 * C::ES), vcol = col0 / PC * 256;
    Frag<T> qf[G][NKB];
    unsigned long long bits[G];
    f32x4 acc[CB][G];
    float m[G], l[G];
    int buf = 0, kt0 = cur.t, idn = page(cur);
    bool fresh = true;
    load_tile(cur, idn, 0);
    if (g0 + 1 < g1) {
        nxt = after(cur);
        idn = page(nxt);
    }
    for (int g = g0;; ++g, buf ^= 1) {
        if (fresh) {
#pragma unroll
            for (int rg = 0; rg < G; ++rg) {
                const int row = rt * RT + row0 + 16 * rg + r16;
                const bool live = row < rows;
                const T *q = (const T *)a.q + ((long)cur.n * rows + (live ? row : 0)) * D;
#pragma unroll
                for (int kb = 0; kb < NKB; ++kb)
                    qf[rg][kb] = live ? load_frag<T>(q + 32 * kb + 8 * gq) : zero_frag<T>();
                const int node = row / a.H;
                bits[rg] = !live || !a.drafts ? 0ull
                         : a.tree ? (unsigned long long)a.tree[(long)cur.n * a.M + node]
                         : node >= 63 ? ~0ull : (2ull << node) - 1;
                m[rg] = -INFINITY;
                l[rg] = 0.f;
#pragma unroll
                for (int cb = 0; cb < CB; ++cb) acc[cb][rg] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
            fresh = false;
        }
        const bool more = g + 1 < g1;
        wait_vm<0>();
        lds_barrier();
        StepPos aft = nxt;
        if (g + 2 < g1) aft = after(nxt);
        if (more) load_tile(nxt, idn, buf ^ 1);
        if (g + 2 < g1) idn = page(aft);

        const char *tile = lds + buf * C::TILE, *there4 = lds + C::OFF_KV + buf * KT + 16 * slab + 4 * gq;
        const int key = cur.t * KT + 16 * slab + 4 * gq;   // first of this lane's four, in the first slab
        // -inf where the row does not see the key.  Without branches: the compiler
        // has lost the masked value of a vector element that two nested ones decide.
        auto mask = [&](f32x4 s, unsigned there, int first, unsigned long long bit) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int d = first + e - cur.len;
                const unsigned in = d < 0 ? 1u : (unsigned)(bit >> (d & 63));
                s[e] = (in & (there >> (8 * e)) & 1u) ? s[e] : -INFINITY;
            }
            return s;
        };
        if constexpr (SPLIT) {
            float *mx = (float *)(lds + C::OFF_MX);
            f32x4 s[G];
            if (wave < NS) {
#pragma unroll
                for (int rg = 0; rg < G; ++rg) s[rg] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int kb = 0; kb < NKB; ++kb) {
                    const Frag<T> kf = kb < R / 32 ? row_frag<T>(tile, nb, kb) : row_frag<T>(tile + C::OFF_R, rb, kb - R / 32);
#pragma unroll
                    for (int rg = 0; rg < G; ++rg) s[rg] = mma(s[rg], kf, qf[rg][kb]);
                }
                const unsigned there = *reinterpret_cast<const unsigned *>(there4);
                if (__any(there != 0x01010101u || key + 3 >= cur.len)) {
#pragma unroll
                    for (int rg = 0; rg < G; ++rg) s[rg] = mask(s[rg], there, key, bits[rg]);
                }
#pragma unroll
                for (int rg = 0; rg < G; ++rg) {
                    const float t = rows_max(fmaxf(fmaxf(s[rg][0], s[rg][1]), fmaxf(s[rg][2], s[rg][3])));
                    if (gq == 0) mx[wave * RT + 16 * rg + r16] = t;
                }
            }
            lds_barrier();
#pragma unroll
            for (int rg = 0; rg < G; ++rg) {
                float t = mx[16 * rg + r16];
#pragma unroll
                for (int w = 1; w < NS; ++w) t = fmaxf(t, mx[w * RT + 16 * rg + r16]);
                const bool up = (t - m[rg]) * c > RAISE;   // false while both are -inf
                if (__any(up)) {
                    const float mn = up ? t : m[rg], al = up ? exp2_hw((m[rg] - mn) * c) : 1.f;
                    m[rg] = mn;
                    l[rg] *= al;
#pragma unroll
                    for (int cb = 0; cb < CB; ++cb) acc[cb][rg] *= al;
                }
                if (wave < NS) {
                    const float mb = m[rg] == -INFINITY ? 0.f : m[rg] * c;
                    f32x4 p;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        p[e] = exp2_hw(__builtin_fmaf(s[rg][e], c, -mb));
                        l[rg] += p[e];
                    }
                    // as the lane's own half of the operand of 32 keys
                    store4((T *)(lds + C::OFF_P + (rg * KT / 32 + wave / 2) * C::PF + lane * 8 * C::ES) + 4 * (wave & 1), p);
                }
            }
            lds_barrier();
#pragma unroll
            for (int kk = 0; kk < KT / 32; ++kk) {
                Frag<T> pf[G];
#pragma unroll
                for (int rg = 0; rg < G; ++rg) pf[rg] = load_frag<T>((const T *)(lds + C::OFF_P + (rg * KT / 32 + kk) * C::PF) + lane * 8);
#pragma unroll
                for (int cb = 0; cb < CB; ++cb) {
                    const Frag<T> vf = col_frag<T, CPR>(tile + 32 * kk * CPR * 16 + vcol, vb, cb);
#pragma unroll
                    for (int rg = 0; rg < G; ++rg) acc[cb][rg] = mma(acc[cb][rg], vf, pf[rg]);
                }
            }
        } else {
            f32x4 s[NS][G];
#pragma unroll
            for (int t = 0; t < NS; ++t) {
#pragma unroll
                for (int rg = 0; rg < G; ++rg) s[t][rg] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int kb = 0; kb < NKB; ++kb) {
                    const Frag<T> kf = kb < R / 32 ? row_frag<T>(tile + 16 * t * CPR * 16, nb, kb)
                                                   : row_frag<T>(tile + C::OFF_R + 16 * t * C::RCPR * 16, rb, kb - R / 32);
#pragma unroll
                    for (int rg = 0; rg < G; ++rg) s[t][rg] = mma(s[t][rg], kf, qf[rg][kb]);
                    if (kb % 3 == 2) GDN_SCHED_FENCE();   // bounds the operands in flight: registers
                }
            }
            unsigned there[NS], all = 0x01010101u;
#pragma unroll
            for (int t = 0; t < NS; ++t) {
                there[t] = *reinterpret_cast<const unsigned *>(there4 + 16 * t);
                all &= there[t];
            }
            if (__any(all != 0x01010101u || key + KT - 13 >= cur.len)) {
#pragma unroll
                for (int t = 0; t < NS; ++t)
#pragma unroll
                    for (int rg = 0; rg < G; ++rg) s[t][rg] = mask(s[t][rg], there[t], key + 16 * t, bits[rg]);
            }
#pragma unroll
            for (int rg = 0; rg < G; ++rg) {
                float mx = -INFINITY;
#pragma unroll
                for (int t = 0; t < NS; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx = fmaxf(mx, s[t][rg][e]);
                mx = rows_max(mx);
                const bool up = (mx - m[rg]) * c > RAISE;
                if (__any(up)) {
                    const float mn = up ? mx : m[rg], al = up ? exp2_hw((m[rg] - mn) * c) : 1.f;
                    m[rg] = mn;
                    l[rg] *= al;
#pragma unroll
                    for (int cb = 0; cb < CB; ++cb) acc[cb][rg] *= al;
                }
                const float mb = m[rg] == -INFINITY ? 0.f : m[rg] * c;
#pragma unroll
                for (int t = 0; t < NS; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float p = exp2_hw(__builtin_fmaf(s[t][rg][e], c, -mb));
                        s[t][rg][e] = p;
                        l[rg] += p;
                    }
            }
#pragma unroll
            for (int t = 0; t < NS; t += 2) {
                Frag<T> pf[G];
#pragma unroll
                for (int rg = 0; rg < G; ++rg) pf[rg] = reg_frag<T>(s[t][rg], s[t + 1][rg]);
#pragma unroll
                for (int cb = 0; cb < CB; ++cb) {
                    const Frag<T> vf = col_frag<T, CPR>(tile + 16 * t * CPR * 16, vb, cb);
#pragma unroll
                    for (int rg = 0; rg < G; ++rg) acc[cb][rg] = mma(acc[cb][rg], vf, pf[rg]);
                    if (cb % 4 == 3) GDN_SCHED_FENCE();
                }
            }
        }
        if (!more || nxt.n != cur.n) {
            // the sequence's (or the share's) last tile: the rows' sums, then write
            float *mx = (float *)(lds + C::OFF_MX), ls[G];
#pragma unroll
            for (int rg = 0; rg < G; ++rg) ls[rg] = rows_sum(l[rg]);
            if constexpr (SPLIT) {
                lds_barrier();
#pragma unroll
                for (int rg = 0; rg < G; ++rg)
                    if (gq == 0 && wave < NS) mx[wave * RT + 16 * rg + r16] = ls[rg];
                lds_barrier();
#pragma unroll
                for (int rg = 0; rg < G; ++rg) {
                    ls[rg] = 0.f;
#pragma unroll
                    for (int w = 0; w < NS; ++w) ls[rg] += mx[w * RT + 16 * rg + r16];
                }
            }
            const bool whole = kt0 == 0 && cur.t + 1 == cur.nkt;
            const long slot = ((long)share * 2 + (kt0 == 0 ? 1 : 0)) * ntile + rt;
            float *po = part + slot * RT * (R + 1), *pl = po + RT * R;
#pragma unroll
            for (int rg = 0; rg < G; ++rg) {
                const int lr = row0 + 16 * rg + r16, row = rt * RT + lr;
                const bool seen = ls[rg] > 0.f;
                const float inv = seen ? 1.f / ls[rg] : 0.f;
                const float lg = seen ? m[rg] * c + __builtin_amdgcn_logf(ls[rg]) : -INFINITY;
                if (row >= rows) continue;
                T *o = (T *)a.o + ((long)cur.n * rows + row) * R + (SPLIT ? 16 * wave * CB : 0) + 4 * gq;
                float *w = po + (long)lr * R + (SPLIT ? 16 * wave * CB : 0) + 4 * gq;
#pragma unroll
                for (int cb = 0; cb < CB; ++cb) {
                    const f32x4 v = seen ? acc[cb][rg] * inv : f32x4{0.f, 0.f, 0.f, 0.f};
                    if (whole) store4(o + 16 * cb, v);
                    else store4(w + 16 * cb, v);
                }
                if (gq == 0 && (!SPLIT || wave == 0)) {
                    if (!whole) pl[lr] = lg;
                    else if (a.lse) a.lse[(long)cur.n * rows + row] = lg * LN2;
                }
            }
            if (!more) break;
            fresh = true;
            kt0 = 0;
        }
        cur = nxt;
        nxt = aft;
    }
}

// Joins the pieces of every sequence that more than one share worked on, and
// writes the sequences that have no key at all.  One workgroup a (sequence, row):
// four waves, each a quarter of the pieces, four of them in flight.
template <typename T, int R>
__global__ __launch_bounds__(256) void latent_join_kernel(LatentStepArgs a, int ntile, int max_shares, int RT)
{
    constexpr int PER = R / 64;   // columns a lane
    __shared__ float sums[4][R];
    __shared__ float tops[4];
    const int rows = a.M * a.H, n = blockIdx.x / rows, row = blockIdx.x % rows;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const StepWs lay(a.N, ntile, RT, R);
    const int *prefix = (const int *)a.ws;
    const int c0 = prefix[n], c1 = prefix[n + 1], total = prefix[a.N], shares = min(max_shares, total);
    int wf = 0, wl = -1;
    if (c1 > c0) {
        wf = (int)(((long)(c0 + 1) * shares - 1) / total);
        wl = (int)(((long)c1 * shares - 1) / total);
        if (wf == wl) return;   // written by its one share
    }
    // piece w of the sequence: the last of share wf, the first of the others
    const long step = (long)2 * ntile * RT * (R + 1);
    const float *first = (const float *)((const char *)a.ws + lay.part) + (long)(row / RT) * RT * (R + 1);
    const float *last = first + (long)ntile * RT * (R + 1);
    const int lr = row % RT;
    auto piece = [&](int w) { return (w == wf ? last : first) + w * step; };
    float top = -INFINITY;
    for (int w = wf + threadIdx.x; w <= wl; w += 256) top = fmaxf(top, piece(w)[RT * R + lr]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
    if (lane == 0) tops[wave] = top;
    __syncthreads();
    top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
    float sum[PER], ls = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) sum[i] = 0.f;
    if (top != -INFINITY) {
#pragma unroll 4
        for (int w = wf + wave; w <= wl; w += 4) {
            const float *p = piece(w);
            const float f = exp2_hw(p[RT * R + lr] - top);
            ls += f;
#pragma unroll
            for (int i = 0; i < PER; i += 4) {
                const f32x4 v = *reinterpret_cast<const f32x4 *>(p + (long)lr * R + i * 64 + lane * 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[i + e] += f * v[e];
            }
        }
    }
    __syncthreads();
    if (lane == 0) tops[wave] = ls;
#pragma unroll
    for (int i = 0; i < PER; i += 4)
        *reinterpret_cast<f32x4 *>(&sums[wave][i * 64 + lane * 4]) = f32x4{sum[i], sum[i + 1], sum[i + 2], sum[i + 3]};
    __syncthreads();
    ls = tops[0] + tops[1] + tops[2] + tops[3];
    const float inv = ls > 0.f ? 1.f / ls : 0.f;
    const int col = threadIdx.x * 4;
    if (col < R) {
        f32x4 v = *reinterpret_cast<const f32x4 *>(&sums[0][col]);
#pragma unroll
        for (int w = 1; w < 4; ++w) v += *reinterpret_cast<const f32x4 *>(&sums[w][col]);
        store4((T *)a.o + ((long)n * rows + row) * R + col, v * inv);
    }
    if (a.lse && threadIdx.x == 0)
        a.lse[(long)n * rows + row] = ls > 0.f ? (top + __builtin_amdgcn_logf(ls)) * LN2 : -INFINITY;
}

template <typename T, int R, bool SPLIT, int G, int NW>
static hipError_t step_launch(const LatentStepArgs &a, hipStream_t st)
{
    typedef StepCfg<T, R, SPLIT, G, NW> C;
    const int rows = a.M * a.H, ntile = (rows + C::RT - 1) / C::RT, shares = step_shares(ntile);
    auto k = latent_step_kernel<T, R, SPLIT, G, NW>;
    const hipError_t e = hipFuncSetAttribute((const void *)k, hipFuncAttributeMaxDynamicSharedMemorySize, C::BYTES);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k, dim3(ntile * shares), dim3(C::NTHR), C::BYTES, st, a, ntile, shares);
    hipLaunchKernelGGL((latent_join_kernel<T, R>), dim3(a.N * rows), dim3(256), 0, st, a, ntile, shares, C::RT);
    return hipGetLastError();
}

template <int R> static hipError_t step_bf16(const LatentStepArgs &a, hipStream_t st)
{
    switch (step_rt(true, a.M * a.H)) {
    case 16: return step_launch<__bf16, R, true, 1, 4>(a, st);
    case 32: return step_launch<__bf16, R, true, 2, 4>(a, st);
    case 64: return step_launch<__bf16, R, false, 1, 4>(a, st);
    default: return step_launch<__bf16, R, false, 1, 8>(a, st);
    }
}

hipError_t latent_step_launch(bool bf16, int r, const LatentStepArgs &a, hipStream_t st)
{
    if (!bf16) return r == 512 ? step_launch<float, 512, true, 1, 4>(a, st) : step_launch<float, 256, true, 1, 4>(a, st);
    return r == 512 ? step_bf16<512>(a, st) : step_bf16<256>(a, st);
}

unsigned long long latent_step_workspace(bool bf16, int N, int M, int H, int r)
{
    const int rt = step_rt(bf16, M * H), ntile = (M * H + rt - 1) / rt;
    return (unsigned long long)StepWs(N, ntile, rt, r).bytes;
}

} // namespace gdn
