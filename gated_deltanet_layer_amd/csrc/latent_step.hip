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

template <typename T, int R, int NRG> struct StepCfg {
    static constexpr int RH = NRG >= 4 ? 2 : 1;             // waves that share a key slab, each with NRG / RH row groups
    static constexpr int NW = 4 * RH, NTHR = 64 * NW;
    static constexpr int D = R + LATENT_ROPE;
    static constexpr int RT = 16 * NRG;
    static constexpr int KT = sizeof(T) == 2 ? 64 : 32;
    static constexpr int NS = KT / 16;                      // 16-key slabs
    static constexpr int CPR = D * (int)sizeof(T) / 16;
    static constexpr int TILE = KT * CPR * 16;
    static constexpr int PCPR = KT * (int)sizeof(T) / 16;   // 8
    static constexpr int OFF_P = 2 * TILE;                  // weights [RT][KT]
    static constexpr int OFF_MX = OFF_P + RT * PCPR * 16;   // [4][RT] tile maxima, then sums
    static constexpr int OFF_KV = OFF_MX + 4 * RT * 4;     // [2][KT] bytes: key is there
    static constexpr int OFF_SCAN = OFF_KV + 2 * KT;        // [NTHR] ints and 4 more
    static constexpr int BYTES = OFF_SCAN + (NTHR + 4) * 4;
    static_assert(PCPR == 8 && BYTES <= 160 * 1024, "LDS");
};

__host__ __device__ inline int step_rt(bool bf16, int rows) { return !bf16 || rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

// Workgroups that share the key tiles of one row tile.
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
__device__ __forceinline__ int step_tiles(const LatentStepArgs &a, int n, int kt) {
    return (int)(((long)step_len(a, n) + a.drafts + kt - 1) / kt);
}

template <typename T, int R, int NRG>
__global__ __launch_bounds__((StepCfg<T, R, NRG>::NTHR), 1) void latent_step_kernel(LatentStepArgs a, int ntile, int shares)
{
    typedef StepCfg<T, R, NRG> C;
    constexpr int D = C::D, KT = C::KT, RT = C::RT, NKB = D / 32, NS = C::NS, CPR = C::CPR;
    constexpr int NTHR = C::NTHR, NW = C::NW, CB = R / 16 / NW, QG = NRG / C::RH;
    extern __shared__ char lds[];
    const int share = blockIdx.x % shares, rt = blockIdx.x / shares;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), r16 = lane_r16(), gq = lane_gq();
    const int rows = a.M * a.H;
    const float c = a.scale * LOG2E;
    const StepWs lay(a.N, ntile, RT, R);
    int *prefix = (int *)a.ws;
    float *part = (float *)((char *)a.ws + lay.part);

    // tiles before each sequence: every thread adds up a run of sequences, then a scan
    int *scan = (int *)(lds + C::OFF_SCAN);
    const int per = (a.N + NTHR - 1) / NTHR, s0 = min(a.N, tid * per), s1 = min(a.N, s0 + per);
    int mine = 0;
    for (int n = s0; n < s1; ++n) mine += step_tiles(a, n, KT);
    scan[tid] = mine;
    __syncthreads();
    for (int d = 1; d < NTHR; d <<= 1) {
        const int v = tid >= d ? scan[tid - d] : 0;
        __syncthreads();
        scan[tid] += v;
        __syncthreads();
    }
    const int total = scan[NTHR - 1];
    const int g0 = (int)((long)share * total / shares), g1 = (int)((long)(share + 1) * total / shares);
    {
        int at = scan[tid] - mine;
        if (share == 0 && rt == 0) {
            for (int n = s0; n < s1; ++n) {
                prefix[n] = at;
                at += step_tiles(a, n, KT);
            }
            if (tid == 0) prefix[a.N] = total;
        }
        at = scan[tid] - mine;
        if (g0 >= at && g0 < at + mine)
            for (int n = s0; n < s1; ++n) {
                const int t = step_tiles(a, n, KT);
                if (g0 >= at && g0 < at + t) {
                    scan[NTHR] = n;
                    scan[NTHR + 1] = g0 - at;
                }
                at += t;
            }
    }
    __syncthreads();
    if (g0 >= g1) return;
    int n = __builtin_amdgcn_readfirstlane(scan[NTHR]), kt = __builtin_amdgcn_readfirstlane(scan[NTHR + 1]);
    int len = step_len(a, n), nkt = step_tiles(a, n, KT);

    // Enqueue the copies of tile t of sequence s into buffer `buf`; the wave's
    // lanes r16 look up the rows that the wave copies.
    constexpr int WR = KT / NW;   // rows a wave copies
    auto load_tile = [&](int s, int slen, int t, int buf) {
        const int key = t * KT + wave * WR + (lane & (WR - 1));
        const char *src = (const char *)&latent_zero;
        bool there = false;
        if (key < slen) {
            const int pg = key / a.page, id = a.table[(long)s * a.width + pg];
            there = id >= 0 && id < a.pages;   // any other page holds nothing
            if (there) src = (const char *)a.cache + ((long)id * a.page + (key - pg * a.page)) * (D * (int)sizeof(T));
        } else if (key - slen < a.drafts) {
            there = true;
            src = (const char *)a.draft + ((long)s * a.M + (key - slen)) * (D * (int)sizeof(T));
        }
        if (lane < WR) lds[C::OFF_KV + buf * KT + wave * WR + lane] = there;
        const int lo = (int)(uintptr_t)src, hi = (int)((uintptr_t)src >> 32);
        char *dst = lds + buf * C::TILE + wave * WR * CPR * 16;
#pragma unroll
        for (int i = 0; i < WR * CPR / 64; ++i) {
            const int slot = i * 64 + lane, row = slot / CPR, ch = (slot % CPR) ^ ((wave * WR + row) & 7);
            const unsigned plo = (unsigned)__shfl(lo, row, 64), phi = (unsigned)__shfl(hi, row, 64);
            const char *p = (const char *)(((uintptr_t)phi << 32) | plo);
            const bool ok = __shfl((int)there, row, 64);
            g2lds16(ok ? p + ch * 16 : p, dst + i * 1024);
        }
    };

    const int slab = wave & 3, rg0 = (wave >> 2) * QG;   // first product: keys and row groups of this wave
    Frag<T> qf[QG][NKB];
    unsigned long long bits[QG];
    f32x4 acc[CB][NRG];
    float m[NRG], l[QG];
    int g = g0, buf = 0, kt0 = kt;
    bool fresh = true;
    load_tile(n, len, kt, 0);
    while (true) {
        if (fresh) {
#pragma unroll
            for (int rg = 0; rg < QG; ++rg) {
                const int row = rt * RT + 16 * (rg0 + rg) + r16;
                const bool live = row < rows;
                const T *q = (const T *)a.q + ((long)n * rows + (live ? row : 0)) * D;
#pragma unroll
                for (int kb = 0; kb < NKB; ++kb)
                    qf[rg][kb] = live ? load_frag<T>(q + 32 * kb + 8 * gq) : zero_frag<T>();
                const int node = row / a.H;
                bits[rg] = !live || !a.drafts ? 0ull
                         : a.tree ? (unsigned long long)a.tree[(long)n * a.M + node]
                         : node >= 63 ? ~0ull : (2ull << node) - 1;
                l[rg] = 0.f;
            }
#pragma unroll
            for (int rg = 0; rg < NRG; ++rg) {
                m[rg] = -INFINITY;
#pragma unroll
                for (int cb = 0; cb < CB; ++cb) acc[cb][rg] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
            fresh = false;
        }
        // the tile after this one
        int n2 = n, kt2 = kt + 1, len2 = len, nkt2 = nkt;
        const bool more = g + 1 < g1;
        if (more && kt2 == nkt) {
            kt2 = 0;
            do {
                ++n2;
                nkt2 = step_tiles(a, n2, KT);
            } while (nkt2 == 0 && n2 + 1 < a.N);   // a tile is left, so a sequence with one follows
            len2 = step_len(a, n2);
        }
        wait_vm<0>();
        lds_barrier();
        if (more) load_tile(n2, len2, kt2, buf ^ 1);

        const char *tile = lds + buf * C::TILE;
        float *mx = (float *)(lds + C::OFF_MX);
        f32x4 s[QG];
        if (slab < NS) {
#pragma unroll
            for (int rg = 0; rg < QG; ++rg) s[rg] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb) {
                const Frag<T> kf = row_frag<T, CPR>(tile, 16 * slab, kb);
#pragma unroll
                for (int rg = 0; rg < QG; ++rg) s[rg] = mma(s[rg], kf, qf[rg][kb]);
            }
            const int key = kt * KT + 16 * slab + 4 * gq;
            const unsigned there = *reinterpret_cast<const unsigned *>(lds + C::OFF_KV + buf * KT + 16 * slab + 4 * gq);
            if (__any(there != 0x01010101u || key + 3 >= len)) {
#pragma unroll
                for (int rg = 0; rg < QG; ++rg)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        // without branches: the compiler has lost the masked value of a
                        // vector element that two nested branches decide
                        const int d = key + e - len;
                        const unsigned in = d < 0 ? 1u : (unsigned)(bits[rg] >> (d & 63));
                        s[rg][e] = (in & (there >> (8 * e)) & 1u) ? s[rg][e] : -INFINITY;
                    }
            }
#pragma unroll
            for (int rg = 0; rg < QG; ++rg) {
                const float t = rows_max(fmaxf(fmaxf(s[rg][0], s[rg][1]), fmaxf(s[rg][2], s[rg][3])));
                if (gq == 0) mx[slab * RT + 16 * (rg0 + rg) + r16] = t;
            }
        }
        lds_barrier();
        float al[NRG];
#pragma unroll
        for (int rg = 0; rg < NRG; ++rg) {
            float t = mx[16 * rg + r16];
#pragma unroll
            for (int w = 1; w < NS; ++w) t = fmaxf(t, mx[w * RT + 16 * rg + r16]);
            const bool up = (t - m[rg]) * c > RAISE;   // false while both are -inf
            const float mn = up ? t : m[rg];
            al[rg] = up ? exp2_hw((m[rg] - mn) * c) : 1.f;
            m[rg] = mn;
            if (__any(up)) {
#pragma unroll
                for (int cb = 0; cb < CB; ++cb) acc[cb][rg] *= al[rg];
            }
        }
#pragma unroll
        for (int rg = 0; rg < QG; ++rg)
            if (slab < NS) {
                // this wave's row groups: rg0 is 0 or NRG / 2, a uniform choice
                const float mr = C::RH == 1 || rg0 == 0 ? m[rg] : m[NRG - QG + rg];
                const float ar = C::RH == 1 || rg0 == 0 ? al[rg] : al[NRG - QG + rg];
                const float mb = mr == -INFINITY ? 0.f : mr * c;
                l[rg] *= ar;
                f32x4 p;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    p[e] = exp2_hw(__builtin_fmaf(s[rg][e], c, -mb));
                    l[rg] += p[e];
                }
                const int row = 16 * (rg0 + rg) + r16, col = 16 * slab + 4 * gq;
                char *pp = lds + C::OFF_P + latent_off<C::PCPR>(row, col * (int)sizeof(T) / 16) + (col * (int)sizeof(T) & 15);
                store4((T *)pp, p);
            }
        lds_barrier();
#pragma unroll
        for (int kk = 0; kk < KT / 32; ++kk) {
            Frag<T> pf[NRG];
#pragma unroll
            for (int rg = 0; rg < NRG; ++rg) pf[rg] = row_frag<T, C::PCPR>(lds + C::OFF_P, 16 * rg, kk);
#pragma unroll
            for (int cb = 0; cb < CB; ++cb) {
                const Frag<T> vf = col_frag<T, CPR>(tile, 32 * kk + 8 * gq, 32 * kk + 8 * gq + 4, wave * CB + cb);
#pragma unroll
                for (int rg = 0; rg < NRG; ++rg) acc[cb][rg] = mma(acc[cb][rg], vf, pf[rg]);
            }
        }
        ++g;
        buf ^= 1;
        if (!more || n2 != n) {
            // the sequence's (or the share's) last tile: add the waves' sums, write
            lds_barrier();
#pragma unroll
            for (int rg = 0; rg < QG; ++rg) {
                const float t = rows_sum(l[rg]);
                if (gq == 0 && slab < NS) mx[slab * RT + 16 * (rg0 + rg) + r16] = t;
            }
            lds_barrier();
            const bool whole = kt0 == 0 && kt + 1 == nkt;
            const long slot = (((long)share * 2 + (kt0 == 0 ? 1 : 0)) * ntile + rt);
            float *po = part + slot * RT * (R + 1), *pl = po + RT * R;
#pragma unroll
            for (int rg = 0; rg < NRG; ++rg) {
                const int lr = 16 * rg + r16, row = rt * RT + lr;
                float ls = 0.f;
#pragma unroll
                for (int w = 0; w < NS; ++w) ls += mx[w * RT + lr];
                const bool seen = ls > 0.f;
                const float inv = seen ? 1.f / ls : 0.f;
                const float lg = seen ? m[rg] * c + __builtin_amdgcn_logf(ls) : -INFINITY;
                if (row < rows) {
#pragma unroll
                    for (int cb = 0; cb < CB; ++cb) {
                        const int col = 16 * (wave * CB + cb) + 4 * gq;
                        const f32x4 v = seen ? acc[cb][rg] * inv : f32x4{0.f, 0.f, 0.f, 0.f};
                        if (whole) store4((T *)a.o + ((long)n * rows + row) * R + col, v);
                        else store4(po + (long)lr * R + col, v);
                    }
                    if (wave == 0 && gq == 0) {
                        if (!whole) pl[lr] = lg;
                        else if (a.lse) a.lse[(long)n * rows + row] = lg * LN2;
                    }
                }
            }
            if (!more) break;
            lds_barrier();
            fresh = true;
            kt0 = 0;
        }
        n = n2; kt = kt2; len = len2; nkt = nkt2;
    }
}

// Joins the pieces of every sequence that more than one share worked on, and
// writes the sequences that have no key at all.  One workgroup a (sequence, four
// rows), one wave a row.
template <typename T, int R>
__global__ __launch_bounds__(256) void latent_join_kernel(LatentStepArgs a, int ntile, int shares, int RT)
{
    const int rows = a.M * a.H, groups = (rows + 3) / 4;
    const int n = blockIdx.x / groups, row = (blockIdx.x % groups) * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
    if (row >= rows) return;
    const StepWs lay(a.N, ntile, RT, R);
    const int *prefix = (const int *)a.ws;
    const float *part = (const float *)((const char *)a.ws + lay.part);
    const int c0 = prefix[n], c1 = prefix[n + 1];
    const long total = prefix[a.N];
    constexpr int PER = R / 64;   // columns a lane
    float sum[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) sum[i] = 0.f;
    float lg = -INFINITY, ls = 0.f;
    if (c1 > c0) {
        const int wf = (int)(((long)(c0 + 1) * shares - 1) / total), wl = (int)(((long)c1 * shares - 1) / total);
        if (wf == wl) return;   // written by its one share
        const int rt = row / RT, lr = row % RT;
        auto piece = [&](int w) { return part + (((long)w * 2 + (w == wf ? 1 : 0)) * ntile + rt) * RT * (R + 1); };
        for (int w = wf; w <= wl; ++w) {
            if (w > wf && w * total / shares == (w + 1) * total / shares) continue;   // a share without a tile
            lg = fmaxf(lg, piece(w)[RT * R + lr]);
        }
        if (lg != -INFINITY)
            for (int w = wf; w <= wl; ++w) {
                if (w > wf && w * total / shares == (w + 1) * total / shares) continue;
                const float *p = piece(w);
                const float f = exp2_hw(p[RT * R + lr] - lg);
                ls += f;
#pragma unroll
                for (int i = 0; i < PER; i += 4) {
                    const f32x4 v = *reinterpret_cast<const f32x4 *>(p + (long)lr * R + i * 64 + lane * 4);
#pragma unroll
                    for (int e = 0; e < 4; ++e) sum[i + e] += f * v[e];
                }
            }
    }
    const float inv = ls > 0.f ? 1.f / ls : 0.f;
    T *o = (T *)a.o + ((long)n * rows + row) * R;
#pragma unroll
    for (int i = 0; i < PER; i += 4)
        store4(o + i * 64 + lane * 4, f32x4{sum[i], sum[i + 1], sum[i + 2], sum[i + 3]} * inv);
    if (a.lse && lane == 0)
        a.lse[(long)n * rows + row] = ls > 0.f ? (lg + __builtin_amdgcn_logf(ls)) * LN2 : -INFINITY;
}

template <typename T, int R, int NRG>
static hipError_t step_launch(const LatentStepArgs &a, hipStream_t st)
{
    typedef StepCfg<T, R, NRG> C;
    const int rows = a.M * a.H, ntile = (rows + C::RT - 1) / C::RT, shares = step_shares(ntile);
    auto k = latent_step_kernel<T, R, NRG>;
    const hipError_t e = hipFuncSetAttribute((const void *)k, hipFuncAttributeMaxDynamicSharedMemorySize, C::BYTES);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k, dim3(ntile * shares), dim3(C::NTHR), C::BYTES, st, a, ntile, shares);
    hipLaunchKernelGGL((latent_join_kernel<T, R>), dim3(a.N * ((rows + 3) / 4)), dim3(256), 0, st, a, ntile, shares, C::RT);
    return hipGetLastError();
}

hipError_t latent_step_launch(bool bf16, int r, const LatentStepArgs &a, hipStream_t st)
{
    const int rt = step_rt(bf16, a.M * a.H);
    if (!bf16) return r == 512 ? step_launch<float, 512, 1>(a, st) : step_launch<float, 256, 1>(a, st);
    if (r == 512)
        return rt == 16 ? step_launch<__bf16, 512, 1>(a, st) : rt == 32 ? step_launch<__bf16, 512, 2>(a, st)
                                                                       : step_launch<__bf16, 512, 4>(a, st);
    return rt == 16 ? step_launch<__bf16, 256, 1>(a, st) : rt == 32 ? step_launch<__bf16, 256, 2>(a, st)
                                                                   : step_launch<__bf16, 256, 4>(a, st);
}

unsigned long long latent_step_workspace(bool bf16, int N, int M, int H, int r)
{
    const int rt = step_rt(bf16, M * H), ntile = (M * H + rt - 1) / rt;
    return (unsigned long long)StepWs(N, ntile, rt, r).bytes;
}

} // namespace gdn
