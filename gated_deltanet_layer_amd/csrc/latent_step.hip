// latent_step.hip -- absorbed latent attention over a paged cache (gfx950): one
// token a sequence, or M drafted tokens (a tree) a sequence.
//
//   row_j = [c_j (r) | k_j^rope (64)], j over the len_n cached tokens, then the drafts
//   s_ij = scale q_i . row_j,   o_i = sum_j softmax_j(s_ij) c_j
//
// All M * H query rows of a sequence read the same cache rows.  A workgroup takes RT
// of the rows and a run of key tiles; each tile is copied once into LDS and serves as
// keys (all columns) and as values (the first r).  Two kernels, by the rows:
//
//   up to 32 (fp32: tiles of 16)  latent_step_kernel.  Four waves; in the first product
//       they split the tile's keys, in the second the r output columns.  Bound by the
//       cache's bytes: 64 sequences of 4100 tokens, 16 heads, r = 512 (229 MB live) 48 us
//       in the kernel, the rate of a plain copy of such a cache; with join and launches
//       52-63 us.  One sequence of 300: 10 us, a chain of latencies (lengths, page,
//       tile, two products), and 4 us of the join.
//   more (bf16)  latent_step_wide_kernel, 64 rows.  At 64 rows a byte of the cache is
//       worth 122 operations, so the matrix cores, LDS and the copies all near their
//       limits: 16 sequences of 4096 x 32 drafts x 32 heads 147-168 us (0.67-0.77 PFLOP/s,
//       matrix cores 35 % busy), 128 of up to 8192 with 128 heads 310-332 us (2.8-3.0 TB/s; a tile is
//       taken from HBM once and from L2 by the second row tile).  A tile of 32
//       keys takes 3,200 cycles, in which the matrix cores work for 1,100 and the LDS,
//       whose score waves read the whole tile each, for some 1,850 (236 KB).
//
// The runs are equal shares of all key tiles of the batch, whatever the lengths:
// the workgroups add up the tiles of all sequences on their own and each takes
// its share, which may begin and end inside a sequence.  Such pieces go to the
// workspace (normalised, with their log-sum-exp) and a second kernel joins them (4-5 us;
// 12-16 where there are thousands of rows).
#include "latent.h"

namespace gdn {

// Up to 32 rows: four waves divide each tile's keys for the scores and the output
// columns for the second product, every wave for all 16 G rows.  Two tiles of 64 keys
// (72 KB each at r = 512) leave room for one workgroup a unit: one is in use while the
// other arrives, which keeps 72 KB a unit in flight, more than the latency of HBM asks
// for.  fp32: 32 keys, and two of the waves have no slab in the first product (8 x 2000
// tokens, r = 256: 17 us).
template <typename T, int R, int G> struct StepCfg {
    static constexpr int NW = 4, D = R + LATENT_ROPE, RT = 16 * G;
    static constexpr int KT = sizeof(T) == 2 ? 64 : 32;
    static constexpr int NS = KT / 16;                      // 16-key slabs
    static constexpr int CB = R / 16 / NW;                  // 16-column blocks of the output a wave
    static constexpr int ES = (int)sizeof(T), CPR = R * ES / 16, RCPR = LATENT_ROPE * ES / 16;
    static constexpr int OFF_R = KT * CPR * 16;             // a tile: [KT][R] latents, [KT][64] rotary keys
    static constexpr int TILE = OFF_R + KT * RCPR * 16;
    static constexpr int PF = 64 * 8 * ES;                  // an operand of weights: 16 rows, 32 keys
    static constexpr int OFF_P = 2 * TILE;                  // [G][KT / 32] of them
    static constexpr int OFF_MX = OFF_P + G * KT / 32 * PF; // [NS][RT] maxima, then sums
    static constexpr int OFF_KV = OFF_MX + NS * RT * 4;     // [2][KT] bytes: key is there
    static constexpr int OFF_SCAN = OFF_KV + 2 * KT;        // [NW + 2] ints
    static constexpr int BYTES = OFF_SCAN + (NW + 2) * 4;
    static_assert(BYTES <= 160 * 1024, "");
};

// More rows (bf16): 64 a workgroup, four waves for the scores, four for the second
// product; see latent_step_wide_kernel.
template <int R> struct WideCfg {
    static constexpr int D = R + LATENT_ROPE, RT = 64, KT = 32, NB = 4;   // NB tile buffers
    static constexpr int CB = R / 64;
    static constexpr int CPR = R / 8, RCPR = LATENT_ROPE / 8;
    static constexpr int OFF_R = KT * CPR * 16, TILE = OFF_R + KT * RCPR * 16;
    static constexpr int OFF_P = NB * TILE;                 // [2][4] operands of weights, 1 KB each
    static constexpr int OFF_AL = OFF_P + 2 * 4 * 1024;     // [2][64] factors of a raised maximum
    static constexpr int OFF_FIN = OFF_AL + 2 * 64 * 4;     // [2][2][64] sums and maxima of a finished sequence
    static constexpr int OFF_KV = OFF_FIN + 2 * 2 * 64 * 4; // [NB][KT] bytes: key is there
    static constexpr int OFF_ID = OFF_KV + NB * KT;         // [4][4][64] pages, by lane of the copying waves
    static constexpr int OFF_SCAN = OFF_ID + 4 * 4 * 64 * 4;    // [8 + 2] ints
    static constexpr int BYTES = OFF_SCAN + 10 * 4;
    static_assert(BYTES <= 160 * 1024, "");
};

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
// The same of a sequence that is uniform, by a scalar load: waiting for it does not
// wait for copies in flight.
__device__ __forceinline__ int step_len_uniform(const LatentStepArgs &a, int n) {
    const int cap = (int)min((long)a.width * a.page, 0x7fffffffL);
    const int v = ((const __attribute__((address_space(4))) int *)(uintptr_t)a.lens)[__builtin_amdgcn_readfirstlane(n)];
    return v < 0 ? 0 : v > cap ? cap : v;
}
__device__ __forceinline__ int step_tiles(int len, int drafts, int kt) { return (len + drafts + kt - 1) / kt; }

// A key tile: tile t of the nkt of sequence n, whose cached length is len.
struct StepPos {
    int n, t, len, nkt;
};

// The tile after p; called only while one is left.
template <int KT> __device__ __forceinline__ StepPos step_after(const LatentStepArgs &a, StepPos p)
{
    if (++p.t == p.nkt) {
        p.t = 0;
        do {
            ++p.n;
            p.len = step_len_uniform(a, p.n);
            p.nkt = step_tiles(p.len, a.drafts, KT);
        } while (p.nkt == 0 && p.n + 1 < a.N);
    }
    return p;
}

// This workgroup's share [g0, g1) of all key tiles and its first tile; false if it
// has none.  Every thread adds up the tiles of a run of sequences, then a scan over
// the workgroup; `first` also writes the tiles before each sequence for the join.
// scan: [NW + 2] ints of LDS.
template <int NW, int KT>
__device__ __forceinline__ bool step_share(const LatentStepArgs &a, int share, int max_shares, bool first, int *scan,
                                           int &g0, int &g1, StepPos &cur)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int per = (a.N + 64 * NW - 1) / (64 * NW), s0 = min(a.N, tid * per), s1 = min(a.N, s0 + per);
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
    if (first) {
        int *prefix = (int *)a.ws, at = incl - mine;
        for (int n = s0; n < s1; ++n) {
            prefix[n] = at;
            at += step_tiles(step_len(a, n), a.drafts, KT);
        }
        if (tid == 0) prefix[a.N] = total;
    }
    if (share >= shares) return false;
    g0 = (int)((long)share * total / shares);
    g1 = (int)((long)(share + 1) * total / shares);
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
    cur.n = __builtin_amdgcn_readfirstlane(scan[NW]);
    cur.t = __builtin_amdgcn_readfirstlane(scan[NW + 1]);
    cur.len = step_len_uniform(a, cur.n);
    cur.nkt = step_tiles(cur.len, a.drafts, KT);
    return true;
}

__device__ __forceinline__ int step_page(const LatentStepArgs &a, int t) {
    return (int)(((unsigned long long)(unsigned)t * a.page_mul) >> a.page_shift);
}

// Row of key `key` of p's sequence (latent_zero: it is not there); id: its page.
template <int ROWB>
__device__ __forceinline__ const char *step_row(const LatentStepArgs &a, const StepPos &p, int key, int id)
{
    const bool cached = key < p.len;
    const bool there = cached ? id >= 0 && id < a.pages : key - p.len < a.drafts;   // any other page holds nothing
    const long slot = (long)id * a.page + (key - step_page(a, key) * a.page), node = (long)p.n * a.M + (key - p.len);
    const char *src = cached ? (const char *)a.cache + slot * ROWB : (const char *)a.draft + node * ROWB;
    return there ? src : (const char *)latent_zero;
}

// -inf where the row does not see the key: s of keys first .. first + 3, `there` their
// flags, bit: the drafts that the row sees.  Without branches: the compiler has lost
// the masked value of a vector element that two nested ones decide.
__device__ __forceinline__ f32x4 step_mask(f32x4 s, unsigned there, int first, int len, unsigned long long bit)
{
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int d = first + e - len;
        const unsigned in = d < 0 ? 1u : (unsigned)(bit >> (d & 63));
        s[e] = (in & (there >> (8 * e)) & 1u) ? s[e] : -INFINITY;
    }
    return s;
}

// A draft that a row does not see has the weight 0 in it, and 0 times a NaN or an
// infinity (a batch of trees padded with drafts that hold anything) is a NaN: rows
// from .. to - 1 of a tile are made finite between the two products, by each wave for
// the columns that it alone multiplies, chunks ch0 .. ch0 + NCH - 1.  A row that sees
// such a draft has its NaN from the score.
template <typename T, int CPR, int NCH> __device__ __forceinline__ void step_finite(char *tile, int from, int to, int ch0)
{
    const unsigned top = sizeof(T) == 2 ? 0x7f80u : 0x7f800000u;   // an exponent of ones
    for (int i = from * NCH + (threadIdx.x & 63); i < to * NCH; i += 64) {
        const int row = i / NCH;
        u32x4 *at = reinterpret_cast<u32x4 *>(tile + row * (CPR * 16) + (((ch0 + i % NCH) ^ swz<CPR>(row)) << 4));
        u32x4 v = *at;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (sizeof(T) == 2) {
                v[e] &= (v[e] & top) == top ? 0xffff0000u : ~0u;
                v[e] &= (v[e] >> 16 & top) == top ? 0x0000ffffu : ~0u;
            } else {
                v[e] = (v[e] & top) == top ? 0u : v[e];
            }
        }
        *at = v;
    }
    asm volatile("" ::: "memory");
}

// The drafts that query row `row` of sequence n sees.
__device__ __forceinline__ unsigned long long step_bits(const LatentStepArgs &a, int n, int row, bool live)
{
    if (!live || !a.drafts) return 0ull;
    const int node = row / a.H;
    if (a.tree) return (unsigned long long)a.tree[(long)n * a.M + node];
    return node >= 63 ? ~0ull : (2ull << node) - 1;
}

template <typename T, int R, int G>
__global__ __launch_bounds__(256, 1) void latent_step_kernel(LatentStepArgs a, int ntile, int max_shares)
{
    typedef StepCfg<T, R, G> C;
    constexpr int D = C::D, KT = C::KT, RT = C::RT, NKB = D / 32, NS = C::NS, CPR = C::CPR, CB = C::CB, NW = C::NW;
    extern __shared__ char lds[];
    const int share = blockIdx.x % max_shares, rt = blockIdx.x / max_shares;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), r16 = lane_r16(), gq = lane_gq();
    const int rows = a.M * a.H;
    const float c = a.scale * LOG2E;
    float *part = (float *)((char *)a.ws + StepWs(a.N, ntile, RT, R).part);
    int g0, g1;
    StepPos cur, nxt;
    if (!step_share<NW, KT>(a, share, max_shares, share == 0 && rt == 0, (int *)(lds + C::OFF_SCAN), g0, g1, cur)) return;

    // The wave copies WR rows of a tile; its lanes look up one each (lanes beyond
    // WR repeat them): page() the page of the lane's row, a tile ahead of its use,
    // load_tile() the copies into buffer `buf`.
    constexpr int WR = KT / NW;
    const int krow = wave * WR + (lane & (WR - 1));
    auto page = [&](const StepPos &p) {
        const int key = p.t * KT + krow;
        return key < p.len ? a.table[(long)p.n * a.width + step_page(a, key)] : -1;
    };
    auto load_tile = [&](const StepPos &p, int id, int buf) {
        const int key = p.t * KT + krow;
        const char *src = step_row<D * C::ES>(a, p, key, id);
        if (lane < WR) lds[C::OFF_KV + buf * KT + krow] = src != (const char *)latent_zero;
        const int lo = (int)(uintptr_t)src, hi = (int)((uintptr_t)src >> 32);
        auto row_ptr = [&](int row) {   // of a row that differs by lane
            return (const char *)(((uintptr_t)(unsigned)__shfl(hi, row, 64) << 32) | (unsigned)__shfl(lo, row, 64));
        };
        char *dst = lds + buf * C::TILE + wave * WR * CPR * 16;
        if constexpr (CPR >= 64) {   // a row is whole instructions: its address is uniform
            static_assert(WR % 8 == 0, "");
#pragma unroll
            for (int i0 = 0; i0 < WR; i0 += 8) {
                unsigned long long q[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) q[i] = lane_address(src, i0 + i);
                settle(q);
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int k = 0; k < CPR / 64; ++k)
                        copy16s((const char *)(uintptr_t)q[i], (unsigned)((k * 64 + (lane ^ swz<CPR>(wave * WR + i0 + i))) * 16),
                                dst + ((i0 + i) * CPR / 64 + k) * 1024);
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
            g2lds16(row_ptr(row) + R * C::ES + ch * 16, rdst + i * 1024);
        }
    };

    // lane parts of the LDS addresses; first product: this wave's slab of keys
    const int nb = row_base<T, CPR>(16 * wave + r16), rb = row_base<T, C::RCPR>(16 * wave + r16);
    // second product: this wave's first 16-column block, as a part inside 256 bytes
    // and whole ones
    constexpr int PC = 16 / C::ES;
    static_assert(CB % PC == 0 || PC % CB == 0, "");
    const int col0 = wave * CB;
    const int vb = col_base<T, CPR>(4 * gq) ^ (col0 % PC * 16 * C::ES), vcol = col0 / PC * 256;
    constexpr int MMAS = C::ES == 2 ? 1 : 8;   // instructions of one mma
    Frag<T> qf[G][NKB];
    unsigned long long bits[G];
    f32x4 acc[CB][G];
    float m[G], l[G];
    int buf = 0, kt0 = cur.t, idn = page(cur);
    bool fresh = true;
    load_tile(cur, idn, 0);
    if (g0 + 1 < g1) {
        nxt = step_after<KT>(a, cur);
        idn = page(nxt);
    }
    for (int g = g0;; ++g, buf ^= 1) {
        if (fresh) {
#pragma unroll
            for (int rg = 0; rg < G; ++rg) {
                const int row = rt * RT + 16 * rg + r16;
                const bool live = row < rows;
                const T *q = (const T *)a.q + ((long)cur.n * rows + (live ? row : 0)) * D;
#pragma unroll
                for (int kb = 0; kb < NKB; ++kb)
                    qf[rg][kb] = live ? load_frag<T>(q + 32 * kb + 8 * gq) : zero_frag<T>();
                bits[rg] = step_bits(a, cur.n, row, live);
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
        if (g + 2 < g1) aft = step_after<KT>(a, nxt);
        // the pages arrived with the tile: nothing of their use moves up to where it would
        // wait for them, and with them for every copy in flight
        asm volatile("" : "+v"(idn));
        if (more) load_tile(nxt, idn, buf ^ 1);
        if (g + 2 < g1) idn = page(aft);

        const char *tile = lds + buf * C::TILE, *there4 = lds + C::OFF_KV + buf * KT + 16 * wave + 4 * gq;
        const int key = cur.t * KT + 16 * wave + 4 * gq;   // first of this lane's four, in the first slab
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
            pipeline<8, NKB * C::ES / 2, NKB * G * MMAS, C::ES / 2, G * MMAS>();
            const unsigned there = *reinterpret_cast<const unsigned *>(there4);
            if (__any(there != 0x01010101u || key + 3 >= cur.len)) {
#pragma unroll
                for (int rg = 0; rg < G; ++rg) s[rg] = step_mask(s[rg], there, key, cur.len, bits[rg]);
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
        if (a.drafts && (cur.t + 1) * KT > cur.len)
            step_finite<T, CPR, CB * 16 / PC>(lds + buf * C::TILE, max(0, cur.len - cur.t * KT),
                                              min(KT, cur.len + a.drafts - cur.t * KT), col0 * 16 / PC);
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
            constexpr int RD = C::ES == 2 ? 2 : 8;   // LDS reads of an operand across the rows
            pipeline<G * C::ES / 2 + 4 * RD, G * C::ES / 2 + CB * RD, CB * G * MMAS, RD, G * MMAS>();
        }
        if (!more || nxt.n != cur.n) {
            // the sequence's (or the share's) last tile: the rows' sums, then write
            float ls[G];
#pragma unroll
            for (int rg = 0; rg < G; ++rg) ls[rg] = rows_sum(l[rg]);
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
            const bool whole = kt0 == 0 && cur.t + 1 == cur.nkt;
            const long slot = ((long)share * 2 + (kt0 == 0 ? 1 : 0)) * ntile + rt;
            float *po = part + slot * RT * (R + 1), *pl = po + RT * R;
#pragma unroll
            for (int rg = 0; rg < G; ++rg) {
                const int lr = 16 * rg + r16, row = rt * RT + lr;
                const bool seen = ls[rg] != 0.f;   // a NaN shows
                const float inv = seen ? 1.f / ls[rg] : 0.f;
                const float lg = seen ? m[rg] * c + __builtin_amdgcn_logf(ls[rg]) : -INFINITY;
                if (row >= rows) continue;
                T *o = (T *)a.o + ((long)cur.n * rows + row) * R + 16 * wave * CB + 4 * gq;
                float *w = po + (long)lr * R + 16 * wave * CB + 4 * gq;
#pragma unroll
                for (int cb = 0; cb < CB; ++cb) {
                    const f32x4 v = seen ? acc[cb][rg] * inv : f32x4{0.f, 0.f, 0.f, 0.f};
                    if (whole) store4(o + 16 * cb, v);
                    else store4(w + 16 * cb, v);
                }
                if (gq == 0 && wave == 0) {
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

// 64 rows of a sequence.  Four waves hold the queries of 16 rows each and compute
// the scores and weights of a tile of 32 keys; four waves hold 64 rows by a quarter
// of the output columns and multiply the weights with the values, a tile behind.  So
// neither needs more registers than two waves a SIMD have, and the matrix cores of
// each SIMD get the products of one kind while the other's wave works on its softmax
// or, the second kind, on the copies of the tiles to come.  Weights change hands as
// whole operands, a lane's own eight values.  With waves that did both products for
// 16 rows each the trees above took 209 us, with the copies before the products 186.
template <int R>
__global__ __launch_bounds__(512, 1) void latent_step_wide_kernel(LatentStepArgs a, int ntile, int max_shares)
{
    typedef __bf16 T;
    typedef WideCfg<R> C;
    constexpr int D = C::D, KT = C::KT, RT = C::RT, NKB = D / 32, CPR = C::CPR, CB = C::CB, NB = C::NB;
    constexpr int WR = KT / 4;                 // rows of a tile that one of the copying waves copies
    constexpr int NV = WR * CPR / 64 + 2;      // its copies a step: latents, rotary keys, pages
    extern __shared__ char lds[];
    const int share = blockIdx.x % max_shares, rt = blockIdx.x / max_shares;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), r16 = lane_r16(), gq = lane_gq();
    const int rows = a.M * a.H;
    const float c = a.scale * LOG2E;
    float *part = (float *)((char *)a.ws + StepWs(a.N, ntile, RT, R).part);
    int g0, g1;
    StepPos pos;
    if (!step_share<8, KT>(a, share, max_shares, share == 0 && rt == 0, (int *)(lds + C::OFF_SCAN), g0, g1, pos)) return;
    const int nt = g1 - g0;
    float *alpha = (float *)(lds + C::OFF_AL), *fin = (float *)(lds + C::OFF_FIN);

    if (wave < 4) {
        const int row = rt * RT + wave * 16 + r16;
        const bool live = row < rows;
        const int nb = row_base<T, CPR>(r16), rb = row_base<T, C::RCPR>(r16);
        Frag<T> qf[NKB];
        unsigned long long bits = 0;
        float m = -INFINITY, l = 0.f;
        int n = -1;
        StepPos p = pos;
        for (int i = 0;; ++i) {
            lds_barrier();   // tile i is there
            if (i == nt) break;
            if (p.n != n) {   // another sequence
                n = p.n;
                const T *q = (const T *)a.q + ((long)n * rows + (live ? row : 0)) * D;
#pragma unroll
                for (int kb = 0; kb < NKB; ++kb) qf[kb] = live ? load_frag<T>(q + 32 * kb + 8 * gq) : zero_frag<T>();
                bits = step_bits(a, n, row, live);
                m = -INFINITY;
                l = 0.f;
            }
            const char *tile = lds + i % NB * C::TILE;
            f32x4 s[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) s[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb)
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const Frag<T> kf = kb < R / 32 ? row_frag<T>(tile + 16 * t * CPR * 16, nb, kb)
                                                   : row_frag<T>(tile + C::OFF_R + 16 * t * C::RCPR * 16, rb, kb - R / 32);
                    s[t] = mma(s[t], kf, qf[kb]);
                }
            pipeline<12, 2 * NKB, 2 * NKB, 2, 2>();
            const int key = p.t * KT + 4 * gq;
            const char *there4 = lds + C::OFF_KV + i % NB * KT + 4 * gq;
            const unsigned th0 = *reinterpret_cast<const unsigned *>(there4), th1 = *reinterpret_cast<const unsigned *>(there4 + 16);
            if (__any((th0 & th1) != 0x01010101u || key + 19 >= p.len)) {
                s[0] = step_mask(s[0], th0, key, p.len, bits);
                s[1] = step_mask(s[1], th1, key + 16, p.len, bits);
            }
            float mx = -INFINITY;
#pragma unroll
            for (int e = 0; e < 4; ++e) mx = fmaxf(mx, fmaxf(s[0][e], s[1][e]));
            mx = rows_max(mx);
            const bool up = (mx - m) * c > RAISE;   // false while both are -inf
            const float mn = up ? mx : m, al = up ? exp2_hw((m - mn) * c) : 1.f;
            m = mn;
            l *= al;
            if (gq == 0) alpha[(i & 1) * 64 + wave * 16 + r16] = al;
            const float mb = m == -INFINITY ? 0.f : m * c;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[t][e] = exp2_hw(__builtin_fmaf(s[t][e], c, -mb));
                    l += s[t][e];
                }
            const Frag<T> pf = reg_frag<T>(s[0], s[1]);
            *reinterpret_cast<bf16x8 *>(lds + C::OFF_P + ((i & 1) * 4 + wave) * 1024 + lane * 16) = pf.v;
            if (i + 1 == nt || p.t + 1 == p.nkt) {   // the sequence's (or the share's) last tile
                const float ls = rows_sum(l);
                if (gq == 0) {
                    fin[(i & 1) * 128 + wave * 16 + r16] = ls;
                    fin[(i & 1) * 128 + 64 + wave * 16 + r16] = m * c;
                }
            }
            if (i + 1 < nt) p = step_after<KT>(a, p);
        }
    } else {
        const int w = wave - 4, col0 = w * CB;   // 16-column blocks of this wave

        // The copies.  Tile i (counted from g0) stands in buffer i % NB.  Step i enqueues
        // tile i + 2; works out the row addresses of i + 3, from pages enqueued two steps
        // before; and enqueues the pages of i + 5.
        // Behind the share's last tile all of this goes to that tile again.  Every step
        // has NV copies a wave, so that all but those of the step before have arrived
        // when NV are left.
        const int krow = w * WR + (lane & (WR - 1));
        const char *ids = lds + C::OFF_ID;   // [4][4 waves][64 lanes]
        constexpr bool WHOLE = CPR == 64;    // a row is one copy: its address is uniform
        const char *row = nullptr;           // of tile i + 2
        auto load_ids = [&](const StepPos &p, int i) {
            const int key = p.t * KT + krow;
            const void *src = key < p.len ? (const void *)(a.table + (long)p.n * a.width + step_page(a, key)) : (const void *)latent_zero;
            copy4(src, ids + (i % 4 * 4 + w) * 256);
        };
        auto page_id = [&](int i) { return *reinterpret_cast<const int *>(ids + (i % 4 * 4 + w) * 256 + lane * 4); };
        auto address = [&](const StepPos &p, int id) { return step_row<D * 2>(a, p, p.t * KT + krow, id); };
        auto of_row = [&](const char *p, int r) {   // of a row that differs by lane
            const int lo = (int)(uintptr_t)p, hi = (int)((uintptr_t)p >> 32);
            return (const char *)(((uintptr_t)(unsigned)__shfl(hi, r, 64) << 32) | (unsigned)__shfl(lo, r, 64));
        };
        auto load_latents = [&](const char *p, int i) {   // as many copies as the wave has column blocks
            char *dst = lds + i % NB * C::TILE + w * WR * CPR * 16;
            if constexpr (WHOLE) {
                unsigned long long b[CB];
#pragma unroll
                for (int k = 0; k < CB; ++k) b[k] = lane_address(p, k);
                settle(b);
#pragma unroll
                for (int k = 0; k < CB; ++k)
                    copy16s((const char *)(uintptr_t)b[k], (unsigned)((lane ^ swz<CPR>(w * WR + k)) * 16), dst + k * 1024);
            } else {
#pragma unroll
                for (int k = 0; k < CB; ++k) {
                    const int r = k * (64 / CPR) + lane / CPR;
                    copy16(of_row(p, r) + ((lane % CPR) ^ swz<CPR>(w * WR + r)) * 16, dst + k * 1024);
                }
            }
        };
        const int rrow = lane / C::RCPR, rch = ((lane % C::RCPR) ^ swz<C::RCPR>(w * WR + rrow)) * 16 + R * 2;
        auto load_rope = [&](const char *p, const char *from, int i) {   // p: the lane's row; from: row rrow
            lds[C::OFF_KV + i % NB * KT + krow] = p != (const char *)latent_zero;   // equal lanes write equal bytes
            copy16(from + rch, lds + i % NB * C::TILE + C::OFF_R + w * WR * C::RCPR * 16);
        };
        static_assert(WR * C::RCPR == 64 && WR * CPR / 64 == CB, "");
        StepPos pa = pos, pi = pos;   // of the tiles whose addresses, and pages, come next
        int na = 0, ni = 0;
        auto advance = [&](StepPos &p, int &n) {
            if (++n < nt) p = step_after<KT>(a, p);
        };
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            load_ids(pi, k);
            advance(pi, ni);
        }
        wait_vm<0>();
        for (int k = 0; k < 2; ++k) {
            const char *r = address(pa, page_id(k));
            load_latents(r, k);
            load_rope(r, of_row(r, rrow), k);
            advance(pa, na);
        }
        row = address(pa, page_id(2));
        advance(pa, na);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the first pages have been read
        load_ids(pi, 4);
        advance(pi, ni);
        wait_vm<0>();

        const int vb = col_base<T, CPR>(4 * gq) ^ (col0 % 8 * 32), vcol = col0 / 8 * 256;
        f32x4 acc[CB][4];
#pragma unroll
        for (int cb = 0; cb < CB; ++cb)
#pragma unroll
            for (int rg = 0; rg < 4; ++rg) acc[cb][rg] = f32x4{0.f, 0.f, 0.f, 0.f};
        StepPos p = pos;   // of the tile before
        int kt0 = pos.t;
        lds_barrier();   // step 0
        load_latents(row, 2);
        load_rope(row, of_row(row, rrow), 2);
        load_ids(pi, 5);
        advance(pi, ni);
        row = address(pa, page_id(3));
        advance(pa, na);
#pragma unroll 1
        for (int i = 1; i <= nt; ++i) {
            wait_vm<NV>();
            lds_barrier();
            const int k = i - 1;
            load_latents(row, i + 2);   // at once: their latency is what a step waits for
            GDN_SCHED_FENCE();
            Frag<T> pf[4];
            float al[4];
            bool up = false;
#pragma unroll
            for (int rg = 0; rg < 4; ++rg) {
                pf[rg] = {*reinterpret_cast<const bf16x8 *>(lds + C::OFF_P + ((k & 1) * 4 + rg) * 1024 + lane * 16)};
                al[rg] = alpha[(k & 1) * 64 + rg * 16 + r16];
                up |= al[rg] != 1.f;
            }
            if (__any(up)) {
#pragma unroll
                for (int cb = 0; cb < CB; ++cb)
#pragma unroll
                    for (int rg = 0; rg < 4; ++rg) acc[cb][rg] *= al[rg];
            }
            const char *tile = lds + k % NB * C::TILE + vcol;
            if (a.drafts && (p.t + 1) * KT > p.len)
                step_finite<T, CPR, CB * 2>(lds + k % NB * C::TILE, max(0, p.len - p.t * KT),
                                            min(KT, p.len + a.drafts - p.t * KT), col0 * 2);
            constexpr int AHEAD = CB < 4 ? CB : 4;   // operands read before their products
            Frag<T> vf[CB];
#pragma unroll
            for (int cb = 0; cb < AHEAD; ++cb) vf[cb] = col_frag<T, CPR>(tile, vb, cb);
            const int id = page_id(i + 3);
            const char *from = of_row(row, rrow), *next = nullptr;
#pragma unroll
            for (int cb = 0; cb < CB; ++cb) {
                GDN_SCHED_FENCE();
                if (cb + AHEAD < CB) vf[cb + AHEAD] = col_frag<T, CPR>(tile, vb, cb + AHEAD);
                if (cb == 0) load_ids(pi, i + 5);
                if (cb == 1) load_rope(row, from, i + 2);
                if (cb == 2) next = address(pa, id);
#pragma unroll
                for (int rg = 0; rg < 4; ++rg) acc[cb][rg] = mma(acc[cb][rg], vf[cb], pf[rg]);
            }
            row = next;
            advance(pi, ni);
            advance(pa, na);
            if (i == nt || p.t + 1 == p.nkt) {
                const bool whole = kt0 == 0 && p.t + 1 == p.nkt;
                const long slot = ((long)share * 2 + (kt0 == 0 ? 1 : 0)) * ntile + rt;
                float *po = part + slot * RT * (R + 1), *pl = po + RT * R;
#pragma unroll
                for (int rg = 0; rg < 4; ++rg) {
                    const int lr = 16 * rg + r16, row = rt * RT + lr;
                    const float ls = fin[(k & 1) * 128 + lr], mc = fin[(k & 1) * 128 + 64 + lr];
                    const bool seen = ls != 0.f;   // a NaN shows
                    const float inv = seen ? 1.f / ls : 0.f;
                    const float lg = seen ? mc + __builtin_amdgcn_logf(ls) : -INFINITY;
                    if (row >= rows) continue;
                    T *o = (T *)a.o + ((long)p.n * rows + row) * R + 16 * col0 + 4 * gq;
                    float *f = po + (long)lr * R + 16 * col0 + 4 * gq;
#pragma unroll
                    for (int cb = 0; cb < CB; ++cb) {
                        const f32x4 v = seen ? acc[cb][rg] * inv : f32x4{0.f, 0.f, 0.f, 0.f};
                        if (whole) store4(o + 16 * cb, v);
                        else store4(f + 16 * cb, v);
                    }
                    if (gq == 0 && w == 0) {
                        if (!whole) pl[lr] = lg;
                        else if (a.lse) a.lse[(long)p.n * rows + row] = lg * LN2;
                    }
                }
#pragma unroll
                for (int cb = 0; cb < CB; ++cb)
#pragma unroll
                    for (int rg = 0; rg < 4; ++rg) acc[cb][rg] = f32x4{0.f, 0.f, 0.f, 0.f};
                kt0 = 0;
            }
            if (i < nt) p = step_after<KT>(a, p);
        }
        wait_vm<0>();   // copies into this LDS end before it is given away
    }
}

// Joins the pieces of every sequence that more than one share worked on, and
// writes the sequences that have no key at all.  WPR waves a row, each with every
// WPR-th piece: four where few rows have many pieces, else one.
template <typename T, int R, int WPR>
__global__ __launch_bounds__(256) void latent_join_kernel(LatentStepArgs a, int ntile, int max_shares, int RT)
{
    constexpr int PER = R / 64;   // columns a lane
    const int rows = a.M * a.H, lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const long at = (long)blockIdx.x * (4 / WPR) + wave / WPR;   // of the N * rows rows
    if (at >= (long)a.N * rows) return;
    const int n = (int)(at / rows), row = (int)(at % rows), w0 = wave % WPR;
    const int *prefix = (const int *)a.ws;
    const int c0 = prefix[n], c1 = prefix[n + 1], total = prefix[a.N], shares = min(max_shares, total);
    int wf = 0, wl = -1;
    if (c1 > c0) {
        wf = (int)(((long)(c0 + 1) * shares - 1) / total);
        wl = (int)(((long)c1 * shares - 1) / total);
        if (wf == wl) return;   // written by its one share (all waves of the row agree)
    }
    // piece w of the sequence: the last of share wf, the first of the others
    const long step = (long)2 * ntile * RT * (R + 1);
    const float *first = (const float *)((const char *)a.ws + StepWs(a.N, ntile, RT, R).part) + (long)(row / RT) * RT * (R + 1);
    const float *last = first + (long)ntile * RT * (R + 1);
    const int lr = row % RT;
    auto piece = [&](int w) { return (w == wf ? last : first) + w * step; };
    float top = -INFINITY;
    for (int w = wf + lane; w <= wl; w += 64) top = fmaxf(top, piece(w)[RT * R + lr]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
    float sum[PER], ls = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) sum[i] = 0.f;
#pragma unroll 4
    for (int w = wf + w0; w <= wl; w += WPR) {
        const float *p = piece(w);
        const float lg = p[RT * R + lr], f = lg == -INFINITY ? 0.f : exp2_hw(lg - top);
        ls += f;
#pragma unroll
        for (int i = 0; i < PER; i += 4) {
            const f32x4 v = *reinterpret_cast<const f32x4 *>(p + (long)lr * R + i * 64 + lane * 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[i + e] += f * v[e];
        }
    }
    if constexpr (WPR > 1) {   // one row a workgroup
        __shared__ float sums[4][R], parts[4];
        if (lane == 0) parts[wave] = ls;
#pragma unroll
        for (int i = 0; i < PER; i += 4)
            *reinterpret_cast<f32x4 *>(&sums[wave][i * 64 + lane * 4]) = f32x4{sum[i], sum[i + 1], sum[i + 2], sum[i + 3]};
        __syncthreads();
        if (wave > 0) return;
        ls = parts[0] + parts[1] + parts[2] + parts[3];
#pragma unroll
        for (int i = 0; i < PER; i += 4)
#pragma unroll
            for (int w = 1; w < 4; ++w) {
                const f32x4 v = *reinterpret_cast<const f32x4 *>(&sums[w][i * 64 + lane * 4]);
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[i + e] += v[e];
            }
    }
    const float inv = ls != 0.f ? 1.f / ls : 0.f;
    T *o = (T *)a.o + at * R;
#pragma unroll
    for (int i = 0; i < PER; i += 4)
        store4(o + i * 64 + lane * 4, f32x4{sum[i], sum[i + 1], sum[i + 2], sum[i + 3]} * inv);
    if (a.lse && lane == 0) a.lse[at] = ls != 0.f ? (top + __builtin_amdgcn_logf(ls)) * LN2 : -INFINITY;
}

template <typename T, int R, typename K>
static hipError_t step_enqueue(K k, int rt, int threads, int lds, const LatentStepArgs &a, hipStream_t st)
{
    const int rows = a.M * a.H, ntile = (rows + rt - 1) / rt, shares = step_shares(ntile);
    const hipError_t e = hipFuncSetAttribute((const void *)k, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k, dim3(ntile * shares), dim3(threads), lds, st, a, ntile, shares);
    // Pieces a sequence: about shares / N.  r = 512, 16 heads: 4 sequences of 2000 tokens
    // 14.9 us with four waves a row, 17.3 with one; 48 of 2000 33.1, 33.4; 64 of 2000 35.5,
    // 35.3; 128 of 2000 63.5, 62.2.
    if (shares > 4 * a.N)
        hipLaunchKernelGGL((latent_join_kernel<T, R, 4>), dim3(a.N * rows), dim3(256), 0, st, a, ntile, shares, rt);
    else
        hipLaunchKernelGGL((latent_join_kernel<T, R, 1>), dim3((a.N * rows + 3) / 4), dim3(256), 0, st, a, ntile, shares, rt);
    return hipGetLastError();
}

template <typename T, int R, int G> static hipError_t step_launch(const LatentStepArgs &a, hipStream_t st)
{
    typedef StepCfg<T, R, G> C;
    return step_enqueue<T, R>(latent_step_kernel<T, R, G>, C::RT, 256, C::BYTES, a, st);
}

template <int R> static hipError_t step_bf16(const LatentStepArgs &a, hipStream_t st)
{
    switch (step_rt(true, a.M * a.H)) {
    case 16: return step_launch<__bf16, R, 1>(a, st);
    case 32: return step_launch<__bf16, R, 2>(a, st);
    default: return step_enqueue<__bf16, R>(latent_step_wide_kernel<R>, WideCfg<R>::RT, 512, WideCfg<R>::BYTES, a, st);
    }
}

hipError_t latent_step_launch(bool bf16, int r, const LatentStepArgs &given, hipStream_t st)
{
    // with L = ceil(log2 page), mul = floor(2^(30 + L) / page) + 1: mul page - 2^(30 + L)
    // is at most 2^L, so t of it stays below 2^(30 + L) and the quotient is exact
    LatentStepArgs a = given;
    int L = 0;
    while ((1LL << L) < a.page) ++L;
    a.page_shift = 30 + L;
    a.page_mul = (unsigned)((1ULL << (30 + L)) / (unsigned)a.page + 1);
    if (!bf16) return r == 512 ? step_launch<float, 512, 1>(a, st) : step_launch<float, 256, 1>(a, st);
    return r == 512 ? step_bf16<512>(a, st) : step_bf16<256>(a, st);
}

unsigned long long latent_step_workspace(bool bf16, int N, int M, int H, int r)
{
    const int rt = step_rt(bf16, M * H), ntile = (M * H + rt - 1) / rt;
    return (unsigned long long)StepWs(N, ntile, rt, r).bytes;
}

} // namespace gdn
