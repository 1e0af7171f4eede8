// attn.h -- arguments and shared device helpers of the grouped-attention kernels
// (gfx950): attn_prologue.hip, attn_fwd.hip, attn_bwd.hip, attn_cache.hip.
#pragma once
#include "attn_plan.h"
#include "latent.h"

namespace gdn {

struct AttnPrologueArgs {
    const void *q_raw, *k_raw;
    const float *w_q, *w_k, *inv_freq;
    const int *pos;
    void *q, *k;                 // forward: outputs; backward: gradients of them (inputs)
    void *dq_raw, *dk_raw;
    float *dw_q, *dw_k;
    float *ws;
    long q_stride, k_stride;     // elements from token to token
    long dq_stride, dk_stride;
    float eps;
    int T, Hq, Hk, R;
};

struct AttnArgs {
    const void *q, *k, *v;
    const int *cu_q, *cu_k;
    void *o;
    float *lse;
    const void *d_o;
    void *dq, *dk, *dv;
    void *ws;
    long qs, ks, vs;             // elements from token to token
    long dqs, dks, dvs;
    float scale;
    int B, Tq, Tk, Hk, G;
    unsigned g_mul;              // r / G = r g_mul >> g_shift for r < 2^30 (set by the launcher)
    int g_shift;
    unsigned g_mul16;            // r / G = r g_mul16 >> 16 for r < 256
};

struct AttnCacheArgs {
    const void *q, *k, *v;
    void *k_cache, *v_cache;
    float *k_scale, *v_scale;
    const int *table, *lens, *cu;
    void *o;
    float *lse;
    void *ws;
    long qs, ks, vs;             // elements from token to token
    float scale;
    int N, T, Hk, G;
    int pages, page, width;
    unsigned bpp_mul;            // block / (page / 16) (set by the launcher)
    int bpp_shift;
};

hipError_t attn_prologue_launch(bool bf16, int D, const AttnPrologueArgs &a, hipStream_t st);
hipError_t attn_prologue_bwd_launch(bool bf16, int D, const AttnPrologueArgs &a, hipStream_t st);
unsigned long long attn_prologue_bwd_workspace(int T, int Hq, int D);
hipError_t attn_fwd_launch(bool bf16, int D, const AttnArgs &a, hipStream_t st);
unsigned long long attn_fwd_workspace(bool bf16, int B, int Tq, int Tk, int Hk, int G, int D);
hipError_t attn_bwd_launch(bool bf16, int D, const AttnArgs &a, hipStream_t st);
unsigned long long attn_bwd_workspace(bool bf16, int B, int Tq, int Tk, int Hk, int G, int D);
hipError_t attn_append_launch(bool bf16, int D, const AttnCacheArgs &a, hipStream_t st);
hipError_t attn_step_launch(bool bf16, int D, const AttnCacheArgs &a, hipStream_t st);
unsigned long long attn_step_workspace(int N, int Hk, int G, int D, int page, int width);

// x / d = x mul >> shift for 0 <= x < 2^30, 1 <= d < 2^15: with shift = 30 + s, 2^s >= d
// the smallest, the error x (mul d - 2^shift) / (d 2^shift) is below 1 / d.
inline void divisor(int d, unsigned &mul, int &shift) {
    int s = 0;
    while ((1 << s) < d) ++s;
    shift = 30 + s;
    mul = (unsigned)(((1ULL << shift) + d - 1) / d);
}

#ifdef __HIPCC__
__device__ __forceinline__ int quotient(int x, unsigned mul, int shift) {
    return (int)((unsigned long long)(unsigned)x * mul >> shift);
}

// Where sequence b stands in the packed rows, in scalar registers.  Offsets that are no
// rising numbers within the tensor give wrong lengths but never rows outside of it.
struct Seq {
    int q0, lq, k0, lk;
};
__device__ __forceinline__ int within(int x, int n) { return x < 0 ? 0 : x > n ? n : x; }
__device__ __forceinline__ Seq seq_lane(const AttnArgs &a, int b) {   // b may differ by lane
    Seq s;
    s.q0 = within(a.cu_q[b], a.Tq);
    s.lq = max(0, within(a.cu_q[b + 1], a.Tq) - s.q0);
    if (a.cu_k) {
        s.k0 = within(a.cu_k[b], a.Tk);
        s.lk = max(0, within(a.cu_k[b + 1], a.Tk) - s.k0);
    } else {   // Tk = Tq
        s.k0 = s.q0;
        s.lk = s.lq;
    }
    return s;
}
__device__ __forceinline__ Seq seq_of(const AttnArgs &a, int b) {
    Seq s = seq_lane(a, b);
    s.q0 = __builtin_amdgcn_readfirstlane(s.q0);
    s.lq = __builtin_amdgcn_readfirstlane(s.lq);
    s.k0 = __builtin_amdgcn_readfirstlane(s.k0);
    s.lk = __builtin_amdgcn_readfirstlane(s.lk);
    return s;
}

// Over the lanes of a wave, by shifts within rows of 16 lanes: the sums up to each lane,
// the sum, and the maximum of values that are not negative.
template <int CTRL> __device__ __forceinline__ int row_shift(int x) {
    return __builtin_amdgcn_update_dpp(0, x, CTRL, 0xf, 0xf, true);   // zeros from outside
}
__device__ __forceinline__ int row_scan(int x) {
    x += row_shift<0x111>(x);
    x += row_shift<0x112>(x);
    x += row_shift<0x114>(x);
    return x + row_shift<0x118>(x);
}
__device__ __forceinline__ int scan_lanes(int x) {
    x = row_scan(x);
    const int a = __builtin_amdgcn_readlane(x, 15), b = a + __builtin_amdgcn_readlane(x, 31);
    const int c = b + __builtin_amdgcn_readlane(x, 47), row = (threadIdx.x & 63) >> 4;
    return x + (row == 0 ? 0 : row == 1 ? a : row == 2 ? b : c);
}
__device__ __forceinline__ int sum_lanes(int x) {
    x = row_scan(x);
    return __builtin_amdgcn_readlane(x, 15) + __builtin_amdgcn_readlane(x, 31) + __builtin_amdgcn_readlane(x, 47) + __builtin_amdgcn_readlane(x, 63);
}
__device__ __forceinline__ int max_lanes(int x) {
    x = max(x, row_shift<0x111>(x));
    x = max(x, row_shift<0x112>(x));
    x = max(x, row_shift<0x114>(x));
    x = max(x, row_shift<0x118>(x));
    return max(max(__builtin_amdgcn_readlane(x, 15), __builtin_amdgcn_readlane(x, 31)),
               max(__builtin_amdgcn_readlane(x, 47), __builtin_amdgcn_readlane(x, 63)));
}

// x, which every lane of the wave has, in a scalar register.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// Item w of a list to which sequence b gives count(b) items: the sequence and the item's
// number within it; -1 where the list is shorter.  Every lane of the wave calls it.
struct Item {
    int b, i;
};
template <typename F> __device__ __forceinline__ Item find_item(int B, int w, F count)
{
    const int lane = threadIdx.x & 63;
    int at = 0;
    for (int b = 0; b < B; b += 64) {
        const int mine = b + lane < B ? count(b + lane) : 0, incl = scan_lanes(mine);
        const int sum = __builtin_amdgcn_readlane(incl, 63);
        if (w < at + sum) {
            const int l = (int)__builtin_ctzll(__ballot(w < at + incl));
            return {b + l, w - at - __builtin_amdgcn_readlane(incl - mine, l)};
        }
        at += sum;
    }
    return {-1, 0};
}

// The last of B sequences with from(b) <= w, for numbers that rise from from(0) <= w on, by
// 64 probes at a time.
template <typename F> __device__ __forceinline__ int find_slot(int B, int w, F from)
{
    const int lane = threadIdx.x & 63;
    int at = 0;
    while (B > 1) {
        const int step = (B + 63) >> 6, b = lane * step;
        const unsigned long long ok = __ballot(b < B && from(at + b) <= w);
        const int l = ok ? 63 - (int)__builtin_clzll(ok) : 0;
        at += l * step;
        B = min(step, B - l * step);
    }
    return uniform(at);
}

// The list of find_item with the last items of all sequences first: item i of every sequence
// stands behind items i + 1 of all of them.  Rows further down a causal sequence have more
// keys, so that the longest work begins first.
template <typename F> __device__ __forceinline__ Item find_last(int B, int w, F count)
{
    const int lane = threadIdx.x & 63;
    const int first = lane < B ? count(lane) : 0;
    auto from = [&](int i) {   // items i and on
        int sum = max(0, first - i);
        for (int b = 64 + lane; b < B; b += 64) sum += max(0, count(b) - i);
        return sum_lanes(sum);
    };
    if (w >= from(0)) return {-1, 0};
    int most = first;
    for (int b = 64 + lane; b < B; b += 64) most = max(most, count(b));
    int lo = 0, hi = max_lanes(most);   // from(lo) > w >= from(hi)
    int behind = 0;                     // from(hi)
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1, n = from(mid);
        if (n > w) lo = mid;
        else hi = mid, behind = n;
    }
    const Item found = find_item(B, w - behind, [&](int b) { return (b < 64 ? first : count(b)) > lo ? 1 : 0; });
    return {found.b, lo};
}

// Row tiles of a sequence: tile t has the tokens from t `per` on.
struct AttnTiles {
    static constexpr int extra = 128;
    int per, off, lq, lk;
    __device__ __forceinline__ AttnTiles(int per, const Seq &s) : per(per), off(s.lk - s.lq), lq(s.lq), lk(s.lk) {}
    __device__ __forceinline__ int count() const { return (lq + per - 1) / per; }
    // keys that the last row of tile t sees
    __device__ __forceinline__ int walk(int t) const { return max(0, off + min((t + 1) * per, lq)); }
    __device__ __forceinline__ int first() const { return off < 0 ? min(-off / per, count()) : 0; }   // tile that sees any
    // keys of the row tiles before t (a tile with keys, or count())
    __device__ __forceinline__ long before(int t) const {
        const int f = first();
        const long n = t - f;
        return n <= 0 ? 0 : n * (off + extra) + (long)per * ((long)t * (t + 1) - (long)f * (f + 1)) / 2;
    }
    __device__ __forceinline__ long all() const {
        const int n = count();
        return n > first() && walk(n - 1) > 0 ? before(n - 1) + walk(n - 1) + extra : 0;
    }
};

// The same of an address.
__device__ __forceinline__ const char *uniform(const void *p) {
    return (const char *)((unsigned)uniform((int)(uintptr_t)p) | (unsigned long long)(unsigned)uniform((int)((uintptr_t)p >> 32)) << 32);
}
// copy16s from an address that a vector instruction may have written last (a readfirstlane,
// or a scalar register that the compiler kept in a vector register's lane): the load reads it
// five wait states after the asm begins.
__device__ __forceinline__ void copy16u(const void *base, unsigned off, const char *lds) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(lds_at(lds)) : "m0");
}

// Operands that a loop holds in registers, there before it begins: the compiler waits for a
// load where its value is first used, and inside of a loop with copies into LDS under way that
// would be a wait for all of them, every time around.
template <typename T> __device__ __forceinline__ void landed(Frag<T> &f) {
    if constexpr (sizeof(T) == 2) asm volatile("" : "+v"(f.v));
    else asm volatile("" : "+v"(f.lo), "+v"(f.hi));
}

// Enqueue the copy of packed rows r0 .. r0 + ROWS - 1 (CPR chunks each, `stride` bytes apart,
// x: row 0) into an LDS tile by 256 threads, tid 0 .. 255; the row and the address may be in
// vector registers, but are the same in every lane.  Rows from n on read as zeros.
template <int CPR, int ROWS> __device__ __forceinline__ void load_tile(char *tile, const char *x, long stride, int r0, int n, int tid)
{
    constexpr int RP = 256 / CPR;
    static_assert(RP % 8 == 0 && ROWS % RP == 0, "");
    const char *p = uniform(x + r0 * stride), *dst = tile + uniform(tid >> 6) * 1024;
    const int row = tid / CPR, left = uniform(n - r0);
#pragma unroll
    for (int i = 0; i < ROWS / RP; ++i) {
        const int ch = ((tid % CPR) ^ swz<CPR>(i * RP + row)) * 16;   // the same for all i, but for row bit 3 where RP is 8
        if (left >= ROWS) copy16u(p + i * RP * stride, (unsigned)(row * (int)stride + ch), dst + i * 4096);
        else copy16(i * RP + row < left ? p + (i * RP + row) * stride + ch : (const char *)latent_zero, dst + i * 4096);
    }
}

// Row tile w of a call's `most`, -1 where there are fewer.  Up to 64 sequences, the tiles with
// the most keys first.  Beyond, where that search would take longer than the tile: tile t of
// sequence b is number cu_q[b] / per + b + t, which leaves gaps, from the last one down.
__device__ __forceinline__ Item find_tile(const AttnArgs &a, int per, int w, int most)
{
    if (a.B <= 64) return find_last(a.B, w, [&](int b) { return AttnTiles(per, seq_lane(a, b)).count(); });
    auto from = [&](int b) { return within(a.cu_q[b], a.Tq) / per + b; };
    const int b = find_slot(a.B, most - 1 - w, from), t = most - 1 - w - from(b);
    return {t >= 0 && t < AttnTiles(per, seq_lane(a, b)).count() ? b : -1, t};
}

// Shares: calls of few owners (row tiles, key tiles) with long walks are cut over a fixed
// number of workgroups, each of which takes an equal run of all that the owners walk by
// (sequence by sequence, head by head, owner by owner), in units of keys or rows.  From that
// follow whole tiles of UT units: those that begin in the run.  `make(seq)` gives a sequence's
// owners of one key head: count(), first() with any work, walk(i), before(i), all().  To the
// walk of an owner belong `extra` units without a tile, as long as a change of owners takes
// (its operands' loads, its results' stores): shares of many short walks would else take
// longer than those of one long walk.
struct Run {   // what a workgroup works on at a time: tiles j .. end of the n of owner t
    int b, h, t, j, end, n;
    Seq s;
};
struct Share {
    Run r;
    long left;   // units of the share behind r
    int x;       // first unit of owner r.t behind r
};
__device__ __forceinline__ long lane_of(long x, int l) {
    const unsigned lo = (unsigned)__builtin_amdgcn_readlane((int)x, l), hi = (unsigned)__builtin_amdgcn_readlane((int)(x >> 32), l);
    return (long)((unsigned long long)hi << 32 | lo);
}

template <int CTRL> __device__ __forceinline__ long row_shift(long x) {
    return (long)((unsigned long long)(unsigned)row_shift<CTRL>((int)(x >> 32)) << 32 | (unsigned)row_shift<CTRL>((int)x));
}
__device__ __forceinline__ long scan_lanes(long x) {
    x += row_shift<0x111>(x);
    x += row_shift<0x112>(x);
    x += row_shift<0x114>(x);
    x += row_shift<0x118>(x);
    const long a = lane_of(x, 15), b = a + lane_of(x, 31), c = b + lane_of(x, 47);
    const int row = (threadIdx.x & 63) >> 4;
    return x + (row == 0 ? 0 : row == 1 ? a : row == 2 ? b : c);
}

// Units of a share: all of the call's over the shares, rounded up; `least` tiles or more.
template <int UT> __device__ __forceinline__ long share_each(long total, int shares, int least) {
    return max((long)least * UT, (total + shares - 1) / shares);
}

// The next run that has a tile; false: none.
template <int UT, typename M> __device__ __forceinline__ bool share_next(const AttnArgs &a, M make, Share &sh)
{
    Run &r = sh.r;
    for (;;) {
        if (sh.left <= 0) return false;
        const auto owners = make(r.s);
        const int walk = r.t < owners.count() ? owners.walk(r.t) : 0, size = walk > 0 ? walk + owners.extra : 0;
        if (sh.x < size) {
            const int n = (int)min(sh.left, (long)(size - sh.x));
            r.n = uniform((walk + UT - 1) / UT);
            r.j = uniform((sh.x + UT - 1) / UT);
            r.end = uniform(min((sh.x + n + UT - 1) / UT, r.n));
            sh.x += n;
            sh.left -= n;
            if (r.j < r.end) {
                r.t = uniform(r.t);
                return true;
            }
        } else {
            sh.x = 0;
            if (r.t + 1 < owners.count()) {
                ++r.t;
            } else if (r.h + 1 < a.Hk && owners.all() > 0) {
                ++r.h;
                r.t = owners.first();
            } else {
                if (r.b + 1 >= a.B) return false;
                r.s = seq_of(a, ++r.b);
                r.h = 0;
                r.t = make(r.s).first();
            }
        }
    }
}

// A share's begin; false: it has none.  Every wave adds up all sequences on its own; the
// first share leaves the units before each, and all of them, in prefix[B + 1] for the join.
template <int UT, typename M> __device__ __forceinline__ bool share_begin(const AttnArgs &a, M make, int share, int shares, int least, long *prefix, Share &sh)
{
    const int lane = threadIdx.x & 63;
    auto of = [&](int b) { return b < a.B ? a.Hk * make(seq_lane(a, b)).all() : 0L; };
    long total = 0, mine = 0, incl = 0;
    for (int b = 0; b < a.B; b += 64) {
        mine = of(b + lane);
        incl = scan_lanes(mine);
        if (share == 0 && b + lane < a.B) prefix[b + lane] = total + incl - mine;
        total += lane_of(incl, 63);
    }
    if (share == 0 && lane == 0) prefix[a.B] = total;
    const long each = share_each<UT>(total, shares, least), g0 = share * each;
    if (g0 >= total) return false;
    long at = 0;
    sh.r.b = 0;
    for (int b = 0; b < a.B; b += 64) {
        if (a.B > 64) {   // else there are those of before
            mine = of(b + lane);
            incl = scan_lanes(mine);
        }
        const long sum = lane_of(incl, 63);
        if (g0 < at + sum) {
            const int l = (int)__builtin_ctzll(__ballot(g0 < at + incl));
            sh.r.b = b + l;
            at += lane_of(incl - mine, l);
            break;
        }
        at += sum;
    }
    sh.r.s = seq_of(a, sh.r.b);
    const auto owners = make(sh.r.s);
    const long one = owners.all(), r = g0 - at;
    sh.r.h = uniform((int)(r / one));
    const long x = r - sh.r.h * one;
    int lo = owners.first(), hi = owners.count();   // the owner: before(t) <= x < before(t + 1)
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (owners.before(mid) <= x) lo = mid;
        else hi = mid;
    }
    sh.r.t = uniform(lo);
    sh.x = uniform((int)(x - owners.before(lo)));
    sh.left = lane_of(min(each, total - g0), 0);
    return true;
}

// The shares that worked on owner i, whose first unit is unit c0 of the call: the first, and
// the last that a tile begins in.
template <int UT, typename O> __device__ __forceinline__ void share_range(long c0, const O &owners, int i, long each, int &first, int &last) {
    const int walk = owners.walk(i), tiles = (walk + UT - 1) / UT;
    first = (int)(c0 / each);
    last = (int)((c0 + walk + owners.extra - 1) / each);
    while (last > first && (last * each - c0 + UT - 1) / UT >= tiles) --last;
}

// The sequence of a packed query (or key) row: the last one that begins at or before it,
// which the row is behind if it is of none.
__device__ __forceinline__ int seq_at(const int *cu, int B, int T, int row) {
    int b = 0, hi = B;
    while (hi - b > 1) {
        const int mid = (b + hi) >> 1;
        if (within(cu[mid], T) <= row) b = mid;
        else hi = mid;
    }
    return b;
}
#endif

// The parts of a row put together: part p < n has o[place(p)][D] and a weight of
// 2^lse[place(p)], or nothing where that is -infinity, and then o may never have been written.
// D / 4 lanes a row take the parts in turn, or, of few rows with many parts each, a whole
// workgroup of 256 does, in GR = 1024 / D groups that take every GR-th.  Returns whether the
// lane holds the row's sum (the first group does), with the base-2 log of the weights.
template <int D, int GR, typename Place>
__device__ __forceinline__ bool join_parts(const float *o, const float *lse, int n, Place place, f32x4 &sum, float &lg)
{
    constexpr int LPR = D / 4;
    const int at = threadIdx.x % LPR * 4, g = GR > 1 ? threadIdx.x / LPR : 0;
    float top = -INFINITY, ls = 0.f;
#pragma unroll 4
    for (int p = g; p < n; p += GR) top = fmaxf(top, lse[place(p)]);
    sum = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int p = g; p < n; p += GR) {
        const long i = place(p);
        const float x = lse[i], f = exp2_hw(x - top);
        const f32x4 v = *reinterpret_cast<const f32x4 *>(o + i * D + at);
        if (x == -INFINITY) continue;
        ls += f;
        sum += f * v;
    }
    if constexpr (GR > 1) {
        __shared__ float os[GR][D];
        __shared__ float st[2][GR];
        store4(os[g] + at, sum);
        if (at == 0) {
            st[0][g] = top;
            st[1][g] = ls;
        }
        __syncthreads();
        if (g > 0) return false;
        top = -INFINITY;
#pragma unroll
        for (int i = 0; i < GR; ++i) top = fmaxf(top, st[0][i]);
        ls = 0.f;
        sum = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < GR; ++i) {
            if (st[1][i] == 0.f) continue;   // of none of the parts; a sum that is NaN stays
            const float f = exp2_hw(st[0][i] - top);
            ls += f * st[1][i];
            sum += f * *reinterpret_cast<const f32x4 *>(os[i] + at);
        }
    }
    if (ls != 0.f) sum = sum * (1.f / ls);
    lg = ls != 0.f ? top + __builtin_amdgcn_logf(ls) : -INFINITY;
    return true;
}

} // namespace gdn
