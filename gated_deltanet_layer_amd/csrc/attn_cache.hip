// attn_cache.hip -- the 8-bit paged cache of grouped attention: appending tokens, and one
// token's attention over it (gfx950).
//
// Keys and values are held as e4m3 with one fp32 scale for 16 tokens of a head (a block); a
// page has a whole number of blocks.  A key block is [16 tokens][D], a value block [D][16
// tokens]: the first product contracts over channels, the second over tokens, and both then
// read their operand from memory as it stands, 16 bytes a lane, without passing through LDS.
// Scales are powers of two, so that a block whose scale has to grow for a new token keeps
// what it holds exactly (but for values that fall below e4m3's smallest normal).
#include "attn.h"

namespace gdn {

constexpr int CACHE_BLOCK = 16;

// Block `blk` of sequence n's tokens for head h: its number among all blocks of the cache
// (pages, then heads, then blocks of the page); -1 if the table names no page.
__device__ __forceinline__ int cache_block(const AttnCacheArgs &a, int n, int h, int blk)
{
    const int bpp = a.page / CACHE_BLOCK, p = quotient(blk, a.bpp_mul, a.bpp_shift);
    const int pg = a.table[(long)n * a.width + p];
    return pg >= 0 && pg < a.pages ? (pg * a.Hk + h) * bpp + blk - p * bpp : -1;
}

// New tokens of sequence n, as positions in it: [lo, hi), the first of them row `row` of the
// new ones.
struct Fresh {
    int lo, hi;
    long row;
};
__device__ __forceinline__ Fresh fresh(const AttnCacheArgs &a, int n)
{
    const int at = a.cu ? within(a.cu[n], a.T) : n, count = a.cu ? max(0, within(a.cu[n + 1], a.T) - at) : 1;
    const int len = max(a.lens[n], 0), first = len - count, lo = max(first, 0);
    return {lo, min(len, a.width * a.page), (long)at + (lo - first)};
}
__device__ __forceinline__ int fresh_blocks(const Fresh &f)
{
    return f.hi > f.lo ? (f.hi - 1) / CACHE_BLOCK - f.lo / CACHE_BLOCK + 1 : 0;
}

// The smallest power of two, 2^-126 or more, that takes amax (given by its bits) to 448 = 1.75 2^8 or less.
__device__ __forceinline__ float pow2_scale(int bits)
{
    const int e = (bits >> 23) - 135 + ((bits & 0x7fffff) > 0x600000);
    return __int_as_float((max(e, -126) + 127) << 23);
}

__device__ __forceinline__ int fp8_moved(int bytes, float by)   // four values, multiplied
{
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(bytes, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(bytes, true);
    return __builtin_amdgcn_cvt_pk_fp8_f32(b[0] * by, b[1] * by, __builtin_amdgcn_cvt_pk_fp8_f32(a[0] * by, a[1] * by, 0, false), true);
}

// A value as it is stored: what is not finite becomes NaN.
__device__ __forceinline__ float stored(float x, float inv)
{
    return (__float_as_int(x) & 0x7fffffff) < 0x7f800000 ? x * inv : __int_as_float(0x7fc00000);
}
__device__ __forceinline__ int magnitude(float x)   // the bits of |x|; 0 where it is not finite
{
    const int bits = __float_as_int(x) & 0x7fffffff;
    return bits < 0x7f800000 ? bits : 0;
}
__device__ __forceinline__ int fp8_four(float a, float b, float c, float d)
{
    return __builtin_amdgcn_cvt_pk_fp8_f32(c, d, __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false), true);
}

// The scale of a block for new values of magnitude `most` (bits), where older ones may stand
// in front; `moved`: what those are multiplied by.
struct BlockScale {
    float scale, inv, moved;
    __device__ __forceinline__ BlockScale(int most, bool older, const float *held) {
        scale = pow2_scale(most);
        const float before = older ? *held : scale;
        if (older) scale = fmaxf(before, scale);
        inv = 1.f / scale;
        moved = before * inv;
    }
};

// Values of 16 tokens from lanes that hold four tokens (4 q .. 4 q + 3 in 16-lane row q) of NC
// channels each, as one dword a channel, to lanes that hold all 16 tokens of NC / 4 channels:
// row q then has channels NC / 4 q and on.  Two rounds of swaps between rows.
template <int NC> __device__ __forceinline__ void turn_tokens(const unsigned (&x)[NC], u32x4 (&w)[NC / 4])
{
    unsigned lo[NC / 2], hi[NC / 2];   // tokens 0-7, tokens 8-15
#pragma unroll
    for (int e = 0; e < NC / 2; ++e) {
        const auto s = __builtin_amdgcn_permlane32_swap(x[e], x[e + NC / 2], false, false);
        lo[e] = s[0];
        hi[e] = s[1];
    }
#pragma unroll
    for (int e = 0; e < NC / 4; ++e) {
        const auto a = __builtin_amdgcn_permlane16_swap(lo[e], lo[e + NC / 4], false, false);
        const auto b = __builtin_amdgcn_permlane16_swap(hi[e], hi[e + NC / 4], false, false);
        w[e] = u32x4{(unsigned)a[0], (unsigned)a[1], (unsigned)b[0], (unsigned)b[1]};
    }
}

// N consecutive values, 4 or a multiple of 8.
template <int N, typename T> __device__ __forceinline__ void load_values(const T *p, float *v)
{
    if constexpr (N == 4 && sizeof(T) == 2) {
        const bf16x4 y = *reinterpret_cast<const bf16x4 *>(p);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = (float)y[e];
    } else if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int c = 0; c < N; c += 8) {
            const bf16x8 y = *reinterpret_cast<const bf16x8 *>(p + c);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[c + e] = (float)y[e];
        }
    } else {
#pragma unroll
        for (int c = 0; c < N; c += 4) {
            const f32x4 y = *reinterpret_cast<const f32x4 *>(p + c);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[c + e] = y[e];
        }
    }
}

// One wave a block, head and kind, 16 bytes a lane to the cache.  Keys: a lane has 16 channels
// of a token.  Values: D / 16 channels of four tokens, turned to D / 64 channels of all.
// Bound by HBM: 16386 new tokens of 8 heads of 128 in bf16 (80 MB in all) take 18 to 20 us, 4.2
// TB/s; with values of four channels by four tokens a lane, stored 4 bytes at a time, 23, and
// keys 4 bytes at a time, too, 26.
template <typename T, int D> __global__ __launch_bounds__(256) void attn_append_kernel(AttnCacheArgs a)
{
    const int unit = blockIdx.y * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    if (unit >= 2 * a.Hk) return;
    const int h = unit >> 1;
    const bool isv = unit & 1;
    Item it = {(int)blockIdx.x, 0};
    if (a.cu) {   // n tokens touch n / 16 + 2 blocks at most: those of a sequence begin at
        auto from = [&](int n) { return within(a.cu[n], a.T) / CACHE_BLOCK + 2 * n; };
        it.b = find_slot(a.N, blockIdx.x, from);
        it.i = (int)blockIdx.x - from(it.b);
    }
    const Fresh f = fresh(a, it.b);
    if (it.i < 0 || it.i >= fresh_blocks(f)) return;
    const int blk = f.lo / CACHE_BLOCK + it.i, base = blk * CACHE_BLOCK;
    const int lo = max(f.lo - base, 0), hi = min(f.hi - base, CACHE_BLOCK);   // slots of new tokens
    const int gb = cache_block(a, it.b, h, blk);
    if (gb < 0) return;
    const long row = f.row + (base - f.lo);   // of slot 0, which may be none
    float *sp = (isv ? a.v_scale : a.k_scale) + gb;
    char *cache = (char *)(isv ? a.v_cache : a.k_cache) + (long)gb * CACHE_BLOCK * D;
    if (isv) {
        constexpr int NC = D / 16, CH = D / 64;
        const int q = lane >> 4, ch = (lane & 15) * NC;
        const T *x = (const T *)a.v + h * D + ch;
        const unsigned slots = (0xffffu >> (16 - hi)) & (0xffffu << lo), older = (1u << lo) - 1;
        const bool part = hi - lo < CACHE_BLOCK;
        u32x4 *p = (u32x4 *)(cache + (ch + q * CH) * CACHE_BLOCK), w[CH], old[CH];
        if (part) {
#pragma unroll
            for (int e = 0; e < CH; ++e) old[e] = p[e];
        }
        float v[4][NC];
        int most = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 4 * q + i;
#pragma unroll
            for (int e = 0; e < NC; ++e) v[i][e] = 0.f;
            if (t >= lo && t < hi) load_values<NC>(x + (row + t) * a.vs, v[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < NC; ++e) most = max(most, magnitude(v[i][e]));
        const BlockScale s(max_lanes(most), lo > 0, sp);
        unsigned four[NC];
#pragma unroll
        for (int e = 0; e < NC; ++e)
            four[e] = fp8_four(stored(v[0][e], s.inv), stored(v[1][e], s.inv), stored(v[2][e], s.inv), stored(v[3][e], s.inv));
        turn_tokens<NC>(four, w);
        if (part) {
#pragma unroll
            for (int e = 0; e < CH; ++e)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    auto bytes = [&](unsigned m) { return (((m >> (4 * i)) & 15u) * 0x00204081u & 0x01010101u) * 0xffu; };
                    unsigned held = old[e][i];
                    if (s.moved != 1.f) held = (held & ~bytes(older)) | ((unsigned)fp8_moved((int)held, s.moved) & bytes(older));
                    w[e][i] = (held & ~bytes(slots)) | (w[e][i] & bytes(slots));
                }
        }
#pragma unroll
        for (int e = 0; e < CH; ++e) p[e] = w[e];
        if (lane == 0) *sp = s.scale;
    } else {
        constexpr int LPR = D / 16, RP = 64 / LPR, NP = 16 / RP;   // lanes a token, tokens at a time, times
        const int t0 = lane / LPR, ch = lane % LPR * 16;
        const T *x = (const T *)a.k + h * D + ch;
        float k[NP][16];
        int most = 0;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int t = i * RP + t0;
#pragma unroll
            for (int e = 0; e < 16; ++e) k[i][e] = 0.f;
            if (t >= lo && t < hi) load_values<16>(x + (row + t) * a.ks, k[i]);
        }
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) most = max(most, magnitude(k[i][e]));
        const BlockScale s(max_lanes(most), lo > 0, sp);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int t = i * RP + t0;
            u32x4 *p = (u32x4 *)(cache + t * D + ch);
            if (t >= lo && t < hi) {
                u32x4 w;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[e] = fp8_four(stored(k[i][4 * e], s.inv), stored(k[i][4 * e + 1], s.inv), stored(k[i][4 * e + 2], s.inv), stored(k[i][4 * e + 3], s.inv));
                *p = w;
            } else if (t < lo && s.moved != 1.f) {
                u32x4 w = *p;
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = fp8_moved((int)w[e], s.moved);
                *p = w;
            }
        }
        if (lane == 0) *sp = s.scale;
    }
}

// --- one token ------------------------------------------------------------------

constexpr int STEP_TILE = 64;       // tokens a tile: four blocks, one for each 16-lane row of a wave
constexpr int STEP_LEAST = 4;       // tiles a workgroup, one for each wave

// Tiles that a table may name and a workgroup takes at once, in one launch (32 over 8 heads of
// 128, in bf16: eight users of 1000 8.7 us, cut 10.7; one of 2000 12.8, cut 10).
constexpr int STEP_WHOLE = 16;

// Rows, at most, that are joined by a workgroup each, not by D / 4 lanes (one user of 100000, 32
// over 4 heads 32 us from 66, 8 over 1 37 from 101; 64 users of 16384 198 from 196).
constexpr int STEP_JOIN = 2048;

// Workgroups to share a call's tiles, `runs` being sequences times key heads.  Two fit a
// compute unit, so 512 run at once; of many sequences with lengths of their own, 768 leave
// smaller remainders (32 over 4 heads, 16 users of 8192 29 us, with 768 34; 64 users of up to
// 16384 125, with 768 116).
__host__ __device__ inline int step_wgs(int runs) { return runs <= 128 ? 512 : 768; }

// Workspace of a call that is cut: int prefix[N + 1] (pieces of cut sequences before each), then
// for each of those pieces and 16 heads float o[16][D] and float lse[16] (base 2), of however
// many heads (as many rows as there are would be an address by a factor only known at run time:
// one user of 100000, 8 heads a key head, 31.9 us from 30.4).  A cut sequence has more tiles than
// `each` (below), so fewer pieces than twice its tiles over `each`, and all of them fewer than
// twice the workgroups that share the tiles.  Whole sequences have none: the workspace does not
// grow with their number.
struct StepWs {
    long o, lse, bytes;
    int wgs;
    __host__ __device__ StepWs(int N, int heads, int d) {
        const int share = step_wgs(N * heads);
        wgs = share + N * heads;
        const long slots = share + (N * heads < share ? N * heads : share);
        o = ((long)(N + 1) * 4 + 255) & ~255L;
        lse = o + slots * 16 * d * 4;
        bytes = lse + slots * 16 * 4;
    }
};
static bool step_cut(int page, int width) { return (long)page * width > STEP_WHOLE * STEP_TILE; }

__device__ __forceinline__ int step_len(const AttnCacheArgs &a, int n) { return a.pages > 0 ? within(a.lens[n], a.width * a.page) : 0; }
__device__ __forceinline__ int step_tiles(const AttnCacheArgs &a, int n) { return (step_len(a, n) + STEP_TILE - 1) / STEP_TILE; }
// Tiles of a piece: all of the call's over the workgroups, rounded up to as many for each wave.
template <typename F> __device__ __forceinline__ int step_each(const AttnCacheArgs &a, int heads, F tiles)
{
    const int lane = threadIdx.x & 63;
    long all = 0;
    for (int n = 0; n < a.N; n += 64) all += sum_lanes(n + lane < a.N ? tiles(n + lane) : 0);
    const int wgs = step_wgs(a.N * heads);
    const long each = (all * heads + wgs - 1) / wgs;
    return max(STEP_LEAST, (int)min((each + 3) & ~3L, 1L << 24));
}
__device__ __forceinline__ int step_pieces(int tiles, int each) { return max(1, (tiles + each - 1) / each); }
__device__ __forceinline__ int step_cuts(int tiles, int each) { return tiles > each ? step_pieces(tiles, each) : 0; }

// bf16 pieces that add up to a value: one of bf16, three of fp32 (8 + 8 + 8 bits).
template <typename T> struct Pieces {
    static constexpr int N = sizeof(T) == 2 ? 1 : 3;
};
template <int N> __device__ __forceinline__ void split4(f32x4 x, bf16x4 (&p)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        p[i] = cvt4(x);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] -= (float)p[i][e];
    }
}

// Eight e4m3 values as bf16, exactly.
__device__ __forceinline__ bf16x8 widen(unsigned lo, unsigned hi) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, 1.f, false), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, 1.f, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, 1.f, false), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, 1.f, true);
    return cat8(__builtin_shufflevector(a, b, 0, 1, 2, 3), __builtin_shufflevector(c, d, 0, 1, 2, 3));
}

// A workgroup has up to 16 query heads of one key head and a run of 64-token tiles of one
// sequence, every wave each fourth of them.  Row i of score tile j is token 4 j + i % 4 of
// block i / 4, so that the 16 weights a lane ends with are those of one block's tokens in
// order: one scale of keys and one of values a lane, and a value operand is 16 tokens of one
// channel as they stand in memory.  A tile's operands are in registers, and the next tile's
// are under way while it is worked on: 16 KB a wave.
// Bound by HBM: 64 users of up to 16384 tokens, 32 over 4 heads of 128 (812 MB), take 158 us,
// 5.1 TB/s, a large copy's rate, and the join 5; one of 300 tokens 6, a launch and the chain
// of table, keys, softmax and values of two tiles.
template <typename T, int D, bool CUT> __global__ __launch_bounds__(256, 2) void attn_step_kernel(AttnCacheArgs a, int ntile)
{
    constexpr int NC = D / 64, NV = D / 16, NP = Pieces<T>::N;
    __shared__ float sums[4][16][D];
    __shared__ float stat[2][4][16];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, r16 = lane_r16(), gq = lane_gq();
    const int heads = a.Hk * ntile, hr = blockIdx.x % heads, h = hr / ntile, g0 = hr % ntile * 16, Hq = a.Hk * a.G;
    int n = blockIdx.x / heads, t0 = 0, t1, pieces = 1, place = 0;   // place: of a piece among those of cut sequences
    if constexpr (CUT) {
        const int first = lane < a.N ? step_tiles(a, lane) : 0;   // most calls have no more sequences
        auto tiles = [&](int b) { return b < 64 ? first : step_tiles(a, b); };   // b: a multiple of 64, and the lane
        const int each = step_each(a, heads, tiles);
        if (blockIdx.x == 0 && wave == 0) {   // for the join
            int *prefix = (int *)a.ws, at = 0;
            for (int b = 0; b < a.N; b += 64) {
                const int mine = b + lane < a.N ? step_cuts(tiles(b + lane), each) : 0, incl = scan_lanes(mine);
                if (b + lane < a.N) prefix[b + lane] = at + incl - mine;
                at += __builtin_amdgcn_readlane(incl, 63);
            }
            if (lane == 0) prefix[a.N] = at;
        }
        // item n of the list of pieces, as find_item does; the whole sequences before it have no place
        Item it = {-1, 0};
        for (int b = 0, at = 0, wholes = 0; b < a.N; b += 64) {
            const int mine = b + lane < a.N ? step_pieces(tiles(b + lane), each) : 0, incl = scan_lanes(mine);
            const int sum = __builtin_amdgcn_readlane(incl, 63);
            const unsigned long long whole = __ballot(mine == 1);
            if (n < at + sum) {
                const int l = (int)__builtin_ctzll(__ballot(n < at + incl));
                it = {b + l, n - at - __builtin_amdgcn_readlane(incl - mine, l)};
                place = n - wholes - (int)__builtin_popcountll(whole & ((1ULL << l) - 1));
                break;
            }
            at += sum;
            wholes += (int)__builtin_popcountll(whole);
        }
        if (it.b < 0) return;
        n = it.b;
        const int nt = __builtin_amdgcn_readfirstlane(step_tiles(a, n));
        pieces = step_pieces(nt, each);
        const int per = (nt + pieces - 1) / pieces;
        t0 = it.i * per;
        t1 = min(nt, t0 + per);
    } else {
        t1 = __builtin_amdgcn_readfirstlane(step_tiles(a, n));
    }
    const int len = __builtin_amdgcn_readfirstlane(step_len(a, n));
    const float c = a.scale * LOG2E;

    bf16x8 qf[2 * NC][NP];
    const bool row = g0 + r16 < a.G;
    {
        const T *q = (const T *)a.q + n * a.qs + (h * a.G + g0 + r16) * D;
#pragma unroll
        for (int i = 0; i < 2 * NC; ++i) {
            const Frag<T> f = row ? load_frag<T>(q + 64 * (i >> 1) + 16 * gq + 8 * (i & 1)) : zero_frag<T>();
            if constexpr (NP == 1) {
                qf[i][0] = f.v;
            } else {
                bf16x4 lo[NP], hi[NP];
                split4(f.lo, lo);
                split4(f.hi, hi);
#pragma unroll
                for (int p = 0; p < NP; ++p) qf[i][p] = cat8(lo[p], hi[p]);
            }
        }
    }
    f32x4 acc[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) acc[v] = f32x4{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f;

    // blocks of the wave's next 16 tiles, one a lane
    int blocks = -1;
    auto lookup = [&](int i) {
        const int blk = (i + (lane >> 2) * 4) * 4 + (lane & 3);
        blocks = blk * CACHE_BLOCK < len ? cache_block(a, n, h, blk) : -1;
    };
    u32x4 kx[4][NC], vx[NV];
    float ks = 0.f, vs = 0.f, nks = 0.f, nvs = 0.f;
    int kb = -1, vb = -1;   // the next tile's block of this lane as a key row, and as a value operand
    auto where = [&](int turn) {
        kb = __shfl(blocks, turn * 4 + (r16 >> 2), 64);
        vb = __shfl(blocks, turn * 4 + gq, 64);
    };
    auto load_k = [&]() {
        const char *p = (const char *)a.k_cache + (long)max(kb, 0) * CACHE_BLOCK * D + (r16 & 3) * D + 16 * gq;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < NC; ++i) kx[j][i] = *(const u32x4 *)(p + 4 * j * D + 64 * i);
        nks = a.k_scale[max(vb, 0)];
    };
    auto load_v = [&]() {
        const char *p = (const char *)a.v_cache + (long)max(vb, 0) * CACHE_BLOCK * D + r16 * CACHE_BLOCK;
#pragma unroll
        for (int v = 0; v < NV; ++v) vx[v] = *(const u32x4 *)(p + v * 16 * CACHE_BLOCK);
        nvs = a.v_scale[max(vb, 0)];
    };
    int turn = 0;
    if (t0 + wave < t1) {
        lookup(t0 + wave);
        where(0);
        load_k();
        load_v();
    }
    for (int i = t0 + wave; i < t1; i += 4) {
        // tokens of this lane's block
        const int count = vb < 0 ? 0 : min(max(len - i * STEP_TILE - gq * CACHE_BLOCK, 0), CACHE_BLOCK);
        const bool part = __any(count < CACHE_BLOCK), more = i + 4 < t1;
        ks = count > 0 ? nks * c : 0.f;
        vs = count > 0 ? nvs : 0.f;
        f32x4 s[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            s[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int x = 0; x < 2 * NC; ++x) {
                const bf16x8 k = widen(kx[j][x >> 1][2 * (x & 1)], kx[j][x >> 1][2 * (x & 1) + 1]);
#pragma unroll
                for (int p = NP - 1; p >= 0; --p) s[j] = mfma_bf16(k, qf[x][p], s[j]);
            }
        }
        if (more) {
            if (++turn == 16) {
                turn = 0;
                lookup(i + 4);
            }
            where(turn);
            load_k();
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[j][e] *= ks;
                if (part) s[j][e] = 4 * j + e < count ? s[j][e] : -INFINITY;
            }
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) mx = fmaxf(mx, s[j][e]);
        mx = rows_max(mx);
        const bool up = mx - m > RAISE;   // false while both are -inf
        if (__any(up)) {
            const float mn = up ? mx : m, al = up ? exp2_hw(m - mn) : 1.f;
            m = mn;
            l *= al;
#pragma unroll
            for (int v = 0; v < NV; ++v) acc[v] *= al;
        }
        const float mb = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float p = exp2_hw(s[j][e] - mb);
                l += p;
                s[j][e] = p * vs;
            }
        if (part) {   // what stands in slots without a token may be a NaN
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int left = count - 4 * w;
                const unsigned keep = left >= 4 ? ~0u : left <= 0 ? 0u : (1u << (8 * left)) - 1;
#pragma unroll
                for (int v = 0; v < NV; ++v) vx[v][w] &= keep;
            }
        }
        // weights (times the values' scale) rounded to bf16 for the matrix cores: half a step
        // each, as the output itself; an fp32 call has them as three bf16 pieces
        bf16x8 pf[2][NP];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            bf16x4 lo[NP], hi[NP];
            split4(s[2 * u], lo);
            split4(s[2 * u + 1], hi);
#pragma unroll
            for (int p = 0; p < NP; ++p) pf[u][p] = cat8(lo[p], hi[p]);
        }
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const bf16x8 x = widen(vx[v][2 * u], vx[v][2 * u + 1]);
#pragma unroll
                for (int p = NP - 1; p >= 0; --p) acc[v] = mfma_bf16(x, pf[u][p], acc[v]);
            }
        if (more) load_v();
    }

    // the waves' sums together
    l = rows_sum(l);
#pragma unroll
    for (int v = 0; v < NV; ++v) *reinterpret_cast<f32x4 *>(&sums[wave][r16][16 * v + 4 * gq]) = acc[v];
    if (gq == 0) {
        stat[0][wave][r16] = m;
        stat[1][wave][r16] = l;
    }
    __syncthreads();
    constexpr int PER = D / 16;   // channels a thread
    const int r = threadIdx.x >> 4, at = (threadIdx.x & 15) * PER;
    if (g0 + r >= a.G) return;
    float top = -INFINITY, total = 0.f, f[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) top = fmaxf(top, stat[0][w][r]);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        f[w] = stat[0][w][r] == -INFINITY ? 0.f : exp2_hw(stat[0][w][r] - top);
        total += f[w] * stat[1][w][r];
    }
    const bool seen = total != 0.f;   // a NaN is seen
    const float inv = seen ? 1.f / total : 0.f, lg = seen ? top + __builtin_amdgcn_logf(total) : -INFINITY;
    const StepWs lay(a.N, heads, D);
    const long orow = (long)n * Hq + h * a.G + g0 + r, slot = ((long)place * heads + hr) * 16 + r;
#pragma unroll
    for (int i = 0; i < PER; i += 4) {
        f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < 4; ++w) x += f[w] * *reinterpret_cast<const f32x4 *>(&sums[w][r][at + i]);
        x = seen ? x * inv : f32x4{0.f, 0.f, 0.f, 0.f};
        if (CUT && pieces > 1) store4((float *)((char *)a.ws + lay.o) + slot * D + at + i, x);
        else store4((T *)a.o + orow * D + at + i, x);
    }
    if (at == 0) {
        if (CUT && pieces > 1) ((float *)((char *)a.ws + lay.lse))[slot] = lg;
        else if (a.lse) a.lse[orow] = lg * LN2;
    }
}

// Joins the pieces of a row: GR groups of D / 4 lanes a row.
template <typename T, int D, int GR> __global__ __launch_bounds__(256) void attn_step_join_kernel(AttnCacheArgs a, int ntile)
{
    constexpr int LPR = D / 4, ROWS = 256 / LPR / GR;   // of a workgroup
    const int Hq = a.Hk * a.G, heads = a.Hk * ntile, at = threadIdx.x % LPR * 4;
    const long row = (long)blockIdx.x * ROWS + (ROWS > 1 ? threadIdx.x / LPR : 0);
    if (row >= (long)a.N * Hq) return;
    const int n = (int)(row / Hq), head = (int)(row - (long)n * Hq), h = head / a.G, g = head - h * a.G;
    const int *prefix = (const int *)a.ws;
    const int p0 = prefix[n], pieces = prefix[n + 1] - p0;
    if (pieces == 0) return;   // written by its one workgroup
    const StepWs lay(a.N, heads, D);
    f32x4 sum;
    float lg;
    if (!join_parts<D, GR>((const float *)((const char *)a.ws + lay.o), (const float *)((const char *)a.ws + lay.lse), pieces,
                           [&](int p) { return ((long)(p0 + p) * heads + h * ntile + (g >> 4)) * 16 + (g & 15); }, sum, lg))
        return;
    store4((T *)a.o + row * D + at, sum);
    if (a.lse && at == 0) a.lse[row] = lg * LN2;
}

template <typename T, int D> static hipError_t append(AttnCacheArgs a, hipStream_t st)
{
    divisor(a.page / CACHE_BLOCK, a.bpp_mul, a.bpp_shift);
    // a sequence's tokens stand in one block more than a sixteenth of them, and one for the begin
    const long items = a.cu ? a.T / CACHE_BLOCK + 2L * a.N : a.N;
    hipLaunchKernelGGL((attn_append_kernel<T, D>), dim3((unsigned)items, (2 * a.Hk + 3) / 4), dim3(256), 0, st, a);
    return hipGetLastError();
}

template <typename T, int D> static hipError_t step(AttnCacheArgs a, hipStream_t st)
{
    const int ntile = (a.G + 15) / 16, heads = a.Hk * ntile;
    divisor(a.page / CACHE_BLOCK, a.bpp_mul, a.bpp_shift);
    if (!step_cut(a.page, a.width)) {
        hipLaunchKernelGGL((attn_step_kernel<T, D, false>), dim3((unsigned)(a.N * heads)), dim3(256), 0, st, a, ntile);
        return hipGetLastError();
    }
    const StepWs lay(a.N, heads, D);
    hipLaunchKernelGGL((attn_step_kernel<T, D, true>), dim3((unsigned)lay.wgs), dim3(256), 0, st, a, ntile);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const long rows = (long)a.N * a.Hk * a.G;
    constexpr int EACH = 1024 / D;
    if (rows <= STEP_JOIN) hipLaunchKernelGGL((attn_step_join_kernel<T, D, EACH>), dim3((unsigned)rows), dim3(256), 0, st, a, ntile);
    else hipLaunchKernelGGL((attn_step_join_kernel<T, D, 1>), dim3((unsigned)((rows + EACH - 1) / EACH)), dim3(256), 0, st, a, ntile);
    return hipGetLastError();
}

hipError_t attn_append_launch(bool bf16, int D, const AttnCacheArgs &a, hipStream_t st)
{
    if (bf16) return D == 128 ? append<__bf16, 128>(a, st) : append<__bf16, 64>(a, st);
    return D == 128 ? append<float, 128>(a, st) : append<float, 64>(a, st);
}

hipError_t attn_step_launch(bool bf16, int D, const AttnCacheArgs &a, hipStream_t st)
{
    if (bf16) return D == 128 ? step<__bf16, 128>(a, st) : step<__bf16, 64>(a, st);
    return D == 128 ? step<float, 128>(a, st) : step<float, 64>(a, st);
}

unsigned long long attn_step_workspace(int N, int Hk, int G, int D, int page, int width)
{
    return N > 0 && step_cut(page, width) ? (unsigned long long)StepWs(N, Hk * ((G + 15) / 16), D).bytes : 0;
}

} // namespace gdn
