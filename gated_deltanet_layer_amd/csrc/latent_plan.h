// latent_plan.h -- how calls of the latent-attention kernels are cut over workgroups.
// Rules on sizes and type alone, without a HIP header: launchers, kernels and host
// programs read the same ones.
#pragma once
#ifdef __HIPCC__
#define GDN_PLAN_FN __host__ __device__ inline
#else
#define GDN_PLAN_FN inline
#endif

namespace gdn {

// --- expanded forward -----------------------------------------------------------

// How a call is cut: 16-row groups a wave, and for small grids either pieces of every
// row tile's keys, or the number of workgroups that share all key tiles of the call.
constexpr int FWD_SHARES = 512;   // two workgroups a compute unit
struct FwdPlan {
    int nr, pieces, each;   // pieces of a row tile, `each` key tiles each (1: whole)
    int shares;             // 0: none
};

// Rows: two groups a wave (each key operand serves two products) once that gives
// every compute unit a workgroup; below that, one (333 rows, 16 heads: 13.5 us from
// 14.4).  Keys: the longest row of a causal call is otherwise its time.  Where there is
// less than two workgroups a unit and a row has eight tiles or more (from 512 workgroups
// on cutting costs more than it gives: 2 x 16 heads of 2048 64 us, 85):
//
// - Shares, where each gets eight tiles or more: 512 workgroups (two a unit) take equal
//   runs of key tiles, whatever rows they are of, the runs of one head on one XCD (bf16,
//   2 heads of 8192 68 us, as pieces 141; 8 of 4096 75, 88; 10 of 2048 41, 51; fp32, 8
//   of 3000 173, 223, 2 x 8 of 1021 42, 48; 10 of 2048 on any XCD 3 us more).  Two row
//   groups from half a workgroup a unit on (2 heads of 8192: 12 us).
// - Pieces of four tiles or more, a workgroup each, where a change of rows inside a share
//   (its queries' loads and its result's stores, which nothing hides) would cost more
//   (8 heads of 1024: 21 us, in shares 5 more; one row of 16 heads over 8192 keys 30, 8
//   more).  Enough to fill the units twice, fp32, whose tiles have half the keys and four
//   times the time, half as many again (2 x 8 heads of 700: 39 us, 5 more without), and 32
//   at most, for the join's sake (one row over 32,768 keys 37 us, with up to 16 59, 64 31,
//   128 40; of 4 heads over 16,384 29, 39, 31, 31; 100 rows over 30,000 44, 62, 46, 56).
//
// Rows of less than eight tiles have neither two pieces of four nor, in less than 512
// workgroups, eight tiles for each of 512 shares.
inline FwdPlan fwd_plan(bool bf16, int B, int Tq, int Tk, int H)
{
    const long bh = (long)B * H, wide = bh * ((Tq + 127) / 128);
    const int kt = bf16 ? 64 : 32, nt = (Tk + kt - 1) / kt;
    FwdPlan p = {bf16 && wide >= 256 ? 2 : 1, 1, nt, 0};
    const long tiles = (Tq + 64 * p.nr - 1) / (64 * p.nr), wgs = bh * tiles;
    if (wgs <= 0 || wgs >= 512 || nt < 8) return p;
    if (wgs * nt - bh * tiles * (tiles - 1) / 2 * (64 * p.nr / kt) >= 8 * 512 && wgs * nt < (1L << 30)) {
        p.shares = FWD_SHARES;
        if (bf16 && wide >= 128) p.nr = 2;
        return p;
    }
    const long fill = bf16 ? 512 : 768;
    long n = wgs < 256 ? (fill + wgs - 1) / wgs : 4;
    if (n > nt / 4) n = nt / 4;
    if (n > 32) n = 32;
    p.each = (int)((nt + n - 1) / n);
    p.pieces = (nt + p.each - 1) / p.each;
    return p;
}

// --- expanded backward ----------------------------------------------------------

// How a call is cut.  Where the workgroups that own rows are too few for the device,
// the rows that walk by are cut into pieces, one workgroup each; the pieces' sums
// stand in the workspace and the last kernel adds them up in order.  The longest walk
// of a causal call is otherwise its time.
struct BwdPlan {
    int kp, qp;        // pieces of the keys (dq), of the query rows (dk, dv)
    int kstep, qstep;  // rows of a piece, whole tiles
};

// Pieces of `tiles` walked tiles, `least` tiles each or more, to give `fill` workgroups:
// at most 16, and 32 where more than that are asked for, as each adds to what the last
// kernel reads.  One row over 65,408 keys 128 us, with 16 207, with as many as there are
// (511) 173; 64 rows of 4 heads over 8192 46 us, 50, 52.  Where fewer are asked for, up to
// 32 are no better: fp32, one head of 1200 54 us with 16, 60; 2 heads of 1000 rows over
// 8000 keys 69, 72.
inline int bwd_pieces(long wgs, long fill, int tiles, int least)
{
    if (wgs <= 0 || wgs >= fill || tiles < 2 * least) return 1;
    long n = (fill + wgs - 1) / wgs;
    const long most = n > 32 ? 32 : 16;
    if (n > tiles / least) n = tiles / least;
    return (int)(n > most ? most : n);
}

inline BwdPlan bwd_plan(bool bf16, int B, int Tq, int Tk, int H)
{
    const int own = bf16 ? 128 : 64, st = bf16 ? 64 : 32;
    const long bh = (long)B * H;
    const int nk = (Tk + st - 1) / st, nq = (Tq + st - 1) / st;
    // dq (two workgroups a unit) is cut below 512 workgroups, dk and dv (one) below 256:
    // 8 heads of 2048 101 us; dq below 256 or 1024 112, 116; dk and dv below 128 or 512 131,
    // 112.  Just below a bound cutting can lose (16 heads of 1920, 240 workgroups: 156 us,
    // dk and dv uncut 140), just above it it would (16 of 2048 163 uncut, 181).
    const int least = bf16 ? 2 : 1;   // 500 rows of 16 heads: 48 us (55 with four); fp32, 257 of 4: 27 us (34 with two)
    const int kp = bwd_pieces(bh * ((Tq + own - 1) / own), 512, nk, least);
    const int qp = bwd_pieces(bh * ((Tk + own - 1) / own), 256, nq, least);
    BwdPlan p;
    p.kstep = (nk + kp - 1) / kp * st;
    p.qstep = (nq + qp - 1) / qp * st;
    p.kp = kp > 1 ? (Tk + p.kstep - 1) / p.kstep : 1;
    p.qp = qp > 1 ? (Tq + p.qstep - 1) / p.qstep : 1;
    return p;
}

// --- absorbed -------------------------------------------------------------------

constexpr int STEP_CUS = 256;   // one workgroup a compute unit: two tiles fill its LDS

// Rows of a workgroup.  fp32 has registers for 16.  bf16: 17 to 32 rows by 32 stand between
// two tiles of 16 and one of 64, never the slowest for long (32 heads, r = 512: 32 sequences
// of 4000 tokens 47 us, by 16 51, by 64 42; 4 of 2000 20, 17, 22; 128 of 2000, r = 256, 45,
// 62, 46); beyond, 64 (64 heads, 64 of 2000: 47 us, two tiles of 32 69; 8 of 2000 27, 26).
GDN_PLAN_FN int step_rt(bool bf16, int rows)
{
    return !bf16 || rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

// Workgroups that may share the key tiles of one row tile: with a multiple of eight the row
// tiles of one share, which read the same keys, land on one XCD.  r = 512, 8 sequences of
// 2000: 5 row tiles 35.5 us, without rounding down 45; 10 tiles 47, 56; 15 tiles 59, 66; 28
// tiles 88, 98.  Where it costs nearly half of the workgroups it loses: 17 tiles (8 for 15)
// 85 us, 72; 20 (8 for 12) 86, 79; fp32, r = 256, 17 tiles 61, 42.
GDN_PLAN_FN int step_shares(int ntile) {
    int g = STEP_CUS / (ntile < 1 ? 1 : ntile);
    if (g >= 8) g &= ~7;
    return g < 1 ? 1 : g;
}

} // namespace gdn
