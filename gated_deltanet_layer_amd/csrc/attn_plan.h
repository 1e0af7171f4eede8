// attn_plan.h -- how calls of the grouped-attention kernels are cut over workgroups.
// Rules on sizes and type alone, without a HIP header: launchers, kernels and host
// programs read the same ones.  What depends on the sequences' lengths, which only the
// device knows, is worked out there.
#pragma once

namespace gdn {

// --- packed forward -------------------------------------------------------------

// The G query heads that share a key head stand side by side in a row tile: row r of a
// tile is token r / G of it, head r % G, and a tile has as many whole tokens as fit.
constexpr int ATTN_SHARES = 512;   // two workgroups a compute unit
struct AttnFwdPlan {
    int nr;        // 16-row groups a wave: a row tile has 64 nr rows
    int tokens;    // of a row tile
    int shares;    // 0: a workgroup for every row tile
    bool halves;   // whose waves take the key tiles in two groups
    long tiles;    // row tiles of one key head, at most
};

// Rows: two groups a wave (each key operand serves two products) once that gives every
// compute unit a workgroup.
//
// Halves: with a workgroup a unit or fewer, and one row group a wave, four more waves take
// every other key tile (32 over 8 heads of 128, 333 rows 11.4 us from 12.8; 8 over 2, 1000
// rows 20 from 26).
//
// Shares: with fewer row tiles than two a unit, the longest row is the call's time unless all
// rows' key tiles are shared equally; but a share begins, changes rows and is joined for
// some 12 us.  Lengths are on the device, so the rule takes the call for up to four sequences
// of equal length, and shares from 20 key tiles a sequence on, or 36 where halves would do in
// bf16 (8 over 2 heads of 128: one sequence of 1000 26 us, in halves 21; of 2048 36, 35; 4
// over 1, of 4096 48, 62; whole, four of 1000 41, 29, one of 4096 64, 81; fp32, D = 64: one of
// 1000 31, 44; three of 1000 53, 57).
inline AttnFwdPlan attn_fwd_plan(bool bf16, int B, int Tq, int Tk, int Hk, int G)
{
    AttnFwdPlan p;
    const long wide = (long)Tq * G / 128 * Hk;
    p.nr = bf16 && wide >= 256 ? 2 : 1;
    p.tokens = 64 * p.nr / G;
    p.tiles = Tq / p.tokens + (B < Tq ? B : Tq);
    const long wgs = ((Tq + p.tokens - 1) / p.tokens) * (long)Hk, each = B > 0 ? Tk / (B < 4 ? B : 4) : 0;
    const long least = !bf16 ? 20 * 32 : p.nr == 1 && wgs <= 256 ? 36 * 64 : 20 * 64;
    p.shares = wgs > 0 && wgs < ATTN_SHARES && each >= least ? ATTN_SHARES : 0;
    p.halves = !p.shares && p.nr == 1 && wgs <= 256;
    return p;
}

// --- packed backward ------------------------------------------------------------

// Rows (of queries, or keys) that a workgroup owns, and that walk by in a tile.
constexpr int attn_own(bool bf16) { return bf16 ? 128 : 64; }
constexpr int attn_walk(bool bf16) { return bf16 ? 64 : 32; }

struct AttnBwdPlan {
    int tokens;          // of a query tile, which has 128 (64) rows
    int kp, kstep;       // pieces of the walked keys (dq), and the keys of one
    int shares;          // workgroups that share the walked rows of all keys (dk, dv)
    long qtiles;         // query tiles of one key head, at most
};

// Pieces of `tiles` walked tiles, `least` tiles each or more, to give `fill` workgroups.
inline int attn_pieces(long wgs, long fill, long tiles, int least)
{
    if (wgs <= 0 || wgs >= fill || tiles < 2 * least) return 1;
    long n = (fill + wgs - 1) / wgs;
    const long most = n > 32 ? 32 : 16;
    if (n > tiles / least) n = tiles / least;
    return (int)(n > most ? most : n);
}

// The walk of one sequence that has all rows is the longest that a call may have.
inline AttnBwdPlan attn_bwd_plan(bool bf16, int B, int Tq, int Tk, int Hk, int G)
{
    AttnBwdPlan p;
    const int own = attn_own(bf16), st = attn_walk(bf16), least = bf16 ? 2 : 1;
    const long rows = (long)Tq * G, nk = (Tk + st - 1) / st;
    p.tokens = own / G;
    p.qtiles = Tq / p.tokens + (B < Tq ? B : Tq);
    const int kp = attn_pieces(Hk * ((long)(Tq + p.tokens - 1) / p.tokens), 512, nk, least);
    p.kstep = (int)((nk + kp - 1) / kp * st);
    p.kp = kp > 1 ? (Tk + p.kstep - 1) / p.kstep : 1;
    // one workgroup a compute unit (two do not fit its LDS), and eight at a time, as there are
    // XCDs; fewer where the call cannot have two tiles for each
    const long tiles = Hk * ((long)(Tk + own - 1) / own + (B < Tk ? B : Tk)) * ((rows + st - 1) / st);
    p.shares = tiles >= 2 * 256 ? 256 : (int)((tiles / 2 + 8) & ~7L);
    return p;
}

} // namespace gdn
