// attn_plan.h -- how calls of the grouped-attention kernels are cut over workgroups.
// Rules on sizes and type alone, without a HIP header: launchers, kernels and host
// programs read the same ones.  What depends on the sequences' lengths, which only the
// device knows, is worked out there.
#pragma once

namespace gdn {

// Row tiles of one key head, at most, and the numbers that they have (find_tile): a sequence
// of l tokens has ceil(l / tokens).
inline long attn_row_tiles(int B, int Tq, int tokens) { return Tq / tokens + (long)(B <= 64 && Tq < B ? Tq : B); }

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
// rows 20 from 26).  Tiles' numbers leave gaps where sequences are many (find_tile), and a launch
// has less than 2^32 threads: 512 a tile until 2^23.
//
// Shares: with fewer row tiles than two a unit, the longest row is the call's time unless all
// rows' key tiles are shared equally; but a share begins, changes rows and is joined for
// some 12 us.  Lengths are on the device, so the rule takes the call for up to four sequences
// of equal length, and shares from 20 key tiles a sequence on; where halves would do in bf16,
// from 36 (8 over 2 heads of 128: one sequence of 1000 26 us, in halves 21; of 2048 36, 35; 4
// over 1, of 4096 48, 62), or from 24 for a few row tiles, which are joined soonest (8 over 2
// heads, 64 tokens of 2000 22 us, in halves 34; D = 64 17, 19, and 64 of 1500 16, 15).  Against
// whole tiles: four of 1000 41, 29, one of 4096 64, 81; fp32, D = 64: one of 1000 31, 44; three
// of 1000 53, 57.
inline AttnFwdPlan attn_fwd_plan(bool bf16, int B, int Tq, int Tk, int Hk, int G)
{
    AttnFwdPlan p;
    const long wide = (long)Tq * G / 128 * Hk;
    p.nr = bf16 && wide >= 256 ? 2 : 1;
    p.tokens = 64 * p.nr / G;
    p.tiles = attn_row_tiles(B, Tq, p.tokens);
    const long wgs = ((Tq + p.tokens - 1) / p.tokens) * (long)Hk, each = B > 0 ? Tk / (B < 4 ? B : 4) : 0;
    const long least = !bf16 ? 20 * 32 : p.nr > 1 || wgs > 256 ? 20 * 64 : wgs > 16 ? 36 * 64 : 24 * 64;
    p.shares = wgs > 0 && wgs < ATTN_SHARES && each >= least ? ATTN_SHARES : 0;
    p.halves = !p.shares && p.nr == 1 && wgs <= 256 && p.tiles * Hk < (1L << 23);
    return p;
}

// --- packed backward ------------------------------------------------------------

// Rows (of queries, or keys) that a workgroup owns, and that walk by in a tile.
constexpr int attn_own(bool bf16) { return bf16 ? 128 : 64; }
constexpr int attn_walk(bool bf16) { return bf16 ? 64 : 32; }

struct AttnBwdPlan {
    int tokens;      // of a query tile, which has attn_own() rows
    long qtiles;     // query tiles of one key head, at most
    int kp, kstep;   // pieces of the keys that walk by them (dq), and the keys of one
    int shares;      // workgroups that share the rows that walk by all keys (dk, dv)
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

inline AttnBwdPlan attn_bwd_plan(bool bf16, int B, int Tq, int Tk, int Hk, int G)
{
    AttnBwdPlan p;
    const int own = attn_own(bf16), st = attn_walk(bf16), least = bf16 ? 4 : 1;
    p.tokens = own / G;
    p.qtiles = attn_row_tiles(B, Tq, p.tokens);
    // dq, below two workgroups a unit: pieces for up to eight sequences of equal length (the
    // lengths are on the device), the last with what a longer one has more, of four tiles (fp32
    // one) or more.  8 over 2 heads of 128: eight sequences of 300 65 us cut, 45 whole; one of
    // 700 43, 55; of 1000 48, 65; of 2048 80, 106; 16 over 4, one of 333 41 both; fp32, D = 64,
    // 4 heads of 300 25 (26 with two), 41.
    const long walk = B > 0 ? (Tk / (B < 8 ? B : 8) + st - 1) / st : 0;
    const int kp = attn_pieces(Hk * ((long)(Tq + p.tokens - 1) / p.tokens), 512, walk, least);
    p.kp = kp;
    p.kstep = (int)(kp > 1 ? (walk + kp - 1) / kp * st : 0);
    // dk and dv: one workgroup a unit (two do not fit its LDS), eight at a time, as there are
    // XCDs; fewer where the call cannot have two tiles for each
    const long tiles = Hk * (Tk / own + (long)(B < Tk ? B : Tk)) * (((long)Tq * G + st - 1) / st);
    p.shares = tiles >= 2 * 256 ? 256 : (int)((tiles / 2 + 8) & ~7L);
    return p;
}

} // namespace gdn
