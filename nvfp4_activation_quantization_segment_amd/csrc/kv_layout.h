// Index arithmetic of the paged 8-bit key/value cache and of the work units
// that its kernels run on.  Plain constexpr C++ (host and device), so that the
// bounds it promises are checked on the CPU.
#pragma once

#include <stdint.h>

namespace nvfp4 {

// Positions of one cache block (one head's keys or values of 64 positions).
constexpr int kKvBlock = 64;

// ---------------------------------------------------------------------------
// Layout inside a block: the order in which the matrix instructions of the
// attention kernels take their operands, so that every load of theirs is 16
// contiguous bytes per lane and whole lines per wave.
//
// Keys [D/16][64][16]: a 32x32x64 instruction multiplies 32 keys by 64 dims;
// lane l holds 32 dims of key l % 32, two 16-byte pieces.
//
// Values [4][D][16]: the scores of a 32x32 tile leave lane l with the 16 keys
// 8 (i / 4) + 4 (l / 32) + i % 4 of query l % 32.  They are used as they lie as
// the second operand of the 32x32x16 products with the values, k-step s taking
// i = 8 (s % 2) .. + 7 of tile s / 2; the first operand then needs the values of
// these keys side by side.  Position t = 32u + 16e + 8m + 4h + j has k-step
// 2u + e, lane half h and place 4m + j, and a 16-byte piece holds the two
// k-steps of one u: piece 2u + h, byte 8e + 4m + j.
// ---------------------------------------------------------------------------
constexpr int kv_key_offset(int t, int d) { return (d / 16) * (kKvBlock * 16) + t * 16 + d % 16; }
constexpr int kv_value_offset(int t, int d, int D) {
    return (2 * (t / 32) + t / 4 % 2) * (D * 16) + d * 16 + 8 * (t / 16 % 2) + 4 * (t / 8 % 2) + t % 4;
}

constexpr int64_t clamp64(int64_t v, int64_t lo, int64_t hi) { return v < lo ? lo : v > hi ? hi : v; }
constexpr int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b < 0 ? 1 : 0); }  // b > 0

// ---------------------------------------------------------------------------
// Work units.  The number of new rows of each sequence is known on the device
// only, so a grid is sized for every way the M rows can be shared out, and a
// sequence's first unit is found from the rows before it.
//
// Tiles of T rows (each of `per` rows per token): a sequence of n tokens has
// ceil(n per / T) of them, and tile_base(b + 1) - tile_base(b) >=
// floor(n per / T) + 1 is never less.
// Blocks of 64 positions: n positions starting anywhere touch at most
// (n + 62) / 64 + 1 <= floor(n / 64) + 2 of them.
//
// With few rows a sequence (single tokens, slots that are mostly empty) fewer
// units do: n tokens have at most n ceil(per / T) tiles and n blocks, so every
// row can have that many of its own.  per_row is that number, or 0 where the
// count above is the smaller one; it is picked on the host.  (256 single tokens
// of 56 heads: written in 17 us instead of 21, attended over 1000 keys and 8
// heads in 102 to 110 instead of 113.)
// ---------------------------------------------------------------------------
constexpr int64_t tile_base(int64_t row, int64_t b, int64_t per, int64_t T) { return row * per / T + b; }
constexpr int64_t tile_units(int64_t M, int64_t B, int64_t per, int64_t T) { return M * per / T + B; }
constexpr int64_t block_base(int64_t row, int64_t b) { return row / kKvBlock + 2 * b; }
constexpr int64_t block_units(int64_t M, int64_t B) { return M / kKvBlock + 2 * B; }
constexpr int32_t tiles_per_row(int64_t M, int64_t B, int64_t per, int64_t T) {
    const int64_t each = (per + T - 1) / T;
    return M * each < tile_units(M, B, per, T) ? (int32_t)each : 0;
}
constexpr int32_t blocks_per_row(int64_t M, int64_t B) { return M < block_units(M, B) ? 1 : 0; }
// First unit of the sequence b whose first row is `row`; of M and B: how many.
constexpr int64_t tile_first(int64_t row, int64_t b, int64_t per, int64_t T, int32_t per_row) {
    return per_row ? row * per_row : tile_base(row, b, per, T);
}
constexpr int64_t block_first(int64_t row, int64_t b, int32_t per_row) { return per_row ? row : block_base(row, b); }

// Heads that one workgroup of the cache's long writer or reader takes: as many
// as leave about 8 workgroups for each of 256 CUs, so that a short call still
// fills the chip, and at most `most`.  The writer looks its angles up once for
// all of them (37,810 x 56 heads: 340 us with 16, 346 with 8, 387 with 2); the
// reader keeps nothing from one to the next (352 us with 2, 356 with 8, 363 with
// 16).
constexpr int kKvWriteHeads = 16, kKvReadHeads = 2;
constexpr int32_t kv_heads_each(int64_t units, int32_t heads, int32_t most) {
    return (int32_t)clamp64(units * heads / 2048, 1, most);
}

// Rows of an attention tile, and which of the two a call takes.  B counts all
// sequences, those without rows too.
// 128-row tiles from 64 rows a sequence (on average) on.  8 sequences, 32 query
// and 8 key/value heads: 128 rows over 30,000 keys 212 us (narrow tiles 328);
// 16 sequences of 64 rows and keys, 56 heads: 20 (35), 16 heads: 10 (16).
// But where they are no more than one for each CU, one after the other of
// their blocks of keys is what takes the time, and a narrow tile's four waves
// share them out without a join: one prompt of 1000 rows and 16 heads 35 us
// (17), 56 heads and 512 rows 34 (24).  Over more than 8192 keys pieces of
// them fill the chip again (16 heads, 512 rows after 16,000: 94, narrow 135),
// and over very few a narrow tile's own start and end are most of it (32 and 8
// heads, 4 sequences of 256 rows: 15, narrow 24).  Over 351 shapes of 64 to
// 4000 rows and both dims the rule is 1% slower on average than the better of
// the two, and 32% at most (16 sequences of 64 rows after 2000 keys, 32 and 8
// heads: 92 us, wide 75); always wide 9%, and 102%.  As slots without rows count
// too, a prompt of 4000 rows, 32 and 8 heads, takes 139 us alone and 178 among
// 255 empty slots.
constexpr int kNarrowRows = 32, kWideRows = 128;
constexpr bool attention_wide(int64_t M, int64_t B, int64_t group, int64_t kv_heads, int64_t blocks) {
    const int64_t wide_tiles = (M * group + kWideRows - 1) / kWideRows * kv_heads;
    return M * group >= 64 * B && !(wide_tiles <= 256 && blocks <= 128 && wide_tiles <= 32 * blocks);
}

// Rows [first, last) of sequence b of row_start, whatever the array holds.
struct RowRange {
    int64_t first, last;
};
constexpr RowRange row_range(int64_t start, int64_t end, int64_t M) {
    const int64_t a = clamp64(start, 0, M);
    return RowRange{a, clamp64(end, a, M)};
}

// A length that a table of `blocks` blocks cannot hold.
constexpr bool kv_length_bad(int64_t len, int64_t blocks) { return len < 0 || len > blocks * kKvBlock; }

// First key that the query at position pos < len does not see: all len keys
// (causal = 0), or those of its own run of `causal` positions and before.
// 32-bit throughout: a 64-bit division is a hundred instructions here.
constexpr int32_t kv_limit(int32_t pos, int32_t len, int32_t causal) {
    if (causal == 0) return len;
    if (pos < 0) return 0;
    if (causal == 1) return pos + 1;
    const int32_t left = causal - pos % causal;  // positions from pos to its run's end
    return left > len - pos ? len : pos + left;
}

// Blocks [first, last) of part s of S of a row tile that sees n blocks (n below
// 2^25, S at most 64).
struct BlockRange {
    int32_t first, last;
};
constexpr BlockRange kv_part(int32_t n, int32_t s, int32_t S) {
    if (S == 1) return BlockRange{0, n};
    const int32_t per = (n + S - 1) / S;
    const int32_t a = s * per < n ? s * per : n;
    return BlockRange{a, a + per < n ? a + per : n};
}

}  // namespace nvfp4
