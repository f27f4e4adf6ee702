// Sizes and choices of the 4-bit products, on the host: the packed layout, which
// kernel a call takes and in which shape, and the workspace (internal to libslim).
// Plain C++ without HIP, so that the rules can be checked where there is no GPU.
#pragma once
#include <math.h>
#include <stddef.h>
#include <stdint.h>

namespace slim {

// ---- 4-bit codes with their scales and zeros, laid out for the products ----
// A record holds 16 rows x 128 columns: 256 words of codes, then a (scale,
// zero) pair per row and group.
inline int64_t q4_row_blocks(int64_t n) { return (n + 15) / 16; }
inline int64_t q4_chunks(int64_t m) { return (m + 127) / 128; }
inline int64_t q4_record_words(int group) { return 256 + 32 * (128 / group); }
inline int64_t q4_matrix_words(int64_t n, int64_t m, int group) {
  return q4_row_blocks(n) * q4_chunks(m) * q4_record_words(group);
}
// ---- Row tiles ----
// Most tiles of tok rows that e ranges covering at most r rows can be cut into.
inline int64_t max_tiles(int64_t r, int64_t e, int64_t tok) {
  const int64_t whole = (r + tok - 1) / tok;
  if (e <= 1) return whole;
  const int64_t ragged = (r + e * (tok - 1)) / tok;
  const int64_t most = ragged < r ? ragged : r;
  return most > whole ? most : whole;
}

// Row tiles to expect: the bounds are on the device, so an expert's last tile
// counts as half, with one standard deviation of their sum (e / 12 is its variance)
// so that a round filled to the last workgroup counts as two; an expert that may
// have rows has one tile at least.
inline double likely_tiles(int64_t r, int64_t e, int64_t tok) {
  if (e == 1) return (double)((r + tok - 1) / tok);
  const double some = (double)(e < r ? e : r), t = (double)r / tok + some / 2 + 0.3 * sqrt(some);
  return t > some ? t : some;
}
// Workgroups of the tile kernel with tiles of tok rows and out outputs.
inline int64_t likely_blocks(int64_t r, int64_t e, int64_t n, int64_t tok, int64_t out) {
  return (int64_t)ceil(likely_tiles(r, e, tok) * (double)((n + out - 1) / out));
}
// 64 rows of Y x 512 output rows in place of 128 x 256 (the same work) where that
// takes fewer rounds of 256 workgroups.
// 8 experts of 11008 x 4096 over 4096 rows, 6 rounds for 7: 390 us against 426; 64
// of 4096 x 2048 over 8192, 5 for 6: 212 against 240; with as many rounds the two
// are alike (8 of 4096 x 4096 over 2048: 120, 118; 8 of 4096 x 11008 over 4096: 453, 444).
inline bool narrow_tiles(int64_t r, int64_t e, int64_t n) {
  return (likely_blocks(r, e, n, 64, 512) + 255) / 256 < (likely_blocks(r, e, n, 128, 256) + 255) / 256;
}
// Workgroups over which the columns are split, four records at least to each and
// all of them in one round.
inline int column_parts(int64_t r, int64_t e, int64_t n, int64_t m) {
  const int64_t blocks = narrow_tiles(r, e, n) ? likely_blocks(r, e, n, 64, 512) : likely_blocks(r, e, n, 128, 256);
  const int64_t most = q4_chunks(m) / 4 < 4 ? q4_chunks(m) / 4 : 4;
  const int64_t parts = 256 / blocks < most ? 256 / blocks : most;
  return parts < 1 ? 1 : (int)parts;
}

// Workspace of the tile kernel: group sums, then what of X it cannot read in
// place, of X's rows or, with a gather of fewer rows than X has or past 32-bit
// offsets, of the gathered rows (compact): the planes of float32 X, or a copy of
// bfloat16 X whose rows do not end with a record or are gathered from too far.
// Without a gather a tile's rows lie together, at any distance from X's first.
// With fewer workgroups than CUs the columns are split over up to four, whose
// sums follow: t = 500, 5000 x 4096 (80 workgroups): 44 us, unsplit 70; t = 1024,
// 4096 x 4096 (128 workgroups, halves): 55 us.
struct TileWs {
  bool compact, copy;
  int parts;
  int64_t nrow;
  size_t planes, partial, bytes;
};
inline TileWs tile_ws(int64_t xrows, int64_t r, int64_t e, int64_t n, int64_t m, int group, bool xbf16, bool gather) {
  TileWs w;
  const size_t nch = (size_t)q4_chunks(m);
  // bytes of a row as the kernel reads it: in place, of the padded copy or of the planes
  const bool padded = m % 128 != 0;
  const uint64_t row = !xbf16 ? 768 * (uint64_t)nch : padded ? 256 * (uint64_t)nch : 2 * (uint64_t)m;
  const bool far = gather && (uint64_t)xrows * row >= 0xfff00000ull;
  w.compact = gather && (r < xrows || far);
  w.copy = xbf16 && (far || padded);
  w.nrow = w.compact ? r : xrows;
  w.planes = ((size_t)w.nrow * nch * (128 / group) * 4 + 15) / 16 * 16;
  w.partial = w.planes + (!xbf16 ? (size_t)w.nrow * 3 * nch * 256 : w.copy ? (size_t)w.nrow * nch * 256 : 0);
  w.parts = column_parts(r, e, n, m);
  w.bytes = w.partial + (w.parts > 1 ? (size_t)w.parts * r * n * 4 : 0);
  return w;
}

// ---- Choices ----
// Which kernel: the shorter of two estimates in us, fitted to measurements (g = 64
// and 128; both are slower alike at 32).  Tiles: 9.5 for the group sums, the first
// loads and the stores, 1.85 for a stage of 128 columns in a round (float32 X, three
// planes: 5.3), and where columns are split 4 and the traffic of the partial sums.
// Streaming: 8, and 6600 (float32 3200) records by 16 rows in one us, the sums' join
// and stores counting as two records.  Measured, tiles - streaming:
//  - t = 2048, 4096 x 11008: 172 - 388; 1537, 2100 x 384: 14 - 17; 1000, 4096 x 2048: 36 -
//    43; 500, 2600 x 1024: 24 - 14; 256, 4096 x 4096: 31 - 24; 256, 4096 x 11008: 48 - 54;
//    130, 4747 x 1088: 25 - 12; 64, 28672 x 8192: 71 - 82; 64, 13824 x 5120: 33 - 28;
//    float32: 1030, 7425 x 640: 40 - 90; 385, 2309 x 1152: 37 - 20.
//  - 8 experts of 11008 x 4096 over 256 rows 68 - 87, over 384 72 - 110; 64 of 1024 x
//    2048 over 3840 rows 40 - 61; 16 of 4096 x 4096 over 512 rows 66 - 65; 18 of 391 x
//    1152 over 2222 rows 27 - 20.
//  - Where they choose the slower: streaming, t = 100, 11008 x 4096: 31 - 33; t = 320, 4096 x
//    4096: 31.7 - 32.5; 8 experts of 11008 x 4096 over 192 rows 64 - 67; and tiles, by more,
//    for float32 t = 2049, 1500 x 320, g = 64: 29 - 24.
inline bool use_tiles(int64_t r, int64_t e, int64_t n, int64_t m, bool xbf16) {
  const int64_t nch = q4_chunks(m);
  const bool narrow = narrow_tiles(r, e, n);
  const int64_t parts = column_parts(r, e, n, m);
  const int64_t rounds = (likely_blocks(r, e, n, narrow ? 64 : 128, narrow ? 512 : 256) * parts + 255) / 256;
  const double stages = (double)(rounds * ((nch + parts - 1) / parts));
  const double tile = 9.5 + stages * (xbf16 ? 1.85 : 5.3) + (parts > 1 ? 4.0 + (double)(parts * r) * n * 1.6e-6 : 0.0);
  const double records = likely_tiles(r, e, 16) * (double)(q4_row_blocks(n) * (nch + 2));
  const double stream = 8.0 + records / (xbf16 ? 6600.0 : 3200.0);
  return tile < stream;
}

// Shape of the streaming kernel, by what fills the 256 CUs.  Measured, us:
//  - 32 rows at a time, bfloat16 only (float32 has not the registers: t = 64, 28672
//    x 8192: 172 against 150 with 16): t = 24, 28672 x 8192: 44.7 against 54; t = 64: 82
//    against 90; t = 256, 4096 x 4096: 23.6 against 25.5; with 128 workgroups (t = 64,
//    4096 x 4096) 13.7 against 9.4 with two row blocks.  An expert's second half tile
//    is mostly empty: 64 of 1024 x 2048 over 2048 rows 42.7 against 40, 8 of 11008 x
//    4096 over 384 110 against 113.
//  - 4, 2 or 1 row blocks a workgroup (X is read once for all of them): t = 16,
//    13824 x 5120: 15.4, 17.4, 25; t = 32, 4096 x 4096: 9.7, 8.0, 11.2; t = 1,
//    4096 x 4096: 8.5, 5.2, 4.7.
//  - 4 waves that load a record ahead; against 8 waves: t = 1, 28672 x 8192, 28.1
//    against 29.5 (g = 32: 39 - 44; float32, 16 rows, g = 32: 61 - 73); against 4 waves
//    with two records at a time: 64 experts of 1024 x 2048, 1024 rows: 27 - 29.
//  - but 8 waves, none ahead, for float32 X with a group to a record, where the records
//    pass more than once (up to 16 rows the stream bounds it) and a wave has two at
//    least; other weights between calls: t = 256, 4096 x 4096: 41.8 against 4 waves' 45.4
//    (g = 64 50.3 - 48.4, g = 32 59.3 - 56.5); t = 48, 13824 x 5120: 42.9 - 45.0; t = 48,
//    22016 x 4096: 53.2 - 57.2 (t = 32 42.4 - 38.0); t = 64, 28672 x 8192: 152.6 - 149.9;
//    t = 1, 28672 x 8192: 46.8 - 43.0; 64 experts of 1024 x 2048, 2048 rows: 65 - 67.7; rows
//    of 12 records, t = 130, 8000 x 1536: 27.4 - 25.5.
//  - 16 waves where a workgroup has a CU to itself: t = 16, 13824 x 5120 (216
//    workgroups): 11.7 against 14.5 with 4 a record ahead; t = 1, 28672 x 8192 (448):
//    31.7 against 28.1.
struct StreamShape {
  int blocks;                // row blocks of 16 outputs a workgroup
  int tiles;                 // 16-row tiles of Y a workgroup
  int waves;
  int records;               // taken by a wave at a time
  bool ahead;                // the next one's loads beside the products
};
inline StreamShape stream_shape(int64_t r, int64_t e, int64_t n, int64_t m, int group, bool xbf16) {
  const int64_t nrb = q4_row_blocks(n), nch = q4_chunks(m), r4 = (nrb + 3) / 4;
  const int64_t rows_per_matrix = (r + e - 1) / e;
  if (xbf16 && rows_per_matrix > (e == 1 ? 16 : 40) && r4 * ((r + 31) / 32) >= 192) return {4, 2, 4, 1, true};
  const int64_t tiles = max_tiles(r, e, 16);
  if (r4 * tiles >= 192) {
    if (nch > 16 && r4 * tiles < 320) return {4, 1, 16, 1, false};
    if (!xbf16 && group == 128 && nch >= 16 && rows_per_matrix > 16) return {4, 1, 8, 1, false};
    return {4, 1, 4, 1, true};
  }
  if ((nrb + 1) / 2 * tiles >= 144) return {2, 1, 8, 2, false};
  return {1, 1, 8, 2, false};
}

}  // namespace slim
