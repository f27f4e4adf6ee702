// Layout of the 4-bit key/value cache and the host-side rules of its
// attention (internal to libslim; plain C++, tested on the CPU).
//
// A page holds `page` tokens of one head as page / 16 records; a record holds
// 16 tokens, dim channels, g channels to a group, k = dim / g:
//   words [0, 2 dim)          key codes: word (16 lg + t) (dim / 32) + j has token t's channels
//                             32 j + 8 lg .. +7, byte b: channel b low, channel b + 4 high nibble
//   words [2 dim, 4 dim)      value codes: byte t % 4 of word (16 (t / 4) + r) (dim / 32) + a has
//                             token t's channel 32 a + 2 r low, 32 a + 2 r + 1 high nibble
//   words 4 dim + 16 q + t    the keys' pair of group q, token t: step (low half) and low end, bfloat16
//   and 16 k words further    the values' pairs
#pragma once
#include <stddef.h>
#include <stdint.h>

namespace slim {

inline bool kv4_shape(int page, int dim, int group) {
  return (page == 16 || page == 32 || page == 64 || page == 128 || page == 256) &&
         (dim == 64 || dim == 128 || dim == 256) && (group == 32 || group == 64 || group == 128) && group <= dim;
}
inline int kv4_record_words(int dim, int group) { return 4 * dim + 32 * (dim / group); }
inline int64_t kv4_page_words(int page, int dim, int group) {
  return (int64_t)(page / 16) * kv4_record_words(dim, group);
}

// How an attention call is cut.  Rows (a sequence's query tokens times the
// query heads of one key head) go in tiles of tm.  Lengths are known on the
// device only, so the tiles' tokens are cut there: into `extra` runs a head
// beyond one for every tile, in proportion to their number.
struct Kv4Plan {
  bool tile;                 // many rows: four waves of 16 nq rows share the tokens; else each wave has its own
  int nq;                    // tiles of 16 rows a wave holds
  int tm;
  int tiles;                 // row tiles of a sequence (uniform)
  int slots;                 // row tiles, at most (uneven queries: some stay idle)
  int extra;                 // runs beyond them, at most; 0: no joining
  int least;                 // tiles of 32 tokens a run has at least (where a sequence has them)
  int most;                  // runs a tile has on average, at most
  size_t ws_bytes;
};

// b sequences, tq query tokens in all (uniform: tq / b each), cap: the tokens
// a row of the page table can name; f32: queries or outputs are float32.
inline Kv4Plan kv4_plan(int64_t b, int64_t tq, bool uniform, int64_t hq, int64_t hkv, int dim, int group, int64_t cap,
                        bool f32) {
  Kv4Plan p;
  const int64_t g = hq / hkv;
  const int64_t per = (uniform ? tq / b : (tq + b - 1) / b) * g;   // rows of a sequence, on average
  const bool wide = !f32 && dim < 256;                             // registers for two tiles of 16 rows
  // Up to 64 rows the stream reads the cache again for every 32 (or 16) of them, from L2, and is still ahead of tiles
  // that most of a workgroup's waves idle in (40 rows of 16 sequences of up to 8192: 72 us, tiles 81; 64 rows: 70 and
  // 78; 96 rows: 108 and 81; float32, 40 rows of 8: 44 and 45).  With four groups a head or more it has too few
  // registers left (40 rows, g = 32: 127 and 81; 32 rows: 81 and 78; heads of 256, g = 64, 48 rows of 8 sequences: 83
  // and 68), unless the context is so short that the first tile's start counts (300 tokens: 14 and 22; 1000: 25 and 21).
  // The average decides for all of a batch, also for one prompt among single tokens.  Such a call takes longer than one
  // for the single tokens and one for the prompt would (us: one call, the two; single tokens over up to 4096): 31 and a
  // prompt of 1024, 32 + 8 heads 83, 29 + 37; 63 and one of 512, 32 + 32 heads 151, 145 + 25; 64 and one of 2048, 64 + 8
  // heads 198, 48 + 105, 32 + 32 heads 277, 147 + 75.
  p.tile = per > (dim / group >= 4 && cap > 512 ? 32 : 64);
  p.nq = wide && per > 16 && !(p.tile && dim / group >= 4) ? 2 : 1;   // (many rows, small groups: 237 TFLOP/s, one 263)
  p.tm = 16 * p.nq * (p.tile ? 4 : 1);
  p.tiles = (int)((per + p.tm - 1) / p.tm);
  p.slots = (int)(uniform ? b * p.tiles : tq * g / p.tm + (b < tq ? b : tq));
  // Few rows: 512 runs, or 768, as many as a CU holds three of, for batches of 16 rows of heads of 128 and g = 128 (us by
  // 512, 768 and 1024 runs: 16 sequences of up to 8192 34.7, 34.8, 37.9; 8 of 32768 46.8, 43.3, 46.9; 5 drafts of 8 over
  // 3001, 40 heads 29.6, 25.5, 29.5).  Elsewhere more gain less or nothing (16 of up to 8192: heads of 64 27.7, 26.3, 27.2;
  // g = 64 39.6, 38.9, 41.4; g = 32 51.5, 48.0, 51.5; heads of 256 54.4, 57.1, 60.8; float32 39.5, 42.7, 44.1; one of 131072
  // tokens, g = 64 41.4, 42.5, 45.2).  Many rows: 512 (one
  // sequence of 65536 tokens: 438 TFLOP/s, 768 384; 2 of 8192, 256 queries: 568 and 497), but some tiles of `slots`
  // are idle where queries are uneven (560, 512 and 768 runs, TFLOP/s: 3 sequences of up to 3000 and 500 queries 419,
  // 362, 402; 8 of up to 2048 and 300 394, 387, 318; 2 of up to 1500 and 900 337, 271, 333).  However many tiles there
  // are, one sequence may be far longer than the others: 256 runs more, unless the table says that none can be.
  const int64_t want = p.tile ? (uniform ? 512 : 560) : b > 1 && !f32 && p.nq == 1 && group == 128 && dim == 128 ? 768 : 512;
  p.least = p.tile && p.slots * hkv >= 256 ? 32 : 8;
  const int64_t units = p.slots * hkv, tokens = (cap + 31) / 32, spare = cap > 2048 ? 256 : 0;
  const int64_t extra = ((want - units > spare ? want - units : spare) + hkv - 1) / hkv;
  const int64_t useful = p.slots * ((tokens + p.least - 1) / p.least - 1);   // runs are no shorter than `least`
  // every wave goes through all lengths to cut: not for thousands of sequences, which fill the card by themselves but
  // for a long one among them (131072 tokens among 1023 of 100, 8 + 1 heads: 155 us, among 1024: 995)
  p.extra = b > 1024 || units * p.tm >= (1 << 23) ? 0 : (int)(extra < useful ? extra : useful);
  const int64_t most = (tokens + p.least - 1) / p.least;
  p.most = (int)(most < p.extra / p.slots + 1 ? most : p.extra / p.slots + 1);
  p.ws_bytes = p.extra > 0 ? (size_t)(p.slots + p.extra) * hkv * p.tm * (dim + 2) * 4 + (size_t)p.slots * 32 : 0;
  return p;
}

}  // namespace slim
