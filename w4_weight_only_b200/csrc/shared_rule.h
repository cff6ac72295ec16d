// How w4a_attn_shared cuts a call: which kernel takes the prefix and the own
// positions, and into how many pieces along the keys.  Host arithmetic on the
// call's sizes alone (the lengths are on the device), apart from the kernels so
// that a test can ask for the choice without a GPU.
#pragma once

namespace w4a {

constexpr int MAX_FEW = 48;    // packed rows of a sequence that few_kernel takes, at most
constexpr int TC_ROWS = 256;   // packed rows of a tile pair
constexpr int FEW_PER_SM = 3;  // CTAs of few_kernel that are resident together, up to 16 packed rows

// Pieces along the keys of equal items of `tiles` 128-key tiles: the count with
// the shortest time, waves x (tiles of a piece + what a piece costs besides:
// its start, its rows of O written and read again, ~3 tiles).  `pairs` items
// are cut in ns, `rest` ones in *ns_rest = half of that when they run at twice
// the speed.
inline int pieces_for(long long pairs, long long rest, bool rest_fast, int tiles, int sms, int cap, int* ns_rest) {
  int best = 1;
  double best_t = 1e30;
  *ns_rest = 1;
  for (int ns = 1; ns <= cap && ns <= (tiles < 1 ? 1 : tiles); ++ns) {
    const int nr = pairs == 0 || !rest_fast ? ns : (ns + 1) / 2;
    const double speed = pairs == 0 && rest_fast ? 0.5 : 1.0;
    const double waves = double((pairs * ns + rest * nr + sms - 1) / sms);
    const double t = waves * (speed * ((tiles + ns - 1) / ns) + 3.0);
    if (t < best_t * 0.999) {
      best_t = t;
      best = ns;
      *ns_rest = nr;
    }
  }
  return best;
}

struct ShPlan {
  long long packed;       // rows x query heads of a KV head
  int few;                // packed rows of a sequence that few_kernel takes
  bool many;              // some sequence may have more
  long long pairs, rest;  // prefix items of whole pair tiles, of the rest of the rows
  bool rest_alt;
  long long own_items;
  int prefix_cap, own_cap;
  int G;
};

inline ShPlan shared_plan(int rows, int batch, int nq, int nkv, int max_new, int sms) {
  const int gq = nq / nkv;
  ShPlan p;
  const long long packed = p.packed = (long long)rows * gq;
  const long long most = (long long)(max_new < rows ? max_new : rows) * gq;  // packed rows of one sequence
  p.few = most <= 16 ? 16 : (most <= 32 ? 32 : MAX_FEW);
  p.many = most > p.few;
  p.pairs = nkv * (packed / TC_ROWS);
  p.rest = packed % TC_ROWS ? nkv : 0;
  p.rest_alt = packed % TC_ROWS <= 128;
  // tiles of the sequences with many rows: at most one partly filled tile each
  long long seqs = packed / (p.few + 1) + 1;
  if (seqs > batch) seqs = batch;
  p.own_items = nkv * (packed / TC_ROWS + seqs);
  auto cap = [&](long long items) {
    const long long c = (2LL * sms + items - 1) / items;
    return int(c < 1 ? 1 : (c > 64 ? 64 : c));
  };
  p.prefix_cap = cap(p.pairs + p.rest);
  p.own_cap = p.many ? cap(p.own_items) : 1;
  p.G = (p.few == 16 ? FEW_PER_SM : 1) * sms;  // CTAs that are resident together
  return p;
}

struct ShChoice {
  int setup;        // what a segment of few_kernel costs besides its tiles, in tiles
  int with_prefix;  // 1: no pass of the prefix's own; every sequence's keys begin with it
  int prefix_few;   // 1: few_kernel takes the prefix too (few packed rows in all)
  int ns_prefix;    // pieces of the prefix, 0 without one of its own
  int ns_rest;      // of them, for the rows behind the last whole pair tile
  int ns_own;       // pieces of the own positions in tc_kernel
  int own_joins;    // 1: tc_kernel's own pieces (one each) take in the prefix's and write the output
  int G;            // CTAs of few_kernel
};

inline ShChoice shared_choice(const ShPlan& p, int batch, int nkv, int hd, int page, int width, int P, int window,
                              int max_new, int sms) {
  const long long packed = p.packed;
  ShChoice c;
  c.G = p.G;
  // (24 sequences of up to 45 rows and 1,500 keys: 54 us with 0, 46 with 3, 44
  // with 5; 16 of 5 rows and 2,048 keys: 25.0 with 0, 23.8 with 1, 23.1 with 2)
  c.setup = p.few == 16 ? 2 : 5;
  // The prefix has no pass of its own where that saves nothing: few positions to
  // read again for every sequence (a launch takes as long as 4,096 of them), or
  // sequences that fill their row tiles by themselves (512 packed rows each on
  // average), for which a tile with the prefix ahead of the own positions does
  // the same work and leaves no pieces to join.  Behind a long prefix such tiles
  // are few and long, and two passes fill the last wave better (~1,000 tokens a
  // sequence: 3 behind 4,000 positions 393 us with a pass of the prefix, 347
  // without; 4 behind 8,192 658 and 692; 4 of ~520 behind 8, 45 and 34).
  c.with_prefix = P > 0 && ((long long)batch * P <= 4096 || (packed >= 512LL * batch && P <= 4096));
  c.prefix_few = P > 0 && !c.with_prefix && packed <= p.few;
  // key tiles that an item can have: all, or what a window reaches
  auto tiles = [&](long long keys) {
    if (window > 0 && keys > (long long)window + max_new + 128) keys = (long long)window + max_new + 128;
    return int((keys + 127) / 128);
  };
  int unused;
  c.ns_prefix = c.ns_rest = P == 0 || c.with_prefix ? 0 : 1;
  if (c.ns_prefix > 0 && !c.prefix_few) {
    // SMs for the prefix.  few_kernel's CTAs fill the others from the start,
    // as many as fit there, so that all run at once: a short prefix is bound by
    // its launch's start and end, a long one with many rows by the tensor
    // cores, few_kernel by memory, which half of the SMs keep busy.  The split
    // is the one with the shortest longer side, by what was measured: 12 us
    // and 0.97 us a key tile of 128 rows for the prefix; 85 GB/s an SM, 6.5 TB/s
    // in all, for 85 % of the keys that the tables have room for (the lengths are
    // on the device, and tables are seldom full).  One after the other unless
    // that is a tenth slower.  (16 sequences behind 8,192 positions: 49 us one
    // after the other, 35 side by side.  100 of up to 1,000 behind 8,192: 103 us
    // with the prefix on the 40 SMs that full tables would leave it, 72 on 48.)
    int budget = sms;
    if (!p.many && p.few == 16) {
      const double unit = 0.97 * (2.0 * p.pairs + (p.rest_alt ? 1.0 : 2.0) * p.rest) * tiles(P);
      double keys = double(width) * page;
      if (window > 0 && keys > double(window) + max_new) keys = double(window) + max_new;
      const double own_bytes = 0.85 * batch * keys * nkv * hd * 4.0, rate = 85e3;
      auto prefix_us = [&](int n) { return 12.0 + unit / n; };
      auto own_us = [&](int n) { return own_bytes / (n * rate < 6.5e6 ? n * rate : 6.5e6); };
      double best = 0.9 * (prefix_us(sms) + own_us(sms));
      for (int n = sms / 4; n <= sms - 8; n += 4) {
        const double t = prefix_us(n) > own_us(sms - n) ? prefix_us(n) : own_us(sms - n);
        if (t < best) {
          best = t;
          budget = n;
        }
      }
      // little of the prefix, much room in the tables: half of the SMs read those as fast as all
      if (budget == sms && unit / 64 < 12.0 && sms >= 128) budget = 64;
      if (budget < sms) c.G = p.G / sms * (sms - budget);
    }
    c.ns_prefix = pieces_for(p.pairs, p.rest, p.rest_alt, tiles(P), budget, p.prefix_cap, &c.ns_rest);
  }
  c.ns_own = 1;
  if (p.many)
    c.ns_own = pieces_for(p.own_items, 0, false, tiles((long long)width * page + (c.with_prefix ? P : 0)), sms, p.own_cap,
                          &unused);
  // one own piece a row, and little of the prefix's to read back: join in the epilogue
  c.own_joins = p.many && c.ns_own == 1 && c.ns_prefix <= 4 && c.ns_rest == c.ns_prefix;
  return c;
}

}  // namespace w4a
