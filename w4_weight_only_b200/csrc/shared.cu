// Attention of a batch whose sequences share a prefix, over the paged KV
// cache (paged.cu).
//
// Row r of sequence b is query token i of its n_b = row_start[b + 1] -
// row_start[b] rows, the last n_b of the sequence's len_b own positions; it
// sits at position p = P + len_b - n_b + i behind the shared prefix of P
// positions and sees positions j <= p, with a window W > 0 also j > p - W:
// positions j < P in the shared pages, the others in the sequence's own.
//   out = softmax(q k^T / sqrt(hd)) v,  query head h over KV head h / gq
// A softmax over a union of key ranges is the join of the softmaxes over the
// ranges: each piece keeps a reference m (log2 units), l = sum 2^(s - m) and
// O = sum 2^(s - m) v in fp32, and pieces join as sum O 2^(m - M) /
// sum l 2^(m - M).  A piece that held none of a row's keys has l = 0 (its O may
// be unwritten) and is left out; every other one counts, so that a NaN or an
// infinity among what a row sees reaches its output whatever the cut: a piece
// with keys has l >= 1, a NaN, or l = 0 where all its scores are -inf.  A row
// sees itself at least, so l = 0 in the end means that every score was -inf, and
// 1 / l makes that the NaN of the formula.  So the work is cut twice: a long prefix apart from the own
// positions, because all rows share its keys (a short one is read ahead of
// each sequence's own, see with_prefix), and both along the keys, to fill the
// SMs when there are few rows.
//
//  - tc_kernel: tcgen05, tiles of 128 packed rows (row x query heads of one
//    KV head) by 128 keys.  The prefix for all rows of the batch, and the own
//    positions of the sequences with many rows.
//  - few_kernel: mma.sync, sequences with at most 16, 32 or 48 packed rows
//    (decode, a few drafted tokens): their own positions, read at memory speed.
//  - join_kernel: joins the pieces of each (row, head) that tc_kernel has not
//    finished itself.
// They are launched one behind the other and overlap (each may start when the
// one before has started); what reads a piece waits for the launch before.
//
// Measured, 40 query heads over 8 of K / V, head_dim 128, GPU time of a call in
// a full queue (a call that finds the queue empty takes the host's 12 to 16 us
// at least):
//   a prompt of 8,192: 636 us, 1,080 TFLOP/s; call after call for seconds 715 us,
//     at 1,735 MHz under the power cap
//   3,722 rows of 4 sequences behind 8,192 positions: 658 us, 1,050 TFLOP/s
//   16 sequences of one row, up to 16,384 own positions: 97 us, 6.2 TB/s
//   16 of one row and up to 2,048 behind 8,192: 35 us
//   64 of one row and up to 1,024 behind 32,768: 102 us, 430 TFLOP/s
//   24 of 5 to 9 rows and up to 1,500 behind 4,097, pages of 16: 86 us
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "ptx.cuh"
#include "shared_rule.h"
#include "tc.cuh"
#include "w4a_internal.h"

namespace w4a {

namespace {

constexpr long long SH_WAIT = 4000000000LL;  // bound on any single wait (~2 s)
constexpr float RESCALE = 8.f;               // the kept reference may fall this far (log2) below the maximum

struct ShArgs {
  const uint16_t* q;
  const int32_t* row_start;
  const int32_t* lens;
  const int32_t* table;
  const int32_t* ptable;
  uint16_t* out;
  uint32_t* err;
  float* o_part;        // [parts][rows * nq][HD]
  float2* ml_part;      // [parts][rows * nq]: (m, l)
  float* o_cont;        // [G][few][HD]: pieces that begin inside a segment
  float2* ml_cont;      // [G][few]
  int rows, batch, nq, nkv, gq, n_pages, page_log2, width, P, window, max_new;
  int ns_prefix;        // pieces of the prefix (slots 0 ..), 0 without one
  int ns_rest;          // of them, for the rows behind the last whole pair tile
  int ns_own;           // pieces of the own positions in tc_kernel (slots ns_prefix ..)
  int few;              // packed rows of a sequence that few_kernel takes (16, 32 or 48)
  int setup;            // what a segment costs besides its tiles, in tiles
  int prefix_few;       // 1: few_kernel takes the prefix too (few packed rows in all)
  int with_prefix;      // 1: no pass of the prefix's own; every sequence's keys begin with it
  int own_joins;        // 1: tc_kernel's own pieces (one each) take in the prefix's and write the output
  int G;                // CTAs of few_kernel
  float scale_log2;     // log2(e) / sqrt(hd)
};

__device__ __forceinline__ void sh_error(uint32_t* err, uint32_t bits) { atomicOr(err, bits); }

// The numbers of a sequence; ok = 0 when they do not fit (n = 0 then).
struct Seq {
  int r0, n, len, ok;
};
__device__ __forceinline__ Seq load_seq(const ShArgs& a, int b) {
  Seq s;
  const int r1 = a.row_start[b + 1];
  s.r0 = a.row_start[b];
  s.len = a.lens[b];
  s.ok = s.r0 >= 0 && r1 >= s.r0 && r1 <= a.rows && r1 - s.r0 <= a.max_new && s.len >= r1 - s.r0 &&
         s.len <= (a.width << a.page_log2);
  s.n = s.ok ? r1 - s.r0 : 0;
  return s;
}
__device__ __forceinline__ int total_rows(const ShArgs& a) { return min(max(a.row_start[a.batch], 0), a.rows); }

// Bounded wait; false (abort flag and error word set) when it runs out or
// another role has given up.
__device__ __forceinline__ bool sh_wait(uint64_t* bar, uint32_t par, volatile int* abort_flag, uint32_t* err) {
  if (mbar_wait_sleep(bar, par)) return true;
  const long long t0 = clock64();
  while (!mbar_wait_sleep(bar, par)) {
    if (*abort_flag) return false;
    if (clock64() - t0 > SH_WAIT) {
      *abort_flag = 1;
      sh_error(err, EW_MBAR_TIMEOUT);
      return false;
    }
  }
  return true;
}
// Copies still in flight land before the CTA may exit.
__device__ __forceinline__ void sh_drain(uint64_t* bar, uint32_t par, uint32_t* err) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, par)) {
    if (clock64() - t0 > SH_WAIT) {
      sh_error(err, EW_DRAIN_TIMEOUT);
      return;
    }
  }
}

// ---------------------------------------------------------------------------
// keys kb .. kb + ROWS - 1 of a page list into a tile of HD / 64 panels
// [ROWS][64] (128-byte swizzle), by the lanes of one warp: one tensor copy per
// page (or part of one) and panel.  Pages at or past key_end are not in the
// list; their rows of the tile keep what was there.
// ---------------------------------------------------------------------------
template <int ROWS>
__device__ __forceinline__ uint32_t load_blocks(int kb, int key_end, int page_log2) {
  const int bs = min(1 << page_log2, ROWS);
  return uint32_t((min(ROWS, key_end - kb) + bs - 1) / bs);  // blocks of bs keys to copy
}
template <int HD, int ROWS>
__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* map, const int32_t* pages, int kb,
                                          int key_end, int kvh, uint64_t* bar, const ShArgs& a, int lane) {
  constexpr int PANELS = HD / 64;
  const int bs = min(1 << a.page_log2, ROWS);
  const int nblk = int(load_blocks<ROWS>(kb, key_end, a.page_log2));
  if (lane < nblk * PANELS) {
    const int blk = lane / PANELS, panel = lane % PANELS;
    const int k0 = kb + blk * bs;
    int id = pages[k0 >> a.page_log2];
    if ((unsigned)id >= (unsigned)a.n_pages) {
      sh_error(a.err, EW_BAD_POS);
      id = a.n_pages;  // outside the tensor: zeros
    }
    tma_load_3d(dst + panel * (ROWS * 128) + blk * bs * 128, map, panel * 64, k0 & ((1 << a.page_log2) - 1),
                id * a.nkv + kvh, bar);
  }
}

// ---------------------------------------------------------------------------
// tc_kernel
// ---------------------------------------------------------------------------
// CTA = one KV head, one tile of packed rows, one run of 128-key tiles.
// Warps 0-3 and 4-7 are two softmax groups (thread = row = TMEM lane), warp 8
// loads, warp 9 issues the MMAs (one thread) and owns the 512 TMEM columns.
// Two groups, so that the tensor core works for one while the other is in its
// softmax:
//  PAIR: two tiles of 128 rows, group i has tile i, both use every K / V tile.
//  ALT (at most 128 rows): one tile of rows, group i has the key tiles of
//        parity i, and the groups' pieces are joined at the end.  A key tile
//        takes half of PAIR's time.
// S_i = Q K^T into TMEM columns [128 i, + 128); a thread takes its row's 128
// scores into registers at once, forms P = 2^(s - m) and writes it back as bf16
// pairs over the first 64 of the same columns (head_dim 64: next to O), where
// the second MMA reads it as its A operand, O_i += P V, V as an MN-major
// operand; it starts on the first 64 keys while the weights of the others are
// formed.  The reference m moves only when the maximum has risen by more than
// 2^8 over it, so O is rescaled rarely; P <= 2^8 is rounded to bf16, 2^-8 of
// each weight at most, while l sums the weights unrounded in fp32.
// What bounds it: a pair of tiles takes ~3,650 clocks a step of 128 keys,
// against 2,140 of the tensor core alone: a group's softmax (~2,000) and the
// latency of its two MMAs (~1,650) follow one another, and the other group's
// fill only part of that.  48 % of the tensor pipe's cycles are busy over a
// prompt of 8,192, 50 % of the special-function unit's.  An item's start and
// end take ~10,000 clocks more, so items are long where there are enough rows.
// Slower were: S in two halves of 64 keys, twice as many softmax warps, waits
// that spin instead of sleep, items handed out by a counter, and loads that
// start ahead of the rows' part of an item's start.
template <int HD>
struct Tc {
  static constexpr int TILE = 128 * HD * 2;                 // 128 rows, bytes
  static constexpr int PANEL = 128 * 128;
  static constexpr int NT = HD == 128 ? 6 : 10;             // tiles in shared memory: Q (ALT 1, PAIR 2), the others the K / V ring
  static constexpr int BARS = 512 + 2 * 256 * 8;            // barriers and small things, the rows' visible keys
  static constexpr int SMEM = NT * TILE + BARS + 1024;
  static constexpr int O_COL = 256;                         // O_i at 256 + i HD
  static constexpr int P_COL(int i) { return HD == 128 ? i * 128 : 384 + i * 64; }
  static constexpr int LD = HD + 4;                         // floats between the rows of O in shared memory
  static_assert(256 * (LD * 4 + 16) <= NT * TILE, "O tiles fit where Q, K and V were");
};
constexpr int TC_THREADS = 320;

template <int HD>
__global__ void __launch_bounds__(TC_THREADS, 1)
    tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
              const __grid_constant__ ShArgs a, const int own, const int lead) {
  using C = Tc<HD>;
  constexpr int TILE = C::TILE, PANEL = C::PANEL, LD = C::LD;
  extern __shared__ uint8_t tc_raw[];
  uint8_t* sm = tc_raw + ((1024u - (smem_addr(tc_raw) & 1023u)) & 1023u);
  uint8_t* sQ = sm;
  uint64_t* q_full = reinterpret_cast<uint64_t*>(sm + C::NT * TILE);
  uint64_t* kv_full = q_full + 1;        // [NT]
  uint64_t* kv_empty = kv_full + C::NT;  // [NT]
  uint64_t* s_full = kv_empty + C::NT;     // [2]: S_i computed (and every earlier MMA done)
  uint64_t* p_full = s_full + 2;         // [2][2]: half of P_i written, O_i rescaled (4 warps arrive)
  uint64_t* o_done = p_full + 4;
  uint32_t* tbase = reinterpret_cast<uint32_t*>(o_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tbase + 1);
  int* s_lo = reinterpret_cast<int*>(tbase + 2);
  int* s_b = s_lo + 1;      // sequence and its first tile
  int* s_warp = s_b + 2;    // [8]
  // a row's visible keys [x, y) in the item's list, and in the prefix ahead of
  // it: read once a tile, before the wait for its scores (in registers over the
  // softmax they would spill)
  volatile int2* s_vis = reinterpret_cast<int2*>(q_full + 64);  // [2][256]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    mbar_init(q_full, 8);
#pragma unroll 1
    for (int s = 0; s < C::NT; ++s) {
      mbar_init(kv_full + s, 1);
      mbar_init(kv_empty + s, 1);
    }
#pragma unroll 1
    for (int s = 0; s < 2; ++s) mbar_init(s_full + s, 1);
#pragma unroll 1
    for (int s = 0; s < 4; ++s) mbar_init(p_full + s, 4);
    mbar_init(o_done, 1);
    *abort_flag = 0;
    *s_lo = a.P;
    s_b[0] = -1;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(tbase, 512);
    tmem_relinquish();
  }

  if (lead) wait_previous_kernel();  // first launch of the call: nothing is read before what came before it is done
  launch_dependents();

  // ---- which item: KV head, rows [base, base + valid) of the packed rows of
  // tokens r0 .., piece of the keys ----
  int kvh, piece, ns, base, valid, r0, b = 0, n = 0, len = 0;
  if (!own) {
    // whole pair tiles in ns_prefix pieces each, then the rest of the rows: a
    // rest of at most 128 rows takes half the time a key, in ns_rest pieces
    const int packed = total_rows(a) * a.gq, whole = a.rows * a.gq / TC_ROWS;
    int x = blockIdx.x;
    const int heads = whole * a.nkv;
    r0 = 0;
    if (x < heads * a.ns_prefix) {
      ns = a.ns_prefix;
      base = (x % whole) * TC_ROWS;
      x /= whole;
    } else {
      x -= heads * a.ns_prefix;
      ns = a.ns_rest;
      base = whole * TC_ROWS;
    }
    kvh = x % a.nkv;
    piece = x / a.nkv;
    valid = min(TC_ROWS, packed - base);
  } else {
    int x = blockIdx.x;
    ns = a.ns_own;
    piece = x % ns;
    x /= ns;
    kvh = x % a.nkv;
    const int want = x / a.nkv;  // tile of the sequences with many rows, in order
    int before = 0;
#pragma unroll 1
    for (int c0 = 0; c0 < a.batch; c0 += 256) {
      int t = 0;
      if (tid < 256 && c0 + tid < a.batch) {
        const Seq s = load_seq(a, c0 + tid);
        if (s.n * a.gq > a.few) t = (s.n * a.gq + TC_ROWS - 1) / TC_ROWS;
      }
      int incl = t;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
      }
      __syncthreads();
      if (warp < 8 && lane == 31) s_warp[warp] = incl;
      __syncthreads();
      int off = before, sum = 0;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        if (w < warp) off += s_warp[w];
        sum += s_warp[w];
      }
      if (t > 0 && want >= off + incl - t && want < off + incl) {
        s_b[0] = c0 + tid;
        s_b[1] = off + incl - t;
      }
      before += sum;
      if (before > want) break;
    }
    __syncthreads();
    b = s_b[0];
    valid = 0;
    base = r0 = 0;
    if (b >= 0) {
      const Seq s = load_seq(a, b);
      n = s.n;
      len = s.len;
      r0 = s.r0;
      const int nt = (n * a.gq + TC_ROWS - 1) / TC_ROWS;
      base = (nt - 1 - (want - s_b[1])) * TC_ROWS;  // the longest rows first
      valid = min(TC_ROWS, n * a.gq - base);
    }
  }

  // the first page ids on their way before the loads need them
  if (warp == 8 && lane == 0 && valid > 0) {
    const bool mine = own && !a.with_prefix;
    prefetch_l2((mine ? a.table + (size_t)b * a.width : a.ptable) +
                (int((long long)(mine ? len : a.P) * piece / ns) >> a.page_log2));
    if (own && a.with_prefix) prefetch_l2(a.table + (size_t)b * a.width);
  }

  // ---- this thread's row: token, head, its query; the visible keys [vlo,
  // vhi) (prefix positions, or own positions) ----
  const bool alt = valid <= 128;
  const int NS = C::NT - (alt ? 1 : 2);  // ring slots
  uint8_t* sR = sm + (alt ? 1 : 2) * TILE;
  const int grp = (warp >> 2) & 1, r = (warp & 3) * 32 + lane;
  const int prow = base + (alt ? 0 : grp * 128) + r;
  const bool live = warp < 8 && prow < base + valid;
  const int row_tok = live ? prow / a.gq : 0;
  const int tok = r0 + row_tok, head = kvh * a.gq + (live ? prow - row_tok * a.gq : 0);
  constexpr int CH = HD / 8, RPI = 32 / CH;  // 16-byte chunks of a row, rows a warp brings at a time
  if (warp < 8) {
    // The rows of Q into shared memory (128-byte swizzle), each warp its 32, a
    // row's chunks side by side (a row per thread took 7,000 clocks; ALT: each
    // group brings every second round).  Dead rows keep what was there.
    const int line = live ? tok * a.nq + head : -1;
    uint8_t* dst = sQ + (alt ? 0 : grp) * TILE + (warp & 3) * 32 * 128;
    const int c = lane % CH;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int row = i * RPI + lane / CH, at = __shfl_sync(0xffffffffu, line, row);
      if (at >= 0 && (!alt || (i & 1) == grp))
        cp_async16(dst + (c >> 3) * PANEL + row * 128 + (((c & 7) ^ (row & 7)) << 4), a.q + (size_t)at * HD + c * 8);
    }
    cp_async_commit();
  }
  // vis: the row's keys of the list that the item is about; k: those that some
  // row of the item sees.  p: the same of the prefix ahead of a sequence's own
  // positions (its end is P)
  int vlo = 0, vhi = 0, vlo_p = a.P, k_lo = 0, k_hi = a.P, p_lo = a.P;
  if (own) {
    k_hi = len - n + (base + valid - 1) / a.gq + 1;
    const int back = a.window ? len - n + base / a.gq - a.window + 1 : -a.P;  // the first row's lowest key, from P on
    k_lo = max(0, back);
    if (a.with_prefix) p_lo = min(a.P, max(0, a.P + back));
    if (live) {
      const int p = len - n + row_tok;  // own position of the row
      vhi = p + 1;
      if (a.window) vlo = max(0, p - a.window + 1);
      if (a.with_prefix) vlo_p = a.window ? min(a.P, max(0, a.P + p - a.window + 1)) : 0;
    }
  } else if (live) {
    vhi = a.P;
    if (a.window) {
      // the row's sequence: the last one that starts at or before it
      int lo = 0, hi = a.batch;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.row_start[mid] <= tok)
          lo = mid;
        else
          hi = mid;
      }
      const Seq s = load_seq(a, lo);
      const int back = s.len - s.n + (tok - s.r0);  // own positions before the row's
      vlo = s.n ? min(a.P, max(0, a.P + back - a.window + 1)) : a.P;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (!own && a.window) {  // uniform
    if (live) atomicMin(s_lo, vlo);
    __syncthreads();
    k_lo = *s_lo;
  }
  const uint32_t tmem = *tbase;
  int t0 = 0, nb = 0;
  const int p_tiles = p_lo < a.P ? ((a.P + 127) >> 7) - (p_lo >> 7) : 0;
  if (k_lo < k_hi && valid > 0) {
    const int nt = p_tiles + ((k_hi + 127) >> 7) - (k_lo >> 7);
    t0 = int((long long)nt * piece / ns);
    nb = int((long long)nt * (piece + 1) / ns) - t0;
  }
  const int groups = valid <= 0 ? 0 : ((alt ? nb > 1 : true) ? 2 : 1);
  // tile t of the item: where its keys are, and which of them are of use
  struct Span {
    const int32_t* pages;
    int kb, lo, hi;
  };
  auto span = [&](int t) {
    t += t0;
    if (t < p_tiles) return Span{a.ptable, ((p_lo >> 7) + t) * 128, p_lo, a.P};
    return Span{own ? a.table + (size_t)b * a.width : a.ptable, ((k_lo >> 7) + t - p_tiles) * 128, k_lo, k_hi};
  };

  if (warp == 8) {
    // ---- loads, in the order in which the MMAs use them: K_0 (K_1) V_0 K_2 V_1 .. (ALT), K_0 V_0 K_1 V_1 .. (PAIR)
    int s = 0, lap = 0;
    bool ok = true;
    auto put = [&](const CUtensorMap* map, int t) {
      if (!ok) return;
      if (lap > 0) {
        int good = 1;
        if (lane == 0) good = sh_wait(kv_empty + s, uint32_t(lap - 1) & 1u, abort_flag, a.err) ? 1 : 0;
        if (!__shfl_sync(0xffffffffu, good, 0)) {
          ok = false;
          return;
        }
      }
      const Span sp = span(t);
      const int bs = min(1 << a.page_log2, 128);
      if (lane == 0) mbar_expect_tx(kv_full + s, load_blocks<128>(sp.kb, sp.hi, a.page_log2) * bs * HD * 2);
      __syncwarp();
      load_tile<HD, 128>(sR + s * TILE, map, sp.pages, sp.kb, sp.hi, kvh, kv_full + s, a, lane);
      if (++s == NS) {
        s = 0;
        ++lap;
      }
    };
    if (alt) {
      if (nb > 0) put(&tmK, 0);
      if (nb > 1) put(&tmK, 1);
#pragma unroll 1
      for (int t = 0; t < nb; ++t) {
        put(&tmV, t);
        if (t + 2 < nb) put(&tmK, t + 2);
      }
    } else {
#pragma unroll 1
      for (int t = 0; t < nb; ++t) {
        put(&tmK, t);
        put(&tmV, t);
      }
    }
    if (lane == 0) {
      // each slot's last load
      for (int i = 0; i < NS; ++i) {
        const int laps = lap + (i < s ? 1 : 0);
        if (laps > 0) sh_drain(kv_full + i, uint32_t(laps - 1) & 1u, a.err);
      }
    }
  } else if (warp == 9) {
    // ---- MMAs (one thread) ----
    if (lane == 0 && nb > 0) {
      const uint32_t idS = umma_idesc_f16(128, 128, true);
      const uint32_t idO = umma_idesc_f16(128, HD, true) | UMMA_B_MN;
      // descriptors of the first tiles; a byte offset adds its sixteenth to the start address
      const uint64_t dQ = umma_desc_sw128(sQ, 0), dK = umma_desc_sw128(sR, 0), dV = umma_desc_mn_sw128(sR, PANEL, 1024);
      auto plus = [](uint64_t d, uint32_t n) { return (d & 0xffffffff00000000ull) | (uint32_t(d) + n); };  // (no carry)
      int s = 0;          // the next ring slot to take
      uint32_t lap = 0;
      auto take = [&](int& slot) {
        slot = s;
        const bool w = sh_wait(kv_full + s, lap & 1u, abort_flag, a.err);
        tc_fence_after();
        if (++s == NS) {
          s = 0;
          ++lap;
        }
        return w;
      };
      auto issue_s = [&](int qi, int ki) {
        const uint64_t q = plus(dQ, uint32_t((alt ? 0 : qi) * (TILE >> 4))), k = plus(dK, uint32_t(ki * (TILE >> 4)));
#pragma unroll
        for (int ks = 0; ks < HD / 16; ++ks) {
          const uint32_t off = uint32_t((ks >> 2) * PANEL + (ks & 3) * 32) >> 4;
          umma_f16(tmem + uint32_t(qi * 128), plus(q, off), plus(k, off), idS, ks > 0 ? 1u : 0u);
        }
        umma_commit(s_full + qi);
      };
      // O_qi (+)= P_qi V: each half of the keys when its weights are there
      auto issue_pv = [&](int qi, int vi, int j) {
        const uint64_t v = plus(dV, uint32_t(vi * (TILE >> 4)));
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (!sh_wait(p_full + qi * 2 + half, uint32_t(j) & 1u, abort_flag, a.err)) return false;
          tc_fence_after();
#pragma unroll
          for (int k4 = 0; k4 < 4; ++k4) {
            const int ks = half * 4 + k4;
            umma_f16_ts(tmem + uint32_t(C::O_COL + qi * HD), tmem + uint32_t(C::P_COL(qi) + ks * 8),
                        plus(v, uint32_t(ks * 16 * 128 >> 4)), idO, (j == 0 && ks == 0) ? 0u : 1u);
          }
        }
        return true;
      };
      bool ok = sh_wait(q_full, 0u, abort_flag, a.err);
      int ks = 0, vs = 0;  // slots of the K and V tiles in use
      if (alt) {
        for (int t = 0; t < 2 && t < nb && ok; ++t) {
          if (!(ok = take(ks))) break;
          issue_s(t, ks);
          umma_commit(kv_empty + ks);
        }
#pragma unroll 1
        for (int t = 0; t < nb && ok; ++t) {
          if (!(ok = take(vs) && issue_pv(t & 1, vs, t >> 1))) break;
          umma_commit(kv_empty + vs);
          if (t + 2 < nb) {
            if (!(ok = take(ks))) break;
            issue_s(t & 1, ks);
            umma_commit(kv_empty + ks);
          }
        }
      } else {
        if (ok && (ok = take(ks))) {
          issue_s(0, ks);
          issue_s(1, ks);
          umma_commit(kv_empty + ks);
        }
#pragma unroll 1
        for (int j = 0; j < nb && ok; ++j) {
          const bool more = j + 1 < nb;
          if (!(ok = take(vs) && issue_pv(0, vs, j))) break;
          if (more) {
            if (!(ok = take(ks))) break;
            issue_s(0, ks);
          }
          if (!(ok = issue_pv(1, vs, j))) break;
          umma_commit(kv_empty + vs);
          if (more) {
            issue_s(1, ks);
            umma_commit(kv_empty + ks);
          }
        }
      }
      umma_commit(o_done);
      // every MMA issued has completed before the tensor memory is freed
      sh_drain(o_done, 0u, a.err);
    }
  } else {
    cp_async_wait<0>();
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) mbar_arrive(q_full);
    s_vis[tid].x = vlo;
    s_vis[tid].y = vhi;
    s_vis[256 + tid].x = vlo_p;
    s_vis[256 + tid].y = a.P;
    // ---- softmax ----
    const uint32_t tl = tmem + (uint32_t((warp & 3) * 32) << 16);
    const uint32_t tS = tl + uint32_t(grp * 128), tP = tl + uint32_t(C::P_COL(grp)),
                   tO = tl + uint32_t(C::O_COL + grp * HD);
    const bool warp_live = __any_sync(0xffffffffu, live);
    float m_run = -INFINITY, l_run = 0.f;
    bool ok = true;
    int j = 0;
    if (grp < groups) {
#pragma unroll 1
      for (int t = alt ? grp : 0; t < nb; t += alt ? 2 : 1, ++j) {
        const bool ahead = t + t0 < p_tiles;  // in the prefix ahead of the own positions
        const int kb = (t + t0 + (ahead ? p_lo >> 7 : (k_lo >> 7) - p_tiles)) * 128;
        // keys that no row sees: their values must be finite (0 x NaN), so
        // group 0 (ALT: the tile's group) clears those rows of V
        const bool edge = (alt || grp == 0) && (kb < (ahead ? p_lo : k_lo) || kb + 128 > (ahead ? a.P : k_hi));
        volatile int2* vis = s_vis + (ahead ? 256 : 0) + tid;
        const int ilo = vis->x - kb, ihi = vis->y - kb;  // visible: ilo <= i < ihi
        const bool part = __any_sync(0xffffffffu, live && (ilo > 0 || ihi < 128));
        if (!__all_sync(0xffffffffu, sh_wait(s_full + grp, uint32_t(j) & 1u, abort_flag, a.err))) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (edge) {
          const uint32_t vi = alt ? uint32_t(t == nb - 1 ? 2 * nb - 1 : 2 * t + 2) : 2u * t + 1u;
          if (!__all_sync(0xffffffffu, sh_wait(kv_full + vi % NS, (vi / NS) & 1u, abort_flag, a.err))) {
            ok = false;
            break;
          }
          if (kb + r < (ahead ? p_lo : k_lo) || kb + r >= (ahead ? a.P : k_hi)) {
            uint8_t* v = sR + (vi % NS) * TILE + r * 128;
#pragma unroll
            for (int c = 0; c < HD / 8; ++c)
              *reinterpret_cast<uint4*>(v + (c >> 3) * PANEL + ((c & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async();
        }
        uint32_t v[4][32];
        uint64_t sum_a = 0, sum_b = 0;
        uint64_t scale2 = 0, nref2 = 0;
        if (warp_live) {
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(tS + uint32_t(32 * c), v[c]);
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld_wait32(v[c]);
          if (part) {
#pragma unroll
            for (int i = 0; i < 128; ++i)
              if (i < ilo || i >= ihi) v[i >> 5][i & 31] = 0xff800000u;  // -inf
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < 32; i += 2)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              mx[c] = fmaxf(fmaxf(mx[c], __uint_as_float(v[c][i])), __uint_as_float(v[c][i + 1]));
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
          if (__any_sync(0xffffffffu, top > m_run + RESCALE)) {  // also the first finite maximum of a row
            const bool up = top > m_run + RESCALE;
            const float alpha = up ? exp2f(m_run - top) : 1.f;  // 0 while the reference was -inf
            if (up) m_run = top;
            l_run *= alpha;
            // the group's previous P V has completed: S_i's barrier follows it
            if (j > 0) {
#pragma unroll 1
              for (int c = 0; c < HD; c += 16) {
                uint32_t o[16];
                tmem_ld16(tO + uint32_t(c), o);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                tmem_st16(tO + uint32_t(c), o);
              }
            }
          }
          const float nref = m_run == -INFINITY ? 0.f : -m_run;
          scale2 = pack_f32x2(a.scale_log2, a.scale_log2);
          nref2 = pack_f32x2(nref, nref);
        }
        // weights of 32 keys.  (Part of them by a polynomial on the FMA pipe, to
        // relieve the special-function unit, was slower at every share: 728 us
        // without, 741 at an eighth, 756 at a quarter, 816 at a half of them,
        // for a prompt of 8,192.)
        auto weights = [&](uint32_t (&w)[32], int c) {
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const uint64_t xa =
                fma_f32x2(pack_f32x2(__uint_as_float(w[i]), __uint_as_float(w[i + 1])), scale2, nref2);
            const uint64_t xb =
                fma_f32x2(pack_f32x2(__uint_as_float(w[i + 2]), __uint_as_float(w[i + 3])), scale2, nref2);
            float x0, x1, x2, x3;
            unpack_f32x2(xa, x0, x1);
            unpack_f32x2(xb, x2, x3);
            const float p0 = ex2_fast(x0), p1 = ex2_fast(x1), p2 = ex2_fast(x2), p3 = ex2_fast(x3);
            sum_a = add_f32x2(sum_a, pack_f32x2(p0, p1));
            sum_b = add_f32x2(sum_b, pack_f32x2(p2, p3));
            w[i >> 1] = cvt_bf16x2(p0, p1);
            w[(i >> 1) + 1] = cvt_bf16x2(p2, p3);
          }
          tmem_st16(tP + uint32_t(16 * c), w);
        };
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (warp_live) {
            weights(v[2 * half], 2 * half);
            weights(v[2 * half + 1], 2 * half + 1);
            tmem_st_wait();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full + grp * 2 + half);
        }
        float s0, s1;
        unpack_f32x2(add_f32x2(sum_a, sum_b), s0, s1);
        l_run += s0 + s1;
      }
    }
    // ---- outputs: the rows of O through shared memory, so that they are
    // written whole; (m, l) of each row beside them ----
    ok = ok && (nb == 0 || __all_sync(0xffffffffu, sh_wait(o_done, 0u, abort_flag, a.err)));
    tc_fence_after();
    const bool join = alt && groups == 2;
    float* sO = reinterpret_cast<float*>(sm) + (alt ? 0 : grp * 128 * LD);  // [128][LD]
    float4* s_row = reinterpret_cast<float4*>(sm + 256 * LD * 4) + (alt ? 0 : grp * 128);
    float* mine = sO + r * LD;
    auto dump = [&](float f, bool add, float g) {
#pragma unroll 1
      for (int c = 0; c < HD; c += 32) {
        uint32_t o[32];
        tmem_ld32(tO + uint32_t(c), o);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          float4 x = make_float4(__uint_as_float(o[i]) * f, __uint_as_float(o[i + 1]) * f,
                                 __uint_as_float(o[i + 2]) * f, __uint_as_float(o[i + 3]) * f);
          float4* d = reinterpret_cast<float4*>(mine + c + i);
          if (add) {
            const float4 y = *d;
            x = make_float4(fmaf(y.x, g, x.x), fmaf(y.y, g, x.y), fmaf(y.z, g, x.z), fmaf(y.w, g, x.w));
          }
          *d = x;
        }
      }
    };
    if (join) {
      if (grp == 1 && warp_live && ok) {
        dump(1.f, false, 0.f);
        s_row[r] = make_float4(m_run, l_run, 0.f, 0.f);
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
    }
    if (grp < (alt ? min(groups, 1) : groups) && warp_live && ok) {
      float f0 = 1.f, f1 = 0.f;
      if (join) {
        const float4 o = s_row[r];
        const float M = fmaxf(m_run, o.x);
        f0 = m_run == -INFINITY ? 0.f : exp2f(m_run - M);
        f1 = o.x == -INFINITY ? 0.f : exp2f(o.x - M);
        m_run = M;
        l_run = l_run * f0 + o.y * f1;
      }
      const bool final = own && a.own_joins;
      const size_t stride = (size_t)a.rows * a.nq;
      const int np = final ? a.ns_prefix : 0;  // (with own_joins every row has as many)
      if (np > 0) wait_previous_kernel();  // the prefix's pieces, made by the launch before this one
      if (final) {
        // the weights of this piece and of the prefix's in the joined row
        const size_t line = (size_t)tok * a.nq + head;
        const float m0 = m_run;
        float L = l_run;
        if (live) {
#pragma unroll 1
          for (int i = 0; i < np; ++i) {
            const float2 ml = a.ml_part[i * stride + line];
            if (ml.y == 0.f) continue;
            const float M = fmaxf(m_run, ml.x);
            L = L * exp2f(m_run - M) + ml.y * exp2f(ml.x - M);
            m_run = M;
          }
        }
        const float inv = 1.f / L;
        const float f = live ? exp2f(m0 - m_run) * inv : 0.f;
        f0 *= f;
        f1 *= f;
        l_run = inv;
      }
      if (nb > 0) dump(f0, join, f1);
      // (m, l), or with the final row (reference, 1 / sum); which row of the outputs
      s_row[r] = make_float4(m_run, l_run, __int_as_float(tok * a.nq + head), 0.f);
      __syncwarp();
      // a warp writes its 32 rows, one after the other, 16 bytes a lane
      const int w0 = (warp & 3) * 32, rows = min(32, valid - (alt ? 0 : grp * 128) - w0);
      const int part = own ? a.ns_prefix + piece : piece;
      constexpr int LPR = HD / 4;  // lanes of a row
      const int sub = lane / LPR, col = (lane % LPR) * 4;
      if (final) {
#pragma unroll 1
        for (int i0 = sub; i0 < rows; i0 += 8 * (32 / LPR)) {
          // eight rows at a time, so that the loads of the prefix's pieces overlap
          float4 x[8], w[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const int i = w0 + min(i0 + u * (32 / LPR), rows - 1);
            x[u] = *reinterpret_cast<const float4*>(sO + i * LD + col);
            w[u] = s_row[i];
          }
#pragma unroll 1
          for (int k = 0; k < np; ++k) {
            float2 ml[8];
            float4 y[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              const size_t line = k * stride + __float_as_int(w[u].z);
              ml[u] = a.ml_part[line];
              y[u] = *reinterpret_cast<const float4*>(a.o_part + line * HD + col);
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              if (ml[u].y == 0.f) continue;  // an empty piece's O was not written
              const float f = exp2f(ml[u].x - w[u].x) * w[u].y;
              x[u] = make_float4(fmaf(y[u].x, f, x[u].x), fmaf(y[u].y, f, x[u].y), fmaf(y[u].z, f, x[u].z),
                                 fmaf(y[u].w, f, x[u].w));
            }
          }
#pragma unroll
          for (int u = 0; u < 8; ++u)
            if (i0 + u * (32 / LPR) < rows)
              *reinterpret_cast<uint2*>(a.out + (size_t)__float_as_int(w[u].z) * HD + col) =
                  make_uint2(cvt_bf16x2(x[u].x, x[u].y), cvt_bf16x2(x[u].z, x[u].w));
        }
      } else {
        float* o_part = a.o_part + part * stride * HD + col;
        if (live) a.ml_part[part * stride + tok * a.nq + head] = make_float2(m_run, l_run);
        if (nb > 0) {
#pragma unroll 8
          for (int i = sub; i < rows; i += 32 / LPR) {
            const float4 x = *reinterpret_cast<const float4*>(sO + (w0 + i) * LD + col);
            const int line = __float_as_int(s_row[w0 + i].z);
            *reinterpret_cast<float4*>(o_part + (size_t)line * HD) = x;
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  wait_previous_kernel();
}

// ---------------------------------------------------------------------------
// few_kernel
// ---------------------------------------------------------------------------
// The 64-key tiles of every (sequence, KV head) with at most 16 MG packed rows
// form one stream (sequence, then KV head, then key), cut into G equal
// runs, one a CTA, whatever the lengths: a CTA takes the segments of its run
// one by one.  A segment that lies in one run is finished there; the piece
// with its first tile goes to the rows' own slot, a piece that begins inside a
// segment to the CTA's (a run has one such piece at most, its first).  A
// segment's start and end take as long as a few tiles, so it counts for `setup`
// tiles more, ahead of its first, which carry no keys.
// Warp (mt, kq) of the 4 MG math warps has m-tile mt (16 rows) and keys 16 kq
// .. + 15 of every tile, and is alone in its loop: scores by mma.sync, a
// softmax of its own over its keys, P straight from the score fragments into
// the second product.  (Sharing P through shared memory, with a quarter of V's
// columns per warp, took two barriers and 2.5 times the instructions per tile,
// and few_kernel ran at their latency, not memory's.)  At a segment's end the
// four key quarters are joined through the stage of its last tile (one
// m-tile), or through memory of their own.  The last warp loads, running ahead
// over segments.  mma.sync, since so few rows would fill a small part of a
// tcgen05 tile.  Up to 16 rows memory bounds this kernel all the same: 16
// sequences of up to 16,384 positions (600 MB) take 97 us, 6.2 TB/s, one of 65,536
// 51 us, 5.3 TB/s; its start and end are ~8 us of each.  With three m-tiles it
// does not get there: 24 sequences of 5 to 9 rows and up to 9,000 positions take
// 158 us with pages of 16 (483 MB, 3.1 TB/s) and 149 with pages of 64 (554 MB,
// 3.7 TB/s): every m-tile reads the K and V fragments for itself, and one CTA an
// SM has three stages in flight.  Up to 16 rows the tensor pipe
// has time to spare, and P goes in as two bf16 terms, P and its rounding
// error, for two products; above rounded to bf16 once.
template <int HD, int MG>
struct Fw {
  static constexpr int TK = 64;                    // keys per tile
  static constexpr int KV = TK * HD * 2;           // bytes of K (or V) per stage
  static constexpr int ROWS = 16 * MG;
  static constexpr int NW = 4 * MG;                // math warps
  static constexpr int THREADS = 32 * (NW + 1);
  static constexpr int PER_SM = MG == 1 ? FEW_PER_SM : 1;  // CTAs that are resident together
  static constexpr int NST = (MG == 1 ? 2 : (MG == 2 ? 4 : 3)) * (HD == 128 ? 1 : 2);  // stages
  static constexpr bool SCR = MG > 1;              // the quarters are joined in memory of their own, all m-tiles at once
  static constexpr bool LO = MG == 1;
  static constexpr int QB = ROWS * HD * 2;
  static constexpr int XB = SCR ? MG * 64 * HD * 4 : 0;
  static constexpr int SMEM = NST * 2 * KV + QB + XB + 1024;
};

// A sequence (or the prefix, b = batch) in the tile stream.
struct FewSeq {
  Seq s;
  int k_lo;    // first key that a row sees
  int k_end;   // keys
  int tiles;   // of the stream: `setup` and its key tiles
  int p_lo;    // the same of the prefix ahead of the own positions
  int p_tiles; // (0: none)
};
__device__ __forceinline__ void few_tiles(const ShArgs& a, FewSeq& f) {
  const int back = a.window ? f.s.len - f.s.n - a.window + 1 : -a.P;  // the first row's lowest key, from P on
  f.k_lo = max(0, back);
  f.k_end = f.s.len;
  f.p_lo = a.with_prefix ? min(a.P, max(0, a.P + back)) : a.P;
  f.p_tiles = f.p_lo < a.P ? ((a.P + 63) >> 6) - (f.p_lo >> 6) : 0;
  f.tiles = f.s.n == 0 || f.s.n * a.gq > a.few
                ? 0
                : f.p_tiles + ((f.s.len + 63) >> 6) - (f.k_lo >> 6) + a.setup;
}
// Tile i of a sequence: its page list, first key, and keys of use.
struct FewSpan {
  const int32_t* pages;
  int kb, lo, hi;
};
__device__ __forceinline__ FewSpan few_span(const ShArgs& a, const FewSeq& f, int b, int i) {
  if (i < f.p_tiles) return FewSpan{a.ptable, ((f.p_lo >> 6) + i) * 64, f.p_lo, a.P};
  return FewSpan{b == a.batch ? a.ptable : a.table + (size_t)b * a.width, ((f.k_lo >> 6) + i - f.p_tiles) * 64, f.k_lo,
                 f.k_end};
}
// The prefix as a last sequence of all rows, when there are few; first_pos:
// the lowest position of a row (INT_MAX: no rows).
__device__ __forceinline__ int few_prefix_lo(const ShArgs& a, int first_pos) {
  return a.window ? min(a.P, max(0, first_pos - a.window + 1)) : 0;
}
__device__ __forceinline__ int few_prefix_tiles(const ShArgs& a, int first_pos) {
  if (!a.prefix_few || first_pos == 0x7fffffff) return 0;
  const int lo = few_prefix_lo(a, first_pos);
  return lo < a.P ? ((a.P + 63) >> 6) - (lo >> 6) + a.setup : 0;
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <int N>
__device__ __forceinline__ void math_barrier() {
  asm volatile("bar.sync 1, %0;" ::"n"(N) : "memory");
}

// The stream's cut: W tiles in G runs (of a tile at least, so that the pieces
// of a segment are those of consecutive CTAs), the first W % G one tile longer.
struct Runs {
  int G, q, r;
  __device__ Runs(int W, int g) : G(min(g, max(W, 1))), q(W / G), r(W - q * G) {}
  __device__ int begin(int c) const { return c * q + min(c, r); }
  __device__ int of(int x) const { return x < r * (q + 1) ? x / (q + 1) : r + (x - r * (q + 1)) / q; }
};

template <int HD, int MG>
__global__ void __launch_bounds__(Fw<HD, MG>::THREADS, Fw<HD, MG>::PER_SM)
    few_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
               const __grid_constant__ ShArgs a, const int lead) {
  using C = Fw<HD, MG>;
  constexpr int NST = C::NST, KV = C::KV, ROWS = C::ROWS, NT = HD / 8;
  extern __shared__ uint8_t fw_raw[];
  uint8_t* sm = fw_raw + ((1024u - (smem_addr(fw_raw) & 1023u)) & 1023u);
  uint8_t* sQ = sm + NST * 2 * KV;
  __shared__ uint64_t full[NST], empty[NST];
  __shared__ float2 s_ml[C::SCR ? MG : 1][4][16];
  __shared__ int s_vlo[ROWS], s_vhi[ROWS], s_vlo_p[ROWS], s_line[ROWS];  // of a packed row: visible keys, token x n_q + head
  __shared__ int s_abort;
  volatile int* abort_flag = &s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, C::NW);
    }
    fence_mbar_init();
    s_abort = 0;
  }
  __syncthreads();
  if (lead) wait_previous_kernel();  // as in tc_kernel
  launch_dependents();
  // the tables' lines on their way (two a CTA), while the lengths are read
  if (tid < 2) {
    const long long at = 32LL * (blockIdx.x + tid * gridDim.x), n = (long long)a.batch * a.width;
    if (at < n) prefetch_l2(a.table + at);
  }
  // ---- the stream and this CTA's run of it: each warp by itself, a sequence
  // a lane (the first 32 stay in registers) ----
  auto tiles_of = [&](int b, int& bad, int& first_pos) {
    if (b >= a.batch) return 0;
    FewSeq f;
    f.s = load_seq(a, b);
    bad |= !f.s.ok;
    if (a.prefix_few && f.s.n > 0) first_pos = min(first_pos, a.P + f.s.len - f.s.n);
    few_tiles(a, f);
    return f.tiles;
  };
  int bad = 0, first_pos = 0x7fffffff;
  const int t_first = tiles_of(lane, bad, first_pos);
  int own_tiles = t_first;
#pragma unroll 4
  for (int b = lane + 32; b < a.batch; b += 32) own_tiles += tiles_of(b, bad, first_pos);
  own_tiles = __reduce_add_sync(0xffffffffu, own_tiles);
  if (a.prefix_few) first_pos = __reduce_min_sync(0xffffffffu, first_pos);
  if (blockIdx.x == 0 && warp == 0 && __any_sync(0xffffffffu, bad) && lane == 0) sh_error(a.err, EW_BAD_SHAPE);
  const int p_lo = few_prefix_lo(a, first_pos), p_tiles = few_prefix_tiles(a, first_pos);
  const int W = (own_tiles + p_tiles) * a.nkv;
  const Runs runs(W, a.G);
  const int cta = int(blockIdx.x);
  const int x_lo = cta < runs.G ? runs.begin(cta) : 0, x_hi = cta < runs.G ? min(runs.begin(cta + 1), W) : 0;
  // the sequence of the run's first tile, and the tiles before it
  int b0 = a.batch, base0 = own_tiles;
  {
    const int y = x_lo / a.nkv;
    int before = 0;
#pragma unroll 1
    for (int c0 = 0; c0 < a.batch; c0 += 32) {
      int incl = c0 == 0 ? t_first : tiles_of(c0 + lane, bad, first_pos);
      const int t = incl;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
      }
      const unsigned past = __ballot_sync(0xffffffffu, before + incl > y);
      if (past) {
        const int l = __ffs(past) - 1;
        b0 = c0 + l;
        base0 = before + __shfl_sync(0xffffffffu, incl - t, l);
        break;
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  auto seq_at = [&](int b) {
    FewSeq f;
    if (b == a.batch) {
      f.s = Seq{0, total_rows(a), 0, 1};
      f.k_lo = p_lo;
      f.k_end = a.P;
      f.p_lo = f.p_tiles = 0;
      f.tiles = p_tiles;
    } else {
      f.s = load_seq(a, b);
      few_tiles(a, f);
    }
    return f;
  };

  if (warp == C::NW) {
    // ---- loads ----
    uint32_t it = 0;
    bool ok = true;
    int b = b0, base = base0;
#pragma unroll 1
    for (int x = x_lo; x < x_hi && ok;) {
      FewSeq f = seq_at(b);
      while (x >= (base + f.tiles) * a.nkv) {
        base += f.tiles;
        f = seq_at(++b);
      }
      const int y = x - base * a.nkv, kvh = y / f.tiles, tv = y - kvh * f.tiles;
      const int nv = min(x_hi - x, f.tiles - tv), t = max(0, tv - a.setup), nt = tv + nv - a.setup - t;
      const int bs = min(1 << a.page_log2, 64);
#pragma unroll 1
      for (int i = 0; i < nt; ++i, ++it) {
        const int s = int(it % NST);
        if (it >= uint32_t(NST)) {
          int good = 1;
          if (lane == 0) good = sh_wait(empty + s, ((it / NST) - 1u) & 1u, abort_flag, a.err) ? 1 : 0;
          if (!__shfl_sync(0xffffffffu, good, 0)) {
            ok = false;
            break;
          }
        }
        const FewSpan sp = few_span(a, f, b, t + i);
        if (lane == 0) mbar_expect_tx(full + s, 2u * load_blocks<64>(sp.kb, sp.hi, a.page_log2) * bs * HD * 2);
        __syncwarp();
        load_tile<HD, 64>(sm + s * 2 * KV, &tmK, sp.pages, sp.kb, sp.hi, kvh, full + s, a, lane);
        load_tile<HD, 64>(sm + s * 2 * KV + KV, &tmV, sp.pages, sp.kb, sp.hi, kvh, full + s, a, lane);
      }
      x += nv;
    }
    if (lane == 0) {
      const uint32_t first = it > uint32_t(NST) ? it - NST : 0u;
#pragma unroll 1
      for (uint32_t j = first; j < it; ++j) sh_drain(full + (j % NST), (j / NST) & 1u, a.err);
    }
  } else {
    // ---- math ----
    constexpr int NTH = C::NW * 32;
    const int g = lane >> 2, tq = lane & 3, mi = lane >> 3, r7 = lane & 7;
    const int kq = warp & 3, mt = warp >> 2;
    // this lane's ldmatrix rows: a 16-byte chunk c of row r is at chunk c ^ (r
    // & 7), so step ks (two chunks) flips bits 5 and 6 of the address
    const uint32_t k_off = (16 * kq + (mi >> 1) * 8 + r7) * 128 + (((mi & 1) ^ r7) << 4);
    const uint32_t v_off = (16 * kq + (mi & 1) * 8 + r7) * 128 + (((mi >> 1) ^ r7) << 4);
    const uint32_t q_at = smem_addr(sQ) + (16 * mt + (mi & 1) * 8 + r7) * 128 + (((mi >> 1) ^ r7) << 4);
    const uint32_t ring = smem_addr(sm);
    uint32_t st = 0, phase = 0;
    int b = b0, base = base0;
    bool ok = true;
#pragma unroll 1
    for (int x = x_lo; x < x_hi;) {  // (a warp whose wait ran out goes on through the barriers, and writes nothing)
      FewSeq f = seq_at(b);
      while (x >= (base + f.tiles) * a.nkv) {
        base += f.tiles;
        f = seq_at(++b);
      }
      const int y = x - base * a.nkv, kvh = y / f.tiles, tv = y - kvh * f.tiles;
      const int nv = min(x_hi - x, f.tiles - tv), t0 = max(0, tv - a.setup), nt = tv + nv - a.setup - t0;
      x += nv;
      if (nt <= 0) continue;  // only of what stands for the segment's start
      const int nrow = f.s.n * a.gq, nmt = (nrow + 15) >> 4;
      // ---- the rows: their lines of q and of the outputs, their visible keys ----
      if (tid < nmt * 16) {
        int vlo = 0, vhi = 0, vlo_p = a.P, line = -1;
        if (tid < nrow) {
          const int i = tid / a.gq;
          line = (f.s.r0 + i) * a.nq + kvh * a.gq + (tid - i * a.gq);
          if (b == a.batch) {
            vhi = a.P;
            if (a.window) {
              int lo = 0, hi = a.batch;
              while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (a.row_start[mid] <= i)
                  lo = mid;
                else
                  hi = mid;
              }
              const Seq s = load_seq(a, lo);
              vlo = s.n ? min(a.P, max(0, a.P + s.len - s.n + (i - s.r0) - a.window + 1)) : a.P;
            }
          } else {
            const int p = f.s.len - f.s.n + i;
            vhi = p + 1;
            if (a.window) vlo = max(0, p - a.window + 1);
            if (a.with_prefix) vlo_p = a.window ? min(a.P, max(0, a.P + p - a.window + 1)) : 0;
          }
        }
        s_vlo_p[tid] = vlo_p;
        s_vlo[tid] = vlo;
        s_vhi[tid] = vhi;
        s_line[tid] = line;
      }
      math_barrier<NTH>();
      // ---- Q into shared memory (128-byte swizzle; zero rows up to whole m-tiles) ----
      for (int i = tid; i < nmt * 16 * (HD / 8); i += NTH) {
        const int row = i / (HD / 8), c = i % (HD / 8), line = s_line[row];
        uint4 q = make_uint4(0u, 0u, 0u, 0u);
        if (line >= 0) q = *reinterpret_cast<const uint4*>(a.q + (size_t)line * HD + c * 8);
        *reinterpret_cast<uint4*>(sQ + (c >> 3) * (ROWS * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4)) = q;
      }
      math_barrier<NTH>();
      // keys that every row sees lie in [in_lo, in_hi)
      const int in_lo = b == a.batch ? (a.window ? a.P : 0) : (a.window ? max(0, f.s.len - a.window) : 0);
      const int in_hi = b == a.batch ? a.P : f.s.len - f.s.n + 1;
      const int in_lo_p = a.window ? a.P + f.s.len - a.window : 0;  // (of the prefix)
      float o[NT][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
      for (int c = 0; c < NT; ++c) o[c][0] = o[c][1] = o[c][2] = o[c][3] = 0.f;
      const bool busy = mt < nmt;
#pragma unroll 1
      for (int i = 0; i < nt; ++i) {
        // (on a failed wait the warps still meet at the barriers below)
        if (!__all_sync(0xffffffffu, sh_wait(full + st, phase, abort_flag, a.err))) ok = false;
        const uint32_t sK = ring + st * 2 * KV, sV = sK + KV;
        const FewSpan sp = few_span(a, f, b, t0 + i);
        const bool ahead = t0 + i < f.p_tiles;  // in the prefix ahead of the own positions
        const int kb = sp.kb, k0 = kb + 16 * kq;
        if (kb < sp.lo || kb + 64 > sp.hi) {
          // values that no row sees must be finite (0 x NaN): clear them
          const int row = lane >> 1, key = k0 + row;
          if (key < sp.lo || key >= sp.hi) {
#pragma unroll
            for (int c = 0; c < HD / 16; ++c) {
              const int ch = (lane & 1) * (HD / 16) + c;
              *reinterpret_cast<uint4*>(sm + st * 2 * KV + KV + (ch >> 3) * (64 * 128) + (16 * kq + row) * 128 +
                                        ((ch & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
            }
          }
          fence_proxy_async();  // before the stage is refilled
          __syncwarp();
        }
        if (busy) {
          float s[2][4] = {};
#pragma unroll
          for (int ks = 0; ks < HD / 16; ++ks) {
            uint32_t kf[4], qf[4];
            ldsm4(kf, ((sK + k_off) ^ ((ks & 3) << 5)) + (ks >> 2) * (64 * 128));
            ldsm4(qf, (q_at ^ ((ks & 3) << 5)) + (ks >> 2) * (ROWS * 128));
            mma_16816(s[0], qf[0], qf[1], qf[2], qf[3], kf[0], kf[1]);
            mma_16816(s[1], qf[0], qf[1], qf[2], qf[3], kf[2], kf[3]);
          }
          const bool edge = ahead ? kb < in_lo_p || kb + 64 > a.P : kb < in_lo || kb + 64 > in_hi;
          uint32_t ph[4], pl[4];
#pragma unroll
          for (int rr = 0; rr < 2; ++rr) {
            float z0 = s[0][2 * rr], z1 = s[0][2 * rr + 1], z2 = s[1][2 * rr], z3 = s[1][2 * rr + 1];
            if (edge) {
              const int row = 16 * mt + g + 8 * rr, off = k0 + 2 * tq;
              const int lo = (ahead ? s_vlo_p[row] : s_vlo[row]) - off, hi = (ahead ? a.P : s_vhi[row]) - off;
              z0 = (0 >= lo && 0 < hi) ? z0 : -INFINITY;
              z1 = (1 >= lo && 1 < hi) ? z1 : -INFINITY;
              z2 = (8 >= lo && 8 < hi) ? z2 : -INFINITY;
              z3 = (9 >= lo && 9 < hi) ? z3 : -INFINITY;
            }
            float M = fmaxf(fmaxf(z0, z1), fmaxf(z2, z3));
            M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 1));
            M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 2)) * a.scale_log2;
            if (M > m[rr] + RESCALE) {
              const float al = exp2f(m[rr] - M);
              m[rr] = M;
              l[rr] *= al;
#pragma unroll
              for (int c = 0; c < NT; ++c) {
                o[c][2 * rr] *= al;
                o[c][2 * rr + 1] *= al;
              }
            }
            const float nref = m[rr] == -INFINITY ? 0.f : -m[rr];
            const float p0 = ex2_fast(fmaf(z0, a.scale_log2, nref)), p1 = ex2_fast(fmaf(z1, a.scale_log2, nref));
            const float p2 = ex2_fast(fmaf(z2, a.scale_log2, nref)), p3 = ex2_fast(fmaf(z3, a.scale_log2, nref));
            l[rr] += (p0 + p1) + (p2 + p3);
            const uint32_t h0 = cvt_bf16x2(p0, p1), h1 = cvt_bf16x2(p2, p3);
            ph[rr] = h0;
            ph[2 + rr] = h1;
            if (C::LO) {
              pl[rr] = cvt_bf16x2(p0 - __uint_as_float(h0 << 16), p1 - __uint_as_float(h0 & 0xffff0000u));
              pl[2 + rr] = cvt_bf16x2(p2 - __uint_as_float(h1 << 16), p3 - __uint_as_float(h1 & 0xffff0000u));
            }
          }
#pragma unroll
          for (int p = 0; p < HD / 16; ++p) {
            uint32_t vf[4];
            ldsm4_t(vf, ((sV + v_off) ^ ((p & 3) << 5)) + (p >> 2) * (64 * 128));
            mma_16816(o[2 * p], ph[0], ph[1], ph[2], ph[3], vf[0], vf[1]);
            mma_16816(o[2 * p + 1], ph[0], ph[1], ph[2], ph[3], vf[2], vf[3]);
            if (C::LO) {
              mma_16816(o[2 * p], pl[0], pl[1], pl[2], pl[3], vf[0], vf[1]);
              mma_16816(o[2 * p + 1], pl[0], pl[1], pl[2], pl[3], vf[2], vf[3]);
            }
          }
        }
        if (C::SCR || i + 1 < nt) {
          __syncwarp();
          if (lane == 0) mbar_arrive(empty + st);
          if (++st == NST) {
            st = 0;
            phase ^= 1;
          }
        }
      }
      // ---- the piece: the four key quarters of each m-tile joined, [quarter]
      // [16 rows][HD] fp32 (16-byte chunks flipped by the row), then written ----
      float* sx = reinterpret_cast<float*>(C::SCR ? sQ + C::QB : sm + st * 2 * KV);
      const bool first = t0 == 0, whole = first && nt == f.tiles - a.setup && b < a.batch && a.ns_prefix == 0;
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        l[rr] += __shfl_xor_sync(0xffffffffu, l[rr], 1);
        l[rr] += __shfl_xor_sync(0xffffffffu, l[rr], 2);
      }
      math_barrier<NTH>();  // the stage has been read
      if (busy) {
        float* sx1 = sx + (C::SCR ? mt * 64 * HD : 0);
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {
          const int row = g + 8 * rr;
          float* d = sx1 + (kq * 16 + row) * HD;
          // (the flip reaches bits 2 to 4 of a column: four bases, 32 columns apart from there)
#pragma unroll
          for (int c1 = 0; c1 < 4; ++c1) {
            float* d1 = d + ((8 * c1 + 2 * tq) ^ (g << 2));
#pragma unroll
            for (int c = c1; c < NT; c += 4)
              *reinterpret_cast<float2*>(d1 + 8 * (c - c1)) = make_float2(o[c][2 * rr], o[c][2 * rr + 1]);
          }
          if (tq == 0) s_ml[C::SCR ? mt : 0][kq][row] = make_float2(m[rr], l[rr]);
        }
      }
      math_barrier<NTH>();
      {
        constexpr int CPR = HD / 4;  // 16-byte chunks of a row
#pragma unroll 2
        for (int it = tid; it < nrow * CPR; it += NTH) {
          const int pr = it / CPR, c4 = it - pr * CPR, row = pr & 15, jt = C::SCR ? pr >> 4 : 0;
          float2 ml[4];
          float4 x[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            ml[k] = s_ml[jt][k][row];
            x[k] = *reinterpret_cast<const float4*>(sx + ((jt * 4 + k) * 16 + row) * HD + ((c4 * 4) ^ ((row & 7) << 2)));
          }
          const float M = fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x));
          float L = 0.f;
          float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float f = ml[k].x == -INFINITY ? 0.f : exp2f(ml[k].x - M);
            L = fmaf(ml[k].y, f, L);
            y = make_float4(fmaf(x[k].x, f, y.x), fmaf(x[k].y, f, y.y), fmaf(x[k].z, f, y.z), fmaf(x[k].w, f, y.w));
          }
          if (!ok) continue;
          const size_t line = size_t(s_line[pr]);
          if (whole) {
            const float inv = 1.f / L;
            *reinterpret_cast<uint2*>(a.out + line * HD + c4 * 4) =
                make_uint2(cvt_bf16x2(y.x * inv, y.y * inv), cvt_bf16x2(y.z * inv, y.w * inv));
          } else {
            const size_t at = first ? (size_t)(b == a.batch ? 0 : a.ns_prefix) * a.rows * a.nq + line
                                    : (size_t)cta * a.few + pr;
            *reinterpret_cast<float4*>((first ? a.o_part : a.o_cont) + at * HD + c4 * 4) = y;
            if (c4 == 0) (first ? a.ml_part : a.ml_cont)[at] = make_float2(M, L);
          }
        }
      }
      fence_proxy_async();  // the stage is refilled by tensor copies
      math_barrier<NTH>();  // and the rows' bounds and Q are free again
      if (!C::SCR) {
        if (lane == 0) mbar_arrive(empty + st);
        if (++st == NST) {
          st = 0;
          phase ^= 1;
        }
      }
    }
  }
  wait_previous_kernel();
}

// ---------------------------------------------------------------------------
// join_kernel: CTA = one head and `tpc` of the tokens with pieces to join (not
// those that tc_kernel has finished), `wpt` warps per token at a time, each
// with every wpt-th piece.
// Where a token's pieces are is worked out before the wait for them (the
// stream's cut again, from the lengths), while they are still being made;
// behind the wait a lane takes a piece's (m, l), then the pieces' O come in
// rounds of eight.
// ---------------------------------------------------------------------------
constexpr int JT = 256, JCH = 8;

template <int HD>
__global__ void __launch_bounds__(JT) join_kernel(const __grid_constant__ ShArgs a, const int tpc, const int wpt) {
  extern __shared__ int s_start[];        // tokens to join before each sequence [batch + 1], then the stream's tiles
  int* cum = s_start + a.batch + 1;       // [batch + 2]
  __shared__ int s_warp[JT / 32], s_tok[JT / 32], s_lo;
  __shared__ float s_acc[JT / 32][HD];
  __shared__ float2 s_ml[JT / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int head = blockIdx.y, kvh = head / a.gq, g = head - kvh * a.gq;
  if (tid == 0) {
    cum[0] = 0;
    s_lo = 0x7fffffff;
    s_start[0] = 0;
  }
  __syncthreads();
  int before = 0, toks = 0;
#pragma unroll 1
  for (int c0 = 0; c0 < a.batch; c0 += JT) {
    int t = 0, nt = 0;
    if (c0 + tid < a.batch) {
      FewSeq f;
      f.s = load_seq(a, c0 + tid);
      few_tiles(a, f);
      t = f.tiles;
      if (!a.own_joins || f.s.n * a.gq <= a.few) nt = f.s.n;
      if (a.prefix_few && f.s.n > 0) atomicMin(&s_lo, a.P + f.s.len - f.s.n);
    }
    int incl = t, itok = nt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, incl, o), v = __shfl_up_sync(0xffffffffu, itok, o);
      if (lane >= o) {
        incl += u;
        itok += v;
      }
    }
    if (lane == 31) {
      s_warp[warp] = incl;
      s_tok[warp] = itok;
    }
    __syncthreads();
    incl += before;
    itok += toks;
#pragma unroll
    for (int w = 0; w < JT / 32; ++w) {
      if (w < warp) {
        incl += s_warp[w];
        itok += s_tok[w];
      }
      before += s_warp[w];
      toks += s_tok[w];
    }
    if (c0 + tid < a.batch) {
      cum[c0 + tid + 1] = incl;
      s_start[c0 + tid + 1] = itok;
    }
    __syncthreads();
  }
  const int ptiles = few_prefix_tiles(a, s_lo), px = before * a.nkv + kvh * ptiles;
  const Runs runs((before + ptiles) * a.nkv, a.G);
  bool waited = false;
  int tok = 0;
  const int x1 = min(toks, int(blockIdx.x + 1) * tpc), share = warp & (wpt - 1);
  // (with wpt > 1 a CTA has one round: tpc = JT / 32 / wpt)
  for (int x = blockIdx.x * tpc + warp / wpt; x < x1; x += JT / 32 / wpt) {
    if (wpt > 1 && lane == 0) s_ml[warp] = make_float2(-INFINITY, -1.f);  // nothing to join
    int b = 0, hi = a.batch;
    while (hi - b > 1) {
      const int mid = (b + hi) >> 1;
      if (s_start[mid] <= x)
        b = mid;
      else
        hi = mid;
    }
    const Seq s = load_seq(a, b);
    tok = s.r0 + x - s_start[b];
    const bool few = s.n * a.gq <= a.few;
    // the pieces: slots [first, first + in_slots), then the CTAs [c0, c0 + nc)
    // of the own positions and [p0, p0 + np) of the prefix
    int first = 0, in_slots = a.ns_prefix + (few ? 1 : a.ns_own), c0 = 0, nc = 0, p0 = 0, np = 0;
    if (few) {
      const int tiles = cum[b + 1] - cum[b], at = cum[b] * a.nkv + kvh * tiles;
      c0 = runs.of(at + a.setup) + 1;
      nc = runs.of(at + tiles - 1) + 1 - c0;
      if (a.ns_prefix == 0 && nc == 0) continue;  // written already
    }
    if (a.prefix_few) {
      if (ptiles == 0) {
        first = 1;  // the window ends behind the prefix: slot 0 was not written
        --in_slots;
      } else {
        p0 = runs.of(px + a.setup) + 1;
        np = runs.of(px + ptiles - 1) + 1 - p0;
      }
    }
    // prefix rows behind the last whole pair tile have fewer pieces: the slots from ns_rest to ns_prefix are not theirs
    const int gap = a.ns_prefix - (tok * a.gq + g >= (a.rows * a.gq & ~(TC_ROWS - 1)) ? a.ns_rest : a.ns_prefix);
    in_slots -= gap;
    const int cut = a.ns_prefix - gap;
    const int total = in_slots + nc + np, crow = (tok - s.r0) * a.gq + g, prow = tok * a.gq + g;
    const size_t line = (size_t)tok * a.nq + head;
    if (!waited) wait_previous_kernel();
    waited = true;
    constexpr int E = HD / 32;
    float acc[E] = {}, L = 0.f, M = -INFINITY;
#pragma unroll 1
    for (int i0 = 0; i0 < total; i0 += 32 * wpt) {
      // a lane's piece: where, and its weight (the address arithmetic of 32
      // pieces at once: a warp by itself takes ~5 clocks an instruction)
      const int i1 = i0 + lane * wpt + share, i = min(i1, total - 1);
      const bool slot = i < in_slots, mine = i < in_slots + nc;
      const size_t at = slot ? (size_t)(first + i + (i >= cut ? gap : 0)) * a.rows * a.nq + line
                             : (size_t)((mine ? c0 + i - in_slots : p0 + i - in_slots - nc) * a.few + (mine ? crow : prow));
      const float2 ml = (slot ? a.ml_part : a.ml_cont)[at];
      const float* src = (slot ? a.o_part : a.o_cont) + at * HD;
      const bool there = i1 < total && ml.y != 0.f;
      float m = there ? ml.x : -INFINITY;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (m > M) {
        const float f = exp2f(M - m);
        M = m;
        L *= f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] *= f;
      }
      const float w = there ? exp2f(ml.x - M) : -1.f;  // (-1: nothing there; a weight may be 0 or NaN)
      if (there) L = fmaf(ml.y, w, L);  // this lane's share; summed below
      const int n32 = min(32, (total - i0 - share + wpt - 1) / wpt);
#pragma unroll 1
      for (int k0 = 0; k0 < n32; k0 += JCH) {
        float x[JCH][E];
#pragma unroll
        for (int k = 0; k < JCH; ++k) {
          // (an index past the last piece is read as that piece, with weight -1)
          const float* s_k = reinterpret_cast<const float*>(
              __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), k0 + k)) + lane * E;
          if (E == 4)
            *reinterpret_cast<float4*>(x[k]) = *reinterpret_cast<const float4*>(s_k);
          else
            *reinterpret_cast<float2*>(x[k]) = *reinterpret_cast<const float2*>(s_k);
        }
#pragma unroll
        for (int k = 0; k < JCH; ++k) {
          const float f = __shfl_sync(0xffffffffu, w, k0 + k);
          // an empty piece's O was not written
#pragma unroll
          for (int e = 0; e < E; ++e) acc[e] = f < 0.f ? acc[e] : fmaf(x[k][e], f, acc[e]);
        }
      }
    }
    // the lanes' shares of L in a fixed order
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    if (wpt > 1) {
#pragma unroll
      for (int e = 0; e < E; ++e) s_acc[warp][lane * E + e] = acc[e];
      if (lane == 0) s_ml[warp] = make_float2(M, L);
    } else {
      const float inv = 1.f / L;
      uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + line * HD + lane * E);
#pragma unroll
      for (int e = 0; e < E; e += 2) dst[e / 2] = cvt_bf16x2(acc[e] * inv, acc[e + 1] * inv);
    }
  }
  if (!waited) wait_previous_kernel();
  if (wpt > 1) {
    // the shares of a token's warps, in order
    __syncthreads();
    const int x = blockIdx.x * tpc + warp / wpt, w0 = warp - share;
    if (share != 0 || x >= x1 || s_ml[w0].y < 0.f) return;
    float M = -INFINITY, L = 0.f;
    for (int w = 0; w < wpt; ++w) M = fmaxf(M, s_ml[w0 + w].x);
    constexpr int E = HD / 32;
    float acc[E] = {};
    for (int w = 0; w < wpt; ++w) {
      const float2 ml = s_ml[w0 + w];
      const float f = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);
      L = fmaf(ml.y, f, L);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(s_acc[w0 + w][lane * E + e], f, acc[e]);
    }
    const float inv = 1.f / L;
    uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + ((size_t)tok * a.nq + head) * HD + lane * E);
#pragma unroll
    for (int e = 0; e < E; e += 2) dst[e / 2] = cvt_bf16x2(acc[e] * inv, acc[e + 1] * inv);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static const EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}

// One layer's pages [n_pages * nkv][page][hd] as boxes of 64 dims x rows keys, 128-byte swizzle.
cudaError_t page_map(CUtensorMap* m, const void* base, int hd, int page, int64_t blocks, int rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {cuuint64_t(hd), cuuint64_t(page), cuuint64_t(blocks)};
  const cuuint64_t strides[2] = {cuuint64_t(hd) * 2, cuuint64_t(page) * hd * 2};
  const cuuint32_t box[3] = {64u, cuuint32_t(rows), 1u};
  const cuuint32_t es[3] = {1, 1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

struct ShLayout {
  size_t ml_part, ml_cont, o_cont, o_part, total;
};
ShLayout shared_layout(const ShPlan& p, int rows, int nq, int hd) {
  auto al = [](size_t x) { return (x + 255) & ~size_t(255); };
  ShLayout L;
  const size_t parts = p.prefix_cap + p.own_cap, lines = parts * rows * nq;
  L.ml_part = 256;
  L.ml_cont = L.ml_part + al(lines * 8);
  L.o_cont = L.ml_cont + al((size_t)p.G * p.few * 8);
  L.o_part = L.o_cont + al((size_t)p.G * p.few * hd * 4);
  L.total = L.o_part + al(lines * hd * 4);
  return L;
}

// Every launch may start before the one in front of it in the stream has
// finished (the kernels wait for it where they need it).
cudaError_t launch(const void* fn, SmemMark& mark, dim3 grid, unsigned threads, int smem, void** args, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = allow_smem(fn, smem, mark);
  if (e != cudaSuccess) return e;
  return cudaLaunchKernelExC(&cfg, fn, args);
}

template <int HD>
cudaError_t launch_shared(ShArgs a, const uint16_t* k, const uint16_t* v, const ShPlan& p, int sms, cudaStream_t st) {
  const int page = 1 << a.page_log2;
  const int64_t blocks = (int64_t)a.n_pages * a.nkv;
  CUtensorMap k128, v128, k64, v64;
  cudaError_t e;
  const bool tc_prefix = a.ns_prefix > 0 && !a.prefix_few;
  if (tc_prefix || p.many) {
    if ((e = page_map(&k128, k, HD, page, blocks, page < 128 ? page : 128)) != cudaSuccess) return e;
    if ((e = page_map(&v128, v, HD, page, blocks, page < 128 ? page : 128)) != cudaSuccess) return e;
  }
  if ((e = page_map(&k64, k, HD, page, blocks, page < 64 ? page : 64)) != cudaSuccess) return e;
  if ((e = page_map(&v64, v, HD, page, blocks, page < 64 ? page : 64)) != cudaSuccess) return e;
  static SmemMark tc_mark, few_mark[3], join_mark;
  int lead = 1;  // the call's first launch
  for (int own = 0; own < 2; ++own) {
    if (own ? !p.many : !tc_prefix) continue;
    const long long items = own ? p.own_items * a.ns_own : p.pairs * a.ns_prefix + p.rest * a.ns_rest;
    void* args[] = {&k128, &v128, &a, &own, &lead};
    e = launch(reinterpret_cast<const void*>(&tc_kernel<HD>), tc_mark, dim3(unsigned(items)), TC_THREADS, Tc<HD>::SMEM, args, st);
    if (e != cudaSuccess) return e;
    lead = 0;
  }
  {
    void* args[] = {&k64, &v64, &a, &lead};
    using F1 = Fw<HD, 1>;
    using F2 = Fw<HD, 2>;
    using F3 = Fw<HD, 3>;
    const void* fn = p.few == 16   ? reinterpret_cast<const void*>(&few_kernel<HD, 1>)
                     : p.few == 32 ? reinterpret_cast<const void*>(&few_kernel<HD, 2>)
                                   : reinterpret_cast<const void*>(&few_kernel<HD, 3>);
    const int smem = p.few == 16 ? F1::SMEM : (p.few == 32 ? F2::SMEM : F3::SMEM);
    const int threads = p.few == 16 ? F1::THREADS : (p.few == 32 ? F2::THREADS : F3::THREADS);
    e = launch(fn, few_mark[p.few / 16 - 1], dim3(unsigned(a.G)), threads, smem, args, st);
    if (e != cudaSuccess) return e;
  }
  // The join: four warps a token while the (token, head) pairs do not fill the
  // SMs, else a warp.
  // The tokens that may have pieces: all, or those of sequences with few rows
  // (a prompt of 8,192: 714 us with a grid over all of them, 669 over nine).
  const long long most = (long long)a.batch * (a.few / a.gq);
  const int toks = a.own_joins && most < a.rows ? int(most) : a.rows;
  const int wpt = toks <= 256 && (long long)toks * a.nq <= 16LL * sms ? 4 : 1;
  long long tpc_l = (long long)toks * a.nq / (8LL * sms) / 8 * 8;  // about eight CTAs an SM
  if (tpc_l > 64) tpc_l = 64;
  const int tpc = wpt > 1 ? JT / 32 / wpt : (tpc_l < 8 ? 8 : int(tpc_l));
  void* args[] = {&a, const_cast<int*>(&tpc), const_cast<int*>(&wpt)};
  return launch(reinterpret_cast<const void*>(&join_kernel<HD>), join_mark,
                dim3(unsigned((toks + tpc - 1) / tpc), unsigned(a.nq)), JT, (2 * a.batch + 3) * 4, args, st);
}

}  // namespace

size_t attn_shared_ws(int rows, int batch, int nq, int nkv, int hd, int max_new, int sms) {
  return shared_layout(shared_plan(rows, batch, nq, nkv, max_new, sms), rows, nq, hd).total;
}

cudaError_t launch_attn_shared(const uint16_t* q, int rows, int batch, int nq, int nkv, int hd, const uint16_t* k,
                               const uint16_t* v, int n_pages, int page, const int32_t* row_start, const int32_t* lens,
                               const int32_t* table, int width, const int32_t* ptable, int P, int window, int max_new,
                               uint16_t* out, uint8_t* ws, int sms, cudaStream_t st) {
  const ShPlan p = shared_plan(rows, batch, nq, nkv, max_new, sms);
  const ShLayout L = shared_layout(p, rows, nq, hd);
  ShArgs a;
  a.q = q;
  a.row_start = row_start;
  a.lens = lens;
  a.table = table;
  a.ptable = ptable;
  a.out = out;
  a.err = reinterpret_cast<uint32_t*>(ws) + 2;
  a.ml_part = reinterpret_cast<float2*>(ws + L.ml_part);
  a.ml_cont = reinterpret_cast<float2*>(ws + L.ml_cont);
  a.o_cont = reinterpret_cast<float*>(ws + L.o_cont);
  a.o_part = reinterpret_cast<float*>(ws + L.o_part);
  a.rows = rows;
  a.batch = batch;
  a.nq = nq;
  a.nkv = nkv;
  a.gq = nq / nkv;
  a.n_pages = n_pages;
  a.page_log2 = 0;
  while ((1 << a.page_log2) < page) ++a.page_log2;
  a.width = width;
  a.P = P;
  a.window = window;
  a.max_new = max_new;
  a.few = p.few;
  const ShChoice c = shared_choice(p, batch, nkv, hd, page, width, P, window, max_new, sms);
  a.setup = c.setup;
  a.with_prefix = c.with_prefix;
  a.prefix_few = c.prefix_few;
  a.ns_prefix = c.ns_prefix;
  a.ns_rest = c.ns_rest;
  a.ns_own = c.ns_own;
  a.own_joins = c.own_joins;
  a.G = c.G;
  a.scale_log2 = float(1.4426950408889634 / sqrt(double(hd)));
  return hd == 64 ? launch_shared<64>(a, k, v, p, sms, st) : launch_shared<128>(a, k, v, p, sms, st);
}

}  // namespace w4a
