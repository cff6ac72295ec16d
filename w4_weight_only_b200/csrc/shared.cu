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
// sum l 2^(m - M).  So the work is cut twice: the prefix apart from the own
// positions, because all rows share its keys, and both along the keys, to
// fill the SMs when there are few rows.
//
//  - tc_kernel: tcgen05, tiles of 128 packed rows (row x query heads of one
//    KV head) by 128 keys.  The prefix for all rows of the batch, and the own
//    positions of the sequences with many rows.
//  - few_kernel: mma.sync, at most 16 packed rows: the own positions of the
//    sequences with few rows (decode), read at memory speed.
//  - join_kernel: joins the pieces of each (row, head).
// They are launched one behind the other and overlap (each may start when the
// one before has started); the join waits for all.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "ptx.cuh"
#include "tc.cuh"
#include "w4a_internal.h"

namespace w4a {

namespace {

constexpr long long SH_WAIT = 4000000000LL;  // bound on any single wait (~2 s)
constexpr int FEW = 16;                      // packed rows of a sequence that few_kernel takes
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
  float* o_cont;        // [G][FEW][HD]: pieces that begin inside a segment
  float2* ml_cont;      // [G][FEW]
  int32_t* cum;         // [batch + 2]: few_kernel's key tiles before each sequence
  int rows, batch, nq, nkv, gq, n_pages, page_log2, width, P, window, max_new;
  int ns_prefix;        // pieces of the prefix (slots 0 ..), 0 without one
  int ns_own;           // pieces of the own positions in tc_kernel (slots ns_prefix ..)
  int prefix_few;       // 1: few_kernel takes the prefix too (few packed rows in all)
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
template <int HD, int ROWS>
__device__ __forceinline__ uint32_t load_blocks(int kb, int key_end, int page_log2) {
  const int bs = min(1 << page_log2, ROWS);
  return uint32_t((min(ROWS, key_end - kb) + bs - 1) / bs);  // blocks of bs keys to copy
}
template <int HD, int ROWS>
__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* map, const int32_t* pages, int kb,
                                          int key_end, int kvh, uint64_t* bar, const ShArgs& a, int lane) {
  constexpr int PANELS = HD / 64;
  const int bs = min(1 << a.page_log2, ROWS);
  const int nblk = int(load_blocks<HD, ROWS>(kb, key_end, a.page_log2));
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
//        parity i, and the groups' pieces are joined at the end.
// S_i = Q K^T into TMEM columns [128 i, + 128); the group reads its rows,
// forms P = 2^(s - m) and writes it back as bf16 pairs over the first 64 of
// the same columns (head_dim 64: next to O), where the second MMA reads it as
// its A operand: O_i += P V, V as an MN-major operand.  The reference m moves
// only when the maximum has risen by more than 2^8 over it, so O is rescaled
// rarely; P <= 2^8 is rounded to bf16, 2^-8 of each weight at most, while l
// sums the weights unrounded in fp32.
template <int HD, bool ALT>
struct Tc {
  static constexpr int TILE = 128 * HD * 2;                 // 128 rows, bytes
  static constexpr int PANEL = 128 * 128;
  static constexpr int NQ = ALT ? 1 : 2;
  static constexpr int NS = HD == 128 ? (ALT ? 5 : 4) : 8;  // K / V ring slots
  static constexpr int ROWS = NQ * 128;
  static constexpr int BARS = 256;
  static constexpr int SMEM = (NQ + NS) * TILE + BARS + 1024;
  static constexpr int O_COL = 256;                         // O_i at 256 + i HD
  static constexpr int P_COL(int i) { return HD == 128 ? i * 128 : 384 + i * 64; }
};
constexpr int TC_THREADS = 320;

template <int HD, bool ALT>
__global__ void __launch_bounds__(TC_THREADS, 1)
    tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
              const __grid_constant__ ShArgs a, const int own) {
  using C = Tc<HD, ALT>;
  constexpr int NS = C::NS, TILE = C::TILE, PANEL = C::PANEL;
  extern __shared__ uint8_t tc_raw[];
  uint8_t* sm = tc_raw + ((1024u - (smem_addr(tc_raw) & 1023u)) & 1023u);
  uint8_t* sQ = sm;
  uint8_t* sR = sm + C::NQ * TILE;
  uint64_t* q_full = reinterpret_cast<uint64_t*>(sR + NS * TILE);
  uint64_t* kv_full = q_full + 1;        // [NS]
  uint64_t* kv_empty = kv_full + NS;     // [NS]
  uint64_t* s_full = kv_empty + NS;      // [2]: S_i computed (and every earlier MMA done)
  uint64_t* p_full = s_full + 2;         // [2]: P_i written, O_i rescaled (4 warps arrive)
  uint64_t* o_done = p_full + 2;
  uint32_t* tbase = reinterpret_cast<uint32_t*>(o_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tbase + 1);
  int* s_lo = reinterpret_cast<int*>(tbase + 2);
  int* s_hi = s_lo + 1;
  int* s_b = s_hi + 1;      // sequence and its first tile
  int* s_warp = s_b + 2;    // [8]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  launch_dependents();

  // ---- which item: KV head, rows [base, base + valid) of the packed rows of
  // tokens r0 .., piece of the keys ----
  int kvh, piece, ns, base, valid, r0, b = 0, n = 0, len = 0;
  if (!own) {
    const int packed = total_rows(a) * a.gq;
    const int ntile = (a.rows * a.gq + C::ROWS - 1) / C::ROWS;
    int x = blockIdx.x;
    base = (x % ntile) * C::ROWS;
    x /= ntile;
    kvh = x % a.nkv;
    piece = x / a.nkv;
    ns = a.ns_prefix;
    r0 = 0;
    valid = min(C::ROWS, packed - base);
  } else {
    int x = blockIdx.x;
    ns = a.ns_own;
    piece = x % ns;
    x /= ns;
    kvh = x % a.nkv;
    const int want = x / a.nkv;  // tile of the sequences with many rows, in order
    if (tid == 0) s_b[0] = -1;
    int before = 0;
#pragma unroll 1
    for (int c0 = 0; c0 < a.batch; c0 += 256) {
      int t = 0;
      if (tid < 256 && c0 + tid < a.batch) {
        const Seq s = load_seq(a, c0 + tid);
        if (s.n * a.gq > FEW) t = (s.n * a.gq + C::ROWS - 1) / C::ROWS;
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
      const int nt = (n * a.gq + C::ROWS - 1) / C::ROWS;
      base = (nt - 1 - (want - s_b[1])) * C::ROWS;  // the longest rows first
      valid = min(C::ROWS, n * a.gq - base);
    }
  }
  if (valid <= 0) {  // uniform: nothing here
    wait_previous_kernel();
    return;
  }

  if (tid == 0) {
    mbar_init(q_full, 8);
#pragma unroll 1
    for (int s = 0; s < NS; ++s) {
      mbar_init(kv_full + s, 1);
      mbar_init(kv_empty + s, 1);
    }
    mbar_init(s_full + 0, 1);
    mbar_init(s_full + 1, 1);
    mbar_init(p_full + 0, 4);
    mbar_init(p_full + 1, 4);
    mbar_init(o_done, 1);
    *abort_flag = 0;
    *s_lo = 0x7fffffff;
    *s_hi = 0;
    fence_mbar_init();
    tma_prefetch_map(&tmK);
    tma_prefetch_map(&tmV);
  }
  if (warp == 9) {
    tmem_alloc(tbase, 512);
    tmem_relinquish();
  }
  __syncthreads();
  // ---- this thread's row: token, head, visible keys [vlo, vhi) (prefix
  // positions, or own positions) ----
  const int grp = (warp >> 2) & 1, r = (warp & 3) * 32 + lane;
  const int prow = base + (ALT ? 0 : grp * 128) + r;
  const bool live = warp < 8 && prow < base + valid;
  const int tok = live ? r0 + prow / a.gq : 0, head = kvh * a.gq + (live ? prow % a.gq : 0);
  int vlo = 0, vhi = 0;
  if (live) {
    if (own) {
      const int p = len - n + prow / a.gq;  // own position of the row
      vhi = p + 1;
      if (a.window) vlo = max(0, p - a.window + 1);
    } else {
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
    if (vlo < vhi) {
      atomicMin(s_lo, vlo);
      atomicMax(s_hi, vhi);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tbase;
  const int k_lo = *s_lo, k_hi = *s_hi;  // keys that some row of the item sees
  int t0 = 0, nb = 0;
  if (k_lo < k_hi) {
    const int f = k_lo >> 7, nt = ((k_hi + 127) >> 7) - f;
    t0 = f + int((long long)nt * piece / ns);
    nb = f + int((long long)nt * (piece + 1) / ns) - t0;
  }
  const int groups = (ALT ? nb > 1 : valid > 128) ? 2 : 1;
  const int32_t* pages = own ? a.table + (size_t)b * a.width : a.ptable;

  if (warp == 8) {
    // ---- loads, in the order in which the MMAs use them: K_0 (K_1) V_0 K_2 V_1 .. (ALT), K_0 V_0 K_1 V_1 .. (PAIR)
    uint32_t it = 0;
    bool ok = true;
    auto put = [&](const CUtensorMap* map, int t) {
      if (!ok) return;
      const int s = int(it % NS);
      if (it >= uint32_t(NS)) {
        int good = 1;
        if (lane == 0) good = sh_wait(kv_empty + s, ((it / NS) - 1u) & 1u, abort_flag, a.err) ? 1 : 0;
        if (!__shfl_sync(0xffffffffu, good, 0)) {
          ok = false;
          return;
        }
      }
      const int kb = (t0 + t) * 128;
      const int bs = min(1 << a.page_log2, 128);
      if (lane == 0) mbar_expect_tx(kv_full + s, load_blocks<HD, 128>(kb, k_hi, a.page_log2) * bs * HD * 2);
      __syncwarp();
      load_tile<HD, 128>(sR + s * TILE, map, pages, kb, k_hi, kvh, kv_full + s, a, lane);
      ++it;
    };
    if (ALT) {
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
      const uint32_t first = it > uint32_t(NS) ? it - NS : 0u;
#pragma unroll 1
      for (uint32_t j = first; j < it; ++j) sh_drain(kv_full + (j % NS), (j / NS) & 1u, a.err);
    }
  } else if (warp == 9) {
    // ---- MMAs (one thread) ----
    if (lane == 0 && nb > 0) {
      const uint32_t idS = umma_idesc_f16(128, 128, true);
      const uint32_t idO = umma_idesc_f16(128, HD, true) | UMMA_B_MN;
      auto ready = [&](uint32_t i) {
        const bool w = sh_wait(kv_full + i % NS, (i / NS) & 1u, abort_flag, a.err);
        tc_fence_after();
        return w;
      };
      auto issue_s = [&](int qi, uint32_t ki) {
        const uint8_t* q = sQ + (ALT ? 0 : qi) * TILE;
        const uint8_t* k = sR + (ki % NS) * TILE;
#pragma unroll
        for (int ks = 0; ks < HD / 16; ++ks) {
          const uint32_t off = uint32_t((ks >> 2) * PANEL + (ks & 3) * 32);
          umma_f16(tmem + uint32_t(qi * 128), umma_desc_sw128(q, off), umma_desc_sw128(k, off), idS, ks > 0 ? 1u : 0u);
        }
        umma_commit(s_full + qi);
      };
      auto issue_pv = [&](int qi, uint32_t vi, bool first) {
        const uint8_t* v = sR + (vi % NS) * TILE;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          umma_f16_ts(tmem + uint32_t(C::O_COL + qi * HD), tmem + uint32_t(C::P_COL(qi) + ks * 8),
                      umma_desc_mn_sw128(v + ks * 16 * 128, PANEL, 1024), idO, (first && ks == 0) ? 0u : 1u);
      };
      auto p_ready = [&](int qi, int j) {
        const bool w = sh_wait(p_full + qi, uint32_t(j) & 1u, abort_flag, a.err);
        tc_fence_after();
        return w;
      };
      bool ok = sh_wait(q_full, 0u, abort_flag, a.err);
      uint32_t it = 0;
      if (ALT) {
        for (int t = 0; t < 2 && t < nb && ok; ++t) {
          ok = ready(it);
          if (!ok) break;
          issue_s(t, it);
          umma_commit(kv_empty + it % NS);
          ++it;
        }
#pragma unroll 1
        for (int t = 0; t < nb && ok; ++t) {
          if (!(ok = ready(it) && p_ready(t & 1, t >> 1))) break;
          issue_pv(t & 1, it, t < 2);
          umma_commit(kv_empty + it % NS);
          ++it;
          if (t + 2 < nb) {
            if (!(ok = ready(it))) break;
            issue_s(t & 1, it);
            umma_commit(kv_empty + it % NS);
            ++it;
          }
        }
      } else {
        if (ok && (ok = ready(0))) {
          issue_s(0, 0);
          if (groups == 2) issue_s(1, 0);
          umma_commit(kv_empty + 0);
        }
#pragma unroll 1
        for (int j = 0; j < nb && ok; ++j) {
          const uint32_t vt = 2u * j + 1u, kn = 2u * j + 2u;
          const bool more = j + 1 < nb;
          if (!(ok = ready(vt) && p_ready(0, j))) break;
          issue_pv(0, vt, j == 0);
          if (more) {
            if (!(ok = ready(kn))) break;
            issue_s(0, kn);
          }
          if (groups == 2) {
            if (!(ok = p_ready(1, j))) break;
            issue_pv(1, vt, j == 0);
            umma_commit(kv_empty + vt % NS);
            if (more) issue_s(1, kn);
          } else {
            umma_commit(kv_empty + vt % NS);
          }
          if (more) umma_commit(kv_empty + kn % NS);
        }
      }
      umma_commit(o_done);
      // every MMA issued has completed before the tensor memory is freed
      sh_drain(o_done, 0u, a.err);
    }
  } else {
    // ---- the rows of Q into shared memory (128-byte swizzle; ALT: half of each row per group) ----
    {
      const uint4* src = reinterpret_cast<const uint4*>(a.q + ((size_t)tok * a.nq + head) * HD);
      constexpr int CH = HD / 8;
      const int c0 = ALT ? grp * (CH / 2) : 0, c1 = ALT ? c0 + CH / 2 : CH;
      uint8_t* dst = sQ + (ALT ? 0 : grp) * TILE + r * 128;
      if (live) {
#pragma unroll 8
        for (int c = c0; c < c1; ++c)
          *reinterpret_cast<uint4*>(dst + (c >> 3) * PANEL + (((c & 7) ^ (r & 7)) << 4)) = src[c];
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    }
    // ---- softmax ----
    const uint32_t tl = tmem + (uint32_t((warp & 3) * 32) << 16);
    const uint32_t tS = tl + uint32_t(grp * 128), tP = tl + uint32_t(C::P_COL(grp)),
                   tO = tl + uint32_t(C::O_COL + grp * HD);
    const bool warp_live = __any_sync(0xffffffffu, live);
    float m_run = -INFINITY, l_run = 0.f;
    bool ok = true;
    const int step = ALT ? 2 : 1;
    int j = 0;
    if (grp < groups) {
#pragma unroll 1
      for (int t = ALT ? grp : 0; t < nb; t += step, ++j) {
        const int kb = (t0 + t) * 128;
        // keys that no row sees: their values must be finite (0 x NaN), so
        // group 0 (ALT: the tile's group) clears those rows of V
        const bool edge = (kb < k_lo || kb + 128 > k_hi) && (ALT || grp == 0);
        if (!__all_sync(0xffffffffu, sh_wait(s_full + grp, uint32_t(j) & 1u, abort_flag, a.err))) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (edge) {
          const uint32_t vi = ALT ? uint32_t(t == nb - 1 ? 2 * nb - 1 : 2 * t + 2) : 2u * t + 1u;
          if (!__all_sync(0xffffffffu, sh_wait(kv_full + vi % NS, (vi / NS) & 1u, abort_flag, a.err))) {
            ok = false;
            break;
          }
          if (kb + r < k_lo || kb + r >= k_hi) {
            uint8_t* v = sR + (vi % NS) * TILE + r * 128;
#pragma unroll
            for (int c = 0; c < HD / 8; ++c)
              *reinterpret_cast<uint4*>(v + (c >> 3) * PANEL + ((c & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async();
        }
        if (warp_live) {
          uint32_t v[128];
#pragma unroll
          for (int c = 0; c < 128; c += 32) tmem_ld32(tS + uint32_t(c), v + c);
          tmem_ld_wait();
          const int ilo = vlo - kb, ihi = vhi - kb;  // visible: ilo <= i < ihi
          if (ilo > 0 || ihi < 128) {
#pragma unroll
            for (int i = 0; i < 128; ++i)
              if (i < ilo || i >= ihi) v[i] = 0xff800000u;  // -inf
          }
          float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
          for (int i = 0; i < 128; i += 4) {
            mx0 = fmaxf(mx0, __uint_as_float(v[i]));
            mx1 = fmaxf(mx1, __uint_as_float(v[i + 1]));
            mx2 = fmaxf(mx2, __uint_as_float(v[i + 2]));
            mx3 = fmaxf(mx3, __uint_as_float(v[i + 3]));
          }
          const float mx = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)) * a.scale_log2;
          float alpha = 1.f;
          if (mx > m_run + RESCALE) {  // also the first finite maximum of the row
            alpha = exp2f(m_run - mx);  // 0 while the reference was -inf
            m_run = mx;
          }
          const float nref = m_run == -INFINITY ? 0.f : -m_run;
          float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
          for (int i = 0; i < 128; i += 2) {
            const float p0 = ex2_fast(fmaf(__uint_as_float(v[i]), a.scale_log2, nref));
            const float p1 = ex2_fast(fmaf(__uint_as_float(v[i + 1]), a.scale_log2, nref));
            sum0 += p0;
            sum1 += p1;
            v[i >> 1] = cvt_bf16x2(p0, p1);
          }
          tmem_st32(tP, v);
          tmem_st32(tP + 32u, v + 32);
          l_run = l_run * alpha + (sum0 + sum1);
          // O rows whose reference moved (the group's previous P V has completed: S_i's barrier follows it)
          if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
            for (int c = 0; c < HD; c += 32) {
              uint32_t o[32];
              tmem_ld32(tO + uint32_t(c), o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st32(tO + uint32_t(c), o);
            }
          }
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + grp);
      }
    }
    // ---- outputs ----
    ok = ok && (nb == 0 || __all_sync(0xffffffffu, sh_wait(o_done, 0u, abort_flag, a.err)));
    tc_fence_after();
    float* xO = reinterpret_cast<float*>(sR);         // ALT: group 1's piece, [HD][128] then (m, l) [128]
    float2* xml = reinterpret_cast<float2*>(xO + HD * 128);
    const bool join = ALT && groups == 2;
    if (join) {
      if (grp == 1 && ok && warp_live) {
#pragma unroll 1
        for (int c = 0; c < HD; c += 32) {
          uint32_t o[32];
          tmem_ld32(tO + uint32_t(c), o);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) xO[(c + i) * 128 + r] = __uint_as_float(o[i]);
        }
        xml[r] = make_float2(m_run, l_run);
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
    }
    if (grp < (ALT ? 1 : groups) && ok && warp_live) {
      const bool direct = own && a.ns_prefix == 0 && a.ns_own == 1;
      float f0 = 1.f, f1 = 0.f;
      if (join) {
        const float2 o = xml[r];
        const float M = fmaxf(m_run, o.x);
        f0 = m_run == -INFINITY ? 0.f : exp2f(m_run - M);
        f1 = o.x == -INFINITY ? 0.f : exp2f(o.x - M);
        m_run = M;
        l_run = l_run * f0 + o.y * f1;
      }
      if (direct) {
        const float inv = l_run > 0.f ? 1.f / l_run : 0.f;
        f0 *= inv;
        f1 *= inv;
      }
      const int part = own ? a.ns_prefix + piece : piece;
      const size_t prow_at = ((size_t)part * a.rows + tok) * a.nq + head;
      if (!direct && live) a.ml_part[prow_at] = make_float2(m_run, l_run);
      if (nb > 0) {
#pragma unroll 1
        for (int c = 0; c < HD; c += 32) {
          uint32_t o[32];
          tmem_ld32(tO + uint32_t(c), o);
          tmem_ld_wait();
          float x[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            x[i] = __uint_as_float(o[i]) * f0;
            if (join) x[i] = fmaf(xO[(c + i) * 128 + r], f1, x[i]);
          }
          if (live) {
            if (direct) {
              uint16_t* dst = a.out + ((size_t)tok * a.nq + head) * HD + c;
#pragma unroll
              for (int i = 0; i < 32; i += 8)
                *reinterpret_cast<uint4*>(dst + i) =
                    make_uint4(cvt_bf16x2(x[i], x[i + 1]), cvt_bf16x2(x[i + 2], x[i + 3]),
                               cvt_bf16x2(x[i + 4], x[i + 5]), cvt_bf16x2(x[i + 6], x[i + 7]));
            } else {
              float* dst = a.o_part + prow_at * HD + c;
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                *reinterpret_cast<float4*>(dst + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
            }
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
// The 64-key tiles of every (sequence, KV head) with at most 16 packed rows
// form one stream (sequence, then KV head, then key), cut into G equal runs,
// one a CTA, whatever the lengths: a CTA takes the segments of its run one by
// one.  A segment that lies in one run is finished there; the piece with its
// first tile goes to the rows' own slot, a piece that begins inside a segment
// to the CTA's (a run has one such piece at most, its first).
// Warps 0-3 compute, warp 4 loads (a ring of stages of 64 K rows and 64 V
// rows, running ahead over segments).  Per tile warp w forms the scores of
// keys 16 w .. + 15 with mma.sync (16 rows by 16 keys), the warps exchange
// their rows' maxima, write P to shared memory, and each multiplies the whole
// P with its quarter of V's columns; so O is never summed across warps.
// mma.sync, since 16 rows would fill an eighth of a tcgen05 tile and memory
// bounds this kernel.  The tensor pipe is idle most of the time, so P goes in
// as two bf16 terms, P and its rounding error, for two products.
template <int HD>
struct Fw {
  static constexpr int TK = 64;                    // keys per tile
  static constexpr int KV = TK * HD * 2;           // bytes of K (or V) per stage
  static constexpr int NST = HD == 128 ? 3 : 6;    // stages
  static constexpr int PB = FEW * TK * 2;          // bytes of one term of P
  static constexpr int SMEM = NST * 2 * KV + 2 * PB + 1024;
};
constexpr int FW_THREADS = 160;

// A sequence (or the prefix, b = batch) in the tile stream.
struct FewSeq {
  Seq s;
  int base;    // prefix: 0; own: P, the position of key 0
  int k_lo;    // first key that a row sees
  int k_end;   // keys
  int tiles;
};
__device__ __forceinline__ int few_tiles(const ShArgs& a, const Seq& s, int* k_lo) {
  *k_lo = a.window ? max(0, s.len - s.n - a.window + 1) : 0;
  if (s.n == 0 || s.n * a.gq > FEW) return 0;
  return ((s.len + 63) >> 6) - (*k_lo >> 6);
}

template <int HD>
__global__ void __launch_bounds__(FW_THREADS)
    few_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
               const __grid_constant__ ShArgs a) {
  using C = Fw<HD>;
  constexpr int NST = C::NST, KV = C::KV, PANELS = HD / 64, NT = HD / 32;  // NT: 8-column tiles of O per warp
  extern __shared__ uint8_t fw_raw[];
  uint8_t* sm = fw_raw + ((1024u - (smem_addr(fw_raw) & 1023u)) & 1023u);
  uint8_t* sP = sm + NST * 2 * KV;
  int* cum = reinterpret_cast<int*>(sP + 2 * C::PB);  // [batch + 2]
  __shared__ uint64_t full[NST], empty[NST];
  __shared__ float s_max[4][FEW], s_sum[4][FEW];
  __shared__ int s_warp[5], s_lo, s_first, s_bad;
  __shared__ int s_abort;
  volatile int* abort_flag = &s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  launch_dependents();
  if (tid == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 4);
    }
    fence_mbar_init();
    s_abort = 0;
    s_lo = 0x7fffffff;
    s_bad = 0;
    cum[0] = 0;
    tma_prefetch_map(&tmK);
    tma_prefetch_map(&tmV);
  }
  __syncthreads();
  // ---- the stream: tiles before each sequence ----
  int before = 0;
#pragma unroll 1
  for (int c0 = 0; c0 < a.batch; c0 += FW_THREADS) {
    int t = 0;
    if (c0 + tid < a.batch) {
      const Seq s = load_seq(a, c0 + tid);
      int lo;
      t = few_tiles(a, s, &lo);
      if (!s.ok) s_bad = 1;
      if (s.n > 0) atomicMin(&s_lo, a.P + s.len - s.n);
    }
    int incl = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int off = before;
#pragma unroll
    for (int w = 0; w < 5; ++w) {
      if (w < warp) off += s_warp[w];
      before += s_warp[w];
    }
    if (c0 + tid < a.batch) cum[c0 + tid + 1] = off + incl;
    __syncthreads();
  }
  // the prefix as a last sequence of all rows, when there are few
  int p_lo = 0;
  if (a.prefix_few && s_lo != 0x7fffffff) {
    p_lo = a.window ? min(a.P, max(0, s_lo - a.window + 1)) : 0;
    if (p_lo < a.P) before += ((a.P + 63) >> 6) - (p_lo >> 6);
  }
  if (tid == 0) cum[a.batch + 1] = before;
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int i = tid; i < a.batch + 2; i += FW_THREADS) a.cum[i] = cum[i];
    if (tid == 0 && s_bad) sh_error(a.err, EW_BAD_SHAPE);
  }
  const long long W = (long long)before * a.nkv;
  const int x_lo = int(W * blockIdx.x / a.G), x_hi = int(W * (blockIdx.x + 1) / a.G);
  // the sequence of the run's first tile
  int b0 = 0;
  {
    int hi = a.batch + 1;
    while (hi - b0 > 1) {
      const int mid = (b0 + hi) >> 1;
      if ((long long)cum[mid] * a.nkv <= x_lo)
        b0 = mid;
      else
        hi = mid;
    }
  }
  auto seq_at = [&](int b) {
    FewSeq f;
    if (b == a.batch) {
      f.s = Seq{0, total_rows(a), 0, 1};
      f.base = 0;
      f.k_lo = p_lo;
      f.k_end = a.P;
    } else {
      f.s = load_seq(a, b);
      f.base = a.P;
      few_tiles(a, f.s, &f.k_lo);
      f.k_end = f.s.len;
    }
    f.tiles = cum[b + 1] - cum[b];
    return f;
  };

  if (warp == 4) {
    // ---- loads ----
    uint32_t it = 0;
    bool ok = true;
    int b = b0;
#pragma unroll 1
    for (int x = x_lo; x < x_hi && ok;) {
      while (x >= cum[b + 1] * a.nkv) ++b;
      const FewSeq f = seq_at(b);
      const int y = x - cum[b] * a.nkv, kvh = y / f.tiles, t = y - kvh * f.tiles;
      const int nt = min(x_hi - x, f.tiles - t);
      const int32_t* pages = b == a.batch ? a.ptable : a.table + (size_t)b * a.width;
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
        const int kb = ((f.k_lo >> 6) + t + i) * 64;
        if (lane == 0)
          mbar_expect_tx(full + s, 2u * load_blocks<HD, 64>(kb, f.k_end, a.page_log2) * bs * HD * 2);
        __syncwarp();
        load_tile<HD, 64>(sm + s * 2 * KV, &tmK, pages, kb, f.k_end, kvh, full + s, a, lane);
        load_tile<HD, 64>(sm + s * 2 * KV + KV, &tmV, pages, kb, f.k_end, kvh, full + s, a, lane);
      }
      x += nt;
    }
    if (lane == 0) {
      const uint32_t first = it > uint32_t(NST) ? it - NST : 0u;
#pragma unroll 1
      for (uint32_t j = first; j < it; ++j) sh_drain(full + (j % NST), (j / NST) & 1u, a.err);
    }
  } else {
    // ---- math ----
    const int g = lane >> 2, tq = lane & 3;
    uint32_t it = 0;
    int b = b0;
    bool ok = true;
#pragma unroll 1
    for (int x = x_lo; x < x_hi && ok;) {
      while (x >= cum[b + 1] * a.nkv) ++b;
      const FewSeq f = seq_at(b);
      const int y = x - cum[b] * a.nkv, kvh = y / f.tiles, t0 = y - kvh * f.tiles;
      const int nt = min(x_hi - x, f.tiles - t0);
      // packed rows g and g + 8 of the segment: tokens, heads, visible keys
      int tok[2], head[2], vlo[2], vhi[2];
      bool live[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int pr = g + 8 * e;
        live[e] = pr < f.s.n * a.gq;
        const int i = live[e] ? pr / a.gq : 0;
        tok[e] = f.s.r0 + i;
        head[e] = kvh * a.gq + (live[e] ? pr - i * a.gq : 0);
        vlo[e] = vhi[e] = 0;
        if (live[e]) {
          if (b == a.batch) {
            vhi[e] = a.P;
            if (a.window) {
              int lo = 0, hi = a.batch;
              while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (a.row_start[mid] <= tok[e])
                  lo = mid;
                else
                  hi = mid;
              }
              const Seq s = load_seq(a, lo);
              vlo[e] = s.n ? min(a.P, max(0, a.P + s.len - s.n + (tok[e] - s.r0) - a.window + 1)) : a.P;
            }
          } else {
            const int p = f.s.len - f.s.n + i;
            vhi[e] = p + 1;
            if (a.window) vlo[e] = max(0, p - a.window + 1);
          }
        }
      }
      // Q as A fragments
      uint32_t qf[HD / 16][4];
#pragma unroll
      for (int ks = 0; ks < HD / 16; ++ks) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int rr = e & 1;
          const size_t at = ((size_t)tok[rr] * a.nq + head[rr]) * HD + ks * 16 + (e >> 1) * 8 + 2 * tq;
          qf[ks][e] = live[rr] ? *reinterpret_cast<const uint32_t*>(a.q + at) : 0u;
        }
      }
      float o[NT][4];
#pragma unroll
      for (int i = 0; i < NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll 1
      for (int i = 0; i < nt; ++i, ++it) {
        const int st = int(it % NST);
        if (!__all_sync(0xffffffffu, sh_wait(full + st, (it / NST) & 1u, abort_flag, a.err))) ok = false;
        // (on a failed wait the warps still meet at the barriers below)
        const uint8_t* sK = sm + st * 2 * KV;
        uint8_t* sV = sm + st * 2 * KV + KV;
        const int kb = ((f.k_lo >> 6) + t0 + i) * 64, k0 = kb + 16 * warp;
        if (kb < f.k_lo || kb + 64 > f.k_end) {
          // values that no row sees must be finite (0 x NaN): clear them
          const int row = lane >> 1, key = k0 + row;
          if (key < f.k_lo || key >= f.k_end) {
#pragma unroll
            for (int c = 0; c < HD / 16; ++c) {
              const int ch = (lane & 1) * (HD / 16) + c;
              *reinterpret_cast<uint4*>(sV + (ch >> 3) * (64 * 128) + (16 * warp + row) * 128 + ((ch & 7) << 4)) =
                  make_uint4(0u, 0u, 0u, 0u);
            }
          }
          fence_proxy_async();  // before the stage is refilled
        }
        float s[2][4] = {};
#pragma unroll
        for (int ks = 0; ks < HD / 16; ++ks) {
          const int mi = lane >> 3, key = 16 * warp + (mi >> 1) * 8 + (lane & 7), ch = 2 * ks + (mi & 1);
          uint32_t k0r, k1r, k2r, k3r;
          ldsm_x4(k0r, k1r, k2r, k3r, sK + (ch >> 3) * (64 * 128) + key * 128 + (((ch & 7) ^ (key & 7)) << 4));
          mma_16816(s[0], qf[ks][0], qf[ks][1], qf[ks][2], qf[ks][3], k0r, k1r);
          mma_16816(s[1], qf[ks][0], qf[ks][1], qf[ks][2], qf[ks][3], k2r, k3r);
        }
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = k0 + j * 8 + 2 * tq + (e & 1), rr = e >> 1;
            s[j][e] = (key >= vlo[rr] && key < vhi[rr]) ? s[j][e] * a.scale_log2 : -INFINITY;
            mx[rr] = fmaxf(mx[rr], s[j][e]);
          }
#pragma unroll
        for (int off = 1; off <= 2; off <<= 1) {
          mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], off));
          mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], off));
        }
        if (tq == 0) {
          s_max[warp][g] = mx[0];
          s_max[warp][g + 8] = mx[1];
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
        float nref[2];
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {
          float M = -INFINITY;
#pragma unroll
          for (int w = 0; w < 4; ++w) M = fmaxf(M, s_max[w][g + 8 * rr]);
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
          nref[rr] = m[rr] == -INFINITY ? 0.f : m[rr];
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int rr = 0; rr < 2; ++rr) {
            const float p0 = ex2_fast(s[j][2 * rr] - nref[rr]), p1 = ex2_fast(s[j][2 * rr + 1] - nref[rr]);
            l[rr] += p0 + p1;
            uint32_t hi, lo;
            split_bf16x2(p0, p1, hi, lo);
            const int row = g + 8 * rr, ch = 2 * warp + j;
            uint8_t* d = sP + row * 128 + ((ch ^ (row & 7)) << 4) + 4 * tq;
            *reinterpret_cast<uint32_t*>(d) = hi;
            *reinterpret_cast<uint32_t*>(d + C::PB) = lo;
          }
        asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          const int mi = lane >> 3;
          const int prow = (mi & 1) * 8 + (lane & 7), pch = 2 * ks + (mi >> 1);
          uint32_t h0, h1, h2, h3, e0, e1, e2, e3;
          const uint8_t* pp = sP + prow * 128 + ((pch ^ (prow & 7)) << 4);
          ldsm_x4(h0, h1, h2, h3, pp);
          ldsm_x4(e0, e1, e2, e3, pp + C::PB);
          const int key = ks * 16 + (mi & 1) * 8 + (lane & 7);
#pragma unroll
          for (int c = 0; c < NT; c += 2) {
            const int ch = warp * NT + c + (mi >> 1);
            uint32_t v0, v1, v2, v3;
            ldsm_x4_t(v0, v1, v2, v3, sV + (ch >> 3) * (64 * 128) + key * 128 + (((ch & 7) ^ (key & 7)) << 4));
            mma_16816(o[c], h0, h1, h2, h3, v0, v1);
            mma_16816(o[c], e0, e1, e2, e3, v0, v1);
            mma_16816(o[c + 1], h0, h1, h2, h3, v2, v3);
            mma_16816(o[c + 1], e0, e1, e2, e3, v2, v3);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + st);
      }
      // ---- the piece's sums: over the quad, then over the warps ----
#pragma unroll
      for (int off = 1; off <= 2; off <<= 1) {
        l[0] += __shfl_xor_sync(0xffffffffu, l[0], off);
        l[1] += __shfl_xor_sync(0xffffffffu, l[1], off);
      }
      if (tq == 0) {
        s_sum[warp][g] = l[0];
        s_sum[warp][g + 8] = l[1];
      }
      asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        const int row = g + 8 * rr;
        float L = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) L += s_sum[w][row];
        if (!live[rr] || !ok) continue;
        const bool first = t0 == 0, whole = first && nt == f.tiles;
        if (whole && b < a.batch && a.ns_prefix == 0) {
          const float inv = L > 0.f ? 1.f / L : 0.f;
          uint16_t* dst = a.out + ((size_t)tok[rr] * a.nq + head[rr]) * HD + warp * NT * 8 + 2 * tq;
#pragma unroll
          for (int c = 0; c < NT; ++c)
            *reinterpret_cast<uint32_t*>(dst + 8 * c) = cvt_bf16x2(o[c][2 * rr] * inv, o[c][2 * rr + 1] * inv);
        } else {
          const size_t at = first ? ((size_t)(b == a.batch ? 0 : a.ns_prefix) * a.rows + tok[rr]) * a.nq + head[rr]
                                  : (size_t)blockIdx.x * FEW + row;
          float* dst = (first ? a.o_part : a.o_cont) + at * HD + warp * NT * 8 + 2 * tq;
#pragma unroll
          for (int c = 0; c < NT; ++c)
            *reinterpret_cast<float2*>(dst + 8 * c) = make_float2(o[c][2 * rr], o[c][2 * rr + 1]);
          if (warp == 0 && tq == 0) (first ? a.ml_part : a.ml_cont)[at] = make_float2(m[rr], L);
        }
      }
      asm volatile("bar.sync 1, 128;" ::: "memory");  // s_sum is free again
      x += nt;
    }
  }
  wait_previous_kernel();
}

// ---------------------------------------------------------------------------
// join_kernel: one CTA per token, one warp per head at a time
// ---------------------------------------------------------------------------
constexpr int JT = 256;

template <int HD>
__global__ void __launch_bounds__(JT) join_kernel(const __grid_constant__ ShArgs a) {
  __shared__ int s_b;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, tok = blockIdx.x;
  if (tid == 0) s_b = -1;
  __syncthreads();
  for (int b = tid; b < a.batch; b += JT)
    if (a.row_start[b] <= tok && tok < a.row_start[b + 1]) s_b = b;
  __syncthreads();
  const int b = s_b;
  wait_previous_kernel();
  if (b < 0) return;
  const Seq s = load_seq(a, b);
  if (tok < s.r0 || tok >= s.r0 + s.n) return;
  const bool few = s.n * a.gq <= FEW;
  const int local = (tok - s.r0) * a.gq;
  const int tiles = few ? a.cum[b + 1] - a.cum[b] : 0, x0 = few ? a.cum[b] * a.nkv : 0;
  const int ptiles = a.prefix_few ? a.cum[a.batch + 1] - a.cum[a.batch] : 0, px0 = a.prefix_few ? a.cum[a.batch] * a.nkv : 0;
  const long long W = (long long)a.cum[a.batch + 1] * a.nkv;
  auto cta_of = [&](long long x) { return int(((x + 1) * a.G - 1) / W); };  // of the run that holds tile x
  constexpr int E = HD / 32;
  for (int head = warp; head < a.nq; head += JT / 32) {
    const int kvh = head / a.gq, g = head - kvh * a.gq;
    // the pieces: slots [first, n_slots), then the CTAs [c0, c1) of the own positions and [p0, p1) of the prefix
    int n_slots = a.ns_prefix + (few ? 1 : a.ns_own), first = 0, c0 = 0, nc = 0, p0 = 0, np = 0;
    if (few) {
      const long long x = x0 + (long long)kvh * tiles;
      c0 = cta_of(x) + 1;
      nc = cta_of(x + tiles - 1) + 1 - c0;
      if (a.ns_prefix == 0 && nc == 0) continue;  // written already
    } else if (a.ns_prefix == 0 && a.ns_own == 1) {
      continue;
    }
    if (a.prefix_few) {
      if (ptiles == 0) {
        first = 1;  // the window ends behind the prefix: slot 0 was not written
      } else {
        const long long x = px0 + (long long)kvh * ptiles;
        p0 = cta_of(x) + 1;
        np = cta_of(x + ptiles - 1) + 1 - p0;
      }
    }
    const int total = (n_slots - first) + nc + np;
    auto piece = [&](int i, const float*& o, float2& ml) {
      if (i < n_slots - first) {
        const size_t at = ((size_t)(first + i) * a.rows + tok) * a.nq + head;
        o = a.o_part + at * HD;
        ml = a.ml_part[at];
      } else {
        i -= n_slots - first;
        const bool mine = i < nc;
        const size_t at = (size_t)(mine ? c0 + i : p0 + i - nc) * FEW + (mine ? local : tok * a.gq) + g;
        o = a.o_cont + at * HD;
        ml = a.ml_cont[at];
      }
    };
    float M = -INFINITY;
    for (int i = lane; i < total; i += 32) {
      const float* o;
      float2 ml;
      piece(i, o, ml);
      if (ml.y > 0.f) M = fmaxf(M, ml.x);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    float acc[E] = {}, L = 0.f;
#pragma unroll 4
    for (int i = 0; i < total; ++i) {
      const float* o;
      float2 ml;
      piece(i, o, ml);
      if (ml.y > 0.f) {
        const float f = exp2f(ml.x - M);
        L = fmaf(ml.y, f, L);
        const float* src = o + lane * E;
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float2 v = *reinterpret_cast<const float2*>(src + e);
          acc[e] = fmaf(v.x, f, acc[e]);
          acc[e + 1] = fmaf(v.y, f, acc[e + 1]);
        }
      }
    }
    const float inv = L > 0.f ? 1.f / L : 0.f;
    uint16_t* dst = a.out + ((size_t)tok * a.nq + head) * HD + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2)
      *reinterpret_cast<uint32_t*>(dst + e) = cvt_bf16x2(acc[e] * inv, acc[e + 1] * inv);
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

// Pieces along the keys of `items` equal items of `tiles` 128-key tiles: the
// count with the shortest time, waves x (tiles of a piece + what a piece costs
// besides: its start, its rows of O written and read again, ~2 tiles).
int pieces_for(long long items, int tiles, int sms, int cap) {
  int best = 1;
  double best_t = 1e30;
  for (int ns = 1; ns <= cap && ns <= (tiles < 1 ? 1 : tiles); ++ns) {
    const double waves = double((items * ns + sms - 1) / sms);
    const double t = waves * ((tiles + ns - 1) / ns + 2.0);
    if (t < best_t * 0.999) {
      best_t = t;
      best = ns;
    }
  }
  return best;
}

struct ShPlan {
  bool many;              // some sequence may have more than FEW packed rows
  bool tc_prefix_alt, tc_own_alt;
  long long prefix_items, own_items;
  int prefix_cap, own_cap;
  int G;
};

ShPlan shared_plan(int rows, int batch, int nq, int nkv, int max_new, int sms) {
  const int gq = nq / nkv;
  ShPlan p;
  const long long packed = (long long)rows * gq;
  const long long most = (long long)(max_new < rows ? max_new : rows) * gq;  // packed rows of one sequence
  p.many = most > FEW;
  p.tc_prefix_alt = packed <= 128;
  p.tc_own_alt = most <= 128;
  p.prefix_items = nkv * ((packed + (p.tc_prefix_alt ? 127 : 255)) / (p.tc_prefix_alt ? 128 : 256));
  // tiles of the sequences with many rows: at most one partly filled tile each
  const long long tr = p.tc_own_alt ? 128 : 256;
  long long seqs = packed / (FEW + 1) + 1;
  if (seqs > batch) seqs = batch;
  p.own_items = nkv * (packed / tr + seqs);
  auto cap = [&](long long items) {
    const long long c = (2LL * sms + items - 1) / items;
    return int(c < 1 ? 1 : (c > 64 ? 64 : c));
  };
  p.prefix_cap = cap(p.prefix_items);
  p.own_cap = p.many ? cap(p.own_items) : 1;
  p.G = 2 * sms;
  return p;
}

struct ShLayout {
  size_t cum, ml_part, ml_cont, o_cont, o_part, total;
};
ShLayout shared_layout(const ShPlan& p, int rows, int batch, int nq, int hd) {
  auto al = [](size_t x) { return (x + 255) & ~size_t(255); };
  ShLayout L;
  const size_t parts = p.prefix_cap + p.own_cap, lines = parts * rows * nq;
  L.cum = 256;
  L.ml_part = L.cum + al((size_t)(batch + 2) * 4);
  L.ml_cont = L.ml_part + al(lines * 8);
  L.o_cont = L.ml_cont + al((size_t)p.G * FEW * 8);
  L.o_part = L.o_cont + al((size_t)p.G * FEW * hd * 4);
  L.total = L.o_part + al(lines * hd * 4);
  return L;
}

cudaError_t launch(const void* fn, unsigned grid, unsigned threads, int smem, bool after, void** args, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = after ? 1 : 0;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  return cudaLaunchKernelExC(&cfg, fn, args);
}

template <int HD>
cudaError_t launch_shared(ShArgs a, const uint16_t* k, const uint16_t* v, const ShPlan& p, int sms, cudaStream_t st) {
  const int page = 1 << a.page_log2;
  const int64_t blocks = (int64_t)a.n_pages * a.nkv;
  CUtensorMap k128, v128, k64, v64;
  cudaError_t e;
  const bool tc_prefix = a.P > 0 && !a.prefix_few;
  if (tc_prefix || p.many) {
    if ((e = page_map(&k128, k, HD, page, blocks, page < 128 ? page : 128)) != cudaSuccess) return e;
    if ((e = page_map(&v128, v, HD, page, blocks, page < 128 ? page : 128)) != cudaSuccess) return e;
  }
  if ((e = page_map(&k64, k, HD, page, blocks, page < 64 ? page : 64)) != cudaSuccess) return e;
  if ((e = page_map(&v64, v, HD, page, blocks, page < 64 ? page : 64)) != cudaSuccess) return e;
  bool after = false;
  for (int own = 0; own < 2; ++own) {
    if (own ? !p.many : !tc_prefix) continue;
    const bool alt = own ? p.tc_own_alt : p.tc_prefix_alt;
    const long long items = (own ? p.own_items : p.prefix_items) * (own ? a.ns_own : a.ns_prefix);
    void* args[] = {&k128, &v128, &a, &own};
    const void* fn = alt ? reinterpret_cast<const void*>(&tc_kernel<HD, true>)
                         : reinterpret_cast<const void*>(&tc_kernel<HD, false>);
    e = launch(fn, unsigned(items), TC_THREADS, alt ? Tc<HD, true>::SMEM : Tc<HD, false>::SMEM, after, args, st);
    if (e != cudaSuccess) return e;
    after = true;
  }
  {
    void* args[] = {&k64, &v64, &a};
    e = launch(reinterpret_cast<const void*>(&few_kernel<HD>), unsigned(a.G), FW_THREADS,
               Fw<HD>::SMEM + ((a.batch + 2) * 4 + 15) / 16 * 16, after, args, st);
    if (e != cudaSuccess) return e;
  }
  void* args[] = {&a};
  return launch(reinterpret_cast<const void*>(&join_kernel<HD>), unsigned(a.rows), JT, 0, true, args, st);
}

}  // namespace

size_t attn_shared_ws(int rows, int batch, int nq, int nkv, int hd, int max_new, int sms) {
  return shared_layout(shared_plan(rows, batch, nq, nkv, max_new, sms), rows, batch, nq, hd).total;
}

cudaError_t launch_attn_shared(const uint16_t* q, int rows, int batch, int nq, int nkv, int hd, const uint16_t* k,
                               const uint16_t* v, int n_pages, int page, const int32_t* row_start, const int32_t* lens,
                               const int32_t* table, int width, const int32_t* ptable, int P, int window, int max_new,
                               uint16_t* out, uint8_t* ws, int sms, cudaStream_t st) {
  const ShPlan p = shared_plan(rows, batch, nq, nkv, max_new, sms);
  const ShLayout L = shared_layout(p, rows, batch, nq, hd);
  ShArgs a;
  a.q = q;
  a.row_start = row_start;
  a.lens = lens;
  a.table = table;
  a.ptable = ptable;
  a.out = out;
  a.err = reinterpret_cast<uint32_t*>(ws) + 2;
  a.cum = reinterpret_cast<int32_t*>(ws + L.cum);
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
  a.prefix_few = P > 0 && rows * a.gq <= FEW;
  // key tiles that an item can have: all, or what a window reaches
  auto tiles = [&](long long keys) {
    if (window > 0 && keys > (long long)window + max_new + 128) keys = (long long)window + max_new + 128;
    return int((keys + 127) / 128);
  };
  a.ns_prefix = P == 0 ? 0 : (a.prefix_few ? 1 : pieces_for(p.prefix_items, tiles(P), sms, p.prefix_cap));
  a.ns_own = p.many ? pieces_for(p.own_items, tiles((long long)width * page), sms, p.own_cap) : 1;
  a.G = p.G;
  a.scale_log2 = float(1.4426950408889634 / sqrt(double(hd)));
  return hd == 64 ? launch_shared<64>(a, k, v, p, sms, st) : launch_shared<128>(a, k, v, p, sms, st);
}

}  // namespace w4a
