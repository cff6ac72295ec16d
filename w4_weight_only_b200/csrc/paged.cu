// The paged KV cache: block tables and slot maps of a step, and QK-norm +
// rotation + append into the pages.  (The attention that reads the pages is
// in shared.cu.)
//
// A layer's K and V are [n_pages][n_kv][page_size][hd] bf16 each, rows in
// plain order; page ids are the same in every layer.  A sequence's own
// positions start behind the prefix that the batch shares: own position i
// (position prefix_len + i) is at page table[b][i / page_size], row
// i % page_size.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "ptx.cuh"
#include "w4a_internal.h"

namespace w4a {

namespace {

// ---------------------------------------------------------------------------
// block tables and slot maps
// ---------------------------------------------------------------------------
// One launch.  Per sequence: held = ceil(len / s) pages, the new length
// len + n (0 for an ended sequence, n = -1), take = ceil(new / s) - held
// pages from the head of the free queue, or freed = held pages to its end.
// The exclusive sums over the sequences of (rows, take, freed) place every
// output.  Every CTA forms those sums itself (a few thousand integers at
// most) and then fills its share of the rows, pages taken and pages freed by
// binary search in them, so no CTA waits for another; CTA 0 also writes the
// per-sequence outputs.  What the CTAs read (lens, n_new, state, the live
// part of the queue, the held part of the table) none of them writes.
// Bound by its chain of loads and scans, not by its bytes (551 KB for 1,024
// sequences with new prompts): 6.3 us of GPU time for 16 sequences of one row,
// 8.4 us for the 1,024.
constexpr int PT = 512;                          // threads
constexpr int PER = MAX_PAGED_BATCH / PT;        // sequences per thread
constexpr int PLAN_ROWS = PT;                    // rows per CTA

struct Sum3 {
  long long rows, take, freed;
};
__device__ __forceinline__ Sum3 operator+(const Sum3& a, const Sum3& b) {
  return Sum3{a.rows + b.rows, a.take + b.take, a.freed + b.freed};
}
__device__ __forceinline__ Sum3 shfl_up(const Sum3& a, int o) {
  return Sum3{__shfl_up_sync(0xffffffffu, a.rows, o), __shfl_up_sync(0xffffffffu, a.take, o),
              __shfl_up_sync(0xffffffffu, a.freed, o)};
}

// The sequence whose range holds x: the last b with start[b] <= x.
__device__ __forceinline__ int seq_of(const int* start, int B, int x) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

struct PlanArgs {
  const int32_t* n_new;
  const int32_t* lens;
  const int32_t* state;
  int32_t* queue;
  int32_t* table;
  int32_t* lens_out;
  int32_t* state_out;
  int32_t* row_start;
  int32_t* slots;
  int32_t* pos;
  uint32_t* err;
  int batch, n_queue, width, page_log2, prefix, max_rows;
};

__global__ void __launch_bounds__(PT) plan_kernel(const PlanArgs a) {
  extern __shared__ int sm_plan[];  // row, take and freed starts, [batch] each, then lens
  int* row0 = sm_plan;
  int* take0 = row0 + a.batch;
  int* free0 = take0 + a.batch;
  int* len0 = free0 + a.batch;
  __shared__ Sum3 wsum[PT / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.batch + PT - 1) / PT;  // sequences of this thread, consecutive
  const int b0 = tid * per;
  const int head = a.state[0], count = a.state[1];  // (loaded with the lengths)
  uint32_t bad = 0;
  Sum3 mine{0, 0, 0}, each[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    each[i] = Sum3{0, 0, 0};
    const int b = b0 + i;
    if (i >= per || b >= a.batch) continue;
    const int n = a.n_new[b], len = a.lens[b];
    const long long end = (long long)len + (n > 0 ? n : 0);
    if (n < -1 || len < 0 || end + a.prefix > 0x7fffffffLL) {
      bad |= EW_BAD_SHAPE;
      continue;
    }
    const int page1 = (1 << a.page_log2) - 1;
    const long long held = ((long long)len + page1) >> a.page_log2, want = (end + page1) >> a.page_log2;
    if (held > a.width || want > a.width) {
      bad |= EW_PAGES;
      continue;
    }
    len0[b] = len;
    each[i] = n < 0 ? Sum3{0, 0, held} : Sum3{n, want - held, 0};
    mine = mine + each[i];
  }
  Sum3 incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sum3 t = shfl_up(incl, o);
    if (lane >= o) incl = incl + t;
  }
  if (lane == 31) wsum[warp] = incl;
  // any sequence's fault fails the plan
  const int shape_bad = __syncthreads_or(int(bad & EW_BAD_SHAPE)), pages_bad = __syncthreads_or(int(bad & EW_PAGES));
  bad = (shape_bad ? EW_BAD_SHAPE : 0u) | (pages_bad ? EW_PAGES : 0u);
  Sum3 base{0, 0, 0}, total{0, 0, 0};
#pragma unroll 1
  for (int w = 0; w < PT / 32; ++w) {
    if (w == warp) base = total;
    total = total + wsum[w];
  }
  const long long N = a.n_queue;
  if (head < 0 || head >= N || count < 0 || count > N || count + total.freed > N)
    bad |= EW_BAD_SHAPE;
  else if (total.take > count + total.freed || total.rows > a.max_rows)
    bad |= EW_PAGES;
  const bool ok = bad == 0u;
  Sum3 at = base + Sum3{incl.rows - mine.rows, incl.take - mine.take, incl.freed - mine.freed};
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = b0 + i;
    if (i >= per || b >= a.batch) continue;
    if (ok) {
      row0[b] = int(at.rows);
      take0[b] = int(at.take);
      free0[b] = int(at.freed);
    }
    if (blockIdx.x == 0) {
      const int n = a.n_new[b], len = a.lens[b];
      a.row_start[b] = ok ? int(at.rows) : 0;
      a.lens_out[b] = !ok ? len : (n < 0 ? 0 : len + n);
    }
    at = at + each[i];
  }
  const int n_rows = ok ? int(total.rows) : 0;
  if (blockIdx.x == 0 && tid == 0) {
    a.row_start[a.batch] = n_rows;
    a.state_out[0] = ok ? int((head + total.take) % N) : head;
    a.state_out[1] = ok ? int(count + total.freed - total.take) : count;
  }
  if (bad && blockIdx.x == 0 && tid == 0) atomicOr(a.err, bad);
  __syncthreads();
  const int first = blockIdx.x * PT + tid, step = gridDim.x * PT;
  // the queue in order: its live entries, then the pages freed by this call
  auto queue_page = [&](int k) {
    if (k < count) return a.queue[head + (long long)k < N ? head + k : int(head + (long long)k - N)];
    const int f = k - count, b = seq_of(free0, a.batch, f);
    return a.table[(size_t)b * a.width + (f - free0[b])];
  };
  auto pages_of = [&](int len) { return int(((long long)len + (1 << a.page_log2) - 1) >> a.page_log2); };
  auto taken_page = [&](int k) {
    const int id = queue_page(k);
    if ((unsigned)id >= (unsigned)a.n_queue) atomicOr(a.err, EW_BAD_POS);
    return id;
  };
  if (ok) {
    for (int k = first; k < int(total.take); k += step) {
      const int b = seq_of(take0, a.batch, k);
      const int held = pages_of(len0[b]);
      a.table[(size_t)b * a.width + held + (k - take0[b])] = taken_page(k);
    }
    for (int f = first; f < int(total.freed); f += step) {
      const int b = seq_of(free0, a.batch, f);
      const int id = a.table[(size_t)b * a.width + (f - free0[b])];
      if ((unsigned)id >= (unsigned)a.n_queue) atomicOr(a.err, EW_BAD_POS);
      a.queue[(head + count + (long long)f) % N] = id;
    }
  }
  for (int r = first; r < a.max_rows; r += step) {
    int slot = -1, p = -1;
    if (r < n_rows) {
      const int b = seq_of(row0, a.batch, r);
      const int own = len0[b] + (r - row0[b]);
      const int held = pages_of(len0[b]);
      const int j = own >> a.page_log2;
      const int id = j < held ? a.table[(size_t)b * a.width + j] : queue_page(take0[b] + (j - held));
      // a page id outside the cache gives no slot: the row is not appended
      if ((unsigned)id < (unsigned)a.n_queue) {
        slot = (id << a.page_log2) + (own & ((1 << a.page_log2) - 1));
      } else {
        atomicOr(a.err, EW_BAD_POS);
      }
      p = a.prefix + own;
    }
    a.slots[r] = slot;
    a.pos[r] = p;
  }
}

// ---------------------------------------------------------------------------
// QK-norm over the whole projections, rotation, append into the pages
// ---------------------------------------------------------------------------
// A CTA takes every gridDim-th row.  The row [q; k; v] (fp32) comes into shared
// memory by asynchronous 16-byte copies, the next one behind it while this one
// is worked on (two buffers), and is read there twice, for the sums of squares
// and for the output.  The rotation of pair (i, i + hd / 2) at the row's
// position is formed once per row: the angle in fp64, reduced to [-pi, pi]
// there (a position of 10^5 has no fraction bits left in fp32), sine and cosine
// in fp32.  Memory bound: 4 bytes read and 2 written per element of the row;
// three CTAs an SM keep 86 KB of a 7,168-wide row's neighbours in flight and
// leave the gains in L1 (one CTA a row, seven an SM, read them from L2 for
// every row: 82.7 us for 8,192 rows).  8,192 such rows take 71 us, 5.0 TB/s;
// the issue slots are busy half of the time, and a row's start (its position's
// angles, its sums across the CTA) is what memory waits for.  16 rows: 5.8 us.
constexpr int QT = 256;

struct PrepArgs {
  const float* y;
  int64_t ld;              // floats between rows
  const float* qg;
  const float* kg;
  const int32_t* pos;
  const int32_t* slots;
  uint16_t* q_out;
  uint16_t* k_pages;
  uint16_t* v_pages;
  uint32_t* err;
  double f[64];
  float ms, eps;
  int rows, nq, nkv, n_pages, page_log2;
};

__device__ __forceinline__ uint2 bf16x4(float a, float b, float c, float d) {
  return make_uint2(cvt_bf16x2(a, b), cvt_bf16x2(c, d));
}

template <int HD>
__global__ void __launch_bounds__(QT, 3) prep_paged_kernel(const __grid_constant__ PrepArgs a) {
  extern __shared__ __align__(16) float rows_sm[];
  __shared__ float2 rot[HD / 2];
  __shared__ float red[2][QT / 32];
  const int tid = threadIdx.x;
  constexpr int h2 = HD / 2, upr = h2 / 4;
  const int qd = a.nq * HD, kd = a.nkv * HD, width = qd + 2 * kd;
  const int n_slots = a.n_pages << a.page_log2;
  auto fetch = [&](int r, int slot, float* dst) {
    if ((unsigned)slot < (unsigned)n_slots) {
      const float* src = a.y + r * a.ld;
      for (int i = tid; i < width / 4; i += QT) cp_async16(dst + 4 * i, src + 4 * i);
    }
    cp_async_commit();
  };
  int r = blockIdx.x, buf = 0;
  int slot = a.slots[r], pos = a.pos[r];
  fetch(r, slot, rows_sm);
  for (;;) {
    const int next = r + gridDim.x;
    int slot_n = -1, pos_n = -1;
    if (next < a.rows) {
      slot_n = a.slots[next];
      pos_n = a.pos[next];
    }
    // (slot -1: a padding row, nothing read, nothing written)
    const bool good = (unsigned)slot < (unsigned)n_slots && pos >= 0;
    if (!good && slot != -1 && tid == 0) atomicOr(a.err, EW_BAD_POS);
    if (good && tid >= QT - h2) {
      const int i = tid - (QT - h2);
      const double ang = double(pos) * a.f[i];
      const double turn = ang - 6.283185307179586476925 * rint(ang * 0.15915494309189533577);
      float sn, cs;
      sincosf(float(turn), &sn, &cs);
      rot[i] = make_float2(cs * a.ms, sn * a.ms);
    }
    float* row = rows_sm + buf * width;
    fetch(next, slot_n, rows_sm + (buf ^ 1) * width);
    cp_async_wait<1>();
    __syncthreads();
    if (good) {
      const float4* row4 = reinterpret_cast<const float4*>(row);
      float sq = 0.f, sk = 0.f;
#pragma unroll 4
      for (int i = tid; i < qd / 4; i += QT) {
        const float4 v = row4[i];
        sq += (v.x * v.x + v.y * v.y) + (v.z * v.z + v.w * v.w);
      }
      for (int i = tid; i < kd / 4; i += QT) {
        const float4 v = row4[qd / 4 + i];
        sk += (v.x * v.x + v.y * v.y) + (v.z * v.z + v.w * v.w);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        sq += __shfl_xor_sync(0xffffffffu, sq, o);
        sk += __shfl_xor_sync(0xffffffffu, sk, o);
      }
      if ((tid & 31) == 0) {
        red[0][tid >> 5] = sq;
        red[1][tid >> 5] = sk;
      }
      __syncthreads();
      sq = sk = 0.f;
#pragma unroll
      for (int w = 0; w < QT / 32; ++w) {
        sq += red[0][w];
        sk += red[1][w];
      }
      const float rq = rsqrtf(sq / float(qd) + a.eps), rk = rsqrtf(sk / float(kd) + a.eps);
      // a thread's unit: four pairs (i .. i + 3, i + hd/2 ..) of one head
      const int nu = (a.nq + a.nkv) * upr;
      // the row's place in a page's first KV head; 1 << page_log2 rows on is the next head's
      const size_t at = (((size_t)(slot >> a.page_log2) * a.nkv) << a.page_log2) + (slot & ((1 << a.page_log2) - 1));
      uint16_t* k_row = a.k_pages + at * HD;
      uint16_t* v_row = a.v_pages + at * HD;
      uint16_t* q_row = a.q_out + (size_t)r * qd;
#pragma unroll 3
      for (int u = tid; u < nu; u += QT) {
        const int h = u / upr, i = (u % upr) * 4;
        const bool isq = h < a.nq;
        const int c = h * HD + i;  // q and k lie one behind the other
        const float rn = isq ? rq : rk;
        const float* gain = isq ? a.qg + c : a.kg + (c - qd);
        const float4 x1 = *reinterpret_cast<const float4*>(row + c), x2 = *reinterpret_cast<const float4*>(row + c + h2);
        const float4 g1 = __ldg(reinterpret_cast<const float4*>(gain)), g2 = __ldg(reinterpret_cast<const float4*>(gain + h2));
        float lo[4], hi[4];
        const float y1[4] = {x1.x * rn * g1.x, x1.y * rn * g1.y, x1.z * rn * g1.z, x1.w * rn * g1.w};
        const float y2[4] = {x2.x * rn * g2.x, x2.y * rn * g2.y, x2.z * rn * g2.z, x2.w * rn * g2.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 cs = rot[i + e];
          lo[e] = y1[e] * cs.x - y2[e] * cs.y;
          hi[e] = y2[e] * cs.x + y1[e] * cs.y;
        }
        uint16_t* dst = isq ? q_row + c : k_row + ((size_t)(h - a.nq) << a.page_log2) * HD + i;
        *reinterpret_cast<uint2*>(dst) = bf16x4(lo[0], lo[1], lo[2], lo[3]);
        *reinterpret_cast<uint2*>(dst + h2) = bf16x4(hi[0], hi[1], hi[2], hi[3]);
      }
      for (int u = tid; u < kd / 4; u += QT) {
        const float4 v = row4[(qd + kd) / 4 + u];
        const int h = (4 * u) / HD, i = 4 * u - h * HD;
        *reinterpret_cast<uint2*>(v_row + ((size_t)h << a.page_log2) * HD + i) = bf16x4(v.x, v.y, v.z, v.w);
      }
    }
    if (next >= a.rows) break;
    __syncthreads();  // the buffer, the rotation and the sums are free again
    r = next;
    slot = slot_n;
    pos = pos_n;
    buf ^= 1;
  }
}

}  // namespace

cudaError_t launch_paged_plan(const int32_t* n_new, const int32_t* lens, const int32_t* state, int32_t* queue,
                              int32_t* table, int32_t* lens_out, int32_t* state_out, int32_t* row_start,
                              int32_t* slots, int32_t* pos, uint32_t* err, int batch, int n_queue, int width, int page,
                              int prefix, int max_rows, cudaStream_t st) {
  int page_log2 = 0;
  while ((1 << page_log2) < page) ++page_log2;
  const PlanArgs a{n_new, lens, state, queue,   table, lens_out,  state_out, row_start, slots,
                   pos,   err,  batch, n_queue, width, page_log2, prefix,    max_rows};
  int grid = (max_rows + PLAN_ROWS - 1) / PLAN_ROWS;
  grid = grid < 1 ? 1 : (grid > 592 ? 592 : grid);
  const int smem = 4 * batch * int(sizeof(int));
  static SmemMark mark;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(&plan_kernel), smem, mark);
  if (e != cudaSuccess) return e;
  plan_kernel<<<grid, PT, smem, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_prep_paged(const float* y, int64_t ld, const float* qg, const float* kg, const int32_t* pos,
                              const int32_t* slots, int rows, uint16_t* q_out, uint16_t* k_pages, uint16_t* v_pages,
                              uint32_t* err, const double* f, float ms, float eps, int nq, int nkv, int hd, int n_pages,
                              int page, int sms, cudaStream_t st) {
  PrepArgs a;
  a.y = y;
  a.ld = ld;
  a.qg = qg;
  a.kg = kg;
  a.pos = pos;
  a.slots = slots;
  a.q_out = q_out;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.err = err;
  for (int i = 0; i < 64; ++i) a.f[i] = f[i];
  a.ms = ms;
  a.eps = eps;
  a.rows = rows;
  a.nq = nq;
  a.nkv = nkv;
  a.n_pages = n_pages;
  a.page_log2 = 0;
  while ((1 << a.page_log2) < page) ++a.page_log2;
  const int smem = 2 * (nq + 2 * nkv) * hd * 4;  // two rows
  const int grid = rows < 3 * sms ? rows : 3 * sms;
  static SmemMark marks[2];
  const void* fn = hd == 64 ? reinterpret_cast<const void*>(&prep_paged_kernel<64>)
                            : reinterpret_cast<const void*>(&prep_paged_kernel<128>);
  const cudaError_t e = allow_smem(fn, smem, marks[hd == 64 ? 0 : 1]);
  if (e != cudaSuccess) return e;
  if (hd == 64)
    prep_paged_kernel<64><<<grid, QT, smem, st>>>(a);
  else
    prep_paged_kernel<128><<<grid, QT, smem, st>>>(a);
  return cudaGetLastError();
}

}  // namespace w4a
