// Attention of a batch whose sequences share a prefix, over the paged KV
// cache (paged.cu).
//
// Row r of sequence b is query token i of its n_b = row_start[b + 1] -
// row_start[b] rows, the last n_b of the sequence's len_b own positions; it
// sits at position p = P + len_b - n_b + i behind the shared prefix of P
// positions and sees positions j <= p, with a window W > 0 also j > p - W:
// positions j < P in the shared pages, the others in the sequence's own.
//   out = softmax(q k^T / sqrt(hd)) v,  query head h over KV head h / (nq / nkv)
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "ptx.cuh"
#include "tc.cuh"
#include "w4a_internal.h"

namespace w4a {

namespace {

struct ShArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  const int32_t* row_start;
  const int32_t* lens;
  const int32_t* table;
  const int32_t* ptable;
  uint16_t* out;
  uint32_t* err;
  int rows, batch, nq, nkv, hd, n_pages, page, width, P, window, max_new;
  float scale_log2;
};

// ---------------------------------------------------------------------------
// one warp per (row, head)
// ---------------------------------------------------------------------------
template <int HD>
__global__ void __launch_bounds__(256) simple_kernel(const ShArgs a) {
  const int warp = (blockIdx.x * 256 + threadIdx.x) >> 5, lane = threadIdx.x & 31;
  const int r = warp / a.nq, h = warp - r * a.nq;
  if (r >= a.rows) return;
  int b = 0;
  for (; b < a.batch; ++b)
    if (r >= a.row_start[b] && r < a.row_start[b + 1]) break;
  if (b == a.batch) return;
  const int r0 = a.row_start[b], n = a.row_start[b + 1] - r0, len = a.lens[b];
  if (n > a.max_new || n > len || (len + a.page - 1) / a.page > a.width) {
    if (lane == 0) atomicOr(a.err, EW_BAD_SHAPE);
    return;
  }
  const int p = a.P + len - n + (r - r0);
  const int lo = a.window ? max(0, p - a.window + 1) : 0;
  const int kvh = h / (a.nq / a.nkv);
  constexpr int E = HD / 32;
  float q[E], o[E] = {};
  for (int e = 0; e < E; ++e) q[e] = bf16_to_f32(a.q[((size_t)r * a.nq + h) * HD + lane * E + e]) * a.scale_log2;
  float m = -INFINITY, l = 0.f;
  for (int j = lo; j <= p; ++j) {
    const int i = j < a.P ? j : j - a.P;
    const int id = j < a.P ? a.ptable[i / a.page] : a.table[(size_t)b * a.width + i / a.page];
    if ((unsigned)id >= (unsigned)a.n_pages) {
      if (lane == 0) atomicOr(a.err, EW_BAD_POS);
      continue;
    }
    const size_t off = (((size_t)id * a.nkv + kvh) * a.page + i % a.page) * HD + lane * E;
    float s = 0.f;
    for (int e = 0; e < E; ++e) s = fmaf(q[e], bf16_to_f32(a.k[off + e]), s);
    for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    const float mn = fmaxf(m, s), c = exp2f(m - mn), x = exp2f(s - mn);
    m = mn;
    l = l * c + x;
    for (int e = 0; e < E; ++e) o[e] = fmaf(x, bf16_to_f32(a.v[off + e]), o[e] * c);
  }
  for (int e = 0; e < E; ++e)
    a.out[((size_t)r * a.nq + h) * HD + lane * E + e] = f32_to_bf16(l > 0.f ? o[e] / l : 0.f);
}

}  // namespace

cudaError_t launch_attn_shared(const uint16_t* q, int rows, int batch, int nq, int nkv, int hd, const uint16_t* k,
                               const uint16_t* v, int n_pages, int page, const int32_t* row_start, const int32_t* lens,
                               const int32_t* table, int width, const int32_t* ptable, int P, int window, int max_new,
                               uint16_t* out, uint8_t* ws, int sms, cudaStream_t st) {
  ShArgs a;
  a.q = q;
  a.k = k;
  a.v = v;
  a.row_start = row_start;
  a.lens = lens;
  a.table = table;
  a.ptable = ptable;
  a.out = out;
  a.err = reinterpret_cast<uint32_t*>(ws) + 2;
  a.rows = rows;
  a.batch = batch;
  a.nq = nq;
  a.nkv = nkv;
  a.hd = hd;
  a.n_pages = n_pages;
  a.page = page;
  a.width = width;
  a.P = P;
  a.window = window;
  a.max_new = max_new;
  a.scale_log2 = float(1.4426950408889634 / sqrt(double(hd)));
  const unsigned grid = unsigned(((int64_t)rows * nq + 7) / 8);
  if (hd == 64)
    simple_kernel<64><<<grid, 256, 0, st>>>(a);
  else
    simple_kernel<128><<<grid, 256, 0, st>>>(a);
  return cudaGetLastError();
}

size_t attn_shared_ws(int rows, int batch, int nq, int nkv, int hd, int max_new, int sms) { return 256; }

}  // namespace w4a
