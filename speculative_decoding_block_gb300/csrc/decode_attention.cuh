// decode_attention.cuh -- attention of one new token per request over the
// paged cache.
//
// Request b holds L cached rows; its new token (optional) is row L.  Query
// head hq of KV head h = hq / (n_q / n_kv) sees the rows
// [max(0, n - window), n), n = L + 1 (n = L without a new row; window 0: all):
//     s_i = q . K_i / sqrt(hd),  p = softmax(s),  o = sum_i p_i V_i,
// with the running maximum and sum of the online softmax, so that K and V
// are read once.  Rows outside the set never take part, whatever they hold.
#pragma once

#include "vsd_common.cuh"

namespace vsd {

constexpr int kMaxGroup = 7;  // query heads per KV head (a model's 17-row verify tile allows no more)

struct DecodeArgs {
  int batch, n_q, n_kv, group, layer, num_pages, ppr, max_tokens, window;
  float scale_log2;         // log2(e) / sqrt(hd)
  const int* lens;          // [B] cached rows (-1: idle slot)
  const int* page_table;    // [max_batch][ppr]
  const __nv_bfloat16* q;   // [B][n_q][hd]
  const __nv_bfloat16* k_new;  // [B][n_kv][hd], nullptr: no new row
  const __nv_bfloat16* v_new;
  __nv_bfloat16 *k_pool, *v_pool;
  __half* out;   // [B][n_q][hd]
  float* lse;    // [B][n_q] or nullptr
  float* score;  // [B][n_kv][max_tokens] or nullptr
  int* status;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// One CTA per (request, KV head); its eight warps walk the rows in turn,
// each with its own running maximum, sum and output per query head, joined
// through shared memory at the end.
constexpr int kDecodeThreads = 256;

template <int HD>
__global__ void __launch_bounds__(kDecodeThreads) decode_attention_kernel(const DecodeArgs a) {
  constexpr int E = HD / 32;  // elements of a row per lane
  constexpr int W = kDecodeThreads / 32;
  __shared__ float m_s[W][kMaxGroup], l_s[W][kMaxGroup], o_s[W][kMaxGroup][HD];
  __shared__ int bad_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x / a.n_kv, h = blockIdx.x % a.n_kv, g = a.group;
  const int L = a.lens[b];
  const bool append = a.k_new != nullptr;
  if (threadIdx.x == 0) bad_s = 0;
  __syncthreads();
  const bool valid = L >= 0 && L + (append ? 1 : 0) <= a.max_tokens;
  if (!valid && L != kIdleSlot && threadIdx.x == 0) atomicOr(a.status, VSD_DEV_BAD_SEQLEN);
  const int n = valid ? L + (append ? 1 : 0) : 0;
  const int lo = a.window > 0 ? max(0, n - a.window) : 0;
  const int* pages = a.page_table + static_cast<size_t>(b) * a.ppr;
  auto row_offset = [&](int i) -> size_t {
    int page = pages[i / kPage];
    if (page < 0 || page >= a.num_pages) {
      bad_s = 1;
      page = 0;
    }
    return (((static_cast<size_t>(a.layer) * a.num_pages + page) * a.n_kv + h) * kPage + i % kPage) * HD;
  };
  float q[kMaxGroup][E], o[kMaxGroup][E], m[kMaxGroup], l[kMaxGroup];
#pragma unroll
  for (int j = 0; j < kMaxGroup; ++j) {
    m[j] = -INFINITY;
    l[j] = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      o[j][e] = 0.0f;
      q[j][e] = j < g ? __bfloat162float(a.q[(static_cast<size_t>(b) * a.n_q + h * g + j) * HD + lane * E + e]) : 0.0f;
    }
  }
  const size_t new_off = (static_cast<size_t>(b) * a.n_kv + h) * HD;
  // scores of row i for every query head of the group, in log2 units
  auto scores = [&](int i, float* s) {
    const __nv_bfloat16* k = (append && i == L) ? a.k_new + new_off : a.k_pool + row_offset(i);
    float kf[E];
#pragma unroll
    for (int e = 0; e < E; ++e) kf[e] = __bfloat162float(k[lane * E + e]);
#pragma unroll
    for (int j = 0; j < kMaxGroup; ++j) {
      float d = 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) d += q[j][e] * kf[e];
      s[j] = warp_sum(d) * a.scale_log2;
    }
  };
  for (int i = lo + warp; i < n; i += W) {
    float s[kMaxGroup];
    scores(i, s);
    const __nv_bfloat16* v = (append && i == L) ? a.v_new + new_off : a.v_pool + row_offset(i);
    float vf[E];
#pragma unroll
    for (int e = 0; e < E; ++e) vf[e] = __bfloat162float(v[lane * E + e]);
#pragma unroll
    for (int j = 0; j < kMaxGroup; ++j) {
      const float mn = fmaxf(m[j], s[j]), mu = mn == -INFINITY ? 0.0f : mn;
      const float c = exp2f(m[j] - mu), p = exp2f(s[j] - mu);
      m[j] = mn;
      l[j] = l[j] * c + p;
#pragma unroll
      for (int e = 0; e < E; ++e) o[j][e] = o[j][e] * c + p * vf[e];
    }
  }
#pragma unroll
  for (int j = 0; j < kMaxGroup; ++j) {
    if (lane == 0) {
      m_s[warp][j] = m[j];
      l_s[warp][j] = l[j];
    }
#pragma unroll
    for (int e = 0; e < E; ++e) o_s[warp][j][lane * E + e] = o[j][e];
  }
  // the new row's page is checked before anything is written
  if (append && valid && threadIdx.x == 0) row_offset(L);
  __syncthreads();
  const bool bad = bad_s != 0;
  if (bad && threadIdx.x == 0) atomicOr(a.status, VSD_DEV_BAD_PAGE);
  const bool empty = bad || n == 0;
  auto join = [&](int j, float& mj, float& lj) {
    mj = -INFINITY;
    for (int w = 0; w < W; ++w) mj = fmaxf(mj, m_s[w][j]);
    if (mj == -INFINITY) mj = 0.0f;
    lj = 0.0f;
    for (int w = 0; w < W; ++w) lj += l_s[w][j] * exp2f(m_s[w][j] - mj);
  };
  for (int i = threadIdx.x; i < g * HD; i += kDecodeThreads) {
    const int j = i / HD, d = i % HD;
    float mj, lj, acc = 0.0f;
    join(j, mj, lj);
    for (int w = 0; w < W; ++w) acc += o_s[w][j][d] * exp2f(m_s[w][j] - mj);
    // one rounding, to the GEMM input type
    a.out[(static_cast<size_t>(b) * a.n_q + h * g) * HD + i] = __float2half_rn(empty ? 0.0f : acc / lj);
    if (d == 0 && a.lse)
      a.lse[static_cast<size_t>(b) * a.n_q + h * g + j] = empty ? -INFINITY : (mj + log2f(lj)) * 0.69314718f;
  }
  if (empty) return;
  if (a.score) {
    float mj[kMaxGroup], lj[kMaxGroup];
    for (int j = 0; j < g; ++j) join(j, mj[j], lj[j]);
    float* score = a.score + (static_cast<size_t>(b) * a.n_kv + h) * a.max_tokens;
    for (int i = lo + warp; i < n; i += W) {
      float s[kMaxGroup];
      scores(i, s);
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < kMaxGroup; ++j)
        if (j < g) sum += exp2f(s[j] - mj[j]) / lj[j];
      if (lane == 0) score[i] = (append && i == L) ? sum : score[i] + sum;
    }
  }
  if (append) {
    const size_t to = row_offset(L);
    for (int d = threadIdx.x; d < HD; d += kDecodeThreads) {
      a.k_pool[to + d] = a.k_new[new_off + d];
      a.v_pool[to + d] = a.v_new[new_off + d];
    }
  }
}

}  // namespace vsd
