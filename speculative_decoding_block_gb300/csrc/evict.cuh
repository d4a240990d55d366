// evict.cuh -- eviction from the paged cache by accumulated attention weight.
//
// A request with L > budget rows keeps, in each layer and KV head, its first
// `sinks` rows, its last `recent` rows and, of those between, the
// budget - sinks - recent rows of the largest score; among equal scores the
// lowest rows; NaN counts as below every number.  Kept rows keep their order
// and move to rows [0, budget) of the same pages.
//
// Moving in place: kept row number j comes from row r_j >= j.  Rows are moved
// in batches of ascending j, each batch read whole before it is written; a
// batch writes rows below those that any later batch reads.
#pragma once

#include "vsd_common.cuh"

namespace vsd {

struct EvictArgs {
  int batch, layers, n_kv, num_pages, ppr, max_tokens, budget, sinks, recent;
  const int* lens;   // [B]
  int* new_lens;     // [B]; nullptr: written by a launch of its own (lens is the same array)
  const int* page_table;
  __nv_bfloat16 *k_pool, *v_pool;
  float* score;      // [layers][B][n_kv][max_tokens]
  int* kept;         // [layers][B][n_kv][budget] or nullptr
  int* status;
};

// Orderable key of a score: NaN lowest, -0 equal to +0.
__device__ __forceinline__ uint32_t score_key(float f) { return f != f ? 0u : float_order_key(f + 0.0f); }

constexpr int kEvictThreads = 256;

// Whether request b's rows [0, L) lie in the pool (every thread of the CTA).
__device__ __forceinline__ bool pages_ok(const int* pages, int L, int num_pages) {
  int ok = 1;
  for (int i = threadIdx.x; i < (L + kPage - 1) / kPage; i += blockDim.x) ok &= pages[i] >= 0 && pages[i] < num_pages;
  return __syncthreads_and(ok);
}

// New length of a request with L rows: min(L, budget); a rejected or idle one keeps its value.
__device__ __forceinline__ int evicted_len(int L, int budget, int max_tokens, bool ok) {
  return (L >= 0 && L <= max_tokens && ok) ? min(L, budget) : L;
}

// One CTA per (layer, request, KV head): radix selection of the smallest kept
// score (four digits of eight bits), then the rows in chunks of 256: keep
// flags, their running count, and the move.
template <int HD>
__global__ void __launch_bounds__(kEvictThreads) evict_kernel(const EvictArgs a) {
  constexpr int V = HD / 8;                    // 16-byte words of a row
  constexpr int RB = kEvictThreads * 8 / (2 * V);  // rows moved per batch (8 words a thread)
  __shared__ int hist[256];
  __shared__ int warp_cnt[kEvictThreads / 32];
  __shared__ int src_s[kEvictThreads];
  __shared__ uint32_t thr_s;
  __shared__ int need_s;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int h = blockIdx.x % a.n_kv, b = (blockIdx.x / a.n_kv) % a.batch, layer = blockIdx.x / a.n_kv / a.batch;
  const int L = a.lens[b];
  const int* pages = a.page_table + static_cast<size_t>(b) * a.ppr;
  const bool valid = L >= 0 && L <= a.max_tokens;
  const bool ok = valid && pages_ok(pages, L, a.num_pages);
  if (layer == 0 && h == 0 && t == 0) {
    if (!valid && L != kIdleSlot) atomicOr(a.status, VSD_DEV_BAD_SEQLEN);
    if (valid && !ok) atomicOr(a.status, VSD_DEV_BAD_PAGE);
    if (a.new_lens) a.new_lens[b] = evicted_len(L, a.budget, a.max_tokens, ok);
  }
  const size_t head = (static_cast<size_t>(layer) * a.batch + b) * a.n_kv + h;
  int* kept = a.kept ? a.kept + head * a.budget : nullptr;
  if (!ok || L <= a.budget) {
    if (kept)
      for (int j = t; j < a.budget; j += kEvictThreads) kept[j] = (ok && j < L) ? j : -1;
    return;
  }
  float* score = a.score ? a.score + head * a.max_tokens : nullptr;  // nullptr only where nothing is chosen
  const int mid0 = a.sinks, mid1 = L - a.recent, want = a.budget - a.sinks - a.recent;
  // the want-th largest key of rows [mid0, mid1), and how many of its equals are kept
  uint32_t prefix = 0;
  int need = want;
  if (want > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      hist[t] = 0;
      __syncthreads();
      for (int i = mid0 + t; i < mid1; i += kEvictThreads) {
        const uint32_t k = score_key(score[i]);
        if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255], 1);
      }
      __syncthreads();
      if (t == 0) {
        int d = 255, left = need;
        for (; d > 0 && hist[d] < left; --d) left -= hist[d];
        thr_s = prefix | (static_cast<uint32_t>(d) << shift);
        need_s = left;
      }
      __syncthreads();
      prefix = thr_s;
      need = need_s;
    }
  }
  const size_t pool_head = (static_cast<size_t>(layer) * a.num_pages * a.n_kv + h) * kPage * HD;
  const size_t page_stride = static_cast<size_t>(a.n_kv) * kPage * HD;
  auto row_ptr = [&](__nv_bfloat16* pool, int i) {
    return reinterpret_cast<uint4*>(pool + pool_head + pages[i / kPage] * page_stride + (i % kPage) * HD);
  };
  int done = 0, ties = 0;  // rows kept and equals of the threshold seen so far
  for (int i0 = 0; i0 < L; i0 += kEvictThreads) {
    const int i = i0 + t;
    const float sc = score && i < L ? score[i] : 0.0f;
    const bool in_mid = i >= mid0 && i < mid1;
    const uint32_t key = score_key(sc);
    const bool tie = in_mid && want > 0 && key == prefix;
    // rank of this row among the equals (block-wide running count)
    const unsigned tb = __ballot_sync(0xFFFFFFFFu, tie);
    if (lane == 0) warp_cnt[warp] = __popc(tb);
    __syncthreads();
    int before = ties, all = 0;
    for (int w = 0; w < kEvictThreads / 32; ++w) {
      if (w < warp) before += warp_cnt[w];
      all += warp_cnt[w];
    }
    before += __popc(tb & ((1u << lane) - 1));
    ties += all;
    __syncthreads();
    const bool keep = i < L && (!in_mid || (want > 0 && (key > prefix || (tie && before < need))));
    const unsigned kb = __ballot_sync(0xFFFFFFFFu, keep);
    if (lane == 0) warp_cnt[warp] = __popc(kb);
    __syncthreads();
    int pos = 0, cnt = 0;
    for (int w = 0; w < kEvictThreads / 32; ++w) {
      if (w < warp) pos += warp_cnt[w];
      cnt += warp_cnt[w];
    }
    pos += __popc(kb & ((1u << lane) - 1));
    if (keep) {
      src_s[pos] = i;
      if (kept) kept[done + pos] = i;
    }
    __syncthreads();
    // the chunk's scores were all read above
    if (keep && score) score[done + pos] = sc;
    for (int r0 = 0; r0 < cnt; r0 += RB) {
      uint4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int x = u * kEvictThreads + t, r = r0 + x / (2 * V), c = x % (2 * V);
        if (r < cnt && src_s[r] != done + r) v[u] = row_ptr(c < V ? a.k_pool : a.v_pool, src_s[r])[c % V];
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int x = u * kEvictThreads + t, r = r0 + x / (2 * V), c = x % (2 * V);
        if (r < cnt && src_s[r] != done + r) row_ptr(c < V ? a.k_pool : a.v_pool, done + r)[c % V] = v[u];
      }
      __syncthreads();
    }
    done += cnt;
    __syncthreads();
  }
}

// Lengths after an eviction whose input and output lengths are one array:
// a launch of its own, behind the last reader of the old lengths.
__global__ void evict_lens_kernel(const EvictArgs a, int* lens) {
  const int b = blockIdx.x;
  const int L = lens[b];
  const int* pages = a.page_table + static_cast<size_t>(b) * a.ppr;
  const bool ok = L >= 0 && L <= a.max_tokens && pages_ok(pages, L, a.num_pages);
  if (threadIdx.x == 0) lens[b] = evicted_len(L, a.budget, a.max_tokens, ok);
}

}  // namespace vsd
