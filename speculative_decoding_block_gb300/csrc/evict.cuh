// evict.cuh -- eviction from the paged cache by accumulated attention weight.
//
// A request with L > budget rows keeps, in each layer and KV head, its first
// `sinks` rows, its last `recent` rows and, of those between, the
// budget - sinks - recent rows of the largest score; among equal scores the
// lowest rows; NaN counts as below every number.  Kept rows keep their order
// and move to rows [0, budget) of the same pages.
//
// Bound by the bytes of the kept rows, read and written once.  A CTA (or,
// where heads are few, a cluster, each CTA with an equal share of the rows) per
// (layer, request, KV head): the smallest kept score by three digits of 11, 11
// and 10 bits of its ordered key, the CTAs' counts added up through distributed
// shared memory; a bit per row for what stays, with a running count per 32
// rows; then the move.  Moving in place: kept row number j comes from row
// r_j >= j, and rows are moved in batches of ascending j, which write rows below
// all that any later batch reads: one barrier per batch is needed, between its
// own reads and its writes.
//
// Measured on fresh caches: 16 requests of 4096 rows cut to 1024, 8 layers, 8
// heads of 128, 203 us for 1.1 GB (79 % of the copy bandwidth; three CTAs of
// 512 threads per SM keep more bytes in flight than two of 256 that read a
// batch ahead, 278 us); 24 layers of one request of 2048 rows cut to 512, 2
// heads of 64, 18 us; 8 heads of 100,000 rows cut to 20,000 143 us (334 with
// every CTA counting all rows).
#pragma once

#include "cluster_mem.cuh"

namespace vsd {

struct EvictArgs {
  int batch, layers, n_kv, num_pages, ppr, max_tokens, budget, sinks, recent;
  int cs;            // CTAs per (layer, request, KV head)
  int words;         // 32-row words of a CTA's share of a request at its longest
  int cache;         // scores kept in shared memory, where a share has no more
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

constexpr int kEvictBins = 2048;
constexpr int kEvictMaxCluster = 8;
// The three forms of the kernel.
struct EvictWide {  // one CTA per SM at most: long batches, so that few barriers stand between the moves
  static constexpr int threads = 512, unroll = 16, window = 4096, per_sm = 1, most_cached = 32768;
  static constexpr bool clusters = true;
};
struct EvictFull {  // all SMs full
  static constexpr int threads = 512, unroll = 4, window = 1024, per_sm = 3, most_cached = 8192;
  static constexpr bool clusters = false;
};
struct EvictShort {  // many short requests: the chain of a CTA's steps is what takes the time, so many of them at once
  // (eight a SM; twelve spilled and took 57 us where these take 52)
  static constexpr int threads = 128, unroll = 8, window = 256, per_sm = 8, most_cached = 1024;
  static constexpr bool clusters = false;
};
// unroll: 16-byte words of a thread per batch; window: kept rows listed at a time, a multiple of a cluster's batch
template <class Form>
constexpr int evict_batch(int hd) { return Form::threads * Form::unroll / (2 * (hd / 8)); }  // rows of a CTA's batch
template <class Form>
int evict_smem_bytes(int words, int cache) { return ((Form::clusters ? 3 : 1) * kEvictBins + 2 * Form::window + 2 * words + cache) * 4; }

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

template <int HD, class Form>
__global__ void __launch_bounds__(Form::threads, Form::per_sm) evict_kernel(const EvictArgs a) {
  constexpr int T = Form::threads, W = T / 32, U = Form::unroll, kWindow = Form::window;
  constexpr bool CL = Form::clusters;
  constexpr int V = HD / 8;  // 16-byte words of a row
  constexpr int RB = evict_batch<Form>(HD);
  constexpr int E = kEvictBins / T;  // bins of a thread
  static_assert(kWindow % (CL ? kEvictMaxCluster * RB : RB) == 0 && RB <= T && E % 4 == 0);
  extern __shared__ __align__(16) uint32_t evict_smem[];
  uint32_t* hists = evict_smem;  // one, or one a digit where other CTAs read it
  uint32_t* win = hists + (CL ? 3 : 1) * kEvictBins;
  uint32_t* place = win + kWindow;    // and where they lie in the layer's pool
  uint32_t* mask = place + kWindow;   // rows that stay, of this CTA's words
  uint32_t* count = mask + a.words;   // of them in front of the word (equals' bits before that)
  float* cache = reinterpret_cast<float*>(count + a.words);
  __shared__ uint32_t red[W], found[3], xch[2][kEvictMaxCluster];
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31, cs = CL ? a.cs : 1;
  const int item = static_cast<int>(blockIdx.x) / cs, rank = static_cast<int>(blockIdx.x) % cs;
  const int h = item % a.n_kv, b = (item / a.n_kv) % a.batch, layer = item / a.n_kv / a.batch;
  const int L = a.lens[b];
  const int* pages = a.page_table + static_cast<size_t>(b) * a.ppr;
  const bool valid = L >= 0 && L <= a.max_tokens;
  const bool ok = valid && pages_ok(pages, L, a.num_pages);
  if (layer == 0 && h == 0 && rank == 0 && t == 0) {
    if (!valid && L != kIdleSlot) atomicOr(a.status, VSD_DEV_BAD_SEQLEN);
    if (valid && !ok) atomicOr(a.status, VSD_DEV_BAD_PAGE);
    if (a.new_lens) a.new_lens[b] = evicted_len(L, a.budget, a.max_tokens, ok);
  }
  int* kept = a.kept ? a.kept + static_cast<size_t>(item) * a.budget : nullptr;
  if (!ok || L <= a.budget) {  // the whole cluster alike
    if (kept && rank == 0)
      for (int64_t j = t; j < a.budget; j += T) kept[j] = (ok && j < L) ? static_cast<int>(j) : -1;
    return;
  }
  float* score = a.score ? a.score + static_cast<size_t>(item) * a.max_tokens : nullptr;  // nullptr only where nothing is chosen
  const int mid0 = a.sinks, mid1 = L - a.recent, want = a.budget - a.sinks - a.recent;
  // this CTA's words of 32 rows, and its rows [r0, r1)
  const int words = (L + 31) / 32, share = (words + cs - 1) / cs, wa = min(words, rank * share), nw = min(words, wa + share) - wa;
  const int r0 = wa * 32, r1 = min(L, r0 + nw * 32);
  auto sync_all = [&]() {
    if (cs > 1) cluster_sync();
    else __syncthreads();
  };
  // sum over the threads before this one; all: of all
  auto block_scan = [&](uint32_t v, uint32_t* all) {
    uint32_t c = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, c, o);
      if (lane >= o) c += y;
    }
    __syncthreads();
    if (lane == 31) red[warp] = c;
    __syncthreads();
    uint32_t pre = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      pre += w < warp ? red[w] : 0;
      sum += red[w];
    }
    *all = sum;
    return pre + c - v;
  };
  // the other ranks' `mine`, summed over the ranks before this one
  auto ranks_before = [&](int turn, uint32_t mine) {
    if (cs == 1) return 0u;
    if (t < cs) st_dsmem_u32(mapa_shared(smem_u32(&xch[turn][rank]), t), mine);
    cluster_sync();
    uint32_t pre = 0;
    for (int r = 0; r < rank; ++r) pre += xch[turn][r];
    return pre;
  };
  for (int i = t; i < (CL ? 3 : 1) * kEvictBins; i += T) hists[i] = 0;
  sync_all();  // and every CTA of the cluster has started

  // ------------------------------------------------------------------ the want-th largest key of rows [mid0, mid1)
  uint32_t thr = 0, need = 0, equals = 0;  // kept: keys above thr and the first `need` of its `equals`
  const bool cached = score && share * 32 <= a.cache;
  if (want > 0) {
    need = static_cast<uint32_t>(want);
#pragma unroll 1
    for (int level = 0; level < 3; ++level) {
      const int shift = level == 0 ? 21 : level == 1 ? 10 : 0, bits = level == 2 ? 10 : 11;
      uint32_t* hist = CL ? hists + level * kEvictBins : hists;
      if (!CL && level) {
        for (int i = t; i < kEvictBins; i += T) hist[i] = 0;
        __syncthreads();
      }
#pragma unroll 4
      for (int i = r0 + t; i < r1; i += T) {
        const float s = level && cached ? cache[i - r0] : score[i];
        if (!level && cached) cache[i - r0] = s;
        const uint32_t k = score_key(s);
        if (i >= mid0 && i < mid1 && (!level || (k >> (shift + bits)) == (thr >> (shift + bits))))
          atomicAdd(&hist[kEvictBins - 1 - ((k >> shift) & ((1u << bits) - 1))], 1u);  // largest first
      }
      sync_all();
      uint32_t n[E], sum = 0, all;
#pragma unroll
      for (int e = 0; e < E; e += 4) {
        uint4 v = *reinterpret_cast<const uint4*>(hist + t * E + e);
        if (cs > 1) {
          v = make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int r = 0; r < kEvictMaxCluster; ++r)
            if (r < cs) {
              const uint4 y = ld_dsmem_v4(mapa_shared(smem_u32(hist + t * E + e), r));
              v = make_uint4(v.x + y.x, v.y + y.y, v.z + y.z, v.w + y.w);
            }
        }
        n[e] = v.x;
        n[e + 1] = v.y;
        n[e + 2] = v.z;
        n[e + 3] = v.w;
        sum += v.x + v.y + v.z + v.w;
      }
      uint32_t before = block_scan(sum, &all);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (before < need && need <= before + n[e]) {  // one thread
          found[0] = static_cast<uint32_t>(kEvictBins - 1 - (t * E + e));
          found[1] = need - before;
          found[2] = n[e];
        }
        before += n[e];
      }
      __syncthreads();
      thr |= found[0] << shift;
      need = found[1];
      equals = found[2];
    }
  }

  // ------------------------------------------------------------------ what stays, a bit per row
#pragma unroll 2
  for (int w = warp; w < nw; w += W) {
    const int i = r0 + w * 32 + lane;
    const bool in_mid = i >= mid0 && i < mid1;
    const uint32_t k = want > 0 && in_mid ? score_key(cached ? cache[i - r0] : score[i]) : 0;
    const bool tie = want > 0 && in_mid && k == thr;
    const uint32_t ties = __ballot_sync(0xFFFFFFFFu, tie);
    const uint32_t stay = __ballot_sync(0xFFFFFFFFu, i < L && (!in_mid || (want > 0 && k > thr)));
    if (lane == 0) {
      mask[w] = stay | (equals <= need ? ties : 0);
      count[w] = ties;
    }
  }
  __syncthreads();
  const int run = (nw + T - 1) / T, w0 = min(nw, t * run), w1 = min(nw, w0 + run);
  uint32_t all;
  if (equals > need) {  // the first ones only
    uint32_t n = 0;
    for (int w = w0; w < w1; ++w) n += __popc(count[w]);
    uint32_t seen = block_scan(n, &all);
    seen += ranks_before(0, all);
    for (int w = w0; w < w1; ++w) {
      const uint32_t ties = count[w];
      uint32_t take = ties;
      for (int drop = static_cast<int>(seen + __popc(ties)) - static_cast<int>(need); drop > 0 && take; --drop) take &= ~(0x80000000u >> __clz(take));
      mask[w] |= take;
      seen += __popc(ties);
    }
  }
  uint32_t n = 0;
  for (int w = w0; w < w1; ++w) n += __popc(mask[w]);
  uint32_t before = block_scan(n, &all);
  before += ranks_before(1, all);
  for (int w = w0; w < w1; ++w) {
    count[w] = before;
    before += __popc(mask[w]);
  }
  __syncthreads();

  // ------------------------------------------------------------------ the move
  // rows of the layer, by their place in it (32 bits: 2^32 rows are more than the device holds)
  const size_t layer_elems = static_cast<size_t>(layer) * a.num_pages * a.n_kv * (kPage * HD);
  auto place_of = [&](int i) { return (static_cast<uint32_t>(pages[i / kPage]) * a.n_kv + h) * kPage + i % kPage; };
  auto row_ptr = [&](int c, uint32_t at) {  // word c of a place's K, then V
    return reinterpret_cast<uint4*>((c < V ? a.k_pool : a.v_pool) + layer_elems + static_cast<size_t>(at) * HD) + c % V;
  };
  // kept rows [first, first + kWindow) into the list of the CTA that moves them (RB rows each in turn)
  auto list = [&](int first) {
    for (int w = warp; w < nw; w += W) {  // a lane per row
      const uint32_t m = mask[w];
      const int j = static_cast<int>(count[w] + __popc(m & ((1u << lane) - 1))) - first;
      if ((m >> lane & 1) && j >= 0 && j < kWindow) {
        const int i = r0 + w * 32 + lane;
        const uint32_t at = place_of(i);
        if (cs > 1) {
          st_dsmem_u32(mapa_shared(smem_u32(&win[j]), (j / RB) % cs), static_cast<uint32_t>(i));
          st_dsmem_u32(mapa_shared(smem_u32(&place[j]), (j / RB) % cs), at);
        } else {
          win[j] = static_cast<uint32_t>(i);
          place[j] = at;
        }
        if (kept) kept[first + j] = i;
      }
    }
  };
  const int step = cs * RB;
#pragma unroll 1
  for (int first = 0; first < a.budget; first += step) {
    if (first % kWindow == 0) {
      list(first);  // (all have read the former list: they are past the barrier of its last batch)
      sync_all();
    }
    // this thread's words of the batch: of K and V rows, a score
    const int j0 = first + rank * RB;
    uint4 v[U];
    float sc = 0.0f;
    uint32_t moved = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int y = u * T + t, j = j0 + y / (2 * V), c = y % (2 * V);
      if (j < a.budget && static_cast<int>(win[j % kWindow]) != j) {
        v[u] = *row_ptr(c, place[j % kWindow]);
        moved |= 1u << u;
      }
    }
    const bool has_score = score && t < RB && j0 + t < a.budget;
    if (has_score) sc = score[win[(j0 + t) % kWindow]];
    sync_all();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int y = u * T + t, j = j0 + y / (2 * V), c = y % (2 * V);
      if (moved >> u & 1) *row_ptr(c, place_of(j)) = v[u];
    }
    if (has_score) score[j0 + t] = sc;
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
