// sample.cuh -- one token from each row of logits, with temperature, top-k,
// top-p, min-p and the caller's uniforms.
//
// Weights w_v = exp((x_v - max x) / T).  In the order of falling logits (equal
// logits: lowest id first) the kept tokens are a prefix: the first k; of
// those the shortest prefix whose mass reaches p times their mass; of those
// the ones with w >= min_p.  So each filter is one threshold logit and a
// number of its equals, and the strictest holds.  The token is the smallest
// id whose cumulative kept mass reaches u times the total.
//
// A token id has to be the one that the definition gives, whatever the order
// of summation, so weights are integers of 2^-44 (sums below 2^18 tokens stay
// under 2^62) and every sum is exact.
#pragma once

#include "vsd_common.cuh"

namespace vsd {

constexpr int kMaxSampleVocab = 1 << 18;
constexpr int kWeightBits = 44;

struct SampleRowArgs {
  const float* logits;  // [rows][ld]
  long long ld;
  int rows, vocab;
  const float* temperature;  // [rows] or nullptr (1)
  const int* top_k;          // [rows] or nullptr (off)
  const float* top_p;        // [rows] or nullptr (off)
  const float* min_p;        // [rows] or nullptr (off)
  const float* u;            // [rows]
  int* tokens;               // [rows]
  float* logprob;            // [rows] or nullptr
};

// Key of a logit in the order of the definition; 0 for those that are never
// sampled (NaN, -inf); -0 equal to +0.
__device__ __forceinline__ uint32_t logit_key(float x) {
  return (x != x || x == -INFINITY) ? 0u : float_order_key(x + 0.0f);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}

constexpr int kSampleThreads = 512;

// One CTA per row, the logits re-read (from L2) by each pass.
__global__ void __launch_bounds__(kSampleThreads) sample_logits_kernel(const SampleRowArgs a) {
  constexpr int W = kSampleThreads / 32;
  __shared__ unsigned long long red[W];
  __shared__ int hist[256];
  __shared__ unsigned long long mass[256];
  __shared__ uint32_t s_key;
  __shared__ int s_need, s_tok;
  __shared__ unsigned long long s_left;
  const int row = blockIdx.x, t = threadIdx.x, warp = t >> 5, lane = t & 31, V = a.vocab;
  const float* x = a.logits + row * a.ld;
  auto block_sum = [&](unsigned long long v) {
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    __syncthreads();
    if (lane == 0) red[warp] = v;
    __syncthreads();
    v = 0;
    for (int w = 0; w < W; ++w) v += red[w];
    return v;
  };
  // the largest logit, lowest id first
  unsigned long long best = 0;
  for (int i = t; i < V; i += kSampleThreads) {
    const uint32_t k = logit_key(x[i]);
    if (k) best = max(best, (static_cast<unsigned long long>(k) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(i)));
  }
  for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xFFFFFFFFu, best, o));
  if (lane == 0) red[warp] = best;
  __syncthreads();
  best = 0;
  for (int w = 0; w < W; ++w) best = max(best, red[w]);
  const float T = a.temperature ? a.temperature[row] : 1.0f;
  if (best == 0 || !(T > 0.0f)) {
    if (t == 0) {
      a.tokens[row] = best ? static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(best)) : -1;
      if (a.logprob) a.logprob[row] = best ? 0.0f : -INFINITY;
    }
    return;
  }
  const uint32_t max_key = static_cast<uint32_t>(best >> 32);
  const double mx = key_logit(max_key), inv_t = 1.0 / static_cast<double>(T);
  auto weight = [&](uint32_t key) -> unsigned long long {
    if (key == 0) return 0;
    if (key == max_key) return 1ull << kWeightBits;
    const double z = (static_cast<double>(key_logit(key)) - mx) * inv_t;
    if (!(z > -100.0)) return 0;  // far below half a step (also an infinite maximum)
    return static_cast<unsigned long long>(__double2ll_rn(exp(z) * static_cast<double>(1ull << kWeightBits)));
  };
  // kept: key > thr, and the first `ties` ids of key == thr
  uint32_t thr = 0;
  int ties = 0;
  auto tighten = [&](uint32_t k, int n) {
    if (k > thr) {
      thr = k;
      ties = n;
    } else if (k == thr) {
      ties = min(ties, n);
    }
  };
  const int top_k = a.top_k ? a.top_k[row] : 0;
  if (top_k > 0 && top_k < V) {
    uint32_t prefix = 0;
    int need = top_k;
    for (int shift = 24; shift >= 0; shift -= 8) {
      __syncthreads();
      if (t < 256) hist[t] = 0;
      __syncthreads();
      for (int i = t; i < V; i += kSampleThreads) {
        const uint32_t k = logit_key(x[i]);
        if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255], 1);
      }
      __syncthreads();
      if (t == 0) {
        int d = 255, left = need;
        for (; d > 0 && hist[d] < left; --d) left -= hist[d];
        s_key = prefix | (static_cast<uint32_t>(d) << shift);
        s_need = left;
      }
      __syncthreads();
      prefix = s_key;
      need = s_need;
    }
    tighten(prefix, need);
  }
  const float top_p = a.top_p ? a.top_p[row] : 1.0f;
  if (top_p < 1.0f) {
    // mass of the tokens kept so far
    unsigned long long sum = 0;
    for (int i = t; i < V; i += kSampleThreads) {
      const uint32_t k = logit_key(x[i]);
      if (k > thr) sum += weight(k);
    }
    const unsigned long long total = block_sum(sum) + (thr ? static_cast<unsigned long long>(ties) * weight(thr) : 0);
    // digit by digit: the key at which the mass from the top reaches p * total
    const double target = fmax(static_cast<double>(top_p), 0.0) * static_cast<double>(total);
    unsigned long long goal = static_cast<unsigned long long>(ceil(target));
    if (goal == 0) goal = 1;
    uint32_t prefix = 0;
    unsigned long long left = goal;
    for (int shift = 24; shift >= 0; shift -= 8) {
      __syncthreads();
      if (t < 256) mass[t] = 0;
      __syncthreads();
      for (int i = t; i < V; i += kSampleThreads) {
        const uint32_t k = logit_key(x[i]);
        if (k <= thr) continue;
        if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&mass[(k >> shift) & 255], weight(k));
      }
      if (t == 0 && thr && (shift == 24 || (thr >> (shift + 8)) == (prefix >> (shift + 8))))
        atomicAdd(&mass[(thr >> shift) & 255], static_cast<unsigned long long>(ties) * weight(thr));
      __syncthreads();
      if (t == 0) {
        int d = 255;
        unsigned long long l = left;
        for (; d > 0 && mass[d] < l; --d) l -= mass[d];
        s_key = prefix | (static_cast<uint32_t>(d) << shift);
        s_left = l;
      }
      __syncthreads();
      prefix = s_key;
      left = s_left;
    }
    const unsigned long long w = weight(prefix);
    const unsigned long long n = w ? (left + w - 1) / w : static_cast<unsigned long long>(V);
    tighten(prefix, static_cast<int>(min(n, static_cast<unsigned long long>(V))));
  }
  const float min_p = a.min_p ? a.min_p[row] : 0.0f;
  const unsigned long long floor_w =
      min_p > 0.0f ? static_cast<unsigned long long>(ceil(fmin(static_cast<double>(min_p), 1.0) * static_cast<double>(1ull << kWeightBits))) : 1ull;
  // total of the kept tokens, by chunks of consecutive ids: each warp owns a range
  const int per = (V + W - 1) / W, w0 = min(V, warp * per), w1 = min(V, w0 + per);
  unsigned long long sum = 0;
  int eq = 0;  // equals of the threshold in this warp's range
  for (int i = w0 + lane; i < w1; i += 32) {
    const uint32_t k = logit_key(x[i]);
    if (k > thr) {
      const unsigned long long w = weight(k);
      if (w >= floor_w) sum += w;
    } else if (k == thr && k) {
      ++eq;
    }
  }
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    eq += __shfl_xor_sync(0xFFFFFFFFu, eq, o);
  }
  __syncthreads();
  if (lane == 0) {
    mass[warp] = sum;
    hist[warp] = eq;
  }
  __syncthreads();
  const unsigned long long wt0 = weight(thr), wt = wt0 >= floor_w ? wt0 : 0;
  unsigned long long before = 0, total = 0;
  int eq_before = 0, eq_all = 0;
  for (int w = 0; w < W; ++w) {
    const unsigned long long m = mass[w] + wt * static_cast<unsigned long long>(max(0, min(hist[w], ties - eq_all)));
    if (w < warp) {
      before += m;
      eq_before += hist[w];
    }
    eq_all += hist[w];
    total += m;
  }
  const float uf = a.u[row];
  unsigned long long goal = static_cast<unsigned long long>(ceil(fmin(fmax(static_cast<double>(uf), 0.0), 1.0) * static_cast<double>(total)));
  goal = max(1ull, min(goal, total));
  if (t == 0) s_tok = -1;
  __syncthreads();
  // the range that holds the goal: its warp walks it 32 ids at a time
  const unsigned long long mine =
      mass[warp] + wt * static_cast<unsigned long long>(max(0, min(hist[warp], ties - eq_before)));
  if (before < goal && goal <= before + mine) {
    unsigned long long run = before;
    int seen = eq_before;
    for (int i0 = w0; i0 < w1; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t k = i < w1 ? logit_key(x[i]) : 0;
      const bool tie = k && k == thr;
      const unsigned tb = __ballot_sync(0xFFFFFFFFu, tie);
      unsigned long long w = 0;
      if (k > thr) {
        w = weight(k);
        if (w < floor_w) w = 0;
      } else if (tie && seen + __popc(tb & ((1u << lane) - 1)) < ties) {
        w = wt;
      }
      seen += __popc(tb);
      unsigned long long c = w;
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xFFFFFFFFu, c, o);
        if (lane >= o) c += y;
      }
      const unsigned hit = __ballot_sync(0xFFFFFFFFu, w > 0 && run + c >= goal);
      if (hit) {
        if (lane == __ffs(hit) - 1) {
          a.tokens[row] = i;
          if (a.logprob)
            a.logprob[row] = static_cast<float>((k == max_key ? 0.0 : (static_cast<double>(key_logit(k)) - mx) * inv_t) -
                                                log(static_cast<double>(total) / static_cast<double>(1ull << kWeightBits)));
        }
        break;
      }
      run += __shfl_sync(0xFFFFFFFFu, c, 31);
    }
  }
}

}  // namespace vsd
