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
// of summation, so weights are integers (2^-44 of a power of two above the
// largest; 2^18 of them stay under 2^63) and every sum is exact.  Their
// relative error has to be far below a token's share of a 150,000-token row,
// which float32 is not: with c = 32 / (T ln 2) in two floats, x c = N + f,
// 2^(N / 32) from a table of 32 pairs and an exponent, exp(f ln 2 / 32) by its
// series in pairs, about 2^-37 in 45 float32 instructions (float64 runs at a
// fiftieth of their rate here).
//
// Rows without filters (sample_plain_kernel) are streamed once; each tile of
// 512 tokens leaves its sum, against a power of two of its own, and the tile
// that holds the sampled mass is read again.
//
// With filters (sample_logits_kernel) a row's logits are read once into the
// shared memory of a cluster of CTAs.  A histogram of their distance from the
// maximum (counts, merged through distributed shared memory) bounds the
// tokens that can be kept; where they are few (1024: nearly always), they are
// gathered in id order in one CTA, which finishes the row alone -- a cluster
// barrier costs about a microsecond, a block's barrier a twentieth.  Else the
// thresholds are found by 11-bit digits of the ordered key over the cluster.
#pragma once

#include "vsd_common.cuh"

namespace vsd {

constexpr int kMaxSampleVocab = 1 << 18;
constexpr int kWeightBits = 44;

struct SampleRowArgs {
  const float* logits;  // [rows][ld]
  long long ld;
  int rows, vocab;
  int cs, per;               // CTAs per row, tokens per CTA (a multiple of 4)
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

// 2^(i / 32) as pairs.
__device__ const float2 kPow32[32] = {
    {0x1.0000000000000p+0f, 0x0.0p+0f}, {0x1.059b0e0000000p+0f, -0x1.9d4f520000000p-25f}, {0x1.0b55860000000p+0f, 0x1.9f31220000000p-25f},
    {0x1.11301e0000000p+0f, -0x1.fdb4960000000p-25f}, {0x1.172b840000000p+0f, -0x1.c157420000000p-27f}, {0x1.1d48740000000p+0f, -0x1.d2e8ca0000000p-25f},
    {0x1.2387a60000000p+0f, 0x1.ceac480000000p-25f}, {0x1.29e9e00000000p+0f, -0x1.5c04240000000p-25f}, {0x1.306fe00000000p+0f, 0x1.4636e20000000p-25f},
    {0x1.371a740000000p+0f, -0x1.18aac60000000p-25f}, {0x1.3dea640000000p+0f, 0x1.8246840000000p-25f}, {0x1.44e0860000000p+0f, 0x1.8624b40000000p-30f},
    {0x1.4bfdae0000000p+0f, -0x1.593abc0000000p-25f}, {0x1.5342b60000000p+0f, -0x1.2c56100000000p-25f}, {0x1.5ab07e0000000p+0f, -0x1.5bd5ec0000000p-27f},
    {0x1.6247ec0000000p+0f, -0x1.f8b5500000000p-25f}, {0x1.6a09e60000000p+0f, 0x1.9fcef40000000p-26f}, {0x1.71f75e0000000p+0f, 0x1.1d8bee0000000p-25f},
    {0x1.7a11480000000p+0f, -0x1.829fd00000000p-25f}, {0x1.82589a0000000p+0f, -0x1.accc7c0000000p-26f}, {0x1.8ace540000000p+0f, 0x1.15506e0000000p-27f},
    {0x1.93737c0000000p+0f, -0x1.e647440000000p-25f}, {0x1.9c49180000000p+0f, 0x1.51f8480000000p-27f}, {0x1.a5503c0000000p+0f, -0x1.b83b540000000p-25f},
    {0x1.ae89fa0000000p+0f, -0x1.a94b140000000p-26f}, {0x1.b7f7700000000p+0f, -0x1.a094380000000p-25f}, {0x1.c199be0000000p+0f, -0x1.3d56b20000000p-27f},
    {0x1.cb720e0000000p+0f, -0x1.8837cc0000000p-27f}, {0x1.d5818e0000000p+0f, -0x1.822dbc0000000p-27f}, {0x1.dfc9740000000p+0f, -0x1.908c940000000p-25f},
    {0x1.ea4afa0000000p+0f, 0x1.52486c0000000p-27f}, {0x1.f507660000000p+0f, -0x1.246eb00000000p-26f}};

// A row's weights.
struct RowWeights {
  float sh, low;   // x' = max(x - sh, low)
  float ch, cl;    // c = 32 / (T ln 2)
  float mo;        // N of the power of two next to the largest weight
  int n_off;       // bits of the rounding constant plus that N
};
constexpr float kRoundMagic = 12582912.0f;  // 1.5 * 2^23: adding it rounds to an integer

// c, capped where 1 / T leaves float32: no two different logits share the mass at one end, all share it at the other.
__device__ __forceinline__ double temperature_scale(float T) {
  return fmin(fmax(46.166241308446828 / static_cast<double>(T), 1e-30), 1e30);
}

// x c must round to an integer below 2^22; beyond that only logits within a
// factor of two of the maximum have weight, and their difference from it is exact.
__device__ __forceinline__ bool needs_shift(float mx, float ch) { return !(fabsf(mx) * ch < 2097152.0f); }

// Weights for logits up to mx (shifted by sh); drop = 1600 / c: that far below, a weight of 2^-50 is nothing.
__device__ __forceinline__ RowWeights row_weights(float mx, float ch, float cl, float sh, float drop) {
  RowWeights r;
  r.ch = ch;
  r.cl = cl;
  r.sh = sh;
  const float m = mx - sh;
  r.low = fmaxf(m - drop, -3.0e38f);
  r.mo = floorf(m * ch * (1.0f / 32.0f)) * 32.0f + 32.0f;  // weights below 1 (and a little)
  r.n_off = __float_as_int(kRoundMagic) + static_cast<int>(r.mo);
  return r;
}

// ceil(share * total), exactly; share in [0, 1] (NaN counts as 0).
__device__ __forceinline__ unsigned long long share_of(unsigned long long total, float share) {
  if (!(share > 0.0f)) return 0;
  if (share >= 1.0f) return total;
  const uint32_t bits = __float_as_uint(share), e = bits >> 23;
  const unsigned long long m = (bits & 0x7FFFFFu) | (e ? 0x800000u : 0u);
  const int s = 150 - static_cast<int>(e ? e : 1u);  // share = m 2^-s, s >= 24
  const unsigned long long hi = __umul64hi(total, m), lo = total * m;
  if (s >= 88) return total != 0;  // the product is below 2^88
  unsigned long long q, rest;
  if (s < 64) {
    q = (hi << (64 - s)) | (lo >> s);
    rest = lo << (64 - s);
  } else {
    q = hi >> (s - 64);
    rest = (s > 64 ? hi << (128 - s) : 0) | lo;
  }
  return q + (rest != 0);
}

// Weight of logit x, in 2^-44; tab: this lane's column of the table.
__device__ __forceinline__ unsigned long long row_weight(const RowWeights& r, float x, const float2* tab) {
  x = fmaxf(x - r.sh, r.low);  // NaN and -inf come out as nothing
  const float uh = __fmul_rn(x, r.ch);  // not to be contracted into the sums below
  const float ul = fmaf(x, r.cl, fmaf(x, r.ch, -uh));
  const float tm = uh + kRoundMagic;
  const float f0 = uh - (tm - kRoundMagic);
  const float f = f0 + ul, fl = ul - (f - f0);  // ul reaches 2^-3 where x c reaches 2^21
  // z = (f + fl) ln 2 / 32
  constexpr float kh = 0x1.62e4300000000p-6f, kl = -0x1.05c6100000000p-34f;
  const float zh = f * kh;
  const float zl = fmaf(fl, kh, fmaf(f, kl, fmaf(f, kh, -zh)));
  const float q = zh * zh * fmaf(zh, fmaf(zh, 1.0f / 24.0f, 1.0f / 6.0f), 0.5f);
  const float sl = zl + q;
  const int n = __float_as_int(tm) - r.n_off;
  const float2 t2 = tab[(n & 31) * 32];
  const float sc = __int_as_float(((n >> 5) + 127) << 23);
  const float ph = t2.x * zh;
  const float pl = fmaf(t2.x, sl, fmaf(t2.y, zh, t2.y) + fmaf(t2.x, zh, -ph));
  // (t + ph + pl) 2^k as integers of 2^-22 and 2^-44
  const float h = t2.x * sc, p = ph * sc, l = pl * sc;
  const float e1 = p + l;
  const float eh = h + e1;
  const float el = (e1 - (eh - h)) + (l - (e1 - p));
  const float i1 = eh + 2.0f;
  const float i2 = ((eh - (i1 - 2.0f)) + el) + 0x1.8p-21f;
  const int a = __float_as_int(i1) - __float_as_int(2.0f), b = __float_as_int(i2) - __float_as_int(0x1.8p-21f);
  return (static_cast<unsigned long long>(static_cast<unsigned int>(a)) << 22) + static_cast<long long>(b);
}

// log of logit x's share of a mass (by one thread of a row: float64).
__device__ __forceinline__ float log_share(const RowWeights& r, float x, float T, unsigned long long total) {
  const double z = (static_cast<double>(x) - static_cast<double>(r.sh)) * temperature_scale(T) - static_cast<double>(r.mo);
  return static_cast<float>(z * 0.021660849392498290 - log(static_cast<double>(total) * (1.0 / static_cast<double>(1ull << kWeightBits))));
}

constexpr int kSampleThreads = 1024;
constexpr int kSampleBins = 2048;
constexpr int kSampleMaxCluster = 8;
constexpr int kSampleList = 1024;  // an entry a thread

// In front of the row's slice.
struct alignas(16) SampleShared {
  float2 tab[32 * 32];                  // [entry][lane]: no bank conflicts
  uint32_t hist[4][kSampleBins];        // masses in 16-bit parts (64-bit atomics are loops here), counts
  unsigned long long list[kSampleList]; // rank 0's: candidates, (key, ~id): larger = earlier in falling order
  unsigned long long ord[kSampleList], vals[kSampleList];
  unsigned long long xch[2][kSampleMaxCluster][3];  // values of each rank
  unsigned long long red[kSampleThreads / 32];
  unsigned long long found[4];          // what the thread that holds a border says
  uint32_t n_list, members;
  float scale[2];                       // c of the row
};

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void st_dsmem_u64(uint32_t addr, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ unsigned long long ld_dsmem_u64(uint32_t addr) {
  unsigned long long v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t atom_add_dsmem(uint32_t addr, uint32_t v) {
  uint32_t old;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(addr), "r"(v) : "memory");
  return old;
}

__device__ __forceinline__ uint32_t ld_dsmem_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
// Adds a weight (below 2^48) to a bin; 2^16 weights fit.
__device__ __forceinline__ void add_mass(uint32_t (*hist)[kSampleBins], int bin, unsigned long long w) {
  const uint32_t low = static_cast<uint32_t>(w), high = static_cast<uint32_t>(w >> 32);
  atomicAdd(&hist[0][bin], low & 0xFFFFu);
  if (low >> 16) atomicAdd(&hist[1][bin], low >> 16);
  if (high) atomicAdd(&hist[2][bin], high);
}

// Inclusive sum over the warp's lanes up to this one.
__device__ __forceinline__ unsigned long long warp_scan(unsigned long long v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

__global__ void __launch_bounds__(kSampleThreads, 1) sample_logits_kernel(const SampleRowArgs a) {
  extern __shared__ __align__(16) uint8_t sample_smem[];
  SampleShared& sh = *reinterpret_cast<SampleShared*>(sample_smem);
  float* xs = reinterpret_cast<float*>(sample_smem + sizeof(SampleShared));
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31, cs = a.cs;
  const int row = static_cast<int>(blockIdx.x) / cs, rank = static_cast<int>(blockIdx.x) % cs;
  const int id0 = min(a.vocab, rank * a.per), n = min(a.vocab, id0 + a.per) - id0;
  const float* src = a.logits + row * a.ld + id0;
  const float T = a.temperature ? a.temperature[row] : 1.0f;
  if (t == 0) sh.n_list = 0;
  if (cs > 1) cluster_arrive();  // the others' memory is touched once all have started
  const float2* tab = sh.tab + lane;

  auto sync_all = [&]() {
    if (cs > 1) cluster_sync();
    else __syncthreads();
  };
  // Three values (the same in every thread) of this rank to all ranks; returns the sums over all ranks in v and over the
  // ranks before this one in pre.  Two buffers in turn.
  int turn = 0;
  auto exchange = [&](unsigned long long* v, unsigned long long* pre) {
    turn ^= 1;
    for (int x = t; x < 3 * cs; x += kSampleThreads)
      st_dsmem_u64(mapa_shared(smem_u32(&sh.xch[turn][rank][x % 3]), x / 3), x % 3 == 0 ? v[0] : x % 3 == 1 ? v[1] : v[2]);
    sync_all();
    v[0] = v[1] = v[2] = pre[0] = pre[1] = pre[2] = 0;
    for (int r = 0; r < cs; ++r)
#pragma unroll
      for (int e = 0; e < 3; ++e) {
        if (r < rank) pre[e] += sh.xch[turn][r][e];
        v[e] += sh.xch[turn][r][e];
      }
  };
  // sum over the CTA's threads, and the sum over the threads before this one
  auto block_scan = [&](unsigned long long v, unsigned long long* before) {
    const unsigned long long c = warp_scan(v, lane);
    __syncthreads();
    if (lane == 31) sh.red[warp] = c;
    __syncthreads();
    const unsigned long long all = warp_scan(sh.red[lane], lane), pre = __shfl_sync(0xFFFFFFFFu, all, max(warp, 1) - 1);
    *before = (warp ? pre : 0) + c - v;
    return __shfl_sync(0xFFFFFFFFu, all, 31);
  };

  // ------------------------------------------------------------------ the slice, and the largest logit (lowest id first)
  unsigned long long best = 0;
  auto look = [&](float x, int i) {
    const uint32_t k = logit_key(x);
    const unsigned long long v = (static_cast<unsigned long long>(k) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(id0 + i));
    best = k && v > best ? v : best;
  };
  {
    // 16-byte loads from the first aligned address on; xs shifted alike
    const int head = min(n, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(src) & 15)) & 15) / 4);
    xs += (4 - head) & 3;
    const int n4 = (n - head) / 4;
    const float4* s4 = reinterpret_cast<const float4*>(src + head);
    float4* d4 = reinterpret_cast<float4*>(xs + head);
#pragma unroll 1
    for (int i0 = t; i0 < n4; i0 += 4 * kSampleThreads) {
      float4 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (i0 + u * kSampleThreads < n4) v[u] = __ldcs(s4 + i0 + u * kSampleThreads);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + u * kSampleThreads;
        if (i < n4) {
          d4[i] = v[u];
          look(v[u].x, head + 4 * i);
          look(v[u].y, head + 4 * i + 1);
          look(v[u].z, head + 4 * i + 2);
          look(v[u].w, head + 4 * i + 3);
        }
      }
    }
    sh.tab[t] = kPow32[t >> 5];
    if (t == kSampleThreads - 1) {
      const double c = temperature_scale(T);
      sh.scale[0] = static_cast<float>(c);
      sh.scale[1] = static_cast<float>(c - static_cast<double>(sh.scale[0]));
    }
    const int rest = n - head - 4 * n4;  // and the ragged ends
    if (t < head + rest) {
      const int i = t < head ? t : head + 4 * n4 + t - head;
      const float x = src[i];
      xs[i] = x;
      look(x, i);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long y = __shfl_xor_sync(0xFFFFFFFFu, best, o);
    best = y > best ? y : best;
  }
  if (lane == 0) sh.red[warp] = best;
  __syncthreads();
  best = sh.red[lane];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long y = __shfl_xor_sync(0xFFFFFFFFu, best, o);
    best = y > best ? y : best;
  }
  if (cs > 1) {
    cluster_wait();
    unsigned long long v[3] = {best, 0, 0}, pre[3];
    exchange(v, pre);
    for (int r = 0; r < cs; ++r) best = sh.xch[turn][r][0] > best ? sh.xch[turn][r][0] : best;
  }
  if (best == 0 || !(T > 0.0f)) {  // the whole cluster alike
    if (rank == 0 && t == 0) {
      a.tokens[row] = best ? static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(best)) : -1;
      if (a.logprob) a.logprob[row] = best ? 0.0f : -INFINITY;
    }
    return;
  }
  uint32_t max_key = static_cast<uint32_t>(best >> 32);
  if (key_logit(max_key) == INFINITY) {  // the infinite logits share the mass: zeros among nothing
    for (int i = t; i < n; i += kSampleThreads) xs[i] = xs[i] == INFINITY ? 0.0f : -INFINITY;
    max_key = logit_key(0.0f);
    __syncthreads();
  }
  const float mx = key_logit(max_key);
  const RowWeights rw =
      row_weights(mx, sh.scale[0], sh.scale[1], needs_shift(mx, sh.scale[0]) ? mx : 0.0f, 1600.0f / sh.scale[0]);
  const int top_k = a.top_k ? a.top_k[row] : 0;
  const float top_p = a.top_p ? a.top_p[row] : 1.0f, min_p = a.min_p ? a.min_p[row] : 0.0f;
  bool cut_k = top_k > 0 && top_k < a.vocab, cut_p = top_p < 1.0f;
  const unsigned long long floor_w = max(1ull, share_of(row_weight(rw, mx, tab), min_p));
  // kept: key > thr, and the first `ties` ids of key == thr, of which there are `equals`
  uint32_t thr = 0;
  int ties = 0, equals = 0;

  // ------------------------------------------------------------------ the tokens that decide, gathered where they are few
  if (cut_k || cut_p) {
    // bins of equal widths below the maximum, the last for all the rest: for counts of 1/64, for masses of 1/51.2 octave, so
    // that 40 octaves are covered
    const float per_unit = cut_k ? 64.0f : 1.6f * rw.ch;
    auto place = [&](float x) { return fminf((mx - fmaxf(x, -3.0e38f)) * per_unit, static_cast<float>(kSampleBins - 1)); };
    for (int i = t; i < 4 * kSampleBins; i += kSampleThreads) sh.hist[0][i] = 0;
    __syncthreads();
    unsigned long long before;
#pragma unroll 4
    for (int i = t; i < n; i += kSampleThreads) {
      const float x = xs[i];
      const int b = static_cast<int>(place(x));
      if (cut_k) {
        if (b < kSampleBins - 1) atomicAdd(&sh.hist[3][b], 1u);
      } else if (x > -INFINITY) {  // (also not NaN)
        atomicAdd(&sh.hist[3][b], 1u);
        add_mass(sh.hist, b, row_weight(rw, x, tab));
      }
    }
    sync_all();
    const int mine = kSampleBins / cs, each = max(1, mine / kSampleThreads), b0 = rank * mine + t * each;
    unsigned long long val[2], cnt[2], val_s = 0, cnt_s = 0, cnt_b;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      val[e] = cnt[e] = 0;
      if (e < each && t * each < mine)
        for (int r = 0; r < cs; ++r) {
          cnt[e] += ld_dsmem_u32(mapa_shared(smem_u32(&sh.hist[3][b0 + e]), r));
          if (!cut_k)
#pragma unroll
            for (int p = 0; p < 3; ++p)
              val[e] += static_cast<unsigned long long>(ld_dsmem_u32(mapa_shared(smem_u32(&sh.hist[p][b0 + e]), r))) << (16 * p);
        }
      if (cut_k) val[e] = cnt[e];
      val_s += val[e];
      cnt_s += cnt[e];
    }
    unsigned long long v[3], pre[3];
    v[0] = block_scan(val_s, &before);
    v[1] = block_scan(cnt_s, &cnt_b);
    v[2] = 0;
    exchange(v, pre);
    before += pre[0];
    cnt_b += pre[1];
    // the goal: k tokens, or p of the row's mass
    unsigned long long goal = cut_k ? static_cast<unsigned long long>(top_k) : max(1ull, share_of(v[0], top_p));
    if (v[0] >= goal) {  // the cluster alike (else there are fewer tokens than k, or the last bin hides the k-th)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (before < goal && goal <= before + val[e])  // one thread of the cluster
          for (int r = 0; r < cs; ++r) {
            st_dsmem_u64(mapa_shared(smem_u32(&sh.found[0]), r), static_cast<unsigned long long>(b0 + e));
            st_dsmem_u64(mapa_shared(smem_u32(&sh.found[1]), r), cnt_b + cnt[e]);
            st_dsmem_u64(mapa_shared(smem_u32(&sh.found[2]), r), cnt[e]);
            st_dsmem_u64(mapa_shared(smem_u32(&sh.found[3]), r), goal - before);
          }
        before += val[e];
        cnt_b += cnt[e];
      }
      sync_all();
      const int last = static_cast<int>(sh.found[0]);  // the bin in which the goal is reached
      const bool complete = sh.found[1] <= kSampleList;  // every token that can be kept fits; else the border bin's tokens may
      const int first = complete ? 0 : last;
      if (complete || sh.found[2] <= kSampleList) {
        if (!complete) goal = sh.found[3];
#pragma unroll 4
        for (int i0 = 0; i0 < n; i0 += kSampleThreads) {
          const int i = i0 + t;
          const float x = i < n ? xs[i] : -INFINITY;
          const int b = static_cast<int>(place(x));
          const bool in = b >= first && b <= last && x > -INFINITY;
          const uint32_t who = __ballot_sync(0xFFFFFFFFu, in);
          if (who) {
            uint32_t at = 0;
            if (lane == __ffs(who) - 1) at = atom_add_dsmem(mapa_shared(smem_u32(&sh.n_list), 0), __popc(who));
            at = __shfl_sync(0xFFFFFFFFu, at, __ffs(who) - 1) + __popc(who & ((1u << lane) - 1));
            if (in && at < kSampleList)
              st_dsmem_u64(mapa_shared(smem_u32(&sh.list[at]), 0),
                           (static_cast<unsigned long long>(logit_key(x)) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(id0 + i)));
          }
        }
        sync_all();
        if (complete && rank != 0) return;
        if (rank == 0) {
          // -------------------------------------------------------------- one CTA has the list: an entry a thread
          const int N = min(static_cast<int>(sh.n_list), kSampleList);
          const unsigned long long ent = t < N ? sh.list[t] : 0;
          const float x = key_logit(static_cast<uint32_t>(ent >> 32));
          const unsigned long long w = t < N ? row_weight(rw, x, tab) : 0;
          const float fine = static_cast<float>(kSampleList) / static_cast<float>(last - first + 1);
          const int bin = t < N ? max(0, min(kSampleList - 1, static_cast<int>((place(x) - static_cast<float>(first)) * fine))) : kSampleList - 1;
          bool keep = t < N;
          // Where the values v, in the order of falling `ord` (bins ascending), reach the goal: the border bin; an entry in it
          // gets what comes before it there, and the bin's part of the goal.
          auto reach = [&](unsigned long long ord, int b, unsigned long long val, unsigned long long to, int* border,
                           unsigned long long* ahead, unsigned long long* rest) {
            sh.hist[0][t] = sh.hist[1][t] = sh.hist[2][t] = 0;
            if (t == 0) sh.members = 0;
            __syncthreads();
            if (val) add_mass(sh.hist, b, val);
            __syncthreads();
            unsigned long long p;
            const unsigned long long h = sh.hist[0][t] + (static_cast<unsigned long long>(sh.hist[1][t]) << 16) +
                                         (static_cast<unsigned long long>(sh.hist[2][t]) << 32);
            block_scan(h, &p);
            if (p < to && to <= p + h) {
              sh.found[0] = static_cast<unsigned long long>(t);
              sh.found[1] = to - p;
            }
            __syncthreads();
            *border = static_cast<int>(sh.found[0]);
            *rest = sh.found[1];
            *ahead = 0;
            if (b == *border && val) {
              const uint32_t at = atomicAdd(&sh.members, 1u);
              sh.ord[at] = ord;
              sh.vals[at] = val;
            }
            __syncthreads();
            if (b == *border && val) {
              const int m = static_cast<int>(sh.members);
              for (int j = 0; j < m; ++j) *ahead += sh.ord[j] > ord ? sh.vals[j] : 0;
            }
            __syncthreads();
          };
          int border;
          unsigned long long ahead, rest;
#pragma unroll 1
          for (int step = cut_k ? 0 : 1; step < (cut_p && (complete || !cut_k) ? 2 : 1); ++step) {
            const unsigned long long val = keep ? (step ? w : 1) : 0;
            if (step && cut_k) goal = max(1ull, share_of(block_scan(val, &before), top_p));
            if (!step && goal >= static_cast<unsigned long long>(N)) continue;  // all stay
            reach(ent, bin, val, goal, &border, &ahead, &rest);
            keep = keep && (bin < border || (bin == border && val && ahead < rest));
          }
          if (complete) {
            const unsigned long long kw = keep && w >= floor_w ? w : 0;
            const unsigned long long total = block_scan(kw, &before);
            const uint32_t low = static_cast<uint32_t>(ent);  // ~id: larger = lower id
            const int id = static_cast<int>(0xFFFFFFFFu - low);
            reach(low, t < N ? min(kSampleList - 1, static_cast<int>(static_cast<float>(id) * (static_cast<float>(kSampleList) / a.vocab))) : 0, kw,
                  max(1ull, share_of(total, a.u[row])), &border, &ahead, &rest);
            if (kw && ahead < rest && rest <= ahead + kw &&
                border == min(kSampleList - 1, static_cast<int>(static_cast<float>(id) * (static_cast<float>(kSampleList) / a.vocab)))) {
              a.tokens[row] = id;
              if (a.logprob) a.logprob[row] = log_share(rw, x, T, total);
            }
            return;
          }
          // the smallest kept key and its numbers, for everybody
          uint32_t k = keep ? static_cast<uint32_t>(ent >> 32) : 0xFFFFFFFFu;
          k = __reduce_min_sync(0xFFFFFFFFu, k);
          if (lane == 0) sh.red[warp] = k;
          __syncthreads();
          k = __reduce_min_sync(0xFFFFFFFFu, static_cast<uint32_t>(sh.red[lane]));
          const bool eq = t < N && static_cast<uint32_t>(ent >> 32) == k;
          const int kept_eq = __syncthreads_count(eq && keep), all_eq = __syncthreads_count(eq);
          if (t < 3 * cs)
            st_dsmem_u64(mapa_shared(smem_u32(&sh.found[t % 3]), t / 3), t % 3 == 0 ? k : static_cast<unsigned long long>(t % 3 == 1 ? kept_eq : all_eq));
        }
        sync_all();
        thr = static_cast<uint32_t>(sh.found[0]);
        ties = static_cast<int>(sh.found[1]);
        equals = static_cast<int>(sh.found[2]);
        if (!cut_k) cut_p = false;  // done
        cut_k = false;
        sync_all();
      }
    }
  }

  // ------------------------------------------------------------------ thresholds by the key's digits, over the cluster
  // Finds the key at which a sum over tokens in falling order reaches a goal: tokens counted (goal = k), or their mass
  // (goal = share of the mass of those kept so far).
  auto select = [&](bool by_mass, float share, unsigned long long goal) {
    uint32_t prefix = 0;
    const unsigned long long w_thr = by_mass && thr ? row_weight(rw, key_logit(thr), tab) : 0;
#pragma unroll 1
    for (int level = 0; level < 3; ++level) {
      const int shift = level == 0 ? 21 : level == 1 ? 10 : 0, bits = level == 2 ? 10 : 11, bins = 1 << bits;
      for (int i = t; i < bins; i += kSampleThreads) sh.hist[0][i] = sh.hist[1][i] = sh.hist[2][i] = 0;
      __syncthreads();
#pragma unroll 2
      for (int i = t; i < n; i += kSampleThreads) {
        const float x = xs[i];
        const uint32_t k = logit_key(x);
        if (k == 0 || (level && (k >> (shift + bits)) != (prefix >> (shift + bits))) || (by_mass && k <= thr)) continue;
        const int bin = bins - 1 - ((k >> shift) & (bins - 1));  // largest first
        if (by_mass) add_mass(sh.hist, bin, row_weight(rw, x, tab));
        else atomicAdd(&sh.hist[0][bin], 1u);
      }
      sync_all();
      // this rank's share of the bins, over all ranks
      const int mine = bins / cs, each = max(1, mine / kSampleThreads), b0 = rank * mine + t * each;
      unsigned long long val[2], sum = 0, before, pre[3];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        val[e] = 0;
        if (e < each && t * each < mine)
          for (int r = 0; r < cs; ++r)
#pragma unroll
            for (int p = 0; p < 3; ++p)
              val[e] += static_cast<unsigned long long>(ld_dsmem_u32(mapa_shared(smem_u32(&sh.hist[p][b0 + e]), r))) << (16 * p);
        // the equals of an earlier threshold, as many as stay
        if (by_mass && thr && e < each && t * each < mine && (!level || (thr >> (shift + bits)) == (prefix >> (shift + bits))) &&
            b0 + e == bins - 1 - static_cast<int>((thr >> shift) & (bins - 1)))
          val[e] += w_thr * static_cast<unsigned long long>(ties);
        sum += val[e];
      }
      unsigned long long v[3] = {block_scan(sum, &before), 0, 0};
      exchange(v, pre);
      before += pre[0];
      if (level == 0) {
        if (by_mass) goal = max(1ull, share_of(v[0], share));
        else if (goal >= v[0]) return;  // no more tokens than that: nothing to cut
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (before < goal && goal <= before + val[e])  // one thread of the cluster
          for (int r = 0; r < cs; ++r) {
            st_dsmem_u64(mapa_shared(smem_u32(&sh.found[0]), r), static_cast<unsigned long long>(b0 + e));
            st_dsmem_u64(mapa_shared(smem_u32(&sh.found[1]), r), goal - before);
            st_dsmem_u64(mapa_shared(smem_u32(&sh.found[2]), r), val[e]);
          }
        before += val[e];
      }
      sync_all();
      prefix |= static_cast<uint32_t>(bins - 1 - static_cast<int>(sh.found[0])) << shift;
      goal = sh.found[1];
    }
    // of the border's equals, as many as the rest of the goal needs
    const unsigned long long v = sh.found[2], w = by_mass ? row_weight(rw, key_logit(prefix), tab) : 1;
    const int need = static_cast<int>((goal + w - 1) / w), have = static_cast<int>(v / w);
    if (prefix != thr) {
      thr = prefix;
      ties = need;
      equals = have;
    } else {
      ties = min(ties, need);
    }
    sync_all();  // everybody has read what was found
  };
  if (cut_k) select(false, 0.0f, static_cast<unsigned long long>(top_k));
  if (cut_p) select(true, top_p, 0);
  const unsigned long long w_thr0 = thr ? row_weight(rw, key_logit(thr), tab) : 0, w_thr = w_thr0 >= floor_w ? w_thr0 : 0;
  const bool all_ties = ties >= equals;  // every equal of the threshold stays (or there is none)
  // weight of token i of the slice; ties are left to the caller
  auto kept_weight = [&](int i, bool* tie) -> unsigned long long {
    const float x = xs[i];
    const uint32_t k = logit_key(x);
    *tie = k && k == thr;
    const unsigned long long w = k > thr ? row_weight(rw, x, tab) : 0;
    return w >= floor_w ? w : 0;
  };
  auto stay = [&](unsigned long long seen, unsigned long long here) -> unsigned long long {  // equals that stay, of `here` after `seen`
    if (all_ties) return here;
    return seen >= static_cast<unsigned long long>(ties) ? 0 : min(here, static_cast<unsigned long long>(ties) - seen);
  };

  // ------------------------------------------------------------------ total, and the token at the goal
  // a run of ids per thread (an odd number of them: no bank conflicts)
  const int len = ((n + kSampleThreads - 1) / kSampleThreads) | 1, i0 = min(n, t * len), i1 = min(n, i0 + len);
  unsigned long long mine = 0, before, seen = 0;
  unsigned int eq = 0;
#pragma unroll 4
  for (int i = i0; i < i1; ++i) {
    bool tie;
    mine += kept_weight(i, &tie);
    eq += tie;
  }
  unsigned long long v[3] = {0, 0, 0}, pre[3];
  if (!all_ties) {
    v[0] = block_scan(eq, &seen);
    exchange(v, pre);
    seen += pre[0];
  }
  mine += w_thr * stay(seen, eq);
  v[0] = block_scan(mine, &before);
  exchange(v, pre);
  before += pre[0];
  const unsigned long long total = v[0], goal = max(1ull, share_of(total, a.u[row]));
  const uint32_t hit = __ballot_sync(0xFFFFFFFFu, before < goal && goal <= before + mine);
  if (!hit) return;  // another warp's (no rank looks into another's memory from here on)
  const int who = __ffs(hit) - 1, end = __shfl_sync(0xFFFFFFFFu, i1, who);
  unsigned long long run = __shfl_sync(0xFFFFFFFFu, before, who);
  seen = __shfl_sync(0xFFFFFFFFu, seen, who);
#pragma unroll 1
  for (int base = __shfl_sync(0xFFFFFFFFu, i0, who); base < end; base += 32) {
    const int i = base + lane;
    bool tie = false;
    unsigned long long w = i < end ? kept_weight(i, &tie) : 0;
    const uint32_t tb = __ballot_sync(0xFFFFFFFFu, tie);
    if (tie) w = w_thr * stay(seen + __popc(tb & ((1u << lane) - 1)), 1);
    seen += __popc(tb);
    const unsigned long long c = run + warp_scan(w, lane);
    const uint32_t got = __ballot_sync(0xFFFFFFFFu, w > 0 && goal <= c);
    if (got) {
      if (lane == __ffs(got) - 1) {
        a.tokens[row] = id0 + i;
        if (a.logprob) a.logprob[row] = log_share(rw, xs[i], T, total);
      }
      break;
    }
    run = __shfl_sync(0xFFFFFFFFu, c, 31);
  }
}

// ------------------------------------------------------------------ rows without filters
constexpr int kPlainThreads = 256;
constexpr int kPlainTile = 512;  // tokens of a warp's tile
constexpr int kPlainMaxTiles = kMaxSampleVocab / kPlainTile;

__global__ void __launch_bounds__(kPlainThreads, 4) sample_plain_kernel(const SampleRowArgs a) {
  constexpr int W = kPlainThreads / 32, E = kPlainTile / 32;
  __shared__ float2 table[32 * 32];
  __shared__ unsigned long long tile_sum[kPlainMaxTiles];
  __shared__ float tile_mo[kPlainMaxTiles];  // the power of two that a tile's sum is against (32nds of an octave)
  __shared__ unsigned long long xch[3][kSampleMaxCluster], red[W];
  __shared__ float scale[2];
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31, cs = a.cs;
  const int row = static_cast<int>(blockIdx.x) / cs, rank = static_cast<int>(blockIdx.x) % cs;
  const int id0 = min(a.vocab, rank * a.per), n = min(a.vocab, id0 + a.per) - id0;
  const float* src = a.logits + row * a.ld + id0;
  const float T = a.temperature ? a.temperature[row] : 1.0f;
  if (cs > 1) cluster_arrive();
  for (int i = t; i < 32 * 32; i += kPlainThreads) table[i] = kPow32[i >> 5];
  if (t == 0) {
    const double c = temperature_scale(T);
    scale[0] = static_cast<float>(c);
    scale[1] = static_cast<float>(c - static_cast<double>(scale[0]));
  }
  const float2* tab = table + lane;
  if (cs > 1) cluster_wait();
  else __syncthreads();
  __syncthreads();
  // every rank's value, for all threads of all ranks; buffers in turn
  auto exchange = [&](int buf, unsigned long long v) -> const unsigned long long* {
    if (cs > 1) {
      if (t < cs) st_dsmem_u64(mapa_shared(smem_u32(&xch[buf][rank]), t), v);
      cluster_sync();
    } else {
      if (t == 0) xch[buf][0] = v;
      __syncthreads();
    }
    return xch[buf];
  };
  auto block_max = [&](unsigned long long v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long y = __shfl_xor_sync(0xFFFFFFFFu, v, o);
      v = y > v ? y : v;
    }
    __syncthreads();
    if (lane == 0) red[warp] = v;
    __syncthreads();
    for (int w = 0; w < W; ++w) v = red[w] > v ? red[w] : v;
    return v;
  };
  const int tiles = (n + kPlainTile - 1) / kPlainTile;
  const bool aligned = (reinterpret_cast<uintptr_t>(src) & 15) == 0;
  auto load = [&](int q, float* x) {
    const int base = q * kPlainTile;
    if (aligned && base + kPlainTile <= n) {
#pragma unroll
      for (int e = 0; e < E; e += 4) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(src + base) + (e / 4) * 32 + lane);
        x[e] = v.x;
        x[e + 1] = v.y;
        x[e + 2] = v.z;
        x[e + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int i = base + e * 32 + lane;
        x[e] = i < n ? src[i] : -INFINITY;
      }
    }
  };
  // id within the slice of element e of tile q as load() deals them
  auto id_of = [&](int q, int e) {
    const int base = q * kPlainTile;
    return base + (aligned && base + kPlainTile <= n ? ((e / 4) * 32 + lane) * 4 + (e & 3) : e * 32 + lane);
  };
  if (!(T > 0.0f)) {  // the largest logit, lowest id first
    unsigned long long best = 0;
    for (int q = warp; q < tiles; q += W) {
      float x[E];
      load(q, x);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const uint32_t k = logit_key(x[e]);
        const unsigned long long v =
            k ? (static_cast<unsigned long long>(k) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(id0 + id_of(q, e))) : 0;
        best = v > best ? v : best;
      }
    }
    best = block_max(best);
    const unsigned long long* all = exchange(0, best);
    for (int r = 0; r < cs; ++r) best = all[r] > best ? all[r] : best;
    if (rank == 0 && t == 0) {
      a.tokens[row] = best ? static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(best)) : -1;
      if (a.logprob) a.logprob[row] = best ? 0.0f : -INFINITY;
    }
    return;
  }
  const float ch = scale[0], cl = scale[1], drop = 1600.0f / ch;
  // Once over the row; a second time, shifted by the row's maximum, where some tile's values are too large for the first.
  float shift = 0.0f;
  bool infinite = false;  // then the infinite logits share the mass: zeros among nothing
  auto prepared = [&](float x) { return infinite ? (x == INFINITY ? 0.0f : -INFINITY) : fmaxf(x, -INFINITY); };  // NaN: -inf
  uint32_t top = 0;
  float mo = 0.0f;
#pragma unroll 1
  for (int pass = 0;; ++pass) {
    uint32_t my_top = 0;
    bool large = false;
    float my_mo = -INFINITY;
#pragma unroll 1
    for (int q = warp; q < tiles; q += W) {
      float x[E];
      load(q, x);
      float m = -INFINITY;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        x[e] = prepared(x[e]);
        m = fmaxf(m, x[e]);
      }
      const uint32_t key = __reduce_max_sync(0xFFFFFFFFu, logit_key(m));
      const float mx = key_logit(key);
      my_top = max(my_top, key);
      unsigned long long sum = 0;
      float t_mo = -INFINITY;
      if (key && (mx - shift) * ch > -2097152.0f && !needs_shift(mx - shift, ch)) {
        const RowWeights rw = row_weights(mx, ch, cl, shift, drop);
#pragma unroll
        for (int e = 0; e < E; ++e) sum += row_weight(rw, x[e], tab);
        t_mo = rw.mo;
      } else if (key && pass == 0) {
        large = true;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
      if (lane == 0) {
        tile_sum[q] = sum;
        tile_mo[q] = t_mo;
      }
      my_mo = fmaxf(my_mo, t_mo);
    }
    // (flag, largest key) and the largest power of two
    const unsigned long long v = block_max((static_cast<unsigned long long>(my_top) << 1) | (large ? 1 : 0));
    const bool cta_large = __syncthreads_or(large);
    const unsigned long long* all = exchange(0, (v & ~1ull) | (cta_large ? 1 : 0));
    bool again = false;
    top = 0;
    for (int r = 0; r < cs; ++r) {
      top = max(top, static_cast<uint32_t>(all[r] >> 1));
      again = again || (all[r] & 1);
    }
    const unsigned long long mv = block_max(my_mo == -INFINITY ? 0 : float_order_key(my_mo));
    const unsigned long long* mos = exchange(1, mv);
    uint32_t mk = 0;
    for (int r = 0; r < cs; ++r) mk = max(mk, static_cast<uint32_t>(mos[r]));
    mo = key_logit(mk);
    if (!again || pass == 1 || top == 0) break;
    shift = key_logit(top);
    if (shift == INFINITY) {
      infinite = true;
      shift = 0.0f;
    }
  }
  if (top == 0) {  // nothing to sample (the cluster alike)
    if (rank == 0 && t == 0) {
      a.tokens[row] = -1;
      if (a.logprob) a.logprob[row] = -INFINITY;
    }
    return;
  }
  // the tiles' sums against the row's power of two; a run of them per thread, in order
  auto octaves = [&](int q) { return tile_mo[q] == -INFINITY ? 63 : min(63, static_cast<int>(mo - tile_mo[q]) >> 5); };
  const int run_len = (tiles + kPlainThreads - 1) / kPlainThreads, q0 = min(tiles, t * run_len), q1 = min(tiles, q0 + run_len);
  unsigned long long mine = 0;
  for (int q = q0; q < q1; ++q) mine += tile_sum[q] >> octaves(q);
  unsigned long long c = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xFFFFFFFFu, c, o);
    if (lane >= o) c += y;
  }
  __syncthreads();
  if (lane == 31) red[warp] = c;
  __syncthreads();
  unsigned long long before = c - mine, own = 0;
  for (int w = 0; w < W; ++w) {
    if (w < warp) before += red[w];
    own += red[w];
  }
  const unsigned long long* all = exchange(2, own);
  unsigned long long total = 0;
  for (int r = 0; r < cs; ++r) {
    if (r < rank) before += all[r];
    total += all[r];
  }
  const unsigned long long goal = max(1ull, share_of(total, a.u[row]));
  const bool hit = before < goal && goal <= before + mine;
  if (!__any_sync(0xFFFFFFFFu, hit)) return;  // (no rank looks into another's memory from here on)
  // this warp finds the tile, reads it again and finds the token
  int q = 0;
  unsigned long long left = 0;
  if (hit) {
    for (q = q0; q < q1 - 1; ++q) {
      const unsigned long long s = tile_sum[q] >> octaves(q);
      if (goal <= before + s) break;
      before += s;
    }
    left = goal - before;
  }
  const int who = __ffs(__ballot_sync(0xFFFFFFFFu, hit)) - 1;
  q = __shfl_sync(0xFFFFFFFFu, q, who);
  left = __shfl_sync(0xFFFFFFFFu, left, who);
  left <<= octaves(q);  // in the tile's own units: at most its sum
  float x[E], m = -INFINITY;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int i = q * kPlainTile + lane * E + e;
    x[e] = i < n ? prepared(src[i]) : -INFINITY;
    m = fmaxf(m, x[e]);
  }
  const float mx = key_logit(__reduce_max_sync(0xFFFFFFFFu, logit_key(m)));
  const RowWeights rw = row_weights(mx, ch, cl, shift, drop);
  unsigned long long sum = 0;
#pragma unroll
  for (int e = 0; e < E; ++e) sum += row_weight(rw, x[e], tab);
  unsigned long long pre = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xFFFFFFFFu, pre, o);
    if (lane >= o) pre += y;
  }
  pre -= sum;
  if (pre < left && left <= pre + sum) {
    int found = 0;
    float xf = 0.0f;
    bool done = false;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      pre += row_weight(rw, x[e], tab);
      if (!done && left <= pre) {
        done = true;
        found = e;
        xf = x[e];
      }
    }
    a.tokens[row] = id0 + q * kPlainTile + lane * E + found;
    if (a.logprob) {
      RowWeights rr = rw;
      rr.mo = mo;
      a.logprob[row] = log_share(rr, xf, T, total);
    }
  }
}

}  // namespace vsd
