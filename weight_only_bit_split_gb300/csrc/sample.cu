// Sampling a token from each row of logits by temperature, top-k, top-p and
// min-p, from given random numbers.
//
// Tokens are ordered by value, largest first, lowest index first among equal
// ones.  With e_i = exp((x_i - max) / T) every filter keeps a prefix of that
// order: top-k the first k, top-p the shortest prefix of those whose mass
// reaches top_p of their mass, min-p the tokens with e_i >= min_p.  So of the
// three only the mass of the shortest prefix matters, and the token drawn is
// the first at which the running mass reaches a target.
//
// Masses are whole multiples of 2^-35, in two parts (of 2^-18, and the signed
// rest): their sums do not depend on the order in which threads add, so equal
// inputs give equal tokens.  A token whose mass rounds to 0 cannot be drawn and
// is left out.
//
// One cluster a row, each CTA a slice of it, kept in shared memory:
//   1. the largest and the smallest value (one exchange);
//   2. a histogram of mass and count over 1024 bins of equal width in x,
//      which keep the order; every CTA sums its share of the bins over the
//      cluster and hands it to all of them;
//   3. the prefix sums, which every CTA then has, give for each filter's edge
//      and for the draw the one or few bins that can hold it;
//   4. the tokens of those bins go to the first CTA, which sorts them and takes
//      every decision exactly: a bin's mass is a whole number, so the running
//      mass at a token is that of the bins in front plus that of the sorted
//      tokens in front.
// Where those bins hold too many tokens (equal values), the same searches are
// made digit by digit over (value, index), a histogram for each 10 bits.
//
// Bound by latency for few rows (about ten dependent steps, four of them
// barriers of the cluster): 1 row of 128000 float32 logits with every filter
// 13.2 us, 32 rows 21.2 us (two CTAs an SM, one wave); by the same steps in
// waves for many: 200 rows of 50257 bf16 logits 43.5 us.  The search by digits
// costs a histogram for each digit: one row of 128000 equal logits 216 us, 200
// rows of 50257 bf16 logits around 100 (some hundred values) 750 us.  All loops
// stay rolled: code that runs once a launch costs the time to fetch it (slices in
// registers, 32 values unrolled in each pass: 6 us a pass instead of 1.5).
#include <cooperative_groups.h>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace wobs {
namespace {

using u64 = unsigned long long;

constexpr int kThreads = 512;
// 2^10 bins: with 2^11 peaked rows cost 8 % more (the bins' own work), flat ones
// 17 % less (fewer tokens to sort): 1x128000 13.1 against 14.2 us, N(0, 1) alone 22.5 against 18.7
constexpr int kBins = 1024, kDigit = 10;
constexpr int kOwn = kBins / kThreads;   // consecutive bins of a thread
constexpr int kSlice = 16383;      // tokens whose parts (at most 2^18, 2^16) 32-bit sums hold
constexpr int kGather = 1536;      // tokens that the first CTA sorts
constexpr int kCount = kThreads;   // up to here by counting
constexpr int kRanges = 4;         // k, p and min-p edges, the draw
constexpr int kMaxCluster = 16;
constexpr float kOne = 34359738368.0f;   // 2^35

// Larger floats to smaller integers; NaN counts as -infinity, -0 as +0.
__device__ __forceinline__ uint32_t order_key(float v) {
  uint32_t b = __float_as_uint(v);
  if (b == 0x80000000u) b = 0u;
  return (b & 0x80000000u) ? b : 0x7FFFFFFFu - b;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k : 0x7FFFFFFFu - k);
}

struct Row {
  float best, bins;      // largest value; bins for each unit of x
  float c_hi, c_lo;      // log2(e) / temperature as a sum of two floats
  float alive;           // below this e < 2^-36, which rounds to no mass
};
struct alignas(8) Mass {
  uint32_t hi;           // multiples of 2^-18
  int lo;                // multiples of 2^-35, at most 2^16 either way
  __device__ __forceinline__ bool none() const { return (hi | static_cast<uint32_t>(lo)) == 0; }
  __device__ __forceinline__ u64 sum() const { return (static_cast<u64>(hi) << 17) + static_cast<u64>(static_cast<long long>(lo)); }
};

// exp((v - best) / T), 0 below alive: the argument of the power of two is rounded
// once.  Above alive it is finite, whatever the temperature (v - best is made so).
__device__ __forceinline__ float weight(const Row& r, float v) {
  const float d = fmaxf(v - r.best, -3.402823466e38f);
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fmaf(d, r.c_hi, d * r.c_lo)));
  return v == r.best ? 1.0f : v >= r.alive ? e : 0.0f;
}
// e in [0, 1]: adding 2^5 rounds it to a multiple of 2^-18, adding 1.5 * 2^-12
// the exact rest to one of 2^-35; both are read off the sums' bits.
__device__ __forceinline__ Mass mass_of(float e) {
  const float h = __fadd_rn(e, 32.0f);
  const float rest = __fsub_rn(e, __fsub_rn(h, 32.0f));
  const float l = __fadd_rn(rest, 1.5f * 0x1p-12f);
  return Mass{__float_as_uint(h) - __float_as_uint(32.0f),
              static_cast<int>(__float_as_uint(l)) - static_cast<int>(__float_as_uint(1.5f * 0x1p-12f))};
}
__device__ __forceinline__ int bin_of(const Row& r, float v) {
  return min(kBins - 1, static_cast<int>((r.best - v) * r.bins));   // v == best where that is infinite: NaN to 0
}
__device__ __forceinline__ u64 place(float v, int i) {
  return (static_cast<u64>(order_key(v)) << 32) | static_cast<unsigned>(i);
}

struct Histogram {
  Mass part[kBins];
  uint32_t cnt[kBins];
};
struct alignas(16) Shared {
  union {
    Histogram h;                   // this CTA's part sums
    struct {
      u64 key[kGather];            // first CTA, later: gathered tokens
      u64 sorted[kCount];
    };
  };
  alignas(16) u64 mass[kBins];     // the row's sums, then the mass up to each bin's end (read as 16-byte vectors)
  alignas(16) uint32_t count[kBins];
  u64 warp_mass[32];
  uint32_t warp_count[32];
  float most[kMaxCluster], least[kMaxCluster];
  u64 parts[kMaxCluster];
  int from[kRanges], to[kRanges];  // bins to gather
  uint32_t gathered;
  u64 prefix, below;               // of a search by digits
  u64 mass_k, mass_p, mass_m, part;
};
// with a slice of 16000 tokens two CTAs share an SM (32 rows of 128000: 44 us with one, 24 us with two)

template <typename T>
__device__ __forceinline__ float load_logit(const T* row, int i) {
  const float v = to_float(row[i]);
  return v == v ? v : -INFINITY;
}

// A CTA's slice of a row: tokens first .. first + n - 1, in shared memory.
struct Slice {
  const float* v;
  int first, n;
};
// Calls f(value, index) for the slice's tokens j0 .. j1 - 1.
template <typename F>
__device__ __forceinline__ void each(const Slice& sl, int j0, int j1, F f) {
#pragma unroll 2
  for (int j = j0 + threadIdx.x; j < j1; j += kThreads) f(sl.v[j], sl.first + j);
}

// Inclusive prefix sums over the bins, kOwn consecutive ones a thread, in place.
__device__ __forceinline__ void scan_bins(Shared& s, bool counts) {
  static_assert(kOwn % 2 == 0 && kBins == kOwn * kThreads, "");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  ulonglong2* mass = reinterpret_cast<ulonglong2*>(s.mass) + kOwn / 2 * tid;
  uint2* count = reinterpret_cast<uint2*>(s.count) + kOwn / 2 * tid;
  ulonglong2 m[kOwn / 2];
  uint2 c[kOwn / 2];
  u64 own = 0;
  uint32_t own_c = 0;
#pragma unroll
  for (int j = 0; j < kOwn / 2; ++j) {
    m[j] = mass[j];
    m[j].x += own;
    own = m[j].y += m[j].x;
  }
  u64 run = own;
  uint32_t run_c = 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 up = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += up;
  }
  if (counts) {
#pragma unroll
    for (int j = 0; j < kOwn / 2; ++j) {
      c[j] = count[j];
      c[j].x += own_c;
      own_c = c[j].y += c[j].x;
    }
    run_c = own_c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(0xffffffffu, run_c, o);
      if (lane >= o) run_c += up;
    }
  }
  if (lane == 31) { s.warp_mass[warp] = run; s.warp_count[warp] = run_c; }
  __syncthreads();
  // the warps in front: every lane adds the same few words
  u64 before = run - own;
  uint32_t before_c = run_c - own_c;
  for (int w = 0; w < warp; ++w) { before += s.warp_mass[w]; before_c += s.warp_count[w]; }
#pragma unroll
  for (int j = 0; j < kOwn / 2; ++j) {
    mass[j] = make_ulonglong2(m[j].x + before, m[j].y + before);
    if (counts) count[j] = make_uint2(c[j].x + before_c, c[j].y + before_c);
  }
  __syncthreads();
}

// Fills every CTA's mass and count with the row's sums of f over the bins, as
// prefix sums (the counts only where `counts` says so); f(value, index, mass)
// gives a bin or -1.
template <typename F>
__device__ void histogram(cg::cluster_group& cluster, Shared& s, const Slice& sl, int slice, bool counts, F f) {
  const int tid = threadIdx.x, n = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  for (int j0 = 0; j0 < slice; j0 += kSlice) {       // the same number of rounds in every CTA
    uint32_t* z = reinterpret_cast<uint32_t*>(&s.h);
    for (int k = tid; k < static_cast<int>(sizeof(Histogram) / 4); k += kThreads) z[k] = 0;
    __syncthreads();
    each(sl, j0, min(sl.n, j0 + kSlice), [&](float v, int i) {
      Mass m;
      const int k = f(v, i, m);
      if (k < 0) return;
      if (counts) atomicAdd(&s.h.cnt[k], 1u);
      if (m.hi) atomicAdd(&s.h.part[k].hi, m.hi);
      atomicAdd(&s.h.part[k].lo, m.lo);
    });
    cluster.sync();
    // This CTA's share of the bins: g lanes a bin read from every g-th CTA each,
    // and write the sum to every g-th.
    const int per = kBins / n, g = n >= 16 ? 4 : n >= 8 ? 2 : 1, bins = 32 / g;
    const int part = (tid & 31) / bins;
    for (int x = (tid >> 5) * bins + (tid & 31) % bins; x < per; x += kThreads / g) {
      const int k = rank * per + x;
      u64 m = j0 && part == 0 ? s.mass[k] : 0ull;
      uint32_t c = j0 && part == 0 ? s.count[k] : 0u;
#pragma unroll 4
      for (int q = part; q < n; q += g) {
        const Histogram* o = &cluster.map_shared_rank(&s, q)->h;
        m += o->part[k].sum();
        if (counts) c += o->cnt[k];
      }
      for (int o = bins; o < 32; o <<= 1) {
        m += __shfl_xor_sync(0xffffffffu, m, o);
        if (counts) c += __shfl_xor_sync(0xffffffffu, c, o);
      }
#pragma unroll 4
      for (int q = part; q < n; q += g) {
        Shared* o = cluster.map_shared_rank(&s, q);
        o->mass[k] = m;
        if (counts) o->count[k] = c;
      }
    }
    cluster.sync();
  }
  scan_bins(s, counts);
}

// The bins at which the running mass first reaches t0 and t1 (1 <= t <= the total).
__device__ __forceinline__ void find_bins(const Shared& s, u64 t0, u64 t1, int* out0, int* out1) {
  const int k0 = kOwn * threadIdx.x;
  u64 below = k0 ? s.mass[k0 - 1] : 0ull;
#pragma unroll
  for (int j = 0; j < kOwn; ++j) {
    const u64 up = s.mass[k0 + j];
    if (below < t0 && t0 <= up) *out0 = k0 + j;
    if (below < t1 && t1 <= up) *out1 = k0 + j;
    below = up;
  }
}

// A fraction of a mass, as a running mass to be reached (1 .. of): f * of
// rounded up, or the first whole number above it.  32 bits of f: exact from
// 2^-8 up.
__device__ __forceinline__ u64 share(float f, u64 of, bool up) {
  if (!(f < 1.f)) return of ? of : 1ull;
  const u64 f32 = static_cast<u64>(__float2uint_rz(fmaxf(f, 0.f) * 4294967296.0f)) << 32;
  const u64 whole = __umul64hi(of, f32);
  const u64 t = up ? whole + (of * f32 != 0ull) : whole + 1ull;
  return max(1ull, min(t, of));
}

// The keys s.key[0 .. n) in ascending order, at the returned place (up to kCount
// of them each thread counts what stands in front of its own: no barriers
// between steps; 512 keys cost about as much as a bitonic sort's 45).
__device__ __noinline__ const u64* sort_keys(Shared& s, int n) {
  if (n <= kCount) {
    if (static_cast<int>(threadIdx.x) < n) {
      const u64 own = s.key[threadIdx.x];
      int at = 0;
#pragma unroll 4
      for (int k = 0; k < n; ++k) at += s.key[k] < own;
      s.sorted[at] = own;
    }
    __syncthreads();
    return s.sorted;
  }
  int size = 2 * kCount;
  while (size < n) size <<= 1;
  // a bitonic network whose runs all ascend (each merge begins by mirroring its
  // second half): keys past n count as the largest and never move
  for (int k = 2; k <= size; k <<= 1) {
    for (int j = k >> 1; j > 0; j >>= 1) {
      const bool mirror = j == (k >> 1);
      for (int x = threadIdx.x; x < size / 2; x += kThreads) {
        const int lo = 2 * x - (x & (j - 1)), hi = mirror ? (lo ^ (k - 1)) : lo + j;
        if (hi >= n) continue;
        const u64 p = s.key[lo], q = s.key[hi];
        if (p > q) {
          s.key[lo] = q;
          s.key[hi] = p;
        }
      }
      __syncthreads();
    }
  }
  return s.key;
}

// The search by digits: the place of the first token in order, among those with
// place <= cut and e >= min_e, at which the running count or mass reaches t.
// Every CTA of the cluster gets it.
__device__ __noinline__ u64 search(cg::cluster_group& cluster, Shared& s, const Row& r, const Slice& sl, int slice, bool by_mass,
                      u64 t, u64 cut, float min_e) {
  u64 prefix = 0, below = 0;
  for (int shift = 64 - kDigit; shift > -kDigit; shift -= kDigit) {
    const int sh = shift < 0 ? 0 : shift, bits = shift < 0 ? kDigit + shift : kDigit;
    histogram(cluster, s, sl, slice, true, [&](float v, int i, Mass& m) -> int {
      const u64 c = place(v, i);
      if (c > cut || (sh + bits < 64 && (c >> (sh + bits)) != (prefix >> (sh + bits)))) return -1;
      const float e = weight(r, v);
      if (!(e >= min_e) || !(v > -INFINITY)) return -1;
      m = mass_of(e);
      return m.none() ? -1 : static_cast<int>((c >> sh) & ((1u << bits) - 1u));
    });
    for (int k = threadIdx.x; k < kBins; k += kThreads) {
      const u64 to = below + (by_mass ? s.mass[k] : s.count[k]);
      const u64 from = below + (k == 0 ? 0ull : by_mass ? s.mass[k - 1] : s.count[k - 1]);
      if (from < t && t <= to) {
        s.prefix = prefix | (static_cast<u64>(k) << sh);
        s.below = from;
      }
    }
    __syncthreads();
    prefix = s.prefix;
    below = s.below;
    __syncthreads();
  }
  return prefix;
}

// The mass of the row's tokens with place <= cut and e >= min_e.
__device__ __noinline__ u64 mass_within(cg::cluster_group& cluster, Shared& s, const Row& r, const Slice& sl, u64 cut, float min_e) {
  u64 m = 0;
  each(sl, 0, sl.n, [&](float v, int i) {
    if (place(v, i) > cut || !(v > -INFINITY)) return;
    const float e = weight(r, v);
    if (e >= min_e) m += mass_of(e).sum();
  });
  if (threadIdx.x == 0) s.part = 0;
  __syncthreads();
  atomicAdd(&s.part, m);
  __syncthreads();
  const int n = static_cast<int>(cluster.num_blocks());
  if (static_cast<int>(threadIdx.x) < n) cluster.map_shared_rank(&s, threadIdx.x)->parts[cluster.block_rank()] = s.part;
  cluster.sync();
  m = 0;
  for (int q = 0; q < n; ++q) m += s.parts[q];
  cluster.sync();
  return m;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(SampleArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  Shared& s = *reinterpret_cast<Shared*>(raw);
  float* values = reinterpret_cast<float*>(raw + sizeof(Shared));
  cg::cluster_group cluster = cg::this_cluster();
  const int n = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  cg::cluster_group::arrival_token started = cluster.barrier_arrive();   // no CTA writes to one that has not begun
  const int m = blockIdx.x / n;
  const T* row = static_cast<const T*>(a.logits) + m * a.ld;
  const int slice = (a.N + n - 1) / n;
  const int first = min(a.N, rank * slice);
  const Slice sl{values, first, min(a.N, first + slice) - first};
  pdl_launch_dependents();
  pdl_wait();
  float most = -INFINITY, least = INFINITY;
#pragma unroll 8
  for (int j = tid; j < sl.n; j += kThreads) {
    const float v = load_logit(row, first + j);
    values[j] = v;
    most = fmaxf(most, v);
    if (v > -INFINITY) least = fminf(least, v);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    least = fminf(least, __shfl_xor_sync(0xffffffffu, least, o));
  }
  float* wm = reinterpret_cast<float*>(s.warp_mass);
  if (lane == 0) { wm[warp] = most; wm[32 + warp] = least; }
  if (tid == 0) s.gathered = 0;
  if (tid < kRanges) { s.from[tid] = 1; s.to[tid] = 0; }      // empty
  __syncthreads();
  most = lane < kThreads / 32 ? wm[lane] : -INFINITY;
  least = lane < kThreads / 32 ? wm[32 + lane] : INFINITY;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    least = fminf(least, __shfl_xor_sync(0xffffffffu, least, o));
  }
  cluster.barrier_wait(std::move(started));
  if (tid < n) {
    Shared* o = cluster.map_shared_rank(&s, tid);
    o->most[rank] = most;
    o->least[rank] = least;
  }
  float temperature = a.temperature ? a.temperature[m] : 1.0f;
  const float given = a.min_p ? a.min_p[m] : 0.f;
  float min_e = given > 0.f ? fminf(given, 1.0f) : 0.f;        // NaN: off
  const float p = a.top_p ? a.top_p[m] : 1.0f;
  const int k = a.top_k ? a.top_k[m] : 0;
  const bool greedy = !(temperature > 0.f);
  if (greedy) temperature = min_e = 1.0f;    // the largest value's tokens alone, and of them the first
  const float u = greedy ? 0.f : a.u[m];
  cluster.sync();
  for (int q = 0; q < n; ++q) {
    most = fmaxf(most, s.most[q]);
    least = fminf(least, s.least[q]);
  }
  if (!(most > -INFINITY)) {           // nothing to draw from
    if (rank == 0 && tid == 0) {
      a.token[m] = -1;
      if (a.prob) a.prob[m] = 0.f;
    }
    return;                            // every CTA of the cluster alike
  }
  Row r;
  r.best = most;
  if (!(most < INFINITY)) temperature = 1.0f;   // only the infinities have a mass, at any temperature
  constexpr float kLog2e = 1.4426950408889634f, kLog2eRest = static_cast<float>(1.4426950408889634 - kLog2e);
  r.c_hi = kLog2e / temperature;
  // the exact remainder's share; at an infinite temperature (c_hi 0: all masses equal) and a tiny one there is none
  r.c_lo = r.c_hi > 0.f && r.c_hi < INFINITY ? (fmaf(-r.c_hi, temperature, kLog2e) + kLog2eRest) / temperature : 0.f;
  r.alive = r.best - 36.1f / r.c_hi;            // -infinity where every token has a mass
  // one width for all bins, over the values that have a mass: (best - x) / T up to 26, where e < 2^-36
  const float span = fminf(r.best - least, 26.f * temperature);
  r.bins = span > 0.f && span < INFINITY ? kBins / span : 0.f;
  if (!(r.bins < INFINITY)) r.bins = 0.f;

  // one comparison for what are most tokens of a peaked row
  histogram(cluster, s, sl, slice, k > 0, [&](float v, int, Mass& mass) -> int {
    if (!(v >= r.alive) || !(v > -INFINITY)) return -1;
    mass = mass_of(weight(r, v));
    return mass.none() ? -1 : bin_of(r, v);
  });

  // the bins that can hold an edge or the draw, found by every CTA alike
  const u64 total = s.mass[kBins - 1];
  const bool has_k = k > 0 && k < static_cast<int>(s.count[kBins - 1]), has_p = p < 1.0f, has_m = min_e > 0.f;
  auto up_to = [&](int b) { return b < 0 ? 0ull : s.mass[min(b, kBins - 1)]; };
  u64 low = total, high = total;       // bounds of the kept mass
  if (has_k) {
    for (int b = tid; b < kBins; b += kThreads)
      if (static_cast<int>(s.count[b]) >= k && (b == 0 || static_cast<int>(s.count[b - 1]) < k)) s.from[0] = s.to[0] = b;
    __syncthreads();
    low = up_to(s.from[0] - 1);
    high = up_to(s.to[0]);
  }
  if (has_p) {
    find_bins(s, share(p, low, true), share(p, high, true), &s.from[1], &s.to[1]);
    __syncthreads();
    low = min(low, up_to(s.from[1] - 1));
    high = min(high, up_to(s.to[1]));
  }
  if (has_m) {
    const int edge = static_cast<int>(fminf(-logf(min_e) * temperature * r.bins, static_cast<float>(kBins)));
    if (tid == 0) { s.from[2] = min(kBins - 1, max(0, edge - 1)); s.to[2] = min(kBins - 1, edge + 1); }   // the logarithm rounds
    low = min(low, up_to(edge - 2));
    high = min(high, up_to(edge + 1));
  }
  find_bins(s, share(u, low, false), share(u, high, false), &s.from[3], &s.to[3]);
  __syncthreads();
  int from[kRanges], to[kRanges];
  int furthest = 0;
#pragma unroll
  for (int q = 0; q < kRanges; ++q) {
    from[q] = s.from[q];
    to[q] = s.to[q];
    furthest = max(furthest, to[q]);
  }
  auto wanted = [&](int b) {
    bool w = false;
#pragma unroll
    for (int q = 0; q < kRanges; ++q) w |= b >= from[q] && b <= to[q];
    return w;
  };
  Shared* lead = cluster.map_shared_rank(&s, 0);
  // most tokens lie beyond the last bin wanted: a comparison, with a bin to spare for its rounding
  const float worth = r.bins > 0.f ? r.best - static_cast<float>(furthest + 2) / r.bins : -INFINITY;
  each(sl, 0, sl.n, [&](float v, int i) {
    if (!(v >= worth) || !(v > -INFINITY) || !wanted(bin_of(r, v)) || mass_of(weight(r, v)).none()) return;
    const uint32_t at = atomicAdd(&lead->gathered, 1u);
    if (at < kGather) lead->key[at] = place(v, i);
  });
  cluster.sync();
  const int many = static_cast<int>(lead->gathered);
  if (many <= kGather) {
    cg::cluster_group::arrival_token read = cluster.barrier_arrive();   // the count has been read
    if (rank != 0) return;
    const u64* sorted = sort_keys(s, many);
    const u64 in_front = from[2] <= to[2] && from[2] > 0 ? s.mass[from[2] - 1] : 0ull;
    // mass and count of the bins in front of bin b that were not gathered: bins
    // 0 .. b - 1 less the ranges' parts of them, each range cut to what those
    // before it (they are few, and may overlap) do not have
    auto not_gathered = [&](int b, u64& mass, int& count) {
      mass = b ? s.mass[b - 1] : 0ull;
      count = b && k > 0 ? static_cast<int>(s.count[b - 1]) : 0;
      int done = 0;                    // bins below are dealt with
#pragma unroll
      for (int x = 0; x < kRanges; ++x) {
        int f = kBins, t = -1;         // the range that begins first among those that reach past `done`
#pragma unroll
        for (int q = 0; q < kRanges; ++q)
          if (from[q] <= to[q] && to[q] >= done && max(from[q], done) < f) { f = max(from[q], done); t = to[q]; }
        t = min(t, b - 1);
        if (f > t) break;
        mass -= s.mass[t] - (f ? s.mass[f - 1] : 0ull);
        if (k > 0) count -= static_cast<int>(s.count[t]) - static_cast<int>(f ? s.count[f - 1] : 0u);
        done = t + 1;
      }
    };
    if (tid == 0) {
      s.mass_k = s.mass_p = s.mass_m = total;
      s.part = 0;
    }
    __syncthreads();
    // some sorted tokens a thread: running mass and count
    constexpr int kPer = kGather / kThreads;
    const int per = many <= kCount ? 1 : kPer;
    u64 upto[kPer], own[kPer];
    float e[kPer];
    u64 sum = 0;
    int bin[kPer];
#pragma unroll 1
    for (int j = 0; j < per; ++j) {
      const int i = tid * per + j;
      own[j] = 0;
      if (i < many) {
        const float v = key_value(static_cast<uint32_t>(sorted[i] >> 32));
        e[j] = weight(r, v);
        own[j] = mass_of(e[j]).sum();
        bin[j] = bin_of(r, v);
      }
      sum += own[j];
      upto[j] = sum;
    }
    u64 run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 other = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += other;
    }
    if (lane == 31) s.warp_mass[warp] = run;
    __syncthreads();
    u64 before = run - sum;
    for (int w = 0; w < warp; ++w) before += s.warp_mass[w];
    u64 part = 0;
#pragma unroll 1
    for (int j = 0; j < per; ++j) {
      const int i = tid * per + j;
      if (i >= many) break;
      u64 mass;
      int count;
      not_gathered(bin[j], mass, count);
      upto[j] += before + mass;
      if (from[0] <= to[0] && count + i + 1 == k) s.mass_k = upto[j];
      if (bin[j] >= from[2] && bin[j] <= to[2] && e[j] >= min_e) part += own[j];
    }
    if (from[2] <= to[2] && part) atomicAdd(&s.part, part);
    __syncthreads();
    if (from[1] <= to[1]) {
      const u64 t = share(p, s.mass_k, true);
#pragma unroll 1
      for (int j = 0; j < per; ++j)
        if (tid * per + j < many && upto[j] >= t && upto[j] - own[j] < t) s.mass_p = upto[j];
    }
    if (from[2] <= to[2] && tid == 0) s.mass_m = in_front + s.part;
    __syncthreads();
    const u64 z = min(s.mass_k, min(s.mass_p, s.mass_m));
    const u64 t = share(u, z, false);
#pragma unroll 1
    for (int j = 0; j < per; ++j) {
      const int i = tid * per + j;
      if (i < many && upto[j] >= t && upto[j] - own[j] < t) {
        a.token[m] = static_cast<int64_t>(sorted[i] & 0xFFFFFFFFull);
        if (a.prob) a.prob[m] = greedy ? 1.f : e[j] * kOne / __ull2float_rn(z);
      }
    }
    cluster.barrier_wait(std::move(read));
    return;
  }

  // too many tokens in the bins: search by digits
  cluster.sync();                      // the count has been read, and the histograms may be written again
  u64 cut = ~0ull;
  if (from[0] <= to[0]) cut = search(cluster, s, r, sl, slice, false, k, cut, 0.f);
  if (from[1] <= to[1]) {
    const u64 z = mass_within(cluster, s, r, sl, cut, 0.f);
    cut = search(cluster, s, r, sl, slice, true, share(p, z, true), cut, 0.f);
  }
  const u64 z = mass_within(cluster, s, r, sl, cut, min_e);
  const u64 at = search(cluster, s, r, sl, slice, true, share(u, z, false), cut, min_e);
  if (rank == 0 && tid == 0) {
    a.token[m] = static_cast<int64_t>(at & 0xFFFFFFFFull);
    if (a.prob) a.prob[m] = greedy ? 1.f : weight(r, key_value(static_cast<uint32_t>(at >> 32))) * kOne / __ull2float_rn(z);
  }
  cluster.sync();                      // no CTA ends while another reads its histogram
}

template <typename T>
cudaError_t launch_t(const SampleArgs& a, int cluster, int smem, cudaStream_t st) {
  auto kernel = sample_kernel<T>;
  static std::atomic<uint64_t> ready{0};                // devices whose kernel may be launched with any of the sizes
  cudaError_t e = once_on_device(ready, [&] {
    constexpr int most = static_cast<int>(sizeof(Shared)) + kSampleMaxN / kMaxCluster * 4;
    static_assert(most <= 227 * 1024, "");
    const cudaError_t first = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    return first != cudaSuccess ? first : cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.M) * cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kernel, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, cudaStream_t st, Launch* info) {
  // Slices of at most kSlice tokens (one histogram round) where the cluster
  // allows it; below that, more CTAs a row while half the GPU would stay empty.
  int cluster = 1;
  while (cluster < kMaxCluster && ((a.N + cluster - 1) / cluster > kSlice ||
                                   (static_cast<int64_t>(a.M) * cluster * 2 <= device_sm_count() && a.N > 2048 * cluster)))
    cluster <<= 1;
  const int smem = static_cast<int>(sizeof(Shared)) + ((a.N + cluster - 1) / cluster + 3) / 4 * 16;
  info->kernel = "sample";
  info->grid_x = a.M * cluster;
  info->block = kThreads;
  info->smem = smem;
  return a.dtype == 1 ? launch_t<__half>(a, cluster, smem, st) : a.dtype == 2 ? launch_t<__nv_bfloat16>(a, cluster, smem, st) : launch_t<float>(a, cluster, smem, st);
}

}  // namespace wobs
