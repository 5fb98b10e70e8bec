// Writing a paged 4-bit key/value cache, and reading its newest tokens back.
//
// Format and decisions are Q4_0's (IEEE float32): per 32 elements of a
// token's head, d = amax / -8 with amax the signed element of the largest
// magnitude (the first on ties), q = clamp(roundf(x / d) + 8, 0, 15), 8 where
// d is 0.  The newest L tokens of sequence b stand at lens[b] - L ..
// lens[b] - 1; positions below 0 (a prompt shorter than L, padded in front)
// and past the sequence's table are left out.
#include "kv4.cuh"

namespace wobs {
namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ void load8_any(const T* p, bool vec, float (&v)[8]) {
  if (vec) {
    if constexpr (sizeof(T) == 2) {
      const uint4 a = *reinterpret_cast<const uint4*>(p);
      const T* tag = nullptr;
      const float2 f0 = to_float2(a.x, tag), f1 = to_float2(a.y, tag), f2 = to_float2(a.z, tag),
                   f3 = to_float2(a.w, tag);
      v[0] = f0.x; v[1] = f0.y; v[2] = f1.x; v[3] = f1.y;
      v[4] = f2.x; v[5] = f2.y; v[6] = f3.x; v[7] = f3.y;
    } else {
      const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_float(p[i]);
  }
}

// Where a thread's elements are: a sequence is a row of the grid, its lanes
// run over [token][head][block][LANES lanes a block].
struct Place {
  int tok, head, blk, j;
  bool in;
};
template <int LANES>
__device__ __forceinline__ Place place_of(const Kv4Args& c, int L) {
  const unsigned per_head = static_cast<unsigned>(c.dim >> 5) * LANES, per_tok = per_head * c.heads;
  const unsigned i = blockIdx.x * kThreads + threadIdx.x;
  const unsigned tok = quotient(i, per_tok), rest = i - tok * per_tok;
  Place p;
  p.tok = static_cast<int>(tok);
  p.in = tok < static_cast<unsigned>(L);
  p.head = static_cast<int>(rest >> (31 - __clz(per_head)));      // dim is a power of two
  const unsigned e = rest & (per_head - 1);
  p.blk = static_cast<int>(e / LANES);
  p.j = static_cast<int>(e % LANES);
  return p;
}

// The code of x in a block of scale d, clamp(roundf(x / d) + 8, 0, 15) with the
// IEEE float32 quotient, in the low byte of the result.
__device__ __forceinline__ uint32_t code_by_division(float x, float d) {
  return static_cast<uint32_t>(min(15, max(0, static_cast<int>(roundf(x / d)) + 8)));
}
// The same by r = 1 / d: adding 1.5 * 2^23 rounds x * r to an integer, the
// nearest one to x / d unless that lies next to half an integer.
//   16-bit x: x and d have significands of 11 bits at most, so x / d is half an
// integer or at least 2^-15 of itself away from one (over all pairs of
// significands).  With r larger by 2^-21, more than its error, halves go away
// from zero and nothing else changes.
//   float32 x: x * r and the rounded quotient are within 2e-6 of x / d (|x / d|
// <= 8), so the codes are right where x * r is further than kNearHalf from a
// half; else the block's lane divides (1 % of the warps, random x).
constexpr float kRound = 12582912.0f, kNearHalf = 1e-5f;
__device__ __forceinline__ uint32_t code_by_reciprocal(float x, float r) {
  return min(__float_as_uint(fmaf(x, r, kRound + 8.0f)), 0x4B40000Fu);
}
__device__ __forceinline__ bool near_half(float x, float r) {
  return fabsf(fmaf(x, r, -(fmaf(x, r, kRound) - kRound))) > 0.5f - kNearHalf;
}
__device__ __forceinline__ float reciprocal(float x) {    // error 2^-23
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// the low bytes of four words
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}
// NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The element of largest magnitude of a block on four lanes (lane j holds
// elements 8j ..), the first one of several; NaN where the block holds one.  It
// is the largest or the smallest element; only where these are of one magnitude
// the first has to be looked for.
__device__ __forceinline__ float largest_of_block(const float (&x)[8], int j) {
  float high = x[0], low = x[0];
#pragma unroll
  for (int e = 1; e < 8; ++e) {
    high = max_nan(high, x[e]);
    low = min_nan(low, x[e]);
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    high = max_nan(high, __shfl_xor_sync(0xffffffffu, high, o));
    low = min_nan(low, __shfl_xor_sync(0xffffffffu, low, o));
  }
  const bool tie = high == -low;
  float amax = high > -low ? high : low;
  if (__any_sync(0xffffffffu, tie)) {
    float first = x[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) first = fabsf(x[e]) > fabsf(first) ? x[e] : first;
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {   // the lower lane's on ties: its elements come first
      const float other = __shfl_xor_sync(0xffffffffu, first, o);
      const bool take = (j & o) ? fabsf(other) >= fabsf(first) : fabsf(other) > fabsf(first);
      first = take ? other : first;
    }
    if (tie) amax = first;
  }
  return amax;
}

// Four lanes a block, eight elements a lane, the keys and the values of the
// same place.  Four prompts of 1500 tokens (8 heads of 128, fp16; 24.6 MB in,
// 6.9 out): 10.2 us, 3.1 TB/s; float32 13.4 us for 56 MB; bound by issue (the
// codes' arithmetic and the places), 18.6 us with a division a code and by every
// index.  The next kernel starts behind it, as behind the read-back: what they
// write may be a product's weights.
template <typename T>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(Kv4Args c, Kv4Source<T> ks, Kv4Source<T> vs, int L) {
  const Place p = place_of<4>(c, L);
  const int b = blockIdx.y, nb = c.dim >> 5;
  pdl_wait();
  const Kv4Length len = kv4_length(c, b);
  const int at = len.given - L + p.tok;
  const Kv4Token token = kv4_token(c, max(at, 0));
  const int page = p.in && at >= 0 && at < len.held ? kv4_page(c, b, token) : -1;
  const bool in = page >= 0;
  float x[2][8];
#pragma unroll
  for (int e = 0; e < 8; ++e) x[0][e] = x[1][e] = 0.f;
  if (in) {
    load8_any(ks.p + b * ks.sb + p.tok * ks.st + p.head * ks.sh + 32 * p.blk + 8 * p.j, ks.vec, x[0]);
    load8_any(vs.p + b * vs.sb + p.tok * vs.st + p.head * vs.sh + 32 * p.blk + 8 * p.j, vs.vec, x[1]);
  }
  const int64_t row = in ? kv4_row(c, page, p.head, token) : 0;
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    const float d = largest_of_block(x[y], p.j) / -8.0f, ad = fabsf(d);
    uint32_t q[8];
    bool divide = !(ad >= 0x1p-100f && ad <= 0x1p100f);
    if (!divide) {
      const float r = sizeof(T) == 2 ? reciprocal(d) * (1.0f + 0x1p-21f) : reciprocal(d);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        q[e] = code_by_reciprocal(x[y][e], r);
        if (sizeof(T) == 4) divide |= near_half(x[y][e], r);
      }
    }
    if (divide) {
#pragma unroll
      for (int e = 0; e < 8; ++e) q[e] = d != 0.0f ? code_by_division(x[y][e], d) : 8u;
    }
    const uint32_t w0 = low_bytes(q[0], q[1], q[2], q[3]), w1 = low_bytes(q[4], q[5], q[6], q[7]);
    // lanes 0 and 1 store elements 0 .. 15 in the low nibbles, those of lanes 2 and 3 in the high ones
    const uint32_t h0 = __shfl_xor_sync(0xffffffffu, w0, 2), h1 = __shfl_xor_sync(0xffffffffu, w1, 2);
    if (in && p.j < 2)
      *reinterpret_cast<uint2*>((y ? c.vq : c.kq) + row * (c.dim >> 1) + 16 * p.blk + 8 * p.j) =
          make_uint2(w0 | (h0 << 4), w1 | (h1 << 4));
    if (in && p.j == 0) (y ? c.vd : c.kd)[row * nb + p.blk] = __float2half_rn(d);
  }
}

// Eight lanes a block, four elements a lane (a warp stores whole lines): (q - 8)
// * d as a float32 product, rounded once to T.  The same tokens as float32 (6.9
// MB in, 49 out): 12.4 us, 4.5 TB/s, where the output comes to DRAM; bound by its
// stores and issue (four lanes a block and two 16-byte stores a lane: 2 us more).
template <typename T>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(Kv4Args c, int L, T* __restrict__ ko, T* __restrict__ vo) {
  const Place p = place_of<8>(c, L);
  const int b = blockIdx.y, nb = c.dim >> 5;
  pdl_wait();
  if (!p.in) return;
  const Kv4Length len = kv4_length(c, b);
  const int at = len.given - L + p.tok;
  const Kv4Token token = kv4_token(c, max(at, 0));
  const int page = at >= 0 && at < len.held ? kv4_page(c, b, token) : -1;
  uint32_t w[2] = {0x88888888u, 0x88888888u};
  float d[2] = {0.f, 0.f};
  if (page >= 0) {
    const int64_t row = kv4_row(c, page, p.head, token);
    const int64_t code = row * (c.dim >> 1) + 16 * p.blk + 4 * (p.j & 3);
    w[0] = *reinterpret_cast<const uint32_t*>(c.kq + code);
    w[1] = *reinterpret_cast<const uint32_t*>(c.vq + code);
    d[0] = __half2float(c.kd[row * nb + p.blk]);
    d[1] = __half2float(c.vd[row * nb + p.blk]);
  }
  const int64_t to = ((static_cast<int64_t>(b) * L + p.tok) * c.heads + p.head) * c.dim + 32 * p.blk + 4 * p.j;
  const int sh = (p.j >> 2) * 4;                // the last four lanes' elements are the high nibbles
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    alignas(16) T o[4];
    const uint32_t n = (w[y] >> sh) & 0x0F0F0F0Fu;      // a code behind the exponent of 2^23: 2^23 + code
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = from_float<T>(d[y] * (__uint_as_float(__byte_perm(n, 0x4B000000u, 0x7440 + e)) - 8388616.0f));
    if constexpr (sizeof(T) == 4) *reinterpret_cast<uint4*>((y ? vo : ko) + to) = *reinterpret_cast<const uint4*>(o);
    else *reinterpret_cast<uint2*>((y ? vo : ko) + to) = *reinterpret_cast<const uint2*>(o);
  }
}

template <typename T>
cudaError_t append_t(const Kv4Args& c, const Kv4Strided& k, const Kv4Strided& v, int L, dim3 grid,
                     cudaStream_t st) {
  auto as = [](const Kv4Strided& s) {
    const int64_t per = 16 / sizeof(T);
    const bool vec = (reinterpret_cast<uintptr_t>(s.p) & 15u) == 0 && s.sb % per == 0 && s.st % per == 0 && s.sh % per == 0;
    return Kv4Source<T>{static_cast<const T*>(s.p), s.sb, s.st, s.sh, vec};
  };
  return launch_k(kv4_append_kernel<T>, grid, dim3(kThreads), 0, st, true, c, as(k), as(v), L);
}

dim3 token_grid(const Kv4Args& c, int B, int L, int lanes_per_block) {
  const int64_t lanes = static_cast<int64_t>(L) * c.heads * (c.dim >> 5) * lanes_per_block;
  return dim3(static_cast<unsigned>((lanes + kThreads - 1) / kThreads), B);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4Args& c, int dtype, const Kv4Strided& k, const Kv4Strided& v, int B, int L,
                              cudaStream_t st, Launch* info) {
  const dim3 grid = token_grid(c, B, L, 4);
  info->kernel = "kv4_append";
  info->grid_x = grid.x;
  info->grid_y = B;
  info->block = kThreads;
  if (dtype == 1) return append_t<__half>(c, k, v, L, grid, st);
  if (dtype == 2) return append_t<__nv_bfloat16>(c, k, v, L, grid, st);
  return append_t<float>(c, k, v, L, grid, st);
}

cudaError_t launch_kv4_read(const Kv4Args& c, int dtype, void* k, void* v, int B, int L, cudaStream_t st,
                            Launch* info) {
  const dim3 grid = token_grid(c, B, L, 8), block(kThreads);
  info->kernel = "kv4_read";
  info->grid_x = grid.x;
  info->grid_y = B;
  info->block = kThreads;
  if (dtype == 1)
    return launch_k(kv4_read_kernel<__half>, grid, block, 0, st, true, c, L, static_cast<__half*>(k), static_cast<__half*>(v));
  if (dtype == 2)
    return launch_k(kv4_read_kernel<__nv_bfloat16>, grid, block, 0, st, true, c, L, static_cast<__nv_bfloat16*>(k),
                    static_cast<__nv_bfloat16*>(v));
  return launch_k(kv4_read_kernel<float>, grid, block, 0, st, true, c, L, static_cast<float*>(k), static_cast<float*>(v));
}

}  // namespace wobs
