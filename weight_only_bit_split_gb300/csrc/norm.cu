// The residual's addition, the root-mean-square norm and the Q8_1 blocks that
// the low-bit products take, in one kernel:
//
//   h = round_R(x + residual)          (stored in the residual's type R)
//   r = 1 / sqrt(sum_k h^2 / K + eps)
//   y = (h * r) * w                    (float32, optionally stored)
//   per 32 elements: Q8_1 of y, with the quantiser's IEEE float32 decisions
//
// The norm is taken of the rounded h, so that the stored residual alone
// determines the output.  Sum, r and y are float32.
//
// And the inverse of the Q8_1 format: the values that the blocks stand for.
#include "common.cuh"

namespace wobs {
namespace {

// Rounds eight values to T in place and stores them (16-byte stores).
template <typename T>
__device__ __forceinline__ void store8(T* p, float (&v)[8]) {
  T o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    o[i] = from_float<T>(v[i]);
    v[i] = to_float(o[i]);
  }
  *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(o);
}
template <>
__device__ __forceinline__ void store8<float>(float* p, float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

__device__ __forceinline__ void store8_any(int dtype, void* p, int64_t at, float (&v)[8]) {
  if (dtype == 1) store8(static_cast<__half*>(p) + at, v);
  else if (dtype == 2) store8(static_cast<__nv_bfloat16*>(p) + at, v);
  else store8(static_cast<float*>(p) + at, v);
}

// Eight elements as they are in memory: one 16-byte load, two for float32.
template <typename T>
struct Raw8 {
  uint4 v[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw8<T> load_raw(const void* p, int64_t at) {
  const uint4* q = reinterpret_cast<const uint4*>(static_cast<const T*>(p) + at);
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) r.v[i] = q[i];
  return r;
}
template <typename T>
__device__ __forceinline__ void widen(const Raw8<T>& r, float (&v)[8]) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<uint4*>(v) = r.v[0];
    *reinterpret_cast<uint4*>(v + 4) = r.v[1];
  } else {
    const uint32_t a[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = to_float2(a[i], static_cast<const T*>(nullptr));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}
__device__ __forceinline__ void load8_any(int dtype, const void* p, int64_t at, float (&v)[8]) {
  if (dtype == 3) widen(load_raw<float>(p, at), v);
  else if (dtype == 2) widen(load_raw<__nv_bfloat16>(p, at), v);
  else widen(load_raw<__half>(p, at), v);
}

constexpr int most_threads(int C) { return C == 2 || C == 4 ? 512 : 1024; }

// One CTA a row; a thread holds C pieces of eight consecutive elements (four
// lanes to a Q8_1 block), so the row is read once.  All loads of a row are
// issued before the first is used.  TX, TR: types of x and of the residual.
// Bound by DRAM latency between a row's phases: 2000 rows of 8192, bf16, 117 MB:
// 23.8 us (4.9 TB/s); with four pieces a thread 24.6, of which 23.0 remain
// without the quantiser and its stores.  Rows past 16384 take eight pieces a
// thread, whose 64 registers spill: 250 rows of 65536, 51.7 us for the same 117
// MB, against 36.3 for 1000 rows of 16384.
// FULL: the threads' pieces are the row exactly.
template <int C, bool FULL, typename TX, typename TR>
__global__ void __launch_bounds__(most_threads(C), C == 2 ? 3 : 1) rmsnorm_q8_1_kernel(RmsNormArgs a) {
  __shared__ float part[32];
  const int pieces = a.K >> 3;
  const int64_t m = blockIdx.x;
  const TX* px = static_cast<const TX*>(a.x) + m * a.ldx;
  const TR* pr = static_cast<const TR*>(a.residual) + m * a.ldr;
  TR* ph = static_cast<TR*>(a.h) + m * a.ldh;
  uint8_t* pq = a.xq + m * (a.K >> 5) * 36;
  auto piece = [&](int c) { return c * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x); };
  auto in = [&](int c) { return FULL || piece(c) < pieces; };   // all four lanes of a block agree: K is a multiple of 32
  float h[C][8];
  float sum = 0.f;
  pdl_launch_dependents();
  pdl_wait();
  Raw8<TX> x[C];
  Raw8<TR> res[C];
  const bool add = a.residual != nullptr;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (!FULL) {
      x[c] = Raw8<TX>{};
      res[c] = Raw8<TR>{};
    }
    if (in(c)) {
      x[c] = load_raw<TX>(px, 8 * piece(c));
      if (add) res[c] = load_raw<TR>(pr, 8 * piece(c));
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c) widen(x[c], h[c]);
  if (add) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float r[8];
      widen(res[c], r);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[c][i] += r[i];
      if (in(c)) store8(ph + 8 * piece(c), h[c]);
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fmaf(h[c][i], h[c][i], sum);
  sum = warp_sum(sum);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
  // the weight arrives during the barrier where a thread has one piece; with
  // more it costs the registers of another CTA, and the caches have it
  float w[8];
  if (C == 1 && in(0)) load8_any(a.w_dtype, a.w, 8 * piece(0), w);
  __syncthreads();
  sum = warp_sum((threadIdx.x & 31) < (blockDim.x >> 5) ? part[threadIdx.x & 31] : 0.f);
  const float r = 1.0f / sqrtf(sum / static_cast<float>(a.K) + a.eps);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (C > 1 && in(c)) load8_any(a.w_dtype, a.w, 8 * piece(c), w);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = in(c) ? __fmul_rn(__fmul_rn(h[c][i], r), w[i]) : 0.f;
    if (a.xq) {
      const float4 v[2] = {make_float4(y[0], y[1], y[2], y[3]), make_float4(y[4], y[5], y[6], y[7])};
      const Q81Part<4> q = q8_1_part_block<4>(v);
      if (in(c)) store_q8_1_part<4>(pq + (piece(c) >> 2) * 36, q, threadIdx.x & 3);
    }
    if (a.y && in(c)) store8_any(a.y_dtype, a.y, m * a.ldy + 8 * piece(c), y);
  }
}

// Eight values a thread: q * d as a float32 product, rounded once to the
// output's type.  2000 rows of 8192 to fp16 (18 MB in, 33 out): 9.0 us, 5.7 TB/s.
// The next kernel starts behind it: what it writes may be a product's weights.
__global__ void __launch_bounds__(256) q8_1_dequant_kernel(const uint8_t* __restrict__ xq, int64_t pieces,
                                                           int dtype, void* __restrict__ out) {
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  pdl_wait();
  if (t >= pieces) return;
  const uint8_t* blk = xq + (t >> 2) * 36;
  const float d = __half2float(*reinterpret_cast<const __half*>(blk));
  const uint32_t* w = reinterpret_cast<const uint32_t*>(blk + 4) + 2 * (t & 3);
  const uint32_t c[2] = {w[0], w[1]};
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    v[i] = d * static_cast<float>(static_cast<int8_t>(c[i >> 2] >> (8 * (i & 3))));
  store8_any(dtype, out, 8 * t, v);
}

}  // namespace

namespace {
template <int C, typename TX>
cudaError_t launch_norm(const RmsNormArgs& a, int M, int block, cudaStream_t st) {
  const bool full = a.K == 8 * C * block;
  auto k = a.r_dtype == 1 ? (full ? rmsnorm_q8_1_kernel<C, true, TX, __half> : rmsnorm_q8_1_kernel<C, false, TX, __half>)
         : a.r_dtype == 2 ? (full ? rmsnorm_q8_1_kernel<C, true, TX, __nv_bfloat16> : rmsnorm_q8_1_kernel<C, false, TX, __nv_bfloat16>)
                          : (full ? rmsnorm_q8_1_kernel<C, true, TX, float> : rmsnorm_q8_1_kernel<C, false, TX, float>);
  return launch_k(k, dim3(M), dim3(block), 0, st, true, a);
}
template <int C>
cudaError_t launch_norm(const RmsNormArgs& a, int M, int block, cudaStream_t st) {
  return a.x_dtype == 1 ? launch_norm<C, __half>(a, M, block, st)
       : a.x_dtype == 2 ? launch_norm<C, __nv_bfloat16>(a, M, block, st) : launch_norm<C, float>(a, M, block, st);
}
}  // namespace

cudaError_t launch_rmsnorm_q8_1(const RmsNormArgs& a, int M, cudaStream_t st, Launch* info) {
  const int pieces = a.K >> 3;
  // Few rows: as many threads as a row has pieces, for the shortest chain.
  // Rows enough to fill the GPU: two pieces a thread, so that three CTAs of 512
  // threads share an SM and some load while others compute (2000 rows of 8192,
  // bf16: 28.3 us with one piece and 1024 threads, 23.8 with two, 24.6 with
  // four and 256 threads; float32 36.2 with two, 41.5 with four).
  const bool many = M >= device_sm_count();
  const int C = pieces <= (many ? 256 : 1024) ? 1 : pieces <= 1024 ? 2 : pieces <= 2048 ? 4 : 8;
  const int block = ((pieces + C - 1) / C + 31) / 32 * 32;
  info->kernel = "rmsnorm_q8_1";
  info->grid_x = M;
  info->block = block;
  return C == 1 ? launch_norm<1>(a, M, block, st) : C == 2 ? launch_norm<2>(a, M, block, st)
       : C == 4 ? launch_norm<4>(a, M, block, st) : launch_norm<8>(a, M, block, st);
}

cudaError_t launch_dequantize_q8_1(const void* xq, int64_t blocks, int dtype, void* out, cudaStream_t st,
                                   Launch* info) {
  const int64_t pieces = 4 * blocks;
  const int grid = static_cast<int>((pieces + 255) / 256);
  info->kernel = "q8_1_dequant";
  info->grid_x = grid;
  info->block = 256;
  return launch_k(q8_1_dequant_kernel, dim3(grid), dim3(256), 0, st, true,
                  static_cast<const uint8_t*>(xq), pieces, dtype, out);
}

}  // namespace wobs
