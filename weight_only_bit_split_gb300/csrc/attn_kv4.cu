// Attention of the newest tokens over a paged 4-bit key/value cache.
//
//   s[j] = scale * sum_b dk[j][b] * sum_{e in b} q[e] (ck[j][e] - 8)
//   p[j] = exp(s[j] - m),  o[e] = sum_j p[j] dv[j][b(e)] (cv[j][e] - 8) / sum_j p[j]
//
// over the tokens j <= lens[b] - L + i of query i; a query without any gives
// zeros.  One pass over the cache with a running maximum m and sum.
//
// Layout.  The queries that share a cache head (L tokens x group heads) are
// the rows of the problem; eight of them fill the narrow side (n) of an
// mma.sync m16n8k16 and the cache's tokens (for the scores) or dims (for the
// output) the wide one, so a group of four or eight query heads wastes half
// of a tile or nothing, and the decoded cache is the A operand of both
// products:
//   S^T[16 tokens][8 rows] += K[16 tokens][16 dims] Q^T[16 dims][8 rows]
//   O^T[16 dims][8 rows]   += V^T[16 dims][16 tokens] P^T[16 tokens][8 rows]
// A Q4_0 block is 16 bytes, one row of an 8x8 b16 matrix, so ldmatrix hands
// lane (g, t) word t of token g's block: eight codes of one token for the
// scores; transposed it hands b16 column g of tokens 2t and 2t + 1: the pair
// of tokens that an A register of V^T holds, for four dims.
//
// Decoding is one mask a register: a code in bits 0..3 or 4..7 of an fp16 is
// the subnormal c * 2^-24 or c * 2^-20, which the matrix unit multiplies
// exactly.  The two scales and the offset 8 leave elsewhere: queries that meet
// the high codes carry a factor 2^-4, rows of O that come from them end with
// 2^20 instead of 2^24; -8 * sum_b dk sum q is a small product of its own, of
// the scales with the blocks' sums of queries (as fp16 pairs high + low).  For
// V the accumulator must not hold a sum eight times larger that cancels at the
// end: with one tile of rows a second product with the constant -8 in A
// follows each one (the matrix unit has time, the issue slots have not), with
// several tiles the codes, decoded once for all of them, become c - 8 first.
//
// Numbers.  A row of queries (fp16 or bf16) is multiplied by the power of two
// that brings its largest element to [2^14, 2^15) and held in fp16; those that
// meet the high codes carry 2^-4 more, so an fp16 element is exact down to
// 2^-24 of the largest, a bf16 one down to 2^-27, and a smaller one is off by
// 2^-35 of the largest at most: what a float32 sum with the largest loses is
// 2^-24.  The offset's low half is an fp16 subnormal, its step 2^-24 of units in
// which the largest query's part is 2^-7 or more: 2^-18 of that part is lost at
// most.  With one query of a row 30 times the others' and key scales around 10
// the outputs' error stays P's (1.6e-5 of sum p |v|); at 1000 times it is 2.5e-4, of
// which an offset held to 2^-22 (1 us of the 117 below) would take a quarter: the
// rest is the float32 sums of codes eight above their values.  A block's scale
// multiplies its float32 sum.  A value's scale varies along the summed axis, so
// it goes into the other operand: p * dv is a float32 product, rounded once to
// fp16.  So that this neither overflows nor loses a token beside one that leads by far,
// what a row's exponentials are relative to is not its largest score but the
// largest s + e - 15 so far, 2^e the least power of two above a token's value
// scales: the largest product lies in [2^14, 2^15), that token's products are
// exact (its p is a power of two), others down to 2^-28 of the largest are
// rounded by half an ulp (2^-11), smaller ones by 2^-39 of it.  Scores are
// rounded before anything is subtracted, the addition of e - 15 (made to lie in
// -40 .. 0) rounds upwards: so also where scores are so large that the addition
// is lost, no product exceeds 2^15 (or a scale beyond that) and the leading
// token's exponential is at least 1.  Maxima, sums and accumulators are float32.
//
// Work.  A CTA step is 128 tokens of one (sequence, cache head, row tile):
// four warps of 32 tokens, each with its own cp.async ring and its own running
// maximum, no CTA barrier inside.  All segments of the call (a sequence's
// steps for one head and row tile) are laid end to end, each with kSegmentCost
// units in front for what it costs beside its steps, and cut into equal
// ranges, one for each resident CTA, so ragged lengths fill the GPU evenly; a
// range's pieces of a segment that others share go to the workspace, and the
// segment's last arrival adds them in range order (fixed sums, whatever the
// arrival order).
#include <cstddef>
#include <type_traits>

#include "kv4.cuh"

namespace wobs {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kWarpTokens = 32;
constexpr int kStepTokens = kWarps * kWarpTokens;
constexpr int kStages = 2;   // of a warp's ring

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <bool TRANS>
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  if constexpr (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// d += a * b, A 16x16 row-major, B 16x8, fp16 operands
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// The four codes of each 16-bit half of w as pairs of fp16 subnormals:
// c * 2^-24 (o[0], o[2]) and c * 2^-20 (o[1], o[3]).
__device__ __forceinline__ void decode(uint32_t w, uint32_t (&o)[4]) {
  o[0] = w & 0x000F000Fu;
  o[1] = w & 0x00F000F0u;
  o[2] = (w >> 8) & 0x000F000Fu;
  o[3] = (w >> 8) & 0x00F000F0u;
}
// The same as c - 8, all of one scale: 1024 + c less 1032, (1024 + 16 c) / 16 less 72, exact in fp16.
__device__ __forceinline__ void decode_signed(uint32_t w, uint32_t (&o)[4]) {
  const __half2 low = __halves2half2(__ushort_as_half(0x6408), __ushort_as_half(0x6408));         // 1032
  const __half2 sixteenth = __halves2half2(__ushort_as_half(0x2C00), __ushort_as_half(0x2C00));
  const __half2 high = __halves2half2(__ushort_as_half(0xD480), __ushort_as_half(0xD480));        // -72
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t x = w >> (8 * i);
    const uint32_t a = (x & 0x000F000Fu) | 0x64006400u, b = (x & 0x00F000F0u) | 0x64006400u;
    const __half2 l = __hsub2(*reinterpret_cast<const __half2*>(&a), low);
    const __half2 h = __hfma2(*reinterpret_cast<const __half2*>(&b), sixteenth, high);
    o[2 * i] = *reinterpret_cast<const uint32_t*>(&l);
    o[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&h);
  }
}
constexpr uint32_t kMinus8Low = 0x80088008u;    // -8 * 2^-24, twice
constexpr uint32_t kMinus8High = 0x80808080u;   // -8 * 2^-20, twice

// DB fp16 scales of one token as float32.
template <int DB>
__device__ __forceinline__ void load_scales(const __half* p, float (&d)[DB]) {
  __half2 h[DB / 2];
  if constexpr (DB == 2) *reinterpret_cast<uint32_t*>(h) = *reinterpret_cast<const uint32_t*>(p);
  else if constexpr (DB == 4) *reinterpret_cast<uint2*>(h) = *reinterpret_cast<const uint2*>(p);
  else *reinterpret_cast<uint4*>(h) = *reinterpret_cast<const uint4*>(p);
#pragma unroll
  for (int i = 0; i < DB / 2; ++i) {
    const float2 f = __half22float2(h[i]);
    d[2 * i] = f.x;
    d[2 * i + 1] = f.y;
  }
}

// e - 15 in -40 .. 0, where 2^e is the least power of two above the largest
// magnitude among DB fp16 scales (a NaN's are NaN whatever this is).
template <int DB>
__device__ __forceinline__ float log2_above(const __half* p) {
  __half2 h[DB / 2];
  if constexpr (DB == 2) *reinterpret_cast<uint32_t*>(h) = *reinterpret_cast<const uint32_t*>(p);
  else if constexpr (DB == 4) *reinterpret_cast<uint2*>(h) = *reinterpret_cast<const uint2*>(p);
  else *reinterpret_cast<uint4*>(h) = *reinterpret_cast<const uint4*>(p);
  __half2 m = __habs2(h[0]);
#pragma unroll
  for (int i = 1; i < DB / 2; ++i) m = __hmax2(m, __habs2(h[i]));
  const float2 f = __half22float2(m);
  // the exponent's field behind that of 2^23
  const float field = __uint_as_float(0x4B000000u | (__float_as_uint(fmaxf(f.x, f.y)) >> 23));
  return fminf(fmaxf(field - (8388608.f + 127.f + 14.f), -40.f), 0.f);
}

// One warp's stage: 32 tokens in two groups of 16.
template <int DB>
struct alignas(128) Stage {
  uint8_t k[2][16 * DB * 16];
  uint8_t v[2][16 * DB * 16];
  __half kd[2][16 * DB];
  __half vd[2][16 * DB];
};

// Slot of a 16-byte block in a group's plane: eight tokens' blocks b fall in
// eight different bank groups.
template <int DB>
__device__ __forceinline__ int block_slot(int row, int b) {
  return row * DB + (b ^ ((row / (8 / DB)) & (DB - 1)));
}

// What the warps' results are joined with, in shared memory.
template <int NT>
struct Join {
  float m[kWarps][8 * NT], l[kWarps][8 * NT], best[8 * NT], sum[8 * NT];
  int last;
};

// Dynamic shared memory (there is no other): the warps' rings, whose place the
// results take between two segments, then the queries.
constexpr int kBatchWords = 3200;   // pieces x rows whose maxima and sums stand in shared memory at a time
template <int DB, int NT>
__host__ __device__ constexpr int join_offset() {   // behind the warps' results, and behind a batch of pieces
  constexpr int results = kWarps * 8 * NT * (32 * DB + 4) * 4, batch = 2 * kBatchWords * 4;
  return results > batch ? results : batch;
}
template <int DB, int NT>
__host__ __device__ constexpr int query_offset() {
  constexpr int ring = static_cast<int>(sizeof(Stage<DB>)) * kStages * kWarps;
  constexpr int join = (join_offset<DB, NT>() + static_cast<int>(sizeof(Join<NT>)) + 15) / 16 * 16;
  return ring > join ? ring : join;
}
template <int DB, int NT>
constexpr int smem_bytes() {
  return query_offset<DB, NT>() + DB * NT * 32 * 16;
}

template <int DB, int NT>
struct Rows {
  float o[DB][2][NT][4];
  float m[NT][2], l[NT][2];
};

// Scores, softmax and values of one warp's 32 tokens.  MASK: some rows do
// not see all of them (column c of tile nt sees tokens below seen[nt][c]).
template <int DB, int NT, bool MASK>
__device__ __forceinline__ void warp_step(const Stage<DB>& st, int lane, const uint4* qs,
                                          const uint32_t (&off)[2][NT], const float (&scale2)[NT][2], int token0,
                                          const int (&seen)[NT][2], unsigned bad, Rows<DB, NT>& r) {
  const int g = lane >> 2;
  const int row = (lane & 7) + (lane & 8);
  const uint32_t lane_off = 16u * block_slot<DB>(row, lane >> 4);
  float s[2][NT][4];
#pragma unroll
  for (int mt = 0; mt < 2; ++mt) {
    float dk[2][DB];
    load_scales<DB>(&st.kd[mt][g * DB], dk[0]);
    load_scales<DB>(&st.kd[mt][(g + 8) * DB], dk[1]);
    // scales 2t, 2t + 1 (modulo DB) of tokens g and g + 8, as an A fragment
    const uint32_t d0 = *reinterpret_cast<const uint32_t*>(&st.kd[mt][g * DB + 2 * (lane & (DB / 2 - 1) & 3)]);
    const uint32_t d1 = *reinterpret_cast<const uint32_t*>(&st.kd[mt][(g + 8) * DB + 2 * (lane & (DB / 2 - 1) & 3)]);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 4; ++i) s[mt][nt][i] = 0.f;
      mma(s[mt][nt], d0, d1, DB == 8 ? d0 : 0u, DB == 8 ? d1 : 0u, off[0][nt], off[1][nt]);
    }
    const uint32_t base = smem_addr(st.k[mt]);
#pragma unroll
    for (int bp = 0; bp < DB / 2; ++bp) {
      uint32_t w[4];
      ldsm4<false>(w, base + (lane_off ^ (32u * bp)));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int b = 2 * bp + h;
        uint32_t lo[4], hi[4];
        decode(w[2 * h], lo);
        decode(w[2 * h + 1], hi);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float acc[4] = {0.f, 0.f, 0.f, 0.f};
          const uint4 q = qs[(b * NT + nt) * 32 + lane];
          mma(acc, lo[0], hi[0], lo[1], hi[1], q.x, q.y);
          mma(acc, lo[2], hi[2], lo[3], hi[3], q.z, q.w);
#pragma unroll
          for (int i = 0; i < 4; ++i) s[mt][nt][i] = fmaf(dk[i >> 1][b], acc[i], s[mt][nt][i]);
        }
      }
    }
  }
  // which of the thread's scores count: tokens g and g + 8 of both groups
  auto out = [&](int mt, int nt, int i) {
    return MASK && (token0 + 16 * mt + g + 8 * (i >> 1) >= seen[nt][i & 1] || ((bad >> (16 * mt)) & 1u));
  };
  // the lane's own token's, then those of its scores' tokens
  const float own = log2_above<DB>(&st.vd[lane >> 4][(lane & 15) * DB]);
  float lg[2][2];
#pragma unroll
  for (int mt = 0; mt < 2; ++mt)
#pragma unroll
    for (int h = 0; h < 2; ++h) lg[mt][h] = __shfl_sync(0xffffffffu, own, 16 * mt + 8 * h + g);
  bool grows = false;
  float mx[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[mt][nt][i] = out(mt, nt, i) ? -INFINITY : __fmul_rn(s[mt][nt][i], scale2[nt][i & 1]);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float v = fmaxf(fmaxf(__fadd_ru(s[0][nt][c], lg[0][0]), __fadd_ru(s[0][nt][c + 2], lg[0][1])),
                      fmaxf(__fadd_ru(s[1][nt][c], lg[1][0]), __fadd_ru(s[1][nt][c + 2], lg[1][1])));
      v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
      v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
      v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
      mx[nt][c] = fmaxf(r.m[nt][c], v);
      grows |= mx[nt][c] > r.m[nt][c];
    }
  }
  if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float alpha = mx[nt][c] == -INFINITY ? 1.f : exp2_approx(r.m[nt][c] - mx[nt][c]);
        r.m[nt][c] = mx[nt][c];
        r.l[nt][c] *= alpha;
#pragma unroll
        for (int b = 0; b < DB; ++b) {
          r.o[b][0][nt][c] *= alpha;
          r.o[b][0][nt][c + 2] *= alpha;
          r.o[b][1][nt][c] *= alpha;
          r.o[b][1][nt][c + 2] *= alpha;
        }
      }
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float m = MASK && r.m[nt][i & 1] == -INFINITY ? 0.f : r.m[nt][i & 1];
      s[0][nt][i] = exp2_approx(__fsub_rn(s[0][nt][i], m));
      s[1][nt][i] = exp2_approx(__fsub_rn(s[1][nt][i], m));
      r.l[nt][i & 1] += s[0][nt][i] + s[1][nt][i];
    }
  }
#pragma unroll
  for (int mt = 0; mt < 2; ++mt) {
    float dv[2][DB];
    load_scales<DB>(&st.vd[mt][g * DB], dv[0]);
    load_scales<DB>(&st.vd[mt][(g + 8) * DB], dv[1]);
    const uint32_t base = smem_addr(st.v[mt]);
#pragma unroll
    for (int bp = 0; bp < DB / 2; ++bp) {
      uint32_t w[4];
      ldsm4<true>(w, base + (lane_off ^ (32u * bp)));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int b = 2 * bp + h;
        uint32_t lo[4], hi[4];       // tokens 2t, 2t + 1 and 2t + 8, 2t + 9
        if (NT == 1) {
          decode(w[2 * h], lo);
          decode(w[2 * h + 1], hi);
        } else {
          decode_signed(w[2 * h], lo);
          decode_signed(w[2 * h + 1], hi);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float p[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)   // a token left out may hold any scale, NaN among them
            p[i] = out(mt, nt, i) ? 0.f : s[mt][nt][i] * dv[i >> 1][b];
          const uint32_t b0 = transpose8x8(pack_half2(p[0], p[1])), b1 = transpose8x8(pack_half2(p[2], p[3]));
          float(&o0)[4] = r.o[b][0][nt];
          float(&o1)[4] = r.o[b][1][nt];
          mma(o0, lo[0], lo[1], hi[0], hi[1], b0, b1);
          mma(o1, lo[2], lo[3], hi[2], hi[3], b0, b1);
          if (NT == 1) {
            mma(o0, kMinus8Low, kMinus8High, kMinus8Low, kMinus8High, b0, b1);
            mma(o1, kMinus8Low, kMinus8High, kMinus8Low, kMinus8High, b0, b1);
          }
        }
      }
    }
  }
}

// Four consecutive outputs.
__device__ __forceinline__ void store_out4(const AttnKv4Args& a, int64_t at, float4 v) {
  if (a.out_dtype == 3) {
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = v;
  } else if (a.out_dtype == 1) {
    const __half2 o[2] = {__floats2half2_rn(v.x, v.y), __floats2half2_rn(v.z, v.w)};
    *reinterpret_cast<uint2*>(static_cast<__half*>(a.out) + at) = *reinterpret_cast<const uint2*>(o);
  } else {
    const __nv_bfloat162 o[2] = {__floats2bfloat162_rn(v.x, v.y), __floats2bfloat162_rn(v.z, v.w)};
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + at) = *reinterpret_cast<const uint2*>(o);
  }
}

// A segment's queries, barriers and join cost about as much as five steps (12 ragged
// sequences with four queries: 41.3 us counted as three, 38.2 as five, 40.1 as eight).
constexpr int kSegmentCost = 5;

__device__ __forceinline__ int steps_of(int len) {   // a sequence without tokens has one (empty) step: its zeros
  return len > 0 ? (len + kStepTokens - 1) / kStepTokens : 1;
}

// Weight of a piece whose maximum is m among pieces whose largest is best.
__device__ __forceinline__ float piece_weight(float m, float best) {
  return best == -INFINITY ? 0.f : exp2_approx(m - best);
}

constexpr int kNoPage = INT32_MIN;

// Three CTAs an SM: 168 registers hold the loop without moves and spills (four
// CTAs with 128: 35 instructions more for 16 tokens, 123 us against 117 on 32
// ragged sequences; two: 125).  The larger accumulators need two.
//
// Measured on GB300 (dim 128, group 4, bf16): 32 sequences up to 32768, 607 MB:
// 117.4 us, 5.2 TB/s, 76 % of the copy rate; one of 131072, 151 MB: 38.3 us, of
// which 10 are its start and the join of 57 pieces a head; one of 1000: 8.7 us.
// Bound by its chains of dependent instructions with three warps a scheduler (280
// for 16 tokens of a head, of which 16 keep the products of probabilities and
// value scales in fp16's range: 114 us without; issue 56 %, ALU pipe 45 %, tensor
// pipe 40 %), not yet by DRAM: with the copies left out 112 us of then 117.
template <int DB, int NT>
__global__ void __launch_bounds__(kThreads, DB * NT == 8 ? 2 : 3)
attn_kv4_kernel(Kv4Args c, AttnKv4Args a, int tiles, int page_shift) {
  constexpr int D = 32 * DB, R = 8 * NT, kPitch = D + 4, kRecord = R * (D + 2);
  constexpr float kLow = NT == 1 ? 0x1p24f : 1.f, kHigh = NT == 1 ? 0x1p20f : 1.f;   // of the value codes' decoding
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  Stage<DB>* ring = reinterpret_cast<Stage<DB>*>(smem) + warp * kStages;
  float* merged = reinterpret_cast<float*>(smem);       // [warp][row][kPitch], between two segments
  Join<NT>& jn = *reinterpret_cast<Join<NT>*>(smem + join_offset<DB, NT>());
  uint4* qs = reinterpret_cast<uint4*>(smem + query_offset<DB, NT>());   // the queries' B fragments, [block][tile][lane]

  pdl_launch_dependents();
  pdl_wait();

  // All units of the call, laid end to end: sequence by sequence, a segment
  // for each (head, row tile).  Every warp finds its CTA's range by itself.
  const int per_seq = c.heads * tiles;
  int64_t total = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int n = b0 + lane < a.B ? steps_of(kv4_length(c, b0 + lane).held) + kSegmentCost : 0;
    total += __reduce_add_sync(0xffffffffu, static_cast<unsigned>(n));
  }
  total *= per_seq;
  const int64_t workers = min(static_cast<int64_t>(gridDim.x), total);
  if (blockIdx.x >= workers) return;
  const int64_t begin = blockIdx.x * total / workers, end = (blockIdx.x + 1) * total / workers;
  int b = 0;
  int64_t before = 0;                                   // units of the sequences in front of b
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int n = b0 + lane < a.B ? steps_of(kv4_length(c, b0 + lane).held) + kSegmentCost : 0;
    int run = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += up;
    }
    const unsigned past = __ballot_sync(0xffffffffu, before + static_cast<int64_t>(run) * per_seq > begin);
    if (past) {
      const int at = __ffs(past) - 1;
      before += static_cast<int64_t>(__shfl_sync(0xffffffffu, run - n, at)) * per_seq;
      b = b0 + at;
      break;
    }
    before += static_cast<int64_t>(__shfl_sync(0xffffffffu, run, 31)) * per_seq;
  }

  const int rows = a.L * a.group, per_page = c.page >> 4;
  // Copies: half a warp takes one of a step's two groups of 16 tokens.  What of
  // its addresses depends on the lane alone: 16-byte pieces of the group's
  // codes, and the pieces of its scales (keys', then values').
  const int half = lane >> 4, hl = lane & 15;
  const uint32_t page_bytes = static_cast<uint32_t>(c.heads) * c.page * (D / 2);
  const int64_t v_delta = c.vq - c.kq;
  const uint32_t lane_dst = smem_addr(ring) + half * (16 * DB * 16) + 16u * block_slot<DB>(hl / DB, hl % DB);
  const bool v_scales = DB < 8 && hl >= 2 * DB;         // 2 * DB pieces of each kind; for DB = 8 a lane takes both
  const uint32_t lane_scale_dst = smem_addr(ring) + half * (32 * DB) + 16u * (hl % (2 * DB)) +
                                  static_cast<uint32_t>(v_scales ? offsetof(Stage<DB>, vd) : offsetof(Stage<DB>, kd));
  const uint8_t* lane_scales = reinterpret_cast<const uint8_t*>(v_scales ? c.vd : c.kd) + 16 * (hl % (2 * DB));
  const int64_t vd_delta = reinterpret_cast<const uint8_t*>(c.vd) - reinterpret_cast<const uint8_t*>(c.kd);

  for (int64_t at = begin; at < end;) {
    const Kv4Length length = kv4_length(c, b);
    const int len = length.held;
    const int nsteps = steps_of(len);
    const int units = nsteps + kSegmentCost;
    const int seg = static_cast<int>((at - before) / units);
    const int64_t seg_first = before + static_cast<int64_t>(seg) * units, seg_steps = seg_first + kSegmentCost;
    const int step0 = static_cast<int>(max(at - seg_steps, static_cast<int64_t>(0)));
    const int step1 = static_cast<int>(min(end - seg_steps, static_cast<int64_t>(nsteps)));
    at = min(end, seg_first + units);
    const int this_b = b;
    if (at == before + static_cast<int64_t>(units) * per_seq) {
      before = at;
      ++b;
    }
    if (step1 <= step0) continue;                       // only the units in front of its steps
    const int head = seg / tiles, row0 = (seg - head * tiles) * R;

    const uint32_t head_bytes = static_cast<uint32_t>(head) * c.page * (D / 2);
    const uint8_t* k_codes = c.kq + head_bytes + 16 * hl;
    const uint8_t* scales = lane_scales + head_bytes / 8;
    const int32_t* table = c.table + this_b * c.ldt;

    // page of this half's group of a step and its byte offset in it; no page past the end
    auto locate = [&](int step, int& page, uint32_t& in_page) {
      const int tok = step * kStepTokens + warp * kWarpTokens + 16 * half;
      page = kNoPage;
      in_page = 0;
      if (step < step1 && tok < len) {
        const int grp = tok >> 4;
        const int p = page_shift >= 0 ? grp >> page_shift : grp / per_page;
        in_page = static_cast<uint32_t>(grp - p * per_page) * (16 * D / 2);
        page = table[p];
      }
    };
    // copies of a step's 32 tokens into ring slot `slot`; bits 0 and 16 of the
    // result: the half's group is not there (past the end, or no such page)
    auto issue = [&](int page, uint32_t in_page, int slot) -> unsigned {
      const uint32_t stage = static_cast<uint32_t>(slot) * static_cast<uint32_t>(sizeof(Stage<DB>));
      const bool bad = static_cast<unsigned>(page) >= static_cast<unsigned>(c.pages);
      if (!bad) {
        const uint64_t off = static_cast<uint64_t>(static_cast<uint32_t>(page)) * page_bytes + in_page;
        const uint8_t* k = k_codes + off;
        const uint8_t* v = k + v_delta;
        const uint32_t dst = lane_dst + stage;
#pragma unroll
        for (int x = 0; x < DB; ++x) {
          // a further 16 pieces are 16 / DB rows on, which turns bits of the swizzle
          constexpr int kTurn = DB == 8 ? 2 : DB == 4 ? 2 : 0;
          const uint32_t d = (dst ^ (16u * ((kTurn * x) & (DB - 1)))) + 256u * x;
          copy16(d, k + 256 * x);
          copy16(d + static_cast<uint32_t>(sizeof(ring->k)), v + 256 * x);
        }
        const uint8_t* sc = scales + (off >> 3);
        if (DB == 8) copy16(lane_scale_dst + stage + static_cast<uint32_t>(sizeof(ring->kd)), sc + vd_delta);
        if (hl < 4 * DB) copy16(lane_scale_dst + stage, sc);
      } else if (page != kNoPage && c.err) {
        *c.err = kErrCacheIndex;
      }
      copy_commit();
      return __ballot_sync(0xffffffffu, bad) & 0x10001u;
    };
    int page;
    uint32_t in_page;
    locate(step0, page, in_page);
    unsigned bad = issue(page, in_page, 0);
    locate(step0 + 1, page, in_page);

    // the queries as B fragments (a warp stores its share), their power of two, each block's sum
    uint32_t off[2][NT];
    float scale2[NT][2];
    int seen[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = row0 + 8 * nt + g;
      const int i = row / a.group;
      const uint16_t* q = static_cast<const uint16_t*>(a.q.p) + this_b * a.q.sb + i * a.q.st +
                          (head * a.group + (row - i * a.group)) * a.q.sh;
      const bool in = row < rows;
      uint32_t raw[DB][4];
      float most = 0.f;
      // of each block the elements (4t, 4t + 2), (16 + 4t, ..), (4t + 1, 4t + 3), (16 + 4t + 1, ..)
      if (a.q_vec) {
#pragma unroll
        for (int blk = 0; blk < DB; ++blk)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint2 v = in ? *reinterpret_cast<const uint2*>(q + 32 * blk + 16 * x + 4 * t) : make_uint2(0u, 0u);
            raw[blk][x] = __byte_perm(v.x, v.y, 0x5410);
            raw[blk][x + 2] = __byte_perm(v.x, v.y, 0x7632);
          }
      } else {
#pragma unroll
        for (int blk = 0; blk < DB; ++blk)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int e = 32 * blk + 16 * (x & 1) + 4 * t + (x >> 1);
            raw[blk][x] = in ? q[e] | (static_cast<uint32_t>(q[e + 2]) << 16) : 0u;
          }
      }
      auto both = [&](uint32_t v) {
        return a.q_dtype == 2 ? to_float2(v, static_cast<const __nv_bfloat16*>(nullptr))
                              : to_float2(v, static_cast<const __half*>(nullptr));
      };
#pragma unroll
      for (int blk = 0; blk < DB; ++blk)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float2 f = both(raw[blk][x]);
          most = fmaxf(most, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
      // 2^e with most * 2^e in [2^14, 2^15); infinities stay as they are
      int e = 14 - (static_cast<int>(__float_as_uint(most) >> 23) - 127);
      e = most > 3.4e38f ? 0 : min(e, 127);
      const float pow2 = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
      // the scale's sign goes into the queries, so that the largest sum has the largest score
      const float up = a.scale < 0.f ? -pow2 : a.scale > 0.f ? pow2 : 0.f * a.scale;
      float hi[DB], lo[DB];
#pragma unroll
      for (int blk = 0; blk < DB; ++blk) {
        float sum = 0.f;
        uint32_t qf[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float2 f = both(raw[blk][x]);
          const float to = (x & 1) ? up * 0.0625f : up;      // these meet the high codes
          const __half2 h = __floats2half2_rn(f.x * to, f.y * to);
          qf[x] = *reinterpret_cast<const uint32_t*>(&h);
          const float2 back = __half22float2(h);
          sum = fmaf(back.x + back.y, (x & 1) ? 16.f : 1.f, sum);
        }
        if ((blk & (kWarps - 1)) == warp) qs[(blk * NT + nt) * 32 + lane] = make_uint4(qf[0], qf[1], qf[2], qf[3]);
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        sum *= -8.f * 0x1p-24f;
        hi[blk] = __half2float(__float2half_rn(sum));
        lo[blk] = sum - hi[blk];
      }
      // B fragment of the offsets: along k the blocks' high parts, then their low parts
      off[0][nt] = off[1][nt] = 0;
#pragma unroll
      for (int p = 0; p < DB / 2; ++p) {
        if (t == p) off[0][nt] = pack_half2(hi[2 * p], hi[2 * p + 1]);
        if (DB < 8 && t == p + DB / 2) off[0][nt] = pack_half2(lo[2 * p], lo[2 * p + 1]);
        if (DB == 8 && t == p) off[1][nt] = pack_half2(lo[2 * p], lo[2 * p + 1]);
      }
      // log2(e) and the powers of two (finite also for queries past 2^117, whose scores then
      // are further apart than any exponential tells); a scale of 0 has made the queries 0
      const float down = fminf((a.scale == 0.f ? 1.f : fabsf(a.scale)) * (1.44269504088896341f * 0x1p24f) / pow2, 3.402823466e38f);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        scale2[nt][x] = __shfl_sync(0xffffffffu, down, 8 * t + 4 * x);
        const int col = row0 + 8 * nt + 2 * t + x;      // rows past the last are computed and dropped
        seen[nt][x] = col < rows ? min(len, max(0, length.given - a.L + col / a.group + 1)) : len;
      }
    }
    const int all_see = min(len, max(0, length.given - a.L + row0 / a.group + 1));   // tokens that every row of the tile sees
    __syncthreads();

    Rows<DB, NT> r;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        r.m[nt][x] = -INFINITY;
        r.l[nt][x] = 0.f;
#pragma unroll
        for (int blk = 0; blk < DB; ++blk)
          r.o[blk][0][nt][x] = r.o[blk][0][nt][x + 2] = r.o[blk][1][nt][x] = r.o[blk][1][nt][x + 2] = 0.f;
      }

    // Two steps a turn, so that the ring's two slots are constants (32 ragged
    // sequences: 113 us against 117; with two row tiles of dim 128 the second
    // step's registers cost more than that).
    constexpr int kUnroll = DB * NT <= 4 ? 2 : 1;
    int slot = 0;
#pragma unroll kUnroll
    for (int step = step0; step < step1; ++step) {
      copy_wait<0>();
      __syncwarp();
      const unsigned next_bad = issue(page, in_page, slot ^ 1);
      locate(step + 2, page, in_page);                  // the table's entry is there a step later
      const int token0 = step * kStepTokens + warp * kWarpTokens;
      if (token0 + kWarpTokens <= all_see && bad == 0)
        warp_step<DB, NT, false>(ring[slot], lane, qs, off, scale2, token0, seen, 0u, r);
      else if (bad != 0x10001u)
        warp_step<DB, NT, true>(ring[slot], lane, qs, off, scale2, token0, seen, bad, r);
      bad = next_bad;
      slot ^= 1;
    }
    copy_wait<0>();
    __syncthreads();               // the ring becomes the place of the warps' results

#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float l = r.l[nt][x];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        const int row = 8 * nt + 2 * t + x;
        if (g == 0) {
          jn.m[warp][row] = r.m[nt][x];
          jn.l[warp][row] = l;
        }
        float* o = merged + (warp * R + row) * kPitch;
#pragma unroll
        for (int blk = 0; blk < DB; ++blk) {
          *reinterpret_cast<float2*>(o + 32 * blk + 2 * g) =
              make_float2(r.o[blk][0][nt][x] * kLow, r.o[blk][1][nt][x] * kLow);
          *reinterpret_cast<float2*>(o + 32 * blk + 16 + 2 * g) =
              make_float2(r.o[blk][0][nt][x + 2] * kHigh, r.o[blk][1][nt][x + 2] * kHigh);
        }
      }
    __syncthreads();

    const int tile_rows = min(R, rows - row0);
    const bool whole = step0 == 0 && step1 == nsteps;
    auto finish = [&](int row, int e, float4 o, float l) {
      const int q = row0 + row, i = q / a.group;
      const float f = l == 0.f ? 0.f : 1.0f / l;       // a NaN sum stays one
      store_out4(a, ((static_cast<int64_t>(this_b) * a.L + i) * c.heads * a.group + head * a.group + (q - i * a.group)) * D + e,
                 make_float4(o.x * f, o.y * f, o.z * f, o.w * f));
    };
    if (tid < R) {                 // the warps' weights take the place of their maxima
      float best = jn.m[0][tid], l = 0.f;
#pragma unroll
      for (int w = 1; w < kWarps; ++w) best = fmaxf(best, jn.m[w][tid]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = piece_weight(jn.m[w][tid], best);
        jn.m[w][tid] = f;
        l = fmaf(f, jn.l[w][tid], l);
      }
      jn.best[tid] = best;
      jn.sum[tid] = l;
    }
    __syncthreads();
    // records of this CTA: 0 for a segment that begins in front of its range, 1 for one that begins in it
    float* record = a.partials + (static_cast<int64_t>(blockIdx.x) * 2 + (seg_first >= begin)) * kRecord;
    for (int x = tid; x < tile_rows * (D / 4); x += kThreads) {
      const int row = x / (D / 4), e = 4 * (x % (D / 4));
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = jn.m[w][row];
        const float4 v = *reinterpret_cast<const float4*>(merged + (w * R + row) * kPitch + e);
        o.x = fmaf(f, v.x, o.x); o.y = fmaf(f, v.y, o.y); o.z = fmaf(f, v.z, o.z); o.w = fmaf(f, v.w, o.w);
      }
      if (whole) finish(row, e, o, jn.sum[row]);
      else __stcg(reinterpret_cast<float4*>(record) + x, o);
    }
    if (!whole) {
      if (tid < tile_rows) {
        __stcg(record + R * D + tid, jn.best[tid]);
        __stcg(record + R * D + R + tid, jn.sum[tid]);
      }
      // workers first .. last hold pieces of this segment
      const int first = static_cast<int>(((seg_steps + 1) * workers + total - 1) / total) - 1;
      const int last = static_cast<int>(((seg_first + units) * workers + total - 1) / total) - 1;
      const int pieces = last - first + 1;
      __syncthreads();
      if (tid == 0) {
        // releases the CTA's record (ordered by the barrier) and acquires those of the CTAs before
        unsigned* counter = a.counters + (static_cast<int64_t>(this_b) * per_seq + seg);
        unsigned prev;
        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(prev) : "l"(counter) : "memory");
        jn.last = prev == static_cast<unsigned>(pieces - 1);
        if (jn.last) *counter = 0u;
      }
      __syncthreads();
      if (jn.last) {
        const float* rec0 = a.partials + static_cast<int64_t>(first) * 2 * kRecord;
        const int skip = seg_first >= static_cast<int64_t>(first) * total / workers ? kRecord : 0;
        auto piece = [&](int p) { return rec0 + static_cast<int64_t>(p) * 2 * kRecord + (p == 0 ? skip : 0); };
        // batches of pieces: their maxima and sums to shared memory, a warp a row
        // turns them into weights, then every thread adds its columns
        constexpr int kBatch = kBatchWords / R;
        float* bm = merged;                             // [row][piece of the batch]: maxima, then weights
        float* bl = merged + R * kBatch;                // sums; jn.m[0][row]: what the batches before are scaled by
        constexpr int kMine = (R * D / 4 + kThreads - 1) / kThreads;
        float4 sum[kMine];
#pragma unroll
        for (int y = 0; y < kMine; ++y) sum[y] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (tid < R) {
          jn.best[tid] = -INFINITY;
          jn.sum[tid] = 0.f;
        }
        for (int p0 = 0; p0 < pieces; p0 += kBatch) {
          const int n = min(kBatch, pieces - p0);
          __syncthreads();
#pragma unroll 4
          for (int x = tid; x < n * tile_rows; x += kThreads) {
            const int p = x / tile_rows, row = x - p * tile_rows;
            const float* rec = piece(p0 + p) + R * D + row;
            bm[row * kBatch + p] = __ldcg(rec);
            bl[row * kBatch + p] = __ldcg(rec + R);
          }
          __syncthreads();
          for (int row = warp; row < tile_rows; row += kWarps) {
            const float old = jn.best[row];
            float best = old, l = 0.f;
            for (int p = lane; p < n; p += 32) best = fmaxf(best, bm[row * kBatch + p]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
            for (int p = lane; p < n; p += 32) {
              const float f = piece_weight(bm[row * kBatch + p], best);
              bm[row * kBatch + p] = f;
              l = fmaf(f, bl[row * kBatch + p], l);
            }
            l = warp_sum(l);
            __syncwarp();
            if (lane == 0) {
              const float f = piece_weight(old, best);
              jn.m[0][row] = f;
              jn.sum[row] = fmaf(jn.sum[row], f, l);
              jn.best[row] = best;
            }
          }
          __syncthreads();
#pragma unroll
          for (int y = 0; y < kMine; ++y) {
            const int x = tid + y * kThreads;
            if (x >= tile_rows * (D / 4)) continue;
            const int row = x / (D / 4);
            const float f0 = jn.m[0][row];
            sum[y] = make_float4(sum[y].x * f0, sum[y].y * f0, sum[y].z * f0, sum[y].w * f0);
            // the columns of kFlight pieces are on their way at a time: 16 where a long
            // context has many (8192 tokens 12.9 us, 13.3 with 12; 20 cost the loop
            // over the cache its registers), 4 where those are all
            auto add = [&](auto flight, int p) {
              constexpr int kFlight = decltype(flight)::value;
              float4 v[kFlight];
#pragma unroll
              for (int z = 0; z < kFlight; ++z)
                v[z] = p + z < n ? __ldcg(reinterpret_cast<const float4*>(piece(p0 + p + z)) + x) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
              for (int z = 0; z < kFlight; ++z) {
                const float f = p + z < n ? bm[row * kBatch + p + z] : 0.f;
                sum[y].x = fmaf(f, v[z].x, sum[y].x); sum[y].y = fmaf(f, v[z].y, sum[y].y);
                sum[y].z = fmaf(f, v[z].z, sum[y].z); sum[y].w = fmaf(f, v[z].w, sum[y].w);
              }
            };
            if (n <= 4) add(std::integral_constant<int, 4>(), 0);
            else
              for (int p = 0; p < n; p += 16) add(std::integral_constant<int, 16>(), p);
          }
        }
#pragma unroll
        for (int y = 0; y < kMine; ++y) {
          const int x = tid + y * kThreads;
          if (x < tile_rows * (D / 4)) finish(x / (D / 4), 4 * (x % (D / 4)), sum[y], jn.sum[x / (D / 4)]);
        }
      }
    }
    __syncthreads();               // before the ring is filled again
  }
}

// Row tiles: as many n8 tiles as the rows fill, at most what the output's
// accumulators leave registers for (64 a thread; dim 64 could hold four tiles, but
// runs as two CTAs an SM then: 37.8 us against 34.1 on 2 sequences of 32 queries).
constexpr int most_tiles(int db) { return db <= 4 ? 2 : 1; }
int tiles_of_eight(int rows, int db) {
  int nt = 1;
  while (nt < most_tiles(db) && 8 * nt < rows) nt *= 2;
  return nt;
}

template <int DB, int NT>
cudaError_t launch_t(const Kv4Args& c, const AttnKv4Args& a, cudaStream_t st, Launch* info) {
  auto kernel = attn_kv4_kernel<DB, NT>;
  constexpr int smem = smem_bytes<DB, NT>();
  static std::atomic<uint64_t> ready{0};                // devices whose kernel has its shared memory
  cudaError_t e = once_on_device(ready, [&] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (e != cudaSuccess) return e;
  const int resident = max_resident_ctas(reinterpret_cast<const void*>(kernel), kThreads, smem);
  const int tiles = (a.L * a.group + 8 * NT - 1) / (8 * NT);
  // no more CTAs than the table has units for
  const int64_t most = static_cast<int64_t>(a.B) * c.heads * tiles *
                       ((static_cast<int64_t>(c.max_pages) * c.page + kStepTokens - 1) / kStepTokens + kSegmentCost);
  int64_t grid = static_cast<int64_t>(device_sm_count()) * (resident < kAttnMaxResident ? resident : kAttnMaxResident);
  if (grid > most) grid = most;
  const int per_page = c.page / 16;
  int shift = -1;
  if ((per_page & (per_page - 1)) == 0)
    for (shift = 0; (1 << shift) < per_page; ++shift) {}
  info->kernel = "attn_kv4";
  info->grid_x = static_cast<int>(grid);
  info->block = kThreads;
  info->smem = smem;
  return launch_k(kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), smem, st, true, c, a, tiles, shift);
}

}  // namespace

size_t attn_kv4_partial_bytes(int dim) {
  const int rows = 8 * most_tiles(dim / 32);
  return static_cast<size_t>(device_sm_count()) * kAttnMaxResident * 2 * rows * (dim + 2) * sizeof(float);
}
int attn_kv4_tiles(int L, int group, int dim) {
  const int rows = L * group, per = 8 * tiles_of_eight(rows, dim / 32);
  return (rows + per - 1) / per;
}

cudaError_t launch_attn_kv4(const Kv4Args& c, const AttnKv4Args& a, cudaStream_t st, Launch* info) {
  const int db = c.dim / 32, nt = tiles_of_eight(a.L * a.group, db);
  if (db == 2) return nt == 1 ? launch_t<2, 1>(c, a, st, info) : launch_t<2, 2>(c, a, st, info);
  if (db == 4) return nt == 1 ? launch_t<4, 1>(c, a, st, info) : launch_t<4, 2>(c, a, st, info);
  return launch_t<8, 1>(c, a, st, info);
}

}  // namespace wobs
