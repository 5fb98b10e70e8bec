// The paged 4-bit key/value cache, as its kernels see it.
//
// Planes: codes [pages][heads][page][dim/2] (Q4_0 blocks of 32 along a
// token's head: byte j of a block holds element j in its low nibble and
// element j + 16 in its high one) and fp16 scales [pages][heads][page][dim/32].
// Token t of sequence b lies in slot t % page of page table[b][t / page].
// Offsets are 64-bit: a cache may hold more than 2^32 bytes.
#pragma once

#include "common.cuh"

namespace wobs {

// Tokens of sequence b: as many as its length says, and those of them that its
// table has room for (0 .. max_pages * page); a length outside that range is
// recorded in the error word.  Positions follow from the given length, so the
// tokens past the table's end are the ones left out.
struct Kv4Length {
  int given, held;
};
__device__ __forceinline__ Kv4Length kv4_length(const Kv4Args& c, int b) {
  const int n = c.lens[b];
  const int64_t most = static_cast<int64_t>(c.max_pages) * c.page;
  if (n < 0 || n > most) {
    if (c.err) *c.err = kErrCacheIndex;
    return n < 0 ? Kv4Length{0, 0} : Kv4Length{n, static_cast<int>(most)};
  }
  return {n, n};
}

// n / d, by a shift where the (uniform) d is a power of two.
__device__ __forceinline__ unsigned quotient(unsigned n, unsigned d) {
  return (d & (d - 1)) == 0 ? n >> (31 - __clz(d)) : n / d;
}

// Where token t of a sequence lies: entry of its table, slot in the page.
struct Kv4Token {
  int entry, slot;
};
__device__ __forceinline__ Kv4Token kv4_token(const Kv4Args& c, int t) {
  const int entry = static_cast<int>(quotient(t, c.page));
  return {entry, t - entry * c.page};
}

// Page of token t of sequence b; -1 (and the error word) where the table
// names a page that the cache does not have.
__device__ __forceinline__ int kv4_page(const Kv4Args& c, int b, Kv4Token t) {
  const int p = c.table[b * c.ldt + t.entry];
  if (p < 0 || p >= c.pages) {
    if (c.err) *c.err = kErrCacheIndex;
    return -1;
  }
  return p;
}

// First slot-of-head index (a token row) of token t in page p.
__device__ __forceinline__ int64_t kv4_row(const Kv4Args& c, int p, int head, Kv4Token t) {
  return (static_cast<int64_t>(p) * c.heads + head) * c.page + t.slot;
}

}  // namespace wobs
