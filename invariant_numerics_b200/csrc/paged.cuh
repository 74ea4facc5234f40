// Ragged-batch descriptors and the row arithmetic shared by the paged-cache
// kernels.
#pragma once

#include "common.cuh"

namespace inv {

// Page of a paged cache: codes of (page, head) are [page_size][128] int16.
struct PagedView {
  int16_t* k;
  int16_t* v;
  float* k_scale;
  float* v_scale;
  int n_pages;
  int n_kv_heads;
  int page_shift;  // log2(page_size)
};

struct RaggedBatch {
  const int32_t* page_table;  // [n_seqs][ld_table]
  int64_t ld_table;
  int n_seqs;
  const int32_t* q_start;  // [n_seqs + 1]
  const int32_t* len;      // [n_seqs]
};

// The entries of the descriptors; every read is checked in the index-checking build.
__device__ __forceinline__ int start_of(const RaggedBatch& rb, int i, [[maybe_unused]] int* status) {
  return INV_IN_BOUNDS(status, i, (int64_t)rb.n_seqs + 1) ? rb.q_start[i] : 0;
}
__device__ __forceinline__ int len_of(const RaggedBatch& rb, int i, [[maybe_unused]] int* status) {
  return INV_IN_BOUNDS(status, i, rb.n_seqs) ? rb.len[i] : 0;
}
__device__ __forceinline__ int page_of(const RaggedBatch& rb, int i, int64_t j, [[maybe_unused]] int* status) {
  return INV_IN_BOUNDS(status, j, rb.ld_table) && INV_IN_BOUNDS(status, i, rb.n_seqs)
             ? rb.page_table[i * rb.ld_table + j]
             : -1;
}

// The last i in [0, n) with key(i) <= x, or -1; key ascending.  One warp: each
// step compares 32 evenly spaced keys, so 32^k candidates take k dependent
// loads (a binary search would take five times as many).
template <class Key>
__device__ __forceinline__ int warp_upper(int n, int64_t x, int lane, Key key) {
  int lo = -1, cnt = n;  // the answer is lo or one of the cnt entries after it
  while (cnt > 0) {
    const int step = (cnt + 31) / 32;
    const int i = lo + min((lane + 1) * step, cnt);
    const unsigned hit = __ballot_sync(0xffffffffu, key(i) <= x);
    const int m = __popc(hit);  // ascending keys: the lanes that hit come first
    const int next = lo + min(m * step, cnt);
    if (m == 32) return next;  // lane 31's entry is the last one
    cnt = min(step - 1, lo + cnt - next);
    lo = next;
  }
  return lo;
}

// log2 scale that brings a value with the given fp32 bits into [2^13, 2^14)
// (bits of a non-negative number; zero and subnormals get the largest one).
__device__ __forceinline__ int norm_exp(float x) { return min(140 - (int)(__float_as_uint(x) >> 23), 126); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// Two INT16 codes (low half first) as binary16 pairs with code / 2 = hi + lo,
// hi = rn16(code / 2), both exact.  t = (code + 32768) >> 6 and l = code & 63
// give code / 2 = 32 (t - 512) + l / 2; T = 1024 + t and U = 1024 + l are formed
// in the binary16 mantissa.  With z = 32 T - 49664 = 32 (t - 512) - 512 (exact),
// hi = rn16(U / 2 + z), and z - hi and lo = U / 2 + (z - hi) are exact again.
// (Splitting into 32 (t - 512) and l / 2 saves two of the seven instructions,
// but then the dropped product lo x_lo reaches 2^-20 of the row's largest code:
// 2.1e-6 against 8.6e-7 of fp32 sums at 300 keys, where hi = rn16 leaves 2^-22
// of each product.)
__device__ __forceinline__ void unpack_code(uint32_t x, uint32_t& hi, uint32_t& lo) {
  uint32_t t, u;
  asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(t) : "r"(x >> 6), "r"(0x03FF03FFu), "r"(0x66006600u));  // (a & b) ^ c
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(u) : "r"(x), "r"(0x003F003Fu), "r"(0x64006400u));       // (a & b) | c
  const uint32_t z = hfma2(t, 0x50005000u, 0xFA10FA10u);  // 32 T - 49664
  hi = hfma2(u, 0x38003800u, z);                          // U / 2 + z
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(z), "r"(hi));
  lo = hfma2(u, 0x38003800u, r);
}

// x = hi + lo up to 2^-22 |x| (not scaled: x is within a normalised range).
__device__ __forceinline__ void split_plain(float x, __half& hi, __half& lo) {
  hi = __float2half_rn(x);
  lo = __float2half_rn(__fsub_rn(x, __half2float(hi)));
}

// Host checks shared by the paged entry points; fills the device views.
inline int check_paged(const inv_paged_kv_cache* c, int n_heads) {
  if (!c || n_heads <= 0) return INV_ERR_INVALID_ARG;
  if (c->head_dim != INV_HEAD_DIM) return INV_ERR_UNSUPPORTED_SHAPE;
  if (c->n_pages <= 0 || c->n_kv_heads <= 0) return INV_ERR_INVALID_ARG;
  const int ps = c->page_size;
  if (ps < 16 || ps > 256 || (ps & (ps - 1)) != 0) return INV_ERR_UNSUPPORTED_SHAPE;
  if (n_heads % c->n_kv_heads != 0) return INV_ERR_UNSUPPORTED_SHAPE;
  // cache rows are 32-bit tensor-map coordinates
  if ((uint64_t)c->n_pages * c->n_kv_heads * ps >= (1ull << 31)) return INV_ERR_UNSUPPORTED_SHAPE;
  return INV_OK;
}

inline PagedView paged_view(const inv_paged_kv_cache& c) {
  int sh = 4;
  while ((1 << sh) < c.page_size) ++sh;
  return {c.k, c.v, c.k_scale, c.v_scale, c.n_pages, c.n_kv_heads, sh};
}

}  // namespace inv
