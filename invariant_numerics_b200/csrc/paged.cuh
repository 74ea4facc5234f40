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

// Two INT16 codes (low half first) as binary16 pairs with code / 2 = hi + lo,
// hi = rn16(code / 2), both exact.  t = (code + 32768) >> 6 and l = code & 63
// give code / 2 = 32 (t - 512) + l / 2 (1024 + t and 1024 + l are formed in the
// binary16 mantissa); the sum rounds to hi and its error is lo.  (Keeping the
// unrounded pair saves 3 of the 8 instructions, but then the dropped product
// lo x_lo reaches 2^-20 of the row's largest code: 2.1e-6 against 8.6e-7 of
// fp32 sums at 300 keys, where hi = rn16 leaves 2^-22 of each product.)
__device__ __forceinline__ void unpack_code(uint32_t x, uint32_t& hi, uint32_t& lo) {
  const uint32_t t = ((x >> 6) & 0x03FF03FFu) ^ 0x66006600u;  // 1024 + t (the xor biases the code)
  const uint32_t l = (x & 0x003F003Fu) | 0x64006400u;         // 1024 + l
  const uint32_t k32 = 0x50005000u, m49152 = 0xFA00FA00u;     // 32, -49152
  const uint32_t kh = 0x38003800u, m512 = 0xE000E000u;        // 1/2, -512
  const __half2 h0 = __hfma2(*reinterpret_cast<const __half2*>(&t), *reinterpret_cast<const __half2*>(&k32),
                             *reinterpret_cast<const __half2*>(&m49152));
  const __half2 l0 = __hfma2(*reinterpret_cast<const __half2*>(&l), *reinterpret_cast<const __half2*>(&kh),
                             *reinterpret_cast<const __half2*>(&m512));
  const __half2 hv = __hadd2_rn(h0, l0);
  const __half2 lv = __hadd2_rn(__hsub2_rn(h0, hv), l0);
  hi = *reinterpret_cast<const uint32_t*>(&hv);
  lo = *reinterpret_cast<const uint32_t*>(&lv);
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
