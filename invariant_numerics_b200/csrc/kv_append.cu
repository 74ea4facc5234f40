// kv_append_paged: head norms, rotary embedding and INT16 quantisation of the
// new tokens' q | k | v rows, K and V going straight to their pages.
#include "paged.cuh"

namespace {

using inv::record_status;

constexpr int kAppendThreads = 256;

// HBM bound (a row reads 512 bytes a head, writes 512 a query and 260 a key or
// value head).  One CTA per row, and one that checks q_start; one warp per head (warp w
// takes heads w, w + 8, ...).  Lane l holds the dims 2l, 2l+1, 64+2l, 65+2l, so a rotary pair (i, i+64) is
// in one lane and a warp's loads are two contiguous 256-byte runs.  A warp requests
// kBatch heads before it looks up the row's sequence, position and page (three
// dependent reads), so that both latencies overlap: 70 us for 8192 rows (32 query, 8
// kv heads) = 5.3 TB/s, 78 with the look-ups first; 5.6 us for 64 sequences of up to
// 5 tokens.  (q_start checked by every row's CTA: 3 us more for the 8192.)
constexpr int kBatch = 6;

__global__ void __launch_bounds__(kAppendThreads)
    kv_append_kernel(const float* __restrict__ qkv, int64_t ld, int T, int Hq, inv::PagedView c, inv::RaggedBatch rb,
                     const float* __restrict__ cos_t, const float* __restrict__ sin_t, int max_pos,
                     const float* __restrict__ q_gain, const float* __restrict__ k_gain, double eps,
                     float* __restrict__ q_out, int* status) {
  constexpr int W = kAppendThreads / 32;
  if (blockIdx.x == 0) {
    // the rows' CTAs see only their own sequence's part of q_start
    for (int j = threadIdx.x; j < rb.n_seqs; j += kAppendThreads) {
      const int q0 = inv::start_of(rb, j, status), q1 = inv::start_of(rb, j + 1, status);
      if (q0 < 0 || q1 < q0 || q1 > T) record_status(status, INV_ERR_INVALID_ARG);
    }
    return;
  }
  const int r = blockIdx.x - 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int Hkv = c.n_kv_heads, H = Hq + 2 * Hkv;
  float2 x[kBatch][2];
  const auto request = [&](int h0) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int h = h0 + j * W;
      const int64_t ix = (int64_t)r * ld + (int64_t)h * 128;
      if (h < H && INV_SPAN_IN_BOUNDS(status, ix, ix + 127, (int64_t)(T - 1) * ld + (int64_t)H * 128)) {
        x[j][0] = reinterpret_cast<const float2*>(qkv + ix)[lane];
        x[j][1] = reinterpret_cast<const float2*>(qkv + ix + 64)[lane];
      }
    }
  };
  request(warp);
  const int i = inv::warp_upper(rb.n_seqs, r, lane, [&](int j) { return inv::start_of(rb, j, status); });
  if (i < 0) return;
  const int q0 = inv::start_of(rb, i, status), q1 = inv::start_of(rb, i + 1, status);
  if (r >= q1) return;  // behind the last sequence
  const int len = inv::len_of(rb, i, status);
  const int64_t pos = (int64_t)len - (q1 - r);
  int page = -1;
  // (r < q0: q_start descends and the search went astray)
  if (q0 >= 0 && r >= q0 && q1 <= T && pos >= 0 && pos < max_pos && len >= q1 - q0 &&
      (pos >> c.page_shift) < rb.ld_table)
    page = inv::page_of(rb, i, pos >> c.page_shift, status);
  if (page < 0 || page >= c.n_pages) {
    if (threadIdx.x == 0) record_status(status, INV_ERR_INVALID_ARG);
    return;
  }
  if (!INV_SPAN_IN_BOUNDS(status, pos * 64, pos * 64 + 63, (int64_t)max_pos * 64)) return;
  const float2 cv0 = reinterpret_cast<const float2*>(cos_t + pos * 64)[lane];
  const float2 sv0 = reinterpret_cast<const float2*>(sin_t + pos * 64)[lane];
  const float cv[2] = {cv0.x, cv0.y}, sv[2] = {sv0.x, sv0.y};
  const int ps = 1 << c.page_shift, off = (int)(pos & (ps - 1));
#pragma unroll 1
  for (int h0 = warp; h0 < H; h0 += kBatch * W) {
    if (h0 != warp) request(h0);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int h = h0 + j * W;
      if (h >= H) break;
      float a[2] = {x[j][0].x, x[j][0].y}, b[2] = {x[j][1].x, x[j][1].y};
      const bool is_v = h >= Hq + Hkv;
      if (!is_v) {
        const float* gain = h < Hq ? q_gain : k_gain;
        if (gain != nullptr) {
          double ss = (double)a[0] * a[0] + (double)a[1] * a[1] + (double)b[0] * b[0] + (double)b[1] * b[1];
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          const float rs = (float)rsqrt(ss * (1.0 / 128.0) + eps);
          const float2 ga = reinterpret_cast<const float2*>(gain)[lane];
          const float2 gb = reinterpret_cast<const float2*>(gain + 64)[lane];
          a[0] = __fmul_rn(__fmul_rn(a[0], rs), ga.x);
          a[1] = __fmul_rn(__fmul_rn(a[1], rs), ga.y);
          b[0] = __fmul_rn(__fmul_rn(b[0], rs), gb.x);
          b[1] = __fmul_rn(__fmul_rn(b[1], rs), gb.y);
        }
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          const float lo = a[d], hi = b[d];
          a[d] = __fsub_rn(__fmul_rn(lo, cv[d]), __fmul_rn(hi, sv[d]));
          b[d] = __fadd_rn(__fmul_rn(hi, cv[d]), __fmul_rn(lo, sv[d]));
        }
      }
      if (h < Hq) {
        const int64_t oq = ((int64_t)r * Hq + h) * 128;
        if (!INV_SPAN_IN_BOUNDS(status, oq, oq + 127, (int64_t)T * Hq * 128)) continue;
        reinterpret_cast<float2*>(q_out + oq)[lane] = make_float2(a[0], a[1]);
        reinterpret_cast<float2*>(q_out + oq + 64)[lane] = make_float2(b[0], b[1]);
        continue;
      }
      const int hk = is_v ? h - Hq - Hkv : h - Hq;
      const int64_t row = ((int64_t)page * Hkv + hk) * ps + off;
      if (!INV_IN_BOUNDS(status, row, (int64_t)c.n_pages * Hkv * ps)) continue;
      float m = fmaxf(fmaxf(fabsf(a[0]), fabsf(a[1])), fmaxf(fabsf(b[0]), fabsf(b[1])));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));  // exact
      const float s = __fdiv_rn(m, 32767.0f);
      const float in[4] = {a[0], a[1], b[0], b[1]};
      int q[4] = {0, 0, 0, 0};
      if (s != 0.0f) {
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const int t = __float2int_rn(__fdiv_rn(in[d], s));  // IEEE division, round half to even
          q[d] = t > 32767 ? 32767 : (t < -32767 ? -32767 : t);
        }
      }
      uint32_t* codes = reinterpret_cast<uint32_t*>((is_v ? c.v : c.k) + row * 128);
      codes[lane] = (uint32_t)(uint16_t)q[0] | ((uint32_t)(uint16_t)q[1] << 16);
      codes[32 + lane] = (uint32_t)(uint16_t)q[2] | ((uint32_t)(uint16_t)q[3] << 16);
      if (lane == 0) (is_v ? c.v_scale : c.k_scale)[row] = s;
    }
  }
}

}  // namespace

extern "C" {

int kv_append_paged(const float* qkv, int64_t ld_qkv, int T, int n_heads, const inv_paged_kv_cache* cache,
                    const int32_t* page_table, int64_t ld_table, int n_seqs, const int32_t* q_start,
                    const int32_t* len, const float* rope_cos, const float* rope_sin, int max_pos,
                    const float* q_gain, const float* k_gain, double eps, float* q_out, inv_stream stream) {
  const int rc = inv::check_paged(cache, n_heads);
  if (rc != INV_OK) return rc;
  if (T < 0 || n_seqs < 0 || ld_table < 0 || max_pos <= 0 || !(eps >= 0.0)) return INV_ERR_INVALID_ARG;
  if (ld_qkv < ((int64_t)n_heads + 2 * (int64_t)cache->n_kv_heads) * 128 || ld_qkv % 4 != 0) return INV_ERR_INVALID_ARG;
  if (T == 0 || n_seqs == 0) return INV_OK;
  if (!qkv || !page_table || !q_start || !len || !rope_cos || !rope_sin || !q_out || !cache->k || !cache->v ||
      !cache->k_scale || !cache->v_scale)
    return INV_ERR_INVALID_ARG;
  const uintptr_t low = reinterpret_cast<uintptr_t>(rope_cos) | reinterpret_cast<uintptr_t>(rope_sin) |
                        reinterpret_cast<uintptr_t>(q_gain) | reinterpret_cast<uintptr_t>(k_gain) |
                        reinterpret_cast<uintptr_t>(q_out);
  if ((low & 7u) || !inv::aligned16(qkv) || !inv::aligned16(cache->k) || !inv::aligned16(cache->v))
    return INV_ERR_INVALID_ARG;
  const inv::RaggedBatch rb = {page_table, ld_table, n_seqs, q_start, len};
  kv_append_kernel<<<(unsigned)T + 1u, kAppendThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      qkv, ld_qkv, T, n_heads, inv::paged_view(*cache), rb, rope_cos, rope_sin, max_pos, q_gain, k_gain, eps, q_out,
      inv::status_ptr());
  INV_CHECK_LAUNCH();
  return INV_OK;
}

}  // extern "C"
