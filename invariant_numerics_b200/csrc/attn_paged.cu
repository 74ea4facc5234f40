// attn_paged: causal attention of ragged chunks of new tokens over a paged
// INT16 KV cache, batch-invariant per row.
//
// Row arithmetic (the same operations, in the same order, whatever kernel,
// tile or split a row is computed in):
//   q_s = q 2^e with max |q_s| in [2^13, 2^14), q_s = q_hi + q_lo in binary16;
//   code / 2 = c_hi + c_lo (unpack_code, exact, c_hi = rn16(code / 2));
//   acc_j  = fp32 tensor-core sum over d in steps of 16: first, per step,
//            c_lo q_hi and c_hi q_lo, then a second round of c_hi q_hi (the
//            small products first, while the accumulator is small);
//   x_j    = acc_j s_K,j;   kappa = (sigma log2 e) 2^(1-e)
//   per block of 128 keys: M' = max(M, max_j x_j), mk = M' kappa,
//            p_j = 2^(x_j kappa - mk), alpha = 2^(mk_old - mk);
//            L_g <- L_g alpha + (sum of p over the 32-key group g)
//            w_j = p_j (s_V,j 2^E), 2^E from the largest s_V of the segment's
//            keys seen so far (brought into [2^13, 2^14)), w = w_hi + w_lo;
//            O  <- O alpha 2^(E - E_old) + sum_j w_j code_j / 2, the sum again
//            cross products first, over keys in steps of 16;
//   segment of 512 keys: o = O 2^(1-E), l = (L_0 + L_1) + (L_2 + L_3), m = mk;
//   segments folded in ascending order with the same running maximum.
// A tensor-core product sum depends neither on the other rows or columns of
// its tile nor on whether mma.sync or tcgen05.mma forms it (checked bit for
// bit in the tests), so decode and prefill rows agree exactly.
#include "paged.cuh"

#include <math.h>

namespace {

using inv::record_status;

constexpr int BLK = INV_PAGED_BLOCK;    // 128 keys: softmax block
constexpr int SEG = INV_PAGED_SEGMENT;  // 512 keys: unit of the split over keys
constexpr int D = INV_HEAD_DIM;

struct AttnArgs {
  const float* q;
  int64_t ld_q;
  int T, Hq, G;
  inv::PagedView c;
  inv::RaggedBatch rb;
  int max_q, max_len, S_max;
  float sigma_l2;   // sigma log2 e
  float* part_o;    // [T][Hq][S_max][128]
  float2* part_ml;  // [T][Hq][S_max]
  float* out;
  __half* out_hi;
  __half* out_lo;
  int* status;
  long long wait_ns;
};

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

__device__ __forceinline__ uint32_t pack_half2(__half lo, __half hi) {
  return (uint32_t)__half_as_ushort(lo) | ((uint32_t)__half_as_ushort(hi) << 16);
}

// Writes one finished output value group of 4 and its binary16 split.
__device__ __forceinline__ void store_out4(const AttnArgs& a, int64_t idx, float4 v) {
  *reinterpret_cast<float4*>(a.out + idx) = v;
  if (a.out_hi) {
    __half h[4], l[4];
    inv::split_hi_lo(v.x, h[0], l[0]);
    inv::split_hi_lo(v.y, h[1], l[1]);
    inv::split_hi_lo(v.z, h[2], l[2]);
    inv::split_hi_lo(v.w, h[3], l[3]);
    if (inv::f16_overflow(v.x) | inv::f16_overflow(v.y) | inv::f16_overflow(v.z) | inv::f16_overflow(v.w))
      record_status(a.status, INV_ERR_RANGE);
    *reinterpret_cast<uint2*>(a.out_hi + idx) = make_uint2(pack_half2(h[0], h[1]), pack_half2(h[2], h[3]));
    *reinterpret_cast<uint2*>(a.out_lo + idx) = make_uint2(pack_half2(l[0], l[1]), pack_half2(l[2], l[3]));
  }
}

// One tile of a sequence's new tokens.
struct Tile {
  int seq, tok0, ntok;  // tokens tok0 .. tok0 + ntok - 1 of the sequence's new ones
  int row0;             // the call's row of token tok0
  int len, n_new;
};

// Tiles are numbered so that sequence i owns the ids q_start[i] / per + i ..:
// ascending in i and never overlapping (floor((a + n) / per) + 1 - floor(a /
// per) >= ceil(n / per)), without a pass over the batch.  False: no such tile.
__device__ __forceinline__ bool find_tile(const AttnArgs& a, int id, int per, int lane, Tile& t) {
  const int i = inv::warp_upper(a.rb.n_seqs, id, lane, [&](int j) { return a.rb.q_start[j] / per + j; });
  if (i < 0) return false;
  const int q0 = a.rb.q_start[i], q1 = a.rb.q_start[i + 1];
  const int tile = id - (q0 / per + i);
  t.seq = i;
  t.n_new = q1 - q0;
  t.tok0 = tile * per;
  if (q0 < 0 || q1 > a.T || t.n_new <= 0 || t.tok0 >= t.n_new) return false;
  t.ntok = min(per, t.n_new - t.tok0);
  t.row0 = q0 + t.tok0;
  t.len = a.rb.len[i];
  if (t.n_new > a.max_q || t.len < t.n_new || t.len > a.max_len) {
    if (lane == 0) record_status(a.status, INV_ERR_INVALID_ARG);
    return false;
  }
  return true;
}

// ------------------------------------------------------- few rows: mma.sync --
//
// One CTA (4 warps) per (tile of up to 8 NT rows, kv head, segment).  A row is
// a (token, query head of the group) pair.  K and V blocks of 128 keys stream
// through a ring of 32 KB slots (2-D TMA, 128-byte swizzle, one box per page
// and half of d).  S^T = K Q^T: warp w owns keys 32w .. 32w+31 of the block
// (rows of two m-tiles), the tile's rows are the MMA columns.  O^T = V^T W:
// warp w owns dims 32w .. 32w+31.  W crosses the warps through shared memory.
constexpr int TH = 128;
constexpr int SLOT = BLK * D * 2;      // 32 KB: codes of one block
constexpr int PSTR = BLK + 8;          // halfs per row of the w and q arrays (conflict-free fragments)

template <int NT, int NST>
struct __align__(1024) FewSmem {
  uint8_t ring[NST * SLOT];
  __half qh[8 * NT * PSTR], ql[8 * NT * PSTR];
  __half wh[8 * NT * PSTR], wl[8 * NT * PSTR];
  float ks[SEG], vs[SEG], pm[SEG];
  float red_m[4][8 * NT];
  float red_l[4][8 * NT];
  float kappa[8 * NT];
  int pages[SEG / 16];
  uint64_t full[NST];
  int abort;
};

// Shared address of code (key r, dim d0 multiple of 8) of a slot: half d0/64,
// row r of 128 bytes, 16-byte chunk xor (r % 8).
__device__ __forceinline__ uint32_t code_addr(uint32_t base, int r, int d0) {
  return base + (d0 >> 6) * (BLK * 128) + r * 128 + ((((d0 & 63) >> 3) ^ (r & 7)) << 4);
}

template <int NT, int NST>
__global__ void __launch_bounds__(TH)
    attn_few_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const __grid_constant__ AttnArgs a) {
  inv::grid_launch_dependents();  // the fold may be scheduled once every CTA has started
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int seg = blockIdx.x % a.S_max, h = blockIdx.y;
  const int G = a.G, per = (8 * NT) / G, Hkv = a.c.n_kv_heads;
  Tile t;
  if (!find_tile(a, blockIdx.x / a.S_max, per, lane, t)) return;
  const int pos0 = t.len - t.n_new + t.tok0;           // position of the tile's first token
  const int key0 = seg * SEG, last = pos0 + t.ntok;    // keys of the tile: 0 .. last - 1
  if (key0 >= last) return;
  const int n_keys = min(SEG, last - key0), nblk = (n_keys + BLK - 1) / BLK;

  extern __shared__ uint8_t smem_raw[];
  using Smem = FewSmem<NT, NST>;
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int sh = a.c.page_shift, ps = 1 << sh;

  if (warp == 0) {
    // page ids of the segment (a segment holds at most 32 pages)
    const int npg = (n_keys + ps - 1) >> sh;
    const int64_t e = (int64_t)(key0 >> sh) + lane;
    int pg = 0;
    if (lane < npg) {
      pg = e < a.rb.ld_table ? a.rb.page_table[t.seq * a.rb.ld_table + e] : -1;
      if (pg < 0 || pg >= a.c.n_pages) {
        record_status(a.status, INV_ERR_INVALID_ARG);
        pg = 0;
      }
    }
    sm.pages[lane] = pg;
    if (lane == 0) {
      for (int i = 0; i < NST; ++i) inv::mbar_init(&sm.full[i], 1);
      sm.abort = 0;
      inv::fence_mbar_init();
    }
  }
  __syncthreads();
  // item 2b = K of block b, 2b + 1 = V of block b; item i lives in slot i % NST
  const int items = 2 * nblk;
  const auto issue = [&](int i) {  // one thread
    const int b = i >> 1, s = i % NST;
    const int kn = min(BLK, n_keys - b * BLK), box = min(ps, BLK), nb = (kn + box - 1) / box;
    inv::mbar_arrive_expect_tx(&sm.full[s], nb * box * D * 2);
    const CUtensorMap* tm = (i & 1) ? &tm_v : &tm_k;
    for (int j = 0; j < nb; ++j) {
      const int kk = key0 + b * BLK + j * box;  // first key of the box
      const int row = (sm.pages[(kk - key0) >> sh] * Hkv + h) * ps + (kk & (ps - 1));
      uint8_t* dst = sm.ring + s * SLOT + j * box * 128;
      inv::tma_load_2d(dst, tm, &sm.full[s], 0, row);
      inv::tma_load_2d(dst + BLK * 128, tm, &sm.full[s], 64, row);
    }
  };
  int issued = 0;
  if (tid == 0)
    for (; issued < NST && issued < items; ++issued) issue(issued);

  // scales of the segment (zero behind its last key), and their running maximum
  {
    float4 kv = make_float4(0.f, 0.f, 0.f, 0.f), vv = kv;
    const int j = 4 * tid;  // keys j .. j+3: one page (page sizes are multiples of 16)
    if (j < n_keys) {
      const int64_t row = ((int64_t)sm.pages[j >> sh] * Hkv + h) * ps + ((key0 + j) & (ps - 1));
      if (INV_SPAN_IN_BOUNDS(a.status, row, row + 3, (int64_t)a.c.n_pages * Hkv * ps)) {
        kv = *reinterpret_cast<const float4*>(a.c.k_scale + row);
        vv = *reinterpret_cast<const float4*>(a.c.v_scale + row);
      }
      if (j + 1 >= n_keys) kv.y = vv.y = 0.0f;
      if (j + 2 >= n_keys) kv.z = vv.z = 0.0f;
      if (j + 3 >= n_keys) kv.w = vv.w = 0.0f;
    }
    *reinterpret_cast<float4*>(sm.ks + j) = kv;
    *reinterpret_cast<float4*>(sm.vs + j) = vv;
    float4 pv;
    pv.x = vv.x;
    pv.y = fmaxf(pv.x, vv.y);
    pv.z = fmaxf(pv.y, vv.z);
    pv.w = fmaxf(pv.z, vv.w);
    float up = pv.w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float x = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up = fmaxf(up, x);
    }
    if (lane == 31) sm.red_m[0][warp] = up;  // (before red_m's first use)
    float before = __shfl_up_sync(0xffffffffu, up, 1);
    if (lane == 0) before = 0.0f;
    __syncthreads();
    for (int w = 0; w < warp; ++w) before = fmaxf(before, sm.red_m[0][w]);
    pv.x = fmaxf(pv.x, before);
    pv.y = fmaxf(pv.y, before);
    pv.z = fmaxf(pv.z, before);
    pv.w = fmaxf(pv.w, before);
    *reinterpret_cast<float4*>(sm.pm + j) = pv;
  }
  // the tile's q rows: scaled by 2^e, split
  for (int r = warp; r < 8 * NT; r += 4) {
    const int tok = r / G, head = r - tok * G;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (tok < t.ntok && tok < per) {
      const int64_t iq = (int64_t)(t.row0 + tok) * a.ld_q + (int64_t)(h * G + head) * D;
      if (INV_SPAN_IN_BOUNDS(a.status, iq, iq + D - 1, (int64_t)(a.T - 1) * a.ld_q + (int64_t)a.Hq * D))
        x = reinterpret_cast<const float4*>(a.q + iq)[lane];
    }
    float m = fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w)));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const int e = inv::norm_exp(m);
    const float f = inv::pow2f(e);
    __half hi[4], lo[4];
    inv::split_plain(__fmul_rn(x.x, f), hi[0], lo[0]);
    inv::split_plain(__fmul_rn(x.y, f), hi[1], lo[1]);
    inv::split_plain(__fmul_rn(x.z, f), hi[2], lo[2]);
    inv::split_plain(__fmul_rn(x.w, f), hi[3], lo[3]);
    *reinterpret_cast<uint2*>(sm.qh + r * PSTR + 4 * lane) = make_uint2(pack_half2(hi[0], hi[1]), pack_half2(hi[2], hi[3]));
    *reinterpret_cast<uint2*>(sm.ql + r * PSTR + 4 * lane) = make_uint2(pack_half2(lo[0], lo[1]), pack_half2(lo[2], lo[3]));
    if (lane == 0) sm.kappa[r] = __fmul_rn(a.sigma_l2, inv::pow2f(1 - e));
  }
  __syncthreads();

  // state of the rows 2c, 2c + 1 of every n-tile (the same in all lanes and warps that share c)
  float kap[NT][2], M[NT][2], mk[NT][2], L[NT][2];
  int E[NT][2], nrow[NT][2];  // nrow: keys of the row in the segment
  float o[NT][2][4];          // O of dims 32 warp + 16 mt + g (+8), rows 2c, 2c + 1
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 8 * nt + 2 * c + i, tok = r / G;
      kap[nt][i] = sm.kappa[r];
      nrow[nt][i] = tok < t.ntok && tok < per ? min(SEG, pos0 + tok + 1 - key0) : 0;
      M[nt][i] = mk[nt][i] = -INFINITY;
      L[nt][i] = 0.0f;
      E[nt][i] = 0;
    }
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) o[nt][mt][0] = o[nt][mt][1] = o[nt][mt][2] = o[nt][mt][3] = 0.0f;
  }

  const auto wait_item = [&](int i) {
    bool ok = true;
    if (lane == 0) ok = inv::mbar_wait(&sm.full[i % NST], (i / NST) & 1, a.wait_ns, &sm.abort, a.status);
    return __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
  };
  const auto refill = [&]() {  // thread 0, after a barrier behind the last reads of the oldest slot
    if (tid == 0 && issued < items && !sm.abort) {
      issue(issued);
      ++issued;
    }
  };
  const uint32_t ring = inv::smem_u32(sm.ring);
  const uint32_t* qh32 = reinterpret_cast<const uint32_t*>(sm.qh);
  const uint32_t* ql32 = reinterpret_cast<const uint32_t*>(sm.ql);
  const uint32_t* wh32 = reinterpret_cast<const uint32_t*>(sm.wh);
  const uint32_t* wl32 = reinterpret_cast<const uint32_t*>(sm.wl);
  bool ok = true;

  for (int b = 0; b < nblk; ++b) {
    // ------------------------------------------------------------- scores --
    ok = wait_item(2 * b) && ok;
    float x[NT][2][4];  // keys 32 warp + 16 mt + g (+8), rows 2c, 2c + 1
    {
      const uint32_t kb = ring + ((2 * b) % NST) * SLOT;
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) x[nt][mt][0] = x[nt][mt][1] = x[nt][mt][2] = x[nt][mt][3] = 0.0f;
        const int lk = 32 * warp + 16 * mt + ((lane >> 3) & 1) * 8 + (lane & 7);
        uint32_t ch[8][4];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          uint32_t w[4], cl[4];
          ldsm_x4(code_addr(kb, lk, 16 * k + (lane >> 4) * 8), w);
#pragma unroll
          for (int i = 0; i < 4; ++i) inv::unpack_code(w[i], ch[k][i], cl[i]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const int w0 = (8 * nt + g) * (PSTR / 2) + 8 * k + c;
            mma16816(x[nt][mt], cl, qh32[w0], qh32[w0 + 4]);
            mma16816(x[nt][mt], ch[k], ql32[w0], ql32[w0 + 4]);
          }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const int w0 = (8 * nt + g) * (PSTR / 2) + 8 * k + c;
            mma16816(x[nt][mt], ch[k], qh32[w0], qh32[w0 + 4]);
          }
        }
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = b * BLK + 32 * warp + 16 * mt + g + 8 * (i >> 1);
          x[nt][mt][i] = key < nrow[nt][i & 1] ? __fmul_rn(x[nt][mt][i], sm.ks[key]) : -INFINITY;
          mx[i & 1] = fmaxf(mx[i & 1], x[nt][mt][i]);
        }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 4));
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 8));
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 16));
      }
      if (g == 0) *reinterpret_cast<float2*>(&sm.red_m[warp][8 * nt + 2 * c]) = make_float2(mx[0], mx[1]);
    }
    inv::fence_proxy_async_smem();  // this thread's K reads before the TMA overwrites the slot
    __syncthreads();
    refill();

    // ------------------------------------------------------------ softmax --
    float beta[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float sc[2], ls[2];
      const float m_old[2] = {mk[nt][0], mk[nt][1]};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 8 * nt + 2 * c + i;
        beta[nt][i] = 1.0f;
        const int seen = min(nrow[nt][i], (b + 1) * BLK);
        if (seen > b * BLK) {
          const float m4 = fmaxf(fmaxf(sm.red_m[0][r], sm.red_m[1][r]), fmaxf(sm.red_m[2][r], sm.red_m[3][r]));
          M[nt][i] = fmaxf(M[nt][i], m4);
          mk[nt][i] = __fmul_rn(M[nt][i], kap[nt][i]);
          const int e_old = E[nt][i];
          E[nt][i] = inv::norm_exp(sm.pm[seen - 1]);
          const float alpha = b == 0 ? 0.0f : inv::ex2(__fsub_rn(m_old[i], mk[nt][i]));
          beta[nt][i] = b == 0 ? 0.0f : __fmul_rn(alpha, inv::pow2f(max(E[nt][i] - e_old, -126)));
          L[nt][i] = __fmul_rn(L[nt][i], alpha);
        }
        sc[i] = inv::pow2f(E[nt][i]);
        ls[i] = 0.0f;
      }
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int rr = i & 1, kk = 32 * warp + 16 * mt + g + 8 * (i >> 1), key = b * BLK + kk;
          float p = 0.0f, w = 0.0f;
          if (key < nrow[nt][rr]) {
            p = inv::ex2(__fmaf_rn(x[nt][mt][i], kap[nt][rr], -mk[nt][rr]));
            w = __fmul_rn(p, __fmul_rn(sm.vs[key], sc[rr]));
          }
          ls[rr] = __fadd_rn(ls[rr], p);
          __half hi, lo;
          inv::split_plain(w, hi, lo);
          sm.wh[(8 * nt + 2 * c + rr) * PSTR + kk] = hi;
          sm.wl[(8 * nt + 2 * c + rr) * PSTR + kk] = lo;
        }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        ls[i] = __fadd_rn(ls[i], __shfl_xor_sync(0xffffffffu, ls[i], 4));
        ls[i] = __fadd_rn(ls[i], __shfl_xor_sync(0xffffffffu, ls[i], 8));
        ls[i] = __fadd_rn(ls[i], __shfl_xor_sync(0xffffffffu, ls[i], 16));
        L[nt][i] = __fadd_rn(L[nt][i], ls[i]);
      }
    }
    __syncthreads();

    // ------------------------------------------------------------- values --
    ok = wait_item(2 * b + 1) && ok;
    {
      const uint32_t vb = ring + ((2 * b + 1) % NST) * SLOT;
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        float acc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.0f;
        uint32_t ch[8][4];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          uint32_t w[4], cl[4];
          ldsm_x4_t(code_addr(vb, 16 * k + (lane >> 4) * 8 + (lane & 7), 32 * warp + 16 * mt + ((lane >> 3) & 1) * 8), w);
#pragma unroll
          for (int i = 0; i < 4; ++i) inv::unpack_code(w[i], ch[k][i], cl[i]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const int w0 = (8 * nt + g) * (PSTR / 2) + 8 * k + c;
            mma16816(acc[nt], cl, wh32[w0], wh32[w0 + 4]);
            mma16816(acc[nt], ch[k], wl32[w0], wl32[w0 + 4]);
          }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const int w0 = (8 * nt + g) * (PSTR / 2) + 8 * k + c;
            mma16816(acc[nt], ch[k], wh32[w0], wh32[w0 + 4]);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (nrow[nt][i & 1] > b * BLK) o[nt][mt][i] = __fmaf_rn(o[nt][mt][i], beta[nt][i & 1], acc[nt][i]);
      }
    }
    inv::fence_proxy_async_smem();  // V reads before the slot is overwritten
    __syncthreads();
    refill();
  }

  // -------------------------------------------------------- segment results --
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
    if (g == 0) *reinterpret_cast<float2*>(&sm.red_l[warp][8 * nt + 2 * c]) = make_float2(L[nt][0], L[nt][1]);
  __syncthreads();
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 8 * nt + 2 * c + i, tok = r / G;
      if (!ok || nrow[nt][i] <= 0) continue;
      const int64_t ro = (int64_t)(t.row0 + tok) * a.Hq + h * G + (r - tok * G);
      const int64_t rs = ro * a.S_max + seg;
      if (!INV_IN_BOUNDS(a.status, rs, (int64_t)a.T * a.Hq * a.S_max)) continue;
      const float un = inv::pow2f(1 - E[nt][i]);
      float* po = a.part_o + rs * D + 32 * warp + g;
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        po[16 * mt] = __fmul_rn(o[nt][mt][i], un);
        po[16 * mt + 8] = __fmul_rn(o[nt][mt][2 + i], un);
      }
      if (warp == 0 && g == 0) {
        const float l = __fadd_rn(__fadd_rn(sm.red_l[0][r], sm.red_l[1][r]), __fadd_rn(sm.red_l[2][r], sm.red_l[3][r]));
        a.part_ml[rs] = make_float2(mk[nt][i], l);
      }
    }
  // no copy may still be landing when the CTA exits (only after a wait gave up)
  if (!ok && tid == 0)
    for (int i = max(0, issued - NST); i < issued; ++i)
      inv::mbar_wait(&sm.full[i % NST], (i / NST) & 1, a.wait_ns, nullptr, a.status);
}

// One warp per (row, head): folds the segments in ascending order.
__global__ void __launch_bounds__(256) attn_fold_kernel(const __grid_constant__ AttnArgs a) {
  inv::grid_wait_prerequisites();
  const int64_t wid = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (wid >= (int64_t)a.T * a.Hq) return;
  const int r = (int)(wid / a.Hq);
  const int i = inv::warp_upper(a.rb.n_seqs, r, lane, [&](int j) { return a.rb.q_start[j]; });
  if (i < 0) return;
  const int q0 = a.rb.q_start[i], q1 = a.rb.q_start[i + 1];
  if (r >= q1 || q0 < 0 || q1 > a.T) return;
  const int n_new = q1 - q0, len = a.rb.len[i];
  if (n_new > a.max_q || len < n_new || len > a.max_len) return;
  const int n = len - (q1 - r) + 1, S = (n + SEG - 1) / SEG;
  const int64_t rs = wid * a.S_max;
  if (!INV_SPAN_IN_BOUNDS(a.status, rs, rs + S - 1, (int64_t)a.T * a.Hq * a.S_max)) return;
  const float4* po = reinterpret_cast<const float4*>(a.part_o + rs * D) + lane;
  float M = -INFINITY, L = 0.0f;
  float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < S; ++s) {
    const float2 ml = a.part_ml[rs + s];
    const float4 v = po[s * 32];
    const float Mn = fmaxf(M, ml.x);
    const float fa = s == 0 ? 0.0f : inv::ex2(__fsub_rn(M, Mn)), fb = inv::ex2(__fsub_rn(ml.x, Mn));
    M = Mn;
    L = __fmaf_rn(L, fa, __fmul_rn(ml.y, fb));
    O.x = __fmaf_rn(O.x, fa, __fmul_rn(v.x, fb));
    O.y = __fmaf_rn(O.y, fa, __fmul_rn(v.y, fb));
    O.z = __fmaf_rn(O.z, fa, __fmul_rn(v.z, fb));
    O.w = __fmaf_rn(O.w, fa, __fmul_rn(v.w, fb));
  }
  const float il = __frcp_rn(L);
  store_out4(a, wid * D + 4 * lane,
             make_float4(__fmul_rn(O.x, il), __fmul_rn(O.y, il), __fmul_rn(O.z, il), __fmul_rn(O.w, il)));
}

template <class F>
int allow_smem(F kernel, size_t bytes, bool (&done)[64]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return INV_ERR_CUDA;
  if (dev >= 0 && dev < 64 && done[dev]) return INV_OK;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess ||
      cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                           (int)cudaSharedmemCarveoutMaxShared) != cudaSuccess)
    return INV_ERR_CUDA;
  if (dev >= 0 && dev < 64) done[dev] = true;
  return INV_OK;
}

int segments(int max_len) { return (max_len + SEG - 1) / SEG; }

template <int NT, int NST>
int launch_few(const AttnArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s) {
  static bool done[64] = {};
  constexpr size_t smem = sizeof(FewSmem<NT, NST>) + 1024;
  const int rc = allow_smem(attn_few_kernel<NT, NST>, smem, done);
  if (rc != INV_OK) return rc;
  const int per = 8 * NT / a.G;
  const int64_t tiles = (int64_t)a.T / per + a.rb.n_seqs;
  if (tiles * a.S_max > 0x7fffffff) return INV_ERR_UNSUPPORTED_SHAPE;
  attn_few_kernel<NT, NST><<<dim3((unsigned)(tiles * a.S_max), a.c.n_kv_heads), TH, smem, s>>>(tk, tv, a);
  INV_CHECK_LAUNCH();
  return INV_OK;
}

int launch_fold(const AttnArgs& a, cudaStream_t s) {
  const int64_t warps = (int64_t)a.T * a.Hq;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)((warps + 7) / 8));
  lc.blockDim = dim3(256);
  lc.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  if (cudaLaunchKernelEx(&lc, attn_fold_kernel, a) != cudaSuccess) return INV_ERR_CUDA;
  INV_CHECK_LAUNCH();
  return INV_OK;
}

}  // namespace

extern "C" {

size_t attn_paged_workspace_size(int T, int n_seqs, int n_heads, int n_kv_heads, int max_q_bound, int max_len_bound) {
  if (T <= 0 || n_seqs <= 0 || n_heads <= 0 || n_kv_heads <= 0 || max_len_bound <= 0) return 0;
  (void)max_q_bound;
  return (size_t)T * n_heads * segments(max_len_bound) * (D * sizeof(float) + sizeof(float2));
}

int attn_paged(const float* q, int64_t ld_q, int T, int n_heads, const inv_paged_kv_cache* cache,
               const int32_t* page_table, int64_t ld_table, int n_seqs, const int32_t* q_start, const int32_t* len,
               int max_q_bound, int max_len_bound, float softmax_scale, float* out, uint16_t* out_hi, uint16_t* out_lo,
               void* workspace, size_t ws_bytes, inv_stream stream) {
  int rc = inv::check_paged(cache, n_heads);
  if (rc != INV_OK) return rc;
  const int G = n_heads / cache->n_kv_heads;
  if (G > 16) return INV_ERR_UNSUPPORTED_SHAPE;
  if (T < 0 || n_seqs < 0 || ld_table < 0 || ld_q < (int64_t)n_heads * D || ld_q % 4 != 0) return INV_ERR_INVALID_ARG;
  if (!(softmax_scale >= 0.0f) || !(softmax_scale <= 1e30f)) return INV_ERR_INVALID_ARG;
  if ((out_hi == nullptr) != (out_lo == nullptr)) return INV_ERR_INVALID_ARG;
  if (T == 0 || n_seqs == 0 || ld_table == 0) return INV_OK;
  if (!q || !page_table || !q_start || !len || !out || !cache->k || !cache->v || !cache->k_scale || !cache->v_scale)
    return INV_ERR_INVALID_ARG;
  if (!inv::aligned16(q) || !inv::aligned16(out) || !inv::aligned16(cache->k) || !inv::aligned16(cache->v) ||
      !inv::aligned16(cache->k_scale) || !inv::aligned16(cache->v_scale) || !inv::aligned16(workspace) ||
      ((reinterpret_cast<uintptr_t>(out_hi) | reinterpret_cast<uintptr_t>(out_lo)) & 7u))
    return INV_ERR_INVALID_ARG;
  const int64_t room = ld_table > 0x7fffffff / cache->page_size ? 0x7fffffff : ld_table * cache->page_size;
  AttnArgs a = {};
  a.max_len = max_len_bound > 0 && max_len_bound < room ? max_len_bound : (int)room;
  a.max_q = max_q_bound > 0 && max_q_bound < T ? max_q_bound : T;
  a.S_max = segments(a.max_len);
  const size_t need = attn_paged_workspace_size(T, n_seqs, n_heads, cache->n_kv_heads, a.max_q, a.max_len);
  if (ws_bytes < need) return INV_ERR_WORKSPACE;
  if (need > 0 && !workspace) return INV_ERR_INVALID_ARG;
  a.q = q;
  a.ld_q = ld_q;
  a.T = T;
  a.Hq = n_heads;
  a.G = G;
  a.c = inv::paged_view(*cache);
  a.rb = {page_table, ld_table, n_seqs, q_start, len};
  a.sigma_l2 = (float)((double)softmax_scale * 1.4426950408889634);
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + (size_t)T * n_heads * a.S_max * D);
  a.out = out;
  a.out_hi = reinterpret_cast<__half*>(out_hi);
  a.out_lo = reinterpret_cast<__half*>(out_lo);
  a.status = inv::status_ptr();
  a.wait_ns = inv::wait_limit_ns();
  const uint64_t rows = (uint64_t)cache->n_pages * cache->n_kv_heads * cache->page_size;
  const uint32_t box = cache->page_size < BLK ? cache->page_size : BLK;
  CUtensorMap tk, tv;
  rc = inv::make_tensor_map_2d(&tk, cache->k, CU_TENSOR_MAP_DATA_TYPE_UINT16, D, rows, 2 * D, 64, box,
                               CU_TENSOR_MAP_SWIZZLE_128B);
  if (rc != INV_OK) return rc;
  rc = inv::make_tensor_map_2d(&tv, cache->v, CU_TENSOR_MAP_DATA_TYPE_UINT16, D, rows, 2 * D, 64, box,
                               CU_TENSOR_MAP_SWIZZLE_128B);
  if (rc != INV_OK) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int rows_tile = a.max_q * G;
  if (rows_tile <= 8)
    rc = launch_few<1, 3>(a, tk, tv, s);
  else if (rows_tile <= 16)
    rc = launch_few<2, 3>(a, tk, tv, s);
  else
    rc = launch_few<4, 3>(a, tk, tv, s);
  if (rc != INV_OK) return rc;
  return launch_fold(a, s);
}

}  // extern "C"
