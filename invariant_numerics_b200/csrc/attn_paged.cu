// attn_paged: causal attention of ragged chunks of new tokens over a paged
// INT16 KV cache, batch-invariant per row.
//
// Row arithmetic (the same operations, in the same order, whatever kernel,
// tile or split a row is computed in):
//   q_s = q 2^e with max |q_s| in [2^13, 2^14), q_s = q_hi + q_lo in binary16
//            (off by 2^-22 |q_s|, or 2^-25 where q_lo is subnormal: 2^-38 of the row's
//            largest value; the same holds for w below);
//   code / 2 = c_hi + c_lo (unpack_code, exact, c_hi = rn16(code / 2));
//   acc_j  = fp32 tensor-core sum over d in steps of 16: first, per step,
//            c_lo q_hi and c_hi q_lo, then a second round of c_hi q_hi (the
//            small products first, while the accumulator is small);
//   x_j    = acc_j s_K,j;   kappa = (sigma log2 e) 2^(1-e)
//   per block of 128 keys: M' = max(M, max_j x_j), mk = M' kappa,
//            p_j = 2^(x_j kappa - mk), alpha = 2^(mk_old - mk);
//            L_g <- L_g alpha + (sum of p over the 16-key group g: key k and
//            k + 8 first, then a tree over k: k xor 2, xor 4, xor 1)
//            w_j = p_j (s_V,j 2^E), 2^E from the largest s_V of the segment's
//            keys seen so far (brought into [2^13, 2^14)), w = w_hi + w_lo;
//            O  <- O alpha 2^(E - E_old) + sum_j w_j code_j / 2, the sum again
//            cross products first, over keys in steps of 16;
//   segment of 512 keys: o = O 2^(1-E), l = ((L_0 + L_1) + (L_2 + L_3)) +
//            ((L_4 + L_5) + (L_6 + L_7)), m = mk;
//   segments folded in ascending order with the same running maximum.
// A tensor-core product sum depends neither on the other rows or columns of
// its tile nor on whether mma.sync or tcgen05.mma forms it (checked bit for
// bit in the tests), so decode and prefill rows agree exactly.
#include "paged.cuh"

#include <math.h>

#include <algorithm>
#include <type_traits>

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
  int few;          // sequences with at most this many new tokens are the mma.sync kernel's
  int direct;       // rows of the tcgen05 kernel are finished there and have no partials
  int by_seq;       // partials indexed by (sequence, token < few) instead of by row
  int segs;         // segments per CTA of the tcgen05 kernel (split over keys)
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

// (Volatile: loaded where it is used.)
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
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

__device__ __forceinline__ void store_out1(const AttnArgs& a, int64_t idx, float v) {
  a.out[idx] = v;
  if (a.out_hi) {
    __half h, l;
    inv::split_hi_lo(v, h, l);
    if (inv::f16_overflow(v)) record_status(a.status, INV_ERR_RANGE);
    a.out_hi[idx] = h;
    a.out_lo[idx] = l;
  }
}

// One tile of a sequence's new tokens.
struct Tile {
  int seq, tok0, ntok;  // tokens tok0 .. tok0 + ntok - 1 of the sequence's new ones
  int row0;             // the call's row of token tok0
  int len, n_new;
};

// Partial results of (row, head): index of segment 0.
__device__ __forceinline__ int64_t part_index(const AttnArgs& a, int seq, int tok, int row, int head) {
  const int64_t r = a.by_seq ? (int64_t)seq * a.few + tok : row;
  return (r * a.Hq + head) * a.S_max;
}
[[maybe_unused]] __device__ __forceinline__ int64_t part_count(const AttnArgs& a) {
  return (a.by_seq ? (int64_t)a.rb.n_seqs * a.few : (int64_t)a.T) * a.Hq * a.S_max;
}

// Checks sequence i's descriptors; fills everything but the tile's tokens.  The
// mma.sync kernel looks at every sequence of a call and records a wrong q_start;
// the other kernels only skip it (recording it there too cost the tcgen05 kernel
// registers: 276 bytes of spill loads against 208).
template <bool kRecordRows = false>
__device__ __forceinline__ bool load_seq(const AttnArgs& a, int i, int lane, Tile& t) {
  const int q0 = inv::start_of(a.rb, i, a.status), q1 = inv::start_of(a.rb, i + 1, a.status);
  if (kRecordRows && lane == 0 && (q0 < 0 || q1 < q0 || q1 > a.T)) record_status(a.status, INV_ERR_INVALID_ARG);
  if (q0 < 0 || q1 <= q0 || q1 > a.T) return false;
  t.seq = i;
  t.row0 = q0;
  t.n_new = q1 - q0;
  t.len = inv::len_of(a.rb, i, a.status);
  if (t.n_new > a.max_q || t.len < t.n_new || t.len > a.max_len) {
    if (lane == 0) record_status(a.status, INV_ERR_INVALID_ARG);
    return false;
  }
  return true;
}

// Tiles are numbered so that sequence i owns the ids q_start[i] / per + i ..:
// ascending in i and never overlapping (floor((a + n) / per) + 1 - floor(a /
// per) >= ceil(n / per)), without a pass over the batch.  False: no such tile (where
// q_start descends, the search may end at a sequence whose ids begin behind id).
__device__ __forceinline__ bool find_tile(const AttnArgs& a, int id, int per, int lane, Tile& t) {
  const int i = inv::warp_upper(a.rb.n_seqs, id, lane, [&](int j) { return inv::start_of(a.rb, j, a.status) / per + j; });
  if (i < 0 || !load_seq(a, i, lane, t)) return false;
  const int j = id - (t.row0 / per + i);
  if (j < 0 || j > (t.n_new - 1) / per) return false;
  t.tok0 = j * per;
  t.ntok = min(per, t.n_new - t.tok0);
  t.row0 += t.tok0;
  return true;
}

__device__ __forceinline__ bool mbar_poll(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(inv::smem_u32(bar)), "r"(parity), "r"(10000u)
      : "memory");
  return ok != 0;
}
// A wait that took long: true once it is to be given up.
__device__ __forceinline__ bool wait_over(unsigned long long& t0, const AttnArgs& a, volatile int* abort) {
  if (*abort) return true;
  const unsigned long long now = inv::global_ns();
  if (t0 == 0) t0 = now;
  if ((long long)(now - t0) <= a.wait_ns) return false;
  record_status(a.status, INV_ERR_TIMEOUT);
  *abort = 1;
  return true;
}
// mbar_wait by a whole warp (kWarp) or one thread, with polls that let the
// hardware suspend it: the waiting warps share their schedulers with working
// ones.  False once any wait of the CTA gave up.
template <bool kWarp>
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity, const AttnArgs& a, int* abort) {
  unsigned long long t0 = 0;
  for (uint32_t i = 1;; ++i) {
    const bool ok = mbar_poll(bar, parity);
    if (kWarp ? __all_sync(0xffffffffu, ok) : ok) return true;
    if ((i & 63u) == 0) {
      const bool over = wait_over(t0, a, abort);
      if (kWarp ? __any_sync(0xffffffffu, over) : over) return false;
    }
  }
}

// One arrival for the whole warp, behind all its lanes' accesses.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) inv::mbar_arrive(bar);
}

// ------------------------------------------------------- few rows: mma.sync --
//
// Persistent CTAs (two a SM), each taking every gridDim.x-th work item = (sequence
// of at most 32 rows, segment, kv head); a row is a (token, query head of the
// group) pair.  Bound by HBM: 520 bytes a key and kv head.
//   warp 8     producer: reads an item's descriptors and page numbers, brings its
//              scales (bulk copies) and its K and V blocks of 128 keys (2-D TMA,
//              128-byte swizzle, a box per page and half of d) into a ring of two
//              32 KB slots, running ahead of the consumers across items, so that
//              an item starts without waiting for memory (one CTA per item spent
//              a quarter of its time there).
//   warps 0-7  S^T = K Q^T: warp w owns keys 16w .. 16w+15 of the block (the rows
//              of an m-tile), the item's rows are the MMA columns.  O^T = V^T W:
//              warp w owns dims 16w .. 16w+15.  W crosses the warps through shared
//              memory.
// An item is computed by the code for its number of tiles of 8 rows, so a decode row
// in a call with prompts or drafts costs what it costs alone (128 x 2048 keys 235 us;
// with the code of four tiles 527, with its idle tiles skipped at run time 361).
// Measured (32 query, 8 kv heads; replays of a graph of the calls, a call among others
// from Python takes 252 us for the first): 128 sequences of 2048 keys 231 us (4.73 TB/s of
// codes, scales and q; without its products 188), 64 of up to 8192 290 us; 32
// sequences over 4096 keys: 4 tokens 183, 5 tokens 237, 8 tokens 297.  Not HBM but the
// warps bound it: loads from shared memory, unpacking, two barriers a block; from
// three tiles on the MMAs' and the softmax's latency too, at two CTAs a SM.  Four warps
// of two m-tiles (264 us for the first case), half-block slots (278) and one CTA a SM
// with four slots (278) were slower.
// The items go round in their order, empty ones included, which a bound far above the
// lengths makes many of (the first case with a bound of 131072: 615 us).  Where the bound's
// number of segments divides gridDim.x / heads, a CTA meets the same segment in every
// sequence: 37 segments, of which 4 hold keys, 1299 us.
constexpr int MAX_NT = 4;  // tiles of 8 rows of an item
constexpr int FEW_WARPS = 8, FEW_T = 32 * FEW_WARPS;
constexpr int TH = FEW_T + 32;
constexpr int SLOT = BLK * D * 2;  // 32 KB: codes of one block
constexpr int NST = 2;

// B fragments of 8 rows: lane (g, c) of k-step k holds, for row g, the pairs
// (16k + 2c, + 1) and (16k + 2c + 8, + 9).  Eight bytes a lane: with hi and lo side by
// side the second round's loads of hi alone met every bank twice, and the scattered
// stores of W four times; shared memory is what the warps wait for most (128 x 2048
// keys: 250 against 234 us).
struct Frags {
  uint2 hi[8][32], lo[8][32];
};

// A work item; n_keys = 0: no more.
struct Item {
  int seq, row0, n_new, pos0, seg, h, n_keys;
};

struct __align__(1024) FewSmem {
  uint8_t ring[NST * SLOT];
  Frags q[MAX_NT], w[MAX_NT];
  float ks[2][SEG], vs[2][SEG];  // scales of this and the next item (unspecified behind their last key)
  float pm[SEG];                 // running maximum of vs
  float red_m[FEW_WARPS][8 * MAX_NT];
  float red_l[FEW_WARPS][8 * MAX_NT];
  float kappa[8 * MAX_NT];
  int nrow[8 * MAX_NT];  // keys of the row in the segment (may be <= 0)
  Item item[2];
  uint64_t full[NST], empty[NST], item_full[2], item_empty[2];
  int abort;
};

// Shared address of code (key r, dim d0 multiple of 8) of a slot: half d0/64,
// row r of 128 bytes, 16-byte chunk xor (r % 8).
__device__ __forceinline__ uint32_t code_addr(uint32_t base, int r, int d0) {
  return base + (d0 >> 6) * (BLK * 128) + r * 128 + ((((d0 & 63) >> 3) ^ (r & 7)) << 4);
}

// Barrier of the consumer warps; true if `bad` holds for any of their threads.
__device__ __forceinline__ bool few_sync_any(bool bad) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)bad), "n"(FEW_T)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void few_sync() { asm volatile("barrier.cta.sync 1, %0;" ::"n"(FEW_T) : "memory"); }

// kLast: the fold is not launched (no sequence has a second segment); the item's
// results are the rows' outputs.
template <bool kLast>
__global__ void __launch_bounds__(TH, 2)
    attn_few_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const __grid_constant__ AttnArgs a) {
  inv::grid_launch_dependents();  // the fold may be scheduled once every CTA has started
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int G = a.G, Hkv = a.c.n_kv_heads;
  extern __shared__ uint8_t smem_raw[];
  FewSmem& sm = *reinterpret_cast<FewSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  if (tid == 0) {
    for (int i = 0; i < NST; ++i) {
      inv::mbar_init(&sm.full[i], 1);
      inv::mbar_init(&sm.empty[i], FEW_WARPS);
    }
    for (int i = 0; i < 2; ++i) {
      inv::mbar_init(&sm.item_full[i], 1);
      inv::mbar_init(&sm.item_empty[i], FEW_WARPS);
    }
    sm.abort = 0;
    inv::fence_mbar_init();
  }
  __syncthreads();
  bool ok = true;

  if (warp == FEW_WARPS) {
    // =============================================================== producer
    const int sh = a.c.page_shift, ps = 1 << sh, box = min(ps, BLK);
    const int64_t items = (int64_t)a.rb.n_seqs * a.S_max * Hkv;
    uint32_t n_item = 0, n_slot = 0;  // items and blocks sent so far
#pragma unroll 1
    for (int64_t id = blockIdx.x; id < items && ok; id += gridDim.x) {
      Item it;
      it.h = (int)(id % Hkv);
      const int64_t rest = id / Hkv;
      it.seg = (int)(rest % a.S_max);
      Tile t;
      if (!load_seq<true>(a, (int)(rest / a.S_max), lane, t) || t.n_new > a.few || t.n_new * G > 8 * MAX_NT) continue;
      const int key0 = it.seg * SEG;
      it.seq = t.seq;
      it.row0 = t.row0;
      it.n_new = t.n_new;
      it.pos0 = t.len - t.n_new;
      it.n_keys = min(SEG, t.len - key0);
      if (it.n_keys <= 0) continue;
      // lane j: page j of the segment (at most 32), as the cache row of this head's first key; -1: none, or a page
      // outside the cache, whose keys and values count as zero (scales 0, whatever codes lie in the slot)
      const int npg = (it.n_keys + ps - 1) >> sh;
      int row = -1;
      if (lane < npg) {
        const int pg = inv::page_of(a.rb, t.seq, (key0 >> sh) + lane, a.status);
        if (pg < 0 || pg >= a.c.n_pages)
          record_status(a.status, INV_ERR_INVALID_ARG);
        else
          row = (pg * Hkv + it.h) << sh;
      }
      const unsigned pages = __ballot_sync(0xffffffffu, row >= 0);
      const int ab = n_item & 1;
      if (n_item >= 2) ok = bar_wait<true>(&sm.item_empty[ab], ((n_item >> 1) - 1) & 1, a, &sm.abort) && ok;
      if (!ok) break;
      if (lane < npg && row < 0) {
        for (int j = 0; j < ps; ++j) sm.ks[ab][(lane << sh) + j] = sm.vs[ab][(lane << sh) + j] = 0.0f;
        inv::fence_proxy_async_smem();  // before a later item's copies to the same place
      }
      __syncwarp();
      if (lane == 0) {
        sm.item[ab] = it;
        inv::mbar_arrive_expect_tx(&sm.item_full[ab], __popc(pages) * ps * 8);
      }
      __syncwarp();
      if (row >= 0 && INV_SPAN_IN_BOUNDS(a.status, row, row + ps - 1, ((int64_t)a.c.n_pages * Hkv) << sh)) {
        inv::bulk_load(sm.ks[ab] + (lane << sh), a.c.k_scale + row, ps * 4, &sm.item_full[ab]);
        inv::bulk_load(sm.vs[ab] + (lane << sh), a.c.v_scale + row, ps * 4, &sm.item_full[ab]);
      }
      ++n_item;
      const int ops = 2 * ((it.n_keys + BLK - 1) / BLK);  // K, V of every block
#pragma unroll 1
      for (int op = 0; op < ops && ok; ++op) {
        const int s = n_slot % NST;
        if (n_slot >= NST) ok = bar_wait<true>(&sm.empty[s], (n_slot / NST - 1) & 1, a, &sm.abort) && ok;
        if (!ok) break;
        const int kb = (op >> 1) * BLK, nb = (min(BLK, it.n_keys - kb) + box - 1) / box;
        // lane j: box j (keys kb + j box ..): both halves of d
        const int kk = kb + lane * box;
        const int r0 = __shfl_sync(0xffffffffu, row, (kk >> sh) & 31);
        const bool in = lane < nb && r0 >= 0;
        const unsigned boxes = __ballot_sync(0xffffffffu, in);
        if (lane == 0) inv::mbar_arrive_expect_tx(&sm.full[s], __popc(boxes) * box * D * 2);
        __syncwarp();
        if (in) {
          const CUtensorMap* tm = (op & 1) ? &tm_v : &tm_k;
          uint8_t* dst = sm.ring + s * SLOT + lane * box * 128;
          inv::tma_load_2d(dst, tm, &sm.full[s], 0, r0 + (kk & (ps - 1)));
          inv::tma_load_2d(dst + BLK * 128, tm, &sm.full[s], 64, r0 + (kk & (ps - 1)));
        }
        ++n_slot;
      }
    }
    // the end mark; after a wait that gave up, no copy may still be landing when the CTA exits
    const int ab = n_item & 1;
    if (ok && n_item >= 2) ok = bar_wait<true>(&sm.item_empty[ab], ((n_item >> 1) - 1) & 1, a, &sm.abort);
    if (ok) {
      if (lane == 0) {
        sm.item[ab].n_keys = 0;
        inv::mbar_arrive(&sm.item_full[ab]);
      }
    } else if (lane == 0) {
      for (uint32_t i = n_slot > NST ? n_slot - NST : 0; i < n_slot; ++i)
        inv::mbar_wait(&sm.full[i % NST], (i / NST) & 1, a.wait_ns, nullptr, a.status);
      for (uint32_t i = n_item > 2 ? n_item - 2 : 0; i < n_item; ++i)
        inv::mbar_wait(&sm.item_full[i & 1], (i >> 1) & 1, a.wait_ns, nullptr, a.status);
    }
    return;
  }

  // ================================================================ consumers
  // acc[nt] = sum over 16 x 8 codes of the m-tile at `ldsm(k)`: cross products first, then hi hi.  The compiler would
  // keep the first round's fragments for the second, or fetch these early, and spill for it: the second round's loads
  // are volatile (4 tokens 203 -> 175 us).  In the first round only one tile gains by that (238 -> 234 us; more tiles
  // lose up to 20 %).
  const auto product = [&](const Frags* f, auto& acc, auto ldsm) {
    constexpr int N = sizeof(acc) / sizeof(acc[0]);
#pragma unroll
    for (int nt = 0; nt < N; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.0f;
    uint32_t ch[8][4];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t w[4], cl[4];
      ldsm(k, w);
#pragma unroll
      for (int i = 0; i < 4; ++i) inv::unpack_code(w[i], ch[k][i], cl[i]);
#pragma unroll
      for (int nt = 0; nt < N; ++nt) {
        const uint2* ph = &f[nt].hi[k][lane];
        const uint2* pl = &f[nt].lo[k][lane];
        const uint2 bh = N == 1 ? lds64(inv::smem_u32(ph)) : *ph, bl = N == 1 ? lds64(inv::smem_u32(pl)) : *pl;
        mma16816(acc[nt], cl, bh.x, bh.y);
        mma16816(acc[nt], ch[k], bl.x, bl.y);
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
#pragma unroll
      for (int nt = 0; nt < N; ++nt) {
        const uint2 b = lds64(inv::smem_u32(&f[nt].hi[k][lane]));
        mma16816(acc[nt], ch[k], b.x, b.y);
      }
    }
  };
  const uint32_t ring = inv::smem_u32(sm.ring);
  const int kk0 = 16 * warp + g;  // this lane's keys in a block: kk0, kk0 + 8
  uint32_t n_slot = 0;

  // One item with its rows in N tiles of 8 columns; false: a wait gave up.
  const auto run_item = [&](auto tiles, const Item& it, int ab) -> bool {
    constexpr int N = decltype(tiles)::value;
    const int rows = it.n_new * G, key0 = it.seg * SEG, nblk = (it.n_keys + BLK - 1) / BLK;
    const float* ks = sm.ks[ab];
    const float* vs = sm.vs[ab];
    // the rows' q, scaled by 2^e and split; lane holds dims 4 lane .. 4 lane + 3
    float4 qx[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int r = warp + FEW_WARPS * i, tok = r / G;
      qx[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows) {
        const int64_t iq = (int64_t)(it.row0 + tok) * a.ld_q + (int64_t)(it.h * G + r - tok * G) * D;
        if (INV_SPAN_IN_BOUNDS(a.status, iq, iq + D - 1, (int64_t)(a.T - 1) * a.ld_q + (int64_t)a.Hq * D))
          qx[i] = reinterpret_cast<const float4*>(a.q + iq)[lane];
      }
    }
    {
      // running maximum of the V scales: keys 2 tid, 2 tid + 1
      const int j = 2 * tid;
      const float s0 = j < it.n_keys ? vs[j] : 0.0f, s1 = j + 1 < it.n_keys ? vs[j + 1] : 0.0f;
      float up = fmaxf(s0, s1);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float x = __shfl_up_sync(0xffffffffu, up, o);
        if (lane >= o) up = fmaxf(up, x);
      }
      if (lane == 31) sm.red_m[0][warp] = up;  // (before red_m's first use)
      float before = __shfl_up_sync(0xffffffffu, up, 1);
      if (lane == 0) before = 0.0f;
      few_sync();
      for (int w = 0; w < warp; ++w) before = fmaxf(before, sm.red_m[0][w]);
      const float p0 = fmaxf(before, s0);
      *reinterpret_cast<float2*>(sm.pm + j) = make_float2(p0, fmaxf(p0, s1));
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int r = warp + FEW_WARPS * i;
      const float4 x = qx[i];
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
      // dims 4 lane, + 1 and + 2, + 3: k-step lane / 4, pairs c = 2 (lane % 2), + 1 of its half (lane % 4) / 2
      const int k = lane >> 2, at = 4 * (r & 7) + 2 * (lane & 1), word = (lane >> 1) & 1;
      uint32_t* dh = reinterpret_cast<uint32_t*>(&sm.q[r >> 3].hi[k][at]) + word;
      uint32_t* dl = reinterpret_cast<uint32_t*>(&sm.q[r >> 3].lo[k][at]) + word;
      dh[0] = pack_half2(hi[0], hi[1]);
      dh[2] = pack_half2(hi[2], hi[3]);
      dl[0] = pack_half2(lo[0], lo[1]);
      dl[2] = pack_half2(lo[2], lo[3]);
      if (lane == 0) {
        sm.kappa[r] = __fmul_rn(a.sigma_l2, inv::pow2f(1 - e));
        sm.nrow[r] = r < rows ? min(SEG, it.pos0 + r / G + 1 - key0) : 0;
      }
    }
    few_sync();

    // lane r of every warp keeps the state of row r; L and O are per thread: L of rows 2c, 2c + 1 of every n-tile over
    // the warp's keys (the same in all lanes that share c), O of these rows, dims 16 warp + g (+8)
    const int nrow_r = lane < 8 * N ? sm.nrow[lane] : 0;
    const float kap_r = lane < 8 * N ? sm.kappa[lane] : 0.0f;
    float M_r = -INFINITY, mk_r = -INFINITY;
    int E_r = 0;
    float L[N][2], o[N][4];
#pragma unroll
    for (int nt = 0; nt < N; ++nt) {
      L[nt][0] = L[nt][1] = 0.0f;
      o[nt][0] = o[nt][1] = o[nt][2] = o[nt][3] = 0.0f;
    }

    bool gone = false;
#pragma unroll 1
    for (int b = 0; b < nblk; ++b) {
      // ----------------------------------------------------------- scores --
      ok = bar_wait<true>(&sm.full[n_slot % NST], (n_slot / NST) & 1, a, &sm.abort) && ok;
      float x[N][4];  // keys kk0 (+8), rows 2c, 2c + 1
      {
        const uint32_t kb = ring + (n_slot % NST) * SLOT;
        product(sm.q, x, [&](int k, uint32_t (&w)[4]) {
          ldsm_x4(code_addr(kb, 16 * warp + ((lane >> 3) & 1) * 8 + (lane & 7), 16 * k + (lane >> 4) * 8), w);
        });
      }
      inv::fence_proxy_async_smem();  // the slot's reads before the TMA overwrites it
      warp_arrive(&sm.empty[n_slot % NST], lane);
      ++n_slot;
      const int key = b * BLK + kk0;
      const float k0 = ks[key], k1 = ks[key + 8];
#pragma unroll
      for (int nt = 0; nt < N; ++nt) {
        float mx[2];
        const int2 nr = *reinterpret_cast<const int2*>(&sm.nrow[8 * nt + 2 * c]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int nri = i == 0 ? nr.x : nr.y;
          x[nt][i] = key < nri ? __fmul_rn(x[nt][i], k0) : -INFINITY;
          x[nt][2 + i] = key + 8 < nri ? __fmul_rn(x[nt][2 + i], k1) : -INFINITY;
          mx[i] = fmaxf(x[nt][i], x[nt][2 + i]);
          mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 4));
          mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 8));
          mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 16));
        }
        if (g == 0) *reinterpret_cast<float2*>(&sm.red_m[warp][8 * nt + 2 * c]) = make_float2(mx[0], mx[1]);
      }
      if (few_sync_any(!ok)) {  // (also: every warp has read the previous block's W)
        gone = true;
        break;
      }

      // ---------------------------------------------------------- softmax --
      float alpha_r = 1.0f, beta_r = 1.0f;
      {
        const int seen = min(nrow_r, (b + 1) * BLK);
        if (seen > b * BLK) {
          float m = sm.red_m[0][lane < 8 * N ? lane : 0];
#pragma unroll
          for (int w = 1; w < FEW_WARPS; ++w) m = fmaxf(m, sm.red_m[w][lane < 8 * N ? lane : 0]);
          M_r = fmaxf(M_r, m);
          const float mk_old = mk_r;
          const int e_old = E_r;
          mk_r = __fmul_rn(M_r, kap_r);
          E_r = inv::norm_exp(sm.pm[seen - 1]);
          alpha_r = b == 0 ? 0.0f : inv::ex2(__fsub_rn(mk_old, mk_r));
          beta_r = b == 0 ? 0.0f : __fmul_rn(alpha_r, inv::pow2f(max(E_r - e_old, -126)));
        }
      }
      const float v0 = vs[key], v1 = vs[key + 8];
#pragma unroll
      for (int nt = 0; nt < N; ++nt) {
        const float2 kap2 = *reinterpret_cast<const float2*>(&sm.kappa[8 * nt + 2 * c]);
        __half* wh = reinterpret_cast<__half*>(&sm.w[nt].hi[warp][4 * (2 * c) + (g >> 1)]) + (g & 1);
        __half* wl = reinterpret_cast<__half*>(&sm.w[nt].lo[warp][4 * (2 * c) + (g >> 1)]) + (g & 1);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int src = 8 * nt + 2 * c + i;
          const float kap = i == 0 ? kap2.x : kap2.y, mk = __shfl_sync(0xffffffffu, mk_r, src);
          const float sc = inv::pow2f(__shfl_sync(0xffffffffu, E_r, src));
          L[nt][i] = __fmul_rn(L[nt][i], __shfl_sync(0xffffffffu, alpha_r, src));
          // (a key the row does not see has x = -inf: p = 0)
          float p0 = 0.0f, p1 = 0.0f, w0 = 0.0f, w1 = 0.0f;
          if (x[nt][i] != -INFINITY) {
            p0 = inv::ex2(__fmaf_rn(x[nt][i], kap, -mk));
            w0 = __fmul_rn(p0, __fmul_rn(v0, sc));
          }
          if (x[nt][2 + i] != -INFINITY) {
            p1 = inv::ex2(__fmaf_rn(x[nt][2 + i], kap, -mk));
            w1 = __fmul_rn(p1, __fmul_rn(v1, sc));
          }
          __half h0, l0, h1, l1;
          inv::split_plain(w0, h0, l0);
          inv::split_plain(w1, h1, l1);
          wh[16 * i] = h0;  // row 2c + i: lane 4 (2c + i) + g / 2
          wh[16 * i + 2] = h1;
          wl[16 * i] = l0;
          wl[16 * i + 2] = l1;
          float s = __fadd_rn(p0, p1);
          s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, 8));
          s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, 16));
          s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, 4));
          L[nt][i] = __fadd_rn(L[nt][i], s);
        }
      }
      few_sync();

      // ----------------------------------------------------------- values --
      ok = bar_wait<true>(&sm.full[n_slot % NST], (n_slot / NST) & 1, a, &sm.abort) && ok;
      {
        const uint32_t vb = ring + (n_slot % NST) * SLOT;
        product(sm.w, x, [&](int k, uint32_t (&w)[4]) {
          ldsm_x4_t(code_addr(vb, 16 * k + (lane >> 4) * 8 + (lane & 7), 16 * warp + ((lane >> 3) & 1) * 8), w);
        });
#pragma unroll
        for (int nt = 0; nt < N; ++nt) {
            const float b0 = __shfl_sync(0xffffffffu, beta_r, 8 * nt + 2 * c), b1 = __shfl_sync(0xffffffffu, beta_r, 8 * nt + 2 * c + 1);
#pragma unroll
          for (int i = 0; i < 4; ++i) o[nt][i] = __fmaf_rn(o[nt][i], (i & 1) ? b1 : b0, x[nt][i]);
        }
      }
      inv::fence_proxy_async_smem();
      warp_arrive(&sm.empty[n_slot % NST], lane);
      ++n_slot;
    }
    if (gone) return false;

    // ------------------------------------------------------ segment results --
#pragma unroll
    for (int nt = 0; nt < N; ++nt)
      if (g == 0) *reinterpret_cast<float2*>(&sm.red_l[warp][8 * nt + 2 * c]) = make_float2(L[nt][0], L[nt][1]);
    inv::fence_proxy_async_smem();  // the scales' reads before the next copy into their buffer
    warp_arrive(&sm.item_empty[ab], lane);
    few_sync();
#pragma unroll
    for (int nt = 0; nt < N; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 8 * nt + 2 * c + i, tok = r / G, head = it.h * G + (r - tok * G);
        const int E = __shfl_sync(0xffffffffu, E_r, r);
        const float mk = __shfl_sync(0xffffffffu, mk_r, r);
        if (!ok || sm.nrow[r] <= 0) continue;
        const float un = inv::pow2f(1 - E);
        const float y0 = __fmul_rn(o[nt][i], un), y1 = __fmul_rn(o[nt][2 + i], un);
        const float l0 = __fadd_rn(__fadd_rn(sm.red_l[0][r], sm.red_l[1][r]), __fadd_rn(sm.red_l[2][r], sm.red_l[3][r]));
        const float l1 = __fadd_rn(__fadd_rn(sm.red_l[4][r], sm.red_l[5][r]), __fadd_rn(sm.red_l[6][r], sm.red_l[7][r]));
        const float l = __fadd_rn(l0, l1);
        if constexpr (kLast) {
          // the fold of one segment: its factor is 1
          const int64_t io = ((int64_t)(it.row0 + tok) * a.Hq + head) * D + 16 * warp + g;
          if (!INV_SPAN_IN_BOUNDS(a.status, io, io + 8, (int64_t)a.T * a.Hq * D)) continue;
          const float il = __frcp_rn(l);
          store_out1(a, io, __fmul_rn(y0, il));
          store_out1(a, io + 8, __fmul_rn(y1, il));
        } else {
          const int64_t rs = part_index(a, it.seq, tok, it.row0 + tok, head) + it.seg;
          if (!INV_IN_BOUNDS(a.status, rs, part_count(a))) continue;
          float* po = a.part_o + rs * D + 16 * warp + g;
          po[0] = y0;
          po[8] = y1;
          if (warp == 0 && g == 0) a.part_ml[rs] = make_float2(mk, l);
        }
      }
    return true;
  };
#pragma unroll 1
  for (uint32_t n_item = 0;; ++n_item) {
    const int ab = n_item & 1;
    ok = bar_wait<true>(&sm.item_full[ab], (n_item >> 1) & 1, a, &sm.abort) && ok;
    if (few_sync_any(!ok)) break;
    const Item it = sm.item[ab];
    if (it.n_keys == 0) break;
    const int tiles = (it.n_new * G + 7) >> 3;
    bool more;
    if (tiles == 1)
      more = run_item(std::integral_constant<int, 1>{}, it, ab);
    else if (tiles == 2)
      more = run_item(std::integral_constant<int, 2>{}, it, ab);
    else if (tiles == 3)
      more = run_item(std::integral_constant<int, 3>{}, it, ab);
    else
      more = run_item(std::integral_constant<int, MAX_NT>{}, it, ab);
    if (!more) break;
  }
}

// --------------------------------------------------------- many rows: tcgen05 --
//
// One CTA per (tile of 128 rows, kv head, range of segments), 20 warps:
//   warps 0-7   softmax: thread (row, half).  Reads its 64 of the block's 128
//               scores from tensor memory, writes w as binary16 hi and lo over
//               them, and adds the finished block's O (its 64 dims) to the
//               registers that hold the segment's sum.
//   warps 8-15  load codes (16 bytes a thread, one operand ahead in registers),
//               unpack them and store hi and lo as swizzled MMA operands.
//   warp 16     issues the MMAs: S = Q K^T (A = Q in tensor memory, B = K in
//               shared memory, K-major), O = W V (A = W in tensor memory, B =
//               V, MN-major).  Order S(i+1), O(i): the tensor core forms the
//               next scores while the softmax of this block runs.
//   warp 17     stores the blocks' scales, the running maximum of V's, and the
//               page numbers the converters need.
// Tensor memory (512 columns): Q hi | Q lo (64 each), two score blocks (128
// each, W in place of the scores), O (128).
// Each product is three chains of 8 MMAs (hi lo, lo hi, hi hi) of 64 clocks, two
// products a block.  Measured: a prompt of 8192 tokens (32 query, 8 kv heads) 2.24 ms in
// a graph, 2.32 as a call: 245 TFLOP/s of useful products and three times that executed,
// 0.45 of the dense rate.  Two chains of about 8K clocks a block bound it, which overlap each other
// and the MMAs: the softmax warps', and unpacking V with the product behind it.
// 16 softmax warps (2.70 ms), separate converters for K and V (2.43) and folding O
// in before the weights (2.30) were slower.
// The roles' loops are kept rolled and each step is written once: unrolled and
// inlined twice they were 34 KB of instructions a block, more than the SM's
// instruction cache holds, and every step ran four times slower.
constexpr int MANY_ROWS = 128;
constexpr int SOFT_T = 256, CONV_T = 256;
constexpr int MANY_T = SOFT_T + CONV_T + 128;
constexpr int MMA_WARP = (SOFT_T + CONV_T) / 32, SCALE_WARP = MMA_WARP + 1;
// Registers a thread: the CTA starts with MANY_REGS for everyone (launch_many
// checks it), each role then takes or returns some; the sum stays the same.
constexpr int MANY_REGS = 96, SOFT_REGS = 152, CONV_REGS = 56, REST_REGS = 56;
static_assert(SOFT_REGS >= MANY_REGS && CONV_REGS <= MANY_REGS && REST_REGS <= MANY_REGS, "an inc must not lower the count, nor a dec raise it");
static_assert(SOFT_T * SOFT_REGS + CONV_T * CONV_REGS + 128 * REST_REGS <= MANY_T * MANY_REGS, "registers of the CTA");
constexpr int OPER = BLK * D * 2;  // bytes of one binary16 operand (hi or lo) of a block
constexpr uint32_t COL_QH = 0, COL_QL = 64, COL_S = 128, COL_O = 384;
constexpr int PAGE_RING = 16, PAGE_AHEAD = 3;  // blocks of page numbers held, and written ahead of the scales

struct __align__(1024) ManySmem {
  uint8_t k[2 * OPER];  // hi, lo; [d half][key][64], 128-byte swizzle
  uint8_t v[2 * OPER];
  uint64_t o_sum[32 * SOFT_T];  // kDirect: sum over the folded segments, [pair of dims][thread]
  // scales of the last 4 blocks: K; V; V 2^E with the whole block's E; running maximum of V in the segment
  float ks[4][BLK], vs[4][BLK], vs2[4][BLK], pm[4][BLK];
  float2 red[2][2][MANY_ROWS];     // [exchange parity][half][row]: maximum, and L of the segment that ended
  int pages[PAGE_RING][BLK / 16];  // page of every 16 keys (-1: none)
  uint64_t q_full, k_full, k_empty, v_full, v_empty, s_full[2], p_full[2], o_full, o_empty, sc_full[4], sc_empty[4],
      row[4], pg_full[PAGE_RING], done;
  uint32_t tmem;
  int abort;
};
constexpr size_t kManySmem = sizeof(ManySmem) + 1024;
static_assert(kManySmem <= 227 * 1024, "shared memory of one SM");

__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

// MN-major operand, 128-byte swizzle: 8 rows of K x 64 elements are 1024 bytes
// (stride SBO between them along K), 64-element groups of N are LBO apart.
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t smem_addr, uint32_t lbo, uint32_t sbo) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(lbo >> 4) << 16;
  d |= static_cast<uint64_t>(sbo >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

// 32 lanes x 32 consecutive columns.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, "
      "%23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two fp32 values in one 64-bit register: one instruction for both, each lane
// rounded as the scalar operation.
__device__ __forceinline__ uint64_t pk(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpk(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Splits two values into binary16 hi and lo pairs (split_plain of each; the
// difference as x - 1 hi, rounded once).
__device__ __forceinline__ void split2(uint64_t x, uint32_t& hi, uint32_t& lo) {
  const float2 v = unpk(x);
  const __half2 h = __floats2half2_rn(v.x, v.y);
  const float2 f = __half22float2(h);
  const float2 d = unpk(fma2(pk(f.x, f.y), pk(-1.0f, -1.0f), x));
  const __half2 l = __floats2half2_rn(d.x, d.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Largest of mx and the 32 scores at TMEM address `src` times the keys' scales
// (kFull: all of them; else the first nv).
template <bool kFull>
__device__ __forceinline__ float score_max(uint32_t src, const float* ks, int nv, float mx) {
  uint32_t v[32];
  tmem_ld32(src, v);
  inv::tmem_wait_ld();
  const float4* k4 = reinterpret_cast<const float4*>(ks);
  float m1 = -INFINITY;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float4 k = k4[j];
    float2 p = unpk(mul2(pk(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1])), pk(k.x, k.y)));
    float2 q = unpk(mul2(pk(__uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3])), pk(k.z, k.w)));
    if constexpr (!kFull) {
      p.x = 4 * j < nv ? p.x : -INFINITY;
      p.y = 4 * j + 1 < nv ? p.y : -INFINITY;
      q.x = 4 * j + 2 < nv ? q.x : -INFINITY;
      q.y = 4 * j + 3 < nv ? q.y : -INFINITY;
    }
    mx = max3(mx, p.x, p.y);
    m1 = max3(m1, q.x, q.y);
  }
  return fmaxf(mx, m1);
}

// Weights of 32 keys: replaces the scores at `src` by w as binary16, 16 columns
// hi and 16 columns lo, and returns the sums of p of either 16 keys (as the group
// sums of the row arithmetic).  kFull: vs holds the scales times 2^E; else the raw ones, and only
// the first nv keys have a weight.
template <bool kFull>
__device__ __forceinline__ float2 weights(uint32_t src, const float* ks, const float* vs, int nv, float kap, float mk,
                                         float vscale) {
  uint32_t v[32];
  tmem_ld32(src, v);
  inv::tmem_wait_ld();
  const float4* k4 = reinterpret_cast<const float4*>(ks);
  const float4* v4 = reinterpret_cast<const float4*>(vs);
  const uint64_t kap2 = pk(kap, kap), mk2 = pk(-mk, -mk);
  uint64_t s[8];
  uint32_t hi[16], lo[16];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float4 k = k4[j], u = v4[j];
    const uint64_t kk[2] = {pk(k.x, k.y), pk(k.z, k.w)};
    uint64_t uu[2] = {pk(u.x, u.y), pk(u.z, u.w)};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = 4 * j + 2 * i;
      const uint64_t x = mul2(pk(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), kk[i]);
      const float2 y = unpk(fma2(x, kap2, mk2));
      float2 pf = make_float2(inv::ex2(y.x), inv::ex2(y.y));
      if constexpr (!kFull) {
        pf.x = e < nv ? pf.x : 0.0f;
        pf.y = e + 1 < nv ? pf.y : 0.0f;
        uu[i] = mul2(uu[i], pk(vscale, vscale));
      }
      const uint64_t p = pk(pf.x, pf.y);
      const int c = (e >> 4) * 4 + ((e >> 1) & 3);  // keys k, k + 1 of the first 8 of 16, with k + 8, k + 9
      s[c] = (e & 8) == 0 ? p : add2(s[c], p);
      uint64_t w = mul2(p, uu[i]);
      if constexpr (!kFull) {  // (a scale behind the row's keys may overflow)
        const float2 wf = unpk(w);
        w = pk(e < nv ? wf.x : 0.0f, e + 1 < nv ? wf.y : 0.0f);
      }
      split2(w, hi[e >> 1], lo[e >> 1]);
    }
  }
  tmem_st16(src, hi);
  tmem_st16(src + 16, lo);
  const float2 a = unpk(add2(add2(s[0], s[1]), add2(s[2], s[3])));
  const float2 b = unpk(add2(add2(s[4], s[5]), add2(s[6], s[7])));
  return make_float2(__fadd_rn(a.x, a.y), __fadd_rn(b.x, b.y));
}

[[maybe_unused]] __device__ __forceinline__ int64_t cache_rows(const AttnArgs& a) {
  return ((int64_t)a.c.n_pages * a.c.n_kv_heads) << a.c.page_shift;
}

// Row of a cached key in the pages of sequence seq, kv head h; -1 behind the
// last key and for a page outside the cache.
__device__ __forceinline__ int64_t cache_row(const AttnArgs& a, int seq, int h, int key, int last) {
  if (key >= last) return -1;
  const int sh = a.c.page_shift, pg = inv::page_of(a.rb, seq, key >> sh, a.status);
  if (pg < 0 || pg >= a.c.n_pages) {
    record_status(a.status, INV_ERR_INVALID_ARG);
    return -1;
  }
  return (((int64_t)pg * a.c.n_kv_heads + h) << sh) + (key & ((1 << sh) - 1));
}

// One lane of the warp (a branch on it leaves the MMA operands in uniform
// registers; on lane == 0 each MMA took 170 clocks to issue instead of 64).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

template <int kRegs>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

template <bool kDirect>
__global__ void __launch_bounds__(MANY_T, 1) attn_many_kernel(const __grid_constant__ AttnArgs a) {
  inv::grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = a.G, per = MANY_ROWS / G, h = blockIdx.y;
  Tile t;
  // the last tiles of a prompt see the most keys: they start first
  if (!find_tile(a, gridDim.x - 1 - blockIdx.x, per, lane, t) || t.n_new <= a.few) return;
  const int pos0 = t.len - t.n_new + t.tok0, last = pos0 + t.ntok;
  const int b0 = blockIdx.z * a.segs * (SEG / BLK);
  const int b1 = min((last + BLK - 1) / BLK, b0 + a.segs * (SEG / BLK));
  const int n = b1 - b0;
  if (n <= 0) return;

  extern __shared__ uint8_t smem_raw[];
  ManySmem& sm = *reinterpret_cast<ManySmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  if (tid == 0) {
    inv::mbar_init(&sm.q_full, SOFT_T / 32);
    inv::mbar_init(&sm.k_full, CONV_T / 32);
    inv::mbar_init(&sm.v_full, CONV_T / 32);
    inv::mbar_init(&sm.k_empty, 1);
    inv::mbar_init(&sm.v_empty, 1);
    inv::mbar_init(&sm.o_full, 1);
    inv::mbar_init(&sm.o_empty, SOFT_T / 32);
    inv::mbar_init(&sm.done, 1);
    for (int i = 0; i < 2; ++i) {
      inv::mbar_init(&sm.s_full[i], 1);
      inv::mbar_init(&sm.p_full[i], SOFT_T / 32);
    }
    for (int i = 0; i < 4; ++i) {
      inv::mbar_init(&sm.sc_full[i], 1);
      inv::mbar_init(&sm.sc_empty[i], SOFT_T / 32);
      inv::mbar_init(&sm.row[i], 2);
    }
    for (int i = 0; i < PAGE_RING; ++i) inv::mbar_init(&sm.pg_full[i], 1);
    sm.abort = 0;
    inv::fence_mbar_init();
  }
  if (warp == MMA_WARP) {
    inv::tmem_alloc(&sm.tmem, 512);
    inv::tmem_relinquish();
  }
  inv::tc_fence_before();
  __syncthreads();
  inv::tc_fence_after();
  const uint32_t tm = sm.tmem;
  bool ok = true;

  if (warp < SOFT_T / 32) {
    // ================================================================ softmax
    regs_inc<SOFT_REGS>();
    const int hf = warp >> 2, r = (warp & 3) * 32 + lane;  // half of the keys and dims, row
    const int tok = r / G, head = h * G + (r - tok * G);
    const bool valid = tok < t.ntok && tok < per;
    const int nrow = valid ? pos0 + tok + 1 : 0;  // keys the row sees
    const uint32_t lanes = tm + ((uint32_t)(warp & 3) << 21);
    float kap;
    {
      float4 x[16];
      float m = 0.0f;
      const int64_t iq = (int64_t)(t.row0 + tok) * a.ld_q + (int64_t)head * D + hf * 64;
      const bool in = valid && INV_SPAN_IN_BOUNDS(a.status, iq, iq + 63, (int64_t)(a.T - 1) * a.ld_q + (int64_t)a.Hq * D);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        x[j] = in ? reinterpret_cast<const float4*>(a.q + iq)[j] : make_float4(0.f, 0.f, 0.f, 0.f);
        m = fmaxf(m, fmaxf(fmaxf(fabsf(x[j].x), fabsf(x[j].y)), fmaxf(fabsf(x[j].z), fabsf(x[j].w))));
      }
      sm.red[0][hf][r].x = m;
      asm volatile("barrier.cta.sync 1, %0;" ::"n"(SOFT_T) : "memory");
      m = fmaxf(m, sm.red[0][hf ^ 1][r].x);
      asm volatile("barrier.cta.sync 1, %0;" ::"n"(SOFT_T) : "memory");
      __syncwarp();  // the tensor memory accesses below are the whole warp's, as all of them
      const int e = inv::norm_exp(m);
      const float f = inv::pow2f(e);
      kap = __fmul_rn(a.sigma_l2, inv::pow2f(1 - e));
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float4 y = x[8 * c + j];
          split2(mul2(pk(y.x, y.y), pk(f, f)), hi[2 * j], lo[2 * j]);
          split2(mul2(pk(y.z, y.w), pk(f, f)), hi[2 * j + 1], lo[2 * j + 1]);
        }
        tmem_st16(lanes + COL_QH + hf * 32 + c * 16, hi);
        tmem_st16(lanes + COL_QL + hf * 32 + c * 16, lo);
      }
      tmem_wait_st();
      inv::tc_fence_before();
      warp_arrive(&sm.q_full, lane);
    }

    if constexpr (kDirect) {
#pragma unroll 1
      for (int j = 0; j < 32; ++j) sm.o_sum[j * SOFT_T + tid] = 0;
    }
    uint64_t O[32];  // the segment's sum, dims 64 hf + 2j, + 1
#pragma unroll
    for (int j = 0; j < 32; ++j) O[j] = 0;
    float M = -INFINITY, mk = -INFINITY;
    float L[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // of the half's 16-key groups
    int E = 0;
    float Mt = -INFINITY, Lt = 0.0f;  // kDirect: folded segments
    float beta = 0.0f;                // of the block whose O is still to be added
    bool add = false;                 // that block has keys of the warp's rows
    uint32_t exch = 0;                // exchanges so far

    // step i: the softmax of block i, then the O of block i - 1, formed meanwhile
#pragma unroll 1
    for (int i = 0; i <= n && ok; ++i) {
      const int b = b0 + i, sl = i & 3;
      const bool first = (b & (SEG / BLK - 1)) == 0, on = i < n;
      const bool ends = i > 0 && (first || !on);  // block i - 1 is the last one of its segment
      const uint32_t sc = lanes + COL_S + (i & 1) * 128 + hf * 64;
      const int nv = nrow - b * BLK - hf * 64;  // visible keys among this thread's 64 (may be <= 0 or > 64)
      const bool row_on = on && nrow > b * BLK;
      const bool any = __any_sync(0xffffffffu, row_on);
      const bool full = on && __all_sync(0xffffffffu, nrow >= (b + 1) * BLK);
      const float* ks = sm.ks[sl] + hf * 64;
      float mx = -INFINITY;
      if (on) {
        ok = bar_wait<true>(&sm.sc_full[sl], (i >> 2) & 1, a, &sm.abort) && ok;
        ok = bar_wait<true>(&sm.s_full[i & 1], (i >> 1) & 1, a, &sm.abort) && ok;
        inv::tc_fence_after();
        if (full) {
#pragma unroll 1
          for (int c = 0; c < 64; c += 32) mx = score_max<true>(sc + c, ks + c, 32, mx);
        } else if (any) {
#pragma unroll 1
          for (int c = 0; c < 64; c += 32) mx = score_max<false>(sc + c, ks + c, nv - c, mx);
        }
      }
      // the row's other half: its maximum, and the L of the segment that ended
      const float mk_s = mk;
      const int E_s = E;
      float l_s = 0.0f;
      if (any || ends) {
        const float lh = __fadd_rn(__fadd_rn(L[0], L[1]), __fadd_rn(L[2], L[3]));
        sm.red[exch & 1][hf][r] = make_float2(mx, lh);
        warp_arrive(&sm.row[warp & 3], lane);
        ok = bar_wait<true>(&sm.row[warp & 3], exch & 1, a, &sm.abort) && ok;
        const float2 other = sm.red[exch & 1][hf ^ 1][r];
        ++exch;
        mx = fmaxf(mx, other.x);
        l_s = __fadd_rn(lh, other.y);
      }
      float beta_n = 1.0f;
      if (on) {
        if (first) {
          M = -INFINITY;
          L[0] = L[1] = L[2] = L[3] = 0.0f;
        }
        if (row_on) {
          M = fmaxf(M, mx);
          mk = __fmul_rn(M, kap);
          E = inv::norm_exp(sm.pm[sl][min(BLK, nrow - b * BLK) - 1]);
          const float alpha = first ? 0.0f : inv::ex2(__fsub_rn(mk_s, mk));
          beta_n = first ? 0.0f : __fmul_rn(alpha, inv::pow2f(max(E - E_s, -126)));
#pragma unroll
          for (int j = 0; j < 4; ++j) L[j] = __fmul_rn(L[j], alpha);
        }
        __syncwarp();
        float2 g = make_float2(0.0f, 0.0f);
        if (full) {
#pragma unroll 1
          for (int c = 0; c < 64; c += 32) {
            if (c != 0) {
              L[0] = __fadd_rn(L[0], g.x);
              L[1] = __fadd_rn(L[1], g.y);
            }
            g = weights<true>(sc + c, ks + c, sm.vs2[sl] + hf * 64 + c, 32, kap, mk, 1.0f);
          }
        } else if (any) {
          const float vscale = inv::pow2f(E);
#pragma unroll 1
          for (int c = 0; c < 64; c += 32) {
            if (c != 0) {
              L[0] = __fadd_rn(L[0], g.x);
              L[1] = __fadd_rn(L[1], g.y);
            }
            g = weights<false>(sc + c, ks + c, sm.vs[sl] + hf * 64 + c, nv - c, kap, mk, vscale);
          }
        }
        L[2] = __fadd_rn(L[2], g.x);
        L[3] = __fadd_rn(L[3], g.y);
        tmem_wait_st();
        inv::tc_fence_before();
        warp_arrive(&sm.p_full[i & 1], lane);
        if (lane == 0) inv::mbar_arrive(&sm.sc_empty[sl]);
      }
      if (i > 0) {
        ok = bar_wait<true>(&sm.o_full, (i - 1) & 1, a, &sm.abort) && ok;
        inv::tc_fence_after();
        if (add) {  // (a row without keys in the block has weights 0 and beta 1)
          const uint64_t b2 = pk(beta, beta);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t v[32];
            tmem_ld32(lanes + COL_O + hf * 64 + c * 32, v);
            inv::tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j)
              O[16 * c + j] = fma2(O[16 * c + j], b2, pk(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])));
          }
        }
        inv::tc_fence_before();
        warp_arrive(&sm.o_empty, lane);
        if (ends) {  // passes the segment on
          const int seg = (b - 1) / (SEG / BLK);
          if (ok && nrow > seg * SEG) {
            const float un = inv::pow2f(1 - E_s);
            const uint64_t un2 = pk(un, un);
            if constexpr (kDirect) {
              const float Mn = fmaxf(Mt, mk_s);
              const float fa = seg == 0 ? 0.0f : inv::ex2(__fsub_rn(Mt, Mn)), fb = inv::ex2(__fsub_rn(mk_s, Mn));
              Mt = Mn;
              Lt = __fmaf_rn(Lt, fa, __fmul_rn(l_s, fb));
              const uint64_t fa2 = pk(fa, fa), fb2 = pk(fb, fb);
              uint64_t* p = sm.o_sum + tid;
#pragma unroll
              for (int j = 0; j < 32; ++j)
                p[j * SOFT_T] = fma2(p[j * SOFT_T], fa2, mul2(mul2(O[j], un2), fb2));
            } else {
              const int64_t rs = part_index(a, t.seq, t.tok0 + tok, t.row0 + tok, head) + seg;
              if (INV_IN_BOUNDS(a.status, rs, part_count(a))) {
                float4* po = reinterpret_cast<float4*>(a.part_o + rs * D + hf * 64);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                  const float2 x = unpk(mul2(O[2 * j], un2)), y = unpk(mul2(O[2 * j + 1], un2));
                  po[j] = make_float4(x.x, x.y, y.x, y.y);
                }
                if (hf == 0) a.part_ml[rs] = make_float2(mk_s, l_s);
              }
            }
          }
        }  // (the next segment's first block has beta 0)
      }
      beta = beta_n;
      add = any;
    }
    if constexpr (kDirect) {
      if (ok && nrow > 0) {
        const float il = __frcp_rn(Lt);
        const int64_t io = ((int64_t)(t.row0 + tok) * a.Hq + head) * D + hf * 64;
        if (INV_SPAN_IN_BOUNDS(a.status, io, io + 63, (int64_t)a.T * a.Hq * D)) {
          for (int j = 0; j < 16; ++j) {
            const uint64_t* p = sm.o_sum + 2 * j * SOFT_T + tid;
            const float2 x = unpk(mul2(p[0], pk(il, il))), y = unpk(mul2(p[SOFT_T], pk(il, il)));
            store_out4(a, io + 4 * j, make_float4(x.x, x.y, y.x, y.y));
          }
        }
      }
    }
  } else if (warp < MMA_WARP) {
    // ============================================================= converters
    regs_dec<CONV_REGS>();
    const int ct = tid - SOFT_T, kr = ct >> 4, ch = ct & 15;  // key kr of every 16, dims 8 ch .. 8 ch + 7
    const int Hkv = a.c.n_kv_heads, sh = a.c.page_shift, ps = 1 << sh;
    // half an operand (64 keys from kh on) of block i into registers; 16 keys lie in one page
    const auto load = [&](const int16_t* codes, int i, int kh, uint4 (&x)[4]) {
      const int key0 = (b0 + i) * BLK + kh + kr;
      const int* pages = sm.pages[i % PAGE_RING] + kh / 16;
      const uint4* src = reinterpret_cast<const uint4*>(codes) + ch;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = key0 + 16 * j, pg = pages[j];
        const int row = ((pg * Hkv + h) << sh) + (key & (ps - 1));  // below 2^31 for a page of the cache
        const bool in = pg >= 0 && key < last && INV_IN_BOUNDS(a.status, row, cache_rows(a));
        x[j] = in ? __ldg(src + (int64_t)row * 16) : make_uint4(0, 0, 0, 0);
      }
    };
    const uint32_t dst0 = (ch >> 3) * (BLK * 128) + kr * 128 + (((ch & 7) ^ (kr & 7)) << 4);
    const auto store = [&](uint8_t* dst, const uint4 (&x)[4]) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint4 hi, lo;
        inv::unpack_code(x[j].x, hi.x, lo.x);
        inv::unpack_code(x[j].y, hi.y, lo.y);
        inv::unpack_code(x[j].z, hi.z, lo.z);
        inv::unpack_code(x[j].w, hi.w, lo.w);
        *reinterpret_cast<uint4*>(dst + j * 2048) = hi;  // 16 keys on
        *reinterpret_cast<uint4*>(dst + j * 2048 + OPER) = lo;
      }
    };
    // Operands in the order they can be stored: K 0, then K i+1 (free once S(i) is formed) before V i (free once
    // O(i-1) is formed).  Operand s: K of block i or V of block i.
    const auto operand = [&](int s, bool& is_v) {
      is_v = s > 0 && (!(s & 1) || s == 2 * n - 1);
      return s == 0 ? 0 : (s & 1) ? (s == 2 * n - 1 ? n - 1 : (s + 1) / 2) : s / 2 - 1;
    };
    // half s & 1 of operand s >> 1, with the next half's codes on their way
    uint4 x[4], y[4];
    ok = bar_wait<true>(&sm.pg_full[0], 0, a, &sm.abort) && ok;
    load(a.c.k, 0, 0, x);
    load(a.c.k, 0, 64, y);
#pragma unroll 1
    for (int s = 0; s < 4 * n && ok; ++s) {
      bool is_v, next_v;
      const int i = operand(s >> 1, is_v);
      if ((s & 1) == 0 && i > 0) ok = bar_wait<true>(is_v ? &sm.v_empty : &sm.k_empty, (i - 1) & 1, a, &sm.abort) && ok;
      store((is_v ? sm.v : sm.k) + dst0 + (s & 1) * (64 * 128), x);
      if (s & 1) {
        inv::fence_proxy_async_smem();
        warp_arrive(is_v ? &sm.v_full : &sm.k_full, lane);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = y[j];
      if (s + 2 < 4 * n) {
        const int ni = operand((s + 2) >> 1, next_v);
        if (!next_v && (s & 1) == 0)
          ok = bar_wait<true>(&sm.pg_full[ni % PAGE_RING], (ni / PAGE_RING) & 1, a, &sm.abort) && ok;
        load(next_v ? a.c.v : a.c.k, ni, (s & 1) * 64, y);
      }
    }
  } else {
    regs_dec<REST_REGS>();
    if (warp == SCALE_WARP) {
    // ================================================================= scales
    float carry = 0.0f;  // largest V scale of the segment so far
    // Page numbers of block j, behind the softmax of block j - 7.  A converter warp reads those of block m last for the
    // second half of its V, which it loads after it has passed on K of block m + 1 and before it passes on K of block
    // m + 2.  So the softmax of block m + 2 is behind these reads, that of block m + 1 is not: the slot may hold pages
    // of block j - 9 and older (tests/test_paged_pipeline.py checks the order of all roles).
    const auto put_pages = [&](int j) {
      if (lane < BLK / 16) {
        const int key = (b0 + j) * BLK + 16 * lane;
        int pg = key < last ? inv::page_of(a.rb, t.seq, key >> a.c.page_shift, a.status) : -1;
        if (key < last && (pg < 0 || pg >= a.c.n_pages)) {
          record_status(a.status, INV_ERR_INVALID_ARG);
          pg = -1;
        }
        sm.pages[j % PAGE_RING][lane] = pg;
      }
      warp_arrive(&sm.pg_full[j % PAGE_RING], lane);
    };
    for (int j = 0; j < min(n, PAGE_AHEAD); ++j) put_pages(j);
#pragma unroll 1
    for (int i = 0; i < n && ok; ++i) {
      // keys 4 lane .. 4 lane + 3 of the block (one page)
      float4 kv = make_float4(0.f, 0.f, 0.f, 0.f), vv = kv;
      const int key = (b0 + i) * BLK + 4 * lane, sl = i & 3;
      const int64_t row = cache_row(a, t.seq, h, key, last);
      if (row >= 0 && INV_SPAN_IN_BOUNDS(a.status, row, row + 3, cache_rows(a))) {
        kv = *reinterpret_cast<const float4*>(a.c.k_scale + row);
        vv = *reinterpret_cast<const float4*>(a.c.v_scale + row);
        if (key + 1 >= last) kv.y = vv.y = 0.0f;
        if (key + 2 >= last) kv.z = vv.z = 0.0f;
        if (key + 3 >= last) kv.w = vv.w = 0.0f;
      }
      if (((b0 + i) & (SEG / BLK - 1)) == 0) carry = 0.0f;
      float4 pv;
      pv.x = vv.x;
      pv.y = fmaxf(pv.x, vv.y);
      pv.z = fmaxf(pv.y, vv.z);
      pv.w = fmaxf(pv.z, vv.w);
      float up = pv.w;
#pragma unroll 1
      for (int o = 1; o < 32; o <<= 1) {
        const float x = __shfl_up_sync(0xffffffffu, up, o);
        if (lane >= o) up = fmaxf(up, x);
      }
      float before = __shfl_up_sync(0xffffffffu, up, 1);
      before = fmaxf(lane == 0 ? 0.0f : before, carry);
      carry = fmaxf(carry, __shfl_sync(0xffffffffu, up, 31));
      const float f = inv::pow2f(inv::norm_exp(carry));
      if (i >= 4) ok = bar_wait<true>(&sm.sc_empty[sl], ((i - 4) >> 2) & 1, a, &sm.abort) && ok;
      if (i + PAGE_AHEAD < n) put_pages(i + PAGE_AHEAD);
      reinterpret_cast<float4*>(sm.ks[sl])[lane] = kv;
      reinterpret_cast<float4*>(sm.vs[sl])[lane] = vv;
      reinterpret_cast<float4*>(sm.vs2[sl])[lane] =
          make_float4(__fmul_rn(vv.x, f), __fmul_rn(vv.y, f), __fmul_rn(vv.z, f), __fmul_rn(vv.w, f));
      reinterpret_cast<float4*>(sm.pm[sl])[lane] =
          make_float4(fmaxf(pv.x, before), fmaxf(pv.y, before), fmaxf(pv.z, before), fmaxf(pv.w, before));
      warp_arrive(&sm.sc_full[sl], lane);
    }
    } else if (warp == MMA_WARP && elect_one()) {
    // ==================================================================== MMA
    constexpr uint32_t ID_S = inv::idesc_f16_f32(MANY_ROWS, BLK);
    constexpr uint32_t ID_O = inv::idesc_f16_f32(MANY_ROWS, D) | (1u << 16);  // B is MN-major
    const uint64_t kdesc = inv::sw128_kmajor_desc(inv::smem_u32(sm.k));
    const uint64_t vdesc = sw128_mnmajor_desc(inv::smem_u32(sm.v), BLK * 128, 1024);
    const auto wait = [&](uint64_t* bar, uint32_t parity) {
      ok = ok && bar_wait<false>(bar, parity, a, &sm.abort);
    };
    wait(&sm.q_full, 0);
#pragma unroll 1
    for (int i = 0; i <= n && ok; ++i) {
      if (i < n) {  // scores of block i
        wait(&sm.k_full, i & 1);
        if (!ok) break;
        inv::tc_fence_after();
        const uint32_t d = tm + COL_S + (i & 1) * 128;
        // operands advance by 32 bytes a step of 16 dims, and to the second half of d after 4
#pragma unroll 1
        for (int k = 0; k < 8; ++k) {
          const uint64_t b = kdesc + (k >> 2) * (BLK * 128 >> 4) + (k & 3) * 2;
          umma_ts(d, tm + COL_QH + 8 * k, b + (OPER >> 4), ID_S, k != 0);
          umma_ts(d, tm + COL_QL + 8 * k, b, ID_S, 1);
        }
#pragma unroll 1
        for (int k = 0; k < 8; ++k)
          umma_ts(d, tm + COL_QH + 8 * k, kdesc + (k >> 2) * (BLK * 128 >> 4) + (k & 3) * 2, ID_S, 1);
        inv::umma_commit(&sm.k_empty);
        inv::umma_commit(&sm.s_full[i & 1]);
      }
      if (i > 0) {  // O of block i - 1
        const int j = i - 1;
        wait(&sm.p_full[j & 1], (j >> 1) & 1);
        wait(&sm.v_full, j & 1);
        if (j > 0) wait(&sm.o_empty, (j - 1) & 1);
        if (!ok) break;
        inv::tc_fence_after();
        const uint32_t w0 = tm + COL_S + (j & 1) * 128, d = tm + COL_O;
#pragma unroll 1
        for (int k = 0; k < 8; ++k) {
          const uint32_t w = w0 + (k >> 1) * 32 + (k & 1) * 8;  // hi; lo 16 columns on
          const uint64_t b = vdesc + k * (2048 >> 4);
          umma_ts(d, w, b + (OPER >> 4), ID_O, k != 0);
          umma_ts(d, w + 16, b, ID_O, 1);
        }
#pragma unroll 1
        for (int k = 0; k < 8; ++k) umma_ts(d, w0 + (k >> 1) * 32 + (k & 1) * 8, vdesc + k * (2048 >> 4), ID_O, 1);
        inv::umma_commit(&sm.v_empty);
        inv::umma_commit(&sm.o_full);
      }
    }
    // every MMA has finished before tensor memory is given back
    inv::umma_commit(&sm.done);
    inv::mbar_wait(&sm.done, 0, a.wait_ns, nullptr, a.status);
    }
  }
  __syncwarp();
  inv::tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    inv::tc_fence_after();
    inv::tmem_dealloc(tm, 512);
  }
}

// One warp per (row, head): folds the segments in ascending order.
__global__ void __launch_bounds__(256) attn_fold_kernel(const __grid_constant__ AttnArgs a) {
  inv::grid_wait_prerequisites();
  const int64_t wid = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (wid >= (int64_t)a.T * a.Hq) return;
  const int r = (int)(wid / a.Hq);
  const int i = inv::warp_upper(a.rb.n_seqs, r, lane, [&](int j) { return inv::start_of(a.rb, j, a.status); });
  if (i < 0) return;
  Tile t;
  if (!load_seq(a, i, lane, t) || r < t.row0 || r >= t.row0 + t.n_new) return;
  if (a.direct && t.n_new > a.few) return;  // its rows are finished already
  const int n = t.len - t.n_new + (r - t.row0) + 1, S = (n + SEG - 1) / SEG;
  const int64_t rs = part_index(a, i, r - t.row0, r, (int)(wid - (int64_t)r * a.Hq));
  if (!INV_SPAN_IN_BOUNDS(a.status, rs, rs + S - 1, part_count(a))) return;
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

constexpr int MAX_GRID_YZ = 65535;
constexpr size_t PART_BYTES = D * sizeof(float) + sizeof(float2);  // of one segment's result

// The longest sequence: a position rounded up to a whole segment stays below 2^31.
constexpr int MAX_LEN = 0x7fffffff - (SEG - 1);

int segments(int max_len) { return max_len / SEG + (max_len % SEG != 0); }

// Sequences with at most this many new tokens (32 rows) take the mma.sync kernel: at 32
// sequences over 4096 keys, 5 tokens of 4 heads (20 rows) take it 237 us and the tcgen05
// kernel 391, 8 tokens (32 rows) 297 and 373.
int few_tokens(int G) { return 8 * MAX_NT / G; }
int64_t many_tiles(int T, int n_seqs, int G) { return (int64_t)T / (MANY_ROWS / G) + n_seqs; }

// How a call's work is cut: by its sizes and bounds, the GPU's number of SMs and the
// partial results that the workspace can hold, and without any effect on the bits.
struct Plan {
  bool many;       // some sequence may have more than few_tokens new tokens
  bool direct;     // a CTA of the tcgen05 kernel takes all segments of its tile and folds them
  bool by_seq;     // partial results by (sequence, token) instead of by row: there are fewer of these
  int segs;        // segments per CTA, unless direct
  int64_t parts;   // (row, head) pairs with partial results
};
Plan make_plan(int T, int n_seqs, int Hq, int Hkv, int max_q, int max_len, int64_t room) {
  const int G = Hq / Hkv, S = segments(max_len), few = few_tokens(G);
  // rows of sequences with few tokens: these always need their partial results, unless one segment is all there is
  const int64_t few_rows = std::min<int64_t>(T, (int64_t)n_seqs * few);
  Plan p = {max_q > few, false, few_rows < T, 1, few_rows * Hq};
  if (!p.many) {
    if (S == 1) p.parts = 0;
    return p;
  }
  // Direct from two CTAs a SM on: each reads its rows' q once and writes no partial results.  Also where the split's
  // results do not fit the workspace: a workspace for many tokens, which are direct, serves calls of fewer.
  const int sms = inv::sm_count();
  const int64_t tiles = (int64_t)T / (MANY_ROWS / G);
  p.direct = (tiles + 1) * Hkv >= 2 * sms || S == 1 || (int64_t)T * Hq > room;
  if (p.direct) {
    p.segs = S;
    return p;
  }
  p.by_seq = false;
  p.parts = (int64_t)T * Hq;
  // Split over keys.  In units of one block of 128 keys (4 us) a CTA costs 2 to start and to finish and 4 per
  // segment; n CTAs that do not all fit at once take their sum over the SMs and half a CTA's time at the end.
  // Measured at 32 query and 8 kv heads, 1 / 2 / 4 segments per CTA: 64 tokens over 8192 keys 81 / 72 / 106 us, 512
  // over 8192 462 / 400 / 408, 512 over 32768 1760 / 1531 / 1403, 32 sequences of 9 over 4096 425 / 376 / 392.
  const int64_t ctas = std::max<int64_t>(1, std::max<int64_t>(tiles, std::min(n_seqs, T / (few + 1)))) * Hkv;
  double best = 0.0;
  for (int segs = 1; segs <= 4; segs *= 2) {
    const int64_t n = ctas * ((S + segs - 1) / segs);
    const double one = 2.0 + 4.0 * segs, t = n <= sms ? one : (4.0 * ctas * S + 2.0 * n) / sms + 0.5 * one;
    if (segs == 1 || t < best) best = t, p.segs = segs;
  }
  p.segs = std::max(p.segs, (S + MAX_GRID_YZ - 1) / MAX_GRID_YZ);
  return p;
}

template <bool kLast>
int launch_few(const AttnArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s) {
  static bool done[64] = {};
  constexpr size_t smem = sizeof(FewSmem) + 1024;
  const int rc = allow_smem(attn_few_kernel<kLast>, smem, done);
  if (rc != INV_OK) return rc;
  const int64_t items = (int64_t)a.rb.n_seqs * a.S_max * a.c.n_kv_heads, fit = 2 * inv::sm_count();
  attn_few_kernel<kLast><<<(unsigned)(items < fit ? items : fit), TH, smem, s>>>(tk, tv, a);
  INV_CHECK_LAUNCH();
  return INV_OK;
}

template <bool kDirect>
int launch_many(const AttnArgs& a, cudaStream_t s) {
  static bool done[64] = {};
  static int regs[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return INV_ERR_CUDA;
  const int rc = allow_smem(attn_many_kernel<kDirect>, kManySmem, done);
  if (rc != INV_OK) return rc;
  if (regs[dev] == 0) {
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, attn_many_kernel<kDirect>) != cudaSuccess) return INV_ERR_CUDA;
    regs[dev] = fa.numRegs;
  }
  // the roles' shares add up to what the CTA starts with; with less, a role would wait for registers for good
  if (regs[dev] != MANY_REGS) return INV_ERR_CUDA;
  const dim3 grid((unsigned)many_tiles(a.T, a.rb.n_seqs, a.G), a.c.n_kv_heads, (a.S_max + a.segs - 1) / a.segs);
  attn_many_kernel<kDirect><<<grid, MANY_T, kManySmem, s>>>(a);
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
  if (n_heads % n_kv_heads != 0 || n_heads / n_kv_heads > 16) return 0;
  const Plan p = make_plan(T, n_seqs, n_heads, n_kv_heads, max_q_bound > 0 && max_q_bound < T ? max_q_bound : T,
                           max_len_bound, INT64_MAX);
  return (size_t)p.parts * segments(max_len_bound) * PART_BYTES;
}

int attn_paged(const float* q, int64_t ld_q, int T, int n_heads, const inv_paged_kv_cache* cache,
               const int32_t* page_table, int64_t ld_table, int n_seqs, const int32_t* q_start, const int32_t* len,
               int max_q_bound, int max_len_bound, float softmax_scale, float* out, uint16_t* out_hi, uint16_t* out_lo,
               void* workspace, size_t ws_bytes, inv_stream stream) {
  int rc = inv::check_paged(cache, n_heads);
  if (rc != INV_OK) return rc;
  const int G = n_heads / cache->n_kv_heads;
  if (G > 16 || cache->n_kv_heads > MAX_GRID_YZ) return INV_ERR_UNSUPPORTED_SHAPE;
  if (T < 0 || n_seqs < 0 || ld_table < 0 || ld_q < (int64_t)n_heads * D || ld_q % 4 != 0) return INV_ERR_INVALID_ARG;
  if (!(softmax_scale >= 0.0f) || !(softmax_scale <= 1e30f)) return INV_ERR_INVALID_ARG;
  if ((out_hi == nullptr) != (out_lo == nullptr)) return INV_ERR_INVALID_ARG;
  if (T == 0 || n_seqs == 0) return INV_OK;
  if (ld_table == 0) return INV_ERR_INVALID_ARG;  // no sequence of the call could have a key
  if (!q || !page_table || !q_start || !len || !out || !cache->k || !cache->v || !cache->k_scale || !cache->v_scale)
    return INV_ERR_INVALID_ARG;
  if (!inv::aligned16(q) || !inv::aligned16(out) || !inv::aligned16(cache->k) || !inv::aligned16(cache->v) ||
      !inv::aligned16(cache->k_scale) || !inv::aligned16(cache->v_scale) || !inv::aligned16(workspace) ||
      ((reinterpret_cast<uintptr_t>(out_hi) | reinterpret_cast<uintptr_t>(out_lo)) & 7u))
    return INV_ERR_INVALID_ARG;
  const int64_t room = ld_table > MAX_LEN / cache->page_size ? MAX_LEN : ld_table * cache->page_size;
  AttnArgs a = {};
  a.max_len = max_len_bound > 0 && max_len_bound < room ? max_len_bound : (int)room;
  a.max_q = max_q_bound > 0 && max_q_bound < T ? max_q_bound : T;
  a.S_max = segments(a.max_len);
  const Plan p = make_plan(T, n_seqs, n_heads, cache->n_kv_heads, a.max_q, a.max_len,
                           (int64_t)std::min<uint64_t>(ws_bytes / (PART_BYTES * a.S_max), INT64_MAX));
  if (ws_bytes / (PART_BYTES * a.S_max) < (uint64_t)p.parts) return INV_ERR_WORKSPACE;
  if (p.parts > 0 && !workspace) return INV_ERR_INVALID_ARG;
  a.q = q;
  a.ld_q = ld_q;
  a.T = T;
  a.Hq = n_heads;
  a.G = G;
  a.c = inv::paged_view(*cache);
  a.rb = {page_table, ld_table, n_seqs, q_start, len};
  a.sigma_l2 = (float)((double)softmax_scale * 1.4426950408889634);
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + (size_t)p.parts * a.S_max * D);
  a.few = few_tokens(G);
  a.direct = p.direct;
  a.by_seq = p.by_seq;
  a.segs = p.segs;
  if ((int64_t)n_seqs * a.S_max > 0x7fffffff || many_tiles(T, n_seqs, G) > 0x7fffffff) return INV_ERR_UNSUPPORTED_SHAPE;
  a.out = out;
  a.out_hi = reinterpret_cast<__half*>(out_hi);
  a.out_lo = reinterpret_cast<__half*>(out_lo);
  a.status = inv::status_ptr();
  a.wait_ns = inv::wait_limit_ns();
  const uint64_t cache_rows = (uint64_t)cache->n_pages * cache->n_kv_heads * cache->page_size;
  const uint32_t box = cache->page_size < BLK ? cache->page_size : BLK;
  CUtensorMap tk, tv;
  rc = inv::make_tensor_map_2d(&tk, cache->k, CU_TENSOR_MAP_DATA_TYPE_UINT16, D, cache_rows, 2 * D, 64, box,
                               CU_TENSOR_MAP_SWIZZLE_128B);
  if (rc != INV_OK) return rc;
  rc = inv::make_tensor_map_2d(&tv, cache->v, CU_TENSOR_MAP_DATA_TYPE_UINT16, D, cache_rows, 2 * D, 64, box,
                               CU_TENSOR_MAP_SWIZZLE_128B);
  if (rc != INV_OK) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool last = !p.many && a.S_max == 1;  // no fold
  rc = last ? launch_few<true>(a, tk, tv, s) : launch_few<false>(a, tk, tv, s);
  if (rc == INV_OK && p.many) rc = p.direct ? launch_many<true>(a, s) : launch_many<false>(a, s);
  if (rc != INV_OK) return rc;
  return last ? INV_OK : launch_fold(a, s);
}

}  // extern "C"
