// softmax_rows and spec_verify: from logits to the tokens of a verification
// step of speculative decoding.
#include "common.cuh"

namespace {

using inv::record_status;

// ------------------------------------------------------------- clusters ----
//
// A row is split over the CTAs of a cluster, each keeping its part in registers,
// so that the row is read once; the parts' results cross by stores into the
// other CTAs' shared memory and one cluster barrier.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// (Without .aligned: a warp may reach them with its threads apart.)
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// Stores 8 bytes at this CTA's shared address p, in the CTA of rank r.
__device__ __forceinline__ void store_cluster(void* p, uint32_t r, uint64_t v) {
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(inv::smem_u32(p)), "r"(r));
  asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(remote), "l"(v) : "memory");
}

constexpr int kMaxCluster = 8;
constexpr int kMaxDraft = 1 << 30;  // counters a block beyond it stay below 2^31

// The larger value; NaN if either is one.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Elements i .. i+3 of a row of n; kVec: 16-byte aligned.
template <bool kVec>
__device__ __forceinline__ float4 load4(const float* p, int i, int n, float none) {
  if (kVec && i + 3 < n) return *reinterpret_cast<const float4*>(p + i);
  float4 v;
  v.x = i < n ? p[i] : none;
  v.y = i + 1 < n ? p[i + 1] : none;
  v.z = i + 2 < n ? p[i + 2] : none;
  v.w = i + 3 < n ? p[i + 3] : none;
  return v;
}
// ----------------------------------------------------------- softmax_rows ----
//
// HBM bound: 8 bytes an element.  Part c of a row (32 THR elements; thread t owns
// every THR-th one from t on: coalesced for any row stride): m_c, s_c = sum exp((x -
// m_c) t); the row: M = max m_c, S = sum_c s_c exp((m_c - M) t) in ascending c; y =
// exp((x - m_c) t) (exp((m_c - M) t) / S).  The maxima keep NaN, so a row with one is
// NaN throughout, wherever it stands.  THR and the number of parts follow from n
// alone, so the order of the sum does too.  21 us for 320 rows of 32000 (3.9 TB/s of
// data that partly stays in L2; one CTA a row that read it again for the sum took 44 us),
// 5 us for 3 rows of 32003: launch, cluster barrier and two trips to memory.
constexpr int kSoftVals = 32;  // elements a thread

template <int THR>
__device__ __forceinline__ float block_max(float m, float* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) red[warp] = m;
  __syncthreads();
  m = red[lane & (THR / 32 - 1)];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}
template <int THR>
__device__ __forceinline__ float block_sum(float s, float* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, o));
  if (lane == 0) red[warp] = s;
  __syncthreads();
  s = lane < THR / 32 ? red[lane] : 0.0f;
#pragma unroll
  for (int o = THR / 64; o > 0; o >>= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, o));
  return s;  // valid in lane 0 of every warp
}

template <int THR>
__global__ void __launch_bounds__(THR, THR == 256 ? 5 : 1024 / THR)
    softmax_kernel(const float* x, int rows, int n, int64_t ld, float it, float* y, int64_t ld_y, int* status) {
  __shared__ float red_m[32], red_s[32];
  __shared__ uint64_t parts[kMaxCluster];  // (m_c, s_c)
  const uint32_t rank = cluster_rank(), parts_n = cluster_size();
  cluster_arrive();  // (every CTA of the cluster runs before another stores into it)
  const int64_t r = blockIdx.x / parts_n;
  const bool in = INV_SPAN_IN_BOUNDS(status, r * ld, r * ld + n - 1, (int64_t)(rows - 1) * ld + n) &&
                  INV_SPAN_IN_BOUNDS(status, r * ld_y, r * ld_y + n - 1, (int64_t)(rows - 1) * ld_y + n);
  const int first = (int)rank * (THR * kSoftVals) + (int)threadIdx.x, left = in ? n - first : 0;  // elements from `first` on
  const float* xr = x + r * ld + first;
  float v[kSoftVals];
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < kSoftVals; ++j) v[j] = j * THR < left ? xr[j * THR] : -INFINITY;
#pragma unroll
  for (int j = 0; j < kSoftVals; ++j) m = max_nan(m, v[j]);
  m = block_max<THR>(m, red_m);
  const bool none = m == -INFINITY;  // nothing but -inf in this part
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int j = 0; j < kSoftVals; ++j) {
    v[j] = none ? 0.0f : expf(__fmul_rn(__fsub_rn(v[j], m), it));
    s[j & 3] = __fadd_rn(s[j & 3], v[j]);
  }
  const float sc = block_sum<THR>(__fadd_rn(__fadd_rn(s[0], s[1]), __fadd_rn(s[2], s[3])), red_s);
  cluster_wait();
  if (threadIdx.x < parts_n) {  // (lane 0's sum goes to every CTA)
    const float s0 = __shfl_sync((1u << parts_n) - 1u, sc, 0);
    store_cluster(&parts[rank], threadIdx.x, ((uint64_t)__float_as_uint(s0) << 32) | __float_as_uint(m));
  }
  __syncwarp();
  cluster_arrive();
  cluster_wait();
  float M = -INFINITY, S = 0.0f;
  for (uint32_t q = 0; q < parts_n; ++q) M = max_nan(M, __uint_as_float((uint32_t)parts[q]));
  for (uint32_t q = 0; q < parts_n; ++q) {
    const float mq = __uint_as_float((uint32_t)parts[q]), sq = __uint_as_float((uint32_t)(parts[q] >> 32));
    if (mq != -INFINITY) S = __fadd_rn(S, __fmul_rn(sq, expf(__fmul_rn(__fsub_rn(mq, M), it))));
  }
  // (a part without weight in a row with NaN: 0 NaN)
  const float f = M == -INFINITY ? 0.0f : __fmul_rn(expf(__fmul_rn(__fsub_rn(m, M), it)), __frcp_rn(S));
  float* yr = y + r * ld_y + first;
#pragma unroll
  for (int j = 0; j < kSoftVals; ++j)
    if (j * THR < left) yr[j * THR] = __fmul_rn(v[j], f);
}

// Rows longer than eight parts: one CTA a row, which reads it three times (indexes are unsigned: the last step of a
// row next to 2^31 ends behind it).
constexpr int kLongThreads = 1024;
__global__ void __launch_bounds__(kLongThreads)
    softmax_long_kernel(const float* x, int rows, int n, int64_t ld, float it, float* y, int64_t ld_y, int* status) {
  __shared__ float red_m[32], red_s[32];
  __shared__ float total;
  const int64_t r = blockIdx.x;
  if (!INV_SPAN_IN_BOUNDS(status, r * ld, r * ld + n - 1, (int64_t)(rows - 1) * ld + n) ||
      !INV_SPAN_IN_BOUNDS(status, r * ld_y, r * ld_y + n - 1, (int64_t)(rows - 1) * ld_y + n))
    return;
  const float* xr = x + r * ld;
  float* yr = y + r * ld_y;
  float m = -INFINITY;
  for (unsigned i = threadIdx.x; i < (unsigned)n; i += kLongThreads) m = max_nan(m, xr[i]);
  m = block_max<kLongThreads>(m, red_m);
  const bool none = m == -INFINITY;
  float s = 0.0f;
  for (unsigned i = threadIdx.x; i < (unsigned)n; i += kLongThreads)
    s = __fadd_rn(s, none ? 0.0f : expf(__fmul_rn(__fsub_rn(xr[i], m), it)));
  s = block_sum<kLongThreads>(s, red_s);
  if (threadIdx.x == 0) total = s;
  __syncthreads();
  const float f = none ? 0.0f : __frcp_rn(total);
  for (unsigned i = threadIdx.x; i < (unsigned)n; i += kLongThreads)
    yr[i] = none ? 0.0f : __fmul_rn(expf(__fmul_rn(__fsub_rn(xr[i], m), it)), f);
}

// ------------------------------------------------------------ spec_verify ----

struct VerifyArgs {
  const float* target;
  int64_t ld_t;
  const float* draft;
  int64_t ld_d;
  int B, max_draft, vocab;
  const int32_t* draft_tokens;
  const int32_t* n_draft;
  const float* u_accept;
  const float* u_sample;
  int32_t* tokens;
  int32_t* n_accepted;
};
// Elements of the buffers, for the index-checking build.
[[maybe_unused]] __device__ __forceinline__ int64_t target_count(const VerifyArgs& a) {
  return ((int64_t)a.B * (a.max_draft + 1) - 1) * a.ld_t + a.vocab;
}
[[maybe_unused]] __device__ __forceinline__ int64_t draft_count(const VerifyArgs& a) {
  return ((int64_t)a.B * a.max_draft - 1) * a.ld_d + a.vocab;
}

// The accepted prefix of sequence b, by one warp, 32 drafts a step: k, or -1 for
// descriptors out of range; m = number of drafts.
__device__ __forceinline__ int accepted_prefix(const VerifyArgs& a, int b, int lane, int& m, int* status, bool record) {
  const int D = a.max_draft, V = a.vocab;
  m = a.n_draft && INV_IN_BOUNDS(status, b, a.B) ? a.n_draft[b] : D;
  bool bad = m < 0 || m > D;
  int k = bad ? -1 : m;
  for (int i0 = 0; !bad && i0 < m; i0 += 32) {
    const int i = i0 + lane;
    bool ok = true, wrong = false;
    const int64_t id = (int64_t)b * D + i;
    if (i < m && INV_IN_BOUNDS(status, id, (int64_t)a.B * D)) {
      const int t = a.draft_tokens[id];
      wrong = t < 0 || t >= V;
      const int64_t ip = ((int64_t)b * (D + 1) + i) * a.ld_t + t, iq = id * a.ld_d + t;
      if (!wrong && INV_IN_BOUNDS(status, ip, target_count(a)) &&
          (!a.draft || INV_IN_BOUNDS(status, iq, draft_count(a)))) {
        const double q = a.draft ? (double)a.draft[iq] : 1.0;
        ok = (double)a.u_accept[id] * q < (double)a.target[ip];
      }
    }
    bad = __any_sync(0xffffffffu, wrong);
    const unsigned no = __ballot_sync(0xffffffffu, !ok);
    if (no != 0 && k == m) k = i0 + __ffs(no) - 1;
  }
  if (bad && record && lane == 0) record_status(status, INV_ERR_INVALID_ARG);
  return bad ? -1 : k;
}

// Everything of the outputs but the next token.
__device__ __forceinline__ void write_prefix(const VerifyArgs& a, int b, int k, [[maybe_unused]] int* status) {
  const int D = a.max_draft;
  const int64_t id = (int64_t)b * D, io = (int64_t)b * (D + 1);
  if (!INV_SPAN_IN_BOUNDS(status, io, io + D, (int64_t)a.B * (D + 1)) || !INV_IN_BOUNDS(status, b, a.B)) return;
  for (int i = threadIdx.x; i <= D; i += blockDim.x)
    if (i != k) a.tokens[io + i] = i < k ? a.draft_tokens[id + i] : -1;
  if (threadIdx.x == 0) a.n_accepted[b] = k < 0 ? 0 : k;
}

// True if rows p_k and q_k of sequence b and its next token lie in their buffers
// (always, except in the index-checking build).
__device__ __forceinline__ bool rows_in_bounds([[maybe_unused]] const VerifyArgs& a, [[maybe_unused]] int b,
                                               [[maybe_unused]] int k, [[maybe_unused]] int m,
                                               [[maybe_unused]] int* status) {
  [[maybe_unused]] const int64_t ip = (int64_t)b * (a.max_draft + 1) + k, iq = (int64_t)b * a.max_draft + k;
  return INV_IN_BOUNDS(status, ip, (int64_t)a.B * (a.max_draft + 1)) &&
         INV_SPAN_IN_BOUNDS(status, ip * a.ld_t, ip * a.ld_t + a.vocab - 1, target_count(a)) &&
         (k >= m || !a.draft || INV_SPAN_IN_BOUNDS(status, iq * a.ld_d, iq * a.ld_d + a.vocab - 1, draft_count(a)));
}

__device__ __forceinline__ double weight(float p, float q) { return p > q ? (double)p - (double)q : 0.0; }

// One cluster per sequence; CTA c owns 16 THR entries of the row, warp w of it a
// run of 512, lane l the entries 4l .. 4l+3 of every 128: 16 in registers.  The
// first dependent reads decide k, then the rows p_k and q_k are read once.  Sums in
// 64 bits: lane, warp, CTA, cluster totals tell which CTA, then which warp and which
// 128 entries the draw falls into; a scan of their lanes ends the search.
// Latency bound (four dependent reads); 8 bytes a vocabulary entry are read.  64
// sequences of 4 drafts over 32000 entries 9.2 us, one of 7 looked-up drafts 4.5 us (29.6
// and 13.6 by one CTA a sequence that read its rows twice).
template <int THR, bool kVec>
__global__ void __launch_bounds__(THR) spec_verify_kernel(const VerifyArgs a, int* status) {
  constexpr int W = THR / 32;
  __shared__ int km[2];
  __shared__ double warp_tot[W];
  __shared__ uint64_t part_tot[2][kMaxCluster];
  const uint32_t rank = cluster_rank(), parts = cluster_size();
  cluster_arrive();
  const int b = (int)(blockIdx.x / parts), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int D = a.max_draft, V = a.vocab;
  if (warp == 0) {
    int m;
    const int k = accepted_prefix(a, b, lane, m, status, rank == 0);
    if (lane == 0) {
      km[0] = k;
      km[1] = m;
    }
  }
  __syncthreads();
  const int k = km[0], m = km[1];
  if (rank == 0) write_prefix(a, b, k, status);
  int32_t* out = a.tokens + (int64_t)b * (D + 1);
  cluster_wait();
  if (k < 0 || !rows_in_bounds(a, b, k, m, status)) return;  // (the same in the whole cluster)
  const float* p = a.target + ((int64_t)b * (D + 1) + k) * a.ld_t;
  const float* q = k < m && a.draft ? a.draft + ((int64_t)b * D + k) * a.ld_d : nullptr;
  const int drop = k < m && !a.draft ? a.draft_tokens[(int64_t)b * D + k] : -1;
  const int e0 = ((int)rank * W + warp) * 512 + 4 * lane;
  float4 pv[4], qv[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    pv[i] = load4<kVec>(p, e0 + 128 * i, V, 0.0f);
    qv[i] = q ? load4<kVec>(q, e0 + 128 * i, V, 0.0f) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  if (drop >= 0) {  // a looked-up draft has q = 1 there (probabilities are at most 1)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = e0 + 128 * i;
      if (drop == e) pv[i].x = 0.0f;
      if (drop == e + 1) pv[i].y = 0.0f;
      if (drop == e + 2) pv[i].z = 0.0f;
      if (drop == e + 3) pv[i].w = 0.0f;
    }
  }
  const double u = a.u_sample[b];
#pragma unroll 1
  for (int round = 0; round < 2; ++round) {  // second round: the fallback to the target's own weights
    double d[4];  // this lane's four entries of each 128
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      d[i] = (weight(pv[i].x, qv[i].x) + weight(pv[i].y, qv[i].y)) + (weight(pv[i].z, qv[i].z) + weight(pv[i].w, qv[i].w));
      s += d[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) warp_tot[warp] = s;
    __syncthreads();
    if (warp == 0) {
      double t = 0.0;
      for (int w = 0; w < W; ++w) t += warp_tot[w];
      if (lane < parts) store_cluster(&part_tot[round][rank], lane, (uint64_t)__double_as_longlong(t));
    }
    cluster_arrive();
    cluster_wait();
    double total = 0.0;
    for (uint32_t c = 0; c < parts; ++c) total += __longlong_as_double((long long)part_tot[round][c]);
    if (total > 0.0) {
      const double thr = u * total;
      // the first part whose end lies beyond the draw (else the last one with weight), then likewise its warp
      uint32_t pick = 0;
      double run = 0.0, before = 0.0;
      for (uint32_t c = 0; c < parts; ++c) {
        const double t = __longlong_as_double((long long)part_tot[round][c]);
        if (t > 0.0) {
          pick = c;
          before = run;
          if (run + t > thr) break;
        }
        run += t;
      }
      if (rank != pick) return;
      int pw = 0;
      run = before;
      for (int w = 0; w < W; ++w) {
        const double t = warp_tot[w];
        if (t > 0.0) {
          pw = w;
          before = run;
          if (run + t > thr) break;
        }
        run += t;
      }
      if (warp != pw) return;
      int last = -1;
      double c0 = before;
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
        // (registers are not indexed: the four are rotated)
        const float4 x = pv[0], y = qv[0];
        const double di = d[0];
        pv[0] = pv[1], pv[1] = pv[2], pv[2] = pv[3];
        qv[0] = qv[1], qv[1] = qv[2], qv[2] = qv[3];
        d[0] = d[1], d[1] = d[2], d[2] = d[3];
        double c = di;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const double up = __shfl_up_sync(0xffffffffu, c, o);
          if (lane >= o) c += up;
        }
        const unsigned some = __ballot_sync(0xffffffffu, di > 0.0);
        const unsigned hit = __ballot_sync(0xffffffffu, di > 0.0 && c0 + c > thr);
        if (some) {
          // the lane whose four entries hold the draw (else the last one with weight)
          const int l = hit ? __ffs(hit) - 1 : 31 - __clz(some);
          const double w[4] = {weight(x.x, y.x), weight(x.y, y.y), weight(x.z, y.z), weight(x.w, y.w)};
          double cc = c0 + (c - di);
          int j = -1;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool past = j >= 0 && cc > thr;  // an earlier entry already exceeds the draw
            cc += w[e];
            if (w[e] > 0.0 && !past) j = e;
          }
          last = __shfl_sync(0xffffffffu, e0 + 128 * i + j, l);
        }
        if (hit) break;
        c0 += __shfl_sync(0xffffffffu, c, 31);
      }
      if (lane == 0) out[k] = last;
      return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      pv[i] = load4<kVec>(p, e0 + 128 * i, V, 0.0f);
      qv[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __syncthreads();
  }
  if (rank == 0 && threadIdx.x == 0) out[k] = -1;
}

// Vocabularies longer than a cluster holds: one CTA a sequence, a contiguous range
// a warp, and the warp the draw falls into walks its range again.
constexpr int kVerifyThreads = 1024;
constexpr int kVerifyWarps = kVerifyThreads / 32;
__global__ void __launch_bounds__(kVerifyThreads) spec_verify_long_kernel(const VerifyArgs a, int* status) {
  __shared__ int km[2];
  __shared__ double tot[kVerifyWarps];
  const int b = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int D = a.max_draft, V = a.vocab;
  if (warp == 0) {
    int m;
    const int k = accepted_prefix(a, b, lane, m, status, true);
    if (lane == 0) {
      km[0] = k;
      km[1] = m;
    }
  }
  __syncthreads();
  const int k = km[0], m = km[1];
  write_prefix(a, b, k, status);
  if (k < 0 || !rows_in_bounds(a, b, k, m, status)) return;
  int32_t* out = a.tokens + (int64_t)b * (D + 1);
  const float* p = a.target + ((int64_t)b * (D + 1) + k) * a.ld_t;
  const float* q = k < m && a.draft ? a.draft + ((int64_t)b * D + k) * a.ld_d : nullptr;
  const int drop = k < m && !a.draft ? a.draft_tokens[(int64_t)b * D + k] : -1;
  // (unsigned: the last warp's range may end behind 2^31)
  const unsigned range = (((unsigned)V + kVerifyWarps - 1) / kVerifyWarps + 31) / 32 * 32;
  const unsigned j0 = min((unsigned)V, warp * range), j1 = min((unsigned)V, j0 + range);
#pragma unroll 1
  for (int round = 0; round < 2; ++round) {
    const auto at = [&](unsigned j) {
      if (round) return weight(p[j], 0.0f);
      return (int)j == drop ? 0.0 : weight(p[j], q ? q[j] : 0.0f);
    };
    double s = 0.0;
    for (unsigned j = j0 + lane; j < j1; j += 32) s += at(j);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) tot[warp] = s;
    __syncthreads();
    double total = 0.0;
#pragma unroll 1
    for (int w = 0; w < kVerifyWarps; ++w) total += tot[w];
    if (total > 0.0) {
      const double thr = (double)a.u_sample[b] * total;
      int pick = 0;
      double run = 0.0, before = 0.0;
#pragma unroll 1
      for (int w = 0; w < kVerifyWarps; ++w) {
        if (tot[w] > 0.0) {
          pick = w;
          before = run;
          if (run + tot[w] > thr) break;
        }
        run += tot[w];
      }
      if (warp != pick) return;
      int last = -1;
      double c0 = before;
      for (unsigned j = j0; j < j1; j += 32) {
        const double w = j + lane < j1 ? at(j + lane) : 0.0;
        double c = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const double up = __shfl_up_sync(0xffffffffu, c, o);
          if (lane >= o) c += up;
        }
        const unsigned some = __ballot_sync(0xffffffffu, w > 0.0);
        const unsigned hit = __ballot_sync(0xffffffffu, w > 0.0 && c0 + c > thr);
        if (some) last = (int)j + 31 - __clz(some);
        if (hit) {
          last = (int)j + __ffs(hit) - 1;
          break;
        }
        c0 += __shfl_sync(0xffffffffu, c, 31);
      }
      if (lane == 0) out[k] = last;
      return;
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) out[k] = -1;
}

// Launches `kernel` with `rows` clusters of `parts` CTAs.
template <class K, class... Args>
int launch_clusters(K kernel, int64_t rows, int parts, int threads, cudaStream_t s, Args... args) {
  if (rows * parts > 0x7fffffff) return INV_ERR_UNSUPPORTED_SHAPE;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)(rows * parts));
  lc.blockDim = dim3(threads);
  lc.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = parts;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  if (cudaLaunchKernelEx(&lc, kernel, args...) != cudaSuccess) return INV_ERR_CUDA;
  INV_CHECK_LAUNCH();
  return INV_OK;
}

template <int THR>
int launch_softmax(const float* x, int rows, int n, int64_t ld, float it, float* y, int64_t ld_y, cudaStream_t s) {
  const int part = THR * kSoftVals, parts = (n + part - 1) / part;
  return launch_clusters(softmax_kernel<THR>, rows, parts, THR, s, x, rows, n, ld, it, y, ld_y, inv::status_ptr());
}

template <int THR>
int launch_verify(bool vec, const VerifyArgs& a, cudaStream_t s) {
  const int part = THR * 16, parts = (a.vocab + part - 1) / part;
  return launch_clusters(vec ? spec_verify_kernel<THR, true> : spec_verify_kernel<THR, false>, a.B, parts, THR, s, a,
                         inv::status_ptr());
}

}  // namespace

extern "C" {

int softmax_rows(const float* logits, int rows, int n, int64_t ld, float inv_temperature, float* probs, int64_t ld_p,
                 inv_stream stream) {
  if (rows < 0 || n <= 0 || ld < n || ld_p < n) return INV_ERR_INVALID_ARG;
  if (!(inv_temperature > 0.0f) || !(inv_temperature <= 3.402823466e38f)) return INV_ERR_INVALID_ARG;
  if (rows == 0) return INV_OK;
  if (!logits || !probs || (logits == probs && ld != ld_p)) return INV_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // The smallest CTAs whose cluster of at most eight holds a row, five a SM: many small CTAs overlap their loads,
  // exponentials and stores.
  if (n <= kMaxCluster * 256 * kSoftVals) return launch_softmax<256>(logits, rows, n, ld, inv_temperature, probs, ld_p, s);
  if (n <= kMaxCluster * 512 * kSoftVals) return launch_softmax<512>(logits, rows, n, ld, inv_temperature, probs, ld_p, s);
  if (n <= kMaxCluster * 1024 * kSoftVals) return launch_softmax<1024>(logits, rows, n, ld, inv_temperature, probs, ld_p, s);
  softmax_long_kernel<<<(unsigned)rows, kLongThreads, 0, s>>>(logits, rows, n, ld, inv_temperature, probs, ld_p,
                                                              inv::status_ptr());
  INV_CHECK_LAUNCH();
  return INV_OK;
}

int spec_verify(const float* target, int64_t ld_target, const float* draft, int64_t ld_draft, int B, int max_draft,
                int vocab, const int32_t* draft_tokens, const int32_t* n_draft, const float* u_accept,
                const float* u_sample, int32_t* tokens, int32_t* n_accepted, inv_stream stream) {
  if (B < 0 || max_draft < 0 || max_draft > kMaxDraft || vocab <= 0 || ld_target < vocab || (draft && ld_draft < vocab))
    return INV_ERR_INVALID_ARG;
  if (B == 0) return INV_OK;
  if (!target || !u_sample || !tokens || !n_accepted || (max_draft > 0 && (!draft_tokens || !u_accept)))
    return INV_ERR_INVALID_ARG;
  const VerifyArgs a = {target,  ld_target,    draft,   ld_draft, B,        max_draft, vocab,
                        draft_tokens, n_draft, u_accept, u_sample, tokens, n_accepted};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool vec = inv::aligned16(target) && inv::aligned16(draft) && ld_target % 4 == 0 && ld_draft % 4 == 0;
  if (vocab <= kMaxCluster * 256 * 16) return launch_verify<256>(vec, a, s);
  if (vocab <= kMaxCluster * 1024 * 16) return launch_verify<1024>(vec, a, s);
  spec_verify_long_kernel<<<(unsigned)B, kVerifyThreads, 0, s>>>(a, inv::status_ptr());
  INV_CHECK_LAUNCH();
  return INV_OK;
}

}  // extern "C"
