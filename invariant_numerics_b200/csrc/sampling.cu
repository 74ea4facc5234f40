// softmax_rows and spec_verify: from logits to the tokens of a verification
// step of speculative decoding.
#include "common.cuh"
#include "paged.cuh"

namespace {

using inv::record_status;

// ----------------------------------------------------------- softmax_rows ----

constexpr int kSoftThreads = 1024;

__device__ __forceinline__ float4 load4(const float* p, int i, int n) {
  float4 v;
  v.x = i < n ? p[i] : -INFINITY;
  v.y = i + 1 < n ? p[i + 1] : -INFINITY;
  v.z = i + 2 < n ? p[i + 2] : -INFINITY;
  v.w = i + 3 < n ? p[i + 3] : -INFINITY;
  return v;
}

// One CTA per row; thread t owns the elements 4t .. 4t+3 of every 4096.
__global__ void __launch_bounds__(kSoftThreads)
    softmax_kernel(const float* __restrict__ x, int rows, int n, int64_t ld, float it, float* y, int64_t ld_y,
                   int* status) {
  __shared__ float red[32];
  __shared__ float bc[2];
  const int64_t r = blockIdx.x;
  if (!INV_SPAN_IN_BOUNDS(status, r * ld, r * ld + n - 1, (int64_t)(rows - 1) * ld + n) ||
      !INV_SPAN_IN_BOUNDS(status, r * ld_y, r * ld_y + n - 1, (int64_t)(rows - 1) * ld_y + n))
    return;
  const float* xr = x + r * ld;
  float* yr = y + r * ld_y;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float m = -INFINITY;
  for (int i = threadIdx.x * 4; i < n; i += 4 * kSoftThreads) {
    const float4 v = load4(xr, i, n);
    m = fmaxf(m, fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) red[warp] = m;
  __syncthreads();
  if (warp == 0) {
    m = red[lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) bc[0] = m;
  }
  __syncthreads();
  m = bc[0];
  const bool none = m == -INFINITY;
  const auto e = [&](float v) { return none ? 0.0f : expf(__fmul_rn(__fsub_rn(v, m), it)); };
  float s = 0.0f;
  for (int i = threadIdx.x * 4; i < n; i += 4 * kSoftThreads) {
    const float4 v = load4(xr, i, n);
    s = __fadd_rn(s, __fadd_rn(__fadd_rn(e(v.x), e(v.y)), __fadd_rn(e(v.z), e(v.w))));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, o));
  if (lane == 0) red[warp] = s;
  __syncthreads();
  if (warp == 0) {
    s = red[lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, o));
    if (lane == 0) bc[1] = s;
  }
  __syncthreads();
  const float inv_s = none ? 0.0f : __frcp_rn(bc[1]);
  for (int i = threadIdx.x * 4; i < n; i += 4 * kSoftThreads) {
    const float4 v = load4(xr, i, n);
    yr[i] = __fmul_rn(e(v.x), inv_s);
    if (i + 1 < n) yr[i + 1] = __fmul_rn(e(v.y), inv_s);
    if (i + 2 < n) yr[i + 2] = __fmul_rn(e(v.z), inv_s);
    if (i + 3 < n) yr[i + 3] = __fmul_rn(e(v.w), inv_s);
  }
}

// ------------------------------------------------------------ spec_verify ----

constexpr int kVerifyThreads = 1024;
constexpr int kVerifyWarps = kVerifyThreads / 32;

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

// One CTA per sequence.  Warp 0 decides the accepted prefix, 32 drafts a step.
// The next token: warp w owns a contiguous range of the vocabulary; the warps'
// totals in 64 bits tell which range the draw falls into, and that warp walks
// its range again.
__global__ void __launch_bounds__(kVerifyThreads) spec_verify_kernel(VerifyArgs a, int* status) {
  __shared__ int k_sh, m_sh;
  __shared__ double tot[kVerifyWarps];
  const int b = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int D = a.max_draft, V = a.vocab;
  const int32_t* x = a.draft_tokens + (int64_t)b * D;
  if (warp == 0) {
    const int m = a.n_draft ? a.n_draft[b] : D;
    bool bad = m < 0 || m > D;
    int k = 0;
    if (!bad) {
      k = m;
      for (int i0 = 0; i0 < m; i0 += 32) {
        const int i = i0 + lane;
        bool ok = true, wrong = false;
        if (i < m) {
          const int t = x[i];
          wrong = t < 0 || t >= V;
          if (!wrong) {
            const double q = a.draft ? (double)a.draft[((int64_t)b * D + i) * a.ld_d + t] : 1.0;
            ok = (double)a.u_accept[(int64_t)b * D + i] * q < (double)a.target[((int64_t)b * (D + 1) + i) * a.ld_t + t];
          }
        }
        bad |= __any_sync(0xffffffffu, wrong);
        const unsigned no = __ballot_sync(0xffffffffu, !ok);
        if (no != 0 && k == m) k = i0 + __ffs(no) - 1;
      }
    }
    if (lane == 0) {
      if (bad) record_status(status, INV_ERR_INVALID_ARG);
      k_sh = bad ? -1 : k;
      m_sh = m;
    }
  }
  __syncthreads();
  const int k = k_sh, m = m_sh;
  int32_t* out = a.tokens + (int64_t)b * (D + 1);
  if (k < 0) {
    for (int i = threadIdx.x; i <= D; i += kVerifyThreads) out[i] = -1;
    if (threadIdx.x == 0) a.n_accepted[b] = 0;
    return;
  }
  for (int i = threadIdx.x; i <= D; i += kVerifyThreads)
    if (i != k) out[i] = i < k ? x[i] : -1;
  if (threadIdx.x == 0) a.n_accepted[b] = k;

  const float* p = a.target + ((int64_t)b * (D + 1) + k) * a.ld_t;
  const float* q = k < m && a.draft ? a.draft + ((int64_t)b * D + k) * a.ld_d : nullptr;
  const int drop = k < m && !a.draft ? x[k] : -1;
  const int range = ((V + kVerifyWarps - 1) / kVerifyWarps + 31) / 32 * 32;
  const int j0 = min(V, warp * range), j1 = min(V, j0 + range);
  for (int plain = 0; plain < 2; ++plain) {  // second time: the fallback to the target's own weights
    const auto weight = [&](int j) {
      const double t = p[j];
      if (plain) return t > 0.0 ? t : 0.0;
      const double u = q ? (double)q[j] : 0.0;
      return j != drop && t > u ? t - u : 0.0;
    };
    double s = 0.0;
    for (int j = j0 + lane; j < j1; j += 32) s += weight(j);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) tot[warp] = s;
    __syncthreads();
    double total = 0.0, before = 0.0;
    for (int w = 0; w < kVerifyWarps; ++w) total += tot[w];
    if (total > 0.0) {
      const double thr = (double)a.u_sample[b] * total;
      // the first range whose end lies beyond the draw (else the last one with weight)
      int pick = -1;
      double run = 0.0;
      for (int w = 0; w < kVerifyWarps; ++w) {
        if (tot[w] > 0.0) {
          pick = w;
          before = run;
          if (run + tot[w] > thr) break;
        }
        run += tot[w];
      }
      if (warp == pick) {
        int last = -1;
        double c0 = before;
        for (int j = j0; j < j1; j += 32) {
          const double w = j + lane < j1 ? weight(j + lane) : 0.0;
          double c = w;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const double up = __shfl_up_sync(0xffffffffu, c, o);
            if (lane >= o) c += up;
          }
          const unsigned pos = __ballot_sync(0xffffffffu, w > 0.0);
          const unsigned hit = __ballot_sync(0xffffffffu, w > 0.0 && c0 + c > thr);
          if (pos) last = j + 31 - __clz(pos);
          if (hit) {
            last = j + __ffs(hit) - 1;
            break;
          }
          c0 += __shfl_sync(0xffffffffu, c, 31);
        }
        if (lane == 0) out[k] = last;
      }
      return;
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) out[k] = -1;
}

}  // namespace

extern "C" {

int softmax_rows(const float* logits, int rows, int n, int64_t ld, float inv_temperature, float* probs, int64_t ld_p,
                 inv_stream stream) {
  if (rows < 0 || n <= 0 || ld < n || ld_p < n) return INV_ERR_INVALID_ARG;
  if (!(inv_temperature > 0.0f) || !(inv_temperature <= 3.402823466e38f)) return INV_ERR_INVALID_ARG;
  if (rows == 0) return INV_OK;
  if (!logits || !probs || (logits == probs && ld != ld_p)) return INV_ERR_INVALID_ARG;
  softmax_kernel<<<(unsigned)rows, kSoftThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      logits, rows, n, ld, inv_temperature, probs, ld_p, inv::status_ptr());
  INV_CHECK_LAUNCH();
  return INV_OK;
}

int spec_verify(const float* target, int64_t ld_target, const float* draft, int64_t ld_draft, int B, int max_draft,
                int vocab, const int32_t* draft_tokens, const int32_t* n_draft, const float* u_accept,
                const float* u_sample, int32_t* tokens, int32_t* n_accepted, inv_stream stream) {
  if (B < 0 || max_draft < 0 || vocab <= 0 || ld_target < vocab || (draft && ld_draft < vocab))
    return INV_ERR_INVALID_ARG;
  if (B == 0) return INV_OK;
  if (!target || !u_sample || !tokens || !n_accepted || (max_draft > 0 && (!draft_tokens || !u_accept)))
    return INV_ERR_INVALID_ARG;
  const VerifyArgs a = {target,  ld_target,    draft,   ld_draft, B,        max_draft, vocab,
                        draft_tokens, n_draft, u_accept, u_sample, tokens, n_accepted};
  spec_verify_kernel<<<(unsigned)B, kVerifyThreads, 0, static_cast<cudaStream_t>(stream)>>>(a, inv::status_ptr());
  INV_CHECK_LAUNCH();
  return INV_OK;
}

}  // extern "C"
