// gdn_step.cu - the gated delta rule's recurrent form for decoding: a few tokens of many sequences, each on its
// own state out of a pool.
//
// Per token, on the state S [dk, dv] of one head (a = log_alpha):
//   p = e^a S^T k,  E = v - p,  S <- e^a S + beta k E^T,  y = S^T q,
// where y = e^a S^T q + beta (k . q) E, so both products with the state are taken of the state before the
// token: one sum over the rows, and one barrier, a token.
//
// Bound by the state's bytes: read and written once a call, whatever T is (256 sequences of 16 heads of 128 x
// 128: 537 MB in 91 us, 87% of the measured copy bandwidth).  A CTA holds 32 columns of one head's state in
// registers: 8 lanes a row, 16 bytes each, 16 rows at a time.  A column group of 32 makes 4 CTAs of a 128 x 128
// state, so that one sequence's 16 heads already reach 64 SMs; five CTAs an SM keep enough loads on their way
// (unbounded registers, 3 or 4 an SM: 113 us), and nothing of the state is kept in the caches on its way
// through (cached: 107).
#include <climits>

#include <cuda_bf16.h>

#include "common.cuh"

namespace sdm {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps, kRows = 4 * kWarps;  // kRows: at a time
constexpr int kCols = 32;

struct StepArgs {
  float *state;
  const uint16_t *q, *k, *v;
  int64_t ld_q, ld_k, ld_v;
  const float *la, *beta;
  const int32_t *slots, *lens;
  int P, B, T, Hk, H, dk, dv, groups;
  uint16_t *y;
  int32_t *err;
};

// sum over the four rows that a warp holds of each column quad
__device__ __forceinline__ float rows_sum(float x) {
  x += __shfl_xor_sync(kFull, x, 8);
  return x + __shfl_xor_sync(kFull, x, 16);
}

template <int NR, bool VEC>  // NR: rows a thread
__global__ void __launch_bounds__(kThreads, 5) gdn_step_kernel(const StepArgs a) {
  __shared__ float part[2][kWarps][2][kCols];  // token parity, warp, S^T k and S^T q
  __shared__ float kq[2][kWarps];
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const int64_t bh = blockIdx.x / a.groups;
  const int c0 = static_cast<int>(blockIdx.x - bh * a.groups) * kCols;
  const int b = static_cast<int>(bh / a.H), h = static_cast<int>(bh % a.H), hk = h / (a.H / a.Hk);
  int slot = b;
  if (a.slots) {
    slot = a.slots[b];
    if (slot < 0 || slot >= a.P) {  // the whole CTA
      if (a.err && tid == 0 && slot >= 0) atomicOr(a.err, SDM_DEVERR_INDEX_RANGE);
      return;
    }
  }
  int T = a.T;
  if (a.lens) {
    T = min(max(a.lens[b], 0), a.T);
    if (a.err && tid == 0 && T != a.lens[b]) atomicOr(a.err, SDM_DEVERR_INDEX_RANGE);
  }
  if (T == 0) return;
  const int r0 = 4 * w + (lane >> 3), c = c0 + 4 * (lane & 7);
  float *S = a.state + (static_cast<int64_t>(slot) * a.H + h) * a.dk * a.dv + c;
  float s[NR][4];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int r = r0 + kRows * i;
    if (VEC) {
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < a.dk && c < a.dv) x = __ldcs(reinterpret_cast<const float4 *>(S + static_cast<int64_t>(r) * a.dv));
      s[i][0] = x.x, s[i][1] = x.y, s[i][2] = x.z, s[i][3] = x.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[i][e] = r < a.dk && c + e < a.dv ? S[static_cast<int64_t>(r) * a.dv + e] : 0.f;
    }
  }
  if (a.slots) {  // a slot that a sequence before this one names, looked for while the state is on its way
    bool repeat = false;
    for (int i = tid; i < b; i += kThreads) repeat |= a.slots[i] == slot;
    if (__syncthreads_or(repeat)) {
      if (a.err && tid == 0) atomicOr(a.err, SDM_DEVERR_INDEX_REPEAT);
      return;
    }
  }
  for (int t = 0; t < T; ++t) {
    const int64_t tok = static_cast<int64_t>(b) * a.T + t;
    const uint16_t *kp = a.k + tok * a.ld_k + hk * a.dk, *qp = a.q + tok * a.ld_q + hk * a.dk;
    float k[NR], q[NR], v[4];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int r = r0 + kRows * i;
      k[i] = r < a.dk ? bf16_to_f32(kp[r]) : 0.f;
      q[i] = r < a.dk ? bf16_to_f32(qp[r]) : 0.f;
    }
    const uint16_t *vp = a.v + tok * a.ld_v + h * a.dv + c;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = c + e < a.dv ? bf16_to_f32(vp[e]) : 0.f;
    const float decay = expf(a.la[tok * a.H + h]), beta = a.beta[tok * a.H + h];
    float pk[4] = {0.f, 0.f, 0.f, 0.f}, pq[4] = {0.f, 0.f, 0.f, 0.f}, dot = 0.f;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      dot = fmaf(k[i], q[i], dot);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        pk[e] = fmaf(k[i], s[i][e], pk[e]);
        pq[e] = fmaf(q[i], s[i][e], pq[e]);
      }
    }
    dot = rows_sum(dot);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      pk[e] = rows_sum(pk[e]);
      pq[e] = rows_sum(pq[e]);
    }
    float(&pt)[kWarps][2][kCols] = part[t & 1];
    if (lane < 8) {
      *reinterpret_cast<float4 *>(&pt[w][0][4 * lane]) = make_float4(pk[0], pk[1], pk[2], pk[3]);
      *reinterpret_cast<float4 *>(&pt[w][1][4 * lane]) = make_float4(pq[0], pq[1], pq[2], pq[3]);
      if (lane == 0) kq[t & 1][w] = dot;
    }
    __syncthreads();  // (the other parity's words are read up to the barrier before this one)
    float e4[4], y4[4];
    float p4[4] = {0.f, 0.f, 0.f, 0.f}, o4[4] = {0.f, 0.f, 0.f, 0.f};
    dot = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      dot += kq[t & 1][i];
      const float4 p = *reinterpret_cast<const float4 *>(&pt[i][0][4 * (lane & 7)]);
      const float4 o = *reinterpret_cast<const float4 *>(&pt[i][1][4 * (lane & 7)]);
      p4[0] += p.x, p4[1] += p.y, p4[2] += p.z, p4[3] += p.w;
      o4[0] += o.x, o4[1] += o.y, o4[2] += o.z, o4[3] += o.w;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      e4[e] = beta * fmaf(-decay, p4[e], v[e]);
      y4[e] = fmaf(dot, e4[e], decay * o4[e]);
    }
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[i][e] = fmaf(k[i], e4[e], decay * s[i][e]);
    if (tid < 8) {
      uint16_t *yp = a.y + (tok * a.H + h) * a.dv + c;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c + e < a.dv) yp[e] = __bfloat16_as_ushort(__float2bfloat16_rn(y4[e]));
    }
  }
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int r = r0 + kRows * i;
    if (r >= a.dk) continue;
    if (VEC) {
      if (c < a.dv)
        __stcs(reinterpret_cast<float4 *>(S + static_cast<int64_t>(r) * a.dv),
               make_float4(s[i][0], s[i][1], s[i][2], s[i][3]));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c + e < a.dv) S[static_cast<int64_t>(r) * a.dv + e] = s[i][e];
    }
  }
}

}  // namespace
}  // namespace sdm

using namespace sdm;

extern "C" int gdn_step(float *state, const uint16_t *q, int64_t ld_q, const uint16_t *k, int64_t ld_k,
                        const uint16_t *v, int64_t ld_v, const float *log_alpha, const float *beta,
                        const int32_t *slots, const int32_t *lens, int P, int B, int T, int Hk, int H, int dk, int dv,
                        uint16_t *y, int32_t *dev_err, void *stream) {
  if (P < 0 || B < 0 || T < 0 || Hk < 0 || H < 0) return set_error(SDM_ERR_INVALID_ARG, "gdn_step: negative size");
  if (B >= 65536 || H >= 65536 || T >= (1 << 20) || dk < 1 || dk > 128 || dv < 1 || dv > 1024 ||
      (H > 0 && (Hk == 0 || H % Hk != 0)) ||
      static_cast<int64_t>(B) * H * ((dv + kCols - 1) / kCols) > INT_MAX)
    return set_error(SDM_ERR_SHAPE, "gdn_step: sizes beyond the limits");
  if (!slots && P < B) return set_error(SDM_ERR_SHAPE, "gdn_step: %d states for %d sequences", P, B);
  if (ld_q < static_cast<int64_t>(Hk) * dk || ld_k < static_cast<int64_t>(Hk) * dk ||
      ld_v < static_cast<int64_t>(H) * dv || ld_q >= (1 << 27) || ld_k >= (1 << 27) || ld_v >= (1 << 27))
    return set_error(SDM_ERR_SHAPE,
                     "gdn_step: a token's row must be at most 2^27 elements from the next and hold its heads");
  if (B == 0 || T == 0 || H == 0) return SDM_OK;
  if ((!state && P > 0) || !q || !k || !v || !log_alpha || !beta || !y)
    return set_error(SDM_ERR_INVALID_ARG, "gdn_step: null pointer");
  if (!aligned(state, 4) || !aligned(q, 2) || !aligned(k, 2) || !aligned(v, 2) || !aligned(log_alpha, 4) ||
      !aligned(beta, 4) || !aligned(y, 2) || !aligned(slots, 4) || !aligned(lens, 4) || !aligned(dev_err, 4))
    return set_error(SDM_ERR_ALIGN, "gdn_step: a pointer is not aligned");
  StepArgs a{state, q, k, v, ld_q, ld_k, ld_v, log_alpha, beta, slots, lens,
             P, B, T, Hk, H, dk, dv, (dv + kCols - 1) / kCols, y, dev_err};
  const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(B) * H * a.groups);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool vec = dv % 4 == 0 && aligned(state, 16);
  auto kernel = vec ? gdn_step_kernel<128 / kRows, true> : gdn_step_kernel<128 / kRows, false>;
  if (dk <= 64) kernel = vec ? gdn_step_kernel<64 / kRows, true> : gdn_step_kernel<64 / kRows, false>;
  kernel<<<grid, kThreads, 0, st>>>(a);
  return check_launch("gdn_step");
}
