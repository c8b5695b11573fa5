// glr_scan.cu - gated linear recurrence with one state per channel, its
// training forward and its backward pass (glr_scan in sdm.h):
//   L_t = -rate sigmoid(r_t), a_t = e^{L_t}, m_t = sqrt(1 - a_t^2),
//   h_t = a_t h_{t-1} + m_t sigmoid(g_t) x_t.
//
// One thread per (sequence, channel), tokens in order (the backward: segments
// of 8 tokens last to first, each recomputed from the state kept before it).
#include <initializer_list>

#include "ckpt8.cuh"

namespace sdm {
namespace {

constexpr int kSeg = 8;  // tokens between the states that the training forward keeps

struct GlrArgs {
  const float *state;   // h_0, or dL/dh_T
  float *state_out;     // h_T, or dL/dh_0
  const void *x, *r, *g;
  int64_t ld_x, ld_r, ld_g, ld_d;
  const int8_t *codes;
  const uint8_t *exps;
  const float *rate;
  const uint8_t *reset;
  const int32_t *lens;
  int B, T, D, S;
  void *y;              // or dy
  float *carry;
  void *dx, *dr, *dg;
  float *part;          // [B][D]: drate of each sequence
  int32_t *err;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rsq(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float sigmoid(float x) { return rcp(1.f + ex2(-kLog2e * x)); }

// One token's decay and its complement: sr = sigmoid(r), a = 2^l with
// l = -rate log2(e) sr, m2 = 1 - a^2.  Near a = 1 the difference cancels, so
// for w = -2 ln a <= 1/4 the series w (1 - w/2 (1 - w/3 (...))) takes over,
// whose first term left out is below 5e-8 of it there; above, 1 - a^2 loses
// two bits at most.
struct Gate {
  float sr, sg, a, m2;
};
__device__ __forceinline__ Gate gate(float r, float g, float rate2) {
  Gate q;
  q.sr = sigmoid(r);
  q.sg = sigmoid(g);
  const float l = rate2 * q.sr;
  q.a = ex2(l);
  const float w = -2.f * kLn2 * l;
  float p = fmaf(w, -1.f / 6.f, 1.f);
  p = fmaf(w * -0.2f, p, 1.f);
  p = fmaf(w * -0.25f, p, 1.f);
  p = fmaf(w * (-1.f / 3.f), p, 1.f);
  p = fmaf(w * -0.5f, p, 1.f);
  q.m2 = w <= 0.25f ? w * p : fmaf(-q.a, q.a, 1.f);
  return q;
}
// 1 / sqrt(m2), and 0 where m2 underflows
__device__ __forceinline__ float inv_m(float m2) { return m2 >= 1.17549435e-38f ? rsq(m2) : 0.f; }

__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t *p) { return bf16_to_f32(*p); }
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t *p, float v) {
  asm("{.reg .b16 h; cvt.rn.bf16.f32 h, %1; st.global.b16 [%0], h;}" ::"l"(p), "f"(v) : "memory");
}

// -rate log2(e), with a rate outside [0, inf) flagged and taken as 0
__device__ __forceinline__ float load_rate(const GlrArgs &a, int c) {
  float v = a.rate[c];
  if (!(v >= 0.f && v < __int_as_float(0x7f800000))) {
    if (a.err) atomicOr(a.err, SDM_DEVERR_RATE);
    v = 0.f;
  }
  return v;
}
__device__ __forceinline__ int load_len(const GlrArgs &a, int b) {
  if (!a.lens) return a.T;
  const int n = a.lens[b];
  if ((n < 0 || n > a.T) && a.err) atomicOr(a.err, SDM_DEVERR_INDEX_RANGE);
  return n < 0 ? 0 : n > a.T ? a.T : n;
}

template <class E>
__global__ void __launch_bounds__(128) glr_forward_kernel(const GlrArgs a) {
  const int c = blockIdx.x * 128 + threadIdx.x, b = blockIdx.y;
  if (c >= a.D) return;
  const int len = load_len(a, b);
  const float rate2 = -kLog2e * load_rate(a, c);
  const int64_t row0 = static_cast<int64_t>(b) * a.T;
  float h = a.state[static_cast<int64_t>(b) * a.D + c];
  for (int t = 0; t < len; ++t) {
    const int64_t row = row0 + t;
    if (a.carry && t % kSeg == 0) a.carry[(static_cast<int64_t>(b) * a.S + t / kSeg) * a.D + c] = h;
    const float x = load1(static_cast<const E *>(a.x) + row * a.ld_x + c);
    const Gate q = gate(load1(static_cast<const E *>(a.r) + row * a.ld_r + c),
                        load1(static_cast<const E *>(a.g) + row * a.ld_g + c), rate2);
    const float u = q.m2 * inv_m(q.m2) * q.sg * x;
    h = fmaf(q.a, a.reset && a.reset[row] ? 0.f : h, u);
    store1(static_cast<E *>(a.y) + row * a.D + c, h);
  }
  a.state_out[static_cast<int64_t>(b) * a.D + c] = h;
}

template <class E, bool K8>
__global__ void __launch_bounds__(128) glr_backward_kernel(const GlrArgs a) {
  const int c = blockIdx.x * 128 + threadIdx.x, b = blockIdx.y;
  if (c >= a.D) return;
  const int len = load_len(a, b);
  const float rate = load_rate(a, c), rate2 = -kLog2e * rate;
  const int64_t row0 = static_cast<int64_t>(b) * a.T;
  const int64_t n = static_cast<int64_t>(a.B) * a.T;
  const int G = ckpt8::groups(a.D);
  auto decoded = [&](int plane, int64_t row) {
    const int64_t i = plane * n + row;
    return static_cast<float>(a.codes[i * a.D + c]) * ckpt8::step(a.exps[i * G + c / ckpt8::kGroup]);
  };
  float dh = a.state ? a.state[static_cast<int64_t>(b) * a.D + c] : 0.f;  // a_{t+1} dh_{t+1}
  float drate = 0.f;
  for (int s = (len + kSeg - 1) / kSeg - 1; s >= 0; --s) {
    float before[kSeg], xs[kSeg];
    Gate q[kSeg];
    float h = a.carry[(static_cast<int64_t>(b) * a.S + s) * a.D + c];
#pragma unroll
    for (int i = 0; i < kSeg; ++i) {
      const int t = s * kSeg + i;
      if (t >= len) break;
      const int64_t row = row0 + t;
      float r, g;
      if (K8) {
        xs[i] = decoded(0, row), r = decoded(1, row), g = decoded(2, row);
      } else {
        xs[i] = load1(static_cast<const E *>(a.x) + row * a.ld_x + c);
        r = load1(static_cast<const E *>(a.r) + row * a.ld_r + c);
        g = load1(static_cast<const E *>(a.g) + row * a.ld_g + c);
      }
      q[i] = gate(r, g, rate2);
      before[i] = a.reset && a.reset[row] ? 0.f : h;
      h = fmaf(q[i].a, before[i], q[i].m2 * inv_m(q[i].m2) * q[i].sg * xs[i]);
    }
#pragma unroll
    for (int i = kSeg - 1; i >= 0; --i) {
      const int t = s * kSeg + i;
      if (t >= len) continue;
      const int64_t row = row0 + t;
      dh += load1(static_cast<const E *>(a.y) + row * a.D + c);
      const float rs = inv_m(q[i].m2), m = q[i].m2 * rs, sx = q[i].sg * xs[i];
      const float dL = q[i].a * dh * fmaf(-q[i].a * rs, sx, before[i]);
      store1(static_cast<E *>(a.dx) + row * a.ld_d + c, dh * m * q[i].sg);
      store1(static_cast<E *>(a.dr) + row * a.ld_d + c, -rate * q[i].sr * (1.f - q[i].sr) * dL);
      store1(static_cast<E *>(a.dg) + row * a.ld_d + c, dh * m * sx * (1.f - q[i].sg));
      drate = fmaf(-q[i].sr, dL, drate);
      dh = a.reset && a.reset[row] ? 0.f : q[i].a * dh;
    }
  }
  a.state_out[static_cast<int64_t>(b) * a.D + c] = dh;
  a.part[static_cast<int64_t>(b) * a.D + c] = drate;
}

// drate[c] = sum over the parts in order
__global__ void __launch_bounds__(128) glr_rate_kernel(const float *part, int parts, int D, float *drate) {
  const int c = blockIdx.x * 128 + threadIdx.x;
  if (c >= D) return;
  float s = 0.f;
  for (int i = 0; i < parts; ++i) s += part[static_cast<int64_t>(i) * D + c];
  drate[c] = s;
}

int check_sizes(const char *fn, int dtype, int B, int T, int D) {
  if (B < 0 || T < 0 || D < 0) return set_error(SDM_ERR_INVALID_ARG, "%s: negative size", fn);
  if (dtype != SDM_DTYPE_F32 && dtype != SDM_DTYPE_BF16) return set_error(SDM_ERR_UNSUPPORTED, "%s: unknown dtype", fn);
  if (B >= 65536 || T >= 1 << 30 || D >= 1 << 24)
    return set_error(SDM_ERR_SHAPE, "%s: need B < 65536, T < 2^30, D < 2^24", fn);
  return SDM_OK;
}

// [B,T,D] tensors of `dtype` with their distance between tokens
int check_rows(const char *fn, const char *name, const void *p, int64_t ld, int dtype, int D) {
  if (!p) return set_error(SDM_ERR_INVALID_ARG, "%s: null pointer (%s)", fn, name);
  if (ld < D || ld >= int64_t(1) << 31) return set_error(SDM_ERR_SHAPE, "%s: need D <= ld < 2^31 (%s)", fn, name);
  if (!aligned(p, dtype == SDM_DTYPE_F32 ? 4 : 2))
    return set_error(SDM_ERR_ALIGN, "%s: %s must be aligned to its element", fn, name);
  return SDM_OK;
}

int check_words(const char *fn, std::initializer_list<const void *> ps) {
  for (const void *p : ps)
    if (!aligned(p, 4)) return set_error(SDM_ERR_ALIGN, "%s: fp32 and int32 arrays must be 4-byte aligned", fn);
  return SDM_OK;
}

dim3 grid_of(int B, int D) { return dim3((D + 127) / 128, B); }

int forward(const char *fn, GlrArgs &a, int dtype, int8_t *codes, uint8_t *exps, cudaStream_t st) {
  int rc = check_sizes(fn, dtype, a.B, a.T, a.D);
  if (rc != SDM_OK) return rc;
  if (a.B == 0 || a.D == 0) return SDM_OK;
  if (!a.state || !a.state_out || !a.rate) return set_error(SDM_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (a.T > 0) {
    if ((rc = check_rows(fn, "x", a.x, a.ld_x, dtype, a.D)) || (rc = check_rows(fn, "r", a.r, a.ld_r, dtype, a.D)) ||
        (rc = check_rows(fn, "g", a.g, a.ld_g, dtype, a.D)) || (rc = check_rows(fn, "y", a.y, a.D, dtype, a.D)))
      return rc;
  }
  if ((rc = check_words(fn, {a.state, a.state_out, a.rate, a.lens, a.carry, a.err}))) return rc;
  const dim3 grid = grid_of(a.B, a.D);
  if (dtype == SDM_DTYPE_F32)
    glr_forward_kernel<float><<<grid, 128, 0, st>>>(a);
  else
    glr_forward_kernel<uint16_t><<<grid, 128, 0, st>>>(a);
  if ((rc = check_launch(fn)) || !codes || a.T == 0) return rc;
  const int64_t rows = static_cast<int64_t>(a.B) * a.T;
  const void *in[3] = {a.x, a.r, a.g};
  const int64_t ld[3] = {a.ld_x, a.ld_r, a.ld_g};
  for (int i = 0; i < 3; ++i)
    if ((rc = launch_ckpt8_pack(in[i], ld[i], dtype, rows, a.D, a.lens, a.T, codes + i * rows * a.D,
                                exps + i * rows * ckpt8::groups(a.D), a.err, st)))
      return rc;
  return SDM_OK;
}

}  // namespace
}  // namespace sdm

using namespace sdm;

extern "C" int glr_scan(const float *state, float *state_out, const void *x, int64_t ld_x, const void *r, int64_t ld_r,
                        const void *g, int64_t ld_g, int dtype, const float *rate, const uint8_t *reset,
                        const int32_t *lens, int B, int T, int D, void *y, int32_t *dev_err, void *stream) {
  GlrArgs a{};
  a.state = state, a.state_out = state_out;
  a.x = x, a.r = r, a.g = g, a.ld_x = ld_x, a.ld_r = ld_r, a.ld_g = ld_g;
  a.rate = rate, a.reset = reset, a.lens = lens;
  a.B = B, a.T = T, a.D = D, a.y = y, a.err = dev_err;
  return forward("glr_scan", a, dtype, nullptr, nullptr, static_cast<cudaStream_t>(stream));
}

extern "C" size_t glr_scan_carry_size(int B, int T, int D) {
  if (check_sizes("glr_scan_carry_size", SDM_DTYPE_F32, B, T, D) != SDM_OK) return 0;
  return sizeof(float) * B * static_cast<size_t>((T + kSeg - 1) / kSeg) * D;
}

extern "C" int glr_scan_train(const float *state, float *state_out, const void *x, int64_t ld_x, const void *r,
                              int64_t ld_r, const void *g, int64_t ld_g, int dtype, const float *rate,
                              const uint8_t *reset, const int32_t *lens, int B, int T, int D, void *y, float *carry,
                              int8_t *codes, uint8_t *exps, int32_t *dev_err, void *stream) {
  if (T > 0 && B > 0 && D > 0 && !carry) return set_error(SDM_ERR_INVALID_ARG, "glr_scan_train: null pointer (carry)");
  if (!codes != !exps) return set_error(SDM_ERR_INVALID_ARG, "glr_scan_train: codes and exps go together");
  GlrArgs a{};
  a.state = state, a.state_out = state_out;
  a.x = x, a.r = r, a.g = g, a.ld_x = ld_x, a.ld_r = ld_r, a.ld_g = ld_g;
  a.rate = rate, a.reset = reset, a.lens = lens;
  a.B = B, a.T = T, a.D = D, a.y = y, a.err = dev_err;
  a.S = (T + kSeg - 1) / kSeg, a.carry = carry;
  return forward("glr_scan_train", a, dtype, codes, exps, static_cast<cudaStream_t>(stream));
}

extern "C" size_t glr_scan_backward_workspace_size(int B, int T, int D) {
  if (check_sizes("glr_scan_backward_workspace_size", SDM_DTYPE_F32, B, T, D) != SDM_OK) return 0;
  return (sizeof(float) * B * static_cast<size_t>(D) + 255) / 256 * 256;
}

extern "C" int glr_scan_backward(const float *dstate, float *dstate_out, const void *x, int64_t ld_x, const void *r,
                                 int64_t ld_r, const void *g, int64_t ld_g, const int8_t *codes, const uint8_t *exps,
                                 int dtype, const float *rate, const uint8_t *reset, const int32_t *lens,
                                 const float *carry, const void *dy, int B, int T, int D, void *dx, void *dr, void *dg,
                                 int64_t ld_d, float *drate, void *workspace, size_t workspace_bytes, int32_t *dev_err,
                                 void *stream) {
  const char *fn = "glr_scan_backward";
  int rc = check_sizes(fn, dtype, B, T, D);
  if (rc != SDM_OK) return rc;
  if (D == 0) return SDM_OK;
  if (!drate || !rate) return set_error(SDM_ERR_INVALID_ARG, "%s: null pointer", fn);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (B > 0) {
    if (!dstate_out) return set_error(SDM_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!codes != !exps) return set_error(SDM_ERR_INVALID_ARG, "%s: codes and exps go together", fn);
    if (codes && (x || r || g))
      return set_error(SDM_ERR_INVALID_ARG, "%s: give x, r and g or their checkpoints, not both", fn);
    if (T > 0) {
      if (!codes &&
          ((rc = check_rows(fn, "x", x, ld_x, dtype, D)) || (rc = check_rows(fn, "r", r, ld_r, dtype, D)) ||
           (rc = check_rows(fn, "g", g, ld_g, dtype, D))))
        return rc;
      if ((rc = check_rows(fn, "dy", dy, D, dtype, D)) || (rc = check_rows(fn, "dx", dx, ld_d, dtype, D)) ||
          (rc = check_rows(fn, "dr", dr, ld_d, dtype, D)) || (rc = check_rows(fn, "dg", dg, ld_d, dtype, D)))
        return rc;
      if (!carry) return set_error(SDM_ERR_INVALID_ARG, "%s: null pointer (carry)", fn);
    }
    const size_t need = glr_scan_backward_workspace_size(B, T, D);
    if (!workspace || workspace_bytes < need)
      return set_error(SDM_ERR_INVALID_ARG, "%s: workspace of %zu bytes needed", fn, need);
    if (!aligned(workspace, 16)) return set_error(SDM_ERR_ALIGN, "%s: workspace must be 16-byte aligned", fn);
  }
  if ((rc = check_words(fn, {dstate, dstate_out, rate, lens, carry, drate, dev_err}))) return rc;
  GlrArgs a{};
  a.state = dstate, a.state_out = dstate_out;
  a.x = x, a.r = r, a.g = g, a.ld_x = ld_x, a.ld_r = ld_r, a.ld_g = ld_g, a.ld_d = ld_d;
  a.codes = codes, a.exps = exps, a.rate = rate, a.reset = reset, a.lens = lens;
  a.B = B, a.T = T, a.D = D, a.S = (T + kSeg - 1) / kSeg;
  a.y = const_cast<void *>(dy), a.carry = const_cast<float *>(carry);
  a.dx = dx, a.dr = dr, a.dg = dg, a.part = static_cast<float *>(workspace), a.err = dev_err;
  if (B > 0) {
    const dim3 grid = grid_of(B, D);
    if (dtype == SDM_DTYPE_F32) {
      if (codes) glr_backward_kernel<float, true><<<grid, 128, 0, st>>>(a);
      else glr_backward_kernel<float, false><<<grid, 128, 0, st>>>(a);
    } else {
      if (codes) glr_backward_kernel<uint16_t, true><<<grid, 128, 0, st>>>(a);
      else glr_backward_kernel<uint16_t, false><<<grid, 128, 0, st>>>(a);
    }
    if ((rc = check_launch(fn))) return rc;
  }
  glr_rate_kernel<<<(D + 127) / 128, 128, 0, st>>>(a.part, B, D, drate);
  return check_launch(fn);
}
