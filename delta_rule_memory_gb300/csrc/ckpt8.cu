// ckpt8.cu - activation checkpoints in 8 bits: pack and unpack.
//
// One pass over memory and little else: a group's largest magnitude is a
// maximum over the absolute values' bits (which order as the values do), then
// one FMA and a byte per element.  Where rows are aligned, a lane holds 8
// neighbouring channels (16 bytes of bf16, two of them for fp32), eight lanes a
// group, and the maximum is three shuffles; else a warp holds four neighbouring
// groups of a row, a lane every 32nd channel of them, and a group's maximum is
// one integer warp reduction.
#include <type_traits>

#include "ckpt8.cuh"

namespace sdm {
namespace {

using ckpt8::kGroup;

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }
__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t *p) { return bf16_to_f32(*p); }
// code * step is exact in bf16 (7 bits), so the upper half of the fp32 bits is it
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t *p, float v) { *p = static_cast<uint16_t>(__float_as_uint(v) >> 16); }

struct Eight {
  float v[8];
};
// eight neighbours as they are loaded
template <class E>
struct Raw;
template <>
struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float *p) {
    a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
  }
  __device__ __forceinline__ Eight eight() const { return Eight{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}}; }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t t = max(max(magnitude(a.x), magnitude(a.y)), max(magnitude(a.z), magnitude(a.w)));
    return max(max(t, max(magnitude(b.x), magnitude(b.y))), max(magnitude(b.z), magnitude(b.w)));
  }
};
template <>
struct Raw<uint16_t> {
  uint4 u;
  __device__ __forceinline__ void load(const uint16_t *p) { u = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ Eight eight() const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    Eight r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.v[2 * i] = __uint_as_float(w[i] << 16);
      r.v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    return r;
  }
  __device__ __forceinline__ uint32_t top() const {  // two magnitudes a word
    const uint32_t m = 0x7fff7fffu;
    const uint32_t t = __vmaxu2(__vmaxu2(u.x & m, u.y & m), __vmaxu2(u.z & m, u.w & m));
    return max(t & 0xffff0000u, t << 16);
  }
};
// one 32-byte store where p allows it: two of 16 bytes write every sector in halves
__device__ __forceinline__ void store8(float *p, const Eight &e) {
  if ((reinterpret_cast<uintptr_t>(p) & 31u) == 0) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(p), "f"(e.v[0]), "f"(e.v[1]),
                 "f"(e.v[2]), "f"(e.v[3]), "f"(e.v[4]), "f"(e.v[5]), "f"(e.v[6]), "f"(e.v[7])
                 : "memory");
    return;
  }
  *reinterpret_cast<float4 *>(p) = make_float4(e.v[0], e.v[1], e.v[2], e.v[3]);
  *reinterpret_cast<float4 *>(p + 4) = make_float4(e.v[4], e.v[5], e.v[6], e.v[7]);
}
__device__ __forceinline__ void store8(uint16_t *p, const Eight &e) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __byte_perm(__float_as_uint(e.v[2 * i]), __float_as_uint(e.v[2 * i + 1]), 0x7632);
  *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// The groups of all rows (or fours of them), G a row, numbered row by row, `on`
// at a time: one division at the start, of 32 bits where they suffice (64-bit
// ones took longer than the packing), then additions.
struct Step {
  int64_t groups;  // of all rows
  int64_t on, rows_on;
  int grps_on, G;
};
Step step_of(int64_t rows, int G, int64_t on) {
  return Step{rows * G, on, on / G, static_cast<int>(on % G), G};
}
// DENSE: the groups are whole and follow one another in x and in codes, so a
// group is as good as a row.
template <bool DENSE>
struct GroupWalk {
  int64_t row;
  int grp;
  __device__ __forceinline__ GroupWalk(int64_t first, const Step &s) {
    if (DENSE) {
      row = first, grp = 0;
    } else if (s.groups <= 0xffffffffll) {
      const uint32_t r = static_cast<uint32_t>(first) / static_cast<uint32_t>(s.G);
      row = r, grp = static_cast<int>(static_cast<uint32_t>(first) - r * s.G);
    } else {
      row = first / s.G, grp = static_cast<int>(first - row * s.G);
    }
  }
  __device__ __forceinline__ void next(const Step &s) {
    if (DENSE) {
      row += s.on;
    } else {
      row += s.rows_on, grp += s.grps_on;
      if (grp >= s.G) grp -= s.G, ++row;
    }
  }
};

// D a multiple of 8, x and its rows aligned to 16 bytes, codes to 8: eight
// threads hold a group, 8 elements each.  kFlight: groups of a thread at a time.  DENSE: whole
// groups with nothing between rows, so the tensor is one row of groups and a
// thread's next address a sum.  bf16 32,768 x 3840: 64 us, 88% of the measured copy
// bandwidth; the arithmetic (max, step, 8 roundings and a packing for 16 bytes)
// is what else the SMs do, and before DENSE it took 74 with four groups in flight and
// six CTAs an SM, 88 with two, 78 with four CTAs.
template <class E, int kFlight, bool DENSE>
__global__ void __launch_bounds__(256, sizeof(E) == 2 ? 6 : 4) pack8_kernel(const E *x, int64_t ld, int64_t rows, int D, const Step s,
                                                       int8_t *codes, uint8_t *exps, int32_t *err) {
  const int64_t thread = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int part = threadIdx.x & 7, G = DENSE ? 1 : s.G;
  if (DENSE) rows = s.groups, D = kGroup, ld = kGroup;
  GroupWalk<DENSE> ahead(thread >> 3, s), w = ahead;
  bool bad = false;
  // whole warps leave together: a warp's four groups are neighbours, and a group
  // behind the last row only skips its loads and stores
  for (int64_t first = (thread >> 5) * 4; first < s.groups; first += kFlight * s.on) {
    Raw<E> e[kFlight];
#pragma unroll
    for (int i = 0; i < kFlight; ++i, ahead.next(s)) {
      const int c = ahead.grp * kGroup + 8 * part;
      e[i] = Raw<E>{};
      if (ahead.row < rows && c < D) e[i].load(x + ahead.row * ld + c);
    }
#pragma unroll
    for (int i = 0; i < kFlight; ++i, w.next(s)) {
      uint32_t top = e[i].top();
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(kFull, top, o));
      const uint32_t byte = ckpt8::exp_byte(top);
      const float inv = ckpt8::inv_step(byte);
      const Eight v = e[i].eight();
      uint32_t q[8];
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const float2 c = __ffma2_rn(make_float2(v.v[j], v.v[j + 1]), make_float2(inv, inv), make_float2(12582912.f, 12582912.f));
        q[j] = __float_as_uint(c.x), q[j + 1] = __float_as_uint(c.y);
      }
      uint2 u;
      u.x = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
      u.y = __byte_perm(__byte_perm(q[4], q[5], 0x0040), __byte_perm(q[6], q[7], 0x0040), 0x5410);
      if (byte == 255u) u = make_uint2(0, 0);
      const int c = w.grp * kGroup + 8 * part;
      if (w.row < rows && c < D) {
        *reinterpret_cast<uint2 *>(codes + w.row * D + c) = u;
        bad |= byte == 255u;
        if (part == 0) exps[w.row * G + w.grp] = static_cast<uint8_t>(byte);
      }
    }
  }
  if (bad && err) atomicOr(err, SDM_DEVERR_NONFINITE);
}

template <class E, int kFlight, bool DENSE>
__global__ void __launch_bounds__(256) unpack8_kernel(const int8_t *codes, const uint8_t *exps, int64_t rows, int D,
                                                      const Step st, E *x, int64_t ld) {
  const int64_t thread = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int part = threadIdx.x & 7, G = DENSE ? 1 : st.G;
  if (DENSE) rows = st.groups, D = kGroup, ld = kGroup;
  GroupWalk<DENSE> w(thread >> 3, st);
  while (w.row < rows) {
    uint2 u[kFlight];
    uint32_t byte[kFlight];
    int64_t row[kFlight];
    int c[kFlight];
    bool in[kFlight];
#pragma unroll
    for (int i = 0; i < kFlight; ++i, w.next(st)) {
      row[i] = w.row, c[i] = w.grp * kGroup + 8 * part;
      in[i] = w.row < rows && c[i] < D;
      u[i] = make_uint2(0, 0), byte[i] = 1;
      if (in[i]) u[i] = *reinterpret_cast<const uint2 *>(codes + row[i] * D + c[i]), byte[i] = exps[row[i] * G + w.grp];
    }
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      const float s = ckpt8::step(byte[i]);
      const float2 a = ckpt8::decode2(u[i].x, s), b = ckpt8::decode2(u[i].x >> 16, s);
      const float2 d = ckpt8::decode2(u[i].y, s), f = ckpt8::decode2(u[i].y >> 16, s);
      if (in[i]) store8(x + row[i] * ld + c[i], Eight{{a.x, a.y, b.x, b.y, d.x, d.y, f.x, f.y}});
    }
  }
}

// any alignment; s counts fours of groups.  fp32 8193 x 1955: 22.5 us and 20.5 (floor 12),
// bound by the instructions of single channels.
constexpr int kFour = 4 * kGroup;
template <class E>
__global__ void __launch_bounds__(256) pack1_kernel(const E *x, int64_t ld, int64_t rows, int D, const Step s,
                                                    int8_t *codes, uint8_t *exps, int32_t *err) {
  const int lane = threadIdx.x & 31, G = ckpt8::groups(D);
  bool bad = false;
  for (GroupWalk<false> w((static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) >> 5, s); w.row < rows; w.next(s)) {
    const int c = w.grp * kFour + lane, left = D - c;  // w is the same in the whole warp
    const E *p = x + w.row * ld + c;
    int8_t *q = codes + w.row * D + c;
    auto four = [&](auto whole) {  // whole: no channel of the four is missing
      auto has = [&](int j) { return decltype(whole)::value || 32 * j < left; };
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = has(j) ? load1(p + 32 * j) : 0.f;
      uint32_t bytes = 0;  // lane i: group i's
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t byte = ckpt8::exp_byte(__reduce_max_sync(kFull, max(magnitude(v[2 * i]), magnitude(v[2 * i + 1]))));
        const float inv = ckpt8::inv_step(byte);
        if (lane == i) bytes = byte;
#pragma unroll
        for (int j = 2 * i; j < 2 * i + 2; ++j)
          if (has(j)) q[32 * j] = byte == 255u ? 0 : static_cast<int8_t>(ckpt8::code_bits(v[j], inv));
      }
      if (lane < 4 && (decltype(whole)::value || 4 * w.grp + lane < G)) {
        exps[w.row * G + 4 * w.grp + lane] = static_cast<uint8_t>(bytes);
        bad |= bytes == 255u;
      }
    };
    if (D - w.grp * kFour >= kFour) four(std::true_type{});
    else four(std::false_type{});
  }
  if (bad && err) atomicOr(err, SDM_DEVERR_NONFINITE);
}

template <class E>
__global__ void __launch_bounds__(256) unpack1_kernel(const int8_t *codes, const uint8_t *exps, int64_t rows, int D,
                                                      const Step s, E *x, int64_t ld) {
  const int lane = threadIdx.x & 31, G = ckpt8::groups(D);
  for (GroupWalk<false> w((static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) >> 5, s); w.row < rows; w.next(s)) {
    const int c = w.grp * kFour + lane, left = D - c;
    const int8_t *q = codes + w.row * D + c;
    E *p = x + w.row * ld + c;
    auto four = [&](auto whole) {
      auto has = [&](int j) { return decltype(whole)::value || 32 * j < left; };
      uint32_t v[8];  // code + 128: below 2^23 + 128 as the low bits of a float
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = has(j) ? static_cast<uint8_t>(q[32 * j]) ^ 0x80u : 0u;
      const uint32_t bytes =
          lane < 4 && (decltype(whole)::value || 4 * w.grp + lane < G) ? exps[w.row * G + 4 * w.grp + lane] : 1;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float step = ckpt8::step(__shfl_sync(kFull, bytes, i));
#pragma unroll
        for (int j = 2 * i; j < 2 * i + 2; ++j)
          if (has(j)) store1(p + 32 * j, (__uint_as_float(v[j] | 0x4b000000u) - 8388736.f) * step);
      }
    };
    if (D - w.grp * kFour >= kFour) four(std::true_type{});
    else four(std::false_type{});
  }
}

// CTAs for `units` of work, `at_once` of them a CTA: a GPU full of CTAs, and
// beyond that as many as give each thread `flight` units
unsigned grid_for(int64_t units, int at_once, int flight) {
  constexpr int kFull = 152 * 8;
  const int64_t most = (units + at_once - 1) / at_once, wanted = (most + flight - 1) / flight;
  const int64_t blocks = wanted > kFull ? wanted : most < kFull ? most : kFull;
  return static_cast<unsigned>(blocks < INT32_MAX ? blocks : INT32_MAX);
}
bool small(int64_t groups) { return groups <= 32 * 152 * 8; }  // one group a thread

// arguments that both directions share
int check(const char *fn, const void *x, int64_t ld, int dtype, int64_t rows, int D, const void *codes,
          const void *exps) {
  if (rows < 0 || D < 0) return set_error(SDM_ERR_INVALID_ARG, "%s: negative size", fn);
  if (dtype != SDM_DTYPE_F32 && dtype != SDM_DTYPE_BF16) return set_error(SDM_ERR_UNSUPPORTED, "%s: unknown dtype", fn);
  if (D >= 1 << 24) return set_error(SDM_ERR_SHAPE, "%s: D must be below 2^24", fn);
  if (rows >= int64_t(1) << 36) return set_error(SDM_ERR_SHAPE, "%s: rows must be below 2^36", fn);
  if (rows == 0 || D == 0) return SDM_OK;
  if (!x || !codes || !exps) return set_error(SDM_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (rows > 1 && (ld < D || ld >= 1 << 27)) return set_error(SDM_ERR_SHAPE, "%s: need D <= ld < 2^27", fn);
  if (!aligned(x, dtype == SDM_DTYPE_F32 ? 4 : 2)) return set_error(SDM_ERR_ALIGN, "%s: x must be aligned to its element", fn);
  return SDM_OK;
}

bool wide(const void *x, int64_t ld, int dtype, int64_t rows, int D, const void *codes) {
  return D % 8 == 0 && aligned(x, 16) && aligned(codes, 8) && (rows == 1 || ld * (dtype == SDM_DTYPE_F32 ? 4 : 2) % 16 == 0);
}

bool dense(int64_t ld, int64_t rows, int D) { return D % kGroup == 0 && (rows == 1 || ld == D); }

template <class E>
void launch_pack(const void *x, int64_t ld, int dtype, int64_t rows, int D, int8_t *codes, uint8_t *exps, int32_t *err,
                 cudaStream_t st) {
  const int G = ckpt8::groups(D);
  const E *p = static_cast<const E *>(x);
  if (wide(x, ld, dtype, rows, D, codes)) {
    const bool one = small(rows * G), flat = dense(ld, rows, D);
    const unsigned grid = grid_for(rows * G, 32, one ? 1 : 4);
    const Step s = step_of(rows, G, static_cast<int64_t>(grid) * 32);
    if (one && flat) pack8_kernel<E, 1, true><<<grid, 256, 0, st>>>(p, ld, rows, D, s, codes, exps, err);
    else if (one) pack8_kernel<E, 1, false><<<grid, 256, 0, st>>>(p, ld, rows, D, s, codes, exps, err);
    else if (flat) pack8_kernel<E, 4, true><<<grid, 256, 0, st>>>(p, ld, rows, D, s, codes, exps, err);
    else pack8_kernel<E, 4, false><<<grid, 256, 0, st>>>(p, ld, rows, D, s, codes, exps, err);
  } else {
    const int U = (G + 3) / 4;
    const unsigned grid = grid_for(rows * U, 8, 1);
    pack1_kernel<<<grid, 256, 0, st>>>(p, ld, rows, D, step_of(rows, U, static_cast<int64_t>(grid) * 8), codes, exps, err);
  }
}

template <class E>
void launch_unpack(const int8_t *codes, const uint8_t *exps, int64_t rows, int D, void *x, int64_t ld, int dtype,
                   cudaStream_t st) {
  const int G = ckpt8::groups(D);
  E *p = static_cast<E *>(x);
  if (wide(x, ld, dtype, rows, D, codes)) {
    const bool one = small(rows * G), flat = dense(ld, rows, D);
    const unsigned grid = grid_for(rows * G, 32, one ? 1 : 2);
    const Step s = step_of(rows, G, static_cast<int64_t>(grid) * 32);
    if (one && flat) unpack8_kernel<E, 1, true><<<grid, 256, 0, st>>>(codes, exps, rows, D, s, p, ld);
    else if (one) unpack8_kernel<E, 1, false><<<grid, 256, 0, st>>>(codes, exps, rows, D, s, p, ld);
    else if (flat) unpack8_kernel<E, 2, true><<<grid, 256, 0, st>>>(codes, exps, rows, D, s, p, ld);
    else unpack8_kernel<E, 2, false><<<grid, 256, 0, st>>>(codes, exps, rows, D, s, p, ld);
  } else {
    const int U = (G + 3) / 4;
    const unsigned grid = grid_for(rows * U, 8, 1);
    unpack1_kernel<<<grid, 256, 0, st>>>(codes, exps, rows, D, step_of(rows, U, static_cast<int64_t>(grid) * 8), p, ld);
  }
}

}  // namespace
}  // namespace sdm

using namespace sdm;

extern "C" int ckpt8_pack(const void *x, int64_t ld, int dtype, int64_t rows, int D, int8_t *codes, uint8_t *exps,
                          int32_t *dev_err, void *stream) {
  const int rc = check("ckpt8_pack", x, ld, dtype, rows, D, codes, exps);
  if (rc != SDM_OK || rows == 0 || D == 0) return rc;
  if (dev_err && !aligned(dev_err, 4)) return set_error(SDM_ERR_ALIGN, "ckpt8_pack: dev_err must be 4-byte aligned");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == SDM_DTYPE_F32) launch_pack<float>(x, ld, dtype, rows, D, codes, exps, dev_err, st);
  else launch_pack<uint16_t>(x, ld, dtype, rows, D, codes, exps, dev_err, st);
  return check_launch("ckpt8_pack");
}

extern "C" int ckpt8_unpack(const int8_t *codes, const uint8_t *exps, int64_t rows, int D, void *x, int64_t ld,
                            int dtype, void *stream) {
  const int rc = check("ckpt8_unpack", x, ld, dtype, rows, D, codes, exps);
  if (rc != SDM_OK || rows == 0 || D == 0) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == SDM_DTYPE_F32) launch_unpack<float>(codes, exps, rows, D, x, ld, dtype, st);
  else launch_unpack<uint16_t>(codes, exps, rows, D, x, ld, dtype, st);
  return check_launch("ckpt8_unpack");
}
