// ckpt8.cu - activation checkpoints in 8 bits: pack and unpack.
//
// One warp per group of 64 channels, two channels a lane: the group's largest
// magnitude is one integer warp reduction over the absolute values' bits
// (which order as the values do), then one FMA and a byte per element.
#include "ckpt8.cuh"

namespace sdm {
namespace {

using ckpt8::kGroup;

__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t *p) { return bf16_to_f32(*p); }
// code * step is exact in bf16 (7 bits), so the upper half of the fp32 bits is it
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t *p, float v) { *p = static_cast<uint16_t>(__float_as_uint(v) >> 16); }

template <class E>
__global__ void __launch_bounds__(256) ckpt8_pack_kernel(const E *x, int64_t ld, int64_t rows, int D, int G,
                                                         int8_t *codes, uint8_t *exps, int32_t *err) {
  const int lane = threadIdx.x & 31;
  const int64_t total = rows * G;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  int bad = 0;
  for (int64_t w = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); w < total; w += warps) {
    const int64_t row = w / G;
    const int grp = static_cast<int>(w - row * G);
    const int c = grp * kGroup + 2 * lane;
    const E *p = x + row * ld + c;
    const float v0 = c < D ? load1(p) : 0.f, v1 = c + 1 < D ? load1(p + 1) : 0.f;
    const uint32_t a0 = __float_as_uint(v0) & 0x7fffffffu, a1 = __float_as_uint(v1) & 0x7fffffffu;
    const uint32_t byte = ckpt8::exp_byte(__reduce_max_sync(kFull, a0 > a1 ? a0 : a1));
    const float inv = ckpt8::inv_step(byte);
    int8_t *q = codes + row * D + c;
    if (c < D) q[0] = byte == 255u ? 0 : static_cast<int8_t>(ckpt8::code_bits(v0, inv));
    if (c + 1 < D) q[1] = byte == 255u ? 0 : static_cast<int8_t>(ckpt8::code_bits(v1, inv));
    if (lane == 0) exps[w] = static_cast<uint8_t>(byte);
    bad |= byte == 255u;
  }
  if (bad && lane == 0 && err) atomicOr(err, SDM_DEVERR_NONFINITE);
}

template <class E>
__global__ void __launch_bounds__(256) ckpt8_unpack_kernel(const int8_t *codes, const uint8_t *exps, int64_t rows,
                                                           int D, int G, E *x, int64_t ld) {
  const int lane = threadIdx.x & 31;
  const int64_t total = rows * G;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  for (int64_t w = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); w < total; w += warps) {
    const int64_t row = w / G;
    const int c = static_cast<int>(w - row * G) * kGroup + 2 * lane;
    const float s = ckpt8::step(exps[w]);
    const int8_t *q = codes + row * D + c;
    E *p = x + row * ld + c;
    if (c < D) store1(p, static_cast<float>(q[0]) * s);
    if (c + 1 < D) store1(p + 1, static_cast<float>(q[1]) * s);
  }
}

unsigned grid_for(int64_t warps) {
  const int64_t blocks = (warps + 7) / 8;
  return static_cast<unsigned>(blocks < 152 * 64 ? blocks : 152 * 64);
}

// arguments that both directions share
int check(const char *fn, const void *x, int64_t ld, int dtype, int64_t rows, int D, const void *codes,
          const void *exps) {
  if (rows < 0 || D < 0) return set_error(SDM_ERR_INVALID_ARG, "%s: negative size", fn);
  if (dtype != SDM_DTYPE_F32 && dtype != SDM_DTYPE_BF16) return set_error(SDM_ERR_UNSUPPORTED, "%s: unknown dtype", fn);
  if (D >= 1 << 24) return set_error(SDM_ERR_SHAPE, "%s: D must be below 2^24", fn);
  if (rows > INT64_MAX / (1 << 26)) return set_error(SDM_ERR_SHAPE, "%s: too many rows", fn);
  if (rows == 0 || D == 0) return SDM_OK;
  if (!x || !codes || !exps) return set_error(SDM_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (rows > 1 && (ld < D || ld >= int64_t(1) << 31)) return set_error(SDM_ERR_SHAPE, "%s: need D <= ld < 2^31", fn);
  if (!aligned(x, dtype == SDM_DTYPE_F32 ? 4 : 2)) return set_error(SDM_ERR_ALIGN, "%s: x must be aligned to its element", fn);
  return SDM_OK;
}

}  // namespace
}  // namespace sdm

using namespace sdm;

extern "C" int ckpt8_pack(const void *x, int64_t ld, int dtype, int64_t rows, int D, int8_t *codes, uint8_t *exps,
                          int32_t *dev_err, void *stream) {
  const int rc = check("ckpt8_pack", x, ld, dtype, rows, D, codes, exps);
  if (rc != SDM_OK || rows == 0 || D == 0) return rc;
  if (dev_err && !aligned(dev_err, 4)) return set_error(SDM_ERR_ALIGN, "ckpt8_pack: dev_err must be 4-byte aligned");
  const int G = ckpt8::groups(D);
  const unsigned grid = grid_for(rows * G);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == SDM_DTYPE_F32)
    ckpt8_pack_kernel<<<grid, 256, 0, st>>>(static_cast<const float *>(x), ld, rows, D, G, codes, exps, dev_err);
  else
    ckpt8_pack_kernel<<<grid, 256, 0, st>>>(static_cast<const uint16_t *>(x), ld, rows, D, G, codes, exps, dev_err);
  return check_launch("ckpt8_pack");
}

extern "C" int ckpt8_unpack(const int8_t *codes, const uint8_t *exps, int64_t rows, int D, void *x, int64_t ld,
                            int dtype, void *stream) {
  const int rc = check("ckpt8_unpack", x, ld, dtype, rows, D, codes, exps);
  if (rc != SDM_OK || rows == 0 || D == 0) return rc;
  const int G = ckpt8::groups(D);
  const unsigned grid = grid_for(rows * G);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == SDM_DTYPE_F32)
    ckpt8_unpack_kernel<<<grid, 256, 0, st>>>(codes, exps, rows, D, G, static_cast<float *>(x), ld);
  else
    ckpt8_unpack_kernel<<<grid, 256, 0, st>>>(codes, exps, rows, D, G, static_cast<uint16_t *>(x), ld);
  return check_launch("ckpt8_unpack");
}
