// mma.cuh - warp-level bf16 matrix products (mma.sync m16n8k16, fp32 sums) on shared-memory tiles, for chains
// whose operands stay in registers.
//
// A tile has 64 rows in panels of 64 columns, each panel row-major with rows of 128 bytes and aligned to 1024;
// the 16-byte piece p of a panel's row r lies at piece p ^ (r & 7), so the eight rows that one ldmatrix phase
// reads lie in different banks (the layout that a tensor copy with the 128-byte swizzle writes).
//
// Fragments (g = lane / 4, t = lane % 4): the accumulator of an m16n8 product holds rows g and g + 8, columns
// 2t and 2t + 1.  Two neighbouring ones are, as they stand, the A fragment of a k = 16 step, so a product's
// result feeds the next product without leaving the registers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "umma.cuh"

namespace sdm {
namespace mma {

using umma::ldsm_x4_trans;

constexpr int kPanel = 64 * 128;

// byte offset of 16-byte piece p (of all panels) of row r
__device__ __forceinline__ uint32_t piece(int r, int p) {
  return static_cast<uint32_t>((p >> 3) * kPanel + r * 128 + (((p & 7) ^ (r & 7)) << 4));
}

__device__ __forceinline__ void ldsm4(uint32_t saddr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(saddr)
               : "memory");
}

// B fragments of two n-tiles (n0 .. n0+15) and one k-step from tile[n][k]: r[0], r[1] of the first, r[2], r[3]
// of the second
__device__ __forceinline__ void b_rows(uint32_t tile, int n0, int k0, int lane, uint32_t (&r)[4]) {
  ldsm4(tile + piece(n0 + ((lane >> 4) << 3) + (lane & 7), (k0 >> 3) + ((lane >> 3) & 1)), r);
}
// the same from tile[k][n]
__device__ __forceinline__ void b_cols(uint32_t tile, int n0, int k0, int lane, uint32_t (&r)[4]) {
  ldsm_x4_trans(tile + piece(k0 + (((lane >> 3) & 1) << 3) + (lane & 7), (n0 >> 3) + (lane >> 4)), r);
}
// A fragment (rows m0 .. m0+15, one k-step) from tile[m][k] ...
__device__ __forceinline__ void a_rows(uint32_t tile, int m0, int k0, int lane, uint32_t (&r)[4]) {
  ldsm4(tile + piece(m0 + (((lane >> 3) & 1) << 3) + (lane & 7), (k0 >> 3) + (lane >> 4)), r);
}
// ... and from tile[k][m]
__device__ __forceinline__ void a_cols(uint32_t tile, int m0, int k0, int lane, uint32_t (&r)[4]) {
  ldsm_x4_trans(tile + piece(k0 + ((lane >> 4) << 3) + (lane & 7), (m0 >> 3) + ((lane >> 3) & 1)), r);
}

// d += a b
__device__ __forceinline__ void fma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ float low2(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float high2(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// x = s[0] + s[1] + ... in bf16, each the rounding of what the ones before leave: two parts keep 16 bits of x,
// three keep all 24 (to 2^-26 relative) as long as they are not below bf16's least step: to 2^-134 absolute.
template <int N>
__device__ __forceinline__ void split(float x0, float x1, uint32_t (&s)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    s[i] = pack2(x0, x1);
    if (i + 1 < N) {
      x0 -= low2(s[i]);
      x1 -= high2(s[i]);
    }
  }
}

// The A fragments, in N parts, of one k-step of an accumulator's columns: c0 and c1 are its n-tiles 2 ks and 2
// ks + 1.  a[part][register].
template <int N>
__device__ __forceinline__ void a_split(const float (&c0)[4], const float (&c1)[4], uint32_t (&a)[N][4]) {
  uint32_t s[N];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i < 2)
      split<N>(c0[2 * i], c0[2 * i + 1], s);
    else
      split<N>(c1[2 * i - 4], c1[2 * i - 3], s);
#pragma unroll
    for (int n = 0; n < N; ++n) a[n][i] = s[n];
  }
}

// transposes an 8x8 matrix of 16-bit elements held one row per four lanes
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(d) : "r"(v));
  return d;
}

// BYTES (4, 8 or 16) global -> shared, asynchronously; zeros where `live` is false (src then only has to be a
// valid address)
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src, bool live) {
  const int n = live ? BYTES : 0;
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;\n" ::"r"(dst), "l"(src), "n"(BYTES), "r"(n) : "memory");
}

template <int PANELS, int THREADS, int BYTES>
__device__ __forceinline__ void load_tile_by(unsigned char *tile, const uint16_t *src, int64_t ld, int live, int width,
                                             int tid) {
  constexpr int pieces = PANELS * 128 / BYTES;
  const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(tile));
#pragma unroll 8
  for (int i = 0; i < 64 * pieces / THREADS; ++i) {
    const int id = tid + i * THREADS, r = id / pieces, p = id % pieces;
    const bool ok = r < live && p * (BYTES / 2) < width;
    copy_async<BYTES>(base + piece(r, p * BYTES / 16) + p * BYTES % 16, ok ? src + r * ld + p * (BYTES / 2) : src, ok);
  }
}

// 64 rows of `width` bf16 (row r at src + r * ld) into a tile, zeros behind `width` and from row `live` on, by
// THREADS threads (a power of two).  bytes: what divides the address, the distance and the width of every row
// (8 or 4: asynchronous copies of that size; else by elements).  Where it is 16, a tensor copy does the same.
template <int PANELS, int THREADS>
__device__ __forceinline__ void load_tile(unsigned char *tile, const uint16_t *src, int64_t ld, int live, int width,
                                          int bytes, int tid) {
  if (bytes >= 8) {
    load_tile_by<PANELS, THREADS, 8>(tile, src, ld, live, width, tid);
  } else if (bytes == 4) {
    load_tile_by<PANELS, THREADS, 4>(tile, src, ld, live, width, tid);
  } else {
    constexpr int pieces = PANELS * 8;
    for (int id = tid; id < 64 * pieces; id += THREADS) {
      const int r = id / pieces, c = id % pieces * 8;
      uint32_t w[4] = {0, 0, 0, 0};
      if (r < live) {
        const uint16_t *s = src + r * ld + c;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c + e < width) w[e >> 1] |= static_cast<uint32_t>(s[e]) << (16 * (e & 1));
      }
      *reinterpret_cast<uint4 *>(tile + piece(r, c / 8)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// rows `live` .. 63 of a tile to zero
template <int PANELS, int THREADS>
__device__ __forceinline__ void clear_rows(unsigned char *tile, int live, int tid) {
  for (int id = live * PANELS * 8 + tid; id < 64 * PANELS * 8; id += THREADS)
    *reinterpret_cast<uint4 *>(tile + piece(id / (PANELS * 8), id % (PANELS * 8))) = make_uint4(0, 0, 0, 0);
}

// a panel of a tensor map's [token][head][channel] (box: 64 tokens, one head, 64 channels), by one thread;
// completes its 8 KB on the mbarrier.  channel: a multiple of 64
__device__ __forceinline__ void tensor_panel(uint32_t dst, const void *map, int channel, int head, int token,
                                             uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];\n" ::"r"(dst),
      "l"(map), "r"(channel), "r"(head), "r"(token), "r"(mbar)
      : "memory");
}

}  // namespace mma
}  // namespace sdm
