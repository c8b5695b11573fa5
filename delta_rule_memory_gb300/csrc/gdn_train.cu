// gdn_train.cu - training of the gated delta rule: the chunked forward that
// keeps what its backward needs, and the backward.
//
// Per sequence and head, S [dk, dv]:
//   S~ = e^{a_t} S (0 at a reset),  E_t = v_t - S~^T k_t,
//   S_t = S~ + beta_t k_t E_t^T,    y_t = S_t^T q_t.
// In a chunk of C = 64 tokens let l_i be the sum of the a's up to token i,
// D_ij = e^{l_i - l_j} for j <= i in one document (else 0), gam_i = D from the
// chunk's start (0 behind a reset), tail_j = D to its end.  With S the state at the
// chunk's start, rows being tokens,
//   Z = V - gam K S,   E = T Z,   T = (I + strict(D o K K^T) diag(beta))^-1,
//   U = beta E,   Y = gam Q S + M U,   M = D o Q K^T,
//   S_end = gam_C S + K^T (tail U).
// Backward, G being the gradient of the state at the chunk's end:
//   dU = M^T dY + tail K G,   dZ = T^T (beta dU),   dV = dZ,
//   G_start = gam_C G + Q^T (gam dY) - K^T (gam dZ),
//   dbeta = (dZ . E) / beta   (dZ is beta times the gradient of beta Z),
//   X = D o dY U^T,   N = -strict(D) o dZ U^T,
//   dQ = gam dY S^T + X K,
//   dK = tail U G^T - gam dZ S^T + X^T Q + (N + N^T) K.
// The decays' gradient needs no product of its own.  y and S_end are linear in
// (S, V), so at every cut the gradient's inner product with the state behind it plus that with the
// values to come is that of the outputs to come; with y_t . dy_t = q_t . dq_t:
//   da_t = <S, G_start> - sum over s < t of (q_s . dq_s - v_s . dv_s)
// (the first term only before the chunk's first reset, the sum from the document's start on).
//
// Kernels.  gdn_prep (every chunk by itself): the decays, T and M.  gdn_chain:
// chunk after chunk, a warp owns 16 value columns and keeps S^T [16, dk] in its
// accumulators; every product of a chunk takes the one before as its A operand
// from registers (mma.cuh), so warps never wait for one another and only the chunk's
// tiles, which are copied a chunk ahead, are shared.  gdn_chain_back: the same
// with G, last chunk to first.  gdn_grad: everything that needs sums over the value columns,
// every chunk by itself.
// mma.sync and not tcgen05: a product here is 64 x 128 x 16..128 and feeds the next one; through tensor
// memory each would be read back, split into bf16 parts and stored for the next,
// which is what bounds the chunk form in gdn_chunk.cu (2.85 us a chunk).
//
// Precision.  q, k, v and dy are exact in bf16.  What is not (S, G, T, M, Z, U, X) is taken in
// three bf16 parts, all 24 bits of it, wherever the result reaches an fp32 output (the states, da, dbeta); in two parts,
// 16 bits, where it only reaches y or dk, which are rounded to bf16's 8.
#include <cuda.h>

#include <algorithm>
#include <climits>

#include "common.cuh"
#include "mma.cuh"
#include "umma.cuh"

namespace sdm {
namespace {

using namespace mma;

constexpr int kSms = 152;
constexpr int kC = 64;                  // tokens of a chunk
constexpr int kTile = kPanel;           // bytes of one bf16 [64][64] tile
constexpr int kTri = 10 * 512;          // ... of a lower triangular one: its ten 16 x 16 blocks
constexpr int kLd = kC + 4;             // fp32 rows of the solve: 16-byte aligned, 4 banks apart
constexpr int kScal = 6 * kC;           // gam, tail, beta, l (two floats), document number
constexpr float kTinyBeta = 1e-18f;     // stands for a smaller |beta|, so that dZ / beta is the limit
constexpr float kLeastLog = -200.f;     // e^-200 is 0 in fp32

struct Gdn {
  const uint16_t *q, *k, *v, *dy;
  int64_t ld_q, ld_k, ld_v, ld_dq, ld_dk, ld_dv;  // elements between tokens
  const float *la, *beta;
  const uint8_t *reset;
  const int32_t *lens;
  int B, T, Hk, H, dk, dv, n;  // n: chunks of a sequence
  int by_qk, by_v, by_dy;      // bytes by which rows of q and k / v / dy can be copied (load_tile)
  int pair_y, pair_qk;         // y (or dv) / dq and dk can be written by pairs
  float *scal;                 // [units][kScal]
  unsigned char *t3, *m3;      // [units][3] triangles
  float *s;                    // [units][16-column tiles][dk tiles of 8][lane][4]: S at the chunk's start
  float *e;                    // [units][tiles][token tiles of 8][lane][4]: E
  float *g;                    // as s, n + 1 a sequence: G at chunk c's start, G_T behind the last
  float *dz;                   // as e: dZ
  const float *state_in;
  float *state_out;
  uint16_t *y, *odq, *odk, *odv;
  float *dla, *dbeta;
  float *pdq, *pdk;            // [B,T,H,dk] where several heads share a key head
  int32_t *err;
};

// A triangle: 16 x 16 blocks row by row, each as four 8 x 8 of 8 rows of 16 bytes
__device__ __forceinline__ constexpr int block_at(int i, int j) { return (i * (i + 1) / 2 + j) * 512; }
// B fragments (two n-tiles, one k-step) of block (n, k), B[k][n] = tri[n][k] ...
__device__ __forceinline__ void tri_rows(uint32_t tri, int n, int k, int lane, uint32_t (&r)[4]) {
  ldsm4(tri + block_at(n, k) + lane * 16, r);
}
// ... and of block (k, n), B[k][n] = tri[k][n]
__device__ __forceinline__ void tri_cols(uint32_t tri, int n, int k, int lane, uint32_t (&r)[4]) {
  ldsm4_t(tri + block_at(k, n) + ((lane & 8) << 5) + ((lane & 16) << 3) + (lane & 7) * 16, r);
}

// A sum of many terms as two floats: to about 2^-46 of the largest partial sum
struct Wide {
  float hi, lo;
};
__device__ __forceinline__ Wide operator+(Wide a, Wide b) {
  const float s = a.hi + b.hi, d = s - a.hi;
  const float l = ((a.hi - (s - d)) + (b.hi - d)) + (a.lo + b.lo), hi = s + l;
  return {hi, l - (hi - s)};
}
__device__ __forceinline__ Wide operator-(Wide a, Wide b) { return a + Wide{-b.hi, -b.lo}; }
__device__ __forceinline__ Wide shfl(Wide x, int lane) {
  return {__shfl_sync(kFull, x.hi, lane), __shfl_sync(kFull, x.lo, lane)};
}
// sums up to each of a warp's lanes
__device__ __forceinline__ Wide running(Wide x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Wide y{__shfl_up_sync(kFull, x.hi, o), __shfl_up_sync(kFull, x.lo, o)};
    if (lane >= o) x = y + x;
  }
  return x;
}

// Tensor maps of q, k, v and dy as [token][head][channel], boxes of one panel;
// set where rows can be copied by 16 bytes
struct Maps {
  CUtensorMap q, k, v, dy;
};

constexpr uint32_t kWaitLimit = 1u << 20;  // polls (about 0.1 s) before a wait gives up

// Wait for a phase of copies.  One that gives up is reported and lets the
// kernel run out, its later waits short.
__device__ __forceinline__ void wait_copies(uint64_t *bar, uint32_t parity, uint32_t &limit, const Gdn &a) {
  if (!umma::mbar_wait(smem_u32(bar), parity, limit)) {
    report_timeout(a.err);
    limit = 64;
  }
}

__device__ __forceinline__ int length_of(const Gdn &a, int b) {
  return a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
}

// ---------------------------------------------------------------------------
// gdn_prep: decays, M and T of one chunk of one head.
// ---------------------------------------------------------------------------
constexpr int kPrepThreads = 128;
static_assert(2 * kC * kLd * 4 >= 4 * kPanel, "the tiles fit where L and X will be");

__device__ __forceinline__ void store_parts3(unsigned char *tiles, uint32_t off, const float *x) {
  uint32_t s[4][3];
#pragma unroll
  for (int i = 0; i < 4; ++i) split<3>(x[2 * i], x[2 * i + 1], s[i]);
#pragma unroll
  for (int p = 0; p < 3; ++p)
    *reinterpret_cast<uint4 *>(tiles + p * kTri + off) = make_uint4(s[0][p], s[1][p], s[2][p], s[3][p]);
}

// the lower blocks of an fp32 [64][kLd] matrix as three triangles
__device__ __forceinline__ void write_tiles(const float *x, unsigned char *tiles, int tid) {
  for (int id = tid; id < kC * 8; id += kPrepThreads) {
    const int i = id >> 3, p = id & 7;
    if (p > 2 * (i >> 4) + 1) continue;
    float v[8];
    *reinterpret_cast<float4 *>(v) = *reinterpret_cast<const float4 *>(x + i * kLd + p * 8);
    *reinterpret_cast<float4 *>(v + 4) = *reinterpret_cast<const float4 *>(x + i * kLd + p * 8 + 4);
    store_parts3(tiles, block_at(i >> 4, p >> 1) + ((i >> 3) & 1) * 256 + (p & 1) * 128 + (i & 7) * 16, v);
  }
}

// out[0..R)[0..4) = sum_k a[r][k] b[k][0..4)
template <int R, int K>
__device__ __forceinline__ void strip(const float *a, int lda, const float *b, int ldb, float (&acc)[R][4]) {
#pragma unroll
  for (int r = 0; r < R; ++r) acc[r][0] = acc[r][1] = acc[r][2] = acc[r][3] = 0.f;
#pragma unroll 4
  for (int k = 0; k < K; k += 4) {
    float4 bv[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) bv[e] = *reinterpret_cast<const float4 *>(b + (k + e) * ldb);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float4 av = *reinterpret_cast<const float4 *>(a + r * lda + k);
      const float aa[4] = {av.x, av.y, av.z, av.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc[r][0] = fmaf(aa[e], bv[e].x, acc[r][0]);
        acc[r][1] = fmaf(aa[e], bv[e].y, acc[r][1]);
        acc[r][2] = fmaf(aa[e], bv[e].z, acc[r][2]);
        acc[r][3] = fmaf(aa[e], bv[e].w, acc[r][3]);
      }
    }
  }
}

// X = L^-1 for unit lower triangular L: the 16 x 16 diagonal blocks by
// substitution (one a warp), then blocks joined two by two,
// X21 = -X22 (L21 X11).  zt: 32 x 36 floats.
__device__ __forceinline__ void invert(const float *L, float *X, float *zt, int tid) {
  const int w = tid >> 5, lane = tid & 31;
  if (lane < 16) {
    const int o = 16 * w;
    float x[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      float acc = r == lane ? 1.f : 0.f;
#pragma unroll
      for (int j = 0; j < r; ++j) acc = fmaf(-L[(o + r) * kLd + o + j], x[j], acc);
      x[r] = acc;
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) X[(o + r) * kLd + o + lane] = x[r];
  } else if (w % 2 == 0) {  // the block right of the diagonal, which the second joining reads
#pragma unroll
    for (int r = 0; r < 16; ++r) X[(16 * w + r) * kLd + 16 * w + lane] = 0.f;
  }
  __syncthreads();
  {  // 16 -> 32: two pairs, 64 threads each, a row's four columns a thread
    const int pr = tid >> 6, r = (tid >> 2) & 15, c = (tid & 3) * 4, o = 32 * pr;
    float acc[1][4];
    strip<1, 16>(L + (o + 16 + r) * kLd + o, kLd, X + o * kLd + o + c, kLd, acc);
    float *z = zt + pr * 16 * 20;
    *reinterpret_cast<float4 *>(z + r * 20 + c) = make_float4(acc[0][0], acc[0][1], acc[0][2], acc[0][3]);
    __syncthreads();
    strip<1, 16>(X + (o + 16 + r) * kLd + o + 16, kLd, z + c, 20, acc);
    *reinterpret_cast<float4 *>(X + (o + 16 + r) * kLd + o + c) = make_float4(-acc[0][0], -acc[0][1], -acc[0][2], -acc[0][3]);
  }
  __syncthreads();
  {  // 32 -> 64
    const int r = (tid >> 3) * 2, c = (tid & 7) * 4;
    float acc[2][4];
    strip<2, 32>(L + (32 + r) * kLd, kLd, X + c, kLd, acc);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<float4 *>(zt + (r + i) * 36 + c) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
    __syncthreads();
    strip<2, 32>(X + (32 + r) * kLd + 32, kLd, zt + c, 36, acc);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<float4 *>(X + (32 + r + i) * kLd + c) = make_float4(-acc[i][0], -acc[i][1], -acc[i][2], -acc[i][3]);
  }
  __syncthreads();
}

// one thread: tensor copies of K and Q, and `more` bytes of its own to come
template <int NK>
__device__ __forceinline__ void load_qk(const Maps &maps, unsigned char *sK, unsigned char *sQ, int hk, int64_t tok,
                                        uint32_t bar, uint32_t more) {
  umma::mbar_expect_tx(bar, 2 * (NK / 4) * kPanel + more);
#pragma unroll
  for (int p = 0; p < NK / 4; ++p) {
    tensor_panel(smem_u32(sK) + p * kPanel, &maps.k, 64 * p, hk, static_cast<int>(tok), bar);
    tensor_panel(smem_u32(sQ) + p * kPanel, &maps.q, 64 * p, hk, static_cast<int>(tok), bar);
  }
}

template <int NK>
__global__ void __launch_bounds__(kPrepThreads) gdn_prep(const Gdn a, const __grid_constant__ Maps maps) {
  constexpr int panels = NK / 4;
  extern __shared__ __align__(1024) unsigned char sm[];
  unsigned char *sK = sm, *sQ = sm + panels * kPanel;
  // L and X take the tiles' place once the products are formed
  float *sL = reinterpret_cast<float *>(sm), *sX = sL + kC * kLd, *zt = sX + kC * kLd, *sc = zt + 32 * 36;
  uint64_t *bar = reinterpret_cast<uint64_t *>(sc + kScal);
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int64_t u = blockIdx.x;
  const int64_t bh = u / a.n;
  const int c = static_cast<int>(u - bh * a.n), b = static_cast<int>(bh / a.H), h = static_cast<int>(bh % a.H);
  const int live = min(length_of(a, b) - c * kC, kC);
  if (live <= 0) return;
  const int64_t tok = static_cast<int64_t>(b) * a.T + c * kC;
  const int hk = h / (a.H / a.Hk);
  if (a.by_qk == 16) {
    if (tid == 0) {
      umma::mbar_init(smem_u32(bar), 1);
      umma::fence_mbar_init();
      load_qk<NK>(maps, sK, sQ, hk, tok, smem_u32(bar), 0);
    }
  } else {
    load_tile<panels, kPrepThreads>(sK, a.k + tok * a.ld_k + hk * a.dk, a.ld_k, live, a.dk, a.by_qk, tid);
    load_tile<panels, kPrepThreads>(sQ, a.q + tok * a.ld_q + hk * a.dk, a.ld_q, live, a.dk, a.by_qk, tid);
    cp_async_commit();
  }
  float *out = a.scal + u * kScal;
  if (w == 0) {
    // l in units of log2, as two floats: a strong decay early in the chunk costs
    // the later, weak ones nothing
    Wide x[2];
    bool r[2];
    float be[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int m = lane + 32 * i;
      const bool ok = m < live;
      float la = ok ? a.la[(tok + m) * a.H + h] : 0.f;
      if (la < kLeastLog) la = kLeastLog;
      const float hi = la * 1.44269502f;  // log2(e) = 1.44269502 + 1.92596303e-8
      x[i] = running({hi, fmaf(la, 1.44269502f, -hi) + la * 1.92596303e-8f}, lane);
      r[i] = ok && a.reset && a.reset[tok + m] != 0;
      be[i] = ok ? a.beta[(tok + m) * a.H + h] : 0.f;
      if (fabsf(be[i]) < kTinyBeta) be[i] = copysignf(kTinyBeta, be[i]);
    }
    x[1] = shfl(x[0], 31) + x[1];
    const Wide end = shfl(x[1], 31);
    const uint32_t b0 = __ballot_sync(kFull, r[0]), b1 = __ballot_sync(kFull, r[1]);
    const uint32_t upto = 0xffffffffu >> (31 - lane);
    const int seg[2] = {__popc(b0 & upto), __popc(b0) + __popc(b1 & upto)}, last = __popc(b0) + __popc(b1);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int m = lane + 32 * i;
      const Wide rest = end - x[i];
      const float v[6] = {seg[i] == 0 ? umma::ex2_approx(x[i].hi) : 0.f, seg[i] == last ? umma::ex2_approx(rest.hi) : 0.f,
                          be[i], x[i].hi, x[i].lo, __int_as_float(seg[i])};
#pragma unroll
      for (int e = 0; e < 6; ++e) {
        sc[e * kC + m] = v[e];
        out[e * kC + m] = v[e];
      }
    }
  }
  cp_async_wait<0>();
  __syncthreads();
  if (a.by_qk == 16) {
    uint32_t limit = kWaitLimit;
    wait_copies(bar, 0, limit, a);
    if (live < kC) {
      clear_rows<panels, kPrepThreads>(sK, live, tid);
      clear_rows<panels, kPrepThreads>(sQ, live, tid);
      __syncthreads();
    }
  }

  // K K^T and Q K^T, a warp 16 rows, up to its diagonal block
  float G[8][4], P[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) G[i][e] = P[i][e] = 0.f;
  const uint32_t uK = smem_u32(sK), uQ = smem_u32(sQ);
#pragma unroll
  for (int ks = 0; ks < NK; ++ks) {
    uint32_t ak[4], aq[4];
    a_rows(uK, 16 * w, 16 * ks, lane, ak);
    a_rows(uQ, 16 * w, 16 * ks, lane, aq);
#pragma unroll
    for (int np = 0; np < 4; ++np) {
      if (np > w) continue;
      uint32_t r[4];
      b_rows(uK, 16 * np, 16 * ks, lane, r);
      fma16816(G[2 * np], ak, r[0], r[1]);
      fma16816(G[2 * np + 1], ak, r[2], r[3]);
      fma16816(P[2 * np], aq, r[0], r[1]);
      fma16816(P[2 * np + 1], aq, r[2], r[3]);
    }
  }
  const float *be = sc + 2 * kC, *lh = sc + 3 * kC, *ll = sc + 4 * kC, *sg = sc + 5 * kC;
  __syncthreads();  // the tiles have been read
#pragma unroll
  for (int nt = 0; nt < 8; ++nt) {
    if (nt > 2 * w + 1) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = 16 * w + g + 8 * (e >> 1), j = 8 * nt + 2 * t + (e & 1);
      const bool on = j <= i && __float_as_int(sg[i]) == __float_as_int(sg[j]);
      const float d = on ? umma::ex2_approx((lh[i] - lh[j]) + (ll[i] - ll[j])) : 0.f;
      sL[i * kLd + j] = on && j < i ? d * G[nt][e] * be[j] : 0.f;
      sX[i * kLd + j] = on ? d * P[nt][e] : 0.f;
    }
  }
  __syncthreads();
  write_tiles(sX, a.m3 + u * (3 * kTri), tid);
  __syncthreads();
  invert(sL, sX, zt, tid);
  write_tiles(sX, a.t3 + u * (3 * kTri), tid);
}

// ---------------------------------------------------------------------------
// The chains.  A CTA has W tiles of 16 value columns of one head, each with two
// warps: the first does what the next chunk waits for (Z, E and the state's
// update), the second everything else (copies of the next chunk's tiles, y,
// the products with dy, what is kept for later).  A tile's state lives in shared memory as its three
// bf16 parts, which are all 24 bits of it, in the order of the A fragments that every
// product with it takes; so the loops over the key channels need not be unrolled over
// registers and stay small enough for the instruction caches.
// ---------------------------------------------------------------------------
template <int NK, int PM, int W>  // PM: parts of M
struct Chain {
  static constexpr int P = NK / 4;  // panels of K and Q
  static constexpr int K = 0, Q = K + P * kPanel, V = Q + P * kPanel, T = V + kPanel, M = T + 3 * kTri, sc = M + PM * kTri,
                       stage = (sc + 3 * kC * 4 + 1023) / 1024 * 1024;
  static constexpr int state = 2 * stage, tokens = state + W * NK * 3 * 512, bars = tokens + W * 8 * 512, size = bars + 16;
};

// A chunk's tiles into a stage; cols: the value columns' tensor.  What tensor and
// bulk copies bring is asked for by one lane of a warp of its own or, where a CTA
// has four tiles and no room for another warp's registers, by one lane of each of
// the second warps (a request holds its warp for a hundred cycles and more).
template <int W>
constexpr int kAskers = W < 4 ? 1 : 4;

template <int NK, int PM, int W>
__device__ __forceinline__ void request_stage(unsigned char *st, uint64_t *bar, const Gdn &a, const Maps &maps, int64_t u,
                                              int64_t tok, int h, int col0, int by_cols, const CUtensorMap *cols_map, int who) {
  using L = Chain<NK, PM, W>;
  constexpr bool all = kAskers<W> == 1;
  const uint32_t mb = smem_u32(bar);
  const int hk = h / (a.H / a.Hk), token = static_cast<int>(tok);
  const bool qk = a.by_qk == 16, cols = by_cols == 16;
  const uint32_t part[4] = {qk ? L::P * kPanel : 0u, qk ? L::P * kPanel : 0u, 3 * kTri + (cols ? kPanel : 0u),
                            PM * kTri + 3 * kC * 4u};
  umma::mbar_expect_tx(mb, all ? part[0] + part[1] + part[2] + part[3] : part[who]);
  if ((all || who == 0) && qk)
#pragma unroll
    for (int p = 0; p < L::P; ++p) tensor_panel(smem_u32(st + L::K) + p * kPanel, &maps.k, 64 * p, hk, token, mb);
  if ((all || who == 1) && qk)
#pragma unroll
    for (int p = 0; p < L::P; ++p) tensor_panel(smem_u32(st + L::Q) + p * kPanel, &maps.q, 64 * p, hk, token, mb);
  if (all || who == 2) {
    umma::bulk_g2s(smem_u32(st + L::T), a.t3 + u * (3 * kTri), 3 * kTri, mb);
    if (cols) tensor_panel(smem_u32(st + L::V), cols_map, col0 & ~63, h, token, mb);
  }
  if (all || who == 3) {
    umma::bulk_g2s(smem_u32(st + L::M), a.m3 + u * (3 * kTri), PM * kTri, mb);
    umma::bulk_g2s(smem_u32(st + L::sc), a.scal + u * kScal, 3 * kC * 4, mb);
  }
}
// ... and the rest, by the second warps
template <int NK, int PM, int W>
__device__ __forceinline__ void copy_stage(unsigned char *st, const Gdn &a, int64_t tok, int h, int col0, int live,
                                           const uint16_t *cols, int64_t ld_cols, int by_cols, int tid) {
  using L = Chain<NK, PM, W>;
  constexpr int threads = 32 * W;
  const int hk = h / (a.H / a.Hk), from = col0 & ~63;  // whole panels of value columns
  if (a.by_qk != 16) {
    load_tile<L::P, threads>(st + L::K, a.k + tok * a.ld_k + hk * a.dk, a.ld_k, live, a.dk, a.by_qk, tid);
    load_tile<L::P, threads>(st + L::Q, a.q + tok * a.ld_q + hk * a.dk, a.ld_q, live, a.dk, a.by_qk, tid);
  }
  if (by_cols != 16)
    load_tile<1, threads>(st + L::V, cols + tok * ld_cols + h * a.dv + from, ld_cols, live, min(64, a.dv - from), by_cols, tid);
  cp_async_commit();
}

// the rows behind a chunk's last token, which tensor copies fill with whatever follows it
template <int NK, int PM, int W>
__device__ __forceinline__ void clear_stage(unsigned char *st, const Gdn &a, int live, int by_cols, int tid) {
  using L = Chain<NK, PM, W>;
  if (a.by_qk == 16) {
    clear_rows<L::P, 32 * W>(st + L::K, live, tid);
    clear_rows<L::P, 32 * W>(st + L::Q, live, tid);
  }
  if (by_cols == 16) clear_rows<1, 32 * W>(st + L::V, live, tid);
  umma::fence_async_smem();
}

// S^T of 16 columns and 8 NT rows of a [dk][dv] matrix as an accumulator, and back
template <int NT>
__device__ __forceinline__ void read_state(const float *m, int row, int dk, int dv, int col, int lane, float (&S)[NT][4]) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = row + 8 * nt + 2 * t + (e & 1), c = col + g + 8 * (e >> 1);
      S[nt][e] = m && r < dk && c < dv ? m[static_cast<int64_t>(r) * dv + c] : 0.f;
    }
}
template <int NT>
__device__ __forceinline__ void write_state(float *m, int row, int dk, int dv, int col, int lane, const float (&S)[NT][4]) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = row + 8 * nt + 2 * t + (e & 1), c = col + g + 8 * (e >> 1);
      if (r < dk && c < dv) m[static_cast<int64_t>(r) * dv + c] = S[nt][e];
    }
}
// accumulators in a row, 16 bytes a lane
template <int N>
__device__ __forceinline__ void put(float4 *m, int lane, const float (&x)[N][4]) {
#pragma unroll
  for (int i = 0; i < N; ++i) m[i * 32 + lane] = make_float4(x[i][0], x[i][1], x[i][2], x[i][3]);
}
template <int N>
__device__ __forceinline__ void get(const float4 *m, int lane, float (&x)[N][4]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float4 v = m[i * 32 + lane];
    x[i][0] = v.x, x[i][1] = v.y, x[i][2] = v.z, x[i][3] = v.w;
  }
}
template <int N>
__device__ __forceinline__ void clear(float (&x)[N][4]) {
#pragma unroll
  for (int i = 0; i < N; ++i) x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0.f;
}
// the parts of a k-step's A fragments of a state, and the state that they are
__device__ __forceinline__ void put_parts(uint4 *m, int lane, const float (&c0)[4], const float (&c1)[4]) {
  uint32_t s[3][4];
  a_split<3>(c0, c1, s);
#pragma unroll
  for (int p = 0; p < 3; ++p) m[p * 32 + lane] = make_uint4(s[p][0], s[p][1], s[p][2], s[p][3]);
}
__device__ __forceinline__ void get_parts(const uint4 *m, int lane, uint32_t (&s)[3][4]) {
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    const uint4 v = m[p * 32 + lane];
    s[p][0] = v.x, s[p][1] = v.y, s[p][2] = v.z, s[p][3] = v.w;
  }
}
__device__ __forceinline__ void join(const uint32_t (&s)[3][4], float (&c0)[4], float (&c1)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float(&c)[4] = i < 2 ? c0 : c1;
    c[2 * (i & 1)] = low2(s[0][i]) + (low2(s[1][i]) + low2(s[2][i]));
    c[2 * (i & 1) + 1] = high2(s[0][i]) + (high2(s[1][i]) + high2(s[2][i]));
  }
}
// x[nt][.] *= f[token]: a token-wise factor on an accumulator whose columns are tokens
template <int N>
__device__ __forceinline__ void scale_tokens(float (&x)[N][4], const float *f, int t) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float2 v = *reinterpret_cast<const float2 *>(f + 8 * i + 2 * t);
    x[i][0] *= v.x, x[i][1] *= v.y, x[i][2] *= v.x, x[i][3] *= v.y;
  }
}

// d (the leading parts' product) and l (the others') += A B for n-tiles 2 np and
// 2 np + 1, over the parts whose numbers sum up to less than max(PA, PB): what
// the others hold is below the last bit kept.  The tensor cores cut sums off
// where an addition would round; kept apart, the many small products do so
// at their own size.
template <int PA, int PB, int N>
__device__ __forceinline__ void products(float (&d)[N][4], float (&l)[N][4], int np, const uint32_t (&a)[PA][4],
                                         const uint32_t (&b)[PB][4]) {
  constexpr int most = PA > PB ? PA : PB;
#pragma unroll
  for (int i = 0; i < PA; ++i)
#pragma unroll
    for (int j = 0; j < PB; ++j)
      if (i + j < most) {
        float(&to)[N][4] = i + j == 0 ? d : l;
        fma16816(to[2 * np], a[i], b[j][0], b[j][1]);
        fma16816(to[2 * np + 1], a[i], b[j][2], b[j][3]);
      }
}
template <int N>
__device__ __forceinline__ void add(float (&d)[N][4], const float (&l)[N][4]) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) d[i][e] += l[i][e];
}

// the three parts of an accumulator over 64 tokens, as A fragments of its four k-steps
__device__ __forceinline__ void split_tokens(const float (&x)[8][4], uint32_t (&a)[4][3][4]) {
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) a_split<3>(x[2 * ks], x[2 * ks + 1], a[ks]);
}

// acc = A B for n-tiles 4 quad .. 4 quad + 3, B = tile[token][n] exact, over 64
// tokens: the small parts first
__device__ __forceinline__ void quad_product(uint32_t tile, int quad, const uint32_t (&a)[4][3][4], int lane,
                                             float (&acc)[4][4]) {
  uint32_t r[4][2][4];
#pragma unroll
  for (int ks = 0; ks < 4; ++ks)
#pragma unroll
    for (int x = 0; x < 2; ++x) b_cols(tile, 32 * quad + 16 * x, 16 * ks, lane, r[ks][x]);
  clear(acc);
#pragma unroll
  for (int p = 2; p >= 0; --p)
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        fma16816(acc[2 * x], a[ks][p], r[ks][x][0], r[ks][x][1]);
        fma16816(acc[2 * x + 1], a[ks][p], r[ks][x][2], r[ks][x][3]);
      }
}

// state <- factor state + sign acc for n-tiles 4 quad .. 4 quad + 3; x: its new values
__device__ __forceinline__ void update_quad(uint4 *parts, int quad, int lane, float factor, float sign,
                                            const float (&acc)[4][4], float (&x)[4][4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint4 *m = parts + (2 * quad + i) * 96;
    uint32_t s[3][4];
    get_parts(m, lane, s);
    join(s, x[2 * i], x[2 * i + 1]);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[2 * i + j][e] = fmaf(factor, x[2 * i + j][e], sign * acc[2 * i + j][e]);
    put_parts(m, lane, x[2 * i], x[2 * i + 1]);
  }
}

// d = the state's product with tile[token][key channel]
template <int NK>
__device__ __forceinline__ void state_product(const uint4 *parts, uint32_t tile, int lane, float (&d)[8][4]) {
  float l[8][4];
  clear(d);
  clear(l);
#pragma unroll 2
  for (int ks = 0; ks < NK; ++ks) {
    uint32_t s[3][4], r[4][4];
    get_parts(parts + ks * 96, lane, s);
#pragma unroll
    for (int np = 0; np < 4; ++np) b_rows(tile, 16 * np, 16 * ks, lane, r[np]);
#pragma unroll
    for (int p = 0; p < 3; ++p)
#pragma unroll
      for (int np = 0; np < 4; ++np) {
        float(&to)[8][4] = p == 0 ? d : l;
        fma16816(to[2 * np], s[p], r[np][0], r[np][1]);
        fma16816(to[2 * np + 1], s[p], r[np][2], r[np][3]);
      }
  }
  add(d, l);
}

// d = X T^T (BACK: X T), X [16 columns][64 tokens] in three parts, T a triangle in three
template <bool BACK>
__device__ __forceinline__ void triangle_product(const float (&x)[8][4], uint32_t tri, int lane, float (&d)[8][4]) {
  float l[8][4];
  clear(d);
  clear(l);
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) {
    uint32_t a[3][4];
    a_split<3>(x[2 * ks], x[2 * ks + 1], a);
#pragma unroll
    for (int np = BACK ? 0 : ks; np < (BACK ? ks + 1 : 4); ++np) {
      uint32_t r[3][4];
#pragma unroll
      for (int p = 0; p < 3; ++p)
        BACK ? tri_cols(tri + p * kTri, np, ks, lane, r[p]) : tri_rows(tri + p * kTri, np, ks, lane, r[p]);
      products(d, l, np, a, r);
    }
  }
  add(d, l);
}

__device__ __forceinline__ void pair_sync(int id) { asm volatile("bar.sync %0, 64;\n" ::"r"(id + 1) : "memory"); }

// a state's parts from and to a [dk][dv] matrix
template <int NK>
__device__ __forceinline__ void load_state(uint4 *parts, const float *m, int dk, int dv, int col, int lane) {
#pragma unroll 1
  for (int ks = 0; ks < NK; ++ks) {
    float x[2][4];
    read_state<2>(m, 16 * ks, dk, dv, col, lane, x);
    put_parts(parts + ks * 96, lane, x[0], x[1]);
  }
}
template <int NK>
__device__ __forceinline__ void store_state(const uint4 *parts, float *m, int dk, int dv, int col, int lane) {
#pragma unroll 1
  for (int ks = 0; ks < NK; ++ks) {
    uint32_t s[3][4];
    float x[2][4];
    get_parts(parts + ks * 96, lane, s);
    join(s, x[0], x[1]);
    write_state<2>(m, 16 * ks, dk, dv, col, lane, x);
  }
}

template <int NK, int W>
__global__ void __launch_bounds__(W < 4 ? 64 * W + 32 : 64 * W, 1) gdn_chain(const Gdn a, const __grid_constant__ Maps maps) {
  using L = Chain<NK, 2, W>;
  constexpr int NT = 2 * NK;
  extern __shared__ __align__(1024) unsigned char sm[];
  const int tid = threadIdx.x, w = (tid >> 5) % W, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int role = tid / (32 * W);
  const int tiles = (a.dv + 15) >> 4, groups = (tiles + W - 1) / W;
  const int64_t bh = blockIdx.x / groups;
  const int col0 = static_cast<int>(blockIdx.x - bh * groups) * (16 * W), col = col0 + 16 * w;
  const int b = static_cast<int>(bh / a.H), h = static_cast<int>(bh % a.H);
  const int len = length_of(a, b), n = (len + kC - 1) / kC;
  const int64_t tok = static_cast<int64_t>(b) * a.T;
  const bool mine = col < a.dv;  // else the warps only help with the copies
  uint4 *hS = reinterpret_cast<uint4 *>(sm + L::state) + w * NK * 96;
  float4 *hE = reinterpret_cast<float4 *>(sm + L::tokens) + w * 8 * 32;
  const int vp = ((col0 & 63) >> 3) + 2 * w;  // the warp's pieces of the value columns' panel
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::bars);
  if (tid == 0) {
    umma::mbar_init(smem_u32(bars), kAskers<W>);
    umma::mbar_init(smem_u32(bars + 1), kAskers<W>);
    umma::fence_mbar_init();
  }
  __syncthreads();
  uint32_t limit = kWaitLimit;

  if (role == 0) {
    if (a.err && a.lens && a.lens[b] != len && tid == 0) atomicOr(a.err, SDM_DEVERR_INDEX_RANGE);
    float S[NT][4];  // the state itself beside its parts
    read_state<NT>(a.state_in ? a.state_in + bh * a.dk * a.dv : nullptr, 0, a.dk, a.dv, col, lane, S);
#pragma unroll
    for (int ks = 0; ks < NK; ++ks) put_parts(hS + ks * 96, lane, S[2 * ks], S[2 * ks + 1]);
    for (int c = 0; c < n; ++c) {
      __syncthreads();
      wait_copies(bars + (c & 1), (c >> 1) & 1, limit, a);
      if (len - c * kC < kC) __syncthreads();  // the second warps clear rows
      if (!mine) continue;
      unsigned char *st = sm + (c & 1) * L::stage;
      const uint32_t uK = smem_u32(st + L::K), uV = smem_u32(st + L::V);
      const float *gam = reinterpret_cast<const float *>(st + L::sc), *tail = gam + kC, *beta = tail + kC;
      float Z[8][4], E[8][4];
      state_product<NK>(hS, uK, lane, Z);
      // Z^T = V^T - gam S^T K^T
#pragma unroll
      for (int np = 0; np < 4; ++np) {
        uint32_t v[4];
        // tile[token][column]: rows of V^T are its columns
        ldsm4_t(uV + piece(16 * np + (((lane >> 4) & 1) << 3) + (lane & 7), vp + ((lane >> 3) & 1)), v);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int nt = 2 * np + x;
          const float2 gm = *reinterpret_cast<const float2 *>(gam + 8 * nt + 2 * t);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t vv = v[2 * x + (e >> 1)];
            Z[nt][e] = fmaf(e & 1 ? -gm.y : -gm.x, Z[nt][e], e & 1 ? high2(vv) : low2(vv));
          }
        }
      }
      triangle_product<false>(Z, smem_u32(st + L::T), lane, E);
      put(hE, lane, E);
      pair_sync(w);  // E is there, S has been read
      // S^T = gam_C S^T + (tail U)^T K
      scale_tokens(E, beta, t);
      scale_tokens(E, tail, t);
      uint32_t ut[4][3][4];
      split_tokens(E, ut);
      const float end = gam[kC - 1];
#pragma unroll
      for (int q = 0; q < NK / 2; ++q) {
        float acc[4][4];
        quad_product(uK, q, ut, lane, acc);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) S[4 * q + i][e] = fmaf(end, S[4 * q + i][e], acc[i][e]);
#pragma unroll
        for (int i = 0; i < 2; ++i) put_parts(hS + (2 * q + i) * 96, lane, S[4 * q + 2 * i], S[4 * q + 2 * i + 1]);
      }
    }
    if (mine) write_state<NT>(a.state_out + bh * a.dk * a.dv, 0, a.dk, a.dv, col, lane, S);
    return;
  }

  const int ltid = tid - 32 * W;
  const auto request = [&](int c) {
    if (lane == 0)
      request_stage<NK, 2, W>(sm + (c & 1) * L::stage, bars + (c & 1), a, maps, bh * a.n + c, tok + c * kC, h, col0, a.by_v,
                              &maps.v, w);
    __syncwarp();
  };
  if (role == 2) {
    for (int c = 0; c <= n; ++c) {
      if (c > 0) __syncthreads();
      if (c < n) request(c);
      if (c > 0 && len - (c - 1) * kC < kC) __syncthreads();
    }
    return;
  }

  const auto copy = [&](int c) {
    copy_stage<NK, 2, W>(sm + (c & 1) * L::stage, a, tok + c * kC, h, col0, min(len - c * kC, kC), a.v, a.ld_v, a.by_v, ltid);
  };
  if (n > 0) {
    if (kAskers<W> > 1) request(0);
    copy(0);
  }
  for (int c = 0; c < n; ++c) {
    const int64_t u = bh * a.n + c;
    unsigned char *st = sm + (c & 1) * L::stage;
    cp_async_wait<0>();
    __syncthreads();
    if (c + 1 < n) {
      if (kAskers<W> > 1) request(c + 1);
      copy(c + 1);
    }
    wait_copies(bars + (c & 1), (c >> 1) & 1, limit, a);
    if (len - c * kC < kC) {
      clear_stage<NK, 2, W>(st, a, len - c * kC, a.by_v, ltid);
      __syncthreads();
    }
    if (!mine) continue;
    const uint32_t uQ = smem_u32(st + L::Q), uM = smem_u32(st + L::M);
    const float *gam = reinterpret_cast<const float *>(st + L::sc), *beta = gam + 2 * kC;
    float Y[8][4], E[8][4];
    clear(Y);
    {  // Y^T = gam S^T Q^T; S is kept
      float4 *kept = reinterpret_cast<float4 *>(a.s) + (u * tiles + (col >> 4)) * (NT * 32);
#pragma unroll 2
      for (int ks = 0; ks < NK; ++ks) {
        uint32_t s[3][4], r[4][4];
        float x[2][4];
        get_parts(hS + ks * 96, lane, s);
#pragma unroll
        for (int np = 0; np < 4; ++np) b_rows(uQ, 16 * np, 16 * ks, lane, r[np]);
        join(s, x[0], x[1]);
        put(kept + 64 * ks, lane, x);
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int np = 0; np < 4; ++np) {
            fma16816(Y[2 * np], s[p], r[np][0], r[np][1]);
            fma16816(Y[2 * np + 1], s[p], r[np][2], r[np][3]);
          }
      }
      scale_tokens(Y, gam, t);
    }
    pair_sync(w);
    get(hE, lane, E);
    put(reinterpret_cast<float4 *>(a.e) + (u * tiles + (col >> 4)) * 256, lane, E);
    scale_tokens(E, beta, t);
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {  // += U^T M^T
      uint32_t us[2][4];
      a_split<2>(E[2 * ks], E[2 * ks + 1], us);
#pragma unroll
      for (int np = ks; np < 4; ++np) {
        uint32_t r[2][4];
#pragma unroll
        for (int p = 0; p < 2; ++p) tri_rows(uM + p * kTri, np, ks, lane, r[p]);
        products(Y, Y, np, us, r);
      }
    }
    // y, rounded once: pairs of tokens turned into pairs of columns
    uint16_t *yc = a.y + (tok * a.H + h) * a.dv + col + 2 * t;
    const int left = a.dv - col - 2 * t;
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
      const int i = c * kC + 8 * nt + g;
      uint16_t *row = yc + i * (static_cast<int64_t>(a.H) * a.dv);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint32_t v = transpose8(pack2(Y[nt][2 * x], Y[nt][2 * x + 1]));
        if (i >= len) continue;
        if (a.pair_y) {
          if (8 * x < left) *reinterpret_cast<uint32_t *>(row + 8 * x) = v;
        } else {
          if (8 * x < left) row[8 * x] = static_cast<uint16_t>(v);
          if (8 * x + 1 < left) row[8 * x + 1] = static_cast<uint16_t>(v >> 16);
        }
      }
    }
  }
}

template <int NK, int W>
__global__ void __launch_bounds__(W < 4 ? 64 * W + 32 : 64 * W, 1) gdn_chain_back(const Gdn a, const __grid_constant__ Maps maps) {
  using L = Chain<NK, 3, W>;
  constexpr int NT = 2 * NK;
  extern __shared__ __align__(1024) unsigned char sm[];
  const int tid = threadIdx.x, w = (tid >> 5) % W, lane = tid & 31, t = lane & 3;
  const int role = tid / (32 * W);
  const int tiles = (a.dv + 15) >> 4, groups = (tiles + W - 1) / W;
  const int64_t bh = blockIdx.x / groups;
  const int col0 = static_cast<int>(blockIdx.x - bh * groups) * (16 * W), col = col0 + 16 * w;
  const int b = static_cast<int>(bh / a.H), h = static_cast<int>(bh % a.H);
  const int len = length_of(a, b), n = (len + kC - 1) / kC;
  const int64_t tok = static_cast<int64_t>(b) * a.T, ld_y = static_cast<int64_t>(a.H) * a.dv;
  const bool mine = col < a.dv;
  uint4 *hG = reinterpret_cast<uint4 *>(sm + L::state) + w * NK * 96;
  float4 *hZ = reinterpret_cast<float4 *>(sm + L::tokens) + w * 8 * 32;  // dY^T M, then dZ^T
  const int vc = (col0 & 63) + 16 * w;  // the warp's columns in the value columns' panel
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::bars);
  if (tid == 0) {
    umma::mbar_init(smem_u32(bars), kAskers<W>);
    umma::mbar_init(smem_u32(bars + 1), kAskers<W>);
    umma::fence_mbar_init();
  }
  __syncthreads();
  uint32_t limit = kWaitLimit;

  if (role == 0) {
    if (a.err && a.lens && a.lens[b] != len && tid == 0) atomicOr(a.err, SDM_DEVERR_INDEX_RANGE);
    load_state<NK>(hG, a.state_in ? a.state_in + bh * a.dk * a.dv : nullptr, a.dk, a.dv, col, lane);
    float4 *kept = reinterpret_cast<float4 *>(a.g) + (bh * (a.n + 1) * tiles + (col >> 4)) * (NT * 32);
    const int64_t step = static_cast<int64_t>(tiles) * (NT * 32);
    if (mine)
#pragma unroll 1
      for (int ks = 0; ks < NK; ++ks) {
        uint32_t s[3][4];
        float x[2][4];
        get_parts(hG + ks * 96, lane, s);
        join(s, x[0], x[1]);
        put(kept + n * step + ks * 64, lane, x);
      }
    for (int c = n - 1; c >= 0; --c) {
      const int it = n - 1 - c;
      __syncthreads();
      wait_copies(bars + (it & 1), (it >> 1) & 1, limit, a);
      if (len - c * kC < kC) __syncthreads();  // the second warps clear rows
      if (!mine) continue;
      unsigned char *st = sm + (it & 1) * L::stage;
      const uint32_t uK = smem_u32(st + L::K);
      const float *gam = reinterpret_cast<const float *>(st + L::sc), *tail = gam + kC, *beta = tail + kC;
      // dU^T = tail G^T K^T + dY^T M
      float U[8][4], Z[8][4];
      state_product<NK>(hG, uK, lane, U);
      scale_tokens(U, tail, t);
      pair_sync(w);  // dY^T M is there, G has been read
      get(hZ, lane, Z);
      add(U, Z);
      scale_tokens(U, beta, t);
      triangle_product<true>(U, smem_u32(st + L::T), lane, Z);  // dZ^T
      put(hZ, lane, Z);
      // G^T = gam_C G^T + (gam dY)^T Q, by the second warp, - (gam dZ)^T K
      scale_tokens(Z, gam, t);
      uint32_t zt[4][3][4];
      split_tokens(Z, zt);
      pair_sync(w);
      float4 *to = kept + c * step;
#pragma unroll 2
      for (int q = 0; q < NK / 2; ++q) {
        float acc[4][4], x[4][4];
        quad_product(uK, q, zt, lane, acc);
        update_quad(hG, q, lane, 1.f, -1.f, acc, x);
        put(to + q * 128, lane, x);
      }
    }
    if (mine) store_state<NK>(hG, a.state_out + bh * a.dk * a.dv, a.dk, a.dv, col, lane);
    return;
  }

  const int ltid = tid - 32 * W;
  const auto request = [&](int c) {
    const int s = (n - 1 - c) & 1;
    if (lane == 0)
      request_stage<NK, 3, W>(sm + s * L::stage, bars + s, a, maps, bh * a.n + c, tok + c * kC, h, col0, a.by_dy, &maps.dy, w);
    __syncwarp();
  };
  if (role == 2) {
    for (int it = 0; it <= n; ++it) {
      const int c = n - 1 - it;
      if (it > 0) __syncthreads();
      if (it < n) request(c);
      if (it > 0 && len - (c + 1) * kC < kC) __syncthreads();
    }
    return;
  }

  const auto copy = [&](int c) {
    copy_stage<NK, 3, W>(sm + ((n - 1 - c) & 1) * L::stage, a, tok + c * kC, h, col0, min(len - c * kC, kC), a.dy, ld_y,
                         a.by_dy, ltid);
  };
  if (n > 0) {
    if (kAskers<W> > 1) request(n - 1);
    copy(n - 1);
  }
  for (int c = n - 1; c >= 0; --c) {
    const int it = n - 1 - c;
    const int64_t u = bh * a.n + c;
    unsigned char *st = sm + (it & 1) * L::stage;
    cp_async_wait<0>();
    __syncthreads();
    if (c > 0) {
      if (kAskers<W> > 1) request(c - 1);
      copy(c - 1);
    }
    wait_copies(bars + (it & 1), (it >> 1) & 1, limit, a);
    if (len - c * kC < kC) {
      clear_stage<NK, 3, W>(st, a, len - c * kC, a.by_dy, ltid);
      __syncthreads();
    }
    if (!mine) continue;
    const uint32_t uQ = smem_u32(st + L::Q), uM = smem_u32(st + L::M), uY = smem_u32(st + L::V);
    const float *gam = reinterpret_cast<const float *>(st + L::sc);
    uint32_t y[4][1][4];
    {
      float R[8][4], l[8][4];
      clear(R);
      clear(l);
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        a_cols(uY, vc, 16 * ks, lane, y[ks][0]);
#pragma unroll
        for (int np = 0; np <= ks; ++np) {
          uint32_t r[3][4];
#pragma unroll
          for (int p = 0; p < 3; ++p) tri_cols(uM + p * kTri, np, ks, lane, r[p]);
          products(R, l, np, y[ks], r);
        }
      }
      add(R, l);
      put(hZ, lane, R);
    }
    uint32_t d3[4][3][4];
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      float d[2][4];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float2 gm = *reinterpret_cast<const float2 *>(gam + 8 * (2 * ks + x) + 2 * t);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t v = y[ks][0][2 * x + (e >> 1)];
          d[x][e] = e & 1 ? gm.y * high2(v) : gm.x * low2(v);
        }
      }
      a_split<3>(d[0], d[1], d3[ks]);
    }
    pair_sync(w);
    const float end = gam[kC - 1];
#pragma unroll 2
    for (int q = 0; q < NK / 2; ++q) {
      float acc[4][4], x[4][4];
      quad_product(uQ, q, d3, lane, acc);
      update_quad(hG, q, lane, end, 1.f, acc, x);
    }
    pair_sync(w);
    float Z[8][4];
    get(hZ, lane, Z);
    put(reinterpret_cast<float4 *>(a.dz) + (u * tiles + (col >> 4)) * 256, lane, Z);
  }
}

// ---------------------------------------------------------------------------
// gdn_grad: the gradients of one chunk of one head.  A warp has an eighth of
// the key channels for 32 tokens, so each element of the two states is needed by
// two warps only: straight from memory, where the chains left it in fragment
// order, split into bf16 parts and turned (8 x 8 at a time) into the B
// fragments of the sums over value columns.  U and dZ are shared: split once, into A fragments
// in shared memory (an A fragment of U holds the B fragments of U^T).
// Value columns come 128 at a time.
// ---------------------------------------------------------------------------
constexpr int kGradThreads = 512;

constexpr int kRing = 3;  // tiles of the states on their way

template <int NK>
struct Grad {
  static constexpr int P = NK / 4;
  static constexpr int K = 0, Q = K + P * kPanel, Y = Q + P * kPanel, V = Y + 2 * kTile, U = V + 2 * kTile,
                       Z = U + 8 * 3 * 4 * 512, ring = Z + 8 * 2 * 4 * 512, part = 2 * NK * 512 /* one state's tile */,
                       sc = ring + kRing * 3 * part, bars = sc + (kScal + 8 * 3 * kC + 8) * 4,
                       size = bars + (2 * kRing + 1) * 8;
  static constexpr int X = U, N = X + 3 * kTile;  // once the value columns are done: X in three parts, N + N^T in two
};

// lanes 4 x + t hold v[16]; the sums over x, two of them a lane (bits 3..1 of the value are the lane's bits 4..2)
__device__ __forceinline__ void sum_rows(float (&v)[16], int lane) {
#pragma unroll
  for (int o = 16; o >= 4; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < o / 2; ++i) {
      const float send = up ? v[i] : v[i + o / 2], keep = up ? v[i + o / 2] : v[i];
      v[i] = keep + __shfl_xor_sync(kFull, send, o);
    }
  }
}

template <int NK>
__global__ void __launch_bounds__(kGradThreads, 1) gdn_grad(const Gdn a, const __grid_constant__ Maps maps) {
  using L = Grad<NK>;
  constexpr int NT = 2 * NK, NW = NK / 4;  // NW: n-tiles of key channels a warp
  extern __shared__ __align__(1024) unsigned char sm[];
  const int tid = threadIdx.x, w = (tid >> 5) & 7, half = tid >> 8, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int64_t u = blockIdx.x, bh = u / a.n;
  const int c = static_cast<int>(u - bh * a.n), b = static_cast<int>(bh / a.H), h = static_cast<int>(bh % a.H);
  const int live = min(length_of(a, b) - c * kC, kC);
  if (live <= 0) return;
  const int64_t tok = static_cast<int64_t>(b) * a.T + c * kC, ld_y = static_cast<int64_t>(a.H) * a.dv;
  const int hk = h / (a.H / a.Hk), tiles = (a.dv + 15) >> 4;
  float *sc = reinterpret_cast<float *>(sm + L::sc);
  float *gam = sc, *tail = sc + kC, *beta = sc + 2 * kC, *lh = sc + 3 * kC, *ll = sc + 4 * kC, *sg = sc + 5 * kC;
  float *rows = sc + kScal /* [8][2][64]: dZ . E and v . dZ */, *flow = rows + 8 * 2 * kC /* [8][64] */,
        *red = flow + 8 * kC;
  const uint32_t uY = smem_u32(sm + L::Y), uV = smem_u32(sm + L::V);
  uint64_t *full = reinterpret_cast<uint64_t *>(sm + L::bars), *empty = full + kRing, *tile_bar = empty + kRing;
  const unsigned char *gS = reinterpret_cast<const unsigned char *>(a.s) + u * tiles * L::part,
                      *gG = reinterpret_cast<const unsigned char *>(a.g) + (bh * (a.n + 1) + c) * tiles * L::part;
  // one thread: the states' tile kt (S, G at the chunk's start and at its end) into the ring
  const auto load_states = [&](int kt) {
    const uint32_t mb = smem_u32(full + kt % kRing), to = smem_u32(sm + L::ring) + (kt % kRing) * 3 * L::part;
    umma::mbar_expect_tx(mb, 3 * L::part);
    umma::bulk_g2s(to, gS + kt * L::part, L::part, mb);
    umma::bulk_g2s(to + L::part, gG + kt * L::part, L::part, mb);
    umma::bulk_g2s(to + 2 * L::part, gG + (static_cast<int64_t>(tiles) + kt) * L::part, L::part, mb);
  };
  // the value columns' tiles from column c0 on
  const auto load_columns = [&](int c0) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int cx = c0 + 64 * x;
      if (cx >= a.dv) continue;
      if (a.by_dy != 16)
        load_tile<1, kGradThreads>(sm + L::Y + x * kTile, a.dy + tok * ld_y + h * a.dv + cx, ld_y, live, min(64, a.dv - cx),
                                   a.by_dy, tid);
      else if (tid == 0)
        tensor_panel(uY + x * kTile, &maps.dy, cx, h, static_cast<int>(tok), smem_u32(tile_bar));
      if (a.by_v != 16)
        load_tile<1, kGradThreads>(sm + L::V + x * kTile, a.v + tok * a.ld_v + h * a.dv + cx, a.ld_v, live,
                                   min(64, a.dv - cx), a.by_v, tid);
      else if (tid == 0)
        tensor_panel(uV + x * kTile, &maps.v, cx, h, static_cast<int>(tok), smem_u32(tile_bar));
    }
    cp_async_commit();
  };
  const auto column_bytes = [&](int c0) {
    return static_cast<uint32_t>(((a.by_dy == 16) + (a.by_v == 16)) * (c0 + 64 < a.dv ? 2 : 1) * kPanel);
  };
  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      umma::mbar_init(smem_u32(full + i), 1);
      umma::mbar_init(smem_u32(empty + i), kGradThreads / 32);
    }
    umma::mbar_init(smem_u32(tile_bar), 1);
    umma::fence_mbar_init();
    const uint32_t more = kScal * 4 + column_bytes(0);
    if (a.by_qk == 16)
      load_qk<NK>(maps, sm + L::K, sm + L::Q, hk, tok, smem_u32(tile_bar), more);
    else
      umma::mbar_expect_tx(smem_u32(tile_bar), more);
    umma::bulk_g2s(smem_u32(sc), a.scal + u * kScal, kScal * 4, smem_u32(tile_bar));
  }
  if (a.by_qk != 16) {
    load_tile<L::P, kGradThreads>(sm + L::K, a.k + tok * a.ld_k + hk * a.dk, a.ld_k, live, a.dk, a.by_qk, tid);
    load_tile<L::P, kGradThreads>(sm + L::Q, a.q + tok * a.ld_q + hk * a.dk, a.ld_q, live, a.dk, a.by_qk, tid);
  }
  load_columns(0);
  if (tid == 0) {
    for (int kt = 0; kt < min(kRing, tiles); ++kt) load_states(kt);
    // what the chunk that is likely to follow here reads first, on its way into L2
    const int64_t next = u + kSms;
    if (next < static_cast<int64_t>(gridDim.x)) {
      const uint32_t bytes = static_cast<uint32_t>(tiles) * 4096;
      umma::prefetch_l2(a.e + next * tiles * 1024, bytes);
      umma::prefetch_l2(a.dz + next * tiles * 1024, bytes);
      umma::prefetch_l2(a.s + next * tiles * (NT * 128), static_cast<uint32_t>(tiles) * L::part);
    }
  }
  uint32_t limit = kWaitLimit;
  if (w >= tiles) rows[(2 * w + half) * kC + lane] = rows[(2 * w + half) * kC + 32 + lane] = 0.f;
  uint4 *sU = reinterpret_cast<uint4 *>(sm + L::U), *sZ = reinterpret_cast<uint4 *>(sm + L::Z);

  // m-tiles 2 half and 2 half + 1
  float dQ[2][NW][4], dA[2][NW][4], dK[2][NW][4], X[2][4], N[2][4];
#pragma unroll
  for (int m = 0; m < 2; ++m) clear(dQ[m]), clear(dA[m]), clear(dK[m]);
  clear(X);
  clear(N);
  float anchor = 0.f;

  for (int c0 = 0; c0 < a.dv; c0 += 128) {
    const int nt_cols = min(8, tiles - (c0 >> 4));  // tiles of 16 columns in this piece
    // half a tile of E and dZ
    float E[4][4], Z[4][4];
    if (w < nt_cols) {
      const int64_t at = (u * tiles + (c0 >> 4) + w) * 256 + half * 128;
      get(reinterpret_cast<const float4 *>(a.e) + at, lane, E);
      get(reinterpret_cast<const float4 *>(a.dz) + at, lane, Z);
    }
    if (c0) {
      __syncthreads();  // the piece before has been read
      if (tid == 0) umma::mbar_expect_tx(smem_u32(tile_bar), column_bytes(c0));
      load_columns(c0);
    }
    cp_async_wait<0>();
    __syncthreads();
    wait_copies(tile_bar, (c0 >> 7) & 1, limit, a);
    if (live < kC) {
      if (a.by_qk == 16 && c0 == 0) {
        clear_rows<L::P, kGradThreads>(sm + L::K, live, tid);
        clear_rows<L::P, kGradThreads>(sm + L::Q, live, tid);
      }
      for (int x = 0; x < 2; ++x) {
        if (a.by_dy == 16) clear_rows<1, kGradThreads>(sm + L::Y + x * kTile, live, tid);
        if (a.by_v == 16) clear_rows<1, kGradThreads>(sm + L::V + x * kTile, live, tid);
      }
      umma::fence_async_smem();
      __syncthreads();
    }
    if (w < nt_cols) {
      uint16_t *dvp = a.odv + tok * a.ld_dv + h * a.dv + c0 + 16 * w + 2 * t;
      float sum[16];  // [dZ . E, v . dZ][n-tile][token of the pair]
#pragma unroll
      for (int np = 0; np < 2; ++np) {
        uint32_t v[4], pu[3][4], pz[2][4];
        ldsm4_t(uV + (w >> 2) * kTile +
                    piece(32 * half + 16 * np + (((lane >> 4) & 1) << 3) + (lane & 7), 2 * (w & 3) + ((lane >> 3) & 1)),
                v);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int nt = 2 * np + x;
          const float2 be = *reinterpret_cast<const float2 *>(beta + 32 * half + 8 * nt + 2 * t);
          sum[2 * nt] = E[nt][0] * Z[nt][0] + E[nt][2] * Z[nt][2];
          sum[2 * nt + 1] = E[nt][1] * Z[nt][1] + E[nt][3] * Z[nt][3];
          sum[8 + 2 * nt] = low2(v[2 * x]) * Z[nt][0] + low2(v[2 * x + 1]) * Z[nt][2];
          sum[8 + 2 * nt + 1] = high2(v[2 * x]) * Z[nt][1] + high2(v[2 * x + 1]) * Z[nt][3];
#pragma unroll
          for (int e = 0; e < 2; ++e) {  // columns 0..7 and 8..15 of the tile
            uint32_t s3[3], s2[2];
            split<3>(be.x * E[nt][2 * e], be.y * E[nt][2 * e + 1], s3);
            split<2>(Z[nt][2 * e], Z[nt][2 * e + 1], s2);
#pragma unroll
            for (int p = 0; p < 3; ++p) pu[p][x + 2 * e] = transpose8(s3[p]);
#pragma unroll
            for (int p = 0; p < 2; ++p) pz[p][x + 2 * e] = transpose8(s2[p]);
            // dv is dZ rounded once, which is its first part
            const int i = 32 * half + 8 * nt + g, left = a.dv - (c0 + 16 * w + 8 * e + 2 * t);
            if (i < live) {
              uint16_t *o = dvp + i * a.ld_dv + 8 * e;
              const uint32_t z = pz[0][x + 2 * e];
              if (a.pair_y) {
                if (left > 0) *reinterpret_cast<uint32_t *>(o) = z;
              } else {
                if (left > 0) o[0] = static_cast<uint16_t>(z);
                if (left > 1) o[1] = static_cast<uint16_t>(z >> 16);
              }
            }
          }
        }
#pragma unroll
        for (int p = 0; p < 3; ++p)
          sU[((w * 3 + p) * 4 + 2 * half + np) * 32 + lane] = make_uint4(pu[p][0], pu[p][1], pu[p][2], pu[p][3]);
#pragma unroll
        for (int p = 0; p < 2; ++p)
          sZ[((w * 2 + p) * 4 + 2 * half + np) * 32 + lane] = make_uint4(pz[p][0], pz[p][1], pz[p][2], pz[p][3]);
      }
      sum_rows(sum, lane);
      float *to = rows + (w * 2 + (lane >> 4)) * kC + 32 * half + 8 * (2 * ((lane >> 3) & 1) + ((lane >> 2) & 1)) + 2 * t;
#pragma unroll
      for (int i = 0; i < 2; ++i) to[i] = c0 ? to[i] + sum[i] : sum[i];
    }
    __syncthreads();

#pragma unroll 1
    for (int kt = 0; kt < nt_cols; ++kt) {
      const int at = (c0 >> 4) + kt, slot = at % kRing;
      const uint32_t parity = (at / kRing) & 1;
      if (tid == 0 && at > 0 && at + kRing - 1 < tiles) {  // the slot of the tile before, once everyone has it
        wait_copies(empty + (at - 1) % kRing, ((at - 1) / kRing) & 1, limit, a);
        load_states(at + kRing - 1);
      }
      __syncwarp();
      wait_copies(full + slot, parity, limit, a);
      float4 fs[NW], f0[NW], f1[NW];
      const float4 *from = reinterpret_cast<const float4 *>(sm + L::ring + slot * 3 * L::part) + w * NW * 32 + lane;
#pragma unroll
      for (int x = 0; x < NW; ++x) {
        fs[x] = from[x * 32], f1[x] = from[2 * NT * 32 + x * 32];
        if (half == 0) f0[x] = from[NT * 32 + x * 32];
      }
      __syncwarp();
      if (lane == 0) umma::mbar_arrive(smem_u32(empty + slot));
      uint32_t bs[NW][3][2], bg[NW][2][2];
#pragma unroll
      for (int x = 0; x < NW; ++x) {
        if (half == 0) anchor += (fs[x].x * f0[x].x + fs[x].y * f0[x].y) + (fs[x].z * f0[x].z + fs[x].w * f0[x].w);
        uint32_t p0[3], p1[3], q0[2], q1[2];
        split<3>(fs[x].x, fs[x].y, p0);
        split<3>(fs[x].z, fs[x].w, p1);
        split<2>(f1[x].x, f1[x].y, q0);
        split<2>(f1[x].z, f1[x].w, q1);
#pragma unroll
        for (int p = 0; p < 3; ++p) bs[x][p][0] = transpose8(p0[p]), bs[x][p][1] = transpose8(p1[p]);
#pragma unroll
        for (int p = 0; p < 2; ++p) bg[x][p][0] = transpose8(q0[p]), bg[x][p][1] = transpose8(q1[p]);
      }
      uint32_t bu[3][2];
#pragma unroll
      for (int p = 0; p < 3; ++p) {
        const uint4 v = sU[((kt * 3 + p) * 4 + (w >> 1)) * 32 + lane];
        bu[p][0] = w & 1 ? v.y : v.x;
        bu[p][1] = w & 1 ? v.w : v.z;
      }
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const int mt = 2 * half + m;
        uint32_t y[4], uu[2][4], z[2][4];
        a_rows(uY + (kt >> 2) * kTile, 16 * mt, 16 * (kt & 3), lane, y);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const uint4 vu = sU[((kt * 3 + p) * 4 + mt) * 32 + lane], vz = sZ[((kt * 2 + p) * 4 + mt) * 32 + lane];
          uu[p][0] = vu.x, uu[p][1] = vu.y, uu[p][2] = vu.z, uu[p][3] = vu.w;
          z[p][0] = vz.x, z[p][1] = vz.y, z[p][2] = vz.z, z[p][3] = vz.w;
        }
#pragma unroll
        for (int p = 0; p < 3; ++p)
#pragma unroll
          for (int x = 0; x < NW; ++x) {
            fma16816(dQ[m][x], y, bs[x][p][0], bs[x][p][1]);
            // parts 0 0, 0 1 and 1 0
            fma16816(dA[m][x], z[p >> 1], bs[x][p & 1][0], bs[x][p & 1][1]);
            fma16816(dK[m][x], uu[p >> 1], bg[x][p & 1][0], bg[x][p & 1][1]);
          }
        if (mt >= (w >> 1))
#pragma unroll
          for (int p = 0; p < 3; ++p) {
            fma16816(X[m], y, bu[p][0], bu[p][1]);
            fma16816(N[m], z[p >> 1], bu[p & 1][0], bu[p & 1][1]);
          }
      }
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) anchor += __shfl_xor_sync(kFull, anchor, o);
  if (lane == 0 && half == 0) red[w] = anchor;
  __syncthreads();  // U has been read

#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const int mt = 2 * half + m;
#pragma unroll
    for (int x = 0; x < NW; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = 16 * mt + g + 8 * (e >> 1);
        dQ[m][x][e] *= gam[i];
        dK[m][x][e] = tail[i] * dK[m][x][e] - gam[i] * dA[m][x][e];
      }
    if (mt < (w >> 1)) continue;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int i = 16 * mt + g + 8 * r, j = 8 * w + 2 * t;
      float xv[2], nv[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const bool on = j + e <= i && __float_as_int(sg[i]) == __float_as_int(sg[j + e]);
        const float d = on ? umma::ex2_approx((lh[i] - lh[j + e]) + (ll[i] - ll[j + e])) : 0.f;
        xv[e] = on ? d * X[m][2 * r + e] : 0.f;
        nv[e] = on && j + e < i ? -d * N[m][2 * r + e] : 0.f;
      }
      uint32_t sx[3], sn[2];
      split<3>(xv[0], xv[1], sx);
      split<2>(nv[0], nv[1], sn);
      const uint32_t off = piece(i, w) + 4 * t;
#pragma unroll
      for (int p = 0; p < 3; ++p) *reinterpret_cast<uint32_t *>(sm + L::X + p * kTile + off) = sx[p];
#pragma unroll
      for (int p = 0; p < 2; ++p) {  // N below the diagonal, N^T above it
        unsigned char *tile = sm + L::N + p * kTile;
        const uint16_t lo = static_cast<uint16_t>(sn[p]), hi = static_cast<uint16_t>(sn[p] >> 16);
        if (j <= i) {
          *reinterpret_cast<uint16_t *>(tile + off) = lo;
          *reinterpret_cast<uint16_t *>(tile + piece(j, i >> 3) + 2 * (i & 7)) = lo;
        }
        if (j + 1 <= i) {
          *reinterpret_cast<uint16_t *>(tile + off + 2) = hi;
          *reinterpret_cast<uint16_t *>(tile + piece(j + 1, i >> 3) + 2 * (i & 7)) = hi;
        }
      }
    }
  }
  __syncthreads();
  const uint32_t uK = smem_u32(sm + L::K), uQ = smem_u32(sm + L::Q), uX = smem_u32(sm + L::X), uN = smem_u32(sm + L::N);
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) {
    uint32_t bk[4], bq[4];  // of 16 key channels: this warp's, or with another's beside them
    constexpr int share = 2 / NW;
    b_cols(uK, 16 * (w / share), 16 * ks, lane, bk);
    b_cols(uQ, 16 * (w / share), 16 * ks, lane, bq);
    if (NW == 1 && (w & 1)) bk[0] = bk[2], bk[1] = bk[3], bq[0] = bq[2], bq[1] = bq[3];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const int mt = 2 * half + m;
      uint32_t f[4];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        a_rows(uN + p * kTile, 16 * mt, 16 * ks, lane, f);
#pragma unroll
        for (int x = 0; x < NW; ++x) fma16816(dK[m][x], f, bk[2 * x], bk[2 * x + 1]);
      }
      if (ks <= mt)
#pragma unroll
        for (int p = 0; p < 3; ++p) {
          a_rows(uX + p * kTile, 16 * mt, 16 * ks, lane, f);
#pragma unroll
          for (int x = 0; x < NW; ++x) fma16816(dQ[m][x], f, bk[2 * x], bk[2 * x + 1]);
        }
      if (ks >= mt)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          a_cols(uX + p * kTile, 16 * mt, 16 * ks, lane, f);
#pragma unroll
          for (int x = 0; x < NW; ++x) fma16816(dK[m][x], f, bq[2 * x], bq[2 * x + 1]);
        }
    }
  }
  // q . dq
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int i = 32 * half + 16 * m + g + 8 * r;
      float qd = 0.f;
#pragma unroll
      for (int x = 0; x < NW; ++x) {
        const uint32_t v = *reinterpret_cast<const uint32_t *>(sm + L::Q + piece(i, w * NW + x) + 4 * t);
        qd += low2(v) * dQ[m][x][2 * r] + high2(v) * dQ[m][x][2 * r + 1];
      }
      qd += __shfl_xor_sync(kFull, qd, 1);
      qd += __shfl_xor_sync(kFull, qd, 2);
      if (t == 0) flow[w * kC + i] = qd;
    }
  __syncthreads();
  if (tid < 32) {  // the decays' gradient: sums before each token
    float x[2], before[2], ez[2];
    int seg[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int m = lane + 32 * i;
      float f = 0.f;
      ez[i] = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        f += flow[e * kC + m] - rows[(2 * e + 1) * kC + m];
        ez[i] += rows[2 * e * kC + m];
      }
      before[i] = x[i] = f;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float y = __shfl_up_sync(kFull, x[i], o);
        if (lane >= o) x[i] += y;
      }
      seg[i] = __float_as_int(sg[m]);
    }
    x[1] += __shfl_sync(kFull, x[0], 31);
    const uint32_t s0 = __ballot_sync(kFull, lane == 0 || seg[0] != __float_as_int(sg[max(lane - 1, 0)]));
    const uint32_t s1 = __ballot_sync(kFull, seg[1] != __float_as_int(sg[lane + 31]));
    before[0] = x[0] - before[0];  // sum over s < t
    before[1] = x[1] - before[1];
    const uint32_t upto = 0xffffffffu >> (31 - lane);
    const float start = ((red[0] + red[1]) + (red[2] + red[3])) + ((red[4] + red[5]) + (red[6] + red[7]));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int m = lane + 32 * i;
      // the first token of this one's document
      const int first = i == 0 ? 31 - __clz(s0 & upto) : (s1 & upto) ? 63 - __clz(s1 & upto) : 31 - __clz(s0);
      const float p0 = __shfl_sync(kFull, before[0], first & 31), p1 = __shfl_sync(kFull, before[1], first & 31);
      if (m < live) {
        a.dla[(tok + m) * a.H + h] = (seg[i] == 0 ? start : 0.f) - (before[i] - (first < 32 ? p0 : p1));
        a.dbeta[(tok + m) * a.H + h] = ez[i] / beta[m];
      }
    }
  }
  // dq and dk
  const int64_t to_q = a.pdq ? static_cast<int64_t>(a.H) * a.dk : a.ld_dq, to_k = a.pdq ? to_q : a.ld_dk;
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int i = 32 * half + 16 * m + g + 8 * r;
      if (i >= live) continue;
      const int64_t oq = (tok + i) * to_q + h * a.dk, ok = (tok + i) * to_k + h * a.dk;
#pragma unroll
      for (int x = 0; x < NW; ++x) {
        const int cc = 8 * (w * NW + x) + 2 * t;
        if (cc >= a.dk) continue;
        const float q0 = dQ[m][x][2 * r], q1 = dQ[m][x][2 * r + 1], k0 = dK[m][x][2 * r], k1 = dK[m][x][2 * r + 1];
        if (a.pdq) {
          a.pdq[oq + cc] = q0;
          a.pdk[ok + cc] = k0;
          if (cc + 1 < a.dk) {
            a.pdq[oq + cc + 1] = q1;
            a.pdk[ok + cc + 1] = k1;
          }
        } else {
          const uint32_t vq = pack2(q0, q1), vk = pack2(k0, k1);
          if (a.pair_qk) {
            *reinterpret_cast<uint32_t *>(a.odq + oq + cc) = vq;
            *reinterpret_cast<uint32_t *>(a.odk + ok + cc) = vk;
          } else {
            a.odq[oq + cc] = static_cast<uint16_t>(vq);
            a.odk[ok + cc] = static_cast<uint16_t>(vk);
            if (cc + 1 < a.dk) {
              a.odq[oq + cc + 1] = static_cast<uint16_t>(vq >> 16);
              a.odk[ok + cc + 1] = static_cast<uint16_t>(vk >> 16);
            }
          }
        }
      }
    }
}

// dq and dk of key heads that several value heads share, heads in order
__global__ void __launch_bounds__(256) gdn_grad_heads(const Gdn a) {
  const int group = a.H / a.Hk;
  const int64_t tok = blockIdx.x;
  if (static_cast<int>(tok % a.T) >= length_of(a, static_cast<int>(tok / a.T))) return;
  for (int i = threadIdx.x; i < a.Hk * a.dk; i += 256) {
    const int hk = i / a.dk, ch = i - hk * a.dk;
    const int64_t o = (tok * a.H + static_cast<int64_t>(hk) * group) * a.dk + ch;
    float q = 0.f, k = 0.f;
    for (int e = 0; e < group; ++e) {
      q += a.pdq[o + static_cast<int64_t>(e) * a.dk];
      k += a.pdk[o + static_cast<int64_t>(e) * a.dk];
    }
    a.odq[tok * a.ld_dq + i] = static_cast<uint16_t>(pack2(q, 0.f));
    a.odk[tok * a.ld_dk + i] = static_cast<uint16_t>(pack2(k, 0.f));
  }
}

// ---------------------------------------------------------------------------
// Host.
// ---------------------------------------------------------------------------
struct Layout {
  int64_t n, units, tiles, state;  // chunks a sequence, chunks in all, 16-column tiles, floats of a kept state
  size_t scal, t3, m3, s, e, saved;
  size_t g, dz, pdq, pdk, work;
};

bool sizes_fit(int B, int T, int Hk, int H, int dk, int dv) {
  return B >= 0 && T >= 0 && H >= 0 && Hk >= 0 && B < 65536 && H < 65536 && T < (1 << 30) && dk >= 1 && dk <= 128 && dv >= 1 &&
         dv <= 1024 && (H == 0 || (Hk > 0 && H % Hk == 0)) &&
         static_cast<int64_t>(B) * H * ((T + kC - 1) / kC) * ((dv + 15) / 16) < INT_MAX &&
         static_cast<int64_t>(B) * H * ((dv + 15) / 16) < INT_MAX && static_cast<int64_t>(B) * T < INT_MAX;
}

Layout layout_of(int B, int T, int Hk, int H, int dk, int dv) {
  Layout l{};
  const auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const int dkp = dk <= 64 ? 64 : 128;
  l.n = (T + kC - 1) / kC;
  l.units = static_cast<int64_t>(B) * H * l.n;
  l.tiles = (dv + 15) / 16;
  l.state = l.tiles * 16 * dkp;
  const size_t units = static_cast<size_t>(l.units);
  l.scal = 0;
  l.t3 = up(l.scal + units * kScal * 4);
  l.m3 = up(l.t3 + units * 3 * kTri);
  l.s = up(l.m3 + units * 3 * kTri);
  l.e = up(l.s + units * l.state * 4);
  l.saved = up(l.e + units * l.tiles * 16 * kC * 4);
  const size_t part = Hk == H ? 0 : static_cast<size_t>(B) * T * H * dk * 4;
  l.g = 0;
  l.dz = up(static_cast<size_t>(B) * H * (l.n + 1) * l.state * 4);
  l.pdq = up(l.dz + units * l.tiles * 16 * kC * 4);
  l.pdk = up(l.pdq + part);
  l.work = up(l.pdk + part);
  return l;
}

int check_common(const char *what, const Gdn &a, const void *saved, size_t saved_bytes, const Layout &l) {
  if (l.units > 0 && (!a.q || !a.k || !a.v || !a.la || !a.beta || !saved))
    return set_error(SDM_ERR_INVALID_ARG, "%s: null pointer", what);
  if (a.ld_q < static_cast<int64_t>(a.Hk) * a.dk || a.ld_k < static_cast<int64_t>(a.Hk) * a.dk ||
      a.ld_v < static_cast<int64_t>(a.H) * a.dv || a.ld_q >= (1 << 27) || a.ld_k >= (1 << 27) || a.ld_v >= (1 << 27))
    return set_error(SDM_ERR_SHAPE, "%s: a token's row must be at most 2^27 elements from the next and hold its heads", what);
  if (!aligned(a.q, 2) || !aligned(a.k, 2) || !aligned(a.v, 2) || !aligned(a.la, 4) || !aligned(a.beta, 4) ||
      !aligned(a.lens, 4) || !aligned(a.err, 4) || !aligned(a.state_in, 4) || !aligned(a.state_out, 4) || !aligned(saved, 16))
    return set_error(SDM_ERR_ALIGN, "%s: a pointer is not aligned", what);
  if (saved_bytes < l.saved) return set_error(SDM_ERR_INVALID_ARG, "%s: saved holds %zu bytes, %zu needed", what, saved_bytes, l.saved);
  return SDM_OK;
}

// the bytes by which rows of `width` bf16 can be copied
int row_bytes(const void *p, int64_t ld, int width) {
  for (int n = 16; n > 2; n /= 2)
    if (width * 2 % n == 0 && ld * 2 % n == 0 && aligned(p, n)) return n;
  return 2;
}

// a tensor map of [tokens][heads][d] bf16, tokens ld elements apart, boxes of 64 tokens x 64 channels
int make_map(CUtensorMap *map, const void *p, int64_t ld, int64_t tokens, int heads, int d) {
  using Encode = decltype(&cuTensorMapEncodeTiled);
  static const Encode encode = [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q;
    return cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
                   q == cudaDriverEntryPointSuccess
               ? reinterpret_cast<Encode>(f)
               : nullptr;
  }();
  if (!encode) return set_error(SDM_ERR_CUDA, "gdn_train: the driver has no cuTensorMapEncodeTiled");
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(tokens)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(ld) * 2};
  const cuuint32_t box[3] = {64, 1, kC}, steps[3] = {1, 1, 1};
  if (encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(p), dims, strides, box, steps,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return set_error(SDM_ERR_CUDA, "gdn_train: cuTensorMapEncodeTiled failed");
  return SDM_OK;
}

int make_maps(Maps *m, const Gdn &a) {
  const int64_t tokens = static_cast<int64_t>(a.B) * a.T;
  int rc = SDM_OK;
  if (tokens == 0) return rc;
  if (a.by_qk == 16) rc = make_map(&m->q, a.q, a.ld_q, tokens, a.Hk, a.dk);
  if (rc == SDM_OK && a.by_qk == 16) rc = make_map(&m->k, a.k, a.ld_k, tokens, a.Hk, a.dk);
  if (rc == SDM_OK && a.by_v == 16) rc = make_map(&m->v, a.v, a.ld_v, tokens, a.H, a.dv);
  if (rc == SDM_OK && a.dy && a.by_dy == 16) rc = make_map(&m->dy, a.dy, static_cast<int64_t>(a.H) * a.dv, tokens, a.H, a.dv);
  return rc;
}

void place_saved(Gdn &a, void *saved, const Layout &l) {
  unsigned char *p = static_cast<unsigned char *>(saved);
  a.n = static_cast<int>(l.n);
  a.scal = reinterpret_cast<float *>(p + l.scal);
  a.t3 = p + l.t3;
  a.m3 = p + l.m3;
  a.s = reinterpret_cast<float *>(p + l.s);
  a.e = reinterpret_cast<float *>(p + l.e);
}

template <typename K>
int launch(K kernel, const char *what, int64_t grid, int threads, int smem, const Gdn &a, const Maps &maps, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return set_error(SDM_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  kernel<<<static_cast<unsigned>(grid), threads, smem, st>>>(a, maps);
  return check_launch(what);
}

// Tiles of 16 columns a CTA: one where every tile can have an SM of its own (its
// two warps then run on schedulers of their own), else two, else four, which share an SM's
// tensor cores and the chunk's tiles.
int chain_width(const Gdn &a, const Layout &l) {
  const int64_t all = l.tiles * a.B * a.H;
  return all <= kSms || l.tiles == 1 ? 1 : all <= 2 * kSms || l.tiles == 2 ? 2 : 4;
}

template <int NK, int W>
int run_chain(const Gdn &a, const Maps &maps, const Layout &l, bool back, cudaStream_t st) {
  const int64_t grid = (l.tiles + W - 1) / W * a.B * a.H;
  return back ? launch(gdn_chain_back<NK, W>, "gdn_backward", grid, W < 4 ? 64 * W + 32 : 64 * W, Chain<NK, 3, W>::size, a, maps, st)
              : launch(gdn_chain<NK, W>, "gdn_train", grid, W < 4 ? 64 * W + 32 : 64 * W, Chain<NK, 2, W>::size, a, maps, st);
}
template <int NK>
int run_chain(const Gdn &a, const Maps &maps, const Layout &l, bool back, cudaStream_t st) {
  const int w = chain_width(a, l);
  return w == 1 ? run_chain<NK, 1>(a, maps, l, back, st)
         : w == 2 ? run_chain<NK, 2>(a, maps, l, back, st) : run_chain<NK, 4>(a, maps, l, back, st);
}

template <int NK>
int run_train(const Gdn &a, const Layout &l, cudaStream_t st) {
  Maps maps{};
  int rc = make_maps(&maps, a);
  if (rc != SDM_OK) return rc;
  if (l.units > 0) {
    rc = launch(gdn_prep<NK>, "gdn_train", l.units, kPrepThreads, (2 * kC * kLd + 32 * 36 + kScal) * 4 + 16, a, maps, st);
    if (rc != SDM_OK) return rc;
  }
  return run_chain<NK>(a, maps, l, false, st);
}

template <int NK>
int run_backward(const Gdn &a, const Layout &l, cudaStream_t st) {
  Maps maps{};
  int rc = make_maps(&maps, a);
  if (rc == SDM_OK) rc = run_chain<NK>(a, maps, l, true, st);
  if (rc != SDM_OK || l.units == 0) return rc;
  rc = launch(gdn_grad<NK>, "gdn_backward", l.units, kGradThreads, Grad<NK>::size, a, maps, st);
  if (rc != SDM_OK || !a.pdq) return rc;
  gdn_grad_heads<<<static_cast<unsigned>(static_cast<int64_t>(a.B) * a.T), 256, 0, st>>>(a);
  return check_launch("gdn_backward");
}

}  // namespace

SDM_STICKY_ACCESSOR(sticky_gdn_train)

}  // namespace sdm

using namespace sdm;

extern "C" size_t gdn_train_saved_size(int B, int T, int Hk, int H, int dk, int dv) {
  return sizes_fit(B, T, Hk, H, dk, dv) ? layout_of(B, T, Hk, H, dk, dv).saved : 0;
}
extern "C" size_t gdn_backward_workspace_size(int B, int T, int Hk, int H, int dk, int dv) {
  return sizes_fit(B, T, Hk, H, dk, dv) ? layout_of(B, T, Hk, H, dk, dv).work : 0;
}

extern "C" int gdn_train(const float *state, float *state_out, const uint16_t *q, int64_t ld_q, const uint16_t *k,
                         int64_t ld_k, const uint16_t *v, int64_t ld_v, const float *log_alpha, const float *beta,
                         const uint8_t *reset, const int32_t *lens, int B, int T, int Hk, int H, int dk, int dv,
                         uint16_t *y, void *saved, size_t saved_bytes, int32_t *dev_err, void *stream) {
  if (B < 0 || T < 0 || Hk < 0 || H < 0) return set_error(SDM_ERR_INVALID_ARG, "gdn_train: negative size");
  if (!sizes_fit(B, T, Hk, H, dk, dv)) return set_error(SDM_ERR_SHAPE, "gdn_train: sizes beyond the limits");
  const Layout l = layout_of(B, T, Hk, H, dk, dv);
  Gdn a{};
  a.q = q; a.k = k; a.v = v;
  a.ld_q = ld_q; a.ld_k = ld_k; a.ld_v = ld_v;
  a.la = log_alpha; a.beta = beta; a.reset = reset; a.lens = lens;
  a.B = B; a.T = T; a.Hk = Hk; a.H = H; a.dk = dk; a.dv = dv;
  a.state_in = state; a.state_out = state_out; a.y = y; a.err = dev_err;
  if (static_cast<int64_t>(B) * H > 0 && (!state_out || (T > 0 && !y))) return set_error(SDM_ERR_INVALID_ARG, "gdn_train: null pointer");
  const int rc = check_common("gdn_train", a, saved, saved_bytes, l);
  if (rc != SDM_OK) return rc;
  if (!aligned(y, 2)) return set_error(SDM_ERR_ALIGN, "gdn_train: a pointer is not aligned");
  if (B == 0 || H == 0) return SDM_OK;
  a.by_qk = std::min(row_bytes(q, ld_q, dk), row_bytes(k, ld_k, dk));
  a.by_v = row_bytes(v, ld_v, dv);
  a.pair_y = dv % 2 == 0 && aligned(y, 4);
  place_saved(a, saved, l);
  return dk <= 64 ? run_train<4>(a, l, static_cast<cudaStream_t>(stream)) : run_train<8>(a, l, static_cast<cudaStream_t>(stream));
}

extern "C" int gdn_backward(const float *dstate, float *dstate_out, const uint16_t *q, int64_t ld_q, const uint16_t *k,
                            int64_t ld_k, const uint16_t *v, int64_t ld_v, const float *log_alpha, const float *beta,
                            const uint8_t *reset, const int32_t *lens, const void *saved, size_t saved_bytes,
                            const uint16_t *dy, int B, int T, int Hk, int H, int dk, int dv, uint16_t *dq, int64_t ld_dq,
                            uint16_t *dk_out, int64_t ld_dk, uint16_t *dv_out, int64_t ld_dv, float *dlog_alpha,
                            float *dbeta, void *workspace, size_t workspace_bytes, int32_t *dev_err, void *stream) {
  if (B < 0 || T < 0 || Hk < 0 || H < 0) return set_error(SDM_ERR_INVALID_ARG, "gdn_backward: negative size");
  if (!sizes_fit(B, T, Hk, H, dk, dv)) return set_error(SDM_ERR_SHAPE, "gdn_backward: sizes beyond the limits");
  const Layout l = layout_of(B, T, Hk, H, dk, dv);
  Gdn a{};
  a.q = q; a.k = k; a.v = v; a.dy = dy;
  a.ld_q = ld_q; a.ld_k = ld_k; a.ld_v = ld_v; a.ld_dq = ld_dq; a.ld_dk = ld_dk; a.ld_dv = ld_dv;
  a.la = log_alpha; a.beta = beta; a.reset = reset; a.lens = lens;
  a.B = B; a.T = T; a.Hk = Hk; a.H = H; a.dk = dk; a.dv = dv;
  a.state_in = dstate; a.state_out = dstate_out; a.err = dev_err;
  a.odq = dq; a.odk = dk_out; a.odv = dv_out; a.dla = dlog_alpha; a.dbeta = dbeta;
  if (static_cast<int64_t>(B) * H > 0 &&
      (!dstate_out || !workspace || (T > 0 && (!dy || !dq || !dk_out || !dv_out || !dlog_alpha || !dbeta))))
    return set_error(SDM_ERR_INVALID_ARG, "gdn_backward: null pointer");
  const int rc = check_common("gdn_backward", a, saved, saved_bytes, l);
  if (rc != SDM_OK) return rc;
  if (ld_dq < static_cast<int64_t>(Hk) * dk || ld_dk < static_cast<int64_t>(Hk) * dk || ld_dv < static_cast<int64_t>(H) * dv ||
      ld_dq >= (1 << 27) || ld_dk >= (1 << 27) || ld_dv >= (1 << 27))
    return set_error(SDM_ERR_SHAPE, "gdn_backward: a token's row must be at most 2^27 elements from the next and hold its heads");
  if (!aligned(dy, 2) || !aligned(dq, 2) || !aligned(dk_out, 2) || !aligned(dv_out, 2) || !aligned(dlog_alpha, 4) ||
      !aligned(dbeta, 4) || !aligned(workspace, 16))
    return set_error(SDM_ERR_ALIGN, "gdn_backward: a pointer is not aligned");
  if (workspace_bytes < l.work)
    return set_error(SDM_ERR_INVALID_ARG, "gdn_backward: workspace of %zu bytes, %zu needed", workspace_bytes, l.work);
  if (B == 0 || H == 0) return SDM_OK;
  a.by_qk = std::min(row_bytes(q, ld_q, dk), row_bytes(k, ld_k, dk));
  a.by_v = row_bytes(v, ld_v, dv);
  a.by_dy = row_bytes(dy, static_cast<int64_t>(H) * dv, dv);
  a.pair_y = dv % 2 == 0 && ld_dv % 2 == 0 && aligned(dv_out, 4);
  a.pair_qk = dk % 2 == 0 && ld_dq % 2 == 0 && ld_dk % 2 == 0 && aligned(dq, 4) && aligned(dk_out, 4);
  place_saved(a, const_cast<void *>(saved), l);
  unsigned char *p = static_cast<unsigned char *>(workspace);
  a.g = reinterpret_cast<float *>(p + l.g);
  a.dz = reinterpret_cast<float *>(p + l.dz);
  if (Hk != H) {
    a.pdq = reinterpret_cast<float *>(p + l.pdq);
    a.pdk = reinterpret_cast<float *>(p + l.pdk);
  }
  return dk <= 64 ? run_backward<4>(a, l, static_cast<cudaStream_t>(stream))
                  : run_backward<8>(a, l, static_cast<cudaStream_t>(stream));
}
