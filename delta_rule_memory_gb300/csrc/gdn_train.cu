// gdn_train.cu - training of the gated delta rule: the chunked forward that keeps what its backward needs, and
// the backward.
//
// Per sequence and head, S [dk, dv]:
//   S~ = e^{a_t} S (0 at a reset),  E_t = v_t - S~^T k_t,
//   S_t = S~ + beta_t k_t E_t^T,    y_t = S_t^T q_t.
// In a chunk of C = 64 tokens let l_i be the sum of the a's up to token i, D_ij = e^{l_i - l_j} for j <= i in
// one document (else 0), gam_i = D from the chunk's start (0 behind a reset), tail_j = D to its end.  With S
// the state at the chunk's start, rows being tokens,
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
// The decays' gradient is the sum of what passes token t's decay, each term with that decay in it:
//   da_t = gam_C <S, G> + sum over i >= t of gam_i (q_i . S dY_i - k_i . S dZ_i)
//        + sum over j < t of tail_j k_j . G U_j + sum over i >= t > j of (X_ij q_i . k_j + N_ij k_i . k_j).
// (A running sum of q . dq - v . dv taken off <S, G_start> is the same and needs no product of its own, but its
// terms do not get smaller with the decay: at e^-8 a token their difference is 5e-4 off, at e^-16 half of it.)
//
// Kernels.  gdn_prep (every chunk by itself): the decays, T and M.  gdn_chain: chunk after chunk, three to eight
// warps a tile of 16 value columns; every product of a chunk takes the one before as its A operand from registers
// or as parts in shared memory (mma.cuh), and the chunk's tiles are copied a chunk ahead.  gdn_chain_back: the same
// with G, last chunk to first.  gdn_grad: everything that needs sums over the value columns, every chunk by
// itself, on tcgen05. The chains use mma.sync: a product there is 64 x 128 x 16 and feeds the next one, so
// through tensor memory each would be read back, split into bf16 parts and stored before the next could start,
// which is what bounds the chunk form in gdn_chunk.cu (2.85 us a chunk for 64 columns, with two parts).
//
// Precision.  q, k, v and dy are exact in bf16.  What is not (S, G, T, M, Z, U, X) is taken in three bf16
// parts, all 24 bits of it; y, dq, dk and dv are rounded to bf16 once, from fp32 sums.
//
// B = 4, T = 4096, H = 16, dk = dv = 128: gdn_prep 89 us, gdn_chain 344 (with two parts behind y 318),
// gdn_chain_back 384, gdn_grad 419.
#include <cuda.h>

#include <algorithm>
#include <climits>

#include "common.cuh"
#include "mma.cuh"
#include "umma.cuh"

namespace sdm {

int test_drop_signal();  // gdn_chunk.cu: the SDM_TEST_DROP_SIGNAL test hook

namespace {

using namespace mma;

constexpr int kSms = 152;
constexpr int kC = 64;                  // tokens of a chunk
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
  int drop;                    // test hook: M is not asked for
};

// A triangle: 16 x 16 blocks row by row, each as four 8 x 8 of 8 rows of 16 bytes
__device__ __forceinline__ constexpr int block_at(int i, int j) { return (i * (i + 1) / 2 + j) * 512; }
// B fragments (two n-tiles, one k-step) of block (n, k), B[k][n] = tri[n][k] ...
__device__ __forceinline__ void tri_rows(uint32_t tri, int n, int k, int lane, uint32_t (&r)[4]) {
  ldsm4(tri + block_at(n, k) + lane * 16, r);
}
// ... and of block (k, n), B[k][n] = tri[k][n]
__device__ __forceinline__ void tri_cols(uint32_t tri, int n, int k, int lane, uint32_t (&r)[4]) {
  ldsm_x4_trans(tri + block_at(k, n) + ((lane & 8) << 5) + ((lane & 16) << 3) + (lane & 7) * 16, r);
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

// 2^x: ex2.approx of the upper float, 2^-22 relative, and what the lower one adds to first order (it is below
// 2^-24 of the upper one, which is at most 2^15 here).  The upper one alone is off by that: 7e-7 of the result at
// e^-20, twice that for a difference of two of them in 32 bits
__device__ __forceinline__ float exp2_wide(Wide x) {
  const float e = umma::ex2_approx(x.hi);
  return fmaf(e, x.lo * 0.693147181f, e);
}

// the decay from token j to a later token i: their sums' difference with its rounding, which is exact where no decay
// in between is above 1
__device__ __forceinline__ float decay_between(Wide i, Wide j) {
  const float hi = i.hi - j.hi;
  return exp2_wide({hi, ((i.hi - hi) - j.hi) + (i.lo - j.lo)});
}

// Tensor maps of q, k, v and dy as [token][head][channel], boxes of one panel; set where rows can be copied by
// 16 bytes
struct Maps {
  CUtensorMap q, k, v, dy;
};

constexpr uint32_t kWaitLimit = 1u << 20;  // polls (about 0.1 s) before a wait gives up
constexpr uint32_t kShortLimit = 1u << 12;  // ... once one has: still far longer than a copy takes

// Wait for a phase of copies.  One that gives up is reported and lets the kernel run to its end, its later
// waits short.
__device__ __forceinline__ bool wait_copies(uint64_t *bar, uint32_t parity, uint32_t &limit, const Gdn &a) {
  if (umma::mbar_wait(smem_u32(bar), parity, limit)) return true;
  report_timeout(a.err);
  limit = kShortLimit;
  return false;
}

// Before a kernel's first access to memory: the kernel before it in the stream has ended and its results are
// there; the next one may be brought up.
__device__ __forceinline__ void before_reading() {
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
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
    // eight lanes, eight rows: 128 bytes in a row of the triangle
    const int i = ((id >> 6) << 3) | (id & 7), p = (id >> 3) & 7;
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

// X = L^-1 for unit lower triangular L: the 16 x 16 diagonal blocks by substitution (one a warp), then blocks
// joined two by two, X21 = -X22 (L21 X11), whose inner products lie in L's upper right quarter.
__device__ __forceinline__ void invert(float *L, float *X, int tid) {
  float *zt = L + 32;
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
    float *z = zt + pr * 16 * kLd;
    *reinterpret_cast<float4 *>(z + r * kLd + c) = make_float4(acc[0][0], acc[0][1], acc[0][2], acc[0][3]);
    __syncthreads();
    strip<1, 16>(X + (o + 16 + r) * kLd + o + 16, kLd, z + c, kLd, acc);
    *reinterpret_cast<float4 *>(X + (o + 16 + r) * kLd + o + c) =
        make_float4(-acc[0][0], -acc[0][1], -acc[0][2], -acc[0][3]);
  }
  __syncthreads();
  {  // 32 -> 64
    const int r = (tid >> 3) * 2, c = (tid & 7) * 4;
    float acc[2][4];
    strip<2, 32>(L + (32 + r) * kLd, kLd, X + c, kLd, acc);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<float4 *>(zt + (r + i) * kLd + c) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
    __syncthreads();
    strip<2, 32>(X + (32 + r) * kLd + 32, kLd, zt + c, kLd, acc);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<float4 *>(X + (32 + r + i) * kLd + c) =
          make_float4(-acc[i][0], -acc[i][1], -acc[i][2], -acc[i][3]);
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
  float *sL = reinterpret_cast<float *>(sm), *sX = sL + kC * kLd, *sc = sX + kC * kLd;
  uint64_t *bar = reinterpret_cast<uint64_t *>(sc + kScal);
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int64_t u = blockIdx.x;
  const int64_t bh = u / a.n;
  const int c = static_cast<int>(u - bh * a.n), b = static_cast<int>(bh / a.H),
      h = static_cast<int>(bh - static_cast<int64_t>(b) * a.H);
  before_reading();
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
    // l in units of log2, as two floats: a strong decay early in the chunk costs the later, weak ones nothing
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
      const float v[6] = {seg[i] == 0 ? exp2_wide(x[i]) : 0.f, seg[i] == last ? exp2_wide(rest) : 0.f,
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
      const float d = on ? decay_between({lh[i], ll[i]}, {lh[j], ll[j]}) : 0.f;
      sL[i * kLd + j] = on && j < i ? d * G[nt][e] * be[j] : 0.f;
      sX[i * kLd + j] = on ? d * P[nt][e] : 0.f;
    }
  }
  __syncthreads();
  write_tiles(sX, a.m3 + u * (3 * kTri), tid);
  __syncthreads();
  invert(sL, sX, tid);
  write_tiles(sX, a.t3 + u * (3 * kTri), tid);
}

// ---------------------------------------------------------------------------
// The chains.  A CTA has W tiles of 16 value columns of one head, each with M + H warps.  M (two or four) do
// what the next chunk waits for, each with its share of the key channels (the sums with the state and its
// update) and of the four groups of 16 tokens (of two warps, 0 and 3, or 1 and 2, the same number of the
// triangle's blocks): sums over all channels and a triangle's products meet in shared memory.  The H others do
// everything else: y, the products with dy, copies.  Warps meet by named barriers, only where one needs what
// another wrote; a stage of copies is asked for again once all have left it.  A tile's state lives in shared
// memory as its three bf16 parts, which are all 24 bits of it, in the order of the A fragments that every
// product with it takes.
// Bound by latency where a tile has an SM to itself (M = H = 4; 1.9 us a chunk forward, 2.0 backward at dk =
// dv = 128; M = 2 and H = 1, all warps meeting once a chunk, took 2.6 and 3.4, one warp for everything 7.6 and
// 6.5).  Where four tiles share an SM (M = 2, H = 1; 5.4 and 6.0 us a chunk) by the tensor cores, about 6,500 of
// 10,500 and of 11,700 cycles, and shared memory beside them: mma.sync runs at 600 TFLOP/s.  Loops are kept
// small: unrolled four times the backward chain is a fifth slower, its instructions no longer at hand.
// ---------------------------------------------------------------------------
template <int NK, bool BACK, int W, int M, int H>
struct Chain {
  static constexpr int P = NK / 4;  // panels of K and Q
  static constexpr int K = 0, Q = K + P * kPanel, V = Q + P * kPanel, T = V + kPanel, sc = T + 3 * kTri,
                       stage = (sc + 3 * kC * 4 + 1023) / 1024 * 1024;
  // places of U: with one, the main warps wait until the helping ones have read the chunk before's
  static constexpr int places = !BACK && W < 4 ? 2 : 1;
  // M is read early in a chunk only, so one place does
  static constexpr int Mq = 2 * stage, state = Mq + 3 * kTri, parts = state + W * NK * 3 * 512,
                       tokens = parts + W * 4 * 3 * 512, sums = tokens + places * W * 8 * 512,
                       bars = sums + (M == 4 ? W * 4 * 8 * 512 : 0), size = bars + 48 + W * 8;
};
static_assert(Chain<8, true, 4, 2, 1>::size <= kMaxSmem && Chain<8, false, 4, 2, 1>::size <= kMaxSmem &&
                  Chain<8, false, 2, 4, 2>::size <= kMaxSmem, "");
template <int W, int M, int H>
constexpr int kChainThreads = 32 * W * (M + H) + (W == 1 ? 32 : 0);

// A chunk's tiles into a stage; cols: the value columns' tensor.  What tensor and bulk copies bring is asked
// for by one lane of a warp of its own or, where a CTA has more tiles than one, whose warps need its registers,
// by one lane of each of the four helping warps (a request holds its warp for a hundred cycles and more; with
// one tile they are what the chain waits for: 794 us in place of 750 backward at B = 1, T = 16384, H = 8).
template <int W>
constexpr int kAskers = W == 1 ? 1 : 4;

template <int NK, bool BACK, int W, int M, int H>
__device__ __forceinline__ void request_stage(unsigned char *st, uint64_t *bar, const Gdn &a, const Maps &maps,
                                              int64_t u, int64_t tok, int h, int col0, int by_cols,
                                              const CUtensorMap *cols_map, int who) {
  using L = Chain<NK, BACK, W, M, H>;
  constexpr bool all = kAskers<W> == 1;
  static_assert(all || W * H == kAskers<W>, "");
  const uint32_t mb = smem_u32(bar);
  const int hk = h / (a.H / a.Hk), token = static_cast<int>(tok);
  const bool qk = a.by_qk == 16, cols = by_cols == 16;
  const uint32_t part[4] = {qk ? L::P * kPanel : 0u, qk ? L::P * kPanel : 0u, 3 * kTri + (cols ? kPanel : 0u),
                            3 * kC * 4u};
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
    umma::bulk_g2s(smem_u32(st + L::sc), a.scal + u * kScal, 3 * kC * 4, mb);
  }
}
__device__ __forceinline__ void request_m(unsigned char *to, uint64_t *bar, const Gdn &a, int64_t u) {
  umma::mbar_expect_tx(smem_u32(bar), 3 * kTri);
  umma::bulk_g2s(smem_u32(to), a.m3 + u * (3 * kTri), 3 * kTri, smem_u32(bar));
}
// ... and the rest, by the helping warps
template <int NK, bool BACK, int W, int M, int H>
__device__ __forceinline__ void copy_stage(unsigned char *st, const Gdn &a, int64_t tok, int h, int col0, int live,
                                           const uint16_t *cols, int64_t ld_cols, int by_cols, int tid) {
  using L = Chain<NK, BACK, W, M, H>;
  constexpr int threads = 32 * W * H;
  const int hk = h / (a.H / a.Hk), from = col0 & ~63;  // whole panels of value columns
  if (a.by_qk != 16) {
    load_tile<L::P, threads>(st + L::K, a.k + tok * a.ld_k + hk * a.dk, a.ld_k, live, a.dk, a.by_qk, tid);
    load_tile<L::P, threads>(st + L::Q, a.q + tok * a.ld_q + hk * a.dk, a.ld_q, live, a.dk, a.by_qk, tid);
  }
  if (by_cols != 16)
    load_tile<1, threads>(st + L::V, cols + tok * ld_cols + h * a.dv + from, ld_cols, live, min(64, a.dv - from),
                          by_cols, tid);
  cp_async_commit();
}

// the rows behind a chunk's last token, which tensor copies fill with whatever follows it
template <int NK, bool BACK, int W, int M, int H>
__device__ __forceinline__ void clear_stage(unsigned char *st, const Gdn &a, int live, int by_cols, int tid) {
  using L = Chain<NK, BACK, W, M, H>;
  if (a.by_qk == 16) {
    clear_rows<L::P, 32 * W * H>(st + L::K, live, tid);
    clear_rows<L::P, 32 * W * H>(st + L::Q, live, tid);
  }
  if (by_cols == 16) clear_rows<1, 32 * W * H>(st + L::V, live, tid);
  umma::fence_async_smem();
}

// S^T of 16 columns and 8 NT rows of a [dk][dv] matrix as an accumulator, and back
template <int NT>
__device__ __forceinline__ void read_state(const float *m, int row, int dk, int dv, int col, int lane,
                                           float (&S)[NT][4]) {
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
__device__ __forceinline__ void write_state(float *m, int row, int dk, int dv, int col, int lane,
                                            const float (&S)[NT][4]) {
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
// d (the leading parts' product) and l (the others') += A B for n-tiles 2 np and 2 np + 1, over the parts whose
// numbers sum up to less than max(PA, PB): what the others hold is below the last bit kept.  The tensor cores
// cut sums off where an addition would round; kept apart, the many small products do so at their own size.
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

// acc = A B for X blocks of 16 columns, B = tile[token][column] exact, over 64 tokens: the small parts first
template <int X>
__device__ __forceinline__ void block_product(uint32_t tile, int block, const uint32_t (&a)[4][3][4], int lane,
                                              float (&acc)[2 * X][4]) {
  uint32_t r[4][X][4];
#pragma unroll
  for (int ks = 0; ks < 4; ++ks)
#pragma unroll
    for (int x = 0; x < X; ++x) b_cols(tile, 16 * (block + x), 16 * ks, lane, r[ks][x]);
  clear(acc);
#pragma unroll
  for (int p = 2; p >= 0; --p)
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)
#pragma unroll
      for (int x = 0; x < X; ++x) {
        fma16816(acc[2 * x], a[ks][p], r[ks][x][0], r[ks][x][1]);
        fma16816(acc[2 * x + 1], a[ks][p], r[ks][x][2], r[ks][x][3]);
      }
}

// state <- factor state + sign acc for X blocks of 16 channels; x: its new values
template <int X>
__device__ __forceinline__ void update_blocks(uint4 *parts, int block, int lane, float factor, float sign,
                                              const float (&acc)[2 * X][4], float (&x)[2 * X][4]) {
#pragma unroll
  for (int i = 0; i < X; ++i) {
    uint4 *m = parts + (block + i) * 96;
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

// d = the product of N k-steps of the state with tile[token][key channel], channels from k0 on; U of them
// unrolled
template <int N, int U>
__device__ __forceinline__ void state_product(const uint4 *parts, uint32_t tile, int k0, int lane, float (&d)[8][4]) {
  float l[8][4];
  clear(d);
  clear(l);
#pragma unroll(U)
  for (int ks = 0; ks < N; ++ks) {
    uint32_t s[3][4], r[4][4];
    get_parts(parts + ks * 96, lane, s);
#pragma unroll
    for (int np = 0; np < 4; ++np) b_rows(tile, 16 * np, k0 + 16 * ks, lane, r[np]);
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

// Of the four groups of 16 tokens, the i-th of warp x of N that share them
template <int N>
__device__ __forceinline__ constexpr int group_of(int x, int i) {
  return N == 1 ? i : N == 4 ? x : x == 0 ? (i ? 3 : 0) : 1 + i;
}
template <int N>
__device__ __forceinline__ constexpr int tile_of(int x, int i) { return 2 * group_of<N>(x, i >> 1) + (i & 1); }
// Sums over all tokens, a part of them with each of M warps: the own groups' n-tiles, and the others' through
// shared memory (of two warps eight tiles, each written by the one that does not keep it; of four all of them)
template <int M>
__device__ __forceinline__ void give_sums(float4 *m, int x, int lane, const float (&d)[8][4], float (&mine)[8 / M][4]) {
  if constexpr (M == 4) {
    put(m + x * 8 * 32, lane, d);
    clear(mine);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int a = i < 2 ? i : i + 4, b = i + 2;  // n-tiles of groups 0 and 3, of 1 and 2
      m[(x ? a : b) * 32 + lane] = x ? make_float4(d[a][0], d[a][1], d[a][2], d[a][3])
                                     : make_float4(d[b][0], d[b][1], d[b][2], d[b][3]);
#pragma unroll
      for (int e = 0; e < 4; ++e) mine[i][e] = x ? d[b][e] : d[a][e];
    }
  }
}
template <int M, int N>
__device__ __forceinline__ void add_tiles(const float4 *m, int x, int lane, float (&mine)[N][4]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float4 v = m[tile_of<M>(x, i) * 32 + lane];
    mine[i][0] += v.x, mine[i][1] += v.y, mine[i][2] += v.z, mine[i][3] += v.w;
  }
}
template <int M>
__device__ __forceinline__ void take_sums(const float4 *m, int x, int lane, float (&mine)[8 / M][4]) {
#pragma unroll
  for (int y = 0; y < (M == 4 ? 4 : 1); ++y) add_tiles<M>(m + y * 8 * 32, x, lane, mine);
}
template <int M, int N>
__device__ __forceinline__ void put_tiles(float4 *m, int x, int lane, const float (&mine)[N][4]) {
#pragma unroll
  for (int i = 0; i < N; ++i)
    m[tile_of<M>(x, i) * 32 + lane] = make_float4(mine[i][0], mine[i][1], mine[i][2], mine[i][3]);
}
template <int M>
__device__ __forceinline__ void put_groups(uint4 *parts, int x, int lane, const float (&mine)[8 / M][4]) {
#pragma unroll
  for (int i = 0; i < 4 / M; ++i) put_parts(parts + group_of<M>(x, i) * 96, lane, mine[2 * i], mine[2 * i + 1]);
}
template <int M, int N>
__device__ __forceinline__ void scale_groups(float (&mine)[N][4], int x, const float *f, int t) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float2 v = *reinterpret_cast<const float2 *>(f + 8 * tile_of<M>(x, i) + 2 * t);
    mine[i][0] *= v.x, mine[i][1] *= v.y, mine[i][2] *= v.x, mine[i][3] *= v.y;
  }
}

// the own groups of X T^T (BACK: X T), X's parts in shared memory, T a triangle in three parts
template <bool BACK, int M>
__device__ __forceinline__ void triangle_product(const uint4 *parts, uint32_t tri, int x, int lane,
                                                 float (&d)[8 / M][4]) {
#pragma unroll
  for (int i = 0; i < 4 / M; ++i) {
    const int n = group_of<M>(x, i), first = BACK ? n : 0, last = BACK ? 3 : n;
    float h[2][4], l[2][4], m[2][4];  // parts 0 0; 0 1 and 1 0; 1 1, 0 2 and 2 0
    clear(h);
    clear(l);
    clear(m);
#pragma unroll 1
    for (int ks = first; ks <= last; ++ks) {
      uint32_t a[3][4], r[3][4];
      get_parts(parts + ks * 96, lane, a);
#pragma unroll
      for (int p = 0; p < 3; ++p)
        BACK ? tri_cols(tri + p * kTri, n, ks, lane, r[p]) : tri_rows(tri + p * kTri, n, ks, lane, r[p]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        fma16816(m[j], a[1], r[1][2 * j], r[1][2 * j + 1]);
        fma16816(l[j], a[0], r[1][2 * j], r[1][2 * j + 1]);
        fma16816(h[j], a[0], r[0][2 * j], r[0][2 * j + 1]);
        fma16816(m[j], a[0], r[2][2 * j], r[2][2 * j + 1]);
        fma16816(l[j], a[1], r[0][2 * j], r[0][2 * j + 1]);
        fma16816(m[j], a[2], r[0][2 * j], r[0][2 * j + 1]);
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) d[2 * i + j][e] = h[j][e] + (l[j][e] + m[j][e]);
  }
}

// a tile's first M warps, or all of them, meet
__device__ __forceinline__ void meet(int id, int threads) {
  asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(threads) : "memory");
}
// ... or only tell the others that they are there
__device__ __forceinline__ void arrive(int id, int threads) {
  asm volatile("bar.arrive %0, %1;\n" ::"r"(id), "r"(threads) : "memory");
}

// where a warp of a chain stands
template <int W>
struct Place {
  int tid, role, w, lane, col0, col, b, h, len, n;  // role: which of the tile's warps
  int64_t bh, tok;
  bool mine;  // else the tile lies behind dv, and its warps only help with the copies
  __device__ __forceinline__ explicit Place(const Gdn &a) {
    tid = threadIdx.x, role = tid / (32 * W), w = (tid >> 5) % W, lane = tid & 31;
    const int tiles = (a.dv + 15) >> 4, groups = (tiles + W - 1) / W;
    bh = blockIdx.x / groups;
    col0 = static_cast<int>(blockIdx.x - bh * groups) * (16 * W), col = col0 + 16 * w;
    b = static_cast<int>(bh / a.H), h = static_cast<int>(bh - static_cast<int64_t>(b) * a.H);
    len = length_of(a, b), n = (len + kC - 1) / kC;
    tok = static_cast<int64_t>(b) * a.T;
    mine = col < a.dv;
  }
};

template <int NK, int W, int M, int H>
__global__ void __launch_bounds__(kChainThreads<W, M, H>, 1) gdn_chain(const Gdn a,
    const __grid_constant__ Maps maps) {
  using L = Chain<NK, false, W, M, H>;
  constexpr int NT = 2 * NK, kOwn = 32 * W * (M + H);  // kOwn: threads before the warp that asks for copies
  constexpr int kBlocks = NK / M, X = kBlocks < 2 ? 1 : 2;        // blocks of 16 channels of a warp's; taken at once
  extern __shared__ __align__(1024) unsigned char sm[];
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::bars);  // two stages there, M there, two stages free, ...
  uint64_t *read = bars + 6;                                     // ... each tile's U read
  if (threadIdx.x == 0) {
    umma::mbar_init(smem_u32(bars), kAskers<W>);
    umma::mbar_init(smem_u32(bars + 1), kAskers<W>);
    umma::mbar_init(smem_u32(bars + 2), 1);
    umma::mbar_init(smem_u32(bars + 3), W * (M + H));
    umma::mbar_init(smem_u32(bars + 4), W * (M + H));
    for (int i = 0; i < W; ++i) umma::mbar_init(smem_u32(read + i), H);
    umma::fence_mbar_init();
  }
  before_reading();
  const Place<W> me(a);
  const int tid = me.tid, w = me.w, lane = me.lane, g = lane >> 2, t = lane & 3, n = me.n, len = me.len, col = me.col,
      h = me.h;
  const int tiles = (a.dv + 15) >> 4;
  uint4 *hS = reinterpret_cast<uint4 *>(sm + L::state) + w * NK * 96,
      *hP = reinterpret_cast<uint4 *>(sm + L::parts) + w * 4 * 96;
  const auto place = [&](int c) {  // U^T, in fp32
    return reinterpret_cast<float4 *>(sm + L::tokens) + ((c % L::places) * W + w) * 8 * 32;
  };
  if (tid == 0 && a.err && a.lens && a.lens[me.b] != len) atomicOr(a.err, SDM_DEVERR_INDEX_RANGE);
  __syncthreads();
  uint32_t limit = tid < kOwn ? kWaitLimit : 4 * kWaitLimit;  // a warp that only asks for copies outwaits the others
  const int pair = 1 + w, all = 1 + W + w, ready = 1 + 2 * W + w;  // barriers
  const bool together = a.by_qk != 16 || a.by_v != 16;  // tiles that the helping warps copy: all warps meet for them
  const auto done = [&](int c) {  // this warp has read the chunk's stage
    __syncwarp();
    if (lane == 0) umma::mbar_arrive(smem_u32(bars + 3 + (c & 1)));
  };
  // ... and so have all others; where that is not seen, nothing more is asked for
  bool ask = true;
  const auto wait_done = [&](int c) { ask = ask && wait_copies(bars + 3 + (c & 1), (c >> 1) & 1, limit, a); };

  if (me.role < M) {
    const int x = me.role, vp = ((me.col0 & 63) >> 3) + 2 * w;  // vp: the tile's pieces of the value columns' panel
    uint4 *own = hS + x * kBlocks * 96;
    float S[2 * kBlocks][4];  // the own channels' state beside its parts
    // a row that starts with a reset does not read it: gam would be 0, but does not take a NaN away.  (Resets further
    // on multiply by 0.  The same there, where a chunk's first token resets, made every chunk 0.1 us longer.)
    const bool given = a.state_in && !(a.reset && n > 0 && a.reset[me.tok] != 0);
    read_state(given ? a.state_in + me.bh * a.dk * a.dv : nullptr, x * kBlocks * 16, a.dk, a.dv, col, lane, S);
#pragma unroll
    for (int ks = 0; ks < kBlocks; ++ks) put_parts(own + ks * 96, lane, S[2 * ks], S[2 * ks + 1]);
    if (me.mine && n > 0) arrive(ready, 32 * (M + H));  // the state's parts are there
    for (int c = 0; c < n; ++c) {
      if (together) __syncthreads();
      wait_copies(bars + (c & 1), (c >> 1) & 1, limit, a);
      if (len - c * kC < kC) __syncthreads();  // the helping warps clear rows
      if (!me.mine) {
        done(c);
        continue;
      }
      float4 *hU = place(c);
      float4 *hX = M == 4 ? reinterpret_cast<float4 *>(sm + L::sums) + w * 32 * 32 : hU;  // partial sums, before U
      unsigned char *st = sm + (c & 1) * L::stage;
      const uint32_t uK = smem_u32(st + L::K), uV = smem_u32(st + L::V);
      const float *gam = reinterpret_cast<const float *>(st + L::sc), *tail = gam + kC, *beta = tail + kC;
      const int64_t at = (me.bh * a.n + c) * tiles + (col >> 4);
      put(reinterpret_cast<float4 *>(a.s) + at * (NT * 32) + x * kBlocks * 64, lane, S);
      float Z[8 / M][4];
      {
        float d[8][4];
        state_product<kBlocks, kBlocks>(own, uK, x * kBlocks * 16, lane, d);
        if (L::places == 1 && c > 0) wait_copies(read + w, (c - 1) & 1, limit, a);
        give_sums<M>(hX, x, lane, d, Z);
      }
      uint32_t v[4 / M][4];
#pragma unroll
      for (int i = 0; i < 4 / M; ++i)  // tile[token][column]: rows of V^T are its columns
        ldsm_x4_trans(
            uV + piece(16 * group_of<M>(x, i) + (((lane >> 4) & 1) << 3) + (lane & 7), vp + ((lane >> 3) & 1)), v[i]);
      meet(pair, 32 * M);
      take_sums<M>(hX, x, lane, Z);
      // Z^T = V^T - gam S^T K^T
#pragma unroll
      for (int i = 0; i < 4 / M; ++i) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 gm = *reinterpret_cast<const float2 *>(gam + 8 * tile_of<M>(x, 2 * i + j) + 2 * t);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t vv = v[i][2 * j + (e >> 1)];
            Z[2 * i + j][e] = fmaf(e & 1 ? -gm.y : -gm.x, Z[2 * i + j][e], e & 1 ? high2(vv) : low2(vv));
          }
        }
      }
      float E[8 / M][4];
      put_groups<M>(hP, x, lane, Z);
      meet(pair, 32 * M);
      triangle_product<false, M>(hP, smem_u32(st + L::T), x, lane, E);
      put_tiles<M>(reinterpret_cast<float4 *>(a.e) + at * 256, x, lane, E);
      scale_groups<M>(E, x, beta, t);
      put_tiles<M>(hU, x, lane, E);
      meet(all, 32 * (M + H));  // U is there, S and Z have been read
      // S^T = gam_C S^T + (tail U)^T K
      scale_groups<M>(E, x, tail, t);
      put_groups<M>(hP, x, lane, E);
      meet(pair, 32 * M);
      uint32_t ut[4][3][4];
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) get_parts(hP + ks * 96, lane, ut[ks]);
      const float end = gam[kC - 1];
#pragma unroll
      for (int q = 0; q < kBlocks; q += X) {
        float acc[2 * X][4];
        block_product<X>(uK, x * kBlocks + q, ut, lane, acc);
#pragma unroll
        for (int i = 0; i < 2 * X; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) S[2 * q + i][e] = fmaf(end, S[2 * q + i][e], acc[i][e]);
#pragma unroll
        for (int i = 0; i < X; ++i) put_parts(own + (q + i) * 96, lane, S[2 * (q + i)], S[2 * (q + i) + 1]);
      }
      if (c + 1 < n) arrive(ready, 32 * (M + H));
      done(c);
    }
    if (me.mine) write_state(a.state_out + me.bh * a.dk * a.dv, x * kBlocks * 16, a.dk, a.dv, col, lane, S);
    return;
  }

  // of four, those with many of the triangle's blocks run beside chain warps with few
  const int ltid = tid - 32 * W * M, z = me.role - M, zg = H == 4 ? 3 - z : z;
  const auto request = [&](int c) {
    if (lane == 0 && ask)
      request_stage<NK, false, W, M, H>(sm + (c & 1) * L::stage, bars + (c & 1), a, maps, me.bh * a.n + c,
                                        me.tok + c * kC, h, me.col0, a.by_v, &maps.v, ltid >> 5);
    __syncwarp();
  };
  const auto ask_m = [&](int c) { if (ask && !a.drop) request_m(sm + L::Mq, bars + 2, a, me.bh * a.n + c); };
  if (tid >= kOwn) {
    for (int c = 0; c <= n; ++c) {
      if (c > 0 && together) __syncthreads();
      if (c > 1) wait_done(c - 2);
      if (lane == 0 && c != 1 && n > 0) ask_m(c == 0 ? 0 : c - 1);  // of chunk 0 at once
      if (c < n) request(c);
      if (c > 0 && len - (c - 1) * kC < kC) __syncthreads();
    }
    return;
  }

  const auto copy = [&](int c) {
    copy_stage<NK, false, W, M, H>(sm + (c & 1) * L::stage, a, me.tok + c * kC, h, me.col0, min(len - c * kC, kC), a.v,
                                   a.ld_v, a.by_v, ltid);
  };
  if (n > 0) {
    if (kAskers<W> > 1) {
      request(0);
      if (ltid == 0) ask_m(0);
    }
    if (together) copy(0);
  }
  for (int c = 0; c < n; ++c) {
    unsigned char *st = sm + (c & 1) * L::stage;
    if (together) {
      cp_async_wait<0>();
      __syncthreads();
      if (c + 1 < n) copy(c + 1);
    }
    wait_copies(bars + (c & 1), (c >> 1) & 1, limit, a);
    if (len - c * kC < kC) {
      clear_stage<NK, false, W, M, H>(st, a, len - c * kC, a.by_v, ltid);
      __syncthreads();
    }
    if (me.mine) meet(ready, 32 * (M + H));
    if (kAskers<W> > 1) {
      if (c > 0) {
        wait_done(c - 1);
        if (ltid == 0) ask_m(c);
      }
      if (c + 1 < n) request(c + 1);
    }
    if (!me.mine) {
      done(c);
      continue;
    }
    const float4 *hU = place(c);
    const auto get_u = [&](int ks, uint32_t(&us)[3][4]) {
      float u[2][4];
      get(hU + ks * 64, lane, u);
      a_split<3>(u[0], u[1], us);
    };
    const auto done_u = [&] {  // this warp has read U
      if (L::places > 1) return;
      __syncwarp();
      if (lane == 0) umma::mbar_arrive(smem_u32(read + w));
    };
    const uint32_t uQ = smem_u32(st + L::Q), uM = smem_u32(sm + L::Mq);
    const float *gam = reinterpret_cast<const float *>(st + L::sc);
    float Y[8 / H][4], l[8 / H][4];  // the own groups of tokens; small products apart
    clear(Y);
    clear(l);
    {  // Y^T = gam S^T Q^T
#pragma unroll(2 * H)
      for (int ks = 0; ks < NK; ++ks) {
        uint32_t s[3][4], r[4 / H][4];
        get_parts(hS + ks * 96, lane, s);
#pragma unroll
        for (int i = 0; i < 4 / H; ++i) b_rows(uQ, 16 * group_of<H>(zg, i), 16 * ks, lane, r[i]);
#pragma unroll
        for (int p = 0; p < 3; ++p)
#pragma unroll
          for (int i = 0; i < 4 / H; ++i) {
            float(&to)[8 / H][4] = p == 0 ? Y : l;
            fma16816(to[2 * i], s[p], r[i][0], r[i][1]);
            fma16816(to[2 * i + 1], s[p], r[i][2], r[i][3]);
          }
      }
      add(Y, l);
      clear(l);
      scale_groups<H>(Y, zg, gam, t);
    }
    wait_copies(bars + 2, c & 1, limit, a);
    if constexpr (H == 4) {  // += U^T M^T, M's fragments read before U is there
      uint32_t r[4][3][4], us[4][3][4];
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
        if (ks <= zg)
#pragma unroll
          for (int p = 0; p < 3; ++p) tri_rows(uM + p * kTri, zg, ks, lane, r[ks][p]);
      meet(all, 32 * (M + H));
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
        if (ks <= zg) get_u(ks, us[ks]);
      done_u();
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
        if (ks <= zg) products(Y, l, 0, us[ks], r[ks]);
      add(Y, l);
    } else {
      meet(all, 32 * (M + H));
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        uint32_t us[3][4];
        get_u(ks, us);
        if (ks == 3) done_u();
#pragma unroll
        for (int i = 0; i < 4 / H; ++i) {
          const int n = group_of<H>(zg, i);
          if (n < ks) continue;
          uint32_t r[3][4];
#pragma unroll
          for (int p = 0; p < 3; ++p) tri_rows(uM + p * kTri, n, ks, lane, r[p]);
          products(Y, l, i, us, r);
        }
      }
      add(Y, l);
    }
    done(c);
    // y, rounded once: pairs of tokens turned into pairs of columns
    uint32_t v[8 / H][2];
#pragma unroll
    for (int i = 0; i < 8 / H; ++i)
#pragma unroll
      for (int x = 0; x < 2; ++x) v[i][x] = transpose8(pack2(Y[i][2 * x], Y[i][2 * x + 1]));
    uint16_t *yc = a.y + (me.tok * a.H + h) * a.dv + col + 2 * t;
    const int left = a.dv - col - 2 * t;
    const int64_t ld_y = static_cast<int64_t>(a.H) * a.dv;
#pragma unroll
    for (int nt = 0; nt < 8 / H; ++nt) {
      const int i = c * kC + 8 * tile_of<H>(zg, nt) + g;
      if (i >= len) continue;
      uint16_t *row = yc + i * ld_y;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (a.pair_y) {
          if (8 * x < left) *reinterpret_cast<uint32_t *>(row + 8 * x) = v[nt][x];
        } else {
          if (8 * x < left) row[8 * x] = static_cast<uint16_t>(v[nt][x]);
          if (8 * x + 1 < left) row[8 * x + 1] = static_cast<uint16_t>(v[nt][x] >> 16);
        }
      }
    }
  }
}

template <int NK, int W, int M, int H>
__global__ void __launch_bounds__(kChainThreads<W, M, H>, 1) gdn_chain_back(const Gdn a,
    const __grid_constant__ Maps maps) {
  using L = Chain<NK, true, W, M, H>;
  constexpr int NT = 2 * NK, kOwn = 32 * W * (M + H);
  constexpr int kBlocks = NK / M, X = kBlocks < 2 ? 1 : 2, XH = NK / H < 2 ? 1 : 2;
  extern __shared__ __align__(1024) unsigned char sm[];
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::bars);  // two stages there, M there, two stages free
  if (threadIdx.x == 0) {
    umma::mbar_init(smem_u32(bars), kAskers<W>);
    umma::mbar_init(smem_u32(bars + 1), kAskers<W>);
    umma::mbar_init(smem_u32(bars + 2), 1);
    umma::mbar_init(smem_u32(bars + 3), W * (M + H));
    umma::mbar_init(smem_u32(bars + 4), W * (M + H));
    umma::fence_mbar_init();
  }
  before_reading();
  const Place<W> me(a);
  const int tid = me.tid, w = me.w, lane = me.lane, t = lane & 3, n = me.n, len = me.len, col = me.col, h = me.h;
  const int tiles = (a.dv + 15) >> 4;
  const int64_t ld_y = static_cast<int64_t>(a.H) * a.dv;
  uint4 *hG = reinterpret_cast<uint4 *>(sm + L::state) + w * NK * 96,
      *hP = reinterpret_cast<uint4 *>(sm + L::parts) + w * 4 * 96;
  float4 *hX = M == 4 ? reinterpret_cast<float4 *>(sm + L::sums) + w * 32 * 32
                      : reinterpret_cast<float4 *>(hP);  // partial sums, before the parts
  float4 *hZ = reinterpret_cast<float4 *>(sm + L::tokens) + w * 8 * 32;  // dY^T M, then dZ^T
  if (tid == 0 && a.err && a.lens && a.lens[me.b] != len) atomicOr(a.err, SDM_DEVERR_INDEX_RANGE);
  __syncthreads();
  uint32_t limit = tid < kOwn ? kWaitLimit : 4 * kWaitLimit;  // a warp that only asks for copies outwaits the others
  const int pair = 1 + w, all = 1 + W + w, read = 1 + 2 * W + w, helpers = 1 + 3 * W;
  const bool together = a.by_qk != 16 || a.by_dy != 16;
  const auto done = [&](int it) {
    __syncwarp();
    if (lane == 0) umma::mbar_arrive(smem_u32(bars + 3 + (it & 1)));
  };
  bool ask = true;
  const auto wait_done = [&](int it) { ask = ask && wait_copies(bars + 3 + (it & 1), (it >> 1) & 1, limit, a); };

  if (me.role < M) {
    const int x = me.role;
    uint4 *own = hG + x * kBlocks * 96;
    float4 *kept = reinterpret_cast<float4 *>(a.g) + (me.bh * (a.n + 1) * tiles + (col >> 4)) * (NT * 32) +
        x * kBlocks * 64;
    const int64_t step = static_cast<int64_t>(tiles) * (NT * 32);
#pragma unroll 1
    for (int ks = 0; ks < kBlocks; ++ks) {
      float y[2][4];
      read_state(a.state_in ? a.state_in + me.bh * a.dk * a.dv : nullptr, 16 * (x * kBlocks + ks), a.dk, a.dv, col,
                 lane, y);
      put_parts(own + ks * 96, lane, y[0], y[1]);
      if (me.mine) put(kept + n * step + ks * 64, lane, y);
      // without a token its bits go on as they are: the parts do not hold infinities
      if (n == 0) write_state(a.state_out + me.bh * a.dk * a.dv, 16 * (x * kBlocks + ks), a.dk, a.dv, col, lane, y);
    }
    for (int c = n - 1; c >= 0; --c) {
      const int it = n - 1 - c;
      if (together) __syncthreads();
      wait_copies(bars + (it & 1), (it >> 1) & 1, limit, a);
      if (len - c * kC < kC) __syncthreads();  // the helping warps clear rows
      if (!me.mine) {
        done(it);
        continue;
      }
      unsigned char *st = sm + (it & 1) * L::stage;
      const uint32_t uK = smem_u32(st + L::K);
      const float *gam = reinterpret_cast<const float *>(st + L::sc), *tail = gam + kC, *beta = tail + kC;
      // dU^T = tail G^T K^T + dY^T M
      float U[8 / M][4], Z[8 / M][4];
      {
        float d[8][4];
        state_product<kBlocks, W < 4 ? kBlocks : 1>(own, uK, x * kBlocks * 16, lane, d);
        if (M == 2) meet(pair, 32 * M);  // the parts, in whose place the sums go, have been read
        give_sums<M>(hX, x, lane, d, U);
      }
      meet(all, 32 * (M + H));  // dY^T M is there
      // G has been read.  Told only behind the meeting: a helping warp meets at `all` again once it is past `read`,
      // so every main warp has to have left that barrier's phase by then, or the helper would be counted in its place
      arrive(read, 32 * (M + H));
      take_sums<M>(hX, x, lane, U);
      scale_groups<M>(U, x, tail, t);
      add_tiles<M>(hZ, x, lane, U);
      scale_groups<M>(U, x, beta, t);
      if (M == 2) meet(pair, 32 * M);  // the partial sums, which lie in the parts' place, have been read
      put_groups<M>(hP, x, lane, U);
      meet(pair, 32 * M);
      triangle_product<true, M>(hP, smem_u32(st + L::T), x, lane, Z);  // dZ^T
      put_tiles<M>(hZ, x, lane, Z);
      meet(all, 32 * (M + H));  // dZ is there, dU has been read, G = gam_C G + Q^T (gam dY)
      // G^T -= (gam dZ)^T K
      scale_groups<M>(Z, x, gam, t);
      put_groups<M>(hP, x, lane, Z);
      meet(pair, 32 * M);
      uint32_t zt[4][3][4];
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) get_parts(hP + ks * 96, lane, zt[ks]);
      float4 *to = kept + c * step;
#pragma unroll 1
      for (int q = 0; q < kBlocks; q += X) {
        float acc[2 * X][4], y[2 * X][4];
        block_product<X>(uK, x * kBlocks + q, zt, lane, acc);
        update_blocks<X>(own, q, lane, 1.f, -1.f, acc, y);
        put(to + q * 64, lane, y);
      }
      done(it);
    }
    if (me.mine && n > 0)
#pragma unroll 1
      for (int ks = 0; ks < kBlocks; ++ks) {
        uint32_t s[3][4];
        float y[2][4];
        get_parts(own + ks * 96, lane, s);
        join(s, y[0], y[1]);
        write_state(a.state_out + me.bh * a.dk * a.dv, 16 * (x * kBlocks + ks), a.dk, a.dv, col, lane, y);
      }
    return;
  }

  const int ltid = tid - 32 * W * M, z = me.role - M, zg = H == 4 ? 3 - z : z;
  const int vc = (me.col0 & 63) + 16 * w;  // vc: the tile's columns in the value columns' panel
  const auto request = [&](int c) {
    const int s = (n - 1 - c) & 1;
    if (lane == 0 && ask)
      request_stage<NK, true, W, M, H>(sm + s * L::stage, bars + s, a, maps, me.bh * a.n + c, me.tok + c * kC, h,
                                       me.col0, a.by_dy, &maps.dy, ltid >> 5);
    __syncwarp();
  };
  if (tid >= kOwn) {
    for (int it = 0; it <= n; ++it) {
      const int c = n - 1 - it;
      if (it > 0 && together) __syncthreads();
      if (it > 1) wait_done(it - 2);
      if (it < n) request(c);
      if (it > 0 && len - (c + 1) * kC < kC) __syncthreads();
    }
    return;
  }

  const auto copy = [&](int c) {
    copy_stage<NK, true, W, M, H>(sm + ((n - 1 - c) & 1) * L::stage, a, me.tok + c * kC, h, me.col0,
                                  min(len - c * kC, kC), a.dy, ld_y, a.by_dy, ltid);
  };
  const auto ask_m = [&](int c) {
    if (ltid == 0 && !a.drop) request_m(sm + L::Mq, bars + 2, a, me.bh * a.n + c);
  };
  if (n > 0) {
    if (kAskers<W> > 1) request(n - 1);
    ask_m(n - 1);
    if (together) copy(n - 1);
  }
  for (int c = n - 1; c >= 0; --c) {
    const int it = n - 1 - c;
    const int64_t u = me.bh * a.n + c;
    unsigned char *st = sm + (it & 1) * L::stage;
    if (together) {
      cp_async_wait<0>();
      __syncthreads();
      if (c > 0) copy(c - 1);
    }
    wait_copies(bars + (it & 1), (it >> 1) & 1, limit, a);
    wait_copies(bars + 2, it & 1, limit, a);
    if (len - c * kC < kC) {
      clear_stage<NK, true, W, M, H>(st, a, len - c * kC, a.by_dy, ltid);
      __syncthreads();
    }
    const uint32_t uQ = smem_u32(st + L::Q), uM = smem_u32(sm + L::Mq), uY = smem_u32(st + L::V);
    const float *gam = reinterpret_cast<const float *>(st + L::sc);
    uint32_t y[4][1][4];
    if (me.mine) {
      float R[8 / H][4], l[8 / H][4];  // the own groups of tokens
      clear(R);
      clear(l);
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        a_cols(uY, vc, 16 * ks, lane, y[ks][0]);
#pragma unroll
        for (int i = 0; i < 4 / H; ++i) {
          const int n = group_of<H>(zg, i);
          if (n > ks) continue;
          uint32_t r[3][4];
#pragma unroll
          for (int p = 0; p < 3; ++p) tri_cols(uM + p * kTri, n, ks, lane, r[p]);
          products(R, l, i, y[ks], r);
        }
      }
      add(R, l);
      put_tiles<H>(hZ, zg, lane, R);
    }
    const auto next = [&] {  // the next chunk's copies, once the stage is free
      if (kAskers<W> == 1 || c == 0) return;
      if (it > 0) wait_done(it - 1);
      request(c - 1);
    };
    if (me.mine) arrive(all, 32 * (M + H));
    meet(helpers, 32 * W * H);  // M has been read
    if (c > 0) ask_m(c - 1);
    if (!me.mine) {
      next();
      done(it);
      continue;
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
    next();
    meet(read, 32 * (M + H));
    const float end = gam[kC - 1];
#pragma unroll 1
    for (int q = z * (NK / H); q < (z + 1) * (NK / H); q += XH) {
      float acc[2 * XH][4], x[2 * XH][4];
      block_product<XH>(uQ, q, d3, lane, acc);
      update_blocks<XH>(hG, q, lane, end, 1.f, acc, x);
    }
    done(it);
    meet(all, 32 * (M + H));
    float4 *to = reinterpret_cast<float4 *>(a.dz) + (u * tiles + (col >> 4)) * 256 + lane;
#pragma unroll
    for (int i = 0; i < 8 / H; ++i) to[tile_of<H>(zg, i) * 32] = hZ[tile_of<H>(zg, i) * 32 + lane];
  }
}

// ---------------------------------------------------------------------------
// gdn_grad: the gradients of one chunk of one head, on the tcgen05 tensor cores. Transposed, every sum over
// value columns has the key channels or two times the tokens as its M = 128 and the tokens as N:
//   [dQ | dKa]^T [128 x 128] = S [dY | dZ]^T        dK^T [128 x 64] = G U^T
//   [X; N]       [128 x 64]  = [dY; dZ] U^T
// and then, with X and N times their decays,
//   [QK; KK] [128 x 64] = [Q; K] K^T,   dQ2^T = K^T X^T,   dK2^T = Q^T X + K^T (N^T + N),
//   dQ = gam dQ + dQ2,   dK = (tail dK - gam dKa) + dK2,
// QK and KK for the decays' gradient and, like dQ2, in X's and N's place; dK2 in dKa's.  The tensor cores cut a
// sum off at each product, towards 0, so a sum with fewer products behind it is nearer: with dQ2 and dK2 on top of
// dQ and dK those were 5.9e-7 and 8.5e-7 off.
// The value columns come 32 at a time, as the chains left them, read ahead by a piece: S by bulk copies, G and the
// rest 16 bytes a lane (a copy of G too would not leave room for a second CTA an SM; states through registers
// alone, whose loads wait for one another at the door, took 404 us where copies took 360).  They are split into
// bf16 parts and stored as the 8 x 8 cores of the operands, where a warp's store is 128 bytes in a row.  K and Q
// come last, in the states' place, while X and N are converted.  The operands of the sums over value columns have
// their rows of 8 along M or N (MN-major); X, N, K and Q serve both ways as they lie.
// With dk <= 64 the products' upper 64 channels are whatever lies behind S and G; rows of a product do not mix,
// and those are not read.  A CTA needs half of an SM's shared memory, registers and tensor memory, so that one's
// conversions run beside the other's products.  A chunk's 240 KB are read and its 48 KB written at 2.8 TB/s; what
// bounds it is the latency of each piece's loads, conversions and products in turn (30,000 cycles a chunk and SM,
// of them 12,100 of issue and about 7,000 of products).  On mma.sync, with accumulators in registers and one CTA
// an SM, it took 705 us, where this form, with two parts behind dk and the decays' gradient by a difference, took 360.
// ---------------------------------------------------------------------------
constexpr int kGradThreads = 256;

struct Grad {
  // a core row of 8 value columns: 16 cores where M or N is 128, 8 where it is 64
  static constexpr int YZ = 0, Z1 = YZ + 8192 /* zeros | the second part of dZ */, Z2 = Z1 + 8192, U = Z2 + 8192,
                       S = U + 3 * 4096, G = S + 3 * 8192, stage = G + 3 * 8192 /* S, a piece ahead */,
                       sc = stage + 16384, rows = sc + kScal * 4 /* [2][64]: dZ . E */,
                       into = rows + 2 * kC * 4 /* [4][64]: gam (q . S dY - k . S dZ) */,
                       out = into + 4 * kC * 4 /* [4][64]: tail k . G U */,
                       inner = out + 4 * kC * 4 /* [8][64]: pairs of tokens */, red = inner + 8 * kC * 4,
                       bars = red + 32, size = bars + 32;
  // once the value columns are done
  static constexpr int X = 0, N = X + 3 * 8192, Q = N + 3 * 8192, K = Q + 16384;
  static constexpr uint32_t dQ = 0, dKa = 64, dK = 128, XN = 192, columns = 256;  // tensor memory
  static constexpr uint32_t QKK = XN, dQ2 = XN, dK2 = dKa;
  static_assert(K + 16384 <= stage, "");
};
static_assert(2 * (Grad::size + 1024) <= 228 * 1024, "two CTAs an SM");

// 64 rows of `width` bf16 as 8 x 8 cores [row / 8][column / 8], zeros from row `live` on
__device__ __forceinline__ void load_cores(unsigned char *to, const uint16_t *src, int64_t ld, int live, int width,
                                           int by, int tid) {
#pragma unroll 4
  for (int i = 0; i < kC * 16 / kGradThreads; ++i) {
    // a warp: 8 rows, 4 pieces of 16 bytes of each
    const int id = tid + i * kGradThreads, r = ((id >> 7) << 3) | (id & 7), p = (id >> 3) & 15, c = p * 8;
    unsigned char *dst = to + (r >> 3) * 2048 + p * 128 + (r & 7) * 16;
    const uint16_t *s = src + r * ld + c;
    if (by == 16) {
      const bool ok = r < live && c < width;
      copy_async<16>(smem_u32(dst), ok ? s : src, ok);
    } else if (by == 8) {
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        const bool ok = r < live && c + e < width;
        copy_async<8>(smem_u32(dst) + 2 * e, ok ? s + e : src, ok);
      }
    } else {
      uint32_t w[4] = {0, 0, 0, 0};
      if (r < live)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c + e < width) w[e >> 1] |= static_cast<uint32_t>(s[e]) << (16 * (e & 1));
      *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// two neighbouring bf16 of a row, of which `left` exist
__device__ __forceinline__ uint32_t load_pair(const uint16_t *p, int left, bool pairs) {
  if (left <= 0) return 0;
  if (pairs) return *reinterpret_cast<const uint32_t *>(p);
  return p[0] | (left > 1 ? static_cast<uint32_t>(p[1]) << 16 : 0);
}

// lanes hold v[16]; the sum over the lanes of v[lane % 16]
__device__ __forceinline__ float sum_lanes(float (&v)[16], int lane) {
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float send = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
      v[i] = keep + __shfl_xor_sync(kFull, send, o);
    }
  }
  return v[0] + __shfl_xor_sync(kFull, v[0], 16);
}

template <int NK>
__global__ void __launch_bounds__(kGradThreads, 2) gdn_grad(const Gdn a) {
  using L = Grad;
  using namespace umma;
  constexpr int NT = 2 * NK, NW = NT / 4;  // NW: 8-channel groups of the states a warp
  extern __shared__ __align__(1024) unsigned char sm[];
  const int tid = threadIdx.x, w = tid >> 5, quarter = w & 3, upper = w >> 2, lane = tid & 31, g = lane >> 2,
      t = lane & 3;
  const unsigned heads = static_cast<unsigned>(a.B) * a.H;
  // chunk by chunk: what the backward chains wrote last, and is still in L2, comes first
  const int c = static_cast<int>(blockIdx.x / heads), bh32 = static_cast<int>(blockIdx.x % heads);
  const int b = bh32 / a.H, h = bh32 - b * a.H;
  const int64_t bh = bh32, u = bh * a.n + c;
  before_reading();
  const int live = min(length_of(a, b) - c * kC, kC);
  if (live <= 0) return;
  const int64_t tok = static_cast<int64_t>(b) * a.T + c * kC, ld_y = static_cast<int64_t>(a.H) * a.dv;
  const int hk = h / (a.H / a.Hk), tiles = (a.dv + 15) >> 4;
  float *sc = reinterpret_cast<float *>(sm + L::sc);
  float *gam = sc, *tail = sc + kC, *beta = sc + 2 * kC, *lh = sc + 3 * kC, *ll = sc + 4 * kC, *sg = sc + 5 * kC;
  float *rows = reinterpret_cast<float *>(sm + L::rows), *into = reinterpret_cast<float *>(sm + L::into),
        *out = reinterpret_cast<float *>(sm + L::out), *inner = reinterpret_cast<float *>(sm + L::inner),
        *red = reinterpret_cast<float *>(sm + L::red);
  uint64_t *bar = reinterpret_cast<uint64_t *>(sm + L::bars);
  uint32_t *holder = reinterpret_cast<uint32_t *>(bar + 2);
  const uint32_t mb = smem_u32(bar), full = smem_u32(bar + 1), base = smem_u32(sm);

  // Two tiles of S at the chunk's start by bulk copies, a piece ahead; the rest of a piece into registers: of tile
  // `upper` of the two, key channels 8 NW quarter .. and tokens 16 quarter .. + 15
  const auto ask_states = [&](int c0) {
    const int ct = c0 >> 4;
    const uint32_t bytes = min(2, tiles - ct) * NT * 512;
    mbar_expect_tx(full, bytes);
    bulk_g2s(base + L::stage, a.s + (u * tiles + ct) * (NT * 128), bytes, full);
  };
  float4 f1[NW];
  float E[2][4], Z[2][4];
  uint32_t yv[2][2];  // dy [n-tile][columns 0..7, 8..15]: a row's pair a lane
  const auto read_end = [&](int c0) {  // G at the chunk's end
    const int ct = (c0 >> 4) + upper;
    const float4 *G = reinterpret_cast<const float4 *>(a.g) +
        (((bh * (a.n + 1) + c + 1) * tiles + ct) * NT + quarter * NW) * 32 + lane;
#pragma unroll
    for (int x = 0; x < NW; ++x) f1[x] = ct < tiles ? G[x * 32] : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  const auto read_tokens = [&](int c0) {
    const int ct = (c0 >> 4) + upper;
    const bool on = ct < tiles;
    const int64_t at = ((u * tiles + ct) * 8 + 2 * quarter) * 32;
    if (on) {
      get(reinterpret_cast<const float4 *>(a.e) + at, lane, E);
      get(reinterpret_cast<const float4 *>(a.dz) + at, lane, Z);
    } else {
      clear(E);
      clear(Z);
    }
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = 16 * quarter + 8 * x + g, cc = 16 * ct + 8 * e + 2 * t, left = i < live ? a.dv - cc : 0;
        yv[x][e] = load_pair(a.dy + (tok + i) * ld_y + h * a.dv + cc, left, a.by_dy >= 4);
      }
  };
  if (tid == 0) {
    mbar_init(mb, 1);
    mbar_init(full, 1);
    fence_mbar_init();
    ask_states(0);
  }
  read_end(0);
  if (tid < kScal / 4) copy_async<16>(smem_u32(sc) + tid * 16, a.scal + u * kScal + tid * 4, true);
  cp_async_commit();
  read_tokens(0);

  if (w == 0) tmem_alloc(smem_u32(holder), L::columns);
  // the halves of zeros beside dZ's second and third part
  {
    const int i = tid >> 6, o = tid & 63;
    *reinterpret_cast<uint4 *>(sm + L::Z1 + i * 2048 + o * 16) = make_uint4(0, 0, 0, 0);
    *reinterpret_cast<uint4 *>(sm + L::Z2 + i * 2048 + o * 16) = make_uint4(0, 0, 0, 0);
  }
  cp_async_wait<0>();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *holder;
  const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
  bool ok = true, there = true;
  uint32_t phase = 0;
  // every thread waits for the products asked for; then the CTA agrees
  const auto products_done = [&]() {
    ok = mbar_wait(mb, phase & 1, kWaitLimit) && there;
    ++phase;
    tc_fence_before();
    ok = __syncthreads_and(ok) != 0;
    tc_fence_after();
    return ok;
  };
  // A and B with rows of 8 along M and N; N = 64 and 128
  const uint32_t mn = (1u << 15) | (1u << 16);
  const uint32_t id64 = idesc_bf16_f32(128, 64) | mn, id128 = idesc_bf16_f32(128, 128) | mn;

  float anchor = 0.f, ez[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
  for (int c0 = 0; c0 < a.dv; c0 += 32) {
    if (c0 && !products_done()) break;  // the piece before has been read
    // ---- the states
    there = mbar_wait(full, (c0 >> 5) & 1, kWaitLimit) && there;
#pragma unroll
    for (int x = 0; x < NW; ++x) {
      float4 fs = make_float4(0.f, 0.f, 0.f, 0.f);
      if ((c0 >> 4) + upper < tiles)
        fs = reinterpret_cast<const float4 *>(sm + L::stage)[(upper * NT + quarter * NW + x) * 32 + lane];
      anchor += (fs.x * f1[x].x + fs.y * f1[x].y) + (fs.z * f1[x].z + fs.w * f1[x].w);
      uint32_t p0[3], p1[3], q0[3], q1[3];
      split<3>(fs.x, fs.y, p0);
      split<3>(fs.z, fs.w, p1);
      split<3>(f1[x].x, f1[x].y, q0);
      split<3>(f1[x].z, f1[x].w, q1);
      unsigned char *o = sm + upper * 4096 + (quarter * NW + x) * 128 + lane * 4;
#pragma unroll
      for (int p = 0; p < 3; ++p) {
        *reinterpret_cast<uint32_t *>(o + L::S + p * 8192) = p0[p];
        *reinterpret_cast<uint32_t *>(o + L::S + p * 8192 + 2048) = p1[p];
        *reinterpret_cast<uint32_t *>(o + L::G + p * 8192) = q0[p];
        *reinterpret_cast<uint32_t *>(o + L::G + p * 8192 + 2048) = q1[p];
      }
    }
    if (c0 + 32 < a.dv) {
      read_end(c0 + 32);
      if (w == 0) {  // once every warp has read the stage
        asm volatile("bar.sync 1, 256;\n" ::: "memory");
        if (lane == 0) ask_states(c0 + 32);
        __syncwarp();
      } else {
        asm volatile("bar.arrive 1, 256;\n" ::: "memory");
      }
    }
    // ---- U, dZ, dy; dv; the sums over value columns
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int nt = 2 * quarter + x;
      const float2 be = *reinterpret_cast<const float2 *>(beta + 8 * nt + 2 * t);
#pragma unroll
      for (int e = 0; e < 2; ++e) {  // columns 0..7 and 8..15 of the tile
        const float e0 = E[x][2 * e], e1 = E[x][2 * e + 1], z0 = Z[x][2 * e], z1 = Z[x][2 * e + 1];
        uint32_t su[3], sz[3];
        split<3>(be.x * e0, be.y * e1, su);
        split<3>(z0, z1, sz);
        const uint32_t y = transpose8(yv[x][e]);
        ez[x][0] = fmaf(e0, z0, ez[x][0]);
        ez[x][1] = fmaf(e1, z1, ez[x][1]);
        const int row = 2 * upper + e;  // of the piece's four core rows
        unsigned char *o = sm + nt * 128 + lane * 4;
        *reinterpret_cast<uint32_t *>(o + L::YZ + row * 2048) = y;
        *reinterpret_cast<uint32_t *>(o + L::YZ + row * 2048 + 1024) = sz[0];
        *reinterpret_cast<uint32_t *>(o + L::Z1 + row * 2048 + 1024) = sz[1];
        *reinterpret_cast<uint32_t *>(o + L::Z2 + row * 2048 + 1024) = sz[2];
#pragma unroll
        for (int p = 0; p < 3; ++p) *reinterpret_cast<uint32_t *>(o + L::U + p * 4096 + row * 1024) = su[p];
        // dv is dZ rounded once, which is its first part
        const uint32_t z = transpose8(sz[0]);
        const int i = 8 * nt + g, cc = c0 + 16 * upper + 8 * e + 2 * t;
        if (i < live) {
          uint16_t *to = a.odv + (tok + i) * a.ld_dv + h * a.dv + cc;
          if (a.pair_y) {
            if (cc < a.dv) *reinterpret_cast<uint32_t *>(to) = z;
          } else {
            if (cc < a.dv) to[0] = static_cast<uint16_t>(z);
            if (cc + 1 < a.dv) to[1] = static_cast<uint16_t>(z >> 16);
          }
        }
      }
    }
    if (c0 + 32 < a.dv) read_tokens(c0 + 32);
    fence_async_smem();
    __syncthreads();
    if (tid == 0) {
      const bool more = c0 > 0;
      const uint64_t yz = smem_desc(base + L::YZ, 2048, 128), z1 = smem_desc(base + L::Z1, 2048, 128),
                     z2 = smem_desc(base + L::Z2, 2048, 128);
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const bool acc = more || ks > 0;
        const uint64_t s0 = smem_desc(base + L::S + ks * 4096, 2048, 128), s1 = s0 + 512, s2 = s0 + 1024;
        const uint64_t g0 = smem_desc(base + L::G + ks * 4096, 2048, 128), g1 = g0 + 512, g2 = g0 + 1024;
        const uint64_t u0 = smem_desc(base + L::U + ks * 2048, 1024, 128), u1 = u0 + 256, u2 = u0 + 512;
        // b1, b2: dZ's second and third part alone
        const uint64_t b = yz + 256 * ks, l1 = z1 + 256 * ks, l2 = z2 + 256 * ks, b1 = l1 + 64, b2 = l2 + 64;
        mma_bf16(tmem + L::dQ, s0, b, id128, acc);
        mma_bf16(tmem + L::dQ, s1, b, id128, true);
        mma_bf16(tmem + L::dQ, s2, b, id128, true);
        mma_bf16(tmem + L::dKa, s0, b1, id64, true);
        mma_bf16(tmem + L::dKa, s1, b1, id64, true);
        mma_bf16(tmem + L::dKa, s0, b2, id64, true);
        mma_bf16(tmem + L::dK, g0, u0, id64, acc);
        mma_bf16(tmem + L::dK, g0, u1, id64, true);
        mma_bf16(tmem + L::dK, g1, u0, id64, true);
        mma_bf16(tmem + L::dK, g1, u1, id64, true);
        mma_bf16(tmem + L::dK, g0, u2, id64, true);
        mma_bf16(tmem + L::dK, g2, u0, id64, true);
        mma_bf16(tmem + L::XN, b, u0, id64, acc);
        mma_bf16(tmem + L::XN, b, u1, id64, true);
        mma_bf16(tmem + L::XN, b, u2, id64, true);
        mma_bf16(tmem + L::XN, l1, u0, id64, true);
        mma_bf16(tmem + L::XN, l1, u1, id64, true);
        mma_bf16(tmem + L::XN, l2, u0, id64, true);
      }
      mma_commit(mb);
    }
  }
  // sums over the columns of 16 tokens, and over the state
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) ez[x][e] += __shfl_xor_sync(kFull, ez[x][e], o);
      if (g == 0) rows[upper * kC + 16 * quarter + 8 * x + 2 * t + e] = ez[x][e];
    }
#pragma unroll
  for (int o = 16; o; o >>= 1) anchor += __shfl_xor_sync(kFull, anchor, o);
  if (lane == 0) red[w] = anchor;

  if (ok && products_done()) {
    load_cores(sm + L::K, a.k + tok * a.ld_k + hk * a.dk, a.ld_k, live, a.dk, a.by_qk, tid);
    load_cores(sm + L::Q, a.q + tok * a.ld_q + hk * a.dk, a.ld_q, live, a.dk, a.by_qk, tid);
    cp_async_commit();
    // ---- X (lanes 0..63) and N (64..127) times their decays: row i, columns 32 upper ..
    const bool is_n = quarter >= 2;
    float pair[2][16];  // they stay, for the decays' gradient
    {
      const int i = 32 * (quarter & 1) + lane;
      const Wide li{lh[i], ll[i]};
      const int si = __float_as_int(sg[i]);
      unsigned char *to = sm + (is_n ? L::N : L::X) + (i >> 3) * 1024 + (i & 7) * 16;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int j0 = 32 * upper + 16 * half;
        float(&x)[16] = pair[half];
        tmem_ld16(lanes + L::XN + j0, x);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int j = j0 + e;
          const bool on = (is_n ? j < i : j <= i) && si == __float_as_int(sg[j]);
          const float d = decay_between(li, {lh[j], ll[j]});
          x[e] = on ? (is_n ? -d : d) * x[e] : 0.f;
        }
#pragma unroll
        for (int e = 0; e < 16; e += 8) {
          uint32_t s[4][3];
#pragma unroll
          for (int p = 0; p < 4; ++p) split<3>(x[e + 2 * p], x[e + 2 * p + 1], s[p]);
          unsigned char *o = to + ((j0 + e) >> 3) * 128;
#pragma unroll
          for (int p = 0; p < 3; ++p)
            *reinterpret_cast<uint4 *>(o + p * 8192) = make_uint4(s[0][p], s[1][p], s[2][p], s[3][p]);
        }
      }
    }
    cp_async_wait<0>();
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0) {
#pragma unroll
      for (int ks = 0; ks < NK; ++ks)  // A and B with rows of 8 along their sum
        mma_bf16(tmem + L::QKK, smem_desc(base + L::Q + ks * 256, 128, 2048),
                 smem_desc(base + L::K + ks * 256, 128, 2048), idesc_bf16_f32(128, 64), ks > 0);
      mma_commit(mb);
    }
    // ---- channel 32 quarter + lane, tokens 32 upper ..: what comes from the states, its part in the decays' gradient
    const int ch = 32 * quarter + lane;
    const bool mine = ch < a.dk;
    {
      const unsigned char *sk = sm + L::K + (ch >> 3) * 128 + (ch & 7) * 2;
      const auto key = [&](int i) {
        return bf16_to_f32(*reinterpret_cast<const uint16_t *>(sk + (i >> 3) * 2048 + (i & 7) * 16));
      };
      const auto query = [&](int i) {
        return bf16_to_f32(*reinterpret_cast<const uint16_t *>(sk + (L::Q - L::K) + (i >> 3) * 2048 + (i & 7) * 16));
      };
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        const int i0 = 32 * upper + 16 * half;
        const float *gi = gam + i0, *ti = tail + i0;
        float x[16], y[16], f[16];
        tmem_ld16(lanes + L::dQ + i0, x);
        tmem_ld16(lanes + L::dKa + i0, y);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          y[e] *= gi[e];
          f[e] = mine ? query(i0 + e) * (gi[e] * x[e]) - key(i0 + e) * y[e] : 0.f;
        }
        const float a0 = sum_lanes(f, lane);
        if (lane < 16) into[quarter * kC + i0 + lane] = a0;
        tmem_ld16(lanes + L::dK + i0, x);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float d = ti[e] * x[e];
          f[e] = mine ? key(i0 + e) * d : 0.f;
          x[e] = d - y[e];
        }
        tmem_st16(lanes + L::dK + i0, x);
        const float b0 = sum_lanes(f, lane);
        if (lane < 16) out[quarter * kC + i0 + lane] = b0;
      }
      tmem_st_wait();
    }
    if (products_done()) {
      const uint32_t idk = idesc_bf16_f32(128, 64) | (1u << 15);  // B with rows of 8 along its sum
      if (tid == 0) {
#pragma unroll
        for (int p = 2; p >= 0; --p)
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            const uint64_t k = smem_desc(base + L::K + ks * 4096, 2048, 128);
            const uint64_t q = smem_desc(base + L::Q + ks * 4096, 2048, 128);
            const uint64_t xc = smem_desc(base + L::X + ks * 2048, 1024, 128);
            const uint64_t nr = smem_desc(base + L::N + ks * 256, 128, 1024);
            const uint64_t nc = smem_desc(base + L::N + ks * 2048, 1024, 128);
            mma_bf16(tmem + L::dK2, q, xc + 512 * p, id64, p < 2 || ks > 0);
            mma_bf16(tmem + L::dK2, k, nr + 512 * p, idk, true);
            mma_bf16(tmem + L::dK2, k, nc + 512 * p, id64, true);
          }
      }
      // ---- the pairs: of row i, the sums over j < t of its terms, which belong to the tokens t <= i
      if (upper <= (quarter & 1)) {
        const bool below = upper < (quarter & 1);  // i >= 32 > j, else i and j in the same half
        float *to = inner + w * kC;
        float sum = 0.f;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float x[16];
          tmem_ld16(lanes + L::QKK + 32 * upper + 16 * half, x);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float term = pair[half][e] * x[e];
            x[e] = below || 16 * half + e <= lane ? sum : 0.f;
            sum += term;
          }
          const float f = sum_lanes(x, lane);
          if (lane < 16) to[32 * upper + 16 * half + lane] = f;
        }
        if (below) {  // tokens t >= 32: rows from t on, all of their terms
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const float y = __shfl_down_sync(kFull, sum, o);
            if (lane + o < 32) sum += y;
          }
          to[32 + lane] = sum;
        }
      }
      tc_fence_before();
      __syncthreads();
      tc_fence_after();
      if (tid == 0) {
#pragma unroll
        for (int p = 2; p >= 0; --p)
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            mma_bf16(tmem + L::dQ2, smem_desc(base + L::K + ks * 4096, 2048, 128),
                     smem_desc(base + L::X + ks * 256, 128, 1024) + 512 * p, idk, p < 2 || ks > 0);
        mma_commit(mb);
      }
    }
    if (ok && products_done()) {
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        const int i0 = 32 * upper + 16 * half, n = mine ? live - i0 : 0;
        const float *gi = gam + i0;
        float x[16], y[16];
        tmem_ld16(lanes + L::dQ + i0, x);
        tmem_ld16(lanes + L::dQ2 + i0, y);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = fmaf(gi[e], x[e], y[e]);
        if (a.pdq) {
          float *o = a.pdq + ((tok + i0) * a.H + h) * a.dk + ch;
#pragma unroll
          for (int e = 0; e < 16; ++e, o += a.H * a.dk)
            if (e < n) *o = x[e];
        } else {
          uint16_t *o = a.odq + (tok + i0) * a.ld_dq + h * a.dk + ch;
#pragma unroll
          for (int e = 0; e < 16; ++e, o += a.ld_dq)
            if (e < n) *o = static_cast<uint16_t>(pack2(x[e], 0.f));
        }
        tmem_ld16(lanes + L::dK + i0, x);
        tmem_ld16(lanes + L::dK2 + i0, y);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] += y[e];
        if (a.pdk) {
          float *o = a.pdk + ((tok + i0) * a.H + h) * a.dk + ch;
#pragma unroll
          for (int e = 0; e < 16; ++e, o += a.H * a.dk)
            if (e < n) *o = x[e];
        } else {
          uint16_t *o = a.odk + (tok + i0) * a.ld_dk + h * a.dk + ch;
#pragma unroll
          for (int e = 0; e < 16; ++e, o += a.ld_dk)
            if (e < n) *o = static_cast<uint16_t>(pack2(x[e], 0.f));
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (!ok) {  // a wait gave up: let the products asked for end (bounded), and report
    if (tid == 0) {
      mma_commit(mb);
      report_timeout(a.err);
    }
    mbar_wait(mb, phase & 1, kWaitLimit);
    __syncthreads();
  }
  if (w == 1) tmem_dealloc(tmem, L::columns);
  if (w == 0) {  // the decays' gradient.  No sum is formed as a difference: what it leaves out may be far larger
    float x[2], y[2];  // what passes the decays up to a token from the states, and on to the state behind it
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int m = lane + 32 * i;
      x[i] = (into[m] + into[kC + m]) + (into[2 * kC + m] + into[3 * kC + m]);
      y[i] = (out[m] + out[kC + m]) + (out[2 * kC + m] + out[3 * kC + m]);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float xx = __shfl_down_sync(kFull, x[i], o), yy = __shfl_up_sync(kFull, y[i], o);
        if (lane + o < 32) x[i] += xx;  // over the tokens from this one on
        if (lane >= o) y[i] += yy;      // up to this one
      }
    }
    x[0] += __shfl_sync(kFull, x[1], 0);
    const float half = __shfl_sync(kFull, y[0], 31);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float last = __shfl_up_sync(kFull, y[i], 1);
      y[i] = (lane ? last : 0.f) + (i ? half : 0.f);  // over those before it
    }
    const float state =
        gam[kC - 1] * (((red[0] + red[1]) + (red[2] + red[3])) + ((red[4] + red[5]) + (red[6] + red[7])));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int m = lane + 32 * i;
      // of the warps that had rows 0..31 / 32..63 of X and N beside columns 0..31 (0, 2 / 1, 3) and 32..63 (- / 5, 7)
      const float *p = inner + m + (i ? 4 * kC : 0);
      const float pairs = (p[i * kC] + p[(2 + i) * kC]) + (inner[kC + m] + inner[3 * kC + m]);
      if (m < live) {
        a.dla[(tok + m) * a.H + h] = state + ((x[i] + y[i]) + pairs);
        a.dbeta[(tok + m) * a.H + h] = (rows[m] + rows[kC + m]) / beta[m];
      }
    }
  }
}

// dq and dk of key heads that several value heads share, heads in order; two channels a thread
__global__ void __launch_bounds__(256) gdn_grad_heads(const Gdn a) {
  const int group = a.H / a.Hk, half = (a.dk + 1) / 2;
  const int64_t tok = blockIdx.x;
  before_reading();
  if (static_cast<int>(tok % a.T) >= length_of(a, static_cast<int>(tok / a.T))) return;
  const bool pairs = a.pair_qk;
  for (int i = threadIdx.x; i < a.Hk * half; i += 256) {
    const int hk = i / half, ch = 2 * (i - hk * half);
    const int64_t from = (tok * a.H + static_cast<int64_t>(hk) * group) * a.dk + ch;
    const bool two = ch + 1 < a.dk;
    float2 q = make_float2(0.f, 0.f), k = q;
    for (int e = 0; e < group; ++e) {
      const float *pq = a.pdq + from + static_cast<int64_t>(e) * a.dk,
          *pk = a.pdk + from + static_cast<int64_t>(e) * a.dk;
      if (pairs) {
        const float2 x = *reinterpret_cast<const float2 *>(pq), y = *reinterpret_cast<const float2 *>(pk);
        q.x += x.x, q.y += x.y, k.x += y.x, k.y += y.y;
      } else {
        q.x += pq[0], k.x += pk[0];
        if (two) q.y += pq[1], k.y += pk[1];
      }
    }
    const uint32_t vq = pack2(q.x, q.y), vk = pack2(k.x, k.y);
    uint16_t *oq = a.odq + tok * a.ld_dq + hk * a.dk + ch, *ok = a.odk + tok * a.ld_dk + hk * a.dk + ch;
    if (pairs) {
      *reinterpret_cast<uint32_t *>(oq) = vq;
      *reinterpret_cast<uint32_t *>(ok) = vk;
    } else {
      oq[0] = static_cast<uint16_t>(vq), ok[0] = static_cast<uint16_t>(vk);
      if (two) oq[1] = static_cast<uint16_t>(vq >> 16), ok[1] = static_cast<uint16_t>(vk >> 16);
    }
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
  return B >= 0 && T >= 0 && H >= 0 && Hk >= 0 && B < 65536 && H < 65536 && T < (1 << 30) && dk >= 1 && dk <= 128 &&
         dv >= 1 && dv <= 1024 && (H == 0 || (Hk > 0 && H % Hk == 0)) &&
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
    return set_error(SDM_ERR_SHAPE, "%s: a token's row must be at most 2^27 elements from the next and hold its heads",
        what);
  if (!aligned(a.q, 2) || !aligned(a.k, 2) || !aligned(a.v, 2) || !aligned(a.la, 4) || !aligned(a.beta, 4) ||
      !aligned(a.lens, 4) || !aligned(a.err, 4) || !aligned(a.state_in, 4) || !aligned(a.state_out, 4) ||
      !aligned(saved, 16))
    return set_error(SDM_ERR_ALIGN, "%s: a pointer is not aligned", what);
  if (saved_bytes < l.saved)
    return set_error(SDM_ERR_INVALID_ARG, "%s: saved holds %zu bytes, %zu needed", what, saved_bytes, l.saved);
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
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q);
    return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<Encode>(f) : nullptr;
  }();
  if (!encode) return set_error(SDM_ERR_CUDA, "gdn_train: the driver has no cuTensorMapEncodeTiled");
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads),
      static_cast<cuuint64_t>(tokens)};
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
  if (rc == SDM_OK && a.dy && a.by_dy == 16)
    rc = make_map(&m->dy, a.dy, static_cast<int64_t>(a.H) * a.dv, tokens, a.H, a.dv);
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

// Every kernel here may be launched while the one before it in the stream still runs (its own set-up then
// overlaps that one's end) and waits for it with before_reading().
template <typename... A>
int launch(void (*kernel)(A...), const char *what, int64_t grid, int threads, int smem, cudaStream_t st, A... args) {
  cudaError_t e = cudaSuccess;
  if (smem > (48 << 10)) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return set_error(SDM_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(static_cast<unsigned>(grid));
  c.blockDim = dim3(static_cast<unsigned>(threads));
  c.dynamicSmemBytes = static_cast<size_t>(smem);
  c.stream = st;
  c.attrs = &early;
  c.numAttrs = 1;
  e = cudaLaunchKernelEx(&c, kernel, args...);
  if (e != cudaSuccess) return set_error(SDM_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  return SDM_OK;
}

// Tiles of 16 columns a CTA: one where every tile can have an SM of its own (1.9 us a chunk forward), else two
// (3.4), else four (5.4), which share an SM's tensor cores and the chunk's tiles; two turns of the SMs with half
// as many would take 3.8 and 6.7.
int chain_width(const Gdn &a, const Layout &l) {
  const int64_t all = l.tiles * a.B * a.H;
  return all <= kSms || l.tiles == 1 ? 1 : all <= 2 * kSms || l.tiles == 2 ? 2 : 4;
}

template <int NK, int W, int M, int H>
int run_chain(const Gdn &a, const Maps &maps, const Layout &l, bool back, cudaStream_t st) {
  const int64_t grid = (l.tiles + W - 1) / W * a.B * a.H;
  return back ? launch(gdn_chain_back<NK, W, M, H>, "gdn_backward", grid, kChainThreads<W, M, H>,
                       Chain<NK, true, W, M, H>::size, st, a, maps)
              : launch(gdn_chain<NK, W, M, H>, "gdn_train", grid, kChainThreads<W, M, H>,
                       Chain<NK, false, W, M, H>::size, st, a, maps);
}
template <int NK>
int run_chain(const Gdn &a, const Maps &maps, const Layout &l, bool back, cudaStream_t st) {
  const int w = chain_width(a, l);
  return w == 1 ? run_chain<NK, 1, 4, 4>(a, maps, l, back, st)
         : w == 2 ? run_chain<NK, 2, 4, 2>(a, maps, l, back, st) : run_chain<NK, 4, 2, 1>(a, maps, l, back, st);
}

template <int NK>
int run_train(const Gdn &a, const Layout &l, cudaStream_t st) {
  Maps maps{};
  int rc = make_maps(&maps, a);
  if (rc != SDM_OK) return rc;
  if (l.units > 0) {
    rc = launch(gdn_prep<NK>, "gdn_train", l.units, kPrepThreads, (2 * kC * kLd + kScal) * 4 + 16, st, a, maps);
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
  rc = launch(gdn_grad<NK>, "gdn_backward", l.units, kGradThreads, Grad::size, st, a);
  if (rc != SDM_OK || !a.pdq) return rc;
  return launch(gdn_grad_heads, "gdn_backward", static_cast<int64_t>(a.B) * a.T, 256, 0, st, a);
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
  a.drop = test_drop_signal();
  if (static_cast<int64_t>(B) * H > 0 && (!state_out || (T > 0 && !y)))
    return set_error(SDM_ERR_INVALID_ARG, "gdn_train: null pointer");
  const int rc = check_common("gdn_train", a, saved, saved_bytes, l);
  if (rc != SDM_OK) return rc;
  if (!aligned(y, 2)) return set_error(SDM_ERR_ALIGN, "gdn_train: a pointer is not aligned");
  if (B == 0 || H == 0) return SDM_OK;
  a.by_qk = std::min(row_bytes(q, ld_q, dk), row_bytes(k, ld_k, dk));
  a.by_v = row_bytes(v, ld_v, dv);
  a.pair_y = dv % 2 == 0 && aligned(y, 4);
  place_saved(a, saved, l);
  return dk <= 64 ? run_train<4>(a, l, static_cast<cudaStream_t>(stream))
                  : run_train<8>(a, l, static_cast<cudaStream_t>(stream));
}

extern "C" int gdn_backward(const float *dstate, float *dstate_out, const uint16_t *q, int64_t ld_q, const uint16_t *k,
                            int64_t ld_k, const uint16_t *v, int64_t ld_v, const float *log_alpha, const float *beta,
                            const uint8_t *reset, const int32_t *lens, const void *saved, size_t saved_bytes,
                            const uint16_t *dy, int B, int T, int Hk, int H, int dk, int dv, uint16_t *dq,
                            int64_t ld_dq, uint16_t *dk_out, int64_t ld_dk, uint16_t *dv_out, int64_t ld_dv,
                            float *dlog_alpha, float *dbeta, void *workspace, size_t workspace_bytes, int32_t *dev_err,
                            void *stream) {
  if (B < 0 || T < 0 || Hk < 0 || H < 0) return set_error(SDM_ERR_INVALID_ARG, "gdn_backward: negative size");
  if (!sizes_fit(B, T, Hk, H, dk, dv)) return set_error(SDM_ERR_SHAPE, "gdn_backward: sizes beyond the limits");
  const Layout l = layout_of(B, T, Hk, H, dk, dv);
  Gdn a{};
  a.q = q; a.k = k; a.v = v; a.dy = dy;
  a.ld_q = ld_q; a.ld_k = ld_k; a.ld_v = ld_v; a.ld_dq = ld_dq; a.ld_dk = ld_dk; a.ld_dv = ld_dv;
  a.la = log_alpha; a.beta = beta; a.reset = reset; a.lens = lens;
  a.B = B; a.T = T; a.Hk = Hk; a.H = H; a.dk = dk; a.dv = dv;
  a.state_in = dstate; a.state_out = dstate_out; a.err = dev_err;
  a.drop = test_drop_signal();
  a.odq = dq; a.odk = dk_out; a.odv = dv_out; a.dla = dlog_alpha; a.dbeta = dbeta;
  if (static_cast<int64_t>(B) * H > 0 &&
      (!dstate_out || !workspace || (T > 0 && (!dy || !dq || !dk_out || !dv_out || !dlog_alpha || !dbeta))))
    return set_error(SDM_ERR_INVALID_ARG, "gdn_backward: null pointer");
  const int rc = check_common("gdn_backward", a, saved, saved_bytes, l);
  if (rc != SDM_OK) return rc;
  if (ld_dq < static_cast<int64_t>(Hk) * dk || ld_dk < static_cast<int64_t>(Hk) * dk ||
      ld_dv < static_cast<int64_t>(H) * dv || ld_dq >= (1 << 27) || ld_dk >= (1 << 27) || ld_dv >= (1 << 27))
    return set_error(SDM_ERR_SHAPE,
                     "gdn_backward: a token's row must be at most 2^27 elements from the next and hold its heads");
  if (!aligned(dy, 2) || !aligned(dq, 2) || !aligned(dk_out, 2) || !aligned(dv_out, 2) || !aligned(dlog_alpha, 4) ||
      !aligned(dbeta, 4) || !aligned(workspace, 16))
    return set_error(SDM_ERR_ALIGN, "gdn_backward: a pointer is not aligned");
  if (workspace_bytes < l.work)
    return set_error(SDM_ERR_INVALID_ARG, "gdn_backward: workspace of %zu bytes, %zu needed", workspace_bytes, l.work);
  if (B == 0 || (H == 0 && (T == 0 || Hk == 0))) return SDM_OK;
  a.by_qk = std::min(row_bytes(q, ld_q, dk), row_bytes(k, ld_k, dk));
  a.by_dy = row_bytes(dy, static_cast<int64_t>(H) * dv, dv);
  a.pair_y = dv % 2 == 0 && ld_dv % 2 == 0 && aligned(dv_out, 4);
  a.pair_qk = dk % 2 == 0 && ld_dq % 2 == 0 && ld_dk % 2 == 0 && aligned(dq, 4) && aligned(dk_out, 4);
  if (H == 0) {  // key heads that no value head reads: sums of nothing
    if (!dq || !dk_out) return set_error(SDM_ERR_INVALID_ARG, "gdn_backward: null pointer");
    return launch(gdn_grad_heads, "gdn_backward", static_cast<int64_t>(B) * T, 256, 0,
                  static_cast<cudaStream_t>(stream), a);
  }
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
