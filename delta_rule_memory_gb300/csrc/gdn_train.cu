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
#include <algorithm>
#include <climits>

#include "common.cuh"
#include "mma.cuh"
#include "umma.cuh"

namespace sdm {
namespace {

using namespace mma;

constexpr int kC = 64;                  // tokens of a chunk
constexpr int kTile = kC * kC * 2;      // bytes of one bf16 [64][64] tile
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
  int vec_qk, vec_v, vec_dy;   // rows of q, k / v / dy can be copied by 16 bytes
  int vec_y;                   // y (or dv) can be written by pairs
  float *scal;                 // [units][kScal]
  unsigned char *t3, *m3;      // [units][3][64][64] bf16 tiles, swizzled (lower blocks)
  float *s;                    // [units][16-column tiles][dk tiles of 8][lane][4]: S at the chunk's start
  float *e;                    // [units][64][dv]
  float *g;                    // as s, n + 1 a sequence: G at chunk c's start, G_T behind the last
  float *dz;                   // [units][64][dv]
  const float *state_in;
  float *state_out;
  uint16_t *y, *odq, *odk, *odv;
  float *dla, *dbeta;
  float *pdq, *pdk;            // [B,T,H,dk] where several heads share a key head
  int32_t *err;
};

__device__ __forceinline__ int length_of(const Gdn &a, int b) {
  return a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
}

// ---------------------------------------------------------------------------
// gdn_prep: decays, M and T of one chunk of one head.
// ---------------------------------------------------------------------------
constexpr int kPrepThreads = 128;

__device__ __forceinline__ void store_parts3(unsigned char *tiles, uint32_t off, const float *x) {
  uint32_t s[4][3];
#pragma unroll
  for (int i = 0; i < 4; ++i) split<3>(x[2 * i], x[2 * i + 1], s[i]);
#pragma unroll
  for (int p = 0; p < 3; ++p)
    *reinterpret_cast<uint4 *>(tiles + p * kTile + off) = make_uint4(s[0][p], s[1][p], s[2][p], s[3][p]);
}

// the lower blocks of an fp32 [64][kLd] matrix as three tiles
__device__ __forceinline__ void write_tiles(const float *x, unsigned char *tiles, int tid) {
  for (int id = tid; id < kC * 8; id += kPrepThreads) {
    const int i = id >> 3, p = id & 7;
    if (p > 2 * (i >> 4) + 1) continue;
    float v[8];
    *reinterpret_cast<float4 *>(v) = *reinterpret_cast<const float4 *>(x + i * kLd + p * 8);
    *reinterpret_cast<float4 *>(v + 4) = *reinterpret_cast<const float4 *>(x + i * kLd + p * 8 + 4);
    store_parts3(tiles, piece(i, p, 128), v);
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

template <int NK>
__global__ void __launch_bounds__(kPrepThreads) gdn_prep(const Gdn a) {
  constexpr int rb = NK * 32;
  extern __shared__ __align__(1024) unsigned char sm[];
  unsigned char *sK = sm, *sQ = sm + kC * rb;
  float *sL = reinterpret_cast<float *>(sm + 2 * kC * rb), *sX = sL + kC * kLd, *sc = sX + kC * kLd;
  float *zt = reinterpret_cast<float *>(sm);  // the K tile's place, once the products are formed
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int64_t u = blockIdx.x;
  const int64_t bh = u / a.n;
  const int c = static_cast<int>(u - bh * a.n), b = static_cast<int>(bh / a.H), h = static_cast<int>(bh % a.H);
  const int live = min(length_of(a, b) - c * kC, kC);
  if (live <= 0) return;
  const int64_t tok = static_cast<int64_t>(b) * a.T + c * kC;
  const int hk = h / (a.H / a.Hk);
  load_tile(sK, rb, a.k + tok * a.ld_k + hk * a.dk, a.ld_k, kC, live, a.dk, a.vec_qk, tid, kPrepThreads);
  load_tile(sQ, rb, a.q + tok * a.ld_q + hk * a.dk, a.ld_q, kC, live, a.dk, a.vec_qk, tid, kPrepThreads);
  cp_async_commit();
  float *out = a.scal + u * kScal;
  if (w == 0) {
    // l in units of log2, summed in 64 bits and kept as two floats: a strong
    // decay early in the chunk costs the later, weak ones nothing
    double x[2];
    bool r[2];
    float be[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int m = lane + 32 * i;
      const bool ok = m < live;
      const float la = ok ? a.la[(tok + m) * a.H + h] : 0.f;
      x[i] = static_cast<double>(la < kLeastLog ? kLeastLog : la) * 1.4426950408889634;
      r[i] = ok && a.reset && a.reset[tok + m] != 0;
      be[i] = ok ? a.beta[(tok + m) * a.H + h] : 0.f;
      if (fabsf(be[i]) < kTinyBeta) be[i] = copysignf(kTinyBeta, be[i]);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(kFull, x[i], o);
        if (lane >= o) x[i] += y;
      }
    }
    x[1] += __shfl_sync(kFull, x[0], 31);
    const double end = __shfl_sync(kFull, x[1], 31);
    const uint32_t b0 = __ballot_sync(kFull, r[0]), b1 = __ballot_sync(kFull, r[1]);
    const uint32_t upto = 0xffffffffu >> (31 - lane);
    const int seg[2] = {__popc(b0 & upto), __popc(b0) + __popc(b1 & upto)}, last = __popc(b0) + __popc(b1);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int m = lane + 32 * i;
      const float hi = static_cast<float>(x[i]), lo = static_cast<float>(x[i] - hi);
      const float v[6] = {seg[i] == 0 ? umma::ex2_approx(hi + lo) : 0.f,
                          seg[i] == last ? umma::ex2_approx(static_cast<float>(end - x[i])) : 0.f,
                          be[i], hi, lo, __int_as_float(seg[i])};
#pragma unroll
      for (int e = 0; e < 6; ++e) {
        sc[e * kC + m] = v[e];
        out[e * kC + m] = v[e];
      }
    }
  }
  cp_async_wait<0>();
  __syncthreads();

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
    a_rows(uK, rb, 16 * w, 16 * ks, lane, ak);
    a_rows(uQ, rb, 16 * w, 16 * ks, lane, aq);
#pragma unroll
    for (int np = 0; np < 4; ++np) {
      if (np > w) continue;
      uint32_t r[4];
      b_rows(uK, rb, 16 * np, 16 * ks, lane, r);
      fma16816(G[2 * np], ak, r[0], r[1]);
      fma16816(G[2 * np + 1], ak, r[2], r[3]);
      fma16816(P[2 * np], aq, r[0], r[1]);
      fma16816(P[2 * np + 1], aq, r[2], r[3]);
    }
  }
  const float *be = sc + 2 * kC, *lh = sc + 3 * kC, *ll = sc + 4 * kC, *sg = sc + 5 * kC;
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
  write_tiles(sX, a.m3 + u * (3 * kTile), tid);
  __syncthreads();
  invert(sL, sX, zt, tid);
  write_tiles(sX, a.t3 + u * (3 * kTile), tid);
}

// ---------------------------------------------------------------------------
// The chains.
// ---------------------------------------------------------------------------
constexpr int kWarps = 4;  // warps of a CTA, 16 value columns each

template <int NK, int PM>  // PM: parts of M
struct Stage {
  static constexpr int rb = NK * 32;
  static constexpr int K = 0, Q = K + kC * rb, T = Q + kC * rb, M = T + 3 * kTile, V = M + PM * kTile,
                       sc = V + kC * 128, size = sc + 3 * kC * 4;
};

// copies of chunk c's tiles into one stage; cols: the value columns' tensor
template <int NK, int PM>
__device__ __forceinline__ void load_stage(unsigned char *st, const Gdn &a, int64_t u, int64_t tok, int h, int col0,
                                           int live, const uint16_t *cols, int64_t ld_cols, bool vec_cols, int tid,
                                           int threads) {
  using L = Stage<NK, PM>;
  const int hk = h / (a.H / a.Hk);
  load_tile(st + L::K, L::rb, a.k + tok * a.ld_k + hk * a.dk, a.ld_k, kC, live, a.dk, a.vec_qk, tid, threads);
  load_tile(st + L::Q, L::rb, a.q + tok * a.ld_q + hk * a.dk, a.ld_q, kC, live, a.dk, a.vec_qk, tid, threads);
  load_tile(st + L::V, 128, cols + tok * ld_cols + h * a.dv + col0, ld_cols, kC, live, min(64, a.dv - col0), vec_cols,
            tid, threads);
  const unsigned char *t3 = a.t3 + u * (3 * kTile), *m3 = a.m3 + u * (3 * kTile);
  const uint32_t dT = smem_u32(st + L::T), dM = smem_u32(st + L::M), ds = smem_u32(st + L::sc);
  for (int id = tid; id < 3 * kTile / 16; id += threads) {
    // of each tile's 64 rows of 8 pieces only the lower blocks hold anything
    const int r = (id >> 3) & 63, p = (id & 7) ^ (r & 7);
    if (p > 2 * (r >> 4) + 1) continue;
    copy16(dT + id * 16, t3 + id * 16, true);
    if (id < PM * (kTile / 16)) copy16(dM + id * 16, m3 + id * 16, true);
  }
  const float *sc = a.scal + u * kScal;
  for (int id = tid; id < 3 * kC / 4; id += threads) copy16(ds + id * 16, sc + id * 4, true);
  cp_async_commit();
}

// S^T of one warp's 16 columns: its registers and a [dk][dv] matrix
template <int NT>
__device__ __forceinline__ void read_state(const float *m, int dk, int dv, int col, int lane, float (&S)[NT][4]) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = 8 * nt + 2 * t + (e & 1), c = col + g + 8 * (e >> 1);
      S[nt][e] = m && r < dk && c < dv ? m[static_cast<int64_t>(r) * dv + c] : 0.f;
    }
}
template <int NT>
__device__ __forceinline__ void write_state(float *m, int dk, int dv, int col, int lane, const float (&S)[NT][4]) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = 8 * nt + 2 * t + (e & 1), c = col + g + 8 * (e >> 1);
      if (r < dk && c < dv) m[static_cast<int64_t>(r) * dv + c] = S[nt][e];
    }
}
// ... and its fragments in a row, 16 bytes a lane
template <int NT>
__device__ __forceinline__ void keep_state(float *m, int lane, const float (&S)[NT][4]) {
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
    reinterpret_cast<float4 *>(m)[nt * 32 + lane] = make_float4(S[nt][0], S[nt][1], S[nt][2], S[nt][3]);
}

// a warp's [16 columns][64 tokens] accumulator into fp32 [64][dv]
__device__ __forceinline__ void keep_tokens(float *m, int dv, int col, int lane, const float (&x)[8][4]) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nt = 0; nt < 8; ++nt)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = 8 * nt + 2 * t + (e & 1), c = col + g + 8 * (e >> 1);
      if (c < dv) m[i * dv + c] = x[nt][e];
    }
}

// d[n] += the product of A's parts and B's parts, n-tiles 2 np and 2 np + 1, whose
// part numbers sum up to less than max(PA, PB): what the others hold is below the last bit kept
template <int PA, int PB, int N>
__device__ __forceinline__ void products(float (&d)[N][4], int np, const uint32_t (&a)[PA][4], const uint32_t (&b)[PB][4]) {
  constexpr int most = PA > PB ? PA : PB;
#pragma unroll
  for (int i = 0; i < PA; ++i)
#pragma unroll
    for (int j = 0; j < PB; ++j)
      if (i + j < most) {
        fma16816(d[2 * np], a[i], b[j][0], b[j][1]);
        fma16816(d[2 * np + 1], a[i], b[j][2], b[j][3]);
      }
}

template <int NK>
__global__ void __launch_bounds__(kWarps * 32, 1) gdn_chain(const Gdn a) {
  using L = Stage<NK, 2>;
  constexpr int NT = 2 * NK, rb = L::rb;
  extern __shared__ __align__(1024) unsigned char sm[];
  const int tid = threadIdx.x, threads = blockDim.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int tiles = (a.dv + 15) >> 4, groups = (tiles + kWarps - 1) / kWarps;
  const int64_t bh = blockIdx.x / groups;
  const int col0 = static_cast<int>(blockIdx.x - bh * groups) * (16 * kWarps), col = col0 + 16 * w;
  const int b = static_cast<int>(bh / a.H), h = static_cast<int>(bh % a.H);
  const int len = length_of(a, b), n = (len + kC - 1) / kC;
  const int64_t tok = static_cast<int64_t>(b) * a.T;
  if (a.err && a.lens && a.lens[b] != len && tid == 0) atomicOr(a.err, SDM_DEVERR_INDEX_RANGE);
  const bool mine = col < a.dv;  // else the warp only helps with the copies

  float S[NT][4];
  read_state<NT>(a.state_in ? a.state_in + bh * a.dk * a.dv : nullptr, a.dk, a.dv, col, lane, S);
  if (n > 0)
    load_stage<NK, 2>(sm, a, bh * a.n, tok, h, col0, min(len, kC), a.v, a.ld_v, a.vec_v, tid, threads);
  for (int c = 0; c < n; ++c) {
    const int64_t u = bh * a.n + c;
    if (c + 1 < n) {
      load_stage<NK, 2>(sm + ((c + 1) & 1) * L::size, a, u + 1, tok + (c + 1) * kC, h, col0, min(len - (c + 1) * kC, kC),
                        a.v, a.ld_v, a.vec_v, tid, threads);
      cp_async_wait<1>();
    } else {
      cp_async_wait<0>();
    }
    __syncthreads();
    if (mine) {
      unsigned char *st = sm + (c & 1) * L::size;
      const uint32_t uK = smem_u32(st + L::K), uQ = smem_u32(st + L::Q), uT = smem_u32(st + L::T),
                     uM = smem_u32(st + L::M), uV = smem_u32(st + L::V);
      const float *gam = reinterpret_cast<const float *>(st + L::sc), *tail = gam + kC, *beta = tail + kC;
      keep_state<NT>(a.s + (u * tiles + (col >> 4)) * (NT * 128), lane, S);
      // S^T K^T and S^T Q^T
      float E[8][4], Y[8][4], Z[8][4];
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) E[i][e] = Y[i][e] = Z[i][e] = 0.f;
#pragma unroll
      for (int ks = 0; ks < NK; ++ks) {
        uint32_t s[3][4];
        a_split<3>(S[2 * ks], S[2 * ks + 1], s);
        const uint32_t s2[2][4] = {{s[0][0], s[0][1], s[0][2], s[0][3]}, {s[1][0], s[1][1], s[1][2], s[1][3]}};
#pragma unroll
        for (int np = 0; np < 4; ++np) {
          uint32_t r[1][4];
          b_rows(uK, rb, 16 * np, 16 * ks, lane, r[0]);
          products(Z, np, s, r);
          b_rows(uQ, rb, 16 * np, 16 * ks, lane, r[0]);
          products(Y, np, s2, r);
        }
      }
      // Z^T = V^T - gam S^T K^T; gam S^T Q^T
#pragma unroll
      for (int np = 0; np < 4; ++np) {
        uint32_t v[4];
        // tile[token][column]: rows of V^T are its columns
        ldsm4_t(uV + piece(16 * np + (((lane >> 4) & 1) << 3) + (lane & 7), 2 * w + ((lane >> 3) & 1), 128), v);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int nt = 2 * np + x;
          const float2 gm = *reinterpret_cast<const float2 *>(gam + 8 * nt + 2 * t);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float gg = e & 1 ? gm.y : gm.x;
            const uint32_t vv = v[2 * x + (e >> 1)];
            Z[nt][e] = fmaf(-gg, Z[nt][e], e & 1 ? high2(vv) : low2(vv));
            Y[nt][e] *= gg;
          }
        }
      }
      // E^T = Z^T T^T
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        uint32_t z[3][4];
        a_split<3>(Z[2 * ks], Z[2 * ks + 1], z);
#pragma unroll
        for (int np = ks; np < 4; ++np) {
          uint32_t r[3][4];
#pragma unroll
          for (int p = 0; p < 3; ++p) b_rows(uT + p * kTile, 128, 16 * np, 16 * ks, lane, r[p]);
          products(E, np, z, r);
        }
      }
      keep_tokens(a.e + u * kC * a.dv, a.dv, col, lane, E);
      // U = beta E;  Y^T += U^T M^T;  S^T = gam_C S^T + (tail U)^T K
      const float end = gam[kC - 1];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[nt][e] *= end;
#pragma unroll
      for (int nt = 0; nt < 8; ++nt) {
        const float2 be = *reinterpret_cast<const float2 *>(beta + 8 * nt + 2 * t);
#pragma unroll
        for (int e = 0; e < 4; ++e) E[nt][e] *= e & 1 ? be.y : be.x;
      }
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        uint32_t us[2][4];
        a_split<2>(E[2 * ks], E[2 * ks + 1], us);
#pragma unroll
        for (int np = ks; np < 4; ++np) {
          uint32_t r[2][4];
#pragma unroll
          for (int p = 0; p < 2; ++p) b_rows(uM + p * kTile, 128, 16 * np, 16 * ks, lane, r[p]);
          products(Y, np, us, r);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float2 tl = *reinterpret_cast<const float2 *>(tail + 8 * (2 * ks + x) + 2 * t);
#pragma unroll
          for (int e = 0; e < 4; ++e) E[2 * ks + x][e] *= e & 1 ? tl.y : tl.x;
        }
        uint32_t ut[3][4];
        a_split<3>(E[2 * ks], E[2 * ks + 1], ut);
#pragma unroll
        for (int np = 0; np < NK; ++np) {
          uint32_t r[1][4];
          b_cols(uK, rb, 16 * np, 16 * ks, lane, r[0]);
          products(S, np, ut, r);
        }
      }
      // y, rounded once: pairs of tokens turned into pairs of columns
#pragma unroll
      for (int nt = 0; nt < 8; ++nt) {
        const int i = c * kC + 8 * nt + g;
        uint16_t *row = a.y + ((tok + i) * a.H + h) * a.dv;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t v = transpose8(pack2(Y[nt][2 * x], Y[nt][2 * x + 1]));
          const int cc = col + 8 * x + 2 * t;
          if (i >= len) continue;
          if (a.vec_y && cc + 1 < a.dv) {
            *reinterpret_cast<uint32_t *>(row + cc) = v;
          } else {
            if (cc < a.dv) row[cc] = static_cast<uint16_t>(v);
            if (cc + 1 < a.dv) row[cc + 1] = static_cast<uint16_t>(v >> 16);
          }
        }
      }
    }
    __syncthreads();
  }
  if (mine) write_state<NT>(a.state_out + bh * a.dk * a.dv, a.dk, a.dv, col, lane, S);
}

template <int NK>
__global__ void __launch_bounds__(kWarps * 32, 1) gdn_chain_back(const Gdn a) {
  using L = Stage<NK, 3>;
  constexpr int NT = 2 * NK, rb = L::rb;
  extern __shared__ __align__(1024) unsigned char sm[];
  const int tid = threadIdx.x, threads = blockDim.x, w = tid >> 5, lane = tid & 31, t = lane & 3;
  const int tiles = (a.dv + 15) >> 4, groups = (tiles + kWarps - 1) / kWarps;
  const int64_t bh = blockIdx.x / groups;
  const int col0 = static_cast<int>(blockIdx.x - bh * groups) * (16 * kWarps), col = col0 + 16 * w;
  const int b = static_cast<int>(bh / a.H), h = static_cast<int>(bh % a.H);
  const int len = length_of(a, b), n = (len + kC - 1) / kC;
  const int64_t tok = static_cast<int64_t>(b) * a.T, ld_y = static_cast<int64_t>(a.H) * a.dv;
  if (a.err && a.lens && a.lens[b] != len && tid == 0) atomicOr(a.err, SDM_DEVERR_INDEX_RANGE);
  const bool mine = col < a.dv;

  float S[NT][4];  // G^T
  read_state<NT>(a.state_in ? a.state_in + bh * a.dk * a.dv : nullptr, a.dk, a.dv, col, lane, S);
  float *kept = a.g + (bh * (a.n + 1) * tiles + (col >> 4)) * (NT * 128);
  const int64_t step = static_cast<int64_t>(tiles) * (NT * 128);
  if (mine) keep_state<NT>(kept + n * step, lane, S);
  if (n > 0)
    load_stage<NK, 3>(sm + ((n - 1) & 1) * L::size, a, bh * a.n + n - 1, tok + (n - 1) * kC, h, col0,
                      min(len - (n - 1) * kC, kC), a.dy, ld_y, a.vec_dy, tid, threads);
  for (int c = n - 1; c >= 0; --c) {
    const int64_t u = bh * a.n + c;
    if (c > 0) {
      load_stage<NK, 3>(sm + ((c - 1) & 1) * L::size, a, u - 1, tok + (c - 1) * kC, h, col0, kC, a.dy, ld_y, a.vec_dy, tid,
                        threads);
      cp_async_wait<1>();
    } else {
      cp_async_wait<0>();
    }
    __syncthreads();
    if (mine) {
      unsigned char *st = sm + (c & 1) * L::size;
      const uint32_t uK = smem_u32(st + L::K), uQ = smem_u32(st + L::Q), uT = smem_u32(st + L::T),
                     uM = smem_u32(st + L::M), uY = smem_u32(st + L::V);
      const float *gam = reinterpret_cast<const float *>(st + L::sc), *tail = gam + kC, *beta = tail + kC;
      // dU^T = tail G^T K^T + dY^T M
      float U[8][4], Z[8][4];
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) U[i][e] = Z[i][e] = 0.f;
#pragma unroll
      for (int ks = 0; ks < NK; ++ks) {
        uint32_t s[3][4];
        a_split<3>(S[2 * ks], S[2 * ks + 1], s);
#pragma unroll
        for (int np = 0; np < 4; ++np) {
          uint32_t r[1][4];
          b_rows(uK, rb, 16 * np, 16 * ks, lane, r[0]);
          products(U, np, s, r);
        }
      }
#pragma unroll
      for (int nt = 0; nt < 8; ++nt) {
        const float2 tl = *reinterpret_cast<const float2 *>(tail + 8 * nt + 2 * t);
#pragma unroll
        for (int e = 0; e < 4; ++e) U[nt][e] *= e & 1 ? tl.y : tl.x;
      }
      uint32_t y[4][1][4];
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        a_cols(uY, 128, 16 * w, 16 * ks, lane, y[ks][0]);
#pragma unroll
        for (int np = 0; np <= ks; ++np) {
          uint32_t r[3][4];
#pragma unroll
          for (int p = 0; p < 3; ++p) b_cols(uM + p * kTile, 128, 16 * np, 16 * ks, lane, r[p]);
          products(U, np, y[ks], r);
        }
      }
      // dZ^T = (beta dU)^T T
#pragma unroll
      for (int nt = 0; nt < 8; ++nt) {
        const float2 be = *reinterpret_cast<const float2 *>(beta + 8 * nt + 2 * t);
#pragma unroll
        for (int e = 0; e < 4; ++e) U[nt][e] *= e & 1 ? be.y : be.x;
      }
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        uint32_t x[3][4];
        a_split<3>(U[2 * ks], U[2 * ks + 1], x);
#pragma unroll
        for (int np = 0; np <= ks; ++np) {
          uint32_t r[3][4];
#pragma unroll
          for (int p = 0; p < 3; ++p) b_cols(uT + p * kTile, 128, 16 * np, 16 * ks, lane, r[p]);
          products(Z, np, x, r);
        }
      }
      keep_tokens(a.dz + u * kC * a.dv, a.dv, col, lane, Z);
      // G^T = gam_C G^T + (gam dY)^T Q - (gam dZ)^T K
      const float end = gam[kC - 1];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[nt][e] *= end;
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        float d[2][4];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float2 gm = *reinterpret_cast<const float2 *>(gam + 8 * (2 * ks + x) + 2 * t);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float gg = e & 1 ? gm.y : gm.x;
            const uint32_t v = y[ks][0][2 * x + (e >> 1)];
            d[x][e] = gg * (e & 1 ? high2(v) : low2(v));
            Z[2 * ks + x][e] *= -gg;
          }
        }
        uint32_t dy3[3][4], dz3[3][4];
        a_split<3>(d[0], d[1], dy3);
        a_split<3>(Z[2 * ks], Z[2 * ks + 1], dz3);
#pragma unroll
        for (int np = 0; np < NK; ++np) {
          uint32_t r[1][4];
          b_cols(uQ, rb, 16 * np, 16 * ks, lane, r[0]);
          products(S, np, dy3, r);
          b_cols(uK, rb, 16 * np, 16 * ks, lane, r[0]);
          products(S, np, dz3, r);
        }
      }
      keep_state<NT>(kept + c * step, lane, S);
    }
    __syncthreads();
  }
  if (mine) write_state<NT>(a.state_out + bh * a.dk * a.dv, a.dk, a.dv, col, lane, S);
}

// ---------------------------------------------------------------------------
// gdn_grad: the gradients of one chunk of one head.  Eight warps: warp (mi, nj)
// has tokens 16 mi .. +15 and half nj of the key channels (of the tokens j, for X and
// N).  The value columns come 64 at a time: E, dZ and the two states are read
// as fp32, split into bf16 parts and stored as tiles.
// ---------------------------------------------------------------------------
constexpr int kGradThreads = 256;

template <int NK>
struct GradSmem {
  static constexpr int rb = NK * 32;
  static constexpr int K = 0, Q = K + kC * rb, Y = Q + kC * rb, U = Y + kTile, Z = U + 3 * kTile, S = Z + 2 * kTile,
                       G = S + 3 * 64 * rb, sc = G + 2 * 64 * rb, size = sc + (kScal + 4 * kC + 16) * 4;
  static constexpr int X = U, N = Z;  // once the value columns are done: X in three parts, N + N^T in two
};

template <int NK>
__global__ void __launch_bounds__(kGradThreads, 1) gdn_grad(const Gdn a) {
  using L = GradSmem<NK>;
  constexpr int rb = L::rb, NT = 2 * NK, NP = NK / 2;  // NP: pairs of n-tiles in half the key channels
  extern __shared__ __align__(1024) unsigned char sm[];
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3, mi = w & 3, nj = w >> 2;
  const int64_t u = blockIdx.x, bh = u / a.n;
  const int c = static_cast<int>(u - bh * a.n), b = static_cast<int>(bh / a.H), h = static_cast<int>(bh % a.H);
  const int live = min(length_of(a, b) - c * kC, kC);
  if (live <= 0) return;
  const int64_t tok = static_cast<int64_t>(b) * a.T + c * kC, ld_y = static_cast<int64_t>(a.H) * a.dv;
  const int hk = h / (a.H / a.Hk), tiles = (a.dv + 15) >> 4;
  float *sc = reinterpret_cast<float *>(sm + L::sc);
  float *gam = sc, *tail = sc + kC, *beta = sc + 2 * kC, *lh = sc + 3 * kC, *ll = sc + 4 * kC, *sg = sc + 5 * kC;
  float *rowEZ = sc + kScal, *rowVZ = rowEZ + kC, *flow = rowVZ + kC /* [2][64] */, *red = flow + 2 * kC;
  load_tile(sm + L::K, rb, a.k + tok * a.ld_k + hk * a.dk, a.ld_k, kC, live, a.dk, a.vec_qk, tid, kGradThreads);
  load_tile(sm + L::Q, rb, a.q + tok * a.ld_q + hk * a.dk, a.ld_q, kC, live, a.dk, a.vec_qk, tid, kGradThreads);
  for (int i = tid; i < kScal; i += kGradThreads) sc[i] = a.scal[u * kScal + i];
  const uint32_t uK = smem_u32(sm + L::K), uQ = smem_u32(sm + L::Q), uY = smem_u32(sm + L::Y), uU = smem_u32(sm + L::U),
                 uZ = smem_u32(sm + L::Z), uS = smem_u32(sm + L::S), uG = smem_u32(sm + L::G);

  float dQ[2 * NP][4], dA[2 * NP][4], dK[2 * NP][4], X[4][4], N[4][4];
#pragma unroll
  for (int i = 0; i < 2 * NP; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) dQ[i][e] = dA[i][e] = dK[i][e] = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) X[i][e] = N[i][e] = 0.f;
  float ez = 0.f, vz = 0.f, anchor = 0.f;
  const int row = tid >> 2, part = tid & 3;  // four threads a token, 16 columns each
  __syncthreads();

  for (int c0 = 0; c0 < a.dv; c0 += 64) {
    const int width = min(64, a.dv - c0);
    load_tile(sm + L::Y, 128, a.dy + tok * ld_y + h * a.dv + c0, ld_y, kC, live, width, a.vec_dy, tid, kGradThreads);
    cp_async_commit();
    {  // E and dZ: U and dZ as tiles, dv, and the sums over a token's columns
      const float *E = a.e + (u * kC + row) * a.dv + c0, *Z = a.dz + (u * kC + row) * a.dv + c0;
      const uint16_t *V = a.v + (tok + row) * a.ld_v + h * a.dv + c0;
      uint16_t *dV = a.odv + (tok + row) * a.ld_dv + h * a.dv + c0;
      const float be = beta[row];
      const bool vec = a.dv % 4 == 0;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int cc = 16 * part + 8 * half;
        float e[8], z[8];
        if (vec && cc + 8 <= width) {
#pragma unroll
          for (int i = 0; i < 8; i += 4) {
            *reinterpret_cast<float4 *>(e + i) = *reinterpret_cast<const float4 *>(E + cc + i);
            *reinterpret_cast<float4 *>(z + i) = *reinterpret_cast<const float4 *>(Z + cc + i);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            e[i] = cc + i < width ? E[cc + i] : 0.f;
            z[i] = cc + i < width ? Z[cc + i] : 0.f;
          }
        }
        if (row < live) {
          if (a.vec_v && cc + 8 <= width) {
            const uint4 vv = *reinterpret_cast<const uint4 *>(V + cc);
            const uint32_t vw[4] = {vv.x, vv.y, vv.z, vv.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) vz += low2(vw[i]) * z[2 * i] + high2(vw[i]) * z[2 * i + 1];
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (cc + i < width) vz += bf16_to_f32(V[cc + i]) * z[i];
          }
          if (a.vec_y && cc + 8 <= width) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint32_t *>(dV + cc + 2 * i) = pack2(z[2 * i], z[2 * i + 1]);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (cc + i < width) dV[cc + i] = static_cast<uint16_t>(pack2(z[i], 0.f));
          }
        }
        uint32_t su[4][3], sz[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ez += e[2 * i] * z[2 * i] + e[2 * i + 1] * z[2 * i + 1];
          split<3>(be * e[2 * i], be * e[2 * i + 1], su[i]);
          split<2>(z[2 * i], z[2 * i + 1], sz[i]);
        }
        const uint32_t off = piece(row, cc >> 3, 128);
#pragma unroll
        for (int p = 0; p < 3; ++p)
          *reinterpret_cast<uint4 *>(sm + L::U + p * kTile + off) = make_uint4(su[0][p], su[1][p], su[2][p], su[3][p]);
#pragma unroll
        for (int p = 0; p < 2; ++p)
          *reinterpret_cast<uint4 *>(sm + L::Z + p * kTile + off) = make_uint4(sz[0][p], sz[1][p], sz[2][p], sz[3][p]);
      }
    }
    // the states: S and G at the chunk's two ends as tiles [column][key channel]; <S, G_start>
    {
      const int ct0 = c0 >> 4;
      const float4 *S = reinterpret_cast<const float4 *>(a.s) + (u * tiles + ct0) * (NT * 32);
      const float4 *G0 = reinterpret_cast<const float4 *>(a.g) + ((bh * (a.n + 1) + c) * tiles + ct0) * (NT * 32);
      const float4 *G1 = G0 + tiles * (NT * 32);
#pragma unroll 4
      for (int id = tid; id < 4 * NT * 32; id += kGradThreads) {
        const int ct = id / (NT * 32), nt = (id >> 5) % NT;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f), x = s;
        if (ct0 + ct < tiles) {
          s = S[id];
          x = G1[id];
          const float4 y = G0[id];
          anchor += (s.x * y.x + s.y * y.y) + (s.z * y.z + s.w * y.w);
        }
        const uint32_t o0 = piece(16 * ct + g, nt, rb) + 4 * t, o1 = piece(16 * ct + g + 8, nt, rb) + 4 * t;
        uint32_t p0[3], p1[3], g0[2], g1[2];
        split<3>(s.x, s.y, p0);
        split<3>(s.z, s.w, p1);
        split<2>(x.x, x.y, g0);
        split<2>(x.z, x.w, g1);
#pragma unroll
        for (int p = 0; p < 3; ++p) {
          *reinterpret_cast<uint32_t *>(sm + L::S + p * 64 * rb + o0) = p0[p];
          *reinterpret_cast<uint32_t *>(sm + L::S + p * 64 * rb + o1) = p1[p];
        }
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          *reinterpret_cast<uint32_t *>(sm + L::G + p * 64 * rb + o0) = g0[p];
          *reinterpret_cast<uint32_t *>(sm + L::G + p * 64 * rb + o1) = g1[p];
        }
      }
    }
    cp_async_wait<0>();
    __syncthreads();
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      uint32_t y[1][4], uu[2][4], z[2][4];
      a_rows(uY, 128, 16 * mi, 16 * ks, lane, y[0]);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        a_rows(uU + p * kTile, 128, 16 * mi, 16 * ks, lane, uu[p]);
        a_rows(uZ + p * kTile, 128, 16 * mi, 16 * ks, lane, z[p]);
      }
#pragma unroll
      for (int np = 0; np < NP; ++np) {
        const int n0 = nj * (NK * 8) + 16 * np;
        uint32_t r[3][4];
#pragma unroll
        for (int p = 0; p < 3; ++p) b_cols(uS + p * 64 * rb, rb, n0, 16 * ks, lane, r[p]);
        products(dQ, np, y, r);
        const uint32_t r2[2][4] = {{r[0][0], r[0][1], r[0][2], r[0][3]}, {r[1][0], r[1][1], r[1][2], r[1][3]}};
        products(dA, np, z, r2);
        uint32_t q[2][4];
#pragma unroll
        for (int p = 0; p < 2; ++p) b_cols(uG + p * 64 * rb, rb, n0, 16 * ks, lane, q[p]);
        products(dK, np, uu, q);
      }
#pragma unroll
      for (int np = 0; np < 2; ++np) {
        const int n0 = 32 * nj + 16 * np;
        if (n0 > 16 * mi) continue;
        uint32_t r[3][4];
#pragma unroll
        for (int p = 0; p < 3; ++p) b_rows(uU + p * kTile, 128, n0, 16 * ks, lane, r[p]);
        products(X, np, y, r);
        const uint32_t r2[2][4] = {{r[0][0], r[0][1], r[0][2], r[0][3]}, {r[1][0], r[1][1], r[1][2], r[1][3]}};
        products(N, np, z, r2);
      }
    }
    __syncthreads();
  }

  // sums over a token's columns and over the state
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    ez += __shfl_xor_sync(kFull, ez, o);
    vz += __shfl_xor_sync(kFull, vz, o);
  }
  if (part == 0) {
    rowEZ[row] = ez;
    rowVZ[row] = vz;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) anchor += __shfl_xor_sync(kFull, anchor, o);
  if (lane == 0) red[w] = anchor;

  const int i0 = 16 * mi + g;
#pragma unroll
  for (int nt = 0; nt < 2 * NP; ++nt)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = i0 + 8 * (e >> 1);
      dQ[nt][e] *= gam[i];
      dK[nt][e] = tail[i] * dK[nt][e] - gam[i] * dA[nt][e];
    }
#pragma unroll
  for (int nt = 0; nt < 4; ++nt) {
    if (32 * nj + 8 * nt > 16 * mi + 15) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = i0 + 8 * (e >> 1), j = 32 * nj + 8 * nt + 2 * t + (e & 1);
      const bool on = j <= i && __float_as_int(sg[i]) == __float_as_int(sg[j]);
      const float d = on ? umma::ex2_approx((lh[i] - lh[j]) + (ll[i] - ll[j])) : 0.f;
      X[nt][e] = on ? d * X[nt][e] : 0.f;
      N[nt][e] = on && j < i ? -d * N[nt][e] : 0.f;
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int i = i0 + 8 * x, j = 32 * nj + 8 * nt + 2 * t;
      uint32_t s[3], m[2];
      split<3>(X[nt][2 * x], X[nt][2 * x + 1], s);
      split<2>(N[nt][2 * x], N[nt][2 * x + 1], m);
      const uint32_t off = piece(i, j >> 3, 128) + 2 * (j & 7);
#pragma unroll
      for (int p = 0; p < 3; ++p) *reinterpret_cast<uint32_t *>(sm + L::X + p * kTile + off) = s[p];
#pragma unroll
      for (int p = 0; p < 2; ++p) {  // N below the diagonal, N^T above it
        unsigned char *tile = sm + L::N + p * kTile;
        const uint16_t lo = static_cast<uint16_t>(m[p]), hi = static_cast<uint16_t>(m[p] >> 16);
        if (j <= i) {
          *reinterpret_cast<uint16_t *>(tile + off) = lo;
          *reinterpret_cast<uint16_t *>(tile + piece(j, i >> 3, 128) + 2 * (i & 7)) = lo;
        }
        if (j + 1 <= i) {
          *reinterpret_cast<uint16_t *>(tile + off + 2) = hi;
          *reinterpret_cast<uint16_t *>(tile + piece(j + 1, i >> 3, 128) + 2 * (i & 7)) = hi;
        }
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) {
    uint32_t x[3][4], xt[2][4], m[2][4];
    const bool low = ks <= mi, up = ks >= mi;
#pragma unroll
    for (int p = 0; p < 2; ++p) a_rows(smem_u32(sm + L::N + p * kTile), 128, 16 * mi, 16 * ks, lane, m[p]);
    if (low)
#pragma unroll
      for (int p = 0; p < 3; ++p) a_rows(smem_u32(sm + L::X + p * kTile), 128, 16 * mi, 16 * ks, lane, x[p]);
    if (up)
#pragma unroll
      for (int p = 0; p < 2; ++p) a_cols(smem_u32(sm + L::X + p * kTile), 128, 16 * mi, 16 * ks, lane, xt[p]);
#pragma unroll
    for (int np = 0; np < NP; ++np) {
      const int n0 = nj * (NK * 8) + 16 * np;
      uint32_t r[1][4];
      b_cols(uK, rb, n0, 16 * ks, lane, r[0]);
      products(dK, np, m, r);
      if (low) products(dQ, np, x, r);
      if (up) {
        b_cols(uQ, rb, n0, 16 * ks, lane, r[0]);
        products(dK, np, xt, r);
      }
    }
  }
  // q . dq, then the outputs
  float qd[2] = {0.f, 0.f};
#pragma unroll
  for (int nt = 0; nt < 2 * NP; ++nt)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const uint32_t v = *reinterpret_cast<const uint32_t *>(sm + L::Q + piece(i0 + 8 * x, nj * NK + nt, rb) + 4 * t);
      qd[x] += low2(v) * dQ[nt][2 * x] + high2(v) * dQ[nt][2 * x + 1];
    }
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    qd[x] += __shfl_xor_sync(kFull, qd[x], 1);
    qd[x] += __shfl_xor_sync(kFull, qd[x], 2);
    if (t == 0) flow[nj * kC + i0 + 8 * x] = qd[x];
  }
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int i = i0 + 8 * x;
    if (i >= live) continue;
#pragma unroll
    for (int nt = 0; nt < 2 * NP; ++nt) {
      const int cc = nj * (NK * 8) + 8 * nt + 2 * t;
      if (cc >= a.dk) continue;
      const float q0 = dQ[nt][2 * x], q1 = dQ[nt][2 * x + 1], k0 = dK[nt][2 * x], k1 = dK[nt][2 * x + 1];
      if (a.pdq) {
        const int64_t o = ((tok + i) * a.H + h) * a.dk + cc;
        a.pdq[o] = q0;
        a.pdk[o] = k0;
        if (cc + 1 < a.dk) {
          a.pdq[o + 1] = q1;
          a.pdk[o + 1] = k1;
        }
      } else {
        uint16_t *oq = a.odq + (tok + i) * a.ld_dq + h * a.dk + cc, *ok = a.odk + (tok + i) * a.ld_dk + h * a.dk + cc;
        const uint32_t vq = pack2(q0, q1), vk = pack2(k0, k1);
        if (a.vec_qk && cc + 1 < a.dk) {
          *reinterpret_cast<uint32_t *>(oq) = vq;
          *reinterpret_cast<uint32_t *>(ok) = vk;
        } else {
          oq[0] = static_cast<uint16_t>(vq);
          ok[0] = static_cast<uint16_t>(vk);
          if (cc + 1 < a.dk) {
            oq[1] = static_cast<uint16_t>(vq >> 16);
            ok[1] = static_cast<uint16_t>(vk >> 16);
          }
        }
      }
    }
  }
  __syncthreads();
  if (w == 0) {  // the decays' gradient: sums before each token, in 64 bits (they cancel)
    double start = 0.0;
    for (int i = 0; i < kGradThreads / 32; ++i) start += red[i];
    double x[2], before[2];
    int seg[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int m = lane + 32 * i;
      before[i] = x[i] = static_cast<double>(flow[m] + flow[kC + m]) - rowVZ[m];
      seg[i] = __float_as_int(sg[m]);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(kFull, x[i], o);
        if (lane >= o) x[i] += y;
      }
    }
    x[1] += __shfl_sync(kFull, x[0], 31);
    const uint32_t s0 = __ballot_sync(kFull, lane == 0 || seg[0] != __float_as_int(sg[max(lane - 1, 0)]));
    const uint32_t s1 = __ballot_sync(kFull, seg[1] != __float_as_int(sg[lane + 31]));
    before[0] = x[0] - before[0];  // sum over s < t
    before[1] = x[1] - before[1];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int m = lane + 32 * i;
      // the first token of this one's document
      const uint32_t upto = 0xffffffffu >> (31 - lane);
      const int first = i == 0 ? 31 - __clz(s0 & upto) : (s1 & upto) ? 63 - __clz(s1 & upto) : 31 - __clz(s0);
      const double p0 = __shfl_sync(kFull, before[0], first & 31), p1 = __shfl_sync(kFull, before[1], first & 31);
      const double base = first < 32 ? p0 : p1;
      if (m < live) {
        const double v = (seg[i] == 0 ? start : 0.0) - (before[i] - base);
        a.dla[(tok + m) * a.H + h] = static_cast<float>(v);
        a.dbeta[(tok + m) * a.H + h] = rowEZ[m] / beta[m];
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
  l.m3 = up(l.t3 + units * 3 * kTile);
  l.s = up(l.m3 + units * 3 * kTile);
  l.e = up(l.s + units * l.state * 4);
  l.saved = up(l.e + units * kC * dv * 4);
  const size_t part = Hk == H ? 0 : static_cast<size_t>(B) * T * H * dk * 4;
  l.g = 0;
  l.dz = up(static_cast<size_t>(B) * H * (l.n + 1) * l.state * 4);
  l.pdq = up(l.dz + units * kC * dv * 4);
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
int launch(K kernel, const char *what, int64_t grid, int threads, int smem, const Gdn &a, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return set_error(SDM_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  kernel<<<static_cast<unsigned>(grid), threads, smem, st>>>(a);
  return check_launch(what);
}

template <int NK>
int run_train(const Gdn &a, const Layout &l, cudaStream_t st) {
  if (l.units > 0) {
    const int rc = launch(gdn_prep<NK>, "gdn_train", l.units, kPrepThreads, 2 * kC * NK * 32 + (2 * kC * kLd + kScal) * 4, a, st);
    if (rc != SDM_OK) return rc;
  }
  const int64_t groups = (l.tiles + kWarps - 1) / kWarps;
  return launch(gdn_chain<NK>, "gdn_train", groups * a.B * a.H, 32 * static_cast<int>(std::min<int64_t>(kWarps, l.tiles)),
                2 * Stage<NK, 2>::size, a, st);
}

template <int NK>
int run_backward(const Gdn &a, const Layout &l, cudaStream_t st) {
  const int64_t groups = (l.tiles + kWarps - 1) / kWarps;
  int rc = launch(gdn_chain_back<NK>, "gdn_backward", groups * a.B * a.H,
                  32 * static_cast<int>(std::min<int64_t>(kWarps, l.tiles)), 2 * Stage<NK, 3>::size, a, st);
  if (rc != SDM_OK || l.units == 0) return rc;
  rc = launch(gdn_grad<NK>, "gdn_backward", l.units, kGradThreads, GradSmem<NK>::size, a, st);
  if (rc != SDM_OK || !a.pdq) return rc;
  gdn_grad_heads<<<static_cast<unsigned>(static_cast<int64_t>(a.B) * a.T), 256, 0, st>>>(a);
  return check_launch("gdn_backward");
}

}  // namespace
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
  a.vec_qk = dk % 8 == 0 && ld_q % 8 == 0 && ld_k % 8 == 0 && aligned(q, 16) && aligned(k, 16);
  a.vec_v = dv % 8 == 0 && ld_v % 8 == 0 && aligned(v, 16);
  a.vec_y = dv % 2 == 0 && aligned(y, 4);
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
  a.vec_qk = dk % 8 == 0 && ld_q % 8 == 0 && ld_k % 8 == 0 && aligned(q, 16) && aligned(k, 16) && ld_dq % 2 == 0 &&
             ld_dk % 2 == 0 && aligned(dq, 4) && aligned(dk_out, 4);
  a.vec_v = dv % 8 == 0 && ld_v % 8 == 0 && aligned(v, 16);
  a.vec_dy = dv % 8 == 0 && aligned(dy, 16);
  a.vec_y = dv % 2 == 0 && ld_dv % 2 == 0 && aligned(dv_out, 4);
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
