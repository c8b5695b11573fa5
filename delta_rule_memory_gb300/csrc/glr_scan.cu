// glr_scan.cu - gated linear recurrence with one state per channel, its
// training forward and its backward pass (glr_scan in sdm.h):
//   L_t = -rate sigmoid(r_t), a_t = e^{L_t}, m_t = sqrt(1 - a_t^2),
//   h_t = a_t h_{t-1} + m_t sigmoid(g_t) x_t.
//
// A run of tokens acts on the state before it as h -> P h + H (P the product
// of its decays, H what it leaves when it starts from 0), and runs compose:
// that splits the sequence.  A warp owns 64 channels (a pair per lane) of 8
// tokens: it forms its run's (P, H), takes the state in front of it from the
// runs before, and steps its tokens through once more with the gates still in
// registers.  Four warps make a CTA (32 tokens), up to eight CTAs a cluster
// (256 tokens, runs exchanged through distributed shared memory), and the
// cluster walks the sequence.  Every input is read once and every output
// written once, no CTA waits for another outside its cluster, and the order of
// every sum is fixed by the sizes.
#include <initializer_list>
#include <type_traits>

#include "ckpt8.cuh"
#include "umma.cuh"

namespace sdm {

int test_drop_signal();  // gdn_chunk.cu: the SDM_TEST_DROP_SIGNAL test hook
SDM_STICKY_ACCESSOR(sticky_glr)

namespace {

constexpr int kSeg = 8;          // tokens of a warp's run, and between the states that the training forward keeps
constexpr int kWarps = 4;        // runs of a CTA
constexpr int kTile = kSeg * kWarps;
constexpr int kChan = 64;        // channels of a CTA, and of a checkpoint's group
constexpr int kMaxCluster = 8;
constexpr int kSMs = 152;
// CTAs that run at once on an SM: bound by registers, for fp32 rows by shared memory
inline int forward_ctas(int dtype) { return dtype == SDM_DTYPE_F32 ? 3 : 5; }
inline int backward_ctas(int dtype) { return dtype == SDM_DTYPE_F32 ? 2 : 3; }
constexpr uint32_t kWaitPolls = 1u << 20;
static_assert(kChan == ckpt8::kGroup, "a warp's channels are one checkpoint group");

struct GlrArgs {
  const float *state;   // h_0, or dL/dh_T
  float *state_out;     // h_T, or dL/dh_0
  const void *x, *r, *g;
  int64_t ld_x, ld_r, ld_g, ld_d;
  int8_t *codes;
  uint8_t *exps;
  const float *rate;
  const uint8_t *reset;
  const int32_t *lens;
  int B, T, D, S;
  int cs;               // CTAs of a cluster
  int drop;             // test hook: the last CTA of a cluster sends nothing
  void *y;              // or dy
  float *carry;
  void *dx, *dr, *dg;
  float *part;          // [B * cs][D]: drate, summed over the tokens of a CTA
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
__device__ __forceinline__ float root(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// pairs of channels: one instruction for two fp32 operations
__device__ __forceinline__ float2 dup(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float2 sigmoid2(float2 v) {
  const float2 z = mul2(v, dup(-kLog2e));
  const float2 d = add2(make_float2(ex2(z.x), ex2(z.y)), dup(1.f));
  return make_float2(rcp(d.x), rcp(d.y));
}

// The decay and its complement: a = 2^l with l = -rate log2(e) sigmoid(r),
// m2 = 1 - a^2.  Near a = 1 the difference cancels, and the series w (1 - w/2
// (1 - w/3 (... (1 - w/6)))) in w = -2 ln a takes over.  It ends with a
// negative term, so it is never above 1 - a^2, and below it by w^7 / 5040 at
// first.  The difference is taken from 1 - 6e-7 in place of 1, which is more than
// a^2's error (2 * 2^-22, ex2.approx) can make up for, so it is never above
// 1 - a^2 either, and the larger of the two is the right one: off by 2.5e-6 of
// it where they meet (w = 0.45), by less elsewhere.
constexpr float kBelow1 = 0.9999994f;
__device__ __forceinline__ float2 decay(float2 l) { return make_float2(ex2(l.x), ex2(l.y)); }
__device__ __forceinline__ float2 complement(float2 l, float2 a) {
  const float2 w = mul2(l, dup(-2.f * kLn2));
  float2 p = fma2(w, dup(-1.f / 720.f), dup(1.f / 120.f));
  p = fma2(w, p, dup(-1.f / 24.f));
  p = fma2(w, p, dup(1.f / 6.f));
  p = fma2(w, p, dup(-0.5f));
  p = fma2(w, p, dup(1.f));
  p = mul2(w, p);
  return make_float2(fmaxf(p.x, __fmaf_rn(-a.x, a.x, kBelow1)), fmaxf(p.y, __fmaf_rn(-a.y, a.y, kBelow1)));
}
// 1 / sqrt(m2), and 0 where m2 underflows
__device__ __forceinline__ float inv_m(float m2) { return m2 >= 1.17549435e-38f ? rsq(m2) : 0.f; }

__device__ __forceinline__ uint32_t bf16_pair(float2 v) {  // nearest even, v.x in the lower half
  uint32_t u;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u) : "f"(v.y), "f"(v.x));
  return u;
}
// a pair of channels to global memory; `two`: both exist
template <bool VEC>
__device__ __forceinline__ void store2(float *p, float2 v, bool two) {
  if (VEC) {
    *reinterpret_cast<float2 *>(p) = v;
  } else {
    p[0] = v.x;
    if (two) p[1] = v.y;
  }
}
template <bool VEC>
__device__ __forceinline__ void store2(uint16_t *p, float2 v, bool two) {
  const uint32_t u = bf16_pair(v);
  if (VEC) {
    *reinterpret_cast<uint32_t *>(p) = u;
  } else {
    p[0] = static_cast<uint16_t>(u);
    if (two) p[1] = static_cast<uint16_t>(u >> 16);
  }
}

// rate, with a value outside [0, inf) flagged and taken as 0
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

// ---- a warp's tokens in shared memory ----
// Rows of 64 channels of E, token i at i * 64 * sizeof(E).  A warp copies and
// reads its own rows only, so no CTA barrier guards them.
template <class E>
struct Rows {
  static constexpr int kRow = kChan * static_cast<int>(sizeof(E));
  static constexpr int kBytes = kSeg * kRow;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// Start copying tokens [0, n) (n <= 8; rows `ld` elements apart, src at the
// first one's first channel of this warp, `chan` of them in range).  VEC: rows
// are 16-byte aligned, 16 bytes a copy, zeros behind the last channel; else
// element by element.
template <class E, bool VEC>
__device__ __forceinline__ void copy_rows(unsigned char *dst, const E *src, int64_t ld, int n, int chan, int lane) {
  if (VEC) {
    constexpr int kPer = Rows<E>::kRow / 16;
    const uint32_t d = smem_u32(dst) + lane * 16;
    const int j = lane % kPer;
    const int left = chan * static_cast<int>(sizeof(E)) - 16 * j;
    const int bytes = left < 0 ? 0 : left > 16 ? 16 : left;
    const E *s = src + (lane / kPer) * ld + (bytes > 0 ? j * (16 / static_cast<int>(sizeof(E))) : 0);
#pragma unroll
    for (int k = 0; k < kSeg * kPer / 32; ++k)
      if (lane / kPer + k * (32 / kPer) < n) cp16(d + k * 512, s + k * (32 / kPer) * ld, bytes);
  } else {
    const int c = 2 * lane;
    if (sizeof(E) == 4) {
#pragma unroll
      for (int i = 0; i < kSeg; ++i) {
        if (i < n && c < chan) cp_async<4>(dst + i * Rows<E>::kRow + lane * 8, src + i * ld + c);
        if (i < n && c + 1 < chan) cp_async<4>(dst + i * Rows<E>::kRow + lane * 8 + 4, src + i * ld + c + 1);
      }
    } else {
      uint32_t v[kSeg];
#pragma unroll
      for (int i = 0; i < kSeg; ++i) {
        const uint16_t *s = reinterpret_cast<const uint16_t *>(src) + i * ld + c;
        const uint32_t lo = i < n && c < chan ? s[0] : 0, hi = i < n && c + 1 < chan ? s[1] : 0;
        v[i] = lo | hi << 16;
      }
#pragma unroll
      for (int i = 0; i < kSeg; ++i) *reinterpret_cast<uint32_t *>(dst + i * Rows<E>::kRow + lane * 4) = v[i];
    }
  }
}
// the same for checkpoint codes: rows of 64 bytes
template <bool VEC>
__device__ __forceinline__ void copy_codes(unsigned char *dst, const int8_t *src, int64_t ld, int n, int chan, int lane) {
  if (VEC) {  // a row is 4 copies, 8 rows 32: one a lane
    const int i = lane >> 2, j = lane & 3, left = chan - 16 * j;
    const int bytes = left < 0 ? 0 : left > 16 ? 16 : left;
    if (i < n) cp16(smem_u32(dst) + lane * 16, src + i * ld + (bytes > 0 ? 16 * j : 0), bytes);
  } else {
    const int c = 2 * lane;
    uint32_t v[kSeg];
#pragma unroll
    for (int i = 0; i < kSeg; ++i) {
      const uint8_t *s = reinterpret_cast<const uint8_t *>(src) + i * ld + c;
      v[i] = (i < n && c < chan ? s[0] : 0) | (i < n && c + 1 < chan ? s[1] : 0) << 8;
    }
#pragma unroll
    for (int i = 0; i < kSeg; ++i) *reinterpret_cast<uint16_t *>(dst + i * kChan + c) = static_cast<uint16_t>(v[i]);
  }
}
__device__ __forceinline__ float2 row_pair(const unsigned char *rows, int i, int lane, const float *) {
  return *reinterpret_cast<const float2 *>(rows + i * Rows<float>::kRow + lane * 8);
}
__device__ __forceinline__ float2 row_pair(const unsigned char *rows, int i, int lane, const uint16_t *) {
  const uint32_t u = *reinterpret_cast<const uint32_t *>(rows + i * Rows<uint16_t>::kRow + lane * 4);
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

// ---- the composition of runs ----
// A run maps v to P v + H; `cut`: it does not depend on v at all (a reset), not
// even where v is NaN.
struct Run {
  float2 P, H;
  bool cut;
};
template <bool CUTS>
__device__ __forceinline__ float2 apply(const Run &q, float2 v) {
  return CUTS && q.cut ? q.H : fma2(q.P, v, q.H);
}

struct Runs {
  float4 warp[2][kWarps][32];
  float4 cta[2][kMaxCluster][32];
  uint32_t warp_cut[2][kWarps], cta_cut[2][kMaxCluster];
  uint64_t full[2];  // mbarriers: every CTA's run of a step has arrived in cta[half]
};

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory"); }
__device__ __forceinline__ uint32_t in_cta(const void *p, int rank) {
  uint32_t d;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(smem_u32(p)), "r"(rank));
  return d;
}
// asynchronous stores into a CTA of the cluster, counted by its mbarrier
__device__ __forceinline__ void send(uint32_t dst, float4 v, uint32_t mbar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];\n" ::"r"(dst),
               "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(mbar)
               : "memory");
}
__device__ __forceinline__ void send(uint32_t dst, uint32_t v, uint32_t mbar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.u32 [%0], %1, [%2];\n" ::"r"(dst), "r"(v), "r"(mbar)
               : "memory");
}
// false: the phase did not complete within the bound
__device__ __forceinline__ bool wait_runs(uint32_t mbar, uint32_t parity) {
  for (uint32_t i = 0; i < kWaitPolls; ++i) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(done)
        : "r"(mbar), "r"(parity)
        : "memory");
    if (done) return true;
    if (i > 64) __nanosleep(64);
  }
  return false;
}

// Where a warp stands in its cluster, and whether a wait of its gave up.
struct Place {
  int warp, lane, rank, cs;
  bool drop;  // test hook: do not send
  bool lost;
};

// Every warp of the cluster gives its run of a step; returns the value in front
// of this warp's run and moves v (the value in front of the step, the same in every
// warp) behind the step.  Runs follow one another by warp and CTA rank, upwards,
// or (REVERSE) downwards.  k counts the calls: the halves of `s` alternate, so
// that one CTA barrier a step is enough (a half is written again two steps on,
// when every reader has passed the barrier between).  Between CTAs a run travels
// by st.async, which needs no fence and no cluster barrier: a fence would wait
// for the warp's stores to global memory as well.  A CTA sends its run of step k + 2
// once it has every run of step k + 1, each sent after its sender had done with
// step k, so a half in use is not overwritten.  CUTS: runs may be cut.
template <bool REVERSE, bool CUTS>
__device__ __forceinline__ float2 compose(Runs &s, int k, Place &at, const Run &mine, float2 &v) {
  const int half = k & 1, warp = at.warp, lane = at.lane, cs = at.cs;
  s.warp[half][warp][lane] = make_float4(mine.P.x, mine.P.y, mine.H.x, mine.H.y);
  if (CUTS && lane == 0) s.warp_cut[half][warp] = mine.cut;
  if (cs > 1 && threadIdx.x == 0) umma::mbar_expect_tx(smem_u32(&s.full[half]), cs * (CUTS ? 516 : 512));
  __syncthreads();
  auto run = [&](const float4 &q, const uint32_t *cut) {
    return Run{make_float2(q.x, q.y), make_float2(q.z, q.w), CUTS && *cut != 0};
  };
  float2 front;
  if (cs == 1) {
    front = v;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      const int j = REVERSE ? kWarps - 1 - i : i;
      if (j == warp) front = v;
      v = apply<CUTS>(run(s.warp[half][j][lane], &s.warp_cut[half][j]), v);
    }
    return front;
  }
  Run all{dup(1.f), dup(0.f), false}, before = all;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    const int j = REVERSE ? kWarps - 1 - i : i;
    if (j == warp) before = all;
    const Run q = run(s.warp[half][j][lane], &s.warp_cut[half][j]);
    all.H = apply<CUTS>(q, all.H);
    all.P = mul2(all.P, q.P);
    if (CUTS) all.cut |= q.cut;
  }
  if (!at.drop)
    for (int i = warp; i < cs; i += kWarps) {  // the warps share out the CTAs that the run goes to
      const uint32_t mbar = in_cta(&s.full[half], i);
      send(in_cta(&s.cta[half][at.rank][lane], i), make_float4(all.P.x, all.P.y, all.H.x, all.H.y), mbar);
      if (CUTS && lane == 0) send(in_cta(&s.cta_cut[half][at.rank], i), static_cast<uint32_t>(all.cut), mbar);
    }
  if (!at.lost) at.lost = !wait_runs(smem_u32(&s.full[half]), k >> 1 & 1);
  front = v;
  for (int i = 0; i < cs; ++i) {
    const int j = REVERSE ? cs - 1 - i : i;
    if (j == at.rank) front = v;
    v = apply<CUTS>(run(s.cta[half][j][lane], &s.cta_cut[half][j]), v);
  }
  return apply<CUTS>(before, front);
}

// Before the first compose, and at the kernel's end.  A CTA whose waits all
// ended well has received everything that is sent to it and may leave; the
// cluster barrier at the end covers those whose wait gave up.
__device__ __forceinline__ void open_runs(Runs &s, const Place &at) {
  if (at.cs == 1) return;
  if (threadIdx.x == 0) {
    umma::mbar_init(smem_u32(&s.full[0]), 1);
    umma::mbar_init(smem_u32(&s.full[1]), 1);
    umma::fence_mbar_init();
  }
  cluster_arrive();
}
__device__ __forceinline__ void close_runs(const Place &at, int32_t *err) {
  if (at.cs == 1) return;
  if (at.lost) report_timeout(err);
  __syncwarp();
  cluster_arrive();
  cluster_wait();
}

// reset flags of tokens [0, n) as bits; the same in every lane
__device__ __forceinline__ uint32_t reset_bits(const uint8_t *reset, int64_t row, int n, int lane) {
  return __ballot_sync(kFull, lane < n && reset[row + lane] != 0);
}

// ---- forward ----
// K8: also the 8-bit checkpoints of x, r and g.  CUTS: with reset flags.
template <class E, bool VEC, bool K8, bool CUTS>
__global__ void __launch_bounds__(kWarps * 32) glr_forward_kernel(const GlrArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  Runs &runs = *reinterpret_cast<Runs *>(smem);
  constexpr int kStage = 3 * Rows<E>::kBytes;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned char *mine = smem + sizeof(Runs) + warp * 2 * kStage;
  const int cs = a.cs, rank = blockIdx.x % cs, c0 = (blockIdx.x / cs) * kChan, b = blockIdx.y;
  Place at{warp, lane, rank, cs, a.drop && rank == cs - 1, false};
  const int c = c0 + 2 * lane, chan = min(kChan, a.D - c0);
  const bool one = c < a.D, two = c + 1 < a.D;
  open_runs(runs, at);
  const int len = load_len(a, b);
  const int64_t row0 = static_cast<int64_t>(b) * a.T;
  const float2 rate2 = make_float2(one ? -kLog2e * load_rate(a, c) : 0.f, two ? -kLog2e * load_rate(a, c + 1) : 0.f);
  const int64_t sc = static_cast<int64_t>(b) * a.D + c;
  float2 v = make_float2(one ? a.state[sc] : 0.f, two ? a.state[sc + 1] : 0.f);
  const int steps = (len + kTile * cs - 1) / (kTile * cs);
  auto first = [&](int step) { return (step * cs + rank) * kTile + warp * kSeg; };
  auto count = [&](int t0) { return max(0, min(kSeg, len - t0)); };
  auto fetch = [&](int step) {
    const int t0 = first(step), n = step < steps ? count(t0) : 0;
    if (n > 0) {
      unsigned char *d = mine + (step & 1) * kStage;
      copy_rows<E, VEC>(d, static_cast<const E *>(a.x) + (row0 + t0) * a.ld_x + c0, a.ld_x, n, chan, lane);
      copy_rows<E, VEC>(d + Rows<E>::kBytes, static_cast<const E *>(a.r) + (row0 + t0) * a.ld_r + c0, a.ld_r, n, chan, lane);
      copy_rows<E, VEC>(d + 2 * Rows<E>::kBytes, static_cast<const E *>(a.g) + (row0 + t0) * a.ld_g + c0, a.ld_g, n, chan, lane);
    }
    cp_async_commit();
  };
  fetch(0);
  if (cs > 1) cluster_wait();  // every CTA of the cluster runs before one writes into another
  int bad = 0;
  for (int step = 0; step < steps; ++step) {
    fetch(step + 1);
    cp_async_wait<1>();
    __syncwarp();
    const int t0 = first(step), n = count(t0);
    const unsigned char *d = mine + (step & 1) * kStage;
    const uint32_t cut = CUTS ? reset_bits(a.reset, row0 + t0, n, lane) : 0;
    float2 f[kSeg], u[kSeg];
#pragma unroll
    for (int i = 0; i < kSeg; ++i) {
      const float2 x = row_pair(d, i, lane, static_cast<const E *>(nullptr));
      const float2 r = row_pair(d + Rows<E>::kBytes, i, lane, static_cast<const E *>(nullptr));
      const float2 g = row_pair(d + 2 * Rows<E>::kBytes, i, lane, static_cast<const E *>(nullptr));
      const float2 l = mul2(rate2, sigmoid2(r)), sg = sigmoid2(g);
      f[i] = decay(l);
      const float2 m2 = complement(l, f[i]);
      u[i] = mul2(mul2(make_float2(root(m2.x), root(m2.y)), sg), x);
      if (K8 && i < n) {
        const int64_t row = row0 + t0 + i, rows = static_cast<int64_t>(a.B) * a.T;
        const int G = ckpt8::groups(a.D);
        const float2 in[3] = {x, r, g};
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          const uint32_t ux = one ? __float_as_uint(in[k].x) & 0x7fffffffu : 0, uy = two ? __float_as_uint(in[k].y) & 0x7fffffffu : 0;
          const uint32_t byte = ckpt8::exp_byte(__reduce_max_sync(kFull, max(ux, uy)));
          const float inv = ckpt8::inv_step(byte);
          const uint32_t q0 = byte == 255u ? 0 : ckpt8::code_bits(in[k].x, inv), q1 = byte == 255u ? 0 : ckpt8::code_bits(in[k].y, inv);
          int8_t *q = a.codes + (k * rows + row) * a.D + c;
          if (VEC) {
            if (one) *reinterpret_cast<uint16_t *>(q) = static_cast<uint16_t>(__byte_perm(q0, q1, 0x0040));
          } else {
            if (one) q[0] = static_cast<int8_t>(q0);
            if (two) q[1] = static_cast<int8_t>(q1);
          }
          if (lane == 0) a.exps[(k * rows + row) * G + c0 / kChan] = static_cast<uint8_t>(byte);
          bad |= byte == 255u;
        }
      }
    }
    if (n < kSeg) {
#pragma unroll
      for (int i = 0; i < kSeg; ++i)
        if (i >= n) f[i] = dup(1.f), u[i] = dup(0.f);
    }
    Run q{f[0], u[0], cut != 0};
    if (CUTS && cut) {
#pragma unroll
      for (int i = 1; i < kSeg; ++i) q.H = cut >> i & 1 ? u[i] : fma2(f[i], q.H, u[i]);
      q.P = dup(0.f);
    } else {
#pragma unroll
      for (int i = 1; i < kSeg; ++i) q.P = mul2(q.P, f[i]), q.H = fma2(f[i], q.H, u[i]);
    }
    float2 h = compose<false, CUTS>(runs, step, at, q, v);
    if (n > 0 && one) {
      if (a.carry) {
        float *k = a.carry + (static_cast<int64_t>(b) * a.S + t0 / kSeg) * a.D + c;
        store2<VEC>(k, h, two);
      }
      E *y = static_cast<E *>(a.y) + (row0 + t0) * a.D + c;
#pragma unroll
      for (int i = 0; i < kSeg; ++i) {
        h = CUTS && cut >> i & 1 ? u[i] : fma2(f[i], h, u[i]);
        if (i < n) store2<VEC>(y + static_cast<int64_t>(i) * a.D, h, two);
      }
    }
  }
  if (rank == 0 && warp == 0 && one) {
    a.state_out[sc] = v.x;
    if (two) a.state_out[sc + 1] = v.y;
  }
  close_runs(at, a.err);
  if (K8 && bad && lane == 0 && a.err) atomicOr(a.err, SDM_DEVERR_NONFINITE);
}

// ---- backward ----
// The same walk from the last token to the first; what runs through it is
// e_t = a_t dh_t, the gradient that reaches h_{t-1}: dh_t = dy_t + e_{t+1}.
// K8: x, r and g come from their checkpoints.
template <class E, bool VEC, bool K8, bool CUTS>
__global__ void __launch_bounds__(kWarps * 32) glr_backward_kernel(const GlrArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  Runs &runs = *reinterpret_cast<Runs *>(smem);
  using I = typename std::conditional<K8, int8_t, E>::type;  // what x, r and g are held in
  constexpr int kStage = 3 * Rows<I>::kBytes + Rows<E>::kBytes;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned char *mine = smem + sizeof(Runs) + warp * 2 * kStage;
  const int cs = a.cs, rank = blockIdx.x % cs, c0 = (blockIdx.x / cs) * kChan, b = blockIdx.y;
  Place at{warp, lane, rank, cs, a.drop && rank == cs - 1, false};
  const int c = c0 + 2 * lane, chan = min(kChan, a.D - c0);
  const bool one = c < a.D, two = c + 1 < a.D;
  open_runs(runs, at);
  const int len = load_len(a, b);
  const int64_t row0 = static_cast<int64_t>(b) * a.T, rows = static_cast<int64_t>(a.B) * a.T;
  const int G = ckpt8::groups(a.D);
  const float2 rate = make_float2(one ? load_rate(a, c) : 0.f, two ? load_rate(a, c + 1) : 0.f);
  const float2 rate2 = mul2(rate, dup(-kLog2e));
  const int64_t sc = static_cast<int64_t>(b) * a.D + c;
  float2 v = make_float2(one && a.state ? a.state[sc] : 0.f, two && a.state ? a.state[sc + 1] : 0.f);
  float2 drate = dup(0.f);
  const int steps = (len + kTile * cs - 1) / (kTile * cs);
  auto first = [&](int step) { return (step * cs + rank) * kTile + warp * kSeg; };
  auto count = [&](int t0) { return max(0, min(kSeg, len - t0)); };
  auto fetch = [&](int step) {
    const int t0 = first(max(step, 0)), n = step >= 0 ? count(t0) : 0;
    if (n > 0) {
      unsigned char *d = mine + (step & 1) * kStage;
      const int64_t row = row0 + t0;
      if constexpr (K8) {
        for (int k = 0; k < 3; ++k)
          copy_codes<VEC>(d + k * Rows<I>::kBytes, a.codes + (k * rows + row) * a.D + c0, a.D, n, chan, lane);
      } else {
        copy_rows<E, VEC>(d, static_cast<const E *>(a.x) + row * a.ld_x + c0, a.ld_x, n, chan, lane);
        copy_rows<E, VEC>(d + Rows<E>::kBytes, static_cast<const E *>(a.r) + row * a.ld_r + c0, a.ld_r, n, chan, lane);
        copy_rows<E, VEC>(d + 2 * Rows<E>::kBytes, static_cast<const E *>(a.g) + row * a.ld_g + c0, a.ld_g, n, chan, lane);
      }
      copy_rows<E, VEC>(d + 3 * Rows<I>::kBytes, static_cast<const E *>(a.y) + row * a.D + c0, a.D, n, chan, lane);
    }
    cp_async_commit();
  };
  fetch(steps - 1);
  if (cs > 1) cluster_wait();
  for (int step = steps - 1; step >= 0; --step) {
    fetch(step - 1);
    const int t0 = first(step), n = count(t0);
    const uint32_t cut = CUTS ? reset_bits(a.reset, row0 + t0, n, lane) : 0;
    float2 h = dup(0.f);
    uint32_t exps = 0;  // lane 8 k + i: plane k, token i
    if (n > 0) {
      const float *k = a.carry + (static_cast<int64_t>(b) * a.S + t0 / kSeg) * a.D + c;
      if (VEC) {
        if (one) h = *reinterpret_cast<const float2 *>(k);
      } else {
        h = make_float2(one ? k[0] : 0.f, two ? k[1] : 0.f);
      }
      if (K8 && lane < 24 && (lane & 7) < n)
        exps = a.exps[((lane >> 3) * rows + row0 + t0 + (lane & 7)) * G + c0 / kChan];
    }
    cp_async_wait<1>();
    __syncwarp();
    const unsigned char *d = mine + (step & 1) * kStage;
    auto input = [&](int k, int i) {
      if constexpr (K8) {
        const uint16_t q = *reinterpret_cast<const uint16_t *>(d + k * Rows<I>::kBytes + i * kChan + 2 * lane);
        const float s = ckpt8::step(__shfl_sync(kFull, exps, 8 * k + i));
        return mul2(make_float2(static_cast<float>(static_cast<int8_t>(q & 0xff)), static_cast<float>(static_cast<int8_t>(q >> 8))), dup(s));
      } else {
        return row_pair(d + k * Rows<I>::kBytes, i, lane, static_cast<const E *>(nullptr));
      }
    };
    // per token: the decay; what dh is multiplied by in dx and dg; and -sr a
    // (h_{t-1} - (a / m) sg x), by which it is in drate (dr: that times rate (1 - sr))
    float2 f[kSeg], cx[kSeg], cg[kSeg], cr[kSeg], ck[kSeg], dy[kSeg];
#pragma unroll
    for (int i = 0; i < kSeg; ++i) {
      const float2 x = input(0, i), sr = sigmoid2(input(1, i)), sg = sigmoid2(input(2, i));
      dy[i] = row_pair(d + 3 * Rows<I>::kBytes, i, lane, static_cast<const E *>(nullptr));
      const float2 l = mul2(rate2, sr);
      f[i] = decay(l);
      const float2 m2 = complement(l, f[i]);
      const float2 rs = make_float2(inv_m(m2.x), inv_m(m2.y));
      const float2 sx = mul2(sg, x), m = mul2(m2, rs);
      cx[i] = mul2(m, sg);
      const float2 u = mul2(m, sx);
      cg[i] = mul2(u, fma2(sg, dup(-1.f), dup(1.f)));
      if (CUTS && cut >> i & 1) h = dup(0.f);
      const float2 nf = mul2(f[i], dup(-1.f));
      cr[i] = mul2(mul2(sr, nf), fma2(mul2(nf, rs), sx, h));
      ck[i] = mul2(rate, fma2(sr, dup(-1.f), dup(1.f)));
      h = fma2(f[i], h, u);
    }
    if (n < kSeg) {
#pragma unroll
      for (int i = 0; i < kSeg; ++i)
        if (i >= n) f[i] = dup(1.f), dy[i] = dup(0.f);
    }
    Run q{dup(1.f), dup(0.f), cut != 0};
    if (CUTS && cut) {
#pragma unroll
      for (int i = kSeg - 1; i >= 0; --i) q.H = cut >> i & 1 ? dup(0.f) : mul2(f[i], add2(dy[i], q.H));
      q.P = dup(0.f);
    } else {
#pragma unroll
      for (int i = kSeg - 1; i >= 0; --i) q.P = mul2(q.P, f[i]), q.H = mul2(f[i], add2(dy[i], q.H));
    }
    float2 e = compose<true, CUTS>(runs, steps - 1 - step, at, q, v);
    if (n > 0) {
      const int64_t at = (row0 + t0) * a.ld_d + c;
#pragma unroll
      for (int i = kSeg - 1; i >= 0; --i) {
        if (i < n) {
          const float2 dh = add2(dy[i], e);
          const float2 w = mul2(dh, cr[i]);
          drate = add2(drate, w);
          if (one) {
            const int64_t o = at + i * a.ld_d;
            store2<VEC>(static_cast<E *>(a.dx) + o, mul2(dh, cx[i]), two);
            store2<VEC>(static_cast<E *>(a.dr) + o, mul2(w, ck[i]), two);
            store2<VEC>(static_cast<E *>(a.dg) + o, mul2(dh, cg[i]), two);
          }
          e = CUTS && cut >> i & 1 ? dup(0.f) : mul2(f[i], dh);
        }
      }
    }
  }
  if (rank == 0 && warp == 0 && one) {
    a.state_out[sc] = v.x;
    if (two) a.state_out[sc + 1] = v.y;
  }
  // drate over the CTA's warps, in their order
  float2 *sum = reinterpret_cast<float2 *>(smem + sizeof(Runs));
  cp_async_wait<0>();
  __syncthreads();
  sum[warp * 32 + lane] = drate;
  __syncthreads();
  if (warp == 0) {
    for (int i = 1; i < kWarps; ++i) drate = add2(drate, sum[i * 32 + lane]);
    float *p = a.part + (static_cast<int64_t>(b) * cs + rank) * a.D + c;
    if (one) p[0] = drate.x;
    if (two) p[1] = drate.y;
  }
  close_runs(at, a.err);
}

// drate[c] = sum over the parts: 32 interleaved sums, then those in order
__global__ void __launch_bounds__(1024) glr_rate_kernel(const float *part, int parts, int D, float *drate) {
  __shared__ float sum[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  float s = 0.f;
  if (c < D)
    for (int i = threadIdx.y; i < parts; i += 32) s += part[static_cast<int64_t>(i) * D + c];
  sum[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && c < D) {
    for (int i = 1; i < 32; ++i) s += sum[i][threadIdx.x];
    drate[c] = s;
  }
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

// CTAs of a cluster: the split of the sequence that leaves the least to the
// busiest SM, in tiles, as long as the whole grid runs at once.
int cluster_size(int B, int T, int D, int per_sm) {
  const int64_t columns = static_cast<int64_t>(B) * ((D + kChan - 1) / kChan);
  int best = 1;
  int64_t least = INT64_MAX;
  for (int cs = 1; cs <= kMaxCluster; ++cs) {
    if (cs > 1 && (columns * cs > int64_t(kSMs) * per_sm || (cs - 1) * kTile >= T)) break;
    const int64_t load = (columns * cs + kSMs - 1) / kSMs * ((T + kTile * cs - 1) / (kTile * cs));
    if (load < least) least = load, best = cs;
  }
  return best;
}

// 16-byte copies of rows, pairwise stores
bool rows_vec(const void *p, int64_t ld, int es) { return aligned(p, 16) && ld * es % 16 == 0; }
bool pairs_vec(const void *p, int64_t ld, int es) { return aligned(p, 2 * es) && ld % 2 == 0; }

template <class K>
int launch(const char *fn, K kernel, size_t smem, const GlrArgs &a, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return set_error(SDM_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((a.D + kChan - 1) / kChan * a.cs, a.B);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = a.cs, at.val.clusterDim.y = 1, at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = a.cs > 1 ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, kernel, a);
  if (e != cudaSuccess) return set_error(SDM_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
  return check_launch(fn);
}

template <class E, bool VEC>
int launch_forward(const char *fn, const GlrArgs &a, cudaStream_t st) {
  const size_t smem = sizeof(Runs) + kWarps * 2 * 3 * Rows<E>::kBytes;
  if (a.reset)
    return a.codes ? launch(fn, glr_forward_kernel<E, VEC, true, true>, smem, a, st)
                   : launch(fn, glr_forward_kernel<E, VEC, false, true>, smem, a, st);
  return a.codes ? launch(fn, glr_forward_kernel<E, VEC, true, false>, smem, a, st)
                 : launch(fn, glr_forward_kernel<E, VEC, false, false>, smem, a, st);
}
template <class E, bool VEC>
int launch_backward(const char *fn, const GlrArgs &a, cudaStream_t st) {
  const size_t smem = sizeof(Runs) + kWarps * 2 * ((a.codes ? 3 * Rows<int8_t>::kBytes : 3 * Rows<E>::kBytes) + Rows<E>::kBytes);
  if (a.reset)
    return a.codes ? launch(fn, glr_backward_kernel<E, VEC, true, true>, smem, a, st)
                   : launch(fn, glr_backward_kernel<E, VEC, false, true>, smem, a, st);
  return a.codes ? launch(fn, glr_backward_kernel<E, VEC, true, false>, smem, a, st)
                 : launch(fn, glr_backward_kernel<E, VEC, false, false>, smem, a, st);
}

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
  if (codes && !aligned(codes, 16)) return set_error(SDM_ERR_ALIGN, "%s: codes must be 16-byte aligned", fn);
  a.codes = codes, a.exps = exps;
  a.drop = test_drop_signal();
  a.cs = cluster_size(a.B, a.T, a.D, forward_ctas(dtype));
  const int es = dtype == SDM_DTYPE_F32 ? 4 : 2;
  const bool vec = rows_vec(a.x, a.ld_x, es) && rows_vec(a.r, a.ld_r, es) && rows_vec(a.g, a.ld_g, es) &&
                   pairs_vec(a.y, a.D, es) && (!a.carry || aligned(a.carry, 8));
  if (dtype == SDM_DTYPE_F32)
    return vec ? launch_forward<float, true>(fn, a, st) : launch_forward<float, false>(fn, a, st);
  return vec ? launch_forward<uint16_t, true>(fn, a, st) : launch_forward<uint16_t, false>(fn, a, st);
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
  return (sizeof(float) * B * kMaxCluster * static_cast<size_t>(D) + 255) / 256 * 256;
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
    if (codes && !aligned(codes, 16)) return set_error(SDM_ERR_ALIGN, "%s: codes must be 16-byte aligned", fn);
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
  a.codes = const_cast<int8_t *>(codes), a.exps = const_cast<uint8_t *>(exps), a.rate = rate, a.reset = reset, a.lens = lens;
  a.B = B, a.T = T, a.D = D, a.S = (T + kSeg - 1) / kSeg;
  a.y = const_cast<void *>(dy), a.carry = const_cast<float *>(carry);
  a.dx = dx, a.dr = dr, a.dg = dg, a.part = static_cast<float *>(workspace), a.err = dev_err;
  a.drop = test_drop_signal();
  a.cs = cluster_size(B, T, D, backward_ctas(dtype));
  if (B > 0) {
    const int es = dtype == SDM_DTYPE_F32 ? 4 : 2;
    const bool in = codes ? D % 16 == 0 : rows_vec(x, ld_x, es) && rows_vec(r, ld_r, es) && rows_vec(g, ld_g, es);
    const bool vec = in && rows_vec(dy, D, es) && pairs_vec(dx, ld_d, es) && pairs_vec(dr, ld_d, es) &&
                     pairs_vec(dg, ld_d, es) && aligned(carry, 8);
    if (dtype == SDM_DTYPE_F32)
      rc = vec ? launch_backward<float, true>(fn, a, st) : launch_backward<float, false>(fn, a, st);
    else
      rc = vec ? launch_backward<uint16_t, true>(fn, a, st) : launch_backward<uint16_t, false>(fn, a, st);
    if (rc) return rc;
  }
  glr_rate_kernel<<<(D + 31) / 32, dim3(32, 32), 0, st>>>(a.part, B * a.cs, D, drate);
  return check_launch(fn);
}
