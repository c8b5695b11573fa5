// glr_scan.cu - gated linear recurrence with one state per channel, its
// training forward and its backward pass (glr_scan in sdm.h):
//   L_t = -rate sigmoid(r_t), a_t = e^{L_t}, m_t = sqrt(1 - a_t^2),
//   h_t = a_t h_{t-1} + m_t sigmoid(g_t) x_t.
//
// A run of tokens acts on the state before it as h -> P h + H (P the product
// of its decays, H what it leaves when it starts from 0), and runs compose:
// that splits the sequence.  A warp owns 64 channels (a pair per lane) of a run
// of 16 tokens (8 in the backward): it forms the run's (P, H), takes the state in
// front of it from the runs before, and steps its tokens through once more with
// the gates still in registers.  Four warps make a CTA, up to sixteen CTAs a
// cluster (runs travel through distributed shared memory), and the cluster
// walks the sequence.  Every input is read once and every output written once,
// no CTA waits for another outside its cluster, and the order of every sum is
// fixed by the sizes.
//
// What bounds it (8 x 4096 x 1920 in bf16, one GB300): the forward moves 8 bytes an
// element and takes 110.6 us, 67% of the measured copy bandwidth; its walk over
// memory alone takes 84 us.  A pair of channels costs 77 instructions, ten of them
// special functions, and 128 registers a thread leave four warps to an SM's
// scheduler, which issues in 63% of the cycles: latency between dependent
// instructions and in the exchange of runs, not memory, is what is left.  Runs of 8
// tokens in 96 registers have more warps, but exchange twice as often: 108.5 us
// where runs of 16 took 106.5, and 304 in place of 215 for one sequence of 32768 x
// 3840.  The backward (14.5 bytes) takes 206 us (65%) for the same reason, at 1.8
// times the instructions.
#include <initializer_list>
#include <type_traits>

#include "ckpt8.cuh"
#include "umma.cuh"

namespace sdm {

int test_drop_signal();  // gdn_chunk.cu: the SDM_TEST_DROP_SIGNAL test hook
SDM_STICKY_ACCESSOR(sticky_glr)

namespace {

constexpr int kSeg = 8;          // tokens between the states that the training forward keeps
constexpr int kForwardRun = 16;  // tokens of a warp's run
constexpr int kBackwardRun = kSeg;
constexpr int kChan = 64;        // channels of a CTA, and of a checkpoint's group
constexpr int kWarps = 4;        // of a CTA
constexpr int kMaxCluster = 16;
constexpr int kSMs = 152;
constexpr int kSteps = 128;      // bytes of a warp's 24 checkpoint steps, and what keeps its rows on 128
constexpr int kForwardRegs = 128, kBackwardRegs = 128;  // of a thread
constexpr uint32_t kWaitPolls = 1u << 18;  // of a cluster's mbarrier, about 1 s, before the wait gives up
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
// pairs of channels: one instruction for two fp32 operations
__device__ __forceinline__ float2 dup(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return fma2(b, dup(-1.f), a); }

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float2 sigmoid2(float2 v) {
  const float2 z = mul2(v, dup(-kLog2e));
  const float2 d = add2(make_float2(ex2(z.x), ex2(z.y)), dup(1.f));
  return make_float2(rcp(d.x), rcp(d.y));
}

// The decay a = e^-y, y = rate sigmoid(r), and e = 1 - a, of which m^2 = 1 - a^2 =
// e (2 - e) is made.  Near a = 1 the exponential unit cannot give e (the difference
// cancels, and its results near 1 are cut off, not rounded: a bias of 2^-25, which a
// horizon of 1 / e tokens multiplies; sums of gradients lost a digit to it).
// So up to y = 0.15, e = y q(y) with q the cubic next to (1 - e^-y) / y there (by
// linear programming, q(0) = 1): off by 5e-8 at most, and a = 1 - e.  Beyond, horizons
// are of a few tokens and the unit's bias counts for little; a is its result itself,
// which keeps a's relative precision however small a is: dr and drate are
// proportional to it, and so is y where a token has no input.
struct Decay {
  float2 a, e;
};
__device__ __forceinline__ Decay decay(float2 y) {
  const float2 l = mul2(y, dup(-kLog2e));
  const float2 far = make_float2(ex2(l.x), ex2(l.y)), rest = fma2(far, dup(-1.f), dup(1.f));
  float2 q = fma2(y, dup(-0.0393375196f), dup(0.166465417f));
  q = fma2(y, q, dup(-0.499995023f));
  q = fma2(y, q, dup(1.f));
  q = mul2(y, q);
  const float2 near = fma2(q, dup(-1.f), dup(1.f));
  const bool x = y.x <= 0.15f, z = y.y <= 0.15f;
  return Decay{make_float2(x ? near.x : far.x, z ? near.y : far.y), make_float2(x ? q.x : rest.x, z ? q.y : rest.y)};
}
// 1 / sqrt(m2), and 0 where m2 underflows
__device__ __forceinline__ float inv_m(float m2) { return m2 >= 1.17549435e-38f ? rsq(m2) : 0.f; }
__device__ __forceinline__ float at_most(float v, float top) {  // NaN stays NaN
  float m;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(v), "f"(top));
  return m;
}
// m sigmoid(g) x with one special function less than its factors take: sigmoid(g)
// = w / d with w = e^g and d = 1 + w, and m / d = m2 / sqrt(d^2 m2).  From g = 26 on
// sigmoid(g) is 1 in fp32, so g is stopped there and d^2 stays in range; a small w
// keeps its digits down to e^-87.  d comes times 2^6 and m2 times 2^12, which keeps
// the root's digits down to m2 = 2^-126; the number added under it keeps its inverse
// finite at m2 = 0.  x comes last: nothing but the term itself overflows.  (With
// 1 / d from e^-g, two instructions less a pair of channels, the term was 0 from g =
// -44 on: 8 x 4096 x 1920 took 107.3 us in place of 110.6.)
__device__ __forceinline__ float2 input_term(float2 e, float2 g, float2 x) {
  const float2 z = mul2(make_float2(at_most(g.x, 26.f), at_most(g.y, 26.f)), dup(kLog2e));
  const float2 w = make_float2(ex2(z.x), ex2(z.y)), d = fma2(w, dup(64.f), dup(64.f));
  const float2 m2 = mul2(e, fma2(e, dup(-4096.f), dup(8192.f)));
  const float2 q = fma2(mul2(d, d), m2, dup(1.17549435e-38f));
  return mul2(mul2(mul2(w, m2), make_float2(rsq(q.x), rsq(q.y))), x);
}

__device__ __forceinline__ uint32_t bf16_pair(float2 v) {  // nearest even, v.x in the lower half
  uint32_t u;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u) : "f"(v.y), "f"(v.x));
  return u;
}
// A pair of channels to global memory, `at` bytes behind a row that is the same
// for the whole warp (an address in two parts costs no 64-bit arithmetic per
// lane); `two`: both channels exist.
template <bool VEC>
__device__ __forceinline__ void store2(float *row, uint32_t at, float2 v, bool two) {
  float *p = reinterpret_cast<float *>(reinterpret_cast<char *>(row) + at);
  if (VEC) {
    *reinterpret_cast<float2 *>(p) = v;
  } else {
    p[0] = v.x;
    if (two) p[1] = v.y;
  }
}
template <bool VEC>
__device__ __forceinline__ void store2(uint16_t *row, uint32_t at, float2 v, bool two) {
  uint16_t *p = reinterpret_cast<uint16_t *>(reinterpret_cast<char *>(row) + at);
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
// 8 rows of 64 channels of I (an activation type, or int8 codes).  A warp
// copies and reads its own rows only, so no CTA barrier guards them.  VEC: rows
// are 16-byte aligned in global memory and dense here.  Else they are copied by the
// aligned 16 bytes that hold them, one piece more than they fill.
template <class I, bool VEC>
struct Rows {
  static constexpr int kRow = kChan * static_cast<int>(sizeof(I)) + (VEC ? 0 : 16);
  static constexpr int kBytes = kSeg * kRow;
  static_assert(kBytes % 128 == 0, "the next rows begin on 128 bytes");
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// A walk over one [tokens, channels] tensor: a warp copies 8 rows at a time and
// moves on by multiples of 16 bytes, so a row's place in its first piece depends
// on its place among the 8 only.  VEC: zeros behind the last channel.
template <class I, bool VEC>
struct Walk {
  static constexpr int kEs = static_cast<int>(sizeof(I)), kRow = Rows<I, VEC>::kRow;
  static constexpr int kPer = kChan * kEs / 16;  // pieces a row
  static constexpr int kRows = 32 / kPer;        // rows a copy of the warp
  static_assert(kSeg % kRows == 0, "a copy of the warp holds whole rows of a run");
  const char *p;   // the first row's first channel of the warp, the same in every lane
  uint32_t row;    // bytes between rows
  uint32_t at;     // this lane's part of a copy, behind p
  int row0, part;  // its row of a copy, and where its piece lies in that row
  int left;        // VEC: its piece's bytes; else the warp's channels

  // `chan` channels exist
  __device__ __forceinline__ Walk(const I *first, int64_t ld, int chan, int lane) {
    row = static_cast<uint32_t>(ld) * kEs;
    p = reinterpret_cast<const char *>(first);
    row0 = lane / kPer, part = 16 * (lane % kPer), left = chan;
    if (VEC) left = max(0, min(16, chan * kEs - part));
    at = row0 * row + (VEC && left == 0 ? 0 : part);
  }
  // how far behind a 16-byte boundary row i begins
  __device__ __forceinline__ uint32_t offset(int i) const {
    return (static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) + i * row) & 15u;
  }
  // start copying rows [0, n)
  __device__ __forceinline__ void copy(unsigned char *dst, int n, int lane) const {
    if constexpr (VEC) {
      const uint32_t d = smem_u32(dst) + lane * 16;
      if (n == kSeg) {
#pragma unroll
        for (int k = 0; k < kSeg / kRows; ++k) cp16(d + k * 512, p + (at + k * kRows * row), left);
      } else {
#pragma unroll
        for (int k = 0; k < kSeg / kRows; ++k)
          if (row0 + k * kRows < n) cp16(d + k * 512, p + (at + k * kRows * row), left);
      }
    } else {
      // only pieces that hold a byte of the row: allocations begin on 16 bytes and
      // more, so such a piece never reaches into unmapped memory
      auto piece = [&](int i, int behind, const char *q) {
        const uint32_t o = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(q)) & 15u;
        if (i < n && behind < static_cast<int>(o) + left * kEs) cp16(smem_u32(dst) + i * kRow + behind, q - o, 16);
      };
#pragma unroll
      for (int k = 0; k < kSeg / kRows; ++k) piece(row0 + k * kRows, part, p + (at + k * kRows * row));
      if (lane < kSeg) piece(lane, 16 * kPer, p + (lane * row + 16 * kPer));
    }
  }
  __device__ __forceinline__ void move(int rows) { p += static_cast<int64_t>(rows) * row; }

  // the lane's channel pair of row i: its bits (16- and 8-bit I); zeros where channels do not exist
  __device__ __forceinline__ uint32_t bits(const unsigned char *rows, int i, int lane) const {
    if constexpr (VEC) {
      if constexpr (kEs == 2) return *reinterpret_cast<const uint32_t *>(rows + i * kRow + lane * 4);
      else return *reinterpret_cast<const uint16_t *>(rows + i * kRow + lane * 2);
    } else {
      const uint32_t o = offset(i) + 2 * kEs * lane;
      const uint32_t *w = reinterpret_cast<const uint32_t *>(rows + i * kRow) + o / 4;
      const uint32_t v = __funnelshift_r(w[0], w[1], 8 * (o & 3u));
      return 2 * lane >= left ? 0u : 2 * lane + 1 >= left ? v & ((1u << (8 * kEs)) - 1u) : v;
    }
  }
  // the pair's values (activations); fp32 off 16 bytes: zeros where channels do
  // not exist only if ZEROS (else their lanes take along what nobody stores: 2 of 37 us)
  template <bool ZEROS = false>
  __device__ __forceinline__ float2 pair(const unsigned char *rows, int i, int lane) const {
    if constexpr (kEs == 4) {
      if constexpr (VEC) {
        return *reinterpret_cast<const float2 *>(rows + i * kRow + lane * 8);
      } else {
        const float *v = reinterpret_cast<const float *>(rows + i * kRow + offset(i)) + 2 * lane;
        return make_float2(!ZEROS || 2 * lane < left ? v[0] : 0.f, !ZEROS || 2 * lane + 1 < left ? v[1] : 0.f);
      }
    } else {
      const uint32_t u = bits(rows, i, lane);
      return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    }
  }
};

// ---- the composition of runs ----
// A run maps v to P v + H.  A run with a reset does not depend on v at all, not
// even where v is NaN: its P is -0, which no product of decays is.  (A flag of its
// own beside P and H, stored, sent and tested apart, held the exchange up: the backward of
// 2 x 8192 x 3840 took 285 us with it in place of 232.)
struct Run {
  float2 P, H;
};
constexpr float kCut = -0.f;
__device__ __forceinline__ bool is_cut(const Run &q) { return __float_as_uint(q.P.x) == 0x80000000u; }
template <bool CUTS>
__device__ __forceinline__ float2 apply(const Run &q, float2 v) {
  const float2 w = fma2(q.P, v, q.H);
  if (!CUTS) return w;
  return is_cut(q) ? q.H : w;
}
// p after q
template <bool CUTS>
__device__ __forceinline__ Run join(const Run &q, const Run &p) {
  Run r{mul2(q.P, p.P), apply<CUTS>(p, q.H)};
  if (CUTS && (is_cut(q) || is_cut(p))) r.P = dup(kCut);
  return r;
}

// In front of a CTA's shared memory; then the warps' rows; then, in a cluster, the CTAs' runs.
// (Rows that begin on 128 bytes are copied faster: the forward of 8 x 4096 x 1920 took
// 111 us at 16 behind a multiple, 108.5 at 32 or 64, 106.5 at 0; fp32, 4 x 4096 x 1920:
// 100, 94 and 90.)
struct alignas(128) Runs {
  float4 warp[2][kWarps][32];
  uint64_t full[2];  // mbarriers: every CTA's run of a step has arrived in its half of the CTAs' runs
};
__host__ __device__ constexpr uint32_t cluster_bytes(int cs) { return cs > 1 ? cs * 1024u : 0u; }

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

// Where a warp stands: its place among the CTA's runs of a step and the CTA's
// place among the cluster's, both in the order in which runs follow one another.
struct Place {
  int warp, lane, rank, cs;
  bool drop;  // test hook: do not send
  bool lost;  // a wait gave up
};

// Every warp of the cluster gives its run of a step; returns the value in front
// of this warp's run and moves v (the value in front of the step, the same in every
// warp) behind the step.  k counts the calls: the halves of `s` alternate, so
// that one CTA barrier a step is enough (a half is written again two steps on,
// when every reader has passed the barrier between).  Between CTAs a run travels
// by st.async, which needs no fence and no cluster barrier: a fence would wait
// for the warp's stores to global memory as well.  A CTA sends its run of step k + 2
// once it has every run of step k + 1, each sent after its sender had done with
// step k, so a half in use is not overwritten.  A wait that gives up is the
// thread's last: an mbarrier whose phase is still open takes no second arrival
// (that faults), so nothing is armed, sent or waited for any more, and the walk
// ends on whatever the buffers hold.  CUTS: runs may be cut.
// kAt: where the CTAs' runs lie behind s.
template <bool CUTS, int kAt>
__device__ __forceinline__ float2 compose(Runs &s, int k, Place &at, const Run &mine, float2 &v) {
  const int half = k & 1, lane = at.lane, cs = at.cs;
  auto slot = [&](int j) { return reinterpret_cast<float4 *>(reinterpret_cast<char *>(&s) + kAt) + (2 * j + half) * 32 + lane; };
  s.warp[half][at.warp][lane] = make_float4(mine.P.x, mine.P.y, mine.H.x, mine.H.y);
  if (cs > 1 && threadIdx.x == 0 && !at.lost) umma::mbar_expect_tx(smem_u32(&s.full[half]), cs * 512);
  __syncthreads();
  auto warp_run = [&](int j) {
    const float4 q = s.warp[half][j][lane];
    return Run{make_float2(q.x, q.y), make_float2(q.z, q.w)};
  };
  auto cta_run = [&](int j) {
    const float4 q = *slot(j);
    return Run{make_float2(q.x, q.y), make_float2(q.z, q.w)};
  };
  if (cs == 1) {
#pragma unroll 4
    for (int j = 0; j < at.warp; ++j) v = apply<CUTS>(warp_run(j), v);
    const float2 front = v;
    v = apply<CUTS>(mine, v);
#pragma unroll 4
    for (int j = at.warp + 1; j < kWarps; ++j) v = apply<CUTS>(warp_run(j), v);
    return front;
  }
  Run before{dup(1.f), dup(0.f)};
#pragma unroll 4
  for (int j = 0; j < at.warp; ++j) before = join<CUTS>(before, warp_run(j));
  if (at.warp == kWarps - 1 && !at.drop && !at.lost) {  // the last warp knows the CTA's run
    const Run q = join<CUTS>(before, mine);
    for (int i = 0; i < cs; ++i)
      send(in_cta(slot(at.rank), i), make_float4(q.P.x, q.P.y, q.H.x, q.H.y), in_cta(&s.full[half], i));
  }
  if (!at.lost) at.lost = !wait_runs(smem_u32(&s.full[half]), k >> 1 & 1);
#pragma unroll 4
  for (int j = 0; j < at.rank; ++j) v = apply<CUTS>(cta_run(j), v);
  const float2 front = v;
#pragma unroll 4
  for (int j = at.rank; j < cs; ++j) v = apply<CUTS>(cta_run(j), v);
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
  __syncwarp();  // the barrier is for whole warps (.aligned)
  cluster_arrive();
}
__device__ __forceinline__ void close_runs(const Place &at, int32_t *err) {
  if (at.cs == 1) return;
  if (at.lost) report_timeout(err);
  __syncwarp();
  cluster_arrive();
  cluster_wait();
}

// lane i < n: token i's reset flag (loaded a step before it is needed)
__device__ __forceinline__ uint32_t reset_flag(const uint8_t *reset, int64_t row, int n, int lane) {
  return lane < n ? reset[row + lane] : 0;
}

// The larger magnitude's bits of a pair; a NaN's are above every number's.
__device__ __forceinline__ uint32_t max_magnitude(float2 v) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(fabsf(v.x)), "f"(fabsf(v.y)));
  return __float_as_uint(m);
}

// The checkpoint of 8 tokens from shared memory to global memory: token i's
// codes are the first 64 bytes of its row in each of the three tensors' rows; lane
// 8 k + i holds the largest magnitude's bits of token i in tensor k.  VEC: 16
// bytes a lane.  Groups with a value that has no code get zeros and 255; returns
// whether there are any.
template <class E, bool VEC>
__device__ __forceinline__ bool put_codes(const GlrArgs &a, unsigned char *q, uint32_t big, int64_t row, int n, int c0,
                                          int chan, int lane) {
  const int64_t rows = static_cast<int64_t>(a.B) * a.T;
  __syncwarp();
  const int k = lane >> 3, i = lane & 7;
  const bool mine = lane < 24 && i < n;
  const uint32_t all = __ballot_sync(kFull, mine && big > ckpt8::kTop);
  for (uint32_t bad = all; bad; bad &= bad - 1) {
    const int j = __ffs(bad) - 1;
    *reinterpret_cast<uint16_t *>(q + (j >> 3) * Rows<E, VEC>::kBytes + (j & 7) * Rows<E, VEC>::kRow + 2 * lane) = 0;
    __syncwarp();
  }
  if (mine) a.exps[(k * rows + row + i) * ckpt8::groups(a.D) + c0 / kChan] = static_cast<uint8_t>(ckpt8::exp_byte(big));
  if (VEC && a.D % 16 == 0) {
    const int j = lane >> 2, at = 16 * (lane & 3);
    if (j < n && at < chan) {
#pragma unroll
      for (int p = 0; p < 3; ++p)
        *reinterpret_cast<int4 *>(a.codes + (p * rows + row + j) * a.D + c0 + at) =
            *reinterpret_cast<const int4 *>(q + p * Rows<E, VEC>::kBytes + j * Rows<E, VEC>::kRow + at);
    }
  } else {
    for (int p = 0; p < 3; ++p)
      for (int j = 0; j < n; ++j) {
        int8_t *o = a.codes + (p * rows + row + j) * a.D + c0;
        const unsigned char *s = q + p * Rows<E, VEC>::kBytes + j * Rows<E, VEC>::kRow;
        if (2 * lane < chan) o[2 * lane] = static_cast<int8_t>(s[2 * lane]);
        if (2 * lane + 1 < chan) o[2 * lane + 1] = static_cast<int8_t>(s[2 * lane + 1]);
      }
  }
  return all != 0;
}

// ---- forward ----
// K8: also the 8-bit checkpoints of x, r and g.  CUTS: with reset flags.
// 8 x 4096 x 1920 in bf16: 110.6 us (67% of the measured copy bandwidth); with the
// carry 112; with checkpoints as well 185 (11.55 bytes an element, 58%: their
// maxima, codes and exponents are three quarters more instructions).  1 x 32768 x 3840,
// one sequence over clusters of 9: 223 us (67%); 2 x 8192 x 3840 with resets: 119
// (62%); fp32, 4 x 4096 x 1920: 91.6 (81%).
template <class E, bool VEC, bool K8, bool CUTS>
__global__ void __maxnreg__(kForwardRegs) glr_forward_kernel(const GlrArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  Runs &runs = *reinterpret_cast<Runs *>(smem);
  constexpr int kBytes = Rows<E, VEC>::kBytes, kHalf = 3 * kBytes, kHalves = kForwardRun / kSeg;
  const int lane = threadIdx.x & 31, warp = __shfl_sync(kFull, threadIdx.x >> 5, 0);
  const int cs = a.cs;
  unsigned char *mine = smem + sizeof(Runs) + warp * kHalves * kHalf;
  const int rank = blockIdx.x % cs, c0 = (blockIdx.x / cs) * kChan, b = blockIdx.y;
  const int c = c0 + 2 * lane, chan = min(kChan, a.D - c0);
  const bool one = c < a.D, two = c + 1 < a.D;
  Place at{warp, lane, rank, cs, a.drop && rank == cs - 1, false};
  const int len = load_len(a, b);
  const float2 rate = make_float2(one ? load_rate(a, c) : 0.f, two ? load_rate(a, c + 1) : 0.f);
  const int64_t sc = static_cast<int64_t>(b) * a.D + c;
  float2 v = make_float2(one ? a.state[sc] : 0.f, two ? a.state[sc + 1] : 0.f);
  open_runs(runs, at);  // behind the state's loads: another CTA may write it in place
  const int tile = kForwardRun * kWarps, tokens = tile * cs;  // tokens of a CTA and of the cluster in a step
  const int steps = (len + tokens - 1) / tokens;
  int t0 = rank * tile + warp * kForwardRun;  // first token of the run
  const int64_t first = static_cast<int64_t>(b) * a.T + t0;
  Walk<E, VEC> wx(static_cast<const E *>(a.x) + first * a.ld_x + c0, a.ld_x, chan, lane);
  Walk<E, VEC> wr(static_cast<const E *>(a.r) + first * a.ld_r + c0, a.ld_r, chan, lane);
  Walk<E, VEC> wg(static_cast<const E *>(a.g) + first * a.ld_g + c0, a.ld_g, chan, lane);
  E *y = static_cast<E *>(a.y) + first * a.D + c0;
  float *carry = a.carry ? a.carry + (static_cast<int64_t>(b) * a.S + t0 / kSeg) * a.D + c0 : nullptr;
  const uint32_t row_bytes = a.D * static_cast<uint32_t>(sizeof(E));
  // the rows of the run's first or second 8 tokens, t the first of them
  auto fetch = [&](int half, int t) {
    const int n = min(kSeg, len - t), on = half == kHalves - 1 ? tokens - kForwardRun + kSeg : kSeg;
    if (n > 0) {
      unsigned char *d = mine + half * kHalf;
      wx.copy(d, n, lane);
      wr.copy(d + kBytes, n, lane);
      wg.copy(d + 2 * kBytes, n, lane);
      wx.move(on), wr.move(on), wg.move(on);
    }
    cp_async_commit();
  };
  for (int half = 0; half < kHalves; ++half) fetch(half, t0 + kSeg * half);
  if (cs > 1) cluster_wait();  // every CTA of the cluster runs before one writes into another
  bool bad = false;            // K8: a group without codes
  const uint8_t *flags = CUTS ? a.reset + static_cast<int64_t>(b) * a.T : nullptr;
  uint32_t flag = CUTS ? reset_flag(flags, t0, min(kForwardRun, len - t0), lane) : 0;
  for (int step = 0; step < steps; ++step, t0 += tokens) {
    const int n = max(0, min(kForwardRun, len - t0));
    const uint32_t cut = CUTS ? __ballot_sync(kFull, flag != 0) : 0;
    if (CUTS) flag = reset_flag(flags, t0 + tokens, min(kForwardRun, len - t0 - tokens), lane);
    float2 f[kForwardRun], u[kForwardRun];
#pragma unroll
    for (int half = 0; half < kHalves; ++half) {
      cp_async_wait<kHalves - 1>();
      __syncwarp();
      unsigned char *d = mine + half * kHalf;
      uint32_t kept = 0;  // K8, lane 8 k + i: the largest magnitude's bits of token i in tensor k
#pragma unroll
      for (int i = 0; i < kSeg; ++i) {
        const float2 x = wx.template pair<K8>(d, i, lane), r = wr.template pair<K8>(d + kBytes, i, lane);
        const float2 g = wg.template pair<K8>(d + 2 * kBytes, i, lane);
        const Decay q = decay(mul2(rate, sigmoid2(r)));
        f[kSeg * half + i] = q.a;
        u[kSeg * half + i] = input_term(q.e, g, x);
        if (K8) {
          // a code goes where the token's inputs were: every lane's are in the maximum below, so they have been read
          const float2 in[3] = {x, r, g};
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            const uint32_t big = __reduce_max_sync(kFull, max_magnitude(in[k]));
            const uint32_t step8 = ckpt8::step_bits(big);
            const float2 code = fma2(in[k], dup(__uint_as_float((254u << 23) - step8)), dup(12582912.f));
            *reinterpret_cast<uint16_t *>(d + k * kBytes + i * Rows<E, VEC>::kRow + 2 * lane) =
                static_cast<uint16_t>(__byte_perm(__float_as_uint(code.x), __float_as_uint(code.y), 0x0040));
            if (lane == 8 * k + i) kept = big;
          }
        }
      }
      if (K8 && n > kSeg * half)
        bad |= put_codes<E, VEC>(a, d, kept, static_cast<int64_t>(b) * a.T + t0 + kSeg * half,
                          min(kSeg, n - kSeg * half), c0, chan, lane);
      __syncwarp();  // the copies go where these rows were read
      fetch(half, t0 + tokens + kSeg * half);
    }
    if (n < kForwardRun) {
#pragma unroll
      for (int i = 0; i < kForwardRun; ++i)
        if (i >= n) f[i] = dup(1.f), u[i] = dup(0.f);
    }
    Run q{f[0], u[0]};
    if (CUTS && cut) {
#pragma unroll
      for (int i = 1; i < kForwardRun; ++i) q.H = cut >> i & 1 ? u[i] : fma2(f[i], q.H, u[i]);
      q.P = dup(kCut);
    } else {
#pragma unroll
      for (int i = 1; i < kForwardRun; ++i) q.P = mul2(q.P, f[i]), q.H = fma2(f[i], q.H, u[i]);
    }
    float2 h = compose<CUTS, sizeof(Runs) + kWarps * kHalves * kHalf>(runs, step, at, q, v);
    if (n > 0 && one) {
      uint32_t o = 2 * lane * static_cast<uint32_t>(sizeof(E));
#pragma unroll
      for (int i = 0; i < kForwardRun; ++i, o += row_bytes) {
        if (i % kSeg == 0 && i < n && carry) store2<VEC>(carry + (i ? a.D : 0), 8u * lane, h, two);
        h = CUTS && cut >> i & 1 ? u[i] : fma2(f[i], h, u[i]);
        if (i < n) store2<VEC>(y, o, h, two);
      }
      if (t0 + n == len) {  // the last token's state, as y has it
        a.state_out[sc] = h.x;
        if (two) a.state_out[sc + 1] = h.y;
      }
    }
    y += static_cast<int64_t>(tokens) * a.D;
    if (carry) carry += static_cast<int64_t>(tokens / kSeg) * a.D;
  }
  if (len == 0 && rank == 0 && warp == 0 && one) {
    a.state_out[sc] = v.x;
    if (two) a.state_out[sc + 1] = v.y;
  }
  close_runs(at, a.err);
  if (K8 && bad && lane == 0 && a.err) atomicOr(a.err, SDM_DEVERR_NONFINITE);
}

// ---- a few tokens: decoding steps ----
// N channels of one sequence a thread (N = 16 bytes of E, or 1 where rows are
// not aligned to that), its tokens in order; the same operations as above, so the
// same bits.  Bound by the launch and latency of one load after another: 6 us for a
// sequence of 1920 channels, 9 for 256 of 3840 (10 MB with the states, which takes 2).
template <class E, int N>
struct alignas(sizeof(E) * N) Pack {
  E v[N];
};
__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(uint16_t v) { return bf16_to_f32(v); }
__device__ __forceinline__ void narrow(float &o, float v) { o = v; }
__device__ __forceinline__ void narrow(uint16_t &o, float v) { o = static_cast<uint16_t>(bf16_pair(make_float2(v, 0.f))); }

template <class E, int N>
__global__ void __launch_bounds__(128) glr_step_kernel(const GlrArgs a) {
  const int per = a.D / N;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x;
  if (i >= static_cast<int64_t>(a.B) * per) return;
  const int b = static_cast<int>(i / per), c = static_cast<int>(i - static_cast<int64_t>(b) * per) * N;
  const int len = load_len(a, b);
  const int64_t sc = static_cast<int64_t>(b) * a.D + c;
  using P = Pack<E, N>;
  using S = Pack<float, N < 4 ? N : 4>;
  constexpr int kS = N < 4 ? N : 4;
  float h[N], rate[N];
#pragma unroll
  for (int j = 0; j < N; j += kS) {
    const S s = *reinterpret_cast<const S *>(a.state + sc + j), q = *reinterpret_cast<const S *>(a.rate + c + j);
#pragma unroll
    for (int l = 0; l < kS; ++l) h[j + l] = s.v[l], rate[j + l] = q.v[l];
  }
  bool bad = false;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const bool ok = rate[j] >= 0.f && rate[j] < __int_as_float(0x7f800000);
    bad |= !ok;
    rate[j] = ok ? rate[j] : 0.f;
  }
  if (bad && a.err) atomicOr(a.err, SDM_DEVERR_RATE);
  const int64_t row0 = static_cast<int64_t>(b) * a.T;
  for (int t = 0; t < len; ++t) {
    const int64_t row = row0 + t;
    const P x = *reinterpret_cast<const P *>(static_cast<const E *>(a.x) + row * a.ld_x + c);
    const P r = *reinterpret_cast<const P *>(static_cast<const E *>(a.r) + row * a.ld_r + c);
    const P g = *reinterpret_cast<const P *>(static_cast<const E *>(a.g) + row * a.ld_g + c);
    const bool cut = a.reset && a.reset[row] != 0;
    P y;
#pragma unroll
    for (int j = 0; j < N; j += 2) {
      const int k = N > 1 ? j + 1 : j;
      const float2 sr = sigmoid2(make_float2(widen(r.v[j]), widen(r.v[k])));
      const Decay q = decay(mul2(make_float2(rate[j], rate[k]), sr));
      const float2 u = input_term(q.e, make_float2(widen(g.v[j]), widen(g.v[k])),
                                  make_float2(widen(x.v[j]), widen(x.v[k])));
      const float2 n = cut ? u : fma2(q.a, make_float2(h[j], h[k]), u);
      h[j] = n.x;
      narrow(y.v[j], n.x);
      if (N > 1) {
        h[k] = n.y;
        narrow(y.v[k], n.y);
      }
    }
    *reinterpret_cast<P *>(static_cast<E *>(a.y) + row * a.D + c) = y;
  }
#pragma unroll
  for (int j = 0; j < N; j += kS) {
    S s;
#pragma unroll
    for (int l = 0; l < kS; ++l) s.v[l] = h[j + l];
    *reinterpret_cast<S *>(a.state_out + sc + j) = s;
  }
}

// ---- backward ----
// The same walk from the last token to the first; what runs through it is
// e_t = a_t dh_t, the gradient that reaches h_{t-1}: dh_t = dy_t + e_{t+1}.
// K8: x, r and g come from their checkpoints.  A run is the 8 tokens between two
// kept states, so the states inside it are recomputed in registers and cost no
// memory.  8 x 4096 x 1920 in bf16: 206 us (65% of the measured copy bandwidth),
// from checkpoints 208 (11.55 bytes an element, 52%: decoding takes the time of the
// bytes it saves); 1 x 32768 x 3840: 408 (66%); 2 x 8192 x 3840 with resets: 228
// (59%); fp32, 4 x 4096 x 1920: 156 (85%).
template <class E, bool VEC, bool K8, bool CUTS>
__global__ void __maxnreg__(kBackwardRegs) glr_backward_kernel(const GlrArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  Runs &runs = *reinterpret_cast<Runs *>(smem);
  using I = typename std::conditional<K8, int8_t, E>::type;  // what x, r and g are held in
  constexpr int kBytes = Rows<I, VEC>::kBytes, kStage = 3 * kBytes + Rows<E, VEC>::kBytes, kOut = K8 ? kSteps : 0;
  const int lane = threadIdx.x & 31, warp = __shfl_sync(kFull, threadIdx.x >> 5, 0);
  const int cs = a.cs;
  unsigned char *mine = smem + sizeof(Runs) + warp * (kStage + kOut);
  const int rank = blockIdx.x % cs, c0 = (blockIdx.x / cs) * kChan, b = blockIdx.y;
  const int c = c0 + 2 * lane, chan = min(kChan, a.D - c0);
  const bool one = c < a.D, two = c + 1 < a.D;
  Place at{kWarps - 1 - warp, lane, cs - 1 - rank, cs, a.drop && rank == 0, false};
  const int len = load_len(a, b);
  const int64_t rows = static_cast<int64_t>(a.B) * a.T;
  const int G = ckpt8::groups(a.D);
  const float2 rate = make_float2(one ? load_rate(a, c) : 0.f, two ? load_rate(a, c + 1) : 0.f);
  const int64_t sc = static_cast<int64_t>(b) * a.D + c;
  float2 v = make_float2(one && a.state ? a.state[sc] : 0.f, two && a.state ? a.state[sc + 1] : 0.f);
  open_runs(runs, at);
  float2 drate = dup(0.f), lost = dup(0.f);  // the sum so far, and what its roundings lost
  const int tile = kBackwardRun * kWarps, tokens = tile * cs;
  const int steps = (len + tokens - 1) / tokens;
  int t0 = ((steps - 1) * cs + rank) * tile + warp * kBackwardRun;  // below 0 with no tokens: nothing is read then
  const int64_t first = static_cast<int64_t>(b) * a.T + t0;
  auto source = [&](const void *p, int64_t ld, int plane) {
    return K8 ? reinterpret_cast<const I *>(a.codes) + (plane * rows + first) * a.D + c0
              : static_cast<const I *>(p) + first * ld + c0;
  };
  Walk<I, VEC> wx(source(a.x, a.ld_x, 0), K8 ? a.D : a.ld_x, chan, lane);
  Walk<I, VEC> wr(source(a.r, a.ld_r, 1), K8 ? a.D : a.ld_r, chan, lane);
  Walk<I, VEC> wg(source(a.g, a.ld_g, 2), K8 ? a.D : a.ld_g, chan, lane);
  Walk<E, VEC> wy(static_cast<const E *>(a.y) + first * a.D + c0, a.D, chan, lane);
  int64_t out = first * a.ld_d + c0;
  const uint32_t out_row = static_cast<uint32_t>(a.ld_d) * static_cast<uint32_t>(sizeof(E));
  auto count = [&](int t) { return t < 0 ? 0 : max(0, min(kSeg, len - t)); };
  auto fetch = [&](int n) {
    if (n > 0) {
      wx.copy(mine, n, lane);
      wr.copy(mine + kBytes, n, lane);
      wg.copy(mine + 2 * kBytes, n, lane);
    }
    wx.move(-tokens), wr.move(-tokens), wg.move(-tokens);
    cp_async_commit();
  };
  auto fetch_dy = [&](int n) {
    if (n > 0) wy.copy(mine + 3 * kBytes, n, lane);
    wy.move(-tokens);
    cp_async_commit();
  };
  // what a step needs besides its rows, loaded a step ahead: flags, the kept
  // state, the checkpoint groups' exponents (lane 8 k + i: plane k, token i)
  const uint8_t *flags = CUTS ? a.reset + static_cast<int64_t>(b) * a.T : nullptr;
  uint32_t flag = 0, exps = 1;
  float2 h0 = dup(0.f);
  auto ahead = [&](int t) {
    const int n = count(t);
    if (CUTS) flag = reset_flag(flags, t, n, lane);
    if (n > 0) {
      const float *k = a.carry + (static_cast<int64_t>(b) * a.S + t / kSeg) * a.D + c;
      if (VEC) {
        if (one) h0 = *reinterpret_cast<const float2 *>(k);
      } else {
        h0 = make_float2(one ? k[0] : 0.f, two ? k[1] : 0.f);
      }
      if (K8 && lane < 24 && (lane & 7) < n)
        exps = a.exps[((lane >> 3) * rows + static_cast<int64_t>(b) * a.T + t + (lane & 7)) * G + c0 / kChan];
    }
  };
  ahead(t0);
  fetch(count(t0));
  fetch_dy(count(t0));
  if (cs > 1) cluster_wait();
  for (int step = 0; step < steps; ++step, t0 -= tokens) {
    const int n = count(t0);
    const uint32_t cut = CUTS ? __ballot_sync(kFull, flag != 0) : 0;
    float2 h = h0;
    if (K8 && lane < 24) reinterpret_cast<float *>(mine + kStage)[lane] = ckpt8::step(exps);
    ahead(t0 - tokens);
    cp_async_wait<1>();
    __syncwarp();
    const unsigned char *d = mine;
    auto input = [&](const Walk<I, VEC> &w, int k, int i) {
      if constexpr (K8) {
        return ckpt8::decode2(w.bits(d + k * kBytes, i, lane), reinterpret_cast<const float *>(mine + kStage)[8 * k + i]);
      } else {
        return w.pair(d + k * kBytes, i, lane);
      }
    };
    // per token: the decay; what dh is multiplied by in dx and dg; and -sr a
    // (h_{t-1} - (a / m) sg x), by which it is in drate (dr: that times rate (1 - sr))
    float2 f[kSeg], cx[kSeg], cg[kSeg], cr[kSeg], ck[kSeg];
    auto dy = [&](int i) { return wy.pair(d + 3 * kBytes, i, lane); };
#pragma unroll
    for (int i = 0; i < kSeg; ++i) {
      const float2 x = input(wx, 0, i), sr = sigmoid2(input(wr, 1, i)), sg = sigmoid2(input(wg, 2, i));
      const Decay q = decay(mul2(rate, sr));
      f[i] = q.a;
      const float2 m2 = mul2(q.e, fma2(q.e, dup(-1.f), dup(2.f)));
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
    cp_async_wait<0>();
    __syncwarp();  // dy is here, and the next inputs go where these were read
    fetch(count(t0 - tokens));
    // dh_i = dy_i + f dd with f and dd those of token i + 1
    Run q{dup(1.f), dup(0.f)};
    float2 ff = dup(0.f), dd = dup(0.f);
    if (n == kSeg && !(CUTS && cut)) {
#pragma unroll
      for (int i = kSeg - 1; i >= 0; --i) q.P = mul2(q.P, f[i]), dd = fma2(ff, dd, dy(i)), ff = f[i];
    } else {
#pragma unroll
      for (int i = kSeg - 1; i >= 0; --i)
        if (i < n) {
          q.P = mul2(q.P, f[i]);
          dd = fma2(ff, dd, dy(i)), ff = f[i];
          if (CUTS && cut >> i & 1) ff = dup(0.f), dd = dup(0.f);
        }
    }
    q.H = mul2(ff, dd);
    if (CUTS && cut) q.P = dup(kCut);
    dd = compose<CUTS, sizeof(Runs) + kWarps * (kStage + kOut)>(runs, step, at, q, v), ff = dup(1.f);
    if (n > 0) {
      E *dx = static_cast<E *>(a.dx) + out, *dr = static_cast<E *>(a.dr) + out, *dg = static_cast<E *>(a.dg) + out;
      uint32_t o = 2 * lane * static_cast<uint32_t>(sizeof(E)) + (kSeg - 1) * out_row;
      float2 part = dup(0.f);
      // `whole`: all 8 tokens exist (a run's only test of n then; with one
      // per token 8 x 4096 x 1920 took 10 us more)
      auto put = [&](auto whole) {
#pragma unroll
        for (int i = kSeg - 1; i >= 0; --i, o -= out_row) {
          asm volatile("" : "+r"(o));  // keeps a row's offset one addition per lane
          if (decltype(whole)::value || i < n) {
            const float2 dh = fma2(ff, dd, dy(i)), w = mul2(dh, cr[i]);
            part = fma2(dh, cr[i], part);
            if (one) {
              store2<VEC>(dx, o, mul2(dh, cx[i]), two);
              store2<VEC>(dr, o, mul2(w, ck[i]), two);
              store2<VEC>(dg, o, mul2(dh, cg[i]), two);
            }
            ff = f[i], dd = dh;
            if (CUTS && cut >> i & 1) ff = dup(0.f), dd = dup(0.f);
          }
        }
      };
      if (n == kSeg) put(std::true_type{});
      else put(std::false_type{});
      // the run's sum joins without loss: thousands of them cancel to a little (two-sum)
      const float2 sum = add2(drate, part), back = sub2(sum, drate);
      lost = add2(lost, add2(sub2(drate, sub2(sum, back)), sub2(part, back)));
      drate = sum;
    }
    out -= tokens * a.ld_d;
    __syncwarp();  // the next dy goes where this was read
    fetch_dy(count(t0 - tokens));
  }
  if (rank == 0 && warp == 0 && one) {
    a.state_out[sc] = v.x;
    if (two) a.state_out[sc + 1] = v.y;
  }
  // drate over the CTA's warps, then over the cluster's CTAs, in their order.  A CTA
  // leaves its sum in CTA 0's slots of the half that the last step did not use:
  // CTA 0 is at most one step behind.
  drate = add2(drate, lost);
  float2 *sum = reinterpret_cast<float2 *>(smem + sizeof(Runs));
  cp_async_wait<0>();
  __syncthreads();
  sum[warp * 32 + lane] = drate;
  __syncthreads();
  if (warp == 0)
    for (int i = 1; i < kWarps; ++i) drate = add2(drate, sum[i * 32 + lane]);
  auto slot = [&](int j) {
    return reinterpret_cast<float2 *>(smem + sizeof(Runs) + kWarps * (kStage + kOut) + (2 * j + (steps & 1)) * 512) + lane;
  };
  if (cs > 1 && warp == 0 && rank > 0)
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};\n" ::"r"(in_cta(slot(rank), 0)), "f"(drate.x), "f"(drate.y)
                 : "memory");
  close_runs(at, a.err);
  if (warp == 0 && rank == 0) {
    for (int i = 1; i < cs; ++i) drate = add2(drate, *slot(i));
    float *p = a.part + static_cast<int64_t>(b) * a.D + c;
    if (one) p[0] = drate.x;
    if (two) p[1] = drate.y;
  }
}

// drate[c] = sum over the sequences' parts: 32 interleaved sums, then those in
// order.  A launch behind the backward's (about 2 us); one sequence needs none.
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
  if (ld < D || ld >= 1 << 27) return set_error(SDM_ERR_SHAPE, "%s: need D <= ld < 2^27 (%s)", fn, name);
  if (!aligned(p, dtype == SDM_DTYPE_F32 ? 4 : 2))
    return set_error(SDM_ERR_ALIGN, "%s: %s must be aligned to its element", fn, name);
  return SDM_OK;
}

int check_words(const char *fn, std::initializer_list<const void *> ps) {
  for (const void *p : ps)
    if (!aligned(p, 4)) return set_error(SDM_ERR_ALIGN, "%s: fp32 and int32 arrays must be 4-byte aligned", fn);
  return SDM_OK;
}

// Shared memory of a CTA without its cluster's runs.
template <class E, bool VEC>
constexpr size_t forward_smem() {
  return sizeof(Runs) + kWarps * kForwardRun / kSeg * 3 * Rows<E, VEC>::kBytes;
}
template <class E, bool VEC>
constexpr size_t backward_smem(bool keep8) {
  return sizeof(Runs) + kWarps * (3 * (keep8 ? Rows<int8_t, VEC>::kBytes : Rows<E, VEC>::kBytes) + Rows<E, VEC>::kBytes +
                                  (keep8 ? kSteps : 0));
}

// CTAs of a cluster.  A walk takes its steps once while the whole grid runs at
// once, however few CTAs an SM has (it then waits for memory and for the runs of others);
// beyond that, between the grid's share of the GPU and whole waves of it times as long.
// Clusters of more than two CTAs find room on 148 of the 152 SMs.  Measured for 8 x 4096 x 1920
// in bf16, forward: 121 us with 2 CTAs (81% of one wave), 119 with 3, 111 with 4, 119
// with 5, 116 with 6, 115 with 8, 132 with 9; backward: 216, 241, 206, 230, 217, 218 and 224;
// 1 x 32768 x 3840, forward: 293 with 4, 248 with 8, 223 with 9; backward: 587, 441, 407.
// More than 8 CTAs only where all of them have room by that count and the walk with 8 has
// more than 16 steps.  The count is too high for large clusters where they would nearly
// fill the GPU: without the second condition 8 x 3000 x 480 backward took 72 us in
// place of 55 and 4 x 8192 x 963 forward 136 in place of 105, and without either
// 12 x 512 x 1285 in fp32 backward 94 in place of 63.  What the second one costs: few
// channels at up to 8192 (backward 4096) tokens would be faster with 16 CTAs, 1 x 4096 x
// 480 by 18.4 us in place of 22.5 and 29 in place of 41, 1 x 6000 x 64 forward by 20.5
// in place of 30.7.
int cluster_size(int B, int T, int D, int run, int regs, size_t smem) {
  const int64_t columns = static_cast<int64_t>(B) * ((D + kChan - 1) / kChan);
  const int tile = run * kWarps;
  int best = 1;
  double least = 1e300;
  for (int cs = 1; cs <= kMaxCluster; ++cs) {
    if (cs > 1 && (cs - 1) * tile >= T) break;
    const int per_sm = min(65536 / (32 * regs) / kWarps, static_cast<int>((227 << 10) / (cluster_bytes(cs) + smem + 1024)));
    const int64_t room = (cs > 2 ? kSMs - 4 : kSMs) * per_sm, ctas = columns * cs;
    if (cs > 8 && (ctas > room || T <= 16 * 8 * tile)) break;
    const int64_t waves = (ctas + room - 1) / room, steps = (T + tile * cs - 1) / (tile * cs);
    const double share = static_cast<double>(ctas) / room;
    const double time = steps * ((share < 1 ? 1 : share) + waves) / 2;
    if (time < 0.95 * least) least = time, best = cs;
  }
  return best;
}
int forward_cluster(int B, int T, int D, int dtype) {
  return cluster_size(B, T, D, kForwardRun, kForwardRegs,
                      dtype == SDM_DTYPE_F32 ? forward_smem<float, true>() : forward_smem<uint16_t, true>());
}
int backward_cluster(int B, int T, int D, int dtype) {
  return cluster_size(B, T, D, kBackwardRun, kBackwardRegs,
                      dtype == SDM_DTYPE_F32 ? backward_smem<float, true>(false) : backward_smem<uint16_t, true>(false));
}

// 16-byte copies of rows, pairwise stores
bool rows_vec(const void *p, int64_t ld, int es) { return aligned(p, 16) && ld * es % 16 == 0; }
bool pairs_vec(const void *p, int64_t ld, int es) { return aligned(p, 2 * es) && ld % 2 == 0; }

// A call that CUDA refused, taken off the thread's own record too: it is not the next launch's.
int refused(const char *fn, cudaError_t e) {
  cudaGetLastError();
  return set_error(SDM_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
}

// layout: the kernel's shared memory without its cluster's runs.  The limit that
// is set is the kernel's, for the largest cluster, and not the call's: between
// here and the launch another thread's call of the same kernel may set it too.
template <class K>
int launch(const char *fn, K kernel, size_t layout, const GlrArgs &a, cudaStream_t st) {
  const size_t smem = layout + cluster_bytes(a.cs);
  cudaError_t e;
  if (smem > 48 << 10) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(layout + cluster_bytes(kMaxCluster)));
    if (e != cudaSuccess) return refused(fn, e);
  }
  if (a.cs > 8) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return refused(fn, e);
  }
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
  return e == cudaSuccess ? SDM_OK : refused(fn, e);
}

// Up to kStepTokens tokens and nothing to keep: one thread walks them all.
constexpr int kStepTokens = 8;
template <class E>
int launch_step(const char *fn, const GlrArgs &a, cudaStream_t st) {
  constexpr int N = 16 / sizeof(E), es = sizeof(E);
  const bool wide = a.D % N == 0 && rows_vec(a.x, a.ld_x, es) && rows_vec(a.r, a.ld_r, es) && rows_vec(a.g, a.ld_g, es) &&
                    rows_vec(a.y, a.D, es) && aligned(a.state, 16) && aligned(a.state_out, 16) && aligned(a.rate, 16);
  const int64_t threads = static_cast<int64_t>(a.B) * (wide ? a.D / N : a.D), blocks = (threads + 127) / 128;
  if (blocks > INT32_MAX) return set_error(SDM_ERR_SHAPE, "%s: B * D too large", fn);
  if (wide) glr_step_kernel<E, N><<<static_cast<unsigned>(blocks), 128, 0, st>>>(a);
  else glr_step_kernel<E, 1><<<static_cast<unsigned>(blocks), 128, 0, st>>>(a);
  return check_launch(fn);
}

template <class E, bool VEC>
int launch_forward(const char *fn, const GlrArgs &a, cudaStream_t st) {
  const size_t smem = forward_smem<E, VEC>();
  if (a.reset)
    return a.codes ? launch(fn, glr_forward_kernel<E, VEC, true, true>, smem, a, st)
                   : launch(fn, glr_forward_kernel<E, VEC, false, true>, smem, a, st);
  return a.codes ? launch(fn, glr_forward_kernel<E, VEC, true, false>, smem, a, st)
                 : launch(fn, glr_forward_kernel<E, VEC, false, false>, smem, a, st);
}
template <class E, bool VEC>
int launch_backward(const char *fn, const GlrArgs &a, cudaStream_t st) {
  const size_t smem = backward_smem<E, VEC>(a.codes != nullptr);
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
  if (a.T <= kStepTokens && !a.carry)
    return dtype == SDM_DTYPE_F32 ? launch_step<float>(fn, a, st) : launch_step<uint16_t>(fn, a, st);
  a.codes = codes, a.exps = exps;
  a.drop = test_drop_signal();
  a.cs = forward_cluster(a.B, a.T, a.D, dtype);
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
  return B < 2 ? 0 : (sizeof(float) * B * static_cast<size_t>(D) + 255) / 256 * 256;
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
    if (need > 0 && (!workspace || workspace_bytes < need))
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
  a.dx = dx, a.dr = dr, a.dg = dg, a.part = B == 1 ? drate : static_cast<float *>(workspace), a.err = dev_err;
  a.drop = test_drop_signal();
  a.cs = backward_cluster(B, T, D, dtype);
  if (B > 0) {
    const int es = dtype == SDM_DTYPE_F32 ? 4 : 2;
    const bool in = codes ? D % 16 == 0 : rows_vec(x, ld_x, es) && rows_vec(r, ld_r, es) && rows_vec(g, ld_g, es);
    const bool vec = in && rows_vec(dy, D, es) && pairs_vec(dx, ld_d, es) && pairs_vec(dr, ld_d, es) &&
                     pairs_vec(dg, ld_d, es) && aligned(carry, 8);
    if (dtype == SDM_DTYPE_F32)
      rc = vec ? launch_backward<float, true>(fn, a, st) : launch_backward<float, false>(fn, a, st);
    else
      rc = vec ? launch_backward<uint16_t, true>(fn, a, st) : launch_backward<uint16_t, false>(fn, a, st);
    if (rc || B == 1) return rc;
  }
  glr_rate_kernel<<<(D + 31) / 32, dim3(32, 32), 0, st>>>(a.part, B, D, drate);
  return check_launch(fn);
}
