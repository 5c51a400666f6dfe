// Attention of new queries over the paged 4-bit cache, many query rows per key
// (prompts, chunks of prompts, long drafts): tcgen05 with the same arithmetic as
// kv4_attend.cu.  Codes are unpacked once per block and tile of keys into shared
// memory as fp16 numbers; S = Q K^T and O += P V have fp32 accumulators in tensor
// memory, P is the tensor-memory operand, over S.  Two ways, by the queries' type:
//   fp16  the unpacked numbers are c - z, exact; scores and probabilities take the
//         scale of their key, x = S s_j scale log2(e), P = 2^(x - m) s'_j, and the only
//         rounding besides fp32's is P's.  That is 2^-11 of each, as much as the output's own,
//         and makes the error 1.4 times that one's (kv4_attend.cu takes two terms).  A second
//         term would fit over the scores, but twice the products and the subtractions in the
//         softmax took 1782 us for 1376 (two chunks of 2048 over 16k), 187 for 173 under the
//         window below.
//   bf16  the unpacked numbers are the keys and values themselves, s (c - z) times a power
//         of two of the step, rounded to fp16 (the scale in two terms, so rounded once; a
//         value's scale in one), and
//         queries are taken to fp16 by a power of two per row, exactly.  That is 2^-11
//         relative per key and value where the output is rounded at 2^-8, and it spares
//         every row reading two numbers per key: reads of the same 16 bytes by all lanes
//         cost four passes through shared memory each, and those were 1000 of the 2400
//         passes per step that bounded the kernel.
// The running maximum m is a whole number, of the weights that P holds (see kv4_attend.cu), and
// moves only when one passes it by 5 binades or more; what was summed before is then scaled by a
// power of two.
//
// One block = up to 256 rows (two tiles of 128; one at head_dim 256) of one
// sequence and key/value head, over its keys 64 at a time.  Warps:
//   0-3, 4-7  softmax of tile 0, of tile 1: a thread owns a row, reads its 64 scores and
//             writes the probabilities over them, so no reduction crosses lanes.  With one
//             tile both take half of its columns: what the step waits for is their latency
//   8, 9      issue the MMAs, of a tile each (one warp needs some 70 cycles per MMA, more
//             than an MMA of 64 keys takes).  Every tile has two S buffers and S runs two steps ahead
//             (S of step j + 2 goes over P of step j behind P V of step j), so the softmax
//             never waits for a product: with 128 keys and one buffer (all of tensor
//             memory) it did, and a step took twice as long.
//   10        numbers: looks up the pages, turns the keys' words into factors, up to 8
//             steps ahead
//   11-15     unpacking: 32 tokens' keys or values at a time, in turn (four such jobs to
//             a step), the next one's codes on their way; rows of 128 bytes, 128-byte
//             swizzled, for both operands (keys K-major, values MN-major)
// Dims stay in the order unpacking yields within each 8 (0 4 1 5 2 6 3 7): queries
// are stored that way and the output is put right when it leaves.
//
// Measured: two chunks of 2048 tokens over 16k, 32 query heads of 128, bf16: 1.27 ms,
// 810 TFLOP/s of the two products; fp16 1.38 ms.  A step of 64 keys takes 2200 to 2800 cycles:
// the softmax of a row some 1900 (600 to 900 for scores and maximum, 1200 for exponentials and
// P), the MMAs 1280 of tensor pipe (S reads 48 KB of shared memory per tile, 384 cycles where
// the products would take 256), issued one behind the other.  A unit costs some 12 us
// beside its steps (division of the work, first loads, output): 1777 tokens under a window
// of 1024, heads of 256, fp16: 172 us, 452 TFLOP/s (204 with one warp to a row); of a step's
// 2600 cycles there, a softmax warp waits 720 for scores, takes 930 to the maximum that two
// warps agree on and 740 to P.  Heads of 256, bf16: the two warps that unpack keys bound it (two
// prompts of 1024 over 6000, 600 us: the MMA warp waits 3000 of 4900 cycles for them).
//
// All waits are bounded; one that gives up records KRONQ_ERR_TIMEOUT in `info`.
#include <type_traits>

#include "kv4_attend.cuh"

namespace kv4 {
namespace {

constexpr int NUM_QUERY_WARPS = 8, MMA_WARP0 = 8, NUM_WARP = 10, UNPACK_WARP0 = 11, THREADS = 512;
constexpr int BN = 64, GROUP = 16, GROUPS = BN / GROUP;    // keys per step; that surely share a page
constexpr int JOB = 32, JOBS = BN / JOB;                   // keys per unpacking job; jobs for a step's keys
constexpr float NO_MAX = -0x1p127f;     // a split's maximum where it saw no key

// Scales in fp16.  The scales of a step's values (bf16: and of its keys) share a power of two
// that is set for each step, 2^V_TOP and 2^K_TOP times [1, 2) for the largest: operands of 15
// times that fit, and ones down to 2^-24 of the largest scale are normal numbers.  A step
// whose scales are further apart than V_SPREAD or K_SPREAD binaries is a wide one: its operands
// are c - z (values: 2^V_TOP of it), exact, and every row takes its keys' scales for itself, so
// that a row that does not see the largest keeps what it sees.  The limits are not a
// matter of speed: by V_SPREAD binaries a row's weights may lie lower in P's range without
// harm; K_SPREAD leaves a key's numbers 2^-19 of themselves exact.
constexpr uint32_t kZeroScale = 0x0d800000u;      // 2^-100: a zero vector's; its score is 0 whatever its factor
constexpr uint32_t V_SPREAD = 8, K_SPREAD = 16;
constexpr uint32_t WIDE = 1u << 31;
constexpr float FAR = 80.f;                       // as in kv4_attend.cu

template <int D>
struct Shape {
  static constexpr int NT = D == 256 ? 1 : 2;        // tiles of 128 rows
  static constexpr int R = 128 * NT;
  static constexpr int HALVES = 2 / NT;              // softmax warps that share a row
  static constexpr int ATOMS = D / 64;               // 128-byte columns of an operand row
  static constexpr int Q_BYTES = R * D * 2;
  static constexpr int KV_BYTES = BN * D * 2;        // keys or values of a stage
  static constexpr int STAGE = 2 * KV_BYTES;
  static constexpr int CH = D / 32;                  // 16-byte chunks of a token's codes
  static constexpr int TPL = 32 / CH;                // tokens per load of a warp
  static constexpr int LOADS = JOB / TPL;            // chunks per lane of a job
  static constexpr int O_COL = 256;                  // tensor memory: S buffers, 64 columns each, then O
  static constexpr int STAGES = D == 256 ? 2 : 4;    // of keys and values: what fits
  static constexpr int LG = D == 256 ? 1 : 2;
  // Unpacking warps.  A job of step j waits for its stage's last user, step j - STAGES; a
  // barrier tells two phases apart, so step j - 2 STAGES must be known to be done.  It is:
  // with four stages the warp's job before was of step j - 2 at the least and waited for S
  // or P V of step j - 6, both behind P V of step j - 8; with two, four warps have one kind
  // of job each and wait for every step.
  static constexpr int UNPACKERS = D == 256 ? 4 : 5;
  static constexpr int SMEM = Q_BYTES + STAGES * STAGE + 1024;
};

// What the other warps need to know of a step's keys.
struct alignas(16) Numbers {
  float fk[BN], sv[BN];      // fp16 queries, wide steps: score factor; value scale x 2^lift
  float far[BN];             // wide steps: log2 of the value scale, for the running maximum
  uint32_t ks[BN];           // bf16: key scale x 2^f as two halves (high term, low term)
  uint16_t vs[BN];           // bf16: value scale x 2^lift
  uint8_t zeros[BN];         // key's zero point | value's << 4
  uint64_t codes[GROUPS];    // address of the group's first key's codes, 0: no page
  // (one read by the softmax warps: each waits its turn behind the unpackers' stores)
  struct alignas(16) All {
    uint32_t absent;         // bit per group: no page; WIDE
    float lift, up;          // of the step's value scales; 2^lift
    float down;              // bf16: 2^-f
  } all;
  float back;                // 2^-lift of what it would be in a step that is not wide, within 2^+-64
};

struct alignas(16) Ctl {
  Numbers num[8];            // step j: num[j & 7]
  uint64_t num_full[8], num_free[8];
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t s_full[2][2], p_ready[2][2];  // per tile and buffer
  uint64_t pv_done[2], o_full, q_full;
  uint32_t tmem;
  int abort;
  float row[256];                        // bf16: score factor of each row
  Unit unit;                             // for the output: nothing of it stays in registers
  Seq seq;
  float2 pair[2][128];                   // what the two threads of a row tell each other
};

// Or of a predicate over the two warps of a barrier.
KQ_DEV bool pair_or(int bar, bool x) {
  uint32_t r;
  __syncwarp();
  asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 q, %2, 0;\n bar.red.or.pred p, %1, 64, q;\n"
               " selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(r)
               : "r"(bar), "r"((uint32_t)x)
               : "memory");
  return r != 0;
}
KQ_DEV void pair_sync(int bar) {
  __syncwarp();
  asm volatile("bar.sync %0, 64;" ::"r"(bar) : "memory");
}

// One lane of a converged warp, the same one every time.  The operands of what it issues
// are computed by the whole warp, so that they live in uniform registers; from one lane's
// registers each would be moved there first (some 100 cycles per MMA).
KQ_DEV bool elect_one() {
  uint32_t e;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(e));
  return e != 0;
}
KQ_DEV uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

KQ_DEV void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

KQ_DEV void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
KQ_DEV void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

KQ_DEV float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

KQ_DEV uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// (volatile: a load stays in front of the waits it is to pass the time of)
KQ_DEV void load16(uint4& v, const uint4* p) {
  asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
}
KQ_DEV uint32_t load4(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

// of a power of two
KQ_DEV float exponent(float x) { return (float)((int)(__float_as_uint(x) >> 23) - 127); }

KQ_DEV float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// 8 codes less their zero point, as 8 halves in the order 0 4 1 5 2 6 3 7.
// z1: 1024 + z in both halves, z2: -(64 + z); exact: 1024 + c and 1024 + 16 c are.
KQ_DEV uint4 codes_f16(uint32_t w, uint32_t z1, uint32_t z2) {
  const __half2 s = __halves2half2(__ushort_as_half(0x2c00), __ushort_as_half(0x2c00));   // 1/16
  const __half2 a = *reinterpret_cast<const __half2*>(&z1), b = *reinterpret_cast<const __half2*>(&z2);
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t v = i ? w >> 8 : w;
    const uint32_t lo = (v & 0x000f000fu) | 0x64006400u, hi = (v & 0x00f000f0u) | 0x64006400u;
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&lo), a);
    const __half2 y = __hfma2(*reinterpret_cast<const __half2*>(&hi), s, b);
    r[2 * i] = *reinterpret_cast<const uint32_t*>(&x);
    r[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&y);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}
KQ_DEV uint32_t mul_half2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
KQ_DEV uint32_t fma_half2(uint32_t a, uint32_t b, uint32_t c) {
  const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b),
                            *reinterpret_cast<const __half2*>(&c));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// v (hi + lo), rounded once (the product with lo is 2^-11 of it)
KQ_DEV uint4 scaled(uint4 v, uint32_t hi, uint32_t lo) {
  return make_uint4(fma_half2(v.x, hi, mul_half2(v.x, lo)), fma_half2(v.y, hi, mul_half2(v.y, lo)),
                    fma_half2(v.z, hi, mul_half2(v.z, lo)), fma_half2(v.w, hi, mul_half2(v.w, lo)));
}
KQ_DEV uint4 scaled(uint4 v, uint32_t s) {
  return make_uint4(mul_half2(v.x, s), mul_half2(v.y, s), mul_half2(v.z, s), mul_half2(v.w, s));
}

template <int D, bool BF>
__global__ void __launch_bounds__(THREADS, 1) kv4_prompt_kernel(const AttendArgs a) {
  using SH = Shape<D>;
  constexpr int NT = SH::NT, R = SH::R, ATOMS = SH::ATOMS;
  // How far weights may pass the running maximum, and where it is put below a new one.
  constexpr float LAG = BF ? 15.f : 14.f, BASE = 9.f;
  constexpr int V_TOP = BF ? 10 : 0, K_TOP = 10;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Ctl ctl;
  uint8_t* q_smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
  uint8_t* kv_smem = q_smem + SH::Q_BYTES;

  Unit u;
  if (!find_unit<R, BN, THREADS>(a, &u)) return;
  const int head = u.head;
  const Seq s = seq_of(a, u.b, nullptr);
  if (threadIdx.x == 0 && head == 0 && u.tile == 0 && u.split == 0)
    a.meta[u.b] = make_int2(u.slot, u.nsplit);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rows = s.n * a.g, r0 = u.tile * R;
  const int last = min(rows, r0 + R) - 1;
  const int q_first = r0 / a.g, q_last = last / a.g;
  const int tiles = NT == 2 && r0 + 128 < rows ? 2 : 1;
  const Span sp = span_of<BN>(a, s, q_first, q_last);
  const int per = ceil_div(sp.nb, u.nsplit);
  const int i0 = u.split * per;
  const int steps = max(0, min(sp.nb, i0 + per) - i0);
  auto lo_of = [&](int q) { return a.window ? max(0, s.L - s.n + q - a.window + 1) : 0; };
  auto hi_of = [&](int q) { return max(0, a.causal ? min(s.L, s.L - s.n + q + 1) : s.L); };
  auto key_of = [&](int i) { return (i < sp.sb ? i : sp.lb + i - sp.sb) * BN; };   // first key of block i

  volatile int* abort = &ctl.abort;
  constexpr int UNPACKERS = SH::UNPACKERS;
  constexpr int STAGES = SH::STAGES, LG = SH::LG, SM = STAGES - 1;    // stage of step j: j & SM, its phase j >> LG
  if (threadIdx.x == 0) {
    for (int i = 0; i < SH::STAGES; ++i) {
      kq::mbar_init(&ctl.k_full[i], JOBS);
      kq::mbar_init(&ctl.k_empty[i], tiles);
      kq::mbar_init(&ctl.v_full[i], JOBS);
      kq::mbar_init(&ctl.v_empty[i], tiles);
    }
    for (int i = 0; i < 2; ++i) {
      for (int k = 0; k < 2; ++k) {
        kq::mbar_init(&ctl.s_full[i][k], 2);   // S itself, and that its keys' numbers are there
        kq::mbar_init(&ctl.p_ready[i][k], 4 * SH::HALVES);
      }
      kq::mbar_init(&ctl.pv_done[i], 1);
    }
    for (int i = 0; i < 8; ++i) {
      kq::mbar_init(&ctl.num_full[i], 1);
      kq::mbar_init(&ctl.num_free[i], 4 * SH::HALVES * tiles + JOBS);   // softmax warps, unpackers of the values
    }
    ctl.unit = u;
    ctl.seq = s;
    kq::mbar_init(&ctl.o_full, tiles);
    kq::mbar_init(&ctl.q_full, NUM_QUERY_WARPS);
    ctl.abort = 0;
    kq::fence_barrier_init();
  }
  if (warp == MMA_WARP0) kq::tmem_alloc(&ctl.tmem, 512);
  kq::tc_fence_before();
  // The barriers are set up and tensor memory is there: every warp comes by here once, those
  // that have something to ask of global memory after asking it.
  auto set_up = [&]() {
    asm volatile("bar.sync 0;" ::: "memory");
    kq::tc_fence_after();
  };

  // a wait of the whole warp: all lanes agree on its outcome
  auto wait = [&](uint64_t* bar, int parity) -> bool {
    return __all_sync(0xffffffffu, kq::mbar_wait(bar, (uint32_t)parity & 1u, abort, a.info));
  };

  if (warp < NUM_QUERY_WARPS) {
    // Queries: rows of 128-byte lines, dims of each 8 in the codes' order.  The softmax
    // warps load them while the first keys are unpacked.
    const float rg = 1.f / (float)a.g;
    constexpr int ALL = R * (D / 8) / (32 * NUM_QUERY_WARPS), PART = ALL < 8 ? ALL : 8;
#pragma unroll 1
    for (int i = 0; i < ALL; i += PART) {
      uint4 v[PART];
#pragma unroll
      for (int k = 0; k < PART; ++k) {
        const int e = threadIdx.x + (i + k) * (32 * NUM_QUERY_WARPS);
        const int r = e / (D / 8), c = e - r * (D / 8);
        v[k] = make_uint4(0u, 0u, 0u, 0u);
        if (r0 + r < rows) {
          // (the quotient is below 2^9 + 1: half a row off an integer, fp32 does not miss it)
          const int qi = q_first + (int)(((float)(r0 + r - q_first * a.g) + 0.5f) * rg);
          const uint16_t* p = a.q + (int64_t)(s.row0 + qi) * a.q_st +
                              (int64_t)(head * a.g + r0 + r - qi * a.g) * a.q_sh + 8 * c;
          if (a.q_vec) {
            load16(v[k], reinterpret_cast<const uint4*>(p));
          } else {
            uint32_t h[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) h[j] = __ldg(p + j);
            v[k] = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
          }
        }
      }
      if (i == 0) set_up();
#pragma unroll
      for (int k = 0; k < PART; ++k) {
        const int e = threadIdx.x + (i + k) * (32 * NUM_QUERY_WARPS);
        const int r = e / (D / 8), c = e - r * (D / 8);
        uint4 w = v[k];
        if (BF) {
          // to fp16 by the power of two that takes the row's largest to about 2^10 (the
          // D / 8 lanes of a row are neighbours)
          float x[8];
          unpack8(w, BF16, x);
          float big = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) big = fmaxf(big, fabsf(x[j]));
#pragma unroll
          for (int o = 1; o < D / 8; o <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
          const int ex = min(max(137 - (int)(__float_as_uint(big) >> 23), -126), 126);
          const float up = __uint_as_float((uint32_t)(127 + ex) << 23);
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] *= up;
          w = pack8(x, FP16);
          if (c == 0) ctl.row[r] = a.scale_log2 * __uint_as_float((uint32_t)(127 - ex) << 23);
        }
        w = make_uint4(__byte_perm(w.x, w.z, 0x5410), __byte_perm(w.x, w.z, 0x7632),
                       __byte_perm(w.y, w.w, 0x5410), __byte_perm(w.y, w.w, 0x7632));
        uint8_t* dst = q_smem + ((r >> 7) * ATOMS + (c >> 3)) * 16384 + (r & 127) * 128 +
                       (((c & 7) ^ (r & 7)) << 4);
        *reinterpret_cast<uint4*>(dst) = w;
      }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) kq::mbar_arrive(&ctl.q_full);
  } else if (warp != NUM_WARP) {
    set_up();
  }

  if (warp >= MMA_WARP0 && warp < MMA_WARP0 + tiles) {
    const int tile = warp - MMA_WARP0;
    // -------------------------------------------------------------- MMAs
    const uint32_t tm = uniform(ctl.tmem), qa = uniform(kq::smem_u32(q_smem)), kv = uniform(kq::smem_u32(kv_smem));
    auto issue_s = [&](int j) {
      constexpr uint32_t idesc = kq::idesc_f16(128, BN, 0, 0, 0);
      const uint32_t d = tm + (2 * tile + (j & 1)) * BN;
      const uint64_t qd = kq::smem_desc(qa + tile * (ATOMS * 16384), 16, 1024, kq::kLayoutSwizzle128B);
      const uint64_t kd = kq::smem_desc(kv + (j & SM) * SH::STAGE, 16, 1024, kq::kLayoutSwizzle128B);
      if (elect_one()) {
#pragma unroll
        for (int at = 0; at < ATOMS; ++at)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            kq::mma_f16(d, qd + ((at * 16384 + kk * 32) >> 4), kd + ((at * (BN * 128) + kk * 32) >> 4), idesc,
                        at || kk);
        kq::mma_commit(&ctl.k_empty[j & SM]);
        kq::mma_commit(&ctl.s_full[tile][j & 1]);
        kq::mbar_arrive(&ctl.s_full[tile][j & 1]);
      }
    };
    auto issue_pv = [&](int j) {
      constexpr uint32_t idesc = kq::idesc_f16(128, D, 0, 0, 1);
      const uint32_t d = tm + SH::O_COL + tile * D, p = tm + (2 * tile + (j & 1)) * BN;
      const uint64_t vd =
          kq::smem_desc(kv + (j & SM) * SH::STAGE + SH::KV_BYTES, BN * 128, 1024, kq::kLayoutSwizzle128B);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < BN / 16; ++kk) mma_f16_ts(d, p + kk * 8, vd + ((kk * 2048) >> 4), idesc, kk > 0 || j > 0);
        kq::mma_commit(&ctl.v_empty[j & SM]);
        kq::mma_commit(&ctl.pv_done[tile]);
      }
    };
    bool ok = wait(&ctl.q_full, 0);
    for (int j = 0; j < min(steps, 2) && ok; ++j) {
      ok = wait(&ctl.k_full[j], 0);
      if (!ok) break;
      kq::tc_fence_after();
      issue_s(j);
    }
    for (int j = 0; j < steps && ok; ++j) {
      ok = wait(&ctl.v_full[j & SM], j >> LG) && wait(&ctl.p_ready[tile][j & 1], j >> 1);
      if (!ok) break;
      kq::tc_fence_after();
      issue_pv(j);
      if (j + 2 < steps) {
        ok = wait(&ctl.k_full[(j + 2) & SM], (j + 2) >> LG);
        if (!ok) break;
        kq::tc_fence_after();
        // (over P, in issue order behind the MMAs that read it)
        issue_s(j + 2);
      }
    }
    // (also after a wait that gave up: nothing is in flight when the block ends)
    if (elect_one()) kq::mma_commit(&ctl.o_full);
    __syncwarp();
    volatile int none = 0;
    kq::mbar_wait(&ctl.o_full, 0, &none, a.info);
    __syncwarp();
  } else if (warp == MMA_WARP0 + 1) {
    // (one tile: nothing to issue)
  } else if (warp == NUM_WARP) {
    // ----------------------------------------------------------- numbers
    // Page numbers are asked for three steps ahead (lane g: group g), words two steps ahead
    // (keys lane and lane + 32): their latencies pass while earlier steps are written.
    const int any_lo = lo_of(q_first), any_hi = hi_of(q_last);
    const int P = a.cache.P;
    auto seen = [&](int t) { return t < any_hi && (t >= any_lo || t < a.sinks); };
    auto ask_page = [&](int j) -> int {
      const int t0 = key_of(i0 + j) + GROUP * lane;
      // (INT32_MIN: nobody sees the group's keys; a negative entry becomes -1)
      if (j >= steps || lane >= GROUPS || !(t0 < any_hi && (t0 + GROUP > any_lo || t0 < a.sinks))) return INT32_MIN;
      return max(-1, (int)load4(reinterpret_cast<const uint32_t*>(a.b.table + u.b * a.b.table_ld + (t0 >> a.cache.lgP))));
    };
    struct Words {
      uint32_t k[2], v[2];
      uint64_t codes;          // lane g: of group g
    };
    auto ask_words = [&](Words& q, int j, int page) {
      const bool here = page >= 0 && page < a.cache.pages;
      if (!here && page != INT32_MIN) kq::record_error(a.info, KRONQ_ERR_INVALID_ARG);
      const int key0 = key_of(i0 + j);
      const uint8_t* blk = a.cache.base + ((int64_t)page * a.cache.heads + head) * (int64_t)a.cache.block_bytes;
      const uint64_t b64 = here ? (uint64_t)blk : 0;
      q.codes = here ? b64 + ((key0 + GROUP * lane) & (P - 1)) * (D / 2) : 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = key0 + lane + 32 * i;
        const uint64_t b = __shfl_sync(0xffffffffu, b64, (lane >> 4) + 2 * i);
        q.k[i] = q.v[i] = 0;
        // what no row sees may be memory that was never written: its scales count as 0
        if (b && seen(t)) {
          const uint32_t* wp = reinterpret_cast<const uint32_t*>(b + (uint64_t)P * D) + (t & (P - 1));
          q.k[i] = load4(wp);
          q.v[i] = load4(wp + P);
        }
      }
    };
    Words cur, nxt, after;
    const int page0 = ask_page(0), page1 = ask_page(1);
    int page = ask_page(2);
    set_up();
    if (steps > 0) ask_words(nxt, 0, page0);
    if (steps > 1) ask_words(after, 1, page1);
    for (int j = 0; j < steps; ++j) {
      cur = nxt;
      nxt = after;
      if (j + 2 < steps) {
        ask_words(after, j + 2, page);
        page = ask_page(j + 3);
      }
      if (j >= 8 && !wait(&ctl.num_free[j & 7], (j >> 3) + 1)) break;
      // Scales are not negative: their bits are in the numbers' order.  (0: nobody sees it.  A
      // zero vector's value scale counts too: its key's score must not decide where the others'
      // weights lie.)
      uint32_t v_top = 0u, v_low = ~0u, k_top = 0u, k_low = ~0u;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t v = cur.v[i] & ~15u, k = cur.k[i] & ~15u;
        if (v && v < 0x7f800000u) {
          v_top = max(v_top, v);
          v_low = min(v_low, v);
        }
        if (BF && k > kZeroScale && k < 0x7f800000u) {
          k_top = max(k_top, k);
          k_low = min(k_low, k);
        }
      }
      v_top = __reduce_max_sync(0xffffffffu, v_top);
      v_low = __reduce_min_sync(0xffffffffu, v_low);
      if (BF) {
        k_top = __reduce_max_sync(0xffffffffu, k_top);
        k_low = __reduce_min_sync(0xffffffffu, k_low);
      }
      const bool wide = v_top > v_low + (V_SPREAD << 23) || (BF && k_top > k_low + (K_SPREAD << 23));
      // 2^lift takes the largest value scale to [1, 2), for bf16 to 2^10 times that
      const int by_top = v_top ? 127 + V_TOP - (int)(v_top >> 23) : 0, lift = wide ? 0 : by_top;
      const float up = __uint_as_float((uint32_t)(127 + lift) << 23);
      Numbers& n = ctl.num[j & 7];
      // bf16: f takes the largest key scale to [1, 2) 2^10
      const int f = wide || !k_top ? 0 : 127 + K_TOP - (int)(k_top >> 23);
      const float kup = __uint_as_float((uint32_t)(127 + f) << 23);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = lane + 32 * i;
        float ks = word_scale(cur.k[i]), vs = word_scale(cur.v[i]) * up;
        if (!BF || wide) {
          const float vk = wide ? vs * (1.f / (1 << V_TOP)) : vs;
          n.fk[t] = BF ? ks : ks * a.scale_log2;
          n.sv[t] = vk;
          if (wide) n.far[t] = fmaxf(log2f(vk), -FAR);
        }
        if (BF) {
          // a value that is not finite must not meet the zero probabilities of rows that do
          // not see it: it counts as 0, and its key makes the score of those that do a NaN
          if (!(vs < INFINITY)) {
            vs = 0.f;
            ks = NAN;
          }
          ks *= kup;
          const __half hi = __float2half_rn(ks);
          const __half2 k2 = __halves2half2(hi, __float2half_rn(ks - __half2float(hi)));
          n.ks[t] = wide ? 0x00003c00u : *reinterpret_cast<const uint32_t*>(&k2);        // 1
          n.vs[t] = __half_as_ushort(__float2half_rn(wide ? (float)(1 << V_TOP) : vs));
        }
        n.zeros[t] = (uint8_t)((cur.k[i] & 15u) | ((cur.v[i] & 15u) << 4));
      }
      const uint32_t there = __ballot_sync(0xffffffffu, cur.codes != 0);
      if (lane < GROUPS) n.codes[lane] = cur.codes;
      if (lane == 0) {
        n.all = {(~there & ((1u << GROUPS) - 1)) | (wide ? WIDE : 0u), (float)lift, up,
                 __uint_as_float((uint32_t)(127 - f) << 23)};
        n.back = __uint_as_float((uint32_t)(127 - min(max(by_top, -64), 64)) << 23);
      }
      __syncwarp();
      if (lane == 0) kq::mbar_arrive(&ctl.num_full[j & 7]);
    }
  } else if (warp >= UNPACK_WARP0) {
    // --------------------------------------------------------- unpacking
    constexpr int TPL = SH::TPL;
    // Lane to (16-byte chunk, token of the load): the 8 lanes of a phase write the two
    // halves of one 128-byte line of 4 tokens, on 8 different chunks of banks.
    const int c = (lane & 1) | (((lane >> 3) & (SH::CH / 2 - 1)) << 1);
    const int ct = ((lane >> 1) & 3) | ((lane / (4 * SH::CH)) << 2);
    // where word k of load i of group 0 goes: (at ^ 16 k) + i (128 TPL), swizzled by the token
    const uint32_t at = kq::smem_u32(kv_smem) + (c >> 1) * (BN * 128) + ct * 128 +
                        (((4 * (c & 1)) ^ (ct & 7)) << 4);
    static_assert(TPL % 8 == 0 || TPL == 4, "the swizzle of a load's tokens");
    auto put = [&](uint32_t base, int i, int k, uint4 v) {
      // (with 4 tokens to a load, every other load's tokens are 4 .. 7 of a line of 8)
      const uint32_t p = ((base ^ (16u * k)) ^ (TPL == 4 && (i & 1) ? 64u : 0u)) + i * (128 * TPL);
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                   : "memory");
    };
    struct Codes {
      uint4 c[SH::LOADS];
    };
    // job n: step n / 4, keys (n & 2 == 0) or values, half n & 1 of the step
    static_assert(JOBS == 2 && JOB == 2 * GROUP, "four jobs to a step, two pages to a job");
    const int jobs = 2 * JOBS * steps;
    const int64_t vrel = (int64_t)a.cache.P * (D / 2);
    auto ask = [&](Codes& q, int n) -> bool {
      const int j = n >> 2, g = n & 1;
      if (!wait(&ctl.num_full[j & 7], j >> 3)) return false;
      const Numbers& num = ctl.num[j & 7];
      const int64_t rel = (n & 2 ? vrel : 0) + ct * (D / 2) + 16 * c;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint64_t p = num.codes[2 * g + h];
#pragma unroll
        for (int i = h * (SH::LOADS / 2); i < (h + 1) * (SH::LOADS / 2); ++i) {
          q.c[i] = make_uint4(0u, 0u, 0u, 0u);
          if (p)
            load16(q.c[i], reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(p) + rel +
                                                          (i - h * (SH::LOADS / 2)) * (TPL * (D / 2))));
        }
      }
      return true;
    };
    Codes cur, nxt;
    int n = warp - UNPACK_WARP0;
    bool ok = n < jobs && warp < UNPACK_WARP0 + UNPACKERS && ask(nxt, n);
    for (; n < jobs && ok; n += UNPACKERS) {
      const int j = n >> 2, g = n & 1, st = j & SM;
      cur = nxt;
      const bool values = n & 2;
      // (these keys' numbers stay until the step's softmax, which waits for this job)
      const Numbers& num = ctl.num[j & 7];
      uint32_t zeros[SH::LOADS], scale[SH::LOADS];
#pragma unroll
      for (int i = 0; i < SH::LOADS; ++i) {
        const int t = JOB * g + i * TPL + ct;
        zeros[i] = num.zeros[t];
        scale[i] = !BF ? 0u : values ? num.vs[t] : num.ks[t];
      }
      if (n + UNPACKERS < jobs) ok = ask(nxt, n + UNPACKERS);
      if (j >= STAGES) ok = ok && wait(values ? &ctl.v_empty[st] : &ctl.k_empty[st], (j >> LG) + 1);
      if (!ok) break;
      const uint32_t dst = at + g * (JOB * 128) + st * SH::STAGE + (values ? SH::KV_BYTES : 0);
      auto unpack = [&](bool of_values) {
#pragma unroll
        for (int i = 0; i < SH::LOADS; ++i) {
          const uint32_t z = of_values ? zeros[i] >> 4 : zeros[i] & 15u;
          const uint32_t z1 = 0x64006400u + z * 0x00010001u, z2 = 0xd400d400u + z * 0x00100010u;
          const uint32_t hi = __byte_perm(scale[i], 0, 0x1010), lo = __byte_perm(scale[i], 0, 0x3232);
          const uint32_t w[4] = {cur.c[i].x, cur.c[i].y, cur.c[i].z, cur.c[i].w};
          if (!BF) {
#pragma unroll
            for (int k = 0; k < 4; ++k) put(dst, i, k, codes_f16(w[k], z1, z2));
          } else if (of_values) {
#pragma unroll
            for (int k = 0; k < 4; ++k) put(dst, i, k, scaled(codes_f16(w[k], z1, z2), hi));
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) put(dst, i, k, scaled(codes_f16(w[k], z1, z2), hi, lo));
          }
        }
      };
      // (heads of 256, bf16: unpacking keys bounds the step, and a copy of the code for either
      // operand is the faster one: 602 us against 652 for two prompts of 1024 over 6000.  Heads
      // of 128 lose 1 % by it, fp16 at 256 14 %.)
      if (!(BF && D == 256))
        unpack(values);
      else if (values)
        unpack(true);
      else
        unpack(false);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        kq::mbar_arrive(values ? &ctl.v_full[st] : &ctl.k_full[st]);
        if (values) kq::mbar_arrive(&ctl.num_free[j & 7]);
      }
    }
  } else if (warp < 4 * tiles * SH::HALVES) {
    // ---------------------------------------------------------- softmax
    // (one tile: two warps share their rows, a half of each step's keys to either, and agree
    // by a barrier of their own on the maximum and on giving up)
    constexpr int HALVES = SH::HALVES, COLS = BN / HALVES;
    const int tile = NT == 2 ? warp >> 2 : 0, part = NT == 2 ? 0 : warp >> 2, bar = 1 + (warp & 3);
    const int tr = (warp & 3) * 32 + lane;              // row within the tile
    const uint32_t tbase = ctl.tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t o_at = tbase + SH::O_COL + tile * D;
    bool ok = wait(&ctl.q_full, 0);
    const float row = BF ? ctl.row[128 * tile + tr] : 0.f;
    const int r = min(last, r0 + 128 * tile + tr);
    const int qi = r / a.g;
    const int lo = lo_of(qi), hi = hi_of(qi);
    // what all rows of the warp see (rows are in order)
    const int all_lo = lo_of(__shfl_sync(0xffffffffu, qi, 31)), all_hi = hi_of(__shfl_sync(0xffffffffu, qi, 0));
    // the running maximum, a whole number; 0 until the row has seen a key
    float m = 0.f;
    // the sum of probabilities, relative to 2^m / back: O's unit follows the weights, and a weight
    // of a scale of 2^100 would push other keys' probabilities out of fp32
    float l = 0.f, back = 0.f, back_max = 0.f;        // back: 0 until a key is seen; back_max: of the warp's rows
    // how far weights may pass the maximum
    auto lag = [&]() { return back > 0.f ? LAG : -0x1.fffffep127f; };
    bool stop = false;
    // Two warps to a row: the larger of their maxima.  Also the only way out of the steps, for
    // both at once: neither waits in vain.
    auto agree = [&](float& high) {
      ctl.pair[part][tr] = make_float2(high, ok ? 1.f : 0.f);
      pair_sync(bar);
      const float2 other = ctl.pair[part ^ 1][tr];
      high = max3(high, other.x, other.x);
      stop = !__all_sync(0xffffffffu, ok && other.y != 0.f);
      ok = ok && !stop;
    };
    // The maximum moves by a whole number; what was summed before turns by a power of two.
    auto move = [&](float high, float to_back, int j) -> float {
      const bool up = high > lag();
      const float by = up ? (high < INFINITY ? ceilf(high) - BASE : high) : 0.f;
      const float al = up && back > 0.f ? exp2_approx(-by) : 1.f;
      if (up) {
        if (back > 0.f) l *= al * (to_back / back);
        back = to_back;
      }
      back_max = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(back)));
      m += by;
      if (j > 0) {
        ok = wait(&ctl.pv_done[tile], j - 1) && ok;
        kq::tc_fence_after();
#pragma unroll 1
        for (int d = part * (D / HALVES); d < (part + 1) * (D / HALVES); d += 16) {
          uint32_t o[16];
          tmem_ld16(o_at + d, o);
          kq::tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * al);
          tmem_st16(o_at + d, o);
        }
      }
      return by;
    };
    // Any step, slowly: masks and per-key numbers always, l's terms for themselves, scores read
    // twice to hold few of them.
    auto any_step = [&](int j, int key0, const Numbers::All& all) {
      const uint32_t s_at = tbase + (2 * tile + (j & 1)) * BN;
      const Numbers& num = ctl.num[j & 7];
      const uint32_t gone = all.absent;
      const bool wide = gone & WIDE, by_key = !BF || wide;
      const float to_x = BF ? row * all.down : 1.f, m0 = m + all.lift;
      float by = 0.f;
      auto scores = [&](int k0, float (&y)[16]) {
        uint32_t x[16];
        tmem_ld16(s_at + k0, x);
        kq::tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int key = key0 + k0 + k;
          const bool seen = !((gone >> (k0 >> 4)) & 1u) && key < hi && (key >= lo || key < a.sinks);
          y[k] = seen ? fmaf(__uint_as_float(x[k]), by_key ? num.fk[k0 + k] * to_x : to_x, -m0) - by : -INFINITY;
        }
      };
      float high = -INFINITY;
#pragma unroll 1
      for (int k0 = COLS * part; k0 < COLS * (part + 1); k0 += 16) {
        float y[16];
        scores(k0, y);
#pragma unroll
        for (int k = 0; k < 16; ++k) high = fmaxf(high, wide ? y[k] + num.far[k0 + k] : y[k]);
      }
      if constexpr (HALVES == 2) {
        pair_sync(bar);        // (the other has read what was told in the step before)
        agree(high);
        if (stop) return;
      }
      if (HALVES == 2 || __any_sync(0xffffffffu, high > lag())) by = move(high, num.back, j);
      const float far = all.lift + exponent(back);
#pragma unroll 1
      for (int k0 = COLS * part; k0 < COLS * (part + 1); k0 += 32) {
        uint32_t pk[16];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float y[16];
          scores(k0 + 16 * c, y);
          float w[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            l += exp2_approx(y[k] + far);
            w[k] = y[k] == -INFINITY ? 0.f : exp2_approx(y[k]) * (by_key ? num.sv[k0 + 16 * c + k] : 1.f);   // (0 times a NaN)
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) pk[8 * c + k] = pack_half2(w[2 * k], w[2 * k + 1]);
        }
        if (HALVES == 2) pair_sync(bar);       // (P of the second half goes over scores of the first)
        tmem_st16(s_at + (k0 >> 1), pk);
      }
    };
    auto step = [&](auto is_masked, int j, int key0, const Numbers::All& all) {
      constexpr bool masked = decltype(is_masked)::value;
      const uint32_t s_at = tbase + (2 * tile + (j & 1)) * BN;
      const Numbers& num = ctl.num[j & 7];
      const uint32_t gone = masked ? all.absent : 0u;
      f32x2 t[COLS / 2];           // scores less lift and the running maximum
      float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      const float less = -m - all.lift, to_x = BF ? row * all.down : 0.f;
      const f32x2 neg_m = pack2(less, less), row2 = pack2(to_x, to_x);
      float xs[COLS / 32][32];
#pragma unroll
      for (int h = 0; h < COLS / 32; ++h) kq::tmem_ld32(s_at + 32 * (h + part), xs[h]);
      kq::tmem_wait_ld();
#pragma unroll
      for (int h = 0; h < COLS / 32; ++h) {
        const int hp = h + part;   // the half of the step's keys
        const float(&x)[32] = xs[h];
        const ulonglong2* fk = reinterpret_cast<const ulonglong2*>(&num.fk[32 * hp]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const ulonglong2 f = BF ? make_ulonglong2(row2, row2) : fk[i];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int e = 4 * i + 2 * k;
            f32x2& tc = t[16 * h + 2 * i + k];
            tc = fma2(pack2(x[e], x[e + 1]), k ? f.y : f.x, neg_m);
            float2 v = unpack2(tc);
            if constexpr (masked) {
              const int key = key0 + 32 * hp + e;
              const bool page = !((gone >> (2 * hp + (e >> 4))) & 1u);
              if (!(page && key < hi && (key >= lo || key < a.sinks))) v.x = -INFINITY;
              if (!(page && key + 1 < hi && (key + 1 >= lo || key + 1 < a.sinks))) v.y = -INFINITY;
              tc = pack2(v.x, v.y);
            }
            top[i & 3] = max3(top[i & 3], v.x, v.y);
          }
        }
      }
      float high = max3(max3(top[0], top[1], top[2]), top[3], top[3]);
      const bool moves = high > lag();
      // (two warps to a row: also before either writes P over scores of the other)
      if (HALVES == 2 ? pair_or(bar, moves || !ok) : __any_sync(0xffffffffu, moves)) {
        if constexpr (HALVES == 2) {
          agree(high);
          if (stop) return;
        }
        const float by = move(high, num.back, j);
        const f32x2 down = pack2(-by, -by);
#pragma unroll
        for (int k = 0; k < COLS / 2; ++k) t[k] = add2(t[k], down);
      }
      const ulonglong2* sv = reinterpret_cast<const ulonglong2*>(num.sv);
      f32x2 sum[2] = {pack2(0.f, 0.f), pack2(0.f, 0.f)};
      const float to_l = all.up * back;
#pragma unroll
      for (int h = 0; h < COLS / 32; ++h) {
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const ulonglong2 f = BF ? make_ulonglong2(0ull, 0ull) : sv[8 * (h + part) + i];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float2 v = unpack2(t[16 * h + 2 * i + k]);
            const f32x2 p = pack2(exp2_approx(v.x), exp2_approx(v.y));
            sum[k] = add2(sum[k], p);
            float2 w = unpack2(BF ? p : mul2(p, k ? f.y : f.x));
            if constexpr (masked && !BF) {                     // (0 times a NaN scale)
              if (v.x == -INFINITY) w.x = 0.f;
              if (v.y == -INFINITY) w.y = 0.f;
            }
            pk[2 * i + k] = pack_half2(w.x, w.y);
          }
        }
        tmem_st16(s_at + 16 * (h + part), pk);
      }
      const float2 ls = unpack2(add2(sum[0], sum[1]));
      l = fmaf(ls.x + ls.y, to_l, l);
    };
    for (int j = 0; j < steps; ++j) {
      ok = ok && wait(&ctl.s_full[tile][j & 1], j >> 1);
      // (of two warps to a row, one that gives up tells the other in step)
      if (HALVES == 1 && !ok) break;
      kq::tc_fence_after();
      const int key0 = key_of(i0 + j);
      const Numbers::All all = ctl.num[j & 7].all;
      // (probabilities that lie far below their place among l's need exponentials of their own)
      // (which of the three copies comes first decides how the compiler lays out the others: 2 x
      // 2048 tokens over 16k, heads of 128, bf16 1267 us this way round, 1399 the other; fp16
      // 1433 and 1380; heads of 64, 2 x 1500 over 6000, 329 and 321)
      if constexpr (BF && D >= 128) {
        if ((all.absent & WIDE) || all.up * back_max > 0x1p30f)
          any_step(j, key0, all);
        else if (!all.absent && key0 + BN <= all_hi && (key0 >= all_lo || key0 + BN <= a.sinks))
          step(std::false_type{}, j, key0, all);
        else
          step(std::true_type{}, j, key0, all);
      } else {
        const bool slow = (all.absent & WIDE) || all.up * back_max > 0x1p30f;
        if (!slow && !all.absent && key0 + BN <= all_hi && (key0 >= all_lo || key0 + BN <= a.sinks))
          step(std::false_type{}, j, key0, all);
        else if (slow)
          any_step(j, key0, all);
        else
          step(std::true_type{}, j, key0, all);
      }
      if (HALVES == 2 && stop) break;
      kq::tmem_wait_st();
      kq::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        kq::mbar_arrive(&ctl.p_ready[tile][j & 1]);
        kq::mbar_arrive(&ctl.num_free[j & 7]);
      }
    }
    // ---- output
    if constexpr (HALVES == 2) {
      pair_sync(bar);
      ctl.pair[part][tr].x = l;
      pair_sync(bar);
      const float other = ctl.pair[part ^ 1][tr].x;
      l = part ? other + l : l + other;
    }
    if (steps > 0) ok = ok && wait(&ctl.o_full, 0);
    kq::tc_fence_after();
    const int row_in = ctl.unit.tile * R + 128 * tile + tr, to_head = ctl.unit.head;
    const bool mine = row_in < ctl.seq.n * a.g;
    const int64_t slot = ((int64_t)ctl.unit.slot * a.cache.heads + to_head) * R + 128 * tile + tr;
    const int to_q = row_in / a.g, hq = to_head * a.g + row_in - to_q * a.g, out_row = ctl.seq.row0 + to_q;
    const bool split = ctl.unit.nsplit > 1;
    if (ok) {
      // Through shared memory (the queries and what lies behind them are not needed any more),
      // so that a warp stores whole rows: a thread has a row, and rows are far apart.  Each
      // warp has its own 32 rows of DP floats; chunk c of 4 of row t lies at c ^ (t & 7).
      static_assert(SH::Q_BYTES + SH::STAGES * SH::STAGE >= R * D * 4, "room for the output");
      constexpr int DP = D / HALVES;                   // dims of this warp's
      float* buf = reinterpret_cast<float*>(q_smem) + warp * 32 * DP;
      const float f = split ? back : l == 0.f ? 0.f : back / l;
      m -= exponent(back);
#pragma unroll 1
      for (int d = 0; d < DP; d += 32) {
        uint32_t o[32];
        if (steps > 0) {
          tmem_ld16(o_at + part * DP + d, reinterpret_cast<uint32_t(&)[16]>(o[0]));
          tmem_ld16(o_at + part * DP + d + 16, reinterpret_cast<uint32_t(&)[16]>(o[16]));
          kq::tmem_wait_ld();
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0u;
        }
#pragma unroll
        for (int k = 0; k < 32; k += 4) {
          // dims 8 (k / 8) + 0..3 are columns 0 2 4 6 of the 8, dims 4..7 columns 1 3 5 7
          const int b = (k & 24) + ((k >> 2) & 1);
          *reinterpret_cast<float4*>(buf + lane * DP + 4 * (((d + k) >> 2) ^ (lane & 7))) =
              make_float4(__uint_as_float(o[b]) * f, __uint_as_float(o[b + 2]) * f,
                          __uint_as_float(o[b + 4]) * f, __uint_as_float(o[b + 6]) * f);
        }
      }
      // where the lane's row goes
      uint64_t to = 0;
      if (mine && split) to = reinterpret_cast<uint64_t>(a.part_o + slot * D + part * DP);
      if (mine && !split)
        to = reinterpret_cast<uint64_t>(static_cast<uint16_t*>(a.out) + (int64_t)out_row * a.o_st +
                                        (int64_t)hq * a.o_sh + part * DP);
      if (mine && split && part == 0) a.part_ml[slot] = {back > 0.f ? m : NO_MAX, l};
      if (mine && !split && part == 0 && a.lse)
        a.lse[(int64_t)out_row * a.Hq + hq] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
      __syncwarp();
      constexpr int CHUNKS = DP / 4;
      auto store = [&](auto is_split) {
#pragma unroll 1
        for (int i = 0; i < DP / 4; i += 8) {
          float4 x[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int t = ((i + k) * 32 + lane) / CHUNKS, c = ((i + k) * 32 + lane) % CHUNKS;
            x[k] = *reinterpret_cast<const float4*>(buf + t * DP + 4 * (c ^ (t & 7)));
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int t = ((i + k) * 32 + lane) / CHUNKS, c = ((i + k) * 32 + lane) % CHUNKS;
            const uint64_t p = __shfl_sync(0xffffffffu, (unsigned long long)to, t);
            if (!p) continue;
            if constexpr (decltype(is_split)::value)
              reinterpret_cast<float4*>(p)[c] = x[k];
            else
              reinterpret_cast<uint2*>(p)[c] = pack4(x[k], BF ? BF16 : FP16);
          }
        }
      };
      if (split)
        store(std::true_type{});
      else
        store(std::false_type{});
    }
  }
  kq::tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP0) {
    kq::tc_fence_after();
    kq::tmem_dealloc(ctl.tmem, 512);
  }
}

template <int D, bool BF>
int launch(const AttendArgs& a, cudaStream_t st) {
  using SH = Shape<D>;
  const long long grid = max_units(a, SH::R, prompt_block(D));
  if (grid > INT32_MAX) return KRONQ_ERR_UNSUPPORTED;
  static kqh::PerDevice attr;
  if (kqh::smem_attr_once(attr, kv4_prompt_kernel<D, BF>, SH::SMEM) <= 0) return KRONQ_ERR_CUDA;
  kv4_prompt_kernel<D, BF><<<(unsigned)grid, THREADS, SH::SMEM, st>>>(a);
  KQ_CHECK_LAUNCH();
  return KRONQ_OK;
}

}  // namespace

int prompt_rows(int D) { return D == 256 ? Shape<256>::R : Shape<128>::R; }
int prompt_block(int D) { return BN; }

int launch_prompt(const AttendArgs& a, int D, cudaStream_t st) {
  if (D == 64) return a.dt == BF16 ? launch<64, true>(a, st) : launch<64, false>(a, st);
  if (D == 128) return a.dt == BF16 ? launch<128, true>(a, st) : launch<128, false>(a, st);
  return a.dt == BF16 ? launch<256, true>(a, st) : launch<256, false>(a, st);
}

}  // namespace kv4
