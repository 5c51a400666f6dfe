// Attention of new queries over the paged 4-bit cache, few query rows per key:
// one pass over the codes with the running maximum and sum of the softmax.
//
//   x_rj = scale log2(e) s_j (sum_d q_rd c_jd - z_j sum_d q_rd)
//   o_r  = sum_j 2^(x_rj - m_r) s'_j (c'_jd - z'_j) / sum_j 2^(x_rj - m_r)
//
// (s, z, c: scale, zero point and codes of key j; primed of value j).  Scales
// and zero points are per token, so they are taken out of both products: the
// tensor cores multiply the bare codes, and 128 codes of a token cost one scale.
//
// What bounds it is not the copy but the chain of a warp's step, from codes to operands
// to scores to probabilities to products: at 16 warps per SM the schedulers issue in 57 % of
// their cycles and no pipe is busier (integer 55, tensor 30, memory 54), and the stalls are
// fixed latencies.  So operands are made with few instructions.  A code in the low bits of a half is the subnormal c 2^-24 (c 2^-20
// four bits up), exact in fp16 x fp16 -> fp32 products, so:
//   keys    unpacking is one AND per two codes and one shift per four pairs; the
//           factors 16 of every other pair go into the queries' fragments;
//   values  the tokens of a dim come together by ldmatrix.trans on bytes (two dims);
//           a byte taken whole is c_even + 16 c_odd, which saves a mask: the odd
//           dim is the difference, taken once at the end.
// (8-bit operands would halve the unpacking: 0000cccc is an e4m3 number and a u8.
// mma.sync on e4m3 is two fp16 MMAs and conversions on this machine, measured 1.6
// times slower over all; on s8 it runs at the fp16 instruction rate, with queries in
// two terms and two sums to convert.)
//
// S^T = K Q^T and O^T = V^T P^T: keys (or dims) are the 16 rows of the MMA and the
// query rows of one key/value head the 8 columns, so a group of 8 or fewer query
// heads wastes none of the code operand.  (A tensor-memory accumulator of 128 lanes
// would be filled the same way, but its operand has to be written to shared or
// tensor memory after unpacking; here the unpacked words are the fragment.)  Between
// the two products the 8 x 8 blocks of probabilities are turned with movmatrix.
//
// One block = one (sequence, tile of 8 NT rows, split of its keys) of one
// key/value head; warp w takes keys 32 w .. of every 128 through a ring of its
// own in shared memory, filled by cp.async two steps ahead: no barrier between
// warps, and some 130 KB in flight per SM.  (Bulk copies from one lane cost
// more: 89 against 20 issued instructions per 16 tokens.)  The running maximum
// is only moved when a weight passes it by 2^5 (all lanes of a column agree by
// vote), so most steps have no cross-lane reduction.
//
// Measured (heads of 128, cold cache): 64 sequences of 4k to 8k tokens, 8 query heads
// a key/value head, bf16: 102 us at an SM clock of 1875 MHz, 4.2 TB/s of codes and words; 4
// sequences of 105k to 131k tokens, 4 query heads, fp16: 116 us at 1760 MHz, 4.6 TB/s (of 6.55
// that a copy moves).  One sequence of 8k is latency: 12.6 us for the two launches.
#include <type_traits>

#include "kv4_attend.cuh"

namespace kv4 {
namespace {

constexpr int THREADS = 128, WARPS = 4, BLK = 128, STEP = BLK / WARPS;

KQ_DEV void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                     uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two 16 x 16 byte blocks (lane l: row l % 16 of block l / 16), turned: register
// 2 i + j of lane (gr, t) holds column 8 j + gr, rows 4t .. 4t + 3 of block i.
KQ_DEV void ldmatrix_turned(uint32_t (&r)[4], uint32_t p) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(p));
}

KQ_DEV uint32_t turn8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

KQ_DEV float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// 2^(x/2).  Maxima follow weights, so where one part saw a value of 10^37 they are 2^100 apart,
// and sums of probabilities that count take a factor that no fp32 number holds: it is applied
// in two halves.
KQ_DEV float exp2_half(float x) { return exp2_approx(0.5f * x); }

// (in rules on ranges only)
KQ_DEV float log2_approx(float x) {
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

KQ_DEV uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

KQ_DEV void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
KQ_DEV void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
KQ_DEV void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int N>
KQ_DEV void lds_words(uint32_t* w, uint32_t p) {
  if constexpr (N == 1)
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(p));
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(p));
  else
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(p));
}

// A step's 32 tokens in shared memory: key codes, value codes (32 x D/2 bytes
// each, in 128-byte lines whose 16-byte chunks are swizzled by the token so that
// neither read has bank conflicts), key words, value words.  They are multiplied
// as two halves of 16.
//
// Probabilities come out of the turn as pairs of neighbouring rows of S and meet
// the values' tokens 4t .. 4t + 3 in lane (gr, t), so row r of the first 8 rows of S
// is the key 4 (r >> 1) + (r & 1), row r of the second 8 the key two tokens on.
// Lane (gr, t) reads D/4 dims of these two keys for row gr.
template <int D>
struct Step {
  static constexpr int TOK = D / 2;                 // bytes of a token's codes
  static constexpr int V = STEP * TOK, KWORDS = 2 * V, VWORDS = KWORDS + 4 * STEP;
  static constexpr int BYTES = VWORDS + 4 * STEP;
  static constexpr int KW = D / 32;                 // key words per lane and token
  static constexpr int VC = D / 32;                 // 16-byte chunks of a token's values
  static constexpr int KLOADS = KW > 4 ? 2 : 1;     // 64 bytes apart: a quad reads 64 at once

  // byte offsets of 16-byte chunk c of the keys, of the values
  KQ_DEV static int key_at(int c) {
    const int tok = c / VC;
    const int x = D == 256 ? 4 * (tok & 1) : D == 128 ? 0 : 4 * ((tok >> 2) & 1);
    return (c ^ x) * 16;
  }
  KQ_DEV static int value_at(int c) {
    const int tok = c / VC;
    const int x = D == 256 ? tok & 7 : D == 128 ? (tok >> 1) & 3 : (tok >> 2) & 1;
    return V + (c ^ x) * 16;
  }
  // where lane (gr, t) reads its first key token (load i of KLOADS); the second
  KQ_DEV static int key_lane(int gr, int t, int i) {
    const int tok = 4 * (gr >> 1) + (gr & 1);
    const int at = tok * TOK + (KLOADS == 2 ? 16 * (t + 4 * i) : t * (D / 8));
    return key_at(at / 16) + at % 16;
  }
  KQ_DEV static int second_key(int off) {
    if constexpr (D == 64) return off ^ 64;         // 2 tokens of 32 bytes: the line's other half
    return off + 2 * TOK;
  }
  // dims of word w of lane t's keys
  KQ_DEV static int key_dim(int t, int w) {
    return KLOADS == 2 ? 32 * (t + 4 * (w >> 2)) + 8 * (w & 3) : t * (D / 4) + 8 * w;
  }
};

// The next 16 steps of a warp: where their halves lie (0: nowhere), and for the last
// 32 steps the first token with flags in its low bits.
struct Plan {
  uint64_t codes[16][2], words[16][2];
  uint32_t first[32];      // token | halves present (1, 2) | some row does not see some key (4)
};

// chunk c (4 floats) of row r of the joining buffer is stored at c ^ this: the 16
// lanes of a phase store 8 floats to each of 4 rows, 2 rows apart
KQ_DEV int join_swizzle(int r) { return 2 * ((r >> 1) & 3); }

// The running maximum before there is one: finite, so that a row that has seen no
// key has sums of 0 and weights of 2^(NO_MAX - max) = 0 or 1, never a NaN.
constexpr float NO_MAX = -0x1p127f;

// Where a row's numbers lie.  With m the row's running maximum, p = 2^(x - m) is summed in
// fp32, and p s' 2^-LIFT, the weight of a value's codes, is what fp16 has to hold.  So m follows
// the largest weight, not the largest score: a new one is put at 2^BASE, and m moves when one
// passes 2^LAG.  It belongs to the row alone: value vectors far larger than the rest do not
// push the rest out of fp16's range in rows that do not see them.  Weights below 2^-35 of the
// row's largest are lost.  LIFT keeps p normal where scales are large (p of a key with scale 2^100
// is 2^(BASE + LIFT - 100) at most); FAR bounds p where they are tiny (zero vectors have
// 2^-100): a score counts at least as a weight 2^FAR below it.
constexpr float BASE = 10.f, LAG = 15.f, LIFT = 8.f, FAR = 80.f;

constexpr int RING = 3;
constexpr int FLUSH = 4;      // steps between subtractions of the zero points' part

// FINE (fp16 outputs): probabilities in two fp16 terms.  One is off by 2^-11, as much as
// the output's own rounding, and the two add up to 1.4 times its error; for bf16 outputs
// it is an eighth of theirs.  A tile of 4 rows has them twice, in the MMA's columns 0 .. 3
// and 4 .. 7: all of a column but its second product is alike, and that one takes the
// second terms; a larger tile takes the product twice.  4 x 128k, 4 query heads, side
// by side: 102 us with one term, 105 in two columns, 119 with two products.
enum Terms { ONE, TWO_COLUMNS, TWO_PRODUCTS };
template <int D, int NT, int TERMS>
__global__ void __launch_bounds__(THREADS, D <= 128 && NT == 1 ? 4 : 2) kv4_attend_kernel(const AttendArgs a) {
  constexpr int ROWS = 8 * NT, R = TERMS == TWO_COLUMNS ? 4 : ROWS;     // columns of the MMAs, rows of a tile
  using SP = Step<D>;
  constexpr int KW = SP::KW, MT = D / 16;
  extern __shared__ __align__(128) uint8_t smem[];   // the warps' rings; then [WARPS][ROWS][D] floats
  float* merge_o = reinterpret_cast<float*>(smem);
  __shared__ float merge_ml[WARPS][ROWS][2];
  __shared__ __align__(16) Plan plans[WARPS];

  Unit u;
  if (!find_unit<R, BLK, THREADS>(a, &u)) return;
  const int head = u.head;
  const Seq s = seq_of(a, u.b, nullptr);
  if (threadIdx.x == 0 && head == 0 && u.tile == 0 && u.split == 0)
    a.meta[u.b] = make_int2(u.slot, u.nsplit);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gr = lane >> 2, t = lane & 3;
  const int rows = s.n * a.g, r0 = u.tile * R;
  const int last = min(rows, r0 + R) - 1;
  const int gq = TERMS == TWO_COLUMNS ? gr & 3 : gr;   // this lane's row of the tile (and + 8)
  int qi[NT];                                       // query of this lane's row (rows behind: the last)
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) qi[nt] = min(last, r0 + 8 * nt + gq) / a.g;
  const int q0 = __shfl_sync(0xffffffffu, qi[0], 0), q1 = last / a.g;
  const Span sp = span_of<BLK>(a, s, q0, q1);
  const int per = ceil_div(sp.nb, u.nsplit);
  const int i0 = u.split * per, i1 = min(sp.nb, i0 + per);

  // the keys each column's row sees: j < chi and (j >= clo or j < sinks); what all
  // of the tile's rows see, and what one of them sees (rows are in order)
  int clo[NT][2], chi[NT][2];
  auto lo_of = [&](int q) { return a.window ? max(0, s.L - s.n + q - a.window + 1) : 0; };
  auto hi_of = [&](int q) { return max(0, a.causal ? min(s.L, s.L - s.n + q + 1) : s.L); };
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int q = __shfl_sync(0xffffffffu, qi[nt], (2 * t + c) * 4);
      chi[nt][c] = hi_of(q);
      clo[nt][c] = lo_of(q);
    }
  const int all_lo = lo_of(q1), all_hi = hi_of(q0), any_lo = lo_of(q0), any_hi = hi_of(q1);

  // ---- keys: the warp's steps are its 32 tokens of every block i0 .. i1 - 1
  const int steps = i1 > i0 ? i1 - i0 : 0;
  const uint32_t ring = kq::smem_u32(smem) + warp * (RING * SP::BYTES);
  Plan& plan = plans[warp];
  auto look_ahead = [&](int st) {        // plans steps st .. st + 15, a half per lane
    const int s1 = st + (lane >> 1);
    const int i = i0 + s1;
    const int j0 = (i < sp.sb ? i : sp.lb + i - sp.sb) * BLK + STEP * warp;
    const int j = j0 + 16 * (lane & 1);
    int64_t page = -1;
    if (s1 < steps && j < any_hi && (j + 16 > any_lo || j < a.sinks)) {
      page = a.b.table[u.b * a.b.table_ld + (j >> a.cache.lgP)];
      if (page < 0 || page >= a.cache.pages) {
        kq::record_error(a.info, KRONQ_ERR_INVALID_ARG);
        page = -1;
      }
    }
    const int P = a.cache.P, slot = j & (P - 1);
    const uint8_t* blk = a.cache.base + (page * a.cache.heads + head) * a.cache.block_bytes;
    const uint32_t both = __ballot_sync(0xffffffffu, page >= 0);
    const uint32_t here = (both >> (lane & ~1)) & 3u;
    plan.codes[s1 & 15][lane & 1] = page >= 0 ? (uint64_t)(blk + slot * SP::TOK) : 0;
    plan.words[s1 & 15][lane & 1] = page >= 0 ? (uint64_t)(blk + P * D + slot * 4) : 0;
    const bool masked = here != 3u || !(j0 + STEP <= all_hi && (j0 >= all_lo || j0 + STEP <= a.sinks));
    if (!(lane & 1)) plan.first[s1 & 31] = (uint32_t)j0 | here | (masked ? 4u : 0u);
    __syncwarp();
  };
  const int vrel = a.cache.P * SP::TOK;                 // value codes behind key codes
  // of the words, lane 8 i + 4 h + c copies chunk c of half h of the keys' (i = 0)
  // or values' (i = 1)
  const int word_half = (lane >> 2) & 1;
  const int wrel = ((lane >> 3) & 1) * a.cache.P * 4 + (lane & 3) * 16;
  auto fetch = [&](int st, uint32_t dst) {      // step st into the stage at dst
    if (st < steps) {
      if ((st & 15) == 0) look_ahead(st);
      const ulonglong2 at = *reinterpret_cast<const ulonglong2*>(plan.codes[st & 15]);
      const uint64_t w = plan.words[st & 15][word_half];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint64_t p = h ? at.y : at.x;
        if (p) {
          const uint8_t* kp = reinterpret_cast<const uint8_t*>(p) + lane * 16;
          const uint8_t* vp = kp + vrel;
#pragma unroll
          for (int c = 0; c < 16 * SP::TOK; c += 512) {
            const int chunk = h * SP::TOK + c / 16 + lane;
            copy16(dst + SP::key_at(chunk), kp + c);
            copy16(dst + SP::value_at(chunk), vp + c);
          }
        }
      }
      if (lane < 16 && w) copy16(dst + SP::KWORDS + lane * 16, reinterpret_cast<const uint8_t*>(w) + wrel);
    }
    copy_commit();
  };
#pragma unroll
  for (int k = 0; k < RING - 1; ++k) fetch(k, ring + k * SP::BYTES);

  // ---- queries: fp16 fragments of q 2^e (e per row: the largest becomes about
  // 2^10, so bf16's range is kept and so are 20 binades below the row's largest)
  uint32_t qf[NT][KW][4];
  float qsum[NT][2], qmul[NT][2];        // of columns 2t, 2t + 1
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = r0 + 8 * nt + gq;
    float x[KW][8];
    float big = 0.f, sum = 0.f;
    if (r < rows) {
      const uint16_t* p = a.q + (int64_t)(s.row0 + qi[nt]) * a.q_st +
                          (int64_t)(head * a.g + r - qi[nt] * a.g) * a.q_sh;
#pragma unroll
      for (int w = 0; w < KW; ++w) load8(p + SP::key_dim(t, w), a.q_vec, a.dt, x[w]);
#pragma unroll
      for (int w = 0; w < KW; ++w)
#pragma unroll
        for (int j = 0; j < 8; ++j) big = fmaxf(big, fabsf(x[w][j]));
    } else {
#pragma unroll
      for (int w = 0; w < KW; ++w)
#pragma unroll
        for (int j = 0; j < 8; ++j) x[w][j] = 0.f;
    }
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
    const int e = min(max(137 - (int)(__float_as_uint(big) >> 23), -126), 126);
    const float up = __uint_as_float((uint32_t)(127 + e) << 23);
    const float down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
    for (int w = 0; w < KW; ++w) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[w][j] *= up;
        sum += x[w][j];
      }
      qf[nt][w][0] = pack_half2(x[w][0], x[w][4]);
      qf[nt][w][1] = pack_half2(x[w][1] * 0.0625f, x[w][5] * 0.0625f);
      qf[nt][w][2] = pack_half2(x[w][2], x[w][6]);
      qf[nt][w][3] = pack_half2(x[w][3] * 0.0625f, x[w][7] * 0.0625f);
    }
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    sum *= -0x1p-24f;
    const float mul = a.scale_log2 * down * 0x1p24f;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      qsum[nt][c] = __shfl_sync(0xffffffffu, sum, (2 * t + c) * 4);
      qmul[nt][c] = __shfl_sync(0xffffffffu, mul, (2 * t + c) * 4);
    }
  }

  // o: tile i's sums of p s' c over dim 16 i + 2 gr (0, 1) and of p s' (c + 16 c of the next
  // dim) (2, 3), for columns 2t, 2t + 1; z: sums of p s' z'
  float o[NT][MT][4], z[NT][4];
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[nt][i][j] = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) z[nt][j] = 0.f;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      m[nt][c] = NO_MAX;        // the running maximum
      l[nt][c] = 0.f;
    }
  }
  // the sums of codes and of zero points nearly cancel (values are centred), and
  // the tensor core rounds its sum towards zero: keep the difference small
  auto flush = [&]() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          o[nt][i][c] -= z[nt][c];
          o[nt][i][2 + c] = fmaf(z[nt][c], -17.f, o[nt][i][2 + c]);
        }
        z[nt][c] = 0.f;
      }
  };

  // byte offsets within a stage of what this lane reads
  const int tok = 4 * (gr >> 1) + (gr & 1);         // its keys: tok + 16 h + 2 k
  int koff[SP::KLOADS];
#pragma unroll
  for (int i = 0; i < SP::KLOADS; ++i) koff[i] = SP::key_lane(gr, t, i);
  const int voff = SP::value_at((lane & 15) * SP::VC + (lane >> 4));
  // one step: two copies of the code, so that steps with every key seen by every
  // row (all but those at the ends) carry no selections
  auto multiply = [&](auto is_masked, uint32_t stage, uint32_t here, int j0) {
    constexpr bool masked = decltype(is_masked)::value;
    const uint32_t wp = stage + SP::KWORDS + 4 * tok, zp = stage + SP::VWORDS + 16 * t;
    // x: scores, after their scale relative to the running maximum
    float x[NT][2][4], sk[2][2], sv[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t kc[2][KW];
      float kz[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t kw, vw;
#pragma unroll
        for (int i = 0; i < SP::KLOADS; ++i)
          lds_words<KW / SP::KLOADS>(
              kc[k] + 4 * i, stage + (k ? SP::second_key(koff[i]) : koff[i]) + 16 * h * SP::TOK);
        lds_words<1>(&kw, wp + 64 * h + 8 * k);
        lds_words<1>(&vw, wp + 4 * STEP + 64 * h + 8 * k);
        sk[h][k] = word_scale(kw);
        kz[k] = word_zero(kw);
        sv[h][k] = word_scale(vw);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int c = 0; c < 2; ++c) x[nt][h][2 * k + c] = kz[k] * qsum[nt][c];
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          const uint32_t ua = kc[0][w], ub = kc[1][w];
          mma16816(x[nt][h], ua & 0x000f000fu, ub & 0x000f000fu, ua & 0x00f000f0u, ub & 0x00f000f0u,
                   qf[nt][w][0], qf[nt][w][1]);
          const uint32_t va = ua >> 8, vb = ub >> 8;
          mma16816(x[nt][h], va & 0x000f000fu, vb & 0x000f000fu, va & 0x00f000f0u, vb & 0x00f000f0u,
                   qf[nt][w][2], qf[nt][w][3]);
        }
      }
    }
    if constexpr (masked) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int j = j0 + tok + 16 * h + 2 * k;
          // what no row sees may be memory that was never written
          if (!((here >> h) & 1) || !(j < any_hi && (j >= any_lo || j < a.sinks))) sv[h][k] = 1.f;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const bool seen = ((here >> h) & 1) && j < chi[nt][c] && (j >= clo[nt][c] || j < a.sinks);
              float& y = x[nt][h][2 * k + c];
              y = seen ? y * (sk[h][k] * qmul[nt][c]) : -INFINITY;
            }
          sk[h][k] = 1.f;                // (applied)
        }
    }
    const float sv_big = fmaxf(fmaxf(sv[0][0], sv[0][1]), fmaxf(sv[1][0], sv[1][1]));
    float top = -INFINITY;
    float y[NT][2][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float f = masked ? 1.f : sk[h][k] * qmul[nt][c];
            y[nt][h][2 * k + c] = fmaf(x[nt][h][2 * k + c], f, -m[nt][c]);
            top = fmaxf(top, y[nt][h][2 * k + c]);
          }
    // (a bound of the lane's largest weight: its largest score with its largest scale)
    if (__any_sync(0xffffffffu, top + log2_approx(sv_big) > LAG + LIFT || top > LAG + LIFT + FAR)) {
      // new maxima (per column, over the lanes of equal t)
      float at[2][2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < 2; ++k) at[h][k] = fmaxf(log2_approx(sv[h][k]), -FAR) - (BASE + LIFT);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float al[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float nm = m[nt][c];
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float& v = y[nt][h][2 * k + c];
              v = x[nt][h][2 * k + c] * (masked ? 1.f : sk[h][k] * qmul[nt][c]);
              nm = fmaxf(nm, v + at[h][k]);
            }
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) nm = fmaxf(nm, __shfl_xor_sync(0xffffffffu, nm, d));
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int k = 0; k < 2; ++k) y[nt][h][2 * k + c] -= nm;
          al[c] = m[nt][c] == nm ? 1.f : exp2_approx(m[nt][c] - nm);
          m[nt][c] = nm;
          l[nt][c] *= al[c];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) z[nt][j] *= al[j & 1];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[nt][i][j] *= al[j & 1];
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t zw[4], pf[NT][2], pl[NT][2];
      lds_words<4>(zw, zp + 64 * h);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float svf = sv[h][k] * (1.f / (1 << (int)LIFT));
          const float p0 = exp2_approx(y[nt][h][2 * k]), p1 = exp2_approx(y[nt][h][2 * k + 1]);
          l[nt][0] += p0;
          l[nt][1] += p1;
          float w0 = p0 * svf, w1 = p1 * svf;
          if constexpr (masked) {        // (0 times a NaN scale)
            if (x[nt][h][2 * k] == -INFINITY) w0 = 0.f;
            if (x[nt][h][2 * k + 1] == -INFINITY) w1 = 0.f;
          }
          const uint32_t hi = pack_half2(w0, w1);
          if constexpr (TERMS != ONE) {
            const float2 up = __half22float2(*reinterpret_cast<const __half2*>(&hi));
            const uint32_t lo = pack_half2(w0 - up.x, w1 - up.y);
            pf[nt][k] = turn8x8(TERMS == TWO_COLUMNS && t >= 2 ? lo : hi);
            if constexpr (TERMS == TWO_PRODUCTS) pl[nt][k] = turn8x8(lo);
          } else {
            pf[nt][k] = turn8x8(hi);
          }
        }
      {
        const uint32_t z01 = __byte_perm(zw[0], zw[1], 0x5410) & 0x000f000fu;
        const uint32_t z23 = __byte_perm(zw[2], zw[3], 0x5410) & 0x000f000fu;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma16816(z[nt], z01, z01, z23, z23, pf[nt][0], pf[nt][1]);
          if constexpr (TERMS == TWO_PRODUCTS) mma16816(z[nt], z01, z01, z23, z23, pl[nt][0], pl[nt][1]);
        }
      }
#pragma unroll
      for (int c = 0; c < SP::VC; c += 2) {
        uint32_t v[4];
        ldmatrix_turned(v, ((stage + voff) ^ (16 * c)) + 16 * h * SP::TOK);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t b01 = __byte_perm(v[i], 0, 0x4140), b23 = __byte_perm(v[i], 0, 0x4342);
          const uint32_t c01 = b01 & 0x000f000fu, c23 = b23 & 0x000f000fu;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma16816(o[nt][2 * c + i], c01, b01, c23, b23, pf[nt][0], pf[nt][1]);
            if constexpr (TERMS == TWO_PRODUCTS)
              mma16816(o[nt][2 * c + i], c01, b01, c23, b23, pl[nt][0], pl[nt][1]);
          }
        }
      }
    }
  };
  int unflushed = 0;
  uint32_t now = ring, next = ring + (RING - 1) * SP::BYTES;
  const uint32_t ring_end = ring + RING * SP::BYTES;
  for (int st = 0; st < steps; ++st) {
    copy_wait<RING - 2>();
    __syncwarp();
    const uint32_t first = plan.first[st & 31], stage = now;
    fetch(st + RING - 1, next);          // into the stage that the last step has left
    now = now + SP::BYTES == ring_end ? ring : now + SP::BYTES;
    next = next + SP::BYTES == ring_end ? ring : next + SP::BYTES;
    if (!(first & 3u)) continue;
    if (first & 4u)
      multiply(std::true_type{}, stage, first & 3u, (int)(first & ~7u));
    else
      multiply(std::false_type{}, stage, 3u, (int)(first & ~7u));
    if (++unflushed == FLUSH) {
      unflushed = 0;
      flush();
    }
  }
  copy_wait<0>();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the merge kernel, which waits
  flush();
  __syncthreads();                       // the rings become the joining buffer

  // ---- join the warps
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], d);
      if (gr == 0) {
        merge_ml[warp][8 * nt + 2 * t + c][0] = m[nt][c];
        merge_ml[warp][8 * nt + 2 * t + c][1] = l[nt][c];
      }
    }
  __syncthreads();
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int r = 8 * nt + 2 * t + c;
      float mx = merge_ml[0][r][0];
#pragma unroll
      for (int w = 1; w < WARPS; ++w) mx = fmaxf(mx, merge_ml[w][r][0]);
      const float root = exp2_half(m[nt][c] - mx), f = root * root;
      const float fe = f * (0x1p24f * (1 << (int)LIFT)), fo = f * (0x1p20f * (1 << (int)LIFT));
      float* row = merge_o + (warp * ROWS + r) * D;
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int d = 16 * i + 2 * gr;
        *reinterpret_cast<float2*>(row + 4 * ((d >> 2) ^ join_swizzle(r)) + (d & 3)) =
            make_float2(o[nt][i][c] * fe, (o[nt][i][2 + c] - o[nt][i][c]) * fo);
      }
    }
  __syncthreads();
  const int64_t slot = ((int64_t)u.slot * a.cache.heads + head) * R;
  for (int e = threadIdx.x; e < R * (D / 4); e += THREADS) {
    const int r = e / (D / 4), d4 = e - r * (D / 4);
    if (r0 + r >= rows) break;
    float mx = merge_ml[0][r][0];
#pragma unroll
    for (int w = 1; w < WARPS; ++w) mx = fmaxf(mx, merge_ml[w][r][0]);
    float ls = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float mw = merge_ml[w][r][0], lw = merge_ml[w][r][1];
      const float root = exp2_half(mw - mx);
      ls += lw * root * root;
      const float4 v =
          *reinterpret_cast<const float4*>(merge_o + (w * ROWS + r) * D + 4 * (d4 ^ join_swizzle(r)));
      acc.x += v.x;
      acc.y += v.y;
      acc.z += v.z;
      acc.w += v.w;
      if (TERMS == TWO_COLUMNS) {        // the second terms
        const float4 x = *reinterpret_cast<const float4*>(merge_o + (w * ROWS + r + 4) * D +
                                                          4 * (d4 ^ join_swizzle(r + 4)));
        acc.x += x.x;
        acc.y += x.y;
        acc.z += x.z;
        acc.w += x.w;
      }
    }
    if (u.nsplit > 1) {
      *reinterpret_cast<float4*>(a.part_o + (slot + r) * D + 4 * d4) = acc;
      if (d4 == 0) a.part_ml[slot + r] = {mx, ls};
      continue;
    }
    const int q = (r0 + r) / a.g, hq = head * a.g + (r0 + r) - q * a.g;
    store_row(a, s.row0 + q, hq, 4 * d4, acc, mx, ls);
  }
}

// Joins the splits of the rows that have some: a block per token and `hpb` query heads.
// Few splits: a warp per row; many: one row at a time, warp w takes the splits w, w + 4, ..
template <int D>
__global__ void __launch_bounds__(THREADS) kv4_merge_kernel(const AttendArgs a, int R, int hpb) {
  constexpr int E = D / 32;
  __shared__ __align__(16) float sum_o[WARPS][D];
  __shared__ float sum_l[WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = blockIdx.x;
  int b = find_sequence(a.b.q_start, a.b.B, i);
  Seq s = seq_of(a, min(max(b, 0), a.b.B - 1), nullptr);
  // the attention kernel's results from here on (every thread waits: this kernel's
  // end stands for that one's too)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int good = a.meta[a.b.B].x;
  if (good < a.b.B) {                    // (starts that go back: the search is over those in front)
    b = good > 0 ? find_sequence(a.b.q_start, good, i) : -1;
    s = seq_of(a, min(max(b, 0), a.b.B - 1), nullptr);
  }
  if (b < 0 || b >= good) return;
  if (i < s.row0 || i >= s.row0 + s.n) return;
  const int2 mt = a.meta[b];
  const int ns = mt.y;
  if (ns <= 1) return;
  if (ns <= 8 && hpb > 1) {
    // lane: chunk of 4 dims (head_dim 256: and the one 32 on; 64: of every other split)
    constexpr int CPL = D == 256 ? 2 : 1, KP = D == 64 ? 2 : 1;
    const int c = lane % (D == 64 ? 16 : 32), k0 = KP == 2 ? lane >> 4 : 0;
    for (int h = warp; h < hpb; h += WARPS) {
      const int hq = blockIdx.y * hpb + h;
      if (hq >= a.Hq) return;
      const int head = hq / a.g, r = (i - s.row0) * a.g + hq - head * a.g;
      const int tile = r / R;
      const int64_t stride = (int64_t)a.cache.heads * R;
      const int64_t s0 = ((int64_t)(mt.x + tile * ns) * a.cache.heads + head) * R + (r - tile * R);
      const Part q = lane < ns ? a.part_ml[s0 + lane * stride] : Part{-INFINITY, 0.f};
      float4 v[8 / KP][CPL];
#pragma unroll
      for (int k = 0; k < 8; k += KP)
#pragma unroll
        for (int j = 0; j < CPL; ++j)
          v[k / KP][j] = k + k0 < ns ? *reinterpret_cast<const float4*>(a.part_o + (s0 + (k + k0) * stride) * D +
                                                                        4 * (c + 32 * j))
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
      float m = q.m;
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
      m = __shfl_sync(0xffffffffu, m, 0);              // (of the splits, lanes 0 .. 7)
      const float root = exp2_half(q.m - m), w = root * root;
      float l = q.l * root * root;
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
      l = __shfl_sync(0xffffffffu, l, 0);
      float4 o[CPL];
#pragma unroll
      for (int j = 0; j < CPL; ++j) o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < 8; k += KP) {
        const float wk = __shfl_sync(0xffffffffu, w, k + k0);
        if (k + k0 >= ns) continue;
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
          o[j].x = fmaf(wk, v[k / KP][j].x, o[j].x);
          o[j].y = fmaf(wk, v[k / KP][j].y, o[j].y);
          o[j].z = fmaf(wk, v[k / KP][j].z, o[j].z);
          o[j].w = fmaf(wk, v[k / KP][j].w, o[j].w);
        }
      }
      if constexpr (KP == 2) {
        o[0].x += __shfl_xor_sync(0xffffffffu, o[0].x, 16);
        o[0].y += __shfl_xor_sync(0xffffffffu, o[0].y, 16);
        o[0].z += __shfl_xor_sync(0xffffffffu, o[0].z, 16);
        o[0].w += __shfl_xor_sync(0xffffffffu, o[0].w, 16);
      }
      if (KP == 1 || lane < 16)
#pragma unroll
        for (int j = 0; j < CPL; ++j) store_row(a, i, hq, 4 * (c + 32 * j), o[j], m, l);
    }
    return;
  }
  for (int h = 0; h < hpb; ++h) {
    const int hq = blockIdx.y * hpb + h;
    if (hq >= a.Hq) return;
    const int head = hq / a.g, r = (i - s.row0) * a.g + hq - head * a.g;
    const int tile = r / R;
    const int64_t stride = (int64_t)a.cache.heads * R;
    const int64_t s0 = ((int64_t)(mt.x + tile * ns) * a.cache.heads + head) * R + (r - tile * R);
    float m = -INFINITY;
    for (int k = lane; k < ns; k += 32) m = fmaxf(m, a.part_ml[s0 + k * stride].m);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    float l = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll 4
    for (int k = warp; k < ns; k += WARPS) {
      const Part q = a.part_ml[s0 + k * stride];
      const float* p = a.part_o + (s0 + k * stride) * D + lane * E;
      float v[E];
      if constexpr (E == 2) {
        const float2 x = *reinterpret_cast<const float2*>(p);
        v[0] = x.x;
        v[1] = x.y;
      } else {
#pragma unroll
        for (int e = 0; e < E; e += 4) {
          const float4 x = *reinterpret_cast<const float4*>(p + e);
          v[e] = x.x;
          v[e + 1] = x.y;
          v[e + 2] = x.z;
          v[e + 3] = x.w;
        }
      }
      const float root = exp2_half(q.m - m), w = root * root;
      l += q.l * root * root;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(w, v[e], o[e]);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) sum_o[warp][lane * E + e] = o[e];
    if (lane == 0) sum_l[warp] = l;
    __syncthreads();
    if (threadIdx.x < D / 4) {
      float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
      float ls = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float4 x = *reinterpret_cast<const float4*>(&sum_o[w][4 * threadIdx.x]);
        t.x += x.x;
        t.y += x.y;
        t.z += x.z;
        t.w += x.w;
        ls += sum_l[w];
      }
      store_row(a, i, hq, 4 * threadIdx.x, t, m, ls);
    }
    __syncthreads();
  }
}

size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }

// (of the device this is written for, not asked for: a workspace's size is the same everywhere)
constexpr int SMS = 148;
// The shortest chunks of keys: one new token over 8k takes 13.4 us with 256 keys, 14.4 with
// 512 (before the join was cheap); 16 and 64 new tokens over 8k with the other kernel 25 and
// 33 us with 256, 23 and 31 with 512, 31 and 41 with 1024.
constexpr int MIN_CHUNK = 2;                         // key blocks
constexpr int PROMPT_MIN_KEYS = 512;
// What a unit costs beside its blocks.  It matters little: with 0 for both, 1 x 8k 13.5 us and
// 12 x 3k 20.6 as with these, 4 x 128k 110 (108); with 5 and 15 they take 14.1, 22.0 and 108.
constexpr float UNIT_COST = 1.5f, PROMPT_UNIT_COST = 5.f;

// How a call is run.  Rows per sequence and key/value head decide (on average: lengths
// are on the device).  The tensor-memory kernel's time is that of 128 rows (256: the
// second tile rides along) whatever there are; the other's grows with every 16 (head_dim
// 256: 8), and per row it is the slower one:
//   rows                 16    24    32    40    48    64    80    96
//   head_dim 128 bf16    43    61    62    75    76   100   133   147     8 sequences of 8k, 8 heads
//                        99   100   100   100   100   101   104   104     (us; this kernel, kv4_prompt.cu)
//                fp16    48    71    72    90    91   122   170   180
//                        97    97    97    98    97    98   100   101
//   head_dim 256 bf16    68    84   110   138   160   197   249   289
//                       210   210   212   212   214   211   214   216
//                fp16    76    95   126   157   183   229   289   336
//                       123   123   123   124   126   127   128   129
//   head_dim 64  bf16    31    45    46    56    57    74   106   108
//                        76    76    76    77    78    78    79    80
//                fp16    34    52    52    64    65    86   123   125
//                        84    84    84    85    85    86    86    87
// fp16 queries stay with this kernel some rows longer than it is the faster one, for its second
// terms (see Terms; the other kernel's error against 64 bits is 1.4 times that of the output's
// rounding).
// Tiles of 8 rows (twice the blocks per SM) where 8 are enough: 16 rows take 42 us with
// them, 39 with tiles of 16.
struct Way {
  bool prompt;
  int R, BLK, min_chunk, resident;
  float unit_cost;
};

Way way_of(int64_t T, int g, int D, int64_t B, int dt) {
  if (T * g > (D == 256 && dt == FP16 ? 40 : 64) * B)
    return {true, prompt_rows(D), prompt_block(D), PROMPT_MIN_KEYS / prompt_block(D), SMS, PROMPT_UNIT_COST};
  const int R = dt == FP16 && T * g <= 4 * B ? 4 : D == 256 || T * g <= 8 * B ? 8 : 16;
  return {false, R, BLK, MIN_CHUNK, SMS * (D == 256 || R == 16 ? 2 : 4), UNIT_COST};
}

struct Layout {
  size_t meta, ml, o, total;
};

Layout layout_of(const Way& w, int D, int heads, int64_t B) {
  const size_t rows = (size_t)max_slots(heads, w.resident) * heads * w.R;
  Layout l;
  l.meta = 0;
  l.ml = up256((size_t)(B + 1) * sizeof(int2));
  l.o = l.ml + up256(rows * sizeof(Part));
  l.total = l.o + up256(rows * D * sizeof(float));
  return l;
}

template <int D, int NT, int TERMS>
int launch(AttendArgs& a, cudaStream_t st) {
  constexpr int ROWS = 8 * NT, R = TERMS == TWO_COLUMNS ? 4 : ROWS;
  const long long grid = max_units(a, R, BLK);
  if (grid > INT32_MAX) return KRONQ_ERR_UNSUPPORTED;
  constexpr int rings = WARPS * RING * Step<D>::BYTES, join = WARPS * ROWS * D * (int)sizeof(float);
  constexpr int smem = rings > join ? rings : join;
  static kqh::PerDevice attr;
  if (kqh::smem_attr_once(attr, kv4_attend_kernel<D, NT, TERMS>, smem) <= 0) return KRONQ_ERR_CUDA;
  kv4_attend_kernel<D, NT, TERMS><<<(unsigned)grid, THREADS, smem, st>>>(a);
  KQ_CHECK_LAUNCH();
  return KRONQ_OK;
}

template <int D>
int launch_merge(const AttendArgs& a, int R, cudaStream_t st) {
  // Query heads of a token to a block: one where the device holds a block for each row or a
  // sequence may have many splits (their number is resident / (heads B) on average, and a warp
  // takes 8), else four; a token's all where there are so many rows that blocks which find
  // nothing to do are the cost.  The whole call in us, heads of 128, bf16:
  //   rows, resident / (heads B)     1      4    all
  //      512    4.6                44.2   49.5   94.7
  //     1024    2.3                63.5   62.3   69.7
  //     4096    1.2                 115    108    123
  //     4096    4.6                90.5   85.0   96.4
  //     2048    9.2                 163    167    267
  //     2048   18.5                61.3   62.8    109
  //    16384    9.2                 206    180    183
  //    65536    4.6                 440    362    360
  //   131072    9.2                1241   1190   1175
  //   262144   18.5                 883    776    747
  const long long rows = (long long)a.T * a.Hq;
  const bool few = a.resident <= 6ll * a.cache.heads * a.b.B;
  const int hpb = rows <= 4 * SMS || (!few && rows <= 8192) ? 1 : rows <= 65536 ? 4 : a.Hq;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.T, (unsigned)((a.Hq + hpb - 1) / hpb));
  cfg.blockDim = dim3(THREADS);
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kv4_merge_kernel<D>, a, R, hpb) != cudaSuccess) return KRONQ_ERR_CUDA;
  KQ_CHECK_LAUNCH();
  return KRONQ_OK;
}

template <int D>
int run(AttendArgs& a, const Way& w, cudaStream_t st) {
  int s;
  if (w.prompt)
    s = launch_prompt(a, D, st);
  else if (w.R == 4)
    s = launch<D, 1, TWO_COLUMNS>(a, st);
  else if (D == 256 || w.R == 8)
    s = a.dt == FP16 ? launch<D, 1, TWO_PRODUCTS>(a, st) : launch<D, 1, ONE>(a, st);
  else
    s = a.dt == FP16 ? launch<D, D == 256 ? 1 : 2, TWO_PRODUCTS>(a, st) : launch<D, D == 256 ? 1 : 2, ONE>(a, st);
  if (s != KRONQ_OK) return s;
  // no sequence can be split when the longest one the table holds is one chunk
  const long long most = (((long long)a.b.max_pages << a.cache.lgP) + w.BLK - 1) / w.BLK;
  return most <= a.min_chunk ? KRONQ_OK : launch_merge<D>(a, w.R, st);
}

}  // namespace
}  // namespace kv4

size_t kq_kv4_attention_ws(int64_t T, int Hq, int heads, int D, int64_t B) {
  if (T < 0 || Hq <= 0 || heads <= 0 || Hq % heads || B <= 0 || (D != 64 && D != 128 && D != 256)) return 0;
  // (for either type)
  const auto need = [&](int dt) { return kv4::layout_of(kv4::way_of(T, Hq / heads, D, B, dt), D, heads, B).total; };
  return std::max(need(kv4::BF16), need(kv4::FP16));
}

int kq_kv4_attention(const void* q, int64_t q_st, int64_t q_sh, int dtype, int64_t T, int Hq, int D,
                     const kv4::Cache& c, const kv4::Batch& b, float scale, int causal, int window,
                     int sinks, void* out, int64_t o_st, int64_t o_sh, float* lse, int32_t* info,
                     void* ws, size_t ws_bytes, cudaStream_t st) {
  using namespace kv4;
  if (dtype != BF16 && dtype != FP16) return KRONQ_ERR_UNSUPPORTED;
  if (T < 0 || T > INT32_MAX || Hq <= 0 || Hq % c.heads || window < 0 || sinks < 0 ||
      (window && !causal) || !(scale == scale))
    return KRONQ_ERR_INVALID_ARG;
  if (T == 0) return KRONQ_OK;
  if (!b.B || !q || !out || !kqh::aligned(q, 2) || !kqh::aligned(out, 8) || q_st < 0 || q_sh < 0 || o_st < 0 ||
      o_sh < 0 || o_st % 4 || o_sh % 4 || !kqh::aligned(lse, 4))
    return KRONQ_ERR_INVALID_ARG;
  // The output may lie over the queries (a block reads its rows before it writes them); any other
  // overlap would be a race.  With equal strides, rows that interleave are told from those that
  // overlap by where they lie within a token.
  const KqRows from = {q, q_st, q_sh, T, Hq, D}, to = {out, o_st, o_sh, T, Hq, D};
  if (!to.apart()) return KRONQ_ERR_INVALID_ARG;
  if (from.meets(to) && !(q == out && (T == 1 || q_st == o_st) && (Hq == 1 || q_sh == o_sh))) {
    const int64_t span = (Hq - 1) * o_sh + D;
    if (T == 1 || q_st != o_st || q_sh != o_sh || o_st < span) return KRONQ_ERR_INVALID_ARG;
    const int64_t at = ((static_cast<const uint16_t*>(out) - static_cast<const uint16_t*>(q)) % o_st + o_st) % o_st;
    if (at < span || at + span > o_st) return KRONQ_ERR_INVALID_ARG;
  }
  if (!ws || !kqh::aligned(ws, 256) || ws_bytes < kq_kv4_attention_ws(T, Hq, c.heads, D, b.B))
    return KRONQ_ERR_WORKSPACE;
  const int g = Hq / c.heads;
  if (T * g > INT32_MAX / 2) return KRONQ_ERR_UNSUPPORTED;
  AttendArgs a = {};
  a.q = static_cast<const uint16_t*>(q);
  a.q_st = q_st;
  a.q_sh = q_sh;
  a.q_vec = kqh::aligned(q, 16) && q_st % 8 == 0 && q_sh % 8 == 0;
  a.out = out;
  a.o_st = o_st;
  a.o_sh = o_sh;
  a.lse = lse;
  a.cache = c;
  a.b = b;
  a.T = (int)T;
  a.Hq = Hq;
  a.g = g;
  a.dt = dtype;
  a.causal = causal;
  a.window = window > (1 << 30) ? 0 : window;    // wider than any sequence
  a.sinks = !a.window ? 0 : sinks > (1 << 30) ? 1 << 30 : sinks;
  a.scale_log2 = scale * 1.4426950408889634f;
  const Way way = way_of(T, g, D, b.B, dtype);
  a.min_chunk = way.min_chunk;
  a.resident = way.resident;
  a.unit_cost = way.unit_cost;
  a.info = info;
  const Layout w = layout_of(way, D, c.heads, b.B);
  uint8_t* base = static_cast<uint8_t*>(ws);
  a.meta = reinterpret_cast<int2*>(base + w.meta);
  a.part_ml = reinterpret_cast<Part*>(base + w.ml);
  a.part_o = reinterpret_cast<float*>(base + w.o);
  return D == 64 ? run<64>(a, way, st) : D == 128 ? run<128>(a, way, st) : run<256>(a, way, st);
}
