// Attention of new queries over the paged 4-bit cache, many query rows per key
// (prompts, chunks of prompts, long drafts): tcgen05 with the same arithmetic as
// kv4_attend.cu.  Codes are unpacked once per block and tile of keys into shared
// memory as the whole numbers c - z (exact in fp16 and bf16), so
//   S = Q K^T      in the queries' type, fp32 accumulators in tensor memory
//   x = S s_j scale log2(e),  p = 2^(x - m),  P = p s'_j (fp16)
//   O += P V       with P as the tensor-memory operand, over S
// and the only rounding besides fp32's is P's.  The running maximum m is a whole
// number and moves only when a score passes it by 8; what was summed before is
// then scaled by a power of two.
//
// One block = up to 256 rows (two tiles of 128; one at head_dim 256) of one
// sequence and key/value head, over its keys in steps of BN (128; 64 at head_dim
// 256).  Warps:
//   0-3, 4-7  softmax of tile 0, of tile 1: a thread owns a row, reads S 32 columns
//             at a time and writes P over it, so no reduction crosses lanes
//   8-11      unpacking: codes of the next step are in registers while this one waits
//             for its stage; rows of 128 bytes, 128-byte swizzled, for both operands
//             (keys K-major, values MN-major)
//   12        issues the MMAs: S of one tile runs beside the softmax of the other
// Dims stay in the order unpacking yields within each 8 (0 4 1 5 2 6 3 7): queries
// are stored that way and the output is put right when it leaves.
//
// All waits are bounded; one that gives up records KRONQ_ERR_TIMEOUT in `info`.
#include <type_traits>

#include "kv4_attend.cuh"

namespace kv4 {
namespace {

constexpr int UNPACK_WARP0 = 8, MMA_WARP = 12, THREADS = 416;
constexpr float NO_MAX = -0x1p100f;     // a whole number; see kv4_attend.cu
constexpr float LAG = 8.f;

template <int D>
struct Shape {
  static constexpr int NT = D == 256 ? 1 : 2;        // tiles of 128 rows
  static constexpr int BN = D == 256 ? 64 : 128;     // keys per step
  static constexpr int R = 128 * NT;
  static constexpr int ATOMS = D / 64;               // 128-byte columns of an operand row
  static constexpr int Q_BYTES = R * D * 2;
  static constexpr int KV_BYTES = BN * D * 2;        // keys or values of a stage
  static constexpr int STAGE = 2 * KV_BYTES;
  static constexpr int TPW = BN / 4;                 // tokens per unpacking warp
  static constexpr int CH = D / 32;                  // 16-byte chunks of a token's codes
  static constexpr int LOADS = TPW * CH / 32;        // chunks per lane (keys; values)
  static constexpr int S_COLS = D == 256 ? 64 : 128;
  static constexpr int O_COL = 256;
  static constexpr int SMEM = Q_BYTES + 2 * STAGE + 1024;
};

struct Ctl {
  uint64_t kv_full[2], kv_empty[2], s_full[2], p_ready[2], scales, pv_done, o_full;
  float fk[2][128], sv[2][128];          // per key: score factor; value scale x fv
  uint32_t absent[2][4];                 // bit per key: no page
  float turn[2], fv[2];                  // fv of the stage over fv of the step before; fv
  float sv_warp[2][4];                   // per step's parity and warp: its largest value scale
  uint32_t tmem;
  int abort;
};

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
// The same in bf16; z1: 128 + z in both halves.
KQ_DEV uint4 codes_bf16(uint32_t w, uint32_t z1) {
  const __nv_bfloat162 a = *reinterpret_cast<const __nv_bfloat162*>(&z1);
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t v = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
    const __nv_bfloat162 x = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), a);
    r[i] = *reinterpret_cast<const uint32_t*>(&x);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

template <int D, bool BF>
__global__ void __launch_bounds__(THREADS, 1) kv4_prompt_kernel(const AttendArgs a) {
  using SH = Shape<D>;
  constexpr int NT = SH::NT, BN = SH::BN, R = SH::R, ATOMS = SH::ATOMS;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Ctl ctl;
  uint8_t* q_smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
  uint8_t* kv_smem = q_smem + SH::Q_BYTES;

  Unit u;
  if (!find_unit<R, BN, THREADS>(a, blockIdx.x, &u)) return;
  const int head = blockIdx.y;
  // (only a batch whose rows overlap can ask for more slots than there are)
  if (u.nsplit > 1 && (u.slot0 < 0 || u.slot0 + (int)blockIdx.x - u.base >= a.slots)) {
    kq::record_error(a.info, KRONQ_ERR_INVALID_ARG);
    return;
  }
  const Seq s = seq_of(a, u.b, nullptr);
  if (threadIdx.x == 0 && head == 0 && u.tile == 0 && u.split == 0)
    a.meta[u.b] = make_int2(u.slot0, u.nsplit);
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
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      kq::mbar_init(&ctl.kv_full[i], 4);
      kq::mbar_init(&ctl.kv_empty[i], 1);
      kq::mbar_init(&ctl.s_full[i], 1);
      kq::mbar_init(&ctl.p_ready[i], 4);
    }
    kq::mbar_init(&ctl.scales, 4);
    kq::mbar_init(&ctl.pv_done, 1);
    kq::mbar_init(&ctl.o_full, 1);
    ctl.abort = 0;
    kq::fence_barrier_init();
  }
  if (warp == MMA_WARP) kq::tmem_alloc(&ctl.tmem, 512);
  // queries: rows of 128-byte lines, dims of each 8 in the codes' order
  for (int e = threadIdx.x; e < R * (D / 8); e += THREADS) {
    const int r = e / (D / 8), c = e - r * (D / 8);
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (r0 + r < rows) {
      const int qi = (r0 + r) / a.g;
      const uint16_t* p = a.q + (int64_t)(s.row0 + qi) * a.q_st +
                          (int64_t)(head * a.g + r0 + r - qi * a.g) * a.q_sh + 8 * c;
      if (a.q_vec) {
        v = __ldg(reinterpret_cast<const uint4*>(p));
      } else {
        uint32_t h[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = __ldg(p + j);
        v = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
      }
      v = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                     __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
    }
    uint8_t* dst = q_smem + ((r >> 7) * ATOMS + (c >> 3)) * 16384 + (r & 127) * 128 +
                   (((c & 7) ^ (r & 7)) << 4);
    *reinterpret_cast<uint4*>(dst) = v;
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  kq::tc_fence_before();
  __syncthreads();
  kq::tc_fence_after();
  const uint32_t tmem = ctl.tmem;

  if (warp == MMA_WARP) {
    // ------------------------------------------------------------- MMAs
    if (lane == 0 && steps > 0) {
      constexpr uint32_t idesc_qk = kq::idesc_f16(128, BN, BF ? 1 : 0, 0, 0);
      constexpr uint32_t idesc_pv = kq::idesc_f16(128, D, 0, 0, 1);
      const uint32_t qa = kq::smem_u32(q_smem), kv = kq::smem_u32(kv_smem);
      auto issue_s = [&](int tile, int buf, int j) {
        const uint32_t ka = kv + (j & 1) * SH::STAGE;
#pragma unroll
        for (int at = 0; at < ATOMS; ++at)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            kq::mma_f16(tmem + buf * SH::S_COLS,
                        kq::smem_desc(qa + (tile * ATOMS + at) * 16384 + kk * 32, 16, 1024, kq::kLayoutSwizzle128B),
                        kq::smem_desc(ka + at * (BN * 128) + kk * 32, 16, 1024, kq::kLayoutSwizzle128B), idesc_qk,
                        at || kk);
        kq::mma_commit(&ctl.s_full[buf]);
      };
      auto issue_pv = [&](int tile, int buf, int j) {
        const uint32_t va = kv + (j & 1) * SH::STAGE + SH::KV_BYTES;
#pragma unroll
        for (int kk = 0; kk < BN / 16; ++kk)
          mma_f16_ts(tmem + SH::O_COL + tile * D, tmem + buf * SH::S_COLS + kk * 8,
                     kq::smem_desc(va + kk * 2048, BN * 128, 1024, kq::kLayoutSwizzle128B), idesc_pv,
                     j > 0 || kk > 0);
      };
      bool ok = kq::mbar_wait(&ctl.kv_full[0], 0, abort, a.info);
      if (ok) {
        kq::tc_fence_after();
        for (int i = 0; i < (NT == 2 ? tiles : 1); ++i) issue_s(i, i, 0);
      }
      for (int j = 0; j < steps && ok; ++j) {
        const bool more = j + 1 < steps;
        if (more) {
          ok = kq::mbar_wait(&ctl.kv_full[(j + 1) & 1], ((j + 1) >> 1) & 1, abort, a.info);
          if (!ok) break;
          kq::tc_fence_after();
        }
        if (NT == 2) {
          for (int i = 0; i < tiles && ok; ++i) {
            ok = kq::mbar_wait(&ctl.p_ready[i], j & 1, abort, a.info);
            if (!ok) break;
            kq::tc_fence_after();
            issue_pv(i, i, j);
            if (i == tiles - 1) kq::mma_commit(&ctl.kv_empty[j & 1]);
            // (over P, in issue order behind the MMAs that read it)
            if (more) issue_s(i, i, j + 1);
          }
        } else {
          if (more) issue_s(0, (j + 1) & 1, j + 1);
          ok = kq::mbar_wait(&ctl.p_ready[j & 1], (j >> 1) & 1, abort, a.info);
          if (!ok) break;
          kq::tc_fence_after();
          issue_pv(0, j & 1, j);
          kq::mma_commit(&ctl.kv_empty[j & 1]);
          kq::mma_commit(&ctl.pv_done);
        }
      }
      // (also after a wait that gave up: nothing is in flight when the block ends)
      kq::mma_commit(&ctl.o_full);
      volatile int none = 0;
      kq::mbar_wait(&ctl.o_full, 0, &none, a.info);
    }
    __syncwarp();
  } else if (warp >= UNPACK_WARP0) {
    // -------------------------------------------------------- unpacking
    const int w = warp - UNPACK_WARP0;
    const int any_lo = lo_of(q_first), any_hi = hi_of(q_last);
    const int c = lane % SH::CH, ct = lane / SH::CH;        // chunk, token within a load
    constexpr int TPL = 32 / SH::CH;                        // tokens per load
    const int at = c >> 1;
    const int x = D == 256 ? at : D == 128 ? 2 * at : 0;    // order in which words are stored
    uint4 kreg[SH::LOADS], vreg[SH::LOADS];
    uint32_t kword = 0, vword = 0;                          // of token TPW w + lane
    bool here = false;
    auto load = [&](int j) {
      const int tok0 = key_of(i0 + j) + SH::TPW * w;
      const int tl = tok0 + (lane & (SH::TPW - 1));
      int64_t page = -1;
      if (tl < any_hi && (tl >= any_lo || tl < a.sinks)) {
        page = a.b.table[u.b * a.b.table_ld + (tl >> a.cache.lgP)];
        if (page < 0 || page >= a.cache.pages) {
          kq::record_error(a.info, KRONQ_ERR_INVALID_ARG);
          page = -1;
        }
      }
      const int P = a.cache.P;
      const uint8_t* blk = a.cache.base + (page * a.cache.heads + head) * (int64_t)a.cache.block_bytes;
      here = page >= 0;
      kword = vword = 0;
      if (here) {
        const uint32_t* wp = reinterpret_cast<const uint32_t*>(blk + P * D) + (tl & (P - 1));
        kword = __ldg(wp);
        vword = __ldg(wp + P);
      }
      const uint32_t seen = __ballot_sync(0xffffffffu, here);
      // the base address of this token's codes
      const uint64_t codes = here ? (uint64_t)(blk + (tl & (P - 1)) * (D / 2)) : 0;
#pragma unroll
      for (int i = 0; i < SH::LOADS; ++i) {
        const int tk = i * TPL + ct;
        const uint64_t p = __shfl_sync(0xffffffffu, codes, tk);
        kreg[i] = vreg[i] = make_uint4(0u, 0u, 0u, 0u);
        if (p) {
          const uint8_t* kp = reinterpret_cast<const uint8_t*>(p) + 16 * c;
          asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(kreg[i].x), "=r"(kreg[i].y), "=r"(kreg[i].z), "=r"(kreg[i].w)
                       : "l"(kp));
          asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(vreg[i].x), "=r"(vreg[i].y), "=r"(vreg[i].z), "=r"(vreg[i].w)
                       : "l"(kp + (int64_t)P * (D / 2)));
        }
      }
      return seen;
    };
    uint32_t seen = 0;
    if (steps > 0) seen = load(0);
    float fv = 0.f;
    bool ok = true;
    for (int j = 0; j < steps; ++j) {
      const int st = j & 1;
      if (j >= 2) {
        ok = kq::mbar_wait(&ctl.kv_empty[st], ((j >> 1) + 1) & 1, abort, a.info);
        if (!__all_sync(0xffffffffu, ok)) break;
      }
      // fv: a power of two that keeps value scales below 2^6 (see kv4_attend.cu)
      float sv = word_scale(vword), big = sv;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
      if (lane == 0) {
        ctl.sv_warp[st][w] = big;
        kq::mbar_arrive(&ctl.scales);
      }
      ok = kq::mbar_wait(&ctl.scales, j & 1, abort, a.info);
      if (!__all_sync(0xffffffffu, ok)) break;
      big = fmaxf(fmaxf(ctl.sv_warp[st][0], ctl.sv_warp[st][1]), fmaxf(ctl.sv_warp[st][2], ctl.sv_warp[st][3]));
      float turn = 1.f;
      if (big > 0.f && (fv == 0.f || big * fv > 64.f)) {
        const int e = min(max(127 - (int)(__float_as_uint(big) >> 23), -100), 100);
        const float nf = __uint_as_float((uint32_t)(127 + e) << 23);
        if (fv != 0.f) turn = nf / fv;
        fv = nf;
      }
      if (lane < SH::TPW) {
        ctl.fk[st][SH::TPW * w + lane] = word_scale(kword) * a.scale_log2;
        ctl.sv[st][SH::TPW * w + lane] = sv * fv;
      }
      if (lane == 0) {
        if (SH::TPW == 32)
          ctl.absent[st][w] = ~seen;
        else
          reinterpret_cast<uint16_t*>(ctl.absent[st])[w] = (uint16_t)~seen;
      }
      if (w == 0 && lane == 0) {
        ctl.turn[st] = turn;
        ctl.fv[st] = fv;
      }
      const uint32_t kz = kword & 15u, vz = vword & 15u;
      uint8_t* kd = kv_smem + st * SH::STAGE + at * (BN * 128);
#pragma unroll
      for (int i = 0; i < SH::LOADS; ++i) {
        const int tk = i * TPL + ct, row = SH::TPW * w + tk;
        const uint32_t z = __shfl_sync(0xffffffffu, kz, tk), zv = __shfl_sync(0xffffffffu, vz, tk);
        const uint32_t z1 = (BF ? 0x43004300u : 0x64006400u) + z * 0x00010001u;
        const uint32_t z2 = 0xd400d400u + z * 0x00100010u;
        const uint32_t y1 = 0x64006400u + zv * 0x00010001u, y2 = 0xd400d400u + zv * 0x00100010u;
        uint32_t kw[4] = {kreg[i].x, kreg[i].y, kreg[i].z, kreg[i].w};
        uint32_t vw[4] = {vreg[i].x, vreg[i].y, vreg[i].z, vreg[i].w};
        auto swap = [](uint32_t& p, uint32_t& q, bool yes) {
          const uint32_t t = p;
          p = yes ? q : p;
          q = yes ? t : q;
        };
        if (D >= 128) {
          // lanes of a phase that write the same lines start with other words
          swap(kw[0], kw[2], x & 2);
          swap(kw[1], kw[3], x & 2);
          swap(vw[0], vw[2], x & 2);
          swap(vw[1], vw[3], x & 2);
        }
        if (D == 256) {
          swap(kw[0], kw[1], x & 1);
          swap(kw[2], kw[3], x & 1);
          swap(vw[0], vw[1], x & 1);
          swap(vw[2], vw[3], x & 1);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint8_t* d = kd + row * 128 + (((4 * (c & 1) + (k ^ x)) ^ (row & 7)) << 4);
          *reinterpret_cast<uint4*>(d) = BF ? codes_bf16(kw[k], z1) : codes_f16(kw[k], z1, z2);
          *reinterpret_cast<uint4*>(d + SH::KV_BYTES) = codes_f16(vw[k], y1, y2);
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) kq::mbar_arrive(&ctl.kv_full[st]);
      if (j + 1 < steps) seen = load(j + 1);
    }
  } else if (warp < 4 * tiles || (NT == 1 && warp < 4)) {
    // ---------------------------------------------------------- softmax
    const int tile = NT == 2 ? warp >> 2 : 0;
    const int tr = (warp & 3) * 32 + lane;              // row within the tile
    const uint32_t tbase = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t o_at = tbase + SH::O_COL + tile * D;
    const int r = min(last, r0 + 128 * tile + tr);
    const int qi = r / a.g;
    const int lo = lo_of(qi), hi = hi_of(qi);
    // what all rows of the warp see (rows are in order)
    const int all_lo = lo_of(__shfl_sync(0xffffffffu, qi, 31)), all_hi = hi_of(__shfl_sync(0xffffffffu, qi, 0));
    float m = NO_MAX, l = 0.f;
    bool ok = true;
    auto step = [&](auto is_masked, int j, int key0) {
      constexpr bool masked = decltype(is_masked)::value;
      const int st = j & 1, buf = NT == 2 ? tile : j & 1;
      const uint32_t s_at = tbase + buf * SH::S_COLS;
      float turn = ctl.turn[st];
#pragma unroll 1
      for (int ch = 0; ch < BN / 32; ++ch) {
        float x[32];
        kq::tmem_ld32(s_at + 32 * ch, x);
        const float4* fk4 = reinterpret_cast<const float4*>(&ctl.fk[st][32 * ch]);
        const float4* sv4 = reinterpret_cast<const float4*>(&ctl.sv[st][32 * ch]);
        const uint32_t gone = masked ? ctl.absent[st][ch] : 0u;
        kq::tmem_wait_ld();
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 f = fk4[i];
          x[4 * i] *= f.x;
          x[4 * i + 1] *= f.y;
          x[4 * i + 2] *= f.z;
          x[4 * i + 3] *= f.w;
          if constexpr (masked) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int key = key0 + 32 * ch + 4 * i + k;
              const bool seen = !((gone >> (4 * i + k)) & 1u) && key < hi && (key >= lo || key < a.sinks);
              if (!seen) x[4 * i + k] = -INFINITY;
            }
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) top = fmaxf(top, x[4 * i + k]);
        }
        const bool up = top > m + LAG;
        if (__any_sync(0xffffffffu, up || turn != 1.f)) {
          // the maximum moves to the next whole number: sums and the probabilities of
          // this step's earlier columns turn by a power of two
          const float nm = up ? (top < INFINITY ? ceilf(top) : top) : m;
          const float al = nm == m ? 1.f : exp2_approx(m - nm);
          m = nm;
          l *= al;
          if (j > 0) {
            if (NT == 1) ok = kq::mbar_wait(&ctl.pv_done, (j - 1) & 1, abort, a.info) && ok;
            __syncwarp();
            kq::tc_fence_after();
            const float f = al * turn;
#pragma unroll 1
            for (int d = 0; d < D; d += 16) {
              uint32_t o[16];
              tmem_ld16(o_at + d, o);
              kq::tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tmem_st16(o_at + d, o);
            }
          }
          turn = 1.f;
          kq::tmem_wait_st();
          const __half2 ah = __float2half2_rn(al);
#pragma unroll 1
          for (int d = 0; d < 16 * ch; d += 16) {
            uint32_t p[16];
            tmem_ld16(s_at + d, p);
            kq::tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&p[k]), ah);
              p[k] = *reinterpret_cast<const uint32_t*>(&v);
            }
            tmem_st16(s_at + d, p);
          }
        }
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 sv = sv4[i];
          const float p0 = exp2_approx(x[4 * i] - m), p1 = exp2_approx(x[4 * i + 1] - m);
          const float p2 = exp2_approx(x[4 * i + 2] - m), p3 = exp2_approx(x[4 * i + 3] - m);
          l += (p0 + p1) + (p2 + p3);
          float v0 = p0 * sv.x, v1 = p1 * sv.y, v2 = p2 * sv.z, v3 = p3 * sv.w;
          if constexpr (masked) {                       // (0 times a NaN scale)
            if (x[4 * i] == -INFINITY) v0 = 0.f;
            if (x[4 * i + 1] == -INFINITY) v1 = 0.f;
            if (x[4 * i + 2] == -INFINITY) v2 = 0.f;
            if (x[4 * i + 3] == -INFINITY) v3 = 0.f;
          }
          pk[2 * i] = pack_half2(v0, v1);
          pk[2 * i + 1] = pack_half2(v2, v3);
        }
        tmem_st16(s_at + 16 * ch, pk);
      }
    };
    for (int j = 0; j < steps; ++j) {
      const int st = j & 1, buf = NT == 2 ? tile : j & 1;
      ok = kq::mbar_wait(&ctl.kv_full[st], (j >> 1) & 1, abort, a.info) && ok;
      ok = ok && kq::mbar_wait(&ctl.s_full[buf], NT == 2 ? j & 1 : (j >> 1) & 1, abort, a.info);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      kq::tc_fence_after();
      const int key0 = key_of(i0 + j);
      uint32_t gone = 0;
#pragma unroll
      for (int i = 0; i < BN / 32; ++i) gone |= ctl.absent[st][i];
      if (gone || !(key0 + BN <= all_hi && (key0 >= all_lo || key0 + BN <= a.sinks)))
        step(std::true_type{}, j, key0);
      else
        step(std::false_type{}, j, key0);
      kq::tmem_wait_st();
      kq::tc_fence_before();
      __syncwarp();
      if (lane == 0) kq::mbar_arrive(&ctl.p_ready[buf]);
    }
    // ---- output
    if (steps > 0) ok = ok && kq::mbar_wait(&ctl.o_full, 0, abort, a.info);
    ok = __all_sync(0xffffffffu, ok);
    kq::tc_fence_after();
    const float rfv = steps > 0 && ctl.fv[(steps - 1) & 1] != 0.f ? 1.f / ctl.fv[(steps - 1) & 1] : 0.f;
    const int rr = 128 * tile + tr;
    const bool mine = r0 + rr < rows;
    const int64_t slot = ((int64_t)(u.slot0 + (int)blockIdx.x - u.base) * a.cache.heads + head) * R + rr;
    const int hq = head * a.g + r - qi * a.g;
    if (ok) {
#pragma unroll 1
      for (int d = 0; d < D; d += 16) {
        uint32_t o[16];
        if (steps > 0) {
          tmem_ld16(o_at + d, o);
          kq::tmem_wait_ld();
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] = 0u;
        }
#pragma unroll
        for (int k = 0; k < 16; k += 4) {
          if (!mine) break;
          // dims 8 (k / 8) + 0..3 are columns 0 2 4 6 of the 8, dims 4..7 columns 1 3 5 7
          const int b = (k & 8) + ((k >> 2) & 1);
          const float4 v = make_float4(__uint_as_float(o[b]) * rfv, __uint_as_float(o[b + 2]) * rfv,
                                       __uint_as_float(o[b + 4]) * rfv, __uint_as_float(o[b + 6]) * rfv);
          if (u.nsplit > 1) {
            *reinterpret_cast<float4*>(a.part_o + slot * D + d + k) = v;
            if (d + k == 0) a.part_ml[slot] = {m, l};
          } else {
            store_row(a, s.row0 + qi, hq, d + k, v, m, l);
          }
        }
        __syncwarp();
      }
    }
  }
  kq::tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    kq::tc_fence_after();
    kq::tmem_dealloc(tmem, 512);
  }
}

template <int D, bool BF>
int launch(const AttendArgs& a, cudaStream_t st) {
  using SH = Shape<D>;
  const long long ux = max_units(a.T, a.g, a.b.B, SH::R, a.cache.heads, a.target);
  if (ux > INT32_MAX) return KRONQ_ERR_UNSUPPORTED;
  static kqh::PerDevice attr;
  if (kqh::smem_attr_once(attr, kv4_prompt_kernel<D, BF>, SH::SMEM) <= 0) return KRONQ_ERR_CUDA;
  const dim3 grid((unsigned)ux, (unsigned)a.cache.heads);
  kv4_prompt_kernel<D, BF><<<grid, THREADS, SH::SMEM, st>>>(a);
  KQ_CHECK_LAUNCH();
  return KRONQ_OK;
}

}  // namespace

int prompt_rows(int D) { return D == 256 ? Shape<256>::R : Shape<128>::R; }
int prompt_block(int D) { return D == 256 ? Shape<256>::BN : Shape<128>::BN; }

int launch_prompt(const AttendArgs& a, int D, cudaStream_t st) {
  if (D == 64) return a.dt == BF16 ? launch<64, true>(a, st) : launch<64, false>(a, st);
  if (D == 128) return a.dt == BF16 ? launch<128, true>(a, st) : launch<128, false>(a, st);
  return a.dt == BF16 ? launch<256, true>(a, st) : launch<256, false>(a, st);
}

}  // namespace kv4
