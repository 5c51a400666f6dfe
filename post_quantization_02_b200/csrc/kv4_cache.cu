// Writing and reading back the paged 4-bit key/value cache (layout: kv4.cuh).
//
// kv4_append_kernel: for each new token the rotation by its position, then the
// signed Hadamard transform (keys and queries), then the 4-bit grid (keys and
// values).  Every step is one fp32 operation with its own rounding, in a fixed
// order, so codes and words are reproducible bit for bit:
//   rotation      y_a = a cos - b sin, y_b = b cos + a sin
//   Hadamard      x -> D^-1/2 H (signs x), butterflies of distance 1, 2, 4, ...
//   grid          lo = min(0, min x), hi = max(0, max x),
//                 s = max((hi - lo) (1/15), 2^-100) rounded to 20 bits, r = 1/s,
//                 zero = clamp(rint(-lo r), 0, 15),
//                 code = clamp(rint(x r) + zero, 0, 15)
// (the library's asymmetric grid with the division by s as a product with
// 1/s, taken once per vector: a division per value would cost more than the
// whole rest).  A vector with a NaN or an infinity, or wider than fp32, gets a
// NaN scale: it reads back as NaN instead of as some other value.
//
// Split: 8 lanes per vector (a query, key or value head of one token), four vectors
// of the same token per warp; lane l holds dims 8 l + 64 r .. + 8, so loads are 16
// bytes per lane and 128 bytes per vector and r, the first three butterflies and the
// last (D/64) are inside the lane, three go by shuffle, and a run of 8 dims is one
// word of codes.  (64 dims per lane, with fewer shuffles, needs 160 registers: a fifth
// slower.)  What bounds it is instructions (70 % of the issue slots) and the loads, stores and
// shuffles among them (76 % of what L1 passes), so fp32 operations go in packed pairs, a
// block looks its token's place up once for all its vectors, and the first vector is
// asked for before that.  Measured: 34k tokens of 64 query and 2 x 8 key/value heads of
// 128, bf16, both rotations: 367 us, 3.6 TB/s read and written; without rotations 268.
#include "kv4.cuh"

namespace {

using namespace kv4;

constexpr int TPB = 128;
constexpr int ITEMS = TPB / 8;      // vectors per block

struct Rows {
  const uint16_t* p;
  int64_t st, sh;     // strides of the token and of the head (elements)
  int vec;
};

struct AppendArgs {
  Rows q, k, v;
  uint16_t* q_out;
  Cache cache;
  Batch b;
  const float* table;         // table_rows x rot: cosines, then sines
  const int32_t* positions;
  const int8_t* signs;
  int64_t table_rows;
  int T, Hq, dt, rot, interleaved;
  int32_t* info;
};

// Where a sequence's token `at` lies: its page, or -1 when it is not a token
// of a cached page.
KQ_DEV int64_t page_of(const Batch& b, const Cache& c, int s, int at) {
  const int pg = at >> c.lgP;
  if (at < 0 || pg >= b.max_pages) return -1;
  const int64_t id = b.table[s * b.table_ld + pg];
  return id >= 0 && id < c.pages ? id : -1;
}

// The index of row i of sequence s among its tokens; negative where the sequence's rows are not
// rows of the tensor or end in front of i (starts that go back).
KQ_DEV int index_of(const Batch& b, int s, int i, int T) {
  const int s0 = b.q_start[s], s1 = b.q_start[s + 1], len = b.kv_len[s];
  return s0 >= 0 && s1 <= T && i < s1 ? len - (s1 - i) : -1;
}

// Block 0 looks for row starts that go back or leave the tensor's rows (after a search, which
// leaves them in L1).
KQ_DEV void check_starts(const Batch& b, int T, int32_t* info) {
  if (blockIdx.x || blockIdx.y) return;
  bool bad = false;
  for (int s = threadIdx.x; s < b.B; s += TPB) {
    const int s0 = b.q_start[s], s1 = b.q_start[s + 1];
    bad |= s0 < 0 || s1 < s0 || s1 > T;
  }
  if (bad) kq::record_error(info, KRONQ_ERR_INVALID_ARG);
}

// Products that are rounded by themselves: packed ones (and fused ones with a zero) are
// contracted with the packed sum behind them.
KQ_DEV f32x2 mul2_rn(f32x2 a, f32x2 b) {
  const float2 x = unpack2(a), y = unpack2(b);
  return pack2(__fmul_rn(x.x, y.x), __fmul_rn(x.y, y.y));
}

// x: dims 8 l + 64 r + 2 i and the next, in the order written above, packed in pairs.
// (Registers are capped for 4 to 6 blocks per SM: 34k tokens 391 us without, 367 with.)
template <int D, int DT>
__global__ void __launch_bounds__(TPB, D == 64 ? 6 : D == 128 ? 5 : 4) kv4_append_kernel(const AppendArgs a) {
  constexpr int R = D / 64;
  const int i = blockIdx.x, l = threadIdx.x & 7;
  const int Hkv = a.cache.heads, items = a.Hq + 2 * Hkv;
  int item = blockIdx.y * ITEMS + (threadIdx.x >> 3);
  const int stride = gridDim.y * ITEMS;
  // the first vector is asked for before its place is looked up (every row may be read)
  uint4 in[R];
  auto source = [&](int it, const Rows** src) -> const uint16_t* {
    const int kind = it < a.Hq ? 0 : it < a.Hq + Hkv ? 1 : 2;
    const int head = kind == 0 ? it : kind == 1 ? it - a.Hq : it - a.Hq - Hkv;
    *src = kind == 0 ? &a.q : kind == 1 ? &a.k : &a.v;
    return (*src)->p + (int64_t)i * (*src)->st + (int64_t)head * (*src)->sh;
  };
  auto ask = [&](int it) {
#pragma unroll
    for (int r = 0; r < R; ++r) in[r] = make_uint4(0u, 0u, 0u, 0u);
    if (it < items) {
      const Rows* src;
      const uint16_t* p = source(it, &src) + 8 * l;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (src->vec) {
          in[r] = __ldg(reinterpret_cast<const uint4*>(p + 64 * r));
        } else {
          uint32_t w[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) w[j] = __ldg(p + 64 * r + j);
          in[r] = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
        }
      }
    }
  };
  ask(item);
  const int s = find_sequence(a.b.q_start, a.b.B, i);
  check_starts(a.b, a.T, a.info);
  if (s < 0 || s >= a.b.B) return;                       // a row of no sequence
  const int at = index_of(a.b, s, i, a.T);
  const int64_t pos = a.positions ? a.positions[i] : at;
  const bool placed = at >= 0 && (!a.rot || (pos >= 0 && pos < a.table_rows));
  const int64_t page = placed ? page_of(a.b, a.cache, s, at) : -1;
  if (page < 0 && threadIdx.x == 0) kq::record_error(a.info, KRONQ_ERR_INVALID_ARG);
  const float* row = a.table + (placed && a.rot ? pos * a.rot : 0);
  const int half = a.rot >> 1;
  // +-1 for each dim of this lane
  f32x2 sg[R][4];
  if (a.signs) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(a.signs + 8 * l + 64 * r));
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t u = k < 2 ? w.x : w.y;
        sg[r][k] = pack2(__uint_as_float(0x3f800000u | ((u << (24 - 16 * (k & 1))) & 0x80000000u)),
                         __uint_as_float(0x3f800000u | ((u << (16 - 16 * (k & 1))) & 0x80000000u)));
      }
    }
  }

  for (; item - (int)(threadIdx.x >> 3) < items; item += stride) {      // (the same in all threads)
    const int kind = item < a.Hq ? 0 : item < a.Hq + Hkv ? 1 : 2;
    const int head = kind == 0 ? item : kind == 1 ? item - a.Hq : item - a.Hq - Hkv;
    const bool ok = item < items && placed && (kind == 0 || page >= 0);
    f32x2 x[R][4];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float v[8];
      unpack8(in[r], DT, v);
#pragma unroll
      for (int k = 0; k < 4; ++k) x[r][k] = pack2(v[2 * k], v[2 * k + 1]);
    }
    if (ok && kind < 2 && a.rot) {
      if (!a.interleaved && a.rot == D && R > 1) {
        // the two halves of a pair are runs r and r + R / 2 of this lane
#pragma unroll
        for (int r = 0; r < R / 2; ++r) {
          const ulonglong2* co = reinterpret_cast<const ulonglong2*>(row + 8 * l + 64 * r);
          const ulonglong2* si = reinterpret_cast<const ulonglong2*>(row + half + 8 * l + 64 * r);
#pragma unroll
          for (int k2 = 0; k2 < 2; ++k2) {
            const ulonglong2 c2 = __ldg(co + k2), s2 = __ldg(si + k2);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const f32x2 c = k ? c2.y : c2.x, sn = k ? s2.y : s2.x;
              f32x2 &u = x[r][2 * k2 + k], &w = x[r + R / 2][2 * k2 + k];
              const f32x2 y = add2(mul2_rn(u, c), mul2_rn(w, neg2(sn)));
              w = add2(mul2_rn(w, c), mul2_rn(u, sn));
              u = y;
            }
          }
        }
      } else if (a.interleaved) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int d = 8 * l + 64 * r;
          if (d >= a.rot) continue;
          const float4 co = __ldg(reinterpret_cast<const float4*>(row + d / 2));
          const float4 si = __ldg(reinterpret_cast<const float4*>(row + half + d / 2));
          const float c4[4] = {co.x, co.y, co.z, co.w}, s4[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 v = unpack2(x[r][k]);
            x[r][k] = add2(mul2_rn(x[r][k], pack2(c4[k], c4[k])), mul2_rn(pack2(v.y, v.x), pack2(-s4[k], s4[k])));
          }
        }
      } else {
        // the other half of each pair is a run of another lane (or of this one): read
        // again, from L1
        const Rows* src;
        const uint16_t* p = source(item, &src);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int d = 8 * l + 64 * r;
          if (d >= a.rot) continue;
          const bool up = d >= half;
          const int e = up ? d - half : d;
          const float g = up ? 1.f : -1.f;
          float o[8];
          load8(p + (up ? e : e + half), src->vec, DT, o);
#pragma unroll
          for (int k2 = 0; k2 < 2; ++k2) {
            const float4 co = __ldg(reinterpret_cast<const float4*>(row + e + 4 * k2));
            const float4 si = __ldg(reinterpret_cast<const float4*>(row + half + e + 4 * k2));
            const f32x2 c[2] = {pack2(co.x, co.y), pack2(co.z, co.w)};
            const f32x2 sn[2] = {pack2(g * si.x, g * si.y), pack2(g * si.z, g * si.w)};
#pragma unroll
            for (int k = 0; k < 2; ++k)
              x[r][2 * k2 + k] = add2(mul2_rn(x[r][2 * k2 + k], c[k]),
                                      mul2_rn(pack2(o[4 * k2 + 2 * k], o[4 * k2 + 2 * k + 1]), sn[k]));
          }
        }
      }
    }
    // (the next vector comes while this one is transformed; what this one's lanes read of each
    // other is read before any of them writes)
    ask(item + stride);
    __syncwarp();

    if (a.signs && __any_sync(0xffffffffu, kind < 2)) {
      f32x2 y[R][4];
      const f32x2 minus = pack2(-1.f, -1.f);
      auto butterfly = [&](f32x2& u, f32x2& w) {
        const f32x2 t = add2(u, w);
        w = fma2(w, minus, u);
        u = t;
      };
#pragma unroll
      for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {                       // distance 1
          const float2 v = unpack2(mul2(x[r][k], sg[r][k]));     // (exact)
          y[r][k] = pack2(__fadd_rn(v.x, v.y), __fsub_rn(v.x, v.y));
        }
        butterfly(y[r][0], y[r][1]);                        // 2
        butterfly(y[r][2], y[r][3]);
        butterfly(y[r][0], y[r][2]);                        // 4
        butterfly(y[r][1], y[r][3]);
      }
#pragma unroll
      for (int h = 1; h < 8; h *= 2) {                      // 8, 16, 32: other lanes
        const float g = (l & h) ? -1.f : 1.f;
        const f32x2 g2 = pack2(g, g);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int k = 0; k < 4; ++k) y[r][k] = fma2(y[r][k], g2, __shfl_xor_sync(0xffffffffu, y[r][k], h));
      }
#pragma unroll
      for (int h = 1; h < R; h *= 2)                        // 64, 128
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (!(r & h))
#pragma unroll
            for (int k = 0; k < 4; ++k) butterfly(y[r][k], y[r + h][k]);
      constexpr float norm = D == 64 ? 0.125f : D == 128 ? 0.08838834764831845f : 0.0625f;
      const f32x2 n2 = pack2(norm, norm);
      if (kind < 2) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int k = 0; k < 4; ++k) x[r][k] = mul2(y[r][k], n2);
      }
    }

    if (kind == 0 && ok) {
      uint16_t* o = a.q_out + ((int64_t)i * a.Hq + head) * D + 8 * l;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 w = unpack2(x[r][k]);
          v[2 * k] = w.x;
          v[2 * k + 1] = w.y;
        }
        *reinterpret_cast<uint4*>(o + 64 * r) = pack8(v, DT);
      }
    }
    // a warp that holds only queries is done with them; in a mixed warp all lanes go on
    if (__all_sync(0xffffffffu, kind == 0 || !ok)) continue;

    float lo = 0.f, hi = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 v = unpack2(x[r][k]);
        lo = min_nan(lo, min_nan(v.x, v.y));
        hi = max_nan(hi, max_nan(v.x, v.y));
      }
#pragma unroll
    for (int h = 1; h < 8; h *= 2) {
      lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, h));
      hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, h));
    }
    if (!ok || kind == 0) continue;
    float sc = fmaxf(__fmul_rn(__fsub_rn(hi, lo), 1.f / 15.f), 0x1p-100f);
    if (!(__fsub_rn(hi, lo) < INFINITY)) sc = INFINITY;     // NaN, infinite or too wide
    sc = __uint_as_float((__float_as_uint(sc) + 8u) & ~15u);
    uint32_t word = 0x7FC00000u, code[R];
#pragma unroll
    for (int r = 0; r < R; ++r) code[r] = 0;
    if (sc < INFINITY) {
      // 1.5 2^23 + y is rounded to a whole number as rint rounds y (|y| <= 16); the code
      // is clamped there and taken from the low bits
      constexpr float M = 12582912.f;
      const float rs = __fdiv_rn(1.f, sc);
      const float z = fminf(fmaxf(rintf(__fmul_rn(-lo, rs)), 0.f), 15.f);
      const f32x2 rs2 = pack2(rs, rs), m2 = pack2(M, M), z2 = pack2(z, z);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 y = unpack2(add2(add2(mul2_rn(x[r][k], rs2), m2), z2));
          code[r] |= (__float_as_uint(fminf(fmaxf(y.x, M), M + 15.f)) & 15u) << (8 * k) |
                     (__float_as_uint(fminf(fmaxf(y.y, M), M + 15.f)) & 15u) << (8 * k + 4);
        }
      word = __float_as_uint(sc) | (uint32_t)z;
    }
    const int P = a.cache.P, slot = at & (P - 1);
    uint8_t* blk = a.cache.base + (page * Hkv + head) * (int64_t)a.cache.block_bytes;
    uint32_t* codes = reinterpret_cast<uint32_t*>(blk + (kind == 2 ? P * (D / 2) : 0)) + slot * (D / 8);
#pragma unroll
    for (int r = 0; r < R; ++r) codes[l + 8 * r] = code[r];
    if (l == 0) (reinterpret_cast<uint32_t*>(blk + P * D) + (kind == 2 ? P : 0))[slot] = word;
  }
}

template <int D>
void launch_append(const AppendArgs& a, dim3 grid, cudaStream_t st) {
  if (a.dt == BF16)
    kv4_append_kernel<D, BF16><<<grid, TPB, 0, st>>>(a);
  else
    kv4_append_kernel<D, FP16><<<grid, TPB, 0, st>>>(a);
}

struct GatherArgs {
  void* k_out;        // T x heads x D
  void* v_out;
  Cache cache;
  Batch b;
  int T, dt;
  int32_t* info;
};

// Reads tokens back as the values they stand for, the last new tokens of each sequence:
// bound by the stores (2 bytes or 4 for half a byte read; bf16 and fp32 write at the same rate,
// though bf16 has the integer pipe at 71 % and fp32 does half the work a byte).  A block takes N tokens; their
// places are looked up once, a warp per token, and 8 lanes read a vector as above.  N = 8
// keeps four vectors of a thread in flight; few tokens are spread instead (N = 1).  34k
// tokens of 2 x 8 heads of 128 as bf16: 41 us, 3.4 TB/s written (N = 1: 50); as fp32 76, 3.7.
template <int D, int N>
__global__ void __launch_bounds__(TPB) kv4_gather_kernel(const GatherArgs a) {
  constexpr int R = D / 64;
  __shared__ const uint8_t* place[N];      // the page's block of head 0, or null
  __shared__ int slots[N];
  const int Hkv = a.cache.heads, P = a.cache.P, lane = threadIdx.x & 31;
  for (int n = threadIdx.x >> 5; n < N; n += TPB / 32) {
    const int i = blockIdx.x * N + n;
    const uint8_t* p = nullptr;
    int slot = 0;
    if (i < a.T) {                         // (the same in the whole warp)
      const int s = find_sequence(a.b.q_start, a.b.B, i);
      if (s >= 0 && s < a.b.B) {
        const int at = index_of(a.b, s, i, a.T);
        const int64_t page = page_of(a.b, a.cache, s, at);
        if (page >= 0) {
          p = a.cache.base + page * Hkv * (int64_t)a.cache.block_bytes;
          slot = at & (P - 1);
        } else if (lane == 0) {
          kq::record_error(a.info, KRONQ_ERR_INVALID_ARG);
        }
      }
    }
    if (lane == 0) {
      place[n] = p;
      slots[n] = slot;
    }
  }
  check_starts(a.b, a.T, a.info);
  __syncthreads();
  const int l = threadIdx.x & 7;
  constexpr int U = N == 1 ? 1 : 4;        // vectors in flight
  for (int e0 = threadIdx.x >> 3; e0 < N * 2 * Hkv; e0 += U * ITEMS) {
    uint32_t word[U], c[U][R];
    int64_t row[U];                        // of the output, + 2^62: values; negative: none
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int e = min(e0 + u * ITEMS, N * 2 * Hkv - 1);
      const int n = N == 1 ? 0 : e / (2 * Hkv), item = e - n * (2 * Hkv);
      const int isv = item >= Hkv, head = isv ? item - Hkv : item, slot = slots[n];
      const bool here = place[n] && e == e0 + u * ITEMS;
      // (without a page the pool's first bytes are read, and nothing is stored)
      const uint8_t* blk = (place[n] ? place[n] : a.cache.base) + head * (int64_t)a.cache.block_bytes;
      const uint32_t* codes =
          reinterpret_cast<const uint32_t*>(blk + (isv ? P * (D / 2) : 0)) + slot * (D / 8);
      word[u] = __ldg(reinterpret_cast<const uint32_t*>(blk + P * D) + (isv ? P : 0) + slot);
#pragma unroll
      for (int r = 0; r < R; ++r) c[u][r] = __ldg(codes + l + 8 * r);
      row[u] = here ? ((((int64_t)(blockIdx.x * N + n) * Hkv + head) * D) | ((int64_t)isv << 62)) : -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (row[u] < 0) continue;
      const float sc = word_scale(word[u]), z = word_zero(word[u]);
      void* out = row[u] >> 62 ? a.v_out : a.k_out;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          x[j] = __fmul_rn(sc, __fsub_rn(__uint_as_float(0x4B000000u | ((c[u][r] >> (4 * j)) & 15u)),
                                         8388608.f + z));
        const int64_t o = (row[u] & ((1ll << 62) - 1)) + 8 * l + 64 * r;
        if (a.dt == FP32) {
          float4* f = reinterpret_cast<float4*>(static_cast<float*>(out) + o);
          f[0] = make_float4(x[0], x[1], x[2], x[3]);
          f[1] = make_float4(x[4], x[5], x[6], x[7]);
        } else {
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + o) = pack8(x, a.dt);
        }
      }
    }
  }
}

template <int D>
void launch_gather(const GatherArgs& a, cudaStream_t st) {
  constexpr int N = 8;
  if (a.T < 8 * kqh::num_sms())
    kv4_gather_kernel<D, 1><<<(unsigned)a.T, TPB, 0, st>>>(a);
  else
    kv4_gather_kernel<D, N><<<(unsigned)((a.T + N - 1) / N), TPB, 0, st>>>(a);
}

}  // namespace

int kq_kv4_views(void* cache, int64_t pages, int page_size, int heads, int D, const int32_t* table,
                 int64_t table_ld, int64_t max_pages, const int32_t* q_start, const int32_t* kv_len,
                 int64_t B, Cache* c, Batch* b) {
  if (D != 64 && D != 128 && D != 256) return KRONQ_ERR_UNSUPPORTED;
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128 && page_size != 256)
    return KRONQ_ERR_UNSUPPORTED;
  // (no sequences: their tensors have no memory; calls with tokens refuse it)
  if (!cache || (B && (!q_start || !kv_len)) || pages <= 0 || pages > INT32_MAX || heads <= 0 ||
      heads > 65535 || B < 0 || B > (1 << 20))
    return KRONQ_ERR_INVALID_ARG;
  if (max_pages < 0 || table_ld < max_pages || (B && max_pages && !table)) return KRONQ_ERR_INVALID_ARG;
  if (max_pages > (1 << 30) / page_size) return KRONQ_ERR_UNSUPPORTED;   // token indices stay below 2^30
  if (!kqh::aligned(cache, 16) || !kqh::aligned(table, 4) || !kqh::aligned(q_start, 4) ||
      !kqh::aligned(kv_len, 4))
    return KRONQ_ERR_INVALID_ARG;
  c->base = static_cast<uint8_t*>(cache);
  c->pages = pages;
  c->P = page_size;
  c->lgP = 31 - __builtin_clz((unsigned)page_size);
  c->heads = heads;
  c->block_bytes = page_size * (D + 8);
  b->table = table;
  b->q_start = q_start;
  b->kv_len = kv_len;
  b->table_ld = table_ld;
  b->B = (int)B;
  b->max_pages = (int)max_pages;
  return KRONQ_OK;
}

namespace {

bool rows_ok(const void* p, int64_t st, int64_t sh, Rows* r) {
  if (!p || !kqh::aligned(p, 2) || st < 0 || sh < 0) return false;
  r->p = static_cast<const uint16_t*>(p);
  r->st = st;
  r->sh = sh;
  r->vec = kqh::aligned(p, 16) && st % 8 == 0 && sh % 8 == 0;
  return true;
}

}  // namespace

int kq_kv4_append(const void* q, int64_t q_st, int64_t q_sh, const void* k, int64_t k_st, int64_t k_sh,
                  const void* v, int64_t v_st, int64_t v_sh, int dtype, int64_t T, int Hq, void* q_out,
                  const float* table, int64_t table_rows, int rot, int interleaved,
                  const int32_t* positions, const int8_t* signs, int D, const Cache& c, const Batch& b,
                  int32_t* info, cudaStream_t st) {
  if (dtype != BF16 && dtype != FP16) return KRONQ_ERR_UNSUPPORTED;
  if (T < 0 || Hq < 0 || Hq > 65535 || rot < 0 || rot > D || rot % 16) return KRONQ_ERR_INVALID_ARG;
  if (rot && (!table || table_rows <= 0 || !kqh::aligned(table, 16))) return KRONQ_ERR_INVALID_ARG;
  if (!kqh::aligned(positions, 4) || !kqh::aligned(signs, 8)) return KRONQ_ERR_INVALID_ARG;
  if (T == 0) return KRONQ_OK;
  if (!b.B) return KRONQ_ERR_INVALID_ARG;
  AppendArgs a = {};
  if (!rows_ok(k, k_st, k_sh, &a.k) || !rows_ok(v, v_st, v_sh, &a.v)) return KRONQ_ERR_INVALID_ARG;
  if (Hq) {
    if (!rows_ok(q, q_st, q_sh, &a.q) || !q_out || !kqh::aligned(q_out, 16)) return KRONQ_ERR_INVALID_ARG;
    // A vector is read by its own 8 lanes before they write it, so queries may be rotated where
    // they lie; any other overlap would be a race.
    const KqRows to = {q_out, (int64_t)Hq * D, D, T, Hq, D};
    const bool in_place = q == q_out && (T == 1 || q_st == to.st) && (Hq == 1 || q_sh == to.sh);
    if ((!in_place && to.meets({q, q_st, q_sh, T, Hq, D})) || to.meets({k, k_st, k_sh, T, c.heads, D}) ||
        to.meets({v, v_st, v_sh, T, c.heads, D}))
      return KRONQ_ERR_INVALID_ARG;
  }
  a.q_out = static_cast<uint16_t*>(q_out);
  a.cache = c;
  a.b = b;
  a.table = table;
  a.positions = positions;
  a.signs = signs;
  a.table_rows = table_rows;
  a.Hq = Hq;
  a.dt = dtype;
  a.rot = rot;
  a.interleaved = interleaved;
  a.info = info;
  if (T > INT32_MAX) return KRONQ_ERR_UNSUPPORTED;
  a.T = (int)T;
  // a block per token; with few tokens their vectors are spread over more blocks (34k tokens
  // of 80 vectors: 367 us, spread 563; 3.8k tokens of 20: 24, spread 30)
  const int passes = (Hq + 2 * c.heads + ITEMS - 1) / ITEMS;
  const dim3 grid((unsigned)T, T < 8 * kqh::num_sms() ? (unsigned)passes : 1u);
  if (D == 64)
    launch_append<64>(a, grid, st);
  else if (D == 128)
    launch_append<128>(a, grid, st);
  else
    launch_append<256>(a, grid, st);
  KQ_CHECK_LAUNCH();
  return KRONQ_OK;
}

int kq_kv4_gather(void* k_out, void* v_out, int dtype, int64_t T, int D, const Cache& c, const Batch& b,
                  int32_t* info, cudaStream_t st) {
  if (dtype != BF16 && dtype != FP16 && dtype != FP32) return KRONQ_ERR_UNSUPPORTED;
  if (T < 0) return KRONQ_ERR_INVALID_ARG;
  if (T == 0) return KRONQ_OK;
  if (!b.B || !k_out || !v_out || !kqh::aligned(k_out, 16) || !kqh::aligned(v_out, 16)) return KRONQ_ERR_INVALID_ARG;
  GatherArgs a = {};
  a.k_out = k_out;
  a.v_out = v_out;
  a.cache = c;
  a.b = b;
  a.dt = dtype;
  a.info = info;
  if (T > INT32_MAX - 8) return KRONQ_ERR_UNSUPPORTED;
  a.T = (int)T;
  if (D == 64)
    launch_gather<64>(a, st);
  else if (D == 128)
    launch_gather<128>(a, st);
  else
    launch_gather<256>(a, st);
  KQ_CHECK_LAUNCH();
  return KRONQ_OK;
}
