// Layout and grid of the paged 4-bit key/value cache, shared by the kernels
// that write it and the kernels that read it.
//
// A page holds P tokens of every key/value head.  The block of one (page,
// head) is contiguous, P (D + 8) bytes:
//   key codes    P x D/2 bytes    byte i of a token: dims 2i (low nibble), 2i+1
//   value codes  P x D/2 bytes
//   key words    P x uint32
//   value words  P x uint32
// so 8 consecutive dims are one 32-bit word with dim j in bits [4j, 4j + 4),
// the order of kronq_pack.  A token's word is its fp32 scale with the low 4
// mantissa bits replaced by the zero point: 4 bytes per 2 D/2 bytes of codes,
// the full fp32 range and 20 significant bits.  value = scale (code - zero).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace kv4 {

enum Dtype { BF16 = 0, FP16 = 1, FP32 = 2 };

// The batch: new tokens of sequence b are rows q_start[b] .. q_start[b+1]-1;
// kv_len[b] tokens are cached once they are in; its t-th page is table[b * ld + t].
struct Batch {
  const int32_t* table;
  const int32_t* q_start;
  const int32_t* kv_len;
  int64_t table_ld;
  int B;
  int max_pages;
};

struct Cache {
  uint8_t* base;
  int64_t pages;
  int P, lgP;
  int heads;
  int block_bytes;   // P (D + 8)
};

KQ_DEV float word_scale(uint32_t w) { return __uint_as_float(w & ~15u); }
// the zero point as a float: exact integers 0 .. 15
KQ_DEV float word_zero(uint32_t w) {
  return __fsub_rn(__uint_as_float(0x4B000000u | (w & 15u)), 8388608.f);
}

// min / max that keep a NaN
KQ_DEV float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
KQ_DEV float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Two fp32 in one 64-bit register: one instruction for both.
using f32x2 = unsigned long long;
KQ_DEV f32x2 pack2(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
KQ_DEV float2 unpack2(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
KQ_DEV f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
KQ_DEV f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
KQ_DEV f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
KQ_DEV f32x2 neg2(f32x2 a) { return a ^ 0x8000000080000000ull; }

KQ_DEV float to_f32(uint16_t h, int dt) {
  return dt == BF16 ? __uint_as_float((uint32_t)h << 16) : __half2float(__ushort_as_half(h));
}

KQ_DEV void unpack8(const uint4& u, int dt, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (dt == BF16) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

KQ_DEV uint4 pack8(const float (&x)[8], int dt) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (dt == BF16) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    } else {
      const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 8 consecutive elements at p: one 16-byte load, or element loads where the
// tensor's address or strides are not multiples of 16 bytes.
KQ_DEV void load8(const uint16_t* p, bool vec, int dt, float (&x)[8]) {
  if (vec) {
    unpack8(__ldg(reinterpret_cast<const uint4*>(p)), dt, x);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = to_f32(__ldg(p + i), dt);
  }
}

// Sequence of token row i: the last b with q_start[b] <= i, found by the whole
// warp 32 probes at a time (i is the same in all lanes).  -1: in front of
// q_start[0]; B: behind the last sequence.
KQ_DEV int find_sequence(const int32_t* __restrict__ q_start, int B, int i) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B + 1;                     // the first entry > i lies in [lo, lo + n]
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int at = lo + lane * step;
    const bool le = at < lo + n && q_start[at] <= i;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    const int c = __clz(~__brev(m));         // probes in front of the first that is > i
    if (c == 0) return lo - 1;
    lo += (c - 1) * step + 1;                // behind the last probe that is <= i
    n = step - 1;
    if (lo + n > B + 1) n = B + 1 - lo;
  }
  return lo - 1;
}

}  // namespace kv4

// Host side (kv4_cache.cu, kv4_attend.cu).
// T x H rows of D 16-bit elements, strides of the token and of the head.
struct KqRows {
  const void* p;
  int64_t st, sh, T, H, D;
  uintptr_t begin() const { return reinterpret_cast<uintptr_t>(p); }
  uintptr_t end() const { return begin() + 2 * ((T - 1) * st + (H - 1) * sh + D); }
  bool meets(const KqRows& o) const { return begin() < o.end() && o.begin() < end(); }    // as ranges
  // no two rows share memory (token-major or head-major)
  bool apart() const {
    return ((H == 1 || sh >= D) && (T == 1 || st >= (H - 1) * sh + D)) ||
           ((T == 1 || st >= D) && (H == 1 || sh >= (T - 1) * st + D));
  }
};
// The checks every entry point of the cache shares; fills the kernels' views.
int kq_kv4_views(void* cache, int64_t pages, int page_size, int heads, int D, const int32_t* table,
                 int64_t table_ld, int64_t max_pages, const int32_t* q_start, const int32_t* kv_len,
                 int64_t B, kv4::Cache* c, kv4::Batch* b);
int kq_kv4_append(const void* q, int64_t q_st, int64_t q_sh, const void* k, int64_t k_st, int64_t k_sh,
                  const void* v, int64_t v_st, int64_t v_sh, int dtype, int64_t T, int Hq, void* q_out,
                  const float* table, int64_t table_rows, int rot, int interleaved,
                  const int32_t* positions, const int8_t* signs, int D, const kv4::Cache& c,
                  const kv4::Batch& b, int32_t* info, cudaStream_t st);
int kq_kv4_gather(void* k_out, void* v_out, int dtype, int64_t T, int D, const kv4::Cache& c,
                  const kv4::Batch& b, int32_t* info, cudaStream_t st);
size_t kq_kv4_attention_ws(int64_t T, int Hq, int heads, int D, int64_t B);
int kq_kv4_attention(const void* q, int64_t q_st, int64_t q_sh, int dtype, int64_t T, int Hq, int D,
                     const kv4::Cache& c, const kv4::Batch& b, float scale, int causal, int window,
                     int sinks, void* out, int64_t o_st, int64_t o_sh, float* lse, int32_t* info,
                     void* ws, size_t ws_bytes, cudaStream_t st);
