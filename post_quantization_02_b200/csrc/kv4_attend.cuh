// What the attention kernels over the 4-bit cache share: arguments, the keys
// a tile of query rows sees, and the division of the work.
//
// Rows of a sequence and key/value head: r = query * group + (query head within
// the group), so a tile of R consecutive rows shares the keys it reads.  Key
// blocks a tile sees: the first `sb` blocks (the sinks) and blocks lb .. he-1
// (the window, or everything); block i of the tile's nb is i < sb ? i : lb + i - sb.
//
// Lengths are on the device (a captured graph serves any), so the division is
// made there: every block adds up the work of the batch, sets the chunk of key
// blocks of one unit, and finds its own (sequence, tile, split) in the running
// sum of units.  The chunk is chosen for whole waves: of eight that give between
// one and two units for each of the `resident` blocks the device holds at a time, the
// one with the least waves x (mean unit + a unit's fixed cost).  A sequence with one split is written
// straight to the output; the units of the others leave partial results, in
// slots counted over those sequences alone, that kv4_merge_kernel joins.
#pragma once

#include <algorithm>

#include "kv4.cuh"

namespace kv4 {

struct Part {            // one (row, split): unnormalised sum relative to 2^m
  float m, l;
};

struct AttendArgs {
  const uint16_t* q;
  int64_t q_st, q_sh;
  int q_vec;             // 16-byte loads fit
  void* out;
  int64_t o_st, o_sh;
  float* lse;            // T x Hq, or null
  Cache cache;
  Batch b;
  int T, Hq, g, dt;
  int causal, window, sinks;
  float scale_log2;      // softmax scale x log2 e
  int min_chunk;         // key blocks
  int resident;          // blocks on the device at a time
  float unit_cost;       // what a unit costs beside its key blocks, in key blocks
  float* part_o;         // slots x heads x R x D
  Part* part_ml;         // slots x heads x R
  int2* meta;            // per sequence: first slot, splits; then the sequences that count
  int32_t* info;
};

struct Seq {
  int row0, n, L;        // first token row, new tokens, cached tokens
};

struct Unit {
  int b, tile, split, nsplit;
  int head, slot;        // its key/value head; its slot, if it is one of several splits
};

struct Span {
  int sb, lb, nb;
};

// bad: set when the batch's numbers contradict each other or the table
KQ_DEV Seq seq_of(const AttendArgs& a, int b, bool* bad) {
  Seq s;
  const int s0 = a.b.q_start[b], s1 = a.b.q_start[b + 1];
  const int len = a.b.kv_len[b];
  const int cap = a.b.max_pages << a.cache.lgP;
  s.row0 = s0;
  s.n = s1 > s0 && s0 >= 0 && s1 <= a.T ? s1 - s0 : 0;
  s.L = len < 0 ? 0 : len > cap ? cap : len;
  if (bad) *bad = s0 < 0 || s1 < s0 || s1 > a.T || len < 0 || len > cap;
  return s;
}

KQ_DEV int ceil_div(int x, int y) { return (x + y - 1) / y; }

template <int R, int BLK>
KQ_DEV void seq_work(const AttendArgs& a, const Seq& s, int* tiles, int* blocks) {
  *tiles = (int)(((long long)s.n * a.g + R - 1) / R);
  int nb = ceil_div(s.L, BLK);
  if (a.window) {
    const long long w = (long long)min(a.sinks, s.L) / BLK + 1 +
                        ((long long)a.window + min(s.n, R / a.g + 2)) / BLK + 2;
    if (w < nb) nb = (int)w;
  }
  *blocks = nb;
}

// Key blocks the rows of queries q0 .. q1 see.
template <int BLK>
KQ_DEV Span span_of(const AttendArgs& a, const Seq& s, int q0, int q1) {
  const int p0 = s.L - s.n + q0, p1 = s.L - s.n + q1;
  const int hi = a.causal ? min(s.L, p1 + 1) : s.L;
  Span r = {0, 0, 0};
  if (hi <= 0) return r;
  const int lo = a.window ? max(0, min(hi, p0 - a.window + 1)) : 0;
  r.sb = ceil_div(min(a.sinks, lo), BLK);
  r.lb = max(r.sb, lo / BLK);
  r.nb = r.sb + max(0, ceil_div(hi, BLK) - r.lb);
  return r;
}

// Units aimed at, in eighths of `resident`.
constexpr int CHOICES = 8;
KQ_DEV int eighths(int k) { return k < 7 ? 8 + k : 16; }

// Finds the block's unit (all threads call it; false: there is none); heads change
// fastest, so blocks without one come last.  Where q_start goes back, the sequences from there
// on have none: their rows may be others' too, and units and slots are counted for rows that
// are one sequence's.  Of up to 32
// sequences every warp finds it by itself, one sequence a lane, without a barrier.
// Work and costs are fp32 sums in one order, so all blocks agree; the chunk is
// rounded up by more than their error, which keeps max_units a bound.
template <int R, int BLK, int THREADS>
KQ_DEV bool find_unit(const AttendArgs& a, Unit* out) {
  constexpr int WARPS = THREADS / 32;
  __shared__ float sums[WARPS];
  __shared__ int firsts[WARPS];
  __shared__ uint32_t counts[WARPS][CHOICES];
  __shared__ unsigned long long wsum[WARPS];
  __shared__ Unit found;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int u = blockIdx.x / a.cache.heads;
  out->head = blockIdx.x - u * a.cache.heads;
  const bool wide = a.b.B > 32;
  const int per = ceil_div(a.b.B, THREADS);
  const int b0 = min(a.b.B, wide ? tid * per : lane), b1 = min(a.b.B, b0 + per);
  int tiles1 = 0, blocks1 = 0;                 // kept when a thread has one sequence
  float work = 0.f;
  int good = a.b.B;                            // the sequences that count
  for (int b = b0; b < b1; ++b) {
    bool bad;
    seq_work<R, BLK>(a, seq_of(a, b, &bad), &tiles1, &blocks1);
    if (bad && blockIdx.x == 0) kq::record_error(a.info, KRONQ_ERR_INVALID_ARG);
    if (bad && a.b.q_start[b + 1] < a.b.q_start[b]) good = min(good, b);
    work += (float)tiles1 * (float)blocks1;
  }
  good = __reduce_min_sync(0xffffffffu, good);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) work += __shfl_xor_sync(0xffffffffu, work, o);
  if (wide) {
    if (lane == 0) {
      sums[warp] = work;
      firsts[warp] = good;
    }
    if (tid == 0) found.b = -1;
    __syncthreads();
    work = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      work += sums[w];
      good = min(good, firsts[w]);
    }
  }
  if (blockIdx.x == 0 && tid == 0) a.meta[a.b.B] = make_int2(good, 0);
  if (b0 >= good) tiles1 = 0;
  // (work counts the others too: the chunk is no smaller for it)
  auto work_of = [&](int b) {
    if (per > 1) seq_work<R, BLK>(a, seq_of(a, b, nullptr), &tiles1, &blocks1);
    if (b >= good) tiles1 = 0;
  };
  work *= a.cache.heads;
  // lane k: the chunk of choice k % CHOICES
  const float aim = 0.125f * (float)(eighths(lane % CHOICES) * a.resident);
  const int mine_c = (int)fmaxf((float)a.min_chunk, ceilf(fminf(__fdividef(work, aim) * (1.00001f + per * 0x1p-23f), 0x1p30f)));
  int chunk = __shfl_sync(0xffffffffu, mine_c, 0);
  if (chunk > a.min_chunk) {                   // (the same in all threads)
    const float mine_r = __frcp_rn((float)mine_c);
    float n[CHOICES], r[CHOICES];
#pragma unroll
    for (int k = 0; k < CHOICES; ++k) {
      n[k] = 0.f;
      r[k] = __shfl_sync(0xffffffffu, mine_r, k);
    }
    for (int b = b0; b < b1; ++b) {
      work_of(b);
#pragma unroll
      for (int k = 0; k < CHOICES; ++k)
        n[k] += (float)tiles1 * fmaxf(1.f, ceilf((float)blocks1 * r[k]));
    }
    uint32_t units = 0;                        // lane k: of choice k % CHOICES
#pragma unroll
    for (int k = 0; k < CHOICES; ++k) {
      const uint32_t x = __reduce_add_sync(0xffffffffu, (uint32_t)n[k]);
      if (lane % CHOICES == k) units = x;
    }
    if (wide) {
      if (lane < CHOICES) counts[warp][lane] = units;
      __syncthreads();
      units = 0;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) units += counts[w][lane % CHOICES];
    }
    const float all = (float)units * a.cache.heads;
    const float waves = __fdividef(all, (float)a.resident);
    const float cost = ceilf(waves) * __fdividef(work, all) + waves * a.unit_cost;
    const uint32_t best =
        __reduce_min_sync(0xffffffffu, (__float_as_uint(cost) & ~7u) | (lane % CHOICES));
    chunk = __shfl_sync(0xffffffffu, mine_c, best & 7);
  }
  // low half: units; high half: those that need a slot
  unsigned long long units = 0;
  for (int b = b0; b < b1; ++b) {
    work_of(b);
    const int ns = max(1, ceil_div(blocks1, chunk));
    const unsigned long long k = (unsigned long long)tiles1 * ns;
    units += k + (ns > 1 ? k << 32 : 0);
  }
  unsigned long long incl = units;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  unsigned long long before = incl - units;
  if (wide) {
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WARPS; ++w)
      if (w < warp) before += wsum[w];
  }
  int base = (int)(uint32_t)before, slot0 = (int)(before >> 32);
  Unit x = {-1, 0, 0, 1, out->head, 0};
  if (u >= base && u < base + (int)(uint32_t)units) {
    for (int b = b0; b < b1; ++b) {
      work_of(b);
      const int ns = max(1, ceil_div(blocks1, chunk)), k = tiles1 * ns;
      if (u < base + k) {
        x.tile = (u - base) / ns;
        x.split = u - base - x.tile * ns;
        x.nsplit = ns;
        x.slot = slot0 + u - base;
        x.b = b;
        break;
      }
      base += k;
      if (ns > 1) slot0 += k;
    }
    if (wide) found = x;
  }
  if (wide) {
    __syncthreads();
    *out = found;
    return found.b >= 0;
  }
  const uint32_t has = __ballot_sync(0xffffffffu, x.b >= 0);
  if (!has) return false;
  const int src = __ffs(has) - 1;
  out->b = src;
  out->tile = __shfl_sync(0xffffffffu, x.tile, src);
  out->split = __shfl_sync(0xffffffffu, x.split, src);
  out->nsplit = __shfl_sync(0xffffffffu, x.nsplit, src);
  out->slot = __shfl_sync(0xffffffffu, x.slot, src);
  return true;
}

KQ_DEV uint2 pack4(float4 o, int dt) {
  if (dt == BF16) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(o.x, o.y), y = __floats2bfloat162_rn(o.z, o.w);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
  }
  const __half2 x = __floats2half2_rn(o.x, o.y), y = __floats2half2_rn(o.z, o.w);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
}

// Four dims from d on of one output row from its sum relative to 2^m; a row
// that saw no key is 0 with a log-sum-exp of -inf.
KQ_DEV void store_row(const AttendArgs& a, int row, int hq, int d, float4 o, float m, float l) {
  const float r = l == 0.f ? 0.f : 1.f / l;
  o.x *= r;
  o.y *= r;
  o.z *= r;
  o.w *= r;
  uint16_t* p = static_cast<uint16_t*>(a.out) + (int64_t)row * a.o_st + (int64_t)hq * a.o_sh + d;
  *reinterpret_cast<uint2*>(p) = pack4(o, a.dt);
  if (a.lse && d == 0)
    a.lse[(int64_t)row * a.Hq + hq] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// kv4_prompt.cu: its rows per tile, keys per block, launch.
int prompt_rows(int D);
int prompt_block(int D);
int launch_prompt(const AttendArgs& a, int D, cudaStream_t st);

// Bounds of what find_unit hands out: a sequence with t tiles and w key blocks
// has t ceil(w / chunk) <= t + t w / chunk units, and at most twice t w / chunk
// when it is split; the sum of t w / chunk is at most 2 resident / heads.  Blocks
// without a unit still look for one, so the grid is also kept to what the table's
// width can give.
inline long long max_units(const AttendArgs& a, int R, int BLK) {    // of all heads
  const long long tiles = (long long)a.T * a.g / R + a.b.B;
  const long long blocks = (((long long)a.b.max_pages << a.cache.lgP) + BLK - 1) / BLK;
  const long long each = (blocks + a.min_chunk - 1) / a.min_chunk;
  return a.cache.heads *
         std::min(tiles + 2 * a.resident / a.cache.heads + 1, tiles * std::max(1ll, each));
}
inline long long max_slots(int heads, int resident) { return 4 * resident / heads + 2; }

}  // namespace kv4
