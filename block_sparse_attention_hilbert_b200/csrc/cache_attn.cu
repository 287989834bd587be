// Attention of a few query tokens over the 8-bit block cache, whole or through
// per-query block lists.
//
//   o = sum_t softmax_t(q . k_t / sqrt(d)) v_t,  k_t = ks[block] * code,  v_t = vs[block] * code
//
// Bound by HBM: 2 d bytes per token and key head, against 4 d FLOP per query
// row of the group that shares the head.  The rows of a group (or of several
// query tokens) fill one 16-row tile of mma.sync.m16n8k16: a tcgen05 tile has
// 64 rows at least and takes its operands from shared memory, so the 8-bit
// codes would have to be widened there and read back, for rows that are mostly
// empty; here the codes go from shared memory to registers and are widened on
// the way (8-bit to fp16 is exact, fp16 x fp16 products are exact in fp32).
//
// Work: an item is (sequence, key head, 16-row tile), or with lists (sequence,
// query, key head, tile of the group's rows); a unit is one 64-token block of
// an item.  The CTAs, one per SM, take equal contiguous shares of all units,
// so ragged lengths balance; an item that several CTAs share is joined by a
// second kernel from fp32 partial sums with their maxima, in CTA order.  In a
// CTA, eight warps take the blocks of a segment in turn, each with a ring of
// its own of three 8 KB tiles filled by TMA (128-byte swizzle, so that both
// the row-wise reads of K and the column-wise reads of V are free of bank
// conflicts), and no barrier until the segment's end.
//
// Rounding: q is scaled per row by a power of two into fp16 (exact for bf16
// values within 2^-14 of the row's largest; below that they keep 2^-24 of it);
// softmax weights are rounded to fp16, taken times 2^14 so that weights down
// to 2^-38 of the row's largest keep a value; a block's P V sum is taken on the codes
// alone and joins the fp32 accumulator times the block's scale, so scales of
// any size mix.  Maxima, sums and accumulators are fp32.
#include <cuda_fp8.h>

#include <type_traits>

#include "common.cuh"
#include "stream.cuh"
#include "tcgen05.cuh"

namespace svsa {

static __device__ unsigned int g_cattn_flags;

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kRing = 3;                    // tiles in flight per warp
constexpr int kRows = 16;                   // query rows of a tile
constexpr float kShift = 14.f;              // weights are held times 2^kShift
constexpr int kMinUnits = 8;                // blocks of a CTA at least, where there are as many

struct AttnArgs {
  CacheArgs c;
  const void* q;                            // [B][heads_q][Tq][d]
  const int32_t* idx;                       // nullable: [B][Tq][heads][cap]
  const int32_t* cnt;
  void* o;                                  // [B][heads_q][Tq][d]
  float* lse;                               // nullable [B][heads_q][Tq]
  float* part;                              // [CTA][2][16][d] sums, then [CTA][2][16][2] maxima and row sums
  int heads_q, Tq, causal, cap, group, tiles, grid;
};

// A contiguous range of an item's blocks.
struct Segment {
  int b, t, h, tile;                        // t: the query (lists) or -1
  int j0, j1;                               // blocks, or list positions
  bool starts, ends;                        // holds the item's first / last unit
};

// Where the units lie.  With lists every item has `cap` units; without, the
// items of sequence b have max(1, blocks of b) units each.
struct Walk {
  long long total;                          // units
  int ctas;                                 // CTAs that take some
};

__device__ __forceinline__ int seq_len(const AttnArgs& p, int b) {
  const int n = __ldg(p.c.len + b);
  return min(max(n, 0), p.c.max_blocks * kBlock);
}
__device__ __forceinline__ int seq_units(const AttnArgs& p, int b) {
  return max(1, (seq_len(p, b) + kBlock - 1) / kBlock);
}

__device__ __forceinline__ int active_ctas(long long total, int grid) {
  const long long c = (total + kMinUnits - 1) / kMinUnits;
  return c < grid ? (int)c : grid;
}
__device__ __forceinline__ long long first_unit(long long total, int ctas, int c) { return total * c / ctas; }
// The CTA that holds unit u: the largest c with floor(total c / ctas) <= u.
__device__ __forceinline__ int cta_of(long long total, int ctas, long long u) {
  return (int)(((u + 1) * ctas - 1) / total);
}

// Sum over the sequences of their units (one item each), and the sequence in
// which unit `u` (of sum * per_seq units) lies with the units before it.  The
// whole CTA calls; `red` has kWarps + 4 words.
__device__ long long scan_sequences(const AttnArgs& p, long long* red) {
  long long s = 0;
  for (int b = threadIdx.x; b < p.c.B; b += blockDim.x) s += seq_units(p, b);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  __syncthreads();
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = s;
  __syncthreads();
  s = 0;
  for (int w = 0; w < (int)blockDim.x / 32; ++w) s += red[w];
  return s;
}

// One warp finds the sequence of unit u: 32 sequences a step.
__device__ void find_sequence(const AttnArgs& p, long long u, long long per_seq, int* b_out, long long* before_out) {
  const int lane = threadIdx.x % 32;
  long long before = 0;
  for (int b0 = 0; b0 < p.c.B; b0 += 32) {
    const long long mine = b0 + lane < p.c.B ? (long long)seq_units(p, b0 + lane) * per_seq : 0;
    long long up = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += v;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, before + up > u);
    if (hit) {
      const int l = __ffs(hit) - 1;
      *b_out = b0 + l;
      *before_out = before + __shfl_sync(0xffffffffu, up - mine, l);
      return;
    }
    before += __shfl_sync(0xffffffffu, up, 31);
  }
  *b_out = p.c.B;
  *before_out = before;
}

// The item of unit u and the unit's place in it.
struct Place {
  int b;
  long long before;                         // units before sequence b (dense)
};

__device__ __forceinline__ void item_of(const AttnArgs& p, const Place& pl, long long u, Segment* s, int* units) {
  if (p.idx) {
    const long long item = u / p.cap;
    s->j0 = (int)(u - item * p.cap);
    *units = p.cap;
    long long r = item;
    s->tile = (int)(r % p.tiles);
    r /= p.tiles;
    s->h = (int)(r % p.c.heads);
    r /= p.c.heads;
    s->t = (int)(r % p.Tq);
    s->b = (int)(r / p.Tq);
  } else {
    const int n = seq_units(p, pl.b);
    const long long in = u - pl.before;
    const int item = (int)(in / n);
    s->j0 = (int)(in - (long long)item * n);
    *units = n;
    s->tile = item % p.tiles;
    s->h = item / p.tiles;
    s->t = -1;
    s->b = pl.b;
  }
}

// Row r of a tile: its query and its head in the group; false past the end.
__device__ __forceinline__ bool row_of(const AttnArgs& p, const Segment& s, int r, int* t, int* g) {
  const int i = s.tile * kRows + r;
  if (s.t >= 0) {
    *t = s.t;
    *g = i;
    return i < p.group;
  }
  *t = i / p.group;
  *g = i - *t * p.group;
  return *t < p.Tq;
}

__device__ __forceinline__ uint32_t h2bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }

// Two 8-bit codes (the low or high half of a word) as a pair of fp16, exactly.
template <bool I8>
struct Widen;
template <>
struct Widen<false> {
  __device__ static void word(uint32_t w, uint32_t out[2]) {
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
        : "=r"(out[0]), "=r"(out[1]) : "r"(w));
  }
};
template <>
struct Widen<true> {
  // 0x6400 | (code + 128) is 1024 + code + 128 in fp16
  __device__ static void word(uint32_t w, uint32_t out[2]) {
    const uint32_t u = w ^ 0x80808080u;
    const __half2 off = __floats2half2_rn(1152.f, 1152.f);
    uint32_t lo = __byte_perm(u, 0x64646464u, 0x4140), hi = __byte_perm(u, 0x64646464u, 0x4342);
    out[0] = h2bits(__hsub2(*reinterpret_cast<__half2*>(&lo), off));
    out[1] = h2bits(__hsub2(*reinterpret_cast<__half2*>(&hi), off));
  }
};

__device__ __forceinline__ void mma16816(float d[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];\n" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

template <typename T>
__device__ __forceinline__ float to_f(T x) { return (float)x; }

// Query fragments.  The products sum over d in any order, so the k index of
// the MMA is laid over d as the reads of K want it: lane c of a quad owns the
// d / 4 consecutive values from c * d / 4 on, four per step.
template <int D, typename T>
__device__ __forceinline__ float load_q(const T* q, bool live, int c, uint32_t lo[D / 16], uint32_t hi[D / 16]) {
  float amax = 0.f;
  bool odd = false;
  const uint4* src = reinterpret_cast<const uint4*>(q + c * (D / 4));
  uint4 raw[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) raw[i] = live ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
  auto pair = [&](int i) {                       // values 2i, 2i + 1 of the lane
    const uint32_t w = reinterpret_cast<const uint32_t*>(raw)[i];
    if constexpr (std::is_same<T, __half>::value) return __half22float2(*reinterpret_cast<const __half2*>(&w));
    else return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  };
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {
    const float2 f = pair(i);
    const float m = fmaxf(fabsf(f.x), fabsf(f.y));
    odd = odd || !(fabsf(f.x) < INFINITY) || !(fabsf(f.y) < INFINITY);
    amax = fmaxf(amax, m);
  }
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  odd = (__ballot_sync(0xffffffffu, odd) >> (threadIdx.x % 32 / 4 * 4)) & 0xfu;
  // 2^e <= amax < 2^(e+1): the row times 2^-e lies in [-2, 2]
  int e = (int)(__float_as_uint(amax) >> 23) - 127;
  e = max(e, -126);
  e = min(e, 126);
  const float down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    const float2 f0 = pair(2 * i), f1 = pair(2 * i + 1);
    lo[i] = h2bits(__floats2half2_rn(f0.x * down, f0.y * down));
    hi[i] = h2bits(__floats2half2_rn(f1.x * down, f1.y * down));
  }
  const float up = __uint_as_float((uint32_t)(127 + e) << 23);
  return odd ? __int_as_float(0x7fffffff) : up;           // a row that is not finite gives NaN
}

// A warp's blocks of the segment, up to 32 at a time: lane i holds the page
// and the scales of the i-th.
struct Window {
  int n;                                     // blocks
  int row;                                   // first row of the block's tile in the tensor maps
  int tok;                                   // first token of the block; past every length for a block left out
  float ks, vs;
};

__device__ __forceinline__ Window load_window(const AttnArgs& p, const Segment& s, int first, int len) {
  Window w;
  const int lane = threadIdx.x % 32;
  const int left = s.j1 - first;
  w.n = left > 0 ? min(32, (left + kWarps - 1) / kWarps) : 0;
  w.row = 0;
  w.tok = 1 << 30;
  w.ks = w.vs = 0.f;
  if (lane < w.n) {
    int j = first + lane * kWarps;
    bool ok = p.idx || len > 0;              // an empty sequence has one unit, and nothing in it
    if (p.idx) {
      const int32_t* list = p.idx + (((long long)s.b * p.Tq + s.t) * p.c.heads + s.h) * p.cap;
      const int before = j > 0 ? __ldg(list + j - 1) : -1;
      j = __ldg(list + j);
      ok = j > before && j >= 0 && j < p.c.max_blocks && (long long)j * kBlock < len;
    }
    int page = ok ? __ldg(p.c.table + (long long)s.b * p.c.max_blocks + j) : -1;
    ok = ok && (unsigned)page < (unsigned)p.c.n_pages;
    if (ok) {
      const long long cell = (long long)page * p.c.heads + s.h;
      w.row = (int)(cell * kBlock);
      w.tok = j * kBlock;
      w.ks = __ldg(p.c.k_scale + cell);
      w.vs = __ldg(p.c.v_scale + cell);
    } else if (p.idx || len > 0) {
      atomicOr(&g_cattn_flags, kFlagIndex);
    }
  }
  return w;
}

template <int D>
struct Smem {
  static constexpr int kTile = kBlock * D;
  static constexpr int kRingBytes = kWarps * kRing * kTile;
  static constexpr int kMergeBytes = kWarps / 2 * kRows * D * 4;
  static constexpr int kTotal = kRingBytes + kMergeBytes + 1024;     // + alignment of the swizzled tiles
};

template <int D, typename T, bool I8>
__global__ void __launch_bounds__(kThreads, 1)
cache_attn_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                  const __grid_constant__ AttnArgs p) {
  constexpr int NT = D / 8;                  // output tiles of 8 columns
  constexpr int KS = D / 16;                 // k steps of Q K^T
  constexpr int TILE = Smem<D>::kTile;
  extern __shared__ uint8_t dyn[];
  __shared__ __align__(8) uint64_t bars[kWarps * kRing];
  __shared__ long long red[kWarps];
  __shared__ float stat_m[kWarps][kRows], stat_l[kWarps][kRows];
  __shared__ Place place;
  __shared__ uint32_t abort_flag;

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, c = lane % 4;
  const uint32_t ring0 = (tc::su32(dyn) + 1023u) & ~1023u;
  float* merge = reinterpret_cast<float*>(dyn + (ring0 - tc::su32(dyn)) + Smem<D>::kRingBytes);
  const uint32_t ring = ring0 + warp * (kRing * TILE);
  const uint32_t bar = tc::su32(bars) + warp * (kRing * 8);
  if (threadIdx.x == 0) abort_flag = 0u;
  if (lane == 0) {
    for (int i = 0; i < kRing; ++i) tc::mbar_init(bar + 8 * i, 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }

  const long long per_seq = (long long)p.c.heads * p.tiles;
  const long long total = p.idx ? (long long)p.c.B * p.Tq * per_seq * p.cap : scan_sequences(p, red) * per_seq;
  const int ctas = active_ctas(total, p.grid);
  if ((int)blockIdx.x >= ctas) return;
  long long u = first_unit(total, ctas, blockIdx.x);
  const long long u_end = first_unit(total, ctas, blockIdx.x + 1);
  if (!p.idx && warp == 0) {
    int b;
    long long before;
    find_sequence(p, u, per_seq, &b, &before);
    if (lane == 0) {
      place.b = b;
      place.before = before;
    }
  }
  if (threadIdx.x == 0) {                    // lengths out of range are clamped, and recorded once
    for (int b = blockIdx.x; b < p.c.B; b += ctas) {
      const int n = __ldg(p.c.len + b);
      if (n < 0 || n > p.c.max_blocks * kBlock) atomicOr(&g_cattn_flags, kFlagIndex);
    }
  }
  __syncthreads();
  Place pl = place;
  volatile uint32_t* dead = &abort_flag;
  uint32_t issued = 0, used = 0;             // tiles of this warp's ring, K and V in turn
  bool alive = true;

  while (u < u_end) {
    // the segment
    Segment s;
    int units;
    item_of(p, pl, u, &s, &units);
    s.starts = s.j0 == 0;
    s.j1 = (int)min((long long)units, s.j0 + (u_end - u));
    s.ends = s.j1 == units;
    u += s.j1 - s.j0;
    const bool whole = s.starts && s.ends;
    if (!p.idx && s.ends && u - pl.before == (long long)units * per_seq) {      // the next sequence
      pl.before = u;
      pl.b += 1;
    }
    const int len = seq_len(p, s.b);
    if (p.idx) {
      const long long r = ((long long)s.b * p.Tq + s.t) * p.c.heads + s.h;
      int n = __ldg(p.cnt + r);
      if (n < 0 || n > p.cap) {
        if (threadIdx.x == 0) atomicOr(&g_cattn_flags, kFlagIndex);
        n = min(max(n, 0), p.cap);
      }
      s.j1 = min(s.j1, n);
    }

    // the query rows of this lane: g and g + 8
    uint32_t qf[KS][4];
    float fac[2];
    int lim[2];                               // keys the row sees
    {
      uint32_t lo[KS], hi[KS];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        int t, hg;
        const bool live = row_of(p, s, g + 8 * r, &t, &hg);
        const T* q = static_cast<const T*>(p.q) + (((long long)s.b * p.heads_q + s.h * p.group + hg) * p.Tq + t) * D;
        fac[r] = load_q<D, T>(q, live, c, lo, hi) * (1.44269504088896340736f / (D == 64 ? 8.f : 11.31370849898476039041f));
        lim[r] = live && p.causal ? max(len - p.Tq + 1 + t, 0) : len;      // (a row past the end counts for nothing)
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          qf[i][r] = lo[i];
          qf[i][r + 2] = hi[i];
        }
      }
    }
    int lim_min = min(lim[0], lim[1]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) lim_min = min(lim_min, __shfl_xor_sync(0xffffffffu, lim_min, o));

    float o[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    // windows of blocks: `cur` is consumed while loads may run into `nxt`
    int at = s.j0 + warp;
    Window cur = load_window(p, s, at, len);
    at += 32 * kWarps;
    Window nxt;
    nxt.n = 0;
    if (at < s.j1) nxt = load_window(p, s, at, len);
    at += 32 * kWarps;
    uint32_t fetched = 0;                     // tiles of `cur` (and on into `nxt`) asked for: K then V of each block

    auto fetch = [&]() {                      // one more tile, if there is one
      const int blk = (int)(fetched >> 1);
      const bool in_cur = blk < cur.n;
      if (!in_cur && blk - cur.n >= nxt.n) return;
      const int row = __shfl_sync(0xffffffffu, in_cur ? cur.row : nxt.row, in_cur ? blk : blk - cur.n);
      if (lane == 0 && alive) {
        const uint32_t slot = issued % kRing;
        tc::mbar_expect_tx(bar + 8 * slot, TILE);
        tc::tma_load_2d(ring + slot * TILE, (fetched & 1) ? &map_v : &map_k, 0, row, bar + 8 * slot);
      }
      ++issued;
      ++fetched;
    };
    auto arrived = [&]() -> uint32_t {        // the next tile in order
      const uint32_t slot = used % kRing, parity = (used / kRing) & 1u;
      if (alive) alive = tc::wait_bar(bar + 8 * slot, parity, dead, 95);
      alive = __all_sync(0xffffffffu, alive);
      ++used;
      return ring + slot * TILE;
    };
#pragma unroll
    for (int i = 0; i < kRing; ++i) fetch();

    while (cur.n > 0) {
      for (int i = 0; i < cur.n; ++i) {
        const float ks = __shfl_sync(0xffffffffu, cur.ks, i), vs = __shfl_sync(0xffffffffu, cur.vs, i);
        const int tok = __shfl_sync(0xffffffffu, cur.tok, i);

        // S = Q K^T: row g of the tile's n-tile nt is token 8 nt + g; a lane
        // reads the d / 4 codes that its fragments hold
        float sc[8][4];
        const uint32_t kt = arrived();
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) {
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[nt][e] = 0.f;
          uint32_t w[D / 16];
          if constexpr (D == 128) {
            const uint4 a = lds128(kt + nt * 1024 + g * 128 + (((2 * c) ^ g) << 4));
            const uint4 b = lds128(kt + nt * 1024 + g * 128 + (((2 * c + 1) ^ g) << 4));
            w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
            w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
          } else {
            const uint4 a = lds128(kt + nt * 512 + g * 64 + ((c ^ (g >> 1)) << 4));
            w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
          }
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            uint32_t f[2];
            Widen<I8>::word(w[k], f);
            mma16816(sc[nt], qf[k], f[0], f[1]);
          }
        }
        __syncwarp();
        fetch();                              // into the K tile's place

        // online softmax of the rows g and g + 8 (log2 units)
        const float f0 = fac[0] * ks, f1 = fac[1] * ks;
        float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) {
          sc[nt][0] *= f0;
          sc[nt][1] *= f0;
          sc[nt][2] *= f1;
          sc[nt][3] *= f1;
        }
        if (tok + kBlock > lim_min) {         // warp-uniform
#pragma unroll
          for (int nt = 0; nt < 8; ++nt) {
            const int t0 = tok + 8 * nt + 2 * c;
            if (t0 >= lim[0]) sc[nt][0] = -INFINITY;
            if (t0 + 1 >= lim[0]) sc[nt][1] = -INFINITY;
            if (t0 >= lim[1]) sc[nt][2] = -INFINITY;
            if (t0 + 1 >= lim[1]) sc[nt][3] = -INFINITY;
          }
        }
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) {
          mx0 = fmaxf(mx0, fmaxf(sc[nt][0], sc[nt][1]));
          mx1 = fmaxf(mx1, fmaxf(sc[nt][2], sc[nt][3]));
        }
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
        const float n0 = fmaxf(m[0], mx0), n1 = fmaxf(m[1], mx1);
        const float z0 = n0 == -INFINITY ? 0.f : n0, z1 = n1 == -INFINITY ? 0.f : n1;
        const float a0 = tc::ex2(m[0] - z0), a1 = tc::ex2(m[1] - z1);
        m[0] = n0;
        m[1] = n1;
        l[0] *= a0;
        l[1] *= a1;
        uint32_t pf[4][4];
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) {
          const float e0 = tc::ex2(sc[nt][0] - z0 + kShift), e1 = tc::ex2(sc[nt][1] - z0 + kShift);
          const float e2 = tc::ex2(sc[nt][2] - z1 + kShift), e3 = tc::ex2(sc[nt][3] - z1 + kShift);
          l[0] += e0 + e1;
          l[1] += e2 + e3;
          pf[nt / 2][nt % 2 * 2] = tc::pack_f16x2(e0, e1);
          pf[nt / 2][nt % 2 * 2 + 1] = tc::pack_f16x2(e2, e3);
        }

        // P V on the codes: n index j of tile nt is column (d / 8) j + nt, so a
        // lane reads d / 8 consecutive codes of its four tokens per step
        float pv[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) pv[n][e] = 0.f;
        const uint32_t vt = arrived();
        const bool edge = tok + kBlock > len;  // rows past the sequence hold anything: zero weights times NaN
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t w[4][D / 32];              // tokens 16 k + 2 c, + 1, + 8, + 9
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int row = 2 * c + (r & 1) + 8 * (r >> 1);
            if constexpr (D == 128) {
              const uint4 a = lds128(vt + k * 2048 + row * 128 + ((g ^ (row & 7)) << 4));
              w[r][0] = a.x; w[r][1] = a.y; w[r][2] = a.z; w[r][3] = a.w;
            } else {
              const uint2 a = lds64(vt + k * 1024 + row * 64 + (((g >> 1) ^ c) << 4) + (g & 1) * 8);
              w[r][0] = a.x; w[r][1] = a.y;
            }
            if (edge && tok + 16 * k + row >= len) {
#pragma unroll
              for (int i2 = 0; i2 < D / 32; ++i2) w[r][i2] = 0u;
            }
          }
#pragma unroll
          for (int i2 = 0; i2 < D / 32; ++i2) {
            // byte pairs (token, token + 1) of columns 4 i2 .. 4 i2 + 3
            uint32_t x[2], y[2], xh[2], yh[2];
            Widen<I8>::word(__byte_perm(w[0][i2], w[1][i2], 0x5140), x);
            Widen<I8>::word(__byte_perm(w[2][i2], w[3][i2], 0x5140), y);
            Widen<I8>::word(__byte_perm(w[0][i2], w[1][i2], 0x7362), xh);
            Widen<I8>::word(__byte_perm(w[2][i2], w[3][i2], 0x7362), yh);
            mma16816(pv[4 * i2], pf[k], x[0], y[0]);
            mma16816(pv[4 * i2 + 1], pf[k], x[1], y[1]);
            mma16816(pv[4 * i2 + 2], pf[k], xh[0], yh[0]);
            mma16816(pv[4 * i2 + 3], pf[k], xh[1], yh[1]);
          }
        }
        __syncwarp();
        fetch();                              // into the V tile's place
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          o[n][0] = o[n][0] * a0 + pv[n][0] * vs;
          o[n][1] = o[n][1] * a0 + pv[n][1] * vs;
          o[n][2] = o[n][2] * a1 + pv[n][2] * vs;
          o[n][3] = o[n][3] * a1 + pv[n][3] * vs;
        }
      }
      fetched -= 2u * (uint32_t)cur.n;
      cur = nxt;
      nxt.n = 0;
      if (at < s.j1) nxt = load_window(p, s, at, len);
      at += 32 * kWarps;
    }

    // join the warps: maxima first, then the sums, upper warps onto lower ones
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if (c == 0) {
        stat_m[warp][g + 8 * r] = m[r];
        stat_l[warp][g + 8 * r] = l[r];
      }
    }
    __syncthreads();
    float scale[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, stat_m[w][g + 8 * r]);
      scale[r] = top == -INFINITY ? 0.f : tc::ex2(m[r] - top);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      o[n][0] *= scale[0];
      o[n][1] *= scale[0];
      o[n][2] *= scale[1];
      o[n][3] *= scale[1];
    }
    if (warp >= kWarps / 2) {
      float* to = merge + (warp - kWarps / 2) * (kRows * D);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) to[(n * 4 + e) * 32 + lane] = o[n][e];
    }
    __syncthreads();
    if (warp < kWarps / 2) {
      float* to = merge + warp * (kRows * D);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) to[(n * 4 + e) * 32 + lane] += o[n][e];
    }
    __syncthreads();
    // warp w finishes element e = w / 2 of the tiles' lanes, half of the tiles
    {
      constexpr int H = NT / 2;
      const int e = warp / 2, half = warp % 2;
      const int row = g + 8 * (e >> 1), col = (D / 4) * c + (D / 8) * (e & 1) + H * half;
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, stat_m[w][row]);
      const float z = top == -INFINITY ? 0.f : top;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum += stat_l[w][row] * tc::ex2(stat_m[w][row] - z);
      float x[H];
#pragma unroll
      for (int n = 0; n < H; ++n) {
        x[n] = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps / 2; ++w) x[n] += merge[w * (kRows * D) + ((half * H + n) * 4 + e) * 32 + lane];
      }
      int t, hg;
      if (row_of(p, s, row, &t, &hg)) {
        if (whole) {
          const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);      // an empty row gives zeros, NaN stays
          const long long orow = ((long long)s.b * p.heads_q + s.h * p.group + hg) * p.Tq + t;
          uint32_t out[H / 2];
#pragma unroll
          for (int n = 0; n < H / 2; ++n) {
            if constexpr (std::is_same<T, __half>::value) out[n] = tc::pack_f16x2(x[2 * n] * inv, x[2 * n + 1] * inv);
            else out[n] = pack_bf16x2(x[2 * n] * inv, x[2 * n + 1] * inv);
          }
          T* dst = static_cast<T*>(p.o) + orow * D + col;
          if constexpr (H == 8) *reinterpret_cast<uint4*>(dst) = make_uint4(out[0], out[1], out[2], out[3]);
          else *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
          if (p.lse && col == 0) p.lse[orow] = (top + log2f(sum) - kShift) * 0.69314718055994530942f;
        } else {
          const long long slot = 2LL * blockIdx.x + (s.starts ? 1 : 0);
          float* dst = p.part + (slot * kRows + row) * D + col;
#pragma unroll
          for (int n = 0; n < H; n += 4) *reinterpret_cast<float4*>(dst + n) = make_float4(x[n], x[n + 1], x[n + 2], x[n + 3]);
          if (col == 0) {
            float* st = p.part + 2LL * p.grid * kRows * D + (slot * kRows + row) * 2;
            st[0] = top;
            st[1] = sum;
          }
        }
      }
    }
    __syncthreads();                           // the statistics and the merge area are free again
  }
}

// Joins the items that several CTAs shared: block (c, row) looks at the item
// that the start of CTA c + 1's share splits, if c holds its first unit.
template <int D, typename T>
__global__ void __launch_bounds__(128) cache_attn_join_kernel(const __grid_constant__ AttnArgs p) {
  constexpr int V = D / 4;                      // lanes of four columns
  constexpr int G = 128 / V;
  __shared__ long long red[4];
  __shared__ Place place;
  __shared__ float4 sums[G][V];
  __shared__ float rowsum[G];
  cudaGridDependencySynchronize();
  const long long per_seq = (long long)p.c.heads * p.tiles;
  const long long total = p.idx ? (long long)p.c.B * p.Tq * per_seq * p.cap : scan_sequences(p, red) * per_seq;
  const int ctas = active_ctas(total, p.grid);
  const int cta = blockIdx.x, row = blockIdx.y;
  if (cta + 1 >= ctas) return;
  const long long u = first_unit(total, ctas, cta + 1);
  Place pl{0, 0};
  if (!p.idx) {
    if (threadIdx.x < 32) {
      int b;
      long long before;
      find_sequence(p, u, per_seq, &b, &before);
      if (threadIdx.x == 0) {
        place.b = b;
        place.before = before;
      }
    }
    __syncthreads();
    pl = place;
  }
  Segment s;
  int units;
  item_of(p, pl, u, &s, &units);
  if (s.j0 == 0) return;                        // the share begins with an item
  const long long u0 = u - s.j0, u1 = u0 + units;
  if (cta_of(total, ctas, u0) != cta) return;   // an earlier CTA holds the item's first unit
  const int last = cta_of(total, ctas, u1 - 1);
  int t, hg;
  if (!row_of(p, s, row, &t, &hg)) return;

  const float* stats = p.part + 2LL * p.grid * kRows * D;
  auto slot_of = [&](int c) { return (2LL * c + (c == cta ? 1 : 0)) * kRows + row; };
  float top = -INFINITY;
  for (int c = cta; c <= last; ++c) top = fmaxf(top, __ldcg(stats + 2 * slot_of(c)));
  const float z = top == -INFINITY ? 0.f : top;
  const int v = threadIdx.x % V, g = threadIdx.x / V;
  float sum = 0.f;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c = cta + g; c <= last; c += G) {
    const long long k = slot_of(c);
    const float w = tc::ex2(__ldcg(stats + 2 * k) - z);
    sum += w * __ldcg(stats + 2 * k + 1);
    const float4 a = __ldcg(reinterpret_cast<const float4*>(p.part + k * D) + v);
    x.x += w * a.x;
    x.y += w * a.y;
    x.z += w * a.z;
    x.w += w * a.w;
  }
  sums[g][v] = x;
  if (v == 0) rowsum[g] = sum;
  __syncthreads();
  if (g != 0) return;
  x = make_float4(0.f, 0.f, 0.f, 0.f);
  sum = 0.f;
#pragma unroll
  for (int i = 0; i < G; ++i) {
    x.x += sums[i][v].x;
    x.y += sums[i][v].y;
    x.z += sums[i][v].z;
    x.w += sums[i][v].w;
    sum += rowsum[i];
  }
  const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
  const long long orow = ((long long)s.b * p.heads_q + s.h * p.group + hg) * p.Tq + t;
  uint2 out;
  if constexpr (std::is_same<T, __half>::value)
    out = make_uint2(tc::pack_f16x2(x.x * inv, x.y * inv), tc::pack_f16x2(x.z * inv, x.w * inv));
  else
    out = make_uint2(pack_bf16x2(x.x * inv, x.y * inv), pack_bf16x2(x.z * inv, x.w * inv));
  *reinterpret_cast<uint2*>(static_cast<T*>(p.o) + orow * D + 4 * v) = out;
  if (p.lse && v == 0) p.lse[orow] = (top + log2f(sum) - kShift) * 0.69314718055994530942f;
}

// Byte view of the codes, [rows, d]: boxes of one block, swizzled over the row.
bool map_codes(CUtensorMap* m, const void* base, long long rows, int d) {
  tc::EncodeTiledFn enc = tc::encode_fn();
  if (enc == nullptr) return false;
  cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)d};
  cuuint32_t box[2] = {(cuuint32_t)d, (cuuint32_t)kBlock};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, typename T, bool I8>
cudaError_t run(const CUtensorMap& mk, const CUtensorMap& mv, const AttnArgs& p, cudaStream_t st) {
  auto kernel = cache_attn_kernel<D, T, I8>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::kTotal);
  if (e != cudaSuccess) return e;
  kernel<<<p.grid, kThreads, Smem<D>::kTotal, st>>>(mk, mv, p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)p.grid, kRows);
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_attn_join_kernel<D, T>, p);
}

}  // namespace

size_t cache_attn_workspace_bytes(int d) { return (size_t)kNumSMs * 2 * kRows * (d + 2) * sizeof(float); }

cudaError_t launch_cache_attn(const CacheArgs& c, const void* q, int heads_q, int Tq, int f16, int causal,
                              const int32_t* idx, const int32_t* cnt, int cap, void* o, float* lse, void* ws,
                              cudaStream_t st) {
  AttnArgs p{};
  p.c = c;
  p.q = q;
  p.idx = idx;
  p.cnt = cnt;
  p.o = o;
  p.lse = lse;
  p.part = static_cast<float*>(ws);
  p.heads_q = heads_q;
  p.Tq = Tq;
  p.causal = causal;
  p.cap = cap;
  p.group = heads_q / c.heads;
  p.tiles = ceil_div(idx ? p.group : (long long)p.group * Tq, kRows);
  p.grid = kNumSMs;
  CUtensorMap mk, mv;
  const long long rows = (long long)c.n_pages * c.heads * kBlock;
  if (!map_codes(&mk, c.k, rows, c.d) || !map_codes(&mv, c.v, rows, c.d)) return cudaErrorInvalidValue;
  cudaError_t e = cudaSuccess;
  auto t = [&](auto D_) {
    auto u = [&](auto z) {
      constexpr int D = decltype(D_)::value;
      using T = decltype(z);
      e = c.i8 ? run<D, T, true>(mk, mv, p, st) : run<D, T, false>(mk, mv, p, st);
    };
    if (f16) u(__half{});
    else u(__nv_bfloat16{});
  };
  if (c.d == 128) t(std::integral_constant<int, 128>{});
  else t(std::integral_constant<int, 64>{});
  return e;
}

cudaError_t cattn_flags(unsigned int* v, cudaStream_t st) { return read_and_clear_flags(g_cattn_flags, v, st); }
cudaError_t cattn_error(unsigned int* code, cudaStream_t st) { return tc::read_error(code, st); }

}  // namespace svsa
