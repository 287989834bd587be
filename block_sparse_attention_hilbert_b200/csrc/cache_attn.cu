// Attention of a few query tokens over the 8-bit block cache, whole or through
// per-query block lists.
//
//   o = sum_t softmax_t(q . k_t / sqrt(d)) v_t,  k_t = ks[block] * code,  v_t = vs[block] * code
//
// Bound by HBM: 2 d bytes per token and key head, against 4 d FLOP per query
// row of the group that shares the head.  The products run transposed on
// mma.sync.m16n8k16, tokens (or output columns) along M and the query rows
// along N, eight at a time: S^T = K Q^T, O^T = V^T P^T.  A tcgen05 tile has 64
// rows at least and takes its operands from shared memory, so the codes would
// have to be widened there and read back, for rows that are mostly empty; here
// they go from shared memory to registers and are widened on the way (8-bit to
// fp16 is exact, fp16 x fp16 products are exact in fp32), and up to eight
// query rows cost half of what a tile of 16 query rows would.
//
// More than 32 (d = 64: 48) query rows per key head, and in large caches more
// than 16 (see tile_rows), take the 128-row tcgen05 tiles of
// cache_attn_rows.cuh instead, over the same items and shares.  So do lists of
// many queries, gathered per tile (see gather_plan).
//
// Work: an item is (sequence, key head, tile of 8 or 16 rows), or with lists
// (sequence, query, key head, tile of the group's rows); a unit is one
// 64-token block of an item.  The CTAs, one per SM, take equal contiguous
// shares of all units, so ragged lengths balance; an item that several CTAs
// share is joined by a second kernel from fp32 partial sums with their maxima,
// in CTA order.  Where items are short, or so many that whole ones balance,
// each goes to one CTA and there is no second kernel.  In a CTA, twelve warps
// (eight with 16 rows) take the blocks of a segment in turn, each with a ring
// of its own of tiles filled by TMA (swizzled over the row, so that both the
// row-wise reads of K and the column-wise reads of V are free of bank
// conflicts), and no barrier until the segment's end.
//
// Rounding: q is scaled per row by a power of two into fp16 (exact for bf16
// values within 2^-14 of the row's largest; below that they keep 2^-24 of it);
// softmax weights are rounded to fp16, taken times 2^14 so that weights down
// to 2^-38 of the row's largest keep a value; a block's P V sum is taken on
// the codes alone and joins the fp32 accumulator times the block's scale, so
// scales of any size mix.  Maxima, sums and accumulators are fp32.
#include <cuda_fp8.h>

#include <type_traits>

#include "common.cuh"
#include "stream.cuh"
#include "tcgen05.cuh"

namespace svsa {

static __device__ unsigned int g_cattn_flags;

namespace {

constexpr int kTileRows = 128;              // of the many-row tiles
constexpr float kShift = 14.f;              // weights are held times 2^kShift
constexpr int kMinUnits = 8;                // blocks of a CTA at least, where there are as many

struct AttnArgs {
  CacheArgs c;
  const void* q;                            // [B][heads_q][Tq][d]
  const int32_t* idx;                       // nullable: [B][Tq][heads][cap]
  const int32_t* cnt;
  void* o;                                  // [B][heads_q][Tq][d]
  float* lse;                               // nullable [B][heads_q][Tq]
  float* part;                              // [CTA][2][rows][d] sums, then [CTA][2][rows][2] maxima and row sums
  int heads_q, Tq, causal, cap, group, tiles, grid;
  int whole;                                // every item goes to one CTA as a whole
  // lists gathered per 128-row tile (idx is null then): per item, the blocks
  // that any of its queries lists, and a bit per query and block
  const int32_t* ucnt;                      // [items]
  const int32_t* ulist;                     // [items][max_blocks]
  const uint32_t* ubits;                    // [items][tile_queries][words]
  int tile_queries, words;
};

// A contiguous range of an item's blocks.
struct Segment {
  int b, t, h, tile;                        // t: the query (lists) or -1
  int j0, j1;                               // blocks, or list positions
};

__device__ __forceinline__ int seq_len(const AttnArgs& p, int b) {
  const int n = __ldg(p.c.len + b);
  return min(max(n, 0), p.c.max_blocks * kBlock);
}
__device__ __forceinline__ int blocks_of(int len) { return max(1, (len + kBlock - 1) / kBlock); }

// What the CTAs share out (counts fit 32 bits, checked on the host): blocks, or
// whole items.  With lists every item counts `cap` blocks, the entries past its
// own count being empty; with gathered lists max(1, its union's blocks);
// without, the items of sequence b have max(1, blocks of b) each.
struct Shares {
  unsigned total, base, rem;
  int ctas;
  __device__ void split(unsigned units, int grid, int least) {
    total = units;
    const unsigned want = (units + least - 1) / least;
    ctas = want < (unsigned)grid ? (int)want : grid;
    base = units / ctas;
    rem = units - base * ctas;                // the first `rem` CTAs take one more
  }
  __device__ unsigned first(int c) const { return base * c + min((unsigned)c, rem); }
  __device__ int of(unsigned u) const {
    const unsigned cut = rem * (base + 1);
    return (int)(u < cut ? u / (base + 1) : rem + (u - cut) / base);
  }
};

// A warp calls; every lane gets the result.
__device__ Shares shares_of(const AttnArgs& p) {
  Shares s;
  const unsigned items = (unsigned)p.c.heads * p.tiles;
  if (p.whole) {
    s.split((unsigned)p.c.B * (p.idx ? p.Tq : 1) * items, p.grid, 1);
  } else if (p.idx) {
    s.split((unsigned)p.c.B * p.Tq * items * p.cap, p.grid, kMinUnits);
  } else if (p.ucnt) {
    unsigned n = 0;
    for (unsigned i = threadIdx.x % 32; i < (unsigned)p.c.B * items; i += 32) n += max(1, __ldg(p.ucnt + i));
    s.split(__reduce_add_sync(0xffffffffu, n), p.grid, kMinUnits);
  } else {
    unsigned n = 0;
    for (int b = threadIdx.x % 32; b < p.c.B; b += 32) n += blocks_of(seq_len(p, b));
    s.split(__reduce_add_sync(0xffffffffu, n) * items, p.grid, kMinUnits);
  }
  return s;
}

// The item at unit u: its sequence, head and tile, u's place in it (j0) and
// its number of units.  `b` and `before` say which sequence (with gathered
// lists: which item) u lies in and how many units lie before that (neither
// with whole items nor with lists).
__device__ __forceinline__ void item_of(const AttnArgs& p, unsigned u, int b, unsigned before, Segment* s, int* units) {
  unsigned item;
  if (p.whole) {
    item = u;
    s->j0 = 0;
    *units = 1;
  } else if (p.ucnt) {
    item = (unsigned)b;
    s->j0 = (int)(u - before);
    *units = max(1, __ldg(p.ucnt + b));
  } else {
    const unsigned n = p.idx ? p.cap : blocks_of(seq_len(p, b));
    item = (u - before) / n;
    s->j0 = (int)(u - before - item * n);
    *units = (int)n;
  }
  s->t = -1;
  s->tile = (int)(item % p.tiles);
  item /= p.tiles;
  if (p.whole || p.idx || p.ucnt) {
    s->h = (int)(item % p.c.heads);
    item /= p.c.heads;
    if (p.idx) {
      s->t = (int)(item % p.Tq);
      item /= p.Tq;
    }
    s->b = (int)item;
  } else {
    s->h = (int)item;
    s->b = b;
  }
}

// The sequence (with gathered lists: the item) of unit u.  A warp calls; 32 a step.
__device__ void find_sequence(const AttnArgs& p, unsigned u, int* b_out, unsigned* before_out) {
  const int lane = threadIdx.x % 32;
  const unsigned items = (unsigned)p.c.heads * p.tiles;
  const int n = p.ucnt ? p.c.B * (int)items : p.c.B;
  unsigned before = 0;
  for (int b0 = 0; b0 < n; b0 += 32) {
    const int b = b0 + lane;
    const unsigned mine = b >= n ? 0u : p.ucnt ? (unsigned)max(1, __ldg(p.ucnt + b)) : blocks_of(seq_len(p, b)) * items;
    unsigned up = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned v = __shfl_up_sync(0xffffffffu, up, o);
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
  *b_out = 0;                                // (u lies below the total, so this is not reached)
  *before_out = 0;
}

// Row r of a tile of ROWS: its query and its head in the group; false past the end.
template <int ROWS>
__device__ __forceinline__ bool row_of(const AttnArgs& p, const Segment& s, int r, int* t, int* g) {
  const int i = s.tile * ROWS + r;
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

// The four codes of a word as two pairs of fp16, exactly.
template <bool I8>
struct Widen;
template <>
struct Widen<false> {
  __device__ static void word(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
        : "=r"(lo), "=r"(hi) : "r"(w));
  }
};
template <>
struct Widen<true> {
  // 0x6400 | (code + 128) is 1024 + code + 128 in fp16
  __device__ static void word(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = w ^ 0x80808080u;
    const __half2 off = __floats2half2_rn(1152.f, 1152.f);
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    lo = h2bits(__hsub2(*reinterpret_cast<__half2*>(&a), off));
    hi = h2bits(__hsub2(*reinterpret_cast<__half2*>(&b), off));
  }
};

// d (16 x 8) += a (16 x 16) b (16 x 8), or d = a b.
__device__ __forceinline__ void mma(float d[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_first(float d[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// An 8 x 8 matrix of 16-bit values (row g of lane 4 g + c: columns 2 c, 2 c + 1), transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
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

// Query fragments of one row.  The products sum over d in any order, so the k
// index of the MMA is laid over d as the reads of K want it: lane c of a quad
// owns the d / 4 consecutive values from c * d / 4 on, four per step.  Returns
// the power of two that the row was divided by.  A row that is not finite is
// NaN throughout: so are its scores, but not the masked ones, and a row that
// sees nothing stays a row that sees nothing.
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
    odd = odd || !(fabsf(f.x) < INFINITY) || !(fabsf(f.y) < INFINITY);
    amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
  }
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  odd = (__ballot_sync(0xffffffffu, odd) >> (threadIdx.x % 32 / 4 * 4)) & 0xfu;
  // 2^e <= amax < 2^(e+1): the row times 2^-e lies in [-2, 2]
  int e = (int)(__float_as_uint(amax) >> 23) - 127;
  e = min(max(e, -126), 126);
  const float down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    const float2 f0 = pair(2 * i), f1 = pair(2 * i + 1);
    lo[i] = odd ? 0x7fff7fffu : h2bits(__floats2half2_rn(f0.x * down, f0.y * down));
    hi[i] = odd ? 0x7fff7fffu : h2bits(__floats2half2_rn(f1.x * down, f1.y * down));
  }
  return __uint_as_float((uint32_t)(127 + e) << 23);
}

// A warp's blocks of the segment, up to 32 at a time: lane i holds the page
// and the scales of the i-th.
struct Window {
  int n;                                     // blocks
  int row;                                   // first row of the block's tile in the tensor maps
  int tok;                                   // first token of the block; past every length for a block left out
  float ks, vs;
};

// With lists, the entry of this lane and the one before it are read ahead of
// what bounds them (`j0 + lane * WARPS < j1` and j1 within the list's capacity).
struct Entry {
  int j, before;
};
template <int WARPS>
__device__ __forceinline__ Entry load_entry(const AttnArgs& p, const Segment& s, int first, int j1) {
  Entry e{first + (int)(threadIdx.x % 32) * WARPS, -1};
  if (p.idx && e.j < j1) {
    const int32_t* list = p.idx + (((long long)s.b * p.Tq + s.t) * p.c.heads + s.h) * p.cap + e.j;
    e.before = e.j > 0 ? __ldg(list - 1) : -1;
    e.j = __ldg(list);
  }
  return e;
}

template <int WARPS>
__device__ __forceinline__ Window load_window(const AttnArgs& p, const Segment& s, int first, int len, Entry e) {
  Window w;
  const int lane = threadIdx.x % 32;
  const int left = s.j1 - first;
  w.n = left > 0 ? min(32, (left + WARPS - 1) / WARPS) : 0;
  w.row = 0;
  w.tok = 1 << 30;
  w.ks = w.vs = 0.f;
  if (lane < w.n) {
    // (an empty sequence has one unit, and nothing in it)
    bool ok = p.idx ? e.j > e.before && e.j >= 0 && e.j < p.c.max_blocks && (long long)e.j * kBlock < len : len > 0;
    const int page = ok ? __ldg(p.c.table + (long long)s.b * p.c.max_blocks + e.j) : -1;
    ok = ok && (unsigned)page < (unsigned)p.c.n_pages;
    if (ok) {
      const long long cell = (long long)page * p.c.heads + s.h;
      w.row = (int)(cell * kBlock);
      w.tok = e.j * kBlock;
      w.ks = __ldg(p.c.k_scale + cell);
      w.vs = __ldg(p.c.v_scale + cell);
    } else if (p.idx || len > 0) {
      atomicOr(&g_cattn_flags, kFlagIndex);
    }
  }
  return w;
}

// Shape of a CTA.  A warp's ring holds its tiles in flight; when a segment is
// done it holds the warp's sums, to be joined.
template <int D, int NR>
struct Cta {
  static constexpr int kWarps = NR == 1 ? 12 : 8;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kTile = kBlock * D;
  static constexpr int kRing = (NR == 1 ? 2 : 3) * (128 / D);        // tiles in flight per warp
  static constexpr int kRows = 8 * NR;
  static constexpr int kPitch = D + 4;                               // floats of a row of sums
  static constexpr int kSmem = kWarps * kRing * kTile + 1024;        // + alignment of the tiles
  static_assert(kRows * kPitch * 4 <= kRing * kTile, "the sums fit the ring");
};

// After a wait that gave up: the warp's copies in flight (tiles used ..
// issued - 1), each waited for with a limit of its own, before the ring holds
// anything else or the CTA goes.
__device__ __noinline__ void wait_in_flight(uint32_t bar, uint32_t ring, uint32_t used, uint32_t issued) {
  for (uint32_t x = used; x < issued; ++x) {
    volatile uint32_t no_abort = 0u;
    tc::wait_bar(bar + 8 * (x % ring), (x / ring) & 1u, &no_abort, 96);
  }
}

// A finished row's four columns from col on, or the CTA's share of them.
template <int D, typename T>
__device__ __forceinline__ void write_out(const AttnArgs& p, const Segment& s, int t, int hg, int col, float4 x, float top,
                                          float sum) {
  const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);      // an empty row gives zeros, NaN stays
  const long long row = ((long long)s.b * p.heads_q + s.h * p.group + hg) * p.Tq + t;
  uint2 out;
  if constexpr (std::is_same<T, __half>::value)
    out = make_uint2(tc::pack_f16x2(x.x * inv, x.y * inv), tc::pack_f16x2(x.z * inv, x.w * inv));
  else
    out = make_uint2(pack_bf16x2(x.x * inv, x.y * inv), pack_bf16x2(x.z * inv, x.w * inv));
  *reinterpret_cast<uint2*>(static_cast<T*>(p.o) + row * D + col) = out;
  if (p.lse && col == 0) p.lse[row] = (top + log2f(sum) - kShift) * 0.69314718055994530942f;
}

template <int D, typename T, bool I8, int NR>
__global__ void __launch_bounds__(Cta<D, NR>::kThreads, 1)
cache_attn_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                  const __grid_constant__ AttnArgs p) {
  using S = Cta<D, NR>;
  constexpr int ROWS = S::kRows, RING = S::kRing, TILE = S::kTile, kWarps = S::kWarps, kThreads = S::kThreads;
  constexpr int MT = D / 16;                 // output tiles of 16 columns; also the k steps of K Q^T
  extern __shared__ uint8_t dyn[];
  __shared__ __align__(8) uint64_t bars[kWarps * RING];
  __shared__ float stat_m[kWarps][ROWS], stat_l[kWarps][ROWS];
  __shared__ uint32_t abort_flag;

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, c = lane % 4;
  const uint32_t ring0 = (tc::su32(dyn) + 1023u) & ~1023u;
  float* const sums = reinterpret_cast<float*>(dyn + (ring0 - tc::su32(dyn)));
  constexpr int SUMS = RING * TILE / 4;      // floats between two warps' rings
  const uint32_t ring = ring0 + warp * (RING * TILE);
  const uint32_t bar = tc::su32(bars) + warp * (RING * 8);
  cudaTriggerProgrammaticLaunchCompletion();  // the joining kernel may take its places; it waits for this one's end
  const Shares sh = shares_of(p);
  if ((int)blockIdx.x >= sh.ctas) return;
  if (threadIdx.x == 0) {
    abort_flag = 0u;
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&map_k)) : "memory");
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&map_v)) : "memory");
  }
  if (lane == 0) {
    for (int i = 0; i < RING; ++i) tc::mbar_init(bar + 8 * i, 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  unsigned u = sh.first(blockIdx.x);
  const unsigned u_end = sh.first(blockIdx.x + 1);
  int seq = 0;
  unsigned before = 0;
  if (!p.idx && !p.whole) find_sequence(p, u, &seq, &before);
  if (threadIdx.x == 0) {                    // lengths out of range are clamped, and recorded
    for (int b = blockIdx.x; b < p.c.B; b += sh.ctas) {
      const int n = __ldg(p.c.len + b);
      if (n < 0 || n > p.c.max_blocks * kBlock) atomicOr(&g_cattn_flags, kFlagIndex);
    }
  }
  __syncthreads();
  volatile uint32_t* dead = &abort_flag;
  uint32_t issued = 0, used = 0;             // tiles of this warp's ring, K and V in turn
  bool alive = true;

  while (u < u_end) {
    Segment s;
    int units;
    item_of(p, u, seq, before, &s, &units);
    const bool starts = s.j0 == 0;
    s.j1 = (int)min((unsigned)units, s.j0 + (u_end - u));
    const bool whole = starts && s.j1 == units;
    u += s.j1 - s.j0;
    if (!p.idx && !p.whole && u - before == (unsigned)units * p.c.heads * p.tiles) {      // the next sequence
      before = u;
      seq += 1;
    }
    if (p.whole && p.idx) s.j1 = p.cap;
    const Entry ahead = load_entry<kWarps>(p, s, s.j0 + warp, s.j1);
    int n = p.idx ? __ldg(p.cnt + ((long long)s.b * p.Tq + s.t) * p.c.heads + s.h) : 0;
    const int len = seq_len(p, s.b);
    if (p.whole && !p.idx) s.j1 = blocks_of(len);
    if (p.idx) {
      if (n < 0 || n > p.cap) {
        if (threadIdx.x == 0) atomicOr(&g_cattn_flags, kFlagIndex);
        n = min(max(n, 0), p.cap);
      }
      s.j1 = min(s.j1, n);
    }

    // windows of blocks: `cur` is consumed while loads may run into `nxt`
    int at = s.j0 + warp;
    Window cur = load_window<kWarps>(p, s, at, len, ahead);
    at += 32 * kWarps;
    Window nxt;
    nxt.n = 0;
    if (at < s.j1) nxt = load_window<kWarps>(p, s, at, len, load_entry<kWarps>(p, s, at, s.j1));
    at += 32 * kWarps;
    uint32_t fetched = 0;                     // tiles of `cur` (and on into `nxt`) asked for: K then V of each block
    auto fetch = [&]() {                      // one more tile, if there is one
      const int blk = (int)(fetched >> 1);
      const bool in_cur = blk < cur.n;
      if (!in_cur && blk - cur.n >= nxt.n) return;
      const int row = __shfl_sync(0xffffffffu, in_cur ? cur.row : nxt.row, in_cur ? blk : blk - cur.n);
      if (lane == 0 && alive) {
        const uint32_t slot = issued % RING;
        tc::mbar_expect_tx(bar + 8 * slot, TILE);
        tc::tma_load_2d(ring + slot * TILE, (fetched & 1) ? &map_v : &map_k, 0, row, bar + 8 * slot);
      }
      ++issued;
      ++fetched;
    };
    auto arrived = [&]() -> uint32_t {        // the next tile in order
      const uint32_t slot = used % RING, parity = (used / RING) & 1u;
      if (alive) {
        alive = __all_sync(0xffffffffu, tc::wait_bar(bar + 8 * slot, parity, dead, 95));
        if (!alive) wait_in_flight(bar, RING, used, issued);
      }
      ++used;
      return ring + slot * TILE;
    };
#pragma unroll
    for (int i = 0; i < RING; ++i) fetch();

    // query row 8 r + g is this lane's fragment; the scores' columns are rows 8 r + 2 c and + 1
    uint32_t qf[NR][MT][2];
    float fac[NR][2];
    int lim[NR][2];                           // keys the row sees
    int lim_min = len;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      uint32_t lo[MT], hi[MT];
      int t, hg;
      const bool live = row_of<ROWS>(p, s, 8 * r + g, &t, &hg);
      const T* q = static_cast<const T*>(p.q) + (((long long)s.b * p.heads_q + s.h * p.group + hg) * p.Tq + t) * D;
      const float f = load_q<D, T>(q, live, c, lo, hi) * (1.44269504088896340736f / (D == 64 ? 8.f : 11.31370849898476039041f));
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        qf[r][i][0] = lo[i];
        qf[r][i][1] = hi[i];
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        fac[r][e] = __shfl_sync(0xffffffffu, f, 4 * (2 * c + e));
        const bool there = row_of<ROWS>(p, s, 8 * r + 2 * c + e, &t, &hg);
        lim[r][e] = there && p.causal ? max(len - p.Tq + 1 + t, 0) : len;      // (a row past the end counts for nothing)
        lim_min = min(lim_min, lim[r][e]);
      }
    }
    lim_min = __reduce_min_sync(0xffffffffu, lim_min);

    F2 o[MT][NR][2];                          // O^T: column g (+ 8) of tile mt, rows 2 c and 2 c + 1
    float m[NR][2];
    F2 l[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      m[r][0] = m[r][1] = -INFINITY;
      l[r] = f2(0.f, 0.f);
#pragma unroll
      for (int n = 0; n < MT; ++n) o[n][r][0] = o[n][r][1] = f2(0.f, 0.f);
    }

    while (cur.n > 0) {
      for (int i = 0; i < cur.n; ++i) {
        const float ks = __shfl_sync(0xffffffffu, cur.ks, i), vs = __shfl_sync(0xffffffffu, cur.vs, i);
        const int tok = __shfl_sync(0xffffffffu, cur.tok, i);

        // S^T = K Q^T: tokens 16 mt + g and + 8 are rows of tile mt; a lane
        // reads the d / 4 codes of each that its fragments hold
        float sc[4][NR][4];
        const uint32_t kt = arrived();
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
          uint32_t w[2][MT];
#pragma unroll
          for (int h8 = 0; h8 < 2; ++h8) {
            if constexpr (D == 128) {
              const uint32_t row = kt + (2 * mt + h8) * 1024 + g * 128;
              const uint4 a = lds128(row + (((2 * c) ^ g) << 4)), b = lds128(row + (((2 * c + 1) ^ g) << 4));
              w[h8][0] = a.x; w[h8][1] = a.y; w[h8][2] = a.z; w[h8][3] = a.w;
              w[h8][4] = b.x; w[h8][5] = b.y; w[h8][6] = b.z; w[h8][7] = b.w;
            } else {
              const uint4 a = lds128(kt + (2 * mt + h8) * 512 + g * 64 + ((c ^ (g >> 1)) << 4));
              w[h8][0] = a.x; w[h8][1] = a.y; w[h8][2] = a.z; w[h8][3] = a.w;
            }
          }
#pragma unroll
          for (int k = 0; k < MT; ++k) {
            uint32_t a[4];
            Widen<I8>::word(w[0][k], a[0], a[2]);
            Widen<I8>::word(w[1][k], a[1], a[3]);
#pragma unroll
            for (int r = 0; r < NR; ++r) {
              if (k == 0) mma_first(sc[mt][r], a, qf[r][k][0], qf[r][k][1]);
              else mma(sc[mt][r], a, qf[r][k][0], qf[r][k][1]);
            }
          }
        }
        __syncwarp();
        fetch();                              // into the K tile's place

        // online softmax of the rows 2 c and 2 c + 1 (log2 units): the scale joins
        // in the exponent, p = 2^(s f - m + 14)
        if (tok + kBlock > lim_min) {         // warp-uniform
#pragma unroll
          for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
              for (int mt = 0; mt < 4; ++mt)
                if (tok + 16 * mt + g + 8 * (e >> 1) >= lim[r][e & 1]) sc[mt][r][e] = -INFINITY;
        }
        uint32_t pf[4][NR][2];
        F2 al[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          float z[2], f[2], a[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            f[e] = fac[r][e] * ks;
            if (f[e] == 0.f) f[e] = 1.17549435e-38f;      // keeps -inf apart from 0 * -inf
            float mx = tc::max3(sc[0][r][e], sc[0][r][e + 2], sc[1][r][e]);
            mx = tc::max3(mx, sc[1][r][e + 2], sc[2][r][e]);
            mx = tc::max3(mx, sc[2][r][e + 2], sc[3][r][e]);
            mx = fmaxf(mx, sc[3][r][e + 2]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float n = fmaxf(m[r][e], mx * f[e]);
            z[e] = n == -INFINITY ? 0.f : n;
            a[e] = tc::ex2(m[r][e] - z[e]);
            m[r][e] = n;
          }
          al[r] = f2(a[0], a[1]);
          const F2 ff = f2(f[0], f[1]), zz = f2(kShift - z[0], kShift - z[1]);
          l[r] = mul2(l[r], al[r]);
#pragma unroll
          for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int h8 = 0; h8 < 2; ++h8) {
              float e0, e1;
              split2(fma2(f2(sc[mt][r][2 * h8], sc[mt][r][2 * h8 + 1]), ff, zz), e0, e1);
              e0 = tc::ex2(e0);
              e1 = tc::ex2(e1);
              l[r] = add2(l[r], f2(e0, e1));
              pf[mt][r][h8] = transpose8(tc::pack_f16x2(e0, e1));
            }
        }

        // O^T += vs V^T P^T on the codes: rows g and g + 8 of tile mt are
        // columns (d / 8) g + 2 mt and + 1, so a lane reads d / 8 consecutive
        // codes of its four tokens per step
        float pv[MT][NR][4];
        const uint32_t vt = arrived();
        if (tok + kBlock > len) {              // rows past the sequence hold anything (zero weights times NaN): clear them
          for (int x = max(len - tok, 0) * (D / 16) + lane; x < kBlock * (D / 16); x += 32)
            tc::st_shared_v4(vt + 16 * x, 0u, 0u, 0u, 0u);      // (the swizzle keeps a 16-byte piece in its row)
          __syncwarp();
        }
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
          }
#pragma unroll
          for (int i2 = 0; i2 < D / 32; ++i2) {
            // byte pairs (token, token + 1) of columns 4 i2 .. 4 i2 + 3
            uint32_t a[4], b[4];
            Widen<I8>::word(__byte_perm(w[0][i2], w[1][i2], 0x5140), a[0], a[1]);
            Widen<I8>::word(__byte_perm(w[2][i2], w[3][i2], 0x5140), a[2], a[3]);
            Widen<I8>::word(__byte_perm(w[0][i2], w[1][i2], 0x7362), b[0], b[1]);
            Widen<I8>::word(__byte_perm(w[2][i2], w[3][i2], 0x7362), b[2], b[3]);
#pragma unroll
            for (int r = 0; r < NR; ++r) {
              if (k == 0) {
                mma_first(pv[2 * i2][r], a, pf[k][r][0], pf[k][r][1]);
                mma_first(pv[2 * i2 + 1][r], b, pf[k][r][0], pf[k][r][1]);
              } else {
                mma(pv[2 * i2][r], a, pf[k][r][0], pf[k][r][1]);
                mma(pv[2 * i2 + 1][r], b, pf[k][r][0], pf[k][r][1]);
              }
            }
          }
        }
        if (tok + kBlock > len) tc::fence_async_smem();        // (the clearing above, before the next tile arrives)
        __syncwarp();
        fetch();                              // into the V tile's place
        const F2 vv = f2(vs, vs);
#pragma unroll
        for (int n = 0; n < MT; ++n)
#pragma unroll
          for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int h8 = 0; h8 < 2; ++h8)
              o[n][r][h8] = fma2(f2(pv[n][r][2 * h8], pv[n][r][2 * h8 + 1]), vv, mul2(o[n][r][h8], al[r]));
      }
      fetched -= 2u * (uint32_t)cur.n;
      cur = nxt;
      nxt.n = 0;
      if (at < s.j1) nxt = load_window<kWarps>(p, s, at, len, load_entry<kWarps>(p, s, at, s.j1));
      at += 32 * kWarps;
    }

    // join the warps: maxima and row sums, then each warp's sums under the common maximum
    // (every tile that this warp asked for has been read, so its ring is free)
    const int rows = min(ROWS, (s.t >= 0 ? p.group : p.group * p.Tq) - s.tile * ROWS);
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      float v[2];
      split2(l[r], v[0], v[1]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        v[e] += __shfl_xor_sync(0xffffffffu, v[e], 4);
        v[e] += __shfl_xor_sync(0xffffffffu, v[e], 8);
        v[e] += __shfl_xor_sync(0xffffffffu, v[e], 16);
        const int row = 8 * r + 2 * c + e;
        if (g == 0) {
          stat_m[warp][row] = m[r][e];
          stat_l[warp][row] = v[e];
        }
        if (row < rows) {
          float* to = sums + warp * SUMS + row * S::kPitch + g * (D / 8);
#pragma unroll
          for (int n = 0; n < MT; n += 2) {
            float x[4][2];
#pragma unroll
            for (int i = 0; i < 4; ++i) split2(o[n + i / 2][r][i % 2], x[i][0], x[i][1]);
            *reinterpret_cast<float4*>(to + 2 * n) = make_float4(x[0][e], x[1][e], x[2][e], x[3][e]);
          }
        }
      }
    }
    __syncthreads();
    for (int x = threadIdx.x; x < rows * (D / 4); x += kThreads) {
      const int row = x / (D / 4), col = x % (D / 4) * 4;
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, stat_m[w][row]);
      const float z = top == -INFINITY ? 0.f : top;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = tc::ex2(stat_m[w][row] - z);
        const float4 v = *reinterpret_cast<const float4*>(sums + w * SUMS + row * S::kPitch + col);
        sum += stat_l[w][row] * f;
        acc.x += v.x * f;
        acc.y += v.y * f;
        acc.z += v.z * f;
        acc.w += v.w * f;
      }
      if (whole) {
        int t, hg;
        row_of<ROWS>(p, s, row, &t, &hg);
        write_out<D, T>(p, s, t, hg, col, acc, top, sum);
      } else {
        const long long slot = (2LL * blockIdx.x + (starts ? 1 : 0)) * ROWS + row;
        *reinterpret_cast<float4*>(p.part + slot * D + col) = acc;
        if (col == 0) {
          float* st = p.part + 2LL * p.grid * ROWS * D + slot * 2;
          st[0] = top;
          st[1] = sum;
        }
      }
    }
    tc::fence_async_smem();                    // the next tiles arrive through the async proxy
    __syncthreads();                           // the statistics and the rings are free again
  }
}

constexpr int kGatherWarps = 32;

// Gathers the lists of one item's queries (a 128-row tile of a key head): a
// bit per query and block, and the ascending list of the blocks that any of
// them lists.  A warp per query sets its bits in shared memory; an entry that
// is not ascending or past the sequence is left out, and recorded.
__global__ void __launch_bounds__(kGatherWarps * 32)
cache_gather_kernel(const __grid_constant__ AttnArgs p, int32_t* ucnt, int32_t* ulist, uint32_t* ubits) {
  extern __shared__ uint32_t rows[];            // [warps][words]
  __shared__ uint32_t all[1024];
  __shared__ int warp_tot[kGatherWarps];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  unsigned item = blockIdx.x;
  const int tile = (int)(item % p.tiles);
  item /= p.tiles;
  const int h = (int)(item % p.c.heads), b = (int)(item / p.c.heads);
  const int t0 = (int)((long long)tile * kTileRows / p.group);
  const int t1 = (int)min(((long long)(tile + 1) * kTileRows - 1) / p.group, (long long)p.Tq - 1);
  const int len = seq_len(p, b);
  for (int i = threadIdx.x; i < p.words; i += blockDim.x) all[i] = 0u;
  __syncthreads();
  uint32_t* mine = rows + warp * p.words;
  for (int t = t0 + warp; t <= t1; t += kGatherWarps) {
    for (int i = lane; i < p.words; i += 32) mine[i] = 0u;
    __syncwarp();
    const long long r = ((long long)b * p.Tq + t) * p.c.heads + h;
    const int32_t* list = p.idx + r * p.cap;
    const int n0 = __ldg(p.cnt + r), n = min(max(n0, 0), p.cap);
    bool bad = n != n0;
    for (int i = lane; i < n; i += 32) {
      const int before = i > 0 ? __ldg(list + i - 1) : -1, j = __ldg(list + i);
      if (j > before && j >= 0 && j < p.c.max_blocks && (long long)j * kBlock < len) atomicOr(&mine[j >> 5], 1u << (j & 31));
      else bad = true;
    }
    if (bad) atomicOr(&g_cattn_flags, kFlagIndex);
    __syncwarp();
    uint32_t* out = ubits + ((long long)blockIdx.x * p.tile_queries + (t - t0)) * p.words;
    for (int i = lane; i < p.words; i += 32) {
      out[i] = mine[i];
      if (mine[i]) atomicOr(&all[i], mine[i]);
    }
    __syncwarp();
  }
  __syncthreads();
  // a thread per word (at most 1024): where its blocks go in the list
  const uint32_t w = threadIdx.x < p.words ? all[threadIdx.x] : 0u;
  int up = __popc(w);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, up, o);
    if (lane >= o) up += v;
  }
  if (lane == 31) warp_tot[warp] = up;
  __syncthreads();
  int at = up - __popc(w);
  for (int i = 0; i < warp; ++i) at += warp_tot[i];
  int32_t* list = ulist + (long long)blockIdx.x * p.c.max_blocks + at;
  for (uint32_t m = w; m; m &= m - 1) *list++ = (int)threadIdx.x * 32 + __ffs(m) - 1;
  if (threadIdx.x == blockDim.x - 1) ucnt[blockIdx.x] = at + __popc(w);
}

#include "cache_attn_rows.cuh"

// Joins the items that several CTAs shared: block (c, y) looks at the item
// that the start of CTA c + 1's share splits, and if c holds its first unit
// joins some of its rows.
template <int D, typename T, int ROWS>
__global__ void __launch_bounds__(128) cache_attn_join_kernel(const __grid_constant__ AttnArgs p) {
  constexpr int V = D / 4;                      // lanes of four columns
  constexpr int G = 128 / V;
  __shared__ float4 sums[G][V];
  __shared__ float rowsum[G];
  // (everything up to the wait reads only what was there before the first kernel)
  const Shares sh = shares_of(p);
  const int cta = blockIdx.x;
  // A block without an item to join leaves; the first one waits all the same,
  // so that this grid does not end before the kernel it joins.
  auto leave = [&]() {
    if ((blockIdx.x | blockIdx.y) == 0) cudaGridDependencySynchronize();
  };
  if (cta + 1 >= sh.ctas) return leave();
  const unsigned u = sh.first(cta + 1);
  int seq = 0;
  unsigned before = 0;
  if (!p.idx) find_sequence(p, u, &seq, &before);      // (a gathered item has no idx)
  Segment s;
  int units;
  item_of(p, u, seq, before, &s, &units);
  if (s.j0 == 0) return leave();                // the share begins with an item
  const unsigned u0 = u - s.j0;
  if (sh.of(u0) != cta) return leave();         // an earlier CTA holds the item's first unit
  const int last = sh.of(u0 + units - 1);

  cudaGridDependencySynchronize();
  const float* stats = p.part + 2LL * p.grid * ROWS * D;
  auto slot_of = [&](int c, int row) { return (2LL * c + (c == cta ? 1 : 0)) * ROWS + row; };
  const int v = threadIdx.x % V, g = threadIdx.x / V;
  const bool few = last - cta < 2 * G;          // a lane group per row, else all of them on one
  for (int base = blockIdx.y * (few ? G : 1); base < ROWS; base += gridDim.y * (few ? G : 1)) {
    const int row = few ? base + g : base;
    int t, hg;
    const bool live = row_of<ROWS>(p, s, row, &t, &hg);       // (rows past the end are the last ones)
    if (!few && !live) return;
    float top = -INFINITY, sum = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (live) {
      if (few) {
#pragma unroll 4
        for (int c = cta; c <= last; ++c) top = fmaxf(top, __ldcg(stats + 2 * slot_of(c, row)));
      } else {
        for (int c = cta + (int)threadIdx.x % 32; c <= last; c += 32) top = fmaxf(top, __ldcg(stats + 2 * slot_of(c, row)));
        top = warp_max(top);
      }
      const float z = top == -INFINITY ? 0.f : top;
#pragma unroll 4
      for (int c = cta + (few ? 0 : g); c <= last; c += few ? 1 : G) {
        const long long k = slot_of(c, row);
        const float w = tc::ex2(__ldcg(stats + 2 * k) - z);
        sum += w * __ldcg(stats + 2 * k + 1);
        const float4 a = __ldcg(reinterpret_cast<const float4*>(p.part + k * D) + v);
        x.x += w * a.x;
        x.y += w * a.y;
        x.z += w * a.z;
        x.w += w * a.w;
      }
    }
    if (few) {
      if (live) write_out<D, T>(p, s, t, hg, 4 * v, x, top, sum);
      continue;
    }
    sums[g][v] = x;
    if (v == 0) rowsum[g] = sum;
    __syncthreads();
    if (g == 0) {
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
      write_out<D, T>(p, s, t, hg, 4 * v, x, top, sum);
    }
    __syncthreads();
  }
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

template <int D, typename T, int ROWS>
cudaError_t join(const AttnArgs& p, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)p.grid, ROWS < 32 ? ROWS : 32);
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_attn_join_kernel<D, T, ROWS>, p);
}

template <int D, typename T, bool I8, int NR>
cudaError_t run(const CUtensorMap& mk, const CUtensorMap& mv, const AttnArgs& p, cudaStream_t st) {
  constexpr auto kernel = cache_attn_kernel<D, T, I8, NR>;
  constexpr int smem = Cta<D, NR>::kSmem;
  cudaError_t e = allow_smem<kernel>(smem);
  if (e != cudaSuccess) return e;
  kernel<<<p.grid, Cta<D, NR>::kThreads, smem, st>>>(mk, mv, p);
  e = cudaGetLastError();
  return e != cudaSuccess || p.whole ? e : join<D, T, 8 * NR>(p, st);
}

template <int D, typename T, bool I8>
cudaError_t run_rows(const AttnArgs& p, cudaStream_t st) {
  auto go = [&](auto L_) {
    constexpr auto kernel = cache_attn_rows_kernel<D, T, I8, decltype(L_)::value>;
    cudaError_t e = allow_smem<kernel>(kRowsSmem);
    if (e != cudaSuccess) return e;
    kernel<<<p.grid, kRowsThreads, kRowsSmem, st>>>(p);
    return cudaGetLastError();
  };
  const cudaError_t e = p.ucnt ? go(std::true_type{}) : go(std::false_type{});
  return e != cudaSuccess || p.whole ? e : join<D, T, kTileRows>(p, st);
}

// Rows of a tile for this many query rows per key head (or per list).  16-row
// tiles widen the codes again for each, 128-row tiles cost the same for one
// row as for 128 and start later.  A visit of a page takes an SM 0.43 us
// per 16-row tile (d = 64: 0.23) and 0.72 us (0.62) on 128 rows, which pay 6 to 9 us
// more to start: 32 rows over 4 caches of 60-65k tokens 188 us in two tiles
// and 168 on 128 rows, over 2 of 2-3k tokens 20 and 25; d = 64, 48 rows: 156 and
// 148, and 17 and 22.  The lengths are on the device, so the caches' room counts.
int tile_rows(long long rows, bool lists, const CacheArgs& c) {
  if (rows <= 8) return 8;
  if (lists || rows <= 16) return 16;
  if (rows > (c.d == 128 ? 32 : 48)) return kTileRows;
  const double more = ceil_div(rows, 16) * (c.d == 128 ? 0.43 : 0.23) - (c.d == 128 ? 0.72 : 0.62);
  return more * c.B * c.heads * c.max_blocks > 10.0 * kNumSMs ? kTileRows : 16;
}

// Lists gathered per 128-row tile of queries: the tile visits every block that
// one of its queries lists, rows masked by a bit per query and block.
struct Gather {
  bool use;
  long long items;
  int tiles, queries, words;                // queries: of a tile at most (one may lie in two)
  size_t bits, list, count, total;          // offsets in the workspace, after the partial sums
};
Gather gather_plan(const CacheArgs& c, int heads_q, int Tq, int cap) {
  Gather g{};
  const long long group = heads_q / c.heads, rows = group * Tq;
  g.tiles = ceil_div(rows, kTileRows);
  g.items = (long long)c.B * c.heads * g.tiles;
  g.queries = (int)std::min<long long>(Tq, (kTileRows - 1) / group + 2);
  g.words = ceil_div(c.max_blocks, 32);
  // Per key head: block visits of the lists' own tiles, 0.33 us of an SM each
  // (0.45 with 16 rows), against those of the gathered tiles, 0.72 us each,
  // and about 30 us more for their start, gathering and joining (over 148 SMs
  // and all heads).
  const long long small = (group + (group <= 8 ? 7 : 15)) / (group <= 8 ? 8 : 16);
  const double heads = (double)c.B * c.heads;
  const double lists = heads * Tq * small * std::min(cap, c.max_blocks) * (group <= 8 ? 0.33 : 0.45);
  const double gathered = heads * g.tiles * c.max_blocks * 0.72 + 30.0 * kNumSMs;
  g.use = Tq > 1 && c.max_blocks <= 32768 && g.items <= 4096 && gathered < lists;
  size_t off = 0;
  auto take = [&](size_t bytes) { const size_t o = off; off += (bytes + 255) & ~(size_t)255; return o; };
  g.count = take((size_t)g.items * 4);
  g.list = take((size_t)g.items * c.max_blocks * 4);
  g.bits = take((size_t)g.items * g.queries * g.words * 4);
  g.total = g.use ? off : 0;
  return g;
}

size_t partial_bytes(int rows, int d) { return ((size_t)kNumSMs * 2 * rows * (d + 2) * sizeof(float) + 255) & ~(size_t)255; }

}  // namespace

size_t cache_attn_workspace_bytes(const CacheArgs& c, int heads_q, int Tq, int cap) {
  // whole cache, and with cap > 0 lists too: the larger
  const long long rows = (long long)heads_q / c.heads * Tq;
  size_t need = partial_bytes(std::max(tile_rows(rows, false, c), 16), c.d);
  if (cap > 0) {
    const Gather g = gather_plan(c, heads_q, Tq, cap);
    if (g.use) need = std::max(need, partial_bytes(kTileRows, c.d) + g.total);
  }
  return need;
}

cudaError_t launch_cache_attn(const CacheArgs& c, const void* q, int heads_q, int Tq, int f16, int causal,
                              const int32_t* idx, const int32_t* cnt, int cap, void* o, float* lse, void* ws,
                              int* launches, cudaStream_t st) {
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
  p.grid = kNumSMs;
  const Gather g = idx ? gather_plan(c, heads_q, Tq, cap) : Gather{};
  const long long rows = idx && !g.use ? p.group : (long long)p.group * Tq;
  const int tile = g.use ? kTileRows : tile_rows(rows, idx != nullptr, c);
  p.tiles = ceil_div(rows, tile);
  cudaError_t e = cudaSuccess;
  if (g.use) {
    char* base = static_cast<char*>(ws) + partial_bytes(kTileRows, c.d);
    p.ucnt = reinterpret_cast<int32_t*>(base + g.count);
    p.ulist = reinterpret_cast<int32_t*>(base + g.list);
    p.ubits = reinterpret_cast<uint32_t*>(base + g.bits);
    p.tile_queries = g.queries;
    p.words = g.words;
    e = allow_smem<cache_gather_kernel>(kGatherWarps * 4096);
    if (e != cudaSuccess) return e;
    cache_gather_kernel<<<(unsigned)g.items, kGatherWarps * 32, kGatherWarps * g.words * 4, st>>>(
        p, reinterpret_cast<int32_t*>(base + g.count), reinterpret_cast<int32_t*>(base + g.list),
        reinterpret_cast<uint32_t*>(base + g.bits));
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    p.idx = p.cnt = idx = nullptr;
  }
  // Whole items per CTA where no item is longer than two rounds of the warps,
  // or where the items, all alike, fill the CTAs to within 5%: the second
  // kernel takes 3 us, and so does a round trip of the partial sums.
  const long long items = (long long)c.B * (idx ? Tq : 1) * c.heads * p.tiles;
  const long long rounds = (items + kNumSMs - 1) / kNumSMs;
  p.whole = !g.use && ((idx ? cap : c.max_blocks) <= 16 || (idx && items * 20 >= rounds * kNumSMs * 19));
  CUtensorMap mk, mv;
  const long long map_rows = (long long)c.n_pages * c.heads * kBlock;
  if (tile <= 16 && (!map_codes(&mk, c.k, map_rows, c.d) || !map_codes(&mv, c.v, map_rows, c.d)))
    return cudaErrorInvalidValue;
  auto by_rows = [&](auto D_, auto z, auto i8) {
    constexpr int D = decltype(D_)::value;
    constexpr bool I8 = decltype(i8)::value;
    using T = decltype(z);
    e = tile == 8    ? run<D, T, I8, 1>(mk, mv, p, st)
        : tile == 16 ? run<D, T, I8, 2>(mk, mv, p, st)
                     : run_rows<D, T, I8>(p, st);
  };
  auto by_code = [&](auto D_, auto z) {
    if (c.i8) by_rows(D_, z, std::true_type{});
    else by_rows(D_, z, std::false_type{});
  };
  auto by_type = [&](auto D_) {
    if (f16) by_code(D_, __half{});
    else by_code(D_, __nv_bfloat16{});
  };
  if (c.d == 128) by_type(std::integral_constant<int, 128>{});
  else by_type(std::integral_constant<int, 64>{});
  *launches = (p.whole ? 1 : 2) + g.use;
  return e;
}

// Units of one call at most (32-bit counters).
long long cache_attn_units(const CacheArgs& c, int heads_q, int Tq, const int32_t* idx, int cap) {
  const long long group = heads_q / c.heads;
  const Gather g = idx ? gather_plan(c, heads_q, Tq, cap) : Gather{};
  if (g.use) return g.items * c.max_blocks;
  const long long rows = idx ? group : group * Tq;
  const int tile = tile_rows(rows, idx != nullptr, c);
  return (long long)c.B * (idx ? Tq : 1) * c.heads * ((rows + tile - 1) / tile) * (idx ? cap : c.max_blocks);
}

cudaError_t cattn_flags(unsigned int* v, cudaStream_t st) { return read_and_clear_flags(g_cattn_flags, v, st); }
cudaError_t cattn_error(unsigned int* code, cudaStream_t st) { return tc::read_error(code, st); }

}  // namespace svsa
