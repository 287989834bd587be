// Attention over the block cache for many query rows per key head (chunks of
// a stream): tcgen05 tiles of 128 rows.  Part of cache_attn.cu, whose items,
// shares and joining kernel it uses.
//
// With more than a few 16-row tiles the time is no longer that of reading the
// codes but of widening them again for every tile and of mma.sync.  Here a
// page is widened once per 128 rows, to fp16 in shared memory in the layout
// that the MMA reads, and both products run on the 5th-generation tensor
// cores, two pages to a step:
//     S [128 x 128] = Q [128 x d] K^T       (fp16, the codes themselves)
//     O_h [128 x d] += P_h [128 x 64] V_h   (h = 0, 1: the step's pages; P in tensor memory)
// Roles: warp 0 issues the MMAs; warp 1 copies the codes; warps 4-11 are two
// softmax warpgroups, one thread per query row each, one for each page of a
// step, with a maximum, a row sum and an accumulator of their own, merged at
// the item's end; warps 2, 3 and 12-15 widen the pages.  Measured on 1560
// queries x 12 heads over 32,760 tokens: 694 us with one page to a step, 645
// with two, 554 with the next step's K widened before this one's V, 404 to 416
// (755 to 778 TFLOP/s) with the copies and the tables in a warp of their own,
// which looks 32 blocks up at a time (510 with both in a seventh widening warp,
// whose time every stage then waits for).
//
// Scales: the key scale joins the softmax's factor.  The value scale goes
// into the weights as an exponent, P = 2^(y - m'), y = s + log2 vs, with a
// reference m' of its own for y, so the fp16 weights are measured against the
// largest contribution to the output whatever the scales; the row sum is
// kept against the maximum of s.  A page whose value scale is zero (or below
// the normal range) has no part in the output: its weights are zeros, it does
// not touch m', and its terms of the row sum are taken on their own.  Both
// references are lazy.  That of s is raised when passed by 2^12.  m' is put
// 2^11 below the largest y and raised when a y passes it by 2^15 (fp16 ends at
// 2^16), so that weights down to 2^-35 of the largest keep a value and those
// down to 2^-25 all of fp16's bits: a tail below one dominant key counts.  When
// one row's m' has to rise, all of its warp's do: with each at its own time, 60
// queries x 12 heads over 32,760 tokens took 54.3 us, now 53.0 (51.7 with m' at
// the largest y and 2^12 of room, which lost such tails).
//
// Bound by the hand-offs of a step (S, softmax, P V): without the widening the
// same loop takes nine tenths of the time.

constexpr int kRowsThreads = 512;               // 16 warps, 128 registers a thread
constexpr int kWideWarps = 6;                   // warps 2, 3 and 12-15
constexpr int kKvStages = 3, kSBufs = 2;        // stages (a step's K or V) in shared memory, steps in S buffers
constexpr float kLazy = 12.f;
constexpr float kHead = 11.f, kRoom = 15.f;     // the largest weights lie between 2^kHead and 2^kRoom
constexpr float kLeastScale = 1.17549435e-38f;  // a value scale below the normal range counts as zero
constexpr float kNone = -3e38f;                 // a reference before the first key
constexpr uint32_t kStep = 32768;               // 128 keys x 128 columns of fp16
constexpr uint32_t kRowsOffKv = kStep, kRowsOffRaw = kRowsOffKv + kKvStages * kStep;
constexpr int kRaw = 5;                         // stages of codes in flight
constexpr uint32_t kRowsOffMisc = kRowsOffRaw + kRaw * 16384;
constexpr int kRowsSmem = (int)kRowsOffMisc + 4096 + 1024;      // + alignment of the tiles
constexpr uint32_t kColO = 256;                 // S buffers at 0 and 128; accumulators at 256, 256 + d

enum : int {
  kBarQFull = 0, kBarQEmpty, kBarKvFull, kBarKvEmpty = kBarKvFull + kKvStages, kBarSFull = kBarKvEmpty + kKvStages,
  kBarPFull = kBarSFull + kSBufs,               // [2 halves][kSBufs]
  kBarSFree = kBarPFull + 2 * kSBufs, kBarOFull = kBarSFree + kSBufs, kBarOEmpty, kBarEnd, kBars
};

struct RowsMisc {
  uint64_t bar[kBars];
  uint64_t raw_full[kRaw], raw_empty[kRaw];     // the stages of codes
  int2 rows[kRaw];                              // rows of their two pages
  uint32_t tmem, abort;
  float fac[kTileRows];
  float xch[2][3][kTileRows];                   // of each half: reference of y, of s, row sum
};
static_assert(sizeof(RowsMisc) <= 4096, "misc region");

__device__ __forceinline__ void tmem_st32u(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
      "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]),
      "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// The CTA's segments, in the order that every role walks them.
struct Segments {
  Shares sh;
  unsigned u, u_end, before, item;              // item: with gathered lists
  int seq;
  // a warp calls; false: nothing for this CTA
  __device__ bool init(const AttnArgs& p) {
    sh = shares_of(p);
    if ((int)blockIdx.x >= sh.ctas) return false;
    u = sh.first(blockIdx.x);
    u_end = sh.first(blockIdx.x + 1);
    seq = 0;
    before = item = 0;
    if (!p.whole) find_sequence(p, u, &seq, &before);
    return true;
  }
  __device__ bool next(const AttnArgs& p, Segment* s, int* len, bool* starts, bool* whole) {
    if (u >= u_end) return false;
    int units;
    item_of(p, u, seq, before, s, &units);
    *starts = s->j0 == 0;
    s->j1 = (int)min((unsigned)units, s->j0 + (u_end - u));
    *whole = *starts && s->j1 == units;
    u += s->j1 - s->j0;
    if (p.ucnt ? s->j1 == units : !p.whole && u - before == (unsigned)units * p.c.heads * p.tiles) {
      before = u;
      seq += 1;
    }
    *len = seq_len(p, s->b);
    if (p.whole) s->j1 = blocks_of(*len);
    if (p.ucnt) {                               // (an item without a block has one unit, and nothing in it)
      item = ((unsigned)s->b * p.c.heads + s->h) * p.tiles + s->tile;
      if (__ldg(p.ucnt + item) == 0) *len = 0;
    }
    return true;
  }
};

// The block of unit j, and its page, or -1 (an empty sequence, a page out of range).
template <bool LISTS>
__device__ __forceinline__ int block_of(const AttnArgs& p, unsigned item, int j) {
  return LISTS ? __ldg(p.ulist + (long long)item * p.c.max_blocks + j) : j;
}
__device__ __forceinline__ int page_of(const AttnArgs& p, int b, int j, int len) {
  if (len <= 0) return -1;
  const int page = __ldg(p.c.table + (long long)b * p.c.max_blocks + j);
  return (unsigned)page < (unsigned)p.c.n_pages ? page : -1;
}

// A segment's stages: K 0, K 1, V 0, K 2, V 1, ..., V steps - 1.
__device__ __forceinline__ int stages_of(const Segment& s) { return (s.j1 - s.j0 + 1) / 2 * 2; }
__device__ __forceinline__ bool is_v(int g, int stages) { return g > 0 && ((g & 1) == 0 || g == stages - 1); }
__device__ __forceinline__ int step_of(int g, int stages) {
  return g == 0 ? 0 : g & 1 ? min((g + 1) / 2, stages / 2 - 1) : g / 2 - 1;
}

template <int D, typename T, bool I8, bool LISTS>
__global__ void __launch_bounds__(kRowsThreads, 1) cache_attn_rows_kernel(const __grid_constant__ AttnArgs p) {
  using namespace tc;
  constexpr int KSTEPS = D / 16;
  extern __shared__ unsigned char rows_mem[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(((uintptr_t)rows_mem + 1023) & ~(uintptr_t)1023);
  RowsMisc* ms = reinterpret_cast<RowsMisc*>(smem + kRowsOffMisc);
  const uint32_t sbase = su32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile uint32_t* dead = &ms->abort;
  auto bar = [&](int i) { return su32(&ms->bar[i]); };

  cudaTriggerProgrammaticLaunchCompletion();
  Segments walk;
  if (!walk.init(p)) return;                    // uniform over the CTA
  if (tid == 0) {
    mbar_init(bar(kBarQFull), 1);
    mbar_init(bar(kBarQEmpty), 1);
    for (int i = 0; i < kKvStages; ++i) {
      mbar_init(bar(kBarKvFull + i), kWideWarps);
      mbar_init(bar(kBarKvEmpty + i), 1);
    }
    for (int i = 0; i < kSBufs; ++i) {
      mbar_init(bar(kBarSFull + i), 1);
      mbar_init(bar(kBarPFull + i), 4);          // the first warpgroup
      mbar_init(bar(kBarPFull + kSBufs + i), 4);
      mbar_init(bar(kBarSFree + i), 1);
    }
    for (int i = 0; i < kRaw; ++i) {
      mbar_init(su32(&ms->raw_full[i]), 1);
      mbar_init(su32(&ms->raw_empty[i]), kWideWarps);
    }
    mbar_init(bar(kBarOFull), 1);
    mbar_init(bar(kBarOEmpty), 8);
    mbar_init(bar(kBarEnd), 1);
    ms->abort = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    for (int b = blockIdx.x; b < p.c.B; b += walk.sh.ctas) {      // lengths out of range are clamped, and recorded
      const int n = __ldg(p.c.len + b);
      if (n < 0 || n > p.c.max_blocks * kBlock) atomicOr(&g_cattn_flags, kFlagIndex);
    }
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(su32(&ms->tmem)), "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms->tmem;
  Segment s;
  int len;
  bool starts, whole;

  if (warp == 0) {
    // ---------------------------------------------------------------- MMA issue
    if (lane == 0) {
      constexpr uint32_t ID_S = idesc_f16(false, false, false, 128, 128);   // Q . K^T
      constexpr uint32_t ID_O = idesc_f16(false, false, true, D, 128);      // P . V, V MN-major
      const uint64_t dQ = sdesc(sbase, 16, 1024);
      const uint64_t dK = sdesc(sbase + kRowsOffKv, 16, 1024);
      const uint64_t dV = sdesc(sbase + kRowsOffKv, 16384, 1024);
      uint32_t n = 0, item = 0;                 // steps before this item (two stages each); items
      bool ok = true;
      while (ok && walk.next(p, &s, &len, &starts, &whole)) {
        ok = wait_bar(bar(kBarQFull), item & 1u, dead, 101);
        const uint32_t first = n, end = n + (uint32_t)stages_of(s) / 2;
        // S runs one step ahead of P V
        for (uint32_t x = first; ok && x <= end; ++x) {
          if (x < end) {
            const uint32_t g = x == first ? 2 * x : 2 * x - 1, st = g % kKvStages, sb = x % kSBufs;
            ok = wait_bar(bar(kBarKvFull + st), (g / kKvStages) & 1u, dead, 102) &&
                 wait_bar(bar(kBarSFree + sb), ((x / kSBufs) & 1u) ^ 1u, dead, 103);
            if (!ok) break;
            tc_fence_after();
            const uint64_t b0 = dK + ((st * kStep) >> 4);
#pragma unroll
            for (int kk = 0; kk < KSTEPS; ++kk) {
              const uint32_t off = (uint32_t)(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4);
              umma_f16(tmem + sb * 128, dQ + off, b0 + off, ID_S, kk > 0 ? 1u : 0u);
            }
            umma_commit(bar(kBarKvEmpty + st));
            umma_commit(bar(kBarSFull + sb));
            if (x == end - 1) umma_commit(bar(kBarQEmpty));
          }
          if (x > first) {
            const uint32_t y = x - 1, g = x == end ? 2 * y + 1 : 2 * y + 2, st = g % kKvStages, sb = y % kSBufs;
            ok = wait_bar(bar(kBarKvFull + st), (g / kKvStages) & 1u, dead, 104) &&
                 (y > first || wait_bar(bar(kBarOEmpty), (item & 1u) ^ 1u, dead, 105));
            const uint64_t b0 = dV + ((st * kStep) >> 4);
#pragma unroll
            for (int h = 0; h < 2 && ok; ++h) {
              ok = wait_bar(bar(kBarPFull + h * kSBufs + sb), (y / kSBufs) & 1u, dead, 106);
              if (!ok) break;
              tc_fence_after();
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                umma_f16_ts(tmem + kColO + h * D, tmem + sb * 128 + 64 * h + kk * 8, b0 + (uint32_t)(((4 * h + kk) * 2048) >> 4),
                            ID_O, (y > first || kk > 0) ? 1u : 0u);
            }
            if (!ok) break;
            umma_commit(bar(kBarKvEmpty + st));
            umma_commit(bar(kBarSFree + sb));
          }
        }
        if (ok) umma_commit(bar(kBarOFull));
        n = end;
        ++item;
      }
      // every MMA issued here has finished before the tensor memory is given back
      umma_commit(bar(kBarEnd));
      volatile uint32_t no_abort = 0u;
      wait_bar(bar(kBarEnd), 0u, &no_abort, 107);
    }
  } else if (warp < 4 || warp >= 12) {
    // ---------------------------------------------------------------- widening
    // Stages of two pages' K or V, in the order in which they are needed: K of
    // the next step before V of this one (V is read a softmax later).  One warp
    // copies the codes to a ring of kRaw stages ahead of time, a bulk copy to a
    // page; six widen them, warp w rows RW w + RPP i of the stage's 128.  The
    // 16-byte pieces lie over the lanes so that neither the loads of codes nor
    // the fp16 stores (swizzled) meet a bank twice.
    constexpr int CPR = D / 16;                  // pieces of a row of codes
    constexpr int RW = 32 / CPR;                 // rows of a pass
    constexpr int RPP = RW * kWideWarps;
    constexpr int P = (2 * kBlock + RPP - 1) / RPP;
    const int ww = warp < 4 ? warp - 2 : warp - 10;      // (-1: the copying warp)
    const int cc = lane & (CPR - 1);
    const int r0 = ww * RW + (D == 128 ? (lane >> 3 & 2) | ((lane >> 2 ^ lane >> 3) & 1) : lane >> 2);
    uint32_t n = 0, asked = 0;                   // stages before this item; copied by now
    bool ok = true;
    while (ok && walk.next(p, &s, &len, &starts, &whole)) {
      const int stages = stages_of(s);           // (a page that is not there is zeros)
      // The copying warp looks blocks up 32 at a time, one to a lane, two batches
      // at hand: the tables' latency is met once in 16 steps.
      int blks[2], pages[2];
      float scales[2];
      auto look = [&](int batch, int* blk, int* page, float* scale) {
        const int j = s.j0 + 32 * batch + lane;
        *blk = 0;
        *page = -1;
        *scale = 0.f;
        if (j < s.j1 && len > 0) {
          *blk = block_of<LISTS>(p, walk.item, j);
          *page = page_of(p, s.b, *blk, len);
          if (*page >= 0) *scale = __ldg(p.c.v_scale + (long long)*page * p.c.heads + s.h);
        }
      };
      // starts the copies of stage g and says how many rows of each page there are
      // (V rows past the sequence, and those of a value scale of zero, are zeros)
      auto ask = [&](int g) {
        const uint32_t to = asked % kRaw;
        if (!__all_sync(0xffffffffu, wait_bar(su32(&ms->raw_empty[to]), ((asked / kRaw) & 1u) ^ 1u, dead, 114))) return false;
        const bool v = is_v(g, stages);
        const int j = 2 * step_of(g, stages), from = (j & 31) + (lane & 1);
        const bool odd = j >> 5 & 1;
        const int blk = __shfl_sync(0xffffffffu, odd ? blks[1] : blks[0], from);
        const int page = __shfl_sync(0xffffffffu, odd ? pages[1] : pages[0], from);
        const float scale = __shfl_sync(0xffffffffu, odd ? scales[1] : scales[0], from);
        int rows = 0;
        if (page >= 0) rows = !v ? kBlock : scale >= kLeastScale ? min(max(len - blk * kBlock, 0), kBlock) : 0;
        const int other = __shfl_sync(0xffffffffu, rows, 1);
        const uint32_t full = su32(&ms->raw_full[to]);
        if (lane == 0) {
          ms->rows[to] = make_int2(rows, other);
          mbar_expect_tx(full, (uint32_t)(rows + other) * D);
        }
        __syncwarp();
        if (rows && lane < 2)
          bulk_load(sbase + kRowsOffRaw + to * 16384 + lane * (kBlock * D),
                    static_cast<const char*>(v ? p.c.v : p.c.k) + ((long long)page * p.c.heads + s.h) * (kBlock * D), (uint32_t)rows * D,
                    full);
        ++asked;
        // the values of a batch's first step are the last to need the batch before
        if (v && (j & 31) == 0) {
          if (odd) look((j >> 5) + 1, &blks[0], &pages[0], &scales[0]);
          else look((j >> 5) + 1, &blks[1], &pages[1], &scales[1]);
        }
        return true;
      };
      if (ww < 0) {
        look(0, &blks[0], &pages[0], &scales[0]);
        for (int g = 0; ok && g < stages; ++g) ok = ask(g);
        n += (uint32_t)stages;
        continue;
      }
      for (int g = 0; g < stages; ++g) {
        const int v = is_v(g, stages);
        const uint32_t x = n + (uint32_t)g, st = x % kKvStages, from_st = x % kRaw;
        ok = ok && wait_bar(su32(&ms->raw_full[from_st]), (x / kRaw) & 1u, dead, 115) &&
             wait_bar(bar(kBarKvEmpty + st), ((x / kKvStages) & 1u) ^ 1u, dead, 108);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t from = sbase + kRowsOffRaw + from_st * 16384 + r0 * D + cc * 16;
        const uint32_t to = sbase + kRowsOffKv + st * kStep + (uint32_t)(cc >> 2) * 16384 + r0 * 128;
        const int2 rows = ms->rows[from_st];
        const bool full = rows.x + rows.y == 2 * kBlock;
        uint4 c[P];                              // all loads before the first store
#pragma unroll
        for (int i = 0; i < P; ++i)
          if (ww * RW + RPP * i < 2 * kBlock) c[i] = lds128(from + i * RPP * D);
        if (!full) {
#pragma unroll
          for (int i = 0; i < P; ++i) {
            const int r = r0 + RPP * i;
            if (r >= kBlock ? r - kBlock >= rows.y : r >= rows.x) c[i] = make_uint4(0u, 0u, 0u, 0u);
          }
        }
#pragma unroll
        for (int i = 0; i < P; ++i) {
          if (ww * RW + RPP * i < 2 * kBlock) {
            uint32_t y[8];
            Widen<I8>::word(c[i].x, y[0], y[1]);
            Widen<I8>::word(c[i].y, y[2], y[3]);
            Widen<I8>::word(c[i].z, y[4], y[5]);
            Widen<I8>::word(c[i].w, y[6], y[7]);
            const uint32_t at = to + i * RPP * 128 + ((((cc & 3) * 2) ^ ((r0 + RPP * i) & 7)) << 4);
            st_shared_v4(at, y[0], y[1], y[2], y[3]);
            st_shared_v4(at ^ 16u, y[4], y[5], y[6], y[7]);
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(kBarKvFull + st));
          mbar_arrive(su32(&ms->raw_empty[from_st]));
        }
      }
      n += (uint32_t)stages;
      if (len > 0 && ok) {                       // pages out of range, recorded
        bool bad = false;
        for (int j = s.j0 + ww * 32 + lane; j < s.j1; j += kWideWarps * 32)
          bad = bad || page_of(p, s.b, block_of<LISTS>(p, walk.item, j), len) < 0;
        if (bad) atomicOr(&g_cattn_flags, kFlagIndex);
      }
    }
    if (ww < 0) {                                // the copies in flight, before the CTA goes
      volatile uint32_t no_abort = 0u;
      for (uint32_t x = asked > kRaw ? asked - kRaw : 0u; x < asked; ++x)
        wait_bar(su32(&ms->raw_full[x % kRaw]), (x / kRaw) & 1u, &no_abort, 116);
    }
  } else {
    // ---------------------------------------------------------------- softmax
    const int wq = warp & 3, half = warp >= 8 ? 1 : 0, row = wq * 32 + lane;
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const uint32_t own = tmem + lane_off + kColO + half * D;      // this half's accumulator
    constexpr int DH = D / 2;                    // columns this thread stores
    uint32_t n = 0, item = 0;
    bool stop = false;
    while (walk.next(p, &s, &len, &starts, &whole)) {
      // Q of the item: two threads per row, fp16 under the row's power of two
      stop = !wait_bar(bar(kBarQEmpty), (item & 1u) ^ 1u, dead, 110);
      {
        const int qi = tid - 128, qr = qi >> 1, hf = qi & 1;
        int t, hg;
        const bool live = row_of<kTileRows>(p, s, qr, &t, &hg);
        const uint4* src = reinterpret_cast<const uint4*>(
            static_cast<const T*>(p.q) + (((long long)s.b * p.heads_q + s.h * p.group + hg) * p.Tq + t) * D + hf * DH);
        uint4 raw[DH / 8];
#pragma unroll
        for (int i = 0; i < DH / 8; ++i) raw[i] = live ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
        auto pair = [&](int i) {
          const uint32_t w = reinterpret_cast<const uint32_t*>(raw)[i];
          if constexpr (std::is_same<T, __half>::value) return __half22float2(*reinterpret_cast<const __half2*>(&w));
          else return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
        };
        float amax = 0.f;
        bool odd = false;
#pragma unroll
        for (int i = 0; i < DH / 2; ++i) {
          const float2 f = pair(i);
          odd = odd || !(fabsf(f.x) < INFINITY) || !(fabsf(f.y) < INFINITY);
          amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        odd = (__ballot_sync(0xffffffffu, odd) >> (lane & ~1)) & 3u;
        int e = (int)(__float_as_uint(amax) >> 23) - 127;
        e = min(max(e, -126), 126);
        const float down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int i = 0; i < DH / 8; ++i) {
          uint32_t x[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = pair(4 * i + k);
            x[k] = h2bits(__floats2half2_rn(f.x * down, f.y * down));
          }
          const int d0 = hf * DH + 8 * i;
          st_shared_v4(sbase + (d0 / 64) * 16384 + qr * 128 + (((d0 % 64 / 8) ^ (qr & 7)) << 4), x[0], x[1], x[2], x[3]);
        }
        if (hf == 0)
          ms->fac[qr] = odd ? __int_as_float(0x7fffffff)
                            : __uint_as_float((uint32_t)(127 + e) << 23) *
                                  (1.44269504088896340736f / (D == 64 ? 8.f : 11.31370849898476039041f));
        fence_async_smem();
      }
      if (named_bar_or(1, 256, stop)) {          // all eight warps agree
        stop = true;
        break;
      }
      if (tid == 128) mbar_arrive(bar(kBarQFull));
      const float fac = ms->fac[row];
      int t, hg;
      const bool live = row_of<kTileRows>(p, s, row, &t, &hg);
      const int lim = live && p.causal ? max(len - p.Tq + 1 + t, 0) : len;

      float ry = kNone, rs = kNone, l = 0.f;     // references of y and s (log2), row sum against rs
      float ytop = kNone;                        // the largest y
      // this half's pages, looked up 32 steps at a time, one to a lane, and the
      // next 32 half way through them: block (-1: not there) and scales
      auto look = [&](int i, int* blk, float* ks, float* vs) {
        const int j = s.j0 + 2 * (i + lane) + half;
        *blk = -1;
        *ks = *vs = 0.f;
        if (j < s.j1 && len > 0) {
          const int b = block_of<LISTS>(p, walk.item, j), page = page_of(p, s.b, b, len);
          if (page >= 0) {
            const long long cell = (long long)page * p.c.heads + s.h;
            *blk = b;
            *ks = __ldg(p.c.k_scale + cell);
            *vs = __ldg(p.c.v_scale + cell);
          }
        }
      };
      int blk_c, blk_n = -1;
      float ks_c, vs_c, ks_n = 0.f, vs_n = 0.f;
      look(0, &blk_c, &ks_c, &vs_c);
      // with gathered lists, whether this row's query lists the page, a step ahead
      const uint32_t* bits = nullptr;
      if (LISTS) bits = p.ubits + ((long long)walk.item * p.tile_queries + (live ? t - (int)((long long)s.tile * kTileRows / p.group) : 0)) * p.words;
      auto lists = [&](int blk) { return !LISTS || blk < 0 || (__ldg(bits + (blk >> 5)) >> (blk & 31) & 1u); };
      bool listed = lists(__shfl_sync(0xffffffffu, blk_c, 0)), listed_n = listed;
      const int steps = stages_of(s) / 2;        // (a page that is not there is masked)
      for (int i = 0; i < steps; ++i) {
        const uint32_t x = n + (uint32_t)i, sb = x % kSBufs;
        if ((i & 31) == 16) look(i + 16, &blk_n, &ks_n, &vs_n);
        const int blk = __shfl_sync(0xffffffffu, blk_c, i & 31), tok = blk < 0 ? 1 << 30 : blk * kBlock;
        const float ks = __shfl_sync(0xffffffffu, ks_c, i & 31), vs = __shfl_sync(0xffffffffu, vs_c, i & 31);
        if ((i & 31) == 31) {
          blk_c = blk_n;
          ks_c = ks_n;
          vs_c = vs_n;
        }
        if (LISTS) listed_n = lists(__shfl_sync(0xffffffffu, blk_c, (i + 1) & 31));
        if (!__all_sync(0xffffffffu, wait_bar(bar(kBarSFull + sb), (x / kSBufs) & 1u, dead, 111))) {
          stop = true;
          break;
        }
        tc_fence_after();
        float v[64];
        tmem_ld32(tmem + lane_off + sb * 128 + 64 * half, v);
        tmem_ld32(tmem + lane_off + sb * 128 + 64 * half + 32, v + 32);
        tmem_wait_ld();
        // (a page that is not there has no key either, and no row sum to take on its own)
        const float f = fac * ks, lv = vs >= kLeastScale ? __log2f(vs) : blk < 0 ? 0.f : -INFINITY;
        // the largest s of the row (log2 units; f >= 0)
        const bool edge = !__all_sync(0xffffffffu, tok + kBlock <= lim);
        if (edge) {
#pragma unroll
          for (int c = 0; c < 64; ++c) v[c] = tok + c < lim ? v[c] * f : -INFINITY;
        }
        float m0 = -INFINITY, m1 = -INFINITY, m2 = -INFINITY, m3 = -INFINITY;
#pragma unroll
        for (int c = 0; c < 64; c += 8) {
          m0 = max3(m0, v[c], v[c + 1]);
          m1 = max3(m1, v[c + 2], v[c + 3]);
          m2 = max3(m2, v[c + 4], v[c + 5]);
          m3 = max3(m3, v[c + 6], v[c + 7]);
        }
        const float top = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3));
        const bool skip = LISTS && !listed;      // (the row's query does not list this page)
        const float smax = skip ? -INFINITY : edge ? top : top * f;
        if (smax > -INFINITY) {
          ytop = fmaxf(ytop, smax + lv);         // (no larger without values)
          if (ry == kNone) ry = ytop - kHead;    // (the accumulator holds zeros)
          if (smax > rs + kLazy) {
            l *= ex2(rs - smax);                 // (of the first key: 0 times 0)
            rs = smax;
          }
        }
        if (__any_sync(0xffffffffu, ytop > ry + kRoom)) {
          // one row's reference has to rise: all of the warp's do, which makes
          // the next time come later
          const float to = fmaxf(ry, ytop - kHead), alpha = ex2(ry - to);
          ry = to;
          // rescale this half's accumulator (factor 1 where nothing changed)
          // once its previous P V product is done; there is one, in this item
          const uint32_t xp = x - 1u, sp = xp % kSBufs;
          if (!__all_sync(0xffffffffu, wait_bar(bar(kBarSFree + sp), (xp / kSBufs) & 1u, dead, 112))) {
            stop = true;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int c0 = 0; c0 < D; c0 += 16) {
            float o[16];
            tmem_ld16(own + c0, o);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 16; ++c) o[c] *= alpha;
            tmem_st16(own + c0, o);
          }
          tmem_wait_st();
        }
        // P = 2^(s + lv - ry) as fp16 pairs over the first 32 of this half's 64 S columns
        uint32_t pk[32];
        const float shift = skip ? -INFINITY : lv - ry;
        const F2 ff = edge ? f2(1.f, 1.f) : f2(f, f), zz = f2(shift, shift);
        // the row sum's terms are 2^gap times the weights; where a tiny value
        // scale makes that too much for fp32, or there are no values (gap is
        // infinite), they are taken on their own
        const float gap = ry - lv - rs;
        float lone = 0.f;
        if (__any_sync(0xffffffffu, gap > 60.f)) {
          const F2 rr = f2(-rs, -rs);
#pragma unroll
          for (int c = 0; c < 64; c += 2) {
            float e0, e1;
            split2(fma2(f2(v[c], v[c + 1]), ff, rr), e0, e1);
            lone += ex2(e0) + ex2(e1);
          }
        }
        F2 sum0 = f2(0.f, 0.f), sum1 = sum0;
#pragma unroll
        for (int c = 0; c < 64; c += 4) {
          float e0, e1, e2, e3;
          split2(fma2(f2(v[c], v[c + 1]), ff, zz), e0, e1);
          split2(fma2(f2(v[c + 2], v[c + 3]), ff, zz), e2, e3);
          e0 = ex2(e0);
          e1 = ex2(e1);
          e2 = ex2(e2);
          e3 = ex2(e3);
          sum0 = add2(sum0, f2(e0, e1));
          sum1 = add2(sum1, f2(e2, e3));
          pk[c / 2] = pack_f16x2(e0, e1);
          pk[c / 2 + 1] = pack_f16x2(e2, e3);
        }
        tmem_st32u(tmem + lane_off + sb * 128 + 64 * half, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarPFull + half * kSBufs + sb));
        float a0, a1;
        split2(add2(sum0, sum1), a0, a1);
        if (!skip) l += gap > 60.f ? lone : (a0 + a1) * ex2(gap);
        listed = listed_n;
      }
      n += (uint32_t)steps;

      // the two halves, merged; then this thread's half of the columns
      const bool ok = !stop && __all_sync(0xffffffffu, wait_bar(bar(kBarOFull), item & 1u, dead, 113));
      ms->xch[half][0][row] = ry;
      ms->xch[half][1][row] = rs;
      ms->xch[half][2][row] = l;
      if (named_bar_or(1, 256, !ok)) {           // all eight warps agree
        stop = true;
        break;
      }
      ++item;
      tc_fence_after();
      const float yA = ms->xch[0][0][row], sA = ms->xch[0][1][row], lA = ms->xch[0][2][row];
      const float yB = ms->xch[1][0][row], sB = ms->xch[1][1][row], lB = ms->xch[1][2][row];
      // (a half without a key has l = 0 and takes no part; NaN stays)
      const float top = fmaxf(lA != 0.f ? sA : -INFINITY, lB != 0.f ? sB : -INFINITY);
      const float z = top == -INFINITY ? 0.f : top;
      const float wA = lA != 0.f ? ex2(yA - z) : 0.f, wB = lB != 0.f ? ex2(yB - z) : 0.f;
      const float sum = (lA != 0.f ? lA * ex2(sA - z) : 0.f) + (lB != 0.f ? lB * ex2(sB - z) : 0.f);
      float* const part = p.part + ((2LL * blockIdx.x + (starts ? 1 : 0)) * kTileRows + row) * D;
#pragma unroll
      for (int c0 = 0; c0 < DH; c0 += 16) {
        float oa[16], ob[16];
        tmem_ld16(tmem + lane_off + kColO + half * DH + c0, oa);
        tmem_ld16(tmem + lane_off + kColO + D + half * DH + c0, ob);
        tmem_wait_ld();
        if (live) {
#pragma unroll
          for (int c = 0; c < 16; c += 4) {
            float r[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) r[k] = (lA != 0.f ? oa[c + k] * wA : 0.f) + (lB != 0.f ? ob[c + k] * wB : 0.f);
            const int col = half * DH + c0 + c;
            const float4 x4 = make_float4(r[0], r[1], r[2], r[3]);
            // (kShift: the joining kernel's sums are held times 2^kShift)
            if (whole) write_out<D, T>(p, s, t, hg, col, x4, top + kShift, sum);
            else *reinterpret_cast<float4*>(part + col) = x4;
          }
        }
      }
      if (!whole && live && half == 0) {
        float* st = p.part + 2LL * p.grid * kTileRows * D + ((2LL * blockIdx.x + (starts ? 1 : 0)) * kTileRows + row) * 2;
        st[0] = top + kShift;
        st[1] = sum;
      }
      // the accumulators, and the exchanged values, are free for the next item
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarOEmpty));
      named_bar(2, 256);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(512u));
  }
}
