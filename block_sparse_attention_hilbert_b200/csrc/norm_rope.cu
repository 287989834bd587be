// Per-head RMS norm of the queries and keys with their position rotation, in
// the pass that also puts the rows in the library's token order, and its
// gradients.
//
// With r = (mean_c x_c^2 + eps)^-1/2 and y = r w x (per row of d values), pair
// i of the row, (a, b) = (y_2i, y_2i+1) or (y_i, y_i+d/2), becomes
//   (a cos t_i - b sin t_i, a sin t_i + b cos t_i),
// t_i the angle of the pair at the token's position on the pair's axis (its
// cosine and sine come from tables).  Backward, with g = the output's gradient
// turned back by -t_i:
//   dw = sum over rows of g r x,   dx = r g w - x r^3 mean_c(g w x).
//
// Both are bound by HBM: 4 bytes per value forward (2 read, 2 written), 6
// backward.  d / 8 lanes hold a row, eight values (four pairs) each, so a
// row's sums are 3 or 4 shuffles and no pair spans two lanes: with the
// (i, i + d/2) pairing a lane takes four values from each half.  A lane group
// keeps its token's four cosines and sines and walks over heads, four rows in
// flight: the tables (fp32, as wide as the row itself) are read once per token
// and head group instead of once per row.
#include "common.cuh"

#include <cuda_fp16.h>

#include <type_traits>

#include "stream.cuh"

namespace svsa {

// Status bits of this translation unit (kFlagIndex: a position or map entry out of range).
static __device__ unsigned int g_rope_flags;

namespace {

constexpr int kThreads = 256;
constexpr int kRowsInFlight = 4;
constexpr int kFwdPerSM = 4, kBwdPerSM = 2;     // CTAs per SM that the registers are held to
constexpr int kStages = 3;                 // steps in the backward's ring
constexpr int kBwdSmem = kStages * 2 * kRowsInFlight * kThreads * 16;

// The call's arguments, and how its heads are split.
struct NormRope : NormRopeArgs {
  int chunks[2];                    // head groups of `hb` heads
  int hb;
};

template <typename T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
  __device__ static float2 load(uint32_t v) { return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&v)); }
  __device__ static uint32_t store(float a, float b) { return pack_bf16x2(a, b); }
};
template <>
struct Pair<__half> {
  __device__ static float2 load(uint32_t v) { return __half22float2(*reinterpret_cast<__half2*>(&v)); }
  __device__ static uint32_t store(float a, float b) {
    __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
  }
};

// The eight values of lane `ch` of a row: 16 bytes in one piece, or, for the
// (i, i + d/2) pairing, 8 bytes from each half.  Either way a[i], b[i] is pair
// 4 * ch + i.
template <int D, bool HALVES>
__device__ __forceinline__ uint4 load_row(const void* row, int ch) {
  if constexpr (HALVES) {
    const uint2 lo = *reinterpret_cast<const uint2*>(static_cast<const char*>(row) + ch * 8);
    const uint2 hi = *reinterpret_cast<const uint2*>(static_cast<const char*>(row) + D + ch * 8);
    return make_uint4(lo.x, lo.y, hi.x, hi.y);
  } else {
    return *reinterpret_cast<const uint4*>(static_cast<const char*>(row) + ch * 16);
  }
}

template <int D, bool HALVES>
__device__ __forceinline__ void store_row(void* row, int ch, uint4 v) {
  if constexpr (HALVES) {
    *reinterpret_cast<uint2*>(static_cast<char*>(row) + ch * 8) = make_uint2(v.x, v.y);
    *reinterpret_cast<uint2*>(static_cast<char*>(row) + D + ch * 8) = make_uint2(v.z, v.w);
  } else {
    *reinterpret_cast<uint4*>(static_cast<char*>(row) + ch * 16) = v;
  }
}

template <typename T, bool HALVES>
__device__ __forceinline__ void unpack(uint4 v, float a[4], float b[4]) {
  const float2 f0 = Pair<T>::load(v.x), f1 = Pair<T>::load(v.y), f2 = Pair<T>::load(v.z), f3 = Pair<T>::load(v.w);
  if constexpr (HALVES) {
    a[0] = f0.x; a[1] = f0.y; a[2] = f1.x; a[3] = f1.y;
    b[0] = f2.x; b[1] = f2.y; b[2] = f3.x; b[3] = f3.y;
  } else {
    a[0] = f0.x; b[0] = f0.y; a[1] = f1.x; b[1] = f1.y;
    a[2] = f2.x; b[2] = f2.y; a[3] = f3.x; b[3] = f3.y;
  }
}

template <typename T, bool HALVES>
__device__ __forceinline__ uint4 pack(const float a[4], const float b[4]) {
  if constexpr (HALVES)
    return make_uint4(Pair<T>::store(a[0], a[1]), Pair<T>::store(a[2], a[3]), Pair<T>::store(b[0], b[1]),
                      Pair<T>::store(b[2], b[3]));
  else
    return make_uint4(Pair<T>::store(a[0], b[0]), Pair<T>::store(a[1], b[1]), Pair<T>::store(a[2], b[2]),
                      Pair<T>::store(a[3], b[3]));
}

// The weights of lane ch, in the same places (ones without a weight vector).
template <int D, bool HALVES>
__device__ __forceinline__ void load_weights(const float* w, int ch, float wa[4], float wb[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int p = 4 * ch + i;
    wa[i] = w ? __ldg(w + (HALVES ? p : 2 * p)) : 1.f;
    wb[i] = w ? __ldg(w + (HALVES ? p + D / 2 : 2 * p + 1)) : 1.f;
  }
}

// Cosines and sines of the lane's four pairs for token n of batch row b; a
// position outside the tables is clamped and recorded.
template <int D>
__device__ __forceinline__ void load_angles(const NormRope& p, int b, int n, int ch, float c[4], float s[4]) {
  const int32_t* at = p.pos + (long long)b * p.pos_stride + (long long)n * p.axes;
  bool bad = false;
  long long row[3];
#pragma unroll
  for (int a = 0; a < 3; ++a) {
    int v = a < p.axes ? __ldg(at + a) : 0;
    if ((unsigned)v >= (unsigned)p.table_rows) {
      bad = bad || a < p.axes;
      v = v < 0 ? 0 : p.table_rows - 1;
    }
    row[a] = (long long)v * (D / 2);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int pair = 4 * ch + i;
    const long long r = pair < p.split1 ? row[0] : pair < p.split2 ? row[1] : row[2];
    c[i] = __ldg(p.cos + r + pair);
    s[i] = __ldg(p.sin + r + pair);
  }
  if (bad) atomicOr(&g_rope_flags, kFlagIndex);
}

template <int LANES>
__device__ __forceinline__ float group_sum(float v, unsigned mask) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(mask, v, o);
  return v;
}

// One lane group per (token, head group); blockIdx.y is the head group, so
// that the groups of a CTA write neighbouring rows of one head.
template <int D, typename T, bool HALVES, bool TURN>
__global__ void __launch_bounds__(kThreads, kFwdPerSM) norm_rope_kernel(const __grid_constant__ NormRope p) {
  constexpr int L = D / 8;                      // lanes per row
  const int ch = threadIdx.x % L;
  const unsigned mask = ((1u << L) - 1) << ((threadIdx.x % 32) / L * L);
  const unsigned tok = blockIdx.x * (kThreads / L) + threadIdx.x / L;
  if (tok >= (unsigned)(p.B * p.rows)) return;                // uniform over the lane group
  const int which = (int)blockIdx.y >= p.chunks[0];
  const int h0 = ((int)blockIdx.y - (which ? p.chunks[0] : 0)) * p.hb;
  const int h1 = min(h0 + p.hb, p.heads[which]);
  const int b = (int)(tok / (unsigned)p.rows), i = (int)(tok - (unsigned)b * p.rows);

  int n = p.map ? __ldg(p.map + i) : i;
  if (n >= p.N || n < -1) {
    atomicOr(&g_rope_flags, kFlagIndex);
    n = -1;
  }
  char* out = static_cast<char*>(p.out[which]) + (((long long)b * p.heads[which]) * p.rows + i) * (2LL * D);
  const long long out_step = (long long)p.rows * (2LL * D);
  if (n < 0) {                                   // a pad row
    for (int h = h0; h < h1; ++h) store_row<D, HALVES>(out + h * out_step, ch, make_uint4(0u, 0u, 0u, 0u));
    return;
  }
  const char* x = static_cast<const char*>(p.x[which]) +
                  2 * ((long long)b * p.stride[which][0] + (long long)n * p.stride[which][2]);
  const long long x_step = 2 * p.stride[which][1];

  float c[4], s[4], wa[4], wb[4];
  uint4 v[kRowsInFlight];
#pragma unroll
  for (int u = 0; u < kRowsInFlight; ++u)
    if (h0 + u < h1) v[u] = load_row<D, HALVES>(x + (h0 + u) * x_step, ch);
  if constexpr (TURN) load_angles<D>(p, b, n, ch, c, s);
  load_weights<D, HALVES>(p.w[which], ch, wa, wb);

  for (int h = h0; h < h1; h += kRowsInFlight) {
    if (h > h0) {
#pragma unroll
      for (int u = 0; u < kRowsInFlight; ++u)
        if (h + u < h1) v[u] = load_row<D, HALVES>(x + (h + u) * x_step, ch);
    }
#pragma unroll
    for (int u = 0; u < kRowsInFlight; ++u) {
      if (h + u >= h1) break;                    // uniform over the lane group
      float a[4], bb[4];
      unpack<T, HALVES>(v[u], a, bb);
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) ss += a[e] * a[e] + bb[e] * bb[e];
      ss = group_sum<L>(ss, mask);
      const float r = rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        a[e] *= r * wa[e];
        bb[e] *= r * wb[e];
        if constexpr (TURN) {
          const float t = a[e] * c[e] - bb[e] * s[e];
          bb[e] = a[e] * s[e] + bb[e] * c[e];
          a[e] = t;
        }
      }
      store_row<D, HALVES>(out + (h + u) * out_step, ch, pack<T, HALVES>(a, bb));
    }
  }
}

// This thread's 16 bytes of a row, copied to its own place in shared memory.
template <int D, bool HALVES>
__device__ __forceinline__ void copy_row(uint32_t to, const char* row, int ch) {
  if constexpr (HALVES) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(to), "l"(row + ch * 8) : "memory");
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(to + 8), "l"(row + D + ch * 8) : "memory");
  } else {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(to), "l"(row + ch * 16) : "memory");
  }
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}

// Backward.  The CTAs are split between q and k (ctas_q of them first) and
// among their head groups; each walks over its token tiles with a fixed
// stride, keeps dw in registers and writes one partial row, so the sums run in
// an order that only the sizes and the grid fix.  The rows come through a ring
// of kStages steps of four rows in shared memory, each thread copying and
// reading only its own bytes (no barrier): with the loads in registers instead
// a warp either waited or computed: 125 us where this takes 116 us (12 heads
// of 32,760 tokens).
template <int D, typename T, bool HALVES, bool TURN>
__global__ void __launch_bounds__(kThreads, kBwdPerSM) norm_rope_bwd_kernel(const __grid_constant__ NormRope p, int ctas_q) {
  constexpr int L = D / 8;
  constexpr int G = kThreads / L;               // lane groups
  extern __shared__ __align__(16) uint8_t ring_mem[];
  __shared__ float red[G][D];
  cudaTriggerProgrammaticLaunchCompletion();    // (the summing kernel may take its place; it waits for this one's end)
  const int ch = threadIdx.x % L, grp = threadIdx.x / L;
  const unsigned mask = ((1u << L) - 1) << ((threadIdx.x % 32) / L * L);
  const int which = (int)blockIdx.x >= ctas_q;
  const int cta = which ? (int)blockIdx.x - ctas_q : (int)blockIdx.x;
  const int ctas = (which ? (int)gridDim.x - ctas_q : ctas_q) / p.chunks[which];      // of one head group
  const int h0 = cta / ctas * p.hb, h1 = min(h0 + p.hb, p.heads[which]);
  const unsigned tokens = (unsigned)(p.B * p.N);
  const unsigned stride = (unsigned)ctas * G;
  const long long x_step = 2 * p.stride[which][1], dx_step = 2 * p.out_stride[which][1];
  const long long dy_step = (long long)p.rows * (2LL * D);
  float wa[4], wb[4], da[4] = {0.f, 0.f, 0.f, 0.f}, db[4] = {0.f, 0.f, 0.f, 0.f};
  load_weights<D, HALVES>(p.w[which], ch, wa, wb);

  // the output row of token tok (-1: none, or no such token)
  auto row_of = [&](unsigned tok) {
    if (tok >= tokens) return -1;
    const int n = (int)(tok % (unsigned)p.N);
    const int i = p.map ? __ldg(p.map + n) : n;
    if (i >= p.rows || i < -1) {
      atomicOr(&g_rope_flags, kFlagIndex);
      return -1;
    }
    return i;
  };
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(ring_mem) + threadIdx.x * 16;
  constexpr uint32_t kPiece = kThreads * 16, kStep = 2 * kRowsInFlight * kPiece;

  // the next step to ask for: heads ph .. ph + 3 of token ptok
  unsigned ptok = (unsigned)(cta % ctas) * G + grp;
  int ph = h0, prow = row_of(ptok), pnext = row_of(ptok + stride), pslot = 0;
  const char *px = nullptr, *pdy = nullptr;
  auto ask = [&]() {
    if (ptok < tokens) {
      if (ph == h0) {
        const int b = (int)(ptok / (unsigned)p.N), n = (int)(ptok - (unsigned)b * p.N);
        px = static_cast<const char*>(p.x[which]) + 2 * ((long long)b * p.stride[which][0] + (long long)n * p.stride[which][2]) + h0 * x_step;
        pdy = static_cast<const char*>(p.dy[which]) + (((long long)b * p.heads[which] + h0) * p.rows + prow) * (2LL * D);
      }
      if (prow >= 0) {
        const uint32_t to = ring + pslot * kStep;
#pragma unroll
        for (int u = 0; u < kRowsInFlight; ++u)
          if (ph + u < h1) {
            copy_row<D, HALVES>(to + (2 * u) * kPiece, px, ch);
            copy_row<D, HALVES>(to + (2 * u + 1) * kPiece, pdy, ch);
            px += x_step;
            pdy += dy_step;
          }
      }
      ph += kRowsInFlight;
      if (ph >= h1) {
        ph = h0;
        ptok += stride;
        prow = pnext;
        pnext = row_of(ptok + stride);
      }
    }
    asm volatile("cp.async.commit_group;\n" ::: "memory");
    pslot = pslot + 1 == kStages ? 0 : pslot + 1;
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) ask();

  unsigned tok = (unsigned)(cta % ctas) * G + grp;
  int row = row_of(tok), slot = 0;
  float c[4], s[4], cn[4], sn[4];
  if (TURN && row >= 0) load_angles<D>(p, (int)(tok / (unsigned)p.N), (int)(tok % (unsigned)p.N), ch, c, s);
  while (tok < tokens) {
    const int b = (int)(tok / (unsigned)p.N), n = (int)(tok - (unsigned)b * p.N);
    char* dx = static_cast<char*>(p.out[which]) +
               2 * ((long long)b * p.out_stride[which][0] + (long long)n * p.out_stride[which][2]) + h0 * dx_step;
    const unsigned later = tok + stride;
    const int row_next = row_of(later);
    if (TURN && row_next >= 0) load_angles<D>(p, (int)(later / (unsigned)p.N), (int)(later % (unsigned)p.N), ch, cn, sn);
    for (int h = h0; h < h1; h += kRowsInFlight) {
      ask();
      asm volatile("cp.async.wait_group %0;\n" ::"n"(kStages - 1) : "memory");
      const uint32_t from = ring + slot * kStep;
      slot = slot + 1 == kStages ? 0 : slot + 1;
#pragma unroll
      for (int u = 0; u < kRowsInFlight; ++u) {
        if (h + u >= h1) break;                  // uniform over the lane group
        uint4 out = make_uint4(0u, 0u, 0u, 0u);  // (a token without an output row has no gradient)
        if (row >= 0) {
          float a[4], bb[4], ga[4], gb[4];
          unpack<T, HALVES>(lds128(from + (2 * u) * kPiece), a, bb);
          unpack<T, HALVES>(lds128(from + (2 * u + 1) * kPiece), ga, gb);
          float ss = 0.f, dot = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (TURN) {
              const float t = ga[e] * c[e] + gb[e] * s[e];
              gb[e] = gb[e] * c[e] - ga[e] * s[e];
              ga[e] = t;
            }
            ss += a[e] * a[e] + bb[e] * bb[e];
            dot += ga[e] * wa[e] * a[e] + gb[e] * wb[e] * bb[e];
          }
          ss = group_sum<L>(ss, mask);
          dot = group_sum<L>(dot, mask);
          const float r = rsqrtf(ss * (1.f / D) + p.eps);
          // (r^2 next to the sum: r^3 alone leaves the fp32 range for rows near 1e-13 when eps is 0)
          const float k = r * (r * (r * dot) * (1.f / D));
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            da[e] += ga[e] * (r * a[e]);
            db[e] += gb[e] * (r * bb[e]);
            a[e] = r * wa[e] * ga[e] - a[e] * k;
            bb[e] = r * wb[e] * gb[e] - bb[e] * k;
          }
          out = pack<T, HALVES>(a, bb);
        }
        store_row<D, HALVES>(dx, ch, out);
        dx += dx_step;
      }
    }
    tok = later;
    row = row_next;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      c[e] = cn[e];
      s[e] = sn[e];
    }
  }
  asm volatile("cp.async.wait_group 0;\n" ::: "memory");
  // lane groups in order, then one partial row per CTA
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int pr = 4 * ch + e;
    red[grp][HALVES ? pr : 2 * pr] = da[e];
    red[grp][HALVES ? pr + D / 2 : 2 * pr + 1] = db[e];
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float t = 0.f;
#pragma unroll
    for (int g = 0; g < G; ++g) t += red[g][threadIdx.x];
    p.part[(long long)blockIdx.x * D + threadIdx.x] = t;
  }
}

// dw[which][c] = sum of the partial rows of q (block 0) or k (block 1), in a fixed order.
template <int D>
__global__ void __launch_bounds__(1024) norm_rope_dw_kernel(const float* __restrict__ part, int ctas_q, int ctas,
                                                            float* dwq, float* dwk) {
  constexpr int G = 1024 / D;
  __shared__ float red[G][D];
  const int which = blockIdx.x, c = threadIdx.x % D, g = threadIdx.x / D;
  float* dw = which ? dwk : dwq;
  if (dw == nullptr) return;
  cudaGridDependencySynchronize();
  const int lo = which ? ctas_q : 0, hi = which ? ctas : ctas_q;
  float t = 0.f;
#pragma unroll 8
  for (int r = lo + g; r < hi; r += G) t += __ldcg(part + (long long)r * D + c);
  red[g][c] = t;
  __syncthreads();
  if (g == 0) {
    t = 0.f;
#pragma unroll
    for (int i = 0; i < G; ++i) t += red[i][c];
    dw[c] = t;
  }
}

// Heads per lane group: a token's tables and indices are then read once for
// that many rows.  One where the call is small and its time is one row's
// latency, else up to 16, in equal groups of whole loads.
int pick_hb(const NormRopeArgs& a, long long tokens, int d) {
  const long long groups = (long long)kNumSMs * (kThreads / (d / 8)) * 4;
  const int most = std::max(a.heads[0], a.heads[1]);
  int hb = 16;
  while (hb > 1 && tokens * ((a.heads[0] + hb - 1) / hb + (a.heads[1] + hb - 1) / hb) < groups) hb >>= 1;
  if (hb < kRowsInFlight) return hb;
  const int parts = (most + hb - 1) / hb, each = (most + parts - 1) / parts;
  return std::min(hb, (each + kRowsInFlight - 1) / kRowsInFlight * kRowsInFlight);
}

NormRope plan(const NormRopeArgs& a, long long tokens, int d) {
  NormRope p{a, {0, 0}, pick_hb(a, tokens, d)};
  for (int w = 0; w < 2; ++w) p.chunks[w] = (a.heads[w] + p.hb - 1) / p.hb;
  return p;
}

template <typename F>
void by_type(int d, int f16, int halves, bool turn, F&& f) {
  auto t = [&](auto D_) {
    auto u = [&](auto z) {
      auto v = [&](auto H_) {
        if (turn) f(D_, z, H_, std::true_type{});
        else f(D_, z, H_, std::false_type{});
      };
      if (halves) v(std::true_type{});
      else v(std::false_type{});
    };
    if (f16) u(__half{});
    else u(__nv_bfloat16{});
  };
  if (d == 128) t(std::integral_constant<int, 128>{});
  else t(std::integral_constant<int, 64>{});
}

// CTAs of q and k in the backward: as many as are resident, in proportion to
// the heads, the same number for each head group, none beyond the work.
void bwd_ctas(const NormRopeArgs& a, int d, int hb, int* cq, int* ck) {
  const int G = kThreads / (d / 8);
  const long long tiles = ((long long)a.B * a.N + G - 1) / G;
  const int total = kNumSMs * kBwdPerSM, heads = a.heads[0] + a.heads[1];
  for (int w = 0; w < 2; ++w) {
    const int chunks = (a.heads[w] + hb - 1) / hb;
    const long long share = chunks ? std::max(1LL, (long long)total * a.heads[w] / heads / chunks) : 0;
    *(w ? ck : cq) = (int)(chunks * std::min(tiles, share));
  }
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, int d, int f16, cudaStream_t st) {
  const long long tokens = (long long)a.B * a.rows;
  const NormRope p = plan(a, tokens, d);
  const int G = kThreads / (d / 8);
  const dim3 grid((unsigned)((tokens + G - 1) / G), (unsigned)(p.chunks[0] + p.chunks[1]));
  by_type(d, f16, a.halves, a.cos != nullptr, [&](auto D_, auto z, auto H_, auto R_) {
    norm_rope_kernel<decltype(D_)::value, decltype(z), decltype(H_)::value, decltype(R_)::value><<<grid, kThreads, 0, st>>>(p);
  });
  return cudaGetLastError();
}

size_t norm_rope_bwd_workspace_bytes(const NormRopeArgs& a, int d) {
  int cq = 0, ck = 0;
  bwd_ctas(a, d, pick_hb(a, (long long)a.B * a.N, d), &cq, &ck);
  return (size_t)(cq + ck) * d * sizeof(float);
}

cudaError_t launch_norm_rope_bwd(const NormRopeArgs& a, int d, int f16, float* dwq, float* dwk, cudaStream_t st) {
  const NormRope p = plan(a, (long long)a.B * a.N, d);
  int cq = 0, ck = 0;
  bwd_ctas(a, d, p.hb, &cq, &ck);
  cudaError_t e = cudaSuccess;
  by_type(d, f16, a.halves, a.cos != nullptr, [&](auto D_, auto z, auto H_, auto R_) {
    constexpr auto kernel = norm_rope_bwd_kernel<decltype(D_)::value, decltype(z), decltype(H_)::value, decltype(R_)::value>;
    e = allow_smem<kernel>(kBwdSmem);
    if (e != cudaSuccess) return;
    kernel<<<cq + ck, kThreads, kBwdSmem, st>>>(p, cq);
    e = cudaGetLastError();
  });
  if (e != cudaSuccess || (dwq == nullptr && dwk == nullptr)) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(1024);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const float* part = a.part;
  return d == 128 ? cudaLaunchKernelEx(&cfg, norm_rope_dw_kernel<128>, part, cq, cq + ck, dwq, dwk)
                  : cudaLaunchKernelEx(&cfg, norm_rope_dw_kernel<64>, part, cq, cq + ck, dwq, dwk);
}

cudaError_t rope_flags(unsigned int* v, cudaStream_t st) { return read_and_clear_flags(g_rope_flags, v, st); }

}  // namespace svsa
