// The 8-bit block cache: appending tokens, and choosing blocks for queries.
//
// cache_append_kernel  one CTA per (sequence, head, block that receives
//   tokens), keys and values apart.  amax of the new rows; the block's scale =
//   the larger of what it had and the smallest power of two that holds amax;
//   the codes of rows that were there are rounded again only when the scale
//   grew.  Then, for keys, the block's mean from the codes: all of them are
//   multiples of the code's last place (1 for int8, 2^-9 for e4m3) and the
//   column sums stay below 2^24 of those, so fp32 sums are exact and the mean
//   does not depend on their order.
//   Bound by HBM for long appends (4 bytes read and 2 written per key and
//   value pair, in 16- and 8-byte pieces), by launch latency for one token.
//
// cache_select_kernel  one cluster of CTAs per (sequence, query, key head).
//   score(block) = max over the group's query heads of q . mean(block), both
//   in 8 bits with power-of-two scales: an integer dot product below 2^21
//   times a power of two, exact in fp32, so that no list depends on the order
//   of a sum and equal scores are really equal (the lower index wins).  Each
//   CTA scores a range of blocks, a warp 32 of them at a time (d / 16 lanes
//   read a mean of d bytes together), and puts the sortable keys into the
//   first CTA's shared memory; that one finds the cap-th largest key by three
//   digits of 11, 11 and 10 bits and writes the list in ascending order.
#include <cooperative_groups.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "common.cuh"
#include "stream.cuh"

namespace cg = cooperative_groups;

namespace svsa {

static __device__ unsigned int g_cache_flags;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

template <typename T>
__device__ __forceinline__ void unpack8(uint4 v, float x[8]);
template <>
__device__ __forceinline__ void unpack8<__nv_bfloat16>(uint4 v, float x[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <typename T>
struct Pair2;
template <>
struct Pair2<__nv_bfloat16> { using type = __nv_bfloat162; };
template <>
struct Pair2<__half> { using type = __half2; };
template <>
__device__ __forceinline__ void unpack8<__half>(uint4 v, float x[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

// The int8 code of y, rounded to nearest even and saturated; NaN gives 0.
__device__ __forceinline__ uint32_t encode_i8(float y) {
  if (y != y) return 0u;
  return (uint32_t)__float2int_rn(fminf(fmaxf(y, -127.f), 127.f)) & 0xffu;
}

// max |x| of packed pairs, NaN and infinities kept.
__device__ __forceinline__ __nv_bfloat162 abs_max(__nv_bfloat162 m, uint32_t w) {
  w &= 0x7fff7fffu;
  return __hmax2_nan(m, *reinterpret_cast<const __nv_bfloat162*>(&w));
}
__device__ __forceinline__ __half2 abs_max(__half2 m, uint32_t w) {
  w &= 0x7fff7fffu;
  return __hmax2_nan(m, *reinterpret_cast<const __half2*>(&w));
}

// Eight codes of x * inv, |x * inv| within the codes.  For int8, adding 1.5 *
// 2^23 leaves the rounded value in the low byte (the product by a power of two
// is exact, so the one rounding is that of the sum).
template <bool I8>
__device__ __forceinline__ uint2 encode8(const float x[8], float inv) {
  uint32_t c[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (I8) {
      uint32_t v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = __float_as_uint(fmaf(x[4 * i + e], inv, 12582912.f));
      c[i] = __byte_perm(__byte_perm(v[0], v[1], 0x0040), __byte_perm(v[2], v[3], 0x0040), 0x5410);
    } else {
      float y[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[4 * i + e] = x[4 * i + e] * inv;
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * i], y[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * i + 2], y[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
      c[i] = lo | hi << 16;
    }
  }
  return make_uint2(c[0], c[1]);
}

template <bool I8>
__device__ __forceinline__ void decode8(uint2 code, float x[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w = i ? code.y : code.x;
    if constexpr (I8) {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[4 * i + e] = (float)(int8_t)(w >> (8 * e));
    } else {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * e)), __NV_E4M3);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r));
        x[4 * i + 2 * e] = f.x;
        x[4 * i + 2 * e + 1] = f.y;
      }
    }
  }
}

struct AppendArgs {
  CacheArgs c;
  const void* x[2];                // k, v
  long long stride[2][3];          // batch, head, token
  const int32_t* n_new;            // nullable
  int32_t* len_out;                // nullable
  int N, wide;                     // wide: blocks that N tokens can touch
};

// 128 threads, eight rows of d = 128 each: what a thread does once per block
// (indices, the maximum, the scale) weighs half of what it does with 256, 29.7
// against 36.0 us for 7800 tokens of two 12-head streams.
constexpr int kAppendThreads = 128;

template <int D, typename T, bool I8>
__global__ void __launch_bounds__(kAppendThreads, 7) cache_append_kernel(const __grid_constant__ AppendArgs p) {
  constexpr int L = D / 8;                 // lanes per row
  constexpr int R = kAppendThreads / L;    // rows per pass
  constexpr int P = kBlock / R;            // passes: 8 (d = 128) or 4 (d = 64)
  constexpr int W = kAppendThreads / 32;
  constexpr float kUnit = I8 ? 1.f : 1.f / 512.f;          // the codes' last place
  __shared__ float wmax[W], wtop[W];
  __shared__ float sums[R][D];
  const int ch = threadIdx.x % L, rl = threadIdx.x / L;
  unsigned id = blockIdx.x;
  const int w = (int)(id & 1u);            // keys or values
  id >>= 1;
  const int x = (int)(id % p.wide);
  id /= p.wide;
  const int h = (int)(id % p.c.heads), b = (int)(id / p.c.heads);

  const int room = p.c.max_blocks * kBlock;
  const int len0 = __ldg(p.c.len + b), new0 = p.n_new ? __ldg(p.n_new + b) : p.N;
  const int len = min(max(len0, 0), room);
  const int n_new = min(min(max(new0, 0), p.N), room - len);
  if (x == 0 && h == 0 && w == 0 && threadIdx.x == 0) {
    if (len != len0 || n_new != new0) atomicOr(&g_cache_flags, kFlagIndex);
    if (p.len_out) p.len_out[b] = len + n_new;
  }
  const int j = len / kBlock + x;                      // block of the sequence
  const int lo = max(len, j * kBlock), hi = min(len + n_new, (j + 1) * kBlock);
  if (lo >= hi) return;
  const int page = __ldg(p.c.table + (long long)b * p.c.max_blocks + j);
  if ((unsigned)page >= (unsigned)p.c.n_pages) {
    if (threadIdx.x == 0) atomicOr(&g_cache_flags, kFlagIndex);
    return;
  }
  const int had = lo - j * kBlock, end = hi - j * kBlock;   // rows [had, end) of the block are new
  const long long cell = (long long)page * p.c.heads + h;
  uint8_t* codes = static_cast<uint8_t*>(w ? p.c.v : p.c.k) + cell * (kBlock * D) + ch * 8;
  float* scale_at = (w ? p.c.v_scale : p.c.k_scale) + cell;
  const bool mean_too = w == 0 && p.c.mean != nullptr;

  // a new row's eight values, or an old row's eight codes
  uint4 raw[P];
  const char* src = static_cast<const char*>(p.x[w]) +
                    2 * ((long long)b * p.stride[w][0] + (long long)h * p.stride[w][1]) + ch * 16;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int r = rl + R * i;
    raw[i] = make_uint4(0u, 0u, 0u, 0u);
    if (r >= had && r < end) {
      raw[i] = *reinterpret_cast<const uint4*>(src + 2 * (long long)(j * kBlock + r - len) * p.stride[w][2]);
    } else if (r < had && mean_too) {
      const uint2 c = *reinterpret_cast<const uint2*>(codes + r * D);
      raw[i].x = c.x;
      raw[i].y = c.y;
    }
  }
  const float start = had > 0 ? *scale_at : 0.f;
  // max |x| of the new rows in their own type, exactly; where it is not finite
  // (rare), once more over the values that are
  float amax;
  {
    using T2 = typename Pair2<T>::type;
    const uint32_t zero = 0u;
    T2 m = *reinterpret_cast<const T2*>(&zero);
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (rl + R * i >= had) m = abs_max(abs_max(abs_max(abs_max(m, raw[i].x), raw[i].y), raw[i].z), raw[i].w);
    float v[8];
    unpack8<T>(make_uint4(*reinterpret_cast<uint32_t*>(&m), 0u, 0u, 0u), v);
    amax = v[0] != v[0] || v[1] != v[1] ? INFINITY : fmaxf(v[0], v[1]);
  }
  auto reduce = [&](float m) {
    m = warp_max(m);
    if (threadIdx.x % 32 == 0) wmax[threadIdx.x / 32] = m;
    __syncthreads();                                   // also: every thread has read the old scale
#pragma unroll
    for (int i = 0; i < W; ++i) m = fmaxf(m, wmax[i]);
    return m;
  };
  amax = reduce(amax);
  const bool odd = !(amax < INFINITY);                 // uniform over the CTA
  if (odd) {
    if (threadIdx.x == 0) atomicOr(&g_cache_flags, kFlagNotFinite);
    __syncthreads();
    amax = 0.f;
    for (int i = 0; i < P; ++i) {
      float v[8];
      unpack8<T>(raw[i], v);
      for (int e = 0; e < 8; ++e)
        if (rl + R * i >= had && fabsf(v[e]) < INFINITY) amax = fmaxf(amax, fabsf(v[e]));
    }
    amax = reduce(amax);
  }
  const float scale = fmaxf(start, pow2_scale(amax, I8));
  const float inv = scale > 0.f ? 1.f / scale : 0.f;
  if (threadIdx.x == 0) *scale_at = scale;
  const bool grew = had > 0 && scale != start;
  const float back = grew ? start / scale : 1.f;

  float total[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int r = rl + R * i;
    uint2* at = reinterpret_cast<uint2*>(codes + r * D);
    uint2 c;
    if (r >= end) continue;
    if (r >= had) {
      float v[8];
      unpack8<T>(raw[i], v);
      if (odd) {                                       // NaN gives 0, an infinity the largest code (0 under the scale 0)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (!(fabsf(v[e]) < INFINITY)) v[e] = v[e] != v[e] ? 0.f : copysignf((I8 ? 127.f : 448.f) * scale, v[e]);
      }
      c = encode8<I8>(v, inv);
      *at = c;
    } else {
      if (!grew && !mean_too) continue;
      c = mean_too ? make_uint2(raw[i].x, raw[i].y) : *at;
      if (grew) {
        float v[8];
        decode8<I8>(c, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = v[e] == v[e] ? v[e] : 0.f;
        c = encode8<I8>(v, back);
        *at = c;
      }
    }
    if (mean_too) {
      float v[8];
      decode8<I8>(c, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) total[e] += v[e];
    }
  }
  if (!mean_too) return;
  *reinterpret_cast<float4*>(&sums[rl][ch * 8]) = make_float4(total[0], total[1], total[2], total[3]);
  *reinterpret_cast<float4*>(&sums[rl][ch * 8 + 4]) = make_float4(total[4], total[5], total[6], total[7]);
  __syncthreads();
  float mean = 0.f;
  if (threadIdx.x < D) {
    float t = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) t += sums[r][threadIdx.x];
    mean = __fdiv_rn(t * (1.f / kUnit), (float)end);
  }
  const float m = warp_max(fabsf(mean));
  if (threadIdx.x % 32 == 0) wtop[threadIdx.x / 32] = m;
  __syncthreads();
  if (threadIdx.x < D) {
    float top = wtop[0];
#pragma unroll
    for (int i = 1; i < D / 32; ++i) top = fmaxf(top, wtop[i]);
    const float s = pow2_scale(top, true);
    p.c.mean[cell * D + threadIdx.x] = (int8_t)encode_i8(s > 0.f ? mean / s : 0.f);
    if (threadIdx.x == 0) p.c.mean_scale[cell] = s * kUnit * scale;
  }
}

// ---------------------------------------------------------------- selection

struct SelectArgs {
  CacheArgs c;
  const void* q;                   // [B][heads_q][Tq][d]
  int32_t* idx;                    // [B][Tq][heads][cap]
  int32_t* cnt;                    // [B][Tq][heads]
  int heads_q, Tq, causal, cap, first, last;
};

constexpr int kBins = 2048;

// Inclusive sums over the CTA's threads of two counts at once (each below 2^16).
__device__ __forceinline__ uint32_t scan_pairs(uint32_t v, uint32_t* warp_tot) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  if (lane == 31) warp_tot[warp] = v;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w)
    if (w < warp) v += warp_tot[w];
  return v;
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads, 5) cache_select_kernel(const __grid_constant__ SelectArgs p) {
  extern __shared__ __align__(16) uint32_t smem[];
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t warp_tot[2][kWarps];
  __shared__ int found[2];
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  // (arrive now, wait before the first write into another CTA's shared memory: it has started by then)
  if (C > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;\n" ::: "memory");
  const int group = p.heads_q / p.c.heads;
  uint32_t* qc = smem;                                     // [group][D / 4]
  float* qs = reinterpret_cast<float*>(qc + group * (D / 4));
  uint32_t* keys = smem + (group * (D / 4 + 1) + 3) / 4 * 4;          // [max_blocks], used in the first CTA

  long long row = blockIdx.x / C;
  const int h = (int)(row % p.c.heads);
  row /= p.c.heads;
  const int t = (int)(row % p.Tq), b = (int)(row / p.Tq);
  const long long out_row = ((long long)b * p.Tq + t) * p.c.heads + h;
  int32_t* idx = p.idx + out_row * p.cap;

  const int len0 = __ldg(p.c.len + b);
  // the group's queries in 8 bits, a warp each
  for (int g = threadIdx.x / 32; g < group; g += kWarps) {
    const int lane = threadIdx.x % 32;
    const char* q = static_cast<const char*>(p.q) + (((long long)b * p.heads_q + h * group + g) * p.Tq + t) * (2LL * D);
    float v[D / 32];
    if constexpr (D == 128) {
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(q) + lane);
      float x[8];
      unpack8<T>(make_uint4(w.x, w.y, 0u, 0u), x);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = x[e];
    } else {
      const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(q) + lane);
      float x[8];
      unpack8<T>(make_uint4(w, 0u, 0u, 0u), x);
      v[0] = x[0];
      v[1] = x[1];
    }
    float amax = 0.f;
    bool odd = false;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) {
      const float a = fabsf(v[e]);
      if (a < INFINITY) amax = fmaxf(amax, a);
      else odd = true;
    }
    if (odd) atomicOr(&g_cache_flags, kFlagNotFinite);
    const float s = pow2_scale(warp_max(amax), true), inv = s > 0.f ? 1.f / s : 0.f;
    uint32_t w = 0u;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) w |= encode_i8(v[e] * inv) << (8 * e);
    if constexpr (D == 128) qc[g * (D / 4) + lane] = w;
    else reinterpret_cast<uint16_t*>(qc + g * (D / 4))[lane] = (uint16_t)w;
    if (lane == 0) qs[g] = s;
  }
  for (int i = threadIdx.x; i < kBins; i += kThreads) hist[i] = 0u;

  const int len = min(max(len0, 0), p.c.max_blocks * kBlock);
  const int seen = p.causal ? max(len - p.Tq + 1 + t, 0) : len;
  const int nb = (seen + kBlock - 1) / kBlock;
  if (rank == 0 && threadIdx.x == 0) {
    p.cnt[out_row] = min(nb, p.cap);
    if (len != len0) atomicOr(&g_cache_flags, kFlagIndex);
  }
  if (nb <= p.cap) {                                       // nothing to choose (uniform over the cluster)
    for (int i = rank * kThreads + threadIdx.x; i < p.cap; i += C * kThreads) idx[i] = i < nb ? i : 0;
    if (C > 1) asm volatile("barrier.cluster.wait.aligned;\n" ::: "memory");
    return;
  }
  __syncthreads();
  if (C > 1) asm volatile("barrier.cluster.wait.aligned;\n" ::: "memory");
  uint32_t* to = C > 1 ? cluster.map_shared_rank(keys, 0) : keys;
  // A warp scores 32 blocks at a time, one per lane in the end; D / 16 lanes
  // read a mean together (whole lines), each a 16-byte piece of as many
  // blocks, and an exchange in halves leaves every lane its block's sum.
  constexpr int L = D / 16;
  const int lane = threadIdx.x % 32, e = lane % L;
  bool bad = false;
  const int32_t* pages = p.c.table + (long long)b * p.c.max_blocks;
  const int step = C * kThreads;
  int j = rank * kThreads + threadIdx.x;
  int page = j < nb ? __ldg(pages + j) : 0;
  for (; j - lane < nb; j += step) {                        // uniform over the warp
    const int next = j + step < nb ? __ldg(pages + j + step) : 0;
    const bool forced = j < p.first || j >= nb - p.last;
    const bool ok = j < nb && (unsigned)page < (unsigned)p.c.n_pages;
    const int cell = ok ? page * p.c.heads + h : h;         // (page 0 in the place of one that is not there)
    const float ms = __ldg(p.c.mean_scale + cell);
    uint4 m[L];
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const int c = __shfl_sync(0xffffffffu, cell, lane - e + i);
      m[i] = __ldg(reinterpret_cast<const uint4*>(p.c.mean + (long long)c * D) + e);
    }
    float best = -INFINITY;
    for (int g = 0; g < group; ++g) {
      const uint4 a = reinterpret_cast<const uint4*>(qc + g * (D / 4))[e];
      int dot[L];
#pragma unroll
      for (int i = 0; i < L; ++i) {
        dot[i] = __dp4a((int)a.x, (int)m[i].x, 0);
        dot[i] = __dp4a((int)a.y, (int)m[i].y, dot[i]);
        dot[i] = __dp4a((int)a.z, (int)m[i].z, dot[i]);
        dot[i] = __dp4a((int)a.w, (int)m[i].w, dot[i]);
      }
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) {
        const bool up = e & o;
#pragma unroll
        for (int i = 0; i < o; ++i) {
          const int give = up ? dot[i] : dot[i + o], keep = up ? dot[i + o] : dot[i];
          dot[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
      }
      best = fmaxf(best, (float)dot[0] * (qs[g] * ms));
    }
    if (j < nb) {
      const uint32_t u = __float_as_uint(best + 0.f);       // -0 becomes +0
      bad = bad || (!ok && !forced);
      to[j] = forced ? 0xffffffffu : !ok ? 0u : (u & 0x80000000u) ? ~u : u | 0x80000000u;
    }
    page = next;
  }
  if (bad) atomicOr(&g_cache_flags, kFlagIndex);
  if (C > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");
    if (rank != 0) return;
    asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
  } else {
    __syncthreads();
  }

  // the cap-th largest key, digit by digit
  uint32_t prefix = 0u;
  int need = p.cap;
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, above = pass == 0 ? 0 : pass == 1 ? 21 : 10;
    const uint32_t mask = pass == 2 ? 1023u : 2047u;
    for (int i = threadIdx.x; i < nb; i += kThreads) {
      const uint32_t key = keys[i];
      if (pass == 0 || (key >> above) == (prefix >> above)) atomicAdd(&hist[(key >> shift) & mask], 1u);
    }
    __syncthreads();
    // thread i holds the eight bins below 2048 - 8 i; the scan counts the keys from the top
    uint32_t c[8], sum = 0u;
    uint4* mine = reinterpret_cast<uint4*>(hist + kBins - 8 - 8 * threadIdx.x);
    const uint4 lo = mine[0], hi = mine[1];
    c[0] = hi.w; c[1] = hi.z; c[2] = hi.y; c[3] = hi.x;
    c[4] = lo.w; c[5] = lo.z; c[6] = lo.y; c[7] = lo.x;
    mine[0] = mine[1] = make_uint4(0u, 0u, 0u, 0u);         // clear for the next digit
#pragma unroll
    for (int e = 0; e < 8; ++e) sum += c[e];
    uint32_t up = scan_pairs(sum, warp_tot[pass & 1]);
    if (up >= (uint32_t)need && up - sum < (uint32_t)need) {
      int at = (int)(up - sum);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (at < need && at + (int)c[e] >= need) {
          found[0] = kBins - 1 - 8 * (int)threadIdx.x - e;
          found[1] = need - at;
        }
        at += (int)c[e];
      }
    }
    __syncthreads();
    prefix |= (uint32_t)found[0] << shift;
    need = found[1];
  }

  // the keys above it, and the first `need` equal to it, in order; a thread
  // takes consecutive keys (an odd number: no bank conflicts)
  const int per = ((nb + kThreads - 1) / kThreads) | 1;
  const int lo = min((int)threadIdx.x * per, nb), hi = min(lo + per, nb);
  uint32_t mine = 0u;                                       // equal << 16 | above
  for (int i = lo; i < hi; ++i) mine += keys[i] > prefix ? 1u : keys[i] == prefix ? 0x10000u : 0u;
  const uint32_t upto = scan_pairs(mine, warp_tot[1]) - mine;
  int gt = (int)(upto & 0xffffu), eq = (int)(upto >> 16);
  for (int i = lo; i < hi; ++i) {
    const uint32_t key = keys[i];
    if (key > prefix || (key == prefix && eq < need)) idx[gt + min(eq, need)] = i;
    gt += key > prefix;
    eq += key == prefix;
  }
}

template <typename F>
void by_d_type(int d, int f16, F&& f) {
  auto t = [&](auto D_) {
    if (f16) f(D_, __half{});
    else f(D_, __nv_bfloat16{});
  };
  if (d == 128) t(std::integral_constant<int, 128>{});
  else t(std::integral_constant<int, 64>{});
}

}  // namespace

cudaError_t launch_cache_append(const CacheArgs& c, const void* k, const void* v, const long long k_stride[3],
                                const long long v_stride[3], const int32_t* n_new, int32_t* len_out, int N, int f16,
                                cudaStream_t st) {
  AppendArgs p{};
  p.c = c;
  p.x[0] = k;
  p.x[1] = v;
  for (int e = 0; e < 3; ++e) {
    p.stride[0][e] = k_stride[e];
    p.stride[1][e] = v_stride[e];
  }
  p.n_new = n_new;
  p.len_out = len_out;
  p.N = N;
  // N tokens touch at most ceil((N - 1) / 64) + 1 blocks, wherever they start
  p.wide = N / kBlock + (N % kBlock > 1) + 1;
  const unsigned grid = (unsigned)((long long)p.wide * c.heads * c.B * 2);
  by_d_type(c.d, f16, [&](auto D_, auto z) {
    constexpr int D = decltype(D_)::value;
    using T = decltype(z);
    if (c.i8) cache_append_kernel<D, T, true><<<grid, kAppendThreads, 0, st>>>(p);
    else cache_append_kernel<D, T, false><<<grid, kAppendThreads, 0, st>>>(p);
  });
  return cudaGetLastError();
}

cudaError_t launch_cache_select(const CacheArgs& c, const void* q, int heads_q, int Tq, int f16, int causal, int cap,
                                int first, int last, int32_t* idx, int32_t* cnt, cudaStream_t st) {
  SelectArgs p{};
  p.c = c;
  p.q = q;
  p.idx = idx;
  p.cnt = cnt;
  p.heads_q = heads_q;
  p.Tq = Tq;
  p.causal = causal;
  p.cap = cap;
  p.first = first;
  p.last = last;
  const long long rows = (long long)c.B * Tq * c.heads;
  // CTAs per row: more while a CTA keeps at least one block per thread and the
  // grid stays within a few CTAs per SM
  int C = 1;
  while (C < 8 && c.max_blocks > C * kThreads && rows * C < kNumSMs * 4) C *= 2;
  const int group = heads_q / c.heads;
  const size_t smem = ((size_t)(group * (c.d / 4 + 1) + 3) / 4 * 4 + c.max_blocks) * 4;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(rows * C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)C;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cudaError_t e = cudaSuccess;
  by_d_type(c.d, f16, [&](auto D_, auto z) {
    constexpr auto kernel = cache_select_kernel<decltype(D_)::value, decltype(z)>;
    // (the most that a call can ask for: the keys of 32768 blocks, 128 heads)
    if (smem > 32768) e = allow_smem<kernel>(32768 * 4 + 128 * 132 + 16);
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, kernel, p);
  });
  return e;
}

cudaError_t cache_flags(unsigned int* v, cudaStream_t st) { return read_and_clear_flags(g_cache_flags, v, st); }

}  // namespace svsa
