// Writing, reading and thinning out the 4-bit key/value cache.
//
//  kv_rows_kernel   : bf16 K and V rows -> NVFP4 (16-channel blocks, E4M3
//                     scale, E2M1 codes) at their slots in the pages, and the
//                     reverse, exact in bf16 (a stored value has at most 6
//                     significant bits); a few rows per sequence
//  kv_pages_kernel  : the same for many rows, a page at a time
//  kv_select_kernel : which slots of a (sequence, KV head) stay: the first,
//                     the last, and the heaviest of the rest
//  kv_move_kernel   : the rows of the kept slots, bit for bit, to new pages
#include <cmath>

#include "kvcache.cuh"

namespace fp4attn {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint4 ld_once(const void* ptr) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(ptr));
  return v;
}

// Eight channels of bf16 -> their 4 code bytes, and the block's scale byte; the
// block's other eight channels are with lane ^ 1.  down is 2^-exp, sixth is
// 2^-exp / 6.  A NaN counts as 0; an infinity saturates (scale 448, code 6).
// Every decision is the exact one, with reciprocals in place of divisions: the
// exact quotient amax / 6 or x / s is either on a boundary of the format (a few
// bits) or 2^-8 of its size away from the next (x has 8 significant bits, 6 and
// s have at most 4), and the computed one is off by less than 2^-21 of itself.
// Rounded to 16 bits (amax / 6) or to fp16's 11 (x / s) it returns to the
// boundary it belongs on and crosses none.
__device__ __forceinline__ uint32_t quant_half(uint4 v, float down, float sixth, uint32_t& scale_byte) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
  auto largest = [&]() {
    uint32_t m2 = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                           __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
    m2 = __vmaxu2(m2, __shfl_xor_sync(0xFFFFFFFFu, m2, 1));
    return max(m2 & 0xFFFFu, m2 >> 16);
  };
  uint32_t m = largest();
  if (__any_sync(0xFFFFFFFFu, m > 0x7F80u)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] &= ~__vcmpgtu2(w[i] & 0x7FFF7FFFu, 0x7F807F80u);
    m = largest();
  }
  const float a6 = __fmul_rn(__uint_as_float(m << 16), sixth);
  scale_byte = cvt_e4m3(__uint_as_float((__float_as_uint(a6) + 0x40u) & 0xFFFFFF80u));
  const uint32_t s2 = e4m3x2_to_half2(scale_byte);
  const float s = __low2float(*reinterpret_cast<const __half2*>(&s2));
  const float inv = __fdividef(down, s);
  uint32_t y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    fmul2(a, b, __uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u), inv, inv);
    const __half2 h = __floats2half2_rn(a, b);
    y[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return s == 0.0f ? 0u : half2x4_to_e2m1x8(y);  // a block whose scale is 0 holds zeros
}

// 4 code bytes and a scale -> 8 bf16 values.  The product of code and scale is
// exact in fp16; 2^exp moves its exponent, and bf16 holds its 6 bits.
__device__ __forceinline__ uint4 decode_half(uint32_t c, uint32_t scale_byte, float up) {
  const uint32_t s = splat_lo(e4m3x2_to_half2(scale_byte));
  uint32_t h[4], o[4];
  e2m1x8_to_half2(c, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t m = hmul2(h[i], s);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&m));
    const __nv_bfloat162 r = __floats2bfloat162_rn(f.x * up, f.y * up);
    o[i] = *reinterpret_cast<const uint32_t*>(&r);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

struct RowsParams {
  KvGeom g;
  uint8_t* pages;
  const __nv_bfloat16 *k, *v;              // append: rows in
  long long k_row, k_head, v_row, v_head;  // strides in elements
  __nv_bfloat16 *ko, *vo;                  // read: rows out [T, heads, D]
  float k_scale, v_scale;                  // append: 2^-exp, read: 2^exp
  float k_sixth, v_sixth;                  // append: 2^-exp / 6
};

// Row offsets that descend or lie outside the tensors: a search for a row's (or
// a page's) sequence may never come to those, so each is looked at, by thread i
// of `all`; the first one's offsets are fetched before the search.
struct OffsetCheck {
  int i, all, from, to;
  __device__ __forceinline__ OffsetCheck(const KvGeom& g, int i_, int all_) : i(i_), all(all_), from(0), to(0) {
    if (g.cu && i < g.B) {
      from = g.cu[i];
      to = g.cu[i + 1];
    }
  }
  __device__ __forceinline__ void report(const KvGeom& g) {
    bool bad = from < 0 || to < from || to > g.T;
    if (g.cu)
      for (i += all; i < g.B; i += all) bad |= g.cu[i] < 0 || g.cu[i + 1] < g.cu[i] || g.cu[i + 1] > g.T;
    if (bad) report_bad_index(g.status);
  }
};

// Few rows per sequence: D / 8 lanes per row and head, every part stored where
// it belongs.  What counts is the chain of dependent loads: 2 us for 8 sequences
// of one row as for 32 of 8.
template <int D, bool READ>
__global__ void __launch_bounds__(kThreads) kv_rows_kernel(const RowsParams p) {
  using P = PageLayout<D>;
  constexpr int kLanes = D / 8;
  const int item = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes, q = threadIdx.x % kLanes;
  const int h = item % p.g.heads, r = item / p.g.heads;
  const bool in = r < p.g.T;
  chain_start();
  uint4 k{}, v{};
  if (!READ && in) {
    k = ld_once(p.k + r * p.k_row + h * p.k_head + q * 8);
    v = ld_once(p.v + r * p.v_row + h * p.v_head + q * 8);
  }
  int b, slot, pg = -1;
  OffsetCheck check(p.g, blockIdx.x * kThreads + threadIdx.x, gridDim.x * kThreads);
  if (in && row_slot(p.g, r, b, slot)) pg = page_of(p.g, b, slot / kPage);
  check.report(p.g);
  // lanes of a row agree on pg; all lanes reach the shuffles
  const int t = pg >= 0 ? slot & (kPage - 1) : 0;
  uint8_t* page = p.pages + (static_cast<long long>(pg) * p.g.heads + h) * P::kBytes;
  if constexpr (READ) {
    if (pg < 0) return;
    const long long at = (static_cast<long long>(r) * p.g.heads + h) * D + q * 8;
    const uint32_t kc = *reinterpret_cast<const uint32_t*>(page + P::k_code(t, 0) + 4 * q);
    const uint32_t vc = *reinterpret_cast<const uint32_t*>(page + P::v_half(t, q));
    const uint32_t ks = page[P::k_scale(t, q >> 1)], vs = page[P::v_scale(t, q >> 1)];
    *reinterpret_cast<uint4*>(p.ko + at) = decode_half(kc, ks, p.k_scale);
    *reinterpret_cast<uint4*>(p.vo + at) = decode_half(vc, vs, p.v_scale);
  } else {
    uint32_t ks, vs;
    const uint32_t kc = quant_half(k, p.k_scale, p.k_sixth, ks), vc = quant_half(v, p.v_scale, p.v_sixth, vs);
    if (pg < 0) return;
    *reinterpret_cast<uint32_t*>(page + P::k_code(t, 0) + 4 * q) = kc;
    *reinterpret_cast<uint32_t*>(page + P::v_half(t, q)) = vc;
    if (!(q & 1)) {
      page[P::k_scale(t, q >> 1)] = static_cast<uint8_t>(ks);
      page[P::v_scale(t, q >> 1)] = static_cast<uint8_t>(vs);
    }
  }
}

// Many rows per sequence: a CTA per page that holds new rows, for kHeads KV
// heads in turn, K and V of each.  A half page (K or V) that is new as a whole
// is put together in shared memory and stored as 36 D contiguous bytes (single
// parts would reach memory as byte- and word-sized pieces of 26 sectors per
// token); one that is not is written part by part.  Reading is the reverse.
// Bound by memory: 16-byte loads and stores whose lanes cover whole rows, and
// the next half page's loads are in flight while one is converted.  38000 rows of
// 8 KV heads, D = 128: append 40 us, 5.0 TB/s; read 32 us, 6.2 TB/s.
//
// CTA x finds its page without a scan: sequence b's pages start at number
// cu[b] / 64 + 2 b.  Between two sequences there are then at least
// floor(n / 64) + 2 numbers, and n rows touch at most floor((n - 1) / 64) + 2.
template <int D, bool READ>
__global__ void __launch_bounds__(kThreads) kv_pages_kernel(const RowsParams p) {
  using P = PageLayout<D>;
  constexpr int kLanes = D / 8, kRows = kThreads / kLanes, kSteps = kPage / kRows;
  constexpr int kVecs = P::kKBytes / 16, kVecSteps = (kVecs + kThreads - 1) / kThreads;
  __shared__ __align__(16) uint8_t buf[2][P::kKBytes];
  const int x = blockIdx.x;
  chain_start();
  if (p.g.cu && blockIdx.y == 0 && x * kThreads < p.g.B)
    OffsetCheck(p.g, x * kThreads + threadIdx.x, gridDim.x * kThreads).report(p.g);
  const int per = p.g.cu ? 0 : p.g.T / p.g.B;
  auto base = [&](int b) { return (p.g.cu ? max(p.g.cu[b], 0) : b * per) / kPage + 2 * b; };
  int lo = 0, hi = p.g.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (base(mid) <= x) lo = mid; else hi = mid;
  }
  int row0, n, L;
  if (!seq_of(p.g, lo, row0, n, L)) {
    if (threadIdx.x == 0) report_bad_index(p.g.status);
    return;
  }
  if (n == 0 || x < base(lo)) return;
  const int first = L - n;  // slot of the first new row
  if (first < 0 && x == base(lo) && threadIdx.x == 0) report_bad_index(p.g.status);
  const int s0 = max(first, 0);
  const int pi = s0 / kPage + (x - base(lo));
  if (pi * kPage >= L) return;
  const int pg = page_of(p.g, lo, pi);
  if (pg < 0) return;
  uint8_t* pages = p.pages + static_cast<long long>(pg) * p.g.heads * P::kBytes;
  const int q = threadIdx.x % kLanes, tr = threadIdx.x / kLanes;
  const int t_lo = max(s0 - pi * kPage, 0), t_hi = min(L - pi * kPage, kPage);  // rows of the page that are new
  const long long rbase = static_cast<long long>(row0) + (pi * kPage - first);  // packed row of the page's row 0
  // half page i: K (even) or V (odd) of head blockIdx.y + i / 2 * gridDim.y
  const int halves = 2 * ((p.g.heads - 1 - static_cast<int>(blockIdx.y)) / static_cast<int>(gridDim.y) + 1);
  auto head_of = [&](int i) { return static_cast<int>(blockIdx.y) + (i >> 1) * static_cast<int>(gridDim.y); };
  auto half_at = [&](int i) { return pages + static_cast<long long>(head_of(i)) * P::kBytes + (i & 1 ? P::kKBytes : 0); };
  // offsets within a half page
  auto code_at = [&](int i, int t) { return i & 1 ? P::v_half(t, q) - P::kVc : P::k_code(t, 0) + 4 * q; };
  auto scale_at = [&](int i, int t) { return i & 1 ? P::v_scale(t, q >> 1) - P::kVc : P::k_scale(t, q >> 1); };
  if constexpr (READ) {
    uint4 r[kVecSteps];
    auto load = [&](int i) {
#pragma unroll
      for (int j = 0; j < kVecSteps; ++j) {
        const int e = j * kThreads + threadIdx.x;
        if (e < kVecs) r[j] = *reinterpret_cast<const uint4*>(half_at(i) + 16 * e);
      }
    };
    load(0);
    for (int i = 0; i < halves; ++i) {
      uint8_t* b = buf[i & 1];
#pragma unroll
      for (int j = 0; j < kVecSteps; ++j) {
        const int e = j * kThreads + threadIdx.x;
        if (e < kVecs) reinterpret_cast<uint4*>(b)[e] = r[j];
      }
      if (i + 1 < halves) load(i + 1);
      __syncthreads();
      __nv_bfloat16* out = i & 1 ? p.vo : p.ko;
      const float up = i & 1 ? p.v_scale : p.k_scale;
#pragma unroll
      for (int j = 0; j < kSteps; ++j) {
        const int t = j * kRows + tr;
        if (t < t_lo || t >= t_hi) continue;
        __stcs(reinterpret_cast<uint4*>(out + ((rbase + t) * p.g.heads + head_of(i)) * D + q * 8),
               decode_half(*reinterpret_cast<const uint32_t*>(b + code_at(i, t)), b[scale_at(i, t)], up));
      }
    }
  } else {
    uint4 r[kSteps];
    auto load = [&](int i) {
      const __nv_bfloat16* src = (i & 1 ? p.v : p.k) + head_of(i) * (i & 1 ? p.v_head : p.k_head) + q * 8;
      const long long row = i & 1 ? p.v_row : p.k_row;
#pragma unroll
      for (int j = 0; j < kSteps; ++j) {
        const int t = j * kRows + tr;
        r[j] = make_uint4(0u, 0u, 0u, 0u);
        if (t >= t_lo && t < t_hi) r[j] = ld_once(src + (rbase + t) * row);
      }
    };
    const bool whole = t_lo == 0 && t_hi == kPage;
    load(0);
    for (int i = 0; i < halves; ++i) {
      uint4 v[kSteps];
#pragma unroll
      for (int j = 0; j < kSteps; ++j) v[j] = r[j];
      if (i + 1 < halves) load(i + 1);
      uint8_t* to = whole ? buf[i & 1] : half_at(i);
#pragma unroll
      for (int j = 0; j < kSteps; ++j) {
        const int t = j * kRows + tr;
        uint32_t sb;
        const uint32_t c = quant_half(v[j], i & 1 ? p.v_scale : p.k_scale, i & 1 ? p.v_sixth : p.k_sixth, sb);
        if (t < t_lo || t >= t_hi) continue;
        *reinterpret_cast<uint32_t*>(to + code_at(i, t)) = c;
        if (!(q & 1)) to[scale_at(i, t)] = static_cast<uint8_t>(sb);
      }
      if (whole) {
        __syncthreads();
        for (int e = threadIdx.x; e < kVecs; e += kThreads)
          *reinterpret_cast<uint4*>(half_at(i) + 16 * e) = reinterpret_cast<const uint4*>(buf[i & 1])[e];
      }
    }
  }
}

// 8 code bytes of V's block b of token t: contiguous for D = 128, two chunks for D = 64.
template <int D>
__device__ __forceinline__ void st_v_codes(uint8_t* page, int t, int b, uint2 c) {
  *reinterpret_cast<uint32_t*>(page + PageLayout<D>::v_half(t, 2 * b)) = c.x;
  *reinterpret_cast<uint32_t*>(page + PageLayout<D>::v_half(t, 2 * b + 1)) = c.y;
}
template <int D>
__device__ __forceinline__ uint2 ld_v_codes(const uint8_t* page, int t, int b) {
  return make_uint2(*reinterpret_cast<const uint32_t*>(page + PageLayout<D>::v_half(t, 2 * b)),
                    *reinterpret_cast<const uint32_t*>(page + PageLayout<D>::v_half(t, 2 * b + 1)));
}

// ---- eviction ---------------------------------------------------------------

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelCtas = 4;          // of the cluster that takes one problem
constexpr int kSelSmem = 40 * 1024;  // slots per CTA whose keys are held in shared memory
constexpr int kBins = 2048;

struct EvictParams {
  KvGeom g;
  uint8_t* pages;
  const float* w;  // [B, heads, W]
  int W;
  const int32_t* new_table;  // [B, new_M]
  int new_M;
  int keep, sinks, recent;
  int32_t* kept;      // [B, heads, keep]
  int32_t* new_lens;  // [B]
  float* new_w;       // [B, heads, W]
};

// Weights as unsigned keys that order as the numbers do; -0 equals 0, a NaN is
// below everything.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// The reverse (a zero comes back as +0, a NaN as one).
__device__ __forceinline__ float key_weight(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

// Length of sequence b as eviction sees it.
__device__ __forceinline__ int evict_len(const EvictParams& p, int b) {
  int L = p.g.lens[b];
  if (L < 0 || L > p.g.M * kPage || L > p.W) {
    if (threadIdx.x == 0) report_bad_index(p.g.status);
    L = 0;
  }
  return L;
}

// A cluster of four CTAs per (sequence, KV head), each with a quarter of the
// slots.  The keep largest keys are found by radix selection, the protected
// slots holding a key above all: three passes over the keys, each a 2048-bin
// histogram of the next 11 (11, 10) key bits of the slots that still match the
// prefix, added up over the cluster, fix the smallest kept key and how many of
// the slots that hold exactly it stay (the lowest ones).  11 bits hold three
// bits of the mantissa, which spreads weights of similar size over bins; zeros,
// which are many, are counted per thread and not by atomics on one bin, the
// protected slots not at all.  The keys are read from memory once where they
// fit in shared memory (KEYS), otherwise in every pass; a thread takes four at
// a time.  A last pass writes the kept slots in order: each warp owns a run of
// slots, a scan over the lanes' counts gives the positions.  What bounds it is
// the work per key and the chain of passes, not memory: 8 problems of 4096 slots
// take 11 us, 128 of up to 32768 take 29.
template <bool KEYS>
__global__ void __launch_bounds__(kSelThreads) kv_select_kernel(const EvictParams p) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ __align__(16) int hist[3][kBins];
  __shared__ int warp_sum[kSelWarps], cnt_hi[kSelWarps], cnt_eq[kSelWarps], total[2];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int rank = cluster_rank();
  const int h = blockIdx.x / kSelCtas, b = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < 3 * kBins / 4; i += kSelThreads) reinterpret_cast<int4*>(hist)[i] = make_int4(0, 0, 0, 0);
  const int L = evict_len(p, b);
  const long long row = static_cast<long long>(b) * p.g.heads + h;
  const float* w = p.w + row * p.W;
  int32_t* kept = p.kept + row * p.keep;
  float* nw = p.new_w + row * p.W;
  const int n = min(L, p.keep), all_tid = rank * kSelThreads + tid;
  if (h == 0 && all_tid == 0) p.new_lens[b] = n;
  for (int i = n + all_tid; i < p.keep; i += kSelCtas * kSelThreads) kept[i] = -1;
  if (L <= p.keep) {
    for (int i = all_tid; i < p.W; i += kSelCtas * kSelThreads) {
      if (i < n) kept[i] = i;
      nw[i] = i < n ? w[i] : 0.0f;
    }
    return;  // (the whole cluster)
  }
  constexpr uint32_t kSafe = 0xFFFFFFFFu;  // above the key of +inf
  const uint32_t zero = weight_key(0.0f);
  const int lo = p.sinks, hi = L - p.recent;  // the unprotected slots
  // this CTA's slots, a multiple of four but for the last
  const int share = ((L + kSelCtas - 1) / kSelCtas + 3) & ~3;
  const int c0 = min(L, rank * share), cnt = min(L, c0 + share) - c0, fours = (cnt + 3) >> 2;
  // Key of the CTA's slot i; behind its last one the lowest key, which is not
  // reached: L > keep, and of equal keys the lowest slots stay (only the last
  // CTA's can be incomplete).
  auto key_of = [&](int i, float x) {
    const int s = c0 + i;
    return i >= cnt ? 0u : s < lo || s >= hi ? kSafe : weight_key(x);
  };
  auto weight = [&](int i) { return w[c0 + min(i, cnt - 1)]; };
  auto four = [&](int v) {
    if constexpr (KEYS) return reinterpret_cast<const uint4*>(keys)[v];
    else
      return make_uint4(key_of(4 * v, weight(4 * v)), key_of(4 * v + 1, weight(4 * v + 1)),
                        key_of(4 * v + 2, weight(4 * v + 2)), key_of(4 * v + 3, weight(4 * v + 3)));
  };
  __syncthreads();
  if constexpr (KEYS) {
    for (int i = tid; i < 4 * fours; i += 4 * kSelThreads) {
      float x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = weight(i + j * kSelThreads);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j * kSelThreads < 4 * fours) keys[i + j * kSelThreads] = key_of(i + j * kSelThreads, x[j]);
    }
    __syncthreads();
  }
  int need = p.keep;
  uint32_t prefix = 0, mask = 0;
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t digit = pass == 2 ? 1023u : 2047u;
    int* hp = hist[pass];
    int zeros = 0;
#pragma unroll 2
    for (int v = tid; v < fours; v += kSelThreads) {
      const uint4 k4 = four(v);
      const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
      const bool m[4] = {(k[0] & mask) == prefix, (k[1] & mask) == prefix, (k[2] & mask) == prefix, (k[3] & mask) == prefix};
      if (!(m[0] || m[1] || m[2] || m[3])) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (k[j] == zero) zeros += m[j];
        else if (m[j] && k[j] != kSafe) atomicAdd(&hp[(k[j] >> shift) & digit], 1);
      }
    }
    zeros = __reduce_add_sync(0xFFFFFFFFu, zeros);
    if (lane == 0 && zeros) atomicAdd(&hp[(zero >> shift) & digit], zeros);
    if (all_tid == 0 && (kSafe & mask) == prefix) atomicAdd(&hp[digit], p.sinks + p.recent);
    cluster_sync();
    if (pass == 0)  // behind the kept ones (written while the others' bins travel)
      for (int i = n + all_tid; i < p.W; i += kSelCtas * kSelThreads) nw[i] = 0.0f;
    // from the top: the bin in which the need-th key lies; kEach bins per
    // thread, added up over the cluster (every CTA does it for itself)
    constexpr int kEach = kBins / kSelThreads;
    const int top = kBins - kEach * (tid + 1);  // the thread's lowest bin
    int c[kEach], mine = 0;                     // from its highest on
#pragma unroll
    for (int j = 0; j < kEach; ++j) c[j] = 0;
#pragma unroll
    for (int r = 0; r < kSelCtas; ++r)
#pragma unroll
      for (int j = 0; j < kEach; j += 4) {
        const uint4 x = cluster_ld4(cluster_map(smem_u32(hp + top + kEach - 4 - j), r));
        c[j] += x.w; c[j + 1] += x.z; c[j + 2] += x.y; c[j + 3] += x.x;
      }
#pragma unroll
    for (int j = 0; j < kEach; ++j) mine += c[j];
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int before = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? warp_sum[lane] : 0) + incl - mine;
    if (before < need && need <= before + mine) {
      int at = 0;
      bool found = false;
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        found |= need <= before + c[j];
        if (!found) {
          before += c[j];
          ++at;
        }
      }
      s_prefix = prefix | (static_cast<uint32_t>(top + kEach - 1 - at) << shift);
      s_need = need - before;
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
    mask |= digit << shift;
  }
  // prefix is now the smallest kept key, need how many slots that hold it stay
  const int run = (fours + kSelThreads - 1) / kSelThreads * 32;  // in fours, of a warp
  const int v0 = min(fours, warp * run), v1 = min(fours, v0 + run);
  // of a lane's four: larger keys, and equal ones in the upper half
  auto count = [&](const uint4& k) {
    return (k.x > prefix) + (k.y > prefix) + (k.z > prefix) + (k.w > prefix) +
           (((k.x == prefix) + (k.y == prefix) + (k.z == prefix) + (k.w == prefix)) << 16);
  };
  int nhi = 0, neq = 0;
#pragma unroll 2
  for (int v = v0 + lane; v < v1; v += 32) {
    const int c = count(four(v));
    nhi += c & 0xFFFF;
    neq += c >> 16;
  }
  nhi = __reduce_add_sync(0xFFFFFFFFu, nhi);
  neq = __reduce_add_sync(0xFFFFFFFFu, neq);
  if (lane == 0) {
    cnt_hi[warp] = nhi;
    cnt_eq[warp] = neq;
  }
  __syncthreads();
  if (warp == 0) {
    const int sh = __reduce_add_sync(0xFFFFFFFFu, lane < kSelWarps ? cnt_hi[lane] : 0);
    const int se = __reduce_add_sync(0xFFFFFFFFu, lane < kSelWarps ? cnt_eq[lane] : 0);
    if (lane == 0) {
      total[0] = sh;
      total[1] = se;
    }
  }
  cluster_sync();
  // larger and equal keys before this warp's run
  int hi_before = 0, eq_before = 0;
  for (int r = 0; r < rank; ++r) {
    hi_before += cluster_ldi(cluster_map(smem_u32(total), r));
    eq_before += cluster_ldi(cluster_map(smem_u32(total + 1), r));
  }
  hi_before += __reduce_add_sync(0xFFFFFFFFu, lane < warp ? cnt_hi[lane] : 0);
  eq_before += __reduce_add_sync(0xFFFFFFFFu, lane < warp ? cnt_eq[lane] : 0);
  for (int vb = v0; vb < v1; vb += 32) {
    const int v = vb + lane;
    uint4 k4 = make_uint4(0u, 0u, 0u, 0u);
    int c = 0;
    if (v < v1) {
      k4 = four(v);
      c = count(k4);
    }
    if (__all_sync(0xFFFFFFFFu, c == 0)) continue;
    int incl = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += y;
    }
    const int all = __shfl_sync(0xFFFFFFFFu, incl, 31), before = incl - c;
    int h_at = hi_before + (before & 0xFFFF), e_at = eq_before + (before >> 16);
    const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
    if (c != 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool is_hi = k[j] > prefix, is_eq = k[j] == prefix;
        if (is_hi || (is_eq && e_at < need)) {
          const int s = c0 + 4 * v + j, at = h_at + min(e_at, need);
          kept[at] = s;
          nw[at] = KEYS && k[j] != kSafe ? key_weight(k[j]) : w[s];
        }
        h_at += is_hi;
        e_at += is_eq;
      }
    }
    hi_before += all & 0xFFFF;
    eq_before += all >> 16;
  }
  cluster_sync();  // nobody leaves while its counts are read
}

// Rows of the kept slots to their new places.  A warp takes 8 new slots and 4
// blocks of one head; every part of a row is moved as stored.  Bound by sectors:
// a row's V lies in 4-byte (D = 64) or 8-byte pieces.  16 sequences, 4096 kept of
// up to 32768, 8 KV heads, D = 64: 25 us.
template <int D>
__global__ void __launch_bounds__(kThreads) kv_move_kernel(const EvictParams p) {
  using P = PageLayout<D>;
  const int h = blockIdx.y, b = blockIdx.z;
  const int lane = threadIdx.x & 31;
  const int item = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int j = item / (D / 64) * 8 + (lane >> 2);
  const int blk = item % (D / 64) * 4 + (lane & 3);
  const int L = evict_len(p, b);
  if (j >= min(L, p.keep)) return;
  const int slot = p.kept[(static_cast<long long>(b) * p.g.heads + h) * p.keep + j];
  const int from = page_of(p.g, b, slot / kPage);
  const int to = p.new_table[static_cast<long long>(b) * p.new_M + j / kPage];
  if (to < 0 || to >= p.g.num_pages) report_bad_index(p.g.status);
  if (from < 0 || to < 0 || to >= p.g.num_pages) return;
  const uint8_t* src = p.pages + (static_cast<long long>(from) * p.g.heads + h) * P::kBytes;
  uint8_t* dst = p.pages + (static_cast<long long>(to) * p.g.heads + h) * P::kBytes;
  const int s = slot & (kPage - 1), t = j & (kPage - 1);
  const uint2 kc = *reinterpret_cast<const uint2*>(src + P::k_code(s, blk));
  const uint2 vc = ld_v_codes<D>(src, s, blk);
  const uint8_t ks = src[P::k_scale(s, blk)], vs = src[P::v_scale(s, blk)];
  *reinterpret_cast<uint2*>(dst + P::k_code(t, blk)) = kc;
  st_v_codes<D>(dst, t, blk, vc);
  dst[P::k_scale(t, blk)] = ks;
  dst[P::v_scale(t, blk)] = vs;
}

// From 256 rows per sequence on, whole pages.  Measured at 8 KV heads, D = 128
// (append / read, us, row by row against page by page): 32 sequences of 8 rows
// 2.1 / 2.1 against 5.0 / 4.5, of 64 4.6 / 3.9 against 6.6 / 5.8, of 256 12.5 /
// 10.7 against 13.2 / 10.2; 5 prompts of 38000 rows in all 45 / 45 against 40 / 31.
template <int D, bool READ>
cudaError_t launch_rows(const RowsParams& p, cudaStream_t s) {
  const long long items = static_cast<long long>(p.g.T) * p.g.heads, per = kThreads / (D / 8);
  if (p.g.T >= 256ll * p.g.B || items >= (1 << 30)) {  // (items are counted in 32 bits)
    const int x = p.g.T / kPage + 2 * p.g.B, most = (sm_count() * 8 + x - 1) / x;
    return launch_chained(kv_pages_kernel<D, READ>, dim3(x, most < p.g.heads ? most : p.g.heads), kThreads, 0, s, p);
  } else {
    return launch_chained(kv_rows_kernel<D, READ>, dim3(static_cast<unsigned>((items + per - 1) / per)), kThreads, 0, s, p);
  }
}

}  // namespace

int check_kv_cache(const fp4attn_kv_cache_t* c) {
  if (!c || !c->pages || !aligned16(c->pages)) return FP4ATTN_ERR_INVALID_ARG;
  if (c->num_pages <= 0 || c->heads <= 0) return FP4ATTN_ERR_INVALID_ARG;
  if (c->k_exp < -32 || c->k_exp > 32 || c->v_exp < -32 || c->v_exp > 32) return FP4ATTN_ERR_INVALID_ARG;
  if (c->D != 64 && c->D != 128) return FP4ATTN_ERR_UNSUPPORTED;
  if (c->heads > 65535) return FP4ATTN_ERR_UNSUPPORTED;
  return FP4ATTN_OK;
}

int check_kv_batch(const fp4attn_kv_batch_t* b, bool rows) {
  if (!b || !b->table || !b->lens) return FP4ATTN_ERR_INVALID_ARG;
  if (b->B <= 0 || b->max_pages <= 0 || b->T < 0) return FP4ATTN_ERR_INVALID_ARG;
  if (rows && !b->cu && b->T % b->B != 0) return FP4ATTN_ERR_INVALID_ARG;
  if (b->B > kMaxKvBatch || b->max_pages > kMaxSlots / kPage || (rows && b->T > kMaxRows)) return FP4ATTN_ERR_UNSUPPORTED;
  return FP4ATTN_OK;
}

KvGeom kv_geom(const fp4attn_kv_cache_t* c, const fp4attn_kv_batch_t* b, DeviceStatus* st) {
  return KvGeom{b->table, b->lens, b->cu, b->B, b->max_pages, b->T, c->num_pages, c->heads, st};
}

}  // namespace fp4attn

using namespace fp4attn;

extern "C" int fp4attn_kv_page_bytes(int heads, int D, size_t* bytes) {
  if (heads <= 0) return FP4ATTN_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return FP4ATTN_ERR_UNSUPPORTED;
  if (!bytes) return FP4ATTN_ERR_INVALID_ARG;
  *bytes = static_cast<size_t>(heads) * 72 * D;
  return FP4ATTN_OK;
}

extern "C" int fp4attn_kv_append(const fp4attn_kv_cache_t* c, const fp4attn_kv_batch_t* b, const void* k,
                                 long long k_row_stride, long long k_head_stride, const void* v,
                                 long long v_row_stride, long long v_head_stride, void* stream) {
  int st = check_kv_cache(c);
  if (st == FP4ATTN_OK) st = check_kv_batch(b, true);
  if (st != FP4ATTN_OK) return st;
  if (b->T == 0) return FP4ATTN_OK;
  if (!k || !v || !aligned16(k) || !aligned16(v)) return FP4ATTN_ERR_INVALID_ARG;
  if ((k_row_stride | k_head_stride | v_row_stride | v_head_stride) & 7) return FP4ATTN_ERR_INVALID_ARG;
  DeviceStatus* ds = device_status_ptr();
  if (!ds) return FP4ATTN_ERR_CUDA;
  RowsParams p{};
  p.g = kv_geom(c, b, ds);
  p.pages = c->pages;
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.k_row = k_row_stride;
  p.k_head = k_head_stride;
  p.v_row = v_row_stride;
  p.v_head = v_head_stride;
  p.k_scale = ldexpf(1.0f, -c->k_exp);
  p.v_scale = ldexpf(1.0f, -c->v_exp);
  p.k_sixth = p.k_scale / 6.0f;
  p.v_sixth = p.v_scale / 6.0f;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cuda_status(c->D == 128 ? launch_rows<128, false>(p, s) : launch_rows<64, false>(p, s));
}

extern "C" int fp4attn_kv_read(const fp4attn_kv_cache_t* c, const fp4attn_kv_batch_t* b, void* k, void* v,
                               void* stream) {
  int st = check_kv_cache(c);
  if (st == FP4ATTN_OK) st = check_kv_batch(b, true);
  if (st != FP4ATTN_OK) return st;
  if (b->T == 0) return FP4ATTN_OK;
  if (!k || !v || !aligned16(k) || !aligned16(v)) return FP4ATTN_ERR_INVALID_ARG;
  DeviceStatus* ds = device_status_ptr();
  if (!ds) return FP4ATTN_ERR_CUDA;
  RowsParams p{};
  p.g = kv_geom(c, b, ds);
  p.pages = c->pages;
  p.ko = static_cast<__nv_bfloat16*>(k);
  p.vo = static_cast<__nv_bfloat16*>(v);
  p.k_scale = ldexpf(1.0f, c->k_exp);
  p.v_scale = ldexpf(1.0f, c->v_exp);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cuda_status(c->D == 128 ? launch_rows<128, true>(p, s) : launch_rows<64, true>(p, s));
}

extern "C" int fp4attn_kv_evict(const fp4attn_kv_cache_t* c, const fp4attn_kv_batch_t* b, const float* weights,
                                int weights_stride, const int32_t* new_table, int new_max_pages, int keep, int sinks,
                                int recent, int32_t* kept, int32_t* new_lens, float* new_weights, void* stream) {
  int st = check_kv_cache(c);
  if (st == FP4ATTN_OK) st = check_kv_batch(b, false);
  if (st != FP4ATTN_OK) return st;
  if (!weights || !new_table || !kept || !new_lens || !new_weights) return FP4ATTN_ERR_INVALID_ARG;
  if (weights == new_weights || new_table == b->table || new_lens == b->lens) return FP4ATTN_ERR_INVALID_ARG;
  if (keep <= 0 || sinks < 0 || recent < 0 || sinks > keep || recent > keep - sinks) return FP4ATTN_ERR_INVALID_ARG;
  if (weights_stride > kMaxSlots) return FP4ATTN_ERR_UNSUPPORTED;
  if (weights_stride < keep || new_max_pages < (keep + kPage - 1) / kPage) return FP4ATTN_ERR_INVALID_ARG;
  DeviceStatus* ds = device_status_ptr();
  if (!ds) return FP4ATTN_ERR_CUDA;
  const EvictParams p{kv_geom(c, b, ds), c->pages, weights, weights_stride, new_table, new_max_pages,
                      keep, sinks, recent, kept, new_lens, new_weights};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // a bound on the lengths that the host knows
  const long long most = static_cast<long long>(b->max_pages) * kPage < weights_stride
                             ? static_cast<long long>(b->max_pages) * kPage : weights_stride;
  const long long share = ((most + kSelCtas - 1) / kSelCtas + 3) & ~3ll;  // of a CTA
  const dim3 grid_select(c->heads * kSelCtas, b->B);
  cudaError_t e = cudaSuccess;
  if (share <= kSelSmem) {
    e = allow_smem<kv_select_kernel<true>>(kSelSmem * 4);
    if (e == cudaSuccess)
      e = launch(kv_select_kernel<true>, grid_select, kSelThreads, static_cast<size_t>(share) * 4, s, kSelCtas, false, p);
  } else {
    e = launch(kv_select_kernel<false>, grid_select, kSelThreads, 0, s, kSelCtas, false, p);
  }
  if (e != cudaSuccess) return FP4ATTN_ERR_CUDA;
  const long long warps = static_cast<long long>((keep + 7) / 8) * (c->D / 64);
  const dim3 grid(static_cast<unsigned>((warps + kThreads / 32 - 1) / (kThreads / 32)), c->heads, b->B);
  // (not chained: the waiting rows' CTAs cost the selection more than they save, 2 us of 18 at 8 problems)
  return cuda_status(launch(c->D == 128 ? kv_move_kernel<128> : kv_move_kernel<64>, grid, kThreads, 0, s, 0, false, p));
}
