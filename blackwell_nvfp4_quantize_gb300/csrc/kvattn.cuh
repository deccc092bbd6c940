// Shared by the attention kernels over the 4-bit key/value cache: arguments,
// the even split of the work, and how partial results are joined.
#pragma once
#include <cfloat>
#include <cmath>

#include "kvcache.cuh"

namespace fp4attn {

constexpr int kNoColumn = -(1 << 30);  // below every slot, and slots stay below 2^30
constexpr float kMaxCap = 1.2379400392853803e27f;  // 2^90: see score_factor
constexpr int kMaxWindow = 1 << 30;       // no sequence is longer; slots minus windows stay within 32 bits
constexpr float kLog2Ef = 1.4426950408889634f;
constexpr float kLn2f = 0.6931471805599453f;

struct KvAttnParams {
  KvGeom g;
  const uint8_t* pages;
  const __nv_bfloat16* q;
  long long q_row, q_head;  // strides in elements
  int G;                    // query heads per KV head
  int max_new;
  float scale;   // softmax_scale 2^k_exp: S to natural-log scores
  float cap;     // 0: none
  int window;    // 0: none
  const float* slopes;  // [heads G] or null
  float v_up;           // 2^v_exp
  __nv_bfloat16* o;     // [T, heads G, D]
  float* lse;           // [T, heads G]
  int* plan;            // for the second kernel: units before each sequence (kvprompt.cu: a Split per run)
  float* part;          // partial results, 2 per run
  const float* lse_in;  // weights kernel
  float* w;             // [B, heads, W]
  int W;
  float decay;
  int ctas;  // of the attention kernel's even split (kvprompt.cu: CTA pairs)
};

// Blocks of kBlock slots that the queries [r0, r1] / G of a sequence see: the
// first, how many (1, and `none`, where they see nothing: the unit still
// writes the rows).
struct Span {
  int first, count;
  bool none;
};
template <int kBlock>
__device__ __forceinline__ Span span_of(int L, int n, int G, int window, int r0, int r1) {
  const int first = L - n;
  const int hi = first + r1 / G;
  if (hi < 0) return Span{0, 1, true};
  int lo = 0;
  if (window > 0) lo = max(0, first + r0 / G - window + 1);
  return Span{lo / kBlock, hi / kBlock - lo / kBlock + 1, false};
}

// Sequence b for the attention kernels; n = 0 after a report where its entries
// are out of range or it has more new tokens than the caller said.
__device__ __forceinline__ void attn_seq(const KvAttnParams& p, int b, int& row0, int& n, int& L) {
  if (!seq_of(p.g, b, row0, n, L) || n > p.max_new) {
    report_bad_index(p.g.status);
    row0 = n = L = 0;
  }
}

// Units per head of a sequence: blocks summed over its tiles of kCols columns.
template <int kCols, int kBlock>
__device__ __forceinline__ int units_of(const KvAttnParams& p, int n, int L) {
  const int R = n * p.G;
  int sum = 0;
#pragma unroll 1
  for (int r = 0; r < R; r += kCols) sum += span_of<kBlock>(L, n, p.G, p.window, r, min(R, r + kCols) - 1).count;
  return sum;
}

// prefix[b] = units before sequence b, prefix[B] = all.  Every thread of the
// CTA takes part; scratch holds one int per warp.
template <int kCols, int kBlock>
__device__ __forceinline__ void plan_units(const KvAttnParams& p, int* prefix, int* scratch) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nwarps = blockDim.x >> 5;
  int carry = 0;
  for (int base = 0; base < p.g.B; base += blockDim.x) {
    int c = 0;
    if (base + tid < p.g.B) {
      int row0, n, L;
      attn_seq(p, base + tid, row0, n, L);
      c = units_of<kCols, kBlock>(p, n, L) * p.g.heads;
    }
    int incl = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += x;
    }
    __syncthreads();
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    int before = carry, all = carry;
    for (int i = 0; i < nwarps; ++i) {
      if (i < warp) before += scratch[i];
      all += scratch[i];
    }
    if (base + tid < p.g.B) prefix[base + tid] = before + incl - c;
    carry = all;
  }
  if (tid == 0) prefix[p.g.B] = carry;
  __syncthreads();
}

struct Unit {
  int b, h, r0, r1;  // columns r0 .. r1 of (sequence, KV head)
  int begin, end;    // the problem's units
  int first;         // its first block
  bool none;
  int row0, n, L;
};

template <int kCols, int kBlock>
__device__ __forceinline__ Unit find_unit(const KvAttnParams& p, const int* prefix, int u) {
  int lo = 0, hi = p.g.B;  // the last b with prefix[b] <= u and units of its own
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= u) lo = mid; else hi = mid;
  }
  Unit x;
  x.b = lo;
  attn_seq(p, lo, x.row0, x.n, x.L);
  const int per_head = (prefix[lo + 1] - prefix[lo]) / p.g.heads;
  x.h = (u - prefix[lo]) / per_head;
  int at = prefix[lo] + x.h * per_head;
  const int R = x.n * p.G;
#pragma unroll 1  // usually one tile: unrolled, decoding takes 3% longer
  for (x.r0 = 0;; x.r0 += kCols) {
    x.r1 = min(R, x.r0 + kCols) - 1;
    const Span s = span_of<kBlock>(x.L, x.n, p.G, p.window, x.r0, x.r1);
    if (u < at + s.count) {
      x.begin = at;
      x.end = at + s.count;
      x.first = s.first;
      x.none = s.none;
      return x;
    }
    at += s.count;
  }
}

__device__ __forceinline__ int run_length(int units, int ctas) { return max(1, (units + ctas - 1) / ctas); }

// What turns a row's S into its log2-domain scores (with a cap: into s / cap),
// where its elements were multiplied by 1 / down, a power of two.  Masked scores
// are -inf when this multiplies them, so it is never 0 there: S is below 2^34,
// and what the least normal number makes of that is as good as 0.  (With a cap
// or slopes the mask comes later, and a subnormal factor is off by 2^-150: below
// 2^-24 of a score's unit for every cap that is accepted.)
template <bool MOD>
__device__ __forceinline__ float score_factor(const KvAttnParams& p, float down) {
  const float f = p.scale * down;
  return MOD ? fminf(p.cap > 0.0f ? f / p.cap : f * kLog2Ef, FLT_MAX) : fminf(fmaxf(f * kLog2Ef, FLT_MIN), FLT_MAX);
}

// Floats of one partial result: O [cols][D], max [cols], sum [cols].
template <int D>
__host__ __device__ constexpr int part_floats(int cols) { return cols * (D + 2); }

// Row r's final values.  top: log2-domain maximum (-inf: nothing seen), sum: of
// 2^(score - top + shift), acc: the same weights times V.
__device__ __forceinline__ float out_o(float acc, float sum, float v_up) { return sum == 0.0f ? 0.0f : acc / sum * v_up; }
__device__ __forceinline__ float out_lse(float top, float sum, float shift) {
  return sum == 0.0f ? -INFINITY : ((top == -INFINITY ? 0.0f : top) + log2f(sum) - shift) * kLn2f;
}
// Factor that brings a partial result with maximum m to the common maximum
// (where nothing was seen at all, 1: a sum that is NaN stays one).
__device__ __forceinline__ float join_factor(float m, float top) { return top == -INFINITY ? 1.0f : ex2_approx(m - top); }

// A problem that begins in one run of the prompt kernel and ends in a later
// one, `last` (-1: the run has none; at most one begins in each).
struct Split {
  int last, row0, h, r0, r1;
  float shift;  // P was held as 2^shift p
};
__device__ __forceinline__ Split* split_of(const KvAttnParams& p, int run) { return reinterpret_cast<Split*>(p.plan) + run; }

// Joins the partial results of such problems, from the records that the runs
// left: block x that of run x, D / 4 lanes per row with four channels each,
// kDeep rows per lane whose loads are in flight together.  (The prompt kernel
// holds every register of its SM, so nothing can be prepared beside it: what the
// blocks had to find out by themselves came on top of its time.)
constexpr int kJoinThreads = 256;
constexpr int kDeep = 2;
template <int D>
constexpr int kJoinRows = kJoinThreads / (D / 4) * kDeep;  // of a block

template <int D, int kCols>
__global__ void __launch_bounds__(kJoinThreads) kv_join_kernel(const KvAttnParams p) {
  constexpr int kLanes = D / 4, kRows = kJoinThreads / kLanes, kPart = part_floats<D>(kCols);
  chain_start();
  const int c0 = blockIdx.x, lane = threadIdx.x % kLanes, col0 = blockIdx.y * kJoinRows<D> + threadIdx.x / kLanes;
  const Split x = *split_of(p, c0);
  if (x.last < 0 || x.r0 + static_cast<int>(blockIdx.y) * kJoinRows<D> > x.r1) return;
  // (usually two results: the maximum so far, and what has been added up under it)
  float top[kDeep], sum[kDeep];
  float4 acc[kDeep];
#pragma unroll
  for (int i = 0; i < kDeep; ++i) {
    top[i] = -INFINITY;
    sum[i] = 0.0f;
    acc[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
  float m[2][kDeep], l[2][kDeep];
  float4 v[2][kDeep];
  auto load = [&](int c, float (&m)[kDeep], float (&l)[kDeep], float4 (&v)[kDeep]) {
    const float* y = p.part + static_cast<long long>(c * 2 + (c == c0 ? 1 : 0)) * kPart;
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      const int col = min(col0 + i * kRows, x.r1 - x.r0);  // behind the last row: that one again
      m[i] = y[kCols * D + col];
      l[i] = y[kCols * D + kCols + col];
      v[i] = *reinterpret_cast<const float4*>(y + col * D + 4 * lane);
    }
  };
  auto add = [&](int c, const float (&m)[kDeep], const float (&l)[kDeep], const float4 (&v)[kDeep]) {
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      const float now = fmaxf(top[i], m[i]), f0 = c == c0 ? 0.0f : join_factor(top[i], now), f1 = join_factor(m[i], now);
      top[i] = now;
      sum[i] = sum[i] * f0 + l[i] * f1;
      acc[i].x = acc[i].x * f0 + v[i].x * f1;
      acc[i].y = acc[i].y * f0 + v[i].y * f1;
      acc[i].z = acc[i].z * f0 + v[i].z * f1;
      acc[i].w = acc[i].w * f0 + v[i].w * f1;
    }
  };
  // the next two results are on their way while one is added
  load(c0, m[0], l[0], v[0]);
  load(c0 + 1, m[1], l[1], v[1]);
#pragma unroll 1
  for (int c = c0; c <= x.last; c += 2) {
    add(c, m[0], l[0], v[0]);
    if (c + 2 <= x.last) load(c + 2, m[0], l[0], v[0]);
    if (c + 1 > x.last) break;
    add(c + 1, m[1], l[1], v[1]);
    if (c + 3 <= x.last) load(c + 3, m[1], l[1], v[1]);
  }
#pragma unroll
  for (int i = 0; i < kDeep; ++i) {
    const int r = x.r0 + col0 + i * kRows;
    if (r > x.r1) return;
    const long long out = static_cast<long long>(x.row0 + r / p.G) * (p.g.heads * p.G) + x.h * p.G + r % p.G;
    const __nv_bfloat162 lo = __floats2bfloat162_rn(out_o(acc[i].x, sum[i], p.v_up), out_o(acc[i].y, sum[i], p.v_up));
    const __nv_bfloat162 hi = __floats2bfloat162_rn(out_o(acc[i].z, sum[i], p.v_up), out_o(acc[i].w, sum[i], p.v_up));
    *reinterpret_cast<uint2*>(p.o + out * D + 4 * lane) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    if (lane == 0) p.lse[out] = out_lse(top[i], sum[i], x.shift);
  }
}

// The plan's part of a workspace, before the partial results (the splits of up to 340 runs of the prompt kernel).
inline size_t plan_bytes() { return (static_cast<size_t>(kMaxKvBatch + 1) * 4 + 255) / 256 * 256; }

// Attention of many queries (kvprompt.cu): runs (CTA pairs), workspace, launch.
int prompt_runs();
size_t prompt_workspace(int D);
cudaError_t launch_prompt(const KvAttnParams& p, int D, cudaStream_t s);

}  // namespace fp4attn
