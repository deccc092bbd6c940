// The 4-bit key/value cache: page layout, batch geometry and the conversions
// shared by its kernels (append, read, attention, weights, eviction).
//
// A page holds kPage tokens of one KV head, K and V, in 72 D contiguous bytes,
// so one bulk copy brings a page into shared memory and the bytes arrive in
// the order in which a warp's lanes take them as MMA fragments:
//   K codes   [64 tokens][D/2 bytes]            lane (g, c): row g, 16-byte (D = 128) chunk c
//   K scales  [t % 8][c][t / 8][S]              lane (g, c): its S = D/64 scales of 8 rows, 8 S bytes
//   V codes   [t / 8][g][t % 8][D/16 bytes]     lane (g, c): channels [g D/8, (g+1) D/8) of tokens 2c, 2c + 1
//   V scales  [block][c][t / 16][4]             lane (g, c): one block, tokens 2c, 2c+1, 2c+8, 2c+9 of 4 groups
// (g = lane / 4, c = lane % 4).  Every one of these reads is one conflict-free
// 8- or 16-byte load per lane.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "fp8.cuh"
#include "internal.h"

namespace fp4attn {

constexpr int kPage = 64;

template <int D>
struct PageLayout {
  static constexpr int S = D / 64;         // K scale bytes per lane and row
  static constexpr int kKc = 0;            // K codes
  static constexpr int kKs = 32 * D;       // K scales
  static constexpr int kKBytes = 36 * D;   // the K half
  static constexpr int kVc = 36 * D;       // V codes
  static constexpr int kVs = 68 * D;       // V scales
  static constexpr int kBytes = 72 * D;
  // byte offsets of token t's parts; b: 16-channel block
  __host__ __device__ static constexpr int k_code(int t, int b) { return kKc + t * (D / 2) + b * 8; }
  __host__ __device__ static constexpr int k_scale(int t, int b) {
    return kKs + (((t & 7) * 4 + b / S) * 8 + (t >> 3)) * S + b % S;
  }
  // the 4 code bytes of V's channels 8 q .. 8 q + 7 (half a chunk for D = 128, one for D = 64)
  __host__ __device__ static constexpr int v_half(int t, int q) {
    return kVc + (((t >> 3) * 8 + (D == 128 ? q >> 1 : q)) * 8 + (t & 7)) * (D / 16) + (D == 128 ? (q & 1) * 4 : 0);
  }
  __host__ __device__ static constexpr int v_scale(int t, int b) {
    return kVs + (b * 4 + ((t & 7) >> 1)) * 16 + (t >> 4) * 4 + ((t >> 3) & 1) * 2 + (t & 1);
  }
};

// Batch geometry, all of it in device memory and therefore checked in the
// kernels: an index outside its range is skipped and reported in the status
// word, never followed.
struct KvGeom {
  const int32_t* table;  // [B, M] page numbers
  const int32_t* lens;   // [B] tokens in the cache, the new ones included
  const int32_t* cu;     // [B + 1] rows of each sequence in packed tensors, or null: T / B each
  int B, M, T;
  int num_pages, heads;
  DeviceStatus* status;
};

__device__ __forceinline__ void report_bad_index(DeviceStatus* st) {
  if (st->bad_index == 0u) st->bad_index = 1u;
}

// Rows [row0, row0 + n) of sequence b and its length; n = 0 (and false) when
// the entries are out of range.
__device__ __forceinline__ bool seq_of(const KvGeom& p, int b, int& row0, int& n, int& L) {
  L = p.lens[b];
  if (p.cu) {
    row0 = p.cu[b];
    n = p.cu[b + 1] - row0;
  } else {
    n = p.T / p.B;
    row0 = b * n;
  }
  if (row0 < 0 || n < 0 || row0 > p.T - n || L < 0 || L > p.M * kPage) {
    row0 = n = L = 0;
    return false;
  }
  return true;
}

// Sequence and slot of packed row r (r < T): false for rows before the first
// sequence or behind the last and, after a report, for rows whose slot or page is out of range.
__device__ __forceinline__ bool row_slot(const KvGeom& p, int r, int& b, int& slot) {
  if (p.cu) {
    int lo = 0, hi = p.B;  // the last b with cu[b] <= r
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.cu[mid] <= r) lo = mid; else hi = mid;
    }
    b = lo;
    const int from = p.cu[0];
    if (r >= p.cu[p.B] || (r < from && from <= p.T)) return false;
  } else {
    b = r / (p.T / p.B);
    if (b >= p.B) return false;
  }
  int row0, n, L;
  if (!seq_of(p, b, row0, n, L)) {
    report_bad_index(p.status);
    return false;
  }
  if (r < row0 || r >= row0 + n) {  // only where cu does not ascend
    report_bad_index(p.status);
    return false;
  }
  slot = L - n + (r - row0);
  if (slot < 0) {
    report_bad_index(p.status);
    return false;
  }
  return true;
}

// Page number of a sequence's slot page, or -1 after a report.
__device__ __forceinline__ int page_of(const KvGeom& p, int b, int pi) {
  const int page = p.table[static_cast<long long>(b) * p.M + pi];
  if (page < 0 || page >= p.num_pages) {
    report_bad_index(p.status);
    return -1;
  }
  return page;
}

// ---- clusters ----------------------------------------------------------------

__device__ __forceinline__ int cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return static_cast<int>(r);
}
__device__ __forceinline__ int cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_nctarank;" : "=r"(r));
  return static_cast<int>(r);
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_map(uint32_t saddr, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ float cluster_ld(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ int cluster_ldi(uint32_t addr) { return __float_as_int(cluster_ld(addr)); }
__device__ __forceinline__ uint4 cluster_ld4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// Host-side checks of the two argument structures (rows: the call takes packed rows).
constexpr int kMaxKvBatch = 2048;
constexpr int kMaxSlots = 1 << 30;  // of a sequence
constexpr int kMaxRows = 1 << 28;   // of a call: rows and slots add up within 32 bits
int check_kv_cache(const fp4attn_kv_cache_t* c);
int check_kv_batch(const fp4attn_kv_batch_t* b, bool rows);
KvGeom kv_geom(const fp4attn_kv_cache_t* c, const fp4attn_kv_batch_t* b, DeviceStatus* st);

// Allows a kernel its dynamic shared memory for the largest batch, once per device.
template <auto kernel>
cudaError_t allow_smem(int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// Launches.  A kernel that starts with chain_start() may come up while the one
// before it in the stream runs, if that one has let it (chain_next), and touches
// no memory before all that came before is done (chain_wait).  Saves a few
// tenths of a microsecond per kernel, more where a kernel prepares before it
// waits (the join behind the attention of few queries).
__device__ __forceinline__ void chain_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void chain_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void chain_start() {
  chain_next();
  chain_wait();
}
// cluster: CTAs per cluster, 0: none.  chained: the kernel waits for the one before it itself.
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, int cluster, bool chained,
                   const A&... args) {
  cudaLaunchAttribute at[2] = {};
  int n = 0;
  if (chained) {
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster > 0) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = cluster;
    at[n].val.clusterDim.y = at[n].val.clusterDim.z = 1;
    ++n;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
template <typename... P, typename... A>
cudaError_t launch_chained(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, const A&... args) {
  return launch(kernel, grid, threads, smem, s, 0, true, args...);
}
template <typename... P, typename... A>
cudaError_t launch_chained_cluster(void (*kernel)(P...), dim3 grid, int cluster, int threads, size_t smem, cudaStream_t s,
                                   const A&... args) {
  return launch(kernel, grid, threads, smem, s, cluster, true, args...);
}

// ---- conversions ----------------------------------------------------------

// Two E2M1 codes of byte i of w -> two fp16 values, exact.
__device__ __forceinline__ void e2m1x8_to_half2(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n.reg .b8 b0, b1, b2, b3;\n"
      "mov.b32 {b0, b1, b2, b3}, %4;\n"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
// The reverse: nearest, ties to even, saturating.
__device__ __forceinline__ uint32_t half2x4_to_e2m1x8(const uint32_t (&h)[4]) {
  uint32_t w;
  asm("{\n.reg .b8 b0, b1, b2, b3;\n"
      "cvt.rn.satfinite.e2m1x2.f16x2 b0, %1;\n"
      "cvt.rn.satfinite.e2m1x2.f16x2 b1, %2;\n"
      "cvt.rn.satfinite.e2m1x2.f16x2 b2, %3;\n"
      "cvt.rn.satfinite.e2m1x2.f16x2 b3, %4;\n"
      "mov.b32 %0, {b0, b1, b2, b3};\n}\n"
      : "=r"(w)
      : "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]));
  return w;
}
// Two E4M3 scales -> two fp16 values, exact (the low byte in the low half).
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t splat_lo(uint32_t h) { return __byte_perm(h, h, 0x1010); }
__device__ __forceinline__ uint32_t splat_hi(uint32_t h) { return __byte_perm(h, h, 0x3232); }

__device__ __forceinline__ float pow2i(int e) {  // 2^e, -126 <= e <= 127
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// tanh(x) to a few units of the last place.  Below 0.6 an odd polynomial
// x - x^3 P(x^2) (least squares on Chebyshev nodes, fitted for this range), so
// that small scores keep their relative precision; above, 1 - 2 / (2^(2 x log2 e) + 1).
constexpr float kTanhSmall = 0.6f;
constexpr float kTanhP0 = 0.33333284f, kTanhP1 = -0.13331491f, kTanhP2 = 0.05374493f, kTanhP3 = -0.0206591f,
                kTanhP4 = 0.00573023f;
__device__ __forceinline__ float tanh_acc(float x) {
  const float a = fabsf(x), x2 = x * x;
  float p = fmaf(kTanhP4, x2, kTanhP3);
  p = fmaf(p, x2, kTanhP2);
  p = fmaf(p, x2, kTanhP1);
  p = fmaf(p, x2, kTanhP0);
  const float small = fmaf(-p * x2, x, x);
  const float t = ex2_approx((a > 20.0f ? 20.0f : a) * 2.885390081777927f);
  const float big = copysignf(1.0f - __fdividef(2.0f, t + 1.0f), x);
  return a < kTanhSmall ? small : big;  // a NaN stays one
}
// a, b -> c tanh(a), c tanh(b) for |a|, |b| < kTanhSmall, two at a time.
__device__ __forceinline__ void tanh2_small(float& a, float& b, float c) {
  float u, v, p, q;
  fmul2(u, v, a, b, a, b);
  ffma2(p, q, u, v, -kTanhP4, -kTanhP4, -kTanhP3, -kTanhP3);
  ffma2(p, q, p, q, u, v, -kTanhP2, -kTanhP2);
  ffma2(p, q, p, q, u, v, -kTanhP1, -kTanhP1);
  ffma2(p, q, p, q, u, v, -kTanhP0, -kTanhP0);
  ffma2(p, q, p, q, u, v, 1.0f, 1.0f);
  fmul2(a, b, a, b, c, c);
  fmul2(a, b, a, b, p, q);
}
// a, b -> c tanh(a), c tanh(b) for |a|, |b| < kTanhTiny, as scores far below
// their cap are: the same kind of polynomial, two terms shorter, two at a time.
constexpr float kTanhTiny = 0.25f;
__device__ __forceinline__ void tanh2_tiny(float& a, float& b, float c) {
  float u, v, p, q;
  fmul2(u, v, a, b, a, b);
  ffma2(p, q, u, v, -0.0512210652f, -0.0512210652f, 0.13322635f, 0.13322635f);
  ffma2(p, q, p, q, u, v, -0.333332121f, -0.333332121f);
  ffma2(p, q, p, q, u, v, 1.0f, 1.0f);
  fmul2(a, b, a, b, c, c);
  fmul2(a, b, a, b, p, q);
}

}  // namespace fp4attn
