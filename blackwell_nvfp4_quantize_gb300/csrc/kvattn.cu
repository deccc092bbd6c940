// Attention of few queries over the 4-bit key/value cache, and the attention
// weight the cached tokens gather.
//
// For a sequence of L cached tokens whose last n are new, query i < n sits at
// slot L - n + i; with s = scale q.k (cap c: c tanh(s / c); slope m:
// - m (slot of i - slot of j)) over the slots j it sees (not after its own
// and, with a window w, fewer than w before it):
//   O_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(s_ij - max),  LSE_i
//   weight_j = decay weight_j + sum over the queries of a KV head of exp(s_ij - LSE_i)
//
// A KV head's group of G query heads times n tokens gives the "columns" of one
// problem, or of several where there are more than a tile's 8 NT.  The kernel is bound by reading the cache (K and V are
// 72 D / 64 bytes per token and KV head, read once), so it is built as streams:
// every warp takes a run of pages, keeps two of them in flight with bulk copies
// into its own part of shared memory, and works alone.  Scores are computed
// transposed, S^T = K q^T (m16n8k16, fp16 operands, fp32 accumulation): 16
// cached tokens by 8 columns, so that 1 to 8 columns cost one MMA and not an
// eighth of one.  K and V become fp16 in registers: E2M1 codes times E4M3
// scales have at most 6 significant bits and lie in [2^-10, 2688], so both are
// exact.  The query row is scaled by a power of two that puts its largest
// element in [2^13, 2^14), which leaves bf16's 8 bits exact in fp16 except for
// elements below 2^-27 of the largest.  P is rounded to fp16 at 2^14 of its
// row maximum (error 2^-12 of the value, independent from token to token;
// what falls below 2^-38 of the maximum is dropped); its sum is kept of the
// unrounded fp32 values.  tcgen05 is of no use here: its A operand would have
// to pass through shared memory as fp16, four times the bytes that arrive.
//
// The conversion E2M1 -> fp16 (4 instructions per 8 codes on the half-rate ALU
// pipe: 8 cycles per word and scheduler, measured; shifts and masks take 29)
// and the scaling (4) are most of the instructions.
//
// Work is split evenly whatever the lengths: all (sequence, head, page) units
// are numbered in a row and every warp takes an equal run of them.  A problem
// that lies in one run is finished there; the others leave partial (O, max,
// sum) triples - one per CTA where its four warps work on the same problem, one
// per warp otherwise - that a second kernel joins in the order of the runs, so
// results do not depend on timing.
//
// Measured (8 KV heads, D = 128; of 6.8 TB/s that a copy reaches): 64 sequences
// to 8192 tokens, 8 query heads per KV head, 63 us and 8 for the join, 4.7 TB/s
// (DRAM 59%, ALU pipe 50%, issue slots 55%; in 45% of the cycles none of a
// scheduler's 2.7 warps can issue); 3 sequences to 131072 tokens 74 us and 9, 5.6
// TB/s; one sequence of 4096 8.2 us.  Gathered weight, 32 sequences to 16384
// tokens: 36 us, 4.4 TB/s (DRAM 51%, ALU pipe 39%, issue slots 51%).
#include <type_traits>

#include "kvattn.cuh"

namespace fp4attn {
namespace {

constexpr int kWarps = 4;  // per CTA
// CTAs of the attention kernel on an SM: three, or two where the columns'
// fragments would not fit 168 registers.
__host__ __device__ constexpr int resident(int D, int nt) { return D * nt >= 192 ? 2 : 3; }
constexpr int kAttnThreads = 32 * kWarps;
constexpr int kAll = 1 << 30;      // one tile: a page serves every column
constexpr float kPShift = 14.0f;   // P is held as 2^14 p

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same with C = 0
__device__ __forceinline__ void mma_16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// The query columns of a warp: fp16 fragments and what turns S into scores.
template <int D, int NT>
struct Columns {
  uint32_t q[NT][D / 8];  // lane (g, c): elements [c D/4, (c+1) D/4) of column g, in pairs
  float cs[NT][2];        // of columns 2c, 2c + 1: log2-domain score per unit of S (with a cap: s / cap)
  float slope[NT][2];     // log2-domain
  int at[NT][2];          // slot of the query; kNoColumn: no such column
  int at_min, at_max;     // over the warp's valid columns
};

template <int D, int NT, bool MOD>
__device__ __forceinline__ void load_columns(const KvAttnParams& p, const Unit& x, Columns<D, NT>& q) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  q.at_min = x.L - x.n + x.r0 / p.G;
  q.at_max = x.L - x.n + x.r1 / p.G;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = x.r0 + nt * 8 + g;
    uint32_t w[D / 8];
    if (r <= x.r1) {
      const uint4* src = reinterpret_cast<const uint4*>(p.q + (x.row0 + r / p.G) * p.q_row +
                                                        (x.h * p.G + r % p.G) * p.q_head + c * (D / 4));
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint4 v = __ldg(src + i);
        w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < D / 8; ++i) w[i] = 0u;
    }
    uint32_t m2 = 0;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) m2 = __vmaxu2(m2, w[i] & 0x7FFF7FFFu);
    uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    const int e = max(static_cast<int>(m >> 7), 20);  // exponent field of the row's largest element
    const float up = pow2i(140 - e), down = pow2i(e - 140);
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
      q.q[nt][i] = pack_half2(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xFFFF0000u) * up);
    const float cs = score_factor<MOD>(p, down);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int col = x.r0 + nt * 8 + 2 * c + k;
      q.cs[nt][k] = __shfl_sync(0xFFFFFFFFu, cs, (2 * c + k) * 4);
      q.at[nt][k] = col <= x.r1 ? x.L - x.n + col / p.G : kNoColumn;
      q.slope[nt][k] = 0.0f;
      if (MOD && p.slopes && col <= x.r1) q.slope[nt][k] = p.slopes[x.h * p.G + col % p.G] * kLog2Ef;
    }
  }
}

// S^T of MT groups of 16 tokens of a page, from group i0 on: s[i][nt] = tokens
// 16 (i0 + i) + g and + 8 by columns 2c, 2c + 1.
template <int D, int NT, int MT>
__device__ __forceinline__ void page_scores(const uint8_t* page, int i0, const uint32_t (&sc)[MT],
                                            const Columns<D, NT>& q, float (&s)[MT][NT][4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const uint8_t* ra = page + (16 * (i0 + i) + g) * (D / 2) + c * (D / 8);
    const uint8_t* rb = ra + 8 * (D / 2);
    uint32_t wa[D / 32], wb[D / 32];
    if constexpr (D == 128) {
      const uint4 a = *reinterpret_cast<const uint4*>(ra), b = *reinterpret_cast<const uint4*>(rb);
      wa[0] = a.x; wa[1] = a.y; wa[2] = a.z; wa[3] = a.w;
      wb[0] = b.x; wb[1] = b.y; wb[2] = b.z; wb[3] = b.w;
    } else {
      const uint2 a = *reinterpret_cast<const uint2*>(ra), b = *reinterpret_cast<const uint2*>(rb);
      wa[0] = a.x; wa[1] = a.y;
      wb[0] = b.x; wb[1] = b.y;
    }
    uint32_t sa[2], sb[2];  // scales of the lane's blocks in rows g and g + 8
    if constexpr (D == 128) {
      const uint32_t xa = e4m3x2_to_half2(sc[i]), xb = e4m3x2_to_half2(sc[i] >> 16);
      sa[0] = splat_lo(xa); sa[1] = splat_hi(xa);
      sb[0] = splat_lo(xb); sb[1] = splat_hi(xb);
    } else {
      const uint32_t xx = e4m3x2_to_half2(sc[i]);
      sa[0] = sa[1] = splat_lo(xx);
      sb[0] = sb[1] = splat_hi(xx);
    }
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
      uint32_t ha[4], hb[4];
      e2m1x8_to_half2(wa[w], ha);
      e2m1x8_to_half2(wb[w], hb);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        ha[k] = hmul2(ha[k], sa[w >> 1]);
        hb[k] = hmul2(hb[k], sb[w >> 1]);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (w == 0) mma_16816_first(s[i][nt], ha[0], hb[0], ha[1], hb[1], q.q[nt][4 * w], q.q[nt][4 * w + 1]);
        else mma_16816(s[i][nt], ha[0], hb[0], ha[1], hb[1], q.q[nt][4 * w], q.q[nt][4 * w + 1]);
        mma_16816(s[i][nt], ha[2], hb[2], ha[3], hb[3], q.q[nt][4 * w + 2], q.q[nt][4 * w + 3]);
      }
    }
  }
}

// The lane's K scales of a page: word i for rows 16 i + g (low) and + 8 (high).
template <int D>
__device__ __forceinline__ void page_k_scales(const uint8_t* page, uint32_t (&sc)[4]) {
  const int lane = threadIdx.x & 31;
  if constexpr (D == 128) {
    const uint4 v = *reinterpret_cast<const uint4*>(page + PageLayout<D>::kKs + lane * 16);
    sc[0] = v.x; sc[1] = v.y; sc[2] = v.z; sc[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(page + PageLayout<D>::kKs + lane * 8);
    sc[0] = v.x & 0xFFFFu; sc[1] = v.x >> 16; sc[2] = v.y & 0xFFFFu; sc[3] = v.y >> 16;
  }
}

// With a cap or slopes, S -> log2-domain scores (otherwise S stays, and its
// factor cs goes into the exponential's multiply-add); -inf where a column does
// not see a token.  slot0: slot of row g of the first group.
template <int D, int NT, int MT, bool MOD>
__device__ __forceinline__ void scores_of(const KvAttnParams& p, const Columns<D, NT>& q, int slot0,
                                          float (&s)[MT][NT][4]) {
  if constexpr (MOD) {
    if (p.cap > 0.0f) {
      bool big = false;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            s[i][nt][k] *= q.cs[nt][k & 1];
            big |= !(fabsf(s[i][nt][k]) < kTanhSmall);
          }
      const float cap = p.cap * kLog2Ef;
      if (__any_sync(0xFFFFFFFFu, big)) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) s[i][nt][k] = cap * tanh_acc(s[i][nt][k]);
      } else {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            tanh2_small(s[i][nt][0], s[i][nt][1], cap);
            tanh2_small(s[i][nt][2], s[i][nt][3], cap);
          }
      }
    } else {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[i][nt][k] *= q.cs[nt][k & 1];
    }
    if (p.slopes) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float far = static_cast<float>(q.at[nt][j] - slot0);
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            s[i][nt][j] = fmaf(-q.slope[nt][j], far - 16.0f * i, s[i][nt][j]);
            s[i][nt][j + 2] = fmaf(-q.slope[nt][j], far - (16.0f * i + 8.0f), s[i][nt][j + 2]);
          }
        }
    }
  }
}

template <int D, int NT, int MT>
__device__ __forceinline__ void mask_scores(const KvAttnParams& p, const Columns<D, NT>& q, int slot0,
                                            float (&s)[MT][NT][4]) {
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int slot = slot0 + 16 * i + 8 * (k >> 1), at = q.at[nt][k & 1];
        if (slot > at || (p.window > 0 && slot <= at - p.window)) s[i][nt][k] = -INFINITY;
      }
}

// One warp's stream of page parts: units [start, start + n) of the run, kStages
// in flight.  The 32 lanes look up 32 pages at a time; lane 0 issues the copies.
// A unit without a page (an index out of range, nothing to see) holds no stage.
template <int kBytes, int kStages>
struct PageStream {
  uint8_t* ring;
  uint64_t* full;
  long long off;     // this lane's page offset: unit base + lane
  int base, n, start;
  uint32_t held = 0, parity = 0;  // per stage: a page is in flight or in place; phase of its barrier

  // unit_of(u): the problem of unit u
  template <typename F>
  __device__ __forceinline__ void look_up(const KvAttnParams& p, F&& unit_of, long long page_bytes, int from) {
    const int lane = threadIdx.x & 31;
    base = from;
    off = -1;
    if (from + lane < n) {
      const int u = start + from + lane;
      const Unit x = unit_of(u);
      if (!x.none) {
        const int pg = page_of(p.g, x.b, x.first + (u - x.begin));
        if (pg >= 0) off = (static_cast<long long>(pg) * p.g.heads + x.h) * page_bytes;
      }
    }
  }
  // Unit k's copy into stage k % kStages, which no lane reads any more.
  template <typename F>
  __device__ __forceinline__ void issue(const KvAttnParams& p, F&& unit_of, long long page_bytes, int k) {
    if (k >= n) return;
    if (k >= base + 32) look_up(p, unit_of, page_bytes, k);
    const long long o = __shfl_sync(0xFFFFFFFFu, off, k - base);
    const int s = k % kStages;
    if (o < 0) return;
    held |= 1u << s;
    if ((threadIdx.x & 31) == 0) {
      fence_proxy_async_smem();  // the lanes' reads of the stage come before the copy's writes
      mbar_arrive_expect_tx(full + s, kBytes);
      bulk_load(ring + s * kBytes, p.pages + o, kBytes, full + s);
    }
  }
  __device__ __forceinline__ bool has(int k) const { return (held >> (k % kStages)) & 1u; }
  __device__ __forceinline__ bool wait(const KvAttnParams& p, int k, volatile int* abort_flag, unsigned site) {
    const int s = k % kStages;
    bool ok = mbar_wait(full + s, (parity >> s) & 1u, abort_flag, p.g.status, site);
    ok = __all_sync(0xFFFFFFFFu, ok);
    if (ok) {  // otherwise drain() waits for it
      parity ^= 1u << s;
      held &= ~(1u << s);
    }
    return ok;
  }
  // After a wait that gave up: no copy may be in flight when the CTA leaves.
  __device__ __forceinline__ void drain(const KvAttnParams& p, volatile int* abort_flag) {
    for (int s = 0; s < kStages; ++s)
      if ((held >> s) & 1u) mbar_wait_drain(full + s, (parity >> s) & 1u, abort_flag, p.g.status, 62);
  }
};

// Shared memory of a CTA whose warps stream parts of kPart bytes: 18 KB each, so
// that three CTAs fit on an SM.
template <int kPart>
struct StreamSmem {
  static constexpr int kRing = 2 * PageLayout<128>::kBytes;  // one warp's
  static constexpr int kStages = kRing / kPart;
  static constexpr int kBars = kWarps * kRing;
  static constexpr int kMisc = kBars + kWarps * kStages * 8;
  static constexpr int kMerge = kMisc + 64;                       // maxima and sums of the four warps
  static constexpr int kPrefix = kMerge + 2 * kWarps * 32 * 4;
  static int bytes(int B) { return kPrefix + (B + 1) * 4; }
};

// Units of a warp's run; a CTA holds kWarps consecutive runs.
__device__ __forceinline__ int warp_run(const KvAttnParams& p, int units) { return run_length(units, p.ctas * kWarps); }

// CLUSTER: instead of the even split, a cluster of CTAs takes one problem, its
// pages shared out among the cluster's warps, and joins the CTAs' results
// through distributed shared memory: one kernel and no workspace, for batches
// whose problems all fit on the GPU at once and are short.
template <int D, int NT, bool MOD, bool CLUSTER>
__global__ void __launch_bounds__(kAttnThreads, resident(D, NT)) kv_attn_kernel(const KvAttnParams p) {
  using L_ = StreamSmem<PageLayout<D>::kBytes>;
  // Groups of 16 tokens per step: the whole page, so that many products are in
  // flight, unless caps and slopes make the step outgrow the instruction cache.
  // 16 sequences of 8192 tokens, 8 KV heads, 16 columns (D = 64 / 128, us): plain
  // 33.0 / 55.3 with 4 groups, 35.7 / 56.9 with 2; capped with slopes 52 / 74 and 49 / 72.
  constexpr int MT = NT == 1 || !MOD ? 4 : 2;
  constexpr int kCols = 8 * NT, kPageBytes = PageLayout<D>::kBytes;
  constexpr int kOStride = D + 4;  // floats per column of a warp's merge area
  static_assert(8 * kOStride * 4 <= L_::kRing, "the merge area takes the ring's place");
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L_::kMisc);
  int* scratch = reinterpret_cast<int*>(smem + L_::kMisc + 16);
  float* sm_m = reinterpret_cast<float*>(smem + L_::kMerge);
  float* sm_l = sm_m + kWarps * 32;
  int* prefix = reinterpret_cast<int*>(smem + L_::kPrefix);

  PageStream<kPageBytes, L_::kStages> st;
  st.ring = smem + warp * L_::kRing;
  st.full = reinterpret_cast<uint64_t*>(smem + L_::kBars) + warp * L_::kStages;
  if (lane == 0) {
    for (int s = 0; s < L_::kStages; ++s) mbar_init(st.full + s, 1);
    if (warp == 0) *abort_flag = 0;
    fence_mbar_init();
  }
  chain_wait();
  chain_next();  // after the wait: the join looks at the lengths before its own
  const int rank = CLUSTER ? cluster_rank() : 0, ranks = CLUSTER ? cluster_size() : 1;
  int cta_start = 0, cta_end = 0;
  Unit x{};
  if constexpr (CLUSTER) {
    const int id = blockIdx.x / ranks, tiles = (p.max_new * p.G + kCols - 1) / kCols;
    x.b = id / (p.g.heads * tiles);
    x.h = id / tiles % p.g.heads;
    x.r0 = id % tiles * kCols;
    attn_seq(p, x.b, x.row0, x.n, x.L);
    if (x.r0 >= x.n * p.G) return;  // (the whole cluster)
    x.r1 = min(x.n * p.G, x.r0 + kCols) - 1;
    const Span s = span_of<kPage>(x.L, x.n, p.G, p.window, x.r0, x.r1);
    x.first = s.first;
    x.none = s.none;
    x.end = s.count;
    const int per = (s.count + ranks * kWarps - 1) / (ranks * kWarps), w = rank * kWarps + warp;
    st.start = min(s.count, w * per);
    st.n = min(s.count, st.start + per) - st.start;
    __syncthreads();
  } else {
    plan_units<kCols, kPage>(p, prefix, scratch);  // ends with a barrier
    const int units = prefix[p.g.B], per = warp_run(p, units);
    cta_start = min(units, static_cast<int>(blockIdx.x) * kWarps * per);
    cta_end = min(units, cta_start + kWarps * per);
    if (cta_start >= cta_end) return;
    if (blockIdx.x == 0)  // for the join
      for (int i = threadIdx.x; i <= p.g.B; i += kAttnThreads) p.plan[i] = prefix[i];
    st.start = min(units, cta_start + warp * per);
    st.n = min(units, st.start + per) - st.start;
  }
  const auto unit_of = [&](int u) {
    if constexpr (CLUSTER) return x;
    else return find_unit<kCols, kPage>(p, prefix, u);
  };
  st.look_up(p, unit_of, kPageBytes, 0);
#pragma unroll 1
  for (int k = 0; k < L_::kStages; ++k) st.issue(p, unit_of, kPageBytes, k);

  bool shared = true;  // the whole CTA works on one problem
  Columns<D, NT> q;
  if constexpr (CLUSTER) {
    load_columns<D, NT, MOD>(p, x, q);
  } else {
    shared = find_unit<kCols, kPage>(p, prefix, cta_start).end >= cta_end;
    x.end = -1;  // none loaded yet
  }
  float o[D / 16][NT][4], m[NT][2], l[NT][2];
  auto clear = [&]() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
      for (int t = 0; t < D / 16; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[t][nt][i] = 0.0f;
    }
  };
  // Column sums over the lanes of a column.
  auto sums = [&]() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        l[nt][j] += __shfl_xor_sync(0xFFFFFFFFu, l[nt][j], 4);
        l[nt][j] += __shfl_xor_sync(0xFFFFFFFFu, l[nt][j], 8);
        l[nt][j] += __shfl_xor_sync(0xFFFFFFFFu, l[nt][j], 16);
      }
  };
  // This warp's result of problem x: final if its run holds the whole problem, otherwise partial.
  auto finish = [&]() {
    sums();
    const bool begins = x.begin >= st.start, whole = begins && x.end <= st.start + st.n;
    float* part = p.part + static_cast<long long>((blockIdx.x * kWarps + warp) * 2 + begins) * part_floats<D>(kCols);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int col = nt * 8 + 2 * c + j, r = x.r0 + col;
        if (r > x.r1) continue;
        if (whole) {
          const long long at = static_cast<long long>(x.row0 + r / p.G) * (p.g.heads * p.G) + x.h * p.G + r % p.G;
          uint32_t h[D / 16];
#pragma unroll
          for (int t = 0; t < D / 16; ++t) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(out_o(o[t][nt][j], l[nt][j], p.v_up),
                                                           out_o(o[t][nt][j + 2], l[nt][j], p.v_up));
            h[t] = *reinterpret_cast<const uint32_t*>(&b);
          }
          uint4* dst = reinterpret_cast<uint4*>(p.o + at * D + g * (D / 8));
#pragma unroll
          for (int t = 0; t < D / 64; ++t) dst[t] = make_uint4(h[4 * t], h[4 * t + 1], h[4 * t + 2], h[4 * t + 3]);
          if (g == 0) p.lse[at] = out_lse(m[nt][j], l[nt][j], kPShift);
        } else {
          float4* dst = reinterpret_cast<float4*>(part + col * D + g * (D / 8));
#pragma unroll
          for (int t = 0; t < D / 32; ++t)
            dst[t] = make_float4(o[2 * t][nt][j], o[2 * t][nt][j + 2], o[2 * t + 1][nt][j], o[2 * t + 1][nt][j + 2]);
          if (g == 0) {
            part[kCols * D + col] = m[nt][j];
            part[kCols * D + kCols + col] = l[nt][j];
          }
        }
      }
  };

  bool ok = true;
  clear();
#pragma unroll 1
  for (int k = 0; k < st.n && ok; ++k) {
    const int u = st.start + k;
    if (!CLUSTER && u >= x.end) {
      if (x.end >= 0) {
        finish();
        clear();
      }
      x = find_unit<kCols, kPage>(p, prefix, u);
      load_columns<D, NT, MOD>(p, x, q);
    }
    if (st.has(k)) {
      ok = st.wait(p, k, abort_flag, 61);
      if (!ok) break;
      const uint8_t* page = st.ring + (k % L_::kStages) * kPageBytes;
      const int slot0 = (x.first + (u - x.begin)) * kPage;
      const bool hides = slot0 + kPage - 1 > q.at_min || (p.window > 0 && slot0 <= q.at_max - p.window);
      const int live = x.L - slot0;  // tokens of the page that are written
      uint32_t ksc[4];
      page_k_scales<D>(page, ksc);
      const int blk = D == 128 ? g : g >> 1;
      const uint4 vsc = *reinterpret_cast<const uint4*>(page + PageLayout<D>::kVs + (blk * 4 + c) * 16);
      const uint32_t vsw[4] = {vsc.x, vsc.y, vsc.z, vsc.w};
#pragma unroll 1  // (two steps side by side took 60 and 83 us)
      for (int i0 = 0; i0 < 4; i0 += MT) {
        float s[MT][NT][4];
        uint32_t ks[MT], vs[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          ks[i] = i0 == 0 ? ksc[i] : ksc[(i + MT) & 3];
          vs[i] = i0 == 0 ? vsw[i] : vsw[(i + MT) & 3];
        }
        page_scores<D, NT, MT>(page, i0, ks, q, s);
        scores_of<D, NT, MT, MOD>(p, q, slot0 + 16 * i0 + g, s);
        if (hides) mask_scores<D, NT, MT>(p, q, slot0 + 16 * i0 + g, s);
        // running maximum of each column, and the probabilities as P^T fragments
        bool grew = false;
        float now[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float t = fmaxf(s[0][nt][j], s[0][nt][j + 2]);
#pragma unroll
            for (int i = 1; i < MT; ++i) t = fmax3(t, s[i][nt][j], s[i][nt][j + 2]);
            t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 4));
            t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 8));
            t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 16));
            if constexpr (!MOD) t *= q.cs[nt][j];
            now[nt][j] = fmaxf(m[nt][j], t);
            grew |= now[nt][j] > m[nt][j];
          }
        if (__any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float alpha[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              alpha[j] = now[nt][j] == -INFINITY ? 1.0f : ex2_approx(m[nt][j] - now[nt][j]);
              m[nt][j] = now[nt][j];
              l[nt][j] *= alpha[j];
            }
#pragma unroll
            for (int t = 0; t < D / 16; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i) o[t][nt][i] *= alpha[i & 1];
          }
        }
        uint32_t pf[MT][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float b0 = kPShift - (m[nt][0] == -INFINITY ? 0.0f : m[nt][0]);
          const float b1 = kPShift - (m[nt][1] == -INFINITY ? 0.0f : m[nt][1]);
          const float f0 = MOD ? 1.0f : q.cs[nt][0], f1 = MOD ? 1.0f : q.cs[nt][1];
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            float p0, p1, p2, p3;
            ffma2(p0, p1, s[i][nt][0], s[i][nt][1], f0, f1, b0, b1);
            ffma2(p2, p3, s[i][nt][2], s[i][nt][3], f0, f1, b0, b1);
            p0 = ex2_approx(p0);
            p1 = ex2_approx(p1);
            p2 = ex2_approx(p2);
            p3 = ex2_approx(p3);
            ffma2(l[nt][0], l[nt][1], p0, p1, 1.0f, 1.0f, l[nt][0], l[nt][1]);
            ffma2(l[nt][0], l[nt][1], p2, p3, 1.0f, 1.0f, l[nt][0], l[nt][1]);
            pf[i][nt][0] = transpose8x8(pack_half2(p0, p1));
            pf[i][nt][1] = transpose8x8(pack_half2(p2, p3));
          }
        }
        // O^T += V^T P^T
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          uint32_t s01 = e4m3x2_to_half2(vs[i]), s89 = e4m3x2_to_half2(vs[i] >> 16);
          if (hides) {  // what lies behind the last token or before every window may be anything: P is 0, V must be finite
            const int t = 16 * (i0 + i) + 2 * c, gone = p.window > 0 ? q.at_min - p.window + 1 - slot0 : 0;
            if (t >= live || t < gone) s01 &= 0xFFFF0000u;
            if (t + 1 >= live || t + 1 < gone) s01 &= 0xFFFFu;
            if (t + 8 >= live || t + 8 < gone) s89 &= 0xFFFF0000u;
            if (t + 9 >= live || t + 9 < gone) s89 &= 0xFFFFu;
          }
          const uint8_t* va = page + PageLayout<D>::kVc + ((2 * (i0 + i)) * 8 + g) * (D / 2) + c * (D / 8);
          const uint8_t* vb = va + 8 * (D / 2);
          uint32_t a[2][D / 64], b[2][D / 64];  // tokens 2c, 2c + 1; 2c + 8, 2c + 9
          if constexpr (D == 128) {
            const uint4 y = *reinterpret_cast<const uint4*>(va), z = *reinterpret_cast<const uint4*>(vb);
            a[0][0] = y.x; a[0][1] = y.y; a[1][0] = y.z; a[1][1] = y.w;
            b[0][0] = z.x; b[0][1] = z.y; b[1][0] = z.z; b[1][1] = z.w;
          } else {
            const uint2 y = *reinterpret_cast<const uint2*>(va), z = *reinterpret_cast<const uint2*>(vb);
            a[0][0] = y.x; a[1][0] = y.y;
            b[0][0] = z.x; b[1][0] = z.y;
          }
#pragma unroll
          for (int w = 0; w < D / 64; ++w) {
            // codes of one channel and two neighbouring tokens side by side
            uint32_t e01[4], o01[4], e89[4], o89[4];
            e2m1x8_to_half2((a[0][w] & 0x0F0F0F0Fu) | ((a[1][w] << 4) & 0xF0F0F0F0u), e01);
            e2m1x8_to_half2(((a[0][w] >> 4) & 0x0F0F0F0Fu) | (a[1][w] & 0xF0F0F0F0u), o01);
            e2m1x8_to_half2((b[0][w] & 0x0F0F0F0Fu) | ((b[1][w] << 4) & 0xF0F0F0F0u), e89);
            e2m1x8_to_half2(((b[0][w] >> 4) & 0x0F0F0F0Fu) | (b[1][w] & 0xF0F0F0F0u), o89);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const uint32_t a0 = hmul2(e01[t], s01), a1 = hmul2(o01[t], s01);
              const uint32_t a2 = hmul2(e89[t], s89), a3 = hmul2(o89[t], s89);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_16816(o[4 * w + t][nt], a0, a1, a2, a3, pf[i][nt][0], pf[i][nt][1]);
            }
          }
        }
      }
      __syncwarp();
    }
    st.issue(p, unit_of, kPageBytes, k + L_::kStages);
  }
  if (!ok) st.drain(p, abort_flag);
  if (!shared) {
    if (x.end >= 0) finish();
    return;
  }
  // Four warps, one problem (a warp without units has an empty result): one
  // partial result, or the final one, eight columns at a time.
  if constexpr (!CLUSTER) x = find_unit<kCols, kPage>(p, prefix, cta_start);
  // (a cluster's partial results: O [cols][D], maxima, sums in the last warp's ring, behind its merge area)
  float* res = reinterpret_cast<float*>(smem + (kWarps - 1) * L_::kRing + 8 * 1024);
  static_assert(8 * 1024 + part_floats<D>(kCols) * 4 <= L_::kRing, "the cluster's result takes the ring's place");
  sums();
  if (g == 0) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        sm_m[warp * 32 + nt * 8 + 2 * c + j] = m[nt][j];
        sm_l[warp * 32 + nt * 8 + 2 * c + j] = l[nt][j];
      }
  }
  const bool begins = x.begin >= cta_start, whole = begins && x.end <= cta_end;
  float* part = p.part + static_cast<long long>(blockIdx.x * kWarps * 2 + begins) * part_floats<D>(kCols);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    if (x.r0 + nt * 8 > x.r1) break;  // no such columns
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int col = nt * 8 + 2 * c + j;
      float top = sm_m[col];
#pragma unroll
      for (int v = 1; v < kWarps; ++v) top = fmaxf(top, sm_m[v * 32 + col]);
      const float f = join_factor(m[nt][j], top);
      float* dst = reinterpret_cast<float*>(st.ring) + (2 * c + j) * kOStride + g * (D / 8);
#pragma unroll
      for (int t = 0; t < D / 16; ++t)
        *reinterpret_cast<float2*>(dst + 2 * t) = make_float2(o[t][nt][j] * f, o[t][nt][j + 2] * f);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 8 * D; i += kAttnThreads) {
      const int cc = i / D, d = i % D, col = nt * 8 + cc, r = x.r0 + col;
      if (r > x.r1) break;
      float acc = 0.0f, top = sm_m[col], sum = 0.0f;
#pragma unroll
      for (int v = 1; v < kWarps; ++v) top = fmaxf(top, sm_m[v * 32 + col]);
#pragma unroll
      for (int v = 0; v < kWarps; ++v) {
        acc += reinterpret_cast<const float*>(smem + v * L_::kRing)[cc * kOStride + d];
        sum += sm_l[v * 32 + col] * join_factor(sm_m[v * 32 + col], top);
      }
      if (!CLUSTER && whole) {
        const long long at = static_cast<long long>(x.row0 + r / p.G) * (p.g.heads * p.G) + x.h * p.G + r % p.G;
        p.o[at * D + d] = __float2bfloat16(out_o(acc, sum, p.v_up));
        if (d == 0) p.lse[at] = out_lse(top, sum, kPShift);
      } else {
        float* to = CLUSTER ? res : part;
        to[col * D + d] = acc;
        if (d == 0) {
          to[kCols * D + col] = top;
          to[kCols * D + kCols + col] = sum;
        }
      }
    }
  }
  if constexpr (CLUSTER) {
    cluster_sync();
    const uint32_t mine = smem_u32(res);
    for (int i = rank * kAttnThreads + threadIdx.x; i < (x.r1 - x.r0 + 1) * D; i += ranks * kAttnThreads) {
      const int col = i / D, d = i % D, r = x.r0 + col;
      float top = -INFINITY, m8[8], l8[8], o8[8];
#pragma unroll
      for (int c8 = 0; c8 < 8; ++c8) {
        if (c8 >= ranks) break;
        const uint32_t at = cluster_map(mine, c8);
        m8[c8] = cluster_ld(at + (kCols * D + col) * 4);
        l8[c8] = cluster_ld(at + (kCols * D + kCols + col) * 4);
        o8[c8] = cluster_ld(at + i * 4);
        top = fmaxf(top, m8[c8]);
      }
      float acc = 0.0f, sum = 0.0f;
#pragma unroll
      for (int c8 = 0; c8 < 8; ++c8) {
        if (c8 >= ranks) break;
        const float f = join_factor(m8[c8], top);
        acc = fmaf(o8[c8], f, acc);
        sum = fmaf(l8[c8], f, sum);
      }
      const long long at = static_cast<long long>(x.row0 + r / p.G) * (p.g.heads * p.G) + x.h * p.G + r % p.G;
      p.o[at * D + d] = __float2bfloat16(out_o(acc, sum, p.v_up));
      if (d == 0) p.lse[at] = out_lse(top, sum, kPShift);
    }
    cluster_sync();  // nobody leaves while its results are read
  }
}

// Joins the partial results: a block per (KV head, sequence, kRows columns), D
// / 4 lanes per column with four channels each.  A lane first takes one partial
// result's maximum and sum, shuffles make the factors; the loads of the first
// eight partial results' channels are in flight meanwhile.  The order of the
// additions is fixed.  Bound by latency: 9 us alone and cold (64 sequences of 8 KV
// heads), 7 behind the attention kernel.
template <int D, int NT>
__global__ void __launch_bounds__(kJoinThreads) kv_join_few_kernel(const KvAttnParams p) {
  constexpr int kCols = 8 * NT, kLanes = D / 4, kRows = kJoinThreads / kLanes, kPart = part_floats<D>(kCols), kAhead = 8;
  __shared__ int prefix[kJoinThreads + 1], scratch[kJoinThreads / 32];
  const int h = blockIdx.x, b = blockIdx.y, lane = threadIdx.x % kLanes;
  const int r = blockIdx.z * kRows + threadIdx.x / kLanes;
  // Small batches: everything but the results themselves before the wait.
  const bool early = p.g.B <= kJoinThreads;
  int row0, n, L, before, units;
  if (early) {
    plan_units<kCols, kPage>(p, prefix, scratch);
    before = prefix[b];
    units = prefix[p.g.B];
  }
  attn_seq(p, b, row0, n, L);
  const int R = n * p.G, first_r = static_cast<int>(blockIdx.z) * kRows;
  // (narrower tiles than the widest come alone)
  static_assert(NT < (D == 128 ? 2 : 4) || kCols % kRows == 0, "a block's columns lie in one tile");
  int skip = h * units_of<kCols, kPage>(p, n, L), count = 0;  // units of the sequence before this problem
  for (int r0 = 0; r0 <= first_r && r0 < R; r0 += kCols) {
    skip += count;
    count = span_of<kPage>(L, n, p.G, p.window, r0, min(R, r0 + kCols) - 1).count;
  }
  chain_next();
  chain_wait();
  if (first_r >= R) return;
  if (!early) {
    before = p.plan[b];
    units = p.plan[p.g.B];
  }
  const int per = warp_run(p, units), run = kWarps * per;
  const int begin = before + skip, end = begin + count;
  const int c0 = begin / run, c1 = (end - 1) / run, w0 = begin / per, w1 = (end - 1) / per;
  if (w0 == w1) return;  // finished in one warp
  // CTAs that worked on this problem alone left one result, the others (the
  // first, the last) one per warp
  const bool alone0 = begin <= c0 * run && end >= min(units, (c0 + 1) * run);
  const bool alone1 = end >= min(units, (c1 + 1) * run);
  if (c0 == c1 && alone0) return;  // finished in one CTA
  const int n0 = alone0 ? 1 : min(w1, c0 * kWarps + kWarps - 1) - w0 + 1;
  const int np = c0 == c1 ? n0 : n0 + (c1 - c0 - 1) + (alone1 ? 1 : w1 - c1 * kWarps + 1);
  auto part = [&](int i) -> const float* {
    int slot;
    if (i < n0) {
      slot = alone0 ? 2 * c0 * kWarps + (begin >= c0 * run) : 2 * (w0 + i) + (begin >= (w0 + i) * per);
    } else {  // behind the first CTA the problem has begun before
      const int c = c0 + 1 + (i - n0);
      slot = 2 * (c < c1 || alone1 ? min(c, c1) * kWarps : c1 * kWarps + (i - n0 - (c1 - c0 - 1)));
    }
    return p.part + static_cast<long long>(slot) * kPart;
  };
  const int col = min(r, R - 1) % kCols;  // lanes without a column repeat the last one
  auto channels = [&](int i) { return *reinterpret_cast<const float4*>(part(i) + col * D + 4 * lane); };
  float4 ahead[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) ahead[i] = i < np ? channels(i) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  // maxima and sums of the first kLanes results stay in the lanes
  const float m0 = lane < np ? part(lane)[kCols * D + col] : -INFINITY;
  const float l0 = lane < np ? part(lane)[kCols * D + kCols + col] : 0.0f;
  float top = m0;
  for (int i = kLanes + lane; i < np; i += kLanes) top = fmaxf(top, part(i)[kCols * D + col]);
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  float sum = 0.0f;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  auto add = [&](const float4& v, float f) {
    acc.x = fmaf(v.x, f, acc.x);
    acc.y = fmaf(v.y, f, acc.y);
    acc.z = fmaf(v.z, f, acc.z);
    acc.w = fmaf(v.w, f, acc.w);
  };
  for (int at = 0; at < np; at += kLanes) {  // np is the same in every lane of the block
    float f = 0.0f, l = 0.0f;
    if (at + lane < np) {
      f = join_factor(at == 0 ? m0 : part(at + lane)[kCols * D + col], top);
      l = at == 0 ? l0 : part(at + lane)[kCols * D + kCols + col];
    }
    sum = fmaf(l, f, sum);
    const int m = min(kLanes, np - at);
    int i = 0;
    if (at == 0) {
#pragma unroll
      for (; i < kAhead; ++i) add(ahead[i], __shfl_sync(0xFFFFFFFFu, f, i, kLanes));
    }
#pragma unroll 8
    for (; i < m; ++i) add(channels(at + i), __shfl_sync(0xFFFFFFFFu, f, i, kLanes));
  }
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if (r >= R) return;
  const long long out = static_cast<long long>(row0 + r / p.G) * (p.g.heads * p.G) + h * p.G + r % p.G;
  const __nv_bfloat162 lo = __floats2bfloat162_rn(out_o(acc.x, sum, p.v_up), out_o(acc.y, sum, p.v_up));
  const __nv_bfloat162 hi = __floats2bfloat162_rn(out_o(acc.z, sum, p.v_up), out_o(acc.w, sum, p.v_up));
  *reinterpret_cast<uint2*>(p.o + out * D + 4 * lane) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  if (lane == 0) p.lse[out] = out_lse(top, sum, kPShift);
}

// ---- gathered weight ----------------------------------------------------------

// The same streams over the K halves of the pages.  A page's columns, 8 NT at
// a time, are summed in column order, so the result does not depend on the
// split, and every slot has one writer.
template <int D, int NT, bool MOD>
__global__ void __launch_bounds__(kAttnThreads, 3) kv_weigh_kernel(const KvAttnParams p) {
  constexpr int kPart = PageLayout<D>::kKBytes, kCols = 8 * NT;
  using L_ = StreamSmem<kPart>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L_::kMisc);
  int* scratch = reinterpret_cast<int*>(smem + L_::kMisc + 16);
  int* prefix = reinterpret_cast<int*>(smem + L_::kPrefix);
  PageStream<kPart, L_::kStages> st;
  st.ring = smem + warp * L_::kRing;
  st.full = reinterpret_cast<uint64_t*>(smem + L_::kBars) + warp * L_::kStages;
  if (lane == 0) {
    for (int s = 0; s < L_::kStages; ++s) mbar_init(st.full + s, 1);
    if (warp == 0) *abort_flag = 0;
    fence_mbar_init();
  }
  chain_start();
  plan_units<kAll, kPage>(p, prefix, scratch);
  const int units = prefix[p.g.B], per = warp_run(p, units);
  st.start = min(units, (static_cast<int>(blockIdx.x) * kWarps + warp) * per);
  st.n = min(units, st.start + per) - st.start;
  if (st.n == 0) return;
  const auto unit_of = [&](int u) { return find_unit<kAll, kPage>(p, prefix, u); };
  st.look_up(p, unit_of, PageLayout<D>::kBytes, 0);
#pragma unroll 1
  for (int k = 0; k < L_::kStages; ++k) st.issue(p, unit_of, PageLayout<D>::kBytes, k);
  Unit x;
  x.end = -1;
  Columns<D, NT> q;
  float lse[NT][2];
  // columns r0 .. of problem x and their LSE in the log2 domain
  auto load = [&](int r0) {
    Unit y = x;
    y.r0 = r0;
    y.r1 = min(x.r1, r0 + kCols - 1);
    load_columns<D, NT, MOD>(p, y, q);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = r0 + nt * 8 + 2 * c + j;
        // a column that is none counts as seeing with infinite LSE: weight 0
        lse[nt][j] = INFINITY;
        if (r <= x.r1) {
          const float v = p.lse_in[static_cast<long long>(x.row0 + r / p.G) * (p.g.heads * p.G) + x.h * p.G + r % p.G];
          lse[nt][j] = v == -INFINITY ? INFINITY : v * kLog2Ef;  // -inf: the row sees nothing
        }
      }
  };
  bool ok = true;
#pragma unroll 1
  for (int k = 0; k < st.n && ok; ++k) {
    const int u = st.start + k;
    if (u >= x.end) {
      x = find_unit<kAll, kPage>(p, prefix, u);
      load(0);
    }
    const int slot0 = (x.first + (u - x.begin)) * kPage;
    const int reach = p.window > 0 ? max(0, x.L - x.n - p.window + 1) : 0;
    // the slots this lane will write: their old weights travel beside the page
    float* w = p.w + (static_cast<long long>(x.b) * p.g.heads + x.h) * p.W + slot0 + 16 * c + g;
    bool mine[2];
    float old[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int slot = slot0 + 16 * c + g + 8 * j;
      mine[j] = !x.none && slot >= reach && slot < x.L;
      if (mine[j] && slot >= p.W) {
        report_bad_index(p.g.status);
        mine[j] = false;
      }
      old[j] = mine[j] ? w[8 * j] : 0.0f;
    }
    float sum[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] = 0.0f;
    if (st.has(k)) {
      ok = st.wait(p, k, abort_flag, 64);
      if (!ok) break;
      const uint8_t* page = st.ring + (k % L_::kStages) * kPart;
      uint32_t ksc[4];
      page_k_scales<D>(page, ksc);
#pragma unroll 1
      for (int r0 = 0; r0 <= x.r1; r0 += kCols) {
        if (r0 > 0) load(r0);
        const bool hides = slot0 + kPage - 1 > q.at_min || (p.window > 0 && slot0 <= q.at_max - p.window);
#pragma unroll
        for (int i0 = 0; i0 < 4; i0 += 2) {
          float s[2][NT][4];
          const uint32_t ks[2] = {ksc[i0], ksc[i0 + 1]};
          page_scores<D, NT, 2>(page, i0, ks, q, s);
          scores_of<D, NT, 2, MOD>(p, q, slot0 + 16 * i0 + g, s);
          if (hides) mask_scores<D, NT, 2>(p, q, slot0 + 16 * i0 + g, s);
          auto add = [&](auto masked) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const float e = ex2_approx(fmaf(s[i][nt][j], MOD ? 1.0f : q.cs[nt][j & 1], -lse[nt][j & 1]));
                  // (a row whose LSE is no number hands none to a token that it does not see)
                  sum[2 * (i0 + i) + (j >> 1)] += masked.value && s[i][nt][j] == -INFINITY ? 0.0f : e;
                }
          };
          if (hides) add(std::true_type{});
          else add(std::false_type{});
        }
      }
      if (x.r1 >= kCols) load(0);
      __syncwarp();
    }
    st.issue(p, unit_of, PageLayout<D>::kBytes, k + L_::kStages);
    // sums over the four lanes of a token; lane c keeps those of group c
    float a[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float give = (c & 2) ? sum[i] : sum[4 + i], keep = (c & 2) ? sum[4 + i] : sum[i];
      a[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, 2);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float give = (c & 1) ? a[j] : a[2 + j], keep = (c & 1) ? a[2 + j] : a[j];
      const float all = keep + __shfl_xor_sync(0xFFFFFFFFu, give, 1);
      if (mine[j]) w[8 * j] = fmaf(p.decay, old[j], all);
    }
  }
  if (!ok) st.drain(p, abort_flag);
}

// ---- host -------------------------------------------------------------------

// Columns per tile in eights: as many as a KV head has, up to 16 (32 for D =
// 64, whose fragments take half the registers).
int tile_nt(int D, long long cols) {
  const int most = D == 128 ? 2 : 4;
  return cols >= 8 * most ? most : cols <= 8 ? 1 : static_cast<int>((cols + 7) / 8);
}

// Columns beyond which the kernel for prompts takes over, whose time hardly
// depends on them up to 512: three tiles for D = 128, two for D = 64.  Measured
// with 8 KV heads (us; this kernel, beyond the limits also the one for prompts):
//   sequences x tokens  D = 128: 48 columns, 64, 80, 96     D = 64: 64 columns, 80, 96, 128
//   1 x 8192     19  19 / 30    28 / 31    28 / 31           19   20 / 26    20 / 26    20 / 27
//   16 x 8192   122  157 / 191  193 / 195  227 / 196         90  126 / 159  129 / 159  160 / 161
//   64 x 4096   252  329 / 390  409 / 395  489 / 402        172  257 / 322  265 / 325  345 / 328
//   64 x 512     91  108 / 84   150 / 86   180 / 88          64  103 / 69   106 / 70   117 / 71
// Many short sequences cross over at the limits, long ones one or two tiles
// later; the lengths, which would tell them apart, are not known on the host.
bool is_prompt(int D, long long cols) { return cols > (D == 128 ? 48 : 64); }
long long tiles_of(int D, long long cols) {
  const int width = 8 * tile_nt(D, cols);
  return (cols + width - 1) / width;
}

template <int D, int NT, bool MOD>
cudaError_t launch_attn(const KvAttnParams& p, int cluster, cudaStream_t s) {
  using L_ = StreamSmem<PageLayout<D>::kBytes>;
  if (cluster > 0) {
    const cudaError_t e = allow_smem<kv_attn_kernel<D, NT, MOD, true>>(L_::bytes(0));
    if (e != cudaSuccess) return e;
    const int tiles = (p.max_new * p.G + 8 * NT - 1) / (8 * NT);
    return launch_chained_cluster(kv_attn_kernel<D, NT, MOD, true>, dim3(p.g.B * p.g.heads * tiles * cluster), cluster,
                                  kAttnThreads, L_::bytes(0), s, p);
  }
  cudaError_t e = allow_smem<kv_attn_kernel<D, NT, MOD, false>>(L_::bytes(kMaxKvBatch));
  if (e != cudaSuccess) return e;
  e = launch_chained(kv_attn_kernel<D, NT, MOD, false>, dim3(p.ctas), kAttnThreads, L_::bytes(p.g.B), s, p);
  if (e != cudaSuccess) return e;
  const int rows = kJoinThreads / (D / 4);
  return launch_chained(kv_join_few_kernel<D, NT>, dim3(p.g.heads, p.g.B, (p.max_new * p.G + rows - 1) / rows), kJoinThreads, 0,
                        s, p);
}

template <int D, int NT, bool MOD>
cudaError_t launch_weigh(const KvAttnParams& p, cudaStream_t s) {
  using L_ = StreamSmem<PageLayout<D>::kKBytes>;
  const cudaError_t e = allow_smem<kv_weigh_kernel<D, NT, MOD>>(L_::bytes(kMaxKvBatch));
  if (e != cudaSuccess) return e;
  return launch_chained(kv_weigh_kernel<D, NT, MOD>, dim3(p.ctas), kAttnThreads, L_::bytes(p.g.B), s, p);
}

// f with the tile width and the kind of score as template arguments.
template <int D, typename F>
cudaError_t by_tile(int nt, bool mod, F&& f) {
  using T = std::true_type;
  using N = std::false_type;
  if (nt == 1) return mod ? f(std::integral_constant<int, 1>{}, T{}) : f(std::integral_constant<int, 1>{}, N{});
  if (D == 128 || nt == 2) return mod ? f(std::integral_constant<int, 2>{}, T{}) : f(std::integral_constant<int, 2>{}, N{});
  if constexpr (D == 64) {
    if (nt == 3) return mod ? f(std::integral_constant<int, 3>{}, T{}) : f(std::integral_constant<int, 3>{}, N{});
    return mod ? f(std::integral_constant<int, 4>{}, T{}) : f(std::integral_constant<int, 4>{}, N{});
  }
  return cudaErrorInvalidValue;
}

int attn_ctas(int D, int nt) { return sm_count() * resident(D, nt); }

// CTAs of the cluster that takes one problem, or 0 for the even split.  The
// widest cluster with which all problems are on the GPU at once, where no warp
// gets more than 8 pages of a sequence as long as the table is wide, or 16 where
// the clusters fill a quarter of the GPU at most.  Measured against the even
// split (D = 128, 4 query heads per KV head, all lengths equal, us): 8 problems of
// 64 pages 8.0 / 13.5, of 512 25.0 / 29.5; 32 of 256 25.0 / 26.6, of 512 44.6 /
// 40.8; 128 of 32 15.6 / 19.6, of 64 24.8 / 24.8, of 128 44.7 / 38.7.
int cluster_of(int D, int nt, long long problems, int max_pages) {
  const int room = attn_ctas(D, nt);
  if (problems > room) return 0;
  int c = 1;  // one page per warp cannot be split further
  while (c < 8 && problems * c * 2 <= room && c * kWarps < max_pages) c *= 2;
  const int most = problems * c * 4 <= room ? 16 : 8;
  return max_pages <= c * kWarps * most ? c : 0;
}

size_t attn_workspace(int D, int B, int heads, int max_pages, long long cols) {
  if (is_prompt(D, cols)) return prompt_workspace(D);
  if (cluster_of(D, tile_nt(D, cols), tiles_of(D, cols) * B * heads, max_pages) > 0) return 0;
  return plan_bytes() + static_cast<size_t>(attn_ctas(D, tile_nt(D, cols))) * kWarps * 2 * (8 * tile_nt(D, cols)) * (D + 2) * sizeof(float);
}

// Limits of the sizes, which are positive.
int check_sizes(int heads, int B, int max_pages, int group, int max_new) {
  if (B > kMaxKvBatch || max_pages > kMaxSlots / kPage) return FP4ATTN_ERR_UNSUPPORTED;
  if (static_cast<long long>(heads) * group > 65535) return FP4ATTN_ERR_UNSUPPORTED;
  const long long cols = static_cast<long long>(max_new) * group;
  if (cols > (1ll << 24)) return FP4ATTN_ERR_UNSUPPORTED;
  // units of all tiles must stay within 32 bits, rounded up to whole runs too
  if (static_cast<long long>(B) * heads * ((cols + 7) / 8) >= (1ll << 30) / max_pages) return FP4ATTN_ERR_UNSUPPORTED;
  return FP4ATTN_OK;
}

// Checks shared by attention and weights.
int check_attn(const fp4attn_kv_cache_t* c, const fp4attn_kv_batch_t* b, const void* q, long long q_row,
               long long q_head, int group, int max_new, float scale, float cap, int window) {
  int st = check_kv_cache(c);
  if (st == FP4ATTN_OK) st = check_kv_batch(b, true);
  if (st != FP4ATTN_OK) return st;
  if (group <= 0 || max_new < 0 || max_new > b->T || window < 0) return FP4ATTN_ERR_INVALID_ARG;
  if (!b->cu && max_new != b->T / b->B) return FP4ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || scale <= 0.0f || !(cap >= 0.0f && cap <= kMaxCap)) return FP4ATTN_ERR_INVALID_ARG;
  const float up = scale * ldexpf(1.0f, c->k_exp);  // what the kernels multiply by
  if (!std::isnormal(up) || (cap > 0.0f && !std::isfinite(up / cap))) return FP4ATTN_ERR_INVALID_ARG;
  if (b->T > 0 && (!q || !aligned16(q) || ((q_row | q_head) & 7))) return FP4ATTN_ERR_INVALID_ARG;
  return check_sizes(c->heads, b->B, b->max_pages, group, max_new);
}

}  // namespace
}  // namespace fp4attn

using namespace fp4attn;

extern "C" int fp4attn_kv_attention_workspace_bytes(int heads, int D, int B, int max_pages, int group, int max_new,
                                                    size_t* bytes) {
  if (heads <= 0 || B <= 0 || max_pages <= 0 || group <= 0 || max_new < 0 || !bytes) return FP4ATTN_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return FP4ATTN_ERR_UNSUPPORTED;
  const int st = check_sizes(heads, B, max_pages, group, max_new);
  if (st != FP4ATTN_OK) return st;
  *bytes = attn_workspace(D, B, heads, max_pages, static_cast<long long>(group) * max_new);
  return FP4ATTN_OK;
}

extern "C" int fp4attn_kv_attention(const fp4attn_kv_cache_t* c, const fp4attn_kv_batch_t* b, const void* q,
                                    long long q_row_stride, long long q_head_stride, int group, int max_new,
                                    float softmax_scale, float softcap, int window, const float* slopes, void* o,
                                    float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  const int st = check_attn(c, b, q, q_row_stride, q_head_stride, group, max_new, softmax_scale, softcap, window);
  if (st != FP4ATTN_OK) return st;
  if (b->T == 0 || max_new == 0) return FP4ATTN_OK;
  if (!o || !lse || !aligned16(o)) return FP4ATTN_ERR_INVALID_ARG;
  const long long cols = static_cast<long long>(group) * max_new;
  const int nt = tile_nt(c->D, cols);
  const size_t need = attn_workspace(c->D, b->B, c->heads, b->max_pages, cols);
  if (need > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < need)) return FP4ATTN_ERR_INVALID_ARG;
  DeviceStatus* ds = device_status_ptr();
  if (!ds) return FP4ATTN_ERR_CUDA;
  KvAttnParams p{};
  p.g = kv_geom(c, b, ds);
  p.pages = c->pages;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_row = q_row_stride;
  p.q_head = q_head_stride;
  p.G = group;
  p.max_new = max_new;
  p.scale = softmax_scale * ldexpf(1.0f, c->k_exp);
  p.cap = softcap;
  p.window = window < kMaxWindow ? window : kMaxWindow;
  p.slopes = slopes;
  p.v_up = ldexpf(1.0f, c->v_exp);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  if (need > 0) {
    p.plan = static_cast<int*>(workspace);
    p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + plan_bytes());
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (is_prompt(c->D, cols)) {
    p.ctas = prompt_runs();
    return cuda_status(launch_prompt(p, c->D, s));
  }
  p.ctas = attn_ctas(c->D, nt);
  const int cluster = cluster_of(c->D, nt, tiles_of(c->D, cols) * b->B * c->heads, b->max_pages);
  const bool mod = softcap > 0.0f || slopes;
  cudaError_t e;
  const auto go = [&](auto d) {
    return by_tile<d.value>(nt, mod, [&](auto n, auto m) { return launch_attn<d.value, n.value, m.value>(p, cluster, s); });
  };
  e = c->D == 128 ? go(std::integral_constant<int, 128>{}) : go(std::integral_constant<int, 64>{});
  return cuda_status(e);
}

extern "C" int fp4attn_kv_accumulate(const fp4attn_kv_cache_t* c, const fp4attn_kv_batch_t* b, const void* q,
                                     long long q_row_stride, long long q_head_stride, int group, int max_new,
                                     float softmax_scale, float softcap, int window, const float* slopes,
                                     const float* lse, float* weights, int weights_stride, float decay,
                                     void* stream) {
  const int st = check_attn(c, b, q, q_row_stride, q_head_stride, group, max_new, softmax_scale, softcap, window);
  if (st != FP4ATTN_OK) return st;
  if (!std::isfinite(decay)) return FP4ATTN_ERR_INVALID_ARG;
  if (b->T == 0 || max_new == 0) return FP4ATTN_OK;
  if (!lse || !weights || weights_stride <= 0) return FP4ATTN_ERR_INVALID_ARG;
  if (weights_stride > kMaxSlots) return FP4ATTN_ERR_UNSUPPORTED;
  DeviceStatus* ds = device_status_ptr();
  if (!ds) return FP4ATTN_ERR_CUDA;
  KvAttnParams p{};
  p.g = kv_geom(c, b, ds);
  p.pages = c->pages;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_row = q_row_stride;
  p.q_head = q_head_stride;
  p.G = group;
  p.max_new = max_new;
  p.scale = softmax_scale * ldexpf(1.0f, c->k_exp);
  p.cap = softcap;
  p.window = window < kMaxWindow ? window : kMaxWindow;
  p.slopes = slopes;
  p.lse_in = lse;
  p.w = weights;
  p.W = weights_stride;
  p.decay = decay;
  p.ctas = sm_count() * 3;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool mod = softcap > 0.0f || slopes;
  const int nt = tile_nt(c->D, static_cast<long long>(group) * max_new);
  cudaError_t e;
  const auto go = [&](auto d) {
    return by_tile<d.value>(nt, mod, [&](auto n, auto m) { return launch_weigh<d.value, n.value, m.value>(p, s); });
  };
  e = c->D == 128 ? go(std::integral_constant<int, 128>{}) : go(std::integral_constant<int, 64>{});
  return cuda_status(e);
}
