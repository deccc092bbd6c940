// Attention of many queries over the 4-bit key/value cache (prompts, chunks of
// prompts): the same operator as kvattn.cu, bound by its products instead of
// by reading the cache.
//
// A KV head's group of G query heads times n tokens gives the rows of one
// problem; a pair of CTAs (a cluster, on the two SMs of a TPC) takes 512 of
// them, in two tiles of 256, over a run of 128-token blocks of the cache (units
// numbered and split evenly as in kvattn.cu, so that no pair waits for another's
// longer problem; what is split is joined by the same kind of second kernel).
// The MMAs are cta_group::2: M = 256 rows, 128 of each CTA, against a K or V^T
// operand of which each CTA holds half, so that a block is converted once for
// 512 rows and every SM stores and reads half of it.  (With one CTA per problem
// the kernel was bound by shared memory: 64 KB of converted operands per block
// and 128 bytes of Q and K per cycle left the tensor cores 40% busy.)  Roles
// (512 threads per CTA):
//   warps 0-3, 4-7  one warpgroup per tile, one thread per row: stages its query
//              row in shared memory (fp16, scaled by a power of two that puts
//              the row's largest element in [2^13, 2^14): exact as in
//              kvattn.cu), turns S into probabilities, rescales O when the
//              reference maximum moves by more than 2^12, writes the result.
//   warps 8-11 turn the pages into the MMAs' operands: K rows of half of each
//              page's tokens, V^T rows of half of the channels (pieces of codes of
//              four tokens, two tokens side by side), both exact, 128-byte
//              swizzled, four stages.
//   warp 12    of the first CTA issues tcgen05.mma (kind::f16): S = Q K^T from
//              shared memory, O += P V with P as fp16 in TMEM, over the columns
//              S came in.
//   warp 13    of the second CTA passes on to it that operands are in place
//              there: what one CTA wrote to its shared memory for an MMA of the
//              other needs a release at cluster scope, which costs the warp about
//              1300 cycles, and this one has the time.
// K and V of a block are handed over together: the hand-offs (a proxy fence and a
// release, which wait for the loads on their way) are what the operands' warps
// have least time for (955 us where one for each took 1000).
// S, P and the products go page by page (64 tokens): a warpgroup alternates
// between its tile's two pages, and while it works on one the tensor core takes
// the other's P, refills its S, and serves the other tile.  TMEM: S 2 x 128 columns, O 2 x D.
// At the end of a problem the next one's queries are staged before the results
// are written, so that its first scores are made meanwhile.
//
// Measured (of 1895 TFLOP/s, a large library product of bf16): D = 128, 2
// sequences of 16384 tokens, 2048 of them new, 40 query heads over 8: 911 us,
// 1413 TFLOP/s, 75%.  The tensor core waits 39% of the time, for the hand-offs of
// a page's chain S -> P -> products; no unit is full (exponentials 31%, ALUs 31%,
// issue slots 47%).  D = 64, 7 prompts of 3333 rows in all, 16 query heads over 4,
// window 1024, capped: 70 us (without the cap 52), of which 31 remain with a
// window of one token: start, join, and for each of the 2
// or 3 problems of a pair its queries, first scores and results.
//
// P is held as 2^(15 - slack) p against a reference maximum that may lag by
// 2^slack (moving it costs a pass over O in TMEM), so that its largest value is
// 2^15.  fp16 is off by 2^-25 at most down there, 2^(slack - 40) of the
// reference, and drops what is smaller; the sum of P is kept of the fp32 values
// before they are rounded.  L tokens together then lose L 2^(slack - 40) of the
// largest |V| at most: the slack is 12 up to 2^17 tokens, where that is 2^-11
// (a quarter of bf16's rounding), and one less with every further doubling, down
// to 1.  (For all lengths alike, a slack of 8 took 984 us in place of 951, of 4 992.)
#include <type_traits>

#include "kvattn.cuh"

namespace fp4attn {
namespace {

constexpr int kRowsPair = 512;
constexpr int kStages = 4;  // of K and V
constexpr int kSeen = 8;    // blocks whose pages the rows' warps may still ask about
constexpr int kBlockKeys = 128;
constexpr int kWarpDq = 8, kWarpMma = 12;
// Four warpgroups: two for the rows, one for the operands, one whose first
// warp issues the MMAs.  The rows' threads hold 64 scores each, and what turns
// them into P, so registers go from the others to them: 2 x 176 + 96 + 64 = 4 x
// 128.  (32 bytes a thread are spilled.)
constexpr int kPromptThreads = 512;
constexpr int kRegsRows = 176, kRegsOperands = 96, kRegsMma = 64;
static_assert(2 * kRegsRows + kRegsOperands + kRegsMma == 4 * 128, "registers of the launch");
constexpr float kPMax = 15.0f;  // P is below 2^kPMax
// How far the reference maximum of a sequence of L tokens may lag, in powers of two.
__device__ __forceinline__ float slack_of(int L) { return static_cast<float>(min(12, max(1, __clz(L - 1) - 3))); }
constexpr uint32_t kColS = 0, kColO = 256;  // tile t: S at 128 t, O at 256 + 128 t

template <int D>
struct PromptSmem {
  static constexpr int kQTile = 128 * D * 2;
  static constexpr int kKTile = kPage * D * 2;             // this CTA's page of the block
  static constexpr int kVTile = (D / 2) * kBlockKeys * 2;  // this CTA's channels
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + 2 * kQTile;
  static constexpr int kV = kK + kStages * kKTile;
  static constexpr int kBars = kV + kStages * kVTile;
  static constexpr int kNumBars = 2 + 3 * kStages + 4 + 4 + 4 + 1 + kStages + kSeen;
  static constexpr int kMisc = kBars + kNumBars * 8;
  static constexpr int kPrefix = kMisc + 128;
  static int bytes(int B) {
    const int n = kPrefix + (B + 1) * 4 + 1024;
    return n > 120 * 1024 ? n : 120 * 1024;  // one CTA per SM: it allocates all of TMEM
  }
};

// fp16 A and B, fp32 accumulation, both operands K-major
__host__ __device__ constexpr uint32_t idesc_f16(uint32_t M, uint32_t N) {
  return (1u << 4) | ((N >> 3) & 0x3Fu) << 17 | ((M >> 4) & 0x1Fu) << 24;
}
// Arrive on bar in both CTAs once every operation issued so far completes.
__device__ __forceinline__ void tc_commit2(uint32_t bar) {
  asm volatile(
      "{\n.reg .pred e;\n.reg .b16 m;\nmov.b16 m, 3;\nelect.sync _|e, 0xffffffff;\n"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n}\n" ::"r"(bar)
      : "memory");
}

// The issuing warp shares its scheduler with two of the rows' warps, which leave
// it one slot in three or four, so what it executes per MMA (32 to 64 cycles
// apart) has to be little.  Descriptors are constants plus the address of shared
// memory, added to their low word in the batch (added outside, for every tile
// and page, they are kept in registers, and spill).
__host__ __device__ constexpr uint32_t desc_low(uint32_t offset) { return (offset >> 4) | (1u << 16); }
constexpr uint32_t kDescHigh = 64u | (1u << 14) | (2u << 29);

// M = 256 over the CTA pair: A and D rows 128 in each CTA (the same offsets), B
// rows N / 2 in each.  The whole warp comes here with operands that are
// the same in every lane; one, elected once per batch, issues the MMAs of a batch
// and the commit that reports them to both CTAs.  (Stages as template arguments
// made four copies of the loop over the blocks: 964 us in place of 928.)
// S of tile T, page PG (32 key rows of the page in each CTA).  q: of the queries'
// tiles in shared memory, k: of the stage, addresses / 16, the same in both CTAs
template <int D, int T, int PG>
__device__ __forceinline__ void issue_qk(uint32_t q, uint32_t k, uint32_t s_full) {
  using L_ = PromptSmem<D>;
  constexpr uint32_t d = kColS + 128 * T + kPage * PG, id = idesc_f16(256, kPage);
  constexpr uint32_t a = desc_low(T * L_::kQTile), b = desc_low(PG * (32 * 128));
  // to the next 64 channels
  constexpr uint64_t da = 128 * 128 / 16 - 6, db = kPage * 128 / 16 - 6;
  if constexpr (D == 128) {
    asm volatile(
      "{\n.reg .pred e, f, t;\n.reg .b64 a, b;\n.reg .b32 lo;\n.reg .b16 m;\nelect.sync _|e, 0xffffffff;\n"
      "setp.ne.b32 f, 0, 0;\nsetp.eq.b32 t, 0, 0;\nadd.u32 lo, %7, %1;\nmov.b64 a, {lo, %9};\nadd.u32 lo, %8, %2;\nmov.b64 b, {lo, %9};\n"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, f;\n"
      "add.s64 a, a, 2;\nadd.s64 b, b, 2;\n"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, t;\n"
      "add.s64 a, a, 2;\nadd.s64 b, b, 2;\n"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, t;\n"
      "add.s64 a, a, 2;\nadd.s64 b, b, 2;\n"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, t;\n"
      "add.s64 a, a, %4;\nadd.s64 b, b, %5;\n"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, t;\n"
      "add.s64 a, a, 2;\nadd.s64 b, b, 2;\n"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, t;\n"
      "add.s64 a, a, 2;\nadd.s64 b, b, 2;\n"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, t;\n"
      "add.s64 a, a, 2;\nadd.s64 b, b, 2;\n"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, t;\n"
      "mov.b16 m, 3;\n@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%6 + %10], m;\n}\n"
        ::"r"(d), "n"(a), "n"(b), "r"(id), "n"(da), "n"(db), "r"(s_full), "r"(q), "r"(k), "n"(kDescHigh), "n"(8 * (2 * T + PG))
        : "memory");
  } else {
    asm volatile(
      "{\n.reg .pred e, f, t;\n.reg .b64 a, b;\n.reg .b32 lo;\n.reg .b16 m;\nelect.sync _|e, 0xffffffff;\n"
      "setp.ne.b32 f, 0, 0;\nsetp.eq.b32 t, 0, 0;\nadd.u32 lo, %7, %1;\nmov.b64 a, {lo, %9};\nadd.u32 lo, %8, %2;\nmov.b64 b, {lo, %9};\n"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, f;\n"
      "add.s64 a, a, 2;\nadd.s64 b, b, 2;\n"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, t;\n"
      "add.s64 a, a, 2;\nadd.s64 b, b, 2;\n"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, t;\n"
      "add.s64 a, a, 2;\nadd.s64 b, b, 2;\n"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, t;\n"
      "mov.b16 m, 3;\n@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%6 + %10], m;\n}\n"
        ::"r"(d), "n"(a), "n"(b), "r"(id), "n"(da), "n"(db), "r"(s_full), "r"(q), "r"(k), "n"(kDescHigh), "n"(8 * (2 * T + PG))
        : "memory");
  }
}
// O of tile T += P V of page PG.  v: of the stage
template <int D, int T, int PG>
__device__ __forceinline__ void issue_pv(uint32_t v, uint32_t o_full, bool acc) {
  constexpr uint32_t d = kColO + 128 * T, a = kColS + 128 * T + kPage * PG, id = idesc_f16(256, D);
  constexpr uint32_t b = desc_low(PG * ((D / 2) * 128));
  asm volatile(
      "{\n.reg .pred e, f, t;\n.reg .b64 b;\n.reg .b32 a, lo;\n.reg .b16 m;\nelect.sync _|e, 0xffffffff;\n"
      "setp.ne.b32 f, %4, 0;\nsetp.eq.b32 t, 0, 0;\nmov.b32 a, %1;\nadd.u32 lo, %6, %2;\nmov.b64 b, {lo, %7};\n"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [a], b, %3, f;\n"
      "add.s32 a, a, 8;\nadd.s64 b, b, 2;\n"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [a], b, %3, t;\n"
      "add.s32 a, a, 8;\nadd.s64 b, b, 2;\n"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [a], b, %3, t;\n"
      "add.s32 a, a, 8;\nadd.s64 b, b, 2;\n"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [a], b, %3, t;\n"
      "mov.b16 m, 3;\n@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%5 + %8], m;\n}\n"
      ::"r"(d), "r"(a), "n"(b), "r"(id), "r"(acc ? 1 : 0), "r"(o_full), "r"(v), "n"(kDescHigh), "n"(8 * (2 * T + PG))
      : "memory");
}
__device__ __forceinline__ void tmem_alloc2(uint32_t* dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(ncols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc2(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// One lane arrives on a barrier of the first CTA (its address there: bar), from
// either CTA: the warp's P is in TMEM.  Between tcgen05 operations of different
// threads it is the tcgen05 fences (before this, and after the wait) that order,
// and the barrier has to say no more than that it was reached.
__device__ __forceinline__ void arrive_tmem(uint32_t bar) {
  asm volatile(
      "{\n.reg .pred e;\nelect.sync _|e, 0xffffffff;\n"
      "@e mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n}\n" ::"r"(bar)
      : "memory");
}
// One lane arrives on a barrier of its own CTA: what the warp wrote to shared
// memory before, and fenced for the MMAs' proxy, is in place there.
__device__ __forceinline__ void arrive_smem(uint32_t bar) {
  __syncwarp();
  asm volatile(
      "{\n.reg .pred e;\nelect.sync _|e, 0xffffffff;\n"
      "@e mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];\n}\n" ::"r"(bar)
      : "memory");
}
// The same from the second CTA on a barrier of the first: also of what the warp
// has acquired from a barrier of its own CTA.
__device__ __forceinline__ void arrive_first(uint32_t bar) {
  __syncwarp();
  asm volatile(
      "{\n.reg .pred e;\nelect.sync _|e, 0xffffffff;\n"
      "@e mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];\n}\n" ::"r"(bar)
      : "memory");
}
// The issuing warp's waits, on arrivals from both CTAs: with the operands' writes
// (SMEM), or for tcgen05 operations alone.
template <bool SMEM>
__device__ __forceinline__ bool pair_try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  if constexpr (SMEM)
    asm volatile(
        "{\n.reg .pred p;\n"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        "selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
  else
    asm volatile(
        "{\n.reg .pred p;\n"
        "mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n"
        "selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
  return ok != 0;
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// 16-byte unit u of a 128-byte row r of a 128-byte-swizzled tile
__device__ __forceinline__ uint32_t swz(int r, int u) { return static_cast<uint32_t>(r * 128 + ((u ^ (r & 7)) << 4)); }

template <int D, bool MOD>
__global__ void __launch_bounds__(kPromptThreads, 1) kv_prompt_kernel(const KvAttnParams p) {
  using L_ = PromptSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // the first CTA's: arrivals of its own warps and of the other CTA's, for K and V of the warp there that passes them on
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + L_::kBars);  // [2] tiles, per segment
  uint64_t* kv_full = q_full + 2;                                   // [kStages]
  uint64_t* p_full = kv_full + kStages;  // [2 tiles][2 pages]; of the warps of both
  // each CTA's own: commits
  uint64_t* k_empty = p_full + 4;
  uint64_t* v_empty = k_empty + kStages;
  uint64_t* s_full = v_empty + kStages;  // [2 tiles][2 pages]
  uint64_t* o_full = s_full + 4;         // [2 tiles][2 pages]
  uint64_t* drain = o_full + 4;
  // the second CTA's: arrivals of its own warps
  uint64_t* kv_mine = drain + 1;
  // each CTA's own: seen[k % kSeen] is written
  uint64_t* seen_full = kv_mine + kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L_::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L_::kMisc + 4);
  // whether the pages of block k count, a bit each, at [k % kSeen]: block k + 8 is staged only after every row is done with k
  uint8_t* seen = smem + L_::kMisc + 8;
  int* scratch = reinterpret_cast<int*>(smem + L_::kMisc + 32);  // 16 ints
  int* prefix = reinterpret_cast<int*>(smem + L_::kPrefix);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  const int rank = cluster_rank();
  const uint32_t first_bars = cluster_map(smem_u32(q_full), 0);  // the first CTA's barriers, in the order above
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + i, 8);  // one arrival per warp, four in each CTA
      for (int h = 0; h < 2; ++h) {
        mbar_init(p_full + 2 * i + h, 8);
        mbar_init(s_full + 2 * i + h, 1);
        mbar_init(o_full + 2 * i + h, 1);
      }
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(kv_full + i, 5);  // four warps and the one that passes on
      mbar_init(kv_mine + i, 4);
      mbar_init(k_empty + i, 1);
      mbar_init(v_empty + i, 1);
    }
    for (int i = 0; i < kSeen; ++i) mbar_init(seen_full + i, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) tmem_alloc2(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the other CTA's barriers are there
  tc_fence_after();
  // (an allocation of all 512 columns begins at column 0)
  const uint32_t tmem_base = *tmem_slot;
  chain_wait();
  chain_next();
  plan_units<kRowsPair, kBlockKeys>(p, prefix, scratch);
  const int units = prefix[p.g.B], per = run_length(units, p.ctas);
  const int pair = blockIdx.x >> 1;
  const int start = min(units, pair * per), end = min(units, start + per);
  if (start >= end) {  // (both CTAs)
    if (rank == 0 && threadIdx.x == 0) split_of(p, pair)->last = -1;
    if (warp == kWarpMma) tmem_dealloc2(tmem_base, 512);
    return;
  }
  if (warp < kWarpDq) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsRows));
    // ---------------------------------------------------------------- softmax
    const int t = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = lane_base + kColS + 128 * t, to = lane_base + kColO + 128 * t;
    int kc = 0, ks = 0;  // blocks of this tile and of the CTA so far
    bool ok = true;
    // the segment at hand: units [u, seg_end) of problem x
    Unit x;
    int u = start, seg_end = start;
    // The next segment from u on that has rows of this tile.
    auto seek = [&]() {
      while (u < end) {
        x = find_unit<kRowsPair, kBlockKeys>(p, prefix, u);
        seg_end = min(end, x.end);
        if (x.r0 + 256 * t <= x.r1) return true;
        ks += seg_end - u;
        u = seg_end;
      }
      return false;
    };
    // this thread's row; rows past the last repeat it and are not written
    const int col = 256 * t + 128 * rank + row;
    const uint4* src = nullptr;
    auto locate_q = [&]() {
      const int r = min(x.r1, x.r0 + col);
      src = reinterpret_cast<const uint4*>(p.q + (x.row0 + r / p.G) * p.q_row + (x.h * p.G + r % p.G) * p.q_head);
    };
    // To shared memory; returns the power of two to undo.  (The row is read twice:
    // held in registers it costs the loop over the pages more than it saves here.)
    auto stage_q = [&]() {
      uint32_t m2 = 0;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const uint4 v = __ldg(src + i);
        m2 = __vmaxu2(__vmaxu2(__vmaxu2(m2, v.x & 0x7FFF7FFFu), v.y & 0x7FFF7FFFu),
                      __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
      }
      const int e = max(static_cast<int>(max(m2 & 0xFFFFu, m2 >> 16) >> 7), 20);
      const float up = pow2i(140 - e);
      uint8_t* qs = smem + L_::kQ + t * L_::kQTile;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const uint4 v = __ldg(src + i);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t h[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          h[j] = half2_of(__uint_as_float(w[j] << 16) * up, __uint_as_float(w[j] & 0xFFFF0000u) * up);
        *reinterpret_cast<uint4*>(qs + (i >> 3) * (128 * 128) + swz(row, i & 7)) = make_uint4(h[0], h[1], h[2], h[3]);
      }
      fence_proxy_async_smem();
      if (rank == 0) arrive_smem(smem_u32(q_full + t));
      else arrive_first(first_bars + 8 * t);
      return pow2i(e - 140);
    };
    float down = 1.0f;
    bool any = seek();
    if (any) {
      locate_q();
      down = stage_q();
    }
    while (any) {
      const int nblk = seg_end - u;
      const bool real = x.r0 + col <= x.r1;
      const int r = min(x.r1, x.r0 + col), at = x.L - x.n + r / p.G;
      // log2-domain score per unit of S (with a cap: s / cap)
      const float cs = score_factor<MOD>(p, down);
      const float slope = MOD && p.slopes ? p.slopes[x.h * p.G + r % p.G] * kLog2Ef : 0.0f;
      const float cap = p.cap * kLog2Ef;
      const float slack = slack_of(x.L), shift = kPMax - slack;
      // S (in TMEM at tp, and in v) -> log2-domain scores; dist: of the first one
      // from the query.  A NaN stays one on either way through the cap.  Scores
      // that are not far below their cap are rare and go through TMEM, so that
      // their longer way is one short loop and not 64 times in the instruction cache.
      auto log2_scores = [&](float (&v)[2][32], uint32_t tp, int dist) {
#pragma unroll
        for (int i = 0; i < 64; i += 2) fmul2(v[i >> 5][i & 31], v[i >> 5][(i & 31) + 1], v[i >> 5][i & 31], v[i >> 5][(i & 31) + 1], cs, cs);
        if (p.cap > 0.0f) {
          float big = 0.0f;
#pragma unroll
          for (int i = 0; i < 64; i += 2) big = fmax3(big, fabsf(v[i >> 5][i & 31]), fabsf(v[i >> 5][(i & 31) + 1]));
          if (__all_sync(0xFFFFFFFFu, big < kTanhTiny)) {
#pragma unroll
            for (int i = 0; i < 64; i += 2) tanh2_tiny(v[i >> 5][i & 31], v[i >> 5][(i & 31) + 1], cap);
          } else {
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              float s[16];
              uint32_t w[16];
              tmem_ld16(tp + 16 * c, s);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(cap * tanh_acc(s[i] * cs));
              tmem_st16(tp + 16 * c, w);
            }
            tmem_wait_st();
            tmem_ld32(tp, v[0]);
            tmem_ld32(tp + 32, v[1]);
            tmem_wait_ld();
          }
        }
        if (p.slopes) {
          const float far = static_cast<float>(dist);
#pragma unroll
          for (int i = 0; i < 64; ++i) v[i >> 5][i & 31] = fmaf(-slope, far - static_cast<float>(i), v[i >> 5][i & 31]);
        }
      };
      // the warp's rows: the first and the last slot they sit at
      const int at_lo = __reduce_min_sync(0xFFFFFFFFu, at), at_hi = __reduce_max_sync(0xFFFFFFFFu, at);
      float m = -INFINITY, l = 0.0f;
      uint32_t pages = 3u;  // of the block at hand: bit i, page i counts
      // page by page: while this warpgroup works on one page's scores, the tensor
      // core takes the other's P and refills its S
      for (int i = 0; i < 2 * nblk; ++i) {
        const int pg = i & 1;
        ok = mbar_wait(s_full + 2 * t + pg, kc & 1, abort_flag, p.g.status, 72);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        if (pg == 0) {  // (by now the barrier's phase is this block's, whichever segments the tile had no rows in)
          ok = mbar_wait(seen_full + ks % kSeen, ks / kSeen & 1, abort_flag, p.g.status, 83);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          pages = seen[ks % kSeen];
        }
        tc_fence_after();
        const uint32_t tp = ts + kPage * pg;
        const int slot0 = (x.first + (u + (i >> 1) - x.begin)) * kBlockKeys + kPage * pg;
        const bool there = (pages >> pg) & 1u;
        // tokens lo < k <= hi of the page are seen
        const int hi = at - slot0, lo = p.window > 0 ? hi - p.window : -1;
        const bool masked = slot0 + kPage - 1 > at_lo || (p.window > 0 && slot0 <= at_hi - p.window) || !there;
        // Bit k: token 32 c + k is seen.
        auto seen_bits = [&](int c) {
          const int up = hi - 32 * c, dn = lo - 32 * c;
          uint32_t bits = up >= 31 ? 0xFFFFFFFFu : up < 0 ? 0u : (2u << up) - 1u;
          if (dn >= 0) bits = dn >= 31 ? 0u : bits & ~((2u << dn) - 1u);
          return there ? bits : 0u;
        };
        // the page's scores in registers; where nothing is done to them, their
        // maximum comes with them out of TMEM
        float v[2][32], mt;
        if (MOD || masked) {
          tmem_ld32(tp, v[0]);
          tmem_ld32(tp + 32, v[1]);
          tmem_wait_ld();
          if constexpr (MOD) log2_scores(v, tp, hi);
          mt = -INFINITY;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if (masked) {
              const uint32_t bits = seen_bits(c);
#pragma unroll
              for (int k = 0; k < 32; ++k) v[c][k] = (bits >> k) & 1u ? v[c][k] : -INFINITY;
            }
#pragma unroll
            for (int k = 0; k < 32; k += 2) mt = fmax3(mt, v[c][k], v[c][k + 1]);
          }
        } else {
          const float a0 = tmem_ld32_max(tp, v[0]), a1 = tmem_ld32_max(tp + 32, v[1]);
          tmem_wait_ld();
          mt = fmaxf(a0, a1);
        }
        if constexpr (!MOD) mt *= cs;
        const bool moves = mt > m + slack;  // (m = -inf: as soon as something is seen)
        if (__any_sync(0xFFFFFFFFu, moves)) {
          const float alpha = moves ? ex2_approx(m - mt) : 1.0f;
          l *= alpha;
          if (moves) m = mt;
          if (i > 0) {
            // the tile's last PV must be in before O is touched
            ok = mbar_wait(o_full + 2 * t + (pg ^ 1), (pg ? kc : kc - 1) & 1, abort_flag, p.g.status, 73);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              float y[16];
              tmem_ld16(to + 16 * c, y);
              tmem_wait_ld();
              uint32_t w[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) w[k] = __float_as_uint(y[k] * alpha);
              tmem_st16(to + 16 * c, w);
            }
          }
        }
        // P over the columns S came in
        const float off = shift - (m == -INFINITY ? 0.0f : m);
        const float f = MOD ? 1.0f : cs;
        float l0 = 0.0f, l1 = 0.0f;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t h[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float a, b;
            ffma2(a, b, v[c][2 * k], v[c][2 * k + 1], f, f, off, off);
            a = ex2_approx(a);
            b = ex2_approx(b);
            ffma2(l0, l1, a, b, 1.0f, 1.0f, l0, l1);
            h[k] = half2_of(a, b);
          }
          tmem_st16(tp + 16 * c, h);
        }
        l += l0 + l1;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        arrive_tmem(first_bars + 8 * (2 + kStages + 2 * t + pg));
        kc += pg;
        ks += pg;
      }
      if (!ok) break;
      const bool whole = u == x.begin && seg_end == x.end;
      const long long out = static_cast<long long>(x.row0 + r / p.G) * (p.g.heads * p.G) + x.h * p.G + r % p.G;
      float* part = p.part + static_cast<long long>(pair * 2 + (u == x.begin ? 1 : 0)) * part_floats<D>(kRowsPair);
      // The next segment's queries are staged and its first scores made while the
      // results are written (its first PV waits for this warp's P, which comes after).
      u = seg_end;
      any = seek();
      if (any) locate_q();
      // the rows' results
      // (page 1's PV of the last block, behind all others; that of the block
      // before was in when page 1's scores came, so the phase is the right one)
      ok = mbar_wait(o_full + 2 * t + 1, (kc - 1) & 1, abort_flag, p.g.status, 74);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      tc_fence_after();
      if (any) down = stage_q();
      const float f = l == 0.0f ? 0.0f : p.v_up / l;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        float v[32];
        tmem_ld32(to + 32 * c, v);
        tmem_wait_ld();
        if (!real) continue;
        if (whole) {
          uint4* dst = reinterpret_cast<uint4*>(p.o + out * D + 32 * c);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const __nv_bfloat162 b = __floats2bfloat162_rn(v[8 * i + 2 * k] * f, v[8 * i + 2 * k + 1] * f);
              h[k] = *reinterpret_cast<const uint32_t*>(&b);
            }
            dst[i] = make_uint4(h[0], h[1], h[2], h[3]);
          }
        } else {
          float4* dst = reinterpret_cast<float4*>(part + col * D + 32 * c);
#pragma unroll
          for (int i = 0; i < 8; ++i) dst[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
      }
      if (real && whole) p.lse[out] = out_lse(m, l, shift);
      if (real && !whole) {
        part[kRowsPair * D + col] = m;
        part[kRowsPair * D + kRowsPair + col] = l;
      }
      tc_fence_before();  // O is read before the next segment's first PV, which waits for this warp's P
    }
  } else if (warp < kWarpMma) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOperands));
    // ---------------------------------------------------------------- operands
    const int w = warp - kWarpDq;
    // K: rows 8 (4 rank + 2 (w & 1) + i) + g of page w / 2, chunk c: of each page every CTA holds 32 rows
    const int g = lane >> 2, c = lane & 3, j0 = 4 * rank + 2 * (w & 1);
    // V: tokens 4 t4 .. 4 t4 + 3 of page w / 2 and of it (16 pieces), this CTA's channel chunk gl: the 16 lanes of a
    // store phase hold the 16 pieces of a row
    const int pv = w >> 1, t4 = lane & 15, gl = (w & 1) * 2 + (lane >> 4), gv = rank * 4 + gl;
    // Two blocks ahead the block's page numbers are read, one block ahead the
    // bytes that the thread needs of the pages; nothing that was read is looked
    // at before the block between is converted, and nothing is read before a
    // proxy fence, which would wait for it.
    struct Block {
      int page[2];  // table entries, where looks() says so
      int first;    // number of the first page
      int lo, L;    // the problem's queries see slots in [lo, L) alone (one comparison below; with two 977 us, not 962)
      int h;
    };
    // Whether page i of a block holds a token that some query sees: others are
    // not looked at (a window's old pages may be back in the pool).
    auto looks = [&](const Block& y, int i) {
      const int from = y.lo & ~(kPage - 1);
      return static_cast<unsigned>((y.first + i) * kPage - from) < static_cast<unsigned>(y.L - from);
    };
    Unit x;
    x.end = -1;
    auto find = [&](int u) {
      Block y{{-1, -1}, 0, 0, 0, 0};
      if (u >= end) return y;
      if (u >= x.end) x = find_unit<kRowsPair, kBlockKeys>(p, prefix, u);
      y.first = 2 * (x.first + (u - x.begin));
      y.lo = p.window > 0 && !x.none ? max(0, x.L - x.n + x.r0 / p.G - p.window + 1) : 0;
      y.L = x.none ? 0 : x.L;
      y.h = x.h;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (looks(y, i)) y.page[i] = p.g.table[static_cast<long long>(x.b) * p.g.M + y.first + i];
      return y;
    };
    // the bytes of page i of a block, or null; a bit per page that counts (one that is not looked at does)
    auto bytes_of = [&](const Block& y, int i) -> const uint8_t* {
      const int page = i ? y.page[1] : y.page[0];
      if (!looks(y, i) || page < 0 || page >= p.g.num_pages) return nullptr;
      return p.pages + (static_cast<long long>(page) * p.g.heads + y.h) * PageLayout<D>::kBytes;
    };
    auto seen_of = [&](const Block& y) {
      uint32_t s = 3u;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (looks(y, i) && (y.page[i] < 0 || y.page[i] >= p.g.num_pages)) {
          report_bad_index(p.g.status);
          s &= ~(1u << i);
        }
      return s;
    };
    uint32_t kw[2][D / 32], ksc, vw[4][D / 64];
    uint16_t vsc[2];
    auto load_k = [&](const uint8_t* src) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint8_t* a = src + (8 * (j0 + i) + g) * (D / 2) + c * (D / 8);
        if constexpr (D == 128) {
          const uint4 v = src ? __ldg(reinterpret_cast<const uint4*>(a)) : make_uint4(0u, 0u, 0u, 0u);
          kw[i][0] = v.x; kw[i][1] = v.y; kw[i][2] = v.z; kw[i][3] = v.w;
        } else {
          const uint2 v = src ? __ldg(reinterpret_cast<const uint2*>(a)) : make_uint2(0u, 0u);
          kw[i][0] = v.x; kw[i][1] = v.y;
        }
      }
      const uint8_t* a = src + PageLayout<D>::kKs + (lane * 8 + j0) * PageLayout<D>::S;
      if constexpr (D == 128) ksc = src ? __ldg(reinterpret_cast<const uint32_t*>(a)) : 0u;
      else ksc = src ? __ldg(reinterpret_cast<const uint16_t*>(a)) : 0u;
    };
    auto load_v = [&](const uint8_t* src) {
      const uint8_t* b = src + PageLayout<D>::kVc + ((t4 >> 1) * 8 + gv) * (D / 2) + (t4 & 1) * (D / 4);
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        const uint4 v = src ? __ldg(reinterpret_cast<const uint4*>(b) + i) : make_uint4(0u, 0u, 0u, 0u);
        if constexpr (D == 128) {
          vw[2 * i][0] = v.x; vw[2 * i][1] = v.y; vw[2 * i + 1][0] = v.z; vw[2 * i + 1][1] = v.w;
        } else {
          vw[0][0] = v.x; vw[1][0] = v.y; vw[2][0] = v.z; vw[3][0] = v.w;
        }
      }
      const int blk = D == 128 ? gv : gv >> 1;
#pragma unroll
      for (int i = 0; i < 2; ++i)  // token pairs 2 c, 2 c + 1 with c = 2 (t4 & 1) + i
        vsc[i] = src ? __ldg(reinterpret_cast<const uint16_t*>(src + PageLayout<D>::kVs + (blk * 4 + 2 * (t4 & 1) + i) * 16 +
                                                               (t4 >> 2) * 4 + ((t4 >> 1) & 1) * 2))
                     : static_cast<uint16_t>(0);
    };
    Block cur = find(start), next = find(start + 1);
    load_k(bytes_of(cur, pv));
    load_v(bytes_of(cur, pv));
    bool ok = true;
    for (int u = start, k = 0; u < end && ok; ++u, ++k) {
      const int s = k % kStages;
      const Block after = find(u + 2);
      if (k >= kStages) {
        ok = mbar_wait(k_empty + s, (k / kStages - 1) & 1, abort_flag, p.g.status, 75);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
      }
      if (w == 0 && lane == 0) {
        seen[k % kSeen] = static_cast<uint8_t>(seen_of(cur));
        mbar_arrive(seen_full + k % kSeen);
      }
      uint8_t* kt = smem + L_::kK + s * L_::kKTile;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 32 * pv + 8 * (2 * (w & 1) + i) + g;
        uint32_t sc[2];
        int flip = 0;
        if constexpr (D == 128) {
          const uint32_t h = e4m3x2_to_half2(ksc >> (16 * i));
          // chunks 2 and 3 take their words in the order 2 3 0 1: the eight
          // lanes of a store phase (two rows, four chunks) then hit eight
          // different 16-byte units, instead of four twice
          flip = c & 2;
          sc[0] = flip ? splat_hi(h) : splat_lo(h);
          sc[1] = flip ? splat_lo(h) : splat_hi(h);
          const uint32_t w0 = kw[i][0], w1 = kw[i][1];
          kw[i][0] = flip ? kw[i][2] : w0;
          kw[i][1] = flip ? kw[i][3] : w1;
          kw[i][2] = flip ? w0 : kw[i][2];
          kw[i][3] = flip ? w1 : kw[i][3];
        } else {
          sc[0] = sc[1] = splat_lo(e4m3x2_to_half2(ksc >> (8 * i)));
        }
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
          uint32_t h[4];
          e2m1x8_to_half2(kw[i][q], h);
#pragma unroll
          for (int y = 0; y < 4; ++y) h[y] = hmul2(h[y], sc[q >> 1]);
          const int unit = c * (D / 32) + (q ^ flip);  // 16-byte unit of the row
          *reinterpret_cast<uint4*>(kt + (unit >> 3) * (kPage * 128) + swz(r, unit & 7)) = make_uint4(h[0], h[1], h[2], h[3]);
        }
      }
      if (k >= kStages) {
        ok = mbar_wait(v_empty + s, (k / kStages - 1) & 1, abort_flag, p.g.status, 76);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
      }
      uint8_t* vt = smem + L_::kV + s * L_::kVTile + pv * ((D / 2) * 128) + (t4 & 1) * 8;
      uint32_t sc[2];
      // what lies before the first token that a query sees, or behind the last, may be anything: P is 0 there, V must
      // be finite
      const int t0 = (cur.first + pv) * kPage + t4 * 4 - cur.lo;
      const unsigned span = cur.L - cur.lo;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        sc[i] = e4m3x2_to_half2(vsc[i]);
        if (static_cast<unsigned>(t0 + 2 * i) >= span) sc[i] &= 0xFFFF0000u;
        if (static_cast<unsigned>(t0 + 2 * i + 1) >= span) sc[i] &= 0xFFFFu;
      }
#pragma unroll
      for (int q = 0; q < D / 64; ++q) {
        uint32_t ev[2][4], od[2][4];  // [token pair][even / odd channel 2 y (+ 1)]
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t a = vw[2 * i][q], b = vw[2 * i + 1][q];
          e2m1x8_to_half2((a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u), ev[i]);
          e2m1x8_to_half2(((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u), od[i]);
        }
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int d = gl * (D / 8) + 8 * q + 2 * y;  // of this CTA's channels
          *reinterpret_cast<uint2*>(vt + swz(d, t4 >> 1)) = make_uint2(hmul2(ev[0][y], sc[0]), hmul2(ev[1][y], sc[1]));
          *reinterpret_cast<uint2*>(vt + swz(d + 1, t4 >> 1)) = make_uint2(hmul2(od[0][y], sc[0]), hmul2(od[1][y], sc[1]));
        }
      }
      fence_proxy_async_smem();
      arrive_smem(smem_u32((rank == 0 ? kv_full : kv_mine) + s));
      load_k(bytes_of(next, pv));
      load_v(bytes_of(next, pv));
      cur = next;
      next = after;
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsMma));
    if (warp == kWarpMma) {
      if (rank == 0) {
        // -------------------------------------------------------------- MMA
        int k = 0, nk[2] = {0, 0}, ns[2] = {0, 0};  // blocks of the pair; blocks and segments of each tile
        bool ok = true;
        const uint32_t bKEmpty = smem_u32(k_empty), bVEmpty = smem_u32(v_empty), bS = smem_u32(s_full), bO = smem_u32(o_full);
        const uint32_t base = (smem_u32(smem) & 0x3FFFFu) >> 4, q = base + L_::kQ / 16;
        auto k_at = [&](int s) { return base + (L_::kK + s * L_::kKTile) / 16; };
        auto v_at = [&](int s) { return base + (L_::kV + s * L_::kVTile) / 16; };
        auto wait_for = [&](auto smem_too, uint64_t* bar, int phase, unsigned site) {
          ok = ok && bounded_wait([&]() { return pair_try_wait<smem_too.value>(bar, phase & 1); }, abort_flag, p.g.status, site);
          ok = __all_sync(0xFFFFFFFFu, ok);
          tc_fence_after();
        };
        auto wait = [&](uint64_t* bar, int phase, unsigned site) { wait_for(std::true_type{}, bar, phase, site); };
        auto wait_p = [&](uint64_t* bar, int phase) { wait_for(std::false_type{}, bar, phase, 79); };
        for (int u = start; u < end && ok;) {
          const Unit x = find_unit<kRowsPair, kBlockKeys>(p, prefix, u);
          const int seg_end = min(end, x.end), nblk = seg_end - u;
          const bool two = x.r0 + 256 <= x.r1;
          wait(kv_full + k % kStages, k / kStages, 77);
          wait(q_full, ns[0]++, 78);
          if (two) wait(q_full + 1, ns[1]++, 78);
          if (!ok) break;
          {
            const int S = k % kStages;
            const uint32_t K = k_at(S);
            issue_qk<D, 0, 0>(q, K, bS);
            if (two) issue_qk<D, 1, 0>(q, K, bS);
            issue_qk<D, 0, 1>(q, K, bS);
            if (two) issue_qk<D, 1, 1>(q, K, bS);
            tc_commit2(bKEmpty + 8 * S);
          }
          for (int j = 0; j < nblk && ok; ++j, ++k, ++nk[0], nk[1] += two) {
            const bool more = j + 1 < nblk;
            const int S = k % kStages, S1 = (k + 1) % kStages;
            if (more) wait(kv_full + S1, (k + 1) / kStages, 80);
            if (!ok) break;
            const uint32_t V = v_at(S), K = k_at(S1);
            // page 0 of the tiles, then page 1: P in, the page's S of the next block out
            wait_p(p_full, nk[0]);
            if (!ok) break;
            issue_pv<D, 0, 0>(V, bO, j > 0);
            if (more) issue_qk<D, 0, 0>(q, K, bS);
            if (two) {
              wait_p(p_full + 2, nk[1]);
              if (!ok) break;
              issue_pv<D, 1, 0>(V, bO, j > 0);
              if (more) issue_qk<D, 1, 0>(q, K, bS);
            }
            wait_p(p_full + 1, nk[0]);
            if (!ok) break;
            issue_pv<D, 0, 1>(V, bO, true);
            if (!two) tc_commit2(bVEmpty + 8 * S);
            if (more) issue_qk<D, 0, 1>(q, K, bS);
            if (two) {
              wait_p(p_full + 3, nk[1]);
              if (!ok) break;
              issue_pv<D, 1, 1>(V, bO, true);
              tc_commit2(bVEmpty + 8 * S);
              if (more) issue_qk<D, 1, 1>(q, K, bS);
            }
            if (more) tc_commit2(bKEmpty + 8 * S1);
          }
          u = seg_end;
        }
        tc_commit2(smem_u32(drain));
      }
    } else if (rank == 1) {
      // ------------------------------------------------------ passing on
      if (warp == kWarpMma + 1) {
        for (int k = 0; k < end - start; ++k) {
          const int s = k % kStages;
          if (!__all_sync(0xFFFFFFFFu, mbar_wait(kv_mine + s, k / kStages & 1, abort_flag, p.g.status, 81))) break;
          arrive_first(first_bars + 8 * (2 + s));
        }
      }
    } else if (warp == kWarpMma + 1) {
      // for the join: the problem that begins in this run and does not end in it
      const Unit x = find_unit<kRowsPair, kBlockKeys>(p, prefix, end - 1);
      const bool split = x.begin >= start && x.end > end;
      if (lane == 0) *split_of(p, pair) = Split{split ? (x.end - 1) / per : -1, x.row0, x.h, x.r0, x.r1, kPMax - slack_of(x.L)};
    }
  }
  tc_fence_before();
  __syncthreads();
  // no operation of the pair is in flight when it frees its columns
  if (warp == kWarpMma) mbar_wait_drain(drain, 0, abort_flag, p.g.status, 82);
  cluster_sync();  // neither CTA leaves while the other's MMAs read it
  tc_fence_after();
  if (warp == kWarpMma) tmem_dealloc2(tmem_base, 512);
}

template <int D, bool MOD>
cudaError_t launch_d(const KvAttnParams& p, cudaStream_t s) {
  using L_ = PromptSmem<D>;
  cudaError_t e = allow_smem<kv_prompt_kernel<D, MOD>>(L_::bytes(kMaxKvBatch));
  if (e != cudaSuccess) return e;
  e = launch_chained_cluster(kv_prompt_kernel<D, MOD>, dim3(2 * p.ctas), 2, kPromptThreads, L_::bytes(p.g.B), s, p);
  if (e != cudaSuccess) return e;
  return launch_chained(kv_join_kernel<D, kRowsPair>, dim3(p.ctas, kRowsPair / kJoinRows<D>), kJoinThreads, 0, s, p);
}

}  // namespace

int prompt_runs() { return sm_count() / 2; }

size_t prompt_workspace(int D) {
  return plan_bytes() + static_cast<size_t>(prompt_runs()) * 2 * kRowsPair * (D + 2) * sizeof(float);
}

cudaError_t launch_prompt(const KvAttnParams& p, int D, cudaStream_t s) {
  const bool mod = p.cap > 0.0f || p.slopes;
  if (D == 128) return mod ? launch_d<128, true>(p, s) : launch_d<128, false>(p, s);
  return mod ? launch_d<64, true>(p, s) : launch_d<64, false>(p, s);
}

}  // namespace fp4attn
