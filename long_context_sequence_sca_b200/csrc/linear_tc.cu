// The projection's products on the 5th-generation tensor cores:
//   C[m, n] = sum_k A(m, k) B(n, k)
// with each operand stored along k (K-major) or along its own rows (MN-major),
// which covers x w^T, du w and du^T x without a transposed copy.
//
// fp32 operands come as three bf16 planes, v = h + m + l to 2^-25 of |v|, and
// the product as the six plane products that reach 2^-24 (the other three are
// below 2^-26): hh, hm, mh, mm, hl, lh.  To the large tiles' kernel they are a
// product six times as deep whose k-blocks come from different planes; at a sixth
// of the bf16 rate this is still several times the rate of the fp32 FMA pipe.
//
// The tensor core cuts its sums instead of rounding them: a step of 16 terms takes
// about 2^-25.5 of the result, 2^-23.5 where all terms have one sign (measured:
// 6e-6 and 1.6e-5 after 256 steps, which shows in the fp32 results: y, pre, db).
// Where it would (fp32, bf16 with pre, and any bf16 product that is deeper than
// kDeep), a product is cut into runs of 1024 (2048; kDeep), whose sums the epilogue
// warps add up in registers with rounding while the next run is under way (kSum),
// and the planes are added in ascending size, or apart from the first.
//
// Persistent, warp-specialised: one thread loads 64-deep k-blocks by TMA into a
// ring of stages, one thread issues tcgen05.mma, eight or sixteen warps empty the
// accumulator (TMEM, two of them in turn), a row per thread.
// With CG = 2 a pair of CTAs shares one 256 x kBN tile: each loads its 128
// rows of A and half the rows of B, so a k-block moves half the bytes per
// multiply-add of a 128 x kBN tile; the even CTA issues the MMAs for both.
#include <type_traits>

#include "common.cuh"
#include "gecko_internal.h"
#include "linear.cuh"

namespace gecko {
namespace {

// ---------------------------------------------------------- pair (CG = 2) --

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The two halves of it, for work between that needs nothing of the other CTAs.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Shared-memory address of `p` in the CTA of rank `rank`.
__device__ __forceinline__ uint32_t map_to(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ void mbar_arrive_at(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// mbar_wait for a barrier on which another CTA of the cluster arrives.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort, int* status) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    if ((it & 63u) == 0) {
      if (*abort) return false;
      if (globaltimer_ns() - t0 > kWaitLimitNs) {
        *abort = 1;
        atomicOr(status, kStatusTimeout);
        return false;
      }
    }
  }
}

template <int CG>
__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  if (CG == 1)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
        "[%2];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
  else   // the barrier may lie in the other CTA of the pair
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], "
        "[%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

template <int CG>
__device__ __forceinline__ void umma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if (CG == 1)
    umma_ss(d, a, b, idesc, accumulate);
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// True for one thread of the (whole) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(p));
  return p != 0;
}

// Arrive on `bar` (of both CTAs of a pair) when the MMAs issued so far are done.
template <int CG>
__device__ __forceinline__ void umma_done(uint64_t* bar) {
  if (CG == 1)
    umma_commit(bar);
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}

template <int CG>
__device__ __forceinline__ void tmem_take(uint32_t* slot, uint32_t cols) {
  if (CG == 1) {
    tmem_alloc(slot, cols);
    tmem_relinquish();
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void tmem_give(uint32_t taddr, uint32_t cols) {
  if (CG == 1)
    tmem_dealloc(taddr, cols);
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols) : "memory");
}

// ------------------------------------------------------------- work split --

constexpr int kBK = 64;              // k-block: one 128-byte swizzle row
constexpr int kBN = 256;             // columns per tile
constexpr int kEpilogueWarp = 4;     // after TMA, MMA, TMEM and an idle warp
constexpr int kBand = 16;            // columns an epilogue warp takes at a time
// Epilogue warps: each of the four row quarters of a tile has two where they hold
// running sums (kSum), else four: what they wait for is each other's loads and
// stores (4096 x 4096 x 512 with SiLU and residual: 39 us with eight warps, with
// sixteen 35 us).
template <bool kSum> constexpr int kEpilogueWarps = kSum ? 8 : 16;
template <bool kSum> constexpr int kGemmThreads = 32 * (kEpilogueWarp + kEpilogueWarps<kSum>);
constexpr int kFewThreads = 384;
// Registers per thread after setmaxnreg: the running sums of 128 columns sit in
// the epilogue warps'.  The split has to fit what the block was launched with
// (setmaxnreg.inc would wait for more forever).
constexpr int kRegsCtl = 56, kRegsEpilogue = 224;
static_assert(128 * kRegsCtl + 256 * kRegsEpilogue <= kGemmThreads<true> * 168,
              "setmaxnreg split above the launch registers");
constexpr int kGroupM = 8;           // tiles of one column band done together (operand reuse in L2)

struct GemmShape {
  int64_t M, N;
  int tiles_m, tiles_n;
  int k_blocks, pairs;            // of one plane product; plane products
  int splits, blocks_per_split;   // the k-blocks in `splits` parts, each its own unit
  int run;                        // k-blocks per run of the accumulator (kSum)
};

// Planes of A and B of each plane product (one pair, 0 and 0, for bf16).
constexpr int kPairs = 6;
__device__ __forceinline__ int plane_a(int left) { return (0x201100 >> (4 * left)) & 15; }
__device__ __forceinline__ int plane_b(int left) { return (0x021010 >> (4 * left)) & 15; }

struct Unit {
  int m, n, split, kb0, kb1;
};

__device__ __forceinline__ Unit unit_at(const GemmShape& g, int u) {
  const int tiles = g.tiles_m * g.tiles_n;
  Unit r;
  r.split = u / tiles;
  const int t = u - r.split * tiles;
  const int band = kGroupM * g.tiles_n, group = t / band, in = t - group * band;
  const int m0 = group * kGroupM, gm = min(kGroupM, g.tiles_m - m0);
  r.n = in / gm;
  r.m = m0 + (in - r.n * gm);
  r.kb0 = r.split * g.blocks_per_split;
  r.kb1 = min(g.k_blocks, r.kb0 + g.blocks_per_split);
  return r;
}

// -------------------------------------------------------------- epilogues --

// A thread owns one row of the tile and takes 16 columns of it at a time,
// straight from registers to global memory: shared memory is busy feeding the
// MMAs (a transpose through it took five times as long as the stores of full
// 32-byte sectors that this makes).  `wide` says that rows and columns of 16 are
// aligned for 32-byte accesses.

__device__ __forceinline__ void store_sector(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// 16 consecutive values.
__device__ __forceinline__ void store16(__nv_bfloat16* p, const float* v, bool wide) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
  if (wide) {
    store_sector(p, w);
  } else {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(p + 8) = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
__device__ __forceinline__ void store16(float* p, const float* v, bool wide) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[8 * h + i]);
    if (wide) {
      store_sector(p + 8 * h, w);
    } else {
      *reinterpret_cast<uint4*>(p + 8 * h) = make_uint4(w[0], w[1], w[2], w[3]);
      *reinterpret_cast<uint4*>(p + 8 * h + 4) = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
}

// Forward: bias, activation, residual.  What has to be read for a band is
// fetched before the sums are waited for.
template <typename T>
struct EpiForward {
  const float* bias;
  const T* residual;
  T* y;
  float* pre;
  OutLayout lay;
  int act;
  bool wide, wide_pre;   // of y; of pre
  struct Fetched {
    float bias[16];
    Vec8<T> residual[2];
  };
  __device__ __forceinline__ int64_t row(int64_t m) const { return lay.row(m); }
  __device__ __forceinline__ void fetch(Fetched& f, int64_t row, int n, bool on) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool in = n + 8 * i < lay.N;
#pragma unroll
      for (int j = 0; j < 8; ++j) f.bias[8 * i + j] = 0.f;
      if (bias && in) load_f8(bias + n + 8 * i, *reinterpret_cast<float(*)[8]>(f.bias + 8 * i));
      if (residual && in && on) f.residual[i].load(residual + row + lay.col(n + 8 * i));
    }
  }
  __device__ __forceinline__ void put(const Fetched& f, int64_t row, int n, int, float* v) const {
    if (n >= lay.N) return;
    const int64_t at[2] = {row + lay.col(n), row + lay.col(n + 8)};
    const bool both = n + 8 < lay.N;
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] += f.bias[i];
    if (pre) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (i == 0 || both) {
          float* p = pre + at[i];
          uint32_t w[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(v[8 * i + j]);
          if (wide_pre) {
            store_sector(p, w);
          } else {
            *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4*>(p + 4) = make_uint4(w[4], w[5], w[6], w[7]);
          }
        }
    }
    if (act == kActSilu) {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = activate<T>(v[i], kActSilu);
    } else if (act == kActGelu) {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = activate<T>(v[i], kActGelu);
    }
    if (residual) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (i == 0 || both) {
          float r[8];
          f.residual[i].get(r);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[8 * i + j] += r[j];
        }
    }
    if (wide) {
      store16(y + at[0], v, true);
    } else {
      store_f8(y + at[0], *reinterpret_cast<float(*)[8]>(v));
      if (both) store_f8(y + at[1], *reinterpret_cast<float(*)[8]>(v + 8));
    }
  }
};

// c[split][m][n]: the product itself (one split), or the parts' sums.
template <typename T>
struct EpiPlain {
  T* c;
  int64_t M;
  int N;
  bool wide;
  struct Fetched {};
  __device__ __forceinline__ int64_t row(int64_t m) const { return m * N; }
  __device__ __forceinline__ void fetch(Fetched&, int64_t, int, bool) const {}
  __device__ __forceinline__ void put(const Fetched&, int64_t row, int n, int split, float* v) const {
    T* p = c + (int64_t)split * M * N + row + n;
    if (n + 8 < N) store16(p, v, wide);
    else if (n < N) store_f8(p, *reinterpret_cast<float(*)[8]>(v));
  }
};

// ----------------------------------------------------------------- kernel --

template <int CG>
struct GemmCfg {
  static constexpr int kA = 128 * kBK * 2, kB = kBN / CG * kBK * 2, kStage = kA + kB;
  static constexpr int kStages = (232448 - 1024 - 512) / kStage > 8 ? 8 : (232448 - 1024 - 512) / kStage;
  static constexpr int kBarOff = kStages * kStage;
  static constexpr int kNumBars = 2 * kStages + 5;   // full, empty; accumulator full, empty; drain
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;
  static constexpr int kAlloc = kMiscOff + 16 + 1024;
  static constexpr uint32_t kTmemCols = 2 * kBN;
  static_assert(kAlloc <= 232448, "shared memory above the per-block limit");
};

template <int CG, bool AMN, bool BMN, bool kSum, class Epi>
__global__ void __launch_bounds__(kGemmThreads<kSum>, 1) gemm_tc_kernel(const __grid_constant__ CUtensorMap ma,
                                                                        const __grid_constant__ CUtensorMap mb,
                                                                        const GemmShape g, const Epi ep, int* status) {
  using Cfg = GemmCfg<CG>;
  constexpr int NS = Cfg::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Cfg::kBarOff);   // used in the even CTA
  uint64_t* empty = full + NS;
  uint64_t* acc_full = empty + NS;    // [2]
  uint64_t* acc_empty = acc_full + 2; // [2], used in the even CTA
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::kMiscOff + 4);

  const int warp = warp_id_uniform(), lane = threadIdx.x % 32;
  const uint32_t rank = CG == 1 ? 0 : cluster_rank();
  const int first = blockIdx.x / CG, step = gridDim.x / CG;
  const int units = g.tiles_m * g.tiles_n * g.splits;
  let_next_start();

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full + i, 1);
      mbar_init(acc_empty + i, kEpilogueWarps<kSum> * CG);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 3 && lane == 0) {
    tma_prefetch_desc(&ma);
    tma_prefetch_desc(&mb);
  }
  if (warp == 2) tmem_take<CG>(tmem_slot, Cfg::kTmemCols);
  wait_for_previous();
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if constexpr (kSum)
    if (warp < kEpilogueWarp) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRegsCtl));
  if (warp == 0) {
    // ------------------------------------------------------- TMA producer --
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int u = first; u < units && ok; u += step) {
        const Unit t = unit_at(g, u);
        const int m0 = (t.m * CG + (int)rank) * 128, n0 = t.n * kBN + (int)rank * (kBN / CG);
        for (int left = g.pairs - 1; left >= 0 && ok; --left) {
          const int za = plane_a(left), zb = plane_b(left);
          for (int kb = t.kb0; kb < t.kb1; ++kb, ++it) {
            const int s = it % NS;
            if (it >= NS && !(ok = mbar_wait_cluster(empty + s, (it / NS - 1) & 1, abort_flag, status))) break;
            if (rank == 0) mbar_arrive_expect_tx(full + s, CG * Cfg::kStage);
            const uint32_t bar = CG == 1 ? smem_u32(full + s) : map_to(full + s, 0);
            uint8_t *pa = smem + s * Cfg::kStage, *pb = pa + Cfg::kA;
            if (AMN) {
#pragma unroll
              for (int i = 0; i < 2; ++i) tma_load<CG>(pa + i * 8192, &ma, bar, m0 + 64 * i, kb * kBK, za);
            } else {
              tma_load<CG>(pa, &ma, bar, kb * kBK, m0, za);
            }
            if (BMN) {
#pragma unroll
              for (int i = 0; i < kBN / CG / 64; ++i)
                tma_load<CG>(pb + i * 8192, &mb, bar, n0 + 64 * i, kb * kBK, zb);
            } else {
              tma_load<CG>(pb, &mb, bar, kb * kBK, n0, zb);
            }
          }
        }
      }
      // the stages' last readers, so that nothing arrives here after the exit;
      // after an abort, the copies issued (both CTAs' land on the even one's barriers)
      for (int i = it > NS ? it - NS : 0; i < it; ++i) {
        if (*abort_flag) {
          if (rank == 0) mbar_wait_drain(full + i % NS, (i / NS) & 1);
        } else {
          mbar_wait_cluster(empty + i % NS, (i / NS) & 1, abort_flag, status);
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // --------------------------------------------------------- MMA issuer --
    if (rank == 0) {   // (the whole warp walks the loop: see gemm_few_kernel)
      const bool leader = elect_one();
      constexpr uint32_t idesc = idesc_bf16_f32(128 * CG, kBN, AMN, BMN);
      const uint32_t base = smem_u32(smem);
      int it = 0, k = 0;
      bool ok = true;
      for (int u = first; u < units && ok; u += step) {
        const Unit t = unit_at(g, u);
        const int blocks = (t.kb1 - t.kb0) * g.pairs;
        for (int kb = 0; kb < blocks && ok; ++k) {   // k counts runs
          const int acc = k & 1, end = kSum ? min(kb + g.run, blocks) : blocks;
          if (k >= 2 && !(ok = __all_sync(0xffffffffu, mbar_wait_cluster(acc_empty + acc, (k / 2 - 1) & 1, abort_flag,
                                                                        status))))
            break;
          tc_fence_after();
          for (uint32_t fresh = 1; kb < end; ++kb, ++it, fresh = 0) {
            const int s = it % NS;
            if (!(ok = __all_sync(0xffffffffu, mbar_wait_cluster(full + s, (it / NS) & 1, abort_flag, status)))) break;
            tc_fence_after();
            const uint32_t a0 = base + s * Cfg::kStage, b0 = a0 + Cfg::kA;
            const SDesc da = AMN ? sdesc_sw128_split(a0, 8192, 1024) : sdesc_sw128_split(a0, 16, 1024);
            const SDesc db = BMN ? sdesc_sw128_split(b0, 8192, 1024) : sdesc_sw128_split(b0, 16, 1024);
            if (leader) {
#pragma unroll
              for (int kk = 0; kk < kBK / 16; ++kk)
                umma<CG>(tmem + acc * kBN, sdesc_at(da, kk * (AMN ? 2048 : 32)), sdesc_at(db, kk * (BMN ? 2048 : 32)),
                         idesc, kk > 0 ? 1u : 1u - fresh);
              umma_done<CG>(empty + s);
            }
          }
          if (ok && leader) umma_done<CG>(acc_full + acc);
        }
      }
      if (!ok) {   // what was issued is done before TMEM is given back
        if (leader) umma_done<CG>(drain);
        mbar_wait_drain(drain, 0);
      }
    }
    __syncwarp();
  } else if (warp >= kEpilogueWarp) {
    if constexpr (kSum) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kRegsEpilogue));
    // ----------------------------------------------------------- epilogue --
    constexpr int kShare = kEpilogueWarps<kSum> / 4;         // warps per row quarter, taking bands in turn
    constexpr int kBands = kBN / kBand / kShare;
    const int q = warp % 4;   // the TMEM lanes a warp may read: rows 32 q ..
    const int first_band = (warp - kEpilogueWarp) / 4;
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16) + first_band * kBand;
    int k = 0;
    bool ok = true;
    for (int u = first; u < units && ok; u += step) {
      const Unit t = unit_at(g, u);
      const int64_t m = ((int64_t)t.m * CG + rank) * 128 + q * 32 + lane;
      const int n0 = t.n * kBN + first_band * kBand;
      const bool on = m < g.M;
      const int64_t row = ep.row(m);
      if constexpr (!kSum) {
        const int acc = k & 1;
        typename Epi::Fetched f;
        ep.fetch(f, row, n0, on);
        ok = __all_sync(0xffffffffu, mbar_wait_cluster(acc_full + acc, (k / 2) & 1, abort_flag, status));
        if (!ok) break;
        ++k;
        tc_fence_after();
#pragma unroll 1
        for (int j = 0; j < kBands; ++j) {
          float v[kBand];
          tmem_ld16p(lanes + acc * kBN + j * kShare * kBand, reinterpret_cast<uint32_t*>(v));
          if (j) ep.fetch(f, row, n0 + j * kShare * kBand, on);
          tmem_wait_ld();
          if (j == kBands - 1) {
            // the accumulator is read: the MMAs of the unit after next may write it
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_at(CG == 1 ? smem_u32(acc_empty + acc) : map_to(acc_empty + acc, 0));
          }
          if (on) ep.put(f, row, n0 + j * kShare * kBand, t.split, v);
        }
      } else {
        float sum[kBands][kBand] = {};
        const int runs = ((t.kb1 - t.kb0) * g.pairs + g.run - 1) / g.run;
        for (int r = 0; r < runs; ++r, ++k) {
          const int acc = k & 1;
          ok = __all_sync(0xffffffffu, mbar_wait_cluster(acc_full + acc, (k / 2) & 1, abort_flag, status));
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int j = 0; j < kBands; j += 2) {
            uint32_t v[2][kBand];
            tmem_ld16p(lanes + acc * kBN + j * kShare * kBand, v[0]);
            tmem_ld16p(lanes + acc * kBN + (j + 1) * kShare * kBand, v[1]);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 2 * kBand; ++i)
              sum[j + i / kBand][i % kBand] += __uint_as_float(v[i / kBand][i % kBand]);
          }
          // the accumulator is read: the run after next may write it
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_at(CG == 1 ? smem_u32(acc_empty + acc) : map_to(acc_empty + acc, 0));
        }
        if (!ok) break;
#pragma unroll
        for (int j = 0; j < kBands; ++j) {
          typename Epi::Fetched f;
          ep.fetch(f, row, n0 + j * kShare * kBand, on);
          if (on) ep.put(f, row, n0 + j * kShare * kBand, t.split, sum[j]);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();
  if (warp == 2) tmem_give<CG>(tmem, Cfg::kTmemCols);
  if (CG == 2) cluster_sync();
}

// Few rows (generation, short prompts) or few tiles: the product is bound by the
// other operand's bytes, or by how long a tile takes, so the work is spread over
// as many SMs as it reaches: tiles of 128 x FN, one per cluster, and the depth
// shared by the cluster's CTAs, each with a part of the k-blocks (balanced, none
// empty).  Their sums meet through distributed shared memory: each CTA leaves its
// rows in the memory of its (now idle) stages and takes an equal share of the
// columns, adding the CTAs' parts in rank order.  One launch, and no working
// memory.
// What keeps the bytes coming is how many stages are on their way, so a stage
// holds only the rows there are (to a multiple of 8): the MMA reads 128 all the
// same, the others from the operand behind, and their results are not used.  (8 x
// 4096 x 4096: 13.4 us with six whole stages, with eleven short ones 12.4.)
// kSums says how the products are summed.  kOne: in one accumulator.  kRuns: a run of
// g.run k-blocks has one to itself, and what is in them (up to four of 128 columns,
// two of 256) is added up as it is read.  (Not always: with a loop over the runs 8 x
// 4096 x 4096 took 8.4 us against 8.1.)  kPlanes3: a stage holds one plane of A and of B,
// loaded once for all of its plane products (with a stage for each product, twice the
// bytes, 256 x 4096 x 1024 took 28.1 us against 25.7 and 64 x 4096 x 4096 70 against
// 58).  The order, middle planes first, gives the stages back as they were taken.  The
// product of the first planes has an accumulator to itself: as many of its sums are
// cut as of a bf16 product's.
constexpr int kFewRing = 196608, kFewMostStages = 12;   // bytes of the ring
template <int FN> constexpr int kFewPitch = FN + 4;     // floats per row left in shared memory
constexpr int kFewMiscOff = kFewRing + (2 * kFewMostStages + 1) * 8;
constexpr int kFewAlloc = kFewMiscOff + 16 + 1024;
static_assert(128 * kFewPitch<256> * 4 <= kFewRing, "the sums have to fit the stages");
static_assert(kFewAlloc <= 232448, "shared memory above the per-block limit");

// Rows of A in a stage.  (Stored along its rows, A comes in whole boxes.)
__host__ __device__ constexpr int few_rows(int64_t M, bool mn) {
  return mn || M > 120 ? 128 : (int)((M + 7) / 8 * 8);
}

enum FewSums { kOne, kRuns, kPlanes3 };

template <FewSums kSums, int FN, bool AMN, bool BMN, class Epi>
__global__ void __launch_bounds__(kFewThreads, 1) gemm_few_kernel(const __grid_constant__ CUtensorMap ma,
                                                                  const __grid_constant__ CUtensorMap mb,
                                                                  const GemmShape g, const Epi ep, int* status) {
  constexpr bool kPlanes = kSums == kPlanes3;
  // TMEM columns: one accumulator; as many as there are; the first planes' product, behind it the others
  constexpr int kAcc = kSums == kOne ? FN : kSums == kRuns ? 512 : 2 * FN;
  const int a_bytes = few_rows(g.M, AMN) * kBK * 2, stage = a_bytes + FN * kBK * 2;
  const int NS = min(kFewMostStages, kFewRing / stage);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kFewRing);
  uint64_t* empty = full + kFewMostStages;
  uint64_t* acc_full = empty + kFewMostStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kFewMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kFewMiscOff + 4);
  const int warp = warp_id_uniform(), lane = threadIdx.x % 32;
  const int S = g.splits, rank = (int)cluster_rank(), tile = blockIdx.x / S;
  const int n0 = tile / g.tiles_m * FN, m0 = tile % g.tiles_m * 128;   // (tiles of one column band together)
  const int rows = (int)min((int64_t)128, g.M - m0);
  const int kb0 = g.k_blocks * rank / S, kb1 = g.k_blocks * (rank + 1) / S;
  // load `it` into a stage: a k-block, or a plane of one (the middle one, the first, the last)
  auto load = [&](int s, int it) {
    uint8_t *pa = smem + s * stage, *pb = pa + a_bytes;
    const uint32_t bar = smem_u32(full + s);
    const int kb = kb0 + (kPlanes ? it / 3 : it), i3 = it % 3, z = !kPlanes || i3 == 1 ? 0 : i3 == 0 ? 1 : 2;
    mbar_arrive_expect_tx(full + s, stage);
    if (AMN) {
#pragma unroll
      for (int i = 0; i < 2; ++i) tma_load<1>(pa + i * 8192, &ma, bar, m0 + 64 * i, kb * kBK, z);
    } else {
      tma_load<1>(pa, &ma, bar, kb * kBK, m0, z);
    }
    if (BMN) {
#pragma unroll
      for (int i = 0; i < FN / 64; ++i) tma_load<1>(pb + i * 8192, &mb, bar, n0 + 64 * i, kb * kBK, z);
    } else {
      tma_load<1>(pb, &mb, bar, kb * kBK, n0, z);
    }
  };
  const int blocks = (kb1 - kb0) * (kPlanes ? 3 : 1);
  int it = 0;   // the loading thread's place
  let_next_start();
  if (warp == 0) {
    if (lane < NS) {
      mbar_init(full + lane, 1);
      mbar_init(empty + lane, 1);
    } else if (lane == kFewMostStages) {
      mbar_init(acc_full, 1);
      *abort_flag = 0;
    }
    fence_mbar_init();
    __syncwarp();
    if (lane == 0) {
      wait_for_previous();
      // the first round of stages is on its way before anything else is set up
      for (; it < NS && it < blocks; ++it) load(it, it);
    }
  }
  if (warp == 2) tmem_take<1>(tmem_slot, kAcc);
  wait_for_previous();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (warp == 0) {
    if (lane == 0) {
      bool ok = true;
      uint32_t phase = 0;   // of the wait for an emptied stage
      for (int s = 0; it < blocks; ++it) {
        if (!(ok = mbar_wait(empty + s, phase, abort_flag, status))) break;
        load(s, it);
        if (++s == NS) s = 0, phase ^= 1;
      }
      if (!ok)   // the copies issued land before the CTA exits
        for (int i = it > NS ? it - NS : 0; i < it; ++i) mbar_wait_drain(full + i % NS, (i / NS) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    // The whole warp walks the loop, so that what one of its threads issues comes
    // from uniform registers (a lone thread took 130 cycles per MMA of 128 columns,
    // twice what the tensor core takes: 8 x 4096 x 4096 10.7 us, so 8.7.  For the
    // loads it was slower: 9.6).
    const bool leader = elect_one();
    constexpr uint32_t idesc = idesc_bf16_f32(128, FN, AMN, BMN);
    const uint32_t base = smem_u32(smem);
    auto product = [&](int sa, int sb, uint32_t acc, bool add) {
      const uint32_t a0 = base + sa * stage, b0 = base + sb * stage + a_bytes;
      const SDesc da = AMN ? sdesc_sw128_split(a0, 8192, 1024) : sdesc_sw128_split(a0, 16, 1024);
      const SDesc db = BMN ? sdesc_sw128_split(b0, 8192, 1024) : sdesc_sw128_split(b0, 16, 1024);
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < kBK / 16; ++kk)
          umma<1>(acc, sdesc_at(da, kk * (AMN ? 2048 : 32)), sdesc_at(db, kk * (BMN ? 2048 : 32)), idesc,
                  add || kk > 0 ? 1u : 0u);
      }
    };
    uint32_t phase = 0;
    int s = 0;
    auto arrived = [&] {
      if (!__all_sync(0xffffffffu, mbar_wait(full + s, phase, abort_flag, status))) return false;
      tc_fence_after();
      return true;
    };
    auto done = [&](uint64_t* bar) {
      if (leader) umma_done<1>(bar);
    };
    auto next = [&] {
      if (++s == NS) s = 0, phase ^= 1;
    };
    if constexpr (kSums == kOne) {
      for (int it = 0; it < blocks; ++it, next()) {
        if (!arrived()) break;
        product(s, s, tmem, it > 0);
        done(empty + s);
      }
    } else if constexpr (kSums == kRuns) {
      uint32_t acc = tmem;
      for (int it = 0, run = 0; it < blocks; ++it, next()) {
        if (!arrived()) break;
        product(s, s, acc, run > 0);
        done(empty + s);
        if (++run == g.run) run = 0, acc += FN;
      }
    } else {
      for (int it = 0; it < blocks; it += 3) {
        const bool add = it > 0;
        if (!arrived()) break;
        const int mid = s;
        product(mid, mid, tmem + FN, add);
        next();
        if (!arrived()) break;
        const int first = s;
        product(first, mid, tmem + FN, true);
        product(mid, first, tmem + FN, true);
        done(empty + mid);
        product(first, first, tmem, add);
        next();
        if (!arrived()) break;
        product(first, s, tmem + FN, true);
        product(s, first, tmem + FN, true);
        done(empty + first);
        done(empty + s);
        next();
      }
    }
    done(acc_full);   // also after an abort: what was issued is done before TMEM is given back
    mbar_wait_drain(acc_full, 0);
    __syncwarp();
  } else if (warp >= kEpilogueWarp) {
    const int q = warp % 4, half = (warp - kEpilogueWarp) / 4, m = q * 32 + lane;
    if (__all_sync(0xffffffffu, mbar_wait(acc_full, 0, abort_flag, status))) {
      tc_fence_after();
      float* to = reinterpret_cast<float*>(smem) + m * kFewPitch<FN> + half * (FN / 2);
      for (int c = 0; c < FN / 2; c += 32) {
        uint32_t v[32];
        tmem_ld32p(tmem + ((uint32_t)(q * 32) << 16) + half * (FN / 2) + c, v);
        if constexpr (kSums == kOne) tmem_wait_ld();
        const int sums = kPlanes ? 2 : kSums == kOne ? 1 : (blocks + g.run - 1) / g.run;
        for (int r = 1; r < sums; ++r) {
          uint32_t w[32];
          tmem_ld32p(tmem + ((uint32_t)(q * 32) << 16) + r * FN + half * (FN / 2) + c, w);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(w[i]));
        }
        if (m < rows)
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<uint4*>(to + c + i) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
      }
    }
  }
  tc_fence_before();
  // this CTA's share of the columns, FN / S, in bands of 16 through the epilogue; what it reads for a
  // thread's first band is on its way meanwhile
  const int own_n = FN / S, bands = own_n / kBand;
  auto band_at = [&](int i, int& m, int& c) {
    m = i / bands;
    c = (i - m * bands) * kBand;
    return n0 + rank * own_n + c;
  };
  typename Epi::Fetched f;
  int m, c, n = band_at(threadIdx.x, m, c);
  if (threadIdx.x < rows * bands) ep.fetch(f, ep.row(m0 + m), n, true);
  __syncthreads();
  if (warp == 2) tmem_give<1>(tmem, kAcc);
  float* own = reinterpret_cast<float*>(smem) + rank * own_n;
  if (S > 1) {
    cluster_sync();
    // four columns at a time from every CTA into this one's rows (nobody else reads those)
    const int quads = own_n / 4;
    for (int i = threadIdx.x; i < rows * quads; i += kFewThreads) {
      const int r0 = i / quads;
      float4* at = reinterpret_cast<float4*>(own + r0 * kFewPitch<FN>) + (i - r0 * quads);
      float4 w[4];
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (r < S)
          asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(w[r].x), "=f"(w[r].y), "=f"(w[r].z), "=f"(w[r].w)
                       : "r"(map_to(at, r))
                       : "memory");
      float4 v = w[0];
#pragma unroll
      for (int r = 1; r < 4; ++r)
        if (r < S) v.x += w[r].x, v.y += w[r].y, v.z += w[r].z, v.w += w[r].w;
      *at = v;
    }
    cluster_arrive();   // (the others' memory is read)
    __syncthreads();
  }
  for (int i = threadIdx.x; i < rows * bands; i += kFewThreads) {
    if (i >= kFewThreads) {
      n = band_at(i, m, c);
      ep.fetch(f, ep.row(m0 + m), n, true);
    }
    if (n >= g.N || *abort_flag) continue;
    float v[kBand];
#pragma unroll
    for (int j = 0; j < kBand; j += 4) {
      const float4 w = *reinterpret_cast<const float4*>(own + m * kFewPitch<FN> + c + j);
      v[j] = w.x, v[j + 1] = w.y, v[j + 2] = w.z, v[j + 3] = w.w;
    }
    ep.put(f, ep.row(m0 + m), n, 0, v);
  }
  if (S > 1) cluster_wait();   // the others have read this CTA's memory
}

// Sum of the parts' sums, then the epilogue: a thread takes 16 columns of a row.
template <class Epi>
__global__ void __launch_bounds__(128) gemm_sum_kernel(const float* part, int splits, int64_t M, int N, const Epi ep) {
  let_next_start();
  wait_for_previous();
  const int bands = (N + kBand - 1) / kBand;
  const int64_t i = (int64_t)blockIdx.x * 128 + threadIdx.x;
  if (i >= M * bands) return;
  const int64_t m = i / bands;
  const int n = (int)(i - m * bands) * kBand;
  float v[kBand];
  typename Epi::Fetched f;
  const int64_t row = ep.row(m);
  ep.fetch(f, row, n, true);
  const float* p = part + m * N + n;
#pragma unroll
  for (int c = 0; c < 2; ++c)
    if (n + 8 * c < N) load_f8(p + 8 * c, *reinterpret_cast<float(*)[8]>(v + 8 * c));
  for (int s = 1; s < splits; ++s) {
    p += M * N;
#pragma unroll
    for (int c = 0; c < 2; ++c)
      if (n + 8 * c < N) {
        float w[8];
        load_f8(p + 8 * c, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[8 * c + j] += w[j];
      }
  }
  ep.put(f, row, n, 0, v);
}

// ------------------------------------------------------------------- host --

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    return cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
                   q == cudaDriverEntryPointSuccess
               ? reinterpret_cast<EncodeTiledFn>(p)
               : nullptr;
  }();
  return fn;
}

struct Operand {
  const void* p;
  int64_t pitch;   // elements between rows
};

// `planes` of [rows, inner] bf16 row-major, boxes of 64 x box_rows with 128-byte
// swizzle; what lies outside a plane reads as zero.
cudaError_t make_map(CUtensorMap* m, const Operand& o, int planes, int64_t rows, int64_t inner, int box_rows) {
  const void* base = o.p;
  const int64_t pitch = o.pitch;
  EncodeTiledFn fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)rows, (cuuint64_t)planes};
  cuuint64_t strides[2] = {(cuuint64_t)pitch * 2, (cuuint64_t)(rows * pitch) * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

struct GemmPlan {
  int cg;        // CTAs per tile; 0: the few-rows kernel
  int few_n;     // and its tiles' columns
  bool sum;      // the accumulator's runs are added up in registers (kSum; kRuns)
  GemmShape g;
};

// k-blocks that the sums of a bf16 result may be cut over: 8192 of the depth, which
// draw a sum of positive terms towards zero by 3.6e-5 (measured; 1/100 of a rounding
// to bf16), one of random signs by 1e-5.  Never emptied, the accumulator took 7.9e-4 off a
// sum of 131072 positive terms, and 6e-3 off one of a million.  Emptying it costs nothing where
// every pair has a tile (dw of 4096 x 4096 over 65536 tokens 1554 us without, 1557 with;
// with runs of 2048 1577), and 5 to 10 % with 40 tiles for 74 pairs (2048 x 1032).
constexpr int kDeep = 128;

// exact: the sums of the accumulator's runs are to be rounded, not cut.  A part
// of one run needs no adding up (of fp32, one run of the last plane product: the
// ones before it are small); nor does one of kDeep for a result rounded to bf16.
GemmPlan gemm_plan(int64_t M, int64_t N, int64_t K, int planes, bool exact) {
  GemmPlan pl;
  auto tiles = [](int64_t x, int64_t t) { return (int)((x + t - 1) / t); };
  GemmShape& g = pl.g;
  g.M = M;
  g.N = N;
  g.tiles_n = tiles(N, kBN);
  g.k_blocks = tiles(K, kBK);
  g.pairs = planes == 3 ? kPairs : 1;
  g.run = planes == 3 ? 16 : exact ? 32 : kDeep;
  // Large tiles.  Few of them: as many parts as fill the GPU, each of eight
  // k-blocks' work at least (below 32 the second kernel costs more than the
  // parts save).
  // (Up to 128 rows fill half a pair's tile, but of much depth the parts gain more: dw of
  // 64 x 912 over 81920 tokens 87 us with the few-rows kernel, 51 so.)
  pl.cg = exact && M <= 128 ? 1 : 2;
  g.tiles_m = tiles(M, 128 * pl.cg);
  const int64_t slots = sm_count() / pl.cg, t = (int64_t)g.tiles_m * g.tiles_n;
  const int64_t work = (int64_t)g.k_blocks * g.pairs;   // k-blocks of a tile
  int64_t splits = work < 32 ? 1 : slots / t;
  if (splits > work / 8) splits = work / 8;
  if (splits > g.k_blocks) splits = g.k_blocks;
  if (splits < 1) splits = 1;
  g.blocks_per_split = (int)((g.k_blocks + splits - 1) / splits);
  g.splits = (g.k_blocks + g.blocks_per_split - 1) / g.blocks_per_split;
  pl.sum = g.blocks_per_split > g.run;

  // Or the few-rows kernel's tiles, of 128 or 256 columns, whose clusters are to be
  // resident all at once (33 of 4 CTAs, 74 of 2: cudaOccupancyMaxActiveClusters; 16
  // of 8 where 15 fit took 20 us against 14).  The times in us that decide were
  // fitted to 24 products from 8 x 4096 x 4096 to 4096 x 2048 x 1024: 256 x 4096 x
  // 4096 takes 20.1 with large tiles, 13.4 and 15.5 with these; 1024 x 1024 x 1024
  // 12.4, 8.9 and 11.6; 1024 x 4096 x 4096 27.5 and, with 256 columns, 27.5.  For
  // fp32 to 30 (with the splitting): 1024 x 1024 x 1024 takes 27.0, 22.0 and 23.7;
  // 1024 x 1024 x 4096 64.1 and, in parts of a run, 56.8 with 256 columns.
  // Up to 128 rows, 128 columns may also come in waves, all but the first bound by the
  // weights' bytes, as large tiles' are there: 8 x 20480 x 4096 takes 39.5 us in two waves and
  // 33.1 with 256 columns in one, 8 x 65536 x 4096 90 in four and 112 with large tiles.
  const int64_t waves = (t * g.splits + slots - 1) / slots;
  const double block = M <= 128 && waves > 1 ? 0.45 : 0.29;
  double best = (g.splits > 1 ? 14.0 + 0.5 * g.splits : 7.5) + block * g.blocks_per_split * g.pairs * waves;
  const int64_t k_blocks = g.k_blocks;
  for (int n : {128, 256}) {
    const int64_t few_tiles = (int64_t)tiles(M, 128) * tiles(N, n);
    if (few_tiles > sm_count() && (M > 128 || n == 256)) continue;
    const int S = few_tiles <= 33 && k_blocks >= 8 ? 4 : few_tiles <= 74 && k_blocks >= 4 ? 2 : 1;
    if (tiles(k_blocks, S) > (exact ? 1 : 512 / n) * g.run) continue;   // (512 columns of accumulators)
    const double part = tiles(k_blocks, S), turns = (double)((few_tiles + sm_count() - 1) / sm_count());
    const double cost = planes == 3  ? turns * (n == 128 ? 7.0 + 1.15 * part : 10.0 + 1.9 * part)
                        : turns > 1  ? turns * (2.6 + 0.34 * part)
                        : n == 128   ? 7.3 + 0.17 * part
                                     : 10.2 + 0.31 * part;
    if (cost > best && pl.cg != 1) continue;   // (one-CTA large tiles only where it must be)
    best = cost;
    pl.cg = 0;
    pl.few_n = n;
    pl.sum = tiles(k_blocks, S) > g.run;
    g.tiles_m = tiles(M, 128);
    g.tiles_n = tiles(N, n);
    g.splits = S;
    g.blocks_per_split = 0;
  }
  return pl;
}

bool aligned32(const void* p) { return reinterpret_cast<uintptr_t>(p) % 32 == 0; }

template <typename T>
EpiPlain<T> plain(void* c, int64_t M, int64_t N) {
  return {static_cast<T*>(c), M, (int)N, aligned32(c) && N * sizeof(T) % 32 == 0};
}

template <class Kernel, class Epi>
cudaError_t launch_gemm(Kernel kern, int ctas, int threads, int cluster, int smem, const CUtensorMap& ma,
                        const CUtensorMap& mb, const GemmShape& g, const Epi& ep, int* status, bool after,
                        cudaStream_t st) {
  if (cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) return e;
  return launch_chained(kern, dim3((unsigned)ctas), threads, smem, cluster, after, st, ma, mb, g, ep, status);
}

template <int CG, bool AMN, bool BMN, bool kSum, class Epi>
cudaError_t run_gemm(const GemmPlan& pl, const CUtensorMap& ma, const CUtensorMap& mb, const Epi& ep, int* status,
                     bool after, cudaStream_t st) {
  const GemmShape& g = pl.g;
  auto kern = gemm_tc_kernel<CG, AMN, BMN, kSum, Epi>;
  static const int regs = [&] {
    cudaFuncAttributes fa;
    return cudaFuncGetAttributes(&fa, kern) == cudaSuccess ? fa.numRegs : 0;
  }();
  if (kSum && 128 * kRegsCtl + 256 * kRegsEpilogue > kGemmThreads<true> * regs) return cudaErrorInvalidConfiguration;
  const int64_t units = (int64_t)g.tiles_m * g.tiles_n * g.splits, slots = sm_count() / CG;
  return launch_gemm(kern, (int)(CG * (units < slots ? units : slots)), kGemmThreads<kSum>, CG, GemmCfg<CG>::kAlloc, ma,
                     mb, g, ep, status, after, st);
}

// A and B: bf16, or (planes = 3) the bf16 planes of fp32 operands.
template <int planes, bool AMN, bool BMN, bool kExact, class Epi>
cudaError_t gemm(int64_t M, int64_t N, int64_t K, const Operand& A, const Operand& B, const Epi& ep, void* ws,
                 int* status, bool after, cudaStream_t st) {
  const GemmPlan pl = gemm_plan(M, N, K, planes, kExact);
  CUtensorMap ma, mb;
  cudaError_t e;
  const int b_rows = pl.cg == 2 ? kBN / 2 : pl.cg == 1 ? kBN : pl.few_n;
  if ((e = AMN ? make_map(&ma, A, planes, K, M, kBK)
               : make_map(&ma, A, planes, M, K, pl.cg == 0 ? few_rows(M, false) : 128))) return e;
  if ((e = BMN ? make_map(&mb, B, planes, K, N, kBK) : make_map(&mb, B, planes, N, K, b_rows))) return e;
  if (pl.cg == 0) {
    constexpr FewSums kSums = planes == 3 ? kPlanes3 : kOne, kDeepSums = kExact ? kSums : kRuns;
    const auto kern = pl.few_n == 128 ? pl.sum ? gemm_few_kernel<kDeepSums, 128, AMN, BMN, Epi>
                                               : gemm_few_kernel<kSums, 128, AMN, BMN, Epi>
                      : pl.sum        ? gemm_few_kernel<kDeepSums, 256, AMN, BMN, Epi>
                                      : gemm_few_kernel<kSums, 256, AMN, BMN, Epi>;
    return launch_gemm(kern, pl.g.tiles_m * pl.g.tiles_n * pl.g.splits, kFewThreads, pl.g.splits, kFewAlloc, ma, mb,
                       pl.g, ep, status, after, st);
  }
  auto product = [&](const auto& out) -> cudaError_t {
    using Out = std::decay_t<decltype(out)>;
    if constexpr (kExact) {
      // (one CTA per tile: only where the few-rows kernel would not be exact)
      if (pl.cg == 1)
        return pl.sum ? run_gemm<1, AMN, BMN, true, Out>(pl, ma, mb, out, status, after, st)
                      : run_gemm<1, AMN, BMN, false, Out>(pl, ma, mb, out, status, after, st);
    }
    if (pl.cg != 2) return cudaErrorInvalidValue;   // (the maps are made for pl.cg)
    return pl.sum ? run_gemm<2, AMN, BMN, true, Out>(pl, ma, mb, out, status, after, st)
                  : run_gemm<2, AMN, BMN, false, Out>(pl, ma, mb, out, status, after, st);
  };
  if (pl.g.splits == 1) return product(ep);
  float* part = static_cast<float*>(ws);
  if ((e = product(EpiPlain<float>{part, M, (int)N, aligned32(part)}))) return e;
  return launch_chained(gemm_sum_kernel<Epi>, dim3((unsigned)((M * ((N + kBand - 1) / kBand) + 127) / 128)), 128, 0, 0,
                        true, st, part, pl.g.splits, M, (int)N, ep);
}

// x or w: rows of the tensor, or of its planes.
Operand operand(const LinearProblem& p, const void* at, int64_t inner) {
  return {at, p.dtype == kBF16 ? inner : plane_pitch(inner)};
}

template <typename T>
cudaError_t forward_tc(const LinearProblem& p, const void* xp, const void* wp, void* ws, bool after, cudaStream_t st) {
  const Operand x = operand(p, xp, p.K), w = operand(p, wp, p.K);
  const int64_t run = p.H ? p.N / p.H : p.N;   // contiguous columns
  const EpiForward<T> ep{p.bias, static_cast<const T*>(p.residual), static_cast<T*>(p.y), p.pre, OutLayout(p), p.act,
                         aligned32(p.y) && run % 16 == 0, aligned32(p.pre)};
  constexpr int planes = sizeof(T) == 4 ? 3 : 1;
  if constexpr (planes == 1)
    if (!p.pre) return gemm<1, false, false, false>(p.M(), p.N, p.K, x, w, ep, ws, p.status, after, st);
  return gemm<planes, false, false, true>(p.M(), p.N, p.K, x, w, ep, ws, p.status, after, st);
}

}  // namespace

size_t gemm_tc_workspace(int64_t M, int64_t N, int64_t K, int dtype) {
  size_t most = 0;
  for (bool exact : {false, true}) {
    const GemmPlan pl = gemm_plan(M, N, K, dtype == kBF16 ? 1 : 3, exact);
    const size_t n = pl.cg == 0 || pl.g.splits == 1 ? 0 : sizeof(float) * (size_t)pl.g.splits * M * N;
    if (n > most) most = n;
  }
  return most;
}

cudaError_t launch_linear_tc(const LinearProblem& p, const void* x, const void* w, void* ws, bool after,
                             cudaStream_t st) {
  return p.dtype == kBF16 ? forward_tc<__nv_bfloat16>(p, x, w, ws, after, st)
                          : forward_tc<float>(p, x, w, ws, after, st);
}

cudaError_t launch_linear_dx_tc(const LinearProblem& p, const void* dup, int64_t du_pitch, const void* wp, void* ws,
                                bool after, cudaStream_t st) {
  const Operand du{dup, du_pitch}, w = operand(p, wp, p.K);
  if (p.dtype == kBF16)
    return gemm<1, false, true, false>(p.M(), p.K, p.N, du, w, plain<__nv_bfloat16>(p.dx, p.M(), p.K), ws, p.status,
                                       after, st);
  return gemm<3, false, true, true>(p.M(), p.K, p.N, du, w, plain<float>(p.dx, p.M(), p.K), ws, p.status, after, st);
}

cudaError_t launch_linear_dw_tc(const LinearProblem& p, const void* dup, int64_t du_pitch, const void* xp, void* ws,
                                bool after, cudaStream_t st) {
  const Operand du{dup, du_pitch}, x = operand(p, xp, p.K);
  if (p.dtype == kBF16)
    return gemm<1, true, true, false>(p.N, p.K, p.M(), du, x, plain<__nv_bfloat16>(p.dw, p.N, p.K), ws, p.status,
                                      after, st);
  return gemm<3, true, true, true>(p.N, p.K, p.M(), du, x, plain<float>(p.dw, p.N, p.K), ws, p.status, after, st);
}

}  // namespace gecko
