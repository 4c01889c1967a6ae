// mx_matmul.cu -- the product of two microscaled 4-bit matrices (include/zipnn.h) on the
// tensor cores: D = A B^T, the scales applied by the matrix instruction itself.
//
// One block computes 128 rows of one operand (P) against BN of the other (Q), over a range of
// the columns, in stages of 256 columns: 128 bytes of codes a row, brought by TMA in the
// 128-byte swizzle that tcgen05.mma reads, and the scales' 512-byte tiles, which lie in memory
// as tcgen05.cp takes them. One thread feeds TMA, one issues the matrix instructions (K = 64
// each, accumulating FP32 in tensor memory), four warps read the sums back and store them.
//
// What bounds it: few rows, what the busy SMs can draw behind 2.7 us of launch, first load and
// sums (1 x 11008 x 4096, 86 blocks and 24 MB: MXFP4 8.7 us and NVFP4 9.6 us where the weights come
// from HBM, over 450 MB of them in turn, 6.9 and 8.1 us where they lie in L2); many rows, the way
// from L2 to shared memory and, repeated, the 1000 W limit (4096 x 11008 x 4096: 72 us, 5.1 PFLOP/s,
// and 77 us in NVFP4; back to back 88 us at 1.6 GHz).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

#include "zipnn.h"
#include "bulk.cuh"
#include "common.cuh"
#include "mx.cuh"
#include "op_ids.h"

namespace zipnn {
namespace {

constexpr int kThreads = 192;
constexpr uint32_t kStageBytesK = 128;  // code bytes of a row in a stage: 256 values
constexpr uint32_t kStageK = 256, kMmaK = 64;
// Polls after which a wait gives up (zipnn_test_mx_wait_limit lowers it for some blocks), and
// always those of the waits that follow one that gave up: for what is still in flight. A poll
// that finds nothing takes some microseconds.
constexpr uint32_t kWaitPolls = 1u << 22;
constexpr uint32_t kOtherPolls = 1u << 10;  // of the other blocks, while a limit is set for some
constexpr uint32_t kNoLimit = kWaitPolls << 6;
std::atomic<uint32_t> g_wait_limit{kNoLimit};  // polls << 6 | mask << 3 | value

// ZIPNN_ERR_TIMEOUT after a wait that gave up, until zipnn_mx_status takes it.
__device__ uint32_t g_mx_status;

struct Args {
  const uint8_t *p_scales, *q_scales;
  const float *ga, *gb;  // the tensors' scales (NVFP4)
  uint8_t* out;
  uint64_t ldo;
  uint32_t p_rows, q_rows, q_tiles;
  uint32_t col_tiles;          // scale tiles along a row
  uint32_t stages, mmas;       // of the whole row
  uint32_t split;              // blocks of a cluster, each a range of the stages
  // One word: with eight bytes more of arguments a product takes 0.1 to 0.4 us longer.
  // Blocks whose number, masked, is `value` (all of them, by default) wait for `polls`.
  uint32_t depth : 3, value : 3, mask : 3, polls : 23;
  uint32_t tmem_cols;
  int type, p_is_n;
};

constexpr uint32_t kAllShared = 227 * 1024;  // of an SM
constexpr uint32_t kSmallest = 80 * 1024;  // below the shared memory of every block here

template <int FMT, int BN>
struct Shape {
  static constexpr uint32_t kTiles = kStageK / (4 * mx_block(FMT));  // scale tiles of a stage along a row: 2 or 4
  static constexpr uint32_t kP = 128 * kStageBytesK, kQ = BN * kStageBytesK, kScales = kTiles * kMxTileBytes;
  static constexpr uint32_t kStage = (kP + kQ + 2 * kScales + 1023) / 1024 * 1024;
  // Stages in flight. Where the grid has more blocks than the device has SMs, two share one
  // (100 x 32000 x 4096: 17.2 us, and 20.3 us with one block and its deeper ring); else a
  // block has the SM's shared memory to itself (128 x 11008 x 4096: 9.6 us, and 10.8 with 3).
  static constexpr uint32_t kHalf = (113 * 1024 - 1280) / kStage, kShared = kHalf < 4 ? kHalf : 4, kAlone = BN <= 64 ? 6 : 5;
  static constexpr uint32_t smem(uint32_t depth) { return depth * kStage + 1024 + 256; }
  static_assert(kShared * kStage >= kSmallest, "the smallest block");
  // Tensor memory: the sums, and a set of scales for each stage in shared memory (4 columns a
  // tile), so that a set is written again only after the instructions that read it are done:
  // the stage's codes were not brought before that either.
  static constexpr uint32_t kScaleCols = 2 * 4 * kTiles;
  static constexpr uint32_t cols(uint32_t depth) {
    const uint32_t used = BN + depth * kScaleCols;
    return used <= 64 ? 64 : used <= 128 ? 128 : used <= 256 ? 256 : 512;
  }
  static_assert(smem(kAlone) <= kAllShared && BN + kAlone * kScaleCols <= 512, "one block to an SM");
  // Two blocks on an SM, of one call or of two, never wait for each other's tensor memory
  // (which could close a ring of clusters): a block that leaves room for another one's shared
  // memory takes at most half of it.
  static_assert(cols(kShared) <= 256 && (cols(kAlone) <= 256 || smem(kAlone) + kSmallest > kAllShared), "tensor memory");
};

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ void tma_2d(void* dst, const CUtensorMap* map, int32_t x, int32_t y, uint64_t* bar) {
  asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
                   smem_addr(dst)),
               "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
               : "memory");
}

// Shared-memory descriptors: rows of 128 bytes in the 128-byte swizzle (groups of 8 rows 1024
// bytes apart), and unswizzled 16-byte rows (groups of 8 rows 128 bytes apart).
__device__ __forceinline__ uint64_t desc_codes(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFF) >> 4) | 1ull << 16 | (uint64_t)(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
__device__ __forceinline__ uint64_t desc_scales(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFF) >> 4) | (uint64_t)(128 >> 4) << 32 | 1ull << 46;
}

__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t addr) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc_scales(addr)) : "memory");
}

// One lane of a warp that is converged here. The loops around the instructions for the tensor
// cores and TMA are run by the whole warp, and only the instructions themselves by this lane:
// their operands live in uniform registers, which a branch on the lane number around the loops
// would put out of reach (a 4096 x 11008 x 4096 product took 118 us so, moving each operand there).
__device__ __forceinline__ bool elect() {
  uint32_t e;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(e));
  return e != 0;
}
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }

// A ring of stages: the place of the next one, and how often the ring was gone round (mod 2).
struct Ring {
  uint32_t at = 0, parity = 0;
  __device__ __forceinline__ void next(uint32_t depth) {
    if (++at == depth) at = 0, parity ^= 1;
  }
};

// Which two of a column's four scale bytes an MXFP4 instruction takes is part of its
// descriptor; an NVFP4 instruction takes all four.
template <int FMT, int BN>
__device__ __forceinline__ constexpr uint32_t instr(uint32_t scale_id) {
  return scale_id << 4 | 1u << 7 | 1u << 10 | (uint32_t)(BN / 8) << 17 | (FMT == kMxFp4 ? 1u : 0u) << 23 | 1u << 27 | scale_id << 29;
}

template <int FMT>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb, bool add) {
  if constexpr (FMT == kMxFp4) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"((uint32_t)add)
        : "memory");
  } else {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"((uint32_t)add)
        : "memory");
  }
}

__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ void load_sums(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; i++) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 load_peer(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ uint32_t load_peer_word(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ uint32_t polls_of(const Args& a) { return (blockIdx.x & a.mask) == a.value ? a.polls : kOtherPolls; }
// A whole warp's wait, of whose outcome its lanes agree, since they go on together. (A look at
// `failed` in it, to give up where another wait has, costs a large product 5 to 17%.)
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint32_t polls) {
  return __all_sync(0xFFFFFFFFu, mbar_wait_bounded(bar, parity, polls));
}

template <typename T>
__device__ __forceinline__ T to_value(float v) {
  if constexpr (sizeof(T) == 4) return v;
  else return T(v);
}
// N values to every `step`th place from `out`, the first n of them.
template <typename T, int N>
__device__ __forceinline__ void put(T* out, uint64_t step, uint32_t n, const float* v) {
  if (n >= (uint32_t)N) {
#pragma unroll
    for (int c = 0; c < N; c++) out[c * step] = to_value<T>(v[c]);
  } else {
#pragma unroll
    for (int c = 0; c < N; c++)
      if ((uint32_t)c < n) out[c * step] = to_value<T>(v[c]);
  }
}
// The product of the two tensors' scales (NVFP4): in FP32 where it is an ordinary number, else
// the sums are scaled in 64 bits, so that neither scale alone takes a result out of range.
struct Scale {
  float f;
  double d;
  bool usual;
};
template <int FMT>
__device__ __forceinline__ Scale scale_of(const Args& a) {
  Scale s = {1.f, 1.0, true};
  if constexpr (FMT == kNvFp4) {
    s.d = (double)*a.ga * (double)*a.gb;
    s.f = (float)s.d;
    s.usual = s.d >= 1e-36 && s.d <= 1e36;
  }
  return s;
}

// The sums of row p of P and rows q .. q + N - 1 of Q, scaled and rounded.
template <int FMT, int N>
__device__ __forceinline__ void store(const Args& a, uint32_t p, uint32_t q, float* v, const Scale& g) {
  if (p >= a.p_rows || q >= a.q_rows) return;
  if constexpr (FMT == kNvFp4) {
    if (g.usual) {
#pragma unroll
      for (int c = 0; c < N; c++) v[c] *= g.f;
    } else {
#pragma unroll
      for (int c = 0; c < N; c++) v[c] = (float)((double)v[c] * g.d);
    }
  }
  const uint64_t at = a.p_is_n ? (uint64_t)q * a.ldo + p : (uint64_t)p * a.ldo + q, step = a.p_is_n ? a.ldo : 1;
  if (a.type == kValFP32) put<float, N>(reinterpret_cast<float*>(a.out) + at, step, a.q_rows - q, v);
  else if (a.type == kValBF16) put<__nv_bfloat16, N>(reinterpret_cast<__nv_bfloat16*>(a.out) + at, step, a.q_rows - q, v);
  else put<__half, N>(reinterpret_cast<__half*>(a.out) + at, step, a.q_rows - q, v);
}

// What a block of a cluster that gave up leaves in place of its sums: a NaN that no sum is, since
// the tensor cores' is 0x7FFFFFFF.
constexpr uint32_t kLost = 0x7FC0DEADu;

// The sums of a block of a cluster lie in its shared memory as (columns / 4, 128 rows, 4).
// This block's share of the columns of this thread's row: every SPLIT-th four, added over the
// blocks in their order. Eight loads are in flight at a time (each takes a good part of a
// microsecond). Nothing is stored where a block's sums are not whole (kLost).
template <int FMT, int SPLIT>
__device__ __forceinline__ void add_peers(const Args& a, const float4* sums, uint32_t rank, uint32_t used, uint32_t p, uint32_t q,
                                          const Scale& g) {
  constexpr uint32_t kAtOnce = 8 / SPLIT;
  for (uint32_t c = rank * 4; c < used; c += kAtOnce * SPLIT * 4) {
    float4 t[kAtOnce][SPLIT];
#pragma unroll
    for (uint32_t k = 0; k < kAtOnce; k++)
#pragma unroll
      for (int r = 0; r < SPLIT; r++)
        if (c + k * SPLIT * 4 < used) t[k][r] = load_peer(peer(smem_addr(sums + (c / 4 + k * SPLIT) * 128 + threadIdx.x), r));
#pragma unroll
    for (uint32_t k = 0; k < kAtOnce; k++) {
      if (c + k * SPLIT * 4 >= used) break;
      float4 v = t[k][0];
      if (k == 0 && c == rank * 4) {  // all of a block's sums are marked, or none
        bool lost = false;
#pragma unroll
        for (int r = 0; r < SPLIT; r++) lost |= __float_as_uint(t[k][r].x) == kLost;
        if (lost) return;
      }
#pragma unroll
      for (int r = 1; r < SPLIT; r++) v.x += t[k][r].x, v.y += t[k][r].y, v.z += t[k][r].z, v.w += t[k][r].w;
      store<FMT, 4>(a, p, q + c + k * SPLIT * 4, &v.x, g);
    }
  }
}

// Waits for the stages that were brought and not used and for the instructions issued, before the
// block's memory goes to another one. Out of line, since it costs products up to 0.1 us in line.
__device__ __noinline__ void drain(uint64_t* full, uint64_t* done, uint32_t issued, uint32_t brought, uint32_t depth) {
  for (uint32_t i = issued; i < brought; i++) mbar_wait_bounded(full + i % depth, i / depth & 1, kWaitPolls);
  mbar_wait_bounded(done, 0, kWaitPolls);
}

template <int FMT, int BN>
__global__ void __launch_bounds__(kThreads) k_mx_matmul(const __grid_constant__ CUtensorMap p_map,
                                                        const __grid_constant__ CUtensorMap q_map, const Args a) {
  using S = Shape<FMT, BN>;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + a.depth * S::kStage);
  uint64_t *empty = full + a.depth, *done = empty + a.depth;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(done + 1);
  volatile uint32_t *failed = tmem_at + 1, *brought = failed + 1, *issued = failed + 2;  // stages brought and used

  const uint32_t warp = uniform(threadIdx.x / 32);
  const uint32_t tile = blockIdx.x / a.split, rank = blockIdx.x % a.split, polls = polls_of(a);
  const uint32_t p0 = tile / a.q_tiles * 128, q0 = tile % a.q_tiles * BN;
  const uint32_t lo = (uint32_t)((uint64_t)a.stages * rank / a.split), hi = (uint32_t)((uint64_t)a.stages * (rank + 1) / a.split);

  // Stage i of the row into place `at` of the ring. Scale tiles that the row does not have are
  // not brought.
  const auto bring = [&](uint32_t i, uint32_t at) {
    uint8_t* st = smem + at * S::kStage;
    uint64_t* bar = full + at;
    const uint32_t t0 = i * S::kTiles, bytes = min(S::kTiles, a.col_tiles - t0) * kMxTileBytes;
    mbar_expect_tx(bar, S::kP + S::kQ + 2 * bytes);
    tma_2d(st, &p_map, (int32_t)(i * kStageBytesK), (int32_t)p0, bar);
    tma_2d(st + S::kP, &q_map, (int32_t)(i * kStageBytesK), (int32_t)q0, bar);
    uint8_t* sc = st + S::kP + S::kQ;
    bulk_g2s(sc, a.p_scales + ((uint64_t)(p0 / 128) * a.col_tiles + t0) * kMxTileBytes, bytes, bar);
    bulk_g2s(sc + S::kScales, a.q_scales + ((uint64_t)(q0 / 128) * a.col_tiles + t0) * kMxTileBytes, bytes, bar);
  };
  const uint32_t early = min(hi - lo, a.depth);  // stages brought before the block has met
  if (warp == 4) {
    if (elect()) {
      prefetch_map(&p_map);
      prefetch_map(&q_map);
      for (uint32_t i = 0; i < a.depth; i++) {
        mbar_init(full + i, 1);
        mbar_init(empty + i, 1);
      }
      mbar_init(done, 1);
      *failed = 0;
      for (uint32_t i = 0; i < early; i++) bring(lo + i, i);
    }
    __syncwarp();
  }
  if (warp == 5) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_at)), "r"(a.tmem_cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = uniform(*reinterpret_cast<volatile uint32_t*>(tmem_at));

  if (warp == 4) {
    const bool one = elect();
    Ring r;
    uint32_t i = lo + early;
    for (; i < hi; i++, r.next(a.depth)) {
      if (!warp_wait(empty + r.at, r.parity, polls)) {
        *failed = 1;
        break;
      }
      if (one) bring(i, r.at);
      __syncwarp();
    }
    *brought = i - lo;
  } else if (warp == 5) {
    const bool one = elect();
    Ring r;
    uint32_t i = lo, left = a.mmas - lo * (kStageK / kMmaK);  // instructions to the end of the row
    for (; i < hi; i++, r.next(a.depth), left -= kStageK / kMmaK) {
      if (!warp_wait(full + r.at, r.parity, polls)) {
        *failed = 1;
        break;
      }
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t st = smem_addr(smem) + r.at * S::kStage, sc = st + S::kP + S::kQ;
      const uint32_t tp = tmem + BN + r.at * S::kScaleCols, tq = tp + 4 * S::kTiles;
      if (one) {
        // scale tiles that the row does not have are copied too: nothing reads them
#pragma unroll
        for (uint32_t t = 0; t < S::kTiles; t++) {
          copy_scales(tp + 4 * t, sc + t * kMxTileBytes);
          copy_scales(tq + 4 * t, sc + S::kScales + t * kMxTileBytes);
        }
#pragma unroll
        for (uint32_t k = 0; k < kStageK / kMmaK; k++) {
          if (k >= left) break;
          const uint32_t t = FMT == kMxFp4 ? k / 2 : k, id = FMT == kMxFp4 ? k % 2 * 2 : 0;
          mma<FMT>(tmem, desc_codes(st + k * 32), desc_codes(st + S::kP + k * 32), instr<FMT, BN>(id), tp + 4 * t,
                   tq + 4 * t, i + k > lo);
        }
        commit(empty + r.at);
      }
      __syncwarp();
    }
    if (one) commit(done);
    __syncwarp();
    *issued = i - lo;
  } else {
    if (!warp_wait(done, 0, polls)) *failed = 1;
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  }
  __syncthreads();
  const bool ok = *failed == 0;
  if (!ok) {
    if (threadIdx.x == 0) atomicMax(&g_mx_status, kStTimeout);
    if (warp == 5) {
      drain(full, done, *issued, *brought, a.depth);
    }
    __syncthreads();
  }
  const Scale g = scale_of<FMT>(a);
  const uint32_t used = min((uint32_t)BN, a.q_rows - q0);  // columns that the output has
  if (a.split == 1) {
    if (warp < 4 && ok) {
#pragma unroll 1
      for (uint32_t c = 0; c < used; c += 16) {
        float v[16];
        load_sums(tmem + (warp * 32 << 16) + c, v);
        store<FMT, 16>(a, p0 + threadIdx.x, q0 + c, v, g);
      }
    }
  } else {
    // each block's sums to its shared memory (its stages are spent), then every block adds its
    // share of the columns over the cluster
    float4* sums = reinterpret_cast<float4*>(smem);
    if (warp < 4) {
#pragma unroll 1
      for (uint32_t c = 0; c < used; c += 16) {
        float v[16];
        load_sums(tmem + (warp * 32 << 16) + c, v);
        if (!ok) {
#pragma unroll
          for (int k = 0; k < 16; k++) v[k] = __uint_as_float(kLost);
        }
#pragma unroll
        for (int k = 0; k < 16; k += 4) sums[(c + k) / 4 * 128 + threadIdx.x] = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
      }
    }
    cluster_sync();
    if (warp < 4) {
      const uint32_t p = p0 + threadIdx.x;
      if (a.split == 2) add_peers<FMT, 2>(a, sums, rank, used, p, q0, g);
      else if (a.split == 4) add_peers<FMT, 4>(a, sums, rank, used, p, q0, g);
      else add_peers<FMT, 8>(a, sums, rank, used, p, q0, g);
    }
    __syncwarp();
    cluster_sync();
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == 5) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(a.tmem_cols));
  }
}

// ---- Two blocks to a tile --------------------------------------------------------------
// Large products are bound by what the codes' tiles cost between L2 and shared memory: a stage
// of a 128 x 128 tile brings 34 KB for 256 cycles of the tensor cores. Here the two blocks of a
// cluster compute 256 x 256 together (cta_group::2): each brings its own 128 rows of P and half
// of the rows of Q, and both read both halves. One thread of the first block issues the
// instructions for both, and the sums of a tile leave tensor memory through the registers of
// eight warps, whose stores overlap with the next tile's instructions. Blocks walk over the
// tiles, one pair on two SMs.
constexpr int kPairThreads = 320, kPairCols = 256;

template <int FMT>
struct PairShape {
  static constexpr int BN = kPairCols;
  static constexpr uint32_t kTiles = kStageK / (4 * mx_block(FMT));
  static constexpr uint32_t kHalves = BN / 128;  // row tiles of Q's scales: every block needs all of them
  static constexpr uint32_t kP = 128 * kStageBytesK, kQ = BN / 2 * kStageBytesK;
  static constexpr uint32_t kSp = kTiles * kMxTileBytes, kSq = kSp * kHalves;
  static constexpr uint32_t kBytes = kP + kQ + kSp + kSq;
  static constexpr uint32_t kStage = (kBytes + 1023) / 1024 * 1024;
  static constexpr uint32_t kScaleCols = 4 * kTiles * (1 + kHalves);
  static constexpr uint32_t kFit = (kAllShared - 1024 - 512) / kStage, kRoom = (512 - BN) / kScaleCols;
  static constexpr uint32_t kDepth = kFit < kRoom ? kFit : kRoom;
  static_assert(kDepth * kStage + 1024 + 512 <= kAllShared, "one block to an SM, with all of the tensor memory");
};

__device__ __forceinline__ void tma_pair_2d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, uint32_t bar) {
  asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
               "l"(map), "r"(x), "r"(y), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void tma_pair_3d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z, uint32_t bar) {
  asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
               "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void pair_copy_scales(uint32_t taddr, uint32_t addr) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc_scales(addr)) : "memory");
}
template <int FMT>
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb, bool add) {
  if constexpr (FMT == kMxFp4) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"((uint32_t)add)
        : "memory");
  } else {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"((uint32_t)add)
        : "memory");
  }
}
// Arrives at the barrier of both blocks when the instructions issued so far are done.
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_addr(bar)),
               "h"((uint16_t)3)
               : "memory");
}
// Arrives at this block's barrier then.
__device__ __forceinline__ void pair_commit_here(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void complete_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void store_peer_word(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void arrive_at(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

__device__ __forceinline__ void load_sums32(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

struct PairMaps {
  CUtensorMap p, q, sp, sq;
};

template <int FMT>
__global__ void __launch_bounds__(kPairThreads, 1) k_mx_matmul_pair(const __grid_constant__ PairMaps maps, const Args a) {
  using S = PairShape<FMT>;
  constexpr int BN = kPairCols;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kDepth * S::kStage);
  uint64_t *empty = full + S::kDepth, *sums_full = empty + S::kDepth, *sums_empty = sums_full + 1;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(sums_empty + 1);
  uint64_t* drained = reinterpret_cast<uint64_t*>(tmem_at + 2);
  // a wait gave up, in either block; stages brought by this block, and those whose places were
  // waited for; stages and tiles whose instructions the first block issued
  volatile uint32_t *failed = tmem_at + 1, *brought = tmem_at + 4, *waited = tmem_at + 5, *issued = tmem_at + 6, *summed = tmem_at + 7;

  const uint32_t warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32, rank = blockIdx.x & 1;
  const uint32_t pairs = gridDim.x / 2, pair = blockIdx.x / 2, polls = polls_of(a);
  const uint32_t tiles = (a.p_rows + 255) / 256 * a.q_tiles;

  // Stage i of a tile into place `at` of the ring: this block's share, whose bytes count at the
  // first block's barrier with the other's.
  const auto bring = [&](uint32_t t, uint32_t i, uint32_t at) {
    const uint32_t p0 = t / a.q_tiles * 256 + rank * 128, q0 = t % a.q_tiles * BN;
    if (rank == 0) mbar_expect_tx(full + at, 2 * S::kBytes);
    const uint32_t st = smem_addr(smem) + at * S::kStage, bar = peer(smem_addr(full + at), 0);
    tma_pair_2d(st, &maps.p, (int32_t)(i * kStageBytesK), (int32_t)p0, bar);
    tma_pair_2d(st + S::kP, &maps.q, (int32_t)(i * kStageBytesK), (int32_t)(q0 + rank * (BN / 2)), bar);
    tma_pair_3d(st + S::kP + S::kQ, &maps.sp, 0, (int32_t)(i * S::kTiles), (int32_t)(p0 / 128), bar);
    tma_pair_3d(st + S::kP + S::kQ + S::kSp, &maps.sq, 0, (int32_t)(i * S::kTiles), (int32_t)(q0 / 128), bar);
  };
  if (warp == 8) {
    if (elect()) {
      prefetch_map(&maps.p);
      prefetch_map(&maps.q);
      prefetch_map(&maps.sp);
      prefetch_map(&maps.sq);
      for (uint32_t i = 0; i < S::kDepth; i++) {
        mbar_init(full + i, 1);
        mbar_init(empty + i, 1);
      }
      mbar_init(sums_full, 1);
      mbar_init(sums_empty, 16);  // eight warps of two blocks
      mbar_init(drained, 1);
      *failed = *issued = *summed = 0;
    }
    __syncwarp();
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_at)), "r"(512u) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  cluster_sync();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = uniform(*reinterpret_cast<volatile uint32_t*>(tmem_at));

  const auto give_up = [&]() {
    *failed = 1;
    store_peer_word(peer(smem_addr(const_cast<uint32_t*>(failed)), rank ^ 1), 1);
  };
  if (warp == 8) {
    const bool one = elect();
    Ring r;
    uint32_t n = 0;  // stages brought so far
    bool ok = true;
    for (uint32_t t = pair; ok && t < tiles; t += pairs) {
      for (uint32_t i = 0; i < a.stages; i++, n++, r.next(S::kDepth)) {
        ok = n < S::kDepth || warp_wait(empty + r.at, r.parity ^ 1, polls);
        if (!ok) break;
        if (one) bring(t, i, r.at);
        __syncwarp();
      }
    }
    *brought = n;
    // the last arrivals at this block's barriers, which the other block's thread sends
    for (uint32_t k = 0; ok && k < S::kDepth; k++) {
      ok = n < S::kDepth || warp_wait(empty + r.at, r.parity ^ 1, polls);
      if (ok) n++, r.next(S::kDepth);
    }
    *waited = n;
    if (!ok) give_up();
  } else if (warp == 9 && rank == 0) {
    const bool one = elect();
    Ring r;
    bool ok = true;
    uint32_t n = 0, turns = 0;  // stages and tiles whose instructions were issued
    for (uint32_t t = pair; t < tiles; t += pairs, turns++) {
      ok = t == pair || warp_wait(sums_empty, (turns & 1) ^ 1, polls);
      if (!ok) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      uint32_t left = a.mmas;
      for (uint32_t i = 0; i < a.stages; i++, n++, r.next(S::kDepth), left -= kStageK / kMmaK) {
        ok = warp_wait(full + r.at, r.parity, polls);
        if (!ok) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t st = smem_addr(smem) + r.at * S::kStage, sc = st + S::kP + S::kQ;
        const uint32_t tp = tmem + BN + r.at * S::kScaleCols, tq = tp + 4 * S::kTiles;
        if (one) {
#pragma unroll
          for (uint32_t j = 0; j < S::kTiles; j++) {
            pair_copy_scales(tp + 4 * j, sc + j * kMxTileBytes);
#pragma unroll
            for (uint32_t h = 0; h < S::kHalves; h++)
              pair_copy_scales(tq + 4 * (j * S::kHalves + h), sc + S::kSp + h * S::kSp + j * kMxTileBytes);
          }
#pragma unroll
          for (uint32_t k = 0; k < kStageK / kMmaK; k++) {
            if (k >= left) break;
            const uint32_t j = FMT == kMxFp4 ? k / 2 : k, id = FMT == kMxFp4 ? k % 2 * 2 : 0;
            // 256 rows: twice the 128 of one block
            pair_mma<FMT>(tmem, desc_codes(st + k * 32), desc_codes(st + S::kP + k * 32), instr<FMT, BN>(id) + (1u << 27), tp + 4 * j,
                          tq + 4 * j * S::kHalves, i + k > 0);
          }
          pair_commit(empty + r.at);
        }
        __syncwarp();
      }
      if (!ok) break;  // no block hears of sums that are not whole
      if (one) pair_commit(sums_full);
      __syncwarp();
    }
    *issued = n, *summed = turns;
    if (!ok) give_up();
  } else if (warp < 8) {
    const Scale g = scale_of<FMT>(a);
    const uint32_t quarter = warp % 4, half = warp / 4, leader_bar = peer(smem_addr(sums_empty), 0);
    constexpr int kCols = BN / 2;  // of one warp
    uint32_t k_tile = 0;
    for (uint32_t t = pair; t < tiles; t += pairs, k_tile++) {
      const uint32_t p = t / a.q_tiles * 256 + rank * 128 + quarter * 32 + lane, q = t % a.q_tiles * BN + half * kCols;
      if (!warp_wait(sums_full, k_tile & 1, polls)) {
        give_up();
        break;
      }
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      float v[kCols];
#pragma unroll
      for (int c = 0; c < kCols; c += 32) load_sums32(tmem + (quarter * 32 << 16) + half * kCols + c, v + c);
      asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) arrive_at(leader_bar);
      store<FMT, kCols>(a, p, q, v, g);
    }
    __syncwarp();
  }
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  cluster_sync();  // neither block's barriers and tensor memory go while the other still uses them
  if (*failed) {  // the same in both blocks by now
    if (threadIdx.x == 0) atomicMax(&g_mx_status, kStTimeout);
    if (warp == 8 || warp == 0) {
      // the arrivals that are still to come for instructions issued: one a stage at `empty`, one
      // a tile at sums_full
      const uint32_t stages = load_peer_word(peer(smem_addr(const_cast<uint32_t*>(issued)), 0));
      const uint32_t sums = load_peer_word(peer(smem_addr(const_cast<uint32_t*>(summed)), 0));
      if (warp == 0) {
        if (sums) mbar_wait_bounded(sums_full, (sums - 1) & 1, kWaitPolls);
      } else {
        // the first kDepth places held no stage yet
        for (uint32_t s = *waited < S::kDepth ? 0 : *waited - S::kDepth; s < stages; s++)
          mbar_wait_bounded(empty + s % S::kDepth, s / S::kDepth & 1, kWaitPolls);
      }
    } else if (warp == 9 && rank == 0) {
      if (elect()) pair_commit_here(drained);
      __syncwarp();
      mbar_wait_bounded(drained, 0, kWaitPolls);
      // the stages brought and not used, at most one in each place. Where only one block has
      // brought its half, the other's bytes, which will not come, are taken off the count.
      const uint32_t first = *brought, second = load_peer_word(peer(smem_addr(const_cast<uint32_t*>(brought)), 1));
      for (uint32_t s = *issued; s < max(first, second); s++) {
        uint64_t* bar = full + s % S::kDepth;
        if (elect()) {
          if (s >= first) mbar_expect_tx(bar, S::kBytes);
          else if (s >= second) complete_tx(bar, S::kBytes);
        }
        __syncwarp();
        mbar_wait_bounded(bar, s / S::kDepth & 1, kWaitPolls);
      }
    }
    __syncthreads();
    cluster_sync();
  }
  if (warp == 9) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
  }
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static std::atomic<void*> cached{nullptr};
  void* f = cached.load(std::memory_order_acquire);
  if (!f) {
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    cached.store(f, std::memory_order_release);
  }
  return reinterpret_cast<EncodeTiled>(f);
}

// Codes as rows of bytes, a box of 128 bytes x `box` rows; zeros outside.
bool code_map(CUtensorMap* m, const void* codes, uint64_t rows, uint64_t row_bytes, uint32_t box) {
  EncodeTiled f = encode_tiled();
  const cuuint64_t dims[2] = {row_bytes, rows}, strides[1] = {row_bytes};
  const cuuint32_t boxes[2] = {kStageBytesK, box}, steps[2] = {1, 1};
  return f && f(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(codes), dims, strides, boxes, steps,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t device_sms(int& dev, int& sms) {
  const cudaError_t e = cudaGetDevice(&dev);
  return e == cudaSuccess ? cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) : e;
}

struct Operand {
  const void* codes;
  const uint8_t* scales;
  uint64_t rows;
};

template <int FMT, int BN>
cudaError_t launch_tiles(const Operand& p, const Operand& q, uint64_t cols, Args a, cudaStream_t st) {
  using S = Shape<FMT, BN>;
  static std::atomic<uint64_t> ready{0};  // devices whose shared-memory limit is set
  int dev = 0, sms = 0;
  cudaError_t e = device_sms(dev, sms);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(k_mx_matmul<FMT, BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kAllShared);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  CUtensorMap pm, qm;
  const uint64_t rb = mx_row_bytes(cols);
  if (!code_map(&pm, p.codes, p.rows, rb, 128) || !code_map(&qm, q.codes, q.rows, rb, BN)) return cudaErrorUnknown;
  const uint64_t q_tiles = mx_div_up(q.rows, BN), tiles = mx_div_up(p.rows, 128) * q_tiles;
  a.q_tiles = (uint32_t)q_tiles;
  // As many blocks to a tile as leave each an SM of its own (16 x 4096 x 4096, 32 tiles: 6.3 us
  // unsplit, 5.4 by 4, 6.7 by 8; 64 x 11008 x 4096, 86 tiles: 8.5 unsplit, 10.0 by 2).
  a.split = 1;
  while (a.split < 8 && tiles * a.split * 2 <= (uint64_t)sms && a.split * 2 <= a.stages) a.split *= 2;
  a.depth = tiles * a.split <= (uint64_t)sms ? S::kAlone : S::kShared;
  a.tmem_cols = S::cols(a.depth);
  if (tiles * a.split > 0x7FFFFFFFull) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((uint32_t)(tiles * a.split));
  cfg.blockDim = dim3(kThreads);
  // Blocks that wait for each other have their SMs to themselves: beside another library's, which
  // may wait for its neighbours as well, two clusters could hold the tensor memory that the
  // other needs. It takes no time, since each block has an SM anyway.
  cfg.dynamicSmemBytes = a.split > 1 ? kAllShared : S::smem(a.depth);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = a.split;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = a.split > 1;
  TimedLaunch t(kIdMxMatmul, st);
  return cudaLaunchKernelEx(&cfg, k_mx_matmul<FMT, BN>, pm, qm, a);
}

// Scale tiles as (row tiles, tiles along a row, 128 words of 4 bytes); zeros outside.
bool scale_map(CUtensorMap* m, const uint8_t* scales, uint64_t row_tiles, uint64_t col_tiles, uint32_t box_tiles, uint32_t box_rows) {
  EncodeTiled f = encode_tiled();
  const cuuint64_t dims[3] = {kMxTileBytes / 4, col_tiles, row_tiles}, strides[2] = {kMxTileBytes, kMxTileBytes * col_tiles};
  const cuuint32_t boxes[3] = {kMxTileBytes / 4, box_tiles, box_rows}, steps[3] = {1, 1, 1};
  return f && f(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<uint8_t*>(scales), dims, strides, boxes, steps,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int FMT>
cudaError_t launch_pairs(const Operand& p, const Operand& q, uint64_t cols, Args a, cudaStream_t st) {
  using S = PairShape<FMT>;
  constexpr int BN = kPairCols;
  static std::atomic<uint64_t> ready{0};
  int dev = 0, sms = 0;
  cudaError_t e = device_sms(dev, sms);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(k_mx_matmul_pair<FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kAllShared);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  PairMaps maps;
  const uint64_t rb = mx_row_bytes(cols);
  if (!code_map(&maps.p, p.codes, p.rows, rb, 128) || !code_map(&maps.q, q.codes, q.rows, rb, BN / 2) ||
      !scale_map(&maps.sp, p.scales, mx_div_up(p.rows, 128), a.col_tiles, S::kTiles, 1) ||
      !scale_map(&maps.sq, q.scales, mx_div_up(q.rows, 128), a.col_tiles, S::kTiles, S::kHalves))
    return cudaErrorUnknown;
  a.q_tiles = (uint32_t)mx_div_up(q.rows, BN);
  const uint64_t tiles = mx_div_up(p.rows, 256) * a.q_tiles, most = (uint64_t)sms / 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((uint32_t)(2 * (tiles < most ? tiles : most)));
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = kAllShared;  // no other block beside these either
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  TimedLaunch t(kIdMxMatmul, st);
  return cudaLaunchKernelEx(&cfg, k_mx_matmul_pair<FMT>, maps, a);
}

template <int FMT>
cudaError_t launch_matmul(bool pairs, const Operand& p, const Operand& q, uint64_t cols, const Args& a, cudaStream_t st) {
  if (pairs) return launch_pairs<FMT>(p, q, cols, a, st);
  // Blocks as wide as the shorter operand's rows: what a wider one adds is read, though it is
  // zeros, and takes room from stages in flight (1 x 32000 x 4096: 13.9 us with 16, 14.8 with
  // 32, 15.9 with 64, 21.0 with 128; 64 x 32000 x 4096: 15.2 with 64, 16.5 with 128).
  if (q.rows <= 16) return launch_tiles<FMT, 16>(p, q, cols, a, st);
  if (q.rows <= 32) return launch_tiles<FMT, 32>(p, q, cols, a, st);
  if (q.rows <= 64) return launch_tiles<FMT, 64>(p, q, cols, a, st);
  return launch_tiles<FMT, 128>(p, q, cols, a, st);
}

inline bool off16(const void* p) { return !p || (reinterpret_cast<uintptr_t>(p) & 15) != 0; }

}  // namespace
}  // namespace zipnn

using namespace zipnn;

extern "C" {

zipnn_status zipnn_mx_matmul(zipnn_mx_format format, const void* a_codes, const void* a_scales, const float* a_global,
                             const void* b_codes, const void* b_scales, const float* b_global, uint64_t m, uint64_t n,
                             uint64_t k, zipnn_value_type type, void* out, uint64_t row_stride, zipnn_stream_t stream) {
  if (!mx_valid(format, m, k) || !mx_valid(format, n, k) || !mx_valid_type(type)) return ZIPNN_ERR_INVALID_ARG;
  if (off16(a_codes) || off16(a_scales) || off16(b_codes) || off16(b_scales) || !out) return ZIPNN_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(out) % mx_value_bytes(type) || row_stride < n || row_stride > kMxMaxStride) return ZIPNN_ERR_INVALID_ARG;
  if (format == ZIPNN_NVFP4 && (!a_global || !b_global || reinterpret_cast<uintptr_t>(a_global) % 4 || reinterpret_cast<uintptr_t>(b_global) % 4))
    return ZIPNN_ERR_INVALID_ARG;
  if (mx_div_up(m, 128) * mx_div_up(n, 128) > 0x7FFFFFFFull) return ZIPNN_ERR_INVALID_ARG;
  if (!device_ok()) return ZIPNN_ERR_UNSUPPORTED;
  // Large products go to pairs of blocks (MXFP4, by pairs and by single blocks: 1024 x 4096 x 4096,
  // 64 tiles, 10.8 and 11.8 us; 640 x 4096 x 4096, 48 tiles, 10.4 and 11.0; 512 x 4096 x 4096, 32
  // tiles, 10.4 and 8.5; 512 x 11008 x 4096, 86 tiles, 16.5 and 17.1). Padding is not looked at:
  // 300 x 11008 x 4096, where nearly half of each tile is padding, takes 16.9 us, and would take
  // 11.6. B's rows lie along the 128 rows of a
  // block, whose lanes then hold neighbours of the output (4096 x 256 x 4096: 9 us, 19 with A's),
  // unless they are few and A's are more.
  const bool pairs = m > 128 && n > 128 && mx_div_up(m, 256) * mx_div_up(n, 256) >= 40;
  const bool p_is_n = n >= 128 || n >= m;
  const Operand a{a_codes, static_cast<const uint8_t*>(a_scales), m}, b{b_codes, static_cast<const uint8_t*>(b_scales), n};
  const Operand &p = p_is_n ? b : a, &q = p_is_n ? a : b;
  Args g = {};
  g.p_scales = p.scales;
  g.q_scales = q.scales;
  g.ga = a_global;
  g.gb = b_global;
  g.out = static_cast<uint8_t*>(out);
  g.ldo = row_stride;
  g.p_rows = (uint32_t)p.rows;
  g.q_rows = (uint32_t)q.rows;
  g.col_tiles = (uint32_t)mx_col_tiles(format, k);
  g.stages = (uint32_t)mx_div_up(k, kStageK);
  g.mmas = (uint32_t)mx_div_up(k, kMmaK);
  g.type = type;
  g.p_is_n = p_is_n;
  const uint32_t limit = g_wait_limit.load(std::memory_order_relaxed);
  g.polls = limit >> 6, g.mask = limit >> 3 & 7, g.value = limit & 7;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = format == ZIPNN_MXFP4 ? launch_matmul<kMxFp4>(pairs, p, q, k, g, st) : launch_matmul<kNvFp4>(pairs, p, q, k, g, st);
  return e == cudaSuccess ? ZIPNN_OK : ZIPNN_ERR_CUDA;
}

zipnn_status zipnn_test_mx_wait_limit(uint32_t polls, uint32_t mask, uint32_t value) {
  if (mask > 7 || value > 7) return ZIPNN_ERR_INVALID_ARG;
  g_wait_limit.store(std::min(polls, kWaitPolls) << 6 | mask << 3 | value, std::memory_order_relaxed);
  return ZIPNN_OK;
}

zipnn_status zipnn_mx_status(zipnn_stream_t stream) {
  if (!device_ok()) return ZIPNN_ERR_UNSUPPORTED;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint32_t v = 0;
  const uint32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_mx_status, 4, 0, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && v) e = cudaMemcpyToSymbolAsync(g_mx_status, &zero, 4, 0, cudaMemcpyHostToDevice, st);
  return e == cudaSuccess ? (zipnn_status)v : ZIPNN_ERR_CUDA;
}

}  // extern "C"
