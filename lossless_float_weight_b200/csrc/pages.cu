// pages.cu -- the pages of a K/V cache (include/zipnn.h): copying them by lists of page
// numbers, and the references, lengths and tables of the sequences that hold them: forks,
// frees and the closing of gaps.
//
// The data is moved once (read and written, nothing else), so HBM bounds the large calls; the
// small ones are bound by launches, and take one or two: a single block decides what the
// call does, and a grid that starts beside it (programmatic dependent launch) does it.
// Measured (32 KB pages, 64 planes): 640 pages scattered 390 us (6.9 TB/s), 174 pages closed up
// 122 us (6.0 TB/s), 5 pages gathered 4.4 us, a fork of one sequence 6.3 us, a free 2.5 us.
#include <algorithm>

#include "zipnn.h"
#include "common.cuh"
#include "op_ids.h"

namespace zipnn {
namespace {

constexpr uint32_t kStInvalid = 1, kStTooSmall = 2;
constexpr int kPlanThreads = 1024, kCopyThreads = 256;
constexpr uint32_t kWindow = 1u << 18;  // page or row numbers marked in shared memory at a time
constexpr uint32_t kChunkVecs = 1024;   // 16 KB of one page are one unit of the copy

// The first words of a workspace. `status` stays until the caller clears it; the others are
// written by every call that uses them.
struct Head {
  uint32_t status, live, pairs, refused;
  unsigned long long next;  // units of the copy that blocks have taken
};

struct Request {
  int32_t row, parent;        // parent == row: the row grows
  uint32_t first, total;      // slots below first are the parent's pages, from there on fresh ones
  uint32_t offset, len;       // into the list of fresh pages; the row's new length
};

struct Pool {
  uint8_t* base;
  uint64_t plane_stride, page_stride;
  uint32_t pages;
};

struct Meta {
  int32_t *refs, *lens, *tables;
  uint32_t seqs, slots, pages, page_tokens;
};

__device__ __forceinline__ void set_status(Head* h, uint32_t v) { atomicCAS(&h->status, 0u, v); }

__device__ __forceinline__ void wait_for_plan() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_dependents_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Copies `count` pages, pair i from src page src_ids[i] to dst page dst_ids[i] (i itself
// without a list; a negative number skips the pair), in every plane. A unit is 16 KB of one
// page of one plane; short pages share a block, a power of two of threads for each. Each
// thread holds up to four 16-byte vectors between its loads and its stores.
struct Units {
  uint32_t chunks, tpu, per_block, lane;  // units of a page and plane; threads of a unit; units of a block; this thread in its unit
  uint64_t all;
  __device__ __forceinline__ Units(uint32_t count, uint32_t planes, uint32_t page_vecs) {
    chunks = (page_vecs + kChunkVecs - 1) / kChunkVecs;
    tpu = 1;
    while (tpu < page_vecs && tpu < kCopyThreads) tpu <<= 1;
    per_block = kCopyThreads / tpu;
    lane = threadIdx.x & (tpu - 1);
    all = (uint64_t)planes * count * chunks;
  }
};

// The units of this block, `first` being the number of its first one.
__device__ __forceinline__ void copy_unit(const Units& n, uint64_t first, const Pool& src, const int32_t* src_ids, const Pool& dst,
                                          const int32_t* dst_ids, uint32_t count, uint32_t page_vecs, Head* head) {
  const uint64_t u = first + threadIdx.x / n.tpu;
  if (u >= n.all) return;
  const uint64_t q = u / n.chunks;
  const uint32_t chunk = (uint32_t)(u - q * n.chunks);
  const uint32_t plane = (uint32_t)(q / count), i = (uint32_t)(q - (uint64_t)plane * count);
  const int64_t s = src_ids ? src_ids[i] : (int64_t)i, d = dst_ids ? dst_ids[i] : (int64_t)i;
  if (s < 0 || d < 0) return;
  if (s >= src.pages || d >= dst.pages) {
    set_status(head, kStInvalid);
    return;
  }
  const uint4* from = reinterpret_cast<const uint4*>(src.base + plane * src.plane_stride + s * src.page_stride);
  uint4* to = reinterpret_cast<uint4*>(dst.base + plane * dst.plane_stride + d * dst.page_stride);
  const uint32_t lo = chunk * kChunkVecs + n.lane, hi = min(page_vecs, (chunk + 1) * kChunkVecs);
  uint4 v[kChunkVecs / kCopyThreads];
#pragma unroll
  for (int k = 0; k < (int)(kChunkVecs / kCopyThreads); k++)
    if (lo + k * n.tpu < hi) v[k] = from[lo + k * n.tpu];
#pragma unroll
  for (int k = 0; k < (int)(kChunkVecs / kCopyThreads); k++)
    if (lo + k * n.tpu < hi) to[lo + k * n.tpu] = v[k];
}

// Within one pool, where the number of pairs was found on the device: a block begins at its own
// place and then takes the next units as it gets done, in the order of memory (head->next
// starts at 0), several at a time where there are many: taking one costs a few nanoseconds in
// which no other block can (17 pages of 1 MB copied beside a fork: 12.6 us, 13.4 with every unit
// taken one by one, the first included).
__device__ __forceinline__ void copy_pairs(const Pool& pool, const int32_t* src_ids, const int32_t* dst_ids, uint32_t count,
                                           uint32_t planes, uint32_t page_vecs, Head* head) {
  __shared__ unsigned long long taken[2];
  const Units n(count, planes, page_vecs);
  const uint64_t at_once = min((uint64_t)8, max((uint64_t)1, n.all / ((uint64_t)gridDim.x * n.per_block * 8)));
  const uint64_t step = at_once * n.per_block, given = gridDim.x * step;
  uint64_t u = blockIdx.x * step;
  for (uint32_t turn = 0; u < n.all; turn ^= 1) {
    if (threadIdx.x == 0) taken[turn] = given < n.all ? given + atomicAdd(&head->next, (unsigned long long)step) : n.all;
    for (uint64_t k = 0; k < at_once; k++) copy_unit(n, u + k * n.per_block, pool, src_ids, pool, dst_ids, count, page_vecs, head);
    __syncthreads();
    u = taken[turn];
  }
}

__global__ void __launch_bounds__(kCopyThreads) k_pages_copy(Pool src, const int32_t* src_ids, Pool dst, const int32_t* dst_ids,
                                                             uint32_t count, uint32_t planes, uint32_t page_vecs, Head* head,
                                                             bool checked) {
  if (checked) {
    wait_for_plan();
    if (*reinterpret_cast<volatile uint32_t*>(&head->refused)) return;
  }
  const Units n(count, planes, page_vecs);
  for (uint64_t u = (uint64_t)blockIdx.x * n.per_block; u < n.all; u += (uint64_t)gridDim.x * n.per_block)
    copy_unit(n, u, src, src_ids, dst, dst_ids, count, page_vecs, head);
}

// Before a copy that could write a page twice, or one that it also reads: every number in its
// range, no destination twice and, within one pool (`same`), no destination among the sources.
__global__ void __launch_bounds__(kPlanThreads) k_pages_check(const int32_t* src_ids, uint32_t src_pages, const int32_t* dst_ids,
                                                              uint32_t dst_pages, uint32_t count, bool same, Head* head) {
  __shared__ uint32_t bits[kWindow / 32];
  let_dependents_start();
  int bad = 0;
  for (uint64_t base = 0; base < dst_pages; base += kWindow) {
    const uint32_t words = (uint32_t)min((uint64_t)kWindow / 32, (dst_pages - base + 31) / 32);
    for (uint32_t i = threadIdx.x; i < words; i += kPlanThreads) bits[i] = 0;
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < count; i += kPlanThreads) {
      const int64_t s = src_ids ? src_ids[i] : (int64_t)i, d = dst_ids ? dst_ids[i] : (int64_t)i;
      if (s < 0 || d < 0) continue;
      if (s >= src_pages || d >= dst_pages) {
        bad = 1;
      } else if ((uint64_t)d >= base && (uint64_t)d < base + kWindow) {
        const uint32_t m = 1u << (d & 31);
        bad |= (atomicOr(&bits[(d - base) >> 5], m) & m) != 0;
      }
    }
    __syncthreads();
    if (same) {
      for (uint32_t i = threadIdx.x; i < count; i += kPlanThreads) {
        const int64_t s = src_ids ? src_ids[i] : (int64_t)i, d = dst_ids ? dst_ids[i] : (int64_t)i;
        if (s < 0 || d < 0 || (uint64_t)s < base || (uint64_t)s >= base + words * 32ull) continue;
        bad |= (bits[(s - base) >> 5] >> (s & 31)) & 1;
      }
    }
    __syncthreads();
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) {
    head->refused = bad ? 1 : 0;
    if (bad) set_status(head, kStInvalid);
  }
}

// Sum over the warps before this one of `v`, summed over the block into `total`.
__device__ __forceinline__ uint32_t warps_before(uint32_t v, uint32_t* smem, uint32_t& total) {
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  __syncthreads();
  if (lane == 0) smem[warp] = v;
  __syncthreads();
  const uint32_t mine = smem[lane];
  total = __reduce_add_sync(0xFFFFFFFFu, mine);
  return __reduce_add_sync(0xFFFFFFFFu, lane < warp ? mine : 0);
}

__device__ __forceinline__ uint32_t lane_scan(uint32_t v) {  // exclusive
  const uint32_t lane = threadIdx.x % 32;
  uint32_t s = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t t = __shfl_up_sync(0xFFFFFFFFu, s, d);
    if (lane >= d) s += t;
  }
  return s - v;
}

// One block: what a fork does. Requests are checked, the fresh pages that each needs counted
// and the lowest free pages listed, in the requests' order; nothing is changed here.
__global__ void __launch_bounds__(kPlanThreads) k_pages_plan_fork(Meta m, const int32_t* rows, const int32_t* parents,
                                                                  const int32_t* new_lens, uint32_t n, Head* head,
                                                                  Request* req, int32_t* fresh, int32_t* pair_src,
                                                                  int32_t* pair_dst) {
  __shared__ uint32_t bits[kWindow / 32];
  __shared__ uint32_t smem[32];
  let_dependents_start();
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const uint64_t room = (uint64_t)m.slots * m.page_tokens;
  for (uint32_t i = threadIdx.x; i < (m.seqs + 31) / 32; i += kPlanThreads) bits[i] = 0;
  __syncthreads();
  int bad = 0;
  uint32_t need = 0, pairs = 0;
  for (uint32_t j0 = 0; j0 < n; j0 += kPlanThreads) {
    const uint32_t j = j0 + threadIdx.x;
    Request r = {0, -1, 0, 0, 0, 0};
    uint32_t part = 0;
    if (j < n) {
      const int32_t row = rows[j], parent = parents[j], len = new_lens[j];
      if (row < 0 || (uint32_t)row >= m.seqs || parent < -1 || parent >= (int32_t)m.seqs || len < 0 || (uint64_t)len > room) {
        bad = 1;
      } else {
        const uint32_t bit = 1u << (row & 31);
        if (atomicOr(&bits[row >> 5], bit) & bit) bad = 1;
        const int32_t old = m.lens[row], have = parent < 0 ? 0 : m.lens[parent];
        if (have < 0 || (uint64_t)have > room || (parent == row ? len < old : old != 0)) {
          bad = 1;  // nothing is derived from such a request
        } else {
          const uint32_t upto = (uint32_t)min(have, len), pt = m.page_tokens;
          r.row = row, r.parent = parent, r.len = (uint32_t)len;
          r.total = ((uint32_t)len + pt - 1) / pt;
          r.first = parent == row ? ((uint32_t)have + pt - 1) / pt : upto / pt;
          part = parent != row && upto % pt != 0;
        }
      }
    }
    // places in the list of fresh pages, and in the list of pages to copy, in request order
    const uint32_t want = r.total - r.first;
    const uint32_t lw = lane_scan(want), lp = lane_scan(part);
    uint32_t all_w, all_p;
    const uint32_t ww = __shfl_sync(0xFFFFFFFFu, lw + want, 31), wp = __shfl_sync(0xFFFFFFFFu, lp + part, 31);
    const uint32_t before_w = warps_before(ww, smem, all_w), before_p = warps_before(wp, smem, all_p);
    r.offset = need + before_w + lw;
    if (j < n) req[j] = r;
    if (part) {
      const uint32_t at = pairs + before_p + lp;
      const int32_t id = m.tables[(uint64_t)r.parent * m.slots + r.first];
      const bool in = id >= 0 && (uint32_t)id < m.pages;
      pair_src[at] = in ? id : -1;
      if (!in) set_status(head, kStCorrupt);
      pair_dst[at] = (int32_t)r.offset;  // its place among the fresh pages, until they are listed
    }
    need += all_w;
    pairs += all_p;
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) {
      head->refused = 1;
      set_status(head, kStInvalid);
    }
    return;
  }
  // the lowest `need` pages without references: each warp counts those of its own range (at
  // most 4096 pages, so that a pool with room at its front is not read to its end), then
  // lists them behind those of the ranges before it
  const uint64_t each = min((uint64_t)4096, ((uint64_t)m.pages + 32 * 32 - 1) / (32 * 32) * 32);
  uint32_t found = 0;
  for (uint64_t base = 0; base < m.pages && found < need; base += 32 * each) {
    const uint64_t lo = base + warp * each, hi = min(lo + each, (uint64_t)m.pages);
    uint32_t mine = 0;
#pragma unroll 8
    for (uint64_t p = lo; p < hi; p += 32) mine += __popc(__ballot_sync(0xFFFFFFFFu, p + lane < hi && m.refs[p + lane] == 0));
    uint32_t all;
    uint32_t at = found + warps_before(mine, smem, all);
    for (uint64_t p = lo; p < hi && at < need; p += 32) {
      const bool is = p + lane < hi && m.refs[p + lane] == 0;
      const uint32_t b = __ballot_sync(0xFFFFFFFFu, is);
      const uint32_t k = at + __popc(b & ((1u << lane) - 1));
      if (is && k < need) fresh[k] = (int32_t)(p + lane);
      at += __popc(b);
    }
    found += all;
  }
  __syncthreads();
  if (found < need) {
    if (threadIdx.x == 0) {
      head->refused = 1;
      set_status(head, kStTooSmall);
    }
    return;
  }
  for (uint32_t i = threadIdx.x; i < pairs; i += kPlanThreads) pair_dst[i] = fresh[pair_dst[i]];
  if (threadIdx.x == 0) {
    head->refused = 0;
    head->pairs = pairs;
    head->next = 0;
  }
}

// The planned fork: tables, references and lengths, a block to a request, and the copies of
// the pages that a fork ends inside of.
__global__ void __launch_bounds__(kCopyThreads) k_pages_fork(Meta m, Pool pool, uint32_t planes, uint32_t page_vecs, uint32_t n,
                                                             Head* head, const Request* req, const int32_t* fresh,
                                                             const int32_t* pair_src, const int32_t* pair_dst) {
  wait_for_plan();
  if (*reinterpret_cast<volatile uint32_t*>(&head->refused)) return;
  for (uint32_t j = blockIdx.x; j < n; j += gridDim.x) {
    const Request r = req[j];
    int32_t* out = m.tables + (uint64_t)r.row * m.slots;
    for (uint32_t s = threadIdx.x; s < r.total; s += kCopyThreads) {
      if (s >= r.first) {
        const int32_t id = fresh[r.offset + s - r.first];
        out[s] = id;
        m.refs[id] = 1;
      } else if (r.parent != r.row) {
        const int32_t id = m.tables[(uint64_t)r.parent * m.slots + s];
        out[s] = id;
        if (id >= 0 && (uint32_t)id < m.pages) atomicAdd(&m.refs[id], 1);
        else set_status(head, kStCorrupt);
      }
    }
    if (threadIdx.x == 0) m.lens[r.row] = (int32_t)r.len;
  }
  copy_pairs(pool, pair_src, pair_dst, *reinterpret_cast<volatile uint32_t*>(&head->pairs), planes, page_vecs, head);
}

// A block to a row: its pages lose a reference each, its slots and its length are cleared. The
// length is taken by exchange, so that a row named twice is freed once.
__global__ void __launch_bounds__(kCopyThreads) k_pages_free(Meta m, const int32_t* rows, uint32_t n, Head* head) {
  __shared__ int32_t len;
  for (uint32_t j = blockIdx.x; j < n; j += gridDim.x) {
    const int32_t row = rows[j];
    if (row < 0 || (uint32_t)row >= m.seqs) {
      if (threadIdx.x == 0) set_status(head, kStInvalid);
      continue;
    }
    __syncthreads();
    if (threadIdx.x == 0) len = atomicExch(&m.lens[row], 0);
    __syncthreads();
    const uint64_t want = len > 0 ? ((uint64_t)len + m.page_tokens - 1) / m.page_tokens : 0;
    if (len < 0 || want > m.slots) {
      if (threadIdx.x == 0) set_status(head, kStCorrupt);
    }
    int32_t* t = m.tables + (uint64_t)row * m.slots;
    for (uint32_t s = threadIdx.x; s < min(want, (uint64_t)m.slots); s += kCopyThreads) {
      const int32_t id = t[s];
      t[s] = -1;
      if (id < 0 || (uint32_t)id >= m.pages) {
        set_status(head, kStCorrupt);
      } else if (atomicSub(&m.refs[id], 1) <= 0) {  // it had none
        atomicAdd(&m.refs[id], 1);
        set_status(head, kStCorrupt);
      }
    }
  }
}

// One block: the pages in use, counted (`live`); those numbered at or past that count, in
// order, move into the free numbers below it, in order. to[p]: where page p >= live goes, -1
// for a page not in use. Each warp takes one range of the pages.
__global__ void __launch_bounds__(kPlanThreads) k_pages_plan_compact(Meta m, Head* head, int32_t* to, int32_t* pair_src,
                                                                     int32_t* pair_dst) {
  __shared__ uint32_t smem[32];
  let_dependents_start();
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const uint64_t each = ((uint64_t)m.pages + 32 * 32 - 1) / (32 * 32) * 32;
  const uint64_t lo = min(warp * each, (uint64_t)m.pages), hi = min(lo + each, (uint64_t)m.pages);
  uint32_t mine = 0;
#pragma unroll 8
  for (uint64_t p = lo; p < hi; p += 32) mine += __popc(__ballot_sync(0xFFFFFFFFu, p + lane < hi && m.refs[p + lane] > 0));
  uint32_t live, below;
  uint32_t used_before = warps_before(mine, smem, live);
  uint32_t kept = 0;  // in use below `live`: they stay
  for (uint64_t p = lo; p < hi && p < live; p += 32)
    kept += __popc(__ballot_sync(0xFFFFFFFFu, p + lane < hi && p + lane < live && m.refs[p + lane] > 0));
  warps_before(kept, smem, below);
  for (uint64_t p = lo; p < hi; p += 32) {
    const uint64_t id = p + lane;
    const bool used = id < hi && m.refs[id] > 0;
    const uint32_t b = __ballot_sync(0xFFFFFFFFu, used);
    const uint32_t u = used_before + __popc(b & ((1u << lane) - 1));  // pages in use before this one
    if (id < hi) {
      if (id >= live) {
        if (used) pair_src[u - below] = (int32_t)id;
        else to[id] = -1;
      } else if (!used) {
        pair_dst[id - u] = (int32_t)id;
      }
    }
    used_before += __popc(b);
  }
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < live - below; i += kPlanThreads) to[pair_src[i]] = pair_dst[i];
  if (threadIdx.x == 0) {
    head->live = live;
    head->pairs = live - below;
    head->next = 0;
  }
}

// The planned moves: the tables' numbers, the references, and the pages.
__global__ void __launch_bounds__(kCopyThreads) k_pages_compact(Meta m, Pool pool, uint32_t planes, uint32_t page_vecs, Head* head,
                                                                const int32_t* to, const int32_t* pair_src, const int32_t* pair_dst) {
  wait_for_plan();
  const uint32_t pairs = *reinterpret_cast<volatile uint32_t*>(&head->pairs);
  if (pairs == 0) return;
  const int32_t live = *reinterpret_cast<volatile int32_t*>(&head->live);
  const uint64_t slots = (uint64_t)m.seqs * m.slots, step = (uint64_t)gridDim.x * kCopyThreads;
  const uint64_t first = (uint64_t)blockIdx.x * kCopyThreads + threadIdx.x;
  for (uint64_t i = first; i < slots; i += step) {
    const int32_t id = m.tables[i];
    if (id < live) continue;
    const int32_t t = (uint32_t)id < m.pages ? to[id] : -1;
    if (t >= 0) m.tables[i] = t;
    else set_status(head, kStCorrupt);
  }
  for (uint64_t i = first; i < pairs; i += step) {
    m.refs[pair_dst[i]] = m.refs[pair_src[i]];
    m.refs[pair_src[i]] = 0;
  }
  copy_pairs(pool, pair_src, pair_dst, pairs, planes, page_vecs, head);
}

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), uint32_t grid, bool dependent, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kCopyThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Blocks for the copy of at most `count` pages. A block that takes one unit and ends, the next
// starting in its place, copies faster than one that walks over many (1.34 GB in 32 KB pages,
// scattered: 390 us with a block a unit, 411 with 148 x 64 blocks, 438 with 148 x 8). Where the
// number of pages is found on the device and may be far below `count`, empty blocks would cost
// more than that: `most` blocks then take units in turn (copy_pairs).
uint32_t copy_grid(uint64_t count, uint32_t planes, uint64_t page_vecs, uint64_t most = 0x7FFFFFFF) {
  uint64_t tpu = 1;
  while (tpu < page_vecs && tpu < (uint64_t)kCopyThreads) tpu <<= 1;
  const uint64_t units = (uint64_t)planes * count * ((page_vecs + kChunkVecs - 1) / kChunkVecs);
  const uint64_t per_block = kCopyThreads / tpu, blocks = units / per_block + (units % per_block != 0);
  return (uint32_t)std::max<uint64_t>(1, std::min<uint64_t>(blocks, most));
}

inline bool bad16(const void* p) { return !p || (reinterpret_cast<uintptr_t>(p) & 15) != 0; }
inline bool bad4(const void* p) { return !p || (reinterpret_cast<uintptr_t>(p) & 3) != 0; }
inline zipnn_status cuda_status(cudaError_t e) { return e == cudaSuccess ? ZIPNN_OK : ZIPNN_ERR_CUDA; }

constexpr uint64_t kMaxStride = 1ull << 46;

// A pool whose pages lie apart: whole 16 bytes, pages within a plane and planes within the
// pool (or pages that hold all their planes) not overlapping.
bool valid_pool(const zipnn_page_pool* p, uint64_t page_bytes) {
  if (!p || bad16(p->base) || p->planes == 0 || p->pages == 0 || p->pages > 0x7FFFFFFFu) return false;
  if (page_bytes == 0 || page_bytes % 16 || page_bytes > (1ull << 32) || p->page_stride % 16 || p->plane_stride % 16) return false;
  if (p->page_stride > kMaxStride || p->plane_stride > kMaxStride) return false;
  // the whole extent within 2^47 bytes, so that no address below wraps
  if (p->page_stride && p->pages - 1 > kMaxStride / p->page_stride) return false;
  if (p->plane_stride && p->planes - 1 > kMaxStride / p->plane_stride) return false;
  const bool planes_out = p->page_stride >= page_bytes && (p->planes == 1 || p->plane_stride / p->pages >= p->page_stride);
  const bool pages_out = (p->planes == 1 || p->plane_stride >= page_bytes) && (p->pages == 1 || p->page_stride / p->planes >= p->plane_stride);
  return planes_out || pages_out;
}

uint64_t pool_end(const zipnn_page_pool* p, uint64_t page_bytes) {
  return reinterpret_cast<uintptr_t>(p->base) + (uint64_t)(p->planes - 1) * p->plane_stride + (uint64_t)(p->pages - 1) * p->page_stride + page_bytes;
}

Pool device_pool(const zipnn_page_pool* p) { return Pool{static_cast<uint8_t*>(p->base), p->plane_stride, p->page_stride, p->pages}; }

constexpr uint64_t kTakers = 148 * 4;  // 122 us for 174 pages of 2 MB; 124 with 148 x 6, 126 with 148 x 8
constexpr uint64_t kHeadBytes = 256;
uint64_t align256(uint64_t x) { return (x + 255) & ~255ull; }

bool valid_table(const zipnn_page_table* t, const zipnn_page_pool* p) {
  return t && !bad4(t->refs) && !bad4(t->lens) && !bad4(t->tables) && t->seqs >= 1 && t->seqs <= kWindow && t->slots >= 1 &&
         t->page_tokens >= 1 && (uint64_t)t->seqs * t->slots <= 0x7FFFFFFFu && t->page_tokens <= 0x7FFFFFFFu && p->pages <= 0x7FFFFFFFu;
}

Meta device_meta(const zipnn_page_table* t, const zipnn_page_pool* p) {
  return Meta{t->refs, t->lens, t->tables, t->seqs, t->slots, p->pages, t->page_tokens};
}

}  // namespace
}  // namespace zipnn

using namespace zipnn;

extern "C" {

size_t zipnn_pages_workspace_bytes(uint32_t seqs, uint32_t pages) {
  return (size_t)(kHeadBytes + align256((uint64_t)seqs * sizeof(Request)) + 3 * align256((uint64_t)pages * 4) +
                  2 * align256((uint64_t)seqs * 4));
}

zipnn_status zipnn_pages_copy(const zipnn_page_pool* src, const int32_t* src_ids, const zipnn_page_pool* dst,
                              const int32_t* dst_ids, uint32_t count, uint64_t page_bytes, void* ws, size_t ws_bytes,
                              zipnn_stream_t stream) {
  if (!valid_pool(src, page_bytes) || !valid_pool(dst, page_bytes) || src->planes != dst->planes || bad16(ws) || count > 0x7FFFFFFFu)
    return ZIPNN_ERR_INVALID_ARG;
  if ((src_ids && bad4(src_ids)) || (dst_ids && bad4(dst_ids))) return ZIPNN_ERR_INVALID_ARG;
  if ((!src_ids && count > src->pages) || (!dst_ids && count > dst->pages)) return ZIPNN_ERR_INVALID_ARG;
  const uint64_t a0 = reinterpret_cast<uintptr_t>(src->base), a1 = pool_end(src, page_bytes);
  const uint64_t b0 = reinterpret_cast<uintptr_t>(dst->base), b1 = pool_end(dst, page_bytes);
  const bool overlap = a0 < b1 && b0 < a1;
  const bool same = src->base == dst->base && src->plane_stride == dst->plane_stride && src->page_stride == dst->page_stride &&
                    src->pages == dst->pages;
  if (overlap && !same) return ZIPNN_ERR_INVALID_ARG;
  if (ws_bytes < kHeadBytes) return ZIPNN_ERR_OUT_TOO_SMALL;
  if (!device_ok()) return ZIPNN_ERR_UNSUPPORTED;
  if (count == 0) return ZIPNN_OK;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  Head* head = static_cast<Head*>(ws);
  // without a list of destinations, and from another pool, no page can be written twice or
  // read after it was written
  const bool check = dst_ids || same;
  cudaError_t e = cudaSuccess;
  if (check) {
    TimedLaunch t(kIdPagesPlan, st);
    k_pages_check<<<1, kPlanThreads, 0, st>>>(src_ids, src->pages, dst_ids, dst->pages, count, same, head);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) {
    TimedLaunch t(kIdPagesMove, st);
    const uint32_t vecs = (uint32_t)(page_bytes / 16);
    e = launch(k_pages_copy, copy_grid(count, src->planes, vecs), check, st, device_pool(src), src_ids, device_pool(dst), dst_ids,
               count, src->planes, vecs, head, check);
  }
  return cuda_status(e);
}

zipnn_status zipnn_pages_fork(const zipnn_page_pool* pool, uint64_t page_bytes, const zipnn_page_table* table,
                              const int32_t* rows, const int32_t* parents, const int32_t* lens, uint32_t count, void* ws,
                              size_t ws_bytes, zipnn_stream_t stream) {
  if (!valid_pool(pool, page_bytes) || !valid_table(table, pool) || bad16(ws)) return ZIPNN_ERR_INVALID_ARG;
  if (count > table->seqs || (count && (bad4(rows) || bad4(parents) || bad4(lens)))) return ZIPNN_ERR_INVALID_ARG;
  if (ws_bytes < zipnn_pages_workspace_bytes(table->seqs, pool->pages)) return ZIPNN_ERR_OUT_TOO_SMALL;
  if (!device_ok()) return ZIPNN_ERR_UNSUPPORTED;
  if (count == 0) return ZIPNN_OK;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* b = static_cast<uint8_t*>(ws);
  Head* head = reinterpret_cast<Head*>(b);
  Request* req = reinterpret_cast<Request*>(b + kHeadBytes);
  b += kHeadBytes + align256((uint64_t)table->seqs * sizeof(Request));
  int32_t* fresh = reinterpret_cast<int32_t*>(b);
  b += 3 * align256((uint64_t)pool->pages * 4);
  int32_t* ps = reinterpret_cast<int32_t*>(b);
  int32_t* pd = reinterpret_cast<int32_t*>(b + align256((uint64_t)table->seqs * 4));
  const Meta m = device_meta(table, pool);
  cudaError_t e;
  {
    TimedLaunch t(kIdPagesPlan, st);
    k_pages_plan_fork<<<1, kPlanThreads, 0, st>>>(m, rows, parents, lens, count, head, req, fresh, ps, pd);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) {
    TimedLaunch t(kIdPagesMove, st);
    const uint32_t vecs = (uint32_t)(page_bytes / 16);
    const uint32_t grid = std::max<uint32_t>(std::min<uint32_t>(count, kTakers), copy_grid(count, pool->planes, vecs, kTakers));
    e = launch(k_pages_fork, grid, true, st, m, device_pool(pool), pool->planes, vecs, count, head, req, fresh, ps, pd);
  }
  return cuda_status(e);
}

zipnn_status zipnn_pages_free(const zipnn_page_pool* pool, uint64_t page_bytes, const zipnn_page_table* table,
                              const int32_t* rows, uint32_t count, int compact, void* ws, size_t ws_bytes,
                              zipnn_stream_t stream) {
  if (!valid_pool(pool, page_bytes) || !valid_table(table, pool) || bad16(ws)) return ZIPNN_ERR_INVALID_ARG;
  if (count > 0x7FFFFFFFu || (count && bad4(rows))) return ZIPNN_ERR_INVALID_ARG;
  if (ws_bytes < zipnn_pages_workspace_bytes(table->seqs, pool->pages)) return ZIPNN_ERR_OUT_TOO_SMALL;
  if (!device_ok()) return ZIPNN_ERR_UNSUPPORTED;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* b = static_cast<uint8_t*>(ws);
  Head* head = reinterpret_cast<Head*>(b);
  b += kHeadBytes + align256((uint64_t)table->seqs * sizeof(Request));
  const uint64_t list = align256((uint64_t)pool->pages * 4);
  int32_t* to = reinterpret_cast<int32_t*>(b);
  int32_t* ps = reinterpret_cast<int32_t*>(b + list);
  int32_t* pd = reinterpret_cast<int32_t*>(b + 2 * list);
  const Meta m = device_meta(table, pool);
  cudaError_t e = cudaSuccess;
  if (count) {
    TimedLaunch t(kIdPagesPlan, st);
    k_pages_free<<<std::min(count, 148u * 8), kCopyThreads, 0, st>>>(m, rows, count, head);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess && compact) {
    TimedLaunch t(kIdPagesPlan, st);
    k_pages_plan_compact<<<1, kPlanThreads, 0, st>>>(m, head, to, ps, pd);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess && compact) {
    TimedLaunch t(kIdPagesMove, st);
    const uint32_t vecs = (uint32_t)(page_bytes / 16);
    e = launch(k_pages_compact, copy_grid(pool->pages / 2 + 1, pool->planes, vecs, kTakers), true, st, m, device_pool(pool), pool->planes, vecs,
               head, to, ps, pd);
  }
  return cuda_status(e);
}

}  // extern "C"
