// Pages of a cache: copying, sharing on a fork, freeing and compacting.
//
// The page state is the caller's: block tables int32[num_seqs,
// max_blocks_per_seq] (negative: no block) and ref_counts int32[num_blocks],
// the number of table entries that name each block (0: free). Allocation takes
// the free blocks with the lowest ids, in a fixed order, so that every result is
// a function of the inputs alone (counts change by atomics, whose sums do not
// depend on their order).
#include <cooperative_groups.h>

#include "../../include/pagedkv.h"
#include "internal.h"

namespace cg = cooperative_groups;

namespace pagedkv {

__device__ uint32_t g_pages_error;

namespace {

// ------------------------------------------------------------------- copy
// pool[dst] = pool[src] for every pair and pool: one read and one write of HBM.
// blockIdx.y is the pool, so that one launch serves every layer's pools; the
// CTAs of a pool stride over the items (pair, 16 KB chunk of the block). A warp
// takes the ids of 32 items with one load per array and skips those that are
// padding by ballot (a compaction's list is as long as the most moves possible).
// Consecutive pairs of one source (a parent's forks) are one item, its chunk
// read once and written to each: reads that hit L2 still share the way to it with
// the writes (480 forks of 32 parents, 64 pools of 64 KB blocks and their scales:
// 554 -> 371 us, 5.4 TB/s written).
// Blocks under 2 KB (scale pools) or not in 16-byte units are copied as one
// flat list of 16-, 4- or 1-byte elements instead, so that no CTA is spent on
// a few bytes.
constexpr uint32_t kMaxPools = 128;  // per launch: 3 KB of kernel parameters
constexpr uint32_t kChunkBytes = 16384, kWideBytes = 2048;
constexpr uint32_t kCopyThreads = 256;
constexpr uint32_t kRun = 16;

struct CopyPool {
  uint8_t* base;
  uint64_t bytes;   // of a block
  uint32_t width;   // bytes per element: 16, 4 or 1
  uint32_t chunks;  // 16 KB chunks of a block; 0: the flat list
};

struct CopyParams {
  CopyPool pool[kMaxPools];
  const int32_t* src;
  const int32_t* dst;
  uint32_t num_pairs, num_blocks;
};

// A pair's block id, -1 for padding. One at or past num_blocks is flagged and
// the pair skipped.
__device__ __forceinline__ int32_t block_id(const CopyParams& p, int32_t id) {
  if (id < 0) return -1;
  if (uint32_t(id) < p.num_blocks) return id;
  atomicOr(&g_pages_error, kErrPageRange);
  return -1;
}

template <typename T>
__device__ __forceinline__ void copy_flat(const CopyParams& p, const CopyPool& pool) {
  const uint64_t per = pool.bytes / sizeof(T), total = per * p.num_pairs;
  T* const base = reinterpret_cast<T*>(pool.base);
  for (uint64_t e = uint64_t(blockIdx.x) * kCopyThreads + threadIdx.x; e < total;
       e += uint64_t(gridDim.x) * kCopyThreads) {
    const uint64_t pair = e / per, at = e % per;
    const int32_t src = block_id(p, p.src[pair]), dst = src >= 0 ? block_id(p, p.dst[pair]) : -1;
    if (src >= 0 && dst >= 0) base[uint64_t(uint32_t(dst)) * per + at] = base[uint64_t(uint32_t(src)) * per + at];
  }
}

__global__ void __launch_bounds__(kCopyThreads) copy_blocks_kernel(const __grid_constant__ CopyParams p) {
  const CopyPool& pool = p.pool[blockIdx.y];
  if (pool.chunks == 0) {
    if (pool.width == 16) copy_flat<uint4>(p, pool);
    else if (pool.width == 4) copy_flat<uint32_t>(p, pool);
    else copy_flat<uint8_t>(p, pool);
    return;
  }
  const uint32_t lane = threadIdx.x & 31;
  const uint64_t items = uint64_t(p.num_pairs) * pool.chunks;
  for (uint64_t i0 = blockIdx.x; i0 < items; i0 += 32ull * gridDim.x) {
    const uint64_t i = i0 + uint64_t(lane) * gridDim.x;
    // A pair whose source is that of the pair before it is copied with that one
    // (runs end at multiples of kRun).
    int32_t src = -1;
    if (i < items) {
      const uint32_t pair = uint32_t(i / pool.chunks);
      src = block_id(p, p.src[pair]);
      if (pair % kRun && p.src[pair - 1] == src) src = -1;
    }
    for (uint32_t todo = __ballot_sync(0xffffffffu, src >= 0); todo; todo &= todo - 1) {
      const uint32_t l = __ffs(todo) - 1;
      const uint64_t it = i0 + uint64_t(l) * gridDim.x;
      const uint32_t pair = uint32_t(it / pool.chunks);
      const uint64_t off = it % pool.chunks * kChunkBytes;
      const int32_t from = __shfl_sync(0xffffffffu, src, l);
      const uint32_t n = uint32_t(pool.bytes - off < kChunkBytes ? pool.bytes - off : kChunkBytes) / 16;
      const uint4* s = reinterpret_cast<const uint4*>(pool.base + uint64_t(uint32_t(from)) * pool.bytes + off);
      constexpr uint32_t kVecs = kChunkBytes / 16 / kCopyThreads;
      uint4 v[kVecs];
#pragma unroll
      for (uint32_t u = 0; u < kVecs; ++u)
        if (threadIdx.x + u * kCopyThreads < n) v[u] = __ldcs(s + threadIdx.x + u * kCopyThreads);
      // lane t: the pair t places on, if it is of the run
      int32_t dst = -1;
      bool same = pair % kRun + lane < kRun && pair + lane < p.num_pairs;
      if (same) {
        same = p.src[pair + lane] == from;
        if (same) dst = block_id(p, p.dst[pair + lane]);
      }
      const uint32_t run = __ffs(~__ballot_sync(0xffffffffu, same)) - 1;  // (kRun < 32: some lane is not of it)
      for (uint32_t t = 0; t < run; ++t) {
        const int32_t to = __shfl_sync(0xffffffffu, dst, t);
        if (to < 0) continue;
        uint4* d = reinterpret_cast<uint4*>(pool.base + uint64_t(uint32_t(to)) * pool.bytes + off);
#pragma unroll
        for (uint32_t u = 0; u < kVecs; ++u)
          if (threadIdx.x + u * kCopyThreads < n) d[threadIdx.x + u * kCopyThreads] = v[u];
      }
    }
  }
}

// ------------------------------------------------------------------- free
// Entries [first, end) of a row (given, or those that a window has left
// behind) become -1 and their blocks' counts drop by one. A count that is 0
// already is flagged and stays.
struct FreeParams {
  int32_t* tables;
  int32_t* refs;
  const int32_t* first;     // null: from the window
  const int32_t* end;
  const int32_t* seq_lens;  // with the window
  uint32_t max_blocks_per_seq, num_blocks, block_size, sliding_window, num_sinks;
};

__global__ void __launch_bounds__(128) free_blocks_kernel(const FreeParams p) {
  const uint32_t row = blockIdx.x;
  int64_t a, b;
  if (p.first) {
    a = __ldg(p.first + row);
    b = __ldg(p.end + row);
    a = a < 0 ? 0 : a;
  } else {
    // as the attention calls cut it; positions below `behind` are out of view
    int64_t L = __ldg(p.seq_lens + row);
    const int64_t cap = int64_t(p.max_blocks_per_seq) * p.block_size;
    if (L > cap) {
      L = cap;
      if (threadIdx.x == 0) atomicOr(&g_pages_error, kErrSeqLenClamped);
    }
    const int64_t behind = L - p.sliding_window;
    a = (int64_t(p.num_sinks) + p.block_size - 1) / p.block_size;
    b = behind > 0 ? behind / p.block_size : 0;
  }
  if (b > int64_t(p.max_blocks_per_seq)) b = p.max_blocks_per_seq;
  int32_t* t = p.tables + uint64_t(row) * p.max_blocks_per_seq;
  for (int64_t j = a + threadIdx.x; j < b; j += blockDim.x) {
    const int32_t id = t[j];
    if (id < 0) continue;
    t[j] = -1;
    if (uint32_t(id) >= p.num_blocks) {
      atomicOr(&g_pages_error, kErrPageRange);
    } else if (atomicSub(p.refs + id, 1) <= 0) {
      atomicAdd(p.refs + id, 1);
      atomicOr(&g_pages_error, kErrPageRange);
    }
  }
}

// ------------------------------------------------------------------- fork
// Two kernels. fork_pages (one CTA: the work is a scan of the counts, in id
// order, up to as many free blocks as there are partial pages) checks the forks
// and gives each partial page a block; fork_rows writes the rows and counts the
// shared blocks. A fork that cannot be made gets the pair (-2, -2), which is
// padding to the copy too.
struct ForkParams {
  int32_t* tables;
  int32_t* seq_lens;
  int32_t* refs;
  const int32_t* src_seqs;
  const int32_t* dst_seqs;
  int32_t* copy_src;
  int32_t* copy_dst;
  uint32_t num_forks, max_blocks_per_seq, num_seqs, num_blocks, block_size;
};

constexpr uint32_t kScanThreads = 1024;

// Inclusive prefix sum of v over the CTA's threads (kScanThreads of them);
// *total gets the sum. s_part: 32 words of shared memory, free again after the
// next __syncthreads.
__device__ __forceinline__ uint32_t block_prefix(uint32_t v, uint32_t* s_part, uint32_t* total) {
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= uint32_t(o)) v += t;
  }
  if (lane == 31) s_part[warp] = v;
  __syncthreads();
  uint32_t w = s_part[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t t = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= uint32_t(o)) w += t;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const uint32_t before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  return v + (warp > 0 ? before : 0u);
}

__global__ void __launch_bounds__(kScanThreads) fork_pages_kernel(const ForkParams p) {
  extern __shared__ uint32_t smem[];
  __shared__ uint32_t s_part[2][32];
  const uint32_t words = (p.num_seqs + 31) / 32;
  uint32_t* const is_dst = smem;           // rows that some fork writes
  uint32_t* const twice = smem + words;    // rows that more than one does
  uint32_t* const fresh = twice + words;   // the free blocks given out, by rank
  const uint32_t tid = threadIdx.x;
  launch_dependents();  // fork_rows, which waits for this grid
  for (uint32_t i = tid; i < 2 * words; i += kScanThreads) smem[i] = 0;
  __syncthreads();
  for (uint32_t i = tid; i < p.num_forks; i += kScanThreads) {
    const int32_t d = __ldg(p.dst_seqs + i);
    if (d < 0 || uint32_t(d) >= p.num_seqs) continue;
    const uint32_t bit = 1u << (d & 31);
    if (atomicOr(&is_dst[d >> 5], bit) & bit) atomicOr(&twice[d >> 5], bit);
  }
  __syncthreads();
  // ranks of the forks that need a block, in fork order
  uint32_t need = 0, flip = 0;
  for (uint32_t i0 = 0; i0 < p.num_forks; i0 += kScanThreads, flip ^= 1) {
    const uint32_t i = i0 + tid;
    int32_t page = -2;  // -2: not made, -1: no partial page
    if (i < p.num_forks) {
      const int32_t s = __ldg(p.src_seqs + i), d = __ldg(p.dst_seqs + i);
      const bool in = s >= 0 && uint32_t(s) < p.num_seqs && d >= 0 && uint32_t(d) < p.num_seqs;
      if (in && !((twice[d >> 5] >> (d & 31)) & 1u) && !((is_dst[s >> 5] >> (s & 31)) & 1u)) {
        const int64_t L = p.seq_lens[s];
        if (L >= 0 && L <= int64_t(p.max_blocks_per_seq) * p.block_size) {
          page = -1;
          if (L % p.block_size) {
            page = p.tables[uint64_t(s) * p.max_blocks_per_seq + uint64_t(L / p.block_size)];
            page = page < 0 ? -1 : page;
            if (page >= 0 && uint32_t(page) >= p.num_blocks) page = -2;
          }
        }
      }
      if (page == -2) atomicOr(&g_pages_error, kErrPageRange);
    }
    uint32_t total;
    const uint32_t incl = block_prefix(page >= 0 ? 1u : 0u, s_part[flip], &total);
    if (i < p.num_forks) {
      p.copy_src[i] = page;
      p.copy_dst[i] = page >= 0 ? int32_t(need + incl - 1) : page;  // the rank, for now
    }
    need += total;
  }
  // the lowest free blocks: 16 ids per thread and step
  uint32_t found = 0;
  for (uint64_t b0 = 0; b0 < p.num_blocks && found < need; b0 += 16 * kScanThreads, flip ^= 1) {
    const uint64_t b = b0 + 16 * uint64_t(tid);
    uint32_t mask = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint64_t bu = b + 4 * u;
      if (bu + 4 <= p.num_blocks) {
        const int4 r = *reinterpret_cast<const int4*>(p.refs + bu);
        mask |= (uint32_t(r.x <= 0) | (uint32_t(r.y <= 0) << 1) | (uint32_t(r.z <= 0) << 2) | (uint32_t(r.w <= 0) << 3))
                << (4 * u);
      } else {
        for (int q = 0; q < 4; ++q)
          if (bu + q < p.num_blocks && p.refs[bu + q] <= 0) mask |= 1u << (4 * u + q);
      }
    }
    uint32_t total;
    uint32_t rank = found + block_prefix(__popc(mask), s_part[flip], &total) - __popc(mask);
    for (; mask && rank < need; mask &= mask - 1, ++rank) fresh[rank] = uint32_t(b) + __ffs(mask) - 1;
    found += total;
  }
  __syncthreads();
  for (uint32_t i = tid; i < p.num_forks; i += kScanThreads) {
    const int32_t rank = p.copy_dst[i];
    if (rank < 0) continue;
    if (uint32_t(rank) < found) {
      p.copy_dst[i] = int32_t(fresh[rank]);
      p.refs[fresh[rank]] = 1;
    } else {
      p.copy_src[i] = p.copy_dst[i] = -2;
      atomicOr(&g_pages_error, kErrNoFreeBlock);
    }
  }
}

__global__ void __launch_bounds__(128) fork_rows_kernel(const ForkParams p) {
  const uint32_t i = blockIdx.x;
  wait_for_prerequisite();
  const int32_t fresh = p.copy_dst[i];
  if (fresh == -2) return;
  const int32_t s = __ldg(p.src_seqs + i), d = __ldg(p.dst_seqs + i);
  const int32_t L = p.seq_lens[s];
  const uint32_t full = uint32_t(L) / p.block_size;
  const int32_t* from = p.tables + uint64_t(s) * p.max_blocks_per_seq;
  int32_t* to = p.tables + uint64_t(d) * p.max_blocks_per_seq;
  for (uint32_t j = threadIdx.x; j < p.max_blocks_per_seq; j += blockDim.x) {
    int32_t id = -1;
    if (j < full) {
      id = from[j];
      if (id >= 0 && uint32_t(id) < p.num_blocks) {
        atomicAdd(p.refs + id, 1);
      } else if (id >= 0) {
        atomicOr(&g_pages_error, kErrPageRange);
        id = -1;
      }
    } else if (j == full) {
      id = fresh;
    }
    to[j] = id;
  }
  if (threadIdx.x == 0) p.seq_lens[d] = L;
}

// ---------------------------------------------------------------- compact
// U blocks are in use; those with an id >= U move to the free ids below U, the
// lowest to the lowest. One launch of one cluster of up to 8 CTAs: each warp
// counts the used blocks of its range of ids (ballots of 32 counts), the counts
// meet in distributed shared memory, and a second pass over the counts (in
// L2 by then) gives every used block >= U and every free block < U its rank,
// which is its place in the list of moves. Then the new ids and counts, then the
// tables, with a cluster barrier before each.
struct CompactParams {
  const int32_t* tables;
  const int32_t* refs;
  int32_t* new_tables;
  int32_t* new_refs;
  int32_t* new_ids;
  int32_t* copy_src;
  int32_t* copy_dst;
  int32_t* num_used;
  uint64_t entries;  // of the tables
  uint32_t num_blocks;
};

constexpr uint32_t kCompactCtas = 8;

__global__ void __launch_bounds__(kScanThreads) compact_kernel(const CompactParams p) {
  cg::cluster_group cluster = cg::this_cluster();
  __shared__ uint32_t s_count;     // used blocks of this CTA's ids
  __shared__ uint32_t s_below;     // used blocks with an id below U (written by the warp that finds it)
  __shared__ uint32_t s_warp[32];  // used blocks of each warp's ids
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster.block_rank(), ctas = cluster.num_blocks();
  // ids in words of 32; this warp's words are [w0, w1)
  const uint32_t words = uint32_t((uint64_t(p.num_blocks) + 31) / 32), per_warp = (words + 32 * ctas - 1) / (32 * ctas);
  const uint32_t w0 = min(words, (rank * 32 + warp) * per_warp), w1 = min(words, w0 + per_warp);
  auto used_word = [&](uint32_t w) {
    const uint64_t id = 32ull * w + lane;
    return __ballot_sync(0xffffffffu, id < p.num_blocks && p.refs[id] > 0);
  };
  uint32_t mine = 0;
#pragma unroll 8
  for (uint32_t w = w0; w < w1; ++w) mine += __popc(used_word(w));
  if (lane == 0) s_warp[warp] = mine;
  __syncthreads();
  uint32_t c = s_warp[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t t = __shfl_up_sync(0xffffffffu, c, o);
    if (lane >= uint32_t(o)) c += t;
  }
  if (tid == 31) s_count = c;
  uint32_t before = __shfl_sync(0xffffffffu, c, warp) - mine;  // used blocks of the CTA's earlier warps
  cluster.sync();
  uint32_t used = 0;
  for (uint32_t r = 0; r < ctas; ++r) {
    const uint32_t n = *cluster.map_shared_rank(&s_count, r);
    if (r < rank) before += n;
    used += n;
  }
  // used blocks below id U: the warp whose words hold it counts up to it
  if (used == p.num_blocks) {
    if (tid == 0) s_below = used;
  } else if (used / 32 >= w0 && used / 32 < w1) {
    uint32_t n = before;
    for (uint32_t w = w0; w < used / 32; ++w) n += __popc(used_word(w));
    n += __popc(used_word(used / 32) & ((1u << (used % 32)) - 1u));
    if (lane < ctas) *cluster.map_shared_rank(&s_below, lane) = n;
  }
  cluster.sync();
  const uint32_t below = s_below, moves = used - below;
  const uint32_t all = ctas * kScanThreads, self = rank * kScanThreads + tid;
  if (self == 0) *p.num_used = int32_t(used);
  for (uint32_t i = moves + self; i < p.num_blocks / 2; i += all) p.copy_src[i] = p.copy_dst[i] = -1;
  // the lists, and the blocks that stay
  for (uint32_t w = w0; w < w1; ++w) {
    const uint64_t id = 32ull * w + lane;
    const uint32_t m = used_word(w);
    const uint32_t n = before + __popc(m & ((1u << lane) - 1u));  // used blocks below id
    before += __popc(m);
    if (id >= p.num_blocks) continue;
    const bool u = (m >> lane) & 1u, low = id < used;
    if (u && !low) {
      p.copy_src[n - below] = int32_t(id);
    } else if (!u && low) {
      p.copy_dst[uint32_t(id) - n] = int32_t(id);
    }
    if (u && low) {
      p.new_ids[id] = int32_t(id);
      p.new_refs[id] = p.refs[id];
    } else if (!u) {
      p.new_ids[id] = -1;
      if (!low) p.new_refs[id] = 0;
    }
  }
  cluster.sync();
  for (uint32_t i = self; i < moves; i += all) {
    const int32_t s = p.copy_src[i], d = p.copy_dst[i];
    p.new_ids[s] = d;
    p.new_refs[d] = p.refs[s];
    p.new_refs[s] = 0;
  }
  cluster.sync();
#pragma unroll 4
  for (uint64_t e = self; e < p.entries; e += all) {
    const int32_t id = p.tables[e];
    int32_t to = -1;
    if (id >= 0) {
      if (uint32_t(id) < p.num_blocks) to = p.new_ids[id];
      if (to < 0) atomicOr(&g_pages_error, kErrPageRange);  // out of range, or a block that counts as free
    }
    p.new_tables[e] = to;
  }
}

}  // namespace

int launch_copy_blocks(void* const* pools, const size_t* block_bytes, uint32_t num_pools, const int32_t* src,
                       const int32_t* dst, uint32_t num_pairs, uint32_t num_blocks, cudaStream_t stream) {
  const DeviceInfo& dev = device_info();
  if (dev.device < 0) return KV_ERR_CUDA;
  for (uint32_t p0 = 0; p0 < num_pools; p0 += kMaxPools) {
    CopyParams c{};
    c.src = src;
    c.dst = dst;
    c.num_pairs = num_pairs;
    c.num_blocks = num_blocks;
    const uint32_t n = num_pools - p0 < kMaxPools ? num_pools - p0 : kMaxPools;
    uint64_t most = 1;  // CTAs that the pool with the most work can use
    for (uint32_t i = 0; i < n; ++i) {
      CopyPool& q = c.pool[i];
      q.base = static_cast<uint8_t*>(pools[p0 + i]);
      q.bytes = block_bytes[p0 + i];
      const uint64_t ends = reinterpret_cast<uintptr_t>(q.base) | q.bytes;
      q.width = ends % 16 == 0 ? 16 : ends % 4 == 0 ? 4 : 1;
      q.chunks = q.width == 16 && q.bytes >= kWideBytes ? uint32_t((q.bytes + kChunkBytes - 1) / kChunkBytes) : 0;
      const uint64_t ctas = q.chunks ? uint64_t(num_pairs) * q.chunks
                                     : (uint64_t(num_pairs) * (q.bytes / q.width) + kCopyThreads - 1) / kCopyThreads;
      most = ctas > most ? ctas : most;
    }
    // eight waves of the 8 CTAs that fit on an SM, shared out among the pools: runs
    // and padding make the CTAs' shares uneven (3,690 moves of 16 KB in 16 pools:
    // two waves 354 us, eight 329, 95% of the copy rate)
    const uint64_t share = (uint64_t(dev.num_sms) * 64 + n - 1) / n;
    const uint32_t gx = uint32_t(most < share ? most : share);
    copy_blocks_kernel<<<dim3(gx, n), kCopyThreads, 0, stream>>>(c);
    if (cudaGetLastError() != cudaSuccess) return KV_ERR_CUDA;
  }
  return KV_OK;
}

cudaError_t launch_free_blocks(int32_t* tables, int32_t* refs, const int32_t* first, const int32_t* end,
                               const int32_t* seq_lens, uint32_t max_blocks_per_seq, uint32_t num_seqs,
                               uint32_t num_blocks, uint32_t block_size, uint32_t sliding_window, uint32_t num_sinks,
                               cudaStream_t stream) {
  FreeParams p{tables, refs, first, end, seq_lens, max_blocks_per_seq, num_blocks, block_size, sliding_window,
               num_sinks};
  free_blocks_kernel<<<num_seqs, 128, 0, stream>>>(p);
  return cudaGetLastError();
}

int launch_fork_blocks(int32_t* tables, int32_t* seq_lens, int32_t* refs, const int32_t* src_seqs,
                       const int32_t* dst_seqs, int32_t* copy_src, int32_t* copy_dst, uint32_t num_forks,
                       uint32_t max_blocks_per_seq, uint32_t num_seqs, uint32_t num_blocks, uint32_t block_size,
                       cudaStream_t stream) {
  ForkParams p{tables,    seq_lens,           refs,     src_seqs,   dst_seqs,  copy_src, copy_dst,
               num_forks, max_blocks_per_seq, num_seqs, num_blocks, block_size};
  const size_t smem = (2ull * ((num_seqs + 31) / 32) + num_forks) * 4;
  constexpr int kMost = 200 * 1024;
  if (smem > kMost) return KV_ERR_UNSUPPORTED;
  static bool set[64] = {false};
  const int dev = device_info().device;
  if (dev < 0 || dev >= 64) return KV_ERR_CUDA;
  if (!set[dev]) {
    if (cudaFuncSetAttribute(fork_pages_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost) != cudaSuccess)
      return KV_ERR_CUDA;
    set[dev] = true;
  }
  fork_pages_kernel<<<1, kScanThreads, smem, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return KV_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(num_forks);
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};  // its launch overlaps the first kernel
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fork_rows_kernel, p) == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

cudaError_t launch_compact_blocks(const int32_t* tables, const int32_t* refs, int32_t* new_tables, int32_t* new_refs,
                                  int32_t* new_ids, int32_t* copy_src, int32_t* copy_dst, int32_t* num_used,
                                  uint32_t max_blocks_per_seq, uint32_t num_seqs, uint32_t num_blocks,
                                  cudaStream_t stream) {
  CompactParams p{tables,   refs,     new_tables, new_refs, new_ids, copy_src,
                  copy_dst, num_used, uint64_t(num_seqs) * max_blocks_per_seq, num_blocks};
  // a CTA per 4096 ids (4 words per warp) or table entries
  const uint64_t work = p.entries > num_blocks ? p.entries : num_blocks;
  uint32_t ctas = 1;
  while (ctas < kCompactCtas && uint64_t(ctas) * 4096 < work) ctas *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kScanThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = ctas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, compact_kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t read_and_clear_pages_error(uint32_t* bits) {
  const uint32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(bits, g_pages_error, sizeof(uint32_t));
  return e != cudaSuccess ? e : cudaMemcpyToSymbol(g_pages_error, &zero, sizeof(uint32_t));
}

}  // namespace pagedkv
