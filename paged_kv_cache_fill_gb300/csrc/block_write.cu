// FP8 cache write with one scale for each block and KV head.
//
// Sequence s brings its last n_s = query_start_loc[s+1] - query_start_loc[s]
// positions (the tokens that a prefill with the same query_start_loc attends
// from). For each cache block that they touch, each head and each of K and V:
//   a  = max |x| over the finite new values of the block and head
//   s' = max(least power of two with a <= 448 s', 2^-60, and the block's
//        present scale where it holds earlier positions of the sequence)
//   new codes      E4M3(x / s'), saturating
//   earlier codes  E4M3(code * s / s') where s' is larger than s
// Powers of two: E4M3 has a floating point of its own, so a finer scale would
// not round any better, x / s' is exact, and a code that is scaled again when
// the scale grows stays exact down to E4M3's subnormal range (with arbitrary
// scales every growth would round every code of the block once more).
//
// HBM-bound: 4 bytes read and 2 written per position and element of a row. One
// task is (block, head, K or V), so that its maximum needs no other CTA: W warps
// of one CTA keep the task's new values in shared memory between the maximum
// and the encoding, one read of the input. Larger tasks (block_size * head_dim >
// 16384) read their input again from L2 instead. Each thread fetches its own
// values (16-byte cp.async into slots that no other thread touches, so only the
// maximum needs a barrier), a step ahead of the one it works on, with 128 KB of
// slots per SM: 117 us (6.3 TB/s, 93% of the copy rate) for 120,000 tokens of 8
// heads of 128, blocks of 64, rows taken out of wider ones. 192 KB (three steps,
// or three CTAs per SM) takes 131 to 133 us, the reads crowding out the writes
// beside them, and values held in registers, nothing fetched ahead, 150. The
// dependent loads that find an item (search, lengths, table) are waited for
// once per CTA: it takes consecutive steps, whose items its threads look up
// side by side. The (sequence, block) items are not known on the host:
// the grid covers the bound num_tokens / block_size + 2 num_seqs, item v of
// which belongs to the last sequence s with floor(query_start_loc[s] /
// block_size) + 2 s <= v (a sequence touches at most n_s / block_size + 2
// blocks, so the ranges do not overlap).
#include "../../include/pagedkv.h"
#include "internal.h"

#include <type_traits>

namespace pagedkv {

__device__ uint32_t g_block_write_error;

namespace {

constexpr uint32_t kWarps = 8;  // per CTA
constexpr int kHeld = 8;        // 16-byte loads per thread of a step
constexpr int kStages = 2;      // steps in flight per CTA, the present one among them
constexpr int kCtasPerSm = 2;
constexpr uint32_t kMaxItems = 32 * kWarps;  // per CTA

struct BlockWriteParams {
  const uint16_t* key;
  const uint16_t* value;
  uint8_t* k_cache;
  uint8_t* v_cache;
  float* k_scales;
  float* v_scales;
  uint32_t key_stride, value_stride;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* qsl;
  uint32_t max_blocks_per_seq, num_seqs, num_tokens, num_kv_heads, block_size, block_shift;
  uint32_t groups;         // steps per item: a step is kWarps warps' tasks
  uint32_t steps_per_cta;
  uint64_t items;
};

__device__ __forceinline__ uint64_t item_base(const BlockWriteParams& p, uint32_t s) {
  const int32_t q = __ldg(p.qsl + s);
  return uint64_t(q > 0 ? uint32_t(q) >> p.block_shift : 0u) + 2ull * s;
}

// The sequence of item v: an 8-ary search (the probes of a round load side by
// side; two rounds for up to 64 sequences). -1: before the first one.
__device__ __forceinline__ int32_t item_seq(const BlockWriteParams& p, uint64_t v) {
  uint32_t lo = 0, hi = p.num_seqs;
  if (item_base(p, 0) > v) return -1;
  while (hi - lo > 1) {
    const uint32_t step = (hi - lo + 7) / 8;
    uint32_t n = 0;
#pragma unroll
    for (uint32_t i = 1; i < 8; ++i) {
      const uint32_t s = lo + i * step;
      n += s < hi && item_base(p, s) <= v ? 1u : 0u;
    }
    lo += n * step;
    hi = lo + step < hi ? lo + step : hi;
  }
  return int32_t(lo);
}

// An item's place: rows [r0, r1) of block `bid` are new, row r's token is
// tok0 + r. bid < 0: nothing to write.
struct Item {
  int32_t tok0, bid;
  uint32_t r0, r1;
};

__device__ __forceinline__ Item item_at(const BlockWriteParams& p, uint64_t v) {
  Item it{0, -1, 0, 0};
  const int32_t s = item_seq(p, v);
  if (s < 0) return it;
  const int32_t qa = __ldg(p.qsl + s), qb = __ldg(p.qsl + s + 1);
  if (qa < 0 || qb < qa || uint32_t(qb) > p.num_tokens) return it;
  const int64_t cap = int64_t(p.max_blocks_per_seq) << p.block_shift;
  const int64_t L = __ldg(p.seq_lens + s), first = L - (int64_t(qb) - qa);
  const int64_t begin = first > 0 ? first : 0, end = L < cap ? L : cap;
  const int64_t lb = (begin >> p.block_shift) + int64_t(v - item_base(p, uint32_t(s)));
  const int64_t blk0 = lb << p.block_shift;
  const int64_t p0 = begin > blk0 ? begin : blk0;
  const int64_t p1 = end < blk0 + int64_t(p.block_size) ? end : blk0 + int64_t(p.block_size);
  if (p0 >= p1) return it;
  it.bid = __ldg(p.block_tables + uint64_t(uint32_t(s)) * p.max_blocks_per_seq + uint64_t(lb));
#ifdef PAGEDKV_DEBUG_BOUNDS
  if (it.bid >= 0 && !dbg_block_ok(it.bid)) it.bid = -1;
#endif
  it.tok0 = int32_t(int64_t(qa) + (blk0 - first));
  it.r0 = uint32_t(p0 - blk0);
  it.r1 = uint32_t(p1 - blk0);
  return it;
}

// 8 BF16 values into this thread's slot of shared memory: asynchronously where
// rows are 16-byte aligned.
template <bool kVec>
__device__ __forceinline__ void fetch8(uint4* slot, const uint16_t* p) {
  if constexpr (kVec) {
    cp_async16(slot, p);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = uint32_t(p[2 * i]) | (uint32_t(p[2 * i + 1]) << 16);
    *slot = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// max over both halves of |x|, as BF16 bit patterns; kFinite: non-finite values as 0
template <bool kFinite>
__device__ __forceinline__ uint32_t amax2(uint32_t m, uint32_t w) {
  uint32_t a = w & 0x7fff7fffu;
  if constexpr (kFinite) a &= ~__vcmpgtu2(a, 0x7f7f7f7fu);
  return __vmaxu2(m, a);
}
template <bool kFinite>
__device__ __forceinline__ uint32_t amax8(uint32_t m, uint4 x) {
  return amax2<kFinite>(amax2<kFinite>(amax2<kFinite>(amax2<kFinite>(m, x.x), x.y), x.z), x.w);
}

__device__ __forceinline__ uint32_t scaled2(uint32_t w, F2 f) {
  const float2 x = f2_split(f2_mul(f2_make(bf16_lo_to_f32(w), bf16_hi_to_f32(w)), f));
  return f32x2_to_e4m3x2_satfinite(x.x, x.y);
}

// The least power of two s, at least 2^-60, with amax <= 448 s = 1.75 * 2^8 s,
// amax a finite BF16 pattern: 2^(exponent - 8), twice that where the fraction
// exceeds 1.75.
__device__ __forceinline__ float pow2_scale(uint32_t amax) {
  int32_t k = int32_t(amax >> 7) - 127 - 8 + ((amax & 0x7fu) > 0x60u ? 1 : 0);
  if (k < -60) k = -60;
  return __uint_as_float(uint32_t(k + 127) << 23);
}

template <int D, int W, bool kVec>
__global__ void __launch_bounds__(32 * kWarps, kCtasPerSm)
    block_write_kernel(const __grid_constant__ BlockWriteParams p) {
  constexpr uint32_t kLanes = D / 8;            // lanes per row
  constexpr uint32_t kStep = W * (32 / kLanes);  // rows that the task's warps load at a time
  extern __shared__ uint4 s_data[];              // [stage][load][thread]
  __shared__ uint32_t s_max[2][kWarps];
  __shared__ Item s_item[kMaxItems];
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // every sequence's metadata, flagged once
  for (uint32_t s = blockIdx.x * blockDim.x + threadIdx.x; s < p.num_seqs; s += gridDim.x * blockDim.x) {
    const int32_t a = __ldg(p.qsl + s), b = __ldg(p.qsl + s + 1);
    if (a < 0 || b < a || uint32_t(b) > p.num_tokens) atomicOr(&g_block_write_error, kErrQueryLayout);
    if (int64_t(__ldg(p.seq_lens + s)) > (int64_t(p.max_blocks_per_seq) << p.block_shift))
      atomicOr(&g_block_write_error, kErrSeqLenClamped);
  }
  // the CTA's items, one per thread (at most kMaxItems, by launch; past the last: none)
  const uint64_t v0 = uint64_t(blockIdx.x) * p.steps_per_cta / p.groups;
  const uint32_t group0 = uint32_t(uint64_t(blockIdx.x) * p.steps_per_cta % p.groups);
  if (threadIdx.x < (group0 + p.steps_per_cta + p.groups - 1) / p.groups)
    s_item[threadIdx.x] = v0 + threadIdx.x < p.items ? item_at(p, v0 + threadIdx.x) : Item{0, -1, 0, 0};
  __syncthreads();

  // One step of the CTA: its warps' tasks (kWarps / W of an item's 2 H: K, then
  // V, of each head). The thread's rows are row0, row0 + kStep, ...; new ones are
  // those with r - r0 < fresh (r1 is at most block_size: the bound covers that
  // too). No task in this warp, or nothing to write: fresh 0.
  struct Step {
    Item it;
    uint32_t head, fresh;
    bool is_v, live;
  };
  const uint32_t row0 = (warp % W) * (32 / kLanes) + lane / kLanes;
  auto step_of = [&](uint32_t i) {
    Step st;
    const uint32_t g = group0 + i;
    st.it = s_item[g / p.groups];
    const uint32_t task = g % p.groups * (kWarps / W) + warp / W;
    st.live = task < 2 * p.num_kv_heads && st.it.bid >= 0;
    st.is_v = task >= p.num_kv_heads;
    st.head = task - (st.is_v ? p.num_kv_heads : 0u);
    st.fresh = st.live ? st.it.r1 - st.it.r0 : 0u;
    return st;
  };
  // Up to kHeld loads of a step, from the k0th on, into a stage
  auto fetch = [&](const Step& st, uint32_t k0, uint4* slot) {
    const uint32_t stride = st.is_v ? p.value_stride : p.key_stride;
    const uint64_t inc = uint64_t(kStep) * stride;
    uint32_t r = row0 + k0 * kStep - st.it.r0;
    const uint16_t* q = (st.is_v ? p.value : p.key) + int64_t(st.it.tok0 + int32_t(row0)) * stride + k0 * inc +
                        st.head * D + (lane % kLanes) * 8;
#pragma unroll
    for (int u = 0; u < kHeld; ++u, q += inc, r += kStep, slot += 32 * kWarps)
      if (r < st.fresh) fetch8<kVec>(slot, q);
  };
  auto stage = [&](uint32_t i) { return s_data + (i % kStages) * (kHeld * 32 * kWarps) + threadIdx.x; };

  const uint32_t row_elems = p.num_kv_heads * D;
  const uint32_t loads = p.block_size / kStep;  // per thread and step
#pragma unroll
  for (uint32_t i = 0; i < kStages - 1; ++i) {
    if (i < p.steps_per_cta) fetch(step_of(i), 0, stage(i));
    cp_async_commit();
  }
  uint32_t turn = 0;  // of s_max: flipped at every barrier, not at every step (steps with nothing to write have none)
  for (uint32_t i = 0; i < p.steps_per_cta; ++i) {
    if (i + kStages - 1 < p.steps_per_cta) fetch(step_of(i + kStages - 1), 0, stage(i + kStages - 1));
    cp_async_commit();
    cp_async_wait<kStages - 1>();
    const Step st = step_of(i);
    if (st.it.bid < 0) continue;  // the whole CTA's
    const uint32_t r0 = st.it.r0;
    uint4* const x = stage(i);
    float* const scale =
        (st.is_v ? p.v_scales : p.k_scales) + uint64_t(uint32_t(st.it.bid)) * p.num_kv_heads + st.head;
    const float old = st.live && r0 > 0 ? *scale : 0.0f;

    // ---- the task's largest magnitude
    auto largest = [&](auto finite) {
      uint32_t m = 0;
      for (uint32_t k0 = 0; k0 < loads; k0 += kHeld) {
        // more rows than a stage holds: in turn, and again from L2 for the encoding
        if (k0 > 0 || (decltype(finite)::value && loads > kHeld)) {
          fetch(st, k0, x);
          cp_async_commit();
          cp_async_wait<0>();
        }
        uint32_t r = row0 + k0 * kStep - r0;
#pragma unroll
        for (int u = 0; u < kHeld; ++u, r += kStep)
          if (r < st.fresh) m = amax8<decltype(finite)::value>(m, x[u * 32 * kWarps]);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
      return max(m & 0xffffu, m >> 16);
    };
    uint32_t m = largest(std::false_type{});
    if (m >= 0x7f80u) m = largest(std::true_type{});  // (the same in every lane) some value is not finite
    if constexpr (W > 1) {
      if (lane == 0) s_max[turn][warp] = m;  // (not over maxima that a slower warp has yet to read)
      __syncthreads();                       // (also: every warp of the task has read the present scale)
#pragma unroll
      for (uint32_t w = 0; w < W; ++w) m = max(m, s_max[turn][warp / W * W + w]);
      turn ^= 1;
    } else {
      __syncwarp();
    }
    if (!st.live) continue;
    const float sc = fmaxf(old, pow2_scale(m));
    const float inv = __frcp_rn(sc);  // exact for powers of two
    if (warp % W == 0 && lane == 0) *scale = sc;

    // ---- the codes
    uint8_t* const dst = (st.is_v ? p.v_cache : p.k_cache) +
                         ((uint64_t(uint32_t(st.it.bid)) << p.block_shift) + row0) * row_elems + st.head * D +
                         (lane % kLanes) * 8;
    const uint64_t inc = uint64_t(kStep) * row_elems;
    const F2 inv2 = f2_make(inv, inv);
    for (uint32_t k0 = 0; k0 < loads; k0 += kHeld) {
      if (loads > kHeld) {
        fetch(st, k0, x);
        cp_async_commit();
        cp_async_wait<0>();
      }
      uint8_t* q = dst + k0 * inc;
      uint32_t r = row0 + k0 * kStep - r0;
#pragma unroll
      for (int u = 0; u < kHeld; ++u, q += inc, r += kStep)
        if (r < st.fresh) {
          const uint4 w = x[u * 32 * kWarps];
          *reinterpret_cast<uint2*>(q) = make_uint2(scaled2(w.x, inv2) | (scaled2(w.y, inv2) << 16),
                                                    scaled2(w.z, inv2) | (scaled2(w.w, inv2) << 16));
        }
    }
    // ---- the block's earlier rows, where its scale grew
    if (r0 > 0 && sc > old) {
      const float ratio = old * inv;
      auto again = [&](uint32_t w) {
        const uint32_t lo = e4m3x2_to_f16x2(uint16_t(w)), hi = e4m3x2_to_f16x2(uint16_t(w >> 16));
        return uint32_t(f32x2_to_e4m3x2_satfinite(f16_lo_to_f32(lo) * ratio, f16_hi_to_f32(lo) * ratio)) |
               (uint32_t(f32x2_to_e4m3x2_satfinite(f16_lo_to_f32(hi) * ratio, f16_hi_to_f32(hi) * ratio)) << 16);
      };
      uint8_t* q = dst;
#pragma unroll 2
      for (uint32_t r = row0; r < r0; r += kStep, q += inc) {
        const uint2 c = *reinterpret_cast<const uint2*>(q);
        *reinterpret_cast<uint2*>(q) = make_uint2(again(c.x), again(c.y));
      }
    }
  }
  cp_async_wait<0>();
}

template <int D, int W, bool kVec>
cudaError_t launch_t(const BlockWriteParams& p, uint32_t grid, cudaStream_t stream) {
  constexpr int kSmem = kStages * kHeld * 32 * kWarps * 16;
  auto kern = block_write_kernel<D, W, kVec>;
  static bool set[64] = {false};  // the shared-memory opt-in, once per device (none during a later stream capture)
  const int dev = device_info().device;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!set[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    set[dev] = true;
  }
  kern<<<grid, 32 * kWarps, kSmem, stream>>>(p);
  return cudaGetLastError();
}

template <int D, bool kVec>
cudaError_t launch_w(uint32_t w, const BlockWriteParams& p, uint32_t grid, cudaStream_t stream) {
  if constexpr (D < 256)  // (head_dim 256 takes two warps or more)
    if (w == 1) return launch_t<D, 1, kVec>(p, grid, stream);
  return w == 2   ? launch_t<D, 2, kVec>(p, grid, stream)
         : w == 4 ? launch_t<D, 4, kVec>(p, grid, stream)
                  : launch_t<D, 8, kVec>(p, grid, stream);
}

template <int D>
cudaError_t launch_d(bool vec, uint32_t w, const BlockWriteParams& p, uint32_t grid, cudaStream_t stream) {
  return vec ? launch_w<D, true>(w, p, grid, stream) : launch_w<D, false>(w, p, grid, stream);
}

}  // namespace

int launch_write_fp8_block(const BlockWriteArgs& a, cudaStream_t stream) {
  BlockWriteParams p{};
  p.key = a.key;
  p.value = a.value;
  p.k_cache = a.k_cache;
  p.v_cache = a.v_cache;
  p.k_scales = a.k_scales;
  p.v_scales = a.v_scales;
  p.key_stride = a.key_stride;
  p.value_stride = a.value_stride;
  p.block_tables = a.block_tables;
  p.seq_lens = a.seq_lens;
  p.qsl = a.query_start_loc;
  p.max_blocks_per_seq = a.max_blocks_per_seq;
  p.num_seqs = a.num_seqs;
  p.num_tokens = a.num_tokens;
  p.num_kv_heads = a.num_kv_heads;
  p.block_size = a.block_size;
  p.block_shift = uint32_t(__builtin_ctz(a.block_size));
  // warps per task: kHeld loads of 256 elements per warp where 8 warps or fewer
  // are enough
  const uint32_t need = a.block_size * a.head_dim / (kHeld * 256);
  const uint32_t w = need <= 1 ? 1 : need <= 2 ? 2 : need <= 4 ? 4 : 8;
  p.groups = (2 * a.num_kv_heads * w + kWarps - 1) / kWarps;
  p.items = (uint64_t(a.num_tokens) >> p.block_shift) + 2ull * a.num_seqs;
  const uint64_t steps = p.items * p.groups;
  // consecutive steps to one CTA of those that fit on the GPU at a time, as far
  // as their items fit in its list
  const uint64_t fit = uint64_t(device_info().num_sms) * kCtasPerSm;
  const uint64_t share = (steps + fit - 1) / fit, most = uint64_t(kMaxItems - 1) * p.groups;
  p.steps_per_cta = uint32_t(share < most ? share : most);
  if (steps / p.steps_per_cta >= 0x7fffffffull) return KV_ERR_UNSUPPORTED;
  const uint32_t grid = uint32_t((steps + p.steps_per_cta - 1) / p.steps_per_cta);
  const uintptr_t ends = reinterpret_cast<uintptr_t>(a.key) | reinterpret_cast<uintptr_t>(a.value);
  const bool vec = ends % 16 == 0 && a.key_stride % 8 == 0 && a.value_stride % 8 == 0;
  cudaError_t e;
  switch (a.head_dim) {
    case 64: e = launch_d<64>(vec, w, p, grid, stream); break;
    case 128: e = launch_d<128>(vec, w, p, grid, stream); break;
    case 256: e = launch_d<256>(vec, w, p, grid, stream); break;
    default: return KV_ERR_UNSUPPORTED;
  }
  return e == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

cudaError_t read_and_clear_block_write_error(uint32_t* bits) {
  const uint32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(bits, g_block_write_error, sizeof(uint32_t));
  return e != cudaSuccess ? e : cudaMemcpyToSymbol(g_block_write_error, &zero, sizeof(uint32_t));
}

#ifdef PAGEDKV_DEBUG_BOUNDS
PAGEDKV_DEBUG_UNIT(block_write)
#endif

}  // namespace pagedkv
