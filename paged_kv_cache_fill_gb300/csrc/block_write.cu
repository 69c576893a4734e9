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
// of one CTA hold the task's new values in registers between the maximum
// and the encoding (kHeld 16-byte loads per lane in flight), one read of the
// input. Larger tasks (block_size * head_dim > 16384) read their input again
// from L2 instead. The (sequence, block) items are not known on the host:
// the grid covers the bound num_tokens / block_size + 2 num_seqs, item v of
// which belongs to the last sequence s with floor(query_start_loc[s] /
// block_size) + 2 s <= v (a sequence touches at most n_s / block_size + 2
// blocks, so the ranges do not overlap).
#include "../../include/pagedkv.h"
#include "internal.h"

namespace pagedkv {

__device__ uint32_t g_block_write_error;

namespace {

constexpr uint32_t kWarps = 8;  // per CTA
constexpr int kHeld = 8;        // 16-byte loads per lane held between the two passes

struct BlockWriteParams {
  const uint16_t* src[2];  // key, value
  uint8_t* cache[2];
  float* scales[2];
  uint32_t stride[2];
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* qsl;
  uint32_t max_blocks_per_seq, num_seqs, num_tokens, num_kv_heads, block_size, block_shift;
  uint32_t groups;  // CTAs per item
};

__device__ __forceinline__ uint64_t item_base(const BlockWriteParams& p, uint32_t s) {
  const int32_t q = __ldg(p.qsl + s);
  return uint64_t(q > 0 ? uint32_t(q) >> p.block_shift : 0u) + 2ull * s;
}

// The sequence of item v (every lane gets it): a 33-ary search, two rounds of
// loads for up to 1024 sequences. -1: before the first one.
__device__ __forceinline__ int32_t item_seq(const BlockWriteParams& p, uint64_t v, uint32_t lane) {
  uint32_t lo = 0, hi = p.num_seqs;
  while (true) {
    const uint32_t step = (hi - lo + 31) / 32;
    const uint32_t s = lo + lane * step;
    const uint32_t m = __ballot_sync(0xffffffffu, s < hi && s >= lo && item_base(p, s) <= v);
    if (m == 0) return -1;
    lo += (31 - __clz(m)) * step;
    if (step == 1) return int32_t(lo);
    hi = lo + step < hi ? lo + step : hi;
  }
}

template <bool kVec>
__device__ __forceinline__ uint4 load8(const uint16_t* p) {
  if constexpr (kVec) {
    return __ldcs(reinterpret_cast<const uint4*>(p));
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = uint32_t(p[2 * i]) | (uint32_t(p[2 * i + 1]) << 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// max over both halves of |x|, as BF16 bit patterns, non-finite values as 0
__device__ __forceinline__ uint32_t amax2(uint32_t m, uint32_t w) {
  const uint32_t a = w & 0x7fff7fffu;
  return __vmaxu2(m, a & ~__vcmpgtu2(a, 0x7f7f7f7fu));
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
__global__ void __launch_bounds__(32 * kWarps) block_write_kernel(const BlockWriteParams p) {
  constexpr uint32_t kLanes = D / 8;            // lanes per row
  constexpr uint32_t kRows = 32 / kLanes;       // rows per load of a warp
  __shared__ uint32_t s_max[kWarps];
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t item = blockIdx.x / p.groups, group = blockIdx.x % p.groups;

  if (group == 0 && threadIdx.x == 0 && item < p.num_seqs) {  // sequence `item`'s metadata, flagged once
    const int32_t a = __ldg(p.qsl + item), b = __ldg(p.qsl + item + 1);
    if (a < 0 || b < a || uint32_t(b) > p.num_tokens) atomicOr(&g_block_write_error, kErrQueryLayout);
    if (int64_t(__ldg(p.seq_lens + item)) > (int64_t(p.max_blocks_per_seq) << p.block_shift))
      atomicOr(&g_block_write_error, kErrSeqLenClamped);
  }
  // ---- the item: rows [r0, r1) of logical block lb of sequence s are new
  // (the same in every warp of the CTA, so every exit below is the whole CTA's)
  const int32_t s = item_seq(p, item, lane);
  if (s < 0) return;
  const int32_t qa = __ldg(p.qsl + s), qb = __ldg(p.qsl + s + 1);
  if (qa < 0 || qb < qa || uint32_t(qb) > p.num_tokens) return;
  const int64_t cap = int64_t(p.max_blocks_per_seq) << p.block_shift;
  const int64_t L = __ldg(p.seq_lens + s), first = L - (int64_t(qb) - qa);
  const int64_t begin = first > 0 ? first : 0, end = L < cap ? L : cap;
  const int64_t lb = (begin >> p.block_shift) + int64_t(uint64_t(item) - item_base(p, uint32_t(s)));
  const int64_t blk0 = lb << p.block_shift;
  const int64_t p0 = begin > blk0 ? begin : blk0;
  const int64_t p1 = end < blk0 + p.block_size ? end : blk0 + int64_t(p.block_size);
  if (p0 >= p1) return;
  const int32_t bid = __ldg(p.block_tables + uint64_t(s) * p.max_blocks_per_seq + uint64_t(lb));
  if (bid < 0) return;
#ifdef PAGEDKV_DEBUG_BOUNDS
  if (!dbg_block_ok(bid)) return;
#endif
  const uint32_t r0 = uint32_t(p0 - blk0), r1 = uint32_t(p1 - blk0);

  // ---- the task: K (tasks 0..H-1) or V of one head
  const uint32_t task = group * (kWarps / W) + warp / W, part = warp % W;
  const bool live = task < 2 * p.num_kv_heads;
  const uint32_t kv = live && task >= p.num_kv_heads ? 1u : 0u;
  const uint32_t head = live ? task - kv * p.num_kv_heads : 0u;
  const uint32_t col = head * D + (lane % kLanes) * 8;
  const uint32_t row_elems = p.num_kv_heads * D;
  const uint32_t loads = p.block_size / (W * kRows);  // per lane: rows (k W + part) kRows + lane / kLanes
  const uint32_t row0 = part * kRows + lane / kLanes;
  const int64_t tok0 = int64_t(qa) + (blk0 - first);  // row r's token is tok0 + r
  uint8_t* dst = p.cache[kv] + (uint64_t(uint32_t(bid)) << p.block_shift) * row_elems + col;
  float* scale = p.scales[kv] + uint64_t(uint32_t(bid)) * p.num_kv_heads + head;
  const float old = live && r0 > 0 ? *scale : 0.0f;

  uint4 x[kHeld];
  auto load = [&](uint32_t k0) {
#pragma unroll
    for (int u = 0; u < kHeld; ++u) {
      const uint32_t r = (k0 + u) * (W * kRows) + row0;
      x[u] = live && k0 + u < loads && r >= r0 && r < r1 ? load8<kVec>(p.src[kv] + uint64_t(tok0 + r) * p.stride[kv] + col)
                                                         : make_uint4(0, 0, 0, 0);
    }
  };
  uint32_t m = 0;
  for (uint32_t k0 = 0; k0 < loads; k0 += kHeld) {
    load(k0);
#pragma unroll
    for (int u = 0; u < kHeld; ++u) m = amax2(amax2(amax2(amax2(m, x[u].x), x[u].y), x[u].z), x[u].w);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
  m = max(m & 0xffffu, m >> 16);
  if constexpr (W > 1) {
    if (lane == 0) s_max[warp] = m;
    __syncthreads();  // (also: every warp of the task has read the present scale)
#pragma unroll
    for (uint32_t w = 0; w < W; ++w) m = max(m, s_max[warp / W * W + w]);
  } else {
    __syncwarp();
  }
  if (!live) return;
  const float sc = fmaxf(old, pow2_scale(m));
  const float inv = __frcp_rn(sc);  // exact for powers of two
  if (part == 0 && lane == 0) *scale = sc;

  const F2 inv2 = f2_make(inv, inv);
  for (uint32_t k0 = 0; k0 < loads; k0 += kHeld) {
    if (loads > kHeld) load(k0);
#pragma unroll
    for (int u = 0; u < kHeld; ++u) {
      const uint32_t r = (k0 + u) * (W * kRows) + row0;
      if (k0 + u < loads && r >= r0 && r < r1)
        *reinterpret_cast<uint2*>(dst + uint64_t(r) * row_elems) =
            make_uint2(scaled2(x[u].x, inv2) | (scaled2(x[u].y, inv2) << 16),
                       scaled2(x[u].z, inv2) | (scaled2(x[u].w, inv2) << 16));
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
    for (uint32_t k0 = 0; k0 < loads; k0 += kHeld) {
      uint2 c[kHeld];
#pragma unroll
      for (int u = 0; u < kHeld; ++u) {
        const uint32_t r = (k0 + u) * (W * kRows) + row0;
        if (k0 + u < loads && r < r0) c[u] = *reinterpret_cast<const uint2*>(dst + uint64_t(r) * row_elems);
      }
#pragma unroll
      for (int u = 0; u < kHeld; ++u) {
        const uint32_t r = (k0 + u) * (W * kRows) + row0;
        if (k0 + u < loads && r < r0)
          *reinterpret_cast<uint2*>(dst + uint64_t(r) * row_elems) = make_uint2(again(c[u].x), again(c[u].y));
      }
    }
  }
}

template <int D, bool kVec>
cudaError_t launch_w(uint32_t w, const BlockWriteParams& p, uint32_t grid, cudaStream_t stream) {
  switch (w) {
    case 1:
      if constexpr (D < 256) block_write_kernel<D, 1, kVec><<<grid, 32 * kWarps, 0, stream>>>(p);
      break;  // (head_dim 256 takes two warps or more)
    case 2: block_write_kernel<D, 2, kVec><<<grid, 32 * kWarps, 0, stream>>>(p); break;
    case 4: block_write_kernel<D, 4, kVec><<<grid, 32 * kWarps, 0, stream>>>(p); break;
    default: block_write_kernel<D, 8, kVec><<<grid, 32 * kWarps, 0, stream>>>(p); break;
  }
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(bool vec, uint32_t w, const BlockWriteParams& p, uint32_t grid, cudaStream_t stream) {
  return vec ? launch_w<D, true>(w, p, grid, stream) : launch_w<D, false>(w, p, grid, stream);
}

}  // namespace

int launch_write_fp8_block(const BlockWriteArgs& a, cudaStream_t stream) {
  BlockWriteParams p{};
  p.src[0] = a.key;
  p.src[1] = a.value;
  p.cache[0] = a.k_cache;
  p.cache[1] = a.v_cache;
  p.scales[0] = a.k_scales;
  p.scales[1] = a.v_scales;
  p.stride[0] = a.key_stride;
  p.stride[1] = a.value_stride;
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
  const uint64_t items = (uint64_t(a.num_tokens) >> p.block_shift) + 2ull * a.num_seqs;
  if (items * p.groups > 0x7fffffffull) return KV_ERR_UNSUPPORTED;
  const uint32_t grid = uint32_t(items * p.groups);
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
