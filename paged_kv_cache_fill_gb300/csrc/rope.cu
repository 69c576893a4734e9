// Rotary positions: kv_rope turns the heads of BF16 rows, kv_append_rope_* a
// step's queries and keys, the keys on their way into the paged cache with the
// values beside them.
//
// Pair i < R/2 of a head (elements i and i + R/2, or 2i and 2i + 1 where pairs
// are interleaved) at position P turns by P f_i and grows by the amplitude a_i:
//   o_x = a (x cos - y sin),  o_y = a (y cos + x sin)
// and elements from R on are copied. The table that the caller builds once
// (kv_rope_table) holds f_i as a 96-bit fraction of a turn and a_i, so P f_i is
// reduced exactly for any int32 position, and sines and cosines come to 2^-43
// (rope.cuh). The rotation (turn2) is within 2^-22 of each result and 2^-38 of
// its pair's magnitude (times the amplitude), and is rounded once: to BF16, or, divided by the cache's
// scale, to E4M3.
//
// Every row is read once and written once, so HBM bounds the long calls and the
// instructions (122 per warp and 16 bytes a lane) come close behind: 120,000
// tokens of 32 + 2 x 8 heads of 128 into an E4M3 K and a BF16 V take 440 us, 6.4
// TB/s or 95% of the copy rate; 9,001 tokens of 15 + 2 x 3 heads of 256 into E4M3
// caches 43 us (62%); 8,192 rows of 32 heads of 128, 134 MB, 27.2 us (73%); one
// token 4.2 us, the launch. With the rotation of rope.cuh, which has nearly twice
// the operations, they were 480, 44 and 29.4 us. A warp handles 256 /
// head_dim tokens at a time with head_dim / 8 lanes per token; a lane owns the
// same four pairs (or eight copied elements) of every head row of its token and
// so computes their sines and cosines once per token. Query, key and value rows
// are one list per token, cut into items of kRows rows of one of the three. A
// warp takes an equal run of consecutive items and fetches them asynchronously
// into a ring of shared memory of its own, kStages - 1 items ahead. (120,000
// tokens, when 4 stages of 4 rows and 2 CTAs per SM took 480 us: 3 stages 487; 6
// stages beside a table in L2 503; 8 rows an item 630; 3 CTAs 570-605.)
#include <string.h>

#include "../../include/pagedkv.h"
#include "internal.h"
#include "quotient.cuh"
#include "rope.cuh"

namespace pagedkv {

__device__ uint32_t g_rope_error;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCtasPerSm = 2;
constexpr uint32_t kRows = 4;           // head rows of an item
constexpr uint32_t kStages = 4;         // items of a warp's ring
constexpr uint32_t kItemBytes = 2048;   // 256 / head_dim tokens x kRows rows
constexpr uint32_t kTableBytes = sizeof(kSinCosTurn);

struct RopeParams {
  const uint16_t* src[3];  // queries, keys, values: row t at element t * stride
  void* dst[3];            // rotated queries, the K pool, the V pool
  uint64_t dst_row[3];     // elements between rows (tokens) or slots
  const uint4* table;      // per pair: turn fraction (96 bits), amplitude
  const int32_t* positions;
  const int64_t* slots;  // null: kv_rope (queries only)
  uint32_t src_stride[3];
  uint32_t heads[3];
  uint32_t first[3];  // first item of each list within a token step
  uint32_t items;     // items of a token step
  uint32_t num_tokens, rotary_dim;
  float sin_sign;     // -1: turned back
  float scale[3], recip[3];
  bool fp8[3];        // E4M3 destination
  bool exact_div;     // some scale outside the range of the division-free quotient
  bool staged;        // sines and cosines from a shared-memory copy of the table
};

// Sines and cosines of two pairs: 16 bits of each and a rest. A BF16 value times 16
// bits is exact, so x ch - y sh is rounded once, by 2^-24 of (the result + 2^-16 M),
// M = |x cos| + |y sin|; the two rests add 2^-24 of the same each and, rounded to 24
// bits themselves, 2^-41 M: below 2^-22 of the result and 2^-38 M.
struct PairTurn {
  F2 ch, cl, sh, nsh, sl, nsl;
};
__device__ __forceinline__ float top16(float v) { return __uint_as_float((__float_as_uint(v) + 0x80u) & 0xffffff00u); }
__device__ __forceinline__ void turn2(F2 x, F2 y, const PairTurn& t, F2& ox, F2& oy) {
  ox = f2_fma(y, t.nsl, f2_fma(x, t.cl, f2_fma(x, t.ch, f2_mul(y, t.nsh))));
  oy = f2_fma(y, t.cl, f2_fma(x, t.sl, f2_fma(y, t.ch, f2_mul(x, t.sh))));
}

// The same where x or y holds infinities: a pair with one takes the 16 bits alone, since its
// products with them and with the rests may have opposite signs.
__device__ __forceinline__ void turn2_infinite(F2 x, F2 y, const PairTurn& t, F2& ox, F2& oy) {
  F2 fx, fy;
  turn2(x, y, t, fx, fy);
  const float2 x2 = f2_split(x), y2 = f2_split(y), a = f2_split(fx), b = f2_split(fy);
  const float2 c = f2_split(f2_fma(x, t.ch, f2_mul(y, t.nsh))), d = f2_split(f2_fma(y, t.ch, f2_mul(x, t.sh)));
  const bool fin0 = fabsf(x2.x) < INFINITY && fabsf(y2.x) < INFINITY;
  const bool fin1 = fabsf(x2.y) < INFINITY && fabsf(y2.y) < INFINITY;
  ox = f2_make(fin0 ? a.x : c.x, fin1 ? a.y : c.y);
  oy = f2_make(fin0 ? b.x : d.x, fin1 ? b.y : d.y);
}

__device__ __forceinline__ uint32_t codes4(const float (&x)[4], float scale, float recip, bool exact_div) {
  float q[4];
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    if (exact_div) {
      q[i] = __fdiv_rn(x[i], scale), q[i + 1] = __fdiv_rn(x[i + 1], scale);
    } else {
      const float2 two = quotient2_rn(x[i], x[i + 1], scale, recip);
      q[i] = two.x, q[i + 1] = two.y;
    }
  }
  return uint32_t(f32x2_to_e4m3x2_satfinite(q[0], q[1])) | (uint32_t(f32x2_to_e4m3x2_satfinite(q[2], q[3])) << 16);
}

struct Meta {  // of an item's tokens
  int64_t slot[4];
  int32_t pos[4];
};

constexpr uint32_t kRingBytes = kWarps * kStages * (kItemBytes + sizeof(Meta));

// kVec: rows of queries, keys, values and rotated queries all on 16-byte boundaries
template <int D, bool kInter, bool kVec>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr uint32_t kLanes = D / 8;         // lanes per token
  constexpr uint32_t kTokens = 32 / kLanes;  // tokens per warp step
  extern __shared__ __align__(128) uint8_t smem[];  // the warps' rings, then the sin/cos table
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const uint32_t sub = lane / kLanes, l = lane % kLanes;
  const uint32_t half = p.rotary_dim / 2;
  const bool is_pair = l < p.rotary_dim / 8;
  // element offsets of the lane's two groups of four
  const uint32_t off_a = kInter || !is_pair ? 8 * l : 4 * l;
  const uint32_t off_b = kInter || !is_pair ? off_a + 4 : half + 4 * l;
  uint16_t* const ring = reinterpret_cast<uint16_t*>(smem + warp * (kStages * kItemBytes)) + sub * (kRows * D);
  Meta* const metas = reinterpret_cast<Meta*>(smem + kWarps * kStages * kItemBytes) + warp * kStages;

  const uint64_t steps = (uint64_t(p.num_tokens) + kTokens - 1) / kTokens, total = steps * p.items;
  const uint64_t share = total / (uint64_t(gridDim.x) * kWarps), more = total % (uint64_t(gridDim.x) * kWarps);
  const uint64_t gw = uint64_t(blockIdx.x) * kWarps + warp;
  const uint32_t n = uint32_t(share + (gw < more ? 1 : 0));  // this warp's items
  const uint64_t first = gw * share + (gw < more ? gw : more);

  // An item: rows head0 .. + kRows - 1 of a list, of the tokens of a step
  struct Place {
    uint32_t step, k, list, head0, t;
    bool valid;
  };
  auto place = [&](uint32_t step, uint32_t k) {
    Place a;
    a.step = step;
    a.k = k;
    a.list = k >= p.first[2] ? 2u : k >= p.first[1] ? 1u : 0u;
    a.head0 = (k - p.first[a.list]) * kRows;
    a.t = step * kTokens + sub;
    a.valid = a.t < p.num_tokens;
    return a;
  };
  auto after = [&](const Place& a) { return a.k + 1 == p.items ? place(a.step + 1, 0) : place(a.step, a.k + 1); };
  auto fetch = [&](const Place& a, uint32_t stage) {
    if (!a.valid) return;
    if (l == 0) {
      if (p.slots) cp_async8(&metas[stage].slot[sub], p.slots + a.t);
      cp_async4(&metas[stage].pos[sub], p.positions + a.t);
    }
    const uint16_t* src = p.src[a.list] + uint64_t(a.t) * p.src_stride[a.list] + uint64_t(a.head0) * D;
    uint16_t* dst = ring + stage * (kItemBytes / 2);
    const uint32_t rows = min(kRows, p.heads[a.list] - a.head0);
    if constexpr (kVec) {
#pragma unroll
      for (uint32_t j = 0; j < kRows; ++j)
        if (j < rows) cp_async16(dst + j * D + 8 * l, src + j * D + 8 * l);
    } else {
#pragma unroll 8
      for (uint32_t e = l; e < rows * D; e += kLanes) dst[e] = src[e];  // (whole sectors, whatever the alignment)
    }
  };

  // the first items are on their way before the set-up below
  Place next = place(uint32_t(first / p.items), uint32_t(first % p.items)), here = next;
#pragma unroll
  for (uint32_t i = 0; i < kStages - 1; ++i) {
    if (i < n) {
      fetch(next, i);
      next = after(next);
    }
    cp_async_commit();
  }
  const float4* table = reinterpret_cast<const float4*>(kSinCosTurn);
  __shared__ uint64_t s_table_bar;
  if (p.staged) {
    float4* const copy = reinterpret_cast<float4*>(smem + kRingBytes);
    table = copy;
    if (threadIdx.x == 0) {
      mbar_init(&s_table_bar, 1);
      fence_mbar_init();
      mbar_arrive_expect_tx(&s_table_bar, kTableBytes);
      bulk_load(copy, kSinCosTurn, kTableBytes, &s_table_bar);
    }
  }
  uint4 g[4];  // the lane's pairs
#pragma unroll
  for (int q = 0; q < 4; ++q) g[q] = is_pair ? __ldg(p.table + 4 * l + q) : make_uint4(0, 0, 0, 0);
  if (p.staged) {
    __syncthreads();
    if (!mbar_wait(&s_table_bar, 0)) {
      // flagged; the copies land (this one's wait bounded) before the CTA releases its shared memory
      if (lane == 0) atomicOr(&g_rope_error, kErrWaitTimeout);
      cp_async_wait<0>();
      mbar_wait(&s_table_bar, 0);
      return;
    }
  }
  PairTurn sc[2];
  uint32_t sc_token = 0xffffffffu;  // whose sines and cosines these are

  for (uint32_t i = 0; i < n; ++i, here = after(here)) {
    if (i + kStages - 1 < n) {
      fetch(next, (i + kStages - 1) % kStages);
      next = after(next);
    }
    cp_async_commit();
    cp_async_wait<kStages - 1>();
    __syncwarp();
    const uint32_t stage = i % kStages;
    const uint16_t* const row0 = ring + stage * (kItemBytes / 2);
    int64_t slot = here.valid ? (p.slots ? metas[stage].slot[sub] : 0) : -1;
#ifdef PAGEDKV_DEBUG_BOUNDS
    if (slot >= 0 && p.slots && !dbg_slot_ok(slot)) slot = -1;  // skipped like padding
#endif
    const uint32_t list = here.list, rows = min(kRows, p.heads[list] - here.head0);
    if (slot >= 0) {
      const bool turn = list < 2 && is_pair;
      if (turn && here.t != sc_token) {
        sc_token = here.t;
        const int32_t pos = metas[stage].pos[sub];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float4 a0 = turn_sincos(pos, g[2 * k], table), a1 = turn_sincos(pos, g[2 * k + 1], table);
          const float s = p.sin_sign;
          const float c0 = top16(a0.z), c1 = top16(a1.z), s0 = top16(a0.x), s1 = top16(a1.x);
          const float r0 = s * ((a0.x - s0) + a0.y), r1 = s * ((a1.x - s1) + a1.y);
          sc[k].ch = f2_make(c0, c1);
          sc[k].cl = f2_make((a0.z - c0) + a0.w, (a1.z - c1) + a1.w);
          sc[k].sh = f2_make(s * s0, s * s1);
          sc[k].nsh = f2_make(-s * s0, -s * s1);
          sc[k].sl = f2_make(r0, r1);
          sc[k].nsl = f2_make(-r0, -r1);
        }
      }
      const F2 amp0 = f2_make(__uint_as_float(g[0].w), __uint_as_float(g[1].w));
      const F2 amp1 = f2_make(__uint_as_float(g[2].w), __uint_as_float(g[3].w));
      const bool fp8 = p.fp8[list];
      const uint64_t at = (list == 0 ? uint64_t(here.t) : uint64_t(slot)) * p.dst_row[list] + uint64_t(here.head0) * D;
#pragma unroll
      for (uint32_t j = 0; j < kRows; ++j) {
        if (j >= rows) continue;
        uint4 w;
        if constexpr (kInter) {
          w = *reinterpret_cast<const uint4*>(row0 + j * D + off_a);
        } else {
          const uint2 a = *reinterpret_cast<const uint2*>(row0 + j * D + off_a);
          const uint2 b = *reinterpret_cast<const uint2*>(row0 + j * D + off_b);
          w = make_uint4(a.x, a.y, b.x, b.y);
        }
        float y[8];  // elements off_a .. + 3 and off_b .. + 3
        if (turn) {
          F2 x01, y01, x23, y23;
          if constexpr (kInter) {
            x01 = f2_make(bf16_lo_to_f32(w.x), bf16_lo_to_f32(w.y));
            y01 = f2_make(bf16_hi_to_f32(w.x), bf16_hi_to_f32(w.y));
            x23 = f2_make(bf16_lo_to_f32(w.z), bf16_lo_to_f32(w.w));
            y23 = f2_make(bf16_hi_to_f32(w.z), bf16_hi_to_f32(w.w));
          } else {
            x01 = f2_make(bf16_lo_to_f32(w.x), bf16_hi_to_f32(w.x));
            x23 = f2_make(bf16_lo_to_f32(w.y), bf16_hi_to_f32(w.y));
            y01 = f2_make(bf16_lo_to_f32(w.z), bf16_hi_to_f32(w.z));
            y23 = f2_make(bf16_lo_to_f32(w.w), bf16_hi_to_f32(w.w));
          }
          F2 ox01, oy01, ox23, oy23;
          const uint32_t m = __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu),
                                      __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
          if (((m + 0x00800080u) & 0x80008000u) != 0) {
            turn2_infinite(x01, y01, sc[0], ox01, oy01);
            turn2_infinite(x23, y23, sc[1], ox23, oy23);
          } else {
            turn2(x01, y01, sc[0], ox01, oy01);
            turn2(x23, y23, sc[1], ox23, oy23);
          }
          const float2 a = f2_split(f2_mul(ox01, amp0)), b = f2_split(f2_mul(ox23, amp1));
          const float2 c = f2_split(f2_mul(oy01, amp0)), d = f2_split(f2_mul(oy23, amp1));
          if constexpr (kInter) {
            y[0] = a.x, y[1] = c.x, y[2] = a.y, y[3] = c.y, y[4] = b.x, y[5] = d.x, y[6] = b.y, y[7] = d.y;
          } else {
            y[0] = a.x, y[1] = a.y, y[2] = b.x, y[3] = b.y, y[4] = c.x, y[5] = c.y, y[6] = d.x, y[7] = d.y;
          }
          if (!fp8)
            w = make_uint4(f32x2_to_bf16x2(y[0], y[1]), f32x2_to_bf16x2(y[2], y[3]), f32x2_to_bf16x2(y[4], y[5]),
                           f32x2_to_bf16x2(y[6], y[7]));
        } else if (fp8) {
          const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) y[2 * q] = bf16_lo_to_f32(ws[q]), y[2 * q + 1] = bf16_hi_to_f32(ws[q]);
        }
        if (fp8) {
          uint8_t* dst = static_cast<uint8_t*>(p.dst[list]) + at + j * D;
          const float ya[4] = {y[0], y[1], y[2], y[3]}, yb[4] = {y[4], y[5], y[6], y[7]};
          const float s = p.scale[list], r = p.recip[list];
          const uint32_t ca = codes4(ya, s, r, p.exact_div), cb = codes4(yb, s, r, p.exact_div);
          if (kInter || !is_pair) {
            *reinterpret_cast<uint2*>(dst + off_a) = make_uint2(ca, cb);
          } else {
            *reinterpret_cast<uint32_t*>(dst + off_a) = ca;
            *reinterpret_cast<uint32_t*>(dst + off_b) = cb;
          }
        } else {
          // (queries that are not aligned go back into the ring, and out from there below; the caches are aligned)
          uint16_t* dst = !kVec && list == 0 ? const_cast<uint16_t*>(row0) + j * D
                                             : static_cast<uint16_t*>(p.dst[list]) + at + j * D;
          if constexpr (kInter) {
            *reinterpret_cast<uint4*>(dst + off_a) = w;
          } else {
            *reinterpret_cast<uint2*>(dst + off_a) = make_uint2(w.x, w.y);
            *reinterpret_cast<uint2*>(dst + off_b) = make_uint2(w.z, w.w);
          }
        }
      }
    }
    __syncwarp();
    if constexpr (!kVec) {
      if (list == 0) {
        if (slot >= 0) {
          uint16_t* dst = static_cast<uint16_t*>(p.dst[0]) + uint64_t(here.t) * p.dst_row[0] + uint64_t(here.head0) * D;
#pragma unroll 8
          for (uint32_t e = l; e < rows * D; e += kLanes) dst[e] = row0[e];
        }
        __syncwarp();
      }
    }
  }
  cp_async_wait<0>();
}

template <int D>
cudaError_t launch_d(bool inter, bool vec, unsigned blocks, const RopeParams& p, cudaStream_t stream) {
  auto kern = inter ? (vec ? rope_kernel<D, true, true> : rope_kernel<D, true, false>)
                    : (vec ? rope_kernel<D, false, true> : rope_kernel<D, false, false>);
  constexpr int kSmem = int(kRingBytes + kTableBytes);
  static bool set[4][64] = {};  // the shared-memory opt-in, once per kernel and device (none during a later capture)
  const int dev = device_info().device;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  bool& done = set[(inter ? 2 : 0) + (vec ? 1 : 0)][dev];
  if (!done) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    done = true;
  }
  kern<<<blocks, kThreads, p.staged ? kSmem : int(kRingBytes), stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t stream) {
  RopeParams p{};
  bool vec = true;
  for (int i = 0; i < 3; ++i) {
    p.src[i] = a.src[i];
    p.dst[i] = a.dst[i];
    p.src_stride[i] = a.src_stride[i];
    p.heads[i] = a.heads[i];
    p.dst_row[i] = i == 0 ? uint64_t(a.q_out_stride) : uint64_t(a.heads[i]) * a.head_dim;
    p.fp8[i] = i == 1 ? a.fp8_k : i == 2 ? a.fp8_v : false;
    p.scale[i] = i == 1 ? a.k_scale : i == 2 ? a.v_scale : 1.0f;
    p.recip[i] = 1.0f / p.scale[i];
    if (p.fp8[i] && !(p.scale[i] >= kFastScaleMin && p.scale[i] <= kFastScaleMax)) p.exact_div = true;
    p.first[i] = p.items;
    p.items += (a.heads[i] + kRows - 1) / kRows;
    if (a.heads[i] && (reinterpret_cast<uintptr_t>(a.src[i]) % 16 || a.src_stride[i] % 8)) vec = false;
  }
  if (a.heads[0] && (reinterpret_cast<uintptr_t>(a.dst[0]) % 16 || a.q_out_stride % 8)) vec = false;
  p.table = reinterpret_cast<const uint4*>(a.table);
  p.positions = a.positions;
  p.slots = a.slots;
  p.num_tokens = a.num_tokens;
  p.rotary_dim = a.rotary_dim;
  p.sin_sign = a.inverse ? -1.0f : 1.0f;

  const uint32_t tokens = 256 / a.head_dim;  // per step
  const uint64_t total = (uint64_t(a.num_tokens) + tokens - 1) / tokens * p.items;
  const uint64_t warps = uint64_t(device_info().num_sms) * kCtasPerSm * kWarps;  // resident
  uint64_t blocks = (total + kWarps - 1) / kWarps;  // an item per warp at least
  if (blocks > warps / kWarps) blocks = warps / kWarps;
  p.staged = total > 2 * warps;  // (below, a warp looks few angles up: from L2)
  switch (a.head_dim) {
    case 64: return launch_d<64>(a.interleaved, vec, unsigned(blocks), p, stream);
    case 128: return launch_d<128>(a.interleaved, vec, unsigned(blocks), p, stream);
    case 256: return launch_d<256>(a.interleaved, vec, unsigned(blocks), p, stream);
    default: return cudaErrorInvalidValue;
  }
}

// ------------------------------------------------------------ the table (host)
int rope_frequencies(double* freqs, uint32_t R, double theta, int scaling, double factor, double trained, double low,
                     double high) {
  const double two_pi = 6.283185307179586477;
  const double base = scaling == KV_ROPE_BASE && R > 2 ? theta * pow(factor, double(R) / (double(R) - 2.0)) : theta;
  // pairs between which KV_ROPE_BY_INDEX interpolates: those that turn `high` and `low` times
  auto pair_of = [&](double turns) { return R * log(trained / (turns * two_pi)) / (2.0 * log(theta)); };
  double lo = 0.0, hi = 0.0;
  if (scaling == KV_ROPE_BY_INDEX) {
    lo = fmax(0.0, floor(pair_of(high)));
    hi = fmin(double(R) - 1.0, ceil(pair_of(low)));
    if (!(hi > lo)) hi = lo + 0.001;
  }
  for (uint32_t i = 0; i < R / 2; ++i) {
    const double f = pow(base, -2.0 * i / R);
    double keep = 1.0;
    if (scaling == KV_ROPE_LINEAR) keep = 0.0;
    if (scaling == KV_ROPE_BY_TURNS) keep = (trained * f / two_pi - low) / (high - low);
    if (scaling == KV_ROPE_BY_INDEX) keep = 1.0 - (i - lo) / (hi - lo);
    keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
    freqs[i] = keep == 1.0 ? f : f * (keep + (1.0 - keep) / factor);
  }
  return KV_OK;
}

void rope_table(uint32_t* table, const double* freqs, uint32_t rotary_dim, float amplitude) {
  for (uint32_t i = 0; i < rotary_dim / 2; ++i) {
    const uint4 g = turn_fraction(freqs[i]);
    table[4 * i] = g.x;
    table[4 * i + 1] = g.y;
    table[4 * i + 2] = g.z;
    memcpy(table + 4 * i + 3, &amplitude, 4);
  }
}

cudaError_t read_and_clear_rope_error(uint32_t* bits) {
  const uint32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(bits, g_rope_error, sizeof(uint32_t));
  return e != cudaSuccess ? e : cudaMemcpyToSymbol(g_rope_error, &zero, sizeof(uint32_t));
}

#ifdef PAGEDKV_DEBUG_BOUNDS
PAGEDKV_DEBUG_UNIT(rope)
#endif

}  // namespace pagedkv
