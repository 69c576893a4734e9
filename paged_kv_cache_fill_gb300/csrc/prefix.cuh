// The plan of a decode over shared prefixes (kv_prefix_plan writes it, the
// paged_decode_attn_*_prefix kernels read it): which positions each group of
// sequences attends together, and the pieces that work is cut into.
//
// A piece is (group, KV head, block of 256 rows, run of 128-key tiles), a row one
// (member, query head of the KV head's group). Its unnormalised outputs go to rows
// base_row + member * num_q_heads + query head of the workspace, and a member's
// pieces are `stride` rows apart, so a sequence needs no more than PlanSeq to find
// them.
#pragma once

#include <stdint.h>

namespace pagedkv {

constexpr uint32_t kPrefixRows = 256;     // rows of a piece, at most
constexpr uint32_t kPrefixTile = 128;     // keys of a tile
constexpr uint32_t kPrefixMaxCtas = 192;  // pieces that groups are split into, at most (one per SM)
constexpr uint32_t kPrefixMaxGroups = 4096;  // (shared memory of the plan's CTAs)

// Key tiles of a piece, at least, where a group has as many (64 members over 2,048
// positions, BF16: pieces of one tile 49 us, of two 40, of four 42)
constexpr uint32_t kMinPieceTiles = 2;

// Shared positions, times the members that save reading them (three at most), below which a
// group's members attend alone: a piece takes 7 us of an SM beside its tiles, as much as
// the decode takes to read them. 256 sequences of 8 KV heads, BF16, 200 own positions each,
// in groups of 2 / 4 / 8 that share the given ones (us a layer: alone, shared):
//   256   90, -     78, 89     63, 72
//   512   128, 138  124, 100   88, 76
//   1024  202, 175  202, 119   148, 85
// (8-bit caches, whose decode reads half as much: internal.h, kMinSavedBytes)
constexpr uint32_t kMinGroupKeys = 1024;

struct PlanHeader {
  uint32_t num_seqs, num_groups, num_q_heads, num_kv_heads;  // what the plan was made for
  uint32_t block_size, max_blocks_per_seq, sliding_window, num_sinks;
  uint32_t num_pieces, pad[23];
};
static_assert(sizeof(PlanHeader) == 128);

struct PlanSeq {
  int32_t eff;     // positions [0, eff) are the group's
  int32_t splits;  // partial results
  int32_t row;     // of the first, its query head 0
  int32_t stride;  // rows between them
};
static_assert(sizeof(PlanSeq) == 16);

struct PlanPiece {
  int32_t first, members, leader, kv_head;
  int32_t row0, limit, win_lo, tile0;
  int32_t tiles, base_row, pad[2];
};
static_assert(sizeof(PlanPiece) == 48);

// Where they lie in the plan's buffer.
struct PlanLayout {
  uint64_t seqs, pieces, bytes;
  uint32_t max_pieces;
};

inline uint64_t prefix_max_pieces(uint64_t num_seqs, uint64_t num_groups, uint64_t num_q_heads, uint64_t num_kv_heads) {
  // every group's blocks of rows (whole ones, and one more; two members share, at least), every KV head; and those that
  // splitting adds
  const uint64_t groups = num_groups < num_seqs / 2 ? num_groups : num_seqs / 2;
  return kPrefixMaxCtas +
         num_kv_heads * (groups + (num_seqs * (num_q_heads / num_kv_heads) + kPrefixRows - 1) / kPrefixRows);
}

inline PlanLayout plan_layout(uint64_t num_seqs, uint64_t num_groups, uint64_t num_q_heads, uint64_t num_kv_heads) {
  PlanLayout l;
  l.seqs = sizeof(PlanHeader);
  l.pieces = l.seqs + num_seqs * sizeof(PlanSeq);
  const uint64_t n = prefix_max_pieces(num_seqs, num_groups, num_q_heads, num_kv_heads);
  l.max_pieces = n < 0xffffffffull ? uint32_t(n) : 0xffffffffu;
  l.bytes = l.pieces + n * sizeof(PlanPiece);
  return l;
}

// Rows of partial results, at most: a piece of each (sequence, query head), and 256 for each piece that splitting adds.
inline uint64_t prefix_max_rows(uint64_t num_seqs, uint64_t num_q_heads) {
  return num_seqs * num_q_heads + uint64_t(kPrefixMaxCtas) * kPrefixRows;
}

// The plan's parts, and whether it was made for this call.
struct PrefixView {
  const PlanHeader* head;  // null: no plan
  const PlanSeq* seqs;
  const PlanPiece* pieces;
  float* part_o;   // [rows][head_dim], unnormalised
  float2* part_ml; // [rows]: running maximum (log2 units) and sum
};

// Whether the plan was made for the shapes and the window of this call.
template <typename Params>
__device__ __forceinline__ bool plan_fits(const PlanHeader* h, const Params& p) {
  const uint4 a = __ldcg(reinterpret_cast<const uint4*>(h)), b = __ldcg(reinterpret_cast<const uint4*>(h) + 1);
  return a.x == p.num_seqs && a.y == p.num_groups && a.z == p.num_q_heads && a.w == p.num_kv_heads &&
         b.x == p.block_size && b.y == p.max_blocks_per_seq && b.z == p.sliding_window && b.w == uint32_t(p.plan_sinks);
}

}  // namespace pagedkv
