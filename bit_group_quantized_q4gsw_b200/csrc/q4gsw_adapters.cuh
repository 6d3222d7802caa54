// q4gsw_adapters.cuh - the plan of a batch over many adapters: its map in
// device memory, shared by the kernel that writes it and those that read it.
//
// int32 words:
//   head   [4]          tiles in use, M, L, kPlanMark: a kernel that is given a plan of
//                       other sizes does nothing (its rows would lie outside the batch)
//   first  [L + 2]      the sorted order's start of adapter a; of the tokens without
//                       one (L); M (L + 1)
//   order  [M]          the tokens, sorted by adapter, those without one last
//   tile   [slots]      the adapter of each tile, kNoAdapter, or kNoTile past the last
//   rows   [slots][16]  the tokens of each tile, -1 where it has fewer
//   pair   [pairs]      the first of two tiles of one adapter (of the second there may be
//                       none: the next tile is another's then), -1 past the last
// (each part padded to 16 bytes).  The number of slots follows from M and L alone,
// so that grids are known on the host: a group of c tokens has ceil(c / 16) tiles,
// together at most (M + 15 g) / 16 for g = min(L + 1, M) groups, and t tiles have
// ceil(t / 2) pairs, together at most (slots + g) / 2.
#pragma once

#include <cstddef>
#include <cstdint>

namespace q4gsw {
namespace ma {

constexpr int kTileRows = 16;
constexpr int kMaxAdapters = 1024;
constexpr int kMaxPlanTokens = 1 << 27;
constexpr int kNoAdapter = -1;
constexpr int kNoTile = -2;
constexpr int kPlanMark = 0x6e616c70;

struct PlanView {
  int32_t* head;
  int32_t* first;
  int32_t* order;
  int32_t* tile;
  int32_t* rows;
  int32_t* pair;
};

__host__ __device__ inline int plan_slots(int M, int L) {
  const int g = L + 1 < M ? L + 1 : M;
  return (int)(((long long)M + 15LL * g) / kTileRows);
}
__host__ __device__ inline int plan_pairs(int M, int L) {
  const int g = L + 1 < M ? L + 1 : M;
  return (plan_slots(M, L) + g) / 2;
}
__host__ __device__ inline size_t plan_pad(size_t words) { return (words + 3) / 4 * 4; }

__host__ __device__ inline PlanView plan_view(int32_t* p, int M, int L) {
  PlanView v;
  v.head = p;
  v.first = v.head + 4;
  v.order = v.first + plan_pad((size_t)L + 2);
  v.tile = v.order + plan_pad((size_t)M);
  v.rows = v.tile + plan_pad((size_t)plan_slots(M, L));
  v.pair = v.rows + (size_t)plan_slots(M, L) * kTileRows;
  return v;
}
__host__ __device__ inline size_t plan_words(int M, int L) {
  const size_t s = (size_t)plan_slots(M, L);
  return 4 + plan_pad((size_t)L + 2) + plan_pad((size_t)M) + plan_pad(s) + s * kTileRows +
         plan_pad((size_t)plan_pairs(M, L));
}

}  // namespace ma
}  // namespace q4gsw
