// cache_attend_ring.cuh - how a warp of the attention kernels streams its tiles
// of keys and values from the cache's pages into shared memory.
//
// Each warp has a ring of stages of its own, filled by asynchronous copies (of
// 16 bytes, or of 4 where the rows are no whole 16-byte vectors), and waits
// for no other warp. The copies run ahead of the arithmetic
// across the ends of rows, and the table entry of a tile is read one tile
// before its copies need it. Tokens outside the row, and elements past the head
// dim, are filled with zeros, whatever their slots hold.
#pragma once

#include "cache_attend.cuh"

namespace cmdx {

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

// N bytes to shared memory, or as many zeros where !take
template <int N>
__device__ __forceinline__ void copy_bytes(uint32_t dst, const void* src, bool take) {
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(take ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 2^x for x <= 0 (a result below 2^-126 is 0)
__device__ __forceinline__ float power_of_two(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Tiles of TOKENS rows of up to DP elements of type T, PITCH bytes apart,
// copied COPY bytes at a time; STAGES stages, WARPS warps to a CTA.
template <class T, int DP, int COPY, int TOKENS, int PITCH, int STAGES, int WARPS>
struct AttendRing {
  static constexpr int CHUNKS = DP * (int)sizeof(T) / COPY;
  static constexpr int kEach = COPY / (int)sizeof(T);             // elements of a copy
  static constexpr int kKeys = TOKENS * PITCH;  // bytes of a stage's keys; the values follow
  static constexpr int kStage = 2 * kKeys;
  static constexpr int kBytes = STAGES * kStage;
  static constexpr int kTile = TOKENS * WARPS;                    // tokens of a CTA's tile
  static constexpr int kRows = CHUNKS < 32 ? 32 / CHUNKS : 1;     // rows that one copy of the warp covers
  static constexpr int kPieces = CHUNKS < 32 ? 1 : CHUNKS / 32;   // and copies that a row takes
  static_assert(CHUNKS < 32 ? 32 % CHUNKS == 0 : CHUNKS % 32 == 0, "a copy covers whole rows");

  const AttendParams& p;
  const AttendRows& rows;
  const AttendShare& share;
  const int lane, warp;
  const uint32_t at;     // the ring's shared address
  const int copy_row, chunk, chunks;
  const bool one_page;   // a tile lies in one page
  // the tile to copy next: the page (-1: none) and slot of this lane's token,
  // lane % TOKENS, and the head's keys and values
  int page = -1, slot = 0;
  const T *k = nullptr, *v = nullptr;
  const int32_t* table = nullptr;
  AttendSegment look;    // the segment of the tile after it
  int look_at = -1;
  uint32_t known[STAGES];  // of the tiles on their way, nearest first: the tokens that have a page
  int stage = 0;         // to be read next

  __device__ __forceinline__ AttendRing(const AttendParams& p_, const AttendRows& r, const AttendShare& s,
                                        const AttendSegment& first, const void* ring)
      : p(p_), rows(r), share(s), lane(threadIdx.x & 31), warp(threadIdx.x >> 5), at(smem_addr(ring)),
        copy_row(lane / CHUNKS), chunk(lane % CHUNKS), chunks(p_.dim / kEach),
        one_page(p_.page.d % TOKENS == 0), look(first) {
    look_up();
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) {
      known[i] = copy(i);
      look_up();
    }
  }

  __device__ __forceinline__ void look_up() {
    page = -1;
    if (look_at < 0 || look_at == look.tiles) {
      if (look_at > 0) look = attend_next(p, rows, share, look, kTile);
      look_at = 0;
      if (look.tiles == 0) return;
      table = p.tables + look.row * p.table_st[0];
      const int head = look.group / p.blocks;
      k = static_cast<const T*>(p.k) + chunk * kEach + head * p.k_st[2];
      v = static_cast<const T*>(p.v) + chunk * kEach + head * p.v_st[2];
    }
    const int token = (look.tile0 + look_at) * kTile + warp * TOKENS + lane % TOKENS;
    const uint32_t column = fast_div32(p.page, (uint32_t)token);
    slot = token - (int)(column * p.page.d);
    if (token >= look.lo && token < look.n) {
      page = __ldg(table + column * p.table_st[1]);
      if (page < 0 || page >= p.n_pages) {
        report(p.status, CMD_CACHE_BAD_PAGE);
        page = -1;
      }
    }
    ++look_at;
  }

  // Copies the next tile into a stage; returns which of its tokens have a page.
  __device__ __forceinline__ uint32_t copy(int into) {
    const uint32_t has = __ballot_sync(~0u, page >= 0) & ((1u << TOKENS) - 1u);
    if (has) {
      const uint32_t dst = at + into * kStage + copy_row * PITCH + chunk * COPY;
      const int64_t one = __shfl_sync(~0u, page, __ffs(has) - 1);
      const int64_t first = __shfl_sync(~0u, slot, 0) + copy_row;
      const T* k0 = k + one * p.k_st[0] + first * p.k_st[1];
      const T* v0 = v + one * p.v_st[0] + first * p.v_st[1];
#pragma unroll
      for (int r = 0; r < TOKENS; r += kRows) {
        const bool in = has >> (r + copy_row) & 1;
        const T *ks = k0 + r * p.k_st[1], *vs = v0 + r * p.v_st[1];
        if (!one_page) {
          const int64_t pg = __shfl_sync(~0u, page, r + copy_row), sl = __shfl_sync(~0u, slot, r + copy_row);
          ks = k + pg * p.k_st[0] + sl * p.k_st[1];
          vs = v + pg * p.v_st[0] + sl * p.v_st[1];
        }
#pragma unroll
        for (int c = 0; c < kPieces; ++c) {
          const bool take = in && chunk + 32 * c < chunks;
          const int e = 32 * c * kEach, to = r * PITCH + 32 * c * COPY;
          copy_bytes<COPY>(dst + to, take ? static_cast<const void*>(ks + e) : p.k, take);
          copy_bytes<COPY>(dst + to + kKeys, take ? static_cast<const void*>(vs + e) : p.v, take);
        }
      }
    }
    copy_commit();
    return has;
  }

  // Waits for the tile to be read next, with another on its way; returns its
  // tokens that have a page and its stage's index.
  __device__ __forceinline__ uint32_t next_tile(int* index) {
    copy_wait<STAGES - 2>();
    __syncwarp();
    known[STAGES - 1] = copy(stage == 0 ? STAGES - 1 : stage - 1);
    look_up();
    const uint32_t here = known[0];
#pragma unroll
    for (int j = 0; j < STAGES - 1; ++j) known[j] = known[j + 1];
    *index = stage;
    stage = stage == STAGES - 1 ? 0 : stage + 1;
    return here;
  }
  // The stage read last, free until the next tile is asked for.
  __device__ __forceinline__ int free_stage() const { return (stage == 0 ? STAGES : stage) - 1; }
};

}  // namespace cmdx
