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

// The first `bytes` of N bytes to shared memory, and zeros for the others.
template <int N>
__device__ __forceinline__ void copy_bytes(uint32_t dst, const void* src, int bytes) {
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
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
  // the tile to copy next: whether this lane's token, lane % TOKENS, is in the
  // row, its page and slot, and the head's keys and values. (The page is not
  // looked at before the copy, so that its load may be on its way until then.)
  bool inside = false;
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
    inside = false;
    if (look_at < 0 || look_at == look.tiles) {
      if (look_at > 0) look = attend_next(p, rows, share, look, kTile);
      look_at = 0;
      if (look.tiles == 0) return;
      table = p.tables + look.row * p.table_st[0];
      const int head = look.group / p.blocks;
      k = static_cast<const T*>(p.k) + head * p.k_st[2];
      v = static_cast<const T*>(p.v) + head * p.v_st[2];
    }
    const int token = (look.tile0 + look_at) * kTile + warp * TOKENS + lane % TOKENS;
    const uint32_t column = fast_div32(p.page, (uint32_t)token);
    slot = token - (int)(column * p.page.d);
    inside = token >= look.lo && token < look.n;
    if (inside) page = table[column * p.table_st[1]];
    ++look_at;
  }

  // One row's keys and values, or zeros where !take.
  __device__ __forceinline__ void copy_row_of(uint32_t dst, const T* ks, const T* vs, bool take) {
#pragma unroll
    for (int c = 0; c < kPieces; ++c) {
      const int piece = chunk + 32 * c;  // (pieces past the head dim are zeros: they read the first one's address, no bytes)
      const int bytes = take && piece < chunks ? COPY : 0, e = piece < chunks ? piece * kEach : 0;
      copy_bytes<COPY>(dst + 32 * c * COPY, ks + e, bytes);
      copy_bytes<COPY>(dst + 32 * c * COPY + kKeys, vs + e, bytes);
    }
  }

  // Copies the next tile into a stage; returns which of its tokens have a page.
  __device__ __forceinline__ uint32_t copy(int into) {
    constexpr uint32_t kAll = (1u << TOKENS) - 1u;
    if (inside && (page < 0 || page >= p.n_pages)) {
      report(p.status, CMD_CACHE_BAD_PAGE);
      inside = false;
    }
    const uint32_t has = __ballot_sync(~0u, inside) & kAll;
    if (has) {
      const uint32_t dst = at + into * kStage + copy_row * PITCH + chunk * COPY;
      if (one_page) {
        const int64_t one = __shfl_sync(~0u, page, __ffs(has) - 1);
        const int64_t first = __shfl_sync(~0u, slot, 0) + copy_row;
        const T* ks = k + one * p.k_st[0] + first * p.k_st[1];
        const T* vs = v + one * p.v_st[0] + first * p.v_st[1];
        const int64_t k_step = kRows * p.k_st[1], v_step = kRows * p.v_st[1];
        if (has == kAll) {
#pragma unroll
          for (int r = 0; r < TOKENS; r += kRows) {
            copy_row_of(dst + r * PITCH, ks, vs, true);
            ks += k_step;
            vs += v_step;
          }
        } else {
#pragma unroll
          for (int r = 0; r < TOKENS; r += kRows) {
            const bool in = has >> (r + copy_row) & 1;
            copy_row_of(dst + r * PITCH, in ? ks : k, in ? vs : v, in);
            ks += k_step;
            vs += v_step;
          }
        }
      } else {
#pragma unroll
        for (int r = 0; r < TOKENS; r += kRows) {
          const int64_t pg = __shfl_sync(~0u, page, r + copy_row), sl = __shfl_sync(~0u, slot, r + copy_row);
          const bool in = has >> (r + copy_row) & 1;
          copy_row_of(dst + r * PITCH, in ? k + pg * p.k_st[0] + sl * p.k_st[1] : k,
                      in ? v + pg * p.v_st[0] + sl * p.v_st[1] : v, in);
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
