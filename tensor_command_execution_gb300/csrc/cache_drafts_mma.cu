// cache_drafts_mma.cu - attention of drafted tokens over a paged cache of
// 16-bit numbers on the warp-level tensor instructions: for heads of more than
// 128 dims (cache_drafts_tc.cu has no form for them), for rows that are not whole
// 16-byte vectors, and for few queries in short tables (cmd_attention_drafts says
// which). cache_drafts_tc.cu has the others.
//
// A tile of 64 tokens lies in shared memory, keys and values, the next one on
// its way; a warp has 16 query rows by some of the tile's tokens, its scores and
// its output in registers, and the online softmax of its rows; warps of the same
// rows are joined at a segment's end. Weights are sums of two 16-bit numbers, as
// in cache_attend_mma.cu. Bound by latency: 24 rows of 16 drafts of up to 374
// tokens, 112 query heads on 16 kv heads of 192 dims take 130 us (its bytes 9),
// with 8 warps on an SM, whose registers are full.
#include "cache_attend_ring.cuh"
#include "cache_drafts.cuh"
#include "cache_mma.cuh"

#ifndef CMDX_COPY
#error "cache_drafts_mma.cu is compiled for each copy size, with -DCMDX_COPY=<16|4|0>"
#endif

namespace cmdx {

namespace {

constexpr int kTile = 64;  // tokens of a tile

// Query rows come in MT tiles of 16, one for each MT-th warp; where there are
// fewer of those than warps, the others take other tokens of a tile. (Wide heads
// leave room for one CTA on an SM: it has eight warps rather than four.)
template <int DP, int MT>
struct Shape {
  static constexpr int kWarps = DP == 256 && MT > 1 ? 8 : 4, kThreads = 32 * kWarps;
  static constexpr int kRows = 16 * MT;
  static constexpr int kSets = kWarps / MT;        // warps that hold states of the same rows
  static constexpr int kMine = kTile / kSets;      // tokens of a warp
  static constexpr int kChunk = kMine < 32 ? kMine : 32;
  static constexpr int kPitch = DP * 2 + 16;       // bytes of a row: an odd number of 16
  static constexpr int kKeys = kTile * kPitch;
  static constexpr int kStage = 2 * kKeys;
  static constexpr int kQueries = 2 * kStage;      // where they lie
  static constexpr int kRest = kQueries + kRows * kPitch;
  static constexpr int kSmem = kRest + (int)(2 * sizeof(DraftTile<kTile>) + sizeof(DraftTree) + sizeof(AttendRows));
  static constexpr int kStatePitch = attend_pitch(DP);
  static constexpr bool kTeams = kWarps == 4;      // (a team's part needs room beside the states)
  static_assert((kSets + (kTeams ? 1 : 0)) * kRows * kStatePitch * 4 <= 2 * kStage, "the states fit the stages");
  static constexpr int kCtas = kSmem <= 113 * 1024 ? 2 : 1;  // of an SM
};

// The rows of a tile (keys only, or keys and values) into a stage, elements
// past the head dim up to a multiple of 16 as zeros, as the rows of tokens
// that have no page.
template <class T, int DP, int kThreads, bool VALUES>
__device__ __forceinline__ void copy_tile(const DraftParams& p, const DraftTile<kTile>& tile, unsigned char* stage, int steps) {
  constexpr int kPitch = DP * 2 + 16, kKeys = kTile * kPitch;
  const T* k = static_cast<const T*>(p.k);
  const T* v = static_cast<const T*>(p.v);
  if constexpr (CMDX_COPY != 0) {
    constexpr int kEach = CMDX_COPY / 2, kChunks = DP / kEach, kOver = kThreads / kChunks;
    const int chunk = threadIdx.x % kChunks, pieces = p.dim / kEach;
    if (chunk * kEach < steps * 16) {
      const int e = chunk < pieces ? chunk * kEach : 0;
      const uint32_t dst = smem_addr(stage) + chunk * CMDX_COPY;
#pragma unroll 8
      for (int r = threadIdx.x / kChunks; r < kTile; r += kOver) {
        const int64_t ks = tile.k[r], vs = tile.v[r];
        const int bytes = ks >= 0 && chunk < pieces ? CMDX_COPY : 0;
        copy_bytes<CMDX_COPY>(dst + r * kPitch, k + (ks >= 0 ? ks : 0) + e, bytes);
        if (VALUES) copy_bytes<CMDX_COPY>(dst + r * kPitch + kKeys, v + (ks >= 0 ? vs : 0) + e, bytes);
      }
    }
  } else {
    for (int i = threadIdx.x; i < kTile * steps * 16; i += kThreads) {
      const int r = i / (steps * 16), e = i - r * steps * 16;
      const bool in = tile.k[r] >= 0 && e < p.dim;
      *reinterpret_cast<T*>(stage + r * kPitch + 2 * e) = in ? k[tile.k[r] + e] : from_float<T>(0.0f);
      if (VALUES) *reinterpret_cast<T*>(stage + kKeys + r * kPitch + 2 * e) = in ? v[tile.v[r] + e] : from_float<T>(0.0f);
    }
  }
  copy_commit();
}

// Query rows [q0, q0 + n) of a kv head, zeros past them and past the head dim.
template <class T, int DP, int kThreads, int ROWS>
__device__ __forceinline__ void load_queries(const DraftParams& p, unsigned char* to, int row, int kv, int q0, int n, int steps) {
  constexpr int kPitch = DP * 2 + 16, kAtOnce = 4;
  const int pieces = steps * 2;  // of 8 numbers
#pragma unroll 1
  for (int i0 = threadIdx.x; i0 < ROWS * pieces; i0 += kThreads * kAtOnce) {
    uint4 x[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int i = i0 + k * kThreads, r = i / pieces, d = 8 * (i - r * pieces);
      x[k] = make_uint4(0, 0, 0, 0);
      if (r < n && d < p.dim) {
        const T* q = draft_query<T>(p, row, kv, q0 + r) + d;
        if (p.q_vectors && p.dim % 8 == 0) {
          x[k] = *reinterpret_cast<const uint4*>(q);
        } else {
          T e[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) e[j] = d + j < p.dim ? q[j] : from_float<T>(0.0f);
          x[k] = *reinterpret_cast<uint4*>(e);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int i = i0 + k * kThreads, r = i / pieces;
      if (r < ROWS) *reinterpret_cast<uint4*>(to + r * kPitch + 16 * (i - r * pieces)) = x[k];
    }
  }
}

// Scores (dot products) of 16 query rows and N tokens.
template <class T, int DP, int N>
__device__ __forceinline__ void scores(float (&s)[N / 8][4], uint32_t queries, uint32_t keys, int steps) {
#pragma unroll
  for (int j = 0; j < N / 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[j][e] = 0.0f;
#pragma unroll
  for (int k = 0; k < DP / 16; ++k) {
    if (k < steps) {
      uint32_t a[4];
      load4(a, queries + k * 32);
#pragma unroll
      for (int j = 0; j < N / 8; j += 2) {
        uint32_t b[4];
        load4(b, keys + j * 8 * (DP * 2 + 16) + k * 32);
        mma<T>(s[j], a, b[0], b[1]);
        mma<T>(s[j + 1], a, b[2], b[3]);
      }
    }
  }
}

template <class T>
constexpr uint32_t kExponent = 0x7f807f80u;
template <>
constexpr uint32_t kExponent<__half> = 0x7c007c00u;
// The parts of x (two numbers of type T) that are infinite or NaN, as a mask.
template <class T>
__device__ __forceinline__ uint32_t not_finite(uint32_t x) {
  constexpr uint32_t lo = kExponent<T> & 0xffffu, hi = kExponent<T> & 0xffff0000u;
  return ((x & lo) == lo ? 0xffffu : 0u) | ((x & hi) == hi ? 0xffff0000u : 0u);
}

template <class T, int DP, int MT>
__global__ void __launch_bounds__((Shape<DP, MT>::kThreads), (Shape<DP, MT>::kCtas)) drafts_mma_kernel(const __grid_constant__ DraftParams p) {
  using S = Shape<DP, MT>;
  constexpr int KS = DP / 16, NC = S::kChunk / 8, kThreads = S::kThreads;
  extern __shared__ __align__(16) unsigned char s_mem[];
  DraftTile<kTile>* s_tile = reinterpret_cast<DraftTile<kTile>*>(s_mem + S::kRest);
  DraftTree& s_tree = *reinterpret_cast<DraftTree*>(s_tile + 2);
  AttendRows& s_rows = *reinterpret_cast<AttendRows*>(&s_tree + 1);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rows_of = warp % MT, set = warp / MT;
  const int gr = lane >> 2, tc = (lane & 3) * 2;
  const int steps = (p.dim + 15) / 16;
  const uint32_t queries = smem_addr(s_mem) + S::kQueries + (rows_of * 16 + (lane & 15)) * S::kPitch + (lane >> 4) * 16;
  const uint32_t key_at = smem_addr(s_mem) + (set * S::kMine + (lane & 7) + (lane >> 4) * 8) * S::kPitch + ((lane >> 3) & 1) * 16;
  const uint32_t value_at = smem_addr(s_mem) + S::kKeys + (set * S::kMine + (lane & 15)) * S::kPitch + (lane >> 4) * 16;

  wait_for_previous();
  let_next_start();
  AttendShare share;
  AttendSegment g;
  if (S::kTeams && p.team) {
    g = attend_team(p, kTile, &share);
  } else {
    if (!attend_begin<T>(p, s_rows, kTile, &share)) return;
    g = attend_first(p, s_rows, share, kTile);
  }
  for (; (S::kTeams && p.team) || g.tiles; g = attend_next(p, s_rows, share, g, kTile)) {
    const AttendHeads heads = attend_heads(p, g.group);
    const int q0 = heads.head0 - heads.kv * p.group, base = g.n - p.drafts;
    if (g.tiles) {  // (none: a team's CTA that has none of a short row)
      draft_place(p, s_tile[0], draft_look(p, g, g.tile0, kTile, true), heads.kv);
      draft_place(p, s_tile[1], draft_look(p, g, g.tile0 + 1, kTile, g.tiles > 1), heads.kv);
      load_queries<T, DP, kThreads, S::kRows>(p, s_mem + S::kQueries, g.row, heads.kv, q0, heads.heads, steps);
      draft_tree<kThreads>(p, s_tree, g.row, base);  // (with barriers: the tiles' places are complete)
      copy_tile<T, DP, kThreads, true>(p, s_tile[0], s_mem, steps);
    }

    // this thread's two query rows
    int draft[2];
    bool live[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = rows_of * 16 + gr + 8 * e;
      draft[e] = (int)fast_div32(p.per, (uint32_t)(q0 + min(r, heads.heads - 1)));
      live[e] = g.tiles && r < heads.heads && s_tree.from[draft[e]] != kNever;
    }
    float o[KS][2][4], m[2] = {-CUDART_INF_F, -CUDART_INF_F}, l[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[k][0][e] = o[k][1][e] = 0.0f;

    for (int i = 0; i < g.tiles; ++i) {
      const int buffer = i & 1;
      if (i + 1 < g.tiles) copy_tile<T, DP, kThreads, true>(p, s_tile[buffer ^ 1], s_mem + (buffer ^ 1) * S::kStage, steps);
      const DraftLook look = draft_look(p, g, g.tile0 + i + 2, kTile, i + 2 < g.tiles);
      if (i + 1 < g.tiles) copy_wait<1>();
      else copy_wait<0>();
      // (before the barrier: draft_place writes them anew below)
      const uint32_t here0 = s_tile[buffer].here[0], here1 = s_tile[buffer].here[1];
      __syncthreads();
      const int t0 = (g.tile0 + i) * kTile;
      const bool masked = (here0 & here1) != ~0u || !draft_all_seen(p, t0, t0 + kTile, base);
      bool infinite = false;  // a value that a masked weight of zero would turn to NaN
      if (masked) {
        bool found = false;
        constexpr int kEach = kThreads / kTile;  // threads to a row
        const unsigned char* v = s_mem + buffer * S::kStage + S::kKeys + threadIdx.x / kEach * S::kPitch;
#pragma unroll 4
        for (int j = threadIdx.x % kEach; j < 2 * steps; j += kEach) {
          const uint4 x = *reinterpret_cast<const uint4*>(v + 16 * j);
          found |= (not_finite<T>(x.x) | not_finite<T>(x.y) | not_finite<T>(x.z) | not_finite<T>(x.w)) != 0;
        }
        infinite = __syncthreads_or(found);
      }
#pragma unroll 1
      for (int c = 0; c < S::kMine; c += S::kChunk) {
        const uint32_t at = buffer * S::kStage + c * S::kPitch;
        const int first = set * S::kMine + c;  // of the chunk, in the tile
        float s[NC][4];
        scores<T, DP, S::kChunk>(s, queries, key_at + at, steps);
        const uint32_t here = first < 32 ? here0 >> first : here1 >> (first - 32);
        float up[2] = {m[0], m[1]};
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int t = 8 * j + tc + (e & 1);
            float x = attend_score(p, s[j][e]);
            if (masked && !((here >> t & 1) && s_tree.sees(p, draft[e >> 1], t0 + first + t, base))) x = -CUDART_INF_F;
            s[j][e] = x;
            up[e >> 1] = fmaxf(up[e >> 1], x);
          }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          up[e] = fmaxf(up[e], __shfl_xor_sync(~0u, up[e], 1));
          up[e] = fmaxf(up[e], __shfl_xor_sync(~0u, up[e], 2));
        }
        if (__any_sync(~0u, up[0] != m[0] || up[1] != m[1])) {
          const float c0 = attend_weight(m[0], up[0]), c1 = attend_weight(m[1], up[1]);
          l[0] *= c0;
          l[1] *= c1;
#pragma unroll
          for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              o[k][b][0] *= c0;
              o[k][b][1] *= c0;
              o[k][b][2] *= c1;
              o[k][b][3] *= c1;
            }
          m[0] = up[0];
          m[1] = up[1];
        }
        uint32_t hi[NC][2], lo[NC][2];
#pragma unroll
        for (int j = 0; j < NC; ++j) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = s[j][e] == -CUDART_INF_F ? 0.0f : power_of_two(s[j][e] - m[e >> 1]);
            l[e >> 1] += x;
            s[j][e] = x;
          }
          split<T>(s[j][0] * kLift<T>, s[j][1] * kLift<T>, &hi[j][0], &lo[j][0]);
          split<T>(s[j][2] * kLift<T>, s[j][3] * kLift<T>, &hi[j][1], &lo[j][1]);
        }
#pragma unroll
        for (int j = 0; j < NC; j += 2) {
          const uint32_t ah[4] = {hi[j][0], hi[j][1], hi[j + 1][0], hi[j + 1][1]};
          const uint32_t al[4] = {lo[j][0], lo[j][1], lo[j + 1][0], lo[j + 1][1]};
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            if (k < steps) {
              uint32_t b[4];
              load4_transposed(b, value_at + at + j * 8 * S::kPitch + k * 32);
              if (infinite) {
#pragma unroll
                for (int e = 0; e < 4; ++e) b[e] &= ~not_finite<T>(b[e]);
              }
              mma<T>(o[k][0], ah, b[0], b[1]);
              mma<T>(o[k][1], ah, b[2], b[3]);
              mma<T>(o[k][0], al, b[0], b[1]);
              mma<T>(o[k][1], al, b[2], b[3]);
            }
          }
        }
        if (infinite) {
          // what was left out above, for the rows that see it
          const unsigned char* v = s_mem + S::kKeys + at + set * S::kMine * S::kPitch;
          for (int t = 0; t < S::kChunk; ++t) {
            bool sees[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) sees[e] = (here >> t & 1) && s_tree.sees(p, draft[e], t0 + first + t, base);
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                if (k < steps) {
                  const uint32_t x = *reinterpret_cast<const uint32_t*>(v + t * S::kPitch + 2 * (16 * k + 8 * b + tc));
                  const uint32_t bad = not_finite<T>(x);
                  const T* y = reinterpret_cast<const T*>(&x);
#pragma unroll
                  for (int e = 0; e < 4; ++e)
                    if (sees[e >> 1] && (bad >> (16 * (e & 1)) & 1)) o[k][b][e] += to_float(y[e & 1]);
                }
              }
          }
        }
      }
      draft_place(p, s_tile[buffer], look, heads.kv);
      __syncthreads();
    }

    // the states into the stages, which are copied to again only after attend_finish
    float* state = reinterpret_cast<float*>(s_mem) + (set * S::kRows + rows_of * 16) * S::kStatePitch;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(~0u, l[e], 1);
      l[e] += __shfl_xor_sync(~0u, l[e], 2);
      float* x = state + (gr + 8 * e) * S::kStatePitch;
      if (tc == 0) {
        x[S::kStatePitch - 4] = live[e] ? m[e] : -CUDART_INF_F;
        x[S::kStatePitch - 3] = live[e] ? l[e] : 0.0f;
      }
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float2 y = make_float2(o[k][b][2 * e] * (1.0f / kLift<T>), o[k][b][2 * e + 1] * (1.0f / kLift<T>));
          if (!live[e]) y = make_float2(0.0f, 0.0f);
          *reinterpret_cast<float2*>(x + 16 * k + 8 * b + tc) = y;
        }
    }
    if (S::kTeams && p.team) {
      attend_finish_team<T, S::kSets, kThreads>(p, g, heads, reinterpret_cast<float*>(s_mem), S::kRows * S::kStatePitch, S::kStatePitch,
                                                reinterpret_cast<float*>(s_mem) + S::kSets * S::kRows * S::kStatePitch);
      return;
    }
    attend_finish<T, S::kSets, kThreads>(p, share, g, heads, reinterpret_cast<float*>(s_mem), S::kRows * S::kStatePitch,
                                         S::kStatePitch);
  }
}

// The weights of every token, added to what p.weights holds, from the maxima
// and sums that the attention has kept: each tile's scores are worked out
// again, and one CTA sums a tile over all of its query rows in their order.
template <class T, int DP, int MT>
__global__ void __launch_bounds__((Shape<DP, MT>::kThreads), 2) weigh_mma_kernel(const __grid_constant__ DraftParams p) {
  using S = Shape<DP, MT>;
  constexpr int NC = S::kMine / 8, kThreads = S::kThreads;
  extern __shared__ __align__(16) unsigned char s_mem[];
  // (two stages of keys alone)
  constexpr int kQueries = 2 * S::kKeys, kRest = kQueries + S::kRows * S::kPitch;
  DraftTile<kTile>* s_tile = reinterpret_cast<DraftTile<kTile>*>(s_mem + kRest);
  DraftTree& s_tree = *reinterpret_cast<DraftTree*>(s_tile + 2);
  AttendRows& s_rows = *reinterpret_cast<AttendRows*>(&s_tree + 1);
  __shared__ float s_sum[MT][kTile];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rows_of = warp % MT, set = warp / MT;
  const int gr = lane >> 2, tc = (lane & 3) * 2;
  const int steps = (p.dim + 15) / 16;
  const uint32_t queries = smem_addr(s_mem) + kQueries + (rows_of * 16 + (lane & 15)) * S::kPitch + (lane >> 4) * 16;
  const uint32_t key_at = smem_addr(s_mem) + (set * S::kMine + (lane & 7) + (lane >> 4) * 8) * S::kPitch + ((lane >> 3) & 1) * 16;

  wait_for_previous();
  let_next_start();
  attend_rows(p, s_rows, kTile);
  const AttendShare share = attend_share(p, s_rows);
  if (share.begin == share.end) return;
  for (AttendSegment g = attend_first(p, s_rows, share, kTile); g.tiles; g = attend_next(p, s_rows, share, g, kTile)) {
    const int kv = g.group, base = g.n - p.drafts;
    const float2* stats = p.stats + ((int64_t)g.row * p.kv_heads + kv) * p.group;
    float* weights = p.weights + g.row * p.w_st[0] + kv * p.w_st[1];
    draft_place(p, s_tile[0], draft_look(p, g, g.tile0, kTile, true), kv);
    draft_place(p, s_tile[1], draft_look(p, g, g.tile0 + 1, kTile, g.tiles > 1), kv);
    draft_tree<kThreads>(p, s_tree, g.row, base);  // (with barriers: the tiles' places are complete)
    copy_tile<T, DP, kThreads, false>(p, s_tile[0], s_mem, steps);
    for (int i = 0; i < g.tiles; ++i) {
      const int buffer = i & 1;
      if (i + 1 < g.tiles) copy_tile<T, DP, kThreads, false>(p, s_tile[buffer ^ 1], s_mem + (buffer ^ 1) * S::kKeys, steps);
      const DraftLook look = draft_look(p, g, g.tile0 + i + 2, kTile, i + 2 < g.tiles);
      if (i + 1 < g.tiles) copy_wait<1>();
      else copy_wait<0>();
      const int t0 = (g.tile0 + i) * kTile;
      const bool mine = threadIdx.x < kTile && s_tile[buffer].k[threadIdx.x] >= 0;
      const float before = mine ? weights[t0 + threadIdx.x] : 0.0f;  // (on its way while the scores are worked out)
      float sum[NC][2];
#pragma unroll
      for (int j = 0; j < NC; ++j) sum[j][0] = sum[j][1] = 0.0f;
      for (int q0 = 0; q0 < p.group; q0 += S::kRows) {
        const int n = min(S::kRows, p.group - q0);
        if (i == 0 || p.group > S::kRows) {  // (one block stays where it is)
          __syncthreads();
          load_queries<T, DP, kThreads, S::kRows>(p, s_mem + kQueries, g.row, kv, q0, n, steps);
        }
        __syncthreads();
        int draft[2];
        float top[2], r[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int q = rows_of * 16 + gr + 8 * e;
          const float2 x = q < n ? stats[q0 + q] : make_float2(0.0f, 0.0f);
          draft[e] = (int)fast_div32(p.per, (uint32_t)(q0 + min(q, n - 1)));
          top[e] = x.x;
          r[e] = x.y == 0.0f ? 0.0f : 1.0f / x.y;
        }
        const uint32_t here0 = s_tile[buffer].here[0], here1 = s_tile[buffer].here[1];
        const bool masked = (here0 & here1) != ~0u || !draft_all_seen(p, t0, t0 + kTile, base);
        const int first = set * S::kMine;
        const uint64_t here = (((uint64_t)here1 << 32) | here0) >> first;
        float s[NC][4];
        scores<T, DP, S::kMine>(s, queries, key_at + buffer * S::kKeys, steps);
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int t = 8 * j + tc + (e & 1);
            const bool seen = !masked || ((here >> t & 1) && s_tree.sees(p, draft[e >> 1], t0 + first + t, base));
            const float x = attend_score(p, s[j][e]);
            if (seen && r[e >> 1] != 0.0f && x != -CUDART_INF_F) sum[j][e & 1] += power_of_two(x - top[e >> 1]) * r[e >> 1];
          }
      }
#pragma unroll
      for (int j = 0; j < NC; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int b = 4; b < 32; b <<= 1) sum[j][e] += __shfl_xor_sync(~0u, sum[j][e], b);
          if (gr == 0) s_sum[rows_of][set * S::kMine + 8 * j + tc + e] = sum[j][e];
        }
      __syncthreads();  // (the tile is read, and the sums are complete)
      if (mine) {
        float x = s_sum[0][threadIdx.x];
#pragma unroll
        for (int j = 1; j < MT; ++j) x += s_sum[j][threadIdx.x];
        weights[t0 + threadIdx.x] = before + x;
      }
      __syncwarp();
      draft_place(p, s_tile[buffer], look, kv);
      __syncthreads();
    }
  }
}

template <class T, int DP, int MT>
cudaError_t launch(const DraftParams& p, cudaStream_t stream) {
  using S = Shape<DP, MT>;
  static PerDevice ready;  // (static storage: zero before first use)
  const cudaError_t e = allow_smem(drafts_mma_kernel<T, DP, MT>, S::kSmem, ready);
  if (e != cudaSuccess) return e;
  return attend_launch<T>(drafts_mma_kernel<T, DP, MT>, p, 2, 152 * S::kCtas, S::kThreads, S::kSmem, kTile, stream, S::kTeams);
}
template <class T, int DP, int MT>
cudaError_t weigh(DraftParams p, cudaStream_t stream) {
  p.blocks = 1;
  p.start_units = 2;
  const int ctas = attend_sides(p.kv_heads, 152 * 2, &p.sides);
  constexpr int smem = Shape<DP, MT>::kSmem - 2 * Shape<DP, MT>::kKeys;
  static PerDevice ready;  // (static storage: zero before first use)
  const cudaError_t e = allow_smem(weigh_mma_kernel<T, DP, MT>, smem, ready);
  if (e != cudaSuccess) return e;
  return launch_chained(weigh_mma_kernel<T, DP, MT>, ctas, Shape<DP, MT>::kThreads, (size_t)smem, stream, p);
}

template <class T, int DP>
cudaError_t by_rows(bool weights, const DraftParams& p, cudaStream_t stream) {
  const int rows = weights ? p.group : p.block_heads;
  if (rows <= 16) return weights ? weigh<T, DP, 1>(p, stream) : launch<T, DP, 1>(p, stream);
  constexpr int two = CMDX_COPY == 16 ? 2 : 4;
  if (rows <= 16 * two) return weights ? weigh<T, DP, two>(p, stream) : launch<T, DP, two>(p, stream);
  return weights ? weigh<T, DP, 4>(p, stream) : launch<T, DP, 4>(p, stream);
}
template <class T>
cudaError_t by_dim(bool weights, const DraftParams& p, cudaStream_t stream) {
  if (p.dim <= 64) return by_rows<T, 64>(weights, p, stream);
  return p.dim <= 128 ? by_rows<T, 128>(weights, p, stream) : by_rows<T, 256>(weights, p, stream);
}

}  // namespace

cudaError_t CMDX_COPY_NAME(drafts_mma_launch)(int dtype, const DraftParams& p, cudaStream_t stream) {
  return dtype == CMD_F16 ? by_dim<__half>(false, p, stream) : by_dim<__nv_bfloat16>(false, p, stream);
}
cudaError_t CMDX_COPY_NAME(weigh_mma_launch)(int dtype, const DraftParams& p, cudaStream_t stream) {
  return dtype == CMD_F16 ? by_dim<__half>(true, p, stream) : by_dim<__nv_bfloat16>(true, p, stream);
}

}  // namespace cmdx
