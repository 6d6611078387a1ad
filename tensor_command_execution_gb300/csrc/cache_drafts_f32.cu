// cache_drafts_f32.cu - attention of drafted tokens over a paged cache of
// 32-bit numbers.
//
// A thread holds R query rows by 2 tokens of the scores, and R rows by 4 dims
// (and every 64th further) of the output; 16 threads share a row, and the two
// halves of a warp 2 R rows, so that a row's maximum, sum and weights stay in
// its warp. Products are binary32 multiply-adds: the tensor units would take a
// 32-bit number as a sum of ones of 11 bits, whose products leave 2^-21 of a
// score, and scores come to weights as powers. 12 rows of 13 drafts, up to 2999
// tokens, window 1100, 16 heads of 80: 33 us of the call's 40 (its bytes: 5.5),
// bound by the latency between a tile's steps (issue slots 44%, 16 warps on an
// SM: registers and stages are full).
#include "cache_attend_ring.cuh"
#include "cache_drafts.cuh"

#ifndef CMDX_COPY
#error "cache_drafts_f32.cu is compiled for each copy size, with -DCMDX_COPY=<16|4>"
#endif

namespace cmdx {

namespace {

constexpr int kTile = 32;  // tokens of a tile

template <int DP, int R>
struct Shape {
  // Few rows to a thread leave much time between its loads and their use: then
  // eight warps share a tile, four with each half of its tokens.
  static constexpr int kSets = R == 2 ? 2 : 1;
  static constexpr int kThreads = 128 * kSets;
  static constexpr int kMine = 2 / kSets;          // tokens of a thread
  static constexpr int kRows = 8 * R;
  static constexpr int kPitch = DP + 4;            // floats of a row: 16-byte vectors of 8 rows meet no bank twice
  static constexpr int kKeys = kTile * kPitch;     // floats
  static constexpr int kStage = 2 * kKeys;
  static constexpr int kQueries = 2 * kStage;
  static constexpr int kWeights = kQueries + kRows * kPitch;
  static constexpr int kWeightPitch = kTile + 4;
  static constexpr int kRest = (kWeights + kRows * kWeightPitch) * 4;  // bytes (the sets' weights side by side)
  static constexpr int kSmem = kRest + (int)(2 * sizeof(DraftTile<kTile>) + sizeof(DraftTree) + sizeof(AttendRows));
  static constexpr int kStatePitch = attend_pitch(DP);
  static_assert((kSets + 1) * kRows * kStatePitch <= 2 * kStage, "the states and a team's part fit the stages");
  static constexpr int kCtas = kSmem <= 113 * 1024 ? 2 : 1;  // of an SM
};

template <int DP, int kThreads, bool VALUES>
__device__ __forceinline__ void copy_tile(const DraftParams& p, const DraftTile<kTile>& tile, float* stage, int steps) {
  constexpr int kPitch = DP + 4, kKeys = kTile * kPitch;
  constexpr int kEach = CMDX_COPY / 4, kChunks = DP / kEach;
  constexpr int kOver = kChunks < kThreads ? kThreads / kChunks : 1, kPieces = kChunks < kThreads ? 1 : kChunks / kThreads;
  const float* k = static_cast<const float*>(p.k);
  const float* v = static_cast<const float*>(p.v);
  const int pieces = p.dim / kEach;
#pragma unroll 4
  for (int r = threadIdx.x / kChunks; r < kTile; r += kOver) {
    const int64_t ks = tile.k[r], vs = tile.v[r];
#pragma unroll
    for (int c = 0; c < kPieces; ++c) {
      const int chunk = threadIdx.x % kChunks + c * kThreads;
      if (chunk * kEach < steps * 4) {
        const int bytes = ks >= 0 && chunk < pieces ? CMDX_COPY : 0, e = chunk < pieces ? chunk * kEach : 0;
        const uint32_t dst = smem_addr(stage + r * kPitch + chunk * kEach);
        copy_bytes<CMDX_COPY>(dst, k + (ks >= 0 ? ks : 0) + e, bytes);
        if (VALUES) copy_bytes<CMDX_COPY>(dst + kKeys * 4, v + (ks >= 0 ? vs : 0) + e, bytes);
      }
    }
  }
  copy_commit();
}

template <int DP, int kThreads, int ROWS>
__device__ __forceinline__ void load_queries(const DraftParams& p, float* to, int row, int kv, int q0, int n, int steps) {
  constexpr int kAtOnce = 8;
#pragma unroll 1
  for (int i0 = threadIdx.x; i0 < ROWS * steps; i0 += kThreads * kAtOnce) {
    float4 x[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int i = i0 + k * kThreads, r = i / steps, d = 4 * (i - r * steps);
      x[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (r < n) {
        const float* q = draft_query<float>(p, row, kv, q0 + r) + d;
        if (p.q_vectors && p.dim % 4 == 0) {
          x[k] = *reinterpret_cast<const float4*>(q);
        } else {
          x[k].x = q[0];
          if (d + 1 < p.dim) x[k].y = q[1];
          if (d + 2 < p.dim) x[k].z = q[2];
          if (d + 3 < p.dim) x[k].w = q[3];
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int i = i0 + k * kThreads, r = i / steps, d = 4 * (i - r * steps);
      if (r < ROWS) *reinterpret_cast<float4*>(to + r * (DP + 4) + d) = x[k];
    }
  }
}

// Dot products of this thread's R rows with N tokens, 16 apart.
template <int DP, int R, int N>
__device__ __forceinline__ void scores(float (&s)[R][N], const float* queries, const float* keys, int steps) {
  constexpr int kPitch = DP + 4;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int e = 0; e < N; ++e) s[r][e] = 0.0f;
#pragma unroll 4
  for (int k = 0; k < steps; ++k) {
    float4 a[N];
#pragma unroll
    for (int e = 0; e < N; ++e) a[e] = *reinterpret_cast<const float4*>(keys + 16 * e * kPitch + 4 * k);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float4 q = *reinterpret_cast<const float4*>(queries + r * kPitch + 4 * k);
#pragma unroll
      for (int e = 0; e < N; ++e) s[r][e] = fmaf(q.x, a[e].x, fmaf(q.y, a[e].y, fmaf(q.z, a[e].z, fmaf(q.w, a[e].w, s[r][e]))));
    }
  }
}

// A tile's values, weighted, to R rows by 4 of every 64 dims (`dims` are left
// from this thread's first). MASKED: a weight of -1 says that the row does not
// see the token, whatever its value (a weight of zero enters: times infinity).
template <int DP, int R, int TOKENS, bool MASKED>
__device__ __forceinline__ void add_values(float (&o)[R][DP / 64][4], const float* weights, const float* values, int dims) {
  constexpr int kPitch = DP + 4, kWeightPitch = kTile + 4;
#pragma unroll 2
  for (int t = 0; t < TOKENS; t += 4) {
    float w[R][4];
#pragma unroll
    for (int r = 0; r < R; ++r) *reinterpret_cast<float4*>(w[r]) = *reinterpret_cast<const float4*>(weights + r * kWeightPitch + t);
#pragma unroll
    for (int j = 0; j < DP / 64; ++j) {
      if (64 * j < dims) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float4 v = *reinterpret_cast<const float4*>(values + (t + e) * kPitch + 64 * j);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const float x = w[r][e];
            const bool none = MASKED && x < 0.0f;
            o[r][j][0] = fmaf(x, none ? 0.0f : v.x, o[r][j][0]);
            o[r][j][1] = fmaf(x, none ? 0.0f : v.y, o[r][j][1]);
            o[r][j][2] = fmaf(x, none ? 0.0f : v.z, o[r][j][2]);
            o[r][j][3] = fmaf(x, none ? 0.0f : v.w, o[r][j][3]);
          }
        }
      }
    }
  }
}

template <int DP, int R>
__global__ void __launch_bounds__((Shape<DP, R>::kThreads), (Shape<DP, R>::kCtas)) drafts_f32_kernel(const __grid_constant__ DraftParams p) {
  using S = Shape<DP, R>;
  constexpr int NJ = DP / 64, N = S::kMine, kThreads = S::kThreads, kTokens = 16 * N;
  extern __shared__ __align__(16) float s_mem[];
  DraftTile<kTile>* s_tile = reinterpret_cast<DraftTile<kTile>*>(reinterpret_cast<unsigned char*>(s_mem) + S::kRest);
  DraftTree& s_tree = *reinterpret_cast<DraftTree*>(s_tile + 2);
  AttendRows& s_rows = *reinterpret_cast<AttendRows*>(&s_tree + 1);
  const int tx = threadIdx.x & 15, r0 = (threadIdx.x >> 4) % 8 * R, set = threadIdx.x / 128, steps = (p.dim + 3) / 4;
  const float* queries = s_mem + S::kQueries + r0 * S::kPitch;
  float* my_weights = s_mem + S::kWeights + r0 * S::kWeightPitch + set * kTokens;

  wait_for_previous();
  let_next_start();
  AttendShare share;
  AttendSegment g;
  if (p.team) {
    g = attend_team(p, kTile, &share);
  } else {
    if (!attend_begin<float>(p, s_rows, kTile, &share)) return;
    g = attend_first(p, s_rows, share, kTile);
  }
  for (; p.team || g.tiles; g = attend_next(p, s_rows, share, g, kTile)) {
    const AttendHeads heads = attend_heads(p, g.group);
    const int q0 = heads.head0 - heads.kv * p.group, base = g.n - p.drafts;
    if (g.tiles) {  // (none: a team's CTA that has none of a short row)
      draft_place(p, s_tile[0], draft_look(p, g, g.tile0, kTile, true), heads.kv);
      draft_place(p, s_tile[1], draft_look(p, g, g.tile0 + 1, kTile, g.tiles > 1), heads.kv);
      load_queries<DP, kThreads, S::kRows>(p, s_mem + S::kQueries, g.row, heads.kv, q0, heads.heads, steps);
      draft_tree<kThreads>(p, s_tree, g.row, base);  // (with barriers: the tiles' places are complete)
      copy_tile<DP, kThreads, true>(p, s_tile[0], s_mem, steps);
    }

    int draft[R];
    float o[R][NJ][4], m[R], l[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      draft[r] = (int)fast_div32(p.per, (uint32_t)(q0 + min(r0 + r, heads.heads - 1)));
      m[r] = -CUDART_INF_F;
      l[r] = 0.0f;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[r][j][e] = 0.0f;
    }

    for (int i = 0; i < g.tiles; ++i) {
      const int buffer = i & 1;
      if (i + 1 < g.tiles) copy_tile<DP, kThreads, true>(p, s_tile[buffer ^ 1], s_mem + (buffer ^ 1) * S::kStage, steps);
      const DraftLook look = draft_look(p, g, g.tile0 + i + 2, kTile, i + 2 < g.tiles);
      if (i + 1 < g.tiles) copy_wait<1>();
      else copy_wait<0>();
      // (before the barrier: draft_place writes it anew below)
      const uint32_t here = s_tile[buffer].here[0];
      __syncthreads();
      const int t0 = (g.tile0 + i) * kTile;
      const bool masked = here != ~0u || !draft_all_seen(p, t0, t0 + kTile, base);
      const float* stage = s_mem + buffer * S::kStage;
      float s[R][N];
      scores<DP, R, N>(s, queries, stage + (set * kTokens + tx) * S::kPitch, steps);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float up = m[r];
        bool hidden[N];
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const int t = set * kTokens + tx + 16 * e;
          float x = attend_score(p, s[r][e]);
          hidden[e] = masked && !((here >> t & 1) && s_tree.sees(p, draft[r], t0 + t, base));
          if (hidden[e]) x = -CUDART_INF_F;
          s[r][e] = x;
          up = fmaxf(up, x);
        }
#pragma unroll
        for (int b = 1; b < 16; b <<= 1) up = fmaxf(up, __shfl_xor_sync(~0u, up, b));
        if (up != m[r]) {
          const float c = attend_weight(m[r], up);
          l[r] *= c;
#pragma unroll
          for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[r][j][e] *= c;
          m[r] = up;
        }
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float w = s[r][e] == -CUDART_INF_F ? 0.0f : exp2f(s[r][e] - m[r]);
          l[r] += w;
          my_weights[r * S::kWeightPitch + tx + 16 * e] = hidden[e] ? -1.0f : w;
        }
      }
      __syncwarp();
      const float* values = stage + S::kKeys + set * kTokens * S::kPitch + 4 * tx;
      if (masked) add_values<DP, R, kTokens, true>(o, my_weights, values, p.dim - 4 * tx);
      else add_values<DP, R, kTokens, false>(o, my_weights, values, p.dim - 4 * tx);
      draft_place(p, s_tile[buffer], look, heads.kv);
      __syncthreads();
    }

    // the states into the stages, which are copied to again only after attend_finish
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int b = 1; b < 16; b <<= 1) l[r] += __shfl_xor_sync(~0u, l[r], b);
      const bool live = g.tiles && r0 + r < heads.heads && s_tree.from[draft[r]] != kNever;
      float* x = s_mem + (set * S::kRows + r0 + r) * S::kStatePitch;
      if (tx == 0) {
        x[S::kStatePitch - 4] = live ? m[r] : -CUDART_INF_F;
        x[S::kStatePitch - 3] = live ? l[r] : 0.0f;
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const float4 y = live ? make_float4(o[r][j][0], o[r][j][1], o[r][j][2], o[r][j][3]) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        *reinterpret_cast<float4*>(x + 4 * tx + 64 * j) = y;
      }
    }
    if (p.team) {
      attend_finish_team<float, S::kSets, kThreads>(p, g, heads, s_mem, S::kRows * S::kStatePitch, S::kStatePitch,
                                                    s_mem + S::kSets * S::kRows * S::kStatePitch);
      return;
    }
    attend_finish<float, S::kSets, kThreads>(p, share, g, heads, s_mem, S::kRows * S::kStatePitch, S::kStatePitch);
  }
}

// The weights of every token (see cache_drafts_mma.cu).
template <int DP, int R>
__global__ void __launch_bounds__((Shape<DP, R>::kThreads), 2) weigh_f32_kernel(const __grid_constant__ DraftParams p) {
  using S = Shape<DP, R>;
  constexpr int N = S::kMine, kThreads = S::kThreads, kTokens = 16 * N;
  extern __shared__ __align__(16) float s_mem[];
  constexpr int kQueries = 2 * S::kKeys, kRest = (kQueries + S::kRows * S::kPitch) * 4;  // (two stages of keys alone)
  DraftTile<kTile>* s_tile = reinterpret_cast<DraftTile<kTile>*>(reinterpret_cast<unsigned char*>(s_mem) + kRest);
  DraftTree& s_tree = *reinterpret_cast<DraftTree*>(s_tile + 2);
  AttendRows& s_rows = *reinterpret_cast<AttendRows*>(&s_tree + 1);
  __shared__ float s_sum[4][kTile];
  const int tx = threadIdx.x & 15, r0 = (threadIdx.x >> 4) % 8 * R, set = threadIdx.x / 128, steps = (p.dim + 3) / 4;

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
    copy_tile<DP, kThreads, false>(p, s_tile[0], s_mem, steps);
    for (int i = 0; i < g.tiles; ++i) {
      const int buffer = i & 1;
      if (i + 1 < g.tiles) copy_tile<DP, kThreads, false>(p, s_tile[buffer ^ 1], s_mem + (buffer ^ 1) * S::kKeys, steps);
      const DraftLook look = draft_look(p, g, g.tile0 + i + 2, kTile, i + 2 < g.tiles);
      if (i + 1 < g.tiles) copy_wait<1>();
      else copy_wait<0>();
      const int t0 = (g.tile0 + i) * kTile;
      const bool mine = threadIdx.x < kTile && s_tile[buffer].k[threadIdx.x] >= 0;
      const float before = mine ? weights[t0 + threadIdx.x] : 0.0f;  // (on its way while the scores are worked out)
      float sum[N] = {};
      for (int q0 = 0; q0 < p.group; q0 += S::kRows) {
        const int n = min(S::kRows, p.group - q0);
        float2 of_row[R];
#pragma unroll
        for (int r = 0; r < R; ++r) of_row[r] = r0 + r < n ? stats[q0 + r0 + r] : make_float2(0.0f, 0.0f);
        if (i == 0 || p.group > S::kRows) {  // (one block stays where it is)
          __syncthreads();
          load_queries<DP, kThreads, S::kRows>(p, s_mem + kQueries, g.row, kv, q0, n, steps);
        }
        __syncthreads();
        const uint32_t here = s_tile[buffer].here[0];
        const bool masked = here != ~0u || !draft_all_seen(p, t0, t0 + kTile, base);
        float s[R][N];
        scores<DP, R, N>(s, s_mem + kQueries + r0 * S::kPitch, s_mem + buffer * S::kKeys + (set * kTokens + tx) * S::kPitch, steps);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float2 x = of_row[r];
          const float w = x.y == 0.0f ? 0.0f : 1.0f / x.y;
          const int draft = (int)fast_div32(p.per, (uint32_t)(q0 + min(r0 + r, n - 1)));
#pragma unroll
          for (int e = 0; e < N; ++e) {
            const int t = set * kTokens + tx + 16 * e;
            const bool seen = !masked || ((here >> t & 1) && s_tree.sees(p, draft, t0 + t, base));
            const float y = attend_score(p, s[r][e]);
            if (seen && w != 0.0f && y != -CUDART_INF_F) sum[e] += exp2f(y - x.x) * w;
          }
        }
      }
#pragma unroll
      for (int e = 0; e < N; ++e) {
        sum[e] += __shfl_xor_sync(~0u, sum[e], 16);
        if ((threadIdx.x & 16) == 0) s_sum[(threadIdx.x >> 5) % 4][set * kTokens + tx + 16 * e] = sum[e];
      }
      __syncthreads();  // (the tile is read, and the sums are complete)
      if (mine) {
        float x = s_sum[0][threadIdx.x];
#pragma unroll
        for (int j = 1; j < 4; ++j) x += s_sum[j][threadIdx.x];
        weights[t0 + threadIdx.x] = before + x;
      }
      __syncwarp();
      draft_place(p, s_tile[buffer], look, kv);
      __syncthreads();
    }
  }
}

template <int DP, int R>
cudaError_t launch(bool weights, DraftParams p, cudaStream_t stream) {
  using S = Shape<DP, R>;
  static PerDevice ready, weigh_ready;  // (static storage: zero before first use)
  if (!weights) {
    const cudaError_t e = allow_smem(drafts_f32_kernel<DP, R>, S::kSmem, ready);
    if (e != cudaSuccess) return e;
    return attend_launch<float>(drafts_f32_kernel<DP, R>, p, 2, 152 * S::kCtas, S::kThreads, S::kSmem, kTile, stream);
  }
  p.blocks = 1;
  p.start_units = 2;
  const int ctas = attend_sides(p.kv_heads, 152 * 2, &p.sides);
  constexpr int smem = (2 * S::kKeys + S::kRows * S::kPitch) * 4 + (S::kSmem - S::kRest);
  const cudaError_t e = allow_smem(weigh_f32_kernel<DP, R>, smem, weigh_ready);
  if (e != cudaSuccess) return e;
  return launch_chained(weigh_f32_kernel<DP, R>, ctas, S::kThreads, (size_t)smem, stream, p);
}

template <int R>
cudaError_t by_dim(bool weights, const DraftParams& p, cudaStream_t stream) {
  if (p.dim <= 64) return launch<64, R>(weights, p, stream);
  return p.dim <= 128 ? launch<128, R>(weights, p, stream) : launch<256, R>(weights, p, stream);
}

}  // namespace

cudaError_t CMDX_COPY_NAME(drafts_f32_launch)(const DraftParams& p, cudaStream_t stream) {
  return p.block_heads <= 16 ? by_dim<2>(false, p, stream) : by_dim<8>(false, p, stream);
}
cudaError_t CMDX_COPY_NAME(weigh_f32_launch)(const DraftParams& p, cudaStream_t stream) {
  return p.group <= 16 ? by_dim<2>(true, p, stream) : by_dim<8>(true, p, stream);
}

}  // namespace cmdx
