// cache_drafts_f32.cu - attention of drafted tokens over a paged cache of
// 32-bit numbers.
//
// A thread holds R query rows by 2 tokens of the scores, and R rows by 4 dims
// (and every 64th further) of the output; 16 threads share a row, and the two
// halves of a warp 2 R rows, so that a row's maximum, sum and weights stay in
// its warp. Products are binary32 multiply-adds: the tensor units take 32-bit
// numbers at three products of 11 bits each, which is no more than the
// multiply-adds' rate at the warp level.
#include "cache_attend_ring.cuh"
#include "cache_drafts.cuh"

#ifndef CMDX_COPY
#error "cache_drafts_f32.cu is compiled for each copy size, with -DCMDX_COPY=<16|4>"
#endif

namespace cmdx {

namespace {

constexpr int kThreads = 128;
constexpr int kTile = 32;  // tokens of a tile

template <int DP, int R>
struct Shape {
  static constexpr int kRows = 8 * R;
  static constexpr int kPitch = DP + 4;            // floats of a row: 16-byte vectors of 8 rows meet no bank twice
  static constexpr int kKeys = kTile * kPitch;     // floats
  static constexpr int kStage = 2 * kKeys;
  static constexpr int kQueries = 2 * kStage;
  static constexpr int kWeights = kQueries + kRows * kPitch;
  static constexpr int kWeightPitch = kTile + 4;
  static constexpr int kRest = (kWeights + kRows * kWeightPitch) * 4;  // bytes
  static constexpr int kSmem = kRest + (int)(2 * sizeof(DraftTile<kTile>) + sizeof(DraftTree) + sizeof(AttendRows));
  static constexpr int kStatePitch = attend_pitch(DP);
  static_assert(kRows * kStatePitch <= 2 * kStage, "the states fit the stages");
  static constexpr int kCtas = kSmem <= 113 * 1024 ? 2 : 1;  // of an SM
};

template <int DP, bool VALUES>
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

template <int DP, int ROWS>
__device__ __forceinline__ void load_queries(const DraftParams& p, float* to, int row, int kv, int q0, int n, int steps) {
  for (int i = threadIdx.x; i < ROWS * steps * 4; i += kThreads) {
    const int r = i / (steps * 4), d = i - r * steps * 4;
    to[r * (DP + 4) + d] = r < n && d < p.dim ? draft_query<float>(p, row, kv, q0 + r)[d] : 0.0f;
  }
}

// Dot products of this thread's R rows with tokens tx and tx + 16 of a tile.
template <int DP, int R>
__device__ __forceinline__ void scores(float (&s)[R][2], const float* queries, const float* keys, int steps) {
  constexpr int kPitch = DP + 4;
#pragma unroll
  for (int r = 0; r < R; ++r) s[r][0] = s[r][1] = 0.0f;
#pragma unroll 4
  for (int k = 0; k < steps; ++k) {
    const float4 a = *reinterpret_cast<const float4*>(keys + 4 * k);
    const float4 b = *reinterpret_cast<const float4*>(keys + 16 * kPitch + 4 * k);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float4 q = *reinterpret_cast<const float4*>(queries + r * kPitch + 4 * k);
      s[r][0] = fmaf(q.x, a.x, fmaf(q.y, a.y, fmaf(q.z, a.z, fmaf(q.w, a.w, s[r][0]))));
      s[r][1] = fmaf(q.x, b.x, fmaf(q.y, b.y, fmaf(q.z, b.z, fmaf(q.w, b.w, s[r][1]))));
    }
  }
}

template <int DP, int R>
__global__ void __launch_bounds__(kThreads, (Shape<DP, R>::kCtas)) drafts_f32_kernel(const __grid_constant__ DraftParams p) {
  using S = Shape<DP, R>;
  constexpr int NJ = DP / 64;
  extern __shared__ __align__(16) float s_mem[];
  DraftTile<kTile>* s_tile = reinterpret_cast<DraftTile<kTile>*>(reinterpret_cast<unsigned char*>(s_mem) + S::kRest);
  DraftTree& s_tree = *reinterpret_cast<DraftTree*>(s_tile + 2);
  AttendRows& s_rows = *reinterpret_cast<AttendRows*>(&s_tree + 1);
  const int tx = threadIdx.x & 15, r0 = (threadIdx.x >> 4) * R, steps = (p.dim + 3) / 4;
  const float* queries = s_mem + S::kQueries + r0 * S::kPitch;
  float* my_weights = s_mem + S::kWeights + r0 * S::kWeightPitch;

  wait_for_previous();
  let_next_start();
  AttendShare share;
  if (!attend_begin<float>(p, s_rows, kTile, &share)) return;
  for (AttendSegment g = attend_first(p, s_rows, share, kTile); g.tiles; g = attend_next(p, s_rows, share, g, kTile)) {
    const AttendHeads heads = attend_heads(p, g.group);
    const int q0 = heads.head0 - heads.kv * p.group, base = g.n - p.drafts;
    draft_place(p, s_tile[0], draft_look(p, g, g.tile0, kTile, true), heads.kv);
    draft_place(p, s_tile[1], draft_look(p, g, g.tile0 + 1, kTile, g.tiles > 1), heads.kv);
    load_queries<DP, S::kRows>(p, s_mem + S::kQueries, g.row, heads.kv, q0, heads.heads, steps);
    draft_tree<kThreads>(p, s_tree, g.row, base);  // (with barriers: the tiles' places are complete)
    copy_tile<DP, true>(p, s_tile[0], s_mem, steps);

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
      if (i + 1 < g.tiles) copy_tile<DP, true>(p, s_tile[buffer ^ 1], s_mem + (buffer ^ 1) * S::kStage, steps);
      const DraftLook look = draft_look(p, g, g.tile0 + i + 2, kTile, i + 2 < g.tiles);
      if (i + 1 < g.tiles) copy_wait<1>();
      else copy_wait<0>();
      __syncthreads();
      const int t0 = (g.tile0 + i) * kTile;
      const uint32_t here = s_tile[buffer].here[0];
      const bool masked = here != ~0u || !draft_all_seen(p, t0, t0 + kTile, base);
      const float* stage = s_mem + buffer * S::kStage;
      float s[R][2];
      scores<DP, R>(s, queries, stage + tx * S::kPitch, steps);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float up = m[r];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int t = tx + 16 * e;
          float x = attend_score(p, s[r][e]);
          if (masked && !((here >> t & 1) && s_tree.sees(p, draft[r], t0 + t, base))) x = -CUDART_INF_F;
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
        for (int e = 0; e < 2; ++e) {
          const float w = s[r][e] == -CUDART_INF_F ? 0.0f : exp2f(s[r][e] - m[r]);
          l[r] += w;
          my_weights[r * S::kWeightPitch + tx + 16 * e] = w;
        }
      }
      __syncwarp();
      const float* values = stage + S::kKeys + 4 * tx;
#pragma unroll 1
      for (int t = 0; t < kTile; t += 4) {
        float w[R][4];
#pragma unroll
        for (int r = 0; r < R; ++r) *reinterpret_cast<float4*>(w[r]) = *reinterpret_cast<const float4*>(my_weights + r * S::kWeightPitch + t);
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            if (4 * tx + 64 * j < p.dim) {
              const float4 v = *reinterpret_cast<const float4*>(values + (t + e) * S::kPitch + 64 * j);
#pragma unroll
              for (int r = 0; r < R; ++r) {
                if (masked && w[r][e] == 0.0f) continue;  // (whatever an unseen token holds)
                o[r][j][0] = fmaf(w[r][e], v.x, o[r][j][0]);
                o[r][j][1] = fmaf(w[r][e], v.y, o[r][j][1]);
                o[r][j][2] = fmaf(w[r][e], v.z, o[r][j][2]);
                o[r][j][3] = fmaf(w[r][e], v.w, o[r][j][3]);
              }
            }
          }
      }
      draft_place(p, s_tile[buffer], look, heads.kv);
      __syncthreads();
    }

    // the states into the stages, which are copied to again only after attend_finish
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int b = 1; b < 16; b <<= 1) l[r] += __shfl_xor_sync(~0u, l[r], b);
      const bool live = r0 + r < heads.heads && s_tree.from[draft[r]] != kNever;
      float* x = s_mem + (r0 + r) * S::kStatePitch;
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
    attend_finish<float, 1, kThreads>(p, share, g, heads, s_mem, 0, S::kStatePitch);
  }
}

// The weights of every token (see cache_drafts_mma.cu).
template <int DP, int R>
__global__ void __launch_bounds__(kThreads, 2) weigh_f32_kernel(const __grid_constant__ DraftParams p) {
  using S = Shape<DP, R>;
  extern __shared__ __align__(16) float s_mem[];
  constexpr int kQueries = 2 * S::kKeys, kRest = (kQueries + S::kRows * S::kPitch) * 4;  // (two stages of keys alone)
  DraftTile<kTile>* s_tile = reinterpret_cast<DraftTile<kTile>*>(reinterpret_cast<unsigned char*>(s_mem) + kRest);
  DraftTree& s_tree = *reinterpret_cast<DraftTree*>(s_tile + 2);
  AttendRows& s_rows = *reinterpret_cast<AttendRows*>(&s_tree + 1);
  __shared__ float s_sum[kThreads / 32][kTile];
  const int tx = threadIdx.x & 15, r0 = (threadIdx.x >> 4) * R, steps = (p.dim + 3) / 4;

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
    copy_tile<DP, false>(p, s_tile[0], s_mem, steps);
    for (int i = 0; i < g.tiles; ++i) {
      const int buffer = i & 1;
      if (i + 1 < g.tiles) copy_tile<DP, false>(p, s_tile[buffer ^ 1], s_mem + (buffer ^ 1) * S::kKeys, steps);
      const DraftLook look = draft_look(p, g, g.tile0 + i + 2, kTile, i + 2 < g.tiles);
      if (i + 1 < g.tiles) copy_wait<1>();
      else copy_wait<0>();
      const int t0 = (g.tile0 + i) * kTile;
      float sum[2] = {0.0f, 0.0f};
      for (int q0 = 0; q0 < p.group; q0 += S::kRows) {
        const int n = min(S::kRows, p.group - q0);
        if (i == 0 || p.group > S::kRows) {  // (one block stays where it is)
          __syncthreads();
          load_queries<DP, S::kRows>(p, s_mem + kQueries, g.row, kv, q0, n, steps);
        }
        __syncthreads();
        const uint32_t here = s_tile[buffer].here[0];
        const bool masked = here != ~0u || !draft_all_seen(p, t0, t0 + kTile, base);
        float s[R][2];
        scores<DP, R>(s, s_mem + kQueries + r0 * S::kPitch, s_mem + buffer * S::kKeys + tx * S::kPitch, steps);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float2 x = r0 + r < n ? stats[q0 + r0 + r] : make_float2(0.0f, 0.0f);
          const float w = x.y == 0.0f ? 0.0f : 1.0f / x.y;
          const int draft = (int)fast_div32(p.per, (uint32_t)(q0 + min(r0 + r, n - 1)));
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int t = tx + 16 * e;
            const bool seen = !masked || ((here >> t & 1) && s_tree.sees(p, draft, t0 + t, base));
            const float y = attend_score(p, s[r][e]);
            if (seen && w != 0.0f && y != -CUDART_INF_F) sum[e] += exp2f(y - x.x) * w;
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        sum[e] += __shfl_xor_sync(~0u, sum[e], 16);
        if ((threadIdx.x & 16) == 0) s_sum[threadIdx.x >> 5][tx + 16 * e] = sum[e];
      }
      __syncthreads();  // (the tile is read, and the sums are complete)
      if (threadIdx.x < kTile && s_tile[buffer].k[threadIdx.x] >= 0) {
        float x = s_sum[0][threadIdx.x];
#pragma unroll
        for (int j = 1; j < kThreads / 32; ++j) x += s_sum[j][threadIdx.x];
        weights[t0 + threadIdx.x] += x;
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
    return attend_launch<float>(drafts_f32_kernel<DP, R>, p, 2, 152 * S::kCtas, kThreads, S::kSmem, kTile, stream, false);
  }
  p.blocks = p.sides = 1;
  p.start_units = 0;
  constexpr int smem = (2 * S::kKeys + S::kRows * S::kPitch) * 4 + (S::kSmem - S::kRest);
  const cudaError_t e = allow_smem(weigh_f32_kernel<DP, R>, smem, weigh_ready);
  if (e != cudaSuccess) return e;
  return launch_chained(weigh_f32_kernel<DP, R>, 152 * 2, kThreads, (size_t)smem, stream, p);
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
