// cache_attend_f32.cu - attention of one new token per sequence over a paged
// cache of 32-bit numbers.
//
// Products and sums stay in binary32 (the tensor units' 32-bit type holds 11
// bits of a factor). Bound by memory for few query heads to a kv head. Each
// warp streams tiles of 8 tokens through a ring of its own. Scores: a lane
// takes an eighth of the head dim of two tokens' keys, so that a query read
// (shared by all lanes of the eighth) serves both, and the sums over the eight
// lanes go by a transposing butterfly that leaves each lane a few finished
// scores. Weighted values: a lane takes 4 elements of the head dim (dims up to
// 64: the half-warps take every other token), the weights being read back from
// shared memory. Rows lie 32 bytes past a multiple of 128 apart: the lanes of
// 4 tokens and 2 neighbouring pieces meet in no bank.
//
// Measured: 24 rows of 2999 tokens, 16 kv heads of 128, one query head each
// 174 us, 6.80 TB/s, the copy peak; 8 query heads to each of 2 kv heads, 96 rows,
// 105 us, 83%, with no unit full (multiply-adds 36%, shared memory 46%, issue
// slots 55%): its 168 registers leave two CTAs of four warps on an SM, too few to
// cover a tile's dependent steps; 12 query heads, in two blocks that each copy
// the cache, 198 us, 44%; 24 rows of 1 to 1100 tokens (16 heads of 80, capped,
// windowed) 19.6 us, 50%, 6 of it the fixed part of two launches.
#include "cache_attend_ring.cuh"

#ifndef CMDX_COPY
#error "cache_attend_f32.cu is compiled for each copy size, with -DCMDX_COPY=<16|4>"
#endif

namespace cmdx {

namespace {

constexpr int kTokens = 8;  // of a warp's tile
constexpr int kWarps = 4;

// Stages of each warp's ring, and CTAs of an SM, for heads of up to DP dims
// and blocks of up to GT query heads.
template <int DP, int GT>
struct Shape {
  static constexpr int kStages = DP == 64 ? 3 : 2;
  static constexpr int kCtas = DP == 256 ? 1 : DP == 64 || GT < 8 ? 3 : 2;
  static constexpr int kPitch = DP * 4 + 32;  // bytes of a row
  using Ring = AttendRing<float, DP, CMDX_COPY, kTokens, kPitch, kStages, kWarps>;
  static constexpr int kQueries = GT * DP * 4;              // bytes of a block's queries
  static constexpr int kWeights = kWarps * kTokens * GT * 4;  // and of the warps' weights
  static constexpr int kSmem = kWarps * Ring::kBytes + kQueries + kWeights + (int)sizeof(AttendRows);
};

template <int DP, int GT>
__global__ void __launch_bounds__(kWarps * 32, Shape<DP, GT>::kCtas)
    attend_f32_kernel(const __grid_constant__ AttendParams p) {
  using S = Shape<DP, GT>;
  using Ring = typename S::Ring;
  constexpr int kScores = 2 * GT;                      // of a lane's two tokens
  constexpr int kHeld = GT > 4 ? GT / 4 : 1;           // finished scores (and heads) of a lane
  constexpr int kQuads = DP > 128 ? DP / 128 : 1;      // groups of 4 dims of a lane
  constexpr int kApart = DP == 64 ? 2 : 1;             // tokens taken at once by the warp's halves
  extern __shared__ __align__(16) unsigned char s_mem[];
  float* s_q = reinterpret_cast<float*>(s_mem + kWarps * Ring::kBytes);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* s_w = s_q + GT * DP + warp * kTokens * GT;    // [token][head]
  AttendRows& s_rows = *reinterpret_cast<AttendRows*>(s_mem + kWarps * Ring::kBytes + S::kQueries + S::kWeights);
  // in the scores: tokens token and token + 4, eighth `part`; finished scores
  // are of token `done` and heads held, held + 1
  const int token = lane & 3, part = lane >> 2;
  const int done = token + (part & 4), held = GT == 1 ? 0 : (part & 3) * kHeld;

  const int quad = DP == 64 ? lane & 15 : lane, half = DP == 64 ? lane >> 4 : 0;  // in the values

  wait_for_previous();
  let_next_start();
  AttendShare share;
  AttendSegment g;
  if (p.team) {
    g = attend_team(p, Ring::kTile, &share);
  } else {
    if (!attend_begin<float>(p, s_rows, Ring::kTile, &share)) return;
    g = attend_first(p, s_rows, share, Ring::kTile);
  }
  Ring ring(p, s_rows, share, g, s_mem + warp * Ring::kBytes);
  for (; p.team || g.tiles; g = attend_next(p, s_rows, share, g, Ring::kTile)) {
    const AttendHeads heads = attend_heads(p, g.group);
    for (int i = threadIdx.x; i < GT * DP; i += kWarps * 32) {
      const int h = i / DP, d = i % DP;
      s_q[i] = h < heads.heads && d < p.dim
                   ? static_cast<const float*>(p.q)[g.row * p.q_st[0] + (heads.head0 + h) * p.q_st[1] + d]
                   : 0.0f;
    }
    __syncthreads();

    // the softmax of heads held + i, and o of this lane's dims
    float m[kHeld], l[kHeld];
    float4 o[GT][kQuads];
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      m[i] = -CUDART_INF_F;
      l[i] = 0.0f;
    }
#pragma unroll
    for (int h = 0; h < GT; ++h)
#pragma unroll
      for (int c = 0; c < kQuads; ++c) o[h][c] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);

    for (int i = 0; i < g.tiles; ++i) {
      int index;
      const uint32_t here = ring.next_tile(&index);
      if (!here) continue;
      const unsigned char* keys = s_mem + warp * Ring::kBytes + index * Ring::kStage;
      float s[kScores];
#pragma unroll
      for (int h = 0; h < kScores; ++h) s[h] = 0.0f;
#pragma unroll
      for (int c = 0; c < DP / 32; ++c) {
        if (32 * c >= p.dim) break;
        const float4 x = *reinterpret_cast<const float4*>(keys + token * S::kPitch + (8 * c + part) * 16);
        const float4 y = *reinterpret_cast<const float4*>(keys + (token + 4) * S::kPitch + (8 * c + part) * 16);
#pragma unroll
        for (int h = 0; h < GT; ++h) {
          const float4 q = *reinterpret_cast<const float4*>(s_q + h * DP + (8 * c + part) * 4);
          s[h] = fmaf(x.x, q.x, s[h]);
          s[h] = fmaf(x.y, q.y, s[h]);
          s[h] = fmaf(x.z, q.z, s[h]);
          s[h] = fmaf(x.w, q.w, s[h]);
          s[GT + h] = fmaf(y.x, q.x, s[GT + h]);
          s[GT + h] = fmaf(y.y, q.y, s[GT + h]);
          s[GT + h] = fmaf(y.z, q.z, s[GT + h]);
          s[GT + h] = fmaf(y.w, q.w, s[GT + h]);
        }
      }
      // over the eight lanes of a token: after each round a lane keeps half of
      // its sums, the upper half where its bit of the round is set
#pragma unroll
      for (int b = 16, n = kScores; b >= 4; b >>= 1) {
        if (n > 1) {
          n >>= 1;
          const bool upper = lane & b;
#pragma unroll
          for (int e = 0; e < kScores / 2; ++e)
            if (e < n) {
              const float give = upper ? s[e] : s[e + n], keep = upper ? s[e + n] : s[e];
              s[e] = keep + __shfl_xor_sync(~0u, give, b);
            }
        } else {
          s[0] += __shfl_xor_sync(~0u, s[0], b);
        }
      }
      const bool in = here >> done & 1;
      float c[kHeld];
      bool moved = false;
#pragma unroll
      for (int j = 0; j < kHeld; ++j) {
        const float x = in ? attend_score(p, s[j]) : -CUDART_INF_F;
        float up = fmaxf(x, __shfl_xor_sync(~0u, x, 1));
        up = fmaxf(up, __shfl_xor_sync(~0u, up, 2));
        up = fmaxf(up, __shfl_xor_sync(~0u, up, 16));
        up = fmaxf(up, m[j]);
        c[j] = m[j] == -CUDART_INF_F ? 0.0f : power_of_two(m[j] - up);
        moved = moved || up != m[j];
        m[j] = up;
        const float w = x == -CUDART_INF_F ? 0.0f : power_of_two(x - up);
        l[j] = fmaf(l[j], c[j], w);
        s_w[done * GT + held + j] = w;
      }
      if (__any_sync(~0u, moved)) {
#pragma unroll
        for (int h = 0; h < GT; ++h) {
          const float ch = __shfl_sync(~0u, c[h % kHeld], h / kHeld * 4);
#pragma unroll
          for (int e = 0; e < kQuads; ++e) scale_by(o[h][e], ch);
        }
      }
      __syncwarp();
#pragma unroll
      for (int t = 0; t < kTokens; t += kApart) {
        float w[GT];
        if constexpr (GT % 4 == 0) {
#pragma unroll
          for (int h = 0; h < GT; h += 4)
            *reinterpret_cast<float4*>(w + h) = *reinterpret_cast<const float4*>(s_w + (t + half) * GT + h);
        } else {
#pragma unroll
          for (int h = 0; h < GT; ++h) w[h] = s_w[(t + half) * GT + h];
        }
#pragma unroll
        for (int e = 0; e < kQuads; ++e) {
          const float4 x = *reinterpret_cast<const float4*>(keys + Ring::kKeys + (t + half) * S::kPitch + (quad + 32 * e) * 16);
#pragma unroll
          for (int h = 0; h < GT; ++h) add_scaled(o[h][e], x, w[h]);
        }
      }
      __syncwarp();  // the weights may be overwritten
    }

    // the warp's state into the stage read last, which is copied to again only
    // with the next tile (a team has no next one: its states go to the first
    // stage, and its CTAs' parts to the second of the first warp)
    unsigned char* states = s_mem + (p.team ? 0 : ring.free_stage()) * Ring::kStage;
    float* state = reinterpret_cast<float*>(states + warp * Ring::kBytes);
    constexpr int kStatePitch = attend_pitch(DP);
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      l[j] += __shfl_xor_sync(~0u, l[j], 1);
      l[j] += __shfl_xor_sync(~0u, l[j], 2);
      l[j] += __shfl_xor_sync(~0u, l[j], 16);
      if (done == 0) {
        float* x = state + (held + j) * kStatePitch;
        x[kStatePitch - 4] = m[j];
        x[kStatePitch - 3] = l[j];
      }
    }
#pragma unroll
    for (int h = 0; h < GT; ++h)
#pragma unroll
      for (int e = 0; e < kQuads; ++e) {
        float4 x = o[h][e];
        if constexpr (DP == 64) {
          x.x += __shfl_xor_sync(~0u, x.x, 16);
          x.y += __shfl_xor_sync(~0u, x.y, 16);
          x.z += __shfl_xor_sync(~0u, x.z, 16);
          x.w += __shfl_xor_sync(~0u, x.w, 16);
        }
        if (half == 0) *reinterpret_cast<float4*>(state + h * kStatePitch + (quad + 32 * e) * 4) = x;
      }
    if (p.team) {
      attend_finish_team<float, kWarps>(p, g, heads, reinterpret_cast<float*>(states), Ring::kBytes / 4, kStatePitch,
                                  reinterpret_cast<float*>(s_mem + Ring::kStage));
      break;
    }
    attend_finish<float, kWarps>(p, share, g, heads, reinterpret_cast<float*>(states), Ring::kBytes / 4, kStatePitch);
  }
}

template <int DP, int GT>
cudaError_t launch(const AttendParams& p, cudaStream_t stream) {
  using S = Shape<DP, GT>;
  static_assert(GT * attend_pitch(DP) * 4 <= S::Ring::kStage, "a warp's state fits a stage");
  static PerDevice ready;  // (static storage: zero before first use)
  const cudaError_t e = allow_smem(attend_f32_kernel<DP, GT>, S::kSmem, ready);
  if (e != cudaSuccess) return e;
  // (a row's beginning as two tiles of 32 tokens: 24 short rows of 16 heads took
  // 28.2 us counted as 0, 20.7 as 1, 21.2 as 2; 64 longer ones of 4 heads with 4
  // query heads each 64.5, 48.4 and 42.2)
  return attend_launch<float>(attend_f32_kernel<DP, GT>, p, 2, 152 * S::kCtas, kWarps * 32, S::kSmem, S::Ring::kTile, stream);
}

template <int DP>
cudaError_t launch_dim(const AttendParams& p, cudaStream_t stream) {
  if (p.block_heads == 1) return launch<DP, 1>(p, stream);
  return p.block_heads <= 4 ? launch<DP, 4>(p, stream) : launch<DP, 8>(p, stream);
}

}  // namespace

cudaError_t CMDX_COPY_NAME(attend_f32_launch)(const AttendParams& p, cudaStream_t stream) {
  if (p.dim <= 64) return launch_dim<64>(p, stream);
  return p.dim <= 128 ? launch_dim<128>(p, stream) : launch_dim<256>(p, stream);
}

}  // namespace cmdx
