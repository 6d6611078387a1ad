// cache_attend_f32.cu - attention of one new token per sequence over a paged
// cache of 32-bit numbers whose rows are whole 16-byte vectors.
//
// Products and sums stay in binary32 (the tensor units' 32-bit type holds 11
// bits of a factor). Bound by memory up to about 8 query heads to a kv head:
// each pair of elements takes 2 multiply-adds a query head, and the SM's 128
// lanes do 128 in the cycle that brings 24 bytes. Each warp streams tiles of
// 8 tokens through a ring of its own; scores are computed with a lane to a
// quarter of a token's key (rows are an odd number of 16 bytes apart, so 8
// tokens are read without bank conflicts), weighted values with a lane to 4
// elements of the head dim (dims up to 64: the half-warps take every other
// token). Queries and weights are read from shared memory as broadcasts.
#include "cache_attend_ring.cuh"

namespace cmdx {

namespace {

constexpr int kTokens = 8;  // of a warp's tile
constexpr int kWarps = 4;

// Stages of each warp's ring, and CTAs of an SM, for heads of up to DP dims
// and blocks of up to GT query heads.
template <int DP, int GT>
struct Shape {
  static constexpr int kStages = DP == 64 ? 3 : 2;
  static constexpr int kCtas = DP == 256 ? 1 : DP == 64 ? 3 : GT == 8 ? 2 : 3;
  static constexpr int kPitch = DP * 4 + 16;  // bytes of a row: an odd number of 16
  using Ring = AttendRing<float, kTokens, DP / 4, kPitch, kStages, kWarps>;
  static constexpr int kQueries = GT * DP * 4;              // bytes of a block's queries
  static constexpr int kWeights = kWarps * kTokens * GT * 4;  // and of the warps' weights
  static constexpr int kSmem = kWarps * Ring::kBytes + kQueries + kWeights + (int)sizeof(AttendRows);
};

template <int DP, int GT>
__global__ void __launch_bounds__(kWarps * 32, Shape<DP, GT>::kCtas) attend_f32_kernel(const __grid_constant__ AttendParams p) {
  using S = Shape<DP, GT>;
  using Ring = typename S::Ring;
  constexpr int kHeld = GT > 4 ? GT / 4 : 1;           // heads whose softmax a lane keeps
  constexpr int kQuads = DP > 128 ? DP / 128 : 1;      // groups of 4 dims of a lane
  constexpr int kApart = DP == 64 ? 2 : 1;             // tokens taken at once by the warp's halves
  extern __shared__ __align__(16) unsigned char s_mem[];
  float* s_q = reinterpret_cast<float*>(s_mem + kWarps * Ring::kBytes);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* s_w = s_q + GT * DP + warp * kTokens * GT;    // [token][head]
  AttendRows& s_rows = *reinterpret_cast<AttendRows*>(s_mem + kWarps * Ring::kBytes + S::kQueries + S::kWeights);
  const int token = lane & 7, part = lane >> 3;        // in the scores
  const int quad = DP == 64 ? lane & 15 : lane, half = DP == 64 ? lane >> 4 : 0;  // in the values

  pdl_wait();
  pdl_trigger();
  AttendShare share;
  if (!attend_begin<float>(p, s_rows, Ring::kTile, &share)) return;
  AttendSegment g = attend_first(p, s_rows, share, Ring::kTile);
  Ring ring(p, s_rows, share, g, s_mem + warp * Ring::kBytes);
  for (; g.tiles; g = attend_next(p, s_rows, share, g, Ring::kTile)) {
    const AttendHeads heads = attend_heads(p, g.group);
    for (int i = threadIdx.x; i < GT * DP; i += kWarps * 32) {
      const int h = i / DP, d = i % DP;
      s_q[i] = h < heads.heads && d < p.dim
                   ? static_cast<const float*>(p.q)[g.row * p.q_st[0] + (heads.head0 + h) * p.q_st[1] + d]
                   : 0.0f;
    }
    __syncthreads();

    // the softmax of head part + 4 i lies with lanes of that part (one query
    // head: with all lanes); o of this lane's dims
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
      float s[GT];
#pragma unroll
      for (int h = 0; h < GT; ++h) s[h] = 0.0f;
#pragma unroll 4
      for (int c = 0; c < DP / 16; ++c) {
        if (16 * c >= p.dim) break;
        const float4 x = *reinterpret_cast<const float4*>(keys + token * S::kPitch + (4 * c + part) * 16);
#pragma unroll
        for (int h = 0; h < GT; ++h) {
          const float4 q = *reinterpret_cast<const float4*>(s_q + h * DP + (4 * c + part) * 4);
          s[h] = fmaf(x.x, q.x, s[h]);
          s[h] = fmaf(x.y, q.y, s[h]);
          s[h] = fmaf(x.z, q.z, s[h]);
          s[h] = fmaf(x.w, q.w, s[h]);
        }
      }
#pragma unroll
      for (int h = 0; h < GT; ++h) {
        s[h] += __shfl_xor_sync(~0u, s[h], 8);
        s[h] += __shfl_xor_sync(~0u, s[h], 16);
      }
      const bool in = here >> token & 1;
      float c[kHeld];
      bool moved = false;
#pragma unroll
      for (int j = 0; j < kHeld; ++j) {
        float x = s[0];
#pragma unroll
        for (int h = 0; h < GT; ++h)
          if (GT > 1 && h / 4 == j) x = part == h % 4 ? s[h] : x;
        x = in ? attend_score(p, x) : -CUDART_INF_F;
        float up = x;
#pragma unroll
        for (int b = 1; b < 8; b <<= 1) up = fmaxf(up, __shfl_xor_sync(~0u, up, b));
        up = fmaxf(up, m[j]);
        c[j] = m[j] == -CUDART_INF_F ? 0.0f : power_of_two(m[j] - up);
        moved = moved || up != m[j];
        m[j] = up;
        const float w = x == -CUDART_INF_F ? 0.0f : power_of_two(x - up);
        l[j] = fmaf(l[j], c[j], w);
        if (GT > 1 || part == 0) s_w[token * GT + (GT > 1 ? part + 4 * j : 0)] = w;
      }
      if (__any_sync(~0u, moved)) {
#pragma unroll
        for (int h = 0; h < GT; ++h) {
          const float ch = __shfl_sync(~0u, c[h / 4], (h % 4) * 8);
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
    // with the next tile
    unsigned char* states = s_mem + ring.free_stage() * Ring::kStage;
    float* state = reinterpret_cast<float*>(states + warp * Ring::kBytes);
    constexpr int kStatePitch = attend_pitch(DP);
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
#pragma unroll
      for (int b = 1; b < 8; b <<= 1) l[j] += __shfl_xor_sync(~0u, l[j], b);
      if (token == 0 && (GT > 1 || part == 0)) {
        float* x = state + (GT > 1 ? part + 4 * j : 0) * kStatePitch;
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
    attend_finish<float, kWarps>(p, share, g, heads, reinterpret_cast<float*>(states), Ring::kBytes / 4, kStatePitch);
  }
}

template <int DP, int GT>
cudaError_t launch(const AttendParams& p, cudaStream_t stream) {
  using S = Shape<DP, GT>;
  static_assert(GT * attend_pitch(DP) * 4 <= S::Ring::kStage, "a warp's state fits a stage");
  static DeviceCache ready;  // (static storage: zero before first use)
  const cudaError_t e = allow_smem(attend_f32_kernel<DP, GT>, S::kSmem, ready);
  if (e != cudaSuccess) return e;
  return attend_launch<float>(attend_f32_kernel<DP, GT>, p, 2, 152 * S::kCtas, kWarps * 32, S::kSmem, S::Ring::kTile, stream);
}

template <int DP>
cudaError_t launch_dim(const AttendParams& p, cudaStream_t stream) {
  if (p.block_heads == 1) return launch<DP, 1>(p, stream);
  return p.block_heads <= 4 ? launch<DP, 4>(p, stream) : launch<DP, 8>(p, stream);
}

}  // namespace

cudaError_t attend_f32_launch(const AttendParams& p, cudaStream_t stream) {
  if (p.dim <= 64) return launch_dim<64>(p, stream);
  return p.dim <= 128 ? launch_dim<128>(p, stream) : launch_dim<256>(p, stream);
}

}  // namespace cmdx
