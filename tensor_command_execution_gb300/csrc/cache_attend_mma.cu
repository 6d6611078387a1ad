// cache_attend_mma.cu - attention of one new token per sequence over a paged
// cache of 16-bit numbers, on the tensor units.
//
// Scores and weighted values are kept transposed: S^T = K q^T is a product of
// 16 tokens by 16 dims with 16 dims by 8 query heads, O^T = V^T P^T one of 16
// dims by 16 tokens with 16 tokens by 8 heads (mma.sync m16n8k16), so the 16
// wide side is always the cache's and up to 8 query heads that share a kv head
// cost no padding beyond 8. The bound is memory: each key and value crosses
// from HBM once, and 24 such products for 8 KB at dim 128 leave the tensor
// units mostly idle, so the warp-level instruction, whose operands come from
// the registers and shared memory of one warp, serves better here than a
// CTA-wide one: every warp streams tiles of 16 tokens of its own through its
// own ring of shared memory (asynchronous 16-byte copies, rows padded by 16
// bytes against bank conflicts) and keeps its own running maximum, sum and
// O^T, and no barrier is met until a row ends.
//
// A weight p is held as the sum of two 16-bit numbers, hi + lo, multiplied
// apart: rounding p itself to 16 bits would add an error as large as the
// output's own rounding. Together they hold p to 2^-16 of itself (bf16) or
// 2^-22 (f16). binary16 has few exponents for that, and rows can be long: beside
// one token that takes nearly all, 10^5 others of 2^-26 each still add up to
// 2^-9. So an f16 weight is lifted by 2^15 first (the largest, 1, to half of the
// largest number), which leaves an error of 2^-40 of the largest weight at most,
// and o is lowered again when a row ends; the sum l takes p as it is. (Unlifted,
// the output of 8192 tokens beside one e^17.5 times as heavy was 25% off.)
// Tokens outside the row are filled with zeros as they are copied, whatever
// their slots hold.
//
// Measured (8 kv heads of 128, 64 query heads): 64 rows of 4096 tokens 181 us in
// bf16 and in f16, 5.95 TB/s, 87% of the copy peak (the launch alone 177; its
// slowest SM ran 10% longer than the mean); 64 rows of 0 to 8192 tokens 49.3 us,
// 71%; two rows of 393217 and 262147 tokens of 2 kv heads (f16) 115.2 us, 86%; one
// row of 700, 6.7 us, the latency of one launch. Tensor units 13% busy, issue
// slots 26%. Dims 136 to 256 in the kernel of 256: 286 to 350 us, 59 to 90%. Rows
// copied in pieces of 4 bytes: 64 rows of 4096 tokens of dim 100, 241 us, 51%,
// bound by the number of copies.
#include "cache_attend_ring.cuh"
#include "cache_mma.cuh"

#ifndef CMDX_COPY
#error "cache_attend_mma.cu is compiled for each copy size, with -DCMDX_COPY=<16|4>"
#endif

namespace cmdx {

namespace {

constexpr int kTokens = 16;  // of a warp's tile
constexpr int kWarps = 4;

// Stages of each warp's ring, and CTAs of an SM, for heads of up to DP dims.
template <class T, int DP, int NT>
struct Shape {
  static constexpr int kStages = 2;
  static constexpr int kCtas = DP == 256 ? 1 : NT == 2 ? 2 : DP == 64 ? 4 : 3;
  static constexpr int kPitch = DP * 2 + 16;                   // bytes of a row: an odd number of 16
  using Ring = AttendRing<T, DP, CMDX_COPY, kTokens, kPitch, kStages, kWarps>;
  static constexpr int kSmem = kWarps * Ring::kBytes + (int)sizeof(AttendRows);
};

// KEEP: the scores are written to p.scores as well, for the weights that the
// tokens get.
template <class T, int DP, int NT, bool KEEP>
__global__ void __launch_bounds__(kWarps * 32, Shape<T, DP, NT>::kCtas)
    attend_mma_kernel(const __grid_constant__ AttendParams p) {
  using S = Shape<T, DP, NT>;
  using Ring = typename S::Ring;
  constexpr int KS = DP / 16;
  extern __shared__ __align__(16) unsigned char s_mem[];
  AttendRows& s_rows = *reinterpret_cast<AttendRows*>(s_mem + kWarps * Ring::kBytes);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // this lane's row and 16-byte piece in the two kinds of fragment loads; its
  // row gr and columns tc, tc + 1 in an 8 by 8 block
  const uint32_t key_at = (lane & 15) * S::kPitch + (lane >> 4) * 16;
  const uint32_t value_at = ((lane >> 4) * 8 + (lane & 7)) * S::kPitch + ((lane >> 3) & 1) * 16 + Ring::kKeys;
  const int gr = lane >> 2, tc = (lane & 3) * 2;

  wait_for_previous();
  let_next_start();
  AttendShare share;
  AttendSegment g;
  if (p.team) {
    g = attend_team(p, Ring::kTile, &share);
  } else {
    if (!attend_begin<T>(p, s_rows, Ring::kTile, &share)) return;
    g = attend_first(p, s_rows, share, Ring::kTile);
  }
  Ring ring(p, s_rows, share, g, s_mem + warp * Ring::kBytes);
  for (; p.team || g.tiles; g = attend_next(p, s_rows, share, g, Ring::kTile)) {
    const AttendHeads heads = attend_heads(p, g.group);
    // the query heads of this block, as the right side of K q^T
    uint32_t q[NT][KS][2];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int h = j * 8 + gr;
      const T* row = static_cast<const T*>(p.q) + g.row * p.q_st[0] + (heads.head0 + min(h, heads.heads - 1)) * p.q_st[1];
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int d = 16 * s + 8 * b + tc;
          uint32_t x = 0;
          if (h < heads.heads && d < p.dim) {
            if (p.q_pairs) {
              x = *reinterpret_cast<const uint32_t*>(row + d);
            } else {
              T e[2] = {row[d], row[d + 1]};
              x = *reinterpret_cast<uint32_t*>(e);
            }
          }
          q[j][s][b] = x;
        }
    }

    float o[NT][KS][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][s][e] = 0.0f;
      m[j][0] = m[j][1] = -CUDART_INF_F;
      l[j][0] = l[j][1] = 0.0f;
    }

    for (int i = 0; i < g.tiles; ++i) {
      int index;
      const uint32_t here = ring.next_tile(&index);
      if (!here) continue;
      const uint32_t at = ring.at + index * Ring::kStage;
      // scores: tokens gr, gr + 8, heads tc, tc + 1; two chains of products
      float s[NT][2][4];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[j][0][e] = s[j][1][e] = 0.0f;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t a[4];
        load4(a, at + key_at + k * 32);
#pragma unroll
        for (int j = 0; j < NT; ++j) mma<T>(s[j][k & 1], a, q[j][k][0], q[j][k][1]);
      }
      const bool in0 = here >> gr & 1, in1 = here >> (gr + 8) & 1;
      uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[e] = (e < 2 ? in0 : in1) ? attend_score(p, s[j][0][e] + s[j][1][e]) : -CUDART_INF_F;
        if constexpr (KEEP) {
          const int t = (g.tile0 + i) * Ring::kTile + warp * kTokens + gr, h = j * 8 + tc;
          float* to = p.scores + (((int64_t)g.row * p.kv_heads + heads.kv) * p.scores_tokens + t) * p.group + heads.head0 - heads.kv * p.group + h;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if ((e < 2 ? in0 : in1) && h + (e & 1) < heads.heads) to[(e < 2 ? 0 : 8 * p.group) + (e & 1)] = x[e];
        }
        float up[2] = {fmaxf(x[0], x[2]), fmaxf(x[1], x[3])};
#pragma unroll
        for (int b = 4; b < 32; b <<= 1) {
          up[0] = fmaxf(up[0], __shfl_xor_sync(~0u, up[0], b));
          up[1] = fmaxf(up[1], __shfl_xor_sync(~0u, up[1], b));
        }
        up[0] = fmaxf(up[0], m[j][0]);
        up[1] = fmaxf(up[1], m[j][1]);
        if (__any_sync(~0u, up[0] != m[j][0] || up[1] != m[j][1])) {
          const float c0 = m[j][0] == -CUDART_INF_F ? 0.0f : power_of_two(m[j][0] - up[0]);
          const float c1 = m[j][1] == -CUDART_INF_F ? 0.0f : power_of_two(m[j][1] - up[1]);
          l[j][0] *= c0;
          l[j][1] *= c1;
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            o[j][k][0] *= c0;
            o[j][k][1] *= c1;
            o[j][k][2] *= c0;
            o[j][k][3] *= c1;
          }
          m[j][0] = up[0];
          m[j][1] = up[1];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = x[e] == -CUDART_INF_F ? 0.0f : power_of_two(x[e] - m[j][e & 1]);
          l[j][e & 1] += x[e];
        }
        split<T>(x[0] * kLift<T>, x[1] * kLift<T>, &hi[j][0], &lo[j][0]);
        split<T>(x[2] * kLift<T>, x[3] * kLift<T>, &hi[j][1], &lo[j][1]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          hi[j][e] = transposed(hi[j][e]);
          lo[j][e] = transposed(lo[j][e]);
        }
      }
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t a[4];
        load4_transposed(a, at + value_at + k * 32);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          mma<T>(o[j][k], a, hi[j][0], hi[j][1]);
          mma<T>(o[j][k], a, lo[j][0], lo[j][1]);
        }
      }
    }

    // the warp's state into the stage read last, which is copied to again only
    // with the next tile (a team has no next one: its states go to the first
    // stage, and its CTAs' parts to the second of the first warp)
    __syncwarp();
    unsigned char* states = s_mem + (p.team ? 0 : ring.free_stage()) * Ring::kStage;
    float* state = reinterpret_cast<float*>(states + warp * Ring::kBytes);
    constexpr int kStatePitch = attend_pitch(DP);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int b = 4; b < 32; b <<= 1) {
        l[j][0] += __shfl_xor_sync(~0u, l[j][0], b);
        l[j][1] += __shfl_xor_sync(~0u, l[j][1], b);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float* x = state + (j * 8 + tc + e) * kStatePitch;
        if (gr == 0) {
          x[kStatePitch - 4] = m[j][e];
          x[kStatePitch - 3] = l[j][e];
        }
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          x[16 * k + gr] = o[j][k][e] * (1.0f / kLift<T>);
          x[16 * k + gr + 8] = o[j][k][2 + e] * (1.0f / kLift<T>);
        }
      }
    }
    if (p.team) {
      attend_finish_team<T, kWarps>(p, g, heads, reinterpret_cast<float*>(states), Ring::kBytes / 4, kStatePitch,
                                  reinterpret_cast<float*>(s_mem + Ring::kStage));
      break;
    }
    attend_finish<T, kWarps>(p, share, g, heads, reinterpret_cast<float*>(states), Ring::kBytes / 4, kStatePitch);
  }
}

template <class T, int DP, int NT, bool KEEP>
cudaError_t launch_kept(const AttendParams& p, cudaStream_t stream) {
  using S = Shape<T, DP, NT>;
  static_assert(NT * 8 * attend_pitch(DP) * 4 <= S::Ring::kStage, "a warp's state fits a stage");
  static PerDevice ready;  // (static storage: zero before first use)
  const cudaError_t e = allow_smem(attend_mma_kernel<T, DP, NT, KEEP>, S::kSmem, ready);
  if (e != cudaSuccess) return e;
  // The beginning of a row as two tiles of 64 tokens. Measured on 64 rows of 0
  // to 8192 tokens (their logarithms even; bf16, dim 128): counted as 0, 66.6
  // us; 1, 49.9; 2, 48.9; 3, 48.6; with 16 query heads to a kv head 120, 74,
  // 58 and 59. On 64 rows of 4096 tokens it costs nothing beyond the noise.
  return attend_launch<T>(attend_mma_kernel<T, DP, NT, KEEP>, p, 2, 152 * S::kCtas, kWarps * 32, S::kSmem, S::Ring::kTile, stream);
}

template <class T, int DP, int NT>
cudaError_t launch(const AttendParams& p, cudaStream_t stream) {
  if constexpr (CMDX_COPY == 16)
    if (p.scores) return launch_kept<T, DP, NT, true>(p, stream);
  return launch_kept<T, DP, NT, false>(p, stream);
}

template <class T>
cudaError_t launch_type(const AttendParams& p, cudaStream_t stream) {
  const bool two = p.block_heads > 8;
  if (p.dim <= 64) return two ? launch<T, 64, 2>(p, stream) : launch<T, 64, 1>(p, stream);
  if (p.dim <= 128) return two ? launch<T, 128, 2>(p, stream) : launch<T, 128, 1>(p, stream);
  return two ? launch<T, 256, 2>(p, stream) : launch<T, 256, 1>(p, stream);
}

}  // namespace

cudaError_t CMDX_COPY_NAME(attend_mma_launch)(int dtype, const AttendParams& p, cudaStream_t stream) {
  return dtype == CMD_F16 ? launch_type<__half>(p, stream) : launch_type<__nv_bfloat16>(p, stream);
}

}  // namespace cmdx
