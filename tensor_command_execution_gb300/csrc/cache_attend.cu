// cache_attend.cu - attention of one new token per sequence over a paged
// cache of 16-bit numbers whose rows are not whole 4-byte words (an odd head
// dim, base or stride): what cache_attend_mma.cu, which copies rows in pieces,
// cannot take.
//
// out = sum_t exp(s_t - lse) v_t, s_t = scale q . k_t, one pass over the
// tokens with a running maximum. A warp takes kStep tokens at a time, a lane
// VEC elements of the head dim, straight from memory to registers; the kStep *
// GT dot products (GT query heads) are summed over the lanes by a transposing
// butterfly that leaves each lane one finished score (31 shuffles for 32
// scores rather than 5 each), where scaling, the cap, the mask and the
// exponential are then done once. Bound by the latency of its loads, element
// by element: 64 rows of 4096 tokens of 8 kv heads of 101 (bf16) 568 us with one
// query head each, 22% of the copy peak, 1116 with eight, which is what an odd
// head dim costs (2060 with each token's page looked up where it is read).
#include "cache_attend.cuh"

namespace cmdx {

namespace {

constexpr int kWarps = 8;
constexpr int kTokens = 16;  // of a warp's tile
constexpr int kRowsBytes = (sizeof(AttendRows) + 15) / 16 * 16;

// VEC elements of a row for this lane (element 32 i + lane), zero past dim.
template <class T, int VEC>
__device__ __forceinline__ void load_row(float (&x)[VEC], const T* row, int lane, int dim) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const int e = 32 * i + lane;
    x[i] = e < dim ? to_float(row[e]) : 0.0f;
  }
}

template <class T, int GT, int VEC>
__global__ void __launch_bounds__(kWarps * 32) attend_simt_kernel(const __grid_constant__ AttendParams p) {
  constexpr int kStep = VEC == 8 && GT == 8 ? 2 : 4;  // tokens at once
  constexpr int NV = kStep * GT;
  constexpr int kDup = 32 / NV;  // lanes that end up with the same score
  constexpr int kPitch = attend_pitch(32 * VEC);
  extern __shared__ __align__(16) unsigned char s_mem[];
  AttendRows& s_rows = *reinterpret_cast<AttendRows*>(s_mem);
  float(*s_state)[GT][kPitch] = reinterpret_cast<float(*)[GT][kPitch]>(s_mem + kRowsBytes);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int tile = kTokens * kWarps;
  wait_for_previous();
  let_next_start();
  AttendShare share;
  if (!attend_begin<T>(p, s_rows, tile, &share)) return;
  const T* kp = static_cast<const T*>(p.k);
  const T* vp = static_cast<const T*>(p.v);
  for (AttendSegment g = attend_first(p, s_rows, share, tile); g.tiles; g = attend_next(p, s_rows, share, g, tile)) {
    const AttendHeads heads = attend_heads(p, g.group);
    float q[GT][VEC], o[GT][VEC];
#pragma unroll
    for (int h = 0; h < GT; ++h) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) q[h][i] = o[h][i] = 0.0f;
      if (h < heads.heads) {
        const T* row = static_cast<const T*>(p.q) + g.row * p.q_st[0] + (heads.head0 + h) * p.q_st[1];
        load_row<T, VEC>(q[h], row, lane, p.dim);
      }
    }
    // this lane's score is that of token lane / kDup / GT and head lane / kDup % GT of a step
    const int my_token = lane / kDup / GT;
    float m = -CUDART_INF_F, l = 0.0f;
    // the page and slot of this lane's token of a tile (lane % 16), read a tile ahead
    const int32_t* table = p.tables + g.row * p.table_st[0];
    int page = 0, slot = 0;
    bool inside = false;
    const auto look_up = [&](int i) {
      const int token = (g.tile0 + i) * tile + warp * kTokens + lane % kTokens;
      inside = i < g.tiles && token >= g.lo && token < g.n;
      const uint32_t column = fast_div32(p.page, (uint32_t)token);
      slot = token - (int)(column * p.page.d);
      if (inside) page = table[column * p.table_st[1]];
    };
    look_up(0);
    for (int i = 0; i < g.tiles; ++i) {
      if (inside && (page < 0 || page >= p.n_pages)) {
        report(p.status, CMD_CACHE_BAD_PAGE);
        inside = false;
      }
      const uint32_t has = __ballot_sync(~0u, inside) & ((1u << kTokens) - 1u);
      const int page_here = inside ? page : 0, slot_here = inside ? slot : 0;
      look_up(i + 1);
      for (int t = 0; t < kTokens; t += kStep) {
        if ((has >> t & ((1u << kStep) - 1u)) == 0) continue;
        float k[kStep][VEC], v[kStep][VEC];
        bool seen[kStep];
#pragma unroll
        for (int j = 0; j < kStep; ++j) {
          seen[j] = has >> (t + j) & 1;
          // (a token outside reads nothing: every element is past a dim of 0)
          const int64_t pg = __shfl_sync(~0u, page_here, t + j), sl = __shfl_sync(~0u, slot_here, t + j);
          const int dim = seen[j] ? p.dim : 0;
          load_row<T, VEC>(k[j], kp + pg * p.k_st[0] + sl * p.k_st[1] + heads.kv * p.k_st[2], lane, dim);
          load_row<T, VEC>(v[j], vp + pg * p.v_st[0] + sl * p.v_st[1] + heads.kv * p.v_st[2], lane, dim);
        }
        float s[NV];
#pragma unroll
        for (int j = 0; j < kStep; ++j)
#pragma unroll
          for (int h = 0; h < GT; ++h) {
            float x = q[h][0] * k[j][0];
#pragma unroll
            for (int e = 1; e < VEC; ++e) x = fmaf(q[h][e], k[j][e], x);
            s[j * GT + h] = x;
          }
        // after each round a lane keeps half of its sums, the upper half
        // where its bit of the round is set
        int n = NV;
#pragma unroll
        for (int b = 16; b > 0; b >>= 1) {
          if (n > 1) {
            n >>= 1;
            const bool upper = lane & b;
#pragma unroll
            for (int e = 0; e < NV / 2; ++e)
              if (e < n) {
                const float give = upper ? s[e] : s[e + n], keep = upper ? s[e + n] : s[e];
                s[e] = keep + __shfl_xor_sync(~0u, give, b);
              }
          } else {
            s[0] += __shfl_xor_sync(~0u, s[0], b);
          }
        }
        bool mine = seen[0];
#pragma unroll
        for (int j = 1; j < kStep; ++j) mine = my_token == j ? seen[j] : mine;
        const float score = mine ? attend_score(p, s[0]) : -CUDART_INF_F;
        float top = score;  // over the step's tokens: the lane bits above a head's
#pragma unroll
        for (int b = kDup * GT; b < 32; b <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, b));
        const float up = fmaxf(m, top);
        if (__any_sync(~0u, up != m)) {
          const float c = m == -CUDART_INF_F ? 0.0f : exp2f(m - up);
          l *= c;
          m = up;
#pragma unroll
          for (int h = 0; h < GT; ++h) {
            const float ch = __shfl_sync(~0u, c, h * kDup);
#pragma unroll
            for (int e = 0; e < VEC; ++e) o[h][e] *= ch;
          }
        }
        const float w = score == -CUDART_INF_F ? 0.0f : exp2f(score - m);
        l += w;
#pragma unroll
        for (int j = 0; j < kStep; ++j)
#pragma unroll
          for (int h = 0; h < GT; ++h) {
            const float x = __shfl_sync(~0u, w, (j * GT + h) * kDup);
#pragma unroll
            for (int e = 0; e < VEC; ++e) o[h][e] = fmaf(x, v[j][e], o[h][e]);
          }
      }
    }
#pragma unroll
    for (int b = kDup * GT; b < 32; b <<= 1) l += __shfl_xor_sync(~0u, l, b);
#pragma unroll
    for (int h = 0; h < GT; ++h) {
      if (lane == h * kDup) {
        s_state[warp][h][kPitch - 4] = m;
        s_state[warp][h][kPitch - 3] = l;
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) s_state[warp][h][32 * e + lane] = o[h][e];
    }
    attend_finish<T, kWarps>(p, share, g, heads, &s_state[0][0][0], GT * kPitch, kPitch);
  }
}

template <class T, int GT, int VEC>
cudaError_t launch(const AttendParams& p, cudaStream_t stream) {
  constexpr int smem = kRowsBytes + kWarps * GT * attend_pitch(32 * VEC) * (int)sizeof(float);
  static PerDevice ready;  // (static storage: zero before first use)
  const cudaError_t e = allow_smem(attend_simt_kernel<T, GT, VEC>, smem, ready);
  if (e != cudaSuccess) return e;
  return attend_launch<T>(attend_simt_kernel<T, GT, VEC>, p, 0, 2 * 152, kWarps * 32, smem, kTokens * kWarps, stream,
                          false);
}

template <class T, int GT>
cudaError_t launch_dim(const AttendParams& p, cudaStream_t stream) {
  if (p.dim <= 64) return launch<T, GT, 2>(p, stream);
  return p.dim <= 128 ? launch<T, GT, 4>(p, stream) : launch<T, GT, 8>(p, stream);
}

template <class T>
cudaError_t launch_type(const AttendParams& p, cudaStream_t stream) {
  return p.block_heads == 1 ? launch_dim<T, 1>(p, stream) : launch_dim<T, 8>(p, stream);
}

}  // namespace

cudaError_t attend_simt_launch(int dtype, const AttendParams& p, cudaStream_t stream) {
  switch (dtype) {
    case CMD_F16: return launch_type<__half>(p, stream);
    case CMD_BF16: return launch_type<__nv_bfloat16>(p, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace cmdx
