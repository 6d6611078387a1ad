// cache_weigh.cu - the weights that one new token's query heads give each token
// of a paged cache, from the scores that the attention has kept.
//
// weights[t] += sum over the heads of exp2(s_t - m) / l: 4 bytes for each score,
// written and read once, where working them out again would read the keys again
// (a decode step of 32 rows to 8192 tokens, 4 query heads to a kv head of 128:
// 50 MB rather than 200: 14 us, where the attention that keeps them takes 70).
// A thread takes a token. Bound by instructions (issue slots 52%) and by the
// rows' and stretches' beginnings.
#include "cache_drafts.cuh"

namespace cmdx {

namespace {

constexpr int kThreads = 256, kEach = 4, kTile = kThreads * kEach;

__global__ void __launch_bounds__(kThreads) weigh_scores_kernel(const __grid_constant__ DraftParams p) {
  constexpr int kHeads = 64;  // of a run: more are gone over in several
  __shared__ AttendRows s_rows;
  __shared__ float2 s_stats[kHeads];  // m, 1 / l
  wait_for_previous();
  let_next_start();
  attend_rows(p, s_rows, kTile);
  const AttendShare share = attend_share(p, s_rows);
  if (share.begin == share.end) return;
  for (AttendSegment g = attend_first(p, s_rows, share, kTile); g.tiles; g = attend_next(p, s_rows, share, g, kTile)) {
    const int64_t list = (int64_t)g.row * p.kv_heads + g.group;
    const float2* stats = p.stats + list * p.group;
    const float* scores = p.scores + list * p.scores_tokens * p.group;
    float* weights = p.weights + g.row * p.w_st[0] + g.group * p.w_st[1];
    const int32_t* table = p.tables + g.row * p.table_st[0];
    for (int h0 = 0; h0 < p.group; h0 += kHeads) {
      const int heads = min(kHeads, p.group - h0);
      __syncthreads();
      if ((int)threadIdx.x < heads) {
        const float2 x = stats[h0 + threadIdx.x];
        s_stats[threadIdx.x] = make_float2(x.x, x.y == 0.0f ? 0.0f : 1.0f / x.y);
      }
      __syncthreads();
      for (int i = 0; i < g.tiles; ++i) {
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
          const int t = (g.tile0 + i) * kTile + k * kThreads + threadIdx.x;
          if (t < g.lo || t >= g.n) continue;
          const int page = table[fast_div32(p.page, (uint32_t)t) * p.table_st[1]];
          if (page < 0 || page >= p.n_pages) continue;  // (reported by the attention; nothing was kept)
          const float* s = scores + (int64_t)t * p.group + h0;
          float sum = 0.0f;
          const auto add = [&](float x, int h) {
            const float2 st = s_stats[h];
            if (st.y != 0.0f && x != -CUDART_INF_F) sum += exp2f(x - st.x) * st.y;
          };
          if (p.group % 4 == 0) {
            for (int h = 0; h < heads; h += 4) {
              const float4 x = *reinterpret_cast<const float4*>(s + h);
              add(x.x, h);
              add(x.y, h + 1);
              add(x.z, h + 2);
              add(x.w, h + 3);
            }
          } else {
            for (int h = 0; h < heads; ++h) add(s[h], h);
          }
          weights[t] += sum;
        }
      }
    }
  }
}

}  // namespace

cudaError_t weigh_scores_launch(const DraftParams& d, cudaStream_t stream) {
  DraftParams p = d;
  p.blocks = p.sides = 1;
  p.start_units = 0;
  return launch_chained(weigh_scores_kernel, 152 * 6, kThreads, 0, stream, p);
}

}  // namespace cmdx
