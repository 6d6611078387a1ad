// cache_weigh_tc.cu - the weights that an attention's queries give each token
// of a paged cache of 16-bit numbers, on the CTA-wide tensor instructions.
//
// weights[t] += sum over the query rows q of a kv head of exp2(s_qt - m_q) / l_q,
// with the maxima m and sums l that the attention has left. The scores are
// worked out again from the keys alone, transposed: 128 tokens by up to 256
// query rows (128 of heads above 128 dims), so that a thread holds all of a token's scores and its sum needs
// no other thread. (Keeping the scores instead would cost 8 bytes for each token
// and query row, more than the keys' 2 dim bytes from dim / 4 rows on.) Two
// groups of four warps take turns, as in cache_drafts_tc.cu. Where a kv head has
// more query rows, so many each are a launch, one after another. No unit
// is full (issue slots 40%, tensor units 14%): a group's loads of scores, its
// exponentials and its turn follow one another, and the slowest CTA counts. Two
// rows of 65536 and 30011 tokens, 32 drafts, 32 query heads on 8 kv heads of 64
// dims: 47 us, for 98 MB of keys 15.
#include <type_traits>

#include "cache_tc.cuh"
#include "cache_attend_ring.cuh"

namespace cmdx {

namespace {

constexpr int kGroup = 128;                // threads of a group, and tokens of a tile
constexpr int kThreads = 2 * kGroup + 64;  // and a warp that issues the products, and one that copies
constexpr int kTile = kTcTile;
static_assert(kTile == kGroup, "a token to a thread");

struct Params : TcParams {
  int32_t row0;  // the first query row of this launch
};

template <int DP>
struct Shape {
  static constexpr int kMostRows = DP == 256 ? 128 : 256;  // of a launch
  static constexpr int kSlot = kTile * DP * 2;
  static constexpr int kSlots = DP == 64 ? 8 : DP == 128 ? 4 : 2;
  static constexpr int kQueries = kMostRows * DP * 2;
  static constexpr int kRest = kQueries + kSlots * kSlot;
};

constexpr int kHereTiles = 16;
struct State {
  uint64_t full[8], empty[8], scores[2], taken[2], queries, end;
  uint32_t tmem;
  uint32_t stop;                    // a wait ran out of time
  uint32_t here[kHereTiles][4];     // which tokens of a tile have a page
  float4 stats[128];                // of two rows: -m, -m, 1 / l, 1 / l
};
template <int DP>
constexpr int kSmem = Shape<DP>::kRest + (int)(sizeof(State) + sizeof(DraftTree) + sizeof(AttendRows)) + 1024;

template <int DP>
__device__ __forceinline__ void copy_keys(const Params& p, State& s, uint32_t ring, const AttendRows& rows, const AttendShare& share) {
  using S = Shape<DP>;
  TmaTiles tiles(p);
  uint32_t issued = 0;
  bool going = true;
  for (AttendSegment g = attend_first(p, rows, share, kTile); g.tiles && going; g = attend_next(p, rows, share, g, kTile)) {
    tiles.begin(g);
    for (int i = 0; i < g.tiles; ++i, ++issued) {
      tiles.look<false>(i);  // (what is wrong has been reported by the attention)
      const uint32_t at = issued % S::kSlots;
      if (!(going = warp_wait(s.stop, smem_u32(&s.empty[at]), (issued / S::kSlots + 1) & 1))) break;
      if (tiles.lane < 4) s.here[issued % kHereTiles][tiles.lane] = tiles.here;
      __syncwarp();
      tiles.copy(p.maps[0], g.group, ring + at * S::kSlot, smem_u32(&s.full[at]));
    }
  }
  for (uint32_t c = issued - min(issued, (uint32_t)S::kSlots); c < issued; ++c)  // (none is on its way when the CTA ends)
    wait_own(s.stop, smem_u32(&s.full[c % S::kSlots]), c / S::kSlots & 1);
}

template <class T, int DP>
__device__ __forceinline__ void issue(const Params& p, State& s, const AttendRows& rows, const AttendShare& share, uint32_t queries, uint32_t ring,
                                      uint32_t tmem, int columns) {
  using S = Shape<DP>;
  const int steps = (p.dim + 15) / 16;
  const uint32_t shape = tcgen05_shape(std::is_same<T, __nv_bfloat16>::value, columns, false), one = elected();
  uint32_t keys = 0, segments = 0, count = 0, items = 0;
  for (AttendSegment g = attend_first(p, rows, share, kTile); g.tiles; g = attend_next(p, rows, share, g, kTile)) {
    wait(s.stop, smem_u32(&s.queries), segments & 1);
    ++segments;
    tcgen05_after_sync();
    const int tiles = __shfl_sync(~0u, g.tiles, 0);
#pragma unroll 1
    for (int i = 0; i < tiles; ++i) {
      const uint32_t w = items & 1, at = keys % S::kSlots;
      ++items;
      wait(s.stop, smem_u32(&s.full[at]), keys / S::kSlots & 1);
      wait(s.stop, smem_u32(&s.taken[w]), (count >> w & 1) ^ 1);  // (the first time: free)
      count ^= 1u << w;
      tcgen05_after_sync();
      const uint64_t a = smem_along_k(ring + at * S::kSlot), b = smem_along_k(queries);
#pragma unroll
      for (int e = 0; e < DP / 16; ++e)
        if (e < steps)
          tcgen05_mma(one, tmem + w * 256, a + (e / 4 * kTile * 128 + e % 4 * 32) / 16, b + (e / 4 * S::kMostRows * 128 + e % 4 * 32) / 16, shape, e > 0);
      tcgen05_commit(one, smem_u32(&s.scores[w]));
      tcgen05_commit(one, smem_u32(&s.empty[at]));
      keys = (keys + 1) % (2 * S::kSlots);
    }
  }
  tcgen05_commit(one, smem_u32(&s.end));
  wait_own(s.stop, smem_u32(&s.end), 0);
}

// Scores that the cap changes, and those of query rows that do not see the
// token, which become -infinity (whatever they are).
__device__ __noinline__ void prepare(const Params& p, const DraftTree& tree, uint32_t at, int columns, int t, int base, bool all) {
  const int per = (int)p.per.d;
  int draft = (int)fast_div32(p.per, (uint32_t)p.row0), head = p.row0 - draft * per;
  bool sees = true;
  if (!all) sees = tree.sees(p, min(draft, p.drafts - 1), t, base);
#pragma unroll 1
  for (int c = 0; c < columns; c += 32) {
    uint32_t x[32], seen = ~0u;
    tmem_load(x, at + c);
    if (!all) {
#pragma unroll 1
      for (int e = 0; e < 32; ++e) {
        if (!sees) seen &= ~(1u << e);
        if (++head == per) {
          head = 0;
          ++draft;
          sees = tree.sees(p, min(draft, p.drafts - 1), t, base);
        }
      }
    }
    tmem_wait_load(x);
    if (p.cap_out != 0.0f) {
#pragma unroll
      for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(p.cap_out * tanhf(__uint_as_float(x[e]) * p.cap_in));
    }
#pragma unroll
    for (int e = 0; e < 32; ++e) x[e] = seen >> e & 1 ? x[e] : __float_as_uint(-CUDART_INF_F);
    tmem_store(at + c, x);
  }
  tmem_wait_store();
}

// What a token gets from the query rows. HIDDEN: scores of -infinity count
// nothing, whatever their row's statistics.
template <bool HIDDEN>
__device__ __forceinline__ float token_sum(const State& s, uint32_t at, int columns, float to_log2) {
  const uint64_t scale = pair(to_log2, to_log2);
  uint64_t part[2] = {0, 0};
#pragma unroll 1
  for (int c = 0; c < columns; c += 32) {
    uint32_t x[32];
    tmem_load(x, at + c);
    tmem_wait_load(x);
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      if (e % 16 == 0 && c + e >= columns) break;  // (columns are a multiple of 16)
      const float4 st = s.stats[(c + e) / 2];
      float2 z = unpair(fma2(pair(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), scale, pair(st.x, st.y)));
      // (a score that is not a number: its row's 1 / l is none either, or the row
      // is zeros beside an infinite key, and 1 / l is 0)
      z.x = fmaxf(z.x, -200.0f);
      z.y = fmaxf(z.y, -200.0f);
      if (HIDDEN) {
        const float a = __uint_as_float(x[e]) == -CUDART_INF_F ? 0.0f : power_of_two(z.x) * st.z;
        const float b = __uint_as_float(x[e + 1]) == -CUDART_INF_F ? 0.0f : power_of_two(z.y) * st.w;
        part[e / 2 & 1] = add2(part[e / 2 & 1], pair(a, b));
      } else {
        part[e / 2 & 1] = fma2(pair(power_of_two(z.x), power_of_two(z.y)), pair(st.z, st.w), part[e / 2 & 1]);
      }
    }
  }
  const float2 both = unpair(add2(part[0], part[1]));
  return both.x + both.y;
}

template <class T, int DP>
__device__ __forceinline__ void sums(const Params& p, State& s, DraftTree& tree, const AttendRows& rows, const AttendShare& share, unsigned char* queries,
                                     uint32_t tmem, int n, int columns) {
  using S = Shape<DP>;
  using Both = SomeThreads<2 * kGroup, 1>;
  const uint32_t w = threadIdx.x / kGroup, token = threadIdx.x % kGroup, at = tmem + w * 256 + ((threadIdx.x / 32 % 4 * 32) << 16);
  uint32_t items = 0, count = 0;
  for (AttendSegment g = attend_first(p, rows, share, kTile); g.tiles; g = attend_next(p, rows, share, g, kTile)) {
    const int kv = g.group, base = g.n - p.drafts;
    const bool planted = !draft_all_seen(p, g.tile0 * kTile, (g.tile0 + g.tiles) * kTile, base);
    Both::sync();  // (the queries before these are no longer read)
    // rows, and what the attention has left of them; padding (a sum of zero) is zeros, whatever it holds
    const float2* stats = p.stats + ((int64_t)g.row * p.kv_heads + kv) * p.group + p.row0;
    for (int q = threadIdx.x; q < columns; q += 2 * kGroup) {
      const float2 x = q < n ? stats[q] : make_float2(0.0f, 0.0f);
      float* to = reinterpret_cast<float*>(&s.stats[q / 2]) + q % 2;
      to[0] = x.y == 0.0f ? 0.0f : -x.x;
      to[2] = x.y == 0.0f ? 0.0f : 1.0f / x.y;
    }
    {
      constexpr int kPieces = DP / 8, kOver = 2 * kGroup / kPieces, kAtOnce = 4;
      const int c = threadIdx.x % kPieces;
      if (c < (p.dim + 15) / 16 * 2) {
        unsigned char* slab = queries + c / 8 * S::kMostRows * 128;
#pragma unroll 1
        for (int r0 = threadIdx.x / kPieces; r0 < columns; r0 += kOver * kAtOnce) {
          uint4 x[kAtOnce];
#pragma unroll
          for (int k = 0; k < kAtOnce; ++k) {
            const int r = r0 + k * kOver;
            x[k] = make_uint4(0, 0, 0, 0);
            if (r < n && c * 8 < p.dim && stats[r].y != 0.0f) {
              const T* q = draft_query<T>(p, g.row, kv, p.row0 + r) + c * 8;
              if (p.q_vectors) {
                x[k] = *reinterpret_cast<const uint4*>(q);
              } else {
                T e[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) e[j] = q[j];
                x[k] = *reinterpret_cast<uint4*>(e);
              }
            }
          }
#pragma unroll
          for (int k = 0; k < kAtOnce; ++k)
            if (r0 + k * kOver < columns) *reinterpret_cast<uint4*>(slab + swizzled(r0 + k * kOver, c % 8)) = x[k];
        }
      }
    }
    fence_async_smem();
    mbar_arrive(smem_u32(&s.queries));
    if (planted) draft_tree<2 * kGroup, Both>(p, tree, g.row, base);
    else Both::sync();  // (the statistics are complete)
    float* weights = p.weights + g.row * p.w_st[0] + kv * p.w_st[1];
    for (int i = 0; i < g.tiles; ++i, ++items) {
      if ((items & 1) != w) continue;
      const int t0 = (g.tile0 + i) * kTile, t = t0 + token;
      float before = 0.0f;
      if (t >= g.lo && t < g.n) before = weights[t];  // (on its way while the scores are worked out)
      wait(s.stop, smem_u32(&s.scores[w]), count & 1);
      ++count;
      tcgen05_after_sync();
      const uint32_t here = s.here[items % kHereTiles][token / 32];
      const bool all = draft_all_seen(p, t0, t0 + kTile, base);
      float sum;
      if (!all || p.cap_out != 0.0f) {
        prepare(p, tree, at, columns, t, base, all);
        sum = token_sum<true>(s, at, columns, p.cap_out != 0.0f ? 1.0f : p.scale_log2);
      } else {
        sum = token_sum<false>(s, at, columns, p.scale_log2);
      }
      tcgen05_before_sync();
      mbar_arrive(smem_u32(&s.taken[w]));
      if (gave_up(s.stop)) {  // (nor is what `here` says known to be the tile's)
        if (t >= g.lo && t < g.n) weights[t] = CUDART_NAN_F;
      } else if (here >> (token % 32) & 1) {
        weights[t] = before + sum;
      }
    }
  }
}

template <class T, int DP>
__global__ void __launch_bounds__(kThreads, 1) weigh_tc_kernel(const __grid_constant__ Params p) {
  using S = Shape<DP>;
  extern __shared__ unsigned char s_raw[];
  unsigned char* s_mem = s_raw + ((1024 - smem_u32(s_raw) % 1024) % 1024);
  State& s = *reinterpret_cast<State*>(s_mem + S::kRest);
  DraftTree& tree = *reinterpret_cast<DraftTree*>(&s + 1);
  AttendRows& rows = *reinterpret_cast<AttendRows*>(&tree + 1);
  const int warp = threadIdx.x / 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kSlots; ++i) {
      mbar_init(smem_u32(&s.full[i]), 1);
      mbar_init(smem_u32(&s.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s.scores[i]), 1);
      mbar_init(smem_u32(&s.taken[i]), kGroup);
    }
    mbar_init(smem_u32(&s.queries), 2 * kGroup);
    mbar_init(smem_u32(&s.end), 1);
    s.stop = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 8) tmem_alloc(smem_u32(&s.tmem), 512);
  wait_for_previous();
  let_next_start();
  attend_rows(p, rows, kTile);
  const AttendShare share = attend_share(p, rows);
  tcgen05_before_sync();
  __syncthreads();
  tcgen05_after_sync();
  const uint32_t tmem = *static_cast<volatile uint32_t*>(&s.tmem);
  const uint32_t queries = smem_u32(s_mem), ring = queries + S::kQueries;
  const int n = min(p.group - p.row0, S::kMostRows), columns = (n + 15) / 16 * 16;
  if (share.begin == share.end) {
  } else if (warp < 8) {
    sums<T, DP>(p, s, tree, rows, share, s_mem, tmem, n, columns);
  } else if (warp == 8) {
    issue<T, DP>(p, s, rows, share, queries, ring, __shfl_sync(~0u, tmem, 0), columns);
  } else {
    copy_keys<DP>(p, s, ring, rows, share);
  }
  tcgen05_before_sync();
  __syncthreads();
  tcgen05_after_sync();
  if (warp == 8) tmem_free(tmem, 512);
  if (threadIdx.x == 0 && s.stop) report(p.status, CMD_CACHE_TIMEOUT);
}

template <class T, int DP>
cudaError_t launch(const Params& p, cudaStream_t stream) {
  static PerDevice ready;  // (static storage: zero before first use)
  static_assert(kSmem<DP> <= 227 * 1024, "the CTA fits an SM");
  cudaError_t e = allow_smem(weigh_tc_kernel<T, DP>, kSmem<DP>, ready);
  Params q = p;
  const int ctas = attend_sides(p.kv_heads, 152, &q.sides);
  for (q.row0 = 0; e == cudaSuccess && q.row0 < q.group; q.row0 += Shape<DP>::kMostRows)
    e = launch_chained(weigh_tc_kernel<T, DP>, ctas, kThreads, (size_t)kSmem<DP>, stream, q);
  return e;
}
template <class T>
cudaError_t by_dim(const Params& p, cudaStream_t stream) {
  if (p.dim <= 64) return launch<T, 64>(p, stream);
  return p.dim <= 128 ? launch<T, 128>(p, stream) : launch<T, 256>(p, stream);
}

}  // namespace

cudaError_t weigh_tma_launch(int dtype, const DraftParams& d, cudaStream_t stream) {
  Params p;
  const cudaError_t e = pool_maps(dtype, d, &p);
  if (e != cudaSuccess) return e;
  p.blocks = 1;
  p.start_units = 4;
  return dtype == CMD_F16 ? by_dim<__half>(p, stream) : by_dim<__nv_bfloat16>(p, stream);
}

}  // namespace cmdx
