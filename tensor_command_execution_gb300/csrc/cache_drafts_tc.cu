// cache_drafts_tc.cu - attention of drafted tokens over a paged cache of
// 16-bit numbers on the CTA-wide tensor instructions (tcgen05).
//
// A CTA takes 128 query rows (drafts times the query heads of a kv head) at a
// time, or 256 as two sets of 128, against tiles of 128 tokens: S = Q K^T into
// tensor memory, the softmax there, O += P V with P read from tensor memory. Two
// groups of four softmax warps, a thread to a query row, take turns, so that the
// tensor units work on one group's products while the other's exponentials are
// worked out: with 256 rows a group has its own rows (and a key or value is read
// once for both), with 128 its own tiles, and the two halves are joined at the
// end of a segment. One warp issues the products, others copy keys and values
// into a ring in the layout that the products read: TMA boxes of the tokens that
// a page and a tile share, where those are 8 or a multiple (a warp for keys, one
// for values), else three warps with 16-byte asynchronous copies.
//
// A weight is held as the sum of two 16-bit numbers, as in cache_attend_mma.cu:
// P takes exactly the columns of S that it came from. O is rescaled only when a
// row's maximum has grown by more than kSlack (in powers of two) since it was
// last taken: weights are up to 2^kSlack then, and f16 ones are lifted by 2^11
// (rather than 2^15), which holds them to no finer than 2^-36 of the largest.
//
// Measured: 4 rows of 64 drafts, up to 16384 tokens, 64 query heads on 8 kv heads
// of 128 dims (512 query rows to a kv head): 136 us with the join, 739 TFLOP/s of
// the attention's products, and with the weights' second halves 1.5 times as many
// on the tensor units, which are busy 56% of the time; the rest is a group's wait
// for its turn at them and segments' beginnings. 16 rows of 24 drafts, 0 to 8192
// tokens, 32 query heads on 8: 43 us, for 79 MB of keys and values 12: segments
// of a few tiles (queries, first keys, last products and states: 10 thousand
// cycles each), and the join.
#include "cache_drafts.cuh"
#include "cache_attend_ring.cuh"
#include "cache_mma.cuh"
#include "cache_tc.cuh"

#ifndef CMDX_TMA
#error "cache_drafts_tc.cu is compiled for both kinds of copies, with -DCMDX_TMA=<1|0>"
#endif

namespace cmdx {

namespace {

constexpr int kGroup = 128;                   // threads of a softmax group, and query rows
constexpr int kLoaders = CMDX_TMA ? 64 : 96;
constexpr int kThreads = 2 * kGroup + 32 + kLoaders;
constexpr int kTile = 128;                    // tokens

// Powers of two: how far a maximum may grow before O is rescaled, and how far
// weights are lifted.
template <class T>
constexpr float kSlack = 8.0f;
template <>
constexpr float kSlack<__half> = 4.0f;
template <class T>
constexpr float kRaise = 0.0f;
template <>
constexpr float kRaise<__half> = 11.0f;
template <class T>
constexpr bool kBf16 = true;
template <>
constexpr bool kBf16<__half> = false;

// x and y rounded to 16 bits, and what that leaves of each, rounded again
template <class T>
__device__ __forceinline__ void split2(float x, float y, uint32_t* hi, uint32_t* lo) {
  if constexpr (kBf16<T>) {
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(*hi) : "f"(y), "f"(x));
    const float2 rest = unpair(add2(pair(x, y), pair(-__uint_as_float(*hi << 16), -__uint_as_float(*hi & 0xffff0000u))));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(*lo) : "f"(rest.y), "f"(rest.x));
  } else {
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(*hi) : "f"(y), "f"(x));
    const float2 h = __half22float2(*reinterpret_cast<const __half2*>(hi));
    const float2 rest = unpair(add2(pair(x, y), pair(-h.x, -h.y)));
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(*lo) : "f"(rest.y), "f"(rest.x));
  }
}

template <int DP, bool WIDE>
struct Shape {
  static constexpr int kRows = WIDE ? 256 : 128;
  static constexpr int kSlot = kTile * DP * 2;    // keys or values of a tile
  static constexpr int kSlots = DP == 64 ? 8 : 4;
  static constexpr int kQueries = kRows * DP * 2;
  static constexpr int kRing = kQueries;
  static constexpr int kRest = kRing + kSlots * kSlot;
  static constexpr int kScores = 0;               // columns of tensor memory: S of each group, then O
  static constexpr int kOut = 256;
};

constexpr int kHereTiles = 8;
struct State {
  uint64_t full[8], empty[8], scores[2], weights[2], done[2], landed, queries, end;
  uint32_t tmem;
  uint32_t stop;                       // a wait ran out of time
  uint32_t here[kHereTiles][4];        // which tokens of a tile have a page
  uint32_t bad[kHereTiles];            // the last of these tiles (counted from 1) whose values are not all finite
  float2 part[2][kGroup];              // maximum and sum of a group's rows
#if !CMDX_TMA
  int64_t k[2][kTile], v[2][kTile];    // offsets of a tile's rows, -1: none
#endif
};
template <int DP, bool WIDE>
constexpr int kSmem = Shape<DP, WIDE>::kRest + (int)(sizeof(State) + sizeof(DraftTree) + sizeof(AttendRows)) + 1024;

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

// ---- the copies -----------------------------------------------------------------
#if CMDX_TMA
template <class T, int DP, bool WIDE>
struct Loader {
  using S = Shape<DP, WIDE>;
  static constexpr int kPieces = DP / 8, kOver = 32 / kPieces;
  const TcParams& p;
  State& s;
  const uint32_t ring;
  TmaTiles tiles;
  const bool values;             // of the two warps one copies keys, one values: each slot is one warp's, which waits for all
                                 // of its turns (a parity says nothing about a barrier that is two turns away)
  uint32_t copies, cleared = 0;  // keys and values in turn; tiles that were

  __device__ __forceinline__ Loader(const TcParams& p_, State& s_, uint32_t ring_)
      : p(p_), s(s_), ring(ring_), tiles(p_), values(threadIdx.x >= 2 * kGroup + 64), copies(values) {
    static_assert(S::kSlots % 2 == 0, "a slot is of keys or of values");
  }

  // Rows of no token become zeros, and so do values that are not finite,
  // whatever their weight: the softmax group is told, and adds them where they
  // are seen.
  __device__ __forceinline__ void clear(uint32_t slot) {
    constexpr int kAtOnce = 8;
    uint32_t here[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) here[k] = __shfl_sync(~0u, tiles.here, k);
    const int lane = tiles.lane, c = lane % kPieces;
    if (c < (p.dim + 15) / 16 * 2) {
      const uint32_t at = slot + c / 8 * kTile * 128;
#pragma unroll 1
      for (int r0 = lane / kPieces; r0 < kTile; r0 += kOver * kAtOnce) {
        uint4 x[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) x[k] = lds128(at + swizzled(r0 + k * kOver, c % 8));
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
          const int r = r0 + k * kOver;
          const uint4 bad = make_uint4(not_finite<T>(x[k].x), not_finite<T>(x[k].y), not_finite<T>(x[k].z), not_finite<T>(x[k].w));
          const uint32_t word = r < 64 ? (r < 32 ? here[0] : here[1]) : (r < 96 ? here[2] : here[3]);
          const bool in = word >> (r & 31) & 1;
          if (in && (bad.x | bad.y | bad.z | bad.w) == 0) continue;
          sts128(at + swizzled(r, c % 8), in ? make_uint4(x[k].x & ~bad.x, x[k].y & ~bad.y, x[k].z & ~bad.z, x[k].w & ~bad.w) : make_uint4(0, 0, 0, 0));
          if (in) *static_cast<volatile uint32_t*>(&s.bad[copies / 2 % kHereTiles]) = copies / 2 + 1;
        }
      }
    }
    fence_async_smem();
    __syncwarp();
  }

  __device__ __forceinline__ void run(const AttendRows& rows, const AttendShare& share, const AttendSegment& head) {
    issue(rows, share, head);
    // (none is on its way when the CTA ends)
    for (uint32_t c = copies - min(copies - values, (uint32_t)S::kSlots); c < copies; c += 2)
      wait_own(s.stop, smem_u32(&s.full[c % S::kSlots]), c / S::kSlots & 1);
  }
  __device__ __forceinline__ void issue(const AttendRows& rows, const AttendShare& share, const AttendSegment& head) {
    for (AttendSegment g = head; g.tiles; g = attend_next(p, rows, share, g, kTile)) {
      const int kv = attend_heads(p, g.group).kv, base = g.n - p.drafts;
      tiles.begin(g);
      for (int i = 0; i < g.tiles; ++i, copies += 2) {
        tiles.look<true>(i);
        const uint32_t at = copies % S::kSlots, slot = ring + at * S::kSlot, full = smem_u32(&s.full[at]);
        if (!warp_wait(s.stop, smem_u32(&s.empty[at]), (copies / S::kSlots + 1) & 1)) return;
        if (!values) {
          if (tiles.lane < 4) s.here[copies / 2 % kHereTiles][tiles.lane] = tiles.here;
          __syncwarp();
          tiles.copy(p.maps[0], kv, slot, full);
          continue;
        }
        const bool all = __all_sync(~0u, tiles.lane >= 4 || tiles.here == ~0u) && draft_all_seen(p, tiles.t0, tiles.t0 + kTile, base);
        tiles.copy(p.maps[1], kv, slot, all ? full : smem_u32(&s.landed));
        if (!all) {
          const uint32_t turn = cleared++ & 1;
          if (!warp_wait(s.stop, smem_u32(&s.landed), turn)) {
            wait_own(s.stop, smem_u32(&s.landed), turn);
            return;
          }
          clear(slot);
          if (tiles.one) mbar_arrive(full);
        }
      }
    }
  }
};
#else
template <class T, int DP, bool WIDE>
struct Loader {
  using S = Shape<DP, WIDE>;
  static constexpr int kChunks = DP / 8, kOver = kLoaders / kChunks;
  const TcParams& p;
  State& s;
  const uint32_t ring;
  const int tid = threadIdx.x - 2 * kGroup - 32, chunk = tid % kChunks, row0 = tid / kChunks, chunks, used;
  uint32_t issued = 0;  // keys and values in turn

  __device__ __forceinline__ Loader(const TcParams& p_, State& s_, uint32_t ring_)
      : p(p_), s(s_), ring(ring_), chunks(p_.dim / 8), used((p_.dim + 15) / 16 * 2) {}

  // Values that are not finite become zeros, whatever their weight, and the
  // softmax group is told: it adds them where they are seen.
  __device__ __forceinline__ void clear(int slot) {
    if (chunk >= chunks) return;
    const uint32_t at = ring + slot * S::kSlot + chunk / 8 * kTile * 128;
    for (int r = row0; r < kTile; r += kOver) {
      const uint32_t a = at + swizzled(r, chunk % 8);
      uint4 x = lds128(a);
      const uint4 bad = make_uint4(not_finite<T>(x.x), not_finite<T>(x.y), not_finite<T>(x.z), not_finite<T>(x.w));
      if ((bad.x | bad.y | bad.z | bad.w) == 0) continue;
      sts128(a, make_uint4(x.x & ~bad.x, x.y & ~bad.y, x.z & ~bad.z, x.w & ~bad.w));
      *static_cast<volatile uint32_t*>(&s.bad[issued / 2 % kHereTiles]) = issued / 2 + 1;
    }
  }
  __device__ __forceinline__ void copy(const T* from, const int64_t* offset, bool mask) {
    const int slot = issued % S::kSlots;
    const uint32_t bar = smem_u32(&s.empty[slot]), parity = (issued / S::kSlots + 1) & 1;
    wait(s.stop, bar, parity);
    if (chunk < used) {
      const bool inside = chunk < chunks;
      const T* at = from + (inside ? chunk * 8 : 0);
      const uint32_t dst = ring + slot * S::kSlot + chunk / 8 * kTile * 128;
      constexpr int kAtOnce = 8;  // (offsets read before the copies that need them)
#pragma unroll 1
      for (int r0 = row0; r0 < kTile; r0 += kOver * kAtOnce) {
        int64_t o[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) o[k] = r0 + k * kOver < kTile ? offset[r0 + k * kOver] : -1;
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
          if (r0 + k * kOver < kTile)
            copy_bytes<16>(dst + swizzled(r0 + k * kOver, chunk % 8), at + (o[k] >= 0 ? o[k] : 0), o[k] >= 0 && inside ? 16 : 0);
      }
    }
    // The arrival comes with the data; the thread that issues the products, not
    // this one, orders them for the products' reads: the fence waits for all of
    // a thread's copies on their way (here it cost 5 to 10 thousand cycles a
    // tile: 4 rows of 64 drafts and 16384 tokens took three quarters longer).
    const uint32_t full = smem_u32(&s.full[slot]);
    if (mask) {
      copy_commit();
      copy_wait<0>();
      clear(slot);
      mbar_arrive(full);
    } else {
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(full) : "memory");
    }
    ++issued;
  }

  __device__ __forceinline__ void run(const AttendRows& rows, const AttendShare& share, const AttendSegment& head) {
    int tile = 0;
    for (AttendSegment g = head; g.tiles; g = attend_next(p, rows, share, g, kTile)) {
      const int kv = attend_heads(p, g.group).kv, base = g.n - p.drafts;
      DraftLook look[2];
      const auto look_up = [&](int i) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          look[e] = {0, 0, false};
          const int t = (g.tile0 + i) * kTile + tid + e * kLoaders;
          if (tid + e * kLoaders < kTile && i < g.tiles && t >= g.lo && t < g.n) {
            const uint32_t column = fast_div32(p.page, (uint32_t)t);
            look[e].inside = true;
            look[e].slot = t - (int)(column * p.page.d);
            look[e].page = p.tables[g.row * p.table_st[0] + column * p.table_st[1]];
          }
        }
      };
      look_up(0);
      for (int i = 0; i < g.tiles; ++i, ++tile) {
        const int b = tile & 1;
        bool all = true;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = tid + e * kLoaders;
          if (r >= kTile) break;  // (whole warps)
          bool in = look[e].inside;
          if (in && (look[e].page < 0 || look[e].page >= p.n_pages)) {
            report(p.status, CMD_CACHE_BAD_PAGE);
            in = false;
          }
          s.k[b][r] = in ? look[e].page * p.k_st[0] + look[e].slot * p.k_st[1] + kv * p.k_st[2] : -1;
          s.v[b][r] = in ? look[e].page * p.v_st[0] + look[e].slot * p.v_st[1] + kv * p.v_st[2] : -1;
          const uint32_t here = __ballot_sync(~0u, in);
          if (threadIdx.x % 32 == 0) s.here[tile % kHereTiles][r / 32] = here;
        }
        look_up(i + 1);
        SomeThreads<kLoaders, 2>::sync();
        const uint32_t* here = s.here[tile % kHereTiles];
        all = (here[0] & here[1] & here[2] & here[3]) == ~0u;
        const int t0 = (g.tile0 + i) * kTile;
        copy(static_cast<const T*>(p.k), s.k[b], false);
        copy(static_cast<const T*>(p.v), s.v[b], !(all && draft_all_seen(p, t0, t0 + kTile, base)));
      }
    }
    copy_commit();
    copy_wait<0>();
  }
};

#endif

// ---- the products -----------------------------------------------------------------
// (What comes from shared memory passes through a shuffle, so that it is known
// to be the same in all lanes.)
template <class T, int DP, bool WIDE>
__device__ __forceinline__ void issue(const DraftParams& p, State& s, const AttendRows& rows, const AttendShare& share,
                                      const AttendSegment& head, uint32_t queries, uint32_t ring, uint32_t tmem) {
  using S = Shape<DP, WIDE>;
  const int steps = (p.dim + 15) / 16;
  const uint32_t qk = tcgen05_shape(kBf16<T>, kTile, false), pv = tcgen05_shape(kBf16<T>, steps * 16, true), one = elected();
  // the copies (keys and values in turn) that the next products read, modulo
  // twice the ring, and how often the groups' weights were waited for
  uint32_t keys = 0, values = 1, segments = 0, count = 0;
  const auto wait_full = [&](uint32_t copy) {
    wait(s.stop, smem_u32(&s.full[copy % S::kSlots]), copy / S::kSlots & 1);
    if (!CMDX_TMA) fence_async_smem();
  };
  for (AttendSegment g = head; g.tiles; g = attend_next(p, rows, share, g, kTile)) {
    wait(s.stop, smem_u32(&s.queries), segments & 1);
    ++segments;
    tcgen05_after_sync();
    const int items = __shfl_sync(~0u, WIDE ? 2 * g.tiles : g.tiles, 0);
    const auto scores = [&](uint32_t w) {
      if (!WIDE || w == 0) wait_full(keys);
      const uint32_t q = queries + (WIDE ? w * kGroup * 128 : 0), at = keys % S::kSlots;
      const uint64_t a = smem_along_k(q), b = smem_along_k(ring + at * S::kSlot);
#pragma unroll
      for (int e = 0; e < DP / 16; ++e)
        if (e < steps)
          tcgen05_mma(one, tmem + S::kScores + w * kTile, a + (e / 4 * S::kRows * 128 + e % 4 * 32) / 16, b + (e / 4 * kTile * 128 + e % 4 * 32) / 16,
                      qk, e > 0);
      tcgen05_commit(one, smem_u32(&s.scores[w]));
      if (!WIDE || w == 1) {
        tcgen05_commit(one, smem_u32(&s.empty[at]));
        keys = (keys + 2) % (2 * S::kSlots);
      }
    };
    scores(0);
    if (items > 1) scores(1);
#pragma unroll 1
    for (int n = 0; n < items; ++n) {
      const uint32_t w = n & 1;
      if (!WIDE || w == 0) wait_full(values);
      wait(s.stop, smem_u32(&s.weights[w]), count >> w & 1);
      count ^= 1u << w;
      tcgen05_after_sync();
      const uint32_t at = values % S::kSlots, weights = tmem + S::kScores + w * kTile, out = tmem + S::kOut + w * 128;
      const uint64_t b = smem_across_k(ring + at * S::kSlot, kTile * 128);
#pragma unroll
      for (int e = 0; e < kTile / 16; ++e) {
        // (a chunk of 32 tokens: 16 columns of the weights' upper parts, 16 of the lower)
        const uint32_t a = weights + e / 2 * 32 + e % 2 * 8;
        tcgen05_mma(one, out, a, b + e * 2048 / 16, pv, n > 1 || e > 0);
        tcgen05_mma(one, out, a + 16, b + e * 2048 / 16, pv, true);
      }
      tcgen05_commit(one, smem_u32(&s.done[w]));
      if (!WIDE || w == 1) {
        tcgen05_commit(one, smem_u32(&s.empty[at]));
        values = (values + 2) % (2 * S::kSlots);
      }
      if (n + 2 < items) scores(w);
    }
  }
  tcgen05_commit(one, smem_u32(&s.end));
  wait_own(s.stop, smem_u32(&s.end), 0);
}

// ---- the softmax --------------------------------------------------------------------
template <class T, int DP, bool WIDE>
struct Softmax {
  using S = Shape<DP, WIDE>;
  const DraftParams& p;
  State& s;
  DraftTree& tree;
  const uint32_t tmem;   // of this warp's lanes
  const int w = threadIdx.x / kGroup, row = threadIdx.x % kGroup;
  uint32_t count = 0;    // items so far
  // of the row: the power of two that its weights are counted from (its maximum
  // when O was last rescaled, less kRaise), and their sum
  float m, l;

  __device__ __forceinline__ Softmax(const DraftParams& p_, State& s_, DraftTree& t, uint32_t tmem_)
      : p(p_), s(s_), tree(t), tmem(tmem_ + ((threadIdx.x / 32 % 4 * 32) << 16)) {}

  __device__ __forceinline__ void load_queries(unsigned char* to, int batch_row, int kv, int q0, int n) {
    constexpr int kPieces = DP / 8, kOver = 2 * kGroup / kPieces, kAtOnce = 8;
    const int c = threadIdx.x % kPieces, r0 = threadIdx.x / kPieces;
    if (c >= (p.dim + 15) / 16 * 2) return;
    unsigned char* slab = to + c / 8 * S::kRows * 128;
#pragma unroll 1
    for (int i = 0; i < S::kRows; i += kOver * kAtOnce) {
      uint4 x[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const int r = r0 + i + k * kOver;
        x[k] = make_uint4(0, 0, 0, 0);
        if (r < n && c * 8 < p.dim) {
          const T* q = draft_query<T>(p, batch_row, kv, q0 + r) + c * 8;
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
      for (int k = 0; k < kAtOnce; ++k) {
        const int r = r0 + i + k * kOver;
        if (r < S::kRows) *reinterpret_cast<uint4*>(slab + swizzled(r, c % 8)) = x[k];
      }
    }
  }

  // Scores that the cap changes, and those of tokens that the row does not see,
  // which become -infinity (whatever they are).
  __device__ __noinline__ void prepare(int draft, int t0, int base, bool all, const uint32_t* here) {
    const uint32_t at = tmem + S::kScores + w * kTile;
#pragma unroll 1
    for (int c = 0; c < kTile / 32; ++c) {
      uint32_t x[32];
      tmem_load(x, at + 32 * c);
      const uint32_t seen = here[c] & (all ? ~0u : tree.sees_of_32(p, draft, t0 + 32 * c, base));
      tmem_wait_load(x);
      if (p.cap_out != 0.0f) {
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(p.cap_out * tanhf(__uint_as_float(x[e]) * p.cap_in));
      }
#pragma unroll
      for (int e = 0; e < 32; ++e) x[e] = seen >> e & 1 ? x[e] : __float_as_uint(-CUDART_INF_F);
      tmem_store(at + 32 * c, x);
    }
    tmem_wait_store();
  }

  // One tile of this group's: the weights of its 128 tokens into the place of
  // their scores.
  __device__ __forceinline__ void item(bool first) {
    const uint32_t at = tmem + S::kScores + w * kTile;
    const float scale = p.cap_out != 0.0f ? 1.0f : p.scale_log2;
    float top = -CUDART_INF_F;
    {
      float up[4] = {top, top, top, top};
#pragma unroll 1
      for (int c = 0; c < kTile; c += 64) {
        uint32_t x[32], y[32];
        tmem_load(x, at + c);
        tmem_load(y, at + c + 32);
        tmem_wait_load(x);
        tmem_wait_load(y);
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
#pragma unroll
          for (int k = 0; k < 4; ++k) up[k] = max3(up[k], __uint_as_float(x[e + k]), __uint_as_float(y[e + k]));
        }
      }
      top = fmaxf(max3(up[0], up[1], up[2]), up[3]) * scale;
    }
    const bool grown = top > m + (kSlack<T> + kRaise<T>);  // (also from -infinity)
    if (__any_sync(~0u, grown)) {
      const float now = top - kRaise<T>, c = grown ? attend_weight(m, now) : 1.0f;
      if (grown) m = now;
      if (!first && __any_sync(~0u, c != 1.0f)) {
        wait(s.stop, smem_u32(&s.done[w]), (count - 1) & 1);
        tcgen05_after_sync();
        rescale(c);
      }
      l *= c;
    }
    const float low = m == -CUDART_INF_F ? 0.0f : -m;
    const uint64_t scale2 = pair(scale, scale), low2 = pair(low, low);
    uint64_t sum[2] = {0, 0};
    uint32_t x[2][32];
    tmem_load(x[0], at);
#pragma unroll 1
    for (int c = 0; c < kTile; c += 64) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        tmem_wait_load(x[b]);
        if (c + 32 * b + 32 < kTile) tmem_load(x[b ^ 1], at + c + 32 * b + 32);
        uint32_t y[32];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const float2 z = unpair(fma2(pair(__uint_as_float(x[b][e]), __uint_as_float(x[b][e + 1])), scale2, low2));
          const float u = power_of_two(z.x), v = power_of_two(z.y);
          sum[e / 2 & 1] = add2(sum[e / 2 & 1], pair(u, v));
          split2<T>(u, v, &y[e / 2], &y[16 + e / 2]);
        }
        tmem_store(at + c + 32 * b, y);
      }
    }
    const float2 all = unpair(add2(sum[0], sum[1]));
    l += all.x + all.y;
    tmem_wait_store();
  }

  __device__ __forceinline__ void rescale(float c) {
    for (int d = 0; d < p.dim; d += 32) {
      uint32_t x[32];
      tmem_load(x, tmem + S::kOut + w * 128 + d);
      tmem_wait_load(x);
#pragma unroll
      for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * c);
      tmem_store(tmem + S::kOut + w * 128 + d, x);
    }
    tmem_wait_store();
  }

  // What the copies left out of a tile's values because it is not finite, to
  // the rows that see it (read again from where it lies).
  __device__ __noinline__ void add_infinite(const AttendSegment& g, int kv, int draft, bool alive, int t0, int base, bool all,
                                            const uint32_t* here) {
    uint32_t seen[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) seen[c] = !alive ? 0u : here[c] & (all ? ~0u : tree.sees_of_32(p, draft, t0 + 32 * c, base));
    for (int d = 0; d < p.dim; d += 32) {
      uint32_t x[32];
      tmem_load(x, tmem + S::kOut + w * 128 + d);
      tmem_wait_load(x);
      for (int t = 0; t < kTile; ++t) {
        if (!(here[t >> 5] >> (t & 31) & 1)) continue;
        const uint32_t column = fast_div32(p.page, (uint32_t)(t0 + t));
        const int slot = t0 + t - (int)(column * p.page.d), page = p.tables[g.row * p.table_st[0] + column * p.table_st[1]];
        const T* v = static_cast<const T*>(p.v) + page * p.v_st[0] + slot * p.v_st[1] + kv * p.v_st[2] + d;
        const bool sees = seen[t >> 5] >> (t & 31) & 1;
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (sees && d + e < p.dim) {
            const float y = to_float(v[e]);
            if (!(fabsf(y) < CUDART_INF_F)) x[e] = __float_as_uint(__uint_as_float(x[e]) + y);
          }
      }
      tmem_store(tmem + S::kOut + w * 128 + d, x);
    }
    tmem_wait_store();
  }

  // Writes 32 elements of the row's (finished or a part's).
  __device__ __forceinline__ void write(const float (&o)[32], float* part, T* out, int d) const {
    if (part) {
#pragma unroll
      for (int e = 0; e < 32; e += 4)
        if (d + e < p.dim) *reinterpret_cast<float4*>(part + d + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
    } else if (p.out_vectors) {
#pragma unroll
      for (int e = 0; e < 32; e += 8)
        if (d + e < p.dim) {
          T y[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) y[k] = from_float<T>(o[e + k]);
          *reinterpret_cast<uint4*>(out + d + e) = *reinterpret_cast<uint4*>(y);
        }
    } else {
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if (d + e < p.dim) out[d + e] = from_float<T>(o[e]);
    }
  }

  // team_part: where a team's part goes
  __device__ __forceinline__ void run(const AttendRows& rows, const AttendShare& share, const AttendSegment& head, unsigned char* queries,
                                      float* team_part) {
    using Both = SomeThreads<2 * kGroup, 1>;
    int tile = 0;
    if (p.team && head.tiles == 0) {
      const AttendHeads heads = attend_heads(p, head.group);
      const int pitch = attend_pitch(p.dim);
      for (int i = threadIdx.x; i < heads.heads * pitch; i += 2 * kGroup) team_part[i] = i % pitch == pitch - 4 ? -CUDART_INF_F : 0.0f;
    }
    for (AttendSegment g = head; g.tiles; g = attend_next(p, rows, share, g, kTile)) {
      const AttendHeads heads = attend_heads(p, g.group);
      const int q0 = heads.head0 - heads.kv * p.group, base = g.n - p.drafts;
      Both::sync();  // (the queries before these, and what they gave, are no longer read)
      load_queries(queries, g.row, heads.kv, q0, heads.heads);
      fence_async_smem();
      mbar_arrive(smem_u32(&s.queries));
      // (where every draft sees all of the segment's tokens, the tree is not asked)
      const int t_begin = g.tile0 * kTile, t_end = t_begin + g.tiles * kTile;
      const bool planted = !draft_all_seen(p, t_begin, t_end, base);
      if (planted) draft_tree<2 * kGroup, Both>(p, tree, g.row, base);

      const int mine = row + (WIDE ? w * kGroup : 0);
      const int draft = (int)fast_div32(p.per, (uint32_t)(q0 + min(mine, heads.heads - 1)));
      const bool alive = mine < heads.heads, live = alive && !(planted && tree.from[draft] == kNever), busy = __any_sync(~0u, alive);
      m = -CUDART_INF_F;
      l = 0.0f;
      bool any = false;
      for (int i = WIDE ? 0 : w; i < g.tiles; i += WIDE ? 1 : 2) {
        const int t0 = (g.tile0 + i) * kTile;
        // (the tile's scores are there: so is what the copies say of it)
        wait(s.stop, smem_u32(&s.scores[w]), count & 1);
        const uint32_t* at = s.here[(tile + i) % kHereTiles];
        const uint32_t here[4] = {at[0], at[1], at[2], at[3]};
        // (the whole warp's, also where a wait gave up and the words are being written)
        const bool all = draft_all_seen(p, t0, t0 + kTile, base), mask = __any_sync(~0u, !all || (here[0] & here[1] & here[2] & here[3]) != ~0u);
        tcgen05_after_sync();
        if (busy) {
          if (mask || p.cap_out != 0.0f) prepare(draft, t0, base, all, here);
          item(!any);
        }
        tcgen05_before_sync();
        mbar_arrive(smem_u32(&s.weights[w]));
        ++count;
        any = true;
        if (mask) {
          wait(s.stop, smem_u32(&s.done[w]), (count - 1) & 1);
          tcgen05_after_sync();
          const bool bad = *static_cast<volatile uint32_t*>(&s.bad[(tile + i) % kHereTiles]) == (uint32_t)(tile + i) + 1;
          if (__all_sync(~0u, bad && !gave_up(s.stop))) {
            add_infinite(g, heads.kv, draft, alive, t0, base, all, here);
            tcgen05_before_sync();  // (the next product comes after this thread's next arrival)
          }
        }
      }
      if (any) wait(s.stop, smem_u32(&s.done[w]), (count - 1) & 1);
      tcgen05_after_sync();
      if (gave_up(s.stop)) l = CUDART_NAN_F;
      tile += g.tiles;

      const int part_pitch = attend_pitch(p.dim);
      float* part = p.team ? team_part : attend_part(p, share, g, threadIdx.x == 0);
      const int h = heads.head0 + mine;
      float top = m, total = l, c[2] = {1.0f, 1.0f};
      bool has[2] = {any, any};
      if (!WIDE) {
        s.part[w][row] = make_float2(m, l);
        Both::sync();  // (the other group's products are done as well)
        tcgen05_after_sync();
        has[0] = true;
        has[1] = g.tiles > 1;
        const float2 a = s.part[0][row], b = has[1] ? s.part[1][row] : make_float2(-CUDART_INF_F, 0.0f);
        top = fmaxf(a.x, b.x);
        c[0] = attend_weight(a.x, top);
        c[1] = attend_weight(b.x, top);
        total = a.y * c[0] + b.y * c[1];
      } else if (p.team) {
        Both::sync();  // (the other group's products have read what the part overwrites)
      }
      if (!live) {
        top = kPadding;
        total = 0.0f;
      }
      T* out = nullptr;
      float scale = 1.0f;
      if (part) {
        part += (h - heads.head0) * part_pitch;
        if (alive && (WIDE || w == 0)) {
          part[part_pitch - 4] = top;
          part[part_pitch - 3] = total;
        }
      } else if (alive) {
        const AttendPlace place = attend_place(p, g.row, h);
        out = static_cast<T*>(p.out) + place.out;
        if (WIDE || w == 0) {
          if (p.lse) p.lse[place.lse] = total == 0.0f ? -CUDART_INF_F : (top + log2f(total)) * CUDART_LN2_F;
          attend_note(p, g.row, h, top, total);
        }
        scale = total == 0.0f ? 0.0f : 1.0f / total;
      }
      if (busy) {
        const int half = WIDE ? DP : DP / 2, d0 = WIDE ? 0 : w * half;
        for (int d = d0; d < d0 + half && d < p.dim; d += 32) {
          float o[32];
          uint32_t x[32];
          if (WIDE) {
            tmem_load(x, tmem + S::kOut + w * 128 + d);
            tmem_wait_load(x);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(x[e]) * scale;
          } else {
            tmem_load(x, tmem + S::kOut + d);
            tmem_wait_load(x);
            const float a = c[0] * scale, b = c[1] * scale;
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = c[0] == 0.0f ? 0.0f : __uint_as_float(x[e]) * a;
            if (has[1]) {
              tmem_load(x, tmem + S::kOut + 128 + d);
              tmem_wait_load(x);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] += c[1] == 0.0f ? 0.0f : __uint_as_float(x[e]) * b;
            }
          }
          if (!(total > 0.0f)) {  // (no token, or a wait gave up)
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = total;
          }
          if (alive) write(o, part, out, d);
        }
      }
      tcgen05_before_sync();  // (what is next issued over O comes after a barrier of these threads)
    }
  }
};

template <class T, int DP, bool WIDE>
__global__ void __launch_bounds__(kThreads, 1) drafts_tc_kernel(const __grid_constant__ TcParams p) {
  using S = Shape<DP, WIDE>;
  extern __shared__ unsigned char s_raw[];
  unsigned char* s_mem = s_raw + ((1024 - smem_u32(s_raw) % 1024) % 1024);
  State& s = *reinterpret_cast<State*>(s_mem + S::kRest);
  DraftTree& tree = *reinterpret_cast<DraftTree*>(&s + 1);
  AttendRows& rows = *reinterpret_cast<AttendRows*>(&tree + 1);
  const int warp = threadIdx.x / 32;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kSlots; ++i) {
      mbar_init(smem_u32(&s.full[i]), CMDX_TMA ? 1 : kLoaders);
      mbar_init(smem_u32(&s.empty[i]), 1);
    }
    for (int i = 0; i < kHereTiles; ++i) s.bad[i] = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s.scores[i]), 1);
      mbar_init(smem_u32(&s.weights[i]), kGroup);
      mbar_init(smem_u32(&s.done[i]), 1);
    }
    mbar_init(smem_u32(&s.landed), 1);
    mbar_init(smem_u32(&s.queries), 2 * kGroup);
    mbar_init(smem_u32(&s.end), 1);
    s.stop = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 2 * kGroup / 32) tmem_alloc(smem_u32(&s.tmem), 512);
  wait_for_previous();
  let_next_start();
  AttendShare share;
  AttendSegment head;
  if (p.team) {
    head = attend_team(p, kTile, &share);
  } else {
    head.tiles = 0;  // (without work)
    if (attend_begin<T>(p, rows, kTile, &share)) head = attend_first(p, rows, share, kTile);
  }
  tcgen05_before_sync();
  __syncthreads();
  tcgen05_after_sync();
  const uint32_t tmem = *static_cast<volatile uint32_t*>(&s.tmem);
  const uint32_t queries = smem_u32(s_mem), ring = queries + S::kRing;
  float* team_part = reinterpret_cast<float*>(s_mem);  // (the queries and the ring have been read by then)
  if (warp < 2 * kGroup / 32) {
    Softmax<T, DP, WIDE> softmax(p, s, tree, tmem);
    softmax.run(rows, share, head, s_mem, team_part);
  } else if (warp == 2 * kGroup / 32) {
    issue<T, DP, WIDE>(p, s, rows, share, head, queries, ring, __shfl_sync(~0u, tmem, 0));
  } else {
    Loader<T, DP, WIDE> loader(p, s, ring);
    loader.run(rows, share, head);
  }
  tcgen05_before_sync();
  __syncthreads();
  tcgen05_after_sync();
  if (warp == 2 * kGroup / 32) tmem_free(tmem, 512);
  if (threadIdx.x == 0 && s.stop) report(p.status, CMD_CACHE_TIMEOUT);
  if (p.team) attend_join_team<T, kThreads>(p, head, attend_heads(p, head.group), team_part);
}

template <class T, int DP, bool WIDE>
cudaError_t launch(const TcParams& p, cudaStream_t stream) {
  static PerDevice ready;  // (static storage: zero before first use)
  static_assert(kSmem<DP, WIDE> <= 227 * 1024, "the CTA fits an SM");
  static_assert(Shape<DP, WIDE>::kRows * attend_pitch(DP) * 4 <= Shape<DP, WIDE>::kRest, "a team's part fits the queries and the ring");
  const cudaError_t e = allow_smem(drafts_tc_kernel<T, DP, WIDE>, kSmem<DP, WIDE>, ready);
  if (e != cudaSuccess) return e;
  return attend_launch<T>(drafts_tc_kernel<T, DP, WIDE>, p, 4, 152, kThreads, kSmem<DP, WIDE>, kTile, stream);
}
template <class T>
cudaError_t launch_type(const TcParams& p, cudaStream_t stream) {
  const bool wide = p.block_heads > kGroup;
  if (p.dim <= 64) return wide ? launch<T, 64, true>(p, stream) : launch<T, 64, false>(p, stream);
  return wide ? launch<T, 128, true>(p, stream) : launch<T, 128, false>(p, stream);
}

}  // namespace

#if CMDX_TMA
bool drafts_tma_fits(int64_t page_size, const int64_t (&sizes)[4], const int64_t (&k_st)[4], const int64_t (&v_st)[4]) {
  if (page_size % 8 || sizes[0] < 1) return false;
  for (int d = 0; d < 3; ++d)
    for (const int64_t st : {k_st[d], v_st[d]})
      if (sizes[d] > 1 && (st == 0 || st >= (int64_t(1) << 38))) return false;
  return tensor_map_encoder() != nullptr;
}

cudaError_t drafts_tma_launch(int dtype, const DraftParams& d, cudaStream_t stream) {
  TcParams p;
  const cudaError_t e = pool_maps(dtype, d, &p);
  if (e != cudaSuccess) return e;
  return dtype == CMD_F16 ? launch_type<__half>(p, stream) : launch_type<__nv_bfloat16>(p, stream);
}
#else
cudaError_t drafts_tc_launch(int dtype, const DraftParams& d, cudaStream_t stream) {
  TcParams p = {};
  static_cast<DraftParams&>(p) = d;
  return dtype == CMD_F16 ? launch_type<__half>(p, stream) : launch_type<__nv_bfloat16>(p, stream);
}
#endif

}  // namespace cmdx
