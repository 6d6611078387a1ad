// cache_rope.cu - rotary positions, and the append of new tokens to a paged
// cache.
//
// Pair (a, b) of a head becomes scale (a cos t - b sin t, b cos t + a sin t),
// with t = position * turns / 2^64 of a turn: a 64-bit wrapping product is
// the angle modulo a turn, exactly, and its upper 32 bits, read as a signed
// number, are half turns in [-1, 1) for sincospi. Backward is the transposed
// rotation, t negated.
//
// Bound by memory: every element is read and written once, at about two
// fused multiply-adds each. A CTA takes a token, or several where heads are
// few, and all of their heads (queries, keys, values), so that an angle is
// computed once, into shared memory, while the elements are already on their
// way: each thread issues its loads first. A thread keeps two 16-byte places
// within the head (in the half layout's rotated part, elements and their
// partners n_pairs further) and goes over heads.
//
// Measured: 4 x 4096 tokens of 40 heads of 128 (bf16) 52.8 us, 6.36 TB/s, 93%
// of the copy peak (a library copy of as many bytes: 54.0 us), with 69% of the
// issue slots taken; 3 x 1537 tokens of 24 heads of 80 (f32, 32 rotated) 13.6
// us, 77%, 2.5 us of it a launch's fixed part; 7 prompts of 1171 tokens into a
// cache (f16, 24 + 2 x 8 heads of 128) 30.0 us, 82%; one token of 16 rows 3.1
// us, all of it fixed. A head is accessed in pieces of one size, so heads of 72
// take 40.9 us (68%) in 8-byte ones, and with 36 rotated 63.2 (44%) in 4-byte
// ones, bound by their instructions.
#include "cache_common.cuh"

namespace cmdx {

namespace {

// Heads a thread has in flight, by the bytes of an access (0: an element) and
// of an element. Measured on 4 x 4096 tokens of 40 bf16 heads: of 128 elements
// (16 bytes, before divisions and strides were narrowed) 2, 56.2 us; 3, 55.7;
// 4, 61.5; of 72 (8 bytes) 3, 54.3; 4, 44.3; 5, 40.9; of 72 with 36 rotated (4
// bytes) 3, 72.1; 4, 69.8; 6, 63.3. f32 heads of 72 (8 bytes) 3, 76.4; 4, 73.4;
// 5, 101.7 (spills).
__host__ __device__ constexpr int rope_loads(int bytes, int element) {
  return bytes == 16 ? 3 : bytes == 8 ? (element == 2 ? 5 : 4) : bytes == 4 ? 6 : 4;
}

// Two 16-bit numbers of a word, and back.
template <class T>
__device__ __forceinline__ float2 unpack(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack<__half>(uint32_t w) { return __half22float2(*reinterpret_cast<__half2*>(&w)); }
template <>
__device__ __forceinline__ float2 unpack<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <class T>
__device__ __forceinline__ uint32_t pack(float x, float y);
template <>
__device__ __forceinline__ uint32_t pack<__half>(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack<__nv_bfloat16>(float x, float y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The pair (a, b) turned: (a c - b s, b c + a s).
__device__ __forceinline__ float2 turned(float a, float b, float2 t) {
  return make_float2(fmaf(a, t.x, -(b * t.y)), fmaf(b, t.x, a * t.y));
}

// Where pair i's cosine and sine lie among the n_pairs of a token, which
// threads read NP at a time: 16 bytes each, next to the other threads' (groups
// = n_pairs / NP of them), so that no two meet in a bank.
template <int NP>
__device__ __forceinline__ int turn_at(int i, int groups) {
  if (NP == 1) return i;
  const int k = i % NP;
  return (k / 2 * groups + i / NP) * 2 + k % 2;
}

// The cosines and sines of one place: pairs 2 i and 2 i + 1 of its NP.
template <int NP>
struct Turns {
  const float2* of_token;
  int group, groups;
  __device__ __forceinline__ float4 two(int i) const {
    return *reinterpret_cast<const float4*>(of_token + turn_at<NP>(group * NP + 2 * i, groups));
  }
  __device__ __forceinline__ float2 one() const { return of_token[group]; }
};

// VE elements of a head: a vector of 16, 8 or 4 bytes when VEC, else up to VE
// of them one by one.
template <class T, int VE, bool VEC>
struct Chunk {
  T x[VE];
  __device__ __forceinline__ void load(const T* p, int n) {
#pragma unroll
    for (int i = 0; i < VE; ++i)
      if (i < n) x[i] = p[i];
  }
  __device__ __forceinline__ void store(T* p, int n) const {
#pragma unroll
    for (int i = 0; i < VE; ++i)
      if (i < n) p[i] = x[i];
  }
  // this chunk's element paired with another's (VE 1)
  __device__ __forceinline__ void turn_with(Chunk& o, const Turns<1>& t) {
    const float2 y = turned(to_float(x[0]), to_float(o.x[0]), t.one());
    x[0] = from_float<T>(y.x);
    o.x[0] = from_float<T>(y.y);
  }
  // neighbours paired (VE 2)
  __device__ __forceinline__ void turn(const Turns<1>& t) {
    const float2 y = turned(to_float(x[0]), to_float(x[VE - 1]), t.one());
    x[0] = from_float<T>(y.x);
    x[VE - 1] = from_float<T>(y.y);
  }
};
template <class T, int VE>
struct Chunk<T, VE, true> {
  static constexpr int kWords = VE * (int)sizeof(T) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p, int) {
    if constexpr (kWords == 4) {
      const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p));
      w[0] = v.x;
      w[1] = v.y;
      w[2] = v.z;
      w[3] = v.w;
    } else if constexpr (kWords == 2) {
      const uint2 v = __ldcs(reinterpret_cast<const uint2*>(p));
      w[0] = v.x;
      w[1] = v.y;
    } else {
      w[0] = __ldcs(reinterpret_cast<const uint32_t*>(p));
    }
  }
  __device__ __forceinline__ void store(T* p, int) const {
    if constexpr (kWords == 4) __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
    else if constexpr (kWords == 2) __stcs(reinterpret_cast<uint2*>(p), make_uint2(w[0], w[1]));
    else __stcs(reinterpret_cast<uint32_t*>(p), w[0]);
  }
  __device__ __forceinline__ void turn_with(Chunk& o, const Turns<VE>& t) {
    // two pairs at a time: of one word, or of two
#pragma unroll
    for (int i = 0; i < VE / 2; ++i) {
      const float4 c = t.two(i);
      if constexpr (sizeof(T) == 4) {
        const float2 y = turned(__uint_as_float(w[2 * i]), __uint_as_float(o.w[2 * i]), make_float2(c.x, c.y));
        const float2 z = turned(__uint_as_float(w[2 * i + 1]), __uint_as_float(o.w[2 * i + 1]), make_float2(c.z, c.w));
        w[2 * i] = __float_as_uint(y.x);
        o.w[2 * i] = __float_as_uint(y.y);
        w[2 * i + 1] = __float_as_uint(z.x);
        o.w[2 * i + 1] = __float_as_uint(z.y);
      } else {
        const float2 a = unpack<T>(w[i]), b = unpack<T>(o.w[i]);
        const float2 y = turned(a.x, b.x, make_float2(c.x, c.y)), z = turned(a.y, b.y, make_float2(c.z, c.w));
        w[i] = pack<T>(y.x, z.x);
        o.w[i] = pack<T>(y.y, z.y);
      }
    }
  }
  // pair i of this chunk turned
  __device__ __forceinline__ void turn_pair(int i, float2 c) {
    if constexpr (sizeof(T) == 4) {
      const float2 y = turned(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]), c);
      w[2 * i] = __float_as_uint(y.x);
      w[2 * i + 1] = __float_as_uint(y.y);
    } else {
      const float2 a = unpack<T>(w[i]);
      const float2 y = turned(a.x, a.y, c);
      w[i] = pack<T>(y.x, y.y);
    }
  }
  __device__ __forceinline__ void turn(const Turns<VE / 2>& t) {
    if constexpr (VE == 2) {
      turn_pair(0, t.one());
    } else {
#pragma unroll
      for (int i = 0; i < VE / 4; ++i) {
        const float4 c = t.two(i);
        turn_pair(2 * i, make_float2(c.x, c.y));
        turn_pair(2 * i + 1, make_float2(c.z, c.w));
      }
    }
  }
};

// How a launch's CTAs are made up: `units` threads to a head, `slots` heads at
// once, `tokens` tokens.
struct RopeShape {
  int units, slots, tokens;
  FastDiv32 by_units, by_slots, by_pairs;
};

// An index times a stride: strides of the vector kernels are below 2^31 (see
// rope_launch's vec), which makes it one instruction.
template <bool NARROW>
__device__ __forceinline__ int64_t stride_of(int64_t index, int64_t stride) {
  return NARROW ? (int64_t)(int32_t)index * (int32_t)stride : index * stride;
}

template <class T, int VE, bool VEC, bool HALF>
__global__ void __launch_bounds__(512, 2) rope_kernel(const __grid_constant__ RopeParams p, const RopeShape shape) {
  constexpr int NP = HALF ? VE : VE / 2;  // pairs of a thread's place
  constexpr int kRopeLoads = rope_loads(VEC ? VE * (int)sizeof(T) : 0, sizeof(T));
  extern __shared__ __align__(16) float2 s_turn[];  // [tokens][n_pairs]: cosine and sine
  const int tid = threadIdx.x;
  const int column = (int)fast_div32(shape.by_units, tid), unit = tid - column * shape.units;
  const int mine = (int)fast_div32(shape.by_slots, column), slot = column - mine * shape.slots;
  const int rot = 2 * p.n_pairs, groups = p.n_pairs / NP;
  // the thread's two places in a head: their first elements, the elements
  // they have (fewer at an odd head's end, 0 for none), and whether they are
  // rotated (in the half layout: with one another)
  int e[2], count[2];
  bool turn[2];
  const int halves = HALF ? p.n_pairs / VE : 0;
  if (HALF && unit < halves) {
    e[0] = unit * VE;
    e[1] = e[0] + p.n_pairs;
    turn[0] = turn[1] = true;
  } else {
    const int from = HALF ? rot : 0, chunks = (p.dim - from + VE - 1) / VE;
    e[0] = from + (unit - halves) * VE;
    e[1] = e[0] + (chunks + 1) / 2 * VE;
    turn[0] = e[0] < rot;
    turn[1] = e[1] < rot;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) count[i] = max(0, min(VE, p.dim - e[i]));

  wait_for_previous();
  let_next_start();

  const int64_t first = (int64_t)blockIdx.x * shape.tokens;
  const int64_t all = p.batch * p.tokens;
  // the CTA's angles, one to a thread: their position and turns are read now
  const auto angle_position = [&](int i) {
    const uint32_t at = (uint32_t)first + fast_div32(shape.by_pairs, i);
    const int64_t ob = fast_div32(p.per_batch, at);
    return at < all ? p.positions[ob * p.pos_st[0] + (at - ob * p.tokens) * p.pos_st[1]] : 0;
  };
  const int angles = shape.tokens * p.n_pairs;
  int32_t angle_at = 0;
  uint64_t angle_turns = 0;
  if (tid < angles) {
    angle_at = angle_position(tid);
    angle_turns = p.turns[tid - fast_div32(shape.by_pairs, tid) * p.n_pairs];
  }
  const bool works = mine < shape.tokens && first + mine < all;
  const uint32_t token = works ? (uint32_t)(first + mine) : 0;
  const int64_t b = fast_div32(p.per_batch, token);
  const int64_t t = token - b * p.tokens;

  // where the cache takes the token: the page and slot, or none
  int32_t page = -1, page_slot = 0;
  if (p.columns >= 0 && works) {
    const int32_t position = p.positions[b * p.pos_st[0] + t * p.pos_st[1]];
    const int32_t row = p.rows ? p.rows[t * p.rows_st] : (int32_t)t;
    if (position >= 0) {
      const uint32_t column = fast_div32(p.page, (uint32_t)position);
      page_slot = position - (int32_t)(column * p.page.d);
      if (row < 0 || row >= p.n_rows || column >= (uint32_t)p.columns) {
        if (unit == 0) report(p.status, CMD_CACHE_BAD_INDEX);
      } else {
        page = p.tables[row * p.table_st[0] + column * p.table_st[1]];
        if (page < 0 || page >= p.n_pages) {
          page = -1;
          if (unit == 0) report(p.status, CMD_CACHE_BAD_PAGE);
        }
      }
    }
  }

  for (int h0 = 0; h0 < p.heads; h0 += kRopeLoads * shape.slots) {
    Chunk<T, VE, VEC> x[kRopeLoads][2];
    T* dst[kRopeLoads];
    bool rotate[kRopeLoads];
#pragma unroll
    for (int i = 0; i < kRopeLoads; ++i) {
      int h = h0 + i * shape.slots + slot;
      dst[i] = nullptr;
      rotate[i] = false;
      if (!works || h >= p.heads) continue;
      int j = 0;
      while (h >= p.s[j].heads) h -= p.s[j++].heads;
      const RopeStream& s = p.s[j];
      const T* src = static_cast<const T*>(s.in) + stride_of<VEC>(b, s.in_st[0]) + stride_of<VEC>(t, s.in_st[1]) +
                     stride_of<VEC>(h, s.in_st[2]);
      if (s.cache) {
        if (page < 0) continue;
        dst[i] = static_cast<T*>(s.out) + stride_of<VEC>(page, s.out_st[0]) + stride_of<VEC>(page_slot, s.out_st[1]) +
                 stride_of<VEC>(h, s.out_st[2]);
      } else {
        dst[i] = static_cast<T*>(s.out) + stride_of<VEC>(b, s.out_st[0]) + stride_of<VEC>(t, s.out_st[1]) +
                 stride_of<VEC>(h, s.out_st[2]);
      }
      rotate[i] = s.rotate;
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (count[k]) x[i][k].load(src + e[k], count[k]);
    }
    if (h0 == 0) {
      for (int i = tid; i < angles; i += blockDim.x) {
        if (i != tid) {
          angle_at = angle_position(i);
          angle_turns = p.turns[i - fast_div32(shape.by_pairs, i) * p.n_pairs];
        }
        const uint64_t phase = (uint64_t)(int64_t)angle_at * angle_turns;
        float s, c;
        sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &s, &c);
        const int k = (int)fast_div32(shape.by_pairs, i);
        s_turn[k * p.n_pairs + turn_at<NP>(i - k * p.n_pairs, groups)] = make_float2(c * p.scale, s * p.sine_scale);
      }
      __syncthreads();
    }
    // (a thread without a token has no place here, and no dst)
    const float2* turns = s_turn + mine * p.n_pairs;
#pragma unroll
    for (int i = 0; i < kRopeLoads; ++i) {
      if (!dst[i]) continue;
      if constexpr (HALF) {
        if (rotate[i] && turn[0]) x[i][0].turn_with(x[i][1], Turns<NP>{turns, e[0] / VE, groups});
      } else {
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (rotate[i] && turn[k]) x[i][k].turn(Turns<NP>{turns, e[k] / VE, groups});
      }
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (count[k]) x[i][k].store(dst[i] + e[k], count[k]);
    }
  }
}

template <class T, int VE, bool VEC, bool HALF>
cudaError_t launch(const RopeParams& p, cudaStream_t stream) {
  RopeShape s;
  constexpr int kRopeLoads = rope_loads(VEC ? VE * (int)sizeof(T) : 0, sizeof(T));
  const int halves = HALF ? p.n_pairs / VE : 0, chunks = (p.dim - (HALF ? 2 * p.n_pairs : 0) + VE - 1) / VE;
  s.units = halves + (chunks + 1) / 2;
  // as many heads at once as leave every thread kRopeLoads of them, or fewer, within 512 threads
  s.slots = 512 / s.units;
  const int rounds = (p.heads + s.slots * kRopeLoads - 1) / (s.slots * kRopeLoads);
  s.slots = (p.heads + rounds * kRopeLoads - 1) / (rounds * kRopeLoads);
  // the tokens that fill whole warps best, within 160 threads (224 were
  // slower than 112 by 2.6%), where there are enough to give every SM eight CTAs
  const int64_t all = p.batch * p.tokens, each = all / (152 * 8);
  const int one = s.units * s.slots;
  s.tokens = 1;
  for (int n = 2; n * one <= 160 && n <= each; ++n) {
    const auto padded = [&](int k) { return (k * one + 31) / 32 * 32; };
    if ((int64_t)n * padded(s.tokens) > (int64_t)s.tokens * padded(n)) s.tokens = n;
  }
  const int threads = (s.units * s.slots * s.tokens + 31) / 32 * 32;
  s.by_units = fast_div_by(s.units);
  s.by_slots = fast_div_by(s.slots);
  s.by_pairs = fast_div_by(p.n_pairs);
  return launch_chained(rope_kernel<T, VE, VEC, HALF>, (int)((all + s.tokens - 1) / s.tokens), threads,
                    (size_t)s.tokens * p.n_pairs * sizeof(float2), stream, p, s);
}

template <class T, int VE, bool VEC>
cudaError_t launch_layout(int layout, const RopeParams& p, cudaStream_t stream) {
  constexpr int kHalf = VEC ? VE : 1;  // (one by one: single elements in the half layout, pairs in the other)
  return layout == CMD_ROPE_HALF ? launch<T, kHalf, VEC, true>(p, stream) : launch<T, VE, VEC, false>(p, stream);
}

// The access: 16, 8 or (16-bit types) 4 bytes, else element by element.
// Measured on 4 x 4096 tokens of 40 bf16 heads: of 80 elements, all rotated (16
// bytes) 38.0 us; of 72 (8 bytes) 40.9, of 72 with 36 rotated (4 bytes) 63.3,
// both 140 element by element.
template <class T>
cudaError_t launch_type(int layout, int bytes, const RopeParams& p, cudaStream_t stream) {
  constexpr int ES = sizeof(T);
  if (bytes == 16) return launch_layout<T, 16 / ES, true>(layout, p, stream);
  if (bytes == 8) return launch_layout<T, 8 / ES, true>(layout, p, stream);
  if constexpr (ES == 2)
    if (bytes == 4) return launch_layout<T, 2, true>(layout, p, stream);
  return launch_layout<T, 2, false>(layout, p, stream);
}

}  // namespace

cudaError_t rope_launch(int dtype, int layout, int bytes, const RopeParams& p, cudaStream_t stream) {
  switch (dtype) {
    case CMD_F32: return launch_type<float>(layout, bytes, p, stream);
    case CMD_F16: return launch_type<__half>(layout, bytes, p, stream);
    case CMD_BF16: return launch_type<__nv_bfloat16>(layout, bytes, p, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace cmdx
