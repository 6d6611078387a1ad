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
// fused multiply-adds each. One CTA takes one token and all of its heads
// (queries, keys, values), so a token's angles are computed once, by n_pairs
// of its threads, into shared memory, while the token's elements are already
// on their way: each thread issues its loads first. A thread keeps one place
// within the head (a vector of 16 bytes, in the half layout with its partner
// n_pairs further) and goes over heads, so its cosines stay in registers.
#include "cache_common.cuh"

namespace cmdx {

namespace {

constexpr int kRopeLoads = 4;  // heads a thread has in flight

// VE elements at p, in one 16-byte access when VEC, else the first n of them one by one.
template <class T, int VE, bool VEC>
struct Chunk {
  T x[VE];
  __device__ __forceinline__ void load(const T* p, int n) {
    if constexpr (VEC) {
      *reinterpret_cast<uint4*>(x) = __ldcs(reinterpret_cast<const uint4*>(p));
    } else {
#pragma unroll
      for (int i = 0; i < VE; ++i)
        if (i < n) x[i] = p[i];
    }
  }
  __device__ __forceinline__ void store(T* p, int n) const {
    if constexpr (VEC) {
      __stcs(reinterpret_cast<uint4*>(p), *reinterpret_cast<const uint4*>(x));
    } else {
#pragma unroll
      for (int i = 0; i < VE; ++i)
        if (i < n) p[i] = x[i];
    }
  }
};

template <class T, int VE, bool VEC, bool HALF>
__global__ void __launch_bounds__(512) rope_kernel(const __grid_constant__ RopeParams p, int units, int head_slots) {
  __shared__ float2 s_turn[CMD_CACHE_MAX_DIM / 2];
  const int tid = threadIdx.x;
  const int unit = tid % units, slot = tid / units;
  const bool works = slot < head_slots;
  const int rot = 2 * p.n_pairs;
  // the thread's place in a head: its first element, and whether it has a
  // partner n_pairs further (half layout, rotated part)
  const int rot_units = (HALF ? p.n_pairs : rot) / VE;
  const bool in_rot = unit < rot_units;
  const int e0 = in_rot ? unit * VE : rot + (unit - rot_units) * VE;
  const int pair0 = HALF ? e0 : e0 / 2;
  const int count = p.dim - e0 < VE ? p.dim - e0 : VE;  // (a head's odd last element)

  pdl_wait();
  pdl_trigger();

  const int64_t token = blockIdx.x;
  const int64_t b = p.batch == 1 ? 0 : token / p.tokens;
  const int64_t t = token - b * p.tokens;
  const int32_t position = p.positions[b * p.pos_st[0] + t * p.pos_st[1]];

  // where the cache takes the token: the offset's page and slot, or none
  int32_t page = -1, page_slot = 0;
  if (p.columns >= 0) {
    const int32_t row = p.rows ? p.rows[t * p.rows_st] : (int32_t)t;
    if (position >= 0) {
      const uint32_t column = fast_div32(p.page, (uint32_t)position);
      page_slot = position - (int32_t)(column * p.page.d);
      if (row < 0 || row >= p.n_rows || column >= (uint32_t)p.columns) {
        if (tid == 0) report(p.status, CMD_CACHE_BAD_INDEX);
      } else {
        page = p.tables[row * p.table_st[0] + column * p.table_st[1]];
        if (page < 0 || page >= p.n_pages) {
          page = -1;
          if (tid == 0) report(p.status, CMD_CACHE_BAD_PAGE);
        }
      }
    }
  }

  auto turn_angles = [&]() {
    for (int i = tid; i < p.n_pairs; i += blockDim.x) {
      const uint64_t phase = (uint64_t)(int64_t)position * p.turns[i];
      float s, c;
      sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &s, &c);
      s_turn[i] = make_float2(c * p.scale, s * p.sine_scale);
    }
    __syncthreads();
  };

  constexpr int NP = HALF ? VE : VE / 2;  // pairs of one thread
  float cs[NP], sn[NP];
  for (int h0 = 0; h0 < p.heads; h0 += kRopeLoads * head_slots) {
    Chunk<T, VE, VEC> a[kRopeLoads], c[kRopeLoads];
    T* dst[kRopeLoads];
    bool turn[kRopeLoads];
#pragma unroll
    for (int i = 0; i < kRopeLoads; ++i) {
      int h = h0 + i * head_slots + slot;
      dst[i] = nullptr;
      turn[i] = false;
      if (!works || h >= p.heads) continue;
      int j = 0;
      while (h >= p.s[j].heads) h -= p.s[j++].heads;
      const RopeStream& s = p.s[j];
      const T* src = static_cast<const T*>(s.in) + b * s.in_st[0] + t * s.in_st[1] + h * s.in_st[2];
      if (s.cache) {
        if (page < 0) continue;
        dst[i] = static_cast<T*>(s.out) + page * s.out_st[0] + page_slot * s.out_st[1] + h * s.out_st[2];
      } else {
        dst[i] = static_cast<T*>(s.out) + b * s.out_st[0] + t * s.out_st[1] + h * s.out_st[2];
      }
      turn[i] = s.rotate;
      a[i].load(src + e0, count);
      if (HALF && in_rot) c[i].load(src + e0 + p.n_pairs, count);
    }
    if (h0 == 0) {
      turn_angles();
      if (in_rot) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const float2 w = s_turn[pair0 + i];
          cs[i] = w.x;
          sn[i] = w.y;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kRopeLoads; ++i) {
      if (!dst[i]) continue;
      if (turn[i] && in_rot) {
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          const float x = to_float(HALF ? a[i].x[k] : a[i].x[(2 * k) % VE]);
          const float y = to_float(HALF ? c[i].x[k] : a[i].x[(2 * k + 1) % VE]);
          const T u = from_float<T>(fmaf(x, cs[k], -(y * sn[k])));
          const T w = from_float<T>(fmaf(y, cs[k], x * sn[k]));
          if (HALF) {
            a[i].x[k] = u;
            c[i].x[k] = w;
          } else {
            a[i].x[(2 * k) % VE] = u;
            a[i].x[(2 * k + 1) % VE] = w;
          }
        }
      }
      a[i].store(dst[i] + e0, count);
      if (HALF && in_rot) c[i].store(dst[i] + e0 + p.n_pairs, count);
    }
  }
}

template <class T, int VE, bool VEC, bool HALF>
cudaError_t launch(const RopeParams& p, cudaStream_t stream) {
  const int rot = 2 * p.n_pairs;
  const int units = (HALF ? p.n_pairs : rot) / VE + (p.dim - rot + VE - 1) / VE;
  // threads: as many heads at once as leave every thread kRopeLoads of them or fewer, within 512 threads
  int slots = 512 / units;
  if (slots < 1) slots = 1;
  const int rounds = (p.heads + slots * kRopeLoads - 1) / (slots * kRopeLoads);
  slots = (p.heads + rounds * kRopeLoads - 1) / (rounds * kRopeLoads);
  const int threads = (units * slots + 31) / 32 * 32;
  return launch_pdl(rope_kernel<T, VE, VEC, HALF>, (int)(p.tokens * p.batch), threads, 0, stream, p, units, slots);
}

template <class T>
cudaError_t launch_type(int layout, bool vec, const RopeParams& p, cudaStream_t stream) {
  constexpr int VE = 16 / sizeof(T);
  if (layout == CMD_ROPE_HALF)
    return vec ? launch<T, VE, true, true>(p, stream) : launch<T, 1, false, true>(p, stream);
  return vec ? launch<T, VE, true, false>(p, stream) : launch<T, 2, false, false>(p, stream);
}

}  // namespace

cudaError_t rope_launch(int dtype, int layout, bool vec, const RopeParams& p, cudaStream_t stream) {
  switch (dtype) {
    case CMD_F32: return launch_type<float>(layout, vec, p, stream);
    case CMD_F16: return launch_type<__half>(layout, vec, p, stream);
    case CMD_BF16: return launch_type<__nv_bfloat16>(layout, vec, p, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace cmdx
