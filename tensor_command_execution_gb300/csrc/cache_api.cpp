// cache_api.cpp - the C ABI of cmd_cache.h: argument checks and launches of
// the paged cache's operators.
#include "../../include/cmd_cache.h"

#include <algorithm>
#include <cmath>
#include <cstring>
#include <initializer_list>
#include <string>
#include <utility>

#include "cache_internal.h"

namespace cmdx {
cmd_status host_fail(cmd_status s, const std::string& msg);
}

namespace {

using cmdx::host_fail;

int elem_size(int dt) { return (dt == CMD_F16 || dt == CMD_BF16) ? 2 : 4; }
bool is_float(int dt) { return dt == CMD_F32 || dt == CMD_F16 || dt == CMD_BF16; }

// A failed check, with its message; thrown inside this file only.
struct Failure {
  cmd_status status;
  std::string message;
};
// (a macro: the message is put together only when the check fails)
#define NEED(ok, status, msg) \
  do {                        \
    if (!(ok)) throw Failure{status, msg}; \
  } while (0)

// Runs f, turning failures (and anything else thrown) into a status.
template <class F>
cmd_status guarded(F f) {
  try {
    return f();
  } catch (const Failure& x) {
    try {
      return host_fail(x.status, x.message);
    } catch (...) {
      return x.status;
    }
  } catch (...) {
    return CMD_ERR_NOMEM;
  }
}

cmd_status launched(cudaError_t e) {
  return e == cudaSuccess ? CMD_OK : host_fail(CMD_ERR_CUDA, cudaGetErrorString(e));
}

// Largest element offset of a view, and an overflow-safe bound on it.
int64_t last_offset(const cmd_operand& o, const char* name) {
  __int128 last = 0;
  for (int d = 0; d < o.rank; ++d) {
    if (o.sizes[d] == 0) return -1;
    last += (__int128)(o.sizes[d] - 1) * o.strides[d];
  }
  NEED(last < ((__int128)1 << 60), CMD_ERR_SHAPE, std::string(name) + " extends past the address space");
  return (int64_t)last;
}

bool empty(const cmd_operand& o) {
  for (int d = 0; d < o.rank; ++d)
    if (o.sizes[d] == 0) return true;
  return false;
}

// Checks that hold for every operand: rank, sizes, strides, pointer. They come
// before anything else that walks an operand's dims.
void check(const cmd_operand& o, const char* name, int rank, bool has_dim = false) {
  NEED(o.rank == rank, CMD_ERR_SHAPE, std::string(name) + " has rank " + std::to_string(o.rank) + ", not " +
                                          std::to_string(rank));
  for (int d = 0; d < rank; ++d) {
    NEED(o.sizes[d] >= 0, CMD_ERR_SHAPE, std::string(name) + " has a negative size");
    NEED(o.strides[d] >= 0, CMD_ERR_SHAPE, std::string(name) + " has a negative stride (strides must be >= 0)");
  }
  NEED(o.ptr || empty(o), CMD_ERR_NULL, std::string(name) + " is NULL");
  NEED(reinterpret_cast<uintptr_t>(o.ptr) % elem_size(o.dtype) == 0, CMD_ERR_ALIGN,
       std::string(name) + " is not aligned to its element size");
  if (has_dim)
    NEED(o.sizes[rank - 1] <= 1 || o.strides[rank - 1] == 1 || empty(o), CMD_ERR_SHAPE,
         std::string(name) + " needs a unit stride along its last dim");
  last_offset(o, name);
}

void check_type(const cmd_operand& o, const char* name, int dtype) {
  NEED(o.dtype == dtype, CMD_ERR_TYPE, std::string(name) + " has another element type than its call needs");
}

void check_sizes(const cmd_operand& o, const char* name, const int64_t* sizes) {
  for (int d = 0; d < o.rank; ++d)
    NEED(o.sizes[d] == sizes[d], CMD_ERR_SHAPE, std::string(name) + " has size " + std::to_string(o.sizes[d]) +
                                                    " in dim " + std::to_string(d) + ", not " + std::to_string(sizes[d]));
}

// Dims by increasing stride.
template <class F>
void sort_dims(int* order, int n, F stride) {
  for (int i = 1; i < n; ++i)
    for (int j = i; j > 0 && stride(order[j]) < stride(order[j - 1]); --j) std::swap(order[j], order[j - 1]);
}

// An output's elements must be distinct: with its dims by increasing stride,
// each stride passes everything below it.
void check_distinct(const cmd_operand& o, const char* name) {
  int order[CMD_MAX_RANK], n = 0;
  for (int d = 0; d < o.rank; ++d) {
    if (o.sizes[d] == 0) return;
    if (o.sizes[d] > 1) order[n++] = d;
  }
  sort_dims(order, n, [&](int d) { return o.strides[d]; });
  int64_t reach = 0;
  for (int i = 0; i < n; ++i) {
    const int d = order[i];
    NEED(o.strides[d] > reach, CMD_ERR_ALIAS, std::string(name) + " is written and overlaps itself");
    reach += (o.sizes[d] - 1) * o.strides[d];
  }
}

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
};
Range range_of(const cmd_operand& o) {
  if (!o.ptr || empty(o)) return {0, 0};
  int64_t last = 0;
  for (int d = 0; d < o.rank; ++d) last += (o.sizes[d] - 1) * o.strides[d];
  const uintptr_t a = reinterpret_cast<uintptr_t>(o.ptr);
  return {a, a + (uintptr_t)(last + 1) * elem_size(o.dtype)};
}
bool meet(const Range& a, const Range& b) { return a.lo < b.hi && b.lo < a.hi; }

bool same_view(const cmd_operand& a, const cmd_operand& b) {
  if (a.ptr != b.ptr || a.rank != b.rank || a.dtype != b.dtype) return false;
  for (int d = 0; d < a.rank; ++d)
    if (a.sizes[d] != b.sizes[d] || (a.sizes[d] > 1 && a.strides[d] != b.strides[d])) return false;
  return true;
}

// Whether two views of one shape interleave without meeting: equal strides,
// and bases less than a stride apart along some dim (keys and values in one
// tensor, say).
bool interleaved(const cmd_operand& a, const cmd_operand& b) {
  if (a.rank != b.rank || a.dtype != b.dtype) return false;
  for (int d = 0; d < a.rank; ++d)
    if (a.strides[d] != b.strides[d] && a.sizes[d] > 1 && b.sizes[d] > 1) return false;
  const int64_t es = elem_size(a.dtype);
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.ptr), pb = reinterpret_cast<uintptr_t>(b.ptr);
  const uintptr_t lo = std::min(pa, pb), hi = std::max(pa, pb);
  if ((hi - lo) % es) return false;
  const int64_t apart = (int64_t)((hi - lo) / es);
  const cmd_operand& first = pa <= pb ? a : b;
  const cmd_operand& second = pa <= pb ? b : a;
  // the dims with strides up to the distance end before it; together with the
  // second view's, and the distance, they fit the strides above, in turn
  int64_t below1 = 0, below2 = 0;
  int order[CMD_MAX_RANK], n = 0;
  for (int d = 0; d < a.rank; ++d) {
    if (std::max(first.sizes[d], second.sizes[d]) <= 1) continue;
    const int64_t st = first.sizes[d] > 1 ? first.strides[d] : second.strides[d];
    if (st <= apart) {
      below1 += (first.sizes[d] - 1) * st;
      below2 += (second.sizes[d] - 1) * st;
    } else {
      order[n++] = d;
    }
  }
  if (below1 >= apart) return false;
  auto stride = [&](int d) { return first.sizes[d] > 1 ? first.strides[d] : second.strides[d]; };
  sort_dims(order, n, stride);
  int64_t reach = apart + below2;
  for (int i = 0; i < n; ++i) {
    const int d = order[i];
    if (stride(d) <= reach) return false;
    reach += (std::max(first.sizes[d], second.sizes[d]) - 1) * stride(d);
  }
  return true;
}

void check_apart(const cmd_operand& out, const char* out_name, const cmd_operand& in, const char* in_name,
                 bool in_place = false) {
  if (!out.ptr || !in.ptr || !meet(range_of(out), range_of(in))) return;
  if (in_place && same_view(out, in)) return;
  if (interleaved(out, in)) return;
  throw Failure{CMD_ERR_ALIAS, std::string(out_name) + " overlaps " + in_name};
}

// Whether rows of a view may be accessed `bytes` at a time.
bool vector_rows(const cmd_operand& o, int bytes) {
  const int es = elem_size(o.dtype);
  if (reinterpret_cast<uintptr_t>(o.ptr) % bytes) return false;
  for (int d = 0; d + 1 < o.rank; ++d)
    if (o.sizes[d] > 1 && o.strides[d] * es % bytes) return false;
  return true;
}

void check_rope(const cmd_rope_spec& r, int64_t dim) {
  NEED(r.layout == CMD_ROPE_HALF || r.layout == CMD_ROPE_INTERLEAVED, CMD_ERR_ARG, "unknown rope layout");
  NEED(r.n_pairs >= 0 && 2 * (int64_t)r.n_pairs <= dim, CMD_ERR_SHAPE, "more rotated elements than the head has");
  NEED(std::isfinite(r.scale), CMD_ERR_ARG, "the rope scale is not finite");
  if (r.n_pairs > 0) {
    NEED(r.turns != nullptr, CMD_ERR_NULL, "turns is NULL");
    NEED(reinterpret_cast<uintptr_t>(r.turns) % 8 == 0, CMD_ERR_ALIGN, "turns is not 8-byte aligned");
  }
}

// The bytes of an access that suit a rotation of these tensors: 16, 8 or 4 (a
// chunk lies wholly in the rotated part, in the half layout in one half of it,
// or past it; strides are below 2^31), else 0.
int rope_bytes(const cmd_rope_spec& r, int64_t dim, std::initializer_list<const cmd_operand*> views) {
  const int es = elem_size((*views.begin())->dtype);
  for (int bytes = 16; bytes > es; bytes /= 2) {
    const int ve = bytes / es;
    bool ok = dim % ve == 0 && (r.layout == CMD_ROPE_HALF ? r.n_pairs : 2 * r.n_pairs) % ve == 0;
    for (const cmd_operand* o : views) {
      if (!o->ptr) continue;
      ok = ok && vector_rows(*o, bytes);
      for (int d = 0; d < o->rank; ++d) ok = ok && (o->sizes[d] <= 1 || o->strides[d] <= 0x7fffffff);
    }
    if (ok) return bytes;
  }
  return 0;
}

// A stream of the rope kernel from operands [batch,] tokens, heads, dim.
cmdx::RopeStream rope_stream(const cmd_operand& in, const cmd_operand& out, bool rotate, bool cache) {
  cmdx::RopeStream s = {};
  s.in = in.ptr;
  s.out = out.ptr;
  const int i = in.rank - 3;  // the dim of tokens
  s.in_st[0] = i ? in.strides[0] : 0;
  s.in_st[1] = in.strides[i];
  s.in_st[2] = in.strides[i + 1];
  if (cache) {
    for (int d = 0; d < 3; ++d) s.out_st[d] = out.strides[d];
  } else {
    s.out_st[0] = i ? out.strides[0] : 0;
    s.out_st[1] = out.strides[i];
    s.out_st[2] = out.strides[i + 1];
  }
  s.heads = (int32_t)in.sizes[i + 1];
  s.rotate = rotate;
  s.cache = cache;
  return s;
}

void rope_common(cmdx::RopeParams& p, const cmd_rope_spec& r, int64_t dim) {
  p.turns = r.turns;
  p.n_pairs = r.n_pairs;
  p.dim = (int32_t)dim;
  p.scale = r.scale;
  p.sine_scale = r.backward ? -r.scale : r.scale;
  p.heads = 0;
  int n = 0;
  for (int j = 0; j < p.n_streams; ++j) {
    if (p.s[j].heads == 0) continue;
    p.heads += p.s[j].heads;
    p.s[n++] = p.s[j];
  }
  p.n_streams = n;
}

void check_status(const int32_t* status) {
  NEED(reinterpret_cast<uintptr_t>(status) % sizeof(int32_t) == 0, CMD_ERR_ALIGN, "status is not 4-byte aligned");
}

void check_heads(int64_t heads) { NEED(heads <= 65536, CMD_ERR_LIMIT, "more than 65536 heads"); }

}  // namespace

extern "C" cmd_status cmd_rope_turns(int32_t n_pairs, double base, int32_t scaling, double factor,
                                     double original_length, double beta_fast, double beta_slow, uint64_t* turns) {
  return guarded([&]() -> cmd_status {
    NEED(n_pairs >= 0, CMD_ERR_SHAPE, "negative number of pairs");
    NEED(turns || n_pairs == 0, CMD_ERR_NULL, "turns is NULL");
    NEED(std::isfinite(base) && (base > 1.0 || (base >= 1.0 && n_pairs <= 1)), CMD_ERR_ARG, "the base must be above 1");
    NEED(scaling >= CMD_ROPE_SCALING_NONE && scaling <= CMD_ROPE_SCALING_PARTS, CMD_ERR_ARG, "unknown scaling");
    if (scaling != CMD_ROPE_SCALING_NONE)
      NEED(std::isfinite(factor) && factor >= 1.0, CMD_ERR_ARG, "the scaling factor must be at least 1");
    const double two_pi = 6.283185307179586476925;
    double lo = 0.0, hi = 0.0;
    if (scaling == CMD_ROPE_SCALING_BASE)
      base *= n_pairs > 1 ? std::pow(factor, (double)n_pairs / (n_pairs - 1)) : factor;
    if (scaling == CMD_ROPE_SCALING_PARTS) {
      NEED(std::isfinite(original_length) && original_length > 0 && std::isfinite(beta_fast) && beta_slow > 0 &&
               beta_fast > beta_slow,
           CMD_ERR_ARG, "scaling by parts needs original_length > 0 and beta_fast > beta_slow > 0");
      NEED(base > 1.0 || n_pairs == 0, CMD_ERR_ARG, "scaling by parts needs a base above 1");
      // the pair that makes `beta` turns over original_length: a real index (past the last pair, where the slowest one
      // makes more: the ramp then ends outside, at most at the rotated elements' number less one)
      auto pair_of = [&](double beta) {
        return n_pairs * std::log(original_length / (beta * two_pi)) / std::log(base);
      };
      lo = std::max(std::floor(pair_of(beta_fast)), 0.0);
      hi = std::min(std::ceil(pair_of(beta_slow)), 2.0 * n_pairs - 1);
      if (hi <= lo) hi = lo + 0.001;
    }
    for (int i = 0; i < n_pairs; ++i) {
      double f = std::pow(base, -(double)i / n_pairs);
      if (scaling == CMD_ROPE_SCALING_LINEAR) f /= factor;
      if (scaling == CMD_ROPE_SCALING_PARTS) {
        const double slow = std::min(std::max((i - lo) / (hi - lo), 0.0), 1.0);
        f = f * (1.0 - slow) + f / factor * slow;
      }
      turns[i] = (uint64_t)std::nearbyint(f / two_pi * 18446744073709551616.0);
    }
    return CMD_OK;
  });
}

extern "C" cmd_status cmd_rope(const cmd_operand* q, const cmd_operand* q_out, const cmd_operand* k,
                               const cmd_operand* k_out, const cmd_operand* positions, const cmd_rope_spec* rope,
                               void* cuda_stream) {
  return guarded([&]() -> cmd_status {
    NEED(positions && rope, CMD_ERR_NULL, "positions or rope is NULL");
    cmdx::RopeParams p;
    std::memset(&p, 0, sizeof p);
    const cmd_operand* ins[2] = {q, k};
    const cmd_operand* outs[2] = {q_out, k_out};
    const char* names[2][2] = {{"q", "q_out"}, {"k", "k_out"}};
    const cmd_operand* like = nullptr;
    bool nothing = false;
    for (int j = 0; j < 2; ++j) {
      if (!ins[j]) continue;
      const cmd_operand& in = *ins[j];
      NEED(outs[j], CMD_ERR_NULL, std::string(names[j][1]) + " is NULL");
      const cmd_operand& out = *outs[j];
      NEED(in.rank == 3 || in.rank == 4, CMD_ERR_SHAPE, std::string(names[j][0]) + " needs rank 3 or 4");
      check(in, names[j][0], in.rank, true);
      check(out, names[j][1], in.rank, true);
      NEED(is_float(in.dtype), CMD_ERR_TYPE, std::string(names[j][0]) + " is no float tensor");
      check_type(out, names[j][1], in.dtype);
      check_sizes(out, names[j][1], in.sizes);
      check_distinct(out, names[j][1]);
      if (like) {
        check_type(in, names[j][0], like->dtype);
        NEED(in.rank == like->rank, CMD_ERR_SHAPE, "q and k differ in rank");
        for (int d = 0; d < in.rank; ++d)
          NEED(d == in.rank - 2 || in.sizes[d] == like->sizes[d], CMD_ERR_SHAPE, "q and k differ in tokens or dim");
      }
      like = &in;
      check_apart(out, names[j][1], in, names[j][0], true);
      check_heads(in.sizes[in.rank - 2]);
      nothing = nothing || in.sizes[in.rank - 3] == 0 || in.sizes[in.rank - 1] == 0 || in.sizes[0] == 0;
      p.s[p.n_streams++] = rope_stream(in, out, true, false);
    }
    NEED(like, CMD_ERR_NULL, "q and k are both absent");
    if (q && k) {
      check_apart(*q_out, "q_out", *k, "k");
      check_apart(*k_out, "k_out", *q, "q");
      check_apart(*q_out, "q_out", *k_out, "k_out");
    }
    const int lead = like->rank - 2;
    check(*positions, "positions", lead);
    check_type(*positions, "positions", CMD_I32);
    check_sizes(*positions, "positions", like->sizes);
    for (int j = 0; j < 2; ++j)
      if (ins[j]) check_apart(*outs[j], names[j][1], *positions, "positions");
    const int64_t dim = like->sizes[like->rank - 1];
    NEED(dim <= CMD_CACHE_MAX_DIM, CMD_ERR_LIMIT, "a head dim above 256");
    check_rope(*rope, dim);
    p.batch = 1;
    p.tokens = like->sizes[like->rank - 3];
    if (like->rank == 4) {
      NEED(like->sizes[0] <= 0x7fffffff, CMD_ERR_LIMIT, "batch above 2^31");
      p.batch = (int32_t)like->sizes[0];
    }
    NEED((__int128)p.batch * p.tokens <= 0x7fffffff, CMD_ERR_LIMIT, "more than 2^31 - 1 tokens");
    p.per_batch = cmdx::fast_div_by((uint32_t)p.tokens);
    p.positions = static_cast<const int32_t*>(positions->ptr);
    p.pos_st[0] = lead == 2 ? positions->strides[0] : 0;
    p.pos_st[1] = positions->strides[lead - 1];
    p.columns = -1;  // no cache
    rope_common(p, *rope, dim);
    if (nothing || p.heads == 0) return CMD_OK;
    const cmd_operand none = {};
    const int bytes = rope_bytes(*rope, dim, {like, q ? q : &none, q ? q_out : &none, k ? k : &none, k ? k_out : &none});
    return launched(cmdx::rope_launch(like->dtype, rope->layout, bytes, p, static_cast<cudaStream_t>(cuda_stream)));
  });
}

namespace {

// The checks of a cache, its table and what goes with them.
void check_cache(const cmd_operand& k_cache, const cmd_operand& v_cache, const cmd_operand& tables) {
  check(k_cache, "k_cache", 4, true);
  check(v_cache, "v_cache", 4, true);
  NEED(is_float(k_cache.dtype), CMD_ERR_TYPE, "k_cache is no float tensor");
  check_type(v_cache, "v_cache", k_cache.dtype);
  check_sizes(v_cache, "v_cache", k_cache.sizes);
  NEED(k_cache.sizes[0] <= 0x7fffffff, CMD_ERR_LIMIT, "more than 2^31 - 1 pages");
  NEED(k_cache.sizes[1] >= 1, CMD_ERR_SHAPE, "a page holds no token");
  NEED(k_cache.sizes[3] <= CMD_CACHE_MAX_DIM, CMD_ERR_LIMIT, "a head dim above 256");
  check_heads(k_cache.sizes[2]);
  check(tables, "tables", 2);
  check_type(tables, "tables", CMD_I32);
  NEED(tables.sizes[0] <= 0x7fffffff, CMD_ERR_LIMIT, "more than 2^31 - 1 table rows");
  NEED((__int128)tables.sizes[1] * k_cache.sizes[1] <= 0x7fff0000, CMD_ERR_LIMIT,
       "table rows that reach past 2^31 - 2^16 tokens");
}

}  // namespace

extern "C" cmd_status cmd_cache_append(const cmd_append_args* args, void* cuda_stream) {
  return guarded([&]() -> cmd_status {
    NEED(args, CMD_ERR_NULL, "args is NULL");
    const cmd_append_args& a = *args;
    check_status(a.status);
    check(a.k, "k", 3, true);
    check(a.v, "v", 3, true);
    check_cache(a.k_cache, a.v_cache, a.tables);
    check_type(a.k, "k", a.k_cache.dtype);
    check_type(a.v, "v", a.k_cache.dtype);
    check_sizes(a.v, "v", a.k.sizes);
    NEED(a.k.sizes[1] == a.k_cache.sizes[2] && a.k.sizes[2] == a.k_cache.sizes[3], CMD_ERR_SHAPE,
         "k and k_cache differ in heads or dim");
    const int64_t tokens = a.k.sizes[0], dim = a.k.sizes[2];
    NEED(tokens <= 0x7fffffff, CMD_ERR_LIMIT, "more than 2^31 - 1 tokens");
    check(a.positions, "positions", 1);
    check_type(a.positions, "positions", CMD_I32);
    check_sizes(a.positions, "positions", &tokens);
    const bool has_rows = a.rows.ptr != nullptr, has_q = a.q.ptr != nullptr;
    if (has_rows) {
      check(a.rows, "rows", 1);
      check_type(a.rows, "rows", CMD_I32);
      check_sizes(a.rows, "rows", &tokens);
    } else {
      NEED(a.tables.sizes[0] == tokens, CMD_ERR_SHAPE, "rows may be absent only where each token has its own table row");
    }
    if (has_q) {
      check(a.q, "q", 3, true);
      check(a.q_out, "q_out", 3, true);
    }
    check_rope(a.rope, dim);
    check_distinct(a.k_cache, "k_cache");
    check_distinct(a.v_cache, "v_cache");
    const struct {
      const cmd_operand* o;
      const char* name;
    } reads[] = {{&a.k, "k"}, {&a.v, "v"}, {&a.tables, "tables"}, {&a.positions, "positions"}, {&a.rows, "rows"}, {&a.q, "q"}};
    for (const auto& r : reads) {
      check_apart(a.k_cache, "k_cache", *r.o, r.name);
      check_apart(a.v_cache, "v_cache", *r.o, r.name);
    }
    check_apart(a.k_cache, "k_cache", a.v_cache, "v_cache");
    cmdx::RopeParams p;
    std::memset(&p, 0, sizeof p);
    if (has_q) {
      NEED(a.rope.n_pairs > 0, CMD_ERR_ARG, "q is given and nothing rotates it");
      check_type(a.q, "q", a.k.dtype);
      check_type(a.q_out, "q_out", a.k.dtype);
      NEED(a.q.sizes[0] == tokens && a.q.sizes[2] == dim, CMD_ERR_SHAPE, "q and k differ in tokens or dim");
      check_sizes(a.q_out, "q_out", a.q.sizes);
      check_distinct(a.q_out, "q_out");
      check_heads(a.q.sizes[1]);
      for (const auto& r : reads) check_apart(a.q_out, "q_out", *r.o, r.name, r.o == &a.q);
      check_apart(a.q_out, "q_out", a.k_cache, "k_cache");
      check_apart(a.q_out, "q_out", a.v_cache, "v_cache");
      p.s[p.n_streams++] = rope_stream(a.q, a.q_out, true, false);
    }
    p.s[p.n_streams++] = rope_stream(a.k, a.k_cache, true, true);
    p.s[p.n_streams++] = rope_stream(a.v, a.v_cache, false, true);
    p.batch = 1;
    p.tokens = tokens;
    p.per_batch = cmdx::fast_div_by((uint32_t)tokens);
    p.positions = static_cast<const int32_t*>(a.positions.ptr);
    p.pos_st[1] = a.positions.strides[0];
    p.tables = static_cast<const int32_t*>(a.tables.ptr);
    p.rows = static_cast<const int32_t*>(a.rows.ptr);
    p.table_st[0] = a.tables.strides[0];
    p.table_st[1] = a.tables.strides[1];
    p.rows_st = has_rows ? a.rows.strides[0] : 0;
    p.n_rows = (int32_t)a.tables.sizes[0];
    p.columns = (int32_t)a.tables.sizes[1];
    p.n_pages = (int32_t)a.k_cache.sizes[0];
    p.page = cmdx::fast_div_by((uint32_t)a.k_cache.sizes[1]);
    p.status = a.status;
    rope_common(p, a.rope, dim);
    if (tokens == 0 || dim == 0 || p.heads == 0) return CMD_OK;
    const cmd_operand none = {};
    const int bytes = rope_bytes(a.rope, dim, {&a.k, &a.v, &a.k_cache, &a.v_cache, &a.q, has_q ? &a.q_out : &none});
    return launched(cmdx::rope_launch(a.k.dtype, a.rope.layout, bytes, p, static_cast<cudaStream_t>(cuda_stream)));
  });
}

namespace {

int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

void check_workspace(const void* ws, int64_t bytes, int64_t want) {
  NEED(ws, CMD_ERR_NULL, "workspace is NULL");
  NEED(reinterpret_cast<uintptr_t>(ws) % 16 == 0, CMD_ERR_ALIGN, "workspace is not 16-byte aligned");
  NEED(bytes >= want, CMD_ERR_LIMIT, "workspace has " + std::to_string(bytes) + " bytes, not " + std::to_string(want));
}

constexpr int64_t kSplitBytes = cmdx::kAttendMaxCtas * sizeof(cmdx::AttendSplit);
static_assert(kSplitBytes % 16 == 0, "the parts are aligned");

int64_t attention_workspace(int64_t q_heads, int64_t kv_heads, int64_t dim) {
  const int64_t heads = std::min<int64_t>(q_heads / kv_heads, cmdx::kAttendMmaHeads);
  return kSplitBytes + 2 * (int64_t)cmdx::kAttendMaxCtas * heads * (round_up(dim, 4) + 4) * 4;
}

}  // namespace

extern "C" cmd_status cmd_attention_workspace(int32_t q_heads, int32_t kv_heads, int32_t dim, int64_t* bytes) {
  return guarded([&]() -> cmd_status {
    NEED(bytes, CMD_ERR_NULL, "bytes is NULL");
    NEED(kv_heads >= 1 && q_heads >= 1 && q_heads % kv_heads == 0, CMD_ERR_SHAPE, "kv_heads must divide q_heads");
    check_heads(q_heads);
    NEED(dim >= 0 && dim <= CMD_CACHE_MAX_DIM, CMD_ERR_LIMIT, "a head dim above 256");
    *bytes = attention_workspace(q_heads, kv_heads, dim);
    return CMD_OK;
  });
}

extern "C" cmd_status cmd_attention_decode(const cmd_attention_args* args, void* cuda_stream) {
  return guarded([&]() -> cmd_status {
    NEED(args, CMD_ERR_NULL, "args is NULL");
    const cmd_attention_args& a = *args;
    check_status(a.status);
    check(a.q, "q", 3, true);
    check(a.out, "out", 3, true);
    check_cache(a.k_cache, a.v_cache, a.tables);
    check_type(a.q, "q", a.k_cache.dtype);
    check_type(a.out, "out", a.k_cache.dtype);
    check_sizes(a.out, "out", a.q.sizes);
    check_distinct(a.out, "out");
    const int64_t rows = a.q.sizes[0], heads = a.q.sizes[1], dim = a.q.sizes[2], kv = a.k_cache.sizes[2];
    NEED(dim == a.k_cache.sizes[3], CMD_ERR_SHAPE, "q and k_cache differ in dim");
    NEED(dim >= 1, CMD_ERR_SHAPE, "a head has no elements");
    NEED(kv >= 1 ? heads % kv == 0 : heads == 0, CMD_ERR_SHAPE, "the cache's heads must divide q's");
    check_heads(heads);
    NEED(rows == a.tables.sizes[0], CMD_ERR_SHAPE, "q and tables differ in rows");
    check(a.lengths, "lengths", 1);
    check_type(a.lengths, "lengths", CMD_I32);
    check_sizes(a.lengths, "lengths", &rows);
    const cmd_operand* ins[] = {&a.q, &a.k_cache, &a.v_cache, &a.tables, &a.lengths};
    const char* names[] = {"q", "k_cache", "v_cache", "tables", "lengths"};
    if (a.lse.ptr) {
      check(a.lse, "lse", 2);
      check_type(a.lse, "lse", CMD_F32);
      check_sizes(a.lse, "lse", a.q.sizes);
      check_distinct(a.lse, "lse");
      for (int i = 0; i < 5; ++i) check_apart(a.lse, "lse", *ins[i], names[i]);
      check_apart(a.lse, "lse", a.out, "out");
    }
    for (int i = 0; i < 5; ++i) check_apart(a.out, "out", *ins[i], names[i]);
    NEED(std::isfinite(a.scale) && a.scale > 0.0f, CMD_ERR_ARG, "scale must be positive");
    NEED(std::isfinite(a.softcap) && a.softcap >= 0.0f, CMD_ERR_ARG, "softcap must be positive, or 0 for none");
    NEED(a.window >= 0, CMD_ERR_ARG, "window must be positive, or 0 for none");
    NEED(a.reserved == 0, CMD_ERR_ARG, "reserved must be 0");
    if (rows == 0 || heads == 0) return CMD_OK;
    check_workspace(a.workspace, a.workspace_bytes, attention_workspace(heads, kv, dim));
    cmdx::AttendParams p;
    std::memset(&p, 0, sizeof p);
    p.kv_heads = (int32_t)kv;
    p.group = (int32_t)(heads / kv);
    p.dim = (int32_t)dim;
    p.n_pages = (int32_t)a.k_cache.sizes[0];
    p.columns = (int32_t)a.tables.sizes[1];
    p.page = cmdx::fast_div_by((uint32_t)a.k_cache.sizes[1]);
    const double log2e = 1.4426950408889634074;
    p.scale_log2 = (float)(a.scale * log2e);
    p.cap_in = a.softcap > 0.0f ? (float)((double)a.scale / a.softcap) : 0.0f;
    p.cap_out = (float)(a.softcap * log2e);
    p.window = a.window;
    for (int d = 0; d < 3; ++d) {
      p.k_st[d] = a.k_cache.strides[d];
      p.v_st[d] = a.v_cache.strides[d];
    }
    for (int d = 0; d < 2; ++d) {
      p.q_st[d] = a.q.strides[d];
      p.out_st[d] = a.out.strides[d];
      p.lse_st[d] = a.lse.ptr ? a.lse.strides[d] : 0;
      p.table_st[d] = a.tables.strides[d];
    }
    p.len_st = a.lengths.strides[0];
    p.k = a.k_cache.ptr;
    p.v = a.v_cache.ptr;
    p.splits = static_cast<cmdx::AttendSplit*>(a.workspace);
    p.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + kSplitBytes);
    p.status = a.status;
    const int es = elem_size(a.q.dtype);
    // bytes of a copy that suit every row of the cache: 16, 4, or fewer. (On rows that suit both, 64 of 4096 tokens, 8 kv
    // heads of 128: bf16 180 us with 16, 217 with 4; 24 f32 ones of 2999 tokens and 16 kv heads 180 and 226.)
    const auto pieces = [&](int n) { return dim * es % n == 0 && vector_rows(a.k_cache, n) && vector_rows(a.v_cache, n); };
    const int copy = pieces(16) ? 16 : pieces(4) ? 4 : 0;
    const int most = copy && es == 2 ? cmdx::kAttendMmaHeads : cmdx::kAttendHeads;
    p.blocks = (p.group + most - 1) / most;
    p.block_heads = (p.group + p.blocks - 1) / p.blocks;
    p.q_pairs = vector_rows(a.q, 4);
    // a launch's units (tiles of rows that fill their tables, for each head) stay below 2^31
    const int64_t row_units = (int64_t)p.kv_heads * p.blocks *
                              (p.columns * a.k_cache.sizes[1] / cmdx::kAttendLeastTile + 2 + cmdx::kAttendMostStart);
    NEED(row_units < 0x7fffffff, CMD_ERR_LIMIT, "a table row's tokens times the heads pass 2^31 tiles of 32");
    const int64_t at_once = std::min<int64_t>(cmdx::kAttendRows, 0x7fffffff / row_units);
    for (int64_t r = 0; r < rows; r += at_once) {
      p.rows = (int32_t)std::min<int64_t>(at_once, rows - r);
      p.q = static_cast<const uint8_t*>(a.q.ptr) + r * a.q.strides[0] * es;
      p.out = static_cast<uint8_t*>(a.out.ptr) + r * a.out.strides[0] * es;
      p.lse = a.lse.ptr ? static_cast<float*>(a.lse.ptr) + r * a.lse.strides[0] : nullptr;
      p.tables = static_cast<const int32_t*>(a.tables.ptr) + r * a.tables.strides[0];
      p.lengths = static_cast<const int32_t*>(a.lengths.ptr) + r * a.lengths.strides[0];
      const cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
      const cudaError_t e = !copy       ? cmdx::attend_simt_launch(a.q.dtype, p, stream)
                            : es == 4   ? (copy == 16 ? cmdx::attend_f32_launch16 : cmdx::attend_f32_launch4)(p, stream)
                                        : (copy == 16 ? cmdx::attend_mma_launch16
                                                      : cmdx::attend_mma_launch4)(a.q.dtype, p, stream);
      if (e != cudaSuccess) return launched(e);
    }
    return CMD_OK;
  });
}

namespace {

// A dense vector, or a table with dense rows, of i32.
void check_ints(const cmd_operand& o, const char* name, int rank) {
  check(o, name, rank, true);
  check_type(o, name, CMD_I32);
  for (int d = 0; d < rank; ++d) NEED(o.sizes[d] <= 0x7fffffff, CMD_ERR_LIMIT, std::string(name) + " is too long");
}

// The pools of a call, and the largest access that suits them all.
cmdx::PoolList pool_list(const cmd_pool* pools, int32_t n, int64_t pages) {
  NEED(n >= 0 && n <= CMD_CACHE_MAX_POOLS, CMD_ERR_LIMIT, "more than 64 pools");
  NEED(pools || n == 0, CMD_ERR_NULL, "pools is NULL");
  cmdx::PoolList l;
  std::memset(&l, 0, sizeof l);
  uint64_t bits = 16;
  for (int i = 0; i < n; ++i) {
    NEED(pools[i].page_bytes >= 0 && pools[i].page_stride >= pools[i].page_bytes, CMD_ERR_SHAPE,
         "a pool's pages overlap (page_stride below page_bytes)");
    NEED((__int128)pools[i].page_stride * pages < ((__int128)1 << 60), CMD_ERR_LIMIT, "a pool extends past the address space");
    if (pools[i].page_bytes == 0 || pages == 0) continue;
    NEED(pools[i].ptr, CMD_ERR_NULL, "a pool's pointer is NULL");
    l.ptr[l.n] = static_cast<uint8_t*>(pools[i].ptr);
    l.stride[l.n] = pools[i].page_stride;
    l.bytes[l.n] = pools[i].page_bytes;
    bits |= reinterpret_cast<uintptr_t>(pools[i].ptr) | (uint64_t)pools[i].page_stride | (uint64_t)pools[i].page_bytes;
    ++l.n;
  }
  l.unit = (int32_t)(bits & (~bits + 1));
  return l;
}

void check_pools_apart(const cmd_operand& o, const char* name, const cmdx::PoolList& l, int64_t pages) {
  for (int i = 0; i < l.n; ++i) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(l.ptr[i]);
    NEED(!meet(range_of(o), {a, a + (uintptr_t)((pages - 1) * l.stride[i] + l.bytes[i])}), CMD_ERR_ALIAS,
         std::string(name) + " overlaps a pool");
  }
}

// Whether two pools share bytes (interleaved pools of one stride do not).
void check_pools(const cmdx::PoolList& l, int64_t pages) {
  for (int i = 0; i < l.n; ++i)
    for (int j = 0; j < i; ++j) {
      const uintptr_t a = reinterpret_cast<uintptr_t>(l.ptr[i]), b = reinterpret_cast<uintptr_t>(l.ptr[j]);
      if (!meet({a, a + (uintptr_t)((pages - 1) * l.stride[i] + l.bytes[i])},
                {b, b + (uintptr_t)((pages - 1) * l.stride[j] + l.bytes[j])}))
        continue;
      bool ok = l.stride[i] == l.stride[j];
      if (ok) {
        const uintptr_t d = (a > b ? a - b : b - a) % (uintptr_t)l.stride[i];
        const int64_t first = a > b ? l.bytes[j] : l.bytes[i], second = a > b ? l.bytes[i] : l.bytes[j];
        ok = (int64_t)d >= first && (int64_t)d + second <= l.stride[i];
      }
      NEED(ok, CMD_ERR_ALIAS, "two pools overlap");
    }
}

// Rows and pages of a select or compact call, whose kernels step through them
// in 32 bits.
constexpr int64_t kMostRows = 1 << 30, kMostPages = 1 << 30;

constexpr int64_t kHeadWords = 16;
int64_t padded(int64_t words) { return round_up(words, 4); }
int64_t select_words(int64_t old_rows, int64_t new_rows, int64_t pages) {
  return kHeadWords + 2 * padded(old_rows) + 4 * padded(new_rows) + padded(pages);
}
int64_t compact_words(int64_t pages) { return kHeadWords + 2 * padded(pages); }

struct Words {
  int32_t* at;
  int32_t* take(int64_t n) {
    int32_t* p = at;
    at += padded(n);
    return p;
  }
};

}  // namespace

extern "C" cmd_status cmd_select_workspace(int64_t old_rows, int64_t new_rows, int64_t pages, int64_t* bytes) {
  return guarded([&]() -> cmd_status {
    NEED(bytes, CMD_ERR_NULL, "bytes is NULL");
    NEED(old_rows >= 0 && new_rows >= 0 && pages >= 0 && old_rows <= 0x7fffffff && new_rows <= 0x7fffffff &&
             pages <= 0x7fffffff,
         CMD_ERR_SHAPE, "negative size, or one above 2^31 - 1");
    *bytes = 4 * select_words(old_rows, new_rows, pages);
    return CMD_OK;
  });
}

extern "C" cmd_status cmd_cache_select(const cmd_select_args* args, void* cuda_stream) {
  return guarded([&]() -> cmd_status {
    NEED(args, CMD_ERR_NULL, "args is NULL");
    const cmd_select_args& a = *args;
    check_status(a.status);
    check_ints(a.tables, "tables", 2);
    check_ints(a.tables_out, "tables_out", 2);
    const int64_t old_rows = a.tables.sizes[0], new_rows = a.tables_out.sizes[0], columns = a.tables.sizes[1];
    NEED(a.tables_out.sizes[1] == columns, CMD_ERR_SHAPE, "tables and tables_out differ in columns");
    NEED(old_rows <= kMostRows && new_rows <= kMostRows, CMD_ERR_LIMIT, "more than 2^30 rows");
    check_distinct(a.tables_out, "tables_out");
    check_ints(a.lengths, "lengths", 1);
    check_sizes(a.lengths, "lengths", &old_rows);
    check_ints(a.lengths_out, "lengths_out", 1);
    check_sizes(a.lengths_out, "lengths_out", &new_rows);
    check_ints(a.parents, "parents", 1);
    check_sizes(a.parents, "parents", &new_rows);
    if (a.grow.ptr) {
      check_ints(a.grow, "grow", 1);
      check_sizes(a.grow, "grow", &new_rows);
    }
    check_ints(a.refs, "refs", 1);
    const int64_t pages = a.refs.sizes[0];
    check_ints(a.refs_out, "refs_out", 1);
    check_sizes(a.refs_out, "refs_out", &pages);
    NEED(pages <= kMostPages, CMD_ERR_LIMIT, "more than 2^30 pages");
    NEED(a.page_size >= 1, CMD_ERR_SHAPE, "a page holds no token");
    NEED((__int128)columns * a.page_size <= 0x7fff0000, CMD_ERR_LIMIT, "table rows that reach past 2^31 - 2^16 tokens");
    const cmdx::PoolList pools = pool_list(a.pools, a.n_pools, pages);
    check_pools(pools, pages);
    const cmd_operand* ins[] = {&a.tables, &a.lengths, &a.refs, &a.parents, &a.grow};
    const char* in_names[] = {"tables", "lengths", "refs", "parents", "grow"};
    const cmd_operand* outs[] = {&a.tables_out, &a.lengths_out, &a.refs_out};
    const char* out_names[] = {"tables_out", "lengths_out", "refs_out"};
    for (int o = 0; o < 3; ++o) {
      for (int i = 0; i < 5; ++i) check_apart(*outs[o], out_names[o], *ins[i], in_names[i]);
      for (int i = 0; i < o; ++i) check_apart(*outs[o], out_names[o], *outs[i], out_names[i]);
      check_pools_apart(*outs[o], out_names[o], pools, pages);
    }
    for (int i = 0; i < 5; ++i) check_pools_apart(*ins[i], in_names[i], pools, pages);
    check_workspace(a.workspace, a.workspace_bytes, 4 * select_words(old_rows, new_rows, pages));
    if (new_rows == 0 && pages == 0) return CMD_OK;
    cmdx::SelectParams p;
    std::memset(&p, 0, sizeof p);
    p.tables = static_cast<const int32_t*>(a.tables.ptr);
    p.lengths = static_cast<const int32_t*>(a.lengths.ptr);
    p.refs = static_cast<const int32_t*>(a.refs.ptr);
    p.parents = static_cast<const int32_t*>(a.parents.ptr);
    p.grow = static_cast<const int32_t*>(a.grow.ptr);
    p.tables_out = static_cast<int32_t*>(a.tables_out.ptr);
    p.lengths_out = static_cast<int32_t*>(a.lengths_out.ptr);
    p.refs_out = static_cast<int32_t*>(a.refs_out.ptr);
    p.table_st = a.tables.strides[0];
    p.table_out_st = a.tables_out.strides[0];
    p.old_rows = (int32_t)old_rows;
    p.new_rows = (int32_t)new_rows;
    p.columns = (int32_t)columns;
    p.pages = (int32_t)pages;
    p.page = cmdx::fast_div_by((uint32_t)a.page_size);
    p.status = a.status;
    Words w = {static_cast<int32_t*>(a.workspace)};
    p.head = w.take(kHeadWords);
    p.first = w.take(old_rows);
    p.children = w.take(old_rows);
    p.keep = w.take(new_rows);
    p.base = w.take(new_rows);
    p.copy_src = w.take(new_rows);
    p.copy_dst = w.take(new_rows);
    p.free_list = w.take(pages);
    return launched(cmdx::select_launch(p, pools, static_cast<cudaStream_t>(cuda_stream)));
  });
}

extern "C" cmd_status cmd_compact_workspace(int64_t pages, int64_t* bytes) {
  return guarded([&]() -> cmd_status {
    NEED(bytes, CMD_ERR_NULL, "bytes is NULL");
    NEED(pages >= 0 && pages <= 0x7fffffff, CMD_ERR_SHAPE, "negative number of pages, or one above 2^31 - 1");
    *bytes = 4 * compact_words(pages);
    return CMD_OK;
  });
}

extern "C" cmd_status cmd_cache_compact(const cmd_compact_args* args, void* cuda_stream) {
  return guarded([&]() -> cmd_status {
    NEED(args, CMD_ERR_NULL, "args is NULL");
    const cmd_compact_args& a = *args;
    check_status(a.status);
    check_ints(a.tables, "tables", 2);
    check_ints(a.tables_out, "tables_out", 2);
    check_sizes(a.tables_out, "tables_out", a.tables.sizes);
    NEED(a.tables.sizes[0] <= kMostRows, CMD_ERR_LIMIT, "more than 2^30 rows");
    check_distinct(a.tables_out, "tables_out");
    check_ints(a.lengths, "lengths", 1);
    check_sizes(a.lengths, "lengths", &a.tables.sizes[0]);
    check_ints(a.refs, "refs", 1);
    const int64_t pages = a.refs.sizes[0], columns = a.tables.sizes[1];
    check_ints(a.refs_out, "refs_out", 1);
    check_sizes(a.refs_out, "refs_out", &pages);
    check_ints(a.page_map_out, "page_map_out", 1);
    check_sizes(a.page_map_out, "page_map_out", &pages);
    NEED(pages <= kMostPages, CMD_ERR_LIMIT, "more than 2^30 pages");
    NEED(a.page_size >= 1, CMD_ERR_SHAPE, "a page holds no token");
    NEED((__int128)columns * a.page_size <= 0x7fff0000, CMD_ERR_LIMIT, "table rows that reach past 2^31 - 2^16 tokens");
    const cmdx::PoolList pools = pool_list(a.pools, a.n_pools, pages);
    check_pools(pools, pages);
    const cmd_operand* ins[] = {&a.tables, &a.lengths, &a.refs};
    const char* in_names[] = {"tables", "lengths", "refs"};
    const cmd_operand* outs[] = {&a.tables_out, &a.refs_out, &a.page_map_out};
    const char* out_names[] = {"tables_out", "refs_out", "page_map_out"};
    for (int o = 0; o < 3; ++o) {
      for (int i = 0; i < 3; ++i) check_apart(*outs[o], out_names[o], *ins[i], in_names[i]);
      for (int i = 0; i < o; ++i) check_apart(*outs[o], out_names[o], *outs[i], out_names[i]);
      check_pools_apart(*outs[o], out_names[o], pools, pages);
    }
    for (int i = 0; i < 3; ++i) check_pools_apart(*ins[i], in_names[i], pools, pages);
    check_workspace(a.workspace, a.workspace_bytes, 4 * compact_words(pages));
    if (a.tables.sizes[0] == 0 && pages == 0) return CMD_OK;
    cmdx::CompactParams p;
    std::memset(&p, 0, sizeof p);
    p.tables = static_cast<const int32_t*>(a.tables.ptr);
    p.lengths = static_cast<const int32_t*>(a.lengths.ptr);
    p.refs = static_cast<const int32_t*>(a.refs.ptr);
    p.tables_out = static_cast<int32_t*>(a.tables_out.ptr);
    p.refs_out = static_cast<int32_t*>(a.refs_out.ptr);
    p.map_out = static_cast<int32_t*>(a.page_map_out.ptr);
    p.table_st = a.tables.strides[0];
    p.table_out_st = a.tables_out.strides[0];
    p.rows = (int32_t)a.tables.sizes[0];
    p.columns = (int32_t)columns;
    p.pages = (int32_t)pages;
    p.page = cmdx::fast_div_by((uint32_t)a.page_size);
    p.status = a.status;
    Words w = {static_cast<int32_t*>(a.workspace)};
    p.head = w.take(kHeadWords);
    p.holes = w.take(pages);
    p.movers = w.take(pages);
    return launched(cmdx::compact_launch(p, pools, static_cast<cudaStream_t>(cuda_stream)));
  });
}

extern "C" cmd_status cmd_cache_status(int32_t* status, int32_t* bits, void* cuda_stream) {
  return guarded([&]() -> cmd_status {
    NEED(status, CMD_ERR_NULL, "status is NULL");
    check_status(status);
    const cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
    int32_t word = 0;
    cudaError_t e = cudaMemcpyAsync(&word, status, sizeof word, cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e == cudaSuccess && word) {
      e = cmdx::status_clear_launch(status, word, stream);
      if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    }
    if (e != cudaSuccess) return launched(e);
    if (bits) *bits = word;
    if (!word) return CMD_OK;
    std::string msg = "on the device:";
    if (word & CMD_CACHE_BAD_PAGE) msg += " a table entry named no page;";
    if (word & CMD_CACHE_BAD_INDEX) msg += " a row, parent, position or length was out of its range;";
    if (word & CMD_CACHE_FULL_TABLE) msg += " a table row had no room;";
    if (word & CMD_CACHE_NO_PAGES) msg += " the pool had no free page;";
    msg.pop_back();
    return host_fail(word & (CMD_CACHE_BAD_PAGE | CMD_CACHE_BAD_INDEX) ? CMD_ERR_ARG : CMD_ERR_LIMIT, msg);
  });
}
