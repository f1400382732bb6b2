// The Python binding's way into the serving-step calls of include/pa.h: their arguments in order,
// each in one 8-byte field, packed by the caller. Marshalling 15 to 31 arguments one by one takes
// ctypes 2 to 3 us on the GPU's host, more than the launch; a packed call takes 0.5.
#include <cstdint>

#include "pa.h"

namespace {

union Field {
  void* p;
  int64_t i;
  double f;
};

// Reads the fields in order; `ok` turns false at an integer that its parameter cannot hold.
struct Fields {
  const Field* at;
  bool ok = true;
  template <typename T>
  T* ptr() {
    return static_cast<T*>((at++)->p);
  }
  int64_t i64() { return (at++)->i; }
  int i32() {
    const int64_t x = (at++)->i;
    ok = ok && x == int64_t(int(x));
    return int(x);
  }
  float f32() { return float((at++)->f); }
  pa_dtype type() { return static_cast<pa_dtype>(i32()); }
  pa_stream_t stream() { return static_cast<pa_stream_t>((at++)->p); }
};

}  // namespace

extern "C" int pa_packed_call(int which, const void* packed) {
  Fields f{static_cast<const Field*>(packed)};
  switch (which) {
    case 0: {
      auto table = f.ptr<int32_t>();
      const int width = f.i32();
      auto lens = f.ptr<int32_t>(), q = f.ptr<int32_t>(), free_blocks = f.ptr<int32_t>();
      const int num_free = f.i32();
      auto head = f.ptr<int32_t>(), lens_out = f.ptr<int32_t>(), head_out = f.ptr<int32_t>(), qsl = f.ptr<int32_t>();
      auto slots = f.ptr<int64_t>();
      auto positions = f.ptr<int32_t>();
      const int S = f.i32(), T = f.i32(), B = f.i32();
      const int64_t NB = f.i64();
      auto s = f.stream();
      if (!f.ok) return PA_ERR_INVALID_ARG;
      return pa_advance_batch(table, width, lens, q, free_blocks, num_free, head, lens_out, head_out, qsl, slots,
                              positions, S, T, B, NB, s);
    }
    case 1: {
      auto q_out = f.ptr<void>(), q = f.ptr<void>(), k = f.ptr<void>(), v = f.ptr<void>();
      const int64_t qs = f.i64(), ks = f.i64(), vs = f.i64();
      auto qw = f.ptr<void>(), kw = f.ptr<void>();
      const float eps = f.f32();
      auto cos_sin = f.ptr<float>();
      const int limit = f.i32(), rot = f.i32(), interleaved = f.i32();
      auto positions = f.ptr<int32_t>();
      const int axes = f.i32();
      int sections[4];
      for (int& x : sections) x = f.i32();  // the first `axes` of them count
      auto slots = f.ptr<int64_t>();
      auto kc = f.ptr<void>(), vc = f.ptr<void>();
      const int64_t T = f.i64(), NB = f.i64();
      const int B = f.i32(), Hq = f.i32(), Hkv = f.i32(), D = f.i32();
      const pa_dtype dt = f.type(), cache = f.type();
      const float k_scale = f.f32(), v_scale = f.f32();
      auto s = f.stream();
      if (!f.ok) return PA_ERR_INVALID_ARG;
      return pa_norm_rope_write(q_out, q, k, v, qs, ks, vs, qw, kw, eps, cos_sin, limit, rot, interleaved, positions, axes,
                                sections, slots, kc, vc, T, NB, B, Hq, Hkv, D, dt, cache, k_scale, v_scale, s);
    }
    case 2: {
      auto bounds = f.ptr<void>(), kc = f.ptr<void>();
      auto table = f.ptr<int32_t>();
      const int width = f.i32();
      auto lens = f.ptr<int32_t>(), qsl = f.ptr<int32_t>();
      const int S = f.i32(), T = f.i32(), max_q = f.i32(), max_s = f.i32(), Hkv = f.i32(), D = f.i32(), B = f.i32();
      const int64_t NB = f.i64();
      const pa_dtype cache = f.type();
      auto s = f.stream();
      if (!f.ok) return PA_ERR_INVALID_ARG;
      return pa_block_bounds(bounds, kc, table, width, lens, qsl, S, T, max_q, max_s, Hkv, D, B, NB, cache, s);
    }
    case 3: {
      auto scores = f.ptr<float>();
      const int score_width = f.i32();
      auto q = f.ptr<void>(), bounds = f.ptr<void>();
      auto table = f.ptr<int32_t>();
      const int width = f.i32();
      auto lens = f.ptr<int32_t>(), qsl = f.ptr<int32_t>();
      const int S = f.i32(), T = f.i32(), max_q = f.i32(), max_s = f.i32(), Hq = f.i32(), Hkv = f.i32(), D = f.i32(),
                B = f.i32();
      const int64_t NB = f.i64();
      auto s = f.stream();
      if (!f.ok) return PA_ERR_INVALID_ARG;
      return pa_block_scores(scores, score_width, q, bounds, table, width, lens, qsl, S, T, max_q, max_s, Hq, Hkv, D, B, NB,
                             s);
    }
    case 4: {
      auto idx = f.ptr<int32_t>();
      const int k = f.i32();
      auto scores = f.ptr<float>();
      const int score_width = f.i32();
      auto lens = f.ptr<int32_t>(), qsl = f.ptr<int32_t>();
      const int S = f.i32(), T = f.i32(), Hkv = f.i32(), B = f.i32(), init = f.i32(), local = f.i32();
      auto s = f.stream();
      if (!f.ok) return PA_ERR_INVALID_ARG;
      return pa_select_blocks(idx, k, scores, score_width, lens, qsl, S, T, Hkv, B, init, local, s);
    }
    case 5: {
      auto out = f.ptr<void>(), q = f.ptr<void>(), kc = f.ptr<void>(), vc = f.ptr<void>();
      auto table = f.ptr<int32_t>();
      const int width = f.i32();
      auto lens = f.ptr<int32_t>(), qsl = f.ptr<int32_t>(), idx = f.ptr<int32_t>();
      const int k = f.i32(), S = f.i32(), T = f.i32(), max_s = f.i32(), Hq = f.i32(), Hkv = f.i32(), D = f.i32(),
                B = f.i32();
      const int64_t NB = f.i64();
      const float scale = f.f32();
      const pa_dtype cache = f.type();
      const float k_scale = f.f32(), v_scale = f.f32();
      auto s = f.stream();
      if (!f.ok) return PA_ERR_INVALID_ARG;
      return pa_attention_sparse(out, q, kc, vc, table, width, lens, qsl, idx, k, S, T, max_s, Hq, Hkv, D, B, NB, scale,
                                 cache, k_scale, v_scale, s);
    }
  }
  return PA_ERR_INVALID_ARG;
}
