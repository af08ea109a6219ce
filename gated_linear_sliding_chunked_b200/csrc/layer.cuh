// Shared parts of the layer operators (short convolution, selective scan,
// block norms): strided rows, vector access, host-side checks.
#pragma once

#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <initializer_list>

#include "../../include/lizard.h"
#include "common.cuh"
#include "kernels.h"

namespace lz {

// ---- device ---------------------------------------------------------------

// Rows of a strided input: element (b, t, 0) stands at b * bs + t * ld.
struct Rows {
  int64_t ld, bs;
  __host__ __device__ size_t at(int b, int t) const { return (size_t)b * bs + (size_t)t * ld; }
};

// Pairs of fp32 values in 64-bit registers: one instruction for two lanes of
// arithmetic (fma.rn.f32x2 and the like), rounded as the scalar ones.
using f2 = unsigned long long;
__device__ __forceinline__ f2 pk(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float lo(f2 x) { return __uint_as_float((uint32_t)x); }
__device__ __forceinline__ float hi(f2 x) { return __uint_as_float((uint32_t)(x >> 32)); }
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// VW consecutive elements as floats (one access: vectors of 4, or of 8 16-bit
// elements to store)
template <int VW>
__device__ __forceinline__ void load_vec(const float* p, float* x) {
  if constexpr (VW == 4) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  } else {
    x[0] = *p;
  }
}
template <int VW>
__device__ __forceinline__ void load_vec(const bf16* p, float* x) {
  static_assert(VW == 4 || VW == 1, "vectors of 4 or single elements");
  if constexpr (VW == 4) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    x[0] = __uint_as_float(u.x << 16);
    x[1] = __uint_as_float(u.x & 0xffff0000u);
    x[2] = __uint_as_float(u.y << 16);
    x[3] = __uint_as_float(u.y & 0xffff0000u);
  } else {
    x[0] = __bfloat162float(*p);
  }
}
template <int VW>
__device__ __forceinline__ void store_vec(float* p, const float* x) {
  if constexpr (VW == 4)
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  else
    *p = x[0];
}
template <int VW>
__device__ __forceinline__ void store_vec(bf16* p, const float* x) {
  if constexpr (VW >= 4) {
    uint32_t q[VW / 2];
#pragma unroll
    for (int e = 0; e < VW / 2; ++e) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
      q[e] = *reinterpret_cast<const uint32_t*>(&h);
    }
    if constexpr (VW == 8)
      *reinterpret_cast<uint4*>(p) = make_uint4(q[0], q[1], q[2], q[3]);
    else
      *reinterpret_cast<uint2*>(p) = make_uint2(q[0], q[1]);
  } else {
    *p = __float2bfloat16_rn(x[0]);
  }
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// 16 bytes to shared memory without waiting
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// sigma(x) (1 / inf = 0 where exp(-x) overflows)
__device__ __forceinline__ float sigmoid(float x) { return rcp(1.f + ex2(-kLog2e * x)); }

// V floats in registers, as pairs where V is even
template <int V>
struct Vec {
  f2 p[V / 2];
  __device__ __forceinline__ float get(int i) const { return i & 1 ? hi(p[i / 2]) : lo(p[i / 2]); }
  __device__ __forceinline__ void fill(float x) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) p[i] = pk(x, x);
  }
  template <typename F>
  __device__ __forceinline__ void set(F f) {  // f(i): value i
#pragma unroll
    for (int i = 0; i < V / 2; ++i) p[i] = pk(f(2 * i), f(2 * i + 1));
  }
  __device__ __forceinline__ void fma(const Vec& a, const Vec& b, const Vec& c) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) p[i] = fma2(a.p[i], b.p[i], c.p[i]);
  }
  __device__ __forceinline__ void mul(const Vec& a, const Vec& b) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) p[i] = mul2(a.p[i], b.p[i]);
  }
  __device__ __forceinline__ void add(const Vec& a) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) p[i] = add2(p[i], a.p[i]);
  }
  __device__ __forceinline__ float sum() const {
    f2 s = p[0];
#pragma unroll
    for (int i = 1; i < V / 2; ++i) s = add2(s, p[i]);
    return lo(s) + hi(s);
  }
  // sigma of every value
  __device__ __forceinline__ void sigmoid(const Vec& a) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const f2 x = mul2(a.p[i], pk(-kLog2e, -kLog2e));
      const f2 y = add2(pk(ex2(lo(x)), ex2(hi(x))), pk(1.f, 1.f));
      p[i] = pk(rcp(lo(y)), rcp(hi(y)));
    }
  }
};
template <>
struct Vec<1> {
  float x;
  __device__ __forceinline__ float get(int) const { return x; }
  __device__ __forceinline__ void fill(float v) { x = v; }
  template <typename F>
  __device__ __forceinline__ void set(F f) { x = f(0); }
  __device__ __forceinline__ void fma(const Vec& a, const Vec& b, const Vec& c) { x = fmaf(a.x, b.x, c.x); }
  __device__ __forceinline__ void mul(const Vec& a, const Vec& b) { x = a.x * b.x; }
  __device__ __forceinline__ void add(const Vec& a) { x += a.x; }
  __device__ __forceinline__ float sum() const { return x; }
  __device__ __forceinline__ void sigmoid(const Vec& a) { x = rcp(1.f + ex2(-kLog2e * a.x)); }
};

// V consecutive elements of a row as they are in memory (V * sizeof(IO) bytes:
// a multiple of 4; V = 1: one element)
template <typename IO, int V>
struct Raw {
  static constexpr int W = (V * (int)sizeof(IO) + 3) / 4;
  uint32_t w[W];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ void load(const IO* p) {
    if constexpr (V * sizeof(IO) == 2) {
      w[0] = *reinterpret_cast<const unsigned short*>(p);
    } else if constexpr (W % 4 == 0) {
#pragma unroll
      for (int i = 0; i < W; i += 4) {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(p) + i / 4);
        w[i] = x.x; w[i + 1] = x.y; w[i + 2] = x.z; w[i + 3] = x.w;
      }
    } else if constexpr (W % 2 == 0) {
      const uint2 x = __ldg(reinterpret_cast<const uint2*>(p));
      w[0] = x.x; w[1] = x.y;
    } else {
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
    }
  }
  // (written out under both conditions: a value kept where there is nothing to
  // load would be selected after the load, which then waits for memory there)
  __device__ __forceinline__ void load_if(const IO* p, bool on) {
    if (on) load(p);
    else zero();
  }
  __device__ __forceinline__ void load_shared(const void* p) {
    static_assert(W == 4, "16 bytes");
    const uint4 x = *reinterpret_cast<const uint4*>(p);
    w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(IO) == 4) return __uint_as_float(w[i]);
    else return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
  // from floats, rounded once
  __device__ __forceinline__ void set(const float* x) {
    if constexpr (sizeof(IO) == 4) {
#pragma unroll
      for (int i = 0; i < V; ++i) w[i] = __float_as_uint(x[i]);
    } else if constexpr (V == 1) {
      const bf16 h = __float2bfloat16_rn(x[0]);
      w[0] = *reinterpret_cast<const unsigned short*>(&h);
    } else {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
  }
  __device__ __forceinline__ void put(IO* p) const {
    if constexpr (V * sizeof(IO) == 2) *reinterpret_cast<unsigned short*>(p) = (unsigned short)w[0];
    else if constexpr (W % 4 == 0) {
#pragma unroll
      for (int i = 0; i < W; i += 4)
        *(reinterpret_cast<uint4*>(p) + i / 4) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    } else if constexpr (W % 2 == 0) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(p) = w[0];
  }
};

template <typename IO, int V>
__device__ __forceinline__ Vec<V> vec_of(const Raw<IO, V>& r) {
  Vec<V> v;
  v.set([&](int i) { return r.get(i); });
  return v;
}
template <typename IO, int V>
__device__ __forceinline__ void raw_of(Raw<IO, V>& r, const Vec<V>& v) {
  float x[V];
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = v.get(i);
  r.set(x);
}

// N consecutive floats from a 16-byte aligned address (any when N is not a
// multiple of 4)
template <int N>
__device__ __forceinline__ void load_floats(const float* p, float* x) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(p + i));
      x[i] = a.x; x[i + 1] = a.y; x[i + 2] = a.z; x[i + 3] = a.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = __ldg(p + i);
  }
}

template <int V>
__device__ __forceinline__ Vec<V> vec_at(const float* p) {
  float x[V];
  load_floats<V>(p, x);
  Vec<V> v;
  v.set([&](int i) { return x[i]; });
  return v;
}

// Tokens of sequence b (lens nullable, clamped to [0, T])
__device__ __forceinline__ int seq_len(const int64_t* lens, int b, int T) {
  if (!lens) return T;
  const long long l = lens[b];
  return l < 0 ? 0 : (l > T ? T : (int)l);
}

// ---- host -----------------------------------------------------------------

// Shared memory beyond 48 KB has to be asked for
template <class Kern>
inline cudaError_t want_smem(Kern k, size_t smem) {
  return smem > 48 * 1024 ? cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)
                          : cudaSuccess;
}

inline lz_status layer_fail(lz_status st, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return (lz_status)set_last_error(st, buf);
}

inline lz_status layer_done(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return (lz_status)set_last_error(LZ_OK, "");
  return layer_fail(LZ_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// A pointer of the call: its name for messages, whether it must be given, and
// the alignment that it needs.
struct PtrRule {
  const void* p;
  const char* name;
  bool required;
  unsigned align;
};

inline lz_status check_ptrs(const char* fn, std::initializer_list<PtrRule> rules) {
  for (const PtrRule& r : rules) {
    if (!r.p) {
      if (r.required) return layer_fail(LZ_ERR_INVALID_ARG, "%s: %s must not be NULL", fn, r.name);
      continue;
    }
    if (reinterpret_cast<uintptr_t>(r.p) % r.align)
      return layer_fail(LZ_ERR_INVALID_ARG, "%s: %s must be %u-byte aligned", fn, r.name, r.align);
  }
  return LZ_OK;
}

// An output that is also an input or another output (by its pointer)
inline lz_status check_distinct(const char* fn, std::initializer_list<const void*> outs,
                                std::initializer_list<const void*> ins) {
  for (const void* const* o = outs.begin(); o != outs.end(); ++o) {
    if (!*o) continue;
    for (const void* const* q = o + 1; q != outs.end(); ++q)
      if (*o == *q) return layer_fail(LZ_ERR_INVALID_ARG, "%s: two outputs overlap", fn);
    for (const void* i : ins)
      if (*o == i) return layer_fail(LZ_ERR_INVALID_ARG, "%s: an output overlaps an input", fn);
  }
  return LZ_OK;
}

inline size_t esize(lz_dtype io) { return io == LZ_BF16 ? 2 : 4; }
inline bool io_ok(lz_dtype io) { return io == LZ_BF16 || io == LZ_F32; }

inline Rows rows_of(const lz_rows& r, int T, int width) {
  if (r.ld == 0) return Rows{width, (int64_t)T * width};
  return Rows{r.ld, r.bs};
}
inline bool rows_ok(const lz_rows& r) {
  return r.ld >= 0 && r.bs >= 0 && r.ld < (int64_t(1) << 40) && r.bs < (int64_t(1) << 50);
}

// Whether 16-byte vectors of VW elements can be read from these rows
inline bool rows_vec(const void* p, const Rows& r, int vw, size_t es) {
  return !p || (reinterpret_cast<uintptr_t>(p) % (vw * es) == 0 && r.ld % vw == 0 && r.bs % vw == 0);
}

constexpr size_t kWsAlign = 256;
inline size_t ws_round(size_t x) { return (x + kWsAlign - 1) / kWsAlign * kWsAlign; }

// Sum of P rows (ld floats apart) of c0 + c1 + c2 columns, in a fixed order,
// handed out to up to three outputs (a NULL output is skipped).
struct SumRowsParams {
  const float* part;
  int P;
  size_t ld;
  float* out0;
  size_t c0;
  float* out1;
  size_t c1;
  float* out2;
  size_t c2;
};
cudaError_t launch_sum_rows(const SumRowsParams& p, cudaStream_t s);

size_t conv_bwd_ws(const lz_conv_dims* d);
size_t scan_ws(const lz_scan_dims* d, int which);
size_t norm_bwd_ws(const lz_norm_dims* d);

}  // namespace lz
