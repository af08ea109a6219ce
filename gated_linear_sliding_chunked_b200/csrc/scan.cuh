// Shared parts of the selective state space scan kernels.
//
// Layout of the work: a channel's states lie across lanes of a warp, 4 states of
// a channel to a thread in the forward, 2 neighbouring states of 2 neighbouring
// channels in the backward; the W scan warps of a block hold 128 W / N channels
// (N rounded up to a power of two) of one sequence.  The tokens are walked in
// tiles.  As many warps more (or twice as many) do what is elementwise in
// (token, channel): while the scan warps walk a tile, they finish the outputs
// of the tile before and prepare the steps (softplus), inputs and gates of the
// tile behind, whose global loads they issued a tile earlier.  One block-wide
// barrier a tile hands the shared memory buffers over.  Without the split the
// scan warps would wait out the loads, the softplus and the stores of every
// tile, with too few warps on an SM to hide it: a layer has only (sequences x
// channels x N/4)/32 of them.  (2 x 8192 tokens, 4096 channels, 16 states:
// forward 1330 -> 775 us, backward 3489 -> 2033 us with the split.)
//
// One exp per (token, channel, state) cannot be done without: 16 a cycle and
// SM, which outweighs the tokens' bytes.
#pragma once

#include "layer.cuh"

namespace lz {
namespace scan {

constexpr int kCk = 16;      // tokens between two saved states

struct ScanParams {
  int B, T, D, G, N, softplus;
  int W;         // scan warps of a block (4 or 7), and elementwise warps
  int nct;       // channel tiles of a group
  int seg, nseg; // tokens of a segment, segments
  bool vec, vecbc;  // rows of 16-byte vectors: u, dt, z, dy and outputs; of 4 elements: B, C
  Rows ru, rdt, rz, rb, rc;
  const void* u;
  const void* dt;
  const float* A;
  const void* Bm;
  const void* Cm;
  const float* Dskip;
  const void* z;
  const float* dtb;
  const float* h0;
  const int64_t* lens;
  void* y;
  float* hT;
  float* states;  // [B][ceil(T/16)][D][N]: the state before every 16th token
  // the segments' effect on the state that enters (forward) or the gradient
  // that leaves (backward): end value from a zero start, sum of delta
  float* segE;    // [nseg][B][D][N]
  float* segD;    // [nseg][B][D]
  // backward
  const void* dy;
  const float* dhT;
  void* du;
  void* ddt;
  void* dz;
  float* dh0;
  float* part;    // [B * nseg][part_ld]: dA, dDskip, ddt_bias
  float* bc;      // [nct][B][T][G][2][N]: dB, dC of a channel tile
  void* dB;
  void* dC;
};

// 2^(A2 d), the decay.  Its errors add up over a state's memory, so their mean
// counts.  The special-function unit's results just below 1 are too small on
// average (measured over the arguments of each binade): by 1.6e-8 to 2.7e-8 for
// exponents of 2^-8 to 1, by 5e-9 to 8e-9 for smaller ones, whose states remember
// longest.  2^-26 in the exponent leaves at most 1.6e-8 of the former and 5e-9 of
// the latter.  (Twice and three times as much centres the fast decays, and takes
// the slow ones off by 1e-8 and 2.4e-8: the gradient of A after 8192 tokens with
// rates of 1 and steps of 0.001 is off by 3.1e-6 with 2^-26, 3.9e-6 with nothing,
// 1.5e-5 with 4.2e-8; torch's products of 32-bit exps by 2.3e-5.  A polynomial took
// half as long again.)
constexpr float kCut = 0x1p-26f;
__device__ __forceinline__ f2 decay(f2 A2, f2 d) {
  const f2 x = fma2(A2, d, pk(kCut, kCut));
  return pk(ex2(lo(x)), ex2(hi(x)));
}

// 2^(A2 d) h + e: a state h carried over a segment whose steps add up to d, with
// what the segment adds to it.  Where rates grow, the factor alone can be more
// than a float holds while its product with h (none, or a small one) is not, so
// that h is multiplied by the factor's root twice.
__device__ __forceinline__ f2 carry(f2 A2, f2 d, f2 h, f2 e) {
  const f2 x = fma2(A2, d, pk(kCut, kCut));
  const f2 r = pk(ex2(fminf(0.5f * lo(x), 127.99f)), ex2(fminf(0.5f * hi(x), 127.99f)));
  return fma2(mul2(h, r), r, e);
}

// softplus(x) = max(x, 0) + log1p(e), e = exp(-|x|), and its derivative
// sigma(x).  log1p(e) = 2 atanh(s) with s = e / (2 + e) <= 1/3, by the series
// s + s^3/3 + .. + s^15/15 (the rest is below 2^-29 of it): accurate relative
// to the result also where e is small, which is where steps live.
__device__ __forceinline__ float softplus_of(float x, float s) {
  const float q = s * s;
  float p = fmaf(q, 1.f / 15.f, 1.f / 13.f);
  p = fmaf(q, p, 1.f / 11.f);
  p = fmaf(q, p, 1.f / 9.f);
  p = fmaf(q, p, 1.f / 7.f);
  p = fmaf(q, p, 1.f / 5.f);
  p = fmaf(q, p, 1.f / 3.f);
  const float t = s + s;
  return fmaxf(x, 0.f) + fmaf(t * q, p, t);
}
__device__ __forceinline__ float softplus(float x) {
  const float e = ex2(-kLog2e * fabsf(x));
  return softplus_of(x, e * rcp(2.f + e));
}
// with sigma(x), both quotients from one reciprocal
__device__ __forceinline__ float softplus(float x, float& sg) {
  const float e = ex2(-kLog2e * fabsf(x)), a = 1.f + e, b = 2.f + e, r = rcp(a * b);
  sg = b * r * (x >= 0.f ? 1.f : e);
  return softplus_of(x, e * a * r);
}

// V consecutive elements of a row as they are in memory
template <typename IO, int V>
struct Pack {
  static constexpr int W = V * (int)sizeof(IO) / 4;
  uint32_t w[W];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(IO) == 4) return __uint_as_float(w[i]);
    else return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
  __device__ __forceinline__ void put(IO* p) const {  // to shared memory
    if constexpr (W == 4) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
  // n of the V elements exist; the rest becomes zero.  In 16-, 8- or 4-byte
  // accesses when vec: the row allows it and n is V or none.  (Written out
  // under both conditions: a value kept where there is nothing to load would be
  // selected after the load, which then waits for memory there and then.)
  __device__ __forceinline__ void load(const IO* p, int n, bool vec) {
    if (vec) {
      if (n > 0) {
        if constexpr (W % 4 == 0) {
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
      } else {
        zero();
      }
    } else {
      zero();
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i < n) {
          if constexpr (sizeof(IO) == 4) w[i] = __float_as_uint(p[i]);
          else w[i / 2] |= (uint32_t)reinterpret_cast<const unsigned short*>(p)[i] << (16 * (i & 1));
        }
    }
  }
};

// V floats from shared memory (16- or 8-byte aligned as V allows)
template <int V>
__device__ __forceinline__ void load_f(const float* p, float* x) {
  if constexpr (V % 4 == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 a = *reinterpret_cast<const float4*>(p + i);
      x[i] = a.x; x[i + 1] = a.y; x[i + 2] = a.z; x[i + 3] = a.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const float2 a = *reinterpret_cast<const float2*>(p + i);
      x[i] = a.x; x[i + 1] = a.y;
    }
  }
}

// V values to consecutive elements, n of which exist
template <typename IO, int V>
__device__ __forceinline__ void store_n(IO* p, const float* x, int n, bool vec) {
  if (vec) {
    if (n > 0) {
      Raw<IO, V> r;
      r.set(x);
      r.put(p);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) p[i] = from_f<IO>(x[i]);
  }
}

// Sum over the lanes that differ in the bits M, M/2 .. LO of the lane index,
// handing the CNT values out over them: each step halves the values a lane
// keeps (the upper half where the bit is set) until one is left, then adds
// whole.  `base` becomes the index of the first value kept.
template <int CNT, int M, int LO, int SZ>
__device__ __forceinline__ void reduce_scatter(float (&v)[SZ], int lane, int& base) {
  if constexpr (M >= LO && M > 0) {
    if constexpr (CNT > 1) {
      constexpr int H = CNT / 2;
      const bool up = lane & M;
#pragma unroll
      for (int i = 0; i < H; ++i) {
        const float send = up ? v[i] : v[i + H], keep = up ? v[i + H] : v[i];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, send, M);
      }
      base += up ? H : 0;
      reduce_scatter<H, M / 2, LO>(v, lane, base);
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], M);
      reduce_scatter<1, M / 2, LO>(v, lane, base);
    }
  }
}

// Row of a [tokens][CH] fp32 tile: CH or a little more, of which x is left over 32 banks
constexpr int row_of(int CH, int x) { return CH + (x - CH % 32 + 32) % 32; }

// Floats from one partial row of the parameter gradients to the next: rows
// are written in vectors of 4
__host__ __device__ inline size_t part_ld(int D, int N) { return ((size_t)D * (N + 2) + 3) / 4 * 4; }

// N rounded up to a power of two, at least 4
inline int states_of(int N) {
  int n = 4;
  while (n < N) n *= 2;
  return n;
}

}  // namespace scan

cudaError_t launch_scan_fwd(const scan::ScanParams& p, bool bf, cudaStream_t s);
cudaError_t launch_scan_bwd(const scan::ScanParams& p, bool bf, cudaStream_t s);

}  // namespace lz
