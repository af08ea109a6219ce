// Shared parts of the selective state space scan kernels.
//
// Layout of the work: a channel's N states lie across L = ceil(N/4) lanes
// (rounded up to a power of two) of a warp, 4 states a lane, and a block of
// 128 threads holds 128/L neighbouring channels of one sequence.  The tokens
// are walked in tiles that are staged in shared memory; the state stays in
// registers.  One exp per (token, channel, state) cannot be done without:
// 16 a cycle and SM, which outweighs the tokens' bytes.
#pragma once

#include "layer.cuh"

namespace lz {
namespace scan {

constexpr int NT = 128;      // threads of a block
constexpr int kCk = 16;      // tokens between two saved states
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct ScanParams {
  int B, T, D, G, N, softplus;
  int nct;       // channel tiles of a group
  int seg, nseg; // tokens of a segment, segments
  bool vec, vecbc;  // 16-byte rows of u, dt, z, dy and outputs; 4-element rows of B, C
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
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ f2 ex2v(f2 x) { return pk(ex2(lo(x)), ex2(hi(x))); }

__device__ __forceinline__ float softplus(float x) { return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))); }

template <int BYTES>
__device__ __forceinline__ void cp_async(void* dst, const void* src) {
  const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(d), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// Stages a tile of TT rows x W elements: rows t0 .. of sequence b, columns c0
// .. ; what lies outside (t >= tmax, column >= cmax) becomes zero.  VW-element
// asynchronous copies where the rows allow them, else plain loads.
template <typename IO, int TT, int W, int VW>
__device__ __forceinline__ void stage(IO* dst, const void* src, const Rows& r, int b, int t0, int tmax, int c0,
                                      int cmax, bool vec) {
  const IO* s = (const IO*)src;
  if (vec) {
    for (int i = threadIdx.x; i < TT * (W / VW); i += NT) {
      const int t = i / (W / VW), c = i % (W / VW) * VW;
      IO* d = dst + t * W + c;
      if (t0 + t < tmax && c0 + c < cmax) {
        cp_async<VW * (int)sizeof(IO)>(d, s + r.at(b, t0 + t) + c0 + c);
      } else {
#pragma unroll
        for (int e = 0; e < VW; ++e) d[e] = from_f<IO>(0.f);
      }
    }
  } else {
    for (int i = threadIdx.x; i < TT * W; i += NT) {
      const int t = i / W, c = i % W;
      dst[i] = t0 + t < tmax && c0 + c < cmax ? s[r.at(b, t0 + t) + c0 + c] : from_f<IO>(0.f);
    }
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

template <int L>
struct Geo {
  static constexpr int CH = NT / L;         // channels of a block
  static constexpr int NP = 4 * L;          // states, padded
  static constexpr int U = L < 4 ? L : 4;   // tokens whose lane sums are formed together
  static constexpr int PAD = 32 / L < 4 ? 4 : 32 / L;
  static constexpr int YS = CH + PAD;       // row of a [tokens][channels] fp32 tile
};

// Floats from one partial row of the parameter gradients to the next: rows
// are written in vectors of 4
__host__ __device__ inline size_t part_ld(int D, int N) { return ((size_t)D * (N + 2) + 3) / 4 * 4; }

inline int lanes_of(int N) {
  int l = 1;
  while (4 * l < N) l *= 2;
  return l;
}

}  // namespace scan

cudaError_t launch_scan_fwd(const scan::ScanParams& p, int L, bool bf, cudaStream_t s);
cudaError_t launch_scan_bwd(const scan::ScanParams& p, int L, bool bf, cudaStream_t s);

}  // namespace lz
