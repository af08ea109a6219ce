// Norms before and after a block, fused with its gate and residual scale:
//   m = rmsnorm_groups(o) w,  out = [r +] m [silu(z)] [s],  n = rmsnorm(out) w2
//
// A row of D features stays in registers between its two norms: every input
// is read once and every output written once, a few operations an element, so
// HBM bandwidth bounds it (forward up to 5 values an element, backward up to
// 8).  A thread holds 16 elements; up to 512 elements a row belongs to 4 to 32
// lanes of a warp (no block-wide synchronisation), longer rows to a block.  The
// forward takes a row a team; the backward's blocks walk the rows with a stride,
// the next row on its way to shared memory while this one is worked on, so that
// the parameter gradients stay in registers and leave as one partial per block.
// At 2 x 8192 rows of 4096 (bf16): forward by 32 heads with a gate 76 to 80 us
// (77 % of the copy bandwidth), backward of everything 246 to 254 us (66 %: two
// sums over a row, with a barrier each, between its loads and its stores); rows
// of 1024: backward 68 us (60 %).  Rows too long for the backward's ring (above 5120
// 32-bit features, 8192 16-bit ones, or 4096 where vectors are single elements) run
// on blocks of up to 1024 threads, whose 64 registers spill: 4096 x 8192 in 32 bits
// 484 us against a floor of 164, 4096 x 16384 in 16 bits 661 us.
#include "layer.cuh"

namespace lz {
namespace {

constexpr int kMaxD = 16384;  // 1024 threads of 16 elements
constexpr int kWarpBlock = 128;  // threads of a block whose rows belong to (parts of) warps

inline int shift_of(int n) {
  int s = 0;
  while ((1 << s) < n) ++s;
  return (1 << s) == n ? s : -1;
}

// How the sums over a group of features are formed: the group is the whole
// row; a power-of-two number of neighbouring lanes; anything else (partial
// sums in shared memory, a warp per group).
enum { GROUP_ROW = 0, GROUP_LANES = 1, GROUP_SMEM = 2 };

struct NormParams {
  int64_t rows;
  int B, T, D, G, heads;
  int dshift;  // log2 of the features of a group, -1 when that is no power of two
  float eps;
  Rows so, sz, sr;
  const void* o;
  const float* w;
  const void* z;
  const float* s;
  const void* r;
  const float* w2;
  void* out;
  void* n;
  // backward
  const void* dout;
  const void* dn;
  void* d_o;
  void* dz;
  void* dr;
  float* part;  // [blocks][3][D]: dw, ds, dw2
  int ring;     // floats of shared memory in front of the rows in flight
  int team, tshift;  // lanes of a row that belongs to a warp or a part of one, log2 of it
};

// Sums of M values over the team that holds a row: 4 to 32 lanes of a warp, or a
// block.  One barrier: a caller alternates between two `red` of M * 32 floats, so
// that a buffer is written again only after a barrier that its readers have passed.
template <bool WARP, int M>
__device__ __forceinline__ void team_sum(float (&v)[M], int team, float* red) {
  if constexpr (WARP) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (team > o) {
#pragma unroll
        for (int i = 0; i < M; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
      }
  } else {
#pragma unroll
    for (int i = 0; i < M; ++i) v[i] = warp_sum(v[i]);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, nw = blockDim.x / 32;
    if (lane < M) {
      float x = v[0];
#pragma unroll
      for (int i = 1; i < M; ++i) x = lane == i ? v[i] : x;
      red[lane * 32 + warp] = x;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < M; ++i) v[i] = warp_sum(lane < nw ? red[i * 32 + lane] : 0.f);
  }
}

// Per-vector partial sums ps[k] -> the sum over each vector's group
template <int E, int VW, bool WARP, int MODE>
__device__ __forceinline__ void group_sum(const NormParams& p, float* ps, int lane, int team, float* red,
                                          float* sm) {
  constexpr int NV = E / VW;
  const int nvec = p.D / VW;
  if constexpr (MODE == GROUP_ROW) {
    float a[1] = {0.f};
#pragma unroll
    for (int k = 0; k < NV; ++k) a[0] += ps[k];
    team_sum<WARP>(a, team, red);
#pragma unroll
    for (int k = 0; k < NV; ++k) ps[k] = a[0];
  } else if constexpr (MODE == GROUP_LANES) {
    const int gv = nvec / p.G;  // lanes of a group: 1, 2, .. 32
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (gv > o) {
#pragma unroll
        for (int k = 0; k < NV; ++k) ps[k] += __shfl_xor_sync(0xffffffffu, ps[k], o);
      }
  } else {  // (block teams only) sm: nvec partials, then G sums
    const int gv = nvec / p.G, warp = threadIdx.x / 32, l = threadIdx.x % 32;
    float* gs = sm + nvec;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = k * team + lane;
      if (v < nvec) sm[v] = ps[k];
    }
    __syncthreads();
    for (int g = warp; g < p.G; g += blockDim.x / 32) {
      float a = 0.f;
      for (int x = l; x < gv; x += 32) a += sm[g * gv + x];
      a = warp_sum(a);
      if (l == 0) gs[g] = a;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = k * team + lane;
      ps[k] = v < nvec ? gs[v / gv] : 0.f;
    }
  }
}

// Where a row's features stand: a run of them, or (heads) a run of D/G in each
// head's [T, D/G].
template <typename IO>
struct RowAt {
  IO* p;
  int64_t head;  // elements from head to head
  int dv, dshift, heads;
  __device__ __forceinline__ IO* at(int c) const {
    if (!heads) return p + c;
    const int g = dshift >= 0 ? c >> dshift : c / dv;
    return p + (g * head + (c - g * dv));
  }
};
template <typename IO>
__device__ __forceinline__ RowAt<IO> row_at(const NormParams& p, IO* base, const Rows& so, int b, int t) {
  const int dv = p.D / p.G;
  const int64_t head = (int64_t)p.T * dv;
  return {base + (p.heads ? b * p.G * head + (int64_t)t * dv : (int64_t)so.at(b, t)), head, dv, p.dshift, p.heads};
}

// Blocks of 256 threads that share an SM in the forward.  16-bit rows of 4096
// features: five (2 x 8192 rows of 32 groups: 80 us against 86 us with the four
// that 60 registers would allow); the others need more registers.
template <typename IO, int VW>
constexpr int kFwdBlocks = VW == 1 ? 4 : sizeof(IO) == 4 ? 3 : 5;

// E: elements of a thread.  FULL: every thread has E features (D is the team's
// threads times E).
template <typename IO, int E, int VW, bool WARP, int MODE, bool FULL, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == 256 ? kFwdBlocks<IO, VW> : 1) norm_fwd_kernel(NormParams p) {
  extern __shared__ __align__(16) float sm[];
  __shared__ float red[2][3 * 32];
  constexpr int NV = E / VW;
  using V = Vec<VW>;
  const int team = WARP ? p.team : blockDim.x;
  const int lane = WARP ? threadIdx.x & (team - 1) : threadIdx.x;
  const int nvec = p.D / VW;
  const int b = blockIdx.y;
  const unsigned ut = WARP ? blockIdx.x * (kWarpBlock >> p.tshift) + (threadIdx.x >> p.tshift) : blockIdx.x;
  const int t = (int)ut;
  const bool live = !WARP || ut < (unsigned)p.T;  // (the lanes of a warp stay together for its sums)
  auto has = [&](int k) { return live && (FULL || k * team + lane < nvec); };
  auto col = [&](int k) { return (k * team + lane) * VW; };
  const int64_t row = ((int64_t)b * p.T + t) * p.D;
  const auto o = row_at<const IO>(p, (const IO*)p.o, p.so, b, t);
  const IO* pz = p.z ? (const IO*)p.z + p.sz.at(b, t) : nullptr;
  const IO* pr = p.r ? (const IO*)p.r + p.sr.at(b, t) : nullptr;
  Raw<IO, VW> ro[NV], rz[NV], rr[NV];  // the row, all of it in flight at once
#pragma unroll
  for (int k = 0; k < NV; ++k) ro[k].load_if(o.at(col(k)), has(k));
  if (pz) {
#pragma unroll
    for (int k = 0; k < NV; ++k) rz[k].load_if(pz + col(k), has(k));
  }
  if (pr) {
#pragma unroll
    for (int k = 0; k < NV; ++k) rr[k].load_if(pr + col(k), has(k));
  }
  V x[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) x[k] = vec_of(ro[k]);
  if (p.w) {
    float ps[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      V q;
      q.mul(x[k], x[k]);
      ps[k] = q.sum();
    }
    group_sum<E, VW, WARP, MODE>(p, ps, lane, team, red[0], sm);
    const float ig = (float)p.G / (float)p.D;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (!has(k)) continue;
      V rs, w = vec_at<VW>(p.w + col(k));
      rs.fill(rsqrtf(ps[k] * ig + p.eps));
      w.mul(w, rs);
      x[k].mul(x[k], w);
    }
  }
  if (pz) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      V z = vec_of(rz[k]), sg;
      sg.sigmoid(z);
      z.mul(z, sg);
      x[k].mul(x[k], z);
    }
  }
  if (p.s) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (has(k)) x[k].mul(x[k], vec_at<VW>(p.s + col(k)));
  }
  if (pr) {
#pragma unroll
    for (int k = 0; k < NV; ++k) x[k].add(vec_of(rr[k]));
  }
  float ss[1] = {0.f};
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    if (!has(k)) continue;
    raw_of(ro[k], x[k]);
    ro[k].put((IO*)p.out + row + col(k));
    // the second norm is that of the stored stream, so that the backward finds
    // the same values in it
    if (p.w2) {
      x[k] = vec_of(ro[k]);
      V q;
      q.mul(x[k], x[k]);
      ss[0] += q.sum();
    }
  }
  if (p.w2) {
    team_sum<WARP>(ss, team, red[1]);
    V rs;
    rs.fill(rsqrtf(ss[0] / (float)p.D + p.eps));
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (!has(k)) continue;
      V w = vec_at<VW>(p.w2 + col(k));
      w.mul(w, rs);
      x[k].mul(x[k], w);
      raw_of(ro[k], x[k]);
      ro[k].put((IO*)p.n + row + col(k));
    }
  }
}

// Backward.  With xh = out rs2 and q = dn w2 the gradient at `out` is
//   e = dout + rs2 (q - xh mean(q xh))           (= dr)
// and with mh = o rs, core = mh w, f = e s:
//   ds = sum e core silu(z)     dz = f core silu'(z)     dw = sum f silu(z) mh
//   do = rs (k - mh mean_group(k mh)),  k = f silu(z) w
template <typename IO, int E, int VW, bool WARP, int MODE, bool FULL, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT <= 512 ? (VW == 1 ? 768 : 512) / MAXT : 1) norm_bwd_kernel(NormParams p) {
  extern __shared__ __align__(16) float sm[];
  __shared__ float red[2][3 * 32];
  constexpr int NV = E / VW;
  using V = Vec<VW>;
  const int team = WARP ? p.team : blockDim.x;
  const int lane = WARP ? threadIdx.x & (team - 1) : threadIdx.x;
  const int nvec = p.D / VW;
  auto col = [&](int k) { return (k * team + lane) * VW; };
  // a warp's rows follow one another: it goes on while the first is there
  const int sub = WARP ? (threadIdx.x & 31) >> p.tshift : 0;
  const int64_t row0 = WARP ? (((int64_t)blockIdx.x * kWarpBlock + threadIdx.x) >> p.tshift) - sub : blockIdx.x;
  const int64_t step = WARP ? (int64_t)gridDim.x * (kWarpBlock >> p.tshift) : gridDim.x;
  auto there = [&](int64_t row, int k) {
    return (!WARP || row < p.rows) && (FULL || k * team + lane < nvec);
  };
  const float ig = (float)p.G / (float)p.D, id = 1.f / (float)p.D;
  const Rows cont{p.D, (int64_t)p.T * p.D};
  // sum over the rows of e silu(z) mh: times s it is dw, times w ds
  V sm0[NV], dw2[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    sm0[k].fill(0.f);
    dw2[k].fill(0.f);
  }
  // RING: the next row is copied to shared memory while this one is worked on,
  // every thread its own vectors (so that no barrier is needed); in registers it
  // would cost 40 of them.  (The threads' vectors lie side by side: where a
  // thread's own did, the copies of a warp's 512 bytes went to 32 places and the
  // whole took 380 us, not 250.)
  constexpr bool RING = VW > 1 && MAXT <= 512;
  enum { O, Z, OUT, DOUT, DN, N_IN };
  struct In {
    Raw<IO, VW> v[N_IN][NV];
  };
  In in;
  uint4* ring = reinterpret_cast<uint4*>(sm + p.ring) + threadIdx.x;  // [2][N_IN][NV][threads]
  const int bd = WARP ? kWarpBlock : blockDim.x;
  auto slot = [&](int st, int i, int k) -> uint4* { return ring + ((st * N_IN + i) * NV + k) * bd; };
  auto fetch = [&](int64_t row, int st) {
    const int b = (int)((unsigned)row / (unsigned)p.T), t = (int)row - b * p.T;
    const size_t at = (size_t)row * p.D;
    auto has = [&](int k) { return there(row, k); };
    auto one = [&](int i, int k, const IO* q) {
      if constexpr (RING) {
        if (has(k)) cp_async16(slot(st, i, k), q);
      } else {
        in.v[i][k].load_if(q, has(k));
      }
    };
    if (p.dn) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        one(OUT, k, (const IO*)p.out + at + col(k));
        one(DN, k, (const IO*)p.dn + at + col(k));
      }
    }
    const auto o = row_at<const IO>(p, (const IO*)p.o, p.so, b, t);
#pragma unroll
    for (int k = 0; k < NV; ++k) one(O, k, o.at(col(k)));
    if (p.dout) {
#pragma unroll
      for (int k = 0; k < NV; ++k) one(DOUT, k, (const IO*)p.dout + at + col(k));
    }
    if (p.z) {
      const IO* pz = (const IO*)p.z + p.sz.at(b, t);
#pragma unroll
      for (int k = 0; k < NV; ++k) one(Z, k, pz + col(k));
    }
    if constexpr (RING) cp_commit();
  };
  int st = 0;
  int64_t row = row0 + sub;
  auto has = [&](int k) { return there(row, k); };
  auto val = [&](int i, int k) -> V {
    if constexpr (RING) {
      Raw<IO, VW> r;
      r.zero();
      if (has(k)) r.load_shared(slot(st, i, k));
      return vec_of(r);
    } else {
      return vec_of(in.v[i][k]);
    }
  };
  int turn = 0;  // of the two buffers of the block's sums
  if (RING && row0 < p.rows) fetch(row, 0);
  for (; row - sub < p.rows; row += step, st ^= RING) {
    if constexpr (RING) {
      if (row - sub + step < p.rows) {
        fetch(row + step, st ^ 1);
        cp_wait<1>();
      } else {
        cp_wait<0>();
      }
    } else {
      fetch(row, 0);
    }
    const int64_t at = row * p.D;
    V e[NV], x[NV];
    float ps[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      x[k] = val(O, k);
      V q;
      q.mul(x[k], x[k]);
      ps[k] = q.sum();
      if (p.dout) e[k] = val(DOUT, k);
      else e[k].fill(0.f);
    }
    // first sums: of out^2, of q out and (one group) of o^2
    float sums[3] = {0.f, 0.f, 0.f};
    if (p.dn) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (!has(k)) continue;
        V xo = val(OUT, k), q = val(DN, k), s;
        q.mul(q, vec_at<VW>(p.w2 + col(k)));
        s.mul(xo, xo);
        sums[0] += s.sum();
        q.mul(q, xo);
        sums[1] += q.sum();
      }
    }
    if constexpr (MODE == GROUP_ROW) {
#pragma unroll
      for (int k = 0; k < NV; ++k) sums[2] += ps[k];
    }
    if (p.dn || (MODE == GROUP_ROW && p.w)) {
      team_sum<WARP>(sums, team, red[turn]);
      turn ^= 1;
    }
    if constexpr (MODE == GROUP_ROW) {
#pragma unroll
      for (int k = 0; k < NV; ++k) ps[k] = sums[2];
    } else {
      if (p.w) group_sum<E, VW, WARP, MODE>(p, ps, lane, team, nullptr, sm);
    }
    if (p.dn) {
      const float r2s = rsqrtf(sums[0] * id + p.eps);
      V r2, m;
      r2.fill(r2s);
      m.fill(-sums[1] * id * r2s * r2s * r2s);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (!has(k)) continue;
        V xo = val(OUT, k), q = val(DN, k);
        q.mul(q, r2);  // dn rs2
        dw2[k].fma(q, xo, dw2[k]);
        e[k].fma(q, vec_at<VW>(p.w2 + col(k)), e[k]);
        e[k].fma(xo, m, e[k]);
      }
    }
    if (p.dr) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (!has(k)) continue;
        Raw<IO, VW> r;
        raw_of(r, e[k]);
        r.put((IO*)p.dr + at + col(k));
      }
    }
    float rs[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      rs[k] = p.w ? rsqrtf(ps[k] * ig + p.eps) : 1.f;
      ps[k] = 0.f;
      if (!has(k)) continue;
      V f;  // w s
      f.fill(rs[k]);
      x[k].mul(x[k], f);  // mh
      if (p.w) {
        f = vec_at<VW>(p.w + col(k));
        if (p.s) f.mul(f, vec_at<VW>(p.s + col(k)));
      } else if (p.s) {
        f = vec_at<VW>(p.s + col(k));
      } else {
        f.fill(1.f);
      }
      if (p.z) {
        const V z = val(Z, k);
        V sg, si, d;
        sg.sigmoid(z);
        si.mul(z, sg);
        if (p.dz) {  // sg + si - si sg
          V one;
          one.fill(1.f);
          d.fill(-1.f);
          d.fma(sg, d, one);
          d.fma(si, d, sg);
          d.mul(d, e[k]);
          d.mul(d, x[k]);
          d.mul(d, f);
          Raw<IO, VW> r;
          raw_of(r, d);
          r.put((IO*)p.dz + at + col(k));
        }
        e[k].mul(e[k], si);
      }
      sm0[k].fma(e[k], x[k], sm0[k]);
      e[k].mul(e[k], f);  // the gradient at mh
      V q;
      q.mul(e[k], x[k]);
      ps[k] = q.sum();
    }
    if (p.w) {
      group_sum<E, VW, WARP, MODE>(p, ps, lane, team, red[turn], sm);
      turn ^= MODE == GROUP_ROW;
    }
    const int b = (int)((unsigned)row / (unsigned)p.T), t = (int)row - b * p.T;
    const auto d_o = row_at<IO>(p, (IO*)p.d_o, cont, b, t);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (!has(k)) continue;
      if (p.w) {
        V m, r;
        m.fill(-ps[k] * ig);
        r.fill(rs[k]);
        e[k].fma(x[k], m, e[k]);
        e[k].mul(e[k], r);
      }
      Raw<IO, VW> r;
      raw_of(r, e[k]);
      r.put(d_o.at(col(k)));
    }
  }
  // ---- the block's partials; the teams of a block of several rows are added
  // in order in shared memory
  auto value = [&](int q, int i, int c) {
    const float a = q == 2 ? dw2[i / VW].get(i % VW) : sm0[i / VW].get(i % VW);
    const float* f = q == 0 ? p.s : q == 1 ? p.w : nullptr;
    return f ? a * f[c] : a;
  };
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    float* part = p.part + ((size_t)blockIdx.x * 3 + q) * p.D;
    if constexpr (WARP) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int c = (i / VW * team + lane) * VW + i % VW;
        if (c < p.D) sm[(threadIdx.x >> p.tshift) * p.D + c] = value(q, i, c);
      }
      __syncthreads();
      for (int c = threadIdx.x; c < p.D; c += kWarpBlock) {
        float tot = 0.f;
        for (int w = 0; w < kWarpBlock >> p.tshift; ++w) tot += sm[w * p.D + c];
        part[c] = tot;
      }
    } else {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int v = k * team + lane;
        if (v < nvec) {
#pragma unroll
          for (int j = 0; j < VW; j += VW < 4 ? 1 : 4) {
            float f[VW < 4 ? 1 : 4];
#pragma unroll
            for (int i = 0; i < (VW < 4 ? 1 : 4); ++i) f[i] = value(q, k * VW + j + i, v * VW + j + i);
            if constexpr (VW < 4) part[v * VW + j] = f[0];
            else *reinterpret_cast<float4*>(part + v * VW + j) = make_float4(f[0], f[1], f[2], f[3]);
          }
        }
      }
    }
  }
}

// ---- host -----------------------------------------------------------------

struct Shape {
  bool warp;    // rows belong to warps or parts of them
  bool full;    // every thread of a team has E features
  int e, vw;    // elements of a thread, of a vector
  int team;     // threads of a row
  int threads;  // of a block
  int mode;
  size_t smem;  // of the group sums
};

// 16 elements a thread; fewer, up to 4096 features, where vectors are single
// elements, whose unpacked values take more registers (8192 rows of 1001 16-bit
// features: forward 8 elements 45 us, 4 elements 51, 16 elements 76; backward 125,
// 109 and 219 us).
Shape shape_of(const lz_norm_dims* d, bool vec, bool bwd) {
  Shape s;
  s.vw = vec ? (int)(16 / esize(d->io)) : 1;
  s.e = vec || d->D > 4096 ? 16 : bwd ? 4 : 8;
  const int nvec = d->D / s.vw;
  const int gd = d->D / d->G;
  const int gv = gd % s.vw == 0 ? gd / s.vw : 0;
  s.mode = d->G == 1 ? GROUP_ROW : (gv >= 1 && gv <= 32 && (gv & (gv - 1)) == 0) ? GROUP_LANES : GROUP_SMEM;
  // short rows: a power-of-two part of a warp each, no smaller than a group
  int lanes = 4;
  while (lanes * s.e < d->D || (s.mode == GROUP_LANES && lanes < gv)) lanes *= 2;
  s.warp = lanes <= 32 && s.mode != GROUP_SMEM;
  s.team = s.warp ? lanes : ((d->D + s.e - 1) / s.e + 31) / 32 * 32;
  s.threads = s.warp ? kWarpBlock : s.team;
  s.full = vec && d->D == s.team * s.e;
  s.smem = s.mode == GROUP_SMEM ? (size_t)(nvec + d->G) * sizeof(float) : 0;
  return s;
}

// Blocks that walk the rows: as many as fit the device at once
template <class Kern>
int grid_rows(Kern k, int64_t rows, int threads, size_t smem, int rows_per_block) {
  const int64_t want = (rows + rows_per_block - 1) / rows_per_block;
  if (want <= 148) return (int)std::max<int64_t>(1, want);
  int wave = resident_ctas(k, threads, smem);
  if (wave <= 0) wave = 148;
  return (int)std::max<int64_t>(1, std::min<int64_t>(want, wave));
}

template <typename IO, int VW, bool WARP, int MODE>
cudaError_t go_fwd(NormParams p, const Shape& sh, cudaStream_t s) {
  constexpr int kT = WARP ? kWarpBlock : 256;
  constexpr int kE = VW > 1 ? 16 : 8;
  p.team = sh.team;
  p.tshift = shift_of(sh.team);
  auto k = norm_fwd_kernel<IO, kE, VW, WARP, MODE, false, kT>;
  if constexpr (VW > 1) {
    if (sh.full) k = norm_fwd_kernel<IO, kE, VW, WARP, MODE, true, kT>;
  }
  if constexpr (!WARP) {
    if (sh.threads > kT) k = norm_fwd_kernel<IO, kE, VW, WARP, MODE, false, 1024>;
    if (sh.e != kE) k = norm_fwd_kernel<IO, 16, VW, WARP, MODE, false, 1024>;
  }
  const cudaError_t e = want_smem(k, sh.smem);
  if (e != cudaSuccess) return e;
  const int rpb = sh.threads / sh.team;
  const dim3 grid((p.T - 1) / rpb + 1, p.B);
  ScopedTiming tm("block_norm_fwd", s);
  k<<<grid, sh.threads, sh.smem, s>>>(p);
  return cudaGetLastError();
}

// Partials of the backward: a bound that needs no device
constexpr int kMaxBlocks = 148 * 8;
int bwd_part_rows(int64_t rows) { return (int)std::min<int64_t>(std::max<int64_t>(rows, 1), kMaxBlocks); }

template <typename IO, int VW, bool WARP, int MODE>
cudaError_t go_bwd(NormParams p, const Shape& sh, int* blocks, cudaStream_t s) {
  const int rpb = sh.threads / sh.team;
  size_t smem = WARP ? (size_t)rpb * p.D * sizeof(float) : sh.smem;
  constexpr int kT = WARP ? kWarpBlock : 256;
  constexpr int kE = VW > 1 ? 16 : 4;
  p.team = sh.team;
  p.tshift = shift_of(sh.team);
  p.ring = (int)((smem + 15) / 16 * 4);
  // two rows in flight beside the sums' scratch
  const size_t ring = (size_t)p.ring * 4 + 2 * 16 * 5 * (kE / VW) * (size_t)sh.threads;
  auto k = norm_bwd_kernel<IO, kE, VW, WARP, MODE, false, kT>;
  if constexpr (VW > 1) {
    if (sh.full) k = norm_bwd_kernel<IO, kE, VW, WARP, MODE, true, kT>;
  }
  bool ringed = VW > 1;
  if constexpr (!WARP) {
    if (sh.threads > kT) k = norm_bwd_kernel<IO, kE, VW, WARP, MODE, false, (VW > 1 ? 512 : 1024)>;
    // rows too long for that
    if (VW > 1 ? sh.threads > 512 || ring > 200 * 1024 : sh.e != kE) {
      k = norm_bwd_kernel<IO, 16, VW, WARP, MODE, false, 1024>;
      ringed = false;
    }
  }
  if (ringed) smem = ring;
  const cudaError_t e = want_smem(k, smem);
  if (e != cudaSuccess) return e;
  const int grid = std::min(grid_rows(k, p.rows, sh.threads, smem, rpb), bwd_part_rows(p.rows));
  *blocks = grid;
  ScopedTiming tm("block_norm_bwd", s);
  k<<<grid, sh.threads, smem, s>>>(p);
  return cudaGetLastError();
}

#define LZ_NORM_DISPATCH(CALL)                                              \
  do {                                                                      \
    if (d->io == LZ_BF16) {                                                 \
      if (sh.vw > 1) LZ_NORM_MODE(CALL, bf16, 8) else LZ_NORM_MODE(CALL, bf16, 1) \
    } else {                                                                \
      if (sh.vw > 1) LZ_NORM_MODE(CALL, float, 4) else LZ_NORM_MODE(CALL, float, 1) \
    }                                                                       \
  } while (0)
#define LZ_NORM_MODE(CALL, IO, VW)                                          \
  {                                                                         \
    if (sh.mode == GROUP_SMEM) e = CALL(IO, VW, false, GROUP_SMEM);         \
    else if (sh.mode == GROUP_ROW) e = sh.warp ? CALL(IO, VW, true, GROUP_ROW) : CALL(IO, VW, false, GROUP_ROW); \
    else e = sh.warp ? CALL(IO, VW, true, GROUP_LANES) : CALL(IO, VW, false, GROUP_LANES); \
  }

lz_status check_norm(const char* fn, const lz_norm_dims* d) {
  if (!d) return layer_fail(LZ_ERR_INVALID_ARG, "%s: dims must not be NULL", fn);
  if (d->B < 0 || d->T < 0 || d->D < 0)
    return layer_fail(LZ_ERR_INVALID_ARG, "%s: B, T, D must be >= 0 (got %d, %d, %d)", fn, d->B, d->T, d->D);
  if (!io_ok(d->io))
    return layer_fail(LZ_ERR_UNSUPPORTED, "%s: io dtype %d is not LZ_F32 or LZ_BF16", fn, (int)d->io);
  if (d->D > kMaxD) return layer_fail(LZ_ERR_UNSUPPORTED, "%s: D must be <= %d (got %d)", fn, kMaxD, d->D);
  if (d->G < 1 || d->D % d->G)
    return layer_fail(LZ_ERR_INVALID_ARG, "%s: G must be a divisor of D (got %d of %d)", fn, d->G, d->D);
  if (d->heads != 0 && d->heads != 1)
    return layer_fail(LZ_ERR_INVALID_ARG, "%s: heads must be 0 or 1 (got %d)", fn, d->heads);
  if (!(d->eps > 0.f && d->eps < 3.0e38f))
    return layer_fail(LZ_ERR_INVALID_ARG, "%s: eps must be finite and > 0", fn);
  if (d->B > 65535 || (int64_t)d->B * d->T >= (int64_t(1) << 31))
    return layer_fail(LZ_ERR_UNSUPPORTED, "%s: B must be <= 65535 and B * T below 2^31", fn);
  if (!rows_ok(d->o) || !rows_ok(d->z) || !rows_ok(d->r))
    return layer_fail(LZ_ERR_INVALID_ARG, "%s: bad row strides", fn);
  return LZ_OK;
}

// heads: a vector must lie within a head
bool norm_vec(const lz_norm_dims* d, const NormParams& p) {
  const size_t es = esize(d->io);
  const int vw = (int)(16 / es);
  if (d->D % vw || (d->D / d->G) % vw) return false;
  return (d->heads || rows_vec(p.o, p.so, vw, es)) && rows_vec(p.z, p.sz, vw, es) && rows_vec(p.r, p.sr, vw, es);
}

}  // namespace

size_t norm_bwd_ws(const lz_norm_dims* d) {
  if (check_norm("lz_layer_workspace_bytes", d) != LZ_OK) return 0;
  return ws_round((size_t)bwd_part_rows((int64_t)d->B * d->T) * 3 * d->D * sizeof(float));
}

}  // namespace lz

using namespace lz;

extern "C" lz_status lz_block_norm_fwd(const lz_norm_dims* d, const void* o, const float* w, const void* z,
                                       const float* s, const void* r, const float* w2, void* out, void* n,
                                       lz_stream stream) {
  const char* fn = "lz_block_norm_fwd";
  lz_status st = check_norm(fn, d);
  if (st != LZ_OK) return st;
  if (d->B == 0 || d->T == 0 || d->D == 0) return layer_done(cudaSuccess, fn);
  const unsigned es = (unsigned)esize(d->io);
  st = check_ptrs(fn, {{o, "o", true, d->heads ? 16 : es}, {w, "w", false, 16}, {z, "z", false, es},
                       {s, "s", false, 16}, {r, "r", false, es}, {w2, "w2", false, 16}, {out, "out", true, 16},
                       {n, "n", w2 != nullptr, 16}});
  if (st == LZ_OK) st = check_distinct(fn, {out, w2 ? n : nullptr}, {o, z, r});
  if (st != LZ_OK) return st;
  NormParams p{};
  p.rows = (int64_t)d->B * d->T;
  p.B = d->B; p.T = d->T; p.D = d->D; p.dshift = shift_of(d->D / d->G); p.G = d->G; p.heads = d->heads; p.eps = d->eps;
  p.so = rows_of(d->o, d->T, d->D);
  p.sz = rows_of(d->z, d->T, d->D);
  p.sr = rows_of(d->r, d->T, d->D);
  p.o = o; p.w = w; p.z = z; p.s = s; p.r = r; p.w2 = w2; p.out = out; p.n = n;
  const Shape sh = shape_of(d, norm_vec(d, p), false);
  cudaError_t e = cudaSuccess;
#define LZ_CALL(IO, VW, WARP, MODE) go_fwd<IO, VW, WARP, MODE>(p, sh, (cudaStream_t)stream)
  LZ_NORM_DISPATCH(LZ_CALL);
#undef LZ_CALL
  return layer_done(e, fn);
}

extern "C" lz_status lz_block_norm_bwd(const lz_norm_dims* d, const void* o, const float* w, const void* z,
                                       const float* s, const float* w2, const void* out, const void* dout,
                                       const void* dn, void* dOo, void* dz, void* dr, float* dw, float* ds,
                                       float* dw2, void* ws, size_t ws_bytes, lz_stream stream) {
  const char* fn = "lz_block_norm_bwd";
  lz_status st = check_norm(fn, d);
  if (st != LZ_OK) return st;
  if (d->D == 0) return layer_done(cudaSuccess, fn);
  const int64_t rows = (int64_t)d->B * d->T;
  const bool data = rows > 0;
  const unsigned es = (unsigned)esize(d->io);
  if (data && !dout && !dn) return layer_fail(LZ_ERR_INVALID_ARG, "%s: dout and dn must not both be NULL", fn);
  st = check_ptrs(fn, {{o, "o", data, d->heads ? 16 : es}, {w, "w", dw != nullptr, 16}, {z, "z", dz != nullptr, es},
                       {s, "s", ds != nullptr, 16}, {w2, "w2", data && (dn || dw2), 16}, {out, "out", data && dn, 16},
                       {dout, "dout", false, 16}, {dn, "dn", data && dw2, 16}, {dOo, "dOo", data, 16},
                       {dz, "dz", false, 16}, {dr, "dr", false, 16}, {dw, "dw", false, 16}, {ds, "ds", false, 16},
                       {dw2, "dw2", false, 16}, {ws, "workspace", true, 256}});
  if (st == LZ_OK) st = check_distinct(fn, {dOo, dz, dr, dw, ds, dw2, ws}, {o, w, z, s, w2, out, dout, dn});
  if (st != LZ_OK) return st;
  const size_t need = norm_bwd_ws(d);
  if (ws_bytes < need)
    return layer_fail(LZ_ERR_INVALID_ARG, "%s: workspace too small (%zu bytes, need %zu)", fn, ws_bytes, need);
  NormParams p{};
  p.rows = rows;
  p.B = d->B; p.T = std::max(d->T, 1); p.D = d->D; p.dshift = shift_of(d->D / d->G); p.G = d->G; p.heads = d->heads; p.eps = d->eps;
  p.so = rows_of(d->o, d->T, d->D);
  p.sz = rows_of(d->z, d->T, d->D);
  p.o = o; p.w = w; p.z = z; p.s = s; p.w2 = w2; p.out = const_cast<void*>(out);
  p.dout = dout; p.dn = dn; p.d_o = dOo; p.dz = dz; p.dr = dr; p.part = (float*)ws;
  const Shape sh = shape_of(d, norm_vec(d, p), true);
  cudaError_t e = cudaSuccess;
  int blocks = 0;
#define LZ_CALL(IO, VW, WARP, MODE) go_bwd<IO, VW, WARP, MODE>(p, sh, &blocks, (cudaStream_t)stream)
  LZ_NORM_DISPATCH(LZ_CALL);
#undef LZ_CALL
  if (e == cudaSuccess && (dw || ds || dw2))
    e = launch_sum_rows({p.part, blocks, (size_t)3 * d->D, dw, (size_t)d->D, ds, (size_t)d->D, dw2, (size_t)d->D},
                        (cudaStream_t)stream);
  return layer_done(e, fn);
}
