// Selective state space scan, forward and single tokens.
//
// Per (token, channel, state): one exp (16 a cycle and SM) and some 10 more
// instructions with everything counted, against 8 bytes a (token, channel): its
// floor is the special-function unit's.  At 2 x 8192 tokens, 4096 channels, 16
// states (bf16, gated) 506 to 537 us: 54 to 57 % of the special-function rate, 62 %
// of the issue slots, neither of them full; its warps wait at the barrier after
// every tile as long as for an issue slot.  Its bytes would take 82 us.
#include "scan.cuh"

namespace lz {
namespace scan {
namespace {

// L: lanes of a channel, 4 states a lane; W: scan warps of a block; WE: its
// elementwise warps
template <int L, int W, int WE>
struct Geo {
  static constexpr int NS = 32 * W, NE = 32 * WE;  // scan threads, elementwise threads
  static constexpr int CH = NS / L;         // channels of a block
  static constexpr int NP = 4 * L;          // states, padded
  static constexpr int U = L < 4 ? L : 4;   // tokens whose lane sums are formed together
  static constexpr int YS = row_of(CH, L == 2 ? 16 : L == 4 ? 8 : 4);
};

// 4 elements of B or C as the scan warps read them from shared memory, as pairs
// of floats.  They stay in the I/O type there: what a warp's shared memory
// loads return to registers, 128 bytes a cycle and SM however many lanes read
// the same words, is what the scan runs out of first.
template <typename IO>
__device__ __forceinline__ void load_bc(const IO* p, f2& x, f2& y) {
  if constexpr (sizeof(IO) == 4) {
    const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(p);
    x = v.x;
    y = v.y;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    x = pk(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u));
    y = pk(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
  }
}

// Tile: 8 elements of (token, channel) for each elementwise thread, as long as
// that is at most 32 tokens.
template <int L, int W, int WE>
struct Tile {
  using G = Geo<L, W, WE>;
  static constexpr int TT = L >= 4 ? 32 : 8 * L;
  static constexpr int EV = TT * G::CH / G::NE;              // elements of a thread: neighbours in a row
  static constexpr int DS = G::CH + 2;                       // row of dd, off the banks of the row before
  static constexpr int BV = TT * L;                          // 4-element vectors of B, and of C
  static constexpr int BN = (BV + G::NE - 1) / G::NE;        // those of a thread
};

template <typename IO, int L, int W, int WE>
struct alignas(16) Smem {
  using X = Tile<L, W, WE>;
  using G = Geo<L, W, WE>;
  float2 dd[2][X::TT * X::DS];  // delta, delta * u
  IO bf[2][X::TT * G::NP], cf[2][X::TT * G::NP];
  float ys[2][X::TT * G::YS];
};

// The scan warps' walk over one tile, U tokens at a time.  The decays and
// inputs of the next U tokens are formed before the state passes through
// these, and the whole tile is one run of instructions, so that the loads and
// exponentials of the former fill the waits of the latter.
template <typename IO, int L, int W, int WE, bool END>
__device__ __forceinline__ void scan_tile(const float2* __restrict__ dd, const IO* __restrict__ bf,
                                          const IO* __restrict__ cf, float* __restrict__ ys, const f2 (&A2)[2],
                                          f2 (&h)[2], float& sumd, int lane, int l, float* states, size_t ck_step,
                                          int ck_left) {
  using G = Geo<L, W, WE>;
  constexpr int NP = G::NP, U = G::U, TT = Tile<L, W, WE>::TT, NG = TT / U;
  f2 a[2][U][2], x[2][U][2];
  auto form = [&](int i, f2 (&a)[2], f2 (&x)[2]) {
    const float2 d = dd[i * Tile<L, W, WE>::DS];
    f2 B0, B1;
    load_bc(bf + i * NP, B0, B1);
    const f2 d2 = pk(d.x, d.x), du2 = pk(d.y, d.y);
    a[0] = decay(A2[0], d2);
    a[1] = decay(A2[1], d2);
    x[0] = mul2(du2, B0);
    x[1] = mul2(du2, B1);
    if (END) sumd += d.x;
  };
  // C h of U tokens: summed over the lanes a step later
  float yv[2][U];
  auto sum_y = [&](int i, float (&v)[U]) {
    int j = 0;
    reduce_scatter<U, L / 2, 1>(v, lane, j);
    if (l % (L / U) == 0) ys[(i + j) * G::YS] = v[0];
  };
#pragma unroll
  for (int j = 0; j < U; ++j) form(j, a[0][j], x[0][j]);
#pragma unroll
  for (int q = 0; q < NG; ++q) {
    const int i = q * U;
    if (!END && i % kCk == 0 && i < ck_left)  // the state before every 16th token
      *reinterpret_cast<float4*>(states + i / kCk * ck_step) = make_float4(lo(h[0]), hi(h[0]), lo(h[1]), hi(h[1]));
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (q + 1 < NG) form(i + U + j, a[(q + 1) & 1][j], x[(q + 1) & 1][j]);
      h[0] = fma2(a[q & 1][j][0], h[0], x[q & 1][j][0]);
      h[1] = fma2(a[q & 1][j][1], h[1], x[q & 1][j][1]);
      if (!END) {
        f2 C0, C1;
        load_bc(cf + (i + j) * NP, C0, C1);
        const f2 y2 = fma2(h[1], C1, mul2(h[0], C0));
        yv[q & 1][j] = lo(y2) + hi(y2);
      }
    }
    if (!END && q > 0) sum_y(i - U, yv[(q + 1) & 1]);
  }
  if (!END) sum_y(TT - U, yv[(NG - 1) & 1]);
}

// One block: 32 W / L channels of one sequence over one segment of its tokens.
// END: only the segment's effect on the state (its end value from a zero
// start and the sum of delta), which the blocks of the later segments fold
// into the state they start from.
template <typename IO, int L, int W, int WE, bool END>
__global__ void __launch_bounds__(32 * (W + WE), W + WE > 8 ? 1 : 2) scan_fwd_kernel(ScanParams p) {
  using G = Geo<L, W, WE>;
  using X = Tile<L, W, WE>;
  constexpr int CH = G::CH, TT = X::TT, EV = X::EV, BN = X::BN, DS = X::DS;
  constexpr int NS = G::NS, NE = G::NE;
  extern __shared__ __align__(16) char raw[];
  using S = Smem<IO, L, W, WE>;
  S& sm = *reinterpret_cast<S*>(raw);
  const int tid = threadIdx.x;
  const int g = blockIdx.x / p.nct, ct = blockIdx.x % p.nct;
  const int b = blockIdx.y, seg = blockIdx.z;
  const int per = p.D / p.G;
  const int c0 = g * per + ct * CH, cmax = (g + 1) * per;  // channels of the block
  const int Tb = seq_len(p.lens, b, p.T);
  const int t0 = seg * p.seg, t1 = min(p.T, t0 + p.seg), te = min(t1, Tb);
  const int ntile = t0 < te ? (te - t0 + TT - 1) / TT : 0;

  if (tid >= NS) {
    // ---- elementwise warps
    const int et = tid - NS;
    const int i = et / (CH / EV), cl = et % (CH / EV) * EV, c = c0 + cl;  // token of the tile, channels
    const int nc = min(EV, cmax - c);                                      // how many of them exist
    struct Tok {
      Pack<IO, EV> u, z;
    };
    struct Next {
      Tok a;
      Pack<IO, EV> dt;
      Pack<IO, 4> b[BN], c[BN];
    };
    // this thread's elements of the next tile to load
    const IO* pu = (const IO*)p.u + p.ru.at(b, t0 + i) + c;
    const IO* pdt = (const IO*)p.dt + p.rdt.at(b, t0 + i) + c;
    const IO* pz = p.z ? (const IO*)p.z + p.rz.at(b, t0 + i) + c : nullptr;
    const IO *pb[BN], *pc[BN];
    int tb[BN], nb[BN];
#pragma unroll
    for (int j = 0; j < BN; ++j) {
      const int v = et + j * NE, n0 = v % L * 4;
      tb[j] = t0 + v / L;
      nb[j] = v < X::BV ? p.N - n0 : 0;
      pb[j] = (const IO*)p.Bm + p.rb.at(b, tb[j]) + g * p.N + n0;
      pc[j] = (const IO*)p.Cm + p.rc.at(b, tb[j]) + g * p.N + n0;
    }
    float bias[EV], Ds[EV];
#pragma unroll
    for (int e = 0; e < EV; ++e) {
      bias[e] = p.dtb && e < nc ? p.dtb[c + e] : 0.f;
      Ds[e] = !END && p.Dskip && e < nc ? p.Dskip[c + e] : 0.f;
    }
    auto load = [&](int k, Next& x) {
      const int n = t0 + k * TT + i < te ? nc : 0;
      x.dt.load(pdt, n, p.vec);
      x.a.u.load(pu, n, p.vec);
      if (!END && p.z) x.a.z.load(pz, n, p.vec);
      pdt += TT * p.rdt.ld;
      pu += TT * p.ru.ld;
      pz += TT * p.rz.ld;
#pragma unroll
      for (int j = 0; j < BN; ++j) {
        const int m = tb[j] < te ? nb[j] : 0;
        x.b[j].load(pb[j], m, p.vecbc);
        if (!END) x.c[j].load(pc[j], m, p.vecbc);
        tb[j] += TT;
        pb[j] += TT * p.rb.ld;
        pc[j] += TT * p.rc.ld;
      }
    };
    auto prepare = [&](int k, const Next& x) {
      const bool live = t0 + k * TT + i < te;
      float2* dd = &sm.dd[k & 1][i * DS + cl];
      float dl[EV];
#pragma unroll
      for (int e = 0; e < EV; ++e) dl[e] = x.dt.get(e) + bias[e];
      if (p.softplus) {
#pragma unroll
        for (int e = 0; e < EV; ++e) dl[e] = softplus(dl[e]);
      }
      // (a channel that is not there has u = 0 and takes nothing up; what its
      // state decays by does not matter)
#pragma unroll
      for (int e = 0; e < EV; ++e) dl[e] = live ? dl[e] : 0.f;
#pragma unroll
      for (int e = 0; e < EV; e += 2)
        *reinterpret_cast<float4*>(dd + e) =
            make_float4(dl[e], dl[e] * x.a.u.get(e), dl[e + 1], dl[e + 1] * x.a.u.get(e + 1));
#pragma unroll
      for (int j = 0; j < BN; ++j) {
        const int v = et + j * NE;
        if (v < X::BV) {
          x.b[j].put(&sm.bf[k & 1][v * 4]);
          if (!END) x.c[j].put(&sm.cf[k & 1][v * 4]);
        }
      }
    };
    auto finish = [&](int k, const Tok& x) {
      const int t = t0 + k * TT + i;
      if (!p.y || t >= te) return;
      float o[EV];
      load_f<EV>(&sm.ys[k & 1][i * G::YS + cl], o);
#pragma unroll
      for (int e = 0; e < EV; ++e) o[e] = fmaf(Ds[e], x.u.get(e), o[e]);
      if (p.z) {
#pragma unroll
        for (int e = 0; e < EV; ++e) {
          const float z = x.z.get(e);
          o[e] *= z * sigmoid(z);
        }
      }
      store_n<IO, EV>((IO*)p.y + ((size_t)b * p.T + t) * p.D + c, o, nc, p.vec);
    };
    // registers: the tokens of the last tile (outputs due), of this one, and
    // the loads of the next
    Next nx;
    Tok last, cur;
    if (ntile > 0) {
      load(0, nx);
      prepare(0, nx);
      cur = nx.a;
      if (ntile > 1) load(1, nx);
    }
    __syncthreads();
    for (int k = 0; k < ntile; ++k) {
      if (k + 1 < ntile) prepare(k + 1, nx);
      const Tok next = nx.a;
      if (k + 2 < ntile) load(k + 2, nx);
      if constexpr (!END)
        if (k > 0) finish(k - 1, last);
      last = cur;
      cur = next;
      __syncthreads();
    }
    if constexpr (!END)
      if (ntile > 0) finish(ntile - 1, last);
    if (!END && p.y) {
      // behind the sequence's end: zeros
      const float zero[EV] = {};
      for (int t = max(t0, te) + i; t < t1; t += TT)
        store_n<IO, EV>((IO*)p.y + ((size_t)b * p.T + t) * p.D + c, zero, nc, p.vec);
    }
    return;
  }

  // ---- scan warps
  const int lane = tid % 32;
  const int cl = tid / L, l = tid % L, c = c0 + cl;  // this thread's channel and lane
  const int n0 = 4 * l;
  const bool on = c < cmax && n0 < p.N;
  const size_t sidx = ((size_t)b * p.D + c) * p.N + n0;  // [B][D][N]
  const size_t sstep = (size_t)p.B * p.D * p.N;
  f2 A2[2] = {0, 0}, h[2] = {0, 0};
  if (on) {
    const float4 a = *reinterpret_cast<const float4*>(p.A + (size_t)c * p.N + n0);
    A2[0] = pk(a.x * kLog2e, a.y * kLog2e);
    A2[1] = pk(a.z * kLog2e, a.w * kLog2e);
    if (!END) {
      if (p.h0) {
        const float4 x = *reinterpret_cast<const float4*>(p.h0 + sidx);
        h[0] = pk(x.x, x.y);
        h[1] = pk(x.z, x.w);
      }
#pragma unroll 4
      for (int s = 0; s < seg; ++s) {
        const float4 x = *reinterpret_cast<const float4*>(p.segE + s * sstep + sidx);
        const float d = p.segD[((size_t)s * p.B + b) * p.D + c];
        h[0] = carry(A2[0], pk(d, d), h[0], pk(x.x, x.y));
        h[1] = carry(A2[1], pk(d, d), h[1], pk(x.z, x.w));
      }
    }
  }
  float sumd = 0.f;
  __syncthreads();
  for (int k = 0; k < ntile; ++k) {
    const float2* dd = sm.dd[k & 1] + cl;
    const IO* bf = sm.bf[k & 1] + n0;
    const IO* cf = sm.cf[k & 1] + n0;
    float* ys = sm.ys[k & 1] + cl;
    // (a tile of 8 tokens starts at a 16th one every other time)
    const int t = t0 + k * TT;
    const bool ck = p.states && on && t % kCk == 0;
    scan_tile<IO, L, W, WE, END>(dd, bf, cf, ys, A2, h, sumd, lane, l,
                          p.states + (((size_t)b * ((p.T + kCk - 1) / kCk) + t / kCk) * p.D + c) * p.N + n0,
                          (size_t)p.D * p.N, ck ? te - t : 0);
    __syncthreads();
  }
  const float4 hv = make_float4(lo(h[0]), hi(h[0]), lo(h[1]), hi(h[1]));
  if (END) {
    if (on) *reinterpret_cast<float4*>(p.segE + seg * sstep + sidx) = hv;
    if (c < cmax && l == 0) p.segD[((size_t)seg * p.B + b) * p.D + c] = sumd;
  } else if (p.hT && on && seg == p.nseg - 1) {
    // (a segment behind the sequence's end passes the state on)
    *reinterpret_cast<float4*>(p.hT + sidx) = hv;
  }
}

template <typename IO, int L, int W, int WE = W>
cudaError_t go(const ScanParams& p, cudaStream_t s) {
  const size_t smem = sizeof(Smem<IO, L, W, WE>);
  if constexpr (W == 4 && WE == 4) {  // (segments only come with such blocks)
    if (p.nseg > 1) {
      cudaError_t e = want_smem(scan_fwd_kernel<IO, L, W, WE, true>, smem);
      if (e != cudaSuccess) return e;
      ScopedTiming tm("scan_fwd_ends", s);
      scan_fwd_kernel<IO, L, W, WE, true><<<dim3(p.G * p.nct, p.B, p.nseg - 1), 32 * (W + WE), smem, s>>>(p);
      e = cudaGetLastError();
      if (e != cudaSuccess) return e;
    }
  }
  const cudaError_t e = want_smem(scan_fwd_kernel<IO, L, W, WE, false>, smem);
  if (e != cudaSuccess) return e;
  ScopedTiming tm("scan_fwd", s);
  scan_fwd_kernel<IO, L, W, WE, false><<<dim3(p.G * p.nct, p.B, p.nseg), 32 * (W + WE), smem, s>>>(p);
  return cudaGetLastError();
}

template <typename IO>
cudaError_t go_any(const ScanParams& p, cudaStream_t s) {
  // blocks with an SM to themselves take twice the elementwise warps: with one
  // scan warp to a scheduler, these are what a tile waits for (1 x 2048 tokens,
  // 4096 channels, 16 states: 97 -> 86 us)
  const bool alone = p.nseg == 1 && (int64_t)p.nct * p.G * p.B <= 148;
  switch (states_of(p.N)) {
    case 4: return alone ? go<IO, 1, 4, 8>(p, s) : go<IO, 1, 4>(p, s);
    case 8: return alone ? go<IO, 2, 4, 8>(p, s) : go<IO, 2, 4>(p, s);
    case 16: return p.W == 7 ? go<IO, 4, 7>(p, s) : alone ? go<IO, 4, 4, 8>(p, s) : go<IO, 4, 4>(p, s);
    case 32: return p.W == 7 ? go<IO, 8, 7>(p, s) : alone ? go<IO, 8, 4, 8>(p, s) : go<IO, 8, 4>(p, s);
    case 64: return p.W == 7 ? go<IO, 16, 7>(p, s) : go<IO, 16, 4>(p, s);
  }
  return cudaErrorInvalidValue;
}

// ---- single tokens --------------------------------------------------------
// The state is read and written once: bound by HBM (or L2, when it fits).
// A thread holds R = 8 states (4 where N is no multiple of 8) of one channel, so
// that what is done once a channel (softplus, the gate, addresses) weighs less;
// its rates stay in registers while it walks sequences, the next one's loads in
// flight.  The L lanes of a channel add their shares of y.
constexpr int kStepThreads = 256;

template <typename IO, int L, int R>
__global__ void __launch_bounds__(kStepThreads, 3) scan_step_kernel(ScanParams p, float* state) {
  constexpr int Q = R / 4;
  const unsigned idx = blockIdx.x * kStepThreads + threadIdx.x;
  const int l = threadIdx.x % L, c = (int)(idx / L), n0 = R * l;
  const bool row = c < p.D, on = row && n0 < p.N;
  const int g = p.G > 1 && row ? c / (p.D / p.G) : 0;
  struct In {
    float4 h[Q];
    Pack<IO, 4> B[Q], C[Q];
    IO u, d, z;
  };
  auto fetch = [&](int b, In& x) {
    const float4* hp = reinterpret_cast<const float4*>(state + ((size_t)b * p.D + c) * p.N + n0);
    const IO* pb = (const IO*)p.Bm + p.rb.at(b, 0) + (size_t)g * p.N + n0;
    const IO* pc = (const IO*)p.Cm + p.rc.at(b, 0) + (size_t)g * p.N + n0;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      if (on) x.h[q] = hp[q];
      else x.h[q] = make_float4(0.f, 0.f, 0.f, 0.f);
      x.B[q].load(pb + 4 * q, on ? 4 : 0, p.vecbc);
      x.C[q].load(pc + 4 * q, on ? 4 : 0, p.vecbc);
    }
    if (on) {
      x.u = ((const IO*)p.u)[p.ru.at(b, 0) + c];
      x.d = ((const IO*)p.dt)[p.rdt.at(b, 0) + c];
      if (p.z) x.z = ((const IO*)p.z)[p.rz.at(b, 0) + c];
    } else {
      x.u = x.d = x.z = from_f<IO>(0.f);
    }
  };
  float4 A[Q];
  float bias = 0.f, Ds = 0.f;
  In nx;
  if ((int)blockIdx.y < p.B) fetch(blockIdx.y, nx);
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    A[q] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (on) A[q] = __ldg(reinterpret_cast<const float4*>(p.A + (size_t)c * p.N + n0) + q);
  }
  if (row && p.dtb) bias = p.dtb[c];
  if (row && p.Dskip) Ds = p.Dskip[c];
  for (int b = blockIdx.y; b < p.B; b += gridDim.y) {
    const In in = nx;
    if (b + (int)gridDim.y < p.B) fetch(b + gridDim.y, nx);
    const float u = to_f(in.u);
    float dl = to_f(in.d) + bias;
    if (p.softplus) dl = softplus(dl);
    const float du = dl * u, d2 = dl * kLog2e;
    float y = 0.f;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      float4 x = in.h[q];
      const Pack<IO, 4>&Bq = in.B[q], &Cq = in.C[q];
      x.x = fmaf(ex2(fmaf(d2, A[q].x, kCut)), x.x, du * Bq.get(0));
      x.y = fmaf(ex2(fmaf(d2, A[q].y, kCut)), x.y, du * Bq.get(1));
      x.z = fmaf(ex2(fmaf(d2, A[q].z, kCut)), x.z, du * Bq.get(2));
      x.w = fmaf(ex2(fmaf(d2, A[q].w, kCut)), x.w, du * Bq.get(3));
      if (on) reinterpret_cast<float4*>(state + ((size_t)b * p.D + c) * p.N + n0)[q] = x;
      y += x.x * Cq.get(0) + x.y * Cq.get(1) + x.z * Cq.get(2) + x.w * Cq.get(3);
    }
#pragma unroll
    for (int m = L / 2; m > 0; m >>= 1) y += __shfl_xor_sync(0xffffffffu, y, m);
    if (row && l == 0) {
      y = fmaf(Ds, u, y);
      if (p.z) {
        const float z = to_f(in.z);
        y *= z * sigmoid(z);
      }
      ((IO*)p.y)[(size_t)b * p.D + c] = from_f<IO>(y);
    }
  }
}

template <typename IO, int L, int R>
cudaError_t go_step(const ScanParams& p, float* state, cudaStream_t s) {
  const int gx = (int)(((size_t)p.D * L + kStepThreads - 1) / kStepThreads);
  // three blocks an SM, each with its share of the sequences
  const int gy = std::max(1, std::min(p.B, 148 * 3 / gx));
  ScopedTiming tm("scan_step", s);
  scan_step_kernel<IO, L, R><<<dim3(gx, gy), kStepThreads, 0, s>>>(p, state);
  return cudaGetLastError();
}

}  // namespace
}  // namespace scan

cudaError_t launch_scan_fwd(const scan::ScanParams& p, bool bf, cudaStream_t s) {
  return bf ? scan::go_any<bf16>(p, s) : scan::go_any<float>(p, s);
}

template <typename IO>
static cudaError_t launch_scan_step(const scan::ScanParams& p, float* state, cudaStream_t s) {
  if (p.N % 8 == 0) {
    switch (scan::states_of(p.N)) {
      case 8: return scan::go_step<IO, 1, 8>(p, state, s);
      case 16: return scan::go_step<IO, 2, 8>(p, state, s);
      case 32: return scan::go_step<IO, 4, 8>(p, state, s);
      case 64: return scan::go_step<IO, 8, 8>(p, state, s);
    }
  }
  switch (scan::states_of(p.N)) {
    case 4: return scan::go_step<IO, 1, 4>(p, state, s);
    case 16: return scan::go_step<IO, 4, 4>(p, state, s);
    case 32: return scan::go_step<IO, 8, 4>(p, state, s);
    case 64: return scan::go_step<IO, 16, 4>(p, state, s);
  }
  return cudaErrorInvalidValue;
}

// ---- host -----------------------------------------------------------------

namespace {

using scan::ScanParams;

lz_status check_scan(const char* fn, const lz_scan_dims* d) {
  if (!d) return layer_fail(LZ_ERR_INVALID_ARG, "%s: dims must not be NULL", fn);
  if (d->B < 0 || d->T < 0 || d->D < 0)
    return layer_fail(LZ_ERR_INVALID_ARG, "%s: B, T, D must be >= 0 (got %d, %d, %d)", fn, d->B, d->T, d->D);
  if (!io_ok(d->io))
    return layer_fail(LZ_ERR_UNSUPPORTED, "%s: io dtype %d is not LZ_F32 or LZ_BF16", fn, (int)d->io);
  if (d->N < 4 || d->N > 64 || d->N % 4)
    return layer_fail(LZ_ERR_UNSUPPORTED, "%s: N must be a multiple of 4 in [4, 64] (got %d)", fn, d->N);
  if (d->G < 1 || d->D % d->G)
    return layer_fail(LZ_ERR_INVALID_ARG, "%s: G must be a divisor of D (got %d of %d)", fn, d->G, d->D);
  if (d->softplus != 0 && d->softplus != 1)
    return layer_fail(LZ_ERR_INVALID_ARG, "%s: softplus must be 0 or 1 (got %d)", fn, d->softplus);
  if (!rows_ok(d->u) || !rows_ok(d->dt) || !rows_ok(d->z) || !rows_ok(d->b) || !rows_ok(d->c))
    return layer_fail(LZ_ERR_INVALID_ARG, "%s: bad row strides", fn);
  // keeps grid dimensions and 32-bit token indices in range
  if (d->B > 65535 || d->T > (1 << 23) || d->D > (1 << 24))
    return layer_fail(LZ_ERR_UNSUPPORTED, "%s: problem too large (B %d, T %d, D %d)", fn, d->B, d->T, d->D);
  return LZ_OK;
}

// Scan warps of a block, channel tiles, and the segments that a sequence is cut
// into when there are too few channels and sequences to fill the device.
//
// Segments: a segmented call runs the recurrence twice (ends, then outputs), so
// it pays from three segments on.  Warps: a block of 7 + 7 warps has an SM to
// itself, blocks of 4 + 4 share one by twos; the kind is taken that leaves the
// fewest scan warps on the busiest of kSMs SMs.  (At 2 sequences of 4096
// channels with 16 states: 148 blocks of 7 against 256 of 4, two of which
// meet on most SMs: 7 warps against 8; the backward takes 1585 us against 1647 us with the sums over its
// channel tiles.)
constexpr int kSMs = 148;
void plan(const lz_scan_dims* d, int* W, int* nct, int* seg, int* nseg) {
  const int N = scan::states_of(d->N), per = d->D / d->G;
  const int64_t gb = (int64_t)d->G * d->B;
  auto tiles = [&](int w) { return (per + 128 * w / N - 1) / (128 * w / N); };
  auto busiest = [&](int w) { return (tiles(w) * gb + kSMs - 1) / kSMs * w; };
  const int64_t base = tiles(4) * gb;
  int n = 1;
  if (base > 0 && base * 3 <= kSMs * 2) n = (int)std::min<int64_t>(32, kSMs * 2 / base);
  *W = N >= 16 && n == 1 && busiest(7) < busiest(4) ? 7 : 4;
  *nct = tiles(*W);
  int len = ((d->T + n - 1) / n + 31) / 32 * 32;
  len = std::max(len, 64);
  // a sequence that is not cut is one segment, however short
  *seg = n > 1 ? len : std::max(1, (d->T + 31) / 32 * 32);
  *nseg = std::max(1, (d->T + *seg - 1) / *seg);
}

size_t state_bytes(const lz_scan_dims* d) {
  return (size_t)d->B * ((d->T + scan::kCk - 1) / scan::kCk) * d->D * d->N * sizeof(float);
}

struct Ws {
  size_t segE, segD, part, bc, states, total;
};
enum { WS_FWD, WS_BWD, WS_BWD_SAVED };  // (saved: the caller has the forward's states)
Ws ws_of(const lz_scan_dims* d, int kind) {
  int W, nct, seg, nseg;
  plan(d, &W, &nct, &seg, &nseg);
  const size_t bd = (size_t)d->B * d->D;
  Ws w{};
  size_t o = 0;
  auto take = [&](size_t bytes) { const size_t at = o; o += ws_round(bytes); return at; };
  w.segE = take(nseg > 1 ? nseg * bd * d->N * sizeof(float) : 0);
  w.segD = take(nseg > 1 ? nseg * bd * sizeof(float) : 0);
  if (kind != WS_FWD) {
    w.part = take((size_t)d->B * nseg * scan::part_ld(d->D, d->N) * sizeof(float));
    w.bc = take((size_t)nct * d->B * d->T * d->G * 2 * d->N * sizeof(float));
    w.states = take(kind == WS_BWD ? state_bytes(d) : 0);  // used when the caller gives none
  }
  w.total = o;
  return w;
}

ScanParams params_of(const lz_scan_dims* d, const void* u, const void* dt, const float* A, const void* Bm,
                     const void* Cm, const float* Dskip, const void* z, const float* dtb) {
  ScanParams p{};
  p.B = d->B; p.T = d->T; p.D = d->D; p.G = d->G; p.N = d->N; p.softplus = d->softplus;
  plan(d, &p.W, &p.nct, &p.seg, &p.nseg);
  const int bcw = d->G * d->N;
  p.ru = rows_of(d->u, d->T, d->D);
  p.rdt = rows_of(d->dt, d->T, d->D);
  p.rz = rows_of(d->z, d->T, d->D);
  p.rb = rows_of(d->b, d->T, bcw);
  p.rc = rows_of(d->c, d->T, bcw);
  p.u = u; p.dt = dt; p.A = A; p.Bm = Bm; p.Cm = Cm; p.Dskip = Dskip; p.z = z; p.dtb = dtb;
  const size_t es = esize(d->io);
  const int vw = (int)(16 / es);
  // the widest run of channels that a thread takes at once is 8: whole runs only
  p.vec = (d->D / d->G) % 8 == 0 && rows_vec(u, p.ru, vw, es) && rows_vec(dt, p.rdt, vw, es) &&
          rows_vec(z, p.rz, vw, es);
  p.vecbc = rows_vec(Bm, p.rb, 4, es) && rows_vec(Cm, p.rc, 4, es);
  return p;
}

}  // namespace

size_t scan_ws(const lz_scan_dims* d, int which) {
  if (check_scan("lz_layer_workspace_bytes", d) != LZ_OK) return 0;
  if (which == LZ_WS_SCAN_STATES) return state_bytes(d);
  return ws_of(d, which == LZ_WS_SCAN_FWD ? WS_FWD : which == LZ_WS_SCAN_BWD ? WS_BWD : WS_BWD_SAVED).total;
}

}  // namespace lz

using namespace lz;

extern "C" lz_status lz_scan_fwd(const lz_scan_dims* d, const void* u, const void* dt, const float* A,
                                 const void* Bm, const void* Cm, const float* Dskip, const void* z,
                                 const float* dt_bias, const float* h0, const int64_t* lens, void* y, float* hT,
                                 float* states, void* ws, size_t ws_bytes, lz_stream stream) {
  const char* fn = "lz_scan_fwd";
  lz_status st = check_scan(fn, d);
  if (st != LZ_OK) return st;
  if (d->B == 0 || d->D == 0 || (d->T == 0 && !hT)) return layer_done(cudaSuccess, fn);
  const unsigned es = (unsigned)esize(d->io);
  const bool data = d->T > 0;
  const Ws w = ws_of(d, WS_FWD);
  st = check_ptrs(fn, {{u, "u", data, es}, {dt, "dt", data, es}, {A, "A", true, 16}, {Bm, "Bm", data, es},
                       {Cm, "Cm", data, es}, {Dskip, "Dskip", false, 16}, {z, "z", false, es},
                       {dt_bias, "dt_bias", false, 16}, {h0, "h0", false, 16}, {lens, "lens", false, 8},
                       {y, "y", false, 16}, {hT, "hT", false, 16}, {states, "states", false, 16},
                       {ws, "workspace", w.total > 0, 256}});
  if (st == LZ_OK) st = check_distinct(fn, {y, hT, states, w.total ? ws : nullptr}, {u, dt, A, Bm, Cm, z, h0});
  if (st != LZ_OK) return st;
  if (ws_bytes < w.total)
    return layer_fail(LZ_ERR_INVALID_ARG, "%s: workspace too small (%zu bytes, need %zu)", fn, ws_bytes, w.total);
  ScanParams p = params_of(d, u, dt, A, Bm, Cm, Dskip, z, dt_bias);
  p.h0 = h0; p.lens = lens; p.y = y; p.hT = hT; p.states = states;
  p.segE = (float*)((char*)ws + w.segE);
  p.segD = (float*)((char*)ws + w.segD);
  return layer_done(launch_scan_fwd(p, d->io == LZ_BF16, (cudaStream_t)stream), fn);
}

static lz_status scan_bwd(const char* fn, int kind, const lz_scan_dims* d, const void* u, const void* dt,
                          const float* A, const void* Bm, const void* Cm, const float* Dskip, const void* z,
                          const float* dt_bias, const float* h0, const int64_t* lens, const void* dy,
                          const float* dhT, const float* states, void* du, void* ddt, float* dA, void* dB, void* dC,
                          float* dDskip, float* ddt_bias, void* dz, float* dh0, void* ws, size_t ws_bytes,
                          lz_stream stream) {
  lz_status st = check_scan(fn, d);
  if (st != LZ_OK) return st;
  if (d->D == 0) return layer_done(cudaSuccess, fn);
  const unsigned es = (unsigned)esize(d->io);
  const bool data = d->T > 0 && d->B > 0;
  const Ws w = ws_of(d, kind);
  st = check_ptrs(fn, {{u, "u", data, es}, {dt, "dt", data, es}, {A, "A", true, 16}, {Bm, "Bm", data, es},
                       {Cm, "Cm", data, es}, {Dskip, "Dskip", false, 16}, {z, "z", data && dz, es},
                       {dt_bias, "dt_bias", false, 16}, {h0, "h0", false, 16}, {lens, "lens", false, 8},
                       {dy, "dy", data, 16}, {dhT, "dhT", false, 16},
                       {states, "states", data && kind == WS_BWD_SAVED, 16},
                       {du, "du", data, 16}, {ddt, "ddt", data, 16}, {dA, "dA", true, 16}, {dB, "dB", data, 16},
                       {dC, "dC", data, 16}, {dDskip, "dDskip", false, 16}, {ddt_bias, "ddt_bias", false, 16},
                       {dz, "dz", false, 16}, {dh0, "dh0", false, 16}, {ws, "workspace", w.total > 0, 256}});
  if (st == LZ_OK)
    st = check_distinct(fn, {du, ddt, dA, dB, dC, dDskip, ddt_bias, dz, dh0, ws},
                        {u, dt, A, Bm, Cm, Dskip, z, dt_bias, h0, dy, dhT, states});
  if (st != LZ_OK) return st;
  if (ws_bytes < w.total)
    return layer_fail(LZ_ERR_INVALID_ARG, "%s: workspace too small (%zu bytes, need %zu)", fn, ws_bytes, w.total);
  ScanParams p = params_of(d, u, dt, A, Bm, Cm, Dskip, z, dt_bias);
  const bool bf = d->io == LZ_BF16;
  cudaStream_t s = (cudaStream_t)stream;
  p.h0 = h0; p.lens = lens;
  p.segE = (float*)((char*)ws + w.segE);
  p.segD = (float*)((char*)ws + w.segD);
  cudaError_t e = cudaSuccess;
  p.states = const_cast<float*>(states);
  if (!states && data) {
    p.states = (float*)((char*)ws + w.states);
    e = launch_scan_fwd(p, bf, s);
  }
  p.dy = dy; p.dhT = dhT; p.du = du; p.ddt = ddt; p.dz = dz; p.dh0 = dh0; p.dB = dB; p.dC = dC;
  p.part = (float*)((char*)ws + w.part);
  p.bc = (float*)((char*)ws + w.bc);
  if (e == cudaSuccess && d->B > 0) e = launch_scan_bwd(p, bf, s);
  if (e == cudaSuccess)
    e = launch_sum_rows({p.part, d->B * p.nseg, scan::part_ld(d->D, d->N), dA, (size_t)d->D * d->N, dDskip,
                         (size_t)d->D, ddt_bias, (size_t)d->D},
                        s);
  return layer_done(e, fn);
}

extern "C" lz_status lz_scan_bwd(const lz_scan_dims* d, const void* u, const void* dt, const float* A,
                                 const void* Bm, const void* Cm, const float* Dskip, const void* z,
                                 const float* dt_bias, const float* h0, const int64_t* lens, const void* dy,
                                 const float* dhT, const float* states, void* du, void* ddt, float* dA, void* dB,
                                 void* dC, float* dDskip, float* ddt_bias, void* dz, float* dh0, void* ws,
                                 size_t ws_bytes, lz_stream stream) {
  return scan_bwd("lz_scan_bwd", WS_BWD, d, u, dt, A, Bm, Cm, Dskip, z, dt_bias, h0, lens, dy, dhT, states, du, ddt,
                  dA, dB, dC, dDskip, ddt_bias, dz, dh0, ws, ws_bytes, stream);
}

extern "C" lz_status lz_scan_bwd_saved(const lz_scan_dims* d, const void* u, const void* dt, const float* A,
                                       const void* Bm, const void* Cm, const float* Dskip, const void* z,
                                       const float* dt_bias, const float* h0, const int64_t* lens, const void* dy,
                                       const float* dhT, const float* states, void* du, void* ddt, float* dA,
                                       void* dB, void* dC, float* dDskip, float* ddt_bias, void* dz, float* dh0,
                                       void* ws, size_t ws_bytes, lz_stream stream) {
  return scan_bwd("lz_scan_bwd_saved", WS_BWD_SAVED, d, u, dt, A, Bm, Cm, Dskip, z, dt_bias, h0, lens, dy, dhT,
                  states, du, ddt, dA, dB, dC, dDskip, ddt_bias, dz, dh0, ws, ws_bytes, stream);
}

extern "C" lz_status lz_scan_step(const lz_scan_dims* d, float* state, const void* u, const void* dt,
                                  const float* A, const void* Bm, const void* Cm, const float* Dskip,
                                  const void* z, const float* dt_bias, void* y, lz_stream stream) {
  const char* fn = "lz_scan_step";
  lz_status st = check_scan(fn, d);
  if (st != LZ_OK) return st;
  if (d->B == 0 || d->D == 0) return layer_done(cudaSuccess, fn);
  const unsigned es = (unsigned)esize(d->io);
  st = check_ptrs(fn, {{state, "state", true, 16}, {u, "u", true, es}, {dt, "dt", true, es}, {A, "A", true, 16},
                       {Bm, "Bm", true, es}, {Cm, "Cm", true, es}, {Dskip, "Dskip", false, 16}, {z, "z", false, es},
                       {dt_bias, "dt_bias", false, 16}, {y, "y", true, 16}});
  if (st == LZ_OK) st = check_distinct(fn, {state, y}, {u, dt, A, Bm, Cm, Dskip, z, dt_bias});
  if (st != LZ_OK) return st;
  lz_scan_dims one = *d;
  one.T = 1;
  ScanParams p = params_of(&one, u, dt, A, Bm, Cm, Dskip, z, dt_bias);
  p.y = y;
  cudaStream_t s = (cudaStream_t)stream;
  return layer_done(d->io == LZ_BF16 ? launch_scan_step<bf16>(p, state, s) : launch_scan_step<float>(p, state, s), fn);
}
