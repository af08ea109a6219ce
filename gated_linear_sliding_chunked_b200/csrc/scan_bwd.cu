// Selective state space scan, backward.
//
// With a = exp(delta A), p_t = a_t h_{t-1}, e = dy silu(z) and g_t the gradient
// of the state after token t:
//   g_t = C_t e_t + a_{t+1} g_{t+1}
//   du = delta sum_n g B + Dskip e      ddelta = u sum_n g B + sum_n A g p
//   dB_t = sum_channels g delta u       dC_t = sum_channels h e
//   dA = sum_t delta g p                dz = dy (sum_n C h + Dskip u) silu'(z)
//
// The states are not kept for every token: the forward saves the one before
// every 16th, and a tile of 16 tokens is run forward again, leaving a and p of
// its tokens in registers, before it is walked back.  So each exp is taken
// once.  dB and dC are sums over all channels: first over a warp's channels
// by halving exchanges, then over the block's warps in shared memory, then
// over the channel tiles in a second kernel, in a fixed order.
#include "scan.cuh"

namespace lz {
namespace scan {
namespace {

constexpr int TB = kCk;  // tokens of a tile
constexpr int kWarps = NT / 32;

template <typename IO, int L>
struct alignas(16) Smem {
  static constexpr int CH = Geo<L>::CH, NP = Geo<L>::NP;
  IO u[2][TB * CH], dt[2][TB * CH], z[2][TB * CH], dy[2][TB * CH];
  IO b[2][TB * NP], c[2][TB * NP];
  float4 q[TB * CH];  // delta, delta u, e, u
  float bf[TB * NP], cf[TB * NP];
  float gB[TB * Geo<L>::YS], gA[TB * Geo<L>::YS], yc[TB * Geo<L>::YS];
  float red[kWarps][TB][2 * NP];  // dB, dC over a warp's channels
};

// END: only the gradient that the segment hands to the one before it when
// none comes from behind (the state gradient before its first token).
template <typename IO, int L, bool END>
__global__ void __launch_bounds__(NT, 2) scan_bwd_kernel(ScanParams p) {
  using G = Geo<L>;
  using S = Smem<IO, L>;
  constexpr int CH = G::CH, NP = G::NP, U = G::U, YS = G::YS;
  constexpr int VW = 16 / (int)sizeof(IO);
  extern __shared__ __align__(16) char raw[];
  S& sm = *reinterpret_cast<S*>(raw);
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int g = blockIdx.x / p.nct, ct = blockIdx.x % p.nct;
  const int b = blockIdx.y, seg = END ? blockIdx.z + 1 : blockIdx.z;
  const int per = p.D / p.G;
  const int c0 = g * per + ct * CH, cmax = (g + 1) * per;
  const int cl = tid / L, l = tid % L, c = c0 + cl;
  const int n0 = 4 * l;
  const bool on = c < cmax && n0 < p.N;
  const int Tb = seq_len(p.lens, b, p.T);
  const int t0 = seg * p.seg, t1 = min(p.T, t0 + p.seg), te = min(t1, Tb);
  const int nck = (p.T + kCk - 1) / kCk;
  const size_t sidx = ((size_t)b * p.D + c) * p.N + n0;
  const size_t sstep = (size_t)p.B * p.D * p.N;

  f2 A2[2] = {0, 0}, gr[2] = {0, 0}, dA[2] = {0, 0};
  if (on) {
    const float4 a = *reinterpret_cast<const float4*>(p.A + (size_t)c * p.N + n0);
    A2[0] = pk(a.x * kLog2e, a.y * kLog2e);
    A2[1] = pk(a.z * kLog2e, a.w * kLog2e);
    if (!END) {
      if (p.dhT) {
        const float4 x = *reinterpret_cast<const float4*>(p.dhT + sidx);
        gr[0] = pk(x.x, x.y);
        gr[1] = pk(x.z, x.w);
      }
      for (int s = p.nseg - 1; s > seg; --s) {
        const float4 x = *reinterpret_cast<const float4*>(p.segE + s * sstep + sidx);
        const float d = p.segD[((size_t)s * p.B + b) * p.D + c];
        gr[0] = fma2(ex2v(mul2(A2[0], pk(d, d))), gr[0], pk(x.x, x.y));
        gr[1] = fma2(ex2v(mul2(A2[1], pk(d, d))), gr[1], pk(x.z, x.w));
      }
    }
  }
  float sumd = 0.f;
  // elementwise work: 4 neighbouring channels and every (NT / (CH/4))-th token
  constexpr int QV = CH / 4, QT = NT / QV;
  const int qc = tid % QV * 4, qt = tid / QV;
  float sD[4] = {0, 0, 0, 0}, sT[4] = {0, 0, 0, 0};  // sums of e u and of ddt

  auto load = [&](int t, int st) {
    stage<IO, TB, CH, VW>(sm.dt[st], p.dt, p.rdt, b, t, te, c0, cmax, p.vec);
    stage<IO, TB, CH, VW>(sm.dy[st], p.dy, Rows{p.D, (int64_t)p.T * p.D}, b, t, te, c0, cmax, p.vec);
    if (p.z) stage<IO, TB, CH, VW>(sm.z[st], p.z, p.rz, b, t, te, c0, cmax, p.vec);
    stage<IO, TB, NP, 4>(sm.c[st], p.Cm, p.rc, b, t, te, g * p.N, g * p.N + p.N, p.vecbc);
    if (!END) {
      stage<IO, TB, CH, VW>(sm.u[st], p.u, p.ru, b, t, te, c0, cmax, p.vec);
      stage<IO, TB, NP, 4>(sm.b[st], p.Bm, p.rb, b, t, te, g * p.N, g * p.N + p.N, p.vecbc);
    }
    cp_commit();
  };
  // behind the sequence's end: zeros
  if (!END) {
    for (int t = max(t0, te); t < t1; ++t)
      for (int i = tid; i < CH; i += NT)
        if (c0 + i < cmax) {
          const size_t at = ((size_t)b * p.T + t) * p.D + c0 + i;
          ((IO*)p.du)[at] = from_f<IO>(0.f);
          ((IO*)p.ddt)[at] = from_f<IO>(0.f);
          if (p.dz) ((IO*)p.dz)[at] = from_f<IO>(0.f);
        }
  }
  int t = t0 < te ? t0 + (te - 1 - t0) / TB * TB : t0 - 1;  // the last tile
  if (t >= t0) load(t, 0);
  int st = 0;
  for (; t >= t0; t -= TB, st ^= 1) {
    f2 h[2] = {0, 0};
    if (!END && on) {
      const float4 x = *reinterpret_cast<const float4*>(p.states + (((size_t)b * nck + t / kCk) * p.D + c) * p.N + n0);
      h[0] = pk(x.x, x.y);
      h[1] = pk(x.z, x.w);
    }
    cp_wait_all();
    __syncthreads();
    for (int i = tid; i < TB * CH; i += NT) {
      float dl = 0.f, u = 0.f, e = 0.f;
      const int cc = c0 + i % CH;
      if (t + i / CH < te && cc < cmax) {
        dl = to_f(sm.dt[st][i]) + (p.dtb ? p.dtb[cc] : 0.f);
        if (p.softplus) dl = softplus(dl);
        e = to_f(sm.dy[st][i]);
        if (p.z) {
          const float z = to_f(sm.z[st][i]);
          e *= z * sigmoid(z);
        }
        if (!END) u = to_f(sm.u[st][i]);
      }
      sm.q[i] = make_float4(dl, dl * u, e, u);
    }
    for (int i = tid; i < TB * NP; i += NT) {
      sm.cf[i] = to_f(sm.c[st][i]);
      if (!END) sm.bf[i] = to_f(sm.b[st][i]);
    }
    __syncthreads();
    if (t - TB >= t0) load(t - TB, st ^ 1);

    if constexpr (END) {
#pragma unroll 4
      for (int i = TB - 1; i >= 0; --i) {
        const float4 q = sm.q[i * CH + cl];
        const ulonglong2 C4 = *reinterpret_cast<const ulonglong2*>(&sm.cf[i * NP + n0]);
        const f2 e2 = pk(q.z, q.z), d2 = pk(q.x, q.x);
        gr[0] = mul2(fma2(e2, C4.x, gr[0]), ex2v(mul2(A2[0], d2)));
        gr[1] = mul2(fma2(e2, C4.y, gr[1]), ex2v(mul2(A2[1], d2)));
        sumd += q.x;
      }
    } else {
    // ---- forward over the tile: a and p = a h_{t-1} of every token
    f2 a[TB][2], pr[TB][2];
#pragma unroll
    for (int i = 0; i < TB; i += U) {
      float yv[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const float4 q = sm.q[(i + j) * CH + cl];
        const ulonglong2 B4 = *reinterpret_cast<const ulonglong2*>(&sm.bf[(i + j) * NP + n0]);
        const f2 d2 = pk(q.x, q.x), du2 = pk(q.y, q.y);
        a[i + j][0] = ex2v(mul2(A2[0], d2));
        a[i + j][1] = ex2v(mul2(A2[1], d2));
        pr[i + j][0] = mul2(a[i + j][0], h[0]);
        pr[i + j][1] = mul2(a[i + j][1], h[1]);
        h[0] = fma2(du2, B4.x, pr[i + j][0]);
        h[1] = fma2(du2, B4.y, pr[i + j][1]);
        if (p.dz) {
          const ulonglong2 C4 = *reinterpret_cast<const ulonglong2*>(&sm.cf[(i + j) * NP + n0]);
          const f2 y2 = fma2(h[1], C4.y, mul2(h[0], C4.x));
          yv[j] = lo(y2) + hi(y2);
        }
      }
      if (p.dz) {
        int j = 0;
        reduce_scatter<U, L / 2, 1>(yv, lane, j);
        if (l % (L / U) == 0) sm.yc[(i + j) * YS + cl] = yv[0];
      }
    }
    // ---- and back
#pragma unroll
    for (int i = TB - U; i >= 0; i -= U) {
      float vB[U], vA[U];
#pragma unroll
      for (int j = U - 1; j >= 0; --j) {
        const int k = i + j;
        const float4 q = sm.q[k * CH + cl];
        const ulonglong2 B4 = *reinterpret_cast<const ulonglong2*>(&sm.bf[k * NP + n0]);
        const ulonglong2 C4 = *reinterpret_cast<const ulonglong2*>(&sm.cf[k * NP + n0]);
        const f2 d2 = pk(q.x, q.x), du2 = pk(q.y, q.y), e2 = pk(q.z, q.z);
        gr[0] = fma2(e2, C4.x, gr[0]);
        gr[1] = fma2(e2, C4.y, gr[1]);
        const f2 dB0 = mul2(gr[0], du2), dB1 = mul2(gr[1], du2);
        const f2 dC0 = mul2(fma2(du2, B4.x, pr[k][0]), e2), dC1 = mul2(fma2(du2, B4.y, pr[k][1]), e2);
        const f2 sB = fma2(gr[1], B4.y, mul2(gr[0], B4.x));
        const f2 gp0 = mul2(gr[0], pr[k][0]), gp1 = mul2(gr[1], pr[k][1]);
        const f2 sA = fma2(gp1, A2[1], mul2(gp0, A2[0]));
        dA[0] = fma2(gp0, d2, dA[0]);
        dA[1] = fma2(gp1, d2, dA[1]);
        gr[0] = mul2(gr[0], a[k][0]);
        gr[1] = mul2(gr[1], a[k][1]);
        vB[j] = lo(sB) + hi(sB);
        vA[j] = lo(sA) + hi(sA);
        float v[8] = {lo(dB0), hi(dB0), lo(dB1), hi(dB1), lo(dC0), hi(dC0), lo(dC1), hi(dC1)};
        int base = 0;
        reduce_scatter<8, 16, L>(v, lane, base);
        // what is left of the 8: 1 for L <= 4 (equal in lanes that differ below
        // bit 2 and from L up), 2 for L = 8, 4 for L = 16
        constexpr int LEFT = L <= 4 ? 1 : L / 4;
        if (L >= 4 || (lane & 3 & ~(L - 1)) == 0) {
#pragma unroll
          for (int x = 0; x < LEFT; ++x) {
            const int y = base + x;
            sm.red[warp][k][(y >> 2) * NP + n0 + (y & 3)] = v[x];
          }
        }
      }
      int j = 0;
      reduce_scatter<U, L / 2, 1>(vB, lane, j);
      j = 0;
      reduce_scatter<U, L / 2, 1>(vA, lane, j);
      if (l % (L / U) == 0) {
        sm.gB[(i + j) * YS + cl] = vB[0];
        sm.gA[(i + j) * YS + cl] = vA[0];
      }
    }
    __syncthreads();
    // ---- the tile's gradients
    for (int i = qt; i < TB; i += QT) {
      const bool live = t + i < te;
      float du[4], dd[4], dz[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int x = i * CH + qc + e, cc = c0 + qc + e;
        if (!live || cc >= cmax) continue;
        const float4 q = sm.q[x];
        const float Ds = p.Dskip ? p.Dskip[cc] : 0.f;
        const float gB = sm.gB[i * YS + qc + e];
        du[e] = fmaf(q.x, gB, Ds * q.z);
        dd[e] = fmaf(q.w, gB, kLn2 * sm.gA[i * YS + qc + e]);
        if (p.softplus) dd[e] *= sigmoid(to_f(sm.dt[st][x]) + (p.dtb ? p.dtb[cc] : 0.f));
        sD[e] = fmaf(q.z, q.w, sD[e]);
        sT[e] += dd[e];
        if (p.dz) {
          const float z = to_f(sm.z[st][x]), sg = sigmoid(z);
          dz[e] = to_f(sm.dy[st][x]) * fmaf(Ds, q.w, sm.yc[i * YS + qc + e]) * sg * (1.f + z * (1.f - sg));
        }
      }
      if (!live) continue;
      const size_t at = ((size_t)b * p.T + t + i) * p.D + c0 + qc;
      if (p.vec) {
        if (c0 + qc < cmax) {
          store_vec<4>((IO*)p.du + at, du);
          store_vec<4>((IO*)p.ddt + at, dd);
          if (p.dz) store_vec<4>((IO*)p.dz + at, dz);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c0 + qc + e < cmax) {
            ((IO*)p.du)[at + e] = from_f<IO>(du[e]);
            ((IO*)p.ddt)[at + e] = from_f<IO>(dd[e]);
            if (p.dz) ((IO*)p.dz)[at + e] = from_f<IO>(dz[e]);
          }
      }
    }
    for (int i = tid; i < TB * 2 * NP; i += NT) {
      const int k = i / (2 * NP), n = i % (2 * NP) % NP, w = i % (2 * NP) / NP;
      if (t + k < te && n < p.N) {
        float s = 0.f;
#pragma unroll
        for (int x = 0; x < kWarps; ++x) s += sm.red[x][k][w * NP + n];
        p.bc[(((((size_t)ct * p.B + b) * p.T + t + k) * p.G + g) * 2 + w) * p.N + n] = s;
      }
    }
    }  // !END
  }
  const float4 gv = make_float4(lo(gr[0]), hi(gr[0]), lo(gr[1]), hi(gr[1]));
  if (END) {
    if (on) *reinterpret_cast<float4*>(p.segE + seg * sstep + sidx) = gv;
    if (c < cmax && l == 0) p.segD[((size_t)seg * p.B + b) * p.D + c] = sumd;
    return;
  }
  if (p.dh0 && on && seg == 0) *reinterpret_cast<float4*>(p.dh0 + sidx) = gv;
  float* part = p.part + ((size_t)b * p.nseg + seg) * part_ld(p.D, p.N);
  if (on)
    *reinterpret_cast<float4*>(part + (size_t)c * p.N + n0) =
        make_float4(lo(dA[0]), hi(dA[0]), lo(dA[1]), hi(dA[1]));
  // sums of e u and ddt over the block's token rows, in order
  __syncthreads();
  float* s1 = &sm.red[0][0][0];
  float* s2 = reinterpret_cast<float*>(sm.q);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    s1[qt * CH + qc + e] = sD[e];
    s2[qt * CH + qc + e] = sT[e];
  }
  __syncthreads();
  for (int i = tid; i < CH; i += NT)
    if (c0 + i < cmax) {
      float x = 0.f, y = 0.f;
      for (int k = 0; k < QT; ++k) {
        x += s1[k * CH + i];
        y += s2[k * CH + i];
      }
      part[(size_t)p.D * p.N + c0 + i] = x;
      part[(size_t)p.D * (p.N + 1) + c0 + i] = y;
    }
}

// dB, dC of a token: the channel tiles' shares added in order.  One thread per
// value; behind a sequence's end zeros.
template <typename IO>
__global__ void __launch_bounds__(256) scan_bc_kernel(ScanParams p) {
  const size_t per = (size_t)p.T * p.G * 2 * p.N, tot = per * p.B;
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= tot) return;
  const int b = (int)(i / per);
  const size_t r = i % per;
  const int n = (int)(r % p.N), w = (int)(r / p.N % 2);
  const size_t tg = r / (2 * p.N);
  const int t = (int)(tg / p.G);
  float s = 0.f;
  if (t < seq_len(p.lens, b, p.T)) {
#pragma unroll 4
    for (int x = 0; x < p.nct; ++x) s += p.bc[(size_t)x * tot + i];
  }
  IO* out = (IO*)(w ? p.dC : p.dB);
  out[((size_t)b * p.T * p.G + tg) * p.N + n] = from_f<IO>(s);
}

template <typename IO, int L>
cudaError_t go(const ScanParams& p, cudaStream_t s) {
  const size_t smem = sizeof(Smem<IO, L>);
  cudaError_t e = cudaSuccess;
  if (smem > 48 * 1024) {
    e = cudaFuncSetAttribute(scan_bwd_kernel<IO, L, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(scan_bwd_kernel<IO, L, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  if (p.nseg > 1) {
    ScopedTiming tm("scan_bwd_ends", s);
    scan_bwd_kernel<IO, L, true><<<dim3(p.G * p.nct, p.B, p.nseg - 1), NT, smem, s>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  {
    ScopedTiming tm("scan_bwd", s);
    scan_bwd_kernel<IO, L, false><<<dim3(p.G * p.nct, p.B, p.nseg), NT, smem, s>>>(p);
  }
  e = cudaGetLastError();
  const size_t n = (size_t)p.B * p.T * p.G * 2 * p.N;
  if (e != cudaSuccess || n == 0) return e;
  ScopedTiming tm("scan_bc_sum", s);
  scan_bc_kernel<IO><<<(unsigned)((n + 255) / 256), 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace
}  // namespace scan

cudaError_t launch_scan_bwd(const scan::ScanParams& p0, int L, bool bf, cudaStream_t s) {
  scan::ScanParams p = p0;
  // gradients are contiguous: vectors of 4 need whole rows of them
  const size_t es = bf ? 2 : 4;
  p.vec = p.vec && rows_vec(p.dy, Rows{p.D, 0}, (int)(16 / es), es);
  switch (L) {
    case 1: return bf ? scan::go<bf16, 1>(p, s) : scan::go<float, 1>(p, s);
    case 2: return bf ? scan::go<bf16, 2>(p, s) : scan::go<float, 2>(p, s);
    case 4: return bf ? scan::go<bf16, 4>(p, s) : scan::go<float, 4>(p, s);
    case 8: return bf ? scan::go<bf16, 8>(p, s) : scan::go<float, 8>(p, s);
    case 16: return bf ? scan::go<bf16, 16>(p, s) : scan::go<float, 16>(p, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace lz
