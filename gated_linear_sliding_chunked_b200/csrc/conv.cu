// Short causal convolution over the tokens, a channel at a time, with its
// activation: y_t = act(bias + sum_{j<K} w_j x_{t-K+1+j}).
//
// Every element is read and written once (forward 2 values, backward 3), with
// 2K + a few operations in between: bound by HBM bandwidth.  A thread holds a
// vector of neighbouring channels and walks a run of tokens with the last K-1
// inputs in registers, so that a token is read once and only the K-1 tokens
// before a run are read twice (they come out of L2).  At 2 x 8192 tokens, 4096
// channels, 4 taps (bf16) the backward takes 98 us: 62 % of the copy
// bandwidth; its 26 instructions an element (counted) and few resident warps
// (166 registers) hold it there.  The forward takes 59 us (69 %).
#include <type_traits>

#include "layer.cuh"

namespace lz {
namespace {

constexpr int NT = 128;

struct ConvParams {
  int B, T, D, silu, run;  // run: tokens of a thread, a multiple of RT
  Rows x;
  const void* px;
  const float* w;
  const float* bias;
  const void* x0;
  const int64_t* lens;
  void* y;
  void* xT;
};

constexpr int RT = 8;  // tokens whose loads are in flight at once

// x at token t of sequence b; the history where t < 0
template <typename IO, int K, int VW>
__device__ __forceinline__ void load_x(const ConvParams& p, int b, int t, int c, Raw<IO, VW>& v) {
  if (t >= 0) v.load((const IO*)p.px + p.x.at(b, t) + c);
  else if (p.x0) v.load((const IO*)p.x0 + ((size_t)b * (K - 1) + (t + K - 1)) * p.D + c);
  else v.zero();
}

// Taps and biases of VW neighbouring channels: w[e * K + j]
template <int K, int VW>
__device__ __forceinline__ void load_taps(const ConvParams& p, int c, float* w, float* bias) {
  load_floats<K * VW>(p.w + (size_t)c * K, w);
  if (p.bias) {
    load_floats<VW>(p.bias + c, bias);
  } else {
#pragma unroll
    for (int e = 0; e < VW; ++e) bias[e] = 0.f;
  }
}

template <typename IO, int K, int VW>
__global__ void __launch_bounds__(NT) conv_fwd_kernel(ConvParams p) {
  const int nvec = p.D / VW;
  const int nrun = max(1, (p.T + p.run - 1) / p.run);
  const unsigned idx = blockIdx.x * NT + threadIdx.x;
  const int b = blockIdx.y;
  const int run = (int)(idx / (unsigned)nvec);
  const int c = (int)(idx - (unsigned)run * nvec) * VW;
  if (run >= nrun) return;
  const int L = seq_len(p.lens, b, p.T);
  if (run == 0 && p.xT) {
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      Raw<IO, VW> v;
      load_x<IO, K, VW>(p, b, L - (K - 1) + j, c, v);
      v.put((IO*)p.xT + ((size_t)b * (K - 1) + j) * p.D + c);
    }
  }
  const int t0 = run * p.run, t1 = min(p.T, t0 + p.run), te = min(t1, L);
  IO* y = (IO*)p.y + ((size_t)b * p.T + t0) * p.D + c;
  const IO* x = (const IO*)p.px + p.x.at(b, t0) + c;
  using V = Vec<VW>;
  V w[K], bias, h[K > 1 ? K - 1 : 1];
  if (t0 < te) {
    Raw<IO, VW> v[RT], g[K > 1 ? K - 1 : 1];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) load_x<IO, K, VW>(p, b, t0 - (K - 1) + j, c, g[j]);
#pragma unroll
    for (int i = 0; i < RT; ++i) v[i].load_if(x + i * p.x.ld, t0 + i < te);
    {
      float wf[K * VW], bf[VW];
      load_taps<K, VW>(p, c, wf, bf);
#pragma unroll
      for (int j = 0; j < K; ++j) w[j].set([&](int e) { return wf[e * K + j]; });
      bias.set([&](int e) { return bf[e]; });
    }
#pragma unroll
    for (int j = 0; j < K - 1; ++j) h[j].set([&](int e) { return g[j].get(e); });
    for (int t = t0;;) {
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        V x, a;
        x.set([&](int e) { return v[i].get(e); });
        a.fma(w[K - 1], x, bias);
#pragma unroll
        for (int j = 0; j < K - 1; ++j) a.fma(w[j], h[j], a);
#pragma unroll
        for (int j = 0; j + 1 < K - 1; ++j) h[j] = h[j + 1];
        if (K > 1) h[K > 1 ? K - 2 : 0] = x;
        float o[VW];
#pragma unroll
        for (int e = 0; e < VW; ++e) o[e] = a.get(e);
        if (p.silu) {
#pragma unroll
          for (int e = 0; e < VW; ++e) o[e] *= sigmoid(o[e]);
        }
        if (t + i < te) store_vec<VW>(y + (size_t)i * p.D, o);
      }
      t += RT;
      if (t >= te) break;
      x += RT * p.x.ld;
      y += (size_t)RT * p.D;
#pragma unroll
      for (int i = 0; i < RT; ++i) v[i].load_if(x + i * p.x.ld, t + i < te);
    }
  }
  if (te < t1) {  // behind the sequence's end: zeros
    Raw<IO, VW> z;
    z.zero();
    IO* yz = (IO*)p.y + ((size_t)b * p.T) * p.D + c;
    for (int t = max(t0, te); t < t1; ++t) z.put(yz + (size_t)t * p.D);
  }
}

template <typename IO, int K, int VW>
__global__ void __launch_bounds__(NT) conv_step_kernel(ConvParams p, void* hist) {
  static_assert(VW == 1 || VW * sizeof(IO) == 16, "the history is read an element or 16 bytes at a time");
  const int c = (blockIdx.x * NT + threadIdx.x) * VW;
  if (c >= p.D) return;
  float w[K * VW], bias[VW];
  load_taps<K, VW>(p, c, w, bias);
  for (int b = blockIdx.y; b < p.B; b += gridDim.y) {
    Raw<IO, VW> h[K];
    IO* hp = (IO*)hist + (size_t)b * (K - 1) * p.D + c;
    h[K - 1].load((const IO*)p.px + p.x.at(b, 0) + c);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      // (plain loads: the history is written below)
#pragma unroll
      for (int i = 0; i < Raw<IO, VW>::W; ++i) h[j].w[i] = 0;
      Raw<IO, VW>& r = h[j];
      const IO* q = hp + (size_t)j * p.D;
      if constexpr (VW == 1) {
        if constexpr (sizeof(IO) == 2) r.w[0] = *reinterpret_cast<const unsigned short*>(q);
        else r.w[0] = *reinterpret_cast<const uint32_t*>(q);
      } else {
        const uint4 u = *reinterpret_cast<const uint4*>(q);
        r.w[0] = u.x; r.w[1] = u.y; r.w[2] = u.z; r.w[3] = u.w;
      }
    }
#pragma unroll
    for (int j = 0; j < K - 1; ++j) h[j + 1].put(hp + (size_t)j * p.D);
    float o[VW];
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      float a = fmaf(w[e * K + K - 1], h[K - 1].get(e), bias[e]);
#pragma unroll
      for (int j = 0; j < K - 1; ++j) a = fmaf(w[e * K + j], h[j].get(e), a);
      o[e] = p.silu ? a * sigmoid(a) : a;
    }
    store_vec<VW>((IO*)p.y + (size_t)b * p.D + c, o);
  }
}

// ---- backward -------------------------------------------------------------
// dp_t = dy_t act'(p_t) needs the inputs up to K-1 tokens back, dx_t =
// sum_j w_j dp_{t+K-1-j} the dp up to K-1 tokens ahead: a run of tokens
// [t0, t1) forms dp for [t0, t1 + K-1) with both windows in registers, RT
// tokens at a time.  A warp holds 32 channel vectors, the block's warps
// neighbouring runs; the parameter gradients stay in registers over the run
// and are added across the warps in shared memory, one partial per block,
// which launch_sum_rows adds up.
constexpr int kWarps = 4;

struct ConvBwdParams {
  ConvParams f;
  const void* dy;
  const void* dxT;
  void* dx;
  void* dx0;
  float* part;  // [blocks over (b, runs)][D*K + D]
};

template <typename IO, int K, int VW>
__global__ void __launch_bounds__(kWarps * 32) conv_bwd_kernel(ConvBwdParams q) {
  __shared__ float red[kWarps][32 * VW];
  constexpr int KW = K > 1 ? K - 1 : 1;
  using V = Vec<VW>;
  const ConvParams& p = q.f;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int b = blockIdx.z;
  const int c = (blockIdx.x * 32 + lane) * VW;
  const bool on = c < p.D;
  const int L = seq_len(p.lens, b, p.T);
  const int t0 = (blockIdx.y * kWarps + warp) * p.run, t1 = min(p.T, t0 + p.run);
  const bool first = t0 == 0 && q.dx0;
  V w[K], bias, xw[KW], dpw[KW], dw[K], db;
  db.fill(0.f);
#pragma unroll
  for (int j = 0; j < K; ++j) dw[j].fill(0.f);
#pragma unroll
  for (int j = 0; j < KW; ++j) {
    dpw[j].fill(0.f);
    xw[j].fill(0.f);
  }
  if (on && (t0 < t1 || first)) {
    {
      float wf[K * VW], bf[VW];
      load_taps<K, VW>(p, c, wf, bf);
#pragma unroll
      for (int j = 0; j < K; ++j) w[j].set([&](int e) { return wf[e * K + j]; });
      bias.set([&](int e) { return bf[e]; });
    }
    if (t0 < L) {
      Raw<IO, VW> g[KW];
#pragma unroll
      for (int j = 0; j < K - 1; ++j) load_x<IO, K, VW>(p, b, t0 - (K - 1) + j, c, g[j]);
#pragma unroll
      for (int j = 0; j < K - 1; ++j) xw[j].set([&](int e) { return g[j].get(e); });
    }
    // s walks the tokens whose dp is formed; dx of token s - (K-1) is then
    // complete.  RT tokens at a time, the next ones' loads in flight.
    const int send = t1 + K - 1, slive = min(send, L);
    // [t0 + RT, sin): whole chunks of this run's own tokens, all live (s < L keeps
    // t below L - (K-1), so that their dx rows get nothing from the final history)
    const int sin = min(t1, L);
    const IO* px = (const IO*)p.px + p.x.at(b, t0) + c;
    const IO* pdy = (const IO*)q.dy + ((size_t)b * p.T + t0) * p.D + c;
    IO* pdx = (IO*)q.dx + ((int64_t)b * p.T + t0 - (K - 1)) * p.D + c;  // (used from token t0 on)
    Raw<IO, VW> nx[RT], ndy[RT];
    auto fetch = [&](int s0) {
      if (s0 + RT <= slive) {
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          nx[i].load(px + i * p.x.ld);
          ndy[i].load(pdy + (int64_t)i * p.D);
        }
      } else {
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          nx[i].load_if(px + i * p.x.ld, s0 + i < slive);
          ndy[i].load_if(pdy + (int64_t)i * p.D, s0 + i < slive);
        }
      }
      px += RT * p.x.ld;
      pdy += (int64_t)RT * p.D;
    };
    auto chunk = [&](int s0, const Raw<IO, VW> (&xv)[RT], const Raw<IO, VW> (&dyv)[RT], auto edge) {
      constexpr bool EDGE = decltype(edge)::value;
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const int s = s0 + i, t = s - (K - 1);
        V x, a, dp, o;
        x.set([&](int e) { return xv[i].get(e); });
        if (p.silu) {
          a.fma(w[K - 1], x, bias);
#pragma unroll
          for (int j = 0; j < K - 1; ++j) a.fma(w[j], xw[j], a);
          dp.set([&](int e) {
            const float v = a.get(e), sg = sigmoid(v), vs = v * sg;
            return dyv[i].get(e) * fmaf(-vs, sg, sg + vs);
          });
          // (dy is zero behind the end, act'(p) need not be finite there)
          if (EDGE && s >= slive) dp.fill(0.f);
        } else {
          dp.set([&](int e) { return dyv[i].get(e); });
        }
        if (!EDGE || s < t1) {  // (tokens of the next run are that run's own)
          db.add(dp);
          dw[K - 1].fma(dp, x, dw[K - 1]);
#pragma unroll
          for (int j = 0; j < K - 1; ++j) dw[j].fma(dp, xw[j], dw[j]);
        }
        // dx_t = sum_j w_j dp_{s-j}
        o.mul(w[0], dp);
#pragma unroll
        for (int j = 1; j < K; ++j) o.fma(w[j], dpw[KW - j], o);
#pragma unroll
        for (int j = 0; j + 1 < K - 1; ++j) {
          xw[j] = xw[j + 1];
          dpw[j] = dpw[j + 1];
        }
        if (K > 1) {
          xw[KW - 1] = x;
          dpw[KW - 1] = dp;
        }
        if (!EDGE || (t < t1 && (t >= t0 || first))) {
          float of[VW];
#pragma unroll
          for (int e = 0; e < VW; ++e) of[e] = o.get(e);
          if (EDGE && q.dxT && t >= L - (K - 1) && t < L) {
            float g[VW];  // token t is this row of the final history
            load_vec<VW>((const IO*)q.dxT + ((size_t)b * (K - 1) + (t - (L - (K - 1)))) * p.D + c, g);
#pragma unroll
            for (int e = 0; e < VW; ++e) of[e] += g[e];
          }
          if (!EDGE || t >= 0) store_vec<VW>(pdx + (int64_t)i * p.D, of);
          else store_vec<VW>((IO*)q.dx0 + ((size_t)b * (K - 1) + t + K - 1) * p.D + c, of);
        }
      }
      pdx += (int64_t)RT * p.D;
    };
    fetch(t0);
    for (int s0 = t0; s0 < send; s0 += RT) {
      Raw<IO, VW> xv[RT], dyv[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        xv[i] = nx[i];
        dyv[i] = ndy[i];
      }
      if (s0 + RT < send) fetch(s0 + RT);
      if (s0 > t0 && s0 + RT <= sin) chunk(s0, xv, dyv, std::false_type{});
      else chunk(s0, xv, dyv, std::true_type{});
    }
  }
  // ---- the block's partial of dw, dbias: warps added in order
  const size_t C = (size_t)p.D * (K + 1);
  float* part = q.part + ((size_t)b * gridDim.y + blockIdx.y) * C;
#pragma unroll
  for (int j = 0; j <= K; ++j) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < VW; ++e) red[warp][lane * VW + e] = j < K ? dw[j < K ? j : 0].get(e) : db.get(e);
    __syncthreads();
    for (int x = threadIdx.x; x < 32 * VW; x += kWarps * 32) {
      const int ch = blockIdx.x * 32 * VW + x;
      if (ch < p.D) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) t += red[k][x];
        part[j < K ? (size_t)ch * K + j : (size_t)p.D * K + ch] = t;
      }
    }
  }
}

// ---- host -----------------------------------------------------------------

lz_status check_conv(const char* fn, const lz_conv_dims* d) {
  if (!d) return layer_fail(LZ_ERR_INVALID_ARG, "%s: dims must not be NULL", fn);
  if (d->B < 0 || d->T < 0 || d->D < 0)
    return layer_fail(LZ_ERR_INVALID_ARG, "%s: B, T, D must be >= 0 (got %d, %d, %d)", fn, d->B, d->T, d->D);
  if (!io_ok(d->io))
    return layer_fail(LZ_ERR_UNSUPPORTED, "%s: io dtype %d is not LZ_F32 or LZ_BF16", fn, (int)d->io);
  if (d->K < 1 || d->K > 8)
    return layer_fail(LZ_ERR_UNSUPPORTED, "%s: taps K must be in [1, 8] (got %d)", fn, d->K);
  if (d->silu != 0 && d->silu != 1)
    return layer_fail(LZ_ERR_INVALID_ARG, "%s: silu must be 0 or 1 (got %d)", fn, d->silu);
  if (!rows_ok(d->x)) return layer_fail(LZ_ERR_INVALID_ARG, "%s: bad row strides", fn);
  if (d->B > 65535) return layer_fail(LZ_ERR_UNSUPPORTED, "%s: B must be <= 65535 (got %d)", fn, d->B);
  // keeps grid dimensions and 32-bit token indices in range
  if (d->T > (1 << 23) || (double)d->T * d->D > (double)(1ll << 34))
    return layer_fail(LZ_ERR_UNSUPPORTED, "%s: problem too large (T %d, D %d)", fn, d->T, d->D);
  return LZ_OK;
}

// Vectors of vw elements where rows and pointers allow it, else single elements
bool conv_vec(const lz_conv_dims* d, const void* x, const Rows& r, int vw) {
  return d->D % vw == 0 && rows_vec(x, r, vw, esize(d->io));
}

// Over sequences 4 channels a thread: with 8 the forward takes 128 registers, not
// 78 (4 taps, 16 bits; 2 x 8192 x 4096: 70 us against 59), and the backward's
// windows do not fit.  BFV: those of a 16-bit vector.
template <template <typename, int, int> class Launch, int BFV, typename P>
cudaError_t dispatch_k(const P& p, int K, bool bf, bool vec, cudaStream_t s) {
  switch (K) {
#define LZ_K(k)                                                                         \
  case k:                                                                               \
    if (bf) return vec ? Launch<bf16, k, BFV>::go(p, s) : Launch<bf16, k, 1>::go(p, s); \
    return vec ? Launch<float, k, 4>::go(p, s) : Launch<float, k, 1>::go(p, s);
    LZ_K(1) LZ_K(2) LZ_K(3) LZ_K(4) LZ_K(5) LZ_K(6) LZ_K(7) LZ_K(8)
#undef LZ_K
  }
  return cudaErrorInvalidValue;
}

template <typename IO, int K, int VW>
struct FwdLaunch {
  static cudaError_t go(const ConvParams& p, cudaStream_t s) {
    const size_t nrun = std::max(1, (p.T + p.run - 1) / p.run);
    const dim3 grid((unsigned)((nrun * (p.D / VW) + NT - 1) / NT), p.B);
    ScopedTiming tm("conv_fwd", s);
    conv_fwd_kernel<IO, K, VW><<<grid, NT, 0, s>>>(p);
    return cudaGetLastError();
  }
};

struct StepParams {
  ConvParams p;
  void* hist;
};
template <typename IO, int K, int VW>
struct StepLaunch {
  static cudaError_t go(const StepParams& q, cudaStream_t s) {
    const int gx = (q.p.D / VW + NT - 1) / NT;
    // a thread keeps its taps over several sequences once the device is full
    const int gy = std::max(1, std::min(q.p.B, 148 * 8 / gx));
    ScopedTiming tm("conv_step", s);
    conv_step_kernel<IO, K, VW><<<dim3(gx, gy), NT, 0, s>>>(q.p, q.hist);
    return cudaGetLastError();
  }
};

// Tokens of a run of the backward, and blocks over a sequence.  The blocks come
// in rounds of as many as the SMs hold at once (by registers, at 4 taps), and a
// run costs its tokens and some 8 more to begin and end: the run whose rounds
// cost the least.
int bwd_blocks(const lz_conv_dims* d, int* run) {
  const bool vec = d->D % 4 == 0;
  const int64_t cols = (int64_t)d->B * ((d->D + (vec ? 127 : 31)) / (vec ? 128 : 32));
  const int64_t slots = 148 * (!vec ? 6 : d->io == LZ_BF16 ? 3 : 2);
  int64_t best = 0;
  int tb = 1;
  for (int r = 256; r >= 8; r -= 8) {
    const int n = std::max(1, (d->T + r * kWarps - 1) / (r * kWarps));
    if (n > 65535) break;  // (a grid's limit)
    const int64_t cost = ((cols * n + slots - 1) / slots) * (r + 8);
    if (!best || cost < best) {
      best = cost;
      *run = r;
      tb = n;
    }
  }
  return tb;
}

template <typename IO, int K, int VW>
struct BwdLaunch {
  static cudaError_t go(const ConvBwdParams& q, cudaStream_t s) {
    const ConvParams& p = q.f;
    const int tb = std::max(1, (p.T + p.run * kWarps - 1) / (p.run * kWarps));
    const dim3 grid((p.D + 32 * VW - 1) / (32 * VW), tb, p.B);
    ScopedTiming tm("conv_bwd", s);
    conv_bwd_kernel<IO, K, VW><<<grid, kWarps * 32, 0, s>>>(q);
    return cudaGetLastError();
  }
};

}  // namespace

size_t conv_bwd_ws(const lz_conv_dims* d) {
  if (check_conv("lz_layer_workspace_bytes", d) != LZ_OK || d->B == 0 || d->D == 0) return 0;
  int run;
  return ws_round((size_t)d->B * bwd_blocks(d, &run) * d->D * (d->K + 1) * sizeof(float));
}

}  // namespace lz

using namespace lz;

extern "C" lz_status lz_conv_fwd(const lz_conv_dims* d, const void* x, const float* w, const float* bias,
                                 const void* x0, const int64_t* lens, void* y, void* xT,
                                 lz_stream stream) {
  const char* fn = "lz_conv_fwd";
  lz_status st = check_conv(fn, d);
  if (st != LZ_OK) return st;
  if (d->B == 0 || d->D == 0 || (d->T == 0 && !xT)) return layer_done(cudaSuccess, fn);
  const bool data = d->T > 0;
  st = check_ptrs(fn, {{x, "x", data, (unsigned)esize(d->io)}, {w, "w", true, 16}, {bias, "bias", false, 16},
                       {x0, "x0", false, 16}, {lens, "lens", false, 8}, {y, "y", data, 16}, {xT, "xT", false, 16}});
  if (st == LZ_OK) st = check_distinct(fn, {y, xT}, {x, x0});
  if (st != LZ_OK) return st;
  ConvParams p{d->B, d->T, d->D, d->silu, RT, rows_of(d->x, d->T, d->D), x, w, bias, x0, lens, y, xT};
  const bool vec = conv_vec(d, x, p.x, 4);
  // long runs re-read less of the input (K - 1 tokens each, from L2); with few
  // of them runs of RT tokens put more threads on the machine
  const size_t vecs = d->D / (vec ? 4 : 1);
  while (p.run < 4 * RT && (size_t)d->B * ((d->T + 2 * p.run - 1) / (2 * p.run)) * vecs >= 148 * 2048) p.run *= 2;
  return layer_done(dispatch_k<FwdLaunch, 4>(p, d->K, d->io == LZ_BF16, vec, (cudaStream_t)stream), fn);
}

extern "C" lz_status lz_conv_bwd(const lz_conv_dims* d, const void* x, const float* w, const float* bias,
                                 const void* x0, const int64_t* lens, const void* dy, const void* dxT, void* dx,
                                 float* dw, float* dbias, void* dx0, void* ws, size_t ws_bytes,
                                 lz_stream stream) {
  const char* fn = "lz_conv_bwd";
  lz_status st = check_conv(fn, d);
  if (st != LZ_OK) return st;
  if (d->D == 0) return layer_done(cudaSuccess, fn);
  const bool data = d->T > 0 && d->B > 0;
  st = check_ptrs(fn, {{x, "x", data, (unsigned)esize(d->io)}, {w, "w", true, 16}, {bias, "bias", false, 16},
                       {x0, "x0", false, 16}, {lens, "lens", false, 8}, {dy, "dy", data, 16},
                       {dxT, "dxT", false, 16}, {dx, "dx", data, 16}, {dw, "dw", true, 16},
                       {dbias, "dbias", false, 16}, {dx0, "dx0", false, 16}, {ws, "workspace", d->B > 0, 256}});
  if (st == LZ_OK) st = check_distinct(fn, {dx, dw, dbias, dx0, ws}, {x, w, bias, x0, dy, dxT});
  if (st != LZ_OK) return st;
  const size_t need = conv_bwd_ws(d);
  if (ws_bytes < need)
    return layer_fail(LZ_ERR_INVALID_ARG, "%s: workspace too small (%zu bytes, need %zu)", fn, ws_bytes, need);
  int run;
  const int tb = bwd_blocks(d, &run);
  ConvBwdParams q{{d->B, d->T, d->D, d->silu, run, rows_of(d->x, d->T, d->D), x, w, bias, x0, lens, nullptr, nullptr},
                  dy, dxT, dx, dx0, (float*)ws};
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = cudaSuccess;
  if (d->B > 0) e = dispatch_k<BwdLaunch, 4>(q, d->K, d->io == LZ_BF16, conv_vec(d, x, q.f.x, 4), s);
  if (e == cudaSuccess)
    e = launch_sum_rows({(const float*)ws, d->B * tb, (size_t)d->D * (d->K + 1), dw, (size_t)d->D * d->K, dbias,
                         (size_t)d->D, nullptr, 0},
                        s);
  return layer_done(e, fn);
}

extern "C" lz_status lz_conv_step(const lz_conv_dims* d, void* hist, const void* x, const float* w,
                                  const float* bias, void* y, lz_stream stream) {
  const char* fn = "lz_conv_step";
  lz_status st = check_conv(fn, d);
  if (st != LZ_OK) return st;
  if (d->B == 0 || d->D == 0) return layer_done(cudaSuccess, fn);
  st = check_ptrs(fn, {{hist, "hist", d->K > 1, 16}, {x, "x", true, (unsigned)esize(d->io)}, {w, "w", true, 16},
                       {bias, "bias", false, 16}, {y, "y", true, 16}});
  if (st == LZ_OK) st = check_distinct(fn, {hist, y}, {x});
  if (st != LZ_OK) return st;
  StepParams q{{d->B, 1, d->D, d->silu, RT, rows_of(d->x, 1, d->D), x, w, bias, nullptr, nullptr, y, nullptr}, hist};
  return layer_done(
      dispatch_k<StepLaunch, 8>(q, d->K, d->io == LZ_BF16, conv_vec(d, x, q.p.x, (int)(16 / esize(d->io))), (cudaStream_t)stream), fn);
}
