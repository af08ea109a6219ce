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
// every 16th (4 bytes a state), and a tile of 16 tokens is run forward again,
// leaving its states in registers, before it is walked back; the decays are
// taken on both ways.  dB and dC are sums over all channels: first within the
// thread, then over a warp's channels by halving exchanges, then over the
// block's warps in shared memory, then over the channel tiles in a second
// kernel, in a fixed order.
//
// Per (token, 4 states of a channel) about 123 instructions, 99 of them the
// scan warps', and 14 warps of 128 registers an SM to issue them.  At 2 x 8192
// tokens, 4096 channels, 16 states (bf16, gated) 1556 to 1574 us, 56 % of the
// issue slots on average (a seventh of the schedulers have one scan warp, the
// others two); what its warps wait for most is the barrier after every tile (1.6
// cycles an instruction).  Its bytes would take 184 us, its exps 480 us.
#include "scan.cuh"

namespace lz {
namespace scan {
namespace {

// A thread holds 2 channels x 2 states: pairs of channels are what the packed
// arithmetic works on, and the sums over channels start within the thread.  (4
// states of one channel to a thread took 28 instructions a token for those
// sums against 14, and moves to repeat each step and input in a pair of
// registers: 1745 us against 1677 us at 2 x 8192 tokens, 4096 channels, 16
// states.)  L: lanes of a channel pair.
template <int L, int W>
struct Geo {
  static constexpr int NS = 32 * W, NE = 32 * W;  // scan threads, elementwise threads
  static constexpr int CH = 2 * NS / L;     // channels of a block
  static constexpr int NP = 2 * L;          // states, padded
  static constexpr int U = L < 8 ? L / 2 : 4;  // tokens whose lane sums are formed together
  static constexpr int YS = row_of(CH, L == 4 ? 16 : L == 8 ? 8 : 4);
  static constexpr int DS = CH / 2 + 1;     // row of a [tokens][channel pairs] tile of 4 words
  static constexpr int EV = kCk * CH / NE > 8 ? 8 : kCk * CH / NE > 1 ? kCk * CH / NE : 2;  // channels of an elementwise thread
};

// 2 elements of B or C as the scan warps read them from shared memory, each
// twice in a register pair.  They stay in the I/O type there: what a warp's
// shared memory loads return to registers, 128 bytes a cycle and SM however
// many lanes read the same words, is what the scan runs out of first.
template <typename IO>
__device__ __forceinline__ void load_bc(const IO* p, f2& x, f2& y) {
  float a, b;
  if constexpr (sizeof(IO) == 4) {
    const float2 v = *reinterpret_cast<const float2*>(p);
    a = v.x;
    b = v.y;
  } else {
    const uint32_t v = *reinterpret_cast<const uint32_t*>(p);
    a = __uint_as_float(v << 16);
    b = __uint_as_float(v & 0xffff0000u);
  }
  x = pk(a, a);
  y = pk(b, b);
}

// A thread's 2 channels x 2 states of an array [.., D][N] (p: its first): s[i]
// is state i of both channels.
__device__ __forceinline__ void load_state(const float* p, int N, bool on0, bool on1, f2 (&s)[2]) {
  float2 a = make_float2(0.f, 0.f), b = a;
  if (on0) a = *reinterpret_cast<const float2*>(p);
  if (on1) b = *reinterpret_cast<const float2*>(p + N);
  s[0] = pk(a.x, b.x);
  s[1] = pk(a.y, b.y);
}
__device__ __forceinline__ void store_state(float* p, int N, bool on0, bool on1, const f2 (&s)[2]) {
  if (on0) *reinterpret_cast<float2*>(p) = make_float2(lo(s[0]), lo(s[1]));
  if (on1) *reinterpret_cast<float2*>(p + N) = make_float2(hi(s[0]), hi(s[1]));
}

constexpr int TB = kCk;  // tokens of a tile
// The parameter gradients are summed over this many tiles at a time: thousands
// of tokens added to one 32-bit sum would cost it bits.  (At 2 x 8192 tokens the
// gradients of Dskip and dt_bias are off by 1.6e-7 and 4.1e-7, with one sum a
// thread by 4.1e-7 and 6.4e-7, for 0.7 % of the time, 1.7 % with 8 states; equal
// terms by 2^-24 for every token that a thread adds up.)
constexpr int kSum = 16;

template <typename IO, int L, int W>
struct alignas(16) Smem {
  using G = Geo<L, W>;
  static constexpr int NP = G::NP;
  float4 q[2][TB * G::DS];       // of a channel pair: delta, delta; delta u, delta u
  float2 qe[2][TB * G::DS];      // e, e
  IO bf[2][TB * NP], cf[2][TB * NP];
  float gB[2][TB * G::YS], gA[2][TB * G::YS], yc[2][TB * G::YS];
  float red[2][W][TB][2 * NP];  // dB, dC over a warp's channels
  ulonglong2 ck[2][G::NS];  // the state before the tile, as the scan threads hold it
  float sum[2][G::EV][G::NE];  // dDskip, ddt_bias of an elementwise thread's channels
};

// The scan warps' walk over one tile, forward and back.  Sums over lanes take
// an exchange's latency a stage, and a shared memory store waits for its
// value while the loads behind it wait for the store; so a token's operands
// are loaded, and the next token's arithmetic done, before its sums over the
// channels are formed and stored.
template <typename IO, int L, int W>
__device__ __forceinline__ void walk_tile(bool want_y, const ulonglong2 h0, const float4* q, const float2* qe,
                                          const IO* bf, const IO* cf, float* gB, float* gA, float* yc, float* red,
                                          f2 (&A2)[2], f2 (&gr)[2], f2 (&dA)[2], int lane, int l) {
  using G = Geo<L, W>;
  constexpr int NP = G::NP, U = G::U, YS = G::YS, DS = G::DS;
  // ---- forward: the state after every token, h[i + 1]
  f2 h[TB + 1][2];
  h[0][0] = h0.x;
  h[0][1] = h0.y;
  {
    f2 a[2][U][2], x[2][U][2];
    auto form = [&](int i, f2 (&a)[U][2], f2 (&x)[U][2]) {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const ulonglong2 d = *reinterpret_cast<const ulonglong2*>(&q[(i + j) * DS]);
        f2 B0, B1;
        load_bc(bf + (i + j) * NP, B0, B1);
        a[j][0] = decay(A2[0], d.x);
        a[j][1] = decay(A2[1], d.x);
        x[j][0] = mul2(d.y, B0);
        x[j][1] = mul2(d.y, B1);
      }
    };
    form(0, a[0], x[0]);
#pragma unroll
    for (int k = 0; k < TB / U; ++k) {
      const int i = k * U;
      if (i + U < TB) form(i + U, a[(k + 1) & 1], x[(k + 1) & 1]);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        h[i + j + 1][0] = fma2(a[k & 1][j][0], h[i + j][0], x[k & 1][j][0]);
        h[i + j + 1][1] = fma2(a[k & 1][j][1], h[i + j][1], x[k & 1][j][1]);
      }
      if (want_y) {
        float yv[2 * U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
          f2 C0, C1;
          load_bc(cf + (i + j) * NP, C0, C1);
          const f2 y2 = fma2(h[i + j + 1][1], C1, mul2(h[i + j + 1][0], C0));
          yv[2 * j] = lo(y2);
          yv[2 * j + 1] = hi(y2);
        }
        int j = 0;
        reduce_scatter<2 * U, L / 2, 1>(yv, lane, j);
        if (l % (L / (2 * U)) == 0) yc[(i + (j >> 1)) * YS + (j & 1)] = yv[0];
      }
    }
  }
  // ---- and back.  a is taken again, which costs less than keeping it (and the
  // compiler is kept from keeping it: 64 more registers would be spilled)
  asm volatile("" : "+l"(A2[0]), "+l"(A2[1]));
  struct Op {
    ulonglong2 d;
    f2 e, B0, B1, C0, C1;
  };
  auto load = [&](int m, Op& o) {
    o.d = *reinterpret_cast<const ulonglong2*>(&q[m * DS]);
    o.e = *reinterpret_cast<const f2*>(&qe[m * DS]);
    load_bc(bf + m * NP, o.B0, o.B1);
    load_bc(cf + m * NP, o.C0, o.C1);
  };
  // dB and dC of token m: over the warp's channels, then to the block's table
  auto sum_bc = [&](int m, float (&v)[4]) {
    int base = 0;
    reduce_scatter<4, 16, L>(v, lane, base);
    // what is left of the 4: 1 for L <= 8 (equal in the lanes that differ in a
    // bit below 8 and not below L), 2 for L = 16, 4 for L = 32
    constexpr int LEFT = L <= 8 ? 1 : L / 8;
    if ((lane & 7 & ~(L - 1)) == 0) {
#pragma unroll
      for (int y = 0; y < LEFT; ++y) {
        const int z = base + y;
        red[m * 2 * NP + (z >> 1) * NP + (z & 1)] = v[y];
      }
    }
  };
  Op op[2];
  float v[2][4];
  load(TB - 1, op[(TB - 1) & 1]);
#pragma unroll
  for (int i = TB - U; i >= 0; i -= U) {
    float vB[2 * U], vA[2 * U];
#pragma unroll
    for (int j = U - 1; j >= 0; --j) {
      const int m = i + j;
      if (m > 0) load(m - 1, op[(m - 1) & 1]);
      const Op& o = op[m & 1];
      const f2 d2 = o.d.x, du2 = o.d.y, e2 = o.e;
      gr[0] = fma2(e2, o.C0, gr[0]);
      gr[1] = fma2(e2, o.C1, gr[1]);
      const f2 dB0 = mul2(gr[0], du2), dB1 = mul2(gr[1], du2);
      const f2 dC0 = mul2(h[m + 1][0], e2), dC1 = mul2(h[m + 1][1], e2);
      const f2 sB = fma2(gr[1], o.B1, mul2(gr[0], o.B0));
      gr[0] = mul2(gr[0], decay(A2[0], d2));
      gr[1] = mul2(gr[1], decay(A2[1], d2));
      const f2 gp0 = mul2(gr[0], h[m][0]), gp1 = mul2(gr[1], h[m][1]);
      const f2 sA = fma2(gp1, A2[1], mul2(gp0, A2[0]));
      dA[0] = fma2(gp0, d2, dA[0]);
      dA[1] = fma2(gp1, d2, dA[1]);
      vB[2 * j] = lo(sB);
      vB[2 * j + 1] = hi(sB);
      vA[2 * j] = lo(sA);
      vA[2 * j + 1] = hi(sA);
      float (&w)[4] = v[m & 1];  // over the thread's two channels
      w[0] = lo(dB0) + hi(dB0);
      w[1] = lo(dB1) + hi(dB1);
      w[2] = lo(dC0) + hi(dC0);
      w[3] = lo(dC1) + hi(dC1);
      if (m + 1 < TB) sum_bc(m + 1, v[(m + 1) & 1]);
    }
    int j = 0;
    reduce_scatter<2 * U, L / 2, 1>(vB, lane, j);
    j = 0;
    reduce_scatter<2 * U, L / 2, 1>(vA, lane, j);
    if (l % (L / (2 * U)) == 0) {
      gB[(i + (j >> 1)) * YS + (j & 1)] = vB[0];
      gA[(i + (j >> 1)) * YS + (j & 1)] = vA[0];
    }
  }
  sum_bc(0, v[0]);
}

// END: only the gradient that the segment hands to the one before it when
// none comes from behind (the state gradient before its first token).
template <typename IO, int L, int W, bool END>
__global__ void __launch_bounds__(64 * W, L >= 8 && W == 4 ? 2 : 1) scan_bwd_kernel(ScanParams p) {
  using G = Geo<L, W>;
  constexpr int CH = G::CH, NP = G::NP, YS = G::YS;
  constexpr int NS = G::NS, NE = G::NE;
  constexpr int EV = G::EV;
  constexpr int ROWT = CH / EV;                                 // threads of a token
  constexpr int PASS = (TB * ROWT + NE - 1) / NE;               // tokens of a thread
  constexpr int BV = TB * NP / 4, BN = (BV + NE - 1) / NE;   // 4-element vectors of B and of C, a thread's
  extern __shared__ __align__(16) char raw[];
  using S = Smem<IO, L, W>;
  S& sm = *reinterpret_cast<S*>(raw);
  const int tid = threadIdx.x;
  const int g = blockIdx.x / p.nct, ct = blockIdx.x % p.nct;
  const int b = blockIdx.y, seg = END ? blockIdx.z + 1 : blockIdx.z;
  const int per = p.D / p.G;
  const int c0 = g * per + ct * CH, cmax = (g + 1) * per;
  const int Tb = seq_len(p.lens, b, p.T);
  const int t0 = seg * p.seg, t1 = min(p.T, t0 + p.seg), te = min(t1, Tb);
  const int ntile = t0 < te ? (te - t0 + TB - 1) / TB : 0;
  // step k of the walk back is tile ntile - 1 - k
  float* part = p.part + ((size_t)b * p.nseg + seg) * part_ld(p.D, p.N);

  if (tid >= NS) {
    // ---- elementwise warps
    const int et = tid - NS;
    const int cl = et % ROWT * EV, c = c0 + cl, i0 = et / ROWT;  // channels; first token of the tile
    constexpr int IS = NE / ROWT;                                // tokens between a thread's
    const int nc = min(EV, cmax - c);
    struct Next {
      Pack<IO, EV> u, dt, z, dy;
    };
    struct Tok {  // what the outputs of a token need
      float delta[EV], e[EV], u[EV], sg[EV], dzf[EV];
    };
    Next nx[PASS];
    Pack<IO, 4> nb[BN], ncv[BN];
    Tok tok[2][PASS];
    float Ds[EV], bias[EV], sD[EV], sT[EV];  // (sums of up to kSum tiles, added to sm.sum)
    const bool many = !END && ntile >= kSum;
#pragma unroll
    for (int e = 0; e < EV; ++e) {
      Ds[e] = p.Dskip && e < nc ? p.Dskip[c + e] : 0.f;
      bias[e] = p.dtb && e < nc ? p.dtb[c + e] : 0.f;
      sD[e] = sT[e] = 0.f;
      if (many) sm.sum[0][e][et] = sm.sum[1][e][et] = 0.f;
    }
    auto flush = [&] {  // (a thread's own words)
#pragma unroll
      for (int e = 0; e < EV; ++e) {
        sm.sum[0][e][et] += sD[e];
        sm.sum[1][e][et] += sT[e];
        sD[e] = sT[e] = 0.f;
      }
    };
    // Pointers to this thread's elements: of the next tile to load, and of the
    // next tile of outputs, from the last tile down.
    const int tl = t0 + (ntile - 1) * TB;
    const int64_t tok0 = (int64_t)b * p.T + tl + i0;  // row of a contiguous array
    const IO* pu = (const IO*)p.u + (p.ru.at(b, 0) + c) + (int64_t)(tl + i0) * p.ru.ld;
    const IO* pdt = (const IO*)p.dt + (p.rdt.at(b, 0) + c) + (int64_t)(tl + i0) * p.rdt.ld;
    const IO* pdy = (const IO*)p.dy + tok0 * p.D + c;
    const IO* pz = (const IO*)p.z + (p.rz.at(b, 0) + c) + (int64_t)(tl + i0) * p.rz.ld;
    const IO *pb[BN], *pc[BN];
    int nbn[BN];
#pragma unroll
    for (int j = 0; j < BN; ++j) {
      const int v = et + j * NE, n0 = v % (L / 2) * 4;
      nbn[j] = v < BV ? p.N - n0 : 0;
      pb[j] = (const IO*)p.Bm + (p.rb.at(b, 0) + g * p.N + n0) + (int64_t)(tl + v / (L / 2)) * p.rb.ld;
      pc[j] = (const IO*)p.Cm + (p.rc.at(b, 0) + g * p.N + n0) + (int64_t)(tl + v / (L / 2)) * p.rc.ld;
    }
    // a saved state: 4 of them, those of the scan thread of the same number
    f2 ck[2] = {0, 0};
    const int ckc = c0 + et / L * 2, ckn = et % L * 2;
    const bool ck0 = !END && ckc < cmax && ckn < p.N, ck1 = !END && ckc + 1 < cmax && ckn < p.N;
    const size_t nck = (p.T + kCk - 1) / kCk;
    const float* pck = p.states + ((b * nck + tl / kCk) * p.D + ckc) * p.N + ckn;
    int64_t out = tok0 * p.D + c;
    // dB, dC: vectors of 4 of a token's [2][N], added over the warps
    constexpr int SV = TB * L, SN = (SV + NE - 1) / NE;
    const int sn = et % (L / 2) * 4, sm_ = et % L / (L / 2), si = et / L;
    const int64_t srow = (int64_t)p.G * 2 * p.N;
    float* pbc = p.bc + (((int64_t)ct * p.B + b) * p.T + tl + si) * srow + (int64_t)(g * 2 + sm_) * p.N + sn;

    // Only tile 0 of the walk, the sequence's last, can have tokens behind the
    // end.
    auto load = [&](int k) {
#pragma unroll
      for (int s = 0; s < PASS; ++s) {
        const int i = i0 + s * IS;
        const int n = i < TB && (k > 0 || tl + i < te) ? nc : 0;
        nx[s].dt.load(pdt + s * IS * p.rdt.ld, n, p.vec);
        nx[s].dy.load(pdy + (int64_t)s * IS * p.D, n, p.vec);
        if (p.z) nx[s].z.load(pz + s * IS * p.rz.ld, n, p.vec);
        if (!END) nx[s].u.load(pu + s * IS * p.ru.ld, n, p.vec);
      }
      pdt -= TB * p.rdt.ld;
      pdy -= (int64_t)TB * p.D;
      pz -= TB * p.rz.ld;
      pu -= TB * p.ru.ld;
#pragma unroll
      for (int j = 0; j < BN; ++j) {
        const int n = k > 0 || tl + (et + j * NE) / (L / 2) < te ? nbn[j] : 0;
        ncv[j].load(pc[j], n, p.vecbc);
        if (!END) nb[j].load(pb[j], n, p.vecbc);
        pc[j] -= TB * p.rc.ld;
        pb[j] -= TB * p.rb.ld;
      }
      if (!END) load_state(pck, p.N, ck0, ck1, ck);
      pck -= (int64_t)p.D * p.N;
    };
    auto prepare = [&](int k, Tok (&tok)[PASS]) {
      if (!END) sm.ck[k & 1][et] = make_ulonglong2(ck[0], ck[1]);
#pragma unroll
      for (int s = 0; s < PASS; ++s) {
        const int i = i0 + s * IS;
        if (i >= TB) continue;
        const bool live = k > 0 || tl + i < te;
        Tok& x = tok[s];
#pragma unroll
        for (int e = 0; e < EV; ++e) {
          x.delta[e] = nx[s].dt.get(e) + bias[e];
          x.e[e] = nx[s].dy.get(e);
          x.u[e] = END ? 0.f : nx[s].u.get(e);
        }
        if (p.softplus) {
#pragma unroll
          for (int e = 0; e < EV; ++e) x.delta[e] = softplus(x.delta[e], x.sg[e]);
        } else {
#pragma unroll
          for (int e = 0; e < EV; ++e) x.sg[e] = 1.f;
        }
        if (p.z) {
#pragma unroll
          for (int e = 0; e < EV; ++e) {
            const float z = nx[s].z.get(e), sz = sigmoid(z), zs = z * sz;
            x.dzf[e] = x.e[e] * fmaf(-zs, sz, sz + zs);
            x.e[e] *= zs;
          }
        }
        // behind the sequence's end e = u = 0, and delta is made 0 (a channel
        // that is not there only needs e = u = 0)
#pragma unroll
        for (int e = 0; e < EV; ++e) x.delta[e] = live ? x.delta[e] : 0.f;
#pragma unroll
        for (int e = 0; e < EV; e += 2) {
          const int at = i * G::DS + (cl + e) / 2;
          sm.q[k & 1][at] = make_float4(x.delta[e], x.delta[e + 1], x.delta[e] * x.u[e], x.delta[e + 1] * x.u[e + 1]);
          sm.qe[k & 1][at] = make_float2(x.e[e], x.e[e + 1]);
        }
      }
#pragma unroll
      for (int j = 0; j < BN; ++j) {
        const int v = et + j * NE;
        if (v < BV) {
          ncv[j].put(&sm.cf[k & 1][v * 4]);
          if (!END) nb[j].put(&sm.bf[k & 1][v * 4]);
        }
      }
    };
    auto finish = [&](int k, const Tok (&tok)[PASS]) {
      const int w = k & 1;
#pragma unroll
      for (int s = 0; s < PASS; ++s) {
        const int i = i0 + s * IS;
        if (i >= TB || !(k > 0 || tl + i < te)) continue;
        float du[EV], dd[EV], dz[EV], gB[EV], gA[EV], yc[EV];
        load_f<EV>(&sm.gB[w][i * YS + cl], gB);
        load_f<EV>(&sm.gA[w][i * YS + cl], gA);
#pragma unroll
        for (int e = 0; e < EV; ++e) {
          du[e] = fmaf(tok[s].delta[e], gB[e], Ds[e] * tok[s].e[e]);
          dd[e] = fmaf(tok[s].u[e], gB[e], kLn2 * gA[e]) * tok[s].sg[e];
          sD[e] = fmaf(tok[s].e[e], tok[s].u[e], sD[e]);
          sT[e] += dd[e];
        }
        const int64_t at = out + (int64_t)s * IS * p.D;
        store_n<IO, EV>((IO*)p.du + at, du, nc, p.vec);
        store_n<IO, EV>((IO*)p.ddt + at, dd, nc, p.vec);
        if (p.dz) {
          load_f<EV>(&sm.yc[w][i * YS + cl], yc);
#pragma unroll
          for (int e = 0; e < EV; ++e) dz[e] = tok[s].dzf[e] * fmaf(Ds[e], tok[s].u[e], yc[e]);
          store_n<IO, EV>((IO*)p.dz + at, dz, nc, p.vec);
        }
      }
      out -= (int64_t)TB * p.D;
#pragma unroll
      for (int j = 0; j < SN; ++j) {
        const int i = si + j * (NE / L);
        if (et + j * NE < SV && sn < p.N && (k > 0 || tl + i < te)) {
          float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int x = 0; x < W; ++x) {
            const float4 r = *reinterpret_cast<const float4*>(&sm.red[w][x][i][sm_ * NP + sn]);
            s.x += r.x; s.y += r.y; s.z += r.z; s.w += r.w;
          }
          *reinterpret_cast<float4*>(pbc + j * (NE / L) * srow) = s;
        }
      }
      pbc -= TB * srow;
    };
    if (!END) {
      // behind the sequence's end: zeros
      const float zero[EV] = {};
      for (int t = max(t0, te) + i0; t < t1; t += IS) {
        const size_t at = ((size_t)b * p.T + t) * p.D + c;
        store_n<IO, EV>((IO*)p.du + at, zero, nc, p.vec);
        store_n<IO, EV>((IO*)p.ddt + at, zero, nc, p.vec);
        if (p.dz) store_n<IO, EV>((IO*)p.dz + at, zero, nc, p.vec);
      }
    }
    if (ntile > 0) {
      load(0);
      prepare(0, tok[0]);
      if (ntile > 1) load(1);
    }
    __syncthreads();
    // tile k - 1's outputs first: its registers then take tile k + 1
    auto step = [&](int k, Tok (&x)[PASS]) {
      if constexpr (!END)
        if (k > 0) finish(k - 1, x);
      if (k + 1 < ntile) prepare(k + 1, x);
      if (k + 2 < ntile) load(k + 2);
      __syncthreads();
    };
    for (int k = 0; k < ntile; k += 2) {
      step(k, tok[1]);
      if (k + 1 < ntile) step(k + 1, tok[0]);
      if constexpr (!END)
        if (many && k % kSum == kSum - 2) flush();
    }
    if constexpr (!END) {
      if (ntile > 0) {
        if (ntile & 1) finish(ntile - 1, tok[0]);
        else finish(ntile - 1, tok[1]);
      }
      if (many) {
#pragma unroll
        for (int e = 0; e < EV; ++e) {
          sD[e] += sm.sum[0][e][et];
          sT[e] += sm.sum[1][e][et];
        }
      }
      // sums of e u and ddt over the block's token rows, in order
      float* s1 = &sm.red[0][0][0][0];
      float* s2 = &sm.gB[0][0];
      static_assert(IS * CH <= 2 * W * TB * 2 * NP && IS * CH <= 2 * TB * YS, "room for the sums");
      asm volatile("bar.sync 1, %0;" ::"n"(NE) : "memory");
#pragma unroll
      for (int e = 0; e < EV; ++e) {
        s1[i0 * CH + cl + e] = sD[e];
        s2[i0 * CH + cl + e] = sT[e];
      }
      asm volatile("bar.sync 1, %0;" ::"n"(NE) : "memory");
      for (int x = et; x < CH; x += NE)
        if (c0 + x < cmax) {
          float u = 0.f, v = 0.f;
          for (int k = 0; k < IS && k < TB; ++k) {
            u += s1[k * CH + x];
            v += s2[k * CH + x];
          }
          part[(size_t)p.D * p.N + c0 + x] = u;
          part[(size_t)p.D * (p.N + 1) + c0 + x] = v;
        }
    }
    return;
  }

  // ---- scan warps
  const int lane = tid % 32, warp = tid / 32;
  const int cl = tid / L * 2, l = tid % L, c = c0 + cl;  // this thread's first channel and its lane
  const int n0 = 2 * l;
  const bool on0 = c < cmax && n0 < p.N, on1 = c + 1 < cmax && n0 < p.N;
  const size_t sidx = ((size_t)b * p.D + c) * p.N + n0;
  const size_t sstep = (size_t)p.B * p.D * p.N;
  f2 A2[2], gr[2] = {0, 0}, dA[2] = {0, 0}, dAt[2] = {0, 0}, sumd = 0;
  load_state(p.A + (size_t)c * p.N + n0, p.N, on0, on1, A2);
  A2[0] = mul2(A2[0], pk(kLog2e, kLog2e));
  A2[1] = mul2(A2[1], pk(kLog2e, kLog2e));
  if (!END) {
    if (p.dhT) load_state(p.dhT + sidx, p.N, on0, on1, gr);
#pragma unroll 4
    for (int s = p.nseg - 1; s > seg; --s) {
      f2 x[2];
      load_state(p.segE + s * sstep + sidx, p.N, on0, on1, x);
      const float* sd = p.segD + ((size_t)s * p.B + b) * p.D + c;
      const f2 d = pk(on0 ? sd[0] : 0.f, on1 ? sd[1] : 0.f);
      gr[0] = carry(A2[0], d, gr[0], x[0]);
      gr[1] = carry(A2[1], d, gr[1], x[1]);
    }
  }
  __syncthreads();
  for (int k = 0; k < ntile; ++k) {
    const int w = k & 1;
    const float4* q = sm.q[w] + cl / 2;
    const float2* qe = sm.qe[w] + cl / 2;
    const IO* bf = sm.bf[w] + n0;
    const IO* cf = sm.cf[w] + n0;
    if constexpr (END) {
#pragma unroll
      for (int i = TB - 1; i >= 0; --i) {
        const f2 d = *reinterpret_cast<const f2*>(&q[i * G::DS]), e = *reinterpret_cast<const f2*>(&qe[i * G::DS]);
        f2 C0, C1;
        load_bc(cf + i * NP, C0, C1);
        gr[0] = mul2(fma2(e, C0, gr[0]), decay(A2[0], d));
        gr[1] = mul2(fma2(e, C1, gr[1]), decay(A2[1], d));
        sumd = add2(sumd, d);
      }
    } else {
      walk_tile<IO, L, W>(p.dz != nullptr, sm.ck[w][tid], q, qe, bf, cf, sm.gB[w] + cl, sm.gA[w] + cl, sm.yc[w] + cl,
                       &sm.red[w][warp][0][0] + n0, A2, gr, dAt, lane, l);
      if (k % kSum == kSum - 1) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          dA[x] = add2(dA[x], dAt[x]);
          dAt[x] = 0;
        }
      }
    }
    __syncthreads();
  }
  if (END) {
    store_state(p.segE + seg * sstep + sidx, p.N, on0, on1, gr);
    float* sd = p.segD + ((size_t)seg * p.B + b) * p.D + c;
    if (l == 0 && on0) sd[0] = lo(sumd);
    if (l == 0 && on1) sd[1] = hi(sumd);
    return;
  }
  dA[0] = add2(dA[0], dAt[0]);
  dA[1] = add2(dA[1], dAt[1]);
  if (p.dh0 && seg == 0) store_state(p.dh0 + sidx, p.N, on0, on1, gr);
  store_state(part + (size_t)c * p.N + n0, p.N, on0, on1, dA);
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

template <typename IO, int L, int W>
cudaError_t go(const ScanParams& p, cudaStream_t s) {
  const size_t smem = sizeof(Smem<IO, L, W>);
  cudaError_t e = cudaSuccess;
  if constexpr (W == 4) {  // (segments only come with such blocks)
    if (p.nseg > 1) {
      e = want_smem(scan_bwd_kernel<IO, L, W, true>, smem);
      if (e != cudaSuccess) return e;
      ScopedTiming tm("scan_bwd_ends", s);
      scan_bwd_kernel<IO, L, W, true><<<dim3(p.G * p.nct, p.B, p.nseg - 1), 64 * W, smem, s>>>(p);
      e = cudaGetLastError();
      if (e != cudaSuccess) return e;
    }
  }
  e = want_smem(scan_bwd_kernel<IO, L, W, false>, smem);
  if (e != cudaSuccess) return e;
  {
    ScopedTiming tm("scan_bwd", s);
    scan_bwd_kernel<IO, L, W, false><<<dim3(p.G * p.nct, p.B, p.nseg), 64 * W, smem, s>>>(p);
  }
  e = cudaGetLastError();
  const size_t n = (size_t)p.B * p.T * p.G * 2 * p.N;
  if (e != cudaSuccess || n == 0) return e;
  ScopedTiming tm("scan_bc_sum", s);
  scan_bc_kernel<IO><<<(unsigned)((n + 255) / 256), 256, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename IO>
cudaError_t go_any(const ScanParams& p, cudaStream_t s) {
  switch (states_of(p.N)) {
    case 4: return go<IO, 2, 4>(p, s);
    case 8: return go<IO, 4, 4>(p, s);
    case 16: return p.W == 7 ? go<IO, 8, 7>(p, s) : go<IO, 8, 4>(p, s);
    case 32: return p.W == 7 ? go<IO, 16, 7>(p, s) : go<IO, 16, 4>(p, s);
    case 64: return p.W == 7 ? go<IO, 32, 7>(p, s) : go<IO, 32, 4>(p, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace
}  // namespace scan

cudaError_t launch_scan_bwd(const scan::ScanParams& p, bool bf, cudaStream_t s) {
  return bf ? scan::go_any<bf16>(p, s) : scan::go_any<float>(p, s);
}

}  // namespace lz
