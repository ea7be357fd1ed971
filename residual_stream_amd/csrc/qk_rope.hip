// Per-head RMSNorm of queries and keys with the rotary position rotation in
// the same pass, forward and backward, and the serving form that writes the
// keys and values of new tokens into a paged cache.
//
// For one head row x[Dh] of a token at position p, with weight w and the
// frequencies f_i (radians per position, i < R/2):
//   u = w ⊙ x·r,  r = (mean_d x² + eps)^(-1/2)
//   y = u turned pair by pair: (a, b) → (a cos θ - b sin θ, a sin θ + b cos θ),
//       θ = p·f_i; the pair is (u[i], u[i + R/2]), or (u[2i], u[2i+1])
//       interleaved; elements from R on pass unturned.
// Backward, with g the gradient of y turned back by θ:
//   dw = Σ_rows g ⊙ x·r,   dx = r·(w ⊙ g - x·r²·mean_d(w ⊙ g ⊙ x)).
//
// A head row is spread over Dh/16 lanes (rounded up to a power of two), 16
// elements a lane chosen so that both members of every pair are in one lane:
// no exchange but the row's sum of squares.  The angle is formed in 64 bits
// as a fraction of a turn (p·f can be 10⁶ radians, where fp32 keeps no phase),
// once per token in LDS for all its heads.  Everything in between is fp32;
// each output is rounded once.
//
// Bound by HBM.  Measured, bf16, 4096 tokens of 40 and 8 heads of 128: forward
// 20 us, 101 MB at 5.0 TB/s (a plain copy reaches 5.2); backward 35 us, 151 MB
// at 4.3 TB/s (two row sums and the weights' products between a row's loads and
// its stores; loads rolled one row ahead made it 4 us slower), and 6 us to sum
// the weights' gradients.
#include "mhc_device.h"
#include "mhc_internal.h"

namespace mhc {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeTokens = 2;    // tokens a workgroup of the forward takes at most
constexpr int kMaxHalfR = 256;    // R/2 at most (Dh ≤ 512)

struct RopeArgs {
  int64_t T;
  int Hq, Hk, Dh, R, interleaved;
  float eps;
  int64_t ldq, ldk, ldv, ldqo, ldko, lddq, lddk;
  const void *q, *k, *v;
  const int32_t* pos;
  const double* freqs;
  const float *qw, *kw;
  void *qo, *ko, *vo;           // ko, vo: caches in the cache form
  const int64_t* slots;
  int64_t n_slots;
  const void *dqo, *dko;
  void *dq, *dk;
  float* part;                  // [workgroups][2][Dh] weight-gradient partials
};

// cos and sin of the tokens' angles into LDS, [token][R/2].
__device__ __forceinline__ void angles(const RopeArgs& a, int64_t t0, int nt, float2* cs) {
  const int h = a.R / 2;
  for (int n = threadIdx.x; n < nt * h; n += kRopeThreads) {
    const int t = n / h, i = n - t * h;
    double turn = (double)a.pos[t0 + t] * a.freqs[i] * 0.15915494309189533577;  // 1 / 2π
    turn -= rint(turn);
    float s, c;
    sincospif(2.0f * (float)turn, &s, &c);
    cs[n] = make_float2(c, s);
  }
}

// The first elements of a lane's two 8-element chunks.
__device__ __forceinline__ void chunks_of(const RopeArgs& a, int u, int& c0, int& c1) {
  if (!a.interleaved && u < a.R / 16) {
    c0 = 8 * u;
    c1 = 8 * u + a.R / 2;
  } else {
    c0 = 16 * u;
    c1 = 16 * u + 8;
  }
}

// Turns v (two chunks of eight) by the pairs' angles; `sign` -1 turns back.
__device__ __forceinline__ void turn(const RopeArgs& a, const float2* cs, int u, float sign, float v[16]) {
  if (u >= a.R / 16) return;
  if (a.interleaved) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 t = cs[8 * u + j];
      const float s = sign * t.y, x = v[2 * j], y = v[2 * j + 1];
      v[2 * j] = x * t.x - y * s;
      v[2 * j + 1] = x * s + y * t.x;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 t = cs[8 * u + j];
      const float s = sign * t.y, x = v[j], y = v[j + 8];
      v[j] = x * t.x - y * s;
      v[j + 8] = x * s + y * t.x;
    }
  }
}

// Sum over the L lanes of a head row (L a power of two, lanes aligned).
template <int L>
__device__ __forceinline__ float row_sum(float s) {
#pragma unroll
  for (int off = 1; off < L; off <<= 1) s += __shfl_xor(s, off, kWave);
  return s;
}

// Forward.  A workgroup takes up to kRopeTokens tokens; its lane groups of L
// walk their head rows (queries, then keys, then in the cache form the values,
// which are copied).
template <int IO, int L, bool CACHE>
__global__ __launch_bounds__(kRopeThreads) void qk_rope_kernel(RopeArgs a, int tokens) {
  __shared__ float2 cs[kRopeTokens * kMaxHalfR];
  const int64_t t0 = (int64_t)blockIdx.x * tokens;
  const int nt = (int)(a.T - t0 < tokens ? a.T - t0 : tokens);
  angles(a, t0, nt, cs);
  __syncthreads();
  const int u = threadIdx.x % L;
  const bool live = u < a.Dh / 16;
  const int heads = a.Hq + a.Hk * (CACHE ? 2 : 1);
  int c0, c1;
  chunks_of(a, live ? u : 0, c0, c1);
  for (int n = threadIdx.x / L; n < nt * heads; n += kRopeThreads / L) {
    const int tt = n / heads, head = n - tt * heads;
    const int64_t t = t0 + tt;
    const bool isq = head < a.Hq, isk = !isq && head < a.Hq + a.Hk;
    const int hh = isq ? head : isk ? head - a.Hq : head - a.Hq - a.Hk;
    int64_t slot = 0;
    if (CACHE && !isq) {
      slot = a.slots[t];
      if (slot < 0 || slot >= a.n_slots) continue;  // (the same for all lanes of the row)
    }
    const void* src = isq ? a.q : isk ? a.k : a.v;
    const int64_t so = t * (isq ? a.ldq : isk ? a.ldk : a.ldv) + (int64_t)hh * a.Dh;
    float x[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] = 0.f;
    if (live) {
      load8<IO>(src, so + c0, x);
      load8<IO>(src, so + c1, x + 8);
    }
    if (isq || isk) {
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < 16; ++j) ss = __builtin_fmaf(x[j], x[j], ss);
      const float r = 1.0f / sqrtf(row_sum<L>(ss) / (float)a.Dh + a.eps);
      const float* w = isq ? a.qw : a.kw;
      float wv[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) wv[j] = 1.f;
      if (w != nullptr && live) {
        load8<kF32>(w, c0, wv);
        load8<kF32>(w, c1, wv + 8);
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] = x[j] * r * wv[j];
      turn(a, cs + tt * (a.R / 2), u, 1.f, x);
    }
    if (live) {
      void* dst = isq ? a.qo : isk ? a.ko : a.vo;
      const int64_t d_o = isq ? t * a.ldqo + (int64_t)hh * a.Dh
                              : CACHE ? (slot * a.Hk + hh) * (int64_t)a.Dh : t * a.ldko + (int64_t)hh * a.Dh;
      store8<IO>(dst, d_o + c0, x);
      store8<IO>(dst, d_o + c1, x + 8);
    }
  }
}

// Backward.  Workgroups walk the tokens with the grid's stride, one or two at a
// time; each lane keeps the weight gradients of its 16 elements of q and of k
// over all its rows, summed over the lane groups at the end into one partial
// row per workgroup (fixed order, no atomics).
template <int IO, int L, int TOKENS>
__global__ __launch_bounds__(kRopeThreads) void qk_rope_bwd_kernel(RopeArgs a) {
  __shared__ float2 cs[TOKENS * kMaxHalfR];
  __shared__ float red[kRopeThreads * 16];
  const int u = threadIdx.x % L;
  const bool live = u < a.Dh / 16;
  const int heads = a.Hq + a.Hk;
  int c0, c1;
  chunks_of(a, live ? u : 0, c0, c1);
  float dwq[16], dwk[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) dwq[j] = dwk[j] = 0.f;
  for (int64_t t0 = (int64_t)blockIdx.x * TOKENS; t0 < a.T; t0 += (int64_t)gridDim.x * TOKENS) {
    const int nt = TOKENS > 1 && a.T - t0 > 1 ? 2 : 1;
    __syncthreads();  // the last tokens' angles have been read
    angles(a, t0, nt, cs);
    __syncthreads();
    for (int n = threadIdx.x / L; n < nt * heads; n += kRopeThreads / L) {
      const int tt = TOKENS > 1 && n >= heads ? 1 : 0, head = n - tt * heads;
      const int64_t t = t0 + tt;
      const bool isq = head < a.Hq;
      const int hh = isq ? head : head - a.Hq;
      const int64_t so = t * (isq ? a.ldq : a.ldk) + (int64_t)hh * a.Dh;
      const int64_t go = t * (isq ? a.ldqo : a.ldko) + (int64_t)hh * a.Dh;
      float x[16], g[16], wv[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] = g[j] = 0.f, wv[j] = 1.f;
      const float* w = isq ? a.qw : a.kw;
      if (live) {
        load8<IO>(isq ? a.q : a.k, so + c0, x);
        load8<IO>(isq ? a.q : a.k, so + c1, x + 8);
        load8<IO>(isq ? a.dqo : a.dko, go + c0, g);
        load8<IO>(isq ? a.dqo : a.dko, go + c1, g + 8);
        if (w != nullptr) {
          load8<kF32>(w, c0, wv);
          load8<kF32>(w, c1, wv + 8);
        }
      }
      turn(a, cs + tt * (a.R / 2), u, -1.f, g);
      float ss = 0.f, sg = 0.f;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        ss = __builtin_fmaf(x[j], x[j], ss);
        sg = __builtin_fmaf(g[j] * wv[j], x[j], sg);
      }
      const float r = 1.0f / sqrtf(row_sum<L>(ss) / (float)a.Dh + a.eps);
      const float m = row_sum<L>(sg) / (float)a.Dh * r * r;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float dw = g[j] * x[j] * r;
        if (isq)
          dwq[j] += dw;
        else
          dwk[j] += dw;
        x[j] = r * (g[j] * wv[j] - x[j] * m);
      }
      if (live) {
        const int64_t d_o = t * (isq ? a.lddq : a.lddk) + (int64_t)hh * a.Dh;
        store8<IO>(isq ? a.dq : a.dk, d_o + c0, x);
        store8<IO>(isq ? a.dq : a.dk, d_o + c1, x + 8);
      }
    }
  }
  if (a.part == nullptr) return;
  constexpr int G = kRopeThreads / L;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 16; ++j) red[j * kRopeThreads + threadIdx.x] = which ? dwk[j] : dwq[j];
    __syncthreads();
    for (int e = threadIdx.x; e < 16 * L; e += kRopeThreads) {
      const int j = e / L, uu = e - j * L;
      if (uu >= a.Dh / 16) continue;
      float s = 0.f;
      for (int gg = 0; gg < G; ++gg) s += red[j * kRopeThreads + gg * L + uu];
      int d0, d1;
      chunks_of(a, uu, d0, d1);
      a.part[((int64_t)blockIdx.x * 2 + which) * a.Dh + (j < 8 ? d0 + j : d1 + j - 8)] = s;
    }
  }
}

// Sum of the workgroups' partial rows: 16 columns a workgroup, 64 row slices
// (at 2048 partial rows 8 us, where 16 slices took 42; at 1024 6).
__global__ __launch_bounds__(1024) void qk_rope_dw_kernel(const float* __restrict__ part, int rows, int Dh,
                                                          float* __restrict__ dqw, float* __restrict__ dkw) {
  __shared__ float red[1024];
  const int c = blockIdx.x * 16 + threadIdx.x % 16, sl = threadIdx.x / 16;
  float s = 0.f;
#pragma unroll 8
  for (int r = sl; r < rows; r += 64) s += part[(int64_t)r * 2 * Dh + c];
  red[threadIdx.x] = s;
  for (int half = 32; half > 0; half >>= 1) {
    __syncthreads();
    if (sl < half) red[threadIdx.x] += red[threadIdx.x + half * 16];
  }
  if (sl == 0) {
    float* o = c < Dh ? dqw : dkw;
    if (o != nullptr) o[c < Dh ? c : c - Dh] = red[threadIdx.x];
  }
}

template <typename F>
void dispatch_lanes(int Dh, F&& f) {
  const int n = Dh / 16;
  if (n <= 1) f(std::integral_constant<int, 1>{});
  else if (n <= 2) f(std::integral_constant<int, 2>{});
  else if (n <= 4) f(std::integral_constant<int, 4>{});
  else if (n <= 8) f(std::integral_constant<int, 8>{});
  else if (n <= 16) f(std::integral_constant<int, 16>{});
  else f(std::integral_constant<int, 32>{});
}

RopeArgs args_of(const mhc_rope_desc& d) {
  RopeArgs a{};
  a.T = d.T;
  a.Hq = d.Hq;
  a.Hk = d.Hk;
  a.Dh = d.Dh;
  a.R = d.R;
  a.interleaved = d.interleaved;
  a.eps = d.eps;
  a.ldq = d.ldq;
  a.ldk = d.ldk;
  a.ldv = d.ldv;
  a.ldqo = d.ldq_out;
  a.ldko = d.ldk_out;
  a.lddq = d.ld_dq;
  a.lddk = d.ld_dk;
  return a;
}

// Two tokens a workgroup at a time where there are enough of them: at T = 4096
// the forward takes 19.7 instead of 20.6 us and the backward 35 instead of 38
// (48 heads leave half of 32 lane groups idle every other round, 96 none); at
// T = 8 the forward would take 8.9 instead of 6.6.
int tokens_of(const mhc_rope_desc& d) { return d.T >= 4096 ? kRopeTokens : 1; }
int bwd_workgroups(const mhc_rope_desc& d) { return (int)(d.T < 1024 ? d.T : 1024); }

}  // namespace

hipError_t launch_qk_rope(const mhc_rope_desc& d, const void* q, const void* k, const void* v, const int32_t* pos,
                          const double* freqs, const float* qw, const float* kw, void* qo, void* ko, void* vo,
                          const int64_t* slots, int64_t n_slots, hipStream_t s) {
  RopeArgs a = args_of(d);
  a.q = q;
  a.k = k;
  a.v = v;
  a.pos = pos;
  a.freqs = freqs;
  a.qw = qw;
  a.kw = kw;
  a.qo = qo;
  a.ko = ko;
  a.vo = vo;
  a.slots = slots;
  a.n_slots = n_slots;
  const int tokens = tokens_of(d);
  const dim3 grid((unsigned)((d.T + tokens - 1) / tokens));
  dispatch_io(d.io, [&](auto io_) {
    dispatch_lanes(d.Dh, [&](auto l_) {
      constexpr int IO = decltype(io_)::value;
      constexpr int L = decltype(l_)::value;
      if (slots != nullptr)
        MHC_LAUNCH((qk_rope_kernel<IO, L, true>), grid, dim3(kRopeThreads), 0, s, a, tokens);
      else
        MHC_LAUNCH((qk_rope_kernel<IO, L, false>), grid, dim3(kRopeThreads), 0, s, a, tokens);
    });
  });
  return hipGetLastError();
}

size_t qk_rope_bwd_workspace_bytes(const mhc_rope_desc& d) {
  return (size_t)bwd_workgroups(d) * 2 * d.Dh * sizeof(float);
}

hipError_t launch_qk_rope_bwd(const mhc_rope_desc& d, const void* dqo, const void* dko, const void* q, const void* k,
                              const int32_t* pos, const double* freqs, const float* qw, const float* kw, void* dq,
                              void* dk, float* dqw, float* dkw, void* ws, hipStream_t s) {
  RopeArgs a = args_of(d);
  a.q = q;
  a.k = k;
  a.pos = pos;
  a.freqs = freqs;
  a.qw = qw;
  a.kw = kw;
  a.dqo = dqo;
  a.dko = dko;
  a.dq = dq;
  a.dk = dk;
  const bool weights = dqw != nullptr || dkw != nullptr;
  a.part = weights ? static_cast<float*>(ws) : nullptr;
  const int nwg = bwd_workgroups(d);
  dispatch_io(d.io, [&](auto io_) {
    dispatch_lanes(d.Dh, [&](auto l_) {
      constexpr int IO = decltype(io_)::value;
      constexpr int L = decltype(l_)::value;
      if (tokens_of(d) > 1)
        MHC_LAUNCH((qk_rope_bwd_kernel<IO, L, 2>), dim3((unsigned)nwg), dim3(kRopeThreads), 0, s, a);
      else
        MHC_LAUNCH((qk_rope_bwd_kernel<IO, L, 1>), dim3((unsigned)nwg), dim3(kRopeThreads), 0, s, a);
    });
  });
  if (weights) MHC_LAUNCH(qk_rope_dw_kernel, dim3((unsigned)(2 * d.Dh / 16)), dim3(1024), 0, s, a.part, nwg, d.Dh, dqw, dkw);
  return hipGetLastError();
}

}  // namespace mhc
