// Masked attention over packed documents, backward (formulas and masks as in
// the forward).  With P_ij = exp(s_ij - lse_i), recomputed from q and k:
//   δ_i  = do_i·o_i,           dP_ij = do_i·v_j,
//   dS_ij = P_ij (dP_ij - δ_i)·(1 - (cap part of s_ij / cap)²)
//   dq_i = scale Σ_j dS_ij k_j,  dk_j = scale Σ_i dS_ij q_i,  dv_j = Σ_i P_ij do_i,
// dk and dv summed over the query heads that share the key head.
//
// Two kernels, each owning what it sums, so that no atomics are needed and the
// results are the same bits every time: one over rows (dq, and δ for the
// other), one over keys (dk, dv).  The scores are formed in both, seven
// products instead of five.  P and dS are rounded to the I/O type for the
// matrix cores; sums, δ and lse are fp32.
#include "attn_core.h"
#include "mhc_internal.h"

namespace mhc {

using namespace attn;

attn::DocMask doc_mask(const mhc_attn_desc& d);

namespace {

constexpr int kRows = 128, kKeys = 64;   // dq: rows of a workgroup, keys of a tile
constexpr int kKeyRows = 128, kQ = 64;   // dk, dv: keys of a workgroup, rows of a tile

struct BwdArgs {
  DocMask mask;
  ScoreMod mod;
  const void *q, *k, *v, *o, *dout;
  const float *slopes, *lse;
  float* delta;  // [Hq][T]
  void *dq, *dk, *dv;
  int Hq, Hk, fill;
  int64_t ldq, ldk, ldv, ldo, lddo, lddq, lddk, lddv;
};

// Score s (log 2 units) and the capping's derivative from a product x.
template <int IO>
__device__ __forceinline__ void score(float x, float pre, ScoreMod mod, float slope2, float dist, float& s, float& dcap) {
  s = x * pre;
  dcap = 1.f;
  if (mod.cap > 0.f) {
    const float t = cap_tanh<IO>(s);
    dcap = 1.f - t * t;
    s = mod.post() * t;
  }
  s = __builtin_fmaf(-slope2, fabsf(dist), s);
}

// Rows: 128 of one query head a workgroup, 32 a wave; key and value tiles of 64.
template <int IO, int DH, bool MOD>
__global__ __launch_bounds__(kThreads, IO == kBF16 ? 2 : 1) void attn_bwd_rows_kernel(BwdArgs a) {
  using T = Tile<IO, DH>;
  constexpr int kTile = kKeys * T::kRow;
  extern __shared__ __attribute__((aligned(256))) char lds[];
  __shared__ int range[8];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave, c = lane & 31, h = lane >> 5;
  const int G = a.Hq / a.Hk;
  const int nt = (a.mask.T + kRows - 1) / kRows;
  const int tile = nt - 1 - (int)(blockIdx.x / a.Hq), x = blockIdx.x % a.Hq;
  const int hk = x % a.Hk, hq = hk * G + x / a.Hk;
  const int i0 = tile * kRows + wave * 32, i = i0 + c;

  int ba, bb, lo, hi, wlo, whi;
  a.mask.bounds(i0, i0 + 31, ba, bb);
  const bool in_doc = a.mask.keys(i, ba, bb, lo, hi);
  wave_range(lo, hi, wlo, whi);
  if (lane == 0) {
    range[wave] = whi > 0 ? wlo : 0x7fffffff;
    range[4 + wave] = whi;
  }
  __syncthreads();
  int blo = min(min(range[0], range[1]), min(range[2], range[3]));
  const int bhi = max(max(range[4], range[5]), max(range[6], range[7]));
  if (bhi == 0) blo = 0;
  const bool live = in_doc && lo < hi;

  Frag<IO> qf[DH / 16], gf[DH / 16];
  float delta = 0.f;
#pragma unroll
  for (int s = 0; s < DH / 16; ++s) {
    const int64_t at = (int64_t)hq * DH + 16 * s + 8 * h;
    if (i < a.mask.T) {
      qf[s] = load_frag<IO>(a.q, i * a.ldq + at);
      gf[s] = load_frag<IO>(a.dout, i * a.lddo + at);
      float ov[8], gv[8];
      load8<IO>(a.o, i * a.ldo + at, ov);
      load8<IO>(a.dout, i * a.lddo + at, gv);
#pragma unroll
      for (int e = 0; e < 8; ++e) delta = __builtin_fmaf(ov[e], gv[e], delta);
    } else {
      qf[s] = gf[s] = zero_frag<IO>();
    }
  }
  delta += other_half(delta);
  float lse2 = 0.f;
  if (live) lse2 = a.lse[(int64_t)hq * a.mask.T + i] * kLog2e;
  if (i < a.mask.T && h == 0) a.delta[(int64_t)hq * a.mask.T + i] = live ? delta : 0.f;

  const char* kb = static_cast<const char*>(a.k) + (int64_t)hk * DH * T::kElem;
  const char* vb = static_cast<const char*>(a.v) + (int64_t)hk * DH * T::kElem;
  Stage<IO, DH, kKeys> sk, sv;
  const float slope2 = MOD && a.slopes != nullptr ? a.slopes[hq] * kLog2e : 0.f;
  const float pre = a.mod.pre();
  f32x16_t acc[DH / 32];
#pragma unroll
  for (int b = 0; b < DH / 32; ++b)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[b][r] = 0.f;
  sk.load(kb + blo * a.ldk * T::kElem, a.ldk, bhi - blo);
  sv.load(vb + blo * a.ldv * T::kElem, a.ldv, bhi - blo);
  int buf = 0;
  for (int key0 = blo; key0 < bhi; key0 += kKeys, buf ^= 1) {
    char* tk = lds + buf * 2 * kTile;
    char* tv = tk + kTile;
    sk.store(tk);
    sv.store(tv);
    const int next = key0 + kKeys;
    if (next < bhi) {
      sk.load(kb + next * a.ldk * T::kElem, a.ldk, bhi - next);
      sv.load(vb + next * a.ldv * T::kElem, a.ldv, bhi - next);
    }
    __syncthreads();
    if (key0 >= whi || next <= wlo) continue;
    const bool partial = __any(live && (lo > key0 || hi < next));
#pragma unroll
    for (int b = 0; b < kKeys / 32; ++b) {
      f32x16_t s, dp;
#pragma unroll
      for (int r = 0; r < 16; ++r) s[r] = dp[r] = 0.f;
#pragma unroll
      for (int n = 0; n < DH / 16; ++n) {
        s = mma(T::row_frag(tk, 32 * b + c, n, h), qf[n], s);
        dp = mma(T::row_frag(tv, 32 * b + c, n, h), gf[n], dp);
      }
      const int l0 = lo - key0 - 32 * b - 4 * h, h0 = hi - key0 - 32 * b - 4 * h;
      const float d0 = (float)(i - key0 - 32 * b - 4 * h);
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int k = 8 * (r >> 2) + (r & 3);
        float sc, dcap = 1.f;
        if constexpr (MOD)
          score<IO>(s[r], pre, a.mod, slope2, d0 - (float)k, sc, dcap);
        else
          sc = s[r] * pre;
        float ds = exp2_fast(sc - lse2) * (dp[r] - delta);
        if constexpr (MOD) ds *= dcap;
        if (partial) ds = k >= l0 && k < h0 ? ds : 0.f;
        s[r] = ds;
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const Frag<IO> ds = frag_of<IO>(s, n);
#pragma unroll
        for (int d = 0; d < DH / 32; ++d) acc[d] = mma(T::col_frag(tk, 32 * b + 16 * n, d, lane), ds, acc[d]);
      }
    }
  }
  if (i >= a.mask.T || (!in_doc && !a.fill)) return;
#pragma unroll
  for (int b = 0; b < DH / 32; ++b) {
    if (!live)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[b][r] = 0.f;
    store_block<IO>(a.dq, i * a.lddq + (int64_t)hq * DH, b, h, acc[b], a.mod.scale);
  }
}

// Keys: 128 of one key head a workgroup, 32 a wave (their key and value rows
// in registers), over the rows that see them, head by head of the group, in
// tiles of 64.  Scores here are S = Q·K^T with the wave's keys as columns.
template <int IO, int DH, bool MOD>
__global__ __launch_bounds__(kThreads, 1) void attn_bwd_keys_kernel(BwdArgs a) {
  using T = Tile<IO, DH>;
  constexpr int kTile = kQ * T::kRow;
  extern __shared__ __attribute__((aligned(256))) char lds[];
  __shared__ int range[8];
  __shared__ float stat[2][2][kQ];  // [buffer][lse in log 2 units, δ][row]
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave, c = lane & 31, h = lane >> 5;
  const int G = a.Hq / a.Hk;
  const int tile = blockIdx.x / a.Hk, hk = blockIdx.x % a.Hk;
  const int j0 = tile * kKeyRows + wave * 32, j = j0 + c;

  int ba, bb, lo, hi, wlo, whi;
  a.mask.bounds(j0, j0 + 31, ba, bb);
  const bool in_doc = a.mask.rows(j, ba, bb, lo, hi);
  wave_range(lo, hi, wlo, whi);
  if (lane == 0) {
    range[wave] = whi > 0 ? wlo : 0x7fffffff;
    range[4 + wave] = whi;
  }
  __syncthreads();
  int blo = min(min(range[0], range[1]), min(range[2], range[3]));
  const int bhi = max(max(range[4], range[5]), max(range[6], range[7]));
  if (bhi == 0) blo = 0;
  const bool live = in_doc && lo < hi;

  Frag<IO> kf[DH / 16], vf[DH / 16];
#pragma unroll
  for (int s = 0; s < DH / 16; ++s) {
    const int64_t at = (int64_t)hk * DH + 16 * s + 8 * h;
    kf[s] = j < a.mask.T ? load_frag<IO>(a.k, j * a.ldk + at) : zero_frag<IO>();
    vf[s] = j < a.mask.T ? load_frag<IO>(a.v, j * a.ldv + at) : zero_frag<IO>();
  }
  f32x16_t dk[DH / 32], dv[DH / 32];
#pragma unroll
  for (int b = 0; b < DH / 32; ++b)
#pragma unroll
    for (int r = 0; r < 16; ++r) dk[b][r] = dv[b][r] = 0.f;
  const float pre = a.mod.pre();

  Stage<IO, DH, kQ> sq, sg;
  float s_lse = 0.f, s_delta = 0.f;
  const int tiles = (bhi - blo + kQ - 1) / kQ, steps = tiles * G;
  auto load = [&](int n) {
    const int g = n / tiles, row0 = blo + (n - g * tiles) * kQ, hq = hk * G + g;
    const int64_t head = (int64_t)hq * DH * T::kElem;
    sq.load(static_cast<const char*>(a.q) + head + row0 * a.ldq * T::kElem, a.ldq, bhi - row0);
    sg.load(static_cast<const char*>(a.dout) + head + row0 * a.lddo * T::kElem, a.lddo, bhi - row0);
    if (threadIdx.x < kQ) {
      const int row = row0 + threadIdx.x;
      s_lse = row < bhi ? a.lse[(int64_t)hq * a.mask.T + row] * kLog2e : 0.f;
      s_delta = row < bhi ? a.delta[(int64_t)hq * a.mask.T + row] : 0.f;
    }
  };
  if (steps > 0) load(0);
  for (int n = 0; n < steps; ++n) {
    const int buf = n & 1, g = n / tiles, row0 = blo + (n - g * tiles) * kQ;
    char* tq = lds + buf * 2 * kTile;
    char* tg = tq + kTile;
    sq.store(tq);
    sg.store(tg);
    if (threadIdx.x < kQ) {
      stat[buf][0][threadIdx.x] = s_lse;
      stat[buf][1][threadIdx.x] = s_delta;
    }
    if (n + 1 < steps) load(n + 1);
    __syncthreads();
    if (row0 >= whi || row0 + kQ <= wlo) continue;
    const bool partial = __any(live && (lo > row0 || hi < row0 + kQ));
    const float slope2 = MOD && a.slopes != nullptr ? a.slopes[hk * G + g] * kLog2e : 0.f;
#pragma unroll
    for (int b = 0; b < kQ / 32; ++b) {
      f32x16_t s, dp;
#pragma unroll
      for (int r = 0; r < 16; ++r) s[r] = dp[r] = 0.f;
#pragma unroll
      for (int m = 0; m < DH / 16; ++m) {
        s = mma(T::row_frag(tq, 32 * b + c, m, h), kf[m], s);
        dp = mma(T::row_frag(tg, 32 * b + c, m, h), vf[m], dp);
      }
      const int l0 = lo - row0 - 32 * b - 4 * h, h0 = hi - row0 - 32 * b - 4 * h;
      const float d0 = (float)(row0 + 32 * b + 4 * h - j);
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4) {
        const float4 lse = *reinterpret_cast<const float4*>(&stat[buf][0][32 * b + 8 * r4 + 4 * h]);
        const float4 del = *reinterpret_cast<const float4*>(&stat[buf][1][32 * b + 8 * r4 + 4 * h]);
        const float lv[4] = {lse.x, lse.y, lse.z, lse.w}, dv4[4] = {del.x, del.y, del.z, del.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 4 * r4 + e, k = 8 * r4 + e;
          float sc, dcap = 1.f;
          if constexpr (MOD)
            score<IO>(s[r], pre, a.mod, slope2, d0 + (float)k, sc, dcap);
          else
            sc = s[r] * pre;
          float p = exp2_fast(sc - lv[e]);
          float ds = p * (dp[r] - dv4[e]);
          if constexpr (MOD) ds *= dcap;
          if (partial) {
            const bool seen = k >= l0 && k < h0;
            p = seen ? p : 0.f;
            ds = seen ? ds : 0.f;
          }
          s[r] = p;
          dp[r] = ds;
        }
      }
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const Frag<IO> p = frag_of<IO>(s, m), ds = frag_of<IO>(dp, m);
#pragma unroll
        for (int d = 0; d < DH / 32; ++d) {
          dv[d] = mma(T::col_frag(tg, 32 * b + 16 * m, d, lane), p, dv[d]);
          dk[d] = mma(T::col_frag(tq, 32 * b + 16 * m, d, lane), ds, dk[d]);
        }
      }
    }
  }
  if (j >= a.mask.T || (!in_doc && !a.fill)) return;
#pragma unroll
  for (int b = 0; b < DH / 32; ++b) {
    if (!live)
#pragma unroll
      for (int r = 0; r < 16; ++r) dk[b][r] = dv[b][r] = 0.f;
    store_block<IO>(a.dk, j * a.lddk + (int64_t)hk * DH, b, h, dk[b], a.mod.scale);
    store_block<IO>(a.dv, j * a.lddv + (int64_t)hk * DH, b, h, dv[b], 1.f);
  }
}

}  // namespace

size_t attn_bwd_workspace_bytes(const mhc_attn_desc& d) { return (size_t)d.Hq * (size_t)d.T * sizeof(float); }

hipError_t launch_attn_bwd(const mhc_attn_desc& d, const void* dout, const void* q, const void* k, const void* v,
                           const void* o, const float* lse, void* dq, void* dk, void* dv, void* ws, hipStream_t s) {
  BwdArgs a{};
  a.mask = doc_mask(d);
  a.mod = {d.scale, d.softcap};
  a.q = q;
  a.k = k;
  a.v = v;
  a.o = o;
  a.dout = dout;
  a.slopes = d.slopes;
  a.lse = lse;
  a.delta = static_cast<float*>(ws);
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.Hq = d.Hq;
  a.Hk = d.Hk;
  a.fill = d.fill_outside;
  a.ldq = d.ldq;
  a.ldk = d.ldk;
  a.ldv = d.ldv;
  a.ldo = d.ldo;
  a.lddo = d.ld_do;
  a.lddq = d.ld_dq;
  a.lddk = d.ld_dk;
  a.lddv = d.ld_dv;
  const dim3 rows((unsigned)((d.T + kRows - 1) / kRows * d.Hq));
  const dim3 keys((unsigned)((d.T + kKeyRows - 1) / kKeyRows * d.Hk));
  hipError_t err = hipErrorInvalidValue;
  dispatch_attn(d.io, d.Dh, d.softcap > 0.f || d.slopes != nullptr, [&](auto io_, auto dh_, auto mod_) {
    constexpr int IO = decltype(io_)::value;
    constexpr int DH = decltype(dh_)::value;
    constexpr bool MOD = decltype(mod_)::value;
    constexpr int lds = 4 * 64 * Tile<IO, DH>::kRow;
    static_assert(kKeys == 64 && kQ == 64, "tile bytes");
    MHC_LAUNCH((attn_bwd_rows_kernel<IO, DH, MOD>), rows, dim3(kThreads), lds, s, a);
    err = hipGetLastError();
    if (err != hipSuccess) return;
    MHC_LAUNCH((attn_bwd_keys_kernel<IO, DH, MOD>), keys, dim3(kThreads), lds, s, a);
    err = hipGetLastError();
  });
  return err;
}

}  // namespace mhc
