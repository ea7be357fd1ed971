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
//
// Measured, bf16, causal, 40 query heads on 8 key heads of 128: 8192 tokens 985
// us over rows (1046 TFLOP/s of the masked half's three products) and 1425 us
// over keys (964 TFLOP/s of its four); nine documents of 4096 tokens with
// capped scores 131 and 141 us, 16 us more for the sum of the pieces; 16 heads
// of 64, 4096 tokens 90 and 110 us.  The matrix cores are busy 53 % and 45 % of
// the time, LDS reads 36 % and 43 %, without bank conflicts, at 1.8 to 1.9 GHz
// under the power limit (a large library product: 68 % busy).
#include "attn_core.h"
#include "mhc_internal.h"

namespace mhc {

using namespace attn;

attn::DocMask doc_mask(const mhc_attn_desc& d);
bool attn_short(const mhc_attn_desc& d);

namespace {

constexpr int kRows = 128, kKeys = 64;   // dq: rows of a workgroup, keys of a tile
constexpr int kKeyRows = 128;            // dk, dv: keys of a workgroup
constexpr int kMaxPieces = 16;

struct BwdArgs {
  DocMask mask;
  ScoreMod mod;
  const void *q, *k, *v, *o, *dout;
  const float *slopes, *lse;
  const uint8_t* rest;  // [T][Hq][Dh] or null
  float* delta;  // [Hq][T]
  float* part;   // [pieces][dk, dv][T][Hk][Dh]
  void *dq, *dk, *dv;
  int Hq, Hk, fill, pieces;
  int64_t ldq, ldk, ldv, ldo, lddo, lddq, lddk, lddv;
};

// Score s (log 2 units) and the capping's derivative from a product x.
template <int IO, int MOD>
__device__ __forceinline__ void score(float x, float pre, ScoreMod mod, float slope2, float dist, float& s, float& dcap) {
  s = x * pre;
  dcap = 1.f;
  if constexpr ((MOD & kCapped) != 0) {
    const float t = cap_tanh<IO>(s);
    dcap = 1.f - t * t;
    s = mod.post() * t;
  }
  if constexpr ((MOD & kSloped) != 0) s = __builtin_fmaf(-slope2, fabsf(dist), s);
}

// The lane's row of the kernels over rows: q and dout fragments, δ and lse.
template <int IO, int DH>
struct BwdRow {
  Frag<IO> qf[DH / 16], gf[DH / 16];
  float delta, lse2;
  __device__ __forceinline__ void load(const BwdArgs& a, int i, int hq, int h, bool live) {
    delta = 0.f;
#pragma unroll
    for (int s = 0; s < DH / 16; ++s) {
      const int64_t at = (int64_t)hq * DH + 16 * s + 8 * h;
      if (i < a.mask.T) {
        qf[s] = load_frag<IO>(a.q, i * a.ldq + at);
        gf[s] = load_frag<IO>(a.dout, i * a.lddo + at);
        float ov[8], gv[8];
        load8<IO>(a.o, i * a.ldo + at, ov);
        load8<IO>(a.dout, i * a.lddo + at, gv);
        if constexpr (IO == kBF16)
          if (a.rest != nullptr) add_rest(a.rest, (int64_t)i * a.Hq * DH + at, ov);
#pragma unroll
        for (int e = 0; e < 8; ++e) delta = __builtin_fmaf(ov[e], gv[e], delta);
      } else {
        qf[s] = gf[s] = zero_frag<IO>();
      }
    }
    delta += other_half(delta);
    lse2 = live ? a.lse[(int64_t)hq * a.mask.T + i] * kLog2e : 0.f;
    settle(qf);
    settle(gf);
    asm volatile("" : "+v"(lse2), "+v"(delta));
  }
};

// dq^T += K^T·dS^T of KB blocks of 32 keys from key0 on (`tk`, the values kTile
// bytes further), masked to the lane's keys [lo, hi) where `partial`.  `rest`
// adds up P (dP - δ), which over all keys is what δ, formed from o, is short of
// Σ P·dP: o carries the roundings of the forward's probabilities.  bf16: dS of
// masked tiles goes in to twice the bits, as the forward's probabilities do.
template <int IO, int DH, int KB, int MOD, int TILE>
__device__ __forceinline__ void rows_step(f32x16_t (&acc)[DH / 32], float& rest, const BwdRow<IO, DH>& row, uint32_t tk, int key0, int lo,
                                          int hi, bool partial, int i, float slope2, ScoreMod mod) {
  using T = Tile<IO, DH>;
  const int lane = threadIdx.x & (kWave - 1), c = lane & 31, h = lane >> 5;
  const uint32_t ra = T::row_addr(tk, c, h), ca = T::col_addr(tk, lane);
  const float pre = mod.pre();
#pragma unroll
  for (int b = 0; b < KB; ++b) {
    f32x16_t s, dp;
#pragma unroll
    for (int r = 0; r < 16; ++r) s[r] = dp[r] = 0.f;
    each<DH / 16>([&](auto n) {
      s = mma(T::template row_frag<n>(ra, 32 * b * T::kRow), row.qf[n], s);
      dp = mma(T::template row_frag<n>(ra, TILE + 32 * b * T::kRow), row.gf[n], dp);
    });
    const float d0 = (float)(i - key0 - 32 * b - 4 * h);
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int k = 8 * (r >> 2) + (r & 3);
      float sc, dcap = 1.f;
      if constexpr (MOD != 0)
        score<IO, MOD>(s[r], pre, mod, slope2, d0 - (float)k, sc, dcap);
      else
        sc = s[r] * pre;
      s[r] = exp2_fast(sc - row.lse2) * (dp[r] - row.delta);
      dp[r] = dcap;
    }
    if (partial) {
      int l0 = lo - key0 - 32 * b - 4 * h, h0 = hi - key0 - 32 * b - 4 * h;
      keep_branch(l0, h0);
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int k = 8 * (r >> 2) + (r & 3);
        s[r] = k >= l0 && k < h0 ? s[r] : 0.f;
      }
    }
    float sum = 0.f;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      sum += s[r];
      if constexpr ((MOD & kCapped) != 0) s[r] *= dp[r];
    }
    rest += sum;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const Frag<IO> ds = frag_of<IO>(s, n);
      each<DH / 32>([&](auto d) { acc[d] = mma(T::template col_frag<d>(ca, (32 * b + 16 * n) * T::kRow), ds, acc[d]); });
    }
    if constexpr (IO == kBF16)
      if (partial)
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const Frag<IO> ds = rest_frag(s, n);
          each<DH / 32>([&](auto d) { acc[d] = mma(T::template col_frag<d>(ca, (32 * b + 16 * n) * T::kRow), ds, acc[d]); });
        }
  }
}

// Rows: 128 of one query head a workgroup, 32 a wave; key and value tiles of 64.
template <int IO, int DH, int MOD>
__global__ __launch_bounds__(kThreads, IO == kBF16 ? 2 : 1) void attn_bwd_rows_kernel(BwdArgs a) {
  using T = Tile<IO, DH>;
  constexpr int kTile = kKeys * T::kRow;
  extern __shared__ __attribute__((aligned(512))) char lds[];
  __shared__ int range[8];
  const int lane = threadIdx.x & (kWave - 1), wave = wave_id(), c = lane & 31, h = lane >> 5;
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

  BwdRow<IO, DH> row;
  row.load(a, i, hq, h, live);

  const char* kb = static_cast<const char*>(a.k) + (int64_t)hk * DH * T::kElem;
  const char* vb = static_cast<const char*>(a.v) + (int64_t)hk * DH * T::kElem;
  Stage<IO, DH, kKeys> sk, sv;
  const float slope2 = (MOD & kSloped) != 0 ? a.slopes[hq] * kLog2e : 0.f;
  float rest = 0.f;
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
    rows_step<IO, DH, kKeys / 32, MOD, kTile>(acc, rest, row, lds_addr(tk), key0, lo, hi, partial, i, slope2, a.mod);
  }
  rest += other_half(rest);
  if (i < a.mask.T && h == 0) a.delta[(int64_t)hq * a.mask.T + i] = live ? row.delta + rest : 0.f;
  if (i >= a.mask.T || (!in_doc && !a.fill)) return;
#pragma unroll
  for (int b = 0; b < DH / 32; ++b) {
    if (!live)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[b][r] = 0.f;
    store_block<IO>(a.dq, i * a.lddq + (int64_t)hq * DH, b, h, acc[b], a.mod.scale);
  }
}

// The same for grids that would not fill the chip: 32 rows a workgroup, held by
// all four waves, which take the key tiles of 32 in turn, each through LDS of
// its own, and add up their sums at the end (fp32, 777 tokens, 8 query heads on
// 2 key heads of 64: 27 us instead of 73).  Not for bf16 heads of 128, where
// the registers do not hold it (8 heads, 2048 tokens: 84 us instead of 72).
template <int IO, int DH, int MOD>
__global__ __launch_bounds__(kThreads, IO == kBF16 ? 2 : 1) void attn_bwd_rows_short_kernel(BwdArgs a) {
  using T = Tile<IO, DH>;
  constexpr int kTile = 32 * T::kRow;
  extern __shared__ __attribute__((aligned(512))) char lds[];
  __shared__ float rests[4][32];
  const int lane = threadIdx.x & (kWave - 1), wave = wave_id(), c = lane & 31, h = lane >> 5;
  const int G = a.Hq / a.Hk;
  const int nt = (a.mask.T + 31) / 32;
  const int x = blockIdx.x % a.Hq, hk = x % a.Hk, hq = hk * G + x / a.Hk;
  const int i0 = (nt - 1 - (int)(blockIdx.x / a.Hq)) * 32, i = i0 + c;

  int ba, bb, lo, hi, wlo, whi;
  a.mask.bounds(i0, i0 + 31, ba, bb);
  const bool in_doc = a.mask.keys(i, ba, bb, lo, hi);
  wave_range(lo, hi, wlo, whi);
  const bool live = in_doc && lo < hi;
  BwdRow<IO, DH> row;
  row.load(a, i, hq, h, live);

  const char* kb = static_cast<const char*>(a.k) + (int64_t)hk * DH * T::kElem;
  const char* vb = static_cast<const char*>(a.v) + (int64_t)hk * DH * T::kElem;
  Stage<IO, DH, 32, kWave> sk, sv;
  const float slope2 = (MOD & kSloped) != 0 ? a.slopes[hq] * kLog2e : 0.f;
  float rest = 0.f;
  f32x16_t acc[DH / 32];
#pragma unroll
  for (int b = 0; b < DH / 32; ++b)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[b][r] = 0.f;
  char* tk = lds + wave * 2 * kTile;
  char* tv = tk + kTile;
  int key0 = wlo + wave * 32;
  if (key0 < whi) {
    sk.load(kb + key0 * a.ldk * T::kElem, a.ldk, whi - key0, lane);
    sv.load(vb + key0 * a.ldv * T::kElem, a.ldv, whi - key0, lane);
  }
  for (; key0 < whi; key0 += 128) {
    sk.store(tk, lane);
    sv.store(tv, lane);
    const int next = key0 + 128;
    if (next < whi) {
      sk.load(kb + next * a.ldk * T::kElem, a.ldk, whi - next, lane);
      sv.load(vb + next * a.ldv * T::kElem, a.ldv, whi - next, lane);
    }
    wave_lds_fence();
    const bool partial = __any(live && (lo > key0 || hi < key0 + 32));
    rows_step<IO, DH, 1, MOD, kTile>(acc, rest, row, lds_addr(tk), key0, lo, hi, partial, i, slope2, a.mod);
    wave_lds_fence();
  }
  if (!live) {
#pragma unroll
    for (int b = 0; b < DH / 32; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[b][r] = 0.f;
  }
  rest += other_half(rest);
  if (lane < 32) rests[wave][c] = rest;
  __syncthreads();  // (every wave is done with its tiles, too)
  if (i < a.mask.T && wave == 0 && h == 0)
    a.delta[(int64_t)hq * a.mask.T + i] = live ? row.delta + ((rests[0][c] + rests[1][c]) + (rests[2][c] + rests[3][c])) : 0.f;
  const f32x16_t sum = sum_waves<DH>(lds, wave, lane, acc, a.mod.scale);
  if (wave >= DH / 32 || i >= a.mask.T || (!in_doc && !a.fill)) return;
  store_block<IO>(a.dq, i * a.lddq + (int64_t)hq * DH, wave, h, sum, 1.f);
}

// Keys: 128 of one key head a workgroup, over the rows that see them, head by
// head of the group, in tiles of Q rows.  Scores here are S = Q·K^T with the
// keys as columns, so that P and dS are the B operands of dv^T = dO^T·P and
// dk^T = Q^T·dS.
//
// Eight waves: a pair for every 32 keys, on the same SIMD.  The first wave of
// a pair forms S and P and sums dv; the second forms dP, takes P from LDS one
// tile later and sums dk.  Each then holds one accumulator and one set of key
// fragments, which leaves room for two waves a SIMD, and the second does its
// vector work (dS of tile n - 1) while the first is at its products (S of tile
// n), and the other way round.  One barrier a tile: tile n is in use by the
// first waves while the second are at q of n - 1 and dout of n.
//
// The (head, row tile) steps of a key tile are cut into `pieces` for
// workgroups of their own where the key tiles are too few to fill the chip;
// each piece then leaves fp32 partial sums that attn_bwd_sum_kernel adds up in
// order.
constexpr int kKeyThreads = 512;

template <int IO, int DH, int MOD, int Q, bool SECOND>
__device__ __forceinline__ void keys_wave(const BwdArgs& a, char* lds, int* range,
                                          float (*stat)[2][Q], int pair, int lane, int thread) {
  using T = Tile<IO, DH>;
  constexpr int QB = Q / 32;
  constexpr int kTile = Q * T::kRow;
  const int c = lane & 31, h = lane >> 5;
  const int G = a.Hq / a.Hk;
  const int hk = blockIdx.x % a.Hk, piece = blockIdx.x / a.Hk % a.pieces, tile = blockIdx.x / a.Hk / a.pieces;
  const int j0 = tile * kKeyRows + pair * 32, j = j0 + c;

  int ba, bb, lo, hi, wlo, whi;
  a.mask.bounds(j0, j0 + 31, ba, bb);
  const bool in_doc = a.mask.rows(j, ba, bb, lo, hi);
  wave_range(lo, hi, wlo, whi);
  if (!SECOND && lane == 0) {
    range[pair] = whi > 0 ? wlo : 0x7fffffff;
    range[4 + pair] = whi;
  }
  Frag<IO> kf[DH / 16];  // keys, or the second wave's values
  {
    const void* p = SECOND ? a.v : a.k;
    const int64_t at = j * (SECOND ? a.ldv : a.ldk) + (int64_t)hk * DH + 8 * h;
#pragma unroll
    for (int s = 0; s < DH / 16; ++s) kf[s] = j < a.mask.T ? load_frag<IO>(p, at + 16 * s) : zero_frag<IO>();
    settle(kf);
  }
  __syncthreads();
  const int end = __builtin_amdgcn_readfirstlane(max(max(range[4], range[5]), max(range[6], range[7])));
  const int low = __builtin_amdgcn_readfirstlane(min(min(range[0], range[1]), min(range[2], range[3])));
  const int blo = end == 0 ? 0 : low;
  const bool live = in_doc && lo < hi;

  f32x16_t acc[DH / 32];  // dv, or the second wave's dk
#pragma unroll
  for (int b = 0; b < DH / 32; ++b)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[b][r] = 0.f;
  const float pre = a.mod.pre();

  // the first waves bring q and the rows' lse, the second dout and δ
  Stage<IO, DH, Q> stage;
  float s_stat = 0.f;
  const int64_t ld = SECOND ? a.lddo : a.ldq;
  const char* src = static_cast<const char*>(SECOND ? a.dout : a.q) + (int64_t)hk * G * DH * T::kElem;
  const float* stats = (SECOND ? a.delta : a.lse) + (int64_t)hk * G * a.mask.T;
  const int tiles = (end - blo + Q - 1) / Q, steps = tiles * G;
  const int per = (steps + a.pieces - 1) / a.pieces;
  const int first = min(piece * per, steps), last = min(first + per, steps);
  auto load = [&](int g, int row0) {
    stage.load(src + (row0 * ld + g * DH) * T::kElem, ld, end - row0, thread);
    if (thread < Q) s_stat = row0 + thread < end ? stats[(int64_t)g * a.mask.T + row0 + thread] : 0.f;
  };
  int g = first < last ? first / tiles : 0, row0 = blo + (first - g * tiles) * Q;  // the next tile's
  if (first < last) load(g, row0);
  const uint32_t base = lds_addr(lds);
  float* ps = reinterpret_cast<float*>(lds + 5 * kTile) + pair * QB * 16 * kWave + lane * 4;
  constexpr int kPs = 4 * QB * 16 * kWave;  // floats of one buffer of P
  f32x16_t s[QB];                           // S and P, or the second wave's dP and dS
  // LDS: three buffers of q (tile n is in use by the first waves while the second
  // still need tile n - 1), two of dout
  int cur = 0, prev = 0;  // q's buffers of tiles n and n - 1
  auto dout_at = [&](int n) { return 3 * kTile + (n & 1) * kTile; };
  // Tile n into its buffer, tile n + 1 on its way.
  auto arrive = [&](int n) {
    stage.store(lds + (SECOND ? dout_at(n) : cur * kTile), thread);
    if (thread < Q) stat[cur][SECOND ? 1 : 0][thread] = SECOND ? s_stat : s_stat * kLog2e;
    row0 += Q;
    if (row0 >= end) {
      row0 = blo;
      ++g;
    }
    if (n + 1 < last) load(g, row0);
    __syncthreads();
  };
  auto next = [&] {
    prev = cur;
    cur = cur == 2 ? 0 : cur + 1;
  };
  auto scores = [&](uint32_t ra) {
#pragma unroll
    for (int b = 0; b < QB; ++b) {
#pragma unroll
      for (int r = 0; r < 16; ++r) s[b][r] = 0.f;
      each<DH / 16>([&](auto m) { s[b] = mma(T::template row_frag<m>(ra, 32 * b * T::kRow), kf[m], s[b]); });
    }
  };
  auto sums = [&](uint32_t ca) {
#pragma unroll
    for (int b = 0; b < QB; ++b)
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const Frag<IO> p = frag_of<IO>(s[b], m);
        each<DH / 32>([&](auto d) { acc[d] = mma(T::template col_frag<d>(ca, (32 * b + 16 * m) * T::kRow), p, acc[d]); });
      }
  };
  if constexpr (!SECOND) {
    for (int n = first; n < last; ++n) {
      const int grow = g, r0 = row0, buf = cur;
      arrive(n);
      next();
      if (r0 >= whi || r0 + Q <= wlo) continue;  // (the pair's two waves alike)
      float* pw = ps + (n & 1) * kPs;
      const bool partial = __any(live && (lo > r0 || hi < r0 + Q));
      scores(T::row_addr(base + buf * kTile, c, h));
      const float slope2 = (MOD & kSloped) != 0 ? a.slopes[hk * G + grow] * kLog2e : 0.f;
      const float d0 = (float)(r0 + 4 * h - j);
#pragma unroll
      for (int b = 0; b < QB; ++b) {
        f32x16_t out;  // P, or P times the capping's derivative, for the second wave
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4) {
          const float4 lse = *reinterpret_cast<const float4*>(&stat[buf][0][32 * b + 8 * r4 + 4 * h]);
          const float lv[4] = {lse.x, lse.y, lse.z, lse.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = 4 * r4 + e;
            float sc, dcap = 1.f;
            if constexpr (MOD != 0)
              score<IO, MOD>(s[b][r], pre, a.mod, slope2, d0 + (float)(32 * b + 8 * r4 + e), sc, dcap);
            else
              sc = s[b][r] * pre;
            s[b][r] = exp2_fast(sc - lv[e]);
            if constexpr ((MOD & kCapped) != 0) out[r] = s[b][r] * dcap;
          }
        }
        if (partial) {
          int l0 = lo - r0 - 32 * b - 4 * h, h0 = hi - r0 - 32 * b - 4 * h;
          keep_branch(l0, h0);
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int k = 8 * (r >> 2) + (r & 3);
            const bool seen = k >= l0 && k < h0;
            s[b][r] = seen ? s[b][r] : 0.f;
            if constexpr ((MOD & kCapped) != 0) out[r] = seen ? out[r] : 0.f;
          }
        }
        if constexpr ((MOD & kCapped) == 0) out = s[b];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<float4*>(pw + (4 * b + i) * kWave * 4) =
              make_float4(out[4 * i], out[4 * i + 1], out[4 * i + 2], out[4 * i + 3]);
      }
      sums(T::col_addr(base + dout_at(n), lane));
    }
    __syncthreads();  // the second waves' last tile
  } else {
    // dS of the tile before, whose first row is rp and whose P lies in `pr`
    auto ds_of = [&](int rp, const float* pr) {
      const bool partial = __any(live && (lo > rp || hi < rp + Q));
#pragma unroll
      for (int b = 0; b < QB; ++b) {
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4) {
          const float4 del = *reinterpret_cast<const float4*>(&stat[prev][1][32 * b + 8 * r4 + 4 * h]);
          const float4 p = *reinterpret_cast<const float4*>(pr + (4 * b + r4) * kWave * 4);
          s[b][4 * r4] = p.x * (s[b][4 * r4] - del.x);
          s[b][4 * r4 + 1] = p.y * (s[b][4 * r4 + 1] - del.y);
          s[b][4 * r4 + 2] = p.z * (s[b][4 * r4 + 2] - del.z);
          s[b][4 * r4 + 3] = p.w * (s[b][4 * r4 + 3] - del.w);
        }
        if (partial) {  // (0 times what is not finite)
          int l0 = lo - rp - 32 * b - 4 * h, h0 = hi - rp - 32 * b - 4 * h;
          keep_branch(l0, h0);
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int k = 8 * (r >> 2) + (r & 3);
            s[b][r] = k >= l0 && k < h0 ? s[b][r] : 0.f;
          }
        }
      }
    };
    int rp = whi;  // (so that nothing is taken for the tile before the first)
    for (int n = first; n < last; ++n) {
      const int r0 = row0;
      arrive(n);
      if (rp < whi && rp + Q > wlo) {
        ds_of(rp, ps + (~n & 1) * kPs);
        sums(T::col_addr(base + prev * kTile, lane));
      }
      if (r0 < whi && r0 + Q > wlo) scores(T::row_addr(base + dout_at(n), c, h));
      rp = r0;
      next();
    }
    __syncthreads();
    if (rp < whi && rp + Q > wlo) {
      ds_of(rp, ps + (~last & 1) * kPs);
      sums(T::col_addr(base + prev * kTile, lane));
    }
  }
  if (j >= a.mask.T) return;
  if (!live) {
#pragma unroll
    for (int b = 0; b < DH / 32; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[b][r] = 0.f;
  }
  const float f = SECOND ? a.mod.scale : 1.f;
  if (a.pieces > 1) {
    const int64_t all = (int64_t)a.mask.T * a.Hk * DH, at = ((int64_t)j * a.Hk + hk) * DH;
#pragma unroll
    for (int b = 0; b < DH / 32; ++b) store_block<kF32>(a.part, (2 * piece + (SECOND ? 0 : 1)) * all + at, b, h, acc[b], f);
    return;
  }
  if (!in_doc && !a.fill) return;
  const int64_t at = j * (SECOND ? a.lddk : a.lddv) + (int64_t)hk * DH;
#pragma unroll
  for (int b = 0; b < DH / 32; ++b) store_block<IO>(SECOND ? a.dk : a.dv, at, b, h, acc[b], f);
}

template <int IO, int DH, int MOD, int Q>
__global__ __launch_bounds__(kKeyThreads, 2) void attn_bwd_keys_kernel(BwdArgs a) {
  // three buffers of a row tile's q and two of its dout, then two of each pair's P
  extern __shared__ __attribute__((aligned(512))) char lds[];
  __shared__ int range[8];
  __shared__ float stat[3][2][Q];  // [buffer][lse in log 2 units, δ][row]
  const int lane = threadIdx.x & (kWave - 1), wave = wave_id(), thread = threadIdx.x % kThreads;
  // The two kinds of wave run loops of their own (joined after each branch, the
  // accumulators were copied between registers every step); both pass the same
  // number of barriers.
  if (wave < 4)
    keys_wave<IO, DH, MOD, Q, false>(a, lds, range, stat, wave, lane, thread);
  else
    keys_wave<IO, DH, MOD, Q, true>(a, lds, range, stat, wave - 4, lane, thread);
}

// Adds up the pieces' partial sums: eight elements a thread, one key row of
// one of dk, dv a time.
template <int IO>
__global__ __launch_bounds__(kThreads) void attn_bwd_sum_kernel(BwdArgs a, int row) {
  const int j = blockIdx.x;
  if (!a.fill && a.mask.docs != nullptr) {
    int ba, bb, s, e, p;
    a.mask.bounds(j, j, ba, bb);
    if (!a.mask.doc(j, ba, bb, s, e, p)) return;
  }
  const int64_t all = (int64_t)a.mask.T * row;
  for (int t = threadIdx.x * 8; t < 2 * row; t += kThreads * 8) {
    const int which = t >= row ? 1 : 0, e = t - which * row;
    float sum[8], v[8];
    load8<kF32>(a.part, which * all + (int64_t)j * row + e, sum);
    for (int n = 1; n < a.pieces; ++n) {
      load8<kF32>(a.part, (2 * n + which) * all + (int64_t)j * row + e, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += v[i];
    }
    store8<IO>(which ? a.dv : a.dk, j * (which ? a.lddv : a.lddk) + e, sum);
  }
}

}  // namespace

static size_t delta_bytes(const mhc_attn_desc& d) { return ((size_t)d.Hq * (size_t)d.T * sizeof(float) + 255) / 256 * 256; }

// Rows of the keys kernel's tiles: 64, which fill a CU's LDS with one workgroup
// (bf16; fp32 takes 32), but 32 for heads of 64 on short documents, where three
// smaller workgroups a CU hide their short loops' ends better.  Measured, 64 and
// 32 rows: heads of 128, T = 8192 1.48 and 1.65 ms, documents of about 450 rows
// 142 and 161 us; heads of 64, one document of 4096 rows 110 and 120 us,
// documents of about 770 rows 47 and 40 us.
static bool tall_tiles(const mhc_attn_desc& d) {
  return d.io == MHC_BF16 && (d.Dh > 64 || d.T / (d.docs != nullptr ? d.n_docs : 1) >= 2048);
}

// Pieces of a key tile's steps: enough workgroups for two on every CU (fp32,
// 777 tokens, 8 query heads on 2 key heads of 64: 35 + 9 us for the sum instead
// of 366; bound by the latency of a workgroup's few steps).  Enough for one and
// for four: 4096 rows in nine uneven documents, 40 heads on 8 of 128, 266 and
// 150 + 25 us instead of 149 + 16; 2048 rows, the same heads, 164 + 10 and 128
// + 24 instead of 109 + 15 (sixteen equal documents of 256 rows would take 53
// instead of 65 + 16 with one, but lengths are not known here).
static int pieces_of(const mhc_attn_desc& d) {
  const int64_t base = (d.T + kKeyRows - 1) / kKeyRows * d.Hk;
  int64_t n = (2 * device_cu_count() + base - 1) / base;
  const int64_t steps = (d.T + 31) / 32 * (d.Hq / d.Hk);
  if (n > (steps + 3) / 4) n = (steps + 3) / 4;  // at least four steps each
  if (n > kMaxPieces) n = kMaxPieces;
  return n < 1 ? 1 : (int)n;
}

size_t attn_bwd_workspace_bytes(const mhc_attn_desc& d) {
  const int pieces = pieces_of(d);
  return delta_bytes(d) + (pieces > 1 ? (size_t)pieces * 2 * (size_t)d.T * d.Hk * d.Dh * sizeof(float) : 0);
}

hipError_t launch_attn_bwd(const mhc_attn_desc& d, const void* dout, const void* q, const void* k, const void* v,
                           const void* o, const float* lse, const void* o_rest, void* dq, void* dk, void* dv, void* ws,
                           hipStream_t s) {
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
  a.rest = static_cast<const uint8_t*>(o_rest);
  a.delta = static_cast<float*>(ws);
  a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + delta_bytes(d));
  a.pieces = pieces_of(d);
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
  const bool small = attn_short(d) && (d.io == MHC_F32 || d.Dh == 64);
  const int per = small ? 32 : kRows;
  const dim3 rows((unsigned)((d.T + per - 1) / per * d.Hq));
  const bool tall = tall_tiles(d);
  const dim3 keys((unsigned)((d.T + kKeyRows - 1) / kKeyRows * d.Hk * a.pieces));
  hipError_t err = hipErrorInvalidValue;
  dispatch_attn(d.io, d.Dh, d.softcap, d.slopes, [&](auto io_, auto dh_, auto mod_) {
    constexpr int IO = decltype(io_)::value;
    constexpr int DH = decltype(dh_)::value;
    constexpr int MOD = decltype(mod_)::value;
    constexpr int row = Tile<IO, DH>::kRow;
    [[maybe_unused]] constexpr int few = 8 * 32 * row > wave_states_bytes<DH>() ? 8 * 32 * row : wave_states_bytes<DH>();
    if constexpr (IO == kF32 || DH == 64)
      if (small) MHC_LAUNCH((attn_bwd_rows_short_kernel<IO, DH, MOD>), rows, dim3(kThreads), few, s, a);
    if (!small)
      MHC_LAUNCH((attn_bwd_rows_kernel<IO, DH, MOD>), rows, dim3(kThreads), 4 * kKeys * row, s, a);
    err = hipGetLastError();
    if (err != hipSuccess) return;
    [[maybe_unused]] constexpr int lds32 = 5 * 32 * row + 2 * 4 * 16 * kWave * 4, lds64 = 2 * lds32;
    if constexpr (IO == kBF16)
      if (tall) MHC_LAUNCH((attn_bwd_keys_kernel<IO, DH, MOD, 64>), keys, dim3(kKeyThreads), lds64, s, a);
    if constexpr (IO == kF32 || DH == 64)
      if (!tall) MHC_LAUNCH((attn_bwd_keys_kernel<IO, DH, MOD, 32>), keys, dim3(kKeyThreads), lds32, s, a);
    err = hipGetLastError();
    if (err != hipSuccess || a.pieces == 1) return;
    MHC_LAUNCH((attn_bwd_sum_kernel<IO>), dim3((unsigned)d.T), dim3(kThreads), 0, s, a, d.Hk * d.Dh);
    err = hipGetLastError();
  });
  return err;
}

}  // namespace mhc
