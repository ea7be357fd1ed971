// Masked attention over packed documents, forward.
//
// For query head h and row i of a packed batch of T tokens:
//   s_ij = cap·tanh(scale·q_i·k_j / cap) - slope_h·|i - j|   (each part optional)
//   o_i  = Σ_j p_ij v_j,  p_i = softmax of s_i over the keys j that row i sees,
//   lse_i = log Σ_j exp s_ij.
// Row i sees the keys of its own document, and with `causal` of those only
// j ≤ i (and i - j < window), or j in the document's prefix.  All these masks
// leave one run of keys [lo, hi) per row, so a tile of rows walks the union of
// its rows' runs and masks only the key tiles that some row sees in part.
//
// A workgroup takes 128 rows of one query head, 32 a wave, and walks the keys
// in tiles of 64, staged through registers into two LDS buffers (one barrier a
// tile).  One pass, with a running maximum and sum per row.  A wave's 32 rows
// hold 64 accumulator and 32 query registers at heads of 128: two waves share
// a SIMD, and one's softmax runs under the other's products.
//
// Measured, bf16, causal, 40 query heads on 8 key heads of 128: 8192 tokens
// 740 us, 930 TFLOP/s of the products that the mask leaves (a large library
// product reaches 1269); 4096 tokens 209 us; nine documents of 4096 tokens
// with capped scores 98 us; 16 heads of 64, 4096 tokens 71 us.  The matrix
// cores are busy 47 % of the time and the vector units about as long (half of
// it the exponentials, at a quarter of the rate), LDS reads 36 %, without bank
// conflicts; power holds the clock at 1.9 GHz.  A version whose eight waves
// took products and softmax strictly in turns needed 12 % fewer cycles and 2 %
// less time here, 5 to 15 % more time on the shorter cases.
#include "attn_core.h"
#include "mhc_internal.h"

namespace mhc {

using namespace attn;

namespace {

constexpr int kRows = 128, kKeys = 64;

struct FwdArgs {
  DocMask mask;
  ScoreMod mod;
  const void *q, *k, *v;
  const float* slopes;
  void* o;
  float* lse;     // [Hq][T] or null
  uint8_t* rest;  // [T][Hq][Dh] or null (bf16)
  int Hq, Hk, fill;
  int64_t ldq, ldk, ldv, ldo;
};

template <int IO, int DH, int MOD>
__global__ __launch_bounds__(kThreads, IO == kBF16 ? 2 : 1) void attn_fwd_kernel(FwdArgs a) {
  using T = Tile<IO, DH>;
  constexpr int kTile = kKeys * T::kRow;
  extern __shared__ __attribute__((aligned(512))) char lds[];  // two buffers of a key and a value tile
  __shared__ int range[16];
  __shared__ int not_finite;  // some value of a masked tile is not
  const int lane = threadIdx.x & (kWave - 1), wave = wave_id(), c = lane & 31, h = lane >> 5;
  // Tiles from the last (under a causal mask the longest) down; the heads of a
  // tile vary fastest, key head first: consecutive workgroups go to the eight
  // XCDs in turn, so with 8 key heads (or a divisor) each XCD's L2 holds one
  // head's keys and values.
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
  int ilo, ihi;
  common_range(lo, hi, ilo, ihi);
  if (lane == 0) {
    range[8 + wave] = ilo;
    range[12 + wave] = ihi;
  }
  if (threadIdx.x == 0) not_finite = 0;
  __syncthreads();
  ilo = max(max(range[8], range[9]), max(range[10], range[11]));
  ihi = min(min(range[12], range[13]), min(range[14], range[15]));
  int blo = min(min(range[0], range[1]), min(range[2], range[3]));
  const int bhi = max(max(range[4], range[5]), max(range[6], range[7]));
  if (bhi == 0) blo = 0;
  // rows of no document take no part: any key tile is whole for them
  const bool live = in_doc && lo < hi;

  Frag<IO> qf[DH / 16];
#pragma unroll
  for (int s = 0; s < DH / 16; ++s)
    qf[s] = i < a.mask.T ? load_frag<IO>(a.q, i * a.ldq + (int64_t)hq * DH + 16 * s + 8 * h) : zero_frag<IO>();

  const char* kb = static_cast<const char*>(a.k) + (int64_t)hk * DH * T::kElem;
  const char* vb = static_cast<const char*>(a.v) + (int64_t)hk * DH * T::kElem;
  Stage<IO, DH, kKeys> sk, sv;
  const float slope2 = (MOD & kSloped) != 0 ? a.slopes[hq] * kLog2e : 0.f;
  settle(qf);
  RowState<DH> st;
  st.init();
  // (rows past bhi read as zeros: no row of the tile sees them)
  sk.load(kb + blo * a.ldk * T::kElem, a.ldk, bhi - blo);
  sv.load(vb + blo * a.ldv * T::kElem, a.ldv, bhi - blo);
  int buf = 0;
  for (int key0 = blo; key0 < bhi; key0 += kKeys, buf ^= 1) {
    char* tk = lds + buf * 2 * kTile;
    char* tv = tk + kTile;
    const int next = key0 + kKeys;
    sk.store(tk);
    if (next < bhi) sk.load(kb + next * a.ldk * T::kElem, a.ldk, bhi - next);
    sv.store(tv);
    if ((key0 < ilo || next > ihi) && sv.store_finite(tv)) not_finite = 1;
    if (next < bhi) sv.load(vb + next * a.ldv * T::kElem, a.ldv, bhi - next);
    __syncthreads();
    if (key0 < whi && next > wlo) {
      const bool partial = __any(live && (lo > key0 || hi < next));
      attend<IO, DH, kKeys / 32, MOD>(st, qf, lds_addr(tk), lds_addr(tv), key0, lo, hi, partial, i, slope2, a.mod);
    }
  }
  if (__builtin_expect(not_finite, 0))
    for (int key0 = blo; key0 < bhi; key0 += kKeys)
      if (key0 < ilo || key0 + kKeys > ihi)
        add_not_finite<IO, DH>(st, max(lo, key0), min(hi, key0 + kKeys), h,
                               [&](int j) { return vb + j * a.ldv * T::kElem; });
  if (i >= a.mask.T || (!in_doc && !a.fill)) return;
  const float l = st.l + other_half(st.l);
  const float inv = !live || l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int b = 0; b < DH / 32; ++b) {
    if (!live)
#pragma unroll
      for (int r = 0; r < 16; ++r) st.o[b][r] = 0.f;
    store_block<IO>(a.o, i * a.ldo + (int64_t)hq * DH, b, h, st.o[b], inv);
    if constexpr (IO == kBF16)
      if (a.rest != nullptr) store_rest(a.rest, ((int64_t)i * a.Hq + hq) * DH, b, h, st.o[b], inv);
  }
  if (a.lse != nullptr && h == 0)
    a.lse[(int64_t)hq * a.mask.T + i] = live ? (st.m + __log2f(l)) * kLn2 : -__builtin_inff();
}

// The same for grids that would not fill the chip: 32 rows a workgroup, held by
// all four waves, which take the key tiles of 32 in turn, each through LDS of
// its own (no barrier in the loop), and join their row states at the end
// (fp32, 777 tokens, 8 query heads on 2 key heads of 64: 21 us instead of 53;
// bound by the latency of a workgroup's few steps).
template <int IO, int DH, int MOD>
__global__ __launch_bounds__(kThreads, IO == kBF16 ? 2 : 1) void attn_fwd_short_kernel(FwdArgs a) {
  using T = Tile<IO, DH>;
  constexpr int kTile = 32 * T::kRow;
  extern __shared__ __attribute__((aligned(512))) char lds[];  // a key and a value tile a wave; then the row states
  __shared__ float stat[256];
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

  Frag<IO> qf[DH / 16];
#pragma unroll
  for (int s = 0; s < DH / 16; ++s)
    qf[s] = i < a.mask.T ? load_frag<IO>(a.q, i * a.ldq + (int64_t)hq * DH + 16 * s + 8 * h) : zero_frag<IO>();
  const char* kb = static_cast<const char*>(a.k) + (int64_t)hk * DH * T::kElem;
  const char* vb = static_cast<const char*>(a.v) + (int64_t)hk * DH * T::kElem;
  Stage<IO, DH, 32, kWave> sk, sv;
  const float slope2 = (MOD & kSloped) != 0 ? a.slopes[hq] * kLog2e : 0.f;
  settle(qf);
  RowState<DH> st;
  st.init();
  char* tk = lds + wave * 2 * kTile;
  char* tv = tk + kTile;
  bool not_finite = false;
  int key0 = wlo + wave * 32;
  if (key0 < whi) {
    sk.load(kb + key0 * a.ldk * T::kElem, a.ldk, whi - key0, lane);
    sv.load(vb + key0 * a.ldv * T::kElem, a.ldv, whi - key0, lane);
  }
  for (; key0 < whi; key0 += 128) {
    const bool partial = __any(live && (lo > key0 || hi < key0 + 32));
    sk.store(tk, lane);
    sv.store(tv, lane);
    if (partial) not_finite |= sv.store_finite(tv, lane);
    const int next = key0 + 128;
    if (next < whi) {
      sk.load(kb + next * a.ldk * T::kElem, a.ldk, whi - next, lane);
      sv.load(vb + next * a.ldv * T::kElem, a.ldv, whi - next, lane);
    }
    wave_lds_fence();
    attend<IO, DH, 1, MOD>(st, qf, lds_addr(tk), lds_addr(tv), key0, lo, hi, partial, i, slope2, a.mod);
    wave_lds_fence();
  }
  if (__builtin_expect(__any(not_finite), 0))
    for (key0 = wlo + wave * 32; key0 < whi; key0 += 128)
      if (__any(live && (lo > key0 || hi < key0 + 32)))
        add_not_finite<IO, DH>(st, max(lo, key0), min(hi, key0 + 32), h, [&](int j) { return vb + j * a.ldv * T::kElem; });
  if (!live) st.init();
  float m, l;
  const f32x16_t sum = join_waves<DH>(lds, stat, wave, lane, st, m, l);
  if (wave >= DH / 32 || i >= a.mask.T || (!in_doc && !a.fill)) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  store_block<IO>(a.o, i * a.ldo + (int64_t)hq * DH, wave, h, sum, inv);
  if constexpr (IO == kBF16)
    if (a.rest != nullptr) store_rest(a.rest, ((int64_t)i * a.Hq + hq) * DH, wave, h, sum, inv);
  if (a.lse != nullptr && wave == 0 && h == 0)
    a.lse[(int64_t)hq * a.mask.T + i] = live ? (m + __log2f(l)) * kLn2 : -__builtin_inff();
}

}  // namespace

// Whether 128 rows a workgroup would leave the chip too empty: fewer workgroups
// than CUs, or than two a CU where documents are long (so that a workgroup is a
// long chain of steps) and the kernels of 32 rows hold their state in registers
// with room to spare (not bf16 heads of 128).  Measured, 128 and 32 rows, the
// forward and the backward's rows kernel, us: bf16, 16 heads of 64, 2309 rows
// 46 + 55 and 34 + 44; the same in documents of 100 rows 16.5 + 19 and 16.4 +
// 23; 4096 rows in 16 documents 17 + 23 and 24 + 35; fp32, 8 heads of 64, 4096
// rows 296 + 418 and 167 + 253; bf16, 40 heads of 128, 1024 rows 36 + 51 and 41
// + 82, but 8 heads of 128, 2048 rows 53 and 29 (forward).
bool attn_short(const mhc_attn_desc& d) {
  const bool roomy = d.io == MHC_F32 || d.Dh == 64;
  const bool chains = d.T / (d.docs != nullptr ? d.n_docs : 1) >= 512;
  return (d.T + kRows - 1) / kRows * d.Hq < (roomy && chains ? 2 : 1) * device_cu_count();
}

attn::DocMask doc_mask(const mhc_attn_desc& d) {
  attn::DocMask m;
  m.docs = d.docs;
  m.prefix = d.prefix;
  m.n_docs = d.docs != nullptr ? d.n_docs : 1;
  m.T = (int)d.T;
  m.causal = d.causal;
  m.window = d.window;
  return m;
}

hipError_t launch_attn(const mhc_attn_desc& d, const void* q, const void* k, const void* v, void* o, float* lse,
                       void* o_rest, hipStream_t s) {
  FwdArgs a{};
  a.mask = doc_mask(d);
  a.mod = {d.scale, d.softcap};
  a.q = q;
  a.k = k;
  a.v = v;
  a.slopes = d.slopes;
  a.o = o;
  a.lse = lse;
  a.rest = static_cast<uint8_t*>(o_rest);
  a.Hq = d.Hq;
  a.Hk = d.Hk;
  a.fill = d.fill_outside;
  a.ldq = d.ldq;
  a.ldk = d.ldk;
  a.ldv = d.ldv;
  a.ldo = d.ldo;
  const bool small = attn_short(d);
  const int rows = small ? 32 : kRows;
  const dim3 grid((unsigned)((d.T + rows - 1) / rows * d.Hq));
  hipError_t err = hipErrorInvalidValue;
  dispatch_attn(d.io, d.Dh, d.softcap, d.slopes, [&](auto io_, auto dh_, auto mod_) {
    constexpr int IO = decltype(io_)::value;
    constexpr int DH = decltype(dh_)::value;
    constexpr int MOD = decltype(mod_)::value;
    constexpr int row = Tile<IO, DH>::kRow;
    constexpr int few = 8 * 32 * row > wave_states_bytes<DH>() ? 8 * 32 * row : wave_states_bytes<DH>();
    if (small)
      MHC_LAUNCH((attn_fwd_short_kernel<IO, DH, MOD>), grid, dim3(kThreads), few, s, a);
    else
      MHC_LAUNCH((attn_fwd_kernel<IO, DH, MOD>), grid, dim3(kThreads), 4 * kKeys * row, s, a);
    err = hipGetLastError();
  });
  return err;
}

}  // namespace mhc
