// Attention of new tokens over a paged cache: single tokens or a chunk per
// sequence, keys and values read through each sequence's page table.
//
// Row t of sequence n is its q_len new tokens' c-th, at position
// p = kv_len - q_len + c; it sees the keys j ≤ p (and p - j < window), or
// j < prefix, of its sequence.  Scores as in the dense calls.
//
// The query heads that share a key head are packed into one tile of rows
// (row = c·G + g), so that the cache is read once for all of them.  Two
// kernels: up to 32 packed rows (single tokens, short drafts) go to four waves
// that take different keys, each with LDS of its own and no barrier in the
// loop; more rows go to the dense kernel's shape (128 rows, 32 a wave, over
// shared key tiles of 64).  Where there are few rows the keys are split over
// workgroups too; every split leaves a normalised partial row and its
// log-sum-exp, and a second kernel joins them.
//
// Table entries outside the cache are never followed: the rows whose keys they
// hold come out as NaN.
//
// Measured, bf16, 40 query heads on 8 key heads of 128.  64 sequences of up to
// 8192 keys, one new token each: 280 us, 1.34 GB at 4.8 TB/s (a plain copy
// reaches 5.2: bound by HBM) and 6 us for the join.  One token over 4099 keys:
// 11 + 6 us, where 3 would read the cache: launches and a chain of three loads.
// 20 heads on 4, three sequences' chunks of up to 700 tokens over up to 6000
// keys with distance slopes: 101 + 11 us, matrix cores busy 28 % of the time,
// the vector units, which have the slopes too, most of the rest.
#include "attn_core.h"
#include "mhc_internal.h"

namespace mhc {

using namespace attn;

namespace {

constexpr int kFewRows = 32, kFewKeys = 32;
constexpr int kRows = 128, kKeys = 64;
constexpr int kMaxSplits = 64;

// Division of 0 ≤ n < 2³¹ by a fixed d: with 2^(l-1) < d ≤ 2^l and
// mul = ⌈2^(31+l)/d⌉, n·mul/2^(31+l) exceeds n/d by less than 1/d.
struct Div {
  uint32_t d, mul, shift;
  __device__ __forceinline__ int operator()(int n) const {
    return d == 1 ? n : (int)(__umulhi((uint32_t)n, mul) >> shift);
  }
};
Div div_of(uint32_t d) {
  Div v{d, 0, 0};
  if (d < 2) return v;
  uint32_t l = 0;
  while ((1ull << l) < d) ++l;
  v.mul = (uint32_t)(((1ull << (31 + l)) + d - 1) / d);
  v.shift = l - 1;
  return v;
}

struct PagedArgs {
  int64_t T;
  int n, max_q, Hq, Hk, window, max_pages, num_pages, page_size, fill, splits, tiles;
  Div by_page, by_group;
  ScoreMod mod;
  const int32_t *cu, *prefix, *kv, *pages;
  const float* slopes;
  const void *q, *kc, *vc;
  void* o;
  float *part_o, *part_l;  // [splits][T][Hq][Dh], [splits][T][Hq]
  int64_t ldq, ldo;
};

// Sequence `s`: its first row, number of rows and number of keys, all within
// the tensors whatever the device arrays hold.
struct Seq {
  int64_t t0, t1;  // rows, of which the first nq are computed
  int nq, nk;
  int before;  // keys before the first new token's own (negative: rows without keys)
};
__device__ __forceinline__ int64_t clamp64(int64_t v, int64_t lo, int64_t hi) { return v < lo ? lo : v > hi ? hi : v; }
__device__ __forceinline__ Seq seq_of(const PagedArgs& a, int s) {
  Seq q;
  if (a.cu == nullptr) {
    q.t0 = s;
    q.t1 = s + 1;
  } else {
    q.t0 = clamp64(a.cu[s], 0, a.T);
    q.t1 = clamp64(a.cu[s + 1], q.t0, a.T);
  }
  q.nq = (int)(q.t1 - q.t0 < a.max_q ? q.t1 - q.t0 : a.max_q);
  q.nk = (int)clamp64(a.kv[s], 0, (int64_t)a.max_pages * a.page_size);
  q.before = (int)clamp64(q.nk - (q.t1 - q.t0), -(int64_t)0x7fffffff, q.nk);
  return q;
}

// The packed row's token, head and keys.
struct Row {
  bool real;
  int64_t at;   // (token, query head) as an index of [T][Hq]
  int64_t tok;
  int hq, pos, lo, hi;
};
__device__ __forceinline__ Row row_of(const PagedArgs& a, int s, const Seq& q, int hk, int pr) {
  const int G = a.Hq / a.Hk;
  Row r;
  const int c = a.by_group(pr), g = pr - c * G;
  r.real = c < q.nq;
  r.tok = q.t0 + c;
  r.hq = hk * G + g;
  r.at = r.tok * a.Hq + r.hq;
  r.pos = q.before + c;
  r.lo = 0;
  r.hi = min(q.nk, max(r.pos + 1, a.prefix != nullptr ? a.prefix[s] : 0));
  if (a.window > 0) r.lo = max(0, r.pos - a.window + 1);
  if (!r.real || r.hi <= r.lo) r.lo = r.hi = 0;
  return r;
}

// Staging of R cache rows by NT threads: as Stage, with each row's entry of
// the page table read one tile ahead of its load (and not looked at before, so
// that nothing waits for it).  Rows past `last` re-read it (they are masked).
template <int IO, int DH, int R, int NT>
struct PagedStage {
  using T = Tile<IO, DH>;
  static constexpr int kN = R * T::kChunks / NT;
  static constexpr int kStep = NT / T::kChunks;
  static_assert(R * T::kChunks % NT == 0 && NT % T::kChunks == 0, "whole passes");
  u32x4_t k[kN], v[kN];
  int64_t at[kN];
  int entry[kN];

  // Address of key r's value row, for a key whose page is in the cache.
  __device__ static __forceinline__ const char* value_row(const PagedArgs& a, const int32_t* table, int hk, int r) {
    const int p = a.by_page(r);
    int e = table[p];
    if ((unsigned)e >= (unsigned)a.num_pages) e = 0;  // (the rows come out as NaN)
    return static_cast<const char*>(a.vc) + (((int64_t)e * a.page_size + (r - p * a.page_size)) * a.Hk + hk) * T::kRow;
  }
  __device__ __forceinline__ void lookup(const PagedArgs& a, const int32_t* table, int thread, int row0, int last) {
#pragma unroll
    for (int n = 0; n < kN; ++n) entry[n] = table[a.by_page(min(row0 + thread / T::kChunks + n * kStep, last))];
  }
  __device__ __forceinline__ void load_k(const PagedArgs& a, int hk, int thread, int row0, int last, bool& bad) {
    const int64_t row = (int64_t)a.Hk * T::kRow;
    const int64_t in = (int64_t)hk * T::kRow + (thread % T::kChunks) * 16;
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      const int r = min(row0 + thread / T::kChunks + n * kStep, last);
      int e = entry[n];
      if ((unsigned)e >= (unsigned)a.num_pages) {
        bad = true;
        e = 0;
      }
      at[n] = (e * a.page_size + (r - a.by_page(r) * a.page_size)) * row + in;
    }
#pragma unroll
    for (int n = 0; n < kN; ++n) k[n] = *reinterpret_cast<const u32x4_t*>(static_cast<const char*>(a.kc) + at[n]);
  }
  __device__ __forceinline__ void load_v(const PagedArgs& a) {  // (after load_k: the same places)
#pragma unroll
    for (int n = 0; n < kN; ++n) v[n] = *reinterpret_cast<const u32x4_t*>(static_cast<const char*>(a.vc) + at[n]);
  }
  __device__ __forceinline__ void load(const PagedArgs& a, int hk, int thread, int row0, int last, bool& bad) {
    load_k(a, hk, thread, row0, last, bad);
    load_v(a);
  }
  __device__ static __forceinline__ void store(char* t, const u32x4_t (&w)[kN], int thread) {
#pragma unroll
    for (int n = 0; n < kN; ++n)
      *reinterpret_cast<u32x4_t*>(t + T::at(thread / T::kChunks + n * kStep, thread % T::kChunks)) = w[n];
  }
  // After store: zeros over the values' infinities and NaN; true if the thread has any.
  __device__ __forceinline__ bool store_finite(char* tv, int thread) const {
    if (__builtin_expect(!any_not_finite<IO>(v), 1)) return false;
#pragma unroll
    for (int n = 0; n < kN; ++n)
      *reinterpret_cast<u32x4_t*>(tv + T::at(thread / T::kChunks + n * kStep, thread % T::kChunks)) = finite_part<IO>(v[n]);
    return true;
  }
};

// Rows that belong to no sequence, zeroed where the call asks for it.
template <int IO, int DH>
__device__ __forceinline__ void fill_rest(const PagedArgs& a) {
  if (!a.fill) return;
  const int64_t first = a.cu != nullptr ? clamp64(a.cu[0], 0, a.T) : 0;
  const int64_t end = a.cu != nullptr ? clamp64(a.cu[a.n], 0, a.T) : a.n;
  const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    if (t >= first && t < end) continue;
    for (int e = threadIdx.x * 8; e < a.Hq * DH; e += blockDim.x * 8) store8<IO>(a.o, t * a.ldo + e, z);
  }
}

// A sequence's rows past max_q likewise, for the heads of key head hk.
template <int IO, int DH>
__device__ __forceinline__ void fill_past(const PagedArgs& a, const Seq& q, int hk) {
  if (!a.fill) return;
  const int G = a.Hq / a.Hk;
  const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int64_t t = q.t0 + q.nq; t < q.t1; ++t)
    for (int e = threadIdx.x * 8; e < G * DH; e += blockDim.x * 8) store8<IO>(a.o, t * a.ldo + (int64_t)hk * G * DH + e, z);
}

// Writes a finished row (or a split's share of it).
template <int IO, int DH>
__device__ __forceinline__ void finish(const PagedArgs& a, const Row& r, int sp, int h, RowState<DH>& st, float l, bool bad) {
  float inv = l == 0.f ? 0.f : 1.f / l;
  if (bad) inv = __builtin_nanf("");
  if (a.splits == 1) {
#pragma unroll
    for (int b = 0; b < DH / 32; ++b) store_block<IO>(a.o, r.tok * a.ldo + (int64_t)r.hq * DH, b, h, st.o[b], inv);
  } else {
    const int64_t at = (int64_t)sp * a.T * a.Hq + r.at;
#pragma unroll
    for (int b = 0; b < DH / 32; ++b) store_block<kF32>(a.part_o, at * DH, b, h, st.o[b], inv);
    if (h == 0) a.part_l[at] = bad ? __builtin_nanf("") : l == 0.f ? -__builtin_inff() : st.m + __log2f(l);
  }
}

// Query fragments of a packed row.
template <int IO, int DH>
__device__ __forceinline__ void load_q(const PagedArgs& a, const Row& r, int h, Frag<IO> (&qf)[DH / 16]) {
#pragma unroll
  for (int s = 0; s < DH / 16; ++s)
    qf[s] = r.real ? load_frag<IO>(a.q, r.tok * a.ldq + (int64_t)r.hq * DH + 16 * s + 8 * h) : zero_frag<IO>();
}

// The keys [lo, hi) of this split, whole tiles of `step` from the row tile's
// first key on.
__device__ __forceinline__ void split_range(int splits, int sp, int step, int& lo, int& hi) {
  const int tiles = (hi - lo + step - 1) / step, per = (tiles + splits - 1) / splits;
  const int64_t a = (int64_t)lo + (int64_t)sp * per * step, b = a + (int64_t)per * step;
  lo = (int)(a < hi ? a : hi);
  hi = (int)(b < hi ? b : hi);
}

// Few rows: one tile of up to 32 packed rows, which every wave holds; the
// waves take the key tiles of 32 in turn and join their row states in LDS.
template <int IO, int DH, int MOD>
__global__ __launch_bounds__(kThreads, IO == kBF16 ? 2 : 1) void attn_paged_few_kernel(PagedArgs a) {
  using T = Tile<IO, DH>;
  constexpr int kTile = kFewKeys * T::kRow;
  extern __shared__ __attribute__((aligned(512))) char lds[];  // a key and a value tile a wave; then the waves' row states
  __shared__ float stat[256];
  __shared__ int any_bad;
  fill_rest<IO, DH>(a);
  const int lane = threadIdx.x & (kWave - 1), wave = wave_id(), c = lane & 31, h = lane >> 5;
  if (threadIdx.x == 0) any_bad = 0;
  __syncthreads();
  const int hk = blockIdx.x % a.Hk;
  const int rest = blockIdx.x / a.Hk, sp = rest % a.splits, s = rest / a.splits;
  const Seq q = seq_of(a, s);
  if (q.nq == 0) return;
  if (sp == 0) fill_past<IO, DH>(a, q, hk);
  const Row r = row_of(a, s, q, hk, c);
  int lo, hi;
  wave_range(r.lo, r.hi, lo, hi);
  split_range(a.splits, sp, kFewKeys, lo, hi);

  Frag<IO> qf[DH / 16];
  load_q<IO, DH>(a, r, h, qf);
  const float slope2 = (MOD & kSloped) != 0 ? a.slopes[r.hq] * kLog2e : 0.f;
  settle(qf);
  RowState<DH> st;
  st.init();
  bool bad = false;
  char* tk = lds + wave * 2 * kTile;
  char* tv = tk + kTile;
  PagedStage<IO, DH, kFewKeys, kWave> sg;
  const int32_t* table = a.pages + (int64_t)s * a.max_pages;
  auto masked = [&](int key0) {
    return __any(r.lo < r.hi && (r.lo > key0 || r.hi < key0 + kFewKeys)) || key0 + kFewKeys > hi;
  };
  bool not_finite = false;
  int key0 = lo + wave * kFewKeys;
  constexpr int kAll = 4 * kFewKeys;
  if (key0 < hi) {
    sg.lookup(a, table, lane, key0, hi - 1);
    sg.load(a, hk, lane, key0, hi - 1, bad);
    if (key0 + kAll < hi) sg.lookup(a, table, lane, key0 + kAll, hi - 1);
  }
  for (; key0 < hi; key0 += kAll) {
    const bool partial = masked(key0);
    sg.store(tk, sg.k, lane);
    sg.store(tv, sg.v, lane);
    if (partial) not_finite |= sg.store_finite(tv, lane);
    if (key0 + kAll < hi) sg.load(a, hk, lane, key0 + kAll, hi - 1, bad);
    if (key0 + 2 * kAll < hi) sg.lookup(a, table, lane, key0 + 2 * kAll, hi - 1);
    wave_lds_fence();
    attend<IO, DH, 1, MOD>(st, qf, lds_addr(tk), lds_addr(tv), key0, r.lo, min(r.hi, hi), partial, r.pos, slope2, a.mod);
    wave_lds_fence();
  }
  if (__builtin_expect(__any(not_finite), 0))
    for (key0 = lo + wave * kFewKeys; key0 < hi; key0 += kAll)
      if (masked(key0))
        add_not_finite<IO, DH>(st, max(r.lo, key0), min(min(r.hi, hi), key0 + kFewKeys), h,
                               [&](int j) { return sg.value_row(a, table, hk, j); });
  if (__any(bad) && lane == 0) any_bad = 1;
  if (r.lo >= r.hi) st.init();  // (unmasked tiles were not for this row)
  float m, l;
  const f32x16_t sum = join_waves<DH>(lds, stat, wave, lane, st, m, l);
  if (wave >= DH / 32 || !r.real) return;
  float inv = l == 0.f ? 0.f : 1.f / l;
  if (any_bad) inv = __builtin_nanf("");
  if (a.splits == 1) {
    store_block<IO>(a.o, r.tok * a.ldo + (int64_t)r.hq * DH, wave, h, sum, inv);
  } else {
    const int64_t at = (int64_t)sp * a.T * a.Hq + r.at;
    store_block<kF32>(a.part_o, at * DH, wave, h, sum, inv);
    if (wave == 0 && h == 0) a.part_l[at] = any_bad ? __builtin_nanf("") : l == 0.f ? -__builtin_inff() : m + __log2f(l);
  }
}

// Many rows: 128 packed rows of one sequence and key head, 32 a wave.
template <int IO, int DH, int MOD>
__global__ __launch_bounds__(kThreads, IO == kBF16 ? 2 : 1) void attn_paged_chunk_kernel(PagedArgs a) {
  using T = Tile<IO, DH>;
  constexpr int kTile = kKeys * T::kRow;
  extern __shared__ __attribute__((aligned(512))) char lds[];
  __shared__ int range[16];
  __shared__ int any_bad;
  __shared__ int not_finite;  // some value of a masked tile is not
  fill_rest<IO, DH>(a);
  const int lane = threadIdx.x & (kWave - 1), wave = wave_id(), c = lane & 31, h = lane >> 5;
  const int hk = blockIdx.x % a.Hk;
  int rest = blockIdx.x / a.Hk;
  const int sp = rest % a.splits;
  rest /= a.splits;
  const int s = rest % a.n, tile = a.tiles - 1 - rest / a.n;
  const int G = a.Hq / a.Hk;
  const Seq q = seq_of(a, s);
  if ((int64_t)tile * kRows >= (int64_t)q.nq * G) return;
  if (sp == 0 && tile == 0) fill_past<IO, DH>(a, q, hk);
  const Row r = row_of(a, s, q, hk, tile * kRows + wave * 32 + c);
  int wlo, whi;
  wave_range(r.lo, r.hi, wlo, whi);
  if (lane == 0) {
    range[wave] = whi > 0 ? wlo : 0x7fffffff;
    range[4 + wave] = whi;
  }
  int ilo, ihi;
  common_range(r.lo, r.hi, ilo, ihi);
  if (lane == 0) {
    range[8 + wave] = ilo;
    range[12 + wave] = ihi;
  }
  if (threadIdx.x == 0) any_bad = not_finite = 0;
  __syncthreads();
  ilo = max(max(range[8], range[9]), max(range[10], range[11]));
  ihi = min(min(range[12], range[13]), min(range[14], range[15]));
  int blo = min(min(range[0], range[1]), min(range[2], range[3]));
  int bhi = max(max(range[4], range[5]), max(range[6], range[7]));
  if (bhi == 0) blo = 0;
  split_range(a.splits, sp, kKeys, blo, bhi);
  ihi = min(ihi, bhi);

  Frag<IO> qf[DH / 16];
  load_q<IO, DH>(a, r, h, qf);
  const float slope2 = (MOD & kSloped) != 0 ? a.slopes[r.hq] * kLog2e : 0.f;
  settle(qf);
  RowState<DH> st;
  st.init();
  bool bad = false;
  PagedStage<IO, DH, kKeys, kThreads> sg;
  const int32_t* table = a.pages + (int64_t)s * a.max_pages;
  if (blo < bhi) {
    sg.lookup(a, table, threadIdx.x, blo, bhi - 1);
    sg.load(a, hk, threadIdx.x, blo, bhi - 1, bad);
    if (blo + kKeys < bhi) sg.lookup(a, table, threadIdx.x, blo + kKeys, bhi - 1);
  }
  int buf = 0;
  for (int key0 = blo; key0 < bhi; key0 += kKeys, buf ^= 1) {
    char* tk = lds + buf * 2 * kTile;
    char* tv = tk + kTile;
    sg.store(tk, sg.k, threadIdx.x);
    if (key0 + kKeys < bhi) sg.load_k(a, hk, threadIdx.x, key0 + kKeys, bhi - 1, bad);
    sg.store(tv, sg.v, threadIdx.x);
    if ((key0 < ilo || key0 + kKeys > ihi) && sg.store_finite(tv, threadIdx.x)) not_finite = 1;
    if (key0 + kKeys < bhi) sg.load_v(a);
    if (key0 + 2 * kKeys < bhi) sg.lookup(a, table, threadIdx.x, key0 + 2 * kKeys, bhi - 1);
    __syncthreads();
    if (key0 < whi && key0 + kKeys > wlo) {
      const bool partial = __any(r.lo < r.hi && (r.lo > key0 || r.hi < key0 + kKeys)) || key0 + kKeys > bhi;
      attend<IO, DH, kKeys / 32, MOD>(st, qf, lds_addr(tk), lds_addr(tv), key0, r.lo, min(r.hi, bhi), partial, r.pos, slope2, a.mod);
    }
  }
  if (__builtin_expect(not_finite, 0))
    for (int key0 = blo; key0 < bhi; key0 += kKeys)
      if (key0 < ilo || key0 + kKeys > ihi)
        add_not_finite<IO, DH>(st, max(r.lo, key0), min(min(r.hi, bhi), key0 + kKeys), h,
                               [&](int j) { return sg.value_row(a, table, hk, j); });
  if (__any(bad) && lane == 0) any_bad = 1;
  __syncthreads();
  if (!r.real) return;
  if (r.lo >= r.hi) st.init();  // (unmasked tiles were not for this row)
  finish<IO, DH>(a, r, sp, h, st, st.l + other_half(st.l), any_bad != 0);
}

// Joins the splits' partial rows: Dh/4 lanes a row of [sequence][c][head], four
// elements each, with a running maximum over the splits, eight of them in
// flight at a time.  Many splits (few rows, a chain of loads each) go to GROUPS
// sets of lanes, which join what they found in LDS.
constexpr int kJoinGroups = 8;
template <int IO, int DH, int GROUPS>
__global__ __launch_bounds__(kThreads) void attn_paged_join_kernel(PagedArgs a) {
  constexpr int kLanes = DH / 4, kPerRow = kLanes * GROUPS;
  __shared__ float found[GROUPS > 1 ? 6 * kThreads : 1];
  const int64_t n = (int64_t)blockIdx.x * (kThreads / kPerRow) + threadIdx.x / kPerRow;
  const int e = threadIdx.x % kLanes * 4, group = threadIdx.x % kPerRow / kLanes;
  const int64_t sc = n / a.Hq;
  const int s = (int)(sc / a.max_q), c = (int)(sc % a.max_q), hq = (int)(n % a.Hq);
  Seq q{};
  if (s < a.n) q = seq_of(a, s);
  const bool real = s < a.n && c < q.nq;
  if (GROUPS == 1 && !real) return;
  const int64_t row = (q.t0 + c) * a.Hq + hq, all = a.T * a.Hq;
  float m = -__builtin_inff(), total = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  constexpr int kAhead = 8;
  auto take = [&](const float (&l)[kAhead], const float4 (&v)[kAhead]) {
    float top = m;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) top = fmaxf(top, l[j]);
    const float base = top == -__builtin_inff() ? 0.f : top, f = exp2_fast(m - base);
    m = top;
    total *= f;
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] *= f;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const float w = exp2_fast(l[j] - base);
      total += w;
      acc[0] = __builtin_fmaf(w, v[j].x, acc[0]);
      acc[1] = __builtin_fmaf(w, v[j].y, acc[1]);
      acc[2] = __builtin_fmaf(w, v[j].z, acc[2]);
      acc[3] = __builtin_fmaf(w, v[j].w, acc[3]);
    }
  };
  if (real)
    for (int i = group; i < a.splits; i += kAhead * GROUPS) {
      float l[kAhead];
      float4 v[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int sp = i + j * GROUPS;
        const int64_t at = min(sp, a.splits - 1) * all + row;
        l[j] = sp < a.splits ? a.part_l[at] : -__builtin_inff();
        v[j] = *reinterpret_cast<const float4*>(a.part_o + at * DH + e);
      }
      take(l, v);
    }
  if constexpr (GROUPS > 1) {
    static_assert(GROUPS == kAhead, "one batch");
    const float mine[6] = {m, total, acc[0], acc[1], acc[2], acc[3]};
#pragma unroll
    for (int k = 0; k < 6; ++k) found[k * kThreads + threadIdx.x] = mine[k];
    __syncthreads();
    if (!real || group != 0) return;
    float sum = 0.f;
    float l[kAhead];
    float4 v[kAhead];
    float top = -__builtin_inff();
#pragma unroll
    for (int j = 0; j < GROUPS; ++j) {
      const int at = threadIdx.x + j * kLanes;
      l[j] = found[at];
      v[j] = make_float4(found[2 * kThreads + at], found[3 * kThreads + at], found[4 * kThreads + at], found[5 * kThreads + at]);
      top = fmaxf(top, l[j]);
    }
    const float base = top == -__builtin_inff() ? 0.f : top;
#pragma unroll
    for (int j = 0; j < GROUPS; ++j) sum = __builtin_fmaf(exp2_fast(l[j] - base), found[kThreads + threadIdx.x + j * kLanes], sum);
    m = -__builtin_inff();
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] = 0.f;
    take(l, v);
    total = sum;
  }
  const float inv = total == 0.f ? 0.f : 1.f / total;
  const int64_t at = (q.t0 + c) * a.ldo + (int64_t)hq * DH + e;
  if constexpr (IO == kBF16)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + at) =
        make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
  else
    *reinterpret_cast<float4*>(static_cast<float*>(a.o) + at) = make_float4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
}

bool few_rows(const mhc_paged_desc& d) { return (int64_t)d.max_q * (d.Hq / d.Hk) <= kFewRows; }
int row_tiles(const mhc_paged_desc& d) {
  return few_rows(d) ? 1 : (int)(((int64_t)d.max_q * (d.Hq / d.Hk) + kRows - 1) / kRows);
}

// Splits of the keys: workgroups for every CU twice over with few rows, and a
// half more than fit with many (64 sequences of up to 8192 keys, single tokens:
// 280 + 6 us for the join with four workgroups a CU, 288 with two and no join;
// 700 tokens over 6000 keys: 101 + 11 us with three a CU, 131 + 10 with two,
// 121 + 12 with four), none with fewer than 128 keys (few) or 256 (many) of a
// full table.
int splits_of(const mhc_paged_desc& d) {
  const int64_t base = (int64_t)d.n_seqs * d.Hk * row_tiles(d);
  const int64_t keys = (int64_t)d.max_pages * d.page_size;
  int64_t want = ((few_rows(d) ? 4 : 3) * device_cu_count() + base - 1) / base;
  const int64_t most = (keys + (few_rows(d) ? 127 : 255)) / (few_rows(d) ? 128 : 256);
  if (want > most) want = most;
  if (want > kMaxSplits) want = kMaxSplits;
  return want < 1 ? 1 : (int)want;
}

}  // namespace

size_t attn_paged_workspace_bytes(const mhc_paged_desc& d) {
  const int splits = splits_of(d);
  if (splits == 1) return 0;
  const size_t rows = (size_t)splits * (size_t)d.T * d.Hq;
  return rows * d.Dh * sizeof(float) + rows * sizeof(float);
}

hipError_t launch_attn_paged(const mhc_paged_desc& d, const void* q, const void* kc, const void* vc, void* o, void* ws,
                             hipStream_t s) {
  PagedArgs a{};
  a.T = d.T;
  a.n = d.n_seqs;
  a.max_q = d.max_q;
  a.Hq = d.Hq;
  a.Hk = d.Hk;
  a.window = d.window;
  a.max_pages = d.max_pages;
  a.num_pages = (int)d.num_pages;
  a.page_size = d.page_size;
  a.fill = d.fill_outside;
  a.splits = splits_of(d);
  a.tiles = row_tiles(d);
  a.by_page = div_of((uint32_t)d.page_size);
  a.by_group = div_of((uint32_t)(d.Hq / d.Hk));
  a.mod = {d.scale, d.softcap};
  a.cu = d.cu_q;
  a.prefix = d.prefix;
  a.kv = d.kv_lens;
  a.pages = d.pages;
  a.slopes = d.slopes;
  a.q = q;
  a.kc = kc;
  a.vc = vc;
  a.o = o;
  a.part_o = static_cast<float*>(ws);
  a.part_l = a.part_o + (size_t)a.splits * (size_t)d.T * d.Hq * d.Dh;
  a.ldq = d.ldq;
  a.ldo = d.ldo;
  const bool few = few_rows(d);
  const dim3 grid((unsigned)((int64_t)d.n_seqs * d.Hk * a.tiles * a.splits));
  hipError_t err = hipErrorInvalidValue;
  dispatch_attn(d.io, d.Dh, d.softcap, d.slopes, [&](auto io_, auto dh_, auto mod_) {
    constexpr int IO = decltype(io_)::value;
    constexpr int DH = decltype(dh_)::value;
    constexpr int MOD = decltype(mod_)::value;
    constexpr int row = Tile<IO, DH>::kRow;
    // few: four waves' tiles, or their fp32 row states
    constexpr int few_lds = 8 * kFewKeys * row > wave_states_bytes<DH>() ? 8 * kFewKeys * row : wave_states_bytes<DH>();
    if (few)
      MHC_LAUNCH((attn_paged_few_kernel<IO, DH, MOD>), grid, dim3(kThreads), few_lds, s, a);
    else
      MHC_LAUNCH((attn_paged_chunk_kernel<IO, DH, MOD>), grid, dim3(kThreads), 4 * kKeys * row, s, a);
    err = hipGetLastError();
    if (err != hipSuccess || a.splits == 1) return;
    const int64_t rows = (int64_t)d.n_seqs * d.max_q * d.Hq;
    auto blocks = [&](int lanes) { return dim3((unsigned)((rows * lanes + kThreads - 1) / kThreads)); };
    if (a.splits > kJoinGroups)
      MHC_LAUNCH((attn_paged_join_kernel<IO, DH, kJoinGroups>), blocks(DH / 4 * kJoinGroups), dim3(kThreads), 0, s, a);
    else
      MHC_LAUNCH((attn_paged_join_kernel<IO, DH, 1>), blocks(DH / 4), dim3(kThreads), 0, s, a);
    err = hipGetLastError();
  });
  return err;
}

}  // namespace mhc
