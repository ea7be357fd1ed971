// Device-side pieces shared by the attention kernels: matrix-core fragments,
// LDS tiles and the rows' visible ranges.
//
// Every product runs on 32x32 accumulator blocks (v_mfma_f32_32x32x16_bf16, or
// eight v_mfma_f32_32x32x2_f32 for fp32).  Lane l = 32·h + c:
//   A operand: row c, B operand: column c, eight elements of the 16-wide inner
//   axis each; the inner index is 8h + e for operands read along a row, and
//   for operands formed from an accumulator 4h + e for e < 4, 8 + 4h + e - 4
//   for the rest (any order serves as long as A and B agree);
//   accumulator: column c, element r is row 8·(r/4) + 4h + r mod 4.
// So a score block whose columns are the lane's own row of the softmax becomes
// the B operand of the next product in the lane that holds it: the
// probabilities never leave the registers.
#pragma once

#include "mhc_device.h"

namespace mhc {
namespace attn {

constexpr int kThreads = 256;  // four waves
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef unsigned u32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned u32x2_t __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) const u32x4_t* lds_u32x4_t;
typedef __attribute__((address_space(3))) s16x4_t* lds_s16x4_t;
typedef __attribute__((address_space(3))) const float* lds_float_t;

// Eight elements of an operand.
template <int IO>
struct Frag;
template <>
struct Frag<kBF16> {
  u32x4_t w;
};
template <>
struct Frag<kF32> {
  float v[8];
};

__device__ __forceinline__ f32x16_t mma(const Frag<kBF16>& a, const Frag<kBF16>& b, f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a.w), __builtin_bit_cast(bf16x8_t, b.w),
                                                 c, 0, 0, 0);
}
__device__ __forceinline__ f32x16_t mma(const Frag<kF32>& a, const Frag<kF32>& b, f32x16_t c) {
#pragma unroll
  for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a.v[e], b.v[e], c, 0, 0, 0);
  return c;
}

// Eight consecutive elements of global memory (16-byte aligned).
template <int IO>
__device__ __forceinline__ Frag<IO> load_frag(const void* base, int64_t i) {
  Frag<IO> f;
  if constexpr (IO == kBF16)
    f.w = *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(base) + i);
  else
    load8<kF32>(base, i, f.v);
  return f;
}
template <int IO>
__device__ __forceinline__ Frag<IO> zero_frag() {
  Frag<IO> f;
  if constexpr (IO == kBF16) {
    f.w = u32x4_t{0, 0, 0, 0};
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) f.v[e] = 0.f;
  }
  return f;
}

// Waits for fragments loaded from global memory here and now.  Without it the
// first use inside a loop waits, every time round, for whatever loads are in
// flight by then: the next tile's.
template <int IO, int N>
__device__ __forceinline__ void settle(Frag<IO> (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (IO == kBF16) {
      asm volatile("" : "+v"(f[i].w));
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) asm volatile("" : "+v"(f[i].v[e]));
    }
  }
}

// The wave's number, known to be the same for all its lanes.
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x / kWave); }

// The operand formed from accumulator elements 8·half .. 8·half + 7 of x.
// bf16: each is rounded once, to the type the matrix cores take.
template <int IO>
__device__ __forceinline__ Frag<IO> frag_of(const f32x16_t& x, int half) {
  Frag<IO> f;
  if constexpr (IO == kBF16) {
#pragma unroll
    for (int e = 0; e < 4; ++e) f.w[e] = pack_bf16x2(x[8 * half + 2 * e], x[8 * half + 2 * e + 1]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) f.v[e] = x[8 * half + e];
  }
  return f;
}

// bf16: the operand formed from what that rounding leaves.
__device__ __forceinline__ Frag<kBF16> rest_frag(const f32x16_t& x, int half) {
  Frag<kBF16> f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float a = x[8 * half + 2 * e], b = x[8 * half + 2 * e + 1];
    const uint32_t p = pack_bf16x2(a, b);
    f.w[e] = pack_bf16x2(a - __uint_as_float(p << 16), b - __uint_as_float(p & 0xffff0000u));
  }
  return f;
}

// A tile of head rows in LDS, 16-byte chunks.  Chunk c of row r lies at place
// c ^ swz(r) of the row.  Sixteen consecutive rows put one chunk on all 64
// banks (reads along the rows), and four consecutive rows, a multiple of four
// the first, put four neighbouring chunks on all of them (32 lanes of a
// transposing read).  A swizzle that kept only eight rows apart cost half as
// many cycles again on either read (SQ_LDS_BANK_CONFLICT).
template <int IO, int DH>
struct Tile {
  static constexpr int kElem = IoT<IO>::bytes;
  static constexpr int kRow = DH * kElem;      // bytes of a row
  static constexpr int kChunks = kRow / 16;    // 16-byte chunks of a row
  static constexpr int kPer = 16 / kElem;      // elements of a chunk
  __device__ static __forceinline__ int swz(int r) {
    return kChunks >= 16 ? (r & 3) << 2 | (r >> 2 & 3) : (r & 2) << 1 | (r >> 2 & 3);
  }
  __device__ static __forceinline__ int at(int r, int c) { return r * kRow + ((c ^ swz(r)) << 4); }

  // Operand along the row: elements 16·s + 8·h + e of row c (+ a multiple of
  // 16, as a byte offset `off`).  `at0` = row_addr(tile, c, h); the chunks of a
  // row differ from it by an exclusive or with a constant (tiles start at
  // multiples of a row, 512 bytes at most).
  __device__ static __forceinline__ uint32_t row_addr(uint32_t tile, int c, int h) {
    return tile + c * kRow + (((kElem == 2 ? h : 2 * h) ^ swz(c)) << 4);
  }
  template <int S>
  __device__ static __forceinline__ Frag<IO> row_frag(uint32_t at0, int off) {
    Frag<IO> f;
    if constexpr (IO == kBF16) {
      f.w = *reinterpret_cast<lds_u32x4_t>((at0 ^ (S << 5)) + off);
    } else {
      const u32x4_t a = *reinterpret_cast<lds_u32x4_t>((at0 ^ (S << 6)) + off);
      const u32x4_t b = *reinterpret_cast<lds_u32x4_t>((at0 ^ (S << 6) ^ 16) + off);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f.v[e] = __uint_as_float(a[e]);
        f.v[4 + e] = __uint_as_float(b[e]);
      }
    }
    return f;
  }

  // Operand across the rows: column 32·D + c of rows r0 + 4h + {0..3} and
  // r0 + 8 + 4h + {0..3} (the order of operands formed from an accumulator),
  // r0 a multiple of 16 in `off` (bytes).  `at0` = col_addr(tile, lane).
  // bf16: ds_read_b64_tr_b16, whose 16 lanes read a 4 x 16 block (lane i the
  // four elements from column 4·(i mod 4) of row i/4) and get its columns;
  // swz(r + 8) = swz(r) ^ 2 is 32 bytes.  fp32: one element a read, row by row.
  __device__ static __forceinline__ uint32_t col_addr(uint32_t tile, int lane) {
    const int h = lane >> 5;
    if constexpr (IO == kBF16) {
      const int i = lane & 15, r = 4 * h + (i >> 2);
      return tile + r * kRow + (((((lane & 16) >> 3) + ((i & 3) >> 1)) ^ swz(r)) << 4) + (i & 1) * 8;
    } else {
      const int c = lane & 31, r = 4 * h;
      return tile + r * kRow + (((c >> 2) ^ swz(r)) << 4) + (c & 3) * 4;
    }
  }
  template <int D>
  __device__ static __forceinline__ Frag<IO> col_frag(uint32_t at0, int off) {
    Frag<IO> f;
    if constexpr (IO == kBF16) {
      const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_s16x4_t>((at0 ^ (D << 6)) + off));
      const s16x4_t hi =
          __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_s16x4_t>((at0 ^ (D << 6) ^ 32) + off + 8 * kRow));
      const u32x2_t a = __builtin_bit_cast(u32x2_t, lo), b = __builtin_bit_cast(u32x2_t, hi);
      f.w = u32x4_t{a.x, a.y, b.x, b.y};
    } else {
      // row 4h + j + 8·(e >> 2), j < 4: swz adds 4j (chunks), and 2 for the upper four
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int j = e & 3, up = e >> 2;
        const uint32_t x = (D << 7) ^ (j << 6) ^ (up << 5);
        f.v[e] = *reinterpret_cast<lds_float_t>((at0 ^ x) + off + (j + 8 * up) * kRow);
      }
    }
    return f;
  }
};

// An LDS pointer's byte address.
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char*)p;
}

// f(integral constant) for 0 .. N - 1, unrolled.
template <int N, typename F>
__device__ __forceinline__ void each(F&& f) {
  if constexpr (N > 0) {
    each<N - 1>(f);
    f(std::integral_constant<int, N - 1>{});
  }
}

// Whether one of N chunks holds an infinity or NaN: the largest magnitude, as
// bit patterns, reaches infinity's.
template <int IO, int N>
__device__ __forceinline__ bool any_not_finite(const u32x4_t (&w)[N]) {
  typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));
  if constexpr (IO == kBF16) {
    u16x2_t m{0, 0};
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, w[n][e] & 0x7fff7fffu));
    return m.x >= 0x7f80u || m.y >= 0x7f80u;
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) m = max(m, w[n][e] & 0x7fffffffu);
    return m >= 0x7f800000u;
  }
}
// A chunk with zeros in their place.
template <int IO>
__device__ __forceinline__ u32x4_t finite_part(u32x4_t w) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const bool top = (w[e] & 0x7f800000u) == 0x7f800000u, low = IO == kBF16 && (w[e] & 0x7f80u) == 0x7f80u;
    w[e] = IO == kBF16 ? (top ? 0u : w[e] & 0xffff0000u) | (low ? 0u : w[e] & 0xffffu) : top ? 0u : w[e];
  }
  return w;
}

// Staging of R head rows by NT threads: global memory to registers, then
// registers to LDS, so that the next tile is on its way while this one is
// used.  Thread i takes chunk i mod C of rows i/C, i/C + NT/C, ...
template <int IO, int DH, int R, int NT = kThreads>
struct Stage {
  using T = Tile<IO, DH>;
  static constexpr int kN = R * T::kChunks / NT;  // chunks a thread
  static constexpr int kStep = NT / T::kChunks;   // rows between a thread's chunks
  static_assert(R * T::kChunks % NT == 0 && NT % T::kChunks == 0, "whole passes");
  u32x4_t w[kN];

  // Rows base + 0 .. base + rows - 1, `ld` elements apart; the buffer's own
  // bounds check returns zeros for rows past the last.
  __device__ __forceinline__ void load(const void* base, int64_t ld, int rows, int thread = threadIdx.x) {
    rows = min(rows, R);
    const int row_bytes = (int)(ld * T::kElem);
    const uint32_t bytes = rows > 0 ? (uint32_t)(rows - 1) * (uint32_t)row_bytes + T::kRow : 0u;
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
    const uint32_t v0 = (uint32_t)(thread / T::kChunks) * (uint32_t)row_bytes + (thread % T::kChunks) * 16u;
#pragma unroll
    for (int n = 0; n < kN; ++n)
      w[n] = __builtin_amdgcn_raw_buffer_load_b128(r, (int)(v0 + (uint32_t)(n * kStep) * (uint32_t)row_bytes), 0, 0);
  }
  __device__ __forceinline__ void store(char* t, int thread = threadIdx.x) const {
#pragma unroll
    for (int n = 0; n < kN; ++n)
      *reinterpret_cast<u32x4_t*>(t + T::at(thread / T::kChunks + n * kStep, thread % T::kChunks)) = w[n];
  }
  // After store: zeros over infinities and NaN; true if the thread has any.
  __device__ __forceinline__ bool store_finite(char* t, int thread = threadIdx.x) const {
    if (__builtin_expect(!any_not_finite<IO>(w), 1)) return false;
#pragma unroll
    for (int n = 0; n < kN; ++n)
      *reinterpret_cast<u32x4_t*>(t + T::at(thread / T::kChunks + n * kStep, thread % T::kChunks)) = finite_part<IO>(w[n]);
    return true;
  }
};

// Entries of the sorted docs[0..cnt) that are ≤ i, for a wave-uniform i: each
// step probes 64 entries, one a lane.  (Unsorted entries give some number in
// 0..cnt, so no access leaves the array.)
__device__ __forceinline__ int count_le(const int32_t* docs, int cnt, int i) {
  const int lane = threadIdx.x & (kWave - 1);
  int lo = 0, hi = cnt;
  while (lo < hi) {
    const int step = (hi - lo + kWave - 1) / kWave;
    const int64_t e = (int64_t)lo + (int64_t)(lane + 1) * step - 1;
    const bool le = e < hi && docs[e] <= i;
    const int c = __popcll(__ballot(le));
    const int64_t nlo = (int64_t)lo + (int64_t)c * step, nhi = nlo + step - 1;
    lo = (int)(nlo < hi ? nlo : hi);
    hi = (int)(nhi < hi ? nhi : hi);
  }
  return lo;
}

// Masks of one packed batch of documents (the dense calls).
struct DocMask {
  const int32_t* docs;    // [n_docs + 1] or null: one document of all T rows
  const int32_t* prefix;  // [n_docs] or null
  int n_docs, T, causal, window;

  // First and last row + 1 of row i's document, and the end of its prefix;
  // false if the row belongs to none.  `a`..`b`: bounds of count_le(i).
  __device__ __forceinline__ bool doc(int i, int a, int b, int& s, int& e, int& p) const {
    if (docs == nullptr) {
      s = 0;
      e = T;
      p = prefix != nullptr ? clampi(prefix[0], 0, T) : 0;
      return i < T;
    }
    while (a < b) {  // largest count c in [a, b] with docs[c - 1] <= i
      const int m = (a + b + 1) >> 1;
      if (docs[m - 1] <= i) a = m; else b = m - 1;
    }
    if (a < 1 || a > n_docs || i >= T) return false;
    s = clampi(docs[a - 1], 0, T);
    e = clampi(docs[a], 0, T);
    p = prefix != nullptr ? (int)min((int64_t)e, (int64_t)s + clampi(prefix[a - 1], 0, T)) : s;
    return i >= s && i < e;
  }
  __device__ static __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

  // Bounds of count_le for the rows i0..i1 (wave-uniform).
  __device__ __forceinline__ void bounds(int i0, int i1, int& a, int& b) const {
    a = b = 0;
    if (docs == nullptr) return;
    a = count_le(docs, n_docs + 1, i0);
    b = count_le(docs, n_docs + 1, i1);
    if (b < a) b = a;
  }
  // Keys [lo, hi) that row i sees (empty for a row of no document).
  __device__ __forceinline__ bool keys(int i, int a, int b, int& lo, int& hi) const {
    int s, e, p;
    lo = hi = 0;
    if (!doc(i, a, b, s, e, p)) return false;
    lo = s;
    hi = e;
    if (causal) {
      hi = max(i + 1, p);
      if (window > 0) lo = max(s, i - window + 1);
    }
    return true;
  }
  // Rows [lo, hi) that see key j.
  __device__ __forceinline__ bool rows(int j, int a, int b, int& lo, int& hi) const {
    int s, e, p;
    lo = hi = 0;
    if (!doc(j, a, b, s, e, p)) return false;
    lo = s;
    hi = e;
    if (causal) {
      lo = j < p ? s : j;
      if (window > 0) hi = (int)min((int64_t)e, (int64_t)j + window);
    }
    return true;
  }
};

// Smallest lo and largest hi over the wave's lanes with lo < hi (lo = hi = 0
// where there is none).
__device__ __forceinline__ void wave_range(int lo, int hi, int& wlo, int& whi) {
  wlo = lo < hi ? lo : 0x7fffffff;
  whi = lo < hi ? hi : 0;
#pragma unroll
  for (int off = kWave / 2; off > 0; off >>= 1) {
    wlo = min(wlo, __shfl_xor(wlo, off, kWave));
    whi = max(whi, __shfl_xor(whi, off, kWave));
  }
  wlo = __builtin_amdgcn_readfirstlane(wlo);
  whi = __builtin_amdgcn_readfirstlane(whi);
  if (whi == 0) wlo = 0;
}

// The other half's value: lane l and l ^ 32.
__device__ __forceinline__ float other_half(float v) { return __shfl_xor(v, 32, kWave); }

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// tanh by one exponential of -2|x|: exact at both ends.  For small |x| the
// difference 1 - e would lose digits, so the odd series takes over there: its
// first dropped term is 62/2835·x⁹, 2⁻²⁶ of x at |x| = 0.17.
__device__ __forceinline__ float tanh_fast(float x) {
  const float t = exp2_fast(-2.f * kLog2e * fabsf(x));
  const float big = (1.f - t) * __builtin_amdgcn_rcpf(1.f + t);
  const float x2 = x * x;
  const float small = fabsf(x) * (1.f + x2 * (-1.f / 3.f + x2 * (2.f / 15.f + x2 * (-17.f / 315.f))));
  return copysignf(fabsf(x) < 0.17f ? small : big, x);
}

// Ties a branch's compares to the branch: otherwise they are folded into
// selects that every tile pays for, masked or not.
__device__ __forceinline__ void keep_branch(int& a, int& b) { asm volatile("" : "+v"(a), "+v"(b)); }

// A wave's own LDS: its writes come before its reads, and these before the
// next writes, without a barrier.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// How scores are formed from the products q·k, in units of log 2 so that exp2
// serves: capped (cap·tanh(scale·x/cap), cap > 0), lowered by slope·distance.
struct ScoreMod {
  float scale, cap;
  // the factor on q·k: to log 2 units at once, or to the tanh's argument
  __host__ __device__ __forceinline__ float pre() const { return cap > 0.f ? scale / cap : scale * kLog2e; }
  __host__ __device__ __forceinline__ float post() const { return cap * kLog2e; }
};

// tanh of the capping.  fp32: tanh_fast.  bf16: 1 - 2/(1 + e^2x), whose
// absolute error of 2⁻²³ moves a score by cap·2⁻²³, far below a rounding of
// its probability to bf16.
template <int IO>
__device__ __forceinline__ float cap_tanh(float x) {
  if constexpr (IO == kF32) return tanh_fast(x);
  return 1.f - 2.f * __builtin_amdgcn_rcpf(1.f + exp2_fast(2.f * kLog2e * x));
}

// What a kernel's scores have besides the scale: bits of a template argument.
enum Mod : int { kCapped = 1, kSloped = 2 };

// The score in log 2 units of x = q·k times mod.pre(), at a signed distance.
template <int IO, int MOD>
__device__ __forceinline__ float modified(float x, ScoreMod mod, float slope2, float dist) {
  if constexpr ((MOD & kCapped) != 0) x = mod.post() * cap_tanh<IO>(x);
  if constexpr ((MOD & kSloped) != 0) x = __builtin_fmaf(-slope2, fabsf(dist), x);
  return x;
}

// Accumulator element r's row within its 32-row block, for lane half h.
__device__ __forceinline__ constexpr int acc_row(int r, int h) { return 8 * (r >> 2) + 4 * h + (r & 3); }

// One accumulator block's worth of an output row: column block `blk` of the
// lane's row, elements 8i + 4h + {0..3}, scaled.
template <int IO>
__device__ __forceinline__ void store_block(void* out, int64_t row, int blk, int h, const f32x16_t& x, float f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t at = row + 32 * blk + 8 * i + 4 * h;
    const float a = x[4 * i] * f, b = x[4 * i + 1] * f, c = x[4 * i + 2] * f, d = x[4 * i + 3] * f;
    if constexpr (IO == kBF16)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = make_uint2(pack_bf16x2(a, b), pack_bf16x2(c, d));
    else
      *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = make_float4(a, b, c, d);
  }
}

// The eight bits of an fp32 output that its bf16 rounding leaves out, as the
// distance of the bit patterns in units of 2⁸ (neighbouring floats are
// neighbouring integers): bf16 word << 16 plus rest << 8 gives the value back
// to 2⁻¹⁶ of itself.
__device__ __forceinline__ uint32_t rest_of(float x, uint32_t bf16_bits) {
  const int d = (int)(__float_as_uint(x) - (bf16_bits << 16)) + 128;
  const int r = d >> 8;
  return (uint32_t)(r > 127 ? 127 : r) & 0xffu;
}
__device__ __forceinline__ void store_rest(uint8_t* rest, int64_t row, int blk, int h, const f32x16_t& x, float f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float a = x[4 * i + 2 * e] * f, b = x[4 * i + 2 * e + 1] * f;
      const uint32_t p = pack_bf16x2(a, b);
      w |= (rest_of(a, p & 0xffffu) | rest_of(b, p >> 16) << 8) << (16 * e);
    }
    *reinterpret_cast<uint32_t*>(rest + row + 32 * blk + 8 * i + 4 * h) = w;
  }
}
// Adds the rest to eight bf16 values widened to fp32.
__device__ __forceinline__ void add_rest(const uint8_t* rest, int64_t at, float v[8]) {
  const uint2 w = *reinterpret_cast<const uint2*>(rest + at);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int r = (int)((e < 4 ? w.x : w.y) << (24 - 8 * (e & 3))) >> 24;
    v[e] = __uint_as_float(__float_as_uint(v[e]) + ((uint32_t)r << 8));
  }
}

// State of the lane's softmax row over the keys seen so far: running maximum
// (log 2 units), this half's share of the sum, and the unnormalised output.
template <int DH>
struct RowState {
  float m, l;
  f32x16_t o[DH / 32];
  __device__ __forceinline__ void init() {
    m = -__builtin_inff();
    l = 0.f;
#pragma unroll
    for (int b = 0; b < DH / 32; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) o[b][r] = 0.f;
  }
};

// Takes KB blocks of 32 keys into the row state: scores by S^T = K·Q^T,
// masked to the lane's keys [lo, hi) where `partial`, then O^T += V^T·P^T.
// `key0`: index of the tile's first key; `pos`: the row's own index.
// The maximum is let lag by up to 2⁶: a new maximum rescales the output only
// when it would overflow that margin (p stays ≤ 64, exact in fp32 sums, and
// bf16 keeps its relative precision at any scale).  bf16: a probability is
// rounded for the second product, which averages out over many keys; a masked
// tile's, which may be all that a row has, go in to twice the bits, by a second
// pass over their rests.
template <int IO, int DH, int KB, int MOD>
__device__ __forceinline__ void attend(RowState<DH>& st, const Frag<IO> (&qf)[DH / 16], uint32_t tk, uint32_t tv,
                                       int key0, int lo, int hi, bool partial, int pos, float slope2, ScoreMod mod) {
  using T = Tile<IO, DH>;
  const int lane = threadIdx.x & (kWave - 1), c = lane & 31, h = lane >> 5;
  const uint32_t ka = T::row_addr(tk, c, h), va = T::col_addr(tv, lane);
  f32x16_t s[KB];
#pragma unroll
  for (int b = 0; b < KB; ++b) {
#pragma unroll
    for (int r = 0; r < 16; ++r) s[b][r] = 0.f;
    each<DH / 16>([&](auto i) { s[b] = mma(T::template row_frag<i>(ka, 32 * b * T::kRow), qf[i], s[b]); });
  }
  float pre = mod.pre();
  if constexpr (MOD != 0) {
    const float d0 = (float)(pos - key0 - 4 * h);
#pragma unroll
    for (int b = 0; b < KB; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        s[b][r] = modified<IO, MOD>(s[b][r] * pre, mod, slope2, d0 - (float)(32 * b + 8 * (r >> 2) + (r & 3)));
    pre = 1.f;
  }
  if (partial) {
    int l0 = lo - key0 - 4 * h, h0 = hi - key0 - 4 * h;
    keep_branch(l0, h0);
#pragma unroll
    for (int b = 0; b < KB; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int k = 32 * b + 8 * (r >> 2) + (r & 3);
        s[b][r] = k >= l0 && k < h0 ? s[b][r] : -__builtin_inff();
      }
  }
  float mx = s[0][0];
#pragma unroll
  for (int b = 0; b < KB; ++b)
#pragma unroll
    for (int r = 0; r < 16; ++r) mx = fmaxf(mx, s[b][r]);
  mx = fmaxf(mx, other_half(mx)) * pre;
  constexpr float kLag = 6.f;
  if (__any(mx > st.m + kLag)) {
    const float m = fmaxf(st.m, mx);
    const float f = m == -__builtin_inff() ? 1.f : exp2_fast(st.m - m);
    st.m = m;
    st.l *= f;
#pragma unroll
    for (int b = 0; b < DH / 32; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) st.o[b][r] *= f;
  }
  const float base = st.m == -__builtin_inff() ? 0.f : st.m;
  float sum = 0.f;
#pragma unroll
  for (int b = 0; b < KB; ++b)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      s[b][r] = exp2_fast(__builtin_fmaf(s[b][r], pre, -base));
      sum += s[b][r];
    }
  st.l += sum;
#pragma unroll
  for (int b = 0; b < KB; ++b)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const Frag<IO> p = frag_of<IO>(s[b], i);
      each<DH / 32>([&](auto d) { st.o[d] = mma(T::template col_frag<d>(va, (32 * b + 16 * i) * T::kRow), p, st.o[d]); });
    }
  if constexpr (IO == kBF16)
    if (partial)
#pragma unroll
      for (int b = 0; b < KB; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const Frag<IO> p = rest_frag(s[b], i);
          each<DH / 32>([&](auto d) { st.o[d] = mma(T::template col_frag<d>(va, (32 * b + 16 * i) * T::kRow), p, st.o[d]); });
        }
}

// LDS bytes of join_waves / sum_waves.
template <int DH>
constexpr int wave_states_bytes() { return 4 * (DH / 32) * 16 * kWave * 4; }

// Values go into masked tiles without their infinities and NaN: in the product
// 0 · NaN would hand them to the rows that do not see their key as well.  This
// adds those of the keys first..end - 1 that the lane's row does see, key by
// key from global memory.  `row(j)`: address of key j's value row.
template <int IO, int DH, typename F>
__device__ __forceinline__ void add_not_finite(RowState<DH>& st, int first, int end, int h, F&& row) {
#pragma unroll 1
  for (int j = first; j < end; ++j) {
    const char* v = row(j);
#pragma unroll
    for (int b = 0; b < DH / 32; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x[4];
        const int at = 32 * b + 8 * i + 4 * h;
        if constexpr (IO == kBF16) {
          const uint2 w = *reinterpret_cast<const uint2*>(v + 2 * at);
          x[0] = __uint_as_float(w.x << 16);
          x[1] = __uint_as_float(w.x & 0xffff0000u);
          x[2] = __uint_as_float(w.y << 16);
          x[3] = __uint_as_float(w.y & 0xffff0000u);
        } else {
          const float4 w = *reinterpret_cast<const float4*>(v + 4 * at);
          x[0] = w.x;
          x[1] = w.y;
          x[2] = w.z;
          x[3] = w.w;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
          st.o[b][4 * i + e] += fabsf(x[e]) < __builtin_inff() ? 0.f : x[e];
      }
  }
}

// Keys that every lane with lo < hi sees, for ranges that do not go back from
// one lane to the next: [ilo, ihi), all keys if there is no such lane.
__device__ __forceinline__ void common_range(int lo, int hi, int& ilo, int& ihi) {
  const uint64_t live = __ballot(lo < hi);
  ilo = live == 0 ? 0 : __builtin_amdgcn_readlane(lo, 31 - __clz((int)(uint32_t)live));
  ihi = live == 0 ? 0x7fffffff : __builtin_amdgcn_readlane(hi, __ffs((int)(uint32_t)live) - 1);
}

// Sums four waves' accumulators x[block] (scaled by f) for the same 32 columns:
// wave w < DH/32 returns block w of the sum.  `lds`: wave_states_bytes, free
// for use by all waves.
template <int DH>
__device__ __forceinline__ f32x16_t sum_waves(char* lds, int wave, int lane, const f32x16_t (&x)[DH / 32], float f) {
  // [wave][column block][element][lane]
  float* acc = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int b = 0; b < DH / 32; ++b)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[((wave * (DH / 32) + b) * 16 + e) * kWave + lane] = x[b][e] * f;
  __syncthreads();
  f32x16_t sum;
  const int b = wave < DH / 32 ? wave : 0;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) t += acc[((w * (DH / 32) + b) * 16 + e) * kWave + lane];
    sum[e] = t;
  }
  return sum;
}

// Joins the row states of four waves that held the same 32 rows over different
// keys: m and l become the whole row's, and wave w < DH/32 returns block w of
// the unnormalised output.  `stat`: [2][4][32] floats.
template <int DH>
__device__ __forceinline__ f32x16_t join_waves(char* lds, float* stat, int wave, int lane, const RowState<DH>& st, float& m,
                                               float& l) {
  const int c = lane & 31;
  const float mine = st.l + other_half(st.l);
  if (lane < 32) {
    stat[wave * 32 + c] = st.m;
    stat[128 + wave * 32 + c] = mine;
  }
  __syncthreads();
  m = fmaxf(fmaxf(stat[c], stat[32 + c]), fmaxf(stat[64 + c], stat[96 + c]));
  const float base = m == -__builtin_inff() ? 0.f : m;
  l = 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w) l += stat[128 + w * 32 + c] * exp2_fast(stat[w * 32 + c] - base);
  return sum_waves<DH>(lds, wave, lane, st.o, exp2_fast(st.m - base));
}

}  // namespace attn

// Calls f(io, head size, score modification) as integral constants for the
// supported kinds.
template <typename F>
__host__ bool dispatch_attn(int io, int dh, float cap, const float* slopes, F&& f) {
  const int mod = (cap > 0.f ? attn::kCapped : 0) | (slopes != nullptr ? attn::kSloped : 0);
  return dispatch_io(io, [&](auto io_) {
    auto with_dh = [&](auto dh_) {
      switch (mod) {
        case 0: f(io_, dh_, std::integral_constant<int, 0>{}); break;
        case 1: f(io_, dh_, std::integral_constant<int, 1>{}); break;
        case 2: f(io_, dh_, std::integral_constant<int, 2>{}); break;
        default: f(io_, dh_, std::integral_constant<int, 3>{}); break;
      }
    };
    if (dh == 64)
      with_dh(std::integral_constant<int, 64>{});
    else if (dh == 128)
      with_dh(std::integral_constant<int, 128>{});
  });
}

}  // namespace mhc
