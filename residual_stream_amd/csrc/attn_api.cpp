// C ABI of the attention sublayer (declared in include/mhc.h): argument
// validation and dispatch.  No allocation, no synchronisation.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>
#include <limits>

#include "mhc.h"
#include "mhc_internal.h"

namespace {

constexpr int64_t kMaxInt = std::numeric_limits<int32_t>::max();
constexpr int64_t kMaxStride = 1 << 22;  // 64 rows of it stay within a buffer's 32-bit range

bool aligned(const void* p, size_t n) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool aligned16(const void* p) { return aligned(p, 16); }
bool optional(const void* p, size_t n) { return p == nullptr || aligned(p, n); }

mhc_status from_hip(hipError_t e) { return e == hipSuccess ? MHC_OK : MHC_ERR_HIP; }

bool workspace_ok(const void* ws, size_t have, size_t need) {
  return need == 0 || (aligned(ws, 256) && have >= need);
}

bool stride_ok(int64_t ld, int64_t heads, int64_t dh) {
  return ld >= heads * dh && ld % 8 == 0 && ld <= kMaxStride;
}

// A head tensor's bytes, first to last.
struct Span {
  const void* p;
  size_t n;
};
Span span(const void* p, int64_t T, int64_t ld, int64_t row, int io) {
  const size_t e = io == MHC_F32 ? 4 : 2;
  return {p, (size_t)((T - 1) * ld + row) * e};
}
Span bytes(const void* p, size_t n) { return {p, n}; }
bool meet(const Span& a, const Span& b) {
  if (a.p == nullptr || b.p == nullptr || a.n == 0 || b.n == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.n && y < x + a.n;
}
// Whether two head tensors share elements: side by side in the rows of one
// buffer (same stride) they do not, although their spans meet.
struct Heads {
  Span s;
  int64_t ld, row;
  size_t e;
};
Heads heads(const void* p, int64_t T, int64_t ld, int64_t row, int io) {
  return {span(p, T, ld, row, io), ld, row, io == MHC_F32 ? (size_t)4 : (size_t)2};
}
bool share(const Heads& a, const Heads& b) {
  if (!meet(a.s, b.s)) return false;
  if (a.ld != b.ld) return true;
  const int64_t pitch = a.ld * (int64_t)a.e;
  int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(b.s.p) - reinterpret_cast<uintptr_t>(a.s.p)) % pitch;
  if (d < 0) d += pitch;  // b's row starts d bytes after a row start of a
  return !(d >= a.row * (int64_t)a.e && d + b.row * (int64_t)b.e <= pitch);
}

mhc_status check_heads(int64_t T, int32_t Hq, int32_t Hk, int32_t io) {
  if (T < 0 || T > kMaxInt) return MHC_ERR_INVALID_ARG;
  if (io != MHC_F32 && io != MHC_BF16) return MHC_ERR_INVALID_ARG;
  if (Hq < 1 || Hk < 1 || Hq % Hk != 0 || Hq > 4096) return MHC_ERR_UNSUPPORTED;
  return MHC_OK;
}

mhc_status check_rope(const mhc_rope_desc* d) {
  if (d == nullptr) return MHC_ERR_INVALID_ARG;
  const mhc_status st = check_heads(d->T, d->Hq, d->Hk, d->io);
  if (st != MHC_OK) return st;
  if (!std::isfinite(d->eps) || d->eps < 0.f) return MHC_ERR_INVALID_ARG;
  if (d->Dh < 16 || d->Dh > 512 || d->Dh % 16 != 0) return MHC_ERR_UNSUPPORTED;
  if (d->R < 16 || d->R > d->Dh || d->R % 16 != 0) return MHC_ERR_UNSUPPORTED;
  return MHC_OK;
}

mhc_status check_scores(int32_t Dh, float scale, float softcap) {
  if (!std::isfinite(scale) || !(scale > 0.f) || !std::isfinite(softcap) || softcap < 0.f) return MHC_ERR_INVALID_ARG;
  return Dh == 64 || Dh == 128 ? MHC_OK : MHC_ERR_UNSUPPORTED;
}

mhc_status check_attn(const mhc_attn_desc* d) {
  if (d == nullptr) return MHC_ERR_INVALID_ARG;
  mhc_status st = check_heads(d->T, d->Hq, d->Hk, d->io);
  if (st == MHC_OK) st = check_scores(d->Dh, d->scale, d->softcap);
  if (st != MHC_OK) return st;
  if (d->window < 0 || (d->docs != nullptr && (d->n_docs < 1 || d->n_docs == kMaxInt))) return MHC_ERR_INVALID_ARG;
  if (!optional(d->docs, 4) || !optional(d->prefix, 4) || !optional(d->slopes, 4)) return MHC_ERR_INVALID_ARG;
  if (!d->causal && (d->window > 0 || d->prefix != nullptr)) return MHC_ERR_UNSUPPORTED;
  if (d->window > 0 && d->prefix != nullptr) return MHC_ERR_UNSUPPORTED;
  if ((d->T + 127) / 128 * d->Hq > kMaxInt) return MHC_ERR_UNSUPPORTED;
  return MHC_OK;
}

mhc_status check_paged(const mhc_paged_desc* d) {
  if (d == nullptr) return MHC_ERR_INVALID_ARG;
  mhc_status st = check_heads(d->T, d->Hq, d->Hk, d->io);
  if (st == MHC_OK) st = check_scores(d->Dh, d->scale, d->softcap);
  if (st != MHC_OK) return st;
  if (d->n_seqs < 0 || d->max_q < 1 || d->window < 0 || d->page_size < 1 || d->max_pages < 1 || d->num_pages < 1)
    return MHC_ERR_INVALID_ARG;
  if (d->cu_q == nullptr && (d->max_q != 1 || d->n_seqs > d->T)) return MHC_ERR_INVALID_ARG;
  if (!optional(d->cu_q, 4) || !optional(d->prefix, 4) || !optional(d->slopes, 4)) return MHC_ERR_INVALID_ARG;
  if (d->window > 0 && d->prefix != nullptr) return MHC_ERR_UNSUPPORTED;
  if (d->num_pages > kMaxInt / d->page_size || (int64_t)d->max_pages * d->page_size > kMaxInt) return MHC_ERR_UNSUPPORTED;
  // the grids: one workgroup per row tile, key head and split (at most 64), one
  // wave per row in the join
  const int64_t rows = (int64_t)d->max_q * (d->Hq / d->Hk), tiles = rows / 128 + 1;
  if (rows > kMaxInt || tiles > kMaxInt / 64 / d->Hk / (d->n_seqs > 0 ? d->n_seqs : 1)) return MHC_ERR_UNSUPPORTED;
  if ((int64_t)d->n_seqs * d->max_q > kMaxInt / d->Hq) return MHC_ERR_UNSUPPORTED;
  return MHC_OK;
}

}  // namespace

extern "C" {

mhc_status mhc_qk_rope(const mhc_rope_desc* d, const void* q, const void* k, const int32_t* positions,
                       const double* freqs, const float* q_weight, const float* k_weight, void* q_out, void* k_out,
                       hipStream_t stream) {
  const mhc_status st = check_rope(d);
  if (st != MHC_OK) return st;
  if (d->T == 0) return MHC_OK;
  const int64_t nq = (int64_t)d->Hq * d->Dh, nk = (int64_t)d->Hk * d->Dh;
  if (!stride_ok(d->ldq, d->Hq, d->Dh) || !stride_ok(d->ldk, d->Hk, d->Dh) || !stride_ok(d->ldq_out, d->Hq, d->Dh) ||
      !stride_ok(d->ldk_out, d->Hk, d->Dh))
    return MHC_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out) || !aligned(positions, 4) ||
      !aligned(freqs, 8) || !optional(q_weight, 16) || !optional(k_weight, 16))
    return MHC_ERR_INVALID_ARG;
  const Heads in[2] = {heads(q, d->T, d->ldq, nq, d->io), heads(k, d->T, d->ldk, nk, d->io)};
  const Heads out[2] = {heads(q_out, d->T, d->ldq_out, nq, d->io), heads(k_out, d->T, d->ldk_out, nk, d->io)};
  for (const Heads& o : out)
    for (const Heads& i : in)
      if (share(o, i)) return MHC_ERR_INVALID_ARG;
  if (share(out[0], out[1])) return MHC_ERR_INVALID_ARG;
  return from_hip(mhc::launch_qk_rope(*d, q, k, nullptr, positions, freqs, q_weight, k_weight, q_out, k_out, nullptr,
                                      nullptr, 0, stream));
}

size_t mhc_qk_rope_bwd_workspace_bytes(const mhc_rope_desc* d) {
  if (check_rope(d) != MHC_OK || d->T == 0) return 0;
  return mhc::qk_rope_bwd_workspace_bytes(*d);
}

mhc_status mhc_qk_rope_bwd(const mhc_rope_desc* d, const void* dq_out, const void* dk_out, const void* q,
                           const void* k, const int32_t* positions, const double* freqs, const float* q_weight,
                           const float* k_weight, void* dq, void* dk, float* dq_weight, float* dk_weight,
                           void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const mhc_status st = check_rope(d);
  if (st != MHC_OK) return st;
  if ((dq_weight != nullptr && q_weight == nullptr) || (dk_weight != nullptr && k_weight == nullptr) ||
      !optional(dq_weight, 16) || !optional(dk_weight, 16))
    return MHC_ERR_INVALID_ARG;
  if (d->T == 0) {  // sums over no tokens
    float* const w[2] = {dq_weight, dk_weight};
    for (float* p : w) {
      if (p == nullptr) continue;
      const hipError_t e = mhc::launch_fill_zero(p, (size_t)d->Dh, stream);
      if (e != hipSuccess) return from_hip(e);
    }
    return MHC_OK;
  }
  const int64_t nq = (int64_t)d->Hq * d->Dh, nk = (int64_t)d->Hk * d->Dh;
  if (!stride_ok(d->ldq, d->Hq, d->Dh) || !stride_ok(d->ldk, d->Hk, d->Dh) || !stride_ok(d->ldq_out, d->Hq, d->Dh) ||
      !stride_ok(d->ldk_out, d->Hk, d->Dh) || !stride_ok(d->ld_dq, d->Hq, d->Dh) || !stride_ok(d->ld_dk, d->Hk, d->Dh))
    return MHC_ERR_INVALID_ARG;
  if (!aligned16(dq_out) || !aligned16(dk_out) || !aligned16(q) || !aligned16(k) || !aligned16(dq) || !aligned16(dk) ||
      !aligned(positions, 4) || !aligned(freqs, 8) || !optional(q_weight, 16) || !optional(k_weight, 16))
    return MHC_ERR_INVALID_ARG;
  const Heads in[4] = {heads(q, d->T, d->ldq, nq, d->io), heads(k, d->T, d->ldk, nk, d->io),
                       heads(dq_out, d->T, d->ldq_out, nq, d->io), heads(dk_out, d->T, d->ldk_out, nk, d->io)};
  const Heads out[2] = {heads(dq, d->T, d->ld_dq, nq, d->io), heads(dk, d->T, d->ld_dk, nk, d->io)};
  for (const Heads& o : out) {
    for (const Heads& i : in)
      if (share(o, i)) return MHC_ERR_INVALID_ARG;
    if (meet(o.s, bytes(workspace, workspace_bytes))) return MHC_ERR_INVALID_ARG;
  }
  if (share(out[0], out[1])) return MHC_ERR_INVALID_ARG;
  if (!workspace_ok(workspace, workspace_bytes, mhc::qk_rope_bwd_workspace_bytes(*d))) return MHC_ERR_INVALID_ARG;
  return from_hip(mhc::launch_qk_rope_bwd(*d, dq_out, dk_out, q, k, positions, freqs, q_weight, k_weight, dq, dk,
                                          dq_weight, dk_weight, workspace, stream));
}

mhc_status mhc_qk_rope_cache(const mhc_rope_desc* d, const void* q, const void* k, const void* v,
                             const int32_t* positions, const double* freqs, const float* q_weight,
                             const float* k_weight, void* q_out, void* k_cache, void* v_cache, const int64_t* slots,
                             int64_t n_slots, hipStream_t stream) {
  const mhc_status st = check_rope(d);
  if (st != MHC_OK) return st;
  if (n_slots < 1 || n_slots > kMaxInt) return MHC_ERR_INVALID_ARG;
  if (d->T == 0) return MHC_OK;
  const int64_t nq = (int64_t)d->Hq * d->Dh, nk = (int64_t)d->Hk * d->Dh;
  if (!stride_ok(d->ldq, d->Hq, d->Dh) || !stride_ok(d->ldk, d->Hk, d->Dh) || !stride_ok(d->ldv, d->Hk, d->Dh) ||
      !stride_ok(d->ldq_out, d->Hq, d->Dh))
    return MHC_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(k_cache) ||
      !aligned16(v_cache) || !aligned(positions, 4) || !aligned(freqs, 8) || !aligned(slots, 8) ||
      !optional(q_weight, 16) || !optional(k_weight, 16))
    return MHC_ERR_INVALID_ARG;
  const Heads in[3] = {heads(q, d->T, d->ldq, nq, d->io), heads(k, d->T, d->ldk, nk, d->io),
                       heads(v, d->T, d->ldv, nk, d->io)};
  const Heads qo = heads(q_out, d->T, d->ldq_out, nq, d->io);
  const Span cache[2] = {span(k_cache, n_slots, nk, nk, d->io), span(v_cache, n_slots, nk, nk, d->io)};
  for (const Heads& i : in)
    if (share(qo, i) || meet(cache[0], i.s) || meet(cache[1], i.s)) return MHC_ERR_INVALID_ARG;
  if (meet(cache[0], cache[1]) || meet(cache[0], qo.s) || meet(cache[1], qo.s)) return MHC_ERR_INVALID_ARG;
  return from_hip(mhc::launch_qk_rope(*d, q, k, v, positions, freqs, q_weight, k_weight, q_out, k_cache, v_cache, slots,
                                      n_slots, stream));
}

mhc_status mhc_attn(const mhc_attn_desc* d, const void* q, const void* k, const void* v, void* o, float* lse,
                    void* o_rest, hipStream_t stream) {
  const mhc_status st = check_attn(d);
  if (st != MHC_OK) return st;
  if (d->T == 0) return MHC_OK;
  const int64_t nq = (int64_t)d->Hq * d->Dh, nk = (int64_t)d->Hk * d->Dh;
  if (!stride_ok(d->ldq, d->Hq, d->Dh) || !stride_ok(d->ldk, d->Hk, d->Dh) || !stride_ok(d->ldv, d->Hk, d->Dh) ||
      !stride_ok(d->ldo, d->Hq, d->Dh))
    return MHC_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !optional(lse, 16) || !optional(o_rest, 16))
    return MHC_ERR_INVALID_ARG;
  if (d->io == MHC_F32 && o_rest != nullptr) return MHC_ERR_INVALID_ARG;
  const Heads in[3] = {heads(q, d->T, d->ldq, nq, d->io), heads(k, d->T, d->ldk, nk, d->io),
                       heads(v, d->T, d->ldv, nk, d->io)};
  const Heads out = heads(o, d->T, d->ldo, nq, d->io);
  const Span l = bytes(lse, (size_t)d->Hq * d->T * 4), r = bytes(o_rest, (size_t)d->T * nq);
  if (meet(l, out.s) || meet(r, out.s) || meet(l, r)) return MHC_ERR_INVALID_ARG;
  for (const Heads& i : in)
    if (share(out, i) || meet(l, i.s) || meet(r, i.s)) return MHC_ERR_INVALID_ARG;
  return from_hip(mhc::launch_attn(*d, q, k, v, o, lse, o_rest, stream));
}

size_t mhc_attn_bwd_workspace_bytes(const mhc_attn_desc* d) {
  if (check_attn(d) != MHC_OK || d->T == 0) return 0;
  return mhc::attn_bwd_workspace_bytes(*d);
}

mhc_status mhc_attn_bwd(const mhc_attn_desc* d, const void* dout, const void* q, const void* k, const void* v,
                        const void* o, const float* lse, const void* o_rest, void* dq, void* dk, void* dv, void* workspace,
                        size_t workspace_bytes, hipStream_t stream) {
  const mhc_status st = check_attn(d);
  if (st != MHC_OK) return st;
  if (d->T == 0) return MHC_OK;
  const int64_t nq = (int64_t)d->Hq * d->Dh, nk = (int64_t)d->Hk * d->Dh;
  if (!stride_ok(d->ldq, d->Hq, d->Dh) || !stride_ok(d->ldk, d->Hk, d->Dh) || !stride_ok(d->ldv, d->Hk, d->Dh) ||
      !stride_ok(d->ldo, d->Hq, d->Dh) || !stride_ok(d->ld_do, d->Hq, d->Dh) || !stride_ok(d->ld_dq, d->Hq, d->Dh) ||
      !stride_ok(d->ld_dk, d->Hk, d->Dh) || !stride_ok(d->ld_dv, d->Hk, d->Dh))
    return MHC_ERR_INVALID_ARG;
  if (!aligned16(dout) || !aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse) ||
      !aligned16(dq) || !aligned16(dk) || !aligned16(dv) || !optional(o_rest, 16))
    return MHC_ERR_INVALID_ARG;
  if (d->io == MHC_F32 && o_rest != nullptr) return MHC_ERR_INVALID_ARG;
  const Heads in[5] = {heads(q, d->T, d->ldq, nq, d->io), heads(k, d->T, d->ldk, nk, d->io),
                       heads(v, d->T, d->ldv, nk, d->io), heads(o, d->T, d->ldo, nq, d->io),
                       heads(dout, d->T, d->ld_do, nq, d->io)};
  const Heads out[3] = {heads(dq, d->T, d->ld_dq, nq, d->io), heads(dk, d->T, d->ld_dk, nk, d->io),
                        heads(dv, d->T, d->ld_dv, nk, d->io)};
  const Span l = bytes(lse, (size_t)d->Hq * d->T * 4), ws = bytes(workspace, workspace_bytes);
  const Span r = bytes(o_rest, (size_t)d->T * nq);
  for (const Heads& x : out) {
    for (const Heads& i : in)
      if (share(x, i)) return MHC_ERR_INVALID_ARG;
    if (meet(x.s, l) || meet(x.s, ws) || meet(x.s, r)) return MHC_ERR_INVALID_ARG;
  }
  if (share(out[0], out[1]) || share(out[0], out[2]) || share(out[1], out[2])) return MHC_ERR_INVALID_ARG;
  for (const Heads& i : in)
    if (meet(i.s, ws)) return MHC_ERR_INVALID_ARG;
  if (meet(l, ws) || meet(r, ws)) return MHC_ERR_INVALID_ARG;
  if (!workspace_ok(workspace, workspace_bytes, mhc::attn_bwd_workspace_bytes(*d))) return MHC_ERR_INVALID_ARG;
  return from_hip(mhc::launch_attn_bwd(*d, dout, q, k, v, o, lse, o_rest, dq, dk, dv, workspace, stream));
}

size_t mhc_attn_paged_workspace_bytes(const mhc_paged_desc* d) {
  if (check_paged(d) != MHC_OK || d->T == 0 || d->n_seqs == 0) return 0;
  return mhc::attn_paged_workspace_bytes(*d);
}

mhc_status mhc_attn_paged(const mhc_paged_desc* d, const void* q, const void* k_cache, const void* v_cache, void* o,
                          void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const mhc_status st = check_paged(d);
  if (st != MHC_OK) return st;
  if (d->T == 0 || d->n_seqs == 0) return MHC_OK;
  const int64_t nq = (int64_t)d->Hq * d->Dh, nk = (int64_t)d->Hk * d->Dh;
  if (!stride_ok(d->ldq, d->Hq, d->Dh) || !stride_ok(d->ldo, d->Hq, d->Dh)) return MHC_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o) || !aligned(d->kv_lens, 4) ||
      !aligned(d->pages, 4))
    return MHC_ERR_INVALID_ARG;
  const Heads in = heads(q, d->T, d->ldq, nq, d->io), out = heads(o, d->T, d->ldo, nq, d->io);
  const int64_t n_slots = d->num_pages * d->page_size;
  const Span kc = span(k_cache, n_slots, nk, nk, d->io), vc = span(v_cache, n_slots, nk, nk, d->io);
  const Span ws = bytes(workspace, workspace_bytes);
  if (share(out, in) || meet(out.s, kc) || meet(out.s, vc)) return MHC_ERR_INVALID_ARG;
  if (meet(ws, in.s) || meet(ws, out.s) || meet(ws, kc) || meet(ws, vc)) return MHC_ERR_INVALID_ARG;
  if (!workspace_ok(workspace, workspace_bytes, mhc::attn_paged_workspace_bytes(*d))) return MHC_ERR_INVALID_ARG;
  return from_hip(mhc::launch_attn_paged(*d, q, k_cache, v_cache, o, workspace, stream));
}

}  // extern "C"
