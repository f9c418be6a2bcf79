// ops_api.cu -- entry points of the operators around the layer (declared in
// include/ittt.h): embedding lookup, layer norm, the gated delta rule, and
// their gradients.  Each validates its descriptors before anything is
// enqueued, takes its scratch and launches its kernels on the caller's stream.
#include <cmath>
#include <cstring>
#include <initializer_list>
#include <new>
#include <string>
#include <vector>

#include "host.h"
#include "ops.h"
#include "rows.cuh"

namespace {

using ittt::host_cuda_fail;
using ittt::host_fail;

bool is_float(int32_t dt) { return dt == ITTT_BF16 || dt == ITTT_FP32; }
int64_t size_of(int32_t dt) { return dt == ITTT_BF16 ? 2 : dt == ITTT_INT64 ? 8 : 4; }

enum Types { kFloats, kFp32Only, kBf16Only, kInts };

// A tensor of these dims whose last dimension is contiguous.  `dense`: every
// other dimension too (outputs and parameters); otherwise the leading strides
// are free, zero included (a broadcast view), but not negative.
ittt_status check(const ittt_tensor* t, const char* name, std::initializer_list<int64_t> shape,
                  Types types, bool dense) {
  if (t == nullptr) return host_fail(ITTT_ERR_INVALID_ARG, "%s: null descriptor", name);
  if (t->data == nullptr) return host_fail(ITTT_ERR_INVALID_ARG, "%s: null data pointer", name);
  const bool ok = types == kFloats ? is_float(t->dtype)
                  : types == kFp32Only ? t->dtype == ITTT_FP32
                  : types == kBf16Only ? t->dtype == ITTT_BF16
                                       : t->dtype == ITTT_INT32 || t->dtype == ITTT_INT64;
  if (!ok) return host_fail(ITTT_ERR_INVALID_ARG, "%s: unsupported dtype %d", name, int(t->dtype));
  if (t->ndim != int(shape.size()))
    return host_fail(ITTT_ERR_INVALID_ARG, "%s: expected %d dims, got %d", name,
                     int(shape.size()), int(t->ndim));
  int k = 0;
  for (int64_t want : shape) {
    if (t->shape[k] != want)
      return host_fail(ITTT_ERR_INVALID_ARG, "%s: dim %d is %lld, expected %lld", name, k,
                       (long long)t->shape[k], (long long)want);
    if (t->stride[k] < 0 && want > 1)
      return host_fail(ITTT_ERR_INVALID_ARG, "%s: negative stride in dim %d", name, k);
    ++k;
  }
  int64_t expect = 1;
  for (k = t->ndim - 1; k >= 0; --k) {
    if ((dense || k == t->ndim - 1) && t->shape[k] > 1 && t->stride[k] != expect)
      return host_fail(ITTT_ERR_INVALID_ARG, dense ? "%s: not dense row-major (dim %d stride %lld)"
                                                   : "%s: last dimension not contiguous (dim %d stride %lld)",
                       name, k, (long long)t->stride[k]);
    expect *= t->shape[k];
  }
  if (reinterpret_cast<uintptr_t>(t->data) % uintptr_t(size_of(t->dtype)) != 0)
    return host_fail(ITTT_ERR_INVALID_ARG, "%s: data pointer not aligned to its elements", name);
  return ITTT_OK;
}

// Bytes from the first to past the last element.
void extent(const ittt_tensor* t, uintptr_t* lo, uintptr_t* hi) {
  int64_t last = 0;
  for (int k = 0; k < t->ndim; ++k) last += (t->shape[k] - 1) * (t->shape[k] > 1 ? t->stride[k] : 0);
  *lo = reinterpret_cast<uintptr_t>(t->data);
  *hi = *lo + uintptr_t((last + 1) * size_of(t->dtype));
}

bool overlap(const ittt_tensor* a, const ittt_tensor* b) {
  if (a == nullptr || b == nullptr) return false;
  uintptr_t a0, a1, b0, b1;
  extent(a, &a0, &a1);
  extent(b, &b0, &b1);
  return a0 < b1 && b0 < a1;
}

// No output may overlap an input or another output.
ittt_status check_apart(std::initializer_list<const ittt_tensor*> writes,
                        std::initializer_list<const ittt_tensor*> reads) {
  for (const ittt_tensor* const* w = writes.begin(); w != writes.end(); ++w) {
    for (const ittt_tensor* r : reads)
      if (overlap(*w, r)) return host_fail(ITTT_ERR_INVALID_ARG, "an output overlaps an input");
    for (const ittt_tensor* const* v = writes.begin(); v != w; ++v)
      if (overlap(*w, *v)) return host_fail(ITTT_ERR_INVALID_ARG, "two output buffers overlap");
  }
  return ITTT_OK;
}

// Columns fill a grid's second dimension in pieces of 32 at least.
constexpr int64_t kMaxColumns = int64_t(1) << 20;

// Elements of the leading dimensions; `rows` views [N, d] or [B, T, d].
ittt_status row_count(const ittt_tensor* t, const char* name, int64_t* N, int64_t* d) {
  if (t == nullptr || (t->ndim != 2 && t->ndim != 3))
    return host_fail(ITTT_ERR_INVALID_ARG, "%s: expected an [N,d] or [B,T,d] descriptor", name);
  for (int k = 0; k < t->ndim; ++k)
    if (t->shape[k] <= 0)
      return host_fail(ITTT_ERR_INVALID_ARG, "%s: sizes must be positive", name);
  *d = t->shape[t->ndim - 1];
  for (int k = 0; k + 1 < t->ndim; ++k)
    if (t->shape[k] >= (int64_t(1) << 31))
      return host_fail(ITTT_ERR_UNSUPPORTED, "%s: 2^31 rows or 2^20 columns and more", name);
  *N = t->ndim == 2 ? t->shape[0] : t->shape[0] * t->shape[1];
  if (*N >= (int64_t(1) << 31) || *d >= kMaxColumns)
    return host_fail(ITTT_ERR_UNSUPPORTED, "%s: 2^31 rows or 2^20 columns and more", name);
  return ITTT_OK;
}

ittt_status check_rows(const ittt_tensor* t, const char* name, const ittt_tensor* like, Types types,
                       bool dense) {
  return like->ndim == 2
             ? check(t, name, {like->shape[0], like->shape[1]}, types, dense)
             : check(t, name, {like->shape[0], like->shape[1], like->shape[2]}, types, dense);
}

ittt::RowView rows(const ittt_tensor* t) {
  ittt::RowView v;
  v.data = t->data;
  v.fp32 = t->dtype == ITTT_FP32;
  v.T = t->shape[t->ndim - 2];
  v.stride_t = v.T > 1 ? t->stride[t->ndim - 2] : 0;
  v.stride_b = t->ndim == 3 && t->shape[0] > 1 ? t->stride[0] : 0;
  if (v.T == 1) {  // [B, 1, d]
    v.T = t->ndim == 3 ? t->shape[0] : 1;
    v.stride_t = v.stride_b;
  } else if (t->ndim == 3 && (t->shape[0] == 1 || v.stride_b == v.T * v.stride_t)) {
    v.T *= t->shape[0];  // evenly spaced rows
  }
  return v;
}

// ids are dense [N] or [B, T]; out or grad_out has one dimension more.
ittt_status check_ids(const ittt_tensor* ids, const ittt_tensor* rows_of, const char* name,
                      int64_t* N, int64_t* d) {
  ittt_status s;
  if ((s = row_count(rows_of, name, N, d))) return s;
  return rows_of->ndim == 2 ? check(ids, "ids", {rows_of->shape[0]}, kInts, true)
                            : check(ids, "ids", {rows_of->shape[0], rows_of->shape[1]}, kInts, true);
}

// ------------------------------------------------------ gated delta rule
ittt::HeadView heads(const ittt_tensor* t) {
  ittt::HeadView v;
  const int n = t->ndim;  // [B, T, H, D], or [B, H, D] for one token a sequence
  auto stride = [&](int k) { return t->shape[k] > 1 ? t->stride[k] : int64_t(0); };
  v.data = t->data;
  v.sb = stride(0);
  v.st = n == 4 ? stride(1) : 0;
  v.sh = stride(n - 2);
  const int64_t es = size_of(t->dtype);
  v.vec = ittt::aligned16(t->data) && (v.sb * es) % 16 == 0 && (v.st * es) % 16 == 0 &&
          (v.sh * es) % 16 == 0;
  return v;
}

ittt::GateView gates(const ittt_tensor* t) {
  auto stride = [&](int k) { return t->shape[k] > 1 ? t->stride[k] : int64_t(0); };
  ittt::GateView v;
  v.data = static_cast<const float*>(t->data);
  v.sb = stride(0);
  v.st = t->ndim == 3 ? stride(1) : 0;
  v.sh = stride(t->ndim - 1);
  return v;
}

// Gates may have any strides.
ittt_status check_gate(const ittt_tensor* t, const char* name, const ittt_tensor* v) {
  if (t == nullptr || t->data == nullptr)
    return host_fail(ITTT_ERR_INVALID_ARG, "%s: null descriptor or data pointer", name);
  if (t->dtype != ITTT_FP32)
    return host_fail(ITTT_ERR_INVALID_ARG, "%s: unsupported dtype %d", name, int(t->dtype));
  if (t->ndim != v->ndim - 1)
    return host_fail(ITTT_ERR_INVALID_ARG, "%s: expected %d dims, got %d", name, int(v->ndim) - 1,
                     int(t->ndim));
  for (int k = 0; k < t->ndim; ++k) {
    if (t->shape[k] != v->shape[k])
      return host_fail(ITTT_ERR_INVALID_ARG, "%s: dim %d is %lld, expected %lld", name, k,
                       (long long)t->shape[k], (long long)v->shape[k]);
    if (t->stride[k] < 0 && t->shape[k] > 1)
      return host_fail(ITTT_ERR_INVALID_ARG, "%s: negative stride in dim %d", name, k);
  }
  if (reinterpret_cast<uintptr_t>(t->data) % 4 != 0)
    return host_fail(ITTT_ERR_INVALID_ARG, "%s: data pointer not aligned to its elements", name);
  return ITTT_OK;
}

ittt_status check_delta_sizes(int64_t B, int64_t T, int64_t Hk, int64_t Hv, int64_t dk, int64_t dv) {
  if (B <= 0 || T <= 0 || Hk <= 0 || Hv <= 0)
    return host_fail(ITTT_ERR_INVALID_ARG, "sizes must be positive (B=%lld T=%lld Hk=%lld Hv=%lld)",
                     (long long)B, (long long)T, (long long)Hk, (long long)Hv);
  if (Hv % Hk != 0)
    return host_fail(ITTT_ERR_INVALID_ARG, "value heads %lld are not a multiple of key heads %lld",
                     (long long)Hv, (long long)Hk);
  if ((dk != 64 && dk != 128) || dv <= 0 || dv % 16 != 0 || dv > 512)
    return host_fail(ITTT_ERR_UNSUPPORTED,
                     "head sizes dk=%lld dv=%lld: dk must be 64 or 128, dv a multiple of 16 up to 512",
                     (long long)dk, (long long)dv);
  if (Hv > 65535 || B >= (int64_t(1) << 31) || T >= (int64_t(1) << 31) ||
      B * T >= (int64_t(1) << 31) || B * Hv * (dv / 16) >= (int64_t(1) << 31))
    return host_fail(ITTT_ERR_UNSUPPORTED, "sizes exceed 32-bit grids");
  return ITTT_OK;
}

// q, k, v, g, beta of a call; fills everything but the map, states and output.
ittt_status check_delta(const ittt_tensor* q, const ittt_tensor* k, const ittt_tensor* v,
                        const ittt_tensor* g, const ittt_tensor* beta, float scale, int ndim,
                        ittt::DeltaArgs* a) {
  ittt_status s;
  memset(static_cast<void*>(a), 0, sizeof(*a));
  if (q == nullptr || q->ndim != ndim || v == nullptr || v->ndim != ndim)
    return host_fail(ITTT_ERR_INVALID_ARG, "q and v: expected %s descriptors",
                     ndim == 4 ? "[B,T,H,dim]" : "[B,H,dim]");
  const int64_t B = v->shape[0], T = ndim == 4 ? v->shape[1] : 1, Hv = v->shape[ndim - 2],
                dv = v->shape[ndim - 1], Hk = q->shape[ndim - 2], dk = q->shape[ndim - 1];
  if ((s = check_delta_sizes(B, T, Hk, Hv, dk, dv))) return s;
  if ((s = ndim == 4 ? check(v, "v", {B, T, Hv, dv}, kFloats, false)
                     : check(v, "v", {B, Hv, dv}, kFloats, false)))
    return s;
  const Types same = v->dtype == ITTT_FP32 ? kFp32Only : kBf16Only;
  if ((s = ndim == 4 ? check(q, "q", {B, T, Hk, dk}, same, false)
                     : check(q, "q", {B, Hk, dk}, same, false)))
    return s;
  if ((s = ndim == 4 ? check(k, "k", {B, T, Hk, dk}, same, false)
                     : check(k, "k", {B, Hk, dk}, same, false)))
    return s;
  if ((s = check_gate(g, "g", v))) return s;
  if ((s = check_gate(beta, "beta", v))) return s;
  if (!std::isfinite(scale)) return host_fail(ITTT_ERR_INVALID_ARG, "scale is not finite");
  a->q = heads(q);
  a->k = heads(k);
  a->v = heads(v);
  a->g = gates(g);
  a->beta = gates(beta);
  a->fp32 = v->dtype == ITTT_FP32;
  a->B = int(B);
  a->T = int(T);
  a->Hk = int(Hk);
  a->Hv = int(Hv);
  a->dk = int(dk);
  a->dv = int(dv);
  a->scale = scale;
  return ITTT_OK;
}

// Sequences of a chunked call: their count, chunks, longest, and for packed
// documents the table (offsets, first chunks) that goes to the device.
struct DeltaDocs {
  int64_t S = 0, nchunks = 0, longest = 0;
  std::vector<int> table;
};
constexpr int64_t kMaxDeltaDocs = int64_t(1) << 22;

ittt_status delta_docs(const int64_t* cu, int64_t num_docs, int64_t B, int64_t T, DeltaDocs* d) {
  if (cu == nullptr) {
    if (num_docs != 0) return host_fail(ITTT_ERR_INVALID_ARG, "num_docs is set but cu_seqlens is NULL");
    d->S = B;
    d->nchunks = B * ((T + 63) / 64);
    d->longest = T;
    return ITTT_OK;
  }
  if (B != 1) return host_fail(ITTT_ERR_INVALID_ARG, "packed documents need B = 1 (got %lld)", (long long)B);
  if (num_docs < 1) return host_fail(ITTT_ERR_INVALID_ARG, "num_docs %lld must be >= 1", (long long)num_docs);
  if (num_docs > kMaxDeltaDocs)
    return host_fail(ITTT_ERR_UNSUPPORTED, "num_docs %lld is too large", (long long)num_docs);
  if (cu[0] != 0) return host_fail(ITTT_ERR_INVALID_ARG, "cu_seqlens[0] must be 0");
  if (cu[num_docs] != T)
    return host_fail(ITTT_ERR_INVALID_ARG, "cu_seqlens[num_docs] = %lld, expected T = %lld",
                     (long long)cu[num_docs], (long long)T);
  for (int64_t i = 0; i < num_docs; ++i)
    if (cu[i + 1] < cu[i] || cu[i + 1] > T)
      return host_fail(ITTT_ERR_INVALID_ARG, "cu_seqlens decreases at document %lld", (long long)i);
  d->S = num_docs;
  try {
    d->table.resize(size_t(2 * (num_docs + 1)));
  } catch (const std::bad_alloc&) {
    return host_fail(ITTT_ERR_OOM, "document table");
  }
  for (int64_t i = 0; i <= num_docs; ++i) {
    d->table[size_t(i)] = int(cu[i]);
    d->table[size_t(num_docs + 1 + i)] = int(d->nchunks);
    if (i < num_docs) {
      d->nchunks += (cu[i + 1] - cu[i] + 63) / 64;
      d->longest = cu[i + 1] - cu[i] > d->longest ? cu[i + 1] - cu[i] : d->longest;
    }
  }
  return ITTT_OK;
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

size_t table_bytes(int64_t num_docs) {
  return num_docs > 0 ? up256(size_t(2 * (num_docs + 1)) * sizeof(int)) : 0;
}

// Sequences up to this long run token by token: a token's step costs about a
// microsecond, a chunk of 64 some 20 us with its two launches.  Token by token /
// by chunk, us: 20 heads of 128 x 128: 8 tokens 12 / 18, 16 tokens 20 / 18,
// 24 tokens 27 / 18, 64 tokens 61 / 18; 64 sequences of 8 such heads: 8 tokens
// 39 / 66, 16 tokens 64 / 66, 20 tokens 78 / 68, 64 tokens 223 / 72.
constexpr int64_t kRecurrentTokens = 16;
bool chunked(const ittt::DeltaArgs& a, const DeltaDocs& d) {
  return !a.fp32 && d.longest > kRecurrentTokens;
}

// Stages the table at the start of the scratch and points the map at it.
ittt_status place_docs(const DeltaDocs& d, int64_t T, unsigned char* ws, cudaStream_t st,
                       ittt::DeltaArgs* a) {
  a->map.ndocs = int(d.S);
  a->map.nchunks = int(d.nchunks);
  a->map.T = int(T);
  a->map.n = int((T + 63) / 64);
  if (d.table.empty()) return ITTT_OK;
  int* table = reinterpret_cast<int*>(ws);
  const ittt_status s = ittt::host_stage_table(table, d.table.data(), d.table.size(), st);
  a->map.cu = table;
  a->map.base = table + (d.S + 1);
  return s;
}

}  // namespace

extern "C" {

size_t ittt_delta_workspace_bytes(int64_t B, int64_t T, int64_t Hv, int64_t num_docs) {
  if (B <= 0 || T <= 0 || Hv <= 0 || Hv > 65535 || num_docs < 0 || num_docs > kMaxDeltaDocs ||
      B >= (int64_t(1) << 31) || T >= (int64_t(1) << 31) || B * T >= (int64_t(1) << 31))
    return 0;
  // packed: every document may end in a partial chunk
  const int64_t chunks = num_docs > 0 ? T / 64 + num_docs : B * ((T + 63) / 64);
  return table_bytes(num_docs) + ittt::delta_scratch(chunks, int(Hv));
}

ittt_status ittt_delta_rule(const ittt_tensor* q, const ittt_tensor* k, const ittt_tensor* v,
                            const ittt_tensor* g, const ittt_tensor* beta, float scale,
                            ittt_tensor* out, ittt_stream_t stream, const ittt_delta_opts* opts) {
  ittt::host_clear_error();
  ittt_delta_opts o;
  memset(&o, 0, sizeof(o));
  if (opts) o = *opts;
  ittt_status s;
  ittt::DeltaArgs a;
  if ((s = check_delta(q, k, v, g, beta, scale, 4, &a))) return s;
  const int64_t B = a.B, T = a.T;
  if ((s = check(out, "out", {B, T, a.Hv, a.dv}, kFloats, true))) return s;
  if (!ittt::aligned16(out->data))
    return host_fail(ITTT_ERR_INVALID_ARG, "out: data pointer not 16-byte aligned");
  DeltaDocs d;
  if ((s = delta_docs(o.cu_seqlens, o.num_docs, B, T, &d))) return s;
  if (o.state_in && (s = check(o.state_in, "state_in", {d.S, a.Hv, a.dv, a.dk}, kFp32Only, true))) return s;
  if (o.state_out && (s = check(o.state_out, "state_out", {d.S, a.Hv, a.dv, a.dk}, kFp32Only, true))) return s;
  if ((o.state_in && !ittt::aligned16(o.state_in->data)) ||
      (o.state_out && !ittt::aligned16(o.state_out->data)))
    return host_fail(ITTT_ERR_INVALID_ARG, "state: data pointer not 16-byte aligned");
  if (d.S * a.Hv * (a.dv / 16) >= (int64_t(1) << 31))
    return host_fail(ITTT_ERR_UNSUPPORTED, "sizes exceed 32-bit grids");
  // in place: every warp reads its rows of the state before it writes them
  const bool in_place = o.state_in && o.state_out && o.state_in->data == o.state_out->data;
  if ((s = check_apart({out, o.state_out}, {q, k, v, g, beta}))) return s;
  if (overlap(out, o.state_in) || (!in_place && overlap(o.state_out, o.state_in)))
    return host_fail(ITTT_ERR_INVALID_ARG, "an output overlaps an input");
  const bool by_chunk = chunked(a, d);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const size_t table = table_bytes(o.cu_seqlens ? o.num_docs : 0);
  ittt::HostScratch ws;
  if ((s = ws.take(table + (by_chunk ? ittt::delta_scratch(d.nchunks, a.Hv) : 0), o.workspace,
                   o.workspace_bytes, st)))
    return s;
  ittt::LaunchEnv env;
  if ((s = ittt::host_env(st, &env))) return s;
  if ((s = place_docs(d, T, ws.base(), st, &a))) return s;
  a.state_in = o.state_in ? static_cast<const float*>(o.state_in->data) : nullptr;
  a.state_out = o.state_out ? static_cast<float*>(o.state_out->data) : nullptr;
  a.out = out->data;
  a.out_fp32 = out->dtype == ITTT_FP32;
  a.ws = ws.base() + table;
  const cudaError_t e =
      by_chunk ? ittt::launch_delta_chunked(env, a) : ittt::launch_delta_recurrent(env, a);
  return e == cudaSuccess ? ITTT_OK : host_cuda_fail(e, "delta rule launch");
}

size_t ittt_delta_grad_workspace_bytes(int64_t B, int64_t T, int64_t Hv, int64_t dk, int64_t dv,
                                       int64_t num_docs) {
  if (num_docs < 0 || num_docs > kMaxDeltaDocs) return 0;
  const std::string saved = ittt_last_error();
  if (check_delta_sizes(B, T, 1, Hv, dk, dv) != ITTT_OK) {
    ittt::set_last_error(saved.c_str());
    return 0;
  }
  const int64_t chunks = num_docs > 0 ? T / 64 + num_docs : B * ((T + 63) / 64);
  return table_bytes(num_docs) +
         ittt::delta_grad_scratch(chunks, int(Hv), int(dk), int(dv));
}

ittt_status ittt_delta_rule_grad(const ittt_tensor* q, const ittt_tensor* k, const ittt_tensor* v,
                                 const ittt_tensor* g, const ittt_tensor* beta,
                                 const ittt_tensor* grad_out, float scale, ittt_tensor* grad_q,
                                 ittt_tensor* grad_k, ittt_tensor* grad_v, ittt_tensor* grad_g,
                                 ittt_tensor* grad_beta, ittt_stream_t stream,
                                 const ittt_delta_grad_opts* opts) {
  ittt::host_clear_error();
  ittt_delta_grad_opts o;
  memset(&o, 0, sizeof(o));
  if (opts) o = *opts;
  ittt_status s;
  ittt::DeltaGradArgs a;
  ittt::DeltaArgs& f = a.f;
  if ((s = check_delta(q, k, v, g, beta, scale, 4, &f))) return s;
  if (f.fp32)
    return host_fail(ITTT_ERR_UNSUPPORTED, "the delta rule's gradient takes bf16 q, k and v");
  const int64_t B = f.B, T = f.T, Hk = f.Hk, Hv = f.Hv, dk = f.dk, dv = f.dv;
  if ((s = check(grad_out, "grad_out", {B, T, Hv, dv}, kBf16Only, false))) return s;
  if ((s = check(grad_q, "grad_q", {B, T, Hk, dk}, kBf16Only, true))) return s;
  if ((s = check(grad_k, "grad_k", {B, T, Hk, dk}, kBf16Only, true))) return s;
  if ((s = check(grad_v, "grad_v", {B, T, Hv, dv}, kBf16Only, true))) return s;
  if ((s = check(grad_g, "grad_g", {B, T, Hv}, kFp32Only, true))) return s;
  if ((s = check(grad_beta, "grad_beta", {B, T, Hv}, kFp32Only, true))) return s;
  DeltaDocs d;
  if ((s = delta_docs(o.cu_seqlens, o.num_docs, B, T, &d))) return s;
  const std::initializer_list<int64_t> states = {d.S, Hv, dv, dk};
  if (o.state_in && (s = check(o.state_in, "state_in", states, kFp32Only, true))) return s;
  if (o.grad_state_out && (s = check(o.grad_state_out, "grad_state_out", states, kFp32Only, true))) return s;
  if (o.grad_state_in && (s = check(o.grad_state_in, "grad_state_in", states, kFp32Only, true))) return s;
  for (const ittt_tensor* t : {static_cast<const ittt_tensor*>(grad_q), static_cast<const ittt_tensor*>(grad_k),
                               static_cast<const ittt_tensor*>(grad_v), o.state_in, o.grad_state_out,
                               static_cast<const ittt_tensor*>(o.grad_state_in)})
    if (t && !ittt::aligned16(t->data))
      return host_fail(ITTT_ERR_INVALID_ARG, "a gradient or state: data pointer not 16-byte aligned");
  if (d.S * Hv * (dv / 16) >= (int64_t(1) << 31) || Hk > 65535)
    return host_fail(ITTT_ERR_UNSUPPORTED, "sizes exceed 32-bit grids");
  if ((s = check_apart({grad_q, grad_k, grad_v, grad_g, grad_beta, o.grad_state_in},
                       {q, k, v, g, beta, grad_out, o.state_in, o.grad_state_out})))
    return s;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const size_t table = table_bytes(o.cu_seqlens ? o.num_docs : 0);
  ittt::HostScratch ws;
  if ((s = ws.take(table + ittt::delta_grad_scratch(d.nchunks, f.Hv, f.dk, f.dv), o.workspace,
                   o.workspace_bytes, st)))
    return s;
  ittt::LaunchEnv env;
  if ((s = ittt::host_env(st, &env))) return s;
  if ((s = place_docs(d, T, ws.base(), st, &f))) return s;
  f.state_in = o.state_in ? static_cast<const float*>(o.state_in->data) : nullptr;
  f.ws = ws.base() + table;
  a.dout = heads(grad_out);
  a.dstate_out = o.grad_state_out ? static_cast<const float*>(o.grad_state_out->data) : nullptr;
  a.dstate_in = o.grad_state_in ? static_cast<float*>(o.grad_state_in->data) : nullptr;
  a.dq = grad_q->data;
  a.dk = grad_k->data;
  a.dv = grad_v->data;
  a.dg = static_cast<float*>(grad_g->data);
  a.dbeta = static_cast<float*>(grad_beta->data);
  const cudaError_t e = ittt::launch_delta_grad(env, a);
  return e == cudaSuccess ? ITTT_OK : host_cuda_fail(e, "delta rule gradient launch");
}

ittt_status ittt_delta_step(const ittt_tensor* q, const ittt_tensor* k, const ittt_tensor* v,
                            const ittt_tensor* g, const ittt_tensor* beta, ittt_tensor* state,
                            const ittt_tensor* slots, float scale, ittt_tensor* out,
                            ittt_stream_t stream) {
  ittt::host_clear_error();
  ittt_status s;
  ittt::DeltaArgs a;
  if ((s = check_delta(q, k, v, g, beta, scale, 3, &a))) return s;
  if ((s = check(out, "out", {a.B, a.Hv, a.dv}, kFloats, true))) return s;
  if (state == nullptr || state->ndim != 4 || state->shape[0] <= 0)
    return host_fail(ITTT_ERR_INVALID_ARG, "state: expected an [S,Hv,dv,dk] descriptor");
  const int64_t S = state->shape[0];
  if ((s = check(state, "state", {S, a.Hv, a.dv, a.dk}, kFp32Only, true))) return s;
  if (!ittt::aligned16(state->data))
    return host_fail(ITTT_ERR_INVALID_ARG, "state: data pointer not 16-byte aligned");
  if (slots && (s = check(slots, "slots", {a.B}, kInts, true))) return s;
  if (!slots && S != a.B)
    return host_fail(ITTT_ERR_INVALID_ARG, "state: %lld rows for %d sequences and no slots",
                     (long long)S, a.B);
  if ((s = check_apart({out, state}, {q, k, v, g, beta, slots}))) return s;
  ittt::LaunchEnv env;
  if ((s = ittt::host_env(reinterpret_cast<cudaStream_t>(stream), &env))) return s;
  a.map.ndocs = a.B;
  a.map.nchunks = a.B;
  a.map.T = 1;
  a.map.n = 1;
  a.state_in = a.state_out = static_cast<float*>(state->data);
  a.slots = slots ? slots->data : nullptr;
  a.slots64 = slots && slots->dtype == ITTT_INT64;
  a.pool = S;
  a.out = out->data;
  a.out_fp32 = out->dtype == ITTT_FP32;
  const cudaError_t e = ittt::launch_delta_recurrent(env, a);
  return e == cudaSuccess ? ITTT_OK : host_cuda_fail(e, "delta step launch");
}

ittt_status ittt_embed(const ittt_tensor* ids, const ittt_tensor* table, float scale,
                       ittt_tensor* out, ittt_stream_t stream) {
  ittt::host_clear_error();
  ittt_status s;
  ittt::EmbedArgs a;
  if ((s = check_ids(ids, out, "out", &a.N, &a.d))) return s;
  if ((s = check_rows(out, "out", out, kFloats, true))) return s;
  if (table == nullptr || table->ndim != 2 || table->shape[0] <= 0)
    return host_fail(ITTT_ERR_INVALID_ARG, "table: expected a [V,d] descriptor");
  a.V = table->shape[0];
  if (a.V >= (int64_t(1) << 31) - 1) return host_fail(ITTT_ERR_UNSUPPORTED, "table: 2^31 rows and more");
  if ((s = check(table, "table", {a.V, a.d}, kFloats, true))) return s;
  if (!std::isfinite(scale)) return host_fail(ITTT_ERR_INVALID_ARG, "scale is not finite");
  if ((s = check_apart({out}, {ids, table}))) return s;
  ittt::LaunchEnv env;
  if ((s = ittt::host_env(reinterpret_cast<cudaStream_t>(stream), &env))) return s;
  a.ids = ids->data;
  a.ids64 = ids->dtype == ITTT_INT64;
  a.table = table->data;
  a.table_fp32 = table->dtype == ITTT_FP32;
  a.scale = scale;
  a.out = out->data;
  a.out_fp32 = out->dtype == ITTT_FP32;
  const cudaError_t e = ittt::launch_embed(env, a);
  return e == cudaSuccess ? ITTT_OK : host_cuda_fail(e, "embedding launch");
}

size_t ittt_embed_grad_workspace_bytes(int64_t N, int64_t d) {
  if (N <= 0 || d <= 0 || N >= (int64_t(1) << 31) || d >= kMaxColumns) return 0;
  return ittt::embed_grad_scratch(N, d);
}

ittt_status ittt_embed_grad(const ittt_tensor* ids, const ittt_tensor* grad_out, float scale,
                            int32_t accumulate, ittt_tensor* grad_table, void* workspace,
                            size_t workspace_bytes, ittt_stream_t stream) {
  ittt::host_clear_error();
  ittt_status s;
  ittt::EmbedGradArgs a;
  if ((s = check_ids(ids, grad_out, "grad_out", &a.N, &a.d))) return s;
  if ((s = check_rows(grad_out, "grad_out", grad_out, kFloats, false))) return s;
  if (grad_table == nullptr || grad_table->ndim != 2 || grad_table->shape[0] <= 0)
    return host_fail(ITTT_ERR_INVALID_ARG, "grad_table: expected a [V,d] descriptor");
  a.V = grad_table->shape[0];
  if (a.V >= (int64_t(1) << 31) - 1)
    return host_fail(ITTT_ERR_UNSUPPORTED, "grad_table: 2^31 rows and more");
  if ((s = check(grad_table, "grad_table", {a.V, a.d}, accumulate ? kFp32Only : kFloats, true)))
    return s;
  if (!ittt::aligned16(grad_table->data))
    return host_fail(ITTT_ERR_INVALID_ARG, "grad_table: data pointer not 16-byte aligned");
  if (!std::isfinite(scale)) return host_fail(ITTT_ERR_INVALID_ARG, "scale is not finite");
  if ((s = check_apart({grad_table}, {ids, grad_out}))) return s;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  ittt::HostScratch ws;
  if ((s = ws.take(ittt::embed_grad_scratch(a.N, a.d), workspace, workspace_bytes, st))) return s;
  ittt::LaunchEnv env;
  if ((s = ittt::host_env(st, &env))) return s;
  a.ids = ids->data;
  a.ids64 = ids->dtype == ITTT_INT64;
  a.dy = rows(grad_out);
  a.scale = scale;
  a.grad = grad_table->data;
  a.grad_fp32 = grad_table->dtype == ITTT_FP32;
  a.accumulate = accumulate != 0;
  a.ws = ws.base();
  const cudaError_t e = ittt::launch_embed_grad(env, a);
  return e == cudaSuccess ? ITTT_OK : host_cuda_fail(e, "embedding gradient launch");
}

ittt_status ittt_layer_norm(const ittt_tensor* x, const ittt_tensor* weight,
                            const ittt_tensor* bias, float eps, ittt_tensor* out,
                            ittt_tensor* mean, ittt_tensor* rstd, ittt_stream_t stream) {
  ittt::host_clear_error();
  ittt_status s;
  ittt::NormArgs a;
  if ((s = row_count(x, "x", &a.N, &a.d))) return s;
  if ((s = check_rows(x, "x", x, kFloats, false))) return s;
  if ((s = check(weight, "weight", {a.d}, kFloats, true))) return s;
  if (bias && (s = check(bias, "bias", {a.d}, kFloats, true))) return s;
  if ((s = check_rows(out, "out", x, kFloats, true))) return s;
  if (mean && (s = check(mean, "mean", {a.N}, kFp32Only, true))) return s;
  if (rstd && (s = check(rstd, "rstd", {a.N}, kFp32Only, true))) return s;
  if (!(eps >= 0.f) || !std::isfinite(eps))
    return host_fail(ITTT_ERR_INVALID_ARG, "eps must be finite and not negative");
  if ((s = check_apart({out, mean, rstd}, {x, weight, bias}))) return s;
  ittt::LaunchEnv env;
  if ((s = ittt::host_env(reinterpret_cast<cudaStream_t>(stream), &env))) return s;
  a.x = rows(x);
  a.weight = weight->data;
  a.w_fp32 = weight->dtype == ITTT_FP32;
  a.bias = bias ? bias->data : nullptr;
  a.b_fp32 = bias && bias->dtype == ITTT_FP32;
  a.eps = eps;
  a.out = out->data;
  a.out_fp32 = out->dtype == ITTT_FP32;
  a.mean = mean ? static_cast<float*>(mean->data) : nullptr;
  a.rstd = rstd ? static_cast<float*>(rstd->data) : nullptr;
  const cudaError_t e = ittt::launch_layer_norm(env, a);
  return e == cudaSuccess ? ITTT_OK : host_cuda_fail(e, "layer norm launch");
}

size_t ittt_layer_norm_grad_workspace_bytes(int64_t N, int64_t d) {
  if (N <= 0 || d <= 0 || N >= (int64_t(1) << 31) || d >= kMaxColumns) return 0;
  return ittt::layer_norm_grad_scratch(N, d);
}

ittt_status ittt_layer_norm_grad(const ittt_tensor* grad_out, const ittt_tensor* x,
                                 const ittt_tensor* weight, const ittt_tensor* mean,
                                 const ittt_tensor* rstd, ittt_tensor* grad_x,
                                 ittt_tensor* grad_weight, ittt_tensor* grad_bias, void* workspace,
                                 size_t workspace_bytes, ittt_stream_t stream) {
  ittt::host_clear_error();
  ittt_status s;
  ittt::NormGradArgs a;
  if ((s = row_count(x, "x", &a.N, &a.d))) return s;
  if ((s = check_rows(x, "x", x, kFloats, false))) return s;
  const Types same = x->dtype == ITTT_FP32 ? kFp32Only : kBf16Only;
  if ((s = check_rows(grad_out, "grad_out", x, same, false))) return s;
  if ((s = check(weight, "weight", {a.d}, kFloats, true))) return s;
  if ((s = check(mean, "mean", {a.N}, kFp32Only, true))) return s;
  if ((s = check(rstd, "rstd", {a.N}, kFp32Only, true))) return s;
  if (grad_x && (s = check_rows(grad_x, "grad_x", x, same, true))) return s;
  if (grad_weight && (s = check(grad_weight, "grad_weight", {a.d}, kFloats, true))) return s;
  if (grad_bias && (s = check(grad_bias, "grad_bias", {a.d}, kFloats, true))) return s;
  if (!grad_x && !grad_weight && !grad_bias)
    return host_fail(ITTT_ERR_INVALID_ARG, "no gradient asked for");
  if ((s = check_apart({grad_x, grad_weight, grad_bias}, {grad_out, x, weight, mean, rstd}))) return s;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  ittt::HostScratch ws;
  if ((s = ws.take(ittt::layer_norm_grad_scratch(a.N, a.d), workspace, workspace_bytes, st))) return s;
  ittt::LaunchEnv env;
  if ((s = ittt::host_env(st, &env))) return s;
  a.dy = rows(grad_out);
  a.x = rows(x);
  a.weight = weight->data;
  a.w_fp32 = weight->dtype == ITTT_FP32;
  a.mean = static_cast<const float*>(mean->data);
  a.rstd = static_cast<const float*>(rstd->data);
  a.dx = grad_x ? grad_x->data : nullptr;
  a.dw = grad_weight ? grad_weight->data : nullptr;
  a.dw_fp32 = grad_weight && grad_weight->dtype == ITTT_FP32;
  a.db = grad_bias ? grad_bias->data : nullptr;
  a.db_fp32 = grad_bias && grad_bias->dtype == ITTT_FP32;
  a.ws = reinterpret_cast<float*>(ws.base());
  const cudaError_t e = ittt::launch_layer_norm_grad(env, a);
  return e == cudaSuccess ? ITTT_OK : host_cuda_fail(e, "layer norm gradient launch");
}

}  // extern "C"
