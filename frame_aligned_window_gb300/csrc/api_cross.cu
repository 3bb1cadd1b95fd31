// C ABI of the attention to an encoder's states (declared in
// include/wsattn.h): argument checks, work split, tensor maps and launches.
#include <cmath>
#include <cstring>

#include "api_args.h"
#include "ops.h"

using wsattn::CrossParams;
using wsattn::CrossView;

namespace {

using namespace wsattn::args;

constexpr int64_t kMaxTokens = (int64_t(1) << 31) - 512;
// TMA strides are below 2^40 bytes.
constexpr int64_t kMaxStride = (int64_t(1) << 39) - 1;

bool scale_ok(float scale) { return scale > 0.f && std::isfinite(scale); }

template <typename A>
bool sizes_ok(const A* a) {
  return a && a->batch >= 0 && a->n_tokens >= 0 && a->n_tokens <= kMaxTokens && a->n_keys >= 0 &&
         a->n_keys <= kMaxTokens && scale_ok(a->scale) &&
         a->q.heads >= 1 && a->k.heads >= 1 && a->v.heads == a->k.heads &&
         a->q.heads % a->k.heads == 0 &&
         (reinterpret_cast<uintptr_t>(a->k_lengths) & 3u) == 0 &&
         (reinterpret_cast<uintptr_t>(a->lse) & 3u) == 0;
}
template <typename A>
bool supported(const A* a) {
  return half_type(a->dtype) && a->head_dim >= 16 && a->head_dim <= 128 && a->head_dim % 16 == 0;
}
// A view whose rows TMA can read (data may be null where there are no elements).
bool tma_view(const wsattn_heads* v, int heads, int batch, int64_t n) {
  auto stride = [](int64_t s, int64_t size) { return size <= 1 || (s % 8 == 0 && s <= kMaxStride); };
  return view_ok(v, 2) && v->heads == heads && aligned16(v->data) && stride(v->stride_b, batch) &&
         stride(v->stride_h, heads) && stride(v->stride_n, n);
}

CrossView view(const wsattn_heads* v) {
  return CrossView{v->data, v->stride_b, v->stride_h, v->stride_n};
}

template <typename A>
void fill_common(const A* a, CrossParams* p) {
  std::memset(p, 0, sizeof(*p));
  p->q = view(&a->q);
  p->k = view(&a->k);
  p->v = view(&a->v);
  p->o = view(&a->out);
  p->lengths = a->k_lengths;
  p->lse = const_cast<float*>(a->lse);
  p->batch = a->batch;
  p->heads = a->q.heads;
  p->kv_heads = a->k.heads;
  p->dim = a->head_dim;
  p->n = static_cast<int>(a->n_tokens);
  p->m = static_cast<int>(a->n_keys);
  p->scale = a->scale;
  p->scale_log2 = static_cast<float>(static_cast<double>(a->scale) * 1.4426950408889634074);
}

}  // namespace

extern "C" {

int wsattn_cross_workspace(const wsattn_cross_args* a, size_t* bytes) {
  if (!bytes || !sizes_ok(a)) return WSATTN_ERR_BAD_ARG;
  if (!supported(a)) return WSATTN_ERR_UNSUPPORTED;
  *bytes = 0;
  return WSATTN_OK;
}

int wsattn_cross(const wsattn_cross_args* a, void*, size_t, void* stream) {
  if (!sizes_ok(a)) return WSATTN_ERR_BAD_ARG;
  if (!supported(a)) return WSATTN_ERR_UNSUPPORTED;
  const int64_t n = a->n_tokens, m = a->n_keys;
  if (!tma_view(&a->q, a->q.heads, a->batch, n) || !tma_view(&a->k, a->k.heads, a->batch, m) ||
      !tma_view(&a->v, a->k.heads, a->batch, m) || !tma_view(&a->out, a->q.heads, a->batch, n) ||
      !apart(&a->out, a->batch, n, a->head_dim))
    return WSATTN_ERR_BAD_ARG;
  if (a->batch == 0 || n == 0) return WSATTN_OK;
  if (!a->q.data || !a->out.data || (m && (!a->k.data || !a->v.data))) return WSATTN_ERR_BAD_ARG;
  CrossParams p;
  fill_common(a, &p);
  p.status = wsattn::op_status_ptr();
  if (!p.status) return WSATTN_ERR_CUDA;
  return wsattn::launch_cross_forward(p, a->dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? WSATTN_OK
             : WSATTN_ERR_CUDA;
}

int wsattn_cross_backward_workspace(const wsattn_cross_grad_args* a, size_t* bytes) {
  if (!bytes || !sizes_ok(a)) return WSATTN_ERR_BAD_ARG;
  if (!supported(a)) return WSATTN_ERR_UNSUPPORTED;
  *bytes = 0;
  return WSATTN_OK;
}

int wsattn_cross_backward(const wsattn_cross_grad_args* a, void*, size_t, void* stream) {
  if (!sizes_ok(a)) return WSATTN_ERR_BAD_ARG;
  if (!supported(a)) return WSATTN_ERR_UNSUPPORTED;
  const int64_t n = a->n_tokens, m = a->n_keys;
  const int h = a->q.heads, e = a->k.heads, b = a->batch;
  if (!tma_view(&a->q, h, b, n) || !tma_view(&a->k, e, b, m) || !tma_view(&a->v, e, b, m) ||
      !tma_view(&a->out, h, b, n) || !tma_view(&a->dout, h, b, n))
    return WSATTN_ERR_BAD_ARG;
  const wsattn_heads* grads[3] = {&a->dq, &a->dk, &a->dv};
  for (int i = 0; i < 3; ++i)
    if (grads[i]->data &&
        (!tma_view(grads[i], i ? e : h, b, i ? m : n) || !apart(grads[i], b, i ? m : n, a->head_dim)))
      return WSATTN_ERR_BAD_ARG;
  if (b == 0 || (!a->dq.data && !a->dk.data && !a->dv.data)) return WSATTN_OK;
  if ((n && (!a->q.data || !a->out.data || !a->dout.data || !a->lse)) ||
      (n && m && (!a->k.data || !a->v.data)))
    return WSATTN_ERR_BAD_ARG;
  CrossParams p;
  fill_common(a, &p);
  p.dout = view(&a->dout);
  p.dq = view(&a->dq);
  p.dk = view(&a->dk);
  p.dv = view(&a->dv);
  p.status = wsattn::op_status_ptr();
  if (!p.status) return WSATTN_ERR_CUDA;
  return wsattn::launch_cross_backward(p, a->dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? WSATTN_OK
             : WSATTN_ERR_CUDA;
}

}  // extern "C"
