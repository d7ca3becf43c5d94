// dckv_attention.cuh -- attention of new tokens over the paged cache (include/dckv_cache.h).
// Included by dckv.cu after dckv_cache.cuh.
#pragma once
#include "dckv_cache.cuh"

namespace dckv {

struct AttnDev {
  const char *q;
  char *out;
  float *lse;
  int64_t qt, qh, ot, oh;
  int64_t n;
  int heads, group, layer, causal;
  float scale;
  int32_t *status;
};

// One block per token, one warp per query head in turn; lane l holds dims l, l + 32, ...
// (the first, plain form: every row reads its keys and values by itself).
template <typename T, int D>
__global__ void __launch_bounds__(CACHE_THREADS) k_attend(const PoolDev p, const BatchDev bt, const AttnDev a) {
  __shared__ int shared_b;
  const int64_t t = blockIdx.x;
  const int b = find_sequence(bt, t, &shared_b);
  if (b < 0) return;
  const int64_t first = __ldg(bt.offsets + b), n = __ldg(bt.offsets + b + 1) - first;
  const int64_t len = __ldg(bt.kv_lens + b);
  if (n > bt.max_new || first < 0 || first + n > bt.n || len < 0 || len > (int64_t)bt.max_pages * p.page_size) {
    if (threadIdx.x == 0) atomicExch(a.status, DCKV_ERANGE);
    return;
  }
  const int64_t seen = a.causal ? len - n + (t - first) + 1 : len;
  const int lane = threadIdx.x & 31;
  constexpr int E = D / 32;
  for (int h = threadIdx.x >> 5; h < a.heads; h += CACHE_THREADS / 32) {
    const T *q = reinterpret_cast<const T *>(a.q) + t * a.qt + h * a.qh;
    const T *k = reinterpret_cast<const T *>(p.k) + a.layer * p.kl + (h / a.group) * p.kh;
    const T *v = reinterpret_cast<const T *>(p.v) + a.layer * p.vl + (h / a.group) * p.vh;
    float x[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      x[e] = to_f(q[lane + 32 * e]) * a.scale;
      o[e] = 0.f;
    }
    for (int64_t j = 0; j < seen; ++j) {
      int row;
      const int64_t page = slot_page(p, bt, b, j, row);
      if (page < 0) {
        if (lane == 0) atomicExch(a.status, DCKV_ERANGE);
        continue;
      }
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) s = fmaf(x[e], to_f(k[page * p.kp + row * p.kr + lane + 32 * e]), s);
      for (int w = 16; w; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
      const float top = fmaxf(m, s), keep = __expf(m - top), w = __expf(s - top);
      l = l * keep + w;
      m = top;
#pragma unroll
      for (int e = 0; e < E; ++e)
        o[e] = fmaf(w, to_f(v[page * p.vp + row * p.vr + lane + 32 * e]), o[e] * keep);
    }
    T *out = reinterpret_cast<T *>(a.out) + t * a.ot + h * a.oh;
#pragma unroll
    for (int e = 0; e < E; ++e) out[lane + 32 * e] = from_f<T>(l > 0.f ? o[e] / l : 0.f);
    if (a.lse && lane == 0) a.lse[t * a.heads + h] = l > 0.f ? m + logf(l) : -INFINITY;
  }
}

}  // namespace dckv

extern "C" size_t dckv_attention_workspace_bytes(const dckv_kv_pool *pool, const dckv_cache_batch *batch, int n_q_heads) {
  PoolDev p;
  BatchDev b;
  if (check_pool(pool, p) != DCKV_OK || check_batch(batch, 0, b) != DCKV_OK) return 0;
  if (n_q_heads < 1 || n_q_heads % p.heads) {
    fail(DCKV_EINVAL, "n_q_heads %d is not a multiple of the pool's heads", n_q_heads);
    return 0;
  }
  return 256;
}

extern "C" int dckv_attention(const dckv_kv_pool *pool, const dckv_cache_batch *batch, const dckv_attention_args *args,
                              int32_t *status, void *workspace, size_t ws_bytes, void *stream) {
  PoolDev p;
  BatchDev b;
  RET(check_pool(pool, p));
  RET(check_batch(batch, args ? args->n_tokens : 0, b));
  if (!args || !args->q || !args->out || !status || !workspace) return fail(DCKV_EINVAL, "a pointer argument is NULL");
  if (((uintptr_t)args->q & 15) || ((uintptr_t)args->out & 15) || ((uintptr_t)args->lse & 3) || ((uintptr_t)status & 3))
    return fail(DCKV_EINVAL, "q and out must be 16-byte, lse and status 4-byte aligned");
  if ((uintptr_t)workspace & 255) return fail(DCKV_EINVAL, "workspace must be 256-byte aligned");
  const int64_t n = args->n_tokens;
  const int hq = args->n_q_heads;
  if (n < 0 || n > 0x7fffffffll) return fail(DCKV_EINVAL, "n_tokens out of range");
  if (hq < 1 || hq > 65535 || hq % p.heads)
    return fail(DCKV_EINVAL, "n_q_heads %d is not a multiple of the pool's heads", hq);
  if (args->layer < 0 || args->layer >= p.n_layers) return fail(DCKV_EINVAL, "layer %d out of range", args->layer);
  if (args->causal != 0 && args->causal != 1) return fail(DCKV_EINVAL, "causal must be 0 or 1");
  if (!std::isfinite(args->scale) || !(args->scale > 0.f)) return fail(DCKV_EINVAL, "scale must be finite and positive");
  AttnDev a{(const char *)args->q, (char *)args->out, args->lse, args->q_token_stride, args->q_head_stride,
            args->out_token_stride, args->out_head_stride, n, hq, hq / p.heads, args->layer, args->causal, args->scale,
            status};
  if (bad_stride(a.qt, n, 8) || bad_stride(a.qh, hq, 8) || bad_stride(a.ot, n, 8) || bad_stride(a.oh, hq, 8))
    return fail(DCKV_EINVAL, "q and out strides must be positive multiples of 8 elements");
  if (n <= 1) a.qt = a.ot = 0;
  if (hq == 1) a.qh = a.oh = 0;
  if (n > 0 && overlaps(a.q, span_bytes(n, a.qt, hq, a.qh, p.dim, 2), a.out, span_bytes(n, a.ot, hq, a.oh, p.dim, 2)))
    return fail(DCKV_EINVAL, "out overlaps q");
  const size_t need = dckv_attention_workspace_bytes(pool, batch, hq);
  if (ws_bytes < need) return fail(DCKV_ECAPACITY, "workspace too small (%zu < %zu)", ws_bytes, need);
  if (n == 0) return DCKV_OK;
  cudaStream_t st = (cudaStream_t)stream;
  DEVICE_SCOPE(pool->device);
  const bool bf = pool->dtype == DCKV_BF16;
  const unsigned g = (unsigned)n;
  if (p.dim == 64) {
    if (bf) k_attend<__nv_bfloat16, 64><<<g, CACHE_THREADS, 0, st>>>(p, b, a);
    else k_attend<__half, 64><<<g, CACHE_THREADS, 0, st>>>(p, b, a);
  } else if (p.dim == 128) {
    if (bf) k_attend<__nv_bfloat16, 128><<<g, CACHE_THREADS, 0, st>>>(p, b, a);
    else k_attend<__half, 128><<<g, CACHE_THREADS, 0, st>>>(p, b, a);
  } else {
    if (bf) k_attend<__nv_bfloat16, 256><<<g, CACHE_THREADS, 0, st>>>(p, b, a);
    else k_attend<__half, 256><<<g, CACHE_THREADS, 0, st>>>(p, b, a);
  }
  ++g_launches;
  CK(cudaGetLastError());
  return DCKV_OK;
}
