// dckv_cache.cuh -- rotary positions and the paged KV cache (include/dckv_cache.h): rotation of
// strided tensors, the append of new keys and values to the pages, and the read-back of pages
// as codec rows.  Included by dckv.cu (error text, device scope, launch count).
//
// All three move each element once and do 3 flops on it at most, so HBM bounds them on long
// inputs and the launch and a chain of dependent loads bound them on short ones.  A block takes one
// token: it looks its slot up and computes its (cos, sin) pairs once, into shared memory, and every
// head (and layer) reads them from there -- the angles cost about as much as the whole copy if each
// head repeats them.  Elements move as 16-byte vectors: a "chunk" is two vectors, the two halves of V
// pairs (half layout) or V whole pairs (interleaved layout).
// Blocks are small (128 threads) where there are many, so that some blocks' loads cover others'
// look-ups.  Measured on four 4,096-token prompts, six layers, 207 MB (appended without a rotation)
// and 258 MB (rows), before evict-first loads and chained launches (38 and 49 us with them): 128
// threads 41 and 53 us; 256 threads 45 and 59; a thread per chunk (384) 62 and 83; first chunk loaded
// before the look-up 48 and 58; four chunks ahead per thread 63 and 88; four tokens per block 44-52 and
// 56-63; blocks of one layer's keys or values 53-65 and 111-119.  These shapes were not measured on
// k_rope (4,096 tokens x 8 heads x 256 in bf16 10.5 us, 49% of the copy rate): the lanes of a
// head read their (cos, sin) pairs 64 bytes apart, eight addresses to a bank, and the loads of x wait
// for the angles.
#pragma once
#include "../../include/dckv_cache.h"
#include "dckv_epilogues.cuh"

namespace dckv {

constexpr int CACHE_THREADS = 256;       // of a block, at most
constexpr int CACHE_MANY_THREADS = 128;  // where the tokens fill the GPU
constexpr int CACHE_MANY_TOKENS = 2368;  // sixteen blocks per SM

// A rotation as the kernels take it (by value): mc and ms scale cos and sin (the magnitude, and
// for the transpose the sign of sin).
struct RopeDev {
  int r = 0;  // rotary_dim; 0: copy
  int interleaved = 0;
  float mc = 1.f, ms = 1.f;
  double turns[DCKV_ROPE_MAX_PAIRS] = {};  // freq / (2 pi): turns per position
};

// Division of n < 2^31 by a divisor known on the host, as a multiplication: with s = ceil(log2 d)
// and m = ceil(2^(31 + s) / d), n m exceeds n 2^(31 + s) / d by less than 2^(31 + s) / d.  (A
// hardware division is some 30 dependent instructions in 32 bits and a subroutine in 64; these
// kernels divide in their set-up, where every instruction is latency.)
struct FastDiv {
  uint32_t d = 1, m = 1u << 31;
  int s = 31;
  FastDiv() = default;
  explicit FastDiv(uint32_t div) : d(div) {
    int l = 0;
    while ((1ull << l) < div) ++l;
    s = 31 + l;
    m = (uint32_t)(((1ull << s) + div - 1) / div);
  }
  __device__ __forceinline__ int div(int n) const { return (int)(((uint64_t)(uint32_t)n * m) >> s); }
};

struct PoolDev {
  char *k, *v;
  int n_layers, heads, dim, page_size;
  FastDiv page_div;
  int64_t n_pages;
  int64_t kl, kp, kr, kh, vl, vp, vr, vh;  // element strides: layer, page, row, head
};

struct BatchDev {
  int batch, max_new, max_pages;
  int64_t n;  // rows of the call's token tensors
  const int32_t *offsets, *kv_lens, *page_table;
  int64_t table_stride;
};

// First in a kernel launched by launch_chained: the kernels before it in the stream are done.
__device__ __forceinline__ void wait_chained() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f(float v) { return v; }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }

// V consecutive elements: 16 bytes, or one element (odd sizes and alignments).
template <typename T, int V>
struct alignas(V * sizeof(T)) Vec {
  T e[V];
};

// A vector that is read once: 16 bytes are fetched evict-first (rows of four prompts 53 -> 51 us).
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> load_once(const T *p) {
  if constexpr (sizeof(Vec<T, V>) == 16) {
    const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(p));
    return *reinterpret_cast<const Vec<T, V> *>(&v);
  } else {
    return *reinterpret_cast<const Vec<T, V> *>(p);
  }
}

// Where chunk c of a rotated vector lies: its two V-element halves at off0 and off1 (off1 < 0:
// absent, the odd last element of a scalar copy).  The first r / (2 V) chunks are pairs, the
// rest copies.
template <int V>
__device__ __forceinline__ bool chunk_at(int c, int dim, const RopeDev &rope, int &off0, int &off1) {
  const int pair_chunks = rope.r / (2 * V);
  if (c < pair_chunks) {
    off0 = rope.interleaved ? 2 * c * V : c * V;
    off1 = rope.interleaved ? off0 + V : rope.r / 2 + c * V;
    return true;
  }
  off0 = rope.r + 2 * (c - pair_chunks) * V;
  off1 = off0 + V < dim ? off0 + V : -1;
  return false;
}

// Rotates the V pairs of chunk c in place, fp32, one rounding.  cs: the token's pairs.
template <typename T, int V>
__device__ __forceinline__ void rotate_chunk(Vec<T, V> &x0, Vec<T, V> &x1, const float2 *cs, int c, bool interleaved) {
  float u[2 * V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    u[j] = to_f(x0.e[j]);
    u[V + j] = to_f(x1.e[j]);
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const float2 w = cs[c * V + j];
    const float a = interleaved ? u[2 * j] : u[j], b = interleaved ? u[2 * j + 1] : u[V + j];
    const float a2 = a * w.x - b * w.y, b2 = b * w.x + a * w.y;
    if (interleaved) {
      u[2 * j] = a2;
      u[2 * j + 1] = b2;
    } else {
      u[j] = a2;
      u[V + j] = b2;
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    x0.e[j] = from_f<T>(u[j]);
    x1.e[j] = from_f<T>(u[V + j]);
  }
}

// One pair's (cos, sin) of the token at position pos, scaled as the mode asks.  The angle is counted
// in turns, in fp64, and its whole turns dropped there, which leaves an argument for sincospif that
// fp32 holds to 2^-25 turns or better.
__device__ __forceinline__ float2 rope_pair(const RopeDev &rope, int pos, int i) {
  const double t = (double)pos * rope.turns[i];
  float c, s;
  sincospif((float)(2.0 * (t - rint(t))), &s, &c);
  return make_float2(c * rope.mc, s * rope.ms);
}

// The (cos, sin) pairs of the block's token; all threads call it.
__device__ __forceinline__ void fill_pairs(const RopeDev &rope, float2 *cs, int pos) {
  for (int i = threadIdx.x; i < rope.r / 2; i += blockDim.x) cs[i] = rope_pair(rope, pos, i);
  __syncthreads();
}

// ------------------------------------------------------------------ rotation of a tensor
struct RopeArgs {
  const char *x;
  char *out;
  int64_t xt, xh, ot, oh;  // element strides: token, head
  int dim, chunks;         // chunks of a head that are moved (in place, dims past rotary_dim stand)
  FastDiv chunk_div;
  int per_token;           // heads * chunks
  const int32_t *positions;
};

template <typename T, int V>
__global__ void __launch_bounds__(CACHE_THREADS) k_rope(const __grid_constant__ RopeDev rope, const RopeArgs a) {
  __shared__ float2 cs[DCKV_ROPE_MAX_PAIRS];
  wait_chained();
  const int64_t t = blockIdx.x;
  fill_pairs(rope, cs, __ldg(a.positions + t));
  const T *x = reinterpret_cast<const T *>(a.x) + t * a.xt;
  T *out = reinterpret_cast<T *>(a.out) + t * a.ot;
  for (int i = threadIdx.x; i < a.per_token; i += blockDim.x) {
    const int h = a.chunk_div.div(i), c = i - h * a.chunks;
    int o0, o1;
    const bool turn = chunk_at<V>(c, a.dim, rope, o0, o1);
    Vec<T, V> x0 = load_once<T, V>(x + h * a.xh + o0), x1 = x0;
    if (o1 >= 0) x1 = load_once<T, V>(x + h * a.xh + o1);
    if (turn) rotate_chunk<T, V>(x0, x1, cs, c, rope.interleaved);
    *reinterpret_cast<Vec<T, V> *>(out + h * a.oh + o0) = x0;
    if (o1 >= 0) *reinterpret_cast<Vec<T, V> *>(out + h * a.oh + o1) = x1;
  }
}

// ------------------------------------------------------------------ tokens, sequences, slots
// Sequence of token t (-1: none), found by each warp for itself: a batch of up to four offsets per
// lane is scanned with one load latency, a larger one bisected.
__device__ __forceinline__ int find_sequence(const BatchDev &bt, int64_t t) {
  const int lane = threadIdx.x & 31;
  if (bt.batch <= 128) {
    int found = -1;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int b = lane + 32 * k;
      if (b < bt.batch && t >= __ldg(bt.offsets + b) && t < __ldg(bt.offsets + b + 1)) found = b;
    }
    return __reduce_max_sync(0xffffffffu, found);
  }
  int lo = 0, hi = bt.batch;  // last b with offsets[b] <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(bt.offsets + mid) <= t) lo = mid; else hi = mid;
  }
  return t >= __ldg(bt.offsets + lo) && t < __ldg(bt.offsets + lo + 1) ? lo : -1;
}

// Page of slot j (below 2^31) of sequence b, or -1 where the table or the pool ends before it.
__device__ __forceinline__ int64_t slot_page(const PoolDev &p, const BatchDev &bt, int b, int64_t j, int &row) {
  row = 0;
  if (j < 0) return -1;
  const int pi = p.page_div.div((int)j);
  row = (int)j - pi * p.page_size;
  if (pi >= bt.max_pages) return -1;
  const int page = __ldg(bt.page_table + b * bt.table_stride + pi);
  return page >= 0 && page < p.n_pages ? page : -1;
}

// Where a token's slot lies: page -1 where the token belongs to no sequence or is left out.
struct TokenSlot {
  int64_t page;
  int row, pos;
};

// Looks up token t; last: its slot counted from the sequence's end (append), else from its start.
__device__ __forceinline__ TokenSlot find_slot(const PoolDev &p, const BatchDev &bt, int64_t t, bool last,
                                               const int32_t *positions, int32_t *status) {
  TokenSlot s{-1, 0, 0};
  const int b = find_sequence(bt, t);
  if (b < 0) return s;
  const int64_t first = __ldg(bt.offsets + b), n = __ldg(bt.offsets + b + 1) - first, len = __ldg(bt.kv_lens + b);
  const int64_t j = last ? len - n + (t - first) : t - first;
  s.page = slot_page(p, bt, b, j, s.row);
  const bool ok = first >= 0 && first + n <= bt.n && (last ? n <= bt.max_new : j < len);
  if (!ok) s.page = -1;
  if (s.page < 0 && (threadIdx.x & 31) == 0) atomicExch(status, DCKV_ERANGE);
  s.pos = positions ? __ldg(positions + t) : (int)j;
  return s;
}

struct AppendDev {
  const char *k, *v, *q;
  char *q_out;
  int64_t kl, kt, kh, vl, vt, vh, qt, qh, ot, oh;
  int per_token;     // (2 layers * heads + q heads) * chunks
  FastDiv head_div;  // by the pool's heads
  const int32_t *positions;
  int32_t *status;
};

// One token: its keys of every layer and head (rotated), values (copied) and queries (rotated).
template <typename T, int V>
__global__ void __launch_bounds__(CACHE_THREADS)
    k_append(const __grid_constant__ RopeDev rope, const PoolDev p, const BatchDev bt, const AppendDev a) {
  __shared__ float2 cs[DCKV_ROPE_MAX_PAIRS];
  wait_chained();
  const int64_t t = blockIdx.x;
  const TokenSlot s = find_slot(p, bt, t, true, a.positions, a.status);
  if (s.page < 0) return;
  if (rope.r) fill_pairs(rope, cs, s.pos);
  const int shift = 31 - __clz(p.dim / (2 * V));  // chunks per vector: a power of two
  const int kv = p.n_layers * p.heads;
  for (int i = threadIdx.x; i < a.per_token; i += blockDim.x) {
    const int vec = i >> shift, c = i - (vec << shift);
    const T *src;
    T *dst;
    bool turn = true;
    if (vec < 2 * kv) {
      const bool is_v = vec >= kv;
      const int lh = is_v ? vec - kv : vec, l = a.head_div.div(lh), h = lh - l * p.heads;
      src = is_v ? reinterpret_cast<const T *>(a.v) + l * a.vl + t * a.vt + h * a.vh
                 : reinterpret_cast<const T *>(a.k) + l * a.kl + t * a.kt + h * a.kh;
      dst = is_v ? reinterpret_cast<T *>(p.v) + l * p.vl + s.page * p.vp + s.row * p.vr + h * p.vh
                 : reinterpret_cast<T *>(p.k) + l * p.kl + s.page * p.kp + s.row * p.kr + h * p.kh;
      turn = !is_v;
    } else {
      const int h = vec - 2 * kv;
      src = reinterpret_cast<const T *>(a.q) + t * a.qt + h * a.qh;
      dst = reinterpret_cast<T *>(a.q_out) + t * a.ot + h * a.oh;
    }
    int o0, o1;
    const bool pairs = chunk_at<V>(c, p.dim, rope, o0, o1);
    Vec<T, V> x0 = load_once<T, V>(src + o0), x1 = load_once<T, V>(src + o1);
    if (turn && pairs) rotate_chunk<T, V>(x0, x1, cs, c, rope.interleaved);
    *reinterpret_cast<Vec<T, V> *>(dst + o0) = x0;
    *reinterpret_cast<Vec<T, V> *>(dst + o1) = x1;
  }
}

struct RowsDev {
  char *rows;
  int64_t row_stride;
  int per_token;     // 2 layers * heads * chunks
  FastDiv head_div;
  const int32_t *positions;
  int32_t *status;
};

// One slot of a prompt as a row [layer][K, V][head][dim], keys rotated back.
template <typename T, int V>
__global__ void __launch_bounds__(CACHE_THREADS)
    k_rows(const __grid_constant__ RopeDev rope, const PoolDev p, const BatchDev bt, const RowsDev a) {
  __shared__ float2 cs[DCKV_ROPE_MAX_PAIRS];
  wait_chained();
  const int64_t t = blockIdx.x;
  const TokenSlot s = find_slot(p, bt, t, false, a.positions, a.status);
  if (s.page < 0) return;
  if (rope.r) fill_pairs(rope, cs, s.pos);
  const int shift = 31 - __clz(p.dim / (2 * V));
  T *row = reinterpret_cast<T *>(a.rows) + t * a.row_stride;
  for (int i = threadIdx.x; i < a.per_token; i += blockDim.x) {
    const int vec = i >> shift, c = i - (vec << shift);  // vec = (layer * 2 + v) * heads + head
    const int lv = a.head_div.div(vec), h = vec - lv * p.heads, l = lv >> 1;
    const bool is_v = lv & 1;
    const T *src = is_v ? reinterpret_cast<const T *>(p.v) + l * p.vl + s.page * p.vp + s.row * p.vr + h * p.vh
                        : reinterpret_cast<const T *>(p.k) + l * p.kl + s.page * p.kp + s.row * p.kr + h * p.kh;
    T *out = row + (int64_t)vec * p.dim;
    int o0, o1;
    const bool pairs = chunk_at<V>(c, p.dim, rope, o0, o1);
    Vec<T, V> x0 = load_once<T, V>(src + o0), x1 = load_once<T, V>(src + o1);
    if (!is_v && pairs) rotate_chunk<T, V>(x0, x1, cs, c, rope.interleaved);
    *reinterpret_cast<Vec<T, V> *>(out + o0) = x0;
    *reinterpret_cast<Vec<T, V> *>(out + o1) = x1;
  }
}

}  // namespace dckv

// ============================================================================ launches
// Launches with programmatic stream serialisation: a kernel's blocks are set up while the kernel
// before it in the stream ends, and wait for it (wait_chained) before they read or write global
// memory.  It is also the cheaper launch (1.9 against 2.7 us per call back to back).
static int launch_chained(const void *kern, dim3 grid, int threads, int smem, int cluster, cudaStream_t st, void **args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  CK(cudaLaunchKernelExC(&cfg, kern, args));
  ++g_launches;
  return DCKV_OK;
}

// ============================================================================ host checks
static int check_device(int device) {
  if (device < 0 || device >= 64) return fail(DCKV_EINVAL, "device %d out of range", device);
  return DCKV_OK;
}

static int check_spec(const dckv_rope_spec *s, int mode, RopeDev &d) {
  if (s->rotary_dim < 2 || s->rotary_dim > 2 * DCKV_ROPE_MAX_PAIRS || s->rotary_dim % 2)
    return fail(DCKV_EINVAL, "rotary_dim %d must be even, 2 .. %d", s->rotary_dim, 2 * DCKV_ROPE_MAX_PAIRS);
  if (s->layout != DCKV_ROPE_HALF && s->layout != DCKV_ROPE_INTERLEAVED)
    return fail(DCKV_EINVAL, "unknown rotary layout %d", s->layout);
  if (mode != DCKV_ROPE_FORWARD && mode != DCKV_ROPE_GRADIENT && mode != DCKV_ROPE_INVERSE)
    return fail(DCKV_EINVAL, "unknown rotary mode %d", mode);
  if (!(s->magnitude >= 0x1p-126) || !(s->magnitude <= 0x1p126))  // it and its inverse are normal fp32 numbers
    return fail(DCKV_EINVAL, "rotary magnitude must be within 2^-126 .. 2^126");
  for (int i = 0; i < s->rotary_dim / 2; ++i) {
    if (!std::isfinite(s->freq[i])) return fail(DCKV_EINVAL, "rotary frequency %d is not finite", i);
    d.turns[i] = s->freq[i] * 0.15915494309189535;  // 1 / (2 pi)
  }
  d.r = s->rotary_dim;
  d.interleaved = s->layout == DCKV_ROPE_INTERLEAVED;
  d.mc = (float)(mode == DCKV_ROPE_INVERSE ? 1.0 / s->magnitude : s->magnitude);
  d.ms = mode == DCKV_ROPE_FORWARD ? d.mc : -d.mc;
  return DCKV_OK;
}

// A stride counts only where its dimension has more than one entry.
static bool bad_stride(int64_t stride, int64_t extent, int64_t multiple) {
  return extent > 1 && (stride <= 0 || stride % multiple || stride >= ((int64_t)1 << 38));
}

static int check_pool(const dckv_kv_pool *p, PoolDev &d) {
  if (!p) return fail(DCKV_EINVAL, "pool is NULL");
  RET(check_device(p->device));
  if (!p->k || !p->v) return fail(DCKV_EINVAL, "a pool pointer is NULL");
  if (((uintptr_t)p->k & 15) || ((uintptr_t)p->v & 15)) return fail(DCKV_EINVAL, "pool must be 16-byte aligned");
  if (p->dtype != DCKV_BF16 && p->dtype != DCKV_FP16) return fail(DCKV_EINVAL, "pool type must be bf16 or fp16");
  if (p->head_dim != 64 && p->head_dim != 128 && p->head_dim != 256)
    return fail(DCKV_EINVAL, "head_dim %d must be 64, 128 or 256", p->head_dim);
  if (p->page_size < 16 || p->page_size > 65536 || p->page_size % 16)
    return fail(DCKV_EINVAL, "page_size %d must be a multiple of 16, 16 .. 65536", p->page_size);
  if (p->n_layers < 1 || p->n_layers > 65535 || p->n_kv_heads < 1 || p->n_kv_heads > 65535 ||
      (int64_t)p->n_layers * p->n_kv_heads > 65535)
    return fail(DCKV_EINVAL, "pool layers or heads out of range");
  if (p->n_pages < 1 || p->n_pages > 0x7fffffffll) return fail(DCKV_EINVAL, "n_pages out of range");
  if (bad_stride(p->k_layer_stride, p->n_layers, 8) || bad_stride(p->v_layer_stride, p->n_layers, 8) ||
      bad_stride(p->k_page_stride, p->n_pages, 8) || bad_stride(p->v_page_stride, p->n_pages, 8) ||
      bad_stride(p->k_row_stride, p->page_size, 8) || bad_stride(p->v_row_stride, p->page_size, 8) ||
      bad_stride(p->k_head_stride, p->n_kv_heads, 8) || bad_stride(p->v_head_stride, p->n_kv_heads, 8))
    return fail(DCKV_EINVAL, "pool strides must be positive multiples of 8 elements");
  d = PoolDev{(char *)p->k,       (char *)p->v,       p->n_layers,     p->n_kv_heads,   p->head_dim,
              p->page_size,       FastDiv((uint32_t)p->page_size), p->n_pages,         p->k_layer_stride, p->k_page_stride, p->k_row_stride,
              p->k_head_stride,   p->v_layer_stride,  p->v_page_stride, p->v_row_stride,  p->v_head_stride};
  return DCKV_OK;
}

static int check_batch(const dckv_cache_batch *b, int64_t n_tokens, BatchDev &d) {
  if (!b) return fail(DCKV_EINVAL, "batch is NULL");
  if (!b->offsets || !b->kv_lens || !b->page_table) return fail(DCKV_EINVAL, "a batch pointer is NULL");
  if (((uintptr_t)b->offsets & 3) || ((uintptr_t)b->kv_lens & 3) || ((uintptr_t)b->page_table & 3))
    return fail(DCKV_EINVAL, "batch arrays must be 4-byte aligned");
  if (b->batch < 1 || b->batch > DCKV_MAX_PROMPTS) return fail(DCKV_EINVAL, "batch %d out of range", b->batch);
  if (b->max_new < 1 || b->max_new > (1 << 30)) return fail(DCKV_EINVAL, "max_new %d out of range", b->max_new);
  if (b->max_pages < 1) return fail(DCKV_EINVAL, "max_pages must be positive");
  if (b->reserved != 0) return fail(DCKV_EINVAL, "reserved fields must be 0");
  if (b->batch > 1 && b->table_stride < b->max_pages)
    return fail(DCKV_EINVAL, "table_stride is smaller than max_pages");
  d = BatchDev{b->batch, b->max_new, b->max_pages, n_tokens, b->offsets, b->kv_lens, b->page_table, b->table_stride};
  return DCKV_OK;
}

// Bytes spanned by [n][heads][dim] with the given element strides (up to 2^38 each: 128 bits).
static unsigned __int128 span_bytes(int64_t n, int64_t ts, int64_t heads, int64_t hs, int64_t dim, int size) {
  return ((unsigned __int128)(n - 1) * ts + (unsigned __int128)(heads - 1) * hs + dim) * size;
}

static bool overlaps(const void *a, unsigned __int128 an, const void *b, unsigned __int128 bn) {
  return (uintptr_t)a < (uintptr_t)b + bn && (uintptr_t)b < (uintptr_t)a + an;
}

// Threads of a token's block: one per chunk up to a bound.
static int block_threads(int64_t n, int per_token) {
  const int most = n >= CACHE_MANY_TOKENS ? CACHE_MANY_THREADS : CACHE_THREADS;
  return std::min(most, (per_token + 31) / 32 * 32);
}

// Whole vectors of v elements: pair chunks, copy chunks and every address.
static bool rope_vectors(int r, int dim, int v) { return r % (2 * v) == 0 && (dim - r) % (2 * v) == 0; }

extern "C" int dckv_rope_init(dckv_rope_spec *out, int rotary_dim, int layout, double base, int scaling, double factor,
                              double original_len, double low, double high, double magnitude) {
  if (!out) return fail(DCKV_EINVAL, "out is NULL");
  if (!std::isfinite(base) || !(base > 1.0)) return fail(DCKV_EINVAL, "rotary base must be finite and above 1");
  if (scaling < DCKV_ROPE_NONE || scaling > DCKV_ROPE_PARTS) return fail(DCKV_EINVAL, "unknown rotary scaling %d", scaling);
  if (scaling != DCKV_ROPE_NONE && (!std::isfinite(factor) || !(factor > 0.0)))
    return fail(DCKV_EINVAL, "rotary factor must be finite and positive");
  if (scaling == DCKV_ROPE_NTK && rotary_dim <= 2) return fail(DCKV_EINVAL, "this scaling needs rotary_dim above 2");
  if (scaling == DCKV_ROPE_PARTS && (!(original_len > 0.0) || !std::isfinite(original_len) || !std::isfinite(low) ||
                                     !std::isfinite(high) || !(high > low)))
    return fail(DCKV_EINVAL, "this scaling needs original_len > 0 and high > low");
  dckv_rope_spec s = {};
  s.rotary_dim = rotary_dim;
  s.layout = layout;
  s.magnitude = magnitude;
  RopeDev d;
  RET(check_spec(&s, DCKV_ROPE_FORWARD, d));  // sizes, layout and magnitude (frequencies are still 0)
  const double b = scaling == DCKV_ROPE_NTK ? base * std::pow(factor, (double)rotary_dim / (rotary_dim - 2)) : base;
  if (!std::isfinite(b) || !(b > 0.0)) return fail(DCKV_EINVAL, "the scaled rotary base is out of range");
  for (int i = 0; i < rotary_dim / 2; ++i) {
    double f = std::pow(b, -2.0 * i / rotary_dim);
    if (scaling == DCKV_ROPE_LINEAR) f /= factor;
    if (scaling == DCKV_ROPE_PARTS) {
      const double turns = original_len * f / 6.283185307179586;
      const double w = std::min(1.0, std::max(0.0, (turns - low) / (high - low)));
      f *= w + (1.0 - w) / factor;
    }
    s.freq[i] = f;
  }
  *out = s;
  return DCKV_OK;
}

extern "C" int dckv_rope(const dckv_rope_spec *spec, int mode, const dckv_rope_args *args, void *stream) {
  if (!args) return fail(DCKV_EINVAL, "a pointer argument is NULL");
  const void *x = args->x;
  void *out = args->out;
  const int32_t *positions = args->positions;
  int64_t x_token_stride = args->x_token_stride, x_head_stride = args->x_head_stride;
  int64_t out_token_stride = args->out_token_stride, out_head_stride = args->out_head_stride;
  const int64_t n_tokens = args->n_tokens;
  const int n_heads = args->n_heads, head_dim = args->head_dim, dtype = args->dtype, device = args->device;
  if (!spec || !x || !out || !positions) return fail(DCKV_EINVAL, "a pointer argument is NULL");
  RET(check_device(device));
  RopeDev rope;
  RET(check_spec(spec, mode, rope));
  if (dtype != DCKV_BF16 && dtype != DCKV_FP16 && dtype != DCKV_FP32) return fail(DCKV_EINVAL, "unknown type %d", dtype);
  const int size = dtype == DCKV_FP32 ? 4 : 2;
  if (((uintptr_t)x & (size - 1)) || ((uintptr_t)out & (size - 1)) || ((uintptr_t)positions & 3))
    return fail(DCKV_EINVAL, "a tensor is not aligned to its elements");
  if (n_tokens < 0 || n_tokens > 0x7fffffffll || n_heads < 1 || n_heads > 65535)
    return fail(DCKV_EINVAL, "n_tokens or n_heads out of range");
  if (head_dim < rope.r || head_dim > 65536) return fail(DCKV_EINVAL, "head_dim %d out of range", head_dim);
  if (bad_stride(x_token_stride, n_tokens, 1) || bad_stride(x_head_stride, n_heads, 1) ||
      bad_stride(out_token_stride, n_tokens, 1) || bad_stride(out_head_stride, n_heads, 1))
    return fail(DCKV_EINVAL, "strides must be positive");
  if (n_tokens == 0) return DCKV_OK;
  const bool same = x == out && (n_tokens == 1 || x_token_stride == out_token_stride) &&
                    (n_heads == 1 || x_head_stride == out_head_stride);
  if (n_tokens == 1) x_token_stride = out_token_stride = 0;
  if (n_heads == 1) x_head_stride = out_head_stride = 0;
  if (!same && overlaps(x, span_bytes(n_tokens, x_token_stride, n_heads, x_head_stride, head_dim, size), out,
                        span_bytes(n_tokens, out_token_stride, n_heads, out_head_stride, head_dim, size)))
    return fail(DCKV_EINVAL, "out overlaps x without being x");
  const int v = 16 / size;
  const bool vec = rope_vectors(rope.r, head_dim, v) && !(((uintptr_t)x | (uintptr_t)out) & 15) &&
                   !((x_token_stride | x_head_stride | out_token_stride | out_head_stride) % v);
  const int vl = vec ? v : 1;
  const int chunks = rope.r / (2 * vl) + (same ? 0 : (head_dim - rope.r + 2 * vl - 1) / (2 * vl));
  const int64_t per_token = (int64_t)n_heads * chunks;
  if (per_token > 0x7fffffffll - 2 * CACHE_THREADS) return fail(DCKV_EINVAL, "n_heads times head_dim is too large");
  const RopeArgs a{(const char *)x, (char *)out, x_token_stride, x_head_stride, out_token_stride, out_head_stride,
                   head_dim, chunks, FastDiv((uint32_t)chunks), (int)per_token, positions};
  cudaStream_t st = (cudaStream_t)stream;
  DEVICE_SCOPE(device);
  const unsigned grid = (unsigned)n_tokens;
  const int threads = block_threads(n_tokens, (int)per_token);
  const void *kern = dtype == DCKV_FP32   ? (vec ? (const void *)k_rope<float, 4> : (const void *)k_rope<float, 1>)
                     : dtype == DCKV_FP16 ? (vec ? (const void *)k_rope<__half, 8> : (const void *)k_rope<__half, 1>)
                     : vec                ? (const void *)k_rope<__nv_bfloat16, 8>
                                          : (const void *)k_rope<__nv_bfloat16, 1>;
  void *kargs[] = {(void *)&rope, (void *)&a};
  return launch_chained(kern, dim3(grid), threads, 0, 1, st, kargs);
}

extern "C" int dckv_cache_append(const dckv_kv_pool *pool, const dckv_cache_batch *batch, const dckv_rope_spec *rope,
                                 const dckv_append_args *args, int32_t *status, void *stream) {
  PoolDev p;
  BatchDev b;
  RopeDev r;
  RET(check_pool(pool, p));
  RET(check_batch(batch, args ? args->n_tokens : 0, b));
  if (!args || !args->k || !args->v || !status) return fail(DCKV_EINVAL, "a pointer argument is NULL");
  if (((uintptr_t)args->k & 15) || ((uintptr_t)args->v & 15) || ((uintptr_t)status & 3) ||
      ((uintptr_t)args->positions & 3))
    return fail(DCKV_EINVAL, "k and v must be 16-byte, status and positions 4-byte aligned");
  if (rope) RET(check_spec(rope, DCKV_ROPE_FORWARD, r));
  if (r.r > p.dim) return fail(DCKV_EINVAL, "rotary_dim is larger than head_dim");
  const int64_t n = args->n_tokens;
  if (n < 0 || n > 0x7fffffffll) return fail(DCKV_EINVAL, "n_tokens out of range");
  if (args->reserved != 0) return fail(DCKV_EINVAL, "reserved fields must be 0");
  if (bad_stride(args->k_layer_stride, p.n_layers, 8) || bad_stride(args->k_token_stride, n, 8) ||
      bad_stride(args->k_head_stride, p.heads, 8) || bad_stride(args->v_layer_stride, p.n_layers, 8) ||
      bad_stride(args->v_token_stride, n, 8) || bad_stride(args->v_head_stride, p.heads, 8))
    return fail(DCKV_EINVAL, "k and v strides must be positive multiples of 8 elements");
  AppendDev a = {};
  a.k = (const char *)args->k;
  a.v = (const char *)args->v;
  a.kl = args->k_layer_stride, a.kt = args->k_token_stride, a.kh = args->k_head_stride;
  a.vl = args->v_layer_stride, a.vt = args->v_token_stride, a.vh = args->v_head_stride;
  a.qt = args->q_token_stride, a.qh = args->q_head_stride;
  a.ot = args->q_out_token_stride, a.oh = args->q_out_head_stride;
  a.positions = args->positions;
  a.status = status;
  int n_q_heads = 0;
  if (args->q) {
    const int hq = args->n_q_heads;
    if (!rope) return fail(DCKV_EINVAL, "q needs a rotation");
    if (!args->q_out) return fail(DCKV_EINVAL, "q_out is NULL");
    if (((uintptr_t)args->q & 15) || ((uintptr_t)args->q_out & 15))
      return fail(DCKV_EINVAL, "q and q_out must be 16-byte aligned");
    if (hq < 1 || hq > 65535) return fail(DCKV_EINVAL, "n_q_heads out of range");
    if (bad_stride(a.qt, n, 8) || bad_stride(a.qh, hq, 8) || bad_stride(a.ot, n, 8) || bad_stride(a.oh, hq, 8))
      return fail(DCKV_EINVAL, "q and q_out strides must be positive multiples of 8 elements");
    if (n <= 1) a.qt = a.ot = 0;
    if (hq == 1) a.qh = a.oh = 0;
    const bool same = args->q == args->q_out && a.qt == a.ot && a.qh == a.oh;
    if (n > 0 && !same && overlaps(args->q, span_bytes(n, a.qt, hq, a.qh, p.dim, 2), args->q_out,
                                   span_bytes(n, a.ot, hq, a.oh, p.dim, 2)))
      return fail(DCKV_EINVAL, "q_out overlaps q without being q");
    a.q = (const char *)args->q;
    a.q_out = (char *)args->q_out;
    n_q_heads = hq;
  }
  if (n == 0) return DCKV_OK;
  cudaStream_t st = (cudaStream_t)stream;
  DEVICE_SCOPE(pool->device);
  const bool vec = rope_vectors(r.r, p.dim, 8);
  a.per_token = (2 * p.n_layers * p.heads + n_q_heads) * (p.dim / (vec ? 16 : 2));
  a.head_div = FastDiv((uint32_t)p.heads);
  const unsigned grid = (unsigned)n;
  const int threads = block_threads(n, a.per_token);
  const void *bf = vec ? (const void *)k_append<__nv_bfloat16, 8> : (const void *)k_append<__nv_bfloat16, 1>;
  const void *hf = vec ? (const void *)k_append<__half, 8> : (const void *)k_append<__half, 1>;
  const void *kern = pool->dtype == DCKV_BF16 ? bf : hf;
  void *kargs[] = {(void *)&r, (void *)&p, (void *)&b, (void *)&a};
  return launch_chained(kern, dim3(grid), threads, 0, 1, st, kargs);
}

extern "C" int dckv_cache_rows(const dckv_kv_pool *pool, const dckv_cache_batch *batch, const dckv_rope_spec *rope,
                               void *rows, int64_t row_stride, int64_t n_tokens, const int32_t *positions,
                               int32_t *status, void *stream) {
  PoolDev p;
  BatchDev b;
  RopeDev r;
  RET(check_pool(pool, p));
  RET(check_batch(batch, n_tokens, b));
  if (!rows || !status) return fail(DCKV_EINVAL, "a pointer argument is NULL");
  if (((uintptr_t)rows & 15) || ((uintptr_t)status & 3) || ((uintptr_t)positions & 3))
    return fail(DCKV_EINVAL, "rows must be 16-byte, status and positions 4-byte aligned");
  if (rope) RET(check_spec(rope, DCKV_ROPE_INVERSE, r));
  if (r.r > p.dim) return fail(DCKV_EINVAL, "rotary_dim is larger than head_dim");
  if (n_tokens < 0 || n_tokens > 0x7fffffffll) return fail(DCKV_EINVAL, "n_tokens out of range");
  if (n_tokens > 1 && (row_stride % 8 || row_stride < (int64_t)2 * p.n_layers * p.heads * p.dim ||
                       row_stride >= ((int64_t)1 << 38)))
    return fail(DCKV_EINVAL, "row_stride must be a multiple of 8 and hold a row");
  if (n_tokens == 0) return DCKV_OK;
  cudaStream_t st = (cudaStream_t)stream;
  DEVICE_SCOPE(pool->device);
  const bool vec = rope_vectors(r.r, p.dim, 8);
  RowsDev a = {};
  a.rows = (char *)rows;
  a.row_stride = row_stride;
  a.per_token = 2 * p.n_layers * p.heads * (p.dim / (vec ? 16 : 2));
  a.head_div = FastDiv((uint32_t)p.heads);
  a.positions = positions;
  a.status = status;
  const unsigned grid = (unsigned)n_tokens;
  const int threads = block_threads(n_tokens, a.per_token);
  const void *bf = vec ? (const void *)k_rows<__nv_bfloat16, 8> : (const void *)k_rows<__nv_bfloat16, 1>;
  const void *hf = vec ? (const void *)k_rows<__half, 8> : (const void *)k_rows<__half, 1>;
  const void *kern = pool->dtype == DCKV_BF16 ? bf : hf;
  void *kargs[] = {(void *)&r, (void *)&p, (void *)&b, (void *)&a};
  return launch_chained(kern, dim3(grid), threads, 0, 1, st, kargs);
}
