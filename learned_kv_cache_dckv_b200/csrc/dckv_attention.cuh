// dckv_attention.cuh -- attention of new tokens over the paged cache (include/dckv_cache.h).
// Included by dckv.cu after dckv_cache.cuh.
//
// Mathematics.  With x_j = log2(e) scale q . k_j, a pass over any subset of a row's slots keeps
// m = max x_j, l = sum 2^(x_j - m) and O = sum 2^(x_j - m) v_j; two subsets join by scaling the
// one with the smaller m by 2^(m1 - m2).  So slots can be split anywhere: over warps, blocks and
// tiles, and the parts added at the end.
//
// Rows.  The g query heads of a KV head read the same keys, so a row tile packs (token, head of
// the group) pairs: packed row i of a sequence is token i / g, head i % g.  The pairs' tiles hold
// whole tokens (128 / g per CTA, the last rows idle where g does not divide 128).
//
// Work.  A unit is (KV head, sequence, row tile); its tiles are the key tiles that its last row
// sees.  The units' tiles stand in one line, head after head, and every block takes an equal,
// contiguous piece of that line, whatever the sequences' lengths: a piece that begins or ends
// inside a unit leaves its part (m, l, O) in the workspace, and a second kernel joins the parts.
// A block finds its piece by itself from the lengths on the device, so the host needs none.
#pragma once
#include "dckv_cache.cuh"

namespace dckv {

constexpr int ATTN_MAX_WORKERS = 160;  // workspace slots; at most one worker per SM

struct AttnDev {
  const char *q;
  char *out;
  float *lse;
  int64_t qt, qh, ot, oh;
  int heads, group, causal;
  FastDiv group_div;
  float scale_log2;
  int32_t *status;
  float4 *part_o;  // [2 workers][rows][dim / 4] (few rows) or [2 workers][dim / 4][rows] (many)
  float2 *part_ml; // [2 workers][rows] (m, l)
  int4 *desc;      // [workers][2]: a split unit that begins here {last worker (-1: none), rows, first
                   // token, first packed row}, {KV head, ...}
  int workers;
};

// What the kernels know of one sequence.
struct SeqView {
  int64_t first;  // first token
  int n, len;     // new tokens, slots in use
};

__device__ __forceinline__ bool load_seq(const BatchDev &bt, int64_t max_slots, int b, SeqView &s) {
  s.first = __ldg(bt.offsets + b);
  const int64_t n = (int64_t)__ldg(bt.offsets + b + 1) - s.first;
  s.len = __ldg(bt.kv_lens + b);
  s.n = (int)n;
  const bool ok = s.first >= 0 && n >= 0 && n <= bt.max_new && s.first + n <= bt.n && s.len >= 0 && s.len <= max_slots;
  if (!ok) s.n = s.len = 0;
  return ok;
}

// Slots that token t of the sequence sees.
__device__ __forceinline__ int seen_slots(const SeqView &s, int t, int causal) {
  return causal ? max(0, s.len - s.n + t + 1) : s.len;
}

// Slots that row tile rt sees (its last row's), -1 where it has no rows.  A sequence's packed
// rows number below 2^31 (checked on the host).
__device__ __forceinline__ int tile_seen(const SeqView &s, int rt, int rows, const AttnDev &a) {
  const int n_rows = s.n * a.group;
  if ((int64_t)rt * rows >= n_rows) return -1;
  const int last = min(n_rows - rt * rows, rows) - 1 + rt * rows;
  return seen_slots(s, a.group_div.div(last), a.causal);
}

// Key tiles of a unit; one that sees no slot still has one, to write its zeros.
__device__ __forceinline__ int unit_tiles(int seen, int key_tile) {
  return seen < 0 ? 0 : max(1, (int)(((uint32_t)seen + key_tile - 1) / (uint32_t)key_tile));
}

// A block's walk along the line of tiles: the current unit and the tiles [t0, t1) of it that
// the block takes.
struct AttnWalk {
  int64_t left;   // tiles of the block's piece from t0 on
  int head, unit; // unit = sequence * row tiles + row tile
  int b, rt;
  SeqView s;
  int seen, tiles, t0, t1;
};

struct AttnShape {
  int rows, key_tile, row_tiles, units, kv_heads;
  FastDiv unit_div;  // by row_tiles
  int64_t max_slots;
};

// Fills the walk's unit fields from (head, unit); t0 is given.
__device__ __forceinline__ void walk_load(AttnWalk &w, const BatchDev &bt, const AttnDev &a, const AttnShape &sh) {
  w.b = sh.unit_div.div(w.unit);
  w.rt = w.unit - w.b * sh.row_tiles;
  load_seq(bt, sh.max_slots, w.b, w.s);
  w.seen = tile_seen(w.s, w.rt, sh.rows, a);
  w.tiles = unit_tiles(w.seen, sh.key_tile);
  w.t1 = (int)min((int64_t)w.tiles, w.t0 + w.left);
}

// Steps to the next unit with tiles; false at the end of the piece.
__device__ __forceinline__ bool walk_next(AttnWalk &w, const BatchDev &bt, const AttnDev &a, const AttnShape &sh) {
  w.left -= w.t1 - w.t0;
  if (w.left <= 0) return false;
  w.t0 = 0;
  do {
    if (++w.unit == sh.units) {
      w.unit = 0;
      if (++w.head >= sh.kv_heads) return false;  // only if the lengths changed under the kernel
    }
    walk_load(w, bt, a, sh);
  } while (w.tiles == 0);
  return true;
}

// How the line is cut.  By default into equal pieces, wherever they begin and end (stream): no
// block waits for another, but a block may pass from unit to unit, which costs it the time of some
// tiles (the old unit's join or output, the new unit's Q).  Where every unit can be cut into equal
// parts of at most T tiles, one part per block, with T at most PLAN_TRIES - 1 steps (a tile, or a
// thirty-second of the piece) above the stream's piece, the parts win: five short ragged chunks took
// 37 us as a stream, 23 us in parts (with the chained launches of the same change).
constexpr int PLAN_TRIES = 4;

struct AttnPlanSmem {
  int64_t warp_sum[32];
  int warp_cnt[32][PLAN_TRIES];
  int unit, off;
};

struct AttnPlan {
  int64_t line;  // tiles of all units and heads
  int workers;   // blocks that take a piece
  int part;      // most tiles of a part; 0: stream
};

// a / b in 32 bits where both fit (64-bit division is a long subroutine).
__device__ __forceinline__ int64_t div_wide(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

// First tile of worker c's piece (stream).
__device__ __forceinline__ int64_t piece_start(const AttnPlan &pl, int c) {
  return div_wide((int64_t)c * pl.line, pl.workers);
}

// Last worker of the unit that begins in worker c's piece (w.t0 = 0).
__device__ __forceinline__ int last_worker(const AttnPlan &pl, const AttnWalk &w, int c) {
  if (pl.part) return c + (w.tiles + pl.part - 1) / pl.part - 1;
  const int64_t end = piece_start(pl, c + 1) - w.left + w.tiles;  // behind the unit's last tile
  return (int)div_wide(end * pl.workers + pl.line - 1, pl.line) - 1;
}

// Part number k of the walk's unit.
__device__ __forceinline__ void walk_part(AttnWalk &w, const AttnPlan &pl, const BatchDev &bt, const AttnDev &a,
                                          const AttnShape &sh, int k) {
  w.t0 = 0;
  w.left = 0x7fffffff;
  walk_load(w, bt, a, sh);
  const int n = (w.tiles + pl.part - 1) / pl.part;
  w.t0 = (int)((int64_t)w.tiles * k / n);
  w.t1 = (int)((int64_t)w.tiles * (k + 1) / n);
  w.left = w.t1 - w.t0;
}

// The plan of up to 32 units, made by each warp for itself, a unit per lane and in 32 bits: no
// barrier, one load latency and little code (its instructions are fetched cold on every call).
// Returns false where the numbers need the block's version below; any: c has a piece.
__device__ __forceinline__ bool warp_plan(const BatchDev &bt, const AttnDev &a, const AttnShape &sh, int tries, int c,
                                          AttnPlan &pl, AttnWalk &w, bool &any) {
  const int lane = threadIdx.x & 31;
  int t = 0;
  if (lane < sh.units) {
    const int b = sh.unit_div.div(lane);
    SeqView s;
    if (!load_seq(bt, sh.max_slots, b, s) && c == 0) atomicExch(a.status, DCKV_ERANGE);
    t = unit_tiles(tile_seen(s, lane - b * sh.row_tiles, sh.rows, a), sh.key_tile);  // below 2^26
  }
  const uint32_t total = __reduce_add_sync(0xffffffffu, (uint32_t)t);
  const uint64_t wide = (uint64_t)total * (uint32_t)sh.kv_heads;
  if (wide >= (1u << 24)) return false;  // line * workers stays below 2^32
  const uint32_t line = (uint32_t)wide, workers = max(1u, min((uint32_t)a.workers, line));
  pl.line = line;
  pl.workers = (int)workers;
  pl.part = 0;
  any = false;
  if (line == 0) return true;
  const uint32_t base = (line + workers - 1) / workers, step = max(1u, base >> 5);
  int mine = t;
  uint32_t pieces = 0;
#pragma unroll 1
  for (int j = 0; j < tries; ++j) {
    const uint32_t part = base + j * step, n = (t + part - 1) / part;
    pieces = __reduce_add_sync(0xffffffffu, n);
    if (pieces * sh.kv_heads <= (uint32_t)a.workers) {
      pl.part = (int)part;
      pl.workers = (int)(pieces * sh.kv_heads);
      mine = (int)n;
      break;
    }
  }
  if (c >= pl.workers) return true;
  // the worker's start along the line of a head's parts or tiles
  const uint32_t start = pl.part ? (uint32_t)c : (uint32_t)c * line / workers, period = pl.part ? pieces : total;
  w.head = (int)(start / period);
  const int pos = (int)(start - w.head * period);
  int at = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, at, o);
    if (lane >= o) at += v;
  }
  at -= mine;
  const int from = __ffs(__ballot_sync(0xffffffffu, pos >= at && pos < at + mine)) - 1;
  const int off = pos - __shfl_sync(0xffffffffu, at, from);
  w.unit = from;
  w.t0 = 0;
  w.left = 0x7fffffff;
  walk_load(w, bt, a, sh);
  if (pl.part) {
    const int n = (w.tiles + pl.part - 1) / pl.part;
    w.t0 = (int)((uint32_t)w.tiles * off / n);
    w.t1 = (int)((uint32_t)w.tiles * (off + 1) / n);
    w.left = w.t1 - w.t0;
  } else {
    w.t0 = off;
    w.left = (int)(((uint32_t)c + 1) * line / workers - start);
    w.t1 = (int)min((int64_t)w.tiles, w.t0 + w.left);
  }
  any = true;
  return true;
}

// Counts every unit's tiles (each thread a run of units, then a block scan), chooses the cut and
// finds worker c's start.  Called by all threads of the block; returns false where c has no piece.
// tries: cuts into parts to look at (1 .. PLAN_TRIES), part sizes from the stream's piece upwards.
template <int THREADS>
__device__ __forceinline__ bool attn_plan(const BatchDev &bt, const AttnDev &a, const AttnShape &sh, int tries, int c,
                                          AttnPlanSmem *sm, AttnPlan &pl, AttnWalk &w) {
  bool any;
  if (sh.units <= 32 && warp_plan(bt, a, sh, tries, c, pl, w, any)) return any;
  constexpr int WARPS = THREADS / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (sh.units + THREADS - 1) / THREADS;
  const int u0 = min(sh.units, tid * per), u1 = min(sh.units, u0 + per);
  int64_t mine = 0;
  int b = -1;
  SeqView s;
  auto tiles_of = [&](int u) {
    const int bu = sh.unit_div.div(u);
    if (bu != b) {
      b = bu;
      const bool ok = load_seq(bt, sh.max_slots, b, s);
      if (!ok && c == 0) atomicExch(a.status, DCKV_ERANGE);
    }
    return unit_tiles(tile_seen(s, u - b * sh.row_tiles, sh.rows, a), sh.key_tile);
  };
  int one = 0;  // the thread's tiles if it has a single unit
  for (int u = u0; u < u1; ++u) mine += one = tiles_of(u);
  int64_t incl = mine;
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) sm->warp_sum[warp] = incl;
  __syncthreads();
  int64_t before = 0, total = 0;
  for (int i = 0; i < WARPS; ++i) {
    const int64_t v = sm->warp_sum[i];
    if (i < warp) before += v;
    total += v;
  }
  pl.line = total * sh.kv_heads;
  pl.workers = (int)max((int64_t)1, min((int64_t)a.workers, pl.line));
  pl.part = 0;
  if (pl.line == 0) return false;
  // parts: sizes base, base + step, ...
  const int64_t base = div_wide(pl.line + pl.workers - 1, pl.workers);
  const int step = (int)max((int64_t)1, min(base >> 5, (int64_t)1 << 20));
  int cnt[PLAN_TRIES], scan[PLAN_TRIES], pieces = 0, pieces_before = 0;
  if (sh.units <= a.workers && base < (1 << 24)) {
#pragma unroll
    for (int j = 0; j < PLAN_TRIES; ++j) cnt[j] = 0;
    for (int u = u0; u < u1; ++u) {
      const int t = per == 1 ? one : tiles_of(u);
#pragma unroll
      for (int j = 0; j < PLAN_TRIES; ++j) {
        const uint32_t part = (uint32_t)base + j * step;
        cnt[j] += (int)((t + part - 1) / part);
      }
    }
#pragma unroll
    for (int j = 0; j < PLAN_TRIES; ++j) {
      scan[j] = cnt[j];
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, scan[j], o);
        if (lane >= o) scan[j] += v;
      }
      if (lane == 31) sm->warp_cnt[warp][j] = scan[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < PLAN_TRIES; ++j) {
      int sum = 0, bef = 0;
      for (int i = 0; i < WARPS; ++i) {
        const int v = sm->warp_cnt[i][j];
        if (i < warp) bef += v;
        sum += v;
      }
      if (j < tries && pl.part == 0 && (int64_t)sum * sh.kv_heads <= a.workers) {
        pl.part = (int)base + j * step;
        pieces = sum;
        pieces_before = bef + scan[j] - cnt[j];
      }
    }
  }
  if (pl.part) {
    pl.workers = pieces * sh.kv_heads;
    if (c >= pl.workers) return false;
    w.head = c / pieces;
    const int pos = c - w.head * pieces;
    int at = pieces_before;
    for (int u = u0; u < u1; ++u) {  // the unit of this worker, in one thread's run
      const int n = (tiles_of(u) + pl.part - 1) / pl.part;
      if (pos >= at && pos < at + n) {
        sm->unit = u;
        sm->off = pos - at;
      }
      at += n;
    }
    __syncthreads();
    w.unit = sm->unit;
    walk_part(w, pl, bt, a, sh, sm->off);
    return true;
  }
  if (c >= pl.workers) return false;
  const int64_t start = piece_start(pl, c);
  w.left = piece_start(pl, c + 1) - start;
  w.head = (int)div_wide(start, total);
  const int64_t pos = start - w.head * total;
  int64_t at = before + incl - mine;
  if (pos >= at && pos < at + mine) {  // the start lies in this thread's run: walk it
    int u = u0;
    for (; u < u1; ++u) {
      const int t = tiles_of(u);
      if (pos < at + t) break;
      at += t;
    }
    sm->unit = u;
    sm->off = (int)(pos - at);
  }
  __syncthreads();
  w.unit = sm->unit;
  w.t0 = sm->off;
  walk_load(w, bt, a, sh);
  return true;
}

// A row's lse from its reference (log2 units) and its sum: -infinity where it saw no slot, NaN where its
// scores held one.
__device__ __forceinline__ float row_lse(float ref, float sum) {
  return sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
}

// ------------------------------------------------------------------ math helpers
__device__ __forceinline__ float exp2_fast(float x) {  // 2 ulp and flush to zero (PTX ex2.approx.ftz)
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 values in one register pair, and sm_100's packed arithmetic on them.
__device__ __forceinline__ uint64_t f2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 un2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.ftz.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.ftz.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Weights are rounded to the cache's type before they multiply V (the tensor cores take no more), each
// relative to itself as long as it is a normal number there.  bf16 has fp32's range, but fp16 ends at
// 2^-14: of weights relative to a row's largest, those below 2^-25 would vanish and those above lose
// bits, and thousands of slots of them count beside one large score.  So in fp16 the reference lies
// below the largest score, and the weights reach up to 2^15, just under its largest number: 2^-25 is
// then 2^-40 of the largest weight for few rows, and 2^-32 or less for the pairs, whose largest may
// first grow by RESCALE_STEPS.
template <typename T>
constexpr float weight_head(float slack) {  // log2 of the largest weight when the reference is set
  return std::is_same<T, __half>::value ? 15.f - slack : 0.f;
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <typename T>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma_16816<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma_16816<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// Where a unit's row r goes: token and query head; false past its last row.
__device__ __forceinline__ bool unit_row(const AttnWalk &w, const AttnDev &a, int rows, int r, int64_t &tok, int &head,
                                         int &seen) {
  const int i = w.rt * rows + r;
  if (i >= w.s.n * a.group) return false;
  const int t = a.group_div.div(i);
  tok = w.s.first + t;
  head = w.head * a.group + i - t * a.group;
  seen = seen_slots(w.s, t, a.causal);
  return true;
}

// The join's description of a split unit that begins in worker c's piece.
__device__ __forceinline__ void describe(const AttnDev &a, const AttnPlan &pl, const AttnWalk &w, int c, int rows) {
  a.desc[2 * c + 1] = make_int4(w.head, 0, 0, 0);
  a.desc[2 * c] = make_int4(last_worker(pl, w, c), min(rows, w.s.n * a.group - w.rt * rows), (int)w.s.first, w.rt * rows);
}

template <typename T>
__device__ __forceinline__ void store4(T *dst, float4 v) {
  uint2 p = make_uint2(pack2<T>(v.x, v.y), pack2<T>(v.z, v.w));
  *reinterpret_cast<uint2 *>(dst) = p;
}

// ------------------------------------------------------------------ few rows: one warp, 16 keys
// Rows 8 NT at most (single tokens of up to 8 or 16 query heads per KV head).  Every K and V byte is
// used for 8 or 16 rows only, so HBM bounds it; the kernel's shape keeps as many loads in flight
// as shared memory holds and no barrier in the loop.  Each of four warps runs its own ring of
// stages (a slice of 16 keys: K and V, fetched by TMA with the 128-byte swizzle) and its own
// (m, l, O), and the four are joined in shared memory at a unit's end.  mma.sync with the keys
// as the M dimension: S^T = K Q^T and O^T = V^T P^T, so that 8 rows fill the N dimension that
// would be padded to 16 (or 128) as M; P^T goes from accumulators to the second product's
// operand through movmatrix.
constexpr int DEC_ATTN_WARPS = 4;
constexpr int DEC_ATTN_THREADS = 32 * DEC_ATTN_WARPS;
constexpr int DEC_SLICE = 16;
constexpr int DEC_KEY_TILE = DEC_SLICE * DEC_ATTN_WARPS;

template <int D, int NT>
struct DecodeAttn {
  static constexpr int ROWS = 8 * NT;
  static constexpr int SLICE_BYTES = DEC_SLICE * D * 2;
  static constexpr int STAGE_BYTES = 2 * SLICE_BYTES;  // K, V
  static constexpr int O_LD = D + 4;                   // floats per row of the join buffer (conflict-free)
  static constexpr int JOIN_BYTES = DEC_ATTN_WARPS * ROWS * (O_LD * 4 + 8);
  static constexpr int FIT = (232448 - 2048 - JOIN_BYTES) / (DEC_ATTN_WARPS * STAGE_BYTES);
  static constexpr int STAGES = FIT > 8 ? 8 : FIT;
  static constexpr int SMEM = 1024 + DEC_ATTN_WARPS * STAGES * STAGE_BYTES + JOIN_BYTES;
  static_assert(STAGES >= 2 && SMEM <= 232448 - 1024, "shared memory");
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(DEC_ATTN_THREADS, 1)
    k_attend_few(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const PoolDev p,
                 const BatchDev bt, const AttnDev a, const AttnShape sh) {
  using C = DecodeAttn<D, NT>;
  extern __shared__ __align__(1024) uint8_t dyn_smem[];
  __shared__ AttnPlanSmem plan_sm;
  __shared__ uint64_t full[DEC_ATTN_WARPS][C::STAGES][2];
  __shared__ int abort_sm;
  uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(dyn_smem) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t *ring = base + warp * C::STAGES * C::STAGE_BYTES;
  float *join_o = reinterpret_cast<float *>(base + DEC_ATTN_WARPS * C::STAGES * C::STAGE_BYTES);
  float2 *join_ml = reinterpret_cast<float2 *>(join_o + DEC_ATTN_WARPS * C::ROWS * C::O_LD);
  volatile int *abort_flag = &abort_sm;

  if (lane == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[warp][s][0], 1);
      mbar_init(&full[warp][s][1], 1);
    }
    if (warp == 0) {
      abort_sm = 0;
      prefetch_tmap(&tm_k);
      prefetch_tmap(&tm_v);
    }
    fence_mbar_init();
  }
  __syncthreads();  // the abort flag is set
  wait_chained();
  AttnPlan pl;
  AttnWalk w;
  const int c = blockIdx.x;
  const bool any = attn_plan<DEC_ATTN_THREADS>(bt, a, sh, 2, c, &plan_sm, pl, w);
  if (threadIdx.x == 0) a.desc[2 * c] = make_int4(-1, 0, 0, 0);
  if (!any) return;
  __syncwarp();

  // the producer's walk runs ahead of the consumer's: same slices, STAGES of them in flight
  AttnWalk pw = w;
  int pt = pw.t0;           // next tile of the producer
  bool more = true;
  uint32_t issued = 0, used = 0;
  auto slice_key = [&](int t) { return t * DEC_KEY_TILE + warp * DEC_SLICE; };
  bool ok = true;
  auto produce = [&]() {  // issues the next slice of this warp, if there is one
    while (more && ok) {
      if (pt >= pw.t1) {
        more = walk_next(pw, bt, a, sh);
        pt = pw.t0;
        continue;
      }
      const int key = slice_key(pt++);
      if (key >= pw.seen) continue;
      if (lane == 0) {
        const int pi = p.page_div.div(key);
        int page = __ldg(bt.page_table + pw.b * bt.table_stride + pi);
        if (page < 0 || page >= p.n_pages) {  // past the pool: the copy fills zeros
          atomicExch(a.status, DCKV_ERANGE);
          page = (int)p.n_pages;
        }
        const int row = key - pi * p.page_size;
        const uint32_t s = issued % C::STAGES;
        uint8_t *dst = ring + s * C::STAGE_BYTES;
        mbar_arrive_expect_tx(&full[warp][s][0], C::SLICE_BYTES);
#pragma unroll
        for (int x = 0; x < D / 64; ++x) tma_load_4d(dst + x * 2048, &tm_k, &full[warp][s][0], 64 * x, row, pw.head, page);
        mbar_arrive_expect_tx(&full[warp][s][1], C::SLICE_BYTES);
#pragma unroll
        for (int x = 0; x < D / 64; ++x)
          tma_load_4d(dst + C::SLICE_BYTES + x * 2048, &tm_v, &full[warp][s][1], 64 * x, row, pw.head, page);
      }
      ++issued;
      return;
    }
  };
  for (int s = 0; s < C::STAGES; ++s) produce();

  bool first_segment = true;
  const int rq = lane >> 2, cq = lane & 3;  // fragment row and column pair
  // ldmatrix source of this lane: matrix lane / 8, its row lane % 8
  const int mi = lane >> 3, mr = lane & 7;
  do {
    // Q^T fragments: row (n) rq of each 8-row tile, dims 16 kk + 2 cq (+ 8)
    uint32_t qf[NT][D / 16][2];
    int seen[2 * NT];
    int min_seen = 0x7fffffff;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      int64_t tok;
      int head, sn;
      const bool valid = unit_row(w, a, C::ROWS, nt * 8 + rq, tok, head, sn);
      const T *q = reinterpret_cast<const T *>(a.q) + (valid ? tok * a.qt + head * a.qh : 0);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        qf[nt][kk][0] = valid ? __ldg(reinterpret_cast<const uint32_t *>(q + kk * 16 + 2 * cq)) : 0u;
        qf[nt][kk][1] = valid ? __ldg(reinterpret_cast<const uint32_t *>(q + kk * 16 + 8 + 2 * cq)) : 0u;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        seen[2 * nt + e] = 0x7fffffff;
        if (unit_row(w, a, C::ROWS, nt * 8 + 2 * cq + e, tok, head, sn)) seen[2 * nt + e] = sn;
        min_seen = min(min_seen, seen[2 * nt + e]);
      }
    }
    min_seen = min(min_seen, w.seen);
    min_seen = min(min_seen, __shfl_xor_sync(0xffffffffu, min_seen, 1));
    min_seen = min(min_seen, __shfl_xor_sync(0xffffffffu, min_seen, 2));

    float o[NT][D / 16][4], m[2 * NT], l[2 * NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
#pragma unroll
    for (int e = 0; e < 2 * NT; ++e) {
      m[e] = -INFINITY;
      l[e] = 0.f;
    }

    for (int t = w.t0; t < w.t1; ++t) {
      const int key0 = slice_key(t);
      if (key0 >= w.seen) break;  // this warp's slices of the unit end here
      const uint32_t st = used % C::STAGES, parity = (used / C::STAGES) & 1u;
      ok = __all_sync(0xffffffffu, ok && mbar_wait(&full[warp][st][0], parity, abort_flag));
      if (!ok) break;
      const uint32_t ks = smem_u32(ring + st * C::STAGE_BYTES), vs = ks + C::SLICE_BYTES;
      // S^T: four partial sums per row tile keep the products' latency apart
      float s4[NT][2][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) s4[nt][i][e] = 0.f;
      {
        const int row = (mi & 1) * 8 + mr, hi = mi >> 1;  // matrices: keys 0-7, 8-15, then dims + 8
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const int chunk = (kk & 3) * 2 + hi;
          uint32_t kf[4];
          ldmatrix_x4(kf, ks + (kk >> 2) * 2048 + row * 128 + ((chunk ^ mr) << 4));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_16816<T>(s4[nt][kk & 1], kf, qf[nt][kk][0], qf[nt][kk][1]);
        }
      }
      const bool edge = key0 + DEC_SLICE > min_seen;
      uint32_t pf[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = (s4[nt][0][e] + s4[nt][1][e]) * a.scale_log2;
          if (edge && key0 + rq + (e >> 1) * 8 >= min(seen[2 * nt + (e & 1)], w.seen)) x[e] = -INFINITY;
        }
        float keep[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = fmaxf(x[e], x[e + 2]);
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
          top = fmaxf(top - weight_head<T>(0.f), m[2 * nt + e]);
          const float ref = top == -INFINITY ? 0.f : top;
          keep[e] = exp2_fast(m[2 * nt + e] - ref);
          m[2 * nt + e] = top;
          x[e] = exp2_fast(x[e] - ref);
          x[e + 2] = exp2_fast(x[e + 2] - ref);
          l[2 * nt + e] = l[2 * nt + e] * keep[e] + x[e] + x[e + 2];
        }
        pf[nt][0] = transpose_8x8(pack2<T>(x[0], x[1]));
        pf[nt][1] = transpose_8x8(pack2<T>(x[2], x[3]));
        if (__any_sync(0xffffffffu, keep[0] != 1.f || keep[1] != 1.f)) {
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            o[nt][i][0] *= keep[0];
            o[nt][i][1] *= keep[1];
            o[nt][i][2] *= keep[0];
            o[nt][i][3] *= keep[1];
          }
        }
      }
      ok = __all_sync(0xffffffffu, mbar_wait(&full[warp][st][1], parity, abort_flag));
      if (!ok) break;
      // rows of V behind the last slot in use may hold anything: their words become 0
      const int live = w.s.len - key0;  // slots of the slice in use
      const bool clean = live >= DEC_SLICE;
      uint32_t keep_lo = 0xffffffffu, keep_hi = 0xffffffffu;
      if (!clean) {
        const int k0 = 2 * cq;
        keep_lo = (k0 < live ? 0xffffu : 0u) | (k0 + 1 < live ? 0xffff0000u : 0u);
        keep_hi = (k0 + 8 < live ? 0xffffu : 0u) | (k0 + 9 < live ? 0xffff0000u : 0u);
      }
      {
        const int row = (mi >> 1) * 8 + mr, hi = mi & 1;  // matrices: dims 0-7, 8-15, then keys + 8
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const int chunk = (i & 3) * 2 + hi;
          uint32_t vf[4];
          ldmatrix_x4_trans(vf, vs + (i >> 2) * 2048 + row * 128 + ((chunk ^ mr) << 4));
          if (!clean) {
            vf[0] &= keep_lo;
            vf[1] &= keep_lo;
            vf[2] &= keep_hi;
            vf[3] &= keep_hi;
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_16816<T>(o[nt][i], vf, pf[nt][0], pf[nt][1]);
        }
      }
      ++used;
      __syncwarp();  // every lane has read the stage
      produce();
    }
    // join the four warps
#pragma unroll
    for (int e = 0; e < 2 * NT; ++e) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 4);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 8);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 16);
    }
    if (!first_segment) __syncthreads();  // the last unit's join has been read
    first_segment = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (lane < 4) {
        join_ml[warp * C::ROWS + nt * 8 + 2 * cq] = make_float2(m[2 * nt], l[2 * nt]);
        join_ml[warp * C::ROWS + nt * 8 + 2 * cq + 1] = make_float2(m[2 * nt + 1], l[2 * nt + 1]);
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          join_o[(warp * C::ROWS + nt * 8 + 2 * cq + (e & 1)) * C::O_LD + i * 16 + rq + (e >> 1) * 8] = o[nt][i][e];
    }
    __syncthreads();
    const bool begins = w.t0 == 0, ends = w.t1 == w.tiles;
    const int slot = begins ? 2 * c + 1 : 2 * c;
    if (begins && !ends && threadIdx.x == 0) describe(a, pl, w, c, C::ROWS);
    constexpr int PER_ROW = D / 4;
    for (int i = threadIdx.x; i < C::ROWS * PER_ROW; i += DEC_ATTN_THREADS) {
      const int r = i / PER_ROW, d = (i - r * PER_ROW) * 4;
      int64_t tok;
      int head, sn;
      if (!unit_row(w, a, C::ROWS, r, tok, head, sn)) break;  // rows ascend
      float2 ml[DEC_ATTN_WARPS];
      float top = -INFINITY;
#pragma unroll
      for (int x = 0; x < DEC_ATTN_WARPS; ++x) {
        ml[x] = join_ml[x * C::ROWS + r];
        top = fmaxf(top, ml[x].x);
      }
      const float ref = top == -INFINITY ? 0.f : top;
      float sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int x = 0; x < DEC_ATTN_WARPS; ++x) {
        const float f = exp2_fast(ml[x].x - ref);
        const float4 v = *reinterpret_cast<const float4 *>(join_o + (x * C::ROWS + r) * C::O_LD + d);
        sum = fmaf(f, ml[x].y, sum);
        acc.x = fmaf(f, v.x, acc.x);
        acc.y = fmaf(f, v.y, acc.y);
        acc.z = fmaf(f, v.z, acc.z);
        acc.w = fmaf(f, v.w, acc.w);
      }
      if (begins && ends) {
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
        store4<T>(reinterpret_cast<T *>(a.out) + tok * a.ot + head * a.oh + d,
                  make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
        if (a.lse && d == 0)
          a.lse[tok * a.heads + head] = row_lse(top, sum);
      } else {
        a.part_o[((int64_t)slot * C::ROWS + r) * (D / 4) + d / 4] = acc;
        if (d == 0) a.part_ml[slot * C::ROWS + r] = make_float2(top, sum);
      }
    }
  } while (walk_next(w, bt, a, sh));
  if (!ok) {  // a wait gave up: let the copies in flight land, then say so
    if (lane == 0) {
      for (uint32_t i = used; i < issued; ++i) {
        mbar_drain(&full[warp][i % C::STAGES][0], (i / C::STAGES) & 1u);
        mbar_drain(&full[warp][i % C::STAGES][1], (i / C::STAGES) & 1u);
      }
      atomicExch(a.status, DCKV_ETIMEOUT);
    }
  }
}

// ------------------------------------------------------------------ many rows: CTA pairs
// More than 8 (dim 256) or 16 packed rows: tcgen05 with cta_group::2.  A pair takes 256 rows (128 per CTA) and
// walks key tiles of 128: S = Q K^T (M 256, N 128) and O += P V (M 256, N dim), each CTA holding
// half of K (64 keys, all dims) and half of V (all keys, half the dims).  A CTA alone would
// stream a whole K and V tile per 128 rows, 64 bytes per clock at the tensor rate and dim 256, all
// that L2 gives an SM; the pair needs half of that.
// TMEM (512 columns): O in the first `dim`, then two S tiles of 128 columns; P overwrites the
// first half of its own S tile as 16-bit pairs and is the A operand of the second product.  (One S
// tile, freed once it is in registers, and two P tiles of their own measured the same.)
// Roles, per CTA: warp 0 loads K and V halves (lanes issue one TMA box each, through the page
// table), warp 1 of the even CTA issues all MMAs, warps 2-9 are the softmax: two threads per
// row, 64 columns each, which exchange the row maximum through shared memory.  While they work
// on tile j the tensor cores run S(j + 1), then O(j).
// The maximum a row's weights refer to moves only when the true one exceeds it by more than
// RESCALE_STEPS in log2: until then P stays below 2^RESCALE_STEPS (2^15 in fp16, see weight_head) and
// O needs no rescaling, which costs a round trip of O through registers.
constexpr int PAIR_ROWS = 256;
constexpr int PAIR_KEYS = 128;
constexpr int PAIR_SOFT_WARPS = 8;
constexpr int PAIR_THREADS = 64 + 32 * PAIR_SOFT_WARPS;
constexpr int ATTN_MAX_PAIRS = 80;
constexpr float RESCALE_STEPS = 8.f;

template <int D>
struct PairAttn {
  static constexpr int Q_BYTES = 128 * D * 2;
  static constexpr int BUF_BYTES = 64 * D * 2;  // half of K, or half of V
  static constexpr int V_ROW = D >= 128 ? 128 : 64;  // bytes of a V half's row in one block
  static constexpr int V_BLOCKS = D >= 128 ? D / 128 : 1;
  static constexpr int AREA = 512 + 2048;  // barriers; exchange, before that the plan
  static constexpr int FIT = (232448 - AREA - Q_BYTES) / BUF_BYTES;
  static constexpr int STAGES = FIT > 10 ? 10 : FIT;
  // All of the SM's shared memory, used or not: no second block that holds TMEM may share the SM.  Two
  // pairs of different kernels, each holding the TMEM of one SM and waiting for the other's, would
  // wait for ever.
  static constexpr int SMEM = 232448;
  static_assert(STAGES >= 4 && Q_BYTES + STAGES * BUF_BYTES + AREA <= SMEM, "shared memory");
};

template <int STAGES>
struct PairBars {
  uint64_t full[STAGES];   // leader: both halves of an item landed
  uint64_t empty[STAGES];  // both: the item's MMAs are done
  uint64_t s_full[2];      // both: S tile computed
  uint64_t p_full[2];      // leader: P written by every softmax warp of the pair
  uint64_t pv_done;        // both: O += P V of a tile done.  S(j) complete implies O(j - 2) complete, so
                           // a warp at tile j may wait here for O(j - 1), not for any later one
  uint64_t o_full;         // both: the unit's last O += P V done
  uint64_t q_empty;        // both: the unit's last S is computed, Q may be replaced
  uint64_t o_empty;        // leader: O read by every softmax warp
  uint64_t fix;            // own: a ragged V half landed
  uint64_t mma_end;        // after a timed-out wait: the MMAs issued so far are done
  GemmTail<STAGES> tail;
};

struct PairMaps {
  int k_box, v_box;     // rows of one TMA box
  int tokens, cta_rows; // of Q in one CTA's tile: tokens, tokens * group
};

template <typename T, int D>
__global__ void __launch_bounds__(PAIR_THREADS, 1)
    k_attend_many(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const __grid_constant__ CUtensorMap tm_q, const PoolDev p, const BatchDev bt, const AttnDev a,
                  const AttnShape sh, const PairMaps mp) {
  using C = PairAttn<D>;
  constexpr int STAGES = C::STAGES;
  constexpr uint32_t S_COL = 256;
  constexpr float HEAD = weight_head<T>(RESCALE_STEPS);
  extern __shared__ __align__(1024) uint8_t dyn_smem[];
  // no room for slack: the swizzled tiles rely on dynamic shared memory starting on 1,024 bytes
  // (it does where a kernel has no static shared memory)
  if (smem_u32(dyn_smem) & 1023u) {
    if (threadIdx.x == 0) atomicExch(a.status, DCKV_ECUDA);
    return;
  }
  uint8_t *q_sm = dyn_smem;
  uint8_t *bufs = dyn_smem + C::Q_BYTES;
  PairBars<STAGES> *bars = reinterpret_cast<PairBars<STAGES> *>(bufs + STAGES * C::BUF_BYTES);
  static_assert(sizeof(PairBars<STAGES>) <= 512 && sizeof(AttnPlanSmem) <= 2048, "barrier area");
  float *xch = reinterpret_cast<float *>(bufs + STAGES * C::BUF_BYTES + 512);  // [tile parity][half][row]
  AttnPlanSmem *plan_sm = reinterpret_cast<AttnPlanSmem *>(xch);
  GemmTail<STAGES> *tail = &bars->tail;
  volatile int *abort_flag = &tail->abort;
  // warp-uniform values, and known to be
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int c = blockIdx.x >> 1;
  uint32_t n_issued = 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->p_full[i], 2 * PAIR_SOFT_WARPS);
    }
    mbar_init(&bars->pv_done, 1);
    mbar_init(&bars->o_full, 1);
    mbar_init(&bars->q_empty, 1);
    mbar_init(&bars->o_empty, 2 * PAIR_SOFT_WARPS);
    mbar_init(&bars->fix, 1);
    mbar_init(&bars->mma_end, 1);
    mbar_init(&tail->drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
    prefetch_tmap(&tm_q);
  }
  if (warp == 1) {
    tmem_alloc_pair(&tail->tmem_base, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_arrive();  // both CTAs' barriers are initialised before any cross-CTA signal
  wait_chained();
  AttnPlan pl;
  AttnWalk w;
  const bool any = attn_plan<PAIR_THREADS>(bt, a, sh, PLAN_TRIES, c, plan_sm, pl, w);
  if (threadIdx.x == 64 && rank == 0) a.desc[2 * c] = make_int4(-1, 0, 0, 0);  // by the thread that may describe
  __syncthreads();  // the plan's shared memory is free
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tail->tmem_base, 0);

  if (!any) {
    // no piece: straight to the teardown (both CTAs of the pair alike)
  } else if (warp == 0) {
    // ---------------------------------------------------------------- K and V (both CTAs)
    int stage = 0;
    uint32_t phase = 0;
    uint32_t fixes = 0, item = 0;
    bool ok = true;
    const uint32_t q_bytes = (uint32_t)mp.cta_rows * D * 2;
    // one item: tile t's K half or V half; the unit's first K brings this CTA's rows of Q with it
    auto load = [&](const AttnWalk &wk, int t, bool is_v, bool with_q) {
      const int key0 = t * PAIR_KEYS + (is_v ? 0 : (int)rank * 64);
      const int box = is_v ? mp.v_box : mp.k_box;
      const int groups = (is_v ? PAIR_KEYS : 64) / box, blocks = is_v ? C::V_BLOCKS : D / 64;
      // this lane's box (at most 32): rows from `key`, page and row in it
      const int g = lane % groups, blk = lane / groups;
      const int key = key0 + g * box;
      int page = (int)p.n_pages, row = 0;  // behind the pool: the copy fills zeros
      if (blk < blocks && key < wk.s.len) {
        const int pi = p.page_div.div(key);
        row = key - pi * p.page_size;
        page = __ldg(bt.page_table + wk.b * bt.table_stride + pi);
        if (page < 0 || page >= p.n_pages) {
          atomicExch(a.status, DCKV_ERANGE);
          page = (int)p.n_pages;
          row = 0;
        }
      }
      // a V box that the sequence's last slot ends in: the rows behind it may hold anything, and
      // 0 * NaN is NaN, so they are cleared before the MMA sees them
      const int last_box = wk.s.len & ~(box - 1);  // first key of the box that holds slot `len`
      const bool ragged = is_v && last_box != wk.s.len && last_box >= key0 && last_box < key0 + PAIR_KEYS;
      ok = mbar_wait(&bars->empty[stage], phase ^ 1u, abort_flag);
      if (ok && with_q && item > 0) ok = mbar_wait(&bars->q_empty, (item - 1) & 1u, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      const uint32_t bytes = C::BUF_BYTES + (with_q ? q_bytes : 0u);
      uint8_t *dst = bufs + stage * C::BUF_BYTES;
      const uint32_t fb = mapa_shared(smem_u32(&bars->full[stage]), 0);
      if (lane == 0) {
        if (rank == 0) mbar_arrive_expect_tx(&bars->full[stage], 2 * bytes);
        if (ragged) mbar_arrive_expect_tx(&bars->fix, C::BUF_BYTES);
        tail->ring[stage] = bytes;
        ++n_issued;
      }
      __syncwarp();
      // rows past the sequence's are other tokens' or zeros; nothing of theirs is written
      if (with_q && lane >= 32 - D / 64) {
        const int x = lane - (32 - D / 64);
        tma_load_3d_pair(q_sm + x * 16384, &tm_q, fb, 64 * x, wk.head * a.group,
                         (int)wk.s.first + (2 * wk.rt + (int)rank) * mp.tokens);
      }
      if (blk < blocks) {
        if (!is_v) {
          tma_load_4d_pair(dst + blk * 8192 + g * box * 128, &tm_k, fb, 64 * blk, row, wk.head, page);
        } else {
          uint8_t *to = dst + (blk * PAIR_KEYS + g * box) * C::V_ROW;
          const int d0 = (int)rank * (D / 2) + blk * 64;
          if (ragged) tma_load_4d(to, &tm_v, &bars->fix, d0, row, wk.head, page);
          else tma_load_4d_pair(to, &tm_v, fb, d0, row, wk.head, page);
        }
      }
      if (ragged) {
        ok = __all_sync(0xffffffffu, mbar_wait(&bars->fix, fixes & 1u, abort_flag));
        if (!ok) mbar_drain(&bars->fix, fixes & 1u);
        ++fixes;
        const int r0 = wk.s.len - key0, n = (last_box + box - wk.s.len) * (C::V_ROW / 16);
        for (int i = lane; i < n * C::V_BLOCKS; i += 32) {
          const int b = i / n, j = i - b * n;
          reinterpret_cast<uint4 *>(dst + (b * PAIR_KEYS + r0) * C::V_ROW)[j] = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_complete_tx_cluster(fb, C::BUF_BYTES);
      }
      if (++stage == STAGES) {
        stage = 0;
        phase ^= 1u;
      }
    };
    do {
      load(w, w.t0, false, true);
      for (int t = w.t0; t < w.t1 && ok; ++t) {
        if (t + 1 < w.t1) load(w, t + 1, false, false);
        if (ok) load(w, t, true, false);
      }
      ++item;
    } while (ok && walk_next(w, bt, a, sh));
    // Q and every stage released: no commit is still in flight towards this CTA when it exits
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&bars->q_empty, (item - 1) & 1u, abort_flag));
    for (int i = 0; i < STAGES && ok; ++i) {
      ok = __all_sync(0xffffffffu, mbar_wait(&bars->empty[stage], phase ^ 1u, abort_flag));
      if (++stage == STAGES) {
        stage = 0;
        phase ^= 1u;
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer (even CTA)
    // The whole warp runs the loop in step and one elected lane issues under a predicate, so that the
    // operands stay in uniform registers (one lane in a branch of its own took 70 clocks per MMA, 24 of
    // them a tile at dim 256; three chunks of up to 300 tokens over 4,000 slots 33.3 -> 31.5 us).
    // Descriptors are a base plus constants (addresses advance in the low word's first 14 bits, which
    // never carry out of them).
    if (rank == 0) {
      constexpr int BF = std::is_same<T, __nv_bfloat16>::value ? 1 : 0;
      const uint32_t id_s = idesc_f16(BF, PAIR_ROWS, PAIR_KEYS);
      const uint32_t id_o = idesc_f16(BF, PAIR_ROWS, D) | IDESC_B_MN_MAJOR;
      const uint32_t issue = elect_one();
      const uint64_t q_desc = sw128_desc(smem_u32(q_sm));
      const uint64_t k_desc0 = sw128_desc(smem_u32(bufs));
      const uint64_t v_desc0 = mn_desc(smem_u32(bufs), C::V_ROW, PAIR_KEYS * C::V_ROW);
      int stage = 0;
      uint32_t phase = 0, tile = 0, item = 0;
      bool ok = true;
      auto scores = [&](uint32_t j) {  // S tile j of the kernel
        ok = __all_sync(0xffffffffu, mbar_wait(&bars->full[stage], phase, abort_flag));
        if (!ok) return;
        tc_fence_after();
        const uint64_t kd = k_desc0 + (uint64_t)(uint32_t)(stage * (C::BUF_BYTES >> 4));
        const uint32_t d = tmem + S_COL + (j & 1u) * PAIR_KEYS;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          umma_f16_pair_if(issue, d, q_desc + (((kk >> 2) * 16384 + (kk & 3) * 32) >> 4),
                           kd + (((kk >> 2) * 8192 + (kk & 3) * 32) >> 4), id_s, kk > 0);
        umma_commit_pair_if(issue, &bars->empty[stage]);
        umma_commit_pair_if(issue, &bars->s_full[j & 1u]);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      };
      do {
        scores(tile);
        const int n = w.t1 - w.t0;
        if (n == 1 && ok) umma_commit_pair_if(issue, &bars->q_empty);
        for (int t = 0; t < n && ok; ++t, ++tile) {
          if (t + 1 < n) scores(tile + 1);
          if (t + 2 == n && ok) umma_commit_pair_if(issue, &bars->q_empty);
          if (ok && t == 0 && item > 0) ok = mbar_wait(&bars->o_empty, (item - 1) & 1u, abort_flag);
          if (ok) ok = mbar_wait(&bars->p_full[tile & 1u], (tile >> 1) & 1u, abort_flag);
          if (ok) ok = mbar_wait_cluster(&bars->full[stage], phase, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          const uint64_t vd = v_desc0 + (uint64_t)(uint32_t)(stage * (C::BUF_BYTES >> 4));
          const uint32_t pt = tmem + S_COL + (tile & 1u) * PAIR_KEYS;
          const uint32_t acc = t > 0;
#pragma unroll
          for (int kk = 0; kk < PAIR_KEYS / 16; ++kk)
            umma_f16_pair_ts_if(issue, tmem, pt + kk * 8, vd + ((kk * 16 * C::V_ROW) >> 4), id_o, kk > 0 ? 1u : acc);
          umma_commit_pair_if(issue, &bars->empty[stage]);
          umma_commit_pair_if(issue, &bars->pv_done);
          if (t + 1 == n) umma_commit_pair_if(issue, &bars->o_full);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        ++item;
      } while (ok && walk_next(w, bt, a, sh));
      if (!ok) {  // leave no MMA in flight (the commit counts the issuing lane's)
        umma_commit_pair_if(issue, &bars->mma_end);
        mbar_drain(&bars->mma_end, 0);
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax (both CTAs)
    const int sw = warp - 2, quarter = warp & 3, half = sw >> 2;
    const int row = quarter * 32 + lane;  // of this CTA's 128
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t l_p[2] = {mapa_shared(smem_u32(&bars->p_full[0]), 0), mapa_shared(smem_u32(&bars->p_full[1]), 0)};
    const uint32_t l_o = mapa_shared(smem_u32(&bars->o_empty), 0);
    bool ok = true;
    uint32_t tile = 0, item = 0;

    do {
      int64_t tok = 0;
      int head = 0, seen = 0x7fffffff;
      const int prow = (int)rank * mp.cta_rows + row;  // row of the pair's tile
      const bool valid = row < mp.cta_rows && unit_row(w, a, sh.rows, prow, tok, head, seen);
      if (!valid) seen = 0x7fffffff;
      const bool work = __any_sync(0xffffffffu, valid);  // the same in both halves of the rows
      float ref = -INFINITY, sum = 0.f;  // ref in log2 units
      for (int t = w.t0; t < w.t1; ++t, ++tile) {
        const uint32_t sb = lanes + S_COL + (tile & 1u) * PAIR_KEYS;
        if (ok) ok = mbar_wait(&bars->s_full[tile & 1u], (tile >> 1) & 1u, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        if (work) {
          uint32_t x[64];
          tmem_ld_32x32b_x32(sb + half * 64, *reinterpret_cast<uint32_t(*)[32]>(x));
          tmem_ld_32x32b_x32(sb + half * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(x + 32));
          tmem_ld_wait();
          const int limit = seen - t * PAIR_KEYS - half * 64;  // columns from here on are masked
          if (__any_sync(0xffffffffu, limit < 64)) {
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (i >= limit) x[i] = 0xff800000u;  // -infinity
          }
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < 64; ++i) m4[i & 3] = fmaxf(m4[i & 3], __uint_as_float(x[i]));
          const float mine = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * a.scale_log2;
          float *xc = xch + (tile & 1u) * 256;
          xc[half * 128 + row] = mine;
          named_bar_sync(1 + quarter, 64);
          const float top = fmaxf(mine, xc[(half ^ 1) * 128 + row]);
          const bool move = top > ref + (HEAD + RESCALE_STEPS);
          if (__any_sync(0xffffffffu, move)) {
            const float next = move ? top - HEAD : ref;
            const float f = move ? exp2_fast(ref - next) : 1.f;
            sum *= f;
            ref = next;
            if (t > w.t0) {  // O of the tiles before: this half's columns
              if (ok) ok = mbar_wait(&bars->pv_done, (tile - 1) & 1u, abort_flag);
              ok = __all_sync(0xffffffffu, ok);
              tc_fence_after();
#pragma unroll 1
              for (int d = half * (D / 2); d < (half + 1) * (D / 2); d += 32) {
                uint32_t o[32];
                tmem_ld_32x32b_x32(lanes + d, o);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                tmem_st_32x32b_x32(lanes + d, o);
              }
              tmem_st_wait();
            }
          }
          const float off = ref == -INFINITY ? 0.f : -ref;
          uint32_t pk[32];
          uint64_t sum2 = f2(0.f, 0.f);
          const uint64_t scale2 = f2(a.scale_log2, a.scale_log2), off2 = f2(off, off);
          // Packed multiply-adds: 408 -> 396 us on 2,048 tokens over 32,768 slots.  Taking every second
          // to fourth pair's exp2 off the special-function unit (a polynomial on the FMA pipe) made
          // dim 128 slower, 415 -> 428-451 us.  Neither that unit (44% busy at dim 64, 42% at 128) nor
          // instruction issue (28%, 27%) bounds the smaller dims: it is the latency of one tile's chain,
          // wait for S - load - maximum - exchange - exp2 - store - signal, with two softmax warps per
          // scheduler and S(j + 1) queued behind O(j - 1), whose P lies in its columns.
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float2 y = un2(fma2(f2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), scale2, off2));
            const float e0 = exp2_fast(y.x), e1 = exp2_fast(y.y);
            sum2 = add2(sum2, f2(e0, e1));
            pk[i] = pack2<T>(e0, e1);
          }
          const float2 two = un2(sum2);
          sum += two.x + two.y;
          tmem_st_32x32b_x32(sb + half * 32, pk);
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(l_p[tile & 1u]);  // TMEM only: ordered by the tcgen05 fences
      }
      // the unit's end: join the halves' sums, read O
      float *xc = xch + (tile & 1u) * 256;
      xc[half * 128 + row] = sum;
      named_bar_sync(1 + quarter, 64);
      sum += xc[(half ^ 1) * 128 + row];
      if (ok) ok = mbar_wait(&bars->o_full, item & 1u, abort_flag);
      ++item;
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      named_bar_sync(1 + quarter, 64);  // sums read before the next unit's maxima overwrite them
      const bool begins = w.t0 == 0, ends = w.t1 == w.tiles;
      const int slot = begins ? 2 * c + 1 : 2 * c;
      const float inv = begins && ends ? (sum > 0.f ? 1.f / sum : 0.f) : 1.f;
      if (work) {
#pragma unroll 1
        for (int d = half * (D / 2); d < (half + 1) * (D / 2); d += 32) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(lanes + d, o);
          tmem_ld_wait();
          if (!valid || !ok) {
          } else if (begins && ends) {
            T *out = reinterpret_cast<T *>(a.out) + tok * a.ot + head * a.oh + d;
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              uint4 v;
              v.x = pack2<T>(__uint_as_float(o[i]) * inv, __uint_as_float(o[i + 1]) * inv);
              v.y = pack2<T>(__uint_as_float(o[i + 2]) * inv, __uint_as_float(o[i + 3]) * inv);
              v.z = pack2<T>(__uint_as_float(o[i + 4]) * inv, __uint_as_float(o[i + 5]) * inv);
              v.w = pack2<T>(__uint_as_float(o[i + 6]) * inv, __uint_as_float(o[i + 7]) * inv);
              *reinterpret_cast<uint4 *>(out + i) = v;
            }
          } else {
            float4 *out = a.part_o + ((int64_t)slot * (D / 4) + d / 4) * PAIR_ROWS + prow;
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<uint4 *>(out + (i / 4) * PAIR_ROWS) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
          }
          __syncwarp();  // the next load is the whole warp's
        }
        if (valid && half == 0 && ok) {
          if (!(begins && ends)) a.part_ml[(int64_t)slot * PAIR_ROWS + prow] = make_float2(ref, sum);
          else if (a.lse) a.lse[tok * a.heads + head] = row_lse(ref, sum);
        }
      }
      if (begins && !ends && rank == 0 && sw == 0 && lane == 0) describe(a, pl, w, c, sh.rows);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(l_o);
    } while (walk_next(w, bt, a, sh));
  }
  __syncthreads();
  pair_teardown<STAGES>(tail, bars->full, n_issued, rank, warp, lane, a.status);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ------------------------------------------------------------------ joining split units
// Block (c, y): if a unit begins in worker c's piece and is split, joins its rows y, y + gridDim.y, ...
// Parts: slot 2 c + 1 (the beginning), then slot 2 i of the workers i up to the last.  With few
// parts each of the eight warps joins a row by itself; with more than JOIN_WARP_PARTS the warps
// share a row, every eighth part each, and add up in shared memory: one warp alone would wait for
// the parts one load latency after the other.
// Few rows: parts are [rows][dim], a warp reads a row's dims side by side.
constexpr int JOIN_WARPS = 8;
constexpr int JOIN_THREADS = 32 * JOIN_WARPS;
constexpr int JOIN_WARP_PARTS = 6;

template <typename T, int D>
__global__ void __launch_bounds__(JOIN_THREADS) k_join_few(const AttnDev a, int rows) {
  constexpr int E = D / 32;  // dims per lane, in vectors of V
  constexpr int V = E >= 4 ? 4 : E;
  __shared__ float acc_sm[JOIN_WARPS][D];
  __shared__ float2 ml_sm[JOIN_WARPS];
  wait_chained();  // the parts are complete
  const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int4 ds = a.desc[2 * c];
  if (ds.x < 0) return;
  const int head0 = a.desc[2 * c + 1].x * a.group;
  const int parts = ds.x - c + 1;
  const bool shared_row = parts > JOIN_WARP_PARTS;
  const int step = shared_row ? JOIN_WARPS : 1;
  for (int r = blockIdx.y + (shared_row ? 0 : warp * gridDim.y); r < ds.y; r += gridDim.y * (shared_row ? 1 : JOIN_WARPS)) {
    float m = -INFINITY, sum = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    // joins one more (m, l, O); the loads of several parts are in flight at once
    auto add = [&](float2 ml, const float *x) {
      const float top = fmaxf(m, ml.x), ref = top == -INFINITY ? 0.f : top;
      const float f0 = exp2_fast(m - ref), f1 = exp2_fast(ml.x - ref);
      m = top;
      sum = sum * f0 + f1 * ml.y;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = acc[e] * f0 + f1 * x[e];
    };
#pragma unroll 4
    for (int i = shared_row ? warp : 0; i < parts; i += step) {
      const int64_t at = (int64_t)(i == 0 ? 2 * c + 1 : 2 * (c + i)) * rows + r;
      const float2 ml = a.part_ml[at];
      float x[E];
#pragma unroll
      for (int v = 0; v < E / V; ++v)
        *reinterpret_cast<Vec<float, V> *>(x + v * V) =
            *reinterpret_cast<const Vec<float, V> *>(reinterpret_cast<const float *>(a.part_o) + at * D + (v * 32 + lane) * V);
      add(ml, x);
    }
    if (shared_row) {
#pragma unroll
      for (int v = 0; v < E / V; ++v)
#pragma unroll
        for (int e = 0; e < V; ++e) acc_sm[warp][(v * 32 + lane) * V + e] = acc[v * V + e];
      if (lane == 0) ml_sm[warp] = make_float2(m, sum);
      __syncthreads();
      if (warp == 0) {
#pragma unroll
        for (int x = 1; x < JOIN_WARPS; ++x) {
          float y[E];
#pragma unroll
          for (int v = 0; v < E / V; ++v)
#pragma unroll
            for (int e = 0; e < V; ++e) y[v * V + e] = acc_sm[x][(v * 32 + lane) * V + e];
          add(ml_sm[x], y);
        }
      }
    }
    if (!shared_row || warp == 0) {
      const int i = ds.w + r, t = a.group_div.div(i);  // packed row of the sequence
      const int64_t tok = (int64_t)ds.z + t;
      const int head = head0 + i - t * a.group;
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
      T *out = reinterpret_cast<T *>(a.out) + tok * a.ot + head * a.oh;
#pragma unroll
      for (int v = 0; v < E / V; ++v) {
        Vec<T, V> y;
#pragma unroll
        for (int e = 0; e < V; ++e) y.e[e] = from_f<T>(acc[v * V + e] * inv);
        *reinterpret_cast<Vec<T, V> *>(out + (v * 32 + lane) * V) = y;
      }
      if (a.lse && lane == 0)
        a.lse[tok * a.heads + head] = row_lse(m, sum);
    }
    if (shared_row) __syncthreads();
  }
}

// Many rows: parts are [dim / 4][rows], as the softmax threads hold them (a row per lane; stores of
// [rows][dim] took 2.3 us of a 64 KB part, 32 lines per store).  A warp joins eight rows at a time
// and JOIN_STEPS values of k: lane = row + 8 q reads the dims 16 k + 4 q .. + 3 of its row, 128 bytes
// of eight rows side by side per q.  (With this layout and join the few rows' cases took 2 us longer.)
constexpr int JOIN_STEPS = 4;

// (m, l, O) of one row's dims in this lane.
struct JoinAcc {
  static constexpr int K = JOIN_STEPS;
  float m = -INFINITY, l = 0.f;
  float4 o[K];
  __device__ __forceinline__ JoinAcc() {
#pragma unroll
    for (int k = 0; k < K; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __device__ __forceinline__ void add(float2 ml, const float4 (&x)[K]) {
    const float top = fmaxf(m, ml.x), ref = top == -INFINITY ? 0.f : top;
    const float f0 = exp2_fast(m - ref), f1 = exp2_fast(ml.x - ref);
    m = top;
    l = l * f0 + f1 * ml.y;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      o[k].x = o[k].x * f0 + f1 * x[k].x;
      o[k].y = o[k].y * f0 + f1 * x[k].y;
      o[k].z = o[k].z * f0 + f1 * x[k].z;
      o[k].w = o[k].w * f0 + f1 * x[k].w;
    }
  }
};

// Adds the parts first, first + step, ... of row r, dims 16 (k0 + k) + 4 q.
template <int D>
__device__ __forceinline__ void join_parts(JoinAcc &acc, const AttnDev &a, int rows, int c, int parts, int first,
                                           int step, int r, int q, int k0) {
  constexpr int K = JOIN_STEPS;
#pragma unroll 4
  for (int i = first; i < parts; i += step) {
    const int64_t slot = i == 0 ? 2 * c + 1 : 2 * (c + i);
    float4 x[K];
    const float2 ml = a.part_ml[slot * rows + r];
#pragma unroll
    for (int k = 0; k < K; ++k) x[k] = a.part_o[(slot * (D / 4) + (k0 + k) * 4 + q) * rows + r];
    acc.add(ml, x);
  }
}

template <typename T>
__device__ __forceinline__ void join_store(const JoinAcc &acc, const AttnDev &a, int4 ds, int head0, int r, int q,
                                           int k0) {
  const int i = ds.w + r, t = a.group_div.div(i);  // packed row of the sequence
  const int64_t tok = (int64_t)ds.z + t;
  const int head = head0 + i - t * a.group;
  const float inv = acc.l > 0.f ? 1.f / acc.l : 0.f;
  T *out = reinterpret_cast<T *>(a.out) + tok * a.ot + head * a.oh + k0 * 16 + q * 4;
#pragma unroll
  for (int k = 0; k < JOIN_STEPS; ++k)
    store4<T>(out + k * 16, make_float4(acc.o[k].x * inv, acc.o[k].y * inv, acc.o[k].z * inv, acc.o[k].w * inv));
  if (a.lse && q == 0 && k0 == 0)
    a.lse[tok * a.heads + head] = row_lse(acc.m, acc.l);
}

template <typename T, int D>
__global__ void __launch_bounds__(JOIN_THREADS) k_join_many(const AttnDev a, int rows) {
  constexpr int CHUNKS = D / 16 / JOIN_STEPS;
  __shared__ float4 acc_sm[JOIN_WARPS][JOIN_STEPS][32];
  __shared__ float2 ml_sm[JOIN_WARPS][32];
  wait_chained();  // the parts are complete
  const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = lane >> 3;
  const int4 ds = a.desc[2 * c];
  if (ds.x < 0) return;
  const int head0 = a.desc[2 * c + 1].x * a.group;
  const int parts = ds.x - c + 1, tasks = ((ds.y + 7) >> 3) * CHUNKS;
  const bool shared_task = parts > JOIN_WARP_PARTS;
  const int first = shared_task ? warp : 0, step = shared_task ? JOIN_WARPS : 1;
  for (int task = shared_task ? blockIdx.y : blockIdx.y * JOIN_WARPS + warp; task < tasks;
       task += gridDim.y * (shared_task ? 1 : JOIN_WARPS)) {
    const int g = task / CHUNKS, k0 = (task - g * CHUNKS) * JOIN_STEPS, row = g * 8 + (lane & 7);
    const int r = min(row, ds.y - 1);
    JoinAcc acc;
    join_parts<D>(acc, a, rows, c, parts, first, step, r, q, k0);
    if (shared_task) {
#pragma unroll
      for (int k = 0; k < JOIN_STEPS; ++k) acc_sm[warp][k][lane] = acc.o[k];
      ml_sm[warp][lane] = make_float2(acc.m, acc.l);
      __syncthreads();
      if (warp == 0) {
#pragma unroll
        for (int x = 1; x < JOIN_WARPS; ++x) {
          float4 y[JOIN_STEPS];
#pragma unroll
          for (int k = 0; k < JOIN_STEPS; ++k) y[k] = acc_sm[x][k][lane];
          acc.add(ml_sm[x][lane], y);
        }
      }
    }
    if ((!shared_task || warp == 0) && row < ds.y) join_store<T>(acc, a, ds, head0, r, q, k0);
    if (shared_task) __syncthreads();
  }
}

}  // namespace dckv

// ============================================================================ host
// One layer of a pool as [pages][heads][page rows][dim]; box: 64 (or 32) dims x box_rows rows,
// swizzled by its row's bytes.
static int map_pages(CUtensorMap *m, const void *ptr, bool bf16, const PoolDev &p, int64_t rs, int64_t hs, int64_t ps,
                     int box_rows, int box_dims = 64) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(DCKV_ECUDA, "cuTensorMapEncodeTiled unavailable");
  cuuint64_t dims[4] = {(cuuint64_t)p.dim, (cuuint64_t)p.page_size, (cuuint64_t)p.heads, (cuuint64_t)p.n_pages};
  // a dimension of one entry has no stride to speak of
  cuuint64_t strides[3] = {(cuuint64_t)rs * 2, (cuuint64_t)(p.heads > 1 ? hs : 8) * 2,
                           (cuuint64_t)(p.n_pages > 1 ? ps : 8) * 2};
  cuuint32_t box[4] = {(cuuint32_t)box_dims, (cuuint32_t)box_rows, 1, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  CUresult r = fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                  const_cast<void *>(ptr), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  box_dims == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(DCKV_ECUDA, "tensor map (pages) encode failed: %d", (int)r);
  return DCKV_OK;
}

struct AttnLayout {
  size_t part_o, part_ml, desc, total;
};

static AttnLayout attn_layout(int rows, int dim) {  // rows: 8, 16 or PAIR_ROWS
  const int workers = rows == PAIR_ROWS ? ATTN_MAX_PAIRS : ATTN_MAX_WORKERS;
  AttnLayout l;
  l.part_o = 0;
  l.part_ml = l.part_o + sizeof(float) * 2ull * workers * rows * dim;
  l.desc = l.part_ml + sizeof(float2) * 2ull * workers * rows;
  l.total = l.desc + 2 * sizeof(int4) * workers;
  return l;
}

// Rows of a tile: 8 or, below dim 256, 16 where every sequence's packed rows fit (k_attend_few),
// else a pair's 256 (k_attend_many).  Measured on 64 ragged sequences of up to 8,192 slots, few / many:
// dim 256, 8 rows 117 / 133 us, 16 rows 160 / 135; dim 128, 8 rows 75 / 112, 16 rows 88 / 110, 24 rows
// (two tiles of 16 at dim 256: 200) many 106; dim 64, 16 rows 72 / 106.  One sequence of 1,000 slots:
// the same within 1 us.  One sequence's chunk sends the whole call to the pairs: 63 single tokens beside
// 512 tokens, 4,096 to 7,939 slots each, 8 heads, 139 / 144 / 189 us at dim 64 / 128 / 256, in two calls
// 96 / 117 / 181.  A group of more than 128 heads does not fit a CTA's rows and takes the few
// rows' tiles, several per token.
static int attn_rows(const BatchDev &b, int group, int dim) {
  const int64_t rows = (int64_t)b.max_new * group;
  const int few = dim < 256 ? 16 : 8;
  return rows <= 8 ? 8 : rows <= few || group > 128 ? few : PAIR_ROWS;
}

// Q as [tokens][heads][dim]; box: 64 dims x a group's heads x the tokens of one CTA's tile.
static int map_queries(CUtensorMap *m, const void *q, bool bf16, int dim, int heads, int64_t n, int64_t hs, int64_t ts,
                       int group, int tokens) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(DCKV_ECUDA, "cuTensorMapEncodeTiled unavailable");
  cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)n};
  cuuint64_t strides[2] = {(cuuint64_t)(heads > 1 ? hs : 8) * 2, (cuuint64_t)(n > 1 ? ts : 8) * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)tokens};
  cuuint32_t es[3] = {1, 1, 1};
  CUresult r = fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(q),
                  dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(DCKV_ECUDA, "tensor map (queries) encode failed: %d", (int)r);
  return DCKV_OK;
}

extern "C" size_t dckv_attention_workspace_bytes(const dckv_kv_pool *pool, const dckv_cache_batch *batch, int n_q_heads) {
  PoolDev p;
  BatchDev b;
  if (check_pool(pool, p) != DCKV_OK || check_batch(batch, 0, b) != DCKV_OK) return 0;
  if (n_q_heads < 1 || n_q_heads > 65535 || n_q_heads % p.heads) {
    fail(DCKV_EINVAL, "n_q_heads %d is not a multiple of the pool's heads", n_q_heads);
    return 0;
  }
  return attn_layout(attn_rows(b, n_q_heads / p.heads, p.dim), p.dim).total;
}

static int sm_count(int device, int &n) {
  static std::atomic<int> known[64];
  n = known[device].load();
  if (n == 0) {
    CK(cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device));
    known[device].store(n);
  }
  return DCKV_OK;
}

// Allows a kernel its dynamic shared memory, once per device.
static int allow_smem(const void *kern, int smem, int device, std::atomic<uint64_t> &done) {
  if (done.load() >> device & 1) return DCKV_OK;
  CK(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
  done.fetch_or(1ull << device);
  return DCKV_OK;
}

static int run_join(const void *kern, const AttnDev &a, int rows, int row_blocks, cudaStream_t st) {
  void *args[] = {(void *)&a, (void *)&rows};
  return launch_chained(kern, dim3((unsigned)a.workers, (unsigned)row_blocks), JOIN_THREADS, 0, 1, st, args);
}

template <typename T, int D, int NT>
static int run_attend_few(const CUtensorMap &mk, const CUtensorMap &mv, const PoolDev &p, const BatchDev &b,
                          const AttnDev &a, const AttnShape &sh, int device, cudaStream_t st) {
  auto kern = k_attend_few<T, D, NT>;
  static std::atomic<uint64_t> allowed{0};
  RET(allow_smem((const void *)kern, DecodeAttn<D, NT>::SMEM, device, allowed));
  void *args[] = {(void *)&mk, (void *)&mv, (void *)&p, (void *)&b, (void *)&a, (void *)&sh};
  RET(launch_chained((const void *)kern, dim3((unsigned)a.workers), DEC_ATTN_THREADS, DecodeAttn<D, NT>::SMEM, 1, st, args));
  return run_join((const void *)k_join_few<T, D>, a, 8 * NT, 8, st);
}

template <typename T, int D>
static int run_attend_many(const CUtensorMap &mk, const CUtensorMap &mv, const CUtensorMap &mq, const PoolDev &p, const BatchDev &b,
                           const AttnDev &a, const AttnShape &sh, const PairMaps &mp, int device, cudaStream_t st) {
  auto kern = k_attend_many<T, D>;
  static std::atomic<uint64_t> allowed{0};
  RET(allow_smem((const void *)kern, PairAttn<D>::SMEM, device, allowed));
  void *args[] = {(void *)&mk, (void *)&mv, (void *)&mq, (void *)&p, (void *)&b, (void *)&a, (void *)&sh, (void *)&mp};
  RET(launch_chained((const void *)kern, dim3((unsigned)(2 * a.workers)), PAIR_THREADS, PairAttn<D>::SMEM, 2, st, args));
  return run_join((const void *)k_join_many<T, D>, a, PAIR_ROWS, 16, st);
}

template <typename T, int D>
static int run_attend(const CUtensorMap &mk, const CUtensorMap &mv, const CUtensorMap &mq, const PoolDev &p, const BatchDev &b,
                      const AttnDev &a, const AttnShape &sh, const PairMaps &mp, int device, cudaStream_t st) {
  if (sh.rows == 8) return run_attend_few<T, D, 1>(mk, mv, p, b, a, sh, device, st);
  if constexpr (D < 256)
    if (sh.rows == 16) return run_attend_few<T, D, 2>(mk, mv, p, b, a, sh, device, st);
  return run_attend_many<T, D>(mk, mv, mq, p, b, a, sh, mp, device, st);
}

// Rows of a TMA box: the largest power of two up to `most` that divides a page, so that no box
// crosses a page (pages are multiples of 16).
static int box_rows(int page_size, int most) {
  int r = 16;
  while (r < most && page_size % (2 * r) == 0) r *= 2;
  return r;
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
  int64_t qt = args->q_token_stride, qh = args->q_head_stride, ot = args->out_token_stride, oh = args->out_head_stride;
  if (bad_stride(qt, n, 8) || bad_stride(qh, hq, 8) || bad_stride(ot, n, 8) || bad_stride(oh, hq, 8))
    return fail(DCKV_EINVAL, "q and out strides must be positive multiples of 8 elements");
  if (n <= 1) qt = ot = 0;
  if (hq == 1) qh = oh = 0;
  if (n > 0 && overlaps(args->q, span_bytes(n, qt, hq, qh, p.dim, 2), args->out, span_bytes(n, ot, hq, oh, p.dim, 2)))
    return fail(DCKV_EINVAL, "out overlaps q");
  const int group = hq / p.heads;
  AttnShape sh;
  const int slot_rows = attn_rows(b, group, p.dim);  // of the workspace's parts
  const bool many = slot_rows == PAIR_ROWS;
  const int cta_tokens = many ? 128 / group : 0;
  sh.rows = many ? 2 * cta_tokens * group : slot_rows;
  sh.key_tile = many ? PAIR_KEYS : DEC_KEY_TILE;
  sh.kv_heads = p.heads;
  const int64_t most_rows = std::min<int64_t>(b.max_new, std::max<int64_t>(n, 1)) * group;
  if (most_rows > 0x7fffffffll - PAIR_ROWS) return fail(DCKV_EINVAL, "max_new times the head group is too large");
  const int64_t row_tiles = (most_rows + sh.rows - 1) / sh.rows;
  if (row_tiles * b.batch > 1ll << 30) return fail(DCKV_EINVAL, "batch times max_new is too large");
  sh.row_tiles = (int)row_tiles;
  sh.unit_div = FastDiv((uint32_t)row_tiles);
  sh.units = (int)(row_tiles * b.batch);
  sh.max_slots = std::min<int64_t>((int64_t)b.max_pages * p.page_size, 0x7fffffffll - 65536);
  const AttnLayout lay = attn_layout(slot_rows, p.dim);
  if (ws_bytes < lay.total) return fail(DCKV_ECAPACITY, "workspace too small (%zu < %zu)", ws_bytes, lay.total);
  if (n == 0) return DCKV_OK;
  cudaStream_t st = (cudaStream_t)stream;
  DEVICE_SCOPE(pool->device);
  int sms;
  RET(sm_count(pool->device, sms));
  char *ws = (char *)workspace;
  const AttnDev a{(const char *)args->q, (char *)args->out, args->lse, qt, qh, ot, oh, hq, group, args->causal,
                  FastDiv((uint32_t)group), args->scale * 1.4426950408889634f, status, (float4 *)(ws + lay.part_o),
                  (float2 *)(ws + lay.part_ml),
                  (int4 *)(ws + lay.desc),
                  many ? std::min(sms / 2, ATTN_MAX_PAIRS) : std::min(sms, ATTN_MAX_WORKERS)};
  const bool bf = pool->dtype == DCKV_BF16;
  CUtensorMap mk, mv;
  const PairMaps mp{many ? box_rows(p.page_size, 64) : DEC_SLICE, many ? box_rows(p.page_size, PAIR_KEYS) : DEC_SLICE,
                    cta_tokens, cta_tokens * group};
  CUtensorMap mq{};
  if (many) RET(map_queries(&mq, args->q, bf, p.dim, hq, n, qh, qt, group, cta_tokens));
  RET(map_pages(&mk, p.k + 2 * args->layer * p.kl, bf, p, p.kr, p.kh, p.kp, mp.k_box));
  RET(map_pages(&mv, p.v + 2 * args->layer * p.vl, bf, p, p.vr, p.vh, p.vp, mp.v_box, many && p.dim == 64 ? 32 : 64));
  if (p.dim == 64)
    return bf ? run_attend<__nv_bfloat16, 64>(mk, mv, mq, p, b, a, sh, mp, pool->device, st)
              : run_attend<__half, 64>(mk, mv, mq, p, b, a, sh, mp, pool->device, st);
  if (p.dim == 128)
    return bf ? run_attend<__nv_bfloat16, 128>(mk, mv, mq, p, b, a, sh, mp, pool->device, st)
              : run_attend<__half, 128>(mk, mv, mq, p, b, a, sh, mp, pool->device, st);
  return bf ? run_attend<__nv_bfloat16, 256>(mk, mv, mq, p, b, a, sh, mp, pool->device, st)
            : run_attend<__half, 256>(mk, mv, mq, p, b, a, sh, mp, pool->device, st);
}
