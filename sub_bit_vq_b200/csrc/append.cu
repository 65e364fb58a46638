// Appending the keys and values of new tokens to the bf16 windows, with the
// position rotation of queries and keys on the way, and the tokens that the
// windows push out staged for the encoder (sm_100a).
//
// Row r of the call belongs to sequence b (the rows [s_b, s_b + n_b) of it,
// n_b = 1 and s_b = b without token_starts) and has position
// p = N_b - n_b + (r - s_b), N_b the length counting the appended rows.
//   rotation   (a, b) -> (a cos - b sin, b cos + a sin), float32, one
//              rounding to bf16 (round to nearest even): every product and sum
//              sees the table's 24 bits, and the cache holds bf16.
//   windows    p < P goes to slot p, the last R tokens to P + (p - P) mod R.
//   staging    the token e = p - R + A >= P, A rows ahead of the one that row r
//              pushes out, goes to row r of the staging slice: from the window
//              when it was cached before the call (e < N_b - n_b), else from row
//              r - R + A of the call. (A = 1 in a decode step: the index of a token
//              is in the pool before the token leaves the window.)
//
// A ring slot that the call overwrites is read (its old token) by the first row of
// the call in its residue class mod R and written by the last. Both are done by
// the thread of the first row, which rotates the last row's token again for it (at
// most R rows of a sequence): read and write stay in one thread, in order, and no
// thread waits for another. Every other row writes only places of its own; what
// the last A rows stage is in slots that the call leaves alone.
//
// Bound: HBM for prompts, the launch for a decode step. Each thread moves two
// 16-byte chunks of a head's row at a time (the two that rotate together), so a
// warp's accesses are whole 128-byte lines; with many rows a block walks eight
// of them, two rows' loads in flight per thread (one, four and eight in flight:
// 133.7, 142.4 and 190 us where two took 132.9, on 32768 tokens: more registers,
// fewer resident warps) and streams past the caches (138.4 us without the hints).
// Measured on B200, 16 + 2 x 16 heads of 128: 32768 tokens in 135 us
// (822 MB, 6.1 TB/s, 93% of the measured copy rate); one token of 8 and 256
// sequences in 2.5 and 3.2 us.

#include "common.cuh"
#include "encode_common.cuh"
#include "internal.h"

namespace loopvq {
namespace {

constexpr int kApThreads = 128;
constexpr int kApRows = 8;                // rows of a CTA when there are many

struct AppendParams {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  int64_t q_stride, k_stride, v_stride;   // elements between tokens
  const float* rope;                      // [n_positions][rot]: cos, then sin
  const int32_t* token_starts;            // [batch + 1] or null
  const int32_t* seq_lens;
  const int32_t* block_table;
  uint16_t* win_k;
  uint16_t* win_v;
  uint16_t* q_out;
  uint16_t* ev_k;                         // staging slices [n_tokens][Hkv][d]
  uint16_t* ev_v;
  int64_t* slots;
  int* status;
  int batch, n_tokens, Hq, Hkv, d, P, R, Pg, n_pages, max_pages_per_seq;
  int rot, n_positions, interleaved, units, lead;   // lead: A
};

// Where a row belongs: sequence (-1: none, nothing is written for the row),
// position, and the number of rows of its sequence from this row on and
// before it.
struct RowInfo {
  int b, p, before, after;                // rows of the sequence before this row, and after it
};

// V consecutive bf16 values.
template <int V>
struct Chunk {
  uint32_t w[V / 2];
};
template <int V, bool STREAM>
__device__ __forceinline__ Chunk<V> load_chunk(const uint16_t* p) {
  Chunk<V> c;
  if constexpr (V == 8) {
    const uint4* s = reinterpret_cast<const uint4*>(p);
    const uint4 t = STREAM ? __ldcs(s) : *s;
    c.w[0] = t.x; c.w[1] = t.y; c.w[2] = t.z; c.w[3] = t.w;
  } else {
    c.w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
  return c;
}
template <int V, bool STREAM>
__device__ __forceinline__ void store_chunk(uint16_t* p, const Chunk<V>& c) {
  if constexpr (V == 8) {
    const uint4 t = make_uint4(c.w[0], c.w[1], c.w[2], c.w[3]);
    if constexpr (STREAM)
      __stcs(reinterpret_cast<uint4*>(p), t);
    else
      *reinterpret_cast<uint4*>(p) = t;
  } else {
    *reinterpret_cast<uint32_t*>(p) = c.w[0];
  }
}

// One unit of a head's row: chunk c0 and (when two) chunk c1.
template <int V>
struct Pair {
  Chunk<V> a, b;
};

template <int V>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Rotates the V pairs of a unit by row p of the table (pairs i0 .. i0 + V - 1).
template <int V>
__device__ __forceinline__ void rotate(Pair<V>& x, const float* cs, int i0, int half, bool interleaved) {
  float co[V], si[V];
  if constexpr (V == 8) {
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const float4 c4 = __ldg(reinterpret_cast<const float4*>(cs + i0 + i));
      const float4 s4 = __ldg(reinterpret_cast<const float4*>(cs + half + i0 + i));
      co[i] = c4.x; co[i + 1] = c4.y; co[i + 2] = c4.z; co[i + 3] = c4.w;
      si[i] = s4.x; si[i + 1] = s4.y; si[i + 2] = s4.z; si[i + 3] = s4.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      co[i] = __ldg(cs + i0 + i);
      si[i] = __ldg(cs + half + i0 + i);
    }
  }
  if (!interleaved) {                     // element i of a with element i of b
#pragma unroll
    for (int w = 0; w < V / 2; ++w) {
      const float2 a = bf16x2_to_float2(x.a.w[w]), b = bf16x2_to_float2(x.b.w[w]);
      x.a.w[w] = pack2<V>(a.x * co[2 * w] - b.x * si[2 * w], a.y * co[2 * w + 1] - b.y * si[2 * w + 1]);
      x.b.w[w] = pack2<V>(b.x * co[2 * w] + a.x * si[2 * w], b.y * co[2 * w + 1] + a.y * si[2 * w + 1]);
    }
  } else {                                // neighbours
#pragma unroll
    for (int w = 0; w < V / 2; ++w) {
      const float2 a = bf16x2_to_float2(x.a.w[w]), b = bf16x2_to_float2(x.b.w[w]);
      const int i = w, k = V / 2 + w;
      x.a.w[w] = pack2<V>(a.x * co[i] - a.y * si[i], a.y * co[i] + a.x * si[i]);
      x.b.w[w] = pack2<V>(b.x * co[k] - b.y * si[k], b.y * co[k] + b.x * si[k]);
    }
  }
}

// The row's sequence and position; every lane of the warp calls it.
__device__ __forceinline__ RowInfo locate_row(const AppendParams& p, int r, int lane) {
  RowInfo f{-1, 0, 0, 0};
  if (r >= p.n_tokens) return f;
  int b = r, lo = r, hi = r + 1;
  if (p.token_starts != nullptr) {
    // the number of ends token_starts[1 .. batch] at or before row r
    int n = 0;
    for (int i = lane; i < p.batch; i += 32) n += __ldg(p.token_starts + 1 + i) <= r ? 1 : 0;
    b = __reduce_add_sync(0xffffffffu, n);
    if (b >= p.batch) return f;           // behind the last sequence
    lo = max(__ldg(p.token_starts + b), 0);
    hi = min(__ldg(p.token_starts + b + 1), p.n_tokens);
    if (r < lo || r >= hi) return f;      // before the first sequence, or starts that do not ascend
  }
  const int N = __ldg(p.seq_lens + b);
  if (N <= 0) return f;                   // no sequence in this row of the batch
  if (N < hi - lo || (p.rot > 0 && N > p.n_positions)) {
    if (lane == 0 && p.status != nullptr) atomicOr(p.status, LOOPVQ_ENCODE_STATUS_BAD_POSITION);
    return f;
  }
  f.b = b;
  f.p = N - (hi - r);
  f.before = r - lo;
  f.after = hi - 1 - r;
  return f;
}

// Pool slot of the token that the row stages, or -1.
__device__ __forceinline__ int64_t evicted_slot(const AppendParams& p, const RowInfo& f) {
  const int v = f.p - p.R + p.lead - p.P; // its index among the quantised tokens
  if (f.b < 0 || v < 0) return -1;
  const int page = v / p.Pg;
  int phys = -1;
  if (page < p.max_pages_per_seq) phys = __ldg(p.block_table + static_cast<int64_t>(f.b) * p.max_pages_per_seq + page);
  if (phys < 0 || phys >= p.n_pages) {
    if (p.status != nullptr) atomicOr(p.status, LOOPVQ_ENCODE_STATUS_BAD_SLOT);
    return -1;
  }
  return static_cast<int64_t>(phys) * p.Pg + v % p.Pg;
}

// Thread = one unit (two chunks of V values that rotate together, or two
// plain ones) of one head of the fused row [q heads][k heads][v heads]; it
// walks the CTA's rows. With eight rows seven blocks share an SM (72 registers; six
// of 76: 143 us against 135 on 32768 tokens).
template <int V, int ROWS>
__global__ void __launch_bounds__(kApThreads, ROWS > 1 ? 7 : 1) append_kernel(const AppendParams p) {
  constexpr int kBatch = ROWS < 2 ? ROWS : 2;
  constexpr bool kStream = ROWS > 1;
  __shared__ RowInfo rows[ROWS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r0 = blockIdx.x * ROWS;
  for (int i = warp; i < ROWS; i += kApThreads / 32) {
    const RowInfo f = locate_row(p, r0 + i, lane);
    if (lane == 0) rows[i] = f;
  }
  const int item = blockIdx.y * kApThreads + tid;
  const int q_heads = p.q != nullptr ? p.Hq : 0;
  const int head = item / p.units, u = item - head * p.units;
  const bool active = head < q_heads + 2 * p.Hkv;
  const bool is_q = head < q_heads, is_v = head >= q_heads + p.Hkv;
  const int h = is_q ? head : is_v ? head - q_heads - p.Hkv : head - q_heads;
  // the unit's chunks
  const int nr = is_v ? 0 : p.rot / (2 * V), n_chunks = p.d / V;
  const bool rotated = u < nr;
  int c0, c1;
  if (rotated) {
    c0 = p.interleaved ? 2 * u : u;
    c1 = p.interleaved ? 2 * u + 1 : u + nr;
  } else {
    c0 = nr + u;                          // 2 nr + (u - nr)
    c1 = c0 + (p.units - nr);
  }
  const bool two = c1 < n_chunks;
  const int e0 = c0 * V, e1 = (two ? c1 : c0) * V;
  const uint16_t* src = is_q ? p.q : is_v ? p.v : p.k;
  const int64_t stride = is_q ? p.q_stride : is_v ? p.v_stride : p.k_stride;
  src += static_cast<int64_t>(h) * p.d;
  auto load = [&](int r) {
    Pair<V> x;
    const uint16_t* s = src + r * stride;
    x.a = load_chunk<V, kStream>(s + e0);
    x.b = load_chunk<V, kStream>(s + e1);
    return x;
  };
  auto put = [&](uint16_t* dst, const Pair<V>& x) {
    store_chunk<V, kStream>(dst + e0, x.a);
    if (two) store_chunk<V, kStream>(dst + e1, x.b);
  };
  auto turn = [&](Pair<V>& x, int pos) {
    if (rotated) rotate<V>(x, p.rope + static_cast<int64_t>(pos) * p.rot, u * V, p.rot / 2, p.interleaved != 0);
  };
  __syncthreads();
  if (blockIdx.y == 0 && p.slots != nullptr && tid < ROWS && r0 + tid < p.n_tokens)
    p.slots[r0 + tid] = evicted_slot(p, rows[tid]);
  if (!active) return;

  auto finish = [&](int i, Pair<V>& x) {  // row i of the CTA, its unit loaded
    const RowInfo f = rows[i];
    const int r = r0 + i;
    turn(x, f.p);
    if (is_q) {
      put(p.q_out + (static_cast<int64_t>(r) * p.Hq + h) * p.d, x);
      return;
    }
    uint16_t* win = (is_v ? p.win_v : p.win_k) + (static_cast<int64_t>(f.b) * p.Hkv + h) * (p.P + p.R) * p.d;
    uint16_t* ev = (is_v ? p.ev_v : p.ev_k) + static_cast<int64_t>(h) * p.d;
    const int64_t ev_row = static_cast<int64_t>(p.Hkv) * p.d;
    const int wait = p.R - p.lead;        // rows from a token to the one that stages it
    if (f.p < p.P)
      put(win + static_cast<int64_t>(f.p) * p.d, x);
    else if (f.after >= wait)             // staged by this or a later row of this call
      put(ev + (r + wait) * ev_row, x);
    // the staged token is one of the window that stays in it
    if (f.after < p.lead && f.before < wait && f.p - wait >= p.P) {
      const uint16_t* kept = win + static_cast<int64_t>(p.P + (f.p - wait - p.P) % p.R) * p.d;
      Pair<V> old;
      old.a = load_chunk<V, kStream>(kept + e0);
      old.b = load_chunk<V, kStream>(kept + e1);
      put(ev + r * ev_row, old);
    }
    if (f.before >= p.R) return;          // (R = 0: every row)
    // first row of its residue class: the old token of the ring slot goes to the
    // row that stages it (unless an earlier call did), the class's last token into
    // the slot
    const int ahead = f.after / p.R * p.R;
    if (f.p + ahead < p.P) return;
    uint16_t* slot = win + static_cast<int64_t>(p.P + (f.p + ahead - p.P) % p.R) * p.d;
    if (f.p - p.R >= p.P && f.before >= p.lead) {
      Pair<V> old;
      old.a = load_chunk<V, kStream>(slot + e0);
      old.b = load_chunk<V, kStream>(slot + e1);
      put(ev + (r - p.lead) * ev_row, old);
    }
    if (ahead > 0) {
      x = load(r + ahead);
      turn(x, f.p + ahead);
    }
    put(slot, x);
  };
  // kBatch rows' loads are in flight before the first is turned and stored
#pragma unroll 1
  for (int i0 = 0; i0 < ROWS; i0 += kBatch) {
    Pair<V> x[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (rows[i0 + i].b >= 0) x[i] = load(r0 + i0 + i);   // CTA-uniform
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (rows[i0 + i].b >= 0) finish(i0 + i, x[i]);
  }
}

}  // namespace

loopvq_status launch_append(const AppendArgs& a) {
  const Geometry& g = *a.geo;
  const int gamma = a.loop_step / g.g, tau = a.loop_step % g.g;
  AppendParams p{};
  p.q = static_cast<const uint16_t*>(a.q);
  p.k = static_cast<const uint16_t*>(a.k);
  p.v = static_cast<const uint16_t*>(a.v);
  p.q_stride = a.q_token_stride;
  p.k_stride = a.k_token_stride;
  p.v_stride = a.v_token_stride;
  p.rope = a.rope;
  p.token_starts = a.token_starts;
  p.seq_lens = a.seq_lens;
  p.block_table = a.block_table;
  p.win_k = static_cast<uint16_t*>(a.win_k);
  p.win_v = static_cast<uint16_t*>(a.win_v);
  p.q_out = static_cast<uint16_t*>(a.q_out);
  const int64_t slice = static_cast<int64_t>(a.n_tokens) * g.Hkv * g.d;
  const int64_t z = (static_cast<int64_t>(a.layer) * g.G + gamma) * 2;
  p.ev_k = static_cast<uint16_t*>(a.evicted) + (z * g.g + tau) * slice;
  p.ev_v = static_cast<uint16_t*>(a.evicted) + ((z + 1) * g.g + tau) * slice;
  p.slots = a.slot_mapping;
  p.status = encode_status_word();
  p.batch = a.batch;
  p.n_tokens = a.n_tokens;
  p.Hq = g.Hq;
  p.Hkv = g.Hkv;
  p.d = g.d;
  p.P = g.P;
  p.R = g.R;
  p.Pg = g.Pg;
  p.n_pages = g.n_pages;
  p.max_pages_per_seq = g.max_pages_per_seq;
  p.rot = a.rot_dim;
  p.n_positions = a.n_positions;
  p.interleaved = a.interleaved;
  p.lead = a.stage_ahead;
  // 16-byte chunks unless the rotated half is not a whole number of them
  const bool wide = a.rot_dim % 16 == 0;
  const int V = wide ? 8 : 2;
  p.units = (g.d + 2 * V - 1) / (2 * V);
  const int64_t items = ((a.q != nullptr ? g.Hq : 0) + 2ll * g.Hkv) * p.units;
  if (items > 65535ll * kApThreads) return LOOPVQ_ERR_UNSUPPORTED;   // the grid's y extent
  const int tiles = static_cast<int>((items + kApThreads - 1) / kApThreads);
  cudaStream_t st = static_cast<cudaStream_t>(a.stream);
  // One row per block while all blocks fit the machine at once or nearly so
  // (latency counts), eight rows per block beyond: measured equal near 16K
  // blocks (heads x rows of 16 x 128: 3556 rows 20.6 against 21.8 us, 7113 rows
  // 37.4 against 34.7; 40 x 96: 1778 rows 21.0 against 22.7, 3556 rows 37.9
  // against 36.6).
  if (static_cast<int64_t>(a.n_tokens) * tiles < 16384) {
    const dim3 grid(a.n_tokens, tiles);
    if (wide)
      append_kernel<8, 1><<<grid, kApThreads, 0, st>>>(p);
    else
      append_kernel<2, 1><<<grid, kApThreads, 0, st>>>(p);
  } else {
    const dim3 grid((a.n_tokens + kApRows - 1) / kApRows, tiles);
    if (wide)
      append_kernel<8, kApRows><<<grid, kApThreads, 0, st>>>(p);
    else
      append_kernel<2, kApRows><<<grid, kApThreads, 0, st>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? LOOPVQ_OK : LOOPVQ_ERR_CUDA;
}

}  // namespace loopvq
