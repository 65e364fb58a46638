// Decode attention for groups of sequences that share a quantised prefix, on
// the tensor cores (sm_100a).
//
// One query per sequence leaves a decode step without a matrix product, but a
// group of sequences over the same tokens is one: with the group's queries as
// the rows of Q,
//   S^T = K Q^T       (M = 128 token rows,  N = query rows, K = d)
//   O^T += V^T P      (M = 128 channels,    N = query rows, K = 128 tokens)
// The tokens (then the channels) are the M side, so the products cost what the
// group's rows need (N = 16, 32 or 64) and not a 128-row tile.
//
// Four kernels, each a programmatic dependent of the one before:
//   shared_table_kernel   the call's codebook slices as fp16 tables, every
//                  sequence's split into shared and own tokens, the shared grid's
//                  starting points. 128 KB a head.
//   shared_prefix_kernel  persistent blocks over the tiles of all units (group, row
//                  tile, head): the tensor-core pipeline below, one record
//                  (m, l, o[d]) per row and block that met it.
//   shared_own_kernel     beside it, on the SMs that it leaves free: a warp per
//                  (sequence, query head, window or chunk of own quantised
//                  tokens), scored against the same tables without a product.
//   shared_merge_kernel   log-sum-exp join of a row's records.
//
// Codewords are dequantised from fp16 tables in shared memory, [E] rows of 256
// bytes holding entry (e, j) at byte j*2c: a lane that reads channel group j
// hits banks that depend on j only, and in the pool's rotated rows lane = slot i
// finds group (s + i) mod J at byte s, so the lookups of a half-warp never
// collide. The tile rows are written so that the same rotation keeps the stores
// free of conflicts too (tile_off). The value tile is the same [token][channel]
// layout read as an M-major operand, so nothing is transposed.
//
// Shared pipeline, 25 warps: 0-7 turn S^T into P (warp w reads TMEM lanes
// 32 (w % 4) .., the column half w / 4), 8-15 fill the K tile and 16-23 the V tile
// (a tile is four index blocks; warp w fills block w % 4, half of its groups), 24
// issues the products. K and V have one buffer each, S^T two, P two (one with 64
// rows); mbarriers hand them over, so the next K tile is filled under the softmax
// and the next V tile under the next scores.
//
// Softmax: per row a reference m, raised only when a score passes it by more
// than kRaise (then to the tile's maximum - kTop), so P = 2^(x - m) stays below
// 2^kRaise and keeps fp16's full precision down to 2^-20 of the maximum; sums
// are float32 over unrounded weights.
//
// Rounding. Keys, values and weights enter the products as fp16: half a step is
// 2^-11 of each value, an eighth of the bf16 output's own. Codebooks are scaled by
// powers of two into fp16's range, one per channel group, queries by one per unit or,
// where its rows differ by more than 2^kRowSpan, one per row (exact but for
// entries 2^-19 below their group's or row's largest). float32 outputs take the
// streaming kernels.
//
// Cost. HBM has to deliver a group's indices once (8 sequences of 16 heads over
// 32696 tokens: 33.5 MB, 5 us); the products are small. What a tile costs is
// shared-memory accesses: 2 x 32 KB of lookups, as much of stores, and the
// products' reads, 1650 cycles of 128 bytes with 16 query rows, 1900 with 64.
// Measured 2200 and 3400 (1900 MHz): 53 us for those 8 sequences, of which 48 in
// the shared grid (7 of them before its first tile), 5 + 1 around it in the tables
// and the merge, against 77.9 us when every sequence streams on its own; 256
// sequences over 16312 tokens 188 us against 1313 (205 with the weights computed
// only once P's buffer is free: with 64 rows there is one).
//
// What lost: the keys in two half tiles of M = 64 (71 us for the 8 sequences: a
// product takes 90-150 cycles of issue under the fill's accesses, 47 alone, so
// more and smaller ones lose); values handed over block by block (73: polls queue
// behind the fill's accesses); one team filling both planes (61); products issued
// by a warp of each fill team instead of one of their own, with 16 softmax warps at
// 64 rows (61, and 233 for the 256 sequences); half a tile filled under the other
// half's products, keys by channels and values by tokens (61 and 243; values only
// 62 and 235): the products slow down under the same plane's fill, and there are
// twice the hand-overs.

#include <cuda_fp16.h>
#include <math.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <numeric>
#include <type_traits>

#include "common.cuh"
#include "group_span.h"
#include "internal.h"
#include "tcgen05.cuh"

namespace loopvq {
namespace {

constexpr int kSoftWarps = 8;             // warps 0-7
constexpr int kDeqWarps = 8;              // warps 8-15 fill the K tile, 16-23 the V tile
constexpr int kKWarp = kSoftWarps, kVWarp = kKWarp + kDeqWarps, kMmaWarp = kVWarp + kDeqWarps;
constexpr int kShWarps = kMmaWarp + 1;
constexpr int kShThreads = kShWarps * 32;
// Registers of a thread: 72 at launch. With 64 query rows the softmax warps need
// more and take what the filling warps give (8 x 104 + 16 x 56 = 24 x 72).
constexpr int kLaunchRegs = 72, kSoftRegs = 104, kDeqRegs = 56;
constexpr int kTileRows = 128;            // token rows of a tile (4 index blocks of up to 32 slots)
constexpr int kMaxRows = 64;              // query rows of a block
constexpr float kRaise = 14.f;            // log2: a weight reaches 2^14 at most
constexpr float kTop = 6.f;               // log2: weight of the maximum after a raise
// A record's o (the window's apart) is 2^-kRecExp of its weighted sum, weights up to
// 2^14, so that it stays in float32 wherever a plain sum of values does; the merge
// takes m and l to the same scale. (Done where the records are written it cost 9 us of
// 187 with 256 sequences.)
constexpr int kRecExp = 14;
constexpr float kUnset = -1e30f;          // reference of a row that has seen no token
// log2: how far the rows of a unit may differ and still share a scale. A row's
// largest entry is then 2^5 at least in fp16, so what its smaller ones lose (half
// of 2^-24) is 2^-30 of it. (A factor per row in every tile cost 3.9 us of 52.9
// with 16 rows, 9 of 93 with 32.)
constexpr int kRowSpan = 8;
#ifndef LOOPVQ_TC_SPIN
#define LOOPVQ_TC_SPIN (1 << 20)
#endif
constexpr int kShSpin = LOOPVQ_TC_SPIN;
constexpr int kShDrainSpin = 1 << 24;

// Shared memory: bytes from the start of the dynamic allocation, which has to
// be window address kShBase (the block's reserved shared memory ends there; the
// host checks it), so that tables and tiles are immediate offsets.
constexpr uint32_t kShBase = 0x400u;
constexpr int kTabBytes = kE * 256;                        // one fp16 codebook slice
constexpr int kKtabOff = 0;
constexpr int kVtabOff = kTabBytes;
constexpr int kKtileOff = 2 * kTabBytes;                   // [16 row groups][2 channel blocks][8][128 B]
constexpr int kTileBytes = kTileRows * 256;
constexpr int kVtileOff = kKtileOff + kTileBytes;
constexpr int kPOff = kVtileOff + kTileBytes;              // [128 tokens] rows of 128 B, or twice of 64 B
constexpr int kQOff = kPOff + kTileRows * 128;             // [2 channel blocks][N][128 B]
constexpr int kQBytes = kMaxRows * 256;
constexpr int kMOff = kQOff + kQBytes;                     // float [64]: references
constexpr int kCmOff = kMOff + kMaxRows * 4;               // float [4][64]: column maxima, then sums
constexpr int kAlOff = kCmOff + 4 * kMaxRows * 4;          // float [64]: factors of a raise
constexpr int kScOff = kAlOff + kMaxRows * 4;              // float [64]: a row's 2^-kq, when the rows differ
constexpr int kLimOff = kScOff + kMaxRows * 4;             // int [64]: a row's shared tokens
constexpr int kNvOff = kLimOff + kMaxRows * 4;             // int [4 tiles][4 blocks]: valid slots
constexpr int kBarOff = kNvOff + 64;                       // mbarriers
constexpr int kSegOff = kBarOff + 96;                      // the block's segment and walk
constexpr int kTmemSlotOff = kSegOff + 144;
constexpr int kShSmem = kTmemSlotOff + 16;
static_assert(kShSmem <= 227 * 1024, "shared memory above 227 KB");

// K and V tile filled, S^T done (per buffer; its K tile is free), P written (per
// buffer), O^T += done (by tile parity; its V tile and P are free).
enum { kBarK = 0, kBarV, kBarS0, kBarS1, kBarP0, kBarP1, kBarO0, kBarO1, kBarTabK, kBarTabV, kBarDrain, kBars };
static_assert(kBars * 8 <= kTmemSlotOff - kBarOff, "barriers fit");

constexpr uint32_t kTmCols = 256, kTmS = 0, kTmO = 128;    // TMEM columns: S^T twice 64, O^T 64

// Where a block of the shared grid is in the list of units: see
// shared_prefix_kernel.
struct Walk {
  int64_t at, end, U, n;          // next cost, the block's last; all blocks' cost; blocks with work
  int g, rt, pos, hkv;            // group, row tile, cost inside the unit, head
  int rows, tiles, S, lo;         // of group g: query rows, shared tiles and tokens, first sequence
  int head, pad[3];               // whose tables are in shared memory
};
static_assert(sizeof(Walk) % 16 == 0, "copied by 16 bytes");

struct SharedParams {
  const uint16_t* q;              // bf16 [B][Hq][d]
  const uint8_t* pool_lg;         // pool at (layer, gamma, head 0)
  int64_t pool_stride_head, page_bytes, plane_bytes;
  const float* cb_k;              // (layer, head 0, gamma, K, tau): [J][E][c]
  const float* cb_v;
  int64_t cb_stride_head;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* group_starts;
  const int32_t* shared_lens;
  const uint16_t* win_k;
  const uint16_t* win_v;
  const unsigned char* tables;    // [Hkv][K, V] fp16 tables of kTabBytes
  const int* exps;                // [Hkv][K, V][32]: a group's table entries are scaled by 2^exps (V: + kRecExp)
  int2* seqs;                     // [B] shared and own quantised tokens of a sequence
  float* srec;                    // [pairs + shared_blocks * N][4 + d] records of the shared blocks
  float* orec;                    // [pairs][NC][4 + d] records of the own chunks
  int* status;
  void* out;
  float* lse;
  int B, n_groups, Hq, Hkv, ratio, W, Pg, n_pages, max_pages_per_seq;
  int max_group, max_shared, max_own;
  int max_vq;                     // tokens that a row of the page table names, or INT_MAX
  Walk* walks;                    // [shared_blocks] where each block starts
  int2* spans;                    // [pairs] first shared record of a row, and their number (N records apart)
  int NC, CH;                     // own records of a pair (window, chunks), tokens of a chunk
  int shared_blocks, own_blocks;  // grids
  int lbpp;                       // log2 of the index blocks of a page
  float scale_log2;
};

template <int J_, int C_>
struct Shape {
  static constexpr int J = J_, C = C_, D = J * C;
  static constexpr int LB = (32 / J) * J;
  static constexpr int GR = (J % 16 == 0) ? 16 : (J % 8 == 0) ? 8 : 4;
  static constexpr int NW = J / 4;                     // index words of a slot
  static constexpr int ENTRY = 2 * C;                  // bytes of an fp16 codeword
  static constexpr int TOK = 4 * LB;                   // tokens of a tile
  static constexpr int RS = 4 + D;                     // floats of a record
  static constexpr int TPS = 32 / J;                   // tokens a warp takes side by side (own tokens)
};

// Shared-memory operand descriptors, low and high word: address and leading
// offset; stride offset, version and swizzle.
constexpr uint32_t kSw128 = 2u, kSw64 = 4u;
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
  return ((saddr >> 4) & 0x3fffu) | ((lbo >> 4) << 16);
}
__device__ __forceinline__ constexpr uint32_t desc_hi(uint32_t sbo, uint32_t swizzle) {
  return (sbo >> 4) | (1u << 14) | (swizzle << 29);
}
__device__ __forceinline__ void tc_mma_f16_words(uint32_t tmem_d, uint32_t alo, uint32_t ahi, uint32_t blo, uint32_t bhi,
                                                 uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %6, 0;\n mov.b64 a, {%1, %2};\n mov.b64 b, {%3, %4};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n}\n" ::"r"(tmem_d), "r"(alo), "r"(ahi), "r"(blo),
      "r"(bhi), "r"(idesc), "r"(accumulate) : "memory");
}
// f16 x f16 -> f32, M = 128; ta, tb: operand is M-major (N-major).
__device__ __forceinline__ uint32_t idesc_f16(int n, uint32_t ta, uint32_t tb) {
  return (1u << 4) | (ta << 15) | (tb << 16) | ((static_cast<uint32_t>(n) >> 3) << 17) | ((128u >> 4) << 24);
}

// Byte offset of (row, byte of the row) in a tile: groups of 8 rows, 2 KB each.
// 8-byte entries: two channel blocks of 8 x 128 bytes, 16-byte pieces swizzled by
// the row. 16-byte entries: pieces of 8 rows x 16 bytes without a swizzle (the
// rotation of the rows would undo it: lane i writes group s + i of row i).
template <int ENTRY>
__device__ __forceinline__ uint32_t tile_off(int row, int byte) {
  if constexpr (ENTRY == 16) return static_cast<uint32_t>((row >> 3) * 2048 + (byte >> 4) * 128 + (row & 7) * 16);
  return static_cast<uint32_t>((row >> 3) * 2048 + (byte >> 7) * 1024 + (row & 7) * 128 +
                               (((byte & 127) & ~15) ^ ((row & 7) << 4)) + (byte & 15));
}

template <int BYTES>
struct Word {
  uint32_t w[BYTES / 4];
};
// Shared word(s) at window address a + OFF.
template <int BYTES, uint32_t OFF>
__device__ __forceinline__ Word<BYTES> lds(uint32_t a) {
  Word<BYTES> r;
  if constexpr (BYTES == 16)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4+%5];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]) : "r"(a), "n"(OFF));
  else
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2+%3];" : "=r"(r.w[0]), "=r"(r.w[1]) : "r"(a), "n"(OFF));
  return r;
}
template <int BYTES, uint32_t OFF>
__device__ __forceinline__ void sts(uint32_t a, const Word<BYTES>& r) {
  if constexpr (BYTES == 16)
    asm volatile("st.shared.v4.b32 [%0+%5], {%1, %2, %3, %4};" ::"r"(a), "r"(r.w[0]), "r"(r.w[1]), "r"(r.w[2]),
                 "r"(r.w[3]), "n"(OFF) : "memory");
  else
    asm volatile("st.shared.v2.b32 [%0+%3], {%1, %2};" ::"r"(a), "r"(r.w[0]), "r"(r.w[1]), "n"(OFF) : "memory");
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// NC columns of this warp's 32 TMEM lanes.
template <int NC>
__device__ __forceinline__ void tld(uint32_t a, uint32_t (&r)[NC]) {
  if constexpr (NC == 32) {
    tld32(a, r);
  } else if constexpr (NC == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(a));
  } else {
    static_assert(NC == 8, "8, 16 or 32 columns");
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(a));
  }
}
__device__ __forceinline__ void tst8(uint32_t a, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(a), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]) : "memory");
}
__device__ __forceinline__ void tld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tst_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
template <int R>
__device__ __forceinline__ void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
__device__ __forceinline__ void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("barrier.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ bool named_or(int id, int threads, bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %3, 0;\n barrier.red.or.pred q, %1, %2, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r) : "r"(id), "r"(threads), "r"(v ? 1u : 0u) : "memory");
  return r != 0u;
}
__device__ __forceinline__ float redux_fmax(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// 2^k for -126 <= k <= 127.
__device__ __forceinline__ float pow2(int k) { return __int_as_float((127 + k) << 23); }

// Power of two that brings values of magnitude `top` just below 2^14. For 0 (or
// no finite value) the largest one: what a table of zeros is multiplied with then
// counts least when the query's own scale is chosen.
__device__ __forceinline__ int scale_exp(float top) {
  return top > 0.f ? min(126, 13 - ilogbf(top)) : 126;     // -114 for the largest floats
}

__device__ __forceinline__ float finite_abs(float v) {
  const float a = fabsf(v);
  return a < INFINITY ? a : 0.f;
}

// Quantised tokens of sequence b.
__device__ __forceinline__ int seq_vq(const SharedParams& p, int b) {
  return max(0, min(max(0, __ldg(p.seq_lens + b)) - p.W, p.max_vq));
}

// Group of sequence b (-1: none; else b is one of the rows that group_info
// counts); every lane of the warp calls it.
__device__ __forceinline__ int group_of(const SharedParams& p, int b, int lane) {
  int n = 0;
  for (int i = lane; i < p.n_groups; i += 32) n += __ldg(p.group_starts + 1 + i) <= b ? 1 : 0;
  const int g = __reduce_add_sync(0xffffffffu, n);
  if (g >= p.n_groups) return -1;
  const GroupSpan s = group_span(__ldg(p.group_starts + g), __ldg(p.group_starts + g + 1), p.B, p.max_group);
  return b >= s.lo && b - s.lo < s.n ? g : -1;
}
__device__ __forceinline__ int group_shared(const SharedParams& p, int g) {
  return max(0, min(__ldg(p.shared_lens + g), p.max_shared));
}

// Tokens of the tensor-core setup of a unit, in tiles: what a block that starts
// a unit spends on its tables, queries, first tile and records.
constexpr int kSetupTiles = 5;

struct Group {
  int lo, rows, S, tiles;         // first sequence, query rows, shared tokens and tiles
  int64_t cost;                   // of its row tiles per head
};
template <int TOK, int N>
__device__ __forceinline__ Group group_info(const SharedParams& p, int g) {
  Group r{0, 0, 0, 0, 0};
  if (g < p.n_groups) {
    const GroupSpan s = group_span(__ldg(p.group_starts + g), __ldg(p.group_starts + g + 1), p.B, p.max_group);
    r.lo = s.lo;
    r.rows = s.n * p.ratio;
    r.S = group_shared(p, g);
    r.tiles = (r.S + TOK - 1) / TOK;
    r.cost = r.tiles > 0 ? static_cast<int64_t>((r.rows + N - 1) / N) * (r.tiles + kSetupTiles) : 0;
  }
  return r;
}

// Where every block of the shared grid starts (one block of kE threads).
template <int TOK, int N>
__device__ void plan_walks(const SharedParams& p) {
  __shared__ int64_t incl[kE];
  __shared__ int64_t part[kE / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // inclusive sums of the costs of groups g0 .. g0 + kE - 1 into incl
  auto scan = [&](int g0) {
    int64_t v = group_info<TOK, N>(p, g0 + tid).cost;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t t = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += t;
    }
    __syncthreads();
    if (lane == 31) part[warp] = v;
    __syncthreads();
    for (int w = 0; w < warp; ++w) v += part[w];
    incl[tid] = v;
    __syncthreads();
  };
  int64_t Ug = 0;
  for (int g0 = 0; g0 < p.n_groups; g0 += kE) {
    scan(g0);
    Ug += incl[kE - 1];
  }
  const int64_t U = Ug * p.Hkv, n = min(static_cast<int64_t>(p.shared_blocks), U);
  for (int c0 = 0; c0 < p.shared_blocks; c0 += kE) {
    const int c = c0 + tid;
    Walk w{};
    w.U = U;
    w.n = n;
    w.head = -1;
    int64_t x = -1;
    if (c < n) {
      w.at = U * c / n;
      w.end = U * (c + 1) / n;
      w.hkv = static_cast<int>(w.at / Ug);
      x = w.at - w.hkv * Ug;
    }
    int64_t before = 0;                                    // cost of the groups before g0
    for (int g0 = 0; g0 < p.n_groups; g0 += kE) {
      if (p.n_groups > kE) scan(g0);                       // (else incl still holds the only sums)
      if (x >= before && x < before + incl[kE - 1]) {
        int a = 0, z = kE - 1;                             // first group whose inclusive sum passes x
        while (a < z) {
          const int mid = (a + z) / 2;
          if (before + incl[mid] > x) z = mid; else a = mid + 1;
        }
        const Group r = group_info<TOK, N>(p, g0 + a);
        const int64_t off = x - before - (a > 0 ? incl[a - 1] : 0);
        const int cost = r.tiles + kSetupTiles;
        w.g = g0 + a;
        w.rt = static_cast<int>(off / cost);
        w.pos = static_cast<int>(off % cost);
        w.lo = r.lo;
        w.rows = r.rows;
        w.S = r.S;
        w.tiles = r.tiles;
      }
      before += incl[kE - 1];
    }
    if (c < p.shared_blocks) p.walks[c] = w;
  }
}

// The codebook slices of one call as fp16 tables: block (4 channel groups, K or
// V, head), thread = codeword. Each group is scaled by a power of two of its
// own. Also the split of every sequence into shared and own tokens and, in a block
// of its own, where the shared grid's blocks start. The shared grid's blocks start
// meanwhile and wait for this grid. 16 heads of 128 read 4.2 MB and write 2.1 MB in
// 5 us, a launch's latency and two dependent loads.
template <int J, int C, int N>
__global__ void __launch_bounds__(kE) shared_table_kernel(const float* cb_k, const float* cb_v, int64_t cb_stride_head,
                                                          unsigned char* tables, int* exps, const SharedParams p) {
  __shared__ float red[4][kE / 32];
  asm volatile("griddepcontrol.launch_dependents;");
  {                                                        // a warp per sequence: its shared and own tokens
    const int lane = threadIdx.x & 31, blocks = gridDim.x * gridDim.y * gridDim.z;
    const int id = (blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x;
    for (int g = id * kE + static_cast<int>(threadIdx.x); g < p.n_groups; g += blocks * kE) {
      const int lo = __ldg(p.group_starts + g), hi = __ldg(p.group_starts + g + 1), s = __ldg(p.shared_lens + g);
      // (the difference is taken of ends inside [0, B] only)
      if ((lo < 0 || hi > p.B || hi < lo || hi - lo > p.max_group || s < 0 || s > p.max_shared) && p.status != nullptr)
        atomicOr(p.status, LOOPVQ_DECODE_STATUS_BAD_GROUP);
    }
    for (int b = id + static_cast<int>(threadIdx.x >> 5) * blocks; b < p.B; b += blocks * (kE / 32)) {
      const int n_vq = seq_vq(p, b), g = group_of(p, b, lane);
      const int s0 = g < 0 ? 0 : min(group_shared(p, g), n_vq), n_own = min(n_vq - s0, p.max_own);
      if (lane == 0) {
        p.seqs[b] = make_int2(s0, n_own);
        if (n_own < n_vq - s0 && p.status != nullptr) atomicOr(p.status, LOOPVQ_DECODE_STATUS_BAD_GROUP);
      }
    }
  }
  if (blockIdx.z == static_cast<unsigned>(p.Hkv)) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && p.shared_blocks > 0) plan_walks<Shape<J, C>::TOK, N>(p);
    return;
  }
  const int j0 = blockIdx.x * 4, kv = blockIdx.y, h = blockIdx.z, e = threadIdx.x;
  const float* cb = (kv ? cb_v : cb_k) + h * cb_stride_head;
  float4 v[4][C / 4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int i = 0; i < C / 4; ++i)
      v[k][i] = __ldg(reinterpret_cast<const float4*>(cb + (static_cast<size_t>(j0 + k) * kE + e) * C) + i);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < C / 4; ++i)
      top = fmaxf(fmaxf(top, fmaxf(finite_abs(v[k][i].x), finite_abs(v[k][i].y))),
                  fmaxf(finite_abs(v[k][i].z), finite_abs(v[k][i].w)));
    top = redux_fmax(top);
    if ((e & 31) == 0) red[k][e >> 5] = top;
  }
  __syncthreads();
  uint32_t w[2 * C];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < kE / 32; ++i) top = fmaxf(top, red[k][i]);
    const int add = kv ? kRecExp : 0, ex = min(scale_exp(top), 126 - add);
    const float f = pow2(ex);
    if (e == 0) exps[(h * 2 + kv) * 32 + j0 + k] = ex + add;
#pragma unroll
    for (int i = 0; i < C / 4; ++i) {
      w[k * (C / 2) + 2 * i] = half2_bits(v[k][i].x * f, v[k][i].y * f);
      w[k * (C / 2) + 2 * i + 1] = half2_bits(v[k][i].z * f, v[k][i].w * f);
    }
  }
  uint4* dst = reinterpret_cast<uint4*>(tables + (static_cast<size_t>(h) * 2 + kv) * kTabBytes + e * 256 + j0 * 2 * C);
#pragma unroll
  for (int i = 0; i < C / 2; ++i) dst[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
}

// Requests a table of a head (which: 0 K, 1 V) into shared memory (one thread).
__device__ __forceinline__ void request_table(const SharedParams& p, unsigned char* sm, int hkv, int which, uint32_t bar) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(kTabBytes) : "memory");
  const unsigned char* src = p.tables + (static_cast<size_t>(hkv) * 2 + which) * kTabBytes;
  for (int part = 0; part < 2; ++part)
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     u32s(sm + which * kTabBytes + part * (kTabBytes / 2))),
                 "l"(src + part * (kTabBytes / 2)), "r"(kTabBytes / 2), "r"(bar) : "memory");
}

// Dequantises this lane's slot of a block: the w_n (up to W0) index words iw of
// its row select entries of the table TAB, stored to its row of the tile TILE
// at the places `at` gives (zeros for a slot at or past nv).
template <int J, int C, int TAB, int TILE, int W0>
__device__ __forceinline__ void fill_block(const uint32_t (&iw)[W0], const uint32_t (&at)[4 * W0], int w_n, int nv,
                                           int lane) {
  constexpr int ENTRY = Shape<J, C>::ENTRY, LB = Shape<J, C>::LB;
  const bool whole = nv >= LB;                             // warp-uniform
#pragma unroll
  for (int w = 0; w < W0; ++w) {
    if (w < w_n) {                                         // warp-uniform
      Word<ENTRY> e[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)                          // codeword row (byte 1) | entry (byte 0)
        e[i] = lds<ENTRY, kShBase + TAB>(__byte_perm(iw[w], at[4 * w + i], 0x5504u | (static_cast<uint32_t>(i) << 4)));
      if (!whole && lane >= nv) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int k = 0; k < ENTRY / 4; ++k) e[i].w[k] = 0u;
      }
      if (lane < LB) {
#pragma unroll
        for (int i = 0; i < 4; ++i) sts<ENTRY, kShBase + TILE>(at[4 * w + i] >> 16, e[i]);
      }
    }
  }
}

// ---- shared blocks ---------------------------------------------------------------

// One run of tiles of a unit (group, row tile, head) in a block, in shared memory.
struct Segment {
  int hkv, rt, lo, rows;          // lo: the group's first sequence; rows: the unit's query rows
  int S, tile0, nt;               // shared tokens of the group, tiles [tile0, tile0 + nt)
  int load;                       // the head's tables are not in shared memory yet
  int64_t rec;                    // record of row 0
  int64_t pad;
};

// Query row c of the unit as (sequence, query head).
template <int N>
__device__ __forceinline__ int64_t pair_of(const SharedParams& p, const Segment& u, int c) {
  const int r = u.rt * N + c;
  return static_cast<int64_t>(u.lo + r / p.ratio) * p.Hq + u.hkv * p.ratio + r % p.ratio;
}

// Returns false when a bounded wait gave up (the status word is flagged, the
// records are NaN and nothing is in flight, or the flag says so).
template <int J, int C, int N>
__device__ bool shared_segment(const SharedParams& p, unsigned char* sm, const Segment& u, uint32_t tmem) {
  using T = Shape<J, C>;
  constexpr int D = T::D, NC = N / 2;
  // P: rows of 64 query rows and one buffer, or of 32 and two (the same bytes)
  constexpr int PP = N > 32 ? 128 : 64, PB = N > 32 ? 1 : 2;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  float* m_ref = reinterpret_cast<float*>(sm + kMOff);
  float* cm = reinterpret_cast<float*>(sm + kCmOff);
  float* al = reinterpret_cast<float*>(sm + kAlOff);
  int* lim = reinterpret_cast<int*>(sm + kLimOff);
  volatile int* nvs = reinterpret_cast<volatile int*>(sm + kNvOff);
  float* sc = reinterpret_cast<float*>(sm + kScOff);
  int* row_top = reinterpret_cast<int*>(sm + kAlOff);      // until the first raise: a row's largest magnitude
  auto bar = [&](int i) { return u32s(sm + kBarOff) + 8u * i; };
  const int rows = u.rows, S = u.S, tile0 = u.tile0, nt = u.nt, hkv = u.hkv;

  // ---- setup: barriers, tables, queries -------------------------------------------
  if (tid == 0) {                                          // (kernel start, or after a segment's last barrier)
    for (int i = 0; i < kBars; ++i) {
      const uint32_t n = (i == kBarK || i == kBarV) ? kDeqWarps : (i == kBarP0 || i == kBarP1) ? kSoftWarps : 1;
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar(i)), "r"(n) : "memory");
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if (u.load) request_table(p, sm, hkv, 0, bar(kBarTabK));
  }
  const int* exk = p.exps + hkv * 64;
  // a row's shared tokens and its unset reference (the last threads; the first ones
  // have the queries)
  if (const int c = kShThreads - 1 - tid; c < N) {
    lim[c] = c < rows ? min(S, seq_vq(p, static_cast<int>(pair_of<N>(p, u, c) / p.Hq))) : INT_MAX;
    m_ref[c] = kUnset;
    row_top[c] = 0;
  }
  // The queries, scaled into fp16 by a power of two 2^kq (against the scales of the
  // key groups): one for all rows while their largest magnitudes are within
  // 2^kRowSpan of each other, else one per row, so that no row's magnitude costs
  // another its bits. Piece = 8 channels of a row.
  int kq;
  bool one_scale;
  {
    constexpr int PIECES = N * D / 8, PER = (PIECES + kShThreads - 1) / kShThreads;
    float v[PER][8], top[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      top[k] = 0.f;
      const int f = tid + k * kShThreads, c = f / (D / 8), part = f % (D / 8);
      uint4 t = make_uint4(0u, 0u, 0u, 0u);
      if (f < PIECES && c < rows) t = *(reinterpret_cast<const uint4*>(p.q + pair_of<N>(p, u, c) * D) + part);
      const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float f2 = pow2(f < PIECES ? -__ldcg(exk + (part * 8 + 2 * i) / C) : 0);
        const float2 a = bf16x2_to_float2(w[i]);
        v[k][2 * i] = a.x * f2;
        v[k][2 * i + 1] = a.y * f2;
        top[k] = fmaxf(top[k], fmaxf(finite_abs(v[k][2 * i]), finite_abs(v[k][2 * i + 1])));
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < PER; ++k) {                        // (magnitudes order as their bits do)
      const int f = tid + k * kShThreads;
      if (f < PIECES) atomicMax(row_top + f / (D / 8), __float_as_int(top[k]));
    }
    __syncthreads();
    {
      const int t0 = row_top[lane % N], t1 = row_top[(lane + 32) % N];
      const int least = min(t0 > 0 ? t0 : INT_MAX, t1 > 0 ? t1 : INT_MAX);   // (zero rows fit any scale)
      kq = scale_exp(__int_as_float(__reduce_max_sync(0xffffffffu, max(t0, t1))));
      const int lo = __reduce_min_sync(0xffffffffu, least);
      one_scale = lo == INT_MAX || scale_exp(__int_as_float(lo)) - kq <= kRowSpan;
      if (const int c = kShThreads - 1 - tid; c < N) sc[c] = pow2(-scale_exp(__int_as_float(row_top[c])));
    }
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int f = tid + k * kShThreads, c = f / (D / 8), byte = (f % (D / 8)) * 16;
      if (f >= PIECES) continue;
      const float f2 = pow2(one_scale ? kq : scale_exp(__int_as_float(row_top[c])));
      *reinterpret_cast<uint4*>(sm + kQOff + (byte >> 7) * (N * 128) + c * 128 + ((byte & 127) ^ ((c & 7) << 4))) =
          make_uint4(half2_bits(v[k][0] * f2, v[k][1] * f2), half2_bits(v[k][2] * f2, v[k][3] * f2),
                     half2_bits(v[k][4] * f2, v[k][5] * f2), half2_bits(v[k][6] * f2, v[k][7] * f2));
    }
  }
  const float scale = one_scale ? ldexpf(p.scale_log2, -kq) : p.scale_log2;
  if constexpr (T::LB < 32) {
    for (int i = tid; i < kTileBytes / 16; i += kShThreads)
      *reinterpret_cast<uint4*>(sm + kVtileOff + i * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
  proxy_fence();
  tc_before();
  __syncthreads();
  tc_after();
  const int min_lim = __reduce_min_sync(0xffffffffu, min(lim[lane % N], lim[(lane + 32) % N]));
  bool failed = false;                                     // this thread's wait gave up
  const int tok0 = tile0 * T::TOK;                         // first token of the split

  if (warp >= kKWarp && warp < kMmaWarp) {
    // ---- dequantisation: a team of eight warps per plane ------------------------------
    if constexpr (N > 32) reg_dec<kDeqRegs>();
    const bool values = warp >= kVWarp;
    const int blk = warp & 3, half = (warp >> 2) & 1;
    constexpr int W0 = (T::NW + 1) / 2;                    // index words of half 0 (half 1: the rest)
    const int w_first = half ? W0 : 0, w_n = half ? T::NW - W0 : W0;
    const int row = blk * 32 + lane;
    // per position: byte 0 its entry's place in a table row, bytes 2-3 its place
    // in a tile (below 32 KB)
    uint32_t at[4 * W0];
#pragma unroll
    for (int w = 0; w < 4 * W0; ++w) {
      const int j = (w_first * 4 + w + lane) % J;
      at[w] = static_cast<uint32_t>(j * T::ENTRY) | (tile_off<T::ENTRY>(row, j * T::ENTRY) << 16);
    }
    // this lane's row in block 0 of page 0 (granule of its first word)
    const uint8_t* rows0 = p.pool_lg + hkv * p.pool_stride_head + (values ? p.plane_bytes : 0) + lane * T::GR +
                           (J == 32 ? half * (T::LB * 16) : 0);
    const int32_t* bt = p.block_table + static_cast<int64_t>(u.lo) * p.max_pages_per_seq;
    const int blk0 = tile0 * 4 + blk;                      // this warp's block of tile i: blk0 + 4 i
    // page-table entries of this warp's blocks of tiles e0 .. e0 + 31 (lane = tile)
    int e0 = 0, entry;
    auto load_entries = [&]() {
      const int b = blk0 + (e0 + lane) * 4;
      entry = e0 + lane < nt && b * T::LB < S ? __ldg(bt + (b >> p.lbpp)) : 0;
      if (entry < 0 || entry >= p.n_pages) {
        if (p.status != nullptr) atomicOr(p.status, LOOPVQ_DECODE_STATUS_BAD_PAGE);
        entry = -1;
      }
    };
    load_entries();
    // the index words of tile i, and the slots that hold a token
    auto load_rows = [&](int i, uint32_t (&w)[W0]) -> int {
      if (i >= e0 + 32) {                                  // warp-uniform
        e0 += 32;
        load_entries();
      }
      const int b = blk0 + i * 4, e = __shfl_sync(0xffffffffu, entry, i & 31);
      const int nv = i < nt && e >= 0 ? min(T::LB, S - b * T::LB) : 0;   // <= 0: none
#pragma unroll
      for (int k = 0; k < W0; ++k) w[k] = 0u;
      if (nv > 0 && lane < T::LB) {
        const uint8_t* r = rows0 + static_cast<int64_t>(e) * p.page_bytes + (b & ((1 << p.lbpp) - 1)) * (T::LB * J);
        if constexpr (J == 32) {
          const uint4 t = __ldcs(reinterpret_cast<const uint4*>(r));
          w[0] = t.x; w[1] = t.y; w[2] = t.z; w[3] = t.w;
        } else {
#pragma unroll
          for (int k = 0; k < W0; ++k) {
            const int byte = (w_first + k) * 4;
            if (k < w_n) w[k] = __ldcs(reinterpret_cast<const uint32_t*>(r + byte / T::GR * (T::LB * T::GR) + byte % T::GR));
          }
        }
      }
      return nv;
    };
    uint32_t w0[W0], w1[W0];                               // tiles i and i + 1
    int nv0 = load_rows(0, w0), nv1 = load_rows(1, w1);
    if (u.load) {
      // the value table follows the key table, so that the first keys need not
      // share the way from L2 with it
      failed = !mbar_wait(bar(kBarTabK), 0, kShSpin);
      if (warp == kVWarp && lane == 0) request_table(p, sm, hkv, 1, bar(kBarTabV));
      if (values) failed = !mbar_wait(bar(kBarTabV), 0, kShSpin) || failed;
    }
#pragma unroll 1
    for (int i = 0; i < nt; ++i) {
      // the tile is free when S^T (K) or O^T (V) of the tile before is done
      if (i > 0)
        failed = !mbar_wait(bar((values ? kBarO0 : kBarS0) + ((i - 1) & 1)), ((i - 1) >> 1) & 1, kShSpin);
      if (__any_sync(0xffffffffu, failed)) {
        failed = true;
        break;
      }
      if (values) {
        fill_block<J, C, kVtabOff, kVtileOff, W0>(w0, at, w_n, nv0, lane);
      } else {
        fill_block<J, C, kKtabOff, kKtileOff, W0>(w0, at, w_n, nv0, lane);
        if (half == 0 && lane == 0) nvs[(i & 3) * 4 + blk] = nv0;
      }
      proxy_fence();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(values ? kBarV : kBarK));
#pragma unroll
      for (int k = 0; k < W0; ++k) w0[k] = w1[k];
      nv0 = nv1;
      nv1 = load_rows(i + 2, w1);                          // lands during the next tile
    }
    if constexpr (N > 32) reg_inc<kLaunchRegs>();
  } else if (warp == kMmaWarp) {
    // ---- the products --------------------------------------------------------------
    if (lane == 0) {
      // descriptors: the high words are constant, the low words the address plus
      // an immediate
      // (K along the channels, V along the tokens; see tile_off for the two layouts)
      constexpr bool SW = T::ENTRY == 8;
      const uint32_t k_hi = desc_hi(2048, SW ? kSw128 : 0u), q_hi = desc_hi(1024, kSw128);
      const uint32_t v_hi = SW ? desc_hi(2048, kSw128) : desc_hi(128, 0u);
      const uint32_t p_hi = desc_hi(PP * 8, PP == 128 ? kSw128 : kSw64);
      const uint32_t k_lo = desc_lo(u32s(sm + kKtileOff), SW ? 16 : 128), q_lo = desc_lo(u32s(sm + kQOff), 16);
      const uint32_t v_lo = desc_lo(u32s(sm + kVtileOff), SW ? 1024 : 2048), p_lo = desc_lo(u32s(sm + kPOff), 16);
      auto product_s = [&](int i) {                        // S^T of tile i
        tc_after();
        const uint32_t d = tmem + kTmS + (i & 1) * 64;
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
          tc_mma_f16_words(d, k_lo + (SW ? (s >> 2) * 1024 + (s & 3) * 32 : s * 256) / 16, k_hi,
                           q_lo + ((s >> 2) * (N * 128) + (s & 3) * 32) / 16, q_hi, idesc_f16(N, 0, 0), s > 0 ? 1u : 0u);
        tc_commit(bar(kBarS0 + (i & 1)));
      };
      // The keys run a tile ahead, so S^T of tile i + 1 is issued before O^T of
      // tile i; its buffer is free since P of tile i - 1 was waited for.
      failed = !mbar_wait(bar(kBarK), 0, kShSpin);
      if (!failed) product_s(0);
#pragma unroll 1
      for (int i = 0; i < nt && !failed; ++i) {
        if (i + 1 < nt) {
          failed = !mbar_wait(bar(kBarK), (i + 1) & 1, kShSpin);
          if (failed) break;
          product_s(i + 1);
        }
        failed = !mbar_wait(bar(kBarP0 + i % PB), (i / PB) & 1, kShSpin) || !mbar_wait(bar(kBarV), i & 1, kShSpin);
        if (failed) break;
        tc_after();
        const uint32_t pb = p_lo + (i % PB) * (kTileRows * PP) / 16;
#pragma unroll
        for (int s = 0; s < 8; ++s)                        // O^T += V^T P, 16 tokens at a time
          tc_mma_f16_words(tmem + kTmO, v_lo + s * 4096 / 16, v_hi, pb + s * (16 * PP) / 16, p_hi, idesc_f16(N, 1, 1),
                           (i > 0 || s > 0) ? 1u : 0u);
        tc_commit(bar(kBarO0 + (i & 1)));
      }
    }
    __syncwarp();
  } else {
    // ---- softmax -------------------------------------------------------------------
    if constexpr (N > 32) reg_inc<kSoftRegs>();
    const int quad = warp & 3, half = warp >> 2, row = quad * 32 + lane, c0 = half * NC;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const int bar_id = 1 + half;                           // the four warps of a column half
    float l[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) l[c] = 0.f;
    // this half's references: in shared memory, but for 16 rows in registers (more
    // rows spilled: 100 us against 96 with 32 rows, 40 heads and 16312 tokens)
    float4 m4[N > 16 ? 1 : NC / 4];
#pragma unroll
    for (int c = 0; c < (N > 16 ? 1 : NC / 4); ++c) m4[c] = make_float4(kUnset, kUnset, kUnset, kUnset);
    auto refs = [&](int c) { return N > 16 ? *reinterpret_cast<const float4*>(m_ref + c0 + c) : m4[c / 4]; };
#pragma unroll 1
    for (int i = 0; i < nt; ++i) {
      failed = !mbar_wait(bar(kBarS0 + (i & 1)), (i >> 1) & 1, kShSpin) || failed;
      __syncwarp();
      tc_after();
      const int nv = nvs[(i & 3) * 4 + quad];
      const bool masked = tok0 + (i + 1) * T::TOK > min_lim;   // some row ends inside this tile
      const int tok = tok0 + i * T::TOK + quad * T::LB + lane;
      // this token's scores, -inf where there is none
      uint32_t sv[NC];
      tld<NC>(lanes + kTmS + (i & 1) * 64 + c0, sv);
      tld_wait();
      if (!one_scale) {                                    // block-uniform; exact, but for scores out of float32's range
#pragma unroll
        for (int c = 0; c < NC; ++c) sv[c] = __float_as_uint(__uint_as_float(sv[c]) * sc[c0 + c]);
      }
      if (nv < 32 && lane >= nv) {                         // no token in this slot
#pragma unroll
        for (int c = 0; c < NC; ++c) sv[c] = 0xff800000u;
      }
      if (masked) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
          if (tok >= lim[c0 + c]) sv[c] = 0xff800000u;
      }
      float mx = -INFINITY;
#pragma unroll
      for (int c = 0; c < NC; c += 4) {
        const float4 mm = refs(c);
        mx = fmaxf(mx, fmaxf(fmaf(__uint_as_float(sv[c]), scale, -mm.x), fmaf(__uint_as_float(sv[c + 1]), scale, -mm.y)));
        mx = fmaxf(mx, fmaxf(fmaf(__uint_as_float(sv[c + 2]), scale, -mm.z), fmaf(__uint_as_float(sv[c + 3]), scale, -mm.w)));
      }
      if (named_or(bar_id, 128, mx > kRaise || failed)) {
        if (i > 0) failed = !mbar_wait(bar(kBarO0 + ((i - 1) & 1)), ((i - 1) >> 1) & 1, kShSpin) || failed;
        if (named_or(bar_id, 128, failed)) {               // uniform over the four warps
          failed = true;
          break;
        }
        __syncwarp();
        tc_after();
        // raise the references that were passed; l and O^T shrink with them. Lane c
        // keeps column c's maximum over the warp's tokens.
        float top = -INFINITY;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const float t = redux_fmax(__uint_as_float(sv[c]) * scale);
          if (lane == c) top = t;
        }
        if (lane < NC) cm[quad * kMaxRows + c0 + lane] = top;
        named_sync(bar_id, 128);
        if (quad == 0 && lane < NC) {
          const int c = c0 + lane;
          const float t = fmaxf(fmaxf(cm[c], cm[kMaxRows + c]), fmaxf(cm[2 * kMaxRows + c], cm[3 * kMaxRows + c]));
          const float was = m_ref[c], now = t > was + kRaise ? t - kTop : was;
          m_ref[c] = now;
          al[c] = fast_exp2(was - now);
        }
        named_sync(bar_id, 128);                           // references and factors written; cm is free
#pragma unroll
        for (int c = 0; c < NC; c += 4) {
          if (N <= 16) m4[c / 4] = *reinterpret_cast<const float4*>(m_ref + c0 + c);
          const float4 f = *reinterpret_cast<const float4*>(al + c0 + c);
          l[c] *= f.x;
          l[c + 1] *= f.y;
          l[c + 2] *= f.z;
          l[c + 3] *= f.w;
        }
        if (i > 0) {
#pragma unroll 1
          for (int c = 0; c < NC; c += 8) {
            uint32_t o[8];
            tld<8>(lanes + kTmO + c0 + c, o);
            tld_wait();
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * al[c0 + c + k]);
            tst8(lanes + kTmO + c0 + c, o);
          }
          tst_wait();
        }
        named_sync(bar_id, 128);                           // the factors are read
      }
      // the weights, in registers until the products that read P's buffer are done
      uint32_t w[NC / 2];
#pragma unroll
      for (int c = 0; c < NC; c += 4) {
        const float4 mm = refs(c);
        const float e0 = fast_exp2(fmaf(__uint_as_float(sv[c]), scale, -mm.x));
        const float e1 = fast_exp2(fmaf(__uint_as_float(sv[c + 1]), scale, -mm.y));
        const float e2 = fast_exp2(fmaf(__uint_as_float(sv[c + 2]), scale, -mm.z));
        const float e3 = fast_exp2(fmaf(__uint_as_float(sv[c + 3]), scale, -mm.w));
        l[c] += e0;
        l[c + 1] += e1;
        l[c + 2] += e2;
        l[c + 3] += e3;
        w[c / 2] = half2_bits(e0, e1);
        w[c / 2 + 1] = half2_bits(e2, e3);
      }
      if (i >= PB) failed = !mbar_wait(bar(kBarO0 + ((i - PB) & 1)), ((i - PB) >> 1) & 1, kShSpin) || failed;
      unsigned char* prow = sm + kPOff + (i % PB) * (kTileRows * PP) + row * PP;
      const int swz = PP == 128 ? row & 7 : (row >> 1) & 3;
#pragma unroll
      for (int c = 0; c < NC; c += 8)
        *reinterpret_cast<uint4*>(prow + ((((c0 + c) >> 3) ^ swz) << 4)) =
            make_uint4(w[c / 2], w[c / 2 + 1], w[c / 2 + 2], w[c / 2 + 3]);
      proxy_fence();
      tc_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarP0 + i % PB));
    }
    if (!failed) failed = !mbar_wait(bar(kBarO0 + ((nt - 1) & 1)), ((nt - 1) >> 1) & 1, kShSpin);
    __syncwarp();
    failed = named_or(bar_id, 128, failed);
    if (!failed) {
      // ---- the rows' records: o from TMEM (lane = channel), m and l ------------------
      tc_after();
      const float unscale = row < D ? pow2(-__ldcg(exk + 32 + row / C)) : 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const float t = warp_sum(l[c]);
        if (lane == 0) cm[quad * kMaxRows + c0 + c] = t;
      }
#pragma unroll 1
      for (int c = 0; c < NC; c += 8) {
        uint32_t o[8];
        tld<8>(lanes + kTmO + c0 + c, o);
        tld_wait();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (c0 + c + k < rows && row < D)
            p.srec[(u.rec + c0 + c + k) * T::RS + 4 + row] = __uint_as_float(o[k]) * unscale;
        }
      }
      named_sync(bar_id, 128);
      if (quad == 0 && lane < NC && c0 + lane < rows) {
        const int c = c0 + lane;
        const float t = cm[c] + cm[kMaxRows + c] + cm[2 * kMaxRows + c] + cm[3 * kMaxRows + c];
        float* rec = p.srec + (u.rec + c) * T::RS;
        rec[0] = t == 0.f ? -INFINITY : m_ref[c];
        rec[1] = t;
      }
    }
    if constexpr (N > 32) reg_dec<kLaunchRegs>();
  }
  const bool any_failed = __syncthreads_or(failed);
  if (any_failed) {
    // a bounded wait gave up: wait for what was issued, flag, poison the records.
    // (The thread that issued the products commits them only here: every other
    // arrival of a segment is waited for before its barriers are invalidated, and
    // one that nobody waits for could come after.)
    if (tid == kMmaWarp * 32) {
      tc_commit(bar(kBarDrain));
      const bool drained = mbar_wait(bar(kBarDrain), 0, kShDrainSpin) &&
                           (!u.load || (mbar_wait(bar(kBarTabK), 0, kShDrainSpin) && mbar_wait(bar(kBarTabV), 0, kShDrainSpin)));
      if (p.status != nullptr)
        atomicOr(p.status, drained ? LOOPVQ_DECODE_STATUS_TIMEOUT
                                   : (LOOPVQ_DECODE_STATUS_TIMEOUT | LOOPVQ_DECODE_STATUS_UNDRAINED));
    }
  }
  __syncthreads();
  if (tid == 0) {
    for (int i = 0; i < kBars; ++i) asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(bar(i)) : "memory");
  }
  return !any_failed;
}

// A persistent grid over the tiles of all units, heads outermost. A unit counts
// kSetupTiles + its tiles; block c of n takes the c-th n-th of the total U, so
// every block does the same work whatever the groups' sizes and lengths, and
// meets one or a few units. Its records go to rows R + c*N .., R the rows of the
// units before: since R and c both grow along the blocks, no two collide.
// 16 x 32696 tokens of d = 128 with 8 rows on 140 blocks: 47.9 us, 36 MB from HBM
// (0.75 TB/s: not the bound), shared-memory lookups and stores at 44% of an SM's
// rate and the products' reads at 26% by their bytes; the rest is the hand-over
// between fill, products and softmax. With 64 rows on 100 blocks, 16312 tokens of
// 16 heads and 4 row tiles: 159 us.
template <int J, int C, int N>
__global__ void __launch_bounds__(kShThreads, 1) shared_prefix_kernel(const SharedParams p) {
  using T = Shape<J, C>;
  extern __shared__ __align__(1024) unsigned char sm[];
  if (u32s(sm) != kShBase) {                               // the host checks this before launching
    if (threadIdx.x == 0 && p.status != nullptr) atomicOr(p.status, LOOPVQ_DECODE_STATUS_SHARED_BASE);
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + kTmemSlotOff);
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(u32s(tmem_slot)),
                 "r"(kTmCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // The walk is kept in shared memory, so that the roles' loops have the registers
  // to themselves.
  Segment* seg = reinterpret_cast<Segment*>(sm + kSegOff);
  Walk* walk = reinterpret_cast<Walk*>(sm + kSegOff + sizeof(Segment));
  static_assert(sizeof(Segment) % 16 == 0 && sizeof(Segment) + sizeof(Walk) <= kTmemSlotOff - kSegOff, "segment and walk fit");
  asm volatile("griddepcontrol.wait;" ::: "memory");       // the tables are written
  asm volatile("griddepcontrol.launch_dependents;");       // ... so the own grid may start
  if (tid < static_cast<int>(sizeof(Walk) / 16))
    reinterpret_cast<uint4*>(walk)[tid] = __ldcg(reinterpret_cast<const uint4*>(p.walks + blockIdx.x) + tid);
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = *tmem_slot;
  bool ok = true;
  while (walk->at < walk->end) {                           // block-uniform
    if (tid == 0) {
      const Walk w = *walk;
      const int cost = w.tiles + kSetupTiles, take = static_cast<int>(min(static_cast<int64_t>(cost - w.pos), w.end - w.at));
      Segment u;
      u.hkv = w.hkv;
      u.rt = w.rt;
      u.lo = w.lo;
      u.rows = min(w.rows - w.rt * N, N);
      u.S = w.S;
      u.tile0 = max(w.pos - kSetupTiles, 0);
      u.nt = max(w.pos + take - kSetupTiles, 0) - u.tile0;
      u.rec = (static_cast<int64_t>(w.hkv) * p.B + w.lo) * p.ratio + w.rt * N + static_cast<int64_t>(blockIdx.x) * N;
      u.load = w.hkv != w.head;
      *seg = u;
      if (u.nt > 0) walk->head = w.hkv;
    }
    __syncthreads();
    if (seg->nt > 0 && ok) ok = shared_segment<J, C, N>(p, sm, *seg, tmem);
    if (seg->nt <= 0 || !ok) {                             // no tiles, or given up
      for (int c = tid; c < seg->rows; c += kShThreads) {
        p.srec[(seg->rec + c) * T::RS] = ok ? -INFINITY : NAN;
        p.srec[(seg->rec + c) * T::RS + 1] = ok ? 0.f : 1.f;
      }
    }
    if (walk->pos == 0) {                                  // the unit's first block: where its rows' records are
      const int64_t at = walk->at, n = walk->n, U = walk->U;
      const int64_t c0 = ((at + 1) * n - 1) / U, c1 = ((at + walk->tiles + kSetupTiles) * n - 1) / U;
      for (int c = tid; c < seg->rows; c += kShThreads)
        p.spans[pair_of<N>(p, *seg, c)] =
            make_int2(static_cast<int>(seg->rec + (c0 - blockIdx.x) * N + c), static_cast<int>(c1 - c0 + 1));
    }
    __syncthreads();                                       // the segment is read
    if (tid == 0) {                                        // next row tile, group with shared tokens, head
      Walk w = *walk;
      w.at += min(static_cast<int64_t>(w.tiles + kSetupTiles - w.pos), w.end - w.at);
      w.pos = 0;
      if (++w.rt * N >= w.rows && w.at < w.end) {
        w.rt = 0;
        Group r;
        do {
          if (++w.g == p.n_groups) {
            w.g = 0;
            ++w.hkv;
          }
          r = group_info<T::TOK, N>(p, w.g);
        } while (r.cost == 0);
        w.lo = r.lo;
        w.rows = r.rows;
        w.S = r.S;
        w.tiles = r.tiles;
      }
      *walk = w;
    }
    __syncthreads();
  }
  tc_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmCols) : "memory");
  }
}

// ---- own blocks ------------------------------------------------------------------

// Per-warp scratch of an own block: value index rows (each twice over, so that
// group j of slot k sits at byte J - k + j of its row), the query in fp16 twice
// over (so that lane i finds group (i + s) mod J at entry i + s), and a block's
// softmax weights in fp16.
constexpr int kOwnPitch = 80;                              // bytes of an index row (conflict-free 16-byte stores)
constexpr int kOwnRows = 0;
constexpr int kOwnQ = 32 * kOwnPitch;
constexpr int kOwnP = kOwnQ + 768;
constexpr int kOwnBytes = kOwnP + 64;
constexpr int kOwnWarps = 16;
constexpr int kOwnFkOff = 2 * kTabBytes;                   // float [32]: 2^-exps of the key groups
constexpr int kOwnScratch = kOwnFkOff + 128;
constexpr int kOwnBarOff = kOwnScratch + kOwnWarps * kOwnBytes;
constexpr int kOwnSmem = kOwnBarOff + 16;
static_assert(kOwnSmem <= 227 * 1024, "shared memory above 227 KB");

// acc += a . b over the two fp16 of each word, products exact, float32 sums
// (mixed-precision multiply-add: no conversion instructions).
__device__ __forceinline__ void dot_f16(float& acc, uint32_t a, uint32_t b) {
  asm("{\n .reg .b16 al, ah, bl, bh;\n mov.b32 {al, ah}, %1;\n mov.b32 {bl, bh}, %2;\n"
      " fma.rn.f32.f16 %0, al, bl, %0;\n fma.rn.f32.f16 %0, ah, bh, %0;\n}\n" : "+f"(acc) : "r"(a), "r"(b));
}
// The same over two bf16.
__device__ __forceinline__ void dot_bf16(float& acc, uint32_t a, uint32_t b) {
  asm("{\n .reg .b16 al, ah, bl, bh;\n mov.b32 {al, ah}, %1;\n mov.b32 {bl, bh}, %2;\n"
      " fma.rn.f32.bf16 %0, al, bl, %0;\n fma.rn.f32.bf16 %0, ah, bh, %0;\n}\n" : "+f"(acc) : "r"(a), "r"(b));
}
// (x, y) += w * v over the two fp16 of v; w the low (0) or high (1) fp16 of its word.
template <int HIGH>
__device__ __forceinline__ void axpy_f16(float& x, float& y, uint32_t w, uint32_t v) {
  if constexpr (HIGH)
    asm("{\n .reg .b16 wl, wh, vl, vh;\n mov.b32 {wl, wh}, %2;\n mov.b32 {vl, vh}, %3;\n"
        " fma.rn.f32.f16 %0, wh, vl, %0;\n fma.rn.f32.f16 %1, wh, vh, %1;\n}\n" : "+f"(x), "+f"(y) : "r"(w), "r"(v));
  else
    asm("{\n .reg .b16 wl, wh, vl, vh;\n mov.b32 {wl, wh}, %2;\n mov.b32 {vl, vh}, %3;\n"
        " fma.rn.f32.f16 %0, wl, vl, %0;\n fma.rn.f32.f16 %1, wl, vh, %1;\n}\n" : "+f"(x), "+f"(y) : "r"(w), "r"(v));
}

// bf16 window of (b, hkv): lane = 4 channels, D/4 lanes a token (two tokens side
// by side at D = 64), rows requested two steps of eight ahead of their sums. The
// scores of eight tokens are summed over the lanes together, half of them
// changing lanes at each of the first three exchanges.
template <int D>
__device__ void own_window(const SharedParams& p, int64_t head, int n_win, const uint16_t* qp, float* rec, int lane) {
  constexpr int LN = D <= 64 ? 16 : 32, SIDES = 32 / LN, U = 8;
  const int side = lane / LN, c4 = lane % LN;              // channels 4 c4 ..
  const bool act = c4 * 4 < D;
  const uint2 q = act ? *reinterpret_cast<const uint2*>(qp + 4 * c4) : make_uint2(0u, 0u);
  const uint16_t* wk = p.win_k + head * p.W * D + 4 * c4;
  const uint16_t* wv = p.win_v + head * p.W * D + 4 * c4;
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  uint2 kr[2][U], vr[2][U];
  auto request = [&](int n0, uint2 (&k)[U], uint2 (&v)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int n = n0 + u * SIDES + side;
      const bool ok = act && n < n_win;
      k[u] = ok ? __ldg(reinterpret_cast<const uint2*>(wk + static_cast<int64_t>(n) * D)) : make_uint2(0u, 0u);
      v[u] = ok ? __ldg(reinterpret_cast<const uint2*>(wv + static_cast<int64_t>(n) * D)) : make_uint2(0u, 0u);
    }
  };
  auto step = [&](int n0, uint2 (&kr)[U], uint2 (&vr)[U]) {
    float x[U];
    uint2 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      x[u] = 0.f;
      dot_bf16(x[u], q.x, kr[u].x);
      dot_bf16(x[u], q.y, kr[u].y);
      v[u] = vr[u];
    }
    request(n0 + 2 * U * SIDES, kr, vr);                   // (past the window: nothing)
#pragma unroll
    for (int h = U / 2, off = LN / 2; h >= 1; h >>= 1, off >>= 1) {
      const bool up = (lane & off) != 0;
#pragma unroll
      for (int i = 0; i < h; ++i) {
        const float give = up ? x[i] : x[i + h], keep = up ? x[i + h] : x[i];
        x[i] = keep + __shfl_xor_sync(0xffffffffu, give, off);
      }
    }
#pragma unroll
    for (int off = LN / 16; off >= 1; off >>= 1) x[0] += __shfl_xor_sync(0xffffffffu, x[0], off);
    // this lane's token: bits LN/2, LN/4, LN/8 of the lane are its number's
    const int mine = ((lane & (LN / 2)) ? 4 : 0) | ((lane & (LN / 4)) ? 2 : 0) | ((lane & (LN / 8)) ? 1 : 0);
    const float xm = n0 + mine * SIDES + side < n_win ? x[0] * p.scale_log2 : -INFINITY;
    const float mx = redux_fmax(xm);
    if (mx > m) {                                          // warp-uniform
      const float f = m == -INFINITY ? 0.f : fast_exp2(m - mx);
      l *= f;
#pragma unroll
      for (int c = 0; c < 4; ++c) o[c] *= f;
      m = mx;
    }
    const float w = fast_exp2(xm - (m == -INFINITY ? 0.f : m));
    if ((lane & (LN / 8 - 1)) == 0) l += w;                // one lane counts a token
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float wu = __shfl_sync(0xffffffffu, w, side * LN + ((u & 4) ? LN / 2 : 0) + ((u & 2) ? LN / 4 : 0) + ((u & 1) ? LN / 8 : 0));
      const float2 a = bf16x2_to_float2(v[u].x), b = bf16x2_to_float2(v[u].y);
      o[0] = fmaf(wu, a.x, o[0]);
      o[1] = fmaf(wu, a.y, o[1]);
      o[2] = fmaf(wu, b.x, o[2]);
      o[3] = fmaf(wu, b.y, o[3]);
    }
  };
  request(0, kr[0], vr[0]);
  request(U * SIDES, kr[1], vr[1]);
#pragma unroll 1
  for (int n0 = 0; n0 < n_win; n0 += 2 * U * SIDES) {
    step(n0, kr[0], vr[0]);
    if (n0 + U * SIDES < n_win) step(n0 + U * SIDES, kr[1], vr[1]);
  }
  l = warp_sum(l);
  if constexpr (SIDES == 2) {
#pragma unroll
    for (int c = 0; c < 4; ++c) o[c] += __shfl_xor_sync(0xffffffffu, o[c], 16);
  }
  if (act && side == 0) *reinterpret_cast<float4*>(rec + 4 + 4 * c4) = make_float4(o[0], o[1], o[2], o[3]);
  if (lane == 0) {
    rec[0] = l == l ? m : NAN;
    rec[1] = l;
  }
}

// Quantised tokens [t0, t1) of sequence b, a block of LB slots at a time.
// Scores: lane = slot, byte s of its rotated key row is group (slot + s) mod J,
// its codeword and the query's channels of that group come from shared memory
// without bank conflicts. Values: lane = (side, group j), token by token.
// Weights are 2^(x - m) with m 14 below the running maximum, so that their fp16
// copies keep full precision down to 2^-28 of it.
template <int J, int C>
__device__ void own_chunk(const SharedParams& p, const uint8_t* pool_h, int b, int t0, int t1, float scale,
                          float unscale, unsigned char* scratch, float* rec, int lane) {
  using T = Shape<J, C>;
  constexpr int LB = T::LB, NW = T::NW;
  const int side = lane / J, j = lane % J;
  const bool act = side < T::TPS;
  const uint32_t sa = u32s(scratch);
  float m = -INFINITY, l = 0.f, o[C];
#pragma unroll
  for (int c = 0; c < C; ++c) o[c] = 0.f;
  const int32_t* bt = p.block_table + static_cast<int64_t>(b) * p.max_pages_per_seq;
  const int b0 = t0 / LB, b1 = (t1 + LB - 1) / LB;
  uint32_t kw[NW], vw[NW];
  auto entry_of = [&](int blk) { return blk < b1 ? __ldg(bt + (blk >> p.lbpp)) : -1; };
  bool ok = false;
  auto request = [&](int blk, int entry) {                 // index rows of a block
    ok = blk < b1 && entry >= 0 && entry < p.n_pages;
    if (blk < b1 && !ok && lane == 0 && p.status != nullptr) atomicOr(p.status, LOOPVQ_DECODE_STATUS_BAD_PAGE);
#pragma unroll
    for (int w = 0; w < NW; ++w) kw[w] = vw[w] = 0u;
    if (!ok || lane >= LB) return;
    const uint8_t* r = pool_h + static_cast<int64_t>(entry) * p.page_bytes + (blk & ((1 << p.lbpp) - 1)) * (LB * J) + lane * T::GR;
#pragma unroll
    for (int w = 0; w < NW; w += T::GR / 4) {
      const uint8_t* a = r + w * 4 / T::GR * (LB * T::GR);
      if constexpr (T::GR == 16) {
        const uint4 k4 = __ldcs(reinterpret_cast<const uint4*>(a));
        const uint4 v4 = __ldcs(reinterpret_cast<const uint4*>(a + p.plane_bytes));
        kw[w] = k4.x; kw[w + 1] = k4.y; kw[w + 2] = k4.z; kw[w + 3] = k4.w;
        vw[w] = v4.x; vw[w + 1] = v4.y; vw[w + 2] = v4.z; vw[w + 3] = v4.w;
      } else {
#pragma unroll
        for (int i = 0; i < T::GR / 4; ++i) {
          kw[w + i] = __ldcs(reinterpret_cast<const uint32_t*>(a) + i);
          vw[w + i] = __ldcs(reinterpret_cast<const uint32_t*>(a + p.plane_bytes) + i);
        }
      }
    }
  };
  int e_next = entry_of(b0);
  request(b0, e_next);
  e_next = entry_of(b0 + 1);
  // the query's channels of group (lane + s) mod J, for every byte s of a row: the
  // same for all blocks, so held in registers
  Word<T::ENTRY> q[J];
#pragma unroll
  for (int i = 0; i < J; ++i) q[i] = lds<T::ENTRY, 0>(sa + kOwnQ + (lane + i) * T::ENTRY);
#pragma unroll 1
  for (int blk = b0; blk < b1; ++blk) {
    // the value rows of this block, each twice
    __syncwarp();
    {
      const uint32_t row = sa + kOwnRows + lane * kOwnPitch;
      if constexpr (J == 32 || J == 16) {
#pragma unroll
        for (int rep = 0; rep < 2; ++rep)
#pragma unroll
          for (int w = 0; w < NW; w += 4) {
            Word<16> t;
            t.w[0] = vw[w]; t.w[1] = vw[w + 1]; t.w[2] = vw[w + 2]; t.w[3] = vw[w + 3];
            sts<16, 0>(row + rep * J + w * 4, t);
          }
      } else {
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(row + w * 4), "r"(vw[w]) : "memory");
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(row + J + w * 4), "r"(vw[w]) : "memory");
        }
      }
    }
    const int tok = blk * LB + lane;
    const bool valid = ok && lane < LB && tok >= t0 && tok < t1;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      Word<T::ENTRY> e[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {                        // codeword row (byte 1) | entry (byte 0)
        const uint32_t at = J == 32 ? static_cast<uint32_t>(lane + 4 * w + i) * T::ENTRY      // byte 0 wraps by itself
                                    : static_cast<uint32_t>((lane + 4 * w + i) % J) * T::ENTRY;
        e[i] = lds<T::ENTRY, kShBase + kKtabOff>(__byte_perm(kw[w], at, 0x7704u | (static_cast<uint32_t>(i) << 4)));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < C / 2; ++c) dot_f16(acc[i], q[4 * w + i].w[c], e[i].w[c]);
    }
    request(blk + 1, e_next);                              // lands under this block's values
    e_next = entry_of(blk + 2);
    const float x = valid ? ((acc[0] + acc[1]) + (acc[2] + acc[3])) * scale : -INFINITY;
    const float mx = redux_fmax(x) - kRaise;
    if (mx > m) {                                          // warp-uniform
      const float f = m == -INFINITY ? 0.f : fast_exp2(m - mx);
      l *= f;
#pragma unroll
      for (int c = 0; c < C; ++c) o[c] *= f;
      m = mx;
    }
    const float w0 = fast_exp2(x - (m == -INFINITY ? 0.f : m));
    l += w0;
    const __half wh = __float2half_rn(w0);
    asm volatile("st.shared.b16 [%0], %1;" ::"r"(sa + kOwnP + lane * 2), "h"(*reinterpret_cast<const uint16_t*>(&wh)) : "memory");
    __syncwarp();
    if (act) {
      const uint32_t row = sa + kOwnRows + side * J * kOwnPitch + j;
      const uint32_t wa = sa + kOwnP + side * J * 2;
#pragma unroll
      for (int k = 0; k < J; k += 4) {
        const Word<8> w4 = lds<8, 0>(wa + k * 2);
        uint32_t iv[4];
        Word<T::ENTRY> e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          asm volatile("ld.shared.u8 %0, [%1];" : "=r"(iv[i]) : "r"(row + (k + i) * kOwnPitch + J - (k + i)));
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = lds<T::ENTRY, kShBase + kVtabOff>(iv[i] * 256u + j * T::ENTRY);
#pragma unroll
        for (int c = 0; c < C / 2; ++c) {
          axpy_f16<0>(o[2 * c], o[2 * c + 1], w4.w[0], e[0].w[c]);
          axpy_f16<1>(o[2 * c], o[2 * c + 1], w4.w[0], e[1].w[c]);
          axpy_f16<0>(o[2 * c], o[2 * c + 1], w4.w[1], e[2].w[c]);
          axpy_f16<1>(o[2 * c], o[2 * c + 1], w4.w[1], e[3].w[c]);
        }
      }
    }
  }
  l = warp_sum(l);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    float t = o[c];
#pragma unroll
    for (int k = 1; k < T::TPS; ++k) t += __shfl_sync(0xffffffffu, o[c], (lane + k * J) & 31);
    o[c] = t * unscale;
  }
  if (lane < J) {
#pragma unroll
    for (int c = 0; c < C; c += 4)
      *reinterpret_cast<float4*>(rec + 4 + lane * C + c) = make_float4(o[c], o[c + 1], o[c + 2], o[c + 3]);
  }
  if (lane == 0) {
    rec[0] = l == l ? m : NAN;
    rec[1] = l;
  }
}

// Runs beside the shared grid, on the SMs that it leaves free: the shared blocks
// start this grid once the tables are written. Without a group's worth of rows
// there is no product to make; the bound is shared memory again, 6 accesses of 128
// bytes a token (two for the keys' lookups, two for the values', two for indices
// and weights): alone on 140 SMs with 1.5 M (sequence, head, token) triples and
// 4096 windows 77.7 us, l1tex at 75%, 62% of the issue slots.
template <int J, int C>
__global__ void __launch_bounds__(kOwnWarps * 32, 1) shared_own_kernel(const SharedParams p) {
  using T = Shape<J, C>;
  constexpr int D = T::D;
  extern __shared__ __align__(1024) unsigned char sm[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t bar = u32s(sm + kOwnBarOff);
  if (u32s(sm) != kShBase) {                               // the host checks this before launching
    if (tid == 0 && p.status != nullptr) atomicOr(p.status, LOOPVQ_DECODE_STATUS_SHARED_BASE);
    return;
  }
  if (tid == 0) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(2u) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  if (p.shared_blocks == 0) asm volatile("griddepcontrol.wait;" ::: "memory");   // this grid follows the tables' own
  float* fk = reinterpret_cast<float*>(sm + kOwnFkOff);
  unsigned char* scratch = sm + kOwnScratch + warp * kOwnBytes;
  uint32_t* qs = reinterpret_cast<uint32_t*>(scratch + kOwnQ);
  // tasks (head, sequence, query head of it, window or chunk), heads outermost; the
  // block takes its share of the list, one or a few heads
  const int per_head = p.B * p.ratio * p.NC;               // (times Hkv below 2^31: checked on the host)
  const int t_lo = static_cast<int>(static_cast<int64_t>(per_head) * p.Hkv * blockIdx.x / gridDim.x);
  const int t_hi = static_cast<int>(static_cast<int64_t>(per_head) * p.Hkv * (blockIdx.x + 1) / gridDim.x);
  int* next = reinterpret_cast<int*>(sm + kOwnBarOff + 8);
  bool failed = false;
  int phase = 0;
  for (int th = t_lo; th < t_hi; ++phase) {                // block-uniform
    const int hkv = th / per_head;
    const int t_end = min(t_hi, (hkv + 1) * per_head);
    const int* exk = p.exps + hkv * 64;
    __syncthreads();                                       // the head before is done with tables and scales
    if (!failed) {
      if (tid < 2) request_table(p, sm, hkv, tid, bar);
      if (tid < J) fk[tid] = pow2(-__ldcg(exk + tid));
      failed = __syncthreads_or(!mbar_wait(bar, phase & 1, kShSpin));
      if (failed && tid == 0) {                            // no copy may outlive the block
        const bool drained = mbar_wait(bar, phase & 1, kShDrainSpin);
        if (p.status != nullptr)
          atomicOr(p.status, drained ? LOOPVQ_DECODE_STATUS_TIMEOUT
                                     : (LOOPVQ_DECODE_STATUS_TIMEOUT | LOOPVQ_DECODE_STATUS_UNDRAINED));
      }
    }
    const float unv = lane < J ? pow2(-__ldcg(exk + 32 + lane)) : 0.f;   // of this lane's record channels
    const uint8_t* pool_h = p.pool_lg + hkv * p.pool_stride_head;
    if (tid == 0) *next = th;
    __syncthreads();
    for (;;) {                                             // a warp takes the next task when it is done with one
      int ti = 0;
      if (lane == 0) ti = atomicAdd(next, 1);
      ti = __shfl_sync(0xffffffffu, ti, 0);
      if (ti >= t_end) break;
      const int t = ti - hkv * per_head;
      const int y = t / p.NC, ck = t - y * p.NC - 1;       // -1: the window
      const int b = y / p.ratio, r = y - b * p.ratio;
      const int64_t pair = static_cast<int64_t>(b) * p.Hq + hkv * p.ratio + r;
      float* rec = p.orec + (pair * p.NC + ck + 1) * T::RS;
      if (failed) {
        if (lane == 0) {
          rec[0] = NAN;
          rec[1] = 1.f;
        }
        continue;
      }
      if (ck < 0) {
        own_window<D>(p, static_cast<int64_t>(b) * p.Hkv + hkv, max(0, min(__ldg(p.seq_lens + b), p.W)), p.q + pair * D, rec, lane);
        continue;
      }
      const int2 seq = __ldcg(p.seqs + b);                  // its shared tokens, its own
      const int c0 = ck * p.CH;
      if (c0 >= seq.y) continue;                           // the merge does not read it
      const int t0 = seq.x + c0, t1 = t0 + min(seq.y - c0, p.CH);
      // the query in fp16 against the scales of the key groups: word i holds
      // channels 2i, 2i + 1 (of D, then around again)
      static_assert((31 + J) * C * 2 <= kOwnP - kOwnQ, "query entries 0 .. 30 + J fit");
      const uint32_t* qw = reinterpret_cast<const uint32_t*>(p.q + pair * D);
      constexpr int QW = (31 + J) * C / 2, PER = (QW + 31) / 32;
      float2 f[PER];
      float top = 0.f;
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        const int i = (lane + 32 * k) % (D / 2);
        f[k] = bf16x2_to_float2(__ldg(qw + i));
        const float g = fk[2 * i / C];
        f[k].x *= g;
        f[k].y *= g;
        top = fmaxf(top, fmaxf(finite_abs(f[k].x), finite_abs(f[k].y)));
      }
      const int kq = scale_exp(redux_fmax(top));
      const float fq = pow2(kq);
      __syncwarp();
#pragma unroll
      for (int k = 0; k < PER; ++k)
        if (lane + 32 * k < QW) qs[lane + 32 * k] = half2_bits(f[k].x * fq, f[k].y * fq);
      __syncwarp();
      own_chunk<J, C>(p, pool_h, b, t0, t1, ldexpf(p.scale_log2, -kq), unv, scratch, rec, lane);
    }
    th = t_end;
  }
  // the merge waits for this grid, which ends after the shared one
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// One warp per (sequence, query head): joins the records that its blocks wrote,
// four requested at a time. 128 pairs with 10 records each take 1 us past the
// kernel before, 4096 pairs 4 us.
template <int D, int N>
__global__ void __launch_bounds__(128) shared_merge_kernel(const SharedParams p) {
  constexpr int RS = 4 + D, NCH = (D + 31) / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");       // every record is written
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t pair = static_cast<int64_t>(blockIdx.x) * 4 + warp;
  if (pair >= static_cast<int64_t>(p.B) * p.Hq) return;
  const int b = static_cast<int>(pair / p.Hq);
  const int2 seq = __ldcg(p.seqs + b);
  const int2 span = seq.x > 0 ? __ldcg(p.spans + pair) : make_int2(0, 0);
  const int ns = span.y, nc = 1 + (seq.y + p.CH - 1) / p.CH;   // the window's record first
  float m = -INFINITY, l = 0.f, o[NCH];
#pragma unroll
  for (int c = 0; c < NCH; ++c) o[c] = 0.f;
  for (int r0 = 0; r0 < ns + nc; r0 += 4) {
    float mr[4], lr[4], v[4][NCH];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = r0 + k;
      mr[k] = -INFINITY;
      lr[k] = 0.f;
      const float* rec = r < ns ? p.srec + (span.x + static_cast<int64_t>(r) * N) * RS : p.orec + (pair * p.NC + r - ns) * RS;
      const bool ok = r < ns + nc;
      if (ok) {
        mr[k] = __ldcg(rec) + (r == ns ? 0.f : static_cast<float>(kRecExp));   // (ns: the window)
        lr[k] = __ldcg(rec + 1) * (r == ns ? 1.f : 1.f / (1 << kRecExp));
      }
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const int ch = c * 32 + lane;
        v[k][c] = ok && ch < D ? __ldcg(rec + 4 + ch) : 0.f;
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (mr[k] == -INFINITY) continue;                    // an empty record
      const float mn = fmaxf(m, mr[k]);
      const float f0 = m == -INFINITY ? 0.f : fast_exp2(m - mn), f1 = fast_exp2(mr[k] - mn);
      l = fmaf(l, f0, lr[k] * f1);
#pragma unroll
      for (int c = 0; c < NCH; ++c) o[c] = fmaf(o[c], f0, v[k][c] * f1);
      m = mn;
    }
  }
  const float inv = (l > 0.f) ? 1.f / l : (l == 0.f ? 0.f : l);   // NaN stays NaN
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int ch = c * 32 + lane;
    if (ch < D) static_cast<__nv_bfloat16*>(p.out)[pair * D + ch] = __float2bfloat16_rn(o[c] * inv);
  }
  if (lane == 0 && p.lse != nullptr) p.lse[pair] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// How a call is cut up; a function of the sizes alone, so that the workspace
// can be sized without a device.
struct SharedPlan {
  int N, NC, CH, shared_blocks, own_blocks;
};
constexpr int kPlanSms = 148;             // blocks that run at once (one per SM of a B200; fewer SMs take waves)
constexpr int kOwnChunk = 256;            // own tokens of a task at least, and chunks of a pair at most
constexpr int kMaxChunks = 64;

// Query rows of a block: the width whose row tiles cost least by the measured
// times of a tile (SM cycles), and the row tiles of a kv-head. Of several groups the
// host knows the largest and the sum: half a row tile of each is taken as empty.
// (61 sequences in 7 uneven groups, 2 query heads a head: 65 us with 32 rows, 69 with
// the 64 that the largest group fills.)
struct RowTiles {
  int N;
  double units, t_tile;
};
RowTiles row_tiles(const Geometry& g, int batch, int n_groups, int max_group) {
  const int ratio = g.Hq / g.Hkv;
  const int64_t most = static_cast<int64_t>(max_group) * ratio;
  const int64_t all = std::min<int64_t>(batch, static_cast<int64_t>(n_groups) * max_group) * ratio;
  RowTiles q{};
  for (int n = 16; n <= kMaxRows; n *= 2) {
    const double cap = static_cast<double>(n_groups) * ((most + n - 1) / n);
    const double u = n_groups > 1 ? std::min(cap, std::max<double>(n_groups, 0.5 * n_groups + static_cast<double>(all) / n)) : cap;
    const double t = n == 16 ? 2200 : n == 32 ? 2500 : 3400;
    if (q.N == 0 || u * t < q.units * q.t_tile) q = RowTiles{n, u, t};
  }
  return q;
}

// Own tokens of a task, and tasks of a pair past its window's.
struct Chunks {
  int CH, n;
};
Chunks own_chunks(const Geometry& g, int batch, int max_own) {
  Chunks q;
  q.CH = static_cast<int64_t>(batch) * g.Hq >= 512 ? 2 * kOwnChunk : kOwnChunk;
  auto chunks = [&] { return max_own / q.CH + (max_own % q.CH != 0 ? 1 : 0); };
  while (chunks() > kMaxChunks) q.CH *= 2;
  q.n = chunks();
  return q;
}

SharedPlan make_plan(const Geometry& g, int batch, int n_groups, int max_group, int max_shared, int max_own) {
  SharedPlan q{};
  const RowTiles r = row_tiles(g, batch, n_groups, max_group);
  const double units = max_shared > 0 ? r.units * g.Hkv : 0, t_tile = r.t_tile;
  const Chunks own = own_chunks(g, batch, max_own);
  q.N = r.N;
  q.CH = own.CH;
  q.NC = 1 + own.n;                                        // the window, and the chunks
  // Both grids together fill the machine once. The own grid gets the number of
  // blocks with which the later of the two ends first, by measured times (SM
  // cycles): a tile; a block's 16 warps' way through a task each, which grows with
  // its tokens; the tables of a head and the warps that run out of its tasks first,
  // more of them where blocks start and end inside heads. (Own tokens, and the
  // shared ones of several groups, as if spread over the upper half of their range.)
  const int tiles = max_shared / (4 * g.LB) + 1;
  const int64_t tasks = static_cast<int64_t>(batch) * g.Hq * q.NC;
  const double t_task = 1500 + 125 * (g.W + 0.75 * max_own * 32 / g.LB) / q.NC;
  const int64_t fit_b = (tasks + 15) / 16 > g.Hkv ? (tasks + 15) / 16 : g.Hkv;
  const int most_b = static_cast<int>(fit_b < kPlanSms ? fit_b : kPlanSms);
  q.own_blocks = most_b;
  if (units > 0) {
    const int last = most_b == kPlanSms ? kPlanSms - 1 : most_b;
    const double work_a = units * ((n_groups > 1 ? 0.75 : 1.0) * tiles + 5) * t_tile;
    double best = 1e300;
    for (int nb = 1; nb <= last; nb += nb < g.Hkv ? 1 : g.Hkv) {
      const double t_a = 8000 + work_a / (kPlanSms - nb);
      const int div = std::gcd(nb, g.Hkv), starts = nb / div;     // a block starts at multiples of 1 / starts heads
      const int heads = (g.Hkv / div + 2 * (starts - 1)) / starts;   // and meets this many at most
      const double t_b = heads * (7000 + (starts > 1 && heads > 1 ? 0.5 : 0.2) * t_task) +
                         std::max(static_cast<double>(tasks) / (16 * nb), static_cast<double>(heads)) * t_task;
      const double t = t_a > t_b ? t_a : t_b;
      if (t < best) {
        best = t;
        q.own_blocks = nb;
      }
    }
  }
  if (units > 0) {                                         // three tiles a block at least
    const double most_a = units * (tiles + 5) / 3;
    const int na = kPlanSms - q.own_blocks;
    q.shared_blocks = most_a < na ? static_cast<int>(most_a) : na;
  }
  return q;
}

// Gives `kernel` its dynamic shared memory on this device (once), after
// checking that the allocation starts where the kernels' addresses need it.
template <typename K>
loopvq_status configure(K kernel, int smem, std::atomic<uint64_t>& configured) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return LOOPVQ_ERR_CUDA;
  const uint64_t bit = (dev >= 0 && dev < 64) ? (1ull << dev) : 0ull;
  if (bit != 0 && (configured.load(std::memory_order_relaxed) & bit)) return LOOPVQ_OK;
  int reserved = -1;
  if (cudaDeviceGetAttribute(&reserved, cudaDevAttrReservedSharedMemoryPerBlock, dev) != cudaSuccess)
    return LOOPVQ_ERR_CUDA;
  cudaFuncAttributes fa{};
  if (cudaFuncGetAttributes(&fa, kernel) != cudaSuccess) return LOOPVQ_ERR_CUDA;
  if (reserved != static_cast<int>(kShBase) || fa.sharedSizeBytes != 0) return LOOPVQ_ERR_UNSUPPORTED;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return LOOPVQ_ERR_CUDA;
  configured.fetch_or(bit, std::memory_order_relaxed);
  return LOOPVQ_OK;
}

// Launches `kernel` as a programmatic dependent of the kernel before it.
template <typename K>
loopvq_status launch_after(K kernel, int64_t blocks, int threads, int smem, cudaStream_t st, const SharedParams& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) return LOOPVQ_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? LOOPVQ_OK : LOOPVQ_ERR_CUDA;
}

template <int J, int C, int N>
loopvq_status launch_prefix(const SharedParams& p, cudaStream_t st) {
  static std::atomic<uint64_t> configured{0};
  const loopvq_status s = configure(shared_prefix_kernel<J, C, N>, kShSmem, configured);
  if (s != LOOPVQ_OK) return s;
  return launch_after(shared_prefix_kernel<J, C, N>, p.shared_blocks, kShThreads, kShSmem, st, p);
}

template <int J, int C>
loopvq_status launch_shared_jc(const SharedParams& p, int N, cudaStream_t st) {
  static std::atomic<uint64_t> configured{0};
  loopvq_status s = configure(shared_own_kernel<J, C>, kOwnSmem, configured);
  if (s != LOOPVQ_OK) return s;
  auto tables = N == 16 ? shared_table_kernel<J, C, 16> : N == 32 ? shared_table_kernel<J, C, 32> : shared_table_kernel<J, C, 64>;
  tables<<<dim3(J / 4, 2, p.Hkv + 1), kE, 0, st>>>(p.cb_k, p.cb_v, p.cb_stride_head, const_cast<unsigned char*>(p.tables),
                                                   const_cast<int*>(p.exps), p);
  if (cudaGetLastError() != cudaSuccess) return LOOPVQ_ERR_CUDA;
  if (p.shared_blocks > 0) {
    s = N == 16 ? launch_prefix<J, C, 16>(p, st) : N == 32 ? launch_prefix<J, C, 32>(p, st) : launch_prefix<J, C, 64>(p, st);
    if (s != LOOPVQ_OK) return s;
  }
  s = launch_after(shared_own_kernel<J, C>, p.own_blocks, kOwnWarps * 32, kOwnSmem, st, p);
  if (s != LOOPVQ_OK) return s;
  const int64_t pairs = static_cast<int64_t>(p.B) * p.Hq;
  switch (N) {
    case 16: return launch_after(shared_merge_kernel<J * C, 16>, (pairs + 3) / 4, 128, 0, st, p);
    case 32: return launch_after(shared_merge_kernel<J * C, 32>, (pairs + 3) / 4, 128, 0, st, p);
    default: return launch_after(shared_merge_kernel<J * C, 64>, (pairs + 3) / 4, 128, 0, st, p);
  }
}

// Byte offsets of the workspace's parts, with room for every way make_plan may
// cut up a call of at most these sizes: a workspace made for a larger batch or
// more own tokens serves a smaller call.
struct SharedLayout {
  size_t srec, orec, tables, exps, walks, spans, seqs, end;
};
SharedLayout make_layout(const Geometry& g, int batch, int max_own) {
  const size_t rec = (4 + static_cast<size_t>(g.d)) * sizeof(float), pairs = static_cast<size_t>(batch) * g.Hq;
  const int chunks = max_own / kOwnChunk + (max_own % kOwnChunk != 0 ? 1 : 0);
  SharedLayout w;
  w.srec = kStatusBytes;
  w.orec = w.srec + (pairs + static_cast<size_t>(kPlanSms) * kMaxRows) * rec;
  w.tables = w.orec + pairs * (1 + std::min(chunks, kMaxChunks)) * rec;
  w.exps = w.tables + static_cast<size_t>(g.Hkv) * 2 * kTabBytes;
  w.walks = w.exps + static_cast<size_t>(g.Hkv) * 64 * sizeof(int);
  w.spans = w.walks + static_cast<size_t>(kPlanSms) * sizeof(Walk);
  w.seqs = w.spans + pairs * sizeof(int2);
  w.end = w.seqs + static_cast<size_t>(batch) * sizeof(int2);
  return w;
}

// Cost of a (query head, quantised token) pair in 10^-6 us on the whole machine,
// measured over the calls of the rule below: in the decode kernels, and as an own
// token of these.
struct TokenCost {
  double decode, own;
};
bool token_cost(const Geometry& g, TokenCost* t) {
  switch (g.J * 100 + g.c) {
    case 3204: *t = TokenCost{14.0, 33.0}; return true;
    case 1604: *t = TokenCost{8.5, 21.0}; return true;
    case 1208: *t = TokenCost{13.0, 38.0}; return true;
    case 1608: *t = TokenCost{8.2, 21.0}; return true;
    case 2404: *t = TokenCost{19.0, 33.0}; return true;
    default: return false;
  }
}

// The calls that the kernels take: the shapes and types that they implement, where
// they are estimated to be faster than the decode kernels, which stream every
// sequence's own row of the page table. Both estimates (us) are fits to 1590 calls
// timed in both forms: 1 to 16 groups of 2 to 128 sequences and up to 120 without
// a group, 0 to 32000 shared and 1 to 32000 own tokens, 4 to 40 heads, the five
// shapes. They are off by a tenth on average and by less than a quarter in nine of
// ten calls; the form that they choose takes 1.01 times the better one's time on
// average, 1.4 times at worst (21 calls lose more than a fifth). What decides is own tokens, which cost more here, against the shared ones
// and the 0.09 us a (sequence, query head) pair that they cost there, these kernels /
// decode kernels, 16 heads of 128, at 1, 500, 2000, 8000 and 32000 own tokens: 4
// sequences over 500 shared ones 18/19, 24/19, 30/24, 43/28, 80/48; 8 over 16000
// 36/50, 36/50, 44/53, 67/61, 162/94; 32 over 2000 23/72, 36/78, 46/85, 131/125; 64
// over none 16/71, 32/114, 66/136, 187/214. 40 heads of 96 (c = 8), 4 sequences over
// 16000: 78/61. Near a tie (a twentieth) the call stays here. Fewer than four query
// rows a group or 64 (sequence, query head) pairs were not fitted.
bool shared_form_pays(const Geometry& g, int batch, int n_groups, int max_group, int max_shared, int max_own) {
  TokenCost cost;
  const double pairs = static_cast<double>(batch) * g.Hq;
  if (static_cast<int64_t>(batch) * (g.Hq / g.Hkv) < 4ll * n_groups || pairs < 64 || !token_cost(g, &cost)) return false;
  // (own tokens, and the shared ones of several groups, as if spread over the upper
  // half of their range)
  const double several = n_groups > 1 ? 0.75 : 1.0, shared = several * max_shared, own = 0.75 * max_own;
  const RowTiles r = row_tiles(g, batch, n_groups, max_group);
  const double tiles = max_shared > 0 ? r.units * g.Hkv * (several * (max_shared / (4 * g.LB) + 1) + kSetupTiles) : 0;
  const double task = std::min(max_own, own_chunks(g, batch, max_own).CH) * 32.0 / g.LB;   // a task's way
  const double here = 16 + 1.25 * tiles * r.t_tile / (kPlanSms * 1900.0) + pairs * own * cost.own * 1e-6 + 0.016 * task;
  const double decode = 13.5 + 0.09 * pairs + pairs * (shared + own) * cost.decode * 1e-6;
  return here <= 1.05 * decode;
}

}  // namespace

// The factor of a score is sm_scale log2(e) 2^-kq, kq >= -114 (the queries' power of
// two): with sm_scale outside 2^-20 .. 2^12 it could leave float32's range.
bool shared_attn_supported(const Geometry& g, int batch, int n_groups, int max_group, int max_shared, int max_own,
                           int out_dtype, float sm_scale) {
  if (!(sm_scale >= 0x1p-20f && sm_scale <= 0x1p12f)) return false;
  if (out_dtype != LOOPVQ_DTYPE_BF16 || n_groups == 0) return false;
  // (records, tasks and a sequence's tokens are counted in 32 bits)
  if (static_cast<int64_t>(batch) * g.Hq * (1 + own_chunks(g, batch, max_own).n) > INT_MAX / 2 ||
      static_cast<int64_t>(max_shared) + max_own > INT_MAX / 2)
    return false;
  return shared_form_pays(g, batch, n_groups, max_group, max_shared, max_own);
}

size_t shared_attn_workspace_bytes(const Geometry& g, int batch, int max_own) {
  return make_layout(g, batch, max_own).end;
}

loopvq_status launch_shared_attn(const SharedArgs& a) {
  const Geometry& g = *a.geo;
  const SharedPlan q = make_plan(g, a.batch, a.n_groups, a.max_group, a.max_shared, a.max_own);
  const int gamma = a.loop_step / g.g, tau = a.loop_step % g.g;
  SharedParams p{};
  p.q = static_cast<const uint16_t*>(a.q);
  p.pool_lg = a.pool + a.layer * g.pool_stride_layer + gamma * g.pool_stride_group;
  p.pool_stride_head = g.pool_stride_head;
  p.page_bytes = g.page_bytes;
  p.plane_bytes = g.plane_bytes;
  p.cb_k = a.codebooks + a.layer * g.cb_stride_layer + gamma * g.cb_stride_group + tau * g.cb_stride_loop;
  p.cb_v = p.cb_k + g.cb_stride_kv;
  p.cb_stride_head = g.cb_stride_head;
  p.block_table = a.block_table;
  p.seq_lens = a.seq_lens;
  p.group_starts = a.group_starts;
  p.shared_lens = a.shared_lens;
  p.win_k = static_cast<const uint16_t*>(a.win_k);
  p.win_v = static_cast<const uint16_t*>(a.win_v);
  char* ws = static_cast<char*>(a.workspace);
  p.status = reinterpret_cast<int*>(ws);
  const SharedLayout w = make_layout(g, a.batch, a.max_own);
  p.srec = reinterpret_cast<float*>(ws + w.srec);
  p.orec = reinterpret_cast<float*>(ws + w.orec);
  p.tables = reinterpret_cast<unsigned char*>(ws + w.tables);
  p.exps = reinterpret_cast<int*>(ws + w.exps);
  p.walks = reinterpret_cast<Walk*>(ws + w.walks);
  p.spans = reinterpret_cast<int2*>(ws + w.spans);
  p.seqs = reinterpret_cast<int2*>(ws + w.seqs);
  p.out = a.out;
  p.lse = a.lse;
  p.B = a.batch;
  p.n_groups = a.n_groups;
  p.Hq = g.Hq;
  p.Hkv = g.Hkv;
  p.ratio = g.Hq / g.Hkv;
  p.W = g.W;
  p.Pg = g.Pg;
  p.n_pages = g.n_pages;
  p.max_pages_per_seq = g.max_pages_per_seq;
  p.max_vq = static_cast<int>(std::min<int64_t>(static_cast<int64_t>(g.max_pages_per_seq) * g.Pg, INT_MAX));
  p.max_group = a.max_group;
  p.max_shared = a.max_shared;
  p.max_own = a.max_own;
  p.NC = q.NC;
  p.CH = q.CH;
  p.shared_blocks = q.shared_blocks;
  p.own_blocks = q.own_blocks;
  while ((1 << p.lbpp) < g.Pg / g.LB) ++p.lbpp;
  p.scale_log2 = a.sm_scale * kLog2e;
  cudaStream_t st = static_cast<cudaStream_t>(a.stream);
  switch (g.J * 100 + g.c) {
    case 3204: return launch_shared_jc<32, 4>(p, q.N, st);
    case 1604: return launch_shared_jc<16, 4>(p, q.N, st);
    case 1208: return launch_shared_jc<12, 8>(p, q.N, st);
    case 1608: return launch_shared_jc<16, 8>(p, q.N, st);
    case 2404: return launch_shared_jc<24, 4>(p, q.N, st);
    default: return LOOPVQ_ERR_UNSUPPORTED;
  }
}

}  // namespace loopvq
