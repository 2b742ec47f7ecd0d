// Decode attention for trees of drafted tokens over paged caches.
//
// Node i of sequence b, at position p_i = t_b + (its number of strict
// ancestors), attends to the compressed entries [0, N(p_i)) (or its selected
// ones), the window rows of positions >= p_i - W and its strict ancestors'
// drafted rows, in one softmax; the cached vector is key and value ([P2] Step
// 3); the output is rotated back by p_i ([P1] "Shared key and value").
//
// The (node, head) pairs of a sequence are flattened into query rows; a group
// of 128 of them shares every cache row it reads (for the selected form a
// group is one node).  A group's row list is cut into tiles of 128 rows: whole
// tiles of compressed rows that every node of the group sees first (dense
// form), then a packed tail of the other compressed rows, the window rows and
// the drafted rows; a selected list is packed throughout.
//
// A group is the work of a pair of CTAs (a cluster of two, cta_group::2
// products): CTA r has 64 of the query rows, loads 64 of a tile's rows as keys
// (all 512 channels) and all 128 rows of channels [256 r, 256 r + 256) as
// values, so that per product each SM feeds half of the B operand, and the 64
// queries (64 KB), the keys (64 KB), the values (64 KB) and the weights (16 KB) fit
// beside 256 + 2 x 64 TMEM columns.  One CTA with 64 queries instead
// (the same tile as key and value) measured 5.7 us a tile: the next tile's
// load waited for the value product, and 64-column products ran at half rate.
//   * S = Q . R^T: M = 128 queries, N = 128 rows, 32 K-steps; two buffers, so the
//     next tile's scores are formed while this one's softmax runs;
//   * 8 softmax warps a CTA, one query and 32 rows a thread (TMEM lanes 0-63: the
//     queries against rows 0-63, lanes 64-127: against rows 64-127): the weights
//     2^(x - m) against a running maximum m that is raised only when some score
//     passes it by 2^8 (one vote a tile), rounded to 16 bits, the products'
//     operand type (half a step of a weight, far below the rows' own rounding);
//     their sum, in fp32, is kept per thread and added up once per group;
//   * O += P . R: M = 128, N = 256, 8 K-steps, twice.
// Keys and values have their own barriers: a key buffer is refilled as soon as its
// scores are formed, a value buffer when its product is done.  Rows come by TMA
// (whole tiles of bf16 rows; both CTAs' copies complete on the first CTA's
// barrier) or through loader warps: 16-byte cp.async, or dequantisation to f16 as
// in the decode kernel.
//
// What bounds it: a buffer's round (product done, copy issued, rows here, product
// issued), since keys and values have one buffer each in two halves.  Measured
// per tile of 128 rows and pair of CTAs: 2.2 us for whole bf16 tiles (the products
// alone would take 1.0 us), 3.2 us for selected bf16 rows, 4.2 us for fp8 rows.
// 256 x 64 query rows x 8,320 bf16 rows x 4 sequences: 245 us called one after
// another (750 TFLOP/s), 215 us in a replayed graph of ten, where a call's set-up
// runs beside the one before.  18 us of latency for one short sequence: 4 us until
// the schedule and the tree are known, two tiles of 4 us each (not overlapped), 3 us
// to finish.
//
// Work split.  When the groups fill the pairs evenly a pair takes whole groups
// (c, c + P, ...); otherwise the tiles of all groups are laid end to end and cut
// into equal runs, a group cut by a run boundary leaving fp32 partial sums
// (O, m, l) that tree_combine merges with log-sum-exp weights.
//
// Rows that no node of the group sees are zero-filled, not loaded.  In the tail a
// row may be hidden from some queries, with weight 0 for them; if it holds an
// infinity or NaN (some score of it is then not finite) it is zeroed as a value
// before the second product, and only the queries that see it get its
// non-finite weight.
#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "internal.h"

namespace dsv4kv {

namespace {

constexpr int kRows = 128;      // rows per tile
constexpr int kKeys = 64;       // rows of a tile that a CTA holds as keys
constexpr int kQ = 64;          // query rows per CTA
constexpr int kGroup = 2 * kQ;  // query rows per pair
constexpr int kDim = 512, kHalf = 256;
constexpr int kQSlab = kQ * 128;        // 64 channels of the queries
constexpr int kQBytes = 8 * kQSlab;     // 64 KB
constexpr int kKSlab = kKeys * 128;     // 64 channels of the keys
constexpr int kKBytes = 8 * kKSlab;     // 64 KB
constexpr int kVSlab = 64 * 128;        // 64 channels of 64 of the values
constexpr int kVPart = 4 * kVSlab;      // 64 values, 32 KB
constexpr int kVBytes = 2 * kVPart;     // 64 KB
constexpr int kPBytes = 2 * kQ * 128;   // weights: 2 chunks of 64 rows
constexpr int kMaxBatch = 1024;
constexpr int kMaxNodes = 256;
constexpr int kRot = 256;       // output rotations kept per group (64 channels: of 8 nodes); others are formed per query
constexpr int kKey0 = 2, kKeyWarps = 4, kVal0 = kKey0 + kKeyWarps;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 0;    // O: 2 x 128 columns
constexpr uint32_t kColS = 256;  // S: 2 buffers of 64 columns
constexpr float kRaise = 8.0f;   // log2 units a score may pass the running maximum by
constexpr float kNoMax = -3.4028235e38f;  // a maximum that nothing has reached yet (finite: x - m of a hidden row is -inf)
// Tiles that cut groups may cost (partial sums, a second part per pair, the merge) before whole groups take longer.
// Whole groups of 10 bf16 tiles against runs of 7: 37 against 48 us; 12 fp8 tiles against 8: 77 against 62 us.  Over 208
// combinations of 8 to 230 groups of 2 to 40 tiles, in bf16 and fp8, 3 is 1.1 % off the faster choice on average.
constexpr int kSplitCost = 3;
// Row scales below this are taken as it: the weight of a stored row carries its scale and the denominator divides it
// out again, which needs a normal reciprocal.  Such a row's fp8 values are below 2^-91 (and rotary ones in bf16 beside
// them far outside of the range that the format's f16 staging keeps).
constexpr float kMinScale = 0x1p-100f;

constexpr int kValWarps = 4, kValRows = kRows / kValWarps;  // (a lane looks up one row)
constexpr int kSoft0 = kVal0 + kValWarps, kSoftWarps = 8;
constexpr int kSoftThreads = 32 * kSoftWarps, kThreads = 32 * (kSoft0 + kSoftWarps);
constexpr int kCols = 32;    // rows of a tile per softmax thread: two warps share a quarter of the TMEM lanes
constexpr int kChans = 128;  // output channels per softmax thread

// Warps: 0 schedule and queries, 1 products, 2-5 keys, 6-9 values, then 8 for the softmax and epilogue.  (16 softmax
// warps leave 72 registers a thread: 241 against 223 us for long dense contexts in bf16, and quantised rows want the
// registers for 8 loads of 16 bytes in flight; 2 value warps: 56 against 53 us for selected rows; two batches of 4 loads
// instead of one of 8: 67 against 62 us for selected fp8 rows.)
template <int FMT>
struct Cfg {
  static constexpr bool kQuant = FMT != DSV4KV_BF16;
  static constexpr bool kRowScale = FMT == DSV4KV_FP8_E4M3_ROW || FMT == DSV4KV_FP8_E4M3_ROW_ROPE_BF16;
  static constexpr uint32_t kIdescQK = kQuant ? idesc_f16(128, 128, 0, 0) : idesc_bf16(128, 128, 0, 0);
  static constexpr uint32_t kIdescPV = kQuant ? idesc_f16(128, 256, 0, 1) : idesc_bf16(128, 256, 0, 1);
};

// A cut group's run of tiles in one pair; slot 2c: the run does not start the group, 2c + 1: it starts it.
struct Rec {
  int valid, b, g, t0, t1, tiles, pad0, pad1;
};

struct Rows {  // one cache
  const int32_t* table;  // null: row i is row i
  int page, tstride;
  int64_t pages;
  const uint8_t* codes;
  const void* scales;
};

struct Params {
  Rows comp, win, draft;
  const int32_t *cu, *parent, *idx;
  const int64_t* t_seq;
  int batch, heads, nodes, max_nodes, window, stride, k;
  int64_t t_max;
  float score_scale;  // sm_scale * log2(e)
  int rope_dim, out_fp32;
  void* out;
  uint32_t* status;
  Rec* rec;       // [2 pairs]
  float4* ml;     // [2 pairs][128]: m, l, position, output row (int bits; -1: none)
  float* o_part;  // [2 pairs][128][512]
  RopeTable rope;
};

struct Seg {  // the part of a group that a pair works on
  int b, g, t0, t1, tiles;  // sequence, group within it, tiles [t0, t1) of `tiles`
  int t, w, m, c0;          // position, window rows, drafted nodes, first node
  int n, full;              // compressed rows listed (the most any node may see), whole tiles that every node sees
};

// Who sees a row: the positions [lo, hi]; a drafted row of the dense form: nobody by its key, but the node's descendants.
struct __align__(8) Key {
  int lo, hi;
};
constexpr int kNever = 0x7fffffff;

struct __align__(16) Ctl {
  // in the pair's first CTA: both CTAs' loads and weights arrive on these
  uint64_t q_ready, k_full[2], v_full[2], p_full[2];
  // in each CTA
  uint64_t q_full, meta, info[2], v_here[2];
  uint64_t s_full[2], k_empty[2], v_empty[2], o_done;
  uint32_t tmem_base;
  volatile int abort;
  int p_max;      // greatest position of the group's nodes
  int node_pos;   // (selected form) the node's position
  int b, g, t0;   // (equal runs) where this pair's run starts
  int whole, share, units;
  __align__(16) Key key[2][kRows];  // the rows of a tile that the loader warps brought
  uint32_t plain[2][4];           // all of a value warp's rows are there and every query sees them
  __align__(16) float scale[2][kRows];
  __align__(16) float lscale[2][kRows];  // log2 of the scale
  __align__(16) float iscale[2][kRows];  // 1 / the scale
  float m[kQ], alpha[kQ];
  float part[8][kQ];        // maxima / sums of a query's eight threads
  int row_pos[kQ];          // position of a query row's node
  uint8_t row_node[kQ];     // and its number within the CTA's
  uint32_t anc[kQ][kMaxNodes / 32];
  int16_t parent[kMaxNodes];
  float2 rot[kRot];         // rotations of the CTA's nodes' outputs, where they fit
  int gpre[kMaxBatch + 1];  // groups before sequence b
};

constexpr size_t kSmemBytes = 1024 + kQBytes + kKBytes + kVBytes + kPBytes + sizeof(Ctl);
static_assert(kSmemBytes <= 232448, "shared memory per CTA");
static_assert(kMaxBatch * sizeof(int) <= kPBytes, "tiles of every sequence in the weights' place");

__device__ __forceinline__ uint64_t globaltimer() {
  uint64_t t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}
constexpr uint64_t kWaitLimitNs = 1000000000ull;  // one second

// Bounded wait; false on timeout (raises the abort flag) or when another role gave up.
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort) {
  const uint64_t t0 = globaltimer();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    if (globaltimer() - t0 > kWaitLimitNs) {
      *abort = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return mbar_try_wait(bar, parity) || wait_slow(bar, parity, abort);
}
// The same for the end of a part of `tiles` tiles: 0.1 ms more for each, some 25 times what one takes.  (A role that is
// stuck in one of them raises the flag after a second.)
__device__ __noinline__ bool wait_part(uint64_t* bar, uint32_t parity, int tiles, volatile int* abort) {
  const uint64_t t0 = globaltimer(), limit = kWaitLimitNs + 100000ull * uint64_t(tiles);
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    if (globaltimer() - t0 > limit) {
      *abort = 1;
      return false;
    }
  }
}
// The products in flight after a wait gave up: bounded, abort or not.
__device__ __noinline__ void wait_drain(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer() - t0 > kWaitLimitNs) return;
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int lane) {
  bool ok = true;
  if (lane == 0) ok = wait_bar(bar, parity, abort);
  return __shfl_sync(kFull, ok, 0);
}
__device__ __forceinline__ bool soft_or(bool pred) {  // over the softmax threads
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred pi, po;\n\tsetp.ne.u32 pi, %1, 0;\n\tbarrier.cta.red.or.pred po, 1, %2, pi;\n\tselp.u32 "
      "%0, 1, 0, po;\n\t}"
      : "=r"(r)
      : "r"(uint32_t(pred)), "n"(kSoftThreads)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void soft_sync() {
  asm volatile("barrier.cta.sync 1, %0;" ::"n"(kSoftThreads) : "memory");
}

__device__ __forceinline__ float exp2_approx(float x) {  // max relative error ~2^-22, far below the weights' 16 bits
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __noinline__ void rotation(double theta_pi, int pos, float* cs, float* sn) {
  rope_rotation(theta_pi, -double(pos), cs, sn);
}

__device__ __forceinline__ int entries(int t, int window, int stride) {
  return t > window ? (t - window) / stride : 0;
}

// First node and number of nodes of sequence b, clamped into the call's.
__device__ __forceinline__ void seq_nodes(const Params& p, int b, int* c0, int* m, uint32_t* status) {
  const int a = p.cu[b], z = p.cu[b + 1];
  int lo = min(max(a, 0), p.nodes), hi = min(max(z, lo), p.nodes);
  hi = min(hi, lo + p.max_nodes);
  if (lo != a || hi != z) set_status(status, DSV4KV_DEV_BAD_LENGTH);
  *c0 = lo;
  *m = hi - lo;
}
__device__ __forceinline__ int seq_len(const Params& p, int b, uint32_t* status) {
  const int64_t t = p.t_seq[b];
  if (t >= 0 && t <= p.t_max) return int(t);
  set_status(status, DSV4KV_DEV_BAD_LENGTH);
  return t < 0 ? 0 : int(p.t_max);
}
__device__ __forceinline__ int groups_of(const Params& p, int m) {
  return p.idx ? m : (m * p.heads + kGroup - 1) / kGroup;  // (heads <= 128: one group a node)
}
// Tiles of a group whose sequence lists n compressed rows.
__device__ __forceinline__ int tiles_of(const Params& p, int n, int w, int m) {
  return ((p.idx ? min(n, p.k) : n) + w + m + kRows - 1) / kRows;
}

// Pool row of logical row i; -1 when its page is outside the pool or the table has no entry for it.
__device__ __forceinline__ int64_t map_row(const Rows& r, int b, int i) {
  if (!r.table) return i;
  const int pi = i / r.page;
  const int32_t pg = pi < r.tstride ? __ldg(r.table + size_t(b) * r.tstride + pi) : -1;
  return pg >= 0 && pg < r.pages ? int64_t(pg) * r.page + (i - pi * r.page) : -1;
}

// Pool rows of the two 64-row halves of whole tile T (pages hold whole halves); false: a bad page.
__device__ __forceinline__ bool tma_rows(const Params& p, int b, int T, int32_t (&row)[2]) {
  bool ok = true;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = kRows * T + 64 * h, pi = i / p.comp.page;
    const int32_t pg = pi < p.comp.tstride ? __ldg(p.comp.table + size_t(b) * p.comp.tstride + pi) : -1;
    ok = ok && pg >= 0 && pg < p.comp.pages;
    row[h] = pg * p.comp.page + (i - pi * p.comp.page);
  }
  return ok;
}

// Row r of tile T: its cache and pool row (null: there is none, or no query of the group sees it) and who sees it.
// Whole tiles (T < s.full) need nothing of the tree; for the others `met` waits for it (warp-uniform), after the index
// and table reads are on their way.  Pages are flagged only for rows that are needed.
template <class Met>
__device__ __forceinline__ const Rows* row_source(const Params& p, const Seg& s, const Ctl* ctl, int T, int r,
                                                  int64_t* row, Key* key, Met met) {
  const int u = kRows * T + r, j = u - s.n;
  const Rows* src = j < 0 ? &p.comp : j < s.w ? &p.win : j - s.w < s.m ? &p.draft : nullptr;
  int i = j < 0 ? u : j < s.w ? j : s.c0 + (j - s.w);
  if (j < 0 && p.idx) i = __ldg(p.idx + size_t(s.c0 + s.g) * p.k + u);
  *row = src && i >= 0 && (j >= 0 || i < entries(s.t + s.m - 1, p.window, p.stride)) ? map_row(*src, s.b, i) : -1;
  *key = Key{0, kNever};
  bool need = src && i >= 0;
  if (T >= s.full) {
    if (!met()) need = false;
    if (j < 0) {
      if (p.idx) {
        const int n = entries(ctl->node_pos, p.window, p.stride);
        if (u >= min(p.k, n)) need = false;
        if (need && i >= n) {
          set_status(p.status, DSV4KV_DEV_BAD_INDEX);
          need = false;
        }
      } else {
        key->lo = p.window + p.stride * (u + 1);  // N(p) > u
        if (key->lo > ctl->p_max) need = false;
      }
    } else if (j < s.w) {  // window row j holds the last position congruent to j
      key->hi = s.t - 1 - (s.t - 1 - j) % p.window + p.window;
      if (p.idx) {
        if (key->hi < ctl->node_pos) need = false;
        key->hi = kNever;
      }
    } else if (j - s.w < s.m) {
      if (!p.idx) *key = Key{kNever, 0};  // (see the ancestor bits)
      else if (!((ctl->anc[0][(j - s.w) >> 5] >> ((j - s.w) & 31)) & 1u)) need = false;
    }
  }
  if (need && *row < 0) set_status(p.status, DSV4KV_DEV_BAD_PAGE);
  if (need && *row >= 0) return src;
  key->lo = kNever;
  return nullptr;
}

// ---------------------------------------------------------------- loader warps
__device__ __forceinline__ uint32_t swz(int r, int ch) { return r * 128 + ((((ch & 63) >> 3) ^ (r & 7)) << 4); }
__device__ __forceinline__ uint8_t* key_cell(uint8_t* sK, int r, int ch) { return sK + (ch >> 6) * kKSlab + swz(r, ch); }
__device__ __forceinline__ uint8_t* val_cell(uint8_t* sV, int r, int ch) {
  return sV + (r >> 6) * kVPart + (ch >> 6) * kVSlab + swz(r & 63, ch);
}

__device__ __forceinline__ const uint8_t* shfl_ptr(const uint8_t* p, int src) {
  return reinterpret_cast<const uint8_t*>(__shfl_sync(kFull, reinterpret_cast<uint64_t>(p), src));
}

__host__ __device__ constexpr int row_bytes(int fmt) {
  return fmt == DSV4KV_BF16 ? 2 * kDim
         : fmt == DSV4KV_FP8_E4M3_ROW ? kDim
         : fmt == DSV4KV_FP4_E2M1_G16 ? kDim / 2
                                      : kDim + 64;
}

// Two bf16 values times `by` as f16, finite ones saturating; infinities become NaN, as NaN stays NaN (x - x is 0 or NaN).
__device__ __forceinline__ uint32_t staged(float lo, float hi, float by) {
  return f32x2_to_f16x2_sat(fmaf(lo, by, lo - lo), fmaf(hi, by, hi - hi));
}

// Dequantises channels [ch0, ch0 + 256) of kR <= 32 rows (row i is lane i's `my`) to f16, in units of 16 bytes of codes:
// 16 fp8 channels, 32 fp4 channels, or 8 bf16 rotary channels (stored as f16 of value / scale: the row's scale is in the
// weights; a scale of 0, which makes the fp8 channels zeros, is staged as 1: my_inv < 0).  A batch is 8 units a lane:
// fetch() issues its loads, put() converts it.
template <int FMT, int kR>
struct Dequant {
  static constexpr bool kRope = FMT == DSV4KV_FP8_E4M3_ROW_ROPE_BF16, kFp4 = FMT == DSV4KV_FP4_E2M1_G16;
  static constexpr int kN = 8;
  uint4 raw[kN];
  uint32_t sc[kFp4 ? kN : 1];

  // units of a row: code units, then (where the channels reach the rotary ones) rotary units
  static __device__ __forceinline__ int body(int ch0) {
    return kFp4 ? kHalf / 32 : kRope && ch0 + kHalf > kDim - 64 ? (kDim - 64 - ch0) / 16 : kHalf / 16;
  }
  static __device__ __forceinline__ int per_row(int ch0) {
    return kRope && ch0 + kHalf > kDim - 64 ? body(ch0) + 8 : body(ch0);
  }
  static __device__ __forceinline__ int batches(int ch0) { return (kR * per_row(ch0) + 32 * kN - 1) / (32 * kN); }

  __device__ __forceinline__ void fetch(const uint8_t* my, const uint8_t* mysc, int ch0, int batch, int lane) {
    const int bd = body(ch0), upr = per_row(ch0);
    // (first all rows' addresses: a shuffle's and then a load's wait for the queue they share would come 8 times over)
    const uint8_t* rows[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) rows[i] = shfl_ptr(my, min((32 * (kN * batch + i) + lane) / upr, kR - 1));
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int x = 32 * (kN * batch + i) + lane, r = x / upr, u = x - r * upr;
      const uint8_t* row = rows[i];
      const bool in = r < kR && row;
      raw[i] = in ? ld_stream_v4(row + (kFp4 ? ch0 / 2 + 16 * u : kRope && u >= bd ? kDim - 64 + 16 * (u - bd) : ch0 + 16 * u))
                  : make_uint4(0, 0, 0, 0);
      if constexpr (kFp4) {
        const uint8_t* srow = shfl_ptr(mysc, min(r, kR - 1));
        sc[i] = in ? *reinterpret_cast<const uint16_t*>(srow + ch0 / 16 + 2 * u) : 0u;
      }
    }
  }
  // cell(row, channel - ch0): where 8 channels go
  template <class Cell>
  __device__ __forceinline__ void put(float my_inv, int ch0, int batch, int lane, Cell cell) const {
    const int bd = body(ch0), upr = per_row(ch0);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int x = 32 * (kN * batch + i) + lane, r = x / upr, u = x - r * upr;
      uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
      float inv = 1.f;
      if constexpr (kRope) inv = __shfl_sync(kFull, my_inv, min(r, kR - 1));
      if (r >= kR) continue;
      if (kRope && inv < 0.f) {
        inv = -inv;
        if (u < bd) w[0] = w[1] = w[2] = w[3] = 0u;
      }
      if constexpr (kFp4) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t s1 = e < 2 ? sc[i] & 0xffu : sc[i] >> 8;
          const uint32_t s2 = e4m3x2_to_f16x2(s1 | (s1 << 8));
          uint32_t h[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) h[j] = hmul2(e2m1x2_to_f16x2((w[e] >> (8 * j)) & 0xffu), s2);
          *reinterpret_cast<uint4*>(cell(r, 32 * u + 8 * e)) = make_uint4(h[0], h[1], h[2], h[3]);
        }
      } else if (kRope && u >= bd) {
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = staged(bf16lo(w[e]), bf16hi(w[e]), inv);
        *reinterpret_cast<uint4*>(cell(r, kDim - 64 - ch0 + 8 * (u - bd))) = make_uint4(h[0], h[1], h[2], h[3]);
      } else {
        uint32_t h[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          h[2 * e] = e4m3x2_to_f16x2(w[e] & 0xffffu);
          h[2 * e + 1] = e4m3x2_to_f16x2(w[e] >> 16);
        }
        *reinterpret_cast<uint4*>(cell(r, 16 * u)) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(cell(r, 16 * u + 8)) = make_uint4(h[4], h[5], h[6], h[7]);
      }
    }
  }
};

// A tail tile in which some score is not finite: if row r's values are not finite the row is zeroed, so that its zero
// weights (queries that do not see it) add zeros.  A query that is not finite itself says nothing.
template <bool kF16>
__device__ __noinline__ void zero_bad_row(uint8_t* sV, int r) {
  const uint32_t e = kF16 ? 0x7c00u : 0x7f80u;
  bool bad = false;
#pragma unroll 1
  for (int ch = 0; ch < kHalf; ch += 8) {
    const uint4 v = *reinterpret_cast<const uint4*>(val_cell(sV, r, ch));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) bad |= (w[k] & e) == e || ((w[k] >> 16) & e) == e;
  }
  if (!bad) return;
#pragma unroll 1
  for (int ch = 0; ch < kHalf; ch += 8) *reinterpret_cast<uint4*>(val_cell(sV, r, ch)) = make_uint4(0, 0, 0, 0);
}

// ---------------------------------------------------------------- the kernel
template <int FMT>
__global__ void __launch_bounds__(kThreads, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_comp,
                const __grid_constant__ Params p) {
  using C = Cfg<FMT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);  // (an offset: the accesses stay shared-memory ones)
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + kQBytes;
  uint8_t* sV = sK + kKBytes;
  uint8_t* sP = sV + kVBytes;
  Ctl* ctl = reinterpret_cast<Ctl*>(sP + kPBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr bool kRotary = FMT == DSV4KV_FP8_E4M3_ROW_ROPE_BF16;
  const int P = gridDim.x / 2, pair = blockIdx.x / 2;
  const int rank = int(cluster_rank());
  volatile int* abort = &ctl->abort;
  pdl_trigger();

  if (tid == 0) {
    mbar_init(&ctl->q_ready, C::kQuant ? 2 * kSoftWarps : 1);
    mbar_init(&ctl->q_full, 1);
    mbar_init(&ctl->meta, kSoftWarps);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&ctl->k_full[x], 2 * kKeyWarps);
      mbar_init(&ctl->v_full[x], kValWarps);
      mbar_init(&ctl->p_full[x], kSoftWarps);
      mbar_init(&ctl->info[x], kValWarps);
      mbar_init(&ctl->v_here[x], kValWarps / 2);
      mbar_init(&ctl->s_full[x], 1);
      mbar_init(&ctl->k_empty[x], 1);
      mbar_init(&ctl->v_empty[x], 1);
    }
    mbar_init(&ctl->o_done, 1);
    ctl->abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  // the pair's barriers exist and both CTAs are there before anything of either reaches the other
  cluster_sync();
  if (warp == 1) tmem_alloc_pair(&ctl->tmem_base, kTmemCols);
  if (tid == 64) {
    prefetch_tmap(&tm_q);
    if (!C::kQuant) prefetch_tmap(&tm_comp);
  }
  tc_fence_before();
  pdl_wait();

  // ---- the batch: groups and tiles of every sequence (in the weights' place), then which part is this pair's
  int* tiles = reinterpret_cast<int*>(sP);
  for (int b = tid; b < p.batch; b += kThreads) {
    int c0, m;
    uint32_t* st = blockIdx.x == 0 ? p.status : nullptr;
    seq_nodes(p, b, &c0, &m, st);
    const int t = seq_len(p, b, st);
    ctl->gpre[b + 1] = groups_of(p, m);
    tiles[b] = m > 0 ? tiles_of(p, entries(t + m - 1, p.window, p.stride), min(t, p.window), m) : 0;
  }
  __syncthreads();
  if (warp == 0) {
    int g = 0, u = 0, most = 0;  // groups, units (tiles of all groups: < 2^31), most tiles of a group
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
      const int b = b0 + lane;
      const int n = b < p.batch ? ctl->gpre[b + 1] : 0, tl = b < p.batch ? tiles[b] : 0;
      int x = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x += y;
      }
      if (b < p.batch) ctl->gpre[b + 1] = g + x;
      g += __shfl_sync(kFull, x, 31);
      u += __reduce_add_sync(kFull, unsigned(n) * unsigned(tl));
      most = max(most, __reduce_max_sync(kFull, n > 0 ? tl : 0));
    }
    if (lane == 0) ctl->gpre[0] = 0;
    __syncwarp();
    // whole groups when that takes no longer than equal runs of tiles plus a merge
    const int share = max(1, (u + P - 1) / P), rounds = (g + P - 1) / P;
    const bool whole = (long long)rounds * most <= share + kSplitCost;
    if (lane == 0) {
      ctl->whole = whole;
      ctl->share = share;
      ctl->units = u;
    }
    const unsigned want = unsigned(share) * unsigned(pair);
    unsigned at = 0;
    for (int b0 = 0; b0 < p.batch && !whole; b0 += 32) {
      const int b = b0 + lane;
      const unsigned tl = b < p.batch ? tiles[b] : 0;
      const unsigned v = b < p.batch ? unsigned(ctl->gpre[b + 1] - ctl->gpre[b]) * tl : 0u;
      unsigned x = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x += y;
      }
      const unsigned ex = at + x - v;
      if (want >= ex && want - ex < v) {
        ctl->b = b;
        ctl->g = (want - ex) / tl;
        ctl->t0 = (want - ex) % tl;
      }
      at += __shfl_sync(kFull, x, 31);
    }
  }
  if (tid < 2 && rank == 0) p.rec[2 * pair + tid].valid = 0;
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  const bool whole = ctl->whole != 0;
  // Every warp walks the pair's parts by itself, so that the loads and scores of the next part run during this one's
  // epilogue.  (equal runs) `left` tiles from (b, g, t0) on; (whole groups) flattened group `g_next`.
  int left = int(max(0ll, min((long long)ctl->share, ctl->units - (long long)ctl->share * pair)));
  int g_next = pair;
  Seg s;
  s.b = ctl->b;
  s.g = ctl->g;
  s.t0 = s.t1 = ctl->t0;
  int cnt = 0, segs = -1;  // tiles and parts done so far: the barriers' phases
  auto next_part = [&]() -> bool {
    const int done = s.t1 - s.t0;  // (0 before the first part)
    if (whole) {
      if (g_next >= ctl->gpre[p.batch]) return false;
      s.b = find_seq(ctl->gpre, p.batch, g_next);
      s.g = g_next - ctl->gpre[s.b];
      s.t0 = 0;
      g_next += P;
    } else {
      left -= done;
      if (left <= 0) return false;
      if (segs >= 0) {
        s.t0 = 0;
        ++s.g;
        while (s.g >= ctl->gpre[s.b + 1] - ctl->gpre[s.b]) {
          ++s.b;
          s.g = 0;
        }
      }
    }
    cnt += done;
    ++segs;
    return true;
  };
  // (the two parts of a step: next_part() sets b, g, t0 and the phases; load_part() the rest)
  auto load_part = [&]() {
    seq_nodes(p, s.b, &s.c0, &s.m, nullptr);
    s.t = seq_len(p, s.b, nullptr);
    s.w = min(s.t, p.window);
    const int n = entries(s.t + s.m - 1, p.window, p.stride);
    s.tiles = tiles_of(p, n, s.w, s.m);
    s.t1 = whole ? s.tiles : min(s.tiles, s.t0 + left);
    s.n = p.idx ? min(p.k, n) : n;
    s.full = p.idx ? 0 : entries(s.t, p.window, p.stride) / kRows;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ queries
    bool ok = true;
    int last = 0;  // tiles of the part before
    while (ok && next_part()) {
      load_part();
      const int row = p.idx ? (s.c0 + s.g) * p.heads + rank * ((p.heads + 1) / 2)
                            : s.c0 * p.heads + kGroup * s.g + rank * kQ;
      if (segs > 0) {  // (its scores have read its queries)
        if (lane == 0) ok = wait_part(&ctl->o_done, (segs - 1) & 1, last, abort);
        ok = __shfl_sync(kFull, ok, 0);
      }
      last = s.t1 - s.t0;
      if (ok && lane == 0) {
        // on the first CTA's barrier, or, to be converted first, on this one's
        if (C::kQuant) mbar_arrive_expect_tx(&ctl->q_full, kQBytes);
        else if (rank == 0) mbar_arrive_expect_tx(&ctl->q_ready, 2 * kQBytes);
        tma_load_3d_pair(sQ, &tm_q, C::kQuant ? smem_u32(&ctl->q_full) : lead_addr(&ctl->q_ready), 0, row, 0);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ products (the first CTA issues them)
    if (rank == 0) {
      const uint32_t me = elect_lane();
      const uint64_t qd = smem_desc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t kd = smem_desc_sw128(smem_u32(sK), 16, 1024);
      const uint64_t pd = smem_desc_sw128(smem_u32(sP), 16, 1024);
      const uint64_t vd = smem_desc_sw128(smem_u32(sV), kVSlab, 1024);
      uint64_t idle = 0;
      auto stuck = [&]() {  // nothing was ready: bounded
        const uint64_t now = globaltimer();
        if (idle == 0) idle = now;
        if (now - idle > kWaitLimitNs) *abort = 1;
        return __any_sync(kFull, *abort != 0) != 0;
      };
      auto ready = [&](uint64_t* bar, uint32_t parity) { return __all_sync(kFull, mbar_test_wait(bar, parity)) != 0; };
      bool ok = true;
      while (ok && next_part()) {
        load_part();
        const int nt = s.t1 - s.t0;
        idle = 0;
        while (ok && !ready(&ctl->q_ready, segs & 1)) ok = !stuck();
        int qk = 0, pv = 0;  // half tiles: 256 channels of the scores, 64 values of the output
        idle = 0;
#pragma unroll 1
        while (ok && pv < 2 * nt) {
          const int tq = cnt + (qk >> 1), tp = cnt + (pv >> 1);
          if ((pv >> 1) < (qk >> 1) && ready(&ctl->p_full[pv & 1], tp & 1) && ready(&ctl->v_full[pv & 1], tp & 1)) {
            tc_fence_after();
            const uint64_t ph = pd + ((pv & 1) * (kQSlab >> 4)), vh = vd + ((pv & 1) * (kVPart >> 4));
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int kr = 0; kr < 4; ++kr)
                mma_f16_pair(me, tmem + kColO + 128 * n, ph + ((kr * 32) >> 4), vh + ((kr * 2048 + 2 * n * kVSlab) >> 4),
                             C::kIdescPV, (pv > 0 || kr > 0) ? 1u : 0u);
            mma_commit_pair(me, &ctl->v_empty[pv & 1]);
            ++pv;
            idle = 0;
          } else if (qk < 2 * nt && (qk >> 1) < (pv >> 1) + 2 && ready(&ctl->k_full[qk & 1], tq & 1)) {
            tc_fence_after();
            const uint32_t d = tmem + kColS + 64 * (tq & 1), on = qk & 1;
            const uint64_t qh = qd + (on * (4 * kQSlab >> 4)), kh = kd + (on * (4 * kKSlab >> 4));
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_f16_pair(me, d, qh + ((c * kQSlab + kk * 32) >> 4), kh + ((c * kKSlab + kk * 32) >> 4), C::kIdescQK,
                             (c | kk) ? 1u : on);
            if (on) mma_commit_pair(me, &ctl->s_full[tq & 1]);
            mma_commit_pair(me, &ctl->k_empty[on]);
            ++qk;
            idle = 0;
          } else {
            ok = !stuck();
          }
        }
        mma_commit_pair(me, &ctl->o_done);  // completes once every product issued so far has
        if (!ok) wait_drain(&ctl->o_done, segs & 1);
      }
    }
  } else if (warp >= kSoft0) {
    // ------------------------------------------------------------ softmax, epilogue
    // TMEM lane 64 h + j: query j against rows 64 h + .. (scores), channels 256 h + .. (output)
    const int wq = warp & 3, cg = (warp - kSoft0) >> 2, h = wq >> 1;
    const int j = 32 * (wq & 1) + lane;            // this thread's query
    const int r0 = 64 * h + kCols * cg;            // its first row of a tile
    const uint32_t lane_base = uint32_t(32 * wq) << 16;
    const int q = tid - 32 * kSoft0;  // (q < 64) the query that this thread keeps the statistics of
    bool dead = false;  // after a wait gave up: skips every access, still takes part in the group's barriers
    while (next_part()) {
      load_part();
      const int nt = s.t1 - s.t0;
      // ---- the group's nodes: [first, last], of them node0 .. node0 + n_nodes - 1 have query rows in this CTA
      int first, last, node0, n_nodes, row0, rows;
      const int f = kGroup * s.g + rank * kQ;  // first query row within the sequence
      if (p.idx) {
        const int hs = (p.heads + 1) / 2;  // the node's heads, half in each CTA
        first = last = node0 = s.g;
        n_nodes = 1;
        row0 = (s.c0 + s.g) * p.heads + rank * hs;
        rows = rank ? p.heads - hs : hs;
      } else {
        const int all = min(kGroup, s.m * p.heads - kGroup * s.g);
        first = kGroup * s.g / p.heads;
        last = (kGroup * s.g + all - 1) / p.heads;
        rows = min(kQ, max(0, all - rank * kQ));
        row0 = s.c0 * p.heads + f;
        node0 = f / p.heads;
        n_nodes = rows > 0 ? (f + rows - 1) / p.heads - node0 + 1 : 0;
      }
      for (int i = q; i < s.m; i += kSoftThreads) {
        int par = p.parent[s.c0 + i];
        if (par < -1 || par >= i) {
          set_status(p.status, DSV4KV_DEV_BAD_TREE);
          par = -1;
        }
        ctl->parent[i] = int16_t(par);
      }
      for (int i = q; i < kQ * (kMaxNodes / 32); i += kSoftThreads) (&ctl->anc[0][0])[i] = 0;
      if (q < kQ) {
        ctl->m[q] = kNoMax;
        ctl->row_node[q] = 0;
        ctl->row_pos[q] = -1;
      }
      if (q == kQ) ctl->p_max = 0;
      soft_sync();
      for (int i = first + q; i <= last; i += kSoftThreads) {
        int d = 0;
        const int gj = i - node0;
        const bool mine = gj >= 0 && gj < n_nodes;
        for (int x = ctl->parent[i]; x >= 0; x = ctl->parent[x]) {
          ++d;
          if (mine) ctl->anc[gj][x >> 5] |= 1u << (x & 31);
        }
        const int at = s.t + d;
        atomicMax(&ctl->p_max, at);
        if (p.idx) ctl->node_pos = at;
        if (mine) {  // its query rows in this CTA
          const int lo = p.idx ? 0 : max(0, i * p.heads - f), hi = p.idx ? rows : min(rows, (i + 1) * p.heads - f);
          for (int x = lo; x < hi; ++x) {
            ctl->row_pos[x] = at;
            ctl->row_node[x] = uint8_t(gj);
          }
        }
      }
      soft_sync();
      if (lane == 0) mbar_arrive(&ctl->meta);
      const bool live = j < rows;
      const int pos = ctl->row_pos[j];
      const uint32_t* anc = ctl->anc[ctl->row_node[j]];
      if (C::kQuant) {  // queries to f16, in place
        if (!dead) dead = !warp_wait(&ctl->q_full, segs & 1, abort, lane);
        if (!dead) {
#pragma unroll 1
          for (int i = q; i < kQBytes / 16; i += kSoftThreads) {
            uint4 v = reinterpret_cast<uint4*>(sQ)[i];
            uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = staged(bf16lo(w[e]), bf16hi(w[e]), 1.f);
            reinterpret_cast<uint4*>(sQ)[i] = v;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive_pair(lead_addr(&ctl->q_ready));
        }
      }
      // the rotations of the CTA's nodes, while the first tiles are on their way
      const bool final_out = s.t0 == 0 && s.t1 == s.tiles;
      const int pairs = p.rope_dim / 2;
      const bool table = n_nodes * pairs <= kRot;
      if (final_out && table)
        for (int x = q; x < n_nodes * pairs; x += kSoftThreads) {
          const int node = x / pairs, at = p.idx ? 0 : max(0, (node0 + node) * p.heads - f);  // its first query row here
          rotation(p.rope.theta_pi[x - node * pairs], ctl->row_pos[at], &ctl->rot[x].x, &ctl->rot[x].y);
        }
      float l = 0.f;
#pragma unroll 1
      for (int i = 0; i < nt; ++i) {
        const int T = s.t0 + i, c = cnt + i, sb = c & 1;
        if (!dead) dead = !warp_wait(&ctl->info[sb], (c >> 1) & 1, abort, lane);
        bool plain = true;
        uint32_t seen = live ? kFull : 0u;
        if (!dead) {
          uint32_t pl = kFull;
#pragma unroll
          for (int x = 0; x < kValWarps; ++x) pl &= ctl->plain[sb][x];
          plain = pl == kFull;
          if (!plain && live) {
            // compressed and window rows by position, drafted ones (consecutive) by the node's ancestor bits
            seen = 0;
            const int4* keys = reinterpret_cast<const int4*>(&ctl->key[sb][r0]);
#pragma unroll
            for (int x = 0; x < kCols; x += 2) {
              const int4 k = keys[x / 2];
              seen |= (pos >= k.x && pos <= k.y ? 1u : 0u) << x;
              seen |= (pos >= k.z && pos <= k.w ? 2u : 0u) << x;
            }
            const int d0 = kRows * T + r0 - s.n - s.w;  // the first row as a drafted node
            if (!p.idx && d0 > -kCols && d0 < s.m) {
              const int w = max(d0, 0) >> 5;
              uint32_t bits = __funnelshift_r(anc[w], w + 1 < kMaxNodes / 32 ? anc[w + 1] : 0u, max(d0, 0) & 31);
              if (d0 < 0) bits <<= -d0;
              seen |= bits;
            }
          }
        }
        if (!dead) dead = !warp_wait(&ctl->s_full[sb], (c >> 1) & 1, abort, lane);
        float d[kCols];  // x - m; where a score passes its maximum by more than 2^8 the maxima are raised first
#pragma unroll 1
        for (int again = 0; again < 2; ++again) {
          bool raise = false;
          float top = -INFINITY;
          if (!dead) {
            tc_fence_after();
            uint32_t raw[kCols];
            tmem_ld32(tmem + lane_base + kColS + 64 * sb + kCols * cg, raw);
            tmem_wait_ld();
            const float m = ctl->m[j];
            if (!plain && again == 0 && T >= s.full) {
              uint32_t odd = 0;
#pragma unroll
              for (int x = 0; x < kCols; ++x) odd |= (raw[x] & 0x7f800000u) == 0x7f800000u ? 1u << x : 0u;
              if (odd) {
                wait_bar(&ctl->v_here[h], c & 1, abort);
                for (int x = 0; x < kCols; ++x)
                  if ((odd >> x) & 1u) zero_bad_row<C::kQuant>(sV, r0 + x);
              }
            }
#pragma unroll
            for (int x = 0; x < kCols; ++x) {
              float v = __uint_as_float(raw[x]) * p.score_scale;
              if (C::kRowScale) v = fmaf(v, ctl->scale[sb][r0 + x], ctl->lscale[sb][r0 + x]);
              d[x] = (seen >> x) & 1u ? v : -INFINITY;
              top = fmaxf(top, d[x]);
            }
            raise = top > m + kRaise;
#pragma unroll
            for (int x = 0; x < kCols; ++x) d[x] -= m;
          }
          if (again || !soft_or(raise)) break;
          ctl->part[2 * cg + h][j] = top;
          soft_sync();
          if (q < kQ) {
            float mx = ctl->part[0][q];
#pragma unroll
            for (int x = 1; x < 4; ++x) mx = fmaxf(mx, ctl->part[x][q]);
            const float m = ctl->m[q];
            const bool up = mx > m + kRaise;
            ctl->alpha[q] = up ? exp2_approx(m - mx) : 1.f;
            if (up) ctl->m[q] = mx;
          }
          soft_sync();
          const float a = ctl->alpha[j];
          l *= a;
          if (i > 0) {  // the accumulator too, once the products before this tile's are in
            if (!dead) dead = !warp_wait(&ctl->v_empty[1], (c - 1) & 1, abort, lane);
            if (!dead) {
              tc_fence_after();
#pragma unroll 1
              for (int x = 0; x < kChans; x += 16) {
                uint32_t o[16];
                const uint32_t addr = tmem + lane_base + kColO + kChans * cg + x;
                tmem_ld16(addr, o);
                tmem_wait_ld();
#pragma unroll
                for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * a);
                tmem_st16(addr, o);
              }
              tmem_wait_st();
            }
            // The next product adds to all 128 lanes but waits for one half's weights only (p_full[h]): no warp hands
            // over weights until all of them have rescaled their lanes.
            tc_fence_before();
            soft_sync();
            tc_fence_after();
          }
        }
        uint32_t pk[kCols / 2];
#pragma unroll
        for (int x = 0; x < kCols; x += 2) {
          const float a = exp2_approx(d[x]), b = exp2_approx(d[x + 1]);
          // the weights the product uses are the ones l sums (row scales: the stored row's weight carries its scale,
          // the denominator's does not)
          pk[x / 2] = C::kQuant ? f32x2_to_f16x2_sat(a, b) : cvt_bf16x2(a, b);
          if (C::kRowScale) {
            l = fmaf(a, ctl->iscale[sb][r0 + x], fmaf(b, ctl->iscale[sb][r0 + x + 1], l));
          } else if (C::kQuant) {
            const float2 w = f16x2_to_f32(pk[x / 2]);
            l += w.x + w.y;
          } else {
            l += bf16lo(pk[x / 2]) + bf16hi(pk[x / 2]);
          }
        }
        // this half of the weights was last read by the previous tile's product
        if (!dead && c > 0) dead = !warp_wait(&ctl->v_empty[h], (c - 1) & 1, abort, lane);
        if (dead) continue;
        uint8_t* prow = sP + h * kQSlab + j * 128;
#pragma unroll
        for (int x = 0; x < kCols / 8; ++x)
          *reinterpret_cast<uint4*>(prow + (((kCols / 8 * cg + x) ^ (j & 7)) << 4)) =
              make_uint4(pk[4 * x], pk[4 * x + 1], pk[4 * x + 2], pk[4 * x + 3]);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_pair(lead_addr(&ctl->p_full[h]));
      }
      // ---- epilogue
      soft_sync();  // (part is free: the last raise has been read)
      ctl->part[2 * cg + h][j] = l;
      soft_sync();
      const int slot = 2 * pair + (s.t0 == 0 ? 1 : 0);
      if (q < kQ) {
        float L = 0.f;
#pragma unroll
        for (int x = 0; x < 4; ++x) L += ctl->part[x][q];
        ctl->alpha[q] = !final_out ? 1.f : L == 0.f ? 0.f : __frcp_rn(L);  // (no row: zeros)
        if (!final_out && !dead) {
          // (a query that is not finite: its NaN has to pass the merge, which skips runs without rows)
          p.ml[size_t(slot) * kGroup + rank * kQ + q] =
              make_float4(L != L ? INFINITY : ctl->m[q], L, __int_as_float(ctl->row_pos[q]),
                          __int_as_float(q < rows ? row0 + q : -1));
          if (q == 0 && rank == 0) p.rec[slot] = Rec{1, s.b, s.g, s.t0, s.t1, s.tiles, 0, 0};
        }
      }
      soft_sync();
      if (!dead) dead = !warp_wait(&ctl->o_done, segs & 1, abort, lane);
      tc_fence_after();
      if (!dead) {
        const float a = ctl->alpha[j];
        const float2* my_rot = ctl->rot + ctl->row_node[j] * pairs;
        const int rch = kDim - p.rope_dim, odd = lane & 1;
        // lane pairs swap 16-byte pieces, so that a store fills whole 32-byte sectors: first the even lane's row
        const bool live_e = (j & ~1) < rows, live_o = (j | 1) < rows;
#pragma unroll 1
        for (int x = 0; x < kChans; x += 16) {
          const int ch = kHalf * h + kChans * cg + x;
          uint32_t o[16];
          tmem_ld16(tmem + lane_base + kColO + kChans * cg + x, o);
          tmem_wait_ld();
#pragma unroll
          for (int y = 0; y < 16; ++y) o[y] = a == 0.f ? 0u : __float_as_uint(__uint_as_float(o[y]) * a);
          if (final_out && ch + 16 > rch && live) {
#pragma unroll
            for (int y = 0; y < 16; y += 2) {
              if (ch + y < rch) continue;
              const int m = (ch + y - rch) >> 1;
              float2 r;
              if (table) r = my_rot[m];
              else rotation(p.rope.theta_pi[m], pos, &r.x, &r.y);
              const float e = __uint_as_float(o[y]), g = __uint_as_float(o[y + 1]);
              o[y] = __float_as_uint(fmaf(e, r.x, -g * r.y));
              o[y + 1] = __float_as_uint(fmaf(e, r.y, g * r.x));
            }
          }
          if (final_out && !p.out_fp32) {
            uint32_t w[8];
#pragma unroll
            for (int y = 0; y < 8; ++y) w[y] = cvt_bf16x2(__uint_as_float(o[2 * y]), __uint_as_float(o[2 * y + 1]));
#pragma unroll
            for (int y = 0; y < 4; ++y) {  // the even lane keeps both rows' first piece, the odd lane the second
              const uint32_t got = __shfl_xor_sync(kFull, odd ? w[y] : w[4 + y], 1);
              if (odd) w[y] = got;
              else w[4 + y] = got;
            }
            uint16_t* dst = static_cast<uint16_t*>(p.out) + size_t(row0 + (j & ~1)) * kDim + ch + 8 * odd;
            if (live_e) *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
            if (live_o) *reinterpret_cast<uint4*>(dst + kDim) = make_uint4(w[4], w[5], w[6], w[7]);
          } else {
#pragma unroll
            for (int z = 0; z < 16; z += 8) {
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const uint32_t got = __shfl_xor_sync(kFull, odd ? o[z + y] : o[z + 4 + y], 1);
                if (odd) o[z + y] = got;
                else o[z + 4 + y] = got;
              }
              float* dst = (final_out ? static_cast<float*>(p.out) + size_t(row0 + (j & ~1)) * kDim
                                      : p.o_part + (size_t(slot) * kGroup + rank * kQ + (j & ~1)) * kDim) + ch + z + 4 * odd;
              if (live_e) *reinterpret_cast<uint4*>(dst) = make_uint4(o[z], o[z + 1], o[z + 2], o[z + 3]);
              if (live_o) *reinterpret_cast<uint4*>(dst + kDim) = make_uint4(o[z + 4], o[z + 5], o[z + 6], o[z + 7]);
            }
          }
        }
      }
      tc_fence_before();
      soft_sync();  // (the statistics and rotations are read; the next part overwrites them)
    }
  } else if (warp >= kVal0) {
    // ------------------------------------------------------------ values, and what the rows are
    const int vw = warp - kVal0, half = vw / (kValWarps / 2);
    // tile T's rows of this warp: the one TMA row, or a row a lane
    struct Set {
      bool tma;
      int32_t row0;
      const uint8_t *my, *mysc;
      float sr;
      Key key;
    };
    int last_met = -1;  // the last part whose nodes were waited for
    bool ok = true;
    auto met = [&]() {
      if (last_met != segs) {
        ok = warp_wait(&ctl->meta, segs & 1, abort, lane);
        last_met = segs;
      }
      return ok;
    };
    auto resolve = [&](Set& e, int T) {
      int32_t trow[2];
      e.tma = !C::kQuant && T < s.full && tma_rows(p, s.b, T, trow);
      e.row0 = half ? trow[1] : trow[0];
      if (e.tma) return;
      int64_t row;
      const Rows* src = row_source(p, s, ctl, T, kValRows * vw + lane, &row, &e.key, met);
      e.my = src ? src->codes + size_t(row) * row_bytes(FMT) : nullptr;
      if (FMT == DSV4KV_FP4_E2M1_G16)
        e.mysc = src ? static_cast<const uint8_t*>(src->scales) + size_t(row) * (kDim / 16) : nullptr;
      if (C::kRowScale) {
        e.sr = src ? static_cast<const float*>(src->scales)[row] : 1.f;
        if (e.sr == 0.f && !kRotary) e.my = nullptr;  // a row of zeros
      }
    };
    while (ok && next_part()) {
      load_part();
      const int nt = s.t1 - s.t0;
      Set cur, nxt;
      Dequant<C::kQuant ? FMT : DSV4KV_FP8_E4M3_ROW, 32> dq;
      resolve(cur, s.t0);
      if (!ok) break;
      if constexpr (C::kQuant) dq.fetch(cur.my, cur.mysc, kHalf * rank, 0, lane);
#pragma unroll 1
      for (int i = 0; i < nt && ok; ++i) {
        const int T = s.t0 + i, c = cnt + i, sb = c & 1;
        float inv = 0.f;
        // (the softmax is done with tile c - 2's: its product has been waited for)
        if (cur.tma) {
          if (lane == 0) ctl->plain[sb][vw] = kFull;
        } else {
          const int r = kValRows * vw + lane;
          if (C::kRowScale) {
            const float sr = cur.sr == 0.f ? 1.f : cur.sr, at_least = fmaxf(sr, kMinScale);
            inv = 1.f / at_least;
            ctl->scale[sb][r] = sr;
            ctl->lscale[sb][r] = __log2f(at_least);
            ctl->iscale[sb][r] = inv;
            if (kRotary && cur.sr == 0.f) inv = -inv;  // (zero but for its rotary channels)
          }
          ctl->key[sb][r] = cur.key;
          const uint32_t plain = __ballot_sync(kFull, cur.key.lo == 0 && cur.key.hi == kNever);
          if (lane == 0) ctl->plain[sb][vw] = plain;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->info[sb]);
        // the next tile's table and index reads: while this one's buffer is in use, or (below) its copies run
        if ((C::kQuant || cur.tma) && i + 1 < nt) resolve(nxt, T + 1);
        if (ok && c > 0) ok = warp_wait(&ctl->v_empty[half], (c - 1) & 1, abort, lane);
        if (!ok) break;
        const uint32_t bar = lead_addr(&ctl->v_full[half]);
        if (cur.tma) {
          if (lane == 0) {
            const bool mine = vw % (kValWarps / 2) == 0;  // one warp a half
            if (mine && rank == 0) mbar_arrive_expect_tx(&ctl->v_full[half], 2 * kVPart);
            else mbar_arrive_pair(bar);
            if (mine) tma_load_3d_pair(sV + half * kVPart, &tm_comp, bar, 0, cur.row0, 4 * rank);
            mbar_arrive(&ctl->v_here[half]);  // (nobody waits for a whole tile's)
          }
          __syncwarp();
        } else {
          if constexpr (C::kQuant) {
            const int nb = dq.batches(kHalf * rank);
            auto cell = [&](int r, int ch) { return val_cell(sV, kValRows * vw + r, ch); };
            dq.put(inv, kHalf * rank, 0, lane, cell);
#pragma unroll 1
            for (int x = 1; x < nb; ++x) {
              dq.fetch(cur.my, cur.mysc, kHalf * rank, x, lane);
              dq.put(inv, kHalf * rank, x, lane, cell);
            }
          } else {
            // 8 lanes a row, 4 rows at a time: 64 channels (a slab) of each, slab after slab
            const uint8_t* rows[8];
#pragma unroll
            for (int y = 0; y < 8; ++y) rows[y] = shfl_ptr(cur.my, (lane >> 3) + 4 * y);
#pragma unroll
            for (int z = 0; z < 8; ++z) {
              const int r = (lane >> 3) + 4 * z;
              const uint8_t* g = rows[z];
              uint8_t* dst = val_cell(sV, kValRows * vw + r, 8 * (lane & 7));
              const uint8_t* src = g ? g + 2 * kHalf * rank + 16 * (lane & 7) : p.draft.codes;
#pragma unroll
              for (int y = 0; y < 4; ++y) cp_async16_zfill(dst + y * kVSlab, src + (g ? 128 * y : 0), g ? 16 : 0);
            }
            cp_async_commit();
            if (i + 1 < nt) resolve(nxt, T + 1);
            cp_async_wait_group<0>();
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&ctl->v_here[half]);
            mbar_arrive_pair(bar);
          }
        }
        cur = nxt;
        if constexpr (C::kQuant)
          if (i + 1 < nt) dq.fetch(cur.my, cur.mysc, kHalf * rank, 0, lane);
      }
    }
  } else {
    // ------------------------------------------------------------ keys (16 rows a warp), 256 channels at a time
    const int kw = warp - kKey0;
    struct Set {
      bool tma;
      int32_t row0;
      const uint8_t *my, *mysc;
      float inv;
    };
    int last_met = -1;
    bool ok = true;
    auto met = [&]() {
      if (last_met != segs) {
        ok = warp_wait(&ctl->meta, segs & 1, abort, lane);
        last_met = segs;
      }
      return ok;
    };
    auto resolve = [&](Set& e, int T) {
      int32_t trow[2];
      e.tma = !C::kQuant && T < s.full && tma_rows(p, s.b, T, trow);
      e.row0 = rank ? trow[1] : trow[0];
      if (e.tma) return;
      int64_t row;
      Key key;
      const Rows* src = row_source(p, s, ctl, T, kKeys * rank + 16 * kw + (lane & 15), &row, &key, met);
      e.my = src ? src->codes + size_t(row) * row_bytes(FMT) : nullptr;
      if (FMT == DSV4KV_FP4_E2M1_G16)
        e.mysc = src ? static_cast<const uint8_t*>(src->scales) + size_t(row) * (kDim / 16) : nullptr;
      if (C::kRowScale) {
        const float sr = src ? static_cast<const float*>(src->scales)[row] : 1.f;
        e.inv = sr == 0.f ? -1.f : 1.f / fmaxf(sr, kMinScale);  // (as the values')
        if (sr == 0.f && !kRotary) e.my = nullptr;
      }
    };
    // the rows of a tile on their way to L2 (the keys' and the values' loads come after): two lanes a row
    auto ahead = [&](const Set& e) {
      constexpr int kBytes = row_bytes(FMT) / 2;
      if (e.my)
#pragma unroll
        for (int x = 0; x < kBytes; x += 128) prefetch_l2(e.my + kBytes * (lane >> 4) + x);
    };
    while (ok && next_part()) {
      load_part();
      const int nt = s.t1 - s.t0;
      Set cur, nxt;
      Dequant<C::kQuant ? FMT : DSV4KV_FP8_E4M3_ROW, 16> dq;
      resolve(cur, s.t0);
      if (!ok) break;
      if constexpr (C::kQuant) dq.fetch(cur.my, cur.mysc, 0, 0, lane);
#pragma unroll 1
      for (int i = 0; i < nt && ok; ++i) {
        const int T = s.t0 + i, c = cnt + i;
        if ((C::kQuant || cur.tma) && i + 1 < nt) {  // (as the values')
          resolve(nxt, T + 1);
          if (C::kQuant) ahead(nxt);
        }
#pragma unroll 1
        for (int x = 0; x < 2 && ok; ++x) {
          if (c > 0) ok = warp_wait(&ctl->k_empty[x], (c - 1) & 1, abort, lane);
          if (!ok) break;
          const uint32_t bar = lead_addr(&ctl->k_full[x]);
          if (cur.tma) {
            if (lane == 0) {
              if (kw == 0 && rank == 0) mbar_arrive_expect_tx(&ctl->k_full[x], kKBytes);
              else mbar_arrive_pair(bar);
              if (kw == 0) tma_load_3d_pair(sK + 4 * x * kKSlab, &tm_comp, bar, 0, cur.row0, 4 * x);
            }
            __syncwarp();
            continue;
          }
          if constexpr (!C::kQuant) {
            const uint8_t* rows[4];  // as the values
#pragma unroll
            for (int z = 0; z < 4; ++z) rows[z] = shfl_ptr(cur.my, (lane >> 3) + 4 * z);
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              const int r = (lane >> 3) + 4 * z;
              const uint8_t* g = rows[z];
              uint8_t* dst = key_cell(sK, 16 * kw + r, kHalf * x + 8 * (lane & 7));
              const uint8_t* src = g ? g + 2 * kHalf * x + 16 * (lane & 7) : p.draft.codes;
#pragma unroll
              for (int y = 0; y < 4; ++y) cp_async16_zfill(dst + y * kKSlab, src + (g ? 128 * y : 0), g ? 16 : 0);
            }
            cp_async_commit();
            if (x == 0) continue;  // (handed over below, while the second half is on its way)
            cp_async_wait_group<1>();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_pair(lead_addr(&ctl->k_full[0]));
            if (i + 1 < nt) resolve(nxt, T + 1);
            cp_async_wait_group<0>();
          } else {
            auto cell = [&](int r, int ch) { return key_cell(sK, 16 * kw + r, kHalf * x + ch); };
            const int nb = dq.batches(kHalf * x);
            dq.put(cur.inv, kHalf * x, 0, lane, cell);
#pragma unroll 1
            for (int y = 1; y < nb; ++y) {
              dq.fetch(cur.my, cur.mysc, kHalf * x, y, lane);
              dq.put(cur.inv, kHalf * x, y, lane, cell);
            }
          }
          if constexpr (C::kQuant)
            if (x == 0) dq.fetch(cur.my, cur.mysc, kHalf, 0, lane);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive_pair(bar);
        }
        if (!ok) cp_async_wait_group<0>();
        cur = nxt;
        if constexpr (C::kQuant)
          if (ok && i + 1 < nt) dq.fetch(cur.my, cur.mysc, 0, 0, lane);
      }
    }
  }
  __syncthreads();
  if (ctl->abort) {
    if (tid == 0) set_status(p.status, DSV4KV_DEV_TIMEOUT);
    // copies that were in flight when a wait gave up have landed long before this
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 1000000ull) {
    }
  }
  // neither CTA leaves while the other may still reach its shared memory or TMEM
  __syncthreads();
  cluster_sync();
  if (warp == 1) tmem_dealloc_pair(tmem, kTmemCols);
  __syncthreads();
  cluster_sync();
}

// Merges the partial sums of the group whose first run ends in pair blockIdx.x / 16 (nothing to do when it did not cut
// one): 16 blocks a group, one warp a query row.
__global__ void __launch_bounds__(256) tree_combine(const __grid_constant__ Params p, int P) {
  const int c = blockIdx.x >> 4, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int j = (blockIdx.x & 15) * 8 + warp;
  pdl_trigger();
  pdl_wait();
  // (most groups are cut once: the next run's record is read along with the first one's)
  const bool any = c + 1 < P;
  const Rec own = p.rec[2 * c + 1];
  Rec r = p.rec[any ? 2 * c + 2 : 2 * c];
  const float4 ml0 = p.ml[size_t(2 * c + 1) * kGroup + j], ml1 = p.ml[size_t(any ? 2 * c + 2 : 2 * c) * kGroup + j];
  if (!own.valid) return;
  const int pos = __float_as_int(ml0.z), row = __float_as_int(ml0.w);
  if (row < 0) return;
  // the runs behind it: first slots of the next pairs, until one ends the group
  float M = ml0.x;
  int last = c;
  for (int end = own.t1; end < own.tiles && last + 1 < P; ++last) {
    if (last > c) r = p.rec[2 * (last + 1)];
    if (!r.valid || r.b != own.b || r.g != own.g) {  // (a run that timed out)
      if (lane == 0) set_status(p.status, DSV4KV_DEV_INCONSISTENT);
      return;
    }
    end = r.t1;
    M = fmaxf(M, last > c ? p.ml[size_t(2 * (last + 1)) * kGroup + j].x : ml1.x);
  }
  float L = 0.f;
  float4 o[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) o[q] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int x = c; x <= last; ++x) {
    const size_t slot = x == c ? 2 * c + 1 : 2 * x;
    const float4 ml = x == c ? ml0 : x == c + 1 ? ml1 : p.ml[slot * kGroup + j];
    if (ml.y == 0.f) continue;  // it saw no row (its O may be unwritten)
    const float w = exp2_approx(ml.x - M);
    L = fmaf(w, ml.y, L);
    const float4* src = reinterpret_cast<const float4*>(p.o_part + (slot * kGroup + j) * kDim) + lane;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float4 v = src[32 * q];
      o[q].x = fmaf(w, v.x, o[q].x);
      o[q].y = fmaf(w, v.y, o[q].y);
      o[q].z = fmaf(w, v.z, o[q].z);
      o[q].w = fmaf(w, v.w, o[q].w);
    }
  }
  const float inv = L == 0.f ? 0.f : __frcp_rn(L);
  const int r0 = kDim - p.rope_dim;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int ch = 128 * q + 4 * lane;
    float v[4] = {o[q].x * inv, o[q].y * inv, o[q].z * inv, o[q].w * inv};
#pragma unroll
    for (int e = 0; e < 4; e += 2)
      if (ch + e >= r0) {
        float cs, sn;
        rotation(p.rope.theta_pi[(ch + e - r0) >> 1], pos, &cs, &sn);
        const float a = v[e], b = v[e + 1];
        v[e] = fmaf(a, cs, -b * sn);
        v[e + 1] = fmaf(a, sn, b * cs);
      }
    const size_t at = size_t(row) * kDim + ch;
    if (p.out_fp32) *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(v[0], v[1], v[2], v[3]);
    else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) = make_uint2(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]));
  }
}

int64_t groups_max(int batch, int heads, int64_t nodes, int k) { return k > 0 ? nodes : nodes * heads / kGroup + batch; }
int64_t tiles_max(int max_nodes, int64_t t_max, int window, int stride, int k) {
  const int64_t n = t_max + max_nodes > window ? (t_max + max_nodes - window) / stride : 0;
  return ((k > 0 ? std::min<int64_t>(n, k) : n) + std::min<int64_t>(t_max, window) + max_nodes + kRows - 1) / kRows;
}
// Pairs of CTAs that a call launches: at most one a tile.
int pairs_of(int batch, int heads, int max_nodes, int64_t nodes, int64_t t_max, int window, int stride, int k) {
  const int64_t units = groups_max(batch, heads, nodes, k) * tiles_max(max_nodes, t_max, window, stride, k);
  return int(std::max<int64_t>(1, std::min<int64_t>(sm_count() / 2, units)));
}

struct Layout {
  size_t rec, ml, o, total;
};
Layout layout(int P) {
  Layout l;
  l.rec = 256;
  l.ml = l.rec + (size_t(2) * P * sizeof(Rec) + 255) / 256 * 256;
  l.o = l.ml + size_t(2) * P * kGroup * sizeof(float4);
  l.total = l.o + size_t(2) * P * kGroup * kDim * sizeof(float);
  return l;
}

template <int FMT>
cudaError_t launch_tree(const CUtensorMap& tq, const CUtensorMap& tc, const Params& p, int P, cudaStream_t stream) {
  static std::atomic<uint64_t> ready{0};
  if (!done_on_device(ready)) {
    const cudaError_t e =
        cudaFuncSetAttribute(tree_kernel<FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmemBytes));
    if (e != cudaSuccess) return e;
    mark_done_on_device(ready);
  }
  return launch_pdl_cluster(tree_kernel<FMT>, dim3(unsigned(2 * P)), dim3(kThreads), kSmemBytes, 2, stream, tq, tc,
                            p);
}

Rows rows_of(const dsv4kv_cache& c, const PageDesc& pg) {
  return Rows{pg.table, pg.page_rows, pg.table_stride, pg.pool_pages, static_cast<const uint8_t*>(c.codes), c.scales};
}

}  // namespace

bool tree_units_ok(int batch, int heads, int max_nodes, int64_t nodes, int64_t t_max, int window, int stride, int k) {
  return groups_max(batch, heads, nodes, k) * tiles_max(max_nodes, t_max, window, stride, k) < (int64_t(1) << 31) - 4096;
}

size_t tree_ws_bytes(int batch, int heads, int max_nodes, int64_t nodes, int64_t t_max, int window, int stride, int k) {
  return layout(pairs_of(batch, heads, max_nodes, nodes, t_max, window, stride, k)).total;
}

dsv4kv_status tree_decode_launch(const TreeArgs& a, void* ws, cudaStream_t stream) {
  const int P = pairs_of(a.batch, a.heads, a.max_nodes, a.nodes, a.t_max, a.window, a.stride, a.idx ? a.k : 0);
  const Layout lay = layout(P);
  uint8_t* base = static_cast<uint8_t*>(ws);
  Params p;
  p.comp = rows_of(a.comp, a.comp_pg);
  p.win = rows_of(a.win, a.win_pg);
  p.draft = rows_of(a.draft, PageDesc{nullptr, 1, 0, 0});
  p.cu = a.cu;
  p.parent = a.parent;
  p.idx = a.idx;
  p.t_seq = a.t_seq;
  p.batch = a.batch;
  p.heads = a.heads;
  p.nodes = int(a.nodes);
  p.max_nodes = a.max_nodes;
  p.window = a.window;
  p.stride = a.stride;
  p.k = a.idx ? a.k : 0;
  p.t_max = a.t_max;
  p.score_scale = a.sm_scale * 1.4426950408889634f;
  p.rope_dim = a.rope_dim;
  p.out_fp32 = a.out_fp32;
  p.out = a.out;
  p.status = reinterpret_cast<uint32_t*>(base);
  p.rec = reinterpret_cast<Rec*>(base + lay.rec);
  p.ml = reinterpret_cast<float4*>(base + lay.ml);
  p.o_part = reinterpret_cast<float*>(base + lay.o);
  rope_table_fill(&p.rope, a.rope_dim, a.rope_base);
  // boxes of 64 rows x 8 (queries) or 4 (keys, values) chunks of 64 channels, chunk after chunk in shared memory
  CUtensorMap tq{}, tc{};
  if (!encode_tmap_3d(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.q, 64, uint64_t(a.nodes) * a.heads, 8, kDim * 2, 128, 64, kQ,
                      8, CU_TENSOR_MAP_SWIZZLE_128B))
    return set_error(DSV4KV_ERR_CUDA, "tree_decode_paged: tensor map of q");
  // (no sequence of a pool without pages has a row to load: any valid map serves)
  const bool none = !a.comp.codes || a.comp.rows == 0;
  if (a.comp.fmt == DSV4KV_BF16 &&
      !encode_tmap_3d(&tc, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, none ? a.q : a.comp.codes, 64, none ? 1 : uint64_t(a.comp.rows),
                      8, kDim * 2, 128, 64, 64, 4, CU_TENSOR_MAP_SWIZZLE_128B))
    return set_error(DSV4KV_ERR_CUDA, "tree_decode_paged: tensor map of the compressed cache");
  cudaError_t e;
  switch (a.comp.fmt) {
    case DSV4KV_BF16: e = launch_tree<DSV4KV_BF16>(tq, tc, p, P, stream); break;
    case DSV4KV_FP8_E4M3_ROW: e = launch_tree<DSV4KV_FP8_E4M3_ROW>(tq, tc, p, P, stream); break;
    case DSV4KV_FP4_E2M1_G16: e = launch_tree<DSV4KV_FP4_E2M1_G16>(tq, tc, p, P, stream); break;
    default: e = launch_tree<DSV4KV_FP8_E4M3_ROW_ROPE_BF16>(tq, tc, p, P, stream); break;
  }
  if (e != cudaSuccess) return set_error(DSV4KV_ERR_CUDA, "tree_kernel: %s", cudaGetErrorString(e));
  dsv4kv_status st = check_launch("tree_kernel");
  if (st != DSV4KV_OK) return st;
  // (a call whose groups fit the pairs and have few tiles never cuts one: see the split rule)
  const int k = a.idx ? a.k : 0;
  const bool never = groups_max(a.batch, a.heads, a.nodes, k) <= P &&
                     tiles_max(a.max_nodes, a.t_max, a.window, a.stride, k) <= kSplitCost + 1;
  if (P > 1 && !never) launch_pdl(tree_combine, dim3(unsigned(16 * P)), dim3(256), 0, stream, p, P);
  return check_launch("tree_combine");
}

}  // namespace dsv4kv
