// Decode attention for trees of drafted tokens over paged caches.
//
// Node i of sequence b, at position p_i = t_b + (its number of strict
// ancestors), attends to the compressed entries [0, N(p_i)) (or its selected
// ones), the window rows of positions >= p_i - W and its strict ancestors'
// drafted rows, in one softmax; the cached vector is key and value ([P2] Step
// 3); the output is rotated back by p_i ([P1] "Shared key and value").
//
// The (node, head) pairs of a sequence are flattened into query rows; a group
// of 64 of them shares every cache row it reads (for the selected form a
// group lies within one node).  A group's row list is cut into tiles of 128
// rows: whole tiles of compressed rows first (dense form), then a packed tail
// of the remaining compressed rows, the window rows and the drafted rows; a
// selected list is packed throughout.
//
// Work split.  One CTA per SM.  When the groups fill the SMs evenly a CTA takes
// whole groups (c, c + P, ...); otherwise the tiles of all groups are laid
// end to end and cut into equal runs, a group cut by a run boundary leaving
// fp32 partial sums (O, m, l) that tree_combine merges with log-sum-exp weights.
//
// A tile (22 warps).  Shared memory holds the queries (64 KB), one tile (128 KB:
// 8 slabs of 64 channels x 128 rows, 128-byte swizzle) and the weights (16 KB).
//   * S^T = R . Q^T: M = 128 rows, N = 64 queries, 32 K-steps (one tcgen05.mma
//     each), into TMEM (lane = row, column = query);
//   * 16 softmax warps, one row and 16 queries a thread: the weights
//     2^(x - m_j) against a running maximum m_j that is raised only when some
//     score passes it by 2^8 (one vote a tile; the column maxima are reduced
//     over the rows only then), rounded to 16 bits and stored row by row, which
//     is the MN-major form of the B operand; l_j sums the rounded weights per
//     thread and is reduced over the rows once per group;
//   * O^T += R^T . P^T: four blocks of M = 128 channels, N = 64, 8 K-steps, from
//     the SAME slabs.  A block's commit frees its two slabs, so the next tile
//     loads behind the products (warp 0 by TMA for whole bf16 tiles, warps
//     2-5 otherwise: 16-byte cp.async, or dequantisation to f16 as in the
//     decode kernel).
// Rows that no node of the batch may read are zero-filled, not loaded.  A loaded
// row that some query of the group does not see has weight 0 for it; if it
// holds an infinity or NaN (its masked score is then not finite) the row is
// zeroed in shared memory before the second product, and only the queries
// that see it get its non-finite weight.
#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "internal.h"

namespace dsv4kv {

namespace {

constexpr int kRows = 128;  // rows per tile
constexpr int kQ = 64;      // query rows per group
constexpr int kDim = 512;
constexpr int kSlabs = kDim / 64;
constexpr int kSlabBytes = kRows * 128;        // 16 KB
constexpr int kTileBytes = kSlabs * kSlabBytes;  // 128 KB
constexpr int kQSlab = kQ * 128;               // 8 KB
constexpr int kQBytes = kSlabs * kQSlab;       // 64 KB
constexpr int kPBytes = kRows * 128;           // 64 weights of 16 bits per row
constexpr int kParts = 4;                      // slab pairs = 128-channel blocks
constexpr int kThreads = 704;
constexpr int kLoad0 = 2, kSoft0 = 6;  // first loader warp (4 of them), first softmax warp (16)
constexpr int kSoftThreads = 512;
constexpr int kCols = 16;          // queries a softmax thread
constexpr int kMaxBatch = 1024;
constexpr int kMaxNodes = 256;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 0;    // O^T: 4 channel blocks x 64 queries
constexpr uint32_t kColS = 256;  // S^T: 64 columns
constexpr float kNoMax = -1e30f;  // a maximum that nothing has reached yet
constexpr float kRaise = 8.0f;   // log2 units a score may pass the running maximum by
constexpr int kSplitCost = 3;    // tiles that a cut group's partial sums and merge cost (see split rule)

template <int FMT>
struct Cfg {
  static constexpr bool kQuant = FMT != DSV4KV_BF16;
  static constexpr bool kRowScale = FMT == DSV4KV_FP8_E4M3_ROW || FMT == DSV4KV_FP8_E4M3_ROW_ROPE_BF16;
  static constexpr uint32_t kIdescQK = kQuant ? idesc_f16(128, kQ, 0, 0) : idesc_bf16(128, kQ, 0, 0);
  static constexpr uint32_t kIdescPV = kQuant ? idesc_f16(128, kQ, 1, 1) : idesc_bf16(128, kQ, 1, 1);
};

// A cut group's run of tiles in one CTA; slot 2c: the run does not start the group, 2c + 1: it starts it.
struct Rec {
  int valid, b, g, t0, t1, tiles, row0, rows;
};
static_assert(sizeof(Rec) == 32, "");

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
  Rec* rec;       // [2 P]
  float4* ml;     // [2 P][64]: m, l, position (int bits)
  float* o_part;  // [2 P][64][512]
  RopeTable rope;
};

struct Seg {  // the part of a group that a CTA works on
  int b, g, t0, t1, tiles;  // sequence, group within it, tiles [t0, t1) of `tiles`
  int t, w, m, c0;          // position, window rows, drafted nodes, first node
  int row0, rows;           // first query row, query rows
  int node0, n_nodes;       // nodes of the group (numbers within the sequence)
  int n, full, rem;         // compressed rows listed, whole tiles of them, rows in the tail
  int n_min;                // least entry count of the group's nodes
};

struct __align__(16) Ctl {
  uint64_t q_full, s_full, p_full, o_done;
  uint64_t full[kParts], empty[kParts];
  uint32_t tmem_base;
  volatile int abort;
  int dmax, n_min;
  int b, g, t0;       // the next part to work on
  int whole, share, units;
  uint32_t ok[2][4];  // rows of a tile that the loader warps brought, one word a warp
  float scale[2][kRows];
  __align__(16) float m[kQ];
  __align__(16) float alpha[kQ];
  float part[4][kQ];  // column maxima / sums of the four row quarters
  int col_pos[kQ];          // position of a column's node
  uint64_t colmask[kQ];     // columns of the group's node j
  int node_n[kQ], node_p[kQ];
  uint32_t anc[kQ][kMaxNodes / 32];
  int16_t parent[kMaxNodes];
  int gpre[kMaxBatch + 1];  // groups before sequence b
  int tiles[kMaxBatch];     // tiles of each group of sequence b
};

constexpr size_t kSmemBytes = 1024 + kQBytes + kTileBytes + kPBytes + sizeof(Ctl);
static_assert(kSmemBytes <= 232448, "shared memory per CTA");

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
// Drains a barrier whose arrivals are certain (copies in flight), abort or not.
__device__ __noinline__ void wait_drain(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer() - t0 > 2 * kWaitLimitNs) return;
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int lane) {
  bool ok = true;
  if (lane == 0) ok = wait_bar(bar, parity, abort);
  return __shfl_sync(kFull, ok, 0);
}
__device__ __forceinline__ bool soft_or(bool pred) {  // over the softmax threads
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred pi, po;\n\tsetp.ne.u32 pi, %1, 0;\n\tbarrier.cta.red.or.pred po, 1, 512, pi;\n\tselp.u32 "
      "%0, 1, 0, po;\n\t}"
      : "=r"(r)
      : "r"(uint32_t(pred))
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void soft_sync() { asm volatile("barrier.cta.sync 1, 512;" ::: "memory"); }

__device__ __forceinline__ float exp2_approx(float x) {  // max relative error ~2^-22, far below the weights' 16 bits
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Reduces v[j] (j < 16) over the 32 lanes: the lane gets column col_of(lane)'s result.  Each step sends half of
// the columns to the lane that keeps them: 16 shuffles instead of 80.
__device__ __forceinline__ int col_of(int lane) {
  return ((lane >> 4) & 1) * 8 + ((lane >> 3) & 1) * 4 + ((lane >> 2) & 1) * 2 + ((lane >> 1) & 1);
}
template <class Op>
__device__ __forceinline__ float reduce_cols(float (&v)[kCols], int lane, Op op) {
#pragma unroll
  for (int h = 8; h >= 1; h >>= 1) {
    const bool up = (lane & (2 * h)) != 0;
#pragma unroll
    for (int j = 0; j < h; ++j) {
      const float keep = up ? v[j + h] : v[j], send = up ? v[j] : v[j + h];
      v[j] = op(keep, __shfl_xor_sync(kFull, send, 2 * h));
    }
  }
  return op(v[0], __shfl_xor_sync(kFull, v[0], 1));
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
  return p.idx ? m * ((p.heads + kQ - 1) / kQ) : (m * p.heads + kQ - 1) / kQ;
}
// Tiles of a group whose sequence lists n compressed rows.
__device__ __forceinline__ int tiles_of(const Params& p, int n, int w, int m) {
  if (p.idx) return (min(n, p.k) + w + m + kRows - 1) / kRows;
  return n / kRows + (n % kRows + w + m + kRows - 1) / kRows;
}

// Pool row of logical row i; -1 (flagged) when its page is outside the pool or the table has no entry for it.
__device__ __forceinline__ int64_t map_row(const Rows& r, int b, int i, uint32_t* status) {
  if (!r.table) return i;
  const int pi = i / r.page;
  const int32_t pg = pi < r.tstride ? __ldg(r.table + size_t(b) * r.tstride + pi) : -1;
  if (pg < 0 || pg >= r.pages) {
    set_status(status, DSV4KV_DEV_BAD_PAGE);
    return -1;
  }
  return int64_t(pg) * r.page + (i - pi * r.page);
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

// What row r of tile T of the group is: compressed row (list number), window row, drafted row.
enum : int { kNone = -1, kComp = 0, kWin = 1, kDraft = 2 };
__device__ __forceinline__ int row_kind(const Params& p, const Seg& s, int T, int r, int* i) {
  int u = kRows * T + r;
  if (T < s.full) {
    *i = u;
    return kComp;
  }
  u -= kRows * s.full;
  if (u < s.rem) {
    *i = kRows * s.full + u;
    return kComp;
  }
  u -= s.rem;
  *i = u;
  if (u < s.w) return kWin;
  u -= s.w;
  *i = u;
  return u < s.m ? kDraft : kNone;
}

// Source of row r of tile T: the cache and its pool row; null when there is none.
__device__ __forceinline__ const Rows* row_source(const Params& p, const Seg& s, int T, int r, int64_t* row) {
  int i;
  const int kind = row_kind(p, s, T, r, &i);
  const Rows* c = nullptr;
  *row = -1;
  if (kind == kComp) {
    if (p.idx) {
      const int32_t e = __ldg(p.idx + size_t(s.c0 + s.node0) * p.k + i);
      if (e >= s.n_min) set_status(p.status, DSV4KV_DEV_BAD_INDEX);
      i = e >= s.n_min ? -1 : e;
    }
    if (i >= 0) *row = map_row(p.comp, s.b, i, p.status);
    c = &p.comp;
  } else if (kind == kWin) {
    *row = map_row(p.win, s.b, i, p.status);
    c = &p.win;
  } else if (kind == kDraft) {
    *row = s.c0 + i;
    c = &p.draft;
  }
  return *row < 0 ? nullptr : c;
}

// ---------------------------------------------------------------- loader warps
// Warp lw owns rows 32 lw .. 32 lw + 31 of a tile; lane l resolves row 32 lw + l.
__device__ __forceinline__ uint8_t* cell(uint8_t* tile, int r, int ch) {  // 16-byte unit of channels ch .. ch + 7
  return tile + (ch >> 6) * kSlabBytes + r * 128 + ((((ch & 63) >> 3) ^ (r & 7)) << 4);
}

__device__ __forceinline__ uint64_t shfl_ptr(const uint8_t* p, int src) {
  return __shfl_sync(kFull, reinterpret_cast<uint64_t>(p), src);
}

__device__ __forceinline__ void put_fp8x16(uint8_t* tile, int r, int ch, const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t h[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    h[2 * e] = e4m3x2_to_f16x2(w[e] & 0xffffu);
    h[2 * e + 1] = e4m3x2_to_f16x2(w[e] >> 16);
  }
  *reinterpret_cast<uint4*>(cell(tile, r, ch)) = make_uint4(h[0], h[1], h[2], h[3]);
  *reinterpret_cast<uint4*>(cell(tile, r, ch + 8)) = make_uint4(h[4], h[5], h[6], h[7]);
}

// A part of the warp's rows in registers (fetch), then as f16 in the tile (put).  Parts 0 .. 3 are the slab pairs
// (128 channels); with bf16 rotary channels pair 3 holds 64 fp8 channels and part 4 the 64 rotary ones.
template <int FMT>
struct QuantPart {
  static constexpr bool kRope = FMT == DSV4KV_FP8_E4M3_ROW_ROPE_BF16;
  static constexpr int kCount = kRope ? 5 : 4;
  static constexpr int kN = FMT == DSV4KV_FP4_E2M1_G16 ? 4 : 8;
  uint4 raw[kN];
  uint32_t sc[FMT == DSV4KV_FP4_E2M1_G16 ? kN : 1];

  // my: this lane's row (codes; null: none), mysc: its fp4 scales
  __device__ __forceinline__ void fetch(const uint8_t* my, const uint8_t* mysc, int part, int lane) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      if constexpr (FMT == DSV4KV_FP4_E2M1_G16) {  // 4 lanes a row: 32 channels, 16 bytes of codes, 2 scales each
        const int r = 8 * i + (lane >> 2), c = lane & 3;
        const uint8_t* row = reinterpret_cast<const uint8_t*>(shfl_ptr(my, r));
        const uint8_t* srow = reinterpret_cast<const uint8_t*>(shfl_ptr(mysc, r));
        raw[i] = row ? ld_stream_v4(row + 64 * part + 16 * c) : make_uint4(0, 0, 0, 0);
        sc[i] = row ? *reinterpret_cast<const uint16_t*>(srow + 8 * part + 2 * c) : 0u;
      } else {  // 8 lanes a row: 16 bytes each
        const int r = 4 * i + (lane >> 3), c = lane & 7;
        const uint8_t* row = reinterpret_cast<const uint8_t*>(shfl_ptr(my, r));
        const bool in = !kRope || part != 3 || c < 4;
        raw[i] = row && in ? ld_stream_v4(row + (kRope && part == 4 ? kDim - 64 : 128 * part) + 16 * c)
                           : make_uint4(0, 0, 0, 0);
      }
    }
  }
  // my_inv: 1 / (this lane's row's scale)
  __device__ __forceinline__ void put(uint8_t* tile, int lw, int part, float my_inv, int lane) const {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      if constexpr (FMT == DSV4KV_FP4_E2M1_G16) {
        const int r = 32 * lw + 8 * i + (lane >> 2), ch = 128 * part + 32 * (lane & 3);
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t s1 = e < 2 ? sc[i] & 0xffu : sc[i] >> 8;
          const uint32_t s2 = e4m3x2_to_f16x2(s1 | (s1 << 8));
          uint32_t h[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) h[j] = hmul2(e2m1x2_to_f16x2((w[e] >> (8 * j)) & 0xffu), s2);
          *reinterpret_cast<uint4*>(cell(tile, r, ch + 8 * e)) = make_uint4(h[0], h[1], h[2], h[3]);
        }
      } else {
        const int rl = 4 * i + (lane >> 3), r = 32 * lw + rl, c = lane & 7;
        if (kRope && part == 4) {  // rotary channels as f16(value / scale): the row's scale is in the weights
          const float inv = __shfl_sync(kFull, my_inv, rl);
          const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
          uint32_t h[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = f32x2_to_f16x2_sat(bf16lo(w[e]) * inv, bf16hi(w[e]) * inv);
          *reinterpret_cast<uint4*>(cell(tile, r, kDim - 64 + 8 * c)) = make_uint4(h[0], h[1], h[2], h[3]);
        } else if (!kRope || part != 3 || c < 4) {
          put_fp8x16(tile, r, 128 * part + 16 * c, raw[i]);
        }
      }
    }
  }
};

__host__ __device__ constexpr int row_bytes(int fmt) {
  return fmt == DSV4KV_BF16 ? 2 * kDim
         : fmt == DSV4KV_FP8_E4M3_ROW ? kDim
         : fmt == DSV4KV_FP4_E2M1_G16 ? kDim / 2
                                      : kDim + 64;
}

// A row hidden from some query (`hid`: columns) whose masked scores are not finite: if the row itself is not finite it
// is zeroed in the tile, so that its zero weights add zeros.  (A query that is not finite itself says nothing.)
template <bool kF16>
__device__ __noinline__ void zero_bad_row(uint8_t* tile, int r, Ctl* ctl, int c) {
  for (int sp = 0; sp < kParts; ++sp) wait_bar(&ctl->full[sp], c & 1, &ctl->abort);  // (complete: orders the row's loads)
  const uint32_t e = kF16 ? 0x7c00u : 0x7f80u;
  bool bad = false;
#pragma unroll 1
  for (int ch = 0; ch < kDim; ch += 8) {
    const uint4 v = *reinterpret_cast<const uint4*>(cell(tile, r, ch));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) bad |= (w[k] & e) == e || ((w[k] >> 16) & e) == e;
  }
  if (!bad) return;
#pragma unroll 1
  for (int ch = 0; ch < kDim; ch += 8) *reinterpret_cast<uint4*>(cell(tile, r, ch)) = make_uint4(0, 0, 0, 0);
}
template <bool kF16>
__device__ __forceinline__ void hide_bad_row(const uint32_t (&raw)[kCols], uint32_t hid, uint8_t* tile, int r, Ctl* ctl,
                                             int c) {
  bool odd = false;
#pragma unroll
  for (int j = 0; j < kCols; ++j) odd |= ((hid >> j) & 1u) && (raw[j] & 0x7f800000u) == 0x7f800000u;
  if (odd) zero_bad_row<kF16>(tile, r, ctl, c);
}

// ---------------------------------------------------------------- the kernel
template <int FMT>
__global__ void __launch_bounds__(kThreads, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_comp,
                const __grid_constant__ Params p) {
  using C = Cfg<FMT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sR = sQ + kQBytes;
  uint8_t* sP = sR + kTileBytes;
  Ctl* ctl = reinterpret_cast<Ctl*>(sP + kPBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int P = gridDim.x, cta = blockIdx.x;
  volatile int* abort = &ctl->abort;
  pdl_trigger();

  if (tid == 0) {
    mbar_init(&ctl->q_full, 1);
    mbar_init(&ctl->s_full, 1);
    mbar_init(&ctl->p_full, kSoftThreads / 32);
    mbar_init(&ctl->o_done, 1);
    for (int i = 0; i < kParts; ++i) {
      mbar_init(&ctl->full[i], 5);  // warp 0 and the four loader warps, every tile
      mbar_init(&ctl->empty[i], 1);
    }
    ctl->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&ctl->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  if (tid == 64) {
    prefetch_tmap(&tm_q);
    if (!C::kQuant) prefetch_tmap(&tm_comp);
  }
  tc_fence_before();
  pdl_wait();

  // ---- the batch: groups and tiles of every sequence, then which part of them is this CTA's
  for (int b = tid; b < p.batch; b += kThreads) {
    int c0, m;
    uint32_t* st = cta == 0 ? p.status : nullptr;
    seq_nodes(p, b, &c0, &m, st);
    const int t = seq_len(p, b, st);
    ctl->gpre[b + 1] = groups_of(p, m);
    ctl->tiles[b] = m > 0 ? tiles_of(p, entries(t + m - 1, p.window, p.stride), min(t, p.window), m) : 0;
  }
  __syncthreads();
  if (warp == 0) {
    int g = 0, u = 0, most = 0;  // groups, units (tiles of all groups: < 2^31), most tiles of a group
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
      const int b = b0 + lane;
      const int n = b < p.batch ? ctl->gpre[b + 1] : 0, tl = b < p.batch ? ctl->tiles[b] : 0;
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
    const unsigned want = whole ? unsigned(cta) : unsigned(share) * unsigned(cta);
    unsigned at = 0;
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
      const int b = b0 + lane;
      const unsigned tl = b < p.batch ? ctl->tiles[b] : 0;
      const unsigned v = b < p.batch ? unsigned(ctl->gpre[b + 1] - ctl->gpre[b]) * (whole ? 1u : tl) : 0u;
      unsigned x = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x += y;
      }
      const unsigned ex = at + x - v;
      if (want >= ex && want - ex < v) {
        const unsigned off = want - ex;
        ctl->b = b;
        ctl->g = whole ? off : off / tl;
        ctl->t0 = whole ? 0 : off % tl;
      }
      at += __shfl_sync(kFull, x, 31);
    }
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  const bool whole = ctl->whole != 0;
  const int G = ctl->gpre[p.batch];
  // (equal runs) tiles of this CTA's run; (whole groups) the flattened group to take next
  int left = int(max(0ll, min((long long)ctl->share, ctl->units - (long long)ctl->share * cta)));
  int g_next = cta;
  if (tid < 2) p.rec[2 * cta + tid].valid = 0;

  int cnt = 0, segs = 0;  // tiles and groups worked on so far: the barriers' phases
  while (whole ? g_next < G : left > 0) {
    // ---- the group: its rows, its nodes and their ancestors
    Seg s;
    s.b = ctl->b;
    s.g = ctl->g;
    s.t0 = ctl->t0;
    s.tiles = ctl->tiles[s.b];
    s.t1 = whole ? s.tiles : min(s.tiles, s.t0 + left);
    seq_nodes(p, s.b, &s.c0, &s.m, nullptr);
    s.t = seq_len(p, s.b, nullptr);
    s.w = min(s.t, p.window);
    if (p.idx) {
      const int gpn = (p.heads + kQ - 1) / kQ, h0 = (s.g % gpn) * kQ;
      s.node0 = s.g / gpn;
      s.n_nodes = 1;
      s.row0 = (s.c0 + s.node0) * p.heads + h0;
      s.rows = min(kQ, p.heads - h0);
    } else {
      const int f = kQ * s.g;
      s.rows = min(kQ, s.m * p.heads - f);
      s.node0 = f / p.heads;
      s.n_nodes = (f + s.rows - 1) / p.heads - s.node0 + 1;
      s.row0 = s.c0 * p.heads + f;
    }
    if (tid == 0) {  // the queries (the previous group's products have read theirs)
      mbar_arrive_expect_tx(&ctl->q_full, kQBytes);
#pragma unroll 1
      for (int c = 0; c < kSlabs; ++c) tma_load_2d(sQ + c * kQSlab, &tm_q, &ctl->q_full, 64 * c, s.row0);
    }
    if (tid == kThreads - 1) {
      ctl->dmax = 0;
      ctl->n_min = 0x7fffffff;
    }
    if (tid < s.m) {  // (at most 256 nodes)
      int par = p.parent[s.c0 + tid];
      if (par < -1 || par >= tid) {
        set_status(p.status, DSV4KV_DEV_BAD_TREE);
        par = -1;
      }
      ctl->parent[tid] = int16_t(par);
    }
    for (int i = tid; i < kQ * (kMaxNodes / 32); i += kThreads) (&ctl->anc[0][0])[i] = 0;
    if (tid < kQ) ctl->m[tid] = kNoMax;
    __syncthreads();
    if (tid < s.m) {
      int d = 0;
      const int gj = tid - s.node0;
      const bool mine = gj >= 0 && gj < s.n_nodes;
      for (int j = ctl->parent[tid]; j >= 0; j = ctl->parent[j]) {
        ++d;
        if (mine) ctl->anc[gj][j >> 5] |= 1u << (j & 31);
      }
      atomicMax(&ctl->dmax, d);
      if (mine) {
        const int pos = s.t + d, n = entries(pos, p.window, p.stride);
        ctl->node_p[gj] = pos;
        ctl->node_n[gj] = n;
        atomicMin(&ctl->n_min, n);
        // its columns: query rows tid * heads .. + heads of the sequence, within the group
        const int lo = p.idx ? 0 : max(0, tid * p.heads - kQ * s.g);
        const int hi = p.idx ? s.rows : min(s.rows, (tid + 1) * p.heads - kQ * s.g);
        ctl->colmask[gj] = (hi >= 64 ? ~0ull : (1ull << hi) - 1) & ~((1ull << lo) - 1);
      }
    }
    __syncthreads();
    s.n_min = ctl->n_min;
    s.n = p.idx ? min(p.k, s.n_min) : entries(s.t + ctl->dmax, p.window, p.stride);
    s.full = p.idx ? 0 : s.n / kRows;
    s.rem = s.n - kRows * s.full;
    // (the deepest node may be less deep than the schedule allowed for: fewer tiles)
    const int exact = s.full + (s.rem + s.w + s.m + kRows - 1) / kRows;
    const int nt = max(0, min(s.t1, exact) - s.t0);

    if (C::kQuant) {  // queries to f16, in place
      if (wait_bar(&ctl->q_full, segs & 1, abort))
#pragma unroll 1
        for (int i = tid; i < kQBytes / 16; i += kThreads) {
          uint4 v = reinterpret_cast<uint4*>(sQ)[i];
          uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = f32x2_to_f16x2_sat(bf16lo(w[e]), bf16hi(w[e]));
          reinterpret_cast<uint4*>(sQ)[i] = v;
        }
      fence_proxy_async_smem();
      __syncthreads();
    }

    if (warp == 0) {
      // ---------------------------------------------------------- TMA: whole tiles of bf16 rows
      if (lane == 0) {
        int issued = 0;
#pragma unroll 1
        for (int i = 0; i < nt; ++i) {
          const int T = s.t0 + i, c = cnt + i;
          int32_t row[2];
          const bool tma = !C::kQuant && T < s.full && tma_rows(p, s.b, T, row);
          bool ok = true;
#pragma unroll 1
          for (int sp = 0; sp < kParts; ++sp) {
            if (c > 0) ok = wait_bar(&ctl->empty[sp], (c - 1) & 1, abort);
            if (!ok) break;
            if (tma) {
              mbar_arrive_expect_tx(&ctl->full[sp], 2 * kSlabBytes);
#pragma unroll
              for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                  tma_load_2d(sR + (2 * sp + x) * kSlabBytes + h * (kSlabBytes / 2), &tm_comp, &ctl->full[sp],
                              64 * (2 * sp + x), row[h]);
            } else {
              mbar_arrive(&ctl->full[sp]);
            }
            issued = kParts * i + sp + 1;
          }
          if (!ok) break;
        }
        // never leave with copies in flight
        wait_drain(&ctl->q_full, segs & 1);
        if (*abort)
          for (int sp = 0; sp < kParts; ++sp) {
            const int last = (issued - 1 - sp) / kParts;  // tile of part sp issued last
            if (issued > sp) wait_drain(&ctl->full[sp], (cnt + last) & 1);
          }
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA
      if (lane == 0) {
        bool ok = wait_bar(&ctl->q_full, segs & 1, abort);
        const uint64_t qd = smem_desc_sw128(smem_u32(sQ), 16, 1024);
        const uint64_t rd = smem_desc_sw128(smem_u32(sR), 16, 1024);
        const uint64_t ad = smem_desc_sw128(smem_u32(sR), kSlabBytes, 1024);
        const uint64_t pd = smem_desc_sw128(smem_u32(sP), 16, 1024);
#pragma unroll 1
        for (int i = 0; i < nt && ok; ++i) {
          const int c = cnt + i;
#pragma unroll 1
          for (int sp = 0; sp < kParts; ++sp) {
            ok = wait_bar(&ctl->full[sp], c & 1, abort);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int x = 0; x < 8; ++x) {  // 128 channels
              const uint32_t ro = (x >> 2) * kSlabBytes + (x & 3) * 32, qo = (x >> 2) * kQSlab + (x & 3) * 32;
              mma_bf16_ss(tmem + kColS, rd + ((2 * sp * kSlabBytes + ro) >> 4), qd + ((2 * sp * kQSlab + qo) >> 4),
                          C::kIdescQK, (sp | x) ? 1u : 0u);
            }
          }
          if (!ok) break;
          mma_commit(&ctl->s_full);
          ok = wait_bar(&ctl->p_full, c & 1, abort);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int ct = 0; ct < kParts; ++ct) {
#pragma unroll
            for (int kr = 0; kr < kRows / 16; ++kr)
              mma_bf16_ss(tmem + kColO + kQ * ct, ad + ((2 * ct * kSlabBytes + kr * 2048) >> 4),
                          pd + ((kr * 2048) >> 4), C::kIdescPV, (i > 0 || kr > 0) ? 1u : 0u);
            mma_commit(&ctl->empty[ct]);
          }
        }
        mma_commit(&ctl->o_done);  // completes once every product issued so far has
      }
    } else if (warp >= kSoft0) {
      // ---------------------------------------------------------- softmax, epilogue
      const int wq = warp & 3, c0 = kCols * ((warp - kSoft0) >> 2);  // row quarter (TMEM lanes), first column
      const uint32_t lane_base = uint32_t(32 * wq) << 16;
      const int r = 32 * wq + lane;   // this thread's row
      const int q = tid - 32 * kSoft0;  // (q < 64) the query that this thread keeps the statistics of
      const uint32_t valid_cols = s.rows - c0 >= kCols ? 0xffffu : s.rows > c0 ? (1u << (s.rows - c0)) - 1u : 0u;
      if (q < kQ) ctl->col_pos[q] = ctl->node_p[p.idx ? 0 : (kQ * s.g + min(q, s.rows - 1)) / p.heads - s.node0];
      float l[kCols];
#pragma unroll
      for (int j = 0; j < kCols; ++j) l[j] = 0.f;
      bool dead = false;
#pragma unroll 1
      for (int i = 0; i < nt; ++i) {
        const int T = s.t0 + i, c = cnt + i;
        // what the row is and who sees it (while the products run)
        uint32_t seen = valid_cols;
        if (p.idx || T >= s.full || kRows * (T + 1) > s.n_min) {
          int x;
          const int kind = row_kind(p, s, T, r, &x);
          if (kind == kNone) {
            seen = 0;
          } else if (kind != kComp || !p.idx) {
            const int wpos = kind == kWin ? s.t - 1 - (s.t - 1 - x) % p.window : 0;
            seen = 0;
#pragma unroll 1
            for (int j = 0; j < s.n_nodes; ++j) {
              const bool v = kind == kComp ? x < ctl->node_n[j]
                             : kind == kWin ? wpos >= ctl->node_p[j] - p.window
                                            : (ctl->anc[j][x >> 5] >> (x & 31)) & 1u;
              if (v) seen |= uint32_t(ctl->colmask[j] >> c0) & 0xffffu;
            }
          }
        }
        if (!dead) dead = !warp_wait(&ctl->s_full, c & 1, abort, lane);
        // (complete, the product has read the tile: orders the loaders' row words and scales before this)
        if (!dead) dead = !warp_wait(&ctl->full[0], c & 1, abort, lane);
        float f = p.score_scale, ls = 0.f, rinv = 1.f;
        if (!dead) {
          tc_fence_after();
          if (!((ctl->ok[c & 1][wq] >> lane) & 1u)) seen = 0;  // no such row, or a bad page
          if (C::kRowScale) {
            const float rs = ctl->scale[c & 1][r];
            f *= rs;
            ls = rs > 0.f ? __log2f(rs) : 0.f;
            rinv = rs > 0.f ? __frcp_rn(rs) : 0.f;
          }
        }
        // x_j - m_j; a score that passes its maximum by more than 2^8 has the maxima raised, then once more
        float d[kCols];
#pragma unroll 1
        for (int again = 0; again < 2; ++again) {
          bool raise = false;
          if (!dead) {
            uint32_t raw[kCols];
            tmem_ld16(tmem + lane_base + kColS + c0, raw);
            tmem_wait_ld();
            if (seen != valid_cols && again == 0) hide_bad_row<C::kQuant>(raw, valid_cols & ~seen, sR, r, ctl, c);
            float top = -INFINITY;
#pragma unroll
            for (int j = 0; j < kCols; ++j) {
              const float x = (seen >> j) & 1u ? fmaf(__uint_as_float(raw[j]), f, ls) : -INFINITY;
              d[j] = x - ctl->m[c0 + j];
              top = fmaxf(top, d[j]);
            }
            raise = top > kRaise;
          }
          if (again || !soft_or(raise)) break;
          // column maxima over the tile's rows; raise the maxima that were passed
          if (!dead) {
            uint32_t raw[kCols];
            float x[kCols];  // the scores themselves: the differences to kNoMax have lost them
            tmem_ld16(tmem + lane_base + kColS + c0, raw);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < kCols; ++j)
              x[j] = (seen >> j) & 1u ? fmaf(__uint_as_float(raw[j]), f, ls) : -INFINITY;
            const float v = reduce_cols(x, lane, [](float a, float b) { return fmaxf(a, b); });
            if (!(lane & 1)) ctl->part[wq][c0 + col_of(lane)] = v;
          }
          soft_sync();
          if (q < kQ) {
            const float mx = fmaxf(fmaxf(ctl->part[0][q], ctl->part[1][q]), fmaxf(ctl->part[2][q], ctl->part[3][q]));
            const float m = ctl->m[q];
            const bool up = mx > m + kRaise;
            ctl->alpha[q] = up ? exp2_approx(m - mx) : 1.f;
            if (up) ctl->m[q] = mx;
          }
          soft_sync();
          if (!dead) {
#pragma unroll
            for (int j = 0; j < kCols; ++j) l[j] *= ctl->alpha[c0 + j];
            if (i > 0) {  // the accumulator too (this tile's scores are in, so the products before them are)
#pragma unroll 1
              for (int ct = 0; ct < kParts; ++ct) {
                uint32_t o[kCols];
                const uint32_t addr = tmem + lane_base + kColO + kQ * ct + c0;
                tmem_ld16(addr, o);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < kCols; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * ctl->alpha[c0 + j]);
                tmem_st16(addr, o);
              }
              tmem_wait_st();
            }
          }
        }
        if (dead) continue;
        uint8_t* prow = sP + r * 128;
#pragma unroll
        for (int u = 0; u < kCols / 8; ++u) {
          uint32_t pk[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = 8 * u + 2 * e;
            const float a = exp2_approx(d[j]), b = exp2_approx(d[j + 1]);
            // the weights the product uses are the ones l sums (row scales: the stored row's weight carries its
            // scale, the denominator's does not)
            pk[e] = C::kQuant ? f32x2_to_f16x2_sat(a, b) : cvt_bf16x2(a, b);
            if (C::kRowScale) {
              l[j] = fmaf(a, rinv, l[j]);
              l[j + 1] = fmaf(b, rinv, l[j + 1]);
            } else if (C::kQuant) {
              const float2 w = f16x2_to_f32(pk[e]);
              l[j] += w.x;
              l[j + 1] += w.y;
            } else {
              l[j] += bf16lo(pk[e]);
              l[j + 1] += bf16hi(pk[e]);
            }
          }
          *reinterpret_cast<uint4*>(prow + (((c0 / 8 + u) ^ (r & 7)) << 4)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->p_full);
      }
      // ---- epilogue
      {
        const float v = reduce_cols(l, lane, [](float a, float b) { return a + b; });
        if (!(lane & 1)) ctl->part[wq][c0 + col_of(lane)] = v;
      }
      if (!dead) dead = !warp_wait(&ctl->o_done, segs & 1, abort, lane);
      tc_fence_after();
      soft_sync();
      const bool final_out = s.t0 == 0 && s.t1 == s.tiles;
      const int slot = 2 * cta + (s.t0 == 0 ? 1 : 0);
      if (!dead && q < kQ) {
        const float L = (ctl->part[0][q] + ctl->part[1][q]) + (ctl->part[2][q] + ctl->part[3][q]);
        ctl->alpha[q] = !final_out ? 1.f : L == 0.f ? 0.f : __frcp_rn(L);  // (no row: zeros)
        if (!final_out) {
          // (a query that is not finite: its NaN has to pass the merge, which skips runs without rows)
          p.ml[size_t(slot) * kQ + q] = make_float4(L != L ? INFINITY : ctl->m[q], L, __int_as_float(ctl->col_pos[q]), 0.f);
          if (q == 0) p.rec[slot] = Rec{1, s.b, s.g, s.t0, s.t1, s.tiles, s.row0, s.rows};
        }
      }
      soft_sync();
      if (!dead && nt > 0) {
        const int r0 = kDim - p.rope_dim, odd = lane & 1;
#pragma unroll 1
        for (int ct = 0; ct < kParts; ++ct) {
          // lane pairs swap, so that each lane has both channels ch, ch + 1 of every other column
          const int ch = 128 * ct + 32 * wq + lane - odd;
          uint32_t o[kCols];
          tmem_ld16(tmem + lane_base + kColO + kQ * ct + c0, o);
          tmem_wait_ld();
          float cs = 1.f, sn = 0.f;
          int pos = -1;
          const bool rot = final_out && ch >= r0;
          const double theta = rot ? p.rope.theta_pi[(ch - r0) >> 1] : 0.0;
#pragma unroll
          for (int jj = 0; jj < kCols / 2; ++jj) {
            const float va = __uint_as_float(o[2 * jj]), vb = __uint_as_float(o[2 * jj + 1]);
            const float got = __shfl_xor_sync(kFull, odd ? va : vb, 1);
            const int col = c0 + 2 * jj + odd;
            const float a = ctl->alpha[col];
            float x = odd ? got : va, y = odd ? vb : got;
            x = a == 0.f ? 0.f : x * a;
            y = a == 0.f ? 0.f : y * a;
            if (rot) {
              const int pc = ctl->col_pos[col];
              if (pc != pos) {
                pos = pc;
                rotation(theta, pos, &cs, &sn);
              }
              const float t = x;
              x = fmaf(t, cs, -y * sn);
              y = fmaf(t, sn, y * cs);
            }
            if (!final_out) {
              *reinterpret_cast<float2*>(p.o_part + (size_t(slot) * kQ + col) * kDim + ch) = make_float2(x, y);
            } else if (col < s.rows) {
              const size_t at = size_t(s.row0 + col) * kDim + ch;
              if (p.out_fp32) *reinterpret_cast<float2*>(static_cast<float*>(p.out) + at) = make_float2(x, y);
              else *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + at) = cvt_bf16x2(x, y);
            }
          }
        }
      }
    } else {
      // ---------------------------------------------------------- loaders
      const int lw = warp - kLoad0, r = 32 * lw + lane;
      bool ok = true;
#pragma unroll 1
      for (int i = 0; i < nt && ok; ++i) {
        const int T = s.t0 + i, c = cnt + i;
        int32_t rows2[2];
        if (!C::kQuant && T < s.full && tma_rows(p, s.b, T, rows2)) {
#pragma unroll 1
          for (int sp = 0; sp < kParts && ok; ++sp) {
            if (c > 0) ok = warp_wait(&ctl->empty[sp], (c - 1) & 1, abort, lane);
            if (ok && lane == 0) {
              if (sp == 0) ctl->ok[c & 1][lw] = kFull;
              mbar_arrive(&ctl->full[sp]);
            }
          }
          continue;
        }
        int64_t row;
        const Rows* src = row_source(p, s, T, r, &row);
        const uint8_t* my = src ? src->codes + size_t(row) * row_bytes(FMT) : nullptr;
        const uint32_t have = __ballot_sync(kFull, src != nullptr);
        if constexpr (!C::kQuant) {
#pragma unroll 1
          for (int sp = 0; sp < kParts && ok; ++sp) {
            if (c > 0) ok = warp_wait(&ctl->empty[sp], (c - 1) & 1, abort, lane);
            if (!ok) break;
            if (sp == 0 && lane == 0) ctl->ok[c & 1][lw] = have;
#pragma unroll 4
            for (int x = 0; x < 16; ++x) {  // 16 lanes a row of the pair's 256 bytes
              const int rl = 2 * x + (lane >> 4), ch = 128 * sp + 8 * (lane & 15);
              const uint8_t* g = reinterpret_cast<const uint8_t*>(shfl_ptr(my, rl));
              cp_async16_zfill(cell(sR, 32 * lw + rl, ch), g ? g + 2 * ch : p.draft.codes, g ? 16 : 0);
            }
            cp_async_commit();
          }
          if (!ok) {
            cp_async_wait_group<0>();
            break;
          }
          auto hand = [&](int sp) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->full[sp]);
          };
          cp_async_wait_group<3>();
          hand(0);
          cp_async_wait_group<2>();
          hand(1);
          cp_async_wait_group<1>();
          hand(2);
          cp_async_wait_group<0>();
          hand(3);
        } else {
          float my_scale = 0.f;
          const uint8_t* mysc = nullptr;
          if (C::kRowScale && src) my_scale = static_cast<const float*>(src->scales)[row];
          if (FMT == DSV4KV_FP4_E2M1_G16 && src)
            mysc = static_cast<const uint8_t*>(src->scales) + size_t(row) * (kDim / 16);
          const float my_inv = my_scale > 0.f ? __frcp_rn(my_scale) : 0.f;
          using Part = QuantPart<FMT>;
          Part part[2];
          part[0].fetch(my, mysc, 0, lane);
#pragma unroll
          for (int k = 0; k < Part::kCount; ++k) {
            const int sp = min(k, kParts - 1);
            if (k + 1 < Part::kCount) part[(k + 1) & 1].fetch(my, mysc, k + 1, lane);
            if (ok && c > 0 && k < kParts) ok = warp_wait(&ctl->empty[sp], (c - 1) & 1, abort, lane);
            if (ok) {
              if (k == 0) {
                if (lane == 0) ctl->ok[c & 1][lw] = have;
                if (C::kRowScale) ctl->scale[c & 1][r] = my_scale;
              }
              part[k & 1].put(sR, lw, k, my_inv, lane);
              if (k < kParts - 1 || k == Part::kCount - 1) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->full[sp]);
              }
            }
          }
        }
      }
    }
    cnt += nt;
    ++segs;
    if (whole) {
      g_next += P;
    } else {
      left -= s.t1 - s.t0;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (ctl->abort) break;
    // ---- the next part
    if (whole) {
      for (int b = tid; b < p.batch; b += kThreads)
        if (ctl->gpre[b] <= g_next && g_next < ctl->gpre[b + 1]) {
          ctl->b = b;
          ctl->g = g_next - ctl->gpre[b];
          ctl->t0 = 0;
        }
    } else if (tid == 0 && left > 0) {
      int b = s.b, g = s.g + 1;
      while (b < p.batch && g >= ctl->gpre[b + 1] - ctl->gpre[b]) {
        ++b;
        g = 0;
      }
      ctl->b = b;
      ctl->g = g;
      ctl->t0 = 0;
    }
    __syncthreads();
  }
  __syncthreads();
  if (tid == 0 && ctl->abort) set_status(p.status, DSV4KV_DEV_TIMEOUT);
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

// Merges the partial sums of the group whose first run ends in CTA blockIdx.x / 8
// (nothing to do when it did not cut one): 8 blocks a group, one warp a query row.
__global__ void __launch_bounds__(256) tree_combine(const __grid_constant__ Params p, int P) {
  const int c = blockIdx.x >> 3, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int j = (blockIdx.x & 7) * 8 + warp;
  pdl_trigger();
  pdl_wait();
  const Rec own = p.rec[2 * c + 1];
  if (!own.valid || j >= own.rows) return;
  // the runs behind it: first slots of the next CTAs, until one ends the group
  float M = kNoMax;
  int last = c;
  {
    int end = own.t1;
    while (end < own.tiles && last + 1 < P) {
      const Rec r = p.rec[2 * (last + 1)];
      if (!r.valid || r.b != own.b || r.g != own.g) {  // (a run that timed out)
        if (lane == 0) set_status(p.status, DSV4KV_DEV_INCONSISTENT);
        return;
      }
      end = r.t1;
      ++last;
    }
  }
  for (int x = c; x <= last; ++x) M = fmaxf(M, p.ml[size_t(x == c ? 2 * c + 1 : 2 * x) * kQ + j].x);
  float L = 0.f;
  float4 o[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) o[q] = make_float4(0.f, 0.f, 0.f, 0.f);
  const int pos = __float_as_int(p.ml[size_t(2 * c + 1) * kQ + j].z);
  for (int x = c; x <= last; ++x) {
    const size_t slot = x == c ? 2 * c + 1 : 2 * x;
    const float4 ml = p.ml[slot * kQ + j];
    if (ml.y == 0.f) continue;  // it saw no row (its O may be unwritten)
    const float w = exp2_approx(ml.x - M);
    L = fmaf(w, ml.y, L);
    const float4* src = reinterpret_cast<const float4*>(p.o_part + (slot * kQ + j) * kDim) + lane;
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
        rope_rotation(p.rope.theta_pi[(ch + e - r0) >> 1], -double(pos), &cs, &sn);
        const float a = v[e], b = v[e + 1];
        v[e] = fmaf(a, cs, -b * sn);
        v[e + 1] = fmaf(a, sn, b * cs);
      }
    const size_t at = size_t(own.row0 + j) * kDim + ch;
    if (p.out_fp32) *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(v[0], v[1], v[2], v[3]);
    else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) = make_uint2(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]));
  }
}

// CTAs that a call launches: at most one a tile.
int grid_of(int batch, int heads, int max_nodes, int64_t nodes, int64_t t_max, int window, int stride, int k) {
  const int64_t n = t_max + max_nodes > window ? (t_max + max_nodes - window) / stride : 0;
  const int64_t rows = (k > 0 ? std::min<int64_t>(n, k) : n) + std::min<int64_t>(t_max, window) + max_nodes;
  const int64_t tiles = rows / kRows + 2;
  const int64_t groups = k > 0 ? nodes * ((heads + kQ - 1) / kQ) : nodes * heads / kQ + batch;
  const int sms = sm_count();
  return groups >= sms ? sms : int(std::max<int64_t>(1, std::min<int64_t>(sms, groups * tiles)));
}

struct Layout {
  size_t rec, ml, o, total;
};
Layout layout(int P) {
  Layout l;
  l.rec = 256;
  l.ml = l.rec + (size_t(2) * P * sizeof(Rec) + 255) / 256 * 256;
  l.o = l.ml + size_t(2) * P * kQ * sizeof(float4);
  l.total = l.o + size_t(2) * P * kQ * kDim * sizeof(float);
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
  return launch_pdl(tree_kernel<FMT>, dim3(unsigned(P)), dim3(kThreads), kSmemBytes, stream, tq, tc, p);
}

Rows rows_of(const dsv4kv_cache& c, const PageDesc& pg) {
  return Rows{pg.table, pg.page_rows, pg.table_stride, pg.pool_pages, static_cast<const uint8_t*>(c.codes), c.scales};
}

}  // namespace

size_t tree_ws_bytes(int batch, int heads, int max_nodes, int64_t nodes, int64_t t_max, int window, int stride, int k) {
  return layout(grid_of(batch, heads, max_nodes, nodes, t_max, window, stride, k)).total;
}

dsv4kv_status tree_decode_launch(const TreeArgs& a, void* ws, cudaStream_t stream) {
  const int P = grid_of(a.batch, a.heads, a.max_nodes, a.nodes, a.t_max, a.window, a.stride, a.idx ? a.k : 0);
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
  CUtensorMap tq{}, tc{};
  if (!encode_tmap_2d(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.q, kDim, uint64_t(a.nodes) * a.heads, kDim * 2, 64, kQ,
                      CU_TENSOR_MAP_SWIZZLE_128B))
    return set_error(DSV4KV_ERR_CUDA, "tree_decode_paged: tensor map of q");
  if (a.comp.fmt == DSV4KV_BF16 && a.comp.codes &&
      !encode_tmap_2d(&tc, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.comp.codes, kDim, uint64_t(a.comp.rows), kDim * 2, 64, 64,
                      CU_TENSOR_MAP_SWIZZLE_128B))
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
  if (P > 1) launch_pdl(tree_combine, dim3(unsigned(8 * P)), dim3(256), 0, stream, p, P);
  return check_launch("tree_combine");
}

}  // namespace dsv4kv
