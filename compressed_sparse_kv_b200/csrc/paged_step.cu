// The cache side of a paged serving step: block tables, slot maps, and the
// append of a ragged batch's new tokens ([P1] hybrid KV cache manager
// paragraph: blocks of a shared pool; "compressor-state blocks").
//
// block_table_kernel.  With pages(t) = ceil(rows(t) / page_rows), sequence b
// gives back entries [pages(t_new), pages(t_old)) of its table row or takes
// A_b = max(0, pages(t_new) - pages(t_old)) pages.  The G pages among the entries
// given back are pushed on the free stack in (b, entry) order, then A = sum A_b are
// popped in (b, entry) order: taken page a is element count + G - 1 - a of the
// grown stack.  An element past the old count is read where it comes from, in a
// shrinking sequence's table row, so pushes and pops need no order between them
// and one launch does both: every CTA forms the prefix sums over the batch
// (passes of warp scans in shared memory) and takes a share of the pages.
// The count is read by every CTA and written by the last one to finish, so
// that it may be updated in place; where some entries given back hold no page, that
// CTA repeats the work with the others' ranks counted out.
//
// slot_map_kernel.  Every CTA forms the prefix sums of the new tokens, then a
// thread finds the sequence of its first token by binary search and walks on;
// 4 tokens a thread, 16-byte stores.
//
// (Times here are of a replayed graph of ten calls; one after another, calls of
// a few us are bound by the host, the prompts take 3 to 4 us more.)  48 prompts of
// up to 65,536 tokens, about 1.7 M in all: tables and map 18.5 us for 35 MB, bound by
// start-up and searches; a decode step of 32 sequences: 7.2 us, two launches'
// latency.  Plain integer divisions in the map: 1.8 and 0.8 us more.
//
// append_paged_kernel (entries of up to 32 taps).  A CTA of 8 warps takes `per`
// consecutive tokens.  It lists the tokens whose row stays in a ring and those
// that emit an entry; a warp copies / rotates one row or sums one entry
// (16 channels a lane, the weights in shared memory, packed fp32 multiply-adds).
// Whole prompts are bound by the latency of the rows' reads at 16 warps an SM: 75,000
// tokens of c4a, 96 MB, in 31 us (3.1 TB/s, its second launch included); a step
// of 32 sequences x 8 tokens, 5.3 us, is latency.  Taps loaded one address at
// a time and scalar multiply-adds: 38 us; 3 CTAs an SM at 80 registers: 42.
//
// append_long_kernel (more taps, c128a).  Every state row is read once but the
// weights, 2 KB a tap, would be read again for each entry; so a cluster of 8 CTAs
// shares the entries of its tokens, CTA r keeping the weights of taps
// [16 r, 16 r + 16) in registers (two channels a thread).  An entry's 16 rows are
// one bulk copy (four entries in flight), the CTAs' sums of 8 entries are
// exchanged through distributed shared memory, and a ninth warp of each CTA
// adds up and stores one of them while the others go on.  110,000 tokens of
// c128a, 124 MB, take 43 us (2.9 TB/s; one CTA an entry with its weights from L2:
// 51), a step of 61 sequences 8.6 us (12.0).
//
// Entries read rows of the raw ring that tokens of the
// same call replace when a sequence has more than lookahead + 1 new ones
// (entry taps reach back to p + 1 + lookahead - (window + k_taps), the row
// replaced by token p' is p' - (window + k_taps)); the ring
// (and the window, whose rows are the last ones too) is then written by a
// second launch, append_rows_kernel, one warp a row (5 us of the prompts' times).
#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "internal.h"
#include "quant_row.cuh"

namespace dsv4kv {

namespace {

constexpr int kTabThreads = 512;
constexpr int kSlotThreads = 256;
constexpr int kSlotPer = 4;  // tokens a thread

// Exclusive prefix sums of f(b), b in [0, batch), into pre[0 .. batch] by all NT
// threads; f packs two counts (low and high half), whose sums stay below 2^32.
template <int NT, class F, class S>
__device__ __forceinline__ uint64_t block_prefix(int batch, F f, S store) {
  __shared__ uint64_t wsum[NT / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint64_t carry = 0;
  for (int b0 = 0; b0 < batch; b0 += NT) {
    const int b = b0 + int(threadIdx.x);
    const uint64_t v = b < batch ? f(b) : 0;
    uint64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t y = __shfl_up_sync(kFull, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) wsum[warp] = x;
    __syncthreads();
    uint64_t before = carry, all = carry;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) {
      if (i < warp) before += wsum[i];
      all += wsum[i];
    }
    if (b < batch) store(b, before + x - v);
    carry = all;
    __syncthreads();
  }
  return carry;
}

__device__ __forceinline__ int64_t clamp_len(int64_t t, int64_t t_max, uint32_t* status) {
  if (t >= 0 && t <= t_max) return t;
  set_status(status, DSV4KV_DEV_BAD_LENGTH);
  return t < 0 ? 0 : t_max;
}

// What a thread of block_table_kernel met: an entry without a page, a stack without one or without room, a bad page number.
enum : uint32_t { kGap = 1, kNoRoom = 2, kBad = 4 };

struct TableParams {
  const int64_t *t_old, *t_new;
  int batch;
  int64_t t_max;
  int window, stride, lookahead, page_rows;
  int32_t* table;
  int table_stride;
  int64_t pool_pages;
  int32_t* free_pages;
  int64_t free_cap;
  const int64_t* free_count;
  int64_t* free_count_out;
  uint32_t* status;  // workspace: status word, then the count of finished CTAs
};

__device__ __forceinline__ int pages_of(const TableParams& p, int64_t t) {
  const int x = int(t);  // t_max + lookahead < 2^31
  const int rows = p.stride == 0 ? min(x, p.window) : max(0, x + p.lookahead - p.window) / p.stride;
  return int((unsigned(rows) + unsigned(p.page_rows) - 1) / unsigned(p.page_rows));
}

__global__ void __launch_bounds__(kTabThreads) block_table_kernel(const TableParams p) {
  extern __shared__ int32_t sm[];
  int32_t *back = sm, *take = back + p.batch + 1;          // prefix sums of the entries given back / taken
  int32_t *first = take + p.batch + 1, *good = first + p.batch + 1;  // a sequence's first such entry; see below
  __shared__ uint32_t seen;
  __shared__ bool again;
  pdl_trigger();
  if (threadIdx.x == 0) seen = 0;
  pdl_wait();
  int64_t count = *p.free_count;
  if (count < 0 || count > p.free_cap) {
    set_status(p.status, DSV4KV_DEV_BAD_LENGTH);
    count = count < 0 ? 0 : p.free_cap;
  }
  const uint64_t sums = block_prefix<kTabThreads>(
      p.batch,
      [&](int b) -> uint64_t {
        const int o = pages_of(p, clamp_len(p.t_old[b], p.t_max, p.status));
        const int n = pages_of(p, clamp_len(p.t_new[b], p.t_max, p.status));
        first[b] = min(o, n);
        return o > n ? uint64_t(o - n) : uint64_t(n - o) << 32;
      },
      [&](int b, uint64_t v) {
        back[b] = int32_t(v & 0xffffffffu);
        take[b] = int32_t(v >> 32);
      });
  const int G = int(sums & 0xffffffffu), A = int(sums >> 32);
  if (threadIdx.x == 0) back[p.batch] = G;
  __syncthreads();
  auto entry = [&](int b, int j) { return p.table[size_t(b) * p.table_stride + first[b] + j]; };
  auto is_page = [&](int32_t pg) { return pg >= 0 && pg < p.pool_pages; };
  // The pushes and pops of threads begin, begin + step, ..; `pages` of the G entries given back hold one: all of them, or
  // (gaps) those that the prefix sums good[] count.  Returns what it met.
  auto move_pages = [&](int begin, int step, bool gaps, int pages) -> uint32_t {
    uint32_t met = 0;
    auto whole = [&](int b) { return !gaps || good[b + 1] - good[b] == back[b + 1] - back[b]; };
    auto given = [&](int r) -> int32_t {  // page r of those given back
      const int b = find_seq(gaps ? good : back, p.batch, r);
      int j = r - (gaps ? good[b] : back[b]);
      if (!whole(b)) {
        int k = j;
        for (j = 0; !is_page(entry(b, j)) || k-- > 0;) ++j;  // (ends: the sequence gives back more than k pages)
      }
      return entry(b, j);
    };
    for (int x = begin; x < G; x += step) {
      const int b = find_seq(back, p.batch, x), j = x - back[b];
      const int32_t pg = entry(b, j);
      if (!is_page(pg)) {
        met |= pg == -1 ? kGap : kGap | kBad;
        continue;
      }
      int r = x;
      if (gaps) {
        r = good[b] + j;
        if (!whole(b))
          for (int i = 0; i < j; ++i) r -= !is_page(entry(b, i));
      }
      if (count + r < p.free_cap) p.free_pages[count + r] = pg;
      else met |= kNoRoom;
    }
    const int64_t top = min(count + pages, p.free_cap);  // the grown stack
    for (int a = begin; a < A; a += step) {
      const int b = find_seq(take, p.batch, a);
      const int64_t at = top - 1 - a;
      int32_t pg = -1;
      if (at < 0) {
        met |= kNoRoom;
      } else {
        pg = at >= count ? given(int(at - count)) : p.free_pages[at];
        if (!is_page(pg)) {
          met |= kBad;
          pg = -1;
        }
      }
      p.table[size_t(b) * p.table_stride + first[b] + (a - take[b])] = pg;
    }
    return met;
  };
  uint32_t met = move_pages(blockIdx.x * kTabThreads + int(threadIdx.x), gridDim.x * kTabThreads, false, G);
  if (met) atomicOr(&seen, met);
  __syncthreads();
  auto finish = [&](uint32_t flags, int pages) {
    if (flags & kNoRoom) set_status(p.status, DSV4KV_DEV_NO_PAGES);
    if (flags & kBad) set_status(p.status, DSV4KV_DEV_BAD_PAGE);
    *p.free_count_out = max(int64_t(0), min(count + pages, p.free_cap) - A);
  };
  // The last CTA to get here (every CTA has read the count) writes it, and the flags of all (a byte of the counter each).
  if (threadIdx.x == 0) {
    __threadfence();
    uint32_t* done = p.status + 1;
    const uint32_t own = 1u + (seen & kGap ? 0x100u : 0u) + (seen & kNoRoom ? 0x10000u : 0u) + (seen & kBad ? 0x1000000u : 0u);
    const uint32_t all = atomicAdd(done, own) + own;
    again = false;
    if ((all & 0xffu) == gridDim.x) {
      *done = 0;
      again = (all & 0xff00u) != 0;
      if (!again) finish((all & 0xff0000u ? kNoRoom : 0u) | (all & 0xff000000u ? kBad : 0u), G);
    }
  }
  __syncthreads();
  if (!again) return;
  // Some entries held no page (the stack had none left when they were taken) and belong not on it: the CTA does all
  // pushes and pops again with the others counted out.  What was written so far lies above the old stack and in the
  // entries taken, none of it read.
  __threadfence();
  for (int b = threadIdx.x; b < p.batch; b += kTabThreads) good[b] = 0;
  if (threadIdx.x == 0) seen = 0;
  __syncthreads();
  for (int x = threadIdx.x; x < G; x += kTabThreads) {
    const int b = find_seq(back, p.batch, x);
    if (is_page(entry(b, x - back[b]))) atomicAdd(&good[b], 1);
  }
  __syncthreads();
  const int pages = int(block_prefix<kTabThreads>(
      p.batch, [&](int b) -> uint64_t { return uint64_t(good[b]); }, [&](int b, uint64_t v) { good[b] = int32_t(v); }));
  if (threadIdx.x == 0) good[p.batch] = pages;
  __syncthreads();
  met = move_pages(threadIdx.x, kTabThreads, true, pages);
  if (met) atomicOr(&seen, met);
  __syncthreads();
  if (threadIdx.x == 0) finish(seen, pages);
}

// Quotients by a divisor of the whole call: floor(n / d) is the high word of n * (floor((2^64 - 1) / d) + 1) for all 32-bit
// n and d > 1 (Lemire, Kaser and Kurz, "Faster remainder by direct computation", 2019).
struct Div {
  uint64_t m;
  int d;
  explicit Div(int by) : m(by > 1 ? ~uint64_t(0) / uint64_t(by) + 1 : 0), d(by) {}
  __device__ __forceinline__ int quot(int n) const { return d == 1 ? n : int(__umul64hi(m, uint64_t(uint32_t(n)))); }
};

struct SlotParams {
  const int64_t *t_old, *t_new;
  int batch;
  int64_t t_max;
  int window, stride, lookahead;
  PageDesc comp, win;
  int capacity;
  int32_t *cu, *seq;
  int64_t* pos;
  int32_t *win_slot, *comp_slot;
  uint32_t* status;
  Div by_window, by_stride, by_comp, by_win;  // window (1 without one), stride, rows a page
};

__device__ __forceinline__ int32_t slot_of(const PageDesc& d, const Div& by, int b, int row, uint32_t* status) {
  const int page = by.quot(row);
  const int32_t pg = __ldg(d.table + size_t(b) * d.table_stride + page);
  if (pg < 0 || pg >= d.pool_pages) {
    set_status(status, DSV4KV_DEV_BAD_PAGE);
    return -1;
  }
  return pg * d.page_rows + (row - page * d.page_rows);  // pool rows < 2^31
}

__global__ void __launch_bounds__(kSlotThreads) slot_map_kernel(const SlotParams p) {
  extern __shared__ int32_t pre[];  // first token of every sequence, clamped to the capacity; its old and new length
  int32_t *old_len = pre + p.batch + 1, *new_len = old_len + p.batch;
  pdl_trigger();
  pdl_wait();
  const uint64_t sum = block_prefix<kSlotThreads>(
      p.batch,
      [&](int b) -> uint64_t {
        const int64_t o = clamp_len(p.t_old[b], p.t_max, p.status), n = clamp_len(p.t_new[b], p.t_max, p.status);
        old_len[b] = int32_t(o);
        new_len[b] = int32_t(n);
        return uint64_t(max(int64_t(0), n - o));
      },
      [&](int b, uint64_t v) {
        pre[b] = int32_t(min(v, uint64_t(p.capacity)));
        if (blockIdx.x == 0) p.cu[b] = pre[b];
      });
  const int total = int(min(sum, uint64_t(p.capacity)));
  if (threadIdx.x == 0) {
    pre[p.batch] = total;
    if (blockIdx.x == 0) {
      p.cu[p.batch] = total;
      if (sum > uint64_t(p.capacity)) set_status(p.status, DSV4KV_DEV_BAD_LENGTH);
    }
  }
  __syncthreads();
  const int64_t stepw = int64_t(gridDim.x) * kSlotThreads * kSlotPer;
  for (int64_t i0 = (int64_t(blockIdx.x) * kSlotThreads + threadIdx.x) * kSlotPer; i0 < p.capacity; i0 += stepw) {
    int32_t sq[kSlotPer], ws[kSlotPer], cs[kSlotPer];
    int64_t ps[kSlotPer];
    int b = i0 < total ? find_seq(pre, p.batch, int(i0)) : 0;
    int o = 0, n = 0, of = -1;
#pragma unroll
    for (int e = 0; e < kSlotPer; ++e) {
      const int i = int(i0) + e;
      sq[e] = ws[e] = cs[e] = -1;
      ps[e] = -1;
      if (i >= total) continue;
      while (pre[b + 1] <= i) ++b;  // (ends: i < pre[batch])
      if (of != b) {
        o = old_len[b];
        n = new_len[b];
        of = b;
      }
      const int pp = o + (i - pre[b]);
      sq[e] = b;
      ps[e] = pp;
      if (p.win.table && pp >= n - p.window) ws[e] = slot_of(p.win, p.by_win, b, pp - p.by_window.quot(pp) * p.window, p.status);
      const int r = pp + 1 + p.lookahead - p.window;  // the entry ends when it is a multiple of the stride
      if (p.comp.table && r > 0) {
        const int n_e = p.by_stride.quot(r);
        if (n_e * p.stride == r) cs[e] = slot_of(p.comp, p.by_comp, b, n_e - 1, p.status);
      }
    }
    if (i0 + kSlotPer <= p.capacity) {
      *reinterpret_cast<int4*>(p.seq + i0) = make_int4(sq[0], sq[1], sq[2], sq[3]);
      *reinterpret_cast<longlong2*>(p.pos + i0) = make_longlong2(ps[0], ps[1]);
      *reinterpret_cast<longlong2*>(p.pos + i0 + 2) = make_longlong2(ps[2], ps[3]);
      *reinterpret_cast<int4*>(p.win_slot + i0) = make_int4(ws[0], ws[1], ws[2], ws[3]);
      *reinterpret_cast<int4*>(p.comp_slot + i0) = make_int4(cs[0], cs[1], cs[2], cs[3]);
    } else {
#pragma unroll
      for (int e = 0; e < kSlotPer; ++e) {
        if (i0 + e >= p.capacity) break;
        p.seq[i0 + e] = sq[e];
        p.pos[i0 + e] = ps[e];
        p.win_slot[i0 + e] = ws[e];
        p.comp_slot[i0 + e] = cs[e];
      }
    }
  }
}

// ------------------------------------------------------------------ append
constexpr int kAppWarps = 8;
constexpr int kAppThreads = 32 * kAppWarps;
constexpr int kD = 512, kPer = kD / 32;
constexpr int kMaxTokens = 512;  // tokens a CTA
constexpr int kLongTaps = 32;    // entries of more taps are summed by a cluster

enum : int { kPartEntries = 1, kPartWindow = 2, kPartRing = 4 };

struct AppendParams {
  const uint16_t* s_new;
  const float* w;
  int batch;
  int tokens, per;  // packed tokens (capacity), tokens a CTA
  const int32_t *cu, *seq;
  const int64_t* pos;
  const int32_t *win_slot, *comp_slot;
  int k_taps, stride, window, lookahead, max_new, rope_dim, parts;
  uint16_t* ring;
  uint8_t *win_codes, *comp_codes;
  void *win_scales, *comp_scales;
  int64_t win_rows, comp_rows;  // pool rows
  uint32_t* status;
  RopeTable rope;
};

struct Tok {
  int i, b, pos, first, slot;  // token, sequence, position, the sequence's first new token, its entry's pool row
};

// A lane holds channels [8 lane, 8 lane + 8) and [256 + 8 lane, ..) of a row, so that every load of it (and store of a
// bf16 row) is one contiguous 512-byte piece; the quantisers want channels [16 lane, 16 lane + 16).
__device__ __forceinline__ void to_consecutive(const float (&x)[kPer], float (&y)[kPer], int lane) {
  const int from = (2 * lane) & 31;  // the lane that holds 8-channel pieces 2 lane (2 lane + 1: the next one)
  const bool upper = lane >= 16;     // of the upper 256 channels
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float a0 = __shfl_sync(kFull, x[e], from), a1 = __shfl_sync(kFull, x[8 + e], from);
    const float b0 = __shfl_sync(kFull, x[e], from + 1), b1 = __shfl_sync(kFull, x[8 + e], from + 1);
    y[e] = upper ? a1 : a0;
    y[8 + e] = upper ? b1 : b0;
  }
}

// Rotates a row's rotary pairs at pos.  theta: pair `lane`'s theta / pi (where there are at most 32 pairs).
__device__ __forceinline__ void rotate_row(float (&x)[kPer], const AppendParams& p, double theta, int pos, int lane) {
  const int r0 = kD - p.rope_dim, pairs = p.rope_dim / 2;
  if (pairs <= 32) {
    // lane m computes pair m; the lanes that own rotary channels (of the second piece) fetch theirs
    float cs_m = 1.f, sn_m = 0.f;
    if (lane < pairs) rope_rotation(theta, double(pos), &cs_m, &sn_m);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const int m = (256 + 8 * lane + e - r0) >> 1;
      const float cs = __shfl_sync(kFull, cs_m, m & 31), sn = __shfl_sync(kFull, sn_m, m & 31);
      if (m >= 0) {
        const float a = x[8 + e], b = x[9 + e];
        x[8 + e] = a * cs - b * sn;
        x[9 + e] = a * sn + b * cs;
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < kPer; e += 2) {
      const int m = ((e < 8 ? 8 * lane + e : 248 + 8 * lane + e) - r0) >> 1;
      if (m >= 0) {
        float cs, sn;
        rope_rotation(p.rope.theta_pi[m], double(pos), &cs, &sn);
        const float a = x[e], b = x[e + 1];
        x[e] = a * cs - b * sn;
        x[e + 1] = a * sn + b * cs;
      }
    }
  }
}

template <int FMT>
__device__ __forceinline__ void store_row(const float (&x)[kPer], int lane, int64_t row, uint8_t* codes, void* scales) {
  if constexpr (FMT == DSV4KV_BF16) {
    uint16_t* dst = reinterpret_cast<uint16_t*>(codes) + size_t(row) * kD + 8 * lane;
#pragma unroll
    for (int q = 0; q < 2; ++q)
      *reinterpret_cast<uint4*>(dst + 256 * q) =
          make_uint4(pack_bf16x2(x[8 * q], x[8 * q + 1]), pack_bf16x2(x[8 * q + 2], x[8 * q + 3]),
                     pack_bf16x2(x[8 * q + 4], x[8 * q + 5]), pack_bf16x2(x[8 * q + 6], x[8 * q + 7]));
  } else {
    float y[kPer];
    to_consecutive(x, y, lane);
    quantize_row<kPer, FMT>(y, lane, size_t(row), codes, scales);
  }
}

__device__ __forceinline__ void unpack8(const uint4& v, float* x) {
  x[0] = bf16lo(v.x); x[1] = bf16hi(v.x);
  x[2] = bf16lo(v.y); x[3] = bf16hi(v.y);
  x[4] = bf16lo(v.z); x[5] = bf16hi(v.z);
  x[6] = bf16lo(v.w); x[7] = bf16hi(v.w);
}

// The state row of position q of token k's sequence: a new token's or the raw ring's (this lane's first piece).
__device__ __forceinline__ const uint16_t* state_row(const AppendParams& p, const Tok& k, int q, int lane) {
  const int i = k.i - (k.pos - q);
  if (i >= k.first) return p.s_new + size_t(i) * kD + 8 * lane;
  const int R = p.window + p.k_taps;
  return p.ring + (size_t(k.b) * R + q % R) * kD + 8 * lane;
}
__device__ __forceinline__ uint4 first_piece(const uint16_t* row) { return *reinterpret_cast<const uint4*>(row); }
__device__ __forceinline__ uint4 second_piece(const uint16_t* row) { return *reinterpret_cast<const uint4*>(row + 256); }

// Sums of channel pairs: one packed fused multiply-add (each half rounded as fmaf rounds) for two channels.
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 pair_value(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ void add2(uint64_t& acc, uint64_t w, uint32_t v) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(w), "l"(pair_of(bf16lo(v), bf16hi(v))));
}
__device__ __forceinline__ void add8(uint64_t* acc, const ulonglong2& w0, const ulonglong2& w1, const uint4& v) {
  add2(acc[0], w0.x, v.x);
  add2(acc[1], w0.y, v.y);
  add2(acc[2], w1.x, v.z);
  add2(acc[3], w1.y, v.w);
}
__device__ __forceinline__ void sums_of(const uint64_t (&acc)[kPer / 2], float (&x)[kPer]) {
#pragma unroll
  for (int e = 0; e < kPer / 2; ++e) {
    const float2 v = pair_value(acc[e]);
    x[2 * e] = v.x;
    x[2 * e + 1] = v.y;
  }
}

__device__ __forceinline__ void app_sync() {  // the 8 working warps (a long entry's CTA has a ninth)
  asm volatile("barrier.cta.sync 1, %0;" ::"n"(kAppThreads) : "memory");
}

// Appends i to list[n ..] where `keep`, in thread order; returns the new length.  The 8 working warps call it.
__device__ __forceinline__ int push_ordered(bool keep, int i, int32_t* list, int n, int* wcnt) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned m = __ballot_sync(kFull, keep);
  if (lane == 0) wcnt[warp] = __popc(m);
  app_sync();
  int before = n, all = n;
#pragma unroll
  for (int k = 0; k < kAppWarps; ++k) {
    if (k < warp) before += wcnt[k];
    all += wcnt[k];
  }
  if (keep) list[before + __popc(m & ((1u << lane) - 1u))] = i;
  app_sync();
  return all;
}

// A token of a list.
__device__ __forceinline__ Tok token(const AppendParams& p, int i) {
  const int b = __ldg(p.seq + i);
  const int pos = int(__ldg(p.pos + i)), slot = __ldg(p.comp_slot + i);
  return Tok{i, b, pos, __ldg(p.cu + b), slot};
}

// Lists the CTA's tokens whose row stays and those that emit an entry, in order; (rows, entries) counted.
__device__ __forceinline__ int2 list_tokens(const AppendParams& p, int32_t* rows, int32_t* ents, int* wcnt) {
  const int i_first = int(blockIdx.x) * p.per, i_end = min(p.tokens, i_first + p.per), R = p.window + p.k_taps;
  int n_rows = 0, n_ents = 0;
  for (int i0 = i_first; i0 < i_end; i0 += kAppThreads) {
    const int i = i0 + int(threadIdx.x);
    bool row = false, ent = false;
    if (i < i_end) {
      const int b = p.seq[i];
      if (b >= 0 && b < p.batch) {
        const int c0 = p.cu[b], c1 = p.cu[b + 1];
        const int64_t pos = p.pos[i];
        const int ws = p.win_slot[i], cs = p.comp_slot[i];
        if (i < c0 || i >= c1 || c0 < 0 || c1 > p.tokens || c1 - c0 > p.max_new || pos < i - c0 || pos >= (int64_t(1) << 31) - p.lookahead - 1) {
          set_status(p.status, DSV4KV_DEV_BAD_LENGTH);
        } else {
          if (ws >= p.win_rows || cs >= p.comp_rows) set_status(p.status, DSV4KV_DEV_BAD_PAGE);
          row = ((p.parts & kPartWindow) && ws >= 0 && ws < p.win_rows) || ((p.parts & kPartRing) && c1 - 1 - i < R);
          ent = (p.parts & kPartEntries) && cs >= 0 && cs < p.comp_rows;
          if (ent && pos + 1 + p.lookahead - p.window < p.stride) {  // no entry ends here
            set_status(p.status, DSV4KV_DEV_BAD_LENGTH);
            ent = false;
          }
        }
      } else if (b != -1) {
        set_status(p.status, DSV4KV_DEV_BAD_LENGTH);
      }
    }
    n_rows = push_ordered(row, i, rows, n_rows, wcnt);
    n_ents = push_ordered(ent, i, ents, n_ents, wcnt);
  }
  return make_int2(n_rows, n_ents);
}

// Ring and window rows of the listed tokens, one warp a row.
template <int FMT>
__device__ __forceinline__ void write_rows(const AppendParams& p, const int32_t* rows, int n_rows, double theta) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, R = p.window + p.k_taps;
  for (int r = warp; r < n_rows; r += kAppWarps) {
    const Tok k = token(p, rows[r]);
    const uint16_t* src = p.s_new + size_t(k.i) * kD + 8 * lane;
    const uint4 v0 = first_piece(src), v1 = second_piece(src);
    if ((p.parts & kPartRing) && p.cu[k.b + 1] - 1 - k.i < R) {
      uint16_t* dst = p.ring + (size_t(k.b) * R + k.pos % R) * kD + 8 * lane;
      *reinterpret_cast<uint4*>(dst) = v0;
      *reinterpret_cast<uint4*>(dst + 256) = v1;
    }
    const int slot = p.win_slot[k.i];
    if ((p.parts & kPartWindow) && slot >= 0 && slot < p.win_rows) {
      float x[kPer];
      unpack8(v0, x);
      unpack8(v1, x + 8);
      rotate_row(x, p, theta, k.pos, lane);
      store_row<FMT>(x, lane, slot, p.win_codes, p.win_scales);
    }
  }
}

template <int FMT>
__global__ void __launch_bounds__(kAppThreads, 2) append_paged_kernel(const __grid_constant__ AppendParams p) {
  __shared__ int32_t rows[kMaxTokens], ents[kMaxTokens];
  __shared__ int wcnt[kAppWarps];
  extern __shared__ __align__(16) float weights[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const double theta = p.rope.theta_pi[lane];
  pdl_trigger();
  pdl_wait();
  const int2 n = list_tokens(p, rows, ents, wcnt);
  const int n_ents = n.y;
  write_rows<FMT>(p, rows, n.x, theta);
  if (n_ents == 0) return;
  // weights [tap][quarter][lane] float4: a lane's two pieces of 8 channels in four conflict-free reads
  ulonglong2* sw = reinterpret_cast<ulonglong2*>(weights);
  for (int i = threadIdx.x; i < p.k_taps * (kD / 4); i += kAppThreads) {
    const int j = i / (kD / 4), c = i % (kD / 4);  // quad c: lane (c / 2) % 32, quarter 2 (c / 64) + c % 2
    sw[(j * 4 + 2 * (c >> 6) + (c & 1)) * 32 + ((c >> 1) & 31)] = reinterpret_cast<const ulonglong2*>(p.w)[i];
  }
  __syncthreads();
  // consecutive entries to one warp: the rows that two entries share come from L1 the second time
  const int per = (n_ents + kAppWarps - 1) / kAppWarps, end = min(n_ents, (warp + 1) * per);
  Tok next = warp * per < end ? token(p, ents[warp * per]) : Tok{};
#pragma unroll 1
  for (int r = warp * per; r < end; ++r) {
    const Tok k = next;
    if (r + 1 < end) next = token(p, ents[r + 1]);
    const int q0 = k.pos + 1 + p.lookahead - p.window - p.k_taps;
    const int i0 = k.i - (k.pos - q0);  // the first tap's token
    uint64_t acc[kPer / 2];
#pragma unroll
    for (int e = 0; e < kPer / 2; ++e) acc[e] = 0;
    auto add = [&](int j, const uint4& a, const uint4& b) {
      const ulonglong2* w = sw + j * 128 + lane;
      add8(acc, w[0], w[32], a);
      add8(acc + 4, w[64], w[96], b);
    };
    int j0 = max(0, -q0);
    if (i0 >= k.first) {  // all taps are new tokens: consecutive rows
      const uint16_t* src = p.s_new + size_t(i0) * kD + 8 * lane;
#pragma unroll 2
      for (; j0 + 4 <= p.k_taps; j0 += 4) {
        uint4 a[4], b[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          a[x] = first_piece(src + (j0 + x) * kD);
          b[x] = second_piece(src + (j0 + x) * kD);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) add(j0 + x, a[x], b[x]);
      }
    }
#pragma unroll 1
    for (; j0 < p.k_taps; j0 += 4) {
      uint4 a[4], b[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if (j0 + x >= p.k_taps) break;
        const uint16_t* src = state_row(p, k, q0 + j0 + x, lane);
        a[x] = first_piece(src);
        b[x] = second_piece(src);
      }
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (j0 + x < p.k_taps) add(j0 + x, a[x], b[x]);
    }
    float x[kPer];
    sums_of(acc, x);
    rotate_row(x, p, theta, q0 + p.k_taps - p.stride, lane);
    store_row<FMT>(x, lane, k.slot, p.comp_codes, p.comp_scales);
  }
}

// Long entries: a cluster of 8 CTAs shares the entries of its CTAs' tokens; CTA r has taps [16 r, 16 r + 16) of each (of
// 128 at a time), whose weights stay in registers: a thread has two channels.
constexpr int kCl = 8;           // CTAs a cluster
constexpr int kRound = kCl;      // entries summed before the CTAs exchange their sums: one a CTA to finish
constexpr int kLongThreads = kAppThreads + 32;
constexpr int kTaps = 16;        // taps a CTA
constexpr int kStages = 4;       // entries' rows in flight
constexpr int kStageBytes = kTaps * kD * 2;
constexpr int kListed = kAppThreads;  // entries whose tokens are looked up at a time
constexpr size_t kLongSmem = kStages * kStageBytes + kRound * kD * sizeof(float);

struct LongCtl {
  uint64_t full[kStages];
  int n_of[kCl];  // entries of every CTA of the cluster
  volatile int dead;
  Tok toks[kListed];
};

__device__ __forceinline__ bool wait_rows(LongCtl* ctl, int st, uint32_t parity) {  // bounded: one second
  if (mbar_try_wait(&ctl->full[st], parity)) return true;
  uint64_t t0, t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t0));
  while (!ctl->dead) {
    if (mbar_try_wait(&ctl->full[st], parity)) return true;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    if (t - t0 > 1000000000ull) ctl->dead = 1;
  }
  return false;
}

template <int FMT>
__global__ void __launch_bounds__(kLongThreads, 2) append_long_kernel(const __grid_constant__ AppendParams p) {
  __shared__ int32_t rows[kMaxTokens], ents[kMaxTokens];
  __shared__ int wcnt[kAppWarps];
  __shared__ LongCtl ctl;
  extern __shared__ __align__(128) uint8_t stages[];
  float* part = reinterpret_cast<float*>(stages + kStages * kStageBytes);  // [CTA][512]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, rank = int(cluster_rank());
  const double theta = p.rope.theta_pi[lane];
  const int R = p.window + p.k_taps;
  const int tp = min(kTaps, (p.k_taps + kCl - 1) / kCl);  // taps a CTA has at a time
  const int chunks = (p.k_taps + kCl * tp - 1) / (kCl * tp);
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&ctl.full[s], 1);
    ctl.dead = 0;
    fence_mbar_init();
  }
  __syncwarp();
  cluster_arrive_relaxed();
  pdl_wait();
  int2 n = make_int2(0, 0);
  if (warp < kAppWarps) n = list_tokens(p, rows, ents, wcnt);
  __syncwarp();
  cluster_wait();
  if (tid < kCl) st_dsmem_u32(dsmem_addr(&ctl.n_of[rank], tid), uint32_t(n.y));
  __syncwarp();
  cluster_sync();
  int total = 0;
#pragma unroll
  for (int r = 0; r < kCl; ++r) total += ctl.n_of[r];
  if (warp == kAppWarps) {
    // the ninth warp adds up and stores this CTA's entry of every round, while the others sum the next round's
    for (int x0 = 0, round = 0; x0 < total; x0 += kListed)
      for (int r0 = 0; r0 < min(kListed, total - x0); r0 += kRound, ++round) {
        if (round) cluster_wait_acquire_div();
        cluster_arrive_release_div();
        cluster_wait_acquire_div();  // every CTA's sums are here
        if (rank < min(kRound, min(kListed, total - x0) - r0) && !ctl.dead) {
          float x[kPer];
#pragma unroll
          for (int y = 0; y < kPer; ++y) x[y] = 0.f;
#pragma unroll 1
          for (int c = 0; c < kCl; ++c)
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              const float4 v = *reinterpret_cast<const float4*>(part + c * kD + 256 * (h >> 1) + 8 * lane + 4 * (h & 1));
              x[4 * h] += v.x; x[4 * h + 1] += v.y; x[4 * h + 2] += v.z; x[4 * h + 3] += v.w;
            }
          const Tok k = ctl.toks[r0 + rank];
          rotate_row(x, p, theta, k.pos + 1 + p.lookahead - p.window - p.stride, lane);
          store_row<FMT>(x, lane, k.slot, p.comp_codes, p.comp_scales);
        }
        cluster_arrive_release_div();  // the sums' place is free
      }
    if (total) cluster_wait_acquire_div();
    return;
  }
  bool rows_done = false;
  int got = 0, put = 0, round = 0;  // stages consumed, issued (thread 0); rounds of entries
  uint64_t w[kTaps];
  for (int base = 0; base < total; base += kListed) {
    const bool again = base > 0;
    if (again) cluster_wait_acquire_div();  // (the tokens of the previous entries are read)
    app_sync();
    const int listed = min(kListed, total - base);
    if (tid < listed) {
      int r = 0, x = base + tid;
      while (x >= ctl.n_of[r]) x -= ctl.n_of[r++];
      ctl.toks[tid] = token(p, int(ld_dsmem_u32(dsmem_addr(&ents[x], r))));
    }
    app_sync();
    // (thread 0) the next slice of an entry's rows: from the raw ring (in two pieces where it wraps) and the new states
    int ir = 0, ic = 0, ie = 0;  // its round's first entry, chunk, entry within the round
    auto issue = [&]() {
      if (ir >= listed || ctl.dead) return;
      const Tok& k = ctl.toks[ir + ie];
      const int j0 = kCl * tp * ic + tp * rank;
      const int q = k.pos + 1 + p.lookahead - p.window - p.k_taps + j0;  // position of the slice's first tap
      const int lo = min(max(0, -q), tp), hi = max(lo, min(tp, p.k_taps - j0));
      const int fresh = min(max(k.first - (k.i - k.pos + q), lo), hi);   // first tap that is a new token
      uint8_t* dst = stages + (put % kStages) * kStageBytes;
      uint64_t* bar = &ctl.full[put % kStages];
      mbar_arrive_expect_tx(bar, uint32_t(hi - lo) * kD * 2);
      if (fresh > lo) {
        const int r0 = (q + lo) % R, a = min(fresh - lo, R - r0);
        const uint16_t* ring = p.ring + size_t(k.b) * R * kD;
        bulk_load_plain(dst + lo * kD * 2, ring + size_t(r0) * kD, uint32_t(a) * kD * 2, bar);
        if (fresh - lo > a) bulk_load_plain(dst + (lo + a) * kD * 2, ring, uint32_t(fresh - lo - a) * kD * 2, bar);
      }
      if (hi > fresh)
        bulk_load_plain(dst + fresh * kD * 2, p.s_new + size_t(k.i - k.pos + q + fresh) * kD, uint32_t(hi - fresh) * kD * 2,
                        bar);
      ++put;
      if (++ie == min(kRound, listed - ir)) {
        ie = 0;
        if (++ic == chunks) {
          ic = 0;
          ir += kRound;
        }
      }
    };
    if (tid == 0)
      for (int s = 0; s < kStages; ++s) issue();
    if (!rows_done) write_rows<FMT>(p, rows, n.x, theta);
    rows_done = true;
    for (int r0 = 0; r0 < listed; r0 += kRound, ++round) {
      const int ne = min(kRound, listed - r0);
      uint64_t acc[kRound];
#pragma unroll
      for (int e = 0; e < kRound; ++e) acc[e] = 0;
      for (int ch = 0; ch < chunks; ++ch) {
        const int j0 = kCl * tp * ch + tp * rank;
        if (chunks > 1 || round == 0) {
#pragma unroll
          for (int x = 0; x < kTaps; ++x)
            w[x] = x < tp && j0 + x < p.k_taps
                       ? __ldg(reinterpret_cast<const unsigned long long*>(p.w + size_t(j0 + x) * kD + 64 * warp) + lane) : 0;
        }
#pragma unroll
        for (int e = 0; e < kRound; ++e) {
          if (e >= ne) break;
          const int q = ctl.toks[r0 + e].pos + 1 + p.lookahead - p.window - p.k_taps + j0;
          const int lo = min(max(0, -q), tp), hi = max(lo, min(tp, p.k_taps - j0));
          const uint32_t* src = reinterpret_cast<const uint32_t*>(stages + (got % kStages) * kStageBytes) + 32 * warp + lane;
          if (wait_rows(&ctl, got % kStages, (got / kStages) & 1)) {
#pragma unroll
            for (int x = 0; x < kTaps; ++x)
              if (x >= lo && x < hi) add2(acc[e], w[x], src[x * (kD / 2)]);
          }
          ++got;
          app_sync();
          if (tid == 0) issue();
        }
      }
      if (round && !(again && r0 == 0)) cluster_wait_acquire_div();  // (the last round's sums are read)
#pragma unroll
      for (int e = 0; e < kRound; ++e)
        if (e < ne) st_dsmem_u64(dsmem_addr(part + rank * kD + 64 * warp + 2 * lane, e), acc[e]);
      cluster_arrive_release_div();
      cluster_wait_acquire_div();
      cluster_arrive_release_div();
    }
  }
  if (!rows_done) write_rows<FMT>(p, rows, n.x, theta);
  pdl_trigger();  // (not earlier: the next kernel's waiting blocks would keep the clusters from starting together)
  if (total) cluster_wait_acquire_div();  // (no CTA leaves while another may still read its list or write its sums)
  if (tid == 0 && ctl.dead) {
    set_status(p.status, DSV4KV_DEV_TIMEOUT);
    uint64_t t0, t;  // copies that were in flight when the wait gave up have landed long before this
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t0));
    do asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    while (t - t0 < 1000000ull);
  }
}

// The rows that a batch of long chunks leaves behind: the last window + k_taps tokens of every sequence into its raw
// ring, the last `window` of them into the window cache.  One warp a row.
template <int FMT>
__global__ void __launch_bounds__(kAppThreads) append_rows_kernel(const __grid_constant__ AppendParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.y, r = blockIdx.x * kAppWarps + warp, R = p.window + p.k_taps;
  const double theta = p.rope.theta_pi[lane];
  pdl_wait();
  pdl_trigger();  // (after the wait, for the same reason: 43 against 60 us a call of c128a prompts, back to back)
  const int c0 = p.cu[b], c1 = p.cu[b + 1];
  if (c0 < 0 || c1 > p.tokens || c1 - c0 > p.max_new || r >= min(c1 - c0, R)) return;  // (flagged by the entries' pass)
  const int i = c1 - 1 - r;
  const uint16_t* src = p.s_new + size_t(i) * kD + 8 * lane;
  const uint4 v0 = first_piece(src), v1 = second_piece(src);
  const int64_t at = __ldg(p.pos + i);
  const int slot = __ldg(p.win_slot + i);
  if (__ldg(p.seq + i) != b || at < i - c0 || at >= (int64_t(1) << 31) - p.lookahead - 1) return;
  uint16_t* dst = p.ring + (size_t(b) * R + int(at) % R) * kD + 8 * lane;
  *reinterpret_cast<uint4*>(dst) = v0;
  *reinterpret_cast<uint4*>(dst + 256) = v1;
  if (slot >= 0 && slot < p.win_rows) {
    float x[kPer];
    unpack8(v0, x);
    unpack8(v1, x + 8);
    rotate_row(x, p, theta, int(at), lane);
    store_row<FMT>(x, lane, slot, p.win_codes, p.win_scales);
  }
}

// Clusters of append_long_kernel that the current device holds at once.
template <int FMT>
int clusters_at_once() {
  static std::atomic<int> cache[64];  // per device; 0 = not queried yet
  std::atomic<int>& slot = cache[current_device()];
  int n = slot.load(std::memory_order_relaxed);
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(2 * sm_count() / kCl * kCl));
    cfg.blockDim = dim3(kLongThreads);
    cfg.dynamicSmemBytes = kLongSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kCl;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, append_long_kernel<FMT>, &cfg) != cudaSuccess || n < 1) n = sm_count() / kCl;
    cudaGetLastError();  // (a refused query only means a guess)
    slot.store(n, std::memory_order_relaxed);
  }
  return n;
}

template <int FMT>
cudaError_t launch_append(AppendParams p, cudaStream_t stream) {
  const bool is_long = p.k_taps > kLongTaps;
  static std::atomic<uint64_t> ready{0};
  if (!done_on_device(ready)) {
    cudaError_t e = cudaFuncSetAttribute(append_paged_kernel<FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         int(kLongTaps * kD * sizeof(float)));
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(append_long_kernel<FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kLongSmem));
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(append_rows_kernel<FMT>, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    mark_done_on_device(ready);
  }
  if (!(p.parts & kPartEntries)) {
    const dim3 grid(unsigned((std::min(p.window + p.k_taps, p.max_new) + kAppWarps - 1) / kAppWarps), unsigned(p.batch));
    return launch_pdl(append_rows_kernel<FMT>, grid, dim3(kAppThreads), 0, stream, p);
  }
  // Few tokens: spread over the SMs; many: runs of up to 128 tokens (short entries, 4 CTAs an SM), or as many as the
  // clusters that run at once share (long ones).
  const int64_t ctas = is_long ? kCl * clusters_at_once<FMT>() : 4 * sm_count();
  p.per = int(std::max<int64_t>(1, std::min<int64_t>((p.tokens + ctas - 1) / ctas, is_long ? kMaxTokens : 128)));
  const int grid = int((int64_t(p.tokens) + p.per - 1) / p.per);
  if (is_long)
    return launch_pdl_cluster(append_long_kernel<FMT>, dim3(unsigned((grid + kCl - 1) / kCl * kCl)), dim3(kLongThreads),
                              kLongSmem, kCl, stream, p);
  return launch_pdl(append_paged_kernel<FMT>, dim3(unsigned(grid)), dim3(kAppThreads), size_t(p.k_taps) * kD * sizeof(float),
                    stream, p);
}

}  // namespace

void rope_table_fill(RopeTable* r, int rope_dim, double rope_base) {
  for (int m = 0; m < 256; ++m)
    r->theta_pi[m] = m >= rope_dim / 2 ? 0.0 : pow(rope_base, -2.0 * double(m) / double(rope_dim)) / 3.141592653589793;
}

dsv4kv_status block_table_update_launch(const int64_t* t_old, const int64_t* t_new, int batch, int64_t t_max, int window,
                                        int stride, int lookahead, int page_rows, int32_t* table, int table_stride,
                                        int64_t pool_pages, int32_t* free_pages, int64_t free_cap,
                                        const int64_t* free_count, int64_t* free_count_out, void* ws,
                                        cudaStream_t stream) {
  const TableParams p{t_old, t_new, batch, t_max, window, stride, lookahead, page_rows, table, table_stride,
                      pool_pages, free_pages, free_cap, free_count, free_count_out, static_cast<uint32_t*>(ws)};
  // a decode step changes at most a page or so per sequence; prompts bring up to table_stride of them
  const int64_t most = int64_t(batch) * table_stride;
  const int grid = int(std::max<int64_t>(1, std::min<int64_t>(64, most / (2 * kTabThreads))));
  const size_t smem = size_t(4 * (batch + 1)) * sizeof(int32_t);
  if (smem > 48 * 1024 - 256) {  // (more than 3054 sequences)
    const cudaError_t e = cudaFuncSetAttribute(block_table_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return set_error(DSV4KV_ERR_CUDA, "block_table_kernel: %s", cudaGetErrorString(e));
  }
  launch_pdl(block_table_kernel, dim3(grid), dim3(kTabThreads), smem, stream, p);
  return check_launch("block_table_kernel");
}

dsv4kv_status slot_map_launch(const int64_t* t_old, const int64_t* t_new, int batch, int64_t t_max, int window,
                              int stride, int lookahead, const PageDesc& comp, const PageDesc& win, int capacity,
                              int32_t* cu, int32_t* seq, int64_t* pos, int32_t* win_slot, int32_t* comp_slot, void* ws,
                              cudaStream_t stream) {
  const SlotParams p{t_old, t_new, batch, t_max, window, stride, lookahead, comp, win, capacity, cu, seq, pos,
                     win_slot, comp_slot, static_cast<uint32_t*>(ws), Div(std::max(window, 1)), Div(stride),
                     Div(comp.page_rows), Div(win.page_rows)};
  const int per = kSlotThreads * kSlotPer;
  const int grid = int(std::max<int64_t>(1, std::min<int64_t>(4 * sm_count(), (int64_t(capacity) + per - 1) / per)));
  const size_t smem = size_t(3 * batch + 1) * sizeof(int32_t);
  if (smem > 48 * 1024 - 256) {  // (more than 4070 sequences)
    const cudaError_t e = cudaFuncSetAttribute(slot_map_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return set_error(DSV4KV_ERR_CUDA, "slot_map_kernel: %s", cudaGetErrorString(e));
  }
  launch_pdl(slot_map_kernel, dim3(grid), dim3(kSlotThreads), smem, stream, p);
  return check_launch("slot_map_kernel");
}

dsv4kv_status append_paged_launch(const void* s_new, const float* w, int batch, int tokens, const int32_t* cu,
                                  const int32_t* seq, const int64_t* pos, const int32_t* win_slot,
                                  const int32_t* comp_slot, int k_taps, int stride, int window, int lookahead,
                                  int64_t max_new, int rope_dim, double rope_base, void* raw_ring,
                                  const dsv4kv_cache& win, const dsv4kv_cache& comp, void* ws, cudaStream_t stream) {
  AppendParams p;
  p.s_new = static_cast<const uint16_t*>(s_new);
  p.w = w;
  p.batch = batch;
  p.tokens = tokens;
  p.cu = cu;
  p.seq = seq;
  p.pos = pos;
  p.win_slot = win_slot;
  p.comp_slot = comp_slot;
  p.k_taps = k_taps;
  p.stride = stride;
  p.window = window;
  p.lookahead = lookahead;
  p.max_new = int(std::min<int64_t>(max_new, tokens));
  p.rope_dim = rope_dim;
  p.ring = static_cast<uint16_t*>(raw_ring);
  p.win_codes = static_cast<uint8_t*>(const_cast<void*>(win.codes));
  p.win_scales = const_cast<void*>(win.scales);
  p.win_rows = window > 0 ? win.rows : 0;
  p.comp_codes = static_cast<uint8_t*>(const_cast<void*>(comp.codes));
  p.comp_scales = const_cast<void*>(comp.scales);
  p.comp_rows = comp.rows;
  p.status = static_cast<uint32_t*>(ws);
  rope_table_fill(&p.rope, rope_dim, rope_base);
  const bool two = max_new > int64_t(lookahead) + 1;
  for (int pass = 0; pass < (two ? 2 : 1); ++pass) {
    p.parts = !two ? kPartEntries | kPartWindow | kPartRing : pass == 0 ? kPartEntries : kPartWindow | kPartRing;
    cudaError_t e;
    switch (comp.fmt) {
      case DSV4KV_BF16: e = launch_append<DSV4KV_BF16>(p, stream); break;
      case DSV4KV_FP8_E4M3_ROW: e = launch_append<DSV4KV_FP8_E4M3_ROW>(p, stream); break;
      case DSV4KV_FP4_E2M1_G16: e = launch_append<DSV4KV_FP4_E2M1_G16>(p, stream); break;
      default: e = launch_append<DSV4KV_FP8_E4M3_ROW_ROPE_BF16>(p, stream); break;
    }
    if (e != cudaSuccess) return set_error(DSV4KV_ERR_CUDA, "append_paged_kernel: %s", cudaGetErrorString(e));
    const dsv4kv_status st = check_launch("append_paged_kernel");
    if (st != DSV4KV_OK) return st;
  }
  return DSV4KV_OK;
}

}  // namespace dsv4kv
