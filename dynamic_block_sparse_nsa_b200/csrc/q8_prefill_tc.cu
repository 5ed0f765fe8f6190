// nsa_prefill_q8 on the sm_100a tensor memory: chunks of queries over the 8-bit
// paged cache, bf16, d = 128, pages of 32 tokens or more. The mathematics is
// that of q8_attend.cu (fp16 products with exact codes, a row scale for q, the
// running maximum m and the output's own reference M); the work plan too, with
// tiles of 256 query rows and chunks of 128 keys.
//
// 4 d flops a row and key make it a matrix kernel: per chunk and tile
// S = Q K^T and O += P V, two 128-row halves each, S (later P) and O of both
// halves in the 512 columns of tensor memory. Roles, one persistent block per
// SM:
//   warps 0-3, 4-7   softmax of a half, a thread per row: S from tensor memory,
//                    P back over it, O rescaled when its reference moves by
//                    more than 2^5, the epilogue;
//   warps 8-11       codes to fp16 K and V tiles in shared memory (128-byte
//                    swizzle), a ring of three;
//   warp 12          copies the pages' codes to shared memory (a head's page is
//                    contiguous: one bulk copy each), three tiles ahead;
//   warp 13          issues the MMAs: while one half's softmax runs, the other
//                    half's products do.
// Where most sequences have rows for one half only (draft tokens), both halves
// take the same rows and alternate chunks (SPLIT), and half 0 joins the two sums
// at the unit's end: 16 sequences of 4 queries over 8191 keys 93 -> 75 us when it
// came in, 77 with the fence behind the converters' loads (a chunk 1.4 us instead
// of 2.4; with one chunk a sequence the call takes 22 us: plan, start and merge).
// A half's chain of softmax (an exponential for every score, 16 a clock and SM,
// is as long as its two products) and products bounds it. 2048 queries of 64
// heads over 16384 keys (4 KV heads): 1.07 ms, 967 TFLOP/s, in short runs, 1.11 ms,
// 929 TFLOP/s, in a program of such calls at the board's power limit. Value scales
// too far apart (q8_attend.cuh) take five times as long. What was measured
// slower: steps of 64 keys with two S tiles a half (the products' overhead
// doubles: 1.15 ms), two threads a row (16 softmax warps: 1.05 ms, short units
// 87 us), 192 registers for the softmax by setmaxnreg (the other
// roles spill: 1.43 ms), MMAs issued under `lane == 0` (1.19 ms).
#include <cuda.h>

#include <algorithm>

#include "q8_attend.cuh"
#include "tcgen05.cuh"

namespace nsa {
namespace {

using q8::Place;
using q8::Plan;
using q8::Seq;

constexpr int D = 128;
constexpr int ROWS = kQ8TcRows;
constexpr int CK = kQ8TcKeys;
constexpr uint32_t ATOM = 16384;   // 128 rows x 64 halves
constexpr uint32_t TILE = 32768;   // 128 rows x 128 halves
constexpr int kThreads = 14 * 32;
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr float kLag = 5.f;        // how far M may fall behind before O is rescaled
constexpr int kRing = 3;           // fp16 tiles: K of chunk 0, V of it, K of chunk 1, ...
constexpr int kRaw = 3;            // tiles of codes under way
constexpr int kFar = 1 << 20;      // beyond every scale's exponent
constexpr int kNanSlots = 4;       // units whose NaN marks are under way
// Floats of a partial: o as [D / 4][ROWS] of 4 components (a thread has a row: a
// warp's stores are contiguous), then lse2 of the rows.
constexpr long kPart = (long)ROWS * D + ROWS;

// Tensor-memory columns of half t: S, later P; and O.
__device__ __forceinline__ uint32_t s_col(int t) { return 128u * t; }
__device__ __forceinline__ uint32_t o_col(int t) { return 256u + 128u * t; }

struct Bars {
  uint64_t q_full[2], s_full[2], p_full[2], o_full[2];
  uint64_t full[kRing], empty[kRing], raw_full[kRaw], raw_empty[kRaw];
  uint64_t fin, marks, stats_full;
  int abort;
  uint32_t tmem;
  int nan_flag[kNanSlots];
  uint32_t live[kRaw];  // pages of the tile that were copied, a bit each
};

struct Smem {
  unsigned char q[2][TILE];
  unsigned char kv[kRing][TILE];
  unsigned char raw[kRaw][CK * D];
  Bars bars;
  float stats[3][128];                 // of half 1's rows in a unit split over the halves
  uint32_t nan_rows[kNanSlots][D][8];  // per component: the tile's tokens that see a NaN value
};

__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                     unsigned* err) {
  if (ptx::mbar_try_wait(bar, parity & 1u)) return true;
  if (*abort) return false;
  if (ptx::mbar_wait(bar, parity & 1u, kWaitNs)) return true;
  atomicOr(err, kErrTimeout);
  *abort = 1;
  return false;
}

// Descriptor of the 16-component step ks of an operand whose first step's
// descriptor is d: K-major (32 bytes a step, four to a 64-component atom), or
// MN-major (16 rows of 128 bytes a step). The address field counts 16 bytes.
__device__ __forceinline__ uint64_t k_step(uint64_t d, int ks) {
  return d + (((ks >> 2) * ATOM + (ks & 3) * 32) >> 4);
}
__device__ __forceinline__ uint64_t mn_step(uint64_t d, int ks) { return d + ((ks * 2048) >> 4); }

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// One lane of a converged warp: the MMAs and commits are its, the control flow
// around them the whole warp's (their operands then stay uniform).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// 16 components as bf16: a 32-byte sector in two stores.
__device__ __forceinline__ void store32(__nv_bfloat16* dst, const float* y) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = ptx::pack_bf16(y[2 * i], y[2 * i + 1]);
  reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
  reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

// A unit: a tile's rows of one KV head.
struct Unit {
  Seq s;
  int b, r0, rows;
  int lo, hi;            // keys that some row sees
  int all_lo, all_hi;    // keys that all rows see
  int tok0, tok1;        // tokens of the rows, of the sequence's new ones
  __device__ __forceinline__ void load(const Q8AttendArgs& a, const Plan& pl, int tile) {
    b = pl.tseq[tile];
    r0 = (tile - pl.tbase[b]) * ROWS;
    s = q8::sequence(a, b);
    rows = min(ROWS, s.n * a.G - r0);
    q8::key_span(a, s, r0, ROWS, lo, hi);
    tok0 = r0 / a.G;
    tok1 = (r0 + rows - 1) / a.G;
    const int at = s.len - s.n;
    all_hi = hi > 0 ? at + tok0 + 1 : 0;
    all_lo = a.keys == q8::KEYS_WINDOW ? at + tok1 + 1 - a.window : 0;
  }
};

// The block's chunks, unit by unit: `n` chunks of the current unit from its
// chunk `first` on. A chunk is `wt` places of the plan, one for each half that
// has rows; a unit's own cost (query rows in, output rows out) is kQ8TcUnit
// places ahead of its chunks. A chunk is the block's that has its first place.
template <bool SPLIT>
struct Walk {
  Place at;
  Unit u;
  long x, end;
  int first, n, seg, wt;
  __device__ __forceinline__ void start(const Q8AttendArgs& a, const Plan& pl, long x0, long x1) {
    x = x0;
    end = x1;
    seg = 0;
    at.init(pl, a.Hkv, x0);
    u.load(a, pl, at.tile);
    settle(a, pl);
  }
  __device__ __forceinline__ int span() const { return (int)min((long)(at.nc - at.c), end - x); }
  __device__ __forceinline__ void settle(const Q8AttendArgs& a, const Plan& pl) {
    while (x < end) {
      wt = SPLIT ? q8::tc_weight(u.rows) : 1;
      first = (max(0, at.c - kQ8TcUnit) + wt - 1) / wt;
      n = (max(0, at.c + span() - kQ8TcUnit) + wt - 1) / wt - first;
      if (n > 0) return;
      step(a, pl);
    }
  }
  __device__ __forceinline__ void step(const Q8AttendArgs& a, const Plan& pl) {
    x += span();
    if (x >= end) return;
    const int tile = at.tile;
    at.c = at.nc - 1;  // (only a unit's last segment is followed by another)
    at.next(pl, a.Hkv);
    if (at.tile != tile) u.load(a, pl, at.tile);
  }
  __device__ __forceinline__ bool done() const { return x >= end; }
  __device__ __forceinline__ void next(const Q8AttendArgs& a, const Plan& pl) {
    ++seg;
    step(a, pl);
    settle(a, pl);
  }
  __device__ __forceinline__ int key0(int i) const { return (u.lo / CK + first + i) * CK; }
  __device__ __forceinline__ bool ends() const { return first + n == (at.nc - kQ8TcUnit) / wt; }
  // Rows for one half only: the halves take alternate chunks of the same rows.
  __device__ __forceinline__ bool split() const { return SPLIT && wt == 1 && n > 1; }
  // Tile j of the 2 n in the order of their use: K and V of chunk c in turn, or
  // (split) each chunk's V behind the next one's K.
  __device__ __forceinline__ void tile(int j, int& c, bool& v) const {
    c = j >> 1;
    v = j & 1;
    if (!split() || j == 0 || j == 2 * n - 1) return;
    c = v ? c + 1 : c - 1;
    v = !v;
  }
};

// Lane j's page of the chunk that begins at key0 (j < 128 / page); -1: none
// (pages before the window may be gone), INT_MAX: not a page number.
__device__ __forceinline__ int page_of(const Q8AttendArgs& a, const Unit& u, int key0, int lane,
                                       int shift) {
  const int first = key0 + (lane << shift);
  if (lane >= CK >> shift || first >= u.hi || first + a.page <= u.lo) return -1;
  const int pid = a.table[(long)u.b * a.max_pages + (first >> shift)];
  return pid < 0 ? INT_MAX : pid;
}

// ---- pages to shared memory (one warp) -------------------------------------------

template <bool SPLIT>
__device__ void copy_pages(const Q8AttendArgs& a, const Plan& pl, long X0, long X1, Smem& sm,
                           int shift, int lane) {
  Bars& B = sm.bars;
  volatile int* abort = &B.abort;
  const uint32_t bytes = (uint32_t)D << shift;
  Walk<SPLIT> w;
  bool ok = true;
  int n = 0;  // the block's tile
  for (w.start(a, pl, X0, X1); ok && !w.done(); w.next(a, pl)) {
    int key0 = w.key0(0);
    int pid = page_of(a, w.u, key0, lane, shift);  // lane j: page j of the chunk
    // the next chunk's, looked up ahead; a number that is none is left out
    auto step = [&] {
      const int now = pid < a.num_pages ? pid : -1;
      if (now != pid) atomicOr(a.err, kErrPage);
      key0 += CK;
      pid = page_of(a, w.u, key0, lane, shift);
      return now;
    };
    // one tile: every lane its page
    auto put = [&](int page, bool v) {
      const bool mine = page >= 0;
      const uint32_t live = __ballot_sync(0xffffffffu, mine);
      const long from = ((long)page * a.Hkv + w.at.h) << (shift + 7);
      const int r = n % kRaw;
      if (n >= kRaw) ok = wait(&B.raw_empty[r], n / kRaw - 1, abort, a.err);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      if (lane == 0) {
        B.live[r] = live;
        ptx::mbar_arrive_expect_tx(&B.raw_full[r], __popc(live) * bytes);
      }
      __syncwarp();
      if (mine)
        ptx::bulk_load(sm.raw[r] + lane * bytes, (v ? a.v_pages : a.k_pages) + from, bytes,
                       &B.raw_full[r]);
      ++n;
    };
    if (w.split()) {
      int now = step();
      put(now, false);
      for (int i = 1; ok && i <= w.n; ++i) {
        const int before = now;
        if (i < w.n) put(now = step(), false);
        if (ok) put(before, true);
      }
    } else {
      for (int i = 0; ok && i < w.n; ++i) {
        const int now = step();
        // (one copy of the code: unrolled, the call of 2048 queries takes 3 % longer)
#pragma unroll 1
        for (int v = 0; ok && v < 2; ++v) put(now, v);
      }
    }
  }
  // every copy has landed before the block ends
  for (int k = n > kRaw ? n - kRaw : 0; k < n; ++k)
    if (!ptx::mbar_wait(&B.raw_full[k % kRaw], (k / kRaw) & 1, kWaitNs)) atomicOr(a.err, kErrTimeout);
}

// ---- codes to fp16 tiles ------------------------------------------------------

struct Converter {
  const Q8AttendArgs& a;
  int warp, lane;  // of the four
  int shift;       // log2 of the page
  __device__ __forceinline__ int row(int k) const { return 16 * k + 4 * warp + (lane >> 3); }

  // Row r's 16 components as two 16-byte pieces of the swizzled tile; lanes of
  // the second half store theirs in the other order, so that the eight lanes
  // of a row cover all banks.
  __device__ __forceinline__ void store(const uint4 (&x)[8], unsigned char* tile) const {
    const int c8 = lane & 7;
    const bool odd = c8 >= 4;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int r = row(k);
      unsigned char* dst = tile + (c8 >> 2) * ATOM + r * 128;
      const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
      uint32_t hx[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        hx[2 * i] = q8::e4m3x2_to_half2((uint16_t)(w[i] & 0xffffu));
        hx[2 * i + 1] = q8::e4m3x2_to_half2((uint16_t)(w[i] >> 16));
      }
      const uint4 p0 = make_uint4(hx[0], hx[1], hx[2], hx[3]);
      const uint4 p1 = make_uint4(hx[4], hx[5], hx[6], hx[7]);
      const int c = (c8 & 3) * 2;
      *reinterpret_cast<uint4*>(dst + (((c + odd) ^ (r & 7)) << 4)) = odd ? p1 : p0;
      *reinterpret_cast<uint4*>(dst + (((c + !odd) ^ (r & 7)) << 4)) = odd ? p0 : p1;
    }
  }

  // NaN values of keys that only some of the tile's tokens see: marked for
  // those, and replaced by zeros (0 * NaN would reach the others).
  // at0: position of the tile's first token, last: index of its last.
  __device__ void mark_nan(uint4 (&x)[8], int at0, int last, int key0, uint32_t (*marks)[8],
                           int* flag) const {
    bool found = false;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) found |= __vcmpeq4(w[i] & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0;
    }
    if (!found) return;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
      const int key = key0 + row(k);
      const int from = max(0, key - at0);
      const int to = a.keys == q8::KEYS_WINDOW ? min(last, key - at0 + a.window - 1) : last;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t bad = __vcmpeq4(w[i] & 0x7f7f7f7fu, 0x7f7f7f7fu);
        if (!bad) continue;
        w[i] &= ~bad;
        for (int y = 0; y < 4; ++y)
          if (bad >> (8 * y) & 1u)
            for (int t = from; t <= to; ++t)
              atomicOr(&marks[(lane & 7) * 16 + 4 * i + y][t >> 5], 1u << (t & 31));
      }
      x[k] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    *flag = 1;
    __threadfence_block();
  }

  template <bool SPLIT>
  __device__ void run(const Plan& pl, long X0, long X1, Smem& sm) const {
    Bars& B = sm.bars;
    volatile int* abort = &B.abort;
    Walk<SPLIT> w;
    int n = 0;  // the block's tile
#pragma unroll 1
    for (w.start(a, pl, X0, X1); !w.done(); w.next(a, pl)) {
      const int lo = w.u.lo, hi = w.u.hi, all_lo = w.u.all_lo, all_hi = w.u.all_hi;
      const int slot = w.seg % kNanSlots, tiles = 2 * w.n;
      int key0 = w.key0(0);
#pragma unroll 1
      for (int i = 0; i < tiles; ++i, ++n) {
        const int r = n % kRaw, buf = n % kRing;
        bool isv = i & 1;
        if (SPLIT) {
          int c;
          w.tile(i, c, isv);
          key0 = w.key0(c);
        }
        wait(&B.raw_full[r], n / kRaw, abort, a.err);
        const uint32_t live = B.live[r];
        uint4 x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          x[k] = *reinterpret_cast<const uint4*>(sm.raw[r] + row(k) * D + (lane & 7) * 16);
        // The next write to the slot is a bulk copy, of the async proxy: without the
        // fence it can overtake these loads, whose data nothing has used yet (one
        // call in 50 of 2600 queries had codes of the copy in place of V's).
        ptx::fence_proxy_async();
        ptx::mbar_arrive(&B.raw_empty[r]);
        if (key0 + CK > all_hi || key0 < all_lo || live != (1u << (CK >> shift)) - 1) {
          // rows that no token sees hold anything: zeros
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int pos = key0 + row(k);
            if (pos < lo || pos >= hi || !(live >> (row(k) >> shift) & 1u))
              x[k] = make_uint4(0, 0, 0, 0);
          }
          if (isv)
            mark_nan(x, w.u.s.len - w.u.s.n + w.u.tok0, w.u.tok1 - w.u.tok0, key0,
                     sm.nan_rows[slot], &B.nan_flag[slot]);
        }
        if (n >= kRing) wait(&B.empty[buf], n / kRing - 1, abort, a.err);
        store(x, sm.kv[buf]);
        ptx::fence_proxy_async();
        ptx::mbar_arrive(&B.full[buf]);
        if (!SPLIT && (i & 1)) key0 += CK;
      }
    }
  }
};

// ---- MMAs (one warp) ----------------------------------------------------------

template <bool SPLIT>
__device__ void issue_mmas(const Q8AttendArgs& a, const Plan& pl, long X0, long X1, Smem& sm) {
  Bars& B = sm.bars;
  volatile int* abort = &B.abort;
  const uint32_t tmem = B.tmem;
  constexpr uint32_t iqk = tc::idesc_f16(128, 128, false, false);
  constexpr uint32_t ipv = tc::idesc_f16(128, 128, false, true);
  const uint64_t dq = tc::sdesc(ptx::smem_u32(sm.q), 16, 1024, tc::kSw128);
  const uint64_t dk = tc::sdesc(ptx::smem_u32(sm.kv), 16, 1024, tc::kSw128);
  const uint64_t dv = tc::sdesc(ptx::smem_u32(sm.kv), ATOM, 1024, tc::kSw128);
  int segs[2] = {0, 0}, tiles[2] = {0, 0};  // per half: units begun, P tiles taken
  Walk<SPLIT> w;
  bool ok = true;
  int n = 0;  // the block's K tile (its V tile is n + 1)
  for (w.start(a, pl, X0, X1); ok && !w.done(); w.next(a, pl)) {
    const int chunks = w.n;
    const bool split = w.split();
    const int halves = w.u.rows > 128 || split ? 2 : 1;
    // (the warp stays together when a wait gives up in some of its lanes)
    auto all = [&](bool r) { return (bool)__all_sync(0xffffffffu, r); };
    auto ready = [&](int k) {
      const bool r = wait(&B.full[k % kRing], k / kRing, abort, a.err);
      tc::fence_after_sync();
      return r;
    };
    auto qk = [&](int t, int k, bool free) {
      const uint64_t qt = dq + ((t * TILE) >> 4), kt = dk + (((k % kRing) * TILE) >> 4);
      if (elect_one()) {
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          tc::mma_ss(tmem + s_col(t), k_step(qt, ks), k_step(kt, ks), iqk, ks > 0);
        tc::commit(&B.s_full[t]);
        if (free) tc::commit(&B.empty[k % kRing]);
      }
      __syncwarp();
    };
    for (int t = 0; t < halves; ++t) ok = ok && wait(&B.q_full[t], segs[t]++, abort, a.err);
    auto pv = [&](int t, int k, bool begun, bool free, bool ends) {
      const uint64_t vt = dv + (((k % kRing) * TILE) >> 4);
      if (elect_one()) {
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          tc::mma_ts(tmem + o_col(t), tmem + s_col(t) + ks * 8, mn_step(vt, ks), ipv,
                     (begun || ks > 0));
        if (free) tc::commit(&B.empty[k % kRing]);
        if (ends) tc::commit(&B.o_full[t]);
      }
      __syncwarp();
    };
    ok = all(ok && ready(n));
    if (split) ok = all(ok && ready(n + 1));
    if (!ok) break;
    for (int t = 0; t < halves; ++t) qk(t, split ? n + t : n, split || t == halves - 1);
    if (split) {
      for (int i = 0; i < chunks; ++i) {
        const int t = i & 1, kv = n + (i < chunks - 1 ? 2 * i + 2 : 2 * i + 1);
        const bool more = i + 2 < chunks;
        const bool r = ready(kv) && (!more || ready(kv + 1));
        ok = all(r && wait(&B.p_full[t], tiles[t]++, abort, a.err));
        if (!ok) break;
        tc::fence_after_sync();
        pv(t, kv, i > 1, true, !more);
        if (more) qk(t, kv + 1, true);
      }
      n += 2 * chunks;
      continue;
    }
    for (int i = 0; ok && i < chunks; ++i, n += 2) {
      const bool more = i + 1 < chunks;
      // (both are converted ahead; no wait then lies between the products but P's)
      const bool kv = ready(n + 1) && (!more || ready(n + 2));
      for (int t = 0; t < halves; ++t) {
        ok = all(kv && wait(&B.p_full[t], tiles[t]++, abort, a.err));
        if (!ok) break;
        tc::fence_after_sync();
        pv(t, n + 1, i > 0, t == halves - 1, !more);
        if (more) qk(t, n + 2, t == halves - 1);
      }
    }
  }
  if (elect_one()) tc::commit(&B.fin);
  if (!ptx::mbar_wait(&B.fin, 0, kWaitNs)) atomicOr(a.err, kErrTimeout);
}

// ---- softmax (a thread per row of half t) -----------------------------------------

struct Softmax {
  const Q8AttendArgs& a;
  Smem& sm;
  int t, row;      // half, row of it
  int r1;          // the half's first row in the unit's
  uint32_t tl;     // the warp's lanes of tensor memory
  int shift;       // log2 of the page
  float qf;        // row factor of the scores
  int lo, hi;      // keys the row sees

  // The row's query, scaled into fp16's range, into the half's tile.
  __device__ __forceinline__ void load_query(const Unit& u, int h) {
    const int r = u.r0 + r1 + row;
    const bool real = r < u.s.n * a.G;
    const int pos = u.s.len - u.s.n + r / a.G;
    // (rows behind the last see everything: their warps need no masks)
    hi = !real ? INT_MAX / 2 : u.hi > 0 ? pos + 1 : 0;
    lo = real && a.keys == q8::KEYS_WINDOW ? max(0, pos + 1 - a.window) : 0;
    uint4 x[16];
    const uint4* src = reinterpret_cast<const uint4*>(
        static_cast<const __nv_bfloat16*>(a.q) + (real ? out_row(u, h, r) : 0) * D);
#pragma unroll
    for (int c = 0; c < 16; ++c) x[c] = real ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
    float big = 0.f;
    bool finite = true;
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float f0 = fabsf(__uint_as_float(w[i] << 16));
        const float f1 = fabsf(__uint_as_float(w[i] & 0xffff0000u));
        if (f0 < INFINITY) big = fmaxf(big, f0);
        if (f1 < INFINITY) big = fmaxf(big, f1);
        finite &= f0 < INFINITY && f1 < INFINITY;
      }
    }
    // 2^up brings the largest component to [2^14, 2^15)
    int up = big > 0.f ? 14 - ((int)(__float_as_uint(big) >> 23) - 127) : 0;
    up = min(max(up, -120), 120);
    // (a negative softmax scale's sign goes into q)
    float mul = a.scale_log2 < 0.f ? -q8::exp2_int(up) : q8::exp2_int(up);
    // (an infinite component makes every score infinite or NaN: the row is NaN)
    if (!finite) mul = __uint_as_float(0x7fffffffu);
    qf = q8::exp2_int(-up) * fabsf(a.scale_log2);
    unsigned char* dst = sm.q[t] + row * 128;
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
      uint32_t y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        y[i] = pack_half(__uint_as_float(w[i] << 16) * mul,
                         __uint_as_float(w[i] & 0xffff0000u) * mul);
      *reinterpret_cast<uint4*>(dst + (c >> 3) * ATOM + (((c & 7) ^ (row & 7)) << 4)) =
          make_uint4(y[0], y[1], y[2], y[3]);
    }
    ptx::fence_proxy_async();
    tc::fence_before_sync();  // (the unit before was read from tensor memory)
    ptx::mbar_arrive(&sm.bars.q_full[t]);
  }

  __device__ __forceinline__ long out_row(const Unit& u, int h, int r) const {
    return ((long)u.s.first + r / a.G) * a.Hq + h * a.G + r % a.G;
  }

  // A chunk's pages as lane j holds them: page j, its scales, log2 of V's.
  struct Pages {
    int pid;
    float ks, vs, lv;
    __device__ __forceinline__ void scales(const Q8AttendArgs& a, int h) {
      if (pid >= a.num_pages) pid = -1;
      ks = vs = 0.f;
      if (pid >= 0) {
        ks = a.k_scale[(long)pid * a.Hkv + h];
        vs = a.v_scale[(long)pid * a.Hkv + h];
      }
    }
  };

  // The running maximum and reference after 32 scores.
  static __device__ __forceinline__ void largest(const uint32_t (&z)[32], float c, float lv,
                                                 float& top, float& ref) {
    const float pm = max32(z) * c;
    top = fmaxf(top, pm);
    ref = fmaxf(ref, pm + fmaxf(lv, -126.f) - 10.f);
  }

  // p * vscale in units of 2^M of 32 scores, as halves to tensor memory (over
  // scores that are read already); sum += p.
  static __device__ __forceinline__ void weights(const uint32_t (&z)[32], uint32_t to, float c,
                                                 float lv, float oref, float base, float& sum) {
    const uint64_t cc = pack2(c, c), off = pack2(lv - oref, lv - oref);
    uint64_t s = pack2(0.f, 0.f);
    uint32_t p[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float p0, p1;
      unpack2(fma2(pack2(__uint_as_float(z[2 * e]), __uint_as_float(z[2 * e + 1])), cc, off), p0, p1);
      p0 = ptx::ex2(p0);
      p1 = ptx::ex2(p1);
      s = add2(s, pack2(p0, p1));
      p[e] = pack_half(p0, p1);
    }
    tc::st16(to, p);
    float s0, s1;
    unpack2(s, s0, s1);
    sum = fmaf(s0 + s1, ptx::ex2(oref - base - lv), sum);
  }

  static __device__ __forceinline__ float max32(const uint32_t (&z)[32]) {
    float x0 = -INFINITY, x1 = -INFINITY, x2 = -INFINITY, x3 = -INFINITY;
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
      x0 = fmaxf(x0, __uint_as_float(z[e]));
      x1 = fmaxf(x1, __uint_as_float(z[e + 1]));
      x2 = fmaxf(x2, __uint_as_float(z[e + 2]));
      x3 = fmaxf(x3, __uint_as_float(z[e + 3]));
    }
    return fmaxf(fmaxf(x0, x1), fmaxf(x2, x3));
  }

  // The lane's four keys' code_room (q8_attend.cuh), a byte each, from the fp16 V
  // tile: a row's largest magnitude.
  static __device__ __forceinline__ uint32_t rooms_of(const unsigned char* tile, int lane) {
    uint32_t rooms = 0;
#pragma unroll 1
    for (int k = 0; k < 4; ++k) {
      const unsigned char* from = tile + (4 * lane + k) * 128;
      __half2 top = __float2half2_rn(0.f);
#pragma unroll
      for (int c = 0; c < 16; ++c) {  // (a row's pieces in any order: lanes on banks of their own)
        const uint4 v =
            *reinterpret_cast<const uint4*>(from + (c >> 3) * ATOM + (((c + lane) & 7) << 4));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          top = __hmax2(top, __habs2(*reinterpret_cast<const __half2*>(&w[i])));
      }
      const uint32_t u = *reinterpret_cast<const uint32_t*>(&top);
      const uint32_t c = max(u & 0xffffu, u >> 16);  // a code's exponent is 8 less in fp16
      const uint32_t room = c == 0u ? q8::kNoCode : min(5u, 23u - (c >> 10));
      rooms |= room << 8 * k;
    }
    return rooms;
  }

  // A chunk's softmax in a unit whose value scales lie far apart: that of
  // q8_attend.cu's apart_softmax. `sc`, `oc`: S and O of the warp's rows, lo and hi
  // count from the chunk's first key, `tile` is its V.
  struct Sums {
    float m, M, l;
  };
  static __device__ __forceinline__ Sums apart_softmax(uint32_t sc, uint32_t oc, int pid, float ks,
                                                    float vlog, int shift, float qf, int lo, int hi,
                                                    const unsigned char* tile, bool begun, float m,
                                                    float M, float l) {
    const int lane = threadIdx.x & 31;
    const uint32_t rooms = rooms_of(tile, lane);
    float top = m, ref = -INFINITY, most = 0.f;
#pragma unroll 1
    for (int g = 0; g < 8; ++g) {
      uint32_t y[16], rw[4];
      tc::ld16_sync(sc + 16 * g, y);
      const int src = (16 * g) >> shift;
      const float cg = fmaxf(qf * __shfl_sync(0xffffffffu, ks, src), 1.17549435e-38f);
      const float lg = fmaxf(__shfl_sync(0xffffffffu, vlog, src), -126.f);
      const bool there = __shfl_sync(0xffffffffu, pid, src) >= 0;
      const int from = there ? lo - 16 * g : 16, to = hi - 16 * g;
#pragma unroll
      for (int k = 0; k < 4; ++k) rw[k] = __shfl_sync(0xffffffffu, rooms, 4 * g + k);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        if (e < from || e >= to) continue;
        const float x = __fmul_rn(__uint_as_float(y[e]), cg);
        const uint32_t room = rw[e >> 2] >> 8 * (e & 3) & 7u;
        top = fmaxf(top, x);
        if (room != q8::kNoCode) ref = fmaxf(ref, x + lg - (float)(room + 10u));
      }
    }
    if (begun) {
#pragma unroll 1
      for (int q4 = 0; q4 < 8; ++q4) {
        uint32_t o[16];
        tc::ld16_sync(oc + 16 * q4, o);
#pragma unroll
        for (int e = 0; e < 16; ++e) most = fmaxf(most, fabsf(__uint_as_float(o[e])));
      }
    }
    const float before = M;
    M = q8::apart_reference(before, ref, most);
    if (__any_sync(0xffffffffu, most > 0.f && M != before)) {
      // in two factors: M may fall by more than fp32's range
      const float half = most > 0.f ? ptx::ex2(0.5f * (before - M)) : 1.f;
#pragma unroll 1
      for (int q4 = 0; q4 < 8; ++q4) {
        uint32_t o[16];
        tc::ld16_sync(oc + 16 * q4, o);
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * half * half);
        tc::st16(oc + 16 * q4, o);
      }
    }
    const float base = top == -INFINITY ? 0.f : top, oref = M == -INFINITY ? 0.f : M;
    float sum = 0.f;
#pragma unroll 1
    for (int g = 0; g < 8; ++g) {
      uint32_t y[16], rw[4], p[8];
      tc::ld16_sync(sc + 16 * g, y);
      const int src = (16 * g) >> shift;
      const float cg = fmaxf(qf * __shfl_sync(0xffffffffu, ks, src), 1.17549435e-38f);
      const float lg = __shfl_sync(0xffffffffu, vlog, src);
      const bool there = __shfl_sync(0xffffffffu, pid, src) >= 0;
      const int from = there ? lo - 16 * g : 16, to = hi - 16 * g;
      const float off = there ? base - oref + lg : 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) rw[k] = __shfl_sync(0xffffffffu, rooms, 4 * g + k);
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        float r[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float d = __fadd_rn(__fmul_rn(__uint_as_float(y[e + k]), cg), -base);
          const bool seen = e + k >= from && e + k < to;
          const uint32_t room = rw[e >> 2] >> 8 * ((e + k) & 3) & 7u;
          sum += seen ? ptx::ex2(d) : 0.f;
          // (values of zeros or NaN: any finite weight does)
          r[k] = seen && room != q8::kNoCode ? ptx::ex2(d + off) : 0.f;
        }
        p[e / 2] = pack_half(r[0], r[1]);
      }
      tc::st8(sc + 8 * g, p);
    }
    return Sums{top, M, l * ptx::ex2(m - base) + sum};
  }
  static __device__ __noinline__ Sums apart_call(uint32_t sc, uint32_t oc, int pid, float ks,
                                                 float vlog, int shift, float qf, int lo, int hi,
                                                 const unsigned char* tile, bool begun, float m,
                                                 float M, float l) {
    return apart_softmax(sc, oc, pid, ks, vlog, shift, qf, lo, hi, tile, begun, m, M, l);
  }

  // The unit's NaN marks, if any, are used up: every row's thread sees the same
  // flag and meets the others before and after they are cleared (two phases of
  // a barrier of 256, where a unit of one half arrives for both).
  __device__ void use_marks(const Unit& u, int slot) const {
    if (!*(volatile int*)&sm.bars.nan_flag[slot]) return;
    const int threads = u.rows > 128 ? 256 : 128;
    for (int phase = 0; phase < 2; ++phase) {
      for (int k = threads; k <= 256; k += 128) ptx::mbar_arrive(&sm.bars.marks);
      wait(&sm.bars.marks, phase, &sm.bars.abort, a.err);
      if (phase) break;
      for (int k = 128 * t + row; k < D * 8; k += threads) (&sm.nan_rows[slot][0][0])[k] = 0;
      if (t == 0 && row == 0) sm.bars.nan_flag[slot] = 0;
    }
  }

  template <bool SPLIT>
  __device__ void run(const Plan& pl, long X0, long X1, int cta, long V, int C) {
    Bars& B = sm.bars;
    volatile int* abort = &B.abort;
    const int lane = threadIdx.x & 31;
    q8::MergeMeta* mm = reinterpret_cast<q8::MergeMeta*>(a.meta);
    int tiles = 0, units = 0;
    int others = 0, splits = 0;  // half 0: units that half 1 had a part in; split ones
    int kv0 = 0;                 // the block's K and V tiles before the unit's
    Walk<SPLIT> w;
    for (w.start(a, pl, X0, X1); !w.done(); kv0 += 2 * w.n, w.next(a, pl)) {
      const Unit& u = w.u;
      // (a unit begins when both halves have ended the one before, so that the
      // converters, two units ahead at most, never reach a half's marks in use)
      const bool split = w.split();
      const int step = split ? 2 : 1;
      r1 = split ? 0 : 128 * t;
      if (t == 1) {
        ptx::mbar_arrive(&B.q_full[0]);
        if (u.rows <= r1) {
          wait(&B.q_full[0], w.seg, abort, a.err);
          continue;
        }
      }
      load_query(u, w.at.h);
      if (u.rows <= r1 + (row & ~31)) {  // no row of the warp is real
        for (int i = split ? t : 0; i < w.n; i += step) {
          wait(&B.s_full[t], tiles++, abort, a.err);
          ptx::mbar_arrive(&B.p_full[t]);
        }
        wait(&B.o_full[t], units++, abort, a.err);
        // (it reads the marks' flag when the others do: all values are in)
        if (split && t == 0) wait(&B.o_full[1], others, abort, a.err);
        others += u.rows > 128 || split;
        splits += split;
        if (split && t == 1)
          ptx::mbar_arrive(&B.stats_full);
        else
          use_marks(u, w.seg % kNanSlots);
        continue;
      }
      float m = -INFINITY, M = -INFINITY, l = 0.f;
      const int chunks = w.n, h = w.at.h;
      int key0 = w.key0(split ? t : 0);
      bool begun = false;
      int low = kFar, high = -kFar;  // log2 of the value scales so far
      Pages pg{page_of(a, u, key0, lane, shift), 0.f, 0.f, 0.f};
      pg.scales(a, h);
      // A chunk's V, for the weights of scales far apart. (Its tile waits for
      // nothing that waits for this softmax: the tile before it in the ring is K's,
      // or a V of which the products were issued ahead of these scores.)
      auto values = [&](int kv) {
        wait(&B.full[kv % kRing], kv / kRing, abort, a.err);
        return sm.kv[kv % kRing];
      };
      auto take = [&](const Sums& now) {
        m = now.m;
        M = now.M;
        l = now.l;
      };
#pragma unroll 1
      for (int i = split ? t : 0; i < chunks; i += step, key0 += step * CK) {
        Pages next{page_of(a, u, key0 + step * CK, lane, shift), 0.f, 0.f, 0.f};
        auto leave = [&] {  // P is written
          tc::st_wait();
          tc::fence_before_sync();
          ptx::mbar_arrive(&B.p_full[t]);
          pg = next;
          begun = true;
        };
        pg.lv = __log2f(pg.vs);
        const bool mine = lane < CK >> shift;
        const bool edge = (mine && pg.pid < 0) || key0 < lo || key0 + CK > hi;
        const bool there = mine && pg.pid >= 0;
        const int level = max(-kFar, __float2int_rd(pg.lv));
        // keys that some row does not see; or, rarely after a unit's first chunk,
        // scales beyond those before, or the smallest ones
        bool masked = __any_sync(0xffffffffu, edge || (there && (level < low || level > high)));
        bool small = false;
        if (masked) {
          const bool tiny = level <= (int)q8::kSmall;
          masked = __any_sync(0xffffffffu, edge);
          small = __any_sync(0xffffffffu, there && tiny);
          low = min(low, (int)__reduce_min_sync(0xffffffffu, there && !tiny ? level : kFar));
          high = max(high, (int)__reduce_max_sync(0xffffffffu, there ? level : -kFar));
        }
        float c[4], lv[4];  // of 32 scores each
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          c[g] = fmaxf(qf * __shfl_sync(0xffffffffu, pg.ks, (32 * g) >> shift), 1.17549435e-38f);
          lv[g] = __shfl_sync(0xffffffffu, pg.lv, (32 * g) >> shift);
        }
        wait(&B.s_full[t], tiles++, abort, a.err);
        tc::fence_after_sync();
        const uint32_t sc = tl + s_col(t);
        const bool far = high - low > q8::spread<__nv_bfloat16>();
        const int kv = kv0 + 2 * i + (split && i < chunks - 1 ? 2 : 1);  // the chunk's V tile
        // (a call here: inline, here or below, the split kernel's chunks take 4 to 9 %
        // longer; the other's take 3 % longer with it, and 1 % less as below)
        if (SPLIT && __builtin_expect(far, 0)) {
          next.scales(a, h);
          take(apart_call(sc, tl + o_col(t), pg.pid, pg.ks, pg.lv, shift, qf, lo - key0, hi - key0,
                          values(kv), begun, m, M, l));
          leave();
          continue;
        }
        float top = m, ref = M;
        uint32_t z0[32], z1[32];
        if (!masked) {
          // (the next 32 scores are on their way from tensor memory meanwhile)
          tc::ld32_nowait(sc, z0);
          tc::ld_wait32(z0);
#pragma unroll
          for (int g = 0; g < 4; g += 2) {
            tc::ld32_nowait(sc + 32 * g + 32, z1);
            largest(z0, c[g], lv[g], top, ref);
            tc::ld_wait32(z1);
            tc::ld32_nowait(sc + (32 * g + 64) % 128, z0);  // at the end: for the weights
            largest(z1, c[g + 1], lv[g + 1], top, ref);
            tc::ld_wait32(z0);
          }
        } else {
#pragma unroll 1
          for (int g = 0; g < 8; ++g) {
            uint32_t y[16];
            tc::ld16_sync(sc + 16 * g, y);
            const int src = (16 * g) >> shift;
            const float cg = fmaxf(qf * __shfl_sync(0xffffffffu, pg.ks, src), 1.17549435e-38f);
            const float lg = __shfl_sync(0xffffffffu, pg.lv, src);
            const int pid = __shfl_sync(0xffffffffu, pg.pid, src);
            const int from = pid >= 0 ? lo - key0 - 16 * g : 16, to = hi - key0 - 16 * g;
            float x = -INFINITY;
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (e >= from && e < to) x = fmaxf(x, __uint_as_float(y[e]));
            x *= cg;
            top = fmaxf(top, x);
            ref = fmaxf(ref, x + fmaxf(lg, -126.f) - 10.f);
          }
        }
        next.scales(a, h);  // on their way during the exponentials
        if (!SPLIT && __builtin_expect(far, 0)) {
          take(apart_softmax(sc, tl + o_col(t), pg.pid, pg.ks, pg.lv, shift, qf, lo - key0,
                             hi - key0, values(kv), begun, m, M, l));
          leave();
          continue;
        }
        const float base = top == -INFINITY ? 0.f : top;
        l *= ptx::ex2(m - base);
        m = top;
        // M follows when it has fallen behind; O is then rescaled. (S being
        // full, the products before it, O's included, are complete.)
        const bool move = ref > M + kLag;
        const float ao = move && M != -INFINITY ? ptx::ex2(M - ref) : 1.f;
        if (move) M = ref;
        if ((SPLIT ? begun : i > 0) && __any_sync(0xffffffffu, ao != 1.f)) {
#pragma unroll 1
          for (int q4 = 0; q4 < 8; ++q4) {
            uint32_t o[16];
            const uint32_t oc = tl + o_col(t) + q4 * 16;
            tc::ld16_sync(oc, o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * ao);
            tc::st16(oc, o);
          }
        }
        const float oref = M == -INFINITY ? 0.f : M;
        // (M is at most the maximum's with the largest scale: p * vscale vanishes
        // before p does beside the smallest scales only)
        const bool apart = __any_sync(0xffffffffu, small || fabsf(base) > 4194304.f);
        float sum = 0.f;
        if (!masked && !apart) {
#pragma unroll
          for (int g = 0; g < 4; g += 2) {
            tc::ld32_nowait(sc + 32 * g + 32, z1);
            weights(z0, sc + 16 * g, c[g], lv[g], oref, base, sum);
            tc::ld_wait32(z1);
            if (g == 0) tc::ld32_nowait(sc + 64, z0);
            weights(z1, sc + 16 * g + 16, c[g + 1], lv[g + 1], oref, base, sum);
            if (g == 0) tc::ld_wait32(z0);
          }
        } else {
          // keys that the row does not see; and p for itself, from a rounded
          // score (see q8_attend.cu)
#pragma unroll 1
          for (int g = 0; g < 8; ++g) {
            const int src = (16 * g) >> shift;
            const float cg = fmaxf(qf * __shfl_sync(0xffffffffu, pg.ks, src), 1.17549435e-38f);
            const float lg = __shfl_sync(0xffffffffu, pg.lv, src);
            const int pid = __shfl_sync(0xffffffffu, pg.pid, src);
            uint32_t y[16], p[8];
            tc::ld16_sync(sc + 16 * g, y);
            const int from = pid >= 0 ? lo - key0 - 16 * g : 16, to = hi - key0 - 16 * g;
            const float off = pid >= 0 ? base - oref + lg : 0.f;
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              float r[2];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const float d = __fadd_rn(__fmul_rn(__uint_as_float(y[e + k]), cg), -base);
                const bool seen = e + k >= from && e + k < to;
                sum += seen ? ptx::ex2(d) : 0.f;
                r[k] = seen ? ptx::ex2(d + off) : 0.f;
              }
              p[e / 2] = pack_half(r[0], r[1]);
            }
            tc::st8(sc + 8 * g, p);
          }
        }
        l += sum;
        leave();
      }

      // ---- epilogue ----
      wait(&B.o_full[t], units++, abort, a.err);
      tc::fence_after_sync();
      const int r = u.r0 + r1 + row;
      const bool real = r < u.s.n * a.G;
      const bool whole = w.first == 0 && w.ends();
      const float base = m == -INFINITY ? 0.f : m, oref = M == -INFINITY ? 0.f : M;
      // in two factors: 2^(M - m) alone can leave fp32's range
      const float half = ptx::ex2(0.5f * (oref - base));
      float f = l == 0.f ? 0.f : half / l;
      float lse2 = l == 0.f ? -INFINITY : m + log2f(l);
      float half1 = 0.f, f1 = 0.f;
      if (split) {
        // half 1 leaves its sums to half 0, which reads its O too (the next unit
        // begins behind that)
        if (t == 1) {
          sm.stats[0][row] = half;
          sm.stats[1][row] = f;
          sm.stats[2][row] = lse2;
          ptx::mbar_arrive(&B.stats_full);
          continue;
        }
        wait(&B.o_full[1], others, abort, a.err);
        wait(&B.stats_full, splits++, abort, a.err);
        tc::fence_after_sync();
        half1 = sm.stats[0][row];
        const float lse1 = sm.stats[2][row], top = fmaxf(lse2, lse1);
        const float b2 = top == -INFINITY ? 0.f : top;
        const float w0 = ptx::ex2(lse2 - b2), w1 = ptx::ex2(lse1 - b2), sum = w0 + w1;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        f *= w0 * inv;
        f1 = sm.stats[1][row] * w1 * inv;
        lse2 = sum == 0.f ? -INFINITY : top + log2f(sum);
      }
      others += u.rows > 128 || split;
      const int slot = w.seg % kNanSlots;
      const bool nan = *(volatile int*)&B.nan_flag[slot] != 0;
      float* part = a.part + (2l * cta + (w.first > 0 ? 0 : 1)) * kPart;
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + (real ? out_row(u, w.at.h, r) : 0) * D;
#pragma unroll 1
      for (int q4 = 0; q4 < 4; ++q4) {
        uint32_t o[32];
        tc::ld32_sync(tl + o_col(t) + 32 * q4, o);
        float y[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) y[e] = __uint_as_float(o[e]) * half * f;
        if (split) {
          tc::ld32_sync(tl + o_col(1) + 32 * q4, o);
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] = fmaf(__uint_as_float(o[e]) * half1, f1, y[e]);
        }
        if (!real) continue;
        if (nan) {
          const int tk = r / a.G - u.tok0;
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (sm.nan_rows[slot][32 * q4 + e][tk >> 5] >> (tk & 31) & 1u)
              y[e] = __uint_as_float(0x7fffffffu);
        }
        if (whole) {
#pragma unroll
          for (int e = 0; e < 32; e += 16) store32(dst + 32 * q4 + e, &y[e]);
        } else {
          float4* to = reinterpret_cast<float4*>(part) + 8 * q4 * ROWS + r1 + row;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            to[e * ROWS] = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
        }
      }
      if (real) {
        if (whole) {
          if (a.lse) a.lse[out_row(u, w.at.h, r)] = lse2 * q8::kLn2;
        } else {
          part[(long)ROWS * D + r1 + row] = lse2;
        }
      }
      if (t == 0 && row == 0 && w.first > 0 && w.ends()) {
        mm[cta].unit = (long)w.at.tile * a.Hkv + w.at.h;
        mm[cta].from = q8::block_of(w.x - w.at.c + kQ8TcUnit, V, C);
      }
      use_marks(u, slot);
    }
  }
};

template <bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    q8_prefill_tc_kernel(const __grid_constant__ Q8AttendArgs a) {
  extern __shared__ unsigned char raw[];
  Smem& sm = *reinterpret_cast<Smem*>(
      (reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  Bars& B = sm.bars;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int t = 0; t < 2; ++t) {
      ptx::mbar_init(&B.q_full[t], t == 0 ? 256 : 128);
      ptx::mbar_init(&B.s_full[t], 1);
      ptx::mbar_init(&B.p_full[t], 128);
      ptx::mbar_init(&B.o_full[t], 1);
    }
    for (int k = 0; k < kRing; ++k) {
      ptx::mbar_init(&B.full[k], 128);
      ptx::mbar_init(&B.empty[k], 1);
    }
    for (int k = 0; k < kRaw; ++k) {
      ptx::mbar_init(&B.raw_full[k], 1);
      ptx::mbar_init(&B.raw_empty[k], 128);
    }
    ptx::mbar_init(&B.fin, 1);
    ptx::mbar_init(&B.marks, 256);
    ptx::mbar_init(&B.stats_full, 128);
    B.abort = 0;
    for (int k = 0; k < kNanSlots; ++k) B.nan_flag[k] = 0;
    ptx::fence_mbar_init();
  }
  for (int k = tid; k < kNanSlots * D * 8; k += kThreads) (&sm.nan_rows[0][0][0])[k] = 0;
  if (warp == 13) {
    tc::tmem_alloc(&B.tmem, 512);
    tc::tmem_relinquish();
  }
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();

  Plan pl{a.plan_pre, a.plan_seq, a.plan_base, nullptr, a.plan_base[a.B], 0};
  const long V = pl.tiles ? pl.pre[pl.tiles] : 0;
  // (two places a block: one chunk of every unit that goes on in it)
  const int C = (int)max(1l, min((long)gridDim.x, (SPLIT ? V / 2 : V)));
  const int cta = blockIdx.x;
  if (tid == 0) reinterpret_cast<q8::MergeMeta*>(a.meta)[cta].unit = -1;
  __syncthreads();
  if (cta < C && V > 0) {
    const long X0 = q8::split(V, cta, C), X1 = q8::split(V, cta + 1, C);
    const int shift = __ffs(a.page) - 1;
    if (warp < 8) {
      Softmax s{a, sm, warp >> 2, (warp & 3) * 32 + lane, 0,
                B.tmem + ((uint32_t)((warp & 3) * 32) << 16), shift, 0.f, 0, 0};
      s.run<SPLIT>(pl, X0, X1, cta, V, C);
    } else if (warp < 12) {
      Converter{a, warp - 8, lane, shift}.run<SPLIT>(pl, X0, X1, sm);
    } else if (warp == 12) {
      copy_pages<SPLIT>(a, pl, X0, X1, sm, shift, lane);
    } else {
      issue_mmas<SPLIT>(a, pl, X0, X1, sm);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 13) tc::tmem_dealloc(B.tmem, 512);
}

// Joins the partials of a unit that lies in several blocks (see q8_attend.cuh):
// block (c, y) does components 16 y .. 16 y + 15 of the unit that ends in
// attention block c, a thread per row.
constexpr int kMergeCols = 16;
__global__ void __launch_bounds__(ROWS)
    q8_prefill_tc_merge_kernel(const __grid_constant__ Q8AttendArgs a) {
  ptx::grid_dep_wait();
  const q8::MergeMeta mm = reinterpret_cast<const q8::MergeMeta*>(a.meta)[blockIdx.x];
  if (mm.unit < 0) return;
  const int row = threadIdx.x, col = kMergeCols * blockIdx.y;
  const int tile = (int)(mm.unit / a.Hkv), h = (int)(mm.unit % a.Hkv);
  const int b = a.plan_seq[tile];
  const int r = (tile - a.plan_base[b]) * ROWS + row;
  int first, n;
  q8::token_range(a.cu, b, a.N, first, n);
  if (r >= n * a.G) return;
  const int np = (int)blockIdx.x - mm.from + 1;
  auto part = [&](int i) { return a.part + (2l * (mm.from + i) + (i == 0 ? 1 : 0)) * kPart; };
  float top = -INFINITY;
#pragma unroll 4
  for (int i = 0; i < np; ++i) top = fmaxf(top, part(i)[(long)ROWS * D + row]);
  const float base = top == -INFINITY ? 0.f : top;
  float acc[kMergeCols] = {}, sum = 0.f;
#pragma unroll 2
  for (int i = 0; i < np; ++i) {
    const float* p = part(i);
    const float w = ptx::ex2(p[(long)ROWS * D + row] - base);
    sum += w;
#pragma unroll
    for (int e = 0; e < kMergeCols / 4; ++e) {
      const float4 x = reinterpret_cast<const float4*>(p)[(col / 4 + e) * ROWS + row];
      acc[4 * e] = fmaf(w, x.x, acc[4 * e]);
      acc[4 * e + 1] = fmaf(w, x.y, acc[4 * e + 1]);
      acc[4 * e + 2] = fmaf(w, x.z, acc[4 * e + 2]);
      acc[4 * e + 3] = fmaf(w, x.w, acc[4 * e + 3]);
    }
  }
  const float f = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int e = 0; e < kMergeCols; ++e) acc[e] *= f;
  const long out = ((long)first + r / a.G) * a.Hq + h * a.G + r % a.G;
  store32(static_cast<__nv_bfloat16*>(a.out) + out * D + col, acc);
  if (col == 0 && a.lse) a.lse[out] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * q8::kLn2;
}

}  // namespace

bool q8_prefill_tc_shape(const nsa_params& p) {
  return p.dtype == NSA_DTYPE_BF16 && p.d == D && p.sel_block >= 32;
}

size_t q8_prefill_tc_part_bytes() { return (size_t)kPart * 4 * 2 * kQ8MaxBlocks; }

cudaError_t launch_q8_prefill_tc(const Q8AttendArgs& a, bool split, cudaStream_t stream) {
  constexpr int smem = sizeof(Smem) + 1024;
  cudaError_t e;
  auto kern = split ? q8_prefill_tc_kernel<true> : q8_prefill_tc_kernel<false>;
  if ((e = ensure_dyn_smem((const void*)kern, smem)) != cudaSuccess) return e;
  {
    TraceScope trace("q8_prefill_tc", stream);
    if ((e = q8::launch_pdl(kern, dim3(a.blocks), dim3(kThreads), smem, stream, a)) !=
        cudaSuccess)
      return e;
  }
  TraceScope trace("q8_prefill_tc_merge", stream);
  return q8::launch_pdl(q8_prefill_tc_merge_kernel, dim3(a.blocks, D / kMergeCols),
                        dim3(ROWS), 0, stream, a);
}

}  // namespace nsa
