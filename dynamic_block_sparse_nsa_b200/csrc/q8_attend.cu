// Attention over the 8-bit paged cache (nsa_decode_q8, and nsa_prefill_q8 where
// the tensor-memory kernel does not apply): any group size, page and dtype.
//
//   z2 = (q . kcode) * kscale[page] * softmax_scale * log2(e)
//   o  = sum_keys 2^(z2 - m) * vscale[page] * vcode / sum_keys 2^(z2 - m)
//
// One pass with the running maximum m and sum l of each row. A single query's
// attention reads every live code once and does 4 G flops a byte-pair, so it is
// bound by HBM; the kernel streams codes and does the products on the warp
// tensor cores (m16n8k16, 16 query rows of a unit, fp32 accumulators). Codes
// become halves exactly (e4m3 is a subset of fp16). fp32 rows are kept as two
// halves each, q = hi + lo and p = hi + lo (22 significant bits), bf16 rows as
// one: q is scaled by a power of two per row into the top of fp16's range, so
// its 8 bits stay exact, and p's rounding (2^-11 relative) is below that of
// the bf16 output (2^-8).
//
// A page's value scale multiplies p before p is rounded to half. So that no
// spread of scales over the pages can push it out of fp16's range, the output
// has a running reference of its own: o is kept in units of 2^M with M the
// largest m_page + log2(vscale) so far (less 10, which puts p * vscale in
// (0, 1024] and its smallest normal 2^-24 below the largest). A scale says
// little of what a row sees: it may be that of a later token, of one before the
// window, or of one written over since. So once the scales of a warp's pages lie
// too far apart (q8::spread), M is the largest p * max |v| of a single key instead,
// and falls to what o holds where an earlier page had set it too high
// (apart_softmax).
//
// Each warp streams its own contiguous share of the chunks (64 keys) through a
// private ring of three cp.async slots, each K or V of a chunk, two of them in
// flight while the third is computed on (no block-wide barrier in the loop).
// Rows outside the sequence, the window or the list are filled with zeros by
// the copy, so no stale byte reaches a product. Lane (g, t) of a B fragment
// reads 16 bytes of key g (K: 16 components, the product's k index permuted
// the same way in q) or the same 16 components of four keys (V), so no
// transposition is needed; the slots' swizzles make both conflict-free.
//
// Measured, 64 query heads on 4 KV heads, d = 128, bf16: one query of each of 32
// sequences of 65536 tokens 330 us, 6.5 TB/s of codes, the rate of a copy; in
// long runs of such calls 370 to 400 us, at the board's power limit. A short call
// is latency: of one key 8.6 us (1.7 of it an empty kernel's; lengths, plan, page,
// scale, codes and query one behind the other, and instructions that no loop has
// warmed the cache with, which are most of its stalls), 2 to 3 for the join of a
// block's warps and as much for a second pass of them: 1000 tokens 14.8 us, of 0.16
// for the bytes. fp32 does each product twice and splits every p, and eight warps
// do not hide the latencies between (issue slots 30 % used, tensor pipe 26 %): 24
// sequences of up to 9001 tokens (40 heads on 8, d = 64) 56 us of 17. More than 16
// heads to a KV head read the codes once for every 16. Value scales too far apart
// take 2 to 2.5 times as long (32 x 16384 tokens 99 and 244 us); the look-out for
// them costs bf16 calls 0 to 3 %, fp32 ones 2 to 5. What was measured slower:
// prefetches of pages into L2 (518 us), chunks of 32 keys (531 us), twelve warps a
// block (fp32 64 us), one copy of the loop's body for both kinds of chunk (350).
#include <algorithm>

#include "q8_attend.cuh"

namespace nsa {
namespace {

using q8::Place;
using q8::Plan;
using q8::Seq;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int CK = 64;       // keys per chunk
constexpr int NS = CK / 8;   // score tiles of 8 keys
constexpr int ROWS = 16;     // query rows per tile
constexpr int kUnitChunks = 4 * kWarps;  // most chunks of a unit that one block takes whole
constexpr int SLOTS = 3;     // of a warp's ring
constexpr int kSmemTiles = 1024;  // tiles whose prefix a block computes itself
constexpr int kFar = 1 << 20;     // beyond every scale's exponent
// First key of an absent page: past every row (of a sequence of up to 2^30 tokens),
// its last still an int.
constexpr int kAbsent = INT_MAX - CK;

template <int D>
struct Geo {
  static constexpr int TILE = CK * D;             // bytes of K or V of a chunk
  static constexpr int RING = SLOTS * TILE;       // a warp's ring
  static constexpr int PART = ROWS * D + ROWS;    // floats of a partial: o, lse2
  static_assert(RING >= PART * 4, "a warp's last partial goes into its ring");
};

// What the computing side needs of a chunk; two chunks are under way.
template <int PP>
struct ChunkMeta {
  float ks[PP], vs[PP];
  int kb[PP];  // position of each page's first key in the chunk
  int state;   // 0: no key of the chunk is seen; 1: some; 2: every key by every row
};

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ float2 unpack_half(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// Four e4m3 codes as two pairs of halves.
__device__ __forceinline__ void e4m3x4_to_half2x2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}

__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

// Byte offset of 16-byte piece c of key r inside a K or V slot. K rows are
// read eight keys at a time (r, r + 4 in one quarter-warp phase), V rows four
// (r .. r + 3) with neighbouring pieces.
template <int D>
__device__ __forceinline__ uint32_t k_off(int r, int c) {
  if (D == 128) return r * 128 + ((c ^ (r & 7)) << 4);
  return ((r & ~7) | ((r & 3) << 1) | ((r >> 2) & 1)) * 64 + (c << 4);
}
template <int D>
__device__ __forceinline__ uint32_t v_off(int r, int c) {
  if (D == 128) return r * 128 + ((c ^ ((r & 3) << 1)) << 4);
  return r * 64 + ((c ^ (r & 2)) << 4);
}

__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

// A unit's sequence and row range.
struct Unit {
  int b, r0, lo, hi;
  Seq s;
  __device__ __forceinline__ void load(const Q8AttendArgs& a, const Plan& pl, int tile) {
    if (pl.tseq) {
      b = pl.tseq[tile];
      r0 = (tile - pl.tbase[b]) * ROWS;
      s = q8::sequence(a, b);
    } else {
      b = tile / pl.rt;
      r0 = (tile - b * pl.rt) * ROWS;
      s.first = b;
      s.n = 1;
      s.len = pl.lens[tile];
      s.ok = s.len >= 0;
      if (!s.ok) s.len = 0;
    }
    q8::key_span(a, s, r0, ROWS, lo, hi);
  }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// The copying side of a warp: its place, the pages ahead of it (one per lane)
// and the chunk being copied.
template <int D, int PP>
struct Feeder {
  static constexpr int PIECES = D / 16, RPI = 32 / PIECES;  // a copy's 512 bytes: RPI rows
  Place at;
  Unit u;
  int gbase;       // entry held by lane 0
  int pid, blk;    // this lane's page and its block number; -1: none
  float ks, vs;
  int cp[PP], ckb[PP], coff;  // the chunk's pages, their first keys, the first key's slot
  int centry;                 // and its first entry
  bool whole;                 // every row of the chunk is a live key
  __device__ __forceinline__ void pages(const Q8AttendArgs& a, int e, int lane) {
    gbase = e;
    const int i = e + lane;
    blk = -1;
    if (a.keys == q8::KEYS_BLOCKS) {
      const int32_t* list = a.sel + ((long)u.b * a.Hkv + at.h) * a.n;
      if (i < a.n) blk = list[i];
      if (blk < 0 || (long)blk * a.page >= u.hi) blk = -1;
      // a block listed twice counts once
      const unsigned same = __match_any_sync(0xffffffffu, blk);
      if (blk >= 0 && (same & ((1u << lane) - 1))) blk = -1;
      for (int k = 0; k < e; ++k)
        if (list[k] == blk) blk = -1;
    } else if ((long)i * a.page < u.hi && (long)(i + 1) * a.page > u.lo) {
      blk = i;  // (a page before the window may be gone)
    }
    pid = blk >= 0 ? a.table[(long)u.b * a.max_pages + blk] : -1;
    if (blk >= 0 && (pid < 0 || pid >= a.num_pages)) {
      atomicOr(a.err, kErrPage);
      pid = blk = -1;
    }
    ks = 0.f;
    vs = 1.f;
    if (pid >= 0) {
      ks = a.k_scale[(long)pid * a.Hkv + at.h];
      vs = a.v_scale[(long)pid * a.Hkv + at.h];
    }
  }

  __device__ __forceinline__ void start(const Q8AttendArgs& a, const Plan& pl, long x) {
    at.init(pl, a.Hkv, x);
    u.load(a, pl, at.tile);
    gbase = INT_MIN / 2;
  }

  // The pages of the chunk at the place.
  __device__ __forceinline__ void look(const Q8AttendArgs& a, ChunkMeta<PP>* meta, int lane) {
    const int ch = at.c + (a.keys == q8::KEYS_BLOCKS ? 0 : u.lo / CK);
    const int shift = __ffs(a.page) - 1;  // (a sequence or a list has up to 2^30 keys)
    const int e = (ch * CK) >> shift;
    coff = PP == 1 ? ch * CK & (a.page - 1) : 0;
    if (e + PP > gbase + 32 || e < gbase) pages(a, e, lane);
    constexpr int w = CK / PP;
    // rows of the tile see from the first token's window to the last token's
    // position; all of them see [full_lo, full_hi)
    const int t0 = u.r0 / a.G, t1 = min(u.s.n - 1, (u.r0 + ROWS - 1) / a.G);
    const int at0 = u.s.len - u.s.n;
    const int full_hi = u.hi > 0 ? at0 + t0 + 1 : 0;
    const int full_lo = a.keys == q8::KEYS_WINDOW ? at0 + t1 + 1 - a.window : 0;
    bool some = false, full = true;
    whole = true;
#pragma unroll
    for (int i = 0; i < PP; ++i) {
      const int src = e - gbase + i;
      cp[i] = __shfl_sync(0xffffffffu, pid, src);
      ckb[i] = __shfl_sync(0xffffffffu, blk, src) * a.page + coff;
      if (cp[i] < 0) ckb[i] = kAbsent;
      some |= ckb[i] < u.hi && ckb[i] + w > u.lo;
      full &= ckb[i] >= full_lo && ckb[i] + w <= full_hi;
      whole &= ckb[i] >= u.lo && ckb[i] + w <= u.hi;
      if (lane == 0) meta->kb[i] = ckb[i];
    }
    if (lane == 0) meta->state = some ? (full ? 2 : 1) : 0;
    centry = e;
  }

  // Their scales: behind the copies, which do not need them.
  __device__ __forceinline__ void scales(ChunkMeta<PP>* meta, int lane) {
#pragma unroll
    for (int i = 0; i < PP; ++i) {
      const int src = centry - gbase + i;
      const float k = __shfl_sync(0xffffffffu, ks, src), v = __shfl_sync(0xffffffffu, vs, src);
      if (lane == 0) {
        meta->ks[i] = k;
        meta->vs[i] = v;
      }
    }
  }

  // Whether the value scales of the unit's pages lie far apart, those just looked
  // up among them. `range`: the warp's, log2 of the least and the largest so far.
  __device__ __forceinline__ bool far(int* range, bool begun, int spread, int lane) const {
    const int level = max(-kFar, __float2int_rd(__log2f(vs)));
    int low = __reduce_min_sync(0xffffffffu, pid >= 0 && level > (int)q8::kSmall ? level : kFar);
    int high = __reduce_max_sync(0xffffffffu, pid >= 0 ? level : -kFar);
    if (begun) {
      low = min(low, range[0]);
      high = max(high, range[1]);
    }
    __syncwarp();
    if (lane == 0) {
      range[0] = low;
      range[1] = high;
    }
    return high - low > spread;
  }

  // Copies K or V of the chunk into a slot.
  template <bool V>
  __device__ __forceinline__ void copy(const Q8AttendArgs& a, uint32_t slot, int lane) {
    const int c = lane % PIECES, rl = lane / PIECES;
    const uint8_t* base = V ? a.v_pages : a.k_pages;
    // copy i's rows lie 512 i bytes behind copy 0's, in the page and in the
    // slot, but for the bit of a K row's swizzle that alternates
    const uint32_t d0 = slot + (V ? v_off<D>(rl, c) : k_off<D>(rl, c));
    const uint32_t d1 = D == 128 && !V ? d0 ^ 64 : d0;
#pragma unroll
    for (int p = 0; p < PP; ++p) {
      const uint8_t* src =
          base + (((long)cp[p] * a.Hkv + at.h) * a.page + coff + rl) * D + c * 16;
      if (whole) {
#pragma unroll
        for (int k = 0; k < CK / PP / RPI; ++k) {
          const int i = p * (CK / PP / RPI) + k;
          cp_async16((i & 1 ? d1 : d0) + 512 * i, src + 512 * k);
        }
      } else {
#pragma unroll
        for (int k = 0; k < CK / PP / RPI; ++k) {
          const int i = p * (CK / PP / RPI) + k;
          const int pos = ckb[p] + k * RPI + rl;
          const bool live = pos >= u.lo && pos < u.hi;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((i & 1 ? d1 : d0) +
                                                                               512 * i),
                       "l"(live ? src + 512 * k : base), "r"(live ? 16 : 0)
                       : "memory");
        }
      }
    }
  }

  __device__ __forceinline__ void next(const Q8AttendArgs& a, const Plan& pl) {
    const int tile = at.tile;
    if (!at.next(pl, a.Hkv)) return;
    gbase = INT_MIN / 2;
    if (at.tile != tile && at.tile < pl.tiles) u.load(a, pl, at.tile);
  }
};

// The computing side: a unit's query rows and its running softmax.
template <typename T, int D>
struct Rows {
  static constexpr int PARTS = sizeof(T) == 4 ? 2 : 1;
  static constexpr int KS = D / 16;  // product steps of 16 components
  static constexpr int NT = D / 8;   // output tiles of 8 components
  uint32_t q[PARTS][KS][4];
  float qf[2];        // row factor of the scores (> 0): 2^shift * |softmax_scale| * log2(e)
  int lo[2], hi[2];   // keys the lane's two rows see
  float o[NT][4];
  float m[2], l[2], M[2];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < NT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    m[0] = m[1] = M[0] = M[1] = -INFINITY;
    l[0] = l[1] = 0.f;
  }

  // Row r of a sequence in q / out: its token's head.
  static __device__ __forceinline__ long row_of(const Q8AttendArgs& a, const Seq& s, int h, int r) {
    return ((long)s.first + r / a.G) * a.Hq + h * a.G + r % a.G;
  }

  // The lane's components of its two query rows, as they are in memory.
  struct Raw {
    uint4 x[2][D / 32 * PARTS];
  };
  __device__ __forceinline__ void fetch(Raw& raw, const Q8AttendArgs& a, const Unit& u, int h,
                                        int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = u.r0 + g + 8 * i;
      const bool real = r < u.s.n * a.G;
      const T* src = static_cast<const T*>(a.q) + (real ? row_of(a, u.s, h, r) : 0) * D + 16 * t;
      // components of step 4 half + j are 16 (4 half + t) + 4 j ..
#pragma unroll
      for (int c = 0; c < D / 32 * PARTS; ++c) {
        const int half = c / (2 * PARTS), piece = c % (2 * PARTS);
        raw.x[i][c] = real ? __ldg(reinterpret_cast<const uint4*>(src + 64 * half) + piece)
                           : make_uint4(0, 0, 0, 0);
      }
    }
  }

  __device__ __forceinline__ void load(const Raw& raw, const Q8AttendArgs& a, const Unit& u,
                                       int lane) {
    const int g = lane >> 2;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = u.r0 + g + 8 * i;
      const bool real = r < u.s.n * a.G;
      const int pos = u.s.len - u.s.n + r / a.G;
      hi[i] = real && u.hi > 0 ? pos + 1 : 0;
      lo[i] = a.keys == q8::KEYS_WINDOW ? max(0, pos + 1 - a.window) : 0;
      float x[D / 4];
      uint32_t m2 = 0;  // largest magnitudes of the even and odd components (bf16)
      float big = 0.f;
#pragma unroll
      for (int c = 0; c < D / 32 * PARTS; ++c) {
        const uint4 v = raw.x[i][c];
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (PARTS == 2) {
            x[4 * c + k] = __uint_as_float(w[k]);
          } else {
            x[(8 * c + 2 * k) % (D / 4)] = __uint_as_float(w[k] << 16);
            x[(8 * c + 2 * k + 1) % (D / 4)] = __uint_as_float(w[k] & 0xffff0000u);
            m2 = __vmaxu2(m2, w[k] & 0x7fff7fffu);  // (order of bits: order of magnitudes)
          }
        }
      }
      if (PARTS == 1 && __vmaxu2(m2, 0x7f7f7f7fu) == 0x7f7f7f7fu) {  // all finite
        big = fmaxf(__uint_as_float(m2 << 16), __uint_as_float(m2 & 0xffff0000u));
      } else {
        // (an infinite component makes every score infinite or NaN: the row is NaN)
#pragma unroll
        for (int j = 0; j < D / 4; ++j) {
          if (fabsf(x[j]) < INFINITY)
            big = fmaxf(big, fabsf(x[j]));
          else
            x[j] = __uint_as_float(0x7fffffffu);
        }
      }
      big = quad_max(big);
      // 2^up brings the largest component to [2^14, 2^15)
      int up = big > 0.f ? 14 - ((int)(__float_as_uint(big) >> 23) - 127) : 0;
      up = min(max(up, -120), 120);
      // (a negative softmax scale's sign goes into q)
      const float mul = a.scale_log2 < 0.f ? -q8::exp2_int(up) : q8::exp2_int(up);
      qf[i] = q8::exp2_int(-up) * fabsf(a.scale_log2);
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const float u0 = x[4 * s + 2 * w] * mul, u1 = x[4 * s + 2 * w + 1] * mul;
          const uint32_t hi2 = pack_half(u0, u1);
          q[0][s][i + 2 * w] = hi2;
          if (PARTS == 2) {
            const float2 f = unpack_half(hi2);
            q[PARTS - 1][s][i + 2 * w] = pack_half(u0 - f.x, u1 - f.y);
          }
        }
    }
  }

  // z[nt][.]: q . kcode of keys 8 nt + t, 8 nt + t + 4 for rows g (0, 1) and g + 8 (2, 3)
  __device__ __forceinline__ void scores(float (&z)[NS][4], uint32_t kbase, int lane) {
    const int g = lane >> 2, t = lane & 3;
    const uint32_t k0 = kbase + k_off<D>((g >> 1) | ((g & 1) << 2), t);
#pragma unroll
    for (int nt = 0; nt < NS; ++nt) {
      z[nt][0] = z[nt][1] = z[nt][2] = z[nt][3] = 0.f;
      float low[4] = {0.f, 0.f, 0.f, 0.f};  // of q's second part: summed apart
#pragma unroll
      for (int half = 0; half < D / 64; ++half) {
        const uint4 v = lds128((half ? k0 ^ 64 : k0) + nt * 8 * D);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t b0, b1;
          e4m3x4_to_half2x2(w[j], b0, b1);
          mma_f16(z[nt], q[0][4 * half + j], b0, b1);
          if (PARTS == 2) mma_f16(low, q[PARTS - 1][4 * half + j], b0, b1);
        }
      }
      if (PARTS == 2) {
#pragma unroll
        for (int x = 0; x < 4; ++x) z[nt][x] += low[x];
      }
    }
  }

  template <int PP>
  __device__ __forceinline__ void mask(float (&z)[NS][4], const ChunkMeta<PP>& meta,
                                       int lane) const {
    const int t = lane & 3;
    constexpr int TP = NS / PP;
#pragma unroll
    for (int nt = 0; nt < NS; ++nt)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int key = meta.kb[nt / TP] + 8 * (nt % TP) + t + 4 * (x & 1);
        if (key < lo[x >> 1] || key >= hi[x >> 1]) z[nt][x] = -INFINITY;
      }
  }

  // code_room of the values of key r of a slot; NaN codes do not count.
  static __device__ __forceinline__ uint32_t room_of(const unsigned char* vst, int r, int lane) {
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      const uint4 v = *reinterpret_cast<const uint4*>(vst + r * D + (c + lane) % (D / 16) * 16);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t u = w[i] & 0x7f7f7f7fu;
        top = __vmaxu4(top, u & ~__vcmpeq4(u, 0x7f7f7f7fu));
      }
    }
    top = max(top & 0xffffu, top >> 16);
    return q8::code_room(max(top & 0xffu, top >> 8));
  }

  // The running softmax of a chunk in a unit whose value scales lie far apart. M is
  // the largest z2 + log2(vscale) - room of a key with values other than zero (less
  // 10), and what o holds; it may fall. p and p * vscale are exponentials of their
  // own: one may vanish and the other not.
  template <int PP>
  __device__ __forceinline__ void apart_softmax(float (&z)[NS][4], const ChunkMeta<PP>& meta,
                                                bool full, const unsigned char* vst, int lane) {
    const int t = lane & 3;
    constexpr int TP = NS / PP;
    if (!full) mask<PP>(z, meta, lane);
    float lv[PP];
#pragma unroll
    for (int p = 0; p < PP; ++p) lv[p] = __log2f(meta.vs[p]);
    uint32_t room[2] = {0, 0};  // of keys t, 8 + t, ..; 4 + t, 12 + t, ..: four bits each
    {
      const uint32_t a = room_of(vst, lane, lane), b = room_of(vst, lane + 32, lane);
#pragma unroll
      for (int nt = 0; nt < NS; ++nt)
#pragma unroll
        for (int y = 0; y < 2; ++y)
          room[y] |= __shfl_sync(0xffffffffu, nt < NS / 2 ? a : b, (8 * nt + t + 4 * y) % 32)
                     << 4 * nt;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float top = m[i], ref = -INFINITY, most_o = 0.f;
#pragma unroll
      for (int nt = 0; nt < NS; ++nt) {
        const float c = fmaxf(qf[i] * meta.ks[nt / TP], 1.17549435e-38f);
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const uint32_t r = room[y] >> 4 * nt & 15u;
          z[nt][2 * i + y] = __fmul_rn(z[nt][2 * i + y], c);
          top = fmaxf(top, z[nt][2 * i + y]);
          if (r != q8::kNoCode)
            ref = fmaxf(ref, z[nt][2 * i + y] + fmaxf(lv[nt / TP], -126.f) - (float)(r + 10u));
        }
      }
      top = quad_max(top);
      ref = quad_max(ref);
#pragma unroll
      for (int j = 0; j < NT; ++j)
        most_o = fmaxf(most_o, fmaxf(fabsf(o[j][2 * i]), fabsf(o[j][2 * i + 1])));
      most_o = quad_max(most_o);
      const float before = M[i];
      M[i] = q8::apart_reference(before, ref, most_o);
      if (__any_sync(0xffffffffu, most_o > 0.f && M[i] != before)) {
        // in two factors: M may fall by more than fp32's range
        const float half = most_o > 0.f ? ptx::ex2(0.5f * (before - M[i])) : 1.f;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          o[j][2 * i] = o[j][2 * i] * half * half;
          o[j][2 * i + 1] = o[j][2 * i + 1] * half * half;
        }
      }
      const float base = top == -INFINITY ? 0.f : top;
      const float oref = M[i] == -INFINITY ? 0.f : M[i];
      const float al = ptx::ex2(m[i] - base);
      m[i] = top;
      float sum = 0.f;
#pragma unroll
      for (int nt = 0; nt < NS; ++nt)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const float d = __fadd_rn(z[nt][2 * i + y], -base);
          sum += ptx::ex2(d);
          // (values of zeros or NaN: any finite weight does)
          z[nt][2 * i + y] = (room[y] >> 4 * nt & 15u) == q8::kNoCode
                                 ? 0.f
                                 : ptx::ex2(d + (base - oref + lv[nt / TP]));
        }
      l[i] = l[i] * al + sum;
    }
  }

  // Running softmax: z becomes p * vscale in units of 2^M; o, l, m, M follow.
  template <int PP>
  __device__ __forceinline__ void softmax(float (&z)[NS][4], const ChunkMeta<PP>& meta, bool full,
                                          int lane) {
    constexpr int TP = NS / PP;  // score tiles of a page
    if (!full) mask<PP>(z, meta, lane);
    float lv[PP];  // log2 of the value scales
#pragma unroll
    for (int p = 0; p < PP; ++p) lv[p] = __log2f(meta.vs[p]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float top = m[i], ref = M[i], c[PP];
#pragma unroll
      for (int p = 0; p < PP; ++p) {
        c[p] = fmaxf(qf[i] * meta.ks[p], 1.17549435e-38f);  // (a masked -inf stays -inf)
        float pm = -INFINITY;
#pragma unroll
        for (int nt = p * TP; nt < (p + 1) * TP; ++nt)
          pm = fmaxf(pm, fmaxf(z[nt][2 * i], z[nt][2 * i + 1]));
        pm = quad_max(pm) * c[p];
        top = fmaxf(top, pm);
        ref = fmaxf(ref, pm + fmaxf(lv[p], -126.f) - 10.f);
      }
      const float base = top == -INFINITY ? 0.f : top;
      const float oref = ref == -INFINITY ? 0.f : ref;
      const float al = ptx::ex2(m[i] - base), ao = ptx::ex2(M[i] - oref);
      m[i] = top;
      M[i] = ref;
      // p * vscale * 2^-M = 2^(z2 + log2(vscale) - M); p itself, for l, is
      // that times 2^-e, e = m + log2(vscale) - M
      float sum = 0.f;
      bool apart = fabsf(base) > 4194304.f;
#pragma unroll
      for (int p = 0; p < PP; ++p) apart |= !(base - oref + lv[p] > -60.f);
      if (__any_sync(0xffffffffu, apart)) {
        // p for itself, from a rounded score: a page of far smaller values than
        // the others' (kSmall), whose p * vscale vanishes and p does not; or scores
        // so large that the exact z2 - m of a fused product is not 0 at the maximum
#pragma unroll
        for (int nt = 0; nt < NS; ++nt)
#pragma unroll
          for (int x = 2 * i; x < 2 * i + 2; ++x) {
            const float d = __fadd_rn(__fmul_rn(z[nt][x], c[nt / TP]), -base);
            sum += ptx::ex2(d);
            z[nt][x] = ptx::ex2(d + (base - oref + lv[nt / TP]));
          }
      } else {
#pragma unroll
        for (int p = 0; p < PP; ++p) {
          const float off = lv[p] - oref;
          float ps = 0.f;
#pragma unroll
          for (int nt = p * TP; nt < (p + 1) * TP; ++nt)
#pragma unroll
            for (int x = 2 * i; x < 2 * i + 2; ++x) {
              z[nt][x] = ptx::ex2(fmaf(z[nt][x], c[p], off));
              ps += z[nt][x];
            }
          sum = fmaf(ps, ptx::ex2(oref - base - lv[p]), sum);
        }
      }
      l[i] = l[i] * al + sum;
      if (__any_sync(0xffffffffu, ao != 1.f)) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          o[j][2 * i] *= ao;
          o[j][2 * i + 1] *= ao;
        }
      }
    }
  }

  // Fragment x of P's k step s: rows g, g + 8 of keys t, t + 4 (x = 0, 1), of 8 + t, 12 + t
  static __device__ __forceinline__ void weights(uint32_t (&a)[PARTS][4], const float (&z)[NS][4],
                                                 int s) {
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const float p0 = z[2 * s + (x >> 1)][2 * (x & 1)], p1 = z[2 * s + (x >> 1)][2 * (x & 1) + 1];
      a[0][x] = pack_half(p0, p1);
      if (PARTS == 2) {
        const float2 f = unpack_half(a[0][x]);
        a[PARTS - 1][x] = pack_half(p0 - f.x, p1 - f.y);
      }
    }
  }

  // Word k of the lane's pieces of keys t, 4 + t, 8 + t, 12 + t (its components
  // 4 k .. 4 k + 3) as the B fragments of output tiles 4 k .. 4 k + 3.
  static __device__ __forceinline__ void fragments(const uint32_t (&w)[4], uint32_t (&b)[4][2]) {
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const uint32_t sel = y ? 0x7362u : 0x5140u;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t x = __byte_perm(w[2 * h], w[2 * h + 1], sel);
        e4m3x4_to_half2x2(x, b[2 * y][h], b[2 * y + 1][h]);
      }
    }
  }

  __device__ __forceinline__ void values(const float (&z)[NS][4], uint32_t vbase, int lane) {
    const int g = lane >> 2, t = lane & 3;
    const uint32_t v0 = vbase + (D == 128 ? v_off<D>(t, g) : v_off<D>(t, g >> 1) + (g & 1) * 8);
    if (PARTS == 1) {
#pragma unroll
      for (int s = 0; s < CK / 16; ++s) {
        uint32_t a[PARTS][4];
        weights(a, z, s);
        uint32_t w[4][D / 32];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t at = v0 + (16 * s + 4 * i) * D;
          if (D == 128) {
            const uint4 v = lds128(at);
            w[i][0] = v.x;
            w[i][1] = v.y;
            w[i][D / 32 - 2] = v.z;
            w[i][D / 32 - 1] = v.w;
          } else {
            const uint2 v = lds64(at);
            w[i][0] = v.x;
            w[i][1] = v.y;
          }
        }
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          const uint32_t wk[4] = {w[0][k], w[1][k], w[2][k], w[3][k]};
          uint32_t b[4][2];
          fragments(wk, b);
#pragma unroll
          for (int j = 0; j < 4; ++j) mma_f16(o[4 * k + j], a[0], b[j][0], b[j][1]);
        }
      }
    } else {
      // fp32: the tensor core's sums of a chunk are short, and added to o in
      // fp32 with rounding to nearest (its own additions truncate)
      uint32_t a[CK / 16][PARTS][4];
#pragma unroll
      for (int s = 0; s < CK / 16; ++s) weights(a[s], z, s);
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        float add[4][4] = {};
#pragma unroll
        for (int s = 0; s < CK / 16; ++s) {
          uint32_t wk[4], b[4][2];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(wk[i]) : "r"(v0 + (16 * s + 4 * i) * D + 4 * k));
          fragments(wk, b);
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int p = PARTS - 1; p >= 0; --p) mma_f16(add[j], a[s][p], b[j][0], b[j][1]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int x = 0; x < 4; ++x) o[4 * k + j][x] += add[j][x];
      }
    }
  }

  // Values that are NaN in keys which some rows of the tile see and others do
  // not: 0 * NaN must not reach the rows that do not. Their codes become zeros
  // in the slot and the rows that see them become NaN. Rare, and only in
  // chunks on the edge of a row's keys.
  template <int PP>
  __device__ void nan_values(unsigned char* vst, const ChunkMeta<PP>& meta, int lane) {
    bool found = false;
    for (int i = lane; i < CK * D / 16; i += 32) {
      const uint4 v = reinterpret_cast<const uint4*>(vst)[i];
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) found |= __vcmpeq4(w[k] & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0;
    }
    if (!__any_sync(0xffffffffu, found)) return;
    const int t = lane & 3;
    constexpr int RUN = D / 4;  // the lane's outputs are components RUN t .. of its rows
#pragma unroll 1
    for (int r = 0; r < CK; ++r) {
      const int key = meta.kb[r / (CK / PP)] + r % (CK / PP);
#pragma unroll
      for (int j = 0; j < RUN; ++j) {
        const int dim = RUN * t + j;
        const uint8_t code = vst[v_off<D>(r, dim / 16) + dim % 16];
        if ((code & 0x7f) == 0x7f) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (key >= lo[i] && key < hi[i])
              o[j % NT][2 * i + j / NT] = __uint_as_float(0x7fffffffu);
        }
      }
    }
    __syncwarp();
    for (int i = lane; i < CK * D / 4; i += 32) {
      uint32_t* w = reinterpret_cast<uint32_t*>(vst) + i;
      *w &= ~__vcmpeq4(*w & 0x7f7f7f7fu, 0x7f7f7f7fu);
    }
    __syncwarp();
  }

  // Ends the unit: o normalised, lse2 = log2 of the sum of 2^z2.
  __device__ __forceinline__ void finish(float (&lse2)[2]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float sum = quad_sum(l[i]);
      const float base = m[i] == -INFINITY ? 0.f : m[i], oref = M[i] == -INFINITY ? 0.f : M[i];
      // in two factors: 2^(M - m) alone can leave fp32's range
      const float half = ptx::ex2(0.5f * (oref - base));
      const float f = sum == 0.f ? 0.f : half / sum;
      lse2[i] = sum == 0.f ? -INFINITY : m[i] + log2f(sum);
      // (a row without keys has o = 0, NaN only where NaN values were marked)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        o[j][2 * i] = o[j][2 * i] * half * f;
        o[j][2 * i + 1] = o[j][2 * i + 1] * half * f;
      }
    }
  }

  // The lane holds components D / 4 * t .. + D / 4 - 1 of its rows: first half
  // of them in o[.][2 i], second in o[.][2 i + 1].
  __device__ __forceinline__ void write(const Q8AttendArgs& a, const Unit& u, int h,
                                        const float (&lse2)[2], int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = u.r0 + g + 8 * i;
      if (r >= u.s.n * a.G) continue;
      const long row = row_of(a, u.s, h, r);
      T* dst = static_cast<T*>(a.out) + row * D + (D / 4) * t;
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int j = 0; j < NT; j += 4) {
          const float v[4] = {o[j][2 * i + c], o[j + 1][2 * i + c], o[j + 2][2 * i + c],
                              o[j + 3][2 * i + c]};
          if (sizeof(T) == 4) {
            *reinterpret_cast<float4*>(dst + NT * c + j) = make_float4(v[0], v[1], v[2], v[3]);
          } else {
            *reinterpret_cast<uint2*>(dst + NT * c + j) =
                make_uint2(ptx::pack_bf16(v[0], v[1]), ptx::pack_bf16(v[2], v[3]));
          }
        }
      if (t == 0 && a.lse) a.lse[row] = lse2[i] * q8::kLn2;
    }
  }

  // A partial keeps the fragments' order: float4 32 j + lane is o[j] of the lane.
  __device__ __forceinline__ void store(float* part, float* part_lse, const float (&lse2)[2],
                                        int lane) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
      reinterpret_cast<float4*>(part)[32 * j + lane] =
          make_float4(o[j][0], o[j][1], o[j][2], o[j][3]);
    if ((lane & 3) == 0) {
      part_lse[lane >> 2] = lse2[0];
      part_lse[(lane >> 2) + 8] = lse2[1];
    }
  }
};

// Output tiles 4 jg .. 4 jg + 3 of fragment lane `lane` to the output's rows.
template <typename T, int D>
__device__ __forceinline__ void write_group(const Q8AttendArgs& a, const Seq& s, int h, int r0,
                                            int jg, int lane, const float4 (&x)[4]) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = r0 + g + 8 * i;
    if (r >= s.n * a.G) continue;
    T* dst = static_cast<T*>(a.out) + Rows<T, D>::row_of(a, s, h, r) * D + (D / 4) * t + 4 * jg;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = i == 0 ? (c ? x[k].y : x[k].x) : (c ? x[k].w : x[k].z);
      if (sizeof(T) == 4)
        *reinterpret_cast<float4*>(dst + D / 8 * c) = make_float4(v[0], v[1], v[2], v[3]);
      else
        *reinterpret_cast<uint2*>(dst + D / 8 * c) =
            make_uint2(ptx::pack_bf16(v[0], v[1]), ptx::pack_bf16(v[2], v[3]));
    }
  }
}

// A warp's unfinished unit: begun before its share or continued behind it.
struct Segment {
  long u0;            // its first chunk's place
  int nc;             // its chunks; 0: no segment
  int tile, h, r0, first, n;
  const float* part;
};
constexpr int kSegs = 2 * kWarps;

template <typename T, int D, int PP>
struct Smem {
  static constexpr int RING = kWarps * Geo<D>::RING;
  static constexpr int META = RING;
  static constexpr int RANGE = META + kWarps * 2 * (int)sizeof(ChunkMeta<PP>);
  static constexpr int SEGS = (RANGE + kWarps * 8 + 15) / 16 * 16;
  static constexpr int LSE = SEGS + kSegs * (int)sizeof(Segment);  // of the segments' rows
  static constexpr int WGT = LSE + kSegs * ROWS * 4;               // their weights in the join
  static constexpr int SUMS = WGT + kSegs * ROWS * 4;
  static constexpr int PRE = SUMS + kWarps * 8;
  static constexpr int LENS = PRE + (kSmemTiles + 1) * 8;
  static constexpr int BYTES = LENS + kSmemTiles * 4;
};

// A warp's share of the chunks, [x0, x1). MULTI: a tile can hold several tokens,
// which see different keys. FAR: apart_softmax for all of them; without, false at
// the first sight of a unit whose value scales lie far apart, the share undone.
template <typename T, int D, int PP, bool MULTI, bool FAR>
__device__ __forceinline__ bool share(const Q8AttendArgs& a, const Plan& pl, unsigned char* smem,
                                      int cta, long x0, long x1) {
  using S = Smem<T, D, PP>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Segment* segs = reinterpret_cast<Segment*>(smem + S::SEGS);
  float* seg_lse = reinterpret_cast<float*>(smem + S::LSE);
  constexpr int TILE = Geo<D>::TILE;
  unsigned char* ring = smem + warp * Geo<D>::RING;
  ChunkMeta<PP>* meta = reinterpret_cast<ChunkMeta<PP>*>(smem + S::META) + warp * 2;
  int* range = reinterpret_cast<int*>(smem + S::RANGE) + warp * 2;
  const uint32_t ring_u = ptx::smem_u32(ring);
  Feeder<D, PP> feed;
  feed.start(a, pl, x0);
  Place at = feed.at;
  Unit u = feed.u;
  Rows<T, D> rows;
  {
    typename Rows<T, D>::Raw raw;
    rows.fetch(raw, a, u, at.h, lane);
    // K and V of the first chunk into slots 0 and 1
    feed.look(a, meta, lane);
    feed.template copy<false>(a, ring_u, lane);
    ptx::cp_async_commit();
    feed.template copy<true>(a, ring_u + TILE, lane);
    ptx::cp_async_commit();
    rows.load(raw, a, u, lane);
    feed.scales(meta, lane);
    if (!FAR && feed.far(range, false, q8::spread<T>(), lane)) {
      ptx::cp_async_wait<0>();  // (the ring is used anew)
      __syncwarp();
      return false;
    }
  }
  rows.clear();
  bool whole = at.c == 0;  // the unit's first chunk is the warp's
  int sk = 0;              // slot of the chunk's K; its V is in the next, the next K behind that
  int mi = 0;
  const int len = (int)(x1 - x0);
  for (int x = 0; x < len; ++x) {
    const int sv = sk + 1 == SLOTS ? 0 : sk + 1, sn = sv + 1 == SLOTS ? 0 : sv + 1;
    ptx::cp_async_wait<1>();  // K
    __syncwarp();
    const bool more = x + 1 < len;
    if (more) {
      feed.next(a, pl);
      feed.look(a, meta + (mi ^ 1), lane);
      feed.template copy<false>(a, ring_u + sn * TILE, lane);
    }
    ptx::cp_async_commit();
    if (more) feed.scales(meta + (mi ^ 1), lane);
    if (!FAR && more && feed.centry == feed.gbase &&
        feed.far(range, feed.at.c > 0, q8::spread<T>(), lane)) {
      ptx::cp_async_wait<0>();  // (the ring is used anew)
      __syncwarp();
      return false;
    }
    const ChunkMeta<PP>& sm = meta[mi];
    const int state = sm.state;
    float z[NS][4];
    if (state) {
      rows.scores(z, ring_u + sk * TILE, lane);
      if (FAR) {
        ptx::cp_async_wait<1>();  // V, which the weights go by
        __syncwarp();
        rows.template apart_softmax<PP>(z, sm, state == 2, ring + sv * TILE, lane);
      } else {
        rows.template softmax<PP>(z, sm, state == 2, lane);
      }
    }
    ptx::cp_async_wait<1>();  // V
    __syncwarp();
    if (more) feed.template copy<true>(a, ring_u + sk * TILE, lane);
    ptx::cp_async_commit();
    if (state) {
      if (MULTI && state == 1)
        rows.template nan_values<PP>(ring + sv * TILE, sm, lane);
      rows.values(z, ring_u + sv * TILE, lane);
    }
    sk = sn;
    mi ^= 1;
    const bool last = at.c + 1 == at.nc;
    if (last || !more) {
      float lse2[2];
      rows.finish(lse2);
      if (whole && last) {
        rows.write(a, u, at.h, lse2, lane);
      } else if (more) {
        float* part = a.hold + ((long)cta * kWarps + warp) * Geo<D>::PART;
        rows.store(part, seg_lse + 2 * warp * ROWS, lse2, lane);
        if (lane == 0)
          segs[2 * warp] = Segment{x0 + x - at.c, at.nc, at.tile, at.h, u.r0, u.s.first, u.s.n, part};
      } else {
        ptx::cp_async_wait<0>();
        __syncwarp();  // the ring is free
        float* part = reinterpret_cast<float*>(ring);
        rows.store(part, seg_lse + (2 * warp + 1) * ROWS, lse2, lane);
        if (lane == 0)
          segs[2 * warp + 1] =
              Segment{x0 + x - at.c, at.nc, at.tile, at.h, u.r0, u.s.first, u.s.n, part};
      }
      if (more) {
        const int tile = at.tile;
        at.next(pl, a.Hkv);
        if (at.tile != tile) u.load(a, pl, at.tile);
        typename Rows<T, D>::Raw raw;
        rows.fetch(raw, a, u, at.h, lane);
        rows.load(raw, a, u, lane);
        rows.clear();
        whole = true;
      }
    } else {
      ++at.c;
    }
  }
  return true;
}

// The plan: that of the launch before, or the block's own (made in shared memory).
template <typename T, int D, int PP>
__device__ __forceinline__ Plan plan_of(const Q8AttendArgs& a, unsigned char* smem) {
  using S = Smem<T, D, PP>;
  if (a.plan_pre)
    return Plan{a.plan_pre, a.plan_seq, a.plan_base, nullptr, a.plan_base[a.B], a.rt};
  return Plan{reinterpret_cast<long*>(smem + S::PRE), nullptr, nullptr,
              reinterpret_cast<int*>(smem + S::LENS), a.tiles, a.rt};
}

// share of a warp with FAR: a call, so that it takes no registers from the other.
template <typename T, int D, int PP, bool MULTI>
__device__ __noinline__ void share_far(const Q8AttendArgs& a, unsigned char* smem, int cta, long X0,
                                       long X1) {
  const int warp = threadIdx.x >> 5;
  share<T, D, PP, MULTI, true>(a, plan_of<T, D, PP>(a, smem), smem, cta,
                               X0 + (X1 - X0) * warp / kWarps, X0 + (X1 - X0) * (warp + 1) / kWarps);
}

template <typename T, int D, int PP, bool MULTI>
__global__ void __launch_bounds__(kThreads, 1)
    q8_attend_kernel(const __grid_constant__ Q8AttendArgs a) {
  using S = Smem<T, D, PP>;
  extern __shared__ __align__(128) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Segment* segs = reinterpret_cast<Segment*>(smem + S::SEGS);
  float* seg_lse = reinterpret_cast<float*>(smem + S::LSE);
  float* seg_wgt = reinterpret_cast<float*>(smem + S::WGT);
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();

  // ---- plan ----
  if (!a.plan_pre) {
    long* pre = reinterpret_cast<long*>(smem + S::PRE);
    long* sums = reinterpret_cast<long*>(smem + S::SUMS);
    int* lens = reinterpret_cast<int*>(smem + S::LENS);
    long base = 0;
    if (tid == 0) pre[0] = 0;
    for (int t0 = 0; t0 < a.tiles; t0 += kThreads) {
      const int tile = t0 + tid;
      long mine = 0;
      if (tile < a.tiles) {
        const int b = tile / a.rt;
        const Seq s = q8::sequence(a, b);
        if (!s.ok && blockIdx.x == 0) atomicOr(a.err, s.err);
        mine = (long)q8::chunks_of(a, s, (tile - b * a.rt) * ROWS, ROWS, CK) * a.Hkv;
        lens[tile] = s.ok ? s.len : -1;
      }
      long run = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long up = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += up;
      }
      if (lane == 31) sums[warp] = run;
      __syncthreads();
      long before = base;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        if (k < warp) before += sums[k];
        base += sums[k];
      }
      if (tile < a.tiles) pre[tile + 1] = before + run;
      __syncthreads();
    }
  }
  const Plan pl = plan_of<T, D, PP>(a, smem);
  if (tid < kSegs) segs[tid].nc = 0;
  __syncthreads();
  const long V = pl.tiles ? pl.pre[pl.tiles] : 0;
  // few chunks: fewer blocks, so that a block's warps share its merge
  const long want = (V + a.min_chunks - 1) / a.min_chunks;
  const int C = (int)(a.by_unit || want >= gridDim.x ? gridDim.x : want > 0 ? want : 1);
  const int cta = blockIdx.x;
  q8::MergeMeta* mm = reinterpret_cast<q8::MergeMeta*>(a.meta);
  if (tid == 0) mm[cta].unit = -1;
  if (cta >= C || V == 0) return;
  long X0 = q8::split(V, cta, C), X1 = q8::split(V, cta + 1, C);
  if (a.by_unit == 1) {
    const long units = (long)pl.tiles * a.Hkv;
    X0 = q8::unit_place(pl, a.Hkv, (int)q8::split(units, cta, C));
    X1 = q8::unit_place(pl, a.Hkv, (int)q8::split(units, cta + 1, C));
  } else if (a.by_unit == 2) {
    X0 = q8::unit_start(pl, a.Hkv, X0);
    X1 = q8::unit_start(pl, a.Hkv, X1);
  }
  const long x0 = X0 + (X1 - X0) * warp / kWarps, x1 = X0 + (X1 - X0) * (warp + 1) / kWarps;

  if (x1 > x0 && !share<T, D, PP, MULTI, false>(a, pl, smem, cta, x0, x1))
    share_far<T, D, PP, MULTI>(a, smem, cta, X0, X1);
  __syncthreads();

  // ---- join the block's segments of each unit ----
  // Lane e of each warp holds segment e; the segments of one unit are a group,
  // a bit mask, led by its lowest. Thread (e, r) weighs row r of segment e.
  static_assert(kSegs * ROWS == kThreads, "a thread for each segment's row");
  const Segment mine = segs[lane % kSegs];
  const bool have = lane < kSegs && mine.nc > 0;
  const unsigned group = __match_any_sync(0xffffffffu, have ? mine.u0 : -1l - lane);
  unsigned leaders = __ballot_sync(0xffffffffu, have && (group & ((1u << lane) - 1)) == 0);
  {
    const int e = tid / ROWS, r = tid % ROWS;
    const unsigned set = __shfl_sync(0xffffffffu, have ? group : 0u, e);
    if (set) {
      float top = -INFINITY, sum = 0.f;
      for (unsigned m = set; m; m &= m - 1) top = fmaxf(top, seg_lse[(__ffs(m) - 1) * ROWS + r]);
      const float base = top == -INFINITY ? 0.f : top;
      for (unsigned m = set; m; m &= m - 1)
        sum += ptx::ex2(seg_lse[(__ffs(m) - 1) * ROWS + r] - base);
      seg_wgt[tid] = sum == 0.f ? 0.f : ptx::ex2(seg_lse[tid] - base) / sum;
      if (__ffs(set) - 1 == e) {
        const Segment& sg = segs[e];
        const float lse2 = sum == 0.f ? -INFINITY : top + log2f(sum);
        const Seq s{sg.first, sg.n, 0, true, 0u};
        if (sg.u0 >= X0 && sg.u0 + sg.nc <= X1) {
          if (sg.r0 + r < sg.n * a.G && a.lse)
            a.lse[Rows<T, D>::row_of(a, s, sg.h, sg.r0 + r)] = lse2 * q8::kLn2;
        } else {
          a.part[(2l * cta + (sg.u0 < X0 ? 0 : 1)) * Geo<D>::PART + ROWS * D + r] = lse2;
          if (r == 0 && sg.u0 < X0 && sg.u0 + sg.nc <= X1) {
            mm[cta].unit = (long)sg.tile * a.Hkv + sg.h;
            mm[cta].from = q8::block_of(sg.u0, V, C);
          }
        }
      }
    }
  }
  __syncthreads();
  // four warps (two for d = 64) join a group, a lane four output tiles of its fragment
  constexpr int JG = D / 32;
  const int jg = warp % JG, g = lane >> 2;
  for (int k = 0; leaders; leaders &= leaders - 1, ++k) {
    if (k % (kWarps / JG) != warp / JG) continue;
    const int lead = __ffs(leaders) - 1;
    const unsigned set = __shfl_sync(0xffffffffu, group, lead);
    float4 acc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (unsigned m = set; m; m &= m - 1) {
      const int e = __ffs(m) - 1;
      const float4* part = reinterpret_cast<const float4*>(segs[e].part) + 128 * jg + lane;
      const float w0 = seg_wgt[e * ROWS + g], w1 = seg_wgt[e * ROWS + g + 8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 x = part[32 * j];
        acc[j].x = fmaf(w0, x.x, acc[j].x);
        acc[j].y = fmaf(w0, x.y, acc[j].y);
        acc[j].z = fmaf(w1, x.z, acc[j].z);
        acc[j].w = fmaf(w1, x.w, acc[j].w);
      }
    }
    const Segment& sg = segs[lead];
    if (sg.u0 >= X0 && sg.u0 + sg.nc <= X1) {
      const Seq s{sg.first, sg.n, 0, true, 0u};
      write_group<T, D>(a, s, sg.h, sg.r0, jg, lane, acc);
    } else {
      float4* slot = reinterpret_cast<float4*>(
          a.part + (2l * cta + (sg.u0 < X0 ? 0 : 1)) * Geo<D>::PART) + 128 * jg + lane;
#pragma unroll
      for (int j = 0; j < 4; ++j) slot[32 * j] = acc[j];
    }
  }
}

// Joins the partials of a unit that lies in several blocks: block (c, jg) does
// output tiles 4 jg .. of the unit that ends in attention block c, from slot
// 2 f + 1 of the block f it begins in and slots 2 i of the blocks behind it up
// to c. Its warps take every kMergeWarps-th partial.
constexpr int kMergeWarps = 8;
template <typename T, int D>
__global__ void __launch_bounds__(32 * kMergeWarps)
    q8_merge_kernel(const __grid_constant__ Q8AttendArgs a) {
  ptx::grid_dep_wait();
  const q8::MergeMeta mm = reinterpret_cast<const q8::MergeMeta*>(a.meta)[blockIdx.x];
  if (mm.unit < 0) return;
  __shared__ float s_top[kMergeWarps][ROWS], s_sum[kMergeWarps][ROWS];
  __shared__ float4 s_acc[kMergeWarps][4][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, jg = blockIdx.y;
  const int g = lane >> 2, t = lane & 3;
  const int n = (int)blockIdx.x - mm.from + 1;
  auto part = [&](int i) { return a.part + (2l * (mm.from + i) + (i == 0 ? 1 : 0)) * Geo<D>::PART; };
  float top[2] = {-INFINITY, -INFINITY};
#pragma unroll 4
  for (int i = 4 * warp + t; i < n; i += 4 * kMergeWarps) {
    const float* l = part(i) + ROWS * D;
    top[0] = fmaxf(top[0], l[g]);
    top[1] = fmaxf(top[1], l[g + 8]);
  }
  top[0] = quad_max(top[0]);
  top[1] = quad_max(top[1]);
  if (t == 0) {
    s_top[warp][g] = top[0];
    s_top[warp][g + 8] = top[1];
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) {
    top[0] = fmaxf(top[0], s_top[w][g]);
    top[1] = fmaxf(top[1], s_top[w][g + 8]);
  }
  const float b0 = top[0] == -INFINITY ? 0.f : top[0], b1 = top[1] == -INFINITY ? 0.f : top[1];
  float4 acc[4];
  float sum[2] = {0.f, 0.f};
#pragma unroll
  for (int j = 0; j < 4; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = warp; i < n; i += kMergeWarps) {
    const float* p = part(i);
    const float w0 = ptx::ex2(p[ROWS * D + g] - b0), w1 = ptx::ex2(p[ROWS * D + g + 8] - b1);
    sum[0] += w0;
    sum[1] += w1;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 x = reinterpret_cast<const float4*>(p)[128 * jg + 32 * j + lane];
      acc[j].x = fmaf(w0, x.x, acc[j].x);
      acc[j].y = fmaf(w0, x.y, acc[j].y);
      acc[j].z = fmaf(w1, x.z, acc[j].z);
      acc[j].w = fmaf(w1, x.w, acc[j].w);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) s_acc[warp][j][lane] = acc[j];
  if (t == 0) {
    s_sum[warp][g] = sum[0];
    s_sum[warp][g + 8] = sum[1];
  }
  __syncthreads();
  if (warp != 0) return;
#pragma unroll
  for (int w = 1; w < kMergeWarps; ++w) {
    sum[0] += s_sum[w][g];
    sum[1] += s_sum[w][g + 8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 x = s_acc[w][j][lane];
      acc[j].x += x.x;
      acc[j].y += x.y;
      acc[j].z += x.z;
      acc[j].w += x.w;
    }
  }
  const float f0 = sum[0] == 0.f ? 0.f : 1.f / sum[0], f1 = sum[1] == 0.f ? 0.f : 1.f / sum[1];
#pragma unroll
  for (int j = 0; j < 4; ++j) acc[j] = make_float4(acc[j].x * f0, acc[j].y * f0, acc[j].z * f1, acc[j].w * f1);
  const int tile = (int)(mm.unit / a.Hkv), h = (int)(mm.unit % a.Hkv);
  const int b = a.plan_pre ? a.plan_seq[tile] : tile / a.rt;
  const int r0 = (tile - (a.plan_pre ? a.plan_base[b] : b * a.rt)) * ROWS;
  Seq s{b, 1, 0, true, 0u};
  if (a.cu) q8::token_range(a.cu, b, a.N, s.first, s.n);
  write_group<T, D>(a, s, h, r0, jg, lane, acc);
  if (jg == 0 && t == 0 && a.lse) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = r0 + g + 8 * i;
      if (r < s.n * a.G)
        a.lse[Rows<T, D>::row_of(a, s, h, r)] =
            sum[i] == 0.f ? -INFINITY : (top[i] + log2f(sum[i])) * q8::kLn2;
    }
  }
}

// The plan of a call with offsets, or of more tiles than a block takes in: the
// tiles of every sequence and the chunks before each tile, `extra` for a unit's own
// cost included. One block.
constexpr int kPlanThreads = 1024;
template <typename I>
__device__ __forceinline__ I block_scan(I mine, I* sums, I& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  I run = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const I up = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += up;
  }
  if (lane == 31) sums[warp] = run;
  __syncthreads();
  static_assert(kPlanThreads == 32 * 32, "a lane for each warp's sum");
  I all = sums[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const I up = __shfl_up_sync(0xffffffffu, all, o);
    if (lane >= o) all += up;
  }
  total = __shfl_sync(0xffffffffu, all, 31);
  const I before = __shfl_sync(0xffffffffu, all, (warp + 31) % 32);
  __syncthreads();
  return (warp ? before : I(0)) + run - mine;
}

__global__ void __launch_bounds__(kPlanThreads) q8_plan_kernel(const Q8AttendArgs a, int tile_rows,
                                                               int chunk, int extra, bool halves) {
  __shared__ long sums[kPlanThreads / 32];
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int tid = threadIdx.x;
  long base = 0, all;
  for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    long mine = 0;
    if (b < a.B) {
      const Seq s = q8::sequence(a, b);
      if (!s.ok) atomicOr(a.err, s.err);
      mine = q8::tiles_of(a, s.n, tile_rows);
    }
    const long at = block_scan(mine, sums, all);
    if (b < a.B) a.plan_base[b] = (int)(base + at);
    base += all;
  }
  const int tiles = (int)(base < a.tiles ? base : a.tiles);
  if (tid == 0) {
    a.plan_base[a.B] = tiles;
    a.plan_pre[0] = 0;
  }
  __syncthreads();
  base = 0;
  for (int t0 = 0; t0 < tiles; t0 += kPlanThreads) {
    const int t = t0 + tid;
    long mine = 0;
    if (t < tiles) {
      int b = 0, last = a.B - 1;  // the last sequence that begins at or before tile t
      while (b < last) {
        const int mid = (b + last + 1) >> 1;
        if (a.plan_base[mid] <= t)
          b = mid;
        else
          last = mid - 1;
      }
      a.plan_seq[t] = b;
      const Seq s = q8::sequence(a, b);
      const int r0 = (t - a.plan_base[b]) * tile_rows;
      const int weight = halves ? q8::tc_weight(s.n * a.G - r0) : 1;
      mine = ((long)q8::chunks_of(a, s, r0, tile_rows, chunk) * weight + extra) * a.Hkv;
    }
    const long at = block_scan(mine, sums, all);
    if (t < tiles) a.plan_pre[t + 1] = base + at + mine;
    base += all;
  }
}

template <typename T, int D, int PP>
cudaError_t launch(const Q8AttendArgs& a, cudaStream_t stream) {
  auto kern = a.cu ? q8_attend_kernel<T, D, PP, true> : q8_attend_kernel<T, D, PP, false>;
  constexpr int smem = Smem<T, D, PP>::BYTES;
  cudaError_t e;
  if ((e = ensure_dyn_smem((const void*)kern, smem)) != cudaSuccess) return e;
  {
    TraceScope trace("q8_attend", stream);
    if ((e = q8::launch_pdl(kern, dim3(a.blocks), dim3(kThreads), smem, stream, a)) != cudaSuccess)
      return e;
  }
  if (a.by_unit) return cudaSuccess;
  TraceScope trace("q8_merge", stream);
  return q8::launch_pdl(q8_merge_kernel<T, D>, dim3(a.blocks, D / 32), dim3(32 * kMergeWarps), 0, stream,
                    a);
}

template <typename T, int D>
cudaError_t launch(const Q8AttendArgs& a, cudaStream_t stream) {
  if (a.page >= CK) return launch<T, D, 1>(a, stream);
  return a.page == 32 ? launch<T, D, 2>(a, stream) : launch<T, D, 4>(a, stream);
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Most tiles a call can have; N is the number of query tokens.
long most_tiles(const nsa_params& p, bool ragged, long N) {
  const int G = p.Hq / p.Hkv;
  if (!ragged) return (long)p.B * ((G + ROWS - 1) / ROWS);
  return N * G / ROWS + p.B;
}

struct Layout {
  size_t part, hold, meta, pre, seq, base, total;
};

// (sized for the most query tokens the parameters allow, B * T)
Layout layout(const nsa_params& p, bool ragged) {
  Layout L{};
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t o = at;
    at += align256(n);
    return o;
  };
  const size_t part = (size_t)(ROWS * p.d + ROWS) * 4;
  const size_t tc = ragged && q8_prefill_tc_shape(p) ? q8_prefill_tc_part_bytes() : 0;
  L.part = take(std::max(part * 2 * kQ8MaxBlocks, tc));
  L.hold = take(part * kWarps * kQ8MaxBlocks);
  L.meta = take(sizeof(q8::MergeMeta) * kQ8MaxBlocks);
  const long tiles = most_tiles(p, ragged, (long)p.B * p.T);
  if (ragged || tiles > kSmemTiles) {
    L.pre = take((size_t)(tiles + 1) * 8);
    L.seq = take((size_t)tiles * 4);
    L.base = take((size_t)(p.B + 1) * 4);
  }
  L.total = at;
  return L;
}

}  // namespace

size_t q8_attend_ws_bytes(const nsa_params& p, bool ragged) {
  return layout(p, ragged).total;
}

cudaError_t launch_q8_attend(const nsa_params& p, Q8AttendArgs a, void* ws, cudaStream_t stream) {
  const bool ragged = a.cu != nullptr;
  const Layout L = layout(p, ragged);
  char* w = static_cast<char*>(ws);
  a.part = reinterpret_cast<float*>(w + L.part);
  a.hold = reinterpret_cast<float*>(w + L.hold);
  a.meta = w + L.meta;
  a.tiles = (int)most_tiles(p, ragged, a.N);
  a.rt = (a.G + ROWS - 1) / ROWS;
  a.blocks = std::min(device_sm_count(), kQ8MaxBlocks);
  a.min_chunks = 8;
  a.plan_pre = nullptr;
  a.plan_seq = nullptr;
  a.plan_base = nullptr;
  // Chunks of queries on the tensor-memory kernel once a sequence has rows to
  // fill a good part of its 128-row tiles with; below that most of the tile is
  // padding, and the kernel here reads the same codes once per 16 rows.
  const bool tc = ragged && q8_prefill_tc_shape(p) && (long)a.N * a.G >= 32l * p.B;
  // Units of few chunks: whole ones to a block, which leaves no partials and
  // saves the merge kernel (3 to 6 us; a pass of a block's warps over a chunk
  // each takes 2 us). With the most chunks a unit can have, that may cost 1.25
  // passes more than an even split does: 4 units of 16 chunks take 14.8 us both
  // ways, of 22 chunks 17.4 us whole and 14.6 split; 128 units of 22 chunks 19
  // and 24.5 us, of 32 chunks 22 and 27. Few chunks and as many units as blocks,
  // or windows and lists, make units alike; else they are dealt by their chunks.
  const long most = a.keys == q8::KEYS_BLOCKS   ? ((long)a.n * a.page + CK - 1) / CK
                    : a.keys == q8::KEYS_WINDOW ? ((long)a.window + ROWS + 2 * CK - 2) / CK
                                                : ((long)a.T + CK - 1) / CK;
  const long units = (long)a.tiles * a.Hkv, per = (units + a.blocks - 1) / a.blocks;
  const double even = (double)units * most / (kWarps * (double)a.blocks);
  a.by_unit = 0;
  if (!tc && most <= kUnitChunks && per * most <= kWarps * (std::max(1.0, even) + 1.25)) {
    a.by_unit = a.keys == q8::KEYS_ALL && units > a.blocks ? 2 : 1;
    a.blocks = (int)std::min<long>(a.blocks, units);
  }
  // (its two halves share the keys where most sequences have rows for one)
  const bool split = tc && (long)a.N * a.G <= kQ8TcRows / 2 * (long)p.B;
  if (tc) a.tiles = (int)((long)a.N * a.G / kQ8TcRows + p.B);
  if (ragged || a.tiles > kSmemTiles) {
    a.plan_pre = reinterpret_cast<long*>(w + L.pre);
    a.plan_seq = reinterpret_cast<int*>(w + L.seq);
    a.plan_base = reinterpret_cast<int*>(w + L.base);
    TraceScope trace("q8_plan", stream);
    const cudaError_t e = q8::launch_pdl(q8_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, a,
                                         tc ? kQ8TcRows : ROWS, tc ? kQ8TcKeys : CK,
                                         tc ? kQ8TcUnit : 0, split);
    if (e != cudaSuccess) return e;
  }
  if (tc) return launch_q8_prefill_tc(a, split, stream);
  const bool bf16 = p.dtype == NSA_DTYPE_BF16;
  using bf = __nv_bfloat16;
  if (p.d == 128) return bf16 ? launch<bf, 128>(a, stream) : launch<float, 128>(a, stream);
  return bf16 ? launch<bf, 64>(a, stream) : launch<float, 64>(a, stream);
}

}  // namespace nsa
