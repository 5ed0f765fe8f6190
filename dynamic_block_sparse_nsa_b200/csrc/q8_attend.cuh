// Work plan shared by the attention kernels over the 8-bit paged cache.
//
// A "tile" is a (sequence, row tile): `rows` consecutive query rows, row r of
// a sequence being head r % G of its token r / G. A unit is a tile and a KV
// head. The keys a tile needs are cut into chunks, and the chunks of all
// units, in order (tile, KV head, chunk), are split evenly over the blocks of
// one resident grid: block c of C takes [V c / C, V (c + 1) / C) of V. A unit
// that lies in one block is finished there; each block leaves the partial
// results of its first unit (begun in an earlier block) in slot 2 c and of its
// last (continued in a later one) in slot 2 c + 1, as a normalised output and
// log-sum-exp, and q8_merge_kernel joins them.
#pragma once

#include <climits>
#include <utility>

#include "ptx.cuh"
#include "q8.cuh"

namespace nsa {
namespace q8 {

enum { KEYS_ALL = NSA_KEYS_ALL, KEYS_WINDOW = NSA_KEYS_WINDOW, KEYS_BLOCKS = NSA_KEYS_BLOCKS };

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Value scales of a unit's pages that lie further apart than 2^spread ("far apart"):
// the output's reference M is then taken from the codes that a row sees and from its
// sums, not from the scales, which other tokens may have set. Up to there a weight's
// smallest place in fp16 lies at least 2^(35 - spread) below the row's largest weight:
// 2^27 for fp32 rows, 2^23 for bf16 ones, 2^3 and 2^14 beyond their types' places.
// Scales up to 2^kSmall do not count: no value under them reaches 1e-30.
template <typename T>
constexpr int spread() {
  return sizeof(T) == 4 ? 8 : 12;
}
constexpr float kSmall = -109.f;

// Places, 0 to 5, by which the largest magnitude c of a key's value codes lies
// below 2^8: a weight may be that much larger beside it in fp16. kNoCode: zeros.
constexpr uint32_t kNoCode = 7u;
__device__ __forceinline__ uint32_t code_room(uint32_t c) {
  return c == 0u ? kNoCode : min(5u, 15u - (c >> 3));
}

// The reference M of a row in such a unit, from its value so far, what the chunk's
// keys ask for (ref: their weights are then at most 2^15) and the largest magnitude
// of the row's sums, in units of 2^M (a key's product is at most 2^19): it falls no
// lower than they reach. A whole number, so that sums follow it exactly.
__device__ __forceinline__ float apart_reference(float M, float ref, float sums) {
  const float held = sums > 0.f ? M + fminf(log2f(sums) - 19.f, 0.f) : -INFINITY;
  const float want = fmaxf(ref, held);
  if (want == -INFINITY || (want <= M && want > M - 4.f)) return M;
  return ceilf(want);
}

// Tiles of sequence b, its first query row, queries and length. A length that
// is out of range (or shorter than the queries) gives ok = false: its rows
// have no keys.
struct Seq {
  int first, n, len;
  bool ok;
  unsigned err;  // its error-word bit when not ok
};

__device__ __forceinline__ Seq sequence(const Q8AttendArgs& a, int b) {
  Seq s;
  s.ok = token_range(a.cu, b, a.N, s.first, s.n);
  s.err = s.ok ? 0u : kErrOffsets;
  s.len = a.seq_lens[b];
  // a single-token call takes an empty sequence; n queries need n tokens
  if (s.len < 0 || s.len > a.T || (a.cu && s.len < s.n)) {
    s.ok = false;
    s.err |= kErrSeqLen;
    s.len = 0;
  }
  return s;
}

__device__ __forceinline__ int tiles_of(const Q8AttendArgs& a, int n, int rows) {
  return (int)(((long)n * a.G + rows - 1) / rows);
}

// Positions [lo, hi) of the keys that rows [r0, r0 + rows) of a sequence see
// (their union). Rows of a bad sequence see none.
__device__ __forceinline__ void key_span(const Q8AttendArgs& a, const Seq& s, int r0, int rows,
                                         int& lo, int& hi) {
  lo = hi = 0;
  if (!s.ok || s.len == 0) return;
  const int t0 = r0 / a.G;
  const int t1 = min(s.n - 1, (r0 + rows - 1) / a.G);
  const int at = s.len - s.n;  // position of the sequence's first query
  hi = at + t1 + 1;
  if (a.keys == KEYS_WINDOW) lo = max(0, at + t0 + 1 - a.window);
}

// Chunks of `chunk` keys that a tile needs; at least one, so that every row is written.
__device__ __forceinline__ int chunks_of(const Q8AttendArgs& a, const Seq& s, int r0, int rows,
                                         int chunk) {
  if (a.keys == KEYS_BLOCKS) return (int)(((long)a.n * a.page + chunk - 1) / chunk);
  int lo, hi;
  key_span(a, s, r0, rows, lo, hi);
  if (hi <= lo) return 1;
  return (hi + chunk - 1) / chunk - lo / chunk;
}

// Places of the tensor-memory kernel's plan for a chunk of a tile: the halves
// of its rows that are not empty.
__device__ __forceinline__ int tc_weight(int rows) { return rows > kQ8TcRows / 2 ? 2 : 1; }

// V c / C, in 32 bits where that holds it (a 64-bit division is slow).
__device__ __forceinline__ long split(long V, int c, int C) {
  if (V <= 0xffffffu && C <= 255) return (uint32_t)V * (uint32_t)c / (uint32_t)C;
  return V * c / C;
}

// Block that holds position x of V positions split over C blocks: the largest
// c with V c / C <= x.
__device__ __forceinline__ int block_of(long x, long V, int C) {
  int c = min(C - 1, (int)((float)x * (float)C / (float)V));
  while (c > 0 && split(V, c, C) > x) --c;
  while (c < C - 1 && split(V, c + 1, C) <= x) ++c;
  return c;
}

// Where the plan's prefix lives and how a tile maps to its sequence.
struct Plan {
  const long* pre;   // chunks (times KV heads) before each tile, [tiles + 1]
  const int* tseq;   // sequence of each tile; null: tile / rt
  const int* tbase;  // first tile of each sequence (with tseq)
  const int* lens;   // without tseq: length of each tile's sequence; -1: a bad one
  int tiles, rt;
};

// A place in the list of chunks: (tile, KV head, chunk).
struct Place {
  int tile, h, c, nc;
  __device__ __forceinline__ void init(const Plan& pl, int hkv, long x) {
    int lo = 0, hi = pl.tiles - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pl.pre[mid] <= x)
        lo = mid;
      else
        hi = mid - 1;
    }
    tile = lo;
    nc = (int)((pl.pre[lo + 1] - pl.pre[lo]) / hkv);
    const int r = (int)(x - pl.pre[lo]);
    h = r / nc;
    c = r - h * nc;
  }
  // Next chunk; true when it belongs to another unit.
  __device__ __forceinline__ bool next(const Plan& pl, int hkv) {
    if (++c < nc) return false;
    c = 0;
    if (++h == hkv) {
      h = 0;
      ++tile;
      if (tile < pl.tiles) nc = (int)((pl.pre[tile + 1] - pl.pre[tile]) / hkv);
    }
    return true;
  }
};

// The place that unit u (of tiles x KV heads) begins at.
__device__ __forceinline__ long unit_place(const Plan& pl, int hkv, int u) {
  const int tile = u / hkv;
  if (tile >= pl.tiles) return pl.pre[pl.tiles];
  return pl.pre[tile] + (u - tile * hkv) * ((pl.pre[tile + 1] - pl.pre[tile]) / hkv);
}

// The first place at or behind x at which a unit begins.
__device__ __forceinline__ long unit_start(const Plan& pl, int hkv, long x) {
  if (x >= pl.pre[pl.tiles]) return x;
  Place at;
  at.init(pl, hkv, x);
  return at.c == 0 ? x : x - at.c + at.nc;
}

// Per block: the unit of slot 2 c when that unit ends in the block (else -1),
// and the block it begins in.
struct MergeMeta {
  long unit;
  int from, pad;
};

// Launches so that the grid may be scheduled while its predecessor in the stream
// drains. The attention kernels wait (grid_dep_wait) before they read; the append's
// pages' kernel waits as it ends: its predecessor, an ordinary launch, is the query
// kernel, of which it reads nothing.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem,
                       cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

}  // namespace q8
}  // namespace nsa
