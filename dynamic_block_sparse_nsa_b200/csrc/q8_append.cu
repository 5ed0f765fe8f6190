// nsa_append_q8: new tokens' keys and values into the 8-bit paged cache, keys
// (and the queries of the same tokens) rotated by their position on the way.
//
//   x'[a], x'[b] = x[a] cos - x[b] sin, x[b] cos + x[a] sin   for each pair
//   s = 2^e, the smallest with max |x'| <= 448 s over the (page, head)'s new
//       components; never below the page's scale unless the call writes the
//       page's first token
//   code = e4m3(x' / s)
// The rotation is fp32, and the only rounding of a stored component is the
// one into its code. A scale that changes re-codes the page's other slots, so
// that they keep their values; both scales being powers of two, that is an
// exponent shift, exact but for codes that fall below e4m3's normal range.
//
// Bound by bytes (each input read once, each output written once) for long
// calls and by latency for one token per sequence. A (page, head) of K or V is
// one block's work: its rows stay in registers between the maximum and the
// codes, and no row is read twice (rows of the rotation table are, by each of the
// two passes). Query rows have a kernel of their own ahead of it, which the pages'
// blocks overlap, or blocks behind the pages' where they are few. With one token
// per sequence a warp takes a (sequence, head) of K or V instead, and more warps
// the query rows.
// Measured, 64 query heads on 4 KV heads, d = 128, bf16: 8192 tokens 64 us, 4.9
// TB/s in and out (loads in flight bound the query rows); 32 sequences of a token
// each 3.4 us. 11 chunks of up to 701 fp32 tokens (12 heads on 3, d = 64) 13 us.
#include <algorithm>

#include "q8_attend.cuh"

namespace nsa {
namespace {

using q8::Vec8;

constexpr int kThreads = 256;
constexpr int kTogether = 2048;  // most blocks of query rows that share the pages' launch

// The two 8-component pieces of a row that thread j of its d / 16 owns: with
// pairs (i, i + rot / 2) they are each other's partners, behind the rotated
// part (and with pairs (2i, 2i + 1)) any two.
__device__ __forceinline__ void pieces(int j, int rot, int& a, int& b) {
  if (j < rot / 16) {
    a = 8 * j;
    b = rot / 2 + 8 * j;
  } else {
    a = 16 * j;
    b = a + 8;
  }
}

// Cosines [8] and sines [8] of a row's pieces at a position: with pairs
// (i, i + rot / 2) those of pairs 8 j .., with pairs (2i, 2i + 1) those of
// 4 j .. 4 j + 3 (piece a) and rot / 4 + 4 j .. (piece b).
template <bool HALF>
__device__ __forceinline__ void turn_of(float (&cs)[16], const Q8AppendArgs& a, int at, int j) {
  if (j >= a.rot / 16) return;
  const float* row = a.rope + (long)at * a.rot;
  const int p0 = HALF ? 8 * j : 4 * j;
  const int p1 = HALF ? 8 * j + 4 : a.rot / 4 + 4 * j;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float* from = row + k * (a.rot / 2);
    *reinterpret_cast<float4*>(&cs[8 * k]) = __ldg(reinterpret_cast<const float4*>(from + p0));
    *reinterpret_cast<float4*>(&cs[8 * k + 4]) = __ldg(reinterpret_cast<const float4*>(from + p1));
  }
}

// Rotates a pair. The products are rounded apart, not fused into the sum: any fp32
// evaluation that rounds each product then gives the same key, and the same code
// where it lies near the middle of two (a fused one may not).
__device__ __forceinline__ void turn_pair(float& u, float& v, float c, float s) {
  const float a = __fsub_rn(__fmul_rn(u, c), __fmul_rn(v, s));
  v = __fadd_rn(__fmul_rn(v, c), __fmul_rn(u, s));
  u = a;
}

// Rotates the 16 components x = [piece a, piece b] of a row.
template <bool HALF>
__device__ __forceinline__ void rotate(float (&x)[16], const float (&cs)[16],
                                       const Q8AppendArgs& a, int j) {
  if (j >= a.rot / 16) return;
  if (HALF) {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn_pair(x[i], x[8 + i], cs[i], cs[8 + i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn_pair(x[2 * i], x[2 * i + 1], cs[i], cs[8 + i]);
  }
}

// Largest magnitude of the finite components; the others become NaN, which is
// how the cache holds them.
__device__ __forceinline__ float finite_max(float (&x)[16]) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float m = fabsf(x[i]);
    if (m < INFINITY)
      a = fmaxf(a, m);
    else
      x[i] = __uint_as_float(0x7fffffffu);
  }
  return a;
}

// Codes of x / s into a page row, and the values they stand for into `held`.
template <typename T>
__device__ __forceinline__ void put_codes(const float (&x)[16], float s, float inv, uint8_t* row,
                                          T* held, int a, int b) {
  uint16_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = q8::float2_to_e4m3x2(x[2 * i] * inv, x[2 * i + 1] * inv);
  const uint32_t* w = reinterpret_cast<const uint32_t*>(c);
  *reinterpret_cast<uint2*>(row + a) = make_uint2(w[0], w[1]);
  *reinterpret_cast<uint2*>(row + b) = make_uint2(w[2], w[3]);
  if (held) {
    float y[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 v = q8::e4m3x2_to_float2(c[i]);
      y[2 * i] = v.x * s;
      y[2 * i + 1] = v.y * s;
    }
    Vec8<T>::store(held + a, y);
    Vec8<T>::store(held + b, y + 8);
  }
}

// Re-codes `bytes` (a multiple of 16) of a page from its old scale to a new
// one. Only a page that the call begins can get a smaller scale: what its stale
// slots then cannot hold becomes NaN.
__device__ __forceinline__ void recode(uint8_t* page, int bytes, float ratio, int thread,
                                       int threads) {
  ratio = fminf(ratio, 0x1p100f);  // (more than enough for NaN; 0 * infinity is none of 0's)
#pragma unroll 4
  for (int at = 16 * thread; at < bytes; at += 16 * threads) {
    uint4 v = *reinterpret_cast<const uint4*>(page + at);
    uint16_t* c = reinterpret_cast<uint16_t*>(&v);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float2 f = q8::e4m3x2_to_float2(c[i]);
      f.x *= ratio;
      f.y *= ratio;
      // 464 is halfway from the largest code to what would follow it
      if (fabsf(f.x) > 464.f) f.x = __uint_as_float(0x7fffffffu);
      if (fabsf(f.y) > 464.f) f.y = __uint_as_float(0x7fffffffu);
      c[i] = q8::float2_to_e4m3x2(f.x, f.y);
    }
    *reinterpret_cast<uint4*>(page + at) = v;
  }
}

// Scale of a (page, head) that gets new components of magnitude up to `a`.
__device__ __forceinline__ float new_scale(float a, float old, bool first) {
  const float need = q8::exp2_int(q8::scale_exponent(a));
  return first ? need : fmaxf(old, need);
}

// Whether sequence b's n tokens at positions from `pos` on fit its table and
// the rotation table.
__device__ __forceinline__ bool place_ok(const Q8AppendArgs& a, int pos, int n) {
  return pos >= 0 && (long)pos + n <= a.T && (a.rot == 0 || (long)pos + n <= a.rope_len);
}

// A row of the queries, at position `at`, rotated into q_out.
template <typename T, bool HALF>
__device__ __forceinline__ void turn_query(const Q8AppendArgs& a, long row, int at, int j) {
  int pa, pb;
  pieces(j, a.rot, pa, pb);
  const T* src = static_cast<const T*>(a.q) + row * a.d;
  float x[16], cs[16];
  Vec8<T>::load(src + pa, x);
  Vec8<T>::load(src + pb, x + 8);
  turn_of<HALF>(cs, a, at, j);
  rotate<HALF>(x, cs, a, j);
  T* dst = static_cast<T*>(a.q_out) + row * a.d;
  Vec8<T>::store(dst + pa, x);
  Vec8<T>::store(dst + pb, x + 8);
}

// One token per sequence: a warp per (sequence, KV head, K or V), then warps
// that take 32 / (d / 16) query rows each.
template <typename T, bool HALF>
__global__ void __launch_bounds__(kThreads) q8_append_step_kernel(Q8AppendArgs a) {
  const int lane = threadIdx.x & 31;
  const long w = blockIdx.x * (long)(kThreads / 32) + (threadIdx.x >> 5);
  const int tpr = a.d / 16;
  const long items = (long)a.B * a.Hkv * 2;
  if (w >= items) {
    const long row = (w - items) * (32 / tpr) + lane / tpr;
    if (!a.q || row >= (long)a.B * a.Hq) return;
    const int pos = a.pos[row / a.Hq];
    if (place_ok(a, pos, 1)) turn_query<T, HALF>(a, row, pos, lane % tpr);
    return;
  }
  const int isv = (int)(w & 1), h = (int)((w >> 1) % a.Hkv), b = (int)((w >> 1) / a.Hkv);
  const int pos = a.pos[b];
  if (!place_ok(a, pos, 1)) {
    if (lane == 0) atomicOr(a.err, kErrAppendPos);
    return;
  }
  const int slot = pos % a.page;
  const int pid = a.table[(long)b * a.max_pages + pos / a.page];
  if (pid < 0 || pid >= a.num_pages) {
    if (lane == 0) atomicOr(a.err, kErrPage);
    return;
  }
  const long ph = (long)pid * a.Hkv + h;
  float* sp = (isv ? a.v_scale : a.k_scale) + ph;
  uint8_t* page = (isv ? a.v_pages : a.k_pages) + ph * a.page * a.d;
  const float old = *sp;
  const long row = (long)b * a.Hkv + h;
  float x[16];
  float amax = 0.f;
  int pa = 0, pb = 0;
  if (lane < tpr) {
    pieces(lane, a.rot, pa, pb);
    const T* src = static_cast<const T*>(isv ? a.v_new : a.k_new) + row * a.d;
    Vec8<T>::load(src + pa, x);
    Vec8<T>::load(src + pb, x + 8);
    if (!isv) {
      float cs[16];
      turn_of<HALF>(cs, a, pos, lane);
      rotate<HALF>(x, cs, a, lane);
    }
    amax = finite_max(x);
  }
  amax = warp_max(amax);
  const float s = new_scale(amax, old, slot == 0);
  if (s != old) {
    recode(page, slot * a.d, old / s, lane, 32);
    recode(page + (slot + 1) * a.d, (a.page - slot - 1) * a.d, old / s, lane, 32);
  }
  if (lane < tpr) {
    T* held = static_cast<T*>(isv ? a.v_out : a.k_out);
    put_codes<T>(x, s, 1.f / s, page + slot * a.d, held ? held + row * a.d : nullptr, pa, pb);
  }
  __syncwarp();  // every lane has read the old scale
  if (lane == 0) *sp = s;
}

// Sequence of token t: the last b with cu[b] <= t (cu ascending).
__device__ __forceinline__ int sequence_of(const int32_t* cu, int B, int t) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] <= t)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// Query rows of a call with offsets: a block takes `tokens` tokens' heads. Each
// thread has one row under way, and many blocks on an SM hide the latency (two
// rows a thread at fewer blocks an SM: 70 us for a call of 8192 tokens with 64
// heads, against 64).
template <typename T, bool HALF>
__device__ __forceinline__ void query_rows(const Q8AppendArgs& a, int tokens, int block) {
  const int tpr = a.d / 16, rpp = kThreads / tpr, j = threadIdx.x % tpr;
  const int t0 = block * tokens;
  const int rows = min(tokens, a.N - t0) * a.Hq;
  int token = -1, at = -1;  // of the row before: a token's heads share them
  for (int r = threadIdx.x / tpr; r < rows; r += rpp) {
    const int t = t0 + (tokens == 1 ? 0 : (int)((uint32_t)r / (uint32_t)a.Hq));
    if (t != token) {
      token = t;
      at = -1;
      const int b = sequence_of(a.cu, a.B, t);
      int f, n;
      if (q8::token_range(a.cu, b, a.N, f, n) && t >= f && t < f + n) {
        const int pos = a.pos[b];
        if (place_ok(a, pos, n)) at = pos + t - f;
      }
    }
    if (at >= 0) turn_query<T, HALF>(a, (long)t0 * a.Hq + r, at, j);
  }
}

template <typename T, bool HALF>
__global__ void __launch_bounds__(kThreads, 5) q8_append_query_kernel(Q8AppendArgs a, int tokens) {
  ptx::grid_dep_launch();  // (the pages' kernel needs nothing from here)
  query_rows<T, HALF>(a, tokens, blockIdx.x);
}

// K and V of a call with offsets: a block per (page of a sequence's new tokens,
// KV head, K or V). NP: passes of the block's threads over a page's rows. Of a
// short call the blocks from `pages` on rotate the query rows.
template <typename T, bool HALF, int NP>
__global__ void __launch_bounds__(kThreads) q8_append_kernel(Q8AppendArgs a, unsigned pages,
                                                             int tokens) {
  if (blockIdx.x >= pages) {
    query_rows<T, HALF>(a, tokens, blockIdx.x - pages);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tpr = a.d / 16, rpp = kThreads / tpr;
  const int j = tid % tpr;
  const long parts = 2l * a.Hkv;
  __shared__ int s_seq, s_page, s_first, s_n, s_pos, s_sum[kThreads / 32];
  __shared__ float s_max[kThreads / 32];
  const int item = (int)(blockIdx.x / parts), part = (int)(blockIdx.x % parts);
  // (a query kernel before this one is not read from, but ends before this one does)
  struct Wait {
    __device__ ~Wait() { ptx::grid_dep_wait(); }
  } wait;
  const int isv = part & 1, h = part >> 1;
  // item -> (sequence, page of its new tokens): sequences take
  // (pos + n - 1) / page - pos / page + 1 items each, in order
  if (tid == 0) s_seq = -1;
  __syncthreads();
  int base = 0;
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const int b = b0 + tid;
    int f = 0, n = 0, pos = 0, mine = 0;
    if (b < a.B) {
      const bool ok = q8::token_range(a.cu, b, a.N, f, n);
      pos = a.pos[b];
      if (!ok || (n > 0 && !place_ok(a, pos, n))) {
        if (blockIdx.x == 0) atomicOr(a.err, ok ? kErrAppendPos : kErrOffsets);
        n = 0;
      }
      if (n > 0) mine = (pos + n - 1) / a.page - pos / a.page + 1;
    }
    int run = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += up;
    }
    if (lane == 31) s_sum[warp] = run;
    __syncthreads();
    int before = base, all = 0;
#pragma unroll
    for (int k = 0; k < kThreads / 32; ++k) {
      if (k < warp) before += s_sum[k];
      all += s_sum[k];
    }
    const int start = before + run - mine;
    if (item >= start && item < start + mine) {
      s_seq = b;
      s_page = pos / a.page + item - start;
      s_first = f;
      s_n = n;
      s_pos = pos;
    }
    base += all;
    __syncthreads();
    // (the first block goes through all of them, for the error word)
    if (blockIdx.x > 0 && (s_seq >= 0 || base > item)) break;
  }
  const int b = s_seq;
  if (b < 0) return;  // more blocks than items
  const int f = s_first, pos = s_pos;
  const int x0 = max(pos, s_page * a.page);  // positions of this page's new tokens
  const int x1 = min(pos + s_n, (int)min((long)(s_page + 1) * a.page, (long)a.T));
  const int slot = x0 - s_page * a.page, rows = x1 - x0;
  const int pid = a.table[(long)b * a.max_pages + s_page];
  int pa, pb;
  pieces(j, a.rot, pa, pb);
  const T* src = static_cast<const T*>(isv ? a.v_new : a.k_new);
  const long row0 = ((long)f + (x0 - pos)) * a.Hkv + h;  // its rows are Hkv apart
  // rows stay as they were read; each of the two passes over them rotates anew
  typename Vec8<T>::Raw raw[NP][2];
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const int r = k * rpp + tid / tpr;
    if (r < rows) {
      const T* p = src + (row0 + (long)r * a.Hkv) * a.d;
      raw[k][0] = Vec8<T>::load_raw(p + pa);
      raw[k][1] = Vec8<T>::load_raw(p + pb);
    }
  }
  auto row_values = [&](int k, int r, float (&x)[16]) {
    Vec8<T>::unpack(raw[k][0], x);
    Vec8<T>::unpack(raw[k][1], x + 8);
    if (!isv) {
      float cs[16];
      turn_of<HALF>(cs, a, x0 + r, j);
      rotate<HALF>(x, cs, a, j);
    }
    return finite_max(x);
  };
  if (pid < 0 || pid >= a.num_pages) {
    if (tid == 0) atomicOr(a.err, kErrPage);
    return;
  }
  const long ph = (long)pid * a.Hkv + h;
  float* sp = (isv ? a.v_scale : a.k_scale) + ph;
  uint8_t* page = (isv ? a.v_pages : a.k_pages) + ph * a.page * a.d;
  const float old = *sp;
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const int r = k * rpp + tid / tpr;
    float x[16];
    if (r < rows) amax = fmaxf(amax, row_values(k, r, x));
  }
  amax = warp_max(amax);
  if (lane == 0) s_max[warp] = amax;
  __syncthreads();  // also: every thread has read the old scale
#pragma unroll
  for (int k = 0; k < kThreads / 32; ++k) amax = fmaxf(amax, s_max[k]);
  const float s = new_scale(amax, old, slot == 0);
  if (tid == 0) *sp = s;
  if (s != old && rows < a.page) {
    recode(page, slot * a.d, old / s, tid, kThreads);
    recode(page + (slot + rows) * a.d, (a.page - slot - rows) * a.d, old / s, tid, kThreads);
  }
  T* held = static_cast<T*>(isv ? a.v_out : a.k_out);
  const float inv = 1.f / s;
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const int r = k * rpp + tid / tpr;
    float x[16];
    if (r < rows) {
      row_values(k, r, x);
      put_codes<T>(x, s, inv, page + (slot + r) * a.d,
                   held ? held + (row0 + (long)r * a.Hkv) * a.d : nullptr, pa, pb);
    }
  }
}

template <typename T, bool HALF>
cudaError_t launch(const Q8AppendArgs& a, cudaStream_t stream) {
  const int tpr = a.d / 16;
  if (!a.cu) {
    TraceScope trace("append_q8", stream);
    long warps = (long)a.B * a.Hkv * 2;
    if (a.q) warps += ((long)a.B * a.Hq + 32 / tpr - 1) / (32 / tpr);
    const long blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
    q8_append_step_kernel<T, HALF><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
  }
  // two rounds of a block's query rows, or one token's heads
  const int tokens = std::max(1, 2 * (kThreads / tpr) / a.Hq);
  const int blocks = a.q ? (a.N + tokens - 1) / tokens : 0;
  // Few of them: one launch for both kinds of blocks (64 query heads, d = 128: 1000
  // tokens 9.4 us against 11.3, and 2 us less on the host; 2000 tokens 16.9 and
  // 17.4; 3000 tokens 29.8 and 27.2, for the pages' registers leave fewer blocks
  // of query rows on an SM).
  // (An ordinary launch, which all work before it precedes: the pages' kernel, launched
  // programmatically behind it, reads its inputs without a wait.)
  const bool together = blocks <= kTogether;
  if (!together) {
    TraceScope trace("append_q8_query", stream);
    q8_append_query_kernel<T, HALF><<<blocks, kThreads, 0, stream>>>(a, tokens);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  // a sequence's n tokens lie on at most n / page + 2 pages
  const long items = (long)a.N / a.page + 2l * (a.B < a.N ? a.B : a.N);
  const int passes = a.page * a.d / 16 / kThreads;  // of the threads over a page's rows
  auto kern = passes <= 1   ? q8_append_kernel<T, HALF, 1>
              : passes == 2 ? q8_append_kernel<T, HALF, 2>
                            : q8_append_kernel<T, HALF, 4>;
  TraceScope trace("append_q8", stream);
  const unsigned pages = (unsigned)(items * a.Hkv * 2);
  if (!together) return q8::launch_pdl(kern, dim3(pages), dim3(kThreads), 0, stream, a, pages, tokens);
  kern<<<pages + blocks, kThreads, 0, stream>>>(a, pages, tokens);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_q8_append(const Q8AppendArgs& a, nsa_dtype dtype, cudaStream_t stream) {
  if (a.style == NSA_ROPE_HALF)
    return dtype == NSA_DTYPE_BF16 ? launch<__nv_bfloat16, true>(a, stream)
                                   : launch<float, true>(a, stream);
  return dtype == NSA_DTYPE_BF16 ? launch<__nv_bfloat16, false>(a, stream)
                                 : launch<float, false>(a, stream);
}

}  // namespace nsa
