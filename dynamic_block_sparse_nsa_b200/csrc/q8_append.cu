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
// codes, so nothing is read twice; blocks behind those rotate query rows. With
// one token per sequence a warp takes a (sequence, head) of K or V instead.
#include "q8.cuh"

namespace nsa {
namespace {

using q8::Vec8;

constexpr int kThreads = 256;

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

// Rotates the 16 components x = [piece a, piece b] of a row by table row
// rope[rot] = [cos | sin].
__device__ __forceinline__ void rotate(float (&x)[16], const float* rope, int rot, int style,
                                       int j) {
  if (j >= rot / 16) return;
  const float* cs = rope;
  const float* sn = rope + rot / 2;
  if (style == NSA_ROPE_HALF) {
    float c[8], s[8];
    Vec8<float>::load(cs + 8 * j, c);
    Vec8<float>::load(sn + 8 * j, s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float u = x[i], v = x[8 + i];
      x[i] = u * c[i] - v * s[i];
      x[8 + i] = v * c[i] + u * s[i];
    }
  } else {
    // pairs 4j .. 4j + 3 in piece a, rot / 4 + 4j .. in piece b
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = (h ? rot / 4 : 0) + 4 * j;
      const float4 c = __ldg(reinterpret_cast<const float4*>(cs + at));
      const float4 s = __ldg(reinterpret_cast<const float4*>(sn + at));
      const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float u = x[8 * h + 2 * i], v = x[8 * h + 2 * i + 1];
        x[8 * h + 2 * i] = u * cc[i] - v * ss[i];
        x[8 * h + 2 * i + 1] = v * cc[i] + u * ss[i];
      }
    }
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

// A row of the queries: rotated into q_out.
template <typename T>
__device__ __forceinline__ void turn_query(const Q8AppendArgs& a, long row, int at, int j) {
  int pa, pb;
  pieces(j, a.rot, pa, pb);
  const T* src = static_cast<const T*>(a.q) + row * a.d;
  float x[16];
  Vec8<T>::load(src + pa, x);
  Vec8<T>::load(src + pb, x + 8);
  rotate(x, a.rope + (long)at * a.rot, a.rot, a.style, j);
  T* dst = static_cast<T*>(a.q_out) + row * a.d;
  Vec8<T>::store(dst + pa, x);
  Vec8<T>::store(dst + pb, x + 8);
}

// One token per sequence: a warp per (sequence, KV head, K or V), then warps
// that take 32 / (d / 16) query rows each.
template <typename T>
__global__ void __launch_bounds__(kThreads) q8_append_step_kernel(Q8AppendArgs a) {
  const int lane = threadIdx.x & 31;
  const long w = blockIdx.x * (long)(kThreads / 32) + (threadIdx.x >> 5);
  const int tpr = a.d / 16;
  const long items = (long)a.B * a.Hkv * 2;
  if (w >= items) {
    const long row = (w - items) * (32 / tpr) + lane / tpr;
    if (!a.q || row >= (long)a.B * a.Hq) return;
    const int pos = a.pos[row / a.Hq];
    if (place_ok(a, pos, 1)) turn_query<T>(a, row, pos, lane % tpr);
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
    if (!isv) rotate(x, a.rope + (long)pos * a.rot, a.rot, a.style, lane);
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

// NP: passes of the block's threads over a page's rows (page * d / 16 / 256).
template <typename T, int NP>
__global__ void __launch_bounds__(kThreads) q8_append_kernel(Q8AppendArgs a, int items,
                                                             int qrows_per_block) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tpr = a.d / 16, rpp = kThreads / tpr;
  const int j = tid % tpr;
  const long parts = 2l * a.Hkv;
  if (blockIdx.x >= items * parts) {
    // query rows
    const long first = (blockIdx.x - items * parts) * qrows_per_block;
    for (int r = tid / tpr; r < qrows_per_block; r += rpp) {
      const long row = first + r;
      const int t = (int)(row / a.Hq);
      if (t >= a.N) return;
      const int b = sequence_of(a.cu, a.B, t);
      int f, n;
      if (!q8::token_range(a.cu, b, a.N, f, n) || t < f || t >= f + n) continue;
      const int pos = a.pos[b];
      if (place_ok(a, pos, n)) turn_query<T>(a, row, pos + t - f, j);
    }
    return;
  }
  __shared__ int s_seq, s_page, s_sum[kThreads / 32];
  __shared__ float s_max[kThreads / 32];
  const int item = (int)(blockIdx.x / parts), part = (int)(blockIdx.x % parts);
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
    }
    base += all;
    __syncthreads();
    // (the first block goes through all of them, for the error word)
    if (blockIdx.x > 0 && (s_seq >= 0 || base > item)) break;
  }
  const int b = s_seq;
  if (b < 0) return;  // more blocks than items
  int f, n;
  q8::token_range(a.cu, b, a.N, f, n);
  const int pos = a.pos[b];
  const int x0 = max(pos, s_page * a.page);                       // positions of this page's
  const int x1 = min(pos + n, (int)min((long)(s_page + 1) * a.page, (long)a.T));  // new tokens
  const int slot = x0 - s_page * a.page, rows = x1 - x0;
  const int pid = a.table[(long)b * a.max_pages + s_page];
  if (pid < 0 || pid >= a.num_pages) {
    if (tid == 0) atomicOr(a.err, kErrPage);
    return;
  }
  const long ph = (long)pid * a.Hkv + h;
  float* sp = (isv ? a.v_scale : a.k_scale) + ph;
  uint8_t* page = (isv ? a.v_pages : a.k_pages) + ph * a.page * a.d;
  const float old = *sp;
  int pa, pb;
  pieces(j, a.rot, pa, pb);
  const T* src = static_cast<const T*>(isv ? a.v_new : a.k_new);
  const long row0 = ((long)f + (x0 - pos)) * a.Hkv + h;  // its rows are Hkv apart
  float x[NP][16];
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const int r = k * rpp + tid / tpr;
    if (r < rows) {
      const T* p = src + (row0 + (long)r * a.Hkv) * a.d;
      Vec8<T>::load(p + pa, x[k]);
      Vec8<T>::load(p + pb, x[k] + 8);
    }
  }
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const int r = k * rpp + tid / tpr;
    if (r < rows) {
      if (!isv) rotate(x[k], a.rope + (long)(x0 + r) * a.rot, a.rot, a.style, j);
      amax = fmaxf(amax, finite_max(x[k]));
    }
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
    if (r < rows)
      put_codes<T>(x[k], s, inv, page + (slot + r) * a.d,
                   held ? held + (row0 + (long)r * a.Hkv) * a.d : nullptr, pa, pb);
  }
}

template <typename T>
cudaError_t launch(const Q8AppendArgs& a, cudaStream_t stream) {
  const int tpr = a.d / 16;
  TraceScope trace("append_q8", stream);
  if (!a.cu) {
    long warps = (long)a.B * a.Hkv * 2;
    if (a.q) warps += ((long)a.B * a.Hq + 32 / tpr - 1) / (32 / tpr);
    const long blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
    q8_append_step_kernel<T><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
  }
  // a sequence's n tokens lie on at most n / page + 2 pages
  const long items = (long)a.N / a.page + 2l * (a.B < a.N ? a.B : a.N);
  const int qrows = 4 * (kThreads / tpr);
  const long qblocks = a.q ? ((long)a.N * a.Hq + qrows - 1) / qrows : 0;
  const unsigned blocks = (unsigned)(items * a.Hkv * 2 + qblocks);
  const int passes = a.page * a.d / 16 / kThreads;
  if (passes <= 1)
    q8_append_kernel<T, 1><<<blocks, kThreads, 0, stream>>>(a, (int)items, qrows);
  else if (passes == 2)
    q8_append_kernel<T, 2><<<blocks, kThreads, 0, stream>>>(a, (int)items, qrows);
  else
    q8_append_kernel<T, 4><<<blocks, kThreads, 0, stream>>>(a, (int)items, qrows);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_q8_append(const Q8AppendArgs& a, nsa_dtype dtype, cudaStream_t stream) {
  return dtype == NSA_DTYPE_BF16 ? launch<__nv_bfloat16>(a, stream) : launch<float>(a, stream);
}

}  // namespace nsa
