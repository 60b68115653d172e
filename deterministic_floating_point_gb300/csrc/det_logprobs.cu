// det_token_logprobs and det_token_logprobs_backward (include/det_model.h).
//
// A row's statistics are S = sum exp(x - m) and T = sum exp(x - m) (x - m)
// with m the row's maximum: lse = m + log S, entropy = log S - T / S, the log
// probability of a token (x[token] - m) - log S.  One CTA takes a row and
// reads it once.  The order of the additions is fixed by element index: thread
// t of 512 takes the pairs (2t, 2t + 1), (2t + 1024, 2t + 1025), ... (single
// elements in f32), keeps its own running maximum and sums relative to it,
// and the 512 triples are joined by a tree.  So a row's bits depend neither on
// the other rows nor on its alignment.
#include "det_model.cuh"

#include <algorithm>

namespace det {
namespace {

constexpr int kRowThreads = 512;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kWords = 16;   // 4-byte words of a thread's chunk

template <typename T> struct Word;   // what a 4-byte word of a row holds
template <> struct Word<float> {
  static constexpr int N = 1;
  static constexpr unsigned kMasked = 0xff800000u;   // -inf
  static __device__ __forceinline__ float get(unsigned w, int) { return __uint_as_float(w); }
  static __device__ __forceinline__ unsigned larger(unsigned a, unsigned b) {
    return __float_as_uint(max_nan(__uint_as_float(a), __uint_as_float(b)));
  }
};
template <> struct Word<__nv_bfloat16> {
  static constexpr int N = 2;
  static constexpr unsigned kMasked = 0xff80ff80u;
  static __device__ __forceinline__ float get(unsigned w, int j) {
    return __uint_as_float(j ? (w & 0xffff0000u) : (w << 16));
  }
  static __device__ __forceinline__ unsigned larger(unsigned a, unsigned b) {
    unsigned r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ unsigned pack(float a, float b) {   // to nearest
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const unsigned*>(&v);
  }
};
template <> struct Word<__half> {
  static constexpr int N = 2;
  static constexpr unsigned kMasked = 0xfc00fc00u;
  static __device__ __forceinline__ float get(unsigned w, int j) {
    return __half2float(__ushort_as_half((unsigned short)(j ? (w >> 16) : w)));
  }
  static __device__ __forceinline__ unsigned larger(unsigned a, unsigned b) {
    unsigned r;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ unsigned pack(float a, float b) {   // to nearest
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const unsigned*>(&v);
  }
};

// Two 32-bit lanes in a 64-bit register.
__device__ __forceinline__ unsigned long long pack_f32x2(float a, float b) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack_f32x2(unsigned long long v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ unsigned long long add_f32x2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long mul_f32x2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long fma_f32x2(unsigned long long a, unsigned long long b,
                                                        unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Word w of a row (elements N w, N w + 1), with masked logits past its end.
template <typename T>
__device__ __forceinline__ unsigned load_word(const T* row, long long w, long long vocab, bool words_aligned) {
  if constexpr (Word<T>::N == 1) {
    return w < vocab ? __float_as_uint(__ldg(row + w)) : Word<T>::kMasked;
  } else {
    const long long e = 2 * w;
    const unsigned short* p = reinterpret_cast<const unsigned short*>(row);
    if (e + 1 < vocab) {
      if (words_aligned) return __ldg(reinterpret_cast<const unsigned*>(p + e));
      return (unsigned)__ldg(p + e) | ((unsigned)__ldg(p + e + 1) << 16);
    }
    if (e < vocab) return (unsigned)__ldg(p + e) | (Word<T>::kMasked & 0xffff0000u);
    return Word<T>::kMasked;
  }
}

// Running maximum and the two sums relative to it (relative to 0 while the
// maximum is -inf: both sums are 0 then).
struct Stat {
  float m, s, t;
};
__device__ __forceinline__ float stat_base(float m) { return m == kNegInf ? 0.0f : m; }
// a and b joined, a's elements the earlier ones.
__device__ __forceinline__ Stat stat_join(const Stat& a, const Stat& b) {
  Stat r;
  r.m = max_nan(a.m, b.m);
  const float base = stat_base(r.m);
  // a side without a logit above -inf has sums of 0; its maximum may not enter (0 * inf)
  const float da = a.m == kNegInf ? 0.0f : a.m - base, db = b.m == kNegInf ? 0.0f : b.m - base;
  const float ca = exp2_approx(da * kLog2e), cb = exp2_approx(db * kLog2e);
  r.s = a.s * ca + b.s * cb;
  r.t = (ca > 0.0f ? ca * fmaf(a.s, da, a.t) : ca) + (cb > 0.0f ? cb * fmaf(b.s, db, b.t) : cb);
  return r;
}

// The sorted list of a warp's best keys, the largest in lane 0; a key is the
// value's order key above the complement of its index, so no two are equal
// and the lowest index wins among equal values.
__device__ __forceinline__ void list_insert(unsigned long long& mine, unsigned long long key, int lane) {
  const int pos = __popc(__ballot_sync(0xffffffffu, mine > key));
  const unsigned long long up = __shfl_up_sync(0xffffffffu, mine, 1);
  if (lane > pos) mine = up;
  else if (lane == pos) mine = key;
}

struct RowOut {
  float *logprob, *entropy, *lse, *top_logprob;
  int32_t* top_index;
};

// The top_k largest of the row, after the pass: `best` is the thread's own
// largest element.  The k-th largest of the two best threads of every warp is
// a lower bound of the row's k-th largest element, so only threads whose best
// reaches it are looked through again, each by its whole warp.
template <typename T>
__device__ void top_alternatives(const T* row, long long vocab, bool words_aligned, float best, int k, float m,
                                 float log_s, long long r, const RowOut& out) {
  __shared__ unsigned sh_best[2 * kRowWarps];
  __shared__ unsigned sh_floor;
  __shared__ unsigned long long sh_list[kRowWarps * DET_MAX_TOP_K];
  __shared__ int sh_count[kRowWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned key = order_key(best);
  const unsigned first = __reduce_max_sync(0xffffffffu, key);
  const int owner = __ffs(__ballot_sync(0xffffffffu, key == first)) - 1;
  const unsigned second = __reduce_max_sync(0xffffffffu, lane == owner ? 0u : key);
  if (lane == 0) {
    sh_best[2 * warp] = first;
    sh_best[2 * warp + 1] = second;
  }
  __syncthreads();
  if (warp == 0) {
    const unsigned b = sh_best[lane];
    int above = 0;
    for (int j = 0; j < 32; ++j) {
      const unsigned o = __shfl_sync(0xffffffffu, b, j);
      above += (o > b || (o == b && j < lane)) ? 1 : 0;
    }
    if (above == k - 1) sh_floor = b;
  }
  __syncthreads();
  const unsigned floor_key = sh_floor;
  const long long words = (vocab + Word<T>::N - 1) / Word<T>::N;
  unsigned long long mine = 0;   // below every key: an element's key has a nonzero complement of its index
  unsigned todo = __ballot_sync(0xffffffffu, key >= floor_key);
  while (todo) {
    const int owner_lane = __ffs(todo) - 1;
    todo &= todo - 1;
    for (long long base = warp * 32 + owner_lane; base < words; base += 32LL * kRowThreads) {
      const long long w = base + (long long)lane * kRowThreads;
      const unsigned word = w < words ? load_word(row, w, vocab, words_aligned) : 0u;
#pragma unroll
      for (int j = 0; j < Word<T>::N; ++j) {
        const long long e = w * Word<T>::N + j;
        unsigned long long cand = 0;
        if (e < vocab) {
          const unsigned ek = order_key(Word<T>::get(word, j));
          if (ek >= floor_key) cand = ((unsigned long long)ek << 32) | (unsigned)~(unsigned)e;
        }
        const unsigned long long worst = __shfl_sync(0xffffffffu, mine, k - 1);
        unsigned hits = __ballot_sync(0xffffffffu, cand > worst);
        while (hits) {
          const int src = __ffs(hits) - 1;
          hits &= hits - 1;
          list_insert(mine, __shfl_sync(0xffffffffu, cand, src), lane);
        }
      }
    }
  }
  const int count = min(k, __popc(__ballot_sync(0xffffffffu, mine != 0)));
  if (lane == 0) sh_count[warp] = count;
  __syncthreads();
  int at = 0, total = 0;
  for (int w = 0; w < kRowWarps; ++w) {
    at += w < warp ? sh_count[w] : 0;
    total += sh_count[w];
  }
  if (lane < count) sh_list[at + lane] = mine;
  __syncthreads();
  if (threadIdx.x < total) {
    const unsigned long long c = sh_list[threadIdx.x];
    int rank = 0;
    for (int j = 0; j < total; ++j) rank += sh_list[j] > c ? 1 : 0;
    if (rank < k) {
      const float x = key_value((unsigned)(c >> 32));
      if (out.top_index) out.top_index[r * k + rank] = (int32_t)~(unsigned)c;
      if (out.top_logprob) out.top_logprob[r * k + rank] = (x - m) - log_s;
    }
  }
}

// A row in chunks of 512 threads x 16 words, a thread's word i of chunk c
// being word (16 c + i) 512 + t: a warp reads 128 neighbouring bytes.  Words
// are 4-byte aligned in memory, except in 16-bit rows that start at an odd
// element (ODD): there a thread reads the aligned word that holds the first of
// its two elements and gets the other from the next lane, whose word holds it
// (the last lane's from an extra word a lane loads for each i).
template <typename T>
struct RowReader {
  const T* row;
  long long vocab, words;
  bool odd;
  const unsigned* base;   // the aligned word with (the first element of) the thread's word 0
  const unsigned* extra;  // of the word behind the warp's last, for i = lane % 16

  __device__ __forceinline__ RowReader(const T* row_, long long vocab_) : row(row_), vocab(vocab_) {
    words = (vocab + Word<T>::N - 1) / Word<T>::N;
    odd = Word<T>::N == 2 && (reinterpret_cast<uintptr_t>(row) & 3);
    const unsigned* aligned = reinterpret_cast<const unsigned*>(reinterpret_cast<uintptr_t>(row) & ~(uintptr_t)3);
    base = aligned + threadIdx.x;
    extra = aligned + (threadIdx.x & 15) * kRowThreads + (threadIdx.x & ~31u) + 32;
  }
  // Raw words of the chunk whose first word is w0.  A word read here lies
  // inside the row; what is not is left to finish().
  __device__ __forceinline__ void start(long long w0, unsigned (&x)[kWords], unsigned& more) const {
    // every aligned word up to index w0 + 16 * 512 is inside the row, and word 0 is not half outside
    const bool inside = odd ? w0 > 0 && 2 * (w0 + kWords * kRowThreads) < vocab
                            : Word<T>::N * (w0 + kWords * kRowThreads) <= vocab;
    if (inside) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) x[i] = __ldg(base + w0 + i * kRowThreads);
      if (odd) more = __ldg(extra + w0);
    } else if (!odd) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) x[i] = load_word(row, w0 + threadIdx.x + i * kRowThreads, vocab, true);
    }
  }
  __device__ __forceinline__ void finish(long long w0, unsigned (&x)[kWords], unsigned more) const {
    if (!odd) return;
    if (w0 > 0 && 2 * (w0 + kWords * kRowThreads) < vocab) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        unsigned next = __shfl_down_sync(0xffffffffu, x[i], 1);
        const unsigned last = __shfl_sync(0xffffffffu, more, i);
        if ((threadIdx.x & 31) == 31) next = last;
        x[i] = __funnelshift_r(x[i], next, 16);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) x[i] = load_word(row, w0 + threadIdx.x + i * kRowThreads, vocab, false);
    }
  }
};

// The chunk's elements added to the thread's statistics.
template <typename T>
__device__ __forceinline__ void add_chunk(Stat& st, const unsigned (&x)[kWords]) {
  constexpr int N = Word<T>::N;
  unsigned mx[kWords / 2];
#pragma unroll
  for (int i = 0; i < kWords / 2; ++i) mx[i] = Word<T>::larger(x[i], x[i + kWords / 2]);
#pragma unroll
  for (int s = kWords / 4; s > 0; s >>= 1)
#pragma unroll
    for (int i = 0; i < s; ++i) mx[i] = Word<T>::larger(mx[i], mx[i + s]);
  float m = Word<T>::get(mx[0], 0);
  if (N == 2) m = max_nan(m, Word<T>::get(mx[0], 1));
  if (!(m <= st.m)) {   // a new maximum (or NaN): the sums so far relative to it
    if (st.m != kNegInf) {
      const float d = st.m - m, f = exp2_approx(d * kLog2e);
      st.t = f > 0.0f ? f * fmaf(st.s, d, st.t) : f;   // no 0 * inf
      st.s *= f;
    }
    st.m = max_nan(st.m, m);
  }
  const float base = stat_base(st.m);
  const unsigned long long minus = pack_f32x2(-base, -base), scale = pack_f32x2(kLog2e, kLog2e);
  unsigned long long s2 = 0, t2 = 0;   // of elements 0 and 1 of the words (f32: even and odd words)
#pragma unroll
  for (int i = 0; i < kWords; i += 3 - N) {
    const float a = Word<T>::get(x[i], 0), b = N == 2 ? Word<T>::get(x[i], 1) : Word<T>::get(x[(i + 1) % kWords], 0);
    const float2 y = unpack_f32x2(mul_f32x2(add_f32x2(pack_f32x2(a, b), minus), scale));
    // 2^-150 is 0 already; without the bound 0 * inf for a masked logit
    const float y0 = max_nan(y.x, -150.0f), y1 = max_nan(y.y, -150.0f);
    const unsigned long long e = pack_f32x2(exp2_approx(y0), exp2_approx(y1));
    s2 = add_f32x2(s2, e);
    t2 = fma_f32x2(e, pack_f32x2(y0, y1), t2);
  }
  const float2 s = unpack_f32x2(s2), t = unpack_f32x2(t2);
  st.s += s.x + s.y;
  st.t = fmaf(t.x + t.y, kLn2, st.t);   // y is d in units of log 2
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads, 2)
token_logprobs_kernel(const T* __restrict__ logits, long long vocab, long long row_stride,
                      const int32_t* __restrict__ tokens, int top_k, RowOut out) {
  __shared__ Stat sh[kRowWarps];
  const long long r = blockIdx.x;
  const T* row = logits + r * row_stride;
  const RowReader<T> reader(row, vocab);
  const bool aligned = !reader.odd;
  Stat st = {kNegInf, 0.0f, 0.0f};
  // the next chunk's loads are in flight while a chunk is added
  constexpr long long kStep = (long long)kRowThreads * kWords;
  unsigned x[kWords], ahead[kWords], more = 0, more_ahead = 0;
  if (reader.words > 0) reader.start(0, x, more);
  for (long long w0 = 0; w0 < reader.words; w0 += kStep) {
    if (w0 + kStep < reader.words) reader.start(w0 + kStep, ahead, more_ahead);
    reader.finish(w0, x, more);
    add_chunk<T>(st, x);
#pragma unroll
    for (int i = 0; i < kWords; ++i) x[i] = ahead[i];
    more = more_ahead;
  }
  const float best = st.m;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    Stat o;
    o.m = __shfl_xor_sync(0xffffffffu, st.m, s);
    o.s = __shfl_xor_sync(0xffffffffu, st.s, s);
    o.t = __shfl_xor_sync(0xffffffffu, st.t, s);
    st = (threadIdx.x & s) ? stat_join(o, st) : stat_join(st, o);
  }
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = st;
  __syncthreads();
  st = sh[0];
  for (int w = 1; w < kRowWarps; ++w) st = stat_join(st, sh[w]);
  const bool empty = st.m == kNegInf;
  const float log_s = empty ? 0.0f : logf(st.s);
  const float base = stat_base(st.m);
  if (threadIdx.x == 0) {
    if (out.lse) out.lse[r] = empty ? kNegInf : base + log_s;
    if (out.entropy) out.entropy[r] = empty ? 0.0f : log_s - st.t / st.s;
    if (out.logprob) {
      const long long tok = tokens[r];
      out.logprob[r] = tok >= 0 && tok < vocab ? (to_f32(row[tok]) - base) - log_s : 0.0f;
    }
  }
  if (top_k > 0) top_alternatives(row, vocab, aligned, best, top_k, base, log_s, r, out);
}

// ---------------------------------------------------------------------------
// The gradient: elementwise once lse and the entropy are known.

constexpr int kGradThreads = 256;
constexpr int kGradVecs = 4;   // 16-byte vectors of a thread
// From this magnitude on 32 bits hold lse to 2^-14 or worse (nothing of log S
// is left of it in a row at the types' lowest values): the row is summed again.
constexpr float kLseFar = 1024.0f;

// The maximum and the log of the sum relative to it of a whole row.
template <typename T>
__device__ float2 row_max_and_log_sum(const T* row, long long vocab) {
  __shared__ float sh[2][kGradThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float m = kNegInf, s = 0.0f;
  for (long long e = threadIdx.x; e < vocab; e += kGradThreads) m = fmaxf(m, to_f32(row[e]));
  for (int d = 1; d < 32; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  if (lane == 0) sh[0][warp] = m;
  __syncthreads();
  for (int w = 0; w < kGradThreads / 32; ++w) m = fmaxf(m, sh[0][w]);
  for (long long e = threadIdx.x; e < vocab; e += kGradThreads) s += exp2_approx((to_f32(row[e]) - m) * kLog2e);
  s = warp_pt(s);
  if (lane == 0) sh[1][warp] = s;
  __syncthreads();
  s = 0.0f;
  for (int w = 0; w < kGradThreads / 32; ++w) s += sh[1][w];
  return make_float2(m, logf(s));
}

// grad[v] = [v == token] g_l - p (c + g_h log p) with c = g_l + g_h * entropy.
struct GradRow {
  float base, log_s;   // log p = (x - base) - log_s
  float gl, gh, c;
  __device__ __forceinline__ float at(float x) const {
    // p is 0 from -150 on already; without the bound 0 * inf for a masked logit
    const float lp = max_nan((x - base) - log_s, -150.0f);
    return -exp2_approx(lp * kLog2e) * fmaf(gh, lp, c);
  }
};

// A CTA takes 256 x 4 vectors of 16 bytes of a row, counted from the row's
// first 16-byte boundary (the same one of both rows: SAME_PHASE), and the
// row's first CTA the elements before it and behind the last vector.  Where
// the rows' boundaries differ it goes by elements.
template <typename T, bool SAME_PHASE>
__global__ void __launch_bounds__(kGradThreads)
token_logprobs_grad_kernel(const T* __restrict__ logits, int vocab, long long row_stride,
                           const int32_t* __restrict__ tokens, const float* __restrict__ lse,
                           const float* __restrict__ entropy, const float* __restrict__ grad_logprob,
                           const float* __restrict__ grad_entropy, T* __restrict__ grad, long long grad_stride,
                           unsigned ctas_per_row) {
  constexpr int E = 16 / sizeof(T), N = Word<T>::N;
  const unsigned r = blockIdx.x / ctas_per_row, part = blockIdx.x - r * ctas_per_row;
  const T* row = logits + r * row_stride;
  T* g = grad + r * grad_stride;
  const int head = SAME_PHASE ? min((int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / (int)sizeof(T), vocab) : 0;
  const int vecs = SAME_PHASE ? (vocab - head) / E : 0;
  const int v0 = part * (kGradThreads * kGradVecs) + threadIdx.x;
  uint4 x[kGradVecs];
  if constexpr (SAME_PHASE) {
#pragma unroll
    for (int i = 0; i < kGradVecs; ++i)
      if (v0 + i * kGradThreads < vecs) x[i] = __ldg(reinterpret_cast<const uint4*>(row + head) + v0 + i * kGradThreads);
  }
  const float l = lse[r];
  const int tok = grad_logprob ? tokens[r] : -1;
  GradRow q;
  q.gl = tok >= 0 && tok < vocab ? grad_logprob[r] : 0.0f;
  q.gh = grad_entropy ? grad_entropy[r] : 0.0f;
  q.c = grad_entropy ? fmaf(q.gh, entropy[r], q.gl) : q.gl;
  q.base = l;
  q.log_s = 0.0f;
  if (fabsf(l) >= kLseFar && fabsf(l) < INFINITY) {
    const float2 ms = row_max_and_log_sum(row, vocab);
    q.base = ms.x;
    q.log_s = ms.y;
  }
  if (l == kNegInf) {   // a row without a logit above -inf: 0 throughout
    q.gl = q.gh = q.c = 0.0f;
    q.base = 0.0f;
  }
  if constexpr (SAME_PHASE) {
#pragma unroll
    for (int i = 0; i < kGradVecs; ++i) {
      const int v = v0 + i * kGradThreads;
      if (v >= vecs) break;
      const unsigned w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      float d[E];
#pragma unroll
      for (int j = 0; j < E; ++j) d[j] = q.at(Word<T>::get(w[j / N], j % N));
      const int at = tok - head - v * E;   // the token's place in the vector
      if (at >= 0 && at < E) {
#pragma unroll
        for (int j = 0; j < E; ++j) d[j] += j == at ? q.gl : 0.0f;
      }
      uint4 o;
      if constexpr (N == 1) {
        o = make_uint4(__float_as_uint(d[0]), __float_as_uint(d[1]), __float_as_uint(d[2]), __float_as_uint(d[3]));
      } else {
        unsigned y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = Word<T>::pack(d[2 * j], d[2 * j + 1]);
        o = make_uint4(y[0], y[1], y[2], y[3]);
      }
      reinterpret_cast<uint4*>(g + head)[v] = o;
    }
    if (part > 0) return;
    for (int k = threadIdx.x; k < vocab - vecs * E; k += kGradThreads) {
      const int e = k < head ? k : vecs * E + k;
      g[e] = from_f32<T>(q.at(to_f32(row[e])) + (e == tok ? q.gl : 0.0f));
    }
  } else {
    const int first = part * (kGradThreads * kGradVecs * E);
    for (int e = first + threadIdx.x; e < min(first + kGradThreads * kGradVecs * E, vocab); e += kGradThreads)
      g[e] = from_f32<T>(q.at(to_f32(row[e])) + (e == tok ? q.gl : 0.0f));
  }
}

template <typename T>
int launch_logprobs(const void* logits, long long rows, long long vocab, long long stride, const int32_t* tokens,
                    int top_k, const RowOut& out, cudaStream_t s) {
  launch_begin("det_token_logprobs", s);
  token_logprobs_kernel<T><<<(unsigned)rows, kRowThreads, 0, s>>>(static_cast<const T*>(logits), vocab, stride, tokens,
                                                                  top_k, out);
  launch_end(s);
  return check_launch("det_token_logprobs");
}

template <typename T>
int launch_grad(const void* logits, long long rows, long long vocab, long long stride, const int32_t* tokens,
                const float* lse, const float* entropy, const float* gl, const float* gh, void* grad,
                long long grad_stride, cudaStream_t s) {
  const long long per = (long long)kGradThreads * kGradVecs * (16 / sizeof(T)), ctas = (vocab + per - 1) / per;
  if (rows * ctas >= (1LL << 31)) return DET_ERR_TOO_LARGE;
  // every row pair starts at the same place of a 16-byte block
  const bool same = ((reinterpret_cast<uintptr_t>(logits) ^ reinterpret_cast<uintptr_t>(grad)) % 16 == 0) &&
                    (rows == 1 || (stride - grad_stride) * (long long)sizeof(T) % 16 == 0);
  launch_begin("det_token_logprobs_backward", s);
  if (same)
    token_logprobs_grad_kernel<T, true><<<(unsigned)(rows * ctas), kGradThreads, 0, s>>>(
        static_cast<const T*>(logits), (int)vocab, stride, tokens, lse, entropy, gl, gh, static_cast<T*>(grad),
        grad_stride, (unsigned)ctas);
  else
    token_logprobs_grad_kernel<T, false><<<(unsigned)(rows * ctas), kGradThreads, 0, s>>>(
        static_cast<const T*>(logits), (int)vocab, stride, tokens, lse, entropy, gl, gh, static_cast<T*>(grad),
        grad_stride, (unsigned)ctas);
  launch_end(s);
  return check_launch("det_token_logprobs_backward");
}

}  // namespace
}  // namespace det

using namespace det;

extern "C" int det_token_logprobs(const void* logits, int64_t rows, int64_t vocab, int64_t row_stride,
                                  const int32_t* tokens, int dtype, float* logprob_out, float* entropy_out,
                                  float* lse_out, int top_k, float* top_logprob_out, int32_t* top_index_out,
                                  void* stream) {
  if (!valid_model_dtype(dtype)) return DET_ERR_DTYPE;
  if (rows < 0 || vocab < 0 || row_stride < 0 || top_k < 0 || top_k > DET_MAX_TOP_K || top_k > vocab)
    return DET_ERR_INVALID_ARG;
  if (rows >= (1LL << 31) || vocab >= (1LL << 31)) return DET_ERR_TOO_LARGE;
  if (rows == 0) return DET_OK;
  if ((vocab > 0 && !logits) || (logprob_out && !tokens)) return DET_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(logits) % model_elem_size(dtype)) return DET_ERR_INVALID_ARG;
  const RowOut out = {logprob_out, entropy_out, lse_out, top_logprob_out, top_index_out};
  const cudaStream_t s = as_stream(stream);
  if (dtype == DET_F32) return launch_logprobs<float>(logits, rows, vocab, row_stride, tokens, top_k, out, s);
  if (dtype == DET_BF16) return launch_logprobs<__nv_bfloat16>(logits, rows, vocab, row_stride, tokens, top_k, out, s);
  return launch_logprobs<__half>(logits, rows, vocab, row_stride, tokens, top_k, out, s);
}

extern "C" int det_token_logprobs_backward(const void* logits, int64_t rows, int64_t vocab, int64_t row_stride,
                                           const int32_t* tokens, int dtype, const float* lse, const float* entropy,
                                           const float* grad_logprob, const float* grad_entropy, void* grad_logits,
                                           int64_t grad_row_stride, void* stream) {
  if (!valid_model_dtype(dtype)) return DET_ERR_DTYPE;
  if (rows < 0 || vocab < 0 || row_stride < 0) return DET_ERR_INVALID_ARG;
  if (rows > 1 && grad_row_stride < vocab) return DET_ERR_INVALID_ARG;   // rows of the result would overlap
  if (rows >= (1LL << 31) || vocab >= (1LL << 28)) return DET_ERR_TOO_LARGE;
  if (rows == 0 || vocab == 0) return DET_OK;
  if (!logits || !lse || !grad_logits || (grad_logprob && !tokens) || (grad_entropy && !entropy))
    return DET_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(logits) % model_elem_size(dtype) ||
      reinterpret_cast<uintptr_t>(grad_logits) % model_elem_size(dtype))
    return DET_ERR_INVALID_ARG;
  const cudaStream_t s = as_stream(stream);
  if (dtype == DET_F32)
    return launch_grad<float>(logits, rows, vocab, row_stride, tokens, lse, entropy, grad_logprob, grad_entropy,
                              grad_logits, grad_row_stride, s);
  if (dtype == DET_BF16)
    return launch_grad<__nv_bfloat16>(logits, rows, vocab, row_stride, tokens, lse, entropy, grad_logprob,
                                      grad_entropy, grad_logits, grad_row_stride, s);
  return launch_grad<__half>(logits, rows, vocab, row_stride, tokens, lse, entropy, grad_logprob, grad_entropy,
                             grad_logits, grad_row_stride, s);
}
