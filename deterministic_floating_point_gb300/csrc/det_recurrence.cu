// det_linear_recurrence and its gradient: h = a[t] h + u[t] along time, for
// every sequence and channel.
//
// A step is the map h -> a h + u; a run of steps is a map of the same kind,
// h -> A h + H with A the product of its decays and H its result from 0.  Time
// is cut into pieces of 16 steps (a warp), spans of 128 (a CTA of 8 warps) and
// of 1,024 (a cluster of 8 CTAs).  A warp reads its piece of 32 words of
// channels into registers once, forms (A, H), the CTA's warps and then the
// cluster's CTAs exchange these through (distributed) shared memory, and each
// warp runs through its piece again, in registers, from the state it now
// knows.  A cluster goes through its sequence in steps of 1,024 and carries
// the state in registers; the next piece is on its way meanwhile.  So every
// input is read once and every output written once, and nothing waits on memory
// that another CTA writes.  Pieces are joined in the order of time, always from
// the same borders, so the bits of a step are a function of the steps before it.
//
// The gradient runs the same way from the end.  With m = a[t] l the value that
// step t hands to step t - 1, l = grad[t] + m, and a piece is m -> A m + M.  The
// states inside a span are formed again from the one kept before it, so that
// gradients of gates see 32-bit states and x, not h, is read.
#include "det_model.cuh"

#include <algorithm>

namespace det {
namespace {

constexpr int kSteps = 16;
constexpr int kWarps = 8;
constexpr int kSpan = kSteps * kWarps;      // of a CTA
constexpr int kMaxCluster = DET_RECURRENCE_SPAN / kSpan;
static_assert(kSpan == DET_RECURRENCE_KEEP, "states are kept at the CTAs' spans");

struct View {
  const void* p;
  long long sb, st;   // elements from one sequence and step to the next
};

// A lane's 32-bit word: two channels in 16 bits, one in 32.
template <typename T> struct Word {
  static constexpr int CH = 4 / sizeof(T);
};

// `n` channels from p; VEC: p is 4-byte aligned (n may still be 1 at the end of the channels).
template <typename T, bool VEC>
__device__ __forceinline__ unsigned load_word(const T* p, int n) {
  if constexpr (sizeof(T) == 4) {
    return *reinterpret_cast<const unsigned*>(p);
  } else {
    if (VEC && n == 2) return *reinterpret_cast<const unsigned*>(p);
    const unsigned short* q = reinterpret_cast<const unsigned short*>(p);
    unsigned w = q[0];
    if (n == 2) w |= (unsigned)q[1] << 16;
    return w;
  }
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_word(T* p, const float (&v)[Word<T>::CH], int n) {
  if constexpr (sizeof(T) == 4) {
    *p = v[0];
  } else {
    const T a = from_f32<T>(v[0]), b = from_f32<T>(v[1]);
    if (VEC && n == 2) {
      *reinterpret_cast<unsigned*>(p) =
          (unsigned)*reinterpret_cast<const unsigned short*>(&a) | (unsigned)*reinterpret_cast<const unsigned short*>(&b) << 16;
    } else {
      p[0] = a;
      if (n == 2) p[1] = b;
    }
  }
}
template <typename T>
__device__ __forceinline__ float unpack(unsigned w, int c) {
  if constexpr (sizeof(T) == 4) return __uint_as_float(w);
  else if constexpr (sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value)
    return __uint_as_float(c ? (w & 0xffff0000u) : (w << 16));
  else return __half2float(__ushort_as_half((unsigned short)(c ? (w >> 16) : w)));
}

// A gate in one 32-bit register.  Decay: itself.  Sigmoid: the smaller of s(z)
// and 1 - s(z), which are e / (1 + e) and 1 / (1 + e) with e = exp(-|z|), with
// the sign of z; both keep their relative accuracy, where 1 - s(z) formed from a
// rounded s(z) would not.  exp is the hardware's approximation for 16-bit
// inputs (relative error below 2^-20 up to |z| = 8) and expf for 32-bit ones.
template <typename T, int FORM>
__device__ __forceinline__ float gate_value(float z) {
  if (FORM == DET_GATE_DECAY) return z;
  const float e = sizeof(T) == 4 ? expf(-fabsf(z)) : exp_approx(-fabsf(z));
  return copysignf(__fdividef(e, 1.0f + e), z);
}
template <int FORM>
__device__ __forceinline__ void gate_parts(float v, float& a, float& rest) {
  if (FORM == DET_GATE_DECAY) {
    a = v;
    rest = 1.0f;
    return;
  }
  const float r = fabsf(v), q = 1.0f - r;
  const bool neg = __float_as_uint(v) >> 31;
  a = neg ? r : q;
  rest = neg ? q : r;
}
// The gate of a step past the end: a = 1, and with x = 0 nothing is added.
template <int FORM>
__device__ __forceinline__ float gate_of_no_step() { return FORM == DET_GATE_DECAY ? 1.0f : 0.0f; }

// The state h after a piece (A, H).  From 0 it is H whatever A is: A may have
// passed the range of 32 bits where h never did.
__device__ __forceinline__ float after(float h, float A, float H) { return h == 0.0f ? H : fmaf(A, h, H); }

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ unsigned cluster_size() {
  unsigned r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// v to the place of `local` in the shared memory of the cluster's CTA `rank`.
__device__ __forceinline__ void st_dsmem(float4* local, unsigned rank, float4 v) {
  unsigned r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(local)), "r"(rank));
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(r), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}

struct Shape {
  int time, channels;
  const int32_t* lengths;
};

// Where a thread works.
template <typename T, bool SHORT>
struct Place {
  int warp, lane, b, c, n;         // n: its channels, from c on
  unsigned rank, ranks;
  int len;                         // of the sequence
  __device__ __forceinline__ explicit Place(const Shape& s) {
    constexpr int CH = Word<T>::CH;
    warp = threadIdx.x >> 5;
    lane = threadIdx.x & 31;
    b = blockIdx.y;
    rank = SHORT ? 0 : cluster_rank();
    ranks = SHORT ? 1 : cluster_size();
    const int tile = SHORT ? blockIdx.x * kWarps + warp : blockIdx.x / ranks;
    c = (tile * 32 + lane) * CH;
    n = max(0, min(CH, s.channels - c));
    len = s.time;
    if (s.lengths) len = max(0, min(len, (int)s.lengths[b]));
  }
};

// The words of steps t0 .. t0 + 15 below len.
template <typename T, bool VEC>
__device__ __forceinline__ void load_piece(unsigned (&w)[kSteps], const View& v, int b, int c, int n, int t0, int len) {
  const T* p = static_cast<const T*>(v.p) + b * v.sb + t0 * v.st + c;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    w[i] = 0;
    if (n > 0 && t0 + i < len) w[i] = load_word<T, VEC>(p + i * v.st, n);
  }
}

// SHORT: at most 16 steps, a piece for each sequence and warp of channels, and
// nothing to exchange; the bits are those of the long form.
template <typename T, int FORM, bool VEC, bool SHORT>
__global__ void __launch_bounds__(32 * kWarps, 2)
recurrence_kernel(View x, View gate, Shape shape, const float* initial, T* out, float* final_out, float* states) {
  constexpr int CH = Word<T>::CH;
  __shared__ float4 s_warp[2][kWarps][32];
  __shared__ float4 s_cta[2][kMaxCluster][32];
  if (!SHORT) cluster_arrive();          // the others' shared memory is written only after they have started
  dep_wait();
  dep_launch();
  const Place<T, SHORT> me(shape);
  const int len = me.len, time = shape.time, channels = shape.channels;
  float carry[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c)
    carry[c] = (initial && c < me.n) ? initial[(long long)me.b * channels + me.c + c] : 0.0f;
  const int stride = SHORT ? kSteps : (int)me.ranks * kSpan;
  const int at = SHORT ? 0 : (int)me.rank * kSpan + me.warp * kSteps;
  const int kept = (time + kSpan - 1) / kSpan;
  unsigned rg[kSteps], rx[kSteps];
  load_piece<T, VEC>(rg, gate, me.b, me.c, me.n, at, len);
  load_piece<T, VEC>(rx, x, me.b, me.c, me.n, at, len);
  if (!SHORT) cluster_wait();
  int parity = 0;
  for (long long s0 = 0; s0 < time; s0 += stride, parity ^= 1) {
    const int t0 = (int)s0 + at;
    float v[kSteps][CH];                 // gates
    unsigned xs[kSteps];
    float A[CH], H[CH], h[CH];
    float4 before = make_float4(1.0f, 0.0f, 1.0f, 0.0f);   // (A, H) of the CTA's pieces before this warp's
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      A[c] = 1.0f;
      H[c] = 0.0f;
    }
    if (s0 < len) {
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        xs[i] = rx[i];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          v[i][c] = t0 + i < len ? gate_value<T, FORM>(unpack<T>(rg[i], c)) : gate_of_no_step<FORM>();
          float a, rest;
          gate_parts<FORM>(v[i][c], a, rest);
          H[c] = fmaf(a, H[c], rest * unpack<T>(xs[i], c));
          A[c] *= a;
        }
      }
      // the next piece is on its way while the states are exchanged
      load_piece<T, VEC>(rg, gate, me.b, me.c, me.n, (int)min(s0 + stride, (long long)len) + at, len);
      load_piece<T, VEC>(rx, x, me.b, me.c, me.n, (int)min(s0 + stride, (long long)len) + at, len);
    }
    if (SHORT || s0 >= len) {
#pragma unroll
      for (int c = 0; c < CH; ++c) h[c] = carry[c];
    } else {
      float4 mine = make_float4(A[0], H[0], 1.0f, 0.0f);
      if (CH == 2) mine.z = A[CH - 1], mine.w = H[CH - 1];
      s_warp[parity][me.warp][me.lane] = mine;
      __syncthreads();
      float4 all = before;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w == me.warp) before = all;
        const float4 q = s_warp[parity][w][me.lane];
        all.y = after(all.y, q.x, q.y);
        all.x *= q.x;
        all.w = after(all.w, q.z, q.w);
        all.z *= q.z;
      }
      if (me.ranks > 1) {
        if (me.warp < (int)me.ranks) st_dsmem(&s_cta[parity][me.rank][me.lane], me.warp, all);
        cluster_arrive();
        cluster_wait();
        float here[2] = {carry[0], carry[CH - 1]}, next[2] = {carry[0], carry[CH - 1]};
        for (unsigned r = 0; r < me.ranks; ++r) {
          if (r == me.rank) here[0] = next[0], here[1] = next[1];
          const float4 q = s_cta[parity][r][me.lane];
          next[0] = after(next[0], q.x, q.y);
          next[1] = after(next[1], q.z, q.w);
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          h[c] = here[c];
          carry[c] = next[c];
        }
      } else {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          h[c] = carry[c];
          carry[c] = c ? after(carry[c], all.z, all.w) : after(carry[c], all.x, all.y);
        }
      }
    }
    if (states && (SHORT || me.warp == 0) && t0 < time) {
#pragma unroll
      for (int c = 0; c < CH; ++c)
        if (c < me.n) states[((long long)me.b * kept + t0 / kSpan) * channels + me.c + c] = h[c];
    }
    T* o = out + ((long long)me.b * time + t0) * channels + me.c;
    if (s0 < len) {
      if (!SHORT && me.warp > 0) {
        h[0] = after(h[0], before.x, before.y);
        if (CH == 2) h[CH - 1] = after(h[CH - 1], before.z, before.w);
      }
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        float r[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          float a, rest;
          gate_parts<FORM>(v[i][c], a, rest);
          h[c] = fmaf(a, h[c], rest * unpack<T>(xs[i], c));
          r[c] = t0 + i < len ? h[c] : 0.0f;
        }
        if (me.n > 0 && t0 + i < time) store_word<T, VEC>(o + (long long)i * channels, r, me.n);
      }
      // the state at the end is that of the last step (steps past it have kept it); the
      // initial state has been read everywhere by now, so it may lie in the same place
      if (final_out && t0 < len && len <= t0 + kSteps) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
          if (c < me.n) final_out[(long long)me.b * channels + me.c + c] = h[c];
      }
    } else {
      const float zero[CH] = {};
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
        if (me.n > 0 && t0 + i < time) store_word<T, VEC>(o + (long long)i * channels, zero, me.n);
    }
  }
  if (final_out && len == 0 && (SHORT || (me.rank == 0 && me.warp == 0))) {
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (c < me.n) final_out[(long long)me.b * channels + me.c + c] = carry[c];
  }
}

template <typename T, int FORM, bool VEC, bool SHORT>
__global__ void __launch_bounds__(32 * kWarps, 2)
recurrence_grad_kernel(View grad, View x, View gate, Shape shape, const float* states, const float* grad_final,
                       T* grad_x, T* grad_gate, float* grad_initial) {
  constexpr int CH = Word<T>::CH;
  __shared__ float4 s_warp[kWarps][32];          // (A, H) of both channels
  __shared__ float2 s_back[kWarps][32];          // M of both
  __shared__ float4 s_cta[2][kMaxCluster][32];   // (A, M) of both
  if (!SHORT) cluster_arrive();
  dep_wait();
  dep_launch();
  const Place<T, SHORT> me(shape);
  const int len = me.len, time = shape.time, channels = shape.channels;
  float carry[CH], first[CH];   // first: what the sequence's first step hands back
#pragma unroll
  for (int c = 0; c < CH; ++c)
    first[c] = carry[c] = (grad_final && c < me.n) ? grad_final[(long long)me.b * channels + me.c + c] : 0.0f;
  const int stride = SHORT ? kSteps : (int)me.ranks * kSpan;
  const int at = SHORT ? 0 : (int)me.rank * kSpan + me.warp * kSteps;
  const int kept = (time + kSpan - 1) / kSpan;
  if (!SHORT) cluster_wait();
  int parity = 0;
  for (long long s0 = time > 0 ? (long long)((time - 1) / stride) * stride : -1; s0 >= 0; s0 -= stride, parity ^= 1) {
    const int t0 = (int)s0 + at;
    T* ox = grad_x + ((long long)me.b * time + t0) * channels + me.c;
    T* og = grad_gate + ((long long)me.b * time + t0) * channels + me.c;
    if (s0 >= len) {
      const float zero[CH] = {};
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
        if (me.n > 0 && t0 + i < time) {
          store_word<T, VEC>(ox + (long long)i * channels, zero, me.n);
          store_word<T, VEC>(og + (long long)i * channels, zero, me.n);
        }
      continue;
    }
    unsigned rg[kSteps], xs[kSteps], gs[kSteps];
    load_piece<T, VEC>(rg, gate, me.b, me.c, me.n, t0, len);
    load_piece<T, VEC>(xs, x, me.b, me.c, me.n, t0, len);
    if (grad.p) {
      load_piece<T, VEC>(gs, grad, me.b, me.c, me.n, t0, len);
    } else {
#pragma unroll
      for (int i = 0; i < kSteps; ++i) gs[i] = 0;
    }
    float h[CH], m[CH], v[kSteps][CH], A[CH], H[CH], M[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      h[c] = (c < me.n && t0 < len) ? states[((long long)me.b * kept + t0 / kSpan) * channels + me.c + c] : 0.0f;
      m[c] = carry[c];
      A[c] = 1.0f;
      H[c] = M[c] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        v[i][c] = t0 + i < len ? gate_value<T, FORM>(unpack<T>(rg[i], c)) : gate_of_no_step<FORM>();
        float a, rest;
        gate_parts<FORM>(v[i][c], a, rest);
        H[c] = fmaf(a, H[c], rest * unpack<T>(xs[i], c));
        A[c] *= a;
        M[c] = fmaf(A[c], unpack<T>(gs[i], c), M[c]);
      }
    }
    if (!SHORT) {
      float4 mine = make_float4(A[0], H[0], A[CH - 1], H[CH - 1]);
      __syncthreads();                     // the piece before has been read
      s_warp[me.warp][me.lane] = mine;
      s_back[me.warp][me.lane] = make_float2(M[0], M[CH - 1]);
      __syncthreads();
      float4 all = make_float4(1.0f, 0.0f, 1.0f, 0.0f);    // (A, M) of the pieces behind, in the order back
      float4 behind = all;
#pragma unroll
      for (int w = kWarps - 1; w >= 0; --w) {
        if (w == me.warp) behind = all;
        const float4 q = s_warp[w][me.lane];
        const float2 b = s_back[w][me.lane];
        all.y = after(all.y, q.x, b.x);
        all.x *= q.x;
        all.w = after(all.w, q.z, b.y);
        all.z *= q.z;
      }
      for (int w = 0; w < me.warp; ++w) {
        const float4 q = s_warp[w][me.lane];
        h[0] = after(h[0], q.x, q.y);
        if (CH == 2) h[CH - 1] = after(h[CH - 1], q.z, q.w);
      }
      if (me.ranks > 1) {
        if (me.warp < (int)me.ranks) st_dsmem(&s_cta[parity][me.rank][me.lane], me.warp, all);
        cluster_arrive();
        cluster_wait();
        float here[2] = {carry[0], carry[CH - 1]}, next[2] = {carry[0], carry[CH - 1]};
        for (int r = (int)me.ranks - 1; r >= 0; --r) {
          if (r == (int)me.rank) here[0] = next[0], here[1] = next[1];
          const float4 q = s_cta[parity][r][me.lane];
          next[0] = after(next[0], q.x, q.y);
          next[1] = after(next[1], q.z, q.w);
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          m[c] = here[c];
          carry[c] = next[c];
        }
      } else {
#pragma unroll
        for (int c = 0; c < CH; ++c) carry[c] = c ? after(carry[c], all.z, all.w) : after(carry[c], all.x, all.y);
      }
      m[0] = after(m[0], behind.x, behind.y);
      if (CH == 2) m[CH - 1] = after(m[CH - 1], behind.z, behind.w);
    }
    float hp[kSteps][CH];                  // the states before the steps
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        hp[i][c] = h[c];
        float a, rest;
        gate_parts<FORM>(v[i][c], a, rest);
        h[c] = fmaf(a, h[c], rest * unpack<T>(xs[i], c));
      }
#pragma unroll
    for (int i = kSteps - 1; i >= 0; --i) {
      float dx[CH], dg[CH];
      const bool inside = t0 + i < len;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        float a, rest;
        gate_parts<FORM>(v[i][c], a, rest);
        const float l = unpack<T>(gs[i], c) + m[c];
        m[c] = inside ? a * l : m[c];
        if (FORM == DET_GATE_DECAY) {
          dx[c] = inside ? l : 0.0f;
          dg[c] = inside ? l * hp[i][c] : 0.0f;
        } else {
          dx[c] = inside ? l * rest : 0.0f;
          dg[c] = inside ? l * rest * (a * (hp[i][c] - unpack<T>(xs[i], c))) : 0.0f;
        }
      }
      if (me.n > 0 && t0 + i < time) {
        store_word<T, VEC>(ox + (long long)i * channels, dx, me.n);
        store_word<T, VEC>(og + (long long)i * channels, dg, me.n);
      }
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) first[c] = m[c];
  }
  if (grad_initial && (SHORT || (me.rank == 0 && me.warp == 0))) {
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (c < me.n) grad_initial[(long long)me.b * channels + me.c + c] = first[c];
  }
}

// A launch over channel tiles and sequences: up to 16 steps without clusters,
// else with as many CTAs a cluster as a sequence fills, at most 8.
template <typename T, typename... KArgs, typename... Args>
int launch_recurrence(const char* name, void (*short_kernel)(KArgs...), void (*kernel)(KArgs...), int batch, int time,
                      int channels, cudaStream_t s, Args... args) {
  const int words = (channels + Word<T>::CH - 1) / Word<T>::CH;
  const bool brief = time <= kSteps;
  int ranks = 1;
  while (ranks < kMaxCluster && ranks * kSpan < time) ranks *= 2;
  const int tiles = (words + 31) / 32;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = brief ? dim3((unsigned)((tiles + kWarps - 1) / kWarps), (unsigned)batch)
                      : dim3((unsigned)tiles * ranks, (unsigned)batch);
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ranks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = brief ? 1 : 2;
  launch_begin(name, s);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, brief ? short_kernel : kernel, args...);
  launch_end(s);
  return e == cudaSuccess ? DET_OK : cuda_fail(e, name);
}

template <typename T, int FORM, bool VEC>
int forward(const View& x, const View& gate, const Shape& shape, int batch, const float* initial, void* out,
            float* final_out, float* states, cudaStream_t s) {
  return launch_recurrence<T>("det_linear_recurrence", recurrence_kernel<T, FORM, VEC, true>,
                              recurrence_kernel<T, FORM, VEC, false>, batch, shape.time, shape.channels, s, x, gate,
                              shape, initial, static_cast<T*>(out), final_out, states);
}
template <typename T, int FORM, bool VEC>
int backward(const View& grad, const View& x, const View& gate, const Shape& shape, int batch, const float* states,
             const float* grad_final, void* grad_x, void* grad_gate, float* grad_initial, cudaStream_t s) {
  return launch_recurrence<T>("det_linear_recurrence_backward", recurrence_grad_kernel<T, FORM, VEC, true>,
                              recurrence_grad_kernel<T, FORM, VEC, false>, batch, shape.time, shape.channels, s, grad,
                              x, gate, shape, states, grad_final, static_cast<T*>(grad_x), static_cast<T*>(grad_gate),
                              grad_initial);
}

int check_shape(int dtype, int form, int64_t batch, int64_t time, int64_t channels) {
  if (!valid_model_dtype(dtype)) return DET_ERR_DTYPE;
  if (form != DET_GATE_DECAY && form != DET_GATE_SIGMOID) return DET_ERR_INVALID_ARG;
  if (batch < 0 || time < 0 || channels < 0) return DET_ERR_INVALID_ARG;
  constexpr int64_t most = (1LL << 31) - (1LL << 16);
  if (batch > 65535 || time >= most || channels >= most) return DET_ERR_TOO_LARGE;
  return DET_OK;
}
bool misaligned(const void* p, int dtype) { return reinterpret_cast<uintptr_t>(p) % model_elem_size(dtype) != 0; }
bool misaligned_floats(const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 != 0; }

}  // namespace
}  // namespace det

using namespace det;

// Two channels a lane go as one word where every row of every operand starts on one.
#define DET_RECURRENCE_PICK(fn, ...)                                                                                  \
  do {                                                                                                               \
    if (dtype == DET_F32)                                                                                            \
      return form == DET_GATE_DECAY ? fn<float, DET_GATE_DECAY, true>(__VA_ARGS__)                                   \
                                    : fn<float, DET_GATE_SIGMOID, true>(__VA_ARGS__);                                \
    if (dtype == DET_BF16)                                                                                           \
      return form == DET_GATE_DECAY ? (words ? fn<__nv_bfloat16, DET_GATE_DECAY, true>(__VA_ARGS__)                  \
                                             : fn<__nv_bfloat16, DET_GATE_DECAY, false>(__VA_ARGS__))                \
                                    : (words ? fn<__nv_bfloat16, DET_GATE_SIGMOID, true>(__VA_ARGS__)                \
                                             : fn<__nv_bfloat16, DET_GATE_SIGMOID, false>(__VA_ARGS__));             \
    return form == DET_GATE_DECAY                                                                                    \
               ? (words ? fn<__half, DET_GATE_DECAY, true>(__VA_ARGS__) : fn<__half, DET_GATE_DECAY, false>(__VA_ARGS__)) \
               : (words ? fn<__half, DET_GATE_SIGMOID, true>(__VA_ARGS__)                                            \
                        : fn<__half, DET_GATE_SIGMOID, false>(__VA_ARGS__));                                         \
  } while (0)

extern "C" int det_linear_recurrence(const void* x, int64_t x_stride_b, int64_t x_stride_t, const void* gate,
                                     int64_t gate_stride_b, int64_t gate_stride_t, int dtype, int form, int64_t batch,
                                     int64_t time, int64_t channels, const float* initial, const int32_t* lengths,
                                     void* out, float* final_out, float* states_out, void* stream) {
  if (const int rc = check_shape(dtype, form, batch, time, channels)) return rc;
  if (batch == 0 || channels == 0) return DET_OK;
  if (time > 0 && (!x || !gate || !out)) return DET_ERR_INVALID_ARG;
  if (x_stride_b < 0 || x_stride_t < 0 || gate_stride_b < 0 || gate_stride_t < 0) return DET_ERR_INVALID_ARG;
  if (misaligned(x, dtype) || misaligned(gate, dtype) || misaligned(out, dtype) || misaligned_floats(initial) ||
      misaligned_floats(lengths) || misaligned_floats(final_out) || misaligned_floats(states_out))
    return DET_ERR_INVALID_ARG;
  const bool words = ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(gate) |
                       reinterpret_cast<uintptr_t>(out)) % 4 == 0) &&
                     ((x_stride_b | x_stride_t | gate_stride_b | gate_stride_t | channels) % 2 == 0);
  const View vx = {x, x_stride_b, x_stride_t}, vg = {gate, gate_stride_b, gate_stride_t};
  const Shape shape = {(int)time, (int)channels, lengths};
  const cudaStream_t s = as_stream(stream);
  DET_RECURRENCE_PICK(forward, vx, vg, shape, (int)batch, initial, out, final_out, states_out, s);
}

extern "C" int det_linear_recurrence_backward(const void* grad, int64_t grad_stride_b, int64_t grad_stride_t,
                                              const void* x, int64_t x_stride_b, int64_t x_stride_t, const void* gate,
                                              int64_t gate_stride_b, int64_t gate_stride_t, int dtype, int form,
                                              int64_t batch, int64_t time, int64_t channels, const float* states,
                                              const float* grad_final, const int32_t* lengths, void* grad_x,
                                              void* grad_gate, float* grad_initial, void* stream) {
  if (const int rc = check_shape(dtype, form, batch, time, channels)) return rc;
  if (batch == 0 || channels == 0) return DET_OK;
  if (time > 0 && (!x || !gate || !states || !grad_x || !grad_gate)) return DET_ERR_INVALID_ARG;
  if (x_stride_b < 0 || x_stride_t < 0 || gate_stride_b < 0 || gate_stride_t < 0 || grad_stride_b < 0 || grad_stride_t < 0)
    return DET_ERR_INVALID_ARG;
  if (misaligned(grad, dtype) || misaligned(x, dtype) || misaligned(gate, dtype) || misaligned(grad_x, dtype) ||
      misaligned(grad_gate, dtype) || misaligned_floats(states) || misaligned_floats(grad_final) ||
      misaligned_floats(lengths) || misaligned_floats(grad_initial))
    return DET_ERR_INVALID_ARG;
  const bool words =
      ((reinterpret_cast<uintptr_t>(grad) | reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(gate) |
        reinterpret_cast<uintptr_t>(grad_x) | reinterpret_cast<uintptr_t>(grad_gate)) % 4 == 0) &&
      ((grad_stride_b | grad_stride_t | x_stride_b | x_stride_t | gate_stride_b | gate_stride_t | channels) % 2 == 0);
  const View vd = {grad, grad_stride_b, grad_stride_t}, vx = {x, x_stride_b, x_stride_t},
             vg = {gate, gate_stride_b, gate_stride_t};
  const Shape shape = {(int)time, (int)channels, lengths};
  const cudaStream_t s = as_stream(stream);
  DET_RECURRENCE_PICK(backward, vd, vx, vg, shape, (int)batch, states, grad_final, grad_x, grad_gate, grad_initial, s);
}
