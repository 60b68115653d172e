// det_linear_recurrence and its gradient: h = a[t] h + u[t] along time, for
// every sequence and channel.
//
// A step is the map h -> a h + u; a run of steps is a map of the same kind,
// h -> A h + H with A the product of its decays and H its result from 0.  Time
// is cut into pieces (a warp), the pieces of a CTA's 8 warps and those of a
// cluster's 8 CTAs.  A warp reads its piece of 32 words of channels into
// registers once, forms (A, H), the CTA's warps and then the cluster's CTAs
// exchange these through (distributed) shared memory, and each warp runs
// through its piece again, in registers, from the state it now knows.  A
// cluster goes through its sequence from one such span to the next and carries
// the state in registers; the next span's words are on their way meanwhile.  So
// every input is read once and every output written once, and nothing waits on
// memory that another CTA writes.  Pieces are joined in the order of time, always
// from the same borders, so the bits of a step are a function of the steps before
// it.
//
// The gradient runs the same way from the end.  With m = a[t] l the value that
// step t hands to step t - 1, l = grad[t] + m, and a piece is m -> A m + M.  The
// states inside a span are formed again from those kept before every 128th step,
// so that the gates' gradients see 32-bit states and x, not h, is read.
//
// What bounds it: bytes, once an element costs few enough instructions (at the
// copy's rate an SM's schedulers have 33 slots for each element forward and
// twice that backward).  So two 16-bit channels of a word are worked on by packed
// 32-bit instructions, whole pieces have no conditions, and gates are computed
// once.
#include "det_model.cuh"

#include <algorithm>
#include <initializer_list>

namespace det {
namespace {

constexpr int kWarps = 8;                   // pieces of a CTA
constexpr int kMaxCluster = 8;
constexpr int kStepsForward = 16;           // of a piece
constexpr int kStepsBackward = 8;           // three inputs, and three values a step between the passes: registers
static_assert(kStepsForward * kWarps * kMaxCluster == DET_RECURRENCE_SPAN, "the documented span");
static_assert(kStepsForward * kWarps == DET_RECURRENCE_KEEP, "states are kept at the forward CTAs' spans");
static_assert(2 * kStepsBackward * kWarps == DET_RECURRENCE_KEEP, "backward every second CTA begins with a kept state");

struct View {
  const void* p;
  long long sb, st;   // elements from one sequence and step to the next
};
struct Shape {
  int time, channels;
  const int32_t* lengths;
  int log2_ranks;     // CTAs of a cluster
  int near;           // a span of a cluster lies within 2^31 bytes in every operand
};

// ---------------------------------------------------------------------------
// A lane's values: two 16-bit channels of a word as a packed pair, one of 32 bits.

using Two = unsigned long long;
__device__ __forceinline__ float add(float a, float b) { return __fadd_rn(a, b); }
__device__ __forceinline__ float mul(float a, float b) { return __fmul_rn(a, b); }
__device__ __forceinline__ float fma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ Two add(Two a, Two b) { return add_f32x2(a, b); }
__device__ __forceinline__ Two mul(Two a, Two b) { return mul_f32x2(a, b); }
__device__ __forceinline__ Two fma(Two a, Two b, Two c) { return fma_f32x2(a, b, c); }
__device__ __forceinline__ void both(float& v, float x) { v = x; }
__device__ __forceinline__ void both(Two& v, float x) { v = pack_f32x2(x, x); }
__device__ __forceinline__ float minus(float a, float b) { return __fsub_rn(a, b); }
__device__ __forceinline__ Two minus(Two a, Two b) { return fma_f32x2(b, pack_f32x2(-1.0f, -1.0f), a); }

template <typename T> struct Lane {
  static constexpr int CH = 2;
  using V = Two;
};
template <> struct Lane<float> {
  static constexpr int CH = 1;
  using V = float;
};
template <typename T> using LaneV = typename Lane<T>::V;

template <typename T>
__device__ __forceinline__ LaneV<T> unpack(unsigned w) {
  if constexpr (sizeof(T) == 4) {
    return __uint_as_float(w);
  } else {
    float a, b;
    unpack_two(w, a, b, T());
    return pack_f32x2(a, b);
  }
}
template <typename T>
__device__ __forceinline__ unsigned pack(LaneV<T> v) {
  if constexpr (sizeof(T) == 4) {
    return __float_as_uint(v);
  } else {
    const float2 f = unpack_f32x2(v);
    return pack_two<T>(f.x, f.y);
  }
}

// `n` channels from p; VEC: p is 4-byte aligned.
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
__device__ __forceinline__ void store_word(T* p, unsigned w, int n) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<unsigned*>(p) = w;
  } else {
    if (VEC && n == 2) {
      *reinterpret_cast<unsigned*>(p) = w;
    } else {
      unsigned short* q = reinterpret_cast<unsigned short*>(p);
      q[0] = (unsigned short)w;
      if (n == 2) q[1] = (unsigned short)(w >> 16);
    }
  }
}

// 32-bit state of a lane's channels in [.., channels] floats at p.
template <int CH, typename V>
__device__ __forceinline__ void load_state(V& v, const float* p, int n) {
  if constexpr (CH == 1) v = n > 0 ? p[0] : 0.0f;
  else v = pack_f32x2(n > 0 ? p[0] : 0.0f, n > 1 ? p[1] : 0.0f);
}
template <int CH, typename V>
__device__ __forceinline__ void store_state(float* p, V v, int n) {
  if constexpr (CH == 1) {
    if (n > 0) p[0] = v;
  } else {
    const float2 f = unpack_f32x2(v);
    if (n > 0) p[0] = f.x;
    if (n > 1) p[1] = f.y;
  }
}

// ---------------------------------------------------------------------------
// Gates: a word of them to the decays a and what is left, 1 - a.
//
// Sigmoid: with e = exp(-z), a = 1 / (1 + e) and 1 - a = e a, which keeps the
// relative accuracy of both where a difference from 1 would lose it.  In 16 bits e
// and the reciprocal are the hardware's approximations (a and 1 - a off by at most
// 8 + |z| units of 2^-24); z is held at -87 and more, so that e stays finite, and
// the a that belongs to -87 is taken off (`floor`, 2^-125): a gate of -inf closes
// for good.  In 32 bits expf, and the smaller one of the two by a division.
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ unsigned at_least(unsigned w, float low, __nv_bfloat16) {
  const __nv_bfloat162 l = __floats2bfloat162_rn(low, low);
  const __nv_bfloat162 m = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&w), l);
  return *reinterpret_cast<const unsigned*>(&m);
}
__device__ __forceinline__ unsigned at_least(unsigned w, float low, __half) {
  const __half2 l = __floats2half2_rn(low, low);
  const __half2 m = __hmax2_nan(*reinterpret_cast<const __half2*>(&w), l);
  return *reinterpret_cast<const unsigned*>(&m);
}
constexpr float kLowestGate = -87.0f;
template <typename T, int FORM>
struct Gates {
  using V = LaneV<T>;
  V floor;
  __device__ __forceinline__ Gates() {
    both(floor, 0.0f);
    if constexpr (FORM == DET_GATE_SIGMOID && sizeof(T) == 2) {
      const float e = exp2_approx(__fmul_rn(kLowestGate, -kLog2e));
      const float a = -rcp_approx(__fadd_rn(e, 1.0f));
      floor = pack_f32x2(a, a);
    }
  }
  __device__ __forceinline__ void operator()(unsigned w, V& a, V& rest) const {
    if constexpr (FORM == DET_GATE_DECAY) {
      a = unpack<T>(w);
      both(rest, 1.0f);
    } else if constexpr (sizeof(T) == 2) {
      const Two t = mul(unpack<T>(at_least(w, kLowestGate, T())), pack_f32x2(-kLog2e, -kLog2e));
      const float2 f = unpack_f32x2(t);
      const Two e = pack_f32x2(exp2_approx(f.x), exp2_approx(f.y));
      const float2 d = unpack_f32x2(add(e, pack_f32x2(1.0f, 1.0f)));
      a = pack_f32x2(rcp_approx(d.x), rcp_approx(d.y));
      rest = mul(e, a);
      a = add(a, floor);
    } else {
      const float z = __uint_as_float(w);
      const float e = expf(-fabsf(z));
      const float less = __fdividef(e, 1.0f + e), more = 1.0f - less;
      a = z < 0.0f ? less : more;
      rest = z < 0.0f ? more : less;
    }
  }
  // rest * x: what a step adds
  __device__ __forceinline__ V input(V rest, V x) const { return FORM == DET_GATE_DECAY ? x : mul(rest, x); }
};

// The state h after a piece (A, H).  Decays above 1 may take A out of the range of
// 32 bits where the states stay in it: from 0 the state is H whatever A is.
template <int FORM>
__device__ __forceinline__ float after(float h, float A, float H) {
  return FORM == DET_GATE_DECAY && h == 0.0f ? H : fmaf(A, h, H);
}
template <int FORM>
__device__ __forceinline__ Two after(Two h, Two A, Two H) {
  if constexpr (FORM == DET_GATE_SIGMOID) {
    return fma(A, h, H);
  } else {
    const float2 g = unpack_f32x2(h), a = unpack_f32x2(A), b = unpack_f32x2(H);
    return pack_f32x2(after<FORM>(g.x, a.x, b.x), after<FORM>(g.y, a.y, b.y));
  }
}

// ---------------------------------------------------------------------------
// Clusters

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// A piece's map: (A, H), or back (A, M).
template <typename V> struct alignas(2 * sizeof(V)) Map {
  V A, H;
};
// v to the place of `local` in the shared memory of the cluster's CTA `rank`, counted
// there on the barrier at the place of `bar`.  (A barrier of the whole cluster
// would first wait for the stores of outputs in flight: 1 x 65,536 x 2,048 in bf16
// took 239 us with it, 202 without.)
__device__ __forceinline__ unsigned remote(const void* local, int rank) {
  unsigned r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(local)), "r"(rank));
  return r;
}
__device__ __forceinline__ void put(Map<Two>* local, unsigned long long* bar, int rank, const Map<Two>& v) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b64 [%0], {%1, %2}, [%3];" ::"r"(
                   remote(local, rank)),
               "l"(v.A), "l"(v.H), "r"(remote(bar, rank))
               : "memory");
}
__device__ __forceinline__ void put(Map<float>* local, unsigned long long* bar, int rank, const Map<float>& v) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::"r"(
                   remote(local, rank)),
               "r"(__float_as_uint(v.A)), "r"(__float_as_uint(v.H)), "r"(remote(bar, rank))
               : "memory");
}
// Waits for a phase of messages, for at most kWaitNs.
__device__ __forceinline__ bool messages_in(unsigned long long* bar, unsigned phase) {
  unsigned long long t0 = 0;
  for (unsigned polls = 0;; ++polls) {
    unsigned done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(phase)
        : "memory");
    if (done) return true;
    if (polls == 0) t0 = globaltimer();
    else if ((polls & 255u) == 0 && globaltimer() - t0 > kWaitNs) return false;
  }
}

// Where a thread works.
template <typename T, bool SHORT>
struct Place {
  int warp, lane, b, c, n;         // n: its channels, from c on
  int rank, ranks;
  int len;                         // of the sequence
  bool whole;                      // every lane of the warp has all its channels, and 32-bit offsets will do
  __device__ __forceinline__ explicit Place(const Shape& s) {
    constexpr int CH = Lane<T>::CH;
    warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    lane = threadIdx.x & 31;
    b = blockIdx.y;
    ranks = SHORT ? 1 : 1 << s.log2_ranks;
    rank = SHORT ? 0 : blockIdx.x & (ranks - 1);             // clusters lie along x
    const int tile = SHORT ? blockIdx.x * kWarps + warp : blockIdx.x >> s.log2_ranks;
    c = (tile * 32 + lane) * CH;
    n = max(0, min(CH, s.channels - c));
    whole = s.near && (tile + 1) * 32 * CH <= s.channels;
    len = s.time;
    if (s.lengths) len = max(0, min(len, (int)s.lengths[b]));
  }
};

// The words of steps s0 + at .. s0 + at + STEPS - 1 below len.  A full piece is read
// at 32-bit offsets from one base, the same for all threads: one addition a word.
template <typename T, bool VEC, int STEPS>
__device__ __forceinline__ void load_piece(unsigned (&w)[STEPS], const View& v, int b, int c, int n, int s0, int at,
                                           int len, bool full) {
  const T* base = static_cast<const T*>(v.p) + (b * v.sb + s0 * v.st);
  if (full) {
    const unsigned step = (unsigned)v.st * (unsigned)sizeof(T);
    unsigned o = (unsigned)at * step + (unsigned)c * (unsigned)sizeof(T);
#pragma unroll
    for (int i = 0; i < STEPS; ++i, o += step)
      w[i] = load_word<T, VEC>(reinterpret_cast<const T*>(reinterpret_cast<const char*>(base) + o), Lane<T>::CH);
  } else {
    const T* p = base + at * v.st + c;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      w[i] = 0;
      if (n > 0 && s0 + at + i < len) w[i] = load_word<T, VEC>(p + i * v.st, n);
    }
  }
}

// ---------------------------------------------------------------------------

// The decays and additions of a piece and its map.  A step past the end is
// (1, 0).
template <typename T, int FORM, bool FULL>
__device__ __forceinline__ void forward_maps(const Gates<T, FORM>& gates, const unsigned (&rg)[kStepsForward],
                                             const unsigned (&rx)[kStepsForward], LaneV<T> (&a)[kStepsForward],
                                             LaneV<T> (&u)[kStepsForward], Map<LaneV<T>>& map, int steps) {
#pragma unroll
  for (int i = 0; i < kStepsForward; ++i) {
    LaneV<T> rest;
    gates(rg[i], a[i], rest);
    u[i] = gates.input(rest, unpack<T>(rx[i]));
    if (!FULL && i >= steps) {
      both(a[i], 1.0f);
      both(u[i], 0.0f);
    }
    map.H = i ? fma(a[i], map.H, u[i]) : u[i];
    map.A = i ? mul(map.A, a[i]) : a[i];
  }
}

// SHORT: at most 16 steps, a piece for each sequence and warp of channels, and
// nothing to exchange; the bits are those of the long form.
template <typename T, int FORM, bool VEC, bool SHORT>
__global__ void __launch_bounds__(32 * kWarps, 2)
recurrence_kernel(View x, View gate, Shape shape, const float* initial, T* out, float* final_out, float* states) {
  using V = LaneV<T>;
  constexpr int CH = Lane<T>::CH, STEPS = kStepsForward, SPAN = STEPS * kWarps;
  __shared__ Map<V> s_warp[2][kWarps][32];
  __shared__ Map<V> s_cta[2][kMaxCluster][32];
  __shared__ unsigned long long s_bar[2];
  if (!SHORT) {
    if (threadIdx.x < 2) mbar_init(&s_bar[threadIdx.x], 1);
    cluster_arrive();                    // the others' shared memory is written only after they have come here
  }
  dep_wait();
  dep_launch();
  const Gates<T, FORM> gates;
  const Place<T, SHORT> me(shape);
  const int len = me.len, time = shape.time, channels = shape.channels;
  const long long row = (long long)me.b * channels + me.c;   // of the sequence's states
  V carry;
  load_state<CH>(carry, initial + row, initial ? me.n : 0);
  const int stride = SHORT ? STEPS : me.ranks * SPAN;
  const int at = SHORT ? 0 : me.rank * SPAN + me.warp * STEPS;
  const int kept = (time + SPAN - 1) / SPAN;
  unsigned rg[STEPS], rx[STEPS];
  bool full = me.whole && at + STEPS <= len;
  load_piece<T, VEC>(rg, gate, me.b, me.c, me.n, 0, at, len, full);
  load_piece<T, VEC>(rx, x, me.b, me.c, me.n, 0, at, len, full);
  if (!SHORT) cluster_wait();
  int round = 0;
  bool lost = false;                     // a wait gave up: results are NaN from there on
  long long s0 = 0;
  for (; s0 < len; s0 += stride, ++round) {
    const int parity = round & 1;
    const int t0 = (int)s0 + at;
    V a[STEPS], u[STEPS];
    Map<V> map;
    const bool all_in = full;
    if (all_in) forward_maps<T, FORM, true>(gates, rg, rx, a, u, map, STEPS);
    else forward_maps<T, FORM, false>(gates, rg, rx, a, u, map, len - t0);
    // the next piece is on its way while the states are exchanged
    if (!SHORT && s0 + stride < len) {
      full = me.whole && s0 + stride + at + STEPS <= len;
      load_piece<T, VEC>(rg, gate, me.b, me.c, me.n, (int)s0 + stride, at, len, full);
      load_piece<T, VEC>(rx, x, me.b, me.c, me.n, (int)s0 + stride, at, len, full);
    }
    V h = carry;
    if (!SHORT) {
      s_warp[parity][me.warp][me.lane] = map;
      __syncthreads();
      if (me.ranks > 1) {
        if (me.warp < me.ranks) {        // warp r tells CTA r
          map = s_warp[parity][0][me.lane];
#pragma unroll
          for (int w = 1; w < kWarps; ++w) {
            const Map<V> q = s_warp[parity][w][me.lane];
            map.H = after<FORM>(map.H, q.A, q.H);
            map.A = mul(map.A, q.A);
          }
          if (!lost) put(&s_cta[parity][me.rank][me.lane], &s_bar[parity], me.warp, map);
        }
        if (threadIdx.x == 0 && !lost) mbar_arrive_expect_tx(&s_bar[parity], me.ranks * 32 * (unsigned)sizeof(Map<V>));
        lost = lost || !messages_in(&s_bar[parity], round >> 1 & 1);
        if (lost) both(h, __int_as_float(0x7fffffff));
        int r = 0;
        for (; r < me.rank; ++r) {
          const Map<V> q = s_cta[parity][r][me.lane];
          h = after<FORM>(h, q.A, q.H);
        }
        carry = h;
        for (; r < me.ranks; ++r) {
          const Map<V> q = s_cta[parity][r][me.lane];
          carry = after<FORM>(carry, q.A, q.H);
        }
      }
      // (a CTA by itself makes one round and needs no carry)
      if (states && me.warp == 0 && t0 < time)
        store_state<CH>(states + ((long long)me.b * kept + t0 / SPAN) * channels + me.c, h, me.n);
      for (int w = 0; w < me.warp; ++w) {
        const Map<V> q = s_warp[parity][w][me.lane];
        h = after<FORM>(h, q.A, q.H);
      }
    } else if (states) {
      store_state<CH>(states + row, h, me.n);
    }
    T* base = out + ((long long)me.b * time + s0) * channels;
    const unsigned step = (unsigned)channels * (unsigned)sizeof(T);
    if (all_in) {
      unsigned o = (unsigned)at * step + (unsigned)me.c * (unsigned)sizeof(T);
#pragma unroll
      for (int i = 0; i < STEPS; ++i, o += step) {
        h = fma(a[i], h, u[i]);
        store_word<T, VEC>(reinterpret_cast<T*>(reinterpret_cast<char*>(base) + o), pack<T>(h), CH);
      }
    } else {
      T* o = base + (long long)at * channels + me.c;
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        h = fma(a[i], h, u[i]);
        if (me.n > 0 && t0 + i < time) store_word<T, VEC>(o + (long long)i * channels, t0 + i < len ? pack<T>(h) : 0u, me.n);
      }
    }
    // the state at the end is that of the last step (steps past it have kept it); the
    // initial state has been read everywhere by now, so it may lie in the same place
    if (final_out && t0 < len && len <= t0 + STEPS) store_state<CH>(final_out + row, h, me.n);
    if (SHORT) carry = h;
  }
  if (final_out && len == 0 && (SHORT || (me.rank == 0 && me.warp == 0))) store_state<CH>(final_out + row, carry, me.n);
  if (!SHORT && me.ranks > 1) {            // no CTA leaves before what it was sent has come
    cluster_arrive();
    cluster_wait();
  }
  // past the sequence's last span
  for (; s0 < time; s0 += stride) {
    const int t0 = (int)s0 + at;
    if (states && (SHORT || me.warp == 0) && t0 < time)
      store_state<CH>(states + ((long long)me.b * kept + t0 / SPAN) * channels + me.c, carry, me.n);
    T* o = out + ((long long)me.b * time + t0) * channels + me.c;
    for (int i = 0; i < STEPS; ++i)
      if (me.n > 0 && t0 + i < time) store_word<T, VEC>(o + (long long)i * channels, 0u, me.n);
  }
}

// ---------------------------------------------------------------------------
// gradient

template <typename T, int FORM, bool FULL>
__device__ __forceinline__ void backward_maps(const Gates<T, FORM>& gates, const unsigned (&rg)[kStepsBackward],
                                              const unsigned (&xs)[kStepsBackward], const unsigned (&gs)[kStepsBackward],
                                              LaneV<T> (&a)[kStepsBackward], LaneV<T> (&rest)[kStepsBackward],
                                              Map<LaneV<T>>& map, LaneV<T>& M, int steps) {
#pragma unroll
  for (int i = 0; i < kStepsBackward; ++i) {
    gates(rg[i], a[i], rest[i]);
    if (!FULL && i >= steps) {
      both(a[i], 1.0f);
      both(rest[i], 0.0f);
    }
    const LaneV<T> u = gates.input(rest[i], unpack<T>(xs[i]));
    map.H = i ? fma(a[i], map.H, u) : u;
    map.A = i ? mul(map.A, a[i]) : a[i];
    M = i ? fma(map.A, unpack<T>(gs[i]), M) : mul(map.A, unpack<T>(gs[i]));
  }
}

template <typename T, int FORM, bool VEC, bool SHORT>
__global__ void __launch_bounds__(32 * kWarps, 2)
recurrence_grad_kernel(View grad, View x, View gate, Shape shape, const float* states, const float* grad_final,
                       T* grad_x, T* grad_gate, float* grad_initial) {
  using V = LaneV<T>;
  constexpr int CH = Lane<T>::CH, STEPS = kStepsBackward, SPAN = STEPS * kWarps;
  __shared__ Map<V> s_warp[2][kWarps][32];       // (A, H)
  __shared__ V s_back[2][kWarps][32];            // M
  __shared__ Map<V> s_cta[2][kMaxCluster][32];   // (A, M)
  __shared__ Map<V> s_pair[2][32];               // (A, H) of the CTA before an odd one, which begins with no kept state
  __shared__ unsigned long long s_bar[2];
  if (!SHORT) {
    if (threadIdx.x < 2) mbar_init(&s_bar[threadIdx.x], 1);
    cluster_arrive();
  }
  dep_wait();
  dep_launch();
  const Gates<T, FORM> gates;
  const Place<T, SHORT> me(shape);
  const int len = me.len, time = shape.time, channels = shape.channels;
  const long long row = (long long)me.b * channels + me.c;
  V carry;
  load_state<CH>(carry, grad_final + row, grad_final ? me.n : 0);
  V first = carry;                               // what the sequence's first step hands back
  const int stride = SHORT ? STEPS : me.ranks * SPAN;
  const int at = SHORT ? 0 : me.rank * SPAN + me.warp * STEPS;
  const int kept = (time + DET_RECURRENCE_KEEP - 1) / DET_RECURRENCE_KEEP;
  // from the sequence's last span back
  const int last = len > 0 ? (len - 1) / stride * stride : -stride;
  for (long long s0 = (long long)last + stride; s0 < time; s0 += stride)
    for (int i = 0; i < STEPS; ++i)
      if (me.n > 0 && s0 + at + i < time) {
        const long long o = ((long long)me.b * time + s0 + at + i) * channels + me.c;
        store_word<T, VEC>(grad_x + o, 0u, me.n);
        store_word<T, VEC>(grad_gate + o, 0u, me.n);
      }
  unsigned rg[STEPS], rx[STEPS], rd[STEPS];
  bool full = false;
  auto load = [&](int s0) {
    full = me.whole && s0 + at + STEPS <= len;
    load_piece<T, VEC>(rg, gate, me.b, me.c, me.n, s0, at, len, full);
    load_piece<T, VEC>(rx, x, me.b, me.c, me.n, s0, at, len, full);
    if (grad.p) {
      load_piece<T, VEC>(rd, grad, me.b, me.c, me.n, s0, at, len, full);
    } else {
#pragma unroll
      for (int i = 0; i < STEPS; ++i) rd[i] = 0;
    }
  };
  if (last >= 0) load(last);
  if (!SHORT) cluster_wait();
  int round = 0;
  bool lost = false;
  for (int s0 = last; s0 >= 0; s0 -= stride, ++round) {
    const int parity = round & 1;
    const int t0 = s0 + at;
    V a[STEPS], rest[STEPS], M;
    Map<V> map;
    const bool all_in = full;
    unsigned xs[STEPS], gs[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) xs[i] = rx[i], gs[i] = rd[i];
    V h;
    load_state<CH>(h, states + ((long long)me.b * kept + t0 / DET_RECURRENCE_KEEP) * channels + me.c, t0 < len ? me.n : 0);
    if (all_in) backward_maps<T, FORM, true>(gates, rg, xs, gs, a, rest, map, M, STEPS);
    else backward_maps<T, FORM, false>(gates, rg, xs, gs, a, rest, map, M, len - t0);
    if (!SHORT && s0 > 0) load(s0 - stride);
    V m = carry;
    if (!SHORT) {
      s_warp[parity][me.warp][me.lane] = map;
      s_back[parity][me.warp][me.lane] = M;
      __syncthreads();
      if (me.ranks > 1) {
        if (me.warp < me.ranks) {                // warp r tells CTA r
          map.A = s_warp[parity][kWarps - 1][me.lane].A;
          map.H = s_back[parity][kWarps - 1][me.lane];
#pragma unroll
          for (int w = kWarps - 2; w >= 0; --w) {
            const V A = s_warp[parity][w][me.lane].A;
            map.H = after<FORM>(map.H, A, s_back[parity][w][me.lane]);
            map.A = mul(map.A, A);
          }
          if (!lost) put(&s_cta[parity][me.rank][me.lane], &s_bar[parity], me.warp, map);
        }
        if (me.warp == 0 && me.rank % 2 == 0 && !lost) {
          map = s_warp[parity][0][me.lane];
#pragma unroll
          for (int w = 1; w < kWarps; ++w) {
            const Map<V> q = s_warp[parity][w][me.lane];
            map.H = after<FORM>(map.H, q.A, q.H);
            map.A = mul(map.A, q.A);
          }
          put(&s_pair[parity][me.lane], &s_bar[parity], me.rank + 1, map);
        }
        if (threadIdx.x == 0 && !lost)
          mbar_arrive_expect_tx(&s_bar[parity], (me.ranks + me.rank % 2) * 32 * (unsigned)sizeof(Map<V>));
        lost = lost || !messages_in(&s_bar[parity], round >> 1 & 1);
        if (lost) both(m, __int_as_float(0x7fffffff));
        int r = me.ranks - 1;
        for (; r > me.rank; --r) {
          const Map<V> q = s_cta[parity][r][me.lane];
          m = after<FORM>(m, q.A, q.H);
        }
        carry = m;
        for (; r >= 0; --r) {
          const Map<V> q = s_cta[parity][r][me.lane];
          carry = after<FORM>(carry, q.A, q.H);
        }
        if (me.rank % 2) {
          const Map<V> q = s_pair[parity][me.lane];
          h = after<FORM>(h, q.A, q.H);
        }
      }
      for (int w = 0; w < me.warp; ++w) {
        const Map<V> q = s_warp[parity][w][me.lane];
        h = after<FORM>(h, q.A, q.H);
      }
      for (int w = kWarps - 1; w > me.warp; --w) m = after<FORM>(m, s_warp[parity][w][me.lane].A, s_back[parity][w][me.lane]);
    }
    // forward again: what l is multiplied by for the gate, without 1 - a
    V factor[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const V xi = unpack<T>(xs[i]);
      factor[i] = FORM == DET_GATE_DECAY ? h : mul(a[i], minus(h, xi));
      h = fma(a[i], h, gates.input(rest[i], xi));
    }
    const long long base = ((long long)me.b * time + s0) * channels;
    if (all_in) {
      const unsigned step = (unsigned)channels * (unsigned)sizeof(T);
      unsigned o = (unsigned)(at + STEPS) * step + (unsigned)me.c * (unsigned)sizeof(T);
      char* bx = reinterpret_cast<char*>(grad_x + base);
      char* bg = reinterpret_cast<char*>(grad_gate + base);
#pragma unroll
      for (int i = STEPS - 1; i >= 0; --i) {
        o -= step;
        const V l = add(unpack<T>(gs[i]), m);
        const V dx = gates.input(rest[i], l);
        m = mul(a[i], l);
        store_word<T, VEC>(reinterpret_cast<T*>(bx + o), pack<T>(dx), CH);
        store_word<T, VEC>(reinterpret_cast<T*>(bg + o), pack<T>(mul(dx, factor[i])), CH);
      }
    } else {
      const long long o = base + (long long)at * channels + me.c;
#pragma unroll
      for (int i = STEPS - 1; i >= 0; --i) {
        const V l = add(unpack<T>(gs[i]), m);
        const V dx = gates.input(rest[i], l);
        const bool inside = t0 + i < len;
        if (inside) m = mul(a[i], l);
        if (me.n > 0 && t0 + i < time) {
          store_word<T, VEC>(grad_x + o + (long long)i * channels, inside ? pack<T>(dx) : 0u, me.n);
          store_word<T, VEC>(grad_gate + o + (long long)i * channels, inside ? pack<T>(mul(dx, factor[i])) : 0u, me.n);
        }
      }
    }
    first = m;
  }
  if (!SHORT && me.ranks > 1) {
    cluster_arrive();
    cluster_wait();
  }
  if (grad_initial && (SHORT || (me.rank == 0 && me.warp == 0))) store_state<CH>(grad_initial + row, first, me.n);
}

// A launch over channel tiles and sequences: a single piece without clusters, else
// with as many CTAs a cluster as a sequence fills, at most 8.
template <typename T, int STEPS, typename... KArgs, typename... Args>
int launch_recurrence(const char* name, void (*short_kernel)(KArgs...), void (*kernel)(KArgs...), int batch,
                      const Shape& shape, cudaStream_t s, Args... args) {
  const int words = (shape.channels + Lane<T>::CH - 1) / Lane<T>::CH;
  const bool brief = shape.time <= STEPS;
  const int ranks = 1 << shape.log2_ranks;
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

// The shape with the cluster's size, and whether 32-bit offsets reach over its spans.
template <typename T, int STEPS>
Shape with_ranks(Shape shape, std::initializer_list<long long> strides) {
  while ((1 << shape.log2_ranks) < kMaxCluster && (STEPS * kWarps << shape.log2_ranks) < shape.time) ++shape.log2_ranks;
  shape.near = 1;
  for (const long long st : strides)
    if (st >= (1LL << 31) || (st * (STEPS * kWarps << shape.log2_ranks) + shape.channels) * (long long)sizeof(T) >= (1LL << 31))
      shape.near = 0;
  return shape;
}

template <typename T, int FORM, bool VEC>
int forward(const View& x, const View& gate, const Shape& shape, int batch, const float* initial, void* out,
            float* final_out, float* states, cudaStream_t s) {
  const Shape sh = with_ranks<T, kStepsForward>(shape, {x.st, gate.st, shape.channels});
  return launch_recurrence<T, kStepsForward>("det_linear_recurrence", recurrence_kernel<T, FORM, VEC, true>,
                                             recurrence_kernel<T, FORM, VEC, false>, batch, sh, s, x, gate, sh, initial,
                                             static_cast<T*>(out), final_out, states);
}
template <typename T, int FORM, bool VEC>
int backward(const View& grad, const View& x, const View& gate, const Shape& shape, int batch, const float* states,
             const float* grad_final, void* grad_x, void* grad_gate, float* grad_initial, cudaStream_t s) {
  const Shape sh = with_ranks<T, kStepsBackward>(shape, {grad.st, x.st, gate.st, shape.channels});
  return launch_recurrence<T, kStepsBackward>(
      "det_linear_recurrence_backward", recurrence_grad_kernel<T, FORM, VEC, true>,
      recurrence_grad_kernel<T, FORM, VEC, false>, batch, sh, s, grad, x, gate, sh, states, grad_final,
      static_cast<T*>(grad_x), static_cast<T*>(grad_gate), grad_initial);
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
  const Shape shape = {(int)time, (int)channels, lengths, 0, 0};
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
  const Shape shape = {(int)time, (int)channels, lengths, 0, 0};
  const cudaStream_t s = as_stream(stream);
  DET_RECURRENCE_PICK(backward, vd, vx, vg, shape, (int)batch, states, grad_final, grad_x, grad_gate, grad_initial, s);
}
