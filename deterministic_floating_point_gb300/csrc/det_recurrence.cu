// det_linear_recurrence and its gradient: h = a[t] h + u[t] along time, for
// every sequence and channel.
//
// A step is the map h -> a h + u; a run of steps is a map of the same kind,
// h -> A h + H with A the product of its decays and H its result from 0.  Time
// is cut into blocks of 128 steps (a CTA) and these into pieces of 8 (a warp, over
// 32 words of channels).  A warp forms its piece's (A, H).  A further warp of the
// CTA joins them and tells the other CTAs of the cluster, which hold the
// sequence's other blocks; another one hears of theirs and tells each warp the
// state its piece begins with.  The warp then runs through its piece again.  Every
// input is read from memory once (copied into shared memory up to three rounds
// ahead, kept in registers between the two passes) and every output written once.
//
// Nothing waits for the chain of states but the second pass: (A, H) of a round do
// not depend on the states, so warps form those of the next round, and CTAs send
// theirs, before the states of this one are known.  Without that the CTAs of a
// cluster spent half of their time on waiting for each other.
//
// Blocks and pieces have fixed borders and are joined one after the other in the
// order of time, by the same operations whatever the number of CTAs that share a
// sequence; so the bits of a step are a function of the steps before it.
//
// The gradient runs the same way from the end.  With m = a[t] l the value that
// step t hands to step t - 1, l = grad[t] + m, and a piece is m -> A m + M.  The
// states inside a block are formed again from the one kept before it, so that the
// gates' gradients see 32-bit states and x, not h, is read.
//
// What bounds it: bytes, once an element costs few enough instructions (at the
// copy's rate an SM's schedulers have 33 slots for each element forward and
// twice that backward).  So two 16-bit channels of a word are worked on by packed
// 32-bit instructions, and whole pieces have no conditions.  8 x 4,096 x 2,048 in bf16: 75 us, 5.4 TB/s
// (gradient 135 us, 5.0 TB/s), at 47% of the issue slots: a CTA fills the SM's shared memory, and its 18
// warps wait for each other twice a round.
#include "../../include/det_test_hooks.h"
#include "det_model.cuh"

#include <algorithm>
#include <initializer_list>
#include <map>
#include <mutex>
#include <tuple>
#include <type_traits>

namespace det {
namespace {

constexpr int kBlock = DET_RECURRENCE_KEEP;  // steps of a CTA; a kept state stands before each
constexpr int kMaxCluster = 8;
constexpr int kSteps = 8;                    // of a piece: two rounds' pieces are in registers at a time
constexpr int kWorkers = kBlock / kSteps;
constexpr int kStages = 3;                   // rounds whose inputs are in shared memory or on their way
static_assert(kBlock == DET_RECURRENCE_SPAN, "decays are multiplied over blocks");

struct View {
  const void* p;
  long long sb, st;   // elements from one sequence and step to the next
};
struct Shape {
  int time, channels;
  const int32_t* lengths;
  int log2_ranks;     // CTAs of a cluster
  float lowest_gate;  // -87, as a value that the compiler does not know: it would work out what belongs to it by itself,
                      // and one step beside the hardware's approximations
  int withheld;       // the round whose message the cluster's first CTA never sends (test hook), else -1
  unsigned long long wait_ns;
};

// ---------------------------------------------------------------------------
// A lane's values: two 16-bit channels of a word as a packed pair, one of 32 bits.

using det::add;
using det::fma;
using det::minus;
using det::mul;
__device__ __forceinline__ float add(float a, float b) { return __fadd_rn(a, b); }
__device__ __forceinline__ float mul(float a, float b) { return __fmul_rn(a, b); }
__device__ __forceinline__ float fma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ void both(float& v, float x) { v = x; }
__device__ __forceinline__ void both(Two& v, float x) { v = twice(x); }
__device__ __forceinline__ float minus(float a, float b) { return __fsub_rn(a, b); }

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
    return two(a, b);
  }
}
template <typename T>
__device__ __forceinline__ unsigned pack(LaneV<T> v) {
  if constexpr (sizeof(T) == 4) {
    return __float_as_uint(v);
  } else {
    const float2 f = (v);
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

// v, after it has arrived: a shuffle needs its value.
__device__ __forceinline__ float here_by_now(float v, int lane) { return __shfl_sync(0xffffffffu, v, lane); }
__device__ __forceinline__ Two here_by_now(Two v, int lane) {
  return two(__shfl_sync(0xffffffffu, v.x, lane), __shfl_sync(0xffffffffu, v.y, lane));
}

// 32-bit state of a lane's channels in [.., channels] floats at p.
template <int CH, typename V>
__device__ __forceinline__ void load_state(V& v, const float* p, int n) {
  if constexpr (CH == 1) v = n > 0 ? p[0] : 0.0f;
  else v = two(n > 0 ? p[0] : 0.0f, n > 1 ? p[1] : 0.0f);
}
template <int CH, typename V>
__device__ __forceinline__ void store_state(float* p, V v, int n) {
  if constexpr (CH == 1) {
    if (n > 0) p[0] = v;
  } else {
    const float2 f = (v);
    if (n > 0) p[0] = f.x;
    if (n > 1) p[1] = f.y;
  }
}

// ---------------------------------------------------------------------------
// Gates: a word of them to the decays a and what is left, 1 - a.
//
// Sigmoid: with e = exp(-z), a = 1 / (1 + e) and 1 - a = e a, which keeps the
// relative accuracy of both where a difference from 1 would lose it.  In 16 bits e
// and the reciprocal are the hardware's approximations: a and 1 - a are off by at most
// 8 + 1.22 |z| units of 2^-24 of their own size.  (The rounded exponent counts |z|
// times.  Half a step of a bf16 gate moves them by 2^-9 |z|, of an f16 one by 2^-12 |z|,
// so a reduction of every gate's range would show in nothing.)  z is held at -87 and
// more, so that e stays finite, and the a that belongs to -87 is taken off (`floor`,
// below 2^-125): a gate of -inf closes for good.  In 32 bits expf, and the smaller one
// of the two by a division.
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
  __device__ __forceinline__ explicit Gates(float lowest) {
    both(floor, 0.0f);
    if constexpr (FORM == DET_GATE_SIGMOID && sizeof(T) == 2) {
      const float e = exp2_approx(__fmul_rn(lowest, -kLog2e));
      const float a = -rcp_approx(__fadd_rn(e, 1.0f));
      floor = two(a, a);
    }
  }
  __device__ __forceinline__ void operator()(unsigned w, V& a, V& rest) const {
    if constexpr (FORM == DET_GATE_DECAY) {
      a = unpack<T>(w);
      both(rest, 1.0f);
    } else if constexpr (sizeof(T) == 2) {
      const Two t = mul(unpack<T>(at_least(w, kLowestGate, T())), two(-kLog2e, -kLog2e));
      const float2 f = (t);
      const Two e = two(exp2_approx(f.x), exp2_approx(f.y));
      const float2 d = (add(e, two(1.0f, 1.0f)));
      a = two(rcp_approx(d.x), rcp_approx(d.y));
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

// The state h after a run of steps (A, H).
template <typename V>
__device__ __forceinline__ V after(V h, V A, V H) { return fma(A, h, H); }
// After whole blocks.  Decays above 1 may take a block's A out of the range of 32 bits
// where the states stay in it: from 0 the state is H whatever A is.
template <int FORM>
__device__ __forceinline__ float after_block(float h, float A, float H) {
  return FORM == DET_GATE_DECAY && h == 0.0f ? H : fmaf(A, h, H);
}
template <int FORM>
__device__ __forceinline__ Two after_block(Two h, Two A, Two H) {
  if constexpr (FORM == DET_GATE_SIGMOID) {
    return fma(A, h, H);
  } else {
    const float2 g = (h), a = (A), b = (H);
    return two(after_block<FORM>(g.x, a.x, b.x), after_block<FORM>(g.y, a.y, b.y));
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
// `bytes` from `from` to the place of `to` in the shared memory of the cluster's CTA `rank`,
// counted there on the barrier at the place of `bar`.  (A barrier of the whole cluster
// in its place would wait for all stores of outputs in flight.)
__device__ __forceinline__ void copy_to(int rank, void* to, const void* from, unsigned bytes, unsigned long long* bar) {
  unsigned dst, remote_bar;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(dst) : "r"(smem_u32(to)), "r"(rank));
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote_bar) : "r"(smem_u32(bar)), "r"(rank));
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "r"(smem_u32(from)), "r"(bytes), "r"(remote_bar)
               : "memory");
}
// Writes to shared memory before it are seen by copies after it.
__device__ __forceinline__ void fence_copies() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// Waits for a phase of messages, for about wait_ns at most.  (The timer is read after
// many polls only: reading it takes as long as a message.)
template <bool CLUSTER>
__device__ __forceinline__ bool messages_in(unsigned long long* bar, unsigned phase, unsigned long long wait_ns) {
  unsigned long long t0 = 0;
  for (unsigned polls = 1;; ++polls) {
    unsigned done;
    if (CLUSTER) {
      asm volatile(
          "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(done)
          : "r"(smem_u32(bar)), "r"(phase)
          : "memory");
    } else {
      done = mbar_try_wait(bar, phase);
    }
    if (done) return true;
    if ((polls & 1023u) == 0) {
      const unsigned long long now = globaltimer();
      if (t0 == 0) t0 = now;
      else if (now - t0 > wait_ns) return false;
    }
  }
}

// Between warps of a CTA: arrive() does not wait, join() waits until all of the
// barrier's threads have come.
template <int BARRIER>
__device__ __forceinline__ void arrive(int threads) {
  asm volatile("bar.arrive %0, %1;" ::"n"(BARRIER), "r"(threads) : "memory");
}
template <int BARRIER>
__device__ __forceinline__ void join(int threads) {
  asm volatile("bar.sync %0, %1;" ::"n"(BARRIER), "r"(threads) : "memory");
}
constexpr int kMapsIn = 1, kStatesIn = 3;      // named barriers, two each for even and odd rounds
// f(0 or 1, k) for every round k, with k's parity as a constant.
template <typename F>
__device__ __forceinline__ void each_round(int rounds, F&& f) {
  for (int k = 0; k < rounds; k += 2) {
    f(std::integral_constant<int, 0>(), k);
    if (k + 1 < rounds) f(std::integral_constant<int, 1>(), k + 1);
  }
}

// ---------------------------------------------------------------------------
// Where a CTA works: blocks rank, rank + ranks, ... of a sequence, 32 words of
// channels.
template <typename T>
struct Place {
  int warp, lane, b, c0, c, n;     // c0: of the tile; n: the lane's channels, from c on
  int rank, ranks, stride, workers;
  int len, rounds;                 // of the sequence
  bool whole;                      // the tile has all its channels
  __device__ __forceinline__ explicit Place(const Shape& s) {
    constexpr int CH = Lane<T>::CH;
    warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    lane = threadIdx.x & 31;
    workers = (blockDim.x >> 5) - 2;
    b = blockIdx.y;
    ranks = 1 << s.log2_ranks;
    stride = ranks * kBlock;
    rank = blockIdx.x & (ranks - 1);             // clusters lie along x
    c0 = (blockIdx.x >> s.log2_ranks) * 32 * CH;
    c = c0 + lane * CH;
    n = max(0, min(CH, s.channels - c));
    whole = c0 + 32 * CH <= s.channels;
    len = s.time;
    if (s.lengths) len = max(0, min(len, (int)s.lengths[b]));
    rounds = (int)(((long long)len + stride - 1) / stride);
  }
};

template <int VEC>
__device__ __forceinline__ void copy_async(void* dst, const void* src, int bytes) {
  if (VEC == 2) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the last one or two committed groups of this thread's copies have arrived.
__device__ __forceinline__ void copies_wait_but_one() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }
__device__ __forceinline__ void copies_wait_but_two() { asm volatile("cp.async.wait_group 2;" ::: "memory"); }
static_assert(kStages == 3, "so many groups are asked for after the one that is waited for");

// Copies a warp's pieces of one operand into its part of shared memory, [kSteps][pitch]
// words, 0 past the sequence and the channels, round after round.  VEC 2: rows of 16-byte
// vectors; 1: of words; 0: of 16-bit elements at any address: the words that hold them,
// one more than the row's if it starts in the middle of one.  (Such a first word's lower half is
// not the row's, but lies beside it in a word.)
__host__ __device__ constexpr int pitch(int vec) { return vec == 0 ? 33 : 32; }
template <typename T, int VEC>
struct Reader {
  const T* p;            // the lane's first element of the next piece
  static constexpr int kRows = VEC == 2 ? 4 : 1;             // that a copy of the warp takes
  static __device__ __forceinline__ int first_channel(const Place<T>& me) {
    return VEC == 2 ? me.c0 + (me.lane & 7) * (4 * Lane<T>::CH) : me.c;
  }
  // first: step of the first round's piece
  __device__ __forceinline__ Reader(const View& v, const Place<T>& me, int first) {
    p = static_cast<const T*>(v.p) + (me.b * v.sb + (first + (VEC == 2 ? me.lane >> 3 : 0)) * v.st + first_channel(me));
  }
  // the piece from step t0 on, with all its steps and channels if full; by: steps to the next round's
  __device__ __forceinline__ void next(unsigned (*to)[pitch(VEC)], const View& v, const Place<T>& me, bool full, int t0,
                                       int by, int channels) {
    const long long step = kRows * v.st;
    if constexpr (VEC == 0) {
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const uintptr_t q = reinterpret_cast<uintptr_t>(p + i * step);
        const int odd = (int)(q >> 1 & 1);
        copy_part(&to[i][me.lane], q & ~(uintptr_t)3, channels - (me.c - odd), t0 + i < me.len, v);
      }
      if (me.lane < kSteps) {           // the rows' last words, a lane a row
        const uintptr_t q = reinterpret_cast<uintptr_t>(p + me.lane * step + (31 - me.lane) * 2);
        const int odd = (int)(q >> 1 & 1);
        copy_part(&to[me.lane][32], (q & ~(uintptr_t)3) + 4, channels - (me.c0 + 64 - odd), t0 + me.lane < me.len, v);
      }
    } else {
      unsigned* dst = VEC == 2 ? &to[me.lane >> 3][(me.lane & 7) * 4] : &to[0][me.lane];
      const int row = VEC == 2 ? me.lane >> 3 : 0;
      const T* q = p;
#pragma unroll
      for (int j = 0; j < kSteps / kRows; ++j, q += step) {
        if (full) {
          copy_async<VEC>(dst + j * kRows * 32, q, VEC == 2 ? 16 : 4);
        } else {
          const bool ok = first_channel(me) < channels && t0 + row + j * kRows < me.len;
          copy_async<VEC>(dst + j * kRows * 32, ok ? q : v.p, ok ? VEC == 2 ? 16 : 4 : 0);   // (0 bytes are read)
        }
      }
    }
    p += by * v.st;
  }
  // A word of which `left` elements are of the tensor.
  static __device__ __forceinline__ void copy_part(unsigned* dst, uintptr_t src, int left, bool valid, const View& v) {
    const int bytes = valid ? max(0, min(2, left)) * 2 : 0;
    copy_async<1>(dst, bytes ? reinterpret_cast<const void*>(src) : reinterpret_cast<const void*>(
                                 reinterpret_cast<uintptr_t>(v.p) & ~(uintptr_t)3), bytes);
  }
};

// A lane's words of a piece, operand `which` of the stage at raw.
template <int VEC> struct Words {
  const unsigned (*raw)[kSteps][pitch(VEC)];
  unsigned odd;          // VEC 0: bits 2 which and 2 which + 1: even and odd rows start in the middle of a word
  int lane;
  bool graded;           // there is an operand 2
  __device__ __forceinline__ unsigned operator()(int which, int i) const {
    if (which == 2 && !graded) return 0u;
    const unsigned w = raw[which][i][lane];
    if constexpr (VEC == 0) return __funnelshift_r(w, raw[which][i][lane + 1], (odd >> (2 * which + (i & 1)) & 1) * 16);
    return w;
  }
  // pieces start at multiples of 8 steps, tiles at even channels: a row's place in its word is a matter of its number
  static __device__ __forceinline__ unsigned odd_rows(const View& v, int b, int which) {
    const unsigned first = (unsigned)((reinterpret_cast<uintptr_t>(v.p) >> 1) + b * v.sb) & 1u;
    return (first | (first ^ ((unsigned)v.st & 1u)) << 1) << (2 * which);
  }
};

// A row of a tile of the outputs.  VEC 0, 16 bits: at an odd element the lanes' words are
// shifted by one element, and the first and the last element go by themselves.
template <typename T, int VEC>
__device__ __forceinline__ void store_row(T* p, unsigned w, int n, bool valid) {
  if constexpr (VEC != 0 || sizeof(T) == 4) {        // (-1: element by element)
    if (valid && n > 0) store_word<T, (VEC > 0)>(p, w, n);
  } else {
    const unsigned before = __shfl_up_sync(0xffffffffu, w, 1);
    const int after = __shfl_down_sync(0xffffffffu, n, 1), lane = threadIdx.x & 31;
    if (!valid || n <= 0) return;
    unsigned short* q = reinterpret_cast<unsigned short*>(p);
    if (reinterpret_cast<uintptr_t>(p) % 4 == 0) {
      store_word<T, true>(p, w, n);
    } else {
      if (lane == 0) q[0] = (unsigned short)w;
      else *reinterpret_cast<unsigned*>(q - 1) = before >> 16 | w << 16;
      if (n == 2 && (lane == 31 || after <= 0)) q[1] = (unsigned short)(w >> 16);
    }
  }
}

// A warp's part of the stages.
template <int VEC> struct Ring {
  unsigned* first;
  int words;             // from one stage to the next
  __device__ __forceinline__ unsigned (*at(int stage) const)[kSteps][pitch(VEC)] {
    return reinterpret_cast<unsigned(*)[kSteps][pitch(VEC)]>(first + stage * words);
  }
};

// ---------------------------------------------------------------------------
// What CTAs of a cluster tell each other: the map of each one's block.  Messages of
// four rounds have places: a CTA may be told of round k + 2 while it still reads those
// of k and k - 1.  (A CTA sends round k + 4 after it has heard of everyone's round k + 2, which
// is sent after round k has been heard: by then its own place is free too.)
// A wait that gives up is the CTA's last: it is `lost`, and waits no more.  It sends one round more at most (the argument above
// holds for that one), so that no message can be taken for another round's.  The others run out of their own waits
// then, if they have rounds left.
template <typename V>
struct Messages {
  alignas(16) Map<V> mine[4][32];
  Map<V> from[4][kMaxCluster][32];
  unsigned long long bar[4];
  int lost;
};
// To how many CTAs the message of this round goes: all of the cluster's, or none.  (Asked for before the round's maps have come,
// where the warp waits anyway, and used as a bound: a branch around the sending took 2% of a long sequence's time.)
template <typename V, typename PLACE>
__device__ __forceinline__ int receivers(const Messages<V>& box, const PLACE& me, int round, int withheld) {
  const bool none = __shfl_sync(0xffffffffu, *(volatile const int*)&box.lost, 0) || (round == withheld && me.rank == 0);
  return none ? 0 : me.ranks;
}
template <typename V, typename PLACE>
__device__ __forceinline__ void send(Messages<V>& box, const PLACE& me, int round, const Map<V>& map, int to) {
  const int k = round & 3;
  if (me.ranks == 1) {                 // no cluster: its instructions must not be used
    box.from[k][0][me.lane] = map;
    __syncwarp();
    if (me.lane == 0) mbar_arrive(&box.bar[k]);
    return;
  }
  box.mine[k][me.lane] = map;
  fence_copies();
  if (me.lane < min(to, 1)) mbar_arrive_expect_tx(&box.bar[k], me.ranks * 32 * (unsigned)sizeof(Map<V>));
  __syncwarp();
  if (me.lane < to)
    copy_to(me.lane, &box.from[k][me.rank][0], &box.mine[k][0], 32 * (unsigned)sizeof(Map<V>), &box.bar[k]);
}
// The state (or what comes back) at the CTA's block, from the one at the cluster's
// blocks, v, which moves on past them.  BACK: from the last block to the first.
template <int FORM, bool BACK, typename V, typename PLACE>
__device__ __forceinline__ V receive(Messages<V>& box, const PLACE& me, int round, V& v, bool& lost,
                                     unsigned long long wait_ns) {
  const int k = round & 3;
  const unsigned phase = round >> 2 & 1;
  lost = lost || !(me.ranks == 1 ? messages_in<false>(&box.bar[k], phase, wait_ns)
                                 : messages_in<true>(&box.bar[k], phase, wait_ns));
  if (lost) {
    both(v, __int_as_float(0x7fffffff));
    if (me.lane == 0) box.lost = 1;
  }
  V here = v;
  const int first = BACK ? me.ranks - 1 : 0, by = BACK ? -1 : 1;
  for (int j = 0, r = first; j < me.ranks; ++j, r += by) {
    if (r == me.rank) here = v;
    const Map<V> q = box.from[k][r][me.lane];
    v = after_block<FORM>(v, q.A, q.H);
  }
  return here;
}

// A cluster's end: no CTA leaves before what it was sent has come.  One that has heard every round has it all; a lost one
// gives what was sent before the barrier a millisecond.
template <typename V>
__device__ __forceinline__ void leave(const Messages<V>& box) {
  cluster_arrive();
  cluster_wait();
  if (box.lost)
    for (const unsigned long long t0 = globaltimer(); globaltimer() - t0 < 1000000;) {
    }
}

// ---------------------------------------------------------------------------

// A piece's decays and what its steps add, and its map.  A step past the end is
// (1, 0).
template <typename T, int FORM, bool FULL, typename WORDS>
__device__ __forceinline__ Map<LaneV<T>> piece_map(const Gates<T, FORM>& gates, const WORDS& words, LaneV<T> (&a)[kSteps],
                                                   LaneV<T> (&u)[kSteps], int steps) {
  Map<LaneV<T>> map;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    LaneV<T> rest;
    gates(words(0, i), a[i], rest);
    u[i] = gates.input(rest, unpack<T>(words(1, i)));
    if (!FULL && i >= steps) {
      both(a[i], 1.0f);
      both(u[i], 0.0f);
    }
    map.H = i ? fma(a[i], map.H, u[i]) : u[i];
    map.A = i ? mul(map.A, a[i]) : a[i];
  }
  return map;
}

template <typename T, int FORM, int VEC>
__global__ void __launch_bounds__(32 * (kWorkers + 2), 1)
recurrence_kernel(View x, View gate, Shape shape, const float* initial, T* out, float* final_out, float* states) {
  using V = LaneV<T>;
  constexpr int CH = Lane<T>::CH;
  extern __shared__ __align__(128) unsigned s_raw[];     // [stages][workers][gate, x][kSteps][32]
  __shared__ Map<V> s_map[2][kWorkers][32];              // of the pieces; then A: the state a piece begins with
  __shared__ Messages<V> s_box;
  if (threadIdx.x < 4) mbar_init(&s_box.bar[threadIdx.x], 1);
  if (threadIdx.x == 0) s_box.lost = 0;
  if (shape.log2_ranks > 0) cluster_arrive();            // a box is written only after its CTA has come here
  dep_wait();
  dep_launch();
  const Place<T> me(shape);
  const int len = me.len, time = shape.time, channels = shape.channels, threads = blockDim.x;
  const long long row = (long long)me.b * channels + me.c;   // of the sequence's states
  V carry;
  load_state<CH>(carry, initial + row, initial && me.warp >= me.workers ? me.n : 0);
  // (the shuffle waits for it: a CTA that has heard of all may write the final state to the same place)
  carry = here_by_now(carry, me.lane);
  if (shape.log2_ranks > 0) cluster_wait();
  else __syncthreads();

  if (me.warp == me.workers) {
    // tells of the CTA's blocks
    each_round(me.rounds, [&](auto parity, int k) {
      constexpr int P = decltype(parity)::value;
      const int to = receivers(s_box, me, k, shape.withheld);
      join<kMapsIn + P>(threads);
      Map<V> map;
      both(map.A, 1.0f);
      both(map.H, 0.0f);
#pragma unroll 1
      for (int w0 = 0; w0 < me.workers; w0 += 4) {           // four at a time are on their way
        Map<V> q[4];
#pragma unroll
        for (int w = 0; w < 4; ++w)
          if (w0 + w < me.workers) q[w] = s_map[P][w0 + w][me.lane];
#pragma unroll
        for (int w = 0; w < 4; ++w)
          if (w0 + w < me.workers) {
            map.H = after(map.H, q[w].A, q[w].H);
            map.A = mul(map.A, q[w].A);
          }
      }
      send(s_box, me, k, map, to);
    });
  } else if (me.warp > me.workers) {
    // hears of the cluster's, and hands out states
    const int kept = (time + kBlock - 1) / kBlock;
    bool lost = false;                 // a wait gave up: states are NaN from there on
    each_round(me.rounds, [&](auto parity, int k) {
      constexpr int P = decltype(parity)::value;
      join<kMapsIn + P>(threads);
      V h = receive<FORM, false>(s_box, me, k, carry, lost, shape.wait_ns);
      const int block = k * me.ranks + me.rank;
      if (states && block < kept) store_state<CH>(states + ((long long)me.b * kept + block) * channels + me.c, h, me.n);
#pragma unroll 1
      for (int w0 = 0; w0 < me.workers; w0 += 4) {
        Map<V> q[4];
#pragma unroll
        for (int w = 0; w < 4; ++w)
          if (w0 + w < me.workers) q[w] = s_map[P][w0 + w][me.lane];
#pragma unroll
        for (int w = 0; w < 4; ++w)
          if (w0 + w < me.workers) {
            s_map[P][w0 + w][me.lane].A = h;
            h = after(h, q[w].A, q[w].H);
          }
      }
      arrive<kStatesIn + P>(threads - 32);
    });
    if (states)                        // past the sequence's last round
      for (int block = me.rounds * me.ranks + me.rank; block < kept; block += me.ranks)
        store_state<CH>(states + ((long long)me.b * kept + block) * channels + me.c, carry, me.n);
    if (final_out && len == 0 && me.rank == 0) store_state<CH>(final_out + row, carry, me.n);
  } else {
    const Gates<T, FORM> gates(shape.lowest_gate);
    const int at = me.rank * kBlock + me.warp * kSteps;
    // the rounds before this one have whole pieces here
    const int whole = me.whole && len >= at + kSteps ? (len - at - kSteps) / me.stride + 1 : 0;
    // and this one has the sequence's last step
    const int end = len > at && (len - 1 - at) % me.stride < kSteps ? (len - 1 - at) / me.stride : -1;
    const Ring<VEC> ring{s_raw + me.warp * (2 * kSteps * pitch(VEC)), me.workers * (2 * kSteps * pitch(VEC))};
    const unsigned odd = VEC == 0 ? Words<VEC>::odd_rows(gate, me.b, 0) | Words<VEC>::odd_rows(x, me.b, 1) : 0u;
    Reader<T, VEC> read_gate(gate, me, at), read_x(x, me, at);
    auto ask = [&](int k, unsigned (*to)[kSteps][pitch(VEC)]) {       // for the piece of round k, if there is one; in the rounds' order
      if (k < me.rounds) {
        read_gate.next(to[0], gate, me, k < whole, k * me.stride + at, me.stride, channels);
        read_x.next(to[1], x, me, k < whole, k * me.stride + at, me.stride, channels);
      }
      copies_commit();
    };
    int taken = 0;                     // stage of the next piece
    auto take = [&](auto parity, int k, V (&a)[kSteps], V (&u)[kSteps]) {
      constexpr int P = decltype(parity)::value;
      copies_wait_but_two();
      __syncwarp();
      unsigned(*w)[kSteps][pitch(VEC)] = ring.at(taken);
      const Words<VEC> words{w, odd, me.lane, false};
      s_map[P][me.warp][me.lane] = k < whole
                                           ? piece_map<T, FORM, true>(gates, words, a, u, kSteps)
                                           : piece_map<T, FORM, false>(gates, words, a, u, len - at - k * me.stride);
      __syncwarp();
      arrive<kMapsIn + P>(threads);
      ask(k + kStages, w);             // into the same stage
      taken = taken + 1 == kStages ? 0 : taken + 1;
    };
    T* o = out + ((long long)me.b * time + at) * channels + me.c;
    auto give = [&](auto parity, int k, const V (&a)[kSteps], const V (&u)[kSteps]) {
      constexpr int P = decltype(parity)::value;
      join<kStatesIn + P>(threads - 32);
      V h = s_map[P][me.warp][me.lane].A;
      T* q = o;
      if (k < whole) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i, q += channels) {
          h = fma(a[i], h, u[i]);
          store_row<T, VEC>(q, pack<T>(h), CH, true);
        }
      } else {
        const int t0 = k * me.stride + at;
#pragma unroll
        for (int i = 0; i < kSteps; ++i, q += channels) {
          h = fma(a[i], h, u[i]);
          store_row<T, VEC>(q, t0 + i < len ? pack<T>(h) : 0u, me.n, t0 + i < time);
        }
      }
      o += (long long)me.stride * channels;
      // the state at the end is that of the last step (steps past it have kept it); the
      // initial state has been read everywhere by now, so it may lie in the same place
      if (k == end && final_out) store_state<CH>(final_out + row, h, me.n);
    };
    constexpr std::integral_constant<int, 0> first;
    constexpr std::integral_constant<int, 1> second;
    V a0[kSteps], u0[kSteps], a1[kSteps], u1[kSteps];
    if (me.rounds > 0) {
      for (int k = 0; k < kStages; ++k) ask(k, ring.at(k));
      take(first, 0, a0, u0);
    }
    for (int k = 0; k < me.rounds; k += 2) {
      if (k + 1 < me.rounds) take(second, k + 1, a1, u1);
      give(first, k, a0, u0);
      if (k + 1 == me.rounds) break;
      if (k + 2 < me.rounds) take(first, k + 2, a0, u0);
      give(second, k + 1, a1, u1);
    }
    // past the sequence's last round
    for (long long t0 = (long long)me.rounds * me.stride + at; t0 < time; t0 += me.stride)
      for (int i = 0; i < kSteps; ++i)
        if (me.n > 0 && t0 + i < time) store_word<T, VEC != 0>(out + ((long long)me.b * time + t0 + i) * channels + me.c, 0u, me.n);
  }
  if (shape.log2_ranks > 0) leave(s_box);
}

// A thread's word of channels of a sequence of at most one piece: the same
// operations, without an exchange (one step of 64 x 4,096 in bf16: 6 us, 18 by the kernel above).
struct Word {
  int b, c, n, len;
  template <typename T>
  __device__ __forceinline__ Word(const Shape& s, T) {
    b = blockIdx.y;
    c = (blockIdx.x * blockDim.x + threadIdx.x) * Lane<T>::CH;
    n = max(0, min(Lane<T>::CH, s.channels - c));
    len = s.time;
    if (s.lengths) len = max(0, min(len, (int)s.lengths[b]));
  }
};
template <typename T, bool VEC, int STEPS>
__device__ __forceinline__ void load_words(unsigned (&w)[STEPS], const View& v, const Word& me) {
  const T* p = static_cast<const T*>(v.p) + (me.b * v.sb + me.c);
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    w[i] = 0;
    if (i < me.len) w[i] = load_word<T, VEC>(p + i * v.st, me.n);
  }
}

template <typename T, int FORM, bool VEC>
__global__ void __launch_bounds__(128)
recurrence_short_kernel(View x, View gate, Shape shape, const float* initial, T* out, float* final_out, float* states) {
  using V = LaneV<T>;
  constexpr int CH = Lane<T>::CH, STEPS = kSteps;
  dep_wait();
  dep_launch();
  const Gates<T, FORM> gates(shape.lowest_gate);
  const Word me(shape, T());
  if (me.n <= 0) return;
  const long long row = (long long)me.b * shape.channels + me.c;
  V h;
  load_state<CH>(h, initial + row, initial ? me.n : 0);
  unsigned rg[STEPS], rx[STEPS];
  load_words<T, VEC>(rg, gate, me);
  load_words<T, VEC>(rx, x, me);
  if (states && shape.time > 0) store_state<CH>(states + row, h, me.n);
  T* o = out + (long long)me.b * shape.time * shape.channels + me.c;
#pragma unroll
  for (int i = 0; i < STEPS; ++i, o += shape.channels) {
    if (i >= shape.time) break;
    V a, rest;
    gates(rg[i], a, rest);
    if (i < me.len) h = fma(a, h, gates.input(rest, unpack<T>(rx[i])));
    store_word<T, VEC>(o, i < me.len ? pack<T>(h) : 0u, me.n);
  }
  if (final_out) store_state<CH>(final_out + row, h, me.n);
}

// ---------------------------------------------------------------------------
// gradient

// A piece's forward map, and back M of m -> A m + M.
template <typename T, int FORM, bool FULL, typename WORDS>
__device__ __forceinline__ Map<LaneV<T>> piece_maps(const Gates<T, FORM>& gates, const WORDS& words, LaneV<T>& M, int steps) {
  using V = LaneV<T>;
  Map<V> map;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    V a, rest;
    gates(words(0, i), a, rest);
    V u = gates.input(rest, unpack<T>(words(1, i)));
    if (!FULL && i >= steps) {
      both(a, 1.0f);
      both(u, 0.0f);
    }
    map.H = i ? fma(a, map.H, u) : u;
    map.A = i ? mul(map.A, a) : a;
    const V d = unpack<T>(words(2, i));
    M = i ? fma(map.A, d, M) : mul(map.A, d);
  }
  return map;
}

// A thread's words of a piece, held in registers.
struct WordsHeld {
  const unsigned (&w)[3][kSteps];
  __device__ __forceinline__ unsigned operator()(int which, int i) const { return w[which][i]; }
};

// The gradients of a piece's steps from the state h before it and what comes back
// behind it, m; m is what it hands back.
template <typename T, int FORM, int VEC, bool FULL, typename WORDS>
__device__ __forceinline__ void piece_gradients(const Gates<T, FORM>& gates, const WORDS& words, LaneV<T> h,
                                                LaneV<T>& m, T* ox, T* og, int channels, int n, int steps, int rows) {
  using V = LaneV<T>;
  constexpr int STEPS = kSteps;
  V a[STEPS], rest[STEPS], factor[STEPS];      // factor: what l (1 - a) is multiplied by for the gate
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    gates(words(0, i), a[i], rest[i]);
    const V xi = unpack<T>(words(1, i));
    factor[i] = FORM == DET_GATE_DECAY ? h : mul(a[i], minus(h, xi));
    h = fma(a[i], h, gates.input(rest[i], xi));
  }
  ox += (long long)(STEPS - 1) * channels;
  og += (long long)(STEPS - 1) * channels;
#pragma unroll
  for (int i = STEPS - 1; i >= 0; --i, ox -= channels, og -= channels) {
    const V l = add(unpack<T>(words(2, i)), m);
    const V dx = gates.input(rest[i], l);
    if (FULL || i < steps) m = mul(a[i], l);
    store_row<T, VEC>(ox, FULL || i < steps ? pack<T>(dx) : 0u, FULL ? Lane<T>::CH : n, FULL || i < rows);
    store_row<T, VEC>(og, FULL || i < steps ? pack<T>(mul(dx, factor[i])) : 0u, FULL ? Lane<T>::CH : n, FULL || i < rows);
  }
}

template <typename T, int FORM, int VEC>
__global__ void __launch_bounds__(32 * (kWorkers + 2), 1)
recurrence_grad_kernel(View grad, View x, View gate, Shape shape, const float* states, const float* grad_final,
                       T* grad_x, T* grad_gate, float* grad_initial) {
  using V = LaneV<T>;
  constexpr int CH = Lane<T>::CH;
  extern __shared__ __align__(128) unsigned s_raw[];     // [stages][workers][gate, x, grad][kSteps][32]
  __shared__ Map<V> s_map[2][kWorkers][32];              // (A, H) of the pieces; then H: the state before a piece
  __shared__ V s_back[2][kWorkers][32];                  // M; then what comes back behind a piece
  __shared__ Messages<V> s_box;                          // (A, M) of the CTAs' blocks
  if (threadIdx.x < 4) mbar_init(&s_box.bar[threadIdx.x], 1);
  if (threadIdx.x == 0) s_box.lost = 0;
  if (shape.log2_ranks > 0) cluster_arrive();
  dep_wait();
  dep_launch();
  const Place<T> me(shape);
  const int len = me.len, time = shape.time, channels = shape.channels, threads = blockDim.x;
  const long long row = (long long)me.b * channels + me.c;
  if (shape.log2_ranks > 0) cluster_wait();
  else __syncthreads();
  // round k takes the blocks from (rounds - 1 - k) * ranks on

  if (me.warp == me.workers) {
    each_round(me.rounds, [&](auto parity, int k) {
      constexpr int P = decltype(parity)::value;
      const int to = receivers(s_box, me, k, shape.withheld);
      join<kMapsIn + P>(threads);
      Map<V> map;
      both(map.A, 1.0f);
      both(map.H, 0.0f);
#pragma unroll 1
      for (int w0 = (me.workers - 1) & ~3; w0 >= 0; w0 -= 4) {
        V A[4], M[4];
#pragma unroll
        for (int w = 0; w < 4; ++w)
          if (w0 + w < me.workers) {
            A[w] = s_map[P][w0 + w][me.lane].A;
            M[w] = s_back[P][w0 + w][me.lane];
          }
#pragma unroll
        for (int w = 3; w >= 0; --w)
          if (w0 + w < me.workers) {
            map.H = after(map.H, A[w], M[w]);
            map.A = mul(map.A, A[w]);
          }
      }
      send(s_box, me, k, map, to);
    });
  } else if (me.warp > me.workers) {
    const int kept = (time + kBlock - 1) / kBlock;
    V carry;
    load_state<CH>(carry, grad_final + row, grad_final ? me.n : 0);
    bool lost = false;
    auto before = [&](int k) {         // the state kept before the CTA's block of round k
      const int block = (me.rounds - 1 - k) * me.ranks + me.rank;
      V h;
      load_state<CH>(h, states + ((long long)me.b * kept + block) * channels + me.c, k < me.rounds && block < kept ? me.n : 0);
      return h;
    };
    V next = before(0);
    each_round(me.rounds, [&](auto parity, int k) {
      constexpr int P = decltype(parity)::value;
      V h = next;
      next = before(k + 1);
      join<kMapsIn + P>(threads);
#pragma unroll 1
      for (int w0 = 0; w0 < me.workers; w0 += 4) {
        Map<V> q[4];
#pragma unroll
        for (int w = 0; w < 4; ++w)
          if (w0 + w < me.workers) q[w] = s_map[P][w0 + w][me.lane];
#pragma unroll
        for (int w = 0; w < 4; ++w)
          if (w0 + w < me.workers) {
            s_map[P][w0 + w][me.lane].H = h;
            h = after(h, q[w].A, q[w].H);
          }
      }
      V m = receive<FORM, true>(s_box, me, k, carry, lost, shape.wait_ns);
#pragma unroll 1
      for (int w0 = (me.workers - 1) & ~3; w0 >= 0; w0 -= 4) {
        V A[4], M[4];
#pragma unroll
        for (int w = 0; w < 4; ++w)
          if (w0 + w < me.workers) {
            A[w] = s_map[P][w0 + w][me.lane].A;
            M[w] = s_back[P][w0 + w][me.lane];
          }
#pragma unroll
        for (int w = 3; w >= 0; --w)
          if (w0 + w < me.workers) {
            s_back[P][w0 + w][me.lane] = m;
            m = after(m, A[w], M[w]);
          }
      }
      arrive<kStatesIn + P>(threads - 32);
    });
    if (grad_initial && len == 0 && me.rank == 0) store_state<CH>(grad_initial + row, carry, me.n);
  } else {
    const Gates<T, FORM> gates(shape.lowest_gate);
    const int at = me.rank * kBlock + me.warp * kSteps, last = (me.rounds - 1) * me.stride + at;
    // from this round on the pieces are whole
    const int whole = me.whole && len >= at + kSteps ? me.rounds - 1 - (len - at - kSteps) / me.stride : me.rounds;
    const Ring<VEC> ring{s_raw + me.warp * (3 * kSteps * pitch(VEC)), me.workers * (3 * kSteps * pitch(VEC))};
    const unsigned odd = VEC == 0 ? Words<VEC>::odd_rows(gate, me.b, 0) | Words<VEC>::odd_rows(x, me.b, 1) |
                                        Words<VEC>::odd_rows(grad, me.b, 2)
                                  : 0u;
    const bool graded = grad.p != nullptr;
    Reader<T, VEC> read_gate(gate, me, last), read_x(x, me, last), read_grad(grad, me, last);
    auto ask = [&](int k, unsigned (*to)[kSteps][pitch(VEC)]) {
      if (k < me.rounds) {
        const int t0 = last - k * me.stride;
        read_gate.next(to[0], gate, me, k >= whole, t0, -me.stride, channels);
        read_x.next(to[1], x, me, k >= whole, t0, -me.stride, channels);
        if (graded) read_grad.next(to[2], grad, me, k >= whole, t0, -me.stride, channels);
      }
      copies_commit();
    };
    int taken = 0, given = 0;          // stages
    auto take = [&](auto parity, int k) {
      constexpr int P = decltype(parity)::value;
      copies_wait_but_one();
      __syncwarp();
      V M;
      unsigned(*w)[kSteps][pitch(VEC)] = ring.at(taken);
      const Words<VEC> words{w, odd, me.lane, graded};
      s_map[P][me.warp][me.lane] =
          k >= whole ? piece_maps<T, FORM, true>(gates, words, M, kSteps)
                     : piece_maps<T, FORM, false>(gates, words, M, len - (last - k * me.stride));
      s_back[P][me.warp][me.lane] = M;
      __syncwarp();
      arrive<kMapsIn + P>(threads);
      taken = taken + 1 == kStages ? 0 : taken + 1;
    };
    long long o = ((long long)me.b * time + last) * channels + me.c;
    auto give = [&](auto parity, int k) {
      constexpr int P = decltype(parity)::value;
      join<kStatesIn + P>(threads - 32);
      const V h = s_map[P][me.warp][me.lane].H;
      V m = s_back[P][me.warp][me.lane];
      unsigned(*w)[kSteps][pitch(VEC)] = ring.at(given);
      if (k >= whole) {
        piece_gradients<T, FORM, VEC, true>(gates, Words<VEC>{w, odd, me.lane, graded}, h, m, grad_x + o, grad_gate + o, channels,
                                                 CH, kSteps, kSteps);
      } else {
        const int t0 = last - k * me.stride;
        piece_gradients<T, FORM, VEC, false>(gates, Words<VEC>{w, odd, me.lane, graded}, h, m, grad_x + o, grad_gate + o,
                                                  channels, me.n, len - t0, time - t0);
      }
      o -= (long long)me.stride * channels;
      if (at == 0 && k + 1 == me.rounds && grad_initial) store_state<CH>(grad_initial + row, m, me.n);
      __syncwarp();
      ask(k + kStages, w);
      given = given + 1 == kStages ? 0 : given + 1;
    };
    // past the sequence's last round
    for (long long t0 = (long long)me.rounds * me.stride + at; t0 < time; t0 += me.stride)
      for (int i = 0; i < kSteps; ++i)
        if (me.n > 0 && t0 + i < time) {
          const long long o = ((long long)me.b * time + t0 + i) * channels + me.c;
          store_word<T, VEC != 0>(grad_x + o, 0u, me.n);
          store_word<T, VEC != 0>(grad_gate + o, 0u, me.n);
        }
    if (me.rounds > 0) {
      ask(0, ring.at(0));
      ask(1, ring.at(1));
      take(std::integral_constant<int, 0>(), 0);
      ask(2, ring.at(2));
    }
    each_round(me.rounds, [&](auto parity, int k) {
      if (k + 1 < me.rounds) take(std::integral_constant<int, 1 - decltype(parity)::value>(), k + 1);
      give(parity, k);
    });
  }
  if (shape.log2_ranks > 0) leave(s_box);
}

template <typename T, int FORM, bool VEC>
__global__ void __launch_bounds__(128)
recurrence_grad_short_kernel(View grad, View x, View gate, Shape shape, const float* states, const float* grad_final,
                             T* grad_x, T* grad_gate, float* grad_initial) {
  using V = LaneV<T>;
  constexpr int CH = Lane<T>::CH, STEPS = kSteps;
  dep_wait();
  dep_launch();
  const Gates<T, FORM> gates(shape.lowest_gate);
  const Word me(shape, T());
  if (me.n <= 0) return;
  const long long row = (long long)me.b * shape.channels + me.c;
  V h, m;
  load_state<CH>(h, states + row, me.len > 0 ? me.n : 0);
  load_state<CH>(m, grad_final + row, grad_final ? me.n : 0);
  unsigned w[3][STEPS];
  load_words<T, VEC>(w[0], gate, me);
  load_words<T, VEC>(w[1], x, me);
#pragma unroll
  for (int i = 0; i < STEPS; ++i) w[2][i] = 0;
  if (grad.p) load_words<T, VEC>(w[2], grad, me);
  const long long o = (long long)me.b * shape.time * shape.channels + me.c;
  piece_gradients<T, FORM, VEC ? 1 : -1, false>(gates, WordsHeld{w}, h, m, grad_x + o, grad_gate + o, shape.channels, me.n,
                                                me.len, shape.time);
  if (grad_initial) store_state<CH>(grad_initial + row, m, me.n);
}

// ---------------------------------------------------------------------------

// CTAs that share a sequence (a cluster), as a logarithm: what costs the least in
// rounds of blocks, with two more for a CTA's start, over the waves of clusters that
// are resident at a time.  (Of 8 CTAs fewer clusters fit than the SMs' number lets
// expect: 16 of them took two waves.)  The bits do not depend on it.  (1 x 65,536 x 256 in bf16 with 1, 2, 4, 8 CTAs,
// when this was chosen: 563, 311, 164, 92 us; with 8 now 84.)
int choose_ranks(const void* kernel, cudaLaunchConfig_t cfg, long long sequences, int time) {
  static std::mutex mu;
  static std::map<std::tuple<const void*, int, int, unsigned, size_t>, int> cache;
  int dev = 0;
  cudaGetDevice(&dev);
  int best = 0;
  long long least = -1;
  for (int l = 0; (1 << l) <= kMaxCluster && (l == 0 || (kBlock << (l - 1)) < time); ++l) {
    int clusters = 0;
    {
      std::lock_guard<std::mutex> lk(mu);
      int& known = cache[{kernel, dev, l, cfg.blockDim.x, cfg.dynamicSmemBytes}];
      if (known == 0) {
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 1u << l;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3(1u << l);
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&known, kernel, &cfg) != cudaSuccess || known <= 0) {
          cudaGetLastError();
          known = -1;
        }
      }
      clusters = known;
    }
    if (clusters <= 0) continue;
    const long long waves = (sequences + clusters - 1) / clusters;
    const long long rounds = ((long long)time + (kBlock << l) - 1) / (kBlock << l);
    const long long cost = waves * (rounds + 2);
    if (least < 0 || cost < least) {
      least = cost;
      best = l;
    }
  }
  return best;
}

// A launch over channel tiles and sequences, a thread a word for single pieces.
template <typename T, int OPERANDS, typename K, typename ARGS>
int launch_recurrence(const char* name, K* short_kernel, K* kernel, int row_words, int batch, Shape shape, cudaStream_t s,
                      ARGS with) {
  const int words = (shape.channels + Lane<T>::CH - 1) / Lane<T>::CH;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (shape.time <= kSteps) {
    cfg.gridDim = dim3((unsigned)((words + 127) / 128), (unsigned)batch);
    cfg.blockDim = dim3(128);
    launch_begin(name, s);
    const cudaError_t e = with(cfg, short_kernel, shape);
    launch_end(s);
    return e == cudaSuccess ? DET_OK : cuda_fail(e, name);
  }
  const int workers = std::min(kWorkers, (shape.time + kSteps - 1) / kSteps);
  const long long tiles = (words + 31) / 32;
  cfg.blockDim = dim3(32 * (workers + 2));
  const size_t round_bytes = (size_t)workers * OPERANDS * kSteps * row_words * 4;
  cfg.dynamicSmemBytes = std::min<long long>(kStages, (shape.time + kBlock - 1) / kBlock) * round_bytes;
  // allowed for the largest at once: a small ring may pass the default limit too, with the static arrays
  cudaError_t e = ensure_dyn_smem((const void*)kernel, (size_t)kStages * kBlock * OPERANDS * row_words * 4);
  if (e != cudaSuccess) return cuda_fail(e, name);
  shape.log2_ranks = choose_ranks((const void*)kernel, cfg, tiles * batch, shape.time);
  const int ranks = 1 << shape.log2_ranks;
  cfg.gridDim = dim3((unsigned)tiles * ranks, (unsigned)batch);
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ranks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  if (ranks > 1) cfg.numAttrs = 2;
  launch_begin(name, s);
  e = with(cfg, kernel, shape);
  launch_end(s);
  return e == cudaSuccess ? DET_OK : cuda_fail(e, name);
}

template <typename T, int FORM, int VEC>
int forward(const View& x, const View& gate, const Shape& shape, int batch, const float* initial, void* out,
            float* final_out, float* states, cudaStream_t s) {
  return launch_recurrence<T, 2>("det_linear_recurrence", recurrence_short_kernel<T, FORM, VEC != 0>,
                                 recurrence_kernel<T, FORM, VEC>, pitch(VEC), batch, shape, s,
                                 [&](const cudaLaunchConfig_t& cfg, auto* kernel, const Shape& sh) {
                                   return cudaLaunchKernelEx(&cfg, kernel, x, gate, sh, initial, static_cast<T*>(out),
                                                             final_out, states);
                                 });
}
template <typename T, int FORM, int VEC>
int backward(const View& grad, const View& x, const View& gate, const Shape& shape, int batch, const float* states,
             const float* grad_final, void* grad_x, void* grad_gate, float* grad_initial, cudaStream_t s) {
  return launch_recurrence<T, 3>("det_linear_recurrence_backward", recurrence_grad_short_kernel<T, FORM, VEC != 0>,
                                 recurrence_grad_kernel<T, FORM, VEC>, pitch(VEC), batch, shape, s,
                                 [&](const cudaLaunchConfig_t& cfg, auto* kernel, const Shape& sh) {
                                   return cudaLaunchKernelEx(&cfg, kernel, grad, x, gate, sh, states, grad_final,
                                                             static_cast<T*>(grad_x), static_cast<T*>(grad_gate),
                                                             grad_initial);
                                 });
}

// How rows are read: 2 where all start on 16 bytes and are whole vectors, 1 where all
// start on a word and are whole words, 0 else.  (8 x 4,096 steps in bf16: 2,048 channels 75 us, 2,046 116, 2,047 178.)
int reading(int dtype, std::initializer_list<const void*> pointers, std::initializer_list<int64_t> strides) {
  uintptr_t all = 0;
  for (const void* p : pointers) all |= reinterpret_cast<uintptr_t>(p);
  for (const int64_t st : strides) all |= (uintptr_t)st * model_elem_size(dtype);
  return all % 16 == 0 ? 2 : all % 4 == 0 ? 1 : 0;
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

// Test hook state (det_test_hooks.h): host-side, read when a call is enqueued.
int g_withheld = -1;
unsigned long long g_wait_ns = kWaitNs;

}  // namespace
}  // namespace det

using namespace det;

extern "C" int det_test_recurrence_withhold(int64_t round, uint64_t timeout_ns) {
  if (round >= 0 && (round > INT32_MAX || timeout_ns == 0 || timeout_ns > kWaitNs)) return DET_ERR_INVALID_ARG;
  g_withheld = round < 0 ? -1 : (int)round;
  g_wait_ns = round < 0 ? kWaitNs : timeout_ns;
  return DET_OK;
}

#define DET_RECURRENCE_FORM(fn, T, VEC, ...) \
  (form == DET_GATE_DECAY ? fn<T, DET_GATE_DECAY, VEC>(__VA_ARGS__) : fn<T, DET_GATE_SIGMOID, VEC>(__VA_ARGS__))
#define DET_RECURRENCE_16(fn, T, ...)                                       \
  (how == 2   ? DET_RECURRENCE_FORM(fn, T, 2, __VA_ARGS__)                  \
   : how == 1 ? DET_RECURRENCE_FORM(fn, T, 1, __VA_ARGS__)                  \
              : DET_RECURRENCE_FORM(fn, T, 0, __VA_ARGS__))
#define DET_RECURRENCE_PICK(fn, ...)                                         \
  (dtype == DET_F32    ? (how == 2 ? DET_RECURRENCE_FORM(fn, float, 2, __VA_ARGS__)  \
                                   : DET_RECURRENCE_FORM(fn, float, 1, __VA_ARGS__)) \
   : dtype == DET_BF16 ? DET_RECURRENCE_16(fn, __nv_bfloat16, __VA_ARGS__)   \
                       : DET_RECURRENCE_16(fn, __half, __VA_ARGS__))

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
  const int how = reading(dtype, {x, gate, out}, {x_stride_b, x_stride_t, gate_stride_b, gate_stride_t, channels});
  const View vx = {x, x_stride_b, x_stride_t}, vg = {gate, gate_stride_b, gate_stride_t};
  const Shape shape = {(int)time, (int)channels, lengths, 0, kLowestGate, g_withheld, g_wait_ns};
  const cudaStream_t s = as_stream(stream);
  return DET_RECURRENCE_PICK(forward, vx, vg, shape, (int)batch, initial, out, final_out, states_out, s);
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
  const int how = reading(dtype, {grad, x, gate, grad_x, grad_gate},
                          {grad_stride_b, grad_stride_t, x_stride_b, x_stride_t, gate_stride_b, gate_stride_t, channels});
  const View vd = {grad, grad_stride_b, grad_stride_t}, vx = {x, x_stride_b, x_stride_t},
             vg = {gate, gate_stride_b, gate_stride_t};
  const Shape shape = {(int)time, (int)channels, lengths, 0, kLowestGate, g_withheld, g_wait_ns};
  const cudaStream_t s = as_stream(stream);
  return DET_RECURRENCE_PICK(backward, vd, vx, vg, shape, (int)batch, states, grad_final, grad_x, grad_gate, grad_initial, s);
}
