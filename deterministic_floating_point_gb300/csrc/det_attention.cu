// det_paged_attention (include/det_model.h): one new token of each sequence
// attends to its paged key-value cache.
//
// A sequence is cut into chunks whose size depends on its own length alone;
// a CTA takes the query heads that share one key-value head over one chunk,
// and a second kernel joins the chunks.  Inside a chunk warp w of 4 takes the
// 16-token tiles w, w + 4, ... with a running maximum (softmax statistics
// and the output are held in 32 bits), so the order of every addition is
// fixed by token index and a sequence's bits do not depend on its batch.
//
// Every key and value is read once for all heads that share it.  At the
// bandwidth of the memory the two products need a few percent of the tensor
// cores' rate, so they run on warp-level matrix instructions, transposed
// (tokens as rows, heads as columns): groups of 8 heads fill a tile exactly,
// each warp loads, multiplies and accumulates on its own without waiting for
// the others, and nothing is staged twice.
#include "det_model.cuh"

#include <algorithm>
#include <type_traits>

namespace det {
namespace {

constexpr int kMaxChunk = 1024;  // most tokens of a chunk

// Tokens of a chunk of a sequence of n tokens.  Short chunks let a short
// sequence use more SMs, long ones spend less on their start and on the join
// (32 sequences of 8,192 tokens, 8 kv heads of 128, as two tiles were kept:
// 183 us at 256, 179 at 512, 175 at 1,024; one of 1,000 tokens: 14, 18 and 24 us);
// a sequence of one chunk needs no join (128 of 500 tokens: 65 us at 256, 58 at 512).
constexpr int kOneChunk = 512, kShort = 1024, kMedium = 16384;
__host__ __device__ inline int chunk_tokens(int n) {
  return n <= kOneChunk ? kOneChunk : n <= kShort ? 256 : n <= kMedium ? 512 : kMaxChunk;
}
__host__ __device__ inline int chunk_count(int n) {
  const int c = chunk_tokens(n);
  return n <= 0 ? 1 : (n - 1) / c + 1;
}
// Most chunks of a sequence of at most n tokens.
inline int most_chunks(int n) {
  int most = chunk_count(n);
  if (n > kShort) most = std::max(most, chunk_count(kShort));
  if (n > kMedium) most = std::max(most, chunk_count(kMedium));
  return most;
}

// A warp's tiles of 16 tokens.  Its shared memory holds the keys of the tile it
// works on and of the next one, and the values of the one it works on: what
// hides the latency of loads and of a tile's chain of products and exponentials
// is the number of warps on an SM, so tiles are as short as the matrix
// instructions allow and no more is fetched ahead than keeps a warp going (32
// sequences of 8,192 tokens, 8 kv heads of 128 dims: 172 us; with the next
// tile's values too, and a CTA fewer on an SM, 177; three whole tiles 209; 128
// sequences of 500 tokens: 51 and 56 us).  With 64 dims and up to 8 heads the
// next tile's values cost no CTA: they are kept too (one sequence of 131,072
// tokens 58 us, without them 63; 128 of 512: 31 and 33).  Rows lie 16 bytes apart
// modulo 128, so that eight rows of a matrix load hit 32 banks.
template <int D> struct Tile {
  static constexpr int kWarps = 4;                  // of a CTA
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kTokens = 16;
  static constexpr int kRowBytes = D * 2;
  static constexpr int kPitch = kRowBytes + 16;
  static constexpr int kBytes = kTokens * kPitch;   // of the keys, and of the values
  // nt tiles of 8 heads: tiles whose values are kept, bytes of a warp and of a CTA
  __host__ __device__ static constexpr int values(int nt) { return D == 64 && nt == 1 ? 2 : 1; }
  __host__ __device__ static constexpr size_t warp_bytes(int nt) { return (2 + values(nt)) * kBytes; }
  __host__ __device__ static constexpr size_t smem_bytes(int nt) { return kWarps * warp_bytes(nt); }
  // the warps' outputs of 8 x nt heads when they are joined, in rows of floats
  // 4 apart modulo 32, so that a warp's writes hit 32 banks
  static constexpr int kOutPitch = D + 4;
  // CTAs on an SM that registers are kept for
  static constexpr int ctas(int nt) {
    return D == 64 ? (nt == 1 ? 6 : nt == 2 ? 4 : 3) : D == 128 ? (nt == 1 ? 4 : 3) : 2;
  }
  static constexpr size_t out_bytes(int nt) { return (size_t)kWarps * 8 * nt * kOutPitch * sizeof(float); }
};

struct AttnArgs {
  const void *q, *k, *v;
  long long q_sb, q_sh, k_sp, k_st, k_sh, v_sp, v_st, v_sh;
  const int32_t *table, *lengths;
  long long table_stride;
  int num_pages, page_size, limit;   // limit: most tokens of a sequence
  int heads, group, head_tiles, max_chunks;
  float scale;
  const void* bias;
  int bias_dtype;
  const int32_t* bounds;
  int num_bounds;
  float* part;      // [batch x heads][max_chunks][D]: the chunk's outputs, not yet divided
  float2* part_ml;  // [batch x heads][max_chunks]: maximum of the scores and sum
  void* out;
  float* lse;
};

__device__ __forceinline__ void cp_async_16(unsigned dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldmatrix_x4(unsigned (&r)[4], unsigned addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(unsigned (&r)[4], unsigned addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ unsigned movmatrix_trans(unsigned a) {
  unsigned d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// c (16 x 8, f32) += a (16 x 16, row major) * b (16 x 8, column major)
template <typename T>
__device__ __forceinline__ void mma_16816(float (&c)[4], const unsigned (&a)[4], unsigned b0, unsigned b1) {
  if constexpr (sizeof(T) == 2 && std::is_same<T, __half>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <typename T> __device__ __forceinline__ unsigned pack2(float lo, float hi) {
  const T a = from_f32<T>(lo), b = from_f32<T>(hi);
  return (unsigned)*reinterpret_cast<const unsigned short*>(&a) |
         ((unsigned)*reinterpret_cast<const unsigned short*>(&b) << 16);
}
template <typename T> __device__ __forceinline__ float2 unpack2(unsigned w) {
  const unsigned short lo = (unsigned short)w, hi = (unsigned short)(w >> 16);
  return make_float2(to_f32(*reinterpret_cast<const T*>(&lo)), to_f32(*reinterpret_cast<const T*>(&hi)));
}

// How the weights of the softmax, at most 1, enter the second product: as 16-bit
// parts that add up to 32-bit accuracy, three of bf16's 8 bits or two of f16's 11.
// f16's smallest normal value is 2^-14, so there they are scaled by 2^15 (exact; the
// outputs are divided by it at the end): held to 2^-22 of themselves from 2^-18 of
// the largest on, and to 2^-40 of the largest below.  A third part in bf16 costs 0 to
// 1.5% with up to 8 heads in a group and 4% with 16 (32 sequences of 8,192 tokens, 32
// heads on 8 x 128, 172.3 and 171.2 us; 32 of 32,768, 32 on 2, 202.4 and 194.4);
// with two, 1.6e-3 to 2.7e-3 of the outputs are not the exact results rounded,
// with three 3e-4 to 9e-4, and 2e-4 to 1.7e-3 if all is done in 32 bits.
template <typename T> constexpr int kWeightParts = std::is_same<T, __half>::value ? 2 : 3;
template <typename T> constexpr float kWeightScale = std::is_same<T, __half>::value ? 32768.0f : 1.0f;

// Number of bounds <= n.
__device__ __forceinline__ int bounds_at_most(const int32_t* bounds, int count, int n) {
  int lo = 0, hi = count;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (bounds[mid] <= n) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

// NT tiles of 8 heads per CTA.  Grid: (chunks, kv heads x head tiles, batch).
// A warp fetches its tiles itself, as groups of asynchronous copies.  Where
// pages hold whole blocks of 16 tokens a block's place is looked up once;
// otherwise every token's.
//
// Bound by the reads of keys and values (both kernels; fraction of the measured
// copy bandwidth): 32 sequences of 8,192 tokens, 8 kv heads of 128 dims for 32
// heads 173 us (91%), for 8 heads 166 us (95%); of 64 dims 97 us (81%), of 256 dims
// and 16 sequences 176 us (90%).  About 10 us of a call are its own: the CTAs'
// first tiles, the last ones, which do not fill the SMs, and the join (of 64 dims
// 128 sequences 351 us, 90%).  With short chunks a CTA's start and end (length,
// page, first tile and join of the warps, some 4 us against 1.3 us a tile) show:
// 128 sequences of 500 tokens 49 us (79%), 64 ragged ones of up to 8,191 tokens
// of 64 dims with the bias 60 us (70%).  Copying whole rows by the bulk engine was
// slower (a copy of 256 bytes every 20 cycles an SM: 296 us for 32 x 8,192).
template <typename T, int D, int NT>
__global__ void __launch_bounds__(Tile<D>::kThreads, Tile<D>::ctas(NT)) attention_chunks_kernel(const __grid_constant__ AttnArgs a) {
  using L = Tile<D>;
  constexpr int W = L::kWarps, kValues = L::values(NT);
  constexpr size_t kWarpBytes = L::warp_bytes(NT), kSmem = L::smem_bytes(NT);
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ long long sh_place[kMaxChunk / 16][2];   // of a block of 16 tokens: its keys and values; -1: skipped
  __shared__ float sh_m[W][8 * NT], sh_l[W][8 * NT];

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int chunk = blockIdx.x, b = blockIdx.z;
  const int g = blockIdx.y / a.head_tiles, h0 = (blockIdx.y % a.head_tiles) * 8 * NT;   // first head in the group
  const bool blocks = a.page_size % 16 == 0;   // chunks begin at multiples of 16
  const int32_t* table = a.table + b * a.table_stride;
  dep_wait();     // launched early: all loads come after, and none is a read-only one, which need not
  dep_launch();   // the join's CTAs come as this kernel's run out
  // A warp looks up its own blocks, a lane one.  The length, the queries and
  // the page, which depends on the length through the chunk's size, are read
  // at once: the page for the size that the longest sequence would have, and
  // again where that was wrong (never in the first chunk).
  static_assert(kMaxChunk / 16 <= 32 * W, "a lane places one block");
  const int block = warp + W * lane;
  const int guess = chunk * chunk_tokens(a.limit) + 16 * block;
  const int length = a.lengths[b];
  int page = -1;
  if (blocks && lane < kMaxChunk / 16 / W && guess < a.limit) page = table[guess / a.page_size];

  // the queries as B operands: column = head (lane / 4), rows = dims
  unsigned qf[D / 16][NT][2];
  const bool words = ((reinterpret_cast<uintptr_t>(a.q) | (a.q_sb | a.q_sh) * 2) & 3) == 0;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int h = h0 + nt * 8 + lane / 4;
    const T* q = static_cast<const T*>(a.q) + b * a.q_sb + (long long)(g * a.group + h) * a.q_sh + 2 * (lane & 3);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        unsigned w = 0;
        if (h < a.group) {
          const unsigned short* p = reinterpret_cast<const unsigned short*>(q + ks * 16 + j * 8);
          w = words ? *reinterpret_cast<const unsigned*>(p) : (unsigned)p[0] | ((unsigned)p[1] << 16);
        }
        qf[ks][nt][j] = w;
      }
  }

  const int n = min(max(length, 0), a.limit);
  const int chunks = chunk_count(n);
  if (chunk >= chunks) return;
  const int size = chunk_tokens(n);
  const int t0 = chunk * size, t1 = min(n, t0 + size);
  const int p0 = t0 / a.page_size;
  int* sh_page = reinterpret_cast<int*>(smem + kSmem);   // of the chunk's pages, where blocks are not whole
  if (blocks) {
    const int j = t0 + 16 * block;
    if (j < t1) {
      const int pj = j / a.page_size, slot = j - pj * a.page_size;
      if (j != guess) page = table[pj];
      const bool valid = page >= 0 && page < a.num_pages;
      sh_place[block][0] = valid ? page * a.k_sp + slot * a.k_st : -1;
      sh_place[block][1] = valid ? page * a.v_sp + slot * a.v_st : -1;
    }
    __syncwarp();
  } else {
    const int pages = t1 > t0 ? (t1 - 1) / a.page_size - p0 + 1 : 0;
    for (int i = threadIdx.x; i < pages; i += L::kThreads) {
      const int p = table[p0 + i];
      sh_page[i] = p >= 0 && p < a.num_pages ? p : -1;
    }
    __syncthreads();
  }

  const T* kbase = static_cast<const T*>(a.k) + g * a.k_sh;
  const T* vbase = static_cast<const T*>(a.v) + g * a.v_sh;
  const unsigned ring = smem_u32(smem + warp * kWarpBytes);   // keys, keys, values
  const int tiles = (t1 - t0 + L::kTokens - 1) / L::kTokens;
  const int mine = (tiles - warp + W - 1) / W;   // tiles of this warp

  // a lane copies 16 bytes of every (32 / C)-th row
  constexpr int C = D / 8, kRows = 32 / C;
  const int row0 = lane / C, col = lane % C;
  // The rows of the warp's tile `it`, of the keys or the values; a bit for
  // each token that is not skipped.  Nothing is read for a skipped token: its
  // row becomes 0, so that 0 * value is 0.
  auto fetch = [&](int it, int which, unsigned to) -> unsigned {
    const int tile = it * W + warp, j0 = t0 + 16 * tile;
    const T* base = (which ? vbase : kbase) + col * 8;
    const long long st = which ? a.v_st : a.k_st;
    const unsigned dst = to + row0 * L::kPitch + col * 16;
    unsigned mask = 0;
    long long from = 0;   // of the block, or of the lane's token (lane % 16)
    if (blocks) {
      from = sh_place[tile][which];
      mask = from < 0 ? 0u : j0 + 16 <= t1 ? 0xffffu : (1u << (t1 - j0)) - 1;
      if (mask == 0xffffu) {
        const T* src = base + from + row0 * st;
#pragma unroll
        for (int i = 0; i < 16 / kRows; ++i) cp_async_16(dst + i * kRows * L::kPitch, src + i * (kRows * st));
        return mask;
      }
    } else {
      const int j = j0 + (lane & 15);
      int page = -1;
      if (j < t1) {
        const int pj = j / a.page_size;
        page = sh_page[pj - p0];
        from = page * (which ? a.v_sp : a.k_sp) + (j - pj * a.page_size) * st;
      }
      mask = __ballot_sync(0xffffffffu, page >= 0) & 0xffffu;
    }
#pragma unroll
    for (int i = 0; i < 16 / kRows; ++i) {
      const int row = i * kRows + row0;
      const long long at = blocks ? from + row * st : __shfl_sync(0xffffffffu, from, row);
      if ((mask >> row) & 1) cp_async_16(dst + i * kRows * L::kPitch, base + at);
      else asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(dst + i * kRows * L::kPitch), "r"(0u) : "memory");
    }
    return mask;
  };

  float o[D / 16][NT][4];
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][nt][j] = 0.0f;
  float m[NT][2], l[NT][2];   // of heads 2 (lane % 4) and + 1; l of this lane's tokens
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      m[nt][j] = kNegInf;
      l[nt][j] = 0.0f;
    }

  unsigned next_mask = mine > 0 ? fetch(0, 0, ring) : 0u;
  cp_async_commit();
  if (kValues == 2 && mine > 0) fetch(0, 1, ring + 2 * L::kBytes);
  if (kValues == 2) cp_async_commit();
  // with a bias: the distance from which on the last bucket holds, and its values
  int far = 0;
  float far_bias[NT][2];
  if (a.bias) {
    far = a.num_bounds > 0 ? a.bounds[a.num_bounds - 1] : 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int h = h0 + nt * 8 + 2 * (lane & 3) + j;
        far_bias[nt][j] =
            h < a.group ? load_as_f32(a.bias, (long long)a.num_bounds * a.heads + g * a.group + h, a.bias_dtype) : 0.0f;
      }
  }
  for (int it = 0; it < mine; ++it) {
    const unsigned ks = ring + (it & 1) * L::kBytes;
    const unsigned vs = ring + (2 + (it & (kValues - 1))) * L::kBytes;
    const unsigned mask = next_mask >> (lane >> 2);   // of this lane's tokens: bits 0 and 8
    if (kValues == 1) {
      fetch(it, 1, vs);
      cp_async_commit();
    }
    if (it + 1 < mine) next_mask = fetch(it + 1, 0, ring + ((it + 1) & 1) * L::kBytes);
    cp_async_commit();
    if (kValues == 2) {
      if (it + 1 < mine) fetch(it + 1, 1, ring + (2 + ((it + 1) & 1)) * L::kBytes);
      cp_async_commit();
    }
    cp_async_wait<1 + kValues>();   // this tile's keys
    __syncwarp();
    float s[NT][4] = {};
    {
      const unsigned row = ks + (lane & 15) * L::kPitch + ((lane >> 4) << 4);
      // two chains, of the even and the odd sixteens of the dims
      float odd[NT][4] = {};
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        unsigned af[4];
        ldmatrix_x4(af, row + 32 * k);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_16816<T>(k & 1 ? odd[nt] : s[nt], af, qf[k][nt][0], qf[k][nt][1]);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[nt][j] += odd[nt][j];
    }
    // the scores, in units of the natural logarithm, since in units of log 2 a
    // bias of the type's lowest value would be -inf; masked tokens to -inf
    const int first = t0 + (it * W + warp) * L::kTokens;
    if (a.bias && n - (first + L::kTokens) >= far) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[nt][j] = fmaf(s[nt][j], a.scale, far_bias[nt][j & 1]);
    } else {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const void* row = nullptr;
        if (a.bias) {
          const int distance = n - 1 - (first + r * 8 + (lane >> 2));
          row = static_cast<const char*>(a.bias) + (long long)bounds_at_most(a.bounds, a.num_bounds, distance) *
                                                       a.heads * (a.bias_dtype == DET_F32 ? 4 : 2);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int h = h0 + nt * 8 + 2 * (lane & 3) + j;
            const float bias = a.bias && h < a.group ? load_as_f32(row, g * a.group + h, a.bias_dtype) : 0.0f;
            s[nt][2 * r + j] = fmaf(s[nt][2 * r + j], a.scale, bias);
          }
      }
    }
    bool raise = false;
    float fresh[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (!(mask & 1)) s[nt][j] = kNegInf;
        if (!(mask & 256)) s[nt][2 + j] = kNegInf;
        float mx = fmaxf(s[nt][j], s[nt][2 + j]);
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        fresh[nt][j] = fmaxf(m[nt][j], mx);
        raise |= fresh[nt][j] > m[nt][j];
      }
    }
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          // nothing was added while the maximum was -inf: any factor will do
          const float f = m[nt][j] == kNegInf ? 1.0f : exp_approx(m[nt][j] - fresh[nt][j]);
          m[nt][j] = fresh[nt][j];
          l[nt][j] *= f;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            o[i][nt][j] *= f;
            o[i][nt][2 + j] *= f;
          }
        }
    }
    // the weights as B operands (column = head), in parts: the weight rounded to
    // 16 bits, and what the rounding left rounded again
    unsigned pw[kWeightParts<T>][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float(&p)[4] = s[nt];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float base = m[nt][j] == kNegInf ? 0.0f : m[nt][j];
        p[j] = exp_approx(p[j] - base);
        p[2 + j] = exp_approx(p[2 + j] - base);
        l[nt][j] += p[j] + p[2 + j];
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float2 left = make_float2(p[2 * half] * kWeightScale<T>, p[2 * half + 1] * kWeightScale<T>);
#pragma unroll
        for (int part = 0; part < kWeightParts<T>; ++part) {
          const unsigned w = pack2<T>(left.x, left.y);
          const float2 r = unpack2<T>(w);
          left = make_float2(left.x - r.x, left.y - r.y);   // exact
          pw[part][nt][half] = movmatrix_trans(w);
        }
      }
    }
    cp_async_wait<kValues>();   // and its values
    __syncwarp();
    {
      const unsigned row = vs + ((lane & 7) + ((lane >> 4) & 1) * 8) * L::kPitch + (((lane >> 3) & 1) << 4);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        unsigned af[4];
        ldmatrix_x4_trans(af, row + 32 * i);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int part = 0; part < kWeightParts<T>; ++part)
            mma_16816<T>(o[i][nt], af, pw[part][nt][0], pw[part][nt][1]);
      }
    }
    __syncwarp();   // its keys and values have been read
  }
  cp_async_wait<0>();

  // join the warps, in order
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], d);
      if (lane < 4) {
        sh_m[warp][nt * 8 + 2 * lane + j] = m[nt][j];
        sh_l[warp][nt * 8 + 2 * lane + j] = l[nt][j];
      }
    }
  __syncthreads();
  constexpr int kPitch = L::kOutPitch;
  float* sh_o = reinterpret_cast<float*>(smem);   // in the place of the tiles
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int col = nt * 8 + 2 * (lane & 3) + j;
      float top = kNegInf;
      for (int w = 0; w < W; ++w) top = fmaxf(top, sh_m[w][col]);
      const float f = (m[nt][j] == kNegInf ? 1.0f : exp_approx(m[nt][j] - top)) * (1.0f / kWeightScale<T>);
      float* dst = sh_o + (size_t)(warp * 8 * NT + col) * kPitch + (lane >> 2);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        dst[i * 16] = o[i][nt][j] * f;
        dst[i * 16 + 8] = o[i][nt][2 + j] * f;
      }
    }
  __syncthreads();
  for (int at = threadIdx.x; at < 8 * NT * D; at += L::kThreads) {
    const int col = at / D, d = at % D;
    if (h0 + col >= a.group) break;
    float top = kNegInf, sum = 0.0f, v = 0.0f;
    for (int w = 0; w < W; ++w) top = fmaxf(top, sh_m[w][col]);
    for (int w = 0; w < W; ++w) {
      const float mw = sh_m[w][col];
      sum += mw == kNegInf ? sh_l[w][col] : sh_l[w][col] * exp_approx(mw - top);
      v += sh_o[(size_t)(w * 8 * NT + col) * kPitch + d];
    }
    const long long bh = (long long)b * a.heads + g * a.group + h0 + col;
    if (chunks == 1) {
      static_cast<T*>(a.out)[bh * D + d] = from_f32<T>(top == kNegInf && sum == 0.0f ? 0.0f : v / sum);
      if (a.lse && d == 0) a.lse[bh] = top == kNegInf && sum == 0.0f ? kNegInf : top + logf(sum);
    } else {
      a.part[(bh * a.max_chunks + chunk) * D + d] = v;
      if (d == 0) a.part_ml[bh * a.max_chunks + chunk] = make_float2(top, sum);
    }
  }
}

// The chunks of the heads of one sequence joined, in the order of the chunks:
// of a few chunks a warp joins a head (a CTA 8 heads, and CTAs beyond the heads
// have nothing to do); of more a CTA joins one, warp w of 8 the chunks w, w + 8,
// ..., and the warps are added in order.  Its CTAs are on the SMs before the
// first kernel ends.  A dependent chain of reads of L2 and the sum; what a CTA a
// head costs is their number (256 sequences of up to 2,000 tokens, 32 heads of 64
// dims, both kernels: 69 us, with a warp a head 58; 8 of 8,192, 128 dims: 49 and 50;
// since lengths are read after the wait, 1 to 2 us more).
constexpr int kJoinWarps = 8;
template <typename T, int D>
__global__ void __launch_bounds__(32 * kJoinWarps) attention_join_kernel(const __grid_constant__ AttnArgs a) {
  constexpr int E = D / 32;
  constexpr int kAhead = 8;                      // chunks in flight
  constexpr int kWarpJoin = D <= 128 ? 16 : 8;   // most chunks that a warp joins
  __shared__ float sh_top[kJoinWarps], sh_sum[kJoinWarps];
  __shared__ float sh_o[kJoinWarps][D];
  const int b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  dep_wait();   // launched early: nothing is read before, the lengths neither
  dep_launch();
  const int chunks = chunk_count(min(max(a.lengths[b], 0), a.limit));
  const bool few = chunks <= kWarpJoin;
  if (chunks == 1 || (few && blockIdx.x * kJoinWarps >= a.heads)) return;   // 1: already in place
  const int h = few ? blockIdx.x * kJoinWarps + warp : blockIdx.x;
  const long long bh = (long long)b * a.heads + h;
  const float2* ml = a.part_ml + bh * a.max_chunks;
  const float* part = a.part + bh * a.max_chunks * D + lane;
  float v[E];
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] = 0.0f;
  float top = kNegInf, sum = 0.0f;

  if (few) {
    if (h >= a.heads) return;
    const float2 x = lane < chunks ? ml[lane] : make_float2(kNegInf, 0.0f);   // a lane's chunk
    float f = 0.0f;
#pragma unroll
    for (int c0 = 0; c0 < kWarpJoin; c0 += kAhead) {
      if (c0 >= chunks) break;
      float y[kAhead][E];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e) y[k][e] = c0 + k < chunks ? part[(c0 + k) * D + e * 32] : 0.0f;
      if (c0 == 0) {
        top = x.x;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        f = x.x == kNegInf ? 1.0f : exp_approx(x.x - top);   // a chunk without a score adds 0
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const float fk = __shfl_sync(0xffffffffu, f, c0 + k);
        sum = fmaf(__shfl_sync(0xffffffffu, x.y, c0 + k), fk, sum);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = fmaf(y[k][e], fk, v[e]);
      }
    }
    const bool none = top == kNegInf && sum == 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) static_cast<T*>(a.out)[bh * D + e * 32 + lane] = from_f32<T>(none ? 0.0f : v[e] / sum);
    if (a.lse && lane == 0) a.lse[bh] = none ? kNegInf : top + logf(sum);
    return;
  }

  float2 x[kAhead];
  float y[kAhead][E];
  auto load = [&](int c0) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int c = c0 + k * kJoinWarps;
      x[k] = c < chunks ? ml[c] : make_float2(kNegInf, 0.0f);
#pragma unroll
      for (int e = 0; e < E; ++e) y[k][e] = c < chunks ? part[(long long)c * D + e * 32] : 0.0f;
    }
  };
  load(warp);
  for (int c = threadIdx.x; c < chunks; c += 32 * kJoinWarps) top = fmaxf(top, ml[c].x);
  for (int d = 1; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  if (lane == 0) sh_top[warp] = top;
  __syncthreads();
  for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, sh_top[w]);
  for (int c0 = warp;;) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const float f = x[k].x == kNegInf ? 1.0f : exp_approx(x[k].x - top);
      sum = fmaf(x[k].y, f, sum);
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = fmaf(y[k][e], f, v[e]);
    }
    c0 += kAhead * kJoinWarps;
    if (c0 >= chunks) break;
    load(c0);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) sh_o[warp][e * 32 + lane] = v[e];
  if (lane == 0) sh_sum[warp] = sum;
  __syncthreads();
  sum = 0.0f;
  for (int w = 0; w < kJoinWarps; ++w) sum += sh_sum[w];
  const bool none = top == kNegInf && sum == 0.0f;
  for (int d = threadIdx.x; d < D; d += 32 * kJoinWarps) {
    float r = 0.0f;
    for (int w = 0; w < kJoinWarps; ++w) r += sh_o[w][d];
    static_cast<T*>(a.out)[bh * D + d] = from_f32<T>(none ? 0.0f : r / sum);
  }
  if (a.lse && threadIdx.x == 0) a.lse[bh] = none ? kNegInf : top + logf(sum);
}

template <typename T, int D, int NT>
int launch_attention(AttnArgs a, int batch, int kv_heads, cudaStream_t s) {
  a.head_tiles = (a.group + 8 * NT - 1) / (8 * NT);
  if ((long long)kv_heads * a.head_tiles > 65535) return DET_ERR_TOO_LARGE;
  const void* kernel = reinterpret_cast<const void*>(&attention_chunks_kernel<T, D, NT>);
  // the ids of a chunk's pages are kept where a page is not made of whole blocks
  const int longest = std::min(a.limit, kMaxChunk);
  const size_t pages = a.page_size % 16 ? (size_t)(longest / a.page_size + 2) * sizeof(int) : 0;
  const size_t smem = std::max(Tile<D>::smem_bytes(NT) + pages, Tile<D>::out_bytes(NT));
  if (const cudaError_t e = ensure_dyn_smem(kernel, smem)) return cuda_fail(e, "det_paged_attention");
  const dim3 grid((unsigned)a.max_chunks, (unsigned)(kv_heads * a.head_tiles), (unsigned)batch);
  launch_begin("det_paged_attention", s);
  const cudaError_t main = launch_dep(attention_chunks_kernel<T, D, NT>, grid, dim3(Tile<D>::kThreads), smem, s, a);
  launch_end(s);
  if (main != cudaSuccess) return cuda_fail(main, "det_paged_attention");
  if (a.max_chunks == 1) return DET_OK;
  launch_begin("det_paged_attention_join", s);
  const cudaError_t e = launch_dep(attention_join_kernel<T, D>, dim3((unsigned)a.heads, (unsigned)batch),
                                   dim3(32 * kJoinWarps), 0, s, a);
  launch_end(s);
  return e == cudaSuccess ? DET_OK : cuda_fail(e, "det_paged_attention_join");
}

// As many heads of a group in one CTA as the registers hold; larger groups
// take several CTAs, which read the cache again.
template <typename T>
int dispatch_attention(const AttnArgs& a, int head_dim, int batch, int kv_heads, cudaStream_t s) {
  if (head_dim == 64) {
    if (a.group <= 8) return launch_attention<T, 64, 1>(a, batch, kv_heads, s);
    if (a.group <= 16) return launch_attention<T, 64, 2>(a, batch, kv_heads, s);
    return launch_attention<T, 64, 4>(a, batch, kv_heads, s);
  }
  if (head_dim == 128) {
    if (a.group <= 8) return launch_attention<T, 128, 1>(a, batch, kv_heads, s);
    return launch_attention<T, 128, 2>(a, batch, kv_heads, s);
  }
  if (a.group <= 8) return launch_attention<T, 256, 1>(a, batch, kv_heads, s);
  return launch_attention<T, 256, 2>(a, batch, kv_heads, s);
}

}  // namespace
}  // namespace det

using namespace det;

extern "C" size_t det_paged_attention_workspace_bytes(int64_t batch, int64_t heads, int64_t head_dim,
                                                      int64_t max_len) {
  if (batch < 0 || heads < 0 || head_dim < 0 || max_len < 0 || max_len >= (1LL << 31)) return 0;
  const size_t chunks = (size_t)most_chunks((int)max_len);
  if (chunks == 1) return kHeaderBytes;
  return kHeaderBytes + align_up((size_t)batch * heads * chunks * sizeof(float2), 256) +
         (size_t)batch * heads * chunks * head_dim * sizeof(float);
}

extern "C" int det_paged_attention(const void* q, int64_t q_stride_b, int64_t q_stride_h, const void* k_cache,
                                   int64_t k_stride_page, int64_t k_stride_token, int64_t k_stride_head,
                                   const void* v_cache, int64_t v_stride_page, int64_t v_stride_token,
                                   int64_t v_stride_head, int64_t num_pages, int64_t page_size,
                                   const int32_t* block_table, int64_t table_stride, int64_t max_pages,
                                   const int32_t* lengths, int64_t batch, int64_t heads, int64_t kv_heads,
                                   int64_t head_dim, int dtype, float scale, const void* bias_table, int bias_dtype,
                                   const int32_t* bias_bounds, int64_t num_bounds, int64_t max_len, void* out,
                                   float* lse_out, void* workspace, size_t workspace_bytes, void* stream) {
  if (dtype != DET_BF16 && dtype != DET_F16) return DET_ERR_DTYPE;
  if (bias_table && !valid_model_dtype(bias_dtype)) return DET_ERR_DTYPE;
  if (batch < 0 || heads < 0 || kv_heads < 0 || num_pages < 0 || page_size < 1 || max_pages < 0 || max_len < 0 ||
      num_bounds < 0 || (head_dim != 64 && head_dim != 128 && head_dim != 256) ||
      (heads > 0 && (kv_heads == 0 || heads % kv_heads != 0)))
    return DET_ERR_INVALID_ARG;
  const int64_t most = (1LL << 31) - 1;
  if (batch > 65535 || kv_heads > 65535 || heads > most / 256 || num_pages > most || page_size > most ||
      max_len > most - kMaxChunk || max_pages > most || num_bounds > DET_MAX_BOUNDS)
    return DET_ERR_TOO_LARGE;
  if (batch == 0 || heads == 0) return DET_OK;
  if (!q || !out || !lengths || (max_pages > 0 && max_len > 0 && !block_table) ||
      (num_pages > 0 && (!k_cache || !v_cache)) || (bias_table && num_bounds > 0 && !bias_bounds))
    return DET_ERR_INVALID_ARG;
  const int64_t strides = k_stride_page | k_stride_token | k_stride_head | v_stride_page | v_stride_token | v_stride_head;
  if (reinterpret_cast<uintptr_t>(k_cache) % 16 || reinterpret_cast<uintptr_t>(v_cache) % 16 || (strides & 7) ||
      reinterpret_cast<uintptr_t>(q) % 2 || reinterpret_cast<uintptr_t>(out) % 2)
    return DET_ERR_INVALID_ARG;
  const int64_t capacity = max_pages > most / page_size ? most : max_pages * page_size;
  const int limit = (int)std::min(max_len, capacity);
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 ||
      workspace_bytes < det_paged_attention_workspace_bytes(batch, heads, head_dim, limit))
    return DET_ERR_WORKSPACE;
  AttnArgs a = {};
  a.q = q, a.k = k_cache, a.v = v_cache;
  a.q_sb = q_stride_b, a.q_sh = q_stride_h;
  a.k_sp = k_stride_page, a.k_st = k_stride_token, a.k_sh = k_stride_head;
  a.v_sp = v_stride_page, a.v_st = v_stride_token, a.v_sh = v_stride_head;
  a.table = block_table, a.lengths = lengths, a.table_stride = table_stride;
  a.num_pages = (int)num_pages, a.page_size = (int)page_size, a.limit = limit;
  a.heads = (int)heads, a.group = (int)(heads / kv_heads);
  a.max_chunks = most_chunks(limit);
  a.scale = scale;
  a.bias = bias_table, a.bias_dtype = bias_dtype, a.bounds = bias_bounds, a.num_bounds = (int)num_bounds;
  unsigned char* ws = static_cast<unsigned char*>(workspace) + kHeaderBytes;
  a.part_ml = reinterpret_cast<float2*>(ws);
  a.part = reinterpret_cast<float*>(ws + align_up((size_t)batch * heads * a.max_chunks * sizeof(float2), 256));
  a.out = out, a.lse = lse_out;
  const cudaStream_t s = as_stream(stream);
  if (dtype == DET_BF16) return dispatch_attention<__nv_bfloat16>(a, (int)head_dim, (int)batch, (int)kv_heads, s);
  return dispatch_attention<__half>(a, (int)head_dim, (int)batch, (int)kv_heads, s);
}
