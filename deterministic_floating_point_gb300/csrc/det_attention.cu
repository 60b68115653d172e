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

constexpr int kTile = 16;        // tokens of a tile
constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = 32 * kAttnWarps;
constexpr int kMaxChunk = 1024;  // most tokens of a chunk

// Tokens of a chunk of a sequence of n tokens.
__host__ __device__ inline int chunk_tokens(long long n) { return n <= 8192 ? 256 : n <= 32768 ? 512 : kMaxChunk; }
__host__ __device__ inline int chunk_count(int n) {
  const int c = chunk_tokens(n);
  return n <= 0 ? 1 : (n - 1) / c + 1;
}
// Most chunks of a sequence of at most n tokens.
inline int most_chunks(int n) {
  int most = chunk_count(n);
  if (n > 8192) most = std::max(most, chunk_count(8192));
  if (n > 32768) most = std::max(most, chunk_count(32768));
  return most;
}

template <int D> __host__ __device__ constexpr int attn_stages() { return D == 64 ? 6 : 3; }
template <int D> __host__ __device__ constexpr size_t attn_smem() {
  return (size_t)kAttnWarps * attn_stages<D>() * kTile * D * 2 * 2;
}

struct AttnArgs {
  const void *q, *k, *v;
  long long q_sb, q_sh, k_sp, k_st, k_sh, v_sp, v_st, v_sh;
  const int32_t *table, *lengths;
  long long table_stride;
  int num_pages, page_size, limit;   // limit: most tokens of a sequence
  int heads, group, head_tiles, max_chunks;
  float scale_log2;
  const void* bias;
  int bias_dtype;
  const int32_t* bounds;
  int num_bounds;
  float* part;      // [batch x heads][max_chunks][D]: the chunk's outputs, not yet divided
  float2* part_ml;  // [batch x heads][max_chunks]: maximum (of log2 scores) and sum
  void* out;
  float* lse;
};

__device__ __forceinline__ void cp_async_16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
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

// Number of bounds <= n.
__device__ __forceinline__ int bounds_at_most(const int32_t* bounds, int count, int n) {
  int lo = 0, hi = count;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(bounds + mid) <= n) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

// NT tiles of 8 heads per CTA.  Grid: (chunks, kv heads x head tiles, batch).
template <typename T, int D, int NT>
__global__ void __launch_bounds__(kAttnThreads) attention_chunks_kernel(const __grid_constant__ AttnArgs a) {
  constexpr int S = attn_stages<D>();
  constexpr int C = D / 8;              // 16-byte pieces of a row
  constexpr int kRowBytes = D * 2;
  constexpr int kTileBytes = kTile * kRowBytes;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int sh_page[kMaxChunk + 1];
  __shared__ unsigned sh_mask[kAttnWarps][S];
  __shared__ float sh_m[kAttnWarps][8 * NT], sh_l[kAttnWarps][8 * NT];

  const int chunk = blockIdx.x, b = blockIdx.z;
  const int g = blockIdx.y / a.head_tiles, h0 = (blockIdx.y % a.head_tiles) * 8 * NT;   // first head in the group
  const int n = min(max(a.lengths[b], 0), a.limit);
  const int chunks = chunk_count(n);
  if (chunk >= chunks) return;
  const int size = chunk_tokens(n);
  const int t0 = chunk * size, t1 = min(n, t0 + size);
  const int p0 = t0 / a.page_size;
  const int pages = t1 > t0 ? (t1 - 1) / a.page_size - p0 + 1 : 0;
  const int32_t* table = a.table + b * a.table_stride + p0;
  for (int i = threadIdx.x; i < pages; i += kAttnThreads) {
    const int p = table[i];
    sh_page[i] = p >= 0 && p < a.num_pages ? p : -1;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

  // the queries as B operands: column = head (lane / 4), rows = dims
  unsigned qf[D / 16][NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int h = h0 + nt * 8 + lane / 4;
    const T* q = static_cast<const T*>(a.q) + b * a.q_sb + (long long)(g * a.group + h) * a.q_sh;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int d = ks * 16 + j * 8 + 2 * (lane & 3);
        unsigned w = 0;
        if (h < a.group) {
          const unsigned short* p = reinterpret_cast<const unsigned short*>(q + d);
          w = (unsigned)__ldg(p) | ((unsigned)__ldg(p + 1) << 16);
        }
        qf[ks][nt][j] = w;
      }
  }
  __syncthreads();

  const T* kbase = static_cast<const T*>(a.k) + g * a.k_sh;
  const T* vbase = static_cast<const T*>(a.v) + g * a.v_sh;
  unsigned char* ring = smem + (size_t)warp * S * 2 * kTileBytes;
  const int tiles = (t1 - t0 + kTile - 1) / kTile;
  const int mine = (tiles - warp + kAttnWarps - 1) / kAttnWarps;   // tiles of this warp (warp <= tiles or <= 0)

  auto load = [&](int it) {
    if (it < mine) {
      const int stage = it % S;
      const int j = t0 + (it * kAttnWarps + warp) * kTile + (lane & 15);
      long long ko = 0, vo = 0;
      int page = -1;
      if (j < t1) {
        const int pj = j / a.page_size, slot = j - pj * a.page_size;
        page = sh_page[pj - p0];
        ko = page * a.k_sp + slot * a.k_st;
        vo = page * a.v_sp + slot * a.v_st;
      }
      const unsigned mask = __ballot_sync(0xffffffffu, page >= 0) & 0xffffu;
      if (lane == 0) sh_mask[warp][stage] = mask;
      unsigned char* ks = ring + (size_t)stage * 2 * kTileBytes;
      unsigned char* vs = ks + kTileBytes;
#pragma unroll
      for (int i = 0; i < kTile * C / 32; ++i) {
        const int at = i * 32 + lane, row = at / C, c = at % C;
        const long long kr = __shfl_sync(0xffffffffu, ko, row), vr = __shfl_sync(0xffffffffu, vo, row);
        const int dst = row * kRowBytes + ((c ^ (row & 7)) << 4);
        if ((mask >> row) & 1) {
          cp_async_16(ks + dst, kbase + kr + c * 8);
          cp_async_16(vs + dst, vbase + vr + c * 8);
        } else {   // nothing is read for a skipped token: 0, so that 0 * value is 0
          *reinterpret_cast<uint4*>(ks + dst) = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(vs + dst) = make_uint4(0, 0, 0, 0);
        }
      }
    }
    cp_async_commit();
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

#pragma unroll
  for (int it = 0; it < S - 1; ++it) load(it);
  for (int it = 0; it < mine; ++it) {
    load(it + S - 1);
    cp_async_wait<S - 1>();
    __syncwarp();
    const int stage = it % S;
    const unsigned ks = smem_u32(ring + (size_t)stage * 2 * kTileBytes), vs = ks + kTileBytes;
    float s[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[nt][j] = 0.0f;
    {
      const int row = lane & 15;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        unsigned af[4];
        ldmatrix_x4(af, ks + row * kRowBytes + (((2 * k + (lane >> 4)) ^ (row & 7)) << 4));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_16816<T>(s[nt], af, qf[k][nt][0], qf[k][nt][1]);
      }
    }
    // scores in units of log 2; masked tokens to -inf
    const unsigned mask = sh_mask[warp][stage] >> (lane >> 2);
    const int j0 = t0 + (it * kAttnWarps + warp) * kTile + (lane >> 2);
    int bucket0 = 0, bucket1 = 0;
    if (a.bias) {
      bucket0 = bounds_at_most(a.bounds, a.num_bounds, n - 1 - j0);
      bucket1 = bounds_at_most(a.bounds, a.num_bounds, n - 9 - j0);
    }
    bool raise = false;
    float fresh[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int h = h0 + nt * 8 + 2 * (lane & 3) + j;
        float x0 = s[nt][j] * a.scale_log2, x1 = s[nt][2 + j] * a.scale_log2;
        if (a.bias && h < a.group) {
          const long long col = g * a.group + h;
          x0 = fmaf(load_as_f32(a.bias, (long long)bucket0 * a.heads + col, a.bias_dtype), kLog2e, x0);
          x1 = fmaf(load_as_f32(a.bias, (long long)bucket1 * a.heads + col, a.bias_dtype), kLog2e, x1);
        }
        s[nt][j] = (mask & 1) ? x0 : kNegInf;
        s[nt][2 + j] = (mask & 256) ? x1 : kNegInf;
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
          const float f = m[nt][j] == kNegInf ? 1.0f : exp2_approx(m[nt][j] - fresh[nt][j]);
          m[nt][j] = fresh[nt][j];
          l[nt][j] *= f;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            o[i][nt][j] *= f;
            o[i][nt][2 + j] *= f;
          }
        }
    }
    // the weights as B operands (column = head), in two parts: the weight
    // rounded to 16 bits and what the rounding left
    unsigned ph[NT][2], pl[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float base = m[nt][j] == kNegInf ? 0.0f : m[nt][j];
        s[nt][j] = exp2_approx(s[nt][j] - base);
        s[nt][2 + j] = exp2_approx(s[nt][2 + j] - base);
        l[nt][j] += s[nt][j] + s[nt][2 + j];
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const unsigned hi = pack2<T>(s[nt][2 * half], s[nt][2 * half + 1]);
        const float2 r = unpack2<T>(hi);
        ph[nt][half] = movmatrix_trans(hi);
        pl[nt][half] = movmatrix_trans(pack2<T>(s[nt][2 * half] - r.x, s[nt][2 * half + 1] - r.y));
      }
    }
    {
      const int row = (lane & 7) + ((lane >> 4) & 1) * 8;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        unsigned af[4];
        ldmatrix_x4_trans(af, vs + row * kRowBytes + (((2 * i + ((lane >> 3) & 1)) ^ (row & 7)) << 4));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_16816<T>(o[i][nt], af, ph[nt][0], ph[nt][1]);
          mma_16816<T>(o[i][nt], af, pl[nt][0], pl[nt][1]);
        }
      }
    }
    __syncwarp();   // the stage is free
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
  constexpr int kPitch = D + 4;   // floats of a row of the joined outputs: the writes below hit 32 banks
  float* sh_o = reinterpret_cast<float*>(smem);
  static_assert((size_t)kAttnWarps * 8 * NT * kPitch * 4 <= attn_smem<D>(), "the outputs fit the ring");
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int col = nt * 8 + 2 * (lane & 3) + j;
      float top = kNegInf;
      for (int w = 0; w < kAttnWarps; ++w) top = fmaxf(top, sh_m[w][col]);
      const float f = m[nt][j] == kNegInf ? 1.0f : exp2_approx(m[nt][j] - top);
      float* dst = sh_o + (size_t)(warp * 8 * NT + col) * kPitch + (lane >> 2);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        dst[i * 16] = o[i][nt][j] * f;
        dst[i * 16 + 8] = o[i][nt][2 + j] * f;
      }
    }
  __syncthreads();
  for (int at = threadIdx.x; at < 8 * NT * D; at += kAttnThreads) {
    const int col = at / D, d = at % D;
    if (h0 + col >= a.group) break;
    float top = kNegInf, sum = 0.0f, v = 0.0f;
    for (int w = 0; w < kAttnWarps; ++w) top = fmaxf(top, sh_m[w][col]);
    for (int w = 0; w < kAttnWarps; ++w) {
      const float mw = sh_m[w][col];
      sum += mw == kNegInf ? sh_l[w][col] : sh_l[w][col] * exp2_approx(mw - top);
      v += sh_o[(size_t)(w * 8 * NT + col) * kPitch + d];
    }
    const long long bh = (long long)b * a.heads + g * a.group + h0 + col;
    if (chunks == 1) {
      static_cast<T*>(a.out)[bh * D + d] = from_f32<T>(top == kNegInf && sum == 0.0f ? 0.0f : v / sum);
      if (a.lse && d == 0) a.lse[bh] = top == kNegInf && sum == 0.0f ? kNegInf : (top + log2f(sum)) * (1.0f / kLog2e);
    } else {
      a.part[(bh * a.max_chunks + chunk) * D + d] = v;
      if (d == 0) a.part_ml[bh * a.max_chunks + chunk] = make_float2(top, sum);
    }
  }
}

// The chunks of one head of one sequence joined: warp w of 4 adds the chunks
// w, w + 4, ..., then the warps are added in order.
template <typename T, int D>
__global__ void __launch_bounds__(kAttnThreads) attention_join_kernel(const __grid_constant__ AttnArgs a) {
  constexpr int E = D / 32;
  __shared__ float sh_top[kAttnWarps], sh_sum[kAttnWarps];
  __shared__ float sh_o[kAttnWarps][D];
  dep_wait();
  const int h = blockIdx.x, b = blockIdx.y;
  const int chunks = chunk_count(min(max(a.lengths[b], 0), a.limit));
  if (chunks == 1) return;   // already in place
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long bh = (long long)b * a.heads + h;
  const float2* ml = a.part_ml + bh * a.max_chunks;
  const float* part = a.part + bh * a.max_chunks * D;
  float top = kNegInf;
  for (int c = threadIdx.x; c < chunks; c += kAttnThreads) top = fmaxf(top, ml[c].x);
  for (int d = 1; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  if (lane == 0) sh_top[warp] = top;
  __syncthreads();
  for (int w = 0; w < kAttnWarps; ++w) top = fmaxf(top, sh_top[w]);
  float v[E], sum = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] = 0.0f;
#pragma unroll 4
  for (int c = warp; c < chunks; c += kAttnWarps) {
    const float2 x = ml[c];
    const float f = x.x == kNegInf ? 1.0f : exp2_approx(x.x - top);   // a chunk without a score adds 0
    sum = fmaf(x.y, f, sum);
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = fmaf(part[(long long)c * D + e * 32 + lane], f, v[e]);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) sh_o[warp][e * 32 + lane] = v[e];
  if (lane == 0) sh_sum[warp] = sum;
  __syncthreads();
  sum = 0.0f;
  for (int w = 0; w < kAttnWarps; ++w) sum += sh_sum[w];
  const bool none = top == kNegInf && sum == 0.0f;
  for (int d = threadIdx.x; d < D; d += kAttnThreads) {
    float r = 0.0f;
    for (int w = 0; w < kAttnWarps; ++w) r += sh_o[w][d];
    static_cast<T*>(a.out)[bh * D + d] = from_f32<T>(none ? 0.0f : r / sum);
  }
  if (a.lse && threadIdx.x == 0) a.lse[bh] = none ? kNegInf : (top + log2f(sum)) * (1.0f / kLog2e);
}

template <typename T, int D, int NT>
int launch_attention(AttnArgs a, int batch, int kv_heads, cudaStream_t s) {
  a.head_tiles = (a.group + 8 * NT - 1) / (8 * NT);
  if ((long long)kv_heads * a.head_tiles > 65535) return DET_ERR_TOO_LARGE;
  const void* kernel = reinterpret_cast<const void*>(&attention_chunks_kernel<T, D, NT>);
  if (const cudaError_t e = ensure_dyn_smem(kernel, attn_smem<D>())) return cuda_fail(e, "det_paged_attention");
  const dim3 grid((unsigned)a.max_chunks, (unsigned)(kv_heads * a.head_tiles), (unsigned)batch);
  launch_begin("det_paged_attention", s);
  attention_chunks_kernel<T, D, NT><<<grid, kAttnThreads, attn_smem<D>(), s>>>(a);
  launch_end(s);
  if (const int rc = check_launch("det_paged_attention")) return rc;
  if (a.max_chunks == 1) return DET_OK;
  launch_begin("det_paged_attention_join", s);
  const cudaError_t e = launch_dep(attention_join_kernel<T, D>, dim3((unsigned)a.heads, (unsigned)batch),
                                   dim3(kAttnThreads), 0, s, a);
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
  a.scale_log2 = scale * kLog2e;
  a.bias = bias_table, a.bias_dtype = bias_dtype, a.bounds = bias_bounds, a.num_bounds = (int)num_bounds;
  unsigned char* ws = static_cast<unsigned char*>(workspace) + kHeaderBytes;
  a.part_ml = reinterpret_cast<float2*>(ws);
  a.part = reinterpret_cast<float*>(ws + align_up((size_t)batch * heads * a.max_chunks * sizeof(float2), 256));
  a.out = out, a.lse = lse_out;
  const cudaStream_t s = as_stream(stream);
  if (dtype == DET_BF16) return dispatch_attention<__nv_bfloat16>(a, (int)head_dim, (int)batch, (int)kv_heads, s);
  return dispatch_attention<__half>(a, (int)head_dim, (int)batch, (int)kv_heads, s);
}
