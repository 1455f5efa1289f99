// CUDA-core attention of mla_decode_tree (any shape; fp32 or bf16 rows; fp32 math), and the merge
// of split key ranges.
//
// A sequence's T drafted tokens and H heads are T * H query rows over the same cache rows, so
// they are tiled together: one CTA takes 8 * RPW of them (8 warps, RPW rows per warp) against a
// range of cache rows, staged 32 at a time in shared memory as fp32. Scores: lane j of a warp
// takes cache row j for the warp's RPW query rows (one conflict-free 16-byte read of the row,
// its pitch D + 4 words, per RPW broadcast reads of the queries). Softmax: running maximum and
// sum in fp32. Values: lane owns r / 32 columns; the weights go through shared memory four cache
// rows at a time. Rows of the cache that precede the drafted ones are seen by every token; for
// the drafted ones the token's mask word decides, and a masked score is replaced, never added to,
// so that nothing of a masked row (NaN included) reaches the result.
// The keys of a sequence are cut into `splits` equal ranges when there are too few query tiles
// to fill the GPU; the merge weighs the ranges by their log-sum-exp, in range order.
#include <cuda_fp8.h>

#include <algorithm>

#include "tree.cuh"

namespace mla {
namespace {

constexpr int kWarps = 8;
constexpr int kKeys = 32;  // cache rows per staged tile (one per lane)

template <typename T> __device__ __forceinline__ float4 load4(const T* p);
template <> __device__ __forceinline__ float4 load4<float>(const float* p) {
  return *(const float4*)p;
}
template <> __device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p) {
  const uint2 u = *(const uint2*)p;
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                     __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}

template <typename T, int RPW, int RW>  // RW: latent columns per lane (r <= 32 * RW)
__global__ void __launch_bounds__(kWarps * 32) tree_simt_kernel(const TreeParams p) {
  constexpr int M = kWarps * RPW;
  extern __shared__ __align__(16) float smem[];
  const int D = p.D, ld = D + 4, r = p.r, quads = D / 4;
  float* s_q = smem;                  // M x D
  float* s_k = s_q + M * D;           // kKeys x ld
  float* s_p = s_k + kKeys * ld;      // M x kKeys
  int* s_blk = (int*)(s_p + M * kKeys);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x % p.splits, tile = blockIdx.x / p.splits;
  const int b = tile / p.tiles, m0 = (tile - b * p.tiles) * M;
  wait_prior_grid();

  const int len = tree_length(p, b, threadIdx.x == 0 && m0 == 0 && split == 0);
  const int first = len - p.T;  // cache row of the first drafted token
  const int rows = p.T * p.H;   // query rows of a sequence
  // this CTA's cache rows, whole tiles of kKeys
  const int tiles = (len + kKeys - 1) / kKeys, per = (tiles + p.splits - 1) / p.splits;
  const int lo = min(split * per, tiles) * kKeys, hi = min((split + 1) * per * kKeys, len);

  const T* Q = (const T*)p.q + ((size_t)b * rows + m0) * D;
  for (int i = threadIdx.x; i < M * quads; i += blockDim.x) {
    const int m = i / quads;
    ((float4*)s_q)[i] = m0 + m < rows ? load4(Q + 4 * (size_t)i) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float o[RPW][RW], mx[RPW], l[RPW];
#pragma unroll
  for (int a = 0; a < RPW; ++a) {
    mx[a] = -INFINITY;
    l[a] = 0.f;
#pragma unroll
    for (int k = 0; k < RW; ++k) o[a][k] = 0.f;
  }
  int tok[RPW];
#pragma unroll
  for (int a = 0; a < RPW; ++a) tok[a] = min((m0 + warp * RPW + a) / p.H, p.T - 1);
  const float* qw = s_q + warp * RPW * D;
  float* pw = s_p + warp * RPW * kKeys;

  for (int t0 = lo; t0 < hi; t0 += kKeys) {
    __syncthreads();  // previous tile consumed (s_q written, the first time)
    if (threadIdx.x < kKeys) {
      const int row = t0 + threadIdx.x;
      int blk = -1;
      if (row < hi) {
        blk = p.table[(size_t)b * p.max_blocks + row / p.bs];
        if (blk < 0 || blk >= p.num_blocks) {
          set_error(p.err, MLA_DEV_OOB_BLOCK);
          blk = -1;
        }
      }
      s_blk[threadIdx.x] = blk;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kKeys * quads; i += blockDim.x) {
      const int t = i / quads, qd = i - t * quads, blk = s_blk[t];
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (blk >= 0)
        v = load4((const T*)p.pool + ((size_t)blk * p.bs + (t0 + t) % p.bs) * D + 4 * qd);
      *(float4*)(s_k + t * ld + 4 * qd) = v;
    }
    __syncthreads();

    // scores of cache row t0 + lane
    float s[RPW];
#pragma unroll
    for (int a = 0; a < RPW; ++a) s[a] = 0.f;
    const float* krow = s_k + lane * ld;
    for (int d = 0; d < D; d += 4) {
      const float4 k = *(const float4*)(krow + d);
#pragma unroll
      for (int a = 0; a < RPW; ++a) {
        const float4 q = *(const float4*)(qw + a * D + d);
        s[a] = fmaf(q.x, k.x, s[a]);
        s[a] = fmaf(q.y, k.y, s[a]);
        s[a] = fmaf(q.z, k.z, s[a]);
        s[a] = fmaf(q.w, k.w, s[a]);
      }
    }
    const bool drafted = t0 + kKeys > first;  // the tile holds drafted rows
    const int node = t0 + lane - first;
#pragma unroll
    for (int a = 0; a < RPW; ++a) {
      bool seen = s_blk[lane] >= 0;
      if (node >= 0 && seen) seen = tree_sees(p, b, tok[a], node);
      s[a] = seen ? s[a] * p.scale : -INFINITY;
      const float m = fmaxf(mx[a], warp_max(s[a]));
      const float alpha = mx[a] == -INFINITY ? 0.f : expf(mx[a] - m);
      const float e = seen && s[a] != -INFINITY ? expf(s[a] - m) : 0.f;
      l[a] = l[a] * alpha + warp_sum(e);
      mx[a] = m;
#pragma unroll
      for (int k = 0; k < RW; ++k) o[a][k] *= alpha;
      pw[a * kKeys + lane] = e;
    }
    __syncwarp();
    if (drafted) {  // a masked row's values are left out, whatever they are
      for (int j = 0; j < kKeys; ++j) {
#pragma unroll
        for (int k = 0; k < RW; ++k) {
          const int d = lane + 32 * k;
          const float v = d < r ? s_k[j * ld + d] : 0.f;
#pragma unroll
          for (int a = 0; a < RPW; ++a) {
            const float e = pw[a * kKeys + j];
            o[a][k] = e == 0.f ? o[a][k] : fmaf(e, v, o[a][k]);
          }
        }
      }
    } else {
      for (int j = 0; j < kKeys; j += 4) {
        float4 e[RPW];
#pragma unroll
        for (int a = 0; a < RPW; ++a) e[a] = *(const float4*)(pw + a * kKeys + j);
#pragma unroll
        for (int k = 0; k < RW; ++k) {
          const int d = lane + 32 * k;
          if (d < r) {
            const float v0 = s_k[j * ld + d], v1 = s_k[(j + 1) * ld + d],
                        v2 = s_k[(j + 2) * ld + d], v3 = s_k[(j + 3) * ld + d];
#pragma unroll
            for (int a = 0; a < RPW; ++a) {
              o[a][k] = fmaf(e[a].x, v0, o[a][k]);
              o[a][k] = fmaf(e[a].y, v1, o[a][k]);
              o[a][k] = fmaf(e[a].z, v2, o[a][k]);
              o[a][k] = fmaf(e[a].w, v3, o[a][k]);
            }
          }
        }
      }
    }
  }

#pragma unroll
  for (int a = 0; a < RPW; ++a) {
    const int m = warp * RPW + a;
    if (m0 + m >= rows) continue;
    const size_t at = (size_t)b * rows + m0 + m;  // (token, head) of the call
    const bool empty = l[a] == 0.f;
    const float inv = empty ? 0.f : 1.f / l[a];
    const float lse = empty ? -INFINITY : mx[a] + logf(l[a]);
    float* dst;
    if (p.splits == 1) {
      dst = p.latent + at * r;
      if (lane == 0 && p.lse) p.lse[at] = lse;
    } else {
      const size_t part = (size_t)split * p.BT * p.H + at;
      dst = p.part_o + part * r;
      if (lane == 0) p.part_lse[part] = lse;
    }
#pragma unroll
    for (int k = 0; k < RW; ++k) {
      const int d = lane + 32 * k;
      if (d < r) dst[d] = empty ? 0.f : o[a][k] * inv;
    }
  }
}

// ---- merge of `splits` ranges: one warp per (token, head) --------------------------------
__global__ void __launch_bounds__(128) tree_merge_kernel(const TreeParams p) {
  __shared__ float s_w[4][kTreeMaxSplits];
  wait_prior_grid();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const size_t n = (size_t)p.BT * p.H, at = (size_t)blockIdx.x * 4 + warp;
  if (at >= n) return;
  float* w = s_w[warp];
  float mx = -INFINITY;
  bool nan = false;
  for (int k = lane; k < p.splits; k += 32) {
    const float x = p.part_lse[k * n + at];
    nan |= x != x;
    mx = fmaxf(mx, x);
  }
  mx = warp_max(mx);
  float z = 0.f;
  for (int k = lane; k < p.splits; k += 32) {
    const float x = p.part_lse[k * n + at];
    const float e = x == -INFINITY ? 0.f : expf(x - mx);
    w[k] = e;
    z += e;
  }
  z = warp_sum(z);
  nan = __any_sync(0xffffffffu, nan);
  const bool empty = mx == -INFINITY && !nan;
  const float inv = empty ? 0.f : 1.f / z;
  __syncwarp();
  for (int d = 4 * lane; d < p.r; d += 128) {
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < p.splits; ++k) {
      const float e = w[k] * inv;
      if (e == 0.f) continue;  // a range without rows
      const float4 v = __ldcs((const float4*)(p.part_o + (k * n + at) * p.r + d));
      acc.x = fmaf(e, v.x, acc.x);
      acc.y = fmaf(e, v.y, acc.y);
      acc.z = fmaf(e, v.z, acc.z);
      acc.w = fmaf(e, v.w, acc.w);
    }
    *(float4*)(p.latent + at * p.r + d) = acc;
  }
  if (lane == 0 && p.lse) p.lse[at] = empty ? -INFINITY : mx + logf(z);
}

template <typename T, int RPW, int RW>
cudaError_t simt_go(const TreeParams& p, cudaStream_t st) {
  const int M = kWarps * RPW;
  const size_t smem = sizeof(float) * ((size_t)M * p.D + kKeys * (p.D + 4) + M * kKeys) +
                      sizeof(int) * kKeys;
  auto k = tree_simt_kernel<T, RPW, RW>;
  const cudaError_t e =
      cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, dim3((unsigned)(p.batch * p.tiles * p.splits)), dim3(kWarps * 32), smem,
                    st, p);
}

template <typename T>
cudaError_t simt_dispatch(const TreeParams& p, cudaStream_t st) {
  if (p.tile_rows == kWarps * 4) {
    if (p.r <= 64) return simt_go<T, 4, 2>(p, st);
    if (p.r <= 128) return simt_go<T, 4, 4>(p, st);
    if (p.r <= 256) return simt_go<T, 4, 8>(p, st);
    return simt_go<T, 4, 16>(p, st);
  }
  if (p.r <= 512) return simt_go<T, 1, 16>(p, st);
  return simt_go<T, 1, 32>(p, st);
}

}  // namespace

cudaError_t launch_tree_simt(const mla_config& c, const TreeParams& p, cudaStream_t st) {
  cudaError_t e = c.dtype == MLA_BF16 ? simt_dispatch<__nv_bfloat16>(p, st)
                                      : simt_dispatch<float>(p, st);
  if (e == cudaSuccess && p.splits > 1) {
    const size_t n = (size_t)p.BT * p.H;
    e = launch_pdl(tree_merge_kernel, dim3((unsigned)((n + 3) / 4)), dim3(128), 0, st, p);
  }
  return e;
}

// Query rows per tile: 32 (four per warp) where r <= 512 and the tile and 32 cache rows fit
// shared memory, else 8.
int tree_simt_tile_rows(const mla_config& c) {
  return c.kv_rank <= 512 && c.kv_rank + c.rope_dim <= 768 ? 4 * kWarps : kWarps;
}

}  // namespace mla
