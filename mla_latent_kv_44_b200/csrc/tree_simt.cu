// CUDA-core attention of mla_decode_tree (any shape; fp32 or bf16 rows; fp32 math), and the merge
// of split key ranges.
//
// A sequence's T drafted tokens and H heads are T * H query rows over the same cache rows, so
// they are tiled together: one CTA takes 8 * RPW of them (8 warps, RPW rows per warp) against a
// range of cache rows, staged 32 * KPL at a time in shared memory as fp32. Scores: lane j of a
// warp takes cache rows j (and j + 32) for the warp's RPW query rows (one conflict-free 16-byte
// read of the row, its pitch D + 4 words, per RPW broadcast reads of the queries). Softmax:
// running maximum and sum in fp32, the warp's rows side by side (their shuffles overlap), the sums
// kept per lane until the end. Values: lane owns r / 32 columns; the weights go through shared
// memory four cache rows at a time. Rows of the cache that precede the drafted ones are seen by
// every token; for the drafted ones the token's mask word decides, and a masked score is
// replaced, never added to, so that nothing of a masked row (NaN included) reaches the result.
// The keys of a sequence are cut into `splits` equal ranges when there are too few query tiles to
// fill the GPU. The second kernel weighs the ranges by their log-sum-exp, in range order, and
// applies W_UV to the merged rows where it has them, in shared memory.
// What bounds it: latency at the sizes that it is for (fp32 models, small heads): a CTA's chain of
// block id, cache rows, scores, softmax, values, and shared-memory reads in scores and values
// (three for eight FMAs). So 64 cache rows go in one tile where two CTAs of that fit an SM (128
// registers a thread: 8 x 5 tokens of 16 heads, r = 64, over 1024 rows 24.7 us; with three CTAs
// and ranges for them 23.4, but 64 x 4 tokens 77 against 72 and 4 x 16 tokens over 4000 rows 47
// against 42; with one 29.6).
#include <algorithm>

#include "tree.cuh"

namespace mla {
namespace {

constexpr int kWarps = 8;

// 2^x, off by 2 ulp at most
__device__ __forceinline__ float ex2_(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T> __device__ __forceinline__ float4 load4(const T* p);
template <> __device__ __forceinline__ float4 load4<float>(const float* p) {
  return *(const float4*)p;
}
template <> __device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p) {
  const uint2 u = *(const uint2*)p;
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                     __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}

template <typename T, int RPW, int KPL, int RW>  // RW: latent columns per lane (r <= 32 * RW)
__global__ void __launch_bounds__(kWarps * 32, KPL == 2 ? 2 : 1)
tree_simt_kernel(const TreeParams p) {
  constexpr int M = kWarps * RPW, kKeys = 32 * KPL;
  extern __shared__ __align__(16) float smem[];
  const int D = p.D, ld = D + 4, r = p.r, quads = D / 4;
  float* s_q = smem;                  // M x D
  float* s_k = s_q + M * D;           // kKeys x ld
  float* s_p = s_k + kKeys * ld;      // M x kKeys
  __shared__ int s_there[kKeys];
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

  // the pool row of a cache row, or -1 (past the range, or a block outside the pool)
  auto place = [&](int row) -> int64_t {
    if (row >= hi) return -1;
    const int at = row / p.bs, blk = p.table[(size_t)b * p.max_blocks + at];
    if (blk < 0 || blk >= p.num_blocks) {
      set_error(p.err, MLA_DEV_OOB_BLOCK);
      return -1;
    }
    return (int64_t)blk * p.bs + (row - at * p.bs);
  };

  // a warp takes every eighth row of a tile; lane j finds where row j of the warp's rows lies, one
  // tile ahead
  constexpr int kPer = kKeys / kWarps;
  int64_t next_at = place(lo + warp + kWarps * (lane % kPer));

  // queries, times softmax_scale / ln 2: scores come out in base-2 units
  const float c2 = p.scale * 1.4426950408889634f;
  const T* Q = (const T*)p.q + ((size_t)b * rows + m0) * D;
  for (int qd = lane; qd < quads; qd += 32) {
    float4 v[RPW];
#pragma unroll
    for (int a = 0; a < RPW; ++a) {
      const int m = warp * RPW + a;
      v[a] = m0 + m < rows ? load4(Q + (size_t)m * D + 4 * qd) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int a = 0; a < RPW; ++a)
      *(float4*)(s_q + (warp * RPW + a) * D + 4 * qd) =
          make_float4(v[a].x * c2, v[a].y * c2, v[a].z * c2, v[a].w * c2);
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
    __syncthreads();  // previous tile consumed
    const int64_t my_at = next_at;
    int64_t at[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) at[j] = __shfl_sync(0xffffffffu, my_at, j) * D;
    for (int qd = lane; qd < quads; qd += 32) {  // all rows' loads, then their stores
      float4 v[kPer];
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        v[j] = at[j] >= 0 ? load4((const T*)p.pool + at[j] + 4 * qd)
                          : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int j = 0; j < kPer; ++j) *(float4*)(s_k + (warp + kWarps * j) * ld + 4 * qd) = v[j];
    }
    if (lane < kPer) s_there[warp + kWarps * lane] = my_at >= 0;
    next_at = place(t0 + kKeys + warp + kWarps * (lane % kPer));
    __syncthreads();
    if (m0 + warp * RPW >= rows) continue;  // this warp has no query rows
    bool there[KPL];
#pragma unroll
    for (int c = 0; c < KPL; ++c) there[c] = s_there[lane + 32 * c];

    // scores of cache rows t0 + lane + 32 c
    float s[RPW][KPL];
#pragma unroll
    for (int a = 0; a < RPW; ++a)
#pragma unroll
      for (int c = 0; c < KPL; ++c) s[a][c] = 0.f;
    const float* krow = s_k + lane * ld;
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
      float4 k[KPL];
#pragma unroll
      for (int c = 0; c < KPL; ++c) k[c] = *(const float4*)(krow + 32 * c * ld + d);
#pragma unroll
      for (int a = 0; a < RPW; ++a) {
        const float4 q = *(const float4*)(qw + a * D + d);
#pragma unroll
        for (int c = 0; c < KPL; ++c) {
          s[a][c] = fmaf(q.x, k[c].x, s[a][c]);
          s[a][c] = fmaf(q.y, k[c].y, s[a][c]);
          s[a][c] = fmaf(q.z, k[c].z, s[a][c]);
          s[a][c] = fmaf(q.w, k[c].w, s[a][c]);
        }
      }
    }
    const bool drafted = t0 + kKeys > first;  // the tile holds drafted rows
    bool seen[RPW][KPL];
#pragma unroll
    for (int a = 0; a < RPW; ++a)
#pragma unroll
      for (int c = 0; c < KPL; ++c) seen[a][c] = there[c];
    if (drafted) {
#pragma unroll
      for (int a = 0; a < RPW; ++a)
#pragma unroll
        for (int c = 0; c < KPL; ++c) {
          const int node = t0 + lane + 32 * c - first;
          if (node >= 0 && there[c]) seen[a][c] = tree_sees(p, b, tok[a], node);
        }
    }
    // the warp's rows side by side, so that their shuffles overlap
    float top[RPW];
#pragma unroll
    for (int a = 0; a < RPW; ++a) {
      top[a] = -INFINITY;
#pragma unroll
      for (int c = 0; c < KPL; ++c) {
        s[a][c] = seen[a][c] ? s[a][c] : -INFINITY;
        top[a] = fmaxf(top[a], s[a][c]);
      }
    }
#pragma unroll
    for (int step = 16; step > 0; step >>= 1)
#pragma unroll
      for (int a = 0; a < RPW; ++a)
        top[a] = fmaxf(top[a], __shfl_xor_sync(0xffffffffu, top[a], step));
#pragma unroll
    for (int a = 0; a < RPW; ++a) {
      const float m = fmaxf(mx[a], top[a]);
      const float alpha = mx[a] == -INFINITY ? 0.f : ex2_(mx[a] - m);
      float sum = 0.f;
#pragma unroll
      for (int c = 0; c < KPL; ++c) {
        const float e = seen[a][c] && s[a][c] != -INFINITY ? ex2_(s[a][c] - m) : 0.f;
        sum += e;
        pw[a * kKeys + lane + 32 * c] = e;
      }
      l[a] = l[a] * alpha + sum;  // the lane's share; summed over the warp at the end
      mx[a] = m;
#pragma unroll
      for (int k = 0; k < RW; ++k) o[a][k] *= alpha;
    }
    __syncwarp();
    // a lane's columns: 64 k + 2 lane and the next
    if (drafted) {  // a masked row's values are left out, whatever they are
      for (int j = 0; j < kKeys; ++j) {
#pragma unroll
        for (int k = 0; k < RW / 2; ++k) {
          const int d = 64 * k + 2 * lane;
          const float2 v = d < r ? *(const float2*)(s_k + j * ld + d) : make_float2(0.f, 0.f);
#pragma unroll
          for (int a = 0; a < RPW; ++a) {
            const float e = pw[a * kKeys + j];
            o[a][2 * k] = e == 0.f ? o[a][2 * k] : fmaf(e, v.x, o[a][2 * k]);
            o[a][2 * k + 1] = e == 0.f ? o[a][2 * k + 1] : fmaf(e, v.y, o[a][2 * k + 1]);
          }
        }
      }
    } else {
#pragma unroll 4
      for (int j = 0; j < kKeys; j += 4) {
        float4 e[RPW];
#pragma unroll
        for (int a = 0; a < RPW; ++a) e[a] = *(const float4*)(pw + a * kKeys + j);
#pragma unroll
        for (int k = 0; k < RW / 2; ++k) {
          const int d = 64 * k + 2 * lane;
          if (d < r) {
            const float* at = s_k + j * ld + d;
            const float2 v0 = *(const float2*)at, v1 = *(const float2*)(at + ld),
                         v2 = *(const float2*)(at + 2 * ld), v3 = *(const float2*)(at + 3 * ld);
#pragma unroll
            for (int a = 0; a < RPW; ++a) {
              float &x = o[a][2 * k], &y = o[a][2 * k + 1];
              x = fmaf(e[a].x, v0.x, x);
              y = fmaf(e[a].x, v0.y, y);
              x = fmaf(e[a].y, v1.x, x);
              y = fmaf(e[a].y, v1.y, y);
              x = fmaf(e[a].z, v2.x, x);
              y = fmaf(e[a].z, v2.y, y);
              x = fmaf(e[a].w, v3.x, x);
              y = fmaf(e[a].w, v3.y, y);
            }
          }
        }
      }
    }
    __syncwarp();  // the warp's weights are read
  }

#pragma unroll
  for (int step = 16; step > 0; step >>= 1)
#pragma unroll
    for (int a = 0; a < RPW; ++a) l[a] += __shfl_xor_sync(0xffffffffu, l[a], step);
#pragma unroll
  for (int a = 0; a < RPW; ++a) {
    const int m = warp * RPW + a;
    if (m0 + m >= rows) continue;
    // row (token, head) of the call, in this range's part
    const size_t at = (size_t)split * p.BT * p.H + (size_t)b * rows + m0 + m;
    const bool empty = l[a] == 0.f;
    const float inv = empty ? 0.f : 1.f / l[a];
    if (lane == 0)
      p.part_lse[at] = empty ? -INFINITY : (mx[a] + log2f(l[a])) * 0.6931471805599453f;
#pragma unroll
    for (int k = 0; k < RW / 2; ++k) {
      const int d = 64 * k + 2 * lane;
      if (d < r)
        *(float2*)(p.part_o + at * r + d) =
            empty ? make_float2(0.f, 0.f) : make_float2(o[a][2 * k] * inv, o[a][2 * k + 1] * inv);
    }
  }
}

// ---- merge of the ranges and W_UV: one CTA per head and NT tokens -------------------------
// (4.3 us of the 24.7: two rounds of loads, of the log-sum-exps and the partial rows, and W_UV.)
// stage: W_UV[h] fits shared memory; it is fetched before the wait for the attention (it is no
// result of it) and read from there.
template <typename T, int NT>
__global__ void __launch_bounds__(128)
tree_simt_out_kernel(const TreeParams p, const T* __restrict__ w_uv, T* __restrict__ o, int dv,
                     int stage) {
  extern __shared__ __align__(16) float s_lat[];  // NT x r, then dv rows of W_UV[h]
  __shared__ float s_w[NT][kTreeMaxSplits];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = p.r;
  const int h = blockIdx.x % p.H, n0 = blockIdx.x / p.H * NT;
  const size_t part = (size_t)p.BT * p.H;
  constexpr int kPiece = 16 / sizeof(T);
  const int pitch = r + kPiece;  // values per row of the copy
  T* s_wuv = (T*)(s_lat + NT * r);
  if (stage) {
    const T* w = w_uv + (size_t)h * dv * r;
    for (int i = threadIdx.x; i < dv * (r / kPiece); i += blockDim.x) {
      const int row = i / (r / kPiece), c = i - row * (r / kPiece);
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                       (uint32_t)__cvta_generic_to_shared(s_wuv + row * pitch + c * kPiece)),
                   "l"(w + (size_t)i * kPiece)
                   : "memory");
    }
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
  wait_prior_grid();
  for (int t = warp; t < NT; t += 4) {  // a warp per token: weights, then the merged row
    const int n = n0 + t;
    if (n >= p.BT) break;
    const size_t at = (size_t)n * p.H + h;
    float mx = -INFINITY;
    bool nan = false;
    for (int k = lane; k < p.splits; k += 32) {
      const float x = p.part_lse[k * part + at];
      nan |= x != x;
      mx = fmaxf(mx, x);
    }
    mx = warp_max(mx);
    nan = __any_sync(0xffffffffu, nan);
    float z = 0.f;
    for (int k = lane; k < p.splits; k += 32) {
      const float x = p.part_lse[k * part + at];
      const float e = x == -INFINITY ? 0.f : expf(x - mx);
      s_w[t][k] = e;
      z += e;
    }
    z = warp_sum(z);
    const bool empty = mx == -INFINITY && !nan;
    const float inv = empty ? 0.f : 1.f / z;
    __syncwarp();
    // r / 4 lanes cover a row; where that is half a warp or less, groups of lanes share the ranges
    const int share = r <= 32 ? 4 : r <= 64 ? 2 : 1, width = 32 / share;
    for (int d = 4 * (lane % width); d < (r + 4 * width - 1) / (4 * width) * (4 * width);
         d += 4 * width) {
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
      for (int k = lane / width; k < (d < r ? p.splits : 0); k += share) {
        const float e = s_w[t][k] * inv;
        // a range without rows holds zeros
        const float4 v = __ldcs((const float4*)(p.part_o + (k * part + at) * r + d));
        a.x = fmaf(e, v.x, a.x);
        a.y = fmaf(e, v.y, a.y);
        a.z = fmaf(e, v.z, a.z);
        a.w = fmaf(e, v.w, a.w);
      }
      for (int step = width; step < 32; step <<= 1) {
        a.x += __shfl_xor_sync(0xffffffffu, a.x, step);
        a.y += __shfl_xor_sync(0xffffffffu, a.y, step);
        a.z += __shfl_xor_sync(0xffffffffu, a.z, step);
        a.w += __shfl_xor_sync(0xffffffffu, a.w, step);
      }
      if (d < r && lane < width) *(float4*)(s_lat + t * r + d) = a;
    }
    if (lane == 0 && p.lse) p.lse[at] = empty ? -INFINITY : mx + logf(z);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  for (int i = threadIdx.x; i < dv; i += blockDim.x) {
    const T* w = stage ? s_wuv + i * pitch : w_uv + ((size_t)h * dv + i) * r;
    float acc[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = 0.f;
#pragma unroll 4
    for (int d = 0; d < r; d += 4) {
      const float4 u = load4(w + d);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float4 v = *(const float4*)(s_lat + t * r + d);
        acc[t] = fmaf(u.x, v.x, acc[t]);
        acc[t] = fmaf(u.y, v.y, acc[t]);
        acc[t] = fmaf(u.z, v.z, acc[t]);
        acc[t] = fmaf(u.w, v.w, acc[t]);
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
      if (n0 + t < p.BT) o[((size_t)(n0 + t) * p.H + h) * dv + i] = from_f32<T>(acc[t]);
  }
}

template <typename T, int RPW, int KPL, int RW>
cudaError_t simt_go(const TreeParams& p, cudaStream_t st) {
  const int M = kWarps * RPW, keys = 32 * KPL;
  const size_t smem = sizeof(float) * ((size_t)M * p.D + keys * (p.D + 4) + M * keys);
  static std::atomic<unsigned long long> devices{0};
  auto k = tree_simt_kernel<T, RPW, KPL, RW>;
  const cudaError_t e = raise_smem_limit((const void*)k, devices);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, dim3((unsigned)(p.batch * p.tiles * p.splits)), dim3(kWarps * 32), smem,
                    st, p);
}

template <typename T, int NT>
cudaError_t simt_out(const TreeParams& p, const void* w_uv, int dv, void* o, cudaStream_t st) {
  const size_t w_bytes = (size_t)dv * (p.r * sizeof(T) + 16);
  const int stage = w_bytes <= 64 * 1024;
  const size_t smem = sizeof(float) * NT * p.r + (stage ? w_bytes : 0);
  static std::atomic<unsigned long long> devices{0};
  auto k = tree_simt_out_kernel<T, NT>;
  const cudaError_t e = raise_smem_limit((const void*)k, devices);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, dim3((unsigned)(p.H * ((p.BT + NT - 1) / NT))), dim3(128), smem, st, p,
                    (const T*)w_uv, (T*)o, dv, stage);
}

template <typename T>
cudaError_t simt_dispatch(const TreeParams& p, const void* w_uv, int dv, void* o,
                          cudaStream_t st) {
  cudaError_t e;
  if (p.tile_rows == kWarps * 4) {
    // 64 cache rows per tile where two CTAs fit an SM, else 32
    if (p.r <= 64 && p.D <= 192) e = simt_go<T, 4, 2, 2>(p, st);
    else if (p.r <= 128 && p.D <= 192) e = simt_go<T, 4, 2, 4>(p, st);
    else if (p.r <= 256) e = simt_go<T, 4, 1, 8>(p, st);
    else e = simt_go<T, 4, 1, 16>(p, st);
  } else {
    e = simt_go<T, 1, 1, 32>(p, st);
  }
  if (e != cudaSuccess) return e;
  // four tokens a CTA while those fill the GPU no more than twice over, else sixteen (W_UV[h] is
  // read once per CTA)
  if ((int64_t)p.H * p.BT <= 4 * 2 * 148 * 4) return simt_out<T, 4>(p, w_uv, dv, o, st);
  return simt_out<T, 16>(p, w_uv, dv, o, st);
}

}  // namespace

cudaError_t launch_tree_simt(const mla_config& c, const TreeParams& p, const void* w_uv, void* o,
                             cudaStream_t st) {
  return c.dtype == MLA_BF16 ? simt_dispatch<__nv_bfloat16>(p, w_uv, c.head_dim_v, o, st)
                             : simt_dispatch<float>(p, w_uv, c.head_dim_v, o, st);
}

// Query rows per tile: 32 (four per warp) where r <= 512, whose tile and 32 cache rows fit shared
// memory whatever d_r is (at most 256), else 8.
int tree_simt_tile_rows(const mla_config& c) { return c.kv_rank <= 512 ? 4 * kWarps : kWarps; }

}  // namespace mla
