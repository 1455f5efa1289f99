// mla_append_slots and mla_commit_tree: cache rows written through a slot map, and the accepted
// path's rows moved together.
//
// append_slots. row = [ RMSNorm(ckv) * gamma || RoPE(krope, pos) ], written to pool row slots[n].
// A drafted token's RoPE position is its depth's while its row is its own, so the position and
// the place are two inputs here. One warp per row, rows dealt round the grid: a lane holds up to
// NP 16-byte pieces of the row (coalesced across the warp), fp32 statistics by a butterfly. The
// angles are p * theta_i in double, as everywhere in the library, and are brought into [-pi, pi]
// in double (Cody and Waite's two-term reduction; exact to a rounding while the angle's turns are
// whole numbers of a double, any position for rope_base >= 1). An fp32 pool then gets the rotation
// in double, rounded once, as mla_append_latent does it. For a bf16 pool, whose rounding is 2^-8,
// sine and cosine are taken in fp32, off by 2^-23 for the angle rounded to fp32 and 2^-22 for
// sincosf: 16,384 rows of 512 take 10.9 us instead of 11.9 from HBM, 8.0 instead of 9.2 from L2
// (fp32 rows, in double, 14.0 and 8.7). theta_i = base^(-2i/d_r) comes from the host as a kernel
// argument: a double pow per lane, and sincos of the whole angle in double, took most of the 16 us
// that 16,384 bf16 rows needed.
// What bounds it: HBM and its latency for prompts (the row in and out: 16,384 tokens, 37.9 MB, 10.9
// us or 3.5 TB/s from HBM, 8.0 with the rows in L2; a warp has a row and the next in flight),
// latency for a decode step (128 tokens: 2.6 us).
#include <algorithm>
#include <cmath>

#include "tree.cuh"

namespace mla {
namespace {

constexpr int kAppendWarps = 8;

template <typename T> struct Piece;  // 16 bytes of a row
template <> struct Piece<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void widen(const uint4 u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *(const uint32_t*)&h;
    }
    *(uint4*)p = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <> struct Piece<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void widen(const uint4 u, float (&v)[4]) {
    v[0] = __uint_as_float(u.x);
    v[1] = __uint_as_float(u.y);
    v[2] = __uint_as_float(u.z);
    v[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ void store(float* p, const float (&v)[4]) {
    *(float4*)p = make_float4(v[0], v[1], v[2], v[3]);
  }
};

struct RopeTheta {
  double t[128];  // d_r <= 256
};

// two neighbouring values
__device__ __forceinline__ float2 load2(const float* p) { return *(const float2*)p; }
__device__ __forceinline__ float2 load2(const __nv_bfloat16* p) {
  const uint32_t u = *(const uint32_t*)p;
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ void store2(float* p, float x, float y) {
  *(float2*)p = make_float2(x, y);
}
__device__ __forceinline__ void store2(__nv_bfloat16* p, float x, float y) {
  *(__nv_bfloat162*)p = __floats2bfloat162_rn(x, y);
}

// Four CTAs per SM, fewer for longer rows: with more the registers no longer hold a row and the
// next (16,384 rows of 512 bf16 out of HBM: 10.5 us at four, 10.8 at three, 12.9 at five; without
// the next row's fetch 12.2, two rows per warp at a time longer still).
constexpr int append_ctas(int pieces) { return pieces <= 2 ? 4 : pieces <= 4 ? 3 : 2; }

template <typename T, int NP>
__global__ void __launch_bounds__(kAppendWarps * 32, append_ctas(NP))
append_slots_kernel(const T* __restrict__ ckv, const T* __restrict__ kr,
                    const float* __restrict__ gamma, const int32_t* __restrict__ pos,
                    const int64_t* __restrict__ slots, T* pool, int64_t pool_rows, int n, int r,
                    int dr, float eps, const __grid_constant__ RopeTheta theta, uint32_t* err) {
  constexpr int E = Piece<T>::N;
  const int lane = threadIdx.x & 31;
  const int warps = gridDim.x * kAppendWarps;
  const int half = dr / 2, D = r + dr;
  const double theta0 = lane < half ? theta.t[lane] : 0.0;
  wait_prior_grid();
  // what a row reads is fetched while the row before is worked on
  uint4 raw[NP];
  float2 k_next;
  int64_t slot_next = -1;
  int pos_next = 0;
  auto fetch = [&](int row) {
    slot_next = slots[row];
    pos_next = pos[row];
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int at = (lane + 32 * k) * E;
      if (at < r) raw[k] = *(const uint4*)(ckv + (size_t)row * r + at);
    }
    if (lane < half) k_next = load2(kr + (size_t)row * dr + 2 * lane);
  };
  int row = blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
  if (row < n) fetch(row);
  for (; row < n; row += warps) {
    const int64_t slot = slot_next;
    const double p = (double)pos_next;
    const float2 k0 = k_next;
    float v[NP][E];
#pragma unroll
    for (int k = 0; k < NP; ++k) Piece<T>::widen(raw[k], v[k]);
    if (row + warps < n) fetch(row + warps);
    if (slot < 0) continue;  // a step's padding
    if (slot >= pool_rows) {
      if (lane == 0) set_error(err, MLA_DEV_OOB_BLOCK);
      continue;
    }
    T* dst = pool + (size_t)slot * D;
    for (int i = lane; i < half; i += 32) {
      const float2 x = i < 32 ? k0 : load2(kr + (size_t)row * dr + 2 * i);
      const double a = p * (i < 32 ? theta0 : theta.t[i]);
      const double turns = rint(a * 0.15915494309189535);  // 1 / (2 pi)
      const double red = fma(-turns, 2.4492935982947064e-16, fma(-turns, 6.283185307179586, a));
      if constexpr (sizeof(T) == 4) {
        double c, s;
        sincos(red, &s, &c);
        store2(dst + r + 2 * i, (float)((double)x.x * c - (double)x.y * s),
               (float)((double)x.x * s + (double)x.y * c));
      } else {
        float c, s;
        sincosf((float)red, &s, &c);
        store2(dst + r + 2 * i, x.x * c - x.y * s, x.x * s + x.y * c);
      }
    }
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < NP; ++k)
      if ((lane + 32 * k) * E < r) {
#pragma unroll
        for (int e = 0; e < E; ++e) ss = fmaf(v[k][e], v[k][e], ss);
      }
    ss = warp_sum(ss);
    const float inv = 1.0f / sqrtf(ss / (float)r + eps);
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int at = (lane + 32 * k) * E;
      if (at < r) {
#pragma unroll
        for (int e = 0; e < E; e += 4) {
          const float4 g = *(const float4*)(gamma + at + e);
          v[k][e] *= inv * g.x;
          v[k][e + 1] *= inv * g.y;
          v[k][e + 2] *= inv * g.z;
          v[k][e + 3] *= inv * g.w;
        }
        Piece<T>::store(dst + at, v[k]);
      }
    }
  }
}

template <typename T, int NP>
cudaError_t append_slots_go(const mla_config& c, const void* ckv, const void* kr,
                            const float* gamma, const int32_t* pos, const int64_t* slots,
                            void* pool, int num_blocks, int n, uint32_t* err, cudaStream_t st) {
  const int grid = std::min((n + kAppendWarps - 1) / kAppendWarps, 148 * append_ctas(NP));
  RopeTheta theta = {};
  // by products in the longest type (64 bits of mantissa): rounded to double, each theta is off by
  // 2^-53 of itself, and so is its angle by another, 2^-52 in all: 4.8e-7 at position 2^31, 2.3e-10
  // at 2^20
  if (c.rope_dim > 0) {
    const long double step = std::pow((long double)c.rope_base, -2.0L / c.rope_dim);
    long double t = 1.0L;
    for (int i = 0; i < c.rope_dim / 2; ++i, t *= step) theta.t[i] = (double)t;
  }
  return launch_pdl(append_slots_kernel<T, NP>, dim3(grid), dim3(kAppendWarps * 32), 0, st,
                    (const T*)ckv, (const T*)kr, gamma, pos, slots, (T*)pool,
                    (int64_t)num_blocks * c.block_size, n, c.kv_rank, c.rope_dim, c.rms_eps, theta,
                    err);
}

}  // namespace

cudaError_t launch_append_slots(const mla_config& c, const void* ckv, const void* kr,
                                const float* gamma, const int32_t* pos, const int64_t* slots,
                                void* pool, int num_blocks, int n, uint32_t* err,
                                cudaStream_t st) {
  // pieces per lane: r values in 16-byte pieces over 32 lanes
  const int np = (c.kv_rank * (c.dtype == MLA_BF16 ? 2 : 4) / 16 + 31) / 32;
#define MLA_GO(T, NP) \
  append_slots_go<T, NP>(c, ckv, kr, gamma, pos, slots, pool, num_blocks, n, err, st)
  if (c.dtype == MLA_BF16) {
    if (np <= 1) return MLA_GO(__nv_bfloat16, 1);
    if (np <= 2) return MLA_GO(__nv_bfloat16, 2);
    return MLA_GO(__nv_bfloat16, 4);
  }
  if (np <= 1) return MLA_GO(float, 1);
  if (np <= 2) return MLA_GO(float, 2);
  if (np <= 4) return MLA_GO(float, 4);
  return MLA_GO(float, 8);
#undef MLA_GO
}

// ------------------------------------------------------------------------------------------
// commit_tree: row P + d <- row P + path[d], d < count, and the new length P + count. A path
// goes down the tree, so it is strictly increasing and path[d] >= d: a row is never overwritten
// before every later d has another source, and moving in order of d is safe in place. One CTA
// per sequence; a thread owns one 16-byte (8-byte) column of the rows and moves it for all d, so
// no two threads touch the same bytes and nothing has to be waited for between rows: kMove loads
// are in flight, then their stores (the stores of rows d .. d + kMove - 1 cannot reach a source
// path[d'] >= d' >= d + kMove). The path is checked before anything moves. What bounds it: latency
// (32 sequences of 4 nodes 2.4 us, 256 of 64 nodes 3.9).
// ------------------------------------------------------------------------------------------
namespace {

constexpr int kMove = 8;
constexpr int kCommitThreads = 128;

template <typename V>
__global__ void __launch_bounds__(kCommitThreads)
commit_tree_kernel(const int32_t* __restrict__ path, const int32_t* __restrict__ count,
                   int width, int T, const int32_t* __restrict__ table, int max_blocks,
                   uint8_t* pool, int num_blocks, int bs, int row_vecs, const int32_t* seq_lens,
                   int32_t* seq_lens_out, uint32_t* err) {
  __shared__ int64_t s_from[MLA_MAX_TREE], s_to[MLA_MAX_TREE];  // rows of the pool, -1: skip
  wait_prior_grid();
  const int b = blockIdx.x, tid = threadIdx.x;
  const int len = seq_lens[b];
  if (len == 0) {  // an empty place of the batch
    __syncthreads();
    if (tid == 0) seq_lens_out[b] = 0;
    return;
  }
  const int n = count[b];
  bool ok = len >= T && (int64_t)len <= (int64_t)max_blocks * bs && n >= 0 && n <= width && n <= T;
  const bool len_ok = len >= T && (int64_t)len <= (int64_t)max_blocks * bs;
  const int first = len - T;
  if (ok) {
    for (int d = tid; d < n; d += kCommitThreads) {
      const int a = path[(size_t)b * width + d];
      const int before = d > 0 ? path[(size_t)b * width + d - 1] : -1;
      if (a <= before || a < 0 || a >= T) {
        ok = false;
        continue;
      }
      const int from = first + a, to = first + d;
      const int bf = table[(size_t)b * max_blocks + from / bs];
      const int bt = table[(size_t)b * max_blocks + to / bs];
      const bool in = bf >= 0 && bf < num_blocks && bt >= 0 && bt < num_blocks;
      if (!in) set_error(err, MLA_DEV_OOB_BLOCK);
      s_from[d] = in && a != d ? (int64_t)bf * bs + from % bs : -1;
      s_to[d] = (int64_t)bt * bs + to % bs;
    }
  }
  ok = __syncthreads_and(ok);
  if (!ok) {
    if (tid == 0) {
      set_error(err, len_ok ? MLA_DEV_BAD_TREE : MLA_DEV_BAD_LENGTH);
      seq_lens_out[b] = len;
    }
    return;
  }
  if (tid == 0) seq_lens_out[b] = first + n;
  V* rows = (V*)pool;
  for (int c = tid; c < row_vecs; c += kCommitThreads) {
    for (int d0 = 0; d0 < n; d0 += kMove) {
      V v[kMove];
#pragma unroll
      for (int u = 0; u < kMove; ++u)
        if (d0 + u < n && s_from[d0 + u] >= 0) v[u] = rows[s_from[d0 + u] * row_vecs + c];
#pragma unroll
      for (int u = 0; u < kMove; ++u)
        if (d0 + u < n && s_from[d0 + u] >= 0) rows[s_to[d0 + u] * row_vecs + c] = v[u];
    }
  }
}

}  // namespace

cudaError_t launch_commit_tree(const mla_config& c, const int32_t* path, const int32_t* count,
                               int width, int T, const int32_t* table, int max_blocks, void* pool,
                               int num_blocks, const int32_t* seq_lens, int32_t* seq_lens_out,
                               int batch, uint32_t* err, cudaStream_t st) {
  // rows are r + d_r values, a multiple of 8: whole 16-byte pieces in both types
  const int row_vecs = (c.kv_rank + c.rope_dim) * (c.dtype == MLA_BF16 ? 2 : 4) / 16;
  return launch_pdl(commit_tree_kernel<uint4>, dim3(batch), dim3(kCommitThreads), 0, st, path,
                    count, width, T, table, max_blocks, (uint8_t*)pool, num_blocks,
                    c.block_size, row_vecs, seq_lens, seq_lens_out, err);
}

}  // namespace mla
