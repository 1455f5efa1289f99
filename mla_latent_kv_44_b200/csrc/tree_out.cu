// The last stages of mla_decode_tree on the tensor-core path: partial results of cut items merged,
// then o[n, h, :] = W_UV[h] latent[n, h, :].
//
// Per head the product is W_UV[h] (d_v x 512) with the call's latent sums of that head (512 x n). A
// CTA keeps 128 rows of W_UV[h] in shared memory (128 KB, loaded by TMA before it waits for the
// kernel in front) and streams the latent rows of 32 tokens, 256 dims at a time, through three
// buffers by cp.async: both bf16 terms of each value (hi = bf16(x), lo = bf16(x - hi); one
// term alone would add as large an error as the rounding of o). M = 128 (dims), N = 32 (tokens):
// 32 MMAs per buffer into one of two tensor-memory accumulators; the epilogue of a tile of
// tokens runs while the next one's products do. What bounds it: the weights' bytes for few
// tokens, the latent rows' for many.
#include <atomic>

#include "tc_ptx.cuh"
#include "tma_map.h"
#include "tree.cuh"
#include "tree_ptx.cuh"

namespace mla {
namespace {

constexpr int kR = 512;
constexpr int kSlabs = kR / 64;
constexpr int kHalf = kSlabs / 2;                  // slabs of one buffer, for each term
constexpr int kDims = 128;                         // rows of W_UV per CTA
constexpr int kTok = 32;                           // tokens per tile
constexpr int kBufs = 3;
constexpr int kThreads = 256;
constexpr int kWSlab = kDims * 128, kBSlab = kTok * 128;
constexpr int kW = 0;
constexpr int kB = kW + kSlabs * kWSlab;           // 128 KB
constexpr int kBBytes = kSlabs * kBSlab;           // 32 KB
constexpr int kBar = kB + kBufs * kBBytes;         // W, products of even and odd buffers
constexpr int kSmem = kBar + 3 * 8 + 16 + 1024;
static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
constexpr unsigned long long kTimeoutNs = 1000000000ull;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t ta, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15}, [%16];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15])
      : "r"(ta)
      : "memory");
}

// D[tmem] (+)= A[smem] . B[smem], descriptors by their low words
__device__ __forceinline__ void mma1(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t id,
                                     uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(id), "r"(acc), "r"(kDescHi)
      : "memory");
}

// ---- merge: one warp per query row of an item in the list of cuts -------------------------
constexpr int kMergeWarps = 8;

__global__ void __launch_bounds__(kMergeWarps * 32) tree_merge_parts_kernel(const TreeParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  wait_prior_grid();
  constexpr int kPer = kTreeTile / kMergeWarps;  // CTAs per tile of query rows
  const int lane = threadIdx.x & 31, m = blockIdx.x % kPer * kMergeWarps + (threadIdx.x >> 5);
  const int member = blockIdx.x / kPer % p.team;
  const int4 cut = p.cuts[blockIdx.x / (kPer * p.team)];
  if (cut.x < 0) return;
  const int b = cut.x / p.groups, mt = (cut.x - b * p.groups) * p.team + member;
  const int row = mt * kTreeTile + m;
  if (row >= p.T * p.H) return;
  auto at = [&](int k) -> size_t {  // the k-th piece's result
    const int slot = k == 0 ? cut.z : 2 * (cut.z / 2 + k);
    return ((size_t)slot * p.team + member) * kTreeTile + m;
  };
  float mx = -INFINITY;
  bool nan = false;
  for (int k = lane; k < cut.y; k += 32) {
    const float x = p.part_lse[at(k)];
    nan |= x != x;
    mx = fmaxf(mx, x);
  }
  mx = warp_max(mx);
  const bool empty = mx == -INFINITY && !__any_sync(0xffffffffu, nan);
  float4 acc[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) acc[u] = make_float4(0.f, 0.f, 0.f, 0.f);
  float z = 0.f;
  if (!empty) {
#pragma unroll 4
    for (int k = 0; k < cut.y; ++k) {
      const size_t part = at(k);
      const float x = p.part_lse[part];
      const float e = x == -INFINITY ? 0.f : expf(x - mx);
      z += e;
      const float4* src = (const float4*)(p.part_o + part * kR) + lane;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float4 v = __ldcs(src + 32 * u);
        acc[u].x = fmaf(e, v.x, acc[u].x);
        acc[u].y = fmaf(e, v.y, acc[u].y);
        acc[u].z = fmaf(e, v.z, acc[u].z);
        acc[u].w = fmaf(e, v.w, acc[u].w);
      }
    }
  }
  const float inv = empty ? 0.f : 1.f / z;
  const size_t out = (size_t)b * p.T * p.H + row;
  uint2* hi = (uint2*)(p.latent_hi + out * kR) + lane;
  uint2* lo = (uint2*)(p.latent_lo + out * kR) + lane;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const float v[4] = {acc[u].x * inv, acc[u].y * inv, acc[u].z * inv, acc[u].w * inv};
    const uint2 h = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    hi[32 * u] = h;
    lo[32 * u] = make_uint2(pack_bf16(v[0] - __uint_as_float(h.x << 16),
                                      v[1] - __uint_as_float(h.x & 0xffff0000u)),
                            pack_bf16(v[2] - __uint_as_float(h.y << 16),
                                      v[3] - __uint_as_float(h.y & 0xffff0000u)));
  }
  if (lane == 0 && p.lse) p.lse[out] = empty ? -INFINITY : mx + logf(z);
}

__global__ void __launch_bounds__(kThreads, 1)
tree_out_kernel(const __grid_constant__ CUtensorMap tm_w, const TreeParams p, int dv, int splits,
                __nv_bfloat16* __restrict__ o) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const uint32_t s_base = saddr(smem);
  const uint32_t bar_w = s_base + kBar, bar_d = bar_w + 8;  // W; the products of a buffer (by i & 1)
  uint32_t* tmem_slot = (uint32_t*)(smem + kBar + 24);
  volatile int* abort_flag = (volatile int*)(smem + kBar + 28);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  // this CTA's head, rows of W_UV and tiles of tokens
  const int split = blockIdx.x % splits, h = (blockIdx.x / splits) % p.H;
  const int dim0 = blockIdx.x / (splits * p.H) * kDims;
  const int tiles = (p.BT + kTok - 1) / kTok;
  const int lo = (int)((int64_t)tiles * split / splits);
  const int hi = (int)((int64_t)tiles * (split + 1) / splits);

  if (tid == 0) {
    for (int i = 0; i < 3; ++i) mbar_init(bar_w + 8 * i, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     saddr(tmem_slot)),
                 "r"(2 * kTok)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  if (warp == 0 && elect_one()) {
    // the weights come from before the attention kernel, which waited for what came before it
    // and is over when the kernel in front of this one writes
    mbar_expect_tx(bar_w, kSlabs * kWSlab);
#pragma unroll
    for (int k = 0; k < kSlabs; ++k)
      tma_load(s_base + kW + k * kWSlab, &tm_w, bar_w, 64 * k, h * dv + dim0);
  }
  __syncwarp();
  wait_prior_grid();

  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (mbar_try(bar, parity)) return;
    const uint64_t t0 = globaltimer();
    while (*abort_flag == 0 && !mbar_try(bar, parity)) {
      if (globaltimer() - t0 > kTimeoutNs) {
        set_error(p.err, MLA_DEV_WAIT_TIMEOUT);
        *abort_flag = 1;
      }
    }
  };
  // buffer i % 3: 32 tokens, 256 dims (half i & 1) of both terms. A thread takes one 16-byte piece
  // (32 per row) of four rows in each term. Sequences without rows read as zeros.
  auto load = [&](int i) {
    const int piece = tid & 31;
    const int n0 = (lo + (i >> 1)) * kTok;
    const uint32_t dst = s_base + kB + (uint32_t)(i % kBufs) * kBBytes + (piece >> 3) * kBSlab;
    bool live[kTok / 8];
#pragma unroll
    for (int u = 0; u < kTok / 8; ++u) {
      const int n = n0 + (tid >> 5) + 8 * u;
      live[u] = n < p.BT && tree_length(p, n / p.T, false) > 0;
      if (n < p.BT && !live[u] && piece == 0 && dim0 == 0 && (i & 1) == 0 && p.lse)
        p.lse[(size_t)n * p.H + h] = -INFINITY;
    }
#pragma unroll
    for (int u = 0; u < kTok / 8; ++u) {
      const int t = (tid >> 5) + 8 * u;
      const uint32_t at = dst + 128u * (uint32_t)t + 16u * (uint32_t)((piece & 7) ^ (t & 7));
      const size_t src = ((size_t)(n0 + t) * p.H + h) * kR + 256 * (i & 1) + 8 * piece;
      if (live[u]) {
        cp_async16(at, p.latent_hi + src);
        cp_async16(at + kHalf * kBSlab, p.latent_lo + src);
      } else {
#pragma unroll
        for (int term = 0; term < 2; ++term)
          asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at + term * kHalf * kBSlab),
                       "r"(0)
                       : "memory");
      }
    }
  };
  auto commit_loads = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };
  // tile i's accumulator (complete) -> o: a thread holds one dim of 16 tokens; neighbours swap, so that each
  // stores two dims of every second token
  auto store = [&](int i) {
    tc_after();
    const int quad = warp & 3, half = warp >> 2;
    uint32_t v[16];
    tmem_ld16(tmem + ((uint32_t)(32 * quad) << 16) + kTok * (i & 1) + 16 * half, v);
    tc_before();
    const int dim = dim0 + 32 * quad + lane, n0 = (lo + i) * kTok + 16 * half;
    const bool even = (lane & 1) == 0;
#pragma unroll
    for (int c = 0; c < 16; c += 2) {
      const uint32_t got = __shfl_xor_sync(0xffffffffu, even ? v[c + 1] : v[c], 1);
      const int n = n0 + c + (even ? 0 : 1);
      const float x = __uint_as_float(even ? v[c] : got), y = __uint_as_float(even ? got : v[c + 1]);
      if (n < p.BT) {
        __nv_bfloat16* dst = o + ((size_t)n * p.H + h) * dv + (dim & ~1);
        if ((dv & 1) == 0) {
          if (dim < dv) *(uint32_t*)dst = pack_bf16(x, y);
        } else {
          if ((dim & ~1) < dv) dst[0] = __float2bfloat16_rn(x);
          if ((dim | 1) < dv) dst[1] = __float2bfloat16_rn(y);
        }
      }
    }
  };

  const int count = 2 * (hi - lo);  // buffers: two per tile of tokens
  if (count > 0) load(0);
  commit_loads();
  if (count > 1) load(1);
  commit_loads();
  constexpr uint32_t id = idesc(kDims, kTok, 0);
  const uint32_t w_lo = desc_lo(s_base + kW, 16), b_lo = desc_lo(s_base + kB, 16);
  for (int i = 0; i < count; ++i) {
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    fence_proxy_async();
    __syncthreads();  // buffer i is in shared memory, and the accumulator it goes to was read
    if (warp == 0) {
      if (i == 0) wait(bar_w, 0);
      __syncwarp();
      tc_after();
      if (elect_one()) {
        const uint32_t b = b_lo + (uint32_t)(i % kBufs) * (kBBytes >> 4);
        const uint32_t a = w_lo + (i & 1) * kHalf * (kWSlab >> 4);
        const uint32_t d = tmem + kTok * ((i >> 1) & 1);
#pragma unroll
        for (int k = 0; k < 2 * kHalf; ++k)  // hi's slabs, then lo's
#pragma unroll
          for (int s = 0; s < 4; ++s)
            mma1(d, a + (k % kHalf) * (kWSlab >> 4) + 2 * s, b + k * (kBSlab >> 4) + 2 * s, id,
                 ((i & 1) || k > 0 || s > 0) ? 1u : 0u);
        tc_commit(bar_d + 8 * (i & 1));
      }
      __syncwarp();
    }
    // the products of buffer i - 1 are over: it takes i + 2; after a tile's second, its result
    if (i > 0) {
      wait(bar_d + 8 * ((i - 1) & 1), ((i - 1) >> 1) & 1);
      __syncwarp();
      if ((i & 1) == 0) store((i >> 1) - 1);
    }
    if (i + 2 < count) load(i + 2);
    commit_loads();
  }
  if (count > 0) {
    wait(bar_d + 8, ((count - 1) >> 1) & 1);
    __syncwarp();
    store((count >> 1) - 1);
  } else {
    wait(bar_w, 0);  // the weights have landed before this CTA may exit
  }
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(2 * kTok)
                 : "memory");
}

}  // namespace

cudaError_t launch_tree_merge(const TreeParams& p, cudaStream_t st) {
  const int ctas = p.ranges * p.team * (kTreeTile / kMergeWarps);
  return launch_pdl(tree_merge_parts_kernel, dim3((unsigned)ctas), dim3(kMergeWarps * 32), 0, st,
                    p);
}

cudaError_t launch_tree_out(const TreeParams& p, const void* w_uv, int dv, void* o,
                            cudaStream_t st) {
  CUtensorMap w;
  if (!make_bf16_map(&w, w_uv, kR, (uint64_t)p.H * dv, kR * 2, kDims)) return cudaErrorInvalidValue;
  static std::atomic<unsigned long long> attr_devices{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? (1ull << dev) : 0ull;
  if (!bit || !(attr_devices.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(tree_out_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    attr_devices.fetch_or(bit, std::memory_order_acq_rel);
  }
  // one CTA per 128 rows of W_UV; its tokens are split where that leaves SMs idle
  const int ctas = p.H * ((dv + kDims - 1) / kDims), tiles = (p.BT + kTok - 1) / kTok;
  const int splits = ctas >= 148 ? 1 : (148 / ctas < tiles ? 148 / ctas : tiles);
  return launch_pdl(tree_out_kernel, dim3((unsigned)(ctas * splits)), dim3(kThreads), kSmem, st,
                    w, p, dv, splits, (__nv_bfloat16*)o);
}

}  // namespace mla
