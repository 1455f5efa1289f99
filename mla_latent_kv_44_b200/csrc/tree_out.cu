// The last stages of mla_decode_tree on the tensor-core path: partial results of cut items merged,
// then o[n, h, :] = W_UV[h] latent[n, h, :].
//
// Per head the product is W_UV[h] (d_v x 512) with the call's latent sums of that head (512 x n). A
// CTA keeps 128 rows of W_UV[h] in shared memory (128 KB, loaded by TMA before it waits for the
// kernel in front) and streams 64 dims of 128 tokens at a time through a ring of three stages,
// both bf16 terms of each value (hi = bf16(x), lo = bf16(x - hi); one term alone would add as large
// an error as the rounding of o). M = 128 (dims), N = the tile's tokens: 8 MMAs per stage into
// one of two tensor-memory accumulators; the epilogue of a tile of tokens runs while the next
// one's products do. (1024 tokens of 128 heads take 59 us, 0.32 GB at 5.4 TB/s; with 32 tokens per
// tile the MMAs' issue took 146.) With few tokens the CTA merges its head's partial
// results itself, into the operand's layout (6 us for 8 tokens, of them the merge 2.8). What
// bounds it: latency and the weights' bytes for few tokens, the latent rows' for many.
#include <atomic>

#include "tc_ptx.cuh"
#include "tma_map.h"
#include "tree.cuh"
#include "tree_ptx.cuh"

namespace mla {
namespace {

constexpr int kR = 512;
constexpr int kSlabs = kR / 64;
constexpr int kDims = 128;                         // rows of W_UV per CTA
constexpr int kTok = 128;                          // tokens per tile
constexpr int kRing = 3;
constexpr int kMergeThreads = 512;                 // of the kernel that merges them
constexpr int kMergeTok = 32;                      // most tokens that are merged here
constexpr int kThreads = 256;
constexpr int kWSlab = kDims * 128, kTerm = kTok * 128;
constexpr int kStage = 2 * kTerm;                  // hi and lo: 32 KB
constexpr int kW = 0;
constexpr int kB = kW + kSlabs * kWSlab;           // 128 KB
constexpr int kBars = kB + kRing * kStage;         // 224 KB
enum Bar {
  kWFull = 0,                  // kSlabs: a slab of W_UV landed
  kFull = kWFull + kSlabs,     // kRing: a stage landed
  kEmpty = kFull + kRing,      // kRing: its products are complete
  kDFull = kEmpty + kRing,     // 2: a tile's products are complete
  kDEmpty = kDFull + 2,        // 2: the epilogue warps read an accumulator
  kNumBars = kDEmpty + 2
};
constexpr int kSmem = kBars + kNumBars * 8 + 16 + 1024;
static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
static_assert(kSlabs * 2 * kMergeTok * 128 <= kRing * kStage, "the merged operand's place");
constexpr unsigned long long kTimeoutNs = 1000000000ull, kSettleNs = 20000000ull;

__device__ __forceinline__ void tma_load3(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x,
                                          int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst), "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// Warp-collective bounded wait.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, uint32_t* err,
                                     volatile int* abort) {
  if (__all_sync(0xffffffffu, mbar_try(bar, parity))) return true;
  const uint64_t t0 = globaltimer();
  for (;;) {
    if (__all_sync(0xffffffffu, mbar_try(bar, parity))) return true;
    const bool late = globaltimer() - t0 > kTimeoutNs;
    if (__any_sync(0xffffffffu, *abort != 0 || late)) {
      if ((threadIdx.x & 31) == 0 && late) {
        set_error(err, MLA_DEV_WAIT_TIMEOUT);
        *abort = 1;
      }
      return false;
    }
  }
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

// ---- merge of a cut item's pieces for one query row, by a warp ---------------------------------
// m: row of the tile. acc: lane's dims 128 u + 4 lane .. + 3, divided by the sum; returns the lse.
__device__ __forceinline__ float merge_row(const TreeParams& p, const int4 cut, int member, int m,
                                           int lane, float4 (&acc)[4]) {
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
#pragma unroll
  for (int u = 0; u < 4; ++u) acc[u] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (empty) return -INFINITY;
  float z = 0.f;
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
  const float inv = 1.f / z;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    acc[u].x *= inv;
    acc[u].y *= inv;
    acc[u].z *= inv;
    acc[u].w *= inv;
  }
  return mx + logf(z);
}
// the two bf16 terms of four values
__device__ __forceinline__ void split4(const float4 v, uint2* hi, uint2* lo) {
  const uint2 h = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
  *hi = h;
  *lo = make_uint2(
      pack_bf16(v.x - __uint_as_float(h.x << 16), v.y - __uint_as_float(h.x & 0xffff0000u)),
      pack_bf16(v.z - __uint_as_float(h.y << 16), v.w - __uint_as_float(h.y & 0xffff0000u)));
}

// One warp per query row of an item in the list of cuts.
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
  float4 acc[4];
  const float lse = merge_row(p, cut, member, m, lane, acc);
  const size_t out = (size_t)b * p.T * p.H + row;
  uint2* hi = (uint2*)(p.latent_hi + out * kR) + lane;
  uint2* lo = (uint2*)(p.latent_lo + out * kR) + lane;
#pragma unroll
  for (int u = 0; u < 4; ++u) split4(acc[u], hi + 32 * u, lo + 32 * u);
  if (lane == 0 && p.lse) p.lse[out] = lse;
}

// kMerge: few tokens, whose cut items this kernel merges itself, straight into the layout of the
// MMA's operand; there is no merge kernel then.
template <bool kMerge>
__global__ void __launch_bounds__(kMerge ? kMergeThreads : kThreads, 1)
tree_out_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_hi,
                const __grid_constant__ CUtensorMap tm_lo, const TreeParams p, int dv, int splits,
                __nv_bfloat16* __restrict__ o) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const uint32_t s_base = saddr(smem);
  auto bar = [&](int i) { return s_base + kBars + 8u * (uint32_t)i; };
  uint32_t* tmem_slot = (uint32_t*)(smem + kBars + kNumBars * 8);
  volatile int* abort = (volatile int*)(smem + kBars + kNumBars * 8 + 4);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  // this CTA's head, rows of W_UV and tiles of tokens
  const int split = blockIdx.x % splits, h = (blockIdx.x / splits) % p.H;
  const int dim0 = blockIdx.x / (splits * p.H) * kDims;
  const int tiles = (p.BT + kTok - 1) / kTok;
  const int lo = (int)((int64_t)tiles * split / splits);
  const int hi = (int)((int64_t)tiles * (split + 1) / splits);

  if (threadIdx.x == 0) {
    for (int i = 0; i < kNumBars; ++i) mbar_init(bar(i), i < kDEmpty ? 1 : 4);
    *abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
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

  const uint32_t w_lo = desc_lo(s_base + kW, 16), b_lo = desc_lo(s_base + kB, 16);
  const int pad = kMerge ? (p.BT + 15) / 16 * 16 : 0;  // tokens of an operand tile
  if (kMerge) {
    if (warp == 0 && elect_one()) {
#pragma unroll
      for (int k = 0; k < kSlabs; ++k) {
        mbar_expect_tx(bar(kWFull + k), kWSlab);
        tma_load(s_base + kW + k * kWSlab, &tm_w, bar(kWFull + k), 64 * k, h * dv + dim0);
      }
    }
    __syncwarp();
    wait_prior_grid();
    int4 cuts[3];  // the list, three entries per lane
    static_assert(kRanges <= 96, "entries held");
#pragma unroll
    for (int i = 0; i < 3; ++i)
      cuts[i] = lane + 32 * i < p.ranges ? p.cuts[lane + 32 * i] : make_int4(-1, 0, 0, 0);
    for (int n = warp; n < p.BT; n += kMergeThreads / 32) {
      const int b = n / p.T, row = (n - b * p.T) * p.H + h;
      const int mt = row / kTreeTile, m = row - mt * kTreeTile;
      const int group = mt / p.team, member = mt - group * p.team, item = b * p.groups + group;
      int4 cut = make_int4(-1, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const uint32_t found = __ballot_sync(0xffffffffu, cuts[i].x == item);
        if (found) {
          const int from = __ffs(found) - 1;
          cut.x = item;
          cut.y = __shfl_sync(0xffffffffu, cuts[i].y, from);
          cut.z = __shfl_sync(0xffffffffu, cuts[i].z, from);
        }
      }
      uint2 hi[4], lo_[4];
      if (cut.x >= 0) {
        float4 acc[4];
        const float lse = merge_row(p, cut, member, m, lane, acc);
#pragma unroll
        for (int u = 0; u < 4; ++u) split4(acc[u], &hi[u], &lo_[u]);
        if (lane == 0 && dim0 == 0 && p.lse) p.lse[(size_t)n * p.H + h] = lse;
      } else {
        // finished by the attention (or of an empty sequence, whose outputs are zeros whatever
        // is here)
        const size_t at = ((size_t)n * p.H + h) * kR;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          hi[u] = *((const uint2*)(p.latent_hi + at) + lane + 32 * u);
          lo_[u] = *((const uint2*)(p.latent_lo + at) + lane + 32 * u);
        }
      }
      // slab 2 u + lane / 16 of 64 dims, term, token: 128-byte rows swizzled by row % 8
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        uint8_t* at = smem + kB + (2 * (2 * u + (lane >> 4)) * pad + n) * 128 +
                      16 * (((lane & 15) >> 1) ^ (n & 7)) + 8 * (lane & 1);
        *(uint2*)at = hi[u];
        *(uint2*)(at + pad * 128) = lo_[u];
      }
    }
    fence_proxy_async();
    __syncthreads();
    if (warp == 1) {
      const uint32_t id = idesc(kDims, pad, 0);
      bool ok = true;
      for (int k = 0; k < kSlabs && ok; ++k) {
        ok = wait(bar(kWFull + k), 0, p.err, abort);
        if (!ok) break;
        tc_after();
        if (elect_one()) {
          const uint32_t a = w_lo + k * (kWSlab >> 4), b = b_lo + k * (2 * pad * 128 >> 4);
#pragma unroll
          for (int s = 0; s < 8; ++s)
            mma1(tmem, a + 2 * (s & 3), b + (s >> 2) * (pad * 128 >> 4) + 2 * (s & 3), id,
                 (k > 0 || s > 0) ? 1u : 0u);
          if (k == kSlabs - 1) tc_commit(bar(kDFull));
        }
        __syncwarp();
      }
    }
  } else if (warp == 0) {
    // ------------------------------------------------------------------------------------ TMA
    // The weights come from before the attention kernel, whose CTAs let the kernels behind it
    // start only once their own wait for what came before is over.
    if (elect_one()) {
#pragma unroll
      for (int k = 0; k < kSlabs; ++k) {
        mbar_expect_tx(bar(kWFull + k), kWSlab);
        tma_load(s_base + kW + k * kWSlab, &tm_w, bar(kWFull + k), 64 * k, h * dv + dim0);
      }
    }
    __syncwarp();
    wait_prior_grid();
    int stage = 0, used = 0;
    uint32_t round = 0;
    bool ok = true;
    for (int i = lo; i < hi && ok; ++i) {
      for (int k = 0; k < kSlabs; ++k, ++used) {
        if (used >= kRing && !wait(bar(kEmpty + stage), round ^ 1, p.err, abort)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          const uint32_t dst = s_base + kB + stage * kStage;
          mbar_expect_tx(bar(kFull + stage), kStage);
          tma_load3(dst, &tm_hi, bar(kFull + stage), 64 * k, h, i * kTok);
          tma_load3(dst + kTerm, &tm_lo, bar(kFull + stage), 64 * k, h, i * kTok);
        }
        __syncwarp();
        if (++stage == kRing) {
          stage = 0;
          round ^= 1;
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------------------------ MMA
    int stage = 0;
    uint32_t round = 0;
    bool ok = true;
    for (int i = 0; i < hi - lo && ok; ++i) {
      const int tokens = min(kTok, p.BT - (lo + i) * kTok);
      const uint32_t id = idesc(kDims, (tokens + 15) / 16 * 16, 0);
      if (i >= 2) ok = wait(bar(kDEmpty + (i & 1)), ((i >> 1) - 1) & 1, p.err, abort);
      for (int k = 0; k < kSlabs && ok; ++k) {
        ok = (i > 0 || wait(bar(kWFull + k), 0, p.err, abort)) &&
             wait(bar(kFull + stage), round, p.err, abort);
        if (!ok) break;
        tc_after();
        if (elect_one()) {
          const uint32_t a = w_lo + k * (kWSlab >> 4), b = b_lo + stage * (kStage >> 4);
          const uint32_t d = tmem + kTok * (i & 1);
#pragma unroll
          for (int s = 0; s < 8; ++s)  // the high term, then the low one
            mma1(d, a + 2 * (s & 3), b + (s >> 2) * (kTerm >> 4) + 2 * (s & 3), id,
                 (k > 0 || s > 0) ? 1u : 0u);
          tc_commit(bar(kEmpty + stage));
          if (k == kSlabs - 1) tc_commit(bar(kDFull + (i & 1)));
        }
        __syncwarp();
        if (++stage == kRing) {
          stage = 0;
          round ^= 1;
        }
      }
    }
  }
  if (warp >= 4 && warp < 8) {
    // ------------------------------------------------------------------------------- epilogue
    // A thread holds one dim of the tile's tokens; neighbours swap, so that each stores two dims
    // of every second token.
    if (!kMerge) wait_prior_grid();
    const int dim = dim0 + 32 * (warp & 3) + lane;
    const bool even = (lane & 1) == 0;
    for (int i = 0; i < hi - lo; ++i) {
      // tokens of sequences without rows (their latent rows were not written): zeros
      const int n0 = (lo + i) * kTok;
      uint32_t none[kTok / 32];
#pragma unroll
      for (int j = 0; j < kTok / 32; ++j) {
        const int mine = n0 + 32 * j + lane;
        const bool is = mine < p.BT && tree_length(p, mine / p.T, false) == 0;
        none[j] = __ballot_sync(0xffffffffu, is);
        if (is && dim0 == 0 && (warp & 3) == 0 && p.lse) p.lse[(size_t)mine * p.H + h] = -INFINITY;
      }
      if (!wait(bar(kDFull + (i & 1)), (i >> 1) & 1, p.err, abort)) break;
      tc_after();
      for (int c0 = 0; c0 < kTok && n0 + c0 < p.BT; c0 += 32) {
        uint32_t v[32];
        tmem_ld32(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + kTok * (i & 1) + c0, v);
        uint32_t empty = none[0];
#pragma unroll
        for (int j = 1; j < kTok / 32; ++j) empty = c0 == 32 * j ? none[j] : empty;
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          const uint32_t got = __shfl_xor_sync(0xffffffffu, even ? v[c + 1] : v[c], 1);
          const int n = n0 + c0 + c + (even ? 0 : 1);
          const bool zero = empty >> (c + (even ? 0 : 1)) & 1;
          const float x = zero ? 0.f : __uint_as_float(even ? v[c] : got);
          const float y = zero ? 0.f : __uint_as_float(even ? got : v[c + 1]);
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
      }
      tc_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kDEmpty + (i & 1)));
    }
  }
  __syncwarp();
  tc_before();
  __syncthreads();
  tc_after();
  if (*abort != 0) {  // loads and products under way without a wait for them end long before this
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < kSettleNs) {
    }
  }
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(2 * kTok)
                 : "memory");
}

// (n, H, 512) bf16 in boxes of 64 dims of one head, 128 tokens
bool latent_map(CUtensorMap* m, const void* base, int n, int H) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)kR, (cuuint64_t)H, (cuuint64_t)n};
  cuuint64_t strides[2] = {kR * 2, (cuuint64_t)H * kR * 2};
  cuuint32_t box[3] = {64, 1, kTok}, estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_tree_out(const TreeParams& p, const void* w_uv, int dv, void* o,
                            cudaStream_t st) {
  CUtensorMap w, hi, lo;
  if (!make_bf16_map(&w, w_uv, kR, (uint64_t)p.H * dv, kR * 2, kDims) ||
      !latent_map(&hi, p.latent_hi, p.BT, p.H) || !latent_map(&lo, p.latent_lo, p.BT, p.H))
    return cudaErrorInvalidValue;
  static std::atomic<unsigned long long> attr_devices{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? (1ull << dev) : 0ull;
  if (!bit || !(attr_devices.load(std::memory_order_acquire) & bit)) {
    for (auto k : {tree_out_kernel<false>, tree_out_kernel<true>}) {
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
      if (e != cudaSuccess) return e;
    }
    attr_devices.fetch_or(bit, std::memory_order_acq_rel);
  }
  // one CTA per 128 rows of W_UV; its tokens are split where that leaves SMs idle
  const int ctas = p.H * ((dv + kDims - 1) / kDims), tiles = (p.BT + kTok - 1) / kTok;
  // Up to 32 tokens the merge is done here: 1 x 8 tokens of 128 heads over 1000 rows take 22.9 us
  // against 27.9 with a merge kernel in between, 32768 rows 70.3 against 76.7, 8 x 4 over 1000 34.9
  // against 37.6, 8 x 4 of 16 heads over 4096 rows 41 against 45; 1 x 48 44.9 against 43.8 (a CTA
  // reads all partial results of its head).
  if (p.BT <= kMergeTok)
    return launch_pdl(tree_out_kernel<true>, dim3((unsigned)ctas), dim3(kMergeThreads), kSmem, st,
                      w, hi, lo, p, dv, 1, (__nv_bfloat16*)o);
  e = launch_pdl(tree_merge_parts_kernel,
                 dim3((unsigned)(p.ranges * p.team * (kTreeTile / kMergeWarps))),
                 dim3(kMergeWarps * 32), 0, st, p);
  if (e != cudaSuccess) return e;
  const int splits = ctas >= 148 ? 1 : (148 / ctas < tiles ? 148 / ctas : tiles);
  return launch_pdl(tree_out_kernel<false>, dim3((unsigned)(ctas * splits)), dim3(kThreads), kSmem,
                    st, w, hi, lo, p, dv, splits, (__nv_bfloat16*)o);
}

}  // namespace mla
