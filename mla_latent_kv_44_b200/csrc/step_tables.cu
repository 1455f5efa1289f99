// mla_build_tables and mla_tree_masks: the integer work of a serving step, from the requests'
// lengths (and a drafted tree's parent indices) to the block tables, slot maps, masks and
// positions that the other calls read.
//
// build_tables. One thread-block cluster does the whole call in one launch, but for the slot map of
// long token lists (a second kernel's). Every CTA scans the
// requests (new tokens, blocks given back, blocks taken: three prefix sums) into its own shared
// memory, so that no offsets travel between CTAs; the CTAs then share the moves and the slot
// map. Three phases are separated by cluster barriers, because each reads what the one before
// wrote in global memory: blocks given back are pushed on the free stack; blocks taken come off
// its top into the table; slots are read from the table. Everything is placed by prefix sums,
// none by atomics: the same inputs give the same tables. A block moved is a thread's, which finds
// its request by a search in the prefix sums (a warp per request: 7.0 us instead of 4.0 for 64
// requests, 14.6 instead of 9.8 for 128 with 32 prompts among them).
// What bounds it: latency (a chain of dependent loads and two barriers) at decode sizes, 4.0 us for
// 64 requests; for prompts also the 16 B written per token (131,072 tokens: 10.2 us, 0.21 TB/s).
#include <algorithm>

#include "tree.cuh"

namespace mla {
namespace {

constexpr int kTabThreads = 1024, kTabSmall = 512;
constexpr int kTabMaxCtas = 8;  // portable cluster size

struct TableParams {
  const int32_t *seq_lens, *new_lens, *held;
  int32_t *table, *free_blocks;
  const int32_t* free_count;
  int32_t *held_out, *free_count_out, *cu, *seq_idx, *pos;
  int64_t* slots;
  uint32_t* err;
  int batch, max_blocks, num_blocks, bs, max_tokens;
  int per_thread;  // tokens per thread and pass: 1 or 4
  bool vec;        // four at a time, 16-byte stores
  bool map_apart;  // the slot map is the second kernel's
};

__device__ __forceinline__ void cluster_barrier(int ctas) {
  if (ctas == 1) {
    __syncthreads();
  } else {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
                 ::: "memory");
  }
}

// Token counts saturate here: above any max_tokens (at most 2^26), below overflow. A request's
// own count is capped at kTokenCap, so that every offset below 2^28 is exact.
constexpr int kTokenSat = 1 << 29, kTokenCap = 1 << 28;

// In place of the first new row: the request is an empty place of a padded batch, and its tokens
// are padding.
constexpr int kPadding = -2147483647 - 1;

// Inclusive scan of three ints over the CTA (a saturating); s holds 3 x 32 ints.
template <int NT>
__device__ void scan3(int* s, int& a, int& b, int& c) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int va = __shfl_up_sync(0xffffffffu, a, o), vb = __shfl_up_sync(0xffffffffu, b, o),
              vc = __shfl_up_sync(0xffffffffu, c, o);
    if (lane >= o) {
      a = min(a + va, kTokenSat);
      b += vb;
      c += vc;
    }
  }
  if (lane == 31) {
    s[warp] = a;
    s[32 + warp] = b;
    s[64 + warp] = c;
  }
  __syncthreads();
  if (warp < 3) {
    int v = lane < NT / 32 ? s[32 * warp + lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v = warp == 0 ? min(v + u, kTokenSat) : v + u;
    }
    s[32 * warp + lane] = v;
  }
  __syncthreads();
  if (warp > 0) {
    a = min(a + s[warp - 1], kTokenSat);
    b += s[32 + warp - 1];
    c += s[64 + warp - 1];
  }
  __syncthreads();
}

// One request as the phases see it.
struct Request {
  int len, fresh, held, want;
  bool ok;
};

__device__ __forceinline__ Request load_request(const TableParams& p, int b) {
  Request q;
  q.len = p.seq_lens[b];
  q.fresh = p.new_lens[b];
  q.held = p.held[b];
  q.ok = q.len >= 0 && (int64_t)q.len <= (int64_t)p.max_blocks * p.bs && q.fresh >= 0 &&
         (q.fresh <= q.len || q.len == 0) && q.held >= 0 && q.held <= p.max_blocks;
  q.want = q.ok ? (int)(((int64_t)q.len + p.bs - 1) / p.bs) : q.held;
  if (!q.ok) q.fresh = 0;
  return q;
}

// The last request with off <= i (offsets rise; off[0] <= i < off[batch]): the one that holds i.
__device__ __forceinline__ int holder(const int* off, int batch, int i) {
  int lo = 0, hi = batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (off[mid] <= i) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Tokens i0 .. i0 + per - 1: one search and one division for all of them while they stay in a
// request. cu: offsets of the requests; start_of(b): its first new row, -1 - row when it was not
// served, kPadding where its tokens are padding; `real` tokens in all.
template <typename F>
__device__ __forceinline__ void map_tokens(const TableParams& p, const int* cu, F start_of,
                                           int64_t i0, int per, int real) {
  int seq[4], row[4];
  int64_t slot[4];
  int b = -1, left = 0, r = 0, at = 0, in = 0, blk = -1;
  bool served = false, padding = false;
  if (p.vec && i0 + 4 <= real) {
    // four tokens of one request, as most are: everything follows from the first (a warp whose
    // lanes part here runs both ways, so a block's end inside the four stays on this one)
    const int i = (int)i0, lo = holder(cu, p.batch, i);
    const int start = start_of(lo);
    if (cu[lo + 1] - i >= 4 && start >= 0 && p.bs >= 4) {
      const int row0 = start + i - cu[lo], at0 = row0 / p.bs, in0 = row0 - at0 * p.bs;
      const int32_t* ids = p.table + (size_t)lo * p.max_blocks + at0;
      const bool ends = in0 + 4 > p.bs;
      const int id = __ldcg(ids), next = ends ? __ldcg(ids + 1) : id;
      if (id >= 0 && id < p.num_blocks && next >= 0 && next < p.num_blocks) {
        const int64_t a = (int64_t)id * p.bs + in0, b4 = (int64_t)next * p.bs + in0 - p.bs;
        int64_t at[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) at[u] = (in0 + u < p.bs ? a : b4) + u;
        *(int4*)(p.seq_idx + i0) = make_int4(lo, lo, lo, lo);
        *(int4*)(p.pos + i0) = make_int4(row0, row0 + 1, row0 + 2, row0 + 3);
        *(longlong2*)(p.slots + i0) = make_longlong2(at[0], at[1]);
        *(longlong2*)(p.slots + i0 + 2) = make_longlong2(at[2], at[3]);
        return;
      }
    }
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int i = (int)i0 + u;
    seq[u] = -1;
    row[u] = 0;
    slot[u] = -1;
    if (u >= per || i >= real) continue;
    bool look = false;
    if (left == 0) {  // the request that holds token i
      if (b >= 0) {
        ++b;
        while (cu[b + 1] <= i) ++b;
      } else {
        b = holder(cu, p.batch, i);
      }
      left = cu[b + 1] - i;
      const int from = start_of(b);
      served = from >= 0;
      padding = from == kPadding;
      r = padding ? 0 : (served ? from : -1 - from) + i - cu[b];
      at = r / p.bs;
      in = r - at * p.bs;
      look = true;
    } else if (in == p.bs) {
      in = 0;
      ++at;
      look = true;
    }
    if (look && served) {
      blk = __ldcg(p.table + (size_t)b * p.max_blocks + at);
      if (blk < 0 || blk >= p.num_blocks) {
        set_error(p.err, MLA_DEV_OOB_BLOCK);
        blk = -1;
      }
    }
    seq[u] = padding ? -1 : b;
    row[u] = padding ? 0 : r;
    if (served && blk >= 0) slot[u] = (int64_t)blk * p.bs + in;
    ++r;
    ++in;
    --left;
  }
  if (p.vec && i0 + 4 <= p.max_tokens) {
    *(int4*)(p.seq_idx + i0) = make_int4(seq[0], seq[1], seq[2], seq[3]);
    *(int4*)(p.pos + i0) = make_int4(row[0], row[1], row[2], row[3]);
    *(longlong2*)(p.slots + i0) = make_longlong2(slot[0], slot[1]);
    *(longlong2*)(p.slots + i0 + 2) = make_longlong2(slot[2], slot[3]);
  } else {
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (u < per && i0 + u < p.max_tokens) {
        p.seq_idx[i0 + u] = seq[u];
        p.pos[i0 + u] = row[u];
        p.slots[i0 + u] = slot[u];
      }
  }
}

template <int NT>
__global__ void __launch_bounds__(NT) build_tables_kernel(const TableParams p) {
  extern __shared__ int s_dyn[];
  int* s_cu = s_dyn;                    // batch + 1: new tokens before request b
  int* s_back = s_cu + p.batch + 1;     // batch + 1: blocks given back by earlier requests
  int* s_take = s_back + p.batch + 1;   // batch + 1: blocks due to earlier requests
  int* s_start = s_take + p.batch + 1;  // batch: as map_tokens takes it
  __shared__ int s_scan[96], s_carry[3];
  const int tid = threadIdx.x, lane = tid & 31;
  const int cta = blockIdx.x, ctas = gridDim.x;
  wait_prior_grid();

  // requests, scanned by every CTA
  const int count = p.free_count[0];
  if (tid < 3) s_carry[tid] = 0;
  for (int base = 0; base < p.batch; base += NT) {
    const int b = base + tid;
    int n = 0, back = 0, take = 0;
    if (b < p.batch) {
      const Request q = load_request(p, b);
      if (!q.ok && cta == 0) set_error(p.err, MLA_DEV_BAD_LENGTH);
      n = min(q.fresh, kTokenCap);
      back = max(q.held - q.want, 0);
      take = max(q.want - q.held, 0);
      s_start[b] = !q.ok ? 0 : q.len == 0 ? kPadding : q.len - q.fresh;
    }
    int a0 = n, a1 = back, a2 = take;
    scan3<NT>(s_scan, a0, a1, a2);
    if (b < p.batch) {
      s_cu[b] = min(s_carry[0] + a0, kTokenSat) - n;
      s_back[b] = s_carry[1] + a1 - back;
      s_take[b] = s_carry[2] + a2 - take;
    }
    __syncthreads();
    if (tid == NT - 1) {
      s_carry[0] = min(s_carry[0] + a0, kTokenSat);
      s_carry[1] += a1;
      s_carry[2] += a2;
    }
    __syncthreads();
  }
  const int tokens = s_carry[0], backs = s_carry[1], takes = s_carry[2];
  if (tid == 0) {
    s_cu[p.batch] = tokens;
    s_back[p.batch] = backs;
    s_take[p.batch] = takes;
  }
  __syncthreads();
  // a stack that cannot be one: no block moves
  const bool stack_ok = count >= 0 && count <= p.num_blocks && backs <= p.num_blocks - count;
  if (!stack_ok && cta == 0 && tid == 0) set_error(p.err, MLA_DEV_BAD_LENGTH);
  const int stack = stack_ok ? count + backs : 0;

  // blocks given back, in (request, index) order: a thread per block, whoever's it was
  const int gtid = cta * NT + tid, threads = ctas * NT;
  if (backs > 0) {
    if (stack_ok) {
      for (int i = gtid; i < backs; i += threads) {
        const int b = holder(s_back, p.batch, i), kept = p.held[b] - (s_back[b + 1] - s_back[b]);
        p.free_blocks[count + i] = p.table[(size_t)b * p.max_blocks + kept + i - s_back[b]];
      }
    }
    cluster_barrier(ctas);
  }

  // blocks taken: the k-th off the top; a request whose share runs past the bottom gets none
  const int most = min(takes, stack);
  for (int i0 = gtid; i0 < most; i0 += 4 * threads) {
    int blk[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + u * threads;
      blk[u] = i < most ? __ldcg(p.free_blocks + (stack - 1 - i)) : 0;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + u * threads;
      if (i >= most) break;
      const int b = holder(s_take, p.batch, i);
      if (s_take[b + 1] > stack) break;  // nor any later one
      if (blk[u] < 0 || blk[u] >= p.num_blocks) set_error(p.err, MLA_DEV_OOB_BLOCK);
      p.table[(size_t)b * p.max_blocks + p.held[b] + i - s_take[b]] = blk[u];
    }
  }
  for (int b = tid; b < p.batch; b += NT) {
    if (s_take[b + 1] > max(s_take[b], stack)) {
      s_start[b] = -1 - s_start[b];
      if (cta == 0) set_error(p.err, MLA_DEV_NO_BLOCKS);
    }
  }
  cluster_barrier(ctas);  // the table is complete, and held and free_count are read

  // counts
  if (cta == 0) {
    int last = 0;  // blocks taken by the requests that were served
    for (int b = tid; b < p.batch; b += NT) {
      const bool served = s_start[b] >= 0;
      const int take = served ? s_take[b + 1] - s_take[b] : 0;
      if (take > 0) last = max(last, s_take[b + 1]);
      p.held_out[b] = p.held[b] + take -
                      (stack_ok ? s_back[b + 1] - s_back[b] : 0);
      p.cu[b] = min(s_cu[b], p.max_tokens);
    }
    last = __reduce_max_sync(0xffffffffu, last);
    if (lane == 0) s_scan[tid >> 5] = last;
    __syncthreads();
    if (tid < 32) {
      last = __reduce_max_sync(0xffffffffu, tid < NT / 32 ? s_scan[tid] : 0);
      if (tid == 0) {
        p.free_count_out[0] = stack_ok ? stack - last : count;
        p.cu[p.batch] = min(tokens, p.max_tokens);
        if (tokens > p.max_tokens) set_error(p.err, MLA_DEV_BAD_LENGTH);
      }
    }
  }

  // tokens
  if (p.map_apart) return;
  const int per = p.per_thread, real = min(tokens, p.max_tokens);
  for (int64_t i0 = (int64_t)gtid * per; i0 < p.max_tokens; i0 += (int64_t)threads * per)
    map_tokens(p, s_cu, [&](int b) { return s_start[b]; }, i0, per, real);
}

// The slot map of long token lists, over the whole GPU: what a request was given follows from the
// first kernel's results (served: as many blocks held as its rows need).
constexpr int kMapThreads = 256;

__global__ void __launch_bounds__(kMapThreads) slot_map_kernel(const TableParams p) {
  extern __shared__ int s_cu[];
  wait_prior_grid();
  for (int b = threadIdx.x; b <= p.batch; b += kMapThreads) s_cu[b] = p.cu[b];
  __syncthreads();
  const int64_t i0 = ((int64_t)blockIdx.x * kMapThreads + threadIdx.x) * p.per_thread;
  if (i0 >= p.max_tokens) return;
  map_tokens(
      p, s_cu,
      [&](int b) {
        const int len = p.seq_lens[b], start = len - p.new_lens[b];
        if (len == 0) return kPadding;
        return (int64_t)p.held_out[b] * p.bs >= len ? start : -1 - start;
      },
      i0, p.per_thread, s_cu[p.batch]);
}

}  // namespace

cudaError_t launch_build_tables(const int32_t* seq_lens, const int32_t* new_lens, int batch,
                                int32_t* table, int max_blocks, int bs, const int32_t* held,
                                int32_t* free_blocks, const int32_t* free_count, int num_blocks,
                                int32_t* held_out, int32_t* free_count_out, int32_t* cu,
                                int32_t* seq_idx, int32_t* pos, int64_t* slots, int max_tokens,
                                uint32_t* err, cudaStream_t st) {
  // one token per thread while that takes one pass of one CTA, else four; and lists that take
  // the cluster more than one pass go to a kernel of their own (131,072 tokens: 17.0 us in the
  // cluster alone)
  const int per = max_tokens <= kTabSmall ? 1 : 4;
  const bool vec = per == 4 && (((uintptr_t)seq_idx | (uintptr_t)pos | (uintptr_t)slots) & 15) == 0;
  const bool apart = max_tokens > kTabMaxCtas * kTabThreads * 4;
  TableParams p{seq_lens, new_lens, held,  table, free_blocks, free_count, held_out,
                free_count_out, cu, seq_idx, pos, slots, err, batch, max_blocks, num_blocks, bs,
                max_tokens, per, vec, apart};
  const size_t smem = sizeof(int) * (4 * (size_t)batch + 3);
  // (the limit of 48 KB without this covers the kernel's static shared memory too)
  if (smem > 40 * 1024) {
    static std::atomic<unsigned long long> devices{0};
    const cudaError_t e =
        raise_smem_limit((const void*)build_tables_kernel<kTabThreads>, devices);
    if (e != cudaSuccess) return e;
  }
  // one CTA while a pass of it covers the tokens and the requests, else a full cluster. A CTA of
  // 512 threads where that is enough: 64 requests take 4.0 us (1024 threads 4.5, 256 4.4), 128
  // with 32 prompts 9.8 (10.2, 13.1).
  const bool small = (apart || max_tokens <= 4 * kTabSmall) && batch <= kTabSmall;
  const int ctas =
      (apart || max_tokens <= 4 * kTabThreads) && batch <= kTabThreads ? 1 : kTabMaxCtas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(small ? kTabSmall : kTabThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  cudaError_t e = small ? cudaLaunchKernelEx(&cfg, build_tables_kernel<kTabSmall>, p)
                        : cudaLaunchKernelEx(&cfg, build_tables_kernel<kTabThreads>, p);
  if (e == cudaSuccess && apart)
    e = launch_pdl(slot_map_kernel, dim3((max_tokens + 4 * kMapThreads - 1) / (4 * kMapThreads)),
                   dim3(kMapThreads), sizeof(int) * ((size_t)batch + 1), st, p);
  return e;
}

// ------------------------------------------------------------------------------------------
// tree_masks: A_t = {t} u A_parent(t), and pos_t = seq_len - T + |A_t| - 1. One thread per node
// walks up its ancestors in shared memory: random trees of T nodes are O(log T) deep, and a
// chain of 256 costs 256 shared-memory reads. Several sequences share a CTA when T is small. What
// bounds it: latency (32 x 4 nodes 1.5 us, 128 x 64 nodes 1.9).
// ------------------------------------------------------------------------------------------
namespace {

template <int W>
__global__ void __launch_bounds__(256)
tree_masks_kernel(const int32_t* __restrict__ parents, int parents_batch,
                  const int32_t* __restrict__ seq_lens, int batch, int T, uint32_t* mask,
                  int32_t* pos, uint32_t* err) {
  __shared__ int s_parent[256];
  wait_prior_grid();
  const int per = 256 / T;  // sequences per CTA (T <= 256)
  const int k = threadIdx.x / T, t = threadIdx.x - k * T;
  const int b = blockIdx.x * per + k;
  const bool live = k < per && b < batch;
  int len = 0;
  if (live) {
    int a = parents[(parents_batch == 1 ? 0 : (size_t)b * T) + t];
    len = seq_lens[b];
    if (a < -1 || a >= t) {  // what an empty place holds is no error
      if (len != 0) set_error(err, MLA_DEV_BAD_TREE);
      a = -1;
    }
    s_parent[threadIdx.x] = a;
  }
  __syncthreads();
  if (!live) return;
  uint32_t w[W];
#pragma unroll
  for (int i = 0; i < W; ++i) w[i] = 0;
  int depth = -1;
  for (int a = t; a >= 0; a = s_parent[k * T + a]) {
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (W == 1 || i == (a >> 5)) w[i] |= 1u << (a & 31);
    ++depth;
  }
  const size_t n = (size_t)b * T + t;
  const int words = (T + 31) / 32;
#pragma unroll
  for (int i = 0; i < W; ++i)
    if (i < words) mask[n * words + i] = w[i];
  const bool bad = len < T;
  if (bad && len != 0 && t == 0) set_error(err, MLA_DEV_BAD_LENGTH);
  pos[n] = bad ? 0 : len - T + depth;
}

}  // namespace

cudaError_t launch_tree_masks(const int32_t* parents, int parents_batch, const int32_t* seq_lens,
                              int batch, int T, uint32_t* mask, int32_t* pos, uint32_t* err,
                              cudaStream_t st) {
  const int per = 256 / T;
  const dim3 grid((batch + per - 1) / per);
  const int words = (T + 31) / 32;
  if (words == 1)
    return launch_pdl(tree_masks_kernel<1>, grid, dim3(256), 0, st, parents, parents_batch,
                      seq_lens, batch, T, mask, pos, err);
  if (words == 2)
    return launch_pdl(tree_masks_kernel<2>, grid, dim3(256), 0, st, parents, parents_batch,
                      seq_lens, batch, T, mask, pos, err);
  if (words <= 4)
    return launch_pdl(tree_masks_kernel<4>, grid, dim3(256), 0, st, parents, parents_batch,
                      seq_lens, batch, T, mask, pos, err);
  return launch_pdl(tree_masks_kernel<8>, grid, dim3(256), 0, st, parents, parents_batch,
                    seq_lens, batch, T, mask, pos, err);
}

}  // namespace mla
