// Tensor-core attention of mla_decode_tree (bf16, r = 512, d_r = 64, cache blocks of a multiple of
// 64 rows, any number of heads), for sm_100a.
//
// A sequence's T drafted tokens and H heads are T * H query rows over the same cache rows. They
// are tiled by 128, whatever token or head a row belongs to; per tile of query rows
//   S = Q . K^T   (128 x keys, K = 576)      O += P . V   (128 x 512, K = keys; V = the latent
//                                                          part of the same rows)
// are dense contractions that a pair of SMs does together (cta_group::2, M = 128: each CTA of a
// cluster of two holds 64 query rows of Q, P, S and O in its own memories, and half of every
// B operand: half of the keys for S, half of the latent dims for O). So a CTA's O takes 256
// tensor-memory columns (its 64 rows in lanes 0-63 for one half of the dims and again in lanes
// 64-127 for the other), which leaves room for two buffers of S over 256 keys; and P stays in the
// SM that computed it: nothing but MMA operands crosses between the two.
//
// Per 256 keys a CTA streams 9 stages of K (128 keys x 64 dims) and 8 of V (64 keys x 128 dims), 16
// KB each, through a ring for each. One warp issues the score products and another P . V, so that
// P . V of a tile runs while the scores of the next are made, waited for and exponentiated. The
// whole warp runs the issue loop and one elected lane issues: from a single thread in a divergent
// branch an MMA took 132 cycles to issue whatever its size, with the warp converged and the
// descriptors' low words at hand 25.
//
// What bounds it. 32 sequences x 16384 rows x 4 tokens of 128 heads take 571 us when run for
// seconds, 1.02 PFLOP/s, 0.73 of the measured sustained rate (the power limit holds the clock near
// 1.4 GHz), and 477 to 509 us, by GPU, in bursts of a few. A tile takes about 7k cycles for 4.35k of
// products. Beside them its softmax takes 4.3k (scores out of TMEM and the maximum 1.7k,
// exponentials 1.7k, P 0.4k, waits), so that any instruction more in it shows: scores read twice to
// save registers 516 us against 493, exponentials begun before the two halves' maxima are exchanged
// 512. The operands come out of L2 at 40 bytes per clock and SM, 11.6 TB/s in all. More query rows
// per pair would halve the operands but for O, which fills the tensor memory beside S.
//
// Few heads (a tile of 128 rows half empty) are bound by the tile's own time, which is that of 128
// rows whatever part of them is real, and by the fixed parts: 3 x 32768 rows x 5 tokens of 16
// heads, 113 MB of cache rows, take 45 us here (2.5 TB/s) and 63 with the merge and W_UV. One short
// sequence is bound by latency: of 15 us for 8 tokens x 1000 rows the schedule takes 2, the first
// loads 1.5, a tile's scores, softmax and P . V 6, the partial results 3.
//
// Softmax: four warps, a thread holds one query row and half of the tile's keys (TMEM lane), two
// threads of a row exchange their maxima; base-2 exponents, the running maximum moved only when
// a tile exceeds it by 2^8, the sum l of the fp32 weights. The same warps rescale O when the
// maximum moves. At a segment's end four other warps write O / l, so that the softmax of the next
// segment goes on meanwhile.
//
// P is rounded to bf16, the type of V in the product: 2^-8 of each weight at most, of random sign,
// which takes the error of o against 64 bits from 1.66e-3 of its norm (its own rounding) to 2.05e-3
// for 8 tokens x 1000 rows, 1.75e-3 for 16384 rows. l adds the weights as they were before that:
// with the rounded ones o gained nothing (2.05e-3, 1.75e-3; 1.85e-3 instead of 2.06e-3 for scores
// four times as large), lse lost (1e-6 off against 1e-4 to 3e-3), and it took 492 us instead of
// 477.
//
// Rows that a token does not see: the prefix (rows before the drafted ones) is seen by all; for
// the drafted rows a thread builds the 32-bit words of its keys from its token's mask, and a
// masked score becomes -inf by selection. P = 0 times a masked row's V would still be NaN if the
// row held NaN, so the V stages that hold drafted rows (or rows past the end) pass through the
// finishing warps, which replace what is not finite by 0 before the MMA may read it.
//
// Warps: 0 TMA of Q and K, 3 of V; 1 issues S, 2 issues P . V (both in the pair's first CTA); 4-7
// softmax; 8-11 fix V and write O. Every wait is bounded: on timeout the kernel sets
// MLA_DEV_WAIT_TIMEOUT, lets what it issued end, frees TMEM and returns. No TMA multicast is used.
#include <atomic>

#include "plan_body.cuh"
#include "tc_ptx.cuh"
#include "tma_map.h"
#include "tree.cuh"
#include "tree_ptx.cuh"

namespace mla {
namespace {

constexpr int kR = 512;
constexpr int kDR = 64;
constexpr int kD = kR + kDR;
constexpr int kM = kTreeTile;             // query rows per pair of CTAs
constexpr int kMH = kM / 2;               // query rows per CTA
constexpr int kRows = 64;                 // cache rows per block of keys
constexpr int kTileBlocks = 4;            // blocks per tile: 256 keys
constexpr int kSlabBytes = 64 * 64 * 2;   // 64 rows x 64 dims bf16: 8 KB
constexpr int kStageBytes = 2 * kSlabBytes;
constexpr int kKRing = 4;                 // stages of the K ring
constexpr int kVRing = 3;                 // stages of the V ring
constexpr int kKStages = kD / 64;         // stages of a tile's K
constexpr int kQBytes = kKStages * kSlabBytes;
constexpr int kPBytes = kTileBlocks * kSlabBytes;
constexpr int kThreads = 384;             // three warpgroups: issue, softmax, finish
constexpr int kFinishWarps = 4;
// 168 registers a thread. (Moving registers to the softmax warps, which hold 128 scores, made the
// compiler spill more in all roles: 540 against 490 us for 32 x 16384 rows x 4 tokens.)
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;           // S buffers at columns 0 and 128
constexpr uint32_t kStageLo = kStageBytes >> 4, kSlabLo = kSlabBytes >> 4;  // in descriptors
constexpr unsigned long long kTimeoutNs = 1000000000ull;  // 1 s per wait
constexpr unsigned long long kSettleNs = 20000000ull;     // 20 ms after an abort

constexpr int kS_K = 0;
constexpr int kS_V = kS_K + kKRing * kStageBytes;         // 64 KB
constexpr int kS_Q = kS_V + kVRing * kStageBytes;         // 112 KB
constexpr int kS_P = kS_Q + kQBytes;                      // 184 KB
constexpr int kS_Red = kS_P + kPBytes;                    // 216 KB: max[2 tiles][2 halves][64]
constexpr int kS_Sum = kS_Red + 4 * kMH * 4;              // l[2 segments][2 halves][64]
constexpr int kS_Inv = kS_Sum + 4 * kMH * 4;              // 1 / l[2 segments][64]
constexpr int kS_Len = kS_Inv + 2 * kMH * 4;
constexpr int kLenCache = 256;
constexpr int kS_Plan = kS_Len + kLenCache * 4;           // 64 ints of the schedule's scans
constexpr int kS_Bar = kS_Plan + 64 * 4;

enum Bar {
  // in the first CTA only (the MMA warps wait): bytes and arrivals come from both CTAs
  kKFull = 0,                  // kKRing: both CTAs' parts of a stage landed
  kVFull = kKFull + kKRing,    // kVRing: ... or were fixed
  kQFull = kVFull + kVRing,    // both CTAs' query rows landed
  kSFree,                      // 2: softmax warps of both CTAs copied an S buffer out
  kPReady = kSFree + 2,        // 2: O rescaled and P's first half of the keys written in both
                               // CTAs; its second half written
  kOFree = kPReady + 2,        // O of the segment was read out in both CTAs
  // in each CTA
  kKEmpty,                     // kKRing: the MMAs reading a stage are complete
  kVEmpty = kKEmpty + kKRing,  // kVRing
  kQEmpty = kVEmpty + kVRing,  // the segment's last S is complete
  kSegDone,                    // the segment's last P . V is complete
  kLReady,                     // 2: 1 / l of an even / odd segment's rows is in shared memory
  kSFull = kLReady + 2,        // 2: an S buffer is complete
  kPvDone = kSFull + 2,        // 2: a tile's P . V is complete over the first half of the keys; all
  kRed = kPvDone + 2,          // the four softmax warps posted their maxima
  kSum,                        // ... their sums
  kFix,                        // kVRing: a stage to be fixed landed
  kFinal = kFix + kVRing,      // 2: all products of an MMA warp are complete
  kNumBars = kFinal + 2
};
constexpr int kSmemBytes = kS_Bar + kNumBars * 8 + 16 + 1024;  // + alignment to 1 KB
static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");

// ------------------------------------------------------------------------------ PTX helpers
// D[tmem of both CTAs] (+)= A[smem] . B[smem], descriptors by their low words
__device__ __forceinline__ void mma2(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t id,
                                     uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(id), "r"(acc), "r"(kDescHi)
      : "memory");
}
// arrives on the barrier at this offset in both CTAs of the pair once the MMAs issued before are
// complete
__device__ __forceinline__ void commit_both(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(bar), "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void commit_one(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}
// load into this CTA's shared memory, bytes counted on a barrier of either CTA of the pair
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                              int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst), "l"(map), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
// Arrival on a barrier of either CTA of the pair. CTA scope on purpose: a release of cluster scope
// waits for everything the thread has in flight (about 1000 cycles here). The memory model does not
// order across the two CTAs at that scope; that it suffices is an assumption about the hardware,
// the one that kernels on pairs of SMs usually make. What it rests on: no thread of the other CTA
// reads what the arrivals hand over, only the tensor core of the writer's own SM does (P and V in
// its shared memory, S and O in its tensor memory), and the writer has put that before the arrival
// itself (tcgen05.wait and fence::before_thread_sync, fence.proxy.async by each writing thread).
__device__ __forceinline__ void arrive_pair(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}

struct Ctl {
  uint32_t* err;
  volatile int* abort;
};

// Warp-collective bounded wait; the result is the same in all 32 lanes. Inlined whole: a call
// would spill the softmax warps' scores.
__device__ __forceinline__ bool wait_slow(uint32_t bar, uint32_t parity, uint32_t* err,
                                          volatile int* abort) {
  uint64_t t0 = 0;
  for (int it = 0;; ++it) {
    if (__all_sync(0xffffffffu, mbar_try_long(bar, parity))) return true;
    if (it == 0) t0 = globaltimer();
    const bool late = (globaltimer() - t0) > kTimeoutNs;
    if (__any_sync(0xffffffffu, *abort != 0 || late)) {
      if ((threadIdx.x & 31) == 0 && late) {
        set_error(err, MLA_DEV_WAIT_TIMEOUT);
        *abort = 1;
      }
      return false;
    }
  }
}
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, const Ctl& c) {
  if (__all_sync(0xffffffffu, mbar_try_long(bar, parity))) return true;
  return wait_slow(bar, parity, c.err, c.abort);
}
// Bounded wait for a phase that normally completed long ago (drains at teardown).
__device__ void drain(uint32_t bar, uint32_t parity, uint32_t* err) {
  const uint64_t t0 = globaltimer();
  bool done = false;
  while (!done && globaltimer() - t0 < kTimeoutNs)
    done = __all_sync(0xffffffffu, mbar_try(bar, parity));
  if (!done && (threadIdx.x & 31) == 0) set_error(err, MLA_DEV_WAIT_TIMEOUT);
}

// One tile: up to four consecutive 64-row chunks of one item.
struct Tile {
  int b, row0, chunk, nb, ntok, len, slot;
  bool first, last;
  __device__ int half_blocks() const { return nb > 2 ? 2 : 1; }  // blocks of keys per CTA
};

// Walks the tiles of the chunks [c, end) of the call's list, identically in every warp of both
// CTAs: the items' chunks lie end to end, so the next item's begin where this one's end.
struct TileWalk {
  const TreeParams* p;
  const int* lens;  // shared memory: rows of items first .. first + kLenCache - 1
  int first, member, range, begin, end;
  int it, x, len, c;  // current item, its first chunk and its rows; current chunk
  int b, row0, stop;  // its sequence, this member's first query row, its end
  bool idle;          // this member has no query rows in it
  __device__ __forceinline__ void enter() {
    b = it / p->groups;
    const int mt = (it - b * p->groups) * p->team + member;
    idle = mt >= p->tiles;
    row0 = mt * kM;
    stop = x + (len + kRows - 1) / kRows;
  }
  __device__ __forceinline__ bool next(Tile& tl) {
    while (c < end) {
      if (c >= stop) {
        x = stop;
        ++it;
        len = it - first < kLenCache ? lens[it - first] : tree_length(*p, it / p->groups, false);
        enter();
        continue;
      }
      const int to = min(stop, end);
      if (idle) {
        c = to;
        continue;
      }
      tl.b = b;
      tl.row0 = row0;
      tl.chunk = c - x;
      tl.nb = min(kTileBlocks, to - c);
      tl.len = len;
      tl.ntok = min(tl.nb * kRows, len - tl.chunk * kRows);
      // an item cut by the range leaves a partial result: a range has at most two, its first
      // and its last
      tl.slot = x >= begin && stop <= end
                    ? -1
                    : (2 * range + (x > begin ? 1 : 0)) * p->team + member;
      tl.first = c == max(x, begin);
      c += tl.nb;
      tl.last = c == to;
      return true;
    }
    return false;
  }
};

// First pool row of a sequence's 64-row chunks, 32 table entries read at a time: lane i holds
// that of chunk base + i. Blocks outside the pool are flagged at use; in place of their rows the
// load takes the rows in front of the pool, which read as zeros, and nobody sees them (InPool).
struct RowWindow {
  int b = -1, base = 0, blk = 0;
  __device__ int get(const TreeParams& p, int seq, int chunk, int lane) {
    const int per = p.bs / kRows;  // chunks per cache block
    const int at = chunk / per;
    if (seq != b || at < base || at >= base + 32) {  // warp-uniform
      b = seq;
      base = at;
      blk = at + lane < p.max_blocks ? p.table[(size_t)seq * p.max_blocks + at + lane] : 0;
    }
    const int id = __shfl_sync(0xffffffffu, blk, at - base);
    if (id < 0 || id >= p.num_blocks) {
      if (lane == 0) set_error(p.err, MLA_DEV_OOB_BLOCK);
      return -kRows;
    }
    return id * p.bs + (chunk - at * per) * kRows;
  }
};

// Whether a sequence's 64-row chunks lie in the pool, looked up for 32 at a time.
struct InPool {
  int b = -1, base = 0;
  uint32_t in = 0;  // bit i: chunk base + i
  // bit i: chunk + i, for a tile's chunks (those behind the table count as in the pool)
  __device__ uint32_t get(const TreeParams& p, int seq, int chunk, int lane) {
    if (seq != b || chunk < base || chunk + kTileBlocks > base + 32) {  // warp-uniform
      b = seq;
      base = chunk;
      const int at = (chunk + lane) / (p.bs / kRows);
      const int id = at < p.max_blocks ? p.table[(size_t)seq * p.max_blocks + at] : 0;
      in = __ballot_sync(0xffffffffu, id >= 0 && id < p.num_blocks);
    }
    return in >> (chunk - base);
  }
};

// A place in a ring of N stages: the stage, the parity of its use, and how many places lie before.
template <int N>
struct Cursor {
  int stage = 0;
  uint32_t round = 0;
  int used = 0;
  __device__ __forceinline__ void step() {
    ++used;
    if (++stage == N) {
      stage = 0;
      round ^= 1;
    }
  }
};

// Whether chunk j of a tile holds drafted rows or rows past the end: its V goes by the fixer.
__device__ __forceinline__ bool needs_fix(const Tile& tl, int j, int T) {
  return (tl.chunk + j + 1) * kRows > tl.len - T;
}

// Bits of the 32 keys from drafted node n0 on (negative: prefix rows, always seen) that token t of
// sequence b sees.
__device__ __forceinline__ uint32_t seen_word(const TreeParams& p, int b, int t, int n0) {
  if (n0 <= -32) return 0xffffffffu;
  auto word = [&](int w) -> uint32_t {  // nodes 32w .. 32w + 31
    if (w < 0 || 32 * w >= p.T) return 0;
    uint32_t m;
    if (p.mask) {
      m = p.mask[((size_t)b * p.T + t) * p.words + w];
    } else {
      m = 32 * w + 31 <= t ? 0xffffffffu : 32 * w > t ? 0 : 0xffffffffu >> (31 - (t & 31));
    }
    const int left = p.T - 32 * w;
    return left < 32 ? m & ((1u << left) - 1) : m;
  };
  if (n0 < 0) return (word(0) << -n0) | ((1u << -n0) - 1);
  const uint32_t lo = word(n0 >> 5), hi = word((n0 >> 5) + 1);
  return __funnelshift_r(lo, hi, n0 & 31);
}

// ------------------------------------------------------------------------------------------
// Schedule. Items are (sequence, group of `team` tiles of query rows); their 64-row chunks of keys
// are laid end to end and cut into R ranges of equal size, one per team of clusters. The members
// of a team walk the same chunks at the same time, each for its own tile of query rows, so the
// cache rows that several tiles need come from HBM once and from L2 for the others. Every CTA
// finds its own range here: a scan of the items' chunk counts, which costs less than a kernel of
// its own in front of this one (5-8 us). The cut items go into a list for the merge.
// ------------------------------------------------------------------------------------------
struct Range {
  int begin, end;  // chunks
  int item, x;     // the item that holds the first chunk, and that item's first chunk
};

// This thread's value summed over the threads up to it (returned) and over all of them.
__device__ int scan_chunks(int v, int* s_warp, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += s_warp[w];
    all += s_warp[w];
  }
  *total = all;
  return v + before;
}

__device__ Range plan_range(const TreeParams& p, int range, int* s_plan, int* s_len) {
  const int tid = threadIdx.x, items = p.batch * p.groups;
  int* s_found = s_plan + 32;  // item, x
  auto rows = [&](int it) {
    if (it >= items) return 0;
    const int b = it / p.groups;
    return tree_length(p, b, blockIdx.x == 0 && it == b * p.groups);
  };
  // all chunks of the call (with one pass of items, this scan is the one that places them too)
  const bool one = items <= kThreads;
  int len = 0, mine = 0, inc = 0, C = 0;
  for (int base = 0; base < items; base += kThreads) {
    int all;
    if (base > 0) __syncthreads();
    len = rows(base + tid);
    mine = (len + kChunk - 1) / kChunk;
    inc = scan_chunks(mine, s_plan, &all);
    C += all;
  }
  // A range holds two chunks at least, four where more would mean many partial results (each is
  // 256 KB): 8 tokens x 1000 rows took 32.4 us cut into single chunks, 32.0 into twos, 29.6 into
  // fours; 3 x 5 tokens of 16 heads x up to 1000 rows 28.9, 26.1 and 30.4.
  const uint32_t c = (uint32_t)C;  // up to 2^31 - 1
  const int R = min(p.ranges, (int)max((c + 3) / 4, min((c + 1) / 2, 32u / (uint32_t)p.team)));
  Range w{0, 0, 0, 0};
  // one CTA per range says whether an item that began in the range before goes on here
  const bool writer = range < p.ranges && (blockIdx.x & 1) == 0 && (blockIdx.x >> 1) % p.team == 0;
  if (range < R) {
    w.begin = first_chunk(range, R, C);
    w.end = first_chunk(range + 1, R, C);
  } else if (writer && tid == 0) {
    p.cuts[range] = make_int4(-1, 0, 0, 0);
  }
  int done = 0;
  for (int base = 0; base < items; base += kThreads) {
    const int it = base + tid;
    int all = 0;
    if (!one) {
      __syncthreads();
      len = rows(it);
      mine = (len + kChunk - 1) / kChunk;
      inc = scan_chunks(mine, s_plan, &all);
    }
    const int x = done + inc - mine, e = x + mine;
    done += all;
    if (mine > 0 && w.begin < w.end && x <= w.begin && w.begin < e) {
      s_found[0] = it;
      s_found[1] = x;
      if (writer) {
        int4 cut = make_int4(-1, 0, 0, 0);
        const int before = range > 0 ? first_chunk(range - 1, R, C) : 0;
        if (x < w.begin && x >= before) {
          const int last = starts_below(e, R, C) - 1;  // the range that holds its last chunk
          cut = make_int4(it, last - (range - 1) + 1, 2 * (range - 1) + (x > before ? 1 : 0), 0);
        }
        p.cuts[range] = cut;
      }
    }
  }
  if (w.begin < w.end) {  // the same in all threads
    __syncthreads();
    w.item = s_found[0];
    w.x = s_found[1];
    const int at = one ? tid - w.item : tid;  // one pass: the lengths are at hand
    if (at >= 0 && at < kLenCache && w.item + at < items) s_len[at] = one ? len : rows(w.item + at);
  }
  return w;
}

// Four lanes with 64 bytes each of a row of their own (w: four 16-byte pieces) change them round,
// so that lane i holds piece i of the group's rows, and write them: a store instruction then
// covers 64 bytes of eight rows. dst: the warp's row 0; only rows below `rows` are written.
__device__ __forceinline__ void put_rows(uint32_t (&w)[16], char* dst, int pitch, int rows,
                                         int lane) {
#pragma unroll
  for (int step = 1; step < 4; step <<= 1) {
    const bool up = lane & step;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (q & step) continue;  // pieces q and q + step change places across the pair
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t &a = w[4 * q + i], &b = w[4 * (q + step) + i];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? a : b, step);
        if (up) a = got;
        else b = got;
      }
    }
  }
  const int r0 = lane & ~3;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (r0 + k < rows)
      *(uint4*)(dst + (size_t)(r0 + k) * pitch + 16 * (lane & 3)) =
          make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
}

// the 16-byte piece with every bf16 that is not finite replaced by 0
__device__ __forceinline__ uint32_t finite2(uint32_t v) {
  if ((v & 0x7f80u) == 0x7f80u) v &= 0xffff0000u;
  if ((v & 0x7f800000u) == 0x7f800000u) v &= 0x0000ffffu;
  return v;
}

}  // namespace

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
tree_tc_kernel(const __grid_constant__ CUtensorMap tm_kv, const __grid_constant__ CUtensorMap tm_q,
               const __grid_constant__ TreeParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const uint32_t s_base = saddr(smem);
  uint32_t* tmem_slot = (uint32_t*)(smem + kS_Bar + kNumBars * 8);
  volatile int* abort_flag = (volatile int*)(smem + kS_Bar + kNumBars * 8 + 4);
  float* s_inv = (float*)(smem + kS_Inv);
  int* s_len = (int*)(smem + kS_Len);
  int* s_plan = (int*)(smem + kS_Plan);
  auto bar = [&](int i) { return s_base + kS_Bar + 8u * (uint32_t)i; };

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const Ctl ctl{p.err, abort_flag};

  if (threadIdx.x == 0) {
    for (int i = 0; i < kKRing; ++i) {
      mbar_init(bar(kKFull + i), 1);
      mbar_init(bar(kKEmpty + i), 1);
    }
    for (int i = 0; i < kVRing; ++i) {
      mbar_init(bar(kVFull + i), 2 * kFinishWarps);
      mbar_init(bar(kVEmpty + i), 1);
      mbar_init(bar(kFix + i), 1);
    }
    mbar_init(bar(kQFull), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kSFree + i), 8);
      mbar_init(bar(kSFull + i), 1);
    }
    mbar_init(bar(kPReady), 8);
    mbar_init(bar(kPReady + 1), 4);
    mbar_init(bar(kQEmpty), 1);
    mbar_init(bar(kSegDone), 1);
    mbar_init(bar(kLReady), 2);
    mbar_init(bar(kLReady + 1), 2);
    mbar_init(bar(kOFree), 2 * kFinishWarps);
    mbar_init(bar(kPvDone), 1);
    mbar_init(bar(kPvDone + 1), 1);
    mbar_init(bar(kRed), 4);
    mbar_init(bar(kSum), 4);
    for (int i = 0; i < 2; ++i) mbar_init(bar(kFinal + i), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     saddr(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  // this CTA's barriers are initialised; waited for behind the schedule, which hides the exchange
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  wait_prior_grid();  // the lengths, Q and the cache rows come from earlier kernels
  // The kernels behind may start on SMs that are done; they wait for this grid before they read
  // its results. Not before the wait above: what they read before theirs (W_UV) must be there.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int cluster = blockIdx.x >> 1;
  const int range = cluster / p.team, member = cluster - range * p.team;
  const Range work = plan_range(p, range, s_plan, s_len);
  tc_before();
  __syncthreads();
  tc_after();
  // barriers of both CTAs initialised before any remote traffic
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

  TileWalk walk{&p, s_len, work.item, member, range, work.begin, work.end,
                work.item, work.x, work.begin < work.end ? s_len[0] : 0, work.begin};
  walk.enter();
  Tile cur;
  bool has = walk.next(cur);

  if (warp >= 4 && warp < 8) {
    // ------------------------------------------------------------------------ softmax, rescale
    // TMEM lane 32 * quad + lane: query row `row` of this CTA, half `half` of the tile's keys
    // in S, and of each 256 latent dims in O
    const int quad = warp & 3, half = quad >> 1;
    const int row = 32 * (quad & 1) + lane;
    const uint32_t tq = tmem + ((uint32_t)(32 * quad) << 16);
    const float c2 = p.scale * 1.4426950408889634f;  // scores in log2 units
    float* red = (float*)(smem + kS_Red);
    float* sum = (float*)(smem + kS_Sum);
    const uint32_t p_row = s_base + kS_P + (uint32_t)(2 * half) * kSlabBytes + (uint32_t)row * 128;
    const uint32_t s_free = peer_addr(bar(kSFree), 0), p_ready = peer_addr(bar(kPReady), 0);
    int t = 0, seg = 0;
    float m_ref = 0.f, l = 0.f;
    InPool pool;
    while (has) {
      const int my_row = cur.row0 + kMH * (int)rank + row;  // of the sequence's T * H
      const int hb = cur.half_blocks();
      const int key0 = half * hb * kRows;  // this thread's first key of the tile
      const int lim = min(cur.ntok - key0, hb * kRows);
      const int node0 = cur.chunk * kRows + key0 - (cur.len - p.T);  // drafted node of column 0
      // this thread's blocks of keys that are in the pool
      const uint32_t in = pool.get(p, cur.b, cur.chunk, lane) >> (half * hb);
      const bool masked = lim < 128 || node0 + 127 >= 0 || (in & 3) != 3;
      uint32_t seen[4];
      if (masked) {
        const int tok = min(my_row / p.H, p.T - 1);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int left = lim - 32 * w;
          const uint32_t bits = left <= 0 ? 0u : seen_word(p, cur.b, tok, node0 + 32 * w);
          seen[w] = left <= 0 || !(in >> (w >> 1) & 1) ? 0u
                    : left < 32 ? bits & ((1u << left) - 1) : bits;
        }
      }
      if (!wait(bar(kSFull + (t & 1)), (t >> 1) & 1, ctl)) break;
      tc_after();
      uint32_t v[128];
      tmem_ld128(tq + 128u * (uint32_t)(t & 1), v);
      tc_before();
      __syncwarp();
      if (lane == 0) arrive_pair(s_free + 8u * (uint32_t)(t & 1));
      if (masked) {
#pragma unroll
        for (int w = 0; w < 4; ++w)
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (!(seen[w] >> k & 1)) v[32 * w + k] = 0xff800000u;
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int k = 0; k < 128; k += 8)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          mx[c] = fmax3(mx[c], __uint_as_float(v[k + 2 * c]), __uint_as_float(v[k + 2 * c + 1]));
      float* rt = red + (t & 1) * 2 * kMH;
      rt[half * kMH + row] = fmax3(mx[0], mx[1], fmaxf(mx[2], mx[3]));
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kRed));
      if (!wait(bar(kRed), t & 1, ctl)) break;
      // a row that sees nothing yet keeps a finite reference: all its weights are exp2(-inf) = 0
      const float mt = fmaxf(fmaxf(rt[row], rt[kMH + row]) * c2, -1e30f);
      float alpha = 1.f;
      if (cur.first) {
        m_ref = mt;
        l = 0.f;
      } else if (mt > m_ref + 8.f) {
        alpha = ex2(m_ref - mt);
        m_ref = mt;
      }
      const float2 c2x2 = make_float2(c2, c2), nm = make_float2(-m_ref, -m_ref);
      float2 s0 = make_float2(0.f, 0.f), s1 = make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < 64; ++k) {
        const float2 x = __ffma2_rn(
            make_float2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), c2x2, nm);
        const float2 e = make_float2(ex2(x.x), ex2(x.y));
        if (k & 1) s1 = __fadd2_rn(s1, e);
        else s0 = __fadd2_rn(s0, e);
        v[k] = pack_bf16(e.x, e.y);
      }
      l = l * alpha + ((s0.x + s0.y) + (s1.x + s1.y));
      // P's halves change hands one by one, so that the tensor core works on one while the other
      // is written. The first may be used once O is rescaled in all lanes, which takes all of the
      // previous tile's P . V: the second half's warps give their part of that before they wait
      // for their own half.
      const bool rescale = !cur.first && __any_sync(0xffffffffu, alpha != 1.f);
      if (t > 0 && !wait(bar(kPvDone), (t - 1) & 1, ctl)) break;
      if (rescale) {
        if (t > 0 && !wait(bar(kPvDone + 1), (t - 1) & 1, ctl)) break;
        tc_after();
#pragma unroll 1
        for (int ch = 0; ch < 8; ++ch) {
          uint32_t o[32];
          tmem_ld32(tq + kColO + 32 * ch, o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
          tmem_st32(tq + kColO + 32 * ch, o);
        }
        tmem_wait_st();
        tc_before();
      }
      if (half == 1) {
        __syncwarp();
        if (lane == 0) arrive_pair(p_ready);
        if (t > 0 && !wait(bar(kPvDone + 1), (t - 1) & 1, ctl)) break;
      }
      // P in the A-operand layout (K-major, 128-byte rows swizzled by row % 8)
#pragma unroll
      for (int cb = 0; cb < 2; ++cb) {
        if (cb < hb) {
#pragma unroll
          for (int u = 0; u < 8; ++u)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                             p_row + cb * kSlabBytes + 16u * (uint32_t)(u ^ (row & 7))),
                         "r"(v[32 * cb + 4 * u]), "r"(v[32 * cb + 4 * u + 1]),
                         "r"(v[32 * cb + 4 * u + 2]), "r"(v[32 * cb + 4 * u + 3])
                         : "memory");
        }
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) arrive_pair(p_ready + 8u * (uint32_t)half);

      if (cur.last) {
        // l with the row's other half of the keys; the finishing warps take over from here
        float* st = sum + (seg & 1) * 2 * kMH;
        st[half * kMH + row] = l;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kSum));
        if (!wait(bar(kSum), seg & 1, ctl)) break;
        if (half == 0) {
          const float total = st[row] + st[kMH + row];
          s_inv[(seg & 1) * kMH + row] = total == 0.f ? 0.f : 1.f / total;
          const float lse = (m_ref + __log2f(total)) * 0.6931471805599453f;
          if (cur.slot >= 0) p.part_lse[(size_t)cur.slot * kM + kMH * rank + row] = lse;
          else if (my_row < p.T * p.H && p.lse) p.lse[(size_t)cur.b * p.T * p.H + my_row] = lse;
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kLReady + (seg & 1)));
        }
        ++seg;
      }
      ++t;
      has = walk.next(cur);
    }
  } else if (warp >= 8) {
    // --------------------------------------------- fixes of V; O / l out at a segment's end
    Cursor<kVRing> at;
    uint32_t fixes = 0;  // per stage: parity of its next fix
    int seg = 0;
    bool ok = true;
    const uint32_t full0 = peer_addr(bar(kVFull), 0), o_free = peer_addr(bar(kOFree), 0);
    const int quad = warp & 3, half = quad >> 1, tid = threadIdx.x - 256;
    const uint32_t to_ = tmem + ((uint32_t)(32 * quad) << 16) + kColO;
    while (ok && has) {
      for (int j = 0; j < cur.nb && ok; ++j) {
        const bool fix = needs_fix(cur, j, p.T);
        // rows of the block: up to `from` are the prefix; from `to` on they lie past the end
        const int from = max(cur.len - p.T - (cur.chunk + j) * kRows, 0);
        const int to = min(cur.len - (cur.chunk + j) * kRows, kRows);
#pragma unroll 1
        for (int dh = 0; dh < 2; ++dh, at.step()) {
          if (!fix) continue;
          if (!wait(bar(kFix + at.stage), fixes >> at.stage & 1, ctl)) {
            ok = false;
            break;
          }
          fixes ^= 1u << at.stage;
          // 16-byte pieces of rows from .. 63 of both slabs, all reads before the writes
          uint4* st = (uint4*)(smem + kS_V + at.stage * kStageBytes);
          uint4 x[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const int i = 8 * from + tid + 128 * (u >> 1);
            if (i < 8 * to) x[u] = st[(u & 1) * (kSlabBytes / 16) + i];
          }
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const int i = 8 * from + tid + 128 * (u >> 1);
            uint4* at_ = st + (u & 1) * (kSlabBytes / 16) + i;
            if (i < 8 * to) {
              const uint4 y = make_uint4(finite2(x[u].x), finite2(x[u].y), finite2(x[u].z),
                                         finite2(x[u].w));
              if (x[u].x != y.x || x[u].y != y.y || x[u].z != y.z || x[u].w != y.w) *at_ = y;
            } else if (i < 8 * kRows) {
              *at_ = make_uint4(0, 0, 0, 0);
            }
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) arrive_pair(full0 + 8u * (uint32_t)at.stage);
        }
      }
      if (ok && cur.last) {
        // (the softmax may be one segment ahead, not two: it needs that one's P . V)
        if (!wait(bar(kLReady + (seg & 1)), (seg >> 1) & 1, ctl) ||
            !wait(bar(kSegDone), seg & 1, ctl))
          break;
        tc_after();
        const float inv = s_inv[(seg & 1) * kMH + 32 * (quad & 1) + lane];
        // A partial result stays in fp32; a finished one becomes two bf16 terms. Lane i of a
        // group of four ends up with piece i of the group's four rows (put_rows), so that 64
        // bytes of a row are written at a time.
        const bool cut = cur.slot >= 0;
        const int r0 = cur.row0 + kMH * (int)rank + 32 * (quad & 1);  // the warp's first row
        const int rows = cut ? 32 : p.T * p.H - r0;                   // rows to write
        const size_t row = cut ? (size_t)cur.slot * kM + kMH * rank + 32 * (quad & 1)
                               : (size_t)cur.b * p.T * p.H + r0;
        char* dst = cut ? (char*)(p.part_o + row * kR) : (char*)(p.latent_hi + row * kR);
        const int64_t lo = (char*)p.latent_lo - (char*)p.latent_hi;
        const int pitch = cut ? kR * 4 : kR * 2;
        // columns 32 ch ..: dims 256 (ch / 4) + 128 half + 32 (ch % 4)
#pragma unroll 1
        for (int ch = 0; ch < 8; ++ch) {
          uint32_t o[32];
          tmem_ld32(to_ + 32 * ch, o);
          const int dim = 256 * (ch >> 2) + 128 * half + 32 * (ch & 3);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * inv);
          uint32_t w[16];
          if (cut) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
#pragma unroll
              for (int i = 0; i < 16; ++i) w[i] = o[16 * u + i];
              put_rows(w, dst + 4 * dim + 64 * u, pitch, rows, lane);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float x = __uint_as_float(o[2 * i]), y = __uint_as_float(o[2 * i + 1]);
              w[i] = pack_bf16(x, y);
              o[i] = pack_bf16(x - __uint_as_float(w[i] << 16),
                               y - __uint_as_float(w[i] & 0xffff0000u));
            }
            put_rows(w, dst + 2 * dim, pitch, rows, lane);
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = o[i];
            put_rows(w, dst + 2 * dim + lo, pitch, rows, lane);
          }
        }
        tc_before();
        __syncwarp();
        if (lane == 0) arrive_pair(o_free);
        ++seg;
      }
      has = walk.next(cur);
    }
  } else {
    if (warp == 0) {
      // --------------------------------------------------------------------------- TMA: Q and K
      // Loads are counted on the first CTA's barriers: it expects the bytes of both CTAs.
      RowWindow win;
      Cursor<kKRing> at;
      int seg = 0;
      bool ok = true;
      const uint32_t bars0 = peer_addr(bar(0), 0);
      while (ok && has) {
        if (cur.first) {
          // the previous segment's S products are done with Q
          if (seg > 0 && !wait(bar(kQEmpty), (seg - 1) & 1, ctl)) break;
          if (elect_one()) {
            if (rank == 0) mbar_expect_tx(bar(kQFull), 2 * kQBytes);
            const int y = cur.b * p.T * p.H + cur.row0 + kMH * (int)rank;
#pragma unroll
            for (int k = 0; k < kKStages; ++k)
              tma_load_pair(s_base + kS_Q + k * kSlabBytes, &tm_q, bars0 + 8 * kQFull, 64 * k, y);
          }
          __syncwarp();
          ++seg;
        }
        // this CTA's blocks of keys; in place of one that the segment does not have, its last (the
        // scores are masked)
        const int hb = cur.half_blocks(), j0 = (int)rank * hb;
        const int y0 = win.get(p, cur.b, cur.chunk + min(j0, cur.nb - 1), lane);
        const int y1 = win.get(p, cur.b, cur.chunk + min(j0 + hb - 1, cur.nb - 1), lane);
#pragma unroll 1
        for (int k = 0; k < kKStages; ++k) {
          if (at.used >= kKRing && !wait(bar(kKEmpty + at.stage), at.round ^ 1, ctl)) {
            ok = false;
            break;
          }
#ifdef MLA_TEST_DROP_ARRIVE
          // test build only: the first pair never loads one stage, so the waits for it run out and
          // the kernel must report MLA_DEV_WAIT_TIMEOUT, let the rest end, free TMEM and return
          if (blockIdx.x < 2 && at.used == 2) {
            at.step();
            continue;
          }
#endif
          if (elect_one()) {
            const uint32_t full = bars0 + 8u * (uint32_t)(kKFull + at.stage);
            const uint32_t dst = s_base + kS_K + at.stage * kStageBytes;
            if (rank == 0) mbar_expect_tx(bar(kKFull + at.stage), 2 * hb * kSlabBytes);
            tma_load_pair(dst, &tm_kv, full, 64 * k, y0);
            if (hb > 1) tma_load_pair(dst + kSlabBytes, &tm_kv, full, 64 * k, y1);
          }
          __syncwarp();
          at.step();
        }
        has = walk.next(cur);
      }
    } else if (warp == 3) {
      // --------------------------------------------------------------------------------- TMA: V
      RowWindow win;
      Cursor<kVRing> at;
      bool ok = true;
      const uint32_t bars0 = peer_addr(bar(0), 0);
      while (ok && has) {
        for (int j = 0; j < cur.nb && ok; ++j) {
          const int y = win.get(p, cur.b, cur.chunk + j, lane);
          const bool fix = needs_fix(cur, j, p.T);
#pragma unroll 1
          for (int dh = 0; dh < 2; ++dh) {
            if (at.used >= kVRing && !wait(bar(kVEmpty + at.stage), at.round ^ 1, ctl)) {
              ok = false;
              break;
            }
            if (elect_one()) {
              const uint32_t dst = s_base + kS_V + at.stage * kStageBytes;
              const int x = 256 * dh + 128 * (int)rank;
              uint32_t full = bars0 + 8u * (uint32_t)(kVFull + at.stage);
              if (fix) {
                full = bar(kFix + at.stage);
                mbar_expect_tx(full, kStageBytes);
              } else if (rank == 0) {
                // all arrivals, which the finishing warps give otherwise
                mbar_arrive_n(bar(kVFull + at.stage), 2 * kFinishWarps - 1);
                mbar_expect_tx(bar(kVFull + at.stage), 2 * kStageBytes);
              }
              tma_load_pair(dst, &tm_kv, full, x, y);
              tma_load_pair(dst + kSlabBytes, &tm_kv, full, x + 64, y);
            }
            __syncwarp();
            at.step();
          }
        }
        has = walk.next(cur);
      }
    } else if (warp == 1 && rank == 0) {
      // ------------------------------------------------------------------------- MMA: S = Q . K^T
      Cursor<kKRing> at;
      int t = 0, seg = 0;
      bool ok = true;
      const uint32_t q_lo = desc_lo(s_base + kS_Q, 16), ring = desc_lo(s_base + kS_K, 16);
      while (ok && has) {
        if (cur.first) {
          if (!wait(bar(kQFull), seg & 1, ctl)) break;
          ++seg;
        }
        // the softmax warps copied out what this buffer held two tiles ago
        if (t >= 2 && !wait(bar(kSFree + (t & 1)), ((t >> 1) - 1) & 1, ctl)) break;
        const uint32_t d = tmem + 128u * (uint32_t)(t & 1);
        const uint32_t id = idesc(128, 128 * cur.half_blocks(), 0);
#pragma unroll 1
        for (int k = 0; k < kKStages; ++k) {
          if (!wait(bar(kKFull + at.stage), at.round, ctl)) {
            ok = false;
            break;
          }
          tc_after();
          if (elect_one()) {
            const uint32_t a = q_lo + kSlabLo * k, b = ring + kStageLo * at.stage;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mma2(d, a + 2 * i, b + 2 * i, id, (k > 0 || i > 0) ? 1u : 0u);
            commit_both(bar(kKEmpty + at.stage));
          }
          __syncwarp();
          at.step();
        }
        if (!ok) break;
        if (elect_one()) {
          commit_both(bar(kSFull + (t & 1)));
          if (cur.last) commit_both(bar(kQEmpty));
        }
        __syncwarp();
        ++t;
        has = walk.next(cur);
      }
    } else if (warp == 2 && rank == 0) {
      // -------------------------------------------------------------------------- MMA: O += P . V
      Cursor<kVRing> at;
      int t = 0, seg = 0;
      bool ok = true;
      const uint32_t p_lo = desc_lo(s_base + kS_P, 16), ring = desc_lo(s_base + kS_V, kSlabBytes);
      while (ok && has) {
        if (cur.first) {
          // the segment before was read out of O
          if (seg > 0 && !wait(bar(kOFree), (seg - 1) & 1, ctl)) break;
          ++seg;
        }
        const int hb = cur.half_blocks();
        // where P's block of keys j lies: the second half of the keys from slab 2 on
        const uint32_t slab = hb > 1 ? kSlabLo : 2 * kSlabLo;
        constexpr uint32_t id = idesc(128, 256, 1);
#pragma unroll 1
        for (int half = 0; half < 2 && ok; ++half) {
          ok = wait(bar(kPReady + half), t & 1, ctl);
          tc_after();
          const int to = half == 0 ? min(hb, cur.nb) : cur.nb;
#pragma unroll 1
          for (int j = half * hb; j < to && ok; ++j) {
#pragma unroll 1
            for (int dh = 0; dh < 2; ++dh) {
              if (!wait(bar(kVFull + at.stage), at.round, ctl)) {
                ok = false;
                break;
              }
              tc_after();
              if (elect_one()) {
                const uint32_t a = p_lo + slab * j, b = ring + kStageLo * at.stage;
                const uint32_t d = tmem + kColO + 128 * dh;
#pragma unroll
                for (int i = 0; i < 4; ++i)  // 16 keys per step; V MN-major: 2 KB apart
                  mma2(d, a + 2 * i, b + 128 * i, id, (cur.first && j == 0 && i == 0) ? 0u : 1u);
                commit_both(bar(kVEmpty + at.stage));
              }
              __syncwarp();
              at.step();
            }
          }
          if (ok && elect_one()) {
            commit_both(bar(kPvDone + half));
            if (half == 1 && cur.last) commit_both(bar(kSegDone));
          }
          __syncwarp();
        }
        ++t;
        has = walk.next(cur);
      }
    }
  }

  // ---------------------------------------------------------------------------------- teardown
  tc_before();
  __syncthreads();
  tc_after();
  if (*abort_flag != 0) {
    // some loads may be under way without a wait for them: each has landed long before this
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < kSettleNs) {
    }
  }
  if ((warp == 1 || warp == 2) && rank == 0) {
    // completes once every MMA that this warp issued is done
    if (elect_one()) commit_one(bar(kFinal + warp - 1));
    __syncwarp();
    drain(bar(kFinal + warp - 1), 0, p.err);
  }
  cluster_sync();  // no MMA, load or remote arrival of the pair is under way any more
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols)
                 : "memory");
}

bool tree_tc_supported(const mla_config& c) {
  return c.dtype == MLA_BF16 && c.kv_rank == kR && c.rope_dim == kDR && c.block_size % kRows == 0;
}

// Clusters that work together on one item: as many as there are tiles of query rows, if the teams
// then leave few of the 74 clusters idle, else a number that does.
void tree_team(int tiles, int* team, int* ranges) {
  int best = 1;
  for (int g = 2; g <= tiles && g <= kRanges; ++g) {
    const int groups = (tiles + g - 1) / g;
    // share of the clusters' time that is used: whole teams, and tiles in the last group
    const double used = (double)(g * (kRanges / g)) / kRanges * tiles / ((double)groups * g);
    if (used >= 0.94) best = g;
  }
  *team = best;
  *ranges = kRanges / best;
}

cudaError_t launch_tree_tc(const TreeParams& p, cudaStream_t st) {
  CUtensorMap kv, qm;
  if (!make_bf16_map(&kv, p.pool, kD, (uint64_t)p.num_blocks * p.bs, kD * 2, kRows) ||
      !make_bf16_map(&qm, p.q, kD, (uint64_t)p.BT * p.H, kD * 2, kMH))
    return cudaErrorInvalidValue;
  // the shared-memory attribute applies to the device current when it is set: once per device
  static std::atomic<unsigned long long> attr_devices{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? (1ull << dev) : 0ull;
  if (!bit || !(attr_devices.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(tree_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSmemBytes);
    if (e != cudaSuccess) return e;
    attr_devices.fetch_or(bit, std::memory_order_acq_rel);
  }
  return launch_pdl(tree_tc_kernel, dim3(2 * kRanges), dim3(kThreads), kSmemBytes, st, kv, qm, p);
}

}  // namespace mla
