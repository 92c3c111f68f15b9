// Paged attention of prompt chunks on pairs of SMs (D = 512, bf16 rows).
//
// For a query row q (a head of a token) and the rows k_i that its token sees:
//   out = sum_i e^{s q.k_i - M} k_i / (sum_i e^{s q.k_i - M} + e^{sink - M})
//
// Neighbouring tokens of a sequence see almost the same rows, so one load of a
// row can serve several of them; what limits how many is TMEM, where an fp32
// output row takes 512 columns.  A cluster of two CTAs works on 128 query rows
// (two tokens of 64 heads, or more tokens of fewer heads): each CTA holds the
// queries, probabilities and outputs of 64, and tcgen05.mma.cta_group::2 shares
// the rows between the two tensor cores: each CTA loads half of every operand.
//   S[128, 256 rows]  = Q K^T      M 128, N 256, K 512: CTA c loads rows 128 c ..
//   O[128, 512]      += P V        M 128, 2 x N 256, K 256: CTA c loads dims 128 c ..
//                                  of each 256
// In TMEM an M = 128 pair accumulator has row l % 64 of a CTA in lane l, columns
// [0, N/2) in lanes 0-63 and [N/2, N) in lanes 64-127: O takes 256 columns, two
// S buffers 128 each, all 512.
//
// K and V stream through a ring of four 16 KB stages each (4 MMAs a stage): K as
// 128 rows x 64 dims, V as 64 rows x 128 dims.  Each has a producer and an
// issuer of its own (one thread cannot issue the copies of both, at about 100
// cycles a copy).  S(t + 2) is issued behind PV(t), so that the tensor pipe has it
// to do while the softmax of tile t + 1, which holds its probabilities in registers
// until PV(t) is done with P, writes them.  Eight warps share the softmax, two on
// each scheduler, so that one's waits cover the other's.
//
// Clusters are persistent and take every n-th pair of token groups (an item).
// Tiles follow one another over the items, and one warp looks the items up ahead
// of the others, so the next queries, keys and logits are there while an item's
// output is written.
//
// Rows that some tokens of the pair see and others do not (the ends of a window,
// the causal diagonal, an unfilled block) need care where they may hold NaN or
// were never written: the logits of the tokens that do not see them are masked,
// but their zero probability times a NaN is a NaN.  Two warps patch such V blocks
// in shared memory before the MMAs read them: rows that no token sees become
// zeros, and in rows that some see non-finite elements do (a token that does see
// the row gets its NaN from the logits).
//
// 2 sequences, 1,918 new tokens of 64 heads over the 3,200 to 5,100 rows up to each:
// 856 us, 1,240 TFLOP/s (0.75 of the measured bf16 matrix rate); under the power cap
// a long run settles at 990 us.  The bound is the tensor pipe's operand reads: a tile of 256
// rows moves 672 KB through each SM's shared memory for 64 MMAs, which take 90 to 100
// cycles each where bare ones take 64, and an item's ends (the patch of its diagonal
// blocks, its output) leave the pipe idle for some 10,000 cycles.
#include <algorithm>
#include <cstring>
#include <cuda_bf16.h>
#include <math_constants.h>
#include "common.cuh"
#include "tc.cuh"
#include "tmap.cuh"
#include "paged.cuh"

namespace csa {

static __device__ uint32_t g_err_pair;

uint32_t read_clear_err_pair() {
  uint32_t v = 0, z = 0;
  cudaMemcpyFromSymbol(&v, g_err_pair, sizeof(v));
  cudaMemcpyToSymbol(g_err_pair, &z, sizeof(z));
  return v;
}

namespace {

constexpr int kD = 512;
constexpr int kBlock = 64;                 // rows of a block: one page box, one slab of P
constexpr int kTileBlocks = 4;             // 256 rows a tile
constexpr int kStages = 4;                 // of each ring
constexpr uint32_t kStage = 16384;         // K: [128 rows][64 dims], V: [2 x 64 dims][64 rows]
constexpr int kKStages = 8;                // stages of a tile's K; its V has two for each block
constexpr uint32_t kSlab = 8192;           // 64 rows x 128 bytes
// warps 0-7 softmax and output, 8 loads Q and K, 11 loads V, 9 issues S and 10 PV
// (in CTA 0), 12 and 13 patch V blocks, 14 looks up items
constexpr int kThreads = 480;
constexpr int kSoft = 256;                 // threads of the softmax
constexpr float kTau = 8.0f;               // lazy-rescale threshold (log2 units)
constexpr uint32_t kSCol = 256;            // S buffers behind the 256 columns of O
constexpr int kItems = 4;                  // items that are looked up ahead

// ---------------------------------------------------------------- pair primitives
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Arrive on the barrier at this offset in CTA 0's shared memory.  The barriers
// of a pair announce shared memory that only the tensor cores read (written by
// TMA, or by threads that fenced it for the async proxy), so arrivals release and
// waits acquire at CTA scope: a cluster-scope release costs 1,000 cycles and more
// each, which 16 stages a tile paid one after another (20,000 cycles a tile).
__device__ __forceinline__ void arrive_leader(uint64_t* bar) {
  asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, 0;\n\t"
               "mbarrier.arrive.shared::cluster.b64 _, [a];\n\t}"
               :: "r"(smem_u32(bar)) : "memory");
}
// Bounded wait on a barrier of this CTA's; gives up after kWaitNs or once
// another warp of the CTA has.  Only the first try is inlined, and the roles'
// loops are not unrolled: seven roles' code shares the instruction caches, and a
// third of the fetches from them missed (chunk over all raw rows 925 us, 870 so).
__device__ __noinline__ bool wait_long(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  uint64_t start = 0;
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63u) == 0) {
      if (*abort_flag) return false;
      const uint64_t now = global_ns();
      if (start == 0) start = now;
      else if (now - start > kWaitNs) break;
    }
  }
  *abort_flag = 1;
  atomicOr(&g_err_pair, DEV_ERR_TIMEOUT_MBAR);
  return false;
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  return mbar_try_wait(bar, parity) || wait_long(bar, parity, abort_flag);
}
// The same, announcing `bytes` of copies that complete there.
__device__ __forceinline__ void expect_leader(uint64_t* bar, uint32_t bytes) {
  asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, 0;\n\t"
               "mbarrier.arrive.expect_tx.shared::cluster.b64 _, [a], %1;\n\t}"
               :: "r"(smem_u32(bar)), "r"(bytes) : "memory");
}
// Tiled copy into this CTA's shared memory that completes on CTA 0's barrier.
__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* map, int32_t x, int32_t y, uint64_t* bar) {
  asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %4, 0;\n\t"
               "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
               " [%0], [%1, {%2, %3}], [a];\n\t}"
               :: "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar))
               : "memory");
}
// The same for a whole warp, with one answer.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  return __all_sync(0xffffffffu, wait(bar, parity, abort_flag));
}
// A V block's copy in this CTA alone, completing on a barrier of its own.
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z, int32_t u,
                                           uint64_t* bar) {
  asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
               " [%0], [%1, {%2, %3, %4, %5}], [%6];"
               :: "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(u),
                  "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tma_load_pair_4d(void* dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z,
                                                int32_t u, uint64_t* bar) {
  asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %6, 0;\n\t"
               "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
               " [%0], [%1, {%2, %3, %4, %5}], [a];\n\t}"
               :: "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(u),
                  "r"(smem_u32(bar)) : "memory");
}
// MMAs and their commits are issued by whole warps in convergent code, with the
// instruction itself predicated on one elected lane: descriptors then stay in
// uniform registers, and 8 MMAs with a wait and a commit issue at the tensor
// pipe's rate (65 cycles an MMA; from a branch that one lane takes, 84 in a bare
// loop).
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
               "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
               :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc));
}
// Arrive on *bar in both CTAs when every MMA issued by the elected lane so far is done.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
               "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}"
               :: "r"(smem_u32(bar)), "h"((uint16_t)3) : "memory");
}
__device__ __forceinline__ void st_shared16(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" :: "r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ float exp2_fast(float x) {     // flushes results below 2^-126 to zero
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}
// Non-finite bf16 halves of a word become zeros.
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
  const uint32_t lo = (w & 0x7f80u) == 0x7f80u ? 0u : w & 0xffffu;
  const uint32_t hi = (w & 0x7f800000u) == 0x7f800000u ? 0u : w & 0xffff0000u;
  return lo | hi;
}

// Two float32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(reinterpret_cast<unsigned long long&>(r))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
        "l"(reinterpret_cast<unsigned long long&>(c)));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(reinterpret_cast<unsigned long long&>(r))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return r;
}

// An item: up to 2 tpc neighbouring tokens of a sequence, and the blocks of 64
// rows that they see, raw rows first, then entries.
struct Work {
  int has;                      // 0: no item (the batch is done)
  int seq, tpc;                 // tokens per CTA
  int64_t tok0, pos0;           // first token: row of the batch, position
  int ntok;                     // tokens of the pair
  int wb0;                      // first block of raw rows
  int nbw, nb;                  // blocks of raw rows, all blocks
  int any_lo[2], any_hi[2];     // rows of each source that some token sees ...
  int all_lo[2], all_hi[2];     // ... and that every token sees
};

// Rows [lo, hi) of source s (0 raw, 1 entries) that a query at position pos sees;
// a table names fewer than 2^31 rows.
__device__ __forceinline__ void seen(const PairParams& p, int s, int64_t pos, int& lo, int& hi) {
  lo = hi = 0;
  if (p.rows[s] == nullptr || pos < 0) return;
  if (s == 0) {
    hi = (int)min(p.cap[0], pos + 1);
    lo = p.W == 0 ? 0 : (int)min((int64_t)hi, max((int64_t)0, pos - p.W + 1));
  } else {
    const int64_t n = pos < 0x7fffffff ? (int64_t)((uint32_t)(pos + 1) / (uint32_t)p.m) : (pos + 1) / p.m;
    hi = (int)min(p.cap[1], n);
  }
}
// Source and first row of block kb.
__device__ __forceinline__ int block_at(const Work& w, int kb, int& row) {
  const int s = kb < w.nbw ? 0 : 1;
  row = (s == 0 ? w.wb0 + kb : kb - w.nbw) * kBlock;
  return s;
}
// Whether every token of the pair sees every row of block kb.
__device__ __forceinline__ bool block_clean(const Work& w, int kb) {
  int row;
  const int s = block_at(w, kb, row);
  return row >= (s ? w.all_lo[1] : w.all_lo[0]) && row + kBlock <= (s ? w.all_hi[1] : w.all_hi[0]);
}

// Tensor maps: the queries as [rows, 512], boxes of 64 x 64; each page store for
// K as [rows, 512], boxes of (at most 64 rows of a page) x 64, and for V as
// [2 of 256 dims][4 of 64][rows][64], boxes of 1 x 2 x rows x 64: a V stage is one
// copy.
struct PairMaps {
  CUtensorMap q, k[2], v[2];
};

// Tile `x` of the batch, counted from the last tile of the last sequence (the
// longest rows of a sequence come first, which leaves short tiles for the end).
// Whole-warp call.
__device__ __forceinline__ void find_work(const PairParams& p, int64_t x, int lane, Work& w) {
  w.has = 0;
  w.ntok = w.nb = w.nbw = 0;
  w.tpc = max(1, 64 / p.H);
  const int per = 2 * w.tpc;
  for (int b0 = p.n_seq - 1; b0 >= 0; b0 -= 32) {
    const int b = b0 - lane;
    int len = 0;
    if (b >= 0) len = seq_len(p.cu_q, b, p.n_tok);
    const int tiles = (len + per - 1) / per;
    int inc = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, x < inc);
    if (hit == 0) {
      x -= __shfl_sync(0xffffffffu, inc, 31);
      continue;
    }
    const int l = __ffs(hit) - 1;
    const int before = __shfl_sync(0xffffffffu, inc - tiles, l);
    const int n = __shfl_sync(0xffffffffu, tiles, l);
    len = __shfl_sync(0xffffffffu, len, l);
    w.seq = b0 - l;
    const int t = n - 1 - (int)(x - before);                 // tile of the sequence
    w.tok0 = (int64_t)p.cu_q[w.seq] + (int64_t)t * per;
    w.ntok = min(per, len - t * per);
    w.pos0 = p.q_pos[w.seq] + (int64_t)t * per;
    w.has = 1;
    const int64_t last = w.pos0 + w.ntok - 1;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      int z;
      seen(p, s, max(w.pos0, (int64_t)0), w.any_lo[s], z);
      seen(p, s, last, z, w.any_hi[s]);
      seen(p, s, last, w.all_lo[s], z);
      seen(p, s, w.pos0, z, w.all_hi[s]);
    }
    w.wb0 = w.any_lo[0] / kBlock;
    w.nbw = w.any_hi[0] > w.any_lo[0] ? (w.any_hi[0] + kBlock - 1) / kBlock - w.wb0 : 0;
    w.nb = w.nbw + (w.any_hi[1] + kBlock - 1) / kBlock;
    return;
  }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
pair_kernel(const __grid_constant__ PairParams p, const __grid_constant__ PairMaps maps) {
  extern __shared__ __align__(1024) uint8_t smem[];          // the kernel has no other shared memory
  pdl_wait();
  pdl_trigger();
  if (smem_u32(smem) & 1023u) {                              // the swizzled slabs start on 1024 bytes
    if (threadIdx.x == 0) atomicOr(&g_err_pair, DEV_ERR_TIMEOUT_MBAR);
    return;
  }
  uint8_t* sQ = smem;                                        // [8 slabs][64 rows][128 B]
  uint8_t* sP = sQ + 8 * kSlab;                              // [4 slabs][64 rows][128 B]
  uint8_t* sK = sP + 4 * kSlab;
  uint8_t* sV = sK + kStages * kStage;
  // Barriers.  A wait tells two neighbouring phases apart, no more: each is waited
  // on by roles that see all of its phases, and none can complete its next phase
  // before all of them have waited for the present one.  What holds it back stands
  // with each.
  // CTA 0: the parts of both CTAs are there.  The stage is loaded again after empty_k /
  // empty_v, which the products issued behind this wait commit.
  uint64_t* full_k = reinterpret_cast<uint64_t*>(sV + kStages * kStage);
  uint64_t* full_v = full_k + kStages;
  // The MMAs that read the stage are done.  Its next products need what its producer
  // loads behind this wait (full_*: both CTAs').
  uint64_t* empty_k = full_v + kStages;
  uint64_t* empty_v = empty_k + kStages;
  // This CTA's part of the V stage is there, to be patched.  The stage is loaded again
  // after empty_v, and full_v needs the patch.
  uint64_t* patch = empty_v + kStages;
  uint64_t* q_full = patch + kStages;                        // CTA 0: the queries of both CTAs; loaded again after q_free
  uint64_t* q_free = q_full + 1;                             // the S products of an item are done; the next need q_full of both CTAs
  // CTA 0: an item's output is out of TMEM in both CTAs.  There is no other output
  // before the PV products issued behind this wait.
  uint64_t* o_free = q_free + 1;
  uint64_t* w_full = o_free + 1;                             // [4] an item is in s_work; the slot is filled again after w_free
  uint64_t* w_free = w_full + kItems;                        // [4] ... and every warp has read it; it is read again after w_full
  // [2] the logits of every other tile; made again after s_free, which all warps that
  // wait here arrive on
  uint64_t* s_full = w_free + kItems;
  uint64_t* s_free = s_full + 2;                             // [2] CTA 0: read by the softmax of both CTAs; read again after s_full
  // CTA 0: P and the rescaled O of both CTAs.  The next tile's follow pv_done, by the
  // wait before them or at the end of the item before.
  uint64_t* p_full = s_free + 2;
  uint64_t* pv_done = p_full + 1;                            // a tile's PV is done; the next needs p_full from all that wait here
  // [2] CTA 0: the MMAs of every other tile's PV are issued.  S(t) waits for PV(t - 2),
  // and the same barrier's PV(t) needs S(t).  One barrier for all tiles would not do:
  // PV(t - 1) does not need S(t) and may be issued before it looks.
  uint64_t* pv_sent = pv_done + 1;
  float* s_x = reinterpret_cast<float*>(pv_sent + 2);        // [2][4][64] maxima / sums of the row quarters
  Work* s_work = reinterpret_cast<Work*>(s_x + 512);         // [4]
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(s_work + kItems);
  int* s_abort = reinterpret_cast<int*>(s_tmem + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t cta = cta_rank();
  const int64_t n_clusters = gridDim.x >> 1, cluster = blockIdx.x >> 1;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full_k[i], 2); mbar_init(&full_v[i], 2); mbar_init(&empty_k[i], 1); mbar_init(&empty_v[i], 1);
      mbar_init(&patch[i], 1);
    }
    for (int i = 0; i < kItems; ++i) { mbar_init(&w_full[i], 1); mbar_init(&w_free[i], 14); }
    mbar_init(q_full, 2); mbar_init(q_free, 1); mbar_init(o_free, 16);
    for (int i = 0; i < 2; ++i) { mbar_init(&s_full[i], 1); mbar_init(&s_free[i], 16); mbar_init(&pv_sent[i], 1); }
    mbar_init(p_full, 16); mbar_init(pv_done, 1);
    *s_abort = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(smem_u32(s_tmem)), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();                                            // barriers and TMEM of both CTAs are set up
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  volatile int* abort_flag = s_abort;

  // Item k of this cluster, from the ring that warp 14 fills.  Whole-warp call; no
  // item: the batch is done, or a wait expired.  The warps of a role that shares a
  // named barrier (bar, of n threads) get one answer.
  auto next_item = [&](uint32_t k, Work& w, uint32_t bar, uint32_t n) -> bool {
    const uint32_t sl = k % kItems;
    bool ok = wait_warp(&w_full[sl], (k / kItems) & 1, abort_flag);
    if (bar != 0 && named_bar_or(bar, n, !ok)) ok = false;
    if (!ok) return false;
    w = s_work[sl];
    __syncwarp();
    if (lane == 0) mbar_arrive(&w_free[sl]);
    return w.has != 0;
  };
  auto tiles_of = [](const Work& w) { return (w.nb + kTileBlocks - 1) / kTileBlocks; };
  auto blocks_of = [](const Work& w, int i) { return min(kTileBlocks, w.nb - kTileBlocks * i); };
  // The tiles of all items in their order (items without rows have none).
  struct Stream {
    Work w;
    uint32_t k = 0, items = 0;   // items read; items with tiles so far, the present one included
    int i = 0, nt = 0;           // tile of the item
  };
  auto advance = [&](Stream& x, uint32_t bar, uint32_t n) -> bool {
    if (++x.i < x.nt) return true;
    do {
      if (!next_item(x.k++, x.w, bar, n)) return false;
      x.nt = tiles_of(x.w);
    } while (x.nt == 0);
    x.i = 0;
    ++x.items;
    return true;
  };
  // Pages of less than 64 rows make several copies of a block: lane 4 kb + j of a
  // producer has part j of block kb of a tile.
  struct Part { int32_t y; int s, rows; bool on; };          // first row of the store, source, rows; whether there is one
  auto part_of = [&](const Stream& x) {
    const int kb = lane >> 2, j = lane & 3;
    Part t{0, 0, kBlock, false};
    if (kb < blocks_of(x.w, x.i)) {
      int row;
      t.s = block_at(x.w, kTileBlocks * x.i + kb, row);
      const PageTable& pt = t.s ? p.pt[1] : p.pt[0];
      t.rows = min(kBlock, 1 << pt.ps_log2);
      t.on = j * t.rows < kBlock;
      if (t.on) {
        const int64_t g = page_row(pt, x.w.seq, row + j * t.rows);
        // A part without a page reads page 0.  It has no visible row, so its logits
        // are masked and its V is patched; or the table is wrong.
        if (g < 0 && row + j * t.rows < (t.s ? x.w.any_hi[1] : x.w.any_hi[0]) &&
            row + (j + 1) * t.rows > (t.s ? x.w.any_lo[1] : x.w.any_lo[0]))
          atomicOr(&g_err_pair, DEV_ERR_BAD_INDEX);
        t.y = (int32_t)max((int64_t)0, g);
      }
    }
    return t;
  };

  if (warp == 14) {
    // ============================ items
    for (uint32_t k = 0;; ++k) {
      const uint32_t sl = k % kItems;
      Work w;
      find_work(p, cluster + (int64_t)k * n_clusters, lane, w);
      if (!wait_warp(&w_free[sl], ((k / kItems) & 1) ^ 1, abort_flag)) break;
      if (lane == 0) {
        s_work[sl] = w;
        mbar_arrive(&w_full[sl]);
      }
      if (!w.has) break;
    }
  } else if (warp == 8) {
    // ============================ queries and K
    const int kb = lane >> 2, j = lane & 3;
    uint32_t st = 0;                                         // stages so far
    bool ok = true;
    Stream x;
    while (ok && advance(x, 0, 0)) {
      const Part t = part_of(x);
      if (x.i == 0) {
        ok = wait_warp(q_free, x.items & 1, abort_flag);
        if (!ok) break;
        if (lane == 0) {
          expect_leader(q_full, 8 * kSlab);
          for (int s = 0; s < 8; ++s)
            tma_load_pair(sQ + s * kSlab, &maps.q, 64 * s, (int32_t)((x.w.tok0 + (int64_t)cta * x.w.tpc) * p.H), q_full);
        }
        __syncwarp();
      }
      // blocks 2 cta, 2 cta + 1 of the tile; absent ones are not loaded (their logits are masked)
      const int n = max(0, min(2, blocks_of(x.w, x.i) - 2 * (int)cta));
      const bool mine = t.on && (kb >> 1) == (int)cta;
      const CUtensorMap* map = t.s ? &maps.k[1] : &maps.k[0];
#pragma unroll 1
      for (int d = 0; d < kKStages; ++d, ++st) {
        const uint32_t sl = st % kStages;
        ok = wait_warp(&empty_k[sl], ((st / kStages) & 1) ^ 1, abort_flag);
        if (!ok) break;
        if (lane == 0) {
          if (n) expect_leader(&full_k[sl], n * kSlab);
          else arrive_leader(&full_k[sl]);
        }
        if (mine) tma_load_pair(sK + sl * kStage + (kb & 1) * kSlab + j * t.rows * 128, map, 64 * d, t.y, &full_k[sl]);
      }
    }
  } else if (warp == 11) {
    // ============================ V
    const int kb = lane >> 2, j = lane & 3;
    uint32_t st = 0;
    bool ok = true;
    Stream x;
    while (ok && advance(x, 0, 0)) {
      const Part t = part_of(x);
      const CUtensorMap* map = t.s ? &maps.v[1] : &maps.v[0];
      const CUtensorMap* part = t.s ? &maps.k[1] : &maps.k[0];
      const int nv = 2 * blocks_of(x.w, x.i);
#pragma unroll 1
      for (int v = 0; v < nv; ++v, ++st) {                   // dims 256 (v & 1) + 128 cta .. of block v / 2
        const uint32_t sl = st % kStages;
        ok = wait_warp(&empty_v[sl], ((st / kStages) & 1) ^ 1, abort_flag);
        if (!ok) break;
        const bool clean = block_clean(x.w, kTileBlocks * x.i + (v >> 1));
        if (lane == 0) {
          if (clean) expect_leader(&full_v[sl], kStage);
          else mbar_expect_tx(&patch[sl], kStage);
        }
        if (t.on && kb == (v >> 1)) {
          // the block's rows lie in both slabs: one copy, or one for each part and slab
          uint8_t* dst = sV + sl * kStage + j * t.rows * 128;
          if (t.rows == kBlock) {
            if (clean) tma_load_pair_4d(dst, map, 0, t.y, 2 * (int)cta, v & 1, &full_v[sl]);
            else tma_load_4d(dst, map, 0, t.y, 2 * (int)cta, v & 1, &patch[sl]);
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int d = 256 * (v & 1) + 128 * (int)cta + 64 * h;
              if (clean) tma_load_pair(dst + h * kSlab, part, d, t.y, &full_v[sl]);
              else tma_load_2d(dst + h * kSlab, part, d, t.y, &patch[sl]);
            }
          }
        }
      }
    }
  } else if (warp == 12 || warp == 13) {
    // ============================ patches of V blocks that not every token sees
    const int lt = tid - 384;                                // 0 .. 63: row of the block
    uint32_t st = 0, uses = 0;                               // uses: bit sl, parity of the next use
    bool ok = true;
    Stream x;
    while (ok && advance(x, 2, 64)) {
      const int nbk = blocks_of(x.w, x.i);
#pragma unroll 1
      for (int v = 0; v < 2 * nbk; ++v, ++st) {
        const int kb = kTileBlocks * x.i + (v >> 1);
        if (block_clean(x.w, kb)) continue;
        int row;
        const int s = block_at(x.w, kb, row);
        row += lt;
        const bool any = row >= (s ? x.w.any_lo[1] : x.w.any_lo[0]) && row < (s ? x.w.any_hi[1] : x.w.any_hi[0]);
        const bool all = row >= (s ? x.w.all_lo[1] : x.w.all_lo[0]) && row < (s ? x.w.all_hi[1] : x.w.all_hi[0]);
        const uint32_t sl = st % kStages;
        ok = wait_warp(&patch[sl], (uses >> sl) & 1, abort_flag);
        uses ^= 1u << sl;
        if (named_bar_or(2, 64, !ok)) ok = false;            // one answer for the two warps
        if (!ok) break;
        if (!all) {
#pragma unroll 4
          for (int q = 0; q < 16; ++q) {                     // the row's 16 pieces of 16 bytes
            uint8_t* at = sV + sl * kStage + (q >> 3) * kSlab + swz128(lt, q & 7);
            uint4 z = make_uint4(0, 0, 0, 0);
            if (any) {
              z = *reinterpret_cast<const uint4*>(at);
              z = make_uint4(finite2(z.x), finite2(z.y), finite2(z.z), finite2(z.w));
            }
            st_shared16(smem_u32(at), z);
          }
        }
        fence_proxy_async_smem();
        named_bar_sync(2, 64);
        if (lt == 0) arrive_leader(&full_v[sl]);
      }
    }
  } else if (warp == 9) {
    // ============================ S (CTA 0)
    const uint32_t idesc = make_idesc(128, 256, 1, 1, 0, 0);
    const uint64_t dQ = smem_desc(smem_u32(sQ), 16, 1024, SWZ_128B);
    const uint64_t dK = smem_desc(smem_u32(sK), 16, 1024, SWZ_128B);
    uint32_t st = 0, t = 0;                                  // stages and tiles so far
    bool ok = cta == 0;
    Stream x;
    for (; advance(x, 0, 0); ++t) {
      if (ok && x.i == 0) ok = wait_warp(q_full, (x.items & 1) ^ 1, abort_flag);
      ok = ok && wait_warp(&pv_sent[t & 1], ((t >> 1) & 1) ^ 1, abort_flag);       // behind PV(t - 2)
      ok = ok && wait_warp(&s_free[t & 1], ((t >> 1) & 1) ^ 1, abort_flag);
      if (!ok) continue;
#pragma unroll 1
      for (int d = 0; d < kKStages; ++d, ++st) {
        const uint32_t sl = st % kStages;
        ok = wait_warp(&full_k[sl], (st / kStages) & 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int m = 0; m < 4; ++m)
          mma_pair(tmem + kSCol + 128 * (t & 1), dQ + ((d * kSlab + m * 32) >> 4), dK + ((sl * kStage + m * 32) >> 4), idesc,
                   (d | m) != 0);
        commit_pair(&empty_k[sl]);
      }
      if (ok) {
        commit_pair(&s_full[t & 1]);
        if (x.i == x.nt - 1) commit_pair(q_free);
      }
    }
  } else if (warp == 10) {
    // ============================ PV (CTA 0)
    const uint32_t idesc = make_idesc(128, 256, 1, 1, 0, 1);
    const uint64_t dP = smem_desc(smem_u32(sP), 16, 1024, SWZ_128B);
    const uint64_t dV = smem_desc(smem_u32(sV), kSlab, 1024, SWZ_128B);
    uint32_t st = 0, t = 0;
    bool ok = cta == 0;
    Stream x;
    for (; advance(x, 0, 0); ++t) {
      // O is overwritten at an item's first tile: the item before must be out of it
      if (ok && x.i == 0) ok = wait_warp(o_free, x.items & 1, abort_flag);
      ok = ok && wait_warp(p_full, t & 1, abort_flag);
      if (!ok) continue;
      const int nv = 2 * blocks_of(x.w, x.i);
#pragma unroll 1
      for (int v = 0; v < nv; ++v, ++st) {
        const uint32_t sl = st % kStages;
        ok = wait_warp(&full_v[sl], (st / kStages) & 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int m = 0; m < 4; ++m)
          mma_pair(tmem + 128 * (v & 1), dP + (((v >> 1) * kSlab + m * 32) >> 4), dV + ((sl * kStage + m * 2048) >> 4), idesc,
                   (x.i | (v >> 1) | m) != 0);
        commit_pair(&empty_v[sl]);
      }
      if (lane == 0) mbar_arrive(&pv_sent[t & 1]);
      if (ok) commit_pair(pv_done);
    }
  } else {
    // ============================ softmax and epilogue
    // Warp w reads lanes 32 (w % 4) .. of TMEM: row r of the CTA, half `half` of an
    // accumulator's columns; and of the 128 columns of an S buffer there the 64 of
    // block 2 half + cg, cg = w / 4.
    const int r = tid & 63, half = (warp >> 1) & 1, cg = warp >> 2;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const float sk = p.sink ? p.sink[r % p.H] * 1.4426950408889634f : -CUDART_INF_F;
    uint32_t g = 0, bc = 0;                                  // tiles and exchanges of the items before
    bool ok = true;
    Work w;
    for (uint32_t k = 0; next_item(k, w, 1, kSoft); ++k) {
      const int nt = tiles_of(w);
      const int tk = (int)cta * w.tpc + r / p.H;             // this row's token of the pair
      const bool valid = r < w.tpc * p.H && tk < w.ntok && w.pos0 + tk >= 0;
      const int64_t pos = valid ? w.pos0 + tk : -1;
      int lo[2], hi[2];
      seen(p, 0, pos, lo[0], hi[0]);
      seen(p, 1, pos, lo[1], hi[1]);
      float m = -CUDART_INF_F, l = 0.f;
      // After a wait that expired the warps only keep their barriers, so that none
      // waits for another for ever.
      for (int i = 0; i < nt; ++i) {
        const uint32_t t = g + i;
        // the columns of the block that the row's token sees: [a, e)
        const int kb = kTileBlocks * i + 2 * half + cg;
        const bool whole = kb < w.nb && block_clean(w, kb);
        int a = 0, e = kBlock;
        if (!whole) {
          e = 0;
          if (kb < w.nb) {
            int row;
            const int s = block_at(w, kb, row);
            a = (s ? lo[1] : lo[0]) - row;
            e = (s ? hi[1] : hi[0]) - row;
          }
        }
        ok = ok && wait_warp(&s_full[t & 1], (t >> 1) & 1, abort_flag);
        tc_fence_after();
        const uint32_t ts = tmem + lane_base + kSCol + 128 * (t & 1) + 64 * cg;
        // This row's logits, those that its token does not see as -inf.  A visible
        // logit of -inf is a non-finite row's, whose V may read as zeros.
        float x[64];
        bool nan = false;
        auto logits = [&]() {
          tmem_ld32(ts, x);
          tmem_ld32(ts + 32, x + 32);
          tmem_wait_ld();
          if (!(whole && valid)) {
#pragma unroll
            for (int q = 0; q < 64; ++q) {
              const bool on = q >= a && q < e && valid;
              nan |= on && x[q] == -CUDART_INF_F;
              x[q] = on ? x[q] : -CUDART_INF_F;
            }
          }
          __syncwarp();
        };
        // probabilities against the maximum m, as bf16 pairs in registers
        uint32_t pk[32];
        float sum = 0.f;
        auto weights = [&]() {
          const float ref = nan ? CUDART_NAN_F : m == -CUDART_INF_F ? 0.f : m;
          float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int q = 0; q < 32; ++q) {
            const float2 z = fma2(make_float2(x[2 * q], x[2 * q + 1]), make_float2(p.scale_log2, p.scale_log2), make_float2(-ref, -ref));
            const float2 y = make_float2(exp2_fast(z.x), exp2_fast(z.y));
            l2[q & 1] = add2(l2[q & 1], y);
            pk[q] = pack2(y.x, y.y);
          }
          sum = (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y);
        };
        // The maximum moves only when it grows by more than 2^kTau, which is rare past
        // the first tiles: the weights are formed against the old one while the four
        // threads of the rows find out, and formed again if it must move.
        float mx = -CUDART_INF_F;
        if (ok) {
          logits();
          float m4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
          for (int q = 4; q < 64; ++q) m4[q & 3] = fmaxf(m4[q & 3], x[q]);
          mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
          weights();
        }
        float alpha = 1.f;
        if (named_bar_or(1, kSoft, !ok || mx * p.scale_log2 > m + kTau)) {
          float* sx = s_x + (bc++ & 1) * 256;
          sx[64 * (2 * half + cg) + r] = mx;
          if (named_bar_or(1, kSoft, !ok)) ok = false;
          if (!ok) continue;
          mx = fmaxf(fmaxf(sx[r], sx[64 + r]), fmaxf(sx[128 + r], sx[192 + r])) * p.scale_log2;
          if (mx > m + kTau) {
            alpha = exp2f(m - mx);                           // 0 the first time
            m = mx;
          }
          __syncwarp();
          logits();
          weights();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_leader(&s_free[t & 1]);
        l = l * alpha + sum;
        // P and O are free once PV(t - 1) is done (of an earlier item: its epilogue waited)
        if (i > 0) {
          ok = wait_warp(pv_done, (t - 1) & 1, abort_flag);
          if (!ok) continue;
          tc_fence_after();
          if (__any_sync(0xffffffffu, alpha != 1.f)) {       // this warp's 128 columns of O
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              float o[32];
              const uint32_t to = tmem + lane_base + 128 * cg + 32 * c;
              tmem_ld32(to, o);
              tmem_wait_ld();
#pragma unroll
              for (int q = 0; q < 32; ++q) o[q] *= alpha;
              tmem_st16(to, o);
              tmem_st16(to + 16, o + 16);
            }
            tmem_wait_st();
            tc_fence_before();
          }
        }
        const uint32_t pb = smem_u32(sP) + (2 * half + cg) * kSlab;
#pragma unroll
        for (int q = 0; q < 8; ++q)
          st_shared16(pb + swz128(r, q), make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]));
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) arrive_leader(p_full);
      }
      // ---------------- epilogue
      float* sx = s_x + (bc++ & 1) * 256;
      sx[64 * (2 * half + cg) + r] = l;
      named_bar_sync(1, kSoft);
      l = (sx[r] + sx[64 + r]) + (sx[128 + r] + sx[192 + r]);
      float coef = 0.f;
      if (valid) {
        if (l != 0.f || sk != -CUDART_INF_F) {               // a NaN sum passes
          const float top = fmaxf(l != 0.f ? m : -CUDART_INF_F, sk);
          const float f = l != 0.f ? exp2f(m - top) : 0.f;
          coef = l != 0.f ? f / (f * l + exp2f(sk - top)) : 0.f;
        }
      }
      g += nt;
      if (nt > 0) ok = ok && wait_warp(pv_done, (g - 1) & 1, abort_flag);
      tc_fence_after();
      // Rows [first, rows) of this CTA are tokens' results.
      const int64_t orow = (w.tok0 + (int64_t)cta * w.tpc) * p.H;
      const int rows = max(0, min(w.tpc, w.ntok - (int)cta * w.tpc)) * p.H;
      const int first = (int)min((int64_t)rows, max((int64_t)0, -(w.pos0 + (int64_t)cta * w.tpc)) * p.H);
#pragma unroll 1
      for (int u = 0; u < 2; ++u) {
        // columns 128 cg + 64 u .. of O: dims 256 cg + 128 half + 64 u ..  Rows of bf16
        // go through P's shared memory (P is done with), so that a warp writes whole
        // lines, not 32 rows of 16 bytes each.
        float o[64];
        if (nt > 0 && ok) {
          __syncwarp();
          tmem_ld32(tmem + lane_base + 128 * cg + 64 * u, o);
          tmem_ld32(tmem + lane_base + 128 * cg + 64 * u + 32, o + 32);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int q = 0; q < 64; ++q) o[q] = 0.f;
        }
        if (u == 1 && nt > 0) {                              // the next item may overwrite O
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_leader(o_free);
        }
#pragma unroll
        for (int q = 0; q < 64; ++q) o[q] = coef == 0.f ? 0.f : o[q] * coef;
        if (p.out_bf16) {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            st_shared16(smem_u32(sP) + (2 * cg + half) * kSlab + swz128(r, q),
                        make_uint4(pack2(o[8 * q], o[8 * q + 1]), pack2(o[8 * q + 2], o[8 * q + 3]),
                                   pack2(o[8 * q + 4], o[8 * q + 5]), pack2(o[8 * q + 6], o[8 * q + 7])));
          named_bar_sync(1, kSoft);
          if (ok) {
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + orow * kD + 128 * (lane >> 3) + 64 * u + 8 * (lane & 7);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const int rr = warp + 8 * q;
              if (rr >= first && rr < rows)
                *reinterpret_cast<uint4*>(out + (int64_t)rr * kD) =
                    *reinterpret_cast<const uint4*>(sP + (lane >> 3) * kSlab + swz128(rr, lane & 7));
            }
          }
          if (u == 0) named_bar_sync(1, kSoft);
        } else if (valid && ok) {
          float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.out) + (orow + r) * kD + 256 * cg + 128 * half + 64 * u);
#pragma unroll
          for (int q = 0; q < 16; ++q) dst[q] = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
        }
      }
    }
    __syncwarp();
  }
  __syncwarp();
  drain_after_abort(abort_flag);
  tc_fence_before();
  __syncthreads();
  cluster_sync();                                            // neither CTA leaves while the other may reach it
  if (warp == 9) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(512));
  }
}

}  // namespace

csa_status_t launch_paged_pair(PairParams& p, cudaStream_t st) {
  PairMaps maps;
  memset(&maps, 0, sizeof(maps));
  if (!encode_2d(&maps.q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p.q, kD, p.n_tok * p.H, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B))
    return fail(CSA_ERR_CUDA, "csa_paged_attention: cuTensorMapEncodeTiled (queries) failed");
  for (int s = 0; s < 2; ++s) {
    if (!p.rows[s]) continue;
    const int ps = 1 << p.pt[s].ps_log2;
    const cuuint64_t rows = (cuuint64_t)p.pt[s].n_pages * ps;
    const cuuint32_t box_rows = (cuuint32_t)std::min(ps, kBlock);
    const cuuint64_t dims[4] = {64, rows, 4, 2}, strides[3] = {kD * 2, 128, 512};
    const cuuint32_t box[4] = {64, box_rows, 2, 1}, step[4] = {1, 1, 1, 1};
    if (!encode_2d(&maps.k[s], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p.rows[s], kD, rows, 64, box_rows, CU_TENSOR_MAP_SWIZZLE_128B) ||
        tmap_encoder()(&maps.v[s], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(p.rows[s]), dims, strides, box, step,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return fail(CSA_ERR_CUDA, "csa_paged_attention: cuTensorMapEncodeTiled (pages) failed");
  }
  const size_t smem = 12 * kSlab + 2 * kStages * kStage + (5 * kStages + 11 + 2 * kItems) * 8 + 512 * 4 + kItems * sizeof(Work) + 16;
  cudaError_t e = cudaFuncSetAttribute(pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return fail(CSA_ERR_CUDA, "csa_paged_attention: cannot reserve %zu bytes of shared memory: %s", smem, cudaGetErrorString(e));
  // Every sequence's last tile may be partly filled: an upper bound of the tiles
  const int per = 2 * std::max(1, 64 / p.H);
  const int64_t tiles = std::min(p.n_tok, p.n_tok / per + p.n_seq);
  if (tiles > 0x3fffffff) return fail(CSA_ERR_UNSUPPORTED, "csa_paged_attention: too many tokens");
  // one cluster for every two SMs (one CTA fits an SM)
  const int64_t clusters = std::min<int64_t>(tiles, num_sms() / 2);
  e = launch_pdl(pair_kernel, dim3((unsigned)(2 * clusters)), dim3(kThreads), smem, st, p, maps);
  if (e != cudaSuccess) return fail(CSA_ERR_CUDA, "csa_paged_attention: launch failed: %s", cudaGetErrorString(e));
  return check_launch("csa_paged_attention");
}

}  // namespace csa
