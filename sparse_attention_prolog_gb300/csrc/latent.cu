// Attention of each sequence's newest tokens over its whole latent cache
// (dsa_latent_attn), on tcgen05.  [V4-TileLang §Sparse Flash Attention] steps
// 3-8 with every visible row in place of a selection.
//
// The (token, head) rows of a sequence lie behind one another in q and out: they
// are cut into blocks of 128 NP rows, whatever H is.  The work is the list of
// (block, tile of 128 cache rows), block by block; persistent clusters take an
// equal stretch of it each, so that sequences of any lengths load all SMs evenly.
// A block that lies in one stretch is finished there; the parts of one that
// several clusters share are merged by latent_merge_kernel.
//
// An O accumulator [128 x 512] in fp32 fills a CTA's tensor memory, so the two
// products live in different CTAs, and P goes from one to the other:
//
//   QK  S = q . K^T (N = 128) and the softmax.  q's latent part is the A operand in
//       tensor memory (256 columns), its rotary part in shared memory; S takes the
//       other 256 columns, twice 128.  A thread has half of a row's columns: two
//       warpgroups, which exchange their maxima, so that a tile's S is read at once
//       and P follows with little delay.  P (bf16) is staged in shared memory and
//       sent by bulk copies, 4 KB a warp, with the factors by which the maximum's
//       growth scales what is in O.
//   PV  O += P . V, V (the first 512 dims of the same rows, from L2) MN-major.
//       Eight warps rescale O where a maximum grew by more than 2^8, and write it
//       at a block's end.
//
// With NP = 1, a warp of the PV CTA fetches the rows of later tiles into the L2: the K ring
// is one tile, and HBM's latency beside the products is longer than a tile's time (541 ->
// 504 us for 32 sequences of 4096 to 131072 rows; four tiles ahead 537, and from the QK CTA,
// whose own copies then wait behind the fetches, it costs more than it gives).  It begins
// when the first rows of V are there, or q would wait behind it (one token at 128K 58.5 ->
// 57.3 us; three tiles ahead in place of two 58.7, four 61.2).
//
// What bounds such a kernel first is not a unit but the single threads that feed them:
// every instruction of theirs takes some five clocks, so their loops are unrolled over a
// tile's units with slots and phases that need no arithmetic, barriers have constant
// addresses, and a tile has few units (nine of K in place of three: 2.25 us a tile in place
// of 1.97 with every row in the L2).  The loaders of K and of V are loops of their own for
// the same reason (one loop with both: 2.25).
//
// Without its loads a tile takes 1.55 us, without its products 1.4, without either 1.17
// (the softmax and P's way); with them NP = 1 takes 1.97 from the L2 and 2.1 from HBM, whose
// rate allows 1.65.  What holds it is the K ring: an SM takes 64 bytes a clock from the L2,
// so a tile of K needs 1.1 us on its way, and a slot is empty while its unit is multiplied.
// NP = 2, whose rings are two tiles, takes 1.3 to 1.4 (its products alone 1.1).
//
// A block's q comes through the K ring, which it fills, and goes on into tensor memory: one
// trip for all of it (through the three staging slots of P, three trips, which cost one token
// over 1000 rows 1 us).
//
// NP = 1: a cluster is one QK and one PV CTA.  NP = 2: two of each, for sequences
// of more than 128 rows: the two QK CTAs run one MMA of M = 256 (cta_group::2), each
// with its own 128 rows of q and half of the tile's K rows, the two PV CTAs likewise
// with half of V's columns, so that an SM loads half of the bytes for the same
// products.
//
// Rows that no token of a block sees (the end of the last tile: they may hold
// anything) are cleared in V before the product; their S is not looked at.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include "dsa_internal.h"
#include "dsa_ptx.cuh"

namespace dsa {
namespace {

constexpr int kDqk = 576, kDv = 512;
constexpr int kTile = 128;                       // cache rows of a tile
constexpr int kAtomsK = kDqk / 64;               // atoms: 64 dims, 128 bytes a row
constexpr int kHalfBytes = 128 * 128;            // 64 columns of a P tile
constexpr uint32_t kTmemS = 256;                 // QK: q's latent part in columns [0, 256), then two S buffers
constexpr int kThreads = 384;                    // 8 softmax / output warps, a loader, an MMA issuer, two for news
constexpr int kLoadWarp = 8, kMmaWarp = 9, kRelayWarp = 10, kNewsWarp = 11;
// A cluster's stretch has at least this many tiles.  (One token over 1000 rows: 22.9 us, with
// at least six 29.3; with one, a call that needs no merge may get it: 4 heads over 256 rows
// 16.0 us in place of 14.9.)
constexpr int kMinShare = 2;
constexpr int kMaxClusters = 256;

// The rings: slots of a unit, [atoms][rows][128 bytes].  K: three atoms of all rows of a
// CTA's part of the tile; V: 64 rows, the columns of a CTA's part of one N = 256 product.
// A ring has the units of NP tiles: a slot's number follows from the unit's.
template <int NP>
struct Ring {
  static constexpr int kKRows = kTile / NP, kKAtoms = 3, kKUnits = kAtomsK / kKAtoms;
  static constexpr int kKBytes = kKAtoms * kKRows * 128, kKSlots = kKUnits * NP;
  static constexpr int kKLoaders = NP == 1 ? 3 : 1;  // warps that load K, a share of a unit's atoms each
  // A block's q fills the ring before its first tile: a load has the bytes that a loader's
  // part of a unit of K has (an atom of 128 rows, or three of 64).
  static constexpr int kQUnits = 3 * NP, kQAtoms = NP == 1 ? 1 : 3, kQLoads = 9 / kQAtoms * NP;
  static constexpr int kQBytes = kKBytes / kKLoaders;
  static constexpr int kVRows = 64, kVAtoms = 4 / NP, kVUnits = 4;
  static constexpr int kVBytes = kVAtoms * kVRows * 128, kVSlots = kVUnits * NP;
};
constexpr int kMaxKSlots = 6, kMaxVSlots = 8;
constexpr int kPSlots = 5, kStages = 3;  // slots of half a tile's P, in the PV CTA and where it is staged
constexpr int kMaxQUnits = 6, kMaxQLoads = 9;
constexpr int kAhead = 2;  // tiles between V's loads and the rows that are fetched into the L2

// Shared memory of a QK CTA: K ring, staging slots of P, q's rotary part, OwnQk.  Of a PV
// CTA: V ring, P slots, the rescale factors.  Behind them, in both, Shared.
struct OwnQk {
  float top[2][2][128];      // [tile parity][column half]: a row's maximum in a tile
  float alpha[kStages][128]; // rescale factors on their way out
  float2 final_ml[2][128];   // (maximum, sum) of each column half at a block's end
};
constexpr int kOffStage = 147456, kOffQrope = kOffStage + kStages * kHalfBytes, kOffOwn = kOffQrope + kHalfBytes;
constexpr int kOffP = 131072, kOffAlpha = kOffP + kPSlots * kHalfBytes;
static_assert(Ring<1>::kKSlots * Ring<1>::kKBytes == kOffStage && Ring<2>::kKSlots * Ring<2>::kKBytes == kOffStage, "K ring");
static_assert(Ring<1>::kVSlots * Ring<1>::kVBytes == kOffP && Ring<2>::kVSlots * Ring<2>::kVBytes == kOffP, "V ring");
constexpr int kOffShared = kOffOwn + sizeof(OwnQk);
static_assert(kOffAlpha + kPSlots * 512 <= kOffShared && kOffShared % 16 == 0, "shared memory of a PV CTA");

struct LatentParams {
  int T, B, n_q, H, max_L;
  float scale_log2;
  const __nv_bfloat16* q;
  const __nv_bfloat16* kv;
  int64_t cache_rows;
  const int32_t* block_table;
  int block_size, max_blocks;
  int k_box, v_box;  // rows of a TMA box of K and of V
  const int32_t* cu;
  const int32_t* kv_len;
  __nv_bfloat16* out;
  float* lse;
  const float* sink;
  int clusters;
  int start;        // tiles that a block's beginning counts as
  float* part_o;    // [2 clusters][64][128 NP][8]: the first and the last part of a stretch, 8 columns of all rows together
  float2* part_ml;  // [2 clusters][128 NP]: (maximum, sum) in log2 units
  int block_rows;   // 128 NP
  int4* desc;       // [clusters]: first row, rows, parts of the block that begins at the end of a stretch
  uint32_t* err;
};

struct __align__(8) Bars {
  // of the barriers that an MMA waits for, those of the pair's first CTA count for both; full ones tell that a
  // CTA's own copies are there
  uint64_t kfull[kMaxKSlots], kempty[kMaxKSlots];
  uint64_t kpeer[kMaxKSlots], vpeer[kMaxVSlots];  // the second CTA's unit of K or V is there
  uint64_t sfull[2], sempty[2];
  uint64_t pfree[kPSlots];        // QK: a P slot of the PV CTA is free
  uint64_t landed[kStages];       // QK: what a staging slot held has arrived there
  uint64_t qload[kMaxQLoads], qread[kMaxQUnits];  // QK: a part of q is in the K ring; a slot's part has been read
  uint64_t mready[4];             // QK: both halves' maxima are known, per pair of warps
  uint64_t qfull;                 // a block's q is in place
  uint64_t ffree;                 // QK: the final (m, l) have been read
  uint64_t vfull[kMaxVSlots], vempty[kMaxVSlots];
  uint64_t vclean[kMaxVSlots];    // PV: rows that nothing sees are cleared in a unit
  uint64_t pfull[kPSlots], pcons[kPSlots];  // PV: P slots
  uint64_t phalf[2];              // PV: the second half of P has arrived in every CTA
  uint64_t oready[2];             // PV: O is scaled for the tile, whose first half has arrived
  uint64_t odone[2];              // PV: a tile's product is in O (even and odd tiles: a warp may look a tile late)
  uint64_t ffull;                 // PV: the final (m, l) lie in the QK CTA
  uint64_t drain;                 // the MMA thread's last commit
};
struct __align__(16) Shared {
  Bars bars;
  long long scan[kThreads / 32];
  long long start_off;
  int start_b;
  uint32_t tmem;
  int abort_flag;         // a wait has run out in this CTA, at the end in any of the cluster
  volatile int progress;  // tiles whose loads have begun, but one
  // Copies begun, for a cluster that gives up: units of K and V by each lane, loads of q by
  // each loader, tiles whose P a softmax warp has sent.
  int k_begun[3][32], q_begun[3], v_begun[32], p_begun[8];
};
constexpr size_t kSmemBytes = kOffShared + sizeof(Shared);
static_assert(kSmemBytes <= 232448, "shared memory of a CTA");

struct Piece {
  int row0, rows;  // of q and out: the block's
  int b, len;      // sequence, its cache rows
  int first_vis;   // cache rows that the sequence's first token sees
  int in_seq;      // rows of the sequence before the block
  int vis;         // cache rows that the block's last token sees
  int t0, t1;      // tiles
  bool begins, ends;
  int to_end;      // of the block's share of the work, what is left for later stretches
};

template <int NP>
struct Walker {
  static constexpr int kBlock = 128 * NP;
  long long left;
  int b, blk, off;
  int n, c0, len, nt, nb;

  __device__ __forceinline__ void load(const LatentParams& P) {
    if (P.cu != nullptr) {
      c0 = min(max(__ldg(P.cu + b), 0), P.T);
      n = min(max(__ldg(P.cu + b + 1), c0), P.T) - c0;
    } else {
      c0 = b * P.n_q;
      n = P.n_q;
    }
    len = min(max(__ldg(P.kv_len + b), 0), P.max_L);
    // (the sequence's tiles for each of its blocks, though the first ones of a prompt see fewer: what
    // that leaves idle is little behind a long context, a third and more where a prompt begins one)
    nt = max(1, (len - 1) / kTile + 1) + P.start;  // so many empty ones in front
    nb = (n * P.H + kBlock - 1) / kBlock;
  }
  __device__ __forceinline__ void start(const LatentParams& P, int b0, long long at, long long count) {
    left = count;
    b = b0;
    n = nb = 0;
    blk = off = 0;
    if (left <= 0) return;
    load(P);
    blk = static_cast<int>(at / nt);
    off = static_cast<int>(at % nt);
  }
  __device__ __forceinline__ bool next(const LatentParams& P, Piece& p) {
    while (true) {
      if (left <= 0) return false;
      while (blk >= nb) {
        if (++b >= P.B) return false;
        blk = 0;
        load(P);
      }
      const int from = off, stop = static_cast<int>(min(static_cast<long long>(nt), off + left));
      const int block = blk;
      left -= stop - from;
      off = stop;
      if (off == nt) {
        off = 0;
        ++blk;
      }
      if (stop <= P.start) continue;  // none of the block's tiles: it begins in the next stretch
      p.b = b;
      p.len = len;
      p.row0 = c0 * P.H + block * kBlock;
      p.rows = min(kBlock, n * P.H - block * kBlock);
      p.in_seq = block * kBlock;
      p.first_vis = len - n + 1;
      p.vis = max(0, p.first_vis + (block * kBlock + p.rows - 1) / P.H);
      p.t0 = max(0, from - P.start);
      p.t1 = max(p.t0, min(stop - P.start, (p.vis + kTile - 1) / kTile));
      p.begins = from <= P.start;
      p.ends = stop == nt;
      p.to_end = nt - stop;
      return true;
    }
  }
};

// Row of the cache at which the rows from s on of a sequence lie (a box of them, in
// one page); cache_rows (past the map: read as zeros) where there are none.
__device__ __forceinline__ int box_row(const LatentParams& P, const Piece& p, int s, bool report) {
  const int none = static_cast<int>(P.cache_rows);
  if (s >= p.len) return none;
  if (P.block_table == nullptr) return p.b * P.max_L + s;  // below cache_rows, so it fits
  const int page = __ldg(P.block_table + static_cast<size_t>(p.b) * P.max_blocks + s / P.block_size);
  if (page < 0 || (static_cast<int64_t>(page) + 1) * P.block_size > P.cache_rows) {
    if (report) atomicOr(P.err, kErrBadIndex);
    return none;
  }
  return page * P.block_size + s % P.block_size;
}

// One thread of the warp (the compiler knows it for one).
__device__ __forceinline__ bool elect_one() {
  uint32_t v;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(v));
  return v != 0;
}

// mbar_wait_polling for a whole warp: all lanes get the same answer, so that what
// follows (tensor memory accesses, votes) is done by all of them or by none.
template <bool kCluster>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint32_t* err, volatile int* abort_flag) {
  auto test = [&]() { return kCluster ? mbar_test_cluster(bar, parity) : mbar_test(bar, parity); };
  if (__all_sync(0xffffffffu, test())) return true;
  const uint64_t limit = wait_limit_ns(err), t0 = globaltimer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (__all_sync(0xffffffffu, test())) return true;
    const bool late = globaltimer_ns() - t0 > limit;
    if (__any_sync(0xffffffffu, late || *abort_flag)) {
      if (late) atomicOr(err, kErrTimeout);
      *abort_flag = 1;
      return false;
    }
  }
}

// Arrives on a barrier of another CTA without ordering this thread's own writes before
// it: for news of what copies and products did, which this thread learned from a
// barrier.  (With .release.cluster an arrival takes 500 ns, and a thread that sends two
// or four a tile holds the whole pipeline up: 2.1 us a tile with nothing else to do.)
__device__ __forceinline__ void arrive_remote_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// The same for one thread.  (Not inlined: the loops of the threads that wait stay short.)
template <bool kCluster>
__device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, uint32_t* err, volatile int* abort_flag) {
  return mbar_wait_polling<kCluster>(bar, parity, err, abort_flag);
}
template <bool kCluster>
__device__ __forceinline__ bool thread_wait(uint64_t* bar, uint32_t parity, uint32_t* err, volatile int* abort_flag) {
  if (kCluster ? mbar_test_cluster(bar, parity) : mbar_test(bar, parity)) return true;
  return wait_on<kCluster>(bar, parity, err, abort_flag);
}

// Tiled load of the box [atoms][rows][64 dims] at an atom and a row.
__device__ __forceinline__ void load_box(void* dst, const void* map, int atom, int row, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(atom), "r"(smem_u32(bar))
      : "memory");
}
// Shared memory of this CTA -> of another of the cluster, counted on its barrier.
__device__ __forceinline__ void bulk_to_peer(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(dst), "r"(smem_u32(src)), "r"(bytes), "r"(bar) : "memory");
}

// Bytes that arrive with half i % 2 of tile i / 2: the first has the rescale factors.
__device__ __forceinline__ uint32_t p_bytes(int i) { return kHalfBytes + (i % 2 == 0 ? 512 : 0); }

template <int NP>
__device__ __forceinline__ void alloc_tmem(uint32_t* result) {
  if (NP == 1) {
    tmem_alloc(result, 512);
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(result)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int NP>
__device__ __forceinline__ void free_tmem(uint32_t addr) {
  if (NP == 1) tmem_dealloc(addr, 512);
  else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(addr) : "memory");
}
// The pair's (or the CTA's) product with A in shared (its descriptor's low word) or in
// tensor memory; kAdd: to what D holds.  All descriptors here have the same high word but
// V's; 32-bit additions and a constant predicate keep an MMA at a few instructions.
template <int NP, bool kAdd>
__device__ __forceinline__ void product_ss(uint32_t d, uint32_t a, uint32_t a_hi, uint32_t b, uint32_t b_hi, uint32_t idesc) {
  if (NP == 1)
    asm volatile("{\n.reg .pred p;\n.reg .b64 x, y;\nsetp.ne.b32 p, %6, 0;\nmov.b64 x, {%1, %2};\nmov.b64 y, {%3, %4};\n"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %5, p;\n}"
                 ::"r"(d), "r"(a), "r"(a_hi), "r"(b), "r"(b_hi), "r"(idesc), "n"(kAdd ? 1 : 0) : "memory");
  else
    asm volatile("{\n.reg .pred p;\n.reg .b64 x, y;\nsetp.ne.b32 p, %6, 0;\nmov.b64 x, {%1, %2};\nmov.b64 y, {%3, %4};\n"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], x, y, %5, p;\n}"
                 ::"r"(d), "r"(a), "r"(a_hi), "r"(b), "r"(b_hi), "r"(idesc), "n"(kAdd ? 1 : 0) : "memory");
}
template <int NP, bool kAdd>
__device__ __forceinline__ void product_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t b_hi, uint32_t idesc) {
  if (NP == 1)
    asm volatile("{\n.reg .pred p;\n.reg .b64 y;\nsetp.ne.b32 p, %5, 0;\nmov.b64 y, {%2, %3};\n"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n}"
                 ::"r"(d), "r"(a), "r"(b), "r"(b_hi), "r"(idesc), "n"(kAdd ? 1 : 0) : "memory");
  else
    asm volatile("{\n.reg .pred p;\n.reg .b64 y;\nsetp.ne.b32 p, %5, 0;\nmov.b64 y, {%2, %3};\n"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], y, %4, p;\n}"
                 ::"r"(d), "r"(a), "r"(b), "r"(b_hi), "r"(idesc), "n"(kAdd ? 1 : 0) : "memory");
}
// Arrives on the barrier, in every CTA of the pair, when the products issued so far are complete.
template <int NP>
__device__ __forceinline__ void commit(uint64_t* bar, uint16_t mask) {
  if (NP == 1) mma_commit(bar);
  else
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 ::"r"(smem_u32(bar)), "h"(mask) : "memory");
}

__device__ __forceinline__ float2 ld_cluster_f32x2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
// Counts bytes on a barrier of this CTA as copied.
__device__ __forceinline__ void mbar_complete_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void st_global_v8(float* p, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// Of a cluster that gave up: waits until every copy into this CTA has landed, when all
// threads of the cluster have stopped.  The lanes and warps that share a unit may have
// stopped at different ones, and its barrier would never complete: what was not begun of a
// unit that one of them did begin is counted here as landed.  (A copy into a slot was begun
// after the slot's last use was complete, so only a ring's last units can be on their way,
// and their phases are the barriers' current ones or just passed.)  Each wait has its limit.
template <int NP>
__device__ __noinline__ void settle(Shared& sh, int role, int k_box, int v_box, uint32_t peer_p_begun) {
  using R = Ring<NP>;
  Bars& bars = sh.bars;
  if (role == 0) {
    const int boxes = R::kKRows / k_box;
    constexpr int kBytes = R::kKBytes / R::kKLoaders;  // of a loader's part of a unit
    int most = 0;
    for (int w = 0; w < R::kKLoaders; ++w)
      for (int l = 0; l < boxes; ++l) most = max(most, sh.k_begun[w][l]);
    for (int i = max(0, most - R::kKSlots); i < most; ++i) {
      uint64_t* full = &bars.kfull[i % R::kKSlots];
      for (int w = 0; w < R::kKLoaders; ++w) {
        if (sh.k_begun[w][0] <= i) mbar_arrive_expect_tx(full, kBytes);
        for (int l = 0; l < boxes; ++l)
          if (sh.k_begun[w][l] <= i) mbar_complete_tx(full, kBytes / boxes);
      }
      if (!mbar_drain(full, (i / R::kKSlots) & 1)) return;
    }
    constexpr int kMine = R::kQLoads / R::kKLoaders;  // loads of a block's q by a loader
    for (int w = 0; w < R::kKLoaders; ++w)
      for (int i = max(0, sh.q_begun[w] - kMine); i < sh.q_begun[w]; ++i)
        if (!mbar_drain(&bars.qload[i % kMine * R::kKLoaders + w], (i / kMine) & 1)) return;
  } else {
    const int boxes = kTile / v_box, per = boxes / 2;
    int most = 0;
    for (int l = 0; l < boxes; ++l) most = max(most, sh.v_begun[l]);
    for (int i = max(0, most - R::kVSlots); i < most; ++i) {
      uint64_t* full = &bars.vfull[i % R::kVSlots];
      const int group = i % R::kVUnits >> 1;  // whose lanes copy this unit
      if (sh.v_begun[0] <= i) mbar_arrive_expect_tx(full, R::kVBytes);
      for (int l = group * per; l < group * per + per; ++l)
        if (sh.v_begun[l] <= i) mbar_complete_tx(full, R::kVBytes / per);
      if (!mbar_drain(full, (i / R::kVSlots) & 1)) return;
    }
    for (int g = 0; g < 2; ++g) {  // P: half g of each tile, from four warps
      int begun[4], tiles = 0;
      for (int w = 0; w < 4; ++w) {
        begun[w] = static_cast<int>(ld_cluster_u32(peer_p_begun + (4 * g + w) * 4));
        tiles = max(tiles, begun[w]);
      }
      for (int t = max(0, tiles - 3); t < tiles; ++t) {  // (older halves have left their staging slots)
        const int at = 2 * t + g;
        uint64_t* full = &bars.pfull[at % kPSlots];
        for (int w = 0; w < 4; ++w)
          if (begun[w] <= t) mbar_complete_tx(full, p_bytes(at) / 4);
        if (!mbar_drain(full, (at / kPSlots) & 1)) return;
      }
    }
  }
}

template <int NP>
__global__ void __launch_bounds__(kThreads, 1)
    latent_attn_kernel(const __grid_constant__ LatentParams P, const __grid_constant__ CUtensorMap k_map,
                       const __grid_constant__ CUtensorMap v_map, const __grid_constant__ CUtensorMap q_map) {
  using R = Ring<NP>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_u32(smem) & 1023u) != 0) {  // (swizzled tiles; it starts at a multiple, as the kernel has no other)
    if (threadIdx.x == 0) atomicOr(P.err, kErrTimeout);
    return;
  }
  Shared& sh = *reinterpret_cast<Shared*>(smem + kOffShared);
  OwnQk& own = *reinterpret_cast<OwnQk*>(smem + kOffOwn);
  Bars& bars = sh.bars;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const int role = rank / NP, side = rank % NP;  // 0: QK, 1: PV; which 128 rows of the block
  const uint32_t first = role * NP;              // rank of the pair's first CTA, which issues its products
  const int cluster = blockIdx.x / (2 * NP);
  volatile int* abort_v = &sh.abort_flag;

  if (tid == 0) {
    for (int i = 0; i < kMaxKSlots; ++i) {
      mbar_init(&bars.kfull[i], R::kKLoaders);
      mbar_init(&bars.kpeer[i], 1);
      mbar_init(&bars.kempty[i], 1);
    }
    for (int i = 0; i < kMaxVSlots; ++i) {
      mbar_init(&bars.vfull[i], 1);
      mbar_init(&bars.vpeer[i], 1);
      mbar_init(&bars.vempty[i], 1);
      mbar_init(&bars.vclean[i], 8 * NP);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.sfull[i], 1);
      mbar_init(&bars.sempty[i], 8 * NP);
      mbar_init(&bars.phalf[i], NP);
      mbar_init(&bars.oready[i], 8 * NP);
      mbar_init(&bars.odone[i], 1);
    }
    for (int i = 0; i < kPSlots; ++i) {
      mbar_init(&bars.pfree[i], 1);
      mbar_init(&bars.pfull[i], 1);
      mbar_init(&bars.pcons[i], 1);
    }
    for (int i = 0; i < kStages; ++i) mbar_init(&bars.landed[i], 1);
    for (int i = 0; i < R::kQLoads; ++i) mbar_init(&bars.qload[i], 1);
    for (int i = 0; i < R::kQUnits; ++i) mbar_init(&bars.qread[i], 8 / NP);
    for (int i = 0; i < 4; ++i) mbar_init(&bars.mready[i], 2);
    mbar_init(&bars.qfull, 8 * NP);
    mbar_init(&bars.ffree, 8);
    mbar_init(&bars.ffull, 8);
    mbar_init(&bars.drain, 1);
    sh.abort_flag = 0;
    sh.progress = 0;
    fence_mbar_init();
    if (role == 1)
      for (int i = 0; i < kPSlots; ++i) mbar_arrive_expect_tx(&bars.pfull[i], p_bytes(i));
  }
  if (warp == 0) alloc_tmem<NP>(&sh.tmem);
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // waited for below
  griddep_wait();
  griddep_launch_dependents();  // the merge's CTAs come as these leave, and wait for the last

  // ------------------------------------------------ this cluster's stretch
  const int each = (P.B + kThreads - 1) / kThreads;
  const int b0 = min(P.B, tid * each), b1 = min(P.B, b0 + each);
  long long mine = 0;
  bool bad = false, falls = false;
  Walker<NP> w;
  for (w.b = b0; w.b < b1; ++w.b) {
    w.load(P);
    mine += static_cast<long long>(w.nb) * w.nt;
    if (P.cu != nullptr) {
      const int c0 = __ldg(P.cu + w.b), c1 = __ldg(P.cu + w.b + 1);
      falls |= c1 < c0;
      bad |= c0 < 0 || c1 < c0 || c1 > P.T || (w.b == 0 && c0 != 0);
    }
    const int len = __ldg(P.kv_len + w.b);
    bad |= len < 0 || len > P.max_L;
  }
  if (bad && blockIdx.x == 0) atomicOr(P.err, kErrBadIndex);
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) sh.scan[warp] = inc;
  tc_fence_before();
  falls = __syncthreads_or(falls);
  tc_fence_after();
  long long before = inc - mine, total = 0;
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) before += sh.scan[i];
    total += sh.scan[i];
  }
  if (falls) {  // counts that decrease: sequences may overlap, and be any multiple of T tokens
    long long tokens = 0;
    for (w.b = b0; w.b < b1; ++w.b) {
      w.load(P);
      tokens += w.n;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) tokens += __shfl_xor_sync(0xffffffffu, tokens, o);
    __syncthreads();  // (the sums above have been read)
    if (lane == 0) sh.scan[warp] = tokens;
    __syncthreads();
    tokens = 0;
    for (int i = 0; i < kThreads / 32; ++i) tokens += sh.scan[i];
    if (tokens > P.T) total = 0;
  }
  const long long active = max(1ll, min(static_cast<long long>(P.clusters), total / kMinShare));
  // stretch c begins at share c + min(c, rest)
  const long long share = total / active, rest = total - share * active;
  const long long lo = cluster < active ? share * cluster + min(static_cast<long long>(cluster), rest) : total;
  const long long hi = cluster < active ? lo + share + (cluster < rest ? 1 : 0) : total;
  if (lo < hi && before <= lo && lo < before + mine) {
    long long at = lo - before;
    for (w.b = b0; w.b < b1; ++w.b) {
      w.load(P);
      const long long size = static_cast<long long>(w.nb) * w.nt;
      if (at < size) break;
      at -= size;
    }
    sh.start_b = w.b;
    sh.start_off = at;
  }
  if (lo >= hi && tid == 0) {
    sh.start_b = 0;
    sh.start_off = 0;
  }
  const uint32_t tmem = sh.tmem;
  const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // every CTA's barriers are initialised
  __syncthreads();                                                      // the stretch is known
  w.start(P, sh.start_b, sh.start_off, hi - lo);
  Piece p;
  // arrives on a barrier of the pair's first CTA; with own_writes, those are visible there
  auto arrive_first = [&](uint64_t* bar, bool own_writes) {
    if (NP == 1) mbar_arrive(bar);
    else if (own_writes) mbar_arrive_remote(mapa(smem_u32(bar), first));
    else arrive_remote_relaxed(mapa(smem_u32(bar), first));
  };

  if (warp < 8 && role == 0) {
    // ------------------------------------------------------------- softmax
    const int g = warp >> 2, wq = warp & 3;  // half of the columns, quadrant of the rows
    const int row = wq * 32 + lane;
    const float ninf = -__int_as_float(0x7f800000);
    const uint32_t peer = NP + side;
    const uint32_t peer_p = mapa(smem_u32(smem + kOffP + wq * 4096), peer);
    const uint32_t peer_alpha = mapa(smem_u32(smem + kOffAlpha + wq * 128), peer);
    const uint32_t peer_pfull = mapa(smem_u32(&bars.pfull[0]), peer);
    const uint32_t peer_ffull = mapa(smem_u32(&bars.ffull), peer);
    const uint64_t scale2 = pack_f32x2(P.scale_log2, P.scale_log2), one2 = pack_f32x2(1.f, 1.f);
    int G = 0, pieces = 0, blocks = 0;  // tiles, pieces and blocks with tiles so far
    auto fetch_q = [&](const Piece& b) {  // four rows a lane
      const int64_t from = static_cast<int64_t>(b.row0) + side * 128 + lane * 4;
      const int64_t n = min(static_cast<int64_t>(4), static_cast<int64_t>(b.row0) + b.rows - from);
      if (n > 0) prefetch_l2(P.q + from * kDqk, static_cast<uint32_t>(n) * (kDqk * 2));
    };
    bool ok = true;
    while (ok && w.next(P, p)) {
      const int nt = p.t1 - p.t0, in_block = side * 128 + row;
      if (nt > 0) {
        // q: this row's latent atoms go from the K ring into tensor memory, half of them each
        // group, the rotary atom into its own place.  The products that read the last
        // block's are complete: every warp has seen its last S.
        if (warp == 7) {  // the next block's comes from the L2
          Walker<NP> after = w;
          Piece next;
          if (after.next(P, next)) fetch_q(next);
        }
#pragma unroll 1
        for (int a = g; ok && a < kAtomsK; a += 2) {
          const int load = NP == 1 ? a : a / 3 * 2 + (row >> 6);  // (of a warp: its rows are of one part)
          ok = warp_wait<false>(&bars.qload[load], blocks & 1, P.err, abort_v);
          if (!ok) break;
          const uint8_t* src = NP == 1 ? smem + a * kHalfBytes
                                       : smem + ((G & 1) * R::kKUnits + load) % R::kKSlots * R::kKBytes + a % 3 * (kHalfBytes / 2);
          uint32_t v[32];
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const uint4 x = *reinterpret_cast<const uint4*>(src + sw128_off(NP == 1 ? row : row & 63, c));
            v[4 * c] = x.x; v[4 * c + 1] = x.y; v[4 * c + 2] = x.z; v[4 * c + 3] = x.w;
          }
          if (a < kAtomsK - 1) {
            tmem_st32(tmem + lane_off + a * 32, v);
          } else {
#pragma unroll
            for (int c = 0; c < 8; ++c)
              *reinterpret_cast<uint4*>(smem + kOffQrope + sw128_off(row, c)) =
                  make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
            fence_proxy_async_smem();
          }
          if (a + 2 >= a / 3 * 3 + 3) {  // this group's last of the slot
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.qread[NP == 1 ? a / 3 : load]);
          }
        }
        ++blocks;
        if (!ok) break;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_first(&bars.qfull, true);
      }
      const int vis = p.first_vis + (p.in_seq + in_block) / P.H;  // rows that this row's token sees
      float m_used = ninf;
      uint64_t l_two = 0;  // two partial sums
      for (int j = 0; j < nt; ++j, ++G) {
        const int par = G & 1, at = 2 * G + g, ps = at % kPSlots, st = at % kStages;
        if (!warp_wait<false>(&bars.sfull[par], (G >> 1) & 1, P.err, abort_v)) { ok = false; break; }
        tc_fence_after();
        uint32_t s0[32], s1[32];
        tmem_ld32(tmem + lane_off + kTmemS + par * kTile + g * 64, s0);
        tmem_ld32(tmem + lane_off + kTmemS + par * kTile + g * 64 + 32, s1);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_first(&bars.sempty[par], false);
        const int lim = vis - (p.t0 + j) * kTile - g * 64;  // columns that this row sees
        if (!__all_sync(0xffffffffu, lim >= 64)) {
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            if (k >= lim) s0[k] = __float_as_uint(ninf);
            if (32 + k >= lim) s1[k] = __float_as_uint(ninf);
          }
        }
        float mx[4] = {ninf, ninf, ninf, ninf};
#pragma unroll
        for (int k = 0; k < 32; ++k) mx[k & 3] = fmaxf(mx[k & 3], fmaxf(__uint_as_float(s0[k]), __uint_as_float(s1[k])));
        float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        own.top[par][g][row] = mt;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.mready[wq]);
        if (!warp_wait<false>(&bars.mready[wq], par, P.err, abort_v)) { ok = false; break; }
        mt = fmaxf(mt, own.top[par][g ^ 1][row]) * P.scale_log2;
        float alpha = 1.f;
        if (mt > m_used + 8.f) {  // also taken when m_used is -inf
          alpha = ex2_approx(m_used - mt);
          m_used = mt;
          l_two = fma_f32x2(l_two, pack_f32x2(alpha, alpha), 0);
        }
        const float shift = m_used == ninf ? 0.f : -m_used;
        const uint64_t shift2 = pack_f32x2(shift, shift);
        uint32_t pk[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          const uint64_t x = k < 16 ? pack_f32x2(__uint_as_float(s0[(2 * k) & 31]), __uint_as_float(s0[(2 * k + 1) & 31]))
                                    : pack_f32x2(__uint_as_float(s1[(2 * k) & 31]), __uint_as_float(s1[(2 * k + 1) & 31]));
          const uint64_t y = fma_f32x2(x, scale2, shift2);
          const float p0 = ex2_approx(lo_f32(y)), p1 = ex2_approx(hi_f32(y));
          l_two = fma_f32x2(pack_f32x2(p0, p1), one2, l_two);
          const __nv_bfloat162 pb = __floats2bfloat162_rn(p0, p1);
          pk[k] = *reinterpret_cast<const uint32_t*>(&pb);
        }
        if (!warp_wait<false>(&bars.landed[st], ((at / kStages) & 1) ^ 1, P.err, abort_v) ||
            !warp_wait<false>(&bars.pfree[ps], ((at / kPSlots) & 1) ^ 1, P.err, abort_v)) {
          ok = false;
          break;
        }
        uint8_t* stage = smem + kOffStage + st * kHalfBytes;
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *reinterpret_cast<uint4*>(stage + sw128_off(row, c)) = make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
        if (g == 0) own.alpha[st][row] = alpha;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          bulk_to_peer(peer_p + ps * kHalfBytes, stage + wq * 4096, 4096, peer_pfull + ps * 8);
          if (g == 0) bulk_to_peer(peer_alpha + ps * 512, &own.alpha[st][wq * 32], 128, peer_pfull + ps * 8);
        }
      }
      if (!ok) break;
      if (!warp_wait<true>(&bars.ffree, (pieces & 1) ^ 1, P.err, abort_v)) { ok = false; break; }
      own.final_ml[g][row] = make_float2(m_used, lo_f32(l_two) + hi_f32(l_two));
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(peer_ffull);
      ++pieces;
    }
    if (!ok) tmem_st_wait();  // (q's, of a block that was given up)
    if (lane == 0) sh.p_begun[warp] = G;
  } else if (warp < 8) {
    // ------------------------------------------------ O: scaling and output
    const int half = warp >> 2, row = (warp & 3) * 32 + lane;
    const float ninf = -__int_as_float(0x7f800000);
    const float* alphas = reinterpret_cast<const float*>(smem + kOffAlpha);
    const uint32_t peer_final = mapa(smem_u32(&own.final_ml[0][0]), side);
    const uint32_t peer_ffree = mapa(smem_u32(&bars.ffree), side);
    int G = 0, pieces = 0, done = 0;  // tiles, blocks, products seen complete
    bool ok = true;
    int tail_row0 = 0, tail_rows = 0, tail_parts = 0;  // the block that this stretch ends inside of
    auto wait_products = [&](int n) {
      while (ok && done < n) {
        ok = warp_wait<false>(&bars.odone[done & 1], (done >> 1) & 1, P.err, abort_v);
        done += ok;
      }
    };
    while (ok && w.next(P, p)) {
      const int nt = p.t1 - p.t0, in_block = side * 128 + row;
      for (int j = 0; j < nt; ++j, ++G) {
        const int par = G & 1, ps = 2 * G % kPSlots;
        if (!warp_wait<false>(&bars.pfull[ps], (2 * G / kPSlots) & 1, P.err, abort_v)) { ok = false; break; }
        const float alpha = alphas[ps * 128 + row];
        const bool rescaled = j > 0 && __any_sync(0xffffffffu, alpha != 1.f);
        if (rescaled) {
          wait_products(G);  // O holds the products before this tile
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int c0 = half * 256; c0 < half * 256 + 256; c0 += 32) {
            uint32_t v[32];
            tmem_ld32(tmem + lane_off + c0, v);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * alpha);
            tmem_st32(tmem + lane_off + c0, v);
          }
          tmem_st_wait();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) arrive_first(&bars.oready[par], rescaled);
        const int live = p.vis - (p.t0 + j) * kTile;  // rows of the tile that the block sees
        if (live < kTile) {
          // (with the products before complete, every unit before this tile's has been there: a
          // wait below cannot take an older phase for its own)
          wait_products(G);
          for (int u = live / R::kVRows * 2; ok && u < R::kVUnits; ++u) {
            const int slot = (G * R::kVUnits + u) % R::kVSlots;
            ok = warp_wait<false>(&bars.vfull[slot], (NP == 1 ? G : G >> 1) & 1, P.err, abort_v);
            if (!ok) break;
            const int from = max(0, live - u / 2 * R::kVRows), rows = R::kVRows - from;
            for (int i = tid; i < rows * R::kVAtoms * 8; i += 256)
              *reinterpret_cast<uint4*>(smem + slot * R::kVBytes + i / (8 * rows) * (R::kVRows * 128) +
                                        (from + (i >> 3) % rows) * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) arrive_first(&bars.vclean[slot], true);
          }
        }
        if (!ok) break;
        wait_products(G);  // at most one product's completion stays unseen
        if (!ok) break;
      }
      wait_products(G);
      if (ok) ok = warp_wait<true>(&bars.ffull, pieces & 1, P.err, abort_v);
      if (!ok) break;
      tc_fence_after();
      const float2 f0 = ld_cluster_f32x2(peer_final + row * 8);
      const float2 f1 = ld_cluster_f32x2(peer_final + (128 + row) * 8);
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(peer_ffree);
      ++pieces;
      float m = fmaxf(f0.x, f1.x);
      // (a sum of 0 says that nothing was seen; one that is not a number stays so)
      float l = (f0.y == 0.f ? 0.f : f0.y * ex2_approx(f0.x - m)) + (f1.y == 0.f ? 0.f : f1.y * ex2_approx(f1.x - m));
      const bool empty = l == 0.f || nt == 0;
      const bool whole = p.begins && p.ends;
      const size_t orow = static_cast<size_t>(p.row0) + in_block;
      if (whole) {
        float factor = empty ? 0.f : 1.f / l, lse2 = empty ? ninf : m + log2f(l);
        if (P.sink != nullptr) {
          // the sink adds 2^s2 to the denominator, taken relative to max(m, s2)
          const float s2 = __ldg(P.sink + (p.in_seq + in_block) % P.H) * 1.4426950408889634f;
          if (empty) {
            lse2 = s2;
          } else {
            const float mx = fmaxf(m, s2), den = l * exp2f(m - mx) + exp2f(s2 - mx);
            factor = exp2f(m - mx) / den;
            lse2 = mx + log2f(den);
          }
        }
        if (in_block < p.rows && half == 0 && P.lse != nullptr) P.lse[orow] = lse2 * 0.69314718055994531f;
        // (stores of 32 bytes a lane, whole sectors: 8 x 64 tokens over 1000 rows 163 us, with 16
        // bytes 174; without any 147)
        __nv_bfloat16* o = P.out + orow * kDv;
#pragma unroll 1
        for (int c0 = half * 256; c0 < half * 256 + 256; c0 += 32) {
          uint32_t v[32], pk[16];
          tmem_ld32(tmem + lane_off + c0, v);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const __nv_bfloat162 pb = __floats2bfloat162_rn(__uint_as_float(v[2 * k]) * factor, __uint_as_float(v[2 * k + 1]) * factor);
            pk[k] = empty ? 0u : *reinterpret_cast<const uint32_t*>(&pb);
          }
          if (in_block < p.rows) {
#pragma unroll
            for (int k = 0; k < 2; ++k) st_global_v8(reinterpret_cast<float*>(o + c0 + 16 * k), pk + 8 * k);
          }
        }
      } else {
        const size_t part = 2 * cluster + (p.begins ? 1 : 0);
        if (half == 0) P.part_ml[part * (128 * NP) + in_block] = make_float2(empty ? ninf : m, empty ? 0.f : l);
        float* o = P.part_o + part * (128 * NP) * kDv + in_block * 8;
        if (__any_sync(0xffffffffu, !empty)) {
#pragma unroll 1
          for (int c0 = half * 256; c0 < half * 256 + 256; c0 += 64) {
            uint32_t v0[32], v1[32];
            tmem_ld32(tmem + lane_off + c0, v0);
            tmem_ld32(tmem + lane_off + c0 + 32, v1);
            tmem_ld_wait();
            if (in_block < p.rows && !empty) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                st_global_v8(o + (c0 / 8 + k) * (128 * NP * 8), v0 + 8 * k);
                st_global_v8(o + (c0 / 8 + 4 + k) * (128 * NP * 8), v1 + 8 * k);
              }
            }
          }
        }
        if (p.begins) {
          // the block ends in the stretch that holds its last tile; this stretch ends with this piece
          const long long last = hi - 1 + p.to_end, edge = (share + 1) * rest;
          const long long holder = last < edge ? last / (share + 1) : rest + (last - edge) / share;
          const int parts = static_cast<int>(holder) - cluster + 1;
          tail_row0 = p.row0;
          tail_rows = p.rows;
          tail_parts = parts;
        }
      }
      tc_fence_before();
    }
    if (tid == 0 && side == 0) P.desc[cluster] = make_int4(tail_row0, tail_rows, tail_parts, 0);
  } else if (role == 0 && (warp == kLoadWarp || (NP == 1 && warp > kMmaWarp))) {
    // ------------------------------------------------------------ q and K
    // Each lane has a box of the tile's rows (a page, or all rows of a unit): it looks up the
    // next tile's while it issues this one's.
    const int boxes = R::kKRows / P.k_box, from = side * R::kKRows + lane * P.k_box;
    const bool plain = P.k_box == R::kKRows;  // a box has all rows of a unit, and its atoms
    const int which = warp == kLoadWarp ? 0 : warp - kMmaWarp;
    int G = 0, issued = 0, blocks = 0, q_issued = 0;  // tiles, units, blocks with tiles and loads of q so far
    bool ok = true;
    auto look_up = [&](int t) { return t < p.t1 && lane < boxes ? box_row(P, p, t * kTile + from, false) : 0; };
    while (ok && w.next(P, p)) {
      if (p.t0 >= p.t1) continue;
      // q, into every slot of the ring, once the last block's is read and its K used up
      if (lane == 0) {
#pragma unroll 1
        for (int u = 0; u < R::kQUnits; ++u)
          ok = ok && (blocks == 0 || thread_wait<false>(&bars.qread[u], (blocks & 1) ^ 1, P.err, abort_v));
#pragma unroll 1
        for (int u = 0; ok && u < R::kQUnits; ++u) {
          // (the phase that the slot's next unit of K waits for)
          const int tile = NP == 1 ? G : G + u / R::kKUnits, slot = ((NP == 1 ? 0 : G & 1) * R::kKUnits + u) % R::kKSlots;
          const int load = NP == 1 ? u * R::kKLoaders + which : u;
          ok = thread_wait<false>(&bars.kempty[slot], ((NP == 1 ? tile : tile >> 1) & 1) ^ 1, P.err, abort_v);
          if (!ok) break;
          mbar_arrive_expect_tx(&bars.qload[load], R::kQBytes);
          load_box(smem + slot * R::kKBytes + which * R::kQBytes, &q_map, NP == 1 ? load : u / 2 * R::kQAtoms,
                   p.row0 + side * 128 + (NP == 1 ? 0 : u % 2 * 64), &bars.qload[load]);
          ++q_issued;
        }
      }
      __syncwarp();
      int row = look_up(p.t0);  // (a trip to memory of its own, while q is on its way)
#pragma unroll 1
      for (int u = 0; u < R::kQUnits; ++u)
        ok = ok && thread_wait<false>(&bars.qread[u], blocks & 1, P.err, abort_v);
      ++blocks;
      ok = __all_sync(0xffffffffu, ok);
      for (int t = p.t0; ok && t < p.t1; ++t, ++G) {
        const int next_row = look_up(t + 1);
        if (lane < boxes) {
          const int ring = NP == 1 ? 0 : G & 1;
          const uint32_t use = ((NP == 1 ? G : G >> 1) & 1) ^ 1;
#pragma unroll
          for (int u = 0; u < R::kKUnits; ++u) {
            constexpr int kAtoms = R::kKAtoms / R::kKLoaders;
            const int slot = ring * R::kKUnits + u;
            ok = ok && thread_wait<false>(&bars.kempty[slot], use, P.err, abort_v);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(&bars.kfull[slot], R::kKBytes / R::kKLoaders);
            uint8_t* dst = smem + slot * R::kKBytes + (which * kAtoms * R::kKRows + lane * P.k_box) * 128;
            if (plain) {
              load_box(dst, &k_map, u * R::kKAtoms + which * kAtoms, row, &bars.kfull[slot]);
            } else {
#pragma unroll
              for (int a = 0; a < kAtoms; ++a)
                load_box(dst + a * R::kKRows * 128, &k_map, u * R::kKAtoms + which * kAtoms + a, row, &bars.kfull[slot]);
            }
            ++issued;
          }
        }
        ok = __all_sync(0xffffffffu, ok);
        row = next_row;
      }
    }
    sh.k_begun[which][lane] = issued;
    if (lane == 0) sh.q_begun[which] = q_issued;
  } else if (role == 1 && warp == kLoadWarp) {
    // ------------------------------------------------------------------ V
    const int boxes = kTile / P.v_box, per = boxes / 2;
    const int group = lane >= per;  // this lane's box is in the units of rows 64 group ..
    const bool plain = P.v_box == R::kVRows;
    int G = 0, issued = 0;
    bool ok = true;
    auto look_up = [&](int t) { return t < p.t1 && lane < boxes ? box_row(P, p, t * kTile + lane * P.v_box, side == 0) : 0; };
    while (ok && w.next(P, p)) {
      if (p.t0 >= p.t1) continue;
      int row = look_up(p.t0);
      for (int t = p.t0; ok && t < p.t1; ++t, ++G) {
        const int next_row = look_up(t + 1);
        if (lane == 0) sh.progress = G;
        if (lane < boxes) {
          const int ring = NP == 1 ? 0 : G & 1;
          const uint32_t use = ((NP == 1 ? G : G >> 1) & 1) ^ 1;
#pragma unroll
          for (int u = 0; u < R::kVUnits; ++u) {
            const int slot = ring * R::kVUnits + u, atom = (u & 1) * 4 + side * R::kVAtoms;
            ok = ok && thread_wait<false>(&bars.vempty[slot], use, P.err, abort_v);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(&bars.vfull[slot], R::kVBytes);
            uint8_t* dst = smem + slot * R::kVBytes + (lane - group * per) * P.v_box * 128;
            if (group == u >> 1) {
              if (plain) {
                load_box(dst, &v_map, atom, row, &bars.vfull[slot]);
              } else {
#pragma unroll
                for (int a = 0; a < R::kVAtoms; ++a)
                  load_box(dst + a * R::kVRows * 128, &v_map, atom + a, row, &bars.vfull[slot]);
              }
            }
            ++issued;
          }
        }
        ok = __all_sync(0xffffffffu, ok);
        row = next_row;
      }
    }
    sh.v_begun[lane] = issued;
  } else if (warp == kMmaWarp && side == 0 && elect_one()) {
    const uint16_t both = role == 0 ? 3 : 12;
    bool ok = true;
    int G = 0;
    if (role == 0) {
      // ------------------------------------------------------ S = q . K^T
      const uint32_t idesc = idesc_f16(128 * NP, kTile, kFmtBF16, 0, 0);
      const uint64_t k_desc = smem_desc(smem_u32(smem), 16, 1024, kSwizzle128B);
      const uint32_t k_lo = static_cast<uint32_t>(k_desc), k_hi = static_cast<uint32_t>(k_desc >> 32);
      const uint32_t qrope_lo = k_lo + (kOffQrope >> 4);
      int blocks = 0;
      while (ok && w.next(P, p)) {
        if (p.t0 >= p.t1) continue;
        ok = thread_wait<NP == 2>(&bars.qfull, blocks & 1, P.err, abort_v);
        ++blocks;
        for (int t = p.t0; ok && t < p.t1; ++t, ++G) {
          const uint32_t s = tmem + kTmemS + (G & 1) * kTile;
          const int ring = NP == 1 ? 0 : G & 1;
          const uint32_t use = (NP == 1 ? G : G >> 1) & 1;
          ok = thread_wait<false>(&bars.sempty[G & 1], ((G >> 1) & 1) ^ 1, P.err, abort_v);
#pragma unroll
          for (int u = 0; u < R::kKUnits; ++u) {
            const int slot = ring * R::kKUnits + u;
            ok = ok && thread_wait<false>(&bars.kfull[slot], use, P.err, abort_v);
            if (NP == 2) ok = ok && thread_wait<false>(&bars.kpeer[slot], use, P.err, abort_v);
            if (!ok) break;
            tc_fence_after();
            const uint32_t kd = k_lo + ((slot * R::kKBytes) >> 4);
#pragma unroll
            for (int kk = 0; kk < R::kKAtoms * 4; ++kk) {
              const int step = u * R::kKAtoms * 4 + kk;
              const uint32_t bd = kd + (((kk / 4) * (R::kKRows * 128) + (kk % 4) * 32) >> 4);
              if (step == 0)
                product_ts<NP, false>(s, tmem, bd, k_hi, idesc);
              else if (step < 32)
                product_ts<NP, true>(s, tmem + step * 8, bd, k_hi, idesc);
              else
                product_ss<NP, true>(s, qrope_lo + (((kk % 4) * 32) >> 4), k_hi, bd, k_hi, idesc);
            }
            commit<NP>(&bars.kempty[slot], both);
          }
          if (ok) commit<NP>(&bars.sfull[G & 1], both);
        }
      }
    } else {
      // ------------------------------------------------------- O += P . V
      const uint32_t idesc = idesc_f16(128 * NP, 256, kFmtBF16, 0, 1);
      const uint64_t v_desc = smem_desc(smem_u32(smem), R::kVRows * 128, 1024, kSwizzle128B);
      const uint64_t p_desc = smem_desc(smem_u32(smem + kOffP), 16, 1024, kSwizzle128B);
      const uint32_t v_lo = static_cast<uint32_t>(v_desc), v_hi = static_cast<uint32_t>(v_desc >> 32);
      const uint32_t p_lo = static_cast<uint32_t>(p_desc), p_hi = static_cast<uint32_t>(p_desc >> 32);
      uint32_t cleaned = 0;  // the phase of each slot's vclean
      int ps = 0;            // slot of the next half of P, and its phase
      uint32_t p_use = 0;
      while (ok && w.next(P, p)) {
        for (int t = p.t0; ok && t < p.t1; ++t, ++G) {
          const int par = G & 1, ring = NP == 1 ? 0 : par, live = p.vis - t * kTile;
          const uint32_t use = (NP == 1 ? G : G >> 1) & 1;
          ok = thread_wait<NP == 2>(&bars.oready[par], (G >> 1) & 1, P.err, abort_v);
#pragma unroll
          for (int u = 0; u < R::kVUnits; ++u) {
            const int slot = ring * R::kVUnits + u;
            if (u == R::kVUnits / 2) {
              if (NP == 1) ok = ok && thread_wait<false>(&bars.pfull[ps], p_use, P.err, abort_v);
              else ok = ok && thread_wait<false>(&bars.phalf[par], (G >> 1) & 1, P.err, abort_v);
            }
            ok = ok && thread_wait<false>(&bars.vfull[slot], use, P.err, abort_v);
            if (NP == 2) ok = ok && thread_wait<false>(&bars.vpeer[slot], use, P.err, abort_v);
            if (ok && (u / 2 + 1) * R::kVRows > live) {  // rows that nothing sees: cleared first
              ok = thread_wait<NP == 2>(&bars.vclean[slot], (cleaned >> slot) & 1, P.err, abort_v);
              cleaned ^= 1u << slot;
            }
            if (!ok) break;
            tc_fence_after();
            const uint32_t pd = p_lo + ((ps * kHalfBytes) >> 4), vd = v_lo + ((slot * R::kVBytes) >> 4);
            const uint32_t d = tmem + (u & 1) * 256;
            if (u < 2 && t == p.t0)
              product_ss<NP, false>(d, pd, p_hi, vd, v_hi, idesc);
            else
              product_ss<NP, true>(d, pd, p_hi, vd, v_hi, idesc);
#pragma unroll
            for (int kk = 1; kk < R::kVRows / 16; ++kk)
              product_ss<NP, true>(d, pd + ((kk * 32) >> 4), p_hi, vd + ((kk * 16 * 128) >> 4), v_hi, idesc);
            commit<NP>(&bars.vempty[slot], both);
            if (u & 1) {
              commit<NP>(&bars.pcons[ps], both);
              if (++ps == kPSlots) { ps = 0; p_use ^= 1; }
            }
          }
          if (ok) commit<NP>(&bars.odone[par], both);
        }
      }
    }
    // every product issued has completed before the tensor memory is freed
    commit<NP>(&bars.drain, both);
    mbar_drain(&bars.drain, 0);
  } else if (warp == kRelayWarp && role == 1 && elect_one()) {
    // -- to the QK CTA: a half of P has arrived, its staging slot is free; a P slot is
    // consumed, and free.  (Pairs) to the first CTA: the second half has arrived.
    const uint32_t peer_pfree = mapa(smem_u32(&bars.pfree[0]), side), peer_landed = mapa(smem_u32(&bars.landed[0]), side);
    const uint32_t first_phalf = mapa(smem_u32(&bars.phalf[0]), first);
    int landed = 0, consumed = 0, end = 0;  // halves
    int l_slot = 0, l_stage = 0, c_slot = 0;
    uint32_t l_use = 0, c_use = 0;
    bool ok = true;
    while (ok && w.next(P, p)) {
      end += 2 * (p.t1 - p.t0);
      int idle = 0;
      uint64_t since = 0;
      while (consumed < end) {
        bool any = false;
        if (landed < end && mbar_test(&bars.pfull[l_slot], l_use)) {
          arrive_remote_relaxed(peer_landed + l_stage * 8);
          if (NP == 2 && (landed & 1)) arrive_remote_relaxed(first_phalf + (landed >> 1 & 1) * 8);
          ++landed;
          if (++l_slot == kPSlots) { l_slot = 0; l_use ^= 1; }
          if (++l_stage == kStages) l_stage = 0;
          any = true;
        }
        if (consumed < landed && mbar_test(&bars.pcons[c_slot], c_use)) {
          mbar_arrive_expect_tx(&bars.pfull[c_slot], p_bytes(consumed + kPSlots));  // for the slot's next use
          arrive_remote_relaxed(peer_pfree + c_slot * 8);
          ++consumed;
          if (++c_slot == kPSlots) { c_slot = 0; c_use ^= 1; }
          any = true;
        }
        if (any) {
          idle = 0;
        } else if (++idle % 64 == 0) {
          const uint64_t now = globaltimer_ns();
          if (idle == 64) since = now;
          const bool late = now - since > wait_limit_ns(P.err);
          if (late) atomicOr(P.err, kErrTimeout);
          if (late || *abort_v) {
            *abort_v = 1;
            ok = false;
            break;
          }
        }
      }
    }
  } else if (NP == 1 && warp == kNewsWarp && role == 1) {
    // --- the tile kAhead on from V's: its rows into the L2, 8 a lane (they lie in one page).
    // No one waits for this warp: it leaves when the others are late.
    bool ok = true;
    int G = 0;
    while (ok && w.next(P, p)) {
      for (int t = p.t0; ok && t < p.t1; ++t, ++G) {
        const int row = lane < kTile / 8 ? box_row(P, p, t * kTile + lane * 8, false) : static_cast<int>(P.cache_rows);
        const uint64_t since = globaltimer_ns();
        while (ok && (G > sh.progress + kAhead || (G == 0 && sh.progress == 0 && !mbar_test(&bars.vfull[0], 0)))) {
          __nanosleep(64);
          ok = !*abort_v && globaltimer_ns() - since <= wait_limit_ns(P.err);
        }
        ok = __all_sync(0xffffffffu, ok);
        if (ok && row < P.cache_rows)
          prefetch_l2(P.kv + static_cast<size_t>(row) * kDqk, static_cast<uint32_t>(min(static_cast<int64_t>(8), P.cache_rows - row)) * (kDqk * 2));
      }
    }
  } else if (NP == 2 && warp == kNewsWarp && side == 1 && elect_one()) {
    // ------------- a unit of this CTA's half has arrived -> the first CTA
    const int units = role == 0 ? R::kKUnits : R::kVUnits, slots = role == 0 ? R::kKSlots : R::kVSlots;
    uint64_t* full = role == 0 ? bars.kfull : bars.vfull;
    const uint32_t peer = mapa(smem_u32(role == 0 ? bars.kpeer : bars.vpeer), first);
    int slot = 0;
    uint32_t ph = 0;
    bool ok = true;
    while (ok && w.next(P, p))
      for (int i = 0; ok && i < (p.t1 - p.t0) * units; ++i) {
        ok = thread_wait<false>(&full[slot], ph, P.err, abort_v);
        if (!ok) break;
        arrive_remote_relaxed(peer + slot * 8);
        if (++slot == slots) { slot = 0; ph ^= 1; }
      }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort_v)
    for (int r = 0; r < 2 * NP; ++r) st_cluster_u32(mapa(smem_u32(&sh.abort_flag), r), 1);
  cluster_sync();  // no CTA leaves while another may still address it
  if (*abort_v) {  // (the same in all of the cluster: nothing more is begun, what was begun lands)
    if (tid == 0) settle<NP>(sh, role, P.k_box, P.v_box, mapa(smem_u32(sh.p_begun), side));
    cluster_sync();
  }
  if (warp == 0) free_tmem<NP>(tmem);
}

// Merges the parts of the blocks that clusters' stretches end inside of:
// out = sum_c 2^(m_c - M) O_c / (sum_c 2^(m_c - M) l_c [+ 2^(sink - M)]).  An item is 32
// rows (a lane each) x 8 columns of a block.  Of a block of few parts a warp takes an item
// with all of them, four in flight at a time; of one of many (one long sequence), eight
// warps take an eighth each of the parts of 4 columns, ten in flight, and their sums meet
// in shared memory.  (At 64K rows: 3 tokens, 25 or 26 parts a block, 73.4 us a call the first
// way, 76.7 the second; 2 x 2 tokens, 18 parts, 64.8 and 71.9; 2 tokens, 38 parts, 63.2 and
// 59.8; 1 x 2 tokens, 36 parts, 52.9 and 50.7.  16 heads over 700 to 9000 rows, two or three
// parts: 82 and 115.)
constexpr int kMergeWarps = 8, kFewParts = 32;

template <int kCols>
struct Merged {
  float acc[kCols], sum, top;  // sum_c 2^(m_c - top) O_c and l_c
  __device__ __forceinline__ Merged() : sum(0.f), top(-INFINITY) {
#pragma unroll
    for (int k = 0; k < kCols; ++k) acc[k] = 0.f;
  }
};

// Adds the parts first, first + step, .. < d.z of the block that begins in cluster c's stretch.
template <int kCols, int kBatch>
__device__ __forceinline__ void add_parts(const LatentParams& P, Merged<kCols>& s, const int4& d, int c, int col, int row, int first, int step) {
  const float ninf = -__int_as_float(0x7f800000);
  for (int c0 = first; c0 < d.z; c0 += kBatch * step) {
    float2 ml[kBatch];
    float4 v[kBatch][kCols / 4];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int part = c0 + b * step;
      ml[b] = make_float2(ninf, 0.f);
#pragma unroll
      for (int k = 0; k < kCols / 4; ++k) v[b][k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row < d.y && part < d.z) {
        const size_t at = part == 0 ? 2 * c + 1 : 2 * (c + part);
        ml[b] = __ldcg(P.part_ml + at * P.block_rows + row);
        const float4* o = reinterpret_cast<const float4*>(P.part_o + ((at * (kDv / 8) + col / 8) * P.block_rows + row) * 8 + col % 8);
#pragma unroll
        for (int k = 0; k < kCols / 4; ++k) v[b][k] = __ldcg(o + k);
      }
    }
    float top = s.top;
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
      if (ml[b].y != 0.f) top = fmaxf(top, ml[b].x);
    const float shift = top == ninf ? 0.f : top, r = exp2f(s.top - shift);
    s.top = top;
    s.sum *= r;
#pragma unroll
    for (int k = 0; k < kCols; ++k) s.acc[k] *= r;
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (ml[b].y == 0.f) continue;  // nothing seen: its O was not written
      const float f = exp2f(ml[b].x - shift);
      s.sum = fmaf(f, ml[b].y, s.sum);
#pragma unroll
      for (int k = 0; k < kCols / 4; ++k) {
        s.acc[4 * k] = fmaf(f, v[b][k].x, s.acc[4 * k]);
        s.acc[4 * k + 1] = fmaf(f, v[b][k].y, s.acc[4 * k + 1]);
        s.acc[4 * k + 2] = fmaf(f, v[b][k].z, s.acc[4 * k + 2]);
        s.acc[4 * k + 3] = fmaf(f, v[b][k].w, s.acc[4 * k + 3]);
      }
    }
  }
}

// The output of an item's row, with the sink as one more term 2^s2 of the denominator.
template <int kCols>
__device__ __forceinline__ void finish_row(const LatentParams& P, Merged<kCols>& s, const int4& d, int col, int row) {
  if (row >= d.y) return;
  const float ninf = -__int_as_float(0x7f800000);
  const int orow = d.x + row;
  if (P.sink != nullptr) {
    const float s2 = __ldg(P.sink + orow % P.H) * 1.4426950408889634f, top = s.sum != 0.f ? fmaxf(s.top, s2) : s2;
    const float shift = top == ninf ? 0.f : top, r = s.sum != 0.f ? exp2f(s.top - shift) : 0.f;
    s.sum = s.sum * r + exp2f(s2 - shift);
#pragma unroll
    for (int k = 0; k < kCols; ++k) s.acc[k] *= r;
    s.top = top;
  }
  const float inv = s.sum != 0.f ? 1.f / s.sum : 0.f;
  uint2* o = reinterpret_cast<uint2*>(P.out + static_cast<size_t>(orow) * kDv + col);
#pragma unroll
  for (int k = 0; k < kCols / 4; ++k) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(s.acc[4 * k] * inv, s.acc[4 * k + 1] * inv);
    const __nv_bfloat162 b = __floats2bfloat162_rn(s.acc[4 * k + 2] * inv, s.acc[4 * k + 3] * inv);
    o[k] = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
  if (col == 0 && P.lse != nullptr) P.lse[orow] = s.sum != 0.f ? (s.top + log2f(s.sum)) * 0.69314718055994531f : ninf;
}

__global__ void __launch_bounds__(32 * kMergeWarps) latent_merge_kernel(const __grid_constant__ LatentParams P) {
  __shared__ float sums[kMergeWarps][6][32];  // a warp's 4 columns, sum and maximum
  __shared__ int4 descs[kMaxClusters];
  __shared__ int begin[kMaxClusters + 1];  // steps of the CTAs before a cluster's block: eight items, or one of many parts
  __shared__ int warp_total[kMergeWarps];
  static_assert(kMaxClusters == 32 * kMergeWarps, "a thread per cluster");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float ninf = -__int_as_float(0x7f800000);
  constexpr int kChunks = kDv / 8;
  griddep_wait();
  {
    int4 d = make_int4(0, 0, 0, 0);
    if (threadIdx.x < P.clusters) d = __ldcg(P.desc + threadIdx.x);
    const int items = d.z == 0 ? 0 : (d.y + 31) / 32 * kChunks;
    const int steps = d.z > kFewParts ? 2 * items : (items + kMergeWarps - 1) / kMergeWarps;
    int inc = steps;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    if (lane == 31) warp_total[warp] = inc;
    descs[threadIdx.x] = d;
    __syncthreads();
    for (int i = 0; i < warp; ++i) inc += warp_total[i];
    begin[threadIdx.x + 1] = inc;
    if (threadIdx.x == 0) begin[0] = 0;
    __syncthreads();
  }
  const int all = begin[kMaxClusters];
  for (int step = blockIdx.x; step < all; step += gridDim.x) {
    int c = 0;  // the last cluster whose steps begin at or before it
#pragma unroll
    for (int o = kMaxClusters / 2; o; o >>= 1)
      if (begin[c + o] <= step) c += o;
    const int4 d = descs[c];
    const int at = step - begin[c];
    if (d.z <= kFewParts) {
      const int item = at * kMergeWarps + warp, col = item % kChunks * 8, row = item / kChunks * 32 + lane;
      Merged<8> s;
      add_parts<8, 4>(P, s, d, c, col, row, 0, 1);
      finish_row(P, s, d, col, row);
      continue;
    }
    const int col = at % (2 * kChunks) * 4, row = at / (2 * kChunks) * 32 + lane;
    {
      Merged<4> s;
      add_parts<4, 10>(P, s, d, c, col, row, warp, kMergeWarps);
#pragma unroll
      for (int k = 0; k < 4; ++k) sums[warp][k][lane] = s.acc[k];
      sums[warp][4][lane] = s.sum;
      sums[warp][5][lane] = s.top;
    }
    __syncthreads();
    if (warp == 0) {
      Merged<4> s;
#pragma unroll
      for (int u = 0; u < kMergeWarps; ++u)
        if (sums[u][4][lane] != 0.f) s.top = fmaxf(s.top, sums[u][5][lane]);
      const float shift = s.top == ninf ? 0.f : s.top;
#pragma unroll
      for (int u = 0; u < kMergeWarps; ++u) {
        const float su = sums[u][4][lane];
        if (su == 0.f) continue;
        const float f = exp2f(sums[u][5][lane] - shift);
        s.sum = fmaf(f, su, s.sum);
#pragma unroll
        for (int k = 0; k < 4; ++k) s.acc[k] = fmaf(f, sums[u][k][lane], s.acc[k]);
      }
      finish_row(P, s, d, col, row);
    }
    __syncthreads();
  }
}

// Whether a call's blocks are 256 rows (NP = 2): where a sequence has more than 128 rows
// on average.  Two blocks of 128 rows read the cache twice, a block of 256 with 128 rows to
// fill it wastes half of its products.  (4 x 2 tokens of 128 heads at 64K 99 us paired, 134
// not; 1024 new tokens 1249 and 1744; 19 sequences of 144 rows at 32K 209 and 273; of 128
// rows 208 and 157.)
bool paired(const dsa_latent_attn_args& a) { return static_cast<long long>(a.T) * a.H > 128ll * a.B; }

template <int NP>
cudaLaunchConfig_t config(int clusters, cudaLaunchAttribute (&attr)[2]) {
  cudaLaunchConfig_t cfg = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2 * NP;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(2 * NP * clusters);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}

// Clusters that the current device holds at once.
template <int NP>
int resident_clusters() {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> known[kMaxDevices];
  int d = -1;
  if (cudaGetDevice(&d) != cudaSuccess || d < 0 || d >= kMaxDevices) return 1;
  int n = known[d].load();
  if (n == 0) {
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = config<NP>(1, attr);
    if (cudaFuncSetAttribute(latent_attn_kernel<NP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kSmemBytes)) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, latent_attn_kernel<NP>, &cfg) != cudaSuccess || n < 1) {
      cudaGetLastError();  // (not to be found by a later launch)
      return 1;
    }
    known[d].store(n);
  }
  return n;
}

// The most blocks that the shape allows: every sequence but one may end in a block's first row.
long long most_blocks(const dsa_latent_attn_args& a) {
  const long long block = paired(a) ? 256 : 128;
  return (static_cast<long long>(a.T) * a.H + std::min(a.T, a.B) * (block - 1)) / block;
}

// What a block costs beside its tiles (its q, its output, the pipeline's start), in tiles:
// stretches are equal with it counted in front of each block.  (Without: 4 x 2 tokens at 64K
// 104 us in place of 99, 2 x 2 tokens 67.7 in place of 64.7, 8 x 64 tokens over 1000 rows 166
// in place of 163, 16 heads over 700 to 9000 rows 82.2 in place of 81.2.)  A single block
// begins but once in any stretch.
int start_tiles(const dsa_latent_attn_args& a) { return most_blocks(a) == 1 ? 0 : paired(a) ? 6 : 3; }

// Clusters of a call: as many as the device holds, but no more than the most tiles
// that the shape allows can keep busy.
int cluster_count(const dsa_latent_attn_args& a) {
  const long long tiles = most_blocks(a) * ((static_cast<long long>(a.max_L) + kTile - 1) / kTile + start_tiles(a));
  const long long most = paired(a) ? resident_clusters<2>() : resident_clusters<1>(), want = tiles / kMinShare;
  return static_cast<int>(std::min<long long>(kMaxClusters, std::max(1ll, std::min(want, most))));
}

struct Workspace {
  size_t ml, desc, bytes;  // the partial outputs come first
  Workspace(int clusters, int block) {
    const size_t parts = static_cast<size_t>(clusters) * 2 * block;
    ml = round_up(parts * kDv * sizeof(float), 256);
    desc = ml + round_up(parts * sizeof(float2), 256);
    bytes = desc + round_up(static_cast<size_t>(clusters) * sizeof(int4), 256);
  }
};

// The rows of a box: what a unit has, or less where pages are smaller.
int box_rows(const dsa_latent_attn_args& a, int unit) {
  if (a.block_table != nullptr)
    while (a.block_size % unit != 0) unit /= 2;
  return unit;
}

// A map of rows of 576 values as [atom][row][64 values].
bool encode_boxes(CUtensorMap& map, const uint16_t* base, int64_t rows, int box, int atoms) {
  const uint64_t dims[3] = {64, static_cast<uint64_t>(rows), kAtomsK};
  const uint64_t strides[2] = {kDqk * 2, 128};
  const uint32_t b[3] = {64, static_cast<uint32_t>(box), static_cast<uint32_t>(atoms)};
  return encode_tmap(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, b, 128);
}

template <int NP>
int launch(LatentParams& P, const dsa_latent_attn_args& a, cudaStream_t s) {
  using R = Ring<NP>;
  P.k_box = box_rows(a, R::kKRows);
  P.v_box = box_rows(a, R::kVRows);
  alignas(64) CUtensorMap k_map, v_map, q_map;
  if (!encode_boxes(k_map, a.kv, a.cache_rows, P.k_box, P.k_box == R::kKRows ? R::kKAtoms / R::kKLoaders : 1) ||
      !encode_boxes(v_map, a.kv, a.cache_rows, P.v_box, P.v_box == R::kVRows ? R::kVAtoms : 1) ||
      !encode_boxes(q_map, a.q, static_cast<int64_t>(a.T) * a.H, R::kKRows, R::kQAtoms))
    return DSA_ERR_CUDA;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = config<NP>(P.clusters, attr);
  cfg.stream = s;
  if (cudaFuncSetAttribute(latent_attn_kernel<NP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(kSmemBytes)) != cudaSuccess)
    return DSA_ERR_CUDA;
  return cuda_status(cudaLaunchKernelEx(&cfg, latent_attn_kernel<NP>, P, k_map, v_map, q_map));
}

}  // namespace

size_t latent_attn_workspace(const dsa_latent_attn_args& a) {
  return Workspace(cluster_count(a), paired(a) ? 256 : 128).bytes;
}

int launch_latent_attn(const dsa_latent_attn_args& a, void* ws, cudaStream_t s) {
  LatentParams P{};
  P.T = a.T; P.B = a.B; P.n_q = a.n_q; P.H = a.H; P.max_L = a.max_L;
  P.scale_log2 = a.scale * 1.4426950408889634f;
  P.q = reinterpret_cast<const __nv_bfloat16*>(a.q);
  P.kv = reinterpret_cast<const __nv_bfloat16*>(a.kv);
  P.cache_rows = a.cache_rows;
  P.block_table = a.block_table; P.block_size = a.block_size; P.max_blocks = a.max_blocks;
  P.cu = a.cu_tokens;
  P.kv_len = a.kv_len;
  P.out = reinterpret_cast<__nv_bfloat16*>(a.out);
  P.lse = a.lse;
  P.sink = a.sink;
  P.clusters = cluster_count(a);
  P.start = start_tiles(a);
  P.block_rows = paired(a) ? 256 : 128;
  const Workspace at(P.clusters, P.block_rows);
  P.part_o = static_cast<float*>(ws);
  P.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) + at.ml);
  P.desc = reinterpret_cast<int4*>(static_cast<uint8_t*>(ws) + at.desc);
  P.err = error_word();
  if (!P.err) return DSA_ERR_CUDA;
  const int st = paired(a) ? launch<2>(P, a, s) : launch<1>(P, a, s);
  if (st != DSA_OK || P.clusters == 1) return st;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  // no more CTAs than items: the most that the clusters can leave
  const long long items = static_cast<long long>(P.clusters) * (P.block_rows / 32) * (kDv / 8), most = 4ll * sm_count();
  cfg.gridDim = dim3(static_cast<unsigned>(items < most ? items : most));
  cfg.blockDim = dim3(32 * kMergeWarps);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, latent_merge_kernel, P));
}

}  // namespace dsa
