// Sparse MLA flash attention over the top-k rows of a 4-bit latent cache, on
// tcgen05.
//
//   out[t,h] = sum_j e^{s_j} v_j / (sum_j e^{s_j} [+ e^{sink[h]}]),
//   s_j = scale q[t,h] . k_j, k_j the dequantised row, v_j its 512 latent dims
//
// Work items (token, block of 128 heads, chunk of selected rows) go round robin
// to persistent 2-CTA clusters; an item is a run of tiles of 128 rows.  An O
// accumulator [128 x 512] in fp32 fills a CTA's tensor memory, so the two
// products live in different CTAs:
//
//   CTA 0: S = q . K^T (M = 128 heads, N = 128 rows, K = 576) and the softmax.
//          The latent part of q is the A operand in tensor memory (256
//          columns), its rotary part in shared memory; S is double-buffered in
//          the other 256 columns, each buffer filled in two halves of N = 64.
//   CTA 1: O += P . V with P sent over by CTA 0 and the values read MN-major from
//          the converted rows.  P goes from a staging buffer by bulk copies between
//          the CTAs' shared memories: 21 bytes a clock, beside the load/store pipe
//          (st.async from the softmax threads took some 2800 clocks a tile and held
//          up the conversion's stores behind it; 3.41 ms for the 4096-token case).
//
// Both convert the rows from 4 bits to bf16, three instructions per pair of dims,
// exact, into one of two 64 KB slots (64 rows x 512 dims, 128B-swizzled), which CTA 0
// reads K-major and CTA 1 MN-major; eight warps fill each while the MMA takes the
// other.  A warp loads its rows into registers a tile ahead, two rows of 16 lanes an
// instruction: 584 clocks of the load path for 128 rows.  Measured against it: 16-byte
// asynchronous copies 812; four lanes a row (which slots of 128 rows x 128 dims for
// N = 128 MMAs ask for) 1854; TMA gathers of four rows 3200, bulk copies of a row 7400.
// N = 64 costs the tensor core 45 clocks a K = 16 step where N = 128 takes 64 for twice
// the rows, which is not what bounds it.  q goes through the same slots of CTA 0, by TMA
// and then into tensor memory.
//
// Measured: 4096 tokens of 128 heads over 2048 of 8192 rows each 2.31 ms, 1012 TFLOP/s;
// 32 sequences of 4096 to 131072 rows 43.0 us; 8 tokens 24.6 us, one 19.3.  With the
// products, the exponentials, the conversion and the row loads taken out the long case
// still takes 1.9 ms: it is bound by the hand-overs between the roles (a buffer of S from
// products to exponentials to P on its way) and by instruction fetch.  No unit is busy for
// more than two thirds of the time, and forms with more code in the loops are slower even
// where they wait less (S in halves of 64 rows 2.48 ms; slots filled by all sixteen warps
// in turn 2.38).  The short cases are bound by their chain of first steps, each through
// cold code: indices, rows, q, the products, and 256 KB of O that one SM writes.
#include <algorithm>
#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include "dsa_internal.h"
#include "dsa_ptx.cuh"
#include "kv4.cuh"

namespace dsa {
namespace {

constexpr int kDqk = 576, kDv = 512;
constexpr int kTile = 128;                 // rows per tile
constexpr int kAtom = 16384;               // 128 rows (or heads) x 128 bytes
constexpr int kHalf = 64;                  // rows of a slot
constexpr int kSlot = 4 * kAtom;           // 64 rows x 512 dims bf16: 8 atoms of 64 rows x 128 bytes
constexpr int kPSlot = 2 * kAtom;          // P [128 heads x 128 rows] bf16
constexpr int kDescs = 8;                  // tile descriptors: how far the lookups run ahead of the slowest role
// Tries of a barrier, measured at 2070 MHz: by one lane while the others of its warp are
// parked 56 clocks at the least (186 in this kernel's long calls), by a whole warp 7790.
constexpr uint64_t kTryNs = 27;
constexpr uint32_t kWarpTries = 139;       // a warp's try in units of the shortest
// 28 warps in seven warpgroups: 0-1 softmax (CTA 0), correction and epilogue
// (CTA 1); 2-5 conversion; 6 MMA issue, row lookups, and q loads and rotary K loads
// (CTA 0) or the news of P's use and arrival (CTA 1).  The launch grants 72 registers
// a thread: 896 x 72 = 256 x 88 + 512 x 64 + 128 x 72.  (ptxas spills two words, 40 bytes
// of stores and 112 of reloads in all; without the softmax or the row lookups none, without
// the conversion 40 and 100.)
constexpr int kThreads = 896;
constexpr int kSoftWarps = 8, kConvWarps = 16, kFirstConv = 8, kMmaWarp = 24, kRowWarp = 25, kAuxWarp = 26,
              kAux2Warp = 27;
constexpr int kRegsLaunch = 72, kRegsSoft = 88, kRegsConv = 64, kRegsLast = 72;
static_assert(256 * kRegsSoft + 512 * kRegsConv + 128 * kRegsLast <= kThreads * kRegsLaunch,
              "register split exceeds the launch allocation");
constexpr uint32_t kPBytes0 = kAtom + 512, kPBytes1 = kAtom;  // the halves of a P tile, the first with the rescale factors
constexpr uint32_t kFinalBytes = 128 * 16;  // per head: two partial softmaxes' maximum and sum
constexpr uint32_t kTmemS = 256;            // CTA 0: q in columns [0, 256), S in [256, 512)

// Dynamic shared memory, after the slots.  CTA 0: q's rotary part, two rotary K
// buffers, P and its rescale factors on their way out, the running maxima.  CTA 1:
// two P slots, the output staging, rescale factors, finals.
constexpr int kOffQrope = 2 * kSlot, kOffKrope = kOffQrope + kAtom, kOffPst = kOffKrope + 2 * kAtom,
              kOffMax = kOffPst + kPSlot + 512, kEnd0 = kOffMax + 1024;
constexpr int kOffP = 2 * kSlot, kOffStage = kOffP + 2 * kPSlot, kOffAlpha = kOffStage + kAtom,
              kOffFinal = kOffAlpha + 1024, kEnd1 = kOffFinal + 2048;
constexpr int kSmem = 1024 + (kEnd0 > kEnd1 ? kEnd0 : kEnd1);
static_assert(kSmem + 1024 + kDescs * 544 <= 232448, "shared memory of a CTA");

struct AttnKv4Params {
  int T, B, n_q, H, topk, max_L, n_chunks, chunk_rows, head_blocks, items;
  float scale_log2;
  const uint8_t* kv4;
  int64_t rows;
  const int32_t* block_table;
  int block_size, max_blocks;  // (a contiguous cache: pages of max_L rows, a sequence each)
  uint32_t page_mul, page_shift;  // i / block_size = i page_mul >> page_shift for 0 <= i < 2^31
  const int32_t* idx;
  uint16_t* out;
  float* lse;
  const float* sink;
  const int32_t* seq;
  float4* part_o;   // [T][n_chunks][512 / 4][H]: each chunk's O, when n_chunks > 1
  float2* part_ml;  // [T][n_chunks][H]: (maximum, sum) in log2 units
  uint32_t* err;
};

// What the roles need to know of a tile.
struct __align__(16) TileDesc {
  int row[kTile];     // its physical rows; -1: read as zeros
  uint32_t valid[4];  // rows that are selected (the others are masked)
  int info;           // rows up to the item's last selected one (0: it selects nothing); + kLast: the item's last tile
};
constexpr int kLast = 1 << 16;
struct Desc {
  int rows;
  bool last;
};

struct __align__(8) Bars {
  uint64_t full[2], empty[2];              // slots (CTA 0: K and q; CTA 1: V)
  uint64_t dfull[kDescs], dempty[kDescs];  // tile descriptors
  uint64_t kpfull[2], kpempty[2];          // CTA 0: rotary K buffers
  uint64_t sfull[2], sempty[2];            // CTA 0: S buffers
  uint64_t mchain[4];                      // CTA 0: a tile's running maxima are known (per warp quadrant)
  uint64_t psent[2][2], pfree[2];          // CTA 0: a half of P has arrived; P slot of CTA 1 free
  uint64_t qgroup[2], qready, qfree, qpfull;  // CTA 0: a slot of q read; all of q stored; MMAs done with q; its rotary part
  uint64_t cdone;                          // CTA 0: every slot of the item is converted
  uint64_t ffree;                          // CTA 0: CTA 1 has read the finals
  uint64_t pfull[2][2], pcons[2];          // CTA 1: P slots (halves of 64 rows)
  uint64_t ready[2], odone[2], ffull;      // CTA 1: correction / MMA
  uint64_t stfull[2], stfree[2], stored;   // CTA 1: output staging; an item's P slot is no more needed for it
  uint64_t lfull[8];                       // CTA 1: output staging of the cluster's last item
  uint64_t mdrain;                         // the MMA thread's last commit
};

__device__ __forceinline__ float neg_inf() { return -__int_as_float(0x7f800000); }

// One thread of the warp.  (The compiler knows it for one: an MMA then takes half
// the instructions that it takes under lane == 0.)
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(e));
  return e != 0;
}
__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
  asm volatile("{\n.reg .b64 st;\nmbarrier.arrive.shared::cta.b64 st, [%0], %1;\n}" ::"r"(smem_u32(bar)), "r"(n) : "memory");
}
__device__ __forceinline__ void tma_load_3d(void* dst, const void* tmap, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_prefetch_3d(const void* tmap, int x, int y, int z) {  // into the L2
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];"
               ::"l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z) : "memory");
}
// Bulk copy to the peer CTA's shared memory, completing on the peer's barrier.
__device__ __forceinline__ void bulk_s2peer(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(dst), "r"(src), "r"(bytes), "r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
      ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// After a wait gave up: waits for a copy that completes on `bar`.  The barrier may
// have moved on to a later use (then the copy has landed, but its parity is gone),
// so this waits a tenth of a millisecond at most, many times a copy's time.
__device__ __forceinline__ void drain_copy(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_test(bar, parity) && globaltimer_ns() - t0 < 100000) {}
}

// Bounded wait for a phase of a barrier, in as little code as will do: the roles of
// this kernel run at the same time, and the two CTAs of a cluster, from one
// instruction cache.  (With the other kernels' waits inlined an earlier form was 133
// KB and a third of the cache's requests missed: 5.97 ms for the 4096-token case;
// taking 3 KB of code that this case never reaches out of an 78 KB form won 5%.)
// Time is counted in tries, a warp's for kWarpTries of a lane's: `limit` of them last
// for the limit in force at the least, and for a lane's waits up to 3.5 times it.
// (Reading the global timer after each failed try instead: 2048 tokens 1305 us for 1204.)
// Who runs out sets *tries to 0 for the CTA's end and leaves its role; the roles that
// wait for it run out in their turn.  The lanes of a waiting warp vote on every try, so
// they go on or give up together (one that left alone would leave the others at the
// next warp barrier) and the loop's branches are uniform: with the vote after the loop
// and the limit in shared memory there were 5 KB more of code, and the 4096-token case
// took 2.45 ms instead of 2.35; with one lane polling for its warp 4.95.
// A wait is by parity: it tells a phase from the one before and the one after only, so
// no role may be two uses of a barrier ahead of or behind the one it waits for.
template <bool kCluster, bool kWarp>
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, uint32_t limit, volatile uint32_t* tries) {
#pragma unroll 1
  for (uint32_t n = 0;; n += kWarp ? kWarpTries : 1) {
    bool done = kCluster ? mbar_probe_cluster(bar, parity) : mbar_probe(bar, parity);
    if (kWarp) done = __all_sync(0xffffffffu, done);
    if (done) return true;
    if (n >= limit) {
      *tries = 0;
      return false;
    }
  }
}
// Waits of one thread, and of a whole warp.
#define WAIT1(bar, parity) wait_phase<false, false>(&(bar), (parity), limit, tries)
#define WAIT1_CLUSTER(bar, parity) wait_phase<true, false>(&(bar), (parity), limit, tries)
#define WAIT(bar, parity) wait_phase<false, true>(&(bar), (parity), limit, tries)
#define WAIT_CLUSTER(bar, parity) wait_phase<true, true>(&(bar), (parity), limit, tries)

__global__ void __launch_bounds__(kThreads, 1)
    attn_kv4_kernel(const __grid_constant__ AttnKv4Params P, const __grid_constant__ CUtensorMap tmap_q,
                    const __grid_constant__ CUtensorMap tmap_o) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ Bars bars;
  __shared__ TileDesc descs[kDescs];
  __shared__ uint32_t tmem_base;
  __shared__ uint32_t wait_tries;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const int cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;
  uint8_t* sP = smem + kOffP;
  float* sAlpha = reinterpret_cast<float*>(smem + kOffAlpha);  // [2][128]
  float* sFinal = reinterpret_cast<float*>(smem + kOffFinal);  // [4][128]: maximum, sum of each softmax warpgroup
  float* sMax = reinterpret_cast<float*>(smem + kOffMax);      // [2][128]: running maxima after even / odd tiles

  if (warp == 1) {  // a barrier a lane
    for (int i = lane; i < static_cast<int>(sizeof(Bars) / 8); i += 32) {
      uint64_t* const b = reinterpret_cast<uint64_t*>(&bars) + i;
      auto in = [&](const uint64_t* first, int n) { return b >= first && b < first + n; };
      uint32_t count = 1;
      if (in(bars.full, 2) || in(bars.qgroup, 2)) count = kConvWarps / 2;
      if (b == &bars.qready || b == &bars.cdone) count = kConvWarps;
      // descriptors are read by the conversion and softmax / correction warps and
      // three more roles: MMA, q and rotary loads / the two that tell of P
      if (in(bars.dempty, kDescs)) count = kConvWarps + kSoftWarps + 3;
      if (in(bars.kpfull, 2)) count = 32;
      if (in(bars.sempty, 2)) count = 4;
      if (in(bars.ready, 2) || b == &bars.ffree || in(bars.stfull, 2) || in(bars.lfull, 8)) count = kSoftWarps;
      mbar_init(b, count);
    }
    fence_mbar_init();
    __syncwarp();
    if (rank == 1 && lane == 0) {
      for (int i = 0; i < 2; ++i) {
        mbar_arrive_expect_tx(&bars.pfull[i][0], kPBytes0);
        mbar_arrive_expect_tx(&bars.pfull[i][1], kPBytes1);
      }
      mbar_arrive_expect_tx(&bars.ffull, kFinalBytes);
    }
  }
  if (warp == 2 && lane == 0)
    wait_tries = static_cast<uint32_t>(min(wait_limit_ns(P.err) / kTryNs + 1, static_cast<uint64_t>(0xffffffffu)));
  if (warp == 0) tmem_alloc(&tmem_base, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  volatile uint32_t* tries = &wait_tries;
  const uint32_t limit = wait_tries;
  const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
  cluster_sync();  // both CTAs' barriers are initialised before any remote use
  griddep_launch_dependents();

  // The next tile's descriptor, for a whole warp or for one thread.
  uint32_t dc = 0;
  auto read_desc = [&](Desc& d) {
    const int info = descs[dc % kDescs].info;
    d.rows = info & (kLast - 1);
    d.last = info >= kLast;
    ++dc;
  };
  auto free_desc = [&]() { mbar_arrive(&bars.dempty[(dc - 1) % kDescs]); };
  auto next_desc1 = [&](Desc& d) -> bool {
    if (!WAIT1(bars.dfull[dc % kDescs], (dc / kDescs) & 1)) return false;
    read_desc(d);
    free_desc();
    return true;
  };

  if (warp >= kFirstConv && warp < kFirstConv + kConvWarps) {
    setmaxnreg_dec<kRegsConv>();
    // ------------------------------------------------- conversion (both CTAs)
    // Eight warps fill a slot, eight rows each, once for q (by TMA; they put it
    // into tensor memory) and once for every tile; what a warp does between two fills
    // goes on while the MMA reads its slot.  A lane converts 32 dims (16 bytes of codes,
    // piece pc) of rows 2 i + rp of its warp's eight.  Lanes are numbered, and odd pairs
    // of pieces stored in another order, so that a quarter warp's stores meet every bank
    // once.
    const int cw = warp - kFirstConv, g = cw >> 3;  // g: its slot
    const int pc = ((lane >> 3) << 2) | (lane & 3), rp = (lane >> 2) & 1;
    const bool swap = (pc & 2) != 0;
    const uint32_t scale_lo = swap ? 0x4441u : 0x4440u;
    const uint32_t slots = smem_u32(smem);
    const uint32_t dst0 = slots + g * kSlot + (pc >> 1) * (kSlot / 8) + ((cw & 7) * 8 + rp) * 128 +
                          ((((pc & 1) * 4) ^ (swap ? 2 : 0) ^ rp) << 4);
    const uint8_t* const src = P.kv4 + pc * 16;
    const int scale_off = kKv4Scales - pc * 14;
    const int my_row = cw * 8 + rp;
    uint4 c[4];  // piece i: row 2 i + my_row
    uint32_t sc[4];
    auto load = [&](int r, uint4& c, uint32_t& s) {
      c = make_uint4(0, 0, 0, 0);
      s = 0;
      if (r >= 0) {
        const uint8_t* p = src + static_cast<size_t>(r) * kKv4Row;
        c = __ldg(reinterpret_cast<const uint4*>(p));
        s = __ldg(reinterpret_cast<const uint16_t*>(p + scale_off));
      }
    };
    uint32_t uses = 0;
    Desc cur{0, false};
    bool ok = WAIT(bars.dfull[0], 0);
    if (ok) {
      const int* rows = descs[0].row + my_row;
      int r[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = rows[2 * i];
      read_desc(cur);
      __syncwarp();
      if (lane == 0) free_desc();
#pragma unroll
      for (int i = 0; i < 4; ++i) load(r[i], c[i], sc[i]);
    }
#pragma unroll 1
    for (int item = cluster, n = 0; item < P.items && ok; item += clusters, ++n) {
      if (rank == 0) {
        // q: 256 dims of the 128 heads a slot (4 atoms), lane = head, two atoms a warp, in
        // 16 registers (in 32, next to a tile's rows: 2.43 ms for 2.31)
        if (n > 0) ok = WAIT(bars.qfree, (n - 1) & 1);
        if (!ok || !WAIT(bars.full[g], uses & 1)) { ok = false; break; }
        tc_fence_after();
#pragma unroll 1
        for (int b = cw & 4, e = b + 4; b < e; ++b) {  // half an atom
          uint32_t r[16];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint4 v = lds128(slots + g * kSlot + (b >> 1) * kAtom + sw128_off((cw & 3) * 32 + lane, (b & 1) * 4 + k));
            r[4 * k] = v.x; r[4 * k + 1] = v.y; r[4 * k + 2] = v.z; r[4 * k + 3] = v.w;
          }
          tmem_st16(tmem + lane_off + (g * 8 + b) * 16, r);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.qgroup[g]);
        if ((cw & 7) == 0) {  // all have read the slot
          if (!WAIT(bars.qgroup[g], n & 1)) { ok = false; break; }
          if (lane == 0) mbar_arrive(&bars.empty[g]);
        }
        ++uses;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.qready);
      }
#pragma unroll 1
      while (ok) {
        if (cur.rows > 0) {
          if (!WAIT(bars.empty[g], (uses & 1) ^ 1)) { ok = false; break; }
          if (cw * 8 < cur.rows) {  // (rows past the last 16 are not read by the MMA)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t dst = (dst0 + i * 256) ^ (i << 5);
              const Kv4Scale lo = kv4_scale(__byte_perm(sc[i], 0, scale_lo)),
                             hi = kv4_scale(__byte_perm(sc[i], 0, scale_lo ^ 1u));
              uint4 w = c[i];
              if (swap) w = make_uint4(w.z, w.w, w.x, w.y);
              sts128(dst, kv4_codes8(w.x, lo));
              sts128(dst ^ 16u, kv4_codes8(w.y, lo));
              sts128(dst ^ 32u, kv4_codes8(w.z, hi));
              sts128(dst ^ 48u, kv4_codes8(w.w, hi));
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.full[g]);  // (the MMA's thread fences the proxies)
          ++uses;
        }
        const bool last = cur.last;
        if (!last || item + clusters < P.items) {  // the next tile's rows, maybe of the next item
          const int* rows = descs[dc % kDescs].row + my_row;
          if (!WAIT(bars.dfull[dc % kDescs], (dc / kDescs) & 1)) { ok = false; break; }
          int r[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) r[i] = rows[2 * i];
          read_desc(cur);
          __syncwarp();
          if (lane == 0) free_desc();  // (before the loads: an arrival waits for those under way)
#pragma unroll
          for (int i = 0; i < 4; ++i) load(r[i], c[i], sc[i]);
        }
        if (last) break;
      }
      if (ok && rank == 0 && lane == 0) mbar_arrive(&bars.cdone);
    }
  } else if (warp < kSoftWarps) {
    setmaxnreg_inc<kRegsSoft>();
    const int hrow = (warp & 3) * 32 + lane, hf = warp >> 2;
    bool ok = true;
    uint32_t tc = 0;
    if (rank == 0) {
      // ------------------------------------------------- softmax (CTA 0)
      // Two warpgroups take tiles in turn (group hf the tiles of S buffer hf), a
      // thread a head's 128 scores; the running maximum goes from tile to tile
      // through shared memory, the sums stay partial until the item ends.
      const uint32_t stage = smem_u32(smem + kOffPst);
      float* stage_alpha = reinterpret_cast<float*>(smem + kOffPst + kPSlot);
      const uint32_t s_tmem = tmem + lane_off + kTmemS + hf * kTile;
      const uint32_t remote_p = mapa(smem_u32(sP), 1) + hf * kPSlot, remote_alpha = mapa(smem_u32(sAlpha), 1) + hf * 512,
                     remote_pfull = mapa(smem_u32(&bars.pfull[hf][0]), 1);
      const uint32_t remote_final = mapa(smem_u32(sFinal), 1) + (hf * 256 + hrow) * 4;
      const uint32_t remote_ffull = mapa(smem_u32(&bars.ffull), 1);
      const uint64_t scale2 = pack_f32x2(P.scale_log2, P.scale_log2), one2 = pack_f32x2(1.f, 1.f);
#pragma unroll 1
      for (int item = cluster, n = 0; item < P.items && ok; item += clusters, ++n) {
        float m_ref = neg_inf(), l_sum = 0.f;  // this group's part: sum relative to m_ref
        bool first = true;
#pragma unroll 1
        while (ok) {
          Desc d;
          const TileDesc& td = descs[dc % kDescs];
          if (!WAIT(bars.dfull[dc % kDescs], (dc / kDescs) & 1)) { ok = false; break; }
          read_desc(d);
          const bool mine = d.rows > 0 && (tc & 1) == static_cast<uint32_t>(hf);
          uint4 valid = make_uint4(0, 0, 0, 0);
          if (mine) valid = *reinterpret_cast<const uint4*>(td.valid);
          __syncwarp();
          if (lane == 0) free_desc();
          if (mine) {
            const uint32_t ph = (tc >> 1) & 1;
            if (!WAIT(bars.sfull[hf], ph)) { ok = false; break; }
            tc_fence_after();
            if ((valid.x & valid.y & valid.z & valid.w) != 0xffffffffu) {  // rows that are not selected
#pragma unroll 1
              for (int x = 0; x < 4; ++x) {
                uint32_t s[32];
                tmem_ld32(s_tmem + x * 32, s);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 32; ++k)
                  if (!((valid.x >> k) & 1u)) s[k] = 0xff800000u;
                tmem_st32(s_tmem + x * 32, s);
                valid = make_uint4(valid.y, valid.z, valid.w, valid.x);
              }
              tmem_st_wait();
            }
            // two passes over the scores, 32 at a time: the maximum, then the
            // exponentials (reading them twice keeps registers and code small)
            float m_tile = neg_inf();
#pragma unroll 1
            for (int x = 0; x * 32 < d.rows; ++x) {
              uint32_t s[32];
              tmem_ld32(s_tmem + x * 32, s);
              tmem_ld_wait();
              float mt[4] = {m_tile, neg_inf(), neg_inf(), neg_inf()};
#pragma unroll
              for (int k = 0; k < 32; ++k) mt[k & 3] = fmaxf(mt[k & 3], __uint_as_float(s[k]));
              m_tile = fmaxf(fmaxf(mt[0], mt[1]), fmaxf(mt[2], mt[3]));
            }
            m_tile *= P.scale_log2;
            // the running maximum moves only when a tile exceeds it by more than 2^8
            if (tc > 0 && !WAIT(bars.mchain[warp & 3], (tc - 1) & 1)) { ok = false; break; }
            const float m_prev = first ? neg_inf() : sMax[((tc - 1) & 1) * 128 + hrow];
            const float m_new = m_tile > m_prev + 8.f ? m_tile : m_prev;
            sMax[(tc & 1) * 128 + hrow] = m_new;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.mchain[warp & 3]);
            const float msub = m_new == neg_inf() ? 0.f : -m_new;  // (nothing selected so far: every p is 0)
            const float alpha = ex2_approx(m_prev + msub);         // 0 from -inf
            l_sum *= ex2_approx(m_ref + msub);
            m_ref = m_new;
            // the exponentials of 64 rows into registers, then into their half of the
            // staging once the previous tile's half has gone, and on their way
            const uint64_t msub2 = pack_f32x2(msub, msub);
            uint64_t sum2[2] = {0, 0};
#pragma unroll 1
            for (int a = 0; a < 2; ++a) {
              uint32_t pk[32];
              if (a * kHalf >= d.rows) {
                // A half without rows is sent for its barrier only, and no product reads it:
                // whatever the registers hold, said without an instruction.  (2048 tokens:
                // zeros take 3% longer, no stores 1.6%, the barrier's count without a copy 3.5%.)
#pragma unroll
                for (int k = 0; k < 32; ++k) asm volatile("" : "=r"(pk[k]));
              } else
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                uint32_t s[32];
                tmem_ld32(s_tmem + a * kHalf + x * 32, s);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                  const uint64_t y =
                      fma_f32x2(pack_f32x2(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1])), scale2, msub2);
                  const float p0 = ex2_approx(lo_f32(y)), p1 = ex2_approx(hi_f32(y));
                  sum2[k & 1] = fma_f32x2(pack_f32x2(p0, p1), one2, sum2[k & 1]);
                  __nv_bfloat162 pb = __floats2bfloat162_rn(p0, p1);
                  pk[x * 16 + k] = *reinterpret_cast<uint32_t*>(&pb);
                }
              }
              if (a == 1) {  // S is read
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.sempty[hf]);
              }
              if (tc > 0 && !WAIT_CLUSTER(bars.psent[hf ^ 1][a], ((tc - 1) >> 1) & 1)) { ok = false; break; }
              if (a == 0) {
                if (!WAIT_CLUSTER(bars.pfree[hf], ph ^ 1)) { ok = false; break; }
                stage_alpha[hrow] = first ? 0.f : alpha;
              }
              const uint32_t row = stage + a * kAtom + hrow * 128, c = (hrow & 7) << 4;
#pragma unroll
              for (int k = 0; k < 8; ++k)
                sts128(row + (c ^ (k << 4)), make_uint4(pk[4 * k], pk[4 * k + 1], pk[4 * k + 2], pk[4 * k + 3]));
              fence_proxy_async_smem();  // generic writes -> bulk copy reads
              __syncwarp();
              if (lane == 0) {
                const uint32_t off = a * kAtom + (warp & 3) * 4096, bar = remote_pfull + a * 8;
                bulk_s2peer(remote_p + off, stage + off, 4096, bar);
                if (a == 0) bulk_s2peer(remote_alpha + (warp & 3) * 128, smem_u32(stage_alpha) + (warp & 3) * 128, 128, bar);
              }
              __syncwarp();
            }
            if (!ok) break;
            l_sum += (lo_f32(sum2[0]) + hi_f32(sum2[0])) + (lo_f32(sum2[1]) + hi_f32(sum2[1]));
          }
          if (d.rows > 0) {
            first = false;
            ++tc;
          }
          if (d.last) break;
        }
        if (ok && n > 0) ok = WAIT_CLUSTER(bars.ffree, (n - 1) & 1);
        if (ok) {
          st_async_b32(remote_final, __float_as_uint(m_ref), remote_ffull);
          st_async_b32(remote_final + 512, __float_as_uint(l_sum), remote_ffull);
        }
      }
    } else {
      // ------------------------------- correction and epilogue (CTA 1)
      const uint32_t remote_ffree = mapa(smem_u32(&bars.ffree), 0);
      uint32_t consumed = 0;  // odone phases observed
      uint32_t stores = 0;    // output atoms
#pragma unroll 1
      for (int item = cluster, n = 0; item < P.items && ok; item += clusters, ++n) {
        const int chunk = item % P.n_chunks, th = item / P.n_chunks, hb = th % P.head_blocks, t = th / P.head_blocks;
        bool first = true;
#pragma unroll 1
        while (ok) {
          Desc d;
          if (!WAIT(bars.dfull[dc % kDescs], (dc / kDescs) & 1)) { ok = false; break; }
          read_desc(d);
          __syncwarp();
          if (lane == 0) free_desc();
          if (d.rows > 0) {
            const uint32_t ps = tc & 1;
            if (!WAIT_CLUSTER(bars.pfull[ps][0], (tc >> 1) & 1)) { ok = false; break; }  // with the rescale factors
            const float alpha = sAlpha[ps * 128 + hrow];
            if (__any_sync(0xffffffffu, alpha != 1.f) && !first) {
              // O must hold the previous tile's product before it is rescaled.
              if (consumed < tc) {
                ok = WAIT(bars.odone[consumed & 1], (consumed >> 1) & 1);
                ++consumed;
              }
              if (!ok) break;
              tc_fence_after();
#pragma unroll 1
              for (int c0 = hf * 256; c0 < hf * 256 + 256; c0 += 32) {
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
            if (lane == 0) mbar_arrive(&bars.ready[ps]);
            // keep at most one completed product unobserved
            if (consumed < tc) {
              ok = WAIT(bars.odone[consumed & 1], (consumed >> 1) & 1);
              ++consumed;
            }
            ++tc;
            first = false;
          }
          if (d.last) break;
        }
        // Every product is in O and the partial softmaxes of each head have arrived:
        // normalise, convert to bf16 into a swizzled staging atom and write it with
        // TMA stores, 64 columns x 128 heads per box (heads past H are clipped by the
        // tensor map), each of the two warps of a head half of the columns.
        if (ok && consumed < tc) {
          ok = WAIT(bars.odone[consumed & 1], (consumed >> 1) & 1);
          ++consumed;
        }
        if (ok) ok = WAIT_CLUSTER(bars.ffull, n & 1);
        if (!ok) break;
        tc_fence_after();
        const float m0 = sFinal[hrow], l0 = sFinal[128 + hrow], m1 = sFinal[256 + hrow], l1 = sFinal[384 + hrow];
        __syncwarp();
        if (warp == 0 && lane == 0) mbar_arrive_expect_tx(&bars.ffull, kFinalBytes);  // the next item's
        if (lane == 0) mbar_arrive_remote(remote_ffree);
        const float m = fmaxf(m0, m1), mz = m == neg_inf() ? 0.f : m;
        const float l = l0 * ex2_approx(m0 - mz) + l1 * ex2_approx(m1 - mz);
        // The sink adds 2^s2 to the denominator, all relative to the larger of the
        // maximum and s2.  (Split chunks get it in the merge.)
        const int h = hb * 128 + hrow;
        float mx = m, num = 1.f, den = l;
        if (P.sink != nullptr && P.n_chunks == 1) {
          const float k2 = (h < P.H ? __ldg(P.sink + h) : neg_inf()) * 1.4426950408889634f;
          mx = fmaxf(m, k2);
          if (mx != neg_inf()) {
            num = ex2_approx(m - mx);
            den = l * num + ex2_approx(k2 - mx);
          }
        }
        const float inv_l = den == 0.f ? 0.f : num / den;
        const float lse2 = den == 0.f ? neg_inf() : mx + log2f(den);  // log2 units
        // The staging is the V slots after the cluster's last item; else an atom of its
        // own and the P slot of the item's last tile, which `stored` gives back.
        const bool final_item = item + clusters >= P.items;
        const uint32_t c = hrow * 128 + (((hf * 4) ^ (hrow & 7)) << 4);
        if (P.n_chunks > 1) {
          // A chunk (its cluster's only item) leaves O as it is, in fp32: lanes are heads,
          // so four columns of 32 heads are a run of 512 bytes, straight from registers.
          // (Rounded to bf16 and through the staging 8 tokens took 24.0 us instead of 24.8
          // and 32 sequences 49.5 instead of 47.2; the output of the 32 was off by 0.0026 of itself
          // instead of 0.0021.)
          if (!first) {  // (what selects nothing writes no O: the merge gives it no weight)
            float4* o = P.part_o + (static_cast<size_t>(t * P.n_chunks + chunk) * (kDv / 4) + hf * (kDv / 8)) * P.H + h;
#pragma unroll 1
            for (int i = 0; i < 8; ++i, o += 8 * P.H) {
              uint32_t v[32];
              tmem_ld32(tmem + lane_off + hf * 256 + i * 32, v);
              tmem_ld_wait();
              if (h < P.H)
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  o[k * P.H] = make_float4(__uint_as_float(v[4 * k]), __uint_as_float(v[4 * k + 1]),
                                           __uint_as_float(v[4 * k + 2]), __uint_as_float(v[4 * k + 3]));
            }
            if (warp == 0 && lane == 0) mbar_arrive(&bars.stored);
          }
        } else if (first) {  // nothing selected: zeros
          if (h < P.H) {
            uint4* o = reinterpret_cast<uint4*>(P.out + (static_cast<size_t>(t) * P.H + h) * kDv + hf * 256);
#pragma unroll 1
            for (int k = 0; k < 32; ++k) o[k] = make_uint4(0, 0, 0, 0);
          }
        } else {
#pragma unroll 1
          for (int i = 0; i < 8; ++i, ++stores) {  // 64 columns a round
            // every store of the last item, or the one before last of this, has read its atom
            // (the cluster's last item has one for every round)
            const uint32_t before = stores - (i == 0 ? 1 : 2);
            if (!final_item && stores > 0 && i != 1 && !WAIT(bars.stfree[before & 1], (before >> 1) & 1)) {
              ok = false;
              break;
            }
            const int b = i % 3;
            const uint32_t atom = final_item ? i * kAtom : b == 0 ? kOffStage : kOffP + ((tc - 1) & 1) * kPSlot + (b - 1) * kAtom;
            const uint32_t row = smem_u32(smem) + atom + c;
            uint32_t v[32];
            tmem_ld32(tmem + lane_off + i * 64 + hf * 32, v);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              __nv_bfloat162 w =
                  __floats2bfloat162_rn(__uint_as_float(v[2 * k]) * inv_l, __uint_as_float(v[2 * k + 1]) * inv_l);
              v[k] = *reinterpret_cast<uint32_t*>(&w);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
              sts128(row ^ (k << 4), make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]));
            fence_proxy_async_smem();
            __syncwarp();
            uint64_t* const full = final_item ? &bars.lfull[i] : &bars.stfull[stores & 1];
            if (lane == 0) mbar_arrive(full);
            if (warp == 0 && lane == 0) {  // the eight warps have written the atom
              if (WAIT1(*full, final_item ? 0 : (stores >> 1) & 1)) {
                tma_store_3d(&tmap_o, smem + atom, i * 64, hb * 128, t);
                bulk_commit_group();
                if (i == 7) {
                  bulk_wait_group_read0();
                  mbar_arrive(&bars.stored);
                } else if (!final_item) {
                  asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                }
                mbar_arrive(&bars.stfree[stores & 1]);
              }
            }
            __syncwarp();
          }
        }
        tc_fence_before();
        if (hf == 0 && h < P.H) {
          if (P.n_chunks == 1) {
            if (P.lse != nullptr) P.lse[static_cast<size_t>(t) * P.H + h] = lse2 * 0.69314718055994531f;
          } else {
            P.part_ml[(static_cast<size_t>(t) * P.n_chunks + chunk) * P.H + h] = make_float2(m, l);
          }
        }
      }
    }
  } else {
    setmaxnreg_inc<kRegsLast>();
    if (warp == kRowWarp) {
      // ---------------------------------------------- row lookups (both CTAs)
      griddep_wait();  // the index rows come from the previous kernel
      bool ok = true;
#pragma unroll 1
      for (int item = cluster; item < P.items && ok; item += clusters) {
        const int chunk = item % P.n_chunks, t = item / P.n_chunks / P.head_blocks;
        int b = t / P.n_q;
        bool bad_seq = false;
        if (P.seq != nullptr) {  // a token outside [0, B) reads no row and gets out = 0
          b = __ldg(P.seq + t);
          bad_seq = b < 0 || b >= P.B;
          if (bad_seq && lane == 0) atomicOr(P.err, kErrBadIndex);
        }
        const int slot_begin = chunk * P.chunk_rows;
        const int rows_here = bad_seq ? 0 : min(P.chunk_rows, P.topk - slot_begin);
        const int32_t* idx = P.idx + static_cast<size_t>(t) * P.topk + slot_begin;
        const int32_t* table = P.block_table == nullptr ? nullptr : P.block_table + static_cast<size_t>(b) * P.max_blocks;
        // rows 4 lane .. 4 lane + 3 of a tile, loaded a tile ahead (the first together
        // with the item's last slot)
        int s[4];
        auto page_of = [&](int i) { return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(i)) * P.page_mul) >> P.page_shift); };
        auto load_idx = [&](int j0, int n) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int i = j0 + 4 * lane + x;
            s[x] = i < n ? __ldg(idx + i) : -1;
          }
        };
        load_idx(0, rows_here);
        // the item ends at its last valid slot, found from the end
        int n_rows = rows_here;
        if (rows_here > 0) {
          const int last = __ldg(idx + rows_here - 1);
          if (last < 0 || last >= P.max_L) {
            n_rows = 0;
#pragma unroll 1
            for (int end = rows_here; end > 0 && n_rows == 0; end -= 256) {
              int mx = -1;
#pragma unroll
              for (int x = 0; x < 8; ++x) {
                const int i = end - 256 + x * 32 + lane;
                const int v = i >= 0 ? __ldg(idx + i) : -1;
                if (v >= 0 && v < P.max_L) mx = i;
              }
#pragma unroll
              for (int o = 16; o; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
              n_rows = mx + 1;
            }
          }
        }
#pragma unroll 1
        for (int j0 = 0; ok; j0 += kTile) {
          // a slot that selects nothing is masked; a row that does not exist is
          // recorded and reads as zeros
          int r[4];
          uint32_t nib = 0;
          bool bad = false;
          {
            int pg[4], off[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              if (s[x] >= P.max_L) s[x] = -1;
              const int i = page_of(s[x]);
              off[x] = s[x] - i * P.block_size;
              pg[x] = s[x] >= 0 && table != nullptr ? __ldg(table + i) : b;
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              r[x] = -1;
              if (s[x] >= 0) {
                nib |= 1u << x;
                const int64_t row = static_cast<int64_t>(pg[x]) * P.block_size + off[x];
                if (pg[x] < 0 || row >= P.rows) bad = true;
                else r[x] = static_cast<int>(row);
              }
            }
          }
          load_idx(j0 + kTile, n_rows);
          if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(P.err, kErrBadIndex);
          nib <<= (lane & 7) * 4;
#pragma unroll
          for (int o = 4; o; o >>= 1) nib |= __shfl_xor_sync(0xffffffffu, nib, o);
          const bool last = j0 + kTile >= n_rows;
          TileDesc& td = descs[dc % kDescs];
          if (!WAIT(bars.dempty[dc % kDescs], ((dc / kDescs) & 1) ^ 1)) { ok = false; break; }
          *reinterpret_cast<int4*>(&td.row[4 * lane]) = make_int4(r[0], r[1], r[2], r[3]);
          if ((lane & 7) == 0) td.valid[lane >> 3] = nib;
          // (up to a multiple of 16, which the second product reads whole: a zero weight
          // does not make up for what a NaN left in the slot, so those rows are zeros)
          if (lane == 0) td.info = max(0, min(kTile, (n_rows - j0 + 15) & ~15)) + (last ? kLast : 0);
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.dfull[dc % kDescs]);
          ++dc;
          if (last) break;
        }
      }
    } else if (warp == kMmaWarp && rank == 0) {
      // ---------------------------------------------- QK^T MMA (CTA 0)
      if (elect_one()) {
        uint32_t tc = 0, uses = 0;  // uses of every slot
        bool ok = true;
        const uint32_t base = smem_u32(smem);
#pragma unroll 1
        for (int item = cluster, n = 0; item < P.items && ok; item += clusters, ++n) {
          ok = WAIT1(bars.qready, n & 1) && WAIT1(bars.qpfull, n & 1);
          if (!ok) break;
          ++uses;
#pragma unroll 1
          while (ok) {
            Desc d;
            if (!next_desc1(d)) { ok = false; break; }
            if (d.rows > 0) {
              const uint32_t sb = tc & 1, ph = (tc >> 1) & 1;
              const uint32_t dt = tmem + kTmemS + sb * kTile;
              if (!WAIT1(bars.sempty[sb], ph ^ 1) || !WAIT1(bars.kpfull[sb], ph)) { ok = false; break; }
              fence_proxy_async_smem();  // cp.async data -> tensor core reads
              tc_fence_after();
              {
                const uint32_t idesc = idesc_f16(128, d.rows, kFmtBF16, 0, 0);
                const uint64_t ad = smem_desc(base + kOffQrope, 16, 1024, kSwizzle128B);
                const uint64_t bd = smem_desc(base + kOffKrope + sb * kAtom, 16, 1024, kSwizzle128B);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) mma_ss(dt, ad + kk * 2, bd + kk * 2, idesc, kk > 0 ? 1u : 0u);
              }
              mma_commit(&bars.kpempty[sb]);
#pragma unroll 1
              for (int x = 0; x < 2; ++x) {
                if (!WAIT1(bars.full[x], uses & 1)) { ok = false; break; }
                fence_proxy_async_smem();  // generic writes -> tensor core reads
                const int n16 = min(kHalf, d.rows - x * kHalf);
                if (n16 > 0) {  // (a slot without rows changes hands all the same)
                  tc_fence_after();
                  const uint32_t idesc = idesc_f16(128, n16, kFmtBF16, 0, 0);
                  uint64_t bd = smem_desc(base + x * kSlot, 16, 1024, kSwizzle128B);
#pragma unroll 1
                  for (int a = 0; a < 8; ++a, bd += kSlot / 8 >> 4)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) mma_ts(dt + x * kHalf, tmem + a * 32 + kk * 8, bd + kk * 2, idesc, 1u);
                }
                mma_commit(&bars.empty[x]);
              }
              if (!ok) break;
              mma_commit(&bars.sfull[sb]);
              ++uses;
              ++tc;
            }
            if (d.last) break;
          }
          if (ok) mma_commit(&bars.qfree);
        }
        // every MMA issued has completed before the tensor memory is freed
        mma_commit(&bars.mdrain);
        mbar_drain(&bars.mdrain, 0);
      }
    } else if (warp == kMmaWarp) {
      // ------------------------------------------------- PV MMA (CTA 1)
      if (elect_one()) {
        uint32_t tc = 0;
        bool ok = true;
        const uint32_t idesc = idesc_f16(128, 256, kFmtBF16, 0, 1);
        const uint32_t vbase = smem_u32(smem), pbase = smem_u32(sP);
#pragma unroll 1
        for (int item = cluster; item < P.items && ok; item += clusters) {
          uint32_t acc = 0;  // the item's first product overwrites O
#pragma unroll 1
          while (ok) {
            Desc d;
            if (!next_desc1(d)) { ok = false; break; }
            if (d.rows > 0) {
              const uint32_t ps = tc & 1;
              if (!WAIT1(bars.ready[ps], (tc >> 1) & 1)) { ok = false; break; }
#pragma unroll 1
              for (int x = 0; x < 2; ++x) {
                if (x == 1 && !WAIT1_CLUSTER(bars.pfull[ps][1], (tc >> 1) & 1)) { ok = false; break; }
                if (!WAIT1(bars.full[x], tc & 1)) { ok = false; break; }
                fence_proxy_async_smem();  // generic writes -> tensor core reads
                tc_fence_after();
                uint64_t ad = smem_desc(pbase + ps * kPSlot + x * kAtom, 16, 1024, kSwizzle128B);
                uint64_t bd = smem_desc(vbase + x * kSlot, kSlot / 8, 1024, kSwizzle128B);
#pragma unroll 1
                for (int r = x * kHalf; r < min(d.rows, (x + 1) * kHalf); r += 16, ad += 2, bd += 16 * 128 >> 4) {
                  mma_ss(tmem, ad, bd, idesc, acc);
                  mma_ss(tmem + 256, ad, bd + (4 * (kSlot / 8) >> 4), idesc, acc);
                  acc = 1;
                }
                mma_commit(&bars.empty[x]);
              }
              if (!ok) break;
              mma_commit(&bars.pcons[ps]);
              mma_commit(&bars.odone[ps]);
              ++tc;
            }
            if (d.last) break;
          }
        }
        mma_commit(&bars.mdrain);
        mbar_drain(&bars.mdrain, 0);
      }
    } else if (warp == kAuxWarp && rank == 0) {
      // ------------------------------------------------------- q loads (CTA 0)
      if (elect_one()) {
        griddep_wait();  // the previous kernel may have written q
        uint32_t uses = 0;
        int q_slots = 0, rope_loads = 0;
        bool ok = true;
#pragma unroll 1
        for (int item = cluster, n = 0; item < P.items && ok; item += clusters, ++n) {
          const int th = item / P.n_chunks, hb = th % P.head_blocks, t = th / P.head_blocks;
          // not before the previous item's last slot is converted: a wait for a slot is
          // by parity, and good for its next use only
          if (n > 0) ok = WAIT1(bars.cdone, (n - 1) & 1);
          q_slots = 0;
#pragma unroll 1
          for (int k = 0; k < 2 && ok; ++k) {
            uint64_t* const full = &bars.full[k];
            if (!WAIT1(bars.empty[k], (uses & 1) ^ 1)) { ok = false; break; }
            mbar_arrive_expect_tx(full, kSlot);
            mbar_arrive_n(full, kConvWarps / 2 - 1);
#pragma unroll 1
            for (int a = 0; a < 4; ++a)
              tma_load_3d(smem + k * kSlot + a * kAtom, &tmap_q, k * 256 + a * 64, hb * 128, t, full);
            q_slots = k + 1;
          }
          if (ok && n > 0) ok = WAIT1(bars.qfree, (n - 1) & 1);
          if (!ok) break;
          mbar_arrive_expect_tx(&bars.qpfull, kAtom);
          tma_load_3d(smem + kOffQrope, &tmap_q, 512, hb * 128, t, &bars.qpfull);
          rope_loads = n + 1;
          ++uses;
          if (item + clusters < P.items) {  // the next item's q, for when its turn comes
            const int next = (item + clusters) / P.n_chunks;
#pragma unroll 1
            for (int k = 0; k < kDqk; k += 64)
              tma_prefetch_3d(&tmap_q, k, next % P.head_blocks * 128, next / P.head_blocks);
          }
#pragma unroll 1
          while (ok) {
            Desc d;
            if (!next_desc1(d)) { ok = false; break; }
            if (d.rows > 0) ++uses;
            if (d.last) break;
          }
        }
        if (*tries == 0) {  // the copies in flight land before the CTA's memory is given up
          for (int k = 0; k < q_slots; ++k) {
            drain_copy(&bars.full[k], 0);
            drain_copy(&bars.full[k], 1);
          }
          if (rope_loads > 0) mbar_drain(&bars.qpfull, (rope_loads - 1) & 1);
        }
      }
    } else if (warp == kAux2Warp && rank == 0) {
      // ------------------------------------------------ rotary K loads (CTA 0)
      // 16-byte asynchronous copies, 8 a row, four rows an instruction, swizzled
      const uint8_t* const rope_src = P.kv4 + kKv4Rope + (lane & 7) * 16;
      uint32_t tc = 0;
      bool ok = true;
#pragma unroll 1
      for (int item = cluster; item < P.items && ok; item += clusters) {
#pragma unroll 1
        while (ok) {
          Desc d;
          if (!WAIT(bars.dfull[dc % kDescs], (dc / kDescs) & 1)) { ok = false; break; }
          const int* rows = descs[dc % kDescs].row + (lane >> 3);
          read_desc(d);
          if (d.rows > 0) {
            const uint32_t rs = tc & 1;
            if (!WAIT(bars.kpempty[rs], ((tc >> 1) & 1) ^ 1)) { ok = false; break; }
            const uint32_t kp = smem_u32(smem + kOffKrope) + rs * kAtom;
#pragma unroll 1
            for (int x0 = 0; x0 < d.rows; x0 += 16, rows += 16) {
#pragma unroll
              for (int x = 0; x < 16; x += 4) {
                const int r = rows[x];  // (a copy of 0 bytes writes zeros)
                cp_async16(kp + x0 * 128 + sw128_off(x + (lane >> 3), lane & 7),
                           rope_src + static_cast<size_t>(max(r, 0)) * kKv4Row, r < 0 ? 0 : 16);
              }
            }
            cp_async_mbar_arrive(&bars.kpfull[rs]);
            ++tc;
          }
          __syncwarp();
          if (lane == 0) free_desc();
          if (d.last) break;
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");  // nothing in flight when the CTA ends
    } else {
      // CTA 1: P slot consumed -> CTA 0 (the slot is free); P arrived -> CTA 0 (its
      // staging is free)
      if (elect_one()) {
        const bool arrived = warp == kAux2Warp;
        const uint32_t remote = mapa(smem_u32(arrived ? &bars.psent[0][0] : &bars.pfree[0]), 0);
        uint32_t tc = 0;
        uint32_t filled = 0;  // items that select something
        bool ok = true;
#pragma unroll 1
        for (int item = cluster; item < P.items && ok; item += clusters) {
#pragma unroll 1
          while (ok) {
            Desc d;
            if (!next_desc1(d)) { ok = false; break; }
            if (d.rows > 0) {
              const uint32_t ps = tc & 1, ph = (tc >> 1) & 1;
              if (arrived) {
#pragma unroll 1
                for (int a = 0; a < 2; ++a) {
                  if (!WAIT1_CLUSTER(bars.pfull[ps][a], ph)) { ok = false; break; }
                  mbar_arrive_remote(remote + (ps * 2 + a) * 8);
                }
              } else {
                if (!WAIT1(bars.pcons[ps], ph)) { ok = false; break; }
                // (the item's output is staged in its last tile's slot)
                if (d.last && !WAIT1(bars.stored, filled++ & 1)) { ok = false; break; }
                mbar_arrive_expect_tx(&bars.pfull[ps][0], kPBytes0);  // arm the slot's next use
                mbar_arrive_expect_tx(&bars.pfull[ps][1], kPBytes1);
                mbar_arrive_remote(remote + ps * 8);
              }
              ++tc;
            }
            if (d.last) break;
          }
        }
      }
    }
  }
  tc_fence_before();
  if (tid == 0 && *tries == 0) {  // copies to the peer may be in flight: far more time than they take
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 100000) {}
  }
  __syncthreads();
  cluster_sync();  // no CTA leaves while its peer may still address it
  if (tid == 0 && *tries == 0) atomicOr(P.err, kErrTimeout);
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// Merges a token's chunks: out = sum_c w_c O_c / (sum_c w_c l_c [+ 2^(sink - M)]) with
// w_c = 2^(m_c - M).  A block takes 32 heads (a lane each) and 16 kCols columns, so
// reads are runs of 512 bytes; its warps share the chunks' maxima and sums through
// shared memory, and the result goes through it to be written in longer runs.  A thread
// has the loads of kBatch chunks of 4 kCols columns in flight, the first of them before
// the maxima arrive.  (The part of a chunk that selects nothing, which nobody wrote, is
// loaded like the others and left out.)  All chunks in one batch and 32 floats a thread
// where there are few chunks, batches of eight and one column group where there are many;
// one call of 128 heads over 2048 rows, us with <2, 4>, <4, 2> and <8, 1>:
//    2 chunks (38 tokens)  38.5  39.5  42.3     9 (8)   26.4  24.2  23.2
//    3        (25)         32.7  32.7  34.2    16 (4)   25.5  24.9  22.4
//    4        (19)         29.4  28.3  29.7    32 (1)   28.3  21.5  19.4
constexpr int kMergeWarps = 4;

template <int kBatch, int kCols>
__global__ void __launch_bounds__(kMergeWarps * 32) attn_kv4_merge_kernel(const AttnKv4Params P) {
  extern __shared__ float2 s_ml[];  // [n_chunks][32]
  __shared__ uint2 s_out[32][kMergeWarps * kCols + 1];
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h0 = blockIdx.y * 32, h = min(h0 + lane, P.H - 1), t = blockIdx.z;
  const int c4 = (blockIdx.x * kMergeWarps + warp) * kCols;
  const float4* src = P.part_o + (static_cast<size_t>(t) * P.n_chunks * (kDv / 4) + c4) * P.H + h;
  float4 o[kBatch][kCols];
  auto load = [&](int c0) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (c0 + i < P.n_chunks)
#pragma unroll
        for (int k = 0; k < kCols; ++k) o[i][k] = __ldcg(src + (static_cast<size_t>(c0 + i) * (kDv / 4) + k) * P.H);
  };
  load(0);
  const float2* ml = P.part_ml + static_cast<size_t>(t) * P.n_chunks * P.H + h;
  for (int c = warp; c < P.n_chunks; c += kMergeWarps) s_ml[c * 32 + lane] = __ldcg(ml + static_cast<size_t>(c) * P.H);
  __syncthreads();
  float M = neg_inf();
#pragma unroll 4
  for (int c = 0; c < P.n_chunks; ++c) M = fmaxf(M, s_ml[c * 32 + lane].x);
  const float Mz = M == neg_inf() ? 0.f : M;  // (nothing selected: every weight is 0)
  float wsum = 0.f;
  float4 acc[kCols];
#pragma unroll
  for (int k = 0; k < kCols; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c0 = 0; c0 < P.n_chunks; c0 += kBatch) {
    if (c0 > 0) load(c0);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const float2 c = c0 + i < P.n_chunks ? s_ml[(c0 + i) * 32 + lane] : make_float2(neg_inf(), 0.f);
      const float w = exp2f(c.x - Mz);
      wsum = fmaf(w, c.y, wsum);  // (a sum that is not a number stays one)
      if (w != 0.f) {  // (an empty chunk has no O)
#pragma unroll
        for (int k = 0; k < kCols; ++k) {
          acc[k].x = fmaf(w, o[i][k].x, acc[k].x);
          acc[k].y = fmaf(w, o[i][k].y, acc[k].y);
          acc[k].z = fmaf(w, o[i][k].z, acc[k].z);
          acc[k].w = fmaf(w, o[i][k].w, acc[k].w);
        }
      }
    }
  }
  float scale = 1.f;
  if (P.sink != nullptr) {
    // one more term 2^s2 in the denominator (a zero-value key); -inf: none
    const float s2 = __ldg(P.sink + h) * 1.4426950408889634f;
    const float mx = fmaxf(M, s2);
    if (mx != neg_inf()) {
      scale = exp2f(M - mx);
      wsum = wsum * scale + exp2f(s2 - mx);
      M = mx;
    }
  }
  scale = wsum == 0.f ? 0.f : scale / wsum;
  if (blockIdx.x == 0 && warp == 0 && h0 + lane < P.H && P.lse != nullptr)
    P.lse[static_cast<size_t>(t) * P.H + h] = wsum == 0.f ? neg_inf() : (M + log2f(wsum)) * 0.69314718055994531f;
#pragma unroll
  for (int k = 0; k < kCols; ++k) {
    const __nv_bfloat162 b0 = __floats2bfloat162_rn(acc[k].x * scale, acc[k].y * scale);
    const __nv_bfloat162 b1 = __floats2bfloat162_rn(acc[k].z * scale, acc[k].w * scale);
    s_out[lane][warp * kCols + k] =
        make_uint2(*reinterpret_cast<const uint32_t*>(&b0), *reinterpret_cast<const uint32_t*>(&b1));
  }
  __syncthreads();
  uint2* out = reinterpret_cast<uint2*>(P.out) + (static_cast<size_t>(t) * P.H + h0) * (kDv / 4) + blockIdx.x * kMergeWarps * kCols;
#pragma unroll
  for (int k = 0; k < kCols; ++k) {
    const int i = k * kMergeWarps * 32 + threadIdx.x, head = i / (kMergeWarps * kCols), x = i % (kMergeWarps * kCols);
    if (h0 + head < P.H) out[static_cast<size_t>(head) * (kDv / 4) + x] = s_out[head][x];
  }
}

template <int kBatch, int kCols>
cudaError_t launch_merge(const AttnKv4Params& P, cudaLaunchConfig_t& cfg) {
  cfg.gridDim = dim3(kDv / 4 / (kMergeWarps * kCols), (P.H + 31) / 32, P.T);
  cfg.blockDim = dim3(kMergeWarps * 32);
  cfg.dynamicSmemBytes = static_cast<size_t>(P.n_chunks) * 32 * sizeof(float2);
  return cudaLaunchKernelEx(&cfg, attn_kv4_merge_kernel<kBatch, kCols>, P);
}

// Chunks per token: as many as the GPU holds clusters for at once, each a multiple of a
// slot's 64 rows.  (Blocks of 64 heads in twice the clusters, where there are enough:
// one token 23.6 us for 21.2, as every row is then converted twice.)
// Whole chunks per token leave clusters idle just past a count that fills them: 128 heads
// over 2048 rows take 38.5 us for 38 tokens (two chunks each, every cluster), 50.6 for 39
// (one each, half of the clusters), 54.1 for 76, 93.0 for 77 (a second round), 102.5 for 152.
void plan(const dsa_attn_kv4_args& a, int& head_blocks, int& n_chunks, int& chunk_rows) {
  head_blocks = (a.H + 127) / 128;
  const long long pairs = static_cast<long long>(a.T) * head_blocks;
  const int target = static_cast<int>(std::max<long long>(1, sm_count() / (2 * pairs)));
  chunk_rows = ((a.topk + target - 1) / target + kHalf - 1) / kHalf * kHalf;
  n_chunks = (a.topk + chunk_rows - 1) / chunk_rows;
}

}  // namespace

size_t attn_kv4_workspace(const dsa_attn_kv4_args& a) {
  int hb, nc, cr;
  plan(a, hb, nc, cr);
  if (nc == 1) return 0;
  const size_t heads = static_cast<size_t>(a.T) * nc * a.H;
  return round_up(heads * kDv * 4, 256) + round_up(heads * sizeof(float2), 256);
}

int launch_attn_kv4(const dsa_attn_kv4_args& a, void* ws, cudaStream_t s) {
  AttnKv4Params P{};
  plan(a, P.head_blocks, P.n_chunks, P.chunk_rows);
  P.T = a.T; P.B = a.B; P.n_q = a.n_q; P.H = a.H; P.topk = a.topk; P.max_L = a.max_L;
  P.items = a.T * P.head_blocks * P.n_chunks;
  P.scale_log2 = a.scale * 1.4426950408889634f;
  P.kv4 = a.kv4; P.rows = a.cache_rows;
  P.block_table = a.block_table; P.block_size = a.block_table ? a.block_size : a.max_L; P.max_blocks = a.max_blocks;
  // With 2^k >= block_size > 2^(k-1) and m = ceil(2^(31+k) / block_size), i m / 2^(31+k) exceeds
  // i / block_size by less than i / 2^(31+k) <= 1 / block_size: the quotients are equal.
  P.page_shift = 0;
  while ((1u << P.page_shift) < static_cast<uint32_t>(P.block_size)) ++P.page_shift;
  P.page_shift += 31;
  P.page_mul = static_cast<uint32_t>(((uint64_t{1} << P.page_shift) + P.block_size - 1) / P.block_size);
  P.idx = a.topk_idx; P.out = a.out; P.lse = a.lse; P.sink = a.sink; P.seq = a.seq_of_token;
  if (P.seq != nullptr) P.n_q = 1;  // ignored with a map
  if (P.n_chunks > 1) {
    P.part_o = static_cast<float4*>(ws);
    P.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) +
                                          round_up(static_cast<size_t>(a.T) * P.n_chunks * a.H * kDv * 4, 256));
  }
  P.err = error_word();
  if (!P.err) return DSA_ERR_CUDA;

  // q [T, H, 576] in 64-dim x 128-head boxes (heads past H read as zeros); the
  // output [T, H, 512] in 64-column x 128-head boxes (heads past H are clipped)
  alignas(64) CUtensorMap tmap_q, tmap_o;
  {
    const uint64_t H = static_cast<uint64_t>(a.H), T = static_cast<uint64_t>(a.T);
    const uint64_t dq[3] = {kDqk, H, T}, sq[2] = {kDqk * 2, H * kDqk * 2};
    const uint64_t od[3] = {kDv, H, T}, os[2] = {kDv * 2, H * kDv * 2};
    const uint32_t box[3] = {64, 128, 1};
    if (!encode_tmap(&tmap_q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.q, dq, sq, box, 128) ||
        !encode_tmap(&tmap_o, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, P.out, od, os, box, 128))
      return DSA_ERR_CUDA;
  }
  cudaError_t e = cudaFuncSetAttribute(attn_kv4_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return DSA_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(2 * std::min(P.items, std::max(1, sm_count() / 2)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, attn_kv4_kernel, P, tmap_q, tmap_o);
  if (e != cudaSuccess) return DSA_ERR_CUDA;
  if (P.n_chunks > 1) {
    cudaLaunchConfig_t c2 = {};
    c2.stream = s;
    c2.attrs = attr;
    c2.numAttrs = 1;
    e = P.n_chunks <= 2 ? launch_merge<2, 4>(P, c2) : P.n_chunks <= 4 ? launch_merge<4, 2>(P, c2) : launch_merge<8, 1>(P, c2);
  }
  return cuda_status(e);
}

}  // namespace dsa
