// Attention of each sequence's newest tokens over its whole latent cache
// (dsa_latent_attn), on tcgen05.  [V4-TileLang §Sparse Flash Attention] steps
// 3-8 with every visible row in place of a selection.
//
// The (token, head) rows of a sequence lie behind one another in q and out: they
// are cut into blocks of 128 rows, whatever H is.  The work is the list of
// (block, tile of 64 cache rows), block by block; persistent clusters of two
// CTAs take an equal stretch of it each, so that sequences of any lengths load
// all SMs evenly.  A block that lies in one stretch is finished there; the parts
// of one that several clusters share are merged by latent_merge_kernel.
//
//   CTA 0  q [128 x 576] in tensor memory, K tiles in shared memory (TMA, one
//          64-dim atom a box, a ring of 9 slots of 3 atoms), S = q . K^T in three
//          buffers.  Two softmax warpgroups take the tiles in turn: the running
//          maximum passes between them as soon as a tile's is known, so one's
//          exponentials overlap the other's loads; P (bf16) goes straight into
//          CTA 1's shared memory with st.async, with the factor by which the
//          maximum's growth scales what is there.
//   CTA 1  O [128 x 512] fp32 fills its tensor memory; V tiles (the first 512 dims
//          of the same rows, from L2) in a ring of 6 slots of 4 atoms; O += P . V.
//          Eight warps rescale O where a maximum grew by more than 2^8, and at a
//          block's end write it.
//
// Rows that no token of a block sees (the end of the last tile: they may hold
// anything) are cleared in V before the product; their S is not looked at.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include "dsa_internal.h"
#include "dsa_ptx.cuh"

namespace dsa {
namespace {

constexpr int kDqk = 576, kDv = 512;
constexpr int kRows = 64;                  // cache rows of a tile
constexpr int kAtomBytes = kRows * 128;    // 64 rows x 64 dims
constexpr int kAtomsK = kDqk / 64, kAtomsV = kDv / 64;
constexpr int kKAtoms = 3, kKSlots = 9, kKParts = kAtomsK / kKAtoms;  // atoms of a slot, slots, slots of a tile
constexpr int kVAtoms = 4, kVSlots = 6, kVParts = kAtomsV / kVAtoms;
constexpr int kSBufs = 3;
constexpr int kPBytesSlot = 128 * kRows * 2;
constexpr uint32_t kPTx = kPBytesSlot + 128 * 4;  // P and the rescale factors of a tile
constexpr uint32_t kTmemS = 288;                  // CTA 0: q in columns [0, 288), then the S buffers
static_assert(kTmemS + kSBufs * kRows <= 512, "tensor memory of CTA 0");
constexpr int kThreads = 384;  // 8 softmax / output warps, a loader, an MMA issuer, a relay, one idle
constexpr int kLoadWarp = 8, kMmaWarp = 9, kRelayWarp = 10;
// A cluster takes at least this many tiles: splitting further costs more in the
// merge than it saves.
constexpr int kMinTiles = 4;

struct LatentParams {
  int T, B, n_q, H, max_L;
  float scale_log2;
  const __nv_bfloat16* q;
  int64_t cache_rows;
  const int32_t* block_table;
  int block_size, max_blocks;
  int box_rows;  // rows of a TMA box: 64, or a smaller page
  const int32_t* cu;
  const int32_t* kv_len;
  __nv_bfloat16* out;
  float* lse;
  const float* sink;
  int clusters;
  float* part_o;    // [2 clusters][128][512]: a cluster's first and last part
  float2* part_ml;  // [2 clusters][128]: (maximum, sum) in log2 units
  int4* desc;       // [clusters]: first row, rows, parts of the block that begins at the end of a stretch
  uint32_t* err;
};

struct __align__(8) Bars {
  uint64_t kfull[kKSlots], kempty[kKSlots];
  uint64_t sfull[kSBufs], sempty[kSBufs];
  uint64_t pfree[2];              // CTA 0: a P slot of CTA 1 is free
  uint64_t mready[2][4];          // the maximum after a group's tile, per warp
  uint64_t qfull;                 // a block's q is in tensor memory
  uint64_t ffree;                 // CTA 0: CTA 1 has read the final (m, l)
  uint64_t vfull[kVSlots], vempty[kVSlots];
  uint64_t pfull[2], pcons[2];    // CTA 1: P slots
  uint64_t oready[2];             // O is scaled for the tile
  uint64_t odone[2];              // a tile's product is in O (even and odd tiles: a warp may look a tile late)
  uint64_t ffull;                 // CTA 1: the final (m, l) lie in CTA 0
  uint64_t drain;                 // the MMA thread's last commit
};

// Shared memory: the ring (CTA 0: K, then OwnA; CTA 1: V, then two P slots), then
// what both CTAs have.
constexpr int kRingBytes = kVSlots * kVAtoms * kAtomBytes + 2 * kPBytesSlot;
struct OwnA {
  float m[2][128];          // running maximum after a softmax group's latest tile
  float2 final_ml[2][128];  // (maximum, sum) of each group at a block's end
};
constexpr int kOwnA = kKSlots * kKAtoms * kAtomBytes;
static_assert(kOwnA + sizeof(OwnA) <= kRingBytes, "ring of CTA 0");
struct __align__(16) Shared {
  float alpha[2][128];  // CTA 1
  Bars bars;
  long long scan[kThreads / 32];
  long long start_off;
  int start_b;
  uint32_t tmem;
  int abort_flag;
};
constexpr size_t kSmemBytes = 1024 + kRingBytes + sizeof(Shared);  // 1024: to align the ring
static_assert(kSmemBytes <= 232448, "shared memory of a CTA");

struct Piece {
  int row0, rows;  // of q and out
  int b, len, first_vis;  // sequence, its rows, rows that the block's first row's token sees
  int in_tok;      // rows of the first token of the sequence before the block: block * 128
  int vis;         // rows that the block's last token sees
  int t0, t1;      // tiles
  bool begins, ends;
};

struct Walker {
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
    nt = max(1, (len + kRows - 1) / kRows);
    nb = (n * P.H + 127) / 128;
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
    if (left <= 0) return false;
    while (blk >= nb) {
      if (++b >= P.B) return false;
      blk = 0;
      load(P);
    }
    p.b = b;
    p.len = len;
    p.row0 = c0 * P.H + blk * 128;
    p.rows = min(128, n * P.H - blk * 128);
    p.in_tok = blk * 128;
    p.first_vis = len - n + 1;
    p.vis = max(0, p.first_vis + (blk * 128 + p.rows - 1) / P.H);
    const int stop = static_cast<int>(min(static_cast<long long>(nt), off + left));
    p.t0 = off;
    p.t1 = max(off, min(stop, (p.vis + kRows - 1) / kRows));
    p.begins = off == 0;
    p.ends = stop == nt;
    left -= stop - off;
    off = stop;
    if (off == nt) {
      off = 0;
      ++blk;
    }
    return true;
  }
};

// Row of the cache at which rows s .. s + box_rows of a sequence lie; cache_rows
// (past the map: read as zeros) where there are none.
__device__ __forceinline__ int box_row(const LatentParams& P, const Piece& p, int s, bool report) {
  if (P.block_table == nullptr) return p.b * P.max_L + s;  // below cache_rows, so it fits
  const int none = static_cast<int>(P.cache_rows);
  if (s >= p.len) return none;
  const int page = __ldg(P.block_table + static_cast<size_t>(p.b) * P.max_blocks + s / P.block_size);
  if (page < 0 || (static_cast<int64_t>(page) + 1) * P.block_size > P.cache_rows) {
    if (report) atomicOr(P.err, kErrBadIndex);
    return none;
  }
  return page * P.block_size + s % P.block_size;
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

__device__ __forceinline__ float2 ld_cluster_f32x2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_global_v8(float* p, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

__global__ void __launch_bounds__(kThreads, 1)
    latent_attn_kernel(const __grid_constant__ LatentParams P, const __grid_constant__ CUtensorMap kv_map) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* ring = smem_raw + (1024u - (smem_u32(smem_raw) & 1023u)) % 1024u;
  Shared& sh = *reinterpret_cast<Shared*>(ring + kRingBytes);
  OwnA& own = *reinterpret_cast<OwnA*>(ring + kOwnA);
  Bars& bars = sh.bars;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const int cluster = blockIdx.x >> 1;
  uint8_t* sP = ring + kVSlots * kVAtoms * kAtomBytes;  // CTA 1
  volatile int* abort_v = &sh.abort_flag;

  if (tid == 0) {
    for (int i = 0; i < kKSlots; ++i) { mbar_init(&bars.kfull[i], 1); mbar_init(&bars.kempty[i], 1); }
    for (int i = 0; i < kSBufs; ++i) { mbar_init(&bars.sfull[i], 1); mbar_init(&bars.sempty[i], 4); }
    for (int i = 0; i < kVSlots; ++i) { mbar_init(&bars.vfull[i], 1); mbar_init(&bars.vempty[i], 1); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.pfree[i], 1);
      mbar_init(&bars.pfull[i], 1);
      mbar_init(&bars.pcons[i], 1);
      mbar_init(&bars.oready[i], 8);
      mbar_init(&bars.odone[i], 1);
      for (int w = 0; w < 4; ++w) mbar_init(&bars.mready[i][w], 1);
    }
    mbar_init(&bars.qfull, 8);
    mbar_init(&bars.ffree, 8);
    mbar_init(&bars.ffull, 8);
    mbar_init(&bars.drain, 1);
    sh.abort_flag = 0;
    fence_mbar_init();
    if (rank == 1) {
      mbar_arrive_expect_tx(&bars.pfull[0], kPTx);
      mbar_arrive_expect_tx(&bars.pfull[1], kPTx);
    }
  }
  if (warp == 0) tmem_alloc(&sh.tmem, 512);
  griddep_wait();

  // ------------------------------------------------ this cluster's stretch
  const int each = (P.B + kThreads - 1) / kThreads;
  const int b0 = min(P.B, tid * each), b1 = min(P.B, b0 + each);
  long long mine = 0;
  bool bad = false;
  Walker w;
  for (w.b = b0; w.b < b1; ++w.b) {
    w.load(P);
    mine += static_cast<long long>(w.nb) * w.nt;
    if (P.cu != nullptr) {
      const int c0 = __ldg(P.cu + w.b), c1 = __ldg(P.cu + w.b + 1);
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
  __syncthreads();
  tc_fence_after();
  long long before = inc - mine, total = 0;
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) before += sh.scan[i];
    total += sh.scan[i];
  }
  const long long active = max(1ll, min(static_cast<long long>(P.clusters), total / kMinTiles));
  const long long lo = cluster < active ? total * cluster / active : total;
  const long long hi = cluster < active ? total * (cluster + 1) / active : total;
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
  cluster_sync();  // the stretch is known; both CTAs' barriers are initialised before any remote use
  w.start(P, sh.start_b, sh.start_off, hi - lo);
  Piece p;

  if (warp < 8 && rank == 0) {
    // ------------------------------------------------------- softmax (CTA 0)
    const int g = warp >> 2, wq = warp & 3;
    const int row = wq * 32 + lane;
    const float ninf = -__int_as_float(0x7f800000);
    const uint32_t remote_p = mapa(smem_u32(sP + g * kPBytesSlot), 1);
    const uint32_t remote_alpha = mapa(smem_u32(&sh.alpha[g][row]), 1);
    const uint32_t remote_pfull = mapa(smem_u32(&bars.pfull[g]), 1);
    const uint32_t remote_ffull = mapa(smem_u32(&bars.ffull), 1);
    int G = 0, pieces = 0;  // tiles and blocks so far
    bool ok = true;
    while (ok && w.next(P, p)) {
      const int nt = p.t1 - p.t0;
      if (nt > 0) {
        // q: this thread's row, atoms [5g, 5 + 4g): global -> tensor memory
        const uint4* qrow = reinterpret_cast<const uint4*>(P.q + static_cast<size_t>(p.row0 + row) * kDqk);
        const bool real = row < p.rows;
#pragma unroll 1
        for (int a = 5 * g; a < 5 + 4 * g; ++a) {
          uint32_t r[32];
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const uint4 v = real ? __ldg(qrow + a * 8 + c) : make_uint4(0, 0, 0, 0);
            r[4 * c] = v.x; r[4 * c + 1] = v.y; r[4 * c + 2] = v.z; r[4 * c + 3] = v.w;
          }
          tmem_st32(tmem + lane_off + a * 32, r);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.qfull);
      }
      const int vis = p.first_vis + (p.in_tok + row) / P.H;  // rows that this row's token sees
      float m_used = ninf, l_sum = 0.f;
      for (int j = 0; j < nt; ++j, ++G) {
        const int sb = G % kSBufs;
        const uint32_t sph = (G / kSBufs) & 1;
        if ((G & 1) != g) {
          // the other group's tile; the block's last one also says that q is read
          if (j + 1 == nt) {
            if (!warp_wait<false>(&bars.sfull[sb], sph, P.err, abort_v)) { ok = false; break; }
          }
          continue;
        }
        if (!warp_wait<false>(&bars.sfull[sb], sph, P.err, abort_v)) { ok = false; break; }
        tc_fence_after();
        float x[kRows];
        {
          uint32_t s0[32], s1[32];
          tmem_ld32(tmem + lane_off + kTmemS + sb * kRows, s0);
          tmem_ld32(tmem + lane_off + kTmemS + sb * kRows + 32, s1);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            x[k] = __uint_as_float(s0[k]);
            x[32 + k] = __uint_as_float(s1[k]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.sempty[sb]);
        const int lim = vis - (p.t0 + j) * kRows;  // columns that this row sees
        if (!__all_sync(0xffffffffu, lim >= kRows)) {
#pragma unroll
          for (int k = 0; k < kRows; ++k)
            if (k >= lim) x[k] = ninf;
        }
        float mt = ninf;
#pragma unroll
        for (int k = 0; k < kRows; ++k) mt = fmaxf(mt, x[k]);
        mt *= P.scale_log2;
        float m_prev = ninf;
        if (j > 0) {
          if (!warp_wait<false>(&bars.mready[g ^ 1][wq], ((G - 1) >> 1) & 1, P.err, abort_v)) { ok = false; break; }
          m_prev = own.m[g ^ 1][row];
        }
        float alpha = 1.f, m_now = m_prev;
        if (mt > m_prev + 8.f) {  // also taken when m_prev is -inf
          m_now = mt;
          alpha = ex2_approx(m_prev - mt);
        }
        own.m[g][row] = m_now;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.mready[g][wq]);
        if (m_now != m_used) {
          l_sum *= ex2_approx(m_used - m_now);  // (0 at the first)
          m_used = m_now;
        }
        uint32_t pk[32];
        float lt = 0.f;
        const float shift = m_now == ninf ? 0.f : m_now;
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          const float p0 = ex2_approx(fmaf(x[2 * k], P.scale_log2, -shift));
          const float p1 = ex2_approx(fmaf(x[2 * k + 1], P.scale_log2, -shift));
          lt += p0 + p1;
          const __nv_bfloat162 pb = __floats2bfloat162_rn(p0, p1);
          pk[k] = *reinterpret_cast<const uint32_t*>(&pb);
        }
        l_sum += lt;
        if (!warp_wait<true>(&bars.pfree[g], ((G >> 1) & 1) ^ 1, P.err, abort_v)) { ok = false; break; }
#pragma unroll
        for (int c = 0; c < 8; ++c)
          st_async_v4(remote_p + sw128_off(row, c), make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]),
                      remote_pfull);
        st_async_b32(remote_alpha, __float_as_uint(alpha), remote_pfull);
      }
      if (!ok) break;
      if (!warp_wait<true>(&bars.ffree, (pieces & 1) ^ 1, P.err, abort_v)) { ok = false; break; }
      own.final_ml[g][row] = make_float2(m_used, l_sum);
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(remote_ffull);
      ++pieces;
    }
    if (!ok) __nanosleep(100000);  // stores on their way to CTA 1 land before either CTA leaves
  } else if (warp < 8) {
    // ----------------------------------------- O: scaling and output (CTA 1)
    const int half = warp >> 2, row = (warp & 3) * 32 + lane;
    const float ninf = -__int_as_float(0x7f800000);
    const uint32_t remote_final = mapa(smem_u32(&own.final_ml[0][0]), 0);
    const uint32_t remote_ffree = mapa(smem_u32(&bars.ffree), 0);
    int G = 0, pieces = 0, done = 0;  // tiles, blocks, products seen complete
    bool ok = true;
    int tail_row0 = 0, tail_rows = 0, tail_parts = 0;  // the block that this stretch ends inside of
    long long at = lo;
    while (ok && w.next(P, p)) {
      const int nt = p.t1 - p.t0;
      for (int j = 0; j < nt; ++j, ++G) {
        const int ps = G & 1;
        if (!warp_wait<true>(&bars.pfull[ps], (G >> 1) & 1, P.err, abort_v)) { ok = false; break; }
        const float alpha = sh.alpha[ps][row];
        if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
          while (ok && done < G) {  // O holds the products before this tile
            ok = warp_wait<false>(&bars.odone[done & 1], (done >> 1) & 1, P.err, abort_v);
            done += ok;
          }
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
        const int live = p.vis - (p.t0 + j) * kRows;  // rows of the tile that the block sees
        if (live < kRows) {
          const int pair = G % (kVSlots / kVParts);
          const uint32_t vph = (G / (kVSlots / kVParts)) & 1;
          for (int i = 0; ok && i < kVParts; ++i)
            ok = warp_wait<false>(&bars.vfull[pair * kVParts + i], vph, P.err, abort_v);
          if (!ok) break;
          uint8_t* v = ring + pair * kAtomsV * kAtomBytes;
          for (int i = tid; i < (kRows - live) * kAtomsV * 8; i += 256)
            *reinterpret_cast<uint4*>(v + ((i >> 3) % kAtomsV) * kAtomBytes + (live + i / (kAtomsV * 8)) * 128 +
                                      (i & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();  // P arrived through st.async, zeros by plain stores; the MMA reads both
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.oready[ps]);
        while (ok && done < G) {  // at most one product's completion stays unseen
          ok = warp_wait<false>(&bars.odone[done & 1], (done >> 1) & 1, P.err, abort_v);
          done += ok;
        }
        if (!ok) break;
      }
      while (ok && done < G) {
        ok = warp_wait<false>(&bars.odone[done & 1], (done >> 1) & 1, P.err, abort_v);
        done += ok;
      }
      if (ok) ok = warp_wait<true>(&bars.ffull, pieces & 1, P.err, abort_v);
      if (!ok) break;
      tc_fence_after();
      const float2 f0 = ld_cluster_f32x2(remote_final + row * 8);
      const float2 f1 = ld_cluster_f32x2(remote_final + (128 + row) * 8);
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(remote_ffree);
      ++pieces;
      float m = fmaxf(f0.x, f1.x);
      // (a sum of 0 says that nothing was seen; one that is not a number stays so)
      float l = (f0.y == 0.f ? 0.f : f0.y * ex2_approx(f0.x - m)) + (f1.y == 0.f ? 0.f : f1.y * ex2_approx(f1.x - m));
      const bool empty = l == 0.f || nt == 0;
      const bool whole = p.begins && p.ends;
      const size_t orow = static_cast<size_t>(p.row0) + row;
      if (whole) {
        float factor = empty ? 0.f : 1.f / l, lse2 = empty ? ninf : m + log2f(l);
        if (P.sink != nullptr) {
          // the sink adds 2^s2 to the denominator, taken relative to max(m, s2)
          const float s2 = __ldg(P.sink + (p.in_tok + row) % P.H) * 1.4426950408889634f;
          if (empty) {
            lse2 = s2;
          } else {
            const float mx = fmaxf(m, s2), den = l * exp2f(m - mx) + exp2f(s2 - mx);
            factor = exp2f(m - mx) / den;
            lse2 = mx + log2f(den);
          }
        }
        if (row < p.rows && half == 0 && P.lse != nullptr) P.lse[orow] = lse2 * 0.69314718055994531f;
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
          if (row < p.rows) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              *reinterpret_cast<uint4*>(o + c0 + 8 * k) = make_uint4(pk[4 * k], pk[4 * k + 1], pk[4 * k + 2], pk[4 * k + 3]);
          }
        }
      } else {
        const int slot = 2 * cluster + (p.begins ? 1 : 0);
        if (half == 0) P.part_ml[static_cast<size_t>(slot) * 128 + row] = make_float2(empty ? ninf : m, empty ? 0.f : l);
        float* o = P.part_o + (static_cast<size_t>(slot) * 128 + row) * kDv;
        if (__any_sync(0xffffffffu, !empty)) {
#pragma unroll 1
          for (int c0 = half * 256; c0 < half * 256 + 256; c0 += 32) {
            uint32_t v[32];
            tmem_ld32(tmem + lane_off + c0, v);
            tmem_ld_wait();
            if (row < p.rows && !empty) {
#pragma unroll
              for (int k = 0; k < 4; ++k) st_global_v8(o + c0 + 8 * k, v + 8 * k);
            }
          }
        }
        if (p.begins) {
          // the block ends in the stretch that holds its last tile
          long long e = at + w.nt;
          int parts = 1;
          while (total * (cluster + parts) / active < e) ++parts;
          tail_row0 = p.row0;
          tail_rows = p.rows;
          tail_parts = parts;
        }
      }
      tc_fence_before();
      at += (p.ends ? w.nt : w.off) - p.t0;
    }
    if (tid == 0) P.desc[cluster] = make_int4(tail_row0, tail_rows, tail_parts, 0);
  } else if (warp == kLoadWarp) {
    // ------------------------------------------------ K (CTA 0) or V (CTA 1)
    const int atoms = rank == 0 ? kKAtoms : kVAtoms, parts = rank == 0 ? kKParts : kVParts;
    const int slots = rank == 0 ? kKSlots : kVSlots;
    uint64_t* full = rank == 0 ? bars.kfull : bars.vfull;
    uint64_t* empty = rank == 0 ? bars.kempty : bars.vempty;
    const int boxes = kRows / P.box_rows;  // boxes of an atom: 1, or a page each
    int slot = 0, issued = 0;
    uint32_t ph = 0;
    bool ok = true;
    while (ok && w.next(P, p)) {
      int row = lane < boxes && p.t0 < p.t1 ? box_row(P, p, p.t0 * kRows + lane * P.box_rows, rank == 0) : 0;
      for (int t = p.t0; ok && t < p.t1; ++t) {
        const int here = row;
        if (t + 1 < p.t1 && lane < boxes) row = box_row(P, p, (t + 1) * kRows + lane * P.box_rows, rank == 0);
        for (int part = 0; part < parts; ++part) {
          if (lane == 0) {
            ok = mbar_wait_polling<false>(&empty[slot], ph ^ 1, P.err, abort_v);
            if (ok) mbar_arrive_expect_tx(&full[slot], atoms * kAtomBytes);
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
          if (lane < boxes) {
            uint8_t* dst = ring + slot * atoms * kAtomBytes + lane * P.box_rows * 128;
            for (int a = 0; a < atoms; ++a)
              tma_load_2d(dst + a * kAtomBytes, &kv_map, (part * atoms + a) * 64, here, &full[slot]);
          }
          __syncwarp();
          ++issued;
          if (++slot == slots) { slot = 0; ph ^= 1; }
        }
      }
    }
    if (!ok && lane == 0) {  // copies in flight land before the CTA leaves
      for (int i = max(0, issued - slots); i < issued; ++i) mbar_drain(&full[i % slots], (i / slots) & 1);
    }
  } else if (warp == kMmaWarp && lane == 0) {
    bool ok = true;
    int G = 0, slot = 0, pieces = 0;
    uint32_t ph = 0;
    if (rank == 0) {
      // ------------------------------------------------------ S = q . K^T
      const uint32_t idesc = idesc_f16(128, kRows, kFmtBF16, 0, 0);
      while (ok && w.next(P, p)) {
        if (p.t0 >= p.t1) continue;
        ok = mbar_wait_polling<false>(&bars.qfull, pieces & 1, P.err, abort_v);
        ++pieces;
        for (int t = p.t0; ok && t < p.t1; ++t, ++G) {
          const int sb = G % kSBufs;
          ok = mbar_wait_polling<false>(&bars.sempty[sb], ((G / kSBufs) & 1) ^ 1, P.err, abort_v);
          for (int part = 0; ok && part < kKParts; ++part) {
            ok = mbar_wait_polling<false>(&bars.kfull[slot], ph, P.err, abort_v);
            if (!ok) break;
            tc_fence_after();
            const uint32_t base = smem_u32(ring + slot * kKAtoms * kAtomBytes);
#pragma unroll
            for (int kk = 0; kk < kKAtoms * 4; ++kk) {
              const uint64_t bd = smem_desc(base + (kk / 4) * kAtomBytes + (kk % 4) * 32, 16, 1024, kSwizzle128B);
              mma_ts(tmem + kTmemS + sb * kRows, tmem + (part * kKAtoms * 4 + kk) * 8, bd, idesc,
                     part > 0 || kk > 0 ? 1u : 0u);
            }
            mma_commit(&bars.kempty[slot]);
            if (++slot == kKSlots) { slot = 0; ph ^= 1; }
          }
          if (ok) mma_commit(&bars.sfull[sb]);
        }
      }
    } else {
      // ------------------------------------------------------- O += P . V
      const uint32_t idesc = idesc_f16(128, 256, kFmtBF16, 0, 1);
      while (ok && w.next(P, p)) {
        for (int t = p.t0; ok && t < p.t1; ++t, ++G) {
          const int ps = G & 1;
          ok = mbar_wait_polling<false>(&bars.oready[ps], (G >> 1) & 1, P.err, abort_v);
          const uint32_t pbase = smem_u32(sP + ps * kPBytesSlot);
          for (int part = 0; ok && part < kVParts; ++part) {
            ok = mbar_wait_polling<false>(&bars.vfull[slot], ph, P.err, abort_v);
            if (!ok) break;
            fence_proxy_async_smem();
            tc_fence_after();
            const uint32_t vbase = smem_u32(ring + slot * kVAtoms * kAtomBytes);
#pragma unroll
            for (int kk = 0; kk < kRows / 16; ++kk) {
              const uint64_t ad = smem_desc(pbase + kk * 32, 16, 1024, kSwizzle128B);
              const uint64_t bd = smem_desc(vbase + kk * 16 * 128, kAtomBytes, 1024, kSwizzle128B);
              mma_ss(tmem + part * 256, ad, bd, idesc, t > p.t0 || kk > 0 ? 1u : 0u);
            }
            mma_commit(&bars.vempty[slot]);
            if (++slot == kVSlots) { slot = 0; ph ^= 1; }
          }
          if (ok) {
            mma_commit(&bars.pcons[ps]);
            mma_commit(&bars.odone[ps]);
          }
        }
      }
    }
    // every product issued has completed before the tensor memory is freed
    mma_commit(&bars.drain);
    mbar_drain(&bars.drain, 0);
  } else if (warp == kRelayWarp && lane == 0 && rank == 1) {
    // ------------------------------------- a P slot is consumed -> CTA 0
    const uint32_t remote_pfree[2] = {mapa(smem_u32(&bars.pfree[0]), 0), mapa(smem_u32(&bars.pfree[1]), 0)};
    bool ok = true;
    int G = 0;
    while (ok && w.next(P, p)) {
      for (int t = p.t0; ok && t < p.t1; ++t, ++G) {
        ok = mbar_wait_polling<false>(&bars.pcons[G & 1], (G >> 1) & 1, P.err, abort_v);
        if (!ok) break;
        mbar_arrive_expect_tx(&bars.pfull[G & 1], kPTx);  // for the slot's next use
        mbar_arrive_remote(remote_pfree[G & 1]);
      }
    }
  }
  griddep_launch_dependents();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no CTA leaves while its peer may still address it
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// Merges the parts of the block that cluster blockIdx.x's stretch ends inside of:
// out = sum_c 2^(m_c - M) O_c / (sum_c 2^(m_c - M) l_c [+ 2^(sink - M)]).  A warp
// takes half a row, 8 columns a lane; the loads of a batch of parts are issued
// before any is used.
constexpr int kMergeBatch = 4;

__global__ void __launch_bounds__(256) latent_merge_kernel(const __grid_constant__ LatentParams P) {
  griddep_wait();
  const int4 d = __ldcg(P.desc + blockIdx.x);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int item = blockIdx.y * 8 + warp, row = item >> 1, half = item & 1;
  if (d.z == 0 || row >= d.y) return;
  const int col = half * 256 + lane * 8;
  const float ninf = -__int_as_float(0x7f800000);
  float acc[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) acc[k] = 0.f;
  float M = ninf, sum = 0.f;
  for (int c0 = 0; c0 < d.z; c0 += kMergeBatch) {
    float2 ml[kMergeBatch];
    float4 v0[kMergeBatch], v1[kMergeBatch];
#pragma unroll
    for (int i = 0; i < kMergeBatch; ++i) {
      const int c = c0 + i;
      ml[i] = make_float2(ninf, 0.f);
      v0[i] = v1[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c < d.z) {
        const size_t at = static_cast<size_t>(c == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + c)) * 128 + row;
        ml[i] = __ldcg(P.part_ml + at);
        const float4* o = reinterpret_cast<const float4*>(P.part_o + at * kDv + col);
        v0[i] = __ldcg(o);
        v1[i] = __ldcg(o + 1);
      }
    }
    float Mb = M;
#pragma unroll
    for (int i = 0; i < kMergeBatch; ++i)
      if (ml[i].y != 0.f) Mb = fmaxf(Mb, ml[i].x);
    const float shift = Mb == ninf ? 0.f : Mb;
    const float r = exp2f(M - shift);
    sum *= r;
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] *= r;
    M = Mb;
#pragma unroll
    for (int i = 0; i < kMergeBatch; ++i) {
      if (ml[i].y == 0.f) continue;  // nothing seen: its O was not written
      const float wc = exp2f(ml[i].x - shift);
      sum = fmaf(wc, ml[i].y, sum);
      const float v[8] = {v0[i].x, v0[i].y, v0[i].z, v0[i].w, v1[i].x, v1[i].y, v1[i].z, v1[i].w};
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = fmaf(wc, v[k], acc[k]);
    }
  }
  const int orow = d.x + row;
  if (P.sink != nullptr) {
    const float s2 = __ldg(P.sink + orow % P.H) * 1.4426950408889634f;
    if (s2 != ninf) {
      if (sum != 0.f) {
        const float mx = fmaxf(M, s2), r = exp2f(M - mx);
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] *= r;
        sum = sum * r + exp2f(s2 - mx);
        M = mx;
      } else {
        M = s2;
        sum = 1.f;
      }
    }
  }
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
  uint32_t pk[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __nv_bfloat162 pb = __floats2bfloat162_rn(acc[2 * k] * inv, acc[2 * k + 1] * inv);
    pk[k] = *reinterpret_cast<const uint32_t*>(&pb);
  }
  *reinterpret_cast<uint4*>(P.out + static_cast<size_t>(orow) * kDv + col) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
  if (half == 0 && lane == 0 && P.lse != nullptr)
    P.lse[orow] = sum != 0.f ? (M + log2f(sum)) * 0.69314718055994531f : ninf;
}

// Clusters of a call: one for each pair of SMs, but no more than the most tiles
// that the shape allows can keep busy.
int cluster_count(const dsa_latent_attn_args& a) {
  const long long blocks = (static_cast<long long>(a.T) * a.H + 127) / 128 + a.B;
  const long long tiles = blocks * ((static_cast<long long>(a.max_L) + kRows - 1) / kRows);
  const long long most = sm_count() / 2, want = tiles / kMinTiles;
  return static_cast<int>(want < 1 ? 1 : want < most ? want : most);
}

}  // namespace

size_t latent_attn_workspace(const dsa_latent_attn_args& a) {
  const size_t n = cluster_count(a);
  return round_up(n * 2 * 128 * kDv * sizeof(float), 256) + round_up(n * 2 * 128 * sizeof(float2), 256) +
         round_up(n * sizeof(int4), 256);
}

int launch_latent_attn(const dsa_latent_attn_args& a, void* ws, cudaStream_t s) {
  LatentParams P{};
  P.T = a.T; P.B = a.B; P.n_q = a.n_q; P.H = a.H; P.max_L = a.max_L;
  P.scale_log2 = a.scale * 1.4426950408889634f;
  P.q = reinterpret_cast<const __nv_bfloat16*>(a.q);
  P.cache_rows = a.cache_rows;
  P.block_table = a.block_table; P.block_size = a.block_size; P.max_blocks = a.max_blocks;
  P.box_rows = a.block_table != nullptr && a.block_size < kRows ? a.block_size : kRows;
  P.cu = a.cu_tokens;
  P.kv_len = a.kv_len;
  P.out = reinterpret_cast<__nv_bfloat16*>(a.out);
  P.lse = a.lse;
  P.sink = a.sink;
  P.clusters = cluster_count(a);
  uint8_t* at = static_cast<uint8_t*>(ws);
  P.part_o = reinterpret_cast<float*>(at);
  at += round_up(static_cast<size_t>(P.clusters) * 2 * 128 * kDv * sizeof(float), 256);
  P.part_ml = reinterpret_cast<float2*>(at);
  at += round_up(static_cast<size_t>(P.clusters) * 2 * 128 * sizeof(float2), 256);
  P.desc = reinterpret_cast<int4*>(at);
  P.err = error_word();
  if (!P.err) return DSA_ERR_CUDA;
  alignas(64) CUtensorMap kv_map;
  {
    const uint64_t dims[2] = {static_cast<uint64_t>(kDqk), static_cast<uint64_t>(a.cache_rows)};
    const uint64_t strides[1] = {static_cast<uint64_t>(kDqk) * 2};
    const uint32_t box[2] = {64, static_cast<uint32_t>(P.box_rows)};
    if (!encode_tmap(&kv_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.kv, dims, strides, box, 128)) return DSA_ERR_CUDA;
  }
  cudaError_t e = cudaFuncSetAttribute(latent_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemBytes));
  if (e != cudaSuccess) return DSA_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(2 * P.clusters);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, latent_attn_kernel, P, kv_map);
  if (e != cudaSuccess) return DSA_ERR_CUDA;
  if (P.clusters > 1) {
    cudaLaunchConfig_t c2 = {};
    c2.gridDim = dim3(P.clusters, 32);
    c2.blockDim = dim3(256);
    c2.stream = s;
    c2.attrs = attr;
    c2.numAttrs = 1;
    e = cudaLaunchKernelEx(&c2, latent_merge_kernel, P);
  }
  return cuda_status(e);
}

}  // namespace dsa
