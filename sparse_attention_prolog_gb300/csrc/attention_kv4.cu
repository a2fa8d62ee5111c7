// Sparse MLA flash attention over the top-k rows of a 4-bit latent cache, on
// tcgen05.
//
//   out[t,h] = sum_j e^{s_j} v_j / (sum_j e^{s_j} [+ e^{sink[h]}]),
//   s_j = scale q[t,h] . k_j, k_j the dequantised row, v_j its 512 latent dims
//
// One 2-CTA cluster per (token, block of 128 heads, chunk of selected rows);
// tiles of 128 rows.  An O accumulator [128 x 512] in fp32 fills a CTA's tensor
// memory, so the two products live in different CTAs:
//
//   CTA 0: S = q . K^T (M = 128 heads, N = 128 rows, K = 576) and the softmax.
//          The latent part of q is the A operand in tensor memory (256
//          columns), its rotary part in shared memory; S is double-buffered in
//          the other 256 columns.  N = 128 runs at the tensor rate (64.4 of 64
//          clocks per K = 16 step; N = 64 takes 45 of 32).
//   CTA 1: O += P . V with P sent over by CTA 0 (st.async) and the values read
//          MN-major from the converted rows.
//
// Both convert the rows they need from 4 bits to bf16: 16 warps load 64-byte
// pieces of a row (4 lanes of 16 bytes, 8 rows at a time) into registers one
// tile ahead, convert (three instructions per pair of dims, exact) and store
// into the 128B-swizzled layout the MMA reads.  A group of four warps fills one
// of four slots: a quarter of the dims of all 128 rows in CTA 0, all dims of 32
// rows in CTA 1, in the order the MMA consumes and frees them; so one tile of
// buffer keeps the tensor core fed while the next tile is converted.
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
constexpr int kSlot = 32768;               // a slot: 128 rows x 128 dims, or 32 rows x 512 dims, bf16
constexpr int kAtom = 16384;               // 128 rows (or heads) x 128 bytes
constexpr int kPSlot = 2 * kAtom;          // P [128 heads x 128 rows] bf16
// 28 warps in seven warpgroups: 0-1 softmax (CTA 0), correction and epilogue
// (CTA 1); 2-5 conversion; 6 MMA issue and the P-slot relay.  The launch
// grants 72 registers a thread: 896 x 72 = 256 x 104 + 512 x 64 + 128 x 40.
constexpr int kThreads = 896;
constexpr int kSoftWarps = 8, kConvWarps = 16, kFirstConv = 8, kMmaWarp = 24, kRelayWarp = 25;
constexpr int kRegsLaunch = 72, kRegsSoft = 104, kRegsConv = 64, kRegsLast = 40;
static_assert(256 * kRegsSoft + 512 * kRegsConv + 128 * kRegsLast <= kThreads * kRegsLaunch,
              "register split exceeds the launch allocation");
constexpr uint32_t kPBytes = 128 * (2 * 128 + 4);  // a P tile and its rescale factors
constexpr uint32_t kFinalBytes = 128 * 12;         // per head: maximum, two partial sums
constexpr uint32_t kTmemS = 256;                   // CTA 0: q in columns [0, 256), S in [256, 512)

// Dynamic shared memory.  CTA 0: four K slots, q's rotary part, two rotary K
// buffers, the row maxima that the two warps of a head exchange.  CTA 1: four V
// slots (the output staging at the end), two P slots, rescale factors, finals.
constexpr int kOffQrope = 4 * kSlot, kOffKrope = kOffQrope + kAtom, kOffMax = kOffKrope + 2 * kAtom;
constexpr int kOffP = 4 * kSlot, kOffAlpha = kOffP + 2 * kPSlot, kOffFinal = kOffAlpha + 1024;
constexpr int kSmem = 1024 + kOffFinal + 2048;
static_assert(kOffMax + 2048 <= kSmem - 1024, "CTA 0 fits CTA 1's allocation");

struct AttnKv4Params {
  int T, B, n_q, H, topk, max_L, n_chunks, chunk_rows, head_blocks;
  float scale_log2;
  const uint16_t* q;
  const uint8_t* kv4;
  int64_t rows;
  const int32_t* block_table;
  int block_size, max_blocks;
  const int32_t* idx;
  uint16_t* out;
  float* lse;
  const float* sink;
  const int32_t* seq;
  uint16_t* part_o;  // [T][n_chunks][H][512] bf16, each chunk's O / l, when n_chunks > 1
  float2* part_ml;   // [T][n_chunks][H]: (maximum, sum) in log2 units
  uint32_t* err;
};

struct __align__(8) Bars {
  uint64_t full[4], empty[4];      // K (CTA 0) or V (CTA 1) slots
  uint64_t rfull[2], rempty[2];    // CTA 0: rotary K buffers
  uint64_t sfull[2], sempty[2];    // CTA 0: S buffers
  uint64_t pfree[2];               // CTA 0: P slot of CTA 1 free
  uint64_t mx[4];                  // CTA 0: row maxima exchanged (per warp quadrant)
  uint64_t pfull[2], pcons[2];     // CTA 1: P slots
  uint64_t ready[2], odone, ffull; // CTA 1: correction / MMA
  uint64_t alldone;                // CTA 1: every PV MMA complete
  uint64_t qready;                 // CTA 0: q is in place
  uint64_t tiles;                  // the chunk's row count is known
  uint64_t mdrain;                 // the MMA thread's last commit
};

__device__ __forceinline__ float neg_inf() { return -__int_as_float(0x7f800000); }

// The page entry that position s needs (its own sequence number where the
// cache is contiguous); loaded a tile before page_row() uses it.
__device__ __forceinline__ int page_of(const AttnKv4Params& P, int b, int s) {
  if (s < 0 || P.block_table == nullptr) return b;
  return __ldg(P.block_table + static_cast<size_t>(b) * P.max_blocks + s / P.block_size);
}
// Physical row of position s (-1: nothing, or recorded and read as zeros).
__device__ __forceinline__ int page_row(const AttnKv4Params& P, int page, int s) {
  if (s < 0) return -1;
  const int64_t row = P.block_table == nullptr ? static_cast<int64_t>(page) * P.max_L + s
                                               : static_cast<int64_t>(page) * P.block_size + s % P.block_size;
  if (row < 0 || row >= P.rows || page < 0) {
    atomicOr(P.err, kErrBadIndex);
    return -1;
  }
  return static_cast<int>(row);
}

__global__ void __launch_bounds__(kThreads, 1)
    attn_kv4_kernel(const __grid_constant__ AttnKv4Params P, const __grid_constant__ CUtensorMap tmap_o) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ Bars bars;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag, last_valid, n_rows_sh;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const int chunk = blockIdx.x >> 1, hb = blockIdx.y, t = blockIdx.z;
  int b = t / P.n_q;
  bool bad_seq = false;
  if (P.seq != nullptr) {  // a token outside [0, B) reads no row and gets out = 0
    b = __ldg(P.seq + t);
    bad_seq = b < 0 || b >= P.B;
    if (bad_seq) {
      if (tid == 0 && rank == 0 && chunk == 0 && hb == 0) atomicOr(P.err, kErrBadIndex);
      b = 0;
    }
  }
  const int slot_begin = chunk * P.chunk_rows;
  const int rows_here = bad_seq ? 0 : max(0, min(P.chunk_rows, P.topk - slot_begin));
  const int32_t* idx_row = P.idx + static_cast<size_t>(t) * P.topk;

  uint8_t* sP = smem + kOffP;
  float* sAlpha = reinterpret_cast<float*>(smem + kOffAlpha);  // [2][128]
  float* sFinal = reinterpret_cast<float*>(smem + kOffFinal);  // [3][128]: maximum, sum, sum
  float* sMax = reinterpret_cast<float*>(smem + kOffMax);      // [2][2][128]

  if (tid == 0) {
    for (int i = 0; i < 4; ++i) { mbar_init(&bars.full[i], 4); mbar_init(&bars.empty[i], 1); mbar_init(&bars.mx[i], 2); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.rfull[i], kConvWarps); mbar_init(&bars.rempty[i], 1);
      mbar_init(&bars.sfull[i], 1); mbar_init(&bars.sempty[i], kSoftWarps); mbar_init(&bars.pfree[i], 1);
      mbar_init(&bars.pfull[i], 1); mbar_init(&bars.pcons[i], 1); mbar_init(&bars.ready[i], kSoftWarps);
    }
    mbar_init(&bars.odone, 1);
    mbar_init(&bars.alldone, 1);
    mbar_init(&bars.ffull, 1);
    mbar_init(&bars.qready, kSoftWarps);
    mbar_init(&bars.tiles, 1);
    mbar_init(&bars.mdrain, 1);
    last_valid = -1;
    abort_flag = 0;
    fence_mbar_init();
    if (rank == 1) {
      mbar_arrive_expect_tx(&bars.pfull[0], kPBytes);
      mbar_arrive_expect_tx(&bars.pfull[1], kPBytes);
      mbar_arrive_expect_tx(&bars.ffull, kFinalBytes);
    }
  }
  if (warp == 0) tmem_alloc(&tmem_base, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  volatile int* abort_v = &abort_flag;
  const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
  auto row_count = [&]() -> int {  // roles other than the conversion warps
    if (!mbar_wait_polling<false>(&bars.tiles, 0, P.err, abort_v)) return 0;
    return n_rows_sh;
  };
  const int q_rows = max(0, min(128, P.H - hb * 128));  // real heads of this block
  cluster_sync();  // both CTAs' barriers are initialised before any remote use
  griddep_launch_dependents();

  if (warp >= kFirstConv && warp < kFirstConv + kConvWarps) {
    setmaxnreg_dec<kRegsConv>();
    // ------------------------------------------------- conversion (both CTAs)
    const int cw = warp - kFirstConv, grp = cw >> 2, wi = cw & 3;
    const int rb = rank == 0 ? wi : grp;  // rows [32 rb, 32 rb + 32) of a tile
    const int dq = rank == 0 ? grp : wi;  // dims [128 dq, 128 dq + 128)
    const int g = lane & 3, r8 = lane >> 2;
    griddep_wait();  // the index rows come from the previous kernel
    // position of this lane's row of tile jj (-1: nothing)
    auto load_pos = [&](int jj) -> int {
      const int i = jj * kTile + rb * 32 + lane;
      const int s = i < rows_here ? __ldg(idx_row + slot_begin + i) : -1;
      return s < P.max_L ? s : -1;
    };
    int s0 = load_pos(0), s1 = load_pos(1), s2 = load_pos(2);
    int n_rows;
    {
      // a valid last slot (every decode chunk) ends the chunk at once; else the
      // conversion warps find the last valid slot together
      const int last = rows_here > 0 ? __ldg(idx_row + slot_begin + rows_here - 1) : -1;
      if (rows_here == 0 || (last >= 0 && last < P.max_L)) {
        n_rows = rows_here;
      } else {
        int mx = -1;
        for (int i = cw * 32 + lane; i < rows_here; i += kConvWarps * 32) {
          const int s = __ldg(idx_row + slot_begin + i);
          if (s >= 0 && s < P.max_L) mx = i;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if (lane == 0 && mx >= 0) atomicMax(&last_valid, mx);
        asm volatile("bar.sync 1, %0;" ::"n"(kConvWarps * 32) : "memory");
        n_rows = last_valid + 1;
      }
      if (cw == 0 && lane == 0) {
        n_rows_sh = n_rows;
        mbar_arrive(&bars.tiles);
      }
    }
    const int n_tiles = (n_rows + kTile - 1) / kTile;
    int page1 = page_of(P, b, s1);
    uint4 c[4];
    uint2 rope[4];
    uint32_t sc[4];
    const uint8_t* src = P.kv4 + dq * 64 + g * 16;
    // one piece (8 rows) of a tile: 16 bytes of codes and 2 scale bytes a lane,
    // and in CTA 0 8 bytes of the rotary dims
    auto load = [&](int i, int row_l) {
      const int row = __shfl_sync(0xffffffffu, row_l, i * 8 + r8);
      c[i] = make_uint4(0, 0, 0, 0);
      rope[i] = make_uint2(0, 0);
      sc[i] = 0;
      if (row >= 0) {
        const uint8_t* p = src + static_cast<size_t>(row) * kKv4Row;
        c[i] = __ldg(reinterpret_cast<const uint4*>(p));
        sc[i] = __ldg(reinterpret_cast<const uint16_t*>(p + (kKv4Scales - dq * 56 - g * 14)));
        if (rank == 0) rope[i] = __ldg(reinterpret_cast<const uint2*>(p + (kKv4Rope - dq * 32 - g * 8)));
      }
    };
    {
      const int row0 = page_row(P, page_of(P, b, s0), s0);
#pragma unroll
      for (int i = 0; i < 4; ++i) load(i, row0);
    }
    // this lane's address in a slot: 16-byte chunk kk ^ C of its row
    const uint32_t C = (g & 2) ^ ((g & 1) << 2) ^ r8;
    const uint32_t row_bytes = rank == 0 ? rb * 32 * 128 : 0;             // first row of the block in its atom
    const uint32_t atom = rank == 0 ? (g >> 1) * kAtom : (dq * 2 + (g >> 1)) * 4096;
    const uint32_t dst = smem_u32(smem) + grp * kSlot + atom + row_bytes + r8 * 128;
    const uint32_t rdst = smem_u32(smem + kOffKrope) + row_bytes + r8 * 128 + ((((dq * 2) + (g >> 1)) ^ r8) << 4) + (g & 1) * 8;
    for (int j = 0; j < n_tiles; ++j) {
      const int row1 = j + 1 < n_tiles ? page_row(P, page1, s1) : -1;
      s1 = s2;
      page1 = page_of(P, b, s1);
      s2 = load_pos(j + 3);
      const int rows_t = min(kTile, n_rows - j * kTile);
      const bool used = rb * 32 < rows_t;  // blocks past the last row are not read by the MMA
      if (rank == 1 && !used) break;       // (only in the last tile)
      if (!mbar_wait_polling<false>(&bars.empty[grp], (j & 1) ^ 1, P.err, abort_v)) break;
      if (rank == 0 && !mbar_wait_polling<false>(&bars.rempty[j & 1], ((j >> 1) & 1) ^ 1, P.err, abort_v)) break;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (used) {
          Kv4Scale lo = kv4_scale(sc[i] & 255u), hi = kv4_scale(sc[i] >> 8);
          uint4 w = c[i];
          if (g & 2) {  // lanes of the second atom store in another order: no bank conflicts
            const Kv4Scale t0 = lo; lo = hi; hi = t0;
            w = make_uint4(c[i].z, c[i].w, c[i].x, c[i].y);
          }
          const uint32_t d = dst + i * 1024;
          auto store = [&](uint32_t kk, const uint4& v) {
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(d + ((kk ^ C) << 4)), "r"(v.x), "r"(v.y),
                         "r"(v.z), "r"(v.w) : "memory");
          };
          store(0, kv4_codes8(w.x, lo));
          store(1, kv4_codes8(w.y, lo));
          store(2, kv4_codes8(w.z, hi));
          store(3, kv4_codes8(w.w, hi));
          if (rank == 0)
            asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(rdst + (j & 1) * kAtom + i * 1024), "r"(rope[i].x),
                         "r"(rope[i].y) : "memory");
        }
        load(i, row1);
      }
      fence_proxy_async_smem();  // generic writes -> tensor core reads
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bars.full[grp]);
        if (rank == 0) mbar_arrive(&bars.rfull[j & 1]);
      }
    }
  } else {
    bool ok = true;
    int n_rows = -1;  // set by each role where it first needs it
    if (warp < kSoftWarps) {
      setmaxnreg_inc<kRegsSoft>();
      const int hrow = (warp & 3) * 32 + lane, hf = warp >> 2;
      if (rank == 0) {
        // ------------------------------------------------- softmax (CTA 0)
        // Two threads per head, each 64 of a tile's 128 rows.
        const uint32_t remote_p = mapa(smem_u32(sP), 1) + hf * kAtom;
        const uint32_t remote_alpha = mapa(smem_u32(sAlpha), 1);
        const uint32_t remote_final = mapa(smem_u32(sFinal), 1);
        const uint32_t remote_pfull[2] = {mapa(smem_u32(&bars.pfull[0]), 1), mapa(smem_u32(&bars.pfull[1]), 1)};
        const uint32_t remote_ffull = mapa(smem_u32(&bars.ffull), 1);
        {
          // q row of this thread's head: 256 latent dims to tensor memory, 32
          // rotary dims to shared memory
          const bool real = hrow < q_rows;
          const uint4* qrow =
              reinterpret_cast<const uint4*>(P.q + (static_cast<size_t>(t) * P.H + hb * 128 + (real ? hrow : 0)) * kDqk);
          uint4 rp[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) rp[i] = real ? __ldg(qrow + 64 + hf * 4 + i) : make_uint4(0, 0, 0, 0);
#pragma unroll 1
          for (int a = 0; a < 2; ++a) {
            uint4 v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = real ? __ldg(qrow + hf * 32 + a * 16 + i) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              uint32_t r[32];
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                r[4 * k] = v[x * 8 + k].x; r[4 * k + 1] = v[x * 8 + k].y;
                r[4 * k + 2] = v[x * 8 + k].z; r[4 * k + 3] = v[x * 8 + k].w;
              }
              tmem_st32(tmem + lane_off + hf * 128 + a * 64 + x * 32, r);
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4*>(smem + kOffQrope + sw128_off(hrow, hf * 4 + i)) = rp[i];
          fence_proxy_async_smem();
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.qready);
        griddep_wait();  // the index rows come from the previous kernel
        float m_used = neg_inf(), l_sum = 0.f;
        auto load_idx = [&](int jj, int& lo, int& hi) {
          const int i = jj * kTile + hf * 64 + lane;
          lo = i < rows_here ? __ldg(idx_row + slot_begin + i) : -1;
          hi = i + 32 < rows_here ? __ldg(idx_row + slot_begin + i + 32) : -1;
        };
        int nx_lo, nx_hi;
        load_idx(0, nx_lo, nx_hi);  // before the row count: one round trip
        n_rows = row_count();
        const int n_tiles = (n_rows + kTile - 1) / kTile;
        const uint64_t scale2 = pack_f32x2(P.scale_log2, P.scale_log2);
        for (int j = 0; j < n_tiles; ++j) {
          const int sb = j & 1, ph = (j >> 1) & 1;
          const uint32_t v_lo = __ballot_sync(0xffffffffu, nx_lo >= 0 && nx_lo < P.max_L);
          const uint32_t v_hi = __ballot_sync(0xffffffffu, nx_hi >= 0 && nx_hi < P.max_L);
          load_idx(j + 1, nx_lo, nx_hi);
          ok = mbar_wait_polling<false>(&bars.sfull[sb], ph, P.err, abort_v) && ok;
          tc_fence_after();
          uint32_t s[64];
          {
            uint32_t(&a)[32] = *reinterpret_cast<uint32_t(*)[32]>(s);
            uint32_t(&c)[32] = *reinterpret_cast<uint32_t(*)[32]>(s + 32);
            tmem_ld32(tmem + lane_off + kTmemS + sb * kTile + hf * 64, a);
            tmem_ld32(tmem + lane_off + kTmemS + sb * kTile + hf * 64 + 32, c);
            tmem_ld_wait();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.sempty[sb]);
          if ((v_lo & v_hi) != 0xffffffffu) {
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              if (!((v_lo >> k) & 1u)) s[k] = 0xff800000u;
              if (!((v_hi >> k) & 1u)) s[32 + k] = 0xff800000u;
            }
          }
          float mt[4] = {neg_inf(), neg_inf(), neg_inf(), neg_inf()};
#pragma unroll
          for (int k = 0; k < 64; ++k) mt[k & 3] = fmaxf(mt[k & 3], __uint_as_float(s[k]));
          float m_tile = fmaxf(fmaxf(mt[0], mt[1]), fmaxf(mt[2], mt[3])) * P.scale_log2;
          // the other 64 rows' maximum, from the warp that holds them
          sMax[(j & 1) * 256 + hf * 128 + hrow] = m_tile;
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.mx[warp & 3]);
          ok = mbar_wait_polling<false>(&bars.mx[warp & 3], j & 1, P.err, abort_v) && ok;
          m_tile = fmaxf(m_tile, sMax[(j & 1) * 256 + (hf ^ 1) * 128 + hrow]);
          float alpha = 1.f;
          if (m_tile > m_used + 8.f) {  // also taken when m_used is -inf
            alpha = ex2_approx(m_used - m_tile);
            l_sum *= alpha;
            m_used = m_tile;
          }
          const float msub = m_used == neg_inf() ? 0.f : -m_used;
          const uint64_t msub2 = pack_f32x2(msub, msub);
          uint64_t sum2[2] = {0, 0};
          const uint64_t one2 = pack_f32x2(1.f, 1.f);
          uint32_t pk[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const uint64_t x = fma_f32x2(pack_f32x2(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1])), scale2, msub2);
            const float p0 = ex2_approx(lo_f32(x)), p1 = ex2_approx(hi_f32(x));
            sum2[k & 1] = fma_f32x2(pack_f32x2(p0, p1), one2, sum2[k & 1]);
            __nv_bfloat162 pb = __floats2bfloat162_rn(p0, p1);
            pk[k] = *reinterpret_cast<uint32_t*>(&pb);
          }
          l_sum += (lo_f32(sum2[0]) + hi_f32(sum2[0])) + (lo_f32(sum2[1]) + hi_f32(sum2[1]));
          ok = mbar_wait_polling<true>(&bars.pfree[sb], ph ^ 1, P.err, abort_v) && ok;
          if (ok) {
            const uint32_t prow = remote_p + sb * kPSlot;
#pragma unroll
            for (int k = 0; k < 8; ++k)
              st_async_v4(prow + sw128_off(hrow, k), make_uint4(pk[4 * k], pk[4 * k + 1], pk[4 * k + 2], pk[4 * k + 3]),
                          remote_pfull[sb]);
            if (hf == 0) st_async_b32(remote_alpha + (sb * 128 + hrow) * 4, __float_as_uint(alpha), remote_pfull[sb]);
          }
        }
        if (hf == 0) st_async_b32(remote_final + hrow * 4, __float_as_uint(m_used), remote_ffull);
        st_async_b32(remote_final + (128 + hf * 128 + hrow) * 4, __float_as_uint(l_sum), remote_ffull);
      } else {
        // ----------------------------------------- correction (CTA 1)
        n_rows = row_count();
        const int n_tiles = (n_rows + kTile - 1) / kTile;
        int consumed = 0;  // odone phases observed
        for (int j = 0; j < n_tiles && ok; ++j) {
          const int ps = j & 1;
          if (!mbar_wait_polling<true>(&bars.pfull[ps], (j >> 1) & 1, P.err, abort_v)) { ok = false; break; }
          const float alpha = sAlpha[ps * 128 + hrow];
          const bool need = __any_sync(0xffffffffu, alpha != 1.f) && j > 0;
          if (need) {
            // O must hold PV of tile j-1 before it is rescaled.
            while (consumed < j) {
              if (!mbar_wait_polling<false>(&bars.odone, consumed & 1, P.err, abort_v)) { ok = false; break; }
              ++consumed;
            }
            if (!ok) break;
            tc_fence_after();
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
          fence_proxy_async_smem();  // P arrived through st.async; the MMA reads it
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.ready[ps]);
          // keep at most one PV completion unobserved
          while (consumed < j) {
            if (!mbar_wait_polling<false>(&bars.odone, consumed & 1, P.err, abort_v)) { ok = false; break; }
            ++consumed;
          }
        }
      }
    } else {
      setmaxnreg_dec<kRegsLast>();
      if (warp == kMmaWarp && rank == 0) {
        // ---------------------------------------------- QK^T MMA (CTA 0)
        if (lane == 0) {
          n_rows = row_count();
          const int n_tiles = (n_rows + kTile - 1) / kTile;
          const uint32_t base = smem_u32(smem);
          if (n_tiles > 0 && mbar_wait_polling<false>(&bars.qready, 0, P.err, abort_v)) tc_fence_after();
          for (int j = 0; j < n_tiles && ok; ++j) {
            const int sb = j & 1;
            const int rows_t = min(kTile, n_rows - j * kTile);
            const uint32_t idesc = idesc_f16(128, (rows_t + 31) & ~31, kFmtBF16, 0, 0);
            const uint32_t d = tmem + kTmemS + sb * kTile;
            if (!mbar_wait_polling<false>(&bars.sempty[sb], ((j >> 1) & 1) ^ 1, P.err, abort_v)) break;
            for (int qd = 0; qd < 4 && ok; ++qd) {
              ok = mbar_wait_polling<false>(&bars.full[qd], j & 1, P.err, abort_v);
              if (!ok) break;
              tc_fence_after();
#pragma unroll
              for (int kk = 0; kk < 8; ++kk) {
                const uint64_t bd = smem_desc(base + qd * kSlot + (kk / 4) * kAtom + (kk % 4) * 32, 16, 1024, kSwizzle128B);
                mma_ts(d, tmem + qd * 64 + kk * 8, bd, idesc, (qd | kk) != 0 ? 1u : 0u);
              }
              mma_commit(&bars.empty[qd]);
            }
            if (!ok || !mbar_wait_polling<false>(&bars.rfull[sb], (j >> 1) & 1, P.err, abort_v)) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const uint64_t ad = smem_desc(base + kOffQrope + kk * 32, 16, 1024, kSwizzle128B);
              const uint64_t bd = smem_desc(base + kOffKrope + sb * kAtom + kk * 32, 16, 1024, kSwizzle128B);
              mma_ss(d, ad, bd, idesc, 1u);
            }
            mma_commit(&bars.rempty[sb]);
            mma_commit(&bars.sfull[sb]);
          }
          // every MMA issued has completed before the tensor memory is freed
          mma_commit(&bars.mdrain);
          mbar_drain(&bars.mdrain, 0);
        }
      } else if (warp == kMmaWarp) {
        // ------------------------------------------------- PV MMA (CTA 1)
        if (lane == 0) {
          n_rows = row_count();
          const int n_tiles = (n_rows + kTile - 1) / kTile;
          const uint32_t idesc = idesc_f16(128, 256, kFmtBF16, 0, 1);
          const uint32_t vbase = smem_u32(smem), pbase = smem_u32(sP);
          for (int j = 0; j < n_tiles && ok; ++j) {
            const int ps = j & 1;
            const int rows_t = min(kTile, n_rows - j * kTile);
            if (!mbar_wait_polling<false>(&bars.ready[ps], (j >> 1) & 1, P.err, abort_v)) break;
            for (int qd = 0; qd * 32 < rows_t; ++qd) {
              ok = mbar_wait_polling<false>(&bars.full[qd], j & 1, P.err, abort_v);
              if (!ok) break;
              tc_fence_after();
#pragma unroll
              for (int kk = 0; kk < 2; ++kk) {
                const uint64_t ad =
                    smem_desc(pbase + ps * kPSlot + (qd >> 1) * kAtom + ((qd & 1) * 2 + kk) * 32, 16, 1024, kSwizzle128B);
#pragma unroll
                for (int nh = 0; nh < 2; ++nh) {
                  const uint64_t bd = smem_desc(vbase + qd * kSlot + nh * 4 * 4096 + kk * 16 * 128, 4096, 1024, kSwizzle128B);
                  mma_ss(tmem + nh * 256, ad, bd, idesc, (j | qd | kk) != 0 ? 1u : 0u);
                }
              }
              mma_commit(&bars.empty[qd]);
            }
            if (!ok) break;
            mma_commit(&bars.pcons[ps]);
            mma_commit(&bars.odone);
            if (j + 1 == n_tiles) mma_commit(&bars.alldone);
          }
          mma_commit(&bars.mdrain);
          mbar_drain(&bars.mdrain, 0);
        }
      } else if (warp == kRelayWarp && rank == 1) {
        // ----------------------------------- relay: P slot consumed -> CTA 0
        if (lane == 0) {
          n_rows = row_count();
          const int n_tiles = (n_rows + kTile - 1) / kTile;
          const uint32_t remote_pfree[2] = {mapa(smem_u32(&bars.pfree[0]), 0), mapa(smem_u32(&bars.pfree[1]), 0)};
          for (int j = 0; j + 2 < n_tiles; ++j) {
            const int ps = j & 1;
            if (!mbar_wait_polling<false>(&bars.pcons[ps], (j >> 1) & 1, P.err, abort_v)) break;
            mbar_arrive_expect_tx(&bars.pfull[ps], kPBytes);  // arm the slot's next use
            mbar_arrive_remote(remote_pfree[ps]);
          }
        }
      }
    }
    if (rank == 1 && warp < kSoftWarps) {
      // ------------------------------------------------- epilogue (CTA 1)
      // Every PV product is in O and (maximum, sums) of each head have arrived:
      // normalise, convert to bf16 into a swizzled staging tile (the free V
      // slots) and write it with TMA stores, 64 columns x 128 heads per box
      // (heads past H are clipped by the tensor map).
      __syncwarp();
      const bool none = n_rows == 0;
      if (ok && !none) ok = mbar_wait_polling<false>(&bars.alldone, 0, P.err, abort_v);
      if (ok) ok = mbar_wait_polling<true>(&bars.ffull, 0, P.err, abort_v);
      tc_fence_after();
      const int hrow = (warp & 3) * 32 + lane, half = warp >> 2;
      const float m = sFinal[hrow], l = sFinal[128 + hrow] + sFinal[256 + hrow];
      const bool empty = !ok || none || l == 0.f;
      const int h = hb * 128 + hrow;
      float inv_l = empty ? 0.f : 1.f / l;
      float lse2 = empty ? neg_inf() : m + log2f(l);  // log2 units
      if (P.sink != nullptr && P.n_chunks == 1) {
        // The sink adds 2^s2 to the denominator; taken relative to max(m, s2) so
        // that neither term overflows.  (Split chunks get it in the merge.)
        const float s2 = (h < P.H ? __ldg(P.sink + h) : neg_inf()) * 1.4426950408889634f;
        if (!empty) {
          const float mx = fmaxf(m, s2);
          const float den = l * exp2f(m - mx) + exp2f(s2 - mx);
          inv_l = exp2f(m - mx) / den;
          lse2 = mx + log2f(den);
        } else {
          lse2 = s2;
        }
      }
#pragma unroll 1
      for (int c0 = half * 256; c0 < half * 256 + 256; c0 += 64) {  // one atom per round
        uint8_t* stage = smem + (c0 / 64) * kAtom;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t v[32], pk[16];
          tmem_ld32(tmem + lane_off + c0 + x * 32, v);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            __nv_bfloat162 w = __floats2bfloat162_rn(__uint_as_float(v[2 * k]) * inv_l, __uint_as_float(v[2 * k + 1]) * inv_l);
            pk[k] = empty ? 0u : *reinterpret_cast<uint32_t*>(&w);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *reinterpret_cast<uint4*>(stage + sw128_off(hrow, x * 4 + k)) =
                make_uint4(pk[4 * k], pk[4 * k + 1], pk[4 * k + 2], pk[4 * k + 3]);
        }
        // the 4 warps of this half have written the atom: store it while they
        // convert the next one
        fence_proxy_async_smem();
        asm volatile("bar.sync %0, 128;" ::"r"(2 + half) : "memory");
        if ((warp & 3) == 0 && lane == 0) {
          tma_store_3d(&tmap_o, stage, c0, hb * 128, P.n_chunks == 1 ? t : t * P.n_chunks + chunk);
          bulk_commit_group();
        }
      }
      if ((warp & 3) == 0 && lane == 0) bulk_wait_group_read0();
      if (half == 0 && h < P.H) {
        if (P.n_chunks == 1) {
          if (P.lse != nullptr) P.lse[static_cast<size_t>(t) * P.H + h] = lse2 * 0.69314718055994531f;
        } else {
          P.part_ml[(static_cast<size_t>(t) * P.n_chunks + chunk) * P.H + h] =
              empty ? make_float2(neg_inf(), 0.f) : make_float2(m, l);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no CTA leaves while its peer may still address it
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// Merges a token's chunks: out = sum_c w_c O_c / (sum_c w_c [+ 2^(sink - M)])
// with w_c = l_c 2^(m_c - M) (O_c already divided by l_c).  One warp per
// (token, head, half of the 512 columns), 8 columns per lane; the loads of a
// batch of chunks are issued together, so a batch costs one memory round trip.
constexpr int kMergeBatch = 8;

__global__ void __launch_bounds__(256) attn_kv4_merge_kernel(const AttnKv4Params P) {
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int item = blockIdx.x * 8 + warp;  // (token, head, column half)
  if (item >= P.T * P.H * 2) return;
  const int th = item >> 1, half = item & 1;
  const int t = th / P.H, h = th % P.H;
  const int col = half * 256 + lane * 8;
  float acc[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) acc[k] = 0.f;
  float M = neg_inf(), wsum = 0.f;
  for (int c0 = 0; c0 < P.n_chunks; c0 += kMergeBatch) {
    float2 ml[kMergeBatch];
    uint4 raw[kMergeBatch];
#pragma unroll
    for (int i = 0; i < kMergeBatch; ++i) {
      ml[i] = make_float2(neg_inf(), 0.f);
      raw[i] = make_uint4(0u, 0u, 0u, 0u);
      if (c0 + i < P.n_chunks) {
        const size_t row = (static_cast<size_t>(t) * P.n_chunks + c0 + i) * P.H + h;
        ml[i] = __ldcg(P.part_ml + row);
        raw[i] = __ldcg(reinterpret_cast<const uint4*>(P.part_o + row * kDv + col));
      }
    }
    float Mb = M;
#pragma unroll
    for (int i = 0; i < kMergeBatch; ++i) Mb = fmaxf(Mb, ml[i].x);
    if (Mb == neg_inf()) continue;  // nothing visible yet
    const float r = exp2f(M - Mb);
    wsum *= r;
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] *= r;
    M = Mb;
#pragma unroll
    for (int i = 0; i < kMergeBatch; ++i) {
      const float wc = ml[i].y * exp2f(ml[i].x - M);  // 0 for an empty chunk
      wsum += wc;
      const uint32_t wds[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        acc[2 * k] = fmaf(wc, bf16lo(wds[k]), acc[2 * k]);
        acc[2 * k + 1] = fmaf(wc, bf16hi(wds[k]), acc[2 * k + 1]);
      }
    }
  }
  if (P.sink != nullptr) {
    // one more term 2^s2 in the denominator (a zero-value key); -inf: none
    const float s2 = __ldg(P.sink + h) * 1.4426950408889634f;
    const float mx = fmaxf(M, s2);
    if (mx != neg_inf()) {
      const float r = exp2f(M - mx);
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] *= r;
      wsum = wsum * r + exp2f(s2 - mx);
      M = mx;
    }
  }
  const float inv = wsum == 0.f ? 0.f : 1.f / wsum;
  uint32_t pk[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    __nv_bfloat162 b2 = __floats2bfloat162_rn(acc[2 * k] * inv, acc[2 * k + 1] * inv);
    pk[k] = *reinterpret_cast<uint32_t*>(&b2);
  }
  *reinterpret_cast<uint4*>(P.out + (static_cast<size_t>(t) * P.H + h) * kDv + col) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
  if (half == 0 && lane == 0 && P.lse != nullptr)
    P.lse[static_cast<size_t>(t) * P.H + h] = wsum == 0.f ? neg_inf() : (M + log2f(wsum)) * 0.69314718055994531f;
}

// Chunks per token: as many clusters as the GPU holds at once, each a
// multiple of 64 rows.
void plan(const dsa_attn_kv4_args& a, int& head_blocks, int& n_chunks, int& chunk_rows) {
  head_blocks = (a.H + 127) / 128;
  const long long pairs = static_cast<long long>(a.T) * head_blocks;
  const int units = (a.topk + 63) / 64;
  const int target = static_cast<int>(std::max<long long>(1, sm_count() / (2 * pairs)));
  chunk_rows = (units + target - 1) / target * 64;
  n_chunks = (a.topk + chunk_rows - 1) / chunk_rows;
}

}  // namespace

size_t attn_kv4_workspace(const dsa_attn_kv4_args& a) {
  int hb, nc, cr;
  plan(a, hb, nc, cr);
  if (nc == 1) return 0;
  const size_t heads = static_cast<size_t>(a.T) * nc * a.H;
  return round_up(heads * kDv * 2, 256) + round_up(heads * sizeof(float2), 256);
}

int launch_attn_kv4(const dsa_attn_kv4_args& a, void* ws, cudaStream_t s) {
  AttnKv4Params P{};
  plan(a, P.head_blocks, P.n_chunks, P.chunk_rows);
  P.T = a.T; P.B = a.B; P.n_q = a.n_q; P.H = a.H; P.topk = a.topk; P.max_L = a.max_L;
  P.scale_log2 = a.scale * 1.4426950408889634f;
  P.q = a.q; P.kv4 = a.kv4; P.rows = a.cache_rows;
  P.block_table = a.block_table; P.block_size = a.block_size; P.max_blocks = a.max_blocks;
  P.idx = a.topk_idx; P.out = a.out; P.lse = a.lse; P.sink = a.sink; P.seq = a.seq_of_token;
  if (P.seq != nullptr) P.n_q = 1;  // ignored with a map
  if (P.n_chunks > 1) {
    P.part_o = static_cast<uint16_t*>(ws);
    P.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) +
                                          round_up(static_cast<size_t>(a.T) * P.n_chunks * a.H * kDv * 2, 256));
  }
  P.err = error_word();
  if (!P.err) return DSA_ERR_CUDA;

  // output (or the chunks' partial outputs): [Z, H, 512] bf16, stored as
  // 64-column x 128-head boxes; heads past H are clipped by the map
  alignas(64) CUtensorMap tmap_o;
  {
    const uint64_t z = static_cast<uint64_t>(a.T) * P.n_chunks;
    const uint64_t dims[3] = {static_cast<uint64_t>(kDv), static_cast<uint64_t>(a.H), z};
    const uint64_t strides[2] = {static_cast<uint64_t>(kDv) * 2, static_cast<uint64_t>(a.H) * kDv * 2};
    const uint32_t box[3] = {64, 128, 1};
    if (!encode_tmap(&tmap_o, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, P.n_chunks == 1 ? P.out : P.part_o, dims, strides,
                     box, 128))
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
  cfg.gridDim = dim3(P.n_chunks * 2, P.head_blocks, a.T);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, attn_kv4_kernel, P, tmap_o);
  if (e != cudaSuccess) return DSA_ERR_CUDA;
  if (P.n_chunks > 1) {
    cudaLaunchConfig_t c2 = {};
    c2.gridDim = dim3((a.T * a.H * 2 + 7) / 8);
    c2.blockDim = dim3(256);
    c2.stream = s;
    c2.attrs = attr;
    c2.numAttrs = 1;
    e = cudaLaunchKernelEx(&c2, attn_kv4_merge_kernel, P);
  }
  return cuda_status(e);
}

}  // namespace dsa
