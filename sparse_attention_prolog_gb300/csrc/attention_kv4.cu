// Sparse MLA flash attention over the top-k rows of a 4-bit latent cache.
//
//   out[t,h] = sum_j e^{s_j} v_j / (sum_j e^{s_j} [+ e^{sink[h]}]),
//   s_j = scale q[t,h] . k_j, k_j the dequantised row, v_j its 512 latent dims
//
// One warp per (token, head): the lane owns a group of 16 latent dims and 2
// rotary dims of q, of each row and of the output; rows are taken one at a
// time with the running maximum and sum of an online softmax.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include "dsa_internal.h"
#include "dsa_ptx.cuh"
#include "kv4.cuh"

namespace dsa {
namespace {

constexpr int kWarps = 8;

struct AttnKv4Params {
  int T, B, n_q, H, topk, max_L;
  float scale;
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
  uint32_t* err;
};

// Physical row of position s of sequence b (-1: recorded, read as zeros).
__device__ __forceinline__ int kv_row(const AttnKv4Params& P, int b, int s) {
  int64_t row = static_cast<int64_t>(b) * P.max_L + s;
  if (P.block_table != nullptr) {
    const int blk = __ldg(P.block_table + static_cast<size_t>(b) * P.max_blocks + s / P.block_size);
    row = blk < 0 ? -1 : static_cast<int64_t>(blk) * P.block_size + s % P.block_size;
  }
  if (row < 0 || row >= P.rows) {
    atomicOr(P.err, kErrBadIndex);
    return -1;
  }
  return static_cast<int>(row);
}

__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16lo(w[i]);
    f[2 * i + 1] = bf16hi(w[i]);
  }
}

__global__ void __launch_bounds__(kWarps * 32) attn_kv4_kernel(const AttnKv4Params P) {
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.x * kWarps + warp, t = blockIdx.y;
  if (h >= P.H) return;
  const float ninf = -__int_as_float(0x7f800000);
  int b = t / P.n_q;
  bool bad_seq = false;
  if (P.seq != nullptr) {
    b = __ldg(P.seq + t);
    bad_seq = b < 0 || b >= P.B;
    if (bad_seq && lane == 0) atomicOr(P.err, kErrBadIndex);
  }
  float q[18], o[16];
  const uint16_t* qr = P.q + (static_cast<size_t>(t) * P.H + h) * 576;
  unpack8(__ldg(reinterpret_cast<const uint4*>(qr + lane * 16)), q);
  unpack8(__ldg(reinterpret_cast<const uint4*>(qr + lane * 16) + 1), q + 8);
  const uint32_t qp = __ldg(reinterpret_cast<const uint32_t*>(qr + 512) + lane);
  q[16] = bf16lo(qp);
  q[17] = bf16hi(qp);
#pragma unroll
  for (int k = 0; k < 16; ++k) o[k] = 0.f;
  float m = ninf, l = 0.f;
  const int32_t* idx = P.idx + static_cast<size_t>(t) * P.topk;
  for (int j0 = 0; j0 < P.topk && !bad_seq; j0 += 32) {
    const int s = j0 + lane < P.topk ? __ldg(idx + j0 + lane) : -1;
    const bool on = s >= 0 && s < P.max_L;
    const int row_l = on ? kv_row(P, b, s) : -1;
    uint32_t todo = __ballot_sync(0xffffffffu, on);
    while (todo) {
      const int src = __ffs(todo) - 1;
      todo &= todo - 1;
      const int row = __shfl_sync(0xffffffffu, row_l, src);
      float v[18];
#pragma unroll
      for (int k = 0; k < 18; ++k) v[k] = 0.f;
      if (row >= 0) {
        const uint8_t* r = P.kv4 + static_cast<size_t>(row) * kKv4Row;
        const uint2 c = *reinterpret_cast<const uint2*>(r + lane * 8);
        const Kv4Scale sc = kv4_scale(r[kKv4Scales + lane]);
        unpack8(kv4_codes8(c.x, sc), v);
        unpack8(kv4_codes8(c.y, sc), v + 8);
        const uint32_t rp = *reinterpret_cast<const uint32_t*>(r + kKv4Rope + lane * 4);
        v[16] = bf16lo(rp);
        v[17] = bf16hi(rp);
      }
      float d = 0.f;
#pragma unroll
      for (int k = 0; k < 18; ++k) d = fmaf(q[k], v[k], d);
#pragma unroll
      for (int x = 16; x; x >>= 1) d += __shfl_xor_sync(0xffffffffu, d, x);
      d *= P.scale;
      const float mn = fmaxf(m, d);
      const float a = m == ninf ? 0.f : expf(m - mn), p = expf(d - mn);
      l = l * a + p;
#pragma unroll
      for (int k = 0; k < 16; ++k) o[k] = fmaf(o[k], a, p * v[k]);
      m = mn;
    }
  }
  float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  float lse = l == 0.f ? ninf : m + logf(l);
  if (P.sink != nullptr) {
    const float sk = __ldg(P.sink + h);
    const float mx = fmaxf(lse, sk);
    if (mx != ninf) {
      const float all = mx + logf(expf(lse - mx) + expf(sk - mx));
      inv *= expf(lse - all);
      lse = all;
    }
  }
  uint32_t pk[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    __nv_bfloat162 w = __floats2bfloat162_rn(o[2 * k] * inv, o[2 * k + 1] * inv);
    pk[k] = *reinterpret_cast<uint32_t*>(&w);
  }
  uint4* dst = reinterpret_cast<uint4*>(P.out + (static_cast<size_t>(t) * P.H + h) * 512 + lane * 16);
  dst[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
  dst[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
  if (lane == 0 && P.lse != nullptr) P.lse[static_cast<size_t>(t) * P.H + h] = lse;
}

}  // namespace

size_t attn_kv4_workspace(const dsa_attn_kv4_args&) { return 0; }

int launch_attn_kv4(const dsa_attn_kv4_args& a, void*, cudaStream_t s) {
  AttnKv4Params P{a.T, a.B, a.n_q, a.H, a.topk, a.max_L, a.scale, a.q, a.kv4, a.cache_rows, a.block_table,
                  a.block_size, a.max_blocks, a.topk_idx, a.out, a.lse, a.sink, a.seq_of_token, error_word()};
  if (!P.err) return DSA_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((a.H + kWarps - 1) / kWarps, a.T);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, attn_kv4_kernel, P));
}

}  // namespace dsa
