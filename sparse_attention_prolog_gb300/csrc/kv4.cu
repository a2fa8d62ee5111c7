// The 4-bit latent cache: rows of bf16 quantised as they are written, and
// read back as bf16 (the layout and the quantiser are stated in dsa.h).
#include <cuda.h>
#include <cuda_runtime.h>
#include "dsa_internal.h"
#include "dsa_ptx.cuh"
#include "kv4.cuh"

namespace dsa {
namespace {

constexpr int kWarps = 8;

struct Kv4Params {
  int n;
  int64_t stride;
  const uint16_t* x;
  uint16_t* out;
  uint8_t* kv4;
  const int64_t* slot;
  int64_t rows;
  uint32_t* err;
};

// Scale byte of a group whose largest |x| is a (finite): a / 7 rounded to 4
// significant bits, on its fp32 bits; the clamps are the ends of the byte's
// range (255 is kept for NaN).
__device__ __forceinline__ uint32_t scale_byte(float a) {
  const uint32_t b = __float_as_uint(a / 7.f);
  const int r = static_cast<int>((b + 0x7ffffu + ((b >> 20) & 1u)) >> 20) - (112 << 3);
  return static_cast<uint32_t>(min(max(r, 0), 254));
}

// One warp per row, one group of 16 dims per lane.
__global__ void __launch_bounds__(kWarps * 32) kv4_write_kernel(const Kv4Params P) {
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  if (i >= P.n) return;
  const int64_t slot = __ldg(P.slot + i);
  if (slot < 0) return;
  if (slot >= P.rows) {
    if (lane == 0) atomicOr(P.err, kErrBadIndex);
    return;
  }
  const uint4* xr = reinterpret_cast<const uint4*>(P.x + i * P.stride);
  uint8_t* dst = P.kv4 + slot * kKv4Row;
  const uint4 v0 = __ldg(xr + 2 * lane), v1 = __ldg(xr + 2 * lane + 1);
  const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
  uint32_t amax = 0;  // |x| as bf16 bits order like integers
#pragma unroll
  for (int k = 0; k < 8; ++k) amax = __vmaxu2(amax, w[k] & 0x7fff7fffu);
  amax = max(amax & 0xffffu, amax >> 16);
  uint32_t u = 255u, c[2] = {0u, 0u};
  if (amax < 0x7f80u) {  // no NaN, no infinity
    u = scale_byte(__uint_as_float(amax << 16));
    const float s = __uint_as_float((u << 20) + (112u << 23));
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      // dims 2k and 2k+1: nibbles k % 4 and 4 + k % 4 of word k / 4
      const int lo = __float2int_rn(fminf(fmaxf(bf16lo(w[k]) / s, -7.f), 7.f));
      const int hi = __float2int_rn(fminf(fmaxf(bf16hi(w[k]) / s, -7.f), 7.f));
      c[k / 4] |= (static_cast<uint32_t>(lo & 15) | (static_cast<uint32_t>(hi & 15) << 16)) << (4 * (k % 4));
    }
  }
  reinterpret_cast<uint2*>(dst)[lane] = make_uint2(c[0], c[1]);
  dst[kKv4Scales + lane] = static_cast<uint8_t>(u);
  if (lane < 8) reinterpret_cast<uint4*>(dst + kKv4Rope)[lane] = __ldg(xr + 64 + lane);
}

// One warp per row, one group of 16 dims per lane.
__global__ void __launch_bounds__(kWarps * 32) kv4_read_kernel(const Kv4Params P) {
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  if (i >= P.n) return;
  int64_t slot = __ldg(P.slot + i);
  if (slot >= P.rows) {
    if (lane == 0) atomicOr(P.err, kErrBadIndex);
    slot = -1;
  }
  uint4* dst = reinterpret_cast<uint4*>(P.out + i * P.stride);
  uint4 o0 = make_uint4(0, 0, 0, 0), o1 = o0, rope = o0;
  if (slot >= 0) {
    const uint8_t* src = P.kv4 + slot * kKv4Row;
    const uint2 c = *reinterpret_cast<const uint2*>(src + lane * 8);
    const Kv4Scale s = kv4_scale(src[kKv4Scales + lane]);
    if (lane < 8) rope = *reinterpret_cast<const uint4*>(src + kKv4Rope + lane * 16);
    o0 = kv4_codes8(c.x, s);
    o1 = kv4_codes8(c.y, s);
  }
  dst[2 * lane] = o0;
  dst[2 * lane + 1] = o1;
  if (lane < 8) dst[64 + lane] = rope;
}

int launch(void (*kernel)(const Kv4Params), const Kv4Params& P, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((P.n - 1) / kWarps + 1);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, kernel, P));
}

}  // namespace

int launch_kv4_write(const dsa_kv4_write_args& a, cudaStream_t s) {
  Kv4Params P{a.n, a.x_stride, a.x, nullptr, a.kv4, a.slot, a.cache_rows, error_word()};
  return P.err ? launch(kv4_write_kernel, P, s) : DSA_ERR_CUDA;
}

int launch_kv4_read(const dsa_kv4_read_args& a, cudaStream_t s) {
  Kv4Params P{a.n, a.out_stride, nullptr, a.out, const_cast<uint8_t*>(a.kv4), a.slot, a.cache_rows, error_word()};
  return P.err ? launch(kv4_read_kernel, P, s) : DSA_ERR_CUDA;
}

}  // namespace dsa
