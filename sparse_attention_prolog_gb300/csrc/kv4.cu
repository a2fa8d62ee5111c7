// The 4-bit latent cache: rows of bf16 quantised as they are written, and
// read back as bf16 (the layout and the quantiser are stated in dsa.h).
#include <cuda.h>
#include <cuda_runtime.h>
#include "dsa_internal.h"
#include "dsa_ptx.cuh"
#include "kv4.cuh"

namespace dsa {
namespace {

// Both kernels are bound by memory.  131071 rows written and read back: 72 us, 5.7 TB/s
// of the 412 MB that cannot be spared (a plain copy: 6.8 TB/s); 262144 rows read: 68 us,
// 6.1 TB/s.  Blocks of 4 warps start and end in smaller steps than larger ones
// (8 warps: 74 and 69 us; 16: 78 and 72).
constexpr int kWarps = 4;

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

// rint(clamp(x / s, -7, 7)) in 4 bits, from r = 1 / s (see kv4_write_kernel).
__device__ __forceinline__ uint32_t code(float x, float r) {
  constexpr float kSnap = 0x1.8p11f, kInt = 0x1.8p23f;  // 1.5 * 2^11, 1.5 * 2^23
  const float q = fminf(fmaxf(fmaf(x, r, kSnap), kSnap - 7.f), kSnap + 7.f);
  return __float_as_uint(q + (kInt - kSnap)) & 15u;
}

// A warp per row: a lane takes the 8 dims of 16 bytes from each half of a row, so
// every load and store of the warp is one run of bytes (a lane per group, whose
// stores leave gaps, took 89 us for the rows above).  Two lanes share a group;
// the even one finds the scale of the group in the first half, the odd one that of the
// second, and they exchange them.
//
// x / s is rounded to a code without a division: r = 1/s is off by 2^-24 of its value,
// x r thus by less than 2^-20.  An x / s that is not halfway between two codes is at least
// 2^-10 away from it (x has 8 significant bits and s has 4; close to a halfway point x
// is above s / 4, so x and s times it are multiples of 2^-6 of s's last place, of which s
// has at most 15), so rounding x r to a multiple of 2^-12 moves halfway points back in
// place and nothing else past them; the second rounding, to even, is the code.
__global__ void __launch_bounds__(kWarps * 32) kv4_write_kernel(const Kv4Params P) {
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  if (i >= P.n) return;
  const uint4* xr = reinterpret_cast<const uint4*>(P.x + i * P.stride) + lane;
  const int64_t slot = __ldg(P.slot + i);
  const uint4 v[2] = {__ldg(xr), __ldg(xr + 32)};
  uint4 rope = make_uint4(0, 0, 0, 0);
  if (lane < 8) rope = __ldg(xr + 64);
  if (slot < 0) return;
  if (slot >= P.rows) {
    if (lane == 0) atomicOr(P.err, kErrBadIndex);
    return;
  }
  uint32_t amax[2];  // |x| as bf16 bits order like integers; both groups of the lane
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t m = 0x7fff7fffu;
    amax[h] = __vmaxu2(__vmaxu2(v[h].x & m, v[h].y & m), __vmaxu2(v[h].z & m, v[h].w & m));
    amax[h] = max(amax[h] & 0xffffu, amax[h] >> 16);
  }
  const bool odd = lane & 1;
  uint32_t a = odd ? amax[0] : amax[1];
  a = max(__shfl_xor_sync(0xffffffffu, a, 1), odd ? amax[1] : amax[0]);
  const bool ok = a < 0x7f80u;  // no NaN, no infinity
  const uint32_t u = ok ? scale_byte(__uint_as_float(a << 16)) : 255u;
  const float r = ok ? __frcp_rn(__uint_as_float((u << 20) + (112u << 23))) : 0.f;
  const float other = __shfl_xor_sync(0xffffffffu, r, 1);
  uint8_t* dst = P.kv4 + slot * kKv4Row;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float rh = odd == (h == 1) ? r : other;
    const uint32_t w[4] = {v[h].x, v[h].y, v[h].z, v[h].w};
    uint32_t c = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)  // dims 2k and 2k+1: nibbles k and 4 + k
      c |= (code(bf16lo(w[k]), rh) | (code(bf16hi(w[k]), rh) << 16)) << (4 * k);
    reinterpret_cast<uint32_t*>(dst)[h * 32 + lane] = rh == 0.f ? 0u : c;
  }
  dst[kKv4Scales + (odd ? 16 : 0) + (lane >> 1)] = static_cast<uint8_t>(u);
  if (lane < 8) reinterpret_cast<uint4*>(dst + kKv4Rope)[lane] = rope;
}

// A warp per row, 8 dims of each half per lane, as above.
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
  uint4* dst = reinterpret_cast<uint4*>(P.out + i * P.stride) + lane;
  uint4 o[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)}, rope = o[0];
  if (slot >= 0) {
    const uint8_t* src = P.kv4 + slot * kKv4Row;
    const uint32_t* w = reinterpret_cast<const uint32_t*>(src) + lane;
    const uint8_t* u = src + kKv4Scales + (lane >> 1);
    const uint32_t w0 = w[0], w1 = w[32], u0 = u[0], u1 = u[16];
    if (lane < 8) rope = *reinterpret_cast<const uint4*>(src + kKv4Rope + lane * 16);
    o[0] = kv4_codes8(w0, kv4_scale(u0));
    o[1] = kv4_codes8(w1, kv4_scale(u1));
  }
  dst[0] = o[0];
  dst[32] = o[1];
  if (lane < 8) dst[64] = rope;
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
