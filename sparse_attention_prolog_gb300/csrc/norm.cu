// Residual addition and RMS norm with a bf16 and/or int8 output
// (dsa_add_rmsnorm).  RMSNorm as in the MLA Prolog, the quantiser as in
// [V4-TileLang §Activation Quantization] steps 1-3.
//
// A row is read once, kept in registers in fp32 (as h, then as z), and written
// once; between lie two reductions over the row, of h^2 and of max |z|.  So the
// kernel moves what it cannot do without, and is bound by HBM when there are
// rows enough and by the launch, one trip to memory and the two reductions when
// there are few.  16384 rows of 7168 with a bf16 residual: y 138 us (6.83 TB/s, a
// copy's rate), y and codes 165 us (6.41 TB/s; the quantiser's instructions beside
// the loads), both with an fp32 residual 228 us (6.70 TB/s); 8 such rows 2.4 to 2.8
// and 3.9 us.
#include <algorithm>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "dsa_internal.h"
#include "dsa_ptx.cuh"

namespace dsa {
namespace {

constexpr int kMaxChunks = 4;  // 8-element chunks of a row that a thread holds

struct NormParams {
  dsa_add_rmsnorm_args a;
  int row_threads;  // threads of a row: 8, 16 or 32 (several rows a CTA), or the whole CTA
  float inv_d;
};

__device__ __forceinline__ float max_abs_nan(float m, float v) {
  // as whole numbers: |v| in order, and a NaN above every number
  return __uint_as_float(max(__float_as_uint(m), __float_as_uint(v) & 0x7fffffffu));
}

// Sum or maximum over the n threads of a row; `part` holds a value per warp of the CTA's.
template <bool kMax>
__device__ __forceinline__ float row_reduce(float v, int n, float* part) {
  auto join = [](float x, float y) { return kMax ? max_abs_nan(x, y) : x + y; };
#pragma unroll
  for (int o = 16; o; o >>= 1)
    if (o < n) v = join(v, __shfl_xor_sync(0xffffffffu, v, o));
  if (n <= 32) return v;
  const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) part[warp] = v;
  __syncthreads();
  v = lane < warps ? part[lane] : 0.f;
#pragma unroll
  for (int o = 16; o; o >>= 1) v = join(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

template <bool kFp16>
__device__ __forceinline__ float2 pair_of(uint32_t w) {
  if (kFp16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// The code of z: rint of the fp32 quotient, in [-127, 127].
__device__ __forceinline__ uint32_t code_of(float z, float s) {
  return static_cast<uint32_t>(__float2int_rn(fminf(fmaxf(z / s, -127.f), 127.f))) & 0xffu;
}

// The codes of 8 values.  A division costs as much as the rest of an element: t = z (1/s)
// is within 127 * 2^-22 < 2^-14 of z / s, so its nearest whole number is the quotient's
// unless t lies that near to a tie; then all 8 are divided.  Adding 1.5 * 2^23 rounds to a
// whole number, ties to even, and leaves it in the low byte.  |z| <= 127 s (1 + 2^-23):
// nothing has to be clamped.
__device__ __forceinline__ uint2 codes_of(const float (&z)[8], float s, float r) {
  constexpr float kRound = 12582912.f;
  uint32_t c[8];
  bool near = !(s > 1e-30f);  // (1 / s would leave fp32's range)
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = z[i] * r, u = t + kRound;
    near |= fabsf(fabsf(t - (u - kRound)) - 0.5f) < 1.f / 16384;
    c[i] = __float_as_uint(u);
  }
  if (near)
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = code_of(z[i], s);
  auto four = [&](int i) {
    return __byte_perm(__byte_perm(c[i], c[i + 1], 0x0040), __byte_perm(c[i + 2], c[i + 3], 0x0040), 0x5410);
  };
  return make_uint2(four(0), four(4));
}

// Rows whose arrays lie at any alignment.  A thread's 8 elements begin at e0 of the row
// (which may be below 0 in its first chunk); elements outside [0, D) are neither read nor
// written.  Inside a row the aligned vectors around the 8 are read and shifted; what they
// have beside them is of the same row.
__device__ __forceinline__ bool inside(int e0, int D) { return e0 >= 8 && e0 + 16 <= D; }
template <int kWords>
__device__ __forceinline__ void shift_words(uint32_t (&w)[kWords], int words) {  // down by 0 to 3
  if (words & 2)
#pragma unroll
    for (int i = 0; i < kWords - 2; ++i) w[i] = w[i + 2];
  if (words & 1)
#pragma unroll
    for (int i = 0; i < kWords - 1; ++i) w[i] = w[i + 1];
}
__device__ __forceinline__ uint4 any_8x16(const uint16_t* row, int e0, int D) {
  if (inside(e0, D)) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(row + e0);
    const uint4* v = reinterpret_cast<const uint4*>(at & ~static_cast<uintptr_t>(15));
    const uint4 x = v[0];
    if ((at & 15) == 0) return x;
    const uint4 y = v[1];
    uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    shift_words(w, static_cast<int>(at >> 2) & 3);
    if (at & 2)
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = e0 + 2 * i;
    w[i] = (e >= 0 && e < D ? row[e] : 0u) | (e + 1 >= 0 && e + 1 < D ? static_cast<uint32_t>(row[e + 1]) << 16 : 0u);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void any_8x32(const float* row, int e0, int D, float (&f)[8]) {
  if (inside(e0, D)) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(row + e0);
    const uint4* v = reinterpret_cast<const uint4*>(at & ~static_cast<uintptr_t>(15));
    const uint4 x = v[0], y = v[1], z = (at & 15) == 0 ? make_uint4(0, 0, 0, 0) : v[2];
    uint32_t w[12] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w, z.x, z.y, z.z, z.w};
    shift_words(w, static_cast<int>(at >> 2) & 3);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = e0 + i >= 0 && e0 + i < D ? row[e0 + i] : 0.f;
}
// 8 values of kBytes each, in words: by vectors where they are whole and aligned, 16-bit
// ones by words where they are whole.
template <int kBytes>
__device__ __forceinline__ void put_8(void* row, int e0, int D, const uint32_t* w) {
  uint8_t* at = static_cast<uint8_t*>(row) + static_cast<int64_t>(e0) * kBytes;
  constexpr int kAlign = kBytes == 1 ? 8 : 16;
  if (e0 >= 0 && e0 + 8 <= D && reinterpret_cast<uintptr_t>(at) % kAlign == 0) {
    if (kBytes == 1) {
      *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int i = 0; i < kBytes / 2; ++i)
        reinterpret_cast<uint4*>(at)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
    return;
  }
  if (kBytes == 2 && e0 >= 0 && e0 + 8 <= D) {
    if (reinterpret_cast<uintptr_t>(at) % 4 == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) reinterpret_cast<uint32_t*>(at)[i] = w[i];
    } else {
      *reinterpret_cast<uint16_t*>(at) = static_cast<uint16_t>(w[0]);
#pragma unroll
      for (int i = 0; i < 3; ++i) *reinterpret_cast<uint32_t*>(at + 2 + 4 * i) = __funnelshift_r(w[i], w[i + 1], 16);
      *reinterpret_cast<uint16_t*>(at + 14) = static_cast<uint16_t>(w[3] >> 16);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (e0 + i < 0 || e0 + i >= D) continue;
    if (kBytes == 1) at[i] = static_cast<uint8_t>(w[i / 4] >> (i % 4 * 8));
    else if (kBytes == 2) reinterpret_cast<uint16_t*>(at)[i] = static_cast<uint16_t>(w[i / 2] >> (i % 2 * 16));
    else reinterpret_cast<uint32_t*>(at)[i] = w[i];
  }
}

// kVec: D and every row allow vectors of 8 elements.  Else chunks begin where the row of
// y (or of the codes) is aligned, and what lies otherwise is shifted into place
// (y and codes of 16384 rows of 7167: 277 us in place of 165, element by element 548; of
// 7168 with rows of x and the residual 7169 apart 372, whose stores of the residual go by
// words).
template <int kChunks, int kThreads, bool kVec, bool kFp16, bool kRes32>
__global__ void __launch_bounds__(kThreads) add_rmsnorm_kernel(const NormParams P) {
  __shared__ float part[2][32];
  const dsa_add_rmsnorm_args& a = P.a;
  const int n = P.row_threads;
  const int me = n <= 32 ? threadIdx.x % n : threadIdx.x;
  const long long at = n <= 32 ? static_cast<long long>(blockIdx.x) * (blockDim.x / n) + threadIdx.x / n : blockIdx.x;
  griddep_wait();
  const int D = at < a.T ? a.D : 0;  // (a row past the last: its threads only take part in the reductions)
  const long long row = min(at, static_cast<long long>(a.T) - 1);
  const bool res = a.residual != nullptr;
  const uint16_t* x = static_cast<const uint16_t*>(a.x) + row * a.x_stride;
  const uint8_t* rin = static_cast<const uint8_t*>(a.residual) + row * a.residual_stride * (kRes32 ? 4 : 2);
  uint8_t* rout = static_cast<uint8_t*>(a.residual_out) + row * a.residual_out_stride * (kRes32 ? 4 : 2);

  // (of a row that needs the last chunk that the threads have, none is left for a skew)
  const int skew = kVec || a.D + 7 > P.row_threads * kChunks * 8 ? 0
                   : a.y ? static_cast<int>(reinterpret_cast<uintptr_t>(a.y + row * a.D) >> 1) & 7
                         : static_cast<int>(reinterpret_cast<uintptr_t>(a.codes + row * a.D)) & 7;

  float h[kChunks][8];
  if (kVec) {
    uint4 xv[kChunks];
    float4 r0[kChunks], r1[kChunks];  // 8 fp32, or 8 bf16 in r0
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      const int e = (me + k * n) * 8;
      const bool on = e < D;
      xv[k] = on ? __ldcs(reinterpret_cast<const uint4*>(x + e)) : make_uint4(0, 0, 0, 0);
      r0[k] = r1[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (res && on) {
        r0[k] = __ldcs(reinterpret_cast<const float4*>(rin + static_cast<size_t>(e) * (kRes32 ? 4 : 2)));
        if (kRes32) r1[k] = __ldcs(reinterpret_cast<const float4*>(rin + static_cast<size_t>(e) * 4 + 16));
      }
    }
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      const int e = (me + k * n) * 8;
      const uint32_t w[4] = {xv[k].x, xv[k].y, xv[k].z, xv[k].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = pair_of<kFp16>(w[i]);
        h[k][2 * i] = f.x;
        h[k][2 * i + 1] = f.y;
      }
      if (!res) continue;
      const float b[8] = {r0[k].x, r0[k].y, r0[k].z, r0[k].w, r1[k].x, r1[k].y, r1[k].z, r1[k].w};
      if (kRes32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[k][i] += b[i];
        if (e < D) {
          float4* o = reinterpret_cast<float4*>(rout + static_cast<size_t>(e) * 4);
          o[0] = make_float4(h[k][0], h[k][1], h[k][2], h[k][3]);
          o[1] = make_float4(h[k][4], h[k][5], h[k][6], h[k][7]);
        }
      } else {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = pair_of<false>(__float_as_uint(b[i]));
          o[i] = bf16_pair(h[k][2 * i] + f.x, h[k][2 * i + 1] + f.y);
          const float2 s = pair_of<false>(o[i]);
          h[k][2 * i] = s.x;
          h[k][2 * i + 1] = s.y;
        }
        if (e < D) *reinterpret_cast<uint4*>(rout + static_cast<size_t>(e) * 2) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  } else {
    uint4 xv[kChunks], rv[kChunks];
    float rf[kRes32 ? kChunks : 1][8];
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      const int e0 = (me + k * n) * 8 - skew;
      xv[k] = any_8x16(x, e0, D);
      if (res && !kRes32) rv[k] = any_8x16(reinterpret_cast<const uint16_t*>(rin), e0, D);
      if (res && kRes32) any_8x32(reinterpret_cast<const float*>(rin), e0, D, rf[kRes32 ? k : 0]);
    }
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      const int e0 = (me + k * n) * 8 - skew;
      const uint32_t w[4] = {xv[k].x, xv[k].y, xv[k].z, xv[k].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = pair_of<kFp16>(w[i]);
        h[k][2 * i] = f.x;
        h[k][2 * i + 1] = f.y;
      }
      if (!res) continue;
      if (kRes32) {
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          h[k][i] += rf[kRes32 ? k : 0][i];
          o[i] = __float_as_uint(h[k][i]);
        }
        put_8<4>(rout, e0, D, o);
      } else {
        const uint32_t v[4] = {rv[k].x, rv[k].y, rv[k].z, rv[k].w};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = pair_of<false>(v[i]);
          o[i] = bf16_pair(h[k][2 * i] + f.x, h[k][2 * i + 1] + f.y);
          const float2 t = pair_of<false>(o[i]);
          h[k][2 * i] = t.x;
          h[k][2 * i + 1] = t.y;
        }
        put_8<2>(rout, e0, D, o);
      }
    }
  }

  float sum = 0.f;
#pragma unroll
  for (int k = 0; k < kChunks; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fmaf(h[k][i], h[k][i], sum);
  sum = row_reduce<false>(sum, n, part[0]);
  const float r = 1.f / sqrtf(sum * P.inv_d + a.eps);

  float top = 0.f;
#pragma unroll
  for (int k = 0; k < kChunks; ++k) {
    if (kVec) {
      const int e = (me + k * n) * 8;
      if (e >= D) continue;
      const float4 g0 = __ldg(reinterpret_cast<const float4*>(a.gamma + e));
      const float4 g1 = __ldg(reinterpret_cast<const float4*>(a.gamma + e) + 1);
      const float g[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) h[k][i] = h[k][i] * r * g[i];
      if (a.y)
        *reinterpret_cast<uint4*>(a.y + row * a.D + e) =
            make_uint4(bf16_pair(h[k][0], h[k][1]), bf16_pair(h[k][2], h[k][3]), bf16_pair(h[k][4], h[k][5]),
                       bf16_pair(h[k][6], h[k][7]));
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max_abs_nan(top, h[k][i]);
    } else {
      const int e0 = (me + k * n) * 8 - skew;
      if (e0 >= D) continue;
      float g[8];
      any_8x32(a.gamma, e0, D, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        h[k][i] = h[k][i] * r * g[i];
        if (e0 + i >= 0 && e0 + i < D) top = max_abs_nan(top, h[k][i]);
      }
      const uint32_t o[4] = {bf16_pair(h[k][0], h[k][1]), bf16_pair(h[k][2], h[k][3]), bf16_pair(h[k][4], h[k][5]),
                             bf16_pair(h[k][6], h[k][7])};
      if (a.y) put_8<2>(a.y + row * a.D, e0, D, o);
    }
  }
  if (a.codes == nullptr) return;
  top = row_reduce<true>(top, n, part[1]);
  float s = top / 127.f;
  const bool fine = s > 0.f && s < __int_as_float(0x7f800000);
  if (a.round_scale && fine) {
    int e;
    const float m = frexpf(s, &e);  // s = m * 2^e, m in [0.5, 1)
    s = ldexpf(1.f, m == 0.5f ? e - 1 : e);
  }
  const float inv_s = 1.f / s;
  if (me == 0 && D > 0) a.code_scale[row] = s;
#pragma unroll
  for (int k = 0; k < kChunks; ++k) {
    if (kVec) {
      const int e = (me + k * n) * 8;
      if (e >= D) continue;
      *reinterpret_cast<uint2*>(a.codes + row * a.D + e) = fine ? codes_of(h[k], s, inv_s) : make_uint2(0u, 0u);
    } else {
      const int e0 = (me + k * n) * 8 - skew;
      if (e0 >= D) continue;
      const uint2 c = fine ? codes_of(h[k], s, inv_s) : make_uint2(0u, 0u);
      const uint32_t o[2] = {c.x, c.y};
      put_8<1>(a.codes + row * a.D, e0, D, o);
    }
  }
}

template <int kChunks, int kThreads, bool kVec>
auto pick(bool fp16, bool res32) {
  return fp16 ? (res32 ? add_rmsnorm_kernel<kChunks, kThreads, kVec, true, true>
                       : add_rmsnorm_kernel<kChunks, kThreads, kVec, true, false>)
              : (res32 ? add_rmsnorm_kernel<kChunks, kThreads, kVec, false, true>
                       : add_rmsnorm_kernel<kChunks, kThreads, kVec, false, false>);
}

// The instance for n threads of `per` chunks each.  Its bound on the threads leaves it as
// many registers as they may have (1024: 64 each, 544: 120, fewer: 255): an instance is for
// the thread counts that need no lower bound.  Two chunks each: up to 128 threads (rows of
// up to 256 chunks, where there are many) or 513 and more (rows of over 1024 chunks).  Four:
// 65 to 512 threads (many rows of up to 2048 chunks), or 513 and more (longer rows; up to
// 544 takes in an unaligned row of 16384, which has a chunk more for its skew).
template <bool kVec>
auto pick_size(int per, int n, bool f, bool r) {
  return per == 1   ? pick<1, 1024, kVec>(f, r)
         : per == 2 ? (n <= 128 ? pick<2, 128, kVec>(f, r) : pick<2, 1024, kVec>(f, r))
         : n <= 256 ? pick<4, 256, kVec>(f, r)
         : n <= 544 ? pick<4, 544, kVec>(f, r)
                    : pick<4, 1024, kVec>(f, r);
}

}  // namespace

int launch_add_rmsnorm(const dsa_add_rmsnorm_args& a, cudaStream_t s) {
  const size_t rsize = a.residual_fp32 ? 4 : 2;
  const bool vec = a.D % 8 == 0 && a.x_stride % 8 == 0 && aligned(a.x, 16) && aligned(a.gamma, 16) &&
                   aligned(a.residual, 16) && aligned(a.residual_out, 16) && a.residual_stride * rsize % 16 == 0 &&
                   a.residual_out_stride * rsize % 16 == 0 && aligned(a.y, 16) && aligned(a.codes, 8);
  const int chunks = vec ? a.D / 8 : std::min((a.D + 14) / 8, kMaxChunks * 1024);  // (room for a skew, but for the longest rows)
  // Threads of a row.  Few rows: one chunk each, so that a row is one trip to memory.  Rows
  // enough to fill the SMs: four chunks each, or two of shorter rows, so that more rows are
  // on their way while others reduce (y and codes of 16384 rows: 7168 wide 225 us with one
  // chunk each and a division a code, 165 with four and the codes as above; 2048 wide 59 and
  // 51 with two, 1536 wide 45 and 40; 512 wide no difference).  Rows of up to 32 chunks: 8
  // to 32 threads, several rows a CTA.
  const bool many = a.T > 4 * sm_count();
  int per = 1;
  while ((chunks + per - 1) / per > 1024) per *= 2;
  if (many && chunks > 64 && chunks <= 2048) per = chunks > 256 ? 4 : 2;
  int n = ((chunks + per - 1) / per + 31) / 32 * 32;
  if (n == 32) n = chunks <= 8 ? 8 : chunks <= 16 ? 16 : 32;
  const int rows = n <= 32 ? 256 / n : 1;
  NormParams P{a, n, 1.f / static_cast<float>(a.D)};
  const bool f = a.x_fp16, r = a.residual_fp32;
  auto kern = vec ? pick_size<true>(per, n, f, r) : pick_size<false>(per, n, f, r);
  static_assert(kMaxChunks * 8 * 1024 >= 32768, "the longest row fits a CTA");
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>((static_cast<long long>(a.T) + rows - 1) / rows));
  cfg.blockDim = dim3(n * rows);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, kern, P));
}

}  // namespace dsa
