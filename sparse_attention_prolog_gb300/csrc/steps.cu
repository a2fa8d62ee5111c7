// Step maps: the block table and the token maps of a step from the lengths of
// its requests (dsa_step_maps).
//
// Two running sums over the requests (tokens, new pages) decide everything: a
// token finds its request, and a new page its own, by a binary search of them.
// B is at most 8192, so every CTA forms both sums itself in shared memory (one
// read of 8 B bytes, from L2 after the first CTA, held in registers) and then
// fills its own stretch of the tables; nothing passes between CTAs, and no page
// entry that this step writes is read (a new page is looked up in the free list).
// What bounds it is the launch and three dependent trips to memory: lengths, page
// entries, stores.  In a graph 32 requests of a token take 2.9 us, 300 with five
// prompt chunks 4.6, 4096 with forty 8.2 (divisions by a page size that is a power
// of two: 3.0, 4.8 and 9.1; lengths read again in every pass and two tokens a
// thread as well: 3.6, 6.0 and 12.0).
#include <algorithm>
#include <cuda_runtime.h>
#include "dsa_internal.h"
#include "dsa_ptx.cuh"

namespace dsa {
namespace {

constexpr int kMaxRequests = 8192;
constexpr size_t shared_bytes(int requests) { return (4 * static_cast<size_t>(requests) + 2) * sizeof(int); }

struct Sums {  // of a request's tokens and new pages
  long long tok, page;
};

__device__ __forceinline__ Sums warp_inclusive(Sums v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, v.tok, o), p = __shfl_up_sync(0xffffffffu, v.page, o);
    if (lane >= o) {
      v.tok += t;
      v.page += p;
    }
  }
  return v;
}

// The last i of [0, n) with run[i] <= v (run[0] = 0 <= v): of the requests that
// begin at the same count, the one that is not empty.
__device__ __forceinline__ int owner(const int* run, int n, int v) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (run[mid] <= v) lo = mid; else hi = mid;
  }
  return lo;
}

// kEach: requests of a thread, which follow one another (read once, in registers).
template <int kEach>
__global__ void __launch_bounds__(1024) step_maps_kernel(const dsa_step_maps_args P, uint32_t* err) {
  extern __shared__ int run[];  // tokens before request b [B + 1], pages before it [B + 1], cached [B], pages held [B]
  __shared__ Sums warp_sum[32];
  __shared__ int cut_sh;       // the first request that is not served
  __shared__ int total_sh[2];  // tokens and pages of those that are
  int* run_tok = run;
  int* run_page = run + P.B + 1;
  int* cached = run_page + P.B + 1;
  int* held = cached + P.B;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, threads = blockDim.x;
  if (tid == 0) cut_sh = P.B;
  griddep_wait();
  const int head = P.free_head == nullptr ? 0 : __ldg(P.free_head);
  const long long avail = head < 0 ? -1 : static_cast<long long>(P.n_free) - head;
  const long long most = static_cast<long long>(P.max_blocks) * P.block_size;
  const int b0 = tid * kEach;
  // whole pages in x rows, and pages that x rows reach into (a shift where pages are a power of two)
  const int shift = (P.block_size & (P.block_size - 1)) == 0 ? __ffs(P.block_size) - 1 : -1;
  auto whole = [&](int x) { return shift >= 0 ? x >> shift : x / P.block_size; };
  auto pages_of = [&](int x) {
    const int q = whole(x);
    return q + (q * P.block_size != x);
  };

  int c[kEach], f[kEach], old[kEach], fresh_pages[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const bool on = b0 + i < P.B;
    c[i] = on ? __ldg(P.cached + b0 + i) : 0;
    f[i] = on ? __ldg(P.fresh + b0 + i) : 0;
  }
  Sums own{0, 0};
  int first_bad = P.B;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    old[i] = fresh_pages[i] = 0;
    if (b0 + i >= P.B) continue;
    if (c[i] < 0 || f[i] < 0 || static_cast<long long>(c[i]) + f[i] > most) {  // lengths that cannot be served
      first_bad = min(first_bad, b0 + i);
      continue;
    }
    old[i] = pages_of(c[i]);
    fresh_pages[i] = pages_of(c[i] + f[i]) - old[i];
    own.tok += f[i];
    own.page += fresh_pages[i];
  }
  Sums inc = warp_inclusive(own, lane);
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    Sums w = lane < (threads >> 5) ? warp_sum[lane] : Sums{0, 0};
    w = warp_inclusive(w, lane);
    warp_sum[lane] = w;
  }
  __syncthreads();
  Sums at{inc.tok - own.tok, inc.page - own.page};  // before request b0
  if (warp > 0) {
    at.tok += warp_sum[warp - 1].tok;
    at.page += warp_sum[warp - 1].page;
  }
  {  // the first request whose running sums pass a limit
    Sums s = at;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      if (b0 + i >= first_bad) break;
      s.tok += f[i];
      s.page += fresh_pages[i];
      if (s.tok > P.T || s.page > avail) first_bad = b0 + i;
    }
  }
  if (first_bad < P.B) atomicMin(&cut_sh, first_bad);
  __syncthreads();
  const int cut = cut_sh;
  if (tid == 0 && cut == P.B) {
    const Sums all = warp_sum[31];
    total_sh[0] = static_cast<int>(all.tok);
    total_sh[1] = static_cast<int>(all.page);
  }
  if (b0 <= cut && cut < min(P.B, b0 + kEach)) {  // sums before the cut
    Sums s = at;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      if (b0 + i >= cut) break;
      s.tok += f[i];
      s.page += fresh_pages[i];
    }
    total_sh[0] = static_cast<int>(s.tok);
    total_sh[1] = static_cast<int>(s.page);
  }
  __syncthreads();
  const int tokens = total_sh[0], pages = total_sh[1];
  const bool writer = blockIdx.x == 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int b = b0 + i;
    if (b >= P.B) break;
    const bool on = b < cut;
    run_tok[b] = on ? static_cast<int>(at.tok) : tokens;
    run_page[b] = on ? static_cast<int>(at.page) : pages;
    cached[b] = c[i];
    held[b] = old[i];
    if (writer) {
      P.cu_tokens[b] = run_tok[b];
      P.kv_len[b] = on ? c[i] + f[i] : c[i];
    }
    if (on) {
      at.tok += f[i];
      at.page += fresh_pages[i];
    }
  }
  if (tid == 0) {
    run_tok[P.B] = tokens;
    run_page[P.B] = pages;
    if (writer) {
      P.cu_tokens[P.B] = tokens;
      P.counts[0] = tokens;
      P.counts[1] = head + pages;
      P.counts[2] = cut;
      if (cut < P.B) atomicOr(err, kErrBadIndex);
    }
  }
  __syncthreads();

  const int stride = gridDim.x * threads;  // (T and the pages end 2^20 below 2^31: the indexes stay inside)
  for (int p = blockIdx.x * threads + tid; p < pages; p += stride) {
    const int b = owner(run_page, P.B, p);
    const int j = held[b] + p - run_page[b];
    P.block_table[static_cast<size_t>(b) * P.max_blocks + j] = __ldg(P.free_pages + head + p);
  }
  const int pad_seq = tokens > 0 ? owner(run_tok, P.B, tokens - 1) : 0;
  for (int t = blockIdx.x * threads + tid; t < P.T; t += stride) {
    int seq = pad_seq, pos = 0;
    int64_t slot = -1;
    if (t < tokens) {
      seq = owner(run_tok, P.B, t);
      pos = cached[seq] + t - run_tok[seq];
      const int j = whole(pos);
      const int page = j < held[seq] ? P.block_table[static_cast<size_t>(seq) * P.max_blocks + j]
                                     : __ldg(P.free_pages + head + run_page[seq] + j - held[seq]);
      if (page >= 0)
        slot = static_cast<int64_t>(page) * P.block_size + (pos - j * P.block_size);
      else
        atomicOr(err, kErrBadIndex);
    }
    P.seq_of_token[t] = seq;
    P.pos[t] = pos;
    P.slot[t] = slot;
  }
  __threadfence();  // (a kernel two further on may read pos and seq_of_token without a wait)
}

}  // namespace

int launch_step_maps(const dsa_step_maps_args& a, cudaStream_t s) {
  uint32_t* err = error_word();
  if (!err) return DSA_ERR_CUDA;
  const int threads = a.B <= 256 ? 256 : 1024;
  const int each = a.B <= 1024 ? 1 : a.B <= 4096 ? 4 : 8;
  auto kern = each == 1 ? step_maps_kernel<1> : each == 4 ? step_maps_kernel<4> : step_maps_kernel<8>;
  // every CTA forms the sums again, so none is started for less than a token a thread
  const long long want = (static_cast<long long>(a.T) + threads - 1) / threads;
  const long long most = std::min(2ll * sm_count() * (1024 / threads), (1ll << 20) / threads);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(want < 1 ? 1 : want < most ? want : most));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = shared_bytes(a.B);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  static_assert(kMaxRequests == 8 * 1024, "requests of a CTA's threads");
  static_assert(shared_bytes(kMaxRequests) <= 200 * 1024 && shared_bytes(1024) <= 40 * 1024, "running sums");
  // What the kernel may ever ask for, not what this call does: the limit is the kernel's, and
  // a call of fewer requests in another host thread would lower it between here and the launch.
  if (each > 1 && cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(shared_bytes(1024 * each))) != cudaSuccess)
    return DSA_ERR_CUDA;
  return cuda_status(cudaLaunchKernelEx(&cfg, kern, a, err));
}

}  // namespace dsa
