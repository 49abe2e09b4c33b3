// kv_pages_copy: pages of the cache onto others (a fork's partly filled pages, a compaction).
//
// Bound by HBM: every byte is read once and written once.  2,048 pages of 64 tokens of 8 heads of 128 in
// bf16 with their digests (1,082 MB): 160 us, 6,760 GB/s of 6,791; 32 pages in FP8 4.8 us.
#include "common.cuh"
#include "launch.h"
#include "profile.h"

namespace dsa {

DSA_CHECK_WORD(page_copy_check_word)

namespace {

constexpr int kThreads = 256, kUnroll = 4;
constexpr int kChunk = kThreads * kUnroll * 16;   // bytes of an array that a CTA copies

// CTA x of a pair: chunk x / 2 of its keys (even x) or values; the first one also takes the
// scales and the digest.
__global__ void __launch_bounds__(kThreads) page_copy_kernel(const PageCopyArgs a) {
  const int per = 2 * a.chunks;
  const int i = blockIdx.x / per, x = blockIdx.x % per;
  grid_dep_wait();
  const int src = a.src[i], dst = a.dst[i];
  DSA_CHECK(src >= 0 && src < a.n_pages && dst >= 0 && dst < a.n_pages);
  if (src < 0 || src >= a.n_pages || dst < 0 || dst >= a.n_pages || src == dst) return;
  char *base = (x & 1) ? a.big[1] : a.big[0];
  const long long at = static_cast<long long>(x >> 1) * kChunk;
  const int pieces = static_cast<int>(min(static_cast<long long>(kChunk), a.big_bytes - at) / 16);
  const uint4 *from = reinterpret_cast<const uint4 *>(base + src * a.big_bytes + at);
  uint4 *to = reinterpret_cast<uint4 *>(base + dst * a.big_bytes + at);
  uint4 u[kUnroll];
#pragma unroll
  for (int k = 0; k < kUnroll; ++k)
    if (static_cast<int>(threadIdx.x) + k * kThreads < pieces) u[k] = __ldcs(from + threadIdx.x + k * kThreads);
#pragma unroll
  for (int k = 0; k < kUnroll; ++k)
    if (static_cast<int>(threadIdx.x) + k * kThreads < pieces) __stcs(to + threadIdx.x + k * kThreads, u[k]);
  if (x == 0) {
    // (16-byte pieces where every page of the array is aligned to them, else bytes)
    for (int s = 0; s < 4; ++s) {
      if (!a.small[s]) continue;
      const int n = a.small_bytes[s];
      const char *f = a.small[s] + static_cast<long long>(src) * n;
      char *t = a.small[s] + static_cast<long long>(dst) * n;
      if (n % 16 == 0 && reinterpret_cast<uintptr_t>(a.small[s]) % 16 == 0) {
        for (int k = threadIdx.x; k < n / 16; k += kThreads)
          reinterpret_cast<uint4 *>(t)[k] = reinterpret_cast<const uint4 *>(f)[k];
      } else {
        for (int k = threadIdx.x; k < n; k += kThreads) t[k] = f[k];
      }
    }
  }
}

}  // namespace

cudaError_t launch_page_copy(const PageCopyArgs &a0, cudaStream_t s) {
  PageCopyArgs a = a0;
  a.chunks = static_cast<int>((a.big_bytes + kChunk - 1) / kChunk);
  // at most 2^31 - 1 CTAs a launch: more pairs in several
  const int per = 2 * a.chunks, most = static_cast<int>(0x7fffffffll / per);
  for (int i = 0; i < a0.n; i += most) {
    a.src = a0.src + i;
    a.dst = a0.dst + i;
    a.n = a0.n - i < most ? a0.n - i : most;
    ProfScope ps("kv_pages_copy", s);
    const cudaError_t e = launch_pdl(page_copy_kernel, dim3(static_cast<unsigned>(a.n) * per), dim3(kThreads), 0, s, a);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace dsa
