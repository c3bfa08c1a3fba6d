// Linear attention with a decay for each head: what its kernels share.
//
//   S_t = a_t S_{t-1} + k_t v_t^T,  o_t = S_t^T q_t,  a_t = exp(log_alpha_t)
// A sequence is cut into chunks of C tokens and segments of `per` chunks.  With b the running
// sum of log2 a inside a chunk (inclusive) and S the state at the chunk's start,
//   O = tril(Q K^T o 2^{b_t - b_s}) V + Diag(2^b) Q S,   S' = 2^{b_C} S + (Diag(2^{b_C - b}) K)^T V.
// Every exponent is <= 0, so nothing overflows for any log_alpha <= 0.  b is summed in 64 bits
// and kept as hi + lo floats: after a strong decay b is large against the differences
// that still matter, and a float's step there would show in the fp32 outputs.  A step below
// 2^-400 counts as 2^-400: both are 0 against any fp32 value, and the sum keeps its digits.
#pragma once

#include <atomic>

#include "kda_internal.cuh"

namespace kda {
namespace lin {

__host__ __device__ inline size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// Segment tables: sbase[b] = segments of the sequences before b (b <= num_seqs); behind them the segments in the order
// in which blocks take them: number (their states' place, in the sequences' order), rows [begin, end), and the sequence
// with a bit that tells its last segment.
struct alignas(16) Segment {
  int id, begin, end, of;
  __device__ __forceinline__ bool last() const { return of & 1; }
  __device__ __forceinline__ int seq() const { return of >> 1; }
};
// Chunks in a segment at most, where segments have more than one: the plan counts the lengths in shared memory.
constexpr int kMaxPer = 64;
// In place of the number of segments, sbase[num_seqs]: the plan found the call's cu_seqlens invalid, or an error latched.
// The word is the call's own, where the library's error word can be read and cleared (by kda_get_device_status on another
// stream) between the plan and the kernels that index by its tables.
constexpr int kRefused = -1;
// Asked by every thread of the block, with the same answer for all, first of all in the kernels behind a plan.
__device__ __forceinline__ bool call_ended(const LinearParams &p, const int *sbase) {
  return __syncthreads_or(device_error_latched(p.err) | (sbase[p.num_seqs] == kRefused));      // both on their way at once
}
inline size_t max_segments(int N, int B, int tokens) { return (size_t)N / tokens + (size_t)B; }
inline size_t table_bytes(int B, size_t segs) { return align256((size_t)(B + 1) * 4) + align256(segs * sizeof(Segment)); }
__device__ __forceinline__ const Segment *segment_table(const int *sbase, int num_seqs) {
  return reinterpret_cast<const Segment *>(sbase + align256((size_t)(num_seqs + 1) * 4) / 4);
}
__device__ __forceinline__ Segment locate(const int *sbase, int num_seqs, int seg) {
  const int4 x = __ldg(reinterpret_cast<const int4 *>(segment_table(sbase, num_seqs) + seg));
  return Segment{x.x, x.y, x.z, x.w};
}

// Lets a kernel have `bytes` of dynamic shared memory: once per device, since the call costs as much as a launch.
template <auto Kernel>
cudaError_t allow_smem(size_t bytes) {
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

__device__ __forceinline__ double shfl_up_f64(double x, int o) {
  return __hiloint2double(__shfl_up_sync(0xFFFFFFFFu, __double2hiint(x), o),
                          __shfl_up_sync(0xFFFFFFFFu, __double2loint(x), o));
}
__device__ __forceinline__ double shfl_f64(double x, int lane) {
  return __hiloint2double(__shfl_sync(0xFFFFFFFFu, __double2hiint(x), lane),
                          __shfl_sync(0xFFFFFFFFu, __double2loint(x), lane));
}

// log2 of a decay: a step below 2^-400 counts as 2^-400, NaN stays NaN (a maximum would drop it, and a broken gate pass
// for a reset).
__device__ __forceinline__ double log2_step(float log_alpha) {
  const double x = (double)log_alpha * 1.4426950408889634074;
  return x < -400.0 ? -400.0 : x;
}
// log2 of token `pos`'s decay for head h; 0 past the end and at pads.
__device__ __forceinline__ double log2_decay(const float *la, int decay_head, const uint8_t *mask, int pos, int end,
                                             int h, int H) {
  if (pos >= end || (mask != nullptr && mask[pos] == 0)) return 0.0;
  return log2_step(la[decay_head ? (size_t)h : (size_t)pos * H + h]);
}

}  // namespace lin
}  // namespace kda
