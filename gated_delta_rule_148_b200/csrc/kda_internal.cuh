// Internal declarations shared by the translation units of libkda.so.
#pragma once

#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "../../include/kda.h"

namespace kda {

// Bits latched in the per-device error word.
enum : unsigned {
  ERR_BIT_CHECK = 1u,     // device-side argument check failed
  ERR_BIT_TIMEOUT = 2u,   // a bounded wait ran out
};

// Per-sequence span of positions a prefill kernel processes: [begin, end)
// in packed rows.  Rows of the sequence outside the span are edge pads.
struct SeqSpan {
  int begin;
  int end;
  int seq_begin;   // cu[b]
  int pad_inside;  // 1 if a pad sits strictly inside [begin, end)
};

struct PrefillParams {
  int num_seqs, N, H, dk, dv, chunk;
  const void *q, *k, *v;
  const float *log_alpha, *beta;
  const int32_t *cu;
  const uint8_t *mask;
  const float *init_state;
  void *o;
  float *final_state;
  const SeqSpan *spans;   // NULL: spans are [cu[b], cu[b+1])
  unsigned *err;          // device error word
  int gate_head;          // 1: log_alpha is [N, H] (one gate per token and head)
  long long wait_cycles;  // limit of every bounded device wait
  int fault;              // test faults (FAULT_*), 0 in normal use
  unsigned *site;         // device word: code of the first bounded wait that ran out
};

// Faults a test can plant with kda_debug_set_fault() to exercise the bounded
// waits; none of them touches memory out of bounds.
enum : int {
  FAULT_STARVE_STATE_LOADS = 1,   // the state pass issues no item loads: its waits run out
};
constexpr long long kDefaultWaitCycles = 4000000000LL;   // ~2 s at 1.9 GHz

struct DecodeParams {
  int B, H, dk, dv;
  const void *q, *k, *v;
  const float *log_alpha, *beta;
  const uint8_t *mask;
  float *state;
  void *o;
  unsigned *err;
  int gate_head;          // 1: log_alpha is [B, H]
};

struct ConvParams {
  int num_seqs, N, D, W;
  const void *x;
  const float *weight, *bias;
  const int32_t *cu;
  const uint8_t *mask;
  const float *state_in;
  float *state_out;
  void *y;
  unsigned *err;
};

struct BackwardParams {
  int num_seqs, N, H, dk, dv;
  const void *q, *k, *v;
  const float *log_alpha, *beta;
  const int32_t *cu;
  const uint8_t *mask;
  const float *init_state;
  const float *d_o, *d_final_state;
  float *gq, *gk, *gv, *gla, *gbeta, *g_init_state;
  void *ws;               // chunk index, per-chunk quantities, states at chunk starts and ends
  unsigned *err;
  int gate_head;
};

// Linear attention with a decay for each head: prefill and (d_o ..) its backward pass.
struct LinearParams {
  int num_seqs, N, H, Hk, dk, dv;
  const void *q, *k, *v;
  const float *log_alpha;
  const int32_t *cu;
  const uint8_t *mask;
  const float *init_state;
  void *o;
  float *final_state;
  int decay_head;         // 1: log_alpha is [H] (a constant of the head)
  void *ws;               // segment table, states at segment starts, ...
  unsigned *err;
  long long wait_cycles;  // limit of every bounded device wait
  unsigned *site;         // device word: code of the first bounded wait that ran out
  const void *d_o;
  const float *d_final;
  void *gq, *gk, *gv;
  float *gla, *g_init;
};

struct LinearDecodeParams {
  int B, H, Hk, dk, dv;
  const void *q, *k, *v;
  const float *log_alpha;
  const uint8_t *mask;
  float *state;
  void *o;
  unsigned *err;
  int decay_head;         // 1: log_alpha is [H]
};

struct NormParams {
  long long rows;
  int D, group;
  const void *x, *residual;
  const float *weight;
  float eps;
  void *y;
  float *scale;
  void *residual_out;
  unsigned *err;
};

struct NormBackwardParams {
  long long rows;
  int D;
  const void *x, *dy, *dr;
  const float *weight;
  float eps;
  void *dx;
  float *dw, *part;       // part: one row of partial sums per block
  unsigned *err;
};

// Launchers (return a CUDA error code; argument checks happen before).
cudaError_t launch_prefill_prepass(const PrefillParams &p, bool bf16, SeqSpan *spans,
                                   cudaStream_t s);
cudaError_t launch_prefill_simt(const PrefillParams &p, bool bf16, cudaStream_t s);
cudaError_t launch_prefill_tc(const PrefillParams &p, cudaStream_t s);  // may return
                                                                          // cudaErrorNotSupported
bool prefill_tc_supported(const PrefillParams &p, bool bf16);
bool prefill_split_supported(const PrefillParams &p, bool bf16);
size_t prefill_split_workspace(int N, int B, int H);
cudaError_t launch_prefill_split(const PrefillParams &p, SeqSpan *spans, void *ws, cudaStream_t s);
// The two-kernel path's chunk index and intra kernel alone (64-row items of every chunk and head).
cudaError_t launch_split_items(const PrefillParams &p, const SeqSpan *spans, int *cbase,
                               unsigned char *items, cudaStream_t s);
// Chunks of 128 or 256 rows: 64-row items merged into chunk items, then the state pass.
bool prefill_bigchunk_supported(const PrefillParams &p, bool bf16);
size_t prefill_bigchunk_workspace(int N, int B, int H, int chunk);
cudaError_t launch_prefill_bigchunk(const PrefillParams &p, SeqSpan *spans, void *ws, cudaStream_t s);
cudaError_t launch_decode(const DecodeParams &p, bool bf16, cudaStream_t s);
cudaError_t launch_short_conv(const ConvParams &p, bool bf16, cudaStream_t s);
size_t backward_workspace(int N, int B, int H, int dk, int dv);
cudaError_t launch_backward(const BackwardParams &p, bool bf16, cudaStream_t s);
size_t linear_prefill_workspace(const LinearParams &p, bool bf16);
cudaError_t launch_linear_prefill(const LinearParams &p, bool bf16, cudaStream_t s);
// bf16 inputs: tensor-core kernels (kda_linear_tc.cu).
size_t linear_prefill_tc_workspace(const LinearParams &p);
cudaError_t launch_linear_prefill_tc(const LinearParams &p, cudaStream_t s);
// States at the segments' starts (part) and their gradients at the segments' ends (rpart).
cudaError_t launch_linear_segment_states_tc(const LinearParams &p, const int *sbase, float *part, float *rpart, float *whole,
                                            size_t segs, cudaStream_t s);
// ... of the backward pass (kda_linear_backward_tc.cu); where the caller's sums over shared inputs find their
// terms: dq, dk per value head (null if none is shared), the decays' gradients per token.
size_t linear_backward_tc_workspace(const LinearParams &p);
cudaError_t launch_linear_backward_tc(const LinearParams &p, float **gq32, float **gk32, float **gla, cudaStream_t s);
size_t linear_backward_workspace(const LinearParams &p, bool bf16);
cudaError_t launch_linear_backward(const LinearParams &p, bool bf16, cudaStream_t s);
cudaError_t launch_linear_decode(const LinearDecodeParams &p, bool bf16, cudaStream_t s);
// cu_seqlens check and table of segments of lo .. hi chunks; states at segment starts (and gradients at their ends).
cudaError_t launch_linear_plan(const LinearParams &p, int *sbase, int chunk, int lo, int hi, int sms, int *order,
                               int *earlier, cudaStream_t s);
cudaError_t launch_linear_chain(const LinearParams &p, const int *sbase, float *part, float *rpart,
                                const float *whole, cudaStream_t s);
// out: 0 the type of x, 1 e4m3, 2 int8.
cudaError_t launch_norm(const NormParams &p, bool bf16, int out, cudaStream_t s);
size_t norm_backward_workspace(long long rows, int D);
cudaError_t launch_norm_backward(const NormBackwardParams &p, bool bf16, cudaStream_t s);

// ---------------------------------------------------------------- a call's kernels, one after another
// A kernel launched with launch_next may be placed on the SMs while the one before it still runs (its launch then costs
// nothing); it begins with after_previous(), which returns when that kernel is complete and its writes are visible.
// A call's first kernel is launched plainly, so that calls do not overlap.
__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <class... P, class... A>
cudaError_t launch_next(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, A &&...args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = block;
  c.dynamicSmemBytes = smem;
  c.stream = s;
  c.attrs = &attr;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, static_cast<P>(args)...);
}

// ---------------------------------------------------------------- helpers
__device__ __forceinline__ float bf16_to_f32(uint16_t h) {
  return __uint_as_float(((unsigned)h) << 16);
}

// To nearest even; NaN stays NaN.
__device__ __forceinline__ uint16_t f32_to_bf16_rne(float f) {
  uint16_t u;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(u) : "f"(f));
  return u;
}

template <bool BF16>
__device__ __forceinline__ float load_elem(const void *base, size_t idx) {
  if (BF16) return bf16_to_f32(reinterpret_cast<const uint16_t *>(base)[idx]);
  return reinterpret_cast<const float *>(base)[idx];
}

template <bool BF16>
__device__ __forceinline__ void store_elem(void *base, size_t idx, float val) {
  if (BF16) reinterpret_cast<uint16_t *>(base)[idx] = f32_to_bf16_rne(val);
  else reinterpret_cast<float *>(base)[idx] = val;
}

// Offset of log_alpha for (row, head h, channel c): [rows, H, dk] or, with a
// head-wise gate, [rows, H] (the same value for every channel).
__device__ __forceinline__ size_t la_index(size_t row, int h, int H, int dk, int c, int gate_head) {
  return gate_head ? row * H + h : (row * H + h) * dk + c;
}

// Records which bounded wait ran out first (codes listed with kda_debug_timeout_site()).
__device__ __forceinline__ void note_timeout(unsigned *site, unsigned code) {
  if (site) atomicCAS(site, 0u, code);
}

__device__ __forceinline__ bool device_error_latched(const unsigned *err) {
  return *reinterpret_cast<const volatile unsigned *>(err) != 0u;
}

// The same answer for every thread of the block, all of which ask.  The word can be set between two warps' looks at it
// (by another block whose wait ran out, by a call on another stream), and a block of which only some warps leave runs on
// without its barriers, its tensor memory or its tables.
__device__ __forceinline__ bool block_leaves(const unsigned *err) { return __syncthreads_or(device_error_latched(err)); }

}  // namespace kda
