// Root-mean-square norm of rows, with the residual's addition, an 8-bit output
// with scales, and the backward pass.
//
//   r = x + residual (rounded to the tensors' type: the residual stream's new value)
//   y = r * rsqrt(mean(r^2) + eps) * w
//   8 bits, per row or per group of 32, 64 or 128 columns:
//     scale = max(max|y|, 2^-100) / 448 (e4m3) or / 127 (int8),  y8 = round(y / scale)
//   backward, g = dy * w, c = rstd:
//     dr = c (g - r c^2 mean(r g)) [+ the gradient that reaches r along the residual]
//     dw = sum over rows of dy * r * c
//
// All of it is bound by HBM: every tensor is read once and written once.  A row belongs to
// TPR threads (8 lanes of a warp up to 1024 threads), each with VPT vectors of 8 columns
// that stay in registers between the statistic and the output, so there is one pass over
// the data and the only exchanges are the row sums (shuffles, and one word per warp through
// shared memory when a row spans warps).  What decides the rate is how many bytes a thread has
// in flight before its first exchange: four 16-byte loads of a tensor (VPT U = 4) in 64
// registers, so that four blocks of 256 threads share an SM, reach 5.2 - 6.4 TB/s of bf16 from 128 to
// 8192 columns (a copy: 6.0); one or two loads 3.0 - 4.7, eight loads (two blocks) 2.5 - 4.0.
// The backward pass keeps dw's columns in registers over all rows of a block and loads the next row
// while the sums of this one are exchanged: 16384 x 4096 bf16 118 -> 96 us (5.6 TB/s).
// The statistic, y and the sums of dw are fp32; r is rounded before the statistic, so
// that the backward pass, which reads the stored r, differentiates what was computed.
#include <cuda_fp8.h>

#include "kda_internal.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace norm {

constexpr float kTiny = 7.888609052210118e-31f;   // 2^-100: keeps 1 / scale finite for an all-zero group

// 8 consecutive elements as loaded: 16 bytes of bf16 or 32 bytes of fp32.
template <bool BF16> struct Raw { uint4 w[BF16 ? 1 : 2]; };

template <bool BF16>
__device__ __forceinline__ Raw<BF16> load8(const void *base, size_t vec) {
  const uint4 *p = reinterpret_cast<const uint4 *>(base) + vec * (BF16 ? 1 : 2);
  Raw<BF16> r;
  r.w[0] = __ldcs(p);
  if constexpr (!BF16) r.w[1] = __ldcs(p + 1);
  return r;
}
template <bool BF16>
__device__ __forceinline__ void unpack8(const Raw<BF16> &r, float (&f)[8]) {
  const uint32_t a[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
  if constexpr (BF16) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[2 * e] = __uint_as_float(a[e] << 16);
      f[2 * e + 1] = __uint_as_float(a[e] & 0xFFFF0000u);
    }
  } else {
    const uint32_t b[4] = {r.w[1].x, r.w[1].y, r.w[1].z, r.w[1].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[e] = __uint_as_float(a[e]);
      f[4 + e] = __uint_as_float(b[e]);
    }
  }
}
// Rounds to nearest even (bf16) or keeps (fp32) the 8 values.
template <bool BF16>
__device__ __forceinline__ Raw<BF16> pack8(const float (&f)[8]) {
  Raw<BF16> r;
  if constexpr (BF16) {
    r.w[0] = make_uint4(tc::pack_bf16x2(f[0], f[1]), tc::pack_bf16x2(f[2], f[3]),
                        tc::pack_bf16x2(f[4], f[5]), tc::pack_bf16x2(f[6], f[7]));
  } else {
    r.w[0] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    r.w[1] = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
  }
  return r;
}
template <bool BF16>
__device__ __forceinline__ void store8(void *base, size_t vec, const Raw<BF16> &r) {
  uint4 *p = reinterpret_cast<uint4 *>(base) + vec * (BF16 ? 1 : 2);
  p[0] = r.w[0];
  if constexpr (!BF16) p[1] = r.w[1];
}

// A NaN wins, so that it reaches the scale instead of being lost in an integer.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Sum (MAX: maximum) over a row's TPR threads of U values; every thread of the block calls it.
template <int TPR, int U, bool MAX>
__device__ __forceinline__ void row_reduce(float (&s)[U], float *red) {
#pragma unroll
  for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1)
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float x = __shfl_xor_sync(0xFFFFFFFFu, s[u], o);
      s[u] = MAX ? max_nan(s[u], x) : s[u] + x;
    }
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, w0 = warp & ~(W - 1);
    __syncthreads();              // the words of the last reduction have been read
    if (lane == 0)
#pragma unroll
      for (int u = 0; u < U; ++u) red[u * 32 + warp] = s[u];
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float x = red[u * 32 + w0];
#pragma unroll
      for (int i = 1; i < W; ++i) x = MAX ? max_nan(x, red[u * 32 + w0 + i]) : x + red[u * 32 + w0 + i];
      s[u] = x;
    }
  }
}

constexpr int OUT_SAME = 0, OUT_E4M3 = 1, OUT_I8 = 2;
__host__ __device__ constexpr int block_threads(int TPR) { return TPR < 256 ? 256 : TPR; }
// 64 registers a thread for bf16, 128 for fp32, whose loads take twice as many
__host__ __device__ constexpr int blocks_per_sm(int TPR, bool bf16) { return (bf16 ? 1024 : 512) / block_threads(TPR); }

// 8 scaled values -> 8 bytes.
template <int OUT>
__device__ __forceinline__ uint2 pack_bytes(const float (&z)[8]) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (OUT == OUT_E4M3) {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(z[4 * i], z[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(z[4 * i + 2], z[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
      w[i] = lo | (hi << 16);
    } else {
      w[i] = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int q = max(-127, min(127, __float2int_rn(z[4 * i + e])));
        w[i] |= (uint32_t)(q & 0xFF) << (8 * e);
      }
    }
  }
  return make_uint2(w[0], w[1]);
}

template <int TPR, int VPT, int U, bool BF16, int OUT>
__global__ void __launch_bounds__(block_threads(TPR), blocks_per_sm(TPR, BF16)) norm_kernel(NormParams p) {
  constexpr int NT = block_threads(TPR), GROUPS = NT / TPR;
  __shared__ float red[U * 32];
  if (block_leaves(p.err)) return;
  const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  const int nvec = p.D / 8;
  const long long row0 = (long long)blockIdx.x * (GROUPS * U) + grp;
  Raw<BF16> rx[U][VPT], rr[U][VPT];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long row = row0 + (long long)u * GROUPS;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int vec = t + i * TPR;
      const size_t at = (size_t)row * nvec + vec;
      const bool in = row < p.rows && vec < nvec;
      rx[u][i] = in ? load8<BF16>(p.x, at) : Raw<BF16>{};
      if (p.residual) rr[u][i] = in ? load8<BF16>(p.residual, at) : Raw<BF16>{};
    }
  }
  float f[U][VPT][8], ss[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long row = row0 + (long long)u * GROUPS;
    ss[u] = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      unpack8<BF16>(rx[u][i], f[u][i]);
      if (p.residual) {
        float g[8];
        unpack8<BF16>(rr[u][i], g);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[u][i][e] += g[e];
        const Raw<BF16> r = pack8<BF16>(f[u][i]);
        const int vec = t + i * TPR;
        if (p.residual_out && row < p.rows && vec < nvec)
          store8<BF16>(p.residual_out, (size_t)row * nvec + vec, r);
        unpack8<BF16>(r, f[u][i]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) ss[u] = fmaf(f[u][i][e], f[u][i][e], ss[u]);
    }
  }
  row_reduce<TPR, U, false>(ss, red);
  const float inv_d = 1.f / (float)p.D;
  float top[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const float rstd = rsqrtf(ss[u] * inv_d + p.eps);
    top[u] = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int vec = t + i * TPR;
      float w[8];
      if (p.weight && vec < nvec) {
        const float4 w0 = __ldg(reinterpret_cast<const float4 *>(p.weight) + 2 * vec);
        const float4 w1 = __ldg(reinterpret_cast<const float4 *>(p.weight) + 2 * vec + 1);
        w[0] = w0.x; w[1] = w0.y; w[2] = w0.z; w[3] = w0.w;
        w[4] = w1.x; w[5] = w1.y; w[6] = w1.z; w[7] = w1.w;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 1.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        f[u][i][e] = f[u][i][e] * rstd * w[e];
        if (OUT != OUT_SAME && p.group == 0) top[u] = max_nan(top[u], vec < nvec ? fabsf(f[u][i][e]) : 0.f);
      }
    }
  }
  if constexpr (OUT == OUT_SAME) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long row = row0 + (long long)u * GROUPS;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int vec = t + i * TPR;
        if (row < p.rows && vec < nvec) store8<BF16>(p.y, (size_t)row * nvec + vec, pack8<BF16>(f[u][i]));
      }
    }
  } else {
    constexpr float kMost = OUT == OUT_E4M3 ? 448.f : 127.f;
    if (p.group == 0) row_reduce<TPR, U, true>(top, red);
    const int lanes_log = p.group == 128 ? 4 : p.group == 64 ? 3 : 2;       // log2 of a group's consecutive lanes
    const int nscale = p.group ? (p.D + p.group - 1) / p.group : 1;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long row = row0 + (long long)u * GROUPS;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int vec = t + i * TPR;
        float m = top[u];
        if (p.group) {
          m = 0.f;
          if (vec < nvec)
#pragma unroll
            for (int e = 0; e < 8; ++e) m = max_nan(m, fabsf(f[u][i][e]));
          if (lanes_log >= 4) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, 8));
          if (lanes_log >= 3) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
          m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
          m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        }
        const float most = max_nan(m, kTiny), inv = kMost / most;
        if (row < p.rows && vec < nvec) {
          float z[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) z[e] = f[u][i][e] * inv;
          reinterpret_cast<uint2 *>(p.y)[(size_t)row * nvec + vec] = pack_bytes<OUT>(z);
          if (p.group == 0 ? vec == 0 : (vec & ((1 << lanes_log) - 1)) == 0)
            p.scale[(size_t)row * nscale + (p.group ? vec >> lanes_log : 0)] = most / kMost;
        }
      }
    }
  }
}

// ---- backward: rows dealt to the blocks in turn; a thread's columns of dw stay in registers
__host__ __device__ constexpr int back_blocks_per_sm(int TPR, bool bf16) { return bf16 && TPR <= 256 ? 2 : 1; }

template <int TPR, int VPT, bool BF16>
__global__ void __launch_bounds__(block_threads(TPR), back_blocks_per_sm(TPR, BF16)) norm_backward_kernel(NormBackwardParams p) {
  constexpr int NT = block_threads(TPR), GROUPS = NT / TPR;
  constexpr bool AHEAD = TPR < 1024;      // the widest rows have no registers for a second one
  __shared__ float red[2 * 32];
  __shared__ float sum[GROUPS > 1 ? GROUPS * TPR * VPT * 8 : 1];
  let_next_start();
  if (block_leaves(p.err)) return;
  const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  const int nvec = p.D / 8;
  float w[VPT][8], dw[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int vec = t + i * TPR;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w[i][e] = (p.weight && vec < nvec) ? __ldg(p.weight + 8 * vec + e) : 1.f;
      dw[i][e] = 0.f;
    }
  }
  const float inv_d = 1.f / (float)p.D;
  const long long step = (long long)gridDim.x * GROUPS;
  Raw<BF16> nx[VPT], ny[VPT], ng[VPT];
  auto fetch = [&](long long row) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int vec = t + i * TPR;
      const size_t at = (size_t)row * nvec + vec;
      const bool in = row < p.rows && vec < nvec;
      nx[i] = in ? load8<BF16>(p.x, at) : Raw<BF16>{};
      ny[i] = in ? load8<BF16>(p.dy, at) : Raw<BF16>{};
      if (p.dr) ng[i] = in ? load8<BF16>(p.dr, at) : Raw<BF16>{};
    }
  };
  const long long first = (long long)blockIdx.x * GROUPS;
  if (AHEAD) fetch(first + grp);
  for (long long base = first; base < p.rows; base += step) {      // the block's rows; each thread comes along to the last
    const long long row = base + grp;
    if (!AHEAD) fetch(row);
    Raw<BF16> cx[VPT], cy[VPT], cg[VPT];
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      cx[i] = nx[i];
      cy[i] = ny[i];
      cg[i] = ng[i];
      float x[8], y[8];
      unpack8<BF16>(cx[i], x);
      unpack8<BF16>(cy[i], y);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s[0] = fmaf(x[e], x[e], s[0]);
        s[1] = fmaf(x[e], y[e] * w[i][e], s[1]);
      }
    }
    if (AHEAD) fetch(row + step);
    row_reduce<TPR, 2, false>(s, red);
    const float rstd = rsqrtf(s[0] * inv_d + p.eps);
    const float back = rstd * rstd * (s[1] * inv_d);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int vec = t + i * TPR;
      if (row >= p.rows || vec >= nvec) continue;
      float x[8], y[8], g[8];
      unpack8<BF16>(cx[i], x);
      unpack8<BF16>(cy[i], y);
      if (p.dr) unpack8<BF16>(cg[i], g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dw[i][e] = fmaf(y[e], x[e] * rstd, dw[i][e]);
        const float d = rstd * fmaf(-x[e], back, y[e] * w[i][e]);
        y[e] = p.dr ? d + g[e] : d;
      }
      store8<BF16>(p.dx, (size_t)row * nvec + vec, pack8<BF16>(y));
    }
  }
  if (p.part == nullptr) return;
  // one row of partial sums per block: the block's row groups added in order
  float *out = p.part + (size_t)blockIdx.x * p.D;
  if constexpr (GROUPS > 1) {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[(grp * VPT + i) * (TPR * 8) + e * TPR + t] = dw[i][e];
    __syncthreads();
    for (int c = threadIdx.x; c < p.D; c += NT) {
      const int vec = c >> 3, i = vec / TPR, tt = vec % TPR;
      float a = 0.f;
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) a += sum[(g * VPT + i) * (TPR * 8) + (c & 7) * TPR + tt];
      out[c] = a;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int vec = t + i * TPR;
      if (vec < nvec) {
        reinterpret_cast<float4 *>(out)[2 * vec] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
        reinterpret_cast<float4 *>(out)[2 * vec + 1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
      }
    }
  }
}

// dw[c] = sum of the blocks' partial rows, in a fixed order: 32 columns x 32 strided shares a block.
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float *part, int parts, int D, float *dw,
                                                       const unsigned *err) {
  __shared__ float s[32][33];
  after_previous();
  if (block_leaves(err)) return;
  const int c = blockIdx.x * 32 + threadIdx.x, y = threadIdx.y;
  float a = 0.f;
  if (c < D)
    for (int i = y; i < parts; i += 32) a += part[(size_t)i * D + c];
  s[y][threadIdx.x] = a;
  __syncthreads();
  if (y == 0 && c < D) {
    a = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) a += s[i][threadIdx.x];
    dw[c] = a;
  }
}

template <int TPR, int VPT, int U, bool SAME = true>
cudaError_t launch(const NormParams &p, bool bf16, int out, cudaStream_t s) {
  constexpr int NT = block_threads(TPR);
  const long long per = (long long)(NT / TPR) * U;
  const unsigned grid = (unsigned)((p.rows + per - 1) / per);
  if (out == OUT_SAME) {
    if constexpr (SAME) {
      if (bf16) norm_kernel<TPR, VPT, U, true, OUT_SAME><<<grid, NT, 0, s>>>(p);
      else norm_kernel<TPR, VPT, U, false, OUT_SAME><<<grid, NT, 0, s>>>(p);
    }
  } else if (bf16) {
    if (out == OUT_E4M3) norm_kernel<TPR, VPT, U, true, OUT_E4M3><<<grid, NT, 0, s>>>(p);
    else norm_kernel<TPR, VPT, U, true, OUT_I8><<<grid, NT, 0, s>>>(p);
  } else {
    if (out == OUT_E4M3) norm_kernel<TPR, VPT, U, false, OUT_E4M3><<<grid, NT, 0, s>>>(p);
    else norm_kernel<TPR, VPT, U, false, OUT_I8><<<grid, NT, 0, s>>>(p);
  }
  return cudaGetLastError();
}

constexpr int kMaxParts = 148 * 2;      // rows of partial sums at most: as many blocks as run at a time

template <int TPR, int VPT>
cudaError_t launch_back(const NormBackwardParams &p, bool bf16, cudaStream_t s) {
  constexpr int NT = block_threads(TPR);
  const long long per = NT / TPR, need = (p.rows + per - 1) / per;
  const long long cap = (long long)kMaxParts / 2 * back_blocks_per_sm(TPR, bf16);
  const unsigned grid = (unsigned)(need < cap ? need : cap);
  if (bf16) norm_backward_kernel<TPR, VPT, true><<<grid, NT, 0, s>>>(p);
  else norm_backward_kernel<TPR, VPT, false><<<grid, NT, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || p.part == nullptr) return e;
  return launch_next(norm_dw_kernel, (unsigned)((p.D + 31) / 32), dim3(32, 32), 0, s, p.part, (int)grid, p.D, p.dw, p.err);
}

}  // namespace norm

size_t norm_backward_workspace(long long rows, int D) {
  const long long parts = rows < norm::kMaxParts ? rows : norm::kMaxParts;
  return (size_t)parts * (size_t)D * 4;
}

// Threads per row so that a thread holds four vectors of 8 columns (of two rows where a row has no more than
// 128 threads of two), from the measurements above.
cudaError_t launch_norm(const NormParams &p, bool bf16, int out, cudaStream_t s) {
  using namespace norm;
  if (p.rows == 0) return cudaSuccess;
  const int nvec = p.D / 8;
  if (nvec <= 16 && out == OUT_SAME) {      // without groups of 16 lanes: fewer exchanges; 5.9 against 5.2 TB/s
    const unsigned grid = (unsigned)((p.rows + 63) / 64);
    if (bf16) norm_kernel<8, 2, 2, true, OUT_SAME><<<grid, 256, 0, s>>>(p);
    else norm_kernel<8, 2, 2, false, OUT_SAME><<<grid, 256, 0, s>>>(p);
    return cudaGetLastError();
  }
  if (nvec <= 16) return launch<16, 1, 4, false>(p, bf16, out, s);
  if (nvec <= 32) return launch<16, 2, 2>(p, bf16, out, s);
  if (nvec <= 64) return launch<32, 2, 2>(p, bf16, out, s);
  if (nvec <= 128) return launch<32, 4, 1>(p, bf16, out, s);
  if (nvec <= 256) return launch<128, 2, 2>(p, bf16, out, s);
  if (nvec <= 512) return launch<128, 4, 1>(p, bf16, out, s);
  if (nvec <= 1024) return launch<256, 4, 1>(p, bf16, out, s);
  return launch<512, 4, 1>(p, bf16, out, s);
}

cudaError_t launch_norm_backward(const NormBackwardParams &p, bool bf16, cudaStream_t s) {
  using namespace norm;
  if (p.rows == 0)
    return p.dw ? cudaMemsetAsync(p.dw, 0, (size_t)p.D * 4, s) : cudaSuccess;
  const int nvec = p.D / 8;
  if (nvec <= 16) return launch_back<8, 2>(p, bf16, s);
  if (nvec <= 32) return launch_back<16, 2>(p, bf16, s);
  if (nvec <= 64) return launch_back<32, 2>(p, bf16, s);
  if (nvec <= 128) return launch_back<64, 2>(p, bf16, s);
  if (nvec <= 256) return launch_back<128, 2>(p, bf16, s);
  if (nvec <= 512) return launch_back<256, 2>(p, bf16, s);
  if (nvec <= 1024) return launch_back<512, 2>(p, bf16, s);
  return launch_back<1024, 2>(p, bf16, s);
}

}  // namespace kda
