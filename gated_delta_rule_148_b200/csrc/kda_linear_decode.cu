// Linear attention with a decay for each head: one token per row on a fp32 state.
//
//   S <- a S + k v^T,  o = S^T q,  a = exp(log_alpha)
//
// Bound by HBM: an active (row, head) reads and writes its d_k x d_v fp32 state once
// (128 KB for d = 128); everything else is below 1 % of the bytes.  A block holds DVS columns of
// one (row, head)'s state in registers between the load and the store: a thread owns 4 consecutive columns
// (16 bytes) of d_k DVS / 1024 rows, all its loads in flight before the first use.  Columns
// never mix, so a small batch is cut into column slices until there are about two blocks
// per SM; a large one keeps whole rows (512-byte rows at d_v = 128).  The sum over d_k is
// taken in registers, by shuffles, and over the warps through shared memory.
#include "kda_internal.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;

template <int DK, int DV, int DVS, bool BF16>
__global__ void __launch_bounds__(kThreads) linear_decode_kernel(LinearDecodeParams p) {
  constexpr int TPR = DVS / 4;                  // threads per state row
  constexpr int GROUPS = kThreads / TPR;        // rows in a pass of the block
  constexpr int RPT = DK / GROUPS;              // rows per thread
  constexpr int SL = DV / DVS;
  static_assert(RPT * GROUPS == DK && TPR <= 32, "tiling");
  __shared__ float red[kThreads / 32][DVS];
  __shared__ float s_k[DK], s_q[DK];

  const int bh = blockIdx.x / SL, c0 = (blockIdx.x % SL) * DVS;
  const int b = bh / p.H, h = bh % p.H;
  const int tid = threadIdx.x, cg = tid % TPR, rg = tid / TPR;

  if (block_leaves(p.err)) return;
  if (p.mask != nullptr && p.mask[b] == 0) {
    for (int j = tid; j < DVS; j += kThreads) store_elem<BF16>(p.o, (size_t)bh * DV + c0 + j, 0.f);
    return;
  }
  float4 *S = reinterpret_cast<float4 *>(p.state + (size_t)bh * DK * DV + c0);
  float4 s[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) s[i] = __ldcs(&S[(size_t)(i * GROUPS + rg) * (DV / 4) + cg]);

  const size_t key = ((size_t)b * p.Hk + h / (p.H / p.Hk)) * DK;
  for (int c = tid; c < 2 * DK; c += kThreads) {
    if (c < DK) s_k[c] = load_elem<BF16>(p.k, key + c);
    else s_q[c - DK] = load_elem<BF16>(p.q, key + c - DK);
  }
  const float a = expf(p.log_alpha[p.decay_head ? h : bh]);
  float v[4], o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = load_elem<BF16>(p.v, (size_t)bh * DV + c0 + 4 * cg + e);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int r = i * GROUPS + rg;
    const float kr = s_k[r], qr = s_q[r];
    s[i].x = fmaf(a, s[i].x, kr * v[0]);
    s[i].y = fmaf(a, s[i].y, kr * v[1]);
    s[i].z = fmaf(a, s[i].z, kr * v[2]);
    s[i].w = fmaf(a, s[i].w, kr * v[3]);
    __stcs(&S[(size_t)r * (DV / 4) + cg], s[i]);
    o[0] = fmaf(qr, s[i].x, o[0]);
    o[1] = fmaf(qr, s[i].y, o[1]);
    o[2] = fmaf(qr, s[i].z, o[2]);
    o[3] = fmaf(qr, s[i].w, o[3]);
  }
#pragma unroll
  for (int off = 16; off >= TPR; off >>= 1)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] += __shfl_xor_sync(0xFFFFFFFFu, o[e], off);
  if ((tid & 31) < TPR)
    *reinterpret_cast<float4 *>(&red[tid >> 5][4 * cg]) = make_float4(o[0], o[1], o[2], o[3]);
  __syncthreads();
  for (int j = tid; j < DVS; j += kThreads) {
    float acc = 0.f;
#pragma unroll
    for (int g = 0; g < kThreads / 32; ++g) acc += red[g][j];
    store_elem<BF16>(p.o, (size_t)bh * DV + c0 + j, acc);
  }
}

template <int DK, int DV, int DVS>
cudaError_t launch(const LinearDecodeParams &p, bool bf16, cudaStream_t s) {
  const unsigned grid = (unsigned)p.B * p.H * (DV / DVS);
  if (bf16) linear_decode_kernel<DK, DV, DVS, true><<<grid, kThreads, 0, s>>>(p);
  else linear_decode_kernel<DK, DV, DVS, false><<<grid, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <int DK, int DV>
cudaError_t launch_dims(const LinearDecodeParams &p, bool bf16, cudaStream_t s) {
  const size_t heads = (size_t)p.B * p.H;
  if (heads * (DV / 32) <= 296) return launch<DK, DV, 32>(p, bf16, s);
  if constexpr (DV == 128) {
    if (heads * 2 <= 296) return launch<DK, DV, 64>(p, bf16, s);
  }
  return launch<DK, DV, DV>(p, bf16, s);
}

}  // namespace

cudaError_t launch_linear_decode(const LinearDecodeParams &p, bool bf16, cudaStream_t s) {
  if (p.B == 0) return cudaSuccess;
  if (p.dk == 128) return p.dv == 128 ? launch_dims<128, 128>(p, bf16, s) : launch_dims<128, 64>(p, bf16, s);
  return p.dv == 128 ? launch_dims<64, 128>(p, bf16, s) : launch_dims<64, 64>(p, bf16, s);
}

}  // namespace kda
