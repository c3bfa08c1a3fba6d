// Linear attention on the tensor cores (bf16 inputs): what its prefill and its backward pass share.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>

#include "kda_linear.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace lintc {

using namespace tc;
using lin::Segment;

constexpr int C = 128;      // rows of a chunk
constexpr long long kDrainCycles = 2000000;      // for what is in flight when a block ends

__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, uint32_t src, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];"
               :: "l"(reinterpret_cast<uint64_t>(map)), "r"(src), "r"(c0), "r"(c1), "r"(c2) : "memory");
}
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
// D (TMEM) += A (TMEM, packed bf16) B (shared memory).
__device__ __forceinline__ void mma_bf16_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred P;\n\tsetp.ne.b32 P, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, P;\n\t}"
      :: "r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}

// Descriptor of a tile's K-step s from that of step 0: one addition in the issuing thread, where computing each
// from its address took longer than the product.
template <int R>
__device__ __forceinline__ uint64_t kmajor_step(uint64_t d, int s) { return d + (uint32_t)(((s >> 2) * R * 128 + (s & 3) * 32) >> 4); }
__device__ __forceinline__ uint64_t mnmajor_step(uint64_t d, int s) { return d + (uint32_t)(16 * s * 128 >> 4); }

// 2^x with results below 2^-126 taken as 0.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 32 fp32 columns of this thread's TMEM lane: issue, and wait for all loads issued before.
__device__ __forceinline__ void tmem_ld32_issue(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// The registers pass through the wait, so that no use of them moves before it.
__device__ __forceinline__ void tmem_ld32_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
      : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
        "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),
        "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]),
        "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]),
        "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]) :: "memory");
}

// The same for 16 columns.
__device__ __forceinline__ void tmem_ld16_issue(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld16_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
      : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
        "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]) :: "memory");
}
// Eight columns stored; one column stored, two loaded.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
               :: "r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st1(uint32_t taddr, float x) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" :: "r"(taddr), "r"(__float_as_uint(x)) : "memory");
}
__device__ __forceinline__ void tmem_ld2(uint32_t taddr, float (&x)[2]) {
  uint32_t r[2];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(r[0]), "+r"(r[1]) :: "memory");
  x[0] = __uint_as_float(r[0]);
  x[1] = __uint_as_float(r[1]);
}

// 8 floats (32 bytes, a whole sector) to global memory.
__device__ __forceinline__ void store_8(float *p, const float *f) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
               :: "l"(p), "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]) : "memory");
}

// Bounded waits of one block.  After one has run out every role leaves its loop; the waits of the
// others then end too.
struct Waits {
  long long limit;
  unsigned *err, *site;
  volatile int *failed;
  static __device__ __forceinline__ bool test(uint64_t *bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred P;\n\tmbarrier.try_wait.parity.shared::cta.b64 P, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, P;\n\t}"
        : "=r"(done) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    return done != 0;
  }
  __device__ __forceinline__ bool operator()(uint64_t *bar, uint32_t phase, unsigned code) const {
    const uint32_t parity = phase & 1;
    if (test(bar, parity)) return true;
    const long long t0 = clock64();
    while (!test(bar, parity)) {
      if (*failed) return false;
      if (clock64() - t0 > limit) {
        note_timeout(site, code);
        atomicOr(err, ERR_BIT_TIMEOUT);
        *failed = 1;
        return false;
      }
    }
    return true;
  }
  // The same by a whole warp, all of whose lanes get the same answer.
  __device__ __forceinline__ bool warp(uint64_t *bar, uint32_t phase, unsigned code) const {
    return __all_sync(0xFFFFFFFFu, (*this)(bar, phase, code));
  }
};

// A chunk's decays, one warp: lane's rows 4 lane .. 4 lane + 3.  Loading is apart from summing, so that the
// next chunk's values are on their way while this one's are used.
struct RawDecays {
  float x[4];
  uint32_t bits;        // bit e: row 4 lane + e is a real token
};
__device__ __forceinline__ RawDecays load_decays(const LinearParams &p, int pos0, int end, int h) {
  RawDecays d;
  const int pos = pos0 + 4 * (threadIdx.x & 31);
  uint8_t m[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const bool in = pos + e < end;
    m[e] = in ? (p.mask != nullptr ? p.mask[pos + e] : (uint8_t)1) : (uint8_t)0;
    d.x[e] = in ? p.log_alpha[p.decay_head ? (size_t)h : (size_t)(pos + e) * p.H + h] : 0.f;
  }
  d.bits = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) d.bits |= (uint32_t)(m[e] != 0) << e;
  return d;
}
// Inclusive sums b of log2 a, the total; word: lanes 0, 8, 16, 24 get the bits of rows 32 (lane / 8) .. + 31.
__device__ __forceinline__ void scan_decays(const RawDecays &d, double (&b)[4], double &total, uint32_t &word) {
  const int lane = threadIdx.x & 31;
  double s = 0.0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if ((d.bits >> e) & 1) s += lin::log2_step(d.x[e]);
    b[e] = s;
  }
  double x = s;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = lin::shfl_up_f64(x, o);
    if (lane >= o) x += y;
  }
  total = lin::shfl_f64(x, 31);
  const double before = lin::shfl_up_f64(x, 1);      // (x - s would carry a NaN back to the lane's rows before it)
#pragma unroll
  for (int e = 0; e < 4; ++e) b[e] += lane ? before : 0.0;
  word = d.bits << (4 * (lane & 7));
  word |= __shfl_xor_sync(0xFFFFFFFFu, word, 1);
  word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2);
  word |= __shfl_xor_sync(0xFFFFFFFFu, word, 4);
}

// A block's n-th item of a list: there and back over the blocks, so that the blocks with the longest item of one
// round take the shortest of the next.
__device__ __forceinline__ int item_of(int n) {
  return n * (int)gridDim.x + (int)(n & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

// 8 bf16 of a 16-byte word as floats.
__device__ __forceinline__ void unpack8(const uint4 &u, float (&f)[8]) {
  const uint32_t a[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = __uint_as_float(a[e] << 16);
    f[2 * e + 1] = __uint_as_float(a[e] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float *f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}
// Rounds 8 floats to bf16 (returned packed) and leaves the remainders in f.
__device__ __forceinline__ uint4 take_bf16(float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    w[e] = pack_bf16x2(f[2 * e], f[2 * e + 1]);
    f[2 * e] -= __uint_as_float(w[e] << 16);
    f[2 * e + 1] -= __uint_as_float(w[e] & 0xFFFF0000u);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// ============================================================ host
inline PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    return nullptr;
  }();
  return fn;
}

// [N, heads, d] bf16 in boxes of `rows` rows of one head and 64 columns with the 128-byte swizzle, or 32 columns
// with the 64-byte one.
inline bool encode(CUtensorMap *map, const void *ptr, int d, int heads, size_t N, int rows = C, int cols = 64) {
  auto fn = encoder();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)N};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)d * 2 * heads};
  const cuuint32_t box[3] = {(cuuint32_t)cols, 1u, (cuuint32_t)rows}, one[3] = {1u, 1u, 1u};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// fp32 [rows][d] in boxes of `box_rows` rows and 32 columns with the 128-byte swizzle.
inline bool encode_f32(CUtensorMap *map, const void *ptr, int d, size_t rows, int box_rows) {
  auto fn = encoder();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, 1u, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 4, (cuuint64_t)d * 4};
  const cuuint32_t box[3] = {32u, 1u, (cuuint32_t)box_rows}, one[3] = {1u, 1u, 1u};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void *>(ptr), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline int sm_count() {
  static std::atomic<int> n[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  int v = n[dev].load(std::memory_order_relaxed);
  if (v == 0) {
    if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0) v = 148;
    n[dev].store(v, std::memory_order_relaxed);
  }
  return v;
}

}  // namespace lintc
}  // namespace kda
