// Linear attention with a decay for each head on the tensor cores (bf16 inputs): prefill.
// Formulas in kda_linear.cuh; chunks of 128 rows, segments of `per` chunks.
//
//   parts   a segment's contribution to the state, sum_s w_s k_s v_s^T with w_s = 2^{b_end - b_s}:
//           the chunks of a segment from the last to the first, so that w needs no second
//           look at the decays, all accumulated in TMEM:  S += K^T (w V).  w V is split into
//           three bf16 parts (24 bits), so the states keep fp32 accuracy.
//   chain   states at the segments' starts (chain_kernel, kda_linear.cu)
//   rows    per chunk  A = Q K^T,  P = A o 2^{b_t - b_s} (bf16, TMEM),  O1 = Q S,  O2 = P V,
//           o = 2^{b_t} O1 + O2,  S <- 2^{b_C} S + K^T (w V), w V in two bf16 parts (2^-17: it only
//           feeds the bf16 operand S of the segment's later chunks).
// Both are persistent blocks with roles: a TMA warp, an MMA thread, a warp that prepares a
// chunk's decays (and clears rows that are pads or belong to the next sequence), and warpgroups
// that move accumulators.  Off the diagonal a warp's 32 rows share a reference row R before them,
// 2^{b_t - b_s} = 2^{b_t - R} 2^{R - b_s}, both factors <= 1: one exponential per row and column
// instead of one per pair.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cmath>

#include "kda_linear.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace lintc {

using namespace tc;
using lin::Segment;

constexpr int C = 128;

// Wait sites reported with a timeout.
enum : unsigned { SITE_PARTS = 41, SITE_ROWS = 51 };

__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void group_sync(int id) { asm volatile("bar.sync %0, 128;" :: "r"(id) : "memory"); }
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

struct Maps {
  CUtensorMap q, k, v, o;
};

// Bounded waits of one block.  After one has run out every role leaves its loop; the waits of the
// others then run out too.
struct Waits {
  long long limit;
  unsigned *err, *site;
  volatile int *failed;
  __device__ __forceinline__ bool operator()(uint64_t *bar, uint32_t parity, unsigned code) const {
    if (*failed) return false;
    if (mbar_wait(bar, parity & 1, limit)) return true;
    note_timeout(site, code);
    atomicOr(err, ERR_BIT_TIMEOUT);
    *failed = 1;
    return false;
  }
};

// Zeroes the rows of a [128][D] tile that are not set in valid (one warp).
template <int D>
__device__ __forceinline__ void clear_rows(unsigned char *tile, const uint32_t *valid) {
  const int lane = threadIdx.x & 31;
  for (int i = lane; i < C * (D / 8); i += 32) {
    const int r = i / (D / 8), c = i % (D / 8);
    if (!((valid[r >> 5] >> (r & 31)) & 1))
      *reinterpret_cast<uint4 *>(tile + row_tile_chunk(r, c >> 3, c & 7, C)) = make_uint4(0, 0, 0, 0);
  }
}

// log2 decays of a chunk by one warp: lane's rows 4 lane .. 4 lane + 3, inclusive sums b and the total.
// word: lanes 0, 8, 16 and 24 get the bits of rows 32 (lane / 8) .. + 31 that are real tokens; returns
// whether all 128 are.
__device__ __forceinline__ bool scan_chunk(const LinearParams &p, int pos0, int end, int h, double (&b)[4],
                                           double &total, uint32_t &word) {
  const int lane = threadIdx.x & 31;
  double s = 0.0;
  uint32_t bits = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int pos = pos0 + 4 * lane + e;
    if (pos < end && (p.mask == nullptr || p.mask[pos] != 0)) bits |= 1u << e;
    s += lin::log2_decay(p.log_alpha, p.decay_head, p.mask, pos, end, h, p.H);
    b[e] = s;
  }
  double x = s;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = lin::shfl_up_f64(x, o);
    if (lane >= o) x += y;
  }
  total = lin::shfl_f64(x, 31);
#pragma unroll
  for (int e = 0; e < 4; ++e) b[e] += x - s;
  word = bits << (4 * (lane & 7));
  word |= __shfl_xor_sync(0xFFFFFFFFu, word, 1);
  word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2);
  word |= __shfl_xor_sync(0xFFFFFFFFu, word, 4);
  return __all_sync(0xFFFFFFFFu, bits == 0xFu);
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

// ============================================================ parts
constexpr int kPartsThreads = 8 * 32 + 64;      // two warpgroups, a TMA + MMA warp, a preparing warp

template <int DK, int DV>
struct PartsSmem {
  static constexpr uint32_t KT = C * DK * 2, VT = C * DV * 2;
  static constexpr uint32_t STAGE = KT + VT, W = 2 * STAGE, TAB = W + 3 * VT;
  // DK = 64: the MMA's rows 64 .. 127 come from the bytes after the K tile and are not used
  static constexpr uint32_t WGT = TAB, VALID = WGT + 2 * C * 4, BARS = VALID + 32, END = BARS + 128;
};

template <int DK, int DV>
__global__ void __launch_bounds__(kPartsThreads, 1)
parts_kernel(LinearParams p, const __grid_constant__ Maps maps, const int *sbase, float *part, float *whole,
             int per) {
  using L = PartsSmem<DK, DV>;
  extern __shared__ __align__(1024) unsigned char sm[];
  if (device_error_latched(p.err)) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nitems = sbase[p.num_seqs] * p.H;
  float *wgt = reinterpret_cast<float *>(sm + L::WGT);
  uint64_t *full = reinterpret_cast<uint64_t *>(sm + L::BARS), *ready = full + 2, *empty = full + 4,
           *w_ready = full + 6, *w_free = full + 7, *s_done = full + 8, *s_free = full + 10, *drain = full + 12;
  uint32_t *tmem_sh = reinterpret_cast<uint32_t *>(full + 13);
  volatile int *failed = reinterpret_cast<volatile int *>(tmem_sh + 1);
  if (warp == 8) tmem_alloc(tmem_sh, 256);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(full + i, 1);
      mbar_init(ready + i, 1);
      mbar_init(empty + i, 1);
      mbar_init(s_done + i, 1);
      mbar_init(s_free + i, 256);
    }
    mbar_init(w_ready, 256);
    mbar_init(w_free, 1);
    mbar_init(drain, 1);
    *failed = 0;
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tm = *tmem_sh;
  const Waits wait{p.wait_cycles, p.err, p.site, failed};
  const int G = p.H / p.Hk;
  int step = 0, n = 0;      // chunks and items that this role has begun

  // the last segment of a sequence matters to the final state only
  auto skip = [&](const Segment &sg) { return sg.last && p.final_state == nullptr; };

  if (warp == 8) {
    // ---------------- loads and MMAs (one thread)
    if (lane == 0) {
      auto load = [&](const Segment &sg, int h, int c, int st) {
        mbar_arrive_expect_tx(full + st, L::STAGE);
        const uint32_t dst = smem_u32(sm + st * L::STAGE);
        const int pos = sg.begin + c * C;
#pragma unroll
        for (int kb = 0; kb < DK / 64; ++kb) tma_load_3d(dst + kb * C * 128, &maps.k, kb * 64, h / G, pos, full + st);
#pragma unroll
        for (int kb = 0; kb < DV / 64; ++kb)
          tma_load_3d(dst + L::KT + kb * C * 128, &maps.v, kb * 64, h, pos, full + st);
      };
      // loads run one chunk ahead of the MMAs, over the items' borders
      int li = blockIdx.x, lc = -1, lstep = 0;
      Segment ls{};
      auto advance = [&]() {            // next (item, chunk) to load
        while (true) {
          if (lc > 0) { --lc; return true; }
          if (lc == 0) li += gridDim.x;
          lc = -1;
          if (li >= nitems) return false;
          ls = lin::locate(p.cu, sbase, p.num_seqs, li / p.H, per * C);
          if (!skip(ls)) { lc = (ls.end - ls.begin + C - 1) / C; }
          else li += gridDim.x;
        }
      };
      bool more = advance();
      bool ok = true;
      auto load_next = [&]() {
        if (!more) return;
        const int st = lstep & 1;
        if (lstep >= 2) ok = ok && wait(empty + st, (lstep >> 1) - 1, SITE_PARTS);
        if (!ok) return;
        load(ls, li % p.H, lc, st);
        ++lstep;
        more = advance();
      };
      load_next();
      for (int i = blockIdx.x; i < nitems && ok; i += gridDim.x) {
        const Segment sg = lin::locate(p.cu, sbase, p.num_seqs, i / p.H, per * C);
        if (skip(sg)) continue;
        const int chunks = (sg.end - sg.begin + C - 1) / C, acc = n & 1;
        if (n >= 2) ok = wait(s_free + acc, (n >> 1) - 1, SITE_PARTS + 1);
        for (int j = 0; j < chunks && ok; ++j, ++step) {
          load_next();
          const int st = step & 1;
          ok = ok && wait(ready + st, step >> 1, SITE_PARTS + 2) && wait(w_ready, step, SITE_PARTS + 3);
          if (!ok) break;
          fence_after_sync();
          const uint32_t sk = smem_u32(sm + st * L::STAGE), sw = smem_u32(sm + L::W);
          const uint32_t id = idesc_bf16(128, DV, 1, 1);
#pragma unroll
          for (int x = 0; x < 3; ++x)
#pragma unroll
            for (int s = 0; s < C / 16; ++s)
              mma_bf16(tm + acc * 128, desc_mnmajor(sk, C, 0, s), desc_mnmajor(sw + x * L::VT, C, 0, s), id,
                       j > 0 || x > 0 || s > 0);
          mma_commit(w_free);
          mma_commit(empty + st);
          if (j == chunks - 1) mma_commit(s_done + acc);
        }
        ++n;
      }
      if (!ok)      // loads in flight land before the block ends
        for (int i = 0; i < lstep; ++i) mbar_wait(full + (i & 1), (i >> 1) & 1, 2000000);
      mma_commit(drain);
      mbar_wait(drain, 0, p.wait_cycles);
    }
  } else if (warp == 9) {
    // ---------------- weights and rows to clear, from a segment's last chunk to its first
    uint32_t *valid = reinterpret_cast<uint32_t *>(sm + L::VALID);
    bool ok = true;
    for (int i = blockIdx.x; i < nitems && ok; i += gridDim.x) {
      const Segment sg = lin::locate(p.cu, sbase, p.num_seqs, i / p.H, per * C);
      if (skip(sg)) continue;
      const int chunks = (sg.end - sg.begin + C - 1) / C, h = i % p.H;
      double after = 0.0;
      for (int j = chunks - 1; j >= 0 && ok; --j, ++step) {
        const int st = step & 1;
        double b[4], total;
        uint32_t word;
        const bool clean = scan_chunk(p, sg.begin + j * C, sg.end, h, b, total, word);
        if (step >= 2) ok = wait(empty + st, (step >> 1) - 1, SITE_PARTS + 4);
        if ((lane & 7) == 0) valid[4 * st + (lane >> 3)] = word;
        __syncwarp();
        float4 w;
        w.x = exp2f((float)(after + (total - b[0])));
        w.y = exp2f((float)(after + (total - b[1])));
        w.z = exp2f((float)(after + (total - b[2])));
        w.w = exp2f((float)(after + (total - b[3])));
        reinterpret_cast<float4 *>(wgt + st * C)[lane] = w;
        after += total;
        ok = ok && wait(full + st, step >> 1, SITE_PARTS + 5);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!clean && ok) {
          clear_rows<DK>(sm + st * L::STAGE, valid + 4 * st);
          clear_rows<DV>(sm + st * L::STAGE + L::KT, valid + 4 * st);
          fence_async_smem();
        }
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(ready + st);
      }
      if (lane == 0) whole[i] = exp2f((float)after);
    }
  } else {
    // ---------------- w V in three parts; at a segment's end the state to global memory
    const int r = tid & 127, half = tid >> 7;          // row of the chunk (of the state), column half
    constexpr int NC = DV / 16;                        // 16-byte words of the half
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    bool ok = true;
    for (int i = blockIdx.x; i < nitems && ok; i += gridDim.x) {
      const Segment sg = lin::locate(p.cu, sbase, p.num_seqs, i / p.H, per * C);
      if (skip(sg)) continue;
      const int chunks = (sg.end - sg.begin + C - 1) / C, acc = n & 1;
      for (int j = 0; j < chunks && ok; ++j, ++step) {
        const int st = step & 1;
        ok = wait(ready + st, step >> 1, SITE_PARTS + 6);
        if (step >= 1) ok = ok && wait(w_free, step - 1, SITE_PARTS + 7);
        if (!ok) break;
        const float w = wgt[st * C + r];
        const unsigned char *sv = sm + st * L::STAGE + L::KT;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const int cc = half * NC + c;
          const uint32_t at = row_tile_chunk(r, cc >> 3, cc & 7, C);
          float f[8];
          unpack8(*reinterpret_cast<const uint4 *>(sv + at), f);
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] *= w;
#pragma unroll
          for (int x = 0; x < 3; ++x) *reinterpret_cast<uint4 *>(sm + L::W + x * L::VT + at) = take_bf16(f);
        }
        fence_async_smem();
        mbar_arrive(w_ready);
      }
      ok = ok && wait(s_done + acc, n >> 1, SITE_PARTS + 8);
      if (!ok) break;
      fence_after_sync();
      float *out = part + ((size_t)i * DK + r) * DV + half * (DV / 2);
#pragma unroll
      for (int c = 0; c < DV / 64; ++c) {
        float v[32];
        tmem_ld32(tm + lanes + acc * 128 + half * (DV / 2) + c * 32, v);
        if (r < DK)
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4 *>(out + c * 32 + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
      }
      fence_before_sync();
      mbar_arrive(s_free + acc);
      ++n;
    }
  }
  fence_before_sync();
  __syncthreads();
  if (warp == 8) {
    fence_after_sync();
    tmem_dealloc(tm, 256);
  }
}

// ============================================================ rows
constexpr int kRowsThreads = 8 * 32 + 96;       // two warpgroups; TMA, MMA and preparing warps

template <int DK, int DV>
struct RowsSmem {
  static constexpr uint32_t QT = C * DK * 2, VT = C * DV * 2;
  static constexpr uint32_t STAGE = 2 * QT + VT, W = 2 * STAGE;      // W: S, then w V, as bf16
  static constexpr uint32_t WB = (DK > C ? DK : C) * DV * 2;
  static constexpr uint32_t HL = W + WB, COLF = HL + 2 * C * 8, VALID = COLF + 192 * 4, WHOLE = VALID + 32;
  static constexpr uint32_t BARS = WHOLE + 8, END = BARS + 15 * 8 + 8;
  static_assert(END <= 232448, "shared memory of a block");
};

template <int DK, int DV>
__global__ void __launch_bounds__(kRowsThreads, 1)
rows_kernel(LinearParams p, const __grid_constant__ Maps maps, const int *sbase, const float *start, int per) {
  using L = RowsSmem<DK, DV>;
  extern __shared__ __align__(1024) unsigned char sm[];
  if (device_error_latched(p.err)) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nitems = sbase[p.num_seqs] * p.H;
  float2 *hl = reinterpret_cast<float2 *>(sm + L::HL);
  uint32_t *valid = reinterpret_cast<uint32_t *>(sm + L::VALID);
  float *whole = reinterpret_cast<float *>(sm + L::WHOLE);
  uint64_t *full = reinterpret_cast<uint64_t *>(sm + L::BARS), *ready = full + 2, *empty = full + 4,
           *a_done = full + 6, *p_ready = full + 7, *w_ready = full + 8, *w_free = full + 9, *o_done = full + 10,
           *o_free = full + 11, *drain = full + 12;
  uint32_t *tmem_sh = reinterpret_cast<uint32_t *>(full + 13);
  volatile int *failed = reinterpret_cast<volatile int *>(tmem_sh + 1);
  if (warp == 8) tmem_alloc(tmem_sh, 512);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(full + i, 1);
      mbar_init(ready + i, 1);
      mbar_init(empty + i, 2);        // the chunk's MMAs, and its output out of the tile
    }
    mbar_init(a_done, 1);
    mbar_init(p_ready, 128);
    mbar_init(w_ready, 128);
    mbar_init(w_free, 1);
    mbar_init(o_done, 1);
    mbar_init(o_free, 128);
    mbar_init(drain, 1);
    *failed = 0;
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tm = *tmem_sh;
  constexpr uint32_t T_S = 0, T_A = 128, T_O1 = 256, T_O2 = 384;      // P overlays A
  const Waits wait{p.wait_cycles, p.err, p.site, failed};
  const int G = p.H / p.Hk;
  int step = 0;
  uint32_t wn = 0;           // fills of W

  if (warp == 9) {
    // ---------------- loads
    if (lane == 0) {
      bool ok = true;
      for (int i = blockIdx.x; i < nitems && ok; i += gridDim.x) {
        const Segment sg = lin::locate(p.cu, sbase, p.num_seqs, i / p.H, per * C);
        const int h = i % p.H;
        for (int pos = sg.begin; pos < sg.end && ok; pos += C, ++step) {
          const int st = step & 1;
          if (step >= 2) ok = wait(empty + st, (step >> 1) - 1, SITE_ROWS);
          if (!ok) break;
          mbar_arrive_expect_tx(full + st, L::STAGE);
          const uint32_t dst = smem_u32(sm + st * L::STAGE);
#pragma unroll
          for (int kb = 0; kb < DK / 64; ++kb) {
            tma_load_3d(dst + kb * C * 128, &maps.q, kb * 64, h / G, pos, full + st);
            tma_load_3d(dst + L::QT + kb * C * 128, &maps.k, kb * 64, h / G, pos, full + st);
          }
#pragma unroll
          for (int kb = 0; kb < DV / 64; ++kb)
            tma_load_3d(dst + 2 * L::QT + kb * C * 128, &maps.v, kb * 64, h, pos, full + st);
        }
      }
      if (!ok)
        for (int i = 0; i < step; ++i) mbar_wait(full + (i & 1), (i >> 1) & 1, 2000000);
    }
  } else if (warp == 8) {
    // ---------------- MMAs
    if (lane == 0) {
      bool ok = true;
      const uint32_t sw = smem_u32(sm + L::W);
      for (int i = blockIdx.x; i < nitems && ok; i += gridDim.x) {
        const Segment sg = lin::locate(p.cu, sbase, p.num_seqs, i / p.H, per * C);
        for (int pos = sg.begin; pos < sg.end && ok; pos += C, ++step) {
          const int st = step & 1;
          const bool last = pos + C >= sg.end;
          const uint32_t sq = smem_u32(sm + st * L::STAGE), sk = sq + L::QT, sv = sk + L::QT;
          ok = wait(ready + st, step >> 1, SITE_ROWS + 1);
          if (!ok) break;
          fence_after_sync();
#pragma unroll
          for (int s = 0; s < DK / 16; ++s)
            mma_bf16(tm + T_A, desc_kmajor(sq, C, 0, s), desc_kmajor(sk, C, 0, s), idesc_bf16(128, C, 0, 0), s > 0);
          mma_commit(a_done);
          if (step > 0) ok = wait(o_free, step - 1, SITE_ROWS + 2);
          ok = ok && wait(w_ready, wn++, SITE_ROWS + 3);
          if (!ok) break;
          fence_after_sync();
#pragma unroll
          for (int s = 0; s < DK / 16; ++s)
            mma_bf16(tm + T_O1, desc_kmajor(sq, C, 0, s), desc_mnmajor(sw, DK, 0, s), idesc_bf16(128, DV, 0, 1), s > 0);
          mma_commit(w_free);
          if (!last)
            for (int x = 0; x < 2 && ok; ++x) {
              ok = wait(w_ready, wn++, SITE_ROWS + 4);
              if (!ok) break;
              fence_after_sync();
#pragma unroll
              for (int s = 0; s < C / 16; ++s)
                mma_bf16(tm + T_S, desc_mnmajor(sk, C, 0, s), desc_mnmajor(sw, C, 0, s), idesc_bf16(128, DV, 1, 1), 1);
              mma_commit(w_free);
            }
          ok = ok && wait(p_ready, step, SITE_ROWS + 5);
          if (!ok) break;
          fence_after_sync();
#pragma unroll
          for (int s = 0; s < C / 16; ++s)
            mma_bf16_ta(tm + T_O2, tm + T_A + 8 * s, desc_mnmajor(sv, C, 0, s), idesc_bf16(128, DV, 0, 1), s > 0);
          mma_commit(o_done);
          mma_commit(empty + st);
        }
      }
      mma_commit(drain);
      mbar_wait(drain, 0, p.wait_cycles);
    }
  } else if (warp == 10) {
    // ---------------- decays and rows to clear
    bool ok = true;
    for (int i = blockIdx.x; i < nitems && ok; i += gridDim.x) {
      const Segment sg = lin::locate(p.cu, sbase, p.num_seqs, i / p.H, per * C);
      const int h = i % p.H;
      for (int pos = sg.begin; pos < sg.end && ok; pos += C, ++step) {
        const int st = step & 1;
        double b[4], total;
        uint32_t word;
        const bool clean = scan_chunk(p, pos, sg.end, h, b, total, word);
        if (step >= 2) ok = wait(empty + st, (step >> 1) - 1, SITE_ROWS + 6);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        if ((lane & 7) == 0) valid[4 * st + (lane >> 3)] = word;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float hi = (float)b[e];
          hl[st * C + 4 * lane + e] = make_float2(hi, (float)(b[e] - (double)hi));
        }
        if (lane == 0) whole[st] = exp2f((float)total);
        __syncwarp();
        ok = wait(full + st, step >> 1, SITE_ROWS + 7);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!clean && ok) {
          clear_rows<DK>(sm + st * L::STAGE + L::QT, valid + 4 * st);
          clear_rows<DV>(sm + st * L::STAGE + 2 * L::QT, valid + 4 * st);
          fence_async_smem();
        }
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(ready + st);
      }
    }
  } else if (warp < 4) {
    // ---------------- P, and the output (thread: row t of the chunk)
    const int t = tid;
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    float *colf = reinterpret_cast<float *>(sm + L::COLF) + 16 * warp * (warp - 1);     // 32 warp entries
    bool ok = true;
    for (int i = blockIdx.x; i < nitems && ok; i += gridDim.x) {
      const Segment sg = lin::locate(p.cu, sbase, p.num_seqs, i / p.H, per * C);
      const int h = i % p.H;
      for (int pos = sg.begin; pos < sg.end && ok; pos += C, ++step) {
        const int st = step & 1;
        ok = wait(ready + st, step >> 1, SITE_ROWS + 8);
        if (!ok) break;
        const float2 *d = hl + st * C;
        const float2 bt = d[t], ref = d[warp > 0 ? 32 * warp - 1 : 0];
        const float rowf = exp2f((bt.x - ref.x) + (bt.y - ref.y)), from = exp2f(bt.x + bt.y);
        for (int x = 0; x < warp; ++x) {
          const float2 bs = d[32 * x + lane];
          colf[32 * x + lane] = exp2f((ref.x - bs.x) + (ref.y - bs.y));
        }
        __syncwarp();
        const bool real = (valid[4 * st + warp] >> lane) & 1;
        ok = wait(a_done, step, SITE_ROWS + 9);
        if (!ok) break;
        fence_after_sync();
#pragma unroll 1
        for (int x = 0; x < 4; ++x) {
          float a[32], w[16];
          if (x <= warp) tmem_ld32(tm + lanes + T_A + 32 * x, a);
          if (x < warp) {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float4 f = *reinterpret_cast<const float4 *>(colf + 32 * x + e);
              a[e] *= rowf * f.x;
              a[e + 1] *= rowf * f.y;
              a[e + 2] *= rowf * f.z;
              a[e + 3] *= rowf * f.w;
            }
          } else if (x == warp) {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float2 bs = d[32 * x + e];
              const float f = exp2f((bt.x - bs.x) + (bt.y - bs.y));
              a[e] = e <= lane ? a[e] * f : 0.f;
            }
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) a[e] = 0.f;
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = __uint_as_float(pack_bf16x2(a[2 * e], a[2 * e + 1]));
          tmem_st16(tm + lanes + T_A + 16 * x, w);
        }
        tmem_st_wait();
        fence_before_sync();
        mbar_arrive(p_ready);
        ok = wait(o_done, step, SITE_ROWS + 10);
        if (!ok) break;
        fence_after_sync();
        unsigned char *tile = sm + st * L::STAGE;           // q's (and k's) tile: no longer read
        const bool whole_chunk = pos + C <= sg.end;
        uint16_t *orow = reinterpret_cast<uint16_t *>(p.o) + ((size_t)(pos + t) * p.H + h) * DV;
#pragma unroll 1
        for (int x = 0; x < DV / 32; ++x) {
          float a[32], b[32];
          tmem_ld32(tm + lanes + T_O1 + 32 * x, a);
          tmem_ld32(tm + lanes + T_O2 + 32 * x, b);
#pragma unroll
          for (int e = 0; e < 32; ++e) a[e] = real ? fmaf(from, a[e], b[e]) : 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint4 u = make_uint4(pack_bf16x2(a[8 * e], a[8 * e + 1]), pack_bf16x2(a[8 * e + 2], a[8 * e + 3]),
                                       pack_bf16x2(a[8 * e + 4], a[8 * e + 5]), pack_bf16x2(a[8 * e + 6], a[8 * e + 7]));
            const int cc = 4 * x + e;
            if (whole_chunk) *reinterpret_cast<uint4 *>(tile + row_tile_chunk(t, cc >> 3, cc & 7, C)) = u;
            else if (pos + t < sg.end) *reinterpret_cast<uint4 *>(orow + 8 * cc) = u;
          }
        }
        fence_before_sync();
        mbar_arrive(o_free);
        if (whole_chunk) fence_async_smem();
        group_sync(1);
        if (tid == 0) {
          if (whole_chunk) {
#pragma unroll
            for (int kb = 0; kb < DV / 64; ++kb) tma_store_3d(&maps.o, smem_u32(tile) + kb * C * 128, kb * 64, h, pos);
            bulk_commit();
            bulk_wait_read();
          }
          mbar_arrive(empty + st);
        }
      }
    }
    if (tid == 0) bulk_wait_all();
  } else {
    // ---------------- S as an operand, S <- 2^{b_C} S, w V (thread: row of the state, then of the chunk)
    const int r = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    bool ok = true;
    for (int i = blockIdx.x; i < nitems && ok; i += gridDim.x) {
      const Segment sg = lin::locate(p.cu, sbase, p.num_seqs, i / p.H, per * C);
      for (int pos = sg.begin; pos < sg.end && ok; pos += C, ++step) {
        const int st = step & 1;
        const bool first = pos == sg.begin, last = pos + C >= sg.end;
        ok = wait(ready + st, step >> 1, SITE_ROWS + 11);
        if (wn > 0) ok = ok && wait(w_free, wn - 1, SITE_ROWS + 12);      // also: S has its last sum
        if (!ok) break;
        fence_after_sync();
        const float keep = whole[st];
        const float *in = start + ((size_t)i * DK + r) * DV;
        if (r < DK || DK == 128) {
#pragma unroll 1
          for (int x = 0; x < DV / 32; ++x) {
            float v[32];
            if (first) {
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float4 f = __ldcs(reinterpret_cast<const float4 *>(in + 32 * x + e));
                v[e] = f.x; v[e + 1] = f.y; v[e + 2] = f.z; v[e + 3] = f.w;
              }
            } else {
              tmem_ld32(tm + lanes + T_S + 32 * x, v);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int cc = 4 * x + e;
              *reinterpret_cast<uint4 *>(sm + L::W + row_tile_chunk(r, cc >> 3, cc & 7, DK)) =
                  make_uint4(pack_bf16x2(v[8 * e], v[8 * e + 1]), pack_bf16x2(v[8 * e + 2], v[8 * e + 3]),
                             pack_bf16x2(v[8 * e + 4], v[8 * e + 5]), pack_bf16x2(v[8 * e + 6], v[8 * e + 7]));
            }
            if (!last) {
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] *= keep;
              tmem_st32(tm + lanes + T_S + 32 * x, v);
            }
          }
          tmem_st_wait();
        }
        fence_async_smem();
        fence_before_sync();
        mbar_arrive(w_ready);
        ++wn;
        if (last) continue;
        const float2 bs = hl[st * C + r], be = hl[st * C + C - 1];
        const float w = exp2f((be.x - bs.x) + (be.y - bs.y));
        const unsigned char *sv = sm + st * L::STAGE + 2 * L::QT;
#pragma unroll 1
        for (int x = 0; x < 2 && ok; ++x) {
          ok = wait(w_free, wn - 1, SITE_ROWS + 13);
          if (!ok) break;
#pragma unroll
          for (int c = 0; c < DV / 8; ++c) {
            const uint32_t at = row_tile_chunk(r, c >> 3, c & 7, C);
            float f[8];
            unpack8(*reinterpret_cast<const uint4 *>(sv + at), f);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] *= w;
            uint4 u = take_bf16(f);
            if (x) u = take_bf16(f);
            *reinterpret_cast<uint4 *>(sm + L::W + at) = u;
          }
          fence_async_smem();
          mbar_arrive(w_ready);
          ++wn;
        }
      }
    }
  }
  fence_before_sync();
  __syncthreads();
  if (warp == 8) {
    fence_after_sync();
    tmem_dealloc(tm, 512);
  }
}

// ============================================================ host
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
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

// [N, heads, d] bf16 in boxes of 128 rows of one head and 64 columns, 128-byte swizzle.
bool encode(CUtensorMap *map, const void *ptr, int d, int heads, int N) {
  auto fn = encoder();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)N};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)d * 2 * heads};
  const cuuint32_t box[3] = {64u, 1u, (cuuint32_t)C}, one[3] = {1u, 1u, 1u};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int sm_count() {
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

// Chunks in a segment: the count with the shortest expected run, in chunk times: rounds of items over the
// SMs, each item `per` chunks and about two more (fill of the pipeline, its state in and out).
int segment_chunks(int N, int B, int H) {
  int best = 1;
  double cost = 1e300;
  for (int per = 1; per <= 32; ++per) {
    const double items = ((double)N / (C * per) + 0.5 * B) * H;
    const double rounds = std::ceil(items / 148.0);
    const double c = rounds * (per + 2.0);
    if (c < cost * 0.999) {
      cost = c;
      best = per;
    }
  }
  return best;
}

template <int DK, int DV>
cudaError_t launch(const LinearParams &p, const Maps &maps, const int *sbase, float *part, float *whole, int per,
                   size_t segs, cudaStream_t s) {
  const size_t items = segs * p.H;
  if (items > 0x7FFFFFFFull) return cudaErrorInvalidValue;
  const unsigned grid = (unsigned)(items < (size_t)sm_count() ? items : (size_t)sm_count());
  cudaError_t e = cudaFuncSetAttribute(parts_kernel<DK, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)PartsSmem<DK, DV>::END);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(rows_kernel<DK, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)RowsSmem<DK, DV>::END);
  if (e != cudaSuccess) return e;
  if (grid) parts_kernel<DK, DV><<<grid, kPartsThreads, PartsSmem<DK, DV>::END, s>>>(p, maps, sbase, part, whole, per);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if ((e = launch_linear_chain(p, sbase, part, nullptr, whole, s)) != cudaSuccess) return e;
  if (grid) rows_kernel<DK, DV><<<grid, kRowsThreads, RowsSmem<DK, DV>::END, s>>>(p, maps, sbase, part, per);
  return cudaGetLastError();
}

}  // namespace lintc

size_t linear_prefill_tc_workspace(const LinearParams &p) {
  using namespace lintc;
  const size_t segs = lin::max_segments(p.N, p.num_seqs, C * segment_chunks(p.N, p.num_seqs, p.H));
  return lin::table_bytes(p.num_seqs) + lin::align256(segs * p.H * 4) + segs * p.H * (size_t)p.dk * p.dv * 4;
}

cudaError_t launch_linear_prefill_tc(const LinearParams &p, cudaStream_t s) {
  using namespace lintc;
  const int per = segment_chunks(p.N, p.num_seqs, p.H);
  const size_t segs = p.N > 0 ? lin::max_segments(p.N, p.num_seqs, C * per) : 0;
  unsigned char *w = static_cast<unsigned char *>(p.ws);
  int *sbase = reinterpret_cast<int *>(w);
  float *whole = reinterpret_cast<float *>(w + lin::table_bytes(p.num_seqs));
  float *part = reinterpret_cast<float *>(w + lin::table_bytes(p.num_seqs) + lin::align256(segs * p.H * 4));
  cudaError_t e = launch_linear_plan(p, sbase, C * per, s);
  if (e != cudaSuccess) return e;
  Maps maps{};
  if (p.N > 0 && !(encode(&maps.q, p.q, p.dk, p.Hk, p.N) && encode(&maps.k, p.k, p.dk, p.Hk, p.N) &&
                   encode(&maps.v, p.v, p.dv, p.H, p.N) && encode(&maps.o, p.o, p.dv, p.H, p.N)))
    return cudaErrorNotSupported;
  if (p.dk == 128)
    return p.dv == 128 ? launch<128, 128>(p, maps, sbase, part, whole, per, segs, s)
                       : launch<128, 64>(p, maps, sbase, part, whole, per, segs, s);
  return p.dv == 128 ? launch<64, 128>(p, maps, sbase, part, whole, per, segs, s)
                     : launch<64, 64>(p, maps, sbase, part, whole, per, segs, s);
}

}  // namespace kda
