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
#include <cmath>

#include "kda_linear_tc.cuh"

namespace kda {
namespace lintc {

// Wait sites reported with a timeout.
enum : unsigned { SITE_PARTS = 41, SITE_ROWS = 51 };

struct Maps {
  CUtensorMap q, k, v, o;
};

// ============================================================ parts
// A ring of four steps: the preparing warp decides which chunk of which segment comes next and writes its
// weights; the others follow.  It goes from a segment's last chunk to its first and stops once every
// weight that is left is 0 in fp32 (decays of 2^-151 and less): those rows are not read, their share is 0.
constexpr int kPartsThreads = 8 * 32 + 64;      // two warpgroups, a TMA + MMA warp, a preparing warp
constexpr int kRing = 4;

struct PartsStep {
  int item;           // segment x H + h; -1: no more
  int pos;            // first row of the chunk
  int h;
  int first, last;    // of the item's chunks, in the order taken
};

template <int DK, int DV>
struct PartsSmem {
  static constexpr uint32_t KT = C * DK * 2, VT = C * DV * 2;
  static constexpr uint32_t STAGE = KT + VT, W = 2 * STAGE;          // W: the three parts of w V
  // DK = 64: the MMA's rows 64 .. 127 come from the bytes after the K tile and are not used
  static constexpr uint32_t WGT = W + 3 * VT, VALID = WGT + kRing * C * 4, STEPS = VALID + kRing * 16;
  static constexpr uint32_t BARS = STEPS + kRing * 32, END = BARS + 20 * 8;
  static_assert(END <= 232448, "shared memory of a block");
};

template <int DK, int DV>
__global__ void __launch_bounds__(kPartsThreads, 1)
parts_kernel(LinearParams p, const __grid_constant__ Maps maps, const int *sbase, float *part, float *whole,
             int per) {
  using L = PartsSmem<DK, DV>;
  extern __shared__ __align__(1024) unsigned char sm[];
  if (device_error_latched(p.err)) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  float *wgt = reinterpret_cast<float *>(sm + L::WGT);
  uint32_t *valid = reinterpret_cast<uint32_t *>(sm + L::VALID);
  volatile PartsStep *steps = reinterpret_cast<volatile PartsStep *>(sm + L::STEPS);
  uint64_t *full = reinterpret_cast<uint64_t *>(sm + L::BARS), *empty = full + 2, *planned = full + 4,
           *done = planned + kRing, *w_ready = done + kRing, *w_free = w_ready + 1, *s_done = w_ready + 2,
           *s_free = s_done + 2, *drain = s_free + 2;
  uint32_t *tmem_sh = reinterpret_cast<uint32_t *>(drain + 1);
  volatile int *failed = reinterpret_cast<volatile int *>(tmem_sh + 1);
  if (warp == 8) tmem_alloc(tmem_sh, 512);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
      mbar_init(s_done + i, 1);
      mbar_init(s_free + i, 256);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(planned + i, 1);
      mbar_init(done + i, 1);
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
  constexpr int kCols = 256;      // TMEM columns of an item's accumulators: DV of w V's first part, DV of the others

  if (warp == 8) {
    // ---------------- loads and MMAs (one thread)
    if (lane == 0) {
      int loaded = 0, n = 0;
      bool ok = true, more = true;
      auto load_next = [&]() {
        if (!more || !ok) return;
        const int rs = loaded % kRing, st = loaded & 1;
        ok = wait(planned + rs, loaded / kRing, SITE_PARTS);
        if (!ok) return;
        const int pos = steps[rs].pos, h = steps[rs].h;
        if (steps[rs].item < 0) { more = false; return; }
        if (loaded >= 2) ok = wait(empty + st, (loaded >> 1) - 1, SITE_PARTS + 1);
        if (!ok) return;
        mbar_arrive_expect_tx(full + st, L::STAGE);
        const uint32_t dst = smem_u32(sm + st * L::STAGE);
#pragma unroll
        for (int kb = 0; kb < DK / 64; ++kb) tma_load_3d(dst + kb * C * 128, &maps.k, kb * 64, h / G, pos, full + st);
#pragma unroll
        for (int kb = 0; kb < DV / 64; ++kb)
          tma_load_3d(dst + L::KT + kb * C * 128, &maps.v, kb * 64, h, pos, full + st);
        ++loaded;
      };
      load_next();
      for (int step = 0; ok && step < loaded; ++step) {
        load_next();
        const int st = step & 1, rs = step % kRing, acc = n & 1;
        const bool first = steps[rs].first != 0, last = steps[rs].last != 0;
        if (first && n >= 2) ok = ok && wait(s_free + acc, (n >> 1) - 1, SITE_PARTS + 2);
        ok = ok && wait(w_ready, step, SITE_PARTS + 3);
        if (!ok) break;
        fence_after_sync();
        const uint32_t sk = smem_u32(sm + st * L::STAGE), sw = smem_u32(sm + L::W), d = tm + acc * kCols;
        if constexpr (DV == 128) {      // first two parts side by side (N = 256), the third into the second's sum
#pragma unroll
          for (int s = 0; s < C / 16; ++s)
            mma_bf16(d, desc_mnmajor(sk, C, 0, s), desc_mnmajor(sw, C, 0, s), idesc_bf16(128, 256, 1, 1), !first || s > 0);
#pragma unroll
          for (int s = 0; s < C / 16; ++s)
            mma_bf16(d + DV, desc_mnmajor(sk, C, 0, s), desc_mnmajor(sw + 2 * L::VT, C, 0, s), idesc_bf16(128, DV, 1, 1), 1);
        } else {
#pragma unroll
          for (int s = 0; s < C / 16; ++s)
            mma_bf16(d, desc_mnmajor(sk, C, 0, s), desc_mnmajor(sw, C, 0, s), idesc_bf16(128, 3 * DV, 1, 1), !first || s > 0);
        }
        mma_commit(w_free);
        mma_commit(empty + st);
        mma_commit(done + rs);
        if (last) {
          mma_commit(s_done + acc);
          ++n;
        }
      }
      if (!ok)      // loads in flight land before the block ends
        for (int i = 0; i < loaded; ++i) mbar_wait(full + (i & 1), (i >> 1) & 1, 2000000);
      mma_commit(drain);
      mbar_wait(drain, 0, p.wait_cycles);
    }
  } else if (warp == 9) {
    // ---------------- the plan
    const int nitems = sbase[p.num_seqs] * p.H;
    int step = 0;
    bool ok = true;
    auto publish = [&](int item, int pos, int h, bool first, bool last) {      // entry reserved by the caller
      if (lane == 0) {
        volatile PartsStep &e = steps[step % kRing];
        e.item = item;
        e.pos = pos;
        e.h = h;
        e.first = first;
        e.last = last;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(planned + step % kRing);
      ++step;
    };
    auto reserve = [&]() {
      if (step >= kRing) ok = wait(done + step % kRing, step / kRing - 1, SITE_PARTS + 4);
      ok = __all_sync(0xFFFFFFFFu, ok);
      return ok;
    };
    for (int i = blockIdx.x; i < nitems && ok; i += gridDim.x) {
      const Segment sg = lin::locate(p.cu, sbase, p.num_seqs, i / p.H, per * C);
      // the last segment of a sequence matters to the final state only
      if (sg.last && p.final_state == nullptr) continue;
      const int chunks = (sg.end - sg.begin + C - 1) / C, h = i % p.H;
      double after = 0.0;
      RawDecays raw = load_decays(p, sg.begin + (chunks - 1) * C, sg.end, h);
      for (int j = chunks - 1; j >= 0; --j) {
        const RawDecays now = raw;
        if (j > 0) raw = load_decays(p, sg.begin + (j - 1) * C, sg.end, h);
        double b[4], total;
        uint32_t word;
        scan_decays(now, b, total, word);
        if (!reserve()) break;
        const int rs = step % kRing;
        float4 w;
        w.x = ex2((float)(after + (total - b[0])));
        w.y = ex2((float)(after + (total - b[1])));
        w.z = ex2((float)(after + (total - b[2])));
        w.w = ex2((float)(after + (total - b[3])));
        reinterpret_cast<float4 *>(wgt + rs * C)[lane] = w;
        if ((lane & 7) == 0) valid[4 * rs + (lane >> 3)] = word;
        after += total;
        const bool last = j == 0 || after < -151.0;
        publish(i, sg.begin + j * C, h, j == chunks - 1, last);
        if (last) break;
      }
      if (lane == 0) whole[i] = ex2((float)after);
    }
    if (ok && reserve()) publish(-1, 0, 0, false, false);
  } else {
    // ---------------- w V in three parts; at a segment's end the state to global memory
    const int r = tid & 127, half = tid >> 7;          // row of the chunk (of the state), column half
    constexpr int NC = DV / 16;                        // 16-byte words of the half
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    int n = 0;
    for (int step = 0;; ++step) {
      const int st = step & 1, rs = step % kRing, acc = n & 1;
      if (!wait.warp(planned + rs, step / kRing, SITE_PARTS + 5)) break;
      const int item = steps[rs].item;
      if (item < 0) break;
      const bool last = steps[rs].last != 0, real = (valid[4 * rs + (r >> 5)] >> (r & 31)) & 1;
      const float w = wgt[rs * C + r];
      if (!wait.warp(full + st, step >> 1, SITE_PARTS + 6)) break;
      unsigned char *sk = sm + st * L::STAGE, *sv = sk + L::KT;
      uint4 u[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int cc = half * NC + c;
        u[c] = real ? *reinterpret_cast<const uint4 *>(sv + row_tile_chunk(r, cc >> 3, cc & 7, C)) : make_uint4(0, 0, 0, 0);
      }
      if (!real)
        for (int c = 0; c < DK / 16; ++c) {
          const int cc = half * (DK / 16) + c;
          *reinterpret_cast<uint4 *>(sk + row_tile_chunk(r, cc >> 3, cc & 7, C)) = make_uint4(0, 0, 0, 0);
        }
      if (step > 0 && !wait.warp(w_free, step - 1, SITE_PARTS + 7)) break;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int cc = half * NC + c;
        const uint32_t at = row_tile_chunk(r, cc >> 3, cc & 7, C);
        float f[8];
        unpack8(u[c], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= w;
#pragma unroll
        for (int x = 0; x < 3; ++x) *reinterpret_cast<uint4 *>(sm + L::W + x * L::VT + at) = take_bf16(f);
      }
      fence_async_smem();
      mbar_arrive(w_ready);
      if (!last) continue;
      if (!wait.warp(s_done + acc, n >> 1, SITE_PARTS + 8)) break;
      fence_after_sync();
      float *out = part + ((size_t)item * DK + r) * DV + half * (DV / 2);
#pragma unroll
      for (int c = 0; c < DV / 64; ++c) {
        const uint32_t col = tm + lanes + acc * kCols + half * (DV / 2) + c * 32;
        uint32_t x[32], y[32];
        float v[32];
        tmem_ld32_issue(col, x);
        tmem_ld32_issue(col + DV, y);
        tmem_ld32_wait(x);
        tmem_ld32_wait(y);
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(x[e]) + __uint_as_float(y[e]);
        if constexpr (DV == 64) {
          tmem_ld32_issue(col + 2 * DV, x);
          tmem_ld32_wait(x);
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] += __uint_as_float(x[e]);
        }
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
    tmem_dealloc(tm, 512);
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
  static constexpr uint32_t BARS = WHOLE + 8, END = BARS + 16 * 8;
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
           *o_free = full + 11, *drain = full + 12, *o_staged = full + 14;
  uint32_t *tmem_sh = reinterpret_cast<uint32_t *>(full + 13);
  volatile int *failed = reinterpret_cast<volatile int *>(tmem_sh + 1);
  if (warp == 8) tmem_alloc(tmem_sh, 512);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(full + i, 1);
      mbar_init(ready + i, 1);
      mbar_init(empty + i, 1);
      mbar_init(o_staged + i, 128);
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
    // ---------------- loads, and stores of whole chunks (from the q tile, and k's where o is wider)
    if (lane == 0) {
      bool ok = true;
      int done_pos[2] = {-1, -1}, done_h[2] = {0, 0};            // the chunk in each stage; pos < 0: its rows were stored directly
      auto retire = [&](int x) {             // chunk number x: its output leaves the stage
        const int st = x & 1;
        ok = ok && wait(o_staged + st, x >> 1, SITE_ROWS);
        if (!ok || done_pos[st] < 0) return;
#pragma unroll
        for (int kb = 0; kb < DV / 64; ++kb)
          tma_store_3d(&maps.o, smem_u32(sm + st * L::STAGE) + kb * C * 128, kb * 64, done_h[st], done_pos[st]);
        bulk_commit();
        bulk_wait_read();
      };
      for (int i = blockIdx.x; i < nitems && ok; i += gridDim.x) {
        const Segment sg = lin::locate(p.cu, sbase, p.num_seqs, i / p.H, per * C);
        const int h = i % p.H;
        for (int pos = sg.begin; pos < sg.end && ok; pos += C, ++step) {
          const int st = step & 1;
          const uint32_t dst = smem_u32(sm + st * L::STAGE);
          if (step >= 2) ok = wait(empty + st, (step >> 1) - 1, SITE_ROWS + 14);
          if (!ok) break;
          mbar_arrive_expect_tx(full + st, L::STAGE);
#pragma unroll
          for (int kb = 0; kb < DV / 64; ++kb)
            tma_load_3d(dst + 2 * L::QT + kb * C * 128, &maps.v, kb * 64, h, pos, full + st);
          if constexpr (DV <= DK)
#pragma unroll
            for (int kb = 0; kb < DK / 64; ++kb)
              tma_load_3d(dst + L::QT + kb * C * 128, &maps.k, kb * 64, h / G, pos, full + st);
          if (step >= 2) retire(step - 2);
          // (a failed wait leaves q's bytes missing: the chunk is never used)
          if (!ok) break;
          if constexpr (DV > DK)
#pragma unroll
            for (int kb = 0; kb < DK / 64; ++kb)
              tma_load_3d(dst + L::QT + kb * C * 128, &maps.k, kb * 64, h / G, pos, full + st);
#pragma unroll
          for (int kb = 0; kb < DK / 64; ++kb)
            tma_load_3d(dst + kb * C * 128, &maps.q, kb * 64, h / G, pos, full + st);
          done_pos[st] = pos + C <= sg.end ? pos : -1;
          done_h[st] = h;
        }
      }
      for (int x = step > 2 ? step - 2 : 0; x < step; ++x) retire(x);
      bulk_wait_all();
      if (!ok)      // loads in flight land before the block ends
        for (int i = 0; i <= step; ++i) mbar_wait(full + (i & 1), (i >> 1) & 1, 2000000);
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
    // ---------------- decays and rows to clear; the next chunk's decays are loaded a chunk ahead
    bool ok = true;
    int ni = blockIdx.x, npos = 0;           // the chunk whose decays are on their way
    Segment ns{};
    auto next = [&]() {
      RawDecays d{};
      if (ni >= nitems) return d;
      d = load_decays(p, npos, ns.end, ni % p.H);
      npos += C;
      if (npos >= ns.end && (ni += gridDim.x) < nitems) {
        ns = lin::locate(p.cu, sbase, p.num_seqs, ni / p.H, per * C);
        npos = ns.begin;
      }
      return d;
    };
    if (ni < nitems) {
      ns = lin::locate(p.cu, sbase, p.num_seqs, ni / p.H, per * C);
      npos = ns.begin;
    }
    RawDecays raw = next();
    for (int i = blockIdx.x; i < nitems && ok; i += gridDim.x) {
      const Segment sg = lin::locate(p.cu, sbase, p.num_seqs, i / p.H, per * C);
      for (int pos = sg.begin; pos < sg.end && ok; pos += C, ++step) {
        const int st = step & 1;
        double b[4], total;
        uint32_t word;
        const RawDecays now = raw;
        raw = next();
        const bool clean = scan_decays(now, b, total, word);
        // the stage's MMAs are done, and its output (which reads the tables) is staged
        if (step >= 2)
          ok = wait(empty + st, (step >> 1) - 1, SITE_ROWS + 6) && wait(o_staged + st, (step >> 1) - 1, SITE_ROWS + 15);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        if ((lane & 7) == 0) valid[4 * st + (lane >> 3)] = word;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float hi = (float)b[e];
          hl[st * C + 4 * lane + e] = make_float2(hi, (float)(b[e] - (double)hi));
        }
        if (lane == 0) whole[st] = ex2((float)total);
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
        ok = wait.warp(ready + st, step >> 1, SITE_ROWS + 8);
        if (!ok) break;
        const float2 *d = hl + st * C;
        const float2 bt = d[t], ref = d[warp > 0 ? 32 * warp - 1 : 0];
        const float rowf = ex2((bt.x - ref.x) + (bt.y - ref.y)), from = ex2(bt.x + bt.y);
        for (int x = 0; x < warp; ++x) {
          const float2 bs = d[32 * x + lane];
          colf[32 * x + lane] = ex2((ref.x - bs.x) + (ref.y - bs.y));
        }
        __syncwarp();
        const bool real = (valid[4 * st + warp] >> lane) & 1;
        ok = wait.warp(a_done, step, SITE_ROWS + 9);
        if (!ok) break;
        fence_after_sync();
        const uint32_t acol = tm + lanes + T_A;
        {
          // the diagonal's 32 columns: each pair by itself
          uint32_t a[32];
          float w[16];
          tmem_ld32_issue(acol + 32 * warp, a);
          float f[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float2 bs = d[32 * warp + e];
            f[e] = ex2(fminf((bt.x - bs.x) + (bt.y - bs.y), 0.f));
          }
          tmem_ld32_wait(a);
          // P's columns 16 x .. lie under A's 16 x .., which A's first pieces must have left
          uint32_t o[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) f[e] = e <= lane ? __uint_as_float(a[e]) * f[e] : 0.f;
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = __uint_as_float(pack_bf16x2(f[2 * e], f[2 * e + 1]));
#pragma unroll
          for (int x = 0; x < 3; ++x) {
            if (x < warp) {
              tmem_ld32_issue(acol + 32 * x, o);
              float g[16];
              tmem_ld32_wait(o);
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float4 c = *reinterpret_cast<const float4 *>(colf + 32 * x + e);
                g[e / 2] = __uint_as_float(pack_bf16x2(__uint_as_float(o[e]) * (rowf * c.x), __uint_as_float(o[e + 1]) * (rowf * c.y)));
                g[e / 2 + 1] = __uint_as_float(pack_bf16x2(__uint_as_float(o[e + 2]) * (rowf * c.z), __uint_as_float(o[e + 3]) * (rowf * c.w)));
              }
              tmem_st16(acol + 16 * x, g);
            }
          }
          tmem_st16(acol + 16 * warp, w);
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = 0.f;
          for (int x = warp + 1; x < 4; ++x) tmem_st16(acol + 16 * x, w);
        }
        tmem_st_wait();
        fence_before_sync();
        mbar_arrive(p_ready);
        ok = wait.warp(o_done, step, SITE_ROWS + 10);
        if (!ok) break;
        fence_after_sync();
        unsigned char *tile = sm + st * L::STAGE;           // q's (and k's) tile: no longer read
        const bool whole_chunk = pos + C <= sg.end;
        uint16_t *orow = reinterpret_cast<uint16_t *>(p.o) + ((size_t)(pos + t) * p.H + h) * DV;
        uint32_t a[2][32], b[2][32];
        tmem_ld32_issue(tm + lanes + T_O1, a[0]);
        tmem_ld32_issue(tm + lanes + T_O2, b[0]);
#pragma unroll
        for (int x = 0; x < DV / 32; ++x) {
          tmem_ld32_wait(a[x & 1]);
          tmem_ld32_wait(b[x & 1]);
          if (x + 1 < DV / 32) {
            tmem_ld32_issue(tm + lanes + T_O1 + 32 * (x + 1), a[(x + 1) & 1]);
            tmem_ld32_issue(tm + lanes + T_O2 + 32 * (x + 1), b[(x + 1) & 1]);
          }
          float f[32];
#pragma unroll
          for (int e = 0; e < 32; ++e)
            f[e] = real ? fmaf(from, __uint_as_float(a[x & 1][e]), __uint_as_float(b[x & 1][e])) : 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint4 u = make_uint4(pack_bf16x2(f[8 * e], f[8 * e + 1]), pack_bf16x2(f[8 * e + 2], f[8 * e + 3]),
                                       pack_bf16x2(f[8 * e + 4], f[8 * e + 5]), pack_bf16x2(f[8 * e + 6], f[8 * e + 7]));
            const int cc = 4 * x + e;
            if (whole_chunk) *reinterpret_cast<uint4 *>(tile + row_tile_chunk(t, cc >> 3, cc & 7, C)) = u;
            else if (pos + t < sg.end) *reinterpret_cast<uint4 *>(orow + 8 * cc) = u;
          }
        }
        fence_before_sync();
        mbar_arrive(o_free);
        if (whole_chunk) fence_async_smem();
        mbar_arrive(o_staged + st);
      }
    }
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
        ok = wait.warp(ready + st, step >> 1, SITE_ROWS + 11);
        if (wn > 0) ok = ok && wait.warp(w_free, wn - 1, SITE_ROWS + 12);      // also: S has its last sum
        if (!ok) break;
        fence_after_sync();
        const float keep = whole[st];
        const float *in = start + ((size_t)i * DK + r) * DV;
        if (r < DK) {
#pragma unroll
          for (int x = 0; x < DV / 32; x += 2) {       // 64 columns at a time
            uint32_t v[2][32];
            if (first) {
#pragma unroll
              for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                  *reinterpret_cast<uint4 *>(&v[y][e]) = __ldcs(reinterpret_cast<const uint4 *>(in + 32 * (x + y) + e));
            } else {
              tmem_ld32_issue(tm + lanes + T_S + 32 * x, v[0]);
              tmem_ld32_issue(tm + lanes + T_S + 32 * (x + 1), v[1]);
              tmem_ld32_wait(v[0]);
              tmem_ld32_wait(v[1]);
            }
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              float f[32];
#pragma unroll
              for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(v[y][e]);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int cc = 4 * (x + y) + e;
                *reinterpret_cast<uint4 *>(sm + L::W + row_tile_chunk(r, cc >> 3, cc & 7, DK)) =
                    make_uint4(pack_bf16x2(f[8 * e], f[8 * e + 1]), pack_bf16x2(f[8 * e + 2], f[8 * e + 3]),
                               pack_bf16x2(f[8 * e + 4], f[8 * e + 5]), pack_bf16x2(f[8 * e + 6], f[8 * e + 7]));
              }
              if (!last) {
#pragma unroll
                for (int e = 0; e < 32; ++e) f[e] *= keep;
                tmem_st32(tm + lanes + T_S + 32 * (x + y), f);
              }
            }
          }
          tmem_st_wait();
        }
        fence_async_smem();
        fence_before_sync();
        mbar_arrive(w_ready);
        ++wn;
        if (last) continue;
        // both parts of w V while Q S runs; each goes to W as the product before it is done
        const float2 bs = hl[st * C + r], be = hl[st * C + C - 1];
        const float w = ex2((be.x - bs.x) + (be.y - bs.y));
        const unsigned char *sv = sm + st * L::STAGE + 2 * L::QT;
        uint4 hi[DV / 8], lo[DV / 8];
#pragma unroll
        for (int c = 0; c < DV / 8; ++c) hi[c] = *reinterpret_cast<const uint4 *>(sv + row_tile_chunk(r, c >> 3, c & 7, C));
#pragma unroll
        for (int c = 0; c < DV / 8; ++c) {
          float f[8];
          unpack8(hi[c], f);
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] *= w;
          hi[c] = take_bf16(f);
          lo[c] = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          ok = ok && wait.warp(w_free, wn - 1, SITE_ROWS + 13);
          if (ok) {
#pragma unroll
            for (int c = 0; c < DV / 8; ++c)
              *reinterpret_cast<uint4 *>(sm + L::W + row_tile_chunk(r, c >> 3, c & 7, C)) = x ? lo[c] : hi[c];
            fence_async_smem();
            mbar_arrive(w_ready);
            ++wn;
          }
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
