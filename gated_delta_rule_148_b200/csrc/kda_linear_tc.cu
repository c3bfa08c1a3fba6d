// Linear attention with a decay for each head on the tensor cores (bf16 inputs): prefill.
// Formulas in kda_linear.cuh; chunks of 128 rows, segments of `per` chunks.
//
//   parts   a segment's contribution to the state, sum_s w_s k_s v_s^T with w_s = 2^{b_end - b_s}:
//           the chunks of a segment from the last to the first, so that w needs no second
//           look at the decays, all accumulated in TMEM:  S += K^T (w V).  w V is split into
//           three bf16 parts (24 bits), so the states keep fp32 accuracy.  REVERSE: the same over q and grad_o from a
//           segment's first chunk on, w_t = 2^{b_t}: its share of the state's gradient at its start.
//   chain   states at the segments' starts (chain_kernel, kda_linear.cu)
//   rows    per chunk  A = Q K^T,  P = A o 2^{b_t - b_s} (bf16, TMEM),  O1 = Q S,  O2 = P V,
//           o = 2^{b_t} O1 + O2,  S <- 2^{b_C} S + K^T (w V), w V in two bf16 parts (2^-17: it only
//           feeds the bf16 operand S of the segment's later chunks).
// Both are persistent blocks with roles: a load warp, an MMA thread, a warp that prepares a chunk's decays, and four
// warpgroups that move accumulators and operands, each a quarter of the columns.  Rows that are pads or belong to the
// next sequence are cleared or masked by their own threads.  Off the diagonal a warp's 32 rows share a reference row R
// before them, 2^{b_t - b_s} = 2^{b_t - R} 2^{R - b_s}, both factors <= 1: one exponential per row and column
// instead of one per pair.
// 131072 tokens, 32 heads, d = 128: shares 78 us where the decays end a share after about five chunks (a mean log of
// -0.18 a token), 560 us where they walk whole segments (-2^-8 a token: keys and values are read twice, 2.1 GB more);
// chain 16 us, rows 1.02 ms (4.3 GB).  Rows is bound by turns of products and warpgroups (the tensor pipe is busy a third
// of the time; 1.04 ms without any load or store, 0.67 ms for these alone), then by power: SM clocks fall to 1.7 - 1.85 GHz.  Chunks of 128: a state's way through TMEM and shared memory
// costs the same for any chunk, the pairs inside grow with it, and 128 rows are the products' own height.
#include <cmath>

#include "kda_linear_tc.cuh"

namespace kda {
namespace lintc {

// Wait sites reported with a timeout.
enum : unsigned { SITE_PARTS = 41, SITE_ROWS = 55 };

struct Maps {
  CUtensorMap q, k, v, o, part;
};

// ============================================================ parts
// A ring of four steps: the preparing warp decides which chunk of which segment comes next and writes its
// weights; the others follow.  It goes from a segment's last chunk to its first (or back) and stops once every
// weight that is left is 0 in fp32 (decays of 2^-151 and less): those rows are not read, their share is 0.
constexpr int kPartsThreads = 16 * 32 + 64;     // four warpgroups, a TMA + MMA warp, a preparing warp
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
  static constexpr uint32_t STAGE = KT + VT, W = 2 * STAGE;          // W: the three parts of w V; the state on its way out
  // DK = 64: the MMA's rows 64 .. 127 come from the bytes after the K tile and are not used
  static constexpr uint32_t WGT = W + 3 * VT, VALID = WGT + kRing * C * 4, STEPS = VALID + kRing * 16;
  static constexpr uint32_t BARS = STEPS + kRing * 32, END = BARS + 24 * 8;
  static_assert(END <= 232448, "shared memory of a block");
};

template <int DK, int DV, bool REVERSE>
__global__ void __launch_bounds__(kPartsThreads, 1)
parts_kernel(LinearParams p, const __grid_constant__ Maps maps, const int *sbase, float *whole) {
  using L = PartsSmem<DK, DV>;
  extern __shared__ __align__(1024) unsigned char sm[];
  after_previous();
  if (lin::call_ended(p, sbase)) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  float *wgt = reinterpret_cast<float *>(sm + L::WGT);
  uint32_t *valid = reinterpret_cast<uint32_t *>(sm + L::VALID);
  volatile PartsStep *steps = reinterpret_cast<volatile PartsStep *>(sm + L::STEPS);
  uint64_t *full = reinterpret_cast<uint64_t *>(sm + L::BARS), *empty = full + 2, *planned = full + 4,
           *done = planned + kRing, *w_ready = done + kRing, *w_free = w_ready + 1, *s_done = w_ready + 2,
           *s_free = s_done + 2, *drain = s_free + 2, *staged = drain + 1, *out_free = drain + 2;
  uint32_t *tmem_sh = reinterpret_cast<uint32_t *>(drain + 3);
  volatile int *failed = reinterpret_cast<volatile int *>(tmem_sh + 1);
  if (warp == 16) tmem_alloc(tmem_sh, 512);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
      mbar_init(s_done + i, 1);
      mbar_init(s_free + i, 512);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(planned + i, 1);
      mbar_init(done + i, 1);
    }
    mbar_init(w_ready, 512);
    mbar_init(w_free, 1);
    mbar_init(staged, 512);
    mbar_init(out_free, 1);
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

  if (warp == 16) {
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
        ok = ok && wait(full + st, step >> 1, SITE_PARTS + 3) && wait(w_ready, step, SITE_PARTS + 3);
        if (!ok) break;
        fence_after_sync();
        const uint32_t d = tm + acc * kCols;
        const uint64_t k = desc_mnmajor(smem_u32(sm + st * L::STAGE), C, 0, 0), v = desc_mnmajor(smem_u32(sm + L::W), C, 0, 0);
        if constexpr (DV == 128) {      // first two parts side by side (N = 256), the third into the second's sum
          const uint64_t v2 = desc_mnmajor(smem_u32(sm + L::W + 2 * L::VT), C, 0, 0);
#pragma unroll
          for (int s = 0; s < C / 16; ++s)
            mma_bf16(d, mnmajor_step(k, s), mnmajor_step(v, s), idesc_bf16(128, 256, 1, 1), !first || s > 0);
#pragma unroll
          for (int s = 0; s < C / 16; ++s)
            mma_bf16(d + DV, mnmajor_step(k, s), mnmajor_step(v2, s), idesc_bf16(128, DV, 1, 1), 1);
        } else {
#pragma unroll
          for (int s = 0; s < C / 16; ++s)
            mma_bf16(d, mnmajor_step(k, s), mnmajor_step(v, s), idesc_bf16(128, 3 * DV, 1, 1), !first || s > 0);
        }
        mma_commit(w_free);
        mma_commit(empty + st);
        mma_commit(done + rs);
        if (last) {
          mma_commit(s_done + acc);
          ++n;
        }
      }
      // loads in flight land before the block ends, whoever gave up
      for (int i = loaded > 2 ? loaded - 2 : 0; i < loaded; ++i) mbar_wait(full + (i & 1), (i >> 1) & 1, kDrainCycles);
      mma_commit(drain);
      mbar_wait(drain, 0, kDrainCycles);
    }
  } else if (warp == 17) {
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
    for (int n_i = 0, i; (i = item_of(n_i)) < nitems && ok; ++n_i) {
      const Segment sg = lin::locate(sbase, p.num_seqs, i / p.H);
      // the last segment of a sequence matters to the final state only (the first to the initial state's gradient)
      if (REVERSE ? p.g_init == nullptr && sg.begin == p.cu[sg.seq()] : p.final_state == nullptr && sg.last()) continue;
      const int chunks = (sg.end - sg.begin + C - 1) / C, h = i % p.H;
      double past = 0.0;                     // log2 of the decay over the chunks taken
      auto at = [&](int x) { return sg.begin + (REVERSE ? x : chunks - 1 - x) * C; };
      RawDecays raw = load_decays(p, at(0), sg.end, h);
      for (int x = 0; x < chunks; ++x) {
        const RawDecays now = raw;
        if (x + 1 < chunks) raw = load_decays(p, at(x + 1), sg.end, h);
        double b[4], total;
        uint32_t word;
        scan_decays(now, b, total, word);
        if (!reserve()) break;
        const int rs = step % kRing;
        float4 w;
        w.x = ex2((float)(past + (REVERSE ? b[0] : total - b[0])));
        w.y = ex2((float)(past + (REVERSE ? b[1] : total - b[1])));
        w.z = ex2((float)(past + (REVERSE ? b[2] : total - b[2])));
        w.w = ex2((float)(past + (REVERSE ? b[3] : total - b[3])));
        reinterpret_cast<float4 *>(wgt + rs * C)[lane] = w;
        if ((lane & 7) == 0) valid[4 * rs + (lane >> 3)] = word;
        past += total;
        const bool last = x == chunks - 1 || past < -151.0;
        publish(sg.id * p.H + h, at(x), h, x == 0, last);
        if (last) break;
      }
      // both directions' sums round apart: a segment's factor has one writer
      if (lane == 0 && (!REVERSE || sg.last())) whole[sg.id * p.H + h] = ex2((float)past);
    }
    if (ok && reserve()) publish(-1, 0, 0, false, false);
  } else {
    // ---------------- w V in three parts; at a segment's end the state to global memory
    const int r = tid & 127, part_of = tid >> 7;       // row of the chunk (of the state), quarter of the columns
    constexpr int COLS = DV / 4, NC = COLS / 8;        // columns, 16-byte words of the quarter
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    int n = 0;
    for (int step = 0;; ++step) {
      const int st = step & 1, rs = step % kRing, acc = n & 1;
      if (!wait.warp(planned + rs, step / kRing, SITE_PARTS + 5)) break;
      const int item = steps[rs].item;
      if (item < 0) break;
      const bool first = steps[rs].first != 0, last = steps[rs].last != 0, real = (valid[4 * rs + (r >> 5)] >> (r & 31)) & 1;
      const float w = wgt[rs * C + r];
      if (!wait.warp(full + st, step >> 1, SITE_PARTS + 6)) break;
      unsigned char *sk = sm + st * L::STAGE, *sv = sk + L::KT;
      uint4 u[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int cc = part_of * NC + c;
        u[c] = real ? *reinterpret_cast<const uint4 *>(sv + row_tile_chunk(r, cc >> 3, cc & 7, C)) : make_uint4(0, 0, 0, 0);
      }
      if (!real)
        for (int c = 0; c < DK / 32; ++c) {
          const int cc = part_of * (DK / 32) + c;
          *reinterpret_cast<uint4 *>(sk + row_tile_chunk(r, cc >> 3, cc & 7, C)) = make_uint4(0, 0, 0, 0);
        }
      if (step > 0 && !wait.warp(w_free, step - 1, SITE_PARTS + 7)) break;
      if (first && n > 0 && !wait.warp(out_free, n - 1, SITE_PARTS + 9)) break;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int cc = part_of * NC + c;
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
      const uint32_t col = tm + lanes + acc * kCols + part_of * COLS;
      float v[COLS];
      if constexpr (DV == 128) {
        uint32_t x[32], y[32];
        tmem_ld32_issue(col, x);
        tmem_ld32_issue(col + DV, y);
        tmem_ld32_wait(x);
        tmem_ld32_wait(y);
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(x[e]) + __uint_as_float(y[e]);
      } else {
        uint32_t x[16], y[16], z[16];
        tmem_ld16_issue(col, x);
        tmem_ld16_issue(col + DV, y);
        tmem_ld16_issue(col + 2 * DV, z);
        tmem_ld16_wait(x);
        tmem_ld16_wait(y);
        tmem_ld16_wait(z);
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(x[e]) + (__uint_as_float(y[e]) + __uint_as_float(z[e]));
      }
      fence_before_sync();
      mbar_arrive(s_free + acc);
      if (r < DK)      // tiles of 32 columns with the 128-byte swizzle
#pragma unroll
        for (int e = 0; e < COLS / 4; ++e) {
          const int cc = part_of * (COLS / 4) + e;
          *reinterpret_cast<float4 *>(sm + L::W + row_tile_chunk(r, cc >> 3, cc & 7, DK)) =
              make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        }
      fence_async_smem();
      mbar_arrive(staged);
      bool gone = true;
      if (tid == 0) {
        gone = wait(staged, n, SITE_PARTS + 10);
        if (gone) {
#pragma unroll
          for (int cb = 0; cb < DV / 32; ++cb)
            tma_store_3d(&maps.part, smem_u32(sm + L::W) + cb * DK * 128, cb * 32, 0, item * DK);
          bulk_commit();
          bulk_wait_read();
          mbar_arrive(out_free);
        }
      }
      if (!__all_sync(0xFFFFFFFFu, gone)) break;
      ++n;
    }
    if (tid == 0) bulk_wait_all();
  }
  fence_before_sync();
  __syncthreads();
  if (warp == 16) {
    fence_after_sync();
    tmem_dealloc(tm, 512);
  }
}

// ============================================================ rows
// Four warpgroups that take each step of a chunk together, a quarter of its columns each (a warpgroup for each step
// measured slower: a step then takes four times as long, and few of them run side by side); TMA, MMA and
// preparing warps.
constexpr int kRowsThreads = 16 * 32 + 96;

template <int DK, int DV>
struct RowsSmem {
  static constexpr uint32_t QT = C * DK * 2, VT = C * DV * 2;
  static constexpr uint32_t STAGE = 2 * QT + VT, W = 2 * STAGE;      // W: S, then w V's first part, as bf16
  static constexpr uint32_t WB = (DK > C ? DK : C) * DV * 2;
  // w V's second part: q's tile, which Q S reads last, where it fits
  static constexpr bool kLoInQ = DV <= DK;
  static constexpr uint32_t LO = W + WB;
  static constexpr uint32_t HL = LO + (kLoInQ ? 0 : VT), COLF = HL + 2 * C * 8, VALID = COLF + 192 * 4, WHOLE = VALID + 32;
  static constexpr uint32_t BARS = WHOLE + 8, END = BARS + 18 * 8;
  static_assert(END <= 232448, "shared memory of a block");
};

template <int DK, int DV>
__global__ void __launch_bounds__(kRowsThreads, 1)
rows_kernel(LinearParams p, const __grid_constant__ Maps maps, const int *sbase, const float *start) {
  using L = RowsSmem<DK, DV>;
  extern __shared__ __align__(1024) unsigned char sm[];
  after_previous();
  if (lin::call_ended(p, sbase)) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nitems = sbase[p.num_seqs] * p.H;
  float2 *hl = reinterpret_cast<float2 *>(sm + L::HL);
  uint32_t *valid = reinterpret_cast<uint32_t *>(sm + L::VALID);
  float *whole = reinterpret_cast<float *>(sm + L::WHOLE);
  uint64_t *full = reinterpret_cast<uint64_t *>(sm + L::BARS), *ready = full + 2, *empty = full + 4, *a_done = full + 6,
           *p_ready = full + 7, *w_ready = full + 8, *qs_done = full + 9, *l_ready = full + 10, *s_done = full + 11,
           *drain = full + 13, *o_staged = full + 14;
  uint32_t *tmem_sh = reinterpret_cast<uint32_t *>(full + 16);
  volatile int *failed = reinterpret_cast<volatile int *>(tmem_sh + 1);
  if (warp == 16) tmem_alloc(tmem_sh, 512);
  if (tid == 0) {
    for (int i = 0; i < 14; ++i) mbar_init(full + i, 1);
    for (int i = 0; i < 2; ++i) mbar_init(o_staged + i, 512);
    mbar_init(p_ready, 512);
    mbar_init(w_ready, 512);
    mbar_init(l_ready, 512);
    *failed = 0;
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tm = *tmem_sh;
  constexpr uint32_t T_S = 0, T_A = 128, T_O1 = 256, T_O2 = 384;
  // P overlays A: its columns 32 x .. 32 x + 31 in 32 x .. 32 x + 15
  const Waits wait{p.wait_cycles, p.err, p.site, failed};
  const int G = p.H / p.Hk;
  // items' segments, loaded an item ahead
  auto segment = [&](int i) { return i < nitems ? lin::locate(sbase, p.num_seqs, i / p.H) : Segment{}; };
  Segment next = segment(item_of(0));
  int step = 0, ln = 0;      // chunks; those among them whose S goes on to another

  if (warp == 17) {
    // ---------------- loads, and stores of whole chunks (from the v tile)
    if (lane == 0) {
      bool ok = true;
      int out_pos[2] = {-1, -1}, out_h[2] = {0, 0};      // the chunk in each stage; pos < 0: its rows were stored directly
      auto store = [&](int st, int x) {                  // chunk number x
        ok = ok && wait(o_staged + st, x >> 1, SITE_ROWS + 2);
        if (!ok || out_pos[st] < 0) return;
#pragma unroll
        for (int kb = 0; kb < DV / 64; ++kb)
          tma_store_3d(&maps.o, smem_u32(sm + st * L::STAGE + 2 * L::QT) + kb * C * 128, kb * 64, out_h[st], out_pos[st]);
        bulk_commit();
        bulk_wait_read();
      };
      for (int n_i = 0, i; (i = item_of(n_i)) < nitems && ok; ++n_i) {
        const Segment sg = next;
        next = segment(item_of(n_i + 1));
        const int h = i % p.H;
        for (int pos = sg.begin; pos < sg.end && ok; pos += C, ++step) {
          const int st = step & 1;
          const uint32_t dst = smem_u32(sm + st * L::STAGE);
          if (step >= 2) ok = wait(empty + st, (step >> 1) - 1, SITE_ROWS);
          if (!ok) break;
          mbar_arrive_expect_tx(full + st, L::STAGE);
#pragma unroll
          for (int kb = 0; kb < DK / 64; ++kb) {
            tma_load_3d(dst + L::QT + kb * C * 128, &maps.k, kb * 64, h / G, pos, full + st);
            tma_load_3d(dst + kb * C * 128, &maps.q, kb * 64, h / G, pos, full + st);
          }
          if (step >= 2) store(st, step - 2);
          if (!ok) break;
#pragma unroll
          for (int kb = 0; kb < DV / 64; ++kb)
            tma_load_3d(dst + 2 * L::QT + kb * C * 128, &maps.v, kb * 64, h, pos, full + st);
          out_pos[st] = pos + C <= sg.end ? pos : -1;
          out_h[st] = h;
        }
      }
      for (int x = step > 2 ? step - 2 : 0; x < step; ++x) store(x & 1, x);
      bulk_wait_all();
      // loads in flight (a begun chunk's too) land before the block ends, whoever gave up
      for (int i = step > 2 ? step - 2 : 0; i < step + !ok; ++i) mbar_wait(full + (i & 1), (i >> 1) & 1, kDrainCycles);
    }
  } else if (warp == 16) {
    // ---------------- MMAs: P V, Q S, the next chunk's A, then S's update, so that the next P is on its way meanwhile
    if (lane == 0) {
      bool ok = true;
      const uint32_t sw = smem_u32(sm + L::W);
      const uint32_t stage[2] = {smem_u32(sm), smem_u32(sm + L::STAGE)};
      auto issue_a = [&](int x) {            // chunk number x
        ok = ok && wait(full + (x & 1), x >> 1, SITE_ROWS + 1);
        if (!ok) return;
        fence_after_sync();
        const uint32_t sq = x & 1 ? stage[1] : stage[0];
        const uint64_t q = desc_kmajor(sq, C, 0, 0), k = desc_kmajor(sq + L::QT, C, 0, 0);
#pragma unroll
        for (int s = 0; s < DK / 16; ++s)
          mma_bf16(tm + T_A, kmajor_step<C>(q, s), kmajor_step<C>(k, s), idesc_bf16(128, C, 0, 0), s > 0);
        mma_commit(a_done);
      };
      if (item_of(0) < nitems) issue_a(0);
      for (int n_i = 0, i; (i = item_of(n_i)) < nitems && ok; ++n_i) {
        const Segment sg = next;
        next = segment(item_of(n_i + 1));
        for (int pos = sg.begin; pos < sg.end && ok; pos += C, ++step) {
          const int st = step & 1;
          const bool last = pos + C >= sg.end, more = !last || item_of(n_i + 1) < nitems;
          const uint32_t sq = st ? stage[1] : stage[0], sk = sq + L::QT, sv = sk + L::QT;
          const uint64_t q = desc_kmajor(sq, C, 0, 0), w = desc_mnmajor(sw, DK, 0, 0), k = desc_mnmajor(sk, C, 0, 0),
                         v = desc_mnmajor(sv, C, 0, 0), hi = desc_mnmajor(sw, C, 0, 0),
                         lo = desc_mnmajor(L::kLoInQ ? sq : smem_u32(sm + L::LO), C, 0, 0);
          ok = wait(p_ready, step, SITE_ROWS + 3);
          if (!ok) break;
          fence_after_sync();
#pragma unroll
          for (int s = 0; s < C / 16; ++s)
            mma_bf16_ta(tm + T_O2, tm + T_A + 32 * (s >> 1) + 8 * (s & 1), mnmajor_step(v, s), idesc_bf16(128, DV, 0, 1),
                        s > 0);
          ok = wait(w_ready, step, SITE_ROWS + 4);
          if (!ok) break;
          fence_after_sync();
#pragma unroll
          for (int s = 0; s < DK / 16; ++s)
            mma_bf16(tm + T_O1, kmajor_step<C>(q, s), mnmajor_step(w, s), idesc_bf16(128, DV, 0, 1), s > 0);
          mma_commit(qs_done);
          // (if it is there: else S's update, which the loads wait for, goes first)
          const bool early = more && Waits::test(full + (st ^ 1), ((step + 1) >> 1) & 1);
          if (early) issue_a(step + 1);
          if (!last) {                       // S += K^T (w V)
            ok = ok && wait(l_ready, ln++, SITE_ROWS + 5);
            if (!ok) break;
            fence_after_sync();
#pragma unroll
            for (int s = 0; s < C / 16; ++s)
              mma_bf16(tm + T_S, mnmajor_step(k, s), mnmajor_step(hi, s), idesc_bf16(128, DV, 1, 1), 1);
#pragma unroll
            for (int s = 0; s < C / 16; ++s)
              mma_bf16(tm + T_S, mnmajor_step(k, s), mnmajor_step(lo, s), idesc_bf16(128, DV, 1, 1), 1);
            mma_commit(s_done);
          }
          mma_commit(empty + st);
          if (more && !early) issue_a(step + 1);
        }
      }
      mma_commit(drain);
      mbar_wait(drain, 0, kDrainCycles);
    }
  } else if (warp == 18) {
    // ---------------- decays; the next chunk's are loaded a chunk ahead
    bool ok = true;
    int nk = 0, ni = item_of(0), npos = 0;   // the chunk whose decays are on their way
    Segment ns{};
    auto next = [&]() {
      RawDecays d{};
      if (ni >= nitems) return d;
      d = load_decays(p, npos, ns.end, ni % p.H);
      npos += C;
      if (npos >= ns.end && (ni = item_of(++nk)) < nitems) {
        ns = lin::locate(sbase, p.num_seqs, ni / p.H);
        npos = ns.begin;
      }
      return d;
    };
    if (ni < nitems) {
      ns = lin::locate(sbase, p.num_seqs, ni / p.H);
      npos = ns.begin;
    }
    RawDecays raw = next();
    for (int n_i = 0, i; (i = item_of(n_i)) < nitems && ok; ++n_i) {
      const Segment sg = lin::locate(sbase, p.num_seqs, i / p.H);
      for (int pos = sg.begin; pos < sg.end && ok; pos += C, ++step) {
        const int st = step & 1;
        double b[4], total;
        uint32_t word;
        const RawDecays now = raw;
        raw = next();
        scan_decays(now, b, total, word);
        // the stage's MMAs are done, and with them the readers of its tables
        if (step >= 2) ok = wait(empty + st, (step >> 1) - 1, SITE_ROWS + 6);
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
        if (lane == 0 && ok) mbar_arrive(ready + st);
      }
    }
  } else {
    // ---------------- thread: row r of the chunk, or of the state; warpgroup y: a quarter of the columns
    const int r = tid & 127, w = warp & 3, y = warp >> 2;
    constexpr int COLS = DV / 4;
    const uint32_t lanes = (uint32_t)(w * 32) << 16;
    float *colf = reinterpret_cast<float *>(sm + L::COLF) + (w * (w - 1) / 2 + y) * 32;      // y < w
    bool ok = true;
    for (int n_i = 0, i; (i = item_of(n_i)) < nitems && ok; ++n_i) {
      const Segment sg = next;
      next = segment(item_of(n_i + 1));
      const int h = i % p.H;
      for (int pos = sg.begin; pos < sg.end && ok; pos += C, ++step) {
        const int st = step & 1;
        const bool first = pos == sg.begin, last = pos + C >= sg.end;
        ok = wait.warp(ready + st, step >> 1, SITE_ROWS + 8) && wait.warp(full + st, step >> 1, SITE_ROWS + 7);
        if (!ok) break;
        const float2 *d = hl + st * C;
        const float2 bt = d[r];
        const uint32_t cols = valid[4 * st + y];         // P's columns that are real rows
        const bool real = (valid[4 * st + w] >> lane) & 1;
        unsigned char *tile_k = sm + st * L::STAGE + L::QT, *tile_v = tile_k + L::QT;
        if (!real) {      // a pad or a row of the next sequence: k and v must not reach S nor o (A's column is masked)
#pragma unroll
          for (int e = 0; e < DK / 32; ++e) {
            const int cc = y * (DK / 32) + e;
            *reinterpret_cast<uint4 *>(tile_k + row_tile_chunk(r, cc >> 3, cc & 7, C)) = make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int e = 0; e < COLS / 8; ++e) {
            const int cc = y * (COLS / 8) + e;
            *reinterpret_cast<uint4 *>(tile_v + row_tile_chunk(r, cc >> 3, cc & 7, C)) = make_uint4(0, 0, 0, 0);
          }
          fence_async_smem();
        }
        const float keep = whole[st], from = ex2(bt.x + bt.y);
        float to, rowf = 0.f;
        {
          const float2 be = d[C - 1];
          to = ex2((be.x - bt.x) + (be.y - bt.y));
        }
        if (y < w) {                         // 2^{b_t - b_ref} and 2^{b_ref - b_s}: the row before the warp's rows
          const float2 ref = d[32 * w - 1], bs = d[32 * y + lane];
          rowf = ex2((bt.x - ref.x) + (bt.y - ref.y));
          colf[lane] = ex2((ref.x - bs.x) + (ref.y - bs.y));
        }
        __syncwarp();

        // P's columns 32 y .. 32 y + 31
        ok = wait.warp(a_done, step, SITE_ROWS + 9);
        if (!ok) break;
        fence_after_sync();
        {
          const uint32_t col = tm + lanes + T_A + 32 * y;
          float g[16];
          if (y > w) {
#pragma unroll
            for (int e = 0; e < 16; ++e) g[e] = 0.f;
          } else {
            uint32_t a[32];
            auto mask = [&](uint32_t (&x)[32]) {
              if (cols != 0xFFFFFFFFu)
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] = (cols >> e) & 1 ? x[e] : 0u;
            };
            tmem_ld32_issue(col, a);
            if (y < w) {
              tmem_ld32_wait(a);
              mask(a);
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float4 c = *reinterpret_cast<const float4 *>(colf + e);
                g[e / 2] = __uint_as_float(pack_bf16x2(__uint_as_float(a[e]) * (rowf * c.x), __uint_as_float(a[e + 1]) * (rowf * c.y)));
                g[e / 2 + 1] = __uint_as_float(pack_bf16x2(__uint_as_float(a[e + 2]) * (rowf * c.z), __uint_as_float(a[e + 3]) * (rowf * c.w)));
              }
            } else {                         // the diagonal: each pair by itself
              float f[32];
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const float2 bs = d[32 * y + e];
                f[e] = ex2((bt.x - bs.x) + (bt.y - bs.y));
              }
              tmem_ld32_wait(a);
              mask(a);
#pragma unroll
              for (int e = 0; e < 32; ++e) f[e] = e <= lane ? __uint_as_float(a[e]) * f[e] : 0.f;
#pragma unroll
              for (int e = 0; e < 16; ++e) g[e] = __uint_as_float(pack_bf16x2(f[2 * e], f[2 * e + 1]));
            }
          }
          tmem_st16(col, g);
          tmem_st_wait();
          fence_before_sync();
          mbar_arrive(p_ready);
        }

        // S as an operand; S <- 2^{b_C} S
        if (!first) ok = wait.warp(s_done, ln - 1, SITE_ROWS + 12);
        else if (step > 0) ok = wait.warp(qs_done, step - 1, SITE_ROWS + 13);      // the item before: W is free
        if (!ok) break;
        fence_after_sync();
        if (r < DK) {
          const uint32_t col = tm + lanes + T_S + y * COLS;
          uint32_t v[COLS];
          if (first) {
            const float *in = start + (((size_t)sg.id * p.H + h) * DK + r) * DV + y * COLS;
#pragma unroll
            for (int e = 0; e < COLS; e += 4)
              *reinterpret_cast<uint4 *>(&v[e]) = __ldcs(reinterpret_cast<const uint4 *>(in + e));
          } else if constexpr (COLS == 32) {
            tmem_ld32_issue(col, v);
            tmem_ld32_wait(v);
          } else {
            tmem_ld16_issue(col, v);
            tmem_ld16_wait(v);
          }
          float f[COLS];
#pragma unroll
          for (int e = 0; e < COLS; ++e) f[e] = __uint_as_float(v[e]);
#pragma unroll
          for (int e = 0; e < COLS / 8; ++e) {
            const int cc = y * (COLS / 8) + e;
            *reinterpret_cast<uint4 *>(sm + L::W + row_tile_chunk(r, cc >> 3, cc & 7, DK)) = pack8(f + 8 * e);
          }
          if (!last) {
#pragma unroll
            for (int e = 0; e < COLS; ++e) f[e] *= keep;
            if constexpr (COLS == 32) tmem_st32(col, f);
            else tmem_st16(col, f);
          }
          tmem_st_wait();
        }
        fence_async_smem();
        fence_before_sync();
        mbar_arrive(w_ready);

        // the two parts of w V, once Q S is done
        if (!last) {
          unsigned char *slo = L::kLoInQ ? sm + st * L::STAGE : sm + L::LO;
          ok = wait.warp(qs_done, step, SITE_ROWS + 14);
          if (!ok) break;
#pragma unroll
          for (int e = 0; e < COLS / 8; ++e) {
            const int cc = y * (COLS / 8) + e;
            const uint32_t at = row_tile_chunk(r, cc >> 3, cc & 7, C);
            float f[8];
            unpack8(*reinterpret_cast<const uint4 *>(tile_v + at), f);
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] *= to;
            *reinterpret_cast<uint4 *>(sm + L::W + at) = take_bf16(f);
            *reinterpret_cast<uint4 *>(slo + at) = take_bf16(f);
          }
          fence_async_smem();
          mbar_arrive(l_ready);
          ++ln;
        }

        // the output: into v's tile, each thread over the words that it alone has read and the products no longer need
        ok = wait.warp(qs_done, step, SITE_ROWS + 10);
        if (!ok) break;
        fence_after_sync();
        {
          const bool whole_chunk = pos + C <= sg.end;
          uint16_t *orow = reinterpret_cast<uint16_t *>(p.o) + ((size_t)(pos + r) * p.H + h) * DV;
          uint32_t a[COLS], b[COLS];
          if constexpr (COLS == 32) {
            tmem_ld32_issue(tm + lanes + T_O1 + y * COLS, a);
            tmem_ld32_issue(tm + lanes + T_O2 + y * COLS, b);
            tmem_ld32_wait(a);
            tmem_ld32_wait(b);
          } else {
            tmem_ld16_issue(tm + lanes + T_O1 + y * COLS, a);
            tmem_ld16_issue(tm + lanes + T_O2 + y * COLS, b);
            tmem_ld16_wait(a);
            tmem_ld16_wait(b);
          }
          float f[COLS];
#pragma unroll
          for (int e = 0; e < COLS; ++e) f[e] = fmaf(from, __uint_as_float(a[e]), __uint_as_float(b[e]));
          if (!real)
#pragma unroll
            for (int e = 0; e < COLS; ++e) f[e] = 0.f;
#pragma unroll
          for (int e = 0; e < COLS / 8; ++e) {
            const int cc = y * (COLS / 8) + e;
            if (whole_chunk) *reinterpret_cast<uint4 *>(tile_v + row_tile_chunk(r, cc >> 3, cc & 7, C)) = pack8(f + 8 * e);
            else if (pos + r < sg.end) *reinterpret_cast<uint4 *>(orow + 8 * cc) = pack8(f + 8 * e);
          }
          if (whole_chunk) fence_async_smem();
          mbar_arrive(o_staged + st);
        }
      }
    }
  }
  fence_before_sync();
  __syncthreads();
  if (warp == 16) {
    fence_after_sync();
    tmem_dealloc(tm, 512);
  }
}

// ============================================================ host
// The fewest chunks in a segment that the plan may take: half of what sequences of equal length would have, in rounds of
// segments over the SMs with two chunks' time for each segment's beginning and end.  It bounds the workspace.
int least_chunks(int N, int B, int H) {
  int best = 1;
  double cost = 1e300;
  for (int per = 1; per <= 32; ++per) {
    const double items = ((double)N / (C * per) + 0.5 * B) * H;
    const double c = std::ceil(items / 148.0) * (per + 2.0);
    if (c < cost * 0.999) {
      cost = c;
      best = per;
    }
  }
  return (best + 1) / 2;
}

template <int DK, int DV>
cudaError_t launch(const LinearParams &p, const Maps &maps, const int *sbase, float *part, float *whole,
                   size_t segs, cudaStream_t s) {
  const size_t items = segs * p.H;
  if (items * DK > 0x7FFFFFFFull) return cudaErrorInvalidValue;      // rows of the states as a tensor map's coordinate
  const unsigned grid = (unsigned)(items < (size_t)sm_count() ? items : (size_t)sm_count());
  cudaError_t e = lin::allow_smem<parts_kernel<DK, DV, false>>(PartsSmem<DK, DV>::END);
  if (e == cudaSuccess) e = lin::allow_smem<rows_kernel<DK, DV>>(RowsSmem<DK, DV>::END);
  if (e != cudaSuccess) return e;
  if (grid) e = launch_next(parts_kernel<DK, DV, false>, grid, kPartsThreads, PartsSmem<DK, DV>::END, s, p, maps, sbase, whole);
  if (e == cudaSuccess) e = launch_linear_chain(p, sbase, part, nullptr, whole, s);
  if (e == cudaSuccess && grid)
    e = launch_next(rows_kernel<DK, DV>, grid, kRowsThreads, RowsSmem<DK, DV>::END, s, p, maps, sbase, part);
  return e;
}

template <int DK, int DV>
cudaError_t launch_shares(const LinearParams &p, const Maps &fwd, const Maps &rev, const int *sbase, float *whole,
                          size_t items, cudaStream_t s) {
  if (items * DK > 0x7FFFFFFFull) return cudaErrorInvalidValue;
  const unsigned grid = (unsigned)(items < (size_t)sm_count() ? items : (size_t)sm_count());
  constexpr int smem = PartsSmem<DK, DV>::END;
  cudaError_t e = lin::allow_smem<parts_kernel<DK, DV, false>>(smem);
  if (e == cudaSuccess) e = lin::allow_smem<parts_kernel<DK, DV, true>>(smem);
  if (e == cudaSuccess) e = launch_next(parts_kernel<DK, DV, false>, grid, kPartsThreads, smem, s, p, fwd, sbase, whole);
  if (e == cudaSuccess) e = launch_next(parts_kernel<DK, DV, true>, grid, kPartsThreads, smem, s, p, rev, sbase, whole);
  return e;
}

}  // namespace lintc

size_t linear_prefill_tc_workspace(const LinearParams &p) {
  using namespace lintc;
  const size_t segs = lin::max_segments(p.N, p.num_seqs, C * least_chunks(p.N, p.num_seqs, p.H));
  return lin::table_bytes(p.num_seqs, segs) + lin::align256(segs * p.H * 4) + segs * p.H * (size_t)p.dk * p.dv * 4;
}

cudaError_t launch_linear_prefill_tc(const LinearParams &p, cudaStream_t s) {
  using namespace lintc;
  const int per = least_chunks(p.N, p.num_seqs, p.H);
  const size_t segs = p.N > 0 ? lin::max_segments(p.N, p.num_seqs, C * per) : 0;
  unsigned char *w = static_cast<unsigned char *>(p.ws);
  int *sbase = reinterpret_cast<int *>(w);
  float *whole = reinterpret_cast<float *>(w + lin::table_bytes(p.num_seqs, segs));
  float *part = reinterpret_cast<float *>(w + lin::table_bytes(p.num_seqs, segs) + lin::align256(segs * p.H * 4));
  cudaError_t e = launch_linear_plan(p, sbase, C, per, 64, sm_count(), nullptr, nullptr, s);
  if (e != cudaSuccess) return e;
  Maps maps{};
  if (p.N > 0 && !(encode(&maps.q, p.q, p.dk, p.Hk, p.N) && encode(&maps.k, p.k, p.dk, p.Hk, p.N) &&
                   encode(&maps.v, p.v, p.dv, p.H, p.N) && encode(&maps.o, p.o, p.dv, p.H, p.N) &&
                   encode_f32(&maps.part, part, p.dv, segs * p.H * p.dk, p.dk)))
    return cudaErrorNotSupported;
  if (p.dk == 128)
    return p.dv == 128 ? launch<128, 128>(p, maps, sbase, part, whole, segs, s)
                       : launch<128, 64>(p, maps, sbase, part, whole, segs, s);
  return p.dv == 128 ? launch<64, 128>(p, maps, sbase, part, whole, segs, s)
                     : launch<64, 64>(p, maps, sbase, part, whole, segs, s);
}

cudaError_t launch_linear_segment_states_tc(const LinearParams &p, const int *sbase, float *part, float *rpart, float *whole,
                                            size_t segs, cudaStream_t s) {
  using namespace lintc;
  Maps fwd{}, rev{};
  const size_t rows = segs * p.H * p.dk;
  if (!(encode(&fwd.k, p.k, p.dk, p.Hk, p.N) && encode(&fwd.v, p.v, p.dv, p.H, p.N) &&
        encode_f32(&fwd.part, part, p.dv, rows, p.dk) && encode(&rev.k, p.q, p.dk, p.Hk, p.N) &&
        encode(&rev.v, p.d_o, p.dv, p.H, p.N) && encode_f32(&rev.part, rpart, p.dv, rows, p.dk)))
    return cudaErrorNotSupported;
  cudaError_t e;
  if (p.dk == 128)
    e = p.dv == 128 ? launch_shares<128, 128>(p, fwd, rev, sbase, whole, segs * p.H, s)
                    : launch_shares<128, 64>(p, fwd, rev, sbase, whole, segs * p.H, s);
  else
    e = p.dv == 128 ? launch_shares<64, 128>(p, fwd, rev, sbase, whole, segs * p.H, s)
                    : launch_shares<64, 64>(p, fwd, rev, sbase, whole, segs * p.H, s);
  return e != cudaSuccess ? e : launch_linear_chain(p, sbase, part, rpart, whole, s);
}

}  // namespace kda
