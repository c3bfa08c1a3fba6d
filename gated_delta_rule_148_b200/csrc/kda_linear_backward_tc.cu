// Linear attention with a decay for each head on the tensor cores (bf16 inputs): gradients.
// Formulas in kda_linear.cuh and kda_linear.cu (grad_kernel); chunks of 128 rows.
//
//   sweep   the states at the chunks' starts, S, and their gradients at the chunks' ends, D.
//           A state's columns never mix, so a block takes 32 columns of d_v of one sequence and
//           head through all chunks:  S <- 2^{b_C} S + K^T (w V), w_s = 2^{b_C - b_s}, with
//           S in registers (fp32), w V split into three bf16 parts (24 bits).  The products do not
//           depend on S, so the chain from chunk to chunk is one multiply-add per element, and four
//           blocks of a head keep it parallel for few heads; for fewer still, segments of a sequence
//           are swept from states of their own (sweep_chunks).  D: the same from the last chunk to
//           the first over q, grad_o with w_t = 2^{b_t}; it also takes <S, D> of each chunk.
//           Both are stored as two bf16 parts (16 bits), the form in which the next step's
//           products read them.
//   grad    per chunk and head, everything else (all chunks in parallel).  With rows s and columns t,
//             A = K Q^T, G = V dO^T, f_st = 2^{b_t - b_s} (t >= s), P = A o f, M = G o f
//             E = dO S^T, F = V D^T (two parts each), U = K D
//             dQ = 2^{b_t} E + M^T K,  dK = 2^{b_C - b_s} F + M Q,  dV = 2^{b_C - b_s} U + P dO
//           M lies in shared memory once and is read K-major (M Q) and MN-major (M^T K); P stays in
//           TMEM over A.  E, F and U are scaled in TMEM, where the second products add to them; on
//           the way the row sums q.E and k.F give the decays' gradients, in fp32.
// 16384 tokens, 32 heads, d = 128: sweeps 131 and 157 us (0.54 and 0.81 GB; a step of a chunk takes 1 us, a chain of
// load, weights, products and state), grad 292 us (1.44 GB, 220 us at the copy rate).  Slow decays change nothing here
// unless segments are swept (8192 tokens, 4 heads: 116 -> 131 us).
// The grad kernel is a persistent block per SM: a load/store warp, an MMA thread, a warp that
// prepares decays, and four warpgroups, whose loops over 32 columns are not unrolled: 96 registers a thread hold one
// round, and the addresses of all rounds spilled (636 -> 608 us for the whole pass over 16384 tokens, 32 heads).
#include "kda_linear_tc.cuh"

namespace kda {
namespace lintc {

// Wait sites reported with a timeout.
enum : unsigned { SITE_SWEEP = 71, SITE_GRAD = 91 };

// State tiles: [chunk x H + h][2 parts][DK][DV] bf16.

// ============================================================ tables
// The sweep's weights of a chunk and head, one warp each: 2^{b_C - b_s}, 2^{b_t}; bits of the real rows, 2^{b_C}.
// Apart from the sweep, where the sums of one chunk took longer than its products.
struct Table {
  float to[C], from[C];
  uint32_t valid[4];
  float whole, pad[3];
};

__global__ void __launch_bounds__(256) table_kernel(LinearParams p, const int *sbase, Table *tables) {
  after_previous();
  if (lin::call_ended(p, sbase)) return;
  const size_t i = (size_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (i >= (size_t)sbase[p.num_seqs] * p.H) return;
  const int lane = threadIdx.x & 31;
  const Segment sg = lin::locate(sbase, p.num_seqs, (int)(i / p.H));
  double b[4], total;
  uint32_t word;
  scan_decays(load_decays(p, sg.begin, sg.end, (int)(i % p.H)), b, total, word);
  Table &t = tables[i];
  reinterpret_cast<float4 *>(t.to)[lane] = make_float4(ex2((float)(total - b[0])), ex2((float)(total - b[1])),
                                                       ex2((float)(total - b[2])), ex2((float)(total - b[3])));
  reinterpret_cast<float4 *>(t.from)[lane] = make_float4(ex2((float)b[0]), ex2((float)b[1]), ex2((float)b[2]), ex2((float)b[3]));
  if ((lane & 7) == 0) t.valid[lane >> 3] = word;
  if (lane == 0) t.whole = ex2((float)total);
}

// ============================================================ sweep
// Roles: a load warp (K tile, 32 columns of V and the weights, three stages ahead), one warpgroup that writes
// w V, an MMA thread, one warpgroup that holds the state, a warp that stores it.  A step's tiles of the state
// leave (and S's arrive) through shared memory, since its rows are 64 bytes apart from each other's neighbours.
constexpr int kSweepThreads = 8 * 32 + 96;
constexpr int kSweepStages = 3;
constexpr int kSlice = 32;                      // d_v columns of a block

template <int DK, bool REVERSE>
struct SweepSmem {
  static constexpr uint32_t KT = C * DK * 2, VT = C * kSlice * 2, STAGE = KT + VT, XT = DK * kSlice * 2;
  // W: three parts of w V, two steps.  DK = 64: the MMA's rows 64 .. 127 come from the bytes after the K tile and
  // are not used
  static constexpr uint32_t W = kSweepStages * STAGE, OUT = W + 2 * 3 * VT, IN = OUT + 2 * XT;
  static constexpr uint32_t WGT = IN + (REVERSE ? 2 * 2 * XT : 0), VALID = WGT + kSweepStages * C * 4;
  static constexpr uint32_t BARS = VALID + kSweepStages * 16, END = BARS + 24 * 8;
  static_assert(END <= 232448, "shared memory of a block");
};

// Byte offset of 16-byte word c of row r in a tile of 32 columns with the 64-byte swizzle.
__device__ __forceinline__ uint32_t slice_at(int r, int c) { return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4)); }

struct SweepMaps {
  CUtensorMap k, v, s, out;      // REVERSE: q, grad_o, the states of the sweep before; the tiles written
};

template <int DK, int DV, bool REVERSE, bool CUT>
__global__ void __launch_bounds__(kSweepThreads, 1)
sweep_kernel(LinearParams p, const __grid_constant__ SweepMaps maps, const int *sbase, const int *order,
             const int *segments, const float *start, const Table *tables, float *through) {
  using L = SweepSmem<DK, REVERSE>;
  extern __shared__ __align__(1024) unsigned char sm[];
  after_previous();
  if (lin::call_ended(p, sbase)) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int SL = DV / kSlice;
  // whole sequences from the longest, or (CUT) segments of them from the states in start
  const int nitems = (CUT ? segments[p.num_seqs] : p.num_seqs) * p.H * SL;
  // a block's items one after the other; the next one's rows are looked up an item ahead
  struct Item {
    int b, h, c0, begin, n, chunk0;      // b: sequence, or segment
  };
  auto look_up = [&](int k) {
    const int i = item_of(k);
    Item x{};
    if (i < nitems) {
      x.c0 = i % SL * kSlice;
      x.h = i / SL % p.H;
      if constexpr (CUT) {
        const Segment sg = lin::locate(segments, p.num_seqs, i / SL / p.H);
        x.b = sg.id;
        x.begin = sg.begin;
        x.n = (sg.end - sg.begin + C - 1) / C;
        x.chunk0 = sbase[sg.seq()] + (sg.begin - p.cu[sg.seq()]) / C;
      } else {
        x.b = order[i / SL / p.H];
        x.begin = p.cu[x.b];
        x.n = (p.cu[x.b + 1] - x.begin + C - 1) / C;
        x.chunk0 = sbase[x.b];
      }
    }
    return x;
  };
  Item next = look_up(0);
  // products: the last chunk's matters to the gradient of the initial state only
  const bool to_init = REVERSE && !CUT && p.g_init != nullptr;
  auto products = [&](const Item &x) { return to_init ? x.n : x.n - 1; };
  auto at = [&](const Item &x, int j) { return REVERSE ? x.n - 1 - j : j; };      // chunk of step j
  // first row of a step's first part in the state tiles
  auto tile_row = [&](const Item &x, int j) { return (int)((((size_t)(x.chunk0 + at(x, j)) * p.H + x.h) * 2) * DK); };
  float *wgt = reinterpret_cast<float *>(sm + L::WGT);
  uint32_t *valid = reinterpret_cast<uint32_t *>(sm + L::VALID);
  uint64_t *full = reinterpret_cast<uint64_t *>(sm + L::BARS), *empty = full + kSweepStages, *w_ready = empty + kSweepStages,
           *done = w_ready + 2, *acc_free = w_ready + 4, *s_full = w_ready + 6, *s_free = w_ready + 8, *staged = w_ready + 10, *out_free = w_ready + 11,
           *drain = w_ready + 12;
  uint32_t *tmem_sh = reinterpret_cast<uint32_t *>(drain + 1);
  volatile int *failed = reinterpret_cast<volatile int *>(tmem_sh + 1);
  if (warp == 8) tmem_alloc(tmem_sh, 256);
  if (tid == 0) {
    for (int i = 0; i < kSweepStages; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(w_ready + i, 128);
      mbar_init(done + i, 1);
      mbar_init(acc_free + i, 128);
      mbar_init(s_full + i, 1);
      mbar_init(s_free + i, 128);
    }
    mbar_init(staged, 128);
    mbar_init(out_free, 1);
    mbar_init(drain, 1);
    *failed = 0;
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tm = *tmem_sh;
  const Waits wait{p.wait_cycles, p.err, p.site, failed};
  if (warp == 9) {
    if (lane == 0) {
      bool ok = true;
      int loaded = 0, states = 0;
      for (int k = 0; item_of(k) < nitems && ok; ++k) {
        const Item x = next;
        next = look_up(k + 1);
        const int n_mma = products(x), hk = x.h / (p.H / p.Hk);
        const Table *table = tables + (size_t)x.chunk0 * p.H + x.h;
        for (int j = 0; j < x.n && ok; ++j) {
          const int pos = x.begin + at(x, j) * C;
          if (j < n_mma) {
            const int st = loaded % kSweepStages;
            if (loaded >= kSweepStages) ok = wait(empty + st, loaded / kSweepStages - 1, SITE_SWEEP);
            if (!ok) break;
            mbar_arrive_expect_tx(full + st, L::STAGE + C * 4 + 16);
            const uint32_t dst = smem_u32(sm + st * L::STAGE);
            const Table &t = table[(size_t)at(x, j) * p.H];
            bulk_load(wgt + st * C, REVERSE ? t.from : t.to, C * 4, full + st);
            bulk_load(valid + st * 4, t.valid, 16, full + st);
#pragma unroll
            for (int kb = 0; kb < DK / 64; ++kb) tma_load_3d(dst + kb * C * 128, &maps.k, kb * 64, hk, pos, full + st);
            tma_load_3d(dst + L::KT, &maps.v, x.c0, x.h, pos, full + st);
            ++loaded;
          }
          if constexpr (REVERSE) {
            const int sl = states & 1;
            if (states >= 2) ok = wait(s_free + sl, (states >> 1) - 1, SITE_SWEEP + 1);
            if (!ok) break;
            mbar_arrive_expect_tx(s_full + sl, 2 * L::XT);
#pragma unroll
            for (int y = 0; y < 2; ++y)
              tma_load_3d(smem_u32(sm + L::IN + (sl * 2 + y) * L::XT), &maps.s, x.c0, 0, tile_row(x, j) + y * DK, s_full + sl);
            ++states;
          }
        }
      }
      // loads in flight land before the block ends, whoever gave up
      for (int i = loaded > kSweepStages ? loaded - kSweepStages : 0; i < loaded; ++i)
        mbar_wait(full + i % kSweepStages, (i / kSweepStages) & 1, kDrainCycles);
      for (int i = states > 2 ? states - 2 : 0; i < states; ++i) mbar_wait(s_full + (i & 1), (i >> 1) & 1, kDrainCycles);
    }
  } else if (warp == 8) {
    if (lane == 0) {
      bool ok = true;
      int m = 0;
      for (int k = 0; item_of(k) < nitems && ok; ++k) {
        const Item x = next;
        next = look_up(k + 1);
        for (int j = 0; j < products(x) && ok; ++j, ++m) {
          const int st = m % kSweepStages, sl = m & 1;
          if (m >= 2) ok = wait(acc_free + sl, (m >> 1) - 1, SITE_SWEEP + 2);
          ok = ok && wait(w_ready + sl, m >> 1, SITE_SWEEP + 3);
          if (!ok) break;
          fence_after_sync();
          const uint64_t kd = desc_mnmajor(smem_u32(sm + st * L::STAGE), C, 0, 0),
                         vd = sdesc(smem_u32(sm + L::W + sl * 3 * L::VT), L::VT, 512, 4);
#pragma unroll
          for (int s = 0; s < C / 16; ++s)
            mma_bf16(tm + sl * 128, mnmajor_step(kd, s), vd + (uint32_t)(s * 16 * 64 >> 4),
                     idesc_bf16(128, 3 * kSlice, 1, 1), s > 0);
          mma_commit(empty + st);
          mma_commit(done + sl);
        }
      }
      mma_commit(drain);
      mbar_wait(drain, 0, kDrainCycles);
    }
  } else if (warp == 10) {
    if (lane == 0) {
      bool ok = true;
      int out = 0;
      for (int k = 0; item_of(k) < nitems && ok; ++k) {
        const Item x = next;
        next = look_up(k + 1);
        for (int j = 0; j < x.n && ok; ++j, ++out) {
          ok = wait(staged, out, SITE_SWEEP + 8);
          if (!ok) break;
#pragma unroll
          for (int y = 0; y < 2; ++y)
            tma_store_3d(&maps.out, smem_u32(sm + L::OUT + y * L::XT), x.c0, 0, tile_row(x, j) + y * DK);
          bulk_commit();
          bulk_wait_read();
          mbar_arrive(out_free);
        }
      }
      bulk_wait_all();
    }
  } else if (warp < 4) {
    // ---------------- w V (thread: row of the chunk)
    const int r = tid;
    bool ok = true;
    int m = 0;
    for (int k = 0; item_of(k) < nitems && ok; ++k) {
      const Item x = next;
      next = look_up(k + 1);
      for (int j = 0; j < products(x) && ok; ++j, ++m) {
        const int sl = m & 1, st = m % kSweepStages;
        ok = wait.warp(full + st, m / kSweepStages, SITE_SWEEP + 4);
        if (!ok) break;
        const bool real = (valid[4 * st + warp] >> lane) & 1;
        const float w = wgt[st * C + r];
        unsigned char *sk = sm + st * L::STAGE;
        uint4 u[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          u[c] = real ? *reinterpret_cast<const uint4 *>(sk + L::KT + slice_at(r, c)) : make_uint4(0, 0, 0, 0);
        if (!real)
#pragma unroll
          for (int c = 0; c < DK / 8; ++c)
            *reinterpret_cast<uint4 *>(sk + row_tile_chunk(r, c >> 3, c & 7, C)) = make_uint4(0, 0, 0, 0);
        if (m >= 2) ok = wait.warp(done + sl, (m >> 1) - 1, SITE_SWEEP + 5);
        if (!ok) break;
        unsigned char *sw = sm + L::W + sl * 3 * L::VT;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float f[8];
          unpack8(u[c], f);
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] *= w;
#pragma unroll
          for (int y = 0; y < 3; ++y) *reinterpret_cast<uint4 *>(sw + y * L::VT + slice_at(r, c)) = take_bf16(f);
        }
        fence_async_smem();
        mbar_arrive(w_ready + sl);
      }
    }
  } else {
    // ---------------- the state (thread: its row)
    const int r = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const float *in = CUT ? start : REVERSE ? p.d_final : p.init_state;
    bool ok = true;
    int out = 0, m = 0;
    for (int k = 0; item_of(k) < nitems && ok; ++k) {
      const Item x = next;
      next = look_up(k + 1);
      const int n_mma = products(x);
      const float *whole = &tables[(size_t)(x.chunk0 + at(x, 0)) * p.H + x.h].whole;
      const ptrdiff_t hop = (REVERSE ? -1 : 1) * (ptrdiff_t)p.H * (ptrdiff_t)(sizeof(Table) / 4);
      const size_t own = (((size_t)x.b * p.H + x.h) * DK + r) * DV + x.c0;
      float S[kSlice];
#pragma unroll
      for (int e = 0; e < kSlice; ++e) S[e] = 0.f;
      if (in != nullptr && r < DK)
#pragma unroll
        for (int e = 0; e < kSlice; e += 4) {
          const float4 f = *reinterpret_cast<const float4 *>(in + own + e);
          S[e] = f.x; S[e + 1] = f.y; S[e + 2] = f.z; S[e + 3] = f.w;
        }
      float ahead = x.n > 0 ? *whole : 0.f;
      for (int j = 0; j < x.n && ok; ++j, ++out) {
        const int sl = out & 1;
        const float a = ahead;
        whole += hop;
        if (j + 1 < x.n) ahead = *whole;
        if (out > 0) ok = wait.warp(out_free, out - 1, SITE_SWEEP + 9);
        if (!ok) break;
        if (r < DK)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = S[8 * c + e];
            *reinterpret_cast<uint4 *>(sm + L::OUT + slice_at(r, c)) = take_bf16(f);
            *reinterpret_cast<uint4 *>(sm + L::OUT + L::XT + slice_at(r, c)) = take_bf16(f);
          }
        fence_async_smem();
        mbar_arrive(staged);
        if constexpr (REVERSE) {
          ok = wait.warp(s_full + sl, out >> 1, SITE_SWEEP + 6);
          if (!ok) break;
          const unsigned char *t = sm + L::IN + sl * 2 * L::XT;
          float dot = 0.f;
          if (r < DK)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              float f[8], g[8];
              unpack8(*reinterpret_cast<const uint4 *>(t + slice_at(r, c)), f);
              unpack8(*reinterpret_cast<const uint4 *>(t + L::XT + slice_at(r, c)), g);
#pragma unroll
              for (int e = 0; e < 8; ++e) dot = fmaf(f[e] + g[e], S[8 * c + e], dot);
            }
          mbar_arrive(s_free + sl);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
          if (lane == 0)
            through[(((size_t)(x.chunk0 + at(x, j)) * p.H + x.h) * SL + x.c0 / kSlice) * 4 + (warp & 3)] = dot;
        }
        if (j >= n_mma) continue;
        ok = wait.warp(done + (m & 1), m >> 1, SITE_SWEEP + 7);
        if (!ok) break;
        fence_after_sync();
        const uint32_t col = tm + lanes + (m & 1) * 128;
        uint32_t u[32], v[32], w[32];
        tmem_ld32_issue(col, u);
        tmem_ld32_issue(col + 32, v);
        tmem_ld32_issue(col + 64, w);
        tmem_ld32_wait(u);
        tmem_ld32_wait(v);
        tmem_ld32_wait(w);
        fence_before_sync();
        mbar_arrive(acc_free + (m & 1));
        ++m;
#pragma unroll
        for (int e = 0; e < 32; ++e)
          S[e] = fmaf(a, S[e], __uint_as_float(u[e]) + (__uint_as_float(v[e]) + __uint_as_float(w[e])));
      }
      if (to_init && ok && r < DK)
#pragma unroll
        for (int e = 0; e < kSlice; e += 4)
          *reinterpret_cast<float4 *>(p.g_init + own + e) = make_float4(S[e], S[e + 1], S[e + 2], S[e + 3]);
    }
  }
  fence_before_sync();
  __syncthreads();
  if (warp == 8) {
    fence_after_sync();
    tmem_dealloc(tm, 256);
  }
}

// ============================================================ grad
constexpr int kGradThreads = 16 * 32 + 96;      // four warpgroups

struct GradMaps {
  CUtensorMap q, k, v, d_o, s, d, gq, gk, gv;
};

template <int DK, int DV>
struct GradSmem {
  static constexpr uint32_t QT = C * DK * 2, VT = C * DV * 2, XT = DK * DV * 2;
  // X: the two parts of S, then of D, then (first) dQ and (second) dV on their way out; M's tile: also dK
  static constexpr uint32_t X1 = QT > VT ? QT : VT;
  static_assert(X1 >= XT && C * C * 2 >= QT, "tiles on their way out");
  static constexpr uint32_t Q = 0, K = QT, V = 2 * QT, O = V + VT, X = O + VT, M = X + 2 * X1, HL = M + C * C * 2;
  // column factors of the blocks (w, x) of 32 x 32 pairs, then the blocks' pair sums; the rest of the decays' sums
  static constexpr uint32_t PAIRS = HL + C * 8, SUMS = PAIRS + 10 * 32 * 4;
  static constexpr uint32_t VALID = SUMS + 10 * 4, BARS = VALID + 16, END = BARS + 32 * 8;
  static_assert(END <= 232448, "shared memory of a block");
};

// Sums of 32 columns over the warp's lanes: lane e gets column e's.
__device__ __forceinline__ float column_sums(float (&x)[32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float give = up ? x[i] : x[i + o], stay = up ? x[i + o] : x[i];
      x[i] = stay + __shfl_xor_sync(0xFFFFFFFFu, give, o);
    }
  }
  return x[0];
}
// Sums over the lanes before (below) this one.
__device__ __forceinline__ float exclusive_sum(float x) {
  const int lane = threadIdx.x & 31;
  float s = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float y = __shfl_up_sync(0xFFFFFFFFu, s, o);
    if (lane >= o) s += y;
  }
  s = __shfl_up_sync(0xFFFFFFFFu, s, 1);
  return lane ? s : 0.f;
}
// Sums over this lane and those after it.
__device__ __forceinline__ float suffix_sum(float s) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float y = __shfl_down_sync(0xFFFFFFFFu, s, o);
    if (lane + o < 32) s += y;
  }
  return s;
}
template <int DK, int DV>
__global__ void __launch_bounds__(kGradThreads, 1)
grad_kernel(LinearParams p, const __grid_constant__ GradMaps maps, const int *sbase, const float *through, float *gq32,
            float *gk32, float *gla) {
  using L = GradSmem<DK, DV>;
  extern __shared__ __align__(1024) unsigned char sm[];
  after_previous();
  if (lin::call_ended(p, sbase)) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nitems = sbase[p.num_seqs] * p.H;
  float2 *hl = reinterpret_cast<float2 *>(sm + L::HL);
  float *extra = reinterpret_cast<float *>(sm + L::HL);     // of the blocks (w, x), w < x: after the pairs' decays are done with
  float *pairs = reinterpret_cast<float *>(sm + L::PAIRS);
  float *sums = reinterpret_cast<float *>(sm + L::SUMS);    // warps' totals: q.E, k.F
  float *whole = sums + 8;                                  // 2^{b_C}
  uint32_t *valid = reinterpret_cast<uint32_t *>(sm + L::VALID);
  uint64_t *full = reinterpret_cast<uint64_t *>(sm + L::BARS), *ready = full + 1, *x_full = full + 2,      // S, S, D, D
           *ag_done = full + 6, *eh_done = full + 7, *e_done = full + 8, *f_done = full + 9, *u_done = full + 10,
           *conv = full + 11, *e_scaled = full + 12, *f_scaled = full + 13, *u_scaled = full + 14, *dq_done = full + 15,
           *dk_done = full + 16, *dv_done = full + 17, *dq_staged = full + 18, *dk_staged = full + 19,
           *dv_staged = full + 20, *m_free = full + 21, *q_free = full + 22, *k_free = full + 23, *v_free = full + 24,
           *tab_free = full + 25, *paired = full + 26, *summed = full + 27, *drain = full + 28;
  uint32_t *tmem_sh = reinterpret_cast<uint32_t *>(full + 29);
  volatile int *failed = reinterpret_cast<volatile int *>(tmem_sh + 1);
  if (warp == 16) tmem_alloc(tmem_sh, 512);
  if (tid == 0) {
    for (int i = 0; i < 29; ++i) mbar_init(full + i, 1);
    // every thread of one to four warpgroups
    mbar_init(conv, 512);
    mbar_init(paired, 512);
    mbar_init(e_scaled, 128);
    mbar_init(f_scaled, 128);
    mbar_init(u_scaled, 256);
    mbar_init(summed, 256);
    mbar_init(dq_staged, 128);
    mbar_init(dk_staged, 128);
    mbar_init(dv_staged, 256);
    mbar_init(q_free, 128);
    mbar_init(k_free, 128);
    mbar_init(v_free, 256);
    mbar_init(tab_free, 128);
    *failed = 0;
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tm = *tmem_sh;
  // A (then P: row block x in columns 32 x .. 32 x + 15), dK; G then dV, and dQ change places from item to item, since
  // the item before gives up dQ first
  constexpr uint32_t T_A = 0, T_K = 384;
  auto t_v = [&](int item) { return item & 1 ? 256u : 128u; };
  auto t_q = [&](int item) { return item & 1 ? 128u : 256u; };
  const Waits wait{p.wait_cycles, p.err, p.site, failed};
  const int G = p.H / p.Hk;
  const bool shared = gq32 != nullptr;
  int it = 0;

  if (warp == 17) {
    // ---------------- loads and stores
    if (lane == 0) {
      bool ok = true;
      int pos_out = -1, h_out = 0;           // the item before: its gradients, if the chunk is whole
      auto store_q = [&]() {
        ok = ok && wait(dq_staged, it - 1, SITE_GRAD);
        if (ok && pos_out >= 0 && !shared)
#pragma unroll
          for (int kb = 0; kb < DK / 64; ++kb)
            tma_store_3d(&maps.gq, smem_u32(sm + L::X) + kb * C * 128, kb * 64, h_out, pos_out);
        bulk_commit();
      };
      auto store_k = [&]() {
        ok = ok && wait(dk_staged, it - 1, SITE_GRAD + 1);
        if (ok && pos_out >= 0 && !shared)
#pragma unroll
          for (int kb = 0; kb < DK / 64; ++kb)
            tma_store_3d(&maps.gk, smem_u32(sm + L::M) + kb * C * 128, kb * 64, h_out, pos_out);
        bulk_commit();
      };
      auto store_v = [&]() {
        ok = ok && wait(dv_staged, it - 1, SITE_GRAD + 2);
        if (ok && pos_out >= 0)
#pragma unroll
          for (int kb = 0; kb < DV / 64; ++kb)
            tma_store_3d(&maps.gv, smem_u32(sm + L::X + L::X1) + kb * C * 128, kb * 64, h_out, pos_out);
        bulk_commit();
      };
      auto one_left = []() { asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory"); };
      auto load_state = [&](const CUtensorMap *map, int i, int x, uint64_t *bar) {      // part x
        mbar_arrive_expect_tx(bar, L::XT);
#pragma unroll
        for (int kb = 0; kb < DV / 64; ++kb)
          tma_load_3d(smem_u32(sm + L::X + x * L::X1) + kb * DK * 128, map, kb * 64, 0, (2 * i + x) * DK, bar);
      };
      for (int i = blockIdx.x; i < nitems && ok; i += gridDim.x, ++it) {
        const Segment sg = lin::locate(sbase, p.num_seqs, i / p.H);
        const int h = i % p.H, pos = sg.begin;
        // each tile once its last reader is done (K, Q: also the row sums, before dK's product)
        if (it > 0) ok = wait(dq_done, it - 1, SITE_GRAD + 3);
        if (!ok) break;
        mbar_arrive_expect_tx(full, 2 * L::QT + 2 * L::VT);
#pragma unroll
        for (int kb = 0; kb < DV / 64; ++kb) tma_load_3d(smem_u32(sm + L::V) + kb * C * 128, &maps.v, kb * 64, h, pos, full);
        if (it > 0) ok = wait(dk_done, it - 1, SITE_GRAD + 4);
        if (!ok) break;
#pragma unroll
        for (int kb = 0; kb < DK / 64; ++kb) {
          tma_load_3d(smem_u32(sm + L::K) + kb * C * 128, &maps.k, kb * 64, h / G, pos, full);
          tma_load_3d(smem_u32(sm + L::Q) + kb * C * 128, &maps.q, kb * 64, h / G, pos, full);
        }
        if (it > 0) {
          store_q();
          ok = ok && wait(dv_done, it - 1, SITE_GRAD + 5);
        }
        if (!ok) break;
#pragma unroll
        for (int kb = 0; kb < DV / 64; ++kb) tma_load_3d(smem_u32(sm + L::O) + kb * C * 128, &maps.d_o, kb * 64, h, pos, full);
        if (it > 0) {
          store_k();
          one_left();
        }
        if (!ok) break;
        load_state(&maps.s, i, 0, x_full);
        if (it > 0) {
          store_v();
          one_left();
          mbar_arrive(m_free);
          bulk_wait_read();
        }
        if (!ok) break;
        load_state(&maps.s, i, 1, x_full + 1);
        ok = wait(eh_done, it, SITE_GRAD + 6);
        if (!ok) break;
        load_state(&maps.d, i, 0, x_full + 2);
        ok = wait(e_done, it, SITE_GRAD + 7);
        if (!ok) break;
        load_state(&maps.d, i, 1, x_full + 3);
        pos_out = pos + C <= sg.end ? pos : -1;
        h_out = h;
      }
      if (it > 0) {
        store_q();
        store_k();
        store_v();
      }
      bulk_wait_all();
      // loads in flight (the last item's, and those of one begun) land before the block ends, whoever gave up
      for (int i = it > 0 ? it - 1 : 0; i < it + !ok; ++i) {
        mbar_wait(full, i & 1, kDrainCycles);
        for (int x = 0; x < 4; ++x) mbar_wait(x_full + x, i & 1, kDrainCycles);
      }
    }
  } else if (warp == 16) {
    // ---------------- MMAs
    if (lane == 0) {
      bool ok = true;
      const uint32_t sx = smem_u32(sm + L::X), smm = smem_u32(sm + L::M);
      // descriptors of step 0, read K-major and MN-major
      const uint64_t qk = desc_kmajor(smem_u32(sm + L::Q), C, 0, 0), qm = desc_mnmajor(smem_u32(sm + L::Q), C, 0, 0),
                     kk = desc_kmajor(smem_u32(sm + L::K), C, 0, 0), km = desc_mnmajor(smem_u32(sm + L::K), C, 0, 0),
                     vk = desc_kmajor(smem_u32(sm + L::V), C, 0, 0), ogk = desc_kmajor(smem_u32(sm + L::O), C, 0, 0),
                     om = desc_mnmajor(smem_u32(sm + L::O), C, 0, 0), xm = desc_mnmajor(sx, DK, 0, 0),
                     xk[2] = {desc_kmajor(sx, DK, 0, 0), desc_kmajor(sx + L::X1, DK, 0, 0)}, mk = desc_kmajor(smm, C, 0, 0), mm = desc_mnmajor(smm, C, 0, 0);
      for (int i = blockIdx.x; i < nitems && ok; i += gridDim.x, ++it) {
        const uint32_t T_V = tm + t_v(it), T_Q = tm + t_q(it);
        // A takes the place of the item before's P and of the row sums beside it, which the third warpgroup reads last
        if (it > 0) ok = wait(tab_free, it - 1, SITE_GRAD + 16);
        ok = ok && wait(full, it, SITE_GRAD + 6);
        if (!ok) break;
        fence_after_sync();
#pragma unroll
        for (int s = 0; s < DK / 16; ++s)
          mma_bf16(tm + T_A, kmajor_step<C>(kk, s), kmajor_step<C>(qk, s), idesc_bf16(128, C, 0, 0), s > 0);
        if (it > 0) ok = wait(q_free, it - 1, SITE_GRAD + 7);
        if (!ok) break;
        fence_after_sync();
#pragma unroll
        for (int s = 0; s < DV / 16; ++s)
          mma_bf16(T_V, kmajor_step<C>(vk, s), kmajor_step<C>(ogk, s), idesc_bf16(128, C, 0, 0), s > 0);
        mma_commit(ag_done);
        if (it > 0) ok = wait(v_free, it - 1, SITE_GRAD + 8);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          ok = ok && wait(x_full + x, it, SITE_GRAD + 9);
          if (!ok) break;
          fence_after_sync();
#pragma unroll
          for (int s = 0; s < DV / 16; ++s)
            mma_bf16(T_Q, kmajor_step<C>(ogk, s), kmajor_step<DK>(xk[x], s), idesc_bf16(128, DK, 0, 0),
                     x > 0 || s > 0);
          mma_commit(x ? e_done : eh_done);
        }
        if (it > 0) ok = ok && wait(k_free, it - 1, SITE_GRAD + 10);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          ok = ok && wait(x_full + 2 + x, it, SITE_GRAD + 11);
          if (!ok) break;
          fence_after_sync();
#pragma unroll
          for (int s = 0; s < DV / 16; ++s)
            mma_bf16(tm + T_K, kmajor_step<C>(vk, s), kmajor_step<DK>(xk[x], s), idesc_bf16(128, DK, 0, 0),
                     x > 0 || s > 0);
        }
        if (!ok) break;
        mma_commit(f_done);
        ok = wait(conv, it, SITE_GRAD + 12);
        if (!ok) break;
        fence_after_sync();
#pragma unroll
        for (int s = 0; s < DK / 16; ++s)
          mma_bf16(T_V, kmajor_step<C>(kk, s), mnmajor_step(xm, s), idesc_bf16(128, DV, 0, 1), s > 0);
        mma_commit(u_done);
        ok = wait(e_scaled, it, SITE_GRAD + 13);
        if (!ok) break;
        fence_after_sync();
#pragma unroll
        for (int s = 0; s < C / 16; ++s)
          mma_bf16(T_Q, mnmajor_step(mm, s), mnmajor_step(km, s), idesc_bf16(128, DK, 1, 1), 1);
        mma_commit(dq_done);
        ok = wait(f_scaled, it, SITE_GRAD + 14);
        if (!ok) break;
        fence_after_sync();
#pragma unroll
        for (int s = 0; s < C / 16; ++s)
          mma_bf16(tm + T_K, kmajor_step<C>(mk, s), mnmajor_step(qm, s), idesc_bf16(128, DK, 0, 1), 1);
        mma_commit(dk_done);
        ok = wait(u_scaled, it, SITE_GRAD + 15);
        if (!ok) break;
        fence_after_sync();
#pragma unroll
        for (int s = 0; s < C / 16; ++s)
          mma_bf16_ta(T_V, tm + T_A + 32 * (s >> 1) + 8 * (s & 1), mnmajor_step(om, s), idesc_bf16(128, DV, 0, 1), 1);
        mma_commit(dv_done);
      }
      mma_commit(drain);
      mbar_wait(drain, 0, kDrainCycles);
    }
  } else if (warp == 18) {
    // ---------------- decays
    bool ok = true;
    RawDecays raw{};
    auto next = [&](int i) {
      if (i < nitems) {
        const Segment sg = lin::locate(sbase, p.num_seqs, i / p.H);
        raw = load_decays(p, sg.begin, sg.end, i % p.H);
      }
    };
    next(blockIdx.x);
    for (int i = blockIdx.x; i < nitems && ok; i += gridDim.x, ++it) {
      double b[4], total;
      uint32_t word;
      const RawDecays now = raw;
      next(i + gridDim.x);
      scan_decays(now, b, total, word);
      if (it > 0) ok = wait.warp(tab_free, it - 1, SITE_GRAD + 16);
      if (!ok) break;
      if ((lane & 7) == 0) valid[lane >> 3] = word;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float hi = (float)b[e];
        hl[4 * lane + e] = make_float2(hi, (float)(b[e] - (double)hi));
      }
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive(ready);
    }
  } else {
    // ---------------- thread: row r of the chunk (as s in P, M, F and U; as t in E and dQ)
    // Warpgroup y: columns 32 y .. 32 y + 31 of P and M; then E and dQ (0), F and dK (1), U and dV (2 and 3, half each)
    const int r = tid & 127, w = warp & 3, y = warp >> 2;
    const uint32_t lanes = (uint32_t)(w * 32) << 16;
    bool ok = true;
    for (int i = blockIdx.x; i < nitems && ok; i += gridDim.x, ++it) {
      const Segment sg = lin::locate(sbase, p.num_seqs, i / p.H);
      const int h = i % p.H, pos = sg.begin;
      const int rows = sg.end - pos;
      const uint32_t T_V = tm + lanes + t_v(it), T_Q = tm + lanes + t_q(it);
      ok = wait.warp(ready, it, SITE_GRAD + 18) && wait.warp(full, it, SITE_GRAD + 17);
      if (!ok) break;
      const float2 br = hl[r];
      const uint32_t cols = valid[y];                  // of the warp's columns: the real rows
      const bool real = (valid[w] >> lane) & 1;
      if (!real) {      // a pad or a row of the next sequence: q, k and grad_o must not reach other rows (sums of whole rows are
                        // masked where they are used)
#pragma unroll
        for (int e = 0; e < DK / 32; ++e) {
          const int cc = y * (DK / 32) + e;
          const uint32_t at = row_tile_chunk(r, cc >> 3, cc & 7, C);
          *reinterpret_cast<uint4 *>(sm + L::Q + at) = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4 *>(sm + L::K + at) = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int e = 0; e < DV / 32; ++e) {
          const int cc = y * (DV / 32) + e;
          *reinterpret_cast<uint4 *>(sm + L::O + row_tile_chunk(r, cc >> 3, cc & 7, C)) = make_uint4(0, 0, 0, 0);
        }
      }
      float fac;      // E's rows are scaled by 2^{b_t}, F's and U's by 2^{b_C - b_s}
      {
        const float2 be = hl[C - 1];
        fac = y == 0 ? ex2(br.x + br.y) : ex2((be.x - br.x) + (be.y - br.y));
        if (tid == 0) *whole = ex2(be.x + be.y);
      }
      float *slot = pairs + (y * (y + 1) / 2 + w) * 32;      // of this warp's block (w <= y)
      float rowf = 0.f;
      if (y > w) {      // 2^{b_t - b_ref} and 2^{b_ref - b_s}: the reference is the row block's last row
        const float2 ref = hl[32 * w + 31], bt = hl[32 * y + lane];
        rowf = ex2((ref.x - br.x) + (ref.y - br.y));
        slot[lane] = ex2((bt.x - ref.x) + (bt.y - ref.y));
      }
      __syncwarp();
      ok = wait.warp(ag_done, it, SITE_GRAD + 19);
      if (it > 0) ok = ok && wait.warp(m_free, it - 1, SITE_GRAD + 20);
      if (!ok) break;
      fence_after_sync();
      unsigned char *mt = sm + L::M;
      float f[32];                       // pairs (s, t) of this row and the warp's columns
      if (y < w) {
        float zero[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) zero[e] = 0.f;
        tmem_st16(tm + lanes + T_A + 32 * y, zero);
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *reinterpret_cast<uint4 *>(mt + row_tile_chunk(r, y >> 1, 4 * (y & 1) + c, C)) = make_uint4(0, 0, 0, 0);
      } else {
        const uint32_t on_cols = real ? cols : 0u;
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          float a[16], g[16];
          tmem_ld16(tm + lanes + T_A + 32 * y + 16 * z, a);
          tmem_ld16(T_V + 32 * y + 16 * z, g);
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            float d[4];
            if (y == w) {
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const float2 bt = hl[32 * y + 16 * z + e + x];
                d[x] = ex2((bt.x - br.x) + (bt.y - br.y));
              }
            } else {
              const float4 cf = *reinterpret_cast<const float4 *>(slot + 16 * z + e);
              d[0] = rowf * cf.x; d[1] = rowf * cf.y; d[2] = rowf * cf.z; d[3] = rowf * cf.w;
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const bool on = (y > w || 16 * z + e + x >= lane) && ((on_cols >> (16 * z + e + x)) & 1);      // t >= s
              a[e + x] = on ? a[e + x] * d[x] : 0.f;
              f[16 * z + e + x] = on ? a[e + x] * g[e + x] : 0.f;
              g[e + x] = on ? g[e + x] * d[x] : 0.f;
            }
          }
          uint32_t pw[8];                // P as packed bf16
#pragma unroll
          for (int e = 0; e < 8; ++e) pw[e] = pack_bf16x2(a[2 * e], a[2 * e + 1]);
          tmem_st8(tm + lanes + T_A + 32 * y + 8 * z, pw);
#pragma unroll
          for (int c = 0; c < 2; ++c)
            *reinterpret_cast<uint4 *>(mt + row_tile_chunk(r, y >> 1, 4 * (y & 1) + 2 * z + c, C)) = pack8(g + 8 * c);
        }
      }
      tmem_st_wait();
      fence_async_smem();
      fence_before_sync();
      mbar_arrive(conv);

      // while the products run: pairs (s, t) with t >= u for column u; on the diagonal block only columns u > s
      float before = 0.f;                // of the rows before this one in the block: their pairs
      if (y >= w) {
        float acc = 0.f;
#pragma unroll
        for (int e = 31; e >= 0; --e) {
          acc += f[e];
          f[e] = (y > w || e > lane) ? acc : 0.f;
        }
        if (y > w) before = exclusive_sum(acc);
        const float col = column_sums(f);
        __syncwarp();
        slot[lane] = col;
      }
      ok = wait.warp(conv, it, SITE_GRAD + 21);      // no more readers of the decays: their place takes sums
      if (!ok) break;
      if (y > w) extra[(y * (y - 1) / 2 + w) * 32 + lane] = before;
      mbar_arrive(paired);

      if (y < 2) {
        // E or F: scaled in place; its rows' products with q or k
        ok = wait.warp(y ? f_done : e_done, it, SITE_GRAD + 22);
        if (!ok) break;
        fence_after_sync();
        float dot = 0.f;
        const unsigned char *tile = sm + (y ? L::K : L::Q);
        const uint32_t col = y ? tm + lanes + T_K : T_Q;
#pragma unroll 1
        for (int x = 0; x < DK / 32; ++x) {
          float v[32];
          tmem_ld32(col + 32 * x, v);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float k[8];
            unpack8(*reinterpret_cast<const uint4 *>(tile + row_tile_chunk(r, x >> 1, 4 * (x & 1) + c, C)), k);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              v[8 * c + e] *= fac;
              dot = fmaf(v[8 * c + e], k[e], dot);
            }
          }
          tmem_st32(col + 32 * x, v);
        }
        tmem_st_wait();
        fence_before_sync();
        mbar_arrive(y ? f_scaled : e_scaled);
        if (!real) dot = 0.f;
        // over the rows from this one on (q.E) or before this one (k.F): to the third warpgroup, in TMEM beside P
        const float sum = y ? exclusive_sum(dot) : suffix_sum(dot);
        if (lane == (y ? 31 : 0)) sums[4 * y + w] = y ? sum + dot : sum;
        tmem_st1(tm + lanes + T_A + 16 + y, sum);
        tmem_st_wait();
        fence_before_sync();
        mbar_arrive(summed);
      } else {
        float g = 0.f;                   // the decay's gradient of row u = r
        if (y == 2) {
          ok = wait.warp(paired, it, SITE_GRAD + 23);
          if (!ok) break;
          float thr = lane < DV / 8 ? through[(size_t)i * (DV / 8) + lane] : 0.f;
          for (int x = 0; x <= w; ++x) g += pairs[(w * (w + 1) / 2 + x) * 32 + lane];
          for (int z = w + 1; z < 4; ++z) {
            g += extra[(z * (z - 1) / 2 + w) * 32 + lane];
            for (int x = 0; x < w; ++x) g += pairs[(z * (z + 1) / 2 + x) * 32];
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) thr += __shfl_xor_sync(0xFFFFFFFFu, thr, o);
          g = fmaf(*whole, thr, g);
        }
        ok = wait.warp(u_done, it, SITE_GRAD + 24);
        if (!ok) break;
        fence_after_sync();
        const uint32_t col = T_V + (y - 2) * (DV / 2);
#pragma unroll 1
        for (int x = 0; x < DV / 64; ++x) {
          float v[32];
          tmem_ld32(col + 32 * x, v);
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] *= fac;
          tmem_st32(col + 32 * x, v);
        }
        tmem_st_wait();
        fence_before_sync();
        mbar_arrive(u_scaled);
        if (y == 2) {
          ok = wait.warp(summed, it, SITE_GRAD + 25);
          if (!ok) break;
          fence_after_sync();
          float qk[2];
          tmem_ld2(tm + lanes + T_A + 16, qk);
          g += qk[0] + qk[1];
          for (int x = w + 1; x < 4; ++x) g += sums[x];
          for (int x = 0; x < w; ++x) g += sums[4 + x];
          // one decay per head: [H, N] for the sum that follows
          if (r < rows) gla[p.decay_head ? (size_t)h * p.N + pos + r : (size_t)(pos + r) * p.H + h] = real ? g : 0.f;
          fence_before_sync();
          mbar_arrive(tab_free);
        }
      }

      // gradients: columns of `col` to 16-byte words word0 .. of the tile, or straight to the row
      auto out = [&](uint32_t col, int cols, unsigned char *tile, int word0, uint16_t *row, float *row32) {
#pragma unroll 1
        for (int x = 0; x < 4; ++x) {
          if (32 * x >= cols) break;
          float f[32];
          tmem_ld32(col + 32 * x, f);
          if (!real)
#pragma unroll
            for (int e = 0; e < 32; ++e) f[e] = 0.f;
          if (row32 != nullptr) {
            if (r < rows)
#pragma unroll
              for (int e = 0; e < 32; e += 8) store_8(row32 + 32 * x + e, f + e);
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int cc = word0 + 4 * x + c;
              if (rows >= C) *reinterpret_cast<uint4 *>(tile + row_tile_chunk(r, cc >> 3, cc & 7, C)) = pack8(f + 8 * c);
              else if (r < rows) *reinterpret_cast<uint4 *>(row + 8 * cc) = pack8(f + 8 * c);
            }
          }
        }
      };
      const size_t token = (size_t)(pos + r) * p.H + h;
      ok = wait.warp(y == 0 ? dq_done : y == 1 ? dk_done : dv_done, it, SITE_GRAD + 26);
      if (!ok) break;
      fence_after_sync();
      if (y >= 2) {
        out(T_V + (y - 2) * (DV / 2), DV / 2, sm + L::X + L::X1, (y - 2) * (DV / 16), reinterpret_cast<uint16_t *>(p.gv) + token * DV, nullptr);
      } else {
        const uint32_t col = y ? tm + lanes + T_K : T_Q;
        if (shared) out(col, DK, nullptr, 0, nullptr, (y ? gk32 : gq32) + token * DK);
        else out(col, DK, y ? mt : sm + L::X, 0, reinterpret_cast<uint16_t *>(y ? p.gk : p.gq) + token * DK, nullptr);
      }
      fence_before_sync();
      mbar_arrive(y == 0 ? q_free : y == 1 ? k_free : v_free);
      if (rows >= C) fence_async_smem();
      mbar_arrive(y == 0 ? dq_staged : y == 1 ? dk_staged : dv_staged);
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
// Chunks in a segment of the sweeps, or 0 to sweep whole sequences.  Few sequences and heads leave SMs idle: then segments,
// about one for each SM, are swept from states computed like the prefill's, in both directions.  A step of both sweeps
// takes 1.8 us and the states with their four more launches 36 to 57 us, so it takes 25 steps less to be worth it; the host
// knows the mean length only, which the longest sequence's steps are no fewer than.  Whole -> segments, d_k = d_v = 128:
// one head of 2048, 4096, 8192, 32768 tokens 63 -> 67, 92 -> 68, 150 -> 74, 547 -> 116 us; 4 heads of 4096, 8192
// 97 -> 85, 175 -> 114 us; 8 of 2048, 4096, 8192 67 -> 85, 113 -> 114, 201 -> 159 us; 16 of 4096, 8192 139 -> 160,
// 239 -> 232 us; 8 heads of two times 2048 82 -> 116 us; 2 heads of 262144 4.22 -> 0.67 ms, 16 of 65536 1.56 -> 1.27 ms.
// 32 heads have no SM for a second segment: two of 64 chunks made 16384 tokens slower, 600 -> 690 us.
inline int sweep_chunks(const LinearParams &p) {
  constexpr int kSms = 148, kWorth = 25;
  const long long lanes = (long long)p.H * (p.dv / kSlice), chunks = ((long long)p.N + C - 1) / C;
  if (p.num_seqs == 0 || lanes > kSms / 2) return 0;      // no SM for a second segment
  const long long segs = kSms / lanes;
  long long per = (chunks + segs - 1) / segs;
  if (per < 2) per = 2;
  if (per > lin::kMaxPer) per = lin::kMaxPer;
  // an SM's steps: more than one segment's where the plan's longest segment leaves more segments than SMs
  const long long steps = per * (((chunks + per - 1) / per * lanes + kSms - 1) / kSms);
  return chunks >= (steps + kWorth) * p.num_seqs ? (int)per : 0;
}

struct BackwardWorkspace {
  int per;      // chunks in a segment of the sweeps; 0: whole sequences
  size_t segs, sbase, order, seg_base, part, rpart, whole, through, tables, s, d, gq32, gk32, gla, bytes;
};
inline BackwardWorkspace backward_layout(const LinearParams &p) {
  const size_t chunks = lin::max_segments(p.N, p.num_seqs, C);
  BackwardWorkspace w{};
  w.per = sweep_chunks(p);
  w.segs = w.per ? lin::max_segments(p.N, p.num_seqs, C * w.per) : 0;
  auto take = [&](size_t n) {
    const size_t at = w.bytes;
    w.bytes += lin::align256(n);
    return at;
  };
  w.sbase = take(lin::table_bytes(p.num_seqs, chunks));
  w.order = take((size_t)p.num_seqs * 4);
  if (w.per) {
    w.seg_base = take(lin::table_bytes(p.num_seqs, w.segs));
    w.part = take(w.segs * p.H * (size_t)p.dk * p.dv * 4);
    w.rpart = take(w.segs * p.H * (size_t)p.dk * p.dv * 4);
    w.whole = take(w.segs * p.H * 4);
  }
  w.through = take(chunks * p.H * (p.dv / 8) * 4);
  w.tables = take(chunks * p.H * sizeof(Table));
  w.s = take(chunks * p.H * (size_t)p.dk * p.dv * 4);
  w.d = take(chunks * p.H * (size_t)p.dk * p.dv * 4);
  const size_t per_head = p.H != p.Hk ? (size_t)p.N * p.H * p.dk * 4 : 0;
  w.gq32 = take(per_head);
  w.gk32 = take(per_head);
  w.gla = take(p.decay_head ? (size_t)p.N * p.H * 4 : 0);
  return w;
}

template <int DK, int DV, bool CUT>
cudaError_t launch_sweeps(const LinearParams &p, const SweepMaps &mf, const SweepMaps &mr, const int *sbase, const int *order,
                          const int *segments, const float *part, const float *rpart, const Table *tables, float *through,
                          size_t items, cudaStream_t s) {
  constexpr int fwd_smem = SweepSmem<DK, false>::END, rev_smem = SweepSmem<DK, true>::END;
  cudaError_t e = lin::allow_smem<sweep_kernel<DK, DV, false, CUT>>(fwd_smem);
  if (e == cudaSuccess) e = lin::allow_smem<sweep_kernel<DK, DV, true, CUT>>(rev_smem);
  const unsigned grid = (unsigned)(items < (size_t)sm_count() ? items : (size_t)sm_count());
  if (e == cudaSuccess)
    e = launch_next(sweep_kernel<DK, DV, false, CUT>, grid, kSweepThreads, fwd_smem, s, p, mf, sbase, order, segments, part,
                    tables, nullptr);
  if (e == cudaSuccess)
    e = launch_next(sweep_kernel<DK, DV, true, CUT>, grid, kSweepThreads, rev_smem, s, p, mr, sbase, order, segments, rpart,
                    tables, through);
  return e;
}

template <int DK, int DV>
cudaError_t launch_backward(const LinearParams &p, const SweepMaps &mf, const SweepMaps &mr, const GradMaps &mg,
                            const BackwardWorkspace &w, size_t items, cudaStream_t s) {
  unsigned char *ws = static_cast<unsigned char *>(p.ws);
  const int *sbase = reinterpret_cast<const int *>(ws + w.sbase), *order = reinterpret_cast<const int *>(ws + w.order);
  float *through = reinterpret_cast<float *>(ws + w.through);
  const size_t sweeps = (w.per ? w.segs : (size_t)p.num_seqs) * p.H * (DV / kSlice);
  if (sweeps > 0x3FFFFFFFull || items * 2 * DK > 0x7FFFFFFFull) return cudaErrorInvalidValue;
  constexpr int grad_smem = GradSmem<DK, DV>::END;
  cudaError_t e = lin::allow_smem<grad_kernel<DK, DV>>(grad_smem);
  if (e != cudaSuccess) return e;
  Table *tables = reinterpret_cast<Table *>(ws + w.tables);
  const int *segments = nullptr;
  const float *part = nullptr, *rpart = nullptr;
  if (w.per) {
    segments = reinterpret_cast<const int *>(ws + w.seg_base);
    float *a = reinterpret_cast<float *>(ws + w.part), *b = reinterpret_cast<float *>(ws + w.rpart);
    e = launch_linear_segment_states_tc(p, segments, a, b, reinterpret_cast<float *>(ws + w.whole), w.segs, s);
    part = a;
    rpart = b;
  }
  if (e == cudaSuccess && items > 0) e = launch_next(table_kernel, (unsigned)((items + 7) / 8), 256, 0, s, p, sbase, tables);
  if (e == cudaSuccess)
    e = w.per ? launch_sweeps<DK, DV, true>(p, mf, mr, sbase, order, segments, part, rpart, tables, through, sweeps, s)
              : launch_sweeps<DK, DV, false>(p, mf, mr, sbase, order, segments, part, rpart, tables, through, sweeps, s);
  if (e != cudaSuccess || p.N == 0) return e;
  const bool shared = p.H != p.Hk;
  float *gla = p.decay_head ? reinterpret_cast<float *>(ws + w.gla) : p.gla;
  const unsigned grid = (unsigned)(items < (size_t)sm_count() ? items : (size_t)sm_count());
  return launch_next(grad_kernel<DK, DV>, grid, kGradThreads, grad_smem, s, p, mg, sbase, through,
                     shared ? reinterpret_cast<float *>(ws + w.gq32) : nullptr,
                     shared ? reinterpret_cast<float *>(ws + w.gk32) : nullptr, gla);
}

}  // namespace lintc

size_t linear_backward_tc_workspace(const LinearParams &p) { return lintc::backward_layout(p).bytes; }

cudaError_t launch_linear_backward_tc(const LinearParams &p, float **gq32, float **gk32, float **gla, cudaStream_t s) {
  using namespace lintc;
  const BackwardWorkspace w = backward_layout(p);
  const size_t items = lin::max_segments(p.N, p.num_seqs, C) * p.H;
  unsigned char *ws = static_cast<unsigned char *>(p.ws);
  const bool shared = p.H != p.Hk;
  *gq32 = shared ? reinterpret_cast<float *>(ws + w.gq32) : nullptr;
  *gk32 = shared ? reinterpret_cast<float *>(ws + w.gk32) : nullptr;
  *gla = p.decay_head ? reinterpret_cast<float *>(ws + w.gla) : p.gla;
  cudaError_t e = launch_linear_plan(p, reinterpret_cast<int *>(ws + w.sbase), C, 1, 1, 1,
                                     reinterpret_cast<int *>(ws + w.order), nullptr, s);
  if (e == cudaSuccess && w.per)
    e = launch_linear_plan(p, reinterpret_cast<int *>(ws + w.seg_base), C, w.per, w.per, 1, nullptr,
                           reinterpret_cast<int *>(ws + w.sbase), s);
  if (e != cudaSuccess) return e;
  GradMaps mg{};
  SweepMaps mf{}, mr{};
  if (p.N > 0) {
    const size_t rows = items * 2 * p.dk;
    const void *st = ws + w.s, *dt = ws + w.d;
    bool ok = encode(&mg.q, p.q, p.dk, p.Hk, p.N) && encode(&mg.k, p.k, p.dk, p.Hk, p.N) &&
              encode(&mg.v, p.v, p.dv, p.H, p.N) && encode(&mg.d_o, p.d_o, p.dv, p.H, p.N) &&
              encode(&mg.gv, p.gv, p.dv, p.H, p.N) && encode(&mg.s, st, p.dv, 1, rows, p.dk) &&
              encode(&mg.d, dt, p.dv, 1, rows, p.dk) && encode(&mf.v, p.v, p.dv, p.H, p.N, C, kSlice) &&
              encode(&mr.v, p.d_o, p.dv, p.H, p.N, C, kSlice) && encode(&mf.out, st, p.dv, 1, rows, p.dk, kSlice) &&
              encode(&mr.out, dt, p.dv, 1, rows, p.dk, kSlice);
    if (!shared) ok = ok && encode(&mg.gq, p.gq, p.dk, p.H, p.N) && encode(&mg.gk, p.gk, p.dk, p.H, p.N);
    if (!ok) return cudaErrorNotSupported;
    mf.k = mg.k;
    mr.k = mg.q;
    mr.s = mf.out;
  }
  if (p.dk == 128)
    return p.dv == 128 ? launch_backward<128, 128>(p, mf, mr, mg, w, items, s)
                       : launch_backward<128, 64>(p, mf, mr, mg, w, items, s);
  return p.dv == 128 ? launch_backward<64, 128>(p, mf, mr, mg, w, items, s)
                     : launch_backward<64, 64>(p, mf, mr, mg, w, items, s);
}

}  // namespace kda
