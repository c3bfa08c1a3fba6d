// Linear attention with a decay for each head: prefill and its backward pass for fp32 inputs (formulas in
// kda_linear.cuh); the plan of segments, the chain and the sums over shared inputs also for bf16 ones, whose
// products are in kda_linear_tc.cu and kda_linear_backward_tc.cu.
//
// Three steps, all parallel over segments and heads except the short middle one:
//   parts    each segment's own contribution to the state,  sum_s 2^{b_end - b_s} k_s v_s^T
//            (and for the backward pass to the gradient of the state at its start,
//            sum_t 2^{b_t} q_t do_t^T, the same product over the same rows in reverse)
//   chain    S <- a S + part over a sequence's segments, one thread per 4 state elements: the
//            parts are replaced by the states at the segments' starts (gradients at their ends)
//   rows     outputs (or gradients) of each segment from the state at its start
// The products run on the tensor cores as 3xTF32: x = hi + lo with tf32 hi, lo, and
// a b = a_h b_l + a_l b_h + a_h b_h, where the dropped term is below 2^-21 of the product.
// Chunks of 64 rows, so that the fp32 tiles of a chunk fit in shared memory.
#include "kda_linear.cuh"

namespace kda {
namespace lin {

constexpr int C = 64;
constexpr int kThreads = 512;       // a chunk's outputs are a chain of short steps: 16 warps hide each other's latency
                                   // (8 warps: gradients of 33 x 8 chunks of 64 x 128 in 93 instead of 80 us)
constexpr int kPartThreads = 256;   // many small blocks side by side: 8 warps each split fewer operands twice (27 / 34 us)
constexpr int kSlice = 64;          // d_v columns of a block in the parts and prefill rows kernels

// ------------------------------------------------------------------ 3xTF32 products
__device__ __forceinline__ void split_tf32(float x, uint32_t &hi, uint32_t &lo) {
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(hi) : "f"(x));
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(lo) : "f"(x - __uint_as_float(hi)));
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// The sums of 16 columns start from zero and are added by fp32 additions that round: chained into the accumulator, each
// of 3 K / 8 products lost up to 2^-23 of the whole sum, as a truncated addition does.  Errors against 64 bits
// 0.6 - 1.6e-6 -> 0.6 - 3.2e-7 for 2 - 8 % of the time (4096 tokens, 16 heads of 128: prefill 369 -> 396 us, backward
// 709 -> 768 us; sums of 8 columns 397 and 787 us, 1.3 - 2.0e-7).
// acc[m][n] += A B for a warp's 16 MT x 8 NT tile over K; a(r, k) and b(k, n) read the operands.
// Entry acc[m][n][e] is row 16 m + lane / 4 + 8 (e / 2), column 8 n + 2 (lane % 4) + e % 2.
template <int MT, int NT, int K, class FA, class FB>
__device__ __forceinline__ void gemm3(float (&acc)[MT][NT][4], FA a, FB b) {
  const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
#pragma unroll 1
  for (int k0 = 0; k0 < K; k0 += 16) {
    uint32_t ah[2][MT][4], al[2][MT][4];
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int k = k0 + 8 * y + t;
        split_tf32(a(16 * m + g, k), ah[y][m][0], al[y][m][0]);
        split_tf32(a(16 * m + g + 8, k), ah[y][m][1], al[y][m][1]);
        split_tf32(a(16 * m + g, k + 4), ah[y][m][2], al[y][m][2]);
        split_tf32(a(16 * m + g + 8, k + 4), ah[y][m][3], al[y][m][3]);
      }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      uint32_t bh[2][2], bl[2][2];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        split_tf32(b(k0 + 8 * y + t, 8 * n + g), bh[y][0], bl[y][0]);
        split_tf32(b(k0 + 8 * y + t + 4, 8 * n + g), bh[y][1], bl[y][1]);
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          mma_tf32(sum, ah[y][m], bl[y]);
          mma_tf32(sum, al[y][m], bh[y]);
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) mma_tf32(sum, ah[y][m], bh[y]);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[m][n][e] += sum[e];
      }
    }
  }
}
template <int MT, int NT>
__device__ __forceinline__ void zero(float (&acc)[MT][NT][4]) {
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[m][n][e] = 0.f;
}
// f(row, column, value) over a thread's accumulator entries.
template <int MT, int NT, class F>
__device__ __forceinline__ void each(float (&acc)[MT][NT][4], F f) {
  const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) f(16 * m + g + 8 * (e >> 1), 8 * n + 2 * t + (e & 1), acc[m][n][e]);
}

// ------------------------------------------------------------------ tiles
// Rows [pos0, pos0 + C) of x [N, heads, d], columns [c0, c0 + W) of head `hd`, with row stride LD.  Rows
// past `end` and pads are zeros and are not read.
template <int W, int LD, int T = kThreads>
__device__ __forceinline__ void load_rows(float *dst, const void *x, int heads, int d, int hd, int c0, int pos0,
                                          int end, const uint8_t *mask) {
  constexpr int V = W / 4;
#pragma unroll 4
  for (int i = threadIdx.x; i < C * V; i += T) {
    const int r = i / V, c = (i % V) * 4, pos = pos0 + r;
    float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
    if (pos < end && (mask == nullptr || mask[pos] != 0))
      u = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(x) + ((size_t)pos * heads + hd) * d + c0 + c);
    *reinterpret_cast<float4 *>(dst + r * LD + c) = u;
  }
}

// A chunk's decays.  Filled by the first warp; the block synchronises after it.
struct Decays {
  float hi[C], lo[C];      // b, log2
  float from[C];           // 2^b: from the chunk's start to the row
  float to[C];             // 2^{b_C - b}: from the row to the chunk's end
  float whole;             // 2^{b_C}
};
__device__ __forceinline__ void chunk_decays(Decays &d, const LinearParams &p, int pos0, int end, int h) {
  const int lane = threadIdx.x & 31;
  double x[2], s;
#pragma unroll
  for (int e = 0; e < 2; ++e) x[e] = log2_decay(p.log_alpha, p.decay_head, p.mask, pos0 + 2 * lane + e, end, h, p.H);
  s = x[0] + x[1];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = shfl_up_f64(s, o);
    if (lane >= o) s += y;
  }
  const double total = shfl_f64(s, 31);
  const double before = shfl_up_f64(s, 1), b[2] = {(lane ? before : 0.0) + x[0], s};
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = 2 * lane + e;
    d.hi[r] = (float)b[e];
    d.lo[r] = (float)(b[e] - (double)d.hi[r]);
    d.from[r] = exp2f((float)b[e]);
    d.to[r] = exp2f((float)(total - b[e]));
  }
  if (lane == 0) d.whole = exp2f((float)total);
}
__device__ __forceinline__ float pair_decay(const Decays &d, int t, int s) {
  return exp2f((d.hi[t] - d.hi[s]) + (d.lo[t] - d.lo[s]));
}

// ------------------------------------------------------------------ plan
// Checks cu_seqlens (nothing else runs if it is invalid), takes the number of chunks in a segment, lo .. hi, and fills
// the segment table, longest segments first.  In the time of a chunk on one SM: a segment costs its chunks and about a half
// more (its state in and out), and its share of the state half of up to six chunks (a share ends where the decays
// are 0 in fp32; six fits a mean log of -0.18 a token, slower decays walk the whole segment).  The longest run over the SMs is no shorter than the mean, nor than r + 1 times the segment in place
// r x SMs, since one SM has r + 1 of the segments up to there.  Against the best of 1, 2, .. 64 chunks, measured one by
// one, the count so taken costs 0 to 5 % more on nine batches of 2048 to 32768 tokens and on 131072 tokens.  The
// lengths are known here only.  order (may be null): the sequences from the longest to the shortest (unsorted beyond
// those whose tables fit in shared memory).  earlier (may be null): the table of the call's plan before this one; both are
// refused or none.
constexpr int kCached = 1024;      // sequences whose tables fit in shared memory
__global__ void __launch_bounds__(1024) plan_kernel(LinearParams p, int *sbase, int chunk, int lo, int hi, int sms,
                                                    int *order, int *earlier) {
  __shared__ int tot[32], carry, bad, most, slot[kMaxPer + 1], s_cu[kCached + 1], s_base[kCached + 1];
  __shared__ int lengths[32][kMaxPer + 1];
  __shared__ unsigned best;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  if (tid == 0) { carry = 0; bad = 0; most = lo; best = 0xFFFFFFFFu; }
  if (tid <= kMaxPer) slot[tid] = 0;
  __syncthreads();
  let_next_start();
  const bool stop = earlier != nullptr && earlier[p.num_seqs] == kRefused;
  if (__syncthreads_or(stop || device_error_latched(p.err))) {
    if (tid == 0) {
      sbase[p.num_seqs] = kRefused;
      if (earlier != nullptr) earlier[p.num_seqs] = kRefused;
    }
    return;
  }
  const bool cached = p.num_seqs <= kCached;
  int wrong = 0, top = 0;
  for (int i = tid; i <= p.num_seqs; i += 1024) {
    const int c = p.cu[i], d = i > 0 ? p.cu[i - 1] : 0;
    if (cached) s_cu[i] = c;
    if (c < 0 || c > p.N || (i == 0 && c != 0) || (i == p.num_seqs && c != p.N) || d > c) wrong = 1;
    top = max(top, c - d);
  }
  if (wrong) atomicOr(&bad, 1);
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  if (lane == 0 && top > 0) atomicMax(&most, (top + chunk - 1) / chunk);
  __syncthreads();
  if (bad) {
    if (tid == 0) {
      atomicOr(p.err, ERR_BIT_CHECK);
      sbase[p.num_seqs] = kRefused;
    }
    return;
  }
  const int *cu = cached ? s_cu : p.cu, *base = cached ? s_base : sbase;
  auto chunks = [&](int b) { return (cu[b + 1] - cu[b] + chunk - 1) / chunk; };
  hi = min(hi, most);      // chunks of the longest sequence (lo at least)
  if (hi > lo) {
    for (int per = lo + w; per <= hi; per += 32) {      // a warp for each count
      for (int n = lane; n <= kMaxPer; n += 32) lengths[w][n] = 0;
      __syncwarp();
      int all = 0, segs = 0;
      for (int b = lane; b < p.num_seqs; b += 32) {
        const int n = chunks(b), f = n / per, rest = n - f * per;
        all += n;
        segs += f + (rest > 0);
        if (f > 0) atomicAdd(&lengths[w][per], f);
        if (rest > 0) atomicAdd(&lengths[w][rest], 1);
      }
      __syncwarp();
      all = __reduce_add_sync(0xFFFFFFFFu, all);
      segs = __reduce_add_sync(0xFFFFFFFFu, segs);
      const int at = lane * sms / p.H;                  // this lane: r = lane
      int place = 0, longest = 0;
#pragma unroll 8
      for (int n = per; n > 0; --n) {
        place += lengths[w][n];
        longest = longest == 0 && place > at ? n : longest;
      }
      const float heads = (float)p.H / (float)sms, mean = ((float)all + 0.5f * (float)segs) * heads;
      int run = (lane + 1) * (longest > 0 ? 2 * longest + 1 : 0);      // in halves of a chunk
      run = __reduce_max_sync(0xFFFFFFFFu, run);
      const float cost = fmaxf(mean, 0.5f * (float)run) + ceilf((float)segs * heads) * 0.5f * (float)min(per, 6);
      // quarters of a chunk's time in 24 bits, then the count
      if (lane == 0) atomicMin(&best, (unsigned)fminf(4.f * cost, 16e6f) << 8 | (unsigned)per);
    }
    __syncthreads();
  }
  const int per = hi > lo ? (int)(best & 0xFFu) : lo;
  for (int b0 = 0; b0 <= p.num_seqs; b0 += 1024) {
    const int b = b0 + tid;
    const int n = b < p.num_seqs ? (chunks(b) + per - 1) / per : 0;
    int x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) tot[w] = x;
    __syncthreads();
    int before = carry;
    for (int i = 0; i < w; ++i) before += tot[i];
    if (b <= p.num_seqs) {
      sbase[b] = before + x - n;
      if (cached) s_base[b] = before + x - n;
    }
    __syncthreads();
    if (tid == 1023) carry = before + x;
    __syncthreads();
  }
  Segment *table = const_cast<Segment *>(segment_table(sbase, p.num_seqs));
  const int segs = carry;
  auto find = [&](int i, int &n) {
    int a = 0, z = p.num_seqs - 1;           // the last sequence whose segments begin at or before i
    while (a < z) {
      const int mid = (a + z + 1) >> 1;
      if (base[mid] <= i) a = mid; else z = mid - 1;
    }
    Segment s;
    const int e = cu[a + 1], tokens = chunk * per;
    s.id = i;
    s.begin = cu[a] + (i - base[a]) * tokens;
    s.end = min(e, s.begin + tokens);
    s.of = a << 1 | (s.begin + tokens >= e ? 1 : 0);
    n = (s.end - s.begin + chunk - 1) / chunk;
    return s;
  };
  if (order != nullptr)
    for (int b = tid; b < p.num_seqs; b += 1024) {
      int place = b;
      if (cached) {
        const int n = cu[b + 1] - cu[b];
        place = 0;
        for (int i = 0; i < p.num_seqs; ++i) {
          const int m = cu[i + 1] - cu[i];
          place += m > n || (m == n && i < b);
        }
      }
      order[place] = b;
    }
  if (per == 1) {
    int n;
    for (int i = tid; i < segs; i += 1024) table[i] = find(i, n);
    return;
  }
  for (int i = tid; i < segs; i += 1024) {
    int n;
    find(i, n);
    atomicAdd(&slot[n], 1);
  }
  __syncthreads();
  if (w == 0) {      // places of the lengths, from the longest: lane's are kMaxPer - 2 lane and the one before it
    const int a = slot[kMaxPer - 2 * lane], b = slot[kMaxPer - 2 * lane - 1];
    int x = a + b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += y;
    }
    slot[kMaxPer - 2 * lane] = x - a - b;
    slot[kMaxPer - 2 * lane - 1] = x - b;
  }
  __syncthreads();
  for (int i = tid; i < segs; i += 1024) {
    int n;
    const Segment s = find(i, n);
    table[atomicAdd(&slot[n], 1)] = s;       // equal lengths in any order: it decides nothing but who computes what
  }
}

// ------------------------------------------------------------------ parts
// Block: segment x head x 64 columns of d_v.  REVERSE: q, do and the rows in reverse.
template <int DK, bool REVERSE>
__device__ __forceinline__ void parts_block(const LinearParams &p, const Segment &sg, int seg, int h, int c0,
                                            float *part, float *whole, float *sm, Decays &dec) {
  constexpr int LK = DK + 4, LV = kSlice + 4, MT = DK / 64;
  float *sk = sm, *sv = sm + C * LK;
  const int warp = threadIdx.x >> 5, m0 = (warp & 3) * 16 * MT, n0 = (warp >> 2) * 32;
  const int hk = h / (p.H / p.Hk);
  float acc[MT][4][4], keep = 1.f;
  zero(acc);
  const int chunks = (sg.end - sg.begin + C - 1) / C;
  for (int j = 0; j < chunks; ++j) {
    const int pos0 = sg.begin + (REVERSE ? chunks - 1 - j : j) * C;
    __syncthreads();
    load_rows<DK, LK, kPartThreads>(sk, REVERSE ? p.q : p.k, p.Hk, DK, hk, 0, pos0, sg.end, p.mask);
    load_rows<kSlice, LV, kPartThreads>(sv, REVERSE ? p.d_o : p.v, p.H, p.dv, h, c0, pos0, sg.end, p.mask);
    if (warp == 0) chunk_decays(dec, p, pos0, sg.end, h);
    __syncthreads();
    const float a = dec.whole, *wgt = REVERSE ? dec.from : dec.to;
    keep *= a;
    each(acc, [&](int, int, float &x) { x *= a; });
    gemm3<MT, 4, C>(acc, [&](int r, int k) { return sk[k * LK + m0 + r] * wgt[k]; },
                    [&](int k, int n) { return sv[k * LV + n0 + n]; });
  }
  float *out = part + ((size_t)seg * p.H + h) * DK * p.dv + c0;
  each(acc, [&](int r, int n, float &x) { out[(size_t)(m0 + r) * p.dv + n0 + n] = x; });
  if (!REVERSE && c0 == 0 && threadIdx.x == 0) whole[(size_t)seg * p.H + h] = keep;
}

template <int DK>
__global__ void __launch_bounds__(kPartThreads) parts_kernel(LinearParams p, const int *sbase, float *part, float *rpart,
                                                         float *whole) {
  extern __shared__ float sm[];
  __shared__ Decays dec;
  after_previous();
  if (call_ended(p, sbase)) return;
  const int slices = p.dv / kSlice;
  const int seg = blockIdx.x / (p.H * slices), h = blockIdx.x / slices % p.H, c0 = (blockIdx.x % slices) * kSlice;
  if (seg >= sbase[p.num_seqs]) return;
  const Segment sg = locate(sbase, p.num_seqs, seg);
  if (blockIdx.y == 0) parts_block<DK, false>(p, sg, seg, h, c0, part, whole, sm, dec);
  else parts_block<DK, true>(p, sg, seg, h, c0, rpart, nullptr, sm, dec);
}
template <int DK> constexpr size_t parts_smem() { return (size_t)C * (DK + 4 + kSlice + 4) * 4; }

// ------------------------------------------------------------------ chain
// grid: (B H, d_k d_v / 1024, 1 or 2); thread: 4 elements of a sequence's and head's state.
// z = 0 forwards from init_state, 1 backwards from the final state's gradient.
__global__ void __launch_bounds__(256) chain_kernel(LinearParams p, const int *sbase, float *part, float *rpart,
                                                    const float *whole) {
  after_previous();
  if (call_ended(p, sbase)) return;
  const bool back = blockIdx.z != 0;
  const size_t bh = blockIdx.x, per = (size_t)p.dk * p.dv;
  const int b = (int)(bh / p.H), h = (int)(bh % p.H);
  const size_t e = (size_t)blockIdx.y * 256 + threadIdx.x;
  const int s0 = sbase[b], s1 = sbase[b + 1];
  const float *in = back ? p.d_final : p.init_state;
  float *out = back ? p.g_init : p.final_state;
  float4 S = in ? reinterpret_cast<const float4 *>(in + bh * per)[e] : make_float4(0.f, 0.f, 0.f, 0.f);
  float *x = back ? rpart : part;
  const int n = s1 - s0;
  constexpr int AHEAD = 8;             // loads in flight ahead of the chain
  for (int i0 = 0; i0 < n; i0 += AHEAD) {
    float4 v[AHEAD];
    float a[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (i0 + i < n) {
        const size_t at = (size_t)(back ? s1 - 1 - i0 - i : s0 + i0 + i) * p.H + h;
        v[i] = reinterpret_cast<const float4 *>(x + at * per)[e];
        a[i] = whole[at];
      }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (i0 + i < n) {
        const size_t at = (size_t)(back ? s1 - 1 - i0 - i : s0 + i0 + i) * p.H + h;
        reinterpret_cast<float4 *>(x + at * per)[e] = S;
        S.x = fmaf(a[i], S.x, v[i].x);
        S.y = fmaf(a[i], S.y, v[i].y);
        S.z = fmaf(a[i], S.z, v[i].z);
        S.w = fmaf(a[i], S.w, v[i].w);
      }
  }
  if (out) reinterpret_cast<float4 *>(out + bh * per)[e] = S;
}

// ------------------------------------------------------------------ prefill rows
template <int DK>
__global__ void __launch_bounds__(kThreads, DK == 64 ? 2 : 1) rows_kernel(LinearParams p, const int *sbase, const float *start) {
  constexpr int LK = DK + 4, LV = kSlice + 4, MT = DK / 64;
  extern __shared__ float sm[];
  __shared__ Decays dec;
  float *sq = sm, *sk = sq + C * LK, *sv = sk + C * LK, *sS = sv + C * LV, *sP = sS + DK * LV;
  after_previous();
  if (call_ended(p, sbase)) return;
  const int slices = p.dv / kSlice;
  const int seg = blockIdx.x / (p.H * slices), h = blockIdx.x / slices % p.H, c0 = (blockIdx.x % slices) * kSlice;
  if (seg >= sbase[p.num_seqs]) return;
  const Segment sg = locate(sbase, p.num_seqs, seg);
  const int hk = h / (p.H / p.Hk);
  const int warp = threadIdx.x >> 5, m0 = (warp & 3) * 16, n0 = (warp >> 2) * 16;
  float S[MT][2][4];                 // rows MT m0 .., columns n0 .. of the state
  const float *in = start + ((size_t)seg * p.H + h) * DK * p.dv + c0;
  each(S, [&](int r, int n, float &x) { x = in[(size_t)(m0 * MT + r) * p.dv + n0 + n]; });
  const int chunks = (sg.end - sg.begin + C - 1) / C;
  for (int j = 0; j < chunks; ++j) {
    const int pos0 = sg.begin + j * C;
    __syncthreads();
    load_rows<DK, LK>(sq, p.q, p.Hk, DK, hk, 0, pos0, sg.end, p.mask);
    load_rows<DK, LK>(sk, p.k, p.Hk, DK, hk, 0, pos0, sg.end, p.mask);
    load_rows<kSlice, LV>(sv, p.v, p.H, p.dv, h, c0, pos0, sg.end, p.mask);
    each(S, [&](int r, int n, float &x) { sS[(m0 * MT + r) * LV + n0 + n] = x; });
    if (warp == 0) chunk_decays(dec, p, pos0, sg.end, h);
    __syncthreads();
    float o[1][2][4], A[1][2][4];
    zero(A);
    if (n0 <= m0 + 15)               // else above the diagonal
      gemm3<1, 2, DK>(A, [&](int r, int k) { return sq[(m0 + r) * LK + k]; },
                      [&](int k, int n) { return sk[(n0 + n) * LK + k]; });
    each(A, [&](int r, int n, float &x) {
      const int t = m0 + r, s = n0 + n;
      sP[t * LV + s] = s <= t ? x * pair_decay(dec, t, s) : 0.f;
    });
    zero(o);
    gemm3<1, 2, DK>(o, [&](int r, int k) { return sq[(m0 + r) * LK + k]; },
                    [&](int k, int n) { return sS[k * LV + n0 + n]; });
    each(o, [&](int r, int, float &x) { x *= dec.from[m0 + r]; });
    __syncthreads();
    gemm3<1, 2, C>(o, [&](int r, int k) { return sP[(m0 + r) * LV + k]; },
                   [&](int k, int n) { return sv[k * LV + n0 + n]; });
    each(o, [&](int r, int n, float &x) {
      const int pos = pos0 + m0 + r;
      if (pos < sg.end) store_elem<false>(p.o, ((size_t)pos * p.H + h) * p.dv + c0 + n0 + n, x);
    });
    if (j + 1 < chunks) {
      each(S, [&](int, int, float &x) { x *= dec.whole; });
      gemm3<MT, 2, C>(S, [&](int r, int k) { return sk[k * LK + m0 * MT + r] * dec.to[k]; },
                      [&](int k, int n) { return sv[k * LV + n0 + n]; });
    }
  }
}
template <int DK> constexpr size_t rows_smem() {
  return (size_t)(2 * C * (DK + 4) + (2 * C + DK) * (kSlice + 4)) * 4;
}

// ------------------------------------------------------------------ gradients of a chunk
// Block: chunk (a segment of one chunk) x head, with the state S at its start and the state's
// gradient D at its end.  With M = tril(dO V^T o 2^{b_t - b_s}), P = tril(Q K^T o 2^{b_t - b_s}):
//   dQ = M K + Diag(2^b) dO S^T,  dK = M^T Q + Diag(2^{b_C-b}) V D^T,  dV = P^T dO + Diag(2^{b_C-b}) K D
//   dlog_alpha_u = sum_{t>=u} 2^{b_t} q_t.S do_t + sum_{s<u} 2^{b_C-b_s} k_s.D v_s + 2^{b_C} <S, D>
//                + sum_{t>=u>s} (q_t.k_s)(do_t.v_s) 2^{b_t-b_s}
// (what passes over row u: to later rows, from earlier rows, through the chunk, inside it).
// S and D are taken in halves of 64 rows, one after the other through the same tile.
template <int DK, int DV>
struct GradSmem {
  static constexpr int LK = DK + 4, LV = DV + 4, LP = C + 4;
  static constexpr int Q = 0, K = Q + C * LK, V = K + C * LK, O = V + C * LV;
  static constexpr int P = O + C * LV, M = P + C * LP, S = M + C * LP, END = S + C * (LV > LP ? LV : LP);
};

// x[row] += sum of f's values over the warp's columns of the row, kept per warp column in part[4][C].
template <int NT, class F>
__device__ __forceinline__ void row_sums(float (&acc)[1][NT][4], float *part, int m0, int wn, F f) {
  const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
  float s[2] = {0.f, 0.f};
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e >> 1] += f(g + 8 * (e >> 1), 8 * n + 2 * t + (e & 1), acc[0][n][e]);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    s[i] += __shfl_xor_sync(0xFFFFFFFFu, s[i], 1);
    s[i] += __shfl_xor_sync(0xFFFFFFFFu, s[i], 2);
    if (t == 0) part[wn * C + m0 + g + 8 * i] += s[i];
  }
}

template <int DK, int DV>
__global__ void __launch_bounds__(kThreads) grad_kernel(LinearParams p, const int *sbase, const float *start,
                                                        const float *dend, float *gq32, float *gk32, float *gla) {
  using L = GradSmem<DK, DV>;
  constexpr int LK = L::LK, LV = L::LV, LP = L::LP, HALVES = DK / 64, NV = DV / 32;
  extern __shared__ float sm[];
  __shared__ Decays dec;
  __shared__ float r_part[4 * C], k_part[4 * C], pair_sum[C], red[kThreads / 32];
  after_previous();
  if (call_ended(p, sbase)) return;
  const int seg = blockIdx.x / p.H, h = blockIdx.x % p.H;
  if (seg >= sbase[p.num_seqs]) return;
  const Segment sg = locate(sbase, p.num_seqs, seg);
  const int hk = h / (p.H / p.Hk), pos0 = sg.begin, tid = threadIdx.x;
  const int warp = tid >> 5, m0 = (warp & 3) * 16, wn = warp >> 2, n0 = wn * 16;
  float *sq = sm + L::Q, *sk = sm + L::K, *sv = sm + L::V, *so = sm + L::O, *sP = sm + L::P, *sM = sm + L::M,
        *sS = sm + L::S;
  load_rows<DK, LK>(sq, p.q, p.Hk, DK, hk, 0, pos0, sg.end, p.mask);
  load_rows<DK, LK>(sk, p.k, p.Hk, DK, hk, 0, pos0, sg.end, p.mask);
  load_rows<DV, LV>(sv, p.v, p.H, DV, h, 0, pos0, sg.end, p.mask);
  load_rows<DV, LV>(so, p.d_o, p.H, DV, h, 0, pos0, sg.end, p.mask);
  if (warp == 0) chunk_decays(dec, p, pos0, sg.end, h);
  if (tid < 4 * C) r_part[tid] = k_part[tid] = 0.f;
  __syncthreads();
  {
    float A[1][2][4], G[1][2][4];
    zero(A);
    zero(G);
    if (n0 <= m0 + 15) {
      gemm3<1, 2, DK>(A, [&](int r, int k) { return sq[(m0 + r) * LK + k]; },
                      [&](int k, int n) { return sk[(n0 + n) * LK + k]; });
      gemm3<1, 2, DV>(G, [&](int r, int k) { return so[(m0 + r) * LV + k]; },
                      [&](int k, int n) { return sv[(n0 + n) * LV + k]; });
    }
    each(G, [&](int r, int n, float &x) {
      const int t = m0 + r, s = n0 + n;
      sM[t * LP + s] = s <= t ? x * pair_decay(dec, t, s) : 0.f;
    });
    each(A, [&](int r, int n, float &x) {
      const int t = m0 + r, s = n0 + n;
      sS[t * LP + s] = s < t ? x * sM[t * LP + s] : 0.f;      // the pairs' shares (own entries)
      sP[t * LP + s] = s <= t ? x * pair_decay(dec, t, s) : 0.f;
    });
  }
  __syncthreads();
  if (tid < C) {                     // column tid: sums over t >= u, in place
    float a = 0.f;
    for (int t = C - 1; t > tid; --t) {
      a += sS[t * LP + tid];
      sS[t * LP + tid] = a;
    }
  }
  __syncthreads();
  if (tid < C) {
    float a = 0.f;
    for (int s = 0; s < tid; ++s) a += sS[tid * LP + s];
    pair_sum[tid] = a;
  }
  const float *gS = start + ((size_t)seg * p.H + h) * DK * DV, *gD = dend + ((size_t)seg * p.H + h) * DK * DV;
  float through = 0.f;
  float av[1][NV][4];
  zero(av);
#pragma unroll 1
  for (int half = 0; half < HALVES; ++half) {
    const int k0 = half * 64;
    __syncthreads();
    for (int i = tid; i < 64 * DV / 4; i += kThreads) {
      const int r = i / (DV / 4), c = i % (DV / 4) * 4;
      const float4 x = *reinterpret_cast<const float4 *>(gS + (size_t)(k0 + r) * DV + c);
      const float4 y = *reinterpret_cast<const float4 *>(gD + (size_t)(k0 + r) * DV + c);
      through += x.x * y.x + x.y * y.y + x.z * y.z + x.w * y.w;
      *reinterpret_cast<float4 *>(sS + r * LV + c) = x;
    }
    __syncthreads();
    float acc[1][2][4];
    zero(acc);
    gemm3<1, 2, DV>(acc, [&](int r, int k) { return so[(m0 + r) * LV + k]; },
                    [&](int k, int n) { return sS[(n0 + n) * LV + k]; });
    each(acc, [&](int r, int, float &x) { x *= dec.from[m0 + r]; });
    row_sums(acc, r_part, m0, wn, [&](int r, int n, float x) { return x * sq[(m0 + r) * LK + k0 + n0 + n]; });
    gemm3<1, 2, C>(acc, [&](int r, int k) { return sM[(m0 + r) * LP + k]; },
                   [&](int k, int n) { return sk[k * LK + k0 + n0 + n]; });
    each(acc, [&](int r, int n, float &x) {
      const int pos = pos0 + m0 + r;
      if (pos >= sg.end) return;
      if (gq32) gq32[((size_t)pos * p.H + h) * DK + k0 + n0 + n] = x;
      else store_elem<false>(p.gq, ((size_t)pos * p.H + h) * DK + k0 + n0 + n, x);
    });
    __syncthreads();
    for (int i = tid; i < 64 * DV / 4; i += kThreads) {
      const int r = i / (DV / 4), c = i % (DV / 4) * 4;
      *reinterpret_cast<float4 *>(sS + r * LV + c) = *reinterpret_cast<const float4 *>(gD + (size_t)(k0 + r) * DV + c);
    }
    __syncthreads();
    zero(acc);
    gemm3<1, 2, DV>(acc, [&](int r, int k) { return sv[(m0 + r) * LV + k]; },
                    [&](int k, int n) { return sS[(n0 + n) * LV + k]; });
    each(acc, [&](int r, int, float &x) { x *= dec.to[m0 + r]; });
    row_sums(acc, k_part, m0, wn, [&](int r, int n, float x) { return x * sk[(m0 + r) * LK + k0 + n0 + n]; });
    gemm3<1, 2, C>(acc, [&](int r, int k) { return sM[k * LP + m0 + r]; },
                   [&](int k, int n) { return sq[k * LK + k0 + n0 + n]; });
    each(acc, [&](int r, int n, float &x) {
      const int pos = pos0 + m0 + r;
      if (pos >= sg.end) return;
      if (gk32) gk32[((size_t)pos * p.H + h) * DK + k0 + n0 + n] = x;
      else store_elem<false>(p.gk, ((size_t)pos * p.H + h) * DK + k0 + n0 + n, x);
    });
    gemm3<1, NV, 64>(av, [&](int r, int k) { return sk[(m0 + r) * LK + k0 + k]; },
                     [&](int k, int n) { return sS[k * LV + wn * (DV / 4) + n]; });
  }
  each(av, [&](int r, int, float &x) { x *= dec.to[m0 + r]; });
  gemm3<1, NV, C>(av, [&](int r, int k) { return sP[k * LP + m0 + r]; },
                  [&](int k, int n) { return so[k * LV + wn * (DV / 4) + n]; });
  each(av, [&](int r, int n, float &x) {
    const int pos = pos0 + m0 + r;
    if (pos < sg.end) store_elem<false>(p.gv, ((size_t)pos * p.H + h) * DV + wn * (DV / 4) + n, x);
  });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) through += __shfl_xor_sync(0xFFFFFFFFu, through, o);
  if ((tid & 31) == 0) red[warp] = through;
  __syncthreads();
  if (tid < C && pos0 + tid < sg.end) {
    float x = 0.f, r = 0.f, k = 0.f;
    for (int i = 0; i < kThreads / 32; ++i) x += red[i];
    for (int t = C - 1; t >= tid; --t) r += (r_part[t] + r_part[C + t]) + (r_part[2 * C + t] + r_part[3 * C + t]);
    for (int s = 0; s < tid; ++s) k += (k_part[s] + k_part[C + s]) + (k_part[2 * C + s] + k_part[3 * C + s]);
    const bool pad = p.mask != nullptr && p.mask[pos0 + tid] == 0;
    const float g = pad ? 0.f : pair_sum[tid] + r + k + dec.whole * x;
    // one decay per head: [H, N] for the sum that follows
    gla[p.decay_head ? (size_t)h * p.N + pos0 + tid : (size_t)(pos0 + tid) * p.H + h] = g;
  }
}

// ------------------------------------------------------------------ sums over shared inputs
// dq, dk of a key head: the value heads' fp32 gradients added in order.  Thread: 4 columns.
template <bool BF16>
__global__ void __launch_bounds__(256) share_kernel(LinearParams p, const int *sbase, const float *gq32,
                                                    const float *gk32) {
  after_previous();
  if (call_ended(p, sbase)) return;
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x, per = p.dk / 4;
  if (i >= (size_t)p.N * p.Hk * per) return;
  const int G = p.H / p.Hk, c = (int)(i % per);
  const size_t row = i / per;          // pos Hk + hk
  const float4 *x = reinterpret_cast<const float4 *>(blockIdx.y ? gk32 : gq32) + row * G * per + c;
  float4 s = x[0];
  for (int g = 1; g < G; ++g) {
    const float4 y = x[g * per];
    s.x += y.x; s.y += y.y; s.z += y.z; s.w += y.w;
  }
  void *out = blockIdx.y ? p.gk : p.gq;
  const size_t at = row * p.dk + 4 * c;
  store_elem<BF16>(out, at, s.x);
  store_elem<BF16>(out, at + 1, s.y);
  store_elem<BF16>(out, at + 2, s.z);
  store_elem<BF16>(out, at + 3, s.w);
}

// The gradient of a head's constant log_alpha: the sum over the tokens, in 64 bits and a fixed order.
__global__ void __launch_bounds__(1024) head_decay_kernel(LinearParams p, const int *sbase, const float *gla) {
  __shared__ double s[32];
  after_previous();
  if (call_ended(p, sbase)) return;
  const int h = blockIdx.x;
  double a = 0.0;
  for (int i = threadIdx.x; i < p.N; i += 1024) a += (double)gla[(size_t)h * p.N + i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    a += __hiloint2double(__shfl_xor_sync(0xFFFFFFFFu, __double2hiint(a), o),
                          __shfl_xor_sync(0xFFFFFFFFu, __double2loint(a), o));
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = a;
  __syncthreads();
  if (threadIdx.x == 0) {
    a = 0.0;
    for (int i = 0; i < 32; ++i) a += s[i];
    p.gla[h] = (float)a;
  }
}

// ------------------------------------------------------------------ host
// Chunks in a segment of the prefill: as many as leave about six blocks per SM, since the
// chain and its states (written and read once per segment) shrink with longer segments.
int segment_chunks(int N, int B, int blocks_per_chunk, int chunk) {
  int per = 1;
  while (per < 64 && ((size_t)N / (chunk * 2 * per) + B) * (size_t)blocks_per_chunk >= 6 * 148) per *= 2;
  return per;
}
size_t state_bytes(const LinearParams &p, size_t segs) { return align256(segs * p.H * (size_t)p.dk * p.dv * 4); }

template <int DK>
cudaError_t launch_parts(const LinearParams &p, const int *sbase, float *part, float *rpart, float *whole, size_t segs,
                         cudaStream_t s) {
  const size_t blocks = segs * p.H * (p.dv / kSlice);
  if (blocks > 0x7FFFFFFFull) return cudaErrorInvalidValue;
  const cudaError_t e = allow_smem<parts_kernel<DK>>(parts_smem<DK>());
  if (e != cudaSuccess) return e;
  if (blocks == 0) return cudaSuccess;
  return launch_next(parts_kernel<DK>, dim3((unsigned)blocks, rpart ? 2 : 1), kPartThreads, parts_smem<DK>(), s, p, sbase,
                     part, rpart, whole);
}
cudaError_t launch_parts_chain(const LinearParams &p, const int *sbase, float *part, float *rpart, float *whole,
                               size_t segs, cudaStream_t s) {
  const cudaError_t e = p.dk == 128 ? launch_parts<128>(p, sbase, part, rpart, whole, segs, s)
                                    : launch_parts<64>(p, sbase, part, rpart, whole, segs, s);
  if (e != cudaSuccess) return e;
  return launch_linear_chain(p, sbase, part, rpart, whole, s);
}

template <int DK>
cudaError_t launch_rows(const LinearParams &p, const int *sbase, const float *start, size_t segs,
                        cudaStream_t s) {
  const cudaError_t e = allow_smem<rows_kernel<DK>>(rows_smem<DK>());
  if (e != cudaSuccess) return e;
  return launch_next(rows_kernel<DK>, (unsigned)(segs * p.H * (p.dv / kSlice)), kThreads, rows_smem<DK>(), s, p, sbase,
                     start);
}

template <int DK, int DV>
cudaError_t launch_grad(const LinearParams &p, const int *sbase, const float *start, const float *dend, float *gq32,
                        float *gk32, float *gla, size_t segs, cudaStream_t s) {
  constexpr size_t smem = (size_t)GradSmem<DK, DV>::END * 4;
  const cudaError_t e = allow_smem<grad_kernel<DK, DV>>(smem);
  if (e != cudaSuccess) return e;
  return launch_next(grad_kernel<DK, DV>, (unsigned)(segs * p.H), kThreads, smem, s, p, sbase, start, dend, gq32, gk32, gla);
}
cudaError_t launch_grad_dims(const LinearParams &p, const int *sbase, const float *start, const float *dend,
                             float *gq32, float *gk32, float *gla, size_t segs, cudaStream_t s) {
  if (p.dk == 128)
    return p.dv == 128 ? launch_grad<128, 128>(p, sbase, start, dend, gq32, gk32, gla, segs, s)
                       : launch_grad<128, 64>(p, sbase, start, dend, gq32, gk32, gla, segs, s);
  return p.dv == 128 ? launch_grad<64, 128>(p, sbase, start, dend, gq32, gk32, gla, segs, s)
                     : launch_grad<64, 64>(p, sbase, start, dend, gq32, gk32, gla, segs, s);
}

}  // namespace lin

cudaError_t launch_linear_plan(const LinearParams &p, int *sbase, int chunk, int lo, int hi, int sms, int *order,
                               int *earlier, cudaStream_t s) {
  lin::plan_kernel<<<1, 1024, 0, s>>>(p, sbase, chunk, lo, hi < lin::kMaxPer ? hi : lin::kMaxPer, sms, order, earlier);
  return cudaGetLastError();
}

cudaError_t launch_linear_chain(const LinearParams &p, const int *sbase, float *part, float *rpart, const float *whole,
                                cudaStream_t s) {
  const unsigned nx = (unsigned)(p.dk * p.dv / 1024);
  return launch_next(lin::chain_kernel, dim3((unsigned)(p.num_seqs * p.H), nx, rpart ? 2 : 1), 256, 0, s, p, sbase, part,
                     rpart, whole);
}

size_t linear_prefill_workspace(const LinearParams &p, bool bf16) {
  using namespace lin;
  if (bf16) return linear_prefill_tc_workspace(p);
  const int per = segment_chunks(p.N, p.num_seqs, p.H * (p.dv / kSlice), C);
  const size_t segs = max_segments(p.N, p.num_seqs, C * per);
  return table_bytes(p.num_seqs, segs) + align256(segs * p.H * 4) + state_bytes(p, segs);
}

cudaError_t launch_linear_prefill(const LinearParams &p, bool bf16, cudaStream_t s) {
  using namespace lin;
  if (p.num_seqs == 0) return cudaSuccess;
  if (bf16) return launch_linear_prefill_tc(p, s);
  const int per = segment_chunks(p.N, p.num_seqs, p.H * (p.dv / kSlice), C), tokens = C * per;
  const size_t segs = max_segments(p.N, p.num_seqs, tokens);
  unsigned char *w = static_cast<unsigned char *>(p.ws);
  int *sbase = reinterpret_cast<int *>(w);
  float *whole = reinterpret_cast<float *>(w + table_bytes(p.num_seqs, segs));
  float *part = reinterpret_cast<float *>(w + table_bytes(p.num_seqs, segs) + align256(segs * p.H * 4));
  cudaError_t e = launch_linear_plan(p, sbase, tokens, 1, 1, 1, nullptr, nullptr, s);
  if (e != cudaSuccess) return e;
  e = launch_parts_chain(p, sbase, part, nullptr, whole, segs, s);
  if (e != cudaSuccess || p.N == 0) return e;
  return p.dk == 128 ? launch_rows<128>(p, sbase, part, segs, s) : launch_rows<64>(p, sbase, part, segs, s);
}

size_t linear_backward_workspace(const LinearParams &p, bool bf16) {
  using namespace lin;
  if (bf16) return linear_backward_tc_workspace(p);
  const size_t segs = max_segments(p.N, p.num_seqs, C);
  size_t n = table_bytes(p.num_seqs, segs) + align256(segs * p.H * 4) + 2 * state_bytes(p, segs);
  if (p.H != p.Hk) n += 2 * align256((size_t)p.N * p.H * p.dk * 4);
  if (p.decay_head) n += align256((size_t)p.N * p.H * 4);
  return n;
}

cudaError_t launch_linear_backward(const LinearParams &p, bool bf16, cudaStream_t s) {
  using namespace lin;
  if (p.num_seqs == 0) return p.decay_head ? cudaMemsetAsync(p.gla, 0, (size_t)p.H * 4, s) : cudaSuccess;
  const bool shared = p.H != p.Hk;
  float *gq32 = nullptr, *gk32 = nullptr, *gla = p.gla;      // per value head; per head and token
  const int *plan = static_cast<const int *>(p.ws);          // first in both workspaces
  cudaError_t e;
  if (bf16) {
    e = launch_linear_backward_tc(p, &gq32, &gk32, &gla, s);
    if (e != cudaSuccess) return e;
  } else {
    const size_t segs = max_segments(p.N, p.num_seqs, C);
    unsigned char *w = static_cast<unsigned char *>(p.ws);
    auto take = [&](size_t n) {
      unsigned char *at = w;
      w += align256(n);
      return reinterpret_cast<float *>(at);
    };
    int *sbase = reinterpret_cast<int *>(take(table_bytes(p.num_seqs, segs)));
    float *whole = take(segs * p.H * 4), *part = take(state_bytes(p, segs)), *rpart = take(state_bytes(p, segs));
    if (shared) {
      gq32 = take((size_t)p.N * p.H * p.dk * 4);
      gk32 = take((size_t)p.N * p.H * p.dk * 4);
    }
    if (p.decay_head) gla = take((size_t)p.N * p.H * 4);
    if ((e = launch_linear_plan(p, sbase, C, 1, 1, 1, nullptr, nullptr, s)) != cudaSuccess) return e;
    e = launch_parts_chain(p, sbase, part, rpart, whole, segs, s);
    if (e != cudaSuccess) return e;
    if (p.N > 0) e = launch_grad_dims(p, sbase, part, rpart, gq32, gk32, gla, segs, s);
    if (e != cudaSuccess) return e;
  }
  if (p.N > 0) {
    if (shared) {
      const size_t n = ((size_t)p.N * p.Hk * (p.dk / 4) + 255) / 256;
      if (n > 0x7FFFFFFFull) return cudaErrorInvalidValue;
      e = bf16 ? launch_next(share_kernel<true>, dim3((unsigned)n, 2), 256, 0, s, p, plan, gq32, gk32)
               : launch_next(share_kernel<false>, dim3((unsigned)n, 2), 256, 0, s, p, plan, gq32, gk32);
      if (e != cudaSuccess) return e;
    }
  }
  return p.decay_head ? launch_next(head_decay_kernel, (unsigned)p.H, 1024, 0, s, p, plan, gla) : cudaSuccess;
}

}  // namespace kda
