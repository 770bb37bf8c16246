// Attention of a few query rows per key head over the 4-bit cache.
//
//   o[i] = sum_t p[i, t] v~[t],  p[i, :] = softmax over the visible t of scale q[i] . k~[t]
//
// in one pass over the codes with a running maximum m and sum l per row:
//   m' = max(m, x),  l' = l 2^(m - m') + 2^(x - m'),  o' = o 2^(m - m') + 2^(x - m') v~.
//
// The rows that share a key head (its query heads times their tokens) are the
// N = 8 columns of m16n8k16 MMAs, so a key or value is decoded once for all of
// them:
//   S^T[16 tokens, 8 rows] = K~[16 tokens, D] . Q^T        A = decoded key codes
//   O^T[D, 8 rows]        += V~^T[D, 16 tokens] . P^T      A = decoded value codes
// S's accumulator fragment becomes P's operand fragment by one 8 x 8 transpose
// in registers (movmatrix) per eight tokens.
//
// Codes are not decoded where the sums can do it: a nibble's bits are the fp16
// subnormal q 2^-24 (or q 2^-20), which the tensor cores multiply exactly, so
//   sum_d Q_d (q_d - z) s = s (2^24 S - z sum_d Q_d)           (keys, per group of dims)
//   sum_t P_t s_t (q_t - z_t) = 2^20 O - sum_t P_t s_t z_t     (values, one scale per token)
// with the last sum one more MMA.  Values with several groups of dims per token
// enter as fp16((q - z) s), one rounding of 2^-11.  P (times the token's scale in
// the first form) is rounded to fp16 once, moved by powers of two to 2^15 .. 2^-24,
// so a long tail of small probabilities is not lost; S, m, l and O are fp32.
// Queries are moved to fp16 by a power of two per row (exact down to 2^-25 of the
// row's largest).
//
// Work split: a tile is one (sequence, key head, RT query rows); it has one step
// per kStepTok keys.  The steps of all tiles are divided evenly over the resident
// CTAs (their number comes from the lengths on the device, so a captured graph
// serves any lengths).  Inside a CTA each warp takes 32 tokens of a step through
// its own ring of cp.async stages (a CTA-wide ring would move its warps in
// lockstep); the warps' results meet in shared memory, while the first stages of
// the CTA's next tile are on their way.  A tile split between CTAs leaves fp32
// partials in the workspace, and the last CTA to arrive adds them in order.  No
// CTA waits for another.
//
// Bound: HBM by its bytes (132 a token and head for both of 128 dims), in fact the
// issue of a stage's instructions: 16 sequences of up to 32768 tokens, 64 query
// heads on 8, take 99 us (4.4 TB/s, 0.68 of the measured copy bandwidth; 104 us in
// seconds of calls at the power cap, 1.87 GHz); the copies alone 77 us, the arithmetic
// alone 93 us.  Of a stage's some 500 instructions the 34 MMAs, which overlap little
// with the logic pipe, cost a quarter.  With groups of 32 dims and zero-points (values
// decoded one by one) 32 sequences of up to 4096 tokens take 36 us (3.1 TB/s; these
// kernels of 128 dims spill up to 20 bytes, 60 with 16 rows, the others nothing).
// Decoding every code before its MMA took 130 us where this takes 99.
#include <algorithm>

#include "kv.cuh"

namespace qk {
namespace {

constexpr int kAtWarps = 4;
constexpr int kAtThreads = kAtWarps * 32;
constexpr int kStageTok = 32;                       // tokens per warp stage: two cache tiles
constexpr int kStepTok = kAtWarps * kStageTok;      // tokens per CTA step
constexpr float kLazy = 4.0f;                       // logits (base 2) may pass the reference by this
constexpr float kPShift = 15.0f - kLazy;            // P carries 2^kPShift, at most 2^15
constexpr int kFlush = 4;                           // stages between two flushes of O
constexpr int kAtMaxCtasPerSm = 3;                  // (4: 128 registers, spills, and no faster)

struct AtArgs {
  const uint16_t* q;
  const uint8_t* cache;
  const int* table;
  const int* lens;
  const int* cu_q;
  uint16_t* out;
  float* lse;
  float* slots;         // [2 * ctas][RT * (D + 2)]
  unsigned* counters;   // [ctas]: arrivals at the tile whose first contributor the CTA is
  long long q_stride, out_stride;
  int batch, total_q, max_q, heads, q_heads, per, page_log2, pages, max_pages;
  int rows_end;         // sequences with this many rows or more are the chunk kernel's
  float scale_log2;     // scale * log2(e)
  int window, split, bf16;
};

// Host and device agree on the rows per tile.
template <int D, int NT>
struct AtCfg {
  static constexpr int RT = 8 * NT;
  static constexpr int PART = RT * (D + 2);   // fp32 per partial: O, m, l
  static constexpr int CTAS = D == 256 || NT == 2 ? 2 : kAtMaxCtasPerSm;   // per SM, by registers
  static constexpr size_t RED = (size_t)kAtWarps * PART * sizeof(float);   // the warps' results
};

// Ring depth: three stages per warp where that many CTAs then fit an SM's shared
// memory beside the buffer of the warps' results (1 KB reserved each), else two.
template <int D, int MODE, int GD, int NT>
constexpr size_t at_smem(int stages) {
  return (size_t)kAtWarps * stages * 2 * kv_tile_bytes(D, D / GD, MODE) + AtCfg<D, NT>::RED;
}
template <int D, int MODE, int GD, int NT>
constexpr int at_stages() {
  return AtCfg<D, NT>::CTAS * (at_smem<D, MODE, GD, NT>(3) + 1024) <= 228 * 1024 ? 3 : 2;
}

// 64-bit division is a long software sequence; almost every one here fits 32 bits.
__device__ __forceinline__ long long div_pos(long long x, long long d) {
  if ((unsigned long long)(x | d) >> 32 == 0) return (long long)((unsigned)x / (unsigned)d);
  return x / d;
}

__device__ __forceinline__ void at_cp16(uint32_t saddr, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(saddr), "l"(src) : "memory");
}
__device__ __forceinline__ void at_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void at_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// D = A . B with a zero accumulator.
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// What a sequence asks for.
struct Seq {
  int len, q0, rows, tiles, steps;
  int base;        // position of its first query (of all it has, computed or not)
  int first, lo;   // first token any of its queries sees; the same down to a stage border
};

__device__ __forceinline__ Seq seq_of(const AtArgs& a, int b, int RT) {
  Seq s;
  const long long most = (long long)a.max_pages << a.page_log2;
  const int len = a.lens[b];
  s.len = len < 0 ? 0 : (len > most ? (int)most : len);
  int nq;
  if (a.cu_q) {
    const int e0 = a.cu_q[b], e1 = a.cu_q[b + 1];
    s.q0 = min(max(e0, 0), a.total_q);
    nq = min(min(max(e1, s.q0), a.total_q) - s.q0, a.max_q);
    s.base = s.len - min(max(e1, s.q0) - s.q0, 1 << 29);
  } else {
    s.q0 = b;
    nq = b < a.total_q ? 1 : 0;
    s.base = s.len - 1;
  }
  s.rows = nq * a.per;
  if (s.rows >= a.rows_end) s.rows = 0;
  s.tiles = (s.rows + RT - 1) / RT;
  s.first = a.window > 0 ? max(0, s.base - a.window + 1) : 0;
  s.lo = s.first & ~(kStageTok - 1);
  s.steps = max(1, (s.len - s.lo + kStepTok - 1) / kStepTok);
  return s;
}

template <int D, int MODE, int GD, int NT>
__global__ void __launch_bounds__(kAtThreads, AtCfg<D, NT>::CTAS)
    kv_attend_kernel(const AtArgs a) {
  constexpr int RT = AtCfg<D, NT>::RT;
  constexpr int G = D / GD;
  constexpr int PB = kv_param_bytes(MODE);
  constexpr int TB = kv_tile_bytes(D, G, MODE);
  constexpr int KROW = D / 2;                 // bytes of a code row
  constexpr int V_OFF = 16 * KROW, KP_OFF = 32 * KROW, VP_OFF = KP_OFF + 16 * G * PB;
  constexpr int KW = D / 32;                  // key words per lane and token: one per 32 dims
  constexpr int VW = D / 64;                  // value words per lane and token
  constexpr int MT = D / 16;                  // value MMA tiles
  constexpr int STAGE = 2 * TB;
  // one scale per token: it multiplies P, and value codes enter undecoded
  constexpr bool kFold = G == 1;
  // token at place k of the MMA's k order (and S's rows): see kv.cuh, the
  // rows read together must sit in different banks
  constexpr int SX = D == 64 ? 2 : 1;
  constexpr int kAtStages = at_stages<D, MODE, GD, NT>();

  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ long long s_scan[kAtWarps], s_scan1[kAtWarps];
  __shared__ long long s_first;
  __shared__ Seq s_seq;
  __shared__ int s_b;
  __shared__ int s_last;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  unsigned char* ring = smem + warp * (kAtStages * STAGE);
  const uint32_t ring_s = smem_u32(ring);

  pdl_wait();
  pdl_launch_dependents();

  // ---- steps of all sequences, this CTA's range of them, and the sequence it
  // starts in (a thread per sequence; more sequences than threads take turns)
  auto units_of = [&](const Seq& s) { return (long long)s.tiles * a.heads * s.steps; };
  Seq mine{};
  long long n_mine = 0, total = 0;
  for (int b = threadIdx.x; b < a.batch; b += kAtThreads) {
    const Seq s = seq_of(a, b, RT);
    if (b == (int)threadIdx.x) {
      mine = s;
      n_mine = units_of(s);
    }
    total += units_of(s);
  }
  // inclusive scan of the first turn within the warp, and the total
  long long inc = n_mine;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, inc, m);
    if (lane >= m) inc += o;
  }
#pragma unroll
  for (int m = 16; m; m >>= 1) total += __shfl_xor_sync(0xffffffffu, total, m);
  if (lane == 31) {
    s_scan[warp] = total;
    s_scan1[warp] = inc;
  }
  __syncthreads();
  total = 0;
  long long before = 0, first_turn = 0;
#pragma unroll
  for (int w = 0; w < kAtWarps; ++w) {
    total += s_scan[w];
    first_turn += s_scan1[w];
    if (w < warp) before += s_scan1[w];
  }
  if (total == 0) return;
  const long long U = total;
  const long long C = U < (long long)gridDim.x ? U : (long long)gridDim.x;   // CTAs with work
  const long long c = blockIdx.x;
  if (c >= C) return;
  long long u = div_pos(c * U, C), u_end = div_pos((c + 1) * U, C);
  {
    auto claim = [&](int b, const Seq& s, long long lo, long long n) {
      if (n > 0 && lo <= u && u < lo + n) {
        s_b = b;
        s_first = lo;
        s_seq = s;
      }
    };
    claim(threadIdx.x, mine, before + inc - n_mine, n_mine);
    long long base = first_turn;
    for (int b0 = kAtThreads; b0 < a.batch && base <= u; b0 += kAtThreads) {   // the same for every thread
      const int b = b0 + threadIdx.x;
      const Seq s = b < a.batch ? seq_of(a, b, RT) : Seq{};
      const long long n = b < a.batch ? units_of(s) : 0;
      long long sum = n;
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, sum, m);
        if (lane >= m) sum += o;
      }
      __syncthreads();
      if (lane == 31) s_scan[warp] = sum;
      __syncthreads();
      long long lo = base + sum - n;
#pragma unroll
      for (int w = 0; w < kAtWarps; ++w) {
        if (w < warp) lo += s_scan[w];
        base += s_scan[w];
      }
      claim(b, s, lo, n);
    }
    __syncthreads();
  }

  // a stretch of steps s0 .. s1 - 1 of one tile of rows
  struct Seg {
    Seq sq;
    long long first;   // unit at which the sequence starts
    int b, tile, head, rt, s0, s1;
  };
  Seg sg;
  sg.b = s_b;
  sg.first = s_first;
  sg.sq = s_seq;

  if (!a.split) {
    // whole tiles only: those that start inside the range
    auto up = [&](long long v) {
      // first tile start at or after v (v in or after the first sequence)
      int bb = sg.b;
      long long f = sg.first;
      Seq s = sg.sq;
      while (true) {
        const long long n = units_of(s);
        if (v < f + n || bb + 1 >= a.batch) break;
        f += n;
        s = seq_of(a, ++bb, RT);
      }
      const long long r = v - f - div_pos(v - f, s.steps) * s.steps;
      return r == 0 ? v : v + s.steps - r;
    };
    const long long ub = up(u), ue = u_end >= U ? U : up(u_end);
    u = ub;
    u_end = ue;
  }
  if (u >= u_end) return;

  auto locate = [&](Seg& s) {   // the stretch that starts at unit u, in s's sequence or after it
    while (u >= s.first + units_of(s.sq)) {
      s.first += units_of(s.sq);
      s.sq = seq_of(a, ++s.b, RT);
    }
    s.tile = (int)div_pos(u - s.first, s.sq.steps);
    s.s0 = (int)(u - s.first - (long long)s.tile * s.sq.steps);
    s.s1 = (int)min((long long)s.sq.steps, s.s0 + (u_end - u));
    s.rt = s.tile / a.heads;
    s.head = s.tile - s.rt * a.heads;
  };

  // ---- copies of this warp's 32 tokens of step s into ring stage st
  const int pm = (1 << a.page_log2) - 1;
  auto token0 = [&](const Seg& s, int step) { return s.sq.lo + (step * kAtWarps + warp) * kStageTok; };
  auto page_at = [&](const Seg& s, int tt) {
    const int id = a.table[(long long)s.b * a.max_pages + (tt >> a.page_log2)];
    return (unsigned)id < (unsigned)a.pages ? id : 0;   // no access outside the cache
  };
  // the page of a step's stage, looked up a step before the copy
  auto page_of_step = [&](const Seg& s, int step) {
    const int t0 = token0(s, step);
    return step < s.s1 && t0 < s.sq.len ? page_at(s, t0) : 0;
  };
  auto issue = [&](const Seg& s, int step, int st, int page) {
    const int t0 = token0(s, step);
    if (step >= s.s1 || t0 >= s.sq.len) return;   // warp-uniform, as below
    auto tile_src = [&](int id, int tt) {
      const long long tile = (((long long)id * a.heads + s.head) << (a.page_log2 - 4)) + ((tt & pm) >> 4);
      return a.cache + tile * TB + lane * 16;
    };
    const uint32_t dst = ring_s + st * STAGE + lane * 16;
    if (a.page_log2 > 4) {
      // the stage's two tiles lie in one page, one after the other
      const uint8_t* src = tile_src(page, t0);
#pragma unroll
      for (int i = 0; i < STAGE / 512; ++i) at_cp16(dst + i * 512, src + i * 512);
      if (STAGE % 512 != 0 && lane * 16 < STAGE % 512) at_cp16(dst + STAGE / 512 * 512, src + STAGE / 512 * 512);
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int tt = t0 + 16 * j;
        if (tt < s.sq.len) {
          const uint8_t* src = tile_src(j == 0 ? page : page_at(s, tt), tt);
#pragma unroll
          for (int i = 0; i < TB / 512; ++i) at_cp16(dst + j * TB + i * 512, src + i * 512);
          if (TB % 512 != 0 && lane * 16 < TB % 512) at_cp16(dst + j * TB + TB / 512 * 512, src + TB / 512 * 512);
        }
      }
    }
  };
  // a stretch's first stages: requested before the stretch before it is merged
  int next_page;
  auto begin = [&](const Seg& s) {
    int page[kAtStages];
#pragma unroll
    for (int i = 0; i < kAtStages; ++i) page[i] = page_of_step(s, s.s0 + i);
#pragma unroll
    for (int i = 0; i < kAtStages - 1; ++i) {
      issue(s, s.s0 + i, i, page[i]);
      at_commit();
    }
    next_page = page[kAtStages - 1];
  };

  locate(sg);
  begin(sg);
  bool first_seg = true;

  while (true) {
    const Seq& sq = sg.sq;
    const int head = sg.head, rt = sg.rt, s0 = sg.s0, s1 = sg.s1;

    // ---- this lane's query rows: column g of each token tile as operand,
    // columns 2t, 2t + 1 of the sums
    uint32_t qf[NT][2 * KW][2];
    float qa[NT][2];       // logit (base 2) per unit of the MMA's sum
    float qb[NT][G][2];    // logit per unit of zero-point: qa times the group's sum of q
    int hi_q[NT][2], lo_q[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = rt * RT + nt * 8 + g;
      const bool ok = row < sq.rows;
      const int qi = ok ? row / a.per : 0, hq = ok ? row - qi * a.per : 0;
      const uint16_t* src = a.q + (long long)(sq.q0 + qi) * a.q_stride + (head * a.per + hq) * D;
      uint4 v[KW];
#pragma unroll
      for (int w = 0; w < KW; ++w)
        v[w] = ok ? *reinterpret_cast<const uint4*>(src + 32 * w + 8 * t) : make_uint4(0, 0, 0, 0);
      uint32_t top = 0;   // largest magnitude bits of the row
#pragma unroll
      for (int w = 0; w < KW; ++w)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t x = (&v[w].x)[k];
          top = max(top, max(x & 0x7FFFu, (x >> 16) & 0x7FFFu));
        }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // times 2^(14 - e) for the largest's exponent e, held inside fp32's normals
      const int e = a.bf16 ? (int)(top >> 7) - 127 : (int)(top >> 10) - 15;
      const int k2 = min(max(14 - e, -126), 126);
      const float mul = __int_as_float((127 + k2) << 23), inv = __int_as_float((127 - k2) << 23);
      float sum[G];
#pragma unroll
      for (int gr = 0; gr < G; ++gr) sum[gr] = 0.0f;
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        float f[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t x = (&v[w].x)[k];
          if (a.bf16) {
            f[2 * k] = __uint_as_float(x << 16);
            f[2 * k + 1] = __uint_as_float(x & 0xFFFF0000u);
          } else {
            const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&x));
            f[2 * k] = h.x;
            f[2 * k + 1] = h.y;
          }
        }
        // dims (p, p + 4) of the word: the pairs the code words yield; the pairs
        // at p = 1, 3 meet codes that stand 16 times higher
#pragma unroll
        for (int p4 = 0; p4 < 4; ++p4) {
          const float m2 = (p4 & 1) ? mul * 0.0625f : mul;
          qf[nt][2 * w + (p4 >> 1)][p4 & 1] = pack2<false>(f[p4] * m2, f[p4 + 4] * m2);
          sum[w / (GD / 32)] += f[p4] * mul + f[p4 + 4] * mul;
        }
      }
#pragma unroll
      for (int gr = 0; gr < G; ++gr) {
        sum[gr] += __shfl_xor_sync(0xffffffffu, sum[gr], 1);
        sum[gr] += __shfl_xor_sync(0xffffffffu, sum[gr], 2);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int col = 2 * t + i;
        const float unit = a.scale_log2 * __shfl_sync(0xffffffffu, inv, 4 * col);
        qa[nt][i] = unit * 16777216.0f;
#pragma unroll
        for (int gr = 0; gr < G; ++gr) {
          qb[nt][gr][i] = unit * __shfl_sync(0xffffffffu, sum[gr], 4 * col);
          if constexpr (MODE == kSYM) qb[nt][gr][i] *= 8.0f;
        }
        const int r2 = rt * RT + nt * 8 + col;
        if (r2 < sq.rows) {
          const int pos = sq.base + r2 / a.per;
          hi_q[nt][i] = min(pos + 1, sq.len);
          lo_q[nt][i] = a.window > 0 ? pos - a.window + 1 : 0;
        } else {
          hi_q[nt][i] = lo_q[nt][i] = 0;
        }
      }
    }
    // tokens every row of the tile sees
    const int r_last = min(sq.rows, rt * RT + RT) - 1;
    const int full_hi = min(sq.len, sq.base + rt * RT / a.per + 1);
    const int full_lo = a.window > 0 ? sq.base + r_last / a.per - a.window + 1 : 0;

    float oacc[MT][NT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) oacc[i][nt][k] = 0.0f;
    float cacc[kFold ? NT : 1][4];   // sum of P (SYM) or P z (ASYM), the zero-points' share of O
#pragma unroll
    for (int nt = 0; nt < (kFold ? NT : 1); ++nt)
#pragma unroll
      for (int k = 0; k < 4; ++k) cacc[nt][k] = 0.0f;
    // moves the zero-points' share out of O: the tensor cores truncate their sums,
    // by up to 2^-24 of a sum of codes that are all positive, so left together O and
    // its share drift apart (32768 tokens on one warp chain: 4e-3 of a flat row's
    // output); taken off every kFlush stages the drift stays below 2^-12 of it
    auto flush = [&]() {
      if constexpr (kFold) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          // the codes stand for q 2^-20
          constexpr float kUnit = (MODE == kSYM ? 8.0f : 1.0f) * 9.5367431640625e-7f;
          const float z0 = cacc[nt][0] * kUnit, z1 = cacc[nt][1] * kUnit;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            oacc[mt][nt][0] -= z0;
            oacc[mt][nt][1] -= z1;
            oacc[mt][nt][2] -= z0;
            oacc[mt][nt][3] -= z1;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) cacc[nt][k] = 0.0f;
        }
      }
    };
    int vexp = 0;                    // exponent field of the largest value scale seen
    float mrow[NT][2], lrow[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mrow[nt][i] = -INFINITY;
        lrow[nt][i] = 0.0f;
      }

    // ---- 32 tokens from a stage; FULL: every row sees all of them
    const int tau0 = (g & 1) ? 4 + ((g >> 1) ^ SX) : (g >> 1);   // token of S's row g
    auto compute = [&]<bool FULL>(const unsigned char* stage, int t0) {
      // S^T = K~ Q^T: the codes are the bits of fp16 subnormals, q 2^-24 (q 2^-20
      // for every other pair); u = logit before its token's scale
      float u[2][NT][4], sk[2][2];
      uint32_t kw[2][2][KW];   // tile; rows g, g + 8
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const unsigned char* rp = stage + j * TB + (tau0 + 8 * h) * KROW;
          if constexpr (D == 64) {
            const uint2 v = *reinterpret_cast<const uint2*>(rp + 8 * t);
            kw[j][h][0] = v.x;
            kw[j][h][1] = v.y;
          } else {
#pragma unroll
            for (int i = 0; i < KW / 4; ++i) {
              const int piece = (t + 4 * i) ^ (D == 256 ? 4 * (tau0 & 1) : 0);
              const uint4 v = *reinterpret_cast<const uint4*>(rp + 16 * piece);
              kw[j][h][4 * i] = v.x;
              kw[j][h][4 * i + 1] = v.y;
              kw[j][h][4 * i + 2] = v.z;
              kw[j][h][4 * i + 3] = v.w;
            }
          }
        }
#pragma unroll
      for (int gr = 0; gr < G; ++gr) {
        float part[2][NT][4];
        // the two tiles' chains of MMAs in turn: each waits for its own last one only
#pragma unroll
        for (int w = gr * (GD / 32); w < (gr + 1) * (GD / 32); ++w) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t w0 = kw[j][0][w], w1 = kw[j][1][w];
              const uint32_t y0 = half ? w0 >> 8 : w0, y1 = half ? w1 >> 8 : w1;
              const uint32_t af[4] = {y0 & 0x000F000Fu, y1 & 0x000F000Fu, y0 & 0x00F000F0u, y1 & 0x00F000F0u};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                if (w == gr * (GD / 32) && half == 0) mma_first(part[j][nt], af, qf[nt][2 * w][0], qf[nt][2 * w][1]);
                else mma_16816<false>(part[j][nt], af, qf[nt][2 * w + half][0], qf[nt][2 * w + half][1]);
              }
            }
          }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float sc[2], z[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const unsigned char* pp = stage + j * TB + KP_OFF + ((tau0 + 8 * h) * G + gr) * PB;
            if constexpr (MODE == kASYM) {
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(pp));
              sc[h] = f.x;
              z[h] = f.y;
            } else {
              sc[h] = __half2float(*reinterpret_cast<const __half*>(pp));
              z[h] = 1.0f;   // qb holds 8 of it
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float v = MODE == kASYM ? fmaf(part[j][nt][i], qa[nt][i & 1], -z[i >> 1] * qb[nt][gr][i & 1])
                                            : fmaf(part[j][nt][i], qa[nt][i & 1], -qb[nt][gr][i & 1]);
              if constexpr (G == 1) u[j][nt][i] = v;
              else u[j][nt][i] = gr == 0 ? sc[i >> 1] * v : fmaf(sc[i >> 1], v, u[j][nt][i]);
            }
          if constexpr (G == 1) {
            sk[j][0] = sc[0];
            sk[j][1] = sc[1];
          } else {
            sk[j][0] = sk[j][1] = 1.0f;
          }
        }
      }

      // this lane's value scales at S's rows (one scale per token): the exponent
      // of the warp's largest keeps P times scale at the top of fp16's range
      [[maybe_unused]] float sv[2][2];
      if constexpr (kFold) {
        uint32_t bits[2][2], top = 0;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            bits[j][h] = *reinterpret_cast<const uint16_t*>(stage + j * TB + VP_OFF + (tau0 + 8 * h) * PB);
            if constexpr (!FULL) {
              // what lies past the sequence or before its window may be anything,
              // and 0 times a NaN found there is a NaN: its scale reads as 0
              const int pos = t0 + 16 * j + 8 * h + tau0;
              if (pos >= sq.len || pos < sq.first) bits[j][h] = 0;
            }
            top = max(top, bits[j][h]);
          }
        const int e = (int)(__reduce_max_sync(0xffffffffu, top) >> 10);
        if (e > vexp) {
          const float f = __int_as_float((127 + max(vexp - e, -126)) << 23);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int k = 0; k < 4; ++k) cacc[nt][k] *= f;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int k = 0; k < 4; ++k) oacc[mt][nt][k] *= f;
          }
          vexp = e;
        }
        const float f = __int_as_float((127 + 14 - vexp) << 23);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) sv[j][h] = __half2float(__ushort_as_half((unsigned short)bits[j][h])) * f;
      }

      // ---- running softmax: the reference m moves only when a logit exceeds it
      // by 2^kLazy, so most stages need no maximum across lanes
      uint32_t pf[2][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float y[2][4], most = -INFINITY;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float v = G == 1 ? fmaf(u[j][nt][i], sk[j][i >> 1], -mrow[nt][i & 1]) : u[j][nt][i] - mrow[nt][i & 1];
            if constexpr (!FULL) {
              const int tok = t0 + 16 * j + 8 * (i >> 1) + tau0;
              if (tok >= hi_q[nt][i & 1] || tok < lo_q[nt][i & 1]) v = -INFINITY;
            }
            y[j][i] = v;
            most = fmaxf(most, v);
          }
        if (__any_sync(0xffffffffu, most > kLazy)) {
#pragma unroll
          for (int c2 = 0; c2 < 2; ++c2) {
            float mx = mrow[nt][c2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int i = 2 * h + c2;
                float v = G == 1 ? u[j][nt][i] * sk[j][h] : u[j][nt][i];
                if constexpr (!FULL) {
                  const int tok = t0 + 16 * j + 8 * h + tau0;
                  if (tok >= hi_q[nt][c2] || tok < lo_q[nt][c2]) v = -INFINITY;
                }
                y[j][i] = v;
                mx = fmaxf(mx, v);
              }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float ref = mx == -INFINITY ? 0.0f : mx;   // nothing seen yet
            const float alpha = exp2_fast(mrow[nt][c2] - ref);
            mrow[nt][c2] = mx;
            lrow[nt][c2] *= alpha;
            if constexpr (kFold) {
              cacc[nt][c2] *= alpha;
              cacc[nt][2 + c2] *= alpha;
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              oacc[mt][nt][c2] *= alpha;
              oacc[mt][nt][2 + c2] *= alpha;
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int h = 0; h < 2; ++h) y[j][2 * h + c2] -= ref;
          }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float p0 = exp2_fast(y[j][2 * h] + kPShift), p1 = exp2_fast(y[j][2 * h + 1] + kPShift);
            lrow[nt][0] += p0;
            lrow[nt][1] += p1;
            if constexpr (kFold) {
              p0 *= sv[j][h];
              p1 *= sv[j][h];
            }
            pf[j][nt][h] = transpose8x8(pack2<false>(p0, p1));
          }
      }

      // ---- O^T += V~^T P^T
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const unsigned char* tp = stage + j * TB;
        const int tok[4] = {t, 4 + (t ^ SX), 8 + t, 12 + (t ^ SX)};
        uint32_t vw[4][VW];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const unsigned char* rp = tp + V_OFF + tok[k] * KROW + (D / 16) * kv_val_piece(D, g, tok[k]);
          if constexpr (D == 64) {
            vw[k][0] = *reinterpret_cast<const uint32_t*>(rp);
          } else if constexpr (D == 128) {
            const uint2 v = *reinterpret_cast<const uint2*>(rp);
            vw[k][0] = v.x;
            vw[k][1] = v.y;
          } else {
            const uint4 v = *reinterpret_cast<const uint4*>(rp);
            vw[k][0] = v.x;
            vw[k][1] = v.y;
            vw[k][2] = v.z;
            vw[k][3] = v.w;
          }
        }
        uint32_t par[4] = {0, 0, 0, 0};
        if constexpr (!kFold || MODE == kASYM) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const unsigned char* pp = tp + VP_OFF + (tok[k] * G + g * (D / 8) / GD) * PB;
            if constexpr (MODE == kASYM) par[k] = *reinterpret_cast<const uint32_t*>(pp);
            else par[k] = *reinterpret_cast<const uint16_t*>(pp);
            if constexpr (!FULL) {
              const int pos = t0 + 16 * j + tok[k];
              if (pos >= sq.len || pos < sq.first) par[k] = 0;
            }
          }
        }
        if constexpr (kFold) {
          // the zero-points' share: sum over tokens of P (times z), in every row
          uint32_t zf[4];
          if constexpr (MODE == kASYM) {
            zf[0] = zf[1] = __byte_perm(par[0], par[1], 0x7632);
            zf[2] = zf[3] = __byte_perm(par[2], par[3], 0x7632);
          } else {
            zf[0] = zf[1] = zf[2] = zf[3] = 0x3C003C00u;
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_16816<false>(cacc[nt], zf, pf[j][nt][0], pf[j][nt][1]);
#pragma unroll
          for (int w = 0; w < VW; ++w) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {   // dims 4 half .. 4 half + 3 of the word
              const uint32_t ab = __byte_perm(vw[0][w], vw[1][w], half ? 0x7632 : 0x5410);
              const uint32_t cd = __byte_perm(vw[2][w], vw[3][w], half ? 0x7632 : 0x5410);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                // all at q 2^-20, 6 bits below the operand's exponent: what the MMA
                // cuts off the smaller of its products stays below 2^-18 of the largest
                const uint32_t ye = e ? ab >> 8 : ab, yf = e ? cd >> 8 : cd;
                const uint32_t af[4] = {(ye * 16u) & 0x00F000F0u, ye & 0x00F000F0u, (yf * 16u) & 0x00F000F0u,
                                        yf & 0x00F000F0u};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma_16816<false>(oacc[4 * w + 2 * half + e][nt], af, pf[j][nt][0], pf[j][nt][1]);
              }
            }
          }
        } else {
          uint32_t sv2[2], bias[2] = {0x64086408u, 0x64086408u}, bias16[2] = {0xD480D480u, 0xD480D480u};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            sv2[h] = __byte_perm(par[2 * h], par[2 * h + 1], 0x5410);
            if constexpr (MODE == kASYM)
              zero_biases(__byte_perm(par[2 * h], par[2 * h + 1], 0x7632), bias[h], bias16[h]);
          }
#pragma unroll
          for (int w = 0; w < VW; ++w) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint32_t d[2][4];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t u2 = __byte_perm(vw[2 * h][w], vw[2 * h + 1][w], half ? 0x7632 : 0x5410);
                decode_nibbles(u2, bias[h], bias16[h], d[h]);
#pragma unroll
                for (int k = 0; k < 4; ++k) d[h][k] = hmul2_u16(d[h][k], sv2[h]);
              }
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint32_t af[4] = {d[0][2 * e], d[0][2 * e + 1], d[1][2 * e], d[1][2 * e + 1]};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma_16816<false>(oacc[4 * w + 2 * half + e][nt], af, pf[j][nt][0], pf[j][nt][1]);
              }
            }
          }
        }
      }
    };

    int st_c = 0, st_f = kAtStages - 1;
    for (int s = s0; s < s1; ++s) {
      issue(sg, s + kAtStages - 1, st_f, next_page);
      next_page = page_of_step(sg, s + kAtStages);
      at_commit();
      at_wait<kAtStages - 1>();
      __syncwarp();
      const int t0 = token0(sg, s);
      if (t0 < sq.len) {   // warp-uniform
        const unsigned char* stage = ring + st_c * STAGE;
        if (t0 + kStageTok <= full_hi && t0 >= full_lo) compute.template operator()<true>(stage, t0);
        else compute.template operator()<false>(stage, t0);
      }
      if ((s - s0) % kFlush == kFlush - 1) flush();
      __syncwarp();   // every lane is done with the stage before it is refilled
      st_c = st_c + 1 == kAtStages ? 0 : st_c + 1;
      st_f = st_f + 1 == kAtStages ? 0 : st_f + 1;
    }
    at_wait<0>();
    flush();

    // ---- the next stretch's first stages are on their way while this one ends
    u += s1 - s0;
    const bool more = u < u_end;
    Seg next = sg;
    if (more) {
      locate(next);
      begin(next);
    }

    // ---- the warps' results through shared memory
    float* wm = reinterpret_cast<float*>(smem + kAtWarps * kAtStages * STAGE);   // [warps][RT]
    float* wl = wm + kAtWarps * RT;                         // [warps][RT]
    float* wo = wl + kAtWarps * RT;                         // [warps][RT][D]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float l = lrow[nt][i];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        const int row = nt * 8 + 2 * t + i;
        if (g == 0) {
          wm[warp * RT + row] = mrow[nt][i];
          wl[warp * RT + row] = l;
        }
        float* dst = wo + (warp * RT + row) * D + g * (D / 8);
        // P carried 2^(14 - vexp) of the value scales
        const float f = kFold ? __int_as_float((127 + vexp - 14 + 20) << 23) : 1.0f;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
          *reinterpret_cast<float2*>(dst + 2 * mt) = make_float2(oacc[mt][nt][i] * f, oacc[mt][nt][2 + i] * f);
      }
    __syncthreads();

    const bool whole = s0 == 0 && s1 == sq.steps;
    const int rows_here = min(RT, sq.rows - rt * RT);
    auto emit = [&](int row, int d4, const float4& o, float m, float l) {
      // four dims of a row: o / l (0 for a row that sees nothing)
      const int r2 = rt * RT + row, qi = r2 / a.per, hq = head * a.per + r2 - qi * a.per;
      const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
      uint2 v;
      if (a.bf16) {
        v.x = pack2<true>(o.x * inv, o.y * inv);
        v.y = pack2<true>(o.z * inv, o.w * inv);
      } else {
        v.x = pack2<false>(o.x * inv, o.y * inv);
        v.y = pack2<false>(o.z * inv, o.w * inv);
      }
      *reinterpret_cast<uint2*>(a.out + (long long)(sq.q0 + qi) * a.out_stride + hq * D + d4) = v;
      if (d4 == 0 && a.lse)
        a.lse[(long long)(sq.q0 + qi) * a.q_heads + hq] =
            l == 0.0f ? -INFINITY : 0.69314718056f * (m + log2f(l) - kPShift);
    };
    float* slot = a.slots + (2 * c + (first_seg ? 0 : 1)) * (long long)AtCfg<D, NT>::PART;
    for (int i = threadIdx.x; i < rows_here * (D / 4); i += kAtThreads) {
      const int row = i / (D / 4), d4 = (i % (D / 4)) * 4;
      float m = -INFINITY;
#pragma unroll
      for (int w = 0; w < kAtWarps; ++w) m = fmaxf(m, wm[w * RT + row]);
      const float ref = m == -INFINITY ? 0.0f : m;
      float l = 0.0f;
      float4 o = make_float4(0, 0, 0, 0);
#pragma unroll
      for (int w = 0; w < kAtWarps; ++w) {
        const float f = exp2_fast(wm[w * RT + row] - ref);
        const float4 v = *reinterpret_cast<const float4*>(wo + (w * RT + row) * D + d4);
        l = fmaf(f, wl[w * RT + row], l);
        o.x = fmaf(f, v.x, o.x);
        o.y = fmaf(f, v.y, o.y);
        o.z = fmaf(f, v.z, o.z);
        o.w = fmaf(f, v.w, o.w);
      }
      if (whole) {
        emit(row, d4, o, m, l);
      } else {
        *reinterpret_cast<float4*>(slot + row * D + d4) = o;
        if (d4 == 0) {
          slot[RT * D + row] = m;
          slot[RT * D + RT + row] = l;
        }
      }
    }
    if (!whole) {
      __syncthreads();
      const long long t_first = sg.first + (long long)sg.tile * sq.steps;
      const long long first = div_pos((t_first + 1) * C - 1, U);
      const long long nb = div_pos((t_first + sq.steps) * C - 1, U) - first + 1;
      unsigned* counter = a.counters + first;   // at most one split tile starts in a CTA's range
      if (threadIdx.x == 0) {
        unsigned prev;
        asm volatile("atom.add.acq_rel.gpu.u32 %0, [%1], 1;" : "=r"(prev) : "l"(counter) : "memory");
        s_last = prev == (unsigned)(nb - 1);
      }
      __syncthreads();
      if (s_last) {
        // `first` left its partial in its second slot if its range began before the tile
        const int first_e = first * U < t_first * C ? 1 : 0;   // floor(first U / C) < t_first
        for (int i = threadIdx.x; i < rows_here * (D / 4); i += kAtThreads) {
          const int row = i / (D / 4), d4 = (i % (D / 4)) * 4;
          float m = -INFINITY, l = 0.0f;
          float4 o = make_float4(0, 0, 0, 0);
          for (long long k = 0; k < nb; ++k) {
            const float* p = a.slots + (2 * (first + k) + (k == 0 ? first_e : 0)) * (long long)AtCfg<D, NT>::PART;
            const float mk = __ldcg(p + RT * D + row), lk = __ldcg(p + RT * D + RT + row);
            const float4 v = __ldcg(reinterpret_cast<const float4*>(p + row * D + d4));
            const float mn = fmaxf(m, mk);
            const float ref = mn == -INFINITY ? 0.0f : mn;
            const float fa = exp2_fast(m - ref), fb = exp2_fast(mk - ref);
            m = mn;
            l = l * fa + lk * fb;
            o.x = o.x * fa + v.x * fb;
            o.y = o.y * fa + v.y * fb;
            o.z = o.z * fa + v.z * fb;
            o.w = o.w * fa + v.w * fb;
          }
          emit(row, d4, o, m, l);
        }
        if (threadIdx.x == 0) *counter = 0u;   // ready for the next call
      }
    }
    if (!more) break;
    __syncthreads();   // the results' buffer is used again
    first_seg = false;
    sg = next;
  }
}

template <int D, int MODE, int GD, int NT>
cudaError_t at_launch(const AtArgs& args, long long most, cudaStream_t stream) {
  auto k = kv_attend_kernel<D, MODE, GD, NT>;
  constexpr size_t smem = at_smem<D, MODE, GD, NT>(at_stages<D, MODE, GD, NT>());
  static_assert(smem <= 227 * 1024, "shared memory of the attention kernel");
  static int occ[64] = {};   // resident CTAs per SM, once per device
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!occ[dev]) {
    int o = 0;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&o, k, kAtThreads, smem);
    if (e == cudaSuccess && o < 1) e = cudaErrorInvalidConfiguration;
    if (e != cudaSuccess) {
      cudaGetLastError();
      return e;
    }
    occ[dev] = o;
  }
  const int ctas = (int)std::min<long long>(
      std::min((long long)occ[dev], (long long)kAtMaxCtasPerSm) * device_sms(), most);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(kAtThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k, args);
  if (e != cudaSuccess) cudaGetLastError();   // report it once, here
  return e;
}

// Sequences with at least this many query rows per key head go to the tensor-core
// kernel, which pays for tiles of 128 rows whatever they hold and splits a tile's
// tokens only as far as SMs are left.  Measured (us, this kernel : that one, 64
// query heads on 8 key heads, SYM, one scale per row):
//   sequences x tokens, dim        64 rows    96 rows    128 rows
//   1 x 32768, 128                 59 : 76    76 : 76    95 : 77
//   8 x 4096, 128                  44 : 53    57 : 53    85 : 54
//   8 x 32768, 128                213 : 307  277 : 303  410 : 304
//   64 x 2048, 128                163 : 131  234 : 145  288 : 141
//   8 x 4096, 64                   33 : 42    42 : 43    61 : 43
//   8 x 4096, 256                  75 : 73   112 : 74   174 : 80
int chunk_rows(int batch, int kv_heads, int dim, int sms) {
  return dim == 256 || (long long)batch * kv_heads >= sms ? 64 : 96;
}

// Query rows per tile: 8 for a key head with up to 8 rows (and for 256 dims,
// whose sums need the registers), else 16.
int at_rows(long long most_rows, int dim) { return most_rows <= 8 || dim == 256 ? 8 : 16; }

struct AtPlan {
  int rows, tiles_max, ctas;
  int chunk_rows;
  bool chunk;       // a sequence may have that many rows
  size_t slots;
};

// The workspace: arrival counters of this kernel's CTAs and of the chunk kernel's
// tiles in a head of the same size for every shape (so that calls of different
// shapes can share a workspace: they leave it zero), then partial results, which
// the two kernels use one after the other.
size_t at_counters(int sms) { return (size_t)sms * kAtMaxCtasPerSm * sizeof(unsigned); }
size_t at_head(int sms) { return (at_counters(sms) + (size_t)sms * sizeof(unsigned) + 255) / 256 * 256; }

AtPlan at_plan(int batch, int max_q, int q_heads, int kv_heads, int dim, int sms) {
  AtPlan p{};
  const int per = q_heads / kv_heads;
  p.chunk_rows = chunk_rows(batch, kv_heads, dim, sms);
  p.chunk = (long long)max_q * per >= p.chunk_rows;
  const long long most_rows = std::min<long long>((long long)max_q * per, p.chunk_rows - 1);
  p.rows = at_rows(most_rows, dim);
  p.tiles_max = (int)((most_rows + p.rows - 1) / p.rows);
  p.ctas = sms * kAtMaxCtasPerSm;
  p.slots = (size_t)2 * p.ctas * p.rows * (dim + 2) * sizeof(float);
  return p;
}

}  // namespace

size_t kv_attend_workspace(int batch, int max_q, int q_heads, int kv_heads, int dim, int sms) {
  const AtPlan p = at_plan(batch, max_q, q_heads, kv_heads, dim, sms);
  const size_t chunk = p.chunk ? kv_chunk_slots(batch, max_q, q_heads, kv_heads, dim, sms) : 0;
  return at_head(sms) + std::max(p.slots, chunk);
}

cudaError_t launch_kv_attend(const KvAttend& p, void* workspace, long long wait_limit, cudaStream_t stream) {
  const KvCache& c = p.cache;
  const int sms = device_sms();
  const AtPlan plan = at_plan(p.batch, p.max_q, p.q_heads, c.heads, c.dim, sms);
  unsigned* counters = static_cast<unsigned*>(workspace);
  float* slots = workspace ? reinterpret_cast<float*>(static_cast<char*>(workspace) + at_head(sms)) : nullptr;
  if (plan.chunk) {
    unsigned* tiles = workspace ? counters + at_counters(sms) / sizeof(unsigned) : nullptr;
    const cudaError_t e = launch_kv_chunk(p, plan.chunk_rows, tiles, slots, wait_limit, stream);
    if (e != cudaSuccess) return e;
  }
  AtArgs a{};
  a.q = static_cast<const uint16_t*>(p.q);
  a.cache = static_cast<const uint8_t*>(c.data);
  a.table = p.table;
  a.lens = p.lens;
  a.cu_q = p.cu_q;
  a.out = static_cast<uint16_t*>(p.out);
  a.lse = p.lse;
  a.q_stride = p.q_stride;
  a.out_stride = p.out_stride;
  a.batch = p.batch;
  a.total_q = p.total_q;
  a.max_q = p.max_q;
  a.heads = c.heads;
  a.q_heads = p.q_heads;
  a.per = p.q_heads / c.heads;
  a.page_log2 = c.page_log2;
  a.pages = c.pages;
  a.max_pages = p.max_pages;
  a.rows_end = plan.chunk_rows;
  a.scale_log2 = p.scale * 1.4426950408889634f;
  a.window = p.window;
  a.bf16 = p.bf16;
  if (workspace) {
    a.split = 1;
    a.counters = counters;
    a.slots = slots;
  }
  // no more CTAs than steps the table could hold
  const long long steps = std::max<long long>(1, (((long long)p.max_pages << c.page_log2) + kStepTok - 1) / kStepTok);
  const long long most = (long long)p.batch * c.heads * plan.tiles_max * steps;
  const int gd = c.dim / c.G;
#define AT_CASE(D, MO, GD, NT) \
  if (c.dim == D && c.mode == MO && gd == GD && plan.rows == 8 * NT) return at_launch<D, MO, GD, NT>(a, most, stream);
#define AT_MODES(D, GD, NT) AT_CASE(D, kSYM, GD, NT) AT_CASE(D, kASYM, GD, NT)
  AT_MODES(64, 32, 1) AT_MODES(64, 64, 1) AT_MODES(64, 32, 2) AT_MODES(64, 64, 2)
  AT_MODES(128, 32, 1) AT_MODES(128, 64, 1) AT_MODES(128, 128, 1)
  AT_MODES(128, 32, 2) AT_MODES(128, 64, 2) AT_MODES(128, 128, 2)
  AT_MODES(256, 32, 1) AT_MODES(256, 64, 1) AT_MODES(256, 128, 1) AT_MODES(256, 256, 1)
#undef AT_MODES
#undef AT_CASE
  return cudaErrorInvalidValue;
}

}  // namespace qk
