// Attention of many query rows per key head over the 4-bit cache (a chunk of a
// prompt behind its prefix): the same sums as kvattend.cu on the 5th-generation
// tensor cores.
//
//   S[128 rows, 128 tokens] = Q . K~^T        A = Q (shared memory), B = K~
//   O[128 rows, D]         += P . V~          A = P (TMEM),          B = V~^T
//
// A row is a query head of a token; a CTA holds NR tiles of 128 rows of one key
// head (two, so that one's softmax runs under the other's MMAs) and walks over
// the visible tokens in tiles of 128.  Bound by the tensor pipe and, as much, by
// the exponentials (16 a cycle and SM: one 128 x 128 tile takes 1024 cycles of
// either).  Warp roles:
//   4 per row tile   softmax: a thread owns a row (its maximum, sum and scale
//                    need no shuffles); S from TMEM, P back into S's columns
//   4                decode: codes from global memory straight to registers, then
//                    K~ = fp16((q - z) s) and V~^T into shared memory (128-byte
//                    swizzle); both row tiles use a decoded tile
//   1                MMA issuer and TMEM owner
// Rounding: K~, V~ and P once each to fp16 (P carries 2^kPShift, so its small
// values keep their bits); S, O, the maximum and the sum are fp32.  The maximum
// is a lazy reference: O is rescaled only when a row passes it by 2^kLazy, by the
// softmax warps themselves, between two MMAs on it.
// Few tiles of rows on long sequences: a tile's tokens are split between CTAs (at
// least kSplitTiles tiles of tokens each); each leaves O, m and l in the workspace
// and the last to arrive adds them in order.
//
// Measured: chunks of 2048 queries x 32 heads on 8 behind prefixes up to 6000
// tokens, 128 dims, take 285 us (826 TFLOP/s, 0.51 of the measured burst rate; 299 us
// in seconds of calls at the power cap, 1.88 GHz); the MMAs alone, unhindered, 165.
// The same with 64 dims 249 us; with 256, one row tile and one stage of keys and
// values, where nothing hides the softmax, 686 (0.42 of the rate).  No spills with one
// scale per row; up to 100 bytes with 256 dims in groups of 32.  A tile of 128 tokens
// takes some 4300 cycles against 2048 of MMAs: S, softmax (2600 cycles, its two groups
// sharing the special function units and issue slots with the decoder) and P V are one
// chain per row tile.  Two S buffers of 64 tokens instead (an MMA of 64 columns takes
// as long as one of 128) 341 us; halves of P handed on early, exponentials on the FMA
// pipes, one pass over S instead of two: no faster; two warps to a row's 128 tokens (16
// softmax warps) 313 us.  Against 64 bits the output is off by 4.4e-4 (2-norm; rounding
// it to fp16 alone 2.1e-4), 2.9e-4 of it K~'s; exact integers as K~ with the keys'
// scales multiplied onto S leave 3.4e-4 and take 328 us.
//
// Every wait is bounded: one that runs out sets the error word and the CTA drains
// its MMAs, frees TMEM and exits.
#include <algorithm>

#include "kv.cuh"

namespace qk {
namespace {

__device__ unsigned g_kv_error = 0;

constexpr int kTok = 128;             // tokens per tile
constexpr int kDecW = 4;              // decode warps
constexpr int kSplitTiles = 8;        // tiles of tokens that are worth a CTA of their own
constexpr int kSplitMost = 16;        // partials the last CTA adds up
constexpr float kLazy = 8.0f;         // logits (base 2) may pass the reference by this
constexpr float kPShift = 15.0f - kLazy;
constexpr long long kDrain = 4000000000ll;   // own MMAs while draining: ~2 s

struct ChArgs {
  const uint16_t* q;
  const uint8_t* cache;
  const int* table;
  const int* lens;
  const int* cu_q;
  uint16_t* out;
  float* lse;
  long long q_stride, out_stride, wait_limit;
  int batch, total_q, max_q, heads, q_heads, per, page_log2, pages, max_pages, tiles_max, min_rows;
  float scale_log2;
  int window, bf16;
  int splits;           // CTAs per tile of rows
  float* slots;         // [tiles][splits][D + 2][128 NR]: O, m, l of a part
  unsigned* counters;   // [tiles]
};

// NR row tiles of 128 and ST stages of K~ and V~ in 227 KB and 512 TMEM columns.
template <int D>
struct ChCfg {
  static constexpr int NR = D == 256 ? 1 : 2;
  static constexpr int ST = D == 256 ? 1 : 2;
  static constexpr int Q_BYTES = 128 * D * 2;
  static constexpr int K_BYTES = kTok * D * 2;
  static constexpr int SOFT = 4 * NR;                       // softmax warps
  static constexpr int THREADS = 32 * (SOFT + kDecW + 4);    // whole warpgroups, for the register split
  // registers per thread: softmax holds a row of 128 S, decode a tile's codes; one
  // warp of each group per SM quarter, within what the launch holds (4 x 128 or 3 x 168)
  static constexpr int R_SOFT = NR == 2 ? 184 : 208;
  static constexpr int R_DEC = NR == 2 ? 96 : 208;
  static constexpr int R_MMA = 48;
  static_assert(NR * R_SOFT + R_DEC + R_MMA <= (NR == 2 ? 512 : 504), "register split");
  static constexpr size_t SMEM = 1024 + (size_t)NR * Q_BYTES + (size_t)ST * 2 * K_BYTES + 256;
  static constexpr int ROWS = 128 * NR;
  static constexpr int PART = ROWS * (D + 2);               // fp32 per partial
  static constexpr int O_COL = 128 * NR;                    // TMEM: S (and P) per row tile, then O
};

// Bounded wait for phase `parity` of `bar`: false (and the CTA's abort flag and the
// error word raised) once `limit` clock cycles pass, or when another thread of the
// CTA has given up.  The clock is read before each try, which may suspend the
// thread for a while.
__device__ __forceinline__ bool ch_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool ch_wait(uint64_t* bar, uint32_t parity, volatile int* abort, long long limit) {
  if (ch_test(bar, parity)) return true;
  const long long t0 = clock64();
  while (true) {
    if (ch_test(bar, parity)) return true;
    if (*abort) return false;
    if (clock64() - t0 > limit) {
      *abort = 1;
      atomicOr(&g_kv_error, 1u);
      return false;
    }
    if (mbar_try(bar, parity)) return true;
  }
}

// Shared-memory matrix descriptor (K-major, 128-byte swizzle, 8-row groups 1024
// bytes apart): the low word holds the address in units of 16 bytes, the high one
// is the same for every tile.
__device__ __forceinline__ uint32_t ch_desc(uint32_t saddr) { return ((saddr >> 4) & 0x3FFF) | (1u << 16); }
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
// Keeps a loop's descriptors from being computed ahead of it, all at once, in
// registers that the MMA warp does not have.
__device__ __forceinline__ uint32_t opaque(uint32_t x) {
  asm volatile("" : "+r"(x));
  return x;
}
// The MMA warp runs its loop as a whole warp, so that descriptors and addresses
// stay in uniform registers (built by one thread they cost some 200 cycles an
// MMA), and one elected lane (`lead`) issues.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
__device__ __forceinline__ void ch_mma(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "mov.b64 da, {%1, %6};\n\tmov.b64 db, {%2, %6};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(lead), "r"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void ch_mma_ta(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "mov.b64 db, {%2, %6};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(lead), "r"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void ch_commit(uint64_t* bar, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(lead)
      : "memory");
}
// Barrier of some warps whose result is the AND of their threads' predicates.
__device__ __forceinline__ bool bar_and(int id, int threads, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.red.and.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)pred), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void ch_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void ch_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 columns of this warp's lanes, not waited for: wait32 before the values are used.
__device__ __forceinline__ void ld32_async(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr));
}
__device__ __forceinline__ void wait32(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])::"memory");
}
__device__ __forceinline__ void st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t r, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float ch_exp2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

template <int D, int MODE, int GD>
__global__ void __launch_bounds__(ChCfg<D>::THREADS, 1) kv_chunk_kernel(const ChArgs a) {
  using Cfg = ChCfg<D>;
  constexpr int NR = Cfg::NR, ST = Cfg::ST;
  constexpr int G = D / GD;
  constexpr int PB = kv_param_bytes(MODE);
  constexpr int TB = kv_tile_bytes(D, G, MODE);
  constexpr int KROW = D / 2;
  constexpr int V_OFF = 16 * KROW, KP_OFF = 32 * KROW, VP_OFF = KP_OFF + 16 * G * PB;
  constexpr int PANEL = 128 * 128;      // 128 rows of one 128-byte swizzle span
  constexpr int VPANEL = D * 128;       // V~^T: D rows of 64 tokens

  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  unsigned char* sQ = base;
  unsigned char* sK = sQ + NR * Cfg::Q_BYTES;
  unsigned char* sV = sK + ST * Cfg::K_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sV + ST * Cfg::K_BYTES);
  uint64_t* k_full = bars;            // [2] decode -> MMA
  uint64_t* k_empty = bars + 2;       // [2] MMA -> decode
  uint64_t* v_full = bars + 4;        // [2]
  uint64_t* v_empty = bars + 6;       // [2]
  uint64_t* s_full = bars + 8;        // [2] MMA -> softmax of row tile r
  uint64_t* p_full = bars + 10;       // [2] softmax -> MMA
  uint64_t* pv_done = bars + 12;      // [2] MMA on O of row tile r finished
  uint64_t* q_full = bars + 14;
  uint64_t* drain = bars + 15;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 16);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* last_flag = abort_flag + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], kDecW);
      mbar_init(&v_full[i], kDecW);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(q_full, Cfg::SOFT);
    mbar_init(drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();
  pdl_launch_dependents();

  // ---- this CTA's tile of rows: the last rows (which see most) first
  const int pairs = a.batch * a.heads;
  const int item = (int)blockIdx.x / a.splits, part = (int)blockIdx.x - item * a.splits;
  const int rt = a.tiles_max - 1 - item / pairs;
  const int pr = item % pairs;
  const int b = pr / a.heads, head = pr - b * a.heads;
  const long long most = (long long)a.max_pages << a.page_log2;
  int len = a.lens[b];
  len = len < 0 ? 0 : (len > most ? (int)most : len);
  int q0, nq, base_pos;   // base_pos: position of the first of all its queries, computed or not
  if (a.cu_q) {
    const int e0 = a.cu_q[b], e1 = a.cu_q[b + 1];
    q0 = min(max(e0, 0), a.total_q);
    nq = min(min(max(e1, q0), a.total_q) - q0, a.max_q);
    base_pos = len - min(max(e1, q0) - q0, 1 << 29);
  } else {
    q0 = b;
    nq = b < a.total_q ? 1 : 0;
    base_pos = len - 1;
  }
  const int rows = nq * a.per;
  if (rows < a.min_rows || rt * 128 * NR >= rows) return;   // another kernel's, or none (no TMEM taken yet)
  const int row0 = rt * 128 * NR, row_end = min(rows, row0 + 128 * NR);
  // tokens any / every row of the CTA sees
  const int first_seq = a.window > 0 ? max(0, base_pos - a.window + 1) : 0;
  const int hi_any = min(len, base_pos + (row_end - 1) / a.per + 1);
  const int lo_any = a.window > 0 ? max(0, base_pos + row0 / a.per - a.window + 1) : 0;
  int j0 = lo_any / kTok;
  int n = hi_any > lo_any ? (hi_any + kTok - 1) / kTok - j0 : 0;
  const int parts = min(a.splits, max(1, n / kSplitTiles));
  if (part >= parts) return;
  {
    const int b0 = (int)((long long)n * part / parts), b1 = (int)((long long)n * (part + 1) / parts);
    j0 += b0;
    n = b1 - b0;
  }
  const int nr = row_end - row0 > 128 ? NR : 1;   // row tiles in use

  constexpr int kMmaWarp = Cfg::SOFT + kDecW;
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  ch_before();
  __syncthreads();
  ch_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < Cfg::SOFT) {
    // ------------------------------------------------------------ softmax
    regs_inc<Cfg::R_SOFT>();
    const int r = warp >> 2;                       // row tile
    const int row_l = (warp & 3) * 32 + lane;      // row of it = TMEM lane
    const int row = row0 + r * 128 + row_l;
    const bool ok = row < rows;
    const int qi = ok ? row / a.per : 0, hq = head * a.per + (ok ? row - qi * a.per : 0);
    const uint32_t tq = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tS = tq + r * 128, tO = tq + Cfg::O_COL + r * D;

    // Q's row: fp16 after a power of two that puts its largest at 2^14 (exact down
    // to 2^-28 of it); dims in the order in which the code words yield them
    float unit = fabsf(a.scale_log2);
    {
      const uint16_t* src = a.q + (long long)(q0 + qi) * a.q_stride + (long long)hq * D;
      uint32_t top = 0;
      uint4 v[D / 8];
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        v[i] = ok ? *reinterpret_cast<const uint4*>(src + 8 * i) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t x = (&v[i].x)[k];
          top = max(top, max(x & 0x7FFFu, (x >> 16) & 0x7FFFu));
        }
      }
      const int e = a.bf16 ? (int)(top >> 7) - 127 : (int)(top >> 10) - 15;
      const int k2 = min(max(14 - e, -126), 126);
      float mul = __int_as_float((127 + k2) << 23);
      // never 0: -inf times it must stay -inf (1e-37 of a finite S is nothing)
      unit = fmaxf(unit * __int_as_float((127 - k2) << 23), 1e-37f);
      if (a.scale_log2 < 0.0f) mul = -mul;         // the row maximum below wants a positive factor
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        float f[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t x = (&v[i].x)[k];
          if (a.bf16) {
            f[2 * k] = __uint_as_float(x << 16);
            f[2 * k + 1] = __uint_as_float(x & 0xFFFF0000u);
          } else {
            const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&x));
            f[2 * k] = h.x;
            f[2 * k + 1] = h.y;
          }
        }
        uint4 o;
        o.x = pack2<false>(f[0] * mul, f[4] * mul);
        o.y = pack2<false>(f[1] * mul, f[5] * mul);
        o.z = pack2<false>(f[2] * mul, f[6] * mul);
        o.w = pack2<false>(f[3] * mul, f[7] * mul);
        *reinterpret_cast<uint4*>(sQ + r * Cfg::Q_BYTES + (i >> 3) * PANEL + row_l * 128 + (((i & 7) ^ (row_l & 7)) << 4)) = o;
      }
    }
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) mbar_arrive(q_full);

    const int pos = base_pos + row / a.per;
    const int hi_q = ok ? min(len, pos + 1) : 0, lo_q = ok && a.window > 0 ? max(0, pos - a.window + 1) : 0;
    const int r_first = row0 + r * 128, r_last = min(rows, r_first + 128) - 1;
    const int full_hi = min(len, base_pos + r_first / a.per + 1);
    const int full_lo = a.window > 0 ? base_pos + r_last / a.per - a.window + 1 : 0;
    float m = -INFINITY, l = 0.0f;
    bool live = true;
    for (int j = 0; r < nr && j < n; ++j) {
      live = ch_wait(&s_full[r], j & 1, abort_flag, a.wait_limit);
      live = __all_sync(0xffffffffu, live);
      if (!live) break;
      ch_after();
      const int t0 = (j0 + j) * kTok;
      float v[kTok];
#pragma unroll
      for (int c = 0; c < kTok; c += 32) ld32_async(tS + c, v + c);
#pragma unroll
      for (int c = 0; c < kTok; c += 32) wait32(v + c);
      if (!(t0 + kTok <= full_hi && t0 >= full_lo)) {   // warp-uniform
        const int hi = hi_q - t0, lo = lo_q - t0;
#pragma unroll
        for (int i = 0; i < kTok; ++i)
          if (i >= hi || i < lo) v[i] = -INFINITY;
      }
      float mx4[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
      for (int i = 4; i < kTok; i += 2) mx4[(i >> 1) & 3] = max3(mx4[(i >> 1) & 3], v[i], v[i + 1]);
      const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * unit;
      const bool up = mx > m + kLazy;              // always at the first visible token
      if (__any_sync(0xffffffffu, up)) {
        const float mn = up ? mx : m;
        const float alpha = up ? ch_exp2(m - mn) : 1.0f;
        m = mn;
        l *= alpha;
        if (j > 0) {   // the MMA on O before S's of this tile has finished
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float o[32];
            ld32_async(tO + c, o);
            wait32(o);
            uint32_t w[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(o[i] * alpha);
            st32(tO + c, w);
          }
        }
      }
      // p = 2^(S unit - m + kPShift); a masked -inf stays one (unit > 0)
      const float sub = kPShift - (m == -INFINITY ? 0.0f : m);
      const uint64_t unit2 = pair(unit, unit), sub2 = pair(sub, sub);
      uint64_t la = pair(0.0f, 0.0f), lb = la;
#pragma unroll
      for (int c = 0; c < kTok; c += 64) {
        uint32_t w[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          float y0, y1;
          unpair(fma2(pair(v[c + 2 * i], v[c + 2 * i + 1]), unit2, sub2), y0, y1);
          y0 = ch_exp2(y0);
          y1 = ch_exp2(y1);
          if (i & 1) la = add2(la, pair(y0, y1));
          else lb = add2(lb, pair(y0, y1));
          w[i] = pack2<false>(y0, y1);
        }
        st32(tS + c / 2, w);   // P over S's columns, which this row has read
      }
      {
        float l0, l1;
        unpair(add2(la, lb), l0, l1);
        l += l0 + l1;
      }
      wait_st();
      ch_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[r]);
    }
    if (live && n > 0 && r < nr) {
      live = ch_wait(&pv_done[r], (n - 1) & 1, abort_flag, a.wait_limit);
      live = __all_sync(0xffffffffu, live);
      ch_after();
    }
    auto emit = [&](int c, const float (&o)[32], float inv) {   // dims c .. c + 31 of the row
      uint16_t* dst = a.out + (long long)(q0 + qi) * a.out_stride + (long long)hq * D + c;
      if (ok) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint4 w;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            // a row that sees nothing gives zeros whatever its place in TMEM holds
            const float x0 = l == 0.0f ? 0.0f : o[8 * i + 2 * k] * inv;
            const float x1 = l == 0.0f ? 0.0f : o[8 * i + 2 * k + 1] * inv;
            (&w.x)[k] = a.bf16 ? pack2<true>(x0, x1) : pack2<false>(x0, x1);
          }
          *reinterpret_cast<uint4*>(dst + 8 * i) = w;
        }
      }
    };
    auto emit_lse = [&]() {
      if (ok && a.lse)
        a.lse[(long long)(q0 + qi) * a.q_heads + hq] =
            l == 0.0f ? -INFINITY : 0.69314718056f * (m + log2f(l) - kPShift);
    };
    if (parts == 1) {
      if (live) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          if (n > 0) {
            ld32_async(tO + c, o);
            wait32(o);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0.0f;
          }
          emit(c, o, inv);
        }
        emit_lse();
      }
    } else {
      const int rw = r * 128 + row_l;
      float* mine = a.slots + ((long long)item * a.splits + part) * Cfg::PART + rw;
      if (live && r < nr) {
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          ld32_async(tO + c, o);
          wait32(o);
#pragma unroll
          for (int i = 0; i < 32; ++i) __stcg(mine + (long long)(c + i) * Cfg::ROWS, o[i]);
        }
        __stcg(mine + (long long)D * Cfg::ROWS, m);
        __stcg(mine + (long long)(D + 1) * Cfg::ROWS, l);
      }
      // all softmax warps: a part that gave up is not counted
      const bool all = bar_and(1, Cfg::SOFT * 32, live);
      if (threadIdx.x == 0 && all) {
        unsigned prev;
        asm volatile("atom.add.acq_rel.gpu.u32 %0, [%1], 1;" : "=r"(prev) : "l"(a.counters + item) : "memory");
        *last_flag = prev == (unsigned)(parts - 1);
      }
      bar_and(1, Cfg::SOFT * 32, true);
      if (all && *last_flag && r < nr) {
        const float* p0 = a.slots + (long long)item * a.splits * Cfg::PART + rw;
        float f[kSplitMost];
        m = -INFINITY;
        for (int k = 0; k < parts; ++k) m = fmaxf(m, __ldcg(p0 + (long long)k * Cfg::PART + (long long)D * Cfg::ROWS));
        const float ref = m == -INFINITY ? 0.0f : m;
        l = 0.0f;
#pragma unroll
        for (int k = 0; k < kSplitMost; ++k) {
          f[k] = 0.0f;
          if (k < parts) {
            const float* pk = p0 + (long long)k * Cfg::PART + (long long)D * Cfg::ROWS;
            f[k] = ch_exp2(__ldcg(pk) - ref);
            l += f[k] * __ldcg(pk + Cfg::ROWS);
          }
        }
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0.0f;
#pragma unroll
          for (int k = 0; k < kSplitMost; ++k) {
            if (k < parts) {   // the same for every thread
#pragma unroll
              for (int i = 0; i < 32; ++i)
                o[i] = fmaf(f[k], __ldcg(p0 + (long long)k * Cfg::PART + (long long)(c + i) * Cfg::ROWS), o[i]);
            }
          }
          emit(c, o, inv);
        }
        emit_lse();
      }
      if (threadIdx.x == 0 && all && *last_flag) a.counters[item] = 0u;   // ready for the next call
    }
  } else if (warp < kMmaWarp) {
    // ------------------------------------------------------------ decode
    if constexpr (NR == 2) regs_dec<Cfg::R_DEC>();
    else regs_inc<Cfg::R_DEC>();
    const int dw = warp - Cfg::SOFT, L = dw * 32 + lane;
    const int* trow = a.table + (long long)b * a.max_pages;
    const int pm = (1 << a.page_log2) - 1;
    const int hi_tok = min(len, (j0 + n) * kTok);     // nothing is read past the last tile
    auto page_of = [&](int tok) {
      const int id = tok < hi_tok ? trow[tok >> a.page_log2] : 0;
      return (unsigned)id < (unsigned)a.pages ? id : 0;   // no access outside the cache
    };
    auto tile_at = [&](int id, int tok) -> const uint8_t* {   // the 16-token tile that holds tok
      const long long t = (((long long)id * a.heads + head) << (a.page_log2 - 4)) + ((tok & pm) >> 4);
      return a.cache + t * TB;
    };
    // keys: eight rows (tokens) x four 16-byte pieces (8-byte for 64 dims) a turn
    constexpr int KP = D == 256 ? 2 : 1;              // pieces per lane and turn
    constexpr int KWP = D == 64 ? 2 : 4;              // words per piece
    const int ktok = lane & 7, kt = lane >> 3;
    // values: eight tokens x one piece (D / 8 dims)
    constexpr int VW = D / 64;                        // words per piece and token
    const int vo = (L & 7) + 8 * (L >> 6), vg = (L >> 3) & 7;
    uint32_t kw[4][KP][KWP], kp[4][G], vw[8][VW], vp[8];
    int kid[4], vid;                                  // pages of the tile to be loaded next
    auto pages_k = [&](int j) {
#pragma unroll
      for (int it = 0; it < 4; ++it) kid[it] = page_of((j0 + j) * kTok + 32 * dw + 8 * it + ktok);
    };
    auto load_k = [&](int j) {
      const int t0 = (j0 + j) * kTok;
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const int tl = 32 * dw + 8 * it + ktok, tok = t0 + tl, at = tok & 15;
#pragma unroll
        for (int i = 0; i < KP; ++i)
#pragma unroll
          for (int w = 0; w < KWP; ++w) kw[it][i][w] = 0;
#pragma unroll
        for (int gr = 0; gr < G; ++gr) kp[it][gr] = 0;
        if (tok < hi_tok) {
          const uint8_t* tp = tile_at(kid[it], tok);
#pragma unroll
          for (int i = 0; i < KP; ++i) {
            if constexpr (D == 64) {
              const uint2 v = *reinterpret_cast<const uint2*>(tp + at * KROW + 8 * kt);
              kw[it][i][0] = v.x;
              kw[it][i][1] = v.y;
            } else {
              const int piece = (kt + 4 * i) ^ (D == 256 ? 4 * (at & 1) : 0);
              const uint4 v = *reinterpret_cast<const uint4*>(tp + at * KROW + 16 * piece);
              kw[it][i][0] = v.x;
              kw[it][i][1] = v.y;
              kw[it][i][KWP - 2] = v.z;
              kw[it][i][KWP - 1] = v.w;
            }
          }
#pragma unroll
          for (int gr = 0; gr < G; ++gr) {
            const uint8_t* pp = tp + KP_OFF + (at * G + gr) * PB;
            kp[it][gr] = MODE == kASYM ? *reinterpret_cast<const uint32_t*>(pp) : *reinterpret_cast<const uint16_t*>(pp);
          }
        }
      }
    };
    auto load_v = [&](int j) {
      const int t0 = (j0 + j) * kTok;
        const int tok0 = t0 + 8 * vo;
        const uint8_t* tp = tile_at(vid, tok0);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int at = (8 * vo + k) & 15;
          vp[k] = 0;
#pragma unroll
          for (int w = 0; w < VW; ++w) vw[k][w] = 0;
          // what lies past the sequence or before its window may be anything: its
          // values count as 0 (0 times a NaN found there would be a NaN)
          if (tok0 + k < hi_tok && tok0 + k >= first_seq) {
            const uint8_t* rp = tp + V_OFF + at * KROW + (D / 16) * kv_val_piece(D, vg, at);
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
              vw[k][VW - 2] = v.z;
              vw[k][VW - 1] = v.w;
            }
            const uint8_t* pp = tp + VP_OFF + (at * G + vg * (D / 8) / GD) * PB;
            vp[k] = MODE == kASYM ? *reinterpret_cast<const uint32_t*>(pp) : *reinterpret_cast<const uint16_t*>(pp);
          }
        }
    };
    // the loads of the next tile's keys run under the decoding of this one's values
    // and the other way round; page indices are fetched a tile before them
    pages_k(0);
    vid = page_of(j0 * kTok + 8 * vo);
    load_k(0);
    load_v(0);
    pages_k(1);
    vid = page_of((j0 + 1) * kTok + 8 * vo);
    for (int j = 0; j < n; ++j) {
      const int s = j % ST;
      const uint32_t ph = ((j / ST) & 1) ^ 1;
      bool ok = ch_wait(&k_empty[s], ph, abort_flag, a.wait_limit);
      if (!__all_sync(0xffffffffu, ok)) break;
      unsigned char* Kt = sK + s * Cfg::K_BYTES;
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const int tl = 32 * dw + 8 * it + ktok;
#pragma unroll
        for (int i = 0; i < KP; ++i)
#pragma unroll
          for (int w = 0; w < KWP; ++w) {
            const int nw = 4 * (w + 4 * i) + kt;      // natural word: dims 8 nw ..
            const uint32_t par = kp[it][(w + 4 * i) * 32 / GD];
            const uint32_t s2 = __byte_perm(par, 0, 0x1010);
            uint32_t bias = 0x64086408u, bias16 = 0xD480D480u;
            if constexpr (MODE == kASYM) zero_biases(__byte_perm(par, 0, 0x3232), bias, bias16);
            uint32_t d[4];
            decode_nibbles(kw[it][i][w], bias, bias16, d);
            uint4 o;
            o.x = hmul2_u16(d[0], s2);
            o.y = hmul2_u16(d[1], s2);
            o.z = hmul2_u16(d[2], s2);
            o.w = hmul2_u16(d[3], s2);
            *reinterpret_cast<uint4*>(Kt + (nw >> 3) * PANEL + tl * 128 + (((nw & 7) ^ (tl & 7)) << 4)) = o;
          }
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&k_full[s]);
      load_k(j + 1);
      pages_k(j + 2);
      ok = ch_wait(&v_empty[s], ph, abort_flag, a.wait_limit);
      if (!__all_sync(0xffffffffu, ok)) break;
      unsigned char* Vt = sV + s * Cfg::K_BYTES + (vo >> 3) * VPANEL;
      uint32_t sv[4], bias[4], bias16[4];
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        sv[h] = __byte_perm(vp[2 * h], vp[2 * h + 1], 0x5410);
        bias[h] = 0x64086408u;
        bias16[h] = 0xD480D480u;
        if constexpr (MODE == kASYM) zero_biases(__byte_perm(vp[2 * h], vp[2 * h + 1], 0x7632), bias[h], bias16[h]);
      }
#pragma unroll
      for (int w = 0; w < VW; ++w)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t d[4][4];
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const uint32_t u = __byte_perm(vw[2 * h][w], vw[2 * h + 1][w], half ? 0x7632 : 0x5410);
            decode_nibbles(u, bias[h], bias16[h], d[h]);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int row = vg * (D / 8) + 8 * w + 4 * half + e;
            uint4 o;
            o.x = hmul2_u16(d[0][e], sv[0]);
            o.y = hmul2_u16(d[1][e], sv[1]);
            o.z = hmul2_u16(d[2][e], sv[2]);
            o.w = hmul2_u16(d[3][e], sv[3]);
            *reinterpret_cast<uint4*>(Vt + row * 128 + (((vo & 7) ^ (row & 7)) << 4)) = o;
          }
        }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&v_full[s]);
      load_v(j + 1);
      vid = page_of((j0 + j + 2) * kTok + 8 * vo);
    }
  } else {
    // ------------------------------------------------------------ MMA issuer
    regs_dec<Cfg::R_MMA>();
    if (warp == kMmaWarp) {
      constexpr uint32_t kIdS = (1u << 4) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
      constexpr uint32_t kIdO = (1u << 4) | (((uint32_t)D >> 3) << 17) | ((128u >> 4) << 24);
      const uint32_t lead = elect_one();
      // the same answer for every lane: the warp stops as one
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, ch_wait(bar, parity, abort_flag, a.wait_limit)) != 0;
      };
      const uint32_t dq = ch_desc(smem_u32(sQ)), dk = ch_desc(smem_u32(sK)), dv = ch_desc(smem_u32(sV));
      // a descriptor's address field counts 16 bytes; offsets stay far inside it
      auto mma_s = [&](int r, int s) {
        const uint32_t qa = opaque(dq + r * (Cfg::Q_BYTES / 16)), ka = opaque(dk + s * (Cfg::K_BYTES / 16));
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (k >> 2) * (PANEL / 16) + 2 * (k & 3);
          ch_mma(tmem + r * 128, qa + off, ka + off, kIdS, k > 0, lead);
        }
        ch_commit(&s_full[r], lead);
      };
      bool ok = n > 0 && wait(q_full, 0) && wait(&k_full[0], 0);
      if (ok) {
        ch_after();
#pragma unroll
        for (int r = 0; r < nr; ++r) mma_s(r, 0);
        ch_commit(&k_empty[0], lead);
      }
      // per row tile: O += P V of tile j, then S of tile j + 1, so that one row
      // tile's softmax runs under the other's MMAs
      for (int j = 0; ok && j < n; ++j) {
        const int s = j % ST, s1 = (j + 1) % ST;
        ok = wait(&v_full[s], (j / ST) & 1);
#pragma unroll
        for (int r = 0; r < nr; ++r) {
          ok = ok && wait(&p_full[r], j & 1);
          if (!ok) break;
          ch_after();
          const uint32_t va = opaque(dv + s * (Cfg::K_BYTES / 16)), pa = opaque(tmem + r * 128);
#pragma unroll
          for (int k = 0; k < kTok / 16; ++k)
            ch_mma_ta(tmem + Cfg::O_COL + r * D, pa + 8 * k, va + (k >> 2) * (VPANEL / 16) + 2 * (k & 3),
                      kIdO, j > 0 || k > 0, lead);
          ch_commit(&pv_done[r], lead);
          if (r == nr - 1) ch_commit(&v_empty[s], lead);
          if (j + 1 < n) {
            if (r == 0) ok = wait(&k_full[s1], ((j + 1) / ST) & 1);
            // P shares S's columns: the MMA that reads it must be done
            ok = ok && wait(&pv_done[r], j & 1);
            if (!ok) break;
            ch_after();
            mma_s(r, s1);
            if (r == nr - 1) ch_commit(&k_empty[s1], lead);
          }
        }
      }
      // every MMA issued has finished before TMEM and the tiles are released
      ch_commit(drain, lead);
      if (!mbar_try(drain, 0)) {
        const long long c0 = clock64();
        while (!mbar_try(drain, 0))
          if (clock64() - c0 > kDrain) break;
      }
    }
  }

  ch_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    ch_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

template <int D, int MODE, int GD>
cudaError_t ch_launch(const ChArgs& args, unsigned ctas, cudaStream_t stream) {
  auto k = kv_chunk_kernel<D, MODE, GD>;
  // one CTA per SM: each takes all of its SM's tensor memory
  constexpr size_t smem = ChCfg<D>::SMEM > 120 * 1024 ? ChCfg<D>::SMEM : 120 * 1024;
  static_assert(smem <= 227 * 1024, "shared memory of the chunk kernel");
  static bool attr_set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return e;
    }
    attr_set[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(ChCfg<D>::THREADS, 1, 1);
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

}  // namespace

namespace {

// Tiles of rows (upper bound) and CTAs per tile: one while the tiles alone fill
// the SMs, else as many as do, at most kSplitMost.
struct ChPlan {
  int tiles_max, splits;
  long long tiles;
  size_t slots;
};
ChPlan ch_plan(int batch, int max_q, int q_heads, int kv_heads, int dim, int sms) {
  ChPlan p{};
  const int rows = 128 * (dim == 256 ? 1 : 2);
  p.tiles_max = (int)(((long long)max_q * (q_heads / kv_heads) + rows - 1) / rows);
  p.tiles = (long long)p.tiles_max * batch * kv_heads;
  p.splits = (int)std::max<long long>(1, std::min<long long>(kSplitMost, sms / p.tiles));
  if (p.splits > 1) p.slots = (size_t)p.tiles * p.splits * rows * (dim + 2) * sizeof(float);
  return p;
}

}  // namespace

size_t kv_chunk_slots(int batch, int max_q, int q_heads, int kv_heads, int dim, int sms) {
  return ch_plan(batch, max_q, q_heads, kv_heads, dim, sms).slots;
}

cudaError_t launch_kv_chunk(const KvAttend& p, int min_rows, unsigned* counters, float* slots,
                            long long wait_limit, cudaStream_t stream) {
  const KvCache& c = p.cache;
  ChArgs a{};
  a.q = static_cast<const uint16_t*>(p.q);
  a.cache = static_cast<const uint8_t*>(c.data);
  a.table = p.table;
  a.lens = p.lens;
  a.cu_q = p.cu_q;
  a.out = static_cast<uint16_t*>(p.out);
  a.lse = p.lse;
  a.q_stride = p.q_stride;
  a.out_stride = p.out_stride;
  a.wait_limit = wait_limit;
  a.batch = p.batch;
  a.total_q = p.total_q;
  a.max_q = p.max_q;
  a.heads = c.heads;
  a.q_heads = p.q_heads;
  a.per = p.q_heads / c.heads;
  a.page_log2 = c.page_log2;
  a.pages = c.pages;
  a.max_pages = p.max_pages;
  a.min_rows = min_rows;
  a.scale_log2 = p.scale * 1.4426950408889634f;
  a.window = p.window;
  a.bf16 = p.bf16;
  // split as the workspace was sized, by max_q; but max_q is the caller's bound and may
  // lie far above the queries there are, so the tiles (whose rows are 32-bit numbers in
  // the kernel) come from those
  const ChPlan plan = ch_plan(p.batch, p.max_q, p.q_heads, c.heads, c.dim, device_sms());
  const ChPlan real = ch_plan(p.batch, std::min(p.max_q, p.total_q), p.q_heads, c.heads, c.dim, device_sms());
  a.tiles_max = real.tiles_max;
  a.splits = 1;
  if (counters && plan.splits > 1) {   // at most a tile per SM then, and a counter each
    a.splits = plan.splits;
    a.counters = counters;
    a.slots = slots;
  }
  const long long ctas = real.tiles * a.splits;
  if (ctas > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  const int gd = c.dim / c.G;
#define CH_CASE(D, MO, GD) \
  if (c.dim == D && c.mode == MO && gd == GD) return ch_launch<D, MO, GD>(a, (unsigned)ctas, stream);
#define CH_MODES(D, GD) CH_CASE(D, kSYM, GD) CH_CASE(D, kASYM, GD)
  CH_MODES(64, 32) CH_MODES(64, 64) CH_MODES(128, 32) CH_MODES(128, 64) CH_MODES(128, 128)
  CH_MODES(256, 32) CH_MODES(256, 64) CH_MODES(256, 128) CH_MODES(256, 256)
#undef CH_MODES
#undef CH_CASE
  return cudaErrorInvalidValue;
}

unsigned kv_read_and_clear_error() {
  unsigned v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_kv_error, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  if (v) cudaMemcpyToSymbol(g_kv_error, &zero, sizeof(zero));
  return v;
}

}  // namespace qk
