// Writing keys and values into the 4-bit cache and reading them back
// (layout: kv.cuh and include/qmm.h).
//
// Both are one pass over their data and bound by memory.  A thread takes one
// 16-byte chunk of a code row, 32 dims: natural words 4i + c of a key row (so that
// the four lanes of a 32-dim block read and write whole 32-byte sectors of k), four
// consecutive ones of a value row.  Its column (head, chunk) is its own for the
// whole call, so the index arithmetic is done once, and it walks over tokens, two
// at a time with their loads in flight together.  A group of dims is some of a
// thread's words in up to eight neighbouring lanes, whose extremes meet in
// shuffles; nothing goes through shared memory.  Measured in short runs at 1965 MHz:
// 16384 tokens x 32 heads x 128 dims read back (bf16) in 57 us, 5.9 TB/s of codes in
// and values out (one 4-byte word per thread: 93 us; values written 64 bytes apart:
// 65 us); 8191 tokens x 32 heads stored (ASYM, groups of 64) and read back in 65 us,
// 5.3 TB/s for both (NaN looked for and codes clamped one by one: 74 us), of which the
// store takes 35 (5.0 TB/s, bound by issue) and the load 31.  In seconds of calls at
// the power cap (1.7 - 1.8 GHz): 59, and 69 = 37 + 31.
#include <algorithm>

#include "kv.cuh"

namespace qk {
namespace {

constexpr int kKvThreads = 128;
constexpr int kUnroll = 2;

struct KvArgs {
  const uint16_t* src[2];   // k, v of a store
  long long stride[2];      // elements between tokens
  uint16_t* dst[2];         // k, v of a load: [tokens][heads][dim]
  const int* slots;
  uint8_t* cache;
  int tokens, heads, page_log2;
  long long slot_end;       // pages << page_log2
  int cols;                 // chunks of keys (of values) per token: heads * dim / 32
  int span;                 // columns per block: min(cols, kKvThreads)
  int tpb;                  // tokens a block takes side by side: kKvThreads / span
};

// This thread's column and its token within the block's; blockIdx.z is 0 for
// keys, 1 for values.
struct KvThread {
  int head, chunk, ty;
  bool on;
};
template <int D>
__device__ __forceinline__ KvThread kv_thread(const KvArgs& a) {
  KvThread t;
  t.ty = (int)threadIdx.x / a.span;
  const int col = blockIdx.x * a.span + (int)threadIdx.x - t.ty * a.span;
  t.on = t.ty < a.tpb && col < a.cols;
  const int c = t.on ? col : 0;
  t.head = c / (D / 32);
  t.chunk = c % (D / 32);
  return t;
}

// Natural word at place i (0 .. 3) of 16-byte chunk c of a row, for a token at
// place `at` of its tile: the inverse of kv_key_word / kv_val_word.
template <int D, bool VAL>
__device__ __forceinline__ int natural_word(int c, int i, int at) {
  if constexpr (VAL) {
    if constexpr (D == 128) c ^= 2 * ((at >> 1) & 1);
    if constexpr (D == 256) c ^= 2 * (at & 3);
    return 4 * c + i;
  } else if constexpr (D == 64) {
    return 4 * (i & 1) + 2 * c + (i >> 1);
  } else if constexpr (D == 128) {
    return 4 * i + c;
  } else {
    c ^= 4 * (at & 1);
    return 4 * (i + (c & 4)) + (c & 3);
  }
}
// Which of the thread's four words share word i's group of GD dims: the group's
// number among them (0 ..), and how many of them there are.
template <int D, int GD, bool VAL>
__host__ __device__ constexpr int local_group(int i) {
  if (VAL) return 0;                              // 32 consecutive dims: one group
  if (D == 64) return GD == 32 ? (i & 1) : 0;     // 32-dim blocks alternate
  return GD >= 128 ? 0 : i * 32 / GD;             // word i lies in block i
}
// Lanes of a row over which a group extends (neighbours): 2^n.
template <int D, int GD, bool VAL>
__host__ __device__ constexpr int group_lanes() {
  if (VAL) return GD / 32;
  if (D == 64) return 2;
  return GD == 256 ? 8 : 4;
}

// First byte of the tile that holds `slot` of a head.
template <int TB>
__device__ __forceinline__ uint8_t* kv_tile(const KvArgs& a, int slot, int head) {
  const int page = slot >> a.page_log2;
  const int in_page = slot & ((1 << a.page_log2) - 1);
  const long long tile = (((long long)page * a.heads + head) << (a.page_log2 - 4)) + (in_page >> 4);
  return a.cache + tile * TB;
}

// Packed 16-bit minimum / maximum (they pass over a NaN; comparisons are exact).
template <bool BF16>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (BF16) asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <bool BF16>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (BF16) asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <bool BF16>
__device__ __forceinline__ float kv_lo(uint32_t w) {
  if constexpr (BF16) return __uint_as_float(w << 16);
  else return __half2float(__ushort_as_half((unsigned short)(w & 0xFFFFu)));
}
template <bool BF16>
__device__ __forceinline__ float kv_hi(uint32_t w) {
  if constexpr (BF16) return __uint_as_float(w & 0xFFFF0000u);
  else return __half2float(__ushort_as_half((unsigned short)(w >> 16)));
}
// The same maximum, NaN if either is one.
template <bool BF16>
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (BF16) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <bool BF16>
__device__ __forceinline__ bool has_nan(uint32_t w) {
  constexpr uint32_t kInf = BF16 ? 0x7F80u : 0x7C00u;
  return (w & 0x7FFFu) > kInf || ((w >> 16) & 0x7FFFu) > kInf;
}
// NaN in either half -> 0 there.
template <bool BF16>
__device__ __forceinline__ uint32_t drop_nan(uint32_t w) {
  constexpr uint32_t kInf = BF16 ? 0x7F80u : 0x7C00u;
  if ((w & 0x7FFFu) > kInf) w &= 0xFFFF0000u;
  if (((w >> 16) & 0x7FFFu) > kInf) w &= 0x0000FFFFu;
  return w;
}

// s = fp16(fl32(absmax / 7)) (SYM) or fp16(fl32((max - min) / 15)) with 0 in the
// range (ASYM, z = rint(-min / s)), code = rint(x / s) + z.
//
// The codes without a division: x and s have at most 11 bits, so x / s is either
// a tie k + 1/2 or at least 2^-12 away from one (with x = X 2^e, s = S 2^f the
// difference is a multiple of 1 / (2 S) or of (x / s) / X).  fma(x, fl(1 / s), 48)
// errs by at most 2^-24 |x / s| < 2^-20 before its rounding to steps of 2^-18 (its
// value lies in 32 .. 64): a tie comes out as the tie, everything else on its own
// side.  Adding 2^23 then rounds half to even at the integers.  NaN counts
// as 0 and infinities saturate: the cache only ever holds finite scales.
template <int D, int MODE, int GD, bool BF16, bool VAL>
__device__ __forceinline__ void store_rows(const KvArgs& a) {
  constexpr bool kA = MODE == kASYM;
  constexpr int G = D / GD, TB = kv_tile_bytes(D, G, MODE), PB = kv_param_bytes(MODE);
  constexpr int NG = VAL ? 1 : local_group<D, GD, VAL>(3) + 1;   // groups among the thread's words
  const KvThread th = kv_thread<D>(a);
  const uint16_t* src = a.src[VAL] + th.head * D;
  const long long stride = a.stride[VAL];
  // blocks in y take token runs of tpb * kUnroll in turn
  for (long long t0 = (long long)blockIdx.y * a.tpb * kUnroll; t0 < a.tokens;
       t0 += (long long)gridDim.y * a.tpb * kUnroll) {
    int slot[kUnroll];
    uint4 v[kUnroll][4];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long long tok = t0 + u * a.tpb + th.ty;
      slot[u] = th.on && tok < a.tokens ? a.slots[tok] : -1;
      if (slot[u] >= a.slot_end) slot[u] = -1;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint16_t* row = src + (t0 + u * a.tpb + th.ty) * stride;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[u][i] = make_uint4(0, 0, 0, 0);
        if (slot[u] >= 0)
          v[u][i] = *reinterpret_cast<const uint4*>(row + 8 * natural_word<D, VAL>(th.chunk, i, slot[u] & 15));
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      uint32_t nan = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4& x = v[u][i];
        nan = max2_nan<BF16>(nan, max2_nan<BF16>(max2_nan<BF16>(x.x, x.y), max2_nan<BF16>(x.z, x.w)));
      }
      if (has_nan<BF16>(nan)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint4& x = v[u][i];
          x.x = drop_nan<BF16>(x.x);
          x.y = drop_nan<BF16>(x.y);
          x.z = drop_nan<BF16>(x.z);
          x.w = drop_nan<BF16>(x.w);
        }
      }
      uint32_t ext[4];   // (largest, -smallest) of each word, then of each local group; 0 included
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4& x = v[u][i];
        const uint32_t mx = max2<BF16>(max2<BF16>(x.x, x.y), max2<BF16>(x.z, x.w));
        const uint32_t mn = min2<BF16>(min2<BF16>(x.x, x.y), min2<BF16>(x.z, x.w)) ^ 0x80008000u;
        const uint32_t e = max2<BF16>(__byte_perm(mx, mn, 0x5410), __byte_perm(mx, mn, 0x7632));
        const int lg = local_group<D, GD, VAL>(i);
        bool first = true;
#pragma unroll
        for (int k = 0; k < i; ++k) first = first && local_group<D, GD, VAL>(k) != lg;
        ext[lg] = first ? e : max2<BF16>(ext[lg], e);
      }
      float r[NG], zf[NG];
      __half sh[NG];
      bool clamp = false;   // a scale that is not the span's to 2^-11: saturated, or below fp16's normals
#pragma unroll
      for (int lg = 0; lg < NG; ++lg) {
#pragma unroll
        for (int m = 1; m < group_lanes<D, GD, VAL>(); m <<= 1)
          ext[lg] = max2<BF16>(ext[lg], __shfl_xor_sync(0xffffffffu, ext[lg], m));
        const float hi = fmaxf(kv_lo<BF16>(ext[lg]), 0.0f), nlo = fmaxf(kv_hi<BF16>(ext[lg]), 0.0f);
        const float span = kA ? __fdiv_rn(hi + nlo, 15.0f) : __fdiv_rn(fmaxf(hi, nlo), 7.0f);
        sh[lg] = __float2half_rn(fminf(span, kKvMaxScale));
        const float s = __half2float(sh[lg]);
        clamp = clamp || s >= kKvMaxScale || s < 6.103515625e-5f;
        r[lg] = s > 0.0f ? __frcp_rn(s) : 0.0f;
        zf[lg] = 8.0f;
        if (kA) zf[lg] = s > 0.0f ? fminf(rintf(__fdiv_rn(nlo, s)), 15.0f) : 0.0f;
      }
      // With s within 2^-11 of its span, SYM codes cannot leave -7 .. 7.  Nor can ASYM ones
      // fall below 0: rint(-x) + rint(x) = 0, and a quotient of two 11-bit numbers that is
      // not a half is 2^-12 away from it, so x r + 48 (off by 2^-18) rounds as x / s does.
      // Two halves rounded up can reach 16.
      uint32_t word[4];
      auto encode = [&]<bool CLAMP>() {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int lg = local_group<D, GD, VAL>(i);
          const float vlo = 48.0f - zf[lg], vhi = 63.0f - zf[lg];
          uint32_t acc = 0;
#pragma unroll
          for (int k = 7; k >= 0; --k) {
            const uint32_t w = (&v[u][i].x)[k >> 1];
            float x = fmaf((k & 1) ? kv_hi<BF16>(w) : kv_lo<BF16>(w), r[lg], 48.0f);
            if (CLAMP) x = fmaxf(x, vlo);
            if (CLAMP || kA) x = fminf(x, vhi);
            // the code is in the sum's low bits, 0x4B000000 + 48 - z above it
            acc = acc * 16u + __float_as_uint(x + 8388608.0f);
          }
          // take the eight offsets off again: 0x4B000000 and 0x4B0000000 survive mod 2^32
          word[i] = acc - (0x4B000000u + 0xB0000000u + 0x11111111u * (uint32_t)(48 - (int)zf[lg]));
        }
      };
      if (clamp) encode.template operator()<true>();
      else encode.template operator()<false>();
      if (slot[u] >= 0) {
        uint8_t* t = kv_tile<TB>(a, slot[u], th.head);
        const int at = slot[u] & 15;
        *reinterpret_cast<uint4*>(t + (VAL ? kKvTile * D / 2 : 0) + at * (D / 2) + 16 * th.chunk) =
            make_uint4(word[0], word[1], word[2], word[3]);
        uint8_t* p = t + kKvTile * D + ((VAL ? kKvTile : 0) + at) * G * PB;
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // the thread with a group's first word writes its parameters
          const int n = natural_word<D, VAL>(th.chunk, i, at), lg = local_group<D, GD, VAL>(i);
          if (n % (GD / 8) == 0) {
            if (kA) *reinterpret_cast<__half2*>(p + n / (GD / 8) * PB) = __halves2half2(sh[lg], __float2half_rn(zf[lg]));
            else *reinterpret_cast<__half*>(p + n / (GD / 8) * PB) = sh[lg];
          }
        }
      }
    }
  }
}

template <int D, int MODE, int GD, bool BF16>
__global__ void __launch_bounds__(kKvThreads) kv_store_kernel(const KvArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  if (blockIdx.z) store_rows<D, MODE, GD, BF16, true>(a);
  else store_rows<D, MODE, GD, BF16, false>(a);
}

// (q - z) s rounded once to the output type: in fp16 one multiplication of exact
// operands, for bf16 the exact fp32 product (5 x 11 bits) converted.  A slot
// outside the cache gives zeros.  Here a thread's words are (D / 32) i + c of both
// kinds of rows: the outputs, eight times the codes, go out in whole sectors.
template <int D, int MODE, int GD, bool BF16, bool VAL>
__device__ __forceinline__ void load_rows(const KvArgs& a) {
  constexpr int G = D / GD, TB = kv_tile_bytes(D, G, MODE), PB = kv_param_bytes(MODE);
  const KvThread th = kv_thread<D>(a);
  if (!th.on) return;
  uint16_t* dst = a.dst[VAL] + th.head * D;
  const long long stride = (long long)a.heads * D;
  for (long long t0 = (long long)blockIdx.y * a.tpb * kUnroll; t0 < a.tokens;
       t0 += (long long)gridDim.y * a.tpb * kUnroll) {
    int slot[kUnroll];
    uint32_t code[kUnroll][4], par[kUnroll][4];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long long tok = t0 + u * a.tpb + th.ty;
      slot[u] = tok < a.tokens ? a.slots[tok] : -1;
      if (slot[u] >= a.slot_end) slot[u] = -1;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
#pragma unroll
      for (int i = 0; i < 4; ++i) code[u][i] = par[u][i] = 0;
      if (slot[u] >= 0) {
        const uint8_t* t = kv_tile<TB>(a, slot[u], th.head);
        const int at = slot[u] & 15;
        const uint8_t* row = t + (VAL ? kKvTile * D / 2 : 0) + at * (D / 2);
        const uint8_t* p = t + kKvTile * D + ((VAL ? kKvTile : 0) + at) * G * PB;
        if constexpr (!VAL && D == 128) {   // the words of one 16-byte chunk
          const uint4 w = *reinterpret_cast<const uint4*>(row + 16 * th.chunk);
          code[u][0] = w.x;
          code[u][1] = w.y;
          code[u][2] = w.z;
          code[u][3] = w.w;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int n = D / 32 * i + th.chunk;
          if constexpr (VAL || D != 128)
            code[u][i] = *reinterpret_cast<const uint32_t*>(row + 4 * (VAL ? kv_val_word(D, n, at) : kv_key_word(D, n, at)));
          const uint8_t* pp = p + n / (GD / 8) * PB;   // (words of one group load the same parameter)
          par[u][i] = MODE == kASYM ? *reinterpret_cast<const uint32_t*>(pp) : *reinterpret_cast<const uint16_t*>(pp);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long long tok = t0 + u * a.tpb + th.ty;
      if (tok >= a.tokens) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t pr = par[u][i];
        uint32_t bias = 0x64086408u, bias16 = 0xD480D480u;
        if (MODE == kASYM) zero_biases(__byte_perm(pr, 0, 0x3232), bias, bias16);
        uint32_t d[4];
        decode_nibbles(code[u][i], bias, bias16, d);   // pairs of dims (p, p + 4)
        uint4 out;
        if constexpr (!BF16) {
          const uint32_t s2 = __byte_perm(pr, 0, 0x1010);
#pragma unroll
          for (int k = 0; k < 4; ++k) d[k] = hmul2_u16(d[k], s2);
          out.x = __byte_perm(d[0], d[1], 0x5410);
          out.y = __byte_perm(d[2], d[3], 0x5410);
          out.z = __byte_perm(d[0], d[1], 0x7632);
          out.w = __byte_perm(d[2], d[3], 0x7632);
        } else {
          const float s = kv_lo<false>(pr);
          float2 f[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) f[k] = __half22float2(*reinterpret_cast<const __half2*>(&d[k]));
          out.x = pack2<true>(f[0].x * s, f[1].x * s);
          out.y = pack2<true>(f[2].x * s, f[3].x * s);
          out.z = pack2<true>(f[0].y * s, f[1].y * s);
          out.w = pack2<true>(f[2].y * s, f[3].y * s);
        }
        if (slot[u] < 0) out = make_uint4(0, 0, 0, 0);   // not (8 - z) times a missing scale
        *reinterpret_cast<uint4*>(dst + tok * stride + 8 * (D / 32 * i + th.chunk)) = out;
      }
    }
  }
}

template <int D, int MODE, int GD, bool BF16>
__global__ void __launch_bounds__(kKvThreads) kv_load_kernel(const KvArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  if (blockIdx.z) load_rows<D, MODE, GD, BF16, true>(a);
  else load_rows<D, MODE, GD, BF16, false>(a);
}

template <class F>
cudaError_t kv_dispatch(const KvCache& c, bool bf16, F&& f) {
  const int gd = c.dim / c.G;
#define KV_CASE(D, MO, GD)                        \
  if (c.dim == D && c.mode == MO && gd == GD)     \
    return bf16 ? f.template operator()<D, MO, GD, true>() : f.template operator()<D, MO, GD, false>();
#define KV_MODES(D, GD) KV_CASE(D, kSYM, GD) KV_CASE(D, kASYM, GD)
  KV_MODES(64, 32) KV_MODES(64, 64) KV_MODES(128, 32) KV_MODES(128, 64) KV_MODES(128, 128)
  KV_MODES(256, 32) KV_MODES(256, 64) KV_MODES(256, 128) KV_MODES(256, 256)
#undef KV_MODES
#undef KV_CASE
  return cudaErrorInvalidValue;
}

cudaError_t kv_launch(void (*k)(KvArgs), const KvArgs& a, cudaStream_t stream) {
  const unsigned gx = (unsigned)((a.cols + a.span - 1) / a.span);
  const long long run = (long long)a.tpb * kUnroll, runs = (a.tokens + run - 1) / run;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(gx, (unsigned)std::min<long long>(runs, 65535), 2);
  cfg.blockDim = dim3(kKvThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k, a);
  if (e != cudaSuccess) cudaGetLastError();   // report it once, here
  return e;
}

KvArgs kv_args(const KvCache& c, const int* slots, int tokens) {
  KvArgs a{};
  a.cache = static_cast<uint8_t*>(c.data);
  a.slots = slots;
  a.tokens = tokens;
  a.heads = c.heads;
  a.page_log2 = c.page_log2;
  a.slot_end = (long long)c.pages << c.page_log2;
  a.cols = c.heads * (c.dim / 32);
  a.span = std::min(a.cols, kKvThreads);
  a.tpb = kKvThreads / a.span;
  return a;
}

}  // namespace

cudaError_t launch_kv_store(const KvCache& c, const void* k, const void* v, bool bf16, long long k_stride,
                            long long v_stride, const int* slots, int tokens, cudaStream_t stream) {
  KvArgs a = kv_args(c, slots, tokens);
  a.src[0] = static_cast<const uint16_t*>(k);
  a.src[1] = static_cast<const uint16_t*>(v);
  a.stride[0] = k_stride;
  a.stride[1] = v_stride;
  return kv_dispatch(c, bf16, [&]<int D, int MO, int GD, bool BF>() {
    return kv_launch(kv_store_kernel<D, MO, GD, BF>, a, stream);
  });
}

cudaError_t launch_kv_load(const KvCache& c, const int* slots, int tokens, bool bf16, void* k, void* v,
                           cudaStream_t stream) {
  KvArgs a = kv_args(c, slots, tokens);
  a.dst[0] = static_cast<uint16_t*>(k);
  a.dst[1] = static_cast<uint16_t*>(v);
  return kv_dispatch(c, bf16, [&]<int D, int MO, int GD, bool BF>() {
    return kv_launch(kv_load_kernel<D, MO, GD, BF>, a, stream);
  });
}

}  // namespace qk
