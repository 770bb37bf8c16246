// Writing keys and values into the 4-bit cache and reading them back
// (layout: kv.cuh and include/qmm.h).
//
// Both are one pass over their data and bound by memory.  A thread takes eight
// dims of one row (16 bytes of k or v, one 32-bit word of codes): the word of a
// (k or v, head) column is its own for the whole call, so the index arithmetic
// is done once, and it walks over tokens, kUnroll at a time with their loads in
// flight together.  A group of GD dims is GD / 8 neighbouring lanes, whose
// largest and smallest values meet in shuffles; nothing goes through shared
// memory.
#include <algorithm>

#include "kv.cuh"

namespace qk {
namespace {

constexpr int kKvThreads = 256;

struct KvArgs {
  const uint16_t* src[2];   // k, v of a store
  long long stride[2];      // elements between tokens
  uint16_t* dst[2];         // k, v of a load: [tokens][heads][dim]
  const int* slots;
  uint8_t* cache;
  int tokens, heads, G, page_log2;
  long long slot_end;       // pages << page_log2
  int cols;                 // words of codes per token: 2 * heads * dim / 8
  int span;                 // columns per block: min(cols, kKvThreads)
  int tpb;                  // tokens a block takes side by side: kKvThreads / span
};

// This thread's column and its token within the block's.
struct KvThread {
  int head, which, n, ty;
  bool on;
};
template <int D>
__device__ __forceinline__ KvThread kv_thread(const KvArgs& a) {
  constexpr int W = D / 8;
  KvThread t;
  t.ty = (int)threadIdx.x / a.span;
  const int col = blockIdx.x * a.span + (int)threadIdx.x - t.ty * a.span;
  t.on = t.ty < a.tpb && col < a.cols;
  const int c = t.on ? col : 0;
  t.n = c % W;
  const int row = c / W;
  t.which = row >= a.heads;
  t.head = row - (t.which ? a.heads : 0);
  return t;
}

// First byte of the tile that holds `slot` of a head.
__device__ __forceinline__ uint8_t* kv_tile(const KvArgs& a, int slot, int head, int TB) {
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
template <int D, int MODE, bool BF16, int U>
__global__ void __launch_bounds__(kKvThreads) kv_store_kernel(const KvArgs a) {
  constexpr bool kA = MODE == kASYM;
  const KvThread th = kv_thread<D>(a);
  const int GL = (D / 8) / a.G;   // lanes per group (4 .. 32)
  const int TB = kv_tile_bytes(D, a.G, MODE);
  const uint16_t* src = (th.which ? a.src[1] : a.src[0]) + th.head * D + th.n * 8;
  const long long stride = th.which ? a.stride[1] : a.stride[0];
  pdl_wait();
  pdl_launch_dependents();
  // blocks in y take token runs of tpb * U in turn
  for (long long t0 = (long long)blockIdx.y * a.tpb * U; t0 < a.tokens; t0 += (long long)gridDim.y * a.tpb * U) {
    int slot[U];
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long tok = t0 + u * a.tpb + th.ty;
      slot[u] = th.on && tok < a.tokens ? a.slots[tok] : -1;
      if (slot[u] >= a.slot_end) slot[u] = -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      v[u] = make_uint4(0, 0, 0, 0);
      if (slot[u] >= 0) v[u] = *reinterpret_cast<const uint4*>(src + (t0 + u * a.tpb + th.ty) * stride);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = drop_nan<BF16>(w[k]);
      // (largest, -smallest) of the group, 0 included
      const uint32_t mx = max2<BF16>(max2<BF16>(w[0], w[1]), max2<BF16>(w[2], w[3]));
      const uint32_t mn = min2<BF16>(min2<BF16>(w[0], w[1]), min2<BF16>(w[2], w[3])) ^ 0x80008000u;
      uint32_t ext = max2<BF16>(__byte_perm(mx, mn, 0x5410), __byte_perm(mx, mn, 0x7632));
      for (int m = 1; m < GL; m <<= 1) ext = max2<BF16>(ext, __shfl_xor_sync(0xffffffffu, ext, m));
      const float hi = fmaxf(kv_lo<BF16>(ext), 0.0f), nlo = fmaxf(kv_hi<BF16>(ext), 0.0f);
      const float span = kA ? __fdiv_rn(hi + nlo, 15.0f) : __fdiv_rn(fmaxf(hi, nlo), 7.0f);
      const __half sh = __float2half_rn(fminf(span, kKvMaxScale));
      const float s = __half2float(sh);
      const float r = s > 0.0f ? __frcp_rn(s) : 0.0f;
      float z = 8.0f;
      if (kA) z = s > 0.0f ? fminf(rintf(__fdiv_rn(nlo, s)), 15.0f) : 0.0f;
      const float vlo = 48.0f - z, vhi = 63.0f - z;
      uint32_t word = 0;
#pragma unroll
      for (int k = 7; k >= 0; --k) {
        const float x = (k & 1) ? kv_hi<BF16>(w[k >> 1]) : kv_lo<BF16>(w[k >> 1]);
        const float q = fminf(fmaxf(fmaf(x, r, 48.0f), vlo), vhi) + 8388608.0f;
        word = word * 16u + __float_as_uint(q);   // the code is in q's low bits, 0x4B000000 + 48 - z above it
      }
      // take the eight offsets off again: 0x4B000000 and 0x4B0000000 survive mod 2^32
      word -= 0x4B000000u + 0xB0000000u + 0x11111111u * (uint32_t)(48 - (int)z);
      if (slot[u] >= 0) {
        uint8_t* t = kv_tile(a, slot[u], th.head, TB);
        const int at = slot[u] & 15;
        const int wi = th.which ? kv_val_word(D, th.n, at) : kv_key_word(D, th.n, at);
        *reinterpret_cast<uint32_t*>(t + th.which * (kKvTile * D / 2) + at * (D / 2) + 4 * wi) = word;
        if (th.n % GL == 0) {
          uint8_t* p = t + kKvTile * D + ((th.which * kKvTile + at) * a.G + th.n / GL) * kv_param_bytes(MODE);
          if (kA) *reinterpret_cast<__half2*>(p) = __halves2half2(sh, __float2half_rn(z));
          else *reinterpret_cast<__half*>(p) = sh;
        }
      }
    }
  }
}

// (q - z) s rounded once to the output type: in fp16 one multiplication of exact
// operands, for bf16 the exact fp32 product (5 x 11 bits) converted.  A slot
// outside the cache gives zeros.
template <int D, int MODE, bool BF16, int U>
__global__ void __launch_bounds__(kKvThreads) kv_load_kernel(const KvArgs a) {
  const KvThread th = kv_thread<D>(a);
  const int GL = (D / 8) / a.G;
  const int TB = kv_tile_bytes(D, a.G, MODE);
  uint16_t* dst = (th.which ? a.dst[1] : a.dst[0]) + th.head * D + th.n * 8;
  const long long stride = (long long)a.heads * D;
  pdl_wait();
  pdl_launch_dependents();
  if (!th.on) return;
  for (long long t0 = (long long)blockIdx.y * a.tpb * U; t0 < a.tokens; t0 += (long long)gridDim.y * a.tpb * U) {
    int slot[U];
    uint32_t word[U], par[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long tok = t0 + u * a.tpb + th.ty;
      slot[u] = tok < a.tokens ? a.slots[tok] : -1;
      if (slot[u] >= a.slot_end) slot[u] = -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      word[u] = par[u] = 0;
      if (slot[u] >= 0) {
        const uint8_t* t = kv_tile(a, slot[u], th.head, TB);
        const int at = slot[u] & 15;
        const int wi = th.which ? kv_val_word(D, th.n, at) : kv_key_word(D, th.n, at);
        word[u] = *reinterpret_cast<const uint32_t*>(t + th.which * (kKvTile * D / 2) + at * (D / 2) + 4 * wi);
        const uint8_t* p = t + kKvTile * D + ((th.which * kKvTile + at) * a.G + th.n / GL) * kv_param_bytes(MODE);
        par[u] = MODE == kASYM ? *reinterpret_cast<const uint32_t*>(p) : *reinterpret_cast<const uint16_t*>(p);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long tok = t0 + u * a.tpb + th.ty;
      if (tok >= a.tokens) continue;
      uint32_t bias = 0x64086408u, bias16 = 0xD480D480u;
      if (MODE == kASYM) zero_biases(__byte_perm(par[u], 0, 0x3232), bias, bias16);
      uint32_t d[4];
      decode_nibbles(word[u], bias, bias16, d);   // pairs of dims (p, p + 4)
      uint4 out;
      if constexpr (!BF16) {
        const uint32_t s2 = __byte_perm(par[u], 0, 0x1010);
#pragma unroll
        for (int k = 0; k < 4; ++k) d[k] = hmul2_u16(d[k], s2);
        out.x = __byte_perm(d[0], d[1], 0x5410);
        out.y = __byte_perm(d[2], d[3], 0x5410);
        out.z = __byte_perm(d[0], d[1], 0x7632);
        out.w = __byte_perm(d[2], d[3], 0x7632);
      } else {
        const float s = kv_lo<false>(par[u]);
        float2 f[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) f[k] = __half22float2(*reinterpret_cast<const __half2*>(&d[k]));
        out.x = pack2<true>(f[0].x * s, f[1].x * s);
        out.y = pack2<true>(f[2].x * s, f[3].x * s);
        out.z = pack2<true>(f[0].y * s, f[1].y * s);
        out.w = pack2<true>(f[2].y * s, f[3].y * s);
      }
      if (slot[u] < 0) out = make_uint4(0, 0, 0, 0);   // not (8 - z) times a missing scale
      *reinterpret_cast<uint4*>(dst + tok * stride) = out;
    }
  }
}

template <class F>
cudaError_t kv_dispatch(int dim, int mode, bool bf16, F&& f) {
#define KV_CASE(D, MO) \
  if (dim == D && mode == MO) return bf16 ? f.template operator()<D, MO, true>() : f.template operator()<D, MO, false>();
  KV_CASE(64, kSYM) KV_CASE(64, kASYM) KV_CASE(128, kSYM) KV_CASE(128, kASYM) KV_CASE(256, kSYM)
  KV_CASE(256, kASYM)
#undef KV_CASE
  return cudaErrorInvalidValue;
}

// Calls whose threads would not fill the GPU take one token per thread (latency:
// more SMs share the work), larger ones four (four loads in flight per thread).
constexpr int kUnroll = 4;
bool kv_small(const KvArgs& a) { return (long long)a.tokens * a.cols <= 2048ll * device_sms(); }

cudaError_t kv_launch(void (*k)(KvArgs), const KvArgs& a, int unroll, cudaStream_t stream) {
  const unsigned gx = (unsigned)((a.cols + a.span - 1) / a.span);
  const long long runs = (a.tokens + (long long)a.tpb * unroll - 1) / ((long long)a.tpb * unroll);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(gx, (unsigned)std::min<long long>(runs, 65535), 1);
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
  a.G = c.G;
  a.page_log2 = c.page_log2;
  a.slot_end = (long long)c.pages << c.page_log2;
  a.cols = 2 * c.heads * (c.dim / 8);
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
  return kv_dispatch(c.dim, c.mode, bf16, [&]<int D, int MO, bool BF>() {
    return kv_small(a) ? kv_launch(kv_store_kernel<D, MO, BF, 1>, a, 1, stream)
                       : kv_launch(kv_store_kernel<D, MO, BF, kUnroll>, a, kUnroll, stream);
  });
}

cudaError_t launch_kv_load(const KvCache& c, const int* slots, int tokens, bool bf16, void* k, void* v,
                           cudaStream_t stream) {
  KvArgs a = kv_args(c, slots, tokens);
  a.dst[0] = static_cast<uint16_t*>(k);
  a.dst[1] = static_cast<uint16_t*>(v);
  return kv_dispatch(c.dim, c.mode, bf16, [&]<int D, int MO, bool BF>() {
    return kv_small(a) ? kv_launch(kv_load_kernel<D, MO, BF, 1>, a, 1, stream)
                       : kv_launch(kv_load_kernel<D, MO, BF, kUnroll>, a, kUnroll, stream);
  });
}

}  // namespace qk
