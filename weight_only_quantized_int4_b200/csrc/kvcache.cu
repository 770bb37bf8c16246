// Writing keys and values into the 4-bit cache and reading them back
// (layout: kv.cuh and include/qmm.h).
//
// Both are one pass over their data and bound by memory: a thread takes eight
// dims of one row (16 bytes of k or v, one 32-bit word of codes), a group of
// GD dims is GD / 8 neighbouring lanes, whose largest and smallest values meet
// in shuffles; nothing goes through shared memory.
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
  long long words;          // tokens * heads * 2 * (dim / 8)
};

template <bool BF16>
__device__ __forceinline__ float kv_widen(uint32_t bits16) {
  if constexpr (BF16) return __uint_as_float(bits16 << 16);
  else return __half2float(__ushort_as_half((unsigned short)bits16));
}

// Word index -> (row of the call, k or v, head, natural word of the row).
template <int D>
__device__ __forceinline__ void kv_split(long long i, int heads, int& tok, int& head, int& which, int& n) {
  constexpr int W = D / 8;
  n = (int)(i % W);
  const long long row = i / W;               // (token, which, head)
  const int rows = 2 * heads;
  tok = (int)(row / rows);
  const int rr = (int)(row - (long long)tok * rows);
  which = rr >= heads;
  head = rr - which * heads;
}

// First byte of the tile that holds `slot` of a head.
template <int D, int MODE>
__device__ __forceinline__ uint8_t* kv_tile(const KvArgs& a, int slot, int head) {
  const long long page = slot >> a.page_log2;
  const int in_page = slot & ((1 << a.page_log2) - 1);
  const long long tile = (page * a.heads + head) * (1 << (a.page_log2 - 4)) + (in_page >> 4);
  return a.cache + tile * kv_tile_bytes(D, a.G, MODE);
}

// One rounding each, in IEEE fp32: s = fp16(absmax / 7) (SYM) or fp16((max -
// min) / 15) with 0 in the range (ASYM, z = rint(-min / s)), code = rint(x / s)
// + z.  For fp16 and bf16 inputs a quotient x / s is either a tie or at least
// 2^-15 away from one (x has at most 11 bits, (2k + 1) s at most 15), so fp32
// decides every code as exact arithmetic would.  NaN counts as 0 and infinities
// saturate: the cache only ever holds finite scales.
template <int D, int MODE, bool BF16>
__global__ void __launch_bounds__(kKvThreads) kv_store_kernel(const KvArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int GL = (D / 8) / a.G;   // lanes per group (4 .. 32)
  const long long step = (long long)gridDim.x * kKvThreads;
  for (long long i0 = (long long)blockIdx.x * kKvThreads; i0 < a.words; i0 += step) {
    const long long i = i0 + threadIdx.x;
    const bool in = i < a.words;   // whole rows: words is a multiple of D / 8
    int tok, head, which, n;
    kv_split<D>(in ? i : 0, a.heads, tok, head, which, n);
    const int slot = in ? a.slots[tok] : -1;
    const bool live = slot >= 0 && slot < a.slot_end;
    float x[8];
    {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (live)
        v = *reinterpret_cast<const uint4*>((which ? a.src[1] : a.src[0]) + tok * (which ? a.stride[1] : a.stride[0]) + head * D + n * 8);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t w = (&v.x)[k];
        x[2 * k] = kv_widen<BF16>(w & 0xFFFFu);
        x[2 * k + 1] = kv_widen<BF16>(w >> 16);
      }
    }
    float lo = 0.0f, hi = 0.0f;   // fminf / fmaxf pass over a NaN
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      lo = fminf(lo, x[k]);
      hi = fmaxf(hi, x[k]);
    }
    for (int m = 1; m < GL; m <<= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, m));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, m));
    }
    const float span = MODE == kASYM ? __fdiv_rn(hi - lo, 15.0f) : __fdiv_rn(fmaxf(hi, -lo), 7.0f);
    const __half sh = __float2half_rn(fminf(span, kKvMaxScale));
    const float s = __half2float(sh);
    float z = 8.0f;
    if (MODE == kASYM) z = s > 0.0f ? fminf(rintf(__fdiv_rn(-lo, s)), 15.0f) : 0.0f;
    uint32_t word = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float xk = x[k] == x[k] ? x[k] : 0.0f;
      const float q = s > 0.0f ? rintf(__fdiv_rn(xk, s)) + z : z;
      word |= (uint32_t)fminf(fmaxf(q, 0.0f), 15.0f) << (4 * k);
    }
    if (live) {
      uint8_t* t = kv_tile<D, MODE>(a, slot, head);
      const int at = slot & 15;
      const int w = which ? kv_val_word(D, n, at) : kv_key_word(D, n, at);
      *reinterpret_cast<uint32_t*>(t + which * (kKvTile * D / 2) + at * (D / 2) + 4 * w) = word;
      if (n % GL == 0) {
        uint8_t* p = t + kKvTile * D +
                     ((which * kKvTile + at) * a.G + n / GL) * kv_param_bytes(MODE);
        if (MODE == kASYM) *reinterpret_cast<__half2*>(p) = __halves2half2(sh, __float2half_rn(z));
        else *reinterpret_cast<__half*>(p) = sh;
      }
    }
  }
}

// (q - z) s in fp32 (exact: 5 x 11 bits), rounded once to the output type.  A
// slot outside the cache gives zeros.
template <int D, int MODE, bool BF16>
__global__ void __launch_bounds__(kKvThreads) kv_load_kernel(const KvArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int GL = (D / 8) / a.G;
  const long long step = (long long)gridDim.x * kKvThreads;
  for (long long i = (long long)blockIdx.x * kKvThreads + threadIdx.x; i < a.words; i += step) {
    int tok, head, which, n;
    kv_split<D>(i, a.heads, tok, head, which, n);
    const int slot = a.slots[tok];
    uint4 out = make_uint4(0, 0, 0, 0);
    if (slot >= 0 && slot < a.slot_end) {
      const uint8_t* t = kv_tile<D, MODE>(a, slot, head);
      const int at = slot & 15;
      const int w = which ? kv_val_word(D, n, at) : kv_key_word(D, n, at);
      const uint32_t word =
          *reinterpret_cast<const uint32_t*>(t + which * (kKvTile * D / 2) + at * (D / 2) + 4 * w);
      const uint8_t* p = t + kKvTile * D + ((which * kKvTile + at) * a.G + n / GL) * kv_param_bytes(MODE);
      float s, z = 8.0f;
      if (MODE == kASYM) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(p));
        s = f.x;
        z = f.y;
      } else {
        s = __half2float(*reinterpret_cast<const __half*>(p));
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float v0 = ((float)((word >> (8 * k)) & 15u) - z) * s;
        const float v1 = ((float)((word >> (8 * k + 4)) & 15u) - z) * s;
        (&out.x)[k] = pack2<BF16>(v0, v1);
      }
    }
    *reinterpret_cast<uint4*>((which ? a.dst[1] : a.dst[0]) + ((long long)tok * a.heads + head) * D + n * 8) = out;
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

cudaError_t kv_launch(void (*k)(KvArgs), const KvArgs& a, cudaStream_t stream) {
  // one word per thread; past 16 resident CTAs' worth per SM the grid strides
  const long long blocks = (a.words + kKvThreads - 1) / kKvThreads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min<long long>(blocks, 16ll * device_sms()), 1, 1);
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
  a.words = (long long)tokens * c.heads * 2 * (c.dim / 8);
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
    return kv_launch(kv_store_kernel<D, MO, BF>, a, stream);
  });
}

cudaError_t launch_kv_load(const KvCache& c, const int* slots, int tokens, bool bf16, void* k, void* v,
                           cudaStream_t stream) {
  KvArgs a = kv_args(c, slots, tokens);
  a.dst[0] = static_cast<uint16_t*>(k);
  a.dst[1] = static_cast<uint16_t*>(v);
  return kv_dispatch(c.dim, c.mode, bf16, [&]<int D, int MO, bool BF>() {
    return kv_launch(kv_load_kernel<D, MO, BF>, a, stream);
  });
}

}  // namespace qk
