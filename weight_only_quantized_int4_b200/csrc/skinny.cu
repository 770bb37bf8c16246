// Decode path: the plan of a call, and its plain kernels (skinny.cuh).
#include "skinny.cuh"

namespace qk {

// Device error word of the decode path.  Its waits are cp.async group waits,
// which always end, so nothing sets it today; qmm_check_error reads it with
// the tensor path's.
__device__ unsigned g_skinny_error = 0;

SkinnyPlan plan_skinny(int M, int N, int K, int bits, int group, int mode, bool bf16, int sms,
                       bool force_streamk) {
  SkinnyPlan p{};
  // token tiles of 8: 1 up to 8 tokens, 2 up to 16, 4 up to 32 (the plain
  // formats; zero-point options stay at 16 tokens per slab)
  p.nt = M <= 8 ? 1 : (M <= 16 || zero_opts(mode) ? 2 : 4);
  const int R = p.nt == 1 ? rb_per_tile<1>() : rb_per_tile<2>();
  p.rows = 16 * R;
  const int nrb = N / 16;
  p.tiles_n = (nrb + R - 1) / R;
  p.slabs = std::max(1, (M + 8 * p.nt - 1) / (8 * p.nt));
  const int nsc = (K + kSC - 1) / kSC;
  const long long units = (long long)p.tiles_n * nsc;
  const int tpg = tiles_per_group(group);
  p.smem = dispatch<true, -1>(bits, mode, bf16, p.nt, tpg, false,
                    [&]<int B, int MO, bool BF, int T, int TP, bool D>() { return smem_bytes<B, MO, T, TP, D>(); });
  const int occ = dispatch<true, -1>(bits, mode, bf16, p.nt, tpg, false,
                           [&]<int B, int MO, bool BF, int T, int TP, bool D>() { return occupancy<B, MO, BF, T, TP, D, false>(); });
  // one resident wave of CTAs; every warp is a stream-K worker with >= 1 unit
  long long warps = (long long)sms * (occ > 0 ? occ : 1) * kWarps;
  const long long cap = std::max<long long>(1, units * 8 / nsc);
  if (!force_streamk && warps >= (long long)p.tiles_n * kWarps) {
    // few row tiles: one CTA per tile, its warps split K, sums added in
    // shared memory (no split-K workspace)
    p.cta_tiles = 1;
    p.splits = p.tiles_n;
    p.warps = p.tiles_n * kWarps;
    p.ws_bytes = 0;
    // at most one tile per SM: each CTA has an SM to itself, so it takes the
    // deep ring (its warps' stages all requested up front on small matrices)
    if (p.tiles_n <= sms && !zero_opts(mode) && p.nt <= 2) {
      p.deep = 1;
      p.smem = dispatch<true, -1>(bits, mode, bf16, p.nt, tpg, true,
                        [&]<int B, int MO, bool BF, int T, int TP, bool D>() { return smem_bytes<B, MO, T, TP, D>(); });
    }
    return p;
  }
  if (warps > cap) warps = cap;
  if (warps > units) warps = units;
  const long long ctas = (warps + kWarps - 1) / kWarps;
  p.splits = (int)ctas;
  p.warps = (int)warps;
  const bool split = !(units % warps == 0 && (units / warps) % nsc == 0);
  if (split) {
    const size_t counters = ((size_t)p.slabs * p.tiles_n * sizeof(unsigned) + 255) / 256 * 256;
    const size_t slots = (size_t)p.slabs * 2 * warps * p.rows * 8 * p.nt * sizeof(float);
    p.ws_bytes = counters + slots;
  } else {
    p.ws_bytes = 0;
  }
  return p;
}

cudaError_t launch_skinny(const Problem& pr, const SkinnyPlan& plan, void* workspace,
                          cudaStream_t stream) {
  if (!pr.epilogue) return launch_skinny_t<false>(pr, plan, workspace, stream);
  switch (pr.mode) {
    case kSYM: return launch_skinny_epi_sym(pr, plan, workspace, stream);
    case kASYM: return launch_skinny_epi_asym(pr, plan, workspace, stream);
    default: return launch_skinny_epi_lut(pr, plan, workspace, stream);
  }
}

}  // namespace qk

// ---------------------------------------------------------------------------
// Decode path with a library-owned scratch buffer, for callers that cannot
// allocate device memory (see qmm_noalloc in qmm.h).
namespace qk {
namespace {

constexpr size_t kStaticScratchBytes = size_t(8) << 20;   // 8 MiB per device
__device__ __align__(256) unsigned char g_static_scratch[kStaticScratchBytes];

// Device address of g_static_scratch on the current device.  The symbol's
// name is only a host-side stand-in, so the address is looked up once per
// device (with that device current) and cached.
cudaError_t static_scratch(void** out) {
  // atomics: host threads making their first call on a device at the same
  // time may both look the address up; they store the same value
  static std::atomic<void*> addr[kMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  void* p = addr[dev].load(std::memory_order_acquire);
  if (!p) {
    e = cudaGetSymbolAddress(&p, g_static_scratch);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return e;
    }
    addr[dev].store(p, std::memory_order_release);
  }
  *out = p;
  return cudaSuccess;
}

}  // namespace

size_t static_scratch_bytes() { return kStaticScratchBytes; }

cudaError_t launch_skinny_static(const Problem& pr, int sms, cudaStream_t stream, bool* too_large) {
  *too_large = false;
  SkinnyPlan plan = plan_skinny(pr.M, pr.N, pr.K, pr.bits, pr.group, pr.mode, pr.bf16, sms);
  const size_t counters = ((size_t)plan.slabs * plan.tiles_n * sizeof(unsigned) + 255) / 256 * 256;
  const size_t slot2 = (size_t)plan.slabs * 2 * plan.rows * 8 * plan.nt * sizeof(float);  // per worker
  if (plan.ws_bytes > kStaticScratchBytes) {
    // fewer stream-K workers so that their partial-sum slots fit
    if (counters + slot2 > kStaticScratchBytes) {
      *too_large = true;
      return cudaSuccess;
    }
    const long long w = (long long)((kStaticScratchBytes - counters) / slot2);
    plan.warps = (int)std::min<long long>(plan.warps, w);
    plan.splits = (plan.warps + kWarps - 1) / kWarps;
    plan.ws_bytes = counters + slot2 * plan.warps;
  }
  void* ws = nullptr;
  if (plan.ws_bytes) {
    cudaError_t e = static_scratch(&ws);
    if (e != cudaSuccess) return e;
    // the arrival counters must start at zero; every call shares the buffer
    e = cudaMemsetAsync(ws, 0, counters, stream);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return e;
    }
  }
  return launch_skinny(pr, plan, ws, stream);
}

}  // namespace qk

namespace qk {
unsigned skinny_read_and_clear_error() {
  unsigned v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_skinny_error, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  if (v) cudaMemcpyToSymbol(g_skinny_error, &zero, sizeof(zero));
  return v;
}
}  // namespace qk
