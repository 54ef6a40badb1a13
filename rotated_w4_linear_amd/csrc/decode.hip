// The small-batch W4 linear without an epilogue of its own
// (w4_decode_kernels.h), the device probe it relies on, and where it fuses the
// transform.
#include <atomic>
#include <mutex>
#include <string>
#include <vector>

#include "w4_decode_kernels.h"

#pragma clang fp contract(off)

namespace paro {
namespace {

// Reads the XCC id of the XCD each workgroup runs on (hardware register 20,
// bits 0..3).
__global__ void xcc_probe_kernel(uint32_t* out) {
  if (threadIdx.x == 0) out[blockIdx.x] = __builtin_amdgcn_s_getreg((3 << 11) | 20) & 0xFu;
}

// Per device: 0 = not probed, 1 = workgroup b runs on the XCD of every other
// workgroup with the same b % 8 and the eight classes use eight XCDs (the
// round-robin dispatch the kernel relies on), 2 = it does not.
std::atomic<int> g_xcd_state[kMaxDevices];

}  // namespace

int xcd_dispatch_probe(int dev) {
  if (dev < 0 || dev >= kMaxDevices) return PARO_ERR_UNSUPPORTED;
  static std::mutex mu;
  std::lock_guard<std::mutex> lock(mu);
  if (g_xcd_state[dev].load(std::memory_order_acquire) != 0) return PARO_OK;
  constexpr int kBlocks = 4096;
  uint32_t* d_out = nullptr;
  hipError_t e = hipMalloc(&d_out, kBlocks * sizeof(uint32_t));
  if (e != hipSuccess) {
    set_error(std::string("device init: hipMalloc: ") + hipGetErrorString(e));
    return PARO_ERR_HIP;
  }
  std::vector<uint32_t> h(kBlocks, 0xFFFFFFFFu);
  hipLaunchKernelGGL(xcc_probe_kernel, dim3(kBlocks), dim3(64), 0, 0, d_out);
  e = hipGetLastError();
  if (e == hipSuccess) e = hipMemcpy(h.data(), d_out, kBlocks * sizeof(uint32_t), hipMemcpyDeviceToHost);
  (void)hipFree(d_out);
  if (e != hipSuccess) {  // nothing is cached: a later call probes again
    set_error(std::string("device init: XCD probe: ") + hipGetErrorString(e));
    return PARO_ERR_HIP;
  }
  bool ok = true;
  uint32_t seen = 0;
  for (int b = 0; b < kBlocks; ++b) {
    if (h[b] != h[b & 7]) ok = false;
    if (h[b] < 32) seen |= 1u << h[b];
    else ok = false;
  }
  if (__builtin_popcount(seen) != 8) ok = false;
  g_xcd_state[dev].store(ok ? 1 : 2, std::memory_order_release);
  return PARO_OK;
}

// The hot path only reads what the probe recorded; a device never probed
// takes the memory-side path, which is correct under any dispatch.
bool xcd_dispatch_is_round_robin() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return false;
  return g_xcd_state[dev].load(std::memory_order_acquire) == 1;
}

bool decode_fuses_rotation(const paro_rotation* r) {
  return r == nullptr || (r->lay.ppl == 1 && r->lay.stages <= 8);
}

// Beyond 16 tokens the N / 128 workgroups that each transform the same
// k-slice make the fused transform the larger cost, and one stand-alone
// transform (4-5 us) before the plain kernel is cheaper: from 33 tokens on
// every layer, from 17 on layers of at least 2^25 weights. Measured,
// graph-replayed, fused against transform-then-plain: 64 tokens, 4096 ->
// 14336 51.4 against 38.8 us, 14336 -> 4096 72.4 against 57.3, 4096 -> 4096
// 21.6 against about 18.4; 32 tokens, 4096 -> 4096 13.7 against about 15.
bool decode_fuses_rotation(const paro_rotation* r, int64_t M, int64_t N, int64_t d) {
  return decode_fuses_rotation(r) && (M <= 16 || (M <= 32 && N * d < (int64_t(1) << 25)));
}

hipError_t launch_w4_decode(const uint16_t* x, const uint8_t* qweight, const uint16_t* scales,
                            const uint8_t* zeros, const uint16_t* bias, uint16_t* y, int64_t M,
                            int64_t N, int64_t d, int group, const paro_rotation* r, void* ws,
                            hipStream_t stream) {
  return launch_w4_decode_epi<kEpiPlain>(x, qweight, scales, zeros, bias, y, M, N, d, group, r, ws, W4Epilogue{},
                                         stream);
}

}  // namespace paro
