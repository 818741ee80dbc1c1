// ffn.cu -- the C ABI of the feed-forward block's operators (include/ffn.h):
// argument validation, the per-device state, launches and status checks.
#include <map>
#include <mutex>
#include <set>
#include <tuple>
#include <utility>

#include "ffn.h"
#include "ffn_launch.h"
#include "launch.h"

using namespace dgb;

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 31;
constexpr int64_t kMaxNormD = 32768;
constexpr int kMaxDevices = 64;

// the status word of the bounded waits, one per device that loads the library
__device__ uint32_t g_ffn_status[4];

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The current device, checked once per device to be one this library has code for.
gemm_status_t current_ffn_device(FfnDevice* out) {
  static std::mutex mu;
  static FfnDevice known[kMaxDevices] = {};
  int dev = 0, major = 0, minor = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();
    return GEMM_ERR_NO_DEVICE;
  }
  try {
    std::lock_guard<std::mutex> lock(mu);
    FfnDevice& d = known[dev];
    if (d.status == nullptr) {
      void* p = nullptr;
      if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
          cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
          cudaDeviceGetAttribute(&d.num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_NO_DEVICE;
      }
      if (major != 10 || minor != 3) return GEMM_ERR_ARCH;
      if (cudaGetSymbolAddress(&p, g_ffn_status) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_CUDA;
      }
      d.status = static_cast<uint32_t*>(p);
    }
    *out = d;
    return GEMM_OK;
  } catch (...) {
    return GEMM_ERR_OOM;
  }
}

gemm_status_t launched(cudaError_t e) {
  if (e == cudaSuccess) return GEMM_OK;
  cudaGetLastError();
  return GEMM_ERR_CUDA;
}

// A row pitch: 0 means dense.  False where it is shorter than a row.
bool pitch(int64_t* ld, int64_t row) {
  if (*ld == 0) *ld = row;
  return *ld >= row && *ld < kMaxDim;
}

gemm_status_t gated_sizes(int64_t M, int64_t F, int64_t K, int32_t dtype, int32_t act, int64_t timeout_ns) {
  if (dtype != FFN_F16 && dtype != FFN_BF16) return GEMM_ERR_UNSUPPORTED_DTYPE;
  if (M < 0 || F < 1 || K < 1 || M >= kMaxDim || 2 * F >= kMaxDim || K >= kMaxDim) return GEMM_ERR_INVALID_ARG;
  if (act < GEMM_ACT_NONE || act > GEMM_ACT_GELU_ERF || timeout_ns < 0) return GEMM_ERR_INVALID_ARG;
  if (K % 8 != 0) return GEMM_ERR_UNSUPPORTED_SHAPE;  // TMA row pitch
  return GEMM_OK;
}

gemm_status_t norm_sizes(int64_t M, int64_t D, int64_t groups, int32_t dtype, int32_t param_dtype, int32_t kind,
                         int32_t flags, bool has_gate) {
  if (dtype < FFN_F16 || dtype > FFN_F32 || (param_dtype != dtype && param_dtype != FFN_F32))
    return GEMM_ERR_UNSUPPORTED_DTYPE;
  if (M < 0 || D < 1 || M >= kMaxDim || D >= kMaxDim) return GEMM_ERR_INVALID_ARG;
  if (kind != FFN_NORM_RMS && kind != FFN_NORM_LAYER) return GEMM_ERR_INVALID_ARG;
  if ((flags & ~(FFN_NORM_POST | FFN_NORM_PRE)) != 0) return GEMM_ERR_INVALID_ARG;
  if (has_gate && (groups < 1 || (M > 0 && (groups > M || M % groups != 0)))) return GEMM_ERR_INVALID_ARG;
  if (D > kMaxNormD) return GEMM_ERR_UNSUPPORTED_SHAPE;
  return GEMM_OK;
}

int elem(int32_t dtype) { return dtype == FFN_F32 ? 4 : 2; }

gemm_status_t norm_grad_sizes(const ffn_norm_grad_t& a) {
  return norm_sizes(a.M, a.D, a.groups, a.dtype, a.param_dtype, a.kind, a.flags,
                    a.gate != nullptr || a.dgate != nullptr);
}

}  // namespace

// A kernel's shared-memory limit is raised once per device.
cudaError_t dgb::allow_smem_once(const void* func, size_t bytes) {
  static std::mutex mu;
  static std::set<std::pair<int, const void*>> done;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  try {
    std::lock_guard<std::mutex> lock(mu);
    if (done.count({dev, func})) return cudaSuccess;
    e = allow_dynamic_smem(func, bytes);
    if (e == cudaSuccess) done.insert({dev, func});
    return e;
  } catch (...) {
    return cudaErrorMemoryAllocation;
  }
}

cudaError_t dgb::resident_ctas(const void* func, int threads, size_t smem, size_t most, int* out) {
  static std::mutex mu;
  static std::map<std::tuple<int, const void*, int, size_t>, int> known;
  cudaError_t e = allow_smem_once(func, most);
  int dev = 0;
  if (e == cudaSuccess) e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  try {
    std::lock_guard<std::mutex> lock(mu);
    const auto key = std::make_tuple(dev, func, threads, smem);
    const auto it = known.find(key);
    if (it != known.end()) {
      *out = it->second;
      return cudaSuccess;
    }
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(out, func, threads, smem);
    if (e == cudaSuccess) known[key] = *out;
    return e;
  } catch (...) {
    return cudaErrorMemoryAllocation;
  }
}

extern "C" {

gemm_status_t ffn_gated(const ffn_gated_t* args, gemm_stream_t stream) {
  if (!args) return GEMM_ERR_INVALID_ARG;
  ffn_gated_t a = *args;
  const gemm_status_t st = gated_sizes(a.M, a.F, a.K, a.dtype, a.activation, a.timeout_ns);
  if (st != GEMM_OK) return st;
  if (!pitch(&a.ld_x, a.K) || !pitch(&a.ld_w, a.K) || !pitch(&a.ld_h, a.F) || !pitch(&a.ld_gu, 2 * a.F))
    return GEMM_ERR_INVALID_ARG;
  if (a.M == 0) return GEMM_OK;
  if (!a.x || !a.w || !a.h) return GEMM_ERR_INVALID_ARG;
  if (!aligned(a.x, 16) || !aligned(a.w, 16) || a.ld_x % 8 != 0 || a.ld_w % 8 != 0 || !aligned(a.h, 2) ||
      !aligned(a.gu, 2))
    return GEMM_ERR_MISALIGNED;
  FfnDevice dev;
  const gemm_status_t ds = current_ffn_device(&dev);
  if (ds != GEMM_OK) return ds;
  return launched(launch_gated(a, dev, reinterpret_cast<cudaStream_t>(stream)));
}

int64_t ffn_gated_backward_workspace(const ffn_gated_grad_t* args) {
  if (!args || gated_sizes(args->M, args->F, args->K, args->dtype, args->activation, args->timeout_ns) != GEMM_OK)
    return -1;
  return (int64_t)gated_backward_workspace(*args);
}

gemm_status_t ffn_gated_backward(const ffn_gated_grad_t* args, gemm_stream_t stream) {
  if (!args) return GEMM_ERR_INVALID_ARG;
  ffn_gated_grad_t a = *args;
  const gemm_status_t st = gated_sizes(a.M, a.F, a.K, a.dtype, a.activation, a.timeout_ns);
  if (st != GEMM_OK) return st;
  if (a.ld_dgu == 0) a.ld_dgu = (2 * a.F + 7) / 8 * 8;
  if (!pitch(&a.ld_x, a.K) || !pitch(&a.ld_w, a.K) || !pitch(&a.ld_gu, 2 * a.F) || !pitch(&a.ld_dh, a.F) ||
      !pitch(&a.ld_dgu, 2 * a.F) || !pitch(&a.ld_dx, a.K) || !pitch(&a.ld_dw, a.K))
    return GEMM_ERR_INVALID_ARG;
  if (a.ld_x % 8 != 0 || a.ld_w % 8 != 0 || a.ld_dgu % 8 != 0 || !aligned(a.x, 16) || !aligned(a.w, 16) ||
      !aligned(a.dgu, 16) || !aligned(a.gu, 2) || !aligned(a.dh, 2) || !aligned(a.dx, 2) || !aligned(a.dw, 2) ||
      !aligned(a.workspace, 32))
    return GEMM_ERR_MISALIGNED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  FfnDevice dev;
  if (a.M == 0) {
    // no token: dw is a sum of nothing
    if (!a.dw) return GEMM_OK;
    const gemm_status_t ds = current_ffn_device(&dev);
    if (ds != GEMM_OK) return ds;
    return launched(cudaMemset2DAsync(a.dw, (size_t)a.ld_dw * 2, 0, (size_t)a.K * 2, (size_t)(2 * a.F), s));
  }
  if (!a.dh || !a.dgu) return GEMM_ERR_INVALID_ARG;
  if (!a.x && (a.dw || !a.gu)) return GEMM_ERR_INVALID_ARG;
  if (!a.workspace && gated_backward_workspace(a) > 0) return GEMM_ERR_INVALID_ARG;
  if (!a.w && (a.dx || !a.gu)) return GEMM_ERR_INVALID_ARG;
  const gemm_status_t ds = current_ffn_device(&dev);
  if (ds != GEMM_OK) return ds;
  return launched(launch_gated_backward(a, dev, s));
}

gemm_status_t ffn_norm(const ffn_norm_t* args, gemm_stream_t stream) {
  if (!args) return GEMM_ERR_INVALID_ARG;
  ffn_norm_t a = *args;
  const gemm_status_t st =
      norm_sizes(a.M, a.D, a.groups, a.dtype, a.param_dtype, a.kind, a.flags, a.gate != nullptr);
  if (st != GEMM_OK) return st;
  if (!pitch(&a.ld_y, a.D) || !pitch(&a.ld_residual, a.D) || !pitch(&a.ld_gate, a.D) || !pitch(&a.ld_s, a.D) ||
      !pitch(&a.ld_n, a.D))
    return GEMM_ERR_INVALID_ARG;
  if (a.M == 0) return GEMM_OK;
  if (!a.y || ((a.flags & FFN_NORM_PRE) != 0) != (a.n != nullptr) || (!a.s && !a.n)) return GEMM_ERR_INVALID_ARG;
  const uintptr_t e = (uintptr_t)elem(a.dtype), pe = (uintptr_t)elem(a.param_dtype);
  if (!aligned(a.y, e) || !aligned(a.residual, e) || !aligned(a.s, e) || !aligned(a.n, e) || !aligned(a.gate, pe) ||
      !aligned(a.post_weight, pe) || !aligned(a.post_bias, pe) || !aligned(a.pre_weight, pe) ||
      !aligned(a.pre_bias, pe))
    return GEMM_ERR_MISALIGNED;
  FfnDevice dev;
  const gemm_status_t ds = current_ffn_device(&dev);
  if (ds != GEMM_OK) return ds;
  return launched(launch_norm(a, dev, reinterpret_cast<cudaStream_t>(stream)));
}

int64_t ffn_norm_backward_workspace(const ffn_norm_grad_t* args) {
  if (!args || norm_grad_sizes(*args) != GEMM_OK) return -1;
  return args->M == 0 ? 0 : (int64_t)norm_backward_workspace(*args);
}

gemm_status_t ffn_norm_backward(const ffn_norm_grad_t* args, gemm_stream_t stream) {
  if (!args) return GEMM_ERR_INVALID_ARG;
  ffn_norm_grad_t a = *args;
  const gemm_status_t st = norm_grad_sizes(a);
  if (st != GEMM_OK) return st;
  if (!pitch(&a.ld_ds, a.D) || !pitch(&a.ld_dn, a.D) || !pitch(&a.ld_y, a.D) || !pitch(&a.ld_s, a.D) ||
      !pitch(&a.ld_gate, a.D) || !pitch(&a.ld_dresidual, a.D) || !pitch(&a.ld_dy, a.D))
    return GEMM_ERR_INVALID_ARG;
  const bool post = (a.flags & FFN_NORM_POST) != 0, pre = (a.flags & FFN_NORM_PRE) != 0;
  if ((!post && (a.dpost_weight || a.dpost_bias)) || (!pre && (a.dpre_weight || a.dpre_bias)))
    return GEMM_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  FfnDevice dev;
  if (a.M == 0) {
    // no row: the parameters' gradients are sums of nothing
    if (!a.dgate && !a.dpost_weight && !a.dpost_bias && !a.dpre_weight && !a.dpre_bias) return GEMM_OK;
    const gemm_status_t ds = current_ffn_device(&dev);
    if (ds != GEMM_OK) return ds;
    cudaError_t e = cudaSuccess;
    if (a.dgate) e = cudaMemsetAsync(a.dgate, 0, (size_t)(a.groups * a.D) * 4, s);
    for (float* p : {a.dpost_weight, a.dpost_bias, a.dpre_weight, a.dpre_bias})
      if (p && e == cudaSuccess) e = cudaMemsetAsync(p, 0, (size_t)a.D * 4, s);
    return launched(e);
  }
  if (pre != (a.dn != nullptr) || (!a.ds && !a.dn) || (pre && !a.s) || ((post || a.dgate) && !a.y))
    return GEMM_ERR_INVALID_ARG;
  const uintptr_t e = (uintptr_t)elem(a.dtype), pe = (uintptr_t)elem(a.param_dtype);
  if (!aligned(a.ds, e) || !aligned(a.dn, e) || !aligned(a.y, e) || !aligned(a.s, e) || !aligned(a.dresidual, e) ||
      !aligned(a.dy, e) || !aligned(a.gate, pe) || !aligned(a.post_weight, pe) || !aligned(a.post_bias, pe) ||
      !aligned(a.pre_weight, pe) || !aligned(a.dgate, 4) || !aligned(a.dpost_weight, 4) || !aligned(a.dpost_bias, 4) ||
      !aligned(a.dpre_weight, 4) || !aligned(a.dpre_bias, 4) || !aligned(a.workspace, 16))
    return GEMM_ERR_MISALIGNED;
  if (norm_backward_workspace(a) > 0 && !a.workspace) return GEMM_ERR_INVALID_ARG;
  const gemm_status_t ds = current_ffn_device(&dev);
  if (ds != GEMM_OK) return ds;
  return launched(launch_norm_backward(a, dev, s));
}

gemm_status_t ffn_check(gemm_stream_t stream) {
  FfnDevice dev;
  const gemm_status_t ds = current_ffn_device(&dev);
  if (ds != GEMM_OK) return ds;
  uint32_t word = 0;
  if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess ||
      cudaMemcpy(&word, dev.status, sizeof(word), cudaMemcpyDeviceToHost) != cudaSuccess ||
      (word != 0 && cudaMemset(dev.status, 0, sizeof(word)) != cudaSuccess)) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  return word != 0 ? GEMM_ERR_DEVICE_TIMEOUT : GEMM_OK;
}

}  // extern "C"
