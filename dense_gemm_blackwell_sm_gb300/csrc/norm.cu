// norm.cu -- host side of the block norms: how rows and columns are split over
// threads, CTAs and clusters, and the workspace of the column sums.
#include "norm.h"

#include <algorithm>

#include "ffn_launch.h"

namespace dgb {

namespace {

int elem_bytes(int32_t dtype) { return dtype == FFN_F32 ? 4 : 2; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// rows that all start on 16-byte boundaries (absent arrays count as aligned)
bool rows16(const void* p, int64_t ld, int bytes) { return p == nullptr || (aligned16(p) && ld * bytes % 16 == 0); }

int round32(int64_t n) { return (int)((n + 31) / 32 * 32); }

}  // namespace

cudaError_t launch_norm(const ffn_norm_t& a, const FfnDevice& dev, cudaStream_t st) {
  const int b = elem_bytes(a.dtype), E = 16 / b;
  NormShape sh{};
  const int64_t vectors = (a.D + E - 1) / E;  // of a row
  const int most = norm_most_vectors(b);
  if (vectors <= 32 * 4 && a.M > 2 * (int64_t)dev.num_sms) {
    // short rows: a warp each, no barrier
    sh.warp_rows = true;
    sh.nv = vectors <= 32 ? 1 : vectors <= 64 ? 2 : 4;
    sh.threads = 256;
    sh.grid = (a.M + 7) / 8;
  } else {
    // a CTA per row, with as many threads as let all rows run at once (short rows),
    // else with as many elements per thread as it can hold, which keeps several rows'
    // loads in flight on an SM
    sh.nv = 1;
    while (sh.nv < most && ((vectors + sh.nv - 1) / sh.nv * a.M > (int64_t)dev.num_sms * 1024 ||
                            vectors > 512 * (int64_t)sh.nv))
      sh.nv *= 2;
    sh.threads = round32((vectors + sh.nv - 1) / sh.nv);
    sh.grid = a.M;
  }
  const int pb = elem_bytes(a.param_dtype);
  sh.aligned = a.D % 8 == 0 && rows16(a.y, a.ld_y, b) && rows16(a.residual, a.ld_residual, b) &&
               rows16(a.s, a.ld_s, b) && rows16(a.n, a.ld_n, b) && rows16(a.gate, a.ld_gate, pb) &&
               aligned16(a.post_weight) && aligned16(a.post_bias) && aligned16(a.pre_weight) && aligned16(a.pre_bias);
  // the ring, where every group has a few rows
  {
    NormShape ring = sh;
    ring.ring = true;
    ring.warp_rows = vectors <= 32 * 4;
    ring.nv = ring.warp_rows ? (vectors <= 32 ? 1 : vectors <= 64 ? 2 : 4)
                             : (vectors <= 256 ? 1 : vectors <= 1024 ? 2 : 4);
    ring.threads = ring.warp_rows ? 256 : round32((vectors + ring.nv - 1) / ring.nv);
    const int groups = ring.warp_rows ? 8 : 1;
    ring.smem = (size_t)groups * kNormStages * (a.residual ? 2 : 1) * norm_slot_bytes(a.D * b);
    if (ring.threads <= 512 && ring.smem <= kNormRingBytes) {
      // (about 100 registers per thread and 6 KB of static shared memory)
      const int64_t per_sm =
          std::max<int64_t>(1, std::min<int64_t>((int64_t)(222 * 1024) / ((int64_t)ring.smem + 6144), 640 / ring.threads));
      ring.grid = std::min<int64_t>(per_sm * dev.num_sms, (a.M + groups - 1) / groups);
      if (a.M >= 2 * ring.grid * groups) sh = ring;
    }
  }
  switch (a.dtype) {
    case FFN_F16: return norm_forward_f16(a, sh, dev, st);
    case FFN_BF16: return norm_forward_bf16(a, sh, dev, st);
    default: return norm_forward_f32(a, sh, dev, st);
  }
}

namespace {

// The split of the backward pass; it depends on the sizes alone, so that the
// workspace can be sized without a device and sums are the same on every call.
NormGradShape grad_shape(const ffn_norm_grad_t& a) {
  constexpr int kResident = 304;  // CTAs of 256 threads: two on each of 152 SMs
  NormGradShape sh{};
  const int64_t threads = (a.D + kNormGradEach - 1) / kNormGradEach;
  sh.cluster = (int)((threads + kNormGradThreads - 1) / kNormGradThreads);
  sh.columns = ((a.D + sh.cluster - 1) / sh.cluster + kNormGradEach - 1) / kNormGradEach * kNormGradEach;
  sh.threads = round32(sh.columns / kNormGradEach);
  sh.lanes = sh.threads == 32 ? 8 : 1;
  const bool gates = a.gate != nullptr || a.dgate != nullptr;
  const int64_t groups = gates ? a.groups : 1;
  int64_t parts = (int64_t)kResident * (kNormGradThreads / (sh.threads * sh.lanes)) * sh.lanes / sh.cluster;
  parts = std::max<int64_t>(1, std::min(parts, a.M));
  if (groups >= parts && groups > 1) {
    sh.many = true;
    sh.parts_per_group = 0;
  } else {
    sh.parts_per_group = (int)std::min(parts / groups, a.M / groups);
    parts = sh.parts_per_group * groups;
  }
  sh.parts = (int)parts;
  sh.bias = a.dpost_bias != nullptr || a.dpre_bias != nullptr || (a.dgate != nullptr && a.post_bias != nullptr);
  return sh;
}

int sums_of(const ffn_norm_grad_t& a, const NormGradShape& sh, NormSums* ws, float* base) {
  int n = 0;
  const int64_t each = (int64_t)sh.parts * a.D;
  auto next = [&](bool need, float** p) {
    *p = nullptr;
    if (need) *p = base ? base + each * n : nullptr, ++n;
  };
  const bool gates = a.dgate != nullptr && !sh.many;
  next(a.dpost_weight != nullptr || gates, &ws->a);
  next(a.dpost_bias != nullptr || (gates && a.post_bias != nullptr), &ws->b);
  next(a.dpre_weight != nullptr, &ws->c);
  next(a.dpre_bias != nullptr, &ws->e);
  return n;
}

}  // namespace

size_t norm_backward_workspace(const ffn_norm_grad_t& a) {
  const NormGradShape sh = grad_shape(a);
  NormSums ws{};
  return (size_t)sums_of(a, sh, &ws, nullptr) * (size_t)sh.parts * (size_t)a.D * 4;
}

cudaError_t launch_norm_backward(const ffn_norm_grad_t& args, const FfnDevice& dev, cudaStream_t st) {
  ffn_norm_grad_t a = args;
  if (a.gate == nullptr && a.dgate == nullptr) a.groups = 1;
  NormGradShape sh = grad_shape(a);
  const int b = elem_bytes(a.dtype), pb = elem_bytes(a.param_dtype);
  sh.aligned = a.D % 8 == 0 && rows16(a.ds, a.ld_ds, b) && rows16(a.dn, a.ld_dn, b) && rows16(a.y, a.ld_y, b) &&
               rows16(a.s, a.ld_s, b) && rows16(a.dresidual, a.ld_dresidual, b) && rows16(a.dy, a.ld_dy, b) &&
               rows16(a.gate, a.ld_gate, pb) && aligned16(a.post_weight) && aligned16(a.pre_weight);
  const int arrays = (a.dn ? 2 : 0) + (a.y ? 1 : 0) + (a.ds ? 1 : 0);
  // three rows ahead where two CTAs still share an SM, else two
  auto bytes = [&](int stages) {
    return (size_t)sh.threads * sh.lanes * 32 * 4 +
           (size_t)sh.lanes * stages * arrays * norm_slot_bytes(sh.columns * elem_bytes(a.dtype));
  };
  sh.stages = bytes(kNormStages) <= 108 * 1024 ? kNormStages : 2;
  sh.smem = bytes(sh.stages);
  NormSums ws{};
  sums_of(a, sh, &ws, static_cast<float*>(a.workspace));
  switch (a.dtype) {
    case FFN_F16: return norm_backward_f16(a, sh, ws, dev, st);
    case FFN_BF16: return norm_backward_bf16(a, sh, ws, dev, st);
    default: return norm_backward_f32(a, sh, ws, dev, st);
  }
}

}  // namespace dgb
