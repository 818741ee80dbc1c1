// norm.cu -- host side of the block norms: how rows and columns are split over
// threads, CTAs and clusters, and the workspace of the column sums.
#include "norm.h"

#include <algorithm>

#include "ffn_launch.h"

namespace dgb {

namespace {

int elem_bytes(int32_t dtype) { return dtype == FFN_F32 ? 4 : 2; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int round32(int64_t n) { return (int)((n + 31) / 32 * 32); }

// rows this far apart start at the same offset to 16-byte boundaries
int row_period(int64_t pitch_bytes) {
  int period = 1;
  while (pitch_bytes * period % 16 != 0) period *= 2;
  return period;
}

}  // namespace

cudaError_t launch_norm(const ffn_norm_t& a, const FfnDevice& dev, cudaStream_t st) {
  const int b = elem_bytes(a.dtype), E = 16 / b;
  // a row that may start off a boundary takes one vector more, if the largest CTA holds that
  // (else k_norm splits it from its start: D > 32761 in 16 bits, D > 32765 in 32)
  const bool aligned = a.D * b % 16 == 0 && aligned16(a.y) && a.ld_y * b % 16 == 0;
  const int most = norm_most_vectors(b);
  const int64_t shifted = (a.D + E - 1 + (aligned ? 0 : E - 1)) / E;
  const int64_t vectors = shifted <= 1024 * most ? shifted : (a.D + E - 1) / E;
  NormShape direct{};
  if (vectors <= 32 * 4 && a.M > 2 * (int64_t)dev.num_sms) {
    // short rows: a warp each, no barrier
    direct.warp_rows = true;
    direct.nv = vectors <= 32 ? 1 : vectors <= 64 ? 2 : 4;
    direct.threads = 256;
    direct.grid = (a.M + 7) / 8;
  } else {
    // a CTA per row, with as many threads as let all rows run at once (short rows),
    // else with as many elements per thread as it can hold, which keeps several rows'
    // loads in flight on an SM
    direct.nv = 1;
    while (direct.nv < most && ((vectors + direct.nv - 1) / direct.nv * a.M > (int64_t)dev.num_sms * 1024 ||
                                vectors > 512 * (int64_t)direct.nv))
      direct.nv *= 2;
    direct.threads = round32((vectors + direct.nv - 1) / direct.nv);
    direct.grid = a.M;
  }
  // The ring, where the rows of all arrays start alike (and, settled at the launch,
  // where every group has a few of them).
  NormShape ring{};
  ring.period = row_period(a.ld_y * b);
  auto alike = [&](const void* p, int64_t ld) {
    return p == nullptr || (((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(a.y)) & 15u) == 0 &&
                            (ld - a.ld_y) * b % 16 == 0);
  };
  const bool layer = a.kind == FFN_NORM_LAYER;
  ring.warp_rows = vectors <= 32 * 4;
  ring.nv = ring.warp_rows ? (vectors <= 32 ? 1 : vectors <= 64 ? 2 : 4) : (!layer && vectors > 1024 ? 4 : 2);
  ring.threads = ring.warp_rows ? 256 : round32((vectors + ring.nv - 1) / ring.nv);
  ring.smem = (size_t)kNormStages * (a.residual ? 2 : 1) * (size_t)(ring.nv * ring.threads * 16);
  const bool ring_ok = alike(a.residual, a.ld_residual) && alike(a.s, a.ld_s) && alike(a.n, a.ld_n) &&
                       (layer || (!a.post_bias && !a.pre_bias)) &&
                       ring.threads <= 512 && ring.smem <= kNormRingBytes;
  const int64_t ld = a.residual ? std::min(a.ld_y, a.ld_residual) : a.ld_y;
  ring.head = aligned16(a.y) ? 0 : rows_at_an_end(ld, E);
  ring.tail = a.M - rows_at_an_end(ld, E);
  const NormShape* maybe_ring = ring_ok ? &ring : nullptr;
  switch (a.dtype) {
    case FFN_F16: return norm_forward_f16(a, direct, maybe_ring, dev, st);
    case FFN_BF16: return norm_forward_bf16(a, direct, maybe_ring, dev, st);
    default: return norm_forward_f32(a, direct, maybe_ring, dev, st);
  }
}

namespace {

// The split of the backward pass; it depends on the sizes alone, so that the
// workspace can be sized without a device and sums are the same on every call.
NormGradShape grad_shape(const ffn_norm_grad_t& a) {
  constexpr int kNumSms = 152;  // each takes 512 threads of this kernel
  const bool gates = a.gate != nullptr || a.dgate != nullptr;
  const int64_t groups = gates ? a.groups : 1;
  auto split = [&](int each) {
    NormGradShape sh{};
    sh.each = each;
    sh.period = row_period(a.D * elem_bytes(a.dtype));
    // columns and threads of a CTA, with room for `spare` columns more; whether the largest
    // cluster holds the row so
    auto cut = [&](int spare) {
      for (sh.cluster = 1;; ++sh.cluster) {
        sh.columns = ((a.D + sh.cluster - 1) / sh.cluster + 15) / 16 * 16;
        sh.threads = round32((sh.columns + spare + each - 1) / each);
        if (sh.threads <= kNormGradThreads) return true;
        if (sh.cluster == 8) return false;
      }
    };
    // a shifted row may need 8 columns more; where they do not fit (D > 32640) rows are split
    // from their starts, and the threads bring those that are off a boundary (2000 x 32640
    // bf16 415 us, 2000 x 32641 1350)
    if (!cut(sh.period > 1 ? 8 : 0)) {
      sh.period = 1;
      cut(0);
    }
    sh.lanes = sh.threads == 32 ? 8 : 1;
    sh.per_sm = 2 * kNormGradThreads / (sh.threads * sh.lanes);
    int64_t parts = (int64_t)kNumSms * sh.per_sm * sh.lanes / sh.cluster;
    // two rows at least per part: a part's sums cost about what a row does
    parts = std::max<int64_t>(1, std::min(parts, (a.M + 1) / 2));
    if (groups >= parts && groups > 1) {
      sh.many = true;
      sh.parts_per_group = 0;
      sh.period = 1;
      parts = std::min(groups, parts);
    } else {
      sh.parts_per_group = (int)std::max<int64_t>(1, std::min(parts / groups, a.M / groups));
      if (sh.parts_per_group < sh.period) sh.period = 1;
      sh.parts_per_group = sh.parts_per_group / sh.period * sh.period;
      parts = sh.parts_per_group * groups;
    }
    sh.parts = (int)parts;
    return sh;
  };
  // 8 columns per thread where one CTA of that many threads takes the row with room to
  // spare, else 16: a row's chain of sums and barriers is shorter then and more rows are
  // under way, until a row needs a cluster (us with 8 and with 16 columns when the rule was
  // made, bf16: 8192 x 1024 32.5 and 40.1 (29.9 today), LayerNorm 45.7 and 79.9 (43.3 today);
  // 8192 x 64 18.9 and 28.8; 8192 x 2048 58.4 and 51.6; 8192 x 4096 in CTAs of 512 threads
  // 123, in clusters of two 175, with 16 columns 85 (78 today))
  NormGradShape sh = split(16);
  if (!sh.many && a.D < 8 * kNormGradThreads) {
    const NormGradShape fine = split(8);
    if (!fine.many && fine.cluster == 1) sh = fine;
  }
  sh.per = (int)(a.M / groups);
  sh.share = sh.many ? NormShare::of(groups, sh.parts)
                     : NormShare::of((sh.per + sh.period - 1) / sh.period, sh.parts_per_group / sh.period);
  sh.bias = a.dpost_bias != nullptr || a.dpre_bias != nullptr || (a.dgate != nullptr && a.post_bias != nullptr);
  return sh;
}

int sums_of(const ffn_norm_grad_t& a, const NormGradShape& sh, NormSums* ws, float* base) {
  int n = 0;
  const int64_t each = (int64_t)sh.parts * sh.cluster * sh.threads * sh.each;
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
  return (size_t)sums_of(a, sh, &ws, nullptr) * (size_t)sh.parts * (size_t)(sh.cluster * sh.threads * sh.each) * 4;
}

cudaError_t launch_norm_backward(const ffn_norm_grad_t& args, const FfnDevice& dev, cudaStream_t st) {
  ffn_norm_grad_t a = args;
  if (a.gate == nullptr && a.dgate == nullptr) a.groups = 1;
  NormGradShape sh = grad_shape(a);
  const int b = elem_bytes(a.dtype);
  const struct {
    const void* p;
    int64_t ld;
  } arrays[6] = {{a.s, a.ld_s}, {a.dn, a.ld_dn}, {a.y, a.ld_y}, {a.ds, a.ld_ds}, {a.dresidual, a.ld_dresidual},
                 {a.dy, a.ld_dy}};
  for (int i = 0; i < 6; ++i) {
    const int64_t off = (sh.period > 1 ? arrays[i].ld - a.D : arrays[i].ld) * b;
    if (arrays[i].p != nullptr && (!aligned16(arrays[i].p) || off % 16 != 0)) sh.slow |= 1u << i;
  }
  int64_t ld = a.dn ? std::min(a.ld_s, a.ld_dn) : a.ld_ds;
  if (a.y) ld = std::min(ld, a.ld_y);
  if (a.ds) ld = std::min(ld, a.ld_ds);
  sh.tail = a.M - rows_at_an_end(ld, 16 / b);
  sh.full = a.dn && a.ds && a.y && a.dresidual && a.dy && (a.flags & FFN_NORM_POST) != 0;
  const int rows = (a.dn ? 2 : 0) + (a.y ? 1 : 0) + (a.ds ? 1 : 0);
  // three rows ahead where the SM holds that for all its CTAs, else two
  auto bytes = [&](int stages) {
    return (size_t)sh.threads * sh.lanes * sh.each * 2 * 4 +
           (size_t)sh.lanes * stages * rows * (size_t)(sh.each * sh.threads * b);
  };
  sh.stages = bytes(kNormStages) * (size_t)sh.per_sm <= 216 * 1024 ? kNormStages : 2;
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
