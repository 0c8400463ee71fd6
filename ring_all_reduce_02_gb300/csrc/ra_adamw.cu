// ra_adamw: argument checks, the overlap rule over many tensors, and the launches.
#include <math.h>

#include <algorithm>
#include <new>
#include <vector>

#include "ra_adamw.cuh"
#include "ra_host.h"

namespace ra {

#define RA_DECLARE_ADAMW(P, G)                                                                                   \
  cudaError_t launch_adamw_small_##P##_##G(bool s8, const AdamArgs<kAdamSmall>& a, uint32_t ctas, cudaStream_t s); \
  cudaError_t launch_adamw_large_##P##_##G(bool s8, const AdamArgs<kAdamLarge>& a, uint32_t ctas, cudaStream_t s);
#define RA_DECLARE_ADAMW_P(P) RA_DECLARE_ADAMW(P, 0) RA_DECLARE_ADAMW(P, 1) RA_DECLARE_ADAMW(P, 2)
RA_DECLARE_ADAMW_P(0)
RA_DECLARE_ADAMW_P(1)
RA_DECLARE_ADAMW_P(2)

using AdamSmallFn = cudaError_t (*)(bool, const AdamArgs<kAdamSmall>&, uint32_t, cudaStream_t);
using AdamLargeFn = cudaError_t (*)(bool, const AdamArgs<kAdamLarge>&, uint32_t, cudaStream_t);
#define RA_ADAMW_ROW(K, P) {launch_adamw_##K##_##P##_0, launch_adamw_##K##_##P##_1, launch_adamw_##K##_##P##_2}
const AdamSmallFn kAdamSmallFns[3][3] = {RA_ADAMW_ROW(small, 0), RA_ADAMW_ROW(small, 1), RA_ADAMW_ROW(small, 2)};
const AdamLargeFn kAdamLargeFns[3][3] = {RA_ADAMW_ROW(large, 0), RA_ADAMW_ROW(large, 1), RA_ADAMW_ROW(large, 2)};

}  // namespace ra

namespace {

struct Span {
  uintptr_t lo, hi;
  bool written;
};

// Sorts spans by address. Lists of tensors mostly come as a few ascending runs
// (slices of flat buffers), so the runs are found and merged.
void sort_spans(std::vector<Span>& v) {
  const auto before = [](const Span& a, const Span& b) { return a.lo < b.lo; };
  std::vector<size_t> ends;  // of the ascending runs
  for (size_t i = 1; i <= v.size(); ++i)
    if (i == v.size() || before(v[i], v[i - 1])) ends.push_back(i);
  std::vector<Span> w(v.size());
  while (ends.size() > 1) {
    size_t begin = 0, kept = 0;
    for (size_t k = 0; k < ends.size(); k += 2) {
      const size_t mid = ends[k], end = k + 1 < ends.size() ? ends[k + 1] : mid;
      std::merge(v.begin() + begin, v.begin() + mid, v.begin() + mid, v.begin() + end, w.begin() + begin, before);
      ends[kept++] = begin = end;
    }
    ends.resize(kept);
    v.swap(w);
  }
}

// Whether a written span overlaps any other.
bool written_overlap(std::vector<Span>& v) {
  sort_spans(v);
  uintptr_t written_to = 0, any_to = 0;
  for (const Span& s : v) {
    if (s.lo < written_to || (s.written && s.lo < any_to)) return true;
    any_to = std::max(any_to, s.hi);
    if (s.written) written_to = std::max(written_to, s.hi);
  }
  return false;
}

// The buffers of a step come as seven lists: parameters, gradients, moments, scales, copies.
constexpr int kLists = 7;
struct Sizes {
  uint64_t param, grad, moment, copy;  // bytes of an element; copy: 0 if there are none
  bool s8;
};
// Tensor t's buffer of a list: its address (null where the list has none for it), its bytes and its alignment.
const void* buffer_of(const ra_adamw_tensor_t& t, int list, const Sizes& z, uint64_t* bytes, uintptr_t* align) {
  const uint64_t scales = (t.count + RA_ADAMW_BLOCK - 1) / RA_ADAMW_BLOCK;
  const void* p[kLists] = {t.param, t.grad, t.exp_avg, t.exp_avg_sq, t.exp_avg_scale, t.exp_avg_sq_scale, t.copy};
  const uint64_t n = list == 4 || list == 5 ? scales : t.count;
  const uint64_t es = list == 0 ? z.param : list == 1 ? z.grad : list <= 3 ? z.moment : list <= 5 ? 4 : z.copy;
  *bytes = n * es, *align = (uintptr_t)es;
  return p[list];
}
bool list_used(int list, const Sizes& z) { return list == 4 || list == 5 ? z.s8 : list < 6 || z.copy; }

bool unit(double x) { return x >= 0.0 && x < 1.0; }
bool sound(double x) { return x >= 0.0 && x < INFINITY; }

// How the kernel may take a tensor's chunks (AdamTensor::layout): in vectors of 8 elements if every buffer is
// as many elements past a vector boundary as the others (fp32 moments: the chunks then start that much early;
// 8-bit blocks start with the tensor, which has to be on a boundary).
uint32_t layout_of(const ra_adamw_tensor_t& t, const Sizes& z) {
  const auto past = [](const void* p, uint64_t es) { return (uint32_t)(reinterpret_cast<uintptr_t>(p) / es % 8); };
  const uint32_t shift = past(t.param, z.param);
  if (past(t.grad, z.grad) != shift || past(t.exp_avg, z.moment) != shift || past(t.exp_avg_sq, z.moment) != shift) return 0;
  if (t.copy != nullptr && past(t.copy, z.copy) != shift) return 0;
  if (z.s8 && shift != 0) return 0;
  return ra::kAdamVec | shift;
}

template <int CAP, class Fn>
ra_status_t launch_all(const ra_adamw_tensor_t* tensors, int ntensors, Fn fn, const ra_adamw_options_t& o, const Sizes& z,
                       ra::AdamScalars s, uint32_t key, cudaStream_t stream) {
  ra::AdamArgs<CAP> a;
  const uint64_t per_cta = (uint64_t)ra::kAdamThreads * ra::adam_lane_elems(z.s8);
  int i = 0;
  while (i < ntensors) {
    uint64_t ctas = 0;
    s.n = 0;
    for (; i < ntensors && s.n < CAP; ++i) {
      const ra_adamw_tensor_t& t = tensors[i];
      const uint32_t layout = t.count ? layout_of(t, z) : 0;
      const uint64_t more = (t.count + (layout & 7u) + per_cta - 1) / per_cta;
      if (ctas + more > 0x7fffffffull) {
        if (s.n == 0) return RA_ERR_UNSUPPORTED;
        break;
      }
      ra::AdamTensor& e = a.t[s.n];
      e.p = t.param, e.g = t.grad, e.m = t.exp_avg, e.v = t.exp_avg_sq;
      e.ms = t.exp_avg_scale, e.vs = t.exp_avg_sq_scale, e.copy = t.copy;
      e.count = t.count;
      e.keep = (float)(1.0 - o.lr * t.weight_decay);
      e.layout = layout;
      e.key = ra::mix32(key + (uint32_t)i * 0xB7E15163u);
      a.cta0[s.n++] = (uint32_t)ctas;
      ctas += more;
    }
    if (ctas == 0) continue;
    a.s = s;
    const cudaError_t err = fn(z.s8, a, (uint32_t)ctas, stream);
    if (err != cudaSuccess) return ra::cuda_failed(err);
  }
  return RA_SUCCESS;
}

}  // namespace

extern "C" ra_status_t ra_adamw(const ra_adamw_tensor_t* tensors, int ntensors, ra_dtype_t param_dtype,
                                ra_dtype_t grad_dtype, const ra_adamw_options_t* options, void* stream) {
  if (ntensors < 0 || (ntensors > 0 && tensors == nullptr) || options == nullptr) return RA_ERR_INVALID_ARG;
  const ra_adamw_options_t& o = *options;
  ra_status_t st = ra::check_float(param_dtype);
  if (st == RA_SUCCESS) st = ra::check_float(grad_dtype);
  if (st != RA_SUCCESS) return st;
  if (o.state != RA_STATE_F32 && o.state != RA_STATE_E4M3) return RA_ERR_INVALID_ARG;
  if (o.step < 1 || !unit(o.beta1) || !unit(o.beta2) || !sound(o.lr) || !sound(o.eps)) return RA_ERR_INVALID_ARG;
  // the kernel's reciprocal of a denormal is infinite, and an element without a gradient would become 0 * infinity
  if (o.eps > 0.0 && o.eps < 0x1p-126) return RA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(o.grad_scale) % 4) return RA_ERR_INVALID_ARG;
  Sizes z{(uint64_t)ra::float_size(param_dtype), (uint64_t)ra::float_size(grad_dtype), 4, 0, o.state == RA_STATE_E4M3};
  if (z.s8) z.moment = 1;
  bool any = false;
  for (int i = 0; i < ntensors; ++i) {
    const ra_adamw_tensor_t& t = tensors[i];
    if (t.count == 0) continue;
    any = true;
    if ((uint64_t)t.count > RA_MAX_COUNT || !sound(t.weight_decay)) return RA_ERR_INVALID_ARG;
    if (t.copy != nullptr && z.copy == 0) {
      st = ra::check_float(o.copy_dtype);
      if (st != RA_SUCCESS) return st;
      z.copy = (uint64_t)ra::float_size(o.copy_dtype);
    }
  }
  if (!any) return RA_SUCCESS;
  // Every buffer by itself, and whether the lists are runs of ascending, separate buffers that keep clear of each
  // other, as slices of flat buffers are: then nothing overlaps (292 tensors: a call of 14 us against 22 with the full check).
  Span extent[kLists + 1];
  int extents = 0;
  bool plain = true;
  for (int list = 0; list < kLists; ++list) {
    if (!list_used(list, z)) continue;
    const bool written = list != 1;
    Span e{UINTPTR_MAX, 0, written};
    for (int i = 0; i < ntensors; ++i) {
      if (tensors[i].count == 0) continue;
      uint64_t bytes;
      uintptr_t align;
      const uintptr_t lo = reinterpret_cast<uintptr_t>(buffer_of(tensors[i], list, z, &bytes, &align));
      if (lo == 0 && list == kLists - 1) continue;  // no copy of this one
      if (lo == 0 || lo % align || lo + bytes < lo) return RA_ERR_INVALID_ARG;
      if (written && lo < e.hi) plain = false;
      e.lo = std::min(e.lo, lo), e.hi = std::max(e.hi, lo + (uintptr_t)bytes);
    }
    extent[extents++] = e;
  }
  const uintptr_t scale = reinterpret_cast<uintptr_t>(o.grad_scale);
  if (scale) extent[extents++] = {scale, scale + 4, false};
  for (int i = 0; i < extents; ++i)
    for (int j = 0; j < i; ++j) plain = plain && (extent[i].hi <= extent[j].lo || extent[j].hi <= extent[i].lo);
  if (!plain) {
    try {
      std::vector<Span> spans;
      spans.reserve((size_t)ntensors * kLists + 1);
      for (int list = 0; list < kLists; ++list) {  // one list after another: each may still be an ascending run
        if (!list_used(list, z)) continue;
        for (int i = 0; i < ntensors; ++i) {
          uint64_t bytes;
          uintptr_t align;
          const uintptr_t lo = reinterpret_cast<uintptr_t>(buffer_of(tensors[i], list, z, &bytes, &align));
          if (tensors[i].count && lo) spans.push_back({lo, lo + (uintptr_t)bytes, list != 1});
        }
      }
      if (scale) spans.push_back({scale, scale + 4, false});
      if (written_overlap(spans)) return RA_ERR_ALIAS;
    } catch (const std::bad_alloc&) {
      return RA_ERR_UNSUPPORTED;  // the host has no room for the list
    }
  }
  ra::AdamScalars s{};
  s.b1 = (float)o.beta1, s.one_minus_b1 = (float)(1.0 - o.beta1);
  s.b2 = (float)o.beta2, s.one_minus_b2 = (float)(1.0 - o.beta2);
  s.inv_sqrt_bc2 = (float)(1.0 / sqrt(1.0 - pow(o.beta2, (double)o.step)));
  s.eps = (float)o.eps;
  s.step_size = (float)(o.lr / (1.0 - pow(o.beta1, (double)o.step)));
  s.one = 1.0f;
  const uint32_t key = ra::mix32((uint32_t)o.seed + ra::mix32((uint32_t)(o.seed >> 32) + (uint32_t)o.step * 0x9E3779B9u));
  s.copy_dtype = o.copy_dtype;
  s.scale = o.grad_scale;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  return ntensors <= ra::kAdamSmall
             ? launch_all<ra::kAdamSmall>(tensors, ntensors, ra::kAdamSmallFns[param_dtype][grad_dtype], o, z, s, key, cs)
             : launch_all<ra::kAdamLarge>(tensors, ntensors, ra::kAdamLargeFns[param_dtype][grad_dtype], o, z, s, key, cs);
}
