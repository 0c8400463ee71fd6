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

ra_status_t add_span(std::vector<Span>& v, const void* p, uint64_t bytes, uintptr_t align, bool written) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  if (lo == 0 || lo % align || lo + bytes < lo) return RA_ERR_INVALID_ARG;
  v.push_back({lo, lo + (uintptr_t)bytes, written});
  return RA_SUCCESS;
}

bool unit(double x) { return x >= 0.0 && x < 1.0; }
bool sound(double x) { return x >= 0.0 && x < INFINITY; }

// How the kernel may take a tensor's chunks (AdamTensor::layout): in vectors of 8 elements if every buffer is
// as many elements past a vector boundary as the others (fp32 moments: the chunks then start that much early;
// 8-bit blocks start with the tensor, which has to be on a boundary).
uint32_t layout_of(const ra_adamw_tensor_t& t, uint64_t pe, uint64_t ge, uint64_t se, uint64_t ce) {
  const auto past = [](const void* p, uint64_t es) { return (uint32_t)(reinterpret_cast<uintptr_t>(p) / es % 8); };
  const uint32_t shift = past(t.param, pe);
  if (past(t.grad, ge) != shift || past(t.exp_avg, se) != shift || past(t.exp_avg_sq, se) != shift) return 0;
  if (t.copy != nullptr && past(t.copy, ce) != shift) return 0;
  if (se == 1 && shift != 0) return 0;
  return ra::kAdamVec | shift;
}

template <int CAP, class Fn>
ra_status_t launch_all(const ra_adamw_tensor_t* tensors, int ntensors, Fn fn, const ra_adamw_options_t& o, uint64_t pe,
                       uint64_t ge, uint64_t ce, ra::AdamScalars s, uint32_t key, cudaStream_t stream) {
  ra::AdamArgs<CAP> a;
  const uint64_t per_cta = (uint64_t)ra::kAdamThreads * ra::adam_lane_elems(o.state == RA_STATE_E4M3);
  int i = 0;
  while (i < ntensors) {
    uint64_t ctas = 0;
    s.n = 0;
    for (; i < ntensors && s.n < CAP; ++i) {
      const ra_adamw_tensor_t& t = tensors[i];
      const uint32_t layout = t.count ? layout_of(t, pe, ge, o.state == RA_STATE_E4M3 ? 1 : 4, ce) : 0;
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
    const cudaError_t err = fn(o.state == RA_STATE_E4M3, a, (uint32_t)ctas, stream);
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
  if (reinterpret_cast<uintptr_t>(o.grad_scale) % 4) return RA_ERR_INVALID_ARG;
  const bool s8 = o.state == RA_STATE_E4M3;
  const uint64_t pe = (uint64_t)ra::float_size(param_dtype), ge = (uint64_t)ra::float_size(grad_dtype);
  const uint64_t se = s8 ? 1 : 4;
  uint64_t ce = 0;
  try {
    std::vector<Span> spans;
    spans.reserve((size_t)ntensors * 7 + 1);
    // one list after another: each is often an ascending run
    for (int list = 0; list < 7; ++list) {
      for (int i = 0; i < ntensors; ++i) {
        const ra_adamw_tensor_t& t = tensors[i];
        if (t.count == 0) continue;
        if ((uint64_t)t.count > RA_MAX_COUNT || !sound(t.weight_decay)) return RA_ERR_INVALID_ARG;
        const uint64_t scales = 4 * ((t.count + RA_ADAMW_BLOCK - 1) / RA_ADAMW_BLOCK);
        switch (list) {
          case 0: st = add_span(spans, t.param, t.count * pe, pe, true); break;
          case 1: st = add_span(spans, t.grad, t.count * ge, ge, false); break;
          case 2: st = add_span(spans, t.exp_avg, t.count * se, se, true); break;
          case 3: st = add_span(spans, t.exp_avg_sq, t.count * se, se, true); break;
          case 4: if (s8) st = add_span(spans, t.exp_avg_scale, scales, 4, true); break;
          case 5: if (s8) st = add_span(spans, t.exp_avg_sq_scale, scales, 4, true); break;
          default:
            if (t.copy == nullptr) break;
            if (ce == 0) {
              st = ra::check_float(o.copy_dtype);
              if (st != RA_SUCCESS) return st;
              ce = (uint64_t)ra::float_size(o.copy_dtype);
            }
            st = add_span(spans, t.copy, t.count * ce, ce, true);
        }
        if (st != RA_SUCCESS) return st;
      }
    }
    if (spans.empty()) return RA_SUCCESS;
    if (o.grad_scale != nullptr) {
      const uintptr_t p = reinterpret_cast<uintptr_t>(o.grad_scale);
      spans.push_back({p, p + 4, false});
    }
    if (written_overlap(spans)) return RA_ERR_ALIAS;
  } catch (const std::bad_alloc&) {
    return RA_ERR_UNSUPPORTED;  // the host has no room for the list
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
             ? launch_all<ra::kAdamSmall>(tensors, ntensors, ra::kAdamSmallFns[param_dtype][grad_dtype], o, pe, ge, ce, s, key, cs)
             : launch_all<ra::kAdamLarge>(tensors, ntensors, ra::kAdamLargeFns[param_dtype][grad_dtype], o, pe, ge, ce, s, key, cs);
}
