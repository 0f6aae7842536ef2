// C ABI of the training operators: argument validation and the AdamW table.  See include/flashkm_train.h for the
// contract.
#include <math.h>

#include <algorithm>
#include <new>
#include <vector>

#include "checks.h"

#include "flashkm_train.h"

using namespace fkm;

namespace {

static_assert(KM_ADAMW_BLOCK == kAdamBlock, "one block size");

int check_rows(int64_t N, int32_t K, int32_t S) {
  if (N < 0 || N >= kMax31) return fail(KM_EINVAL, "N=%lld must be 0 to 2^31 - 1", (long long)N);
  if (K < 1) return fail(KM_EINVAL, "K=%d must be >= 1", K);
  if (S < 1 || S > K) return fail(KM_EINVAL, "S=%d must be 1 to K=%d", S, K);
  if (S > KM_ROUTE_MAX_S) return fail(KM_EUNSUPPORTED, "unsupported S=%d (1 to %d)", S, KM_ROUTE_MAX_S);
  return KM_OK;
}
int check_score(int32_t score) {
  if (score != KM_SOFTMAX && score != KM_SIGMOID) return fail(KM_EUNSUPPORTED, "unsupported score %d", score);
  return KM_OK;
}

constexpr int64_t kMaxTensors = 1 << 20, kMaxNumel = (int64_t)1 << 40;

// Chunks of a table; -1 and the error text for invalid arguments.
int64_t count_chunks(const km_adamw_tensor* t, int32_t count) {
  if (count < 1 || count > kMaxTensors) {
    fail(KM_EINVAL, "count=%d must be 1 to %lld", count, (long long)kMaxTensors);
    return -1;
  }
  if (!t) {
    fail(KM_EINVAL, "tensors must be non-null");
    return -1;
  }
  int64_t chunks = 0;
  for (int32_t i = 0; i < count; ++i) {
    if (t[i].numel < 0 || t[i].numel >= kMaxNumel) {
      fail(KM_EINVAL, "tensor %d: numel=%lld must be 0 to 2^40 - 1", i, (long long)t[i].numel);
      return -1;
    }
    chunks += (t[i].numel + kAdamChunk - 1) / kAdamChunk;
  }
  if (chunks >= kMax31) {
    fail(KM_EINVAL, "too many elements: %lld chunks of %d", (long long)chunks, kAdamChunk);
    return -1;
  }
  return chunks;
}

// A range of memory that a step reads or writes.
struct Range {
  uintptr_t from, to;
  int32_t tensor;
  const char* name;
  bool out;
};

int check_tensors(const km_adamw_tensor* t, int32_t count, int pdt, int gdt, int bits) {
  const uint64_t psz = dtype_size(pdt), gsz = dtype_size(gdt);
  std::vector<Range> ranges;
  ranges.reserve((size_t)count * 7);
  const bool masters = t[0].master != nullptr;
  for (int32_t i = 0; i < count; ++i) {
    const km_adamw_tensor& x = t[i];
    if ((x.master != nullptr) != masters)
      return fail(KM_EINVAL, "tensor %d: a master copy for every tensor or for none", i);
    if (!(x.decay >= 0.f) || x.decay == INFINITY) return fail(KM_EINVAL, "tensor %d: decay must be finite and >= 0", i);
    const uint64_t n = (uint64_t)x.numel, scales = (n + kAdamBlock - 1) / kAdamBlock * 4;
    const Arr arrs[] = {{"param", x.param, n * psz, (unsigned)psz, true},
                        {"grad", x.grad, n * gsz, (unsigned)gsz, false},
                        {"master", x.master, masters ? n * 4 : 0, 4, true},
                        {"exp_avg", x.exp_avg, bits == 8 ? n : n * 4, bits == 8 ? 1u : 4u, true},
                        {"exp_avg_sq", x.exp_avg_sq, bits == 8 ? n : n * 4, bits == 8 ? 1u : 4u, true},
                        {"exp_avg_scale", x.exp_avg_scale, bits == 8 ? scales : 0, 4, true},
                        {"exp_avg_sq_scale", x.exp_avg_sq_scale, bits == 8 ? scales : 0, 4, true}};
    for (const Arr& a : arrs) {
      if (a.bytes && !a.p) return fail(KM_EINVAL, "tensor %d: %s must be non-null", i, a.name);
      if ((uintptr_t)a.p % a.align)
        return fail(KM_EINVAL, "tensor %d: misaligned pointer: %s needs %u bytes", i, a.name, a.align);
      if (a.bytes) ranges.push_back(Range{(uintptr_t)a.p, (uintptr_t)a.p + a.bytes, i, a.name, a.out});
    }
  }
  // in the order of their addresses a written range may meet no other; gradients may meet each other
  std::sort(ranges.begin(), ranges.end(), [](const Range& a, const Range& b) { return a.from < b.from; });
  const Range *any = nullptr, *out = nullptr;  // that reach furthest so far
  for (const Range& r : ranges) {
    const Range* hit = r.out ? any : out;
    if (hit && r.from < hit->to)
      return fail(KM_EINVAL, "%s of tensor %d overlaps %s of tensor %d", r.name, r.tensor, hit->name, hit->tensor);
    if (!any || r.to > any->to) any = &r;
    if (r.out && (!out || r.to > out->to)) out = &r;
  }
  return KM_OK;
}

int check_bits(int32_t bits) {
  if (bits != 32 && bits != 8) return fail(KM_EUNSUPPORTED, "unsupported bits=%d (32 or 8)", bits);
  return KM_OK;
}

}  // namespace

extern "C" {

int kmeans_route(const void* logits, int32_t dtype, int64_t N, int32_t K, const float* bias, int32_t score,
                 int32_t groups, int32_t top_groups, int32_t group_best, int32_t S, int32_t renormalise, float scale,
                 const uint8_t* valid, int32_t* ids, float* weights, float* chosen, void* stream) {
  err_buf()[0] = 0;
  if (int rc = check_type(dtype, "dtype")) return rc;
  if (int rc = check_score(score)) return rc;
  if (int rc = check_rows(N, K, S)) return rc;
  if (groups < 1 || K % groups) return fail(KM_EINVAL, "groups=%d must divide K=%d", groups, K);
  if (groups > KM_ROUTE_MAX_GROUPS)
    return fail(KM_EUNSUPPORTED, "unsupported groups=%d (1 to %d)", groups, KM_ROUTE_MAX_GROUPS);
  if (top_groups < 1 || top_groups > groups)
    return fail(KM_EINVAL, "top_groups=%d must be 1 to groups=%d", top_groups, groups);
  if (group_best != 1 && group_best != 2) return fail(KM_EINVAL, "group_best=%d must be 1 or 2", group_best);
  const uint64_t n = (uint64_t)N, sz = dtype_size(dtype);
  const Arr arrs[] = {{"logits", logits, n * K * sz, (unsigned)sz, false},
                      {"bias", bias, bias ? (uint64_t)K * 4 : 0, 4, false},
                      {"valid", valid, valid ? n : 0, 1, false},
                      {"ids", ids, n * S * 4, 4, true},
                      {"weights", weights, n * S * 4, 4, true},
                      {"chosen", chosen, n * S * 4, 4, true}};
  if (int rc = check_arrays(arrs)) return rc;
  if (n == 0) return KM_OK;
  // groups that all stay change nothing
  const bool grouped = top_groups < groups;
  const RouteCall c{logits,     N,         K,     bias, score == KM_SOFTMAX, grouped ? groups : 1, top_groups,
                    group_best, S,         renormalise != 0, scale, valid, ids, weights, chosen};
  KM_HIP(launch_route(dtype, c, (hipStream_t)stream), "route launch");
  return KM_OK;
}

int kmeans_route_grad(const void* logits, int32_t dtype, int64_t N, int32_t K, const int32_t* ids, const float* chosen,
                      const float* dweights, int32_t S, int32_t score, int32_t renormalise, float scale,
                      int32_t accumulate, void* dlogits, void* stream) {
  err_buf()[0] = 0;
  if (int rc = check_type(dtype, "dtype")) return rc;
  if (int rc = check_score(score)) return rc;
  if (int rc = check_rows(N, K, S)) return rc;
  const uint64_t n = (uint64_t)N, sz = dtype_size(dtype);
  const bool dense = score == KM_SOFTMAX && !renormalise;
  const Arr arrs[] = {{"logits", logits, dense ? n * K * sz : 0, dense ? (unsigned)sz : 1, false},
                      {"ids", ids, n * S * 4, 4, false},
                      {"chosen", chosen, dense ? 0 : n * S * 4, dense ? 1u : 4u, false},
                      {"dweights", dweights, n * S * 4, 4, false},
                      {"dlogits", dlogits, n * K * sz, (unsigned)sz, true}};
  if (int rc = check_arrays(arrs)) return rc;
  if (n == 0) return KM_OK;
  const RouteGradCall c{logits, N,     K,         ids, chosen, dweights, S, score == KM_SOFTMAX, renormalise != 0,
                        scale,  accumulate != 0, dlogits};
  KM_HIP(launch_route_grad(dtype, c, (hipStream_t)stream), "route gradient launch");
  return KM_OK;
}

int64_t kmeans_adamw_chunks(const km_adamw_tensor* tensors, int32_t count) {
  err_buf()[0] = 0;
  return count_chunks(tensors, count);
}

size_t kmeans_adamw_table_bytes(const km_adamw_tensor* tensors, int32_t count) {
  err_buf()[0] = 0;
  const int64_t chunks = count_chunks(tensors, count);
  return chunks < 0 ? 0 : al256(adam_map_at(count) + (size_t)chunks * 4);
}

int kmeans_adamw_table(const km_adamw_tensor* tensors, int32_t count, int32_t param_dtype, int32_t grad_dtype,
                       int32_t bits, void* table, size_t table_bytes) {
  err_buf()[0] = 0;
  try {
    if (int rc = check_type(param_dtype, "param dtype")) return rc;
    if (int rc = check_type(grad_dtype, "grad dtype")) return rc;
    if (int rc = check_bits(bits)) return rc;
    const int64_t chunks = count_chunks(tensors, count);
    if (chunks < 0) return KM_EINVAL;
    if (tensors[0].master && param_dtype == KM_F32)
      return fail(KM_EINVAL, "an fp32 parameter needs no master copy");
    if (int rc = check_tensors(tensors, count, param_dtype, grad_dtype, bits)) return rc;
    const size_t need = kmeans_adamw_table_bytes(tensors, count);
    if (!table) return fail(KM_EINVAL, "table must be non-null");
    if ((uintptr_t)table % alignof(AdamItem)) return fail(KM_EINVAL, "misaligned pointer: table");
    if (table_bytes < need) return fail(KM_EWORKSPACE, "table too small: %zu bytes given, %zu needed", table_bytes, need);
    auto* items = static_cast<AdamItem*>(table);
    auto* map = reinterpret_cast<int32_t*>(static_cast<char*>(table) + adam_map_at(count));
    // the alignment at which four elements of an array are moved at once
    auto four = [](const void* p, uint64_t size) { return (uintptr_t)p % (4 * size < 16 ? 4 * size : 16) == 0; };
    const uint64_t ssz = bits == 8 ? 1 : 4;
    int64_t first = 0;
    for (int32_t i = 0; i < count; ++i) {
      const km_adamw_tensor& t = tensors[i];
      const bool aligned = four(t.param, dtype_size(param_dtype)) && four(t.grad, dtype_size(grad_dtype)) &&
                           four(t.master, 4) && four(t.exp_avg, ssz) && four(t.exp_avg_sq, ssz);
      items[i] = AdamItem{t.param,          t.grad,  t.master, t.exp_avg, t.exp_avg_sq, t.exp_avg_scale,
                          t.exp_avg_sq_scale, t.numel, first,    t.decay,   aligned};
      const int64_t mine = (t.numel + kAdamChunk - 1) / kAdamChunk;
      for (int64_t c = 0; c < mine; ++c) map[first + c] = i;
      first += mine;
    }
    return KM_OK;
  } catch (const std::bad_alloc&) {
    return fail(KM_ENOMEM, "out of host memory");
  } catch (...) {
    return fail(KM_EINVAL, "unexpected exception");
  }
}

int kmeans_adamw(const void* table, int32_t count, int64_t chunks, int32_t param_dtype, int32_t grad_dtype,
                 int32_t bits, int32_t masters, double lr, double beta1, double beta2, double eps, double weight_decay,
                 int64_t step, const float* lr_at, const int64_t* step_at, const float* grad_scale_at,
                 const uint8_t* skip_at, void* stream) {
  err_buf()[0] = 0;
  if (int rc = check_type(param_dtype, "param dtype")) return rc;
  if (int rc = check_type(grad_dtype, "grad dtype")) return rc;
  const bool stochastic = bits == (8 | KM_ADAMW_STOCHASTIC);
  if (stochastic) bits = 8;
  if (int rc = check_bits(bits)) return rc;
  if (count < 1 || count > kMaxTensors) return fail(KM_EINVAL, "count=%d must be 1 to %lld", count, (long long)kMaxTensors);
  if (chunks < 0 || chunks >= kMax31) return fail(KM_EINVAL, "chunks=%lld must be 0 to 2^31 - 1", (long long)chunks);
  if (masters && param_dtype == KM_F32) return fail(KM_EINVAL, "an fp32 parameter needs no master copy");
  if (!(beta1 >= 0 && beta1 < 1)) return fail(KM_EINVAL, "beta1=%g must be in [0, 1)", beta1);
  if (!(beta2 >= 0 && beta2 < 1)) return fail(KM_EINVAL, "beta2=%g must be in [0, 1)", beta2);
  if (!(eps >= 0) || isinf(eps)) return fail(KM_EINVAL, "eps=%g must be finite and >= 0", eps);
  if (!lr_at && !isfinite(lr)) return fail(KM_EINVAL, "lr=%g must be finite", lr);
  if (!isfinite(weight_decay)) return fail(KM_EINVAL, "weight_decay=%g must be finite", weight_decay);
  if (!step_at && step < 1) return fail(KM_EINVAL, "step=%lld must be >= 1", (long long)step);
  if (!table) return fail(KM_EINVAL, "table must be non-null");
  if ((uintptr_t)table & 255) return fail(KM_EINVAL, "table must be 256-byte aligned");
  if ((uintptr_t)lr_at % 4) return fail(KM_EINVAL, "misaligned pointer: lr_at needs 4 bytes");
  if ((uintptr_t)step_at % 8) return fail(KM_EINVAL, "misaligned pointer: step_at needs 8 bytes");
  if ((uintptr_t)grad_scale_at % 4) return fail(KM_EINVAL, "misaligned pointer: grad_scale_at needs 4 bytes");
  if (chunks == 0) return KM_OK;
  const AdamCall c{table, count, chunks, bits,  masters != 0, lr,      beta1,         beta2,
                   eps,   weight_decay,  step,  lr_at, step_at, grad_scale_at, skip_at, stochastic};
  KM_HIP(launch_adamw(param_dtype, grad_dtype, c, (hipStream_t)stream), "adamw launch");
  return KM_OK;
}

}  // extern "C"
