// C ABI of the codebook operators: argument validation and workspace
// carve-up.  See include/flashkm_codebook.h for the contract.
#include "kernels.h"
#include "workspace.h"

#include "flashkm_codebook.h"

using namespace fkm;

namespace {

int hip_fail(hipError_t e, const char* what) { return fail(KM_EHIP, "%s: %s", what, hipGetErrorString(e)); }

#define KM_HIP(expr, what)                           \
  do {                                               \
    hipError_t e_ = (expr);                          \
    if (e_ != hipSuccess) return hip_fail(e_, what); \
  } while (0)

constexpr int32_t kMaxD = 1 << 20;
constexpr int64_t kMax31 = (int64_t)1 << 31;

bool known_type(int dt) { return dt == KM_F32 || dt == KM_F16 || dt == KM_BF16; }

int check_sizes(int64_t N, int32_t K, int32_t B) {
  if (B < 1) return fail(KM_EINVAL, "B=%d must be >= 1", B);
  if (K < 1) return fail(KM_EINVAL, "K=%d must be >= 1", K);
  if (N < 0) return fail(KM_EINVAL, "N=%lld must be >= 0", (long long)N);
  if (N >= kMax31 || N * B >= kMax31) return fail(KM_EINVAL, "B*N must be < 2^31");
  if ((int64_t)B * K >= kMax31) return fail(KM_EINVAL, "B*K must be < 2^31");
  return KM_OK;
}

int check_d(int32_t D) {
  if (D < 1 || D > kMaxD) return fail(KM_EUNSUPPORTED, "unsupported D=%d (1 to %d)", D, kMaxD);
  return KM_OK;
}

int check_type(int dt, const char* name) {
  if (!known_type(dt)) return fail(KM_EUNSUPPORTED, "unsupported %s %d", name, dt);
  return KM_OK;
}

// One array of a call: its name, address, bytes and element size.
struct Arr {
  const char* name;
  const void* p;
  uint64_t bytes;
  unsigned align;
  bool out;
};

// Present and aligned where it has elements; no output overlaps another array.
template <int M>
int check_arrays(const Arr (&a)[M]) {
  for (const Arr& x : a) {
    if (x.bytes && !x.p) return fail(KM_EINVAL, "%s must be non-null", x.name);
    if ((uintptr_t)x.p % x.align) return fail(KM_EINVAL, "misaligned pointer: %s needs %u bytes", x.name, x.align);
  }
  for (int i = 0; i < M; ++i)
    for (int j = 0; j < M; ++j) {
      if (i == j || !a[i].out || !a[i].bytes || !a[j].bytes) continue;
      const uint64_t p = (uintptr_t)a[i].p, q = (uintptr_t)a[j].p;
      if (p < q + a[j].bytes && q < p + a[i].bytes) return fail(KM_EINVAL, "%s overlaps %s", a[i].name, a[j].name);
    }
  return KM_OK;
}

// The smallest workspace size: what a shape without need of one is given.
constexpr size_t kNoWorkspace = 256;

int check_workspace(const void* ws, size_t ws_bytes, size_t need) {
  if (need == kNoWorkspace) return KM_OK;
  if (ws_bytes < need) return fail(KM_EWORKSPACE, "workspace too small: %zu bytes given, %zu needed", ws_bytes, need);
  if (!ws) return fail(KM_EINVAL, "workspace pointer is null");
  if (((uintptr_t)ws & 255) != 0) return fail(KM_EINVAL, "workspace must be 256-byte aligned");
  return KM_OK;
}

// ---- workspaces --------------------------------------------------------------
struct GradLayout {
  size_t kv0, kv1, hist, dtot, frag[3], any[3], total;
};
GradLayout grad_layout(int64_t N, int K, int D, int B) {
  GradLayout L{};
  const int64_t n = N * B;
  if (n <= kGradDirect) {
    L.total = kNoWorkspace;
    return L;
  }
  size_t o = kNoWorkspace;
  L.kv0 = o;   o = al256(o + (size_t)(n + kSlack) * 8);
  L.kv1 = o;   o = al256(o + (size_t)(n + kSlack) * 8);
  L.hist = o;  o = al256(o + (size_t)sort_hist_words(N, B, K) * 4);
  L.dtot = o;  o = al256(o + ((size_t)1 << kSortWideBits) * 4);
  for (int i = 0; i < 3; ++i) {
    const size_t units = (size_t)grad_units(n, D, i);
    L.frag[i] = o;  o = al256(o + units * 2 * ((D + 3) / 4 * 4) * 4);
    L.any[i] = o;   o = al256(o + units * 2 * 4);
  }
  L.total = o;
  return L;
}

struct BalanceLayout {
  size_t part, cpart, vpart, terms, ms, total;
};
BalanceLayout balance_layout(int64_t N, int K, int B) {
  BalanceLayout L{};
  const bool wide = K > kBalanceMaxK;
  const int64_t chunks = wide ? balance_wide_chunks(N) : balance_split(N, B, K).chunks;
  const size_t cells = wide || chunks > 1 ? (size_t)B * chunks * K : 0;  // one chunk is finished where it is summed
  if (!cells) {
    L.total = kNoWorkspace;
    return L;
  }
  size_t o = kNoWorkspace;
  L.part = o;   o = al256(o + cells * 4);
  L.cpart = o;  o = al256(o + (wide ? 0 : cells * 4));
  L.vpart = o;  o = al256(o + (wide ? (size_t)B : (size_t)B * chunks) * 4);
  L.terms = o;  o = al256(o + (size_t)B * (((size_t)K + kBalanceJoinCols - 1) / kBalanceJoinCols) * 8);
  L.ms = o;     o = al256(o + (wide ? (size_t)B * N * 8 : 0));
  L.total = o;
  return L;
}

int check_grad_shape(int64_t N, int32_t K, int32_t D, int32_t B) {
  if (int rc = check_sizes(N, K, B)) return rc;
  return check_d(D);
}

// A workgroup per instance at least, and a launch's threads are counted in 32 bits.
int check_balance_sizes(int64_t N, int32_t K, int32_t B) {
  if (int rc = check_sizes(N, K, B)) return rc;
  if (B > (1 << 22)) return fail(KM_EINVAL, "B=%d must be <= %d", B, 1 << 22);
  return KM_OK;
}
int check_balance_shape(int64_t N, int32_t K, int32_t B, int32_t S) {
  if (int rc = check_balance_sizes(N, K, B)) return rc;
  if (S < 1) return fail(KM_EINVAL, "S=%d must be >= 1", S);
  if (N * B * (int64_t)S >= kMax31) return fail(KM_EINVAL, "B*N*S must be < 2^31");
  return KM_OK;
}

}  // namespace

extern "C" {

int kmeans_embed(const void* table, int32_t table_dtype, int64_t N, int32_t K, int32_t D, int32_t B,
                 const int32_t* ids, float scale, void* out, int32_t out_dtype, void* stream) {
  err_buf()[0] = 0;
  if (int rc = check_type(table_dtype, "table dtype")) return rc;
  if (int rc = check_type(out_dtype, "out dtype")) return rc;
  if (int rc = check_sizes(N, K, B)) return rc;
  if (int rc = check_d(D)) return rc;
  const uint64_t n = (uint64_t)N * B, tsz = dtype_size(table_dtype), osz = dtype_size(out_dtype);
  const Arr arrs[] = {{"table", table, (uint64_t)B * K * D * tsz, (unsigned)tsz, false},
                      {"ids", ids, n * 4, 4, false},
                      {"out", out, n * D * osz, (unsigned)osz, true}};
  if (int rc = check_arrays(arrs)) return rc;
  if (n == 0) return KM_OK;
  KM_HIP(launch_embed(table_dtype, out_dtype, table, ids, N, K, D, B, scale, out, (hipStream_t)stream),
         "embed launch");
  return KM_OK;
}

size_t kmeans_embed_grad_workspace_bytes(int64_t N, int32_t K, int32_t D, int32_t B) {
  if (check_grad_shape(N, K, D, B) != KM_OK) return 0;
  return grad_layout(N, K, D, B).total;
}

int kmeans_embed_grad(const void* dout, int32_t dout_dtype, int64_t N, int32_t K, int32_t D, int32_t B,
                      const int32_t* ids, float scale, int32_t accumulate, void* grad, int32_t grad_dtype, void* ws,
                      size_t ws_bytes, void* stream) {
  err_buf()[0] = 0;
  if (int rc = check_type(dout_dtype, "dout dtype")) return rc;
  if (int rc = check_type(grad_dtype, "grad dtype")) return rc;
  if (int rc = check_grad_shape(N, K, D, B)) return rc;
  const GradLayout L = grad_layout(N, K, D, B);
  if (int rc = check_workspace(ws, ws_bytes, L.total)) return rc;
  const uint64_t n = (uint64_t)N * B, isz = dtype_size(dout_dtype), gsz = dtype_size(grad_dtype);
  const Arr arrs[] = {{"dout", dout, n * D * isz, (unsigned)isz, false},
                      {"ids", ids, n * 4, 4, false},
                      {"grad", grad, (uint64_t)B * K * D * gsz, (unsigned)gsz, true},
                      {"workspace", ws, L.total == kNoWorkspace ? 0 : L.total, 1, true}};
  if (int rc = check_arrays(arrs)) return rc;
  if (n == 0 && accumulate) return KM_OK;
  char* base = static_cast<char*>(ws);
  hipStream_t s = (hipStream_t)stream;
  GradBuffers buf{};
  buf.sort.kv[0] = reinterpret_cast<uint2*>(base + L.kv0);
  buf.sort.kv[1] = reinterpret_cast<uint2*>(base + L.kv1);
  buf.sort.hist = reinterpret_cast<uint32_t*>(base + L.hist);
  buf.sort.hist_words = (int64_t)((L.dtot - L.hist) / 4);
  buf.sort.dtot = reinterpret_cast<uint32_t*>(base + L.dtot);
  for (int i = 0; i < 3; ++i) {
    buf.frag[i] = reinterpret_cast<float*>(base + L.frag[i]);
    buf.any[i] = reinterpret_cast<uint32_t*>(base + L.any[i]);
  }
  KM_HIP(launch_embed_grad(dout_dtype, grad_dtype, dout, ids, N, K, D, B, scale, accumulate != 0, grad, buf, s),
         "embed gradient launch");
  return KM_OK;
}

size_t kmeans_balance_workspace_bytes(int64_t N, int32_t K, int32_t B, int32_t S) {
  if (check_balance_shape(N, K, B, S) != KM_OK) return 0;
  return balance_layout(N, K, B).total;
}

int kmeans_balance(const void* logits, int32_t dtype, int64_t N, int32_t K, int32_t B, const int32_t* labels,
                   int32_t S, const uint8_t* valid, float* loss, int32_t* counts, float* prob, float* lse, float* coef,
                   void* ws, size_t ws_bytes, void* stream) {
  err_buf()[0] = 0;
  if (int rc = check_type(dtype, "dtype")) return rc;
  if (int rc = check_balance_shape(N, K, B, S)) return rc;
  const BalanceLayout L = balance_layout(N, K, B);
  if (int rc = check_workspace(ws, ws_bytes, L.total)) return rc;
  const uint64_t n = (uint64_t)N * B, e = (uint64_t)B * K, sz = dtype_size(dtype);
  const Arr arrs[] = {{"logits", logits, n * K * sz, (unsigned)sz, false},
                      {"labels", labels, n * S * 4, 4, false},
                      {"valid", valid, valid ? n : 0, 1, false},
                      {"loss", loss, (uint64_t)B * 4, 4, true},
                      {"counts", counts, e * 4, 4, true},
                      {"prob", prob, e * 4, 4, true},
                      {"lse", lse, n * 4, 4, true},
                      {"coef", coef, e * 4, 4, true},
                      {"workspace", ws, L.total == kNoWorkspace ? 0 : L.total, 1, true}};
  if (int rc = check_arrays(arrs)) return rc;
  char* base = static_cast<char*>(ws);
  BalanceBuffers buf{};
  buf.part = reinterpret_cast<float*>(base + L.part);
  buf.cpart = reinterpret_cast<int32_t*>(base + L.cpart);
  buf.vpart = reinterpret_cast<int32_t*>(base + L.vpart);
  buf.terms = reinterpret_cast<double*>(base + L.terms);
  buf.ms = reinterpret_cast<float2*>(base + L.ms);
  KM_HIP(launch_balance(dtype, logits, N, K, B, labels, S, valid, loss, counts, prob, lse, coef, buf,
                        (hipStream_t)stream),
         "balance launch");
  return KM_OK;
}

int kmeans_balance_grad(const void* logits, int32_t dtype, int64_t N, int32_t K, int32_t B, const float* lse,
                        const float* coef, const float* dloss, void* dlogits, void* stream) {
  err_buf()[0] = 0;
  if (int rc = check_type(dtype, "dtype")) return rc;
  if (int rc = check_balance_sizes(N, K, B)) return rc;
  const uint64_t n = (uint64_t)N * B, e = (uint64_t)B * K, sz = dtype_size(dtype);
  const Arr arrs[] = {{"logits", logits, n * K * sz, (unsigned)sz, false},
                      {"lse", lse, n * 4, 4, false},
                      {"coef", coef, e * 4, 4, false},
                      {"dloss", dloss, (uint64_t)B * 4, 4, false},
                      {"dlogits", dlogits, n * K * sz, (unsigned)sz, true}};
  if (int rc = check_arrays(arrs)) return rc;
  if (n == 0) return KM_OK;
  KM_HIP(launch_balance_grad(dtype, logits, N, K, B, lse, coef, dloss, dlogits, (hipStream_t)stream),
         "balance gradient launch");
  return KM_OK;
}

}  // extern "C"
