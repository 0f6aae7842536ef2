// Balance loss of the use of K choices by N rows, with counts, and its
// gradient (formulas in flashkm_codebook.h).
//
// Exponentials are taken of differences from the row's maximum, formed before the scaling by log2(e), so logits of the
// type's lowest value stay finite differences.
#include "kernels.h"
#include "vecio.h"

namespace fkm {

namespace {

__device__ __forceinline__ float wave_max_f32(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}

// lse of every row (+inf for an invalid one) and its (maximum, 1 / sum of
// exponentials), (0, 0) for a row that leaves no probability: the
// probabilities come from these, since a large lse has lost the sum's low
// bits.  One wave per row.
template <class T>
__global__ __launch_bounds__(256) void balance_lse_kernel(const typename T::raw* __restrict__ logits, int64_t n, int K,
                                                          const uint8_t* __restrict__ valid, float* __restrict__ lse,
                                                          float2* __restrict__ ms) {
  const int lane = lane_id();
  for (int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); i < n; i += (int64_t)gridDim.x * 4) {
    if (valid && !valid[i]) {
      if (lane == 0) lse[i] = INFINITY, ms[i] = make_float2(0.f, 0.f);
      continue;
    }
    const typename T::raw* row = logits + i * K;
    float m = -INFINITY;
    bool nan = false;
    for (int k = lane; k < K; k += 64) {
      const float f = T::to_f32(row[k]);
      nan |= f != f;
      m = fmaxf(m, f);
    }
    m = wave_max_f32(m);
    float sum = 0.f;
    if (m > -INFINITY)
      for (int k = lane; k < K; k += 64) sum += expf(T::to_f32(row[k]) - m);
    sum = wave_sum_f32(sum);
    if (__ballot(nan)) sum = NAN;
    const bool none = m == -INFINITY && sum == 0.f;
    if (lane == 0) {
      lse[i] = none ? -INFINITY : m + logf(sum);
      ms[i] = none ? make_float2(0.f, 0.f) : make_float2(m, 1.f / sum);
    }
  }
}

// part[b, chunk, k] = fp64 sum of p[b, i, k] over the chunk's valid rows; one
// thread per column.
template <class T>
__global__ __launch_bounds__(256) void balance_cols_kernel(const typename T::raw* __restrict__ logits, int64_t N,
                                                           int K, int64_t chunks, int kblocks, int64_t units,
                                                           const float2* __restrict__ ms, double* __restrict__ part) {
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t bc = u / kblocks;
    const int k = (int)(u - bc * kblocks) * 256 + threadIdx.x;
    if (k >= K) continue;
    const int64_t b = bc / chunks, c = bc - b * chunks;
    const int64_t i0 = c * kBalanceRows, i1 = i0 + kBalanceRows < N ? i0 + kBalanceRows : N;
    double sum = 0.0;
    for (int64_t i = i0; i < i1; ++i) {
      const float2 z = ms[b * N + i];
      if (z.y == 0.f) continue;
      sum += (double)(expf(T::to_f32(logits[(b * N + i) * K + k]) - z.x) * z.y);
    }
    part[bc * K + k] = sum;
  }
}

__global__ __launch_bounds__(256) void balance_zero_kernel(int32_t* __restrict__ counts, int64_t entries,
                                                           int32_t* __restrict__ nvalid, int B) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < entries; i += (int64_t)gridDim.x * 256) {
    counts[i] = 0;
    if (i < B) nvalid[i] = 0;
  }
}

// Integer counts by atomics: exact, whatever their order.
__global__ __launch_bounds__(256) void balance_count_kernel(const int32_t* __restrict__ labels, int64_t n, uint32_t N,
                                                            uint32_t K, int S, const uint8_t* __restrict__ valid,
                                                            int32_t* __restrict__ counts,
                                                            int32_t* __restrict__ nvalid) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    if (valid && !valid[i]) continue;
    const int64_t b = (uint32_t)i / N;
    atomicAdd(&nvalid[b], 1);
    for (int s = 0; s < S; ++s) {
      const uint32_t l = (uint32_t)labels[i * S + s];
      if (l < K) atomicAdd(&counts[b * K + l], 1);
    }
  }
}

// One workgroup per instance: prob, coef and the loss.
__global__ __launch_bounds__(256) void balance_finish_kernel(const double* __restrict__ part, int64_t chunks, int K,
                                                             int S, const int32_t* __restrict__ counts,
                                                             const int32_t* __restrict__ nvalid,
                                                             float* __restrict__ loss, float* __restrict__ prob,
                                                             float* __restrict__ coef) {
  __shared__ double tmp[4];
  const int64_t b = blockIdx.x;
  const double T = nvalid[b];
  const double per = T > 0 ? 1.0 / T : 0.0;
  double sum = 0.0;
  for (int k = threadIdx.x; k < K; k += 256) {
    double p = 0.0;
    for (int64_t c = 0; c < chunks; ++c) p += part[(b * chunks + c) * K + k];
    p *= per;
    const double share = (double)counts[b * K + k] * ((double)K / S) * per;
    prob[b * K + k] = (float)p;
    coef[b * K + k] = (float)(share * per);
    sum += share * p;
  }
  sum = wave_sum_f64(sum);
  if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) loss[b] = (float)(((tmp[0] + tmp[1]) + tmp[2]) + tmp[3]);
}

template <class T>
__global__ __launch_bounds__(256) void balance_grad_kernel(const typename T::raw* __restrict__ logits, int64_t n,
                                                           uint32_t N, int K, const float* __restrict__ lse,
                                                           const float* __restrict__ coef,
                                                           const float* __restrict__ dloss,
                                                           typename T::raw* __restrict__ dlogits) {
  const int lane = lane_id();
  for (int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); i < n; i += (int64_t)gridDim.x * 4) {
    const int64_t b = (uint32_t)i / N;
    const float z = lse[i];
    const bool none = z == INFINITY || z == -INFINITY;
    const float* cf = coef + b * K;
    // the row's maximum and sum again: an lse of large magnitude does not hold
    // the sum's logarithm
    float m = -INFINITY, sum = 0.f, dot = 0.f;
    if (!none) {
      for (int k = lane; k < K; k += 64) m = fmaxf(m, T::to_f32(logits[i * K + k]));
      m = wave_max_f32(m);
      for (int k = lane; k < K; k += 64) {
        const float e = expf(T::to_f32(logits[i * K + k]) - m);
        sum += e;
        dot = fmaf(e, cf[k], dot);
      }
    }
    sum = wave_sum_f32(sum);
    dot = wave_sum_f32(dot) / sum;
    const float w = dloss[b] / sum;
    for (int k = lane; k < K; k += 64)
      dlogits[i * K + k] =
          round_to<T>(none ? 0.f : w * expf(T::to_f32(logits[i * K + k]) - m) * (cf[k] - dot));
  }
}

int64_t capped(int64_t blocks) { return blocks < 1 ? 1 : blocks < (1 << 22) ? blocks : (1 << 22); }

template <class T>
hipError_t balance_t(const void* logits, int64_t N, int K, int B, const int32_t* labels, int S, const uint8_t* valid,
                     float* loss, int32_t* counts, float* prob, float* lse, float* coef, const BalanceBuffers& buf,
                     hipStream_t s) {
  const int64_t n = N * B;
  const auto* x = static_cast<const typename T::raw*>(logits);
  const int64_t entries = (int64_t)B * K;
  balance_zero_kernel<<<dim3((unsigned)capped((entries + 255) / 256)), dim3(256), 0, s>>>(counts, entries, buf.nvalid,
                                                                                           B);
  if (n) {
    balance_lse_kernel<T><<<dim3((unsigned)capped((n + 3) / 4)), dim3(256), 0, s>>>(x, n, K, valid, lse, buf.ms);
    balance_count_kernel<<<dim3((unsigned)capped((n + 255) / 256)), dim3(256), 0, s>>>(labels, n, (uint32_t)N,
                                                                                        (uint32_t)K, S, valid, counts,
                                                                                        buf.nvalid);
  }
  const int64_t chunks = balance_chunks(N);
  const int kblocks = (K + 255) / 256;
  const int64_t units = B * chunks * kblocks;
  balance_cols_kernel<T><<<dim3((unsigned)capped(units)), dim3(256), 0, s>>>(x, N, K, chunks, kblocks, units, buf.ms,
                                                                              buf.part);
  balance_finish_kernel<<<dim3((unsigned)B), dim3(256), 0, s>>>(buf.part, chunks, K, S, counts, buf.nvalid, loss, prob,
                                                                coef);
  return hipGetLastError();
}

template <class T>
hipError_t balance_grad_t(const void* logits, int64_t N, int K, int B, const float* lse, const float* coef,
                          const float* dloss, void* dlogits, hipStream_t s) {
  const int64_t n = N * B;
  balance_grad_kernel<T><<<dim3((unsigned)capped((n + 3) / 4)), dim3(256), 0, s>>>(
      static_cast<const typename T::raw*>(logits), n, (uint32_t)N, K, lse, coef, dloss,
      static_cast<typename T::raw*>(dlogits));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_balance(int dt, const void* logits, int64_t N, int K, int B, const int32_t* labels, int S,
                          const uint8_t* valid, float* loss, int32_t* counts, float* prob, float* lse, float* coef,
                          const BalanceBuffers& buf, hipStream_t s) {
  switch (dt) {
    case DT_F32: return balance_t<F32>(logits, N, K, B, labels, S, valid, loss, counts, prob, lse, coef, buf, s);
    case DT_F16: return balance_t<F16>(logits, N, K, B, labels, S, valid, loss, counts, prob, lse, coef, buf, s);
    case DT_BF16: return balance_t<BF16>(logits, N, K, B, labels, S, valid, loss, counts, prob, lse, coef, buf, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_balance_grad(int dt, const void* logits, int64_t N, int K, int B, const float* lse,
                               const float* coef, const float* dloss, void* dlogits, hipStream_t s) {
  switch (dt) {
    case DT_F32: return balance_grad_t<F32>(logits, N, K, B, lse, coef, dloss, dlogits, s);
    case DT_F16: return balance_grad_t<F16>(logits, N, K, B, lse, coef, dloss, dlogits, s);
    case DT_BF16: return balance_grad_t<BF16>(logits, N, K, B, lse, coef, dloss, dlogits, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace fkm
