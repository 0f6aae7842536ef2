// AdamW step over the tensors of a table (formulas in flashkm_train.h).
//
// Bound by bytes: a value's parameter, gradient and two states are read once and all but the gradient written once (28
// bytes with fp32 everywhere; 16 1/16 with bf16 parameters and gradients, fp32 copies and states in 8 bits; parameters
// that have copies are not read).  A workgroup takes a chunk of 4,096 values of one tensor, a lane four neighbours at a
// time, so every access is up to 16 bytes a lane and a wave's four times 64 values are one block of a scale: its largest
// magnitude is a reduction over the wave's lanes.  Measured: 8.4 million fp32 values 40 us (5.9 TB/s), 124 million bf16
// values with copies 610 (5.7), 350 million with states in 8 bits 993 (5.7; a copy of 4 GiB moves 4.7).  With 8 bits the
// vector units are busy four fifths of that time: a third of the instructions are the codes and their scales; rounded
// stochastically (a hash for four values, three products, a conversion a code instead of one for two) 1.5 % more time.
#include <type_traits>

#include "kernels.h"
#include "teams.h"
#include "vecio.h"

namespace fkm {

namespace {

// What a step's values share.
struct Rates {
  float b1, c1, b2, c2;  // the betas and 1 - beta
  float eps, lr_wd, rate, root;  // lr * weight_decay, lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
  uint32_t key;                  // of the step's random words
};
struct Live {  // what is read on the device, where it is there
  const float* lr;
  const int64_t* step;
  const float* gscale;
  const uint8_t* skip;
  double lr_, b1, b2, wd;
  int64_t step_;
};

__host__ __device__ inline void set_step(Rates& r, double lr, double b1, double b2, double wd, int64_t step) {
  uint64_t x = (uint64_t)step * 0x9E3779B97F4A7C15ull;
  x = (x ^ x >> 32) * 0xD6E8FEB86659FD93ull;
  x = (x ^ x >> 32) * 0xA0761D6478BD642Full;
  r.key = (uint32_t)(x ^ x >> 32);
  r.lr_wd = (float)(lr * wd);
  r.rate = (float)(lr / (1.0 - pow(b1, (double)step)));
  r.root = (float)(1.0 / sqrt(1.0 - pow(b2, (double)step)));
}

// A state's value in 8 bits: a format's conversions, its code for a block's largest magnitude (a power of two), and the
// least code of a positive value.
// Rounded to nearest, or stochastically: the conversion adds the random word's 20 (e4m3) or 21 (e5m2) upper bits to the
// bits that it drops, those of subnormal codes among them.  18 and 19 of these are random and a one follows: the
// expectation is the value itself to 2^-19 of a step, and a block's largest, which scaling may leave one unit of fp32
// beside its code, is neither carried past it nor dropped below it.
struct E4M3 {
  static constexpr float kTop = 256.f, kLeast = 0.f;
  __device__ static uint32_t pack(const float (&y)[4]) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], w, true);
  }
  __device__ static uint32_t pack(const float (&y)[4], const uint32_t (&random)[4]) {
    uint32_t r[4];  // (the random bits' other end, so that m's errors are not v's)
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = ((random[e] >> 16 | random[e] << 16) & 0xFFFFC000u) | 0x2000u;
    int w = __builtin_amdgcn_cvt_sr_fp8_f32(y[0], r[0], 0, 0);
    w = __builtin_amdgcn_cvt_sr_fp8_f32(y[1], r[1], w, 1);
    w = __builtin_amdgcn_cvt_sr_fp8_f32(y[2], r[2], w, 2);
    return (uint32_t)__builtin_amdgcn_cvt_sr_fp8_f32(y[3], r[3], w, 3);
  }
  __device__ static void unpack(uint32_t w, float (&y)[4]) {
    const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    y[0] = a[0], y[1] = a[1], y[2] = b[0], y[3] = b[1];
  }
};
struct E5M2 {
  static constexpr float kTop = 32768.f, kLeast = 0x1p-16f;
  __device__ static uint32_t pack(const float (&y)[4]) {
    int w = __builtin_amdgcn_cvt_pk_bf8_f32(y[0], y[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_bf8_f32(y[2], y[3], w, true);
  }
  __device__ static uint32_t pack(const float (&y)[4], const uint32_t (&random)[4]) {
    uint32_t r[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = (random[e] & 0xFFFFE000u) | 0x1000u;
    int w = __builtin_amdgcn_cvt_sr_bf8_f32(y[0], r[0], 0, 0);
    w = __builtin_amdgcn_cvt_sr_bf8_f32(y[1], r[1], w, 1);
    w = __builtin_amdgcn_cvt_sr_bf8_f32(y[2], r[2], w, 2);
    return (uint32_t)__builtin_amdgcn_cvt_sr_bf8_f32(y[3], r[3], w, 3);
  }
  __device__ static void unpack(uint32_t w, float (&y)[4]) {
    const auto a = __builtin_amdgcn_cvt_pk_f32_bf8((int)w, false), b = __builtin_amdgcn_cvt_pk_f32_bf8((int)w, true);
    y[0] = a[0], y[1] = a[1], y[2] = b[0], y[3] = b[1];
  }
};

// Codes of a wave's 256 values and their scale (in every lane).  A NaN or an infinity leaves the others' scale alone: the
// maximum passes a NaN over, and infinities are looked for only where it is one.  Where the largest is below 2^-100, m is
// held as zeros.  v, of smaller values still, is not: a positive v that went to 0 would leave its element's step to eps.
// Its scale is 2^-133 at least, so that the least code stays a positive number (2^-149), and its codes are formed from
// values times 2^100.
template <class Q, bool SR>
__device__ __forceinline__ uint32_t to_codes(const float (&x)[4], float& scale, const uint32_t (&random)[4]) {
  float high = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
  high = team_max<64>(high);
  float inv, y[4] = {x[0], x[1], x[2], x[3]};
  if (high >= 0x1p-100f && high < INFINITY) {  // uniform over the wave
    inv = Q::kTop / high, scale = high * (1.f / Q::kTop);
  } else {
    const bool inf = high == INFINITY;
    if (inf) {
      high = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) high = fabsf(x[e]) < INFINITY ? fmaxf(high, fabsf(x[e])) : high;
      high = team_max<64>(high);
    }
    if (high >= 0x1p-100f) {
      inv = Q::kTop / high, scale = high * (1.f / Q::kTop);
    } else if (Q::kLeast > 0.f && (high > 0.f || inf)) {
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] *= 0x1p100f;
      high = fmaxf(high * 0x1p100f, 0x1p-33f * Q::kTop);
      inv = Q::kTop / high, scale = high * (0x1p-100f / Q::kTop);
    } else {
      inv = scale = 0.f;
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    y[e] *= inv;
    if (Q::kLeast > 0.f && x[e] > 0.f) y[e] = y[e] < Q::kLeast ? Q::kLeast : y[e];
  }
  if constexpr (SR) return Q::pack(y, random);
  else return Q::pack(y);
}

// Random words of a lane's four values: a hash of their place in the table and the step's key, and three products of it.
// (The same for a value whatever its arrays' alignment.)
__device__ __forceinline__ void random_words(uint32_t place, uint32_t key, uint32_t (&w)[4]) {
  uint32_t x = place + key;
  x = (x ^ x >> 16) * 0x9E3779B1u;
  x = (x ^ x >> 15) * 0x6A09E667u;
  w[0] = x ^ x >> 16;
  w[1] = w[0] * 0xBB67AE85u, w[2] = w[0] * 0x3C6EF373u, w[3] = w[0] * 0xA54FF53Bu;
}

// Square root to one unit in the last place.  (The instruction takes values below the normal range as 0: scaled first.)
__device__ __forceinline__ float quick_sqrt(float v) {
  const bool low = v < 0x1p-96f;
  const float s = __builtin_amdgcn_sqrtf(low ? v * 0x1p64f : v);
  return low ? s * 0x1p-32f : s;
}

// A pointer of the table: the same in all lanes (in scalar registers, so that accesses are an address and a lane's
// distance from it) and to global memory (what is read from memory could be any address, which takes flat accesses).
template <class X>
__device__ __forceinline__ X* uniform(X* x) {
  const uint64_t b = (uint64_t)x;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)b), hi = __builtin_amdgcn_readfirstlane((uint32_t)(b >> 32));
  typedef __attribute__((address_space(1))) X Global;
  return (X*)(Global*)((uint64_t)hi << 32 | lo);
}

// The sums and products of m and v are rounded one by one, as the formula has them: what is held in 8 bits then does
// not depend on which of them a compiler joins.
template <class TP, class TG, bool MASTER, int BITS, bool STREAM, bool SR>
__global__ __launch_bounds__(256) void adamw_kernel(const char* __restrict__ table, int64_t map_at, int64_t chunks,
                                                    Rates r, Live live) {
#pragma clang fp contract(off)
  constexpr int U = kAdamChunk / 1024;  // groups of four values a lane
  constexpr bool Q8 = BITS == 8;
  if (live.skip && *live.skip) return;
  if (live.step || live.lr) {
    __shared__ Rates shared;
    if (threadIdx.x == 0) {
      shared = r;
      set_step(shared, live.lr ? (double)*live.lr : live.lr_, live.b1, live.b2, live.wd,
               live.step ? *live.step : live.step_);
    }
    __syncthreads();
    r = shared;
  }
  const float gscale = live.gscale ? *live.gscale : 1.f;
  const int32_t* map = reinterpret_cast<const int32_t*>(table + map_at);
  for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    AdamItem t = reinterpret_cast<const AdamItem*>(table)[map[c]];
    auto* p = uniform(static_cast<typename TP::raw*>(t.p));
    auto* g = uniform(static_cast<const typename TG::raw*>(t.g));
    t.master = uniform(t.master), t.sm = uniform(t.sm), t.sv = uniform(t.sv);
    using S = std::conditional_t<Q8, uint8_t, float>;
    auto* tm = uniform(static_cast<S*>(t.m));
    auto* tv = uniform(static_cast<S*>(t.v));
    const int64_t base = (c - t.first) * kAdamChunk;
    const float keep = 1.f - r.lr_wd * t.decay;
    auto at = [&](int u) { return base + u * 1024 + (int64_t)threadIdx.x * 4; };
    auto words = [&](int u, uint32_t (&w)[4]) {
      if constexpr (SR) random_words(((uint32_t)c * U + u) * 256 + threadIdx.x, r.key, w);
    };
    auto take = [](auto& pack, const auto* from) {
      if constexpr (STREAM) pack.load_nt(from);
      else pack.load(from);
    };
    auto put = [](const auto& pack, auto* to) {
      if constexpr (STREAM) pack.store_nt(to);
      else pack.store(to);
    };
    auto take4 = [](const uint8_t* from, uint32_t i) {
      const auto* q = reinterpret_cast<const uint32_t*>(from + i);
      return STREAM ? __builtin_nontemporal_load(q) : *q;
    };
    auto put4 = [](uint8_t* to, uint32_t i, uint32_t w) {
      auto* q = reinterpret_cast<uint32_t*>(to + i);
      if constexpr (STREAM) __builtin_nontemporal_store(w, q);
      else *q = w;
    };
    // the lane's group u: values p, g, m, v in, and p, m, v out
    auto step = [&](float (&pv)[4], const float (&gv)[4], float (&mv)[4], float (&vv)[4]) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float gr = gv[e] * gscale;
        mv[e] = mv[e] * r.b1 + gr * r.c1;
        vv[e] = vv[e] * r.b2 + (gr * gr) * r.c2;
        // With states in 32 bits the root and the quotient are good to one unit each: 2^25 values in 166 us, 171 rounded
        // in full.  With 8 bits a lane waits less for them, and in full they cost nothing (200 million values 525 us, 541).
        const float d = (Q8 ? sqrtf(vv[e]) : quick_sqrt(vv[e])) * r.root + r.eps;
        // 0 / 0 only where eps is 0 and nothing has moved
        const float q = mv[e] == 0.f && d == 0.f ? 0.f : Q8 ? mv[e] / d : mv[e] * __builtin_amdgcn_rcpf(d);
        pv[e] = pv[e] * keep - q * r.rate;
      }
    };
    if (t.aligned && base + kAdamChunk <= t.numel) {  // uniform over the workgroup
      // (one address for the workgroup, and a lane's distance from it)
      const uint32_t own = threadIdx.x * 4;
      auto* p0 = p + base;
      const auto* g0 = g + base;
      float* w0 = t.master + base;
      auto *m0 = tm + base, *v0 = tv + base;
      float *sm0 = t.sm + base / kAdamBlock, *sv0 = t.sv + base / kAdamBlock;
      Pack<TP, 4> pp[U];
      Pack<F32, 4> pm[U], m[U], v[U];
      Pack<TG, 4> gg[U];
      uint32_t mq[U], vq[U];
      float sm[U], sv[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t i = own + u * 1024;
        if constexpr (MASTER) take(pm[u], w0 + i);
        else take(pp[u], p0 + i);
        take(gg[u], g0 + i);
        if constexpr (Q8) {
          mq[u] = take4(m0, i);
          vq[u] = take4(v0, i);
          sm[u] = sm0[i / kAdamBlock], sv[u] = sv0[i / kAdamBlock];
        } else {
          take(m[u], m0 + i);
          take(v[u], v0 + i);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t i = own + u * 1024;
        float pv[4], gv[4], mv[4], vv[4];
        if constexpr (MASTER) pm[u].unpack(pv);
        else pp[u].unpack(pv);
        gg[u].unpack(gv);
        if constexpr (Q8) {
          E4M3::unpack(mq[u], mv);
          E5M2::unpack(vq[u], vv);
#pragma unroll
          for (int e = 0; e < 4; ++e) mv[e] *= sm[u], vv[e] *= sv[u];
        } else {
          m[u].unpack(mv);
          v[u].unpack(vv);
        }
        step(pv, gv, mv, vv);
        pp[u].pack(pv);
        put(pp[u], p0 + i);
        if constexpr (MASTER) {
          pm[u].pack(pv);
          put(pm[u], w0 + i);
        }
        if constexpr (Q8) {
          float a, b;
          uint32_t w[4];
          words(u, w);
          const uint32_t ma = to_codes<E4M3, SR>(mv, a, w), va = to_codes<E5M2, SR>(vv, b, w);
          put4(m0, i, ma);
          put4(v0, i, va);
          if (i % kAdamBlock == 0) sm0[i / kAdamBlock] = a, sv0[i / kAdamBlock] = b;
        } else {
          m[u].pack(mv);
          v[u].pack(vv);
          put(m[u], m0 + i);
          put(v[u], v0 + i);
        }
      }
    } else {
      // a tensor's end, or arrays at odd addresses: element by element
      for (int u = 0; u < U; ++u) {
        const int64_t i = at(u);
        float pv[4] = {}, gv[4] = {}, mv[4] = {}, vv[4] = {};
        uint32_t mq = 0, vq = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (i + e >= t.numel) continue;
          pv[e] = MASTER ? t.master[i + e] : TP::to_f32(p[i + e]);
          gv[e] = TG::to_f32(g[i + e]);
          if constexpr (Q8) {
            mq |= (uint32_t)tm[i + e] << 8 * e;
            vq |= (uint32_t)tv[i + e] << 8 * e;
          } else {
            mv[e] = tm[i + e];
            vv[e] = tv[i + e];
          }
        }
        if constexpr (Q8) {
          E4M3::unpack(mq, mv);
          E5M2::unpack(vq, vv);
          const float a = i < t.numel ? t.sm[i / kAdamBlock] : 0.f, b = i < t.numel ? t.sv[i / kAdamBlock] : 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) mv[e] *= a, vv[e] *= b;
        }
        step(pv, gv, mv, vv);
        if constexpr (Q8) {
          float a, b;
          uint32_t w[4];
          words(u, w);
          mq = to_codes<E4M3, SR>(mv, a, w), vq = to_codes<E5M2, SR>(vv, b, w);  // all lanes of the wave take part
          if (i % kAdamBlock == 0 && i < t.numel) t.sm[i / kAdamBlock] = a, t.sv[i / kAdamBlock] = b;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (i + e >= t.numel) continue;
          p[i + e] = round_to<TP>(pv[e]);
          if constexpr (MASTER) t.master[i + e] = pv[e];
          if constexpr (Q8) {
            tm[i + e] = (uint8_t)(mq >> 8 * e);
            tv[i + e] = (uint8_t)(vq >> 8 * e);
          } else {
            tm[i + e] = mv[e];
            tv[i + e] = vv[e];
          }
        }
      }
    }
  }
}

// Steps that move this many bytes (half of the last cache) are streamed past the caches: 124 million bf16 values with
// fp32 copies 607 us, 652 not so; 33.5 million fp32 values 161 and 178; 4.2 million 21.7 and 18.7.
constexpr int64_t kStream = (int64_t)1 << 27;

template <class TP, class TG, bool MASTER>
hipError_t adamw_t(const AdamCall& c, hipStream_t s) {
  Rates r{(float)c.b1, (float)(1.0 - c.b1), (float)c.b2, (float)(1.0 - c.b2), (float)c.eps, 0.f, 0.f, 0.f, 0u};
  set_step(r, c.lr, c.b1, c.b2, c.wd, c.step_at ? 1 : c.step);
  const Live live{c.lr_at, c.step_at, c.gscale_at, c.skip_at, c.lr, c.b1, c.b2, c.wd, c.step};
  const int64_t grid = c.chunks < (1 << 22) ? c.chunks : (1 << 22);
  const auto* table = static_cast<const char*>(c.table);
  const int64_t map_at = (int64_t)adam_map_at(c.count);
  const int64_t each = (MASTER ? TP::SZ + 8 : 2 * TP::SZ) + TG::SZ + (c.bits == 8 ? 4 : 16);
  const bool stream = c.chunks * kAdamChunk * each >= kStream;
  auto go = [&](auto kernel) {
    kernel<<<dim3((unsigned)grid), dim3(256), 0, s>>>(table, map_at, c.chunks, r, live);
  };
  if (c.bits == 8 && c.stochastic) {
    if (stream) go(adamw_kernel<TP, TG, MASTER, 8, true, true>);
    else go(adamw_kernel<TP, TG, MASTER, 8, false, true>);
  } else if (c.bits == 8) {
    if (stream) go(adamw_kernel<TP, TG, MASTER, 8, true, false>);
    else go(adamw_kernel<TP, TG, MASTER, 8, false, false>);
  } else {
    if (stream) go(adamw_kernel<TP, TG, MASTER, 32, true, false>);
    else go(adamw_kernel<TP, TG, MASTER, 32, false, false>);
  }
  return hipGetLastError();
}
template <class TP>
hipError_t adamw_g(int gdt, const AdamCall& c, hipStream_t s) {
  auto go = [&](auto tg) {
    using TG = decltype(tg);
    if constexpr (TP::SZ == 2) {
      if (c.masters) return adamw_t<TP, TG, true>(c, s);
    }
    return adamw_t<TP, TG, false>(c, s);
  };
  switch (gdt) {
    case DT_F32: return go(F32{});
    case DT_F16: return go(F16{});
    case DT_BF16: return go(BF16{});
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_adamw(int pdt, int gdt, const AdamCall& c, hipStream_t s) {
  switch (pdt) {
    case DT_F32: return adamw_g<F32>(gdt, c, s);
    case DT_F16: return adamw_g<F16>(gdt, c, s);
    case DT_BF16: return adamw_g<BF16>(gdt, c, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace fkm
