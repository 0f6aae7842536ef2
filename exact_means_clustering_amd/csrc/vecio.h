// Vectors of V elements of a storage type, converted to and from fp32 (internal).
#pragma once

#include "common.h"

namespace fkm {

// fp32 -> storage, rounded to nearest even once (infinities and NaN kept).
template <class T> __device__ __forceinline__ typename T::raw round_to(float f);
template <> __device__ __forceinline__ float round_to<F32>(float f) { return f; }
template <> __device__ __forceinline__ uint16_t round_to<F16>(float f) {
  return __builtin_bit_cast(uint16_t, (_Float16)f);
}
template <> __device__ __forceinline__ uint16_t round_to<BF16>(float f) {
  return __builtin_bit_cast(uint16_t, (__bf16)f);
}

// The 16-bit types' -infinity.
template <class T> constexpr uint32_t neg_inf_bits() { return 0; }
template <> constexpr uint32_t neg_inf_bits<F16>() { return 0xFC00u; }
template <> constexpr uint32_t neg_inf_bits<BF16>() { return 0xFF80u; }

// 16 * words bytes of V elements, moved with the widest accesses that the
// V elements' own size allows (16 bytes for V = 8, or 4 of fp32).  The address
// is aligned to the smaller of 16 bytes and the vector's size.
template <class T, int V> struct Pack {
  static constexpr int BYTES = V * T::SZ;
  static constexpr int UNIT = BYTES >= 16 ? 16 : BYTES;  // bytes per access
  static constexpr int W = BYTES >= 4 ? BYTES / 4 : 1;    // 32-bit words held
  uint32_t w[W];

  __device__ __forceinline__ void load(const typename T::raw* p) {
    if constexpr (BYTES >= 16) {
#pragma unroll
      for (int i = 0; i < BYTES / 16; ++i) {
        const uint4 v = reinterpret_cast<const uint4*>(p)[i];
        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
      }
    } else if constexpr (BYTES == 8) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x, w[1] = v.y;
    } else if constexpr (BYTES == 4) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    }
  }
  // the same, streamed past the caches (data read once)
  __device__ __forceinline__ void load_nt(const typename T::raw* p) {
    if constexpr (BYTES >= 16) {
#pragma unroll
      for (int i = 0; i < BYTES / 16; ++i) {
        const uint4 v = fkm::load_nt(reinterpret_cast<const uint4*>(p) + i);
        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
      }
    } else {
      load(p);
    }
  }
  __device__ __forceinline__ void store(typename T::raw* p) const {
    if constexpr (BYTES >= 16) {
#pragma unroll
      for (int i = 0; i < BYTES / 16; ++i)
        reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else if constexpr (BYTES == 8) {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else if constexpr (BYTES == 4) {
      *reinterpret_cast<uint32_t*>(p) = w[0];
    } else {
      *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
    }
  }
  // the same, streamed past the caches (data written once and not read here)
  __device__ __forceinline__ void store_nt(typename T::raw* p) const {
    if constexpr (BYTES >= 16) {
      typedef unsigned int v4u __attribute__((ext_vector_type(4)));
#pragma unroll
      for (int i = 0; i < BYTES / 16; ++i)
        __builtin_nontemporal_store(v4u{w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]},
                                    reinterpret_cast<v4u*>(p) + i);
    } else {
      store(p);
    }
  }
  // The same at an address aligned to its elements only (the hardware takes
  // unaligned global accesses; the compiler is told the alignment it has).
  struct __attribute__((packed, aligned(T::SZ))) Loose {
    uint32_t w[W];
  };
  __device__ __forceinline__ void load_loose(const typename T::raw* p) {
    static_assert(BYTES >= 4, "whole words");
    const Loose v = *reinterpret_cast<const Loose*>(p);
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = v.w[i];
  }
  __device__ __forceinline__ void store_loose(typename T::raw* p) const {
    Loose v;
#pragma unroll
    for (int i = 0; i < W; ++i) v.w[i] = w[i];
    *reinterpret_cast<Loose*>(p) = v;
  }
  // The first n < V elements only; the others keep what they hold.
  __device__ __forceinline__ void load_head(const typename T::raw* p, int n) {
#pragma unroll
    for (int i = 0; i < V - 1; ++i) {
      if (i >= n) continue;
      if constexpr (T::SZ == 4) {
        w[i] = __float_as_uint(p[i]);
      } else {
        const uint32_t h = p[i];
        w[i / 2] = (i & 1) ? (w[i / 2] & 0xFFFFu) | h << 16 : (w[i / 2] & 0xFFFF0000u) | h;
      }
    }
  }
  // Elements from `from` to before `to` only.
  __device__ __forceinline__ void store_range(typename T::raw* p, int from, int to) const {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (i < from || i >= to) continue;
      if constexpr (T::SZ == 4) p[i] = __uint_as_float(w[i]);
      else p[i] = (uint16_t)((i & 1) ? w[i / 2] >> 16 : w[i / 2]);
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ void fill_neg_inf() {
    constexpr uint32_t h = T::SZ == 4 ? 0xFF800000u : neg_inf_bits<T>();
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = T::SZ == 4 ? h : h | h << 16;
  }
  __device__ __forceinline__ void unpack(float* o) const {
    if constexpr (T::SZ == 4) {
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = T::to_f32((uint16_t)((i & 1) ? w[i / 2] >> 16 : w[i / 2] & 0xFFFFu));
    }
  }
  __device__ __forceinline__ void pack(const float* o) {
    if constexpr (T::SZ == 4) {
#pragma unroll
      for (int i = 0; i < V; ++i) w[i] = __float_as_uint(o[i]);
    } else if constexpr (V == 1) {
      w[0] = round_to<T>(o[0]);
    } else {
#pragma unroll
      for (int i = 0; i < V / 2; ++i)
        w[i] = (uint32_t)round_to<T>(o[2 * i]) | (uint32_t)round_to<T>(o[2 * i + 1]) << 16;
    }
  }
};

// The widest vector (8, 4 or 1 elements, `most` at most) in which rows of D
// elements at these addresses can be moved: it must divide the row, and both
// addresses must be aligned to the smaller of 16 bytes and the vector's size.
// `most` is 16 bytes of what is streamed past the caches: a lane that moves
// two 16-byte words of it makes every access of the wave touch half of each
// 32 bytes (949,595 fp32 rows of 128 looked up: 210 us with 8, 81 with 4).
inline int vec_width(int D, int most, const void* a, int a_size, const void* b, int b_size) {
  for (int v : {8, 4}) {
    if (v > most) continue;
    const int na = v * a_size < 16 ? v * a_size : 16, nb = v * b_size < 16 ? v * b_size : 16;
    if (D % v == 0 && (uintptr_t)a % na == 0 && (uintptr_t)b % nb == 0) return v;
  }
  return 1;
}

}  // namespace fkm
