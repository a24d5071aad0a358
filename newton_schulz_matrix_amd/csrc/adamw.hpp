// adamw.hpp - one AdamW step over many tensors.
//
//   g = s g0,  m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//   p = p - lr wd p - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
//
// Bound by memory: every element of p, g, m and v is read once and p, m and v
// are written once, 22 bytes an element with 16-bit p and g and fp32 moments,
// 10 with 8-bit moments.  Measured (MI355X): 38.6M fp32 masters with bf16
// gradients and copies 214 us (5.0 TB/s), 524M bf16 parameters with 8-bit
// moments 1123 us (4.7), as a copy of that size; 50 vectors of 768 6 us.
//
// The tensors come as a table in the kernel's arguments (no copy to the
// device, no workspace), so a launch takes up to kAdamwItems of them, cut into
// chunks that the blocks take in turn.
//
// 8-bit moments: blocks of 256 elements, each with the largest magnitude `top`
// of its block in fp32 and e4m3 codes for x * (1 / top * 448).  The second moment
// is held by its root: v = g^2 spans twice the exponents of m, its root the
// same, and an error of the root is what the update sees.  A positive root
// below the smallest code (2^-9 of 448, 2^-17.8 of the block's largest) takes
// that code: as 0 it would make the next update of that element as large as
// its gradient's share of the second moment allows.  The step itself uses the
// moments before they are rounded.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "xent.hpp"

namespace nsk {

constexpr int kAdamwItems = 54;                   // tensors of one launch: 4 KB of arguments
constexpr int kAdamwThreads = 256;
constexpr int kStateBlock = 256;                  // elements that share a scale
// 16 lanes take a block, each two groups of 8 elements half a block apart, so
// that neighbours' 16-byte vectors lie side by side.  (32 lanes with a group
// each spent a fifth more instructions per element, on addresses and on the
// blocks' scales, and arithmetic was 70 % of the time.)
constexpr int kAdamwGroups = 2, kAdamwLanes = kStateBlock / (8 * kAdamwGroups);
constexpr int kAdamwChunk = kAdamwThreads * 8 * kAdamwGroups;
constexpr float kCodeTop = 448.f;                 // the largest e4m3 number
constexpr float kCodeLeast = 0x1p-9f;             // and the smallest positive one
constexpr float kScaleLeast = 0x1p-100f;          // keeps 448 / top finite

struct AdamwItem {
  void* p;
  const void* g;
  void *m, *v;
  float* scales;  // [2][blocks of 256]: 8-bit moments; null: fp32 ones
  void* copy;     // p rounded to another type, or null
  int64_t n;
  float lr, decay;
};

struct AdamwArgs {
  AdamwItem item[kAdamwItems];
  int32_t types[kAdamwItems];  // ns_dtype of p, g and copy in bits 0, 4 and 8
  int32_t first[kAdamwItems];  // an item's first chunk
  int count, chunks;
  float b1, a1, b2, a2;  // a = 1 - b
  float eps, c1, c2;     // 1 / (1 - b1^t), 1 / sqrt(1 - b2^t); from d_step where that is given
  double log_b1, log_b2;
  const int32_t* d_step;
  const float *d_grad_scale, *d_lr_scale;
  int32_t* d_status;
  int32_t status_bits;
};

static_assert(sizeof(AdamwArgs) <= 4096, "kernel arguments");

// Eight consecutive elements of a type known at run time, as raw vectors and
// as floats; `left`: how many of them there are.  The type is the same for a
// whole block, so its branches cost no divergence.
struct Eight {
  u32x4_t q[2];
};
template <typename T>
__device__ __forceinline__ void load_eight(const T* s, int64_t left, Eight& r) {
  constexpr int N = 8 / kVec<T>;
  if (left >= 8) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      r.q[i] = *reinterpret_cast<const typename Vec16<sizeof(T)>::type*>(s + i * kVec<T>);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      r.q[i] = u32x4_t{0u, 0u, 0u, 0u};
      T* e = reinterpret_cast<T*>(&r.q[i]);
#pragma unroll
      for (int k = 0; k < kVec<T>; ++k)
        if (i * kVec<T> + k < left) e[k] = s[i * kVec<T> + k];
    }
  }
}
template <typename T>
__device__ __forceinline__ void floats_of(const Eight& r, float (&f)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] = to_f32<T>(reinterpret_cast<const T*>(&r.q[k / kVec<T>])[k % kVec<T>]);
}
// Returns nonfinite_bits of what was stored.
template <typename T>
__device__ __forceinline__ uint32_t store_eight(T* d, int64_t left, const float (&f)[8]) {
  constexpr int N = 8 / kVec<T>;
  Eight r;
#pragma unroll
  for (int k = 0; k < 8; ++k) reinterpret_cast<T*>(&r.q[k / kVec<T>])[k % kVec<T>] = from_f32<T>(f[k]);
  uint32_t found = 0;
  if (left >= 8) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      *reinterpret_cast<typename Vec16<sizeof(T)>::type*>(d + i * kVec<T>) = r.q[i];
#pragma unroll
      for (int k = 0; k < 4; ++k) found |= nonfinite_bits<T>(r.q[i][k]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < left) {
        d[k] = reinterpret_cast<const T*>(&r.q[k / kVec<T>])[k % kVec<T>];
        found |= nonfinite_bits<T>(one_bits(d[k]));
      }
  }
  return found & kNonfiniteMask<T>;
}

// Calls f(T{}) for an ns_dtype.
template <class F>
__device__ __forceinline__ void of_type(int type, F&& f) {
  if (type == NS_FP32)
    f(float{});
  else if (type == NS_BF16)
    f(__bf16{});
  else
    f(_Float16{});
}

// Eight e4m3 codes.
struct Codes {
  uint32_t w[2];
};
__device__ __forceinline__ Codes load_codes(const uint8_t* s, int64_t left) {
  typedef uint32_t u32x2_b __attribute__((ext_vector_type(2), aligned(1)));
  Codes c{{0u, 0u}};
  if (left >= 8) {
    const u32x2_b q = *reinterpret_cast<const u32x2_b*>(s);
    c.w[0] = q[0];
    c.w[1] = q[1];
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < left) c.w[k / 4] |= (uint32_t)s[k] << (8 * (k % 4));
  }
  return c;
}
__device__ __forceinline__ void store_codes(uint8_t* d, int64_t left, const Codes& c) {
  typedef uint32_t u32x2_b __attribute__((ext_vector_type(2), aligned(1)));
  if (left >= 8) {
    *reinterpret_cast<u32x2_b*>(d) = u32x2_b{c.w[0], c.w[1]};
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < left) d[k] = (uint8_t)(c.w[k / 4] >> (8 * (k % 4)));
  }
}
__device__ __forceinline__ void decode(const Codes& c, float unit, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.w[i], false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.w[i], true);
    f[4 * i] = lo[0] * unit;
    f[4 * i + 1] = lo[1] * unit;
    f[4 * i + 2] = hi[0] * unit;
    f[4 * i + 3] = hi[1] * unit;
  }
}
// Codes of f * inv; ROOT: positive numbers take the smallest code at least.
template <bool ROOT>
__device__ __forceinline__ Codes encode(const float (&f)[8], float inv) {
  float q[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    q[k] = f[k] * inv;
    if (ROOT) q[k] = f[k] > 0.f ? fmaxf(q[k], kCodeLeast) : f[k];
  }
  Codes c;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i], q[4 * i + 1], 0, false);
    c.w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i + 2], q[4 * i + 3], w, true);
  }
  return c;
}

// Largest of 16 lanes' values (>= 0, NaN passed over), in every one of them.
template <int CTRL>
__device__ __forceinline__ float max_dpp(float v) {
  const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false);
  return fmaxf(v, __builtin_bit_cast(float, o));
}
__device__ __forceinline__ float block_max(float v) {
  static_assert(kAdamwLanes == 16, "a row of the data-parallel moves");
  v = max_dpp<0xB1>(v);
  v = max_dpp<0x4E>(v);
  v = max_dpp<0x141>(v);
  return max_dpp<0x140>(v);
}

// The square root, rounded to nearest (codes and scales are made of it, and
// equal moments give equal ones whoever computes them): the hardware's
// reciprocal root, one Newton step for the root s and half its reciprocal h,
// and the residual's last correction.  The compiler's own sequence takes twice
// the instructions, for moments of 2^-100 and more and zero.  An infinite
// moment counts as the largest finite one, whose root is kRootTop.  A NaN
// stays one (fminf would make it the largest number, whose root would become
// the scale of the whole block): the maxima of a block pass it over, and its
// code is e4m3's NaN.
constexpr float kRootTop = 0x1.fffffep63f, kRootLeast = 0x1p-100f;
__device__ __forceinline__ float root_of(float v) {
  v = v > 0x1.fffffep127f ? 0x1.fffffep127f : v;
  const float y = __builtin_amdgcn_rsqf(fmaxf(v, 0x1p-126f));
  float s = v * y, h = 0.5f * y;
  const float r = fmaf(-h, s, 0.5f);
  s = fmaf(s, r, s);
  h = fmaf(h, r, h);
  return fmaf(fmaf(-s, s, v), h, s);
}
// Of a moment below kRootLeast, whose residual would fall among the subnormal
// numbers and which the reciprocal root does not take below 2^-126.  Only where
// the least of eight moments but zeros is one, which costs 6 us of 1123 at 524M
// 8-bit moments; scaling every moment costs 20, and going there for zeros took
// 1237 us where most moments are (rows of an embedding that no token met).
__device__ __forceinline__ float root_of_small(float v) { return root_of(v * 0x1p64f) * 0x1p-32f; }

// The moments' update, each operation rounded on its own (no fused
// multiply-adds): a code is then what its formula in fp32 gives, whoever
// computes it.
__device__ __forceinline__ void next_moments(float b1, float a1, float b2, float a2, float g, float& m, float& v) {
#pragma clang fp contract(off)
  m = b1 * m + a1 * g;
  v = b2 * v + a2 * g * g;
}

static __global__ void __launch_bounds__(kAdamwThreads) k_adamw(AdamwArgs a) {
  float c1 = a.c1, c2 = a.c2;
  if (a.d_step) {
    const double t = (double)*a.d_step;
    c1 = (float)(-1.0 / expm1(t * a.log_b1));
    c2 = (float)(1.0 / sqrt(-expm1(t * a.log_b2)));
  }
  const float gs = a.d_grad_scale ? *a.d_grad_scale : 1.f, lrs = a.d_lr_scale ? *a.d_lr_scale : 1.f;
  // The first chunk's tensor: the last one that begins at or before it.  Each
  // lane looks at one tensor: one read of the arguments and not one after the
  // other, as in a search (50 vectors, captured: 6.2 us a step, not 6.5).
  static_assert(kAdamwItems <= 64, "a lane each");
  const int lane = (int)threadIdx.x & 63;
  int i = __popcll(__ballot(lane < a.count && a.first[lane < a.count ? lane : 0] <= (int)blockIdx.x)) - 1;
  bool bad = false;
  constexpr int kG = kAdamwGroups;
  // A thread's place in a chunk: block, lane and with it the first group.
  const int place = (int)threadIdx.x / kAdamwLanes * kStateBlock + (int)threadIdx.x % kAdamwLanes * 8;
  constexpr int kApart = kAdamwLanes * 8;
  for (int chunk = blockIdx.x; chunk < a.chunks; chunk += gridDim.x) {
    while (i + 1 < a.count && a.first[i + 1] <= chunk) ++i;
    const AdamwItem& it = a.item[i];
    const int64_t e0 = (int64_t)(chunk - a.first[i]) * kAdamwChunk + place;
    const int types = a.types[i], pt = types & 15, gt = types >> 4 & 15, ct = types >> 8 & 15;
    const bool coded = it.scales != nullptr;
    const int64_t block = e0 / kStateBlock, blocks = (it.n + kStateBlock - 1) / kStateBlock;
    Eight rp[kG], rg[kG], rm[kG], rv[kG];
    Codes cm[kG], cv[kG];
    float um = 0.f, uv = 0.f;
    of_type(gt, [&](auto t) {
#pragma unroll
      for (int j = 0; j < kG; ++j) load_eight(reinterpret_cast<const decltype(t)*>(it.g) + e0 + j * kApart, it.n - e0 - j * kApart, rg[j]);
    });
    of_type(pt, [&](auto t) {
#pragma unroll
      for (int j = 0; j < kG; ++j) load_eight(reinterpret_cast<const decltype(t)*>(it.p) + e0 + j * kApart, it.n - e0 - j * kApart, rp[j]);
    });
    if (coded) {
#pragma unroll
      for (int j = 0; j < kG; ++j) {
        cm[j] = load_codes(reinterpret_cast<const uint8_t*>(it.m) + e0 + j * kApart, it.n - e0 - j * kApart);
        cv[j] = load_codes(reinterpret_cast<const uint8_t*>(it.v) + e0 + j * kApart, it.n - e0 - j * kApart);
      }
      if (block < blocks) {
        um = it.scales[block] * (1.f / kCodeTop);
        uv = it.scales[blocks + block] * (1.f / kCodeTop);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kG; ++j) {
        load_eight(reinterpret_cast<const float*>(it.m) + e0 + j * kApart, it.n - e0 - j * kApart, rm[j]);
        load_eight(reinterpret_cast<const float*>(it.v) + e0 + j * kApart, it.n - e0 - j * kApart, rv[j]);
      }
    }
    const float lr = it.lr * lrs, keep = 1.f - lr * it.decay, lrc = lr * c1;
    float m[kG][8], root[kG][8], tm = 0.f, tv = 0.f;
#pragma unroll
    for (int j = 0; j < kG; ++j) {
      const int64_t e = e0 + j * kApart, left = it.n - e;
      float p[8], g[8], v[8];
      float least = 1.f;
      of_type(pt, [&](auto t) { floats_of<decltype(t)>(rp[j], p); });
      of_type(gt, [&](auto t) { floats_of<decltype(t)>(rg[j], g); });
      if (coded) {
        decode(cm[j], um, m[j]);
        decode(cv[j], uv, v);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] *= v[k];
      } else {
        floats_of<float>(rm[j], m[j]);
        floats_of<float>(rv[j], v);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        next_moments(a.b1, a.a1, a.b2, a.a2, g[k] * gs, m[j][k], v[k]);
        root[j][k] = root_of(v[k]);
        least = fminf(least, v[k]);
      }
      if (least < kRootLeast) {
        // Zeros, whose root is right, wrap to the top.
        uint32_t key = ~0u;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t u = __float_as_uint(v[k]) - 1u;
          key = u < key ? u : key;
        }
        if (key < __float_as_uint(kRootLeast) - 1u) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (v[k] < kRootLeast) root[j][k] = root_of_small(v[k]);
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        // The hardware's reciprocal is good to a step of fp32; only the step
        // is made of it.
        p[k] = fmaf(-lrc * m[j][k], __builtin_amdgcn_rcpf(fmaf(root[j][k], c2, a.eps)), p[k] * keep);
        tm = fmaxf(tm, fabsf(m[j][k]));
        tv = fmaxf(tv, root[j][k]);
      }
      if (left <= 0) continue;
      if (!coded) {
        bad |= (store_eight(reinterpret_cast<float*>(it.m) + e, left, m[j]) |
                store_eight(reinterpret_cast<float*>(it.v) + e, left, v)) != 0;
      }
      of_type(pt, [&](auto t) { bad |= store_eight(reinterpret_cast<decltype(t)*>(it.p) + e, left, p) != 0; });
      if (it.copy)
        of_type(ct, [&](auto t) { bad |= store_eight(reinterpret_cast<decltype(t)*>(it.copy) + e, left, p) != 0; });
    }
    if (!coded) continue;
    // All lanes of a block take part, those past the tensor's end with zeros.
    // An infinite moment may leave p finite; a NaN does not.
    bad |= !(tm < __builtin_inff() && tv < kRootTop);
    tm = fmaxf(block_max(tm), kScaleLeast);
    tv = fmaxf(block_max(tv), kScaleLeast);
    const float im = 1.f / tm * kCodeTop, iv = 1.f / tv * kCodeTop;
#pragma unroll
    for (int j = 0; j < kG; ++j) {
      const int64_t e = e0 + j * kApart, left = it.n - e;
      if (left <= 0) continue;
      store_codes(reinterpret_cast<uint8_t*>(it.m) + e, left, encode<false>(m[j], im));
      store_codes(reinterpret_cast<uint8_t*>(it.v) + e, left, encode<true>(root[j], iv));
    }
    if (threadIdx.x % kAdamwLanes == 0 && block < blocks) {
      it.scales[block] = tm;
      it.scales[blocks + block] = tv;
    }
  }
  if (a.d_status) report_status(a.d_status, a.status_bits, bad);
}

}  // namespace nsk
