// Internal interfaces of the feed-forward operators: the norms around a block
// (hc_norm.hip), the matrix products (hc_gemm.hip) and their activations
// (shared by the products' epilogues and the element-wise backward kernels).
#pragma once

#include "hc_device.h"

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace hc {

// ------------------------------------------------------------------ activations

enum Act : int { ACT_NONE = 0, ACT_RELU = 1, ACT_SILU = 2, ACT_GELU = 3, ACT_GELU_TANH = 4, ACT_SIGMOID = 5 };

constexpr float GELU_C = 0.7978845608028654f;   // sqrt(2 / pi)
constexpr float GELU_A = 0.044715f;
constexpr float RSQRT2 = 0.7071067811865476f;
constexpr float RSQRT2PI = 0.3989422804014327f;

// Sigmoid for values that are then rounded to 16 bits: hardware exponential and
// reciprocal (about 1 ulp each), relative error below 2^-20 for |x| < 16 and an exact
// 0 or 1 in the limits. An epilogue of 64 gated outputs per thread costs about 3 us
// per tile with it, about 12 with expf and a division.
__device__ __forceinline__ float sigmoid_fast(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -1.4426950408889634f));
}
// Phi(x), the normal distribution function, for the same use. Phi(-a) = exp(-a^2 / 2) m(a) for
// a >= 0, with m(a) = t P(t), t = 1 / (1 + 0.36 a): P has degree 6 and was fitted so that the
// largest relative error over 0 <= a <= 15 is least (1.1e-6). With the fp32 steps' rounding the
// relative error is below 2.2e-6 for |x| < 6 and 7e-6 beyond (the exponent's own rounding), far
// below half a step of fp16 (4.9e-4) down to where the result leaves the normal numbers of T.
__device__ __forceinline__ float phi_fast(float x) {
  const float a = fabsf(x);
  const float t = __builtin_amdgcn_rcpf(fmaf(0.36f, a, 1.0f));
  float p = fmaf(0.04649430513381958f, t, -0.17784516513347626f);
  p = fmaf(p, t, 0.17835372686386108f);
  p = fmaf(p, t, 0.02832658961415291f);
  p = fmaf(p, t, 0.13907690346240997f);
  p = fmaf(p, t, 0.14188815653324127f);
  p = fmaf(p, t, 0.14370496571063995f);
  const float tail = p * t * __builtin_amdgcn_exp2f(a * a * -0.7213475204444817f);
  return x < 0.0f ? tail : 1.0f - tail;
}
template <DT D> __device__ __forceinline__ float sigmoid_of(float x) {
  return D == DT::F32 ? sigmoid(x) : sigmoid_fast(x);
}
template <DT D> __device__ __forceinline__ float phi_of(float x) {
  return D == DT::F32 ? 0.5f * erfcf(-x * RSQRT2) : phi_fast(x);
}
// s = sigmoid(x) and c = 1 - s, both with their full relative accuracy (a subtraction from one
// would leave c, and so the slope s c, few correct bits for large x): with e = exp(-x) they are
// 1 / (1 + e) and e / (1 + e). An infinite e is taken as the largest value, so that c stays finite
// where s is 0.
template <DT D> __device__ __forceinline__ void sigmoid_both(float x, float& s, float& c) {
  const float e = D == DT::F32 ? expf(-x) : __builtin_amdgcn_exp2f(x * -1.4426950408889634f);
  s = D == DT::F32 ? 1.0f / (1.0f + e) : __builtin_amdgcn_rcpf(1.0f + e);
  c = fminf(e, 3.4028234663852886e38f) * s;
}
__device__ __forceinline__ float relu(float x) { return x > 0.0f ? x : (x <= 0.0f ? 0.0f : x); }  // NaN stays NaN
__device__ __forceinline__ float gelu_arg(float x) { return 2.0f * GELU_C * (x + GELU_A * x * x * x); }

// N values x replaced by act(x), for outputs of type D. GELU as x * Phi(x) with Phi's tail
// computed as such (fp32: erfc(-x / sqrt 2) / 2, whose relative error grows as x^2 2^-24 with its
// argument's rounding; 16 bits: phi_fast) and GELU_TANH as x * sigmoid(2 t): they equal the usual
// forms and keep their relative accuracy for negative x, where 1 + erf and 1 + tanh cancel.
template <DT D, int N> __device__ __forceinline__ void act_n(int kind, float* x) {
  switch (kind) {
    case ACT_RELU:
#pragma unroll
      for (int e = 0; e < N; ++e) x[e] = relu(x[e]);
      break;
    case ACT_SILU:
#pragma unroll
      for (int e = 0; e < N; ++e) x[e] = x[e] * sigmoid_of<D>(x[e]);
      break;
    case ACT_GELU:
#pragma unroll
      for (int e = 0; e < N; ++e) x[e] = x[e] * phi_of<D>(x[e]);
      break;
    case ACT_GELU_TANH:
#pragma unroll
      for (int e = 0; e < N; ++e) x[e] = x[e] * sigmoid_of<D>(gelu_arg(x[e]));
      break;
    case ACT_SIGMOID:
#pragma unroll
      for (int e = 0; e < N; ++e) x[e] = sigmoid_of<D>(x[e]);
      break;
    default: break;
  }
}

// N values x replaced by act(x), and their slopes act'(x) in d.
template <DT D, int N> __device__ __forceinline__ void act_slope_n(int kind, float* x, float* d) {
  switch (kind) {
    case ACT_RELU:
#pragma unroll
      for (int e = 0; e < N; ++e) {
        d[e] = x[e] > 0.0f ? 1.0f : (x[e] <= 0.0f ? 0.0f : x[e]);  // NaN stays NaN
        x[e] = relu(x[e]);
      }
      break;
    case ACT_SILU:
#pragma unroll
      for (int e = 0; e < N; ++e) {
        float s, c;
        sigmoid_both<D>(x[e], s, c);
        d[e] = s * (1.0f + x[e] * c);
        x[e] = x[e] * s;
      }
      break;
    case ACT_GELU:
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float phi = phi_of<D>(x[e]), h = -0.5f * x[e] * x[e];
        const float g = D == DT::F32 ? expf(h) : __builtin_amdgcn_exp2f(h * 1.4426950408889634f);
        d[e] = phi + x[e] * (g * RSQRT2PI);
        x[e] = x[e] * phi;
      }
      break;
    case ACT_GELU_TANH:
#pragma unroll
      for (int e = 0; e < N; ++e) {  // 1 - tanh(t)^2 = 4 s (1 - s) with s = sigmoid(2 t)
        float s, c;
        sigmoid_both<D>(gelu_arg(x[e]), s, c);
        const float v = __builtin_amdgcn_fmed3f(x[e], -32.0f, 32.0f);  // beyond, s c is 0 and x^3 may be infinite
        d[e] = s + 2.0f * v * s * c * GELU_C * (1.0f + 3.0f * GELU_A * v * v);
        x[e] = x[e] * s;
      }
      break;
    case ACT_SIGMOID:
#pragma unroll
      for (int e = 0; e < N; ++e) {
        float s, c;
        sigmoid_both<D>(x[e], s, c);
        d[e] = s * c;
        x[e] = s;
      }
      break;
    default:
#pragma unroll
      for (int e = 0; e < N; ++e) d[e] = 1.0f;
      break;
  }
}

// ------------------------------------------------------------------ element access

// Eight elements from any element-aligned address, n of them valid (the others
// read as 0). ALN: every address is 16-byte aligned and n is always at least 8.
typedef unsigned u32x4_h __attribute__((ext_vector_type(4), aligned(2)));
typedef unsigned u32x4_w __attribute__((ext_vector_type(4), aligned(4)));

template <DT D, bool ALN> __device__ __forceinline__ uint4 ld16(const void* p) {
  if constexpr (ALN) return *(const uint4*)p;
  else if constexpr (D == DT::F32) return to_uint4(*(const u32x4_w*)p);
  else return to_uint4(*(const u32x4_h*)p);
}
template <DT D, bool ALN> __device__ __forceinline__ void st16(void* p, uint4 v) {
  if constexpr (ALN) *(uint4*)p = v;
  else if constexpr (D == DT::F32) *(u32x4_w*)p = to_u32x4(v);
  else *(u32x4_h*)p = to_u32x4(v);
}

template <DT D, bool ALN>
__device__ __forceinline__ void load8(const void* base, int64_t i, int n, float* x) {
  if constexpr (D == DT::F32) {
    const float* p = (const float*)base + i;
    if (ALN || n >= 8) {
      const f32x4 a = __builtin_bit_cast(f32x4, to_u32x4(ld16<D, ALN>(p)));
      const f32x4 b = __builtin_bit_cast(f32x4, to_u32x4(ld16<D, ALN>(p + 4)));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = a[e];
        x[4 + e] = b[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = e < n ? p[e] : 0.0f;
    }
  } else {
    const uint16_t* p = (const uint16_t*)base + i;
    if (ALN || n >= 8) {
      unpack8<D>(ld16<D, ALN>(p), x);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = e < n ? widen<D>(p[e]) : 0.0f;
    }
  }
}

// A buffer descriptor of `bytes` bytes from base (the same in every lane). Loads past its end
// give zeros, stores there are dropped.
typedef __amdgpu_buffer_rsrc_t rsrc_t;
__device__ __forceinline__ rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00020000);
}

// Eight elements as they are stored (half the registers of their fp32 values for 16-bit T).
template <DT D> struct Raw8 {
  u32x4 v;
};
template <> struct Raw8<DT::F32> {
  u32x4 v, w;
};
// From any element-aligned address, n of them valid.
template <DT D> __device__ __forceinline__ Raw8<D> load_raw8(const void* base, int64_t i, int n) {
  Raw8<D> r;
  if constexpr (D == DT::F32) {
    float x[8];
    load8<D, false>(base, i, n, x);
    r.v = __builtin_bit_cast(u32x4, f32x4{x[0], x[1], x[2], x[3]});
    r.w = __builtin_bit_cast(u32x4, f32x4{x[4], x[5], x[6], x[7]});
  } else {
    const uint16_t* p = (const uint16_t*)base + i;
    if (n >= 8) {
      r.v = to_u32x4(ld16<D, false>(p));
    } else {
      uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int e = 0; e < 7; ++e)
        if (e < n) w[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
      r.v = u32x4{w[0], w[1], w[2], w[3]};
    }
  }
  return r;
}
template <DT D> __device__ __forceinline__ Raw8<D> zero_raw8() {
  Raw8<D> r;
  r.v = u32x4{0u, 0u, 0u, 0u};
  if constexpr (D == DT::F32) r.w = r.v;
  return r;
}
template <DT D> __device__ __forceinline__ void unpack_raw8(const Raw8<D>& r, float* x) {
  if constexpr (D == DT::F32) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = __uint_as_float(r.v[e]);
      x[4 + e] = __uint_as_float(r.w[e]);
    }
  } else {
    unpack8<D>(to_uint4(r.v), x);
  }
}

// Rounds eight values to T and stores the first n.
template <DT D, bool ALN>
__device__ __forceinline__ void store8(void* base, int64_t i, int n, const float* x) {
  if constexpr (D == DT::F32) {
    float* p = (float*)base + i;
    if (ALN || n >= 8) {
      st16<D, ALN>(p, to_uint4(__builtin_bit_cast(u32x4, f32x4{x[0], x[1], x[2], x[3]})));
      st16<D, ALN>(p + 4, to_uint4(__builtin_bit_cast(u32x4, f32x4{x[4], x[5], x[6], x[7]})));
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < n) p[e] = x[e];
    }
  } else {
    uint16_t* p = (uint16_t*)base + i;
    if (ALN || n >= 8) {
      st16<D, ALN>(p, pack8<D>(x));
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < n) p[e] = (uint16_t)to_bits<D>(x[e]);
    }
  }
}

// ------------------------------------------------------------------ norms

struct NormArgs {
  const void *y, *res, *gate, *post, *pre;  // res: the residual (forward) or residual_out (backward)
  const void *dres, *dn;                    // backward: gradients of residual_out and normed, or null
  void *res_out, *normed;                   // forward
  void *dy, *d_residual, *d_gate;           // backward, each or null
  void *d_post, *d_pre;                     // backward: the scales' gradients, each or null
  float* partial;                           // backward: [groups][2][hidden] sums of the scales' gradients
  int64_t rows, gate_stride;
  int hidden, gate_kind, post_norm;
  float alpha, eps;
};

hipError_t launch_norm(const NormArgs& a, int dtype, bool aligned, hipStream_t s);
// Workgroups of the backward kernel, each with one row of partial sums: at most this many for
// this many rows or fewer.
int norm_backward_most_groups(int64_t rows, int64_t hidden);
hipError_t launch_norm_backward(const NormArgs& a, int dtype, bool aligned, hipStream_t s);

// out0[c], out1[c] (each or null) = T(sum over r, in a fixed order, of partial[r * pitch + c]
// and of partial[r * pitch + cols + c]) for c < cols.
hipError_t launch_column_sums(const float* partial, int nrows, int64_t pitch, int64_t cols, void* out0, void* out1,
                              int dtype, hipStream_t s);

// ------------------------------------------------------------------ products

// One product out[m][n] = epilogue(sum over k of P(m, k) Q(k, n)) or a pair of
// them. P(m, k) is p[m * ldp + k], or p[k * ldp + m] with p_trans; Q(k, n) is
// q[k * ldq + n], or q[n * ldq + k] with q_trans.
//   segments = 2: out = P0 Q0 + P1 Q1 (one sum over both contractions).
//   batch = 2: two products out[b] = P_b Q_b in one launch.
//   dual: g = P0 Q0 + bias0, u = P0 Q1 + bias1, out[0] = act(g) * u.
struct Product {
  const void* p[2];
  const void* q[2];
  int64_t ldp, ldq, ldr;
  int64_t M;
  int N, K;
  bool p_trans, q_trans, dual;
  int segments, batch;
  const void* bias[2];
  const void* residual;
  void* out[2];   // [M, N] contiguous
  void* save[2];  // pre-activations [M, N] (dual: g and u), or null
  int act;
};

// scratch: product_scratch() bytes (hc_plan.h); counters: HCLRMIX_COUNTER_BYTES, zero.
hipError_t launch_product(const Product& p, int dtype, void* scratch, unsigned* counters, hipStream_t s);

// dz = dy * act'(p) [rows, cols] into d0 and, with partial not null, the column sums of dz
// before its rounding into b0 [cols] (partial: grad_groups(rows) rows of scratch). Glu form
// (u not null): d0 = dy * u * act'(p), d1 = dy * act(p), sums into b0 and b1, scratch rows of
// 2 * cols. d0 and d1 may be null (only sums wanted).
// dz is rounded to T because it is an operand of the 16-bit matrix units in both products that
// follow. That costs their results one rounding more: 2.3e-3 from the 64-bit definition in bf16
// (2.9e-4 in fp16, relative 2-norm), where one rounding of the result alone is 1.7e-3 (2.1e-4);
// from the products of the rounded dz they are those 1.7e-3 (2.1e-4). A second product with what
// the rounding left off would take that away for twice the matrix work.
int grad_groups(int64_t rows);
hipError_t launch_act_grad(const void* dy, const void* p, const void* u, void* d0, void* d1, float* partial, void* b0,
                           void* b1, int64_t rows, int64_t cols, int act, int dtype, bool aligned, hipStream_t s);

// Writes zeros (n bytes, a multiple of 2).
hipError_t launch_zero(void* p, size_t n, hipStream_t s);

}  // namespace hc
