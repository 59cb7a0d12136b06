// residual_norm: the norms before and after a block, fused with the block's
// gate and residual scale, and its backward pass.
//
//   z = (post_norm ? y * ry : y) * post,   r' = res + alpha * gate * z,
//   n = (r' * rr) * pre,   ry = 1 / sqrt(mean y^2 + eps), rr likewise of r'.
//
// Backward, with D the gradient of r', t = dn * pre, q = alpha * gate * D * post:
//   D  = dr' + rr * (t - r' * rr^2 * mean(t * r'))
//   dy = ry * (q - y * ry^2 * mean(q * y))   (post_norm; else q)
//   d_res = D; d_gate = alpha * z * D (summed over the row for a gate per row);
//   d_post = sum over rows of alpha * gate * D * (y * ry);
//   d_pre  = sum over rows of dn * (r' * rr).
//
// Both are bounded by HBM: forward reads two rows and writes two, backward
// reads four and writes two, and every element is held in registers between
// the row sums, so each is read once.
#include "hc_ffn.h"
#include "hc_internal.h"

namespace hc {

// Sums of N values over the W waves that share a row; every thread of them
// gets the same bits: each wave's butterfly, then the wave sums in order.
// red: this row group's LDS, one use per call site and row parity.
template <int W, int N>
__device__ __forceinline__ void row_sums(float* v, float* red, int wave, int lane) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_allsum(v[i]);
  if constexpr (W > 1) {
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) red[wave * N + i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = red[i];
    for (int w = 1; w < W; ++w)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = v[i] + red[w * N + i];
  }
}

__device__ __forceinline__ float rinv_rms(float ss, int H, float eps) { return 1.0f / sqrtf(ss / (float)H + eps); }

// One row per W waves; lane-chunk i of a row's thread t is chunk t + 64 W i
// (eight elements), NV of them at most.
template <DT D, bool ALN, int W, int NV>
__global__ __launch_bounds__(W > 4 ? 64 * W : 256) void k_norm(const NormArgs a) {
  constexpr int RPB = W > 4 ? 1 : 4 / W;  // rows per workgroup
  __shared__ float red[2 * W];
  const int lane = threadIdx.x & 63, wave = (threadIdx.x >> 6) % W;
  const int t = 64 * wave + lane;
  const int64_t m = (int64_t)blockIdx.x * RPB + (threadIdx.x >> 6) / W;
  if (W < 4 && m >= a.rows) return;  // wave-uniform; rows that share a workgroup share no LDS (W == 1)
  const int H = a.hidden, nch = (H + 7) >> 3;
  const int64_t row = m * H;

  float y[NV][8], r[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int ch = t + 64 * W * i, h = 8 * ch;
    if (ch < nch) {
      load8<D, ALN>(a.y, row + h, H - h, y[i]);
      if (a.res) load8<D, ALN>(a.res, row + h, H - h, r[i]);
    }
    if (ch >= nch || !a.res) {
#pragma unroll
      for (int e = 0; e < 8; ++e) r[i][e] = 0.0f;
    }
    if (ch >= nch) {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[i][e] = 0.0f;
    }
  }
  float coef = a.alpha;
  if (a.gate_kind == 1) coef = coef * ld<D>(a.gate, m * a.gate_stride);
  float ry = 1.0f;
  if (a.post_norm) {
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(y[i][e], y[i][e], ss);
    row_sums<W, 1>(&ss, red, wave, lane);
    ry = rinv_rms(ss, H, a.eps);
  }
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int ch = t + 64 * W * i, h = 8 * ch;
    if (ch < nch) {
      float w[8], g[8];
      if (a.post) load8<D, ALN>(a.post, h, H - h, w);
      if (a.gate_kind == 2) load8<D, ALN>(a.gate, row + h, H - h, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float z = y[i][e] * ry;
        if (a.post) z = z * w[e];
        if (a.gate_kind == 2) z = z * g[e];
        r[i][e] = fmaf(coef, z, r[i][e]);
        ss = fmaf(r[i][e], r[i][e], ss);
      }
      store8<D, ALN>(a.res_out, row + h, H - h, r[i]);
    }
  }
  if (!a.normed) return;  // uniform
  row_sums<W, 1>(&ss, red + W, wave, lane);
  const float rr = rinv_rms(ss, H, a.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int ch = t + 64 * W * i, h = 8 * ch;
    if (ch < nch) {
      float w[8];
      if (a.pre) load8<D, ALN>(a.pre, h, H - h, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        r[i][e] = r[i][e] * rr;
        if (a.pre) r[i][e] = r[i][e] * w[e];
      }
      store8<D, ALN>(a.normed, row + h, H - h, r[i]);
    }
  }
}

// Backward: workgroup b takes rows b, b + gridDim.x, ...; W waves per row,
// and the scales' gradient sums of its rows stay in registers until the end.
template <DT D, bool ALN, int W, int NV>
__global__ __launch_bounds__(64 * W) void k_norm_bwd(const NormArgs a) {
  __shared__ float red[2][5 * W];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, t = threadIdx.x;
  const int H = a.hidden, nch = (H + 7) >> 3;
  float apost[NV][8], apre[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) apost[i][e] = apre[i][e] = 0.0f;

  int parity = 0;
  for (int64_t m = blockIdx.x; m < a.rows; m += gridDim.x, parity ^= 1) {
    const int64_t row = m * H;
    float y[NV][8], r[NV][8], d[NV][8], n[NV][8];
    float s[3] = {0.0f, 0.0f, 0.0f};  // r'^2, t r', y^2
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int ch = t + 64 * W * i, h = 8 * ch;
#pragma unroll
      for (int e = 0; e < 8; ++e) y[i][e] = r[i][e] = d[i][e] = n[i][e] = 0.0f;
      if (ch < nch) {
        load8<D, ALN>(a.y, row + h, H - h, y[i]);
        load8<D, ALN>(a.res, row + h, H - h, r[i]);
        if (a.dres) load8<D, ALN>(a.dres, row + h, H - h, d[i]);
        if (a.dn) load8<D, ALN>(a.dn, row + h, H - h, n[i]);
      }
    }
    float coef = a.alpha;
    if (a.gate_kind == 1) coef = coef * ld<D>(a.gate, m * a.gate_stride);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int ch = t + 64 * W * i, h = 8 * ch;
      if (ch < nch) {
        float w[8];
        if (a.pre) load8<D, ALN>(a.pre, h, H - h, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float tt = a.pre ? n[i][e] * w[e] : n[i][e];
          s[0] = fmaf(r[i][e], r[i][e], s[0]);
          s[1] = fmaf(tt, r[i][e], s[1]);
          s[2] = fmaf(y[i][e], y[i][e], s[2]);
        }
      }
    }
    row_sums<W, 3>(s, red[parity], wave, lane);
    const float rr = rinv_rms(s[0], H, a.eps);
    const float cr = a.dn ? rr * rr * (s[1] / (float)H) : 0.0f;
    const float ry = a.post_norm ? rinv_rms(s[2], H, a.eps) : 1.0f;
    float u[2] = {0.0f, 0.0f};  // q y, z D
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int ch = t + 64 * W * i, h = 8 * ch;
      if (ch < nch) {
        float w[8], p[8], g[8];
        if (a.pre) load8<D, ALN>(a.pre, h, H - h, w);
        if (a.post) load8<D, ALN>(a.post, h, H - h, p);
        if (a.gate_kind == 2) load8<D, ALN>(a.gate, row + h, H - h, g);
        float dgate[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (a.dn) {
            const float tt = a.pre ? n[i][e] * w[e] : n[i][e];
            apre[i][e] = fmaf(n[i][e], r[i][e] * rr, apre[i][e]);
            d[i][e] = fmaf(rr, fmaf(-r[i][e], cr, tt), d[i][e]);
          }
          const float yh = y[i][e] * ry;
          const float z = a.post ? yh * p[e] : yh;
          const float zd = z * d[i][e];
          u[1] = u[1] + zd;
          dgate[e] = a.alpha * zd;
          float dz = coef * d[i][e];
          if (a.gate_kind == 2) dz = dz * g[e];
          apost[i][e] = fmaf(dz, yh, apost[i][e]);
          const float q = a.post ? dz * p[e] : dz;
          u[0] = fmaf(q, y[i][e], u[0]);
          n[i][e] = q;
        }
        if (a.d_residual) store8<D, ALN>(a.d_residual, row + h, H - h, d[i]);
        if (a.d_gate && a.gate_kind == 2) store8<D, ALN>(a.d_gate, row + h, H - h, dgate);
      }
    }
    if (a.post_norm || (a.d_gate && a.gate_kind == 1)) row_sums<W, 2>(u, red[parity] + 3 * W, wave, lane);
    if (a.d_gate && a.gate_kind == 1 && t == 0) st<D>(a.d_gate, m, a.alpha * u[1]);
    if (a.dy) {
      const float cy = a.post_norm ? ry * ry * (u[0] / (float)H) : 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int ch = t + 64 * W * i, h = 8 * ch;
        if (ch < nch) {
#pragma unroll
          for (int e = 0; e < 8; ++e) n[i][e] = ry * fmaf(-y[i][e], cy, n[i][e]);
          store8<D, ALN>(a.dy, row + h, H - h, n[i]);
        }
      }
    }
  }
  if (!a.partial) return;
  float* post = a.partial + (size_t)blockIdx.x * 2 * H;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int ch = t + 64 * W * i, h = 8 * ch;
    if (ch < nch) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (h + e < H) {
          post[h + e] = apost[i][e];
          post[H + h + e] = apre[i][e];
        }
    }
  }
}

// Four partial rows are added per thread in ascending order, 16 threads share
// a column, and their sums are added in thread order.
template <DT D>
__global__ __launch_bounds__(256) void k_column_sums(const float* __restrict__ partial, int nrows, int64_t pitch,
                                                     int64_t cols, void* out0, void* out1) {
  __shared__ float red[16][17];
  const int c = threadIdx.x & 15, g = threadIdx.x >> 4;
  const int64_t col = (int64_t)blockIdx.x * 16 + c;
  void* out = blockIdx.y ? out1 : out0;
  float s = 0.0f;
  if (col < cols) {
    const float* p = partial + blockIdx.y * cols + col;
    for (int r = g; r < nrows; r += 16) s = s + p[(int64_t)r * pitch];
  }
  red[g][c] = s;
  __syncthreads();
  if (g == 0 && col < cols && out) {
    s = red[0][c];
    for (int i = 1; i < 16; ++i) s = s + red[i][c];
    st<D>(out, col, s);
  }
}

__global__ __launch_bounds__(256) void k_zero(uint16_t* p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = 0;
}

// ------------------------------------------------------------------ launches

template <DT D, bool ALN> static hipError_t norm_fwd(const NormArgs& a, hipStream_t s) {
  const int nch = (a.hidden + 7) / 8;
  const unsigned rows = (unsigned)a.rows;
  if (nch <= 64 * 8 && a.rows >= 1024) {
    const dim3 grid((rows + 3) / 4);
    if (nch <= 64 * 4) return launch(nullptr, k_norm<D, ALN, 1, 4>, grid, dim3(256), 0, s, a);
    return launch(nullptr, k_norm<D, ALN, 1, 8>, grid, dim3(256), 0, s, a);
  }
  if (nch <= 256 * 2) return launch(nullptr, k_norm<D, ALN, 4, 2>, dim3(rows), dim3(256), 0, s, a);
  if (nch <= 1024 * 2) return launch(nullptr, k_norm<D, ALN, 16, 2>, dim3(rows), dim3(1024), 0, s, a);
  return launch(nullptr, k_norm<D, ALN, 16, 4>, dim3(rows), dim3(1024), 0, s, a);
}

hipError_t launch_norm(const NormArgs& a, int dtype, bool aligned, hipStream_t s) {
  if (dtype == 16) return aligned ? norm_fwd<DT::BF16, true>(a, s) : norm_fwd<DT::BF16, false>(a, s);
  if (dtype == 10) return aligned ? norm_fwd<DT::F16, true>(a, s) : norm_fwd<DT::F16, false>(a, s);
  return aligned ? norm_fwd<DT::F32, true>(a, s) : norm_fwd<DT::F32, false>(a, s);
}

int norm_backward_groups(int64_t rows) { return (int)(rows < 768 ? rows : 768); }

template <DT D, bool ALN> static hipError_t norm_bwd(const NormArgs& a, int groups, hipStream_t s) {
  const int nch = (a.hidden + 7) / 8;
  const dim3 grid((unsigned)groups);
  if (nch <= 256) return launch(nullptr, k_norm_bwd<D, ALN, 4, 1>, grid, dim3(256), 0, s, a);
  if (nch <= 512) return launch(nullptr, k_norm_bwd<D, ALN, 4, 2>, grid, dim3(256), 0, s, a);
  if (nch <= 1024) return launch(nullptr, k_norm_bwd<D, ALN, 16, 1>, grid, dim3(1024), 0, s, a);
  if (nch <= 2048) return launch(nullptr, k_norm_bwd<D, ALN, 16, 2>, grid, dim3(1024), 0, s, a);
  return launch(nullptr, k_norm_bwd<D, ALN, 16, 4>, grid, dim3(1024), 0, s, a);
}

hipError_t launch_norm_backward(const NormArgs& a, int dtype, bool aligned, int groups, hipStream_t s) {
  if (dtype == 16) return aligned ? norm_bwd<DT::BF16, true>(a, groups, s) : norm_bwd<DT::BF16, false>(a, groups, s);
  if (dtype == 10) return aligned ? norm_bwd<DT::F16, true>(a, groups, s) : norm_bwd<DT::F16, false>(a, groups, s);
  return aligned ? norm_bwd<DT::F32, true>(a, groups, s) : norm_bwd<DT::F32, false>(a, groups, s);
}

hipError_t launch_column_sums(const float* partial, int nrows, int64_t pitch, int64_t cols, void* out0, void* out1,
                              int dtype, hipStream_t s) {
  const dim3 grid((unsigned)((cols + 15) / 16), out1 ? 2 : 1);
  if (dtype == 16) return launch(nullptr, k_column_sums<DT::BF16>, grid, dim3(256), 0, s, partial, nrows, pitch, cols, out0, out1);
  if (dtype == 10) return launch(nullptr, k_column_sums<DT::F16>, grid, dim3(256), 0, s, partial, nrows, pitch, cols, out0, out1);
  return launch(nullptr, k_column_sums<DT::F32>, grid, dim3(256), 0, s, partial, nrows, pitch, cols, out0, out1);
}

hipError_t launch_zero(void* p, size_t n, hipStream_t s) {
  const int64_t c = (int64_t)(n / 2);
  if (c == 0) return hipSuccess;
  return launch(nullptr, k_zero, dim3((unsigned)(c > 65536 * 256 ? 65536 : (c + 255) / 256)), dim3(256), 0, s,
                (uint16_t*)p, c);
}

}  // namespace hc
