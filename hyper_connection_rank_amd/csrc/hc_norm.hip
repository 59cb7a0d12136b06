// residual_norm: the norms before and after a block, fused with the block's
// gate and residual scale, and its backward pass.
//
//   z = (post_norm ? y * ry : y) * post,   r' = res + alpha * gate * z,
//   n = (r' * rr) * pre,   ry = 1 / sqrt(mean y^2 + eps), rr likewise of r'.
//
// Backward, with D the gradient of r', t = dn * pre and p = D * post (* gate per element):
//   D  = dr' + rr * (t - r' * rr^2 * mean(t * r'))
//   dy = coef * ry * (p - y * ry^2 * mean(p * y))  (post_norm; else coef * p),
//   with coef = alpha (* gate per row);
//   d_res = D; d_gate = alpha * z * D, for a gate per row alpha * ry * sum(p * y);
//   d_post = sum over rows of coef * ry * D * y (* gate per element);
//   d_pre  = sum over rows of dn * r' * rr.
// So a row needs three sums (r'^2, t r', y^2) and then one (p y).
//
// Both are bounded by HBM: forward reads two rows and writes two, backward reads four and
// writes two. Every element is read once and held in registers between the row sums, in its
// stored form. A row is shared by as many waves as it has 64 chunks of eight elements (up to
// eight waves; then two and four chunks a thread), so no lane is idle for want of a power of
// two. Workgroups stay for several rows (persistent grid) and load the next row's elements
// before they work on the current one, so that the row sums' latency does not empty the
// memory pipeline; the scales are loaded once.
// Measured: forward 8192 x 2560 bf16 30 us (5.6 TB/s; a copy reaches 6.1), 8192 x 4096 fp16 46
// (5.8); backward 8192 x 4096 fp16 69 us and 5 for the scales' gradients (5.4), 8192 x 2560
// bf16 61 (4.1), 1021 x 2057 fp32 22 and 6 (2.4). Rows that are not 16-byte aligned are read and
// written under a condition per chunk, so that the compiler waits for everything in flight (see
// RowChunks): 8192 x 2057 bf16 33 us forward (4.1) and 90 backward (2.2).
#include "hc_ffn.h"
#include "hc_internal.h"

#include <algorithm>

namespace hc {

constexpr int MAX_WAVES = 16;

// Sums of N values over the W waves that share a row; every thread of them
// gets the same bits: each wave's butterfly, then the wave sums in order.
// red: LDS that no wave can still be reading (see the callers).
template <bool ONE, int N>
__device__ __forceinline__ void row_sums(float* v, float* red, int W, int wave, int lane) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_allsum(v[i]);
  if constexpr (!ONE) {
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) red[wave * N + i] = v[i];
    }
    // Only LDS is waited for: the next row's loads stay in flight.
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = red[i];
    for (int w = 1; w < W; ++w)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = v[i] + red[w * N + i];
  }
}

__device__ __forceinline__ float rinv_rms(float ss, float inv_h, float eps) { return 1.0f / sqrtf(fmaf(ss, inv_h, eps)); }

// A thread's chunks of one row. Aligned rows go through a buffer descriptor of the row, so
// that no access is conditional: lanes past the row's end, a row that does not exist (live
// false) and a tensor that is not given read zeros and write nothing. The compiler can then
// count the operations in flight, and a wait for the next row's loads does not also wait for
// this row's stores (which took a row from about 2 us to 4.5).
template <DT D, bool ALN, int NV> struct RowChunks {
  static constexpr int ES = D == DT::F32 ? 4 : 2;
  Raw8<D> c[NV];

  __device__ __forceinline__ void load(const void* base, int64_t row, int H, int t, int stride, bool live = true) {
    if constexpr (ALN) {
      const rsrc_t r = make_rsrc((const char*)base + row * ES, base && live ? H * ES : 0);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int o = 8 * ES * (t + stride * i);
        c[i].v = __builtin_amdgcn_raw_buffer_load_b128(r, o, 0, 2);  // non-temporal: read once
        if constexpr (D == DT::F32) c[i].w = __builtin_amdgcn_raw_buffer_load_b128(r, o + 16, 0, 2);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int h = 8 * (t + stride * i);
        c[i] = base && live && h < H ? load_raw8<D>(base, row + h, H - h) : zero_raw8<D>();
      }
    }
  }
  // As load(), with ones for a tensor that is not given.
  __device__ __forceinline__ void load_scale(const void* base, int H, int t, int stride) {
    load(base, 0, H, t, stride);
    if (!base) {
      constexpr uint32_t one = D == DT::F32 ? 0x3F800000u : D == DT::BF16 ? 0x3F803F80u : 0x3C003C00u;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        c[i].v = u32x4{one, one, one, one};
        if constexpr (D == DT::F32) c[i].w = c[i].v;
      }
    }
  }
  // Makes the compiler unpack the chunks again where they are used next, instead of keeping
  // their fp32 values (twice the registers of 16-bit T) from one pass to the other.
  __device__ __forceinline__ void renew() {
    if constexpr (D != DT::F32) {
#pragma unroll
      for (int i = 0; i < NV; ++i) asm volatile("" : "+v"(c[i].v));
    }
  }
};
// Rounds a row's values x and stores them.
template <DT D, bool ALN, int NV>
__device__ __forceinline__ void store_row(void* base, int64_t row, int H, int t, int stride, const float (*x)[8]) {
  constexpr int ES = D == DT::F32 ? 4 : 2;
  if constexpr (ALN) {
    const rsrc_t r = make_rsrc((const char*)base + row * ES, base ? H * ES : 0);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int o = 8 * ES * (t + stride * i);
      if constexpr (D == DT::F32) {
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, f32x4{x[i][0], x[i][1], x[i][2], x[i][3]}), r, o, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, f32x4{x[i][4], x[i][5], x[i][6], x[i][7]}), r, o + 16, 0, 0);
      } else {
        __builtin_amdgcn_raw_buffer_store_b128(to_u32x4(pack8<D>(x[i])), r, o, 0, 0);
      }
    }
  } else if (base) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int h = 8 * (t + stride * i);
      if (h < H) store8<D, ALN>(base, row + h, H - h, x[i]);
    }
  }
}

// Row m's gate as it is stored (0 without a gate per row and past the last row). The load is
// unconditional and its value is first looked at a row later: a wait for it here would also
// wait for the row loads issued before it.
template <DT D> __device__ __forceinline__ uint32_t load_row_gate(const NormArgs& a, int64_t m) {
  constexpr int ES = D == DT::F32 ? 4 : 2;
  const rsrc_t r = make_rsrc((const char*)a.gate + m * a.gate_stride * ES, a.gate_kind == 1 && m < a.rows ? ES : 0);
  if constexpr (D == DT::F32) return __builtin_amdgcn_raw_buffer_load_b32(r, 0, 0, 0);
  else return __builtin_amdgcn_raw_buffer_load_b16(r, 0, 0, 0);
}
// alpha times the row's gate.
template <DT D> __device__ __forceinline__ float row_coef(const NormArgs& a, uint32_t gate) {
  if (a.gate_kind != 1) return a.alpha;
  if constexpr (D == DT::F32) return a.alpha * __uint_as_float(gate);
  else return a.alpha * widen<D>(gate);
}

// A workgroup's place: ONE: four rows per workgroup, a wave each (no LDS shared); otherwise
// one row for all of its waves.
struct NormPlace {
  int lane, W, wave, sub, t, stride;
  int64_t first, step;
};
template <bool ONE> __device__ __forceinline__ NormPlace norm_place() {
  NormPlace p;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  p.lane = threadIdx.x & 63;
  p.W = ONE ? 1 : (int)(blockDim.x >> 6);
  p.wave = ONE ? 0 : wv;
  p.sub = ONE ? wv : 0;
  p.t = 64 * p.wave + p.lane;
  p.stride = 64 * p.W;
  p.first = ONE ? (int64_t)blockIdx.x * 4 + wv : (int64_t)blockIdx.x;
  p.step = (int64_t)gridDim.x * (ONE ? 4 : 1);
  return p;
}

// NV: chunks of a thread; chunk i of thread t is chunk t + 64 W i of the row.
// AHEAD: the next row is loaded while the current one is worked on (where registers allow).
// GE: a gate per element.
template <DT D, bool ALN, int NV, bool ONE, bool AHEAD, bool GE>
__global__ __launch_bounds__(ONE ? 256 : NV == 1 ? 512 : 1024) void k_norm(const NormArgs a) {
  __shared__ float red[2][2 * MAX_WAVES];
  const NormPlace pl = norm_place<ONE>();
  const int H = a.hidden, t = pl.t, S = pl.stride;
  const float inv_h = 1.0f / (float)H;
  RowChunks<D, ALN, NV> post, pre, y, r;
  post.load_scale(a.post, H, t, S);
  pre.load_scale(a.pre, H, t, S);
  int64_t m = pl.first;
  uint32_t row_gate = load_row_gate<D>(a, m);
  if constexpr (AHEAD) {
    y.load(a.y, m * H, H, t, S, m < a.rows);
    r.load(a.res, m * H, H, t, S, m < a.rows);
  }
  // A row's sums use red[parity]: a wave writes them again two rows later, after the barrier
  // of the row between, which every wave passes after its last read of this row's.
  for (int parity = 0; m < a.rows; m += pl.step, parity ^= 1) {
    const int64_t row = m * H, next = m + pl.step;
    RowChunks<D, ALN, NV> ny, nr, gate;
    // Loads complete in order: this row's gate goes before the next row's elements, and the
    // next row's coefficient with them.
    if constexpr (GE) gate.load(a.gate, row, H, t, S);
    if constexpr (!AHEAD) {
      y.load(a.y, row, H, t, S);
      r.load(a.res, row, H, t, S);
    } else {
      ny.load(a.y, next * H, H, t, S, next < a.rows);
      nr.load(a.res, next * H, H, t, S, next < a.rows);
    }
    const float coef = row_coef<D>(a, row_gate);
    row_gate = load_row_gate<D>(a, next);
    float c = coef;
    if (a.post_norm) {
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float x[8];
        unpack_raw8<D>(y.c[i], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
      }
      row_sums<ONE, 1>(&ss, red[parity], pl.W, pl.wave, pl.lane);
      c = coef * rinv_rms(ss, inv_h, a.eps);
      y.renew();
    }
    float o[NV][8], ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float x[8], w[8], g[8];
      unpack_raw8<D>(y.c[i], x);
      unpack_raw8<D>(r.c[i], o[i]);
      unpack_raw8<D>(post.c[i], w);
      if constexpr (GE) unpack_raw8<D>(gate.c[i], g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float z = x[e] * w[e];
        if constexpr (GE) z = z * g[e];
        o[i][e] = fmaf(c, z, o[i][e]);
        ss = fmaf(o[i][e], o[i][e], ss);
      }
    }
    store_row<D, ALN, NV>(a.res_out, row, H, t, S, o);
    if (a.normed) {
      row_sums<ONE, 1>(&ss, red[parity] + MAX_WAVES, pl.W, pl.wave, pl.lane);
      const float rr = rinv_rms(ss, inv_h, a.eps);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float w[8];
        unpack_raw8<D>(pre.c[i], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[i][e] = (o[i][e] * rr) * w[e];
      }
      store_row<D, ALN, NV>(a.normed, row, H, t, S, o);
    }
    if constexpr (AHEAD) {
      y = ny;
      r = nr;
    }
  }
}

// Backward: the scales' gradient sums of a workgroup's rows stay in registers until the end.
// A gradient or scale that is not given reads as zeros or ones, and costs no branch.
template <DT D, bool ALN, int NV, bool ONE, int WAVES, bool AHEAD, bool GE>
__global__ __launch_bounds__(ONE ? 256 : 64 * WAVES) void k_norm_bwd(const NormArgs a) {
  __shared__ float red[2][4 * MAX_WAVES];
  const NormPlace pl = norm_place<ONE>();
  const int H = a.hidden, t = pl.t, S = pl.stride, sub = pl.sub;
  const float inv_h = 1.0f / (float)H;
  float apost[NV][8], apre[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) apost[i][e] = apre[i][e] = 0.0f;

  RowChunks<D, ALN, NV> post, pre, y, r, d, n;
  post.load_scale(a.post, H, t, S);
  pre.load_scale(a.pre, H, t, S);
  int64_t m = pl.first;
  uint32_t row_gate = load_row_gate<D>(a, m);
  if constexpr (AHEAD) {
    y.load(a.y, m * H, H, t, S, m < a.rows);
    r.load(a.res, m * H, H, t, S, m < a.rows);
    d.load(a.dres, m * H, H, t, S, m < a.rows);
    n.load(a.dn, m * H, H, t, S, m < a.rows);
  }
  for (int parity = 0; m < a.rows; m += pl.step, parity ^= 1) {  // red[parity]: see k_norm
    const int64_t row = m * H, next = m + pl.step;
    RowChunks<D, ALN, NV> ny, nr, nd, nn, gate;
    if constexpr (GE) gate.load(a.gate, row, H, t, S);
    if constexpr (!AHEAD) {
      y.load(a.y, row, H, t, S);
      r.load(a.res, row, H, t, S);
      d.load(a.dres, row, H, t, S);
      n.load(a.dn, row, H, t, S);
    } else {
      ny.load(a.y, next * H, H, t, S, next < a.rows);
      nr.load(a.res, next * H, H, t, S, next < a.rows);
      nd.load(a.dres, next * H, H, t, S, next < a.rows);
      nn.load(a.dn, next * H, H, t, S, next < a.rows);
    }
    const float coef = row_coef<D>(a, row_gate);
    row_gate = load_row_gate<D>(a, next);
    float s[3] = {0.0f, 0.0f, 0.0f};  // r'^2, t r', y^2
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float yv[8], rv[8], nv[8], w[8];
      unpack_raw8<D>(y.c[i], yv);
      unpack_raw8<D>(r.c[i], rv);
      unpack_raw8<D>(n.c[i], nv);
      unpack_raw8<D>(pre.c[i], w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s[0] = fmaf(rv[e], rv[e], s[0]);
        s[1] = fmaf(nv[e] * w[e], rv[e], s[1]);
        s[2] = fmaf(yv[e], yv[e], s[2]);
      }
    }
    row_sums<ONE, 3>(s, red[parity], pl.W, pl.wave, pl.lane);
    y.renew();
    r.renew();
    n.renew();
    const float rr = rinv_rms(s[0], inv_h, a.eps);
    const float cr = rr * (rr * (rr * (s[1] * inv_h)));  // in this order rr^3 of tiny or huge rows stays in range
    const float ry = a.post_norm ? rinv_rms(s[2], inv_h, a.eps) : 1.0f;
    const float cp = coef * ry;
    float u = 0.0f;  // p y
    float q[NV][8], dv[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float yv[8], rv[8], nv[8], w[8], p[8], g[8], dgate[8];
      unpack_raw8<D>(y.c[i], yv);
      unpack_raw8<D>(r.c[i], rv);
      unpack_raw8<D>(n.c[i], nv);
      unpack_raw8<D>(d.c[i], dv[i]);
      unpack_raw8<D>(pre.c[i], w);
      unpack_raw8<D>(post.c[i], p);
      if constexpr (GE) unpack_raw8<D>(gate.c[i], g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float nr_ = nv[e] * rr;
        apre[i][e] = fmaf(nr_, rv[e], apre[i][e]);
        dv[i][e] = fmaf(-rv[e], cr, fmaf(nr_, w[e], dv[i][e]));
        float dy_ = dv[i][e] * yv[e];
        q[i][e] = dv[i][e] * p[e];
        if constexpr (GE) {
          dgate[e] = a.alpha * ry * (q[i][e] * yv[e]);
          dy_ = dy_ * g[e];
          q[i][e] = q[i][e] * g[e];
        }
        apost[i][e] = fmaf(dy_, cp, apost[i][e]);
        u = fmaf(q[i][e], yv[e], u);
      }
      if constexpr (GE) store_row<D, ALN, 1>(a.d_gate, row, H, t + S * i, S, &dgate);
    }
    store_row<D, ALN, NV>(a.d_residual, row, H, t, S, dv);
    row_sums<ONE, 1>(&u, red[parity] + 3 * MAX_WAVES, pl.W, pl.wave, pl.lane);
    y.renew();
    if (!GE && a.d_gate && t == 0) st<D>(a.d_gate, m, a.alpha * ry * u);
    const float cy = a.post_norm ? ry * (ry * (u * inv_h)) : 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float yv[8];
      unpack_raw8<D>(y.c[i], yv);
#pragma unroll
      for (int e = 0; e < 8; ++e) q[i][e] = cp * fmaf(-yv[e], cy, q[i][e]);
    }
    store_row<D, ALN, NV>(a.dy, row, H, t, S, q);
    if constexpr (AHEAD) {
      y = ny;
      r = nr;
      d = nd;
      n = nn;
    }
  }
  if (!a.d_post && !a.d_pre) return;
  if constexpr (ONE) {  // the four waves' sums, in wave order (H <= 512 here)
    __shared__ float add[4][2][512];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        add[sub][0][8 * (t + S * i) + e] = apost[i][e];
        add[sub][1][8 * (t + S * i) + e] = apre[i][e];
      }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * H; c += 256) {
      const int k = c >= H, h = c - k * H;
      float v = add[0][k][h];
#pragma unroll
      for (int j = 1; j < 4; ++j) v = v + add[j][k][h];
      void* out = k ? a.d_pre : a.d_post;
      if (gridDim.x > 1) a.partial[(size_t)blockIdx.x * 2 * H + c] = v;
      else if (out) st<D>(out, h, v);
    }
  } else {
    float* part = a.partial + (size_t)blockIdx.x * 2 * H;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int h = 8 * (t + S * i);
      if (h < H) {
        if (gridDim.x == 1) {
          if (a.d_post) store8<D, ALN>(a.d_post, h, H - h, apost[i]);
          if (a.d_pre) store8<D, ALN>(a.d_pre, h, H - h, apre[i]);
        } else {
          store8<DT::F32, false>(part, h, H - h, apost[i]);
          store8<DT::F32, false>(part, H + h, H - h, apre[i]);
        }
      }
    }
  }
}

// 16 lanes of VEC columns each per workgroup, 64 threads per column group; each adds every
// 64th row, eight loads at a time, and their sums are added in thread order. (Eight loads at
// once: a row after the other costs a memory latency each, 29 us for 768 rows.)
template <DT D, int VEC>
__global__ __launch_bounds__(1024) void k_column_sums(const float* __restrict__ partial, int nrows, int64_t pitch,
                                                      int64_t cols, void* out0, void* out1) {
  typedef float vec_t __attribute__((ext_vector_type(VEC)));
  __shared__ vec_t red[64][17];
  const int c = threadIdx.x & 15, g = threadIdx.x >> 4;
  const int64_t col = ((int64_t)blockIdx.x * 16 + c) * VEC;
  void* out = blockIdx.y ? out1 : out0;
  if (!out) return;  // the whole workgroup
  vec_t s = 0.0f;
  if (col < cols) {
    const float* p = partial + blockIdx.y * cols + col;
    for (int r = g; r < nrows; r += 512) {
      vec_t v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = *(const vec_t*)(p + (int64_t)min(r + 64 * i, nrows - 1) * pitch);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (r + 64 * i < nrows) s = s + v[i];
    }
  }
  red[g][c] = s;
  __syncthreads();
  // 16 lanes x VEC columns: one thread each, 64 sums
  if ((int)threadIdx.x < 16 * VEC) {
    const int cc = threadIdx.x / VEC, e = threadIdx.x % VEC;
    const int64_t k = ((int64_t)blockIdx.x * 16 + cc) * VEC + e;
    if (k < cols) {
      float v = red[0][cc][e];
      for (int i = 1; i < 64; ++i) v = v + red[i][cc][e];
      st<D>(out, k, v);
    }
  }
}

__global__ __launch_bounds__(256) void k_zero(uint16_t* p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = 0;
}

// ------------------------------------------------------------------ launches

// Waves that share a row: rows of up to 512 elements one each, four to a workgroup; above,
// one chunk a thread up to eight waves, then two and four chunks. Backward keeps eight waves
// up to 16384 elements: with sixteen a thread has 128 registers instead of 256 (8192 columns: 161
// us against 102). Up to two chunks a thread the registers suffice. Four (backward above 8192
// columns) need more than there are: 224 to 660 bytes a thread go to scratch with eight waves and
// 764 to 1232 with sixteen (above 16384 columns). In bf16 3200 x 10240 takes 218 us (1.8 TB/s),
// 2000 x 16384 193 (2.0) and 1000 x 32768 443 (0.9). Forward four chunks (above 16384 columns) spill
// 80 to 216 bytes in fp32 and 24 to 48 with a gate per element (1000 x 32768: fp32 121 us, 4.3
// TB/s; bf16 52, 5.1).
struct NormShape {
  int nv, waves, threads, rows;  // rows per workgroup
};
static NormShape norm_shape(int64_t hidden, bool backward) {
  const int nch = (int)((hidden + 7) / 8);
  if (nch <= 64) return {1, 1, 256, 4};
  const int nv = nch <= 512 ? 1 : nch <= (backward ? 1024 : 2048) ? 2 : 4;
  const int w = (nch + 64 * nv - 1) / (64 * nv);
  return {nv, w, 64 * w, 1};
}

// Workgroups: at most `most`, and no more than share the rows evenly.
static int norm_groups(int64_t rows, int per_group, int64_t most) {
  const int64_t sets = (rows + per_group - 1) / per_group;
  const int64_t turns = (sets + most - 1) / most;
  return (int)((sets + turns - 1) / turns);
}

template <typename K> static hipError_t run_norm(const NormArgs& a, unsigned groups, int threads, K k, K kg, hipStream_t s) {
  return launch(nullptr, a.gate_kind == 2 ? kg : k, dim3(groups), dim3((unsigned)threads), 0, s, a);
}

template <DT D, bool ALN> static hipError_t norm_fwd(const NormArgs& a, hipStream_t s) {
  const NormShape sh = norm_shape(a.hidden, false);
  // Persistent: up to 24 waves per compute unit (their rows and the next ones are in flight).
  const unsigned g = (unsigned)norm_groups(a.rows, sh.rows, 256 * std::max(1, 24 / (sh.waves * sh.rows)));
  if (sh.waves == 1) return run_norm(a, g, sh.threads, k_norm<D, ALN, 1, true, true, false>, k_norm<D, ALN, 1, true, true, true>, s);
  if (sh.nv == 1) return run_norm(a, g, sh.threads, k_norm<D, ALN, 1, false, true, false>, k_norm<D, ALN, 1, false, true, true>, s);
  if (sh.nv == 2) return run_norm(a, g, sh.threads, k_norm<D, ALN, 2, false, D != DT::F32, false>, k_norm<D, ALN, 2, false, D != DT::F32, true>, s);
  return run_norm(a, g, sh.threads, k_norm<D, ALN, 4, false, false, false>, k_norm<D, ALN, 4, false, false, true>, s);
}

hipError_t launch_norm(const NormArgs& a, int dtype, bool aligned, hipStream_t s) {
  if (dtype == 16) return aligned ? norm_fwd<DT::BF16, true>(a, s) : norm_fwd<DT::BF16, false>(a, s);
  if (dtype == 10) return aligned ? norm_fwd<DT::F16, true>(a, s) : norm_fwd<DT::F16, false>(a, s);
  return aligned ? norm_fwd<DT::F32, true>(a, s) : norm_fwd<DT::F32, false>(a, s);
}

// Up to 4 rows one workgroup takes them all and writes the scales' gradients itself: one
// launch less. Above, every group adds 2 * hidden fp32 sums of traffic.
static int64_t backward_most(const NormShape& sh) { return 256 * std::max(1, std::min(4, 16 / (sh.waves * sh.rows))); }
static int norm_backward_groups(int64_t rows, int64_t hidden) {
  if (rows <= 4) return 1;
  const NormShape sh = norm_shape(hidden, true);
  return norm_groups(rows, sh.rows, backward_most(sh));
}
int norm_backward_most_groups(int64_t rows, int64_t hidden) {
  if (rows <= 4) return 1;
  const NormShape sh = norm_shape(hidden, true);
  return (int)std::min((rows + sh.rows - 1) / sh.rows, backward_most(sh));
}

template <DT D, bool ALN, int NV, bool ONE, int WAVES, bool AHEAD>
static hipError_t norm_bwd_as(const NormArgs& a, int groups, int threads, hipStream_t s) {
  return run_norm(a, (unsigned)groups, threads, k_norm_bwd<D, ALN, NV, ONE, WAVES, AHEAD, false>,
                  k_norm_bwd<D, ALN, NV, ONE, WAVES, AHEAD, true>, s);
}
template <DT D, bool ALN> static hipError_t norm_bwd(const NormArgs& a, int groups, hipStream_t s) {
  const NormShape sh = norm_shape(a.hidden, true);
  if (sh.waves == 1) return norm_bwd_as<D, ALN, 1, true, 4, true>(a, groups, sh.threads, s);
  if (sh.nv == 1) return norm_bwd_as<D, ALN, 1, false, 8, true>(a, groups, sh.threads, s);
  if (sh.nv == 2) return norm_bwd_as<D, ALN, 2, false, 8, false>(a, groups, sh.threads, s);
  if (sh.waves <= 8) return norm_bwd_as<D, ALN, 4, false, 8, false>(a, groups, sh.threads, s);
  return norm_bwd_as<D, ALN, 4, false, 16, false>(a, groups, sh.threads, s);
}

hipError_t launch_norm_backward(const NormArgs& a, int dtype, bool aligned, hipStream_t s) {
  const int groups = norm_backward_groups(a.rows, a.hidden);
  hipError_t e;
  if (dtype == 16) e = aligned ? norm_bwd<DT::BF16, true>(a, groups, s) : norm_bwd<DT::BF16, false>(a, groups, s);
  else if (dtype == 10) e = aligned ? norm_bwd<DT::F16, true>(a, groups, s) : norm_bwd<DT::F16, false>(a, groups, s);
  else e = aligned ? norm_bwd<DT::F32, true>(a, groups, s) : norm_bwd<DT::F32, false>(a, groups, s);
  if (e != hipSuccess || groups == 1 || (!a.d_post && !a.d_pre)) return e;
  return launch_column_sums(a.partial, groups, 2 * (int64_t)a.hidden, a.hidden, a.d_post, a.d_pre, dtype, s);
}

hipError_t launch_column_sums(const float* partial, int nrows, int64_t pitch, int64_t cols, void* out0, void* out1,
                              int dtype, hipStream_t s) {
  const bool vec = cols % 4 == 0 && pitch % 4 == 0;  // scratch itself is 16-byte aligned
  const dim3 grid((unsigned)((cols + (vec ? 63 : 15)) / (vec ? 64 : 16)), out1 ? 2 : 1);
  auto run = [&](auto k4, auto k1) {
    return vec ? launch(nullptr, k4, grid, dim3(1024), 0, s, partial, nrows, pitch, cols, out0, out1)
               : launch(nullptr, k1, grid, dim3(1024), 0, s, partial, nrows, pitch, cols, out0, out1);
  };
  if (dtype == 16) return run(k_column_sums<DT::BF16, 4>, k_column_sums<DT::BF16, 1>);
  if (dtype == 10) return run(k_column_sums<DT::F16, 4>, k_column_sums<DT::F16, 1>);
  return run(k_column_sums<DT::F32, 4>, k_column_sums<DT::F32, 1>);
}

hipError_t launch_zero(void* p, size_t n, hipStream_t s) {
  const int64_t c = (int64_t)(n / 2);
  if (c == 0) return hipSuccess;
  return launch(nullptr, k_zero, dim3((unsigned)(c > 65536 * 256 ? 65536 : (c + 255) / 256)), dim3(256), 0, s,
                (uint16_t*)p, c);
}

}  // namespace hc
