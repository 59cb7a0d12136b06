// Matrix products with fused epilogues: hclrmix_linear and hclrmix_glu and the
// products of their backward passes.
//
// Every product is out[m][n] = sum over k of P(m, k) Q(k, n), where each operand's
// contraction index k runs either along its rows in memory ("direct") or down its
// columns ("transposed"):
//   forward   x [M, K] direct,        W [K, N] transposed
//   dx        dz [M, N] direct,       W [K, N] direct (contraction over N)
//   dW        x [M, K] transposed,    dz [M, N] transposed (contraction over M)
// A workgroup computes a BM x BN tile with 16x16x32 matrix-core steps. Both
// operands' tiles go through LDS in the order they have in memory, 16-byte chunks
// permuted inside a row so that the fragment reads spread over the banks; a
// transposed operand's fragments come from the transposing LDS read.
//
// The matrix op is given Q's fragment as its first operand, so a lane's result
// holds four consecutive columns n of one row m: bias, residual and the stores of
// the epilogue are then one 8-byte access per four elements.
//
// Few tiles: the contraction is split over workgroups. Each writes its fp32 tile
// to scratch with agent-coherent stores and counts itself in; the last one adds
// the parts in ascending order, whichever order they arrived in, and runs the
// epilogue.
#include "hc_ffn.h"
#include "hc_internal.h"

#include "../../include/hclrmix.h"

#include <algorithm>

namespace hc {

// Most workgroup tiles of a product whose contraction is split: one arrival
// counter each in the workspace's prefix.
constexpr int MAX_SPLIT_TILES = HCLRMIX_COUNTER_BYTES / 4;

// Kernel arguments: a Product and its schedule.
struct Gemm {
  const void* p[2];
  const void* q[2];
  int64_t ldp, ldq, ldr;
  int64_t M;
  int N, K;
  const void* bias[2];
  const void* residual;
  void* out[2];
  void* save[2];
  int act, segments;
  int tiles_m, tiles_n, splits;
  int vec4;         // four consecutive columns of every [M, N] tensor and bias are 4-element aligned
  float* partial;   // [tile][split][BM * BN] fp32 (splits > 1)
  unsigned* counters;
};

// Counter i sits in line i % 32 of the 4 KB prefix.
__device__ __forceinline__ unsigned* counter_at(unsigned* base, int i) { return base + (i & 31) * 32 + (i >> 5); }

// Chunk permutation of an LDS row: the slot that holds chunk c of row r (and the
// chunk that slot c holds). Direct tiles (rows of BK): a fragment read takes one
// chunk of 16 consecutive rows, so the low three bits of c change with r.
// Transposed tiles (rows of R columns): a transposing read takes 32 bytes of rows
// r .. r+3 and r+8 .. r+11 in one half wave, so whole 32-byte units move with r.
template <bool TR, int CPR> __device__ __forceinline__ int swz(int r, int c) {
  if constexpr (!TR) {
    return c ^ (r & 7);
  } else if constexpr (CPR >= 16) {
    return c ^ (((r & 3) | ((r >> 1) & 4)) << 1);
  } else {
    return c ^ ((((r >> 1) & 1) | ((r >> 2) & 2)) << 1);
  }
}

// One operand's tile: R indices of the output by BK of the contraction.
template <DT D, bool TR, int R, int BK, int THREADS> struct Tile {
  static constexpr int CPR = (TR ? R : BK) / 8;  // 16-byte chunks per LDS row
  static constexpr int ROWS = TR ? BK : R;
  static constexpr int NI = ROWS * CPR / THREADS;  // chunks a thread stages
  static constexpr int BYTES = ROWS * CPR * 16;
  static_assert(ROWS * CPR % THREADS == 0 && CPR >= 8, "tile shape");

  // Reads this thread's chunks of the tile at output index r0 and contraction
  // index k0 of an operand with nr output indices and K contraction indices.
  template <bool ALN>
  static __device__ __forceinline__ void fetch(const void* base, int64_t ld, int64_t r0, int64_t nr, int k0, int K,
                                               int tid, uint4* v) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int c = i * THREADS + tid, row = c / CPR, ch = c % CPR;
      const int64_t mr = TR ? (int64_t)k0 + row : r0 + row;        // memory row
      const int64_t mc = TR ? r0 + 8 * ch : (int64_t)k0 + 8 * ch;  // memory column
      const int64_t left = (TR ? nr : (int64_t)K) - mc;            // columns from here on
      const bool in = mr < (TR ? (int64_t)K : nr) && left > 0;
      const uint16_t* src = (const uint16_t*)base + mr * ld + mc;
      v[i] = make_uint4(0u, 0u, 0u, 0u);
      if (in) {
        if (ALN || left >= 8) {
          v[i] = ld16<D, ALN>(src);
        } else {
          uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
          for (int e = 0; e < 7; ++e)
            if (e < left) w[e >> 1] |= (uint32_t)src[e] << (16 * (e & 1));
          v[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
  }
  static __device__ __forceinline__ void put(unsigned char* lds, int tid, const uint4* v) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int c = i * THREADS + tid, row = c / CPR, ch = c % CPR;
      *(uint4*)(lds + (row * CPR + swz<TR, CPR>(row, ch)) * 16) = v[i];
    }
  }
  // Fragment of output indices r .. r+15 and contraction indices k .. k+31: lane l
  // holds (r + l % 16, k + 8 (l / 16) + 0..7).
  static __device__ __forceinline__ s16x8 frag(const unsigned char* lds, int r, int k, int lane) {
    const int g = lane >> 4, j = lane & 15;
    if constexpr (!TR) {
      const int row = r + j;
      return __builtin_bit_cast(s16x8, *(const uint4*)(lds + (row * CPR + swz<TR, CPR>(row, (k >> 3) + g)) * 16));
    } else {
      const int kr = k + 8 * g + (j >> 2), cb = j & 3;
      lds_u8* p = (lds_u8*)(lds + (kr * CPR + swz<TR, CPR>(kr, (r >> 3) + (cb >> 1))) * 16 + 8 * (cb & 1));
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * CPR * 16));
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  }
};

// ------------------------------------------------------------------ epilogue

// Four consecutive elements of a row, n of them valid.
template <DT D> __device__ __forceinline__ void ld4(const void* base, int64_t i, int n, bool vec, float* x) {
  if (vec && n >= 4) {
    if constexpr (D == DT::F32) {
      const f32x4 v = *(const f32x4*)((const float*)base + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = v[e];
    } else {
      unpack4<D>(*(const u32x2*)((const uint16_t*)base + i), x);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = e < n ? ld<D>(base, i + e) : 0.0f;
  }
}
template <DT D> __device__ __forceinline__ void st4(void* base, int64_t i, int n, bool vec, const float* x) {
  if (vec && n >= 4) {
    if constexpr (D == DT::F32) *(f32x4*)((float*)base + i) = f32x4{x[0], x[1], x[2], x[3]};
    else *(u32x2*)((uint16_t*)base + i) = u32x2{pack2<D>(x[0], x[1]), pack2<D>(x[2], x[3])};
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < n) st<D>(base, i + e, x[e]);
  }
}

// Columns n .. n+3 of row m: v (and u of a dual product) hold the fp32 sums.
template <DT D, bool DUAL>
__device__ __forceinline__ void finish4(const Gemm& a, int b, int64_t m, int n, float* v, float* u) {
  const int left = a.N - n;
  if (m >= a.M || left <= 0) return;
  const int64_t i = m * a.N + n;
  float t[4];
  if constexpr (DUAL) {
    if (a.bias[0]) {
      ld4<D>(a.bias[0], n, left, a.vec4, t);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = v[e] + t[e];
    }
    if (a.bias[1]) {
      ld4<D>(a.bias[1], n, left, a.vec4, t);
#pragma unroll
      for (int e = 0; e < 4; ++e) u[e] = u[e] + t[e];
    }
    if (a.save[0]) {
      st4<D>(a.save[0], i, left, a.vec4, v);
      st4<D>(a.save[1], i, left, a.vec4, u);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = act_f(a.act, v[e]) * u[e];
    st4<D>(a.out[0], i, left, a.vec4, v);
  } else {
    if (a.bias[0]) {
      ld4<D>(a.bias[0], n, left, a.vec4, t);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = v[e] + t[e];
    }
    if (a.save[0]) st4<D>(a.save[0], i, left, a.vec4, v);
    if (a.act != ACT_NONE) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = act_f(a.act, v[e]);
    }
    if (a.residual) {
      ld4<D>(a.residual, m * a.ldr + n, left, a.vec4, t);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = v[e] + t[e];
    }
    st4<D>(a.out[b], i, left, a.vec4, v);
  }
}

typedef __amdgpu_buffer_rsrc_t rsrc_t;
__device__ __forceinline__ rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00020000);
}
constexpr int AGENT = 16;  // sc1: the access is coherent across the chip's L2s

// Split sums: this workgroup's tile (NA vectors per thread) goes to scratch; the
// last of the tile's workgroups to arrive gets the sum of all parts in ascending
// order and true, the others false.
template <int NA, int THREADS>
__device__ __forceinline__ bool join_splits(const Gemm& a, int tile, int split, f32x4* acc, int tid) {
  __shared__ int is_last;
  constexpr uint32_t PART = NA * THREADS * 16;  // bytes of one part
  float* base = a.partial + (size_t)tile * a.splits * (PART / 4);
  {
    const rsrc_t r = make_rsrc((const char*)base + (size_t)split * PART, PART);
#pragma unroll
    for (int i = 0; i < NA; ++i)
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc[i]), r, (i * THREADS + tid) * 16, 0, AGENT);
  }
  // Each thread's stores have completed before any thread counts the workgroup in.
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  unsigned* counter = counter_at(a.counters, tile);
  if (tid == 0)
    is_last = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (unsigned)(a.splits - 1);
  __syncthreads();
  if (!is_last) return false;
  if (tid == 0) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);  // zero for the next call
#pragma unroll
  for (int i = 0; i < NA; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int s = 0; s < a.splits; ++s) {
    const rsrc_t r = make_rsrc((const char*)base + (size_t)s * PART, PART);
#pragma unroll
    for (int i = 0; i < NA; ++i)
      acc[i] = acc[i] + __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (i * THREADS + tid) * 16, 0, AGENT));
  }
  return true;
}

// Block id -> (batch, tile row, tile column, split). Consecutive block ids go to
// the eight XCDs in turn; each XCD gets a contiguous range of tiles, ordered so
// that workgroups running together share the operands' tiles in its L2: groups of
// eight tile rows, tile rows fastest, then tile columns.
struct Place {
  int b, tm, tn, split, tile;
};
__device__ __forceinline__ Place place(const Gemm& a) {
  const int total = gridDim.x, id = blockIdx.x;
  const int xcd = id & 7, per = total >> 3, rem = total & 7;
  int w = xcd * per + (xcd < rem ? xcd : rem) + (id >> 3);
  Place r;
  r.split = w % a.splits;
  w /= a.splits;
  const int tiles = a.tiles_m * a.tiles_n;
  r.tile = w;
  r.b = w / tiles;
  w -= r.b * tiles;
  constexpr int GM = 8;
  const int per_group = GM * a.tiles_n, group = w / per_group, in = w - group * per_group;
  const int rows = min(GM, a.tiles_m - group * GM);
  r.tm = group * GM + in % rows;
  r.tn = in / rows;
  return r;
}

// ------------------------------------------------------------------ 16-bit kernel

// BM x BN tile, WM x WN waves, contraction steps of BK. Dual: the tile's BN
// columns are BN / 2 of g and the same BN / 2 of u.
template <DT D, bool PT, bool QT, bool DUAL, int BM, int BN, int BK, int WM, int WN, bool ALN>
__global__ __launch_bounds__(64 * WM * WN) void k_product(const Gemm a) {
  constexpr int THREADS = 64 * WM * WN, NQ = DUAL ? 2 : 1;
  constexpr int FM = BM / WM / 16, FN = BN / WN / 16, FQ = FN / NQ;
  typedef Tile<D, PT, BM, BK, THREADS> TP;
  typedef Tile<D, QT, BN / NQ, BK, THREADS> TQ;
  __shared__ __attribute__((aligned(16))) unsigned char lds[TP::BYTES + NQ * TQ::BYTES];
  unsigned char* const lq = lds + TP::BYTES;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave / WN, wn = wave % WN;
  const Place pl = place(a);
  const int64_t m0 = (int64_t)pl.tm * BM;
  const int n0 = pl.tn * (BN / NQ);

  f32x4 acc[FM * FN];
#pragma unroll
  for (int i = 0; i < FM * FN; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  const int kt = (a.K + BK - 1) / BK, steps = kt * a.segments;
  const int t0 = (int)((int64_t)steps * pl.split / a.splits), t1 = (int)((int64_t)steps * (pl.split + 1) / a.splits);
  uint4 vp[TP::NI], vq[NQ][TQ::NI];
  auto fetch = [&](int t) {
    const int seg = t >= kt, k0 = (t - seg * kt) * BK, b = seg + pl.b;
    TP::template fetch<ALN>(a.p[b], a.ldp, m0, a.M, k0, a.K, tid, vp);
#pragma unroll
    for (int i = 0; i < NQ; ++i) TQ::template fetch<ALN>(a.q[b + i], a.ldq, n0, a.N, k0, a.K, tid, vq[i]);
  };
  if (t0 < t1) fetch(t0);
  for (int t = t0; t < t1; ++t) {
    __syncthreads();
    TP::put(lds, tid, vp);
#pragma unroll
    for (int i = 0; i < NQ; ++i) TQ::put(lq + i * TQ::BYTES, tid, vq[i]);
    __syncthreads();
    if (t + 1 < t1) fetch(t + 1);
#pragma unroll
    for (int k = 0; k < BK; k += 32) {
      s16x8 fp[FM], fq[FN];
#pragma unroll
      for (int i = 0; i < FM; ++i) fp[i] = TP::frag(lds, (wm * FM + i) * 16, k, lane);
#pragma unroll
      for (int j = 0; j < FN; ++j)
        fq[j] = TQ::frag(lq + (j / FQ) * TQ::BYTES, (wn * FQ + j % FQ) * 16, k, lane);
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i * FN + j] = mfma<D>(fq[j], fp[i], acc[i * FN + j]);
    }
  }

  if (a.splits > 1 && !join_splits<FM * FN, THREADS>(a, pl.tile, pl.split, acc, tid)) return;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int64_t m = m0 + (wm * FM + i) * 16 + (lane & 15);
#pragma unroll
    for (int j = 0; j < FQ; ++j) {
      const int n = n0 + (wn * FQ + j) * 16 + 4 * (lane >> 4);
      float v[4], u[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = acc[i * FN + j][e];
        if constexpr (DUAL) u[e] = acc[i * FN + FQ + j][e];
      }
      finish4<D, DUAL>(a, pl.b, m, n, v, u);
    }
  }
}

// ------------------------------------------------------------------ fp32 kernel

// The same product in fp32 with 16x16x4 fp32 matrix-core steps. Both operands'
// tiles sit in LDS as [output index][16 contraction indices], rows 20 floats apart
// (16 lanes' 16-byte reads then fall on distinct banks); lane l reads contraction
// indices 4 (l / 16) .. +3 of its row, and step e of four uses the e-th of them.
// Sums over 512 contraction indices are taken before they are added to the total,
// so that a long contraction's rounding grows with its square root at a slower rate.
template <bool TR, int R, int THREADS> struct Tile32 {
  static constexpr int LD = 20;
  static constexpr int BK = 16;
  static constexpr int CHUNKS = R * BK / 4;  // four floats each
  static constexpr int NI = (CHUNKS + THREADS - 1) / THREADS;

  static __device__ __forceinline__ void fetch(const void* base, int64_t ld, int64_t r0, int64_t nr, int k0, int K,
                                               bool aln, int tid, f32x4* v) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int c = i * THREADS + tid;
      const int row = TR ? c / (R / 4) : c / 4, ch = TR ? c % (R / 4) : c % 4;
      const int64_t mr = TR ? (int64_t)k0 + row : r0 + row;
      const int64_t mc = TR ? r0 + 4 * ch : (int64_t)k0 + 4 * ch;
      const int64_t left = (TR ? nr : (int64_t)K) - mc;
      const float* src = (const float*)base + mr * ld + mc;
      v[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      if (c < CHUNKS && mr < (TR ? (int64_t)K : nr) && left > 0) {
        if (aln) {
          v[i] = *(const f32x4*)src;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (e < left) v[i][e] = src[e];
        }
      }
    }
  }
  static __device__ __forceinline__ void put(float* lds, int tid, const f32x4* v) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int c = i * THREADS + tid;
      if (c < CHUNKS) {
        if constexpr (!TR) {
          *(f32x4*)(lds + (c / 4) * LD + 4 * (c % 4)) = v[i];
        } else {
          const int k = c / (R / 4), r = 4 * (c % (R / 4));
#pragma unroll
          for (int e = 0; e < 4; ++e) lds[(r + e) * LD + k] = v[i][e];
        }
      }
    }
  }
  static __device__ __forceinline__ f32x4 frag(const float* lds, int r, int lane) {
    return *(const f32x4*)(lds + (r + (lane & 15)) * LD + 4 * (lane >> 4));
  }
};

template <bool PT, bool QT, bool DUAL, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void k_product32(const Gemm a, const bool aln) {
  constexpr int THREADS = 64 * WM * WN, NQ = DUAL ? 2 : 1, BK = 16;
  constexpr int FM = BM / WM / 16, FN = BN / WN / 16, FQ = FN / NQ, NA = FM * FN;
  typedef Tile32<PT, BM, THREADS> TP;
  typedef Tile32<QT, BN / NQ, THREADS> TQ;
  __shared__ __attribute__((aligned(16))) float lds[(BM + BN) * TP::LD];
  float* const lq = lds + BM * TP::LD;
  constexpr int LQ = (BN / NQ) * TP::LD;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave / WN, wn = wave % WN;
  const Place pl = place(a);
  const int64_t m0 = (int64_t)pl.tm * BM;
  const int n0 = pl.tn * (BN / NQ);

  f32x4 acc[NA], tot[NA];
#pragma unroll
  for (int i = 0; i < NA; ++i) acc[i] = tot[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const int kt = (a.K + BK - 1) / BK, steps = kt * a.segments;
  const int t0 = (int)((int64_t)steps * pl.split / a.splits), t1 = (int)((int64_t)steps * (pl.split + 1) / a.splits);
  f32x4 vp[TP::NI], vq[NQ][TQ::NI];
  auto fetch = [&](int t) {
    const int seg = t >= kt, k0 = (t - seg * kt) * BK, b = seg + pl.b;
    TP::fetch(a.p[b], a.ldp, m0, a.M, k0, a.K, aln, tid, vp);
#pragma unroll
    for (int i = 0; i < NQ; ++i) TQ::fetch(a.q[b + i], a.ldq, n0, a.N, k0, a.K, aln, tid, vq[i]);
  };
  if (t0 < t1) fetch(t0);
  for (int t = t0; t < t1; ++t) {
    __syncthreads();
    TP::put(lds, tid, vp);
#pragma unroll
    for (int i = 0; i < NQ; ++i) TQ::put(lq + i * LQ, tid, vq[i]);
    __syncthreads();
    if (t + 1 < t1) fetch(t + 1);
    f32x4 fp[FM], fq[FN];
#pragma unroll
    for (int i = 0; i < FM; ++i) fp[i] = TP::frag(lds, (wm * FM + i) * 16, lane);
#pragma unroll
    for (int j = 0; j < FN; ++j) fq[j] = TQ::frag(lq + (j / FQ) * LQ, (wn * FQ + j % FQ) * 16, lane);
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[i * FN + j] = __builtin_amdgcn_mfma_f32_16x16x4f32(fq[j][e], fp[i][e], acc[i * FN + j], 0, 0, 0);
    if (((t - t0) & 31) == 31) {
#pragma unroll
      for (int i = 0; i < NA; ++i) {
        tot[i] = tot[i] + acc[i];
        acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NA; ++i) acc[i] = tot[i] + acc[i];

  if (a.splits > 1 && !join_splits<NA, THREADS>(a, pl.tile, pl.split, acc, tid)) return;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int64_t m = m0 + (wm * FM + i) * 16 + (lane & 15);
#pragma unroll
    for (int j = 0; j < FQ; ++j) {
      const int n = n0 + (wn * FQ + j) * 16 + 4 * (lane >> 4);
      float v[4], u[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = acc[i * FN + j][e];
        if constexpr (DUAL) u[e] = acc[i * FN + FQ + j][e];
      }
      finish4<DT::F32, DUAL>(a, pl.b, m, n, v, u);
    }
  }
}

// ------------------------------------------------------------------ schedule

// Tile shape and split of a product.
struct Plan {
  int bm, bn, bk;
  int tiles_m, tiles_n, splits;
};

static Plan make_plan(int dtype, int64_t M, int64_t N, int64_t K, bool p_trans, bool dual, int segments, int batch) {
  Plan p;
  const bool few = M <= 16 && !p_trans;
  p.bm = few ? 16 : 128;
  p.bn = few && !dual ? 64 : 128;
  p.bk = dtype == HCLRMIX_F32 ? 16 : (few ? 128 : 64);
  const int cols = dual ? p.bn / 2 : p.bn;
  p.tiles_m = (int)((M + p.bm - 1) / p.bm);
  p.tiles_n = (int)((N + cols - 1) / cols);
  const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n * batch;
  const int64_t steps = (K + p.bk - 1) / p.bk * segments;
  int64_t s = 1;
  if (tiles <= MAX_SPLIT_TILES && tiles < 384) s = std::min<int64_t>(768 / tiles, steps / (few ? 2 : 4));
  p.splits = (int)std::max<int64_t>(1, std::min<int64_t>(s, 64));
  return p;
}

size_t product_scratch(int dtype, int64_t M, int64_t N, int64_t K, bool p_trans, bool dual, int segments, int batch) {
  if (M == 0) return 0;
  const Plan p = make_plan(dtype, M, N, K, p_trans, dual, segments, batch);
  if (p.splits == 1) return 0;
  return (size_t)p.tiles_m * p.tiles_n * batch * p.splits * p.bm * p.bn * 4;
}

template <DT D, bool PT, bool QT, bool DUAL>
static hipError_t go16(const Gemm& g, const Plan& p, bool aln, unsigned grid, hipStream_t s) {
  if constexpr (!PT) {
    if (p.bm == 16)
      return aln ? launch(nullptr, k_product<D, PT, QT, DUAL, 16, DUAL ? 128 : 64, 128, 1, 4, true>, dim3(grid), dim3(256),
                          0, s, g)
                 : launch(nullptr, k_product<D, PT, QT, DUAL, 16, DUAL ? 128 : 64, 128, 1, 4, false>, dim3(grid), dim3(256),
                          0, s, g);
  }
  return aln ? launch(nullptr, k_product<D, PT, QT, DUAL, 128, 128, 64, 2, 2, true>, dim3(grid), dim3(256), 0, s, g)
             : launch(nullptr, k_product<D, PT, QT, DUAL, 128, 128, 64, 2, 2, false>, dim3(grid), dim3(256), 0, s, g);
}

template <bool PT, bool QT, bool DUAL>
static hipError_t go32(const Gemm& g, const Plan& p, bool aln, unsigned grid, hipStream_t s) {
  if constexpr (!PT) {
    if (p.bm == 16)
      return launch(nullptr, k_product32<PT, QT, DUAL, 16, DUAL ? 128 : 64, 1, 4>, dim3(grid), dim3(256), 0, s, g, aln);
  }
  return launch(nullptr, k_product32<PT, QT, DUAL, 128, 128, 2, 2>, dim3(grid), dim3(256), 0, s, g, aln);
}

template <bool PT, bool QT, bool DUAL>
static hipError_t go(const Gemm& g, const Plan& p, int dtype, bool aln, unsigned grid, hipStream_t s) {
  if (dtype == HCLRMIX_F32) return go32<PT, QT, DUAL>(g, p, aln, grid, s);
  return dtype == HCLRMIX_BF16 ? go16<DT::BF16, PT, QT, DUAL>(g, p, aln, grid, s)
                               : go16<DT::F16, PT, QT, DUAL>(g, p, aln, grid, s);
}

hipError_t launch_product(const Product& p, int dtype, void* scratch, unsigned* counters, hipStream_t s) {
  if (p.M == 0) return hipSuccess;
  const Plan pl = make_plan(dtype, p.M, p.N, p.K, p.p_trans, p.dual, p.segments, p.batch);
  Gemm g{};
  const uintptr_t es = dtype == HCLRMIX_F32 ? 4 : 2, a16 = 16 / es;
  // 16-byte accesses: rows start on them and their ends do too.
  bool aln = p.ldp % a16 == 0 && p.ldq % a16 == 0 && (p.p_trans ? p.M : (int64_t)p.K) % (int64_t)a16 == 0 &&
             (p.q_trans ? p.N : p.K) % (int64_t)a16 == 0;
  bool v4 = p.N % 4 == 0 && (!p.residual || p.ldr % 4 == 0);
  auto on = [](const void* q, uintptr_t to) { return ((uintptr_t)q & (to - 1)) == 0; };
  for (int i = 0; i < 2; ++i) {
    g.p[i] = p.p[i];
    g.q[i] = p.q[i];
    g.bias[i] = p.bias[i];
    g.out[i] = p.out[i];
    g.save[i] = p.save[i];
    aln = aln && on(p.p[i], 16) && on(p.q[i], 16);
    v4 = v4 && on(p.bias[i], 4 * es) && on(p.out[i], 4 * es) && on(p.save[i], 4 * es);
  }
  v4 = v4 && on(p.residual, 4 * es);
  g.ldp = p.ldp;
  g.ldq = p.ldq;
  g.ldr = p.ldr;
  g.M = p.M;
  g.N = p.N;
  g.K = p.K;
  g.residual = p.residual;
  g.act = p.act;
  g.segments = p.segments;
  g.tiles_m = pl.tiles_m;
  g.tiles_n = pl.tiles_n;
  g.splits = pl.splits;
  g.vec4 = v4;
  g.partial = (float*)scratch;
  g.counters = counters;
  const int64_t grid = (int64_t)pl.tiles_m * pl.tiles_n * p.batch * pl.splits;
  if (grid > 0x3FFFFF) return hipErrorInvalidValue;
  const unsigned n = (unsigned)grid;
  if (p.dual) return go<false, true, true>(g, pl, dtype, aln, n, s);
  if (p.p_trans) return go<true, true, false>(g, pl, dtype, aln, n, s);
  return p.q_trans ? go<false, true, false>(g, pl, dtype, aln, n, s) : go<false, false, false>(g, pl, dtype, aln, n, s);
}

// ------------------------------------------------------------------ activation gradients

constexpr int GRAD_ROWS = 32;  // rows per group, at least

int grad_groups(int64_t rows) {
  const int64_t g = (rows + GRAD_ROWS - 1) / GRAD_ROWS;
  return (int)(g < 64 ? g : 64);
}

// A thread takes eight columns of its group's rows (a contiguous range),
// ascending, and holds their column sums.
template <DT D, bool ALN, bool GLU>
__global__ __launch_bounds__(256) void k_act_grad(const void* dy, const void* p, const void* u, void* d0, void* d1,
                                                  float* partial, int64_t rows, int64_t cols, int act) {
  const int64_t c = ((int64_t)blockIdx.x * 64 + (threadIdx.x & 63)) * 8;
  const int sub = threadIdx.x >> 6;
  __shared__ float red[4][64][9];
  const int64_t r0 = rows * blockIdx.y / gridDim.y, r1 = rows * (blockIdx.y + 1) / gridDim.y;
  float s0[8], s1[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) s0[e] = s1[e] = 0.0f;
  const int left = (int)(cols - c < 8 ? cols - c : 8);
  if (left > 0) {
    for (int64_t r = r0 + sub; r < r1; r += 4) {
      const int64_t i = r * cols + c;
      float g[8], x[8], y[8], v[8];
      load8<D, ALN>(dy, i, left, g);
      if (p) load8<D, ALN>(p, i, left, x);
      if (GLU) load8<D, ALN>(u, i, left, y);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float df = 1.0f, f = 0.0f;
        if (p) f = act_df(act, x[e], df);
        if (GLU) {
          const float a = g[e] * y[e] * df, b = g[e] * f;
          s0[e] = s0[e] + a;
          s1[e] = s1[e] + b;
          g[e] = a;
          v[e] = b;
        } else {
          g[e] = g[e] * df;
          s0[e] = s0[e] + g[e];
        }
      }
      if (d0) store8<D, ALN>(d0, i, left, g);
      if (GLU && d1) store8<D, ALN>(d1, i, left, v);
    }
  }
  if (!partial) return;
#pragma unroll
  for (int h = 0; h < (GLU ? 2 : 1); ++h) {
    if (h) __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) red[sub][threadIdx.x & 63][e] = h ? s1[e] : s0[e];
    __syncthreads();
    for (int j = threadIdx.x; j < 512; j += 256) {
      const int64_t col = (int64_t)blockIdx.x * 512 + j;
      if (col < cols)
        partial[((int64_t)blockIdx.y * (GLU ? 2 : 1) + h) * cols + col] =
            ((red[0][j >> 3][j & 7] + red[1][j >> 3][j & 7]) + red[2][j >> 3][j & 7]) + red[3][j >> 3][j & 7];
    }
  }
}

template <DT D, bool ALN>
static hipError_t act_grad(const void* dy, const void* p, const void* u, void* d0, void* d1, float* partial,
                           int64_t rows, int64_t cols, int act, hipStream_t s) {
  const dim3 grid((unsigned)((cols + 511) / 512), (unsigned)grad_groups(rows));
  return u ? launch(nullptr, k_act_grad<D, ALN, true>, grid, dim3(256), 0, s, dy, p, u, d0, d1, partial, rows, cols, act)
           : launch(nullptr, k_act_grad<D, ALN, false>, grid, dim3(256), 0, s, dy, p, u, d0, d1, partial, rows, cols, act);
}

hipError_t launch_act_grad(const void* dy, const void* p, const void* u, void* d0, void* d1, float* partial,
                           int64_t rows, int64_t cols, int act, int dtype, bool aligned, hipStream_t s) {
  if (rows == 0) return hipSuccess;
  if (dtype == HCLRMIX_BF16)
    return aligned ? act_grad<DT::BF16, true>(dy, p, u, d0, d1, partial, rows, cols, act, s)
                   : act_grad<DT::BF16, false>(dy, p, u, d0, d1, partial, rows, cols, act, s);
  if (dtype == HCLRMIX_F16)
    return aligned ? act_grad<DT::F16, true>(dy, p, u, d0, d1, partial, rows, cols, act, s)
                   : act_grad<DT::F16, false>(dy, p, u, d0, d1, partial, rows, cols, act, s);
  return aligned ? act_grad<DT::F32, true>(dy, p, u, d0, d1, partial, rows, cols, act, s)
                 : act_grad<DT::F32, false>(dy, p, u, d0, d1, partial, rows, cols, act, s);
}

}  // namespace hc
