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
// holds four consecutive columns n of one row m: one 16-byte access per vector
// where sums go to LDS or scratch.
//
// Few tiles: the contraction is split over workgroups. Each writes its fp32 tile
// to scratch with agent-coherent stores and counts itself in; the last one adds
// the parts in ascending order, whichever order they arrived in, and runs the
// epilogue.
#include "hc_ffn.h"
#include "hc_internal.h"
#include "hc_plan.h"

#include "../../include/hclrmix.h"

#include <algorithm>

namespace hc {

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
  int tiles_m, tiles_n;
  int whole;        // tiles taken by one workgroup each (the first ones); the rest are split
  int splits;       // parts of a split tile
  int vec8;         // N is a multiple of 8 and every [M, N] tensor and bias 16-byte aligned
  float* partial;   // [split tile][split][min(BM, M) * BN] fp32
  unsigned* counters;
};

// Counter i sits in line i % 32 of the 4 KB prefix.
__device__ __forceinline__ unsigned* counter_at(unsigned* base, int i) { return base + (i & 31) * 32 + (i >> 5); }

// Chunk permutation of an LDS row: the slot that holds chunk c of row r (and the
// chunk that slot c holds). Direct tiles (rows of 128 bytes): a fragment read takes one
// chunk of 16 consecutive rows, so the low three bits of c change with r.
// Transposed tiles (rows of R columns), 16-bit: a transposing read takes 32 bytes of rows
// r .. r+3 and r+8 .. r+11 in one half wave, so whole 32-byte units move with r; fp32: a
// read takes 64 bytes of rows r, r+4, r+8 and r+12, so 64-byte units move with r / 4.
template <DT D, bool TR, int CPR> __device__ __forceinline__ int swz(int r, int c) {
  if constexpr (!TR) {
    return c ^ (r & 7);
  } else if constexpr (D == DT::F32) {
    return c ^ (((r >> 2) & 3) << 2);
  } else if constexpr (CPR >= 16) {
    return c ^ (((r & 3) | ((r >> 1) & 4)) << 1);
  } else {
    return c ^ ((((r >> 1) & 1) | ((r >> 2) & 2)) << 1);
  }
}

// One operand's tile: R indices of the output by BK of the contraction (128 bytes).
template <DT D, bool TR, int R, int THREADS> struct Tile {
  static constexpr int ES = D == DT::F32 ? 4 : 2, EPC = 16 / ES;  // bytes of an element, elements of a chunk
  static constexpr int BK = 128 / ES;
  static constexpr int CPR = (TR ? R : BK) / EPC;  // 16-byte chunks per LDS row
  static constexpr int ROWS = TR ? BK : R;
  static constexpr int NI = ROWS * CPR / THREADS;  // chunks a thread stages
  static constexpr int BYTES = ROWS * CPR * 16;
  static constexpr int KSTEP = D == DT::F32 ? 16 : 32;  // contraction indices of one fragment
  static_assert(ROWS * CPR % THREADS == 0 && CPR >= (D == DT::F32 && TR ? 16 : 8), "tile shape");
  typedef typename Store<D>::type elem_t;

  // Reads this thread's chunks of the tile at output index r0 and contraction
  // index k0 of a 16-bit operand with nr output indices and K contraction indices, at any
  // element-aligned address.
  static __device__ __forceinline__ void fetch(const void* base, int64_t ld, int64_t r0, int64_t nr, int k0, int K,
                                               int tid, uint4* v) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int c = i * THREADS + tid, row = c / CPR, ch = c % CPR;
      const int64_t mr = TR ? (int64_t)k0 + row : r0 + row;            // memory row
      const int64_t mc = TR ? r0 + EPC * ch : (int64_t)k0 + EPC * ch;  // memory column
      const int64_t left = (TR ? nr : (int64_t)K) - mc;                // columns from here on
      const bool in = mr < (TR ? (int64_t)K : nr) && left > 0;
      const elem_t* src = (const elem_t*)base + mr * ld + mc;
      v[i] = make_uint4(0u, 0u, 0u, 0u);
      if (in) {
        if (left >= EPC) {
          v[i] = ld16<D, false>(src);
        } else {
          uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
          for (int e = 0; e < EPC - 1; ++e)
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
      *(uint4*)(lds + (row * CPR + swz<D, TR, CPR>(row, ch)) * 16) = v[i];
    }
  }
  // Fragment of output indices r .. r+15 and contraction indices k .. k+KSTEP-1. 16-bit: lane l
  // holds (r + l % 16, k + 8 (l / 16) + 0..7); fp32: (r + l % 16, k + 4 (l / 16) + 0..3), one
  // value for each of four matrix ops.
  static __device__ __forceinline__ auto frag(const unsigned char* lds, int r, int k, int lane) {
    const int g = lane >> 4, j = lane & 15;
    if constexpr (!TR) {
      const int row = r + j;
      const uint4 v = *(const uint4*)(lds + (row * CPR + swz<D, TR, CPR>(row, k / EPC + g)) * 16);
      if constexpr (D == DT::F32) return __builtin_bit_cast(f32x4, v);
      else return __builtin_bit_cast(s16x8, v);
    } else if constexpr (D == DT::F32) {
      f32x4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int kr = k + 4 * g + e;
        v[e] = *(const float*)(lds + (kr * CPR + swz<D, TR, CPR>(kr, (r >> 2) + (j >> 2))) * 16 + 4 * (j & 3));
      }
      return v;
    } else {
      const int kr = k + 8 * g + (j >> 2), cb = j & 3;
      lds_u8* p = (lds_u8*)(lds + (kr * CPR + swz<D, TR, CPR>(kr, (r >> 3) + (cb >> 1))) * 16 + 8 * (cb & 1));
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * CPR * 16));
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  }
};
template <DT D> struct Frag { typedef s16x8 type; };
template <> struct Frag<DT::F32> { typedef f32x4 type; };

// ------------------------------------------------------------------ epilogue

// The tile's fp32 sums go through LDS once more, so that every global access of the epilogue is
// eight consecutive elements of a row and neighbouring lanes follow each other: whole cache
// lines. (Stores straight from the matrix-core layout, four elements of 16 rows per
// instruction, write 32 bytes of a line at a time.)

// Eight columns n .. n+7 of row m: v (and u of a dual product) hold the fp32 sums.
template <DT D, bool DUAL, bool ALN>
__device__ __forceinline__ void finish8(const Gemm& a, int b, int64_t m, int n, float* v, float* u) {
  const int left = a.N - n;
  const int64_t i = m * a.N + n;
  // Every load first: one memory latency for all.
  float t[8], w[8];
  if (a.bias[0]) load8<D, ALN>(a.bias[0], n, left, t);
  if constexpr (DUAL) {
    if (a.bias[1]) load8<D, ALN>(a.bias[1], n, left, w);
  } else {
    if (a.residual) load8<D, ALN>(a.residual, m * a.ldr + n, left, w);
  }
  if (a.bias[0]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = v[e] + t[e];
  }
  if constexpr (DUAL) {
    if (a.bias[1]) {
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] = u[e] + w[e];
    }
    if (a.save[0]) {
      store8<D, ALN>(a.save[0], i, left, v);
      store8<D, ALN>(a.save[1], i, left, u);
    }
    act_n<D, 8>(a.act, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = v[e] * u[e];
    store8<D, ALN>(a.out[0], i, left, v);
  } else {
    if (a.save[0]) store8<D, ALN>(a.save[0], i, left, v);
    act_n<D, 8>(a.act, v);
    if (a.residual) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = v[e] + w[e];
    }
    store8<D, ALN>(a.out[b], i, left, v);
  }
}

// Place of column quad c (four floats) of row r in the LDS image of [rows][BN] sums: the quads
// of 16 consecutive rows, which one write instruction covers, fall on distinct banks.
template <int BN> __device__ __forceinline__ int sum_at(int r, int c) { return r * BN + 4 * (c ^ (r & 15)); }

// Rows m0 .. m0+ROWS-1, columns from n0 on, from their LDS image (after a barrier).
template <DT D, bool DUAL, int ROWS, int BN, int THREADS>
__device__ __forceinline__ void finish_rows(const Gemm& a, int b, const float* sums, int64_t m0, int n0, int tid) {
  constexpr int COLS = DUAL ? BN / 2 : BN, CH = COLS / 8;  // chunks of eight output columns per row
  const int rows = (int)min((int64_t)ROWS, a.M - m0);
  for (int i = tid; i < rows * CH; i += THREADS) {
    const int r = i / CH, c = i - r * CH, n = n0 + 8 * c;
    if (n >= a.N) continue;
    float v[8], u[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x4 x = *(const f32x4*)(sums + sum_at<BN>(r, 2 * c + h));
      f32x4 y = x;
      if constexpr (DUAL) y = *(const f32x4*)(sums + sum_at<BN>(r, COLS / 4 + 2 * c + h));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[4 * h + e] = x[e];
        u[4 * h + e] = y[e];
      }
    }
    if (a.vec8) finish8<D, DUAL, true>(a, b, m0 + r, n, v, u);
    else finish8<D, DUAL, false>(a, b, m0 + r, n, v, u);
  }
}

constexpr uint32_t OUTSIDE = 0x80000000u;  // an offset past every descriptor's end: loads give zeros, stores nothing
constexpr int AGENT = 16;  // sc1: the access is coherent across the chip's L2s

// Split sums: this workgroup's tile goes to scratch; the last of the tile's workgroups to
// arrive gets the sum of all parts in ascending order and true, the others false. A part is
// [columns / 4][rows that exist] of four floats: vector i of a thread is row row(i) and
// column group quad(i), and rows past the last one are neither written nor read. A tile's parts
// have room for part_size() floats each.
template <int NA, int BM, int BN, typename Row, typename Quad>
__device__ __forceinline__ bool join_splits(const Gemm& a, int slot, int split, int64_t m0, f32x4* acc, int tid, Row row,
                                            Quad quad) {
  __shared__ int is_last;
  const int rows = (int)min((int64_t)BM, a.M - m0);
  const uint32_t part = (uint32_t)rows * (BN / 4) * 16;  // bytes of one part
  const char* base = (const char*)(a.partial + (size_t)slot * a.splits * ((int)min((int64_t)BM, a.M) * BN));
  auto at = [&](int i) { return row(i) < rows ? (uint32_t)(quad(i) * rows + row(i)) * 16u : OUTSIDE; };
  {
    const rsrc_t r = make_rsrc(base + (size_t)split * part, part);
#pragma unroll
    for (int i = 0; i < NA; ++i)
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc[i]), r, at(i), 0, AGENT);
  }
  // Each thread's stores have completed before any thread counts the workgroup in.
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  unsigned* counter = counter_at(a.counters, slot);
  if (tid == 0)
    is_last = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (unsigned)(a.splits - 1);
  __syncthreads();
  if (!is_last) return false;
  if (tid == 0) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);  // zero for the next call
  // Parts are read several at a time (up to 16 loads in flight per thread): one after
  // the other, each would cost a memory latency.
  constexpr int AT = NA >= 16 ? 1 : 16 / NA;
#pragma unroll
  for (int i = 0; i < NA; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int s0 = 0; s0 < a.splits; s0 += AT) {
    f32x4 v[AT][NA];
#pragma unroll
    for (int j = 0; j < AT; ++j) {
      const rsrc_t r = make_rsrc(base + (size_t)min(s0 + j, a.splits - 1) * part, part);
#pragma unroll
      for (int i = 0; i < NA; ++i)
        v[j][i] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at(i), 0, AGENT));
    }
#pragma unroll
    for (int j = 0; j < AT; ++j)
      if (s0 + j < a.splits) {
#pragma unroll
        for (int i = 0; i < NA; ++i) acc[i] = acc[i] + v[j][i];
      }
  }
  return true;
}

// Block id -> (batch, tile row, tile column, split). Consecutive block ids go to
// the eight XCDs in turn; each XCD gets a contiguous range of tiles, ordered so
// that workgroups running together share the operands' tiles in its L2: groups of
// eight tile rows, tile rows fastest, then tile columns.
struct Place {
  int b, tm, tn;
  int splits, split;  // parts of this tile (1: whole) and which one this is
  int slot;           // index among the split tiles
};
__device__ __forceinline__ int xcd_order(int id, int total) {
  const int xcd = id & 7, per = total >> 3, rem = total & 7;
  return xcd * per + (xcd < rem ? xcd : rem) + (id >> 3);
}
__device__ __forceinline__ Place place(const Gemm& a) {
  const int id = blockIdx.x;
  Place r;
  int tile;
  if (id < a.whole) {
    tile = xcd_order(id, a.whole);
    r.splits = 1;
    r.split = r.slot = 0;
  } else {
    const int w = xcd_order(id - a.whole, (int)gridDim.x - a.whole);
    r.splits = a.splits;
    r.slot = w / a.splits;
    r.split = w - r.slot * a.splits;
    tile = a.whole + r.slot;
  }
  const int tiles = a.tiles_m * a.tiles_n;
  r.b = tile / tiles;
  tile -= r.b * tiles;
  constexpr int GM = 8;
  const int per_group = GM * a.tiles_n, group = tile / per_group, in = tile - group * per_group;
  const int rows = min(GM, a.tiles_m - group * GM);
  r.tm = group * GM + in % rows;
  r.tn = in / rows;
  return r;
}

// ------------------------------------------------------------------ direct staging

// Stages a tile by loads that write LDS themselves: no registers and no LDS
// write instructions. One instruction per wave fills 1 KB of consecutive LDS,
// so the chunk permutation is applied to the addresses instead. Loads go
// through a buffer descriptor of the tile; lanes whose chunk lies outside the
// operand get an offset beyond it, for which the load writes zeros.
__device__ __forceinline__ u32x4 raw_desc(const void* base) {
  const uint64_t b = (uint64_t)base;
  return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)b),
               (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(b >> 32)), 0x7FFFFFF0u, 0x00020000u};
}
__device__ __forceinline__ uint32_t lds_offset(const void* p) { return (uint32_t)(uintptr_t)(const lds_u8*)p; }
// Lane l: W bytes (16 or 4) from offset off of the descriptor to LDS byte dst + W l (dst
// the same in every lane). Written out because the compiler, which cannot tell the stage
// being filled from the one being read, would wait for the load before every LDS read. m0 is a
// register of the compiler's own (it warns of any asm that writes it): named as written, so that
// no value that the compiler put there itself is taken to have survived.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
template <int W, bool STREAM> __device__ __forceinline__ void lds_load(u32x4 desc, uint32_t off, uint32_t dst) {
  static_assert(W == 16 || W == 4, "width");
  if constexpr (W == 4 && STREAM)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen nt lds"
                 : : "s"(dst), "v"(off), "s"(desc) : "memory", "m0");
  else if constexpr (W == 4)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                 : : "s"(dst), "v"(off), "s"(desc) : "memory", "m0");
  else if constexpr (STREAM)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen nt lds"
                 : : "s"(dst), "v"(off), "s"(desc) : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 : : "s"(dst), "v"(off), "s"(desc) : "memory", "m0");
}
#pragma clang diagnostic pop

// Where an operand's next tile starts and how many contraction indices it has from
// there in its segment; steps go through the first segment, then the second.
template <DT D, bool TR> struct Cursor {
  static constexpr int ES = D == DT::F32 ? 4 : 2, BK = 128 / ES;
  const char* p;
  const char* p1;  // the second segment's start
  int64_t step;    // bytes from one tile to the next
  int k, k1;
  __device__ __forceinline__ void init(const void* q0, const void* q1, int64_t ld, int64_t r0, int K, int segments, int t,
                                       int steps) {
    const int64_t first = ES * (TR ? r0 : r0 * ld);
    step = ES * (TR ? BK * ld : (int64_t)BK);
    const int kt = (K + BK - 1) / BK;
    p = (const char*)q0 + first;
    p1 = (const char*)q1 + first;
    k = K;
    k1 = segments == 2 ? K : 0;
    if (t >= kt) {
      p = p1;
      k1 = 0;
      t -= kt;
    }
    p += t * step;
    k -= t * BK;
    // A split's range may end before its segments do.
    stop = steps;
  }
  int stop;  // tiles left to load
  __device__ __forceinline__ void next() {
    p += step;
    k -= BK;
    --stop;
    const bool turn = k <= 0;
    p = turn ? p1 : p;
    k = turn ? k1 : k;
    k1 = turn ? 0 : k1;
    k = stop > 0 ? k : 0;
  }
};

// W: bytes a lane loads at once, 16 where rows start and end on 16 bytes, else (fp32) one
// element's 4: four times the instructions, but at any address (3243 x 1963 -> 4216 in fp32:
// 517 us, 701 with the chunks going through registers).
template <DT D, bool TR, int R, int THREADS, int W> struct Direct {
  typedef Tile<D, TR, R, THREADS> T;
  static constexpr int PER = 16 / W;      // instructions that fill 1 KB
  static constexpr int NL = T::NI * PER;  // loads of a thread
  static_assert(TR || THREADS / T::CPR % 8 == 0 || T::NI == 1, "every chunk of a thread has the same place in its row");
  static_assert(W == 16 || W == T::ES, "a load is a chunk or an element");
  uint32_t off[NL];  // byte offset of this lane's loads from the tile's first element
  int kk[PER];       // contraction index of the first PER loads inside the tile
  __device__ __forceinline__ void init(int64_t ld, int64_t r0, int64_t nr, int tid) {
    const int lane = tid & 63;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int c = i / PER * THREADS + (tid - lane) + (i % PER * 64 + lane) * W / 16;  // the chunk
      const int row = c / T::CPR, ch = swz<D, TR, T::CPR>(row, c % T::CPR);
      const int col = T::EPC * ch + (W == 16 ? 0 : lane & (PER - 1));
      const bool in = TR ? r0 + col < nr : r0 + row < nr;
      off[i] = in ? (uint32_t)(row * (int)ld + col) * T::ES : OUTSIDE;
      if (i < PER) kk[i] = TR ? row : col;
    }
  }
  // The tile at p, k contraction indices of which exist, into LDS from byte address lds on
  // (this wave's part).
  // STREAM: data that one workgroup alone reads, once (non-temporal loads).
  template <bool STREAM = false>
  __device__ __forceinline__ void stage(const char* p, int k, uint32_t lds, int wave) const {
    const u32x4 r = raw_desc(p);
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const uint32_t o = kk[i % PER] + (TR ? i / PER * (THREADS / T::CPR) : 0) < k ? off[i] : OUTSIDE;
      lds_load<W, STREAM>(r, o, __builtin_amdgcn_readfirstlane(lds + (i / PER * THREADS + wave * 64) * 16 + i % PER * 64 * W));
    }
  }
};

// Waits until at most N of this wave's loads are in flight (they complete in order).
template <int N> __device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

// Workgroup barrier once this wave's LDS operations are done; its global loads stay in flight.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// BM x BN tile, WM x WN waves, contraction steps of 128 bytes staged in a ring of NST buffers: the
// loads of step t + NST - 1 are issued once every wave is done with step t - 1, whose buffer
// they fill. With many rows two buffers of a 128 x 128 tile (64 KB) leave room for two
// workgroups per compute unit, whose loads, matrix ops and epilogues overlap. With few rows
// the product streams its weights: three or more buffers keep about 100 KB of loads in
// flight per compute unit.
// Measured: 1 x 2560 -> 2 x 10240 in bf16 22.5 us (105 MB of weights, 4.7 TB/s; reading them
// alone in such tiles 16.5 us), 48 x 4096 -> 2 x 12288 in fp16 44.6 us (201 MB, 4.5 TB/s), 8 x
// 10240 -> 2560 17.4 us (reading alone 10; the join of the parts 5), fp32 3200 x 2048 -> 2 x
// 4096 811 us (132 TFLOP/s).
template <DT D, bool PT, bool QT, bool DUAL, int BM, int BN, int NST, int WM, int WN, bool ALN>
__global__ __launch_bounds__(64 * WM * WN, BM == 128 ? 2 : 1) void k_product_ring(const Gemm a) {
  constexpr int THREADS = 64 * WM * WN, NQ = DUAL ? 2 : 1;
  constexpr int PR = BM < 32 ? 32 : BM;  // staged rows of P: every thread has a chunk; those past M load nothing
  constexpr bool FEW = BM <= 64;
  constexpr int FM = BM / WM / 16, FN = BN / WN / 16, FQ = FN / NQ;
  typedef Tile<D, PT, PR, THREADS> TP;
  typedef Tile<D, QT, BN / NQ, THREADS> TQ;
  constexpr int BK = TP::BK, KS = TP::KSTEP;
  typedef typename Frag<D>::type frag_t;
  constexpr bool DIRECT = ALN || D == DT::F32;  // loads write LDS themselves
  constexpr int W = ALN ? 16 : 4;               // bytes of a direct load per lane
  static_assert(DIRECT || NST == 2, "register staging uses two buffers");
  constexpr int STAGE = TP::BYTES + NQ * TQ::BYTES;
  __shared__ __attribute__((aligned(1024))) unsigned char lds[NST * STAGE];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave / WN, wn = wave % WN;
  const Place pl = place(a);
  const int64_t m0 = (int64_t)pl.tm * BM;
  const int n0 = pl.tn * (BN / NQ);

  f32x4 acc[FM * FN];
#pragma unroll
  for (int i = 0; i < FM * FN; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  const int kt = (a.K + BK - 1) / BK, steps = kt * a.segments;
  const int t0 = (int)((int64_t)steps * pl.split / pl.splits), t1 = (int)((int64_t)steps * (pl.split + 1) / pl.splits);
  // fp32: sums over 512 contraction indices are taken before they are added to the total, so
  // that the rounding of a long contraction does not grow with its length.
  constexpr bool BLOCKED = D == DT::F32;
  f32x4 total[BLOCKED ? FM * FN : 1];
  if constexpr (BLOCKED) {
#pragma unroll
    for (int i = 0; i < FM * FN; ++i) total[i] = acc[i];
  }
  auto multiply = [&](const unsigned char* cur, int t) {
    const unsigned char* curq = cur + TP::BYTES;
#pragma unroll
    for (int k = 0; k < BK; k += KS) {
      frag_t fp[FM], fq[FN];
#pragma unroll
      for (int j = 0; j < FN; ++j) fq[j] = TQ::frag(curq + (j / FQ) * TQ::BYTES, (wn * FQ + j % FQ) * 16, k, lane);
#pragma unroll
      for (int i = 0; i < FM; ++i) fp[i] = TP::frag(cur, (wm * FM + i) * 16, k, lane);
      if constexpr (D == DT::F32) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
              acc[i * FN + j] = __builtin_amdgcn_mfma_f32_16x16x4f32(fq[j][e], fp[i][e], acc[i * FN + j], 0, 0, 0);
      } else {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j) acc[i * FN + j] = mfma<D>(fq[j], fp[i], acc[i * FN + j]);
      }
    }
    if constexpr (BLOCKED) {
      if (((t - t0) & 15) == 15) {
#pragma unroll
        for (int i = 0; i < FM * FN; ++i) {
          total[i] = total[i] + acc[i];
          acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
      }
    }
  };

  if constexpr (DIRECT) {
    Direct<D, PT, PR, THREADS, W> dp;
    Direct<D, QT, BN / NQ, THREADS, W> dq;
    constexpr int LOADS = dp.NL + NQ * dq.NL;  // of a wave, per step
    static_assert((NST - 2) * LOADS < 64, "the wait counts up to 63 loads");
    dp.init(a.ldp, m0, BM < PR ? min(a.M, m0 + BM) : a.M, tid);
    dq.init(a.ldq, n0, a.N, tid);
    Cursor<D, PT> cp;
    Cursor<D, QT> cq[NQ];
    cp.init(a.p[pl.b], a.p[1], a.ldp, m0, a.K, a.segments, t0, t1 - t0);
#pragma unroll
    for (int i = 0; i < NQ; ++i) cq[i].init(a.q[pl.b + i], a.q[1], a.ldq, n0, a.K, a.segments, t0, t1 - t0);
    const uint32_t l0 = lds_offset(lds);
    const int w = __builtin_amdgcn_readfirstlane(wave);
    auto stage = [&](int buf) {
      const uint32_t to = l0 + buf * STAGE;
      dp.stage(cp.p, cp.k, to, w);
      cp.next();
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        if (FEW && a.tiles_m == 1) dq.template stage<true>(cq[i].p, cq[i].k, to + TP::BYTES + i * TQ::BYTES, w);
        else dq.stage(cq[i].p, cq[i].k, to + TP::BYTES + i * TQ::BYTES, w);
        cq[i].next();
      }
    };
#pragma unroll
    for (int i = 0; i < NST - 1; ++i) stage(i);
    int buf = 0;
    for (int t = t0; t < t1; ++t) {
      // This wave's loads of step t have arrived and its LDS reads of step t - 1 are done; then
      // everyone's. Loads past the last step write zeros, so the count in flight is constant.
      wait_loads<(NST - 2) * LOADS>();
      lds_barrier();
      stage(buf == 0 ? NST - 1 : buf - 1);
      multiply(lds + buf * STAGE, t);
      buf = buf == NST - 1 ? 0 : buf + 1;
    }
    wait_loads<0>();  // LDS must not be given up with loads into it in flight
  } else {
    // 16-bit rows at any address: through registers, the next step's loads issued before
    // this step's matrix ops and written to the other buffer after them.
    uint4 vp[TP::NI], vq[NQ][TQ::NI];
    auto fetch = [&](int t) {
      const int seg = t >= kt, k0 = (t - seg * kt) * BK, b = seg + pl.b;
      TP::fetch(a.p[b], a.ldp, m0, BM < PR ? min(a.M, m0 + BM) : a.M, k0, a.K, tid, vp);
#pragma unroll
      for (int i = 0; i < NQ; ++i) TQ::fetch(a.q[b + i], a.ldq, n0, a.N, k0, a.K, tid, vq[i]);
    };
    auto put = [&](int buf) {
      TP::put(lds + buf * STAGE, tid, vp);
#pragma unroll
      for (int i = 0; i < NQ; ++i) TQ::put(lds + buf * STAGE + TP::BYTES + i * TQ::BYTES, tid, vq[i]);
    };
    fetch(t0);
    put(0);
    lds_barrier();
    for (int t = t0; t < t1; ++t) {
      const int buf = (t - t0) & 1;
      if (t + 1 < t1) fetch(t + 1);
      multiply(lds + buf * STAGE, t);
      if (t + 1 < t1) put(buf ^ 1);
      lds_barrier();
    }
  }
  if constexpr (BLOCKED) {
#pragma unroll
    for (int i = 0; i < FM * FN; ++i) acc[i] = total[i] + acc[i];
  }

  // Column quad of vector i in the tile: the columns of Q0, then those of Q1.
  auto quad = [&](int i) {
    const int j = i % FN;
    return ((j / FQ) * (BN / NQ) + (wn * FQ + j % FQ) * 16) / 4 + (lane >> 4);
  };
  if (pl.splits > 1 &&
      !join_splits<FM * FN, BM, BN>(a, pl.slot, pl.split, m0, acc, tid, [&](int i) { return (wm * FM + i / FN) * 16 + (lane & 15); },
                                    quad))
    return;
  static_assert(BM * BN * 4 <= NST * STAGE, "the sums fit the staging buffers");
  float* const sums = (float*)lds;
  lds_barrier();
#pragma unroll
  for (int i = 0; i < FM * FN; ++i)
    *(f32x4*)(sums + sum_at<BN>((wm * FM + i / FN) * 16 + (lane & 15), quad(i))) = acc[i];
  lds_barrier();
  finish_rows<D, DUAL, BM, BN, THREADS>(a, pl.b, sums, m0, n0, tid);
}

// 256 x 256 tile, contraction steps of 64, eight waves, for products with many tiles. Wave
// (wm, wn) owns 64 rows of each half of the tile's rows and 64 columns (dual: 32 of g, the
// same 32 of u). A step has two phases of 32 matrix ops per wave, one per half of the rows.
// A fragment's registers are filled again as soon as their last matrix op is issued: during
// phase 0 with P's second half, during phase 1 with the next step's Q and first half of P, so
// that LDS reads run under the matrix ops all along.
// There are two LDS buffers and one barrier a phase, in its middle. There a wave waits for its
// LDS reads of the phase before (lgkmcnt counts the younger ones) and for its own global loads
// of what the next phase reads; behind the barrier both hold for every wave. So behind phase
// 0's barrier the loads of step t + 2 go to Q and the first half of P, behind phase 1's to the
// second half, and a load has two phases to arrive. Loads past the last step write zeros into
// free buffers, so that the number of loads in flight is the same in every phase.
// Measured: 8192^3 in bf16 1244 to 1315 TFLOP/s (by layout); the matrix units are half busy at
// 1.7 to 2.0 GHz, which is the power limit (on zeros the same product is 13 % faster). Two wave
// groups half a phase apart with two barriers a phase: 1165 to 1230.
template <DT D, bool PT, bool QT, bool DUAL>
__global__ __launch_bounds__(512) void k_product_wide(const Gemm a) {
  constexpr int THREADS = 512, NQ = DUAL ? 2 : 1, BK = 64, FM = 8, FN = 4, FQ = FN / NQ;
  typedef Tile<D, PT, 128, THREADS> TP;
  typedef Tile<D, QT, 256 / NQ, THREADS> TQ;
  constexpr int QBYTES = NQ * TQ::BYTES, STAGE = QBYTES + 2 * TP::BYTES;
  constexpr int LQ = NQ * TQ::NI, LP = TP::NI;  // loads of a wave for Q, and for half of P
  __shared__ __attribute__((aligned(1024))) unsigned char lds[2 * STAGE];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 2, wn = wave & 3;
  const Place pl = place(a);
  const int64_t m0 = (int64_t)pl.tm * 256;
  const int n0 = pl.tn * (256 / NQ);

  f32x4 acc[FM * FN];
#pragma unroll
  for (int i = 0; i < FM * FN; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  const int kt = (a.K + BK - 1) / BK, steps = kt * a.segments;
  const int t0 = (int)((int64_t)steps * pl.split / pl.splits), t1 = (int)((int64_t)steps * (pl.split + 1) / pl.splits);
  Direct<D, PT, 128, THREADS, 16> dp[2];
  Direct<D, QT, 256 / NQ, THREADS, 16> dq;
  dp[0].init(a.ldp, m0, a.M, tid);
  dp[1].init(a.ldp, m0 + 128, a.M, tid);
  dq.init(a.ldq, n0, a.N, tid);
  Cursor<D, PT> cp[2];
  Cursor<D, QT> cq[NQ];
#pragma unroll
  for (int h = 0; h < 2; ++h) cp[h].init(a.p[pl.b], a.p[1], a.ldp, m0 + 128 * h, a.K, a.segments, t0, t1 - t0);
#pragma unroll
  for (int i = 0; i < NQ; ++i) cq[i].init(a.q[pl.b + i], a.q[1], a.ldq, n0, a.K, a.segments, t0, t1 - t0);
  const uint32_t l0 = lds_offset(lds);
  const int w = __builtin_amdgcn_readfirstlane(wave);
  auto load_q = [&](int buf) {
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      dq.stage(cq[i].p, cq[i].k, l0 + buf * STAGE + i * TQ::BYTES, w);
      cq[i].next();
    }
  };
  auto load_p = [&](int buf, int h) {
    dp[h].stage(cp[h].p, cp[h].k, l0 + buf * STAGE + QBYTES + h * TP::BYTES, w);
    cp[h].next();
  };
  load_q(0);
  load_p(0, 0);
  load_p(0, 1);
  load_q(1);
  load_p(1, 0);
  load_p(1, 1);
  wait_loads<LQ + 2 * LP>();
  __builtin_amdgcn_s_barrier();
  s16x8 fq[2][FN], fp[2][FM / 2];
  const unsigned char* cur = lds;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
#pragma unroll
    for (int j = 0; j < FN; ++j) fq[k][j] = TQ::frag(cur + (j / FQ) * TQ::BYTES, (wn * FQ + j % FQ) * 16, 32 * k, lane);
#pragma unroll
    for (int i = 0; i < FM / 2; ++i) fp[k][i] = TP::frag(cur + QBYTES, (wm * 4 + i) * 16, 32 * k, lane);
  }
  for (int t = t0; t < t1; ++t) {
    const int buf = (t - t0) & 1;
    const unsigned char* next = lds + (buf ^ 1) * STAGE;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const unsigned char* np = half == 0 ? cur + QBYTES + TP::BYTES : next + QBYTES;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int i = 0; i < FM / 2; ++i) {
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int j = 0; j < FN; ++j) {
            f32x4& c = acc[(half * FM / 2 + i) * FN + j];
            c = mfma<D>(fq[k][j], fp[k][i], c);
          }
          __builtin_amdgcn_sched_barrier(0);
          fp[k][i] = TP::frag(np, (wm * 4 + i) * 16, 32 * k, lane);
          if (half == 1 && i == FM / 2 - 1) {
#pragma unroll
            for (int j = 0; j < FN; ++j)
              fq[k][j] = TQ::frag(next + (j / FQ) * TQ::BYTES, (wn * FQ + j % FQ) * 16, 32 * k, lane);
          }
          if (k == 0 && i == FM / 2 - 1) {
            // Everything read before this phase has arrived (younger: this phase's fragments so far).
            if (half == 0) wait_loads<LP>();
            else wait_loads<LQ + LP>();
            asm volatile("s_waitcnt lgkmcnt(%0)" : : "n"(min(15, half == 0 ? (PT ? 8 : 4) : (PT ? 8 : 4) + (QT ? 8 : 4))) : "memory");
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
            if (half == 0) {
              load_q(buf);
              load_p(buf, 0);
            } else {
              load_p(buf, 1);
            }
          }
        }
      }
    }
    cur = next;
  }
  wait_loads<0>();  // LDS must not be given up with loads into it in flight

  // Column quad of vector i in the tile: the columns of Q0, then those of Q1.
  auto quad = [&](int i) {
    const int j = i % FN;
    return ((j / FQ) * (256 / NQ) + (wn * FQ + j % FQ) * 16) / 4 + (lane >> 4);
  };
  if (pl.splits > 1 &&
      !join_splits<FM * FN, 256, 256>(a, pl.slot, pl.split, m0, acc, tid, [&](int i) { return (i / FN / 4) * 128 + (wm * 4 + i / FN % 4) * 16 + (lane & 15); },
                                    quad))
    return;
  float* const sums = (float*)lds;  // 128 rows at a time
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    lds_barrier();
#pragma unroll
    for (int i = 0; i < FM * FN / 2; ++i)
      *(f32x4*)(sums + sum_at<256>((wm * 4 + i / FN) * 16 + (lane & 15), quad(i))) = acc[half * FM * FN / 2 + i];
    lds_barrier();
    finish_rows<D, DUAL, 128, 256, THREADS>(a, pl.b, sums, m0 + 128 * half, n0, tid);
  }
}

// ------------------------------------------------------------------ launches

// k_product_ring for one tile shape; rows staged through registers take two buffers.
template <DT D, bool PT, bool QT, bool DUAL, int BM, int BN, int NST, int WM, int WN>
static hipError_t ring(const Gemm& g, bool aln, unsigned n, hipStream_t s) {
  constexpr int ODD = D == DT::F32 ? NST : 2;
  return launch(nullptr, aln ? k_product_ring<D, PT, QT, DUAL, BM, BN, NST, WM, WN, true> : k_product_ring<D, PT, QT, DUAL, BM, BN, ODD, WM, WN, false>,
                dim3(n), dim3(64 * WM * WN), 0, s, g);
}

template <DT D, bool PT, bool QT, bool DUAL>
static hipError_t go(const Gemm& g, const Shape& sh, bool aln, unsigned n, hipStream_t s) {
  constexpr int BN = DUAL ? 128 : 64;
  if constexpr (D != DT::F32) {  // aligned operands only
    if (sh.bm == 256) return launch(nullptr, k_product_wide<D, PT, QT, DUAL>, dim3(n), dim3(512), 0, s, g);
    if constexpr (!PT) {
      if (sh.bm == 16 && sh.bn == 256)
        return launch(nullptr, k_product_ring<D, PT, QT, DUAL, 16, 256, 3, 1, 4, true>, dim3(n), dim3(256), 0, s, g);
      if (sh.bm == 64 && sh.bn == 256)
        return launch(nullptr, k_product_ring<D, PT, QT, DUAL, 64, 256, 3, 1, 4, true>, dim3(n), dim3(256), 0, s, g);
    }
  }
  if constexpr (!PT) {
    if (sh.bm == 16) return ring<D, PT, QT, DUAL, 16, BN, DUAL ? 3 : 4, 1, 4>(g, aln, n, s);
  }
  if (sh.bm == 64) return ring<D, PT, QT, DUAL, 64, BN, 3, 2, 2>(g, aln, n, s);
  return ring<D, PT, QT, DUAL, 128, 128, 2, 2, 2>(g, aln, n, s);
}

template <DT D> static hipError_t go_layout(const Product& p, const Gemm& g, const Shape& sh, bool aln, unsigned n, hipStream_t s) {
  if (p.dual) return go<D, false, true, true>(g, sh, aln, n, s);
  if (p.p_trans) return go<D, true, true, false>(g, sh, aln, n, s);
  return p.q_trans ? go<D, false, true, false>(g, sh, aln, n, s) : go<D, false, false, false>(g, sh, aln, n, s);
}

hipError_t launch_product(const Product& p, int dtype, void* scratch, unsigned* counters, hipStream_t s) {
  if (p.M == 0) return hipSuccess;
  Gemm g{};
  const uintptr_t es = dtype == HCLRMIX_F32 ? 4 : 2, a16 = 16 / es;
  // 16-byte accesses: rows start on them and their ends do too.
  bool aln = p.ldp % a16 == 0 && p.ldq % a16 == 0 && (p.p_trans ? p.M : (int64_t)p.K) % (int64_t)a16 == 0 &&
             (p.q_trans ? p.N : p.K) % (int64_t)a16 == 0;
  bool v8 = p.N % 8 == 0 && (!p.residual || p.ldr % (int64_t)a16 == 0);
  auto on = [](const void* q, uintptr_t to) { return ((uintptr_t)q & (to - 1)) == 0; };
  for (int i = 0; i < 2; ++i) {
    g.p[i] = p.p[i];
    g.q[i] = p.q[i];
    g.bias[i] = p.bias[i];
    g.out[i] = p.out[i];
    g.save[i] = p.save[i];
    aln = aln && on(p.p[i], 16) && on(p.q[i], 16);
    v8 = v8 && on(p.bias[i], 16) && on(p.out[i], 16) && on(p.save[i], 16);
  }
  v8 = v8 && on(p.residual, 16);
  const Plan pl = make_plan(dtype, p.M, p.N, p.K, p.p_trans, p.dual, p.segments, p.batch, aln);
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
  g.whole = (int)pl.whole;
  g.splits = pl.splits;
  g.vec8 = v8;
  g.partial = (float*)scratch;
  g.counters = counters;
  const int64_t grid = pl.whole + pl.rest * pl.splits;
  if (grid > 0x3FFFFF) return hipErrorInvalidValue;
  const unsigned n = (unsigned)grid;
  if (dtype == HCLRMIX_F32) return go_layout<DT::F32>(p, g, *pl.shape, aln, n, s);
  return dtype == HCLRMIX_BF16 ? go_layout<DT::BF16>(p, g, *pl.shape, aln, n, s)
                               : go_layout<DT::F16>(p, g, *pl.shape, aln, n, s);
}

// ------------------------------------------------------------------ activation gradients

// One group up to 64 rows (its sums are the result, without a second launch), then one for
// every 16 rows up to 128 groups, so that few columns still fill the chip (2011 x 4096: 18.9 us
// with 32 groups).
int grad_groups(int64_t rows) { return rows <= 64 ? 1 : (int)std::min<int64_t>((rows + 15) / 16, 128); }

// A thread takes eight columns of its group's rows (a contiguous range),
// ascending, and holds their column sums. With one group the sums are the
// bias gradients themselves (b0, b1); otherwise they go to partial.
// Bounded by HBM: 4096 x 10240 bf16 with a gate, 420 MB in 73 us (5.7 TB/s).
template <DT D, bool ALN, bool GLU>
__global__ __launch_bounds__(256) void k_act_grad(const void* dy, const void* p, const void* u, void* d0, void* d1,
                                                  float* partial, void* b0, void* b1, int64_t rows, int64_t cols, int act) {
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
      float g[8], x[8], y[8], df[8];
      load8<D, ALN>(dy, i, left, g);
      if (p) {
        load8<D, ALN>(p, i, left, x);
        act_slope_n<D, 8>(act, x, df);
      }
      if (GLU) {
        load8<D, ALN>(u, i, left, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] = g[e] * x[e];
          g[e] = g[e] * y[e] * df[e];
          s0[e] = s0[e] + g[e];
          s1[e] = s1[e] + x[e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (p) g[e] = g[e] * df[e];
          s0[e] = s0[e] + g[e];
        }
      }
      if (d0) store8<D, ALN>(d0, i, left, g);
      if (GLU && d1) store8<D, ALN>(d1, i, left, x);
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
      if (col < cols) {
        const float sum =
            ((red[0][j >> 3][j & 7] + red[1][j >> 3][j & 7]) + red[2][j >> 3][j & 7]) + red[3][j >> 3][j & 7];
        if (gridDim.y == 1) st<D>(h ? b1 : b0, col, sum);
        else partial[((int64_t)blockIdx.y * (GLU ? 2 : 1) + h) * cols + col] = sum;
      }
    }
  }
}

template <DT D, bool ALN>
static hipError_t act_grad(const void* dy, const void* p, const void* u, void* d0, void* d1, float* partial, void* b0,
                           void* b1, int64_t rows, int64_t cols, int act, hipStream_t s) {
  const dim3 grid((unsigned)((cols + 511) / 512), (unsigned)grad_groups(rows));
  return u ? launch(nullptr, k_act_grad<D, ALN, true>, grid, dim3(256), 0, s, dy, p, u, d0, d1, partial, b0, b1, rows, cols, act)
           : launch(nullptr, k_act_grad<D, ALN, false>, grid, dim3(256), 0, s, dy, p, u, d0, d1, partial, b0, b1, rows, cols, act);
}

hipError_t launch_act_grad(const void* dy, const void* p, const void* u, void* d0, void* d1, float* partial, void* b0,
                           void* b1, int64_t rows, int64_t cols, int act, int dtype, bool aligned, hipStream_t s) {
  if (rows == 0) return hipSuccess;
  auto run = [&](auto f) { return f(dy, p, u, d0, d1, partial, b0, b1, rows, cols, act, s); };
  hipError_t e;
  if (dtype == HCLRMIX_BF16) e = run(aligned ? act_grad<DT::BF16, true> : act_grad<DT::BF16, false>);
  else if (dtype == HCLRMIX_F16) e = run(aligned ? act_grad<DT::F16, true> : act_grad<DT::F16, false>);
  else e = run(aligned ? act_grad<DT::F32, true> : act_grad<DT::F32, false>);
  const int groups = grad_groups(rows);
  if (e == hipSuccess && partial && groups > 1)
    e = launch_column_sums(partial, groups, (u ? 2 : 1) * cols, cols, b0, b1, dtype, s);
  return e;
}

}  // namespace hc
