// The key-value cache in pages: one new token's attention over it (hclrmix_paged_attention), rows stored into it
// (hclrmix_cache_store) and the tables that say where tokens live (hclrmix_page_map).
#include "hc_attn.h"
#include "hc_internal.h"

#include <algorithm>

namespace hc {

// ------------------------------------------------------------------ attention of one token

// A workgroup takes one sequence, one key head with up to 16 of the query heads that share it, and a part of the
// sequence's keys; its waves take tiles of keys in turn, each through buffers of its own, so no wave waits for
// another before the end. As in hc_attn.hip the products are transposed (16 x 16 results here: few rows).
// The cache's rows are read once, by loads that write LDS directly; they bound the kernel.

template <DT D, int NB> struct PagedShape {
  typedef Rows<D, NB> T;
  static constexpr int KT = T::RB <= 128 ? 64 : T::RB >= 1024 && D == DT::F32 ? 16 : 32;  // keys of a tile
  static constexpr int TILE = KT * T::RB;
  static constexpr int RING = 4 * TILE;  // bytes of a wave: two buffers of K and V
  static constexpr int WAVES = RING * 4 <= 131072 ? 4 : 2;
};

struct PagedSeq {
  int len, lo, first;       // keys; the window's first; first tokens
  int head, begin, count;   // tiles [0, head) and from begin on, as one list
  int parts, per;           // parts that the list is cut into, tiles of each
  __device__ __forceinline__ int tile(int i) const { return i < head ? i : i - head + begin; }
};
template <int KT> __device__ __forceinline__ PagedSeq paged_seq(const PagedArgs& a, int b) {
  PagedSeq s;
  s.len = (int)min((int64_t)max(a.lengths[b], 0), (int64_t)a.most_pages * a.page);
  s.lo = a.window ? max(s.len - a.window, 0) : 0;
  s.first = min(a.sinks, s.len);
  const int sink_tiles = (s.first + KT - 1) / KT, end = (s.len + KT - 1) / KT;
  s.begin = s.lo / KT;
  s.head = min(sink_tiles, s.begin);
  if (s.head == s.begin) s.head = s.begin = 0;
  s.count = s.head + end - s.begin;
  const int chunk = a.chunk / KT;
  s.parts = max(1, min(a.splits, (s.count + chunk - 1) / chunk));
  s.per = (s.count + s.parts - 1) / s.parts;
  return s;
}

__device__ __forceinline__ float quarters_max(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return halves_max(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float quarters_sum(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return halves_sum(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

// Where part s of a query head's result lies: dim floats, and its maximum and sum after all of them.
__device__ __forceinline__ float* part_values(const PagedArgs& a, int64_t head, int s) {
  return a.partial + (head * a.splits + s) * a.dim;
}
__device__ __forceinline__ float* part_sums(const PagedArgs& a, int64_t head, int s) {
  return a.partial + (int64_t)a.batch * a.heads * a.splits * a.dim + (head * a.splits + s) * 2;
}

template <DT D, int NB, bool ALN>
__global__ __launch_bounds__((64 * PagedShape<D, NB>::WAVES)) void k_paged(const PagedArgs a) {
  typedef PagedShape<D, NB> F;
  typedef Rows<D, NB> T;
  typedef typename T::piece piece;
  constexpr int KT = F::KT, WAVES = F::WAVES, KB = KT / 16;
  constexpr int STEP = D == DT::F32 ? 16 : 32, STEPS = 32 * NB / STEP;  // contraction of a score
  constexpr int DB = 2 * NB;                                           // blocks of 16 columns
  constexpr int NL = F::TILE / 1024;                                   // loads that fill a tile
  static_assert(16 * 32 * NB * 4 <= F::RING, "a wave's sums fit its buffers");
  __shared__ __attribute__((aligned(1024))) unsigned char lds[WAVES * F::RING];
  __shared__ float stat[WAVES][2][16];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 4;

  // Parts fastest, so that a sequence's parts are in flight together.
  const int blocks = (a.group + 15) / 16;  // of rows
  int id = blockIdx.x;
  const int part = id % a.splits;
  id /= a.splits;
  const int rb = id % blocks;
  id /= blocks;
  const int kvh = id % a.kv_heads, b = id / a.kv_heads;
  const PagedSeq s = paged_seq<KT>(a, b);
  if (part >= s.parts) return;
  const int t0 = part * s.per, t1 = min(t0 + s.per, s.count);
  const int rows = min(16, a.group - rb * 16), head0 = kvh * a.group + rb * 16;

  piece q[STEPS];
  {
    const int r = min(lane & 15, rows - 1);
    const char* p = (const char*)a.q + ((int64_t)b * a.sq.b + (int64_t)(head0 + r) * a.sq.h) * T::ES;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) q[i] = __builtin_bit_cast(piece, chunk16<D, ALN>(p, (4 * i + g) * T::EPC, a.dim));
  }
  f32x4 o[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d) o[d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  float m = NEG_INF, l = 0.0f;
  const float c = a.scale * LOG2E;
  unsigned char* const ring = lds + wave * F::RING;

  // Lane l looks after key l % KT of a tile: the page that holds it, one tile ahead of its loads.
  const int* table = a.table + (int64_t)b * a.table_stride;
  auto page_of = [&](int i) {
    const int j = s.tile(min(i, s.count - 1)) * KT + (lane & (KT - 1));
    return j < s.len ? table[j / a.page] : -1;
  };
  // Its row's offset in the caches, or -1: not seen, or on a page that the cache does not have.
  auto offset_of = [&](int i, int page) {
    const int j = s.tile(i) * KT + (lane & (KT - 1));
    const bool in = j < s.len && (j >= s.lo || j < s.first) && page >= 0 && page < a.pages;
    return in ? (int64_t)page * a.sc.b + (int64_t)(j % a.page) * a.sc.t + (int64_t)kvh * a.sc.h : (int64_t)-1;
  };
  auto stage = [&](int64_t at, unsigned char* to) {
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int row = (i * 64 + lane) / T::CPR, col = ((lane % T::CPR) ^ T::swz(row)) * T::EPC;
      const uint32_t lo = __shfl((uint32_t)at, row, 64), hi = __shfl((uint32_t)((uint64_t)at >> 32), row, 64);
      const int64_t from = (int64_t)((uint64_t)hi << 32 | lo);
      if constexpr (ALN) {
        const bool in = from >= 0 && col < a.dim;
        const char* kp = in ? (const char*)a.k + (from + col) * T::ES : (const char*)zeros16;
        const char* vp = in ? (const char*)a.v + (from + col) * T::ES : (const char*)zeros16;
        const uint32_t dst = __builtin_amdgcn_readfirstlane(lds_offset(to) + i * 1024);
        lds_load_from(kp, dst);
        lds_load_from(vp, dst + F::TILE);
      } else {
        uint4 kv = make_uint4(0u, 0u, 0u, 0u), vv = kv;
        if (from >= 0) {
          kv = chunk16<D, false>((const char*)a.k + from * T::ES, col, a.dim);
          vv = chunk16<D, false>((const char*)a.v + from * T::ES, col, a.dim);
        }
        *(uint4*)(to + i * 1024 + lane * 16) = kv;
        *(uint4*)(to + F::TILE + i * 1024 + lane * 16) = vv;
      }
    }
  };

  int buf = 0, i = t0 + wave;
  int64_t at = -1, next = -1;
  int page = 0;
  if (i < t1) {
    at = offset_of(i, page_of(i));
    stage(at, ring);
    page = page_of(i + WAVES);
  }
  for (; i < t1; i += WAVES, buf ^= 1) {
    // Tile i has arrived (and the pages of the next); the reads of the tile before it are done.
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    const bool more = i + WAVES < t1;
    if (more) {
      next = offset_of(i + WAVES, page);
      stage(next, ring + (buf ^ 1) * 2 * F::TILE);
      page = page_of(i + 2 * WAVES);
    }
    const unsigned char* kt = ring + buf * 2 * F::TILE;
    const unsigned char* vt = kt + F::TILE;
    const uint64_t seen = __ballot(at >= 0);  // bit j: key j of the tile
    f32x4 x[KB];
#pragma unroll
    for (int k = 0; k < KB; ++k) {
      x[k] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int st = 0; st < STEPS; ++st) {
        const int row = 16 * k + (lane & 15);
        const piece f = __builtin_bit_cast(piece, *(const uint4*)(kt + row * T::RB + (((4 * st + g) ^ T::swz(row)) << 4)));
        if constexpr (D == DT::F32) {
#pragma unroll
          for (int e = 0; e < 4; ++e) x[k] = __builtin_amdgcn_mfma_f32_16x16x4f32(f[e], q[st][e], x[k], 0, 0, 0);
        } else {
          x[k] = mfma<D>(f, q[st], x[k]);
        }
      }
    }
    float top = NEG_INF;
#pragma unroll
    for (int k = 0; k < KB; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[k][e] = (seen >> (16 * k + 4 * g + e)) & 1 ? x[k][e] : NEG_INF;
        top = fmaxf(top, x[k][e]);
      }
    top = quarters_max(top) * c;
    const float grown = fmaxf(m, top);
    if (__ballot(grown > m)) {
      const float f = grown == NEG_INF ? 1.0f : __builtin_amdgcn_exp2f(m - grown);
      m = grown;
      l *= f;
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[d][e] *= f;
    }
    // fp16 weights 2^15 times as large: fewer fall below fp16's normal numbers.
    const float base = (D == DT::F16 ? 15.0f : 0.0f) - (m == NEG_INF ? 0.0f : m);
#pragma unroll
    for (int k = 0; k < KB; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[k][e] = __builtin_amdgcn_exp2f(fmaf(x[k][e], c, base));
        l += x[k][e];
      }
    if constexpr (D == DT::F32) {
#pragma unroll
      for (int k = 0; k < KB; ++k)
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int row = 16 * k + 4 * g + e, ch = 4 * d + ((lane & 15) >> 2);
            const float f = *(const float*)(vt + row * T::RB + ((ch ^ T::swz(row)) << 4) + 4 * (lane & 3));
            o[d] = __builtin_amdgcn_mfma_f32_16x16x4f32(f, x[k][e], o[d], 0, 0, 0);
          }
    } else {
#pragma unroll
      for (int k = 0; k < KB; k += 2) {  // contraction over 32 keys: this lane's are 16 k + 4 g .. + 3 and 16 keys further
        const u32x4 w = {pack2<D>(x[k][0], x[k][1]), pack2<D>(x[k][2], x[k][3]), pack2<D>(x[k + 1][0], x[k + 1][1]),
                         pack2<D>(x[k + 1][2], x[k + 1][3])};
        const s16x8 p = __builtin_bit_cast(s16x8, w);
#pragma unroll
        for (int d = 0; d < DB; ++d) {
          const int j = lane & 15, row = 16 * k + 4 * g + (j >> 2), ch = 2 * d + ((j & 3) >> 1);
          lds_u8* v0 = (lds_u8*)(vt + row * T::RB + ((ch ^ T::swz(row)) << 4) + 8 * (j & 1));
          lds_u8* v1 = v0 + 16 * T::RB;  // the permutation repeats every 16 rows
          const s16x4 f0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)v0);
          const s16x4 f1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)v1);
          o[d] = mfma<D>(__builtin_shufflevector(f0, f1, 0, 1, 2, 3, 4, 5, 6, 7), p, o[d]);
        }
      }
    }
    at = next;
  }

  // The waves' results joined in their order: sums of each row in LDS [row][32 NB], in this wave's own buffers.
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  l = quarters_sum(l);
  float* const mine = (float*)ring;
#pragma unroll
  for (int d = 0; d < DB; ++d) *(f32x4*)(mine + (lane & 15) * (32 * NB) + 16 * d + 4 * g) = o[d];
  if (lane < 16) {
    stat[wave][0][lane] = m;
    stat[wave][1][lane] = l;
  }
  __syncthreads();
  for (int e = tid; e < rows * a.dim; e += 64 * WAVES) {
    const int r = e / a.dim, col = e - r * a.dim;
    float top = stat[0][0][r];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) top = fmaxf(top, stat[w][0][r]);
    float sum = 0.0f, y = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      const float f = stat[w][0][r] == NEG_INF ? 0.0f : __builtin_amdgcn_exp2f(stat[w][0][r] - top);
      sum = sum + f * stat[w][1][r];
      y = y + f * ((const float*)(lds + w * F::RING))[r * (32 * NB) + col];
    }
    const int64_t head = (int64_t)b * a.heads + head0 + r;
    if (s.parts == 1) {
      st<D>(a.out, (int64_t)b * a.so.b + (int64_t)(head0 + r) * a.so.h + col, sum == 0.0f ? 0.0f : y / sum);
    } else {
      part_values(a, head, part)[col] = y;
      if (col == 0) {
        part_sums(a, head, part)[0] = top;
        part_sums(a, head, part)[1] = sum;
      }
    }
  }
}

// The parts of one query head joined in ascending order.
template <DT D, int KT> __global__ __launch_bounds__(256) void k_paged_join(const PagedArgs a) {
  __shared__ float sum4[4], y4[4][256];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t head = blockIdx.x;
  const int b = (int)(head / a.heads), h = (int)(head - (int64_t)b * a.heads);
  const PagedSeq s = paged_seq<KT>(a, b);
  if (s.parts == 1) return;
  const int used = (s.count + s.per - 1) / s.per;  // parts that hold tiles
  // Wave w takes the parts w, w + 4, ...; the maximum first.
  float top = NEG_INF;
  for (int p = lane; p < used; p += 64) top = fmaxf(top, part_sums(a, head, p)[0]);
#pragma unroll
  for (int d = 32; d; d >>= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
  float sum = 0.0f, y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int p = wave; p < used; p += 4) {
    const float pm = part_sums(a, head, p)[0];
    const float f = pm == NEG_INF ? 0.0f : __builtin_amdgcn_exp2f(pm - top);
    sum = sum + f * part_sums(a, head, p)[1];
    const float* v = part_values(a, head, p);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (lane + 64 * i < a.dim) y[i] = y[i] + f * v[lane + 64 * i];
  }
  if (lane == 0) sum4[wave] = sum;
#pragma unroll
  for (int i = 0; i < 4; ++i) y4[wave][lane + 64 * i] = y[i];
  __syncthreads();
  if (tid < a.dim) {
    const float total = ((sum4[0] + sum4[1]) + sum4[2]) + sum4[3];
    const float v = ((y4[0][tid] + y4[1][tid]) + y4[2][tid]) + y4[3][tid];
    st<D>(a.out, (int64_t)b * a.so.b + (int64_t)h * a.so.h + tid, total == 0.0f ? 0.0f : v / total);
  }
}

namespace {

// Parts: enough workgroups to fill the card several times over where the sequences are long, each with at least
// two tiles a wave, and no more than 1024 keys where there are many anyway (ragged lengths even out).
template <DT D, int NB> void plan(PagedArgs& a) {
  typedef PagedShape<D, NB> F;
  const int64_t most = std::max<int64_t>((int64_t)a.most_pages * a.page, 1);  // keys
  const int64_t pairs = (int64_t)a.batch * a.kv_heads * ((a.group + 15) / 16);
  const int64_t least = 2 * F::KT * F::WAVES;
  int64_t chunk = most * pairs / 1024;
  chunk = std::min<int64_t>(std::max(chunk, least), 1024);
  chunk = (chunk + F::KT - 1) / F::KT * F::KT;
  a.chunk = (int)chunk;
  // A launch holds 2^24 workgroups of 256 threads.
  a.splits = (int)std::min<int64_t>(std::min<int64_t>((most + chunk - 1) / chunk, 128), std::max<int64_t>((1 << 23) / pairs, 1));
}

// The most workgroups times parts that plan() gives to as many pairs and keys or fewer: it ascends in both.
template <DT D, int NB> int64_t most_parts(const PagedArgs& a) {
  typedef PagedShape<D, NB> F;
  const int64_t most = std::max<int64_t>((int64_t)a.most_pages * a.page, 1), least = 2 * F::KT * F::WAVES;
  const int64_t pairs = (int64_t)a.batch * a.kv_heads * ((a.group + 15) / 16);
  return std::min(pairs * std::min<int64_t>((most + least - 1) / least, 128),
                  std::max<int64_t>(1024 + pairs, pairs * std::min<int64_t>((most + 1023) / 1024, 128)));
}

template <DT D, int NB> hipError_t go(PagedArgs a, bool aligned, hipStream_t s) {
  typedef PagedShape<D, NB> F;
  plan<D, NB>(a);
  const int64_t groups = (int64_t)a.batch * a.kv_heads * ((a.group + 15) / 16) * a.splits;
  const dim3 grid((unsigned)groups), block(64 * F::WAVES);
  if (aligned) hipLaunchKernelGGL((k_paged<D, NB, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((k_paged<D, NB, false>), grid, block, 0, s, a);
  if (a.splits > 1)
    hipLaunchKernelGGL((k_paged_join<D, F::KT>), dim3((unsigned)(a.batch * a.heads)), dim3(256), 0, s, a);
  return hipGetLastError();
}
template <DT D> hipError_t go_dim(const PagedArgs& a, bool aligned, hipStream_t s) {
  if (a.dim <= 64) return go<D, 2>(a, aligned, s);
  if (a.dim <= 128) return go<D, 4>(a, aligned, s);
  return go<D, 8>(a, aligned, s);
}
template <DT D> int64_t parts_dim(const PagedArgs& a) {
  return a.dim <= 64 ? most_parts<D, 2>(a) : a.dim <= 128 ? most_parts<D, 4>(a) : most_parts<D, 8>(a);
}

}  // namespace

hipError_t launch_paged(PagedArgs a, int dtype, bool aligned, hipStream_t s) {
  switch (dtype) {
    case (int)DT::F32: return go_dim<DT::F32>(a, aligned, s);
    case (int)DT::F16: return go_dim<DT::F16>(a, aligned, s);
    default: return go_dim<DT::BF16>(a, aligned, s);
  }
}

size_t paged_scratch(const PagedArgs& a, int dtype) {
  if (a.batch == 0) return 0;
  const int64_t parts = dtype == (int)DT::F32 ? parts_dim<DT::F32>(a) : parts_dim<DT::BF16>(a);  // fp16 has bf16's shapes
  const int blocks = (a.group + 15) / 16;
  return (size_t)parts * ((a.group + blocks - 1) / blocks) * ((size_t)a.dim + 2) * sizeof(float);
}

// ------------------------------------------------------------------ rows into the cache

// One thread per 16 bytes of a row (aligned) or per element. Bound by HBM, or by the launch for a step's tokens.
template <typename E> __global__ __launch_bounds__(256) void k_store(const StoreArgs a, int per_head) {
  const int64_t n = a.tokens * a.kv_heads * per_head;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / per_head;
    const int c = (int)(i - row * per_head);
    const int64_t t = row / a.kv_heads;
    const int h = (int)(row - t * a.kv_heads);
    const int slot = a.slots[t];
    if (slot < 0) continue;
    const int64_t page = slot / a.page;
    if (page >= a.pages) continue;
    const int64_t to = page * a.sc.b + (int64_t)(slot - (int)page * a.page) * a.sc.t + (int64_t)h * a.sc.h + c;
    ((E*)a.kc)[to] = ((const E*)a.k)[t * a.sk.t + (int64_t)h * a.sk.h + c];
    ((E*)a.vc)[to] = ((const E*)a.v)[t * a.sv.t + (int64_t)h * a.sv.h + c];
  }
}

hipError_t launch_store(const StoreArgs& a0, int dtype, bool aligned, hipStream_t s) {
  StoreArgs a = a0;
  const int es = dtype == (int)DT::F32 ? 4 : 2, unit = aligned ? 16 / es : 1;
  for (Strides3* x : {&a.sk, &a.sv, &a.sc}) {  // in units
    x->b /= unit;
    x->t /= unit;
    x->h /= unit;
  }
  const int per_head = a.dim / unit;
  const int64_t n = a.tokens * a.kv_heads * per_head;
  const dim3 grid((unsigned)std::min<int64_t>((n + 255) / 256, 1 << 20)), block(256);
  if (aligned) hipLaunchKernelGGL(k_store<uint4>, grid, block, 0, s, a, per_head);
  else if (es == 4) hipLaunchKernelGGL(k_store<uint32_t>, grid, block, 0, s, a, per_head);
  else hipLaunchKernelGGL(k_store<uint16_t>, grid, block, 0, s, a, per_head);
  return hipGetLastError();
}

// ------------------------------------------------------------------ tables

// Two sums over the requests (new tokens, pages to take), then one number per token and per page. The sums are of
// 64 bits and are written held to 32.
constexpr int MAP_THREADS = 1024;

__device__ __forceinline__ int to_int(int64_t x) { return (int)min(x, (int64_t)0x7FFFFFFF); }
struct Request {
  int64_t cached, fresh, held, missing;
};
__device__ __forceinline__ Request request(const MapArgs& a, int b) {
  Request r;
  r.cached = max(a.cached[b], 0);
  r.fresh = max(a.fresh[b], 0);
  r.held = (r.cached + a.page - 1) / a.page;
  r.missing = (r.cached + r.fresh + a.page - 1) / a.page - r.held;
  return r;
}
__device__ __forceinline__ int64_t wave_scan(int64_t x, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t y = __shfl_up((long long)x, d, 64);
    if (lane >= d) x += y;
  }
  return x;
}
// Inclusive sums of x and y over the workgroup's threads.
__device__ __forceinline__ void group_scan(int64_t& x, int64_t& y, int64_t (*part)[2], int tid) {
  const int lane = tid & 63, wave = tid >> 6;
  x = wave_scan(x, lane);
  y = wave_scan(y, lane);
  if (lane == 63) {
    part[wave][0] = x;
    part[wave][1] = y;
  }
  __syncthreads();
  int64_t px = 0, py = 0;
  for (int w = 0; w < wave; ++w) {
    px += part[w][0];
    py += part[w][1];
  }
  x += px;
  y += py;
  __syncthreads();
}

// The last index i with sums[i] <= t (sums ascend from 0, n + 1 of them; t < sums[n]).
__device__ __forceinline__ int find_in(const int* sums, int n, int t) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ __launch_bounds__(MAP_THREADS) void k_page_sums(const MapArgs a) {
  __shared__ int64_t part[MAP_THREADS / 64][2];
  __shared__ int64_t carry[2];
  const int tid = threadIdx.x;
  if (tid == 0) {
    carry[0] = carry[1] = 0;
    a.starts[0] = a.taken[0] = 0;
  }
  __syncthreads();
  for (int b0 = 0; b0 < a.batch; b0 += MAP_THREADS) {
    const int b = b0 + tid;
    int64_t x = 0, y = 0;
    if (b < a.batch) {
      const Request r = request(a, b);
      x = r.fresh;
      y = r.missing;
      a.lengths[b] = to_int(r.cached + r.fresh);
    }
    group_scan(x, y, part, tid);
    x += carry[0];
    y += carry[1];
    if (b < a.batch) {
      a.starts[b + 1] = to_int(x);
      a.taken[b + 1] = to_int(y);
    }
    __syncthreads();
    if (tid == MAP_THREADS - 1) {
      carry[0] = x;
      carry[1] = y;
    }
    __syncthreads();
  }
}

__device__ __forceinline__ void fill_maps(const MapArgs& a, const int* starts, const int* taken) {
  const int64_t first = a.free_start ? max(*a.free_start, 0) : 0;
  const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, all = (int64_t)gridDim.x * blockDim.x;
  const int tokens = starts[a.batch], pages = taken[a.batch];
  auto page_from = [&](int64_t u) { return first + u < a.free_count ? a.free_pages[first + u] : -1; };
  for (int64_t t = id; t < a.tokens; t += all) {
    int pos = 0, slot = -1;
    if (t < tokens) {
      const int b = find_in(starts, a.batch, (int)t);
      const int64_t held = ((int64_t)max(a.cached[b], 0) + a.page - 1) / a.page;
      const int64_t p = (int64_t)max(a.cached[b], 0) + t - starts[b], at = p / a.page;
      pos = to_int(p);
      int page = -1;
      if (at < a.most_pages) page = at < held ? a.table[b * a.table_stride + at] : page_from(taken[b] + at - held);
      const int64_t x = (int64_t)page * a.page + (p - at * a.page);
      slot = page >= 0 && x <= 0x7FFFFFFF ? (int)x : -1;
    }
    a.positions[t] = pos;
    a.slots[t] = slot;
  }
  for (int64_t u = id; u < pages; u += all) {
    const int b = find_in(taken, a.batch, (int)u);
    const int64_t held = ((int64_t)max(a.cached[b], 0) + a.page - 1) / a.page, at = held + u - taken[b];
    if (at < a.most_pages) a.table[b * a.table_stride + at] = page_from(u);
  }
}

__global__ __launch_bounds__(256) void k_page_fill(const MapArgs a) { fill_maps(a, a.starts, a.taken); }

hipError_t launch_page_map(const MapArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(k_page_sums, dim3(1), dim3(MAP_THREADS), 0, s, a);
  const int64_t n = std::max<int64_t>(a.tokens, a.batch);
  if (a.batch > 0 || a.tokens > 0)
    hipLaunchKernelGGL(k_page_fill, dim3((unsigned)std::min<int64_t>((n + 255) / 256, 2048)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace hc
