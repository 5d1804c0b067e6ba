// Attention of one new token per sequence over a paged key-value cache (sage_paged_attn).
//
//   t_j = sm_scale q.k_j, capped to cap tanh(t_j / cap), less slope |pos_q - pos_j|
//   out = sum_j softmax(t)_j v_j over the sequence's held tokens, lse = ln sum_j exp t_j
//
// Every held K and V row is read once, so DRAM bounds it. The query heads of one key/value
// head are the (at most 16) rows of an m16n8k16 product: a tcgen05 tile would have 128 rows, of which
// a decode step fills the same few, and the tensor work here is a small part of what the memory
// time allows.
//
// Split: the (sequence, head, 64-key tile) items of the whole batch form one line, cut into equal
// ranges, one per CTA, so the load is even whatever the lengths (which only the device knows). Each
// warp takes 16 keys of a tile through its own ring of cp.async stages and keeps its own running
// maximum, sum and accumulator; no barrier runs inside a range. At a (sequence, head)'s last tile
// in a range the warps are merged in a fixed order; a result that lies in one range is written
// out, others go to the workspace and the join kernel sums them in the order of the ranges, so
// results do not depend on timing.
#include <cmath>

#include "../../include/sageattn.h"
#include "launch.h"
#include "paged.cuh"
#include "sm103_ptx.cuh"

namespace sage {
namespace {

constexpr int kWarps = 4;
constexpr int kKeys = 16;                  // keys per warp and tile
constexpr int kTile = kWarps * kKeys;      // keys per tile
constexpr int kCtas = 304;                 // two resident CTAs per SM
constexpr int kRows = 16;                  // query heads per row block
constexpr int kMinTiles = 2;               // tiles a CTA takes at least
constexpr float kLog2eF = 1.4426950408889634f, kLn2F = 0.6931471805599453f;

struct DecodeArgs {
  PagedView c;
  const void* q; int64_t q_sb, q_sh;
  void* o; int64_t o_sb, o_sh;
  float* lse;               // [batch, hq] or null
  const float* slopes;      // [hq] or null
  const int* q_pos;         // [batch] or null (length - 1)
  float sm_scale, cap;
  int hq, group, row_blocks, max_len, vec;
  // workspace
  int* err;                 // status word
  int* cta_err;             // [kCtas]
  float* part_o;            // [kCtas][2][kRows][dp]
  float* part_ml;           // [kCtas][2][kRows][2]
  float* lse2;              // [batch, hq], base 2 (with mass)
  float* scores;            // [batch, hq, score_pitch], base 2 (with mass) or null
  int64_t score_pitch;
};

template <int DP>
struct DecodeCfg {
  static constexpr int kStages = DP == 128 ? 3 : 6;
  static constexpr int kRowBytes = DP * 2;
  static constexpr int kTileBytes = kKeys * kRowBytes;        // K or V of one warp's tile
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kWarpBytes = kStages * kStageBytes;
  static constexpr int kOffMerge = kWarps * kWarpBytes;       // two warps' accumulators
  static constexpr int kOffMl = kOffMerge + 2 * kRows * DP * 4;
  static constexpr int kSmem = kOffMl + kWarps * kRows * 2 * 4 + 64;
};

// Tiles of a sequence of n tokens.
__device__ __forceinline__ int tiles_of(int n) { return (n + kTile - 1) / kTile; }

// Total number of (sequence, head, tile) items and, for the item index `at`, its sequence and its place
// there. All threads call it; lengths that are out of range count as 0 and set `bad`.
struct Found {
  long long total, base;
  int b;
};
__device__ Found find_item(const DecodeArgs& a, int heads, long long at, bool& bad) {
  __shared__ long long s_sum[32];
  __shared__ long long s_base;
  __shared__ int s_b;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  if (threadIdx.x == 0) { s_b = a.c.batch; s_base = 0; }
  long long run = 0;
  for (int b0 = 0; b0 < a.c.batch; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    long long n = 0;
    if (b < a.c.batch) {
      const int len = checked_len(a.c, b, a.max_len);
      if (len < 0) bad = true;
      n = (long long)tiles_of(max(len, 0)) * heads;
    }
    long long inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    __syncthreads();
    if (lane == 31) s_sum[warp] = inc;
    __syncthreads();
    long long before = run, all = 0;
    for (int w = 0; w < nw; ++w) {
      if (w < warp) before += s_sum[w];
      all += s_sum[w];
    }
    const long long lo = before + inc - n;
    if (n > 0 && at >= lo && at < lo + n) { s_b = b; s_base = lo; }
    run += all;
  }
  __syncthreads();
  return {run, s_base, s_b};
}

// CTAs that share `total` items, and the first item of CTA i.
__device__ __forceinline__ int ctas_of(long long total) {
  const long long g = (total + kMinTiles - 1) / kMinTiles;
  return (int)(g < kCtas ? g : kCtas);
}
__device__ __forceinline__ long long first_item(long long total, int ctas, int i) {
  return total * i / ctas;
}

// One place on the line of items.
struct Cursor {
  int b, h, tile, tiles, len;  // h: head * row_blocks + row block
};
__device__ __forceinline__ void next_item(const DecodeArgs& a, int heads, Cursor& u) {
  if (++u.tile < u.tiles) return;
  u.tile = 0;
  if (++u.h < heads) return;
  u.h = 0;
  do {
    ++u.b;
    u.len = u.b < a.c.batch ? max(checked_len(a.c, u.b, a.max_len), 0) : 0;
  } while (u.b < a.c.batch && u.len == 0);
  u.tiles = tiles_of(u.len);
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
template <typename T>
__device__ __forceinline__ T round_to(float x) {
  if constexpr (std::is_same<T, __half>::value) return __float2half_rn(x);
  else return __float2bfloat16_rn(x);
}

// The 16 keys of item u that belong to this warp into one stage: K rows, then V rows, 16-byte chunk c of
// row r at chunk c ^ (r & 7). `page` is the page of row (lane & 15) or -1 where nothing is read;
// such rows and the channels past d become zero, so they add exactly nothing.
template <typename T, int DP>
__device__ __forceinline__ void load_stage(const DecodeArgs& a, const Cursor& u, int page, int slot,
                                           uint8_t* stage) {
  using C = DecodeCfg<DP>;
  const int lane = threadIdx.x & 31;
  const int h = u.h / a.row_blocks;
  const T* kb = static_cast<const T*>(a.c.k) + h * a.c.k_sh;
  const T* vb = static_cast<const T*>(a.c.v) + h * a.c.v_sh;
  constexpr int kChunks = DP / 8, kRowsPer = 32 / kChunks;  // rows that one pass of the warp covers
  const int c = lane % kChunks;
  const uint32_t base = smem_u32(stage);
#pragma unroll
  for (int i = 0; i < kKeys / kRowsPer; ++i) {
    const int r = i * kRowsPer + lane / kChunks;
    const int pg = __shfl_sync(0xffffffffu, page, r), sl = __shfl_sync(0xffffffffu, slot, r);
    const bool in = pg >= 0 && c * 8 < a.c.d;
    const int off = r * C::kRowBytes + ((c ^ (r & 7)) << 4);
    const T* ks = in ? kb + pg * a.c.k_sp + sl * a.c.k_st + c * 8 : kb;
    const T* vs = in ? vb + pg * a.c.v_sp + sl * a.c.v_st + c * 8 : vb;
    if (a.vec) {
      cp_async16(base + off, ks, in ? 16 : 0);
      cp_async16(base + C::kTileBytes + off, vs, in ? 16 : 0);
    } else {
      // rows that no 16-byte load fits: element loads
      T* kd = reinterpret_cast<T*>(stage + off);
      T* vd = reinterpret_cast<T*>(stage + C::kTileBytes + off);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const bool ok = in && c * 8 + e < a.c.d;
        kd[e] = ok ? ks[e] : T(0.0f);
        vd[e] = ok ? vs[e] : T(0.0f);
      }
    }
  }
}

// Page (or -1) and slot of this lane's row (lane & 15) of this warp's part of item u.
__device__ __forceinline__ void find_page(const DecodeArgs& a, const Cursor& u, bool live, int& page, int& slot,
                                          int& err) {
  page = -1;
  slot = 0;
  const int key = u.tile * kTile + (threadIdx.x >> 5) * kKeys + (threadIdx.x & 15);
  if (!live || key >= u.len) return;
  const int i = key / a.c.page_size;
  slot = key - i * a.c.page_size;
  const int pg = __ldg(&a.c.table[u.b * a.c.table_stride + i]);
  if (pg >= 0 && pg < a.c.num_pages) page = pg;
  else err = kDevPage;
}

// Rows r0 and r0 + 8 of a finished (sequence, head) from one warp's accumulators.
template <typename T, int DP>
__device__ __forceinline__ void write_rows(const DecodeArgs& a, int b, int row0, int rows,
                                           const float (&o)[DP / 8][4], float m0, float m1, float l0, float l1) {
  const int lane = threadIdx.x & 31, cq = (lane & 3) * 2;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int r = (lane >> 2) + half * 8;
    if (r >= rows) continue;
    const float m = half ? m1 : m0, l = half ? l1 : l0;
    const float inv = l != 0.f ? 1.0f / l : 0.f;
    T* dst = static_cast<T*>(a.o) + b * a.o_sb + (row0 + r) * a.o_sh;
#pragma unroll
    for (int n = 0; n < DP / 8; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (n * 8 + cq + e < a.c.d) dst[n * 8 + cq + e] = round_to<T>(o[n][2 * half + e] * inv);
    if ((lane & 3) == 0) {
      const float l2 = l != 0.f ? m + log2f(l) : -INFINITY;
      if (a.lse) a.lse[(int64_t)b * a.hq + row0 + r] = l2 * kLn2F;
      if (a.scores) a.lse2[(int64_t)b * a.hq + row0 + r] = l2;
    }
  }
}

template <typename T, int DP>
__global__ void __launch_bounds__(kWarps * 32, 2) decode_kernel(const DecodeArgs a) {
  using C = DecodeCfg<DP>;
  constexpr int S = C::kStages, KS = DP / 16, NT = DP / 8;
  extern __shared__ __align__(128) uint8_t sm[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int heads = a.c.hkv * a.row_blocks;
  uint8_t* const ring = sm + warp * C::kWarpBytes;
  float* const merge = reinterpret_cast<float*>(sm + C::kOffMerge);
  float* const ml = reinterpret_cast<float*>(sm + C::kOffMl);
  pdl_wait();
  bool bad = false;
  int err = 0;
  // total first (any item index finds it), then this CTA's first item
  const long long total = find_item(a, heads, 0, bad).total;
  const int ctas = total > 0 ? ctas_of(total) : 0;
  const int me = blockIdx.x;
  if (bad) err = kDevSeqlens;
  long long left = 0;
  Cursor cu{a.c.batch, 0, 0, 1, 0};
  if (me < ctas) {
    const long long i0 = first_item(total, ctas, me);
    left = first_item(total, ctas, me + 1) - i0;
    const Found f = find_item(a, heads, i0, bad);
    cu.b = f.b;
    cu.len = checked_len(a.c, cu.b, a.max_len);
    cu.tiles = tiles_of(cu.len);
    const long long in = i0 - f.base;
    cu.h = (int)(in / cu.tiles);
    cu.tile = (int)(in - (long long)cu.h * cu.tiles);
  }
  pdl_trigger();

  // ---- fill the ring: S - 1 stages in flight, the page of the stage after them already read
  Cursor ld = cu;
  long long to_load = left;
  int page, slot;
  find_page(a, ld, to_load > 0, page, slot, err);
#pragma unroll 1
  for (int s = 0; s < S - 1; ++s) {
    if (to_load > 0) {
      load_stage<T, DP>(a, ld, page, slot, ring + s * C::kStageBytes);
      next_item(a, heads, ld);
      --to_load;
      find_page(a, ld, to_load > 0, page, slot, err);
    }
    cp_async_commit();
  }

  float o[NT][4], m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
  uint32_t qf[KS][4];
  float sl0 = 0.f, sl1 = 0.f;
  int qpos = 0, rows = 0, row0 = 0, tile0 = 0, pieces = 0;
  bool fresh = true;
  const float scale2 = a.sm_scale * kLog2eF;
  const float cap_in = a.cap > 0.f ? a.sm_scale / a.cap : 0.f, cap_out = a.cap * kLog2eF;
  int stage = 0;
  const int r0 = lane >> 2, cq = (lane & 3) * 2;

#pragma unroll 1
  for (; left > 0; --left) {
    if (fresh) {
      // a new (sequence, head): its query rows as the A operand, its statistics
      fresh = false;
      tile0 = cu.tile;
      const int h = cu.h / a.row_blocks, rb = cu.h - h * a.row_blocks;
      row0 = h * a.group + rb * kRows;
      rows = min(kRows, a.group - rb * kRows);
      const T* qb = static_cast<const T*>(a.q) + cu.b * a.q_sb;
      auto at = [&](int r, int c) {
        return r < rows && c < a.c.d ? qb[(row0 + r) * a.q_sh + c] : T(0.0f);
      };
      auto two = [&](int r, int c) {
        T x[2] = {at(r, c), at(r, c + 1)};
        return *reinterpret_cast<const uint32_t*>(x);
      };
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        qf[k][0] = two(r0, k * 16 + cq);
        qf[k][1] = two(r0 + 8, k * 16 + cq);
        qf[k][2] = two(r0, k * 16 + 8 + cq);
        qf[k][3] = two(r0 + 8, k * 16 + 8 + cq);
      }
      sl0 = sl1 = 0.f;
      if (a.slopes) {
        if (r0 < rows) sl0 = __ldg(&a.slopes[row0 + r0]) * kLog2eF;
        if (r0 + 8 < rows) sl1 = __ldg(&a.slopes[row0 + r0 + 8]) * kLog2eF;
      }
      qpos = a.q_pos ? __ldg(&a.q_pos[cu.b]) : cu.len - 1;
#pragma unroll
      for (int n = 0; n < NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
      m0 = m1 = -INFINITY;
      l0 = l1 = 0.f;
    }
    // the stage after the ones in flight goes where the previous item was
    {
      __syncwarp();
      const int fill = stage == 0 ? S - 1 : stage - 1;
      if (to_load > 0) {
        load_stage<T, DP>(a, ld, page, slot, ring + fill * C::kStageBytes);
        next_item(a, heads, ld);
        --to_load;
        find_page(a, ld, to_load > 0, page, slot, err);
      }
      cp_async_commit();
      cp_async_wait<S - 1>();
      __syncwarp();
    }
    const int key0 = cu.tile * kTile + warp * kKeys;
    if (key0 < cu.len) {
      const uint32_t kb = smem_u32(ring + stage * C::kStageBytes), vb = kb + C::kTileBytes;
      // S = Q K^T: lanes 0-7 / 8-15 address keys 0-7 at channels +0 / +8, 16-23 / 24-31 keys 8-15
      float s[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
      {
        const int r = (lane & 7) + ((lane >> 4) << 3);
        const uint32_t row = kb + r * C::kRowBytes;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          uint32_t b[4];
          const int c = 2 * k + ((lane >> 3) & 1);
          ldsm4(row + ((c ^ (r & 7)) << 4), b);
          mma16816<T>(s[0], qf[k], b[0], b[1]);
          mma16816<T>(s[1], qf[k], b[2], b[3]);
        }
      }
      // scores in base 2; lane holds keys 8 n + cq, + 1 of rows r0 (s[n][0..1]) and r0 + 8
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int key = key0 + n * 8 + cq + e;
          float x0 = s[n][e], x1 = s[n][2 + e];
          if (a.cap > 0.f) {
            x0 = tanhf(x0 * cap_in) * cap_out;
            x1 = tanhf(x1 * cap_in) * cap_out;
          } else {
            x0 *= scale2;
            x1 *= scale2;
          }
          const bool in = key < cu.len;
          if (a.slopes) {
            int kp = key;
            if (a.c.pos && in) {
              const int i = key / a.c.page_size;
              const int pg = __ldg(&a.c.table[cu.b * a.c.table_stride + i]);
              if (pg >= 0 && pg < a.c.num_pages)
                kp = __ldg(&a.c.pos[plane_at(a.c, pg, cu.h / a.row_blocks, key - i * a.c.page_size)]);
            }
            const float dist = fabsf((float)((long long)qpos - kp));
            x0 = fmaf(-sl0, dist, x0);
            x1 = fmaf(-sl1, dist, x1);
          }
          s[n][e] = in ? x0 : -INFINITY;
          s[n][2 + e] = in ? x1 : -INFINITY;
        }
      if (a.scores) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int key = key0 + n * 8 + cq + e;
            if (key < cu.len) {
              float* dst = a.scores + ((int64_t)cu.b * a.hq + row0 + r0) * a.score_pitch + key;
              if (r0 < rows) dst[0] = s[n][e];
              if (r0 + 8 < rows) dst[8 * a.score_pitch] = s[n][2 + e];
            }
          }
      }
      // running maximum and sum of the rows (the four lanes of a row agree on the maximum)
      float x0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
      float x1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
#pragma unroll
      for (int w = 1; w < 4; w <<= 1) {
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, w));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, w));
      }
      const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
      const float u0 = n0 == -INFINITY ? 0.f : n0, u1 = n1 == -INFINITY ? 0.f : n1;
      if (__any_sync(0xffffffffu, n0 > m0 || n1 > m1)) {
        const float f0 = ex2_approx(m0 - u0), f1 = ex2_approx(m1 - u1);
        l0 *= f0;
        l1 *= f1;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          o[n][0] *= f0; o[n][1] *= f0;
          o[n][2] *= f1; o[n][3] *= f1;
        }
        m0 = n0;
        m1 = n1;
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        s[n][0] = ex2_approx(s[n][0] - u0);
        s[n][1] = ex2_approx(s[n][1] - u0);
        s[n][2] = ex2_approx(s[n][2] - u1);
        s[n][3] = ex2_approx(s[n][3] - u1);
      }
      l0 += (s[0][0] + s[0][1]) + (s[1][0] + s[1][1]);
      l1 += (s[0][2] + s[0][3]) + (s[1][2] + s[1][3]);
      // P in the operands' 16-bit type (the one rounding of the weights; their sum stays in
      // 32 bits), which is already the A operand's layout; O += P V
      const uint32_t p[4] = {pack2<T>(s[0][0], s[0][1]), pack2<T>(s[0][2], s[0][3]),
                             pack2<T>(s[1][0], s[1][1]), pack2<T>(s[1][2], s[1][3])};
      {
        const int r = (lane & 7) + (((lane >> 3) & 1) << 3);  // keys 0-7 / 8-15
        const uint32_t row = vb + r * C::kRowBytes;
#pragma unroll
        for (int n = 0; n < NT; n += 2) {
          uint32_t b[4];
          const int c = n + (lane >> 4);
          ldsm4t(row + ((c ^ (r & 7)) << 4), b);
          mma16816<T>(o[n], p, b[0], b[1]);
          mma16816<T>(o[n + 1], p, b[2], b[3]);
        }
      }
    }
    stage = stage + 1 == S ? 0 : stage + 1;
    const bool seg_end = cu.tile + 1 == cu.tiles || left == 1;
    if (seg_end) {
      // ---- merge the warps: sums of a row over its four lanes, then over the warps
#pragma unroll
      for (int w = 1; w < 4; w <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, w);
        l1 += __shfl_xor_sync(0xffffffffu, l1, w);
      }
      if ((lane & 3) == 0) {
        ml[(warp * kRows + r0) * 2] = m0;
        ml[(warp * kRows + r0) * 2 + 1] = l0;
        ml[(warp * kRows + r0 + 8) * 2] = m1;
        ml[(warp * kRows + r0 + 8) * 2 + 1] = l1;
      }
      __syncthreads();
      float M0 = -INFINITY, M1 = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        M0 = fmaxf(M0, ml[(w * kRows + r0) * 2]);
        M1 = fmaxf(M1, ml[(w * kRows + r0 + 8) * 2]);
      }
      const float U0 = M0 == -INFINITY ? 0.f : M0, U1 = M1 == -INFINITY ? 0.f : M1;
      float L0 = 0.f, L1 = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        L0 += ml[(w * kRows + r0) * 2 + 1] * ex2_approx(ml[(w * kRows + r0) * 2] - U0);
        L1 += ml[(w * kRows + r0 + 8) * 2 + 1] * ex2_approx(ml[(w * kRows + r0 + 8) * 2] - U1);
      }
      const float f0 = ex2_approx(m0 - U0), f1 = ex2_approx(m1 - U1);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        o[n][0] *= f0; o[n][1] *= f0;
        o[n][2] *= f1; o[n][3] *= f1;
      }
      // pairs (0, 2) and (1, 3), then (0, 1)
#pragma unroll
      for (int step = 2; step >= 1; step >>= 1) {
        if (warp >= step && warp < 2 * step) {
          float* dst = merge + (warp - step) * kRows * DP;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            *reinterpret_cast<float2*>(dst + r0 * DP + n * 8 + cq) = make_float2(o[n][0], o[n][1]);
            *reinterpret_cast<float2*>(dst + (r0 + 8) * DP + n * 8 + cq) = make_float2(o[n][2], o[n][3]);
          }
        }
        __syncthreads();
        if (warp < step) {
          const float* src = merge + warp * kRows * DP;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const float2 x = *reinterpret_cast<const float2*>(src + r0 * DP + n * 8 + cq);
            const float2 y = *reinterpret_cast<const float2*>(src + (r0 + 8) * DP + n * 8 + cq);
            o[n][0] += x.x; o[n][1] += x.y;
            o[n][2] += y.x; o[n][3] += y.y;
          }
        }
        __syncthreads();
      }
      if (warp == 0) {
        // the whole (sequence, head) in this range: the result; a part of it: to the workspace
        const bool whole = tile0 == 0 && cu.tile + 1 == cu.tiles;
        if (whole) {
          write_rows<T, DP>(a, cu.b, row0, rows, o, M0, M1, L0, L1);
        } else {
          const int64_t at = ((int64_t)me * 2 + (pieces > 0)) * kRows;
          float* po = a.part_o + at * DP;
          float* pm = a.part_ml + at * 2;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int r = r0 + half * 8;
            if (r < rows) {
#pragma unroll
              for (int n = 0; n < NT; ++n)
                *reinterpret_cast<float2*>(po + r * DP + n * 8 + cq) =
                    make_float2(o[n][2 * half], o[n][2 * half + 1]);
              if ((lane & 3) == 0)
                *reinterpret_cast<float2*>(pm + r * 2) = make_float2(half ? M1 : M0, half ? L1 : L0);
            }
          }
        }
      }
      ++pieces;
      fresh = true;
    }
    next_item(a, heads, cu);
  }
  cp_async_wait<0>();
  // this CTA's error, collected by the join kernel (no word to clear before the call)
  __shared__ int s_err[kWarps];
  const int we = __reduce_max_sync(0xffffffffu, err);
  if (lane == 0) s_err[warp] = we;
  __syncthreads();
  if (threadIdx.x == 0) {
    int e = 0;
    for (int w = 0; w < kWarps; ++w) e = max(e, s_err[w]);
    a.cta_err[me] = e;
  }
}

// ------------------------------------------------------------------------------------- join
// One CTA per (row block of a head, sequence): the results that lie in several ranges summed in
// the order of the ranges; sequences that hold nothing get 0 and -inf. CTA (0, 0) also collects the status.
constexpr int kJoinThreads = 256;

template <typename T, int DP>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const DecodeArgs a) {
  __shared__ float s_w[kCtas][kRows];       // weight of each range's piece
  __shared__ float s_m[kRows], s_l[kRows];
  __shared__ __align__(16) float s_acc[kJoinThreads * 4];
  __shared__ long long s_before[kJoinThreads / 32], s_all[kJoinThreads / 32];
  const int heads = a.c.hkv * a.row_blocks;
  const int hb = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  if (hb == 0 && b == 0) {
    int e = 0;
    for (int i = tid; i < kCtas; i += kJoinThreads) e = max(e, a.cta_err[i]);
    e = __reduce_max_sync(0xffffffffu, e);
    if (lane == 0) s_all[warp] = e;
    __syncthreads();
    if (tid == 0) {
      for (int w = 0; w < kJoinThreads / 32; ++w) e = max(e, (int)s_all[w]);
      *a.err = e;
    }
    __syncthreads();
  }
  // items before this sequence, and in all
  long long before = 0, all = 0;
  for (int i = tid; i < a.c.batch; i += kJoinThreads) {
    const long long n = (long long)tiles_of(max(checked_len(a.c, i, a.max_len), 0)) * heads;
    all += n;
    if (i < b) before += n;
  }
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) {
    all += __shfl_xor_sync(0xffffffffu, all, w);
    before += __shfl_xor_sync(0xffffffffu, before, w);
  }
  if (lane == 0) { s_before[warp] = before; s_all[warp] = all; }
  __syncthreads();
  before = all = 0;
  for (int w = 0; w < kJoinThreads / 32; ++w) { before += s_before[w]; all += s_all[w]; }

  const int len = max(checked_len(a.c, b, a.max_len), 0);
  const int h = hb / a.row_blocks, rb = hb - h * a.row_blocks;
  const int row0 = h * a.group + rb * kRows, rows = min(kRows, a.group - rb * kRows);
  if (len == 0) {
    for (int i = tid; i < rows * a.c.d; i += kJoinThreads) {
      const int r = i / a.c.d, c = i - r * a.c.d;
      static_cast<T*>(a.o)[b * a.o_sb + (row0 + r) * a.o_sh + c] = T(0.0f);
    }
    if (a.lse && tid < rows) a.lse[(int64_t)b * a.hq + row0 + tid] = -INFINITY;
    return;
  }
  const long long t0 = before + (long long)hb * tiles_of(len), t1 = t0 + tiles_of(len);
  const int ctas = ctas_of(all);
  // the ranges that hold t0 and t1 - 1: range i is [all i / ctas, all (i + 1) / ctas)
  auto range_of = [&](long long t) { return (int)(((t + 1) * ctas - 1) / all); };
  const int c0 = range_of(t0), c1 = range_of(t1 - 1);
  if (c0 == c1) return;  // written by its own range
  const int parts = c1 - c0 + 1;
  auto piece = [&](int c) { return (int64_t)c * 2 + (first_item(all, ctas, c) < t0 ? 1 : 0); };
  // row statistics: one warp per row
  for (int r = warp; r < rows; r += kJoinThreads / 32) {
    float m = -INFINITY;
    for (int p = lane; p < parts; p += 32) m = fmaxf(m, a.part_ml[(piece(c0 + p) * kRows + r) * 2]);
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
    const float u = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    for (int p = lane; p < parts; p += 32) {
      const float2 x = *reinterpret_cast<const float2*>(a.part_ml + (piece(c0 + p) * kRows + r) * 2);
      const float w = ex2_approx(x.x - u);
      s_w[p][r] = w;
      l += x.y * w;
    }
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
    if (lane == 0) { s_m[r] = m; s_l[r] = l; }
  }
  __syncthreads();
  // accumulators, four channels per thread; threads left over take every n-th piece
  const int cells = rows * (DP / 4);
  const int sets = cells >= kJoinThreads ? 1 : kJoinThreads / cells;
  for (int base = 0; base < cells; base += kJoinThreads) {
    const int set = sets > 1 ? tid / cells : 0;
    const int cell = sets > 1 ? tid - set * cells : base + tid;
    const bool on = set < sets && cell < cells;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const int r = on ? cell / (DP / 4) : 0, c = on ? (cell - r * (DP / 4)) * 4 : 0;
    if (on) {
#pragma unroll 4
      for (int p = set; p < parts; p += sets) {
        const float4 x = *reinterpret_cast<const float4*>(a.part_o + (piece(c0 + p) * kRows + r) * DP + c);
        const float w = s_w[p][r];
        acc.x = fmaf(w, x.x, acc.x); acc.y = fmaf(w, x.y, acc.y);
        acc.z = fmaf(w, x.z, acc.z); acc.w = fmaf(w, x.w, acc.w);
      }
    }
    if (sets > 1) {
      *reinterpret_cast<float4*>(&s_acc[tid * 4]) = acc;
      __syncthreads();
      if (tid < cells)
        for (int s = 1; s < sets; ++s) {
          const float4 x = *reinterpret_cast<const float4*>(&s_acc[(s * cells + tid) * 4]);
          acc.x += x.x; acc.y += x.y; acc.z += x.z; acc.w += x.w;
        }
    }
    if (on && set == 0) {
      const float inv = s_l[r] != 0.f ? 1.0f / s_l[r] : 0.f;
      T* dst = static_cast<T*>(a.o) + b * a.o_sb + (row0 + r) * a.o_sh + c;
      const float y[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c + e < a.c.d) dst[e] = round_to<T>(y[e]);
    }
  }
  if (tid < rows) {
    const float l2 = s_l[tid] != 0.f ? s_m[tid] + log2f(s_l[tid]) : -INFINITY;
    if (a.lse) a.lse[(int64_t)b * a.hq + row0 + tid] = l2 * kLn2F;
    if (a.scores) a.lse2[(int64_t)b * a.hq + row0 + tid] = l2;
  }
}

// --------------------------------------------------------------------------- accumulated weight
// mass += sum over the group's heads of 2^(t - lse2): the scores written by the decode kernel, one thread per
// key. Added atomically, since two sequences may share a page; a page of one sequence gets one
// addition, whose result does not depend on any order.
__global__ void __launch_bounds__(256) mass_kernel(const DecodeArgs a) {
  pdl_wait();
  const int b = blockIdx.z, h = blockIdx.y;
  const int len = max(checked_len(a.c, b, a.max_len), 0);
  const int key = blockIdx.x * 256 + threadIdx.x;
  if (key >= len) return;
  const int i = key / a.c.page_size;
  const int page = __ldg(&a.c.table[b * a.c.table_stride + i]);
  if (page < 0 || page >= a.c.num_pages) return;
  const int64_t row = (int64_t)b * a.hq + h * a.group;
  const float* s = a.scores + row * a.score_pitch + key;
  float sum = 0.f;
#pragma unroll 8
  for (int g = 0; g < a.group; ++g) {
    const float l2 = a.lse2[row + g];
    sum += l2 == -INFINITY ? 0.f : ex2_approx(s[g * a.score_pitch] - l2);
  }
  atomicAdd(&a.c.mass[plane_at(a.c, page, h, key - i * a.c.page_size)], sum);
}

// ------------------------------------------------------------------------------------- host
struct DecodeLayout {
  size_t err, part_o, part_ml, lse2, scores, total;
  int64_t pitch;
};
size_t up256(size_t x) { return (x + 255) / 256 * 256; }
bool decode_layout(int batch, int hq, int hkv, int64_t max_len, int d, bool mass, DecodeLayout* L) {
  if (batch < 0 || hq < 1 || hkv < 1 || hq % hkv || max_len < 0 || d < 1 || d > 128) return false;
  const int dp = d <= 64 ? 64 : 128;
  size_t o = 256 + up256(4 * kCtas);  // status word, then the CTAs' errors
  auto take = [&](size_t bytes) { const size_t at = o; o += up256(bytes); return at; };
  L->err = 256;
  L->part_o = take((size_t)kCtas * 2 * kRows * dp * 4);
  L->part_ml = take((size_t)kCtas * 2 * kRows * 2 * 4);
  L->pitch = (max_len + 3) / 4 * 4;
  L->lse2 = take(mass ? (size_t)batch * hq * 4 : 0);
  L->scores = take(mass ? (size_t)batch * hq * L->pitch * 4 : 0);
  L->total = o;
  return true;
}

template <typename T, int DP>
cudaError_t launch_decode_t(const DecodeArgs& a, cudaStream_t st) {
  static std::atomic<int> limits[64];
  cudaError_t e = raise_smem_limit(decode_kernel<T, DP>, DecodeCfg<DP>::kSmem, limits);
  if (e != cudaSuccess) return e;
  e = launch_pdl(decode_kernel<T, DP>, dim3(kCtas), dim3(kWarps * 32), DecodeCfg<DP>::kSmem, st, a);
  if (e != cudaSuccess) return e;
  e = launch_pdl(join_kernel<T, DP>, dim3(a.c.hkv * a.row_blocks, a.c.batch), dim3(kJoinThreads), 0, st, a);
  if (e != cudaSuccess || !a.scores || a.max_len == 0) return e;
  return launch_pdl(mass_kernel, dim3((a.max_len + 255) / 256, a.c.hkv, a.c.batch), dim3(256), 0, st, a);
}

}  // namespace
}  // namespace sage

using namespace sage;

extern "C" {

size_t sage_paged_attn_workspace_size(int batch, int heads_q, int heads_kv, int max_seqlen, int head_dim,
                                      int accumulate) {
  DecodeLayout L;
  return decode_layout(batch, heads_q, heads_kv, max_seqlen, head_dim, accumulate != 0, &L) ? L.total : 0;
}

int sage_paged_attn(const sage_packed* q, const sage_paged_cache* cache, const sage_packed* out, float* lse,
                    const float* slopes, const int32_t* q_positions, int batch, int heads_q, int heads_kv,
                    int max_seqlen, int head_dim, int dtype, int tensor_layout, float sm_scale, float softcap,
                    void* workspace, size_t workspace_bytes, void* stream) {
  if (!q || !cache || !out) return SAGE_ERR_INVALID_ARG;
  DecodeArgs a{};
  bool vec = false;
  int s = make_paged_view(cache, batch, heads_kv, head_dim, dtype, tensor_layout, &a.c, &vec);
  if (s != SAGE_OK) return s;
  if (heads_q < 1 || max_seqlen < 0 || batch > 65535 || !(softcap >= 0.f) || std::isinf(softcap))
    return SAGE_ERR_INVALID_ARG;
  if (heads_q % heads_kv) return SAGE_ERR_GQA;
  if (batch == 0) return SAGE_OK;
  if (!q->data || !out->data) return SAGE_ERR_INVALID_ARG;
  for (const sage_packed* t : {q, out})
    if (reinterpret_cast<uintptr_t>(t->data) % 2 || t->stride_token < 0 || t->stride_head < 0) return SAGE_ERR_STRIDE;
  for (const void* p : {(const void*)lse, (const void*)slopes, (const void*)q_positions})
    if (reinterpret_cast<uintptr_t>(p) % 4) return SAGE_ERR_INVALID_ARG;
  DecodeLayout L;
  if (!decode_layout(batch, heads_q, heads_kv, max_seqlen, head_dim, cache->mass != nullptr, &L))
    return SAGE_ERR_INVALID_ARG;
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 || workspace_bytes < L.total)
    return SAGE_ERR_WORKSPACE;
  if (!sage_device_supported()) return SAGE_ERR_DEVICE;
  a.q = q->data; a.q_sb = q->stride_token; a.q_sh = q->stride_head;
  a.o = out->data; a.o_sb = out->stride_token; a.o_sh = out->stride_head;
  a.lse = lse;
  a.slopes = slopes;
  a.q_pos = q_positions;
  a.sm_scale = std::isnan(sm_scale) || sm_scale <= 0.f ? (float)(1.0 / std::sqrt((double)head_dim)) : sm_scale;
  a.cap = softcap;
  a.hq = heads_q;
  a.group = heads_q / heads_kv;
  a.row_blocks = (a.group + kRows - 1) / kRows;
  a.max_len = max_seqlen;
  a.vec = vec ? 1 : 0;
  char* w = static_cast<char*>(workspace);
  a.err = reinterpret_cast<int*>(w);
  a.cta_err = reinterpret_cast<int*>(w + L.err);
  a.part_o = reinterpret_cast<float*>(w + L.part_o);
  a.part_ml = reinterpret_cast<float*>(w + L.part_ml);
  if (cache->mass) {
    a.lse2 = reinterpret_cast<float*>(w + L.lse2);
    a.scores = reinterpret_cast<float*>(w + L.scores);
    a.score_pitch = L.pitch;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == SAGE_F16)
    e = head_dim <= 64 ? launch_decode_t<__half, 64>(a, st) : launch_decode_t<__half, 128>(a, st);
  else
    e = head_dim <= 64 ? launch_decode_t<__nv_bfloat16, 64>(a, st) : launch_decode_t<__nv_bfloat16, 128>(a, st);
  return e == cudaSuccess ? SAGE_OK : note_cuda_failure(e, "paged attention");
}

}  // extern "C"
