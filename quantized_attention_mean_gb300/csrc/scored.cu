// Attention with modified scores on 16-bit operands (sage_scored_attn): tanh cap, distance bias,
// causal, prefix and document masks.
//
//   s = sm_scale q.k; s = cap tanh(s / cap); s -= slope |i + q_offset - j|; softmax over visible j; times v
//
// One CTA owns two 128-row query tiles (A, B) of one (sequence, head) and walks the 128-key tiles that any of its
// rows may see:
//   warp 8      TMA: Q once, then K and V tiles through rings of stages, straight from the caller's tensors
//   warps 9, 10 issue tile A's and tile B's MMAs: S = Q K^T (both operands in shared memory) and O += P V with P
//               in tensor memory and V in its own row order (an MN-major operand), so nothing is transposed
//   warp 11     with documents: zeroes the V rows of padding before their tile is multiplied
//   warps 0-3, 4-7   softmax of tile A / B, one thread per row: S from tensor memory, score
//               modification, mask, running maximum and sum, P written over S's columns
// P overlays its own S buffer: P V of an item and the product that refills the buffer are
// issued in this order by one thread, and MMAs of a thread run in order. Three S buffers rotate over the items
// at head_dim 64, two at 128 (512 columns hold no more beside O).
// O is rescaled only when a row's maximum has grown by more than 2^8 since the last rescale: P then
// stays below 2^8 and the sum is exact in the same frame, so no precision is lost.
#include <cmath>

#include "../../include/sageattn.h"
#include "launch.h"
#include "problem.cuh"
#include "sm103_ptx.cuh"

namespace sage {
namespace {

constexpr int kThreads = 384;
constexpr uint32_t kRegsSoft = 224, kRegsCtl = 56;  // 2 * 128 * 224 + 128 * 56 = 384 * 168
constexpr float kL2e = 1.4426950408889634f, kL2 = 0.6931471805599453f;
constexpr float kNegInf = -INFINITY;
constexpr int kMaxSplits = 16;

struct DocTile {
  int lo, hi;  // smallest and largest non-negative id; lo > hi: none
  int mixed;   // more than one id, or padding
  int pad;     // some padding
};

struct ScoredArgs {
  int batch, hq, hkv, nq, nk, d, dtype, causal, splits, k_tiles, q_offset, vec;
  float c2;           // sm_scale log2(e)
  float cap2, cap_k, cap_x;  // cap log2(e); 2 sm_scale log2(e) / cap; sm_scale / cap
  void* o; int64_t o_sb, o_sh, o_sn;
  float* lse;
  const float* slopes;
  const int* prefix;
  const int* doc_q;
  const int* doc_k;
  // workspace
  int* err;
  DocTile* doc_tiles;  // [batch][k_tiles]
  float* part_o;       // [splits][batch * hq * nq][dp]
  float* part_ml;      // [splits][batch * hq * nq][2]
};

template <int DP>
struct Cfg {
  static constexpr int kChunks = DP / 64;
  static constexpr int kQBytes = 128 * DP * 2, kKBytes = 128 * DP * 2, kVBytes = 128 * DP * 2;
  static constexpr int kKStages = DP == 128 ? 3 : 4, kVStages = DP == 128 ? 2 : 4;
  // tensor memory: S of tile x at 128 x; P over S (head_dim 128) or beside it; then O
  static constexpr bool kOver = DP == 128;
  static constexpr uint32_t kTmemP = kOver ? 0 : 256, kPitchP = kOver ? 128 : 64;
  static constexpr uint32_t kTmemO = kOver ? 256 : 384;
  static constexpr int kOffK = 2 * kQBytes, kOffV = kOffK + kKStages * kKBytes;
  static constexpr int kOffBar = kOffV + kVStages * kVBytes;
  static constexpr int kNumBars = 1 + 2 * kKStages + 3 * kVStages + 12;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kSmem = kOffMisc + 64 + 1024;
  static_assert(kTmemO + 2 * DP <= 512 && kSmem <= 232448, "tensor and shared memory");
};

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcpf(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// 32 columns of tensor memory and their largest value (both valid after a tcgen05.wait::ld).
__device__ __forceinline__ void ld32_max(uint32_t taddr, uint32_t (&r)[32], float& m) {
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, %32, [%33];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=f"(m)
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void wait_ld_max(float (&m)[4]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : "+f"(m[0]), "+f"(m[1]), "+f"(m[2]), "+f"(m[3]) : : "memory");
}

// O of a row times alpha, in tensor memory.
template <int DP>
__device__ __forceinline__ void rescale_o(uint32_t tO, float alpha) {
#pragma unroll 1
  for (int c = 0; c < DP / 32; ++c) {
    uint32_t o[32];
    tmem_ld32(tO + c * 32, o);
    tmem_wait_ld(o);
#pragma unroll
    for (int u = 0; u < 32; u += 2) {
      float f0, f1;
      mul2(f0, f1, __uint_as_float(o[u]), __uint_as_float(o[u + 1]), alpha, alpha);
      o[u] = __float_as_uint(f0);
      o[u + 1] = __float_as_uint(f1);
    }
    tmem_st32(tO + c * 32, o);
  }
}

// What every role of a CTA has to agree on.
struct Work {
  int b, h, split;
  int q0;            // first query row of tile A
  bool has_b;
  int j0, j1;        // key tiles
  int j1a;           // tile A's end (one less where the last tile is behind all of its rows)
};

// CAP / BIAS: the score modification that is compiled in; the masks are a matter of each tile.
template <int DP, bool BF16, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kThreads, 1)
    scored_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const ScoredArgs a) {
  using C = Cfg<DP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sK = sm + C::kOffK;
  uint8_t* sV = sm + C::kOffV;
  uint64_t* q_full = reinterpret_cast<uint64_t*>(sm + C::kOffBar);
  uint64_t* k_full = q_full + 1;
  uint64_t* k_empty = k_full + C::kKStages;
  uint64_t* v_full = k_empty + C::kKStages;
  uint64_t* v_empty = v_full + C::kVStages;
  uint64_t* v_clean = v_empty + C::kVStages;
  uint64_t* s_full = v_clean + C::kVStages;  // [2] scores of a tile are in tensor memory
  uint64_t* s_free = s_full + 2;             // [2] and in registers (P beside S)
  uint64_t* p_half = s_free + 2;             // [2] P of the first 64 keys is written (P over S)
  uint64_t* p_full = p_half + 2;             // [2] all of P is
  uint64_t* o_full = p_full + 2;             // [2] P V is done
  uint64_t* drain = o_full + 2;              // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + C::kOffMisc + 4);
  int* s_red = reinterpret_cast<int*>(sm + C::kOffMisc + 16);  // [4] document and tile ranges

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Work w;
  w.h = blockIdx.x;
  w.b = blockIdx.z / a.splits;
  w.split = blockIdx.z - w.b * a.splits;
  // the pairs with the most keys first when causal
  const int pair = a.causal ? (int)(gridDim.y - 1 - blockIdx.y) : (int)blockIdx.y;
  w.q0 = pair * 256;
  w.has_b = a.nq - w.q0 > 128;
  const int hk = w.h / (a.hq / a.hkv);
  const int rows = min(256, a.nq - w.q0);

  if (threadIdx.x == 0) {
    const int nx = w.has_b ? 2 : 1;
    mbar_init(q_full, 1);
    for (int i = 0; i < C::kKStages; ++i) { mbar_init(&k_full[i], 1); mbar_init(&k_empty[i], nx); }
    for (int i = 0; i < C::kVStages; ++i) {
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], nx);
      mbar_init(&v_clean[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 128);
      mbar_init(&p_half[i], 128);
      mbar_init(&p_full[i], 128);
      mbar_init(&o_full[i], 1);
      mbar_init(&drain[i], 1);
    }
    *abort_flag = 0;
    s_red[0] = INT32_MAX;  // smallest id of the rows
    s_red[1] = -1;         // largest
    s_red[2] = INT32_MAX;  // first tile with such ids
    s_red[3] = -1;         // last
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();

  // ---- the key tiles of this CTA
  const int prefix = a.prefix ? __ldg(&a.prefix[w.b]) : 0;
  // keys that rows [.., row] may see at most
  auto limit_of = [&](int row) -> int {
    if (!a.causal) return a.nk;
    long long n = (long long)row + a.q_offset + 1;
    n = n > prefix ? n : prefix;
    return (int)(n < 0 ? 0 : n < a.nk ? n : a.nk);
  };
  int lo = 0, hi = (limit_of(w.q0 + rows - 1) + 127) / 128;
  int hi_a = (limit_of(w.q0 + min(rows, 128) - 1) + 127) / 128;
  int my_doc = 0;
  if (a.doc_q) {
    my_doc = -1;
    if (threadIdx.x < rows) {
      my_doc = __ldg(&a.doc_q[(int64_t)w.b * a.nq + w.q0 + threadIdx.x]);
      if (my_doc >= 0) { atomicMin(&s_red[0], my_doc); atomicMax(&s_red[1], my_doc); }
    }
    __syncthreads();
    const int dlo = s_red[0], dhi = s_red[1];
    for (int j = threadIdx.x; j < hi; j += kThreads) {
      const DocTile t = a.doc_tiles[(int64_t)w.b * a.k_tiles + j];
      if (t.lo <= t.hi && t.hi >= dlo && t.lo <= dhi) { atomicMin(&s_red[2], j); atomicMax(&s_red[3], j); }
    }
    __syncthreads();
    lo = min(s_red[2], hi);
    hi = min(hi, s_red[3] + 1);
  }
  if (hi < lo) hi = lo;
  if (a.splits > 1) {
    const int n = hi - lo;
    const int x0 = lo + (int)((long long)n * w.split / a.splits), x1 = lo + (int)((long long)n * (w.split + 1) / a.splits);
    lo = x0;
    hi = x1;
  }
  w.j0 = lo;
  w.j1 = hi;
  w.j1a = w.has_b ? max(lo, min(hi, max(hi_a, hi - 1))) : hi;
  const int n_tiles = w.j1 - w.j0;
  const int n_a = w.j1a - w.j0;  // tile A may leave out the last key tile

  if (warp >= 8) {
    regs_dec<kRegsCtl>();
    if (warp == 8) {
      // ========================================================= TMA producer
      if (lane == 0 && n_tiles > 0) {
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
        mbar_arrive_expect_tx(q_full, (w.has_b ? 2 : 1) * C::kQBytes);
        for (int t = 0; t < (w.has_b ? 2 : 1); ++t)
          for (int c = 0; c < C::kChunks; ++c)
            tma_load_4d(sm + t * C::kQBytes + c * 16384, &tmQ, q_full, c * 64, w.q0 + t * 128, w.h, w.b);
        int nk = 0, nv = 0;
        bool ok = true;
        for (int j = 0; j < n_tiles; ++j) {
          const int sk = j % C::kKStages, sv = j % C::kVStages, row = (w.j0 + j) * 128;
          if (j >= C::kKStages) ok = mbar_wait(&k_empty[sk], ((j / C::kKStages) - 1) & 1, abort_flag);
          if (!ok) break;
          mbar_arrive_expect_tx(&k_full[sk], C::kKBytes);
          for (int c = 0; c < C::kChunks; ++c)
            tma_load_4d(sK + sk * C::kKBytes + c * 16384, &tmK, &k_full[sk], c * 64, row, hk, w.b);
          ++nk;
          if (j >= C::kVStages) ok = mbar_wait(&v_empty[sv], ((j / C::kVStages) - 1) & 1, abort_flag);
          if (!ok) break;
          mbar_arrive_expect_tx(&v_full[sv], C::kVBytes);
          for (int c = 0; c < C::kChunks; ++c)
            tma_load_4d(sV + sv * C::kVBytes + c * 16384, &tmV, &v_full[sv], c * 64, row, hk, w.b);
          ++nv;
        }
        if (!ok) {
          // copies in flight land before the shared memory goes away
          volatile int never = 0;
          mbar_wait(q_full, 0, &never);
          for (int j = max(0, nk - C::kKStages); j < nk; ++j)
            mbar_wait(&k_full[j % C::kKStages], (j / C::kKStages) & 1, &never);
          for (int j = max(0, nv - C::kVStages); j < nv; ++j)
            mbar_wait(&v_full[j % C::kVStages], (j / C::kVStages) & 1, &never);
          record_error(a.err, kDevTimeout);
        }
      }
    } else if (warp == 11) {
      // ================================== padding: its V rows become zero (they may hold anything)
      if (a.doc_k) {
        bool ok = true;
        for (int j = 0; j < n_tiles && ok; ++j) {
          const int sv = j % C::kVStages;
          ok = __all_sync(0xffffffffu, mbar_wait(&v_full[sv], (j / C::kVStages) & 1, abort_flag));
          if (!ok) break;
          const DocTile t = a.doc_tiles[(int64_t)w.b * a.k_tiles + w.j0 + j];
          if (t.pad) {
            for (int i = 0; i < 4; ++i) {
              const int row = i * 32 + lane, key = (w.j0 + j) * 128 + row;
              if (key < a.nk && __ldg(&a.doc_k[(int64_t)w.b * a.nk + key]) < 0)
                for (int c = 0; c < C::kChunks; ++c)
                  for (int u = 0; u < 8; ++u)
                    *reinterpret_cast<uint4*>(sV + sv * C::kVBytes + c * 16384 + row * 128 + u * 16) =
                        make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&v_clean[sv]);
        }
        if (!ok && lane == 0) record_error(a.err, kDevTimeout);
      }
    } else if (n_tiles > 0 && (warp == 9 || (!C::kOver && w.has_b))) {
      // ========================================================= MMA issuers
      const int me = warp - 9;
      const uint64_t dq = sdesc_sw128(smem_u32(sm)), dk = sdesc_sw128(smem_u32(sK));
      const uint64_t dv = sdesc_sw128_mn(smem_u32(sV), 16384);
      const uint32_t fmt = BF16 ? 1 : 0;
      const uint32_t id_qk = make_idesc(1, fmt, fmt, 128, 128), id_pv = make_idesc(1, fmt, fmt, 128, DP) | kIdescTransB;
      uint64_t* const v_in = a.doc_k ? v_clean : v_full;
      auto wait_all = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag));
      };
      // scores of query tile x against key tile j
      auto issue_qk = [&](int x, int j) {
        const int st = j % C::kKStages;
        if (!wait_all(&k_full[st], (j / C::kKStages) & 1)) return false;
        tc_fence_after();
        const uint64_t qx = dq + static_cast<uint64_t>((x * C::kQBytes) >> 4);
        const uint64_t kx = dk + static_cast<uint64_t>((st * C::kKBytes) >> 4);
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
          const uint32_t off = ((k >> 2) * 16384 + (k & 3) * 32) >> 4;
          mma_f16_ss_warp(tmem + x * 128, qx + off, kx + off, id_qk, k > 0);
        }
        mma_commit_warp(&s_full[x]);
        mma_commit_warp(&k_empty[st]);
        return true;
      };
      // O of query tile x += P V of key tile j
      auto issue_pv = [&](int x, int j) {
        const int sv = j % C::kVStages;
        if (!wait_all(&v_in[sv], (j / C::kVStages) & 1)) return false;
        if (C::kOver && !wait_all(&p_half[x], j & 1)) return false;
        if (!C::kOver && !wait_all(&p_full[x], j & 1)) return false;
        tc_fence_after();
        const uint32_t d_o = tmem + C::kTmemO + x * DP, a_p = tmem + C::kTmemP + x * C::kPitchP;
        const uint64_t vx = dv + static_cast<uint64_t>((sv * C::kVBytes) >> 4);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (C::kOver && k == 4) {
            if (!wait_all(&p_full[x], j & 1)) return false;
            tc_fence_after();
          }
          mma_f16_ts_warp(d_o, a_p + k * 8, vx + ((k * 2048) >> 4), id_pv, (j > 0 || k > 0) ? 1u : 0u);
        }
        mma_commit_warp(&o_full[x]);
        mma_commit_warp(&v_empty[sv]);
        return true;
      };
      bool ok = wait_all(q_full, 0);
      if constexpr (C::kOver) {
        // One issuer, the tiles in turn, P V and the next scores of one tile together: the tiles then stay half a
        // period apart, one in its softmax while the other has the tensor core. (An issuer per tile
        // lets them fall into step, both in the softmax and then both waiting: 1.5 times slower.)
        const int nx = w.has_b ? 2 : 1;
        for (int x = 0; x < nx && ok; ++x)
          if (x == 1 || n_a > 0) ok = issue_qk(x, 0);
        for (int j = 0; j < n_tiles && ok; ++j)
          for (int x = 0; x < nx && ok; ++x) {
            const int n = x == 0 ? n_a : n_tiles;
            if (j >= n) continue;
            ok = issue_pv(x, j);
            if (ok && j + 1 < n) ok = issue_qk(x, j + 1);
          }
      } else {
        // An issuer per tile: the next scores as soon as the softmax holds the last ones, then P V.
        const int n = me == 0 ? n_a : n_tiles;
        if (ok && n > 0) ok = issue_qk(me, 0);
        for (int j = 0; j < n && ok; ++j) {
          if (j + 1 < n) {
            ok = wait_all(&s_free[me], j & 1) && issue_qk(me, j + 1);
            if (!ok) break;
          }
          ok = issue_pv(me, j);
        }
      }
      // every MMA has finished before tensor memory is released
      mma_commit_warp(&drain[me]);
      volatile int never = 0;
      mbar_wait(&drain[me], 0, &never);
      __syncwarp();
      if (!ok && lane == 0) record_error(a.err, kDevTimeout);
    }
  } else {
    regs_inc<kRegsSoft>();
    // =========================================================== softmax of tile x
    const int x = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int row = w.q0 + x * 128 + r;
    const bool active = x == 0 || w.has_b, valid = active && row < a.nq;
    const uint32_t tS = tmem + lane_base + x * 128, tP = tmem + lane_base + C::kTmemP + x * C::kPitchP;
    const uint32_t tO = tmem + lane_base + C::kTmemO + x * DP;
    const int my_tiles = x == 0 ? n_a : n_tiles;
    const int limit = valid ? limit_of(row) : 0;
    const int dq = a.doc_q ? my_doc : 0;
    const int pos = row + a.q_offset;
    float slope = 0.f;
    if constexpr (BIAS) slope = __ldg(&a.slopes[w.h]) * kL2e;
    // cap tanh(s / cap) = cap - 2 cap / (1 + e^(2 s / cap)): the quotient of two scores
    const float cap_m2 = -2.0f * a.cap2;
    auto cap_rcp = [&](float& t0, float& t1) {
      mul2(t0, t1, t0, t1, a.cap_k, a.cap_k);
      t0 = ex2f(t0);
      t1 = ex2f(t1);
      add2(t0, t1, t0, t1, 1.0f, 1.0f);
      t0 = rcpf(t0);
      t1 = rcpf(t1);
    };
    const float cap_c[7] = {a.cap2 * 0.9999999403953552f,   a.cap2 * -0.33332881331443787f, a.cap2 * 0.13325709104537964f,
                            a.cap2 * -0.05347844585776329f, a.cap2 * 0.020331112667918205f, a.cap2 * -0.006239818874746561f,
                            a.cap2 * 0.0010531365405768156f};
    // the same for |s| <= cap, less the frame: x = s / cap times a polynomial of x^2 (the minimax
    // one of tanh(x) / x on [0, 1], found by exchange; the largest error of tanh is 1.1e-7 in fp32)
    auto cap_poly = [&](float& t0, float& t1, float off) {
      mul2(t0, t1, t0, t1, a.cap_x, a.cap_x);
      float z0, z1, y0, y1;
      mul2(z0, z1, t0, t1, t0, t1);
      fma2(y0, y1, z0, z1, cap_c[6], cap_c[6], cap_c[5], cap_c[5]);
#pragma unroll
      for (int i = 4; i >= 0; --i) fma2(y0, y1, y0, y1, z0, z1, cap_c[i], cap_c[i]);
      fma2(t0, t1, t0, t1, y0, y1, off, off);
    };
    float m = kNegInf;  // the frame's maximum, base 2
    float l = 0.f;
    bool ok = true;
    if (active) {
      for (int j = 0; j < my_tiles; ++j) {
        ok = __all_sync(0xffffffffu, mbar_wait(&s_full[x], j & 1, abort_flag));
        if (!ok) break;
        tc_fence_after();
        const int kv0 = (w.j0 + j) * 128;
        // ---- which keys of the tile this row sees, as bits (only where some row of the warp misses one)
        bool whole = limit - kv0 >= 128;
        if (a.doc_k) {
          const DocTile t = a.doc_tiles[(int64_t)w.b * a.k_tiles + w.j0 + j];
          whole = whole && !t.mixed && t.lo == dq;
        }
        whole = whole || !valid;  // (rows behind the last one are not written)
        const bool masked = !__all_sync(0xffffffffu, whole);
        uint32_t s[4][32];
        float t_max = kNegInf, alpha = 1.0f, m_use = 0.f;
        float g0 = 0.f, g1 = 0.f, g2 = 0.f, g3 = 0.f;
        // S is in registers
        auto release_s = [&]() {
          if constexpr (!C::kOver) {
            tc_fence_before();
            mbar_arrive(&s_free[x]);
          }
        };
        // The frame is kept unless the maximum grew by more than 8. P V of the last tile is waited for here:
        // O may then be rescaled and P overwritten (it also keeps p_full at most one phase ahead of its issuer).
        auto reframe = [&]() {
          const bool grow = t_max > m + 8.0f || (m == kNegInf && t_max > kNegInf);
          const float m_new = grow ? t_max : m;
          m_use = m_new == kNegInf ? 0.f : m_new;
          alpha = grow ? ex2f(m - m_use) : 1.0f;
          m = m_new;
          if (j > 0) {
            ok = __all_sync(0xffffffffu, mbar_wait(&o_full[x], (j - 1) & 1, abort_flag));
            if (!ok) return;
            tc_fence_after();
            if (__any_sync(0xffffffffu, alpha != 1.0f)) rescale_o<DP>(tO, alpha);
          }
        };
        // P = 2^(t - m), summed in 32 bits, rounded once to the operands' type. FORM: 0 s holds the
        // scores t; 1 the products; 2, 3 the products to be capped, by quotient or by polynomial
        auto weights = [&](auto form) {
          constexpr int FORM = decltype(form)::value;
          const float c_off = FORM == 2 ? a.cap2 - m_use : -m_use;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t pw[16];
#pragma unroll
            for (int u = 0; u < 32; u += 4) {
              float e[4];
#pragma unroll
              for (int v = 0; v < 4; v += 2) {
                float t0 = __uint_as_float(s[c][u + v]), t1 = __uint_as_float(s[c][u + v + 1]);
                if constexpr (FORM == 0) add2(t0, t1, t0, t1, c_off, c_off);
                if constexpr (FORM == 1) fma2(t0, t1, t0, t1, a.c2, a.c2, c_off, c_off);
                if constexpr (FORM == 2) {
                  cap_rcp(t0, t1);
                  fma2(t0, t1, t0, t1, cap_m2, cap_m2, c_off, c_off);
                }
                if constexpr (FORM == 3) cap_poly(t0, t1, c_off);
                e[v] = ex2f(t0);
                e[v + 1] = ex2f(t1);
              }
              add2(g0, g1, g0, g1, e[0], e[1]);
              add2(g2, g3, g2, g3, e[2], e[3]);
              pw[u / 2] = pack16<BF16>(e[0], e[1]);
              pw[u / 2 + 1] = pack16<BF16>(e[2], e[3]);
            }
#pragma unroll
            for (int u = 0; u < 16; ++u) s[c >> 1][(c & 1) * 16 + u] = pw[u];
            if (c & 1) {
              tmem_st32(tP + (c >> 1) * 32, s[c >> 1]);
              if (C::kOver && c == 1) {
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&p_half[x]);
              }
            }
          }
        };
        if (!BIAS && !masked) {
          // products; the cap and the scale keep their order, so their largest gives the maximum
          float cm[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) ld32_max(tS + c * 32, s[c], cm[c]);
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_wait_ld(s[c]);
          wait_ld_max(cm);
          release_s();
          const float top = fmaxf(max3(cm[0], cm[1], cm[2]), cm[3]);
          if constexpr (CAP) {
            float big = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int u = 0; u < 32; u += 2)
                big = max3(big, fabsf(__uint_as_float(s[c][u])), fabsf(__uint_as_float(s[c][u + 1])));
            t_max = fmaf(rcpf(1.0f + ex2f(top * a.cap_k)), cap_m2, a.cap2);
            reframe();
            if (!ok) break;
            if (__all_sync(0xffffffffu, big * a.cap_x <= 1.0f)) weights(std::integral_constant<int, 3>{});
            else weights(std::integral_constant<int, 2>{});
          } else {
            t_max = top * a.c2;
            reframe();
            if (!ok) break;
            weights(std::integral_constant<int, 1>{});
          }
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, s[c]);
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_wait_ld(s[c]);
          release_s();
          // scores in base 2: capped or scaled, then biased
          auto scores = [&](auto bias_at) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int u = 0; u < 32; u += 2) {
                float t0 = __uint_as_float(s[c][u]), t1 = __uint_as_float(s[c][u + 1]);
                if constexpr (CAP) {
                  cap_rcp(t0, t1);
                  if constexpr (BIAS) fma2(t0, t1, t0, t1, cap_m2, cap_m2, bias_at(c * 32 + u), bias_at(c * 32 + u + 1));
                  else fma2(t0, t1, t0, t1, cap_m2, cap_m2, a.cap2, a.cap2);
                } else if constexpr (BIAS) {
                  fma2(t0, t1, t0, t1, a.c2, a.c2, bias_at(c * 32 + u), bias_at(c * 32 + u + 1));
                } else {
                  mul2(t0, t1, t0, t1, a.c2, a.c2);
                }
                s[c][u] = __float_as_uint(t0);
                s[c][u + 1] = __float_as_uint(t1);
              }
          };
          if constexpr (BIAS) {
            // The bias is linear along a tile that lies on one side of every row's position (or
            // whose other side the causal mask hides)
            const float dist = static_cast<float>(pos - kv0);  // exact below 2^24
            const float add = CAP ? a.cap2 : 0.f;
            const bool all_left = __all_sync(0xffffffffu, kv0 + 127 <= pos || (a.causal && prefix <= 0));
            const bool all_right = __all_sync(0xffffffffu, kv0 >= pos);
            if (all_left || all_right) {
              const float step = all_left ? slope : -slope, base = fmaf(-step, dist, add);
              scores([&](int u) { return fmaf(step, static_cast<float>(u), base); });
            } else {
              scores([&](int u) { return fmaf(-slope, fabsf(dist - static_cast<float>(u)), add); });
            }
          } else {
            scores([](int) { return 0.f; });
          }
          if (masked) {
            uint32_t bits[4];
            const int n = limit - kv0;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int k = n - c * 32;
              bits[c] = k >= 32 ? 0xffffffffu : k <= 0 ? 0u : (1u << k) - 1u;
            }
            if (a.doc_k) {
              int id[4];
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const int key = kv0 + c * 32 + lane;
                id[c] = key < a.nk ? __ldg(&a.doc_k[(int64_t)w.b * a.nk + key]) : -1;
              }
              // each document among the warp's rows in turn: its keys by ballot
              uint32_t todo = __ballot_sync(0xffffffffu, dq >= 0);
              uint32_t mine[4] = {0, 0, 0, 0};
              while (todo) {
                const int one = __shfl_sync(0xffffffffu, dq, __ffs(todo) - 1);
                const bool me = dq == one;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                  const uint32_t v = __ballot_sync(0xffffffffu, id[c] == one);
                  if (me) mine[c] = v;
                }
                todo &= ~__ballot_sync(0xffffffffu, me);
              }
#pragma unroll
              for (int c = 0; c < 4; ++c) bits[c] &= mine[c];
            }
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int u = 0; u < 32; ++u)
                if (!(bits[c] >> u & 1u)) s[c][u] = __float_as_uint(kNegInf);
          }
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int u = 0; u < 32; u += 2)
              t_max = max3(t_max, __uint_as_float(s[c][u]), __uint_as_float(s[c][u + 1]));
          reframe();
          if (!ok) break;
          weights(std::integral_constant<int, 0>{});
        }
        l = fmaf(l, alpha, (g0 + g1) + (g2 + g3));
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&p_full[x]);
      }
      // ---- out = O / l and the log-sum-exp; a split writes O and its frame to the workspace
      if (ok && my_tiles > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(&o_full[x], (my_tiles - 1) & 1, abort_flag));
        tc_fence_after();
      }
      if (ok) {
        const int64_t line = ((int64_t)w.b * a.hq + w.h) * a.nq + row;
        const bool seen = my_tiles > 0 && l != 0.f;
        const float inv = seen ? 1.0f / l : 0.f;
        uint16_t* const dst = static_cast<uint16_t*>(a.o) + w.b * a.o_sb + w.h * a.o_sh + row * a.o_sn;
        float* const part = a.part_o + ((int64_t)w.split * a.batch * a.hq * a.nq + line) * DP;
#pragma unroll 1
        for (int c = 0; c < DP / 32 && c * 32 < a.d; ++c) {
          uint32_t o[32];
          if (my_tiles > 0) {
            tmem_ld32(tO + c * 32, o);
            tmem_wait_ld(o);
          }
          if (!seen)
#pragma unroll
            for (int u = 0; u < 32; ++u) o[u] = 0u;
          if (valid && a.splits > 1) {
#pragma unroll
            for (int u = 0; u < 32; u += 4)
              *reinterpret_cast<uint4*>(part + c * 32 + u) = make_uint4(o[u], o[u + 1], o[u + 2], o[u + 3]);
          } else if (valid && a.vec) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (c * 32 + q * 8 < a.d) {
                uint4 v;
                const float* f = reinterpret_cast<const float*>(o) + q * 8;
                v.x = pack16<BF16>(f[0] * inv, f[1] * inv);
                v.y = pack16<BF16>(f[2] * inv, f[3] * inv);
                v.z = pack16<BF16>(f[4] * inv, f[5] * inv);
                v.w = pack16<BF16>(f[6] * inv, f[7] * inv);
                *reinterpret_cast<uint4*>(dst + c * 32 + q * 8) = v;
              }
          } else if (valid) {
#pragma unroll
            for (int u = 0; u < 32; ++u)
              if (c * 32 + u < a.d)
                dst[c * 32 + u] = static_cast<uint16_t>(pack16<BF16>(__uint_as_float(o[u]) * inv, 0.f) & 0xffffu);
          }
        }
        if (valid) {
          if (a.splits > 1)
            *reinterpret_cast<float2*>(a.part_ml + ((int64_t)w.split * a.batch * a.hq * a.nq + line) * 2) =
                make_float2(seen ? m : kNegInf, seen ? l : 0.f);
          else if (a.lse)
            a.lse[line] = seen ? (m + __log2f(l)) * kL2 : kNegInf;
        }
      }
      if (!ok) record_error(a.err, kDevTimeout);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Clears the status word; with documents, the ids that each tile of 128 keys holds.
__global__ void __launch_bounds__(128) scored_setup_kernel(const ScoredArgs a) {
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *a.err = 0;
  if (!a.doc_k) return;
  __shared__ int s_lo, s_hi, s_pad;
  if (threadIdx.x == 0) { s_lo = INT32_MAX; s_hi = -1; s_pad = 0; }
  __syncthreads();
  const int key = blockIdx.x * 128 + threadIdx.x;
  if (key < a.nk) {
    const int id = __ldg(&a.doc_k[(int64_t)blockIdx.y * a.nk + key]);
    if (id >= 0) { atomicMin(&s_lo, id); atomicMax(&s_hi, id); }
    else s_pad = 1;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    DocTile t;
    t.lo = s_lo; t.hi = s_hi; t.pad = s_pad;
    t.mixed = s_pad || s_lo != s_hi;
    a.doc_tiles[(int64_t)blockIdx.y * a.k_tiles + blockIdx.x] = t;
  }
}

// Splits joined: one warp per row.
template <bool BF16, int DP>
__global__ void __launch_bounds__(128) scored_join_kernel(const ScoredArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t lines = (int64_t)a.batch * a.hq * a.nq, line = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  pdl_wait();
  if (line >= lines) return;
  float m = kNegInf;
  for (int s = 0; s < a.splits; ++s) m = fmaxf(m, a.part_ml[(s * lines + line) * 2]);
  const float u = m == kNegInf ? 0.f : m;
  float l = 0.f, acc[DP / 32];
#pragma unroll
  for (int c = 0; c < DP / 32; ++c) acc[c] = 0.f;
  for (int s = 0; s < a.splits; ++s) {
    const float2 x = *reinterpret_cast<const float2*>(a.part_ml + (s * lines + line) * 2);
    const float f = ex2f(x.x - u);
    l = fmaf(x.y, f, l);
#pragma unroll
    for (int c = 0; c < DP / 32; ++c)
      if (c * 32 < a.d) acc[c] = fmaf(a.part_o[(s * lines + line) * DP + c * 32 + lane], f, acc[c]);
  }
  const float inv = l != 0.f ? 1.0f / l : 0.f;
  const int64_t bh = line / a.nq;
  const int row = (int)(line - bh * a.nq), b = (int)(bh / a.hq), h = (int)(bh - (int64_t)b * a.hq);
  uint16_t* dst = static_cast<uint16_t*>(a.o) + b * a.o_sb + h * a.o_sh + row * a.o_sn;
#pragma unroll
  for (int c = 0; c < DP / 32; ++c)
    if (c * 32 + lane < a.d) dst[c * 32 + lane] = static_cast<uint16_t>(pack16<BF16>(acc[c] * inv, 0.f) & 0xffffu);
  if (a.lse && lane == 0) a.lse[line] = l != 0.f ? (m + __log2f(l)) * kL2 : kNegInf;
}

// No keys at all: 0 and -inf.
__global__ void __launch_bounds__(128) scored_empty_kernel(const ScoredArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t lines = (int64_t)a.batch * a.hq * a.nq, line = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (line == 0 && lane == 0) *a.err = 0;
  if (line >= lines) return;
  const int64_t bh = line / a.nq;
  const int row = (int)(line - bh * a.nq), b = (int)(bh / a.hq), h = (int)(bh - (int64_t)b * a.hq);
  for (int c = lane; c < a.d; c += 32)
    static_cast<uint16_t*>(a.o)[b * a.o_sb + h * a.o_sh + row * a.o_sn + c] = 0;
  if (a.lse && lane == 0) a.lse[line] = kNegInf;
}

// Rows that TMA cannot address (odd head_dim or strides, unaligned or broadcast tensors), copied
// once into rows of dp channels: [batch][heads][n][dp], zeros behind d.
struct CopyArgs {
  const uint16_t* src; int64_t sb, sh, sn;
  uint16_t* dst;
  int heads, n, d, dp;
  int64_t lines;
};
__global__ void __launch_bounds__(128) scored_copy_kernel(const CopyArgs a) {
  const int lane = threadIdx.x & 31;
  for (int64_t line = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5); line < a.lines; line += (int64_t)gridDim.x * 4) {
    const int64_t bh = line / a.n;
    const int row = (int)(line - bh * a.n), b = (int)(bh / a.heads), h = (int)(bh - (int64_t)b * a.heads);
    const uint16_t* src = a.src + b * a.sb + h * a.sh + row * a.sn;
    for (int c = lane; c < a.dp; c += 32) a.dst[line * a.dp + c] = c < a.d ? src[c] : (uint16_t)0;
  }
}

// ------------------------------------------------------------------------------------- host
size_t up256(size_t x) { return (x + 255) / 256 * 256; }
struct ScoredLayout {
  size_t tiles, part_o, part_ml, copy[3], total;
  int dp, splits, k_tiles;
};
// Key splits: where the (head, pair of query tiles) items leave SMs idle, as many as fill one wave, of at
// least four key tiles each.
int splits_of(int batch, int hq, int nq, int nk) {
  const int64_t items = (int64_t)batch * hq * ((nq + 255) / 256), tiles = (nk + 127) / 128;
  int64_t s = items > 0 ? 152 / items : 1;
  if (s > tiles / 4) s = tiles / 4;
  if (s > kMaxSplits) s = kMaxSplits;
  return s < 1 ? 1 : (int)s;
}
bool scored_layout(int batch, int hq, int hkv, int nq, int nk, int d, int packed, ScoredLayout* L) {
  if (batch < 0 || hq < 1 || hkv < 1 || hq % hkv || nq < 0 || nk < 0 || d < 1 || d > 128) return false;
  L->dp = d <= 64 ? 64 : 128;
  L->splits = splits_of(batch, hq, nq, nk);
  L->k_tiles = (int)(((int64_t)nk + 127) / 128);
  size_t o = 256;
  auto take = [&](size_t bytes) { const size_t at = o; o += up256(bytes); return at; };
  L->tiles = take((size_t)batch * L->k_tiles * sizeof(DocTile));
  const size_t lines = (size_t)batch * hq * nq;
  L->part_o = take(L->splits > 1 ? L->splits * lines * L->dp * 4 : 0);
  L->part_ml = take(L->splits > 1 ? L->splits * lines * 8 : 0);
  for (int i = 0; i < 3; ++i) {
    const size_t rows = (size_t)batch * (i == 0 ? hq : hkv) * (i == 0 ? nq : nk);
    L->copy[i] = take(packed ? 0 : rows * L->dp * 2);
  }
  L->total = o;
  return true;
}

template <int DP, bool BF16, bool CAP, bool BIAS>
cudaError_t launch_scored_t(const ScoredArgs& a, const CUtensorMap* maps, dim3 grid, cudaStream_t st) {
  static std::atomic<int> limits[64];
  cudaError_t e = raise_smem_limit(scored_kernel<DP, BF16, CAP, BIAS>, Cfg<DP>::kSmem, limits);
  if (e != cudaSuccess) return e;
  return launch_pdl(scored_kernel<DP, BF16, CAP, BIAS>, grid, dim3(kThreads), Cfg<DP>::kSmem, st, maps[0], maps[1],
                    maps[2], a);
}
template <int DP, bool BF16>
cudaError_t launch_scored(const ScoredArgs& a, const CUtensorMap* maps, dim3 grid, cudaStream_t st) {
  const bool cap = a.cap2 > 0.f, bias = a.slopes != nullptr;
  cudaError_t e = cap ? (bias ? launch_scored_t<DP, BF16, true, true>(a, maps, grid, st)
                              : launch_scored_t<DP, BF16, true, false>(a, maps, grid, st))
                      : (bias ? launch_scored_t<DP, BF16, false, true>(a, maps, grid, st)
                              : launch_scored_t<DP, BF16, false, false>(a, maps, grid, st));
  if (e != cudaSuccess || a.splits == 1) return e;
  const int64_t blocks = ((int64_t)a.batch * a.hq * a.nq + 3) / 4;
  return launch_pdl(scored_join_kernel<BF16, DP>, dim3((unsigned)blocks), dim3(128), 0, st, a);
}

struct View {
  const void* p;
  int64_t sb, sh, sn;
  int heads, n;
};

}  // namespace
}  // namespace sage

using namespace sage;

extern "C" {

size_t sage_scored_attn_workspace_size(int batch, int heads_q, int heads_kv, int seqlen_q, int seqlen_k, int head_dim,
                                       int packed) {
  ScoredLayout L;
  return scored_layout(batch, heads_q, heads_kv, seqlen_q, seqlen_k, head_dim, packed, &L) ? L.total : 0;
}

int sage_scored_attn(const sage_tensor* q, const sage_tensor* k, const sage_tensor* v, const sage_tensor* out,
                     float* lse, const float* slopes, const int32_t* prefix_lens, const int32_t* doc_q,
                     const int32_t* doc_k, int batch, int heads_q, int heads_kv, int seqlen_q, int seqlen_k,
                     int head_dim, int dtype, int tensor_layout, int is_causal, float sm_scale, float softcap,
                     int q_offset, int return_lse, void* workspace, size_t workspace_bytes, void* stream) {
  if (!q || !k || !v || !out) return SAGE_ERR_INVALID_ARG;
  if (head_dim < 1 || head_dim > 128) return SAGE_ERR_HEAD_DIM;
  if (dtype != SAGE_F16 && dtype != SAGE_BF16) return SAGE_ERR_DTYPE;
  if (tensor_layout != SAGE_HND && tensor_layout != SAGE_NHD) return SAGE_ERR_INVALID_ARG;
  if (batch < 0 || heads_q < 1 || heads_kv < 1 || seqlen_q < 0 || seqlen_k < 0 || !(softcap >= 0.f) ||
      std::isinf(softcap) || (prefix_lens && !is_causal) || !doc_q != !doc_k || (return_lse && !lse))
    return SAGE_ERR_INVALID_ARG;
  if (heads_q % heads_kv) return SAGE_ERR_GQA;
  for (const void* p : {(const void*)lse, (const void*)slopes, (const void*)prefix_lens, (const void*)doc_q, (const void*)doc_k})
    if (reinterpret_cast<uintptr_t>(p) % 4) return SAGE_ERR_INVALID_ARG;
  if (batch == 0 || seqlen_q == 0) return SAGE_OK;
  const sage_tensor* ts[4] = {q, k, v, out};
  View view[4];
  for (int i = 0; i < 4; ++i) {
    const sage_tensor* t = ts[i];
    const bool keys = i == 1 || i == 2;
    if (!t->data && !(keys && seqlen_k == 0)) return SAGE_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(t->data) % 2) return SAGE_ERR_STRIDE;
    for (int s = 0; s < 3; ++s)
      if (t->stride[s] < 0) return SAGE_ERR_STRIDE;
    const int hi = tensor_layout == SAGE_HND ? 1 : 2, ni = tensor_layout == SAGE_HND ? 2 : 1;
    view[i] = {t->data, t->stride[0], t->stride[hi], t->stride[ni], keys ? heads_kv : heads_q, keys ? seqlen_k : seqlen_q};
  }
  ScoredLayout L;
  // rows that TMA addresses: 16-byte aligned, no zero stride of a dimension that is walked
  bool fits[4];
  for (int i = 0; i < 4; ++i) {
    const View& t = view[i];
    bool ok = head_dim % 8 == 0 && reinterpret_cast<uintptr_t>(t.p) % 16 == 0;
    const int64_t str[3] = {t.sb, t.sh, t.sn}, len[3] = {batch, t.heads, t.n};
    for (int s = 0; s < 3; ++s)
      if (len[s] > 1) ok = ok && str[s] > 0 && str[s] % 8 == 0 && str[s] < (1LL << 38);
    fits[i] = ok;
  }
  const bool packed = fits[0] && fits[1] && fits[2];
  if (!scored_layout(batch, heads_q, heads_kv, seqlen_q, seqlen_k, head_dim, packed, &L)) return SAGE_ERR_INVALID_ARG;
  const int64_t pairs = ((int64_t)seqlen_q + 255) / 256;
  if (seqlen_k > 0x7fffff00 || seqlen_q > 0x7fffff00 || (int64_t)q_offset + seqlen_q > 0x7fffff00 ||
      q_offset < -0x7fffff00 || pairs > 65535 || (int64_t)batch * L.splits > 65535 || (int64_t)batch * heads_q * seqlen_q > (1LL << 32))
    return SAGE_ERR_INVALID_ARG;
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 || workspace_bytes < L.total)
    return SAGE_ERR_WORKSPACE;
  if (!sage_device_supported()) return SAGE_ERR_DEVICE;
  char* w = static_cast<char*>(workspace);
  ScoredArgs a{};
  a.batch = batch; a.hq = heads_q; a.hkv = heads_kv; a.nq = seqlen_q; a.nk = seqlen_k; a.d = head_dim;
  a.dtype = dtype; a.causal = is_causal ? 1 : 0; a.splits = L.splits; a.k_tiles = L.k_tiles; a.q_offset = q_offset;
  a.vec = fits[3] ? 1 : 0;
  const float scale =
      std::isnan(sm_scale) || sm_scale <= 0.f ? (float)(1.0 / std::sqrt((double)head_dim)) : sm_scale;
  a.c2 = (float)(scale * 1.4426950408889634);
  a.cap2 = (float)(softcap * 1.4426950408889634);
  a.cap_x = softcap > 0.f ? scale / softcap : 0.f;
  a.cap_k = softcap > 0.f ? (float)(2.0 * 1.4426950408889634 * scale / softcap) : 0.f;
  a.o = out->data; a.o_sb = view[3].sb; a.o_sh = view[3].sh; a.o_sn = view[3].sn;
  a.lse = return_lse ? lse : nullptr;
  a.slopes = slopes; a.prefix = prefix_lens; a.doc_q = doc_q; a.doc_k = doc_k;
  a.err = reinterpret_cast<int*>(w);
  a.doc_tiles = reinterpret_cast<DocTile*>(w + L.tiles);
  a.part_o = reinterpret_cast<float*>(w + L.part_o);
  a.part_ml = reinterpret_cast<float*>(w + L.part_ml);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (seqlen_k == 0) {
    scored_empty_kernel<<<(unsigned)(((int64_t)batch * heads_q * seqlen_q + 3) / 4), 128, 0, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SAGE_OK : note_cuda_failure(e, "scored attention");
  }
  CUtensorMap maps[3];
  cudaError_t e = cudaSuccess;
  for (int i = 0; i < 3 && e == cudaSuccess; ++i) {
    View& t = view[i];
    int inner = head_dim;
    if (!packed) {
      CopyArgs c{static_cast<const uint16_t*>(t.p), t.sb, t.sh, t.sn, reinterpret_cast<uint16_t*>(w + L.copy[i]),
                 t.heads, t.n, head_dim, L.dp, (int64_t)batch * t.heads * t.n};
      const int64_t blocks = (c.lines + 3) / 4;
      scored_copy_kernel<<<(unsigned)(blocks < 4864 ? blocks : 4864), 128, 0, st>>>(c);
      e = cudaGetLastError();
      t = {c.dst, (int64_t)t.heads * t.n * L.dp, (int64_t)t.n * L.dp, L.dp, t.heads, t.n};
      inner = L.dp;
    }
    // a stride that is never walked (its dimension is 1 long) is given a legal value
    const int64_t sn = t.n > 1 ? t.sn : 128, sh = t.heads > 1 ? t.sh : 128, sb = batch > 1 ? t.sb : 128;
    if (!make_map4(&maps[i], dtype == SAGE_BF16, t.p, inner, t.n, t.heads, batch, sn * 2, sh * 2, sb * 2, 64, 128))
      return note_cuda_failure(cudaErrorInvalidValue, "cuTensorMapEncodeTiled");
  }
  if (e == cudaSuccess) {
    scored_setup_kernel<<<doc_k ? dim3(L.k_tiles, batch) : dim3(1), 128, 0, st>>>(a);
    e = cudaGetLastError();
  }
  const dim3 grid(heads_q, (unsigned)pairs, (unsigned)(batch * L.splits));
  if (e == cudaSuccess) {
    if (dtype == SAGE_BF16)
      e = L.dp == 64 ? launch_scored<64, true>(a, maps, grid, st) : launch_scored<128, true>(a, maps, grid, st);
    else
      e = L.dp == 64 ? launch_scored<64, false>(a, maps, grid, st) : launch_scored<128, false>(a, maps, grid, st);
  }
  return e == cudaSuccess ? SAGE_OK : note_cuda_failure(e, "scored attention");
}

}  // extern "C"
