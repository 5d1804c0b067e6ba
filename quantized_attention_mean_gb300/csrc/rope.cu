// Norms of queries and keys for each head and their rotation by position, in one pass (sage_qk_norm_rope).
//
//   y = x / sqrt(mean_c x_c^2 + eps) * w_c            over the d channels of a (token, head) row
//   (y_i, y_j) -> (y_i cos a - y_j sin a, y_j cos a + y_i sin a),  a = position * inv_freq[p]
//   for the pairs p < rot / 2: (i, j) = (p, p + rot / 2), or (2 p, 2 p + 1) interleaved
//
// Every row is read and written once, so DRAM bounds it. A warp takes some heads of one token: 32 / lanes rows at a
// time, whose lanes hold the same channels of every row, so that weights, cosines and sines stay in registers over the
// heads. A lane owns two runs of V channels that hold whole pairs, so a rotation needs no exchange between lanes and
// the mean of squares one butterfly. The angle is taken in turns modulo one, as a 64-bit fixed-point product of the
// position and inv_freq / 2 pi, which is off by 2^-52 of itself (its constant and its product are rounded) and 2^-65: the angle
// by 2^-52 of itself and 2^-65 of a turn per position, 5e-7 inv_freq + 4e-10 at 2^31. 32-bit floats would lose an angle at position
// 2^20 by 0.06. All arithmetic on values is in 32 bits, rounded once.
//
// 8192 tokens of 32 + 8 heads, head_dim 128, bf16 (168 MB): 31.4 us, 5.35 TB/s, 79% of a copy; 64 tokens: 4.2 us of GPU time.
// 8194 tokens of 16 + 16 heads, head_dim 72, 36 channels in neighbouring pairs (76 MB): 21.9 us, since a row of 72 channels leaves
// two lanes of 32 and a seventh of the others idle and a token's sines and products serve fewer channels.
#include <cmath>

#include "../../include/sageattn.h"
#include "launch.h"
#include "sm103_ptx.cuh"

namespace sage {
namespace {

constexpr int kRopeWarps = 4, kRopeBlocks = 4;  // of an SM
constexpr int kMaxPairs = 64;
// Means of squares that fp32 holds with all their bits: below, the squares of a row lose theirs; above, their sum may overflow.
constexpr float kLeastSquare = 0x1p-90f, kMostSquare = 0x1p120f;

struct RopeArgs {
  const void* x[2];          // q, k
  void* y[2];
  int64_t xs[2][3], ys[2][3];  // element strides of batch, token, head
  const void* w[2];          // or null
  const int* pos; int64_t pos_sb;  // null: the token's place in its row
  const float* freq;
  int heads[2], chunks;      // chunks: warps that share a token's heads
  int batch, n, d, rot;
  int interleaved, w32, lanes;  // lanes of a row: a power of two, or where more rows fit a warp as many as it has slots
  int64_t items;
  float eps, inv_d;
};

template <typename T, int V> struct Run;  // V channels as one access
template <typename T> struct Run<T, 8> { using type = uint4; };
template <typename T> struct Run<T, 4> { using type = uint2; };
template <typename T> struct Run<T, 2> { using type = uint32_t; };
template <typename T> struct Run<T, 1> { using type = uint16_t; };

// A run, where heads are left: one predicated access, no branch. (Volatile: an output may be its input.)
__device__ __forceinline__ void load_if(uint4& r, const void* p, int left) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.gt.s32 p, %5, 0;\n\t@p ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
               : "+r"(r.x), "+r"(r.y), "+r"(r.z), "+r"(r.w) : "l"(p), "r"(left) : "memory");
}
__device__ __forceinline__ void store_if(void* p, const uint4& r, int left) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.gt.s32 p, %5, 0;\n\t@p st.global.v4.u32 [%4], {%0, %1, %2, %3};\n\t}" ::"r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w), "l"(p), "r"(left)
               : "memory");
}
__device__ __forceinline__ void load_if(uint2& r, const void* p, int left) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.gt.s32 p, %3, 0;\n\t@p ld.global.v2.u32 {%0, %1}, [%2];\n\t}"
               : "+r"(r.x), "+r"(r.y) : "l"(p), "r"(left) : "memory");
}
__device__ __forceinline__ void store_if(void* p, const uint2& r, int left) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.gt.s32 p, %3, 0;\n\t@p st.global.v2.u32 [%2], {%0, %1};\n\t}" ::"r"(r.x), "r"(r.y), "l"(p), "r"(left)
               : "memory");
}
__device__ __forceinline__ void load_if(uint32_t& r, const void* p, int left) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.gt.s32 p, %2, 0;\n\t@p ld.global.u32 %0, [%1];\n\t}"
               : "+r"(r) : "l"(p), "r"(left) : "memory");
}
__device__ __forceinline__ void store_if(void* p, const uint32_t& r, int left) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.gt.s32 p, %2, 0;\n\t@p st.global.u32 [%1], %0;\n\t}" ::"r"(r), "l"(p), "r"(left)
               : "memory");
}
__device__ __forceinline__ void load_if(uint16_t& r, const void* p, int left) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.gt.s32 p, %2, 0;\n\t@p ld.global.u16 %0, [%1];\n\t}"
               : "+h"(r) : "l"(p), "r"(left) : "memory");
}
__device__ __forceinline__ void store_if(void* p, const uint16_t& r, int left) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.gt.s32 p, %2, 0;\n\t@p st.global.u16 [%1], %0;\n\t}" ::"h"(r), "l"(p), "r"(left)
               : "memory");
}

// Two fp32 values in a pair of registers.
using Pair = unsigned long long;
__device__ __forceinline__ Pair make_pair2(float lo, float hi) {
  Pair p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(lo), "f"(hi));
  return p;
}
__device__ __forceinline__ void split_pair2(Pair p, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p)); }
__device__ __forceinline__ Pair mul_pair2(Pair x, Pair y) {
  Pair z;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(z) : "l"(x), "l"(y));
  return z;
}
__device__ __forceinline__ Pair fma_pair2(Pair x, Pair y, Pair z) {
  Pair w;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(w) : "l"(x), "l"(y), "l"(z));
  return w;
}

template <typename T>
__device__ __forceinline__ T narrow(float x) {
  if constexpr (std::is_same<T, __half>::value) return __float2half_rn(x);
  else return __float2bfloat16_rn(x);
}

// First channels of the two runs of slot x, and which of the runs lie within the row.
template <int V, bool PAIRS>
__device__ __forceinline__ void slot_runs(const RopeArgs& a, int x, int (&c)[2], bool (&on)[2]) {
  const int half = a.rot / 2, turned = half / V;
  if (PAIRS) {
    c[0] = 2 * x * V;
    c[1] = c[0] + V;
  } else if (x < turned) {
    c[0] = x * V;
    c[1] = half + x * V;
  } else {
    c[0] = a.rot + 2 * (x - turned) * V;
    c[1] = c[0] + V;
  }
  on[0] = c[0] < a.d;
  on[1] = c[1] < a.d;
}

// N floats from shared memory, at a multiple of N floats (N >= 4: of four).
template <int N>
__device__ __forceinline__ void copy_run(float* to, const float* from) {
  if constexpr (N >= 4) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 f = *reinterpret_cast<const float4*>(from + i);
      to[i] = f.x; to[i + 1] = f.y; to[i + 2] = f.z; to[i + 3] = f.w;
    }
  } else if constexpr (N == 2) {
    const float2 f = *reinterpret_cast<const float2*>(from);
    to[0] = f.x; to[1] = f.y;
  } else {
    to[0] = *from;
  }
}

// Two 16-bit values of a register.
template <typename T>
__device__ __forceinline__ void widen2(uint32_t x, float& lo, float& hi) {
  if constexpr (std::is_same<T, __half>::value) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x));
    lo = f.x;
    hi = f.y;
  } else {
    lo = __uint_as_float(x << 16);
    hi = __uint_as_float(x & 0xffff0000u);
  }
}

// SLOTS: pairs of runs per lane. PAIRS: neighbouring channels are turned. A warp takes a share of one token's heads, first
// of q, then of k, `rows` heads at a time. The next kAhead such steps are in flight, the first ones before the position is
// known. With x' = x w a pair becomes f (x'_i cos - x'_j sin, x'_j cos + x'_i sin), f the row's norm: the products of weights
// with cosines and sines are the same for all heads, which leaves six operations for two values.
// LANES: of a row, or 0: a.lanes. ANY: rows whose mean of squares fp32 does not hold are taken by a power of two first; what
// looks for them in the loop costs 2 to 8%, so that only calls that may have some do (bf16 with eps below kLeastSquare).
// At 128 registers the forms of neighbouring pairs on five or six lanes spill one (4 bytes).
template <typename T, int V, int SLOTS, bool PAIRS, int LANES, bool ANY>
__global__ void __launch_bounds__(kRopeWarps * 32, kRopeBlocks) rope_kernel(const RopeArgs a) {
  using R = typename Run<T, V>::type;
  constexpr int kAhead = V == 8 ? 4 : 2, N = SLOTS * V / 2;  // N: pairs of a lane, two by two
  __shared__ unsigned long long s_turns[kMaxPairs];
  __shared__ __align__(16) float2 s_cs[kRopeWarps][128];  // of the channels' pairs, (1, 0) past the turned ones
  __shared__ __align__(16) float s_w[2][128];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int pairs = a.rot / 2;
  pdl_wait();
  pdl_trigger();
  for (int k = threadIdx.x; k < pairs; k += kRopeWarps * 32) {
    // turns per position modulo 1, in units of 2^-64 (one of a negative frequency is not taken from one, which would round it)
    const float freq = __ldg(&a.freq[k]);
    double f = (double)fabsf(freq) * 0.15915494309189533577;
    f -= floor(f);
    const unsigned long long turns = __double2ull_rn(f * 18446744073709551616.0);
    s_turns[k] = freq < 0.f ? 0ull - turns : turns;
  }
  for (int k = threadIdx.x; k < 256; k += kRopeWarps * 32) {
    const int i = k >> 7, c = k & 127;
    const void* w = a.w[i];
    s_w[i][c] = c >= a.d ? 0.f : !w ? 1.f : a.w32 ? __ldg(static_cast<const float*>(w) + c) : to_f32<T>(static_cast<const T*>(w)[c]);
  }
  for (int k = pairs + lane; k < 128; k += 32) s_cs[warp][k] = make_float2(1.f, 0.f);
  __syncthreads();
  const int lanes = LANES ? LANES : a.lanes;
  const int sub = lane % lanes, row = lane / lanes, rows = 32 / lanes;  // (lanes of no row: 32 is no multiple of five)
  int c[SLOTS][2];
  bool on[SLOTS][2];
#pragma unroll
  for (int s = 0; s < SLOTS; ++s) slot_runs<V, PAIRS>(a, sub + s * lanes, c[s], on[s]);
  int off[SLOTS][2];  // taken off a count of heads, it leaves none
#pragma unroll
  for (int s = 0; s < SLOTS; ++s)
#pragma unroll
    for (int u = 0; u < 2; ++u) off[s][u] = on[s][u] && row < rows ? 0 : -(1 << 30);
  R raw[kAhead][SLOTS][2];  // (runs behind the row stay zero)
#pragma unroll
  for (int k = 0; k < kAhead; ++k)
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) raw[k][s][0] = raw[k][s][1] = R{};

  for (int64_t item = (int64_t)blockIdx.x * kRopeWarps + warp; item < a.items; item += (int64_t)gridDim.x * kRopeWarps) {
    int64_t token = item;
    int chunk = 0, b = 0;
    if (a.items <= 0x7fffffff) {  // (32-bit divisions)
      if (a.chunks > 1) token = (int)item / a.chunks;
      if (a.batch > 1) b = (int)token / a.n;
    } else {
      token = item / a.chunks;
      b = (int)(token / a.n);
    }
    chunk = (int)(item - token * a.chunks);
    const int i = (int)(token - (int64_t)b * a.n);
    // steps: those of q's heads, filled up to a multiple of kAhead, then k's
    const int hq0 = (int)((int64_t)a.heads[0] * chunk / a.chunks), nq = (int)((int64_t)a.heads[0] * (chunk + 1) / a.chunks) - hq0;
    const int hk0 = (int)((int64_t)a.heads[1] * chunk / a.chunks), nk = (int)((int64_t)a.heads[1] * (chunk + 1) / a.chunks) - hk0;
    const int steps_q = ((nq + rows - 1) / rows + kAhead - 1) / kAhead * kAhead, steps = steps_q + (nk + rows - 1) / rows;
    auto at = [&](const int64_t (&st)[3], int h0) { return b * st[0] + i * st[1] + (h0 + row) * st[2]; };
    // what is fetched next: this lane's row, the heads that are left from it on, the steps until k's
    const T* fx = static_cast<const T*>(a.x[0]) + at(a.xs[0], hq0);
    int64_t f_stride = rows * a.xs[0][2];
    int f_left = nq - row, f_steps = steps_q;
    auto fetch = [&](R (&to)[SLOTS][2]) {
      if (f_steps-- == 0) {
        fx = static_cast<const T*>(a.x[1]) + at(a.xs[1], hk0);
        f_stride = rows * a.xs[1][2];
        f_left = nk - row;
      }
#pragma unroll
      for (int s = 0; s < SLOTS; ++s)
#pragma unroll
        for (int u = 0; u < 2; ++u) load_if(to[s][u], fx + c[s][u], f_left + off[s][u]);
      fx += f_stride;
      f_left -= rows;
    };
    long long p = i;
    if (pairs > 0 && a.pos) p = __ldg(&a.pos[b * a.pos_sb + i]);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) fetch(raw[k]);
    // ---- cosines and sines of the token, two pairs per lane
    __syncwarp();
    for (int k = lane; k < pairs; k += 32) {
      const long long turns = (long long)(s_turns[k] * (unsigned long long)p);  // modulo one, in [-1/2, 1/2)
      float sn, cs;
      sincospif(__ll2float_rn(turns) * 0x1p-63f, &sn, &cs);
      s_cs[warp][k] = make_float2(cs, sn);
    }
    __syncwarp();
    T* y = nullptr;  // where this lane's row goes
    int64_t y_stride = 0;
    Pair ca[N], cb[N], da[N], db[N];  // (x_i, x_j) -> (x_i ca + x_j cb, x_j da + x_i db)
#pragma unroll 1
    for (int base = 0, left = 0, live = 0; base < steps; base += kAhead) {
      if (base == 0 || base == steps_q) {
        const int w = base < steps_q ? 0 : 1;
        y = static_cast<T*>(a.y[w]) + at(a.ys[w], w ? hk0 : hq0);
        y_stride = rows * a.ys[w][2];
        left = w ? nk : nq;
        live = left - row;
        // weights of a run and cosines and sines of the pairs that follow one another from k on (neither leaves its array:
        // slots past the row end below channel 128 too)
        float p[4][SLOTS * V];
        auto put = [&](int e, float wi, float wj, const float2& t) {
          p[0][e] = wi * t.x;
          p[1][e] = -wj * t.y;
          p[2][e] = wj * t.x;
          p[3][e] = wi * t.y;
        };
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
          float wt[2][V];
          copy_run<V>(wt[0], &s_w[w][c[s][0]]);
          copy_run<V>(wt[1], &s_w[w][c[s][1]]);
          float2 t[V];
          if constexpr (PAIRS && V > 1) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              copy_run<V>(reinterpret_cast<float*>(t), &s_cs[warp][c[s][u] / 2].x);
#pragma unroll
              for (int z = 0; z < V / 2; ++z) put(s * V + u * (V / 2) + z, wt[u][2 * z], wt[u][2 * z + 1], t[z]);
            }
          } else {
            copy_run<2 * V>(reinterpret_cast<float*>(t), &s_cs[warp][PAIRS ? c[s][0] / 2 : c[s][0]].x);
#pragma unroll
            for (int z = 0; z < V; ++z) put(s * V + z, wt[0][z], wt[1][z], t[z]);
          }
        }
#pragma unroll
        for (int e = 0; e < N; ++e) {
          ca[e] = make_pair2(p[0][2 * e], p[0][2 * e + 1]);
          cb[e] = make_pair2(p[1][2 * e], p[1][2 * e + 1]);
          da[e] = make_pair2(p[2][2 * e], p[2][2 * e + 1]);
          db[e] = make_pair2(p[3][2 * e], p[3][2 * e + 1]);
        }
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        Pair xi[N], xj[N];
        if constexpr (V == 1) {
          auto one = [&](int s, int u) { return to_f32<T>(*reinterpret_cast<const T*>(&raw[k][s][u])); };
          xi[0] = make_pair2(one(0, 0), one(SLOTS - 1, 0));
          xj[0] = make_pair2(one(0, 1), one(SLOTS - 1, 1));
        } else {
#pragma unroll
          for (int s = 0; s < SLOTS; ++s) {
            float f[2][V];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int e = 0; e < V; e += 2)
                widen2<T>(reinterpret_cast<const uint32_t*>(&raw[k][s][u])[e / 2], f[u][e], f[u][e + 1]);
#pragma unroll
            for (int e = 0; e < V; e += 2) {
              // pairs e and e + 1
              if (PAIRS && V == 2) {
                xi[s] = make_pair2(f[0][0], f[1][0]);
                xj[s] = make_pair2(f[0][1], f[1][1]);
              } else if (PAIRS) {
                const int u = e / (V / 2), z = 2 * e % V;
                xi[s * V / 2 + e / 2] = make_pair2(f[u][z], f[u][(z + 2) % V]);
                xj[s * V / 2 + e / 2] = make_pair2(f[u][z + 1], f[u][(z + 3) % V]);
              } else {
                xi[s * V / 2 + e / 2] = make_pair2(f[0][e], f[0][e + 1]);
                xj[s * V / 2 + e / 2] = make_pair2(f[1][e], f[1][e + 1]);
              }
            }
          }
        }
        fetch(raw[k]);
        if (left <= 0) continue;  // (a step that fills up, for the whole warp)
        auto over_row = [&](float x, auto join) {
          if (LANES > 0 ? (LANES & (LANES - 1)) == 0 : (lanes & (lanes - 1)) == 0) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
              if (o < lanes) x = join(x, __shfl_xor_sync(0xffffffffu, x, o));
            return x;
          }
          // in the order of the lanes, so that all of a row get the same
          float all = 0.f;
#pragma unroll
          for (int o = 0; o < (LANES > 0 ? LANES : 16); ++o)
            if (o < lanes) all = join(all, __shfl_sync(0xffffffffu, x, (row * lanes + o) & 31));
          return all;
        };
        auto squares = [&]() {
          Pair s2 = mul_pair2(xi[0], xi[0]), t2 = mul_pair2(xj[0], xj[0]);
#pragma unroll
          for (int e = 1; e < N; ++e) {
            s2 = fma_pair2(xi[e], xi[e], s2);
            t2 = fma_pair2(xj[e], xj[e], t2);
          }
          float s0, s1, t0, t1;
          split_pair2(s2, s0, s1);
          split_pair2(t2, t0, t1);
          return over_row((s0 + s1) + (t0 + t1), [](float x, float y) { return x + y; });
        };
        float v = fmaf(squares(), a.inv_d, a.eps);
        if constexpr (ANY) {
          const bool odd = live > 0 && row < rows && !(v > kLeastSquare && v < kMostSquare);
          if (__any_sync(0xffffffffu, odd)) {
            // its largest channel, or the root of eps, comes to about one
            float most = 0.f;
#pragma unroll
            for (int e = 0; e < N; ++e) {
              float x0, x1, x2, x3;
              split_pair2(xi[e], x0, x1);
              split_pair2(xj[e], x2, x3);
              most = fmaxf(fmaxf(most, fmaxf(fabsf(x0), fabsf(x1))), fmaxf(fabsf(x2), fabsf(x3)));
            }
            most = fmaxf(over_row(most, [](float x, float y) { return fmaxf(x, y); }), sqrtf(a.eps));
            const int e0 = max(1, min(253, (int)(__float_as_uint(most) >> 23)));
            const float up = odd ? __uint_as_float((uint32_t)(254 - e0) << 23) : 1.f;
            const Pair up2 = make_pair2(up, up);
#pragma unroll
            for (int e = 0; e < N; ++e) {
              xi[e] = mul_pair2(xi[e], up2);
              xj[e] = mul_pair2(xj[e], up2);
            }
            v = fmaf(squares(), a.inv_d, a.eps * up * up);
          }
        }
        const float f = rsqrtf(v);
        const Pair f2 = make_pair2(f, f);
        float zi[2 * N], zj[2 * N];
#pragma unroll
        for (int e = 0; e < N; ++e) {
          split_pair2(mul_pair2(f2, fma_pair2(xi[e], ca[e], mul_pair2(xj[e], cb[e]))), zi[2 * e], zi[2 * e + 1]);
          split_pair2(mul_pair2(f2, fma_pair2(xj[e], da[e], mul_pair2(xi[e], db[e]))), zj[2 * e], zj[2 * e + 1]);
        }
#pragma unroll
        for (int s = 0; s < SLOTS; ++s)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            R r;
            T* t = reinterpret_cast<T*>(&r);
#pragma unroll
            for (int e = 0; e < V; ++e) {
              const int z = PAIRS && V > 1 ? s * V + u * (V / 2) + e / 2 : s * V + e;
              t[e] = narrow<T>((PAIRS && V > 1 ? e & 1 : u) ? zj[z] : zi[z]);
            }
            store_if(y + c[s][u], r, live + off[s][u]);
          }
        y += y_stride;
        left -= rows;
        live -= rows;
      }
    }
  }
}

template <typename T, bool PAIRS>
cudaError_t launch_rope(const RopeArgs& a, int v, int blocks, cudaStream_t st) {
  const dim3 g(blocks), t(kRopeWarps * 32);
  if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    if (a.eps < kLeastSquare) {  // (fp16 rows have no such squares)
      if (v == 8) return launch_pdl(rope_kernel<T, 8, 1, PAIRS, 0, true>, g, t, 0, st, a);
      if (v == 4) return launch_pdl(rope_kernel<T, 4, 1, PAIRS, 0, true>, g, t, 0, st, a);
      if (v == 2) return launch_pdl(rope_kernel<T, 2, 1, PAIRS, 0, true>, g, t, 0, st, a);
      return launch_pdl(rope_kernel<T, 1, 2, PAIRS, 0, true>, g, t, 0, st, a);
    }
  }
  if (v == 8 && a.lanes == 8) return launch_pdl(rope_kernel<T, 8, 1, PAIRS, 8, false>, g, t, 0, st, a);
  if (v == 8 && a.lanes == 5) return launch_pdl(rope_kernel<T, 8, 1, PAIRS, 5, false>, g, t, 0, st, a);
  if (v == 8 && a.lanes == 6) return launch_pdl(rope_kernel<T, 8, 1, PAIRS, 6, false>, g, t, 0, st, a);
  if (v == 8 && a.lanes == 4) return launch_pdl(rope_kernel<T, 8, 1, PAIRS, 4, false>, g, t, 0, st, a);
  if (v == 8) return launch_pdl(rope_kernel<T, 8, 1, PAIRS, 0, false>, g, t, 0, st, a);
  if (v == 4) return launch_pdl(rope_kernel<T, 4, 1, PAIRS, 0, false>, g, t, 0, st, a);
  if (v == 2) return launch_pdl(rope_kernel<T, 2, 1, PAIRS, 0, false>, g, t, 0, st, a);
  return launch_pdl(rope_kernel<T, 1, 2, PAIRS, 0, false>, g, t, 0, st, a);
}

}  // namespace
}  // namespace sage

using namespace sage;

extern "C" int sage_qk_norm_rope(const sage_tensor* q, const sage_tensor* k, const sage_tensor* q_out,
                                 const sage_tensor* k_out, const int32_t* positions, int64_t positions_stride,
                                 const float* inv_freq, const void* q_weight, const void* k_weight, int weight_dtype,
                                 int batch, int heads_q, int heads_kv, int seqlen, int head_dim, int rot_dim, int dtype,
                                 int tensor_layout, int interleaved, float eps, void* stream) {
  if (!q || !k || !q_out || !k_out) return SAGE_ERR_INVALID_ARG;
  if (head_dim < 1 || head_dim > 128) return SAGE_ERR_HEAD_DIM;
  if (dtype != SAGE_F16 && dtype != SAGE_BF16) return SAGE_ERR_DTYPE;
  if ((q_weight || k_weight) && weight_dtype != dtype && weight_dtype != SAGE_F32) return SAGE_ERR_DTYPE;
  if (tensor_layout != SAGE_HND && tensor_layout != SAGE_NHD) return SAGE_ERR_INVALID_ARG;
  if (batch < 0 || seqlen < 0 || (int64_t)batch * seqlen > 0x7fffffff || heads_q < 1 || heads_kv < 1 || rot_dim < 0 || rot_dim > head_dim || rot_dim % 2 ||
      !(eps >= 0.f) || std::isinf(eps) || positions_stride < 0 || (rot_dim > 0 && !inv_freq))
    return SAGE_ERR_INVALID_ARG;
  if (batch == 0 || seqlen == 0) return SAGE_OK;
  RopeArgs a{};
  const sage_tensor* t[2][2] = {{q, q_out}, {k, k_out}};
  const int heads[2] = {heads_q, heads_kv};
  const int hi = tensor_layout == SAGE_HND ? 1 : 2, ni = tensor_layout == SAGE_HND ? 2 : 1;
  // channels that one access takes: what every address, stride and the place of a pair's second half allow
  int v = 8;
  auto fits = [&](int64_t x) { while (x % v) v /= 2; };
  fits(head_dim);
  if (!interleaved) fits(rot_dim / 2);
  for (int i = 0; i < 2; ++i) {
    for (int o = 0; o < 2; ++o) {
      const sage_tensor& s = *t[i][o];
      if (!s.data) return SAGE_ERR_INVALID_ARG;
      if (reinterpret_cast<uintptr_t>(s.data) % 2) return SAGE_ERR_STRIDE;
      const int64_t st[3] = {s.stride[0], s.stride[ni], s.stride[hi]};
      const int len[3] = {batch, seqlen, heads[i]};
      fits(static_cast<int64_t>(reinterpret_cast<uintptr_t>(s.data) / 2 % 8));
      for (int x = 0; x < 3; ++x) {
        // (rows that are written must not coincide)
        if (st[x] < 0 || (o && len[x] > 1 && st[x] == 0)) return SAGE_ERR_STRIDE;
        if (len[x] > 1) fits(st[x]);
        (o ? a.ys : a.xs)[i][x] = st[x];
      }
    }
    a.x[i] = t[i][0]->data;
    a.y[i] = t[i][1]->data;
    a.heads[i] = heads[i];
  }
  a.w[0] = q_weight;
  a.w[1] = k_weight;
  a.w32 = weight_dtype == SAGE_F32;
  for (const void* p : a.w)
    if (reinterpret_cast<uintptr_t>(p) % (a.w32 ? 4 : 2)) return SAGE_ERR_INVALID_ARG;
  for (const void* p : {(const void*)positions, (const void*)inv_freq})
    if (reinterpret_cast<uintptr_t>(p) % 4) return SAGE_ERR_INVALID_ARG;
  if (!sage_device_supported()) return SAGE_ERR_DEVICE;
  a.pos = positions;
  a.pos_sb = positions_stride;
  a.freq = inv_freq;
  a.batch = batch; a.n = seqlen; a.d = head_dim; a.rot = rot_dim;
  a.interleaved = interleaved != 0;
  a.eps = eps;
  a.inv_d = 1.0f / static_cast<float>(head_dim);
  // slots of a row: its rotated pairs of runs, then the other channels two runs at a time
  const int turned = a.interleaved ? 0 : rot_dim / 2 / v, rest = head_dim - 2 * turned * v;
  const int slots = turned + (rest + 2 * v - 1) / (2 * v);
  a.lanes = 1;
  while (a.lanes < slots && a.lanes < 32) a.lanes *= 2;
  if (slots < 16 && 32 / slots > 32 / a.lanes) a.lanes = slots;
  const int64_t tokens = (int64_t)batch * seqlen;
  // a token's heads are shared by several warps where there are few tokens
  const int rows = 32 / a.lanes, most = ((heads_q > heads_kv ? heads_q : heads_kv) + rows - 1) / rows;
  const int64_t want = (152 * kRopeBlocks * kRopeWarps + tokens - 1) / tokens;
  a.chunks = (int)(want < most ? want : most);
  a.items = tokens * a.chunks;
  const int64_t blocks = (a.items + kRopeWarps - 1) / kRopeWarps;
  const int grid = (int)(blocks < 152 * kRopeBlocks ? blocks : 152 * kRopeBlocks);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      dtype == SAGE_F16 ? (a.interleaved ? launch_rope<__half, true>(a, v, grid, st) : launch_rope<__half, false>(a, v, grid, st))
                        : (a.interleaved ? launch_rope<__nv_bfloat16, true>(a, v, grid, st)
                                         : launch_rope<__nv_bfloat16, false>(a, v, grid, st));
  return e == cudaSuccess ? SAGE_OK : note_cuda_failure(e, "norm and rotation");
}
