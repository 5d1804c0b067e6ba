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
// position and inv_freq / 2 pi (off by 2^-54 of inv_freq and 2^-65 per position, however far that is); 32-bit floats would
// lose an angle at position 2^20 by 0.06. All arithmetic on values is in 32 bits, rounded once.
#include <cmath>

#include "../../include/sageattn.h"
#include "launch.h"

namespace sage {
namespace {

constexpr int kRopeWarps = 8;
constexpr int kMaxPairs = 64;

struct RopeArgs {
  const void* x[2];          // q, k
  void* y[2];
  int64_t xs[2][3], ys[2][3];  // element strides of batch, token, head
  const void* w[2];          // or null
  const int* pos; int64_t pos_sb;  // null: the token's place in its row
  const float* freq;
  int heads[2], chunks[2];   // chunks: items that share a token's heads
  int batch, n, d, rot;
  int interleaved, w32, lanes;  // lanes of a row: a power of two
  int64_t items;
  float eps, inv_d;
};

template <typename T, int V> struct Run;  // V channels as one access
template <typename T> struct Run<T, 8> { using type = uint4; };
template <typename T> struct Run<T, 4> { using type = uint2; };
template <typename T> struct Run<T, 2> { using type = uint32_t; };
template <typename T> struct Run<T, 1> { using type = uint16_t; };

template <typename T>
__device__ __forceinline__ T narrow(float x) {
  if constexpr (std::is_same<T, __half>::value) return __float2half_rn(x);
  else return __float2bfloat16_rn(x);
}

// First channels of the two runs of slot x, and the first pair; `on`: which of the runs lie within the row.
template <int V>
__device__ __forceinline__ void slot_runs(const RopeArgs& a, int x, int (&c)[2], bool (&on)[2]) {
  const int half = a.rot / 2, turned = half / V;
  if (a.interleaved) {
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

// SLOTS: pairs of runs per lane.
template <typename T, int V, int SLOTS>
__global__ void __launch_bounds__(kRopeWarps * 32) rope_kernel(const RopeArgs a) {
  using R = typename Run<T, V>::type;
  __shared__ unsigned long long s_turns[kMaxPairs];
  __shared__ float2 s_cs[kRopeWarps][kMaxPairs];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int pairs = a.rot / 2;
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x < pairs) {
    // turns per position modulo 1, in units of 2^-64
    double f = (double)__ldg(&a.freq[threadIdx.x]) * 0.15915494309189533577;
    f -= floor(f);
    s_turns[threadIdx.x] = __double2ull_rn(f * 18446744073709551616.0);
  }
  __syncthreads();
  const int sub = lane & (a.lanes - 1), row = lane / a.lanes, rows = 32 / a.lanes;
  int c[SLOTS][2];
  bool on[SLOTS][2];
#pragma unroll
  for (int s = 0; s < SLOTS; ++s) slot_runs<V>(a, sub + s * a.lanes, c[s], on[s]);
  const int per_token = a.chunks[0] + a.chunks[1];

  for (int64_t item = (int64_t)blockIdx.x * kRopeWarps + warp; item < a.items; item += (int64_t)gridDim.x * kRopeWarps) {
    const int64_t token = item / per_token;
    int chunk = (int)(item - token * per_token);
    const int which = chunk < a.chunks[0] ? 0 : 1;
    if (which) chunk -= a.chunks[0];
    const int b = (int)(token / a.n), i = (int)(token - (int64_t)b * a.n);
    // ---- cosines and sines of the token, two pairs per lane
    __syncwarp();
    if (pairs > 0) {
      const long long p = a.pos ? __ldg(&a.pos[b * a.pos_sb + i]) : i;
      for (int k = lane; k < pairs; k += 32) {
        const long long turns = (long long)(s_turns[k] * (unsigned long long)p);  // modulo one, in [-1/2, 1/2)
        float sn, cs;
        sincospif(__ll2float_rn(turns) * 0x1p-63f, &sn, &cs);
        s_cs[warp][k] = make_float2(cs, sn);
      }
    }
    __syncwarp();
    float2 cs[SLOTS][V];
    float w[SLOTS][2][V];
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        // the e-th pair of a slot: channels e of both runs, or two neighbours of one of them
        int pr;
        bool turned;
        if (a.interleaved) {
          pr = (V == 1 ? c[s][0] : e < V / 2 ? c[s][0] + 2 * e : c[s][1] + 2 * (e - V / 2)) / 2;
          turned = pr < pairs;
        } else {
          pr = c[s][0] + e;
          turned = pr < pairs;
        }
        cs[s][e] = turned ? s_cs[warp][pr] : make_float2(1.f, 0.f);
      }
      const void* wp = a.w[which];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          w[s][u][e] = 1.f;
          if (wp && on[s][u])
            w[s][u][e] = a.w32 ? __ldg(static_cast<const float*>(wp) + c[s][u] + e)
                               : to_f32<T>(static_cast<const T*>(wp)[c[s][u] + e]);
        }
    }
    // ---- the heads of this item
    const int heads = a.heads[which], h0 = (int)((int64_t)heads * chunk / a.chunks[which]),
              h1 = (int)((int64_t)heads * (chunk + 1) / a.chunks[which]);
    const T* xb = static_cast<const T*>(a.x[which]) + b * a.xs[which][0] + i * a.xs[which][1];
    T* yb = static_cast<T*>(a.y[which]) + b * a.ys[which][0] + i * a.ys[which][1];
#pragma unroll 2
    for (int h = h0 + row; h - row < h1; h += rows) {
      const bool live = h < h1;
      float y[SLOTS][2][V];
      float sum = 0.f;
#pragma unroll
      for (int s = 0; s < SLOTS; ++s)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          R r{};
          if (live && on[s][u]) r = *reinterpret_cast<const R*>(xb + h * a.xs[which][2] + c[s][u]);
          const T* t = reinterpret_cast<const T*>(&r);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            y[s][u][e] = to_f32<T>(t[e]);
            sum = fmaf(y[s][u][e], y[s][u][e], sum);
          }
        }
      for (int o = a.lanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const float f = rsqrtf(fmaf(sum, a.inv_d, a.eps));
#pragma unroll
      for (int s = 0; s < SLOTS; ++s) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 0; e < V; ++e) y[s][u][e] = y[s][u][e] * f * w[s][u][e];
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float *p, *q;
          if (V > 1 && a.interleaved) {
            p = e < V / 2 ? &y[s][0][(2 * e) % V] : &y[s][1][(2 * e) % V];
            q = e < V / 2 ? &y[s][0][(2 * e + 1) % V] : &y[s][1][(2 * e + 1) % V];
          } else {
            p = &y[s][0][e];
            q = &y[s][1][e];
          }
          const float x0 = *p, x1 = *q;
          *p = x0 * cs[s][e].x - x1 * cs[s][e].y;
          *q = x1 * cs[s][e].x + x0 * cs[s][e].y;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (!live || !on[s][u]) continue;
          R r;
          T* t = reinterpret_cast<T*>(&r);
#pragma unroll
          for (int e = 0; e < V; ++e) t[e] = narrow<T>(y[s][u][e]);
          *reinterpret_cast<R*>(yb + h * a.ys[which][2] + c[s][u]) = r;
        }
      }
    }
  }
}

template <typename T>
cudaError_t launch_rope(const RopeArgs& a, int v, int blocks, cudaStream_t st) {
  const dim3 g(blocks), t(kRopeWarps * 32);
  if (v == 8) return launch_pdl(rope_kernel<T, 8, 1>, g, t, 0, st, a);
  if (v == 4) return launch_pdl(rope_kernel<T, 4, 1>, g, t, 0, st, a);
  if (v == 2) return launch_pdl(rope_kernel<T, 2, 1>, g, t, 0, st, a);
  return launch_pdl(rope_kernel<T, 1, 2>, g, t, 0, st, a);
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
  if (batch < 0 || seqlen < 0 || heads_q < 1 || heads_kv < 1 || rot_dim < 0 || rot_dim > head_dim || rot_dim % 2 ||
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
  const int64_t tokens = (int64_t)batch * seqlen;
  // a token's heads are shared by several warps where there are few tokens
  const int rows = 32 / a.lanes;
  for (int i = 0; i < 2; ++i) {
    const int most = (heads[i] + rows - 1) / rows;
    const int64_t want = (152 * 24 + tokens - 1) / tokens;
    a.chunks[i] = (int)(want < most ? want : most);
    if (a.chunks[i] < 1) a.chunks[i] = 1;
  }
  a.items = tokens * (a.chunks[0] + a.chunks[1]);
  const int64_t blocks = (a.items + kRopeWarps - 1) / kRopeWarps;
  const int grid = (int)(blocks < 152 * 3 ? blocks : 152 * 3);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == SAGE_F16 ? launch_rope<__half>(a, v, grid, st) : launch_rope<__nv_bfloat16>(a, v, grid, st);
  return e == cudaSuccess ? SAGE_OK : note_cuda_failure(e, "norm and rotation");
}
