// norm_step.cu -- the residual step between two blocks with given stream weights: the norm after
// a block fused with its gate and residual scale, the residual streams, and the norm before the next
// block; and its gradients.
//
// Per token, with F the block's output, a the gate (1, its value or its sigmoid), s the residual
// scale and n = 1 or 4 streams:
//   r_F = (mean F^2 + eps)^(-1/2),  h_i = s a_i gpost_i,  Z = h F r_F  (r_F = gpost = 1 without post norm)
//   X'_k = u_k Z + sum_j C_jk X_j,  yh = sum_k p_k X'_k,  r_y = (mean yh^2 + eps)^(-1/2),
//   y = gpre yh r_y.
// Everything between the bf16 inputs and the bf16 outputs X', y is float32: one rounding each.
// Gradients (G_k that of X'_k in all):
//   T = sum gpre gy yh,  gyh = r_y gpre gy - (r_y^3 T / d) yh,  G_k = gXp_k + p_k gyh,
//   gX_j = sum_k C_jk G_k,  gC_jk = G_k . X_j,  gu_k = G_k . Z,  gp_k = gyh . X'_k,
//   q = sum_k u_k G_k (the gradient of Z),  S = sum h q F,  gF = r_F h q - (r_F^3 S / d) F,
//   ggate = s gpost F r_F q (times a (1 - a) for the sigmoid),
//   ggpost += s a F r_F q,  ggpre += gy yh r_y  over the tokens.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "internal.h"
#include "mx8.cuh"

namespace mhc {
namespace {

constexpr int NT = 256;              // threads of a block
constexpr int NW = NT / 32;

// Sums of V values over the block, in the same order for every call; the result in every thread.
template <int V>
__device__ __forceinline__ void block_sums(float (&v)[V], float* scratch) {
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
  if (l == 0)
#pragma unroll
    for (int i = 0; i < V; ++i) scratch[w * V + i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float t = 0.f;
    for (int k = 0; k < NW; ++k) t += scratch[k * V + i];
    v[i] = t;
  }
  __syncthreads();
}

struct C8 {
  f2 v[4];
};
__device__ __forceinline__ C8 unpack8(uint4 w) {
  return C8{{bf2_to_f2(w.x), bf2_to_f2(w.y), bf2_to_f2(w.z), bf2_to_f2(w.w)}};
}
__device__ __forceinline__ uint4 pack8(const C8& c) {
  return make_uint4(f2_to_bf2(c.v[0]), f2_to_bf2(c.v[1]), f2_to_bf2(c.v[2]), f2_to_bf2(c.v[3]));
}
__device__ __forceinline__ C8 gain8(const float* g, int c) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(g) + 2 * c);
  const float4 b = __ldg(reinterpret_cast<const float4*>(g) + 2 * c + 1);
  return C8{{f2{a.x, a.y}, f2{a.z, a.w}, f2{b.x, b.y}, f2{b.z, b.w}}};
}
__device__ __forceinline__ f2 both(float v) { return f2{v, v}; }
__device__ __forceinline__ float sigmoid_n(float z) { return 1.0f / (1.0f + expf(-z)); }

// Row `row` of a tensor, chunk c of 8 features: bf16, or MXFP8 codes and scales.
template <bool CK>
__device__ __forceinline__ C8 load8(const void* x, const uint8_t* scales, int64_t row, int c, int d) {
  if (!CK) return unpack8(__ldg(reinterpret_cast<const uint4*>(x) + row * (d / 8) + c));
  const uint2 v = __ldg(reinterpret_cast<const uint2*>(x) + row * (d / 8) + c);
  const f2 s = both(scale_value(__ldg(scales + row * ((d + MX_BLOCK - 1) / MX_BLOCK) + c / 4)));
  return C8{{decode2(v.x, s), decode2(v.x >> 16, s), decode2(v.y, s), decode2(v.y >> 16, s)}};
}

// The stream weights of a token: cc[j][k] the weight of input stream j in output stream k.
template <int NS>
struct Weights {
  float p[NS], u[NS], cc[NS][NS];
};
template <int NS>
__device__ __forceinline__ Weights<NS> load_weights(const NormArgs& P, int64_t t) {
  Weights<NS> w;
  const int64_t row = (P.flags & FLAG_WEIGHTS_SHARED) ? 0 : t;
#pragma unroll
  for (int k = 0; k < NS; ++k) {
    w.p[k] = P.pre ? __ldg(P.pre + row * NS + k) : 1.f;
    w.u[k] = P.post ? __ldg(P.post + row * NS + k) : 1.f;
#pragma unroll
    for (int j = 0; j < NS; ++j)
      w.cc[j][k] = P.comb ? __ldg(P.comb + row * NS * NS + ((P.flags & 1u) ? k * NS + j : j * NS + k)) : 1.f;
  }
  return w;
}

// The gate's values and its derivative for one chunk (ones where there is none).
__device__ __forceinline__ void gate8(const NormArgs& P, int64_t t, int c, C8& a, C8& da) {
#pragma unroll
  for (int i = 0; i < 4; ++i) a.v[i] = da.v[i] = both(1.f);
  if (!P.gate) return;
  a = unpack8(__ldg(reinterpret_cast<const uint4*>(P.gate) + t * (P.d / 8) + c));
  if (!(P.flags & FLAG_GATE_SIGMOID)) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a.v[i] = f2{sigmoid_n(a.v[i].x), sigmoid_n(a.v[i].y)};
    da.v[i] = f2{a.v[i].x * (1.f - a.v[i].x), a.v[i].y * (1.f - a.v[i].y)};
  }
}

template <int NS>
__global__ void __launch_bounds__(NT) norm_step_kernel(const NormArgs P) {
  extern __shared__ float yh_s[];
  __shared__ float scratch[NW];
  const int chunks = P.d / 8;
  for (int64_t t = blockIdx.x; t < P.N; t += gridDim.x) {
    const Weights<NS> w = load_weights<NS>(P, t);
    float r = 1.f;
    if (P.gain_post) {
      f2 s{0.f, 0.f};
      for (int c = threadIdx.x; c < chunks; c += NT) {
        const C8 f = load8<false>(P.F, nullptr, t, c, P.d);
#pragma unroll
        for (int i = 0; i < 4; ++i) s = fma2(f.v[i], f.v[i], s);
      }
      float v[1] = {s.x + s.y};
      block_sums<1>(v, scratch);
      r = rsqrtf(__fdiv_rn(v[0], static_cast<float>(P.d)) + P.eps);
    }
    f2 s{0.f, 0.f};
    for (int c = threadIdx.x; c < chunks; c += NT) {
      const C8 f = load8<false>(P.F, nullptr, t, c, P.d);
      C8 x[NS], a, da;
#pragma unroll
      for (int j = 0; j < NS; ++j) x[j] = load8<false>(P.X, nullptr, t * NS + j, c, P.d);
      gate8(P, t, c, a, da);
      const C8 g = P.gain_post ? gain8(P.gain_post, c) : C8{{both(1.f), both(1.f), both(1.f), both(1.f)}};
      C8 xp[NS];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f2 h = mul2(mul2(both(P.res_scale), a.v[i]), g.v[i]);
        const f2 z = mul2(mul2(h, f.v[i]), both(r));
        f2 yh{0.f, 0.f};
#pragma unroll
        for (int k = 0; k < NS; ++k) {
          f2 v = mul2(both(w.u[k]), z);
#pragma unroll
          for (int j = 0; j < NS; ++j) v = fma2(both(w.cc[j][k]), x[j].v[i], v);
          xp[k].v[i] = v;
          yh = fma2(both(w.p[k]), v, yh);
        }
        s = fma2(yh, yh, s);
        yh_s[8 * c + 2 * i] = yh.x;
        yh_s[8 * c + 2 * i + 1] = yh.y;
      }
#pragma unroll
      for (int k = 0; k < NS; ++k) reinterpret_cast<uint4*>(P.X_out)[(t * NS + k) * chunks + c] = pack8(xp[k]);
    }
    float v[1] = {s.x + s.y};
    block_sums<1>(v, scratch);
    const float ry = rsqrtf(__fdiv_rn(v[0], static_cast<float>(P.d)) + P.eps);
    for (int c = threadIdx.x; c < chunks; c += NT) {
      const C8 g = gain8(P.gain_pre, c);
      C8 o;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        o.v[i] = mul2(g.v[i], mul2(f2{yh_s[8 * c + 2 * i], yh_s[8 * c + 2 * i + 1]}, both(ry)));
      reinterpret_cast<uint4*>(P.y)[t * chunks + c] = pack8(o);
    }
  }
}

// One block per token at a time. Each thread owns the same chunks of every token, so the
// parameter gradients gather in the block's own row of the workspace without atomics.
template <int NS, bool CK>
__global__ void __launch_bounds__(NT) norm_step_backward_kernel(const NormArgs P) {
  constexpr int NSUM = 1 + 2 * NS + NS * NS;
  extern __shared__ float q_s[];
  __shared__ float scratch[NW * NSUM];
  const int chunks = P.d / 8;
  const float fd = static_cast<float>(P.d);
  float* part = P.partial + blockIdx.x * static_cast<int64_t>(norm_partial_floats(P.d));
  float* part_post = part + P.d;
  float* part_w = part + 2 * P.d;
  bool first = true;
  float shared_sum = 0.f;   // thread i < 2 NS + NS^2: the i-th weight's gradient over this block's tokens
  for (int64_t t = blockIdx.x; t < P.N; t += gridDim.x) {
    const Weights<NS> w = load_weights<NS>(P, t);
    float r = 1.f;
    if (P.gain_post) {
      f2 s{0.f, 0.f};
      for (int c = threadIdx.x; c < chunks; c += NT) {
        const C8 f = load8<CK>(P.F, P.F_scale, t, c, P.d);
#pragma unroll
        for (int i = 0; i < 4; ++i) s = fma2(f.v[i], f.v[i], s);
      }
      float v[1] = {s.x + s.y};
      block_sums<1>(v, scratch);
      r = rsqrtf(__fdiv_rn(v[0], fd) + P.eps);
    }
    auto forward = [&](int c, C8 (&x)[NS], C8& f, C8& a, C8& da, C8& g, C8& z, C8 (&xp)[NS], C8& yh) {
      f = load8<CK>(P.F, P.F_scale, t, c, P.d);
#pragma unroll
      for (int j = 0; j < NS; ++j) x[j] = load8<CK>(P.X, P.X_scale, t * NS + j, c, P.d);
      gate8(P, t, c, a, da);
      g = P.gain_post ? gain8(P.gain_post, c) : C8{{both(1.f), both(1.f), both(1.f), both(1.f)}};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        z.v[i] = mul2(mul2(mul2(mul2(both(P.res_scale), a.v[i]), g.v[i]), f.v[i]), both(r));
        yh.v[i] = both(0.f);
#pragma unroll
        for (int k = 0; k < NS; ++k) {
          f2 v = mul2(both(w.u[k]), z.v[i]);
#pragma unroll
          for (int j = 0; j < NS; ++j) v = fma2(both(w.cc[j][k]), x[j].v[i], v);
          xp[k].v[i] = v;
          yh.v[i] = fma2(both(w.p[k]), v, yh.v[i]);
        }
      }
    };
    f2 sy{0.f, 0.f}, st{0.f, 0.f};
    for (int c = threadIdx.x; c < chunks; c += NT) {
      C8 x[NS], f, a, da, g, z, xp[NS], yh;
      forward(c, x, f, a, da, g, z, xp, yh);
      const C8 gn = gain8(P.gain_pre, c);
      const C8 gy = load8<false>(P.gy, nullptr, t, c, P.d);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sy = fma2(yh.v[i], yh.v[i], sy);
        st = fma2(mul2(gn.v[i], gy.v[i]), yh.v[i], st);
      }
    }
    float v2[2] = {sy.x + sy.y, st.x + st.y};
    block_sums<2>(v2, scratch);
    const float ry = rsqrtf(__fdiv_rn(v2[0], fd) + P.eps);
    const float tau = ry * ry * ry * v2[1] / fd;
    f2 acc[NSUM];
#pragma unroll
    for (int i = 0; i < NSUM; ++i) acc[i] = both(0.f);
    for (int c = threadIdx.x; c < chunks; c += NT) {
      C8 x[NS], f, a, da, g, z, xp[NS], yh, G[NS], gx[NS], gg;
      forward(c, x, f, a, da, g, z, xp, yh);
      const C8 gn = gain8(P.gain_pre, c);
      const C8 gy = load8<false>(P.gy, nullptr, t, c, P.d);
#pragma unroll
      for (int k = 0; k < NS; ++k) G[k] = load8<false>(P.gXp, nullptr, t * NS + k, c, P.d);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f2 gyh = fma2(mul2(both(ry), gn.v[i]), gy.v[i], mul2(both(-tau), yh.v[i]));
        f2 q = both(0.f);
#pragma unroll
        for (int k = 0; k < NS; ++k) {
          G[k].v[i] = fma2(both(w.p[k]), gyh, G[k].v[i]);
          q = fma2(both(w.u[k]), G[k].v[i], q);
          acc[1 + k] = fma2(gyh, xp[k].v[i], acc[1 + k]);
          acc[1 + NS + k] = fma2(G[k].v[i], z.v[i], acc[1 + NS + k]);
#pragma unroll
          for (int j = 0; j < NS; ++j)
            acc[1 + 2 * NS + j * NS + k] = fma2(G[k].v[i], x[j].v[i], acc[1 + 2 * NS + j * NS + k]);
        }
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          f2 v = both(0.f);
#pragma unroll
          for (int k = 0; k < NS; ++k) v = fma2(both(w.cc[j][k]), G[k].v[i], v);
          gx[j].v[i] = v;
        }
        // h q F, the gain's and the gate's gradients
        const f2 fr = mul2(f.v[i], both(r));
        const f2 sq = mul2(both(P.res_scale), q);
        const f2 hq = mul2(mul2(sq, a.v[i]), g.v[i]);
        acc[0] = fma2(hq, f.v[i], acc[0]);
        gg.v[i] = mul2(mul2(mul2(sq, g.v[i]), fr), da.v[i]);
        q_s[8 * c + 2 * i] = hq.x;
        q_s[8 * c + 2 * i + 1] = hq.y;
        const f2 ip = mul2(gy.v[i], mul2(yh.v[i], both(ry)));
        const f2 io = mul2(mul2(sq, a.v[i]), fr);
        float* pp = part + 8 * c + 2 * i;
        float* po = part_post + 8 * c + 2 * i;
        pp[0] = first ? ip.x : pp[0] + ip.x;
        pp[1] = first ? ip.y : pp[1] + ip.y;
        po[0] = first ? io.x : po[0] + io.x;
        po[1] = first ? io.y : po[1] + io.y;
      }
#pragma unroll
      for (int j = 0; j < NS; ++j) reinterpret_cast<uint4*>(P.gX)[(t * NS + j) * chunks + c] = pack8(gx[j]);
      if (P.gate) reinterpret_cast<uint4*>(P.ggate)[t * chunks + c] = pack8(gg);
    }
    float v[NSUM];
#pragma unroll
    for (int i = 0; i < NSUM; ++i) v[i] = acc[i].x + acc[i].y;
    block_sums<NSUM>(v, scratch);
    const float cf = P.gain_post ? r * r * r * v[0] / fd : 0.f;
    for (int c = threadIdx.x; c < chunks; c += NT) {
      const C8 f = load8<CK>(P.F, P.F_scale, t, c, P.d);
      C8 o;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        o.v[i] = fma2(both(r), f2{q_s[8 * c + 2 * i], q_s[8 * c + 2 * i + 1]}, mul2(both(-cf), f.v[i]));
      reinterpret_cast<uint4*>(P.gF)[t * chunks + c] = pack8(o);
    }
    if (P.pre) {
#pragma unroll
      for (int i = 1; i < NSUM; ++i) {
        if (threadIdx.x != i - 1) continue;
        if (P.flags & FLAG_WEIGHTS_SHARED) {
          shared_sum += v[i];
        } else if (i <= NS) {
          P.gpre[t * NS + i - 1] = v[i];
        } else if (i <= 2 * NS) {
          P.gpost[t * NS + i - 1 - NS] = v[i];
        } else {
          const int e = i - 1 - 2 * NS, j = e / NS, k = e % NS;
          P.gcomb[t * NS * NS + ((P.flags & 1u) ? k * NS + j : e)] = v[i];
        }
      }
    }
    first = false;
  }
  if ((P.flags & FLAG_WEIGHTS_SHARED) && threadIdx.x < NSUM - 1) part_w[threadIdx.x] = shared_sum;
}

// Sums of the blocks' partial rows, in the blocks' order: 32 columns a block, 8 threads a column.
__global__ void __launch_bounds__(256) norm_reduce_kernel(const NormArgs P, int rows) {
  __shared__ float red[8][33];
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  const int cols = norm_partial_floats(P.d);
  float v = 0.f;
  if (col < cols)
    for (int r = g; r < rows; r += 8) v += P.partial[r * static_cast<int64_t>(cols) + col];
  red[g][lane] = v;
  __syncthreads();
  if (g != 0 || col >= cols) return;
  float t = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) t += red[k][lane];
  const int n = P.n, e = col - 2 * P.d;
  if (col < P.d) {
    P.ggain_pre[col] = t;
  } else if (e < 0) {
    if (P.gain_post) P.ggain_post[col - P.d] = t;
  } else if (P.flags & FLAG_WEIGHTS_SHARED) {
    if (e < n) {
      P.gpre[e] = t;
    } else if (e < 2 * n) {
      P.gpost[e - n] = t;
    } else if (e < 2 * n + n * n) {
      const int i = e - 2 * n, j = i / n, k = i % n;
      P.gcomb[(P.flags & 1u) ? k * n + j : i] = t;
    }
  }
}

int norm_sms() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return sms;
}

template <typename K>
cudaError_t launch_rows(K kernel, const NormArgs& a, int64_t grid, cudaStream_t stream) {
  const int smem = a.d * 4;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  kernel<<<static_cast<unsigned>(grid), NT, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_step(const NormArgs& a, cudaStream_t stream) {
  const int sms = norm_sms();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const int64_t grid = std::min<int64_t>(a.N, static_cast<int64_t>(sms) * 8);
  return a.n == 1 ? launch_rows(norm_step_kernel<1>, a, grid, stream)
                  : launch_rows(norm_step_kernel<4>, a, grid, stream);
}

int norm_backward_rows(int64_t N) {
  return static_cast<int>(std::min<int64_t>(N, 2 * static_cast<int64_t>(norm_sms())));
}

cudaError_t launch_norm_step_backward(const NormArgs& a, cudaStream_t stream) {
  const int rows = norm_backward_rows(a.N);
  if (rows <= 0) return cudaErrorInvalidDevice;
  cudaError_t e;
  if (a.X_scale != nullptr)
    e = a.n == 1 ? launch_rows(norm_step_backward_kernel<1, true>, a, rows, stream)
                 : launch_rows(norm_step_backward_kernel<4, true>, a, rows, stream);
  else
    e = a.n == 1 ? launch_rows(norm_step_backward_kernel<1, false>, a, rows, stream)
                 : launch_rows(norm_step_backward_kernel<4, false>, a, rows, stream);
  if (e != cudaSuccess) return e;
  norm_reduce_kernel<<<(norm_partial_floats(a.d) + 31) / 32, 256, 0, stream>>>(a, rows);
  return cudaGetLastError();
}

}  // namespace mhc
