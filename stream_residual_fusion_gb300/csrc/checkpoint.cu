// checkpoint.cu -- bf16 rows to MXFP8 activation checkpoints and back.
//
// Save reads 2d bytes of a row and writes d + ceil(d / 32); load the reverse. Both are bound by
// memory. One thread per 8 features (a 16-byte bf16 chunk against 8 bytes of codes), so a warp moves
// contiguous runs; the four threads of a block of 32 share its largest magnitude by shuffles.
#include <cuda_runtime.h>

#include <algorithm>

#include "internal.h"
#include "mx8.cuh"

namespace mhc {
namespace {

constexpr int CKP_THREADS = 256;

// One thread per chunk of 8 features; rows padded to whole blocks of four chunks, so that the
// four threads of a block are neighbours. `pc` chunks a padded row, `chunks` of them in the row.
__global__ void __launch_bounds__(CKP_THREADS) save_kernel(const uint4* __restrict__ x,
                                                           uint2* __restrict__ codes,
                                                           uint8_t* __restrict__ scales,
                                                           int64_t total, int chunks, int pc) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * CKP_THREADS;
  for (int64_t i0 = blockIdx.x * static_cast<int64_t>(CKP_THREADS); i0 < total; i0 += step) {
    const int64_t i = i0 + threadIdx.x;
    const int64_t row = i / pc;
    const int c = static_cast<int>(i - row * pc);
    const bool in = i < total && c < chunks;
    const uint4 v = in ? __ldg(x + row * chunks + c) : make_uint4(0u, 0u, 0u, 0u);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    bool odd;
    uint32_t m = finite_max8(w, odd);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const uint32_t e = scale_code_of(m);
    if (in) {
      codes[row * chunks + c] = encode8(w, e, odd);
      if ((c & 3) == 0) scales[row * (pc / 4) + c / 4] = static_cast<uint8_t>(e);
    }
  }
}

__global__ void __launch_bounds__(CKP_THREADS) load_kernel(const uint2* __restrict__ codes,
                                                           const uint8_t* __restrict__ scales,
                                                           uint4* __restrict__ x, int64_t total,
                                                           int chunks, int blocks) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * CKP_THREADS;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(CKP_THREADS) + threadIdx.x; i < total; i += step) {
    const int64_t row = i / chunks;
    const int c = static_cast<int>(i - row * chunks);
    const uint2 v = __ldg(codes + i);
    const float sv = scale_value(__ldg(scales + row * blocks + c / 4));
    const f2 s{sv, sv};
    x[i] = make_uint4(f2_to_bf2(decode2(v.x, s)), f2_to_bf2(decode2(v.x >> 16, s)),
                      f2_to_bf2(decode2(v.y, s)), f2_to_bf2(decode2(v.y >> 16, s)));
  }
}

int ckpt_grid(int64_t work) {
  const int sms = std::max(1, device_info().sms);
  const int64_t blocks = (work + CKP_THREADS - 1) / CKP_THREADS;
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(blocks, static_cast<int64_t>(sms) * 16)));
}

}  // namespace

cudaError_t launch_checkpoint_save(const void* x, void* codes, void* scales, int64_t rows, int d,
                                   cudaStream_t stream) {
  const int chunks = d / 8, pc = (chunks + 3) / 4 * 4;
  const int64_t total = rows * pc;
  save_kernel<<<ckpt_grid(total), CKP_THREADS, 0, stream>>>(static_cast<const uint4*>(x),
                                                            static_cast<uint2*>(codes),
                                                            static_cast<uint8_t*>(scales), total, chunks, pc);
  return cudaGetLastError();
}

cudaError_t launch_checkpoint_load(const void* codes, const void* scales, void* x, int64_t rows, int d,
                                   cudaStream_t stream) {
  const int chunks = d / 8;
  const int64_t total = rows * chunks;
  load_kernel<<<ckpt_grid(total), CKP_THREADS, 0, stream>>>(
      static_cast<const uint2*>(codes), static_cast<const uint8_t*>(scales), static_cast<uint4*>(x), total,
      chunks, (chunks + 3) / 4);
  return cudaGetLastError();
}

}  // namespace mhc
