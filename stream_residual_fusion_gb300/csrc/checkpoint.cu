// checkpoint.cu -- bf16 rows to MXFP8 activation checkpoints and back.
//
// Save reads 2d bytes of a row and writes d + ceil(d / 32); load the reverse. Both are bound by
// memory. One thread per 8 features (a 16-byte bf16 chunk against 8 bytes of codes), so a warp moves
// contiguous runs; the four threads of a block of 32 share its largest magnitude by shuffles. Each
// thread has CKP_EACH chunks in flight. Rows of whole blocks (d a multiple of 32) are one long run of
// chunks; others are walked row by row, padded to whole blocks of four chunks.
//
// Save was bound by integer instructions (ALU pipe 89% busy, 4-byte halves taken apart for the
// maximum) until the maximum went to two half words at a time and infinities and NaNs to a branch of
// their own. 8-bit checkpoints of 32,768 x 4 x 5,120 and 32,768 x 5,120 features, saved and loaded:
// 593 us from 691, the time in which a plain copy moves the same bytes.
#include <cuda_runtime.h>

#include "internal.h"
#include "mx8.cuh"

namespace mhc {
namespace {

constexpr int CKP_THREADS = 256;
constexpr int CKP_EACH = 4;

// Chunk i of the padded rows: its row and its place c in the row (`in`: it is one of the row's own).
struct Chunk {
  int64_t row;
  int c;
  bool in;
};
// `pc` chunks a padded row, `chunks` of them the row's own; WHOLE: the same, rows need not be told apart.
template <bool WHOLE>
__device__ __forceinline__ Chunk chunk_at(int64_t i, int64_t total, int chunks, int pc) {
  if (WHOLE) return Chunk{0, 0, i < total};
  Chunk k;
  if (total <= 0x7fffffff) k.row = static_cast<uint32_t>(i) / static_cast<uint32_t>(pc);   // a far cheaper division
  else k.row = i / pc;
  k.c = static_cast<int>(i - k.row * pc);
  k.in = i < total && k.c < chunks;
  return k;
}

template <bool WHOLE>
__global__ void __launch_bounds__(CKP_THREADS) save_kernel(const uint4* __restrict__ x,
                                                           uint2* __restrict__ codes,
                                                           uint8_t* __restrict__ scales,
                                                           int64_t total, int chunks, int pc) {
  const int64_t i0 = blockIdx.x * static_cast<int64_t>(CKP_THREADS * CKP_EACH) + threadIdx.x;
  const int lane = threadIdx.x & 31;
  uint4 v[CKP_EACH];
  Chunk k[CKP_EACH];
#pragma unroll
  for (int q = 0; q < CKP_EACH; ++q) {
    const int64_t i = i0 + q * CKP_THREADS;
    k[q] = chunk_at<WHOLE>(i, total, chunks, pc);
    v[q] = k[q].in ? __ldcs(x + (WHOLE ? i : k[q].row * chunks + k[q].c)) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int q = 0; q < CKP_EACH; ++q) {
    const int64_t i = i0 + q * CKP_THREADS;
    const uint32_t w[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
    uint32_t m = max_halves8(w);
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
    m = max_of_halves(m);
    uint2 c;
    uint32_t e;
    if (__any_sync(0xffffffffu, m >= 0x7f80u)) {   // rare: an infinity or a NaN in one of the warp's blocks
      m = finite_max_halves8(w);
      m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
      e = scale_code_of(max_of_halves(m));
      c = encode8<true>(w, e);
    } else {
      e = scale_code_of(m);
      c = encode8<false>(w, e);
    }
    if (k[q].in) __stcs(codes + (WHOLE ? i : k[q].row * chunks + k[q].c), c);
    if (WHOLE) {   // the warp's eight scale codes are neighbours: two words
      uint32_t p = e | (__shfl_down_sync(0xffffffffu, e, 4) << 8);
      p |= __shfl_down_sync(0xffffffffu, p, 8) << 16;
      const int64_t b = i / 4;
      if ((lane & 15) == 0 && i + 15 < total) {
        *reinterpret_cast<uint32_t*>(scales + b) = p;
      } else if ((lane & 3) == 0 && i - (lane & 15) + 15 >= total && k[q].in) {   // the last, partial word
        scales[b] = static_cast<uint8_t>(e);
      }
    } else if (k[q].in && (k[q].c & 3) == 0) {
      scales[k[q].row * (pc / 4) + k[q].c / 4] = static_cast<uint8_t>(e);
    }
  }
}

template <bool WHOLE>
__global__ void __launch_bounds__(CKP_THREADS) load_kernel(const uint2* __restrict__ codes,
                                                           const uint8_t* __restrict__ scales,
                                                           uint4* __restrict__ x, int64_t total, int chunks,
                                                           int pc) {
  const int64_t i0 = blockIdx.x * static_cast<int64_t>(CKP_THREADS * CKP_EACH) + threadIdx.x;
  uint2 v[CKP_EACH];
  uint32_t e[CKP_EACH];
  int64_t at[CKP_EACH];
#pragma unroll
  for (int q = 0; q < CKP_EACH; ++q) {
    const int64_t i = i0 + q * CKP_THREADS;
    const Chunk k = chunk_at<WHOLE>(i, total, chunks, pc);
    at[q] = k.in ? (WHOLE ? i : k.row * chunks + k.c) : -1;
    if (k.in) {
      v[q] = __ldcs(codes + at[q]);
      e[q] = __ldg(scales + (WHOLE ? i / 4 : k.row * (pc / 4) + k.c / 4));
    }
  }
#pragma unroll
  for (int q = 0; q < CKP_EACH; ++q) {
    if (at[q] < 0) continue;
    const float sv = scale_value(e[q]);
    const f2 s{sv, sv};
    __stcs(x + at[q], make_uint4(f2_to_bf2(decode2(v[q].x, s)), f2_to_bf2(decode2(v[q].x >> 16, s)),
                                 f2_to_bf2(decode2(v[q].y, s)), f2_to_bf2(decode2(v[q].y >> 16, s))));
  }
}

unsigned ckpt_blocks(int64_t total) {
  return static_cast<unsigned>((total + CKP_THREADS * CKP_EACH - 1) / (CKP_THREADS * CKP_EACH));
}

}  // namespace

cudaError_t launch_checkpoint_save(const void* x, void* codes, void* scales, int64_t rows, int d,
                                   cudaStream_t stream) {
  const int chunks = d / 8, pc = (chunks + 3) / 4 * 4;
  const int64_t total = rows * pc;
  auto run = [&](auto kernel) {
    kernel<<<ckpt_blocks(total), CKP_THREADS, 0, stream>>>(static_cast<const uint4*>(x), static_cast<uint2*>(codes),
                                                           static_cast<uint8_t*>(scales), total, chunks, pc);
    return cudaGetLastError();
  };
  return pc == chunks ? run(save_kernel<true>) : run(save_kernel<false>);
}

cudaError_t launch_checkpoint_load(const void* codes, const void* scales, void* x, int64_t rows, int d,
                                   cudaStream_t stream) {
  const int chunks = d / 8, pc = (chunks + 3) / 4 * 4;
  const int64_t total = rows * pc;
  auto run = [&](auto kernel) {
    kernel<<<ckpt_blocks(total), CKP_THREADS, 0, stream>>>(static_cast<const uint2*>(codes),
                                                           static_cast<const uint8_t*>(scales),
                                                           static_cast<uint4*>(x), total, chunks, pc);
    return cudaGetLastError();
  };
  return pc == chunks ? run(load_kernel<true>) : run(load_kernel<false>);
}

}  // namespace mhc
