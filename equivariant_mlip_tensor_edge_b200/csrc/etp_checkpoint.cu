// 8-bit activation checkpoints: store and restore (the code is in etp_checkpoint.h).
//
// Both are one pass over memory. Store moves sizeof(T) + 1 + 1/32 bytes a value, restore the same.
#include "etp_checkpoint.h"

#include <algorithm>

#include "etp_internal.h"

namespace etp {
namespace {

constexpr int kThreads = 256;

// Rows of whole blocks (cols % 32 == 0) in aligned memory: the array is a run of blocks, 8 lanes to a
// block and 4 values to a lane. A thread has kFlight such vectors under way.
constexpr int kFlight = 4;

template <class T>
__global__ void __launch_bounds__(kThreads) k_store_whole(long long n_vec, bool int8, const T* __restrict__ x,
                                                          uint8_t* __restrict__ q, uint8_t* __restrict__ scale) {
  const long long stride = static_cast<long long>(gridDim.x) * kThreads;
  const long long n_round = (n_vec + 31) & ~31LL;   // whole warps stay together for the shuffles
  for (long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i < n_round; i += kFlight * stride) {
    float v[kFlight][4];
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      if (i + k * stride < n_vec) load_v<T, 4>(x + (i + k * stride) * 4, v[k]);
      else v[k][0] = v[k][1] = v[k][2] = v[k][3] = 0.0f;
    }
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const long long at = i + k * stride;
      float m = max_abs(max_abs(v[k][0], v[k][1]), max_abs(v[k][2], v[k][3]));
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) m = max_abs(m, __shfl_xor_sync(0xffffffffu, m, o));
      const unsigned byte = scale_byte(m, int8);
      if (at < n_vec) {
        __stcs(reinterpret_cast<unsigned*>(q) + at, encode4(v[k], inv_scale(byte), byte == kCkptBad, int8));
        if ((at & 7) == 0) scale[at >> 3] = static_cast<uint8_t>(byte);
      }
    }
  }
}

template <class T>
__device__ __forceinline__ float held(float v) {   // the type's finite range; NaN passes
  return v > Limits<T>::max ? Limits<T>::max : v < -Limits<T>::max ? -Limits<T>::max : v;
}

template <class T>
__global__ void __launch_bounds__(kThreads) k_restore_whole(long long n_vec, bool int8, const uint8_t* __restrict__ q,
                                                            const uint8_t* __restrict__ scale, T* __restrict__ x) {
  const long long stride = static_cast<long long>(gridDim.x) * kThreads;
  for (long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i < n_vec; i += kFlight * stride) {
    unsigned codes[kFlight];
    unsigned byte[kFlight];
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const long long at = min(i + k * stride, n_vec - 1);
      codes[k] = __ldg(reinterpret_cast<const unsigned*>(q) + at);
      byte[k] = __ldg(scale + (at >> 3));
    }
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      float v[4];
      decode4(codes[k], scale_of(byte[k]), int8, v);
#pragma unroll
      for (int h = 0; h < 4; ++h) v[h] = held<T>(v[h]);
      if (i + k * stride < n_vec) store_v<T, 4>(x + (i + k * stride) * 4, v);
    }
  }
}

// Any row length: a warp to a block of a row, a lane to a value, four blocks under way. A warp's next
// block is `stride` blocks on, d_row rows and d_block blocks of one: no division.
struct Walk {
  long long row;
  int block;
  __device__ __forceinline__ void next(int d_row, int d_block, int blocks) {
    row += d_row;
    block += d_block;
    if (block >= blocks) {
      block -= blocks;
      ++row;
    }
  }
};

template <class T>
__global__ void __launch_bounds__(kThreads) k_store_any(long long rows, int cols, int blocks, int d_row, int d_block,
                                                        bool int8, const T* __restrict__ x, uint8_t* __restrict__ q,
                                                        uint8_t* __restrict__ scale) {
  const int lane = threadIdx.x & 31;
  const long long first = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  Walk w{first / blocks, static_cast<int>(first % blocks)};
  while (w.row < rows) {
    Walk at[kFlight];
    float v[kFlight];
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      at[k] = w;
      const int col = w.block * kCkptBlock + lane;
      v[k] = w.row < rows && col < cols ? to_f32<T>(x[w.row * cols + col]) : 0.0f;
      w.next(d_row, d_block, blocks);
    }
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      if (at[k].row >= rows) break;
      // as integers the patterns of |x| order like the values, with infinity and NaN on top
      const float m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(v[k]))));
      const unsigned byte = scale_byte(m, int8);
      const int col = at[k].block * kCkptBlock + lane;
      if (col < cols)
        q[at[k].row * cols + col] = static_cast<uint8_t>(encode(v[k], inv_scale(byte), byte == kCkptBad, int8));
      if (lane == 0) scale[at[k].row * blocks + at[k].block] = static_cast<uint8_t>(byte);
    }
  }
}

template <class T>
__global__ void __launch_bounds__(kThreads) k_restore_any(long long rows, int cols, int blocks, int d_row, int d_block,
                                                          bool int8, const uint8_t* __restrict__ q,
                                                          const uint8_t* __restrict__ scale, T* __restrict__ x) {
  const int lane = threadIdx.x & 31;
  const long long first = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  Walk w{first / blocks, static_cast<int>(first % blocks)};
  while (w.row < rows) {
    Walk at[kFlight];
    unsigned code[kFlight], byte[kFlight];
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      at[k] = w;
      const int col = w.block * kCkptBlock + lane;
      const bool here = w.row < rows && col < cols;
      code[k] = here ? q[w.row * cols + col] : 0u;
      byte[k] = here ? scale[w.row * blocks + w.block] : 1u;
      w.next(d_row, d_block, blocks);
    }
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const int col = at[k].block * kCkptBlock + lane;
      if (at[k].row < rows && col < cols)
        x[at[k].row * cols + col] = from_f32<T>(held<T>(decode(code[k], scale_of(byte[k]), int8)));
    }
  }
}

// blocks for so many threads or warps of work, kFlight items to each, up to what is resident twice over
int grid_for(long long items, int per_block) {
  const long long g = (items + static_cast<long long>(per_block) * kFlight - 1) / (static_cast<long long>(per_block) * kFlight);
  return static_cast<int>(std::min<long long>(g, 148 * 16));
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

template <class T>
etp_status store_t(bool int8, long long rows, int cols, const void* x, uint8_t* q, uint8_t* scale, cudaStream_t s) {
  const T* xt = static_cast<const T*>(x);
  const int blocks = (cols + kCkptBlock - 1) / kCkptBlock;
  if (cols % kCkptBlock == 0 && aligned(x, 4 * sizeof(T)) && aligned(q, 4)) {
    const long long n_vec = rows * (cols / 4);
    k_store_whole<T><<<grid_for(n_vec, kThreads), kThreads, 0, s>>>(n_vec, int8, xt, q, scale);
  } else {
    const int grid = grid_for(rows * blocks, kThreads / 32), warps = grid * (kThreads / 32);
    k_store_any<T><<<grid, kThreads, 0, s>>>(rows, cols, blocks, warps / blocks, warps % blocks, int8, xt, q, scale);
  }
  return cuda_status(cudaGetLastError(), "checkpoint store launch");
}

template <class T>
etp_status restore_t(bool int8, long long rows, int cols, const uint8_t* q, const uint8_t* scale, void* x, cudaStream_t s) {
  T* xt = static_cast<T*>(x);
  const int blocks = (cols + kCkptBlock - 1) / kCkptBlock;
  if (cols % kCkptBlock == 0 && aligned(x, 4 * sizeof(T)) && aligned(q, 4)) {
    const long long n_vec = rows * (cols / 4);
    k_restore_whole<T><<<grid_for(n_vec, kThreads), kThreads, 0, s>>>(n_vec, int8, q, scale, xt);
  } else {
    const int grid = grid_for(rows * blocks, kThreads / 32), warps = grid * (kThreads / 32);
    k_restore_any<T><<<grid, kThreads, 0, s>>>(rows, cols, blocks, warps / blocks, warps % blocks, int8, q, scale, xt);
  }
  return cuda_status(cudaGetLastError(), "checkpoint restore launch");
}

}  // namespace

namespace ckpt {

etp_status store(etp_ckpt_format format, etp_dtype dtype, long long rows, int cols, const void* x, uint8_t* q,
                 uint8_t* scale, cudaStream_t s) {
  const bool int8 = format == ETP_CKPT_INT8;
  switch (dtype) {
    case ETP_F32: return store_t<float>(int8, rows, cols, x, q, scale, s);
    case ETP_BF16: return store_t<__nv_bfloat16>(int8, rows, cols, x, q, scale, s);
    default: return store_t<__half>(int8, rows, cols, x, q, scale, s);
  }
}

etp_status restore(etp_ckpt_format format, etp_dtype dtype, long long rows, int cols, const uint8_t* q,
                   const uint8_t* scale, void* x, cudaStream_t s) {
  const bool int8 = format == ETP_CKPT_INT8;
  switch (dtype) {
    case ETP_F32: return restore_t<float>(int8, rows, cols, q, scale, x, s);
    case ETP_BF16: return restore_t<__nv_bfloat16>(int8, rows, cols, q, scale, x, s);
    default: return restore_t<__half>(int8, rows, cols, q, scale, x, s);
  }
}

}  // namespace ckpt
}  // namespace etp
