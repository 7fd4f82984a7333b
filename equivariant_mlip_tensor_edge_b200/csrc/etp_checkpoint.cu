// 8-bit activation checkpoints: store and restore (the code is in etp_checkpoint.h).
//
// Both are one pass over memory. Store moves sizeof(T) + 1 + 1/32 bytes a value, restore the same.
#include "etp_checkpoint.h"
#include "etp_internal.h"

namespace etp {
namespace {

constexpr int kThreads = 256;

// rows of whole blocks (cols % 32 == 0) in aligned memory: the array is a run of blocks, 8 lanes to a
// block and 4 values to a lane
template <class T>
__global__ void __launch_bounds__(kThreads) k_store_whole(long long n_vec, bool int8, const T* __restrict__ x,
                                                          uint8_t* __restrict__ q, uint8_t* __restrict__ scale) {
  const long long stride = static_cast<long long>(gridDim.x) * kThreads;
  const long long n_round = (n_vec + 31) & ~31LL;   // whole warps stay together for the shuffles
  for (long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i < n_round; i += stride) {
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (i < n_vec) load_v<T, 4>(x + i * 4, v);
    float m = max_abs(max_abs(v[0], v[1]), max_abs(v[2], v[3]));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = max_abs(m, __shfl_xor_sync(0xffffffffu, m, o));
    const unsigned byte = scale_byte(m, int8);
    if (i < n_vec) {
      reinterpret_cast<unsigned*>(q)[i] = encode4(v, inv_scale(byte), byte == kCkptBad, int8);
      if ((i & 7) == 0) scale[i >> 3] = static_cast<uint8_t>(byte);
    }
  }
}

// any row length: a warp to a block, a lane to a value
template <class T>
__global__ void __launch_bounds__(kThreads) k_store_any(long long rows, int cols, int blocks, bool int8,
                                                        const T* __restrict__ x, uint8_t* __restrict__ q,
                                                        uint8_t* __restrict__ scale) {
  const int lane = threadIdx.x & 31;
  const long long n = rows * blocks, stride = static_cast<long long>(gridDim.x) * (kThreads / 32);
  for (long long b = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); b < n; b += stride) {
    const long long row = b / blocks;
    const int col = static_cast<int>(b - row * blocks) * kCkptBlock + lane;
    const float v = col < cols ? to_f32<T>(x[row * cols + col]) : 0.0f;
    float m = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) m = max_abs(m, __shfl_xor_sync(0xffffffffu, m, o));
    const unsigned byte = scale_byte(m, int8);
    if (col < cols) q[row * cols + col] = static_cast<uint8_t>(encode(v, inv_scale(byte), byte == kCkptBad, int8));
    if (lane == 0) scale[b] = static_cast<uint8_t>(byte);
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
  for (long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i < n_vec; i += stride) {
    float v[4];
    decode4(__ldg(reinterpret_cast<const unsigned*>(q) + i), scale_of(__ldg(scale + (i >> 3))), int8, v);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = held<T>(v[k]);
    store_v<T, 4>(x + i * 4, v);
  }
}

template <class T>
__global__ void __launch_bounds__(kThreads) k_restore_any(long long rows, int cols, int blocks, bool int8,
                                                          const uint8_t* __restrict__ q,
                                                          const uint8_t* __restrict__ scale, T* __restrict__ x) {
  const int lane = threadIdx.x & 31;
  const long long n = rows * blocks, stride = static_cast<long long>(gridDim.x) * (kThreads / 32);
  for (long long b = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); b < n; b += stride) {
    const long long row = b / blocks;
    const int col = static_cast<int>(b - row * blocks) * kCkptBlock + lane;
    if (col < cols)
      x[row * cols + col] = from_f32<T>(held<T>(decode(q[row * cols + col], scale_of(scale[b]), int8)));
  }
}

int grid_for(long long items, int per_block) {
  const long long g = (items + per_block - 1) / per_block;
  return static_cast<int>(g < 148 * 16 ? g : 148 * 16);
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
    k_store_any<T><<<grid_for(rows * blocks, kThreads / 32), kThreads, 0, s>>>(rows, cols, blocks, int8, xt, q, scale);
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
    k_restore_any<T><<<grid_for(rows * blocks, kThreads / 32), kThreads, 0, s>>>(rows, cols, blocks, int8, q, scale, xt);
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
