// 8-bit activation checkpoints: store and restore (the code is in etp_checkpoint.h).
//
// Both are one pass over memory. Store moves sizeof(T) + 1 + 1/32 bytes a value, restore the same.
#include "etp_checkpoint.h"

#include <algorithm>

#include "etp_internal.h"

namespace etp {
namespace {

constexpr int kThreads = 256;

template <class T>
__device__ __forceinline__ float held(float v) {   // the type's finite range; NaN passes
  return v > Limits<T>::max ? Limits<T>::max : v < -Limits<T>::max ? -Limits<T>::max : v;
}

// Aligned rows of whole vectors of 4 (cols % 4 == 0): 8 lanes to a block, a vector to a lane, kFlight
// vectors of a thread under way. A group of 8 lanes goes on by `stride` blocks, some rows
// and d_block blocks of one: no division. Bound by memory: 8000 rows of 2048 float32 stored and fetched in
// 30 us, 85 % of the measured copy rate.
constexpr int kFlight = 4;

struct Steps {
  long long n, stride, d_off;   // blocks in all; blocks and values to a lane group's next block
  int cols, blocks, d_block, wrap;
};

struct Walk {
  long long index, off;         // of the block among all, of its first value
  int block;                    // in its row
  __device__ __forceinline__ void next(const Steps& s) {
    index += s.stride;
    off += s.d_off;
    block += s.d_block;
    if (block >= s.blocks) {
      block -= s.blocks;
      off += s.wrap;
    }
  }
};

// kWhole: rows of whole blocks, one run of them (30 us where the general form takes 34)
template <class T, bool kStore, bool kWhole>
__global__ void __launch_bounds__(kThreads) k_vectors(Steps s, bool int8, T* __restrict__ x, uint8_t* __restrict__ q,
                                                      uint8_t* __restrict__ scale) {
  const int in_block = (threadIdx.x & 7) * 4;
  const long long first = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) >> 3;
  Walk w{first, first * kCkptBlock + in_block, 0};
  if (!kWhole) {
    w.block = static_cast<int>(first % s.blocks);
    w.off = first / s.blocks * s.cols + w.block * kCkptBlock + in_block;
  }
  const unsigned group = 0xffu << (threadIdx.x & 24u);   // the lanes of a block, which end together
  while (w.index < s.n) {
    long long index[kFlight], off[kFlight];
    bool here[kFlight];
    float v[kFlight][4];
    unsigned codes[kFlight], byte[kFlight];
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      index[k] = w.index;
      off[k] = w.off;
      here[k] = w.index < s.n && (kWhole || w.block * kCkptBlock + in_block < s.cols);
      if (kStore) {
        if (here[k]) load_v<T, 4>(x + w.off, v[k]);
        else v[k][0] = v[k][1] = v[k][2] = v[k][3] = 0.0f;
      } else {
        codes[k] = here[k] ? __ldcs(reinterpret_cast<const unsigned*>(q + w.off)) : 0u;
        byte[k] = here[k] ? __ldg(scale + w.index) : 1u;
      }
      if (kWhole) {
        w.index += s.stride;
        w.off += s.stride * kCkptBlock;
      } else {
        w.next(s);
      }
    }
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      if (kStore) {
        float m = max_abs(max_abs(v[k][0], v[k][1]), max_abs(v[k][2], v[k][3]));
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) m = max_abs(m, __shfl_xor_sync(group, m, o));
        const unsigned b = scale_byte(m, int8);
        if (here[k]) {
          __stcs(reinterpret_cast<unsigned*>(q + off[k]), encode4(v[k], inv_scale(b), b == kCkptBad, int8));
          if (in_block == 0) scale[index[k]] = static_cast<uint8_t>(b);
        }
      } else if (here[k]) {
        decode4(codes[k], scale_of(byte[k]), int8, v[k]);
#pragma unroll
        for (int h = 0; h < 4; ++h) v[k][h] = held<T>(v[k][h]);
        store_v<T, 4>(x + off[k], v[k]);
      }
    }
  }
}

template <class T, bool kStore>
void launch_vectors(bool int8, long long rows, int cols, int blocks, T* x, uint8_t* q, uint8_t* scale, cudaStream_t s) {
  // up to twice what is resident
  const long long per = kThreads / 8 * kFlight;
  const int grid = static_cast<int>(std::min<long long>((rows * blocks + per - 1) / per, 148 * 16));
  Steps p;
  p.n = rows * blocks;
  p.stride = grid * (kThreads / 8);
  p.cols = cols;
  p.blocks = blocks;
  p.d_block = static_cast<int>(p.stride % blocks);
  p.d_off = p.stride / blocks * cols + static_cast<long long>(p.d_block) * kCkptBlock;
  p.wrap = static_cast<int>(cols - static_cast<long long>(blocks) * kCkptBlock);
  if (cols % kCkptBlock == 0) k_vectors<T, kStore, true><<<grid, kThreads, 0, s>>>(p, int8, x, q, scale);
  else k_vectors<T, kStore, false><<<grid, kThreads, 0, s>>>(p, int8, x, q, scale);
}

// Any row length and alignment. A block takes a run of up to kUnit values, whole rows or a part of one
// that starts at a block's first value, through shared memory: outside 16 bytes at a time, inside value by
// value, as they are not aligned. Bound by the instructions of the single accesses and, between a
// unit's arrival and its leaving, by how many blocks an SM has under way: 16411 rows of 1153 bfloat16
// stored and fetched in 48 us, 37 % of the copy rate (units of 4096 values and 256 threads: 64 us; a lane
// to a value: 90 us; single accesses to global memory: 123 us).
constexpr int kUnit = 6144, kUnitThreads = 128;

struct Units {
  long long n, rows;
  int cols, blocks;          // of a row
  int unit_rows, seg, per_row;   // rows of a unit, or columns of one of a row's per_row units
  unsigned blocks_m;         // division by a row's blocks, for the numbers of a unit
};

// Bytes [from, from + n) of a unit, between global memory and shared memory of the same alignment.
template <bool kIn>
__device__ __forceinline__ void move_bytes(char* shared, char* global, int n) {
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(global) & 15u), head = min((16 - off) & 15, n);
  const int body = (n - head) >> 4, tail = n - head - (body << 4);
  char* s = shared + off;
  for (int i = threadIdx.x; i < body; i += kUnitThreads) {
    uint4* g = reinterpret_cast<uint4*>(global + head) + i;
    uint4* t = reinterpret_cast<uint4*>(s + head) + i;
    if (kIn) *t = __ldcs(g);
    else __stcs(g, *t);
  }
  if (threadIdx.x < head + tail) {
    const int i = threadIdx.x < head ? threadIdx.x : n - tail + threadIdx.x - head;
    if (kIn) s[i] = global[i];
    else global[i] = s[i];
  }
}

template <class T, bool kStore, bool kInt8, int kLanes>
__global__ void __launch_bounds__(kUnitThreads, 6) k_units(Units p, T* x, uint8_t* q, uint8_t* scale) {
  __shared__ __align__(16) char values[kUnit * sizeof(T) + 16];
  __shared__ __align__(16) char codes[kUnit + 32];
  __shared__ __align__(16) char scales[kUnit + 16];
  // kLanes: that share a block of 32, or a shorter row
  constexpr int per_warp = 32 / kLanes;
  const int lane = threadIdx.x & 31, in_block = lane & (kLanes - 1), first = lane / kLanes;
  for (long long u = blockIdx.x; u < p.n; u += gridDim.x) {
    const long long group = p.per_row > 1 ? u / p.per_row : u, row0 = group * p.unit_rows;
    const int c0 = static_cast<int>(u - group * p.per_row) * p.seg;
    const int nr = static_cast<int>(min(static_cast<long long>(p.unit_rows), p.rows - row0)), nc = min(p.seg, p.cols - c0);
    const int blocks = (nc + kCkptBlock - 1) / kCkptBlock, items = nr * blocks, n = nr * nc;
    T* gx = x + row0 * p.cols + c0;
    uint8_t* gq = q + row0 * p.cols + c0;
    uint8_t* gs = scale + row0 * p.blocks + c0 / kCkptBlock;
    T* sx = reinterpret_cast<T*>(values + (reinterpret_cast<uintptr_t>(gx) & 15u));
    uint8_t* sq = reinterpret_cast<uint8_t*>(codes) + (reinterpret_cast<uintptr_t>(gq) & 15u);
    uint8_t* ss = reinterpret_cast<uint8_t*>(scales) + (reinterpret_cast<uintptr_t>(gs) & 15u);
    if (kStore) {
      move_bytes<true>(values, reinterpret_cast<char*>(gx), n * static_cast<int>(sizeof(T)));
    } else {
      move_bytes<true>(codes, reinterpret_cast<char*>(gq), n);
      move_bytes<true>(scales, reinterpret_cast<char*>(gs), items);
    }
    __syncthreads();
    // Two blocks to a lane, 4 values of each (or one short row of at most 4 to each): 4 lanes' values in
    // 32 bytes keep the accesses of a warp at two a bank.
    const int end = (items + 2 * per_warp - 1) / (2 * per_warp);
    for (int it = threadIdx.x >> 5; it < end; it += kUnitThreads / 32) {
      int at[2], count[2];
      float v[2][4];
      unsigned codes4[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int b = (it * 2 + h) * per_warp + first;
        const int r = p.per_row > 1 ? 0 : p.blocks_m ? static_cast<int>(__umulhi(b, p.blocks_m)) : b;
        const int col = (b - r * blocks) * kCkptBlock + in_block * 4;
        at[h] = r * nc + col;
        count[h] = b < items ? min(max(nc - col, 0), 4) : 0;
        if (kStore) {
          if (count[h] == 4) {
#pragma unroll
            for (int k = 0; k < 4; ++k) v[h][k] = to_f32<T>(sx[at[h] + k]);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) v[h][k] = k < count[h] ? to_f32<T>(sx[at[h] + k]) : 0.0f;
          }
        } else if (count[h] > 0) {
          // what stands behind the last value of a row is the next one's, or room in shared memory
          const uint8_t* from = sq + at[h];
          codes4[h] = from[0] | from[1] << 8 | from[2] << 16 | static_cast<unsigned>(from[3]) << 24;
          decode4(codes4[h], scale_of(ss[b]), kInt8, v[h]);
        }
      }
      if (kStore) {
        float m[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) m[h] = max_abs(max_abs(v[h][0], v[h][1]), max_abs(v[h][2], v[h][3]));
#pragma unroll
        for (int o = 1; o < kLanes; o *= 2)
#pragma unroll
          for (int h = 0; h < 2; ++h) m[h] = max_abs(m[h], __shfl_xor_sync(0xffffffffu, m[h], o));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const unsigned byte = scale_byte(m[h], kInt8);
          codes4[h] = encode4(v[h], inv_scale(byte), byte == kCkptBad, kInt8);
          const int b = (it * 2 + h) * per_warp + first;
          if (in_block == 0 && b < items) ss[b] = static_cast<uint8_t>(byte);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (count[h] == 4) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (kStore) sq[at[h] + k] = static_cast<uint8_t>(codes4[h] >> (8 * k));
            else sx[at[h] + k] = from_f32<T>(held<T>(v[h][k]));
          }
        } else {
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            if (k >= count[h]) continue;
            if (kStore) sq[at[h] + k] = static_cast<uint8_t>(codes4[h] >> (8 * k));
            else sx[at[h] + k] = from_f32<T>(held<T>(v[h][k]));
          }
        }
      }
    }
    __syncthreads();
    if (kStore) {
      move_bytes<false>(codes, reinterpret_cast<char*>(gq), n);
      move_bytes<false>(scales, reinterpret_cast<char*>(gs), items);
    } else {
      move_bytes<false>(values, reinterpret_cast<char*>(gx), n * static_cast<int>(sizeof(T)));
    }
    __syncthreads();
  }
}

template <class T, bool kStore>
void launch_units(bool int8, long long rows, int cols, int blocks, T* x, uint8_t* q, uint8_t* scale, cudaStream_t s) {
  Units p;
  p.rows = rows;
  p.cols = cols;
  p.blocks = blocks;
  p.per_row = (cols - 1) / kUnit + 1;
  p.seg = p.per_row > 1 ? kUnit : cols;
  p.unit_rows = p.per_row > 1 ? 1 : kUnit / cols;
  p.n = (rows + p.unit_rows - 1) / p.unit_rows * p.per_row;
  p.blocks_m = blocks > 1 ? static_cast<unsigned>(((1ULL << 32) + blocks - 1) / blocks) : 0u;
  const int grid = static_cast<int>(std::min<long long>(p.n, 148 * 16));
  auto run = [&](auto kernel) { kernel<<<grid, kUnitThreads, 0, s>>>(p, x, q, scale); };
  if (int8) cols > 4 ? run(k_units<T, kStore, true, 8>) : run(k_units<T, kStore, true, 1>);
  else cols > 4 ? run(k_units<T, kStore, false, 8>) : run(k_units<T, kStore, false, 1>);
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

template <class T, bool kStore>
etp_status run(bool int8, long long rows, int cols, void* x, uint8_t* q, uint8_t* scale, cudaStream_t s) {
  T* xt = static_cast<T*>(x);
  const int blocks = (cols - 1) / kCkptBlock + 1;   // cols > 0; cols + 31 may not fit an int
  if (cols % 4 == 0 && aligned(x, 4 * sizeof(T)) && aligned(q, 4))
    launch_vectors<T, kStore>(int8, rows, cols, blocks, xt, q, scale, s);
  else
    launch_units<T, kStore>(int8, rows, cols, blocks, xt, q, scale, s);
  return cuda_status(cudaGetLastError(), kStore ? "checkpoint store launch" : "checkpoint restore launch");
}

template <bool kStore>
etp_status run_type(etp_ckpt_format format, etp_dtype dtype, long long rows, int cols, void* x, uint8_t* q,
                    uint8_t* scale, cudaStream_t s) {
  const bool int8 = format == ETP_CKPT_INT8;
  switch (dtype) {
    case ETP_F32: return run<float, kStore>(int8, rows, cols, x, q, scale, s);
    case ETP_BF16: return run<__nv_bfloat16, kStore>(int8, rows, cols, x, q, scale, s);
    default: return run<__half, kStore>(int8, rows, cols, x, q, scale, s);
  }
}

}  // namespace

namespace ckpt {

etp_status store(etp_ckpt_format format, etp_dtype dtype, long long rows, int cols, const void* x, uint8_t* q,
                 uint8_t* scale, cudaStream_t s) {
  return run_type<true>(format, dtype, rows, cols, const_cast<void*>(x), q, scale, s);
}

etp_status restore(etp_ckpt_format format, etp_dtype dtype, long long rows, int cols, const uint8_t* q,
                   const uint8_t* scale, void* x, cudaStream_t s) {
  return run_type<false>(format, dtype, rows, cols, x, const_cast<uint8_t*>(q), const_cast<uint8_t*>(scale), s);
}

}  // namespace ckpt
}  // namespace etp
