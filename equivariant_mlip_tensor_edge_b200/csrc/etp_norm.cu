// Group norm with an activation on node rows, channels last, forward and backward.
//
// Row n holds components (l, m) = 0 .. (L+1)^2 - 1 of C channels each. A structure is a run of rows
// [node_ptr[s], node_ptr[s+1]); a group is C / G neighbouring channels. Over the rows of a structure,
// the channels of a group and the components of a rank:
//
//   mu = mean x (l = 0 only; a mean of l > 0 is not invariant under rotations),
//   r_l = 1 / sqrt(mean (x - mu)^2 + eps),   xhat = (x - mu) r_l,
//   y_lm = xhat_lm w_l + (l = 0) b,          out_lm = y_lm f(y_0),  f = 1 or the logistic function:
//
// SiLU on the scalars and the same channel's gate on the other ranks. Backward, with g = dL/dout:
//
//   dy_lm = g_lm f,  dy_0 += f' sum_lm g_lm y_lm,   dw_l = sum dy xhat,  db = sum dy_0,   h = w dy,
//   dx = r_l (h - xhat mean(h xhat) - (l = 0) mean(h)).
//
// Either direction needs a structure's sums before its first output: two sweeps over the rows. One
// cooperative launch does both. Each block owns a run of rows; a structure inside one block's rows is
// swept twice by that block alone, and one that crosses blocks (two at most for a block: the one that
// reaches in from before and the one that goes on behind) leaves partial sums, which meet after the
// grid barrier. Sums are kept in 64 bits: mu and the mean square cancel where mu is far larger than
// the spread. Every sum has one order, so equal calls give equal bits.
//
// A thread holds V neighbouring channels (V = 4 where channels and group size divide by 4, else 1)
// and walks a row's components, so a component is one coalesced access for the threads of a row and
// the gate of a channel stays in its thread.
#include <cooperative_groups.h>

#include "etp_checkpoint.h"
#include "etp_internal.h"
#include "etp_norm.h"

namespace cg = cooperative_groups;

namespace etp {
namespace norm {
namespace {

constexpr int kThreads = 256;

struct Shape {
  int n_nodes, n_structs, rows;   // rows: a block's share
  int channels, groups, cg;       // cg: channels of a group
  int cv, rp;                     // vectors of a row's component; rows a block reads side by side
  const int* ptr;                 // NULL: one structure of all rows
};

__device__ __forceinline__ int clamp_row(const Shape& s, int v) { return min(max(v, 0), s.n_nodes); }
__device__ __forceinline__ int begin_of(const Shape& s, int i) { return s.ptr ? clamp_row(s, __ldg(s.ptr + i)) : 0; }
__device__ __forceinline__ int end_of(const Shape& s, int i) {
  return s.ptr ? clamp_row(s, __ldg(s.ptr + i + 1)) : s.n_nodes;
}

// Number of structures that end at or before row r, by the whole block: every round probes up to
// kThreads places of the remaining range.
__device__ int ended_by(const Shape& s, int r) {
  int lo = 0, hi = s.n_structs;
  while (lo < hi) {
    const int step = (hi - lo + kThreads - 1) / kThreads;
    const long long p = lo + static_cast<long long>(threadIdx.x) * step;
    const int c = __syncthreads_count(p < hi && end_of(s, static_cast<int>(p)) <= r);
    if (c == 0) break;
    if (static_cast<long long>(lo) + static_cast<long long>(c) * step < hi) hi = lo + c * step;
    lo = lo + (c - 1) * step + 1;
  }
  return lo;
}

// What a block has to do: rows [r0, r1); structures [first, last) lie whole inside; head reaches in
// from before or past the end on both sides, tail starts inside and goes on behind.
struct Span {
  int r0, r1, first, last;
  int head, head_a, head_b, head_slot;   // structure (-1: none), its rows in the block, partial slot
  int tail, tail_a;
};

__device__ Span span_of(const Shape& s) {
  Span w;
  w.r0 = min(static_cast<long long>(blockIdx.x) * s.rows, static_cast<long long>(s.n_nodes));
  w.r1 = min(w.r0 + s.rows, s.n_nodes);
  const int a = ended_by(s, w.r0), b = ended_by(s, w.r1);
  w.head = w.tail = -1;
  w.head_a = w.head_b = w.head_slot = w.tail_a = 0;
  w.first = a;
  w.last = b;
  if (a < s.n_structs) {
    const int lo = begin_of(s, a), hi = end_of(s, a);
    if (lo < w.r1 && (lo < w.r0 || hi > w.r1)) {
      w.head = a;
      w.head_a = max(lo, w.r0);
      w.head_b = min(hi, w.r1);
      w.head_slot = lo < w.r0 ? 0 : 1;
      w.first = a + 1;
    }
  }
  if (b < s.n_structs && b != w.head) {
    const int lo = begin_of(s, b);
    if (lo < w.r1) {
      w.tail = b;
      w.tail_a = max(lo, w.r0);
    }
  }
  return w;
}

// ---------------------------------------------------------------- sums over a block

// acc[q][thread] -> sum[q * groups + g], over the threads of a group's channels in thread order.
template <int Q>
__device__ void sum_groups(const Shape& s, double (&acc)[Q][kThreads], double* red, double* sum) {
  const int nq = Q * s.groups, cvg = s.cv / s.groups, n = s.rp * cvg;
  int parts = 1;
  while (parts < 32 && nq * parts * 2 <= kThreads && parts < n) parts *= 2;
  __syncthreads();
  for (int base = 0; base < nq; base += kThreads / parts) {
    const int i = base + threadIdx.x / parts, part = threadIdx.x % parts;
    double t = 0.0;
    if (i < nq) {
      const int q = i / s.groups, g = i - q * s.groups;
      for (int k = part; k < n; k += parts) {
        const int r = k / cvg;
        t += acc[q][r * s.cv + g * cvg + (k - r * cvg)];
      }
    }
    red[threadIdx.x] = t;
    __syncthreads();
    const int j = base + threadIdx.x;
    if (threadIdx.x < kThreads / parts && j < nq) {
      t = 0.0;
      for (int k = 0; k < parts; ++k) t += red[threadIdx.x * parts + k];
      sum[j] = t;
    }
    __syncthreads();
  }
}

// sum[i] = sum over the blocks that hold rows [a, b) of one structure of their partials, in block order
__device__ void gather_partials(const Shape& s, const double* part, int nq, int a, int b, double* red, double* sum) {
  const int c0 = a / s.rows, c1 = (b - 1) / s.rows;
  int parts = 1;
  while (parts < 32 && nq * parts * 2 <= kThreads) parts *= 2;
  __syncthreads();
  for (int base = 0; base < nq; base += kThreads / parts) {
    // neighbouring threads read neighbouring sums of one block
    const int w = kThreads / parts, i = base + threadIdx.x % w, p = threadIdx.x / w;
    double t = 0.0;
    if (i < nq)
      for (int c = c0 + p; c <= c1; c += parts) t += part[(static_cast<size_t>(c) * 2 + (c == c0 ? 1 : 0)) * nq + i];
    red[threadIdx.x] = t;
    __syncthreads();
    if (threadIdx.x < w && i < nq) {
      t = 0.0;
      for (int k = 0; k < parts; ++k) t += red[k * w + threadIdx.x];
      sum[i] = t;
    }
    __syncthreads();
  }
}

__device__ __forceinline__ float logistic(float t) { return __fdividef(1.0f, 1.0f + __expf(-t)); }

// ---------------------------------------------------------------- forward

struct FwdArgs {
  Shape s;
  const void* x;
  const float *weight, *bias;
  float eps;
  int act, zero_rest;
  void* out;
  float* stats;
  uint8_t *q, *scale;   // the checkpoint of x, or NULL
  int int8;
  double* part;
};

template <int V>
__device__ __forceinline__ void load_affine(const float* p, int col, float fill, float (&v)[V]) {
#pragma unroll
  for (int k = 0; k < V; ++k) v[k] = p ? __ldg(p + col + k) : fill;
}

template <class T, int L, int V>
struct Fwd {
  static constexpr int K = (L + 1) * (L + 1), Q = L + 2;
  static constexpr int kLanes = kCkptBlock / V;   // threads that share a checkpoint block

  // sums of rows [a, b): sum[0] = sum x (l = 0), sum[1 + l] = sum x^2
  static __device__ void sums(const FwdArgs& p, int a, int b, double (&acc)[Q][kThreads], double* red, double* sum) {
    const Shape& s = p.s;
    const int row = threadIdx.x / s.cv, col = (threadIdx.x - row * s.cv) * V;
    double t[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) t[q] = 0.0;
    if (row < s.rp) {
      const T* base = static_cast<const T*>(p.x) + col;
      for (int n = a + row; n < b; n += s.rp) {
        const T* xr = base + static_cast<size_t>(n) * K * s.channels;
        float v[K][V];
#pragma unroll
        for (int m = 0; m < K; ++m) load_v<T, V>(xr + m * s.channels, v[m]);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const double d = v[0][k];
          t[0] += d;
          t[1] = fma(d, d, t[1]);
        }
#pragma unroll
        for (int l = 1; l <= L; ++l) {
          // no cancellation here: a row's squares are added in 32 bits
          float u = 0.0f;
#pragma unroll
          for (int m = l * l; m < (l + 1) * (l + 1); ++m)
#pragma unroll
            for (int k = 0; k < V; ++k) u = fmaf(v[m][k], v[m][k], u);
          t[1 + l] += u;
        }
      }
    }
#pragma unroll
    for (int q = 0; q < Q; ++q) acc[q][threadIdx.x] = t[q];
    sum_groups<Q>(s, acc, red, sum);
  }

  // statistics of a structure of n rows from its sums, to st[Q * groups] (mu, r_0 .. r_L)
  static __device__ void finish(const FwdArgs& p, int structure, int n, bool write, const double* sum, float* st) {
    const int G = p.s.groups;
    for (int i = threadIdx.x; i < Q * G; i += kThreads) {
      const int q = i / G, g = i - q * G;
      float v;
      if (q == 0) {
        v = static_cast<float>(sum[g] / (static_cast<double>(n) * p.s.cg));
      } else {
        const int l = q - 1;
        const double size = static_cast<double>(n) * p.s.cg * (2 * l + 1);
        double var = sum[i] / size;
        if (l == 0) {
          const double mu = sum[g] / size;
          var = var - mu * mu;
          if (var < 0.0) var = 0.0;
        }
        v = static_cast<float>(1.0 / sqrt(var + static_cast<double>(p.eps)));
      }
      st[i] = v;
      if (write) p.stats[static_cast<size_t>(structure) * Q * G + i] = v;
    }
    __syncthreads();
  }

  static __device__ __forceinline__ void keep(const FwdArgs& p, int n, int m, int col, const float (&v)[V]) {
    unsigned top = 0;
#pragma unroll
    for (int k = 0; k < V; ++k) top = max(top, abs_bits(v[k]));
    // the lanes of a block hold the same row, so they are here together
    const unsigned lane = threadIdx.x & 31;
    const unsigned mask = kLanes == 32 ? 0xffffffffu : 0xffu << (lane & 24u);
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) top = max(top, __shfl_xor_sync(mask, top, o));
    const unsigned byte = scale_byte(top, p.int8);
    const size_t at = (static_cast<size_t>(n) * K + m) * p.s.channels + col;
    if constexpr (V == 4) *reinterpret_cast<unsigned*>(p.q + at) = encode4(v, inv_scale(byte), byte == kCkptBad, p.int8);
    else p.q[at] = static_cast<uint8_t>(encode(v[0], inv_scale(byte), byte == kCkptBad, p.int8));
    if ((lane & (kLanes - 1)) == 0) p.scale[at / kCkptBlock] = static_cast<uint8_t>(byte);
  }

  static __device__ void apply(const FwdArgs& p, int a, int b, const float* st) {
    const Shape& s = p.s;
    const int row = threadIdx.x / s.cv, col = (threadIdx.x - row * s.cv) * V;
    if (row >= s.rp) return;
    const int g = col / s.cg;
    float w[L + 1][V], bias[V];
    load_affine<V>(p.bias, col, 0.0f, bias);
    const float mu = st[g];
#pragma unroll
    for (int l = 0; l <= L; ++l) {
      load_affine<V>(p.weight ? p.weight + l * s.channels : nullptr, col, 1.0f, w[l]);
      const float r = st[(1 + l) * s.groups + g];
#pragma unroll
      for (int k = 0; k < V; ++k) w[l][k] *= l == 0 ? 1.0f : r;
    }
    const float r0 = st[s.groups + g];
    for (int n = a + row; n < b; n += s.rp) {
      const size_t at = static_cast<size_t>(n) * K * s.channels + col;
      const T* xr = static_cast<const T*>(p.x) + at;
      T* yr = static_cast<T*>(p.out) + at;
      float v[K][V], f[V];
#pragma unroll
      for (int m = 0; m < K; ++m) load_v<T, V>(xr + m * s.channels, v[m]);
      if (p.q) {
#pragma unroll
        for (int m = 0; m < K; ++m) keep(p, n, m, col, v[m]);
      }
#pragma unroll
      for (int k = 0; k < V; ++k) {
        v[0][k] = fmaf((v[0][k] - mu) * r0, w[0][k], bias[k]);
        f[k] = p.act ? logistic(v[0][k]) : 1.0f;
        v[0][k] *= f[k];
      }
      store_v<T, V>(yr, v[0]);
#pragma unroll
      for (int l = 1; l <= L; ++l)
#pragma unroll
        for (int m = l * l; m < (l + 1) * (l + 1); ++m) {
#pragma unroll
          for (int k = 0; k < V; ++k) v[m][k] = v[m][k] * w[l][k] * f[k];
          store_v<T, V>(yr + m * s.channels, v[m]);
        }
    }
  }

  // rows of the block's share that belong to no structure: their checkpoint, and zeros where asked for
  static __device__ void rest(const FwdArgs& p, int a, int b) {
    const Shape& s = p.s;
    const int row = threadIdx.x / s.cv, col = (threadIdx.x - row * s.cv) * V;
    if (row >= s.rp || (!p.q && !p.zero_rest)) return;
    for (int n = a + row; n < b; n += s.rp)
      for (int m = 0; m < K; ++m) {
        const size_t at = (static_cast<size_t>(n) * K + m) * s.channels + col;
        float v[V];
        if (p.q) {
          load_v<T, V>(static_cast<const T*>(p.x) + at, v);
          keep(p, n, m, col, v);
        }
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = 0.0f;
        if (p.zero_rest) store_v<T, V>(static_cast<T*>(p.out) + at, v);
      }
  }
};

template <class T, int L, int V>
__global__ void __launch_bounds__(kThreads) k_norm_fwd(FwdArgs p) {
  using F = Fwd<T, L, V>;
  constexpr int Q = F::Q;
  __shared__ double acc[Q][kThreads];
  __shared__ double red[kThreads];
  __shared__ double sum[Q * kMaxGroups];
  __shared__ float st[Q * kMaxGroups];
  const Shape& s = p.s;
  const int nq = Q * s.groups;
  const Span w = span_of(s);
  double* mine = p.part + static_cast<size_t>(blockIdx.x) * 2 * nq;
  if (w.head >= 0) {
    F::sums(p, w.head_a, w.head_b, acc, red, sum);
    for (int i = threadIdx.x; i < nq; i += kThreads) mine[w.head_slot * nq + i] = sum[i];
    __syncthreads();
  }
  if (w.tail >= 0) {
    F::sums(p, w.tail_a, w.r1, acc, red, sum);
    for (int i = threadIdx.x; i < nq; i += kThreads) mine[nq + i] = sum[i];
    __syncthreads();
  }
  for (int i = w.first; i < w.last; ++i) {
    const int a = max(begin_of(s, i), w.r0), b = min(end_of(s, i), w.r1);
    if (a >= b) continue;
    F::sums(p, a, b, acc, red, sum);
    F::finish(p, i, b - a, true, sum, st);
    F::apply(p, a, b, st);
    __syncthreads();
  }
  // structures without rows have zero statistics
  if (s.ptr)
    for (long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i < s.n_structs;
         i += static_cast<long long>(gridDim.x) * kThreads)
      if (begin_of(s, static_cast<int>(i)) >= end_of(s, static_cast<int>(i)))
        for (int k = 0; k < nq; ++k) p.stats[i * nq + k] = 0.0f;
  if (s.ptr) {
    F::rest(p, w.r0, min(w.r1, begin_of(s, 0)));
    F::rest(p, max(w.r0, end_of(s, s.n_structs - 1)), w.r1);
  }
  if (gridDim.x > 1) cg::this_grid().sync();
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    const int i = k ? w.tail : w.head;
    if (i < 0) continue;
    const int lo = begin_of(s, i), hi = end_of(s, i);
    gather_partials(s, p.part, nq, lo, hi, red, sum);
    F::finish(p, i, hi - lo, lo >= w.r0, sum, st);
    F::apply(p, k ? w.tail_a : w.head_a, k ? w.r1 : w.head_b, st);
    __syncthreads();
  }
}

// ---------------------------------------------------------------- backward

struct BwdArgs {
  Shape s;
  const void* x;                 // the input, or NULL: its checkpoint
  const uint8_t *q, *scale;
  int int8;
  const float *stats, *weight, *bias;
  int act, zero_rest;
  const void* grad;
  void* grad_x;
  float *grad_weight, *grad_bias;
  double* part;
  float* chan;                   // [blocks][L + 2][C]: sums over the block's rows (db, dw_0 .. dw_L)
};

template <class T, int L, int V, bool kKept>
struct Bwd {
  static constexpr int K = (L + 1) * (L + 1), Q = L + 2;

  // a thread's channels: constants of its column and of the structure at hand
  struct Column {
    int row, col, g;
    float w[L + 1][V], bias[V], mu, r[L + 1];
  };

  static __device__ __forceinline__ void column(const BwdArgs& p, Column& c) {
    c.row = threadIdx.x / p.s.cv;
    c.col = (threadIdx.x - c.row * p.s.cv) * V;
    if (c.row >= p.s.rp) c.col = 0;
    c.g = c.col / p.s.cg;
    load_affine<V>(p.bias, c.col, 0.0f, c.bias);
#pragma unroll
    for (int l = 0; l <= L; ++l)
      load_affine<V>(p.weight ? p.weight + l * p.s.channels : nullptr, c.col, 1.0f, c.w[l]);
  }

  static __device__ __forceinline__ void structure(const BwdArgs& p, int i, Column& c) {
    const float* st = p.stats + static_cast<size_t>(i) * Q * p.s.groups + c.g;
    c.mu = __ldg(st);
#pragma unroll
    for (int l = 0; l <= L; ++l) c.r[l] = __ldg(st + (1 + l) * p.s.groups);
  }

  static __device__ __forceinline__ void load_x(const BwdArgs& p, int n, int m, int col, float (&v)[V]) {
    const size_t row = static_cast<size_t>(n) * K * p.s.channels;
    const int at = m * p.s.channels + col;
    if constexpr (kKept) {
      const int blocks = (K * p.s.channels + kCkptBlock - 1) / kCkptBlock;
      const float sc = scale_of(__ldg(p.scale + static_cast<size_t>(n) * blocks + at / kCkptBlock));
      if constexpr (V == 4) decode4(__ldg(reinterpret_cast<const unsigned*>(p.q + row + at)), sc, p.int8, v);
      else v[0] = decode(__ldg(p.q + row + at), sc, p.int8);
    } else {
      load_v<T, V>(static_cast<const T*>(p.x) + row + at, v);
    }
  }

  // One row: xhat and dy of every component, handed to put(l, m, xhat, dy); component 0 comes last,
  // because its dy holds the sum over all of them.
  template <class Put>
  static __device__ __forceinline__ void row(const BwdArgs& p, const Column& c, int n, Put&& put) {
    const T* gr = static_cast<const T*>(p.grad) + static_cast<size_t>(n) * K * p.s.channels + c.col;
    float x[K][V], g[K][V], f[V], t[V];
#pragma unroll
    for (int m = 0; m < K; ++m) {
      load_x(p, n, m, c.col, x[m]);
      load_v<T, V>(gr + m * p.s.channels, g[m]);
    }
#pragma unroll
    for (int k = 0; k < V; ++k) {
      x[0][k] = (x[0][k] - c.mu) * c.r[0];
      const float y = fmaf(x[0][k], c.w[0][k], c.bias[k]);
      f[k] = p.act ? logistic(y) : 1.0f;
      t[k] = g[0][k] * y;
    }
#pragma unroll
    for (int l = 1; l <= L; ++l)
#pragma unroll
      for (int m = l * l; m < (l + 1) * (l + 1); ++m) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
          x[m][k] *= c.r[l];
          t[k] = fmaf(g[m][k], x[m][k] * c.w[l][k], t[k]);
          g[m][k] *= f[k];
        }
        put(l, m, x[m], g[m]);
      }
#pragma unroll
    for (int k = 0; k < V; ++k) g[0][k] = p.act ? fmaf(f[k] * (1.0f - f[k]), t[k], g[0][k] * f[k]) : g[0][k];
    put(0, 0, x[0], g[0]);
  }

  // sum[0] = sum h (l = 0), sum[1 + l] = sum h xhat over rows [a, b); own adds db and dw_l of the
  // thread's channels
  static __device__ void sums(const BwdArgs& p, const Column& c, int a, int b, float (&own)[Q][V],
                              double (&acc)[Q][kThreads], double* red, double* sum) {
    float here[Q][V];
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int k = 0; k < V; ++k) here[q][k] = 0.0f;
    if (c.row < p.s.rp)
      for (int n = a + c.row; n < b; n += p.s.rp)
        row(p, c, n, [&](int l, int m, const float (&xh)[V], const float (&dy)[V]) {
#pragma unroll
          for (int k = 0; k < V; ++k) {
            here[1 + l][k] = fmaf(dy[k], xh[k], here[1 + l][k]);
            if (m == 0) here[0][k] += dy[k];
          }
        });
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      double t = 0.0;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        t = fma(static_cast<double>(here[q][k]), static_cast<double>(c.w[q == 0 ? 0 : q - 1][k]), t);
        own[q][k] += here[q][k];
      }
      acc[q][threadIdx.x] = t;
    }
    sum_groups<Q>(p.s, acc, red, sum);
  }

  static __device__ void apply(const BwdArgs& p, const Column& c, int a, int b, int n_rows, const double* sum) {
    if (c.row >= p.s.rp || !p.grad_x) return;
    float along[L + 1];
    const double size = static_cast<double>(n_rows) * p.s.cg;
    const float level = static_cast<float>(sum[c.g] / size);
#pragma unroll
    for (int l = 0; l <= L; ++l) along[l] = static_cast<float>(sum[(1 + l) * p.s.groups + c.g] / (size * (2 * l + 1)));
    for (int n = a + c.row; n < b; n += p.s.rp) {
      T* xr = static_cast<T*>(p.grad_x) + static_cast<size_t>(n) * K * p.s.channels + c.col;
      row(p, c, n, [&](int l, int m, const float (&xh)[V], const float (&dy)[V]) {
        float d[V];
#pragma unroll
        for (int k = 0; k < V; ++k) {
          d[k] = fmaf(dy[k], c.w[l][k], -xh[k] * along[l]);
          if (m == 0) d[k] -= level;
          d[k] *= c.r[l];
        }
        store_v<T, V>(xr + m * p.s.channels, d);
      });
    }
  }

  static __device__ void rest(const BwdArgs& p, const Column& c, int a, int b) {
    if (c.row >= p.s.rp || !p.zero_rest || !p.grad_x) return;
    const float zero[V] = {};
    for (int n = a + c.row; n < b; n += p.s.rp)
      for (int m = 0; m < K; ++m)
        store_v<T, V>(static_cast<T*>(p.grad_x) + (static_cast<size_t>(n) * K + m) * p.s.channels + c.col, zero);
  }
};

template <class T, int L, int V, bool kKept>
__global__ void __launch_bounds__(kThreads) k_norm_bwd(BwdArgs p) {
  using B = Bwd<T, L, V, kKept>;
  constexpr int Q = B::Q;
  __shared__ double acc[Q][kThreads];
  __shared__ double red[kThreads];
  __shared__ double sum[Q * kMaxGroups];
  const Shape& s = p.s;
  const int nq = Q * s.groups;
  const Span w = span_of(s);
  typename B::Column c;
  B::column(p, c);
  float own[Q][V];
#pragma unroll
  for (int q = 0; q < Q; ++q)
#pragma unroll
    for (int k = 0; k < V; ++k) own[q][k] = 0.0f;
  double* mine = p.part + static_cast<size_t>(blockIdx.x) * 2 * nq;
  if (w.head >= 0) {
    B::structure(p, w.head, c);
    B::sums(p, c, w.head_a, w.head_b, own, acc, red, sum);
    for (int i = threadIdx.x; i < nq; i += kThreads) mine[w.head_slot * nq + i] = sum[i];
    __syncthreads();
  }
  if (w.tail >= 0) {
    B::structure(p, w.tail, c);
    B::sums(p, c, w.tail_a, w.r1, own, acc, red, sum);
    for (int i = threadIdx.x; i < nq; i += kThreads) mine[nq + i] = sum[i];
    __syncthreads();
  }
  for (int i = w.first; i < w.last; ++i) {
    const int a = max(begin_of(s, i), w.r0), b = min(end_of(s, i), w.r1);
    if (a >= b) continue;
    B::structure(p, i, c);
    B::sums(p, c, a, b, own, acc, red, sum);
    B::apply(p, c, a, b, b - a, sum);
    __syncthreads();
  }
  if (s.ptr) {
    B::rest(p, c, w.r0, min(w.r1, begin_of(s, 0)));
    B::rest(p, c, max(w.r0, end_of(s, s.n_structs - 1)), w.r1);
  }
  // the block's channel sums, over the rows it reads side by side
  float* flat = reinterpret_cast<float*>(&acc[0][0]);
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < V; ++k) flat[threadIdx.x * V + k] = own[q][k];
    __syncthreads();
    for (int i = threadIdx.x; i < s.channels; i += kThreads) {
      float t = 0.0f;
      for (int r = 0; r < s.rp; ++r) t += flat[r * s.channels + i];
      p.chan[(static_cast<size_t>(blockIdx.x) * Q + q) * s.channels + i] = t;
    }
  }
  __syncthreads();
  if (gridDim.x > 1) cg::this_grid().sync();
  // dw and db: 8 sums at a time, 32 lanes to a sum's blocks
  for (int base = blockIdx.x * 8; base < Q * s.channels; base += gridDim.x * 8) {
    const int i = base + (threadIdx.x & 7), lane = threadIdx.x >> 3;
    double t = 0.0;
    if (i < Q * s.channels)
      for (int b = lane; b < gridDim.x; b += kThreads / 8) t += p.chan[static_cast<size_t>(b) * Q * s.channels + i];
    red[threadIdx.x] = t;
    __syncthreads();
    if (lane == 0 && i < Q * s.channels) {
      t = 0.0;
      for (int k = 0; k < kThreads / 8; ++k) t += red[k * 8 + threadIdx.x];
      const int q = i / s.channels;
      if (q == 0 && p.grad_bias) p.grad_bias[i] = static_cast<float>(t);
      if (q > 0 && p.grad_weight) p.grad_weight[i - s.channels] = static_cast<float>(t);
    }
    __syncthreads();
  }
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    const int i = k ? w.tail : w.head;
    if (i < 0) continue;
    const int lo = begin_of(s, i), hi = end_of(s, i);
    gather_partials(s, p.part, nq, lo, hi, red, sum);
    B::structure(p, i, c);
    B::apply(p, c, k ? w.tail_a : w.head_a, k ? w.r1 : w.head_b, hi - lo, sum);
    __syncthreads();
  }
}

// ---------------------------------------------------------------- launch

int vector_width(int channels, int groups) {
  return channels % 4 == 0 && (channels / groups) % 4 == 0 ? 4 : 1;
}

// A block for every rp rows at most, and no more blocks than run at once: the grid barrier needs
// them all on the device.
Shape shape_of(int n_nodes, int n_structs, int channels, int groups, int width, const int* ptr, int resident, int* blocks) {
  Shape s;
  s.n_nodes = n_nodes;
  s.n_structs = n_structs;
  s.channels = channels;
  s.groups = groups;
  s.cg = channels / groups;
  s.cv = channels / width;
  s.rp = kThreads / s.cv;
  s.ptr = ptr;
  long long b = (static_cast<long long>(n_nodes) + s.rp - 1) / s.rp;
  if (b > resident) b = resident;
  if (b < 1) b = 1;
  s.rows = static_cast<int>((n_nodes + b - 1) / b);
  *blocks = s.rows > 0 ? (n_nodes + s.rows - 1) / s.rows : 1;
  return s;
}

template <class Kernel, class Args>
etp_status launch(Kernel kernel, Args& p, int n_nodes, int n_structs, int channels, int groups, int width, const int* ptr,
                  int& per_sm, cudaStream_t stream, const char* what) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess && per_sm == 0) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kThreads, 0);
  if (e != cudaSuccess) return cuda_status(e, what);
  int resident = per_sm * sms, blocks = 0;
  if (resident > kMaxBlocks) resident = kMaxBlocks;
  p.s = shape_of(n_nodes, n_structs, channels, groups, width, ptr, resident, &blocks);
  void* args[] = {&p};
  if (blocks == 1) e = cudaLaunchKernel(reinterpret_cast<const void*>(kernel), dim3(1), dim3(kThreads), args, 0, stream);
  else e = cudaLaunchCooperativeKernel(reinterpret_cast<const void*>(kernel), dim3(blocks), dim3(kThreads), args, 0, stream);
  return cuda_status(e, what);
}

template <class T, int L, int V>
etp_status fwd_launch(const Call& c, FwdArgs& p, cudaStream_t s) {
  static int per_sm = 0;
  return launch(k_norm_fwd<T, L, V>, p, c.n_nodes, c.n_structs, c.channels, c.groups, V, c.node_ptr, per_sm, s, "group norm launch");
}
template <class T, int L, int V, bool kKept>
etp_status bwd_launch(const Call& c, BwdArgs& p, cudaStream_t s) {
  static int per_sm = 0;
  return launch(k_norm_bwd<T, L, V, kKept>, p, c.n_nodes, c.n_structs, c.channels, c.groups, V, c.node_ptr, per_sm, s,
                "group norm backward launch");
}

template <class T, int V>
etp_status fwd_rank(const Call& c, FwdArgs& p, cudaStream_t s) {
  switch (c.lmax) {
    case 0: return fwd_launch<T, 0, V>(c, p, s);
    case 1: return fwd_launch<T, 1, V>(c, p, s);
    case 2: return fwd_launch<T, 2, V>(c, p, s);
    default: return fwd_launch<T, 3, V>(c, p, s);
  }
}
template <class T, int V, bool kKept>
etp_status bwd_rank(const Call& c, BwdArgs& p, cudaStream_t s) {
  switch (c.lmax) {
    case 0: return bwd_launch<T, 0, V, kKept>(c, p, s);
    case 1: return bwd_launch<T, 1, V, kKept>(c, p, s);
    case 2: return bwd_launch<T, 2, V, kKept>(c, p, s);
    default: return bwd_launch<T, 3, V, kKept>(c, p, s);
  }
}
template <class T>
etp_status fwd_type(const Call& c, FwdArgs& p, int width, cudaStream_t s) {
  return width == 4 ? fwd_rank<T, 4>(c, p, s) : fwd_rank<T, 1>(c, p, s);
}
template <class T>
etp_status bwd_type(const Call& c, BwdArgs& p, int width, cudaStream_t s) {
  if (p.q) return width == 4 ? bwd_rank<T, 4, true>(c, p, s) : bwd_rank<T, 1, true>(c, p, s);
  return width == 4 ? bwd_rank<T, 4, false>(c, p, s) : bwd_rank<T, 1, false>(c, p, s);
}

size_t partial_bytes(const Call& c) {
  return align256(static_cast<size_t>(kMaxBlocks) * 2 * (c.lmax + 2) * c.groups * sizeof(double));
}

}  // namespace

__global__ void k_check_ptr(const int* ptr, int n_structs, int n_nodes, int* flag) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i > n_structs) return;
  const int v = ptr[i];
  if (v < 0 || v > n_nodes || (i < n_structs && ptr[i + 1] < v)) *flag = 1;
}

etp_status validate(const Call& c, void* ws, cudaStream_t s) {
  if (!c.node_ptr) return ETP_OK;
  int* flag = static_cast<int*>(ws);
  int bad = 0;
  cudaError_t e = cudaMemsetAsync(flag, 0, sizeof(int), s);
  if (e == cudaSuccess) {
    k_check_ptr<<<c.n_structs / 256 + 1, 256, 0, s>>>(c.node_ptr, c.n_structs, c.n_nodes, flag);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) e = cudaMemcpyAsync(&bad, flag, sizeof(int), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_status(e, "node_ptr validation");
  if (!bad) return ETP_OK;
  set_error("node_ptr must be ascending and stay within [0, n_nodes]");
  return ETP_ERR_BAD_GRAPH;
}

bool supported(int lmax, int channels, int groups) {
  return lmax >= 0 && lmax <= kMaxL && channels >= 1 && groups >= 1 && groups <= kMaxGroups && channels % groups == 0 &&
         channels / vector_width(channels, groups) <= kThreads;
}

size_t workspace_bytes(const Call& c, bool backward) {
  size_t n = partial_bytes(c);
  if (backward) n += align256(static_cast<size_t>(kMaxBlocks) * (c.lmax + 2) * c.channels * sizeof(float));
  return n;
}

etp_status forward(const Call& c, const void* x, const float* weight, const float* bias, float eps, void* out,
                   float* stats, etp_ckpt_format format, uint8_t* q, uint8_t* scale, void* ws, cudaStream_t s) {
  const int width = vector_width(c.channels, c.groups);
  FwdArgs p;
  p.x = x;
  p.weight = weight;
  p.bias = bias;
  p.eps = eps;
  p.act = c.activation;
  p.zero_rest = c.zero_rest;
  p.out = out;
  p.stats = stats;
  p.int8 = format == ETP_CKPT_INT8;
  p.part = static_cast<double*>(ws);
  // the norm writes the checkpoint itself where no block of 32 crosses a component's end
  const bool fused = format != ETP_CKPT_NONE && c.channels % kCkptBlock == 0;
  p.q = fused ? q : nullptr;
  p.scale = fused ? scale : nullptr;
  if (format != ETP_CKPT_NONE && !fused) {
    const int dim = c.channels * (c.lmax + 1) * (c.lmax + 1);
    etp_status st = ckpt::store(format, c.dtype, c.n_nodes, dim, x, q, scale, s);
    if (st != ETP_OK) return st;
  }
  switch (c.dtype) {
    case ETP_F32: return fwd_type<float>(c, p, width, s);
    case ETP_BF16: return fwd_type<__nv_bfloat16>(c, p, width, s);
    default: return fwd_type<__half>(c, p, width, s);
  }
}

etp_status backward(const Call& c, const void* x, etp_ckpt_format format, const uint8_t* q, const uint8_t* scale,
                    const float* stats, const float* weight, const float* bias, const void* grad_out, void* grad_x,
                    float* grad_weight, float* grad_bias, void* ws, cudaStream_t s) {
  BwdArgs p;
  p.x = x;
  p.q = format == ETP_CKPT_NONE ? nullptr : q;
  p.scale = scale;
  p.int8 = format == ETP_CKPT_INT8;
  p.stats = stats;
  p.weight = weight;
  p.bias = bias;
  p.act = c.activation;
  p.zero_rest = c.zero_rest;
  p.grad = grad_out;
  p.grad_x = grad_x;
  p.grad_weight = grad_weight;
  p.grad_bias = grad_bias;
  p.part = static_cast<double*>(ws);
  p.chan = reinterpret_cast<float*>(static_cast<char*>(ws) + partial_bytes(c));
  const int width = vector_width(c.channels, c.groups);
  switch (c.dtype) {
    case ETP_F32: return bwd_type<float>(c, p, width, s);
    case ETP_BF16: return bwd_type<__nv_bfloat16>(c, p, width, s);
    default: return bwd_type<__half>(c, p, width, s);
  }
}

}  // namespace norm
}  // namespace etp
