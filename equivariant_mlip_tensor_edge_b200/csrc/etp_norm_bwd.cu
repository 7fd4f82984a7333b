// Group norm on node rows: the backward (etp_norm_sweep.h has the method).
#include "etp_norm_sweep.h"

namespace etp {
namespace norm {
namespace {

// ---------------------------------------------------------------- backward

// Streams: grad_out, x or its codes, the codes' scales.
template <class T, int L, int V, bool kKept>
struct Bwd {
  static constexpr int K = (L + 1) * (L + 1), Q = L + 2, kStreams = kKept ? 3 : 2;
  static constexpr bool kBackward = true;
  using Sum = float;
  static constexpr int kRows = K == 1 ? 2 : 1;   // rows at once: more loads under way where a row has few

  static constexpr int kAcc = 4 * Q;

  float own[Q][V], here[Q][V];    // db and dw_l: of the block's rows, of the structure at hand
  float w[L + 1][V], bias[V], r[L + 1], mu;
  float level, along[L + 1];

  __device__ Bwd(const Args& p, const Place& at) {
    load_affine<V>(p.bias, at.col, 0.0f, bias);
#pragma unroll
    for (int l = 0; l <= L; ++l) load_affine<V>(p.weight ? p.weight + l * p.s.channels : nullptr, at.col, 1.0f, w[l]);
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int k = 0; k < V; ++k) own[q][k] = 0.0f;
    clear();
  }
  __device__ void clear() {
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int k = 0; k < V; ++k) here[q][k] = 0.0f;
  }
  __device__ void enter_up(const Args& p, const Place& at, int structure) {
    const float* st = p.stats_in + static_cast<size_t>(structure) * Q * p.s.groups.d + at.g;
    mu = __ldg(st);
#pragma unroll
    for (int l = 0; l <= L; ++l) r[l] = __ldg(st + (1 + l) * p.s.groups.d);
  }

  static __device__ __forceinline__ void load_x(const Args& p, const char* const (&src)[kStreams], int m, int col,
                                                float (&v)[V]) {
    const int at = m * p.s.channels;
    if constexpr (kKept) {
      const float sc = scale_of(static_cast<uint8_t>(src[2][(at + col) / kCkptBlock]));
      load_codes<V>(reinterpret_cast<const uint8_t*>(src[1]) + at, sc, p.int8, v);
    } else {
      lds_v<T, V>(src[1] + at * static_cast<int>(sizeof(T)), v);
    }
  }

  // component 0 of a row: xhat, g, f = phi(y_0) and g y
  struct Scalar {
    float xh[V], g[V], f[V], gy[V];
  };
  __device__ __forceinline__ void scalar(const Args& p, const char* const (&src)[kStreams], int col, Scalar& a) {
    load_x(p, src, 0, col, a.xh);
    lds_v<T, V>(src[0], a.g);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      a.xh[k] = (a.xh[k] - mu) * r[0];
      const float y = fmaf(a.xh[k], w[0][k], bias[k]);
      a.f[k] = p.act ? logistic(y) : 1.0f;
      a.gy[k] = a.g[k] * y;
    }
  }
  // dy_0 = g_0 f + f' sum g y; without an activation f' = 0
  static __device__ __forceinline__ float dy0(const Args& p, const Scalar& a, int k) {
    return p.act ? fmaf(a.f[k] * (1.0f - a.f[k]), a.gy[k], a.g[k] * a.f[k]) : a.g[k];
  }

  // Of rank l > 0 a row adds f sum_m g xhat to dw_l, w_l sum_m g xhat to g y: one multiply-add a value.
  template <int R>
  __device__ __forceinline__ void add(const Args& p, const Place&, const char* const (&src)[kStreams],
                                      const int (&step)[kStreams], int col) {
#pragma unroll
    for (int h = 0; h < R; ++h) {
      const char* from[kStreams];
#pragma unroll
      for (int k = 0; k < kStreams; ++k) from[k] = src[k] + h * step[k];
      add_row(p, from, col);
    }
  }
  __device__ __forceinline__ void add_row(const Args& p, const char* const (&src)[kStreams], int col) {
    Scalar a;
    scalar(p, src, col, a);
#pragma unroll
    for (int l = 1; l <= L; ++l) {
      float x[V], g[V], u[V];
#pragma unroll
      for (int m = l * l; m < (l + 1) * (l + 1); ++m) {
        load_x(p, src, m, col, x);
        lds_v<T, V>(src[0] + m * p.s.channels * static_cast<int>(sizeof(T)), g);
#pragma unroll
        for (int k = 0; k < V; ++k) u[k] = m == l * l ? g[k] * x[k] : fmaf(g[k], x[k], u[k]);
      }
#pragma unroll
      for (int k = 0; k < V; ++k) {
        u[k] *= r[l];
        a.gy[k] = fmaf(u[k], w[l][k], a.gy[k]);
        here[1 + l][k] = fmaf(u[k], a.f[k], here[1 + l][k]);
      }
    }
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const float dy = dy0(p, a, k);
      here[0][k] += dy;
      here[1][k] = fmaf(dy, a.xh[k], here[1][k]);
    }
  }
  // sum h (l = 0) and sum h xhat of every rank; a row's place for sums: [Q][cv] of 32 bits
  __device__ void leave(char* acc, int cv, int i) {
    float* f = reinterpret_cast<float*>(acc);
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      float t = 0.0f;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        t = fmaf(here[q][k], w[q == 0 ? 0 : q - 1][k], t);
        own[q][k] += here[q][k];
      }
      f[q * cv + i] = t;
    }
  }
  static __device__ __forceinline__ float first(const char* acc, int, int i) { return reinterpret_cast<const float*>(acc)[i]; }
  static __device__ __forceinline__ float second(const char* acc, int cv, int l, int i) {
    return reinterpret_cast<const float*>(acc)[(1 + l) * cv + i];
  }
  // mean h (l = 0) and mean h xhat
  static __device__ float2 value(const Args& p, int l, int n, double s0, double s1) {
    const double inv = reciprocal(static_cast<double>(n) * p.s.cg * (2 * l + 1));
    return make_float2(static_cast<float>(s0 * inv), static_cast<float>(s1 * inv));
  }
  __device__ void enter_down(const Args& p, const Place& at, int structure, const float* means) {
    enter_up(p, at, structure);
    level = means[at.g];
#pragma unroll
    for (int l = 0; l <= L; ++l) along[l] = means[(1 + l) * p.s.groups.d + at.g];
  }
  // outputs of rows n, n - rp, ..; inside: they belong to a structure
  template <int R>
  __device__ __forceinline__ void put(const Args& p, const Place& at, const char* const (&src)[kStreams],
                                      const int (&step)[kStreams], int col, int n, bool inside) {
#pragma unroll
    for (int h = 0; h < R; ++h) {
      const char* from[kStreams];
#pragma unroll
      for (int k = 0; k < kStreams; ++k) from[k] = src[k] - h * step[k];
      put_row(p, at, from, col, n - h * p.s.rp, inside);
    }
  }
  __device__ __forceinline__ void put_row(const Args& p, const Place& at, const char* const (&src)[kStreams], int col, int n,
                                          bool inside) {
    T* out = static_cast<T*>(p.out) + static_cast<size_t>(n) * K * p.s.channels + at.col;
    if (!inside) {
      const float zero[V] = {};
      for (int m = 0; m < K; ++m) store_v<T, V>(out + m * p.s.channels, zero);
      return;
    }
    Scalar a;
    scalar(p, src, col, a);
#pragma unroll
    for (int l = 1; l <= L; ++l) {
      // dx = g (r w f) - x (r^2 mean h xhat)
      float x[V], g[V], u[V], c[V];
      const float back = r[l] * r[l] * along[l];
#pragma unroll
      for (int k = 0; k < V; ++k) c[k] = r[l] * w[l][k] * a.f[k];
#pragma unroll
      for (int m = l * l; m < (l + 1) * (l + 1); ++m) {
        load_x(p, src, m, col, x);
        lds_v<T, V>(src[0] + m * p.s.channels * static_cast<int>(sizeof(T)), g);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          u[k] = m == l * l ? g[k] * x[k] : fmaf(g[k], x[k], u[k]);
          g[k] = fmaf(g[k], c[k], -x[k] * back);
        }
        store_v<T, V>(out + m * p.s.channels, g);
      }
#pragma unroll
      for (int k = 0; k < V; ++k) a.gy[k] = fmaf(u[k] * r[l], w[l][k], a.gy[k]);
    }
#pragma unroll
    for (int k = 0; k < V; ++k) a.g[k] = r[0] * (fmaf(dy0(p, a, k), w[0][k], -a.xh[k] * along[0]) - level);
    store_v<T, V>(out, a.g);
  }
  __device__ bool wants_outside(const Args& p) const { return p.zero_rest; }
};

template <class T, int L, int V, bool kKept>
etp_status bwd_launch(const Call& c, Args& p, cudaStream_t s) {
  const int dim = Bwd<T, L, V, kKept>::K * c.channels, size = static_cast<int>(sizeof(T));
  const int row_bytes[kMaxStreams] = {dim * size, kKept ? dim : dim * size, kKept ? (dim + kCkptBlock - 1) / kCkptBlock : 0};
  return launch<Bwd<T, L, V, kKept>, V>(c, p, row_bytes, s, "group norm backward launch");
}

template <class T, int V, bool kKept>
etp_status bwd_rank(const Call& c, Args& p, cudaStream_t s) {
  switch (c.lmax) {
    case 0: return bwd_launch<T, 0, V, kKept>(c, p, s);
    case 1: return bwd_launch<T, 1, V, kKept>(c, p, s);
    case 2: return bwd_launch<T, 2, V, kKept>(c, p, s);
    default: return bwd_launch<T, 3, V, kKept>(c, p, s);
  }
}
template <class T, bool kKept>
etp_status bwd_type(const Call& c, Args& p, int width, cudaStream_t s) {
  switch (width) {
    case 4: return bwd_rank<T, 4, kKept>(c, p, s);
    case 2: return bwd_rank<T, 2, kKept>(c, p, s);
    default: return bwd_rank<T, 1, kKept>(c, p, s);
  }
}

template <bool kKept>
etp_status bwd_kept(const Call& c, Args& p, int width, cudaStream_t s) {
  switch (c.dtype) {
    case ETP_F32: return bwd_type<float, kKept>(c, p, width, s);
    case ETP_BF16: return bwd_type<__nv_bfloat16, kKept>(c, p, width, s);
    default: return bwd_type<__half, kKept>(c, p, width, s);
  }
}

}  // namespace

etp_status launch_backward(const Call& c, Args& p, bool kept, int width, cudaStream_t s) {
  return kept ? bwd_kept<true>(c, p, width, s) : bwd_kept<false>(c, p, width, s);
}

}  // namespace norm
}  // namespace etp
