// Group norm on node rows: the forward (etp_norm_sweep.h has the method).
#include "etp_norm_sweep.h"

namespace etp {
namespace norm {
namespace {

// ---------------------------------------------------------------- forward

template <class T, int L, int V>
struct Fwd {
  static constexpr int K = (L + 1) * (L + 1), Q = L + 2, kStreams = 1;
  static constexpr bool kBackward = false;
  using Sum = double;
  static constexpr int kRows = K == 1 ? 4 : K == 4 ? 2 : 1;   // rows at once: more loads under way where a row has few
  static constexpr int kLanes = kCkptBlock / V;   // threads that share a checkpoint block

  static constexpr int kAcc = 16 + 4 * L;         // bytes of a thread's sums: two of 64 bits, L of 32

  double t[Q];                                    // sum x (l = 0) and sum x^2 of every rank
  float w[L + 1][V], bias[V], wr[L + 1][V], mu;   // wr: w_l r_l of the structure at hand

  __device__ Fwd(const Args& p, const Place& at) {
    load_affine<V>(p.bias, at.col, 0.0f, bias);
#pragma unroll
    for (int l = 0; l <= L; ++l) load_affine<V>(p.weight ? p.weight + l * p.s.channels : nullptr, at.col, 1.0f, w[l]);
    clear();
  }
  __device__ void clear() {
#pragma unroll
    for (int q = 0; q < Q; ++q) t[q] = 0.0;
  }
  __device__ void enter_up(const Args&, const Place&, int) {}

  // Of l > 0 a row's squares (at most 28 to a thread, no cancellation) are added in 32 bits; the rest in 64.
  // Rows `step` bytes apart.
  template <int R>
  __device__ void add(const Args& p, const Place&, const char* const (&src)[kStreams], const int (&step)[kStreams], int) {
    float v[R][K][V];
#pragma unroll
    for (int h = 0; h < R; ++h)
#pragma unroll
      for (int m = 0; m < K; ++m)
        lds_v<T, V>(src[0] + h * step[0] + m * p.s.channels * static_cast<int>(sizeof(T)), v[h][m]);
#pragma unroll
    for (int h = 0; h < R; ++h) {
      double s0 = 0.0, s1 = 0.0;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const double d = v[h][0][k];
        s0 += d;
        s1 = fma(d, d, s1);
      }
      t[0] += s0;
      t[1] += s1;
#pragma unroll
      for (int l = 1; l <= L; ++l) {
        float row = 0.0f;
#pragma unroll
        for (int m = l * l; m < (l + 1) * (l + 1); ++m)
#pragma unroll
          for (int k = 0; k < V; ++k) row = fmaf(v[h][m][k], v[h][m][k], row);
        t[1 + l] += row;
      }
    }
  }
  // A row's place for sums: [2][cv] of 64 bits, [L][cv] rounded to 32 (2^-24 of a thread's sum once; in 64
  // they cost a tenth of the ring, and 17.6 -> 19.1 us for 600 molecules of 96 channels in 16 bits).
  __device__ void leave(char* acc, int cv, int i) {
    double* d = reinterpret_cast<double*>(acc);
    d[i] = t[0];
    d[cv + i] = t[1];
    float* f = reinterpret_cast<float*>(d + 2 * cv);
#pragma unroll
    for (int l = 1; l <= L; ++l) f[(l - 1) * cv + i] = static_cast<float>(t[1 + l]);
  }
  static __device__ __forceinline__ double first(const char* acc, int, int i) { return reinterpret_cast<const double*>(acc)[i]; }
  static __device__ __forceinline__ double second(const char* acc, int cv, int l, int i) {
    const double* d = reinterpret_cast<const double*>(acc);
    return l == 0 ? d[cv + i] : reinterpret_cast<const float*>(d + 2 * cv)[(l - 1) * cv + i];
  }

  // Statistics of rank l of n rows of a group, from sum x (l = 0) and sum x^2: r_l, and mu for l = 0. The
  // variance of l = 0 is (N sum x^2 - (sum x)^2) / N^2, with the rounding errors of both products added
  // back: what cancels is as good as the sums are.
  static __device__ float2 value(const Args& p, int l, int n, double s0, double s1) {
    const double count = static_cast<double>(n) * p.s.cg * (2 * l + 1), inv = reciprocal(count);
    double var = s1 * inv;
    if (l == 0) {
      const double a = count * s1, b = s0 * s0;
      var = ((a - b) + (fma(count, s1, -a) - fma(s0, s0, -b))) * inv * inv;
    }
    if (var < 0.0) var = 0.0;   // not fmax, which would drop a NaN
    return make_float2(l == 0 ? static_cast<float>(s0 * inv) : 0.0f,
                       rsqrtf(static_cast<float>(var + static_cast<double>(p.eps))));
  }

  __device__ __forceinline__ void enter_down(const Args& p, const Place& at, int, const float* st) {
    mu = st[at.g];
#pragma unroll
    for (int l = 0; l <= L; ++l) {
      const float r = st[(1 + l) * p.s.groups.d + at.g];
#pragma unroll
      for (int k = 0; k < V; ++k) wr[l][k] = w[l][k] * r;
    }
  }

  // Checkpoint codes of N vectors of a row, `apart` values from one to the next: N reductions side by side,
  // as each is a chain of shuffles.
  template <int N>
  static __device__ __forceinline__ void keep(const Args& p, size_t at, int apart, const float (&v)[N][V]) {
    float top[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      top[i] = max_abs(v[i][0], v[i][V - 1]);
#pragma unroll
      for (int k = 1; k < V - 1; ++k) top[i] = max_abs(top[i], v[i][k]);
    }
    // the lanes of a block hold the same row, so they are here together
    const unsigned lane = threadIdx.x & 31;
    const unsigned mask = kLanes == 32 ? 0xffffffffu : ((1u << (kLanes & 31)) - 1u) << (lane & (32u - kLanes));
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) top[i] = max_abs(top[i], __shfl_xor_sync(mask, top[i], o));
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const unsigned byte = scale_byte(top[i], p.int8);
      const size_t to = at + i * apart;
      store_codes<V>(p.q + to, v[i], inv_scale(byte), byte == kCkptBad, p.int8);
      if ((lane & (kLanes - 1)) == 0) p.scale[to / kCkptBlock] = static_cast<uint8_t>(byte);
    }
  }

  // components [M, M + N) of a row; f: the gate, made by component 0
  template <int M, int N>
  __device__ __forceinline__ void put_part(const Args& p, const char* src, size_t first, bool inside, float (&f)[V]) {
    const int C = p.s.channels;
    float v[N][V];
#pragma unroll
    for (int i = 0; i < N; ++i) lds_v<T, V>(src + (M + i) * C * static_cast<int>(sizeof(T)), v[i]);
    if (p.q) keep<N>(p, first + M * C, C, v);
    if (!inside && !p.zero_rest) return;
    T* out = static_cast<T*>(p.out) + first + M * C;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int m = M + i, l = m == 0 ? 0 : m < 4 ? 1 : m < 9 ? 2 : 3;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        if (m == 0) {
          v[i][k] = fmaf(v[i][k] - mu, wr[0][k], bias[k]);
          f[k] = p.act ? logistic(v[i][k]) : 1.0f;
          v[i][k] *= f[k];
        } else {
          v[i][k] = v[i][k] * (wr[l <= L ? l : L][k] * f[k]);
        }
        if (!inside) v[i][k] = 0.0f;
      }
      store_v<T, V>(out + i * C, v[i]);
    }
  }

  // outputs of rows n, n - rp, ..; inside: they belong to a structure
  template <int R>
  __device__ __forceinline__ void put(const Args& p, const Place& at, const char* const (&src)[kStreams],
                                      const int (&step)[kStreams], int, int n, bool inside) {
#pragma unroll
    for (int h = 0; h < R; ++h) {
      const size_t first = static_cast<size_t>(n - h * p.s.rp) * K * p.s.channels + at.col;
      const char* from = src[0] - h * step[0];
      float f[V];
      put_part<0, K < 4 ? 1 : 4>(p, from, first, inside, f);
      if constexpr (K > 4) put_part<4, K == 9 ? 5 : 4>(p, from, first, inside, f);
      if constexpr (K > 9) put_part<8, 4>(p, from, first, inside, f);
      if constexpr (K > 9) put_part<12, 4>(p, from, first, inside, f);
    }
  }
  __device__ bool wants_outside(const Args& p) const { return p.q || p.zero_rest; }
};

template <class T, int L, int V>
etp_status fwd_launch(const Call& c, Args& p, cudaStream_t s) {
  const int row_bytes[kMaxStreams] = {Fwd<T, L, V>::K * c.channels * static_cast<int>(sizeof(T)), 0, 0};
  return launch<Fwd<T, L, V>, V>(c, p, row_bytes, s, "group norm launch");
}
template <class T, int V>
etp_status fwd_rank(const Call& c, Args& p, cudaStream_t s) {
  switch (c.lmax) {
    case 0: return fwd_launch<T, 0, V>(c, p, s);
    case 1: return fwd_launch<T, 1, V>(c, p, s);
    case 2: return fwd_launch<T, 2, V>(c, p, s);
    default: return fwd_launch<T, 3, V>(c, p, s);
  }
}
template <class T>
etp_status fwd_type(const Call& c, Args& p, int width, cudaStream_t s) {
  switch (width) {
    case 4: return fwd_rank<T, 4>(c, p, s);
    case 2: return fwd_rank<T, 2>(c, p, s);
    default: return fwd_rank<T, 1>(c, p, s);
  }
}

}  // namespace

etp_status launch_forward(const Call& c, Args& p, int width, cudaStream_t s) {
  switch (c.dtype) {
    case ETP_F32: return fwd_type<float>(c, p, width, s);
    case ETP_BF16: return fwd_type<__nv_bfloat16>(c, p, width, s);
    default: return fwd_type<__half>(c, p, width, s);
  }
}

}  // namespace norm
}  // namespace etp
