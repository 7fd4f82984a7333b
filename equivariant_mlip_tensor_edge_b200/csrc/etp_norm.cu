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
// Either direction needs a structure's sums before its first output: two sweeps over the rows, bound by
// memory. One cooperative launch does both. A block owns a run of rows, which one warp brings into
// shared memory tile by tile with bulk copies, through a ring of slots that the other warps read. The
// first sweep goes up, the second comes down, so what the ring holds at the turn (all of it, where the
// rows fit on the chip) is not read again, and what comes next was read last and is likely in L2. A
// structure that crosses blocks (two at most for a block: one that reaches in from before, one that goes
// on behind) leaves partial sums, which meet after the grid barrier between the sweeps. Sums are kept in
// 64 bits: mu and the mean square cancel where mu is far larger than the spread. Every sum has one
// order, so equal calls give equal bits.
//
// A thread holds V neighbouring channels (V = 4 where channels and group size divide by 4, else 1) of
// every rp-th row and walks the row's components, so a channel's gate stays in its thread. Sums stay in
// the thread's registers until its last row of a structure, which leaves them in shared memory. The
// warps meet to add them up once for the rows that the ring holds, not at every structure's end.
#include <cooperative_groups.h>

#include <climits>
#include <string>

#include "etp_checkpoint.h"
#include "etp_internal.h"
#include "etp_norm.h"
#include "etp_tc_common.h"

namespace cg = cooperative_groups;

namespace etp {
namespace norm {
namespace {

constexpr int kThreads = 480;             // that compute; a further warp copies
constexpr int kBlock = kThreads + 32;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxSlots = 16;
constexpr int kMaxTileRows = 64;
constexpr int kTileBytes = 24 * 1024;     // aim of a tile
constexpr int kMaxStreams = 3;
constexpr int kBlocksPerSm = 1;
constexpr int kSmem = (227 / kBlocksPerSm - 1) * 1024;   // dynamic, for a block

struct Shape {
  int n_nodes, n_structs, rows;   // rows: a block's share
  int channels, groups, cg;       // cg: channels of a group
  int cv, rp;                     // vectors of a row's component; rows a block reads side by side
  const int* ptr;                 // NULL: one structure of all rows
};

// Shared memory: ring slots of tile_rows rows of every stream, tables for the rows and the structure
// ends of each slot's tile, and the threads' sums at their last rows of a structure. Those are kept by
// row, in a ring as long as the rows that warps can be apart.
struct Ring {
  int tile_rows, slots, slot_bytes, acc_rows, acc_bytes;
  int off[kMaxStreams];
  int o_rows, o_ends, o_sum, o_edge, o_acc, o_ring, bytes;
  const char* src[kMaxStreams];
  int row_bytes[kMaxStreams];        // 0: stream not used
};

// A structure's end inside a block's rows: rows [a, b) of it lie in the block. slot < 0: all of it;
// 0 / 1: it began before / goes on behind, and its sums are partial.
struct alignas(16) End {
  int structure, a, b, slot;
};

__device__ __forceinline__ int clamp_row(const Shape& s, int v) { return min(max(v, 0), s.n_nodes); }
__device__ __forceinline__ int begin_of(const Shape& s, int i) { return s.ptr ? clamp_row(s, __ldg(s.ptr + i)) : 0; }
__device__ __forceinline__ int end_of(const Shape& s, int i) {
  return s.ptr ? clamp_row(s, __ldg(s.ptr + i + 1)) : s.n_nodes;
}

// Numbers of structures that end at or before rows ra <= rb, by one warp: every round probes 32 places
// for each.
__device__ void ended_by(const Shape& s, int ra, int rb, int* na, int* nb) {
  const int lane = threadIdx.x & 31;
  int lo[2] = {0, 0}, hi[2] = {s.n_structs, s.n_structs};
  while (lo[0] < hi[0] || lo[1] < hi[1]) {
    int step[2], end[2];
    bool probe[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      step[k] = (hi[k] - lo[k] + 31) / 32;
      const long long at = lo[k] + static_cast<long long>(lane) * step[k];
      probe[k] = at < hi[k];
      end[k] = probe[k] ? end_of(s, static_cast<int>(at)) : 0;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = __popc(__ballot_sync(0xffffffffu, probe[k] && end[k] <= (k ? rb : ra)));
      if (lo[k] >= hi[k]) continue;
      if (c == 0) {
        hi[k] = lo[k];
        continue;
      }
      if (static_cast<long long>(lo[k]) + static_cast<long long>(c) * step[k] < hi[k]) hi[k] = lo[k] + c * step[k];
      lo[k] += (c - 1) * step[k] + 1;
    }
  }
  *na = lo[0];
  *nb = lo[1];
}

struct Shared {
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  int4 tile[kMaxSlots];              // structure of all rows or kMixed, its end, structures ended so far, -
  uint64_t gate;
  int copies[kMaxSlots];
  int abort, first, behind;          // structures that end in the block's rows: [first, behind)
  int head, tail;                    // structures that cross the block's first / last row, or -1
};
constexpr int kMixed = -2;

// Slot and parity of consecutive tiles' copies.
struct Turn {
  int slot;
  uint32_t parity;
  __device__ void next(int slots) {
    if (++slot == slots) {
      slot = 0;
      parity ^= 1u;
    }
  }
};

// The compute warps meet here while copies are under way. A barrier with a bounded wait, unlike the
// hardware's: a warp that gave up on a copy does not come.
struct Gate {
  uint32_t parity = 0;
  __device__ bool meet(Shared* sh, int* err) {
    __syncwarp();
    tc::mbar_arrive_lane0(&sh->gate, threadIdx.x & 31);
    const bool ok = tc::warp_wait(&sh->gate, parity, &sh->abort, err, 3);
    parity ^= 1u;
    return ok;
  }
};

__device__ __forceinline__ void meet_compute() { asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory"); }

__device__ __forceinline__ float logistic(float t) { return __fdividef(1.0f, 1.0f + __expf(-t)); }

// 1 / v for a count: a 32-bit reciprocal and one Newton step, 2^-46 off
__device__ __forceinline__ double reciprocal(double v) {
  const double r = __frcp_rn(static_cast<float>(v));
  return fma(r, fma(-v, r, 1.0), r);
}

template <class T, int V>
__device__ __forceinline__ void lds_v(const char* p, float (&v)[V]) {
  if constexpr (V == 1) {
    v[0] = to_f32<T>(*reinterpret_cast<const T*>(p));
  } else if constexpr (sizeof(T) == 4) {
    const float4 t = *reinterpret_cast<const float4*>(p);
    v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
  } else {
    union { uint2 u; T h[4]; } t;
    t.u = *reinterpret_cast<const uint2*>(p);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = to_f32<T>(t.h[k]);
  }
}

template <int V>
__device__ __forceinline__ void load_affine(const float* p, int col, float fill, float (&v)[V]) {
#pragma unroll
  for (int k = 0; k < V; ++k) v[k] = p ? __ldg(p + col + k) : fill;
}

struct Args {
  Shape s;
  Ring ring;
  const float *weight, *bias, *stats_in;
  float eps;
  int act, zero_rest, int8;
  void* out;                  // out, or grad_x (may be NULL)
  float* table;               // [structures][Q][groups]: statistics, or the backward's means
  uint8_t *q, *scale;         // the checkpoint to write, or NULL
  float *grad_weight, *grad_bias;
  double* part;               // [blocks][2][Q][groups]: sums of the structures that cross blocks
  float* chan;                // [blocks][Q][C]: db, dw_0 .. dw_L of a block's rows
  int* err;
};

// A thread's place: its first row of rp, its channels, their group
struct Place {
  int row, col, g;
};

// ---------------------------------------------------------------- forward

template <class T, int L, int V>
struct Fwd {
  static constexpr int K = (L + 1) * (L + 1), Q = L + 2, kStreams = 1;
  static constexpr bool kBackward = false;
  using Sum = double;
  static constexpr int kLanes = kCkptBlock / V;   // threads that share a checkpoint block

  static constexpr int kAcc = 16 + 4 * L;         // bytes of a thread's sums: two of 64 bits, L of 32

  double t[2];
  float u[L + 1];
  float w[L + 1][V], bias[V], r[L + 1], mu;

  __device__ Fwd(const Args& p, const Place& at) {
    load_affine<V>(p.bias, at.col, 0.0f, bias);
#pragma unroll
    for (int l = 0; l <= L; ++l) load_affine<V>(p.weight ? p.weight + l * p.s.channels : nullptr, at.col, 1.0f, w[l]);
    clear();
  }
  __device__ void clear() {
    t[0] = t[1] = 0.0;
#pragma unroll
    for (int l = 0; l <= L; ++l) u[l] = 0.0f;
  }
  __device__ void enter_up(const Args&, const Place&, int) {}

  // t += x, x^2 (l = 0); u_l += x^2 (no cancellation: in 32 bits)
  __device__ void add(const Args& p, const Place&, const char* const (&src)[kStreams], int) {
    float v[V];
    lds_v<T, V>(src[0], v);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const double d = v[k];
      t[0] += d;
      t[1] = fma(d, d, t[1]);
    }
#pragma unroll
    for (int l = 1; l <= L; ++l) {
      float row = 0.0f;
#pragma unroll
      for (int m = l * l; m < (l + 1) * (l + 1); ++m) {
        lds_v<T, V>(src[0] + m * p.s.channels * static_cast<int>(sizeof(T)), v);
#pragma unroll
        for (int k = 0; k < V; ++k) row = fmaf(v[k], v[k], row);
      }
      u[l] += row;
    }
  }
  // a row's place for sums: [2][cv] of 64 bits, [L][cv] of 32
  __device__ void leave(char* acc, int cv, int i) {
    double* d = reinterpret_cast<double*>(acc);
    d[i] = t[0];
    d[cv + i] = t[1];
    float* f = reinterpret_cast<float*>(d + 2 * cv);
#pragma unroll
    for (int l = 1; l <= L; ++l) f[(l - 1) * cv + i] = u[l];
  }
  static __device__ __forceinline__ double first(const char* acc, int, int i) { return reinterpret_cast<const double*>(acc)[i]; }
  static __device__ __forceinline__ double second(const char* acc, int cv, int l, int i) {
    const double* d = reinterpret_cast<const double*>(acc);
    return l == 0 ? d[cv + i] : reinterpret_cast<const float*>(d + 2 * cv)[(l - 1) * cv + i];
  }

  // Statistics of rank l of n rows of a group, from sum x (l = 0) and sum x^2: r_l, and mu for l = 0.
  static __device__ float2 value(const Args& p, int l, int n, double s0, double s1) {
    const double inv = reciprocal(static_cast<double>(n) * p.s.cg * (2 * l + 1));
    const double m = l == 0 ? s0 * inv : 0.0;
    double var = fma(-m, m, s1 * inv);
    if (var < 0.0) var = 0.0;   // not fmax, which would drop a NaN
    return make_float2(static_cast<float>(m), rsqrtf(static_cast<float>(var + static_cast<double>(p.eps))));
  }

  __device__ void enter_down(const Args& p, const Place& at, int, const float* st) {
    mu = st[at.g];
#pragma unroll
    for (int l = 0; l <= L; ++l) r[l] = st[(1 + l) * p.s.groups + at.g];
  }

  static __device__ __forceinline__ void keep(const Args& p, size_t at, const float (&v)[V]) {
    unsigned top = 0;
#pragma unroll
    for (int k = 0; k < V; ++k) top = max(top, abs_bits(v[k]));
    // the lanes of a block hold the same row, so they are here together
    const unsigned lane = threadIdx.x & 31;
    const unsigned mask = kLanes == 32 ? 0xffffffffu : 0xffu << (lane & 24u);
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) top = max(top, __shfl_xor_sync(mask, top, o));
    const unsigned byte = scale_byte(top, p.int8);
    if constexpr (V == 4) *reinterpret_cast<unsigned*>(p.q + at) = encode4(v, inv_scale(byte), byte == kCkptBad, p.int8);
    else p.q[at] = static_cast<uint8_t>(encode(v[0], inv_scale(byte), byte == kCkptBad, p.int8));
    if ((lane & (kLanes - 1)) == 0) p.scale[at / kCkptBlock] = static_cast<uint8_t>(byte);
  }

  // outputs of row n; inside: it belongs to a structure
  __device__ void put(const Args& p, const Place& at, const char* const (&src)[kStreams], int, int n, bool inside) {
    const size_t first = static_cast<size_t>(n) * K * p.s.channels + at.col;
    T* out = static_cast<T*>(p.out) + first;
    float v[V], f[V];
    lds_v<T, V>(src[0], v);
    if (p.q) keep(p, first, v);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      v[k] = fmaf((v[k] - mu) * r[0], w[0][k], bias[k]);
      f[k] = p.act ? logistic(v[k]) : 1.0f;
      v[k] = inside ? v[k] * f[k] : 0.0f;
    }
    if (inside || p.zero_rest) store_v<T, V>(out, v);
#pragma unroll
    for (int l = 1; l <= L; ++l)
#pragma unroll
      for (int m = l * l; m < (l + 1) * (l + 1); ++m) {
        lds_v<T, V>(src[0] + m * p.s.channels * static_cast<int>(sizeof(T)), v);
        if (p.q) keep(p, first + m * p.s.channels, v);
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = inside ? v[k] * (r[l] * w[l][k]) * f[k] : 0.0f;
        if (inside || p.zero_rest) store_v<T, V>(out + m * p.s.channels, v);
      }
  }
  __device__ bool wants_outside(const Args& p) const { return p.q || p.zero_rest; }
};

// ---------------------------------------------------------------- backward

// Streams: grad_out, x or its codes, the codes' scales.
template <class T, int L, int V, bool kKept>
struct Bwd {
  static constexpr int K = (L + 1) * (L + 1), Q = L + 2, kStreams = kKept ? 3 : 2;
  static constexpr bool kBackward = true;
  using Sum = float;

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
    const float* st = p.stats_in + static_cast<size_t>(structure) * Q * p.s.groups + at.g;
    mu = __ldg(st);
#pragma unroll
    for (int l = 0; l <= L; ++l) r[l] = __ldg(st + (1 + l) * p.s.groups);
  }

  static __device__ __forceinline__ void load_x(const Args& p, const char* const (&src)[kStreams], int m, int col,
                                                float (&v)[V]) {
    const int at = m * p.s.channels;
    if constexpr (kKept) {
      const float sc = scale_of(static_cast<uint8_t>(src[2][(at + col) / kCkptBlock]));
      if constexpr (V == 4) decode4(*reinterpret_cast<const unsigned*>(src[1] + at), sc, p.int8, v);
      else v[0] = decode(static_cast<uint8_t>(src[1][at]), sc, p.int8);
    } else {
      lds_v<T, V>(src[1] + at * static_cast<int>(sizeof(T)), v);
    }
  }

  // xhat and dy of every component of a row, handed to use(l, m, xhat, dy); component 0 comes last,
  // because its dy holds the sum over all of them
  template <class Use>
  __device__ __forceinline__ void row(const Args& p, const char* const (&src)[kStreams], int col, Use&& use) {
    float x[V], g[V], x0[V], g0[V], f[V], u[V];
    load_x(p, src, 0, col, x0);
    lds_v<T, V>(src[0], g0);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      x0[k] = (x0[k] - mu) * r[0];
      const float y = fmaf(x0[k], w[0][k], bias[k]);
      f[k] = p.act ? logistic(y) : 1.0f;
      u[k] = g0[k] * y;
    }
#pragma unroll
    for (int l = 1; l <= L; ++l)
#pragma unroll
      for (int m = l * l; m < (l + 1) * (l + 1); ++m) {
        load_x(p, src, m, col, x);
        lds_v<T, V>(src[0] + m * p.s.channels * static_cast<int>(sizeof(T)), g);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          x[k] *= r[l];
          u[k] = fmaf(g[k], x[k] * w[l][k], u[k]);
          g[k] *= f[k];
        }
        use(l, m, x, g);
      }
#pragma unroll
    for (int k = 0; k < V; ++k) g0[k] = p.act ? fmaf(f[k] * (1.0f - f[k]), u[k], g0[k] * f[k]) : g0[k];
    use(0, 0, x0, g0);
  }

  __device__ void add(const Args& p, const Place&, const char* const (&src)[kStreams], int col) {
    row(p, src, col, [&](int l, int m, const float (&xh)[V], const float (&dy)[V]) {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        here[1 + l][k] = fmaf(dy[k], xh[k], here[1 + l][k]);
        if (m == 0) here[0][k] += dy[k];
      }
    });
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
    for (int l = 0; l <= L; ++l) along[l] = means[(1 + l) * p.s.groups + at.g];
  }
  __device__ void put(const Args& p, const Place& at, const char* const (&src)[kStreams], int col, int n, bool inside) {
    T* out = static_cast<T*>(p.out) + static_cast<size_t>(n) * K * p.s.channels + at.col;
    if (!inside) {
      const float zero[V] = {};
      for (int m = 0; m < K; ++m) store_v<T, V>(out + m * p.s.channels, zero);
      return;
    }
    row(p, src, col, [&](int l, int m, const float (&xh)[V], const float (&dy)[V]) {
      float d[V];
#pragma unroll
      for (int k = 0; k < V; ++k) {
        d[k] = fmaf(dy[k], w[l][k], -xh[k] * along[l]);
        if (m == 0) d[k] -= level;
        d[k] *= r[l];
      }
      store_v<T, V>(out + m * p.s.channels, d);
    });
  }
  __device__ bool wants_outside(const Args& p) const { return p.zero_rest; }
};

// ---------------------------------------------------------------- the two sweeps

struct Work {
  int r0, r1, tiles;
};

// number of a tile's copy among its slot's: up the tiles once, then down over those the ring lost
__device__ __forceinline__ Turn turn_of(const Ring& ring, int tiles, int tile, bool down) {
  const int slot = tile % ring.slots, n = (tiles - 1 - slot) / ring.slots + 1;
  const int number = down ? n + ((n - 1) * ring.slots + slot - tile) / ring.slots - 1 : tile / ring.slots;
  return Turn{slot, static_cast<uint32_t>(number & 1)};
}

// Starts a tile's copies into its slot, a lane to a stream: the aligned bytes around the tile, and by
// hand the last bytes of an array that do not fill 16.
template <int kStreams>
__device__ __forceinline__ void copy_tile(const Args& p, Shared* sh, char* smem, int slot, int t0, int t1) {
  const Ring& ring = p.ring;
  const int lane = threadIdx.x & 31;
  char* dst = smem + ring.o_ring + static_cast<size_t>(slot) * ring.slot_bytes;
  if (lane < kStreams) {
    const size_t rb = ring.row_bytes[lane], e = t1 * rb, a = (t0 * rb) & ~static_cast<size_t>(15);
    const size_t whole = (p.s.n_nodes * rb) & ~static_cast<size_t>(15);
    const size_t b = max(a, min((e + 15) & ~static_cast<size_t>(15), whole));
    const uint32_t bytes = static_cast<uint32_t>(b - a);
    tc::mbar_expect_tx(&sh->full[slot], bytes);
    if (bytes) tc::bulk_g2s(dst + ring.off[lane], ring.src[lane] + a, bytes, &sh->full[slot]);
    if (lane == 0) ++sh->copies[slot];
  }
  if (t1 == p.s.n_nodes) {
#pragma unroll
    for (int k = 0; k < kStreams; ++k) {
      const size_t rb = ring.row_bytes[k], e = t1 * rb, a = (t0 * rb) & ~static_cast<size_t>(15);
      const size_t b = max(a, e & ~static_cast<size_t>(15));
      if (b + lane < e) dst[ring.off[k] + (b - a) + lane] = ring.src[k][b + lane];
    }
  }
}

// Writes the tables of a tile: the structure of every row, and the structures that end here, after the
// *ended of the tiles before. `last` keeps the structure found last, which covers whole tiles of a large
// one.
__device__ __forceinline__ void describe_tile(const Args& p, const Work& w, Shared* sh, char* smem, int slot, int t0,
                                              int t1, End* last, int* ended) {
  const Shape& s = p.s;
  const Ring& ring = p.ring;
  const int lane = threadIdx.x & 31;
  End* ends = reinterpret_cast<End*>(smem + ring.o_ends);
  const int room = ring.slots * ring.tile_rows;
  if (last->structure >= 0 && last->a <= t0 && last->b >= t1) {
    const int n_ends = last->b == t1;
    if (lane == 0) {
      if (n_ends) ends[*ended % room] = *last;
      sh->tile[slot] = make_int4(last->structure, last->b, *ended + n_ends, 0);
    }
    *ended += n_ends;
  } else {
    int2* rows = reinterpret_cast<int2*>(smem + ring.o_rows) + slot * ring.tile_rows;
    for (int base = t0; base < t1; base += 32) {
      const int n = base + lane;
      int lo = sh->first, hi = sh->behind;      // the first structure that ends behind row n
      while (lo < hi) {
        const int mid = lo + (hi - lo) / 2;
        if (end_of(s, mid) > n) hi = mid;
        else lo = mid + 1;
      }
      End end{-1, 0, 0, -1};
      if (n < t1 && lo < s.n_structs) {
        const int sa = begin_of(s, lo), sb = end_of(s, lo);
        if (sa <= n && n < sb) {
          end.structure = lo;
          end.a = max(sa, w.r0);
          end.b = min(sb, w.r1);
          end.slot = sa < w.r0 ? 0 : sb > w.r1 ? 1 : -1;
        }
      }
      const bool ends_here = end.structure >= 0 && end.b == n + 1;
      const unsigned votes = __ballot_sync(0xffffffffu, ends_here);
      if (n < t1) rows[n - t0] = make_int2(end.structure, end.b);
      if (ends_here) ends[(*ended + __popc(votes & ((1u << lane) - 1u))) % room] = end;
      *ended += __popc(votes);
      const int from = min(31, t1 - 1 - base);
      last->structure = __shfl_sync(0xffffffffu, end.structure, from);
      last->a = __shfl_sync(0xffffffffu, end.a, from);
      last->b = __shfl_sync(0xffffffffu, end.b, from);
      last->slot = __shfl_sync(0xffffffffu, end.slot, from);
    }
    const bool one = last->structure >= 0 && last->a <= t0;   // and it reaches to the last row
    if (lane == 0) sh->tile[slot] = make_int4(one ? last->structure : kMixed, last->b, *ended, 0);
  }
  __syncwarp();
  tc::mbar_arrive_lane0(&sh->full[slot], lane);
}

// The sums of the structures ended with numbers [from, to), by all warps, from the threads' sums at their
// last rows (the last rp rows of a structure hold one of every thread): several lanes to a group and
// rank, then the statistics, or partial sums where the structure crosses blocks.
template <class Op>
__device__ void close(const Args& p, const Work& w, const char* acc, const End* ends, int from, int to) {
  constexpr int kRanks = Op::Q - 1;
  using Sum = typename Op::Sum;
  const Shape& s = p.s;
  const int G = s.groups, nq = Op::Q * G, cvg = s.cv / G, lane = threadIdx.x & 31;
  const int per = kRanks * G, items = (to - from) * per, room = p.ring.slots * p.ring.tile_rows;
  int parts = 1;
  while (parts < 32 && items * parts * 2 <= kThreads) parts *= 2;
  for (int base = (threadIdx.x / 32) * (32 / parts); base < items; base += kThreads / parts) {
    const int it = base + lane / parts, part = lane & (parts - 1);
    Sum a0 = 0, a1 = 0, b0 = 0, b1 = 0;     // two chains each: a sum waits for its last addend, not for its loads
    End e{-1, 0, 0, -1};
    int l = 0, g = 0;
    if (it < items) {
      const int k = it / per;
      e = ends[(from + k) % room];
      l = (it - k * per) / G;
      g = it - k * per - l * G;
      const int rows = min(s.rp, e.b - e.a);
      int at = (e.b - rows - w.r0 + part) % p.ring.acc_rows;
      for (int r = part; r < rows; r += parts) {
        const char* row = acc + static_cast<size_t>(at) * p.ring.acc_bytes;
        at += parts;
        if (at >= p.ring.acc_rows) at -= p.ring.acc_rows;
        int j = g * cvg;
        for (const int end = j + cvg - 1; j < end; j += 2) {
          if (l == 0) {
            a0 += Op::first(row, s.cv, j);
            b0 += Op::first(row, s.cv, j + 1);
          }
          a1 += Op::second(row, s.cv, l, j);
          b1 += Op::second(row, s.cv, l, j + 1);
        }
        if (cvg & 1) {
          if (l == 0) a0 += Op::first(row, s.cv, j);
          a1 += Op::second(row, s.cv, l, j);
        }
      }
    }
    double s0 = static_cast<double>(a0) + b0, s1 = static_cast<double>(a1) + b1;
    for (int o = parts / 2; o > 0; o /= 2) {
      s0 += __shfl_xor_sync(0xffffffffu, s0, o);
      s1 += __shfl_xor_sync(0xffffffffu, s1, o);
    }
    if (part == 0 && it < items) {
      if (e.slot < 0) {
        const float2 v = Op::value(p, l, e.b - e.a, s0, s1);
        float* at = p.table + static_cast<size_t>(e.structure) * nq + g;
        if (l == 0) at[0] = v.x;
        at[(1 + l) * G] = v.y;
      } else {
        double* at = p.part + (static_cast<size_t>(blockIdx.x) * 2 + e.slot) * nq + g;
        if (l == 0) at[0] = s0;
        at[(1 + l) * G] = s1;
      }
    }
  }
}

// sum[i] = sum over the blocks that hold rows [a, b) of one structure of their partials, in block order
__device__ void gather_partials(const Shape& s, const double* part, int nq, int a, int b, double* red, double* sum) {
  const int c0 = a / s.rows, c1 = (b - 1) / s.rows;
  const int parts = max(1, min(kThreads / nq, c1 - c0 + 1)), width = min(nq, kThreads);
  meet_compute();
  for (int base = 0; base < nq; base += width) {
    // neighbouring threads read neighbouring sums of one block
    const int k = threadIdx.x / width, i = base + threadIdx.x - k * width;
    double t = 0.0;
    if (i < nq && k < parts) {
      int c = c0 + k;
      if (k == 0) {
        t = part[(static_cast<size_t>(c) * 2 + 1) * nq + i];
        c += parts;
      }
      for (; c + 7 * parts <= c1; c += 8 * parts) {
        double v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = part[static_cast<size_t>(c + j * parts) * 2 * nq + i];
#pragma unroll
        for (int j = 0; j < 8; ++j) t += v[j];
      }
      for (; c <= c1; c += parts) t += part[static_cast<size_t>(c) * 2 * nq + i];
    }
    red[threadIdx.x] = t;
    meet_compute();
    if (threadIdx.x < width && i < nq) {
      t = 0.0;
      for (int j = 0; j < parts; ++j) t += red[j * width + threadIdx.x];
      sum[i] = t;
    }
    meet_compute();
  }
}

template <class Op, int V>
__global__ void __launch_bounds__(kBlock, kBlocksPerSm) k_norm(const __grid_constant__ Args p) {
  constexpr int Q = Op::Q, kStreams = Op::kStreams;
  extern __shared__ __align__(128) char smem[];
  __shared__ Shared sh;
  const Shape& s = p.s;
  const Ring& ring = p.ring;
  const int nq = Q * s.groups, lane = threadIdx.x & 31;
  Work w;
  w.r0 = static_cast<int>(min(static_cast<long long>(blockIdx.x) * s.rows, static_cast<long long>(s.n_nodes)));
  w.r1 = static_cast<int>(min(static_cast<long long>(w.r0) + s.rows, static_cast<long long>(s.n_nodes)));
  w.tiles = (w.r1 - w.r0 + ring.tile_rows - 1) / ring.tile_rows;
  const int held = min(w.tiles, ring.slots);

  if (threadIdx.x >= kThreads) {   // the copying warp
    if (lane == 0) {
      for (int k = 0; k < ring.slots; ++k) {
        tc::mbar_init(&sh.full[k], kStreams + 1);
        tc::mbar_init(&sh.empty[k], kWarps);
        sh.copies[k] = 0;
      }
      tc::mbar_init(&sh.gate, kWarps);
      sh.abort = 0;
      if (blockIdx.x == 0) *p.err = 0;
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
    for (int k = 0; k < held; ++k) {
      const int t0 = w.r0 + k * ring.tile_rows;
      copy_tile<kStreams>(p, &sh, smem, k, t0, min(t0 + ring.tile_rows, w.r1));
    }
    __syncthreads();
    End last{-1, 0, 0, -1};
    bool ok = true;
    int ended = 0;
    Turn turn{0, 1};
    for (int k = 0; k < w.tiles; ++k) {
      const int t0 = w.r0 + k * ring.tile_rows, t1 = min(t0 + ring.tile_rows, w.r1);
      if (k >= held) {
        ok = tc::warp_wait(&sh.empty[turn.slot], turn.parity, &sh.abort, p.err, 1);
        if (!ok) break;
        copy_tile<kStreams>(p, &sh, smem, turn.slot, t0, t1);
      }
      describe_tile(p, w, &sh, smem, turn.slot, t0, t1, &last, &ended);
      turn.next(ring.slots);
    }
    __syncthreads();
    if (gridDim.x > 1) cg::this_grid().sync();
    last.structure = -1;
    ended = 0;
    if (p.out)
      for (int k = w.tiles - held - 1; k >= 0 && ok; --k) {
        const int t0 = w.r0 + k * ring.tile_rows, t1 = t0 + ring.tile_rows;
        turn = turn_of(ring, w.tiles, k, true);
        ok = tc::warp_wait(&sh.empty[turn.slot], turn.parity ^ 1u, &sh.abort, p.err, 1);
        if (!ok) break;
        copy_tile<kStreams>(p, &sh, smem, turn.slot, t0, t1);
        describe_tile(p, w, &sh, smem, turn.slot, t0, t1, &last, &ended);
      }
    // the warps that compute wait for every copy, unless one of them gave up
    if (!ok || *static_cast<volatile int*>(&sh.abort))
      for (int k = 0; k < ring.slots; ++k)
        if (sh.copies[k] > 0) tc::mbar_wait_drain(&sh.full[k], (sh.copies[k] - 1) & 1);
    return;
  }

  if (threadIdx.x < 32) {
    int first, behind, head = -1, tail = -1;
    ended_by(s, w.r0, w.r1, &first, &behind);
    if (first < s.n_structs) {
      const int lo = begin_of(s, first);
      if (lo < w.r1 && (lo < w.r0 || end_of(s, first) > w.r1)) head = first;
    }
    if (behind < s.n_structs && behind != head && begin_of(s, behind) < w.r1) tail = behind;
    if (lane == 0) {
      sh.first = first;
      sh.behind = behind;
      sh.head = head;
      sh.tail = tail;
    }
  }
  Place at;
  at.row = threadIdx.x / s.cv;
  at.col = (threadIdx.x - at.row * s.cv) * V;
  if (at.row >= s.rp) at.col = 0;
  at.g = at.col / s.cg;
  // bytes of a value in each stream; a row's scales are indexed from its first
  int elem[kStreams];
#pragma unroll
  for (int k = 0; k < kStreams; ++k) elem[k] = k < 2 ? ring.row_bytes[k] / (Op::K * s.channels) : 0;
  char* acc = smem + ring.o_acc;
  double* sum = reinterpret_cast<double*>(smem + ring.o_sum);
  float* edge = reinterpret_cast<float*>(smem + ring.o_edge);
  const int2* rows = reinterpret_cast<const int2*>(smem + ring.o_rows);
  const End* ends = reinterpret_cast<const End*>(smem + ring.o_ends);
  // this thread's channels of row t0 of a tile
  auto sources = [&](int slot, int t0, const char* (&src)[kStreams]) {
    const char* base = smem + ring.o_ring + static_cast<size_t>(slot) * ring.slot_bytes;
#pragma unroll
    for (int k = 0; k < kStreams; ++k)
      src[k] = base + ring.off[k] + ((static_cast<unsigned>(t0) * static_cast<unsigned>(ring.row_bytes[k])) & 15u) +
               at.col * elem[k];
  };
  Op op(p, at);
  // structures without rows have zero statistics
  if (!Op::kBackward && s.ptr)
    for (long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i < s.n_structs;
         i += static_cast<long long>(gridDim.x) * kThreads)
      if (begin_of(s, static_cast<int>(i)) >= end_of(s, static_cast<int>(i)))
        for (int k = 0; k < nq; ++k) p.table[i * nq + k] = 0.0f;
  __syncthreads();

  int step[kStreams];
#pragma unroll
  for (int k = 0; k < kStreams; ++k) step[k] = s.rp * ring.row_bytes[k];
  auto leave = [&](int row) {
    op.leave(acc + static_cast<size_t>((row - w.r0) % ring.acc_rows) * ring.acc_bytes, s.cv, at.col / V);
    op.clear();
  };
  // A slot is free once the structures that end in its tile are summed up: no warp can then be so far
  // ahead that it overwrites what the threads left. Where the ring is shorter than the block's rows, half
  // of it waits for that while the other half is read.
  const int half = ring.slots / 2;
  int current = -1, released = 0, closed = 0, ended = 0;
  int n = at.row < s.rp ? w.r0 + at.row : INT_MAX;
  Turn turn{0, 0}, release{0, 0};
  Gate gate;
  for (int tile = 0; tile < w.tiles; ++tile) {
    const int slot = turn.slot, t0 = w.r0 + tile * ring.tile_rows, t1 = min(t0 + ring.tile_rows, w.r1);
    if (!tc::warp_wait(&sh.full[slot], turn.parity, &sh.abort, p.err, 2)) break;
    const int4 about = sh.tile[slot];
    if (n < t1) {
      const char* src[kStreams];
      sources(slot, t0, src);
#pragma unroll
      for (int k = 0; k < kStreams; ++k) src[k] += (n - t0) * ring.row_bytes[k];
      if (about.x != kMixed) {
        if (about.x != current) {
          current = about.x;
          op.enter_up(p, at, current);
        }
        do {
          op.add(p, at, src, at.col);
          n += s.rp;
#pragma unroll
          for (int k = 0; k < kStreams; ++k) src[k] += step[k];
        } while (n < t1);
        if (n >= about.y) leave(n - s.rp);
      } else {
        for (; n < t1; n += s.rp) {
          const int2 e = rows[slot * ring.tile_rows + n - t0];
          if (e.x >= 0) {
            if (e.x != current) {
              current = e.x;
              op.enter_up(p, at, current);
            }
            op.add(p, at, src, at.col);
            if (n + s.rp >= e.y) leave(n);
          }
#pragma unroll
          for (int k = 0; k < kStreams; ++k) src[k] += step[k];
        }
      }
    }
    ended = about.z;
    turn.next(ring.slots);
    if (released < w.tiles - ring.slots && (ended == closed || tile - released + 1 >= half)) {
      if (ended > closed) {
        if (!gate.meet(&sh, p.err)) break;
        close<Op>(p, w, acc, ends, closed, ended);
        closed = ended;
      }
      __syncwarp();
      for (; released <= tile && released < w.tiles - ring.slots; ++released) {
        tc::mbar_arrive_lane0(&sh.empty[release.slot], lane);
        release.next(ring.slots);
      }
    }
  }
  meet_compute();
  if (!*static_cast<volatile int*>(&sh.abort) && ended > closed) close<Op>(p, w, acc, ends, closed, ended);
  if constexpr (Op::kBackward) {
    // the block's channel sums, over the rows it reads side by side
    float* flat = reinterpret_cast<float*>(sum);
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      meet_compute();
#pragma unroll
      for (int k = 0; k < V; ++k) flat[threadIdx.x * V + k] = op.own[q][k];
      meet_compute();
      for (int i = threadIdx.x; i < s.channels; i += kThreads) {
        float t = 0.0f;
        for (int r = 0; r < s.rp; ++r) t += flat[r * s.channels + i];
        p.chan[(static_cast<size_t>(blockIdx.x) * Q + q) * s.channels + i] = t;
      }
    }
  }
  __syncthreads();
  if (gridDim.x > 1) cg::this_grid().sync();
  if (sh.abort) return;

  if constexpr (Op::kBackward) {
    // dw and db: 8 sums at a time, the other threads of a sum take its blocks in turn
    for (int base = blockIdx.x * 8; base < Q * s.channels; base += gridDim.x * 8) {
      const int i = base + (threadIdx.x & 7), k = threadIdx.x >> 3;
      double t = 0.0;
      if (i < Q * s.channels)
        for (int b = k; b < gridDim.x; b += kThreads / 8) t += p.chan[static_cast<size_t>(b) * Q * s.channels + i];
      sum[threadIdx.x] = t;
      meet_compute();
      if (k == 0 && i < Q * s.channels) {
        t = 0.0;
        for (int j = 0; j < kThreads / 8; ++j) t += sum[j * 8 + threadIdx.x];
        const int q = i / s.channels;
        if (q == 0 && p.grad_bias) p.grad_bias[i] = static_cast<float>(t);
        if (q > 0 && p.grad_weight) p.grad_weight[i - s.channels] = static_cast<float>(t);
      }
      meet_compute();
    }
    if (!p.out) return;
  }
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    const int i = k ? sh.tail : sh.head;
    if (i < 0) continue;
    const int lo = begin_of(s, i), hi = end_of(s, i);
    gather_partials(s, p.part, nq, lo, hi, sum, sum + kThreads);
    const double* all = sum + kThreads;
    for (int j = threadIdx.x; j < nq - s.groups; j += kThreads) {
      const int l = j / s.groups, g = j - l * s.groups;
      const float2 v = Op::value(p, l, hi - lo, all[g], all[s.groups + j]);
      float* to = edge + k * nq;
      if (l == 0) to[g] = v.x;
      to[s.groups + j] = v.y;
      if (!Op::kBackward && lo >= w.r0) {
        to = p.table + static_cast<size_t>(i) * nq;
        if (l == 0) to[g] = v.x;
        to[s.groups + j] = v.y;
      }
    }
  }
  meet_compute();

  current = -1;
  // the last row of this thread
  n = at.row < s.rp && at.row < w.r1 - w.r0 ? w.r0 + at.row + (w.r1 - w.r0 - 1 - at.row) / s.rp * s.rp : -1;
  turn = turn_of(ring, w.tiles, w.tiles - 1, false);
  for (int tile = w.tiles - 1; tile >= 0; --tile) {
    const int slot = turn.slot, t0 = w.r0 + tile * ring.tile_rows;
    if (tile < w.tiles - ring.slots &&
        !tc::warp_wait(&sh.full[slot], turn_of(ring, w.tiles, tile, true).parity, &sh.abort, p.err, 2))
      return;
    if (n >= t0) {
      const int about = sh.tile[slot].x;
      const char* src[kStreams];
      sources(slot, t0, src);
#pragma unroll
      for (int k = 0; k < kStreams; ++k) src[k] += (n - t0) * ring.row_bytes[k];
      auto enter = [&](int i) {
        if (i != current) {
          current = i;
          op.enter_down(p, at, i, i == sh.head ? edge : i == sh.tail ? edge + nq : p.table + static_cast<size_t>(i) * nq);
        }
      };
      if (about != kMixed) {
        enter(about);
        do {
          op.put(p, at, src, at.col, n, true);
          n -= s.rp;
#pragma unroll
          for (int k = 0; k < kStreams; ++k) src[k] -= step[k];
        } while (n >= t0);
      } else {
        for (; n >= t0; n -= s.rp) {
          const int i = rows[slot * ring.tile_rows + n - t0].x;
          if (i >= 0) enter(i);
          if (i >= 0 || op.wants_outside(p)) op.put(p, at, src, at.col, n, i >= 0);
#pragma unroll
          for (int k = 0; k < kStreams; ++k) src[k] -= step[k];
        }
      }
    }
    if (tile >= ring.slots) {
      __syncwarp();
      tc::mbar_arrive_lane0(&sh.empty[slot], lane);
    }
    if (--turn.slot < 0) turn.slot = ring.slots - 1;
  }
}

// ---------------------------------------------------------------- launch

int vector_width(int channels, int groups) {
  return channels % 4 == 0 && (channels / groups) % 4 == 0 ? 4 : 1;
}

int round_up(int v, int to) { return (v + to - 1) / to * to; }

// Shared memory of a call: the sums, and slots with their tables and places for sums in what is left.
bool plan_ring(const Shape& s, int q, int acc_thread, const int (&row_bytes)[kMaxStreams], Ring* r) {
  int per_row = 0;
  for (int k = 0; k < kMaxStreams; ++k) per_row += row_bytes[k];
  r->tile_rows = kTileBytes / per_row;
  if (r->tile_rows < 1) r->tile_rows = 1;
  if (r->tile_rows > kMaxTileRows) r->tile_rows = kMaxTileRows;
  int at = 0, in_slot = 0;
  for (int k = 0; k < kMaxStreams; ++k) {
    r->row_bytes[k] = row_bytes[k];
    r->off[k] = in_slot;
    if (row_bytes[k]) in_slot += round_up(row_bytes[k] * r->tile_rows + 32, 128);
  }
  r->slot_bytes = in_slot;
  r->acc_bytes = round_up(acc_thread * s.cv, 8);
  const int nq = q * s.groups;
  r->o_sum = at;
  at += round_up((kThreads + (nq > kThreads ? nq : kThreads)) * static_cast<int>(sizeof(double)), 128);
  r->o_edge = at;
  at += round_up(2 * nq * static_cast<int>(sizeof(float)), 128);
  const int row_cost = r->acc_bytes + static_cast<int>(sizeof(int2) + sizeof(End));
  r->slots = (kSmem - 512 - at - s.rp * r->acc_bytes) / (in_slot + r->tile_rows * row_cost);
  if (r->slots > kMaxSlots) r->slots = kMaxSlots;
  if (r->slots < 2) return false;
  r->acc_rows = r->slots * r->tile_rows + s.rp;
  r->o_acc = at;
  at += round_up(r->acc_rows * r->acc_bytes, 128);
  r->o_rows = at;
  at += round_up(r->slots * r->tile_rows * static_cast<int>(sizeof(int2)), 128);
  r->o_ends = at;
  at += round_up(r->slots * r->tile_rows * static_cast<int>(sizeof(End)), 128);
  r->o_ring = at;
  r->bytes = at + r->slots * r->slot_bytes;
  return true;
}

Shape shape_of(const Call& c, int width) {
  Shape s;
  s.n_nodes = c.n_nodes;
  s.n_structs = c.n_structs;
  s.rows = 0;
  s.channels = c.channels;
  s.groups = c.groups;
  s.cg = c.channels / c.groups;
  s.cv = c.channels / width;
  s.rp = kThreads / s.cv;
  s.ptr = c.node_ptr;
  return s;
}

template <class Op, int V>
etp_status launch(const Call& c, Args& p, const int (&row_bytes)[kMaxStreams], cudaStream_t stream, const char* what) {
  auto kernel = k_norm<Op, V>;
  p.s = shape_of(c, V);
  if (!plan_ring(p.s, Op::Q, Op::kAcc, row_bytes, &p.ring)) {
    set_error(std::string(what) + ": rows too long");
    return ETP_ERR_UNSUPPORTED;
  }
  // what the device says about a kernel and a size of shared memory is asked for once in a row
  static thread_local int known_dev = -1, known_bytes = 0, sms = 0, per_sm = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev != known_dev || p.ring.bytes != known_bytes)) {
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kBlock, p.ring.bytes);
    known_dev = e == cudaSuccess ? dev : -1;
    known_bytes = p.ring.bytes;
  }
  if (e != cudaSuccess) return cuda_status(e, what);
  // A block for every rp rows at most, and no more blocks than run at once: the grid barrier needs
  // them all on the device.
  long long blocks = (static_cast<long long>(c.n_nodes) + p.s.rp - 1) / p.s.rp;
  long long resident = static_cast<long long>(per_sm) * sms;
  if (resident > kMaxBlocks) resident = kMaxBlocks;
  if (blocks > resident) blocks = resident;
  if (blocks < 1) blocks = 1;
  p.s.rows = static_cast<int>((c.n_nodes + blocks - 1) / blocks);
  blocks = (static_cast<long long>(c.n_nodes) + p.s.rows - 1) / p.s.rows;
  void* args[] = {&p};
  const dim3 grid(static_cast<unsigned>(blocks)), block(kBlock);
  const void* fn = reinterpret_cast<const void*>(kernel);
  if (blocks == 1) e = cudaLaunchKernel(fn, grid, block, args, p.ring.bytes, stream);
  else e = cudaLaunchCooperativeKernel(fn, grid, block, args, p.ring.bytes, stream);
  return cuda_status(e, what);
}

template <class T, int L, int V>
etp_status fwd_launch(const Call& c, Args& p, cudaStream_t s) {
  const int row_bytes[kMaxStreams] = {Fwd<T, L, V>::K * c.channels * static_cast<int>(sizeof(T)), 0, 0};
  return launch<Fwd<T, L, V>, V>(c, p, row_bytes, s, "group norm launch");
}
template <class T, int L, int V, bool kKept>
etp_status bwd_launch(const Call& c, Args& p, cudaStream_t s) {
  const int dim = Bwd<T, L, V, kKept>::K * c.channels, size = static_cast<int>(sizeof(T));
  const int row_bytes[kMaxStreams] = {dim * size, kKept ? dim : dim * size, kKept ? (dim + kCkptBlock - 1) / kCkptBlock : 0};
  return launch<Bwd<T, L, V, kKept>, V>(c, p, row_bytes, s, "group norm backward launch");
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
template <class T, int V, bool kKept>
etp_status bwd_rank(const Call& c, Args& p, cudaStream_t s) {
  switch (c.lmax) {
    case 0: return bwd_launch<T, 0, V, kKept>(c, p, s);
    case 1: return bwd_launch<T, 1, V, kKept>(c, p, s);
    case 2: return bwd_launch<T, 2, V, kKept>(c, p, s);
    default: return bwd_launch<T, 3, V, kKept>(c, p, s);
  }
}
template <class T>
etp_status fwd_type(const Call& c, Args& p, int width, cudaStream_t s) {
  return width == 4 ? fwd_rank<T, 4>(c, p, s) : fwd_rank<T, 1>(c, p, s);
}
template <class T>
etp_status bwd_type(const Call& c, Args& p, bool kept, int width, cudaStream_t s) {
  if (kept) return width == 4 ? bwd_rank<T, 4, true>(c, p, s) : bwd_rank<T, 1, true>(c, p, s);
  return width == 4 ? bwd_rank<T, 4, false>(c, p, s) : bwd_rank<T, 1, false>(c, p, s);
}

// workspace: [error word][partial sums][means per structure][channel sums per block], the last two
// for the backward
size_t partial_bytes(const Call& c) {
  return align256(static_cast<size_t>(kMaxBlocks) * 2 * (c.lmax + 2) * c.groups * sizeof(double));
}
size_t mean_bytes(const Call& c) {
  return align256(static_cast<size_t>(c.n_structs) * (c.lmax + 2) * c.groups * sizeof(float));
}

__global__ void k_check_ptr(const int* ptr, int n_structs, int n_nodes, int* flag) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i > n_structs) return;
  const int v = ptr[i];
  if (v < 0 || v > n_nodes || (i < n_structs && ptr[i + 1] < v)) *flag = 1;
}

// Waits for the stream and reads the int at the start of the workspace.
etp_status read_flag(void* ws, int* value, cudaStream_t s, const char* what) {
  cudaError_t e = cudaMemcpyAsync(value, ws, sizeof(int), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  return e == cudaSuccess ? ETP_OK : cuda_status(e, what);
}

}  // namespace

etp_status validate(const Call& c, void* ws, cudaStream_t s) {
  if (!c.node_ptr) return ETP_OK;
  cudaError_t e = cudaMemsetAsync(ws, 0, sizeof(int), s);
  if (e == cudaSuccess) {
    k_check_ptr<<<c.n_structs / 256 + 1, 256, 0, s>>>(c.node_ptr, c.n_structs, c.n_nodes, static_cast<int*>(ws));
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return cuda_status(e, "node_ptr validation");
  int bad = 0;
  etp_status st = read_flag(ws, &bad, s, "node_ptr validation");
  if (st != ETP_OK || !bad) return st;
  set_error("node_ptr must be ascending and stay within [0, n_nodes]");
  return ETP_ERR_BAD_GRAPH;
}

etp_status finished(void* ws, cudaStream_t s, const char* who) {
  int code = 0;
  etp_status st = read_flag(ws, &code, s, who);
  if (st != ETP_OK || !code) return st;
  set_error(std::string(who) + ": a bounded pipeline wait gave up (code " + std::to_string(code) + "); the output is incomplete");
  return ETP_ERR_CUDA;
}

bool supported(int lmax, int channels, int groups) {
  return lmax >= 0 && lmax <= kMaxL && channels >= 1 && groups >= 1 && groups <= kMaxGroups && channels % groups == 0 &&
         channels / vector_width(channels, groups) <= kMaxVectors && channels * (lmax + 1) * (lmax + 1) <= kGenMaxDim;
}

size_t workspace_bytes(const Call& c, bool backward) {
  size_t n = 256 + partial_bytes(c);
  if (backward) n += mean_bytes(c) + align256(static_cast<size_t>(kMaxBlocks) * (c.lmax + 2) * c.channels * sizeof(float));
  return n;
}

etp_status forward(const Call& c, const void* x, const float* weight, const float* bias, float eps, void* out,
                   float* stats, etp_ckpt_format format, uint8_t* q, uint8_t* scale, void* ws, cudaStream_t s) {
  Args p{};
  p.ring.src[0] = static_cast<const char*>(x);
  p.weight = weight;
  p.bias = bias;
  p.eps = eps;
  p.act = c.activation;
  p.zero_rest = c.zero_rest;
  p.out = out;
  p.table = stats;
  p.int8 = format == ETP_CKPT_INT8;
  p.err = static_cast<int*>(ws);
  p.part = reinterpret_cast<double*>(static_cast<char*>(ws) + 256);
  // the norm writes the checkpoint itself where no block of 32 crosses a component's end
  const bool fused = format != ETP_CKPT_NONE && c.channels % kCkptBlock == 0;
  p.q = fused ? q : nullptr;
  p.scale = fused ? scale : nullptr;
  if (format != ETP_CKPT_NONE && !fused) {
    const int dim = c.channels * (c.lmax + 1) * (c.lmax + 1);
    etp_status st = ckpt::store(format, c.dtype, c.n_nodes, dim, x, q, scale, s);
    if (st != ETP_OK) return st;
  }
  const int width = vector_width(c.channels, c.groups);
  switch (c.dtype) {
    case ETP_F32: return fwd_type<float>(c, p, width, s);
    case ETP_BF16: return fwd_type<__nv_bfloat16>(c, p, width, s);
    default: return fwd_type<__half>(c, p, width, s);
  }
}

etp_status backward(const Call& c, const void* x, etp_ckpt_format format, const uint8_t* q, const uint8_t* scale,
                    const float* stats, const float* weight, const float* bias, const void* grad_out, void* grad_x,
                    float* grad_weight, float* grad_bias, void* ws, cudaStream_t s) {
  const bool kept = format != ETP_CKPT_NONE;
  Args p{};
  p.ring.src[0] = static_cast<const char*>(grad_out);
  p.ring.src[1] = kept ? reinterpret_cast<const char*>(q) : static_cast<const char*>(x);
  p.ring.src[2] = reinterpret_cast<const char*>(scale);
  p.int8 = format == ETP_CKPT_INT8;
  p.stats_in = stats;
  p.weight = weight;
  p.bias = bias;
  p.act = c.activation;
  p.zero_rest = c.zero_rest;
  p.out = grad_x;
  p.grad_weight = grad_weight;
  p.grad_bias = grad_bias;
  p.err = static_cast<int*>(ws);
  char* at = static_cast<char*>(ws) + 256;
  p.part = reinterpret_cast<double*>(at);
  p.table = reinterpret_cast<float*>(at += partial_bytes(c));
  p.chan = reinterpret_cast<float*>(at + mean_bytes(c));
  const int width = vector_width(c.channels, c.groups);
  switch (c.dtype) {
    case ETP_F32: return bwd_type<float>(c, p, kept, width, s);
    case ETP_BF16: return bwd_type<__nv_bfloat16>(c, p, kept, width, s);
    default: return bwd_type<__half>(c, p, kept, width, s);
  }
}

}  // namespace norm
}  // namespace etp
