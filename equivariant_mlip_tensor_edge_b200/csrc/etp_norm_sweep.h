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
// on behind) leaves partial sums, which meet after the grid barrier between the sweeps. The forward keeps
// its sums in 64 bits, but for a row's squares of l > 0 and a thread's sum of them as it is passed on. The
// backward adds in 32 bits within a block, a thread's rows and then the threads (joining the threads in 64
// bits took the backward of 4000 structures from 24.4 to 25.9 us), and in 64 from block to block. Every
// sum has one order, so equal calls give equal bits.
//
// A thread holds V neighbouring channels (V = 4, 2 or 1, as the group size divides by it) of every rp-th
// row and walks the row's components, so a channel's gate stays in its thread. Sums stay in
// the thread's registers until its last row of a structure, which leaves them in shared memory. The
// warps meet to add them up once for the rows that the ring holds, not at every structure's end.
//
// Measured on one B200 (148 SMs, 6449 GB/s copy rate), times of the kernel alone: 32768 rows of 9 x 128
// float32, one structure, forward: 75 us for 302 MB read and written once, 62 % of the copy rate. In a
// chain of calls 382 MB cross DRAM: 231 read (the ring and L2 spare 71 of the second sweep's 151 MB), 151
// written, part of it during the next call. 8 structures of 1000 rows of 16 x 128 float32, backward from
// int8: 44 us, 53 %. Small calls are bound by the chain launch - first tile - sums - grid barrier -
// outputs: 21 rows 6.7 us, 1000 rows of 576 backward 12.3 us. Between, by the warps' dependent
// instructions: 15 warps an SM issue in 25 to 47 % of the cycles (twice as many with half the registers were
// 5 to 24 % slower).
#pragma once

#include <cooperative_groups.h>

#include <algorithm>
#include <climits>
#include <string>

#include "etp_checkpoint.h"
#include "etp_internal.h"
#include "etp_norm.h"
#include "etp_tc_common.h"

namespace cg = cooperative_groups;

namespace etp {
namespace norm {

constexpr int kThreads = 480;             // that compute; a further warp copies
constexpr int kBlock = kThreads + 32;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxSlots = 16;
constexpr int kMaxTileRows = 256;
// Aim of a tile with its tables, three slots or more: fewer turns for the warps than with 24 KB (60001
// rows of 252 bfloat16 28 us for 38, 8 cells of 1000 atoms backward 44 for 46).
constexpr int kTileBytes = 64 * 1024;
constexpr int kMaxStreams = 3;
// What L2 (126 MB) is to hold for the second sweep; rows before that, and outputs, are evicted first (151
// MB of rows: 75 us, without 77).
constexpr long long kL2Bytes = 90LL << 20;
constexpr int kSmem = 226 * 1024;         // dynamic, of the 227 KB that a block can have

// Division by a number known at launch, for n d below 2^32: a multiplication (an integer division takes
// some 200 cycles, and most are on the way of the whole block).
struct Div {
  int d;
  unsigned m;
  __device__ __forceinline__ int of(int n) const { return m ? static_cast<int>(__umulhi(n, m)) : n; }
};
inline Div div_by(int d) { return Div{d, d > 1 ? static_cast<unsigned>(((1ULL << 32) + d - 1) / d) : 0u}; }

struct Shape {
  int n_nodes, n_structs, rows;   // rows: a block's share
  int channels, cg;               // cg: channels of a group
  int cv, cvg, rp;                // vectors of a row's component, of a group; rows a block reads side by side
  Div groups, per;                // per: ranks times groups, the sums of a structure
  const int* ptr;                 // NULL: one structure of all rows
};

// Shared memory: ring slots of tile_rows rows of every stream, tables for the rows and the structure
// ends of each slot's tile, and the threads' sums at their last rows of a structure. Those are kept by
// row, in a ring as long as the rows that warps can be apart.
struct Ring {
  int tile_rows, slots, slot_bytes, acc_rows, acc_bytes;
  int tiles, tiles_last;          // of a block, of the last block
  int l2_tiles;                   // of a block's, that L2 can hold until the sweep down
  int off[kMaxStreams], elem[kMaxStreams];   // elem: bytes of a value; 0 for scales, indexed by value
  int o_rows, o_ends, o_sum, o_edge, o_acc, o_ring, bytes;
  const char* src[kMaxStreams];
  int row_bytes[kMaxStreams];        // 0: stream not used
};

// A structure's end inside a block's rows: n rows of it lie in the block, and the places for sums of its
// last rows end before `place`. slot < 0: all of it is here; 0 / 1: it began before / goes on behind, and
// its sums are partial.
struct alignas(16) End {
  int structure, n, place, slot;
};

__device__ __forceinline__ int clamp_row(const Shape& s, int v) { return min(max(v, 0), s.n_nodes); }
__device__ __forceinline__ int begin_of(const Shape& s, int i) { return s.ptr ? clamp_row(s, __ldg(s.ptr + i)) : 0; }
__device__ __forceinline__ int end_of(const Shape& s, int i) {
  return s.ptr ? clamp_row(s, __ldg(s.ptr + i + 1)) : s.n_nodes;
}

// Numbers of structures that end at or before rows ra <= rb, by one warp: every round probes 32 places
// for each.
static __device__ void ended_by(const Shape& s, int ra, int rb, int* na, int* nb) {
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
  // the structures that cross the block's first / last row (-1: none), their rows, and the blocks that
  // hold them, the first of which writes what concerns all
  int edge[2], edge_n[2], from_block[2], to_block[2];
};
constexpr int kMixed = -2;

// Parities of the barriers of all slots, as a waiting warp goes through them.
struct Phases {
  uint32_t bits = 0;
  __device__ __forceinline__ uint32_t of(int slot) const { return (bits >> slot) & 1u; }
  __device__ __forceinline__ void pass(int slot) { bits ^= 1u << slot; }
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
  } else if constexpr (V == 2) {
    union { typename Pair<sizeof(T)>::type u; T h[2]; } t;
    t.u = *reinterpret_cast<const typename Pair<sizeof(T)>::type*>(p);
    v[0] = to_f32<T>(t.h[0]);
    v[1] = to_f32<T>(t.h[1]);
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

etp_status launch_forward(const Call& c, Args& p, int width, cudaStream_t s);
etp_status launch_backward(const Call& c, Args& p, bool kept, int width, cudaStream_t s);

// A thread's place: its first row of rp, its channels, their group
struct Place {
  int row, col, g;
};

// ---------------------------------------------------------------- the two sweeps

struct Work {
  int r0, r1, tiles;
};

// A bulk copy of data that nobody reads again soon: first to leave L2.
__device__ __forceinline__ void bulk_g2s_once(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  uint64_t policy;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
                   tc::sptr(dst)),
               "l"(src), "r"(bytes), "r"(tc::sptr(bar)), "l"(policy)
               : "memory");
}

// Bytes that rows [t0, t1) of an array of n_rows rows take: [a, b) by a bulk copy, in whole units of 16, and
// [b, e), if any, by hand: bytes of the array behind its last whole unit.
struct TileBytes {
  size_t a, b, e;
};
__host__ __device__ inline TileBytes tile_bytes(int t0, int t1, int n_rows, int row_bytes) {
  const size_t unit = 15, rb = static_cast<size_t>(row_bytes), whole = (n_rows * rb) & ~unit;
  TileBytes t;
  t.a = (t0 * rb) & ~unit;
  t.e = t1 * rb;
  t.b = (t.e + unit) & ~unit;
  if (t.b > whole) t.b = whole;
  if (t.b < t.a) t.b = t.a;
  return t;
}
// Whether that can leave bytes to copy by hand: not with 16 rows or more behind the tile.
__host__ __device__ inline bool near_end(int t1, int n_rows) { return n_rows - t1 < 16; }

// Starts a tile's copies into its slot, a lane to a stream, and does those by hand. once: it will not be
// found in L2 again.
template <int kStreams>
__device__ __forceinline__ void copy_tile(const Args& p, Shared* sh, char* smem, int slot, int t0, int t1, bool once) {
  const Ring& ring = p.ring;
  const int lane = threadIdx.x & 31;
  char* dst = smem + ring.o_ring + static_cast<size_t>(slot) * ring.slot_bytes;
  if (lane < kStreams) {
    const TileBytes t = tile_bytes(t0, t1, p.s.n_nodes, ring.row_bytes[lane]);
    const uint32_t bytes = static_cast<uint32_t>(t.b - t.a);
    tc::mbar_expect_tx(&sh->full[slot], bytes);
    if (bytes && once) bulk_g2s_once(dst + ring.off[lane], ring.src[lane] + t.a, bytes, &sh->full[slot]);
    else if (bytes) tc::bulk_g2s(dst + ring.off[lane], ring.src[lane] + t.a, bytes, &sh->full[slot]);
    if (lane == 0) ++sh->copies[slot];
  }
  if (near_end(t1, p.s.n_nodes)) {
#pragma unroll
    for (int k = 0; k < kStreams; ++k) {
      const TileBytes t = tile_bytes(t0, t1, p.s.n_nodes, ring.row_bytes[k]);
      if (t.b + lane < t.e) dst[ring.off[k] + (t.b - t.a) + lane] = ring.src[k][t.b + lane];
    }
    tc::fence_proxy_async();   // before a later bulk copy into the same bytes
  }
}

// What describe_tile knows from tile to tile: the structure found last, which covers whole tiles of a
// large one, and how many ended (their number, and its place in the ring of ends).
struct Seen {
  int structure = -1, a = 0, b = 0, slot = -1;
  int ended = 0, at = 0;
};

// Writes the tables of a tile: the structure of every row, and the structures that end here. place: that
// of the tile's first row for sums.
__device__ __forceinline__ void describe_tile(const Args& p, const Work& w, Shared* sh, char* smem, int slot, int t0,
                                              int t1, int place, Seen* seen) {
  const Shape& s = p.s;
  const Ring& ring = p.ring;
  const int lane = threadIdx.x & 31;
  End* ends = reinterpret_cast<End*>(smem + ring.o_ends);
  const int room = ring.slots * ring.tile_rows;
  auto write_end = [&](int number, const Seen& e) {
    int at = seen->at + number, end = place + e.b - t0;
    if (at >= room) at -= room;
    if (end >= ring.acc_rows) end -= ring.acc_rows;
    ends[at] = End{e.structure, e.b - e.a, end, e.slot};
  };
  if (seen->structure >= 0 && seen->a <= t0 && seen->b >= t1) {
    const int n_ends = seen->b == t1;
    if (lane == 0) {
      if (n_ends) write_end(0, *seen);
      sh->tile[slot] = make_int4(seen->structure, seen->b, seen->ended + n_ends, 0);
    }
    seen->ended += n_ends;
    seen->at += n_ends;
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
      Seen e;
      if (n < t1 && lo < s.n_structs) {
        const int sa = begin_of(s, lo), sb = end_of(s, lo);
        if (sa <= n && n < sb) {
          e.structure = lo;
          e.a = max(sa, w.r0);
          e.b = min(sb, w.r1);
          e.slot = sa < w.r0 ? 0 : sb > w.r1 ? 1 : -1;
        }
      }
      const bool ends_here = e.structure >= 0 && e.b == n + 1;
      const unsigned votes = __ballot_sync(0xffffffffu, ends_here);
      if (n < t1) rows[n - t0] = make_int2(e.structure, e.b);
      if (ends_here) write_end(__popc(votes & ((1u << lane) - 1u)), e);
      seen->ended += __popc(votes);
      seen->at += __popc(votes);
      if (seen->at >= room) seen->at -= room;
      const int from = min(31, t1 - 1 - base);
      seen->structure = __shfl_sync(0xffffffffu, e.structure, from);
      seen->a = __shfl_sync(0xffffffffu, e.a, from);
      seen->b = __shfl_sync(0xffffffffu, e.b, from);
      seen->slot = __shfl_sync(0xffffffffu, e.slot, from);
    }
    const bool one = seen->structure >= 0 && seen->a <= t0;   // and it reaches to the last row
    if (lane == 0) sh->tile[slot] = make_int4(one ? seen->structure : kMixed, seen->b, seen->ended, 0);
  }
  if (seen->at >= room) seen->at -= room;
  __syncwarp();
  tc::mbar_arrive_lane0(&sh->full[slot], lane);
}

// The sums of `count` ended structures, from place `from` of the ring of ends on, by all warps, from the
// threads' sums at their last rows (the last rp rows of a structure hold one of every thread): 2^lg lanes
// to a group and rank, then the statistics, or partial sums where the structure crosses blocks.
template <class Op>
__device__ __forceinline__ void close(const Args& p, const char* acc, const End* ends, int from, int count) {
  using Sum = typename Op::Sum;
  const Shape& s = p.s;
  const int G = s.groups.d, nq = s.per.d + G, lane = threadIdx.x & 31;
  const int items = count * s.per.d, room = p.ring.slots * p.ring.tile_rows;
  int lg = 0;
  while (lg < 5 && (items << (lg + 1)) <= kThreads) ++lg;
  const int parts = 1 << lg, part = lane & (parts - 1);
#pragma unroll 1
  for (int base = (threadIdx.x >> 5) << (5 - lg); base < items; base += kThreads >> lg) {
    const int it = base + (lane >> lg);
    Sum a0 = 0, a1 = 0, b0 = 0, b1 = 0;     // two chains each: a sum waits for its last addend, not for its loads
    End e{-1, 0, 0, -1};
    int l = 0, g = 0;
    if (it < items) {
      const int k = s.per.of(it), i = it - k * s.per.d;
      int at = from + k;
      if (at >= room) at -= room;
      e = ends[at];
      l = s.groups.of(i);
      g = i - l * G;
      const int rows = min(s.rp, e.n);
      int place = e.place - rows + part;
      if (place < 0) place += p.ring.acc_rows;
      if (place >= p.ring.acc_rows) place -= p.ring.acc_rows;
#pragma unroll 1
      for (int r = part; r < rows; r += parts) {
        const char* row = acc + place * p.ring.acc_bytes;
        place += parts;
        if (place >= p.ring.acc_rows) place -= p.ring.acc_rows;
        int j = g * s.cvg;
#pragma unroll 1
        for (const int end = j + s.cvg - 1; j < end; j += 2) {
          if (l == 0) {
            a0 += Op::first(row, s.cv, j);
            b0 += Op::first(row, s.cv, j + 1);
          }
          a1 += Op::second(row, s.cv, l, j);
          b1 += Op::second(row, s.cv, l, j + 1);
        }
        if (s.cvg & 1) {
          if (l == 0) a0 += Op::first(row, s.cv, j);
          a1 += Op::second(row, s.cv, l, j);
        }
      }
    }
    double s0 = static_cast<double>(a0) + b0, s1 = static_cast<double>(a1) + b1;
#pragma unroll 1
    for (int o = parts / 2; o > 0; o /= 2) {
      s0 += __shfl_xor_sync(0xffffffffu, s0, o);
      s1 += __shfl_xor_sync(0xffffffffu, s1, o);
    }
    if (part == 0 && it < items) {
      if (e.slot < 0) {
        const float2 v = Op::value(p, l, e.n, s0, s1);
        float* at = p.table + static_cast<size_t>(e.structure) * nq + g;
        if (l == 0) at[0] = v.x;
        at[(1 + l) * G] = v.y;
      } else {
        double* at = p.part + (blockIdx.x * 2 + e.slot) * nq + g;
        if (l == 0) at[0] = s0;
        at[(1 + l) * G] = s1;
      }
    }
  }
}

// The statistics of the structures that cross this block's ends: the partial sums of all the blocks that
// hold their rows, in block order, some threads to a sum (the two structures' sums side by side).
template <class Op>
__device__ __forceinline__ void gather(const Args& p, const Shared& sh, double* red, double* sum, float* edge) {
  const Shape& s = p.s;
  const int G = s.groups.d, nq = s.per.d + G;
  const bool head = sh.edge[0] >= 0, tail = sh.edge[1] >= 0;
  if (!head && !tail) return;
  const int first = head ? 0 : 1, both = head && tail ? 2 : 1;
  const int width = nq * both;                      // sums to gather
#pragma unroll 1
  for (int base = 0; base < width; base += kThreads) {
    const int here = min(width - base, kThreads);
    int parts = 1;
    while (here * (parts + 1) <= kThreads && parts < 16) ++parts;
    int k = 0, j = threadIdx.x;                     // thread k of sum j
    while (j >= here && k < parts) {
      j -= here;
      ++k;
    }
    double t = 0.0;
    if (k < parts) {
      int i = base + j, e = first;
      if (i >= nq) {
        i -= nq;
        e = 1;
      }
      const int c0 = sh.from_block[e], c1 = sh.to_block[e];
      const double* from = p.part + i;
#pragma unroll 1
      for (int c = c0 + k; c <= c1; c += 12 * parts) {
        double v[12];
#pragma unroll
        for (int h = 0; h < 12; ++h) {
          const int b = c + h * parts;
          v[h] = b <= c1 ? from[(b * 2 + (b == c0)) * nq] : 0.0;
        }
#pragma unroll
        for (int h = 0; h < 12; ++h) t += v[h];
      }
      red[threadIdx.x] = t;
    }
    meet_compute();
    if (threadIdx.x < here) {
      for (int h = 1; h < parts; ++h) t += red[h * here + threadIdx.x];
      sum[base + threadIdx.x] = t;
    }
    meet_compute();
  }
#pragma unroll 1
  for (int k = first; k < 2; ++k) {
    const int structure = sh.edge[k];
    if (structure < 0) continue;
    const double* all = sum + (k - first) * nq;
#pragma unroll 1
    for (int j = threadIdx.x; j < s.per.d; j += kThreads) {
      const int l = s.groups.of(j), g = j - l * G;
      const float2 v = Op::value(p, l, sh.edge_n[k], all[g], all[G + j]);
      float* to = edge + k * nq;
      if (l == 0) to[g] = v.x;
      to[G + j] = v.y;
      if (!Op::kBackward && sh.from_block[k] == blockIdx.x) {
        to = p.table + static_cast<size_t>(structure) * nq;
        if (l == 0) to[g] = v.x;
        to[G + j] = v.y;
      }
    }
  }
  meet_compute();
}

template <class Op, int V>
__global__ void __launch_bounds__(kBlock, 1) k_norm(const __grid_constant__ Args p) {
  constexpr int Q = Op::Q, kStreams = Op::kStreams;
  extern __shared__ __align__(128) char smem[];
  __shared__ Shared sh;
  const Shape& s = p.s;
  const Ring& ring = p.ring;
  const int lane = threadIdx.x & 31;
  Work w;
  w.r0 = blockIdx.x * s.rows;
  w.r1 = blockIdx.x == gridDim.x - 1 ? s.n_nodes : w.r0 + s.rows;
  w.tiles = blockIdx.x == gridDim.x - 1 ? ring.tiles_last : ring.tiles;
  const int held = min(w.tiles, ring.slots), last_once = w.tiles - ring.slots - ring.l2_tiles;

  // The last warp copies, the others compute. All of them meet at the same three places: before the first
  // sweep, behind it, and at the grid barrier.
  const bool copies = threadIdx.x >= kThreads;
  if (copies) {
    if (lane < ring.slots) {
      tc::mbar_init(&sh.full[lane], kStreams + 1);
      tc::mbar_init(&sh.empty[lane], kWarps);
      sh.copies[lane] = 0;
    }
    if (lane == 0) {
      tc::mbar_init(&sh.gate, kWarps);
      sh.abort = 0;
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncwarp();
#pragma unroll 1
    for (int k = 0; k < held; ++k) {
      const int t0 = w.r0 + k * ring.tile_rows;
      copy_tile<kStreams>(p, &sh, smem, k, t0, min(t0 + ring.tile_rows, w.r1), k < last_once);
    }
  }

  if (threadIdx.x < 32) {
    int first, behind, edge[2] = {-1, -1};
    ended_by(s, w.r0, w.r1, &first, &behind);
    if (first < s.n_structs) {
      const int lo = begin_of(s, first);
      if (lo < w.r1 && (lo < w.r0 || end_of(s, first) > w.r1)) edge[0] = first;
    }
    if (behind < s.n_structs && behind != edge[0] && begin_of(s, behind) < w.r1) edge[1] = behind;
    if (lane == 0) {
      sh.first = first;
      sh.behind = behind;
    }
    if (lane < 2) {
      const int i = lane == 0 ? edge[0] : edge[1];
      sh.edge[lane] = i;
      if (i >= 0) {
        const int lo = begin_of(s, i), hi = end_of(s, i);
        sh.edge_n[lane] = hi - lo;
        sh.from_block[lane] = lo / s.rows;
        sh.to_block[lane] = (hi - 1) / s.rows;
      }
    }
  }
  Place at;
  at.row = threadIdx.x / s.cv;
  at.col = (threadIdx.x - at.row * s.cv) * V;
  if (at.row >= s.rp) at.col = 0;
  at.g = at.col / s.cg;
  char* acc = smem + ring.o_acc;
  double* sum = reinterpret_cast<double*>(smem + ring.o_sum);
  float* edge = reinterpret_cast<float*>(smem + ring.o_edge);
  const int2* rows = reinterpret_cast<const int2*>(smem + ring.o_rows);
  const End* ends = reinterpret_cast<const End*>(smem + ring.o_ends);
  // this thread's channels of row n of a tile
  auto sources = [&](int slot, int t0, int n, const char* (&src)[kStreams]) {
    const char* base = smem + ring.o_ring + slot * ring.slot_bytes;
#pragma unroll
    for (int k = 0; k < kStreams; ++k)
      src[k] = base + ring.off[k] + ((static_cast<unsigned>(t0) * static_cast<unsigned>(ring.row_bytes[k])) & 15u) +
               (n - t0) * ring.row_bytes[k] + at.col * ring.elem[k];
  };
  int step[kStreams];
#pragma unroll
  for (int k = 0; k < kStreams; ++k) step[k] = s.rp * ring.row_bytes[k];
  Op op(p, at);
  // structures without rows have zero statistics
  if (!Op::kBackward && s.ptr && !copies)
    for (long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i < s.n_structs;
         i += static_cast<long long>(gridDim.x) * kThreads)
      if (begin_of(s, static_cast<int>(i)) >= end_of(s, static_cast<int>(i)))
        for (int k = 0; k < s.per.d + s.groups.d; ++k) p.table[i * (s.per.d + s.groups.d) + k] = 0.0f;
  __syncthreads();

  // A slot is free once the structures that end in its tile are summed up: no warp can then be so far
  // ahead that it overwrites what the threads left. Where the ring is shorter than the block's rows, half
  // of it waits for that while the other half is read.
  const int half = ring.slots / 2, lost = w.tiles - ring.slots, room = ring.slots * ring.tile_rows;
  int current = -1, n = at.row < s.rp ? w.r0 + at.row : INT_MAX;
  int place = copies ? 0 : at.row;     // for sums: of the tile's first row, of row n
  int slot = 0, ended = 0, closed = 0, closed_at = 0, released = 0, released_slot = 0;
  Phases phases;                       // of the full slots, of the empty ones where this warp copies
  Gate gate;
  auto forward = [&](const char* (&src)[kStreams], int rows_done) {
    n += rows_done * s.rp;
    if ((place += rows_done * s.rp) >= ring.acc_rows) place -= ring.acc_rows;
#pragma unroll
    for (int k = 0; k < kStreams; ++k) src[k] += rows_done * step[k];
  };
  auto leave = [&](int where) {
    op.leave(acc + where * ring.acc_bytes, s.cv, at.col / V);
    op.clear();
  };
  if (copies) {
    Seen seen;
#pragma unroll 1
    for (int k = 0; k < w.tiles; ++k) {
      const int t0 = w.r0 + k * ring.tile_rows, t1 = min(t0 + ring.tile_rows, w.r1);
      if (k >= held) {
        if (!tc::warp_wait(&sh.empty[slot], phases.of(slot), &sh.abort, p.err, 1)) break;
        phases.pass(slot);
        copy_tile<kStreams>(p, &sh, smem, slot, t0, t1, k < last_once);
      }
      describe_tile(p, w, &sh, smem, slot, t0, t1, place, &seen);
      if (++slot == ring.slots) slot = 0;
      if ((place += ring.tile_rows) >= ring.acc_rows) place -= ring.acc_rows;
    }
  } else {
#pragma unroll 1
    for (int tile = 0; tile < w.tiles; ++tile) {
      const int t0 = w.r0 + tile * ring.tile_rows, t1 = min(t0 + ring.tile_rows, w.r1);
      if (!tc::warp_wait(&sh.full[slot], phases.of(slot), &sh.abort, p.err, 2)) break;
      phases.pass(slot);
      const int4 about = sh.tile[slot];
      if (n < t1) {
        const char* src[kStreams];
        sources(slot, t0, n, src);
        if (about.x != kMixed) {
          if (about.x != current) {
            current = about.x;
            op.enter_up(p, at, current);
          }
          if constexpr (Op::kRows > 1) {
#pragma unroll 1
            while (n + (Op::kRows - 1) * s.rp < t1) {
              op.template add<Op::kRows>(p, at, src, step, at.col);
              forward(src, Op::kRows);
            }
          }
#pragma unroll 1
          while (n < t1) {
            op.template add<1>(p, at, src, step, at.col);
            forward(src, 1);
          }
          if (n >= about.y) leave(place >= s.rp ? place - s.rp : place - s.rp + ring.acc_rows);
        } else {
#pragma unroll 1
          while (n < t1) {
            const int2 e = rows[slot * ring.tile_rows + n - t0];
            if (e.x >= 0) {
              if (e.x != current) {
                current = e.x;
                op.enter_up(p, at, current);
              }
              op.template add<1>(p, at, src, step, at.col);
              if (n + s.rp >= e.y) leave(place);
            }
            forward(src, 1);
          }
        }
      }
      ended = about.z;
      if (released < lost && (ended == closed || tile - released + 1 >= half)) {
        if (ended > closed) {
          if (!gate.meet(&sh, p.err)) break;
          close<Op>(p, acc, ends, closed_at, ended - closed);
          closed_at += ended - closed;
          if (closed_at >= room) closed_at -= room;
          closed = ended;
        }
        __syncwarp();
        for (; released <= tile && released < lost; ++released) {
          tc::mbar_arrive_lane0(&sh.empty[released_slot], lane);
          if (++released_slot == ring.slots) released_slot = 0;
        }
      }
      if (++slot == ring.slots) slot = 0;
    }
    meet_compute();
    if (ended > closed) close<Op>(p, acc, ends, closed_at, ended - closed);
    if constexpr (Op::kBackward) {
      // The block's channel sums, over the rows it reads side by side, in the room of the sums that are
      // done with.
      float* flat = reinterpret_cast<float*>(acc);
      const int one = s.rp * s.channels;
      float* chan = p.chan + static_cast<size_t>(blockIdx.x) * Q * s.channels;
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        meet_compute();
        if (at.row < s.rp) {
#pragma unroll
          for (int k = 0; k < V; ++k) flat[at.row * s.channels + at.col + k] = op.own[q][k];
        }
        meet_compute();
#pragma unroll 1
        for (int i = threadIdx.x; i < s.channels; i += kThreads) {
          float t[4] = {};
#pragma unroll 1
          for (int r = i; r < one; r += 4 * s.channels)
#pragma unroll
            for (int h = 0; h < 4; ++h) t[h] += r + h * s.channels < one ? flat[r + h * s.channels] : 0.0f;
          chan[q * s.channels + i] = (t[0] + t[1]) + (t[2] + t[3]);
        }
      }
    }
  }
  __syncthreads();
  const bool gave_up = *static_cast<volatile int*>(&sh.abort) != 0;   // by all threads before anyone goes on
  if (gridDim.x > 1) cg::this_grid().sync();
  else __syncthreads();

  if (copies) {
    if (p.out && !gave_up) {
      // down again, from the slot of the last tile that the ring lost
      Seen seen;
      if (held == ring.slots && --slot < 0) slot = ring.slots - 1;
#pragma unroll 1
      for (int k = w.tiles - held - 1; k >= 0; --k) {
        const int t0 = w.r0 + k * ring.tile_rows;
        if (!tc::warp_wait(&sh.empty[slot], phases.of(slot), &sh.abort, p.err, 1)) break;
        phases.pass(slot);
        copy_tile<kStreams>(p, &sh, smem, slot, t0, t0 + ring.tile_rows, true);
        describe_tile(p, w, &sh, smem, slot, t0, t0 + ring.tile_rows, 0, &seen);
        if (--slot < 0) slot = ring.slots - 1;
      }
    }
    // the block may not end before its copies have, also where a wait gave up
    for (int k = 0; k < ring.slots; ++k)
      if (sh.copies[k] > 0) tc::mbar_wait_drain(&sh.full[k], (sh.copies[k] - 1) & 1);
    return;
  }
  if (gave_up) return;

  if constexpr (Op::kBackward) {
    // dw and db: a warp to a sum, its lanes to the blocks
    const int sums = Q * s.channels;
#pragma unroll 1
    for (int i = blockIdx.x * kWarps + (threadIdx.x >> 5); i < sums; i += gridDim.x * kWarps) {
      double t = 0.0;
#pragma unroll 4
      for (int b = lane; b < gridDim.x; b += 32) t += p.chan[static_cast<size_t>(b) * sums + i];
#pragma unroll
      for (int o = 16; o > 0; o /= 2) t += __shfl_xor_sync(0xffffffffu, t, o);
      if (lane == 0) {
        if (i < s.channels && p.grad_bias) p.grad_bias[i] = static_cast<float>(t);
        if (i >= s.channels && p.grad_weight) p.grad_weight[i - s.channels] = static_cast<float>(t);
      }
    }
    if (!p.out) return;
  }
  gather<Op>(p, sh, sum, sum + kThreads, edge);

  current = -1;
  const int nq = s.per.d + s.groups.d;
  auto enter = [&](int i) {
    if (i != current) {
      current = i;
      op.enter_down(p, at, i, i == sh.edge[0] ? edge : i == sh.edge[1] ? edge + nq : p.table + static_cast<size_t>(i) * nq);
    }
  };
  n = at.row < s.rp ? n - s.rp : -1;   // the last row of this thread, if it has any
#pragma unroll 1
  for (int tile = w.tiles - 1; tile >= 0; --tile) {
    const int t0 = w.r0 + tile * ring.tile_rows;
    if (--slot < 0) slot = min(ring.slots, w.tiles) - 1;
    if (tile < lost) {
      if (!tc::warp_wait(&sh.full[slot], phases.of(slot), &sh.abort, p.err, 2)) return;
      phases.pass(slot);
    }
    if (n >= t0) {
      const int about = sh.tile[slot].x;
      const char* src[kStreams];
      sources(slot, t0, n, src);
      auto back = [&](int rows_done) {
        n -= rows_done * s.rp;
#pragma unroll
        for (int k = 0; k < kStreams; ++k) src[k] -= rows_done * step[k];
      };
      if (about != kMixed) {
        enter(about);
        if constexpr (Op::kRows > 1) {
#pragma unroll 1
          while (n - (Op::kRows - 1) * s.rp >= t0) {
            op.template put<Op::kRows>(p, at, src, step, at.col, n, true);
            back(Op::kRows);
          }
        }
#pragma unroll 1
        while (n >= t0) {
          op.template put<1>(p, at, src, step, at.col, n, true);
          back(1);
        }
      } else {
#pragma unroll 1
        while (n >= t0) {
          const int i = rows[slot * ring.tile_rows + n - t0].x;
          if (i >= 0) enter(i);
          if (i >= 0 || op.wants_outside(p)) op.template put<1>(p, at, src, step, at.col, n, i >= 0);
          back(1);
        }
      }
    }
    if (tile >= ring.slots) {
      __syncwarp();
      tc::mbar_arrive_lane0(&sh.empty[slot], lane);
    }
  }
}

// ---------------------------------------------------------------- launch

inline int round_up(int v, int to) { return (v + to - 1) / to * to; }

// Shared memory of a call: the sums, and slots with their tables and places for sums in what is left.
inline bool plan_ring(const Shape& s, int q, int dim, int acc_thread, const int (&row_bytes)[kMaxStreams], Ring* r) {
  int per_row = 0;
  for (int k = 0; k < kMaxStreams; ++k) per_row += row_bytes[k];
  r->acc_bytes = round_up(acc_thread * s.cv, 8);
  const int row_cost = r->acc_bytes + static_cast<int>(sizeof(int2) + sizeof(End));
  r->tile_rows = std::min(std::max(kTileBytes / (per_row + row_cost), 1), kMaxTileRows);
  int at = 0, in_slot = 0;
  for (int k = 0; k < kMaxStreams; ++k) {
    r->row_bytes[k] = row_bytes[k];
    r->elem[k] = k < 2 ? row_bytes[k] / dim : 0;
    r->off[k] = in_slot;
    if (row_bytes[k]) in_slot += round_up(row_bytes[k] * r->tile_rows + 32, 128);
  }
  r->slot_bytes = in_slot;
  const int nq = q * s.groups.d;
  r->o_sum = at;
  at += round_up((kThreads + std::max(2 * nq, kThreads)) * static_cast<int>(sizeof(double)), 128);
  r->o_edge = at;
  at += round_up(2 * nq * static_cast<int>(sizeof(float)), 128);
  // rows that a thread can be ahead, and room for rp rows of the backward's channel sums
  const int more = std::max(s.rp, (s.rp * s.channels * static_cast<int>(sizeof(float)) + r->acc_bytes - 1) / r->acc_bytes);
  r->slots = (kSmem - 512 - at - more * r->acc_bytes) / (in_slot + r->tile_rows * row_cost);
  if (r->slots > kMaxSlots) r->slots = kMaxSlots;
  if (r->slots < 2) return false;
  r->acc_rows = r->slots * r->tile_rows + more;
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

inline Shape shape_of(const Call& c, int width) {
  Shape s;
  s.n_nodes = c.n_nodes;
  s.n_structs = c.n_structs;
  s.rows = 0;
  s.channels = c.channels;
  s.groups = div_by(c.groups);
  s.per = div_by((c.lmax + 1) * c.groups);
  s.cg = c.channels / c.groups;
  s.cv = c.channels / width;
  s.cvg = s.cg / width;
  s.rp = kThreads / s.cv;
  s.ptr = c.node_ptr;
  return s;
}

// Shape, shared memory and number of blocks of a call on a device of `sms` SMs; false: rows too long.
inline bool plan_call(const Call& c, int width, int q, int dim, int acc_thread, const int (&row_bytes)[kMaxStreams],
                      int sms, Shape* s, Ring* ring, long long* blocks) {
  *s = shape_of(c, width);
  if (!plan_ring(*s, q, dim, acc_thread, row_bytes, ring)) return false;
  // A block for every rp rows at most, and no more blocks than run at once (one on an SM): the grid
  // barrier needs them all on the device.
  const long long n = c.n_nodes, most = std::min(sms, kMaxBlocks);
  *blocks = std::max(1LL, std::min((n + s->rp - 1) / s->rp, most));
  s->rows = static_cast<int>((n + *blocks - 1) / *blocks);
  *blocks = (n + s->rows - 1) / s->rows;
  auto tiles = [&](long long rows) { return static_cast<int>((rows + ring->tile_rows - 1) / ring->tile_rows); };
  ring->tiles = tiles(s->rows);
  ring->tiles_last = tiles(n - (*blocks - 1) * s->rows);
  ring->l2_tiles = static_cast<int>(kL2Bytes / *blocks / ring->slot_bytes);
  return true;
}

template <class Op, int V>
etp_status launch(const Call& c, Args& p, const int (&row_bytes)[kMaxStreams], cudaStream_t stream, const char* what) {
  auto kernel = k_norm<Op, V>;
  static thread_local int known_dev = -1, sms = 0;   // a device is asked once in a row
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && dev != known_dev) {
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    known_dev = e == cudaSuccess ? dev : -1;
  }
  if (e != cudaSuccess) return cuda_status(e, what);
  long long blocks = 0;
  if (!plan_call(c, V, Op::Q, Op::K * c.channels, Op::kAcc, row_bytes, sms, &p.s, &p.ring, &blocks)) {
    set_error(std::string(what) + ": rows too long");
    return ETP_ERR_UNSUPPORTED;
  }
  void* args[] = {&p};
  const dim3 grid(static_cast<unsigned>(blocks)), block(kBlock);
  const void* fn = reinterpret_cast<const void*>(kernel);
  if (blocks == 1) e = cudaLaunchKernel(fn, grid, block, args, p.ring.bytes, stream);
  else e = cudaLaunchCooperativeKernel(fn, grid, block, args, p.ring.bytes, stream);
  if (e != cudaSuccess) cudaGetLastError();   // reported here, not by the next call
  return cuda_status(e, what);
}

}  // namespace norm
}  // namespace etp
