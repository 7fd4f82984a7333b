// Host replay of the group norm's launch plan: every byte that a tile's rows hold comes into its slot, by
// the bulk copy or by hand, and no copy leaves its array or its slot. Prints what is not so.
#include <cstdio>
#include <cstring>
#include <vector>

#include "etp_norm_sweep.h"

using namespace etp::norm;

namespace etp {
void set_error(const std::string&) {}
etp_status cuda_status(cudaError_t, const char*) { return ETP_ERR_CUDA; }
}  // namespace etp

static long long tiles_seen = 0, by_hand = 0, wrong = 0;

static void replay(const etp::norm::Call& c, int width, int acc, const int (&row_bytes)[kMaxStreams], int sms) {
  Shape s;
  Ring ring;
  long long blocks = 0;
  const int dim = c.channels * (c.lmax + 1) * (c.lmax + 1);
  if (!plan_call(c, width, c.lmax + 2, dim, acc, row_bytes, sms, &s, &ring, &blocks)) return;
  const int streams = row_bytes[2] ? 3 : row_bytes[1] ? 2 : 1;
  for (long long b = 0; b < blocks; ++b) {
    const int r0 = static_cast<int>(b * s.rows), r1 = b == blocks - 1 ? c.n_nodes : r0 + s.rows;
    const int tiles = b == blocks - 1 ? ring.tiles_last : ring.tiles;
    if ((r1 - r0 + ring.tile_rows - 1) / ring.tile_rows != tiles) ++wrong;
    for (int k = 0; k < tiles; ++k) {
      const int t0 = r0 + k * ring.tile_rows, t1 = std::min(t0 + ring.tile_rows, r1);
      ++tiles_seen;
      for (int i = 0; i < streams; ++i) {
        const size_t rb = row_bytes[i], all = static_cast<size_t>(c.n_nodes) * rb;
        const TileBytes t = tile_bytes(t0, t1, c.n_nodes, row_bytes[i]);
        const size_t room = (i + 1 < streams ? ring.off[i + 1] : ring.slot_bytes) - ring.off[i];
        size_t have = t.b;                       // bytes of the array in the slot: [t.a, have)
        if (near_end(t1, c.n_nodes) && t.e > t.b) {
          have = t.e;
          ++by_hand;
          if (t.e - t.b > 32) ++wrong;           // a byte to a lane
        }
        const bool fits = t.a % 16 == 0 && t.b % 16 == 0 && t.a <= t.b && t.b <= all && have - t.a <= room &&
                          t.a == (t0 * rb & ~static_cast<size_t>(15));
        if (!fits || have < t1 * rb) {
          if (wrong < 5)
            std::printf("lmax %d, %d channels, %d groups, %d rows, stream %d of %d bytes a row: rows %d..%d end at byte %zu, there to %zu\n",
                        c.lmax, c.channels, c.groups, c.n_nodes, i, row_bytes[i], t0, t1, t1 * rb, have);
          ++wrong;
        }
      }
    }
  }
}

int main() {
  const int shapes[][4] = {{2, 32, 4, 4}, {1, 32, 4, 4}, {0, 64, 8, 4}, {0, 1, 1, 1}, {0, 2, 1, 2}, {0, 4, 1, 4}, {0, 5, 1, 1},
                           {0, 6, 3, 2}, {1, 1, 1, 1}, {1, 3, 1, 1}, {2, 50, 5, 2}, {3, 128, 16, 4}, {0, 252, 7, 4}};
  std::vector<int> rows;
  for (int n = 1; n <= 2500; ++n) rows.push_back(n);
  for (int n = 2501; n <= 3000000; n = n * 5 / 4 + 3) rows.push_back(n);
  for (const auto& sh : shapes)
    for (int n : rows)
      for (int sms : {148, 132, 1})
        for (int size : {2, 4}) {
          etp::norm::Call c{};
          c.lmax = sh[0];
          c.channels = sh[1];
          c.groups = sh[2];
          c.n_nodes = n;
          c.n_structs = 1;
          const int l = c.lmax, dim = c.channels * (l + 1) * (l + 1);
          const int forward[kMaxStreams] = {dim * size, 0, 0}, rows_in[kMaxStreams] = {dim * size, dim * size, 0},
                    kept[kMaxStreams] = {dim * size, dim, (dim + 31) / 32};
          replay(c, sh[3], 16 + 4 * l, forward, sms);
          for (int width : {sh[3], std::min(sh[3], 2)}) {
            replay(c, width, 4 * (l + 2), rows_in, sms);
            replay(c, width, 4 * (l + 2), kept, sms);
          }
        }
  std::printf("%lld tiles, %lld with bytes by hand, %lld wrong\n", tiles_seen, by_hand, wrong);
  return wrong != 0;
}
