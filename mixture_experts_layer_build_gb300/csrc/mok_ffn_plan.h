// mok_ffn_plan.h -- how the feed-forward block's contractions are cut into tiles and dealt out to CTA pairs (plain C++, no
// CUDA types, so host tests can drive it).
#pragma once
#include <cstdint>
#include <initializer_list>

#if defined(__CUDACC__)
#define MOK_PLAN_FN __host__ __device__ __forceinline__
#else
#define MOK_PLAN_FN inline
#endif

namespace mok {

constexpr int kFfnBK = 64;  // bf16 of K per block: one 128-byte swizzle row
constexpr int64_t kFfnMaxTokens = (int64_t{1} << 31) - 257;  // row indices of padded tiles stay within 31 bits

// Limit of the wait for a tile of k_blocks K blocks, where that of other waits is `base`: 2 us more for every block, which
// takes 0.2 to 0.45.  (K blocks of a weight gradient are 64 tokens: 2 s alone cover 284 million tokens at 0.45.)
MOK_PLAN_FN uint64_t tile_wait_ns(uint64_t base, int64_t k_blocks) {
  return base + static_cast<uint64_t>(k_blocks) * 2000u;
}

inline int64_t tiles_of(int64_t n, int64_t tile) { return (n + tile - 1) / tile; }

// ---- the CTA pairs' tiles (mok_ffn_pair.cu) ----

// How a launch's tiles are dealt out to its `pairs` CTA pairs.  Job 0 is the row-tiled contraction, job 1 the weight
// gradients; in the forward, the same contraction's last rows in narrower tiles.  The first job's units go round
// robin: pairs below `rem` get `quot` + 1, the rest `quot`.  Of the second job's, every pair gets `each`, round robin,
// and the pairs from `rem` on `extra` before them.
struct PairPlan {
  int32_t pairs;
  int32_t first;        // which job goes first
  int32_t quot, rem;
  int32_t each, extra;
  int32_t units[2];
};

// Slots of pair `pair`.
MOK_PLAN_FN int plan_steps(const PairPlan& g, int pair) {
  return g.quot + (pair < g.rem ? 1 : 0) + g.each + (pair >= g.rem ? g.extra : 0);
}
// Job and unit of the pair's i-th slot; false when it is empty.
MOK_PLAN_FN bool plan_unit(const PairPlan& g, int pair, int i, int& job, int& u) {
  const int mine = g.quot + (pair < g.rem ? 1 : 0);
  if (i < mine) {
    u = i * g.pairs + pair;
    job = g.first;
    return true;
  }
  const int j = i - mine, e = pair >= g.rem ? g.extra : 0;
  u = j < e ? g.each * g.pairs + j * (g.pairs - g.rem) + (pair - g.rem) : (j - e) * g.pairs + pair;
  job = 1 - g.first;
  return u < g.units[job];
}

constexpr int kGroupM = 4;  // M tiles of one band of the tile order

// Tile u of an m_tiles x n_tiles output in bands of kGroupM M tiles, M fastest within a band.
MOK_PLAN_FN void ordered_tile(int u, int m_tiles, int n_tiles, int& m, int& n) {
  const int band = u / (kGroupM * n_tiles), r = u - band * (kGroupM * n_tiles);
  const int left = m_tiles - band * kGroupM, rows = left < kGroupM ? left : kGroupM;
  n = r / rows;
  m = band * kGroupM + (r - n * rows);
}

// The plan of a launch with units[j] tiles of k[j] K blocks of job j on at most `pairs` pairs, the job with the longer
// K first unless `rows_first`; returns the K blocks of the pair that has the most.
inline int64_t make_plan(const int64_t (&units)[2], const int64_t (&k)[2], bool rows_first, int pairs, PairPlan* g) {
  const int first = units[0] && (!units[1] || rows_first || k[0] >= k[1]) ? 0 : 1, second = 1 - first;
  const int64_t total = units[0] + units[1], n = total < pairs ? total : pairs;
  g->pairs = static_cast<int32_t>(n);
  g->first = first;
  g->units[0] = static_cast<int32_t>(units[0]);
  g->units[1] = static_cast<int32_t>(units[1]);
  const int64_t quot = units[first] / n, rem = units[first] % n;
  g->quot = static_cast<int32_t>(quot);
  g->rem = static_cast<int32_t>(rem);
  const int64_t ca = (quot + 1) * k[first], cb = quot * k[first];  // K blocks of a pair below rem, and of the rest
  int64_t end = rem ? ca : cb;                                     // no pair ends before its first job
  g->each = g->extra = 0;
  if (units[second]) {
    // the earliest end by which the pairs can have taken all of the second job: it is reached either by a whole
    // number of units behind `ca` or behind `cb`
    const int64_t ks = k[second];
    auto room = [&](int64_t t) { return (rem ? rem * ((t - ca) / ks) : 0) + (n - rem) * ((t - cb) / ks); };
    const int64_t share = (units[0] * k[0] + units[1] * k[1]) / n;  // none can end before an even share
    const int64_t least = end > share ? end : share;
    int64_t best = -1;
    for (int64_t c : {rem ? ca : cb, cb}) {
      int64_t t = c + (least > c ? (least - c + ks - 1) / ks * ks : 0);
      while (room(t) < units[second]) t += ks;
      if (best < 0 || t < best) best = t;
    }
    end = best;
    const int64_t nb = (end - cb) / ks, na = rem ? (end - ca) / ks : nb;
    g->each = static_cast<int32_t>(na);
    g->extra = static_cast<int32_t>(nb - na);
  }
  return end;
}

// What a 64-wide K block takes on a pair, in ns: measured 300 at 256 columns, 270 and 240 at 224 and 192 (the loads
// from L2 bound it: 128 + columns / 2 rows of 128 bytes per CTA), 205 to 285 at 128.
constexpr int64_t block_ns(int bn) { return bn == 256 ? 300 : bn == 224 ? 270 : bn == 192 ? 240 : 220; }

// The tile width of the least cost, and that cost: the longest pair's time, a tile counted as its K blocks and one more
// for what it costs besides them, three for a row-tiled one where those go first (rows_first: an epilogue there stands
// at the end of some pairs).  tiles(bn, units) gives each job's tiles.  Against counting K blocks x (columns + 16):
// 41 training sizes 0.976 of the time on average, 0.82 to 1.03; T = 9602, H = 4024, I = 848 forward 205 -> 170 us,
// T = 2675, H = 3992, I = 536 training 143 -> 132.
struct Width {
  int bn;  // 0: there are no tiles
  int64_t cost;
};
template <class Tiles>
Width best_width(std::initializer_list<int> widths, const int64_t (&k)[2], bool rows_first, int pairs, Tiles&& tiles) {
  const int64_t k1[2] = {k[0] + (rows_first ? 3 : 1), k[1] + 1};
  Width best{0, 0};
  for (int bn : widths) {
    int64_t units[2] = {0, 0};
    PairPlan g;
    tiles(bn, units);
    if (!units[0] && !units[1]) return Width{0, 0};
    const int64_t c = make_plan(units, k1, rows_first, pairs, &g) * block_ns(bn);
    if (!best.bn || c < best.cost) best = Width{bn, c};
  }
  return best;
}

// A forward tile's time: its K blocks and three more.
constexpr int64_t fwd_cost(int64_t k_blocks, int bn) { return (k_blocks + 3) * block_ns(bn); }

// Widths of GATEUP or DOWN: the first m_split M tiles in tiles of bn0 columns, the others of bn1.
struct FwdSplit {
  int bn0, bn1;  // bn1 = 0: no others
  int64_t m_split;
};

// The widths of least cost for M rows, N output columns, K.  With up to four rounds of tiles, the M tiles that do not
// fill whole rounds may take a narrower width, so that the last round is shorter rather than part empty: T = 4096,
// H = 2048, I = 1024 40.7 -> 38.3 us (76 pairs; 256 columns in nine of 16 M tiles, 192 in seven), T = 700, H = I = 3400
// 66.4 -> 64.1.
inline FwdSplit fwd_split(bool gate_up, int64_t M, int64_t N, int64_t K, int pairs) {
  const int64_t mt = tiles_of(M, 256), kb = tiles_of(K, kFfnBK), cols = gate_up ? 2 * N : N;
  constexpr int kWidths[4] = {256, 224, 192, 128};
  FwdSplit best{0, 0, mt};
  int64_t cost = 0;
  for (int w : kWidths) {
    if (gate_up && w == 224) continue;  // half of the columns are gate columns, in whole 32-column chunks
    const int64_t c = (mt * tiles_of(cols, w) + pairs - 1) / pairs * fwd_cost(kb, w);
    if (!best.bn0 || c < cost) best.bn0 = w, cost = c;
  }
  for (int w : kWidths) {
    const int64_t n = tiles_of(cols, w), rounds = mt * n / pairs, m = rounds * pairs / n;
    if ((gate_up && w == 224) || rounds < 1 || rounds > 3 || m <= 0 || m >= mt) continue;
    for (int v : kWidths) {
      if (v >= w || (gate_up && v == 224)) continue;
      PairPlan g;
      const int64_t units[2] = {m * n, (mt - m) * tiles_of(cols, v)};
      const int64_t c = make_plan(units, {fwd_cost(kb, w), fwd_cost(kb, v)}, true, pairs, &g);
      if (c < cost) best = FwdSplit{w, v, m}, cost = c;
    }
  }
  return best;
}

// What a launch of the backward does: its row-tiled contraction (DACT in phase 1, DX in phase 2), dWg and dWu, dWd.
struct BwdJobs {
  bool rows, gate_up, down;
};
inline void bwd_tiles(int phase, int64_t T, int64_t H, int64_t I, const BwdJobs& j, int w, int64_t* units) {
  units[0] = j.rows ? tiles_of(T, 256) * tiles_of(phase == 1 ? I : H, w) : 0;
  units[1] = (j.gate_up ? 2 * tiles_of(I, 256) * tiles_of(H, w) : 0) + (j.down ? tiles_of(H, 256) * tiles_of(I, w) : 0);
}
// DACT's tiles go before dWd's, whose MMAs then hide its epilogue.
constexpr bool rows_first(int phase) { return phase == 1; }

inline Width bwd_width(int phase, int64_t T, int64_t H, int64_t I, const BwdJobs& j, int pairs) {
  const int64_t k[2] = {phase == 1 ? tiles_of(H, kFfnBK) : 2 * tiles_of(I, kFfnBK), tiles_of(T, kFfnBK)};
  return best_width({256, 224, 192, 128}, k, rows_first(phase), pairs,
                    [&](int w, int64_t* u) { bwd_tiles(phase, T, H, I, j, w, u); });
}
// The two phases' jobs: dact, dx: whether the row-tiled contractions are in them; gate_up, down: which weight gradients
// are wanted.  dWd goes with DACT where the two launches then cost less.
inline void bwd_jobs(int64_t T, int64_t H, int64_t I, bool dact, bool dx, bool gate_up, bool down, int pairs, BwdJobs* one,
                     BwdJobs* two) {
  const BwdJobs with{dact, false, down}, rest{dx, gate_up, false}, without{dact, false, false}, all{dx, gate_up, down};
  auto cost = [&](const BwdJobs& a, const BwdJobs& b) {
    return bwd_width(1, T, H, I, a, pairs).cost + bwd_width(2, T, H, I, b, pairs).cost;
  };
  const bool apart = !dact || cost(without, all) <= cost(with, rest);
  *one = apart ? without : with;
  *two = apart ? all : rest;
}

// ---- tile kernel or pairs ----

enum FfnVariant : int { F_GATEUP = 0, F_DOWN, F_DACT, F_DX };  // the row-tiled contractions (M = T)

// Whether a row-tiled contraction runs on pairs of CTAs: where their narrowest tiles, 256 x 128, are enough for
// half of the pairs, or a quarter up to 1024 tokens; below, the tile kernel, which can split K.  In the backward,
// where weight gradients fill the other pairs, an eighth is enough from 384 tokens on, and a quarter below if three
// quarters of the tiles' rows are tokens.  Measured at H = 4096, I = 1536, a training step with every contraction
// on the tile kernel and on pairs: 67.6 and 74.9 us for 256 tokens, 151 and 96.7 for 1024; the quarter: T = 1000,
// H = 1000, I = 512 16.1 -> 14.8 forward, but T = 1500, H = I = 640 12.9 -> 13.8; the backward's: 384 tokens at H =
// 2048, I = 1024 49.6 -> 44.4, 1024 tokens 62.7 -> 52.3; 150 tokens at H = 4096, I = 1536 would lose 66.4 -> 70.4.
inline bool ffn_on_pairs(int var, int64_t M, int64_t N, int sms) {
  const int cols = var == F_GATEUP ? 64 : 128;
  const int64_t mt = tiles_of(M, 256), tiles = mt * tiles_of(N, cols);
  int part = M <= 1024 ? 4 : 2;  // of the pairs that has tiles
  if (var >= F_DACT) part = M > 384 ? 8 : 4 * M >= 3 * 256 * mt ? 4 : 2;
  return M > 128 && 2 * part * tiles >= sms;
}

}  // namespace mok
