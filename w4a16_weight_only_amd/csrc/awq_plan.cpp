// Host-only launch planning of the AWQ W4A16 library (declarations and the plan
// structures in awq_plan.h).  Every choice below is measured on MI355X; the comments
// give the measurements that decided it.
#include "awq_plan.h"

#include "../../include/awq_w4a16.h"

namespace awq {

int64_t groups_of(int64_t K, int64_t group_size) { return group_size == -1 ? 1 : K / group_size; }

// Effective group length passed to kernels: -1 means one group spanning K.
int eff_group(int64_t K, int64_t group_size) { return (int)(group_size == -1 ? K : group_size); }

int format_check(int64_t K, int64_t N, int64_t group_size) {
  if (K < 1 || N < 1 || N % 8 != 0) return AWQ_ERR_SHAPE;
  if (group_size == -1) return AWQ_OK;
  if (group_size <= 0 || K % group_size != 0) return AWQ_ERR_GROUP;
  return AWQ_OK;
}

int limits_check(int64_t M, int64_t K, int64_t N, int64_t group_size) {
  int st = format_check(K, N, group_size);
  if (st != AWQ_OK) return st;
  if (M < 0) return AWQ_ERR_SHAPE;
  if (K % 32 != 0 || N % 32 != 0) return AWQ_ERR_UNSUPPORTED;
  if (group_size != -1 && group_size % 32 != 0) return AWQ_ERR_UNSUPPORTED;
  if (K > kMaxDim || N > kMaxDim || M > kMaxDim) return AWQ_ERR_UNSUPPORTED;
  // The tile family's 1-D grid must stay below 2^31 workgroups.
  if (((M + 127) / 128) * ((N + 63) / 64) >= (int64_t(1) << 31)) return AWQ_ERR_UNSUPPORTED;
  return AWQ_OK;
}

constexpr int kSkinnyWgPer2Cu = 4;  // 4-wave skinny workgroups counted per two compute units

// Skinny plan for M <= kSkinnyMaxM, or false when no launch shape fits the
// kernel's limits (at most kSkinnyMaxSplits splits, at most kSkinnyMaxGroups
// quantization groups per workgroup).
bool plan_skinny(int64_t M, int64_t K, int64_t N, int64_t g, int cus, SkinnyPlan& s) {
  // The kernel addresses qweight with 32-bit byte offsets.
  if (K * (N / 2) >= (int64_t(1) << 32) - 4096) return false;
  const int64_t T = K / kKStep;
  const int64_t gsteps = g / kKStep;  // g already resolved (-1 -> K)
  s.n_tiles = (int)((N + kSkinnyCols - 1) / kSkinnyCols);
  // One or two rows: 4-row plans (4 waves, splits meet in fixed-point atomics).
  // From three rows the atomics cost more than fp32 partials and the reduce kernel
  // (every split costs one returning atomic per row and column; M = 3, 4: 10-25%
  // faster with partials; M = 2 mixed, within 7% either way).  Three or four rows
  // on a layer whose 8-wave grid would take more than four rounds (above ~32 MB of
  // packed weights) take 4-row plans with partials: their smaller LDS reduction
  // buffer lets more workgroups share a compute unit (4096 x 114688: 69.5 -> 62.8
  // us; 8192 x 28672: 37.3 -> 33.3 us; routed experts at 3-4 tokens 6-10%); on
  // smaller layers they measured 0-3% slower than the 16-row plans.  Five to eight
  // rows on those layers take 8-row plans for the same reason (32 KB of LDS
  // reduction buffer instead of 64 KB; 4096 x 114688 M = 8: 73.8 -> 68.2 us;
  // 8192 x 28672 M = 6: 38.6 -> 35.6 us).  16-row plans
  // take 8 waves, or 4 waves (two per CU, shorter workgroups overlapping each
  // other's fixed phases) on those large layers: measured 8-15% faster on
  // 8192 x 28672, 28672 x 8192 and 4096 x 114688, 10-25% slower on layers of up
  // to 22 MB.
  const bool large = T * s.n_tiles > (int64_t)8 * cus * 4;
  s.mrows = (M <= 2 || (M <= 4 && large)) ? 4 : ((M <= 8 && large) ? 8 : 16);
  s.atomic = M <= 2;
  s.waves = (s.mrows == 4 || large) ? 4 : 8;
  const int64_t W = s.waves;
  // Whole grid resident in one round, counting two 4-wave workgroups per CU (three
  // fit when every wave stays inside one group; counting three gives more splits,
  // which measured slower at four rows) and one 8-wave workgroup (large LDS
  // reduction buffer).
  const int64_t cap = s.waves == 4 ? (int64_t)cus * kSkinnyWgPer2Cu / 2 : (int64_t)cus;
  int64_t L = (T * s.n_tiles + W * cap - 1) / (W * cap);
  const int64_t l_min = (T + W * kSkinnyMaxSplits - 1) / (W * kSkinnyMaxSplits);
  if (L < l_min) L = l_min;
  // At least two k-steps per wave, so that each wave's second step is in flight
  // while its first is multiplied (measured faster than one step per wave even
  // at half the workgroups); four for two rows, whose splits each cost one atomic
  // per row and column (half the splits measured faster).
  const int64_t l_floor = M == 2 ? 4 : 2;
  if (L < l_floor) L = l_floor;
  if (L > T) L = T;
  // 4-row plans on a grid of more than two rounds: keep each wave's run inside one
  // group (at most 4 k-steps).  Such waves need no per-group LDS tables and fewer
  // registers, so three workgroups share a compute unit, and the extra splits cost
  // one atomic (or partial) per output element each; on 16-row plans the extra
  // splits outweigh the gain (measured on 4096 x 114688, 8192 x 28672 and
  // 28672 x 8192 layers).
  if (s.mrows == 4 && gsteps < T && L > gsteps && T * s.n_tiles > W * cap * 2) L = gsteps < 4 ? gsteps : 4;
  auto splits_of = [&](int64_t l) { return (T + W * l - 1) / (W * l); };
  if (gsteps >= T) {
    s.single_group = true;  // one group spans K
  } else if (L <= gsteps) {
    while (gsteps % L != 0) ++L;  // stays <= gsteps: each wave's run in one group
    s.single_group = true;
  } else {
    s.single_group = false;
    // A workgroup's run of W*L steps may touch at most kSkinnyMaxGroups groups.
    if ((W * L - 1) / gsteps + 2 > kSkinnyMaxGroups) {
      int64_t l2 = ((int64_t)(kSkinnyMaxGroups - 2) * gsteps + 1) / W;
      if (l2 < 1) l2 = 1;
      if (l2 <= gsteps) {
        while (gsteps % l2 != 0) --l2;
        s.single_group = true;
      }
      L = l2;
    }
  }
  // 8- and 16-row plans whose waves span several groups: take one-group runs of at most 4
  // k-steps instead when that lowers (rounds of resident workgroups) x (k-steps
  // per wave + 2); the 2 stands for a workgroup's fixed cost (group data, the
  // reduction, the partial stores).  The round count decides it: 5.25 rounds of
  // 7-step waves lose to 7 full rounds of 4-step waves (4096 x 114688), while
  // 1 or 2 full rounds beat 2 or 3.5 (11008 x 4096, 28672 x 8192); measured.
  if (s.mrows >= 8 && !s.single_group) {
    int64_t l1 = gsteps < 4 ? gsteps : 4;
    while (gsteps % l1 != 0) --l1;
    auto cost = [&](int64_t l) { return (s.n_tiles * splits_of(l) + cap - 1) / cap * (l + 2); };
    if (splits_of(l1) <= kSkinnyMaxSplits && cost(l1) < cost(L)) {
      L = l1;
      s.single_group = true;
    }
  }
  if (splits_of(L) > kSkinnyMaxSplits) return false;
  s.L = (int)L;
  s.splits = (int)splits_of(L);
  // fp32 partials: the workgroup of a tile that arrives last sums them when the grid takes
  // two or more rounds of resident workgroups (its tail then overlaps the next round's
  // loads), and for 16-row plans only from five rounds (their partials are twice the
  // 8-row plans'); otherwise a reduce kernel does.  Measured, µs per call: 4 x 8192 x
  // 28672 34.2 -> 31.5, 3 / 8 / 16 x 4096 x 114688 61.3 / 67.4 / 77.9 -> 56.0 / 60.8 /
  // 75.0; 16 x 8192 x 28672 (four rounds) 43.9 -> 44.5; one-round grids 2-15% slower
  // fused (16 x 4096 x 11008 13.2 -> 13.6, 8 x 11008 x 4096 14.0 -> 16.3), where the
  // write-through of the partials, the arrival and the partial loads sit on the
  // critical path instead of the reduce launch.
  const int64_t per_cu = s.waves == 8 ? 1 : (s.mrows == 16 ? 2 : 3);
  const int64_t rounds = ((int64_t)s.n_tiles * s.splits + per_cu * cus - 1) / (per_cu * cus);
  s.fused = s.splits > 1 && rounds >= 2 && (s.mrows <= 8 || rounds >= 5);
  return true;
}

// Decode plan (fp16, 1 <= M <= 16), or false when the layer is outside its limits: a
// wave's k-steps must lie in one quantization group, the splits fit the fixed-point
// format, and qweight stays below 4 GiB (32-bit buffer offsets).  One workgroup per
// (512-column tile, K split) of waves * ks k-steps.
bool plan_decode(int64_t M, int64_t K, int64_t N, int64_t g, DecodePlan& d) {
  // Up to four rows: the returning fixed-point adds (M x N x splits of them) stay cheap
  // enough.  From five rows they cost more than the skinny family's fp32 partials (M = 8
  // on 11008 x 4096: 15.6 / 17.9 us for g-1 / g64 against 12.3 / 14.2), which keeps those.
  if (M < 1 || M > kDecodeMaxM) return false;
  if (K * (N / 2) >= (int64_t(1) << 32) - 4096) return false;
  const int64_t T = K / kKStep;
  d.mp = M <= 2 ? (int)M : 4;
  auto splits_of = [&](int ks, int waves) { return (T + (int64_t)ks * waves - 1) / ((int64_t)ks * waves); };
  auto ok = [&](int ks, int waves) {
    return (g == K || g % (kKStep * ks) == 0) && splits_of(ks, waves) <= kFxMaxSplits;
  };
  // Half-width tiles (256 columns, 4 waves): two k-steps per wave when g is K or a
  // multiple of 64, else one; the workgroup's waves then form 1, 2 or 4 parts that each
  // lie in one quantization group, summed and scaled apart after the wave reduction.
  // Half the columns per workgroup halves the K splits for the same grid, and with them
  // the fixed-point adds and how many meet at each address.  Measured, us per call, full
  // tiles -> half: 1 x 4096 x 4096 g128 6.38 -> 5.39, g64 6.88 -> 5.49, g32 6.97 -> 5.61;
  // 2 x 4096 x 4096 g128 8.00 -> 6.04; 1 x 4096 x 11008 g128 10.15 -> 8.33; 1 x 11008 x
  // 4096 g-1 9.02 -> 8.25, g32 11.18 -> 9.90; 2 x 11008 x 4096 g64 10.48 -> 9.42; 1 x 8192
  // x 28672 g128 35.9 -> 27.6.  Beyond 127 splits, full tiles: two k-steps per wave on 8
  // waves (one on 4 waves up to 128 k-steps), each wave scaling its own sums unless the
  // workgroup lies in one group.
  const int hks = (g == K || g % (2 * kKStep) == 0) ? 2 : 1;
  if (splits_of(hks, 4) <= kFxMaxSplits) {
    d.words = kDecodeWords / 2;
    d.ks = hks;
    d.waves = 4;
  } else {
    d.words = kDecodeWords;
    const int pref_ks = T <= 128 ? 1 : 2, pref_w = T <= 128 ? 4 : 8;
    const int cand[4][2] = {{pref_ks, pref_w}, {1, 4}, {1, 8}, {2, 8}};
    d.ks = 0;
    for (const auto& c : cand)
      if (ok(c[0], c[1])) {
        d.ks = c[0];
        d.waves = c[1];
        break;
      }
    if (d.ks == 0) return false;
  }
  d.n_tiles = (int)((N / 8 + d.words - 1) / d.words);
  d.splits = (int)splits_of(d.ks, d.waves);
  // Three or four rows: only while the grid stays within two rounds of three workgroups
  // per CU (1536 workgroups) or N <= 8192, and N <= 32768 (the adds' words stay under
  // 1.5 MB).  Measured against the skinny family, us per call: 3 x 2048 x 4096 8.90 ->
  // 5.91, 3 x 4096 x 4096 9.49 -> 6.95, 4 x 4096 x 4096 9.36 -> 7.39, 4 x 11008 x 4096
  // g64 13.68 -> 10.93, 4 x 4096 x 22016 17.46 -> 16.01, 4 x 28672 x 8192 35.8 -> 32.9;
  // kept on the skinny family: 3 x 8192 x 16384 20.5 (21.2 here), 4 x 8192 x 28672 32.3
  // (34.6), 3 x 4096 x 114688 56.0 (60.1).
  if (M > 2) {
    const int64_t grid = (int64_t)d.n_tiles * d.splits;
    if (N > 32768 || (grid > 1536 && N > 8192)) return false;
  }
  const int64_t span = (int64_t)kKStep * d.ks * d.waves;
  d.late = (g == K || g % span == 0) ? 1 : d.words == kDecodeWords ? 0 : (g % (span / 2) == 0 ? 2 : 4);
  return true;
}

int64_t decode_entries(const DecodePlan& d) { return (int64_t)d.n_tiles * 8 * d.words * d.mp; }

int64_t skinny_accum_entries(const SkinnyPlan& s) { return (int64_t)s.n_tiles * s.mrows * kSkinnyCols; }

// One launch of the tile family over M rows.
TileLaunch plan_tile(int64_t M, int64_t K, int64_t N, int cus) {
  auto tiles = [&](int v) {
    return ((M + kTileBM[v] - 1) / kTileBM[v]) * ((N + kTileBN[v] - 1) / kTileBN[v]);
  };
  // Row tile by M: 256 x 128 above 128 rows, 64 x 128 above 32, 32 x 128 below (a
  // tile taller than M wastes MFMA rows and x loads: 32 x 128 against 64 x 128 at
  // 17-32 rows measured 6-25% faster; at 65-128 rows two 64 x 128 row tiles beat
  // one 128 x 64 tile by 4-13%, and at 33-64 one 64 x 128 tile beats two 32 x 128).
  // Above 128 rows the product is MFMA-bound: K is split only while the tiles
  // leave compute units idle.  At or below 128 rows the weight stream dominates
  // and K is split to about two workgroups per compute unit (rounded down;
  // measured best over 1 to 4 per unit on 4096- to 28672-wide layers).  Every
  // split keeps at least 8 k-tiles.
  const int64_t fill = (int64_t)cus * 3 / 4;
  int v = M > 128 ? 0 : (M > 32 ? 1 : 2);
  // 129-192 rows with K <= 4096, where the 256-row tiles would be split over K: up to
  // three 64 x 128 row tiles instead (M = 130 on 4096 x 4096: 28.7 -> 21.8 us; M = 176
  // on 4096 x 11008: 61.1 -> 57.6 us).  With longer K (each weight dequantised by up
  // to three workgroups: M = 144 on 8192 x 8192 52.5 -> 69.6 us) or an unsplit grid
  // (M = 192 on 4096 x 28672: 83.8 -> 115.6 us) the 256-row tiles stay.
  if (v == 0 && M <= 192 && K <= 4096 && tiles(0) < fill) v = 1;
  const int64_t KT = (K + kTileBK - 1) / kTileBK;
  int64_t splits = 1;
  if (v == 0) {
    if (tiles(v) < fill) splits = ((int64_t)cus + tiles(v) - 1) / tiles(v);
  } else {
    splits = 2 * (int64_t)cus / tiles(v);
    if (splits < 1) splits = 1;
  }
  const int64_t max_splits = KT / 8 > 1 ? KT / 8 : 1;
  if (splits > max_splits) splits = max_splits;
  const int64_t kps = (KT + splits - 1) / splits;
  splits = (KT + kps - 1) / kps;
  TileLaunch t;
  t.tp.variant = v;
  t.tp.splits = (int)splits;
  t.tp.kps = (int)kps;
  t.block = kTileThreads[v];
  t.grid_x = tile_blocks((M + kTileBM[v] - 1) / kTileBM[v], N, kTileBN[v]);
  t.workgroups = tiles(v) * splits;
  return t;
}

Plan make_plan(int64_t M, int64_t K, int64_t N, int64_t g, int cus, bool bf16) {
  Plan p;
  if (!bf16 && plan_decode(M, K, N, g, p.dp)) {
    p.family = 2;
    p.grid_x = p.dp.n_tiles;
    p.grid_y = p.dp.splits;
    p.block = 64 * p.dp.waves;
    if (p.dp.splits > 1) p.accum_bytes = decode_entries(p.dp) * 12;  // word + side word
    return p;
  }
  if (M <= kSkinnyMaxM && plan_skinny(M, K, N, g, cus, p.sk)) {
    p.family = 0;
    p.grid_x = p.sk.n_tiles;
    p.grid_y = p.sk.splits;
    p.block = 64 * p.sk.waves;
    // 4-row fp16 plans: 64-bit fixed-point accumulators per tile entry; 16-row
    // plans and every bfloat16 plan: fp32 partials per (tile, split, entry).
    if (p.sk.splits > 1) {
      if (p.sk.atomic && !bf16) {
        p.accum_bytes = skinny_accum_entries(p.sk) * 12;
      } else {
        p.partial_bytes = (int64_t)p.sk.n_tiles * p.sk.splits * p.sk.mrows * kSkinnyCols * 4;
        if (p.sk.fused) p.accum_bytes = (int64_t)p.sk.n_tiles * 4;  // one arrival counter per column tile
      }
    }
  } else {
    p.family = 1;
    // A partly filled last 256-row tile whose workgroups would take one more round of
    // the compute units (one 256 x 128 workgroup per unit) goes to a second launch with
    // its own row tile and K splits: M = 2100 on 4096 x 4096, 137 -> 104 us; M = 1100,
    // 97 -> 77 us.  Where the round count stays, one launch is faster (M = 300 or
    // 600: the second launch's fixed cost and its reduce).
    const TileLaunch all = plan_tile(M, K, N, cus);
    p.rows1 = M;
    p.tile = all;
    const int64_t r = M % kTileBM[0];
    if (all.tp.variant == 0 && M > kTileBM[0] && r != 0) {
      const TileLaunch main = plan_tile(M - r, K, N, cus);
      if (main.rounds(cus) < all.rounds(cus)) {
        p.rows1 = M - r;
        p.tile = main;
        p.tail = plan_tile(r, K, N, cus);
      }
    }
    p.tp = p.tile.tp;
    p.block = p.tile.block;
    p.grid_x = p.tile.grid_x;
    p.grid_y = p.tile.tp.splits;
    const int64_t b1 = p.tile.tp.splits > 1 ? p.tile.tp.splits * p.rows1 * N * 4 : 0;
    const int64_t b2 = p.tail.tp.splits > 1 ? p.tail.tp.splits * (M - p.rows1) * N * 4 : 0;
    p.partial_bytes = b1 > b2 ? b1 : b2;  // the launches run in stream order
  }
  return p;
}

// Blocks of the tile grid (see the block order in tile_kernel): row_units units per
// run of 256 / bn column tiles, in whole runs of 8 (256 / bn) blocks.
int64_t tile_blocks(int64_t row_units, int64_t N, int bn) {
  const int64_t ct = 256 / bn;
  const int64_t n_tiles = (N + bn - 1) / bn;
  const int64_t units = row_units * ((n_tiles + ct - 1) / ct);
  return 8 * ct * ((units + 7) / 8);
}

// Grouped variants by slots per expert: 256 x 128 from 192, 64 x 128 above 32, and
// 32 x 128 for the few rows per expert of decode-sized batches, where the weights
// dominate and a smaller x tile lets four workgroups share a CU.  Below 192 rows two
// or three 64 x 128 row tiles beat one 256 x 128 tile that leaves rows idle; from
// 192 the larger tile wins (768 tokens over 8 experts, top-2: 300 against 390 us).
int moe_tile_variant(int64_t avg_rows, int* block_rows) {
  const int v = avg_rows >= 192 ? 0 : (avg_rows > 32 ? 1 : 2);
  *block_rows = kTileBM[v];
  return v;
}

RtnPlan rtn_plan(int64_t K, int64_t N, int g) {
  RtnPlan p;
  p.block = 64 * kRtnWaves;
  p.cols = 8 * kRtnWordCols;
  const int64_t ncb = (N + p.cols - 1) / p.cols;
  const int64_t G = K / g;
  if (g <= kRtnSlices * kRtnMaxFusedCache) {
    int cache = 1;
    while (kRtnSlices * cache < g) cache *= 2;
    p.cache = cache;
    p.two_pass = false;
    p.cpg = 1;
    p.scratch_bytes = 0;
  } else {
    p.cache = kRtnChunkCache;
    p.two_pass = true;
    p.cpg = (g + kRtnSlices * kRtnChunkCache - 1) / (kRtnSlices * kRtnChunkCache);
    p.scratch_bytes = G * p.cpg * 2 * (N / 8) * 16;
  }
  p.grid = G * p.cpg * ncb;
  return p;
}

int validate_pack(int64_t K, int64_t N, int64_t group_size, int64_t qweight_rows, int64_t qweight_cols,
                  int64_t qzeros_rows, int64_t qzeros_cols, int64_t scales_rows, int64_t scales_cols,
                  int64_t bias_len) {
  const int st = format_check(K, N, group_size);
  if (st != AWQ_OK) return st;
  const int64_t G = groups_of(K, group_size);
  if (qweight_rows != K || qweight_cols != N / 8) return AWQ_ERR_SHAPE;
  if (qzeros_rows != G || qzeros_cols != N / 8) return AWQ_ERR_SHAPE;
  if (scales_rows != G || scales_cols != N) return AWQ_ERR_SHAPE;
  if (bias_len != -1 && bias_len != N) return AWQ_ERR_SHAPE;
  return AWQ_OK;
}

namespace {

constexpr int64_t k2p32 = int64_t(1) << 32;

// HIP takes a launch's size in 32-bit work-item counts per dimension; grid y stays
// below 2^16 workgroups.
bool grid_fits(int64_t gx, int64_t gy, int64_t block) { return gx >= 1 && gy >= 1 && gx * block < k2p32 && gy < 65536; }

// One tile launch over `rows` rows: its grid, the 32-bit byte offsets of a tile's x
// rows from the tile's first row, and the grid of its split reduce (one thread per
// four outputs).
bool tile_launch_fits(const TileLaunch& t, int64_t rows, int64_t K, int64_t N) {
  if (!grid_fits(t.grid_x, t.tp.splits, t.block)) return false;
  if ((int64_t)kTileBM[t.tp.variant] * K * 2 >= k2p32) return false;
  if (t.tp.splits > 1 && rows * N / 4 + 256 >= k2p32) return false;
  return true;
}

}  // namespace

int plan_gemm(int64_t M, int64_t K, int64_t N, int64_t group_size, int cus, bool bf16, Plan& p) {
  p = Plan{};
  const int st = limits_check(M, K, N, group_size);
  if (st != AWQ_OK) return st;
  if (M == 0) return AWQ_OK;
  p = make_plan(M, K, N, eff_group(K, group_size), cus < 1 ? 1 : cus, bf16);
  bool ok;
  if (p.family == 1)
    ok = tile_launch_fits(p.tile, p.rows1, K, N) && (p.rows1 == M || tile_launch_fits(p.tail, M - p.rows1, K, N));
  else
    ok = grid_fits(p.grid_x, p.grid_y, p.block);
  return ok ? AWQ_OK : AWQ_ERR_UNSUPPORTED;
}

int64_t moe_tiles(int64_t S, int64_t E, int64_t block_rows) {
  const int64_t big = int64_t(1) << 40;
  if (S < 0 || E < 1 || block_rows < 1 || S >= big || E >= big) return -1;
  return (S + block_rows - 1) / block_rows + E;
}

int plan_moe(int64_t T, int64_t topk, int64_t E, int64_t K, int64_t N, int64_t group_size, int cus, MoePlan& mp) {
  mp = MoePlan{};
  if (T < 0 || topk < 1 || E < 1) return AWQ_ERR_SHAPE;
  if (T > kMaxDim || topk > kMaxDim) return AWQ_ERR_UNSUPPORTED;
  int st = limits_check(T * topk, K, N, group_size);
  if (st != AWQ_OK) return st;
  if (E > 1024 || T * topk >= (int64_t(1) << 30)) return AWQ_ERR_UNSUPPORTED;
  if (T * K * 2 >= k2p32) return AWQ_ERR_UNSUPPORTED;  // gathered rows use 32-bit offsets
  if (T == 0) return AWQ_OK;
  if (cus < 1) cus = 1;
  const int64_t S = T * topk;
  const int g = eff_group(K, group_size);
  // Few tokens: the skinny family batched over experts, each block taking up to 16
  // of its expert's routed tokens as rows, no alignment pass.  Up to 16 tokens always;
  // up to 64 when the experts average at most 8 slots (most experts then need one
  // 16-row chunk and stream their weights once) and each expert's packed weight is at
  // least 2 MB (shorter streams lose to the grouped tiles: per-block fixed costs and
  // the empty later chunks weigh more).  Measured, 4096 -> 2048 layers, 64 experts
  // top-2: 17 tokens 81.9 -> 47.2 us, 64 tokens 111.6 -> 85.5 us; 2048 -> 1024, 128
  // experts top-8, 64 tokens: 70.8 on the tiles against 94.6.
  mp.tiles_e = (N + kSkinnyCols - 1) / kSkinnyCols;
  mp.chunks = (T + kSkinnyMaxM - 1) / kSkinnyMaxM;
  const bool few = T <= kSkinnyMaxM || (T <= kSkinnyExpertsMaxT && S <= 8 * E && K * (N / 2) >= (int64_t(1) << 21));
  const int64_t blocks = E * mp.chunks * mp.tiles_e;
  if (few && blocks < (int64_t(1) << 31) &&
      plan_skinny(T < kSkinnyMaxM ? T : kSkinnyMaxM, K, blocks * kSkinnyCols, g, cus, mp.sk) &&
      grid_fits(mp.sk.n_tiles, mp.sk.splits, 64 * mp.sk.waves)) {
    mp.skinny = true;
    if (mp.sk.splits > 1) {
      if (mp.sk.atomic) mp.accum_bytes = skinny_accum_entries(mp.sk) * 12;
      else mp.partial_bytes = (int64_t)mp.sk.n_tiles * mp.sk.splits * mp.sk.mrows * kSkinnyCols * 4;
    }
    return AWQ_OK;
  }
  mp.sk = SkinnyPlan{};
  mp.variant = moe_tile_variant(S / E, &mp.block_rows);
  mp.tiles = moe_tiles(S, E, mp.block_rows);
  // Grids of the launches: 256-row tables take a second launch of two 64-row parts
  // per entry on 256 threads.
  const int bn = kTileBN[mp.variant];
  if (!grid_fits(tile_blocks(mp.tiles, N, bn), 1, kTileThreads[mp.variant])) return AWQ_ERR_UNSUPPORTED;
  if (mp.variant == 0 && !grid_fits(tile_blocks(mp.tiles * 2, N, bn), 1, kTileThreads[1])) return AWQ_ERR_UNSUPPORTED;
  // Scratch: tile table (16-byte entries), offsets, sorted slots.
  mp.scratch_bytes = mp.tiles * 16 + (E + 1 + S + 4) * 4;
  return AWQ_OK;
}

int plan_route(int64_t T, int64_t E, int64_t row_stride, int64_t groups, int64_t topk_groups, int group_top,
               int64_t topk) {
  if (T < 0 || E < 1 || row_stride < E || groups < 1 || topk < 1 || topk_groups < 1) return AWQ_ERR_SHAPE;
  if (E % groups != 0 || topk_groups > groups || (group_top != 1 && group_top != 2)) return AWQ_ERR_SHAPE;
  if (topk > topk_groups * (E / groups)) return AWQ_ERR_SHAPE;
  if (E > 1024 || topk > kRouteMaxTopk || groups > kRouteMaxGroups || T > kMaxDim) return AWQ_ERR_UNSUPPORTED;
  if (row_stride > (int64_t(1) << 40)) return AWQ_ERR_UNSUPPORTED;
  return AWQ_OK;
}

int plan_norm(int64_t T, int64_t H, int64_t x_stride, int64_t residual_stride, int64_t gates) {
  if (T < 0 || H < 1 || x_stride < H || residual_stride < H || gates < 0) return AWQ_ERR_SHAPE;
  if (gates > 0 && T % gates != 0) return AWQ_ERR_SHAPE;
  if (H > kNormMaxH || T > kMaxDim) return AWQ_ERR_UNSUPPORTED;
  if (x_stride > (int64_t(1) << 36) || residual_stride > (int64_t(1) << 36)) return AWQ_ERR_UNSUPPORTED;
  return AWQ_OK;
}

namespace {

int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// Entries of at most `rows` rows that S slots over E experts can make: an expert with slots
// has one per `rows` of them, so at most one each for min(E, S) experts and one more per
// full block.
int64_t entry_bound(int64_t S, int64_t E, int64_t rows) {
  const int64_t experts = E < S ? E : S;
  const int64_t b = experts + S / rows;
  return b < S ? b : S;
}

// Entries of `rows` rows, about, that T tokens' slots make.
int64_t active_entries(int64_t T, int64_t topk, int64_t E, int64_t rows) {
  // Experts with rows, about, where a token's are distinct: E (1 - (1 - topk / E)^T).
  const int64_t S = T * topk;
  double idle = 1.0;
  for (int64_t t = 0; t < T && idle > 1e-3; ++t) idle *= topk < E ? 1.0 - (double)topk / (double)E : 0.0;
  int64_t active = (int64_t)((double)E * (1.0 - idle) + 0.5);
  if (active < 1) active = 1;
  // Their entries: one each, or, of several, half an entry more than the rows fill (one expert's
  // last is as full as its rows make it).
  const int64_t full = (2 * S + (active - 1) * rows + 2 * rows - 1) / (2 * rows);
  return full > active ? full : active;
}

// K splits of `tiles` column tiles on workgroups of kStreamWaves waves, one per compute unit at a time,
// that meet inside the kernel; returns the cost in hundredths of a microsecond (MI355X, a call in a
// graph).  350 beside the stream; a k-step of 32 takes a compute unit's waves 100 to 125 by the rows (32
// rows, which unpacking and rescaling bound: 120 and 220 for every 32 rows of a group), or what HBM gives (160 with all
// of the units at it); a round of workgroups 100 beside; the join of the splits 250 (32 rows 450) and
// a share by the rows for each, and of 32 rows 900 for every round after the first: its workgroups begin anew
// and leave 32 or 64 KB of sums each (us, fp16, splits over rounds: 300 x 2048 -> 8192, g 64, 1 over 2 38, 2 over
// 3 46, 4 over 5 66; 96 x 8192 -> 8192, 2 over 1 35, 3 over 2 50, 8 over 3 55).  Measured against forced split counts, us: 1 x 4096 -> 4096 fp16, 4, 8, 12, 16
// splits 10.4, 8.3, 8.2, 8.9 (8 chosen); 16 x 4096 -> 4096 bf16, 4, 8, 12, 16: 13.0, 12.1, 11.8, 14.0 (8);
// 4 x 4096 -> 2 x 11008, 3, 4, 5, 6: 20.7, 16.7, 16.4, 23.0 (4); 32 x 4096 -> 2 x 11008, 2, 3, 4, 5: 35.9, 30.6,
// 27.9, 28.4 (4); 1 x 11008 -> 4096, 4, 8, 12, 16: 19.2, 13.1, 11.4, 11.9 (11); 16 x 8192 -> 28672, 1, 2, 3, 4:
// 55.0, 34.9, 42.7, 39.0 (2).  (The stream's part is from before the waves' priorities: one round without
// splits takes 0.75 to 0.95 of what it says.  Over ten weights, 17 to 1400 rows and both types the choice of splits and
// tiles is 1.8% slower than the best of all of them in the mean, 36% at most.)
int64_t choose_splits8(int64_t tiles, int64_t ksteps, int64_t g, bool gated, int rows, int64_t cus, int& splits,
                       int& steps) {
  const int64_t parts = gated ? kStreamWaves / 2 : kStreamWaves;
  const int64_t step = rows == 1 ? 100 : rows <= 8 ? 105 : rows == 16 ? 125 : 120 + 220 * 32 / g;
  const int64_t share = rows == 1 ? 20 : rows <= 8 ? 25 : rows == 16 ? 37 : gated ? 95 : 70;
  int64_t best = -1, last = 0;
  for (int64_t want = 1; want <= kExpertMaxSplits && last != 1; ++want) {
    const int64_t st = (ksteps + want * parts - 1) / (want * parts);
    if (best >= 0 && st == last) continue;  // the same splits
    last = st;
    const int64_t sp = (ksteps + st * parts - 1) / (st * parts);
    const int64_t rounds = (tiles * sp + cus - 1) / cus;
    const int64_t hbm = 160 * tiles * sp / (rounds * cus);
    int64_t cost = 350 + rounds * (st * (hbm > step ? hbm : step) + 100);
    if (sp > 1) cost += (rows == 32 ? 450 : 250) + sp * share * (gated ? 2 : 1);
    if (sp > 1 && rows == 32) cost += (rounds - 1) * 900;
    if (best >= 0 && cost >= best) continue;
    best = cost;
    steps = (int)st;
    splits = (int)sp;
  }
  return best;
}

// Row tiles of M rows, where they cost less than `best`: their height and K splits.  In hundredths of a
// microsecond: a k-tile of 64 takes a tile of 256, 192, 128, 64 rows 166, 145, 110, 88 (unpacking the
// weights is the same for all), and 0.4 more with groups of 32; a round of tiles 800 beside; the
// splits' fp32 sums are written and read at 6 TB/s by a kernel more.  Streamed / best tiles (height / splits),
// us in a graph: 4096 -> 4096 fp16, 500 rows 31.9 / 36.5 (128 / 4), 750 59.7 / 45.9 (192 / 4), 1500 92 / 71.5 (192 / 2);
// 11008 -> 4096 bfloat16, 80 rows 32.2 / 34.9 (64 / 8), 200 49.3 / 42.0 (128 / 8), 1000 158 / 110 (256 / 4); 4096 ->
// 2 x 11008, 80 rows 57.0 / 46.1 (128 / 2), 500 182 / 111 (256 / 1); 2048 -> 8192, g 64, 200 rows 21.4 / 30.3, 300
// 40.3 / 34.8 (192 / 4), 1000 80 / 50.6 (128 / 1).
void choose_tiles(int64_t M, int64_t K, int64_t N, int64_t g, int64_t cus, bool gated, int64_t best, DensePlan& p) {
  const int64_t cols = gated ? kExpertTileCols / 2 : kExpertTileCols, wide = gated ? 2 * N : N;
  const int64_t tiles_n = (N + cols - 1) / cols;
  // Splits are whole groups and whole k-tiles; one group, pairs of k-tiles.
  int64_t unit = g == K ? 128 : g;
  if (unit % 64 != 0) unit *= 2;
  const int heights[4] = {256, 192, 128, 64}, cost[4] = {166, 145, 110, 88};
  for (int i = 0; i < 4; ++i) {
    const int64_t tiles = (M + heights[i] - 1) / heights[i] * tiles_n;
    for (int64_t want = 1; want <= 8; ++want) {
      const int64_t kps = want == 1 ? K : (K / want + unit - 1) / unit * unit;
      const int64_t splits = (K + kps - 1) / kps;
      if (splits != want) continue;
      const int64_t rounds = (tiles * splits + cus - 1) / cus;
      int64_t c = rounds * ((kps + 63) / 64 * (cost[i] + cost[i] * 2 / 5 * 32 / g) + 800);
      if (splits > 1) c += 400 + 2 * splits * M * wide * 4 / 60000;
      if (best >= 0 && c >= best) continue;
      best = c;
      p = DensePlan{};
      p.rows = heights[i];
      p.col_tiles = (int)tiles_n;
      p.splits = (int)splits;
      p.kps = (int)kps;
      p.grid = tiles * splits;
      if (splits > 1) p.sums_bytes = splits * M * wide * 4;
    }
  }
}

// K splits of a streaming plan.  In tenths of a microsecond (MI355X): a workgroup alone on a
// compute unit takes 7 per k-step and wave, two together 12, and each round of two 30 for its
// fixed part, so the busiest compute unit's n workgroups decide; every split also writes and
// reads its fp32 sums once (4 TB/s), and splits of a gated product cost the kernel that joins
// them.  Measured against forced split counts, us per call: one token through 8 x 4096 -> 14336,
// gated: 1, 2, 3, 4, 9 splits 56, 35.6, 36.5, 32.5, 34.3 (4 chosen: 448 workgroups); 45 tokens
// over 64 x 2048 -> 1408: 1, 2, 3, 9 splits 65.3, 67.4, 70.5, 71.3 (1 chosen); one expert 4096 ->
// 4096, 256 rows: 2, 3 splits 33.5, 37.3 (2), 1024 rows: 1, 2 splits 80, 88 (1).
void choose_splits(int64_t T, int64_t topk, int64_t E, int64_t K, int64_t wide, int64_t cus, bool gated, ExpertPlan& p) {
  const int64_t S = T * topk;
  const int64_t entries = active_entries(T, topk, E, p.block_rows);
  const int64_t parts = gated ? 2 : 4;  // waves of a workgroup along K
  const int64_t ksteps = K / 32;
  int64_t best = -1;
  for (int64_t want = 1; want <= kExpertMaxSplits; ++want) {
    const int64_t steps = (ksteps + want * parts - 1) / (want * parts);
    const int64_t splits = (ksteps + steps * parts - 1) / (steps * parts);
    const int64_t n = (entries * p.col_tiles * splits + cus - 1) / cus;
    int64_t cost = steps * (12 * (n / 2) + 7 * (n % 2)) + 30 * ((n + 1) / 2);
    if (!gated || splits > 1) cost += splits * S * wide / 50000;
    if (gated && splits > 1) cost += 45;
    if (best >= 0 && cost >= best) continue;
    best = cost;
    p.steps = (int)steps;
    p.splits = (int)splits;
  }
}

int plan_expert(int64_t T, int64_t topk, int64_t E, int64_t K, int64_t N, int cus, bool gated, ExpertPlan& p) {
  p = ExpertPlan{};
  const int64_t S = T * topk;
  const int64_t wide = gated ? 2 * N : N;
  if (K * (wide / 2) >= k2p32 - 4096) return AWQ_ERR_UNSUPPORTED;  // 32-bit offsets into one expert's weight
  // Few rows per expert, or too few row tiles to fill a third of the card.  Streamed / tiles, us:
  // 8 x 14336 -> 4096, top 2, 512 tokens (64 tiles) 286 / 355, 768 (96) 398 / 373, 1024 (128) 514 /
  // 374; one expert 4096 -> 4096, 1024 rows (64) 80 / 121, 2048 (128) 147 / 128; 80 tiles: 8 x 4096
  // -> 2048, 1200 tokens 104 / 118, gate_up of 600 tokens 8 x 4096 -> 2048 127 / 114.
  const int64_t tile_cols = gated ? kExpertTileCols / 2 : kExpertTileCols;
  const int64_t row_tiles = (S + kExpertTileRows - 1) / kExpertTileRows * ((N + tile_cols - 1) / tile_cols);
  p.stream = S <= kExpertStreamRows * E || 3 * row_tiles <= cus;
  if (p.stream) {
    p.ranked = S <= kExpertRankSlots;
    p.rows = S <= 4 ? 4 : S <= 8 ? 8 : S < kExpertWideRows * E ? 16 : 32;
    p.block_rows = p.rows == 32 ? 32 : 16;
    p.col_tiles = (int)((N + kExpertStreamCols - 1) / kExpertStreamCols);
    p.tiles = p.ranked ? entry_bound(S, E, p.block_rows) : moe_tiles(S, E, p.block_rows);
    p.by_xcd = p.tiles >= kExpertXcdEntries;
    if (p.by_xcd) p.tiles = round_up(p.tiles, 8);
    choose_splits(T, topk, E, K, wide, cus, gated, p);
    p.grid = p.tiles * p.col_tiles * p.splits;
    p.sums_bytes = gated && p.splits == 1 ? 0 : round_up(p.splits * S * wide * 4, 256);
    if (!p.ranked) p.table_bytes = round_up(p.tiles * 16 + (E + 1 + S) * 4, 256);
  } else {
    p.rows = p.block_rows = kExpertTileRows;
    p.tiles = moe_tiles(S, E, p.block_rows);
    p.col_tiles = (int)((N + tile_cols - 1) / tile_cols);
    p.grid = 2 * p.tiles * p.col_tiles;  // long entries, then short ones
    p.table_bytes = round_up(p.tiles * 16 + (E + 1 + S) * 4, 256);
    p.sums_bytes = gated ? 0 : round_up(S * N * 4, 256);
  }
  return grid_fits(p.grid, 1, p.stream ? 256 : 512) ? AWQ_OK : AWQ_ERR_UNSUPPORTED;
}

}  // namespace

namespace {

// The sizes of one or both products of routed experts.
int check_experts(int64_t T, int64_t topk, int64_t E, int64_t K, int64_t inner, int64_t N, int64_t group_size, bool up,
                  bool down) {
  if (T < 0 || topk < 1 || E < 1) return AWQ_ERR_SHAPE;
  if (inner < 1 || inner > kMaxDim) return inner < 1 ? AWQ_ERR_SHAPE : AWQ_ERR_UNSUPPORTED;
  if (T > kMaxDim || topk > kMaxDim || E > 1024) return AWQ_ERR_UNSUPPORTED;
  const int64_t S = T * topk;
  // h: read with 32-bit offsets, written by one thread per four values.
  if (S <= kMaxDim && S * inner * 2 >= k2p32 - 4096) return AWQ_ERR_UNSUPPORTED;
  if (up) {
    const int st = limits_check(S, K, 2 * inner, group_size);
    if (st != AWQ_OK) return st;
    if (inner % 32 != 0) return AWQ_ERR_UNSUPPORTED;  // the halves meet on a whole 16-byte piece
    if (T * K * 2 >= k2p32 - 4096) return AWQ_ERR_UNSUPPORTED;  // gathered rows use 32-bit offsets
  }
  if (down) {
    const int st = limits_check(S, inner, N, group_size);
    if (st != AWQ_OK) return st;
    if (T * (N / 4) + 256 >= k2p32) return AWQ_ERR_UNSUPPORTED;  // one thread per four outputs
  }
  return AWQ_OK;
}

}  // namespace

int plan_experts(int64_t T, int64_t topk, int64_t E, int64_t K, int64_t inner, int64_t N, int64_t group_size,
                 int cus, bool up, bool down, ExpertsPlan& p) {
  p = ExpertsPlan{};
  const int ok = check_experts(T, topk, E, K, inner, N, group_size, up, down);
  if (ok != AWQ_OK) return ok;
  const int64_t S = T * topk;
  if (T == 0) return AWQ_OK;
  if (cus < 1) cus = 1;
  if (up) {
    const int st = plan_expert(T, topk, E, K, inner, cus, true, p.up);
    if (st != AWQ_OK) return st;
    p.sorted_bytes = p.up.table_bytes;
    p.sums_bytes = p.up.sums_bytes;
    if (down) p.h_bytes = round_up(S * inner * 2, 256);
  }
  if (down) {
    const int st = plan_expert(T, topk, E, inner, N, cus, false, p.down);
    if (st != AWQ_OK) return st;
    if (p.down.table_bytes > p.sorted_bytes) p.sorted_bytes = p.down.table_bytes;
    if (p.down.sums_bytes > p.sums_bytes) p.sums_bytes = p.down.sums_bytes;
    p.two_terms = up && p.up.ranked && p.down.ranked && p.down.rows <= 16;
    if (p.two_terms) p.h_bytes *= 2;
  }
  return AWQ_OK;
}

int plan_layer(int64_t T, int64_t topk, int64_t E, int64_t K, int64_t inner, int64_t N, int64_t group_size, int cus,
               LayerPlan& p) {
  p = LayerPlan{};
  int st = check_experts(T, topk, E, K, inner, N, group_size, true, true);
  if (st != AWQ_OK || T == 0) return st;
  const int64_t S = T * topk;
  if (S > kExpertRankSlots) return AWQ_ERR_UNSUPPORTED;
  if (K * inner >= k2p32 - 4096 || inner * (N / 2) >= k2p32 - 4096) return AWQ_ERR_UNSUPPORTED;  // one expert's weight
  if (cus < 1) cus = 1;
  p.rows = T == 1 ? 1 : T <= 4 ? 4 : T <= 8 ? 8 : 16;  // a token goes to an expert once
  p.router_waves = E <= 16 ? 8 : E <= 64 ? 4 : E <= 128 ? 2 : 1;
  p.up_tiles = (int)((inner + kExpertStreamCols - 1) / kExpertStreamCols);
  p.down_tiles = (int)((N + kExpertStreamCols - 1) / kExpertStreamCols);
  const int64_t active = active_entries(T, topk, E, 16);
  choose_splits8(active * p.up_tiles, K / 32, eff_group(K, group_size), true, p.rows, cus, p.up_splits, p.up_steps);
  choose_splits8(active * p.down_tiles, inner / 32, eff_group(inner, group_size), false, p.rows, cus, p.down_splits,
                 p.down_steps);
  if (p.rows == 1 && p.down_steps * kStreamWaves * 32 > kLayerCols) p.rows = 4;
  const int64_t entries = entry_bound(S, E, 16);
  const int64_t up_items = entries * p.up_tiles * p.up_splits, down_items = entries * p.down_tiles * p.down_splits;
  const int64_t items = up_items > down_items ? up_items : down_items;
  if (up_items >= (int64_t(1) << 30) || down_items >= (int64_t(1) << 30)) return AWQ_ERR_UNSUPPORTED;
  p.workgroups = items < cus ? items : cus;  // one per compute unit
  p.n_counts = (16 + kExpertRankSlots) * kLayerStride + p.down_tiles + (p.up_splits > 1 && p.rows > 1 ? entries * p.up_tiles : 0);
  p.counts_bytes = round_up(p.n_counts * 4, 256);
  p.logits_bytes = round_up(T * E * 4, 256);
  p.ids_bytes = round_up(S * 4, 256);
  p.h_bytes = round_up(2 * S * inner * 2, 256);
  if (p.rows == 1) p.up_bytes = round_up(S * p.up_splits * 2 * inner * 4, 256);
  else if (p.up_splits > 1) p.up_bytes = round_up(entries * p.up_tiles * p.up_splits * 2 * p.rows * kExpertStreamCols * 4, 256);
  p.down_bytes = round_up(p.down_splits * S * N * 4, 256);
  // 32-bit offsets into h and the sums.
  if (2 * S * inner * 2 >= k2p32 || p.down_splits * S * N * 4 >= k2p32 || p.up_bytes >= k2p32) return AWQ_ERR_UNSUPPORTED;
  return AWQ_OK;
}

int plan_dense(int64_t M, int64_t K, int64_t N, int64_t group_size, int cus, bool gated, DensePlan& p) {
  p = DensePlan{};
  if (N < 1 || N > kMaxDim) return N < 1 ? AWQ_ERR_SHAPE : AWQ_ERR_UNSUPPORTED;
  const int64_t wide = gated ? 2 * N : N;
  const int st = limits_check(M, K, wide, group_size);
  if (st != AWQ_OK) return st;
  if (N % 32 != 0) return AWQ_ERR_UNSUPPORTED;                     // halves of whole 16-byte pieces
  if (K * (wide / 2) >= k2p32 - 4096) return AWQ_ERR_UNSUPPORTED;  // 32-bit offsets into the weight
  if (M == 0) return AWQ_OK;
  if (cus < 1) cus = 1;
  // 32-bit offsets into x (streamed) or a tile's rows of it.
  const bool can_stream = M * K * 2 < k2p32 - 4096, can_tile = int64_t(kExpertTileRows) * K * 2 < k2p32 - 4096;
  int64_t best = -1;
  if (can_stream) {
    p.stream = true;
    p.rows = M == 1 ? 1 : M <= 4 ? 4 : M <= 8 ? 8 : M <= 16 ? 16 : 32;
    const int64_t block_rows = p.rows == 32 ? 32 : 16;
    p.col_tiles = (int)((N + kExpertStreamCols - 1) / kExpertStreamCols);
    const int64_t tiles = (M + block_rows - 1) / block_rows * p.col_tiles;
    best = choose_splits8(tiles, K / 32, eff_group(K, group_size), gated, p.rows, cus, p.splits, p.steps);
    p.grid = tiles * p.splits;
    if (p.splits > 1) {
      p.counter_bytes = tiles * 4;
      p.sums_bytes = p.grid * p.rows * (gated ? 2 : 1) * kExpertStreamCols * 4;
    }
  }
  if (can_tile && M > kExpertStreamRows) choose_tiles(M, K, N, eff_group(K, group_size), cus, gated, best, p);
  if (p.grid == 0) return AWQ_ERR_UNSUPPORTED;
  const bool join = !p.stream && p.splits > 1;  // a thread per eight columns
  if (join && !grid_fits((M * (N / 8) + 255) / 256, 1, 256)) return AWQ_ERR_UNSUPPORTED;
  return grid_fits(p.grid, 1, 512) && p.grid < (int64_t(1) << 31) ? AWQ_OK : AWQ_ERR_UNSUPPORTED;
}

int plan_rtn(int64_t K, int64_t N, int64_t group_size, int sym, RtnPlan& p) {
  p = RtnPlan{};
  const int st = format_check(K, N, group_size);
  if (st != AWQ_OK) return st;
  if (sym != 0 && sym != 1) return AWQ_ERR_SHAPE;
  if (K > kMaxDim || N > kMaxDim) return AWQ_ERR_UNSUPPORTED;
  p = rtn_plan(K, N, eff_group(K, group_size));
  return grid_fits(p.grid, 1, p.block) ? AWQ_OK : AWQ_ERR_UNSUPPORTED;
}

}  // namespace awq
