// Sweep of the routed-expert planner (plan_experts and plan_route in
// w4a16_weight_only_amd/csrc/awq_plan.cpp), built on the CPU with the address and
// undefined-behaviour sanitizers.  Each plan is checked against what the kernels rely on:
//   - launches fit HIP's limits, and cover every entry and column tile;
//   - a table has an entry for every block of rows any routing can make;
//   - the K splits of a streaming plan cover every k-step once, none of them empty;
//   - rows kept hold every entry a workgroup can get;
//   - the workspace holds table, offsets and slots, h, and the sums of all splits;
//   - bad arguments give the documented status.
// Prints "plans checked: <n>" and exits 0, or prints the first failures and exits 1.
#include <cinttypes>
#include <cstdio>
#include <cstdlib>
#include <initializer_list>

#include "../include/awq_w4a16.h"
#include "../w4a16_weight_only_amd/csrc/awq_plan.h"

using namespace awq;

namespace {

long g_checked = 0, g_failed = 0;
char g_ctx[512];

void fail(const char* what, int line) {
  std::fprintf(stderr, "FAIL line %d: %s  [%s]\n", line, what, g_ctx);
  if (++g_failed >= 20) std::exit(1);
}
#define CHECK(c) \
  do {           \
    if (!(c)) fail(#c, __LINE__); \
  } while (0)

constexpr int64_t k2p32 = int64_t(1) << 32;
constexpr int64_t kDim = int64_t(1) << 24;

// Blocks of `rows` slots that S slots over E experts can make at most: the experts with
// slots number at most min(E, S), and a block short of full needs an expert of its own.
int64_t most_blocks(int64_t S, int64_t E, int64_t rows) {
  const int64_t e = E < S ? E : S;
  // e experts with one slot each, the other S - e slots in whole blocks on top of one.
  return e + (S - e) / rows;
}

void check_product(const ExpertPlan& p, int64_t S, int64_t E, int64_t K, int64_t N, bool gated) {
  const int64_t wide = gated ? 2 * N : N;
  CHECK(p.grid >= 1 && p.grid * (p.stream ? 256 : 512) < k2p32);
  CHECK(p.rows >= 1 && p.block_rows >= 1);
  CHECK(p.tiles >= most_blocks(S, E, p.block_rows));
  if (p.stream) {
    CHECK(p.rows == 4 || p.rows == 8 || p.rows == 16 || p.rows == 32);
    CHECK(p.rows >= (S < p.block_rows ? S : p.block_rows));
    CHECK((int64_t)p.col_tiles * 256 >= N && (int64_t)(p.col_tiles - 1) * 256 < N);
    CHECK(p.grid == p.tiles * p.col_tiles * p.splits);
    if (p.by_xcd) CHECK(p.tiles % 8 == 0);
    const int64_t run = (int64_t)p.steps * (gated ? 2 : 4), T = K / 32;
    CHECK(p.steps >= 1 && p.splits >= 1 && p.splits <= kExpertMaxSplits);
    CHECK(run * p.splits >= T && run * (p.splits - 1) < T);
    CHECK(K * wide / 2 < k2p32);
    if (p.ranked) CHECK(S <= 64 && p.table_bytes == 0);
    if (!gated || p.splits > 1) CHECK(p.sums_bytes >= p.splits * S * wide * 4);
    else CHECK(p.sums_bytes == 0);
  } else {
    CHECK(p.splits == 1 && p.block_rows == 256 && !p.ranked);
    CHECK((int64_t)p.col_tiles * (gated ? 128 : 256) >= N);
    CHECK(p.grid == 2 * p.tiles * p.col_tiles);
    if (!gated) CHECK(p.sums_bytes >= S * N * 4);
  }
  if (!p.ranked) CHECK(p.table_bytes >= p.tiles * 16 + (E + 1 + S) * 4);
  CHECK(p.table_bytes % 256 == 0 && p.sums_bytes % 256 == 0);
}

bool product_ok(int64_t S, int64_t K, int64_t N, int64_t gs) {
  return K >= 1 && N >= 1 && K % 32 == 0 && N % 32 == 0 && K <= kDim && N <= kDim && S <= kDim &&
         (gs == -1 || (gs > 0 && gs % 32 == 0 && K % gs == 0));
}

void check(int64_t T, int64_t topk, int64_t E, int64_t K, int64_t inner, int64_t N, int64_t gs, int cus) {
  for (int halves = 1; halves <= 3; ++halves) {
    const bool up = halves & 1, down = halves & 2;
    std::snprintf(g_ctx, sizeof g_ctx,
                  "T=%" PRId64 " topk=%" PRId64 " E=%" PRId64 " K=%" PRId64 " inner=%" PRId64 " N=%" PRId64
                  " g=%" PRId64 " cus=%d up=%d down=%d",
                  T, topk, E, K, inner, N, gs, cus, up, down);
    ExpertsPlan p;
    const int st = plan_experts(T, topk, E, K, inner, N, gs, cus, up, down, p);
    ++g_checked;
    CHECK(st == AWQ_OK || st == AWQ_ERR_SHAPE || st == AWQ_ERR_GROUP || st == AWQ_ERR_UNSUPPORTED);
    if (T < 0 || topk < 1 || E < 1 || inner < 1 || (up && K < 1) || (down && N < 1)) {
      CHECK(st != AWQ_OK);
      continue;
    }
    if (st != AWQ_OK) continue;
    CHECK(T <= kDim && topk <= kDim && E <= 1024);
    const int64_t S = T * topk;
    if (up) CHECK(product_ok(S, K, 2 * inner, gs) && inner % 32 == 0 && T * K * 2 < k2p32);
    if (down) CHECK(product_ok(S, inner, N, gs) && T * (N / 4) < k2p32);
    CHECK(S * inner * 2 < k2p32);
    if (T == 0) {
      CHECK(p.workspace_bytes() == 0);
      continue;
    }
    if (up) check_product(p.up, S, E, K, inner, true);
    if (down) check_product(p.down, S, E, inner, N, false);
    CHECK(p.sorted_bytes >= (up ? p.up.table_bytes : 0) && p.sorted_bytes >= (down ? p.down.table_bytes : 0));
    CHECK(p.sums_bytes >= (up ? p.up.sums_bytes : 0) && p.sums_bytes >= (down ? p.down.sums_bytes : 0));
    CHECK(p.h_bytes >= (up && down ? S * inner * 2 : 0) && p.h_bytes % 256 == 0);
    if (p.two_terms) CHECK(S <= 64 && p.down.rows <= 16 && p.h_bytes % 512 == 0 && p.h_bytes >= 4 * S * inner);
    CHECK(p.workspace_bytes() == p.sorted_bytes + p.h_bytes + p.sums_bytes);
  }
}

uint64_t g_state = 88172645463325252ull;
uint64_t next() {
  g_state ^= g_state << 13;
  g_state ^= g_state >> 7;
  g_state ^= g_state << 17;
  return g_state;
}

}  // namespace

int main() {
  const int64_t edges[] = {INT64_MIN, -1, 0, 1, 31, 32, 33, 64, 4096, kDim - 32, kDim, kDim + 1, INT64_MAX};
  for (int64_t T : edges)
    for (int64_t topk : edges)
      for (int64_t E : {int64_t(-1), int64_t(0), int64_t(1), int64_t(1024), int64_t(1025), INT64_MAX})
        for (int64_t K : edges)
          for (int64_t inner : edges) check(T, topk, E, K, inner, 4096, -1, 256);
  for (int64_t gs : {int64_t(-2), int64_t(-1), int64_t(0), int64_t(16), int64_t(32), int64_t(96), INT64_MIN, INT64_MAX})
    for (int64_t N : edges) check(3, 2, 8, 96, 192, N, gs, 256);
  const int64_t groups[] = {32, 64, 96, 128, -1};
  for (int i = 0; i < 400000; ++i) {
    const int64_t gs = groups[next() % 5];
    const int64_t step = gs == -1 ? 32 : gs;
    const int64_t E = 1 + (int64_t)(next() % (next() % 4 == 0 ? 1024 : 64));
    const int64_t topk = 1 + (int64_t)(next() % 12);
    const int64_t T = (int64_t)(next() % (uint64_t(1) << (1 + next() % 17)));
    const int64_t K = step * (1 + (int64_t)(next() % 200)), inner = step * (1 + (int64_t)(next() % 200));
    const int64_t N = 32 * (1 + (int64_t)(next() % 1000));
    check(T, topk, E, K, inner, N, gs, next() % 8 == 0 ? 1 + (int)(next() % 304) : 256);
  }
  long routes = 0;
  for (int64_t T : edges)
    for (int64_t E : edges)
      for (int64_t groups_n : {int64_t(-1), int64_t(0), int64_t(1), int64_t(8), int64_t(64), int64_t(65), INT64_MAX})
        for (int64_t keep : {int64_t(0), int64_t(1), int64_t(4), INT64_MAX})
          for (int64_t topk : {int64_t(0), int64_t(1), int64_t(8), int64_t(64), int64_t(65), INT64_MAX}) {
            std::snprintf(g_ctx, sizeof g_ctx, "route T=%" PRId64 " E=%" PRId64 " groups=%" PRId64 " keep=%" PRId64
                          " topk=%" PRId64, T, E, groups_n, keep, topk);
            const int st = plan_route(T, E, E, groups_n, keep, 1, topk);
            ++routes;
            if (st != AWQ_OK) continue;
            CHECK(T >= 0 && T <= kDim && E >= 1 && E <= 1024 && groups_n >= 1 && groups_n <= 64 && E % groups_n == 0);
            CHECK(keep >= 1 && keep <= groups_n && topk >= 1 && topk <= 64 && topk <= keep * (E / groups_n));
          }
  if (g_failed) return 1;
  std::printf("plans checked: %ld\n", g_checked + routes);
  return 0;
}
