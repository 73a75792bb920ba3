// The planners of awq_gemm_fused and awq_moe_layer (plan_dense and plan_layer in
// w4a16_weight_only_amd/csrc/awq_plan.cpp), on the CPU.  Without arguments: a sweep of sizes, each plan checked
// against what the kernels rely on (launches within HIP's limits that cover every row and column; K
// splits that cover K once, none of them empty, each whole groups where it is row tiles'; 32-bit
// offsets; a workspace that holds what is written).  Prints "plans checked: <n>" and exits 0, or prints the
// first failures and exits 1.  With "query": lines "M K N group_size gated" in, "status stream rows splits" out.
#include <cinttypes>
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "../include/awq_w4a16.h"
#include "../w4a16_weight_only_amd/csrc/awq_plan.h"

using namespace awq;

namespace {

long g_checked = 0, g_failed = 0;
char g_ctx[256];

void fail(const char* what, int line) {
  std::fprintf(stderr, "FAIL line %d: %s  [%s]\n", line, what, g_ctx);
  if (++g_failed >= 20) std::exit(1);
}
#define CHECK(c) \
  do {           \
    if (!(c)) fail(#c, __LINE__); \
  } while (0)

constexpr int64_t k2p32 = int64_t(1) << 32;

void check_splits(int64_t ksteps, int splits, int steps, bool gated) {
  const int64_t run = (int64_t)steps * (gated ? kStreamWaves / 2 : kStreamWaves);
  CHECK(steps >= 1 && splits >= 1 && splits <= kExpertMaxSplits);
  CHECK(run * splits >= ksteps && run * (splits - 1) < ksteps);
}

void dense(int64_t M, int64_t K, int64_t N, int64_t gs, bool gated, int cus) {
  std::snprintf(g_ctx, sizeof g_ctx, "dense M %" PRId64 " K %" PRId64 " N %" PRId64 " g %" PRId64 " gated %d cus %d", M, K, N, gs, gated, cus);
  DensePlan p;
  const int st = plan_dense(M, K, N, gs, cus, gated, p);
  ++g_checked;
  const int64_t wide = gated ? 2 * N : N;
  if (limits_check(M, K, wide, gs) != AWQ_OK) {
    CHECK(st != AWQ_OK);
    return;
  }
  if (st != AWQ_OK) {
    CHECK(st == AWQ_ERR_UNSUPPORTED);
    CHECK(N % 32 != 0 || K * wide / 2 >= k2p32 - 4096 || 256 * K * 2 >= k2p32 - 4096 || M * K * 2 >= k2p32 - 4096 || M * N > (int64_t(1) << 30));
    return;
  }
  if (M == 0) {
    CHECK(p.grid == 0 && p.sums_bytes == 0 && p.counter_bytes == 0);
    return;
  }
  const int64_t g = gs == -1 ? K : gs;
  CHECK(N % 32 == 0 && K * wide / 2 < k2p32);
  CHECK(p.grid >= 1 && p.grid * 512 < k2p32);
  if (p.stream) {
    CHECK(p.rows == 1 || p.rows == 4 || p.rows == 8 || p.rows == 16 || p.rows == 32);
    CHECK(p.rows == 32 || p.rows >= M);
    const int64_t blocks = p.rows == 32 ? (M + 31) / 32 : 1;
    CHECK((int64_t)p.col_tiles * 256 >= N && (int64_t)(p.col_tiles - 1) * 256 < N);
    CHECK(p.grid == blocks * p.col_tiles * p.splits);
    check_splits(K / 32, p.splits, p.steps, gated);
    CHECK(M * K * 2 < k2p32);
    const int64_t share = (int64_t)p.rows * (gated ? 2 : 1) * 256 * 4;
    CHECK(share * p.splits < k2p32);
    if (p.splits > 1) {
      CHECK(p.counter_bytes >= blocks * p.col_tiles * 4);
      CHECK(p.sums_bytes >= p.grid * share);
    }
  } else {
    CHECK(p.rows == 64 || p.rows == 128 || p.rows == 192 || p.rows == 256);
    const int64_t cols = gated ? 128 : 256, blocks = (M + p.rows - 1) / p.rows;
    CHECK((int64_t)p.col_tiles * cols >= N && (int64_t)(p.col_tiles - 1) * cols < N);
    CHECK(p.grid == blocks * p.col_tiles * p.splits);
    CHECK((int64_t)p.kps * p.splits >= K && (int64_t)p.kps * (p.splits - 1) < K);
    if (p.splits > 1) {
      CHECK(p.kps % 64 == 0 && (g == K || p.kps % g == 0));
      CHECK(g != K || p.kps % 128 == 0);
      CHECK(p.sums_bytes >= p.splits * M * wide * 4);
      CHECK((M * (N / 8) + 255) / 256 * 256 < k2p32);
    } else {
      CHECK(p.kps == K);
    }
    CHECK(256 * K * 2 < k2p32);
  }
}

void layer(int64_t T, int64_t topk, int64_t E, int64_t K, int64_t inner, int64_t N, int64_t gs, int cus) {
  std::snprintf(g_ctx, sizeof g_ctx, "layer T %" PRId64 " topk %" PRId64 " E %" PRId64 " K %" PRId64 " inner %" PRId64 " N %" PRId64 " g %" PRId64 " cus %d", T, topk, E, K, inner, N, gs, cus);
  LayerPlan p;
  const int st = plan_layer(T, topk, E, K, inner, N, gs, cus, p);
  ++g_checked;
  ExpertsPlan parts;
  const int ps = plan_experts(T, topk, E, K, inner, N, gs, cus, true, true, parts);
  if (ps != AWQ_OK || T == 0 || T * topk > kExpertRankSlots) {
    CHECK(T == 0 || st != AWQ_OK);
    return;
  }
  if (st != AWQ_OK) {
    CHECK(st == AWQ_ERR_UNSUPPORTED && (4 * T * topk * inner > k2p32 / 64 || T * topk * N > k2p32 / 512 || inner > (1 << 20) || N > (1 << 20)));
    return;
  }
  const int64_t S = T * topk;
  const int64_t entries = (E < S ? E : S) + (S - (E < S ? E : S)) / 16;  // at most
  CHECK(p.rows == 1 || p.rows == 4 || p.rows == 8 || p.rows == 16);
  CHECK(p.rows == 16 || p.rows >= T);
  if (p.rows == 1) CHECK(T == 1 && (int64_t)p.down_steps * kStreamWaves * 32 <= kLayerCols);
  CHECK((int64_t)p.up_tiles * 256 >= inner && (int64_t)(p.up_tiles - 1) * 256 < inner);
  CHECK((int64_t)p.down_tiles * 256 >= N && (int64_t)(p.down_tiles - 1) * 256 < N);
  check_splits(K / 32, p.up_splits, p.up_steps, true);
  check_splits(inner / 32, p.down_splits, p.down_steps, false);
  CHECK(entries * p.up_tiles * p.up_splits < (1 << 30) && entries * p.down_tiles * p.down_splits < (1 << 30));
  CHECK(p.workgroups >= 1 && p.workgroups <= (cus < 1 ? 1 : cus));
  CHECK(p.router_waves == 1 || p.router_waves == 2 || p.router_waves == 4 || p.router_waves == 8);
  CHECK(p.n_counts * 4 <= p.counts_bytes && p.counts_bytes % 256 == 0);
  CHECK(p.n_counts >= (16 + kExpertRankSlots) * kLayerStride + p.down_tiles);
  CHECK(p.logits_bytes >= T * E * 4 && p.ids_bytes >= S * 4 && p.h_bytes >= 4 * S * inner && p.down_bytes >= p.down_splits * S * N * 4);
  CHECK(4 * S * inner < k2p32 && p.down_splits * S * N * 4 < k2p32 && p.up_bytes < k2p32);
  if (p.rows == 1) {
    CHECK(p.up_bytes >= S * p.up_splits * 2 * inner * 4);
  } else if (p.up_splits > 1) {
    CHECK(p.up_bytes >= entries * p.up_tiles * p.up_splits * 2 * p.rows * 256 * 4);
    CHECK(p.n_counts >= (16 + kExpertRankSlots) * kLayerStride + p.down_tiles + entries * p.up_tiles);
  }
  CHECK(K * inner < k2p32 && inner * N / 2 < k2p32);
  CHECK(p.logits_bytes % 256 == 0 && p.ids_bytes % 256 == 0 && p.h_bytes % 256 == 0 && p.up_bytes % 256 == 0);
}

uint64_t g_state = 88172645463325252ull;
uint64_t rnd() {
  g_state ^= g_state << 13;
  g_state ^= g_state >> 7;
  g_state ^= g_state << 17;
  return g_state;
}
int64_t log_size(int bits) {  // 1 .. 2^bits, spread over the logarithm
  const int b = (int)(rnd() % (uint64_t)(bits + 1));
  return (int64_t)(rnd() % ((uint64_t(1) << b) | 1)) + (int64_t(1) << b) / 2 + 1;
}

}  // namespace

int main(int argc, char** argv) {
  if (argc > 1 && std::strcmp(argv[1], "query") == 0) {
    int64_t M, K, N, gs;
    int gated;
    while (std::scanf("%" SCNd64 " %" SCNd64 " %" SCNd64 " %" SCNd64 " %d", &M, &K, &N, &gs, &gated) == 5) {
      DensePlan p;
      const int st = plan_dense(M, K, N, gs, 256, gated != 0, p);
      std::printf("%d %d %d %d\n", st, (int)p.stream, p.rows, p.splits);
    }
    return 0;
  }
  const int cus[] = {256, 1, 64, 304};
  const int64_t groups[] = {-1, 32, 64, 96, 128, 160, 256, 384, 1024};
  for (long i = 0; i < 400000; ++i) {
    const int64_t gs = groups[rnd() % 9];
    const int64_t step = gs == -1 ? 32 : gs;
    const int64_t K = rnd() % 50 == 0 ? log_size(25) : step * ((log_size(rnd() % 4 == 0 ? 24 : 15) + step - 1) / step);
    const int64_t N = rnd() % 50 == 0 ? log_size(25) : 32 * ((log_size(rnd() % 4 == 0 ? 24 : 15) + 31) / 32);
    const int64_t M = rnd() % 100 == 0 ? 0 : log_size(rnd() % 4 == 0 ? 25 : 13);
    dense(M, K, N, gs, rnd() % 2, cus[rnd() % 4]);
  }
  for (long i = 0; i < 400000; ++i) {
    const int64_t gs = groups[rnd() % 9];
    const int64_t step = gs == -1 ? 32 : gs;
    const int64_t K = rnd() % 50 == 0 ? log_size(25) : step * ((log_size(rnd() % 4 == 0 ? 22 : 14) + step - 1) / step);
    const int64_t inner = rnd() % 50 == 0 ? log_size(25) : step * ((log_size(rnd() % 4 == 0 ? 22 : 14) + step - 1) / step);
    const int64_t N = rnd() % 50 == 0 ? log_size(25) : 32 * ((log_size(rnd() % 4 == 0 ? 22 : 14) + 31) / 32);
    const int64_t topk = 1 + (int64_t)(rnd() % 66);
    const int64_t T = rnd() % 20 == 0 ? (int64_t)(rnd() % 80) : (int64_t)(rnd() % (uint64_t)(64 / (topk > 64 ? 64 : topk) + 1));
    layer(T, topk, log_size(10), K, inner, N, gs, cus[rnd() % 4]);
  }
  if (g_failed) return 1;
  std::printf("plans checked: %ld\n", g_checked);
  return 0;
}
