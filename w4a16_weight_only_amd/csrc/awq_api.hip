// C ABI of the AWQ W4A16 library: argument checks, launch planning, workspace.
// The declarations and their contracts are in include/awq_w4a16.h.
#include <map>
#include <mutex>
#include <utility>
#include <vector>

#include "../../include/awq_w4a16.h"
#include "awq_kernels.h"

using namespace awq;

namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Compute units of the current device (cached per device ordinal).
int device_cus() {
  static std::mutex mu;
  static std::map<int, int> cache;
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return 256;
  std::lock_guard<std::mutex> lock(mu);
  auto it = cache.find(dev);
  if (it != cache.end()) return it->second;
  int cus = 256;
  if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0)
    cus = 256;
  cache[dev] = cus;
  return cus;
}

// Compute units for host-only plan queries: the current device's, or 256 (MI355X)
// when no device is visible.
int query_cus() {
  static const bool visible = [] {
    int count = 0;
    const bool any = hipGetDeviceCount(&count) == hipSuccess && count > 0;
    if (!any) (void)hipGetLastError();
    return any;
  }();
  return visible ? device_cus() : 256;
}

// Library-owned split-K workspace, one per (device, stream), in two buffers:
//   accum    fixed-point words and their float side words; zeroed once at allocation
//            and left zero by every call that uses them, so they never hold anything
//            else between calls;
//   partial  fp32 scratch, fully written before it is read in each call.
// A buffer that must grow is replaced, and the old one is retired, never freed while
// the library is loaded (a graph captured earlier may still hold its address and replay
// into it); awq_release_workspace() frees retired and current buffers on request.  A
// stream that is being captured cannot grow its workspace: that call fails with
// AWQ_ERR_UNSUPPORTED before enqueueing anything.
// Some calls are several launches that hand something over in these buffers (partial sums,
// an alignment's table).  Of two threads' calls on one stream each makes all of its launches
// before the other begins: a call holds the workspace's `launches` from when it gets the
// buffers until its last launch.
typedef std::unique_lock<std::mutex> Launches;
struct Buffer {
  void* ptr = nullptr;
  int64_t bytes = 0;
};
struct Workspace {
  Buffer accum, partial;
  std::mutex launches;
};

std::mutex g_ws_mu;
std::map<std::pair<int, hipStream_t>, Workspace> g_ws;
std::vector<std::pair<int, void*>> g_retired;  // (device, buffer) replaced by a larger one

int ensure(int dev, Buffer& b, int64_t need, bool zero, hipStream_t stream) {
  if (need <= 0 || (b.ptr && need <= b.bytes)) return AWQ_OK;
  hipStreamCaptureStatus cap = hipStreamCaptureStatusNone;
  if (hipStreamIsCapturing(stream, &cap) != hipSuccess) return AWQ_ERR_HIP;
  if (cap != hipStreamCaptureStatusNone) return AWQ_ERR_UNSUPPORTED;
  const int64_t bytes = need + need / 4;  // headroom against frequent regrowth
  void* ptr = nullptr;
  if (hipMalloc(&ptr, (size_t)bytes) != hipSuccess) return AWQ_ERR_HIP;
  // Zeroed in stream order, before any kernel of this stream can use the buffer.
  if (zero && hipMemsetAsync(ptr, 0, (size_t)bytes, stream) != hipSuccess) {
    (void)hipFree(ptr);
    return AWQ_ERR_HIP;
  }
  if (b.ptr) g_retired.emplace_back(dev, b.ptr);
  b.ptr = ptr;
  b.bytes = bytes;
  return AWQ_OK;
}

// The workspace of the current device and the stream, whose launches the caller then holds.
int hold_workspace(hipStream_t stream, int* dev, Workspace** ws, Launches& held) {
  if (hipGetDevice(dev) != hipSuccess) return AWQ_ERR_HIP;
  {
    std::lock_guard<std::mutex> lock(g_ws_mu);
    *ws = &g_ws[{*dev, stream}];
  }
  held = Launches((*ws)->launches);
  return AWQ_OK;
}

int get_workspace(const Plan& p, hipStream_t stream, uint64_t** accum, float** partial, Launches& held) {
  int dev = 0;
  Workspace* ws = nullptr;
  int st = hold_workspace(stream, &dev, &ws, held);
  if (st != AWQ_OK) return st;
  std::lock_guard<std::mutex> lock(g_ws_mu);
  st = ensure(dev, ws->accum, p.accum_bytes, true, stream);
  if (st != AWQ_OK) return st;
  st = ensure(dev, ws->partial, p.partial_bytes, false, stream);
  if (st != AWQ_OK) return st;
  *accum = reinterpret_cast<uint64_t*>(ws->accum.ptr);
  *partial = reinterpret_cast<float*>(ws->partial.ptr);
  return AWQ_OK;
}

// Scratch that is fully written before it is read within one call: the partial
// buffer of the same (device, stream) workspace.
int get_scratch(int64_t bytes, hipStream_t stream, void** out, Launches& held) {
  int dev = 0;
  Workspace* ws = nullptr;
  int st = hold_workspace(stream, &dev, &ws, held);
  if (st != AWQ_OK) return st;
  std::lock_guard<std::mutex> lock(g_ws_mu);
  st = ensure(dev, ws->partial, bytes, false, stream);
  if (st != AWQ_OK) return st;
  *out = ws->partial.ptr;
  return AWQ_OK;
}

// Allocation-free workspace for awq_gemm_noalloc: one file-scope device array per GPU
// (each device that runs the library holds its own copy until the process ends).  The
// first kScratchWordBytes hold fixed-point words and their side words, zero between
// calls like the workspace above (a fill kernel clears them on the device's first call);
// the rest holds fp32 partials, fully written before they are read in each call.  The
// two regions never trade places, so neither kind of plan can break the other's
// invariant.  In host code `scratch` only names the symbol: kernels get the address
// hipGetSymbolAddress returns for the current device.
constexpr int64_t kScratchWordBytes = int64_t(2) << 20;
constexpr int64_t kScratchPartialBytes = int64_t(62) << 20;
__device__ __align__(256) unsigned char scratch[kScratchWordBytes + kScratchPartialBytes];

__global__ void zero_words_kernel(u32x4_t* p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x)
    p[i] = u32x4_t{0u, 0u, 0u, 0u};
}

std::mutex g_scratch_mu;
struct StaticScratch {
  void* ptr;  // address of `scratch` on the device
  std::mutex launches;
};
std::map<int, StaticScratch> g_scratch;  // by device

int get_static_scratch(hipStream_t stream, void** out, Launches& held) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return AWQ_ERR_HIP;
  StaticScratch* at = nullptr;
  {
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    auto it = g_scratch.find(dev);
    if (it == g_scratch.end()) {
      void* ptr = nullptr;
      if (hipGetSymbolAddress(&ptr, HIP_SYMBOL(scratch)) != hipSuccess || ptr == nullptr) return AWQ_ERR_HIP;
      hipLaunchKernelGGL(zero_words_kernel, dim3(256), dim3(256), 0, stream, static_cast<u32x4_t*>(ptr),
                         kScratchWordBytes / 16);
      if (hipGetLastError() != hipSuccess) return AWQ_ERR_HIP;
      it = g_scratch.try_emplace(dev).first;
      it->second.ptr = ptr;
    }
    at = &it->second;
  }
  held = Launches(at->launches);
  *out = at->ptr;
  return AWQ_OK;
}

// The split-K buffers of plan p: the stream's grown workspace, or (noalloc) the static
// scratch, AWQ_ERR_UNSUPPORTED when the plan needs more than it holds.
int workspace_for(const Plan& p, hipStream_t stream, bool noalloc, uint64_t** accum, float** partial, Launches& held) {
  if (!noalloc) return get_workspace(p, stream, accum, partial, held);
  if (p.accum_bytes > kScratchWordBytes || p.partial_bytes > kScratchPartialBytes) return AWQ_ERR_UNSUPPORTED;
  void* base = nullptr;
  const int st = get_static_scratch(stream, &base, held);
  if (st != AWQ_OK) return st;
  *accum = static_cast<uint64_t*>(base);
  *partial = reinterpret_cast<float*>(static_cast<unsigned char*>(base) + kScratchWordBytes);
  return AWQ_OK;
}

}  // namespace

extern "C" {

const char* awq_status_string(int status) {
  switch (status) {
    case AWQ_OK: return "AWQ_OK";
    case AWQ_ERR_NULL: return "AWQ_ERR_NULL: a required pointer is NULL";
    case AWQ_ERR_SHAPE: return "AWQ_ERR_SHAPE: tensor shapes disagree with K, N, group_size (or N % 8 != 0)";
    case AWQ_ERR_GROUP: return "AWQ_ERR_GROUP: group_size must be -1 or a positive divisor of K";
    case AWQ_ERR_ALIGN: return "AWQ_ERR_ALIGN: tensor base pointers must be 16-byte aligned";
    case AWQ_ERR_UNSUPPORTED:
      return "AWQ_ERR_UNSUPPORTED: needs K % 32 == 0, N % 32 == 0, group_size -1 or a multiple of 32, sizes <= 2^24, "
             "launches within the grid and offset limits (or a workspace the call may not allocate)";
    case AWQ_ERR_HIP: return "AWQ_ERR_HIP: the HIP runtime reported an error";
    default: return "AWQ: unknown status";
  }
}

int awq_validate_pack(int64_t K, int64_t N, int64_t group_size, int64_t qweight_rows,
                      int64_t qweight_cols, int64_t qzeros_rows, int64_t qzeros_cols,
                      int64_t scales_rows, int64_t scales_cols, int64_t bias_len) {
  return validate_pack(K, N, group_size, qweight_rows, qweight_cols, qzeros_rows, qzeros_cols, scales_rows,
                       scales_cols, bias_len);
}

int awq_release_workspace(void) {
  std::lock_guard<std::mutex> lock(g_ws_mu);
  int cur = 0;
  if (hipGetDevice(&cur) != hipSuccess) return AWQ_ERR_HIP;
  int st = AWQ_OK;
  auto release = [&](int dev, void* ptr) {
    if (hipSetDevice(dev) != hipSuccess || hipDeviceSynchronize() != hipSuccess || hipFree(ptr) != hipSuccess)
      st = AWQ_ERR_HIP;
  };
  for (auto& r : g_retired) release(r.first, r.second);
  g_retired.clear();
  for (auto& w : g_ws) {
    if (w.second.accum.ptr) release(w.first.first, w.second.accum.ptr);
    if (w.second.partial.ptr) release(w.first.first, w.second.partial.ptr);
  }
  g_ws.clear();
  if (hipSetDevice(cur) != hipSuccess) st = AWQ_ERR_HIP;
  return st;
}

int awq_check_limits(int64_t M, int64_t K, int64_t N, int64_t group_size) {
  Plan p;
  return plan_gemm(M, K, N, group_size, query_cus(), false, p);
}

int awq_gemm_plan(int64_t M, int64_t K, int64_t N, int64_t group_size, int* family, int* splits,
                  int* grid_x, int* grid_y, int* block, int64_t* workspace_bytes) {
  Plan p;
  const int st = plan_gemm(M, K, N, group_size, query_cus(), false, p);
  if (st != AWQ_OK) return st;
  if (family) *family = p.family;
  if (splits) *splits = p.family == 2 ? p.dp.splits : (p.family == 0 ? p.sk.splits : p.tp.splits);
  if (grid_x) *grid_x = (int)p.grid_x;
  if (grid_y) *grid_y = p.grid_y;
  if (block) *block = p.block;
  if (workspace_bytes) *workspace_bytes = p.workspace_bytes();
  return AWQ_OK;
}

int awq_gemm_plan_tail(int64_t M, int64_t K, int64_t N, int64_t group_size, int64_t* rows, int* splits,
                       int* grid_x, int* grid_y, int* block) {
  Plan p;
  const int st = plan_gemm(M, K, N, group_size, query_cus(), false, p);
  if (st != AWQ_OK) return st;
  const bool tail = p.family == 1 && p.rows1 < M;
  if (rows) *rows = tail ? M - p.rows1 : 0;
  if (splits) *splits = tail ? p.tail.tp.splits : 0;
  if (grid_x) *grid_x = tail ? (int)p.tail.grid_x : 0;
  if (grid_y) *grid_y = tail ? p.tail.tp.splits : 0;
  if (block) *block = tail ? p.tail.block : 0;
  return AWQ_OK;
}

namespace {
int dequant_common(const int32_t* qweight, const int32_t* qzeros, const void* scales_f16, int64_t K, int64_t N,
                   int64_t group_size, void* out, bool f16, hipStream_t stream) {
  const int st = limits_check(0, K, N, group_size);
  if (st != AWQ_OK) return st;
  if (!qweight || !qzeros || !scales_f16 || !out) return AWQ_ERR_NULL;
  if (!aligned16(qweight) || !aligned16(qzeros) || !aligned16(scales_f16) || !aligned16(out))
    return AWQ_ERR_ALIGN;
  hipError_t e = awq::launch_dequant(qweight, qzeros, static_cast<const uint16_t*>(scales_f16), (int)K,
                                     (int)N, eff_group(K, group_size), out, f16, stream);
  return e == hipSuccess ? AWQ_OK : AWQ_ERR_HIP;
}
}  // namespace

int awq_dequant(const int32_t* qweight, const int32_t* qzeros, const void* scales_f16, int64_t K,
                int64_t N, int64_t group_size, float* out, struct ihipStream_t* stream) {
  return dequant_common(qweight, qzeros, scales_f16, K, N, group_size, out, false, stream);
}

int awq_dequant_f16(const int32_t* qweight, const int32_t* qzeros, const void* scales_f16, int64_t K,
                    int64_t N, int64_t group_size, void* out_f16, struct ihipStream_t* stream) {
  return dequant_common(qweight, qzeros, scales_f16, K, N, group_size, out_f16, true, stream);
}

int awq_quantize_rtn(const void* w_f16, int64_t K, int64_t N, int64_t group_size, int sym, int32_t* qweight,
                     int32_t* qzeros, void* scales_f16, struct ihipStream_t* stream) {
  RtnPlan p;
  int st = plan_rtn(K, N, group_size, sym, p);
  if (st != AWQ_OK) return st;
  const int g = eff_group(K, group_size);
  if (!w_f16 || !qweight || !qzeros || !scales_f16) return AWQ_ERR_NULL;
  if (!aligned16(w_f16) || !aligned16(qweight) || !aligned16(qzeros) || !aligned16(scales_f16))
    return AWQ_ERR_ALIGN;
  void* scratch = nullptr;
  Launches held;
  if (p.scratch_bytes > 0) {
    st = get_scratch(p.scratch_bytes, stream, &scratch, held);
    if (st != AWQ_OK) return st;
  }
  hipError_t e = awq::launch_quantize_rtn(static_cast<const uint16_t*>(w_f16), (int)K, (int)N, g, sym != 0, qweight,
                                          qzeros, static_cast<uint16_t*>(scales_f16), scratch, stream);
  return e == hipSuccess ? AWQ_OK : AWQ_ERR_HIP;
}

namespace {
int gemm_common(const void* x_f16, const int32_t* qweight, const int32_t* qzeros, const void* scales_f16,
                const void* bias_f16, int64_t M, int64_t K, int64_t N, int64_t group_size, void* y_f16,
                bool bf16, hipStream_t stream, bool noalloc = false) {
  const int st = limits_check(M, K, N, group_size);
  if (st != AWQ_OK) return st;
  if (M == 0) return AWQ_OK;
  if (!x_f16 || !qweight || !qzeros || !scales_f16 || !y_f16) return AWQ_ERR_NULL;
  if (!aligned16(x_f16) || !aligned16(qweight) || !aligned16(qzeros) || !aligned16(scales_f16) ||
      !aligned16(y_f16) || (bias_f16 && !aligned16(bias_f16)))
    return AWQ_ERR_ALIGN;
  const int g = eff_group(K, group_size);
  Plan p;
  const int pst = plan_gemm(M, K, N, group_size, device_cus(), bf16, p);
  if (pst != AWQ_OK) return pst;
  const auto* x = static_cast<const uint16_t*>(x_f16);
  const auto* sc = static_cast<const uint16_t*>(scales_f16);
  const auto* b = static_cast<const uint16_t*>(bias_f16);
  auto* y = static_cast<uint16_t*>(y_f16);
  hipError_t e;
  Launches held;
  if (p.family == 2) {
    uint64_t* accum = nullptr;
    float* partial = nullptr;
    if (p.dp.splits > 1) {
      const int ws = workspace_for(p, stream, noalloc, &accum, &partial, held);
      if (ws != AWQ_OK) return ws;
    }
    float* side = accum ? reinterpret_cast<float*>(accum + decode_entries(p.dp)) : nullptr;
    e = awq::launch_decode(x, qweight, qzeros, sc, b, (int)M, (int)K, (int)N, g, p.dp, accum, side, y, stream);
  } else if (p.family == 0) {
    uint64_t* accum = nullptr;
    float* partial = nullptr;
    if (p.sk.splits > 1) {
      const int ws = workspace_for(p, stream, noalloc, &accum, &partial, held);
      if (ws != AWQ_OK) return ws;
    }
    // Fixed-point plans: the float side words follow the accumulator words.
    if (p.sk.splits > 1 && p.sk.atomic && !bf16)
      partial = reinterpret_cast<float*>(accum + (int64_t)p.sk.n_tiles * p.sk.mrows * awq::kSkinnyCols);
    e = awq::launch_skinny(x, qweight, qzeros, sc, b, (int)M, (int)K, (int)N, g, p.sk, bf16, accum, partial, y,
                           stream);
  } else {
    uint64_t* accum = nullptr;
    float* partial = nullptr;
    if (p.tp.splits > 1 || p.tail.tp.splits > 1) {
      const int ws = workspace_for(p, stream, noalloc, &accum, &partial, held);
      if (ws != AWQ_OK) return ws;
    }
    e = awq::launch_tile(x, qweight, qzeros, sc, b, (int)p.rows1, (int)K, (int)N, g, p.tp, bf16, partial, y,
                         stream);
    if (e == hipSuccess && p.rows1 < M)
      e = awq::launch_tile(x + p.rows1 * K, qweight, qzeros, sc, b, (int)(M - p.rows1), (int)K, (int)N, g,
                           p.tail.tp, bf16, partial, y + p.rows1 * N, stream);
  }
  return e == hipSuccess ? AWQ_OK : AWQ_ERR_HIP;
}
}  // namespace

int64_t awq_moe_tiles(int64_t S, int64_t E, int64_t block_rows) { return moe_tiles(S, E, block_rows); }

int awq_moe_align(const int32_t* expert_ids, int64_t S, int64_t E, int64_t block_rows, int32_t* offsets,
                  int32_t* sorted_slots, int32_t* tile_table, struct ihipStream_t* stream) {
  if (S < 0 || E < 1 || block_rows < 1) return AWQ_ERR_SHAPE;
  if (E > 1024 || S >= (int64_t(1) << 30)) return AWQ_ERR_UNSUPPORTED;
  if (!offsets || !tile_table || (S > 0 && (!expert_ids || !sorted_slots))) return AWQ_ERR_NULL;
  if (!aligned16(tile_table)) return AWQ_ERR_ALIGN;
  const int64_t tiles = awq_moe_tiles(S, E, block_rows);
  hipError_t e = awq::launch_moe_align(expert_ids, (int)S, (int)E, (int)block_rows, (int)tiles, offsets, sorted_slots,
                                       tile_table, stream);
  return e == hipSuccess ? AWQ_OK : AWQ_ERR_HIP;
}

int awq_moe_gemm(const void* x_f16, const int32_t* qweight, const int32_t* qzeros, const void* scales_f16,
                 const int32_t* expert_ids, int64_t T, int64_t topk, int64_t E, int64_t K, int64_t N,
                 int64_t group_size, void* y_f16, struct ihipStream_t* stream) {
  MoePlan mp;
  int st = plan_moe(T, topk, E, K, N, group_size, 0, mp);  // sizes only
  if (st != AWQ_OK) return st;
  if (T == 0) return AWQ_OK;
  if (!x_f16 || !qweight || !qzeros || !scales_f16 || !expert_ids || !y_f16) return AWQ_ERR_NULL;
  if (!aligned16(x_f16) || !aligned16(qweight) || !aligned16(qzeros) || !aligned16(scales_f16) || !aligned16(y_f16))
    return AWQ_ERR_ALIGN;
  st = plan_moe(T, topk, E, K, N, group_size, device_cus(), mp);
  if (st != AWQ_OK) return st;
  const int64_t S = T * topk;
  const int g = eff_group(K, group_size);
  const int64_t G = K / g;
  const auto* x = static_cast<const uint16_t*>(x_f16);
  const auto* sc = static_cast<const uint16_t*>(scales_f16);
  auto* y = static_cast<uint16_t*>(y_f16);
  Launches held;
  if (mp.skinny) {
    Plan p;
    p.accum_bytes = mp.accum_bytes;
    p.partial_bytes = mp.partial_bytes;
    uint64_t* accum = nullptr;
    float* partial = nullptr;
    if (mp.sk.splits > 1) {
      st = get_workspace(p, stream, &accum, &partial, held);
      if (st != AWQ_OK) return st;
      if (mp.sk.atomic) partial = reinterpret_cast<float*>(accum + skinny_accum_entries(mp.sk));
    }
    const SkinnyExperts ex{expert_ids, (int)topk, (int)mp.tiles_e, (int)mp.chunks, (int)E, K * (N / 8), G * (N / 8),
                           G * N};
    hipError_t e = launch_skinny_experts(x, qweight, qzeros, sc, (int)T, (int)K, (int)N, g, mp.sk, ex, accum, partial,
                                         y, stream);
    return e == hipSuccess ? AWQ_OK : AWQ_ERR_HIP;
  }
  // Scratch: tile table (16-byte entries), offsets, sorted slots; written by the
  // alignment kernel before the product reads it, on the same stream.
  void* scratch = nullptr;
  st = get_scratch(mp.scratch_bytes, stream, &scratch, held);
  if (st != AWQ_OK) return st;
  int32_t* table = static_cast<int32_t*>(scratch);
  int32_t* offsets = table + 4 * mp.tiles;
  int32_t* sorted = offsets + E + 1;
  hipError_t e = launch_moe_align(expert_ids, (int)S, (int)E, mp.block_rows, (int)mp.tiles, offsets, sorted, table,
                                  stream);
  if (e != hipSuccess) return AWQ_ERR_HIP;
  MoeTiles moe{sorted, table, (int)topk, (int)mp.tiles, K * (N / 8), G * (N / 8), G * N};
  e = launch_tile_grouped(x, qweight, qzeros, sc, (int)K, (int)N, g, mp.variant, moe, y, stream);
  return e == hipSuccess ? AWQ_OK : AWQ_ERR_HIP;
}

int awq_moe_route(const void* logits, int logits_type, int64_t T, int64_t E, int64_t row_stride, const float* bias,
                  int score, int64_t groups, int64_t topk_groups, int group_top, int64_t topk, int renormalize,
                  float scale, float* weights, int32_t* expert_ids, struct ihipStream_t* stream) {
  const int st = plan_route(T, E, row_stride, groups, topk_groups, group_top, topk);
  if (st != AWQ_OK) return st;
  if (logits_type != AWQ_F16 && logits_type != AWQ_BF16 && logits_type != AWQ_F32) return AWQ_ERR_UNSUPPORTED;
  if (score != AWQ_SOFTMAX && score != AWQ_SIGMOID) return AWQ_ERR_UNSUPPORTED;
  if (T == 0) return AWQ_OK;
  if (!logits || !weights || !expert_ids) return AWQ_ERR_NULL;
  const uintptr_t unit = logits_type == AWQ_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(logits) % unit != 0 || reinterpret_cast<uintptr_t>(bias) % 4 != 0 ||
      reinterpret_cast<uintptr_t>(weights) % 4 != 0 || reinterpret_cast<uintptr_t>(expert_ids) % 4 != 0)
    return AWQ_ERR_ALIGN;
  RouteArgs a;
  a.logits = logits;
  a.bias = bias;
  a.weights = weights;
  a.ids = expert_ids;
  a.T = T;
  a.row_stride = row_stride;
  a.E = (int)E;
  a.type = logits_type;
  a.topk = (int)topk;
  a.groups = (int)groups;
  a.topk_groups = (int)topk_groups;
  a.group_top = group_top;
  a.softmax = score == AWQ_SOFTMAX;
  a.renormalize = renormalize != 0;
  a.scale = scale;
  return awq::launch_route(a, stream) == hipSuccess ? AWQ_OK : AWQ_ERR_HIP;
}

namespace {

// Whether two byte ranges share a byte.
bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a != nullptr && b != nullptr && a0 < b0 + (uintptr_t)b_bytes && b0 < a0 + (uintptr_t)a_bytes;
}

}  // namespace

int awq_gemm_fused_plan(int64_t M, int64_t K, int64_t N, int64_t group_size, int gated, int64_t* workspace_bytes,
                        int64_t* counter_bytes) {
  DensePlan p;
  const int st = plan_dense(M, K, N, group_size, query_cus(), gated != 0, p);
  if (st != AWQ_OK) return st;
  if (workspace_bytes) *workspace_bytes = p.sums_bytes;
  if (counter_bytes) *counter_bytes = p.counter_bytes;
  return AWQ_OK;
}

int awq_gemm_fused(const void* x, int act, const int32_t* qweight, const int32_t* qzeros, const void* scales_f16,
                   const void* bias, int activation, int gated, const void* residual, float scale, int64_t M,
                   int64_t K, int64_t N, int64_t group_size, void* y, void* workspace, int64_t workspace_bytes,
                   void* counters, int64_t counter_bytes, struct ihipStream_t* stream) {
  DensePlan d;
  const int st = plan_dense(M, K, N, group_size, query_cus(), gated != 0, d);
  if (st != AWQ_OK) return st;
  if (act != AWQ_F16 && act != AWQ_BF16) return AWQ_ERR_UNSUPPORTED;
  if (activation < AWQ_ACT_NONE || activation > AWQ_ACT_GELU_TANH) return AWQ_ERR_UNSUPPORTED;
  if (M == 0) return AWQ_OK;
  if (!x || !qweight || !qzeros || !scales_f16 || !y) return AWQ_ERR_NULL;
  if ((d.sums_bytes > 0 && !workspace) || (d.counter_bytes > 0 && !counters)) return AWQ_ERR_NULL;
  for (const void* p : {x, (const void*)qweight, (const void*)qzeros, scales_f16, bias, residual, (const void*)y,
                        (const void*)workspace})
    if (!aligned16(p)) return AWQ_ERR_ALIGN;
  if (reinterpret_cast<uintptr_t>(counters) % 4 != 0) return AWQ_ERR_ALIGN;
  if (workspace_bytes < d.sums_bytes || counter_bytes < d.counter_bytes) return AWQ_ERR_UNSUPPORTED;
  // Workgroups write y while others still read x.  The residual is read where y is written, by the
  // same thread: y may be the residual.
  const int64_t y_bytes = M * N * 2;
  if (overlap(y, y_bytes, x, M * K * 2) || (y != residual && overlap(y, y_bytes, residual, y_bytes)))
    return AWQ_ERR_UNSUPPORTED;
  DenseProduct p;
  p.x = static_cast<const uint16_t*>(x);
  p.qweight = reinterpret_cast<const uint32_t*>(qweight);
  p.qzeros = reinterpret_cast<const uint32_t*>(qzeros);
  p.scales = static_cast<const uint16_t*>(scales_f16);
  p.M = (int)M;
  p.K = (int)K;
  p.N = (int)N;
  p.g = eff_group(K, group_size);
  p.gated = gated != 0;
  p.bf16 = act == AWQ_BF16;
  p.sums = static_cast<float*>(workspace);
  p.counters = static_cast<uint32_t*>(counters);
  const Epilogue e{static_cast<const uint16_t*>(bias), static_cast<const uint16_t*>(residual), static_cast<uint16_t*>(y),
                   scale, activation};
  const hipError_t err = d.stream ? awq::launch_fused_stream(p, e, d, stream) : awq::launch_fused_tiles(p, e, d, stream);
  return err == hipSuccess ? AWQ_OK : AWQ_ERR_HIP;
}

int awq_add_norm(const void* x, int act, int64_t T, int64_t H, int64_t x_stride, const void* residual,
                 int residual_type, int64_t residual_stride, const void* gate, int64_t gates, float scale,
                 const void* post_weight, const void* post_bias, const void* weight, const void* bias, int kind,
                 int unit_offset, float eps, void* y, void* r, struct ihipStream_t* stream) {
  const int st = plan_norm(T, H, x_stride, residual ? residual_stride : H, gate ? gates : 0);
  if (st != AWQ_OK) return st;
  if (act != AWQ_F16 && act != AWQ_BF16) return AWQ_ERR_UNSUPPORTED;
  const bool r32 = residual_type == AWQ_F32;
  if ((residual || r) && !r32 && residual_type != act) return AWQ_ERR_UNSUPPORTED;
  if (kind != AWQ_RMS && kind != AWQ_LAYER) return AWQ_ERR_UNSUPPORTED;
  if (gate && gates == 0) return AWQ_ERR_SHAPE;
  if (T == 0) return AWQ_OK;
  if (!x || (!y && !r) || (y && !weight) || (post_bias && !post_weight) || (bias && !y)) return AWQ_ERR_NULL;
  const uintptr_t unit = r32 ? 4 : 2;
  for (const void* p : {x, gate, post_weight, post_bias, weight, bias, (const void*)y})
    if (reinterpret_cast<uintptr_t>(p) % 2 != 0) return AWQ_ERR_ALIGN;
  if (reinterpret_cast<uintptr_t>(residual) % unit != 0 || reinterpret_cast<uintptr_t>(r) % unit != 0) return AWQ_ERR_ALIGN;
  // A row is read whole before it is written, so r may take residual's place and y that of x, row
  // for row; nothing else that is read or written may share memory with them.
  const int64_t x_bytes = ((T - 1) * x_stride + H) * 2, y_bytes = T * H * 2, r_bytes = T * H * (int64_t)unit;
  const int64_t res_bytes = ((T - 1) * residual_stride + H) * (int64_t)unit;
  auto clash = [&](const void* out, int64_t bytes, const void* same, int64_t same_stride, int64_t same_unit,
                   int64_t out_unit) {
    auto meets = [&](const void* in, int64_t in_bytes, int64_t stride, int64_t in_unit) {
      const bool in_place = in == same && in == out && stride == same_stride && (T == 1 || stride == H) &&
                            in_unit == same_unit && in_unit == out_unit;
      return !in_place && overlap(out, bytes, in, in_bytes);
    };
    return meets(x, x_bytes, x_stride, 2) || meets(residual, res_bytes, residual_stride, (int64_t)unit) ||
           overlap(out, bytes, gate, gates * H * 2) || overlap(out, bytes, post_weight, H * 2) ||
           overlap(out, bytes, post_bias, H * 2) || overlap(out, bytes, weight, H * 2) || overlap(out, bytes, bias, H * 2);
  };
  if (clash(y, y_bytes, x, x_stride, 2, 2) || clash(r, r_bytes, residual, residual_stride, (int64_t)unit, (int64_t)unit) ||
      overlap(y, y_bytes, r, r_bytes))
    return AWQ_ERR_UNSUPPORTED;
  NormArgs a;
  a.x = static_cast<const uint16_t*>(x);
  a.gate = static_cast<const uint16_t*>(gate);
  a.post_weight = static_cast<const uint16_t*>(post_weight);
  a.post_bias = static_cast<const uint16_t*>(post_bias);
  a.weight = static_cast<const uint16_t*>(weight);
  a.bias = static_cast<const uint16_t*>(bias);
  a.residual = residual;
  a.y = static_cast<uint16_t*>(y);
  a.r = r;
  a.T = T;
  a.x_stride = x_stride;
  a.residual_stride = residual_stride;
  a.gate_rows = gate ? T / gates : 1;
  a.H = (int)H;
  a.scale = scale;
  a.eps = eps;
  a.bf16 = act == AWQ_BF16;
  a.r32 = r32;
  a.layer = kind == AWQ_LAYER;
  a.unit_offset = unit_offset != 0;
  return awq::launch_norm(a, stream) == hipSuccess ? AWQ_OK : AWQ_ERR_HIP;
}

int64_t awq_moe_workspace(int64_t T, int64_t topk, int64_t E, int64_t K, int64_t inner, int64_t N,
                          int64_t group_size) {
  if (K < 0 || N < 0 || (K == 0 && N == 0)) return AWQ_ERR_SHAPE;
  ExpertsPlan p;
  const int st = plan_experts(T, topk, E, K, inner, N, group_size, query_cus(), K > 0, N > 0, p);
  return st == AWQ_OK ? p.workspace_bytes() : st;
}

namespace {

// The packed weight of one half: [E, K, n] as the header lays it out.
struct Packed {
  const int32_t *qweight, *qzeros;
  const void* scales;
  int check() const {
    if (!qweight || !qzeros || !scales) return AWQ_ERR_NULL;
    return aligned16(qweight) && aligned16(qzeros) && aligned16(scales) ? AWQ_OK : AWQ_ERR_ALIGN;
  }
};

// The gated half (up), the second half (down), or both with h between them in the workspace.
int experts_common(const void* x, int act, const Packed* up, const Packed* down, const int32_t* ids,
                   const float* weights, int64_t T, int64_t topk, int64_t E, int64_t K, int64_t inner, int64_t N,
                   int64_t group_size, void* out, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  ExpertsPlan p;
  int st = plan_experts(T, topk, E, K, inner, N, group_size, query_cus(), up != nullptr, down != nullptr, p);
  if (st != AWQ_OK) return st;
  const bool nan_weights = down && (act & AWQ_NAN_WEIGHTS) != 0;
  if (nan_weights) act -= AWQ_NAN_WEIGHTS;
  if (act != AWQ_F16 && act != AWQ_BF16) return AWQ_ERR_UNSUPPORTED;
  if (T == 0) return AWQ_OK;
  if (!x || !ids || !out || !workspace || (down && !weights)) return AWQ_ERR_NULL;
  for (const Packed* w : {up, down})
    if (w && (st = w->check()) != AWQ_OK) return st;
  if (!aligned16(x) || !aligned16(out) || !aligned16(workspace)) return AWQ_ERR_ALIGN;
  if (reinterpret_cast<uintptr_t>(ids) % 4 != 0 || reinterpret_cast<uintptr_t>(weights) % 4 != 0) return AWQ_ERR_ALIGN;
  if (workspace_bytes < p.workspace_bytes()) return AWQ_ERR_UNSUPPORTED;

  const int64_t S = T * topk;
  // The gated product alone writes h while other workgroups still read x; in the others nothing
  // reads x or h any more when y is written.
  const uintptr_t x0 = reinterpret_cast<uintptr_t>(x), h0 = reinterpret_cast<uintptr_t>(out);
  if (!down && x0 < h0 + (uintptr_t)(S * inner * 2) && h0 < x0 + (uintptr_t)(T * K * 2)) return AWQ_ERR_UNSUPPORTED;
  char* ws = static_cast<char*>(workspace);
  uint16_t* h = reinterpret_cast<uint16_t*>(ws + p.sorted_bytes);
  float* sums = reinterpret_cast<float*>(ws + p.sorted_bytes + p.h_bytes);
  ExpertProduct q{};
  q.ids = ids;
  q.S = (int)S;
  q.E = (int)E;
  q.bf16 = act == AWQ_BF16;
  q.sums = sums;
  // Slots sorted by expert, in blocks of the product's rows; kept for the next product where
  // that takes the same blocks.
  int sorted_for = 0;
  auto product = [&](const Packed& w, const ExpertPlan& ep) {
    q.qweight = reinterpret_cast<const uint32_t*>(w.qweight);
    q.qzeros = reinterpret_cast<const uint32_t*>(w.qzeros);
    q.scales = static_cast<const uint16_t*>(w.scales);
    int32_t* table = reinterpret_cast<int32_t*>(ws);
    int32_t* offsets = table + 4 * ep.tiles;
    int32_t* sorted = offsets + E + 1;
    if (ep.ranked) return awq::launch_expert_stream(q, ep, nullptr, nullptr, stream);
    if (sorted_for != ep.block_rows) {
      const hipError_t e = awq::launch_moe_align(ids, (int)S, (int)E, ep.block_rows, (int)ep.tiles, offsets, sorted,
                                                 table, stream);
      if (e != hipSuccess) return e;
      sorted_for = ep.block_rows;
    }
    return ep.stream ? awq::launch_expert_stream(q, ep, sorted, table, stream)
                     : awq::launch_expert_tiles(q, ep, sorted, table, stream);
  };
  hipError_t e = hipSuccess;
  if (up) {
    q.x = static_cast<const uint16_t*>(x);
    q.row_div = (int)topk;
    q.K = (int)K;
    q.N = (int)inner;
    q.g = eff_group(K, group_size);
    q.gated = true;
    q.h = down ? h : static_cast<uint16_t*>(out);
    if (p.two_terms) q.h_rest = reinterpret_cast<uint16_t*>(reinterpret_cast<char*>(h) + p.h_bytes / 2);
    e = product(*up, p.up);
    if (e == hipSuccess && p.up.splits > 1)
      e = awq::launch_expert_gate(sums, ids, (int)S, (int)E, (int)inner, p.up.splits, q.bf16, q.h, q.h_rest,
                                  stream);
  }
  if (e == hipSuccess && down) {
    q.x = up ? h : static_cast<const uint16_t*>(x);
    q.x_rest = q.h_rest;
    q.row_div = 1;
    q.K = (int)inner;
    q.N = (int)N;
    q.g = eff_group(inner, group_size);
    q.gated = false;
    e = product(*down, p.down);
    if (e == hipSuccess)
      e = awq::launch_expert_combine(sums, ids, weights, (int)T, (int)topk, (int)E, (int)N, p.down.splits, q.bf16,
                                     nan_weights, static_cast<uint16_t*>(out), stream);
  }
  return e == hipSuccess ? AWQ_OK : AWQ_ERR_HIP;
}

}  // namespace

int64_t awq_moe_layer_workspace(int64_t T, int64_t topk, int64_t E, int64_t K, int64_t inner, int64_t N,
                                int64_t group_size) {
  LayerPlan p;
  const int st = plan_layer(T, topk, E, K, inner, N, group_size, query_cus(), p);
  return st == AWQ_OK ? p.workspace_bytes() : st;
}

int awq_moe_layer(const void* x, int act, const void* router, int router_type, int round_logits, const float* bias,
                  int score, int64_t groups, int64_t topk_groups, int group_top, int64_t topk, int renormalize,
                  float scale, const int32_t* up_qweight, const int32_t* up_qzeros, const void* up_scales_f16,
                  const int32_t* down_qweight, const int32_t* down_qzeros, const void* down_scales_f16,
                  const void* residual, int64_t T, int64_t E, int64_t K, int64_t inner, int64_t N, int64_t group_size,
                  void* y, void* workspace, int64_t workspace_bytes, void* counters, int64_t counter_bytes,
                  struct ihipStream_t* stream) {
  int st = plan_route(T, E, E, groups, topk_groups, group_top, topk);
  if (st != AWQ_OK) return st;
  LayerPlan p;
  st = plan_layer(T, topk, E, K, inner, N, group_size, query_cus(), p);
  if (st != AWQ_OK) return st;
  if (act != AWQ_F16 && act != AWQ_BF16) return AWQ_ERR_UNSUPPORTED;
  if (router_type != act && router_type != AWQ_F32) return AWQ_ERR_UNSUPPORTED;
  if (score != AWQ_SOFTMAX && score != AWQ_SIGMOID) return AWQ_ERR_UNSUPPORTED;
  if (T == 0) return AWQ_OK;
  if (!x || !router || !y || !workspace || !counters) return AWQ_ERR_NULL;
  const Packed up{up_qweight, up_qzeros, up_scales_f16}, down{down_qweight, down_qzeros, down_scales_f16};
  for (const Packed* w : {&up, &down})
    if ((st = w->check()) != AWQ_OK) return st;
  if (!aligned16(x) || !aligned16(router) || !aligned16(y) || !aligned16(residual) || !aligned16(workspace))
    return AWQ_ERR_ALIGN;
  if (reinterpret_cast<uintptr_t>(bias) % 4 != 0 || reinterpret_cast<uintptr_t>(counters) % 4 != 0) return AWQ_ERR_ALIGN;
  if (workspace_bytes < p.workspace_bytes() || counter_bytes < AWQ_MOE_LAYER_COUNTERS) return AWQ_ERR_UNSUPPORTED;
  // Nobody reads x any more when y is written; the residual is read where y is, by the same thread.
  if (y != residual && overlap(y, T * N * 2, residual, T * N * 2)) return AWQ_ERR_UNSUPPORTED;
  LayerArgs a;
  char* ws = static_cast<char*>(workspace);
  auto part = [&](int64_t bytes) {
    char* at = ws;
    ws += bytes;
    return static_cast<void*>(at);
  };
  a.counts = static_cast<uint32_t*>(part(p.counts_bytes));
  a.logits = static_cast<float*>(part(p.logits_bytes));
  a.ids = static_cast<int32_t*>(part(p.ids_bytes));
  a.weights = static_cast<float*>(part(p.ids_bytes));
  a.h = static_cast<uint16_t*>(part(p.h_bytes));
  a.up_sums = static_cast<float*>(part(p.up_bytes));
  a.down_sums = static_cast<float*>(part(p.down_bytes));
  a.x = static_cast<const uint16_t*>(x);
  a.residual = static_cast<const uint16_t*>(residual);
  a.router = router;
  a.y = static_cast<uint16_t*>(y);
  a.up_qweight = reinterpret_cast<const uint32_t*>(up_qweight);
  a.up_qzeros = reinterpret_cast<const uint32_t*>(up_qzeros);
  a.up_scales = static_cast<const uint16_t*>(up_scales_f16);
  a.down_qweight = reinterpret_cast<const uint32_t*>(down_qweight);
  a.down_qzeros = reinterpret_cast<const uint32_t*>(down_qzeros);
  a.down_scales = static_cast<const uint16_t*>(down_scales_f16);
  a.arrivals = static_cast<uint32_t*>(counters);
  a.n_counts = p.n_counts;
  a.T = (int)T;
  a.topk = (int)topk;
  a.E = (int)E;
  a.K = (int)K;
  a.inner = (int)inner;
  a.N = (int)N;
  a.g_up = eff_group(K, group_size);
  a.g_down = eff_group(inner, group_size);
  a.router_waves = p.router_waves;
  a.up_tiles = p.up_tiles;
  a.up_splits = p.up_splits;
  a.up_steps = p.up_steps;
  a.down_tiles = p.down_tiles;
  a.down_splits = p.down_splits;
  a.down_steps = p.down_steps;
  a.bf16 = act == AWQ_BF16;
  a.router32 = router_type == AWQ_F32;
  a.round_logits = round_logits != 0;
  RouteArgs r{};
  r.bias = bias;
  r.T = T;
  r.E = (int)E;
  r.topk = (int)topk;
  r.groups = (int)groups;
  r.topk_groups = (int)topk_groups;
  r.group_top = group_top;
  r.softmax = score == AWQ_SOFTMAX;
  r.renormalize = renormalize != 0;
  r.scale = scale;
  return awq::launch_layer(a, r, p, stream) == hipSuccess ? AWQ_OK : AWQ_ERR_HIP;
}

int awq_moe_gate_up(const void* x, int act, const int32_t* qweight, const int32_t* qzeros, const void* scales_f16,
                    const int32_t* expert_ids, int64_t T, int64_t topk, int64_t E, int64_t K, int64_t inner,
                    int64_t group_size, void* h, void* workspace, int64_t workspace_bytes,
                    struct ihipStream_t* stream) {
  const Packed up{qweight, qzeros, scales_f16};
  return experts_common(x, act, &up, nullptr, expert_ids, nullptr, T, topk, E, K, inner, 0, group_size, h, workspace,
                        workspace_bytes, stream);
}

int awq_moe_down(const void* h, int act, const int32_t* qweight, const int32_t* qzeros, const void* scales_f16,
                 const int32_t* expert_ids, const float* weights, int64_t T, int64_t topk, int64_t E, int64_t K,
                 int64_t N, int64_t group_size, void* y, void* workspace, int64_t workspace_bytes,
                 struct ihipStream_t* stream) {
  const Packed down{qweight, qzeros, scales_f16};
  return experts_common(h, act, nullptr, &down, expert_ids, weights, T, topk, E, 0, K, N, group_size, y, workspace,
                        workspace_bytes, stream);
}

int awq_moe_mlp(const void* x, int act, const int32_t* up_qweight, const int32_t* up_qzeros,
                const void* up_scales_f16, const int32_t* down_qweight, const int32_t* down_qzeros,
                const void* down_scales_f16, const int32_t* expert_ids, const float* weights, int64_t T, int64_t topk,
                int64_t E, int64_t K, int64_t inner, int64_t N, int64_t group_size, void* y, void* workspace,
                int64_t workspace_bytes, struct ihipStream_t* stream) {
  const Packed up{up_qweight, up_qzeros, up_scales_f16}, down{down_qweight, down_qzeros, down_scales_f16};
  return experts_common(x, act, &up, &down, expert_ids, weights, T, topk, E, K, inner, N, group_size, y, workspace,
                        workspace_bytes, stream);
}

int awq_gemm(const void* x_f16, const int32_t* qweight, const int32_t* qzeros, const void* scales_f16,
             const void* bias_f16, int64_t M, int64_t K, int64_t N, int64_t group_size, void* y_f16,
             struct ihipStream_t* stream) {
  return gemm_common(x_f16, qweight, qzeros, scales_f16, bias_f16, M, K, N, group_size, y_f16, false, stream);
}

int awq_gemm_noalloc(const void* x_f16, const int32_t* qweight, const int32_t* qzeros, const void* scales_f16,
                     const void* bias_f16, int64_t M, int64_t K, int64_t N, int64_t group_size, void* y_f16,
                     struct ihipStream_t* stream) {
  return gemm_common(x_f16, qweight, qzeros, scales_f16, bias_f16, M, K, N, group_size, y_f16, false, stream, true);
}

int awq_gemm_bf16(const void* x_bf16, const int32_t* qweight, const int32_t* qzeros, const void* scales_f16,
                  const void* bias_bf16, int64_t M, int64_t K, int64_t N, int64_t group_size, void* y_bf16,
                  struct ihipStream_t* stream) {
  return gemm_common(x_bf16, qweight, qzeros, scales_f16, bias_bf16, M, K, N, group_size, y_bf16, true, stream);
}

}  // extern "C"
