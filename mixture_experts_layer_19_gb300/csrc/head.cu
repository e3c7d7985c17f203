// head.cu -- the C ABI of the loss head (include/moe.h): argument checks,
// workspace layout, tensor maps and the kernel sequence of cross entropy and
// distillation, forward and backward.
//
// Forward   [teacher entries] -> [row list, compact X] -> logits + softmax
//           statistics GEMM -> losses
// Backward  [teacher entries] -> row list, compact X -> per vocabulary piece:
//           D GEMM, dX GEMM (fp32 sums), dW GEMM -> dX rounding
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <mutex>
#include <string>

#include "head.h"
#include "kernels.h"
#include "moe.h"

namespace {

using namespace moe;

constexpr int kMaxDevices = 64;

// Default piece of D: this much, but no fewer columns than keep its products wide (16 KB per token, the
// larger of the two from 16384 tokens on).
constexpr int64_t kPieceBytes = int64_t(256) << 20, kPieceColumns = 8192;

moe_status_t bad(const char* where, const char* what, moe_status_t s = MOE_ERR_INVALID_ARG) {
  set_error_detail((std::string(where) + ": " + what).c_str());
  return s;
}
moe_status_t cuda_bad(const char* where, const char* what, cudaError_t e) {
  set_error_detail((std::string(where) + ": " + what + ": " + cudaGetErrorString(e)).c_str());
  return MOE_ERR_CUDA;
}

struct DeviceFacts {
  bool ready = false;
  int sms = 0, pairs = 0;
};
DeviceFacts g_facts[kMaxDevices];
std::mutex g_facts_mu;

// Facts of the current device, and its context bound to the calling thread
// (the tensor-map encoder is a driver call).
moe_status_t device_facts(const char* where, DeviceFacts* out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaSetDevice(dev);
  if (e != cudaSuccess) return cuda_bad(where, "no usable current device", e);
  if (dev < 0 || dev >= kMaxDevices) return bad(where, "device ordinal out of range", MOE_ERR_UNSUPPORTED);
  std::lock_guard<std::mutex> lock(g_facts_mu);
  DeviceFacts& f = g_facts[dev];
  if (!f.ready) {
    int major = 0, minor = 0;
    cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    if (major != 10 || minor != 3)
      return bad(where, "this library is built for sm_103a (GB300) only", MOE_ERR_UNSUPPORTED);
    if ((e = cudaDeviceGetAttribute(&f.sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess ||
        (e = head_gemm_prepare()) != cudaSuccess || (e = head_gemm_max_pairs(&f.pairs)) != cudaSuccess)
      return cuda_bad(where, "kernel attributes", e);
    f.pairs = std::min(f.pairs, f.sms / 2);
    if (f.pairs < 1) return bad(where, "no room for a CTA pair", MOE_ERR_CUDA);
    f.ready = true;
  }
  *out = f;
  return MOE_OK;
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

// bf16, row-major [rows, cols] with row stride ld: boxes of 64 columns (128
// bytes, 128-byte swizzle) and box_r rows; reads past the edges give zeros.
bool map_k(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int64_t ld, int box_r) {
  auto enc = encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  cuuint32_t box[2] = {64, (cuuint32_t)box_r};
  cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

struct Layout {
  int64_t Tp, piece, ldl;   // padded rows, columns of one piece, leading dimension of the D piece
  int K, nsplit;
  bool pair_z, pair_x, pair_w;   // CTA pairs for the logits, dX and dW products
  int arows, bn;            // rows of A per CTA (without pairs), columns of a tile in the logits products
  bool sums;                // dX needs the fp32 sums (several pieces or splits)
  int64_t blocks;           // blocks of 128 vocabulary columns
  size_t counts, scale, rec, inv, ids, probs, first, cnt, plogp, xc, part, zt, dl, acc, total;
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Time of one product in units of one K slice of a pair's 256 x 256 tile
// (0.27 us at 1.9 GHz): whole waves of tiles, each as long as its nkb slices or
// its epilogue (epi slices, overlapped with the next tile's products), and the last
// epilogue, which nothing overlaps.  A single CTA's slice moves 48 KB into its SM
// where a pair moves 32 per SM, and takes 1.1 times as long (4096 x 7168 x
// 65536 forward: 2508 us against 2393), 1.3 where rows do not end on 32 bytes
// (520 x 1000 x 50001 backward: 197 against 175).  A pair's epilogues wait for
// each other (1000 x 256 x 30000 forward: 34.5 us against 28.2 with single CTAs).
constexpr double kEpiLogits = 12, kEpiGrad = 6, kEpiPair = 1.25, kStart = 16;
struct Cost {
  int sms, pairs;
  double single;     // a single CTA's slice
  double of(int64_t m, int64_t ncols, double nkb, double epi, int splits, bool pair) const {
    const int64_t tiles = ceil_div(m, pair ? 256 : 128) * ceil_div(ncols, kHeadBN) * splits;
    const double tile = pair ? std::max(nkb, kEpiPair * epi) : std::max(single * nkb, epi);
    return (double)ceil_div(tiles, pair ? pairs : sms) * tile + kStart;
  }
  bool pair_pays(int64_t m, int64_t ncols, double nkb, double epi) const {
    return of(m, ncols, nkb, epi, 1, true) <= of(m, ncols, nkb, epi, 1, false);
  }
};

Layout layout(const moe_head_config_t& c, bool distill, bool backward, int sms, int pairs) {
  Layout L{};
  const Cost cost{sms, pairs, c.d % 16 == 0 ? 1.1 : 1.3};
  L.K = distill ? c.K : 1;
  L.Tp = std::max<int64_t>(up(c.T, kHeadRowPad), kHeadRowPad);
  L.nsplit = 1;
  if (backward) {
    int64_t p = c.piece > 0 ? up(c.piece, 256) : std::max(kPieceBytes / (2 * L.Tp), kPieceColumns);
    const int64_t n = std::max<int64_t>(1, ceil_div(up(c.V, 256), p));
    L.piece = up(ceil_div(c.V, n), 256);        // pieces of equal size
    L.ldl = L.piece;
    const int64_t cols = std::min<int64_t>(L.piece, c.V);
    // dX has few tiles when T is small: its K, the piece, is split until they
    // fill the SMs.  Splitting costs another launch (12 slices), and each split
    // the traffic of its fp32 sums, written and read at 5 TB/s, and a load in
    // that launch's chain.
    const double per_split = 0.25 + 6e-6 * (double)c.T * c.d;
    const int64_t nkb = ceil_div(cols, 64);
    double best = 0;
    for (int pair = 0; pair < (c.T > 128 ? 2 : 1); ++pair)
      for (int s = 1; s <= 48 && s <= nkb; ++s) {
        const double t = cost.of(c.T, c.d, (double)nkb / s, kEpiGrad, s, pair != 0) +
                         (s > 1 ? 12.0 + per_split * (s - 1) : 0.0);
        if ((s == 1 && !pair) || t < best) {
          best = t;
          L.nsplit = s;
          L.pair_x = pair != 0;
        }
      }
    // dW of few tokens is bound by its writes, which single CTAs, each on its own
    // tile, keep going better than pairs (64 x 7168 x 131072: 383 us against 503,
    // 300 x 2048 x 32768 98 against 105; 520 x 1000 x 50001 143 against 123)
    L.pair_w = c.T >= 384 && cost.pair_pays(cols, c.d, (double)ceil_div(c.T, 64), kEpiGrad);
    L.sums = L.nsplit > 1 || L.piece < c.V;
  }
  const int64_t zcols = backward ? std::min<int64_t>(L.piece, c.V) : c.V;
  L.pair_z = cost.pair_pays(c.T, zcols, (double)ceil_div(c.d, 64), kEpiLogits);
  // One row tile waits for W: no pair (its second half would have no rows).  Up
  // to 64 tokens fetch no more rows of X than they have, and where the vocabulary
  // has fewer tiles of 256 columns than there are SMs, narrower ones let more
  // SMs fetch (64 x 4096 x 8192 backward: 67.7 us against 60.2; 224 columns for 32768
  // entries, 147 tiles instead of 128, gained nothing).
  if (c.T <= 128) L.pair_z = false;
  L.arows = c.T > 64 ? 128 : c.T > 16 ? 64 : 16;
  L.bn = L.arows < 128 ? (int)std::min<int64_t>(kHeadBN, up(ceil_div(zcols, sms), 64)) : kHeadBN;
  size_t o = 0;
  auto take = [&o](size_t bytes) {
    const size_t at = o;
    o += (bytes + 255) & ~size_t(255);
    return at;
  };
  L.counts = take(16);
  L.scale = take(4);
  L.rec = take(L.Tp * 16);
  L.inv = take(c.T * 4);
  L.blocks = 2 * ceil_div(c.V, kHeadBN);
  L.ids = distill ? take((size_t)c.T * L.K * 4) : 0;
  L.first = distill ? take((size_t)c.T * L.blocks * 2) : 0;
  L.probs = distill ? take((size_t)c.T * L.K * 4) : 0;
  L.cnt = distill ? take(c.T * 4) : 0;
  L.plogp = distill ? take(c.T * 4) : 0;
  L.xc = take((size_t)L.Tp * c.d * 2);
  if (!backward) {
    L.part = take((size_t)ceil_div(c.V, L.bn) * 2 * L.Tp * 8);
    L.zt = take((size_t)c.T * L.K * 4);
  } else {
    L.dl = take((size_t)L.Tp * L.ldl * 2);
    L.acc = L.sums ? take((size_t)L.nsplit * L.Tp * c.d * 4) : 0;
  }
  L.total = o;
  return L;
}

HeadRows rows_of(const Layout& L, void* ws, bool distill) {
  char* b = static_cast<char*>(ws);
  HeadRows r{};
  r.n_active = reinterpret_cast<int32_t*>(b + L.counts);
  r.scale = reinterpret_cast<float*>(b + L.scale);
  r.rec = reinterpret_cast<int4*>(b + L.rec);
  r.inv = reinterpret_cast<int32_t*>(b + L.inv);
  r.blocks = L.blocks;
  if (distill) {
    r.ids = reinterpret_cast<int32_t*>(b + L.ids);
    r.first = reinterpret_cast<uint16_t*>(b + L.first);
    r.probs = reinterpret_cast<float*>(b + L.probs);
    r.cnt = reinterpret_cast<int32_t*>(b + L.cnt);
    r.plogp = reinterpret_cast<float*>(b + L.plogp);
  }
  r.Xc = b + L.xc;
  r.part = reinterpret_cast<float2*>(b + L.part);
  r.zt = reinterpret_cast<float*>(b + L.zt);
  r.dl = b + L.dl;
  r.acc = reinterpret_cast<float*>(b + L.acc);
  return r;
}

moe_status_t check_config(const char* where, const moe_head_config_t* c, bool distill) {
  if (!c) return bad(where, "null config");
  if (c->T < 0 || c->T > (1 << 20)) return bad(where, "T must be in [0, 2^20]");
  if (c->V < 1 || c->V > (1 << 24)) return bad(where, "V must be in [1, 2^24]");
  if (c->d < 8 || c->d > (1 << 16) || c->d % 8 != 0)
    return bad(where, "d must be a multiple of 8 in [8, 2^16]", MOE_ERR_UNSUPPORTED);
  if (distill && (c->K < 1 || c->K > kHeadMaxEntries)) return bad(where, "K must be in [1, 1024]");
  if (distill && !(c->temperature > 0.0f && std::isfinite(c->temperature)))
    return bad(where, "temperature must be positive and finite");
  if (c->piece < 0 || c->piece > (1 << 24)) return bad(where, "piece must be in [0, 2^24]");
  if (c->wait_timeout_ns < 0) return bad(where, "wait_timeout_ns must not be negative");
  return MOE_OK;
}

bool ok_ptr(const void* p, unsigned align) { return p && (reinterpret_cast<uintptr_t>(p) & (align - 1)) == 0; }

struct HeadCall {
  const char* where;
  const moe_head_config_t* cfg;
  const void *X, *W, *labels, *teacher, *ids;   // labels, or teacher and ids
  const float* dloss;                           // backward
  const float* lse_in;
  float *loss, *lse_out;
  void *dX, *dW;
  void* ws;
  size_t ws_bytes;
  int32_t* status;
  cudaStream_t st;
};

moe_status_t run_head(const HeadCall& h, bool distill, bool backward) {
  const char* w = h.where;
  moe_status_t s = check_config(w, h.cfg, distill);
  if (s != MOE_OK) return s;
  const moe_head_config_t& c = *h.cfg;
  const unsigned id_align = c.ids_int64 ? 8 : 4;
  if (backward && h.dW && !ok_ptr(h.dW, 16)) return bad(w, "misaligned dW");
  DeviceFacts f;
  if (c.T == 0) {
    if (backward && h.dW) {
      if ((s = device_facts(w, &f)) != MOE_OK) return s;
      const cudaError_t e = cudaMemsetAsync(h.dW, 0, (size_t)c.V * c.d * 2, h.st);
      if (e != cudaSuccess) return cuda_bad(w, "memset of dW", e);
    }
    return MOE_OK;
  }
  if (!ok_ptr(h.X, 16) || !ok_ptr(h.W, 16)) return bad(w, "null or misaligned X or W");
  if (distill ? (!ok_ptr(h.teacher, c.teacher_bf16 ? 2 : 4) || !ok_ptr(h.ids, id_align)) : !ok_ptr(h.labels, id_align))
    return bad(w, "null or misaligned targets");
  if (backward ? (!ok_ptr(h.dloss, 4) || !ok_ptr(h.lse_in, 4)) : (!ok_ptr(h.loss, 4) || !ok_ptr(h.lse_out, 4)))
    return bad(w, "null or misaligned row vector");
  if (backward && h.dX && !ok_ptr(h.dX, 16)) return bad(w, "misaligned dX");
  if (backward && !h.dX && !h.dW) return MOE_OK;
  if (!ok_ptr(h.ws, 256)) return bad(w, "null or misaligned workspace (256 bytes)");
  if (h.status && !ok_ptr(h.status, 4)) return bad(w, "misaligned status");
  if ((s = device_facts(w, &f)) != MOE_OK) return s;
  const Layout L = layout(c, distill, backward, f.sms, f.pairs);
  if (h.ws_bytes < L.total) return bad(w, "workspace smaller than moe_head_workspace_bytes");
  const HeadRows r = rows_of(L, h.ws, distill);
  const int T = (int)c.T;
  const float temp = distill ? c.temperature : 1.0f;

  HeadArgs a{};
  a.n_active = r.n_active;
  a.rec = r.rec;
  a.ids = r.ids;
  a.probs = r.probs;
  a.first = r.first;
  a.blocks = L.blocks;
  a.scale = r.scale;
  a.part = r.part;
  a.zt = r.zt;
  a.status = h.status;
  a.timeout_ns = c.wait_timeout_ns > 0 ? (uint64_t)c.wait_timeout_ns : 2000000000ull;
  a.Tp = L.Tp;
  a.T = T;
  a.d = c.d;
  a.K = L.K;
  a.nsplit = 1;
  a.bn = L.bn;
  a.inv_temp = 1.0f / temp;
  a.out_scale = temp;
  a.stall = (c.debug_flags & MOE_DEBUG_STALL_TEST) ? 1 : 0;

  bool ok = map_k(&a.mapA0, h.X, c.d, T, c.d, L.arows) && map_k(&a.mapA1, r.Xc, c.d, L.Tp, c.d, L.arows) &&
            map_k(&a.mapB0, h.W, c.d, c.V, c.d, L.pair_z ? 128 : L.bn);
  HeadArgs ax{}, aw{};
  if (backward) {
    a.dl = static_cast<__nv_bfloat16*>(r.dl);
    a.ldl = L.ldl;
    ax = a;
    ax.nsplit = L.nsplit;
    ax.acc = r.acc;
    ok = ok && map_k(&ax.mapA0, r.dl, L.ldl, L.Tp, L.ldl, L.pair_x ? 128 : L.arows) &&
         map_k(&ax.mapB0, h.W, c.d, c.V, c.d, 64);
    aw = a;
    aw.dW = static_cast<__nv_bfloat16*>(h.dW);
    aw.beside = h.dX != nullptr;
    ok = ok && map_k(&aw.mapA0, r.dl, L.ldl, L.Tp, L.ldl, 64) && map_k(&aw.mapB0, h.X, c.d, T, c.d, 64) &&
         map_k(&aw.mapB1, r.Xc, c.d, L.Tp, c.d, 64);
  }
  if (!ok) return bad(w, "tensor map encoding failed", MOE_ERR_CUDA);

  (void)cudaGetLastError();   // an error read below belongs to these launches
  cudaError_t e = cudaSuccess;
  if (distill)
    e = launch_head_entries(h.teacher, c.teacher_bf16 != 0, h.ids, c.ids_int64 != 0, T, L.K, c.V, a.inv_temp, r, h.st);
  // One row tile forward takes as long with every token's row as without some
  // of them, and rows do not mix: no list of the rows that count is made.
  const bool listed = backward || T > 128;
  if (e == cudaSuccess && listed)
    e = launch_head_prep(h.labels, c.ids_int64 != 0, h.dloss, h.lse_in, h.X, T, c.d, c.V, r,
                         backward ? h.dX : nullptr, f.sms, h.st);
  if (e != cudaSuccess) return cuda_bad(w, "row kernels", e);

  auto go = [&](int kind, bool pair, const HeadArgs& args, int64_t m, int64_t ncols, int splits) {
    const int64_t tiles = ceil_div(m, pair ? 256 : 128) * ceil_div(ncols, kind <= kHeadDl ? L.bn : kHeadBN) * splits;
    const int64_t workers = std::min<int64_t>(tiles, pair ? f.pairs : f.sms);
    return head_gemm_launch(kind, pair, L.arows, args, (int)workers * (pair ? 2 : 1), h.st);
  };
  if (!backward) {
    a.v0 = 0;
    a.vlen = c.V;
    HeadRows rl = r;
    if (!listed) {
      a.n_active = nullptr;
      a.labels = h.labels;
      a.cnt = r.cnt;
      a.ids64 = c.ids_int64 != 0;
      a.V = c.V;
      rl.inv = nullptr;
    }
    e = go(kHeadLse, L.pair_z, a, T, c.V, 1);
    if (e == cudaSuccess)
      e = launch_head_loss(h.labels, c.ids_int64 != 0, T, c.V, L.K, (int)(2 * ceil_div(c.V, L.bn)), L.Tp, temp, distill,
                           rl, h.loss, h.lse_out, h.st);
    return e == cudaSuccess ? MOE_OK : cuda_bad(w, "launch", e);
  }
  for (int64_t v0 = 0; v0 < c.V && e == cudaSuccess; v0 += L.piece) {
    const int64_t vlen = std::min<int64_t>(L.piece, c.V - v0);
    a.v0 = ax.v0 = aw.v0 = v0;
    a.vlen = ax.vlen = aw.vlen = vlen;
    ax.add = v0 > 0;
    ax.dX = L.nsplit == 1 && v0 + vlen == c.V ? static_cast<__nv_bfloat16*>(h.dX) : nullptr;
    e = go(kHeadDl, L.pair_z, a, T, vlen, 1);
    // a short last piece may have fewer K slices than splits: the empty ones add zeros
    if (e == cudaSuccess && h.dX) e = go(kHeadDX, L.pair_x, ax, T, c.d, L.nsplit);
    if (e == cudaSuccess && h.dW) e = go(kHeadDW, L.pair_w, aw, vlen, c.d, 1);
  }
  if (e == cudaSuccess && h.dX && L.nsplit > 1)
    e = launch_head_dx(T, c.d, L.nsplit, L.Tp, temp, r, h.dX, f.sms, h.st);
  return e == cudaSuccess ? MOE_OK : cuda_bad(w, "launch", e);
}

moe_status_t guarded(const HeadCall& h, bool distill, bool backward) {
  try {
    return run_head(h, distill, backward);
  } catch (...) {
    return MOE_ERR_INTERNAL;
  }
}

}  // namespace

extern "C" {

moe_status_t moe_head_workspace_bytes(const moe_head_config_t* cfg, int32_t distill, int32_t backward, size_t* bytes) {
  const char* w = "moe_head_workspace_bytes";
  try {
    if (!bytes) return bad(w, "null argument");
    moe_status_t s = check_config(w, cfg, distill != 0);
    if (s != MOE_OK) return s;
    *bytes = 0;
    if (cfg->T == 0) return MOE_OK;
    DeviceFacts f;
    if ((s = device_facts(w, &f)) != MOE_OK) return s;
    *bytes = layout(*cfg, distill != 0, backward != 0, f.sms, f.pairs).total;
    return MOE_OK;
  } catch (...) {
    return MOE_ERR_INTERNAL;
  }
}

moe_status_t moe_head_info(const moe_head_config_t* cfg, int32_t distill, int32_t backward, int32_t* plan) {
  const char* w = "moe_head_info";
  try {
    if (!plan) return bad(w, "null argument");
    moe_status_t s = check_config(w, cfg, distill != 0);
    if (s != MOE_OK) return s;
    std::fill(plan, plan + 6, 0);
    if (cfg->T == 0) return MOE_OK;
    DeviceFacts f;
    if ((s = device_facts(w, &f)) != MOE_OK) return s;
    const Layout L = layout(*cfg, distill != 0, backward != 0, f.sms, f.pairs);
    plan[0] = L.pair_z ? 2 : 1;
    plan[3] = L.bn;
    if (backward) {
      plan[1] = L.pair_x ? 2 : 1;
      plan[2] = L.pair_w ? 2 : 1;
      plan[4] = L.nsplit;
      plan[5] = (int32_t)ceil_div(cfg->V, L.piece);
    }
    return MOE_OK;
  } catch (...) {
    return MOE_ERR_INTERNAL;
  }
}

moe_status_t moe_cross_entropy_forward(const moe_head_config_t* cfg, const void* X, const void* W, const void* labels,
                                       float* loss, float* lse, void* workspace, size_t workspace_bytes,
                                       int32_t* status, moe_stream_t stream) {
  return guarded({"moe_cross_entropy_forward", cfg, X, W, labels, nullptr, nullptr, nullptr, nullptr, loss, lse,
                  nullptr, nullptr, workspace, workspace_bytes, status, reinterpret_cast<cudaStream_t>(stream)},
                 false, false);
}

moe_status_t moe_cross_entropy_backward(const moe_head_config_t* cfg, const float* dloss, const void* X, const void* W,
                                        const void* labels, const float* lse, void* dX, void* dW, void* workspace,
                                        size_t workspace_bytes, int32_t* status, moe_stream_t stream) {
  return guarded({"moe_cross_entropy_backward", cfg, X, W, labels, nullptr, nullptr, dloss, lse, nullptr, nullptr, dX,
                  dW, workspace, workspace_bytes, status, reinterpret_cast<cudaStream_t>(stream)},
                 false, true);
}

moe_status_t moe_distill_forward(const moe_head_config_t* cfg, const void* X, const void* W, const void* teacher,
                                 const void* ids, float* loss, float* lse, void* workspace, size_t workspace_bytes,
                                 int32_t* status, moe_stream_t stream) {
  return guarded({"moe_distill_forward", cfg, X, W, nullptr, teacher, ids, nullptr, nullptr, loss, lse, nullptr,
                  nullptr, workspace, workspace_bytes, status, reinterpret_cast<cudaStream_t>(stream)},
                 true, false);
}

moe_status_t moe_distill_backward(const moe_head_config_t* cfg, const float* dloss, const void* X, const void* W,
                                  const void* teacher, const void* ids, const float* lse, void* dX, void* dW,
                                  void* workspace, size_t workspace_bytes, int32_t* status, moe_stream_t stream) {
  return guarded({"moe_distill_backward", cfg, X, W, nullptr, teacher, ids, dloss, lse, nullptr, nullptr, dX, dW,
                  workspace, workspace_bytes, status, reinterpret_cast<cudaStream_t>(stream)},
                 true, true);
}

}  // extern "C"
