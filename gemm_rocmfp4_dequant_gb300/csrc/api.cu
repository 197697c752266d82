// C ABI of the ROCmFP4 library (declared in include/rocmfp4.h): host-side
// argument checks, per-device state, and kernel dispatch.
#include <atomic>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <string>

#include "../../include/rocmfp4.h"
#include "kernels.h"

namespace {

using namespace rocmfp4;

struct DeviceState {
  bool ready = false;
  int sms = 0;
  int occ[2][2][4] = {};             // stream kernel CTAs per SM [variant][act][log2 mb]
  int64_t wmax = 0;                  // workspace capacity in warps
  float* ws = nullptr;               // 2 * wmax records of kStreamTileRows * 8 floats
  uint32_t* cnt = nullptr;           // wmax split counters
  uint32_t* err = nullptr;           // kernel error bits
  float* tcws = nullptr;             // tensor-core kernel: split-tile partials
  uint32_t* tccnt = nullptr;         // tensor-core kernel: split-tile counters
  float* attn_ws = nullptr;          // decode attention: split partials
  unsigned long long* vfirst = nullptr;
  float* lp_ws = nullptr;            // log probabilities: records of split rows
  uint32_t* lp_cnt = nullptr;        // log probabilities: arrivals per split row
  bool norm_ready = false;           // RMS norm: kernels prepared
  uint32_t* moe_bars = nullptr;      // mixture of experts: barrier counters
  float* paged_ws = nullptr;         // paged attention: parts of split row tiles, from its first call on
  uint32_t* paged_cnt = nullptr;     // paged attention: arrivals per split row tile
  float* moe_ws = nullptr;           // mixture of experts: router logits and hidden values, from its first call on
};

constexpr int kMaxDevices = 64;
std::mutex g_mu;
DeviceState g_dev[kMaxDevices];
std::atomic<uint64_t> g_launches{0};
thread_local std::string t_last_error;

rocmfp4_status fail(rocmfp4_status st, const std::string& msg) {
  t_last_error = msg;
  return st;
}

rocmfp4_status cuda_fail(cudaError_t e, const char* what) {
  return fail(ROCMFP4_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool valid_variant(int v) { return v == ROCMFP4_DUAL || v == ROCMFP4_FAST; }
bool valid_dtype(int t) { return t == ROCMFP4_OUT_F32 || t == ROCMFP4_OUT_BF16 || t == ROCMFP4_OUT_F16; }
bool aligned_to(const void* p, int dtype) {
  return (reinterpret_cast<uintptr_t>(p) & (dtype == ROCMFP4_OUT_F32 ? 3u : 1u)) == 0;
}
bool valid_act(int a) { return a == ROCMFP4_ACT_F16 || a == ROCMFP4_ACT_BF16; }

int64_t block_bytes_of(int v) { return v == ROCMFP4_DUAL ? 18 : 17; }

// The mixture of experts' workspace (36 MiB) is made at its first call, not at
// every user's first call.  That call may stand in a graph's capture, which
// an allocation would end but for the relaxed mode (nothing here touches a stream).
rocmfp4_status moe_set_up(DeviceState& d) {
  cudaError_t e = moe_prepare();
  if (e != cudaSuccess) return cuda_fail(e, "mixture-of-experts kernel set-up");
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  if ((e = cudaThreadExchangeStreamCaptureMode(&mode)) != cudaSuccess) return cuda_fail(e, "cudaThreadExchangeStreamCaptureMode");
  float* ws = nullptr;
  e = cudaMalloc(&ws, sizeof(float) * kMoeWsFloats);
  cudaThreadExchangeStreamCaptureMode(&mode);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMalloc");
  d.moe_ws = ws;
  return ROCMFP4_OK;
}

// Paged attention's workspace (57 MiB on 152 SMs), made in the same manner.
rocmfp4_status paged_set_up(DeviceState& d) {
  cudaError_t e = paged_attn_prepare();
  if (e == cudaSuccess) e = paged_few_prepare();
  if (e != cudaSuccess) return cuda_fail(e, "paged attention kernel set-up");
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  if ((e = cudaThreadExchangeStreamCaptureMode(&mode)) != cudaSuccess) return cuda_fail(e, "cudaThreadExchangeStreamCaptureMode");
  float* ws = nullptr;
  e = cudaMalloc(&ws, sizeof(float) * paged_attn_ws_floats(d.sms));
  cudaThreadExchangeStreamCaptureMode(&mode);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMalloc");
  d.paged_ws = ws;
  return ROCMFP4_OK;
}

enum class Needs { kProducts, kNorm, kMoe, kPaged };

// Per-device set-up on first use: SM count, kernel attributes, occupancy and
// the workspace of the split-tile reduction; and what `needs` has beside that.
rocmfp4_status device_state(DeviceState** out, Needs needs = Needs::kProducts) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return fail(ROCMFP4_ERR_UNSUPPORTED, "device index out of range");
  std::lock_guard<std::mutex> lk(g_mu);
  DeviceState& d = g_dev[dev];
  if (!d.ready) {
    if ((e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
      return cuda_fail(e, "cudaDeviceGetAttribute");
    if ((e = stream_init_driver()) != cudaSuccess) return cuda_fail(e, "cuTensorMapEncodeTiled entry point");
    if ((e = tc_prepare()) != cudaSuccess) return cuda_fail(e, "tensor-core kernel set-up");
    if ((e = attn_prepare()) != cudaSuccess) return cuda_fail(e, "attention kernel set-up");
    int best = 1;
    for (int v = 0; v < 2; ++v)
      for (int a = 0; a < 2; ++a)
        for (int lm = 0; lm < 4; ++lm) {
          int& o = d.occ[v][a][lm];
          if ((e = stream_prepare(v, a, 1 << lm)) != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
          if ((e = stream_occupancy(v, a, 1 << lm, &o)) != cudaSuccess) return cuda_fail(e, "occupancy");
          if (o < 1) return fail(ROCMFP4_ERR_UNSUPPORTED, "streaming kernel does not fit on this device");
          best = o > best ? o : best;
        }
    d.wmax = (int64_t)d.sms * best * kStreamWarpsPerCta;
    if ((e = cudaMalloc(&d.ws, sizeof(float) * kStreamTileRows * 8 * 2 * d.wmax)) != cudaSuccess) return cuda_fail(e, "cudaMalloc");
    if ((e = cudaMalloc(&d.cnt, sizeof(uint32_t) * d.wmax)) != cudaSuccess) return cuda_fail(e, "cudaMalloc");
    if ((e = cudaMalloc(&d.err, sizeof(uint32_t))) != cudaSuccess) return cuda_fail(e, "cudaMalloc");
    if ((e = cudaMalloc(&d.vfirst, sizeof(unsigned long long))) != cudaSuccess) return cuda_fail(e, "cudaMalloc");
    if ((e = cudaMemset(d.cnt, 0, sizeof(uint32_t) * d.wmax)) != cudaSuccess) return cuda_fail(e, "cudaMemset");
    if ((e = cudaMalloc(&d.tcws, sizeof(float) * tc_ws_floats(d.sms))) != cudaSuccess) return cuda_fail(e, "cudaMalloc");
    if ((e = cudaMalloc(&d.tccnt, sizeof(uint32_t) * tc_cnt_words(d.sms))) != cudaSuccess)
      return cuda_fail(e, "cudaMalloc");
    if ((e = cudaMemset(d.tccnt, 0, sizeof(uint32_t) * tc_cnt_words(d.sms))) != cudaSuccess)
      return cuda_fail(e, "cudaMemset");
    if ((e = cudaMalloc(&d.attn_ws, sizeof(float) * attn_ws_floats(d.sms))) != cudaSuccess)
      return cuda_fail(e, "cudaMalloc");
    if ((e = cudaMalloc(&d.lp_ws, logprobs_ws_bytes(d.sms))) != cudaSuccess) return cuda_fail(e, "cudaMalloc");
    if ((e = cudaMalloc(&d.lp_cnt, sizeof(uint32_t) * logprobs_cnt_words(d.sms))) != cudaSuccess)
      return cuda_fail(e, "cudaMalloc");
    if ((e = cudaMemset(d.lp_cnt, 0, sizeof(uint32_t) * logprobs_cnt_words(d.sms))) != cudaSuccess)
      return cuda_fail(e, "cudaMemset");
    if ((e = cudaMalloc(&d.moe_bars, sizeof(uint32_t) * kMoeBarWords)) != cudaSuccess) return cuda_fail(e, "cudaMalloc");
    if ((e = cudaMemset(d.moe_bars, 0, sizeof(uint32_t) * kMoeBarWords)) != cudaSuccess) return cuda_fail(e, "cudaMemset");
    if ((e = cudaMalloc(&d.paged_cnt, sizeof(uint32_t) * kPagedCtas * d.sms)) != cudaSuccess) return cuda_fail(e, "cudaMalloc");
    if ((e = cudaMemset(d.paged_cnt, 0, sizeof(uint32_t) * kPagedCtas * d.sms)) != cudaSuccess) return cuda_fail(e, "cudaMemset");
    if ((e = cudaMemset(d.err, 0, sizeof(uint32_t))) != cudaSuccess) return cuda_fail(e, "cudaMemset");
    if ((e = cudaDeviceSynchronize()) != cudaSuccess) return cuda_fail(e, "cudaDeviceSynchronize");
    d.ready = true;
  }
  if (needs == Needs::kNorm && !d.norm_ready) {
    if ((e = norm_prepare()) != cudaSuccess) return cuda_fail(e, "RMS norm kernel set-up");
    d.norm_ready = true;
  }
  if (needs == Needs::kMoe && d.moe_ws == nullptr) {
    const rocmfp4_status st = moe_set_up(d);
    if (st != ROCMFP4_OK) return st;
  }
  if (needs == Needs::kPaged && d.paged_ws == nullptr) {
    const rocmfp4_status st = paged_set_up(d);
    if (st != ROCMFP4_OK) return st;
  }
  *out = &d;
  return ROCMFP4_OK;
}

// The state of the current device if an allocating entry point has set it
// up there, else nullptr (never creates it).
DeviceState* existing_state() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lk(g_mu);
  return g_dev[dev].ready ? &g_dev[dev] : nullptr;
}

rocmfp4_status check_shape(int64_t N, int64_t K, int variant) {
  if (!valid_variant(variant)) return fail(ROCMFP4_ERR_INVALID_ARG, "unknown variant");
  if (N < 0 || K < 0) return fail(ROCMFP4_ERR_INVALID_ARG, "negative size");
  if (K % 32 != 0) return fail(ROCMFP4_ERR_INVALID_ARG, "K must be a multiple of 32");
  return ROCMFP4_OK;
}

// Warps of a single-product streaming launch for `tiles` tiles of `nspans`
// units of `unit_bytes` weight bytes, M activation rows, with room for `cap`
// warps.  Units go to warps in contiguous equal ranges, four warps to a CTA.
// When the tiles can be dealt out whole to CTAs that each stream at most
// kAlignedCtaBytes of weights (and M <= 4), the grid has one CTA per run of
// whole tiles: a tile is then split only between the warps of one CTA
// (whenever the CTAs divide the tiles evenly), and the reduction never
// takes its cross-CTA level, whose two L2 round trips at the end of the
// launch cost more than the extra warps gain.  Otherwise (long rows, or
// 8 activation rows) every warp that fits takes a share, which keeps more
// bytes in flight.
constexpr int64_t kAlignedCtaBytes = 40 * 4608;  // 40 dual units of 32 rows x 256 weights
}  // namespace

int64_t rocmfp4::stream_warps(int64_t tiles, int64_t nspans, int64_t unit_bytes, int64_t M, int64_t cap) {
  const int64_t units = tiles * nspans;
  const int64_t maxc = cap / kStreamWarpsPerCta;
  const int64_t tpc = (tiles + maxc - 1) / maxc;  // tiles per CTA
  if (M <= 4 && tpc * nspans * unit_bytes <= kAlignedCtaBytes) {
    const int64_t w = (tiles + tpc - 1) / tpc * kStreamWarpsPerCta;
    return units < w ? units : w;
  }
  return units < cap ? units : cap;
}

namespace {

rocmfp4_status product(const void* W, const void* X, float* Y, int64_t M, int64_t N, int64_t K, int variant,
                       int act, cudaStream_t s) {
  rocmfp4_status st = check_shape(N, K, variant);
  if (st != ROCMFP4_OK) return st;
  if (!valid_act(act)) return fail(ROCMFP4_ERR_INVALID_ARG, "unknown activation type");
  if (M < 0) return fail(ROCMFP4_ERR_INVALID_ARG, "negative size");
  if (M == 0 || N == 0) return ROCMFP4_OK;
  if (Y == nullptr) return fail(ROCMFP4_ERR_INVALID_ARG, "Y is NULL");
  if (K > 0 && W == nullptr) return fail(ROCMFP4_ERR_INVALID_ARG, "W is NULL");
  if (K == 0) {
    cudaError_t e = cudaMemsetAsync(Y, 0, sizeof(float) * M * N, s);
    return e == cudaSuccess ? ROCMFP4_OK : cuda_fail(e, "cudaMemsetAsync");
  }
  if (X == nullptr) return fail(ROCMFP4_ERR_INVALID_ARG, "X is NULL");
  DeviceState* d = nullptr;
  if ((st = device_state(&d)) != ROCMFP4_OK) return st;

  const int64_t row_bytes = K / 32 * block_bytes_of(variant);
  const int64_t ku = stream_weights_per_unit(variant);
  // The streaming kernel indexes units and tiles in 32 bits.
  const bool stream_ok = K % ku == 0 && aligned16(W) && aligned16(X) &&
                         (N + kStreamTileRows - 1) / kStreamTileRows * (K / ku) < (int64_t(1) << 31);
  const uint16_t* Xh = static_cast<const uint16_t*>(X);
  // More than 8 activation rows: the tensor-core kernel reads W once per
  // 256-token tile instead of once per 8 rows.
  const bool tc_ok = M > 8 && K % tc_k_multiple(variant) == 0 && aligned16(W) && aligned16(X) &&
                     M < (int64_t(1) << 31) && N < (int64_t(1) << 31) && K < (int64_t(1) << 31);
  if (tc_ok) {
    TcArgs a{static_cast<const uint8_t*>(W), Xh, Y, M, N, K, row_bytes, d->tcws, d->tccnt, d->err};
    cudaError_t e = launch_gemm_tc(variant, act, a, s);
    if (e != cudaSuccess) return cuda_fail(e, "tensor-core kernel launch");
    g_launches.fetch_add(1);
    return ROCMFP4_OK;
  }
  if (!stream_ok || M > 8) {
    GenericArgs a{static_cast<const uint8_t*>(W), Xh, Y, N, K, row_bytes, M};
    cudaError_t e = launch_gemm_generic(variant, act, a, s);
    if (e != cudaSuccess) return cuda_fail(e, "generic kernel launch");
    g_launches.fetch_add(1);
    return ROCMFP4_OK;
  }
  const int64_t nspans = K / ku;
  const int64_t tiles = (N + kStreamTileRows - 1) / kStreamTileRows;
  const int64_t units = tiles * nspans;
  for (int64_t m0 = 0; m0 < M; m0 += 8) {
    const int mc = (int)(M - m0 < 8 ? M - m0 : 8);
    const int mb = stream_mb_for(mc);
    const int lm = mb == 1 ? 0 : mb == 2 ? 1 : mb == 4 ? 2 : 3;
    const int64_t cap = (int64_t)d->sms * d->occ[variant][act][lm] * kStreamWarpsPerCta;
    const int64_t wact = stream_warps(tiles, nspans, ku * block_bytes_of(variant), mc, cap);
    const int ctas = (int)((wact + kStreamWarpsPerCta - 1) / kStreamWarpsPerCta);
    GemvArgs a{};
    a.W = static_cast<const uint8_t*>(W);
    a.X = Xh + m0 * K;
    a.Y = Y + m0 * N;
    a.N = N;
    a.K = K;
    a.row_bytes = row_bytes;
    a.M = mc;
    a.nspans = nspans;
    a.units = units;
    a.wact = wact;
    a.ws = d->ws;
    a.cnt = d->cnt;
    a.err = d->err;
    // A grid of at most two CTAs per SM takes the deeper rings (M <= 2).
    a.deep = mb <= 2 && ctas <= 2 * d->sms ? 1 : 0;
    cudaError_t e = launch_gemv_stream(variant, act, a, ctas, s);
    if (e != cudaSuccess) return cuda_fail(e, "streaming kernel launch");
    g_launches.fetch_add(1);
  }
  return ROCMFP4_OK;
}

rocmfp4_status chain(const rocmfp4_gemv_op* ops, int count, int64_t M, int variant, int act, cudaStream_t s) {
  if (count < 0) return fail(ROCMFP4_ERR_INVALID_ARG, "negative count");
  if (count == 0) return ROCMFP4_OK;
  if (ops == nullptr) return fail(ROCMFP4_ERR_INVALID_ARG, "ops is NULL");
  if (!valid_act(act)) return fail(ROCMFP4_ERR_INVALID_ARG, "unknown activation type");
  if (M < 0) return fail(ROCMFP4_ERR_INVALID_ARG, "negative size");
  for (int i = 0; i < count; ++i) {
    const rocmfp4_gemv_op& op = ops[i];
    rocmfp4_status st = check_shape(op.N, op.K, variant);
    if (st != ROCMFP4_OK) return fail(st, "product " + std::to_string(i) + ": " + t_last_error);
    if (M == 0 || op.N == 0) continue;
    if (op.Y == nullptr || (op.K > 0 && (op.W == nullptr || op.X == nullptr)))
      return fail(ROCMFP4_ERR_INVALID_ARG, "product " + std::to_string(i) + ": NULL pointer");
  }
  if (M == 0) return ROCMFP4_OK;
  // One launch per product, in order, exactly as rocmfp4_gemm_ex would run
  // it.  Streaming launches are programmatic dependent launches: a product's
  // weights stream while the previous product finishes, and its activations
  // are read only once the previous launch has completed.  (One cooperative
  // launch with a grid barrier between products measured slower at every
  // size, from N = 256 to the layer's matrices.)
  for (int i = 0; i < count; ++i) {
    if (ops[i].N == 0) continue;
    rocmfp4_status st = product(ops[i].W, ops[i].X, ops[i].Y, M, ops[i].N, ops[i].K, variant, act, s);
    if (st != ROCMFP4_OK) return st;
  }
  return ROCMFP4_OK;
}

// Fused gate/up product (M <= 8): W holds 2I rows, the I gate rows then the
// I up rows; Y[m][i] = SiLU(gate_i . x_m) * (up_i . x_m).
rocmfp4_status gate_up(const void* W, const void* X, float* Y, int64_t M, int64_t I, int64_t K, int variant, int act,
                       cudaStream_t s) {
  rocmfp4_status st = check_shape(I, K, variant);
  if (st != ROCMFP4_OK) return st;
  if (!valid_act(act)) return fail(ROCMFP4_ERR_INVALID_ARG, "unknown activation type");
  if (M < 0) return fail(ROCMFP4_ERR_INVALID_ARG, "negative size");
  if (M == 0 || I == 0) return ROCMFP4_OK;
  if (M > 8) return fail(ROCMFP4_ERR_UNSUPPORTED, "gate/up product: at most 8 activation rows");
  if (Y == nullptr) return fail(ROCMFP4_ERR_INVALID_ARG, "Y is NULL");
  if (K > 0 && W == nullptr) return fail(ROCMFP4_ERR_INVALID_ARG, "W is NULL");
  if (K == 0) {  // SiLU(0) * 0
    cudaError_t e = cudaMemsetAsync(Y, 0, sizeof(float) * M * I, s);
    return e == cudaSuccess ? ROCMFP4_OK : cuda_fail(e, "cudaMemsetAsync");
  }
  if (X == nullptr) return fail(ROCMFP4_ERR_INVALID_ARG, "X is NULL");
  DeviceState* d = nullptr;
  if ((st = device_state(&d)) != ROCMFP4_OK) return st;
  const int64_t ku = stream_weights_per_unit(variant);
  const int64_t nspans = K / ku;
  const int64_t tiles = (I + kStreamTileRows / 2 - 1) / (kStreamTileRows / 2);  // 16 gate and 16 up rows each
  const int64_t units = tiles * nspans;
  if (K % ku != 0 || !aligned16(W) || !aligned16(X) || units >= (int64_t(1) << 31))
    return fail(ROCMFP4_ERR_UNSUPPORTED,
                "gate/up product: K must be a multiple of 256 (dual) or 512 (single-scale), W and X 16-byte aligned");
  const int mb = stream_mb_for((int)M);
  const int lm = mb == 1 ? 0 : mb == 2 ? 1 : mb == 4 ? 2 : 3;
  const int64_t cap = (int64_t)d->sms * d->occ[variant][act][lm] * kStreamWarpsPerCta;
  GemvArgs a{};
  a.W = static_cast<const uint8_t*>(W);
  a.X = static_cast<const uint16_t*>(X);
  a.Y = Y;
  a.N = I;
  a.K = K;
  a.row_bytes = K / 32 * block_bytes_of(variant);
  a.M = (int)M;
  a.nspans = nspans;
  a.units = units;
  a.wact = stream_warps(tiles, nspans, ku * block_bytes_of(variant), M, cap);
  a.ws = d->ws;
  a.cnt = d->cnt;
  a.err = d->err;
  a.epi = 1;
  const int ctas = (int)((a.wact + kStreamWarpsPerCta - 1) / kStreamWarpsPerCta);
  cudaError_t e = launch_gemv_stream(variant, act, a, ctas, s);
  if (e != cudaSuccess) return cuda_fail(e, "streaming kernel launch");
  g_launches.fetch_add(1);
  return ROCMFP4_OK;
}

rocmfp4_status decode_attention(const void* q, const void* K, const void* V, const int32_t* lens, float* out,
                                int64_t B, int64_t H, int64_t Hkv, int64_t D, int64_t Tmax, float scale, int variant,
                                int act, cudaStream_t s) {
  if (!valid_variant(variant)) return fail(ROCMFP4_ERR_INVALID_ARG, "unknown variant");
  if (!valid_act(act)) return fail(ROCMFP4_ERR_INVALID_ARG, "unknown activation type");
  if (B < 0 || H < 0 || Hkv < 1 || D < 0 || Tmax < 0) return fail(ROCMFP4_ERR_INVALID_ARG, "negative or zero size");
  if (H % Hkv != 0) return fail(ROCMFP4_ERR_INVALID_ARG, "H must be a multiple of Hkv");
  if (D % 32 != 0) return fail(ROCMFP4_ERR_INVALID_ARG, "D must be a multiple of 32");
  if (B == 0 || H == 0) return ROCMFP4_OK;
  if (out == nullptr || q == nullptr || lens == nullptr) return fail(ROCMFP4_ERR_INVALID_ARG, "NULL pointer");
  if (Tmax > 0 && (K == nullptr || V == nullptr)) return fail(ROCMFP4_ERR_INVALID_ARG, "NULL pointer");
  if (D != 64 && D != 128) return fail(ROCMFP4_ERR_UNSUPPORTED, "decode attention: D must be 64 or 128");
  if (H / Hkv > 8) return fail(ROCMFP4_ERR_UNSUPPORTED, "decode attention: at most 8 query heads per KV head");
  if (Tmax % 32 != 0) return fail(ROCMFP4_ERR_UNSUPPORTED, "decode attention: Tmax must be a multiple of 32");
  if (Tmax > 0 && (!aligned16(K) || !aligned16(V)))
    return fail(ROCMFP4_ERR_UNSUPPORTED, "decode attention: K and V must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(lens) & 3u) != 0) return fail(ROCMFP4_ERR_INVALID_ARG, "lens misaligned");
  if (B * H >= (int64_t(1) << 31) || B * Hkv * Tmax >= (int64_t(1) << 40) || Tmax >= (int64_t(1) << 31))
    return fail(ROCMFP4_ERR_UNSUPPORTED, "decode attention: sizes too large");
  if (!(scale == scale)) return fail(ROCMFP4_ERR_INVALID_ARG, "scale is NaN");
  if (Tmax == 0) {  // no token anywhere: zeros
    cudaError_t e = cudaMemsetAsync(out, 0, sizeof(float) * B * H * D, s);
    return e == cudaSuccess ? ROCMFP4_OK : cuda_fail(e, "cudaMemsetAsync");
  }
  DeviceState* d = nullptr;
  rocmfp4_status st = device_state(&d);
  if (st != ROCMFP4_OK) return st;
  AttnArgs a{static_cast<const uint16_t*>(q), static_cast<const uint8_t*>(K), static_cast<const uint8_t*>(V), lens,
             out, d->attn_ws, B, H, Hkv, D, Tmax, scale, d->err};
  int launches = 0;
  cudaError_t e = launch_decode_attention(variant, act, a, d->sms, s, &launches);
  g_launches.fetch_add((uint64_t)launches);
  if (e != cudaSuccess) return cuda_fail(e, "decode attention launch");
  return ROCMFP4_OK;
}

rocmfp4_status add_rmsnorm(NormArgs a, int64_t group, cudaStream_t s) {
  if (!valid_dtype(a.x_type) || !valid_dtype(a.weight_type) || (a.residual && !valid_dtype(a.residual_type)))
    return fail(ROCMFP4_ERR_INVALID_ARG, "unknown type");
  if (!valid_act(a.y_act)) return fail(ROCMFP4_ERR_INVALID_ARG, "unknown activation type");
  if (a.M < 0 || a.D < 0) return fail(ROCMFP4_ERR_INVALID_ARG, "negative size");
  if (group != 0 && group != 32 && group != 64 && group != 128)
    return fail(ROCMFP4_ERR_INVALID_ARG, "group must be 0 (the row), 32, 64 or 128");
  if (!(a.eps >= 0.f) || a.eps > 3.4e38f) return fail(ROCMFP4_ERR_INVALID_ARG, "eps must be finite and not negative");
  if (a.M == 0) return ROCMFP4_OK;
  if (a.D == 0) return fail(ROCMFP4_ERR_INVALID_ARG, "D must be positive");
  if (a.x == nullptr || a.weight == nullptr || (a.residual != nullptr && a.residual_out == nullptr) ||
      (a.y == nullptr && a.q == nullptr) || (a.q == nullptr) != (a.scales == nullptr))
    return fail(ROCMFP4_ERR_INVALID_ARG, "NULL pointer");
  if (a.ldx < a.D || (a.residual && (a.ldr < a.D || a.ldro < a.D)))
    return fail(ROCMFP4_ERR_INVALID_ARG, "row stride below D");
  if (a.residual == a.residual_out && a.residual && a.ldr != a.ldro)
    return fail(ROCMFP4_ERR_INVALID_ARG, "residual updated in place needs one stride");
  if (!aligned_to(a.x, a.x_type) || !aligned_to(a.weight, a.weight_type) || !aligned_to(a.y, ROCMFP4_OUT_F16) ||
      !aligned_to(a.scales, ROCMFP4_OUT_F32) ||
      (a.residual && (!aligned_to(a.residual, a.residual_type) || !aligned_to(a.residual_out, a.residual_type))))
    return fail(ROCMFP4_ERR_INVALID_ARG, "misaligned pointer");
  if (a.D > norm_max_width()) return fail(ROCMFP4_ERR_UNSUPPORTED, "RMS norm: D at most 32768");
  if (a.M >= (int64_t(1) << 31)) return fail(ROCMFP4_ERR_UNSUPPORTED, "RMS norm: M too large");
  DeviceState* d = nullptr;
  rocmfp4_status st = device_state(&d, Needs::kNorm);
  if (st != ROCMFP4_OK) return st;
  a.err = d->err;
  cudaError_t e = launch_norm(a, d->sms, s);
  if (e != cudaSuccess) return cuda_fail(e, "RMS norm launch");
  g_launches.fetch_add(1);
  return ROCMFP4_OK;
}

rocmfp4_status moe(MoeArgs a, int variant, int act, cudaStream_t s) {
  if (!valid_variant(variant)) return fail(ROCMFP4_ERR_INVALID_ARG, "unknown variant");
  if (!valid_act(act)) return fail(ROCMFP4_ERR_INVALID_ARG, "unknown activation type");
  if (!valid_dtype(a.router_type)) return fail(ROCMFP4_ERR_INVALID_ARG, "unknown type");
  if (a.route != ROCMFP4_ROUTE_SOFTMAX && a.route != ROCMFP4_ROUTE_SOFTMAX_TOPK && a.route != ROCMFP4_ROUTE_SIGMOID)
    return fail(ROCMFP4_ERR_INVALID_ARG, "unknown route");
  if (a.M < 0) return fail(ROCMFP4_ERR_INVALID_ARG, "negative size");
  if (a.E < 1 || a.top_k < 1 || a.top_k > a.E) return fail(ROCMFP4_ERR_INVALID_ARG, "1 <= top_k <= E is needed");
  if (a.K < 32 || a.I < 32 || a.K % 32 != 0 || a.I % 32 != 0)
    return fail(ROCMFP4_ERR_INVALID_ARG, "K and I must be positive multiples of 32");
  if (!(a.route_scale >= -3.4e38f && a.route_scale <= 3.4e38f)) return fail(ROCMFP4_ERR_INVALID_ARG, "route_scale must be finite");
  if (a.M == 0) return ROCMFP4_OK;
  if (!a.X || !a.router || !a.Wgu || !a.Wd || !a.Y) return fail(ROCMFP4_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned_to(a.Y, 0) || !aligned_to(a.ids, 0) || !aligned_to(a.probs, 0))
    return fail(ROCMFP4_ERR_INVALID_ARG, "misaligned pointer");
  if (a.M > kMoeMaxTokens || a.E > kMoeMaxExperts || a.top_k > kMoeMaxTop || a.K > kMoeMaxWidth || a.I > kMoeMaxWidth ||
      a.M * a.top_k * a.I > kMoeMaxHidden)
    return fail(ROCMFP4_ERR_UNSUPPORTED,
                "mixture of experts: at most 32 tokens, 512 experts, 16 choices, widths of 32768 and 2^22 hidden values");
  if (!aligned16(a.X) || !aligned16(a.router) || !aligned16(a.Wgu) || !aligned16(a.Wd))
    return fail(ROCMFP4_ERR_UNSUPPORTED, "mixture of experts: X, router, Wgu and Wd must be 16-byte aligned");
  DeviceState* d = nullptr;
  rocmfp4_status st = device_state(&d, Needs::kMoe);
  if (st != ROCMFP4_OK) return st;
  a.ws = d->moe_ws;
  a.bars = d->moe_bars;
  a.err = d->err;
  cudaError_t e = launch_moe(variant, act, a, d->sms, s);
  if (e != cudaSuccess) return cuda_fail(e, "mixture-of-experts launch");
  g_launches.fetch_add(1);
  return ROCMFP4_OK;
}

rocmfp4_status logprobs(LogprobsArgs a, int64_t top_n, cudaStream_t s) {
  if (!valid_dtype(a.type)) return fail(ROCMFP4_ERR_INVALID_ARG, "unknown type");
  if (a.M < 0 || a.V < 0 || top_n < 0) return fail(ROCMFP4_ERR_INVALID_ARG, "negative size");
  if (!(a.scale >= 1e-30f && a.scale <= 1e30f)) return fail(ROCMFP4_ERR_INVALID_ARG, "scale must be from 1e-30 to 1e30");
  if (a.M == 0) return ROCMFP4_OK;
  if (a.V == 0) return fail(ROCMFP4_ERR_INVALID_ARG, "V must be positive");
  if (a.ld < a.V) return fail(ROCMFP4_ERR_INVALID_ARG, "row stride below V");
  if (top_n > a.V) return fail(ROCMFP4_ERR_INVALID_ARG, "top_n above V");
  if (a.logits == nullptr || (a.targets != nullptr && a.logprob == nullptr) ||
      (top_n > 0 && (a.top_ids == nullptr || a.top_logprobs == nullptr)))
    return fail(ROCMFP4_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned_to(a.logits, a.type) || !aligned_to(a.targets, 0) || !aligned_to(a.logprob, 0) ||
      !aligned_to(a.entropy, 0) || !aligned_to(a.top_ids, 0) || !aligned_to(a.top_logprobs, 0))
    return fail(ROCMFP4_ERR_INVALID_ARG, "misaligned pointer");
  if (top_n > kMaxTop) return fail(ROCMFP4_ERR_UNSUPPORTED, "log probabilities: top_n at most 32");
  if (a.V >= (int64_t(1) << 31) - 64 || a.M >= (int64_t(1) << 31))
    return fail(ROCMFP4_ERR_UNSUPPORTED, "log probabilities: sizes too large");
  DeviceState* d = nullptr;
  rocmfp4_status st = device_state(&d);
  if (st != ROCMFP4_OK) return st;
  a.top_n = (int)top_n;
  a.ws = d->lp_ws;
  a.cnt = d->lp_cnt;
  cudaError_t e = launch_logprobs(a, d->sms, s);
  if (e != cudaSuccess) return cuda_fail(e, "log probabilities launch");
  g_launches.fetch_add(1);
  return ROCMFP4_OK;
}

// The cache description of a call, checked, as the kernels see it.
rocmfp4_status paged_args(const rocmfp4_paged_cache* c, PagedArgs* out) {
  if (c == nullptr) return fail(ROCMFP4_ERR_INVALID_ARG, "cache is NULL");
  if (!valid_variant(c->variant)) return fail(ROCMFP4_ERR_INVALID_ARG, "unknown variant");
  if (c->B < 0 || c->table_width < 0 || c->num_pages < 0) return fail(ROCMFP4_ERR_INVALID_ARG, "negative size");
  if (c->Hkv < 1 || c->D < 32 || c->page_size < 1) return fail(ROCMFP4_ERR_INVALID_ARG, "Hkv, D and page_size must be positive");
  if (c->D % 32 != 0) return fail(ROCMFP4_ERR_INVALID_ARG, "D must be a multiple of 32");
  if (c->table_stride != 0 && c->table_stride < c->table_width) return fail(ROCMFP4_ERR_INVALID_ARG, "table_stride below table_width");
  if (!c->cu || (c->B > 0 && !c->lens) || (c->table_width > 0 && !c->table) || (c->num_pages > 0 && (!c->K || !c->V)))
    return fail(ROCMFP4_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned_to(c->cu, 0) || !aligned_to(c->lens, 0) || !aligned_to(c->table, 0))
    return fail(ROCMFP4_ERR_INVALID_ARG, "misaligned pointer");
  if (!aligned16(c->K) || !aligned16(c->V)) return fail(ROCMFP4_ERR_UNSUPPORTED, "paged cache: K and V must be 16-byte aligned");
  const int64_t most = int64_t(1) << 31;
  if (c->page_size % 16 != 0) return fail(ROCMFP4_ERR_UNSUPPORTED, "paged cache: page_size must be a multiple of 16");
  if (c->D > 256) return fail(ROCMFP4_ERR_UNSUPPORTED, "paged cache: D at most 256");
  if (c->B >= most || c->table_width >= most || c->num_pages >= most || c->page_size >= most || c->Hkv > 65536 ||
      c->table_width > (most >> 1) / c->page_size)
    return fail(ROCMFP4_ERR_UNSUPPORTED, "paged cache: sizes too large");
  PagedArgs& p = *out;
  p.K = static_cast<uint8_t*>(c->K);
  p.V = static_cast<uint8_t*>(c->V);
  p.table = c->table;
  p.lens = c->lens;
  p.cu = c->cu;
  p.ldt = c->table_stride;
  p.B = (int)c->B;
  p.width = (int)c->table_width;
  p.num_pages = (int)c->num_pages;
  p.page_size = (int)c->page_size;
  p.Hkv = (int)c->Hkv;
  p.D = (int)c->D;
  return ROCMFP4_OK;
}

// Whether rows of `width` bytes, `stride` apart, touch the `bytes` from `out` on; rows with gaps count whole.
bool rows_touch(const void* x, int64_t rows, int64_t stride, int64_t width, const void* out, int64_t bytes) {
  if (x == nullptr || rows == 0 || bytes == 0) return false;
  const unsigned __int128 a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(out);
  return a < b + bytes && b < a + (unsigned __int128)(rows - 1) * stride + width;
}

// Shared by rocmfp4_rotary and rocmfp4_rope_append (`cache` not NULL).
rocmfp4_status rope(RopeArgs a, const rocmfp4_paged_cache* cache, cudaStream_t s) {
  rocmfp4_status st;
  if (a.paged) {
    if ((st = paged_args(cache, &a.cache)) != ROCMFP4_OK) return st;
    a.D = cache->D;
  }
  if (!valid_dtype(a.type)) return fail(ROCMFP4_ERR_INVALID_ARG, "unknown type");
  if (!valid_act(a.act)) return fail(ROCMFP4_ERR_INVALID_ARG, "unknown activation type");
  if (a.M < 0 || a.H < 0) return fail(ROCMFP4_ERR_INVALID_ARG, "negative size");
  if (a.D < 32 || a.D % 32 != 0) return fail(ROCMFP4_ERR_INVALID_ARG, "D must be a positive multiple of 32");
  if (a.rot < 0 || a.rot > a.D || a.rot % 2 != 0) return fail(ROCMFP4_ERR_INVALID_ARG, "rot must be even, from 0 to D");
  if (!(a.amplitude >= -3.4e38f && a.amplitude <= 3.4e38f)) return fail(ROCMFP4_ERR_INVALID_ARG, "amplitude must be finite");
  if (a.M == 0 || (a.paged && a.cache.B == 0) || (!a.paged && a.H == 0)) return ROCMFP4_OK;
  const int64_t widths[3] = {a.H * a.D, a.paged ? a.cache.Hkv * a.D : 0, a.paged ? a.cache.Hkv * a.D : 0};
  for (int i = 0; i < 3; ++i) {
    if (widths[i] == 0) {
      a.x[i] = nullptr;
      continue;
    }
    if (a.x[i] == nullptr) return fail(ROCMFP4_ERR_INVALID_ARG, "NULL pointer");
    if (!aligned_to(a.x[i], a.type)) return fail(ROCMFP4_ERR_INVALID_ARG, "misaligned pointer");
    if (a.ld[i] < widths[i]) return fail(ROCMFP4_ERR_INVALID_ARG, "row stride below the heads' width");
  }
  if ((a.H > 0 && a.q_out == nullptr) || (a.rot > 0 && a.freq == nullptr) || (!a.paged && a.rot > 0 && a.positions == nullptr))
    return fail(ROCMFP4_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned_to(a.freq, 0) || !aligned_to(a.positions, 0) || !aligned_to(a.q_out, ROCMFP4_OUT_F16))
    return fail(ROCMFP4_ERR_INVALID_ARG, "misaligned pointer");
  if (a.D > 256) return fail(ROCMFP4_ERR_UNSUPPORTED, "rotary positions: D at most 256");
  if (a.H > 65536 || a.M * (a.D / 32) >= (int64_t(1) << 31)) return fail(ROCMFP4_ERR_UNSUPPORTED, "rotary positions: sizes too large");
  if ((reinterpret_cast<uintptr_t>(a.q_out) & 7u) != 0)
    return fail(ROCMFP4_ERR_UNSUPPORTED, "rotary positions: the output must be 8-byte aligned");
  // Partners of a pair may be read by another block after a value's output: in place the results would depend on the order.
  const int64_t size = a.type == ROCMFP4_OUT_F32 ? 4 : 2;
  for (int i = 0; i < 3; ++i)
    if (rows_touch(a.x[i], a.M, a.ld[i] * size, widths[i] * size, a.q_out, a.M * widths[0] * 2))
      return fail(ROCMFP4_ERR_INVALID_ARG, "the output must not overlap the inputs");
  DeviceState* d = nullptr;
  if ((st = device_state(&d)) != ROCMFP4_OK) return st;
  a.cache.err = d->err;
  cudaError_t e = launch_rope(a.paged ? cache->variant : 0, a, d->sms, s);
  if (e != cudaSuccess) return cuda_fail(e, "rotary positions launch");
  g_launches.fetch_add(1);
  return ROCMFP4_OK;
}

rocmfp4_status cache_read(const rocmfp4_paged_cache* cache, CacheReadArgs a, int type, cudaStream_t s) {
  rocmfp4_status st = paged_args(cache, &a.cache);
  if (st != ROCMFP4_OK) return st;
  if (!valid_dtype(type)) return fail(ROCMFP4_ERR_INVALID_ARG, "unknown type");
  if (a.M < 0) return fail(ROCMFP4_ERR_INVALID_ARG, "negative size");
  if (a.M == 0 || a.cache.B == 0) return ROCMFP4_OK;
  if (a.k_out == nullptr && a.v_out == nullptr) return fail(ROCMFP4_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned_to(a.k_out, type) || !aligned_to(a.v_out, type)) return fail(ROCMFP4_ERR_INVALID_ARG, "misaligned pointer");
  if (!aligned16(a.k_out) || !aligned16(a.v_out)) return fail(ROCMFP4_ERR_UNSUPPORTED, "reading a cache: outputs must be 16-byte aligned");
  if (a.M >= (int64_t(1) << 31)) return fail(ROCMFP4_ERR_UNSUPPORTED, "reading a cache: M too large");
  DeviceState* d = nullptr;
  if ((st = device_state(&d)) != ROCMFP4_OK) return st;
  a.cache.err = d->err;
  cudaError_t e = launch_cache_read(cache->variant, type, a, d->sms, s);
  if (e != cudaSuccess) return cuda_fail(e, "cache read launch");
  g_launches.fetch_add(1);
  return ROCMFP4_OK;
}

rocmfp4_status paged_attention(const rocmfp4_paged_cache* cache, PagedAttnArgs a, int64_t H, int64_t window, int act,
                               cudaStream_t s) {
  rocmfp4_status st = paged_args(cache, &a.cache);
  if (st != ROCMFP4_OK) return st;
  if (!valid_act(act)) return fail(ROCMFP4_ERR_INVALID_ARG, "unknown activation type");
  if (a.M < 0 || H < 0 || window < 0) return fail(ROCMFP4_ERR_INVALID_ARG, "negative size");
  if (H % cache->Hkv != 0) return fail(ROCMFP4_ERR_INVALID_ARG, "H must be a multiple of Hkv");
  if (!(a.scale >= 1e-30f && a.scale <= 1e30f)) return fail(ROCMFP4_ERR_INVALID_ARG, "scale must be from 1e-30 to 1e30");
  if (a.causal != 0 && a.causal != 1) return fail(ROCMFP4_ERR_INVALID_ARG, "causal is 0 or 1");
  if (!a.causal && window != 0) return fail(ROCMFP4_ERR_INVALID_ARG, "a window needs causal");
  if (a.M == 0 || H == 0 || a.cache.B == 0) return ROCMFP4_OK;
  if (a.q == nullptr || a.out == nullptr) return fail(ROCMFP4_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned_to(a.q, ROCMFP4_OUT_F16) || !aligned_to(a.out, ROCMFP4_OUT_F16))
    return fail(ROCMFP4_ERR_INVALID_ARG, "misaligned pointer");
  if (a.ldq < H * cache->D) return fail(ROCMFP4_ERR_INVALID_ARG, "row stride below the heads' width");
  if (cache->D != 64 && cache->D != 128) return fail(ROCMFP4_ERR_UNSUPPORTED, "paged attention: D must be 64 or 128");
  if (!aligned16(a.q) || a.ldq % 8 != 0 || !aligned16(a.out))
    return fail(ROCMFP4_ERR_UNSUPPORTED, "paged attention: q's rows and out must be 16-byte aligned");
  if (a.M * H >= (int64_t(1) << 31) || H > 65536) return fail(ROCMFP4_ERR_UNSUPPORTED, "paged attention: sizes too large");
  a.H = (int)H;
  a.window = window >= (int64_t(1) << 31) ? 0 : (int)window;  // no sequence is as long
  DeviceState* d = nullptr;
  if ((st = device_state(&d, Needs::kPaged)) != ROCMFP4_OK) return st;
  a.cache.err = d->err;
  a.ws = d->paged_ws;
  a.cnt = d->paged_cnt;
  // At most 16 (row, head) pairs a sequence and KV head, on the average: the kernel of few rows, tiles of 8; else tiles of 128
  // and 256.  Measured, few against many: 16 rows: 41 / 62 us (32768 tokens), 68 / 69 (16 sequences of 4096), 71 / 86 (64 of 1000),
  // 19 / 27 (9 of 3001, D = 64); 20 to 24 rows: 52 / 62, 90 / 70, 100 / 89, 23 / 28.  The lengths of the chunks are on the device:
  // either kernel is right for any.  A batch of unequal chunks is served by the one that its average names: 64 single tokens over
  // 4096 with 512 rows over 16384 take 479 us, in two calls 111 + 167.
  const bool few = a.M * (H / cache->Hkv) <= 16 * (int64_t)cache->B;
  cudaError_t e = few ? launch_paged_few(cache->variant, act, a, d->sms, s) : launch_paged_attention(cache->variant, act, a, d->sms, s);
  if (e != cudaSuccess) return cuda_fail(e, "paged attention launch");
  g_launches.fetch_add(1);
  return ROCMFP4_OK;
}

}  // namespace

namespace rocmfp4 {
void set_last_error(const std::string& message) { t_last_error = message; }
void count_launch() { g_launches.fetch_add(1); }
}  // namespace rocmfp4

extern "C" {

size_t rocmfp4_block_bytes(rocmfp4_variant variant) {
  return valid_variant(variant) ? (size_t)block_bytes_of(variant) : 0;
}

size_t rocmfp4_row_bytes(int64_t K, rocmfp4_variant variant) {
  if (!valid_variant(variant) || K < 0 || K % 32 != 0) return 0;
  return (size_t)(K / 32 * block_bytes_of(variant));
}

rocmfp4_status rocmfp4_gemv(const void* W, const void* x, float* y, int64_t N, int64_t K,
                            rocmfp4_variant variant) {
  return product(W, x, y, 1, N, K, variant, ROCMFP4_ACT_F16, nullptr);
}

rocmfp4_status rocmfp4_gemv_ex(const void* W, const void* x, float* y, int64_t N, int64_t K,
                               rocmfp4_variant variant, rocmfp4_act act, rocmfp4_stream_t stream) {
  return product(W, x, y, 1, N, K, variant, act, reinterpret_cast<cudaStream_t>(stream));
}

rocmfp4_status rocmfp4_gemm(const void* W, const void* X, float* Y, int64_t M, int64_t N, int64_t K,
                            rocmfp4_variant variant) {
  return product(W, X, Y, M, N, K, variant, ROCMFP4_ACT_BF16, nullptr);
}

rocmfp4_status rocmfp4_gemm_ex(const void* W, const void* X, float* Y, int64_t M, int64_t N, int64_t K,
                               rocmfp4_variant variant, rocmfp4_act act, rocmfp4_stream_t stream) {
  return product(W, X, Y, M, N, K, variant, act, reinterpret_cast<cudaStream_t>(stream));
}

rocmfp4_status rocmfp4_gemv_gate_up(const void* W, const void* X, float* Y, int64_t M, int64_t I, int64_t K,
                                    rocmfp4_variant variant, rocmfp4_act act, rocmfp4_stream_t stream) {
  return gate_up(W, X, Y, M, I, K, variant, act, reinterpret_cast<cudaStream_t>(stream));
}

rocmfp4_status rocmfp4_decode_attention(const void* q, const void* K, const void* V, const int32_t* lens, float* out,
                                        int64_t B, int64_t H, int64_t Hkv, int64_t D, int64_t Tmax, float scale,
                                        rocmfp4_variant variant, rocmfp4_act act, rocmfp4_stream_t stream) {
  return decode_attention(q, K, V, lens, out, B, H, Hkv, D, Tmax, scale, variant, act,
                          reinterpret_cast<cudaStream_t>(stream));
}

rocmfp4_status rocmfp4_add_rmsnorm(const void* x, rocmfp4_out_dtype x_type, int64_t ldx, const void* residual,
                                   void* residual_out, rocmfp4_out_dtype residual_type, int64_t ldr, int64_t ldro,
                                   const void* weight, rocmfp4_out_dtype weight_type, float eps, void* y,
                                   rocmfp4_act y_type, void* q, float* scales, int64_t group, int64_t M, int64_t D,
                                   rocmfp4_stream_t stream) {
  NormArgs a{};
  a.x = x;
  a.residual = residual;
  a.residual_out = residual_out;
  a.weight = weight;
  a.y = y;
  a.q = static_cast<uint8_t*>(q);
  a.scales = scales;
  a.M = M;
  a.D = D;
  a.ldx = ldx;
  a.ldr = ldr;
  a.ldro = ldro;
  a.x_type = x_type;
  a.residual_type = residual_type;
  a.weight_type = weight_type;
  a.y_act = y_type;
  a.group = (int)group;
  a.eps = eps;
  return add_rmsnorm(a, group, reinterpret_cast<cudaStream_t>(stream));
}

rocmfp4_status rocmfp4_moe(const void* X, const void* router, rocmfp4_out_dtype router_type, const void* Wgu,
                           const void* Wd, float* Y, int32_t* ids, float* probs, int64_t M, int64_t E, int64_t top_k,
                           int64_t K, int64_t I, rocmfp4_route route, float route_scale, rocmfp4_variant variant,
                           rocmfp4_act act, rocmfp4_stream_t stream) {
  MoeArgs a{};
  a.X = static_cast<const uint16_t*>(X);
  a.router = router;
  a.Wgu = static_cast<const uint8_t*>(Wgu);
  a.Wd = static_cast<const uint8_t*>(Wd);
  a.Y = Y;
  a.ids = ids;
  a.probs = probs;
  a.M = M;
  a.E = E;
  a.top_k = top_k;
  a.K = K;
  a.I = I;
  a.router_type = router_type;
  a.route = route;
  a.route_scale = route_scale;
  return moe(a, variant, act, reinterpret_cast<cudaStream_t>(stream));
}

rocmfp4_status rocmfp4_logprobs(const void* logits, rocmfp4_out_dtype type, int64_t ld, const int32_t* targets,
                                float scale, float* logprob, float* entropy, int32_t* top_ids, float* top_logprobs,
                                int64_t top_n, int64_t M, int64_t V, rocmfp4_stream_t stream) {
  LogprobsArgs a{};
  a.logits = logits;
  a.targets = targets;
  a.logprob = logprob;
  a.entropy = entropy;
  a.top_ids = top_ids;
  a.top_logprobs = top_logprobs;
  a.M = M;
  a.V = V;
  a.ld = ld;
  a.scale = scale;
  a.type = type;
  return logprobs(a, top_n, reinterpret_cast<cudaStream_t>(stream));
}

rocmfp4_status rocmfp4_rotary(const void* x, rocmfp4_out_dtype x_type, int64_t ldx, const int32_t* positions,
                              const float* freq, int64_t rot, int interleaved, float amplitude, void* y,
                              rocmfp4_act y_type, int64_t M, int64_t H, int64_t D, rocmfp4_stream_t stream) {
  RopeArgs a{};
  a.x[0] = x;
  a.ld[0] = ldx;
  a.positions = positions;
  a.freq = freq;
  a.q_out = static_cast<uint16_t*>(y);
  a.M = M;
  a.H = H;
  a.D = D;
  a.rot = rot;
  a.type = x_type;
  a.act = y_type;
  a.interleaved = interleaved;
  a.amplitude = amplitude;
  return rope(a, nullptr, reinterpret_cast<cudaStream_t>(stream));
}

rocmfp4_status rocmfp4_rope_append(const rocmfp4_paged_cache* cache, const void* q, const void* k, const void* v,
                                   rocmfp4_out_dtype type, int64_t ldq, int64_t ldk, int64_t ldv,
                                   const int32_t* positions, const float* freq, int64_t rot, int interleaved,
                                   float amplitude, void* q_out, rocmfp4_act q_type, int64_t M, int64_t H,
                                   rocmfp4_stream_t stream) {
  RopeArgs a{};
  a.x[0] = q;
  a.x[1] = k;
  a.x[2] = v;
  a.ld[0] = ldq;
  a.ld[1] = ldk;
  a.ld[2] = ldv;
  a.positions = positions;
  a.freq = freq;
  a.q_out = static_cast<uint16_t*>(q_out);
  a.M = M;
  a.H = H;
  a.rot = rot;
  a.type = type;
  a.act = q_type;
  a.interleaved = interleaved;
  a.paged = 1;
  a.amplitude = amplitude;
  return rope(a, cache, reinterpret_cast<cudaStream_t>(stream));
}

rocmfp4_status rocmfp4_cache_read(const rocmfp4_paged_cache* cache, void* k_out, void* v_out, rocmfp4_out_dtype type,
                                  int64_t M, rocmfp4_stream_t stream) {
  CacheReadArgs a{};
  a.k_out = k_out;
  a.v_out = v_out;
  a.M = M;
  return cache_read(cache, a, type, reinterpret_cast<cudaStream_t>(stream));
}

rocmfp4_status rocmfp4_paged_attention(const void* q, int64_t ldq, const rocmfp4_paged_cache* cache, void* out, int64_t M,
                                       int64_t H, float scale, int causal, int64_t window, rocmfp4_act act,
                                       rocmfp4_stream_t stream) {
  PagedAttnArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.ldq = ldq;
  a.out = static_cast<uint16_t*>(out);
  a.M = M;
  a.causal = causal;
  a.scale = scale;
  return paged_attention(cache, a, H, window, act, reinterpret_cast<cudaStream_t>(stream));
}

rocmfp4_status rocmfp4_gemv_chain(const rocmfp4_gemv_op* ops, int count, int64_t M, rocmfp4_variant variant,
                                  rocmfp4_act act, rocmfp4_stream_t stream) {
  return chain(ops, count, M, variant, act, reinterpret_cast<cudaStream_t>(stream));
}

rocmfp4_status rocmfp4_gemv_chain_mixed(const rocmfp4_gemv_op* ops, const rocmfp4_variant* variants, int count,
                                        int64_t M, rocmfp4_act act, rocmfp4_stream_t stream) {
  if (count < 0) return fail(ROCMFP4_ERR_INVALID_ARG, "negative count");
  if (count == 0) return ROCMFP4_OK;
  if (ops == nullptr || variants == nullptr) return fail(ROCMFP4_ERR_INVALID_ARG, "ops or variants is NULL");
  if (!valid_act(act)) return fail(ROCMFP4_ERR_INVALID_ARG, "unknown activation type");
  if (M < 0) return fail(ROCMFP4_ERR_INVALID_ARG, "negative size");
  // every product is checked before any launch, as in a single-layout chain
  for (int i = 0; i < count; ++i) {
    const rocmfp4_gemv_op& op = ops[i];
    rocmfp4_status st = check_shape(op.N, op.K, variants[i]);
    if (st != ROCMFP4_OK) return fail(st, "product " + std::to_string(i) + ": " + t_last_error);
    if (M == 0 || op.N == 0) continue;
    if (op.Y == nullptr || (op.K > 0 && (op.W == nullptr || op.X == nullptr)))
      return fail(ROCMFP4_ERR_INVALID_ARG, "product " + std::to_string(i) + ": NULL pointer");
  }
  // runs of products with one layout, each a single-layout chain, in order
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  for (int i = 0; i < count;) {
    int n = 1;
    while (i + n < count && variants[i + n] == variants[i]) ++n;
    rocmfp4_status st = chain(ops + i, n, M, variants[i], act, s);
    if (st != ROCMFP4_OK) return st;
    i += n;
  }
  return ROCMFP4_OK;
}

rocmfp4_status rocmfp4_dequant(const void* W, void* out, rocmfp4_out_dtype out_dtype, int64_t N, int64_t K,
                               rocmfp4_variant variant, rocmfp4_stream_t stream) {
  rocmfp4_status st = check_shape(N, K, variant);
  if (st != ROCMFP4_OK) return st;
  if (out_dtype != ROCMFP4_OUT_F32 && out_dtype != ROCMFP4_OUT_BF16 && out_dtype != ROCMFP4_OUT_F16)
    return fail(ROCMFP4_ERR_INVALID_ARG, "unknown output type");
  const int64_t nblocks = N * (K / 32);
  if (nblocks == 0) return ROCMFP4_OK;
  if (W == nullptr) return fail(ROCMFP4_ERR_INVALID_ARG, "W is NULL");
  if (out == nullptr) return fail(ROCMFP4_ERR_INVALID_ARG, "out is NULL");
  cudaError_t e = launch_dequant(variant, out_dtype, static_cast<const uint8_t*>(W), out, nblocks,
                                 reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "dequant launch");
  g_launches.fetch_add(1);
  return ROCMFP4_OK;
}

rocmfp4_status rocmfp4_quantize(const void* src, rocmfp4_act src_type, void* W, int64_t N, int64_t K,
                                rocmfp4_variant variant, rocmfp4_stream_t stream) {
  rocmfp4_status st = check_shape(N, K, variant);
  if (st != ROCMFP4_OK) return st;
  if (!valid_act(src_type)) return fail(ROCMFP4_ERR_INVALID_ARG, "unknown source type");
  const int64_t nblocks = N * (K / 32);
  if (nblocks == 0) return ROCMFP4_OK;
  if (src == nullptr || W == nullptr) return fail(ROCMFP4_ERR_INVALID_ARG, "NULL pointer");
  if ((reinterpret_cast<uintptr_t>(src) & 1u) != 0) return fail(ROCMFP4_ERR_INVALID_ARG, "src misaligned");
  cudaError_t e = launch_quantize(variant, src_type, static_cast<const uint16_t*>(src), static_cast<uint8_t*>(W),
                                  nblocks, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "quantize launch");
  g_launches.fetch_add(1);
  return ROCMFP4_OK;
}

rocmfp4_status rocmfp4_copy(void* dst, const void* src, int64_t bytes, rocmfp4_stream_t stream) {
  if (bytes < 0) return fail(ROCMFP4_ERR_INVALID_ARG, "negative size");
  if (bytes == 0) return ROCMFP4_OK;
  if (dst == nullptr || src == nullptr) return fail(ROCMFP4_ERR_INVALID_ARG, "NULL pointer");
  const uintptr_t d = reinterpret_cast<uintptr_t>(dst), sp = reinterpret_cast<uintptr_t>(src);
  if ((d < sp ? sp - d : d - sp) < (uintptr_t)bytes) return fail(ROCMFP4_ERR_INVALID_ARG, "overlapping ranges");
  // Each side must be memory a kernel on the current device can address:
  // its own device memory, managed memory, or pinned host memory (through
  // its device pointer).  Pageable host memory and another device's memory
  // are refused rather than handed to the kernel.
  int cur = 0;
  cudaError_t ce = cudaGetDevice(&cur);
  if (ce != cudaSuccess) return cuda_fail(ce, "cudaGetDevice");
  void* ends[2] = {dst, const_cast<void*>(src)};
  for (void*& p : ends) {
    cudaPointerAttributes at{};
    cudaError_t e = cudaPointerGetAttributes(&at, p);
    if (e != cudaSuccess) return cuda_fail(e, "cudaPointerGetAttributes");
    if (at.type == cudaMemoryTypeUnregistered)
      return fail(ROCMFP4_ERR_INVALID_ARG, "pageable host memory: pin it (cudaHostAlloc / cudaHostRegister)");
    if (at.type == cudaMemoryTypeDevice && at.device != cur)
      return fail(ROCMFP4_ERR_INVALID_ARG, "device memory of another device");
    if (at.type == cudaMemoryTypeHost) {
      if (at.devicePointer == nullptr) return fail(ROCMFP4_ERR_INVALID_ARG, "host memory not mapped for the device");
      p = at.devicePointer;
    }
  }
  cudaError_t e = launch_copy(ends[0], ends[1], bytes, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "copy launch");
  g_launches.fetch_add(1);
  return ROCMFP4_OK;
}

rocmfp4_status rocmfp4_validate(const void* W, int64_t N, int64_t K, rocmfp4_variant variant,
                                int64_t* first_bad_block, rocmfp4_stream_t stream) {
  if (first_bad_block) *first_bad_block = -1;
  rocmfp4_status st = check_shape(N, K, variant);
  if (st != ROCMFP4_OK) return st;
  const int64_t nblocks = N * (K / 32);
  if (nblocks == 0) return ROCMFP4_OK;
  if (W == nullptr) return fail(ROCMFP4_ERR_INVALID_ARG, "W is NULL");
  DeviceState* d = nullptr;
  if ((st = device_state(&d)) != ROCMFP4_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  unsigned long long first = ~0ull;
  cudaError_t e = cudaMemcpyAsync(d->vfirst, &first, sizeof(first), cudaMemcpyHostToDevice, s);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemcpyAsync");
  if ((e = launch_validate(variant, static_cast<const uint8_t*>(W), nblocks, d->vfirst, s)) != cudaSuccess)
    return cuda_fail(e, "validate launch");
  g_launches.fetch_add(1);
  if ((e = cudaMemcpyAsync(&first, d->vfirst, sizeof(first), cudaMemcpyDeviceToHost, s)) != cudaSuccess)
    return cuda_fail(e, "cudaMemcpyAsync");
  if ((e = cudaStreamSynchronize(s)) != cudaSuccess) return cuda_fail(e, "cudaStreamSynchronize");
  if (first == ~0ull) return ROCMFP4_OK;
  if (first_bad_block) *first_bad_block = (int64_t)first;
  return ROCMFP4_ERR_INVALID_SCALE;
}

uint32_t rocmfp4_device_error_bits(rocmfp4_stream_t stream) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint32_t bits = 0;
  // The allocating entry points' workspace, only if one exists: the query
  // itself never creates it.
  if (DeviceState* d = existing_state()) {
    if (cudaMemcpyAsync(&bits, d->err, sizeof(bits), cudaMemcpyDeviceToHost, s) != cudaSuccess) return 0xFFFFFFFFu;
    if (cudaStreamSynchronize(s) != cudaSuccess) return 0xFFFFFFFFu;
    if (bits != 0) {
      // A kernel gave up waiting: its split counters may be left set, so clear them.
      cudaMemsetAsync(d->err, 0, sizeof(uint32_t), s);
      cudaMemsetAsync(d->cnt, 0, sizeof(uint32_t) * d->wmax, s);
      cudaMemsetAsync(d->tccnt, 0, sizeof(uint32_t) * tc_cnt_words(d->sms), s);
      cudaMemsetAsync(d->moe_bars, 0, sizeof(uint32_t) * kMoeBarWords, s);
      cudaMemsetAsync(d->paged_cnt, 0, sizeof(uint32_t) * kPagedCtas * d->sms, s);
      if (cudaStreamSynchronize(s) != cudaSuccess) return 0xFFFFFFFFu;
    }
  }
  // The allocation-free entry point's fixed array, if it was set up here.
  uint32_t nb = 0;
  if (noalloc_error_bits(s, &nb) != cudaSuccess) return 0xFFFFFFFFu;
  return bits | nb;
}

const char* rocmfp4_status_string(rocmfp4_status status) {
  switch (status) {
    case ROCMFP4_OK: return "ROCMFP4_OK";
    case ROCMFP4_ERR_INVALID_ARG: return "ROCMFP4_ERR_INVALID_ARG";
    case ROCMFP4_ERR_UNSUPPORTED: return "ROCMFP4_ERR_UNSUPPORTED";
    case ROCMFP4_ERR_INVALID_SCALE: return "ROCMFP4_ERR_INVALID_SCALE";
    case ROCMFP4_ERR_CUDA: return "ROCMFP4_ERR_CUDA";
  }
  return "ROCMFP4_UNKNOWN_STATUS";
}

const char* rocmfp4_last_error(void) { return t_last_error.c_str(); }

uint64_t rocmfp4_launch_count(void) { return g_launches.load(); }

void rocmfp4_shutdown(void) {
  std::lock_guard<std::mutex> lk(g_mu);
  int cur = 0;
  cudaGetDevice(&cur);
  for (int dev = 0; dev < kMaxDevices; ++dev) {
    DeviceState& d = g_dev[dev];
    if (!d.ready) continue;
    cudaSetDevice(dev);
    cudaDeviceSynchronize();
    cudaFree(d.ws);
    cudaFree(d.cnt);
    cudaFree(d.err);
    cudaFree(d.tcws);
    cudaFree(d.tccnt);
    cudaFree(d.attn_ws);
    cudaFree(d.vfirst);
    cudaFree(d.lp_ws);
    cudaFree(d.lp_cnt);
    cudaFree(d.moe_ws);
    cudaFree(d.moe_bars);
    cudaFree(d.paged_ws);
    cudaFree(d.paged_cnt);
    d = DeviceState{};
  }
  cudaSetDevice(cur);
}

}  // extern "C"
