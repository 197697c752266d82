// Host-side launch interface between api.cu and the kernel translation units.
#pragma once
#include <cstdint>
#include <string>
#include <cuda_runtime.h>

#include "moe_layout.h"
#include "paged.h"

namespace rocmfp4 {

// Host-side bookkeeping shared by the C entry points (api.cu).
void set_last_error(const std::string& message);  // text of rocmfp4_last_error()
void count_launch();                              // one more kernel for rocmfp4_launch_count()

// Streaming product Y[M][N] = X[M][K] . W[N][K]^T for M <= 8.
struct GemvArgs {
  const uint8_t* W;      // N x row_bytes packed blocks (2N rows, gate then up, when epi)
  const uint16_t* X;     // M x K activations (fp16 or bf16 bits)
  float* Y;              // M x N outputs
  int64_t N, K, row_bytes;
  int M;
  int64_t nspans;        // K / weights-per-unit
  int64_t units;         // ceil(N/32) * nspans, or ceil(N/16) * nspans when epi
  int64_t wact;          // active warps (<= units)
  float* ws;             // 2 * wact records of 32 x 8 floats
  uint32_t* cnt;         // wact counters, zero between calls
  uint32_t* err;         // error bits
  int epi = 0;           // 1: Y = SiLU(gate rows . x) * (up rows . x)
  int deep = 0;          // 1: deeper per-warp rings, two CTAs per SM (plain products, M <= 2)
};

constexpr int kStreamWarpsPerCta = 4;
constexpr int kStreamTileRows = 32;
int stream_mb_for(int M);                   // staged activation rows: 1, 2, 4 or 8
int stream_weights_per_unit(int variant);   // 256 (dual) or 512 (single-scale)
size_t stream_smem_bytes(int variant, int mb, int deep);
cudaError_t stream_prepare(int variant, int act, int mb);  // sets the dynamic smem attribute
cudaError_t stream_occupancy(int variant, int act, int mb, int* ctas_per_sm);
cudaError_t stream_init_driver();           // resolves cuTensorMapEncodeTiled once
cudaError_t launch_gemv_stream(int variant, int act, const GemvArgs& a, int ctas, cudaStream_t s);
// Active warps of a single-product streaming launch over `tiles` tiles of
// `nspans` units of `unit_bytes` weight bytes, M activation rows, with room
// for `cap` warps (api.cu).
int64_t stream_warps(int64_t tiles, int64_t nspans, int64_t unit_bytes, int64_t M, int64_t cap);
// Error bits of the allocation-free entry point's fixed scratch on the
// current device (noalloc.cu): 0 when it has not been set up there.  Reads
// and clears them, and on a non-zero result zeroes its split counters.
cudaError_t noalloc_error_bits(cudaStream_t s, uint32_t* bits);

// Tensor-core product Y[M][N] = X[M][K] . W[N][K]^T (tcgen05, decoded weights
// in tensor memory).  Needs K % tc_k_multiple(variant) == 0, W and X 16-byte
// aligned, and M, N, K below 2^31.
struct TcArgs {
  const uint8_t* W;
  const uint16_t* X;
  float* Y;
  int64_t M, N, K, row_bytes;
  float* ws;       // split-tile partials: tc_ws_floats(sms) floats
  uint32_t* cnt;   // split-tile counters: tc_cnt_words(sms) words, zero between launches
  uint32_t* err;
};
int tc_k_multiple(int variant);   // 256 (dual) or 512 (single-scale)
size_t tc_ws_floats(int sms);     // one partial tile of 128 x 256 fp32 per SM
size_t tc_cnt_words(int sms);     // one counter per tile of the split region (at most 2 per SM)
cudaError_t tc_prepare();         // resolves cuTensorMapEncodeTiled, sets the smem attributes
cudaError_t launch_gemm_tc(int variant, int act, const TcArgs& a, cudaStream_t s);

// Decode attention over a ROCmFP4 K/V cache (attention.cu): q [B][H][D],
// K and V [B][Hkv][Tmax] rows of D/32 blocks, lens [B], out [B][H][D] fp32.
// D is 64 or 128, H / Hkv at most 8, Tmax a multiple of 32, K and V 16-byte
// aligned.  One split launch, plus a combine launch when the cache is split.
constexpr int kAttnMaxD = 128;
struct AttnArgs {
  const uint16_t* q;
  const uint8_t* K;
  const uint8_t* V;
  const int32_t* lens;
  float* out;
  float* ws;  // attn_ws_floats(sms) floats
  int64_t B, H, Hkv, D, Tmax;
  float scale;
  uint32_t* err;
};
size_t attn_ws_floats(int sms);
cudaError_t attn_prepare();
cudaError_t launch_decode_attention(int variant, int act, const AttnArgs& a, int sms, cudaStream_t s, int* launches);

// Residual addition and RMS norm (norm.cu).  Types are rocmfp4_out_dtype
// values; row strides ld* in elements; y, q and scales are contiguous.
struct NormArgs {
  const void* x;
  const void* residual;  // nullptr: none
  void* residual_out;
  const void* weight;
  void* y;           // nullptr: not wanted
  uint8_t* q;        // nullptr: not wanted
  float* scales;     // M x ceil(D / group), or M when group is 0
  int64_t M, D, ldx, ldr, ldro;
  int x_type, residual_type, weight_type, y_act, group;
  float eps;
  uint32_t* err;
};
int64_t norm_max_width();  // largest D
cudaError_t norm_prepare();  // sets the smem attributes
cudaError_t launch_norm(const NormArgs& a, int sms, cudaStream_t s);

// Log probabilities, entropy and top alternatives of rows of logits (logprobs.cu).
constexpr int kMaxTop = 32;
struct LogprobsArgs {
  const void* logits;
  const int32_t* targets;  // nullptr: none
  float* logprob;          // [M], with targets
  float* entropy;          // [M], nullptr: not wanted
  int32_t* top_ids;        // [M][top_n]
  float* top_logprobs;     // [M][top_n]
  int64_t M, V, ld;
  float scale;
  int type, top_n;
  int splits;              // CTAs that share a row (set by the launch)
  float* ws;               // logprobs_ws_bytes(sms) bytes, 8-byte aligned
  uint32_t* cnt;           // logprobs_cnt_words(sms) words, zero between launches
};
size_t logprobs_ws_bytes(int sms);
size_t logprobs_cnt_words(int sms);
cudaError_t launch_logprobs(const LogprobsArgs& a, int sms, cudaStream_t s);

// Mixture-of-experts layer for M <= kMoeMaxTokens tokens (moe.cu).  X, router,
// Wgu and Wd 16-byte aligned; K and I multiples of 32, at most kMoeMaxWidth;
// E <= kMoeMaxExperts; top_k <= min(E, kMoeMaxTop); M * top_k * I at most
// kMoeMaxHidden.  One cooperative launch of one CTA per SM.
struct MoeArgs {
  const uint16_t* X;   // M x K
  const void* router;  // E x K
  const uint8_t* Wgu;  // E x (I gate rows, I up rows) of K weights
  const uint8_t* Wd;   // E x K rows of I weights
  float* Y;            // M x K
  int32_t* ids;        // M x top_k, nullptr: not wanted
  float* probs;        // M x top_k, nullptr: not wanted
  float* ws;           // kMoeWsFloats floats
  uint32_t* bars;      // kMoeBarWords words, zero between launches
  uint32_t* err;
  int64_t M, E, top_k, K, I;
  int router_type, route;
  float route_scale;
};
cudaError_t moe_prepare();
cudaError_t launch_moe(int variant, int act, const MoeArgs& a, int sms, cudaStream_t s);

// Rotary positions of rows of q, k and v heads; q to fp16 / bf16, k and v into
// the pages (paged.cu).  Without `paged`, q alone, at `positions`.
struct RopeArgs {
  const void* x[3];          // q, k, v: rows of heads of D values
  int64_t ld[3];             // row strides in elements
  const int32_t* positions;  // [M], nullptr: the tokens' places in their sequences
  const float* freq;         // [rot / 2]
  uint16_t* q_out;           // [M][H][D]
  int64_t M, H, D, rot;
  int type, act, interleaved, paged;
  float amplitude;
  PagedArgs cache;
};
cudaError_t launch_rope(int variant, const RopeArgs& a, int sms, cudaStream_t s);

struct CacheReadArgs {
  void* k_out;  // [M][Hkv][D], nullptr: not wanted
  void* v_out;
  int64_t M;
  PagedArgs cache;
};
cudaError_t launch_cache_read(int variant, int type, const CacheReadArgs& a, int sms, cudaStream_t s);

// Attention of rows of queries over the pages of their sequences
// (paged_attention.cu).  D is 64 or 128, page_size a multiple of 16.
struct PagedAttnArgs {
  const uint16_t* q;  // [M] rows of H heads, ldq apart
  int64_t ldq;
  uint16_t* out;      // [M][H][D]
  int64_t M;
  int H, causal, window;
  float scale;
  float* ws;          // paged_attn_ws_floats(sms) floats
  uint32_t* cnt;      // kPagedCtas * sms words, zero between launches
  PagedArgs cache;
};
constexpr int kPagedCtas = 2;  // CTAs an SM of a launch, at most
size_t paged_attn_ws_floats(int sms);
cudaError_t paged_attn_prepare();
// The same for few rows (paged_few.cu).
cudaError_t paged_few_prepare();
cudaError_t launch_paged_few(int variant, int act, const PagedAttnArgs& a, int sms, cudaStream_t s);
cudaError_t launch_paged_attention(int variant, int act, const PagedAttnArgs& a, int sms, cudaStream_t s);

// Any K % 32 == 0, any alignment: one warp per (row, column chunk).
struct GenericArgs {
  const uint8_t* W;
  const uint16_t* X;
  float* Y;
  int64_t N, K, row_bytes;
  int64_t M;
};
cudaError_t launch_gemm_generic(int variant, int act, const GenericArgs& a, cudaStream_t s);

// Dequantisation to fp32 / bf16 / fp16 (out_dtype 0/1/2), flat over blocks.
cudaError_t launch_dequant(int variant, int out_dtype, const uint8_t* W, void* out, int64_t nblocks,
                           cudaStream_t s);

// First block with a non-finite scale byte -> atomicMin into *first (init INT64_MAX).
// Quantiser fp16 / bf16 (act 0 / 1) -> ROCmFP4 blocks, one thread per block
// of 32 consecutive source values.
cudaError_t launch_quantize(int variant, int act, const uint16_t* src, uint8_t* W, int64_t nblocks, cudaStream_t s);
cudaError_t launch_validate(int variant, const uint8_t* W, int64_t nblocks, unsigned long long* first,
                            cudaStream_t s);

// Stream-ordered copy of `bytes` bytes by a kernel (programmatic dependent
// launch); each pointer is device memory or device-addressable host memory.
cudaError_t launch_copy(void* dst, const void* src, int64_t bytes, cudaStream_t s);

}  // namespace rocmfp4
