// Limits of the mixture-of-experts layer, and where its kernel keeps what in
// shared memory and in the workspace.  Plain C++, no CUDA: the sizes can be
// walked through on any machine.
#pragma once
#include <cstddef>
#include <cstdint>

namespace rocmfp4 {

constexpr int kMoeMaxTokens = 32, kMoeMaxExperts = 512, kMoeMaxTop = 16, kMoeMaxWidth = 32768;
constexpr int64_t kMoeMaxHidden = int64_t(1) << 22;  // M * top_k * I
// router logits, activation scales, largest hidden values, hidden values in
// fp32 and as two fp16 parts (rows padded to 512), activations (likewise),
// room for a read past the last
constexpr size_t kMoeWsFloats = (size_t)kMoeMaxTokens * (kMoeMaxExperts + 1 + kMoeMaxTop) + 2 * kMoeMaxHidden +
                                (size_t)kMoeMaxTokens * kMoeMaxTop * 512 + (size_t)kMoeMaxTokens * (kMoeMaxWidth + 512) / 2 + 256;
constexpr int kMoeBarWords = 4;

constexpr int kMoeWarps = 16;
constexpr int kMoeTileRows = 16;
constexpr int kMoeMaxStages = 6;
constexpr int kMoeSmemMax = 227 * 1024 - (kMoeWarps * 640 + 6144);  // dynamic; the rest is the kernel's static shared memory
constexpr int kMoeSlack = 32;                                       // word reads past the last row slot
constexpr int kMoeReadAhead = 1024;                                 // bytes that may be read past the last hidden value

// A span: bytes of a row, and the blocks in them.
constexpr int moe_span_bytes(int variant) { return variant == 0 ? 144 : 272; }
constexpr int moe_span_blocks(int variant) { return variant == 0 ? 8 : 16; }

// A stage of ns spans: aligned rows as ns boxes of 16 rows x one span (36 or 68
// words: rows an odd multiple of 16 bytes apart, whose reads meet no bank
// twice), unaligned ones as 16 slots of ns spans, with room for their place
// within 16 bytes and to end in.
constexpr int moe_row_pitch(int variant, bool aligned, int ns) {
  return aligned ? moe_span_bytes(variant) : ns * moe_span_bytes(variant) + 32;
}

struct MoeLayout {
  // Bytes from the start of dynamic shared memory.  The selection of the
  // experts has its keys and candidates from off_select on, where the outputs,
  // sums and ring come later; the next starts behind select_bytes of it.
  int off_mask, off_list, off_slot, off_unscale, off_y, off_acc, off_ring, off_select, select_bytes;
  int acc_floats;              // a warp's sums of a tile, by group
  int ns, stages, stage_bytes;  // spans of a stage; ring of a warp
  int bytes;                   // of dynamic shared memory
  // Workspace, in floats from its start.
  int64_t ws_logits, ws_unscale, ws_amax, ws_h, ws_x, ws_hi, ws_lo, ws_end;
};

// False where the kernel's shared memory or the workspace would not hold it.
// Sizes within the limits above all fit.
inline bool moe_layout(int variant, bool aligned, int64_t M, int64_t E, int64_t top_k, int64_t K, int64_t I, MoeLayout* l) {
  const auto up = [](int64_t v, int to) { return (int)((v + to - 1) / to * to); };
  l->off_mask = up(M * top_k * 4, 16);
  l->off_list = l->off_mask + up(E * 4, 16);
  l->off_slot = l->off_list + up(E * 2, 16);
  l->off_unscale = l->off_slot + up(M * E, 16);
  l->off_y = l->off_unscale + up(M * 4, 16);
  l->off_acc = l->off_y + kMoeWarps * kMoeTileRows * (int)M * 4;
  l->acc_floats = (int)(M + 3) / 4 * 128;
  l->off_ring = up(l->off_acc + kMoeWarps * l->acc_floats * 4, 128);
  l->ns = variant == 0 ? 2 : 1;
  const int each = aligned ? l->ns * kMoeTileRows * moe_span_bytes(variant) : kMoeTileRows * moe_row_pitch(variant, false, l->ns);
  l->stage_bytes = up(each, 128);
  const int room = (kMoeSmemMax - l->off_ring - kMoeSlack) / (kMoeWarps * l->stage_bytes);
  l->stages = room < kMoeMaxStages ? room : kMoeMaxStages;
  l->bytes = l->off_ring + kMoeWarps * l->stages * l->stage_bytes + kMoeSlack;
  // A warp a token: the order of every expert's logit, 4 bytes, in 8 E bytes,
  // then candidates of 8 bytes.  The ring of many tokens is too small for them
  // (one stage, 68 to 80 KB, against 128 KB for 16 warps and 512 experts); with
  // the outputs and sums in front of it all sizes fit but some of 16 tokens
  // and nearly 512 experts, for which a launch asks for up to 4 KB more.
  l->off_select = l->off_y;
  l->select_bytes = 16 * (int)E;
  const int select_end = l->off_select + (M < kMoeWarps ? (int)M : kMoeWarps) * l->select_bytes;
  if (select_end > l->bytes) l->bytes = select_end;

  const int64_t per = moe_span_blocks(variant), x_span = per * 64, choices = M * top_k;  // bytes of a span's fp16 activations
  const int64_t spans_k = (K / 32 + per - 1) / per, spans_i = (I / 32 + per - 1) / per;
  l->ws_logits = 0;
  l->ws_unscale = l->ws_logits + kMoeMaxTokens * kMoeMaxExperts;
  l->ws_amax = l->ws_unscale + kMoeMaxTokens;
  l->ws_h = l->ws_amax + kMoeMaxTokens * kMoeMaxTop;
  l->ws_x = l->ws_h + choices * I;
  l->ws_hi = l->ws_x + M * spans_k * x_span / 4;
  l->ws_lo = l->ws_hi + choices * spans_i * x_span / 4;
  l->ws_end = l->ws_lo + choices * spans_i * x_span / 4;

  return l->stages >= 1 && l->bytes <= kMoeSmemMax && l->ws_end + kMoeReadAhead / 4 <= (int64_t)kMoeWsFloats;
}

}  // namespace rocmfp4
