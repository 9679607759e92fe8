// The one-kernel layer for a few tokens: what its host side and its kernel share.
#pragma once

#include "moe_internal.h"

namespace moe {

constexpr int kFewMaxT = 8;
constexpr int kFewMaxSlots = kFewMaxT * 16 + 1;  // touched experts: at most T * top_k, and the shared one

// Counters of a handle, all zero between calls.
constexpr int kFewScoresDone = 0;                          // blocks whose router scores are written
constexpr int kFewBlocksDone = 1;                          // blocks that have ended
constexpr int kFewSlotDone = 2;                            // [slot] h blocks written
constexpr int kFewColsDone = kFewSlotDone + kFewMaxSlots;  // [d / 64][T] expert rows written in these columns
inline __host__ __device__ int few_counters(int d) { return kFewColsDone + d / 64 * kFewMaxT; }

struct FewArgs {
  const __nv_bfloat16* x;   // [T, d]
  const float* router_w;    // [E, d], NULL on a hash layer
  const float* bias;        // [E]
  const int32_t* tok;       // [T] (hash layer)
  const int32_t* table;     // [V, k]
  float* scores;            // [T, E] sqrt(softplus(logit))
  uint8_t* h;               // [T, k + 1, f] E4M3 codes
  uint8_t* h_s;             // [T, k + 1, f / 32]
  float* rows;              // [T, k + 1, d] weighted expert rows
  int* counters;
  int32_t* ws_ids;
  float* ws_w;
  int32_t* out_ids;         // may be NULL
  float* out_w;             // may be NULL
  __nv_bfloat16* out;       // [T, d]
  int* status;
  uint64_t budget_ns;
  int T, d, f, E, k, V, has_shared, stages;
  int red_shift;            // buffers of partial products: 2 (1) or 1 (0)
  int stall;                // issue no weight copies (moe_testing_stall_loads)
  float route_scale, limit;
};

// Stages of the weight ring that fit beside T rows of d columns; 0 if too few.
int few_stages(int T, int d, int* red_shift = nullptr);

// Tensor maps of one expert set for this kernel: a copy brings the K groups kg .. kg + 3 of 64 weight rows.
//   w13   {64 B, 128 rows, gate / up, f / 128, experts * d / 128}, box {64, 32, 2, 1, 4}, 64-byte swizzle
//   w2    {64 B, 256 rows, d / 256, experts * f / 128}, box {64, 64, 1, 4}, 64-byte swizzle
//   sf13  {128 words, gate / up, f / 128, experts * d / 128}, box {128, 2, 1, 4}
//   sf2   {128 words, row half, d / 256, experts * f / 128}, box {128, 1, 1, 4}
struct FewMaps {
  CUtensorMap w13, w2, sf13, sf2;
};
cudaError_t launch_few_tokens(const FewMaps& routed, const FewMaps& shared, FewArgs a, int num_sms, cudaStream_t s);

}  // namespace moe
