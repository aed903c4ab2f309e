// gate.h -- launchers of the router's gate and balance loss (include/muon_block.h).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace muon {

constexpr int kGateMaxExperts = 1024;

struct GateArgs {
  const void* logits;      // [tokens][experts], rows ldz apart
  const uint8_t* mask;     // null, or a token's share in the batch (0: none)
  float* weights;          // [tokens][top]
  int32_t* ids;
  const float* dweights;   // gradient
  void* dlogits;           // contiguous
  int64_t tokens, ldz;
  int32_t experts, top, normalize;
};
hipError_t launch_gate(const GateArgs& a, int dtype, hipStream_t s);
hipError_t launch_gate_grad(const GateArgs& a, int dtype, hipStream_t s);

struct BalanceArgs {
  const void* logits;
  const uint8_t* mask;
  const void* ids;         // [tokens][top]
  float* loss;
  int32_t* counts;         // [experts]
  float* shares;           // [experts + 1]: c_e / (T top), then experts / T
  float* part;             // workspace [blocks][experts]: sums of probabilities
  int32_t* part_counts;    // [blocks][experts + 1]: counts, and the block's tokens
  const float* dloss;      // gradient
  void* dlogits;
  int64_t tokens, ldz;
  int32_t experts, top, ids64;
};
int balance_blocks(int64_t tokens, int experts);
hipError_t launch_balance(const BalanceArgs& a, int dtype, hipStream_t s);
hipError_t launch_balance_grad(const BalanceArgs& a, int dtype, hipStream_t s);

}  // namespace muon
