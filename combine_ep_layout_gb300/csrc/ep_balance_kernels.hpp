// ep_balance_kernels.hpp -- host-side interface between the C ABI of the router's
// training losses (ep_balance_api.cpp, include/ep_gb300_balance.h) and their kernels.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace epg {

struct BalanceParams {
  const void* logits;       // [n, E], rows row_stride elements apart
  int64_t row_stride;
  const int64_t* idx;       // [n, K]
  int n, experts, topk;
  bool bf16, sigmoid;
  const int32_t* offsets;   // [G + 1] or null: one sequence
  int sequences;            // G
  // forward
  int32_t* counts;          // [G, E]
  float* prob_sums;         // [G, E]
  int32_t* tokens;          // [G + 1]
  float* loss;              // [2]
  // backward
  const int32_t* counts_in;
  const int32_t* tokens_in;
  const float* grad_loss;   // [2]
  void* grad;               // [n, E], rows grad_stride elements apart
  int64_t grad_stride;
  bool accumulate;
  // workspace (BalanceWorkspace): a row of sums for each pair of a block and a sequence
  // that it has tokens of, each final block's part of the losses, the tickets
  float* sums;              // [blocks + G][2 E + 2]
  float* parts;             // [G, column blocks, 2]
  int32_t* ticket;          // [1], zero between launches
  int blocks;               // of the first kernel
  int num_sms;
};

// Experts that one final block adds up.
constexpr int kBalanceColumns = 32;

// Blocks of the first kernel for n tokens, and the workspace's sizes in words.
int BalanceBlocks(int n, int experts, int num_sms);
inline size_t BalanceSumWords(int blocks, int sequences, int experts) {
  return (static_cast<size_t>(blocks) + sequences) * (2 * static_cast<size_t>(experts) + 2);
}
inline size_t BalancePartWords(int sequences, int experts) {
  return static_cast<size_t>(sequences) * ((experts + kBalanceColumns - 1) / kBalanceColumns) * 2;
}

// Whether the first kernel's one block does everything.
inline bool BalanceAlone(const BalanceParams& p) { return p.n > 0 && p.blocks == 1 && p.sequences == 1; }

cudaError_t LaunchBalance(const BalanceParams& p, cudaStream_t s);
cudaError_t LaunchBalanceBackward(const BalanceParams& p, cudaStream_t s);

}  // namespace epg
