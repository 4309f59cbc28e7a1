// vocab.h -- what the vocabulary operators' two translation units share:
// vocab.cu (argument checks, row packing, reductions) and vocab_gemm.cu (the
// matrix products over the vocabulary and their epilogues).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"

namespace fp8rl {

// Columns of the vocabulary that one softmax partial covers.
constexpr int kVocabPart = 128;
// Row counts, and pieces of the vocabulary, are padded to this in the
// workspace: the tile's rows and columns.
constexpr int kVocabPad = 256;

// One call's operands on the packed rows: row c of `x` is the hidden state of
// token map[c]; tokens without a target are not in it.  n_rows (device) is
// their number, at most rows_cap.
struct VocabArgs {
  const __nv_bfloat16* x;   // [rows_pad, H]
  const __nv_bfloat16* w;   // [V, H], row stride ldw
  int64_t ldw;
  int H, V;
  int rows_cap, rows_pad;
  const int32_t* n_rows;
  const int32_t* map;       // [rows_pad] token of each packed row
  float scale;              // logits = scale * x w^T
  // sparse target distribution: K = 0, one target tgt[c] of probability 1;
  // K > 0, entries ids/p[map[c] * K + j], ids ascending, absent ones INT_MAX
  const int32_t* tgt;
  const int32_t* ids;
  const float* p;
  int K;
  // forward: per (column part, row) the maximum of x w^T and the sum of
  // exp(scale * (x w^T - maximum)) less 1, the maximum's own term ((-inf, -1)
  // for nothing); the entries' x w^T ([row] or [row, K])
  float2* part;             // [ceil(V / kVocabPart), rows_pad]
  float* zt;
  // backward: log-sum-exp and signed, scaled upstream gradient of each row;
  // G = gcoef * (softmax - target distribution)
  const float* lse;
  const float* gcoef;
  __nv_bfloat16* g[2];      // [rows_pad, vc] each: alternating pieces of G
  int vc;                   // columns of a piece, a multiple of kVocabPad
  int slices;               // dX: sums over this many parts of a piece
  float* dx;                // [slices, rows_pad, H] FP32, or null
  __nv_bfloat16* dw;        // [V, H], or null
  uint32_t* status;
};

// Softmax partials and target logits of every row over the whole vocabulary.
fp8rl_status vocab_forward(const VocabArgs& a, const DeviceState* ds, cudaStream_t stream);
// G, dx (per slice) and dw over the whole vocabulary, piece by piece.
fp8rl_status vocab_backward(const VocabArgs& a, const DeviceState* ds, cudaStream_t stream);
// Slices that give the dX product of `rows` x H enough tiles to fill the GPU.
int vocab_dx_slices(int64_t rows, int64_t H, int64_t vc);

}  // namespace fp8rl
