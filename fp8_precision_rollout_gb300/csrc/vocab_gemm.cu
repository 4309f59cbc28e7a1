// vocab_gemm.cu -- the matrix products of the vocabulary operators.
//
//   forward   A = X W^T, reduced in the epilogue to softmax partials;
//   G         the same product, turned into gcoef * (softmax - targets), BF16;
//   dX        G W, FP32 sums over the vocabulary pieces;
//   dW        G^T X.
//
// Plain tiles: 64 x 64 outputs per CTA, 256 threads, 4 x 4 FP32 accumulators
// each, operands staged through shared memory 16 deep.
#include <algorithm>

#include "vocab.h"

namespace fp8rl {
namespace {

constexpr int kT = 64, kD = 16;
constexpr float kLog2e = 1.4426950408889634f;
enum { kStats = 0, kGrad = 1, kDx = 2, kDw = 3 };

struct Operand {
  const __nv_bfloat16* p;
  int64_t ld_mn, ld_k;   // element strides
};

template <int kEpi>
__global__ void __launch_bounds__(256) vocab_gemm_kernel(VocabArgs a, Operand A, Operand B, int v0,
                                                         int vc, int first) {
  __shared__ float sA[kD][kT + 4], sB[kD][kT + 4];
  __shared__ float red[kT][18], ties[kT][16];
  const int n = *a.n_rows;
  const int m0 = blockIdx.y * kT, c0 = blockIdx.x * kT;
  const int M = kEpi == kDw ? vc : n;
  const int N = kEpi == kStats ? a.V : (kEpi == kGrad ? vc : a.H);
  const int K = kEpi == kDx ? vc : (kEpi == kDw ? n : a.H);
  // G keeps zero rows up to its row padding, so every tile of it is written
  if (m0 >= M && kEpi != kGrad) return;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < K; k0 += kD) {
    for (int i = tid; i < kT * kD; i += 256) {
      const int mn = i / kD, k = i % kD;
      sA[k][mn] = (m0 + mn < M && k0 + k < K)
                      ? __bfloat162float(A.p[(m0 + mn) * A.ld_mn + (k0 + k) * A.ld_k]) : 0.0f;
      sB[k][mn] = (c0 + mn < N && k0 + k < K)
                      ? __bfloat162float(B.p[(c0 + mn) * B.ld_mn + (k0 + k) * B.ld_k]) : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kD; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sA[k][ty * 4 + i], sB[k][tx * 4 + j], acc[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i) {
    const int r = m0 + ty * 4 + i;
    if (kEpi == kStats) {
      float mx = -INFINITY;
      for (int j = 0; j < 4; ++j)
        if (c0 + tx * 4 + j < N) mx = fmaxf(mx, acc[i][j]);
      for (int o = 8; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
      float s = 0.0f, cnt = 0.0f;
      for (int j = 0; j < 4; ++j)
        if (c0 + tx * 4 + j < N) {
          if (acc[i][j] == mx)
            cnt += mx == -INFINITY ? 0.0f : 1.0f;
          else
            s += exp2f((acc[i][j] - mx) * (a.scale * kLog2e));
        }
      red[ty * 4 + i][tx] = s;
      ties[ty * 4 + i][tx] = cnt;
      if (tx == 0) red[ty * 4 + i][16] = mx;
    }
    if (r >= n && kEpi != kDw && kEpi != kGrad) continue;
    if (kEpi == kStats || kEpi == kGrad) {
      const bool ok = r < n;
      const int base = kEpi == kStats ? 0 : v0;
      const int64_t tok = (ok && a.K) ? a.map[r] : 0;
      for (int j = 0; j < 4; ++j) {
        const int c = c0 + tx * 4 + j;
        const int v = base + c;
        float q = 0.0f;
        if (kEpi == kGrad && ok && c < N)
          q = exp2f(fmaf(acc[i][j], a.scale * kLog2e, -a.lse[r] * kLog2e));
        if (ok && c < N) {
          if (a.K == 0) {
            if (a.tgt[r] == v) {
              if (kEpi == kStats) a.zt[r] = acc[i][j];
              q -= 1.0f;
            }
          } else {
            for (int k = 0; k < a.K; ++k)
              if (a.ids[tok * a.K + k] == v) {
                if (kEpi == kStats) a.zt[(int64_t)r * a.K + k] = acc[i][j];
                q -= a.p[tok * a.K + k];
              }
          }
        }
        if (kEpi == kGrad && c < a.ldg)
          a.g[(int64_t)r * a.ldg + c] = __float2bfloat16_rn(ok && c < N ? a.gcoef[r] * q : 0.0f);
      }
    } else {
      for (int j = 0; j < 4; ++j) {
        const int c = c0 + tx * 4 + j;
        if (r >= M || c >= N) continue;
        if (kEpi == kDx) {
          float* d = a.dx + (int64_t)r * a.H + c;
          *d = first ? acc[i][j] : *d + acc[i][j];
        } else {
          a.dw[(int64_t)(v0 + r) * a.H + c] = __float2bfloat16_rn(acc[i][j]);
        }
      }
    }
  }
  if (kEpi == kStats) {
    __syncthreads();
    if (tid < kT && m0 + tid < n) {
      float s = 0.0f, cnt = 0.0f;
      for (int j = 0; j < 16; ++j) s += red[tid][j];
      for (int j = 0; j < 16; ++j) cnt += ties[tid][j];
      s += cnt - 1.0f;
      a.part[(int64_t)blockIdx.x * a.rows_pad + m0 + tid] = make_float2(red[tid][16], s);
    }
  }
}

inline unsigned up(int64_t x) { return (unsigned)((x + kT - 1) / kT); }

}  // namespace

fp8rl_status vocab_forward(const VocabArgs& a, const DeviceState*, cudaStream_t stream) {
  const Operand A = {a.x, a.H, 1}, B = {a.w, a.ldw, 1};
  vocab_gemm_kernel<kStats><<<dim3(up(a.V), up(a.rows_cap)), 256, 0, stream>>>(a, A, B, 0, a.V, 0);
  return cuda_check(cudaGetLastError(), "vocab_gemm_kernel launch");
}

fp8rl_status vocab_backward_piece(const VocabArgs& a, int v0, int vc, bool first,
                                  const DeviceState*, cudaStream_t stream) {
  const Operand X = {a.x, a.H, 1}, W = {a.w + (int64_t)v0 * a.ldw, a.ldw, 1};
  vocab_gemm_kernel<kGrad>
      <<<dim3(up(vc), up(a.rows_pad)), 256, 0, stream>>>(a, X, W, v0, vc, 0);
  if (a.dx) {
    const Operand G = {a.g, a.ldg, 1}, Wt = {W.p, 1, a.ldw};
    vocab_gemm_kernel<kDx>
        <<<dim3(up(a.H), up(a.rows_cap)), 256, 0, stream>>>(a, G, Wt, v0, vc, first);
  }
  if (a.dw) {
    const Operand Gt = {a.g, 1, a.ldg}, Xt = {a.x, 1, a.H};
    vocab_gemm_kernel<kDw><<<dim3(up(a.H), up(vc)), 256, 0, stream>>>(a, Gt, Xt, v0, vc, 0);
  }
  return cuda_check(cudaGetLastError(), "vocab_gemm_kernel launch");
}

}  // namespace fp8rl
