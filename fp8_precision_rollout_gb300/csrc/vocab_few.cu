// vocab_few.cu -- softmax partials and target logits of one row or two: the
// log-probability of a token that has just been sampled.
//
// The work is one read of the vocabulary weights (2 V H bytes; 1.07 GB and 158
// us at 131072 x 4096 and the measured 6.79 TB/s) with 2 n FLOP per weight; it
// takes 159 us.
// Plain FP32 FMAs keep up with it (packed pairs, 64 in sequence, then a tree),
// and their sums are exact enough for a single nearly certain token, whose
// log-probability's relative error is its logit's absolute one.
//
// A CTA of 16 warps per SM holds the rows as FP32 in shared memory (two planes
// of float4, so that a warp's 16-byte reads are conflict-free).  Each warp takes
// a contiguous range of the vocabulary, four weights rows at a time: a lane
// loads 16 bytes of each, converts them once and uses them for all n rows,
// reading the rows' values once for the four.  The 4 n sums are reduced by
// halving (a lane ends with one of them), so the softmax's exponentials and the
// search for targets run on all lanes at once; each lane keeps a running
// (maximum, sum) of its own stream, joined at the end.
#include <algorithm>
#include <climits>
#include <mutex>

#include "sm100_ptx.cuh"
#include "vocab.h"

namespace fp8rl {
namespace {

constexpr int kWarps = 16, kThreads = kWarps * 32, kRows = 4;
constexpr int kMaxK = 256;

__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
  return (uint64_t)lo | ((uint64_t)hi << 32);
}
// Both halves: an IEEE FP32 FMA each.
__device__ __forceinline__ void fma2(uint64_t& acc, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(a), "l"(b));
}
__device__ __forceinline__ uint4 load_once(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <int NT>
__global__ void __launch_bounds__(kThreads, 1) few_kernel(const VocabArgs a) {
  extern __shared__ ulonglong2 xs[];      // [NT][2 planes][H / 8]: 4 floats each
  __shared__ int32_t sids[NT][kMaxK];
  __shared__ float wm[kWarps][NT], wr[kWarps][NT];
  ptx::grid_dependency_wait();
  ptx::grid_dependents_launch();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = min(*a.n_rows, NT);
  const int vecs = a.H / 8, K = max(a.K, 1);
  for (int i = tid; i < NT * vecs; i += kThreads) {
    const int t = i / vecs, c = i - t * vecs;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (t < n) v = reinterpret_cast<const uint4*>(a.x + (int64_t)t * a.ldx)[c];
    xs[(t * 2) * vecs + c] = make_ulonglong2(pack2(v.x << 16, v.x & 0xFFFF0000u), pack2(v.y << 16, v.y & 0xFFFF0000u));
    xs[(t * 2 + 1) * vecs + c] = make_ulonglong2(pack2(v.z << 16, v.z & 0xFFFF0000u), pack2(v.w << 16, v.w & 0xFFFF0000u));
  }
  for (int i = tid; i < n * K; i += kThreads) {
    const int t = i / K, k = i - t * K;
    sids[t][k] = a.K ? a.ids[(int64_t)a.map[t] * K + k] : a.tgt[t];
  }
  __syncthreads();

  // this lane's sum after the halving: token lt, weights row lr of the four
  constexpr int kSums = NT * kRows, kDup = 32 / kSums;
  const int lt = (lane / kDup) / kRows, lr = (lane / kDup) % kRows;
  const bool mine = lt < n;
  const float k2 = a.scale * 1.4426950408889634f;
  float m = -INFINITY, r = -1.0f;
  int cur = 0;
  const int64_t w = (int64_t)blockIdx.x * kWarps + warp, nw = (int64_t)gridDim.x * kWarps;
  const int v0 = (int)(a.V * w / nw), v1 = (int)(a.V * (w + 1) / nw);
  for (int v = v0; v < v1; v += kRows) {
    uint64_t acc[NT][kRows];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < kRows; ++i) acc[t][i] = 0;
    const uint4* wp[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i)      // (past the range: the last row again, not used)
      wp[i] = reinterpret_cast<const uint4*>(a.w + (int64_t)min(v + i, v1 - 1) * a.ldw);
#pragma unroll 2
    for (int c = lane; c < vecs; c += 32) {
      uint4 q[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) q[i] = load_once(wp[i] + c);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint64_t f[kRows][2];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const uint32_t x = half ? q[i].z : q[i].x, y = half ? q[i].w : q[i].y;
          f[i][0] = pack2(x << 16, x & 0xFFFF0000u);
          f[i][1] = pack2(y << 16, y & 0xFFFF0000u);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const ulonglong2 h = xs[(t * 2 + half) * vecs + c];
#pragma unroll
          for (int i = 0; i < kRows; ++i) {
            fma2(acc[t][i], f[i][0], h.x);
            fma2(acc[t][i], f[i][1], h.y);
          }
        }
      }
    }
    float z[kSums];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < kRows; ++i)
        z[t * kRows + i] = __uint_as_float((uint32_t)acc[t][i]) + __uint_as_float((uint32_t)(acc[t][i] >> 32));
#pragma unroll
    for (int o = 16, left = kSums; o; o >>= 1) {
      if (left > 1) {
        left >>= 1;
#pragma unroll
        for (int i = 0; i < left; ++i) {
          const float keep = (lane & o) ? z[i + left] : z[i], give = (lane & o) ? z[i] : z[i + left];
          z[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, o);
        }
      } else {
        z[0] += __shfl_xor_sync(0xFFFFFFFFu, z[0], o);
      }
    }
    const int row = v + lr;
    if (mine && row < v1) {
      vocab_join(m, r, z[0], z[0] == -INFINITY ? -1.0f : 0.0f, k2);
      while (cur < K && sids[lt][cur] < row) ++cur;
      for (; cur < K && sids[lt][cur] == row; ++cur)
        if (lane % kDup == 0) a.zt[(int64_t)lt * K + cur] = z[0];
    }
    __syncwarp();
  }
  // the four streams of a token, then the warps'
#pragma unroll
  for (int o = kDup; o < kDup * kRows; o <<= 1) {
    const float m2 = __shfl_xor_sync(0xFFFFFFFFu, m, o), r2 = __shfl_xor_sync(0xFFFFFFFFu, r, o);
    vocab_join(m, r, m2, r2, k2);
  }
  if (lr == 0 && lane % kDup == 0) {
    wm[warp][lt] = m;
    wr[warp][lt] = r;
  }
  __syncthreads();
  if (tid < n) {
    m = wm[0][tid];
    r = wr[0][tid];
    for (int i = 1; i < kWarps; ++i) vocab_join(m, r, wm[i][tid], wr[i][tid], k2);
    a.part[(int64_t)blockIdx.x * a.rows_pad + tid] = make_float2(m, r);
  }
}

template <int NT>
fp8rl_status launch_few(const VocabArgs& a, const DeviceState* ds, cudaStream_t stream) {
  static bool done[64] = {false};
  static std::mutex mu;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!done[ds->device & 63]) {
      const fp8rl_status st = cuda_check(
          cudaFuncSetAttribute(few_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kVocabFewBytes),
          "cudaFuncSetAttribute(few)");
      if (st != FP8RL_OK) return st;
      done[ds->device & 63] = true;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ds->sm_count);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)NT * a.H * 4;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_check(cudaLaunchKernelEx(&cfg, few_kernel<NT>, a), "few_kernel launch");
}

}  // namespace

fp8rl_status vocab_forward_few(const VocabArgs& a, const DeviceState* ds, cudaStream_t stream) {
  return a.rows_cap == 1 ? launch_few<1>(a, ds, stream) : launch_few<2>(a, ds, stream);
}

}  // namespace fp8rl
