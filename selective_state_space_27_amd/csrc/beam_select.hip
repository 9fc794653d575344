// Beam search's selection (gfx950).  Definitions in include/mambascan.h.
//
// Two launches: every beam's best candidates (its logits in order, with the
// log of the sum of their exponentials), then the best of a sequence's beams.
// Totals are in 64 bits: candidates of one beam can differ by one unit of an
// fp32 logit near zero while their totals are tens.
#include "beam.hpp"
#include "launch.hpp"

namespace mss {
namespace {

constexpr int kThreadsBeam = 256;

template <typename T, typename F>
__device__ __forceinline__ T reduce(T v, T* lds, F&& f) {
  for (int m = 1; m < 64; m <<= 1) v = f(v, (T)__shfl_xor(v, m, 64));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  T r = lds[0];
  for (int w = 1; w < kThreadsBeam / 64; ++w) r = f(r, lds[w]);
  return r;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreadsBeam) beam_rows_kernel(BeamSelectParams p, Candidate* out) {
  __shared__ double dlds[4];
  __shared__ float flds[4];
  __shared__ unsigned long long klds[4];
  __shared__ int ilds[4];
  const int64_t row = blockIdx.x;
  const int vocab = (int)p.vocab, n = (int)(p.n_out < p.vocab ? p.n_out : p.vocab);
  Candidate* mine = out + row * p.n_out;
  const int64_t first = row % p.beams * p.vocab;
  const float score = p.scores[row];
  const bool valid = score < __builtin_inff();
  if (p.finished != nullptr && p.finished[row] != 0) {
    for (int j = threadIdx.x; j < n; j += kThreadsBeam) {
      const int64_t token = j == 0 ? p.eos : j - 1 < p.eos ? j - 1 : j;
      mine[j] = {j == 0 && valid ? (double)score : -__builtin_inf(), first + token};
    }
    return;
  }
  auto at = [&](int v) {
    if constexpr (BF16) return bf16_to_f32(static_cast<const uint16_t*>(p.logits)[row * p.stride + v]);
    else return static_cast<const float*>(p.logits)[row * p.stride + v];
  };
  float top = -__builtin_inff();
  int bad = 0;
  for (int v = threadIdx.x; v < vocab; v += kThreadsBeam) {
    const float l = at(v);
    bad |= !(l < __builtin_inff());
    top = fmaxf(top, l);
  }
  top = reduce(top, flds, [](float a, float b) { return fmaxf(a, b); });
  bad = reduce(bad, ilds, [](int a, int b) { return a | b; });
  if (bad || !valid || score == -__builtin_inff() || top == -__builtin_inff()) {  // no candidate: places in order
    for (int j = threadIdx.x; j < n; j += kThreadsBeam) mine[j] = {-__builtin_inf(), first + j};
    return;
  }
  double sum = 0.0;
  for (int v = threadIdx.x; v < vocab; v += kThreadsBeam) sum += (double)expf(at(v) - top);
  sum = reduce(sum, dlds, [](double a, double b) { return a + b; });
  const double lse = (double)top + log(sum);
  unsigned long long last = ~0ull;
  for (int j = 0; j < n; ++j) {
    unsigned long long best = 0;
    for (int v = threadIdx.x; v < vocab; v += kThreadsBeam) {
      const unsigned long long k = key_of(at(v), (uint32_t)v);
      if (k < last && k > best) best = k;
    }
    last = reduce(best, klds, [](unsigned long long a, unsigned long long b) { return a > b ? a : b; });
    if (threadIdx.x == 0)
      mine[j] = {(double)score + ((double)value_of((uint32_t)(last >> 32)) - lse), first + place_of(last)};
  }
}

__global__ void __launch_bounds__(kThreadsBeam) beam_merge_kernel(BeamSelectParams p, const Candidate* in) {
  __shared__ Candidate lds[kThreadsBeam];
  const int64_t b = blockIdx.x;
  const int per = (int)(p.n_out < p.vocab ? p.n_out : p.vocab), total = per * (int)p.beams;
  const Candidate* mine = in + b * p.beams * p.n_out;
  Candidate last = {__builtin_inf(), -1};
  for (int j = 0; j < (int)p.n_out; ++j) {
    Candidate best = {-__builtin_inf(), INT64_MAX};
    for (int i = threadIdx.x; i < total; i += kThreadsBeam) {
      const Candidate c = mine[(int64_t)(i / per) * p.n_out + i % per];
      if (before(last, c) && before(c, best)) best = c;
    }
    lds[threadIdx.x] = best;
    __syncthreads();
    for (int h = kThreadsBeam / 2; h > 0; h >>= 1) {
      if ((int)threadIdx.x < h && before(lds[threadIdx.x + h], lds[threadIdx.x]))
        lds[threadIdx.x] = lds[threadIdx.x + h];
      __syncthreads();
    }
    last = lds[0];
    __syncthreads();
    if (threadIdx.x == 0) {
      const int64_t o = b * p.n_out + j, parent = last.place / p.vocab, token = last.place - parent * p.vocab;
      p.out_scores[o] = (float)last.total;
      p.parents[o] = parent;
      p.tokens[o] = token;
      if (p.out_finished != nullptr)
        p.out_finished[o] = token == p.eos || (p.finished != nullptr && p.finished[b * p.beams + parent] != 0);
    }
  }
}

}  // namespace

size_t beam_select_workspace_bytes(int64_t batch, int64_t beams, int64_t, int64_t n_out) {
  return (size_t)(batch * beams * n_out) * sizeof(Candidate);
}

hipError_t launch_beam_select(const BeamSelectParams& p, hipStream_t stream) {
  Candidate* cand = static_cast<Candidate*>(p.workspace);
  const dim3 rows((unsigned)(p.batch * p.beams));
  if (p.bf16) hipLaunchKernelGGL(beam_rows_kernel<true>, rows, dim3(kThreadsBeam), 0, stream, p, cand);
  else hipLaunchKernelGGL(beam_rows_kernel<false>, rows, dim3(kThreadsBeam), 0, stream, p, cand);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(beam_merge_kernel, dim3((unsigned)p.batch), dim3(kThreadsBeam), 0, stream, p, cand);
  return hipGetLastError();
}

}  // namespace mss
