// Beam search's selection (gfx950).  Definitions in include/mambascan.h.
//
// Two launches.  The first cuts every beam's logits into slices, one workgroup
// each: a slice is read once into registers and leaves its maximum, the sum of its
// exponentials and its n_out best candidates.  The second, a workgroup per
// sequence, forms the beams' totals from those (in 64 bits: candidates of one
// beam can differ by one unit of a logit near zero while their totals are tens)
// and takes the best.
//
// The best n of many, in either launch: the threads' maxima, the 64 lanes' over
// all waves, give a bound that at least n candidates are not below, and few
// others (with 8192 logits and n = 16 some 20); those go to LDS and are ranked
// there, each by counting what comes before it.  Where more pass than there is room
// for (ties, a sorted row), the bound is raised by bisection first, and among equals
// the place.
#include "beam.hpp"
#include "launch.hpp"
#include "recurrence.hpp"
#include "rows.hpp"

namespace mss {
namespace {

constexpr int kThreadsRow = 256, kWavesRow = kThreadsRow / 64;
constexpr int kThreadsMerge = 512, kWavesMerge = kThreadsMerge / 64;
constexpr int kRoom = 512;     // candidates ranked in LDS
constexpr int kMaxOut = 64;    // n_out

struct Slice {
  double sum;  // of exp(logit - top)
  float top;   // -infinity: no candidate; +infinity: the beam has none
  int count;   // of candidates listed
};

struct BeamArgs {
  BeamSelectParams p;
  Slice* slices;    // [rows][nslices]
  uint64_t* lists;  // [batch][n_out][beams][nslices]: every slice's best, every slice's second, ..
  int nslices;
};

// Sum over the workgroup, in a fixed order; every thread gets it.  `lds` is free
// to be written when the call begins, and again after the next barrier.
template <int WAVES>
__device__ __forceinline__ int block_sum(int v, int* lds) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m, 64);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  int s = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) s += lds[w];
  __syncthreads();
  return s;
}

// VE logits at `at` as loaded; NV vectors a thread.
template <bool BF16, int NV>
struct Logits {
  static constexpr int kVec = BF16 ? 8 : 4;
  static constexpr int kSlice = kThreadsRow * NV * kVec;
  u32x4 raw[NV];
  __device__ __forceinline__ float at(int j, int e) const {
    if constexpr (BF16) return e & 1 ? bf16_hi(raw[j][e >> 1]) : bf16_lo(raw[j][e >> 1]);
    else return __uint_as_float(raw[j][e]);
  }
  static __device__ __forceinline__ int place(int first, int j, int e) {
    return first + (j * kThreadsRow + (int)threadIdx.x) * kVec + e;
  }
  static __device__ __forceinline__ uint64_t key(const void* row, int place) {
    const float v = BF16 ? bf16_to_f32(static_cast<const uint16_t*>(row)[BF16 ? place : 0])
                         : static_cast<const float*>(row)[BF16 ? 0 : place];
    return key_of(ordered_bits(v), (uint32_t)place);
  }
  // Past the row's end: -infinity.
  __device__ __forceinline__ void load(const void* row, int first, int vocab) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int at = place(first, j, 0), n = vocab - at;
      if constexpr (BF16) {
        const uint16_t* p = static_cast<const uint16_t*>(row) + at;
        if (n >= kVec) {
          raw[j] = *reinterpret_cast<const u32x4_a2*>(p);
        } else {
          raw[j] = u32x4{0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u};
#pragma unroll
          for (int e = 0; e < kVec - 1; ++e)
            if (e < n) raw[j][e >> 1] = (raw[j][e >> 1] & (e & 1 ? 0xffffu : 0xffff0000u)) | (uint32_t)p[e] << (16 * (e & 1));
        }
      } else {
        const uint32_t* p = static_cast<const uint32_t*>(row) + at;
        if (n >= kVec) {
          raw[j] = *reinterpret_cast<const u32x4_a4*>(p);
        } else {
#pragma unroll
          for (int e = 0; e < kVec; ++e) raw[j][e] = e < n ? p[e] : 0xff800000u;
        }
      }
    }
  }
};

template <bool BF16, int NV>
__global__ void __launch_bounds__(kThreadsRow) beam_rows_kernel(BeamArgs a) {
  typedef Logits<BF16, NV> L;
  __shared__ float lds_top[kWavesRow][64], lds_sum[kWavesRow];
  __shared__ uint64_t lds_keys[kRoom];
  __shared__ int lds_bad[kWavesRow], lds_count, lds_add[kWavesRow];
  const BeamSelectParams& p = a.p;
  const int64_t row = blockIdx.y;
  if (p.finished != nullptr && p.finished[row] != 0) return;  // its logits are not looked at
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, first = (int)blockIdx.x * L::kSlice;
  const int n = (int)p.n_out;
  const void* base = static_cast<const char*>(p.logits) + row * p.stride * (BF16 ? 2 : 4);
  L l;
  l.load(base, first, (int)p.vocab);

  float top = -__builtin_inff();
  bool fine = true;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < L::kVec; ++e) {
      const float v = l.at(j, e);
      fine = fine && v < __builtin_inff();
      top = fmaxf(top, v);
    }
  lds_top[wave][lane] = top;
  const bool bad = __any(!fine);
  if (lane == 0) lds_bad[wave] = bad;
  if (threadIdx.x == 0) lds_count = 0;
  __syncthreads();
  float group = lds_top[0][lane];
  int anybad = lds_bad[0];
#pragma unroll
  for (int w = 1; w < kWavesRow; ++w) {
    group = fmaxf(group, lds_top[w][lane]);
    anybad |= lds_bad[w];
  }
  float most = group;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) most = fmaxf(most, __shfl_xor(most, m, 64));
  Slice* out = a.slices + row * a.nslices + blockIdx.x;
  if (anybad || most == -__builtin_inff()) {
    if (threadIdx.x == 0) *out = Slice{0.0, anybad ? __builtin_inff() : most, 0};
    return;
  }
  // Sixteen bits of the bound: for bf16 all there are, for fp32 as fine as bf16.
  uint32_t bound = wave_threshold<16>(ordered_bits(group), n);
  if (bound <= kOrderedNegInf) bound = kOrderedNegInf + 1;
  const float least = value_of(bound);

  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float part = 0.0f;
#pragma unroll
    for (int e = 0; e < L::kVec; ++e) part += exp_neg<true>(most - l.at(j, e));
    sum += part;
  }
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) sum += __shfl_xor(sum, m, 64);
  if (lane == 0) lds_sum[wave] = sum;

  // The few that pass are read again: their registers cannot be indexed.
  auto keep = [&](uint32_t mask) {
    for (; mask != 0; mask &= mask - 1) {
      const int i = __builtin_ctz(mask), at = atomicAdd(&lds_count, 1);
      if (at < kRoom) lds_keys[at] = L::key(base, L::place(first, i / L::kVec, i % L::kVec));
    }
  };
  if (top >= least) {
    uint32_t mask = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < L::kVec; ++e) mask |= (l.at(j, e) >= least ? 1u : 0u) << (j * L::kVec + e);
    keep(mask);
  }
  __syncthreads();
  int count = lds_count;
  if (count > kRoom) {
    // A bound that n to kRoom candidates are not below; where equals allow none, the
    // n-th largest value and the place up to which its equals are taken.
    uint32_t exact = 0;
    bool tied = true;
    for (int b = 31; b >= 0 && tied; --b) {
      const uint32_t with = exact | 1u << b;
      int c = 0;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < L::kVec; ++e) c += ordered_bits(l.at(j, e)) >= with;
      c = block_sum<kWavesRow>(c, lds_add);
      if (c >= n) exact = with, tied = c > kRoom;
    }
    int until = L::kSlice;  // past the first place, of what is taken of the equals
    if (tied) {
      int above = 0;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < L::kVec; ++e) above += ordered_bits(l.at(j, e)) > exact;
      above = block_sum<kWavesRow>(above, lds_add);
      until = 0;
      for (int b = 13; b >= 0; --b) {
        const int with = until | 1 << b;
        int c = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int e = 0; e < L::kVec; ++e)
            c += ordered_bits(l.at(j, e)) == exact && L::place(first, j, e) < first + with;
        if (block_sum<kWavesRow>(c, lds_add) < n - above) until = with;
      }
    }
    if (threadIdx.x == 0) lds_count = 0;
    __syncthreads();
    uint32_t mask = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < L::kVec; ++e) {
        const uint32_t o = ordered_bits(l.at(j, e));
        const bool in = o > exact || (o == exact && L::place(first, j, e) <= first + until);
        mask |= (in ? 1u : 0u) << (j * L::kVec + e);
      }
    keep(mask);
    __syncthreads();
    count = lds_count;
  }
  const int64_t seq = row / p.beams, across = p.beams * a.nslices;
  uint64_t* list = a.lists + seq * n * across + (row - seq * p.beams) * a.nslices + blockIdx.x;
  for (int i = threadIdx.x; i < count; i += kThreadsRow) {
    const uint64_t mine = lds_keys[i];
    int rank = 0;
    for (int o = 0; o < count; ++o) rank += lds_keys[o] > mine;
    if (rank < n) list[rank * across] = mine;
  }
  if (threadIdx.x == 0) {
    double s = 0.0;
#pragma unroll
    for (int w = 0; w < kWavesRow; ++w) s += (double)lds_sum[w];
    *out = Slice{s, most, count < n ? count : n};
  }
}

__global__ void __launch_bounds__(kThreadsMerge) beam_merge_kernel(BeamArgs a) {
  // A beam's totals are base + (logit - top), base = score - log sum exp(logit - top);
  // -infinity: no candidates.  (Not base - top + logit: logits may be the type's lowest.)
  __shared__ double lds_base[64];
  __shared__ float lds_most[64];
  __shared__ uint64_t lds_best[kWavesMerge][64], lds_keys[kRoom];
  __shared__ uint32_t lds_places[kRoom], lds_out[kMaxOut];
  __shared__ int lds_count, lds_add[kWavesMerge];
  const BeamSelectParams& p = a.p;
  const int64_t b = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int beams = (int)p.beams, n = (int)p.n_out, vocab = (int)p.vocab;
  const float* scores = p.scores + b * beams;
  const uint8_t* finished = p.finished != nullptr ? p.finished + b * beams : nullptr;
  const Slice* slices = a.slices + b * beams * a.nslices;
  const uint64_t* lists = a.lists + b * beams * a.nslices * n;

  for (int k = wave; k < beams; k += kWavesMerge) {
    const float score = scores[k];
    const bool over = finished != nullptr && finished[k] != 0;
    float top = -__builtin_inff();
    if (!over)
      for (int s = lane; s < a.nslices; s += 64) top = fmaxf(top, slices[k * a.nslices + s].top);
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) top = fmaxf(top, __shfl_xor(top, m, 64));
    double sum = 0.0;
    if (!over && __builtin_fabsf(top) < __builtin_inff())
      for (int s = lane; s < a.nslices; s += 64) {
        const Slice t = slices[k * a.nslices + s];
        if (t.count > 0) sum += t.sum * exp((double)t.top - (double)top);
      }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) sum += __shfl_xor(sum, m, 64);
    const bool none = !(score < __builtin_inff()) || score == -__builtin_inff() ||
                      (!over && !(__builtin_fabsf(top) < __builtin_inff()));
    if (lane == 0) {
      lds_base[k] = none ? -__builtin_inf() : over ? (double)score : (double)score - log(sum);
      lds_most[k] = top;
    }
  }
  if (threadIdx.x == 0) lds_count = 0;
  __syncthreads();

  // The i-th item: its total's ordered bits (kOrderedNegInf64: no candidate) and
  // place.  In the order of the lists, so that neighbouring threads, whose maxima
  // make the bound, look at the same rank of different slices.
  const int across = beams * a.nslices, items = across * n;
  auto item = [&](int i, uint32_t& place) -> uint64_t {
    const int rank = i / across, at = i - rank * across, k = at / a.nslices;
    const double base = lds_base[k];
    place = 0;
    if (base == -__builtin_inf()) return kOrderedNegInf64;
    if (finished != nullptr && finished[k] != 0) {
      place = (uint32_t)k * vocab + (uint32_t)p.eos;
      return rank == 0 && at == k * a.nslices ? ordered_bits(base) : kOrderedNegInf64;
    }
    if (rank >= slices[at].count) return kOrderedNegInf64;
    const uint64_t key = lists[i];
    place = (uint32_t)k * vocab + place_of(key);
    return ordered_bits(base + ((double)value_of((uint32_t)(key >> 32)) - (double)lds_most[k]));
  };
  uint32_t place;
  uint64_t best = kOrderedNegInf64;
  for (int i = threadIdx.x; i < items; i += kThreadsMerge) {
    const uint64_t o = item(i, place);
    best = o > best ? o : best;
  }
  lds_best[wave][lane] = best;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWavesMerge; ++w) best = lds_best[w][lane] > best ? lds_best[w][lane] : best;
  uint64_t bound = wave_threshold<32>(best, n);
  if (bound <= kOrderedNegInf64) bound = kOrderedNegInf64 + 1;
  for (int i = threadIdx.x; i < items; i += kThreadsMerge) {
    const uint64_t o = item(i, place);
    if (o >= bound) {
      const int at = atomicAdd(&lds_count, 1);
      if (at < kRoom) lds_keys[at] = o, lds_places[at] = place;
    }
  }
  __syncthreads();
  int count = lds_count;
  if (count > kRoom) {  // as above
    uint64_t exact = 0;
    bool tied = true;
    for (int bit = 63; bit >= 0 && tied; --bit) {
      const uint64_t with = exact | 1ull << bit;
      int c = 0;
      for (int i = threadIdx.x; i < items; i += kThreadsMerge) c += item(i, place) >= with;
      c = block_sum<kWavesMerge>(c, lds_add);
      if (c >= n) exact = with, tied = c > kRoom;
    }
    uint32_t until = ~0u;
    if (tied) {
      int above = 0;
      for (int i = threadIdx.x; i < items; i += kThreadsMerge) above += item(i, place) > exact;
      above = block_sum<kWavesMerge>(above, lds_add);
      until = 0;
      for (int bit = 30; bit >= 0; --bit) {
        const uint32_t with = until | 1u << bit;
        int c = 0;
        for (int i = threadIdx.x; i < items; i += kThreadsMerge) c += item(i, place) == exact && place < with;
        if (block_sum<kWavesMerge>(c, lds_add) < n - above) until = with;
      }
    }
    if (threadIdx.x == 0) lds_count = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < items; i += kThreadsMerge) {
      const uint64_t o = item(i, place);
      if (o > exact || (o == exact && place <= until)) {
        const int at = atomicAdd(&lds_count, 1);
        if (at < kRoom) lds_keys[at] = o, lds_places[at] = place;
      }
    }
    __syncthreads();
    count = lds_count;
  }
  auto put = [&](int j, float score, uint32_t at) {
    const int64_t o = b * n + j;
    const int parent = (int)(at / (uint32_t)vocab), token = (int)(at - (uint32_t)parent * (uint32_t)vocab);
    p.out_scores[o] = score;
    p.parents[o] = parent;
    p.tokens[o] = token;
    if (p.out_finished != nullptr) p.out_finished[o] = token == p.eos || (finished != nullptr && finished[parent] != 0);
  };
  const int found = count < n ? count : n;
  for (int i = threadIdx.x; i < count; i += kThreadsMerge) {
    const uint64_t mine = lds_keys[i];
    const uint32_t at = lds_places[i];
    int rank = 0;
    for (int o = 0; o < count; ++o) rank += lds_keys[o] > mine || (lds_keys[o] == mine && lds_places[o] < at);
    if (rank < n) put(rank, (float)value_of(mine), at);
    if (rank < n) lds_out[rank] = at;
  }
  if (found == n) return;
  // Fewer candidates than asked for: all are listed, the others follow in order of place.
  __syncthreads();
  if ((int)threadIdx.x < n) {
    int before = 0;
    bool taken = false;
    for (int j = 0; j < found; ++j) {
      before += lds_out[j] < threadIdx.x;
      taken = taken || lds_out[j] == threadIdx.x;
    }
    const int rank = (int)threadIdx.x - before;
    if (!taken && rank < n - found) put(found + rank, -__builtin_inff(), threadIdx.x);
  }
}

// Slices of 8192 logits where they fill the card twice; else of 2048, for the time
// that a workgroup takes for its slice.
constexpr int64_t kWideSlice = 8192, kNarrowSlice = 2048;
bool wide_slices(int64_t rows, int64_t vocab) { return rows * ((vocab + kWideSlice - 1) / kWideSlice) >= 512; }
int64_t slices_of(int64_t rows, int64_t vocab) {
  const int64_t s = wide_slices(rows, vocab) ? kWideSlice : kNarrowSlice;
  return (vocab + s - 1) / s;
}
size_t lists_offset(int64_t rows, int64_t vocab) { return (size_t)(rows * slices_of(rows, vocab)) * sizeof(Slice); }

template <bool BF16, int NV>
void launch_rows(const BeamArgs& a, hipStream_t stream) {
  static_assert(Logits<BF16, NV>::kSlice == kWideSlice || Logits<BF16, NV>::kSlice == kNarrowSlice, "");
  hipLaunchKernelGGL((beam_rows_kernel<BF16, NV>), dim3((unsigned)a.nslices, (unsigned)(a.p.batch * a.p.beams)),
                     dim3(kThreadsRow), 0, stream, a);
}

}  // namespace

size_t beam_select_workspace_bytes(int64_t batch, int64_t beams, int64_t vocab, int64_t n_out) {
  const int64_t rows = batch * beams;
  return lists_offset(rows, vocab) + (size_t)(rows * slices_of(rows, vocab) * n_out) * sizeof(uint64_t);
}

hipError_t launch_beam_select(const BeamSelectParams& p, hipStream_t stream) {
  const int64_t rows = p.batch * p.beams;
  char* ws = static_cast<char*>(p.workspace);
  const BeamArgs a{p, reinterpret_cast<Slice*>(ws), reinterpret_cast<uint64_t*>(ws + lists_offset(rows, p.vocab)),
                   (int)slices_of(rows, p.vocab)};
  const bool wide = wide_slices(rows, p.vocab);
  if (p.bf16) wide ? launch_rows<true, 4>(a, stream) : launch_rows<true, 1>(a, stream);
  else wide ? launch_rows<false, 8>(a, stream) : launch_rows<false, 2>(a, stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(beam_merge_kernel, dim3((unsigned)p.batch), dim3(kThreadsMerge), 0, stream, a);
  return hipGetLastError();
}

}  // namespace mss
