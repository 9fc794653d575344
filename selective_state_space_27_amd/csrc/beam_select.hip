// Beam search's selection (gfx950).  Definitions in include/mambascan.h.
//
// Two launches.  The first cuts every beam's logits into slices, one workgroup
// each: a slice is read once into registers and leaves its maximum, the sum of its
// exponentials and its n_out best candidates.  The second, a workgroup per
// sequence, forms the beams' totals from those (in 64 bits: candidates of one
// beam can differ by one unit of a logit near zero while their totals are tens)
// and takes the best; of equal totals the lower beam's, in a beam the larger logit's
// (tiny logits may differ where 64 bits of a total do not), then the lower token's.
//
// The best n of many, in either launch: the maxima of groups of threads give a bound
// that at least n candidates are not below, and few others (with 8192 logits and n =
// 16 some 20); those go to LDS and are ranked there, each by counting what comes
// before it.  Where more pass than there is room for (ties, a sorted row), the bound is
// raised first, bit by bit where need be.
//
// 32 x 8 x 50277 bf16 (25.7 MB): 10 us the slices, 7 us the merge (all logits equal: 33
// in all); 8 x 16 x 250001 fp32 (128 MB), n = 32: 27 us and 12 us (110).  The first is
// bound by memory where logits are many (4.8 TB/s), else by the latency of its steps,
// as the second always is.
#include "beam.hpp"
#include "launch.hpp"
#include "recurrence.hpp"
#include "rows.hpp"

namespace mss {
namespace {

constexpr int kThreadsRow = 256, kWavesRow = kThreadsRow / 64;
constexpr int kHeld = 16;      // totals a thread of the merge holds
// Candidates ranked in LDS; more are narrowed down first (which takes as long as
// ranking about as many).
constexpr int kRoom = 512, kRoomMerge = 1024;
constexpr int kMaxOut = 64;    // n_out

// What decides between equal totals, larger first: 6 bits of the beam, the logit, 24 of
// the token.
__device__ __forceinline__ uint64_t second_of(int beam, uint64_t key) {
  return (uint64_t)(63 - beam) << 56 | (key >> 32) << 24 | (0xffffffu - place_of(key));
}
__device__ __forceinline__ uint32_t place_of_second(uint64_t second, int vocab) {
  return (63 - (uint32_t)(second >> 56)) * (uint32_t)vocab + (0xffffffu - ((uint32_t)second & 0xffffffu));
}

struct Slice {
  double sum;  // of exp(logit - top)
  float top;   // -infinity: no candidate; +infinity: the beam has none
  int count;   // of candidates listed
};

constexpr size_t kHeader = 16;  // of the workspace: the status word, which nothing sets

struct BeamArgs {
  BeamSelectParams p;
  Slice* slices;    // [rows][nslices]
  uint64_t* lists;  // [batch][n_out][beams][nslices]: every slice's best, every slice's second, ..
  int nslices;
};

// Maximum over the wave's lanes, which every one of them gets.
__device__ __forceinline__ float lanes_max(float v) {
  v = fmaxf(v, dpp_f32<kDppXor1>(v));
  v = fmaxf(v, dpp_f32<kDppXor2>(v));
  v = fmaxf(v, dpp_f32<kDppHalfMirror>(v));
  v = fmaxf(v, dpp_f32<kDppMirror>(v));
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1]));
}

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

// Sum over the threads before this one, and over all; `lds` as there.
template <int WAVES>
__device__ __forceinline__ int block_before(int v, int* lds, int& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int s = v;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const int t = __shfl_up(s, m, 64);
    s += lane >= m ? t : 0;
  }
  if (lane == 63) lds[wave] = s;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    before += w < wave ? lds[w] : 0;
    total += lds[w];
  }
  __syncthreads();
  return before + s - v;
}

// VE logits at `at` as loaded; NV vectors a thread.
template <bool BF16, int NV>
struct Logits {
  static constexpr int kVec = BF16 ? 8 : 4;
  static constexpr int kSlice = kThreadsRow * NV * kVec;
  u32x4 raw[NV];
  static __device__ __forceinline__ float value(u32x4 v, int e) {
    if constexpr (BF16) return e & 1 ? bf16_hi(v[e >> 1]) : bf16_lo(v[e >> 1]);
    else return __uint_as_float(v[e]);
  }
  __device__ __forceinline__ float at(int j, int e) const { return value(raw[j], e); }
  static __device__ __forceinline__ int place(int first, int j, int e) {
    return first + (j * kThreadsRow + (int)threadIdx.x) * kVec + e;
  }
  // From `at` on; past the row's end: -infinity.
  static __device__ __forceinline__ u32x4 load(const void* row, int at, int vocab) {
    const int n = vocab - at;
    u32x4 v;
    if constexpr (BF16) {
      const uint16_t* p = static_cast<const uint16_t*>(row) + at;
      if (n >= kVec) {
        v = *reinterpret_cast<const u32x4_a2*>(p);
      } else {
        v = u32x4{0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u};
#pragma unroll
        for (int e = 0; e < kVec - 1; ++e)
          if (e < n) v[e >> 1] = (v[e >> 1] & (e & 1 ? 0xffffu : 0xffff0000u)) | (uint32_t)p[e] << (16 * (e & 1));
      }
    } else {
      const uint32_t* p = static_cast<const uint32_t*>(row) + at;
      if (n >= kVec) {
        v = *reinterpret_cast<const u32x4_a4*>(p);
      } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e) v[e] = e < n ? p[e] : 0xff800000u;
      }
    }
    return v;
  }
  // f(ordered bits) of every logit of the thread, read again.
  template <class F>
  static __device__ __forceinline__ void again(const void* row, int first, int vocab, F f) {
#pragma unroll 1
    for (int j = 0; j < NV; ++j) {
      const u32x4 v = load(row, place(first, j, 0), vocab);
#pragma unroll
      for (int e = 0; e < kVec; ++e) f(ordered_bits(value(v, e)));
    }
  }
};

template <bool BF16, int NV>
__global__ void __launch_bounds__(kThreadsRow) beam_rows_kernel(BeamArgs a) {
  typedef Logits<BF16, NV> L;
  __shared__ uint32_t lds_top[kWavesRow][64];  // ordered bits
  __shared__ float lds_sum[kWavesRow];
  __shared__ uint64_t lds_keys[kRoom];
  __shared__ int lds_count, lds_add[kWavesRow];
  const BeamSelectParams& p = a.p;
  // A row's slices side by side (as the grid's axes, rows first, 32 x 8 x 50277 took 18.0
  // us instead of 16.1).
  const uint32_t slice = blockIdx.x % (uint32_t)a.nslices;
  const int64_t row = blockIdx.x / (uint32_t)a.nslices;
  if (blockIdx.x == 0 && threadIdx.x == 0) *static_cast<int*>(a.p.workspace) = 0;
  if (p.finished != nullptr && p.finished[row] != 0) return;  // its logits are not looked at
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, first = (int)slice * L::kSlice;
  const int n = (int)p.n_out;
  const void* base = static_cast<const char*>(p.logits) + row * p.stride * (BF16 ? 2 : 4);
  L l;
#pragma unroll
  for (int j = 0; j < NV; ++j) l.raw[j] = L::load(base, L::place(first, j, 0), (int)p.vocab);

  float top = -__builtin_inff();
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < L::kVec; ++e) top = fmaxf(top, l.at(j, e));
  lds_top[wave][lane] = ordered_bits(top);
  if (threadIdx.x == 0) lds_count = 0;
  __syncthreads();
  uint32_t group = lds_top[0][lane];
#pragma unroll
  for (int w = 1; w < kWavesRow; ++w) group = max(group, lds_top[w][lane]);
  const float most = lanes_max(value_of(group));
  Slice* out = a.slices + row * a.nslices + slice;
  // (Where there is a NaN beside infinities the sum below shows it.)
  if (most == __builtin_inff()) {
    if (threadIdx.x == 0) *out = Slice{0.0, most, 0};
    return;
  }
  // Sixteen bits of the bound: for bf16 all there are, for fp32 as fine as bf16.
  uint32_t bound = lds_threshold<16, kWavesRow>(lds_top, n > kLanesEnough, n);
  if (bound <= kOrderedNegInf) bound = kOrderedNegInf + 1;
  const float least = value_of(bound);

  // A slice of nothing but -infinity: terms of exp(-(lowest - -infinity)) = 0.
  const float from = fmaxf(most, -3.4028235e38f);
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float part = 0.0f;
#pragma unroll
    for (int e = 0; e < L::kVec; ++e) part += exp_neg<!BF16>(from - l.at(j, e));
    sum += part;
  }
  sum = lanes_sum<64>(sum);
  if (lane == 0) lds_sum[wave] = sum;

  // Few pass.
  auto keep = [&](uint32_t ordered, int place) {
    const int at = atomicAdd(&lds_count, 1);
    if (at < kRoom) lds_keys[at] = key_of(ordered, (uint32_t)place);
  };
  if (top >= least) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < L::kVec; ++e)
        if (l.at(j, e) >= least) keep(ordered_bits(l.at(j, e)), L::place(first, j, e));
  }
  __syncthreads();
  int count = lds_count;
  if (count > kRoom) {
    // Mostly many equal the bound, and fewer than n are above it: it is the n-th largest.
    // Else a bound that n to kRoom candidates are not below, or, where equals allow
    // none, the n-th largest.  Of its equals the first are taken.  The logits are read
    // again, from the caches: kept in registers for this they would take half of the
    // waves' room (8 x 16 x 250001 fp32: 40.3 us, so 38.2).
    const auto all = [&](auto f) { L::again(base, first, (int)p.vocab, f); };
    const auto number = [&](auto f) {
      int c = 0;
      all([&](uint32_t o) { c += f(o); });
      return block_sum<kWavesRow>(c, lds_add);
    };
    // (A negative bf16's ordered bits end in ones.)
    const auto whole = [](uint32_t o) { return BF16 && !(o >> 31) ? o | 0xffffu : o; };
    uint32_t exact = whole(bound);
    int above = number([&](uint32_t o) { return o > exact; });
    if (above >= n) {
      const bool high = BF16 || number([&](uint32_t o) { return o > (bound | 0xffffu); }) >= n;
      if (high) exact = 0;
      bool tied = true;
      for (int b = high ? 31 : 15; b >= (BF16 ? 16 : 0) && tied; --b) {
        const uint32_t with = exact | 1u << b;
        const int c = number([&](uint32_t o) { return o >= with; });
        if (c >= n) exact = with, tied = c > kRoom;
      }
      exact = whole(exact);
      if (tied) above = number([&](uint32_t o) { return o > exact; });
      else exact -= 1, above = n;  // none of its equals apart from the others
    }
    if (threadIdx.x == 0) lds_count = 0;
    __syncthreads();
    int left = n - above;  // of the equals
#pragma unroll 1
    for (int j = 0; j < NV; ++j) {
      const u32x4 v = L::load(base, L::place(first, j, 0), (int)p.vocab);
      int equals = 0, total;
#pragma unroll
      for (int e = 0; e < L::kVec; ++e) equals += ordered_bits(L::value(v, e)) == exact;
      int before = block_before<kWavesRow>(equals, lds_add, total);
#pragma unroll
      for (int e = 0; e < L::kVec; ++e) {
        const uint32_t o = ordered_bits(L::value(v, e));
        if (o > exact || (o == exact && before < left)) keep(o, L::place(first, j, e));
        before += o == exact;
      }
      left -= total;
    }
    __syncthreads();
    count = lds_count;
  }
  const int64_t seq = row / p.beams, across = p.beams * a.nslices;
  uint64_t* list = a.lists + seq * n * across + (row - seq * p.beams) * a.nslices + slice;
  for (int i = threadIdx.x; i < count; i += kThreadsRow) {
    const uint64_t mine = lds_keys[i];
    int rank = 0;
#pragma unroll 8
    for (int o = 0; o < count; ++o) rank += lds_keys[o] > mine;
    if (rank < n) list[rank * across] = mine;
  }
  if (threadIdx.x == 0) {
    double s = 0.0;
#pragma unroll
    for (int w = 0; w < kWavesRow; ++w) s += (double)lds_sum[w];
    *out = s == s ? Slice{s, most, count < n ? count : n} : Slice{0.0, __builtin_inff(), 0};
  }
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS) beam_merge_kernel(BeamArgs a) {
  constexpr int WAVES = THREADS / 64;
  // A beam's totals are base + (logit - top), base = score - log sum exp(logit - top);
  // -infinity: no candidates.  (Not base - top + logit: logits may be the type's lowest.)
  __shared__ double lds_base[64], lds_term[THREADS];
  __shared__ float lds_most[64];
  __shared__ uint32_t lds_top[64];  // ordered bits
  __shared__ int lds_over[64];
  __shared__ uint32_t lds_bound;
  __shared__ uint64_t lds_keys[kRoomMerge];
  __shared__ uint32_t lds_best[WAVES][64];  // the upper halves
  __shared__ uint64_t lds_seconds[kRoomMerge];
  __shared__ uint32_t lds_out[kMaxOut];
  __shared__ int lds_count, lds_add[WAVES];
  const BeamSelectParams& p = a.p;
  const int64_t b = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int beams = (int)p.beams, n = (int)p.n_out, vocab = (int)p.vocab;
  const float* scores = p.scores + b * beams;
  const uint8_t* finished = p.finished != nullptr ? p.finished + b * beams : nullptr;
  const Slice* slices = a.slices + b * beams * a.nslices;
  const uint64_t* lists = a.lists + b * beams * a.nslices * n;

  // A thread looks at one slice, at every step-th rank of its list from r0 on.  What it
  // reads does not depend on anything read before, so it is all under way at once.
  const int across = beams * a.nslices, items = across * n;
  const int step = max(THREADS / across, 1), r0 = (int)threadIdx.x / across, at0 = (int)threadIdx.x - r0 * across;
  const bool held = across <= THREADS && n <= step * kHeld;  // holds<THREADS>
  const int k0 = at0 / a.nslices;
  uint64_t key[kHeld];
  Slice own{};
  bool over0 = false;
  if (held) {
#pragma unroll
    for (int j = 0; j < kHeld; ++j)
      if (j * step < n) key[j] = lists[min(r0 + j * step, n - 1) * across + at0];
    own = slices[at0];
    over0 = finished != nullptr && finished[k0] != 0;
  }
  const float score = (int)threadIdx.x < beams ? scores[threadIdx.x] : 0.0f;
  const bool over = (int)threadIdx.x < beams && finished != nullptr && finished[threadIdx.x] != 0;
  if (threadIdx.x < 64) lds_top[threadIdx.x] = 0;
  if (threadIdx.x == 0) lds_count = 0;
  __syncthreads();
  // Every beam's largest logit, the sum of its slices' sums, its base.
  if (held) {
    if (r0 == 0 && !over0) atomicMax(&lds_top[k0], ordered_bits(own.top));
    __syncthreads();
    const float top = value_of(lds_top[k0]);
    if (r0 == 0)
      lds_term[at0] = !over0 && own.count > 0 && top < __builtin_inff() ? own.sum * exp((double)own.top - (double)top) : 0.0;
    __syncthreads();
  } else {
    for (int k = wave; k < beams; k += WAVES) {
      float top = -__builtin_inff();
      for (int s = lane; s < a.nslices; s += 64) top = fmaxf(top, slices[k * a.nslices + s].top);
      top = lanes_max(top);
      double sum = 0.0;
      for (int s = lane; s < a.nslices; s += 64) {
        const Slice t = slices[k * a.nslices + s];
        if (t.count > 0 && top < __builtin_inff()) sum += t.sum * exp((double)t.top - (double)top);
      }
#pragma unroll
      for (int m = 1; m < 64; m <<= 1) sum += __shfl_xor(sum, m, 64);
      if (lane == 0) lds_top[k] = ordered_bits(top), lds_base[k] = sum;
    }
    __syncthreads();
  }
  if ((int)threadIdx.x < beams) {
    const int k = threadIdx.x;
    double sum = 0.0;
    if (held)
      for (int s = 0; s < a.nslices; ++s) sum += lds_term[k * a.nslices + s];
    else
      sum = lds_base[k];
    const float top = value_of(lds_top[k]);
    const bool none = !(score < __builtin_inff()) || score == -__builtin_inff() ||
                      (!over && !(__builtin_fabsf(top) < __builtin_inff()));
    lds_base[k] = none ? -__builtin_inf() : over ? (double)score : (double)score - log(sum);
    lds_most[k] = top;
    lds_over[k] = over;
  }
  __syncthreads();

  // The i-th item: its total's ordered bits (kOrderedNegInf64: no candidate) and what
  // decides between equal ones.  In the order of the lists, so that neighbouring threads, whose maxima
  // make the bound, look at the same rank of different slices.
  auto item = [&](int i, uint64_t& second) -> uint64_t {
    const int rank = i / across, at = i - rank * across, k = at / a.nslices;
    const uint64_t key = lists[i];
    const int listed = slices[at].count;
    const double base = lds_base[k];
    const bool over = lds_over[k] != 0;
    second = second_of(k, over ? key_of(0, (uint32_t)p.eos) : key);
    const bool is = base != -__builtin_inf() && (over ? rank == 0 && at == k * a.nslices : rank < listed);
    const double total = over ? base : base + ((double)value_of((uint32_t)(key >> 32)) - (double)lds_most[k]);
    return is ? ordered_bits(total) : kOrderedNegInf64;
  };
  uint64_t second;
  auto keep = [&](uint64_t o, uint64_t then) {
    const int to = atomicAdd(&lds_count, 1);
    if (to < kRoomMerge) lds_keys[to] = o, lds_seconds[to] = then;
  };
  uint64_t o[kHeld], best = kOrderedNegInf64;
  if (held) {
    const double base = lds_base[k0], most = (double)lds_most[k0];
    const bool none = r0 >= step || base == -__builtin_inf();
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      o[j] = kOrderedNegInf64;
      if (j * step >= n) continue;
      const int r = r0 + j * step;
      if (over0) key[j] = key_of(0, (uint32_t)p.eos);
      const double total = over0 ? base : base + ((double)value_of((uint32_t)(key[j] >> 32)) - most);
      if (!none && (over0 ? r == 0 && at0 == k0 * a.nslices : r < own.count && r < n)) o[j] = ordered_bits(total);
      best = o[j] > best ? o[j] : best;
    }
  } else {
#pragma unroll 4
    for (int i = threadIdx.x; i < items; i += THREADS) {
      const uint64_t t = item(i, second);
      best = t > best ? t : best;
    }
  }
  lds_best[wave][lane] = (uint32_t)(best >> 32);
  __syncthreads();
  if (wave == 0) {
    const uint32_t t = lds_threshold<24, WAVES>(lds_best, n > 8, n);
    if (lane == 0) lds_bound = t;
  }
  __syncthreads();
  uint64_t bound = (uint64_t)lds_bound << 32;
  if (bound <= kOrderedNegInf64) bound = kOrderedNegInf64 + 1;
  if (held) {
    if (best >= bound)
#pragma unroll
      for (int j = 0; j < kHeld; ++j)
        if (o[j] >= bound) keep(o[j], second_of(k0, key[j]));
  } else {
#pragma unroll 4
    for (int i = threadIdx.x; i < items; i += THREADS) {
      const uint64_t t = item(i, second);
      if (t >= bound) keep(t, second);
    }
  }
  __syncthreads();
  int count = lds_count;
  if (count > kRoomMerge) {  // as for a row, reading the lists each time
    int past = 0;  // of other prefixes than the bound's
    for (int i = threadIdx.x; i < items; i += THREADS) past += item(i, second) > (bound | 0xffffffffffull);
    const bool high = block_sum<WAVES>(past, lds_add) >= n;
    uint64_t exact = high ? 0 : bound;
    bool tied = true;
    for (int bit = high ? 63 : 39; bit >= 0 && tied; --bit) {
      const uint64_t with = exact | 1ull << bit;
      int c = 0;
      for (int i = threadIdx.x; i < items; i += THREADS) c += item(i, second) >= with;
      c = block_sum<WAVES>(c, lds_add);
      if (c >= n) exact = with, tied = c > kRoomMerge;
    }
    // (Fewer than n candidates: all of them, and none of what is not one.)
    if (exact <= kOrderedNegInf64) exact = kOrderedNegInf64 + 1, tied = false;
    uint64_t least = 0;  // of the equals' second keys
    if (tied) {
      int above = 0;
      for (int i = threadIdx.x; i < items; i += THREADS) above += item(i, second) > exact;
      above = block_sum<WAVES>(above, lds_add);
      for (int bit = 61; bit >= 0; --bit) {
        const uint64_t with = least | 1ull << bit;
        int c = 0;
        for (int i = threadIdx.x; i < items; i += THREADS) c += item(i, second) == exact && second >= with;
        if (block_sum<WAVES>(c, lds_add) >= n - above) least = with;
      }
    }
    if (threadIdx.x == 0) lds_count = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < items; i += THREADS) {
      const uint64_t o = item(i, second);
      if (o > exact || (o == exact && second >= least)) keep(o, second);
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
  for (int i = threadIdx.x; i < count; i += THREADS) {
    const uint64_t mine = lds_keys[i];
    const uint64_t then = lds_seconds[i];
    int rank = 0;
#pragma unroll 8
    for (int o = 0; o < count; ++o) {
      const uint64_t other = lds_keys[o];
      rank += (other > mine) | ((other == mine) & (lds_seconds[o] > then));
    }
    if (rank < n) {
      const uint32_t at = place_of_second(then, vocab);
      put(rank, (float)value_of(mine), at);
      lds_out[rank] = at;
    }
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

// 256 threads where they hold the lists, whose barriers take less time (16 x 8 x 32000
// bf16, n = 16: 13.2 us, with 1024 14.3; 64 x 4 x 32000 fp32: 15.1 and 15.7).
template <int THREADS>
bool holds(int64_t across, int64_t n) { return across <= THREADS && n <= THREADS / across * kHeld; }

// Slices of 8192 logits where there is much to do or to merge (16 x 8 x 32000 bf16:
// 13.2 us, with slices of 2048 15.1; 4 x 16 x 32000: 13.4 and 16.3), else of 2048, for
// the time that a workgroup takes for its slice (1 x 5 x 50277: 10.8 and 10.0) or
// for rows that are no longer (256 x 16 x 1500: 25.6 and 18.6).  16 x 4 x 32000 and 64 x 8
// x 5000 take the same time either way.
constexpr int64_t kWideSlice = 8192, kNarrowSlice = 2048;
constexpr int64_t kManySlices = 1280, kManyLists = 128;  // narrow ones: of the call, of a sequence
int64_t slices_of(int64_t batch, int64_t beams, int64_t vocab, bool& wide) {
  const int64_t narrow = (vocab + kNarrowSlice - 1) / kNarrowSlice;
  wide = narrow > 1 && (batch * beams * narrow > kManySlices || beams * narrow > kManyLists);
  return wide ? (vocab + kWideSlice - 1) / kWideSlice : narrow;
}

size_t lists_offset(int64_t slices) { return kHeader + (size_t)slices * sizeof(Slice); }

template <bool BF16, int NV>
void launch_rows(const BeamArgs& a, hipStream_t stream) {
  static_assert(Logits<BF16, NV>::kSlice == kWideSlice || Logits<BF16, NV>::kSlice == kNarrowSlice, "");
  hipLaunchKernelGGL((beam_rows_kernel<BF16, NV>), dim3((unsigned)(a.p.batch * a.p.beams * a.nslices)),
                     dim3(kThreadsRow), 0, stream, a);
}

}  // namespace

int64_t beam_select_workgroups(int64_t batch, int64_t beams, int64_t vocab) {
  bool wide;
  return batch * beams * slices_of(batch, beams, vocab, wide);
}

size_t beam_select_workspace_bytes(int64_t batch, int64_t beams, int64_t vocab, int64_t n_out) {
  const int64_t slices = beam_select_workgroups(batch, beams, vocab);
  return lists_offset(slices) + (size_t)(slices * n_out) * sizeof(uint64_t);
}

hipError_t launch_beam_select(const BeamSelectParams& p, hipStream_t stream) {
  bool wide;
  const int64_t nslices = slices_of(p.batch, p.beams, p.vocab, wide);
  char* ws = static_cast<char*>(p.workspace);
  const BeamArgs a{p, reinterpret_cast<Slice*>(ws + kHeader),
                   reinterpret_cast<uint64_t*>(ws + lists_offset(p.batch * p.beams * nslices)), (int)nslices};
  if (p.bf16) wide ? launch_rows<true, 4>(a, stream) : launch_rows<true, 1>(a, stream);
  else wide ? launch_rows<false, 8>(a, stream) : launch_rows<false, 2>(a, stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (holds<256>(p.beams * a.nslices, p.n_out))
    hipLaunchKernelGGL(beam_merge_kernel<256>, dim3((unsigned)p.batch), dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL(beam_merge_kernel<1024>, dim3((unsigned)p.batch), dim3(1024), 0, stream, a);
  return hipGetLastError();
}

}  // namespace mss
