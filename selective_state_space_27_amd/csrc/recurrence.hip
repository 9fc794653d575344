// Gated linear recurrence: scan over whole sequences and its gradient (gfx950).
// Definitions in include/mambascan.h, arithmetic in recurrence.hpp.
//
// h_t = a_t h_{t-1} + b_t is cut along t: a wave holds T steps of 64 V channels
// (V neighbouring ones a lane) in registers and runs them from a zero state,
// which gives per channel the product A of its decays and its end state H; a
// workgroup's W waves, side by side in time, fold these in LDS; workgroups hand
// states on through memory (Chain).  Then every wave adds what its entering
// state has become at each step.  Inputs are read once and outputs written once,
// whatever the length.
//
// Where a packed sequence starts, what was before counts as zero even if it is
// NaN: A is not multiplied in but skipped (a start is the same for all channels,
// so the choice is a scalar one).
#include "launch.hpp"
#include "norm_common.hpp"
#include "recurrence.hpp"

namespace mss {
namespace {

// ------------------------------------------------------------ pieces in order
// A piece is one workgroup's steps of one stream (64 V channels of a batch row).
// Pieces take their place in order of start (a ticket): s-th in its stream, all
// streams' s-th before any (s+1)-th.  A piece that has its own A and H publishes
// them, looks back for the nearest piece whose end state is known, folds what
// lies between from there on, and publishes its own end state.  The fold is the
// same sequence of operations wherever it begins, so results do not depend on
// timing.  What is waited for belongs to pieces that have started and that
// publish it before they wait themselves.
//
// Values move through relaxed agent-scope atomics, coherent across the dies.  A
// word that is all ones has not been written: the buffers are filled with that
// before, and a NaN of those bits is replaced by another.  So one load tells
// whether a value is there and what it is; flags beside the values took a wait
// for the stores, one load more for each look and two more for each hand-over.
constexpr int kMaxSpinsChain = 1 << 20;
constexpr uint32_t kUnset = 0xffffffffu;
constexpr int kChainHeader = 64;  // bytes before the values: status word, ticket

constexpr int kManyStreams = 96;

struct Chain {
  int* status;    // null: one piece a stream, nothing is handed on
  int* ticket;
  uint64_t* own;  // [place][stream][64 V]: A, H
  float* end;     // [place][stream][64 V]
  int streams;
};

// Status word and ticket to 0, the rest (n times 16 bytes) to unset.
__global__ void __launch_bounds__(256) chain_clear_kernel(u32x4* p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const uint32_t v = i < kChainHeader / 16 ? 0u : kUnset;
    p[i] = u32x4{v, v, v, v};
  }
}

__device__ __forceinline__ uint32_t set_bits(float v) {
  const uint32_t u = __float_as_uint(v);
  return u == kUnset ? 0x7fc00000u : u;
}
template <int V>
__device__ __forceinline__ void put_end(float* p, const float (&h)[V]) {
  if constexpr (V == 2) {
    __hip_atomic_store(reinterpret_cast<uint64_t*>(p), (uint64_t)set_bits(h[1]) << 32 | set_bits(h[0]),
                       __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  } else {
    __hip_atomic_store(reinterpret_cast<uint32_t*>(p), set_bits(h[0]), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
}
template <int V>
__device__ __forceinline__ void put_own(uint64_t* p, const float (&a)[V], const float (&h)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v)
    __hip_atomic_store(p + v, (uint64_t)set_bits(h[v]) << 32 | set_bits(a[v]), __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
}
template <int V>
__device__ __forceinline__ uint64_t load_end(const float* p) {
  if constexpr (V == 2)
    return __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  else
    return __hip_atomic_load(reinterpret_cast<const uint32_t*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ bool is_set(uint64_t w) { return (uint32_t)w != kUnset; }

// One look at the last N places before `place`: whether an end state is there and
// everything after it, and if so what enters the piece.
template <int V, int N>
__device__ __forceinline__ bool chain_look(const Chain& c, int place, int stream, float (&carry)[V]) {
  const int lane = threadIdx.x & 63;
  uint64_t end[N], own[N][V];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int at = place - 1 - i > 0 ? place - 1 - i : 0;
    const int64_t off = ((int64_t)at * c.streams + stream) * (64 * V) + lane * V;
    end[i] = load_end<V>(c.end + off);
    if (i + 1 < N)
#pragma unroll
      for (int v = 0; v < V; ++v)
        own[i][v] = __hip_atomic_load(c.own + off + v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  int near = -1;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (near >= 0) break;
    if (__all(is_set(end[i]))) near = i;
    bool there = i + 1 < N;
#pragma unroll
    for (int v = 0; v < V; ++v) there = there && is_set(own[i + 1 < N ? i : 0][v]);
    if (near < 0 && !__all(there)) return false;
  }
  if (near < 0) return false;
#pragma unroll
  for (int i = N - 1; i >= 0; --i) {
    if (i == near) {
      carry[0] = __uint_as_float((uint32_t)end[i]);
      if constexpr (V == 2) carry[1] = __uint_as_float((uint32_t)(end[i] >> 32));
    }
    if (i < near)
#pragma unroll
      for (int v = 0; v < V; ++v)
        carry[v] = __builtin_fmaf(__uint_as_float((uint32_t)own[i][v]), carry[v],
                                  __uint_as_float((uint32_t)(own[i][v] >> 32)));
  }
  return true;
}

// What enters the piece at `place` of `stream` (wave 0's lanes; `first` at place
// 0), given its own A and H; publishes what later pieces need.  `cut`: a sequence
// starts inside, so its end state does not depend on what enters.
template <int V>
__device__ __forceinline__ void chain_carry(const Chain& c, int place, int stream, bool last, bool cut,
                                            const float (&own_a)[V], const float (&own_h)[V], const float (&first)[V],
                                            float (&carry)[V]) {
  const int64_t off = ((int64_t)place * c.streams + stream) * (64 * V) + (threadIdx.x & 63) * V;
  if (cut && !last) put_end<V>(c.end + off, own_h);
  if (place == 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) carry[v] = first[v];
  } else {
    if (!cut && !last) put_own<V>(c.own + off, own_a, own_h);
    // With many streams the piece before has mostly ended; with few, several of a
    // stream are under way at once.
    bool found = c.streams >= kManyStreams && chain_look<V, 1>(c, place, stream, carry);
    for (int spins = 0; !found; ++spins) {
      found = chain_look<V, 4>(c, place, stream, carry);
      if (!found && spins > kMaxSpinsChain) {  // never expected; keeps every wait finite, reported through the status word
        if ((threadIdx.x & 63) == 0) __hip_atomic_store(c.status, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
        for (int v = 0; v < V; ++v) carry[v] = 0.0f;
        break;
      }
    }
  }
  if (cut || last) return;
  float h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = __builtin_fmaf(own_a[v], carry[v], own_h[v]);
  put_end<V>(c.end + off, h);
}

// ------------------------------------------------------------ rows
// V neighbouring channels of a row as loaded: two bf16 in a word, or one value.
template <bool BF16, int V>
__device__ __forceinline__ uint32_t load_raw_at(const void* row, uint32_t ch) {
  if constexpr (BF16 && V == 1) return static_cast<const uint16_t*>(row)[ch];
  else if constexpr (BF16) return *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(row) + ch);
  else return static_cast<const uint32_t*>(row)[ch];
}
template <bool BF16, int V>
__device__ __forceinline__ float widen_at(uint32_t w, int v) {
  if constexpr (!BF16) return __uint_as_float(w);
  else return v == 0 ? bf16_lo(w) : bf16_hi(w);
}
template <bool BF16, int V>
__device__ __forceinline__ void store_at(void* row, uint32_t ch, const float (&o)[V]) {
  if constexpr (BF16 && V == 1) static_cast<uint16_t*>(row)[ch] = f32_to_bf16(o[0]);
  else if constexpr (BF16) *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(row) + ch) = pack_bf16x2(o[0], o[1]);
  else static_cast<float*>(row)[ch] = o[0];
}
// Rows r0, r0 + 1, .. of a tensor, a wave's lanes at channel ch; past the last of n
// rows the last is repeated.  WHOLE: there are T.
template <bool BF16, int V, int T, bool WHOLE>
__device__ __forceinline__ void load_rows(const void* p, int64_t r0, int64_t stride, uint32_t ch, int n,
                                          uint32_t (&raw)[T]) {
  const char* row = static_cast<const char*>(p) + r0 * stride * (BF16 ? 2 : 4);
  const int64_t step = stride * (BF16 ? 2 : 4);
#pragma unroll
  for (int j = 0; j < T; ++j) {
    raw[j] = load_raw_at<BF16, V>(row, ch);
    if (WHOLE || j + 1 < n) row += step;
  }
}

// Where a wave works: which piece, its steps, its lane's channels.
template <int V, int W, int T>
struct WavePlace {
  int place, stream, wave;
  int64_t b, t0;     // batch row, first step
  int n;             // steps that exist
  uint32_t ch;       // first channel, kept inside the row
  bool ok;           // whether it exists
};

// `piece` in order along time; a lane past the last channel repeats it.
template <int V, int W, int T>
__device__ __forceinline__ WavePlace<V, W, T> wave_place(int64_t id, int streams, int blocks, int64_t pieces,
                                                         bool reversed, int64_t seqlen, int64_t dim) {
  WavePlace<V, W, T> w;
  w.place = (int)(id / streams);
  w.stream = (int)(id - (int64_t)w.place * streams);
  w.wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  w.b = w.stream / blocks;
  const int64_t piece = reversed ? pieces - 1 - w.place : w.place;
  w.t0 = piece * (W * T) + w.wave * T;
  const int64_t left = seqlen - w.t0;
  w.n = left < 0 ? 0 : left < T ? (int)left : T;
  const int64_t c = (int64_t)(w.stream - (int)w.b * blocks) * (64 * V) + (threadIdx.x & 63) * V;
  w.ok = c < dim;
  w.ch = (uint32_t)(w.ok ? c : dim - V);
  return w;
}

// Bit j: a sequence starts at the wave's step j.
template <int T>
__device__ __forceinline__ uint64_t start_bits(const uint8_t* starts, int64_t row, int n) {
  if (starts == nullptr) return 0;
  const int lane = threadIdx.x & 63;
  return __ballot(lane < n && starts[row + (lane < n ? lane : 0)] != 0);
}

// ------------------------------------------------------------ forward
struct FwdArgs {
  RecurrenceFwdParams p;
  Chain chain;
  int blocks;      // of channels
  int64_t pieces;  // of a stream
};

template <bool BF16, int V, int W, int T>
__global__ void __launch_bounds__(W * 64) recurrence_fwd_kernel(FwdArgs a) {
  __shared__ float lds_a[W][64 * V], lds_h[W][64 * V], lds_carry[64 * V];
  __shared__ int lds_cut[W], lds_id;
  const RecurrenceFwdParams& p = a.p;
  int64_t id = blockIdx.x;
  if (a.chain.status != nullptr) {
    if (threadIdx.x == 0) lds_id = atomicAdd(a.chain.ticket, 1);
    __syncthreads();
    id = __builtin_amdgcn_readfirstlane(lds_id);
  } else if (id == 0 && threadIdx.x == 0) {
    *static_cast<int*>(p.workspace) = 0;  // the status word: nothing waits
  }
  const auto w = wave_place<V, W, T>(id, a.chain.streams, a.blocks, a.pieces, false, p.seqlen, p.dim);
  const int lane = threadIdx.x & 63;
  const int64_t row0 = w.b * p.seqlen + w.t0;

  uint32_t rx[T], ra[T], ri[T];
  const auto load = [&](auto whole) {
    load_rows<BF16, V, T, whole()>(p.gate_a, row0, p.gate_a_stride, w.ch, w.n, ra);
    load_rows<BF16, V, T, whole()>(p.gate_x, row0, p.gate_x_stride, w.ch, w.n, ri);
    load_rows<BF16, V, T, whole()>(p.x, row0, p.x_stride, w.ch, w.n, rx);
  };
  if (w.n == T) load(std::true_type{});
  else if (w.n > 0) load(std::false_type{});
  const uint64_t starts = w.n > 0 ? start_bits<T>(p.starts, row0, w.n) : 0;
  const bool plain = w.n == T && starts == 0;
  float k[V];
  bool low = true;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    k[v] = p.c * softplus_of(p.lam[w.ch + v]);
    low = low && k[v] <= kPolySmall;
  }

  // From a zero state: after each step the state and the product of the decays.
  float pr[T][V], hl[T][V], ha[V], hh[V];
#pragma unroll
  for (int v = 0; v < V; ++v) ha[v] = 1.0f, hh[v] = 0.0f;
  const auto local = [&](auto whole, auto small) {
#pragma unroll
    for (int j = 0; j < T; ++j) {
      if (!whole() && j >= w.n) break;
      const bool start = !whole() && (starts >> j & 1);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float mj = one_minus_exp<small()>(k[v] * sigmoid_of<!BF16>(widen_at<BF16, V>(ra[j], v)));
        const float in = __builtin_amdgcn_sqrtf(mj * (2.0f - mj)) * sigmoid_of<!BF16>(widen_at<BF16, V>(ri[j], v)) *
                         widen_at<BF16, V>(rx[j], v);
        hh[v] = (start ? 0.0f : __builtin_fmaf(-mj, hh[v], hh[v])) + in;
        ha[v] = __builtin_fmaf(-mj, ha[v], ha[v]);
        hl[j][v] = hh[v];
        pr[j][v] = ha[v];
      }
    }
  };
  if (plain) {
    if (__all(low)) local(std::true_type{}, std::true_type{});
    else local(std::true_type{}, std::false_type{});
  } else if (w.n > 0) {
    local(std::false_type{}, std::false_type{});
  }
#pragma unroll
  for (int v = 0; v < V; ++v) lds_a[w.wave][lane * V + v] = ha[v], lds_h[w.wave][lane * V + v] = hh[v];
  if (lane == 0) lds_cut[w.wave] = starts != 0;
  __syncthreads();

  if (w.wave == 0) {
    float first[V], carry[V];
#pragma unroll
    for (int v = 0; v < V; ++v) first[v] = p.h0 != nullptr && w.place == 0 ? p.h0[w.b * p.dim + w.ch + v] : 0.0f;
    if (a.chain.status == nullptr) {
#pragma unroll
      for (int v = 0; v < V; ++v) carry[v] = first[v];
    } else {
      bool cut = starts != 0;
      for (int i = 1; i < W; ++i) {
        const bool c = lds_cut[i] != 0;
        cut |= c;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float ai = lds_a[i][lane * V + v], hi = lds_h[i][lane * V + v];
          hh[v] = c ? hi : __builtin_fmaf(ai, hh[v], hi);
          ha[v] *= ai;
        }
      }
      chain_carry<V>(a.chain, w.place, w.stream, w.place + 1 == a.pieces, cut, ha, hh, first, carry);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) lds_carry[lane * V + v] = carry[v];
  }
  __syncthreads();

  if (w.n == 0) return;
  float q[V];
#pragma unroll
  for (int v = 0; v < V; ++v) q[v] = lds_carry[lane * V + v];
  for (int i = 0; i < w.wave; ++i) {
    const bool c = lds_cut[i] != 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float hi = lds_h[i][lane * V + v];
      q[v] = c ? hi : __builtin_fmaf(lds_a[i][lane * V + v], q[v], hi);
    }
  }
  if (!w.ok) return;
  if (p.states != nullptr && w.t0 % kRecurrenceChunk == 0) {
    const int64_t chunks = (p.seqlen + kRecurrenceChunk - 1) / kRecurrenceChunk;
#pragma unroll
    for (int v = 0; v < V; ++v) p.states[(w.b * chunks + w.t0 / kRecurrenceChunk) * p.dim + w.ch + v] = q[v];
  }
  char* y = static_cast<char*>(p.y) + row0 * p.y_stride * (BF16 ? 2 : 4);
  const auto apply = [&](auto whole) {
#pragma unroll
    for (int j = 0; j < T; ++j) {
      if (!whole() && j >= w.n) break;
      const bool cut = !whole() && (starts & ((2ull << j) - 1)) != 0;
      float o[V];
#pragma unroll
      for (int v = 0; v < V; ++v) o[v] = cut ? hl[j][v] : __builtin_fmaf(pr[j][v], q[v], hl[j][v]);
      store_at<BF16, V>(y, w.ch, o);
      y += p.y_stride * (BF16 ? 2 : 4);
      if (p.h_last != nullptr && w.t0 + j == p.seqlen - 1)
#pragma unroll
        for (int v = 0; v < V; ++v) p.h_last[w.b * p.dim + w.ch + v] = o[v];
    }
  };
  if (plain) apply(std::true_type{});
  else apply(std::false_type{});
}

// ------------------------------------------------------------ backward
struct BwdArgs {
  RecurrenceBwdParams p;
  Chain chain;
  float* part;     // [batch][pieces][dim]
  int blocks;
  int64_t pieces;
};

// Below, beta = sqrt(2 m) and s / beta = sqrt(m / 2) add nothing to what they meet
// (the reciprocal root takes such an m for 0).
constexpr float kLeastNormal = 1.1754944e-38f;

// One piece is one chunk: W T = kRecurrenceChunk.
template <bool BF16, int V, int W, int T>
__global__ void __launch_bounds__(W * 64) recurrence_bwd_kernel(BwdArgs a) {
  static_assert(W * T == kRecurrenceChunk, "");
  __shared__ float lds_a[W][64 * V], lds_h[W][64 * V], lds_e[W][64 * V], lds_carry[64 * V];
  __shared__ int lds_cut[W], lds_id;
  const RecurrenceBwdParams& p = a.p;
  int64_t id = blockIdx.x;
  if (a.chain.status != nullptr) {
    if (threadIdx.x == 0) lds_id = atomicAdd(a.chain.ticket, 1);
    __syncthreads();
    id = __builtin_amdgcn_readfirstlane(lds_id);
  } else if (id == 0 && threadIdx.x == 0) {
    *static_cast<int*>(p.workspace) = 0;  // the status word: nothing waits
  }
  const auto w = wave_place<V, W, T>(id, a.chain.streams, a.blocks, a.pieces, true, p.seqlen, p.dim);
  const int lane = threadIdx.x & 63;
  const int64_t row0 = w.b * p.seqlen + w.t0, piece = a.pieces - 1 - w.place;

  uint32_t rx[T], ra[T], ri[T], rd[T];
  const auto load = [&](auto whole) {
    load_rows<BF16, V, T, whole()>(p.gate_a, row0, p.gate_a_stride, w.ch, w.n, ra);
    load_rows<BF16, V, T, whole()>(p.gate_x, row0, p.gate_x_stride, w.ch, w.n, ri);
    load_rows<BF16, V, T, whole()>(p.x, row0, p.x_stride, w.ch, w.n, rx);
    load_rows<BF16, V, T, whole()>(p.dy, row0, p.dy_stride, w.ch, w.n, rd);
  };
  if (w.n == T) load(std::true_type{});
  else if (w.n > 0) load(std::false_type{});
  const uint64_t starts = w.n > 0 ? start_bits<T>(p.starts, row0, w.n) : 0;
  const bool plain = w.n == T && starts == 0;
  float k[V], sp[V], before[V];  // before: the state entering the piece, then this wave's steps
  bool low = true;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    sp[v] = softplus_of(p.lam[w.ch + v]);
    k[v] = p.c * sp[v];
    low = low && k[v] <= kPolySmall;
    before[v] = p.states[(w.b * a.pieces + piece) * p.dim + w.ch + v];
  }

  // From a zero state forwards (hl), from a zero gradient backwards (e).
  float m[T][V], hl[T][V], ha[V], hh[V], e[V];
#pragma unroll
  for (int v = 0; v < V; ++v) ha[v] = 1.0f, hh[v] = 0.0f, e[v] = 0.0f;
  const auto local = [&](auto whole, auto small) {
#pragma unroll
    for (int j = 0; j < T; ++j) {
      if (!whole() && j >= w.n) break;
      const bool start = !whole() && (starts >> j & 1);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float mj = one_minus_exp<small()>(k[v] * sigmoid_of<!BF16>(widen_at<BF16, V>(ra[j], v)));
        const float in = __builtin_amdgcn_sqrtf(mj * (2.0f - mj)) * sigmoid_of<!BF16>(widen_at<BF16, V>(ri[j], v)) *
                         widen_at<BF16, V>(rx[j], v);
        m[j][v] = mj;
        hh[v] = (start ? 0.0f : __builtin_fmaf(-mj, hh[v], hh[v])) + in;
        ha[v] = __builtin_fmaf(-mj, ha[v], ha[v]);
        hl[j][v] = hh[v];
      }
    }
#pragma unroll
    for (int j = T - 1; j >= 0; --j) {
      if (!whole() && j >= w.n) continue;
      const bool start = !whole() && (starts >> j & 1);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float g = widen_at<BF16, V>(rd[j], v) + e[v];
        e[v] = start ? 0.0f : __builtin_fmaf(-m[j][v], g, g);
      }
    }
  };
  if (plain) {
    if (__all(low)) local(std::true_type{}, std::true_type{});
    else local(std::true_type{}, std::false_type{});
  } else if (w.n > 0) {
    local(std::false_type{}, std::false_type{});
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    lds_a[w.wave][lane * V + v] = ha[v];
    lds_h[w.wave][lane * V + v] = hh[v];
    lds_e[w.wave][lane * V + v] = e[v];
  }
  if (lane == 0) lds_cut[w.wave] = starts != 0;
  __syncthreads();

  if (w.wave == 0) {
    float first[V], carry[V], ea[V], ee[V];
    bool cut = false;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      first[v] = p.dh_last != nullptr && w.place == 0 ? p.dh_last[w.b * p.dim + w.ch + v] : 0.0f;
      ea[v] = 1.0f, ee[v] = 0.0f;
    }
    if (a.chain.status == nullptr) {
#pragma unroll
      for (int v = 0; v < V; ++v) carry[v] = first[v];
    } else {
      for (int i = W - 1; i >= 0; --i) {
        const bool c = lds_cut[i] != 0;
        cut |= c;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float ai = lds_a[i][lane * V + v], ei = lds_e[i][lane * V + v];
          ee[v] = c ? ei : __builtin_fmaf(ai, ee[v], ei);
          ea[v] *= ai;
        }
      }
      chain_carry<V>(a.chain, w.place, w.stream, w.place + 1 == a.pieces, cut, ea, ee, first, carry);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) lds_carry[lane * V + v] = carry[v];
  }
  // The states before each step, from the one that enters the piece.
  for (int i = 0; i < w.wave; ++i) {
    const bool c = lds_cut[i] != 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float hi = lds_h[i][lane * V + v];
      before[v] = c ? hi : __builtin_fmaf(lds_a[i][lane * V + v], before[v], hi);
    }
  }
  const auto enter = [&](auto whole) {
    float q[V];
#pragma unroll
    for (int v = 0; v < V; ++v) q[v] = before[v];
#pragma unroll
    for (int j = 0; j < T; ++j) {
      if (!whole() && j >= w.n) break;
      const bool start = !whole() && (starts >> j & 1);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        q[v] = start ? 0.0f : __builtin_fmaf(-m[j][v], q[v], q[v]);
        hl[j][v] += q[v];
      }
    }
  };
  if (plain) enter(std::true_type{});
  else if (w.n > 0) enter(std::false_type{});
  __syncthreads();

#pragma unroll
  for (int v = 0; v < V; ++v) e[v] = lds_carry[lane * V + v];
  for (int i = W - 1; i > w.wave; --i) {
    const bool c = lds_cut[i] != 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float ei = lds_e[i][lane * V + v];
      e[v] = c ? ei : __builtin_fmaf(lds_a[i][lane * V + v], e[v], ei);
    }
  }
  float dlam[V];
#pragma unroll
  for (int v = 0; v < V; ++v) dlam[v] = 0.0f;
  const int64_t es = BF16 ? 2 : 4;
  char* dx = static_cast<char*>(p.dx) + (row0 + w.n) * p.dx_stride * es;
  char* da = static_cast<char*>(p.dgate_a) + (row0 + w.n) * p.dgate_a_stride * es;
  char* di = static_cast<char*>(p.dgate_x) + (row0 + w.n) * p.dgate_x_stride * es;
  const auto grads = [&](auto whole) {
#pragma unroll
    for (int j = T - 1; j >= 0; --j) {
      if (!whole() && j >= w.n) continue;
      const bool start = !whole() && (starts >> j & 1);
      float ox[V], oa[V], oi[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float rr, rest;
        const float r = sigmoid_of<!BF16>(widen_at<BF16, V>(ra[j], v), rr);
        const float i = sigmoid_of<!BF16>(widen_at<BF16, V>(ri[j], v), rest);
        const float s = finite_decay(k[v] * r), mj = m[j][v], dec = 1.0f - mj, beta2 = mj * (2.0f - mj);
        const float inv = __builtin_amdgcn_rsqf(beta2), beta = mj >= kLeastNormal ? beta2 * inv : mj;
        const float g = widen_at<BF16, V>(rd[j], v) + e[v];
        const float gi = g * i, gix = gi * widen_at<BF16, V>(rx[j], v);
        const float from_beta = dec * dec * (mj >= kLeastNormal ? s * inv : mj) * gix;
        const float prev = j > 0 ? hl[j > 0 ? j - 1 : 0][v] : before[v];
        const float big = from_beta - (start ? 0.0f : s * dec * (g * prev));
        ox[v] = gi * beta;
        oi[v] = gix * beta * rest;
        oa[v] = big * rr;
        dlam[v] += big;
        e[v] = start ? 0.0f : __builtin_fmaf(-mj, g, g);
      }
      dx -= p.dx_stride * es, da -= p.dgate_a_stride * es, di -= p.dgate_x_stride * es;
      if (w.ok) {
        store_at<BF16, V>(dx, w.ch, ox);
        store_at<BF16, V>(da, w.ch, oa);
        store_at<BF16, V>(di, w.ch, oi);
      }
    }
  };
  if (plain) grads(std::true_type{});
  else if (w.n > 0) grads(std::false_type{});
  if (w.wave == 0 && piece == 0 && p.dh0 != nullptr && w.ok)
#pragma unroll
    for (int v = 0; v < V; ++v) p.dh0[w.b * p.dim + w.ch + v] = e[v];
  __syncthreads();  // lds_h has been read
#pragma unroll
  for (int v = 0; v < V; ++v) lds_h[w.wave][lane * V + v] = dlam[v];
  __syncthreads();
  if (w.wave == 0 && w.ok) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float sum = 0.0f;
      for (int i = 0; i < W; ++i) sum += lds_h[i][lane * V + v];
      a.part[(w.b * a.pieces + piece) * p.dim + w.ch + v] = sum * softplus_rate(p.lam[w.ch + v], sp[v]);
    }
  }
}

// ------------------------------------------------------------ launch
constexpr int kWaves = 8;
constexpr int kFwdSteps = 16, kBwdSteps = kRecurrenceChunk / kWaves;  // of a wave

struct Cut {
  int64_t blocks, pieces, streams;
  size_t own, end, bytes;  // offsets in the workspace
};
Cut cut_of(int64_t batch, int64_t seqlen, int64_t dim, int v, int steps) {
  Cut c;
  c.blocks = (dim + 64 * v - 1) / (64 * v);
  c.streams = batch * c.blocks;
  c.pieces = (seqlen + steps - 1) / steps;
  const size_t n = c.pieces > 1 ? (size_t)(c.streams * c.pieces) * (64 * v) : 0;
  c.own = kChainHeader;
  c.end = c.own + n * sizeof(uint64_t);
  c.bytes = c.end + n * sizeof(float);
  return c;
}

hipError_t start_chain(const Cut& c, void* workspace, Chain& chain, hipStream_t stream) {
  char* base = static_cast<char*>(workspace);
  chain.streams = (int)c.streams;
  chain.status = nullptr;
  if (c.pieces == 1) return hipSuccess;
  chain.status = reinterpret_cast<int*>(base);
  chain.ticket = chain.status + 1;
  chain.own = reinterpret_cast<uint64_t*>(base + c.own);
  chain.end = reinterpret_cast<float*>(base + c.end);
  const int64_t n = (int64_t)(c.bytes / 16), groups = (n + 1023) / 1024;
  hipLaunchKernelGGL(chain_clear_kernel, dim3((unsigned)(groups < 2048 ? groups : 2048)), dim3(256), 0, stream,
                     reinterpret_cast<u32x4*>(base), n);
  return hipGetLastError();
}

// Two bf16 channels a lane need rows of whole words.
bool pairs(const void* p, int64_t stride) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0 && stride % 2 == 0; }

template <bool BF16, int V>
hipError_t launch_fwd(const RecurrenceFwdParams& p, hipStream_t stream) {
  const Cut c = cut_of(p.batch, p.seqlen, p.dim, V, kWaves * kFwdSteps);
  FwdArgs a{p, {}, (int)c.blocks, c.pieces};
  const hipError_t e = start_chain(c, p.workspace, a.chain, stream);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((recurrence_fwd_kernel<BF16, V, kWaves, kFwdSteps>), dim3((unsigned)(c.streams * c.pieces)),
                     dim3(kWaves * 64), 0, stream, a);
  return hipGetLastError();
}

size_t bwd_part_offset(const Cut& c) { return (c.bytes + 255) / 256 * 256; }

template <bool BF16, int V>
hipError_t launch_bwd(const RecurrenceBwdParams& p, hipStream_t stream) {
  const Cut c = cut_of(p.batch, p.seqlen, p.dim, V, kRecurrenceChunk);
  BwdArgs a{p, {}, reinterpret_cast<float*>(static_cast<char*>(p.workspace) + bwd_part_offset(c)), (int)c.blocks,
            c.pieces};
  hipError_t e = start_chain(c, p.workspace, a.chain, stream);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((recurrence_bwd_kernel<BF16, V, kWaves, kBwdSteps>), dim3((unsigned)(c.streams * c.pieces)),
                     dim3(kWaves * 64), 0, stream, a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  SumPartialsArgs s{};
  s.part = a.part;
  s.dweight = p.dlam;
  s.nparts = p.batch * c.pieces;
  s.cols = p.dim;
  s.nout = 1;
  return launch_sum_partials(s, stream);
}

}  // namespace

// Whether channels go in pairs depends on the call's addresses: room for either.
size_t recurrence_fwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim, bool bf16) {
  const size_t one = cut_of(batch, seqlen, dim, 1, kWaves * kFwdSteps).bytes;
  const size_t two = bf16 ? cut_of(batch, seqlen, dim, 2, kWaves * kFwdSteps).bytes : 0;
  return one > two ? one : two;
}

hipError_t launch_recurrence_fwd(const RecurrenceFwdParams& p, hipStream_t stream) {
  if (!p.bf16) return launch_fwd<false, 1>(p, stream);
  const bool two = p.dim % 2 == 0 && pairs(p.x, p.x_stride) && pairs(p.gate_a, p.gate_a_stride) &&
                   pairs(p.gate_x, p.gate_x_stride) && pairs(p.y, p.y_stride);
  return two ? launch_fwd<true, 2>(p, stream) : launch_fwd<true, 1>(p, stream);
}

size_t recurrence_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim, bool bf16) {
  const Cut one = cut_of(batch, seqlen, dim, 1, kRecurrenceChunk), two = cut_of(batch, seqlen, dim, 2, kRecurrenceChunk);
  const size_t a = bwd_part_offset(one), b = bf16 ? bwd_part_offset(two) : 0;
  return (a > b ? a : b) + (size_t)(batch * one.pieces * dim) * sizeof(float);
}

hipError_t launch_recurrence_bwd(const RecurrenceBwdParams& p, hipStream_t stream) {
  if (!p.bf16) return launch_bwd<false, 1>(p, stream);
  const bool two = p.dim % 2 == 0 && pairs(p.dy, p.dy_stride) && pairs(p.x, p.x_stride) &&
                   pairs(p.gate_a, p.gate_a_stride) && pairs(p.gate_x, p.gate_x_stride) && pairs(p.dx, p.dx_stride) &&
                   pairs(p.dgate_a, p.dgate_a_stride) && pairs(p.dgate_x, p.dgate_x_stride);
  return two ? launch_bwd<true, 2>(p, stream) : launch_bwd<true, 1>(p, stream);
}

}  // namespace mss
