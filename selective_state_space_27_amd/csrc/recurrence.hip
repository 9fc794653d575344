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
//
// Bound by memory where there is enough to do: 4 x 8192 x 5120 bf16 forward 260 us (1.34
// GB at 5.1 TB/s; a 1 GiB copy reaches 5.13), backward 507 us (2.35 GB, 4.6 TB/s);
// 131072 x 2560 forward 525 us (5.1); 4 x 8192 x 2560 fp32 235 and 431 us (5.7, 5.5).  The
// vector unit follows: busy 59% of the forward and 73% of the backward (31 and 72
// instructions for 64 values, five and eight of them transcendental, at a quarter of the
// rate).  Odd rows of fp32 with starts (3 x 4099 x 1001) run at 4 TB/s.
//
// These are layers whose decays are slow (k up to kPolySmall).  A wave with a faster
// channel takes the general code, for all of its channels the same time whether one of
// them is fast or all: 4 x 8192 x 5120 bf16 270 and 553 us, 131072 x 2560 forward 562,
// 4 x 8192 x 2560 fp32 244 and 437, 3 x 4099 x 1001 54 and 86 (slow: 52 and 87).
//
// Up to 128 steps the forward is a single launch of 5.5 us, and so is the backward of up
// to 64 steps of one batch row; more steps take a launch more to clear the words that
// pieces hand on, and dlam from more than one piece or row one to sum it.
#include "launch.hpp"
#include "norm_common.hpp"
#include "recurrence.hpp"

namespace mss {
namespace {

// ------------------------------------------------------------ pieces in order
// A piece is one workgroup's steps of one stream (64 V channels of a batch row).
// Pieces take their place in order of start (a ticket): s-th in its stream, all
// s-th of a share of the streams before any (s+1)-th of it.  A piece that has its own A and H publishes
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
constexpr uint32_t kUnset = 0xffffffffu, kNaN = 0x7fc00000u, kCutMark = 0x7fc0c0c0u;
constexpr int kGroup = 8;  // pieces
constexpr int kChainHeader = 64;  // bytes before the values: status word, tickets

struct Chain {
  int* status;    // null: one piece a stream, nothing is handed on
  int* ticket;    // one for each share of the streams
  uint64_t* own;  // [place][stream][64 V]: A, H
  float* end;     // [place][stream][64 V]
  uint64_t* group_own;  // [group][stream][64 V], or null: no groups
  float* group_end;
  uint32_t streams;
  uint32_t shares;      // of the streams: 1, or one for each die
  uint32_t each, more;  // streams of a share, and how many shares have one more
};

// Status word and tickets to 0, the rest (n times 16 bytes) to unset.
__global__ void __launch_bounds__(256) chain_clear_kernel(u32x4* p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const uint32_t v = i < kChainHeader / 16 ? 0u : kUnset;
    p[i] = u32x4{v, v, v, v};
  }
}

__device__ __forceinline__ uint32_t set_bits(float v) {
  const uint32_t u = __float_as_uint(v);
  return u == kUnset ? kNaN : u;
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

// Never expected; keeps every wait finite, reported through the status word.
__device__ __forceinline__ bool gives_up(const Chain& c, int spins) {
  if (spins <= kMaxSpinsChain) return false;
  if ((threadIdx.x & 63) == 0) __hip_atomic_store(c.status, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return true;
}

// Mostly the piece before has ended (a first look at four places: 2 x 16384 x 5120
// backward 556 us, with one at one place 523; with 20 streams or fewer the same).
template <int V>
__device__ __forceinline__ void chain_wait(const Chain& c, int place, int stream, float (&carry)[V]) {
  bool found = chain_look<V, 1>(c, place, stream, carry);
  for (int spins = 0; !found; ++spins) {
    found = chain_look<V, 4>(c, place, stream, carry);
    if (!found && gives_up(c, spins)) {
#pragma unroll
      for (int v = 0; v < V; ++v) carry[v] = 0.0f;
      break;
    }
  }
}

// What enters the piece at `place` of `stream` (wave 0's lanes; `first` the stream),
// given its own A and H; publishes what later pieces need.  `cut`: a sequence
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
    chain_wait<V>(c, place, stream, carry);
  }
  if (cut || last) return;
  float h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = __builtin_fmaf(own_a[v], carry[v], own_h[v]);
  put_end<V>(c.end + off, h);
}

// The same with few streams, where the way of a state from piece to piece is what
// takes the time (a look is a trip to memory, and one brings it four pieces on).  Eight
// pieces are a group, whose A and H its last piece forms and hands on as above, so a
// look brings a state four groups on; inside its group a piece folds what is before it.
// Each of these folds, too, is always the same.  A piece in which a sequence starts has
// a mark for its A.
template <int V>
__device__ __forceinline__ void group_fold(const Chain& c, int from, int n, int stream, float (&a)[V], float (&x)[V],
                                           bool& cut) {
  uint64_t own[4][V];
  for (int spins = 0;; ++spins) {
    bool there = true;
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int64_t off = ((int64_t)(from + (q < n ? q : 0)) * c.streams + stream) * (64 * V);
        own[q][v] = __hip_atomic_load(c.own + off + (threadIdx.x & 63) * V + v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        there = there && is_set(own[q][v]);
      }
    if (__all(there) || gives_up(c, spins)) break;
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (q >= n) continue;
    const bool mark = __any((uint32_t)own[q][0] == kCutMark);
    cut = cut || mark;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float pa = __uint_as_float((uint32_t)own[q][v]), px = __uint_as_float((uint32_t)(own[q][v] >> 32));
      x[v] = mark ? px : __builtin_fmaf(pa, x[v], px);
      a[v] *= pa;
    }
  }
}
template <int V>
__device__ __forceinline__ void group_carry(const Chain& c, int place, int stream, bool last, bool cut,
                                            const float (&own_a)[V], const float (&own_h)[V], const float (&first)[V],
                                            float (&carry)[V]) {
  const int group = place / kGroup, before = place % kGroup;
  const int64_t lane = (threadIdx.x & 63) * V;
  if (!last) {
    const float mark = __uint_as_float(kCutMark);
    float pa[V];
#pragma unroll
    for (int v = 0; v < V; ++v) pa[v] = cut ? mark : __float_as_uint(own_a[v]) == kCutMark ? __uint_as_float(kNaN) : own_a[v];
    put_own<V>(c.own + ((int64_t)place * c.streams + stream) * (64 * V) + lane, pa, own_h);
  }
  float a[V], x[V];
#pragma unroll
  for (int v = 0; v < V; ++v) a[v] = 1.0f, x[v] = 0.0f;
  bool apart = false;  // a sequence starts in the group, before this piece
  for (int q = 0; q < before; q += 4)
    group_fold<V>(c, group * kGroup + q, before - q < 4 ? before - q : 4, stream, a, x, apart);
  const bool hands = before == kGroup - 1 && !last;
  const int64_t off = ((int64_t)group * c.streams + stream) * (64 * V) + lane;
  float ga[V], gx[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    ga[v] = a[v] * own_a[v];
    gx[v] = cut ? own_h[v] : __builtin_fmaf(own_a[v], x[v], own_h[v]);
  }
  if (hands && (apart || cut)) put_end<V>(c.group_end + off, gx);
  else if (hands && group > 0) put_own<V>(c.group_own + off, ga, gx);
  if (apart) {
#pragma unroll
    for (int v = 0; v < V; ++v) carry[v] = x[v];
    return;
  }
  float enters[V];
  if (group == 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) enters[v] = first[v];
  } else {
    Chain g = c;
    g.own = c.group_own;
    g.end = c.group_end;
    chain_wait<V>(g, group, stream, enters);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    carry[v] = __builtin_fmaf(a[v], enters[v], x[v]);
    gx[v] = __builtin_fmaf(ga[v], enters[v], gx[v]);
  }
  if (hands && !cut) put_end<V>(c.group_end + off, gx);
}

// Which piece a workgroup works on.  Neighbouring workgroups start on different dies,
// each with a cache of its own, while a row's neighbouring channels have lines in common
// where rows are not whole lines.  So each die has a share of neighbouring streams, and
// takes from another's when its own has run out (there are as many pieces as
// workgroups: each finds one).  Only the speed depends on which die a workgroup runs on.
struct Turn {
  int place, stream;
};
constexpr uint32_t kDies = 8;
__device__ __forceinline__ Turn take_turn(const Chain& c, uint32_t pieces, Turn* lds) {
  const auto first = [&](uint32_t g) { return g * c.each + (g < c.more ? g : c.more); };
  const uint32_t mask = c.shares - 1, own = blockIdx.x & mask;
  if (c.status == nullptr) return Turn{0, (int)(first(own) + (blockIdx.x >> __popc(mask)))};
  if (threadIdx.x == 0) {
    for (uint32_t i = 0; i < c.shares; ++i) {
      const uint32_t g = (own + i) & mask, n = c.each + (g < c.more);
      if (n == 0) continue;
      const uint32_t t = (uint32_t)atomicAdd(c.ticket + g, 1);
      if (t < n * pieces) {
        const uint32_t place = t / n;
        *lds = Turn{(int)place, (int)(first(g) + t - place * n)};
        break;
      }
    }
  }
  __syncthreads();
  return Turn{__builtin_amdgcn_readfirstlane(lds->place), __builtin_amdgcn_readfirstlane(lds->stream)};
}

// ------------------------------------------------------------ rows
// Rows r0, r0 + 1, .. of a tensor, one descriptor each (its base in scalar
// registers, a lane's channel as the offset: no address arithmetic in the vector
// unit).  A row's bytes fit 32 bits.
template <bool BF16>
struct Rows {
  char* at;
  int64_t step;
  uint32_t bytes;
  __device__ __forceinline__ Rows(const void* p, int64_t r0, int64_t stride, int64_t dim)
      : at(static_cast<char*>(const_cast<void*>(p)) + r0 * stride * (BF16 ? 2 : 4)),
        step(stride * (BF16 ? 2 : 4)),
        bytes((uint32_t)dim * (BF16 ? 2 : 4)) {}
  __device__ __forceinline__ rsrc_t row(int j) const { return make_rsrc(at + j * step, bytes); }
};

// V neighbouring channels as loaded: two bf16 in a word, or one value.  Of T rows
// only n exist; the rest read as `none`.
template <bool BF16, int V, int T>
__device__ __forceinline__ void load_rows(const Rows<BF16>& r, uint32_t off, int n, uint32_t none, uint32_t (&raw)[T]) {
  const auto load = [&](int j) -> uint32_t {
    if constexpr (BF16 && V == 1) return buf_load_u16(r.row(j), off);
    else return buf_load_u32(r.row(j), off);
  };
  if (n == T) {
#pragma unroll
    for (int j = 0; j < T; ++j) raw[j] = load(j);
  } else {
#pragma unroll
    for (int j = 0; j < T; ++j) raw[j] = j < n ? load(j < n ? j : 0) : none;
  }
}
// Gates of minus infinity and inputs of zero make a step that changes nothing.
template <bool BF16>
constexpr uint32_t kClosed = BF16 ? 0xff80ff80u : 0xff800000u;

template <bool BF16, int V>
__device__ __forceinline__ float widen_at(uint32_t w, int v) {
  if constexpr (!BF16) return __uint_as_float(w);
  else return v == 0 ? bf16_lo(w) : bf16_hi(w);
}
// Stores that do not take the place of what is read next in the caches (backward of 8 x
// 2048 x 1536: 93 -> 80 us, 4 x 8192 x 5120: 507 -> 502), for whole lines; parts of lines
// go to memory one by one then.
constexpr int kNonTemporal = 2;
// Rows past the n-th are not stored, nor what a lane without channels has.
template <bool BF16, int V, int AUX>
__device__ __forceinline__ void store_row(const Rows<BF16>& r, int j, int n, uint32_t off, const float (&o)[V]) {
  const rsrc_t d = make_rsrc(r.at + j * r.step, j < n ? r.bytes : 0u);
  if constexpr (BF16 && V == 1) {
    buf_store_u16(d, off, f32_to_bf16(o[0]));
  } else {
    uint32_t v;
    if constexpr (BF16) v = pack_bf16x2(o[0], o[1]);
    else v = __float_as_uint(o[0]);
    __builtin_amdgcn_raw_buffer_store_b32(v, d, (int)off, 0, AUX);
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
  bool any_rate;     // the workgroup takes the polynomial for all decays whatever its channels'
  uint32_t in, out;  // its offset in a row for loads, and for stores
};

// `piece` in order along time.  A lane past the last channel repeats it, and so does
// one with half a pair, as the second of the last two: what two lanes write there is
// the same.  Where that one is alone in its workgroup the other of the two belongs to
// the workgroup before as well, and both have to take the same polynomial.
template <bool BF16, int V, int W, int T>
__device__ __forceinline__ WavePlace<V, W, T> wave_place(Turn turn, int blocks, int64_t pieces, bool reversed,
                                                         int64_t seqlen, int64_t dim) {
  WavePlace<V, W, T> w;
  w.place = turn.place;
  w.stream = turn.stream;
  w.wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  w.b = w.stream / blocks;
  const int64_t piece = reversed ? pieces - 1 - w.place : w.place;
  w.t0 = piece * (W * T) + w.wave * T;
  const int64_t left = seqlen - w.t0;
  w.n = left < 0 ? 0 : left < T ? __builtin_amdgcn_readfirstlane((int)left) : T;
  const int64_t c = (int64_t)(w.stream - (int)w.b * blocks) * (64 * V) + (threadIdx.x & 63) * V;
  w.ok = c < dim;
  w.ch = (uint32_t)(c + V <= dim ? c : dim - V);
  w.in = w.ch * (BF16 ? 2u : 4u);
  w.out = w.ok ? w.in : kOffNone;
  w.any_rate = V == 2 && dim % (64 * V) == 1 && w.stream - (int)w.b * blocks >= blocks - 2;
  return w;
}

// Whether a sequence starts at the wave's step `lane` (the load comes before the
// rows', so that it is not waited for behind them); bit j of the wave's: at step j.
__device__ __forceinline__ uint32_t start_mark(const uint8_t* starts, int64_t row, int n) {
  const int lane = threadIdx.x & 63;
  return lane < n ? starts[row + lane] : 0u;
}

// Bit i: a sequence starts in wave i's steps.
template <int W>
__device__ __forceinline__ uint32_t cut_bits(const int* lds_cut) {
  return (uint32_t)__ballot(lds_cut[threadIdx.x & (W - 1)] != 0) & ((1u << W) - 1);
}

// Folds the waves lo .. hi - 1, in order (REVERSED: from the last), onto (a, x):
// x <- A x + X, a <- A a; where a sequence starts x is X alone (and a has no
// meaning any more).  Four waves' values are read at a time: one after the other
// the fold would take eight times LDS's latency.
template <int V, int W, bool REVERSED>
__device__ __forceinline__ void fold_waves(const float (*lds_a)[64 * V], const float (*lds_x)[64 * V], uint32_t cuts,
                                           int lo, int hi, float (&a)[V], float (&x)[V]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int g = 0; g < W; g += 4) {
    float la[4][V], lx[4][V];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int i = REVERSED ? W - 1 - g - q : g + q;
#pragma unroll
      for (int v = 0; v < V; ++v) la[q][v] = lds_a[i][lane * V + v], lx[q][v] = lds_x[i][lane * V + v];
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int i = REVERSED ? W - 1 - g - q : g + q;
      if (i < lo || i >= hi) continue;
      const bool cut = cuts >> i & 1;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        x[v] = cut ? lx[q][v] : __builtin_fmaf(la[q][v], x[v], lx[q][v]);
        a[v] *= la[q][v];
      }
    }
  }
}

// ------------------------------------------------------------ forward
struct FwdArgs {
  RecurrenceFwdParams p;
  Chain chain;
  int blocks;      // of channels
  int64_t pieces;  // of a stream
};

// GROUPS apart: in one kernel each would cost the other registers (131072 x 512 bf16
// backward 266 us, so 258).
template <bool BF16, int V, int W, int T, bool STARTS, bool GROUPS>
__global__ void __launch_bounds__(W * 64) __attribute__((amdgpu_waves_per_eu(4))) recurrence_fwd_kernel(FwdArgs a) {
  __shared__ float lds_a[W][64 * V], lds_h[W][64 * V], lds_carry[64 * V];
  __shared__ int lds_cut[W];
  __shared__ Turn lds_turn;
  const RecurrenceFwdParams& p = a.p;
  const Turn turn = take_turn(a.chain, (uint32_t)a.pieces, &lds_turn);
  if (a.chain.status == nullptr && blockIdx.x == 0 && threadIdx.x == 0)
    *static_cast<int*>(p.workspace) = 0;  // the status word: nothing waits
  const auto w = wave_place<BF16, V, W, T>(turn, a.blocks, a.pieces, false, p.seqlen, p.dim);
  const int lane = threadIdx.x & 63;
  const int64_t row0 = w.b * p.seqlen + w.t0;

  const uint32_t mark = STARTS ? start_mark(p.starts, row0, w.n) : 0u;
  float lam[V];
#pragma unroll
  for (int v = 0; v < V; ++v) lam[v] = p.lam[w.ch + v];
  uint32_t rx[T], ra[T], ri[T];
  load_rows<BF16, V, T>(Rows<BF16>(p.gate_a, row0, p.gate_a_stride, p.dim), w.in, w.n, kClosed<BF16>, ra);
  load_rows<BF16, V, T>(Rows<BF16>(p.gate_x, row0, p.gate_x_stride, p.dim), w.in, w.n, kClosed<BF16>, ri);
  load_rows<BF16, V, T>(Rows<BF16>(p.x, row0, p.x_stride, p.dim), w.in, w.n, 0u, rx);
  const uint64_t starts = STARTS ? __ballot(mark != 0) : 0;
  float k[V];
  bool slow = !w.any_rate;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    k[v] = decay_rate(p.c, lam[v]);
    slow = slow && k[v] <= kPolySmall;
  }

  // From a zero state: after each step the state and the product of the decays.
  float pr[T][V], hl[T][V], ha[V], hh[V];
#pragma unroll
  for (int v = 0; v < V; ++v) ha[v] = 1.0f, hh[v] = 0.0f;
  const auto local = [&](auto small) {
#pragma unroll
    for (int j = 0; j < T; ++j) {
      const bool start = STARTS && (starts >> j & 1);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float m = decay_of<small(), !BF16>(k[v] * sigmoid_of<!BF16>(widen_at<BF16, V>(ra[j], v)));
        const float u = beta_of(rest_of<small()>(m)) * sigmoid_of<!BF16>(widen_at<BF16, V>(ri[j], v));
        hh[v] = __builtin_fmaf(u, widen_at<BF16, V>(rx[j], v), start ? 0.0f : decayed<small()>(m, hh[v]));
        ha[v] = decayed<small()>(m, ha[v]);
        hl[j][v] = hh[v];
        pr[j][v] = ha[v];
      }
      if (j % 2 == 1) __builtin_amdgcn_sched_barrier(0);  // in the order that the loads arrive (275 -> 270 us)
    }
  };
  if (__all(slow)) local(std::true_type{});
  else local(std::false_type{});
#pragma unroll
  for (int v = 0; v < V; ++v) lds_a[w.wave][lane * V + v] = ha[v], lds_h[w.wave][lane * V + v] = hh[v];
  if (STARTS && lane == 0) lds_cut[w.wave] = starts != 0;
  __syncthreads();
  const uint32_t cuts = STARTS ? cut_bits<W>(lds_cut) : 0u;

  if (w.wave == 0) {
    float first[V], carry[V];
#pragma unroll
    for (int v = 0; v < V; ++v) first[v] = p.h0 != nullptr && w.place < kGroup ? p.h0[w.b * p.dim + w.ch + v] : 0.0f;
    if (a.chain.status == nullptr) {
#pragma unroll
      for (int v = 0; v < V; ++v) carry[v] = first[v];
    } else {
      fold_waves<V, W, false>(lds_a, lds_h, cuts, 1, W, ha, hh);
      if constexpr (!GROUPS)
        chain_carry<V>(a.chain, w.place, w.stream, w.place + 1 == a.pieces, cuts != 0, ha, hh, first, carry);
      else
        group_carry<V>(a.chain, w.place, w.stream, w.place + 1 == a.pieces, cuts != 0, ha, hh, first, carry);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) lds_carry[lane * V + v] = carry[v], ha[v] = 1.0f, hh[v] = 0.0f;
  } else {  // from the piece's first step to the wave's
#pragma unroll
    for (int v = 0; v < V; ++v) ha[v] = 1.0f, hh[v] = 0.0f;
    fold_waves<V, W, false>(lds_a, lds_h, cuts, 0, w.wave, ha, hh);
  }
  __syncthreads();

  if (w.n == 0) return;
  float q[V];
  const bool apart = (cuts & ((1u << w.wave) - 1)) != 0;
#pragma unroll
  for (int v = 0; v < V; ++v) q[v] = apart ? hh[v] : __builtin_fmaf(ha[v], lds_carry[lane * V + v], hh[v]);
  if (p.states != nullptr && w.ok && w.t0 % kRecurrenceChunk == 0) {
    const int64_t chunks = (p.seqlen + kRecurrenceChunk - 1) / kRecurrenceChunk;
#pragma unroll
    for (int v = 0; v < V; ++v) p.states[(w.b * chunks + w.t0 / kRecurrenceChunk) * p.dim + w.ch + v] = q[v];
  }
  const Rows<BF16> y(p.y, row0, p.y_stride, p.dim);
#pragma unroll
  for (int j = 0; j < T; ++j) {
    const bool cut = STARTS && (starts & ((2ull << j) - 1)) != 0;
    float o[V];
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = cut ? hl[j][v] : __builtin_fmaf(pr[j][v], q[v], hl[j][v]);
    store_row<BF16, V, kNonTemporal>(y, j, w.n, w.out, o);
    if (p.h_last != nullptr && w.ok && w.t0 + j == p.seqlen - 1)
#pragma unroll
      for (int v = 0; v < V; ++v) p.h_last[w.b * p.dim + w.ch + v] = o[v];
  }
}

// ------------------------------------------------------------ backward
struct BwdArgs {
  RecurrenceBwdParams p;
  Chain chain;
  float* part;     // [batch][pieces][dim]
  int blocks;
  int64_t pieces;
};

// Least beta^2 whose reciprocal root is taken: below, what it is multiplied by is next to
// nothing or 0, which must not meet an infinity.
constexpr float kLeastNormal = 1.1754944e-38f;

// One piece is one chunk: W T = kRecurrenceChunk.  Of a step, m and h_{t-1} stay in
// registers until the gradients, the gates' exponentials in LDS (each lane its
// own).  With w = dx x:
//   dx = g i beta,  dgate_x = w (1 - i),  G = s a (a w / beta^2 - g h_{t-1}).
template <bool BF16, int V, int W, int T, bool STARTS, int AUX, bool GROUPS>
__global__ void __launch_bounds__(W * 64) __attribute__((amdgpu_waves_per_eu(4))) recurrence_bwd_kernel(BwdArgs a) {
  static_assert(W * T == kRecurrenceChunk, "");
  extern __shared__ __align__(16) float lds_kept[];  // [2][W][T][64 V]
  __shared__ float lds_a[W][64 * V], lds_h[W][64 * V], lds_e[W][64 * V], lds_carry[64 * V];
  __shared__ int lds_cut[W];
  __shared__ Turn lds_turn;
  const RecurrenceBwdParams& p = a.p;
  const Turn turn = take_turn(a.chain, (uint32_t)a.pieces, &lds_turn);
  if (a.chain.status == nullptr && blockIdx.x == 0 && threadIdx.x == 0)
    *static_cast<int*>(p.workspace) = 0;  // the status word: nothing waits
  const auto w = wave_place<BF16, V, W, T>(turn, a.blocks, a.pieces, true, p.seqlen, p.dim);
  const int lane = threadIdx.x & 63;
  const int64_t row0 = w.b * p.seqlen + w.t0, piece = a.pieces - 1 - w.place;

  const uint32_t mark = STARTS ? start_mark(p.starts, row0, w.n) : 0u;
  float lam[V], before[V];  // before: the state entering the piece, then this wave's steps
#pragma unroll
  for (int v = 0; v < V; ++v) {
    lam[v] = p.lam[w.ch + v];
    before[v] = p.states[(w.b * a.pieces + piece) * p.dim + w.ch + v];
  }
  uint32_t rx[T], ra[T], ri[T], rd[T];
  load_rows<BF16, V, T>(Rows<BF16>(p.gate_a, row0, p.gate_a_stride, p.dim), w.in, w.n, kClosed<BF16>, ra);
  load_rows<BF16, V, T>(Rows<BF16>(p.gate_x, row0, p.gate_x_stride, p.dim), w.in, w.n, kClosed<BF16>, ri);
  load_rows<BF16, V, T>(Rows<BF16>(p.x, row0, p.x_stride, p.dim), w.in, w.n, 0u, rx);
  load_rows<BF16, V, T>(Rows<BF16>(p.dy, row0, p.dy_stride, p.dim), w.in, w.n, 0u, rd);
  const uint64_t starts = STARTS ? __ballot(mark != 0) : 0;
  float k[V];
  bool slow = !w.any_rate;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    k[v] = decay_rate(p.c, lam[v]);
    slow = slow && k[v] <= kPolySmall;
  }

  // From a zero state forwards (hl); what the gradients of dy here leave behind, e =
  // sum a_0 .. a_j dy_j up to a start.
  typedef float vec __attribute__((ext_vector_type(V)));
  vec* const exp_a = reinterpret_cast<vec*>(lds_kept) + w.wave * (T * 64) + lane;
  vec* const exp_x = exp_a + W * T * 64;
  float m[T][V], hl[T][V], ha[V], hh[V], e[V];
#pragma unroll
  for (int v = 0; v < V; ++v) ha[v] = 1.0f, hh[v] = 0.0f, e[v] = 0.0f;
  const auto local = [&](auto small) {
#pragma unroll
    for (int j = 0; j < T; ++j) {
      const bool start = STARTS && (starts >> j & 1), cut = STARTS && (starts & ((2ull << j) - 1)) != 0;
      vec ea, ex;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        ea[v] = exp_neg<!BF16>(widen_at<BF16, V>(ra[j], v));
        ex[v] = exp_neg<!BF16>(widen_at<BF16, V>(ri[j], v));
        m[j][v] = decay_of<small(), !BF16>(k[v] * rcp_fast(1.0f + ea[v]));
        hh[v] = __builtin_fmaf(beta_of(rest_of<small()>(m[j][v])) * rcp_fast(1.0f + ex[v]), widen_at<BF16, V>(rx[j], v),
                               start ? 0.0f : decayed<small()>(m[j][v], hh[v]));
        ha[v] = decayed<small()>(m[j][v], ha[v]);
        e[v] = cut ? e[v] : __builtin_fmaf(ha[v], widen_at<BF16, V>(rd[j], v), e[v]);
        hl[j][v] = hh[v];
      }
      exp_a[j * 64] = ea;
      exp_x[j * 64] = ex;
    }
  };
  if (__all(slow)) local(std::true_type{});
  else local(std::false_type{});
#pragma unroll
  for (int v = 0; v < V; ++v) {
    lds_a[w.wave][lane * V + v] = ha[v];
    lds_h[w.wave][lane * V + v] = hh[v];
    lds_e[w.wave][lane * V + v] = e[v];
  }
  if (STARTS && lane == 0) lds_cut[w.wave] = starts != 0;
  __syncthreads();
  const uint32_t cuts = STARTS ? cut_bits<W>(lds_cut) : 0u;

  float ea[V], ee[V];  // from the piece's last step to the wave's
#pragma unroll
  for (int v = 0; v < V; ++v) ea[v] = 1.0f, ee[v] = 0.0f;
  fold_waves<V, W, true>(lds_a, lds_e, cuts, w.wave + 1, W, ea, ee);
  if (w.wave == 0) {
    float first[V], carry[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
      first[v] = p.dh_last != nullptr && w.place < kGroup ? p.dh_last[w.b * p.dim + w.ch + v] : 0.0f;
    if (a.chain.status == nullptr) {
#pragma unroll
      for (int v = 0; v < V; ++v) carry[v] = first[v];
    } else {
      float pa[V], pe[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        pa[v] = ha[v] * ea[v];
        pe[v] = starts != 0 ? e[v] : __builtin_fmaf(ha[v], ee[v], e[v]);
      }
      if constexpr (!GROUPS)
        chain_carry<V>(a.chain, w.place, w.stream, w.place + 1 == a.pieces, cuts != 0, pa, pe, first, carry);
      else
        group_carry<V>(a.chain, w.place, w.stream, w.place + 1 == a.pieces, cuts != 0, pa, pe, first, carry);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) lds_carry[lane * V + v] = carry[v];
  }
  // The states before each step, from the one that enters the piece.
  fold_waves<V, W, false>(lds_a, lds_h, cuts, 0, w.wave, ha, before);
  float q[V];
#pragma unroll
  for (int v = 0; v < V; ++v) q[v] = before[v];
  const auto states = [&](auto small) {
#pragma unroll
    for (int j = 0; j < T; ++j) {
      const bool start = STARTS && (starts >> j & 1);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        q[v] = start ? 0.0f : decayed<small()>(m[j][v], q[v]);
        hl[j][v] += q[v];
      }
    }
  };
  if (__all(slow)) states(std::true_type{});
  else states(std::false_type{});
  __syncthreads();

  const bool apart = (cuts >> w.wave >> 1) != 0;
#pragma unroll
  for (int v = 0; v < V; ++v) e[v] = apart ? ee[v] : __builtin_fmaf(ea[v], lds_carry[lane * V + v], ee[v]);
  // Widened again from here on: values kept wide would not fit the registers.
#pragma unroll
  for (int j = 0; j < T; ++j) asm volatile("" : "+v"(rx[j]), "+v"(rd[j]));
  float dlam[V];
#pragma unroll
  for (int v = 0; v < V; ++v) dlam[v] = 0.0f;
  const Rows<BF16> dx(p.dx, row0, p.dx_stride, p.dim), da(p.dgate_a, row0, p.dgate_a_stride, p.dim),
      di(p.dgate_x, row0, p.dgate_x_stride, p.dim);
  const auto gradients = [&](auto small) {
#pragma unroll
    for (int j = T - 1; j >= 0; --j) {
      const bool start = STARTS && (starts >> j & 1);
      float ox[V], oa[V], oi[V];
      const vec ka = exp_a[j * 64], kx = exp_x[j * 64];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float rest_r, rest_i;
        const float r = sigmoid_from(ka[v], rest_r), i = sigmoid_from(kx[v], rest_i);
        const float n = rest_of<small()>(m[j][v]), dec = factor_of<small()>(m[j][v]), beta2 = __builtin_fmaf(-n, dec, -n);
        const float inv = __builtin_amdgcn_rsqf(__builtin_amdgcn_fmed3f(beta2, kLeastNormal, 2.0f));
        const float g = widen_at<BF16, V>(rd[j], v) + e[v];
        const float prev = j > 0 ? hl[j > 0 ? j - 1 : 0][v] : before[v];
        ox[v] = g * i * (beta2 * inv);
        const float wx = ox[v] * widen_at<BF16, V>(rx[j], v);
        oi[v] = wx * rest_i;
        const float big = k[v] * r * dec * __builtin_fmaf(dec * (inv * inv), wx, start ? 0.0f : -g * prev);
        oa[v] = big * rest_r;
        dlam[v] += j < w.n ? big : 0.0f;
        e[v] = start ? 0.0f : decayed<small()>(m[j][v], g);
      }
      store_row<BF16, V, AUX>(dx, j, w.n, w.out, ox);
      store_row<BF16, V, AUX>(da, j, w.n, w.out, oa);
      store_row<BF16, V, AUX>(di, j, w.n, w.out, oi);
      if (j % 2 == 0) __builtin_amdgcn_sched_barrier(0);  // no more than two steps at once: registers
    }
  };
  if (__all(slow)) gradients(std::true_type{});
  else gradients(std::false_type{});
  if (w.wave == 0 && piece == 0 && p.dh0 != nullptr && w.ok)
#pragma unroll
    for (int v = 0; v < V; ++v) p.dh0[w.b * p.dim + w.ch + v] = e[v];
  // (lds_h was last read before the barrier above.)
#pragma unroll
  for (int v = 0; v < V; ++v) lds_h[w.wave][lane * V + v] = dlam[v];
  __syncthreads();
  if (w.wave == 0 && w.ok) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < W; ++i) sum += lds_h[i][lane * V + v];
      a.part[(w.b * a.pieces + piece) * p.dim + w.ch + v] = sum * softplus_rate(lam[v], softplus_of(lam[v]));
    }
  }
}

// ------------------------------------------------------------ launch
// Longer pieces make a shorter chain, fewer waves shorter waits inside a workgroup: in
// an earlier form, 4 x 8192 x 5120 forward 291 us and 131072 x 2560 793 us; with 4 waves
// of 16 steps 323 and 1101, 8 of 8 328 and 1142, 16 of 8 393 and 940.  16 steps of the
// backward do not fit the registers.
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

// 131072 x 512 bf16 (4 streams) 238 us forward and 467 backward, with groups 137 and 258; 65536
// x 1001 fp32 (16) 242 and 471, 234 and 466; with 20 to 160 streams groups take up to 6% longer
// (4 x 8192 x 5120: 257 and 507, 269 and 539).
constexpr int64_t kFewStreams = 16, kManyPieces = 32;

hipError_t start_chain(const Cut& c, uint32_t shares, void* workspace, Chain& chain, hipStream_t stream) {
  char* base = static_cast<char*>(workspace);
  chain.streams = (uint32_t)c.streams;
  chain.group_own = nullptr;
  chain.shares = c.pieces == 1 ? kDies : shares;
  chain.each = chain.streams / chain.shares;
  chain.more = chain.streams % chain.shares;
  chain.status = nullptr;
  if (c.pieces == 1) return hipSuccess;
  chain.status = reinterpret_cast<int*>(base);
  chain.ticket = chain.status + 1;
  chain.own = reinterpret_cast<uint64_t*>(base + c.own);
  chain.end = reinterpret_cast<float*>(base + c.end);
  // Groups: their words take the place of the pieces' end states, of which there are none.
  const bool grouped = c.streams <= kFewStreams && c.pieces >= kManyPieces;
  const int64_t half = (int64_t)(c.bytes - c.end) / 2;
  chain.group_end = grouped ? chain.end : nullptr;
  chain.group_own = grouped ? reinterpret_cast<uint64_t*>(base + c.end + half) : nullptr;
  const int64_t n = (int64_t)(c.bytes / 16), groups = (n + 255) / 256;
  hipLaunchKernelGGL(chain_clear_kernel, dim3((unsigned)(groups < 2048 ? groups : 2048)), dim3(256), 0, stream,
                     reinterpret_cast<u32x4*>(base), n);
  return hipGetLastError();
}

// bf16 channels go in pairs, a word a lane, which the hardware reads and writes at any
// alignment (at odd ones, 3 x 4099 x 1001, 39 us forward and 61 us backward, against 43
// and 70 with one channel a lane); a row of one channel has none.
bool in_pairs(int64_t dim, bool bf16) { return bf16 && dim > 1; }

template <bool BF16, int V>
hipError_t launch_fwd(const RecurrenceFwdParams& p, hipStream_t stream) {
  const Cut c = cut_of(p.batch, p.seqlen, p.dim, V, kWaves * kFwdSteps);
  FwdArgs a{p, {}, (int)c.blocks, c.pieces};
  const hipError_t e = start_chain(c, 1, p.workspace, a.chain, stream);
  if (e != hipSuccess) return e;
  const auto kernel = a.chain.group_own != nullptr
                          ? p.starts != nullptr ? recurrence_fwd_kernel<BF16, V, kWaves, kFwdSteps, true, true>
                                                : recurrence_fwd_kernel<BF16, V, kWaves, kFwdSteps, false, true>
                          : p.starts != nullptr ? recurrence_fwd_kernel<BF16, V, kWaves, kFwdSteps, true, false>
                                                : recurrence_fwd_kernel<BF16, V, kWaves, kFwdSteps, false, false>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)(c.streams * c.pieces)), dim3(kWaves * 64), 0, stream, a);
  return hipGetLastError();
}

// Rows of which the 64 channels of a wave are whole half lines.
template <bool BF16>
bool whole_lines(const void* p, int64_t stride) {
  return ((reinterpret_cast<uintptr_t>(p) | (uint64_t)stride * (BF16 ? 2 : 4)) & 63u) == 0;
}
// Gradients of other rows.  A share of the streams for each die where there are many
// (25 to 100 MB a tensor: with 8 streams of fp32 shares take 9 to 14% more time, with 16 3
// to 9% more, 24 and 32 2% less to 6% more, 48 2 to 5% less, 64 10 to 11%, 264 8 to 14%;
// bf16 gains a third of that).  And plain stores for large tensors: up to 32 MB a tensor,
// all seven in the 256 MB cache, they take 0 to 7% less time; from 40 to 64 MB, where some
// of what is read next is still there, 9 to 21% more; from 80 MB on 6 to 23% less (24 to
// 160 MB of 2099 and 1001 fp32 and 1537 bf16 channels).  The rule takes the upper border.
// The forward, with one output beside three inputs, has neither: shares take up to 13% less
// with 48 streams and more and 80 MB or less, but 0 to 6% more from 100 MB on, and with
// fewer streams up to 19% more; plain stores 2% less to 13% more.
constexpr int64_t kManyStreams = 48, kNearBytes = 64ll << 20;

size_t bwd_part_offset(const Cut& c) { return (c.bytes + 255) / 256 * 256; }

template <bool BF16, int V>
hipError_t launch_bwd(const RecurrenceBwdParams& p, hipStream_t stream) {
  const Cut c = cut_of(p.batch, p.seqlen, p.dim, V, kRecurrenceChunk);
  // One piece of one row writes dlam itself.
  const int64_t parts = p.batch * c.pieces;
  float* part = reinterpret_cast<float*>(static_cast<char*>(p.workspace) + bwd_part_offset(c));
  BwdArgs a{p, {}, parts > 1 ? part : p.dlam, (int)c.blocks, c.pieces};
  const bool whole = whole_lines<BF16>(p.dx, p.dx_stride) && whole_lines<BF16>(p.dgate_a, p.dgate_a_stride) &&
                     whole_lines<BF16>(p.dgate_x, p.dgate_x_stride);
  hipError_t e = start_chain(c, !whole && c.streams >= kManyStreams ? kDies : 1, p.workspace, a.chain, stream);
  if (e != hipSuccess) return e;
  const bool past = whole || p.batch * p.seqlen * p.dim * (BF16 ? 2 : 4) <= kNearBytes;
  constexpr int kNT = kNonTemporal;
  const auto kernel = a.chain.group_own != nullptr
                          ? p.starts != nullptr ? recurrence_bwd_kernel<BF16, V, kWaves, kBwdSteps, true, kNT, true>
                                                : recurrence_bwd_kernel<BF16, V, kWaves, kBwdSteps, false, kNT, true>
                      : past
                          ? p.starts != nullptr ? recurrence_bwd_kernel<BF16, V, kWaves, kBwdSteps, true, kNT, false>
                                                : recurrence_bwd_kernel<BF16, V, kWaves, kBwdSteps, false, kNT, false>
                          : p.starts != nullptr ? recurrence_bwd_kernel<BF16, V, kWaves, kBwdSteps, true, 0, false>
                                                : recurrence_bwd_kernel<BF16, V, kWaves, kBwdSteps, false, 0, false>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)(c.streams * c.pieces)), dim3(kWaves * 64),
                     2 * kRecurrenceChunk * 64 * V * sizeof(float), stream, a);
  e = hipGetLastError();
  if (e != hipSuccess || parts == 1) return e;
  SumPartialsArgs s{};
  s.part = a.part;
  s.dweight = p.dlam;
  s.nparts = parts;
  s.cols = p.dim;
  s.nout = 1;
  return launch_sum_partials(s, stream);
}

}  // namespace

size_t recurrence_fwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim, bool bf16) {
  return cut_of(batch, seqlen, dim, in_pairs(dim, bf16) ? 2 : 1, kWaves * kFwdSteps).bytes;
}

hipError_t launch_recurrence_fwd(const RecurrenceFwdParams& p, hipStream_t stream) {
  if (!p.bf16) return launch_fwd<false, 1>(p, stream);
  return in_pairs(p.dim, true) ? launch_fwd<true, 2>(p, stream) : launch_fwd<true, 1>(p, stream);
}

size_t recurrence_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim, bool bf16) {
  const Cut c = cut_of(batch, seqlen, dim, in_pairs(dim, bf16) ? 2 : 1, kRecurrenceChunk);
  return bwd_part_offset(c) + (size_t)(batch * c.pieces * dim) * sizeof(float);
}

hipError_t launch_recurrence_bwd(const RecurrenceBwdParams& p, hipStream_t stream) {
  if (!p.bf16) return launch_bwd<false, 1>(p, stream);
  return in_pairs(p.dim, true) ? launch_bwd<true, 2>(p, stream) : launch_bwd<true, 1>(p, stream);
}

}  // namespace mss
