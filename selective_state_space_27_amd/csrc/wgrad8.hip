// Weight gradient of a linear layer whose input was kept in 8 bits (gfx950):
//   dW[o, i] = sum_t dY[t, o] X[t, i],  X = q 2^(e - 127)  (rows.hpp)
// on v_mfma_f32_32x32x16_bf16 with fp32 accumulation.  X's values are exact in
// bf16, so nothing is rounded before the products.
//
// Both operands lie with the summed axis t slow, so a tile of 32 steps is
// staged in LDS as it lies in memory (t-major), X widened on the way, and the
// matrix operands (eight steps of one column per lane) come out of LDS by
// transposing reads.  A staged row is cut into chunks of 64 bytes, chunk c of
// row t stored at c ^ (t % 4): the four rows that a transposing read touches
// then lie in different banks.
//
// What bounds it: the power that the matrix cores may draw.  With random operands
// the clock falls to 1.6 to 1.7 GHz of 2.4, by the card (matrix cores busy 71% of the
// cycles); with dY zero the same call, in the same cycles to 4%, runs at 2.0 GHz, with
// both zero at 2.24 GHz (1.50, 1.15 and 1.01 ms on one card).  256 x 256 tiles, eight
// waves of 128 x 64: a wave reads 6 KB of LDS for 8 products, so LDS (1026 cycles for
// 64 steps by its counter, reads and writes) stays well under the matrix cores'
// 2048.  With dY loaded straight into LDS five stages ahead, the next stage's first
// operands read before the barrier, and LDS reads and the widening of X issued
// between the products, 32768 x 10576 x 2560 takes 1.43 to 1.50 ms by the card,
// 1240 TFLOP/s at best (a bf16 matrix product of 8192^3 by the vendor's
// library, many in a row, reaches 1390, 1790 on zeros; its product of
// this very shape and layout 812).  On the way: 623 TFLOP/s with one stage ahead
// through registers, 665 without bounds checks inside, 886 with the transfers
// into LDS, 989 with their addresses kept instead of computed, 1033 and 1163 with
// the cut tiles' sums joined wider and cut less, 1203 with no LDS bank conflicts
// and the order of issue given, 1240 with the first loads in order and no
// branches at the end.
//
// Output tiles past the last full set of the card's CUs are cut along t into
// `splits` parts each, whose fp32 sums go to the workspace and are added in
// order by a second kernel: the result does not depend on scheduling.
#include <type_traits>

#include "launch.hpp"
#include "rows.hpp"
#include "ssd_common.hpp"

namespace mss {
namespace {

using ssd::f32x16;
using ssd::mfma;

constexpr int kDK = 32;  // steps of a stage

struct Args {
  const uint16_t* dy;
  const int8_t* q;
  const uint8_t* scale;
  void* dw;
  float* part;  // [cut][splits][BM][BN], 16-byte aligned
  int64_t dy_stride;
  int64_t tokens;
  int outs, ins, pitch;
  int acols;      // outs in whole vectors of eight: what a row of dy holds
  int mt, nt;     // tiles
  int whole;      // tiles taken whole, before the cut ones
  int splits;
  int stages;     // of all tokens
  bool dw_bf16, accumulate;
  int* status;
};

__device__ __forceinline__ void put(const Args& a, int64_t i, float v) {
  if (a.dw_bf16) {
    uint16_t* p = static_cast<uint16_t*>(a.dw) + i;
    *p = f32_to_bf16(a.accumulate ? bf16_to_f32(*p) + v : v);
  } else {
    float* p = static_cast<float*>(a.dw) + i;
    *p = a.accumulate ? *p + v : v;
  }
}

// Tile `i` of the order: bands of eight tile rows, column by column.
__host__ __device__ __forceinline__ void tile_at(int mt, int nt, int i, int& m, int& n) {
  const int band = i / (8 * nt), r = i - band * 8 * nt;
  const int left = mt - band * 8, rows = left < 8 ? left : 8;
  n = r / rows;
  m = band * 8 + r - n * rows;
}

// Byte offset of 16-byte slot `s` of staged row t of `width` bytes.
__device__ __forceinline__ int stage_slot(int t, int s, int width) {
  return t * width + ((((s >> 2) ^ (t & 3)) << 2 | (s & 3)) << 4);
}

// Eight (q, scale) as bf16: exact, so the high halves of the fp32 products.
__device__ __forceinline__ u32x4 widen_bf16(uint32_t w0, uint32_t w1, uint32_t e) {
  Raw<kSrcP8> r;
  r.a = u32x2{w0, w1};
  r.e = e;
  float v[8];
  widen<kSrcP8>(r, v);
  u32x4 o;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    o[j] = __builtin_amdgcn_perm(__float_as_uint(v[2 * j + 1]), __float_as_uint(v[2 * j]), 0x07060302u);
  return o;
}

// The tile and the stages of a workgroup.  Workgroups go to the eight XCDs in
// turn; each XCD takes a run of neighbouring tiles (bands of eight tile rows,
// column by column), so that the 32 it holds at a time share their operands in
// its L2.
struct Item {
  int m, n;         // tile
  int part;         // its part among the cut ones, or -1: the whole sum
  int first, last;  // stages
};
__device__ __forceinline__ int xcd_run(int b, int total) {
  const int x = b & 7, q = total >> 3, r = total & 7;
  return x * q + min(x, r) + (b >> 3);
}
__device__ __forceinline__ Item item_of(const Args& a) {
  Item it;
  int tile;
  if ((int)blockIdx.x < a.whole) {
    tile = xcd_run(blockIdx.x, a.whole);
    it.part = -1, it.first = 0, it.last = a.stages;
  } else {
    const int cut = a.mt * a.nt - a.whole, i = xcd_run(blockIdx.x - a.whole, cut * a.splits);
    const int s = i / cut;
    tile = i - s * cut;
    it.part = tile * a.splits + s;
    tile += a.whole;
    it.first = (int)((int64_t)a.stages * s / a.splits);
    it.last = (int)((int64_t)a.stages * (s + 1) / a.splits);
  }
  tile_at(a.mt, a.nt, tile, it.m, it.n);
  return it;
}

// f(i, j) for every tile, the indices constants (an accumulator stays in registers).
template <int TM, int TN, int I = 0, typename F>
__device__ __forceinline__ void each_tile(F&& f) {
  if constexpr (I < TM * TN) {
    f(std::integral_constant<int, I / TN>{}, std::integral_constant<int, I % TN>{});
    each_tile<TM, TN, I + 1>(f);
  }
}

// A wave's accumulators to dW, added to it with ACC: elements past dW's edges go to
// an offset past the descriptor's end, where loads give 0 and stores are dropped,
// so no element branches (with a branch for each, a 128 x 128 tile took 5.6 us).
template <bool BF16, bool ACC, int BM, int BN, int TM, int TN>
__device__ __forceinline__ void store_tile(const Args& a, const Item& it, const f32x16 (&acc)[TM][TN], int lm, int ln) {
  constexpr uint32_t kBytes = BF16 ? 2 : 4;
  const rsrc_t dst = make_rsrc(static_cast<char*>(a.dw) + (int64_t)it.m * BM * a.ins * kBytes, 0x7fffff00u);
  each_tile<TM, TN>([&](auto i, auto j) {
    const int m = lm + 32 * i.value, n = it.n * BN + ln + 32 * j.value;
    const int rows = n < a.ins ? a.outs - it.m * BM : 0;
    uint32_t off[16];
    float v[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int mr = m + 8 * (r >> 2) + (r & 3);
      off[r] = mr < rows ? ((uint32_t)mr * (uint32_t)a.ins + (uint32_t)n) * kBytes : kOffNone;
      v[r] = acc[i.value][j.value][r];
    }
    if constexpr (ACC) {
      float old[16];
#pragma unroll
      for (int r = 0; r < 16; ++r)
        old[r] = BF16 ? bf16_to_f32(buf_load_u16(dst, off[r])) : __uint_as_float(buf_load_u32(dst, off[r]));
#pragma unroll
      for (int r = 0; r < 16; ++r) v[r] += old[r];
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      if constexpr (BF16) buf_store_u16(dst, off[r], f32_to_bf16(v[r]));
      else buf_store_u32(dst, off[r], __float_as_uint(v[r]));
    }
  });
}

// A wave's accumulators: row 8 (r / 4) + r % 4 from lm, column ln of each 32 x 32 tile.
template <int BM, int BN, int TM, int TN>
__device__ __forceinline__ void write_tile(const Args& a, const Item& it, const f32x16 (&acc)[TM][TN], int lm, int ln) {
  if (it.part >= 0) {
    float* p = a.part + ((int64_t)it.part * BM + lm) * BN + ln;
    each_tile<TM, TN>([&](auto i, auto j) {
#pragma unroll
      for (int r = 0; r < 16; ++r)
        p[(32 * i.value + 8 * (r >> 2) + (r & 3)) * BN + 32 * j.value] = acc[i.value][j.value][r];
    });
    return;
  }
  if (a.dw_bf16) {
    if (a.accumulate) store_tile<true, true, BM, BN>(a, it, acc, lm, ln);
    else store_tile<true, false, BM, BN>(a, it, acc, lm, ln);
  } else {
    if (a.accumulate) store_tile<false, true, BM, BN>(a, it, acc, lm, ln);
    else store_tile<false, false, BM, BN>(a, it, acc, lm, ln);
  }
}

// dY's rows copied to aligned ones of whole vectors of eight (zeros past the
// last column), for rows that cannot go into LDS as they lie: 16-byte transfers
// need 16-byte aligned rows, and a last vector that ends with the row must not
// be read past it.  Reading and writing dY once costs less than the product
// through registers did: 32768 x 10575 x 2560 2.61 ms that way.
__global__ void __launch_bounds__(256) wgrad8_align_kernel(const uint16_t* src, int64_t stride, uint16_t* dst,
                                                           int64_t tokens, int outs, uint32_t vecs) {
  constexpr int kVecs = 4;
  const int64_t first = (int64_t)blockIdx.x * (256 * kVecs), row0 = first / vecs;
  const uint32_t rem0 = (uint32_t)(first - row0 * vecs);
  u32x4 v[kVecs];
  int64_t row[kVecs];
  int col[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const uint32_t t = rem0 + i * 256 + threadIdx.x, r = t / vecs;
    row[i] = row0 + r;
    col[i] = (int)(t - r * vecs) * 8;
    v[i] = load_raw<kSrcBf16>(src + row[i] * stride, nullptr, col[i], row[i] < tokens ? outs - col[i] : 0).a;
  }
#pragma unroll
  for (int i = 0; i < kVecs; ++i)
    if (row[i] < tokens) *reinterpret_cast<u32x4*>(dst + row[i] * ((int64_t)vecs * 8) + col[i]) = v[i];
}

// Instruction classes of __builtin_amdgcn_sched_group_barrier.
constexpr int kSchedValu = 0x002, kSchedMfma = 0x008, kSchedLdsRead = 0x100;
// vmcnt limit (bits 3:0 and 15:14), the other counters not waited for.
constexpr int vmcnt(int n) { return (n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8); }

// The products of a tile, WM x WN waves of TM x TN tiles of 32 x 32.  Six tiles of
// dY and three of X are staged; dY's rows are 16-byte aligned, whole vectors of
// eight and at most 2^23 elements apart.
template <int WM, int WN, int TM, int TN>
__global__ void __launch_bounds__(WM* WN * 64) wgrad8_kernel(Args a) {
  constexpr int BM = WM * TM * 32, BN = WN * TN * 32, WA = BM * 2, WB = BN * 2;
  constexpr int kTA = kDK * WA, kTX = kDK * WB;
  constexpr int kPieces = kTA / 1024 / (WM * WN);  // 1 KB transfers of a wave and stage
  static_assert(kTA % (1024 * WM * WN) == 0 && WM * WN * 64 * 16 == kDK * BN, "");
  // One array per staged tile: the compiler then knows which transfer a read may alias.
  __shared__ __align__(1024) unsigned char a0[kTA], a1[kTA], a2[kTA], a3[kTA], a4[kTA], a5[kTA];
  __shared__ __align__(1024) unsigned char x0[kTX], x1[kTX], x2[kTX];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  if (blockIdx.x == 0 && tid == 0) *a.status = 0;
  const Item it = item_of(a);
  const int m0 = it.m * BM, n0 = it.n * BN;
  const int64_t te = min((int64_t)it.last * kDK, a.tokens);  // end of this part's steps

  // This lane's offsets: of dY (row and 16-byte slot of piece wave + p waves), q and scale.
  uint32_t aoff[kPieces];
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {
    const int byte = (wave + p * WM * WN) * 1024 + lane * 16, t = byte / WA, pos = byte % WA / 16;
    aoff[p] = ((uint32_t)t * (uint32_t)a.dy_stride + ((((pos >> 2) ^ (t & 3)) << 2 | (pos & 3)) << 3)) * 2;
  }
  const int xt = tid / (BN / 16), xc = tid % (BN / 16) * 16, spitch = a.pitch >> 5;
  const uint32_t qoff = (uint32_t)xt * a.pitch + xc, soff = (uint32_t)xt * spitch + (xc >> 5);
  // X's two slots of a thread swap places in every other 128 bytes: eight lanes,
  // which write every second slot of 256 bytes, then meet all banks (20% of the
  // LDS cycles were conflicts without).
  const int xflip = (xc >> 6 & 1) << 4;
  const int xs0 = stage_slot(xt, xc / 8, WB) ^ xflip, xs1 = stage_slot(xt, xc / 8 + 1, WB) ^ xflip;

  // Where the next transfer of dY starts and the steps left from there, and the
  // same of X.  With 64 steps left, a stage's accesses end inside the tensors
  // however narrow they are (32 rows, and columns past the last one run on for
  // at most 32 rows more); with fewer, the descriptor ends with the part, and
  // what lies past it reads as zeros.
  const char* pa = reinterpret_cast<const char*>(a.dy + (int64_t)it.first * kDK * a.dy_stride + m0);
  const int8_t* pq = a.q + (int64_t)it.first * kDK * a.pitch + n0;
  const uint8_t* ps = a.scale + (int64_t)it.first * kDK * spitch + (n0 >> 5);
  int64_t left_a = te - (int64_t)it.first * kDK, left_x = left_a;  // not kept while `open`
  const int64_t step_a = a.dy_stride * (2 * kDK), step_q = (int64_t)a.pitch * kDK, step_s = (int64_t)spitch * kDK;
  constexpr uint32_t kOpen = 0x7fffff00u;
  auto load_a = [&](auto open, unsigned char* dst) {
    uint32_t bytes = kOpen;
    if constexpr (!open.value) {
      const int n = (int)max(min(left_a, (int64_t)64), (int64_t)0);
      if (n < 64) bytes = n == 0 ? 0u : ((uint32_t)(n - 1) * (uint32_t)a.dy_stride + (uint32_t)(a.acols - m0)) * 2u;
      left_a -= kDK;
    }
    const rsrc_t r = make_rsrc(pa, bytes);
#pragma unroll
    for (int p = 0; p < kPieces; ++p)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          r, (__attribute__((address_space(3))) void*)(dst + (wave + p * WM * WN) * 1024), 16, (int)aoff[p], 0, 0, 0);
    pa += step_a;
  };
  struct QRegs {
    u32x4 q;
    uint32_t e;
  };
  auto load_q = [&](auto open) {
    uint32_t qbytes = kOpen, sbytes = kOpen;
    if constexpr (!open.value) {
      const int n = (int)max(min(left_x, (int64_t)64), (int64_t)0);
      if (n < 64) {
        qbytes = n == 0 ? 0u : (uint32_t)(n * a.pitch - n0);
        sbytes = n == 0 ? 0u : (uint32_t)(n * spitch - (n0 >> 5));
      }
      left_x -= kDK;
    }
    const rsrc_t rq = make_rsrc(pq, qbytes), rs = make_rsrc(ps, sbytes);
    QRegs v;
    v.q = buf_load_u32x4(rq, qoff);
    v.e = __builtin_amdgcn_raw_buffer_load_b8(rs, (int)soff, 0, 0);
    pq += step_q, ps += step_s;
    return v;
  };
  auto put_x = [&](unsigned char* dst, const QRegs& v) {
    *reinterpret_cast<u32x4*>(dst + xs0) = widen_bf16(v.q[0], v.q[1], v.e);
    *reinterpret_cast<u32x4*>(dst + xs1) = widen_bf16(v.q[2], v.q[3], v.e);
  };

  f32x16 acc[TM][TN] = {};
  const int wm = wave / WN * (TM * 32), wn = wave % WN * (TN * 32);
  const int i16 = lane & 15, hf = lane >> 5, gc = (lane >> 4) & 1;
  typedef short v4s __attribute__((ext_vector_type(4)));
  const int frow = 8 * hf + (i16 >> 2), fsub = gc * 32 + (i16 & 3) * 8;
  int fca[TM], fcb[TN];  // offsets of the operand reads
#pragma unroll
  for (int i = 0; i < TM; ++i) fca[i] = frow * WA + (((wm >> 5) + i) ^ (i16 >> 2)) * 64 + fsub;
#pragma unroll
  for (int j = 0; j < TN; ++j)
    fcb[j] = frow * WB + (((wn >> 5) + j) ^ (i16 >> 2)) * 64 + (fsub ^ ((((wn >> 5) + j) >> 1 & 1) << 4));
  auto rd = [&](const unsigned char* p, int width) -> u32x4 {
    const u32x2 lo = __builtin_bit_cast(
        u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)(p)));
    const u32x2 hi = __builtin_bit_cast(
        u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)(p + 4 * width)));
    return u32x4{lo[0], lo[1], hi[0], hi[1]};
  };
  constexpr int kReads = 2 * (TM + TN);  // of one set of operands
  static_assert(kReads <= 15, "");
  struct Ops {
    u32x4 a[TM], b[TN];
  };
  // X before dY in a stage's loads: widening X then leaves three stages of dY in
  // flight instead of two (loads come back in order), which the short stages of
  // four waves need (8191 x 768 x 1536: 34 us, 36 the other way); with eight
  // waves the order of issue that it fixes costs more (32768 x 10576 x 2560: 1.48
  // ms, 1.43 the other way).
  constexpr bool kXFirst = WM * WN == 4;
  auto operands = [&](const unsigned char* sa, const unsigned char* sx, int kk) {
    Ops o;
#pragma unroll
    for (int i = 0; i < TM; ++i) o.a[i] = rd(sa + fca[i] + kk * 16 * WA, WA);
#pragma unroll
    for (int j = 0; j < TN; ++j) o.b[j] = rd(sx + fcb[j] + kk * 16 * WB, WB);
    return o;
  };
  auto products = [&](const Ops& o) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = mfma(o.a[i], o.b[j], acc[i][j]);
  };

  // Stage s of six (the arrays a stage uses are then constants).  On entry its
  // first operands are in registers, its other ones and those of stage s + 1
  // are staged once the barrier is passed, and dY of s + 2 .. s + 4 and q of s
  // + 2, s + 3 are on their way.
  QRegs q0, q1;
  Ops f0;
  auto stage = [&](auto open, unsigned char* sa, unsigned char* sx, unsigned char* sa1, unsigned char* sx1, unsigned char* sx2,
                   unsigned char* dst, QRegs& q) {
    // This wave's dY of stage s + 1 has landed (at least the loads of three stages
    // were issued after it), its X of s + 1 is written and all it read but the
    // operands just asked for (kReads, of tiles that stay) is in registers.  The
    // empty assembly keeps memory accesses on their side.
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((vmcnt(3 * (kPieces + 2)) & ~(15 << 8)) | (kReads << 8));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    const QRegs now = q;
    if constexpr (kXFirst) {
      q = load_q(open);
      asm volatile("" ::: "memory");
      load_a(open, dst);
    } else {
      load_a(open, dst);
      q = load_q(open);
    }
    const Ops f1 = operands(sa, sx, 1);
    products(f0);
    put_x(sx2, now);
    // Order of issue: the LDS reads between the first four products, most of the
    // widening between the other four.
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __builtin_amdgcn_sched_group_barrier(kSchedMfma, 1, 0);
      __builtin_amdgcn_sched_group_barrier(kSchedLdsRead, 3, 0);
      __builtin_amdgcn_sched_group_barrier(kSchedValu, 4, 0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __builtin_amdgcn_sched_group_barrier(kSchedMfma, 1, 0);
      __builtin_amdgcn_sched_group_barrier(kSchedValu, 8, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
    f0 = operands(sa1, sx1, 0);
    products(f1);
#pragma unroll
    for (int i = 0; i < 6; ++i) {
      __builtin_amdgcn_sched_group_barrier(kSchedMfma, 1, 0);
      __builtin_amdgcn_sched_group_barrier(kSchedLdsRead, 2, 0);
    }
  };
  const std::false_type bounded;
  // In this order: what a stage waits for counts the loads issued after it, and
  // the first stages' are these.  The empty assembly keeps it.
  const auto in_order = [] { asm volatile("" ::: "memory"); };
  load_a(bounded, a0);
  load_a(bounded, a1);
  {
    const QRegs p0 = load_q(bounded), p1 = load_q(bounded);
    in_order();
    load_a(bounded, a2);
    in_order();
    load_a(bounded, a3);
    in_order();
    q0 = load_q(bounded);
    in_order();
    load_a(bounded, a4);
    in_order();
    q1 = load_q(bounded);
    in_order();
    put_x(x0, p0);
    put_x(x1, p1);
  }
  // dY of the first two stages has landed (three transfers and two loads of X were
  // issued after it), their X is written.
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(vmcnt(3 * kPieces + 4) & ~(15 << 8));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  f0 = operands(a0, x0, 0);
  auto six = [&](auto open) {
    stage(open, a0, x0, a1, x1, x2, a5, q0);
    stage(open, a1, x1, a2, x2, x0, a0, q1);
    stage(open, a2, x2, a3, x0, x1, a1, q0);
    stage(open, a3, x0, a4, x1, x2, a2, q1);
    stage(open, a4, x1, a5, x2, x0, a3, q0);
    stage(open, a5, x2, a0, x0, x1, a4, q1);
  };
  // Six stages at a time (past the part's end with zeros): those whose
  // transfers, up to five stages ahead, have 64 steps left, then the rest.
  int st = it.first;
  const int open_end = (int)((te >> 5) - 12);
  for (; st < open_end; st += 6) six(std::true_type{});
  left_a = te - (int64_t)(st + 5) * kDK, left_x = te - (int64_t)(st + 4) * kDK;
  for (; st < it.last; st += 6) six(bounded);
  write_tile<BM, BN, TM, TN>(a, it, acc, wm + 4 * hf, wn + (lane & 31));
}

// The cut tiles: their parts added in order, four neighbouring sums a thread.
// grid (BM BN / 1024, tile), 256 threads.
template <int BM, int BN>
__global__ void __launch_bounds__(256) wgrad8_join_kernel(Args a) {
  int tm, tn;
  tile_at(a.mt, a.nt, a.whole + blockIdx.y, tm, tn);
  const int i = (blockIdx.x * 256 + threadIdx.x) * 4, m = tm * BM + i / BN, n = tn * BN + i % BN;
  if (m >= a.outs || n >= a.ins) return;
  const float* p = a.part + (int64_t)blockIdx.y * a.splits * (BM * BN) + i;
  f32x4 v = {};
  for (int s = 0; s < a.splits; s += 8) {
    f32x4 t[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      t[j] = s + j < a.splits
                 ? __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p + (int64_t)(s + j) * (BM * BN)))
                 : f32x4{};
#pragma unroll
    for (int j = 0; j < 8; ++j) v += t[j];
  }
  const int64_t o = (int64_t)m * a.ins + n;
  if (a.ins % 4 == 0 && !a.accumulate) {
    if (a.dw_bf16)
      *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.dw) + o) =
          u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    else
      *reinterpret_cast<f32x4*>(static_cast<float*>(a.dw) + o) = v;
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (n + j < a.ins) put(a, o + j, v[j]);
}

// How a product is laid over the card.
struct Plan {
  bool big;  // 256 x 256 tiles (one workgroup on a CU), else 128 x 128 (two)
  int mt, nt, whole, splits, stages;
  double us;  // estimate
};

// Tiles of one size.  The tiles past the last full set are cut along t into the
// number of parts that takes the least time: a CU takes 0.88 us for a stage of a
// 256-wide tile and 0.28 us for one of a 128-wide (whether it holds one or two of
// them), 3 us to start, the join 3 us and the parts' sums, written and read, 5
// TB/s; a part has 8 stages or more.  (That parts run whole groups of six stages is
// left out.  Counting the CUs' turns alone cut the
// in_proj shape above in 14 where 3 is best: 1.69 ms.)
Plan plan_with(bool big, int64_t tokens, int64_t outs, int64_t ins) {
  Plan p;
  p.big = big;
  const int bt = big ? 256 : 128, slots = big ? 256 : 512;
  const double stage = big ? 0.88 : 0.28, join = (double)(bt * bt) * 8 / 5e6;
  p.mt = (int)((outs + bt - 1) / bt);
  p.nt = (int)((ins + bt - 1) / bt);
  p.stages = (int)((tokens + kDK - 1) / kDK);
  const int tiles = p.mt * p.nt, rest = tiles % slots;
  p.whole = tiles - rest;
  const double before = p.whole / 256 * (p.stages * stage);
  p.us = 1e30;
  for (int s = 1; s <= 128 && (s == 1 || s * 8 <= p.stages); ++s) {
    const int parts = rest * s;
    const double us = before + 3.0 + (double)((parts + 255) / 256) * ((double)p.stages / s * stage) +
                      (s > 1 ? 3.0 + parts * join : 0.0);
    if (us < p.us) p.us = us, p.splits = s;
  }
  if (p.splits == 1) p.whole = tiles;
  return p;
}

// The layout with the smaller estimate: 256-wide tiles where there are enough of
// them or long enough sums (32768 x 2560 x 768: 123 us, 128-wide 158), 128-wide
// ones for little work (4096 x 2048 x 2048: 45 us, 256-wide 54; 8191 x 768 x
// 1536: 35 and 37).
Plan plan_of(int64_t tokens, int64_t outs, int64_t ins) {
  const Plan a = plan_with(true, tokens, outs, ins), b = plan_with(false, tokens, outs, ins);
  return a.us <= b.us ? a : b;
}

// Whether dY's rows can go into LDS as they lie.
bool direct(const void* dy, int64_t dy_stride, int64_t outs) {
  return (reinterpret_cast<uintptr_t>(dy) & 15) == 0 && dy_stride % 8 == 0 && outs % 8 == 0 && dy_stride <= (1 << 23);
}

size_t parts_bytes(const Plan& p) {
  const size_t tile = p.big ? 256 * 256 : 128 * 128;
  return (size_t)(p.mt * p.nt - p.whole) * (size_t)p.splits * tile * sizeof(float);
}

template <int WM, int WN, int TM, int TN>
hipError_t launch_cfg(const Args& a, hipStream_t stream) {
  constexpr int BM = WM * TM * 32, BN = WN * TN * 32;
  const int cut = a.mt * a.nt - a.whole;
  hipLaunchKernelGGL((wgrad8_kernel<WM, WN, TM, TN>), dim3((unsigned)(a.whole + cut * a.splits)), dim3(WM * WN * 64), 0,
                     stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || cut == 0) return e;
  hipLaunchKernelGGL((wgrad8_join_kernel<BM, BN>), dim3(BM * BN / 1024, (unsigned)cut), dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

size_t wgrad8_workspace_bytes(const void* dy, int64_t dy_stride, int64_t tokens, int64_t outs, int64_t ins) {
  const size_t copy = direct(dy, dy_stride, outs) ? 0 : (size_t)tokens * (size_t)((outs + 7) / 8 * 16);
  return 256 + parts_bytes(plan_of(tokens, outs, ins)) + copy;
}

hipError_t launch_wgrad8(const Wgrad8Params& p, hipStream_t stream) {
  const Plan pl = plan_of(p.tokens, p.outs, p.ins);
  char* ws = static_cast<char*>(p.workspace);
  Args a;
  a.dy = static_cast<const uint16_t*>(p.dy);
  a.dy_stride = p.dy_stride;
  if (!direct(p.dy, p.dy_stride, p.outs)) {
    uint16_t* copy = reinterpret_cast<uint16_t*>(ws + 256 + parts_bytes(pl));
    const uint32_t vecs = (uint32_t)((p.outs + 7) / 8);
    hipLaunchKernelGGL(wgrad8_align_kernel, dim3((unsigned)((p.tokens * vecs + 1023) / 1024)), dim3(256), 0, stream, a.dy,
                       p.dy_stride, copy, p.tokens, (int)p.outs, vecs);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    a.dy = copy;
    a.dy_stride = (int64_t)vecs * 8;
  }
  a.q = p.q;
  a.scale = p.scale;
  a.dw = p.dw;
  a.part = reinterpret_cast<float*>(ws + 256);
  a.tokens = p.tokens;
  a.outs = (int)p.outs;
  a.acols = (int)((p.outs + 7) / 8 * 8);
  a.ins = (int)p.ins;
  a.pitch = (int)((p.ins + 31) / 32 * 32);
  a.mt = pl.mt, a.nt = pl.nt, a.whole = pl.whole, a.splits = pl.splits, a.stages = pl.stages;
  a.dw_bf16 = p.dw_bf16;
  a.accumulate = p.accumulate;
  a.status = static_cast<int*>(p.workspace);
  return pl.big ? launch_cfg<2, 4, 4, 2>(a, stream) : launch_cfg<2, 2, 2, 2>(a, stream);
}

}  // namespace mss
