// Weight gradient of a linear layer whose input was kept in 8 bits (gfx950):
//   dW[o, i] = sum_t dY[t, o] X[t, i],  X = q 2^(e - 127)  (rows.hpp)
// on v_mfma_f32_32x32x16_bf16 with fp32 accumulation.  X's values are exact in
// bf16, so nothing is rounded before the products.
//
// Both operands lie with the summed axis t slow, so a tile of 64 steps is
// staged in LDS as it lies in memory (t-major), X widened on the way, and the
// matrix operands (eight steps of one column per lane) come out of LDS by
// transposing reads.  A staged row is cut into chunks of 64 bytes, chunk c of
// row t stored at c ^ (t % 4): the four rows that a transposing read touches
// then lie in different banks.
//
// Output tiles that do not fill the card's last round are cut along t into
// `splits` parts each, whose fp32 sums go to the workspace and are added in
// order by a second kernel: the result does not depend on scheduling.
#include "launch.hpp"
#include "rows.hpp"
#include "ssd_common.hpp"

namespace mss {
namespace {

using ssd::f32x16;
using ssd::mfma;

constexpr int kBK = 64;  // steps of a stage

struct Args {
  const uint16_t* dy;
  const int8_t* q;
  const uint8_t* scale;
  void* dw;
  float* part;  // [cut][splits][BM][BN]
  int64_t dy_stride;
  int64_t tokens;
  int outs, ins, pitch;
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

template <int WM, int WN, int TM, int TN>  // waves, and 32 x 32 tiles of a wave
struct Cfg {
  static constexpr int kThreads = WM * WN * 64, BM = WM * TM * 32, BN = WN * TN * 32;
  static constexpr int kARows = kThreads * 8 / BM;  // rows of dY a pass of 16-byte loads covers
  static constexpr int kBRows = kThreads * 16 / BN; // rows of q
  static constexpr int kAPass = kBK / kARows, kBPass = kBK / kBRows;
};

// Byte offset of 16-byte slot `s` of staged row t of `width` bytes.
__device__ __forceinline__ int stage_slot(int t, int s, int width) {
  return t * width + ((((s >> 2) ^ (t & 3)) << 2 | (s & 3)) << 4);
}

// Eight (q, scale) as bf16: exact, so the high halves of the fp32 products.
__device__ __forceinline__ u32x4 widen_bf16(uint32_t w0, uint32_t w1, uint32_t scale_bits) {
  Raw<kSrcP8> r;
  r.a = u32x2{w0, w1};
  r.scale = scale_bits;
  float v[8];
  widen<kSrcP8>(r, v);
  u32x4 o;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    o[j] = __builtin_amdgcn_perm(__float_as_uint(v[2 * j + 1]), __float_as_uint(v[2 * j]), 0x07060302u);
  return o;
}

template <typename C, int WM, int WN, int TM, int TN>
__global__ void __launch_bounds__(C::kThreads) wgrad8_kernel(Args a) {
  constexpr int BM = C::BM, BN = C::BN, WA = BM * 2, WB = BN * 2;
  constexpr int kStage = kBK * (WA + WB);  // [64][BM] of dY, [64][BN] of X, bf16
  __shared__ __align__(16) unsigned char smem[2 * kStage];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (blockIdx.x == 0 && tid == 0) *a.status = 0;
  // The tile and the stages of this workgroup.
  int tile = blockIdx.x, part = -1, first = 0, last = a.stages;
  if (tile >= a.whole) {
    part = tile - a.whole;
    tile = a.whole + part / a.splits;
    const int s = part % a.splits;
    first = (int)((int64_t)a.stages * s / a.splits);
    last = (int)((int64_t)a.stages * (s + 1) / a.splits);
  }
  const int m0 = tile / a.nt * BM, n0 = tile % a.nt * BN;

  u32x4 ra[C::kAPass];
  struct QRegs {
    u32x4 q;
    uint32_t scale;
  } rb[C::kBPass];
  auto fetch = [&](int st) {
#pragma unroll
    for (int p = 0; p < C::kAPass; ++p) {
      const int64_t t = (int64_t)st * kBK + p * C::kARows + tid / (BM / 8);
      const int c = m0 + tid % (BM / 8) * 8;
      ra[p] = load_raw<kSrcBf16>(a.dy + t * a.dy_stride, nullptr, c, t < a.tokens ? a.outs - c : 0).a;
    }
#pragma unroll
    for (int p = 0; p < C::kBPass; ++p) {
      const int64_t t = (int64_t)st * kBK + p * C::kBRows + tid / (BN / 16);
      const int c = n0 + tid % (BN / 16) * 16;
      rb[p].q = u32x4{};
      rb[p].scale = 0;
      if (t < a.tokens && c < a.pitch) {  // the pitch is whole blocks of 32
        rb[p].q = *reinterpret_cast<const u32x4*>(a.q + t * a.pitch + c);
        rb[p].scale = (uint32_t)a.scale[t * (a.pitch >> 5) + (c >> 5)] << 23;
      }
    }
  };
  auto commit = [&](unsigned char* st) {
#pragma unroll
    for (int p = 0; p < C::kAPass; ++p) {
      const int t = p * C::kARows + tid / (BM / 8);
      *reinterpret_cast<u32x4*>(st + stage_slot(t, tid % (BM / 8), WA)) = ra[p];
    }
    unsigned char* sb = st + kBK * WA;
#pragma unroll
    for (int p = 0; p < C::kBPass; ++p) {
      const int t = p * C::kBRows + tid / (BN / 16), s = tid % (BN / 16) * 2;
      *reinterpret_cast<u32x4*>(sb + stage_slot(t, s, WB)) = widen_bf16(rb[p].q[0], rb[p].q[1], rb[p].scale);
      *reinterpret_cast<u32x4*>(sb + stage_slot(t, s + 1, WB)) = widen_bf16(rb[p].q[2], rb[p].q[3], rb[p].scale);
    }
  };

  f32x16 acc[TM][TN] = {};
  const int wm = wave / WN * (TM * 32), wn = wave % WN * (TN * 32);
  const int i16 = lane & 15, hf = lane >> 5, gc = (lane >> 4) & 1;
  // Steps kk*16 + 8 hf .. + 8 of column base + lane % 32 (base a multiple of
  // 32): two transposing reads of four rows.  Lane i of a 16-lane group
  // addresses row i / 4 of the four, columns 4 (i % 4) .. + 4 of the group's 16.
  typedef short v4s __attribute__((ext_vector_type(4)));
  auto frag = [&](const unsigned char* st, int kk, int base, int width) -> u32x4 {
    const int t = kk * 16 + 8 * hf + (i16 >> 2);
    const unsigned char* p = st + t * width + ((base >> 5) ^ (i16 >> 2)) * 64 + gc * 32 + (i16 & 3) * 8;
    const u32x2 lo = __builtin_bit_cast(
        u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)(p)));
    const u32x2 hi = __builtin_bit_cast(
        u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)(p + 4 * width)));
    return u32x4{lo[0], lo[1], hi[0], hi[1]};
  };

  if (first < last) {
    fetch(first);
    commit(smem);
  }
  for (int st = first; st < last; ++st) {
    unsigned char* cur = smem + ((st - first) & 1) * kStage;
    __syncthreads();  // this stage is written, and the other one read
    if (st + 1 < last) fetch(st + 1);
#pragma unroll
    for (int kk = 0; kk < kBK / 16; ++kk) {
      u32x4 fa[TM], fb[TN];
#pragma unroll
      for (int i = 0; i < TM; ++i) fa[i] = frag(cur, kk, wm + 32 * i, WA);
#pragma unroll
      for (int j = 0; j < TN; ++j) fb[j] = frag(cur + kBK * WA, kk, wn + 32 * j, WB);
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = mfma(fa[i], fb[j], acc[i][j]);
    }
    if (st + 1 < last) commit(smem + ((st + 1 - first) & 1) * kStage);
  }
  // Accumulators: row 8 (r / 4) + 4 hf + r % 4, column lane % 32 of a 32 x 32 tile.
  const int lc = lane & 31;
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int m = wm + 32 * i + 8 * (r >> 2) + 4 * hf + (r & 3), n = wn + 32 * j + lc;
        if (part >= 0) a.part[((int64_t)part * BM + m) * BN + n] = acc[i][j][r];
        else if (m0 + m < a.outs && n0 + n < a.ins) put(a, (int64_t)(m0 + m) * a.ins + n0 + n, acc[i][j][r]);
      }
}

// The cut tiles: their parts added in order.  grid (tile, BM / 4 rows of four), BN threads.
template <int BM, int BN>
__global__ void __launch_bounds__(BN) wgrad8_join_kernel(Args a) {
  const int tile = a.whole + blockIdx.x, m0 = tile / a.nt * BM, n = tile % a.nt * BN + threadIdx.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = blockIdx.y * 4 + i;
    if (m0 + m >= a.outs || n >= a.ins) continue;
    const float* p = a.part + ((int64_t)blockIdx.x * a.splits * BM + m) * BN + threadIdx.x;
    float v = 0.f;
    for (int s = 0; s < a.splits; ++s) v += p[(int64_t)s * BM * BN];
    put(a, (int64_t)(m0 + m) * a.ins + n, v);
  }
}

// How a product is laid over the card.
struct Plan {
  bool big;  // 256 x 256 tiles (one workgroup per CU), else 128 x 128 (two)
  int mt, nt, whole, splits, stages;
};

Plan plan_of(int64_t tokens, int64_t outs, int64_t ins) {
  Plan p;
  const int64_t t256 = ((outs + 255) / 256) * ((ins + 255) / 256);
  p.big = t256 >= 128;
  const int bt = p.big ? 256 : 128, slots = p.big ? 256 : 512;
  p.mt = (int)((outs + bt - 1) / bt);
  p.nt = (int)((ins + bt - 1) / bt);
  p.stages = (int)((tokens + kBK - 1) / kBK);
  const int tiles = p.mt * p.nt, rest = tiles % slots;
  p.whole = tiles - rest;
  // Parts of the tiles past the last full round: the fewest that leave the
  // least time, ceil(rest * s / slots) / s rounds, each part at least 4 stages.
  p.splits = 1;
  double best = 1e30;
  for (int s = 1; s <= 64 && s * 4 <= (p.stages > 4 ? p.stages : 4); ++s) {
    const double rounds = (double)((rest * s + slots - 1) / slots) / s;
    if (rounds < best * 0.97) best = rounds, p.splits = s;
  }
  if (p.splits == 1) p.whole = tiles;
  return p;
}

template <int WM, int WN, int TM, int TN>
hipError_t launch_cfg(const Args& a, hipStream_t stream) {
  typedef Cfg<WM, WN, TM, TN> C;
  const int cut = a.mt * a.nt - a.whole;
  hipLaunchKernelGGL((wgrad8_kernel<C, WM, WN, TM, TN>), dim3((unsigned)(a.whole + cut * a.splits)), dim3(C::kThreads), 0,
                     stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || cut == 0) return e;
  hipLaunchKernelGGL((wgrad8_join_kernel<C::BM, C::BN>), dim3((unsigned)cut, C::BM / 4), dim3(C::BN), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

size_t wgrad8_workspace_bytes(int64_t tokens, int64_t outs, int64_t ins) {
  const Plan p = plan_of(tokens, outs, ins);
  const size_t tile = p.big ? 256 * 256 : 128 * 128;
  return 256 + (size_t)(p.mt * p.nt - p.whole) * (size_t)p.splits * tile * sizeof(float);
}

hipError_t launch_wgrad8(const Wgrad8Params& p, hipStream_t stream) {
  const Plan pl = plan_of(p.tokens, p.outs, p.ins);
  Args a;
  a.dy = static_cast<const uint16_t*>(p.dy);
  a.q = p.q;
  a.scale = p.scale;
  a.dw = p.dw;
  a.part = reinterpret_cast<float*>(static_cast<char*>(p.workspace) + 256);
  a.dy_stride = p.dy_stride;
  a.tokens = p.tokens;
  a.outs = (int)p.outs;
  a.ins = (int)p.ins;
  a.pitch = (int)((p.ins + 31) / 32 * 32);
  a.mt = pl.mt, a.nt = pl.nt, a.whole = pl.whole, a.splits = pl.splits, a.stages = pl.stages;
  a.dw_bf16 = p.dw_bf16;
  a.accumulate = p.accumulate;
  a.status = static_cast<int*>(p.workspace);
  return pl.big ? launch_cfg<2, 4, 4, 2>(a, stream) : launch_cfg<2, 2, 2, 2>(a, stream);
}

}  // namespace mss
