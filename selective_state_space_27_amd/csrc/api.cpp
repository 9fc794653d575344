// C-ABI entry points of libmambascan: host-side validation, then launch.
// Everything here runs on the host before any HIP call; on any error nothing
// is enqueued and no output is touched.
#include <hip/hip_runtime.h>

#include <stdint.h>
#include <string.h>

#include <mutex>

#include "../../include/mambascan.h"
#include "launch.hpp"

namespace {

thread_local int g_last_hip_error = 0;

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
};

Range range_of(const void* p, size_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Range{a, a + bytes};
}

bool overlaps(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

size_t elem_size(mss_dtype t) { return t == MSS_BF16 ? 2 : 4; }

bool dtype_ok(mss_dtype t) { return t == MSS_FP32 || t == MSS_BF16; }

// An output range must not overlap any of the listed (non-null) input ranges.
bool output_clear(const void* out, size_t out_bytes, const void* const* ins, const size_t* in_bytes, int n) {
  if (out == nullptr) return true;
  const Range o = range_of(out, out_bytes);
  for (int i = 0; i < n; ++i)
    if (ins[i] != nullptr && overlaps(o, range_of(ins[i], in_bytes[i]))) return false;
  return true;
}

mss_status hip_status(hipError_t e) {
  if (e == hipSuccess) return MSS_OK;
  g_last_hip_error = static_cast<int>(e);
  return MSS_ERR_HIP;
}

constexpr int64_t kMaxIndex = INT32_MAX;

// Scratch of mss_selective_scan_fwd_noalloc, for callers that cannot allocate:
// one copy per GPU, held until the process ends.  In host code `scratch`
// names a host-side stand-in; its device address, different on each GPU,
// comes from hipGetSymbolAddress with that GPU current and is kept per device.
constexpr size_t kNoAllocScratchBytes = size_t{64} << 20;
static __device__ __align__(256) unsigned char scratch[kNoAllocScratchBytes];

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices] = {};

// The current device's scratch address, looked up on its first use there.
hipError_t scratch_of_current_device(void** out) {
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return hipErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (g_scratch_ptr[dev] == nullptr) {
    void* p = nullptr;
    e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    if (e != hipSuccess) return e;
    if (p == nullptr) return hipErrorInvalidSymbol;
    g_scratch_ptr[dev] = p;
  }
  *out = g_scratch_ptr[dev];
  return hipSuccess;
}

}  // namespace

extern "C" {

const char* mss_status_string(mss_status s) {
  switch (s) {
    case MSS_OK: return "MSS_OK";
    case MSS_ERR_NULL: return "MSS_ERR_NULL: a required pointer is NULL";
    case MSS_ERR_SHAPE: return "MSS_ERR_SHAPE: a size is not positive or is too large";
    case MSS_ERR_DTYPE: return "MSS_ERR_DTYPE: unknown dtype";
    case MSS_ERR_ALIGN: return "MSS_ERR_ALIGN: a pointer is not 16-byte aligned";
    case MSS_ERR_UNSUPPORTED: return "MSS_ERR_UNSUPPORTED: shape or option not implemented";
    case MSS_ERR_WORKSPACE: return "MSS_ERR_WORKSPACE: workspace missing or too small";
    case MSS_ERR_ALIAS: return "MSS_ERR_ALIAS: an output overlaps an input";
    case MSS_ERR_HIP: return "MSS_ERR_HIP: a HIP call failed";
    case MSS_ERR_WAIT: return "MSS_ERR_WAIT: a bounded wait between workgroups gave up; the outputs are not valid";
  }
  return "unknown mss_status";
}

int mss_last_hip_error(void) { return g_last_hip_error; }

int mss_abi_version(void) { return MSS_ABI_VERSION; }

mss_status mss_workspace_status(const void* workspace, void* hip_stream) {
  if (workspace == nullptr) return MSS_ERR_NULL;
  hipError_t e = hipStreamSynchronize(static_cast<hipStream_t>(hip_stream));
  int word = 0;
  if (e == hipSuccess) e = hipMemcpy(&word, workspace, sizeof(word), hipMemcpyDeviceToHost);
  if (e != hipSuccess) return hip_status(e);
  return word == 0 ? MSS_OK : MSS_ERR_WAIT;
}

// ------------------------------------------------------------ selective scan
static mss_status scan_check_shape(int64_t batch, int64_t dim, int64_t dstate, int64_t seqlen, mss_dtype t) {
  if (!dtype_ok(t)) return MSS_ERR_DTYPE;
  if (batch <= 0 || dim <= 0 || dstate <= 0 || seqlen <= 0) return MSS_ERR_SHAPE;
  if (batch > 65535 || seqlen >= (1LL << 24) || dim * seqlen > kMaxIndex || dim * dstate > kMaxIndex ||
      batch * dim > kMaxIndex)
    return MSS_ERR_SHAPE;
  if (dstate > 128) return MSS_ERR_UNSUPPORTED;
  return MSS_OK;
}

size_t mss_selective_scan_workspace_size(int64_t batch, int64_t dim, int64_t dstate, int64_t seqlen,
                                         mss_dtype io_dtype, uint32_t flags) {
  (void)flags;
  if (scan_check_shape(batch, dim, dstate, seqlen, io_dtype) != MSS_OK) return 0;
  return mss::scan_workspace_bytes(batch, dim, dstate, seqlen);
}

// The selective scan forward's checks before the workspace's: pointers,
// shape, flags, alignment (`extra`, a 4-byte output, only needs 4 bytes).
static mss_status scan_fwd_check_args(const void* u, const void* delta, const float* A, const void* B, const void* C,
                                      const float* D, const void* z, const float* h0, const void* y,
                                      const float* h_last, int64_t batch, int64_t dim, int64_t dstate, int64_t seqlen,
                                      mss_dtype io_dtype, uint32_t flags, const void* workspace, const void* extra) {
  if (!u || !delta || !A || !B || !C || !y) return MSS_ERR_NULL;
  mss_status st = scan_check_shape(batch, dim, dstate, seqlen, io_dtype);
  if (st != MSS_OK) return st;
  if (flags & ~MSS_FLAG_DECAY_GENERAL) return MSS_ERR_UNSUPPORTED;
  const void* all[] = {u, delta, A, B, C, D, z, h0, y, h_last, workspace};
  for (const void* p : all)
    if (p && !aligned16(p)) return MSS_ERR_ALIGN;
  if (extra && (reinterpret_cast<uintptr_t>(extra) & 3u)) return MSS_ERR_ALIGN;
  return MSS_OK;
}

// ... and after it: no output overlaps an input (the workspace, `need` bytes,
// counts as one) or another output (`extra`, 4 bytes, nullable).
static mss_status scan_fwd_check_alias(const void* u, const void* delta, const float* A, const void* B,
                                       const void* C, const float* D, const void* z, const float* h0, const void* y,
                                       const float* h_last, int64_t batch, int64_t dim, int64_t dstate,
                                       int64_t seqlen, mss_dtype io_dtype, const void* workspace, size_t need,
                                       const void* extra) {
  const size_t es = elem_size(io_dtype);
  const size_t nbdl = (size_t)batch * dim * seqlen;
  const size_t nbnl = (size_t)batch * dstate * seqlen;
  const size_t nstate = (size_t)batch * dim * dstate * sizeof(float);
  const void* ins[] = {u, delta, A, B, C, D, z, h0, workspace};
  const size_t in_bytes[] = {nbdl * es, nbdl * es, (size_t)dim * dstate * 4, nbnl * es, nbnl * es,
                             (size_t)dim * 4, nbdl * es, nstate, need};
  if (!output_clear(y, nbdl * es, ins, in_bytes, 9)) return MSS_ERR_ALIAS;
  if (!output_clear(h_last, nstate, ins, in_bytes, 9)) return MSS_ERR_ALIAS;
  if (h_last && overlaps(range_of(y, nbdl * es), range_of(h_last, nstate))) return MSS_ERR_ALIAS;
  if (extra) {
    const Range e = range_of(extra, sizeof(int));
    if (!output_clear(extra, sizeof(int), ins, in_bytes, 9)) return MSS_ERR_ALIAS;
    if (overlaps(e, range_of(y, nbdl * es))) return MSS_ERR_ALIAS;
    if (h_last && overlaps(e, range_of(h_last, nstate))) return MSS_ERR_ALIAS;
  }
  return MSS_OK;
}

static mss::ScanParams scan_params(const void* u, const void* delta, const float* A, const void* B, const void* C,
                                   const float* D, const void* z, const float* h0, void* y, float* h_last,
                                   int64_t batch, int64_t dim, int64_t dstate, int64_t seqlen, mss_dtype io_dtype,
                                   uint32_t flags, void* workspace) {
  mss::ScanParams p;
  p.u = u;
  p.delta = delta;
  p.A = A;
  p.B = B;
  p.C = C;
  p.D = D;
  p.z = z;
  p.h0 = h0;
  p.y = y;
  p.h_last = h_last;
  p.batch = batch;
  p.dim = dim;
  p.dstate = dstate;
  p.seqlen = seqlen;
  p.bf16 = io_dtype == MSS_BF16;
  p.force_general = (flags & MSS_FLAG_DECAY_GENERAL) != 0;
  p.workspace = workspace;
  return p;
}

mss_status mss_selective_scan_fwd(const void* u, const void* delta, const float* A, const void* B, const void* C,
                                  const float* D, const void* z, const float* h0, void* y, float* h_last,
                                  int64_t batch, int64_t dim, int64_t dstate, int64_t seqlen, mss_dtype io_dtype,
                                  uint32_t flags, void* workspace, size_t workspace_bytes, void* hip_stream) {
  mss_status st = scan_fwd_check_args(u, delta, A, B, C, D, z, h0, y, h_last, batch, dim, dstate, seqlen, io_dtype,
                                      flags, workspace, nullptr);
  if (st != MSS_OK) return st;
  const size_t need = mss::scan_workspace_bytes(batch, dim, dstate, seqlen);
  if (!workspace || workspace_bytes < need) return MSS_ERR_WORKSPACE;
  st = scan_fwd_check_alias(u, delta, A, B, C, D, z, h0, y, h_last, batch, dim, dstate, seqlen, io_dtype, workspace,
                            need, nullptr);
  if (st != MSS_OK) return st;
  const mss::ScanParams p = scan_params(u, delta, A, B, C, D, z, h0, y, h_last, batch, dim, dstate, seqlen, io_dtype,
                                        flags, workspace);
  return hip_status(mss::launch_scan(p, static_cast<hipStream_t>(hip_stream)));
}

mss_status mss_selective_scan_fwd_noalloc(const void* u, const void* delta, const float* A, const void* B,
                                          const void* C, const float* D, const void* z, const float* h0, void* y,
                                          float* h_last, int64_t batch, int64_t dim, int64_t dstate, int64_t seqlen,
                                          mss_dtype io_dtype, uint32_t flags, int* wait_status, void* hip_stream) {
  mss_status st = scan_fwd_check_args(u, delta, A, B, C, D, z, h0, y, h_last, batch, dim, dstate, seqlen, io_dtype,
                                      flags, nullptr, wait_status);
  if (st != MSS_OK) return st;
  st = scan_fwd_check_alias(u, delta, A, B, C, D, z, h0, y, h_last, batch, dim, dstate, seqlen, io_dtype, nullptr, 0,
                            wait_status);
  if (st != MSS_OK) return st;
  if (mss::scan_workspace_bytes(batch, dim, dstate, seqlen) > kNoAllocScratchBytes) return MSS_ERR_WORKSPACE;
  void* ws = nullptr;
  const hipError_t e = scratch_of_current_device(&ws);
  if (e != hipSuccess) return hip_status(e);
  mss::ScanParams p = scan_params(u, delta, A, B, C, D, z, h0, y, h_last, batch, dim, dstate, seqlen, io_dtype, flags,
                                  ws);
  p.status = wait_status;
  return hip_status(mss::launch_scan(p, static_cast<hipStream_t>(hip_stream)));
}

mss_status mss_selective_scan_fwd_fused(const void* x, const float* conv_w, const float* conv_b,
                                        const void* delta_raw, const float* delta_bias, const float* A,
                                        const void* B, const void* C, const float* D, const void* z,
                                        const float* h0, void* y, float* h_last, int64_t batch, int64_t dim,
                                        int64_t dstate, int64_t seqlen, mss_dtype io_dtype, uint32_t flags,
                                        void* workspace, size_t workspace_bytes, void* hip_stream) {
  if (!x || !conv_w || !delta_raw || !A || !B || !C || !y) return MSS_ERR_NULL;
  mss_status st = scan_check_shape(batch, dim, dstate, seqlen, io_dtype);
  if (st != MSS_OK) return st;
  if (flags & ~(MSS_FLAG_DECAY_GENERAL | MSS_FLAG_CONV_SILU | MSS_FLAG_DELTA_SOFTPLUS)) return MSS_ERR_UNSUPPORTED;
  const void* all[] = {x, conv_w, conv_b, delta_raw, delta_bias, A, B, C, D, z, h0, y, h_last, workspace};
  for (const void* p : all)
    if (p && !aligned16(p)) return MSS_ERR_ALIGN;
  const size_t need = mss::scan_workspace_bytes(batch, dim, dstate, seqlen);
  if (!workspace || workspace_bytes < need) return MSS_ERR_WORKSPACE;

  const size_t es = elem_size(io_dtype);
  const size_t nbdl = (size_t)batch * dim * seqlen;
  const size_t nbnl = (size_t)batch * dstate * seqlen;
  const size_t nstate = (size_t)batch * dim * dstate * sizeof(float);
  const void* ins[] = {x, conv_w, conv_b, delta_raw, delta_bias, A, B, C, D, z, h0, workspace};
  const size_t in_bytes[] = {nbdl * es, (size_t)dim * 16, (size_t)dim * 4, nbdl * es, (size_t)dim * 4,
                             (size_t)dim * dstate * 4, nbnl * es, nbnl * es, (size_t)dim * 4, nbdl * es, nstate,
                             need};
  if (!output_clear(y, nbdl * es, ins, in_bytes, 12)) return MSS_ERR_ALIAS;
  if (!output_clear(h_last, nstate, ins, in_bytes, 12)) return MSS_ERR_ALIAS;
  if (h_last && overlaps(range_of(y, nbdl * es), range_of(h_last, nstate))) return MSS_ERR_ALIAS;

  mss::ScanParams p;
  p.u = x;
  p.delta = delta_raw;
  p.A = A;
  p.B = B;
  p.C = C;
  p.D = D;
  p.z = z;
  p.h0 = h0;
  p.y = y;
  p.h_last = h_last;
  p.batch = batch;
  p.dim = dim;
  p.dstate = dstate;
  p.seqlen = seqlen;
  p.bf16 = io_dtype == MSS_BF16;
  p.force_general = (flags & MSS_FLAG_DECAY_GENERAL) != 0;
  p.workspace = workspace;
  p.fused = true;
  p.conv_w = conv_w;
  p.conv_b = conv_b;
  p.delta_bias = delta_bias;
  p.conv_silu = (flags & MSS_FLAG_CONV_SILU) != 0;
  p.delta_softplus = (flags & MSS_FLAG_DELTA_SOFTPLUS) != 0;
  return hip_status(mss::launch_scan(p, static_cast<hipStream_t>(hip_stream)));
}

// --------------------------------------------------- selective scan backward
// The forward's limits (d_state <= 128).  Up to 32 states the gradient
// kernels take them all (up to 4 states per wave); above, slices of 32 run
// one after the other.
static mss_status scan_bwd_check_shape(int64_t batch, int64_t dim, int64_t dstate, int64_t seqlen, mss_dtype t) {
  return scan_check_shape(batch, dim, dstate, seqlen, t);
}

static size_t scan_bwd_need(int64_t batch, int64_t dim, int64_t dstate, int64_t seqlen) {
  return dstate > 32 ? mss::scan_bwd_wide_workspace_bytes(batch, dim, seqlen)
                     : mss::scan_bwd_workspace_bytes(batch, dim, dstate, seqlen);
}

size_t mss_selective_scan_bwd_workspace_size(int64_t batch, int64_t dim, int64_t dstate, int64_t seqlen,
                                             mss_dtype io_dtype, uint32_t flags) {
  (void)flags;
  if (scan_bwd_check_shape(batch, dim, dstate, seqlen, io_dtype) != MSS_OK) return 0;
  return scan_bwd_need(batch, dim, dstate, seqlen);
}

mss_status mss_selective_scan_bwd(const void* u, const void* delta, const float* A, const void* B, const void* C,
                                  const float* D, const void* z, const float* h0, const void* dy,
                                  const float* dh_last, void* du, void* ddelta, float* dA, void* dB, void* dC,
                                  float* dD, void* dz, float* dh0, int64_t batch, int64_t dim, int64_t dstate,
                                  int64_t seqlen, mss_dtype io_dtype, uint32_t flags, void* workspace,
                                  size_t workspace_bytes, void* hip_stream) {
  if (!u || !delta || !A || !B || !C || !dy || !du || !ddelta || !dA || !dB || !dC) return MSS_ERR_NULL;
  if ((z == nullptr) != (dz == nullptr)) return MSS_ERR_NULL;
  mss_status st = scan_bwd_check_shape(batch, dim, dstate, seqlen, io_dtype);
  if (st != MSS_OK) return st;
  if (flags & ~MSS_FLAG_DECAY_GENERAL) return MSS_ERR_UNSUPPORTED;
  const void* all[] = {u, delta, A, B, C, D, z, h0, dy, dh_last, du, ddelta, dA, dB, dC, dD, dz, dh0, workspace};
  for (const void* p : all)
    if (p && !aligned16(p)) return MSS_ERR_ALIGN;
  const size_t need = scan_bwd_need(batch, dim, dstate, seqlen);
  if (!workspace || workspace_bytes < need) return MSS_ERR_WORKSPACE;

  const size_t es = elem_size(io_dtype);
  const size_t nbdl = (size_t)batch * dim * seqlen * es;
  const size_t nbnl = (size_t)batch * dstate * seqlen * es;
  const size_t nA = (size_t)dim * dstate * 4, nD = (size_t)dim * 4;
  const size_t nstate = (size_t)batch * dim * dstate * sizeof(float);
  const void* ins[] = {u, delta, A, B, C, D, z, h0, dy, dh_last, workspace};
  const size_t in_bytes[] = {nbdl, nbdl, nA, nbnl, nbnl, nD, nbdl, nstate, nbdl, nstate, need};
  void* outs[] = {du, ddelta, dA, dB, dC, dD, dz, dh0};
  const size_t out_bytes[] = {nbdl, nbdl, nA, nbnl, nbnl, nD, nbdl, nstate};
  for (int i = 0; i < 8; ++i) {
    if (!output_clear(outs[i], out_bytes[i], ins, in_bytes, 11)) return MSS_ERR_ALIAS;
    for (int j = i + 1; j < 8; ++j)
      if (outs[i] && outs[j] && overlaps(range_of(outs[i], out_bytes[i]), range_of(outs[j], out_bytes[j])))
        return MSS_ERR_ALIAS;
  }

  mss::ScanBwdParams p;
  p.fwd.u = u;
  p.fwd.delta = delta;
  p.fwd.A = A;
  p.fwd.B = B;
  p.fwd.C = C;
  p.fwd.D = D;
  p.fwd.z = z;
  p.fwd.h0 = h0;
  p.fwd.y = nullptr;
  p.fwd.h_last = nullptr;
  p.fwd.batch = batch;
  p.fwd.dim = dim;
  p.fwd.dstate = dstate;
  p.fwd.seqlen = seqlen;
  p.fwd.bf16 = io_dtype == MSS_BF16;
  p.fwd.force_general = (flags & MSS_FLAG_DECAY_GENERAL) != 0;
  p.fwd.workspace = workspace;
  p.dy = dy;
  p.dh_last = dh_last;
  p.du = du;
  p.ddelta = ddelta;
  p.dA = dA;
  p.dB = dB;
  p.dC = dC;
  p.dD = dD;
  p.dz = dz;
  p.dh0 = dh0;
  if (dstate > 32) return hip_status(mss::launch_scan_bwd_wide(p, static_cast<hipStream_t>(hip_stream)));
  return hip_status(mss::launch_scan_bwd(p, static_cast<hipStream_t>(hip_stream)));
}

// ------------------------------------------ fused scan (prologue) backward
size_t mss_selective_scan_fused_bwd_workspace_size(int64_t batch, int64_t dim, int64_t dstate, int64_t seqlen,
                                                   mss_dtype io_dtype, uint32_t flags) {
  (void)flags;
  if (scan_bwd_check_shape(batch, dim, dstate, seqlen, io_dtype) != MSS_OK) return 0;
  return mss::scan_fused_bwd_workspace_bytes(batch, dim, dstate, seqlen);
}

mss_status mss_selective_scan_fused_bwd(const void* x, const float* conv_w, const float* conv_b,
                                        const void* delta_raw, const float* delta_bias, const float* A,
                                        const void* B, const void* C, const float* D, const void* z,
                                        const float* h0, const void* dy, const float* dh_last, void* dx,
                                        void* ddelta_raw, float* dconv_w, float* dconv_b, float* ddelta_bias,
                                        float* dA, void* dB, void* dC, float* dD, void* dz, float* dh0,
                                        int64_t batch, int64_t dim, int64_t dstate, int64_t seqlen,
                                        mss_dtype io_dtype, uint32_t flags, void* workspace, size_t workspace_bytes,
                                        void* hip_stream) {
  if (!x || !conv_w || !delta_raw || !A || !B || !C || !dy || !dx || !ddelta_raw || !dconv_w || !dA || !dB || !dC)
    return MSS_ERR_NULL;
  if ((z == nullptr) != (dz == nullptr)) return MSS_ERR_NULL;
  mss_status st = scan_bwd_check_shape(batch, dim, dstate, seqlen, io_dtype);
  if (st != MSS_OK) return st;
  if (flags & ~(MSS_FLAG_DECAY_GENERAL | MSS_FLAG_CONV_SILU | MSS_FLAG_DELTA_SOFTPLUS)) return MSS_ERR_UNSUPPORTED;
  const void* all[] = {x, conv_w, conv_b, delta_raw, delta_bias, A, B, C, D, z, h0, dy, dh_last, dx, ddelta_raw,
                       dconv_w, dconv_b, ddelta_bias, dA, dB, dC, dD, dz, dh0, workspace};
  for (const void* p : all)
    if (p && !aligned16(p)) return MSS_ERR_ALIGN;
  const size_t need = mss::scan_fused_bwd_workspace_bytes(batch, dim, dstate, seqlen);
  if (!workspace || workspace_bytes < need) return MSS_ERR_WORKSPACE;

  const size_t es = elem_size(io_dtype);
  const size_t nbdl = (size_t)batch * dim * seqlen * es;
  const size_t nbnl = (size_t)batch * dstate * seqlen * es;
  const size_t nA = (size_t)dim * dstate * 4, nD = (size_t)dim * 4;
  const size_t nstate = (size_t)batch * dim * dstate * sizeof(float);
  const void* ins[] = {x, conv_w, conv_b, delta_raw, delta_bias, A, B, C, D, z, h0, dy, dh_last, workspace};
  const size_t in_bytes[] = {nbdl, nD * 4, nD, nbdl, nD, nA, nbnl, nbnl, nD, nbdl, nstate, nbdl, nstate, need};
  void* outs[] = {dx, ddelta_raw, dconv_w, dconv_b, ddelta_bias, dA, dB, dC, dD, dz, dh0};
  const size_t out_bytes[] = {nbdl, nbdl, nD * 4, nD, nD, nA, nbnl, nbnl, nD, nbdl, nstate};
  for (int i = 0; i < 11; ++i) {
    if (!output_clear(outs[i], out_bytes[i], ins, in_bytes, 14)) return MSS_ERR_ALIAS;
    for (int j = i + 1; j < 11; ++j)
      if (outs[i] && outs[j] && overlaps(range_of(outs[i], out_bytes[i]), range_of(outs[j], out_bytes[j])))
        return MSS_ERR_ALIAS;
  }

  mss::ScanFusedBwdParams p;
  p.x = x;
  p.delta_raw = delta_raw;
  p.conv_w = conv_w;
  p.conv_b = conv_b;
  p.delta_bias = delta_bias;
  p.conv_silu = (flags & MSS_FLAG_CONV_SILU) != 0;
  p.softplus = (flags & MSS_FLAG_DELTA_SOFTPLUS) != 0;
  p.A = A;
  p.B = B;
  p.C = C;
  p.D = D;
  p.z = z;
  p.h0 = h0;
  p.dy = dy;
  p.dh_last = dh_last;
  p.dx = dx;
  p.ddelta_raw = ddelta_raw;
  p.dconv_w = dconv_w;
  p.dconv_b = dconv_b;
  p.ddelta_bias = ddelta_bias;
  p.dA = dA;
  p.dB = dB;
  p.dC = dC;
  p.dD = dD;
  p.dz = dz;
  p.dh0 = dh0;
  p.batch = batch;
  p.dim = dim;
  p.dstate = dstate;
  p.seqlen = seqlen;
  p.bf16 = io_dtype == MSS_BF16;
  p.force_general = (flags & MSS_FLAG_DECAY_GENERAL) != 0;
  p.workspace = workspace;
  return hip_status(mss::launch_scan_fused_bwd(p, static_cast<hipStream_t>(hip_stream)));
}

// -------------------------------------------------------------- state update
mss_status mss_state_update(float* h, const void* u, const void* delta, const float* A, const void* B,
                            const void* C, const float* D, const void* z, void* y, int64_t batch, int64_t dim,
                            int64_t dstate, mss_dtype io_dtype, uint32_t flags, void* hip_stream) {
  if (!h || !u || !delta || !A || !B || !C || !y) return MSS_ERR_NULL;
  if (!dtype_ok(io_dtype)) return MSS_ERR_DTYPE;
  if (batch <= 0 || dim <= 0 || dstate <= 0) return MSS_ERR_SHAPE;
  // At most 2^28 rows: 8 threads per row above 64 states keeps the grid below
  // 2^31 work-items, and every state offset below 2^35 elements.
  if (batch > (int64_t{1} << 28) || dim > (int64_t{1} << 28) || batch * dim > (int64_t{1} << 28))
    return MSS_ERR_SHAPE;
  if (dstate > 128) return MSS_ERR_UNSUPPORTED;
  if (flags != 0) return MSS_ERR_UNSUPPORTED;
  const void* all[] = {h, u, delta, A, B, C, D, z, y};
  for (const void* p : all)
    if (p && !aligned16(p)) return MSS_ERR_ALIGN;
  const size_t es = elem_size(io_dtype);
  const size_t nbd = (size_t)batch * dim;
  const size_t nstate = nbd * dstate * sizeof(float);
  const void* ins[] = {u, delta, A, B, C, D, z};
  const size_t in_bytes[] = {nbd * es, nbd * es, (size_t)dim * dstate * 4, (size_t)batch * dstate * es,
                             (size_t)batch * dstate * es, (size_t)dim * 4, nbd * es};
  if (!output_clear(h, nstate, ins, in_bytes, 7)) return MSS_ERR_ALIAS;
  if (!output_clear(y, nbd * es, ins, in_bytes, 7)) return MSS_ERR_ALIAS;
  if (overlaps(range_of(y, nbd * es), range_of(h, nstate))) return MSS_ERR_ALIAS;

  mss::UpdateParams p;
  p.h = h;
  p.u = u;
  p.delta = delta;
  p.A = A;
  p.B = B;
  p.C = C;
  p.D = D;
  p.z = z;
  p.y = y;
  p.batch = batch;
  p.dim = dim;
  p.dstate = dstate;
  p.bf16 = io_dtype == MSS_BF16;
  return hip_status(mss::launch_state_update(p, static_cast<hipStream_t>(hip_stream)));
}

// ---------------------------------------------------------- Mamba-3 update
mss_status mss_mamba3_state_update(float* h, const void* x, const void* x_prev, const float* delta, const float* A,
                                   const float* theta, const void* B, const void* B_prev, const void* C,
                                   const float* D, const void* z, void* y, int64_t batch, int64_t nheads,
                                   int64_t headdim, int64_t ngroups, int64_t dstate, int64_t rank,
                                   mss_dtype io_dtype, uint32_t flags, void* hip_stream) {
  if (!h || !x || !delta || !A || !B || !C || !y) return MSS_ERR_NULL;
  if ((x_prev == nullptr) != (B_prev == nullptr)) return MSS_ERR_NULL;
  const bool cplx = (flags & MSS_FLAG_COMPLEX_STATE) != 0;
  if (cplx && !theta) return MSS_ERR_NULL;
  if (!dtype_ok(io_dtype)) return MSS_ERR_DTYPE;
  if (batch <= 0 || nheads <= 0 || headdim <= 0 || ngroups <= 0 || dstate <= 0 || rank <= 0) return MSS_ERR_SHAPE;
  // Grid (headdim/16, nheads, batch); state offsets within 2^40 floats.
  if (batch > 65535 || nheads > 65535 || batch * nheads * headdim > (int64_t{1} << 28)) return MSS_ERR_SHAPE;
  if (flags & ~MSS_FLAG_COMPLEX_STATE) return MSS_ERR_UNSUPPORTED;
  if (headdim % 16 != 0 || headdim > 4096 || !(dstate == 64 || dstate == 128 || dstate == 256) || rank > 8 ||
      nheads % ngroups != 0)
    return MSS_ERR_UNSUPPORTED;
  const void* all[] = {h, delta, A, theta, D};
  for (const void* p : all)
    if (p && !aligned16(p)) return MSS_ERR_ALIGN;
  const size_t es = elem_size(io_dtype);
  const size_t nx = (size_t)batch * nheads * rank * headdim * es;
  const size_t nbc = (size_t)batch * ngroups * rank * dstate * es;
  const size_t nstate = (size_t)batch * nheads * headdim * dstate * sizeof(float) * (cplx ? 2 : 1);
  const void* ins[] = {x, x_prev, delta, A, theta, B, B_prev, C, D, z};
  const size_t in_bytes[] = {nx, nx, (size_t)batch * nheads * 4, (size_t)nheads * 4,
                             (size_t)nheads * dstate * 4, nbc, nbc, nbc, (size_t)nheads * 4, nx};
  if (!output_clear(h, nstate, ins, in_bytes, 10)) return MSS_ERR_ALIAS;
  if (!output_clear(y, nx, ins, in_bytes, 10)) return MSS_ERR_ALIAS;
  if (overlaps(range_of(y, nx), range_of(h, nstate))) return MSS_ERR_ALIAS;

  mss::Mamba3Params p;
  p.h = h;
  p.x = x;
  p.x_prev = x_prev;
  p.delta = delta;
  p.A = A;
  p.theta = cplx ? theta : nullptr;
  p.B = B;
  p.B_prev = B_prev;
  p.C = C;
  p.D = D;
  p.z = z;
  p.y = y;
  p.batch = batch;
  p.nheads = nheads;
  p.headdim = headdim;
  p.ngroups = ngroups;
  p.dstate = dstate;
  p.rank = rank;
  p.bf16 = io_dtype == MSS_BF16;
  return hip_status(mss::launch_mamba3_step(p, static_cast<hipStream_t>(hip_stream)));
}

// ----------------------------------------------------------------------- SSD
static mss_status ssd_check_shape(int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim,
                                  int64_t ngroups, int64_t dstate, int64_t chunk, mss_dtype t) {
  if (!dtype_ok(t)) return MSS_ERR_DTYPE;
  if (batch <= 0 || seqlen <= 0 || nheads <= 0 || headdim <= 0 || ngroups <= 0 || dstate <= 0 || chunk <= 0)
    return MSS_ERR_SHAPE;
  // Byte offsets inside one batch entry of y (fp32) and of B, C must fit 32
  // bits, with every descriptor at most 2^32 - 256 bytes (the kernels' "no
  // element" offset lies past it).
  if (seqlen * nheads * headdim > (int64_t{1} << 30) - 64 || seqlen * ngroups * dstate >= (int64_t{1} << 30) ||
      batch > 65535 || nheads > 65535)
    return MSS_ERR_SHAPE;
  if (t != MSS_BF16) return MSS_ERR_UNSUPPORTED;
  if (!(headdim == 64 || headdim == 128) || dstate % 16 != 0 || dstate > 256 ||
      !(chunk == 64 || chunk == 128 || chunk == 256))
    return MSS_ERR_UNSUPPORTED;
  // Grids: at most 2 * (chunks x 64-row head slices x batch) workgroups of
  // 512 threads, below 2^32 work-items.
  if (((seqlen + chunk - 1) / chunk) * nheads * (headdim / 64) * batch >= (int64_t{1} << 22)) return MSS_ERR_SHAPE;
  if (nheads % ngroups != 0) return MSS_ERR_UNSUPPORTED;
  return MSS_OK;
}

size_t mss_ssd_workspace_size(int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim, int64_t ngroups,
                              int64_t dstate, int64_t chunk, mss_dtype in_dtype) {
  if (ssd_check_shape(batch, seqlen, nheads, headdim, ngroups, dstate, chunk, in_dtype) != MSS_OK) return 0;
  return mss::ssd_workspace_bytes(batch, seqlen, nheads, headdim, ngroups, dstate, chunk);
}

mss_status mss_ssd_chunk_fwd(const void* x, const float* delta, const float* A, const void* B, const void* C,
                             const float* D, const void* z, const float* h0, float* y, float* chunk_states,
                             float* h_last, int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim,
                             int64_t ngroups, int64_t dstate, int64_t chunk, mss_dtype in_dtype, uint32_t flags,
                             void* workspace, size_t workspace_bytes, void* hip_stream) {
  if (!x || !delta || !A || !B || !C || !y) return MSS_ERR_NULL;
  mss_status st = ssd_check_shape(batch, seqlen, nheads, headdim, ngroups, dstate, chunk, in_dtype);
  if (st != MSS_OK) return st;
  if (flags != 0) return MSS_ERR_UNSUPPORTED;
  const void* all[] = {x, delta, A, B, C, D, z, h0, y, chunk_states, h_last, workspace};
  for (const void* p : all)
    if (p && !aligned16(p)) return MSS_ERR_ALIGN;
  const size_t need = mss::ssd_workspace_bytes(batch, seqlen, nheads, headdim, ngroups, dstate, chunk);
  if (!workspace || workspace_bytes < need) return MSS_ERR_WORKSPACE;

  const size_t es = elem_size(in_dtype);
  const size_t nx = (size_t)batch * seqlen * nheads * headdim;
  const size_t nbc = (size_t)batch * seqlen * ngroups * dstate;
  const size_t nstate = (size_t)batch * nheads * headdim * dstate * sizeof(float);
  const size_t nchunks = (size_t)((seqlen + chunk - 1) / chunk);
  const void* ins[] = {x, delta, A, B, C, D, z, h0, workspace};
  const size_t in_bytes[] = {nx * es, (size_t)batch * seqlen * nheads * 4, (size_t)nheads * 4, nbc * es,
                             nbc * es, (size_t)nheads * 4, nx * es, nstate, need};
  const void* outs[] = {y, chunk_states, h_last};
  const size_t out_bytes[] = {nx * 4, nstate * nchunks, nstate};
  for (int i = 0; i < 3; ++i) {
    if (!output_clear(outs[i], out_bytes[i], ins, in_bytes, 9)) return MSS_ERR_ALIAS;
    for (int j = i + 1; j < 3; ++j)
      if (outs[i] && outs[j] && overlaps(range_of(outs[i], out_bytes[i]), range_of(outs[j], out_bytes[j])))
        return MSS_ERR_ALIAS;
  }

  mss::SSDParams p;
  p.x = x;
  p.delta = delta;
  p.A = A;
  p.B = B;
  p.C = C;
  p.D = D;
  p.z = z;
  p.h0 = h0;
  p.y = y;
  p.chunk_states = chunk_states;
  p.h_last = h_last;
  p.batch = batch;
  p.seqlen = seqlen;
  p.nheads = nheads;
  p.headdim = headdim;
  p.ngroups = ngroups;
  p.dstate = dstate;
  p.chunk = chunk;
  p.workspace = workspace;
  return hip_status(mss::launch_ssd(p, static_cast<hipStream_t>(hip_stream)));
}


// The forward's limits with chunk 64 (d_state up to 256).  Up to 128 states
// one pass takes them all; above, two halves run one after the other.
static mss_status ssd_bwd_check_shape(int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim,
                                      int64_t ngroups, int64_t dstate, mss_dtype t) {
  return ssd_check_shape(batch, seqlen, nheads, headdim, ngroups, dstate, 64, t);
}

static size_t ssd_bwd_need(int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim, int64_t ngroups,
                           int64_t dstate) {
  return dstate > 128 ? mss::ssd_bwd_halves_workspace_bytes(batch, seqlen, nheads, headdim, ngroups)
                      : mss::ssd_bwd_workspace_bytes(batch, seqlen, nheads, headdim, ngroups, dstate);
}

size_t mss_ssd_bwd_workspace_size(int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim,
                                  int64_t ngroups, int64_t dstate, mss_dtype in_dtype) {
  if (ssd_bwd_check_shape(batch, seqlen, nheads, headdim, ngroups, dstate, in_dtype) != MSS_OK) return 0;
  return ssd_bwd_need(batch, seqlen, nheads, headdim, ngroups, dstate);
}

mss_status mss_ssd_chunk_bwd(const void* x, const float* delta, const float* A, const void* B, const void* C,
                             const float* D, const void* z, const float* h0, const float* dy, const float* dh_last,
                             float* dx, float* ddelta, float* dA, float* dB, float* dC, float* dD, float* dz,
                             float* dh0, int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim,
                             int64_t ngroups, int64_t dstate, mss_dtype in_dtype, uint32_t flags, void* workspace,
                             size_t workspace_bytes, void* hip_stream) {
  if (!x || !delta || !A || !B || !C || !dy || !dx || !ddelta || !dA || !dB || !dC) return MSS_ERR_NULL;
  if ((z == nullptr) != (dz == nullptr)) return MSS_ERR_NULL;
  mss_status st = ssd_bwd_check_shape(batch, seqlen, nheads, headdim, ngroups, dstate, in_dtype);
  if (st != MSS_OK) return st;
  if (flags != 0) return MSS_ERR_UNSUPPORTED;
  const void* all[] = {x, delta, A, B, C, D, z, h0, dy, dh_last, dx, ddelta, dA, dB, dC, dD, dz, dh0, workspace};
  for (const void* p : all)
    if (p && !aligned16(p)) return MSS_ERR_ALIGN;
  const size_t need = ssd_bwd_need(batch, seqlen, nheads, headdim, ngroups, dstate);
  if (!workspace || workspace_bytes < need) return MSS_ERR_WORKSPACE;

  const size_t es = elem_size(in_dtype);
  const size_t nx = (size_t)batch * seqlen * nheads * headdim;
  const size_t nbc = (size_t)batch * seqlen * ngroups * dstate;
  const size_t nstate = (size_t)batch * nheads * headdim * dstate * sizeof(float);
  const size_t ndl = (size_t)batch * seqlen * nheads * 4;
  const void* ins[] = {x, delta, A, B, C, D, z, h0, dy, dh_last, workspace};
  const size_t in_bytes[] = {nx * es, ndl, (size_t)nheads * 4, nbc * es, nbc * es, (size_t)nheads * 4, nx * es,
                             nstate, nx * 4, nstate, need};
  const void* outs[] = {dx, ddelta, dA, dB, dC, dD, dz, dh0};
  const size_t out_bytes[] = {nx * 4, ndl, (size_t)nheads * 4, nbc * 4, nbc * 4, (size_t)nheads * 4, nx * 4, nstate};
  for (int i = 0; i < 8; ++i) {
    if (!output_clear(outs[i], out_bytes[i], ins, in_bytes, 11)) return MSS_ERR_ALIAS;
    for (int j = i + 1; j < 8; ++j)
      if (outs[i] && outs[j] && overlaps(range_of(outs[i], out_bytes[i]), range_of(outs[j], out_bytes[j])))
        return MSS_ERR_ALIAS;
  }

  mss::SSDBwdParams p;
  p.x = x;
  p.delta = delta;
  p.A = A;
  p.B = B;
  p.C = C;
  p.D = D;
  p.z = z;
  p.h0 = h0;
  p.dy = dy;
  p.dh_last = dh_last;
  p.dx = dx;
  p.ddelta = ddelta;
  p.dA = dA;
  p.dB = dB;
  p.dC = dC;
  p.dD = dD;
  p.dz = dz;
  p.dh0 = dh0;
  p.batch = batch;
  p.seqlen = seqlen;
  p.nheads = nheads;
  p.headdim = headdim;
  p.ngroups = ngroups;
  p.dstate = dstate;
  p.workspace = workspace;
  if (dstate > 128) return hip_status(mss::launch_ssd_bwd_halves(p, static_cast<hipStream_t>(hip_stream)));
  return hip_status(mss::launch_ssd_bwd(p, static_cast<hipStream_t>(hip_stream)));
}

// ------------------------------------------------- norms around the mixer
namespace {

// Rows of a [rows, cols] tensor in memory.
struct RowSet {
  const void* p;        // null: absent
  int64_t stride, cols; // bytes
  int64_t rows;
};

RowSet row_set(const void* p, int64_t stride, int64_t rows, int64_t cols, mss_dtype t) {
  const int64_t es = (int64_t)elem_size(t);
  return RowSet{p, stride * es, cols * es, rows};
}
RowSet dense_set(const void* p, int64_t bytes) { return RowSet{p, bytes, bytes, 1}; }

Range span_of(const RowSet& s) { return range_of(s.p, (size_t)((s.rows - 1) * s.stride + s.cols)); }

// Whether two row sets share a byte: exactly for rows of the same stride
// (slices of one wider buffer interleave), by their whole spans otherwise.
bool rows_overlap(const RowSet& a, const RowSet& b) {
  if (a.p == nullptr || b.p == nullptr || !overlaps(span_of(a), span_of(b))) return false;
  if (a.rows == 1 || b.rows == 1 || a.stride != b.stride) return true;
  const int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p));
  const int64_t m = ((d % a.stride) + a.stride) % a.stride;  // b's start within a row of a
  return m < a.cols || a.stride - m < b.cols;
}

// Every output against every input and the outputs before it.
bool outputs_clear(const RowSet* outs, int nouts, const RowSet* ins, int nins) {
  for (int o = 0; o < nouts; ++o) {
    for (int i = 0; i < nins; ++i)
      if (rows_overlap(outs[o], ins[i])) return false;
    for (int i = 0; i < o; ++i)
      if (rows_overlap(outs[o], outs[i])) return false;
  }
  return true;
}

constexpr int64_t kMaxSpan = 1LL << 47;
constexpr int64_t kNormCols = 16384;

// Sizes: positive; a stride holds its row; spans that a 64-bit byte offset holds.
bool rows_ok(int64_t rows, int64_t cols) { return rows > 0 && cols > 0 && cols < (1LL << 30) && rows < kMaxSpan / cols; }
bool stride_ok(const void* p, int64_t stride, int64_t rows, int64_t cols) {
  return p == nullptr || (stride >= cols && stride < kMaxSpan / rows);
}

bool elem_aligned(const void* p, mss_dtype t) { return (reinterpret_cast<uintptr_t>(p) & (elem_size(t) - 1)) == 0; }
bool f32_aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool i64_aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

int64_t pitch8(int64_t cols) { return (cols + 31) / 32 * 32; }
RowSet q_set(const void* q, int64_t rows, int64_t cols) { return dense_set(q, rows * pitch8(cols)); }
RowSet scale_set(const void* s, int64_t rows, int64_t cols) { return dense_set(s, rows * (pitch8(cols) / 32)); }

// The type pairs that the norm kernels take: the wide tensor at least as wide as the other.
mss_status norm_types(mss_dtype io, mss_dtype wide) {
  if (!dtype_ok(io) || !dtype_ok(wide)) return MSS_ERR_DTYPE;
  return io == MSS_FP32 && wide == MSS_BF16 ? MSS_ERR_UNSUPPORTED : MSS_OK;
}

bool eps_ok(float eps) { return eps > 0.f && eps < __builtin_inff(); }

}  // namespace

mss_status mss_add_norm_fwd(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                            const float* weight, const float* post_weight, const float* gamma, float scale, float eps,
                            void* out, int64_t out_stride, void* residual_out, int64_t residual_out_stride,
                            int8_t* out_q, uint8_t* out_scale, int64_t rows, int64_t cols, mss_dtype io_dtype,
                            mss_dtype res_dtype, uint32_t flags, void* hip_stream) {
  if (!x || !weight || !out || !residual_out || (out_q == nullptr) != (out_scale == nullptr)) return MSS_ERR_NULL;
  if (!rows_ok(rows, cols)) return MSS_ERR_SHAPE;
  mss_status st = norm_types(io_dtype, res_dtype);
  if (st != MSS_OK) return st;
  if (!stride_ok(x, x_stride, rows, cols) || !stride_ok(residual, residual_stride, rows, cols) ||
      !stride_ok(out, out_stride, rows, cols) || !stride_ok(residual_out, residual_out_stride, rows, cols))
    return MSS_ERR_SHAPE;
  if (flags != 0 || cols > kNormCols || !eps_ok(eps)) return MSS_ERR_UNSUPPORTED;
  if (!elem_aligned(x, io_dtype) || !elem_aligned(out, io_dtype) || !elem_aligned(residual, res_dtype) ||
      !elem_aligned(residual_out, res_dtype) || !f32_aligned(weight) || !f32_aligned(post_weight) ||
      !f32_aligned(gamma) || !aligned16(out_q))
    return MSS_ERR_ALIGN;
  const RowSet ins[] = {row_set(x, x_stride, rows, cols, io_dtype),
                        row_set(residual, residual_stride, rows, cols, res_dtype), dense_set(weight, cols * 4),
                        dense_set(post_weight, cols * 4), dense_set(gamma, cols * 4)};
  const RowSet outs[] = {row_set(out, out_stride, rows, cols, io_dtype),
                         row_set(residual_out, residual_out_stride, rows, cols, res_dtype), q_set(out_q, rows, cols),
                         scale_set(out_scale, rows, cols)};
  if (!outputs_clear(outs, 4, ins, 5)) return MSS_ERR_ALIAS;
  mss::AddNormFwdParams p;
  p.x = x;
  p.residual = residual;
  p.weight = weight;
  p.post_weight = post_weight;
  p.gamma = gamma;
  p.out = out;
  p.residual_out = residual_out;
  p.out_q = out_q;
  p.out_scale = out_scale;
  p.x_stride = x_stride;
  p.residual_stride = residual_stride;
  p.out_stride = out_stride;
  p.residual_out_stride = residual_out_stride;
  p.rows = rows;
  p.cols = cols;
  p.scale = scale;
  p.eps = eps;
  p.io_bf16 = io_dtype == MSS_BF16;
  p.res_bf16 = res_dtype == MSS_BF16;
  return hip_status(mss::launch_add_norm_fwd(p, static_cast<hipStream_t>(hip_stream)));
}

size_t mss_add_norm_bwd_workspace_size(int64_t rows, int64_t cols, int64_t ngrads) {
  if (!rows_ok(rows, cols) || cols > kNormCols || ngrads < 1 || ngrads > 3) return 0;
  return mss::add_norm_bwd_workspace_bytes(rows, cols, (int)ngrads);
}

mss_status mss_add_norm_bwd(const void* dout, int64_t dout_stride, const void* dresidual_out,
                            int64_t dresidual_out_stride, const void* r, int64_t r_stride, const uint8_t* r_scale,
                            const void* x, int64_t x_stride, const uint8_t* x_scale, const float* weight,
                            const float* post_weight, const float* gamma, float scale, float eps, void* dx,
                            int64_t dx_stride, void* dresidual, int64_t dresidual_stride, float* dweight,
                            float* dpost_weight, float* dgamma, int64_t rows, int64_t cols, mss_dtype io_dtype,
                            mss_dtype res_dtype, uint32_t flags, void* workspace, size_t workspace_bytes,
                            void* hip_stream) {
  if (!dout || !r || !weight || !dweight || (post_weight == nullptr) != (dpost_weight == nullptr) ||
      (gamma == nullptr) != (dgamma == nullptr) || ((post_weight || gamma) && !x))
    return MSS_ERR_NULL;
  if (!rows_ok(rows, cols)) return MSS_ERR_SHAPE;
  mss_status st = norm_types(io_dtype, res_dtype);
  if (st != MSS_OK) return st;
  const bool packed = r_scale != nullptr, use_x = post_weight || gamma;
  if (!use_x) x = nullptr, x_scale = nullptr;
  if (!stride_ok(dout, dout_stride, rows, cols) || !stride_ok(dresidual_out, dresidual_out_stride, rows, cols) ||
      (!packed && (!stride_ok(r, r_stride, rows, cols) || !stride_ok(x, x_stride, rows, cols))) ||
      !stride_ok(dx, dx_stride, rows, cols) || !stride_ok(dresidual, dresidual_stride, rows, cols))
    return MSS_ERR_SHAPE;
  if (flags != 0 || cols > kNormCols || !eps_ok(eps) || (use_x && (x_scale != nullptr) != packed))
    return MSS_ERR_UNSUPPORTED;
  if (!elem_aligned(dout, io_dtype) || !elem_aligned(dresidual_out, res_dtype) || !elem_aligned(dx, io_dtype) ||
      !elem_aligned(dresidual, res_dtype) || !f32_aligned(weight) || !f32_aligned(post_weight) || !f32_aligned(gamma) ||
      !f32_aligned(dweight) || !f32_aligned(dpost_weight) || !f32_aligned(dgamma) ||
      (packed ? !aligned16(r) || !aligned16(x) : !elem_aligned(r, res_dtype) || !elem_aligned(x, io_dtype)) ||
      !aligned16(workspace))
    return MSS_ERR_ALIGN;
  const int ngrads = 1 + (post_weight != nullptr) + (gamma != nullptr);
  const size_t need = mss::add_norm_bwd_workspace_bytes(rows, cols, ngrads);
  if (!workspace || workspace_bytes < need) return MSS_ERR_WORKSPACE;
  const RowSet ins[] = {row_set(dout, dout_stride, rows, cols, io_dtype),
                        row_set(dresidual_out, dresidual_out_stride, rows, cols, res_dtype),
                        packed ? q_set(r, rows, cols) : row_set(r, r_stride, rows, cols, res_dtype),
                        packed ? q_set(x, rows, cols) : row_set(x, x_stride, rows, cols, io_dtype),
                        scale_set(r_scale, rows, cols), scale_set(x_scale, rows, cols), dense_set(weight, cols * 4),
                        dense_set(post_weight, cols * 4), dense_set(gamma, cols * 4),
                        dense_set(workspace, (int64_t)need)};
  const RowSet outs[] = {row_set(dx, dx_stride, rows, cols, io_dtype),
                         row_set(dresidual, dresidual_stride, rows, cols, res_dtype), dense_set(dweight, cols * 4),
                         dense_set(dpost_weight, cols * 4), dense_set(dgamma, cols * 4)};
  if (!outputs_clear(outs, 5, ins, 10)) return MSS_ERR_ALIAS;
  mss::AddNormBwdParams p;
  p.dout = dout;
  p.dresidual_out = dresidual_out;
  p.r = r;
  p.r_scale = r_scale;
  p.x = x;
  p.x_scale = x_scale;
  p.weight = weight;
  p.post_weight = post_weight;
  p.gamma = gamma;
  p.dx = dx;
  p.dresidual = dresidual;
  p.dweight = dweight;
  p.dpost_weight = dpost_weight;
  p.dgamma = dgamma;
  p.dout_stride = dout_stride;
  p.dresidual_out_stride = dresidual_out_stride;
  p.r_stride = r_stride;
  p.x_stride = x_stride;
  p.dx_stride = dx_stride;
  p.dresidual_stride = dresidual_stride;
  p.rows = rows;
  p.cols = cols;
  p.scale = scale;
  p.eps = eps;
  p.io_bf16 = io_dtype == MSS_BF16;
  p.res_bf16 = res_dtype == MSS_BF16;
  p.workspace = workspace;
  return hip_status(mss::launch_add_norm_bwd(p, static_cast<hipStream_t>(hip_stream)));
}

// Shape checks that both directions of the gated norm share.
static mss_status gated_norm_shape(int64_t rows, int64_t cols, int64_t ngroups, mss_dtype y_dtype, mss_dtype io_dtype) {
  if (!rows_ok(rows, cols) || ngroups <= 0) return MSS_ERR_SHAPE;
  const mss_status st = norm_types(io_dtype, y_dtype);
  if (st != MSS_OK) return st;
  if (ngroups > 65535 || cols % ngroups != 0 || cols / ngroups > kNormCols) return MSS_ERR_UNSUPPORTED;
  return MSS_OK;
}
static bool groups_pack(int64_t cols, int64_t ngroups) { return ngroups == 1 || cols / ngroups % 32 == 0; }

mss_status mss_gated_norm_fwd(const void* y, int64_t y_stride, const void* z, int64_t z_stride, const float* weight,
                              float eps, void* out, int64_t out_stride, int8_t* y_q, uint8_t* y_scale, int8_t* z_q,
                              uint8_t* z_scale, int8_t* out_q, uint8_t* out_scale, int64_t rows, int64_t cols,
                              int64_t ngroups, mss_dtype y_dtype, mss_dtype io_dtype, uint32_t flags,
                              void* hip_stream) {
  const bool keep = y_q != nullptr;
  if (!y || !weight || !out || keep != (y_scale != nullptr) || (out_q == nullptr) != (out_scale == nullptr) ||
      (z_q != nullptr) != (keep && z) || (z_scale != nullptr) != (keep && z))
    return MSS_ERR_NULL;
  mss_status st = gated_norm_shape(rows, cols, ngroups, y_dtype, io_dtype);
  if (st != MSS_OK) return st;
  if (!stride_ok(y, y_stride, rows, cols) || !stride_ok(z, z_stride, rows, cols) ||
      !stride_ok(out, out_stride, rows, cols))
    return MSS_ERR_SHAPE;
  if ((flags & ~MSS_FLAG_NORM_FIRST) || !eps_ok(eps) || ((keep || out_q) && !groups_pack(cols, ngroups)))
    return MSS_ERR_UNSUPPORTED;
  if (!elem_aligned(y, y_dtype) || !elem_aligned(z, io_dtype) || !elem_aligned(out, io_dtype) || !f32_aligned(weight) ||
      !aligned16(y_q) || !aligned16(z_q) || !aligned16(out_q))
    return MSS_ERR_ALIGN;
  const RowSet ins[] = {row_set(y, y_stride, rows, cols, y_dtype), row_set(z, z_stride, rows, cols, io_dtype),
                        dense_set(weight, cols * 4)};
  const RowSet outs[] = {row_set(out, out_stride, rows, cols, io_dtype), q_set(y_q, rows, cols),
                         scale_set(y_scale, rows, cols), q_set(z_q, rows, cols), scale_set(z_scale, rows, cols),
                         q_set(out_q, rows, cols), scale_set(out_scale, rows, cols)};
  if (!outputs_clear(outs, 7, ins, 3)) return MSS_ERR_ALIAS;
  mss::GatedNormFwdParams p;
  p.y = y;
  p.z = z;
  p.weight = weight;
  p.out = out;
  p.y_q = y_q;
  p.y_scale = y_scale;
  p.z_q = z_q;
  p.z_scale = z_scale;
  p.out_q = out_q;
  p.out_scale = out_scale;
  p.y_stride = y_stride;
  p.z_stride = z_stride;
  p.out_stride = out_stride;
  p.rows = rows;
  p.cols = cols;
  p.ngroups = ngroups;
  p.eps = eps;
  p.y_bf16 = y_dtype == MSS_BF16;
  p.io_bf16 = io_dtype == MSS_BF16;
  p.norm_first = (flags & MSS_FLAG_NORM_FIRST) != 0;
  return hip_status(mss::launch_gated_norm_fwd(p, static_cast<hipStream_t>(hip_stream)));
}

size_t mss_gated_norm_bwd_workspace_size(int64_t rows, int64_t cols, int64_t ngroups) {
  if (gated_norm_shape(rows, cols, ngroups, MSS_FP32, MSS_FP32) != MSS_OK) return 0;
  return mss::gated_norm_bwd_workspace_bytes(rows, cols, ngroups);
}

mss_status mss_gated_norm_bwd(const void* dout, int64_t dout_stride, const void* y, int64_t y_stride,
                              const uint8_t* y_scale, const void* z, int64_t z_stride, const uint8_t* z_scale,
                              const float* weight, float eps, void* dy, int64_t dy_stride, void* dz, int64_t dz_stride,
                              float* dweight, int64_t rows, int64_t cols, int64_t ngroups, mss_dtype y_dtype,
                              mss_dtype io_dtype, uint32_t flags, void* workspace, size_t workspace_bytes,
                              void* hip_stream) {
  if (!dout || !y || !weight || !dy || !dweight || (z == nullptr) != (dz == nullptr)) return MSS_ERR_NULL;
  mss_status st = gated_norm_shape(rows, cols, ngroups, y_dtype, io_dtype);
  if (st != MSS_OK) return st;
  const bool packed = y_scale != nullptr;
  if (!stride_ok(dout, dout_stride, rows, cols) || !stride_ok(dy, dy_stride, rows, cols) ||
      !stride_ok(dz, dz_stride, rows, cols) ||
      (!packed && (!stride_ok(y, y_stride, rows, cols) || !stride_ok(z, z_stride, rows, cols))))
    return MSS_ERR_SHAPE;
  if ((flags & ~MSS_FLAG_NORM_FIRST) || !eps_ok(eps) || (z_scale != nullptr) != (packed && z) ||
      (packed && !groups_pack(cols, ngroups)))
    return MSS_ERR_UNSUPPORTED;
  if (!elem_aligned(dout, io_dtype) || !elem_aligned(dy, y_dtype) || !elem_aligned(dz, io_dtype) ||
      !f32_aligned(weight) || !f32_aligned(dweight) ||
      (packed ? !aligned16(y) || !aligned16(z) : !elem_aligned(y, y_dtype) || !elem_aligned(z, io_dtype)) ||
      !aligned16(workspace))
    return MSS_ERR_ALIGN;
  const size_t need = mss::gated_norm_bwd_workspace_bytes(rows, cols, ngroups);
  if (!workspace || workspace_bytes < need) return MSS_ERR_WORKSPACE;
  const RowSet ins[] = {row_set(dout, dout_stride, rows, cols, io_dtype),
                        packed ? q_set(y, rows, cols) : row_set(y, y_stride, rows, cols, y_dtype),
                        packed ? q_set(z, rows, cols) : row_set(z, z_stride, rows, cols, io_dtype),
                        scale_set(y_scale, rows, cols), scale_set(z_scale, rows, cols), dense_set(weight, cols * 4),
                        dense_set(workspace, (int64_t)need)};
  const RowSet outs[] = {row_set(dy, dy_stride, rows, cols, y_dtype), row_set(dz, dz_stride, rows, cols, io_dtype),
                         dense_set(dweight, cols * 4)};
  if (!outputs_clear(outs, 3, ins, 7)) return MSS_ERR_ALIAS;
  mss::GatedNormBwdParams p;
  p.dout = dout;
  p.y = y;
  p.y_scale = y_scale;
  p.z = z;
  p.z_scale = z_scale;
  p.weight = weight;
  p.dy = dy;
  p.dz = dz;
  p.dweight = dweight;
  p.dout_stride = dout_stride;
  p.y_stride = y_stride;
  p.z_stride = z_stride;
  p.dy_stride = dy_stride;
  p.dz_stride = dz_stride;
  p.rows = rows;
  p.cols = cols;
  p.ngroups = ngroups;
  p.eps = eps;
  p.y_bf16 = y_dtype == MSS_BF16;
  p.io_bf16 = io_dtype == MSS_BF16;
  p.norm_first = (flags & MSS_FLAG_NORM_FIRST) != 0;
  p.workspace = workspace;
  return hip_status(mss::launch_gated_norm_bwd(p, static_cast<hipStream_t>(hip_stream)));
}

// ------------------------------------------------- 8-bit checkpoints
static mss_status ckpt8_check(const void* x, int64_t x_stride, const void* q, const void* scale, int64_t rows,
                              int64_t cols, mss_dtype dtype, bool pack) {
  if (!x || !q || !scale) return MSS_ERR_NULL;
  if (!rows_ok(rows, cols)) return MSS_ERR_SHAPE;
  if (!dtype_ok(dtype)) return MSS_ERR_DTYPE;
  // A launch holds fewer than 2^32 threads, each of four vectors of eight.
  if (!stride_ok(x, x_stride, rows, cols) || rows >= (1LL << 36) / pitch8(cols)) return MSS_ERR_SHAPE;
  if (!elem_aligned(x, dtype) || !aligned16(q)) return MSS_ERR_ALIGN;
  const RowSet a[] = {row_set(x, x_stride, rows, cols, dtype)};
  const RowSet b[] = {q_set(q, rows, cols), scale_set(scale, rows, cols)};
  if (pack ? !outputs_clear(b, 2, a, 1) : !outputs_clear(a, 1, b, 2)) return MSS_ERR_ALIAS;
  return MSS_OK;
}

mss_status mss_pack8(const void* x, int64_t x_stride, int8_t* q, uint8_t* scale, int64_t rows, int64_t cols,
                     mss_dtype dtype, void* hip_stream) {
  const mss_status st = ckpt8_check(x, x_stride, q, scale, rows, cols, dtype, true);
  if (st != MSS_OK) return st;
  const mss::Ckpt8Params p{x, nullptr, q, scale, x_stride, rows, cols, dtype == MSS_BF16};
  return hip_status(mss::launch_pack8(p, static_cast<hipStream_t>(hip_stream)));
}

mss_status mss_unpack8(const int8_t* q, const uint8_t* scale, void* x, int64_t x_stride, int64_t rows, int64_t cols,
                       mss_dtype dtype, void* hip_stream) {
  const mss_status st = ckpt8_check(x, x_stride, q, scale, rows, cols, dtype, false);
  if (st != MSS_OK) return st;
  const mss::Ckpt8Params p{nullptr, x, const_cast<int8_t*>(q), const_cast<uint8_t*>(scale), x_stride, rows, cols,
                           dtype == MSS_BF16};
  return hip_status(mss::launch_unpack8(p, static_cast<hipStream_t>(hip_stream)));
}

// (A launch of the copy that aligns dy holds fewer than 2^32 threads, each of four vectors of eight.)
static bool wgrad8_shape_ok(int64_t tokens, int64_t outs, int64_t ins) {
  return tokens > 0 && outs > 0 && ins > 0 && tokens <= (1LL << 35) && outs <= (1LL << 20) && ins <= (1LL << 20) &&
         outs * ins <= (1LL << 34) && tokens < (1LL << 36) / (outs + 7);
}

size_t mss_wgrad8_workspace_size(const void* dy, int64_t dy_stride, int64_t tokens, int64_t outs, int64_t ins) {
  return wgrad8_shape_ok(tokens, outs, ins) ? mss::wgrad8_workspace_bytes(dy, dy_stride, tokens, outs, ins) : 0;
}

mss_status mss_wgrad8(const void* dy, int64_t dy_stride, const int8_t* q, const uint8_t* scale, void* dw,
                      int64_t tokens, int64_t outs, int64_t ins, mss_dtype dy_dtype, mss_dtype dw_dtype,
                      uint32_t flags, void* workspace, size_t workspace_bytes, void* hip_stream) {
  if (!dy || !q || !scale || !dw) return MSS_ERR_NULL;
  if (!dtype_ok(dy_dtype) || !dtype_ok(dw_dtype)) return MSS_ERR_DTYPE;
  if (!wgrad8_shape_ok(tokens, outs, ins) || !stride_ok(dy, dy_stride, tokens, outs)) return MSS_ERR_SHAPE;
  if (dy_dtype != MSS_BF16 || (flags & ~MSS_FLAG_ACCUMULATE)) return MSS_ERR_UNSUPPORTED;
  if (!elem_aligned(dy, dy_dtype) || !aligned16(q) || !aligned16(dw) || !aligned16(workspace)) return MSS_ERR_ALIGN;
  const size_t need = mss::wgrad8_workspace_bytes(dy, dy_stride, tokens, outs, ins);
  if (!workspace || workspace_bytes < need) return MSS_ERR_WORKSPACE;
  const RowSet in[] = {row_set(dy, dy_stride, tokens, outs, dy_dtype), q_set(q, tokens, ins),
                       scale_set(scale, tokens, ins), dense_set(workspace, (int64_t)need)};
  const RowSet out[] = {dense_set(dw, outs * ins * (int64_t)elem_size(dw_dtype))};
  if (!outputs_clear(out, 1, in, 4)) return MSS_ERR_ALIAS;
  const mss::Wgrad8Params p{dy,   q,    scale, dw, dy_stride, tokens, outs, ins, dw_dtype == MSS_BF16,
                            (flags & MSS_FLAG_ACCUMULATE) != 0, workspace};
  return hip_status(mss::launch_wgrad8(p, static_cast<hipStream_t>(hip_stream)));
}

// ------------------------------------------------- gated linear recurrence
namespace {

bool rate_ok(float c) { return c > 0.f && c < __builtin_inff(); }

mss_status recurrence_shape(int64_t batch, int64_t seqlen, int64_t dim, mss_dtype t) {
  if (!dtype_ok(t)) return MSS_ERR_DTYPE;
  if (batch <= 0 || seqlen <= 0 || dim <= 0) return MSS_ERR_SHAPE;
  // Workgroups of a launch, each of up to 512 threads: fewer than 2^32 threads.
  constexpr int64_t most = 1LL << 23;
  if (batch >= most || seqlen >= most * 64 || dim >= (1LL << 29)) return MSS_ERR_SHAPE;
  const int64_t chunks = batch * ((seqlen + 63) / 64);
  if (chunks >= most || chunks * ((dim + 63) / 64) >= most) return MSS_ERR_SHAPE;
  return rows_ok(batch * seqlen, dim) ? MSS_OK : MSS_ERR_SHAPE;
}

}  // namespace

size_t mss_gated_recurrence_workspace_size(int64_t batch, int64_t seqlen, int64_t dim, mss_dtype io_dtype) {
  if (recurrence_shape(batch, seqlen, dim, io_dtype) != MSS_OK) return 0;
  return mss::recurrence_fwd_workspace_bytes(batch, seqlen, dim, io_dtype == MSS_BF16);
}

size_t mss_gated_recurrence_bwd_workspace_size(int64_t batch, int64_t seqlen, int64_t dim, mss_dtype io_dtype) {
  if (recurrence_shape(batch, seqlen, dim, io_dtype) != MSS_OK) return 0;
  return mss::recurrence_bwd_workspace_bytes(batch, seqlen, dim, io_dtype == MSS_BF16);
}

mss_status mss_gated_recurrence_fwd(const void* x, int64_t x_stride, const void* gate_a, int64_t gate_a_stride,
                                    const void* gate_x, int64_t gate_x_stride, const float* lam, float c,
                                    const float* h0, const uint8_t* starts, void* y, int64_t y_stride, float* h_last,
                                    float* states, int64_t batch, int64_t seqlen, int64_t dim, mss_dtype io_dtype,
                                    uint32_t flags, void* workspace, size_t workspace_bytes, void* hip_stream) {
  if (!x || !gate_a || !gate_x || !lam || !y) return MSS_ERR_NULL;
  const mss_status st = recurrence_shape(batch, seqlen, dim, io_dtype);
  if (st != MSS_OK) return st;
  const int64_t rows = batch * seqlen;
  if (!stride_ok(x, x_stride, rows, dim) || !stride_ok(gate_a, gate_a_stride, rows, dim) ||
      !stride_ok(gate_x, gate_x_stride, rows, dim) || !stride_ok(y, y_stride, rows, dim))
    return MSS_ERR_SHAPE;
  if (flags != 0 || !rate_ok(c)) return MSS_ERR_UNSUPPORTED;
  if (!elem_aligned(x, io_dtype) || !elem_aligned(gate_a, io_dtype) || !elem_aligned(gate_x, io_dtype) ||
      !elem_aligned(y, io_dtype) || !f32_aligned(lam) || !f32_aligned(h0) || !f32_aligned(h_last) ||
      !f32_aligned(states) || !aligned16(workspace))
    return MSS_ERR_ALIGN;
  const size_t need = mss::recurrence_fwd_workspace_bytes(batch, seqlen, dim, io_dtype == MSS_BF16);
  if (!workspace || workspace_bytes < need) return MSS_ERR_WORKSPACE;
  const int64_t chunks = batch * ((seqlen + mss::kRecurrenceChunk - 1) / mss::kRecurrenceChunk);
  const RowSet ins[] = {row_set(x, x_stride, rows, dim, io_dtype), row_set(gate_a, gate_a_stride, rows, dim, io_dtype),
                        row_set(gate_x, gate_x_stride, rows, dim, io_dtype), dense_set(lam, dim * 4),
                        dense_set(h0, batch * dim * 4), dense_set(starts, rows),
                        dense_set(workspace, (int64_t)need)};
  const RowSet outs[] = {row_set(y, y_stride, rows, dim, io_dtype), dense_set(h_last, batch * dim * 4),
                         dense_set(states, chunks * dim * 4)};
  if (!outputs_clear(outs, 3, ins, 7)) return MSS_ERR_ALIAS;
  mss::RecurrenceFwdParams p;
  p.x = x;
  p.gate_a = gate_a;
  p.gate_x = gate_x;
  p.lam = lam;
  p.h0 = h0;
  p.starts = starts;
  p.y = y;
  p.h_last = h_last;
  p.states = states;
  p.x_stride = x_stride;
  p.gate_a_stride = gate_a_stride;
  p.gate_x_stride = gate_x_stride;
  p.y_stride = y_stride;
  p.batch = batch;
  p.seqlen = seqlen;
  p.dim = dim;
  p.c = c;
  p.bf16 = io_dtype == MSS_BF16;
  p.workspace = workspace;
  return hip_status(mss::launch_recurrence_fwd(p, static_cast<hipStream_t>(hip_stream)));
}

mss_status mss_gated_recurrence_bwd(const void* dy, int64_t dy_stride, const void* x, int64_t x_stride,
                                    const void* gate_a, int64_t gate_a_stride, const void* gate_x,
                                    int64_t gate_x_stride, const float* lam, float c, const uint8_t* starts,
                                    const float* states, const float* dh_last, void* dx, int64_t dx_stride,
                                    void* dgate_a, int64_t dgate_a_stride, void* dgate_x, int64_t dgate_x_stride,
                                    float* dlam, float* dh0, int64_t batch, int64_t seqlen, int64_t dim,
                                    mss_dtype io_dtype, uint32_t flags, void* workspace, size_t workspace_bytes,
                                    void* hip_stream) {
  if (!dy || !x || !gate_a || !gate_x || !lam || !states || !dx || !dgate_a || !dgate_x || !dlam) return MSS_ERR_NULL;
  const mss_status st = recurrence_shape(batch, seqlen, dim, io_dtype);
  if (st != MSS_OK) return st;
  const int64_t rows = batch * seqlen;
  if (!stride_ok(dy, dy_stride, rows, dim) || !stride_ok(x, x_stride, rows, dim) ||
      !stride_ok(gate_a, gate_a_stride, rows, dim) || !stride_ok(gate_x, gate_x_stride, rows, dim) ||
      !stride_ok(dx, dx_stride, rows, dim) || !stride_ok(dgate_a, dgate_a_stride, rows, dim) ||
      !stride_ok(dgate_x, dgate_x_stride, rows, dim))
    return MSS_ERR_SHAPE;
  if (flags != 0 || !rate_ok(c)) return MSS_ERR_UNSUPPORTED;
  if (!elem_aligned(dy, io_dtype) || !elem_aligned(x, io_dtype) || !elem_aligned(gate_a, io_dtype) ||
      !elem_aligned(gate_x, io_dtype) || !elem_aligned(dx, io_dtype) || !elem_aligned(dgate_a, io_dtype) ||
      !elem_aligned(dgate_x, io_dtype) || !f32_aligned(lam) || !f32_aligned(states) || !f32_aligned(dh_last) ||
      !f32_aligned(dlam) || !f32_aligned(dh0) || !aligned16(workspace))
    return MSS_ERR_ALIGN;
  const size_t need = mss::recurrence_bwd_workspace_bytes(batch, seqlen, dim, io_dtype == MSS_BF16);
  if (!workspace || workspace_bytes < need) return MSS_ERR_WORKSPACE;
  const int64_t chunks = batch * ((seqlen + mss::kRecurrenceChunk - 1) / mss::kRecurrenceChunk);
  const RowSet ins[] = {row_set(dy, dy_stride, rows, dim, io_dtype), row_set(x, x_stride, rows, dim, io_dtype),
                        row_set(gate_a, gate_a_stride, rows, dim, io_dtype),
                        row_set(gate_x, gate_x_stride, rows, dim, io_dtype), dense_set(lam, dim * 4),
                        dense_set(starts, rows), dense_set(states, chunks * dim * 4),
                        dense_set(dh_last, batch * dim * 4), dense_set(workspace, (int64_t)need)};
  const RowSet outs[] = {row_set(dx, dx_stride, rows, dim, io_dtype),
                         row_set(dgate_a, dgate_a_stride, rows, dim, io_dtype),
                         row_set(dgate_x, dgate_x_stride, rows, dim, io_dtype), dense_set(dlam, dim * 4),
                         dense_set(dh0, batch * dim * 4)};
  if (!outputs_clear(outs, 5, ins, 9)) return MSS_ERR_ALIAS;
  mss::RecurrenceBwdParams p;
  p.dy = dy;
  p.x = x;
  p.gate_a = gate_a;
  p.gate_x = gate_x;
  p.lam = lam;
  p.starts = starts;
  p.states = states;
  p.dh_last = dh_last;
  p.dx = dx;
  p.dgate_a = dgate_a;
  p.dgate_x = dgate_x;
  p.dlam = dlam;
  p.dh0 = dh0;
  p.dy_stride = dy_stride;
  p.x_stride = x_stride;
  p.gate_a_stride = gate_a_stride;
  p.gate_x_stride = gate_x_stride;
  p.dx_stride = dx_stride;
  p.dgate_a_stride = dgate_a_stride;
  p.dgate_x_stride = dgate_x_stride;
  p.batch = batch;
  p.seqlen = seqlen;
  p.dim = dim;
  p.c = c;
  p.bf16 = io_dtype == MSS_BF16;
  p.workspace = workspace;
  return hip_status(mss::launch_recurrence_bwd(p, static_cast<hipStream_t>(hip_stream)));
}

mss_status mss_gated_recurrence_step(const float* h, const int64_t* parents, const void* x, int64_t x_stride,
                                     const void* gate_a, int64_t gate_a_stride, const void* gate_x,
                                     int64_t gate_x_stride, const float* lam, float c, float* h_out, void* y,
                                     int64_t y_stride, int64_t batch, int64_t beams, int64_t dim, mss_dtype io_dtype,
                                     uint32_t flags, void* hip_stream) {
  if (!h || !x || !gate_a || !gate_x || !lam || !h_out || !y) return MSS_ERR_NULL;
  if (!dtype_ok(io_dtype)) return MSS_ERR_DTYPE;
  constexpr int64_t most = 1LL << 31;
  if (batch <= 0 || beams <= 0 || dim <= 0 || batch > most / beams || batch * beams > most / dim) return MSS_ERR_SHAPE;
  const int64_t rows = batch * beams;
  if (!stride_ok(x, x_stride, rows, dim) || !stride_ok(gate_a, gate_a_stride, rows, dim) ||
      !stride_ok(gate_x, gate_x_stride, rows, dim) || !stride_ok(y, y_stride, rows, dim))
    return MSS_ERR_SHAPE;
  if (flags != 0 || !rate_ok(c)) return MSS_ERR_UNSUPPORTED;
  if (!elem_aligned(x, io_dtype) || !elem_aligned(gate_a, io_dtype) || !elem_aligned(gate_x, io_dtype) ||
      !elem_aligned(y, io_dtype) || !f32_aligned(h) || !f32_aligned(h_out) || !f32_aligned(lam) || !i64_aligned(parents))
    return MSS_ERR_ALIGN;
  // In place each thread reads its own element of h before it writes it.
  const bool in_place = h_out == h && parents == nullptr;
  const RowSet ins[] = {row_set(x, x_stride, rows, dim, io_dtype), row_set(gate_a, gate_a_stride, rows, dim, io_dtype),
                        row_set(gate_x, gate_x_stride, rows, dim, io_dtype), dense_set(lam, dim * 4),
                        dense_set(parents, rows * 8), dense_set(in_place ? nullptr : h, rows * dim * 4)};
  const RowSet outs[] = {dense_set(h_out, rows * dim * 4), row_set(y, y_stride, rows, dim, io_dtype)};
  if (!outputs_clear(outs, 2, ins, 6)) return MSS_ERR_ALIAS;
  mss::RecurrenceStepParams p;
  p.h = h;
  p.parents = parents;
  p.x = x;
  p.gate_a = gate_a;
  p.gate_x = gate_x;
  p.lam = lam;
  p.h_out = h_out;
  p.y = y;
  p.x_stride = x_stride;
  p.gate_a_stride = gate_a_stride;
  p.gate_x_stride = gate_x_stride;
  p.y_stride = y_stride;
  p.rows = rows;
  p.beams = beams;
  p.dim = dim;
  p.c = c;
  p.bf16 = io_dtype == MSS_BF16;
  return hip_status(mss::launch_recurrence_step(p, static_cast<hipStream_t>(hip_stream)));
}

// ------------------------------------------------- beam search
static mss_status beam_shape(int64_t batch, int64_t beams, int64_t vocab, int64_t n_out) {
  if (batch <= 0 || beams <= 0 || vocab <= 0 || n_out <= 0 || batch > 65535 || vocab > (1LL << 24)) return MSS_ERR_SHAPE;
  if (beams > 64 || n_out > 64 || n_out > beams * vocab) return MSS_ERR_UNSUPPORTED;
  // Workgroups of 256 threads: fewer than 2^32 threads.
  return mss::beam_select_workgroups(batch, beams, vocab) < (1LL << 24) ? MSS_OK : MSS_ERR_SHAPE;
}

size_t mss_beam_select_workspace_size(int64_t batch, int64_t beams, int64_t vocab, int64_t n_out) {
  return beam_shape(batch, beams, vocab, n_out) == MSS_OK ? mss::beam_select_workspace_bytes(batch, beams, vocab, n_out)
                                                          : 0;
}

mss_status mss_beam_select(const void* logits, int64_t logits_stride, const float* scores, const uint8_t* finished,
                           int64_t eos, float* out_scores, int64_t* parents, int64_t* tokens, uint8_t* out_finished,
                           int64_t batch, int64_t beams, int64_t vocab, int64_t n_out, mss_dtype io_dtype,
                           uint32_t flags, void* workspace, size_t workspace_bytes, void* hip_stream) {
  if (!logits || !scores || !out_scores || !parents || !tokens) return MSS_ERR_NULL;
  if (!dtype_ok(io_dtype)) return MSS_ERR_DTYPE;
  const mss_status st = beam_shape(batch, beams, vocab, n_out);
  if (st != MSS_OK) return st;
  const int64_t rows = batch * beams;
  if (!stride_ok(logits, logits_stride, rows, vocab)) return MSS_ERR_SHAPE;
  if (flags != 0 || eos < -1 || eos >= vocab || (eos < 0 && (finished || out_finished))) return MSS_ERR_UNSUPPORTED;
  if (!elem_aligned(logits, io_dtype) || !f32_aligned(scores) || !f32_aligned(out_scores) || !i64_aligned(parents) ||
      !i64_aligned(tokens) || !aligned16(workspace))
    return MSS_ERR_ALIGN;
  const size_t need = mss::beam_select_workspace_bytes(batch, beams, vocab, n_out);
  if (!workspace || workspace_bytes < need) return MSS_ERR_WORKSPACE;
  const RowSet ins[] = {row_set(logits, logits_stride, rows, vocab, io_dtype), dense_set(scores, rows * 4),
                        dense_set(finished, rows), dense_set(workspace, (int64_t)need)};
  const RowSet outs[] = {dense_set(out_scores, batch * n_out * 4), dense_set(parents, batch * n_out * 8),
                         dense_set(tokens, batch * n_out * 8), dense_set(out_finished, batch * n_out)};
  if (!outputs_clear(outs, 4, ins, 4)) return MSS_ERR_ALIAS;
  mss::BeamSelectParams p;
  p.logits = logits;
  p.scores = scores;
  p.finished = finished;
  p.out_scores = out_scores;
  p.parents = parents;
  p.tokens = tokens;
  p.out_finished = out_finished;
  p.stride = logits_stride;
  p.batch = batch;
  p.beams = beams;
  p.vocab = vocab;
  p.n_out = n_out;
  p.eos = eos;
  p.bf16 = io_dtype == MSS_BF16;
  p.workspace = workspace;
  return hip_status(mss::launch_beam_select(p, static_cast<hipStream_t>(hip_stream)));
}

mss_status mss_reorder_states(void* const* states, const int64_t* row_bytes, int64_t count, const int64_t* parents,
                              int64_t batch, int64_t beams, void* hip_stream) {
  if (!states || !row_bytes || !parents) return MSS_ERR_NULL;
  if (count <= 0 || batch <= 0 || batch > 65535 || beams <= 0) return MSS_ERR_SHAPE;
  if (beams > 64) return MSS_ERR_UNSUPPORTED;
  for (int64_t s = 0; s < count; ++s) {
    if (!states[s]) return MSS_ERR_NULL;
    if (row_bytes[s] <= 0 || row_bytes[s] > (1LL << 30)) return MSS_ERR_SHAPE;
  }
  if (!i64_aligned(parents)) return MSS_ERR_ALIGN;
  const int64_t rows = batch * beams;
  for (int64_t s = 0; s < count; ++s) {
    const Range r = range_of(states[s], (size_t)(rows * row_bytes[s]));
    if (overlaps(r, range_of(parents, (size_t)rows * 8))) return MSS_ERR_ALIAS;
    for (int64_t o = 0; o < s; ++o)
      if (overlaps(r, range_of(states[o], (size_t)(rows * row_bytes[o])))) return MSS_ERR_ALIAS;
  }
  const mss::ReorderParams p{states, row_bytes, count, parents, batch, beams};
  return hip_status(mss::launch_reorder_states(p, static_cast<hipStream_t>(hip_stream)));
}

}  // extern "C"
