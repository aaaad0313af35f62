// C ABI of the attention library: argument validation, TMA tensor maps,
// kernel dispatch and the device status word. See include/fa.h.
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <mutex>

#include <cuda.h>
#include <cuda_runtime.h>

#include "fa.h"
#include "fa_kernels.h"

namespace {

// Status words set by kernels whose bounded waits ran out, one per stream:
// a call launched on a stream reports to that stream's word, which
// fa_device_status(stream) reads and clears. Slot 0 is shared by the streams
// beyond the first kStatusSlots - 1 that a device sees.
constexpr int kStatusSlots = 256;
__device__ unsigned g_status_words[kStatusSlots];
// SM cycles and nanoseconds summed over the CTAs of the forward and dK/dV
// kernels since the last fa_sm_clock_mhz (diagnostic, device-wide).
__device__ unsigned long long g_clock_acc[2];

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

constexpr int kMaxDevices = 64;
struct DeviceState {
  std::once_flag once;
  bool arch_ok = false;
  int num_sms = 0;
  unsigned* status = nullptr;           // device address of g_status_words on this device
  unsigned long long* clock_acc = nullptr;  // device address of g_clock_acc on this device
  std::mutex mu;                        // guards the stream -> slot table below
  const void* owner[kStatusSlots] = {}; // owner[i]: the stream whose calls report to slot i (i >= 1)
  int used = 1;
};
DeviceState g_dev[kMaxDevices];

// The status word of `stream` on this device: the slot the stream was given
// the first time it was seen, or the shared slot 0 once the table is full.
unsigned* stream_slot(DeviceState& s, const void* stream) {
  std::lock_guard<std::mutex> lock(s.mu);
  for (int i = 1; i < s.used; ++i)
    if (s.owner[i] == stream) return s.status + i;
  if (s.used < kStatusSlots) {
    s.owner[s.used] = stream;
    return s.status + s.used++;
  }
  return s.status;
}

// Checks the current device once (compute capability 10.3), resolves the
// device address of the status words on it and returns the word of `stream`.
fa_status device_state(const void* stream, unsigned** status_out, int* num_sms = nullptr,
                       unsigned long long** clock_acc = nullptr) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FA_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevices) return FA_ERR_UNSUPPORTED;
  DeviceState& s = g_dev[dev];
  std::call_once(s.once, [&s, dev] {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess) return;
    if (cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess) return;
    s.arch_ok = (major == 10 && minor == 3);
    if (cudaDeviceGetAttribute(&s.num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) s.num_sms = 0;
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_status_words) == cudaSuccess) s.status = static_cast<unsigned*>(p);
    void* c = nullptr;
    if (cudaGetSymbolAddress(&c, g_clock_acc) == cudaSuccess) s.clock_acc = static_cast<unsigned long long*>(c);
  });
  if (!s.arch_ok) return FA_ERR_ARCH;
  if (!s.status || !s.clock_acc || s.num_sms <= 0) return FA_ERR_CUDA;
  *status_out = stream_slot(s, stream);
  if (num_sms) *num_sms = s.num_sms;
  if (clock_acc) *clock_acc = s.clock_acc;
  return FA_OK;
}

unsigned long long wait_limit_ns() {
  static unsigned long long ns = [] {
    const char* e = std::getenv("FA_WAIT_LIMIT_MS");
    long ms = e ? std::strtol(e, nullptr, 10) : 0;
    if (ms <= 0) ms = 2000;
    return static_cast<unsigned long long>(ms) * 1000000ull;
  }();
  return ns;
}

// FA_TEST_STALL=1 (read at every call): the tensor-core issuer first waits on
// a barrier nothing ever arrives on, so the bounded wait runs out and the
// call reports FA_ERR_TIMEOUT; for exercising failure detection without any
// fault. Off unless set.
int test_stall() {
  const char* e = std::getenv("FA_TEST_STALL");
  return (e && e[0] == '1') ? 1 : 0;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// FP8 head dimensions: multiples of 16 up to 256 (a row of one-byte codes
// must be a multiple of 16 bytes for TMA). The attention kernels are built
// for 128 and 256; a smaller d runs in the next one up, its columns past d
// read as zeros and never stored.
bool fp8_dim(int d) { return d >= 16 && d <= 256 && d % 16 == 0; }

// 3-D map over a [BH, N, d] tensor: dims (d, N, BH), one box = 128 rows by 128
// bytes with 128-byte swizzle. Rows past N read as zero and are not written by
// stores. row, head: distances between rows and between heads in elements.
bool make_map_strided(CUtensorMap* m, const void* ptr, int elt_bytes, int d, int N, long long BH, long long row,
                      long long head, int box_rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(BH)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(row) * elt_bytes, static_cast<cuuint64_t>(head) * elt_bytes};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / elt_bytes), static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUtensorMapDataType dt = elt_bytes == 1   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                 : elt_bytes == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                  : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
  const CUresult r = enc(m, dt, 3,
                         const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// The same over a dense tensor.
bool make_map(CUtensorMap* m, const void* ptr, int elt_bytes, int d, int N, long long BH, int box_rows = 128) {
  return make_map_strided(m, ptr, elt_bytes, d, N, BH, d, static_cast<long long>(d) * N, box_rows);
}

fa_status check_sizes(int B, int Hq, int Hkv, int N, int d, float scale) {
  if (B < 1 || Hq < 1 || Hkv < 1 || N < 1) return FA_ERR_INVALID_ARG;
  if (Hq % Hkv != 0) return FA_ERR_INVALID_ARG;
  // head dims up to 256 in steps of 8 (16-byte rows for TMA); the kernels are
  // built for 64, 128, 192 and 256 and a smaller d runs in the next one up,
  // the columns past d read as zeros and never written. The backward stops
  // at 128 (bwd_dim).
  if (d < 8 || d > 256 || d % 8 != 0) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_INVALID_ARG;
  const long long BH = static_cast<long long>(B) * Hq;
  const long long nq = (N + 127) / 128;
  if (BH > (1LL << 24) || ((nq + 1) / 2) * BH >= (1LL << 31)) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// The one-pass backward kernels hold dK, dV, S^T and dP^T of a 128-key tile
// in TMEM (4 x d columns of 512): up to d = 128. Above that the three-pass
// backward (fa_bwd_wide.cu) serves fa_bwd, fa_bwd_kv, fa_bwd_deterministic
// and fa_bwd_noalloc; the single phases and the block-sparse backward stop at 128.
fa_status bwd_dim(int d, bool wide_ok = false) { return d > 128 && !wide_ok ? FA_ERR_UNSUPPORTED : FA_OK; }

fa_status fwd_common(int elt, const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq,
                     int Hkv, int N, int d, int causal, float scale, void* stream,
                     const unsigned char* mask = nullptr, long long mask_sb = 0, long long mask_sh = 0,
                     int Nk = -1, bool use_pair = false) {
  if (Nk < 0) Nk = N;
  if (!q || !k || !v || !o || !lse) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse)) return FA_ERR_INVALID_ARG;
  fa_status st = check_sizes(B, Hq, Hkv, N, d, scale);
  if (st != FA_OK) return st;
  if (Nk < 1) return FA_ERR_INVALID_ARG;
  if (elt == 4 && d != 64) return FA_ERR_UNSUPPORTED;
  const bool wide = d > 128;                // one query tile per CTA, V in 64-key halves
  if (wide && mask) return FA_ERR_UNSUPPORTED;
  // fa_fwd_pair: CTA pairs (cta_group::2), K loaded in 64-row halves; bf16,
  // 64 < d <= 128, dense only
  const bool pair = use_pair;
  if (pair && (elt != 2 || mask || d <= 64 || d > 128)) return FA_ERR_UNSUPPORTED;
  unsigned* status = nullptr;
  unsigned long long* clock_acc = nullptr;
  st = device_state(stream, &status, nullptr, &clock_acc);
  if (st != FA_OK) return st;
  CUtensorMap mq, mk, mv, mo;
  const long long BHq = static_cast<long long>(B) * Hq, BHkv = static_cast<long long>(B) * Hkv;
  if (!make_map(&mq, q, elt, d, N, BHq) || !make_map(&mk, k, elt, d, Nk, BHkv, pair ? 64 : 128) ||
      !make_map(&mv, v, elt, d, Nk, BHkv, wide ? 64 : 128) || !make_map(&mo, o, elt, d, N, BHq))
    return FA_ERR_CUDA;
  fa::FwdParams p{};
  p.lse = lse;
  p.status = status;
  p.clock_acc = clock_acc;
  p.N = N;
  p.Nk = Nk;
  p.causal_off = Nk - N;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.BH = static_cast<int>(BHq);
  p.causal = causal ? 1 : 0;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.timeout_ns = wait_limit_ns();
  p.test_stall = test_stall();
  p.mask = mask;
  p.mask_sb = mask_sb;
  p.mask_sh = mask_sh;
  p.mask_nt = (N + 127) / 128;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = wide ? fa::launch_fwd_wide(d, mq, mk, mv, mo, p, s)
                        : pair ? fa::launch_fwd_pair(mq, mk, mv, mo, p, s)
                               : fa::launch_fwd(elt, d, mq, mk, mv, mo, p, s);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

struct BwdWorkspace {
  size_t off_lse2, off_d, off_dq, total;   // off_dq: the bytes the deterministic backward needs
  size_t off_count, off_list, total_sparse;  // block-sparse: per dK/dV CTA, its step count and step list
};

BwdWorkspace bwd_workspace(int B, int Hq, int Hkv, int N, int d) {
  const size_t BH = static_cast<size_t>(B) * Hq;
  const size_t NQP = static_cast<size_t>((N + 127) / 128) * 128;
  BwdWorkspace w;
  w.off_lse2 = 0;
  w.off_d = align256(BH * NQP * 4);
  w.off_dq = w.off_d + align256(BH * NQP * 4);
  w.total = w.off_dq + align256(BH * static_cast<size_t>(N) * d * 4);
  const size_t ctas = (NQP / 128) * static_cast<size_t>(B) * Hkv;
  const size_t G = static_cast<size_t>(Hq / (Hkv > 0 ? Hkv : 1));
  w.off_count = w.total;
  w.off_list = w.off_count + align256(ctas * 4);
  w.total_sparse = w.off_list + align256(ctas * G * (NQP / 128) * 4);
  return w;
}

// Validates sizes and workspace, resolves the device, fills BwdParams. With
// lse_d_only the workspace only has to hold the LSE and D parts.
fa_status bwd_setup(int B, int Hq, int Hkv, int N, int d, int causal, float scale, void* workspace,
                    size_t workspace_bytes, fa::BwdParams* p, int* num_sms, void* stream, bool lse_d_only = false,
                    const unsigned char* mask = nullptr, long long mask_sb = 0, long long mask_sh = 0,
                    int Nk = -1) {
  if (Nk < 0) Nk = N;
  fa_status st = check_sizes(B, Hq, Hkv, N, d, scale);
  if (st != FA_OK) return st;
  if (Nk < 1 || check_sizes(B, Hq, Hkv, Nk, d, scale) != FA_OK) return FA_ERR_INVALID_ARG;
  // above d = 128 only the three-pass backward, which needs the LSE and D parts alone
  st = bwd_dim(d, lse_d_only && !mask);
  if (st != FA_OK) return st;
  const BwdWorkspace w = bwd_workspace(B, Hq, Hkv, N, d);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
      workspace_bytes < (mask ? w.total_sparse : (lse_d_only ? w.off_dq : w.total)))
    return FA_ERR_WORKSPACE;
  unsigned* status = nullptr;
  unsigned long long* clock_acc = nullptr;
  st = device_state(stream, &status, num_sms, &clock_acc);
  if (st != FA_OK) return st;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p->ws_lse2 = reinterpret_cast<float*>(ws + w.off_lse2);
  p->ws_d = reinterpret_cast<float*>(ws + w.off_d);
  // a workspace sized for the LSE and D parts alone has no dQ accumulator:
  // nothing may write past its end
  p->ws_dq = lse_d_only ? nullptr : reinterpret_cast<float*>(ws + w.off_dq);
  p->status = status;
  p->clock_acc = clock_acc;
  p->N = N;
  p->NQP = ((N + 127) / 128) * 128;
  p->Nk = Nk;
  p->NKP = ((Nk + 127) / 128) * 128;
  p->causal_off = Nk - N;
  p->Hq = Hq;
  p->Hkv = Hkv;
  p->BH = B * Hq;
  p->BHkv = B * Hkv;
  p->causal = causal ? 1 : 0;
  p->scale = scale;
  p->scale_log2 = scale * 1.4426950408889634f;
  p->timeout_ns = wait_limit_ns();
  p->test_stall = test_stall();
  p->mask = mask;
  p->mask_sb = mask_sb;
  p->mask_sh = mask_sh;
  p->mask_nt = (N + 127) / 128;
  p->ws_count = mask ? reinterpret_cast<int*>(ws + w.off_count) : nullptr;
  p->ws_list = mask ? reinterpret_cast<unsigned*>(ws + w.off_list) : nullptr;
  return FA_OK;
}

}  // namespace

extern "C" {

size_t fa_bwd_workspace_bytes(int B, int Hq, int Hkv, int N, int d) {
  if (check_sizes(B, Hq, Hkv, N, d, 1.0f) != FA_OK) return 0;
  const BwdWorkspace w = bwd_workspace(B, Hq, Hkv, N, d);
  return d > 128 ? w.off_dq : w.total;      // the three-pass backward keeps no dQ accumulator
}

size_t fa_bwd_blocksparse_workspace_bytes(int B, int Hq, int Hkv, int N, int d) {
  if (check_sizes(B, Hq, Hkv, N, d, 1.0f) != FA_OK || bwd_dim(d) != FA_OK || (N + 127) / 128 > fa::kMaskMaxTiles)
    return 0;
  return bwd_workspace(B, Hq, Hkv, N, d).total_sparse;
}

fa_status fa_bwd_blocksparse(const void* q, const void* k, const void* v, const void* o, const float* lse,
                             const void* dO, void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes,
                             const unsigned char* block_mask, long long mask_stride_b, long long mask_stride_h,
                             int B, int Hq, int Hkv, int N, int d, int causal, float scale, void* stream) {
  const void* ptrs[] = {q, k, v, o, lse, dO, dq, dk, dv};
  for (const void* ptr : ptrs)
    if (!ptr || !aligned16(ptr)) return FA_ERR_INVALID_ARG;
  if (!block_mask || mask_stride_b < 0 || mask_stride_h < 0) return FA_ERR_INVALID_ARG;
  if ((N + 127) / 128 > fa::kMaskMaxTiles) return FA_ERR_UNSUPPORTED;
  fa::BwdParams p{};
  int num_sms = 0;
  fa_status st = bwd_setup(B, Hq, Hkv, N, d, causal, scale, workspace, workspace_bytes, &p, &num_sms, stream, false,
                           block_mask, mask_stride_b, mask_stride_h);
  if (st != FA_OK) return st;
  fa::BwdMaps m;
  const long long BHq = static_cast<long long>(B) * Hq, BHkv = static_cast<long long>(B) * Hkv;
  if (!make_map(&m.q, q, 2, d, N, BHq) || !make_map(&m.k, k, 2, d, N, BHkv) || !make_map(&m.v, v, 2, d, N, BHkv) ||
      !make_map(&m.dO, dO, 2, d, N, BHq) || !make_map(&m.dk, dk, 2, d, N, BHkv) || !make_map(&m.dv, dv, 2, d, N, BHkv) ||
      !make_map(&m.dqacc, p.ws_dq, 4, d, N, BHq))
    return FA_ERR_CUDA;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = fa::launch_bwd_pre(d, o, dO, lse, p, num_sms, s);
  if (e == cudaSuccess) e = fa::launch_bwd_blocklist(p, s);
  if (e == cudaSuccess) e = fa::launch_bwd_dkdv(d, m, p, s);
  if (e == cudaSuccess) e = fa::launch_bwd_dq(d, dq, p, num_sms, s);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_bwd_preprocess(const void* o, const float* lse, const void* dO, void* workspace,
                            size_t workspace_bytes, int B, int Hq, int Hkv, int N, int d, void* stream) {
  if (!o || !lse || !dO || !aligned16(o) || !aligned16(lse) || !aligned16(dO)) return FA_ERR_INVALID_ARG;
  fa::BwdParams p{};
  int num_sms = 0;
  fa_status st = bwd_setup(B, Hq, Hkv, N, d, 0, 1.0f, workspace, workspace_bytes, &p, &num_sms, stream);
  if (st != FA_OK) return st;
  const cudaError_t e = fa::launch_bwd_pre(d, o, dO, lse, p, num_sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"

namespace {
fa_status bwd_dkdv_common(const void* q, const void* k, const void* v, const void* dO, void* dk, void* dv,
                          void* workspace, size_t workspace_bytes, int B, int Hq, int Hkv, int N, int Nk, int d,
                          int causal, float scale, void* stream) {
  const void* ptrs[] = {q, k, v, dO, dk, dv};
  for (const void* ptr : ptrs)
    if (!ptr || !aligned16(ptr)) return FA_ERR_INVALID_ARG;
  fa::BwdParams p{};
  int num_sms = 0;
  fa_status st = bwd_setup(B, Hq, Hkv, N, d, causal, scale, workspace, workspace_bytes, &p, &num_sms, stream, false,
                           nullptr, 0, 0, Nk);
  if (st != FA_OK) return st;
  fa::BwdMaps m;
  const long long BHq = static_cast<long long>(B) * Hq, BHkv = static_cast<long long>(B) * Hkv;
  if (!make_map(&m.q, q, 2, d, N, BHq) || !make_map(&m.k, k, 2, d, Nk, BHkv) ||
      !make_map(&m.v, v, 2, d, Nk, BHkv) || !make_map(&m.dO, dO, 2, d, N, BHq) ||
      !make_map(&m.dk, dk, 2, d, Nk, BHkv) || !make_map(&m.dv, dv, 2, d, Nk, BHkv) ||
      !make_map(&m.dqacc, p.ws_dq, 4, d, N, BHq))
    return FA_ERR_CUDA;
  const cudaError_t e = fa::launch_bwd_dkdv(d, m, p, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}
}  // namespace

namespace {
// Head dims 136..256: the three passes of fa_bwd_wide.cu after the
// preprocess (no dQ accumulator in the workspace).
fa_status bwd_wide(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO,
                   void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes, int B, int Hq, int Hkv,
                   int N, int Nk, int d, int causal, float scale, void* stream) {
  const void* ptrs[] = {q, k, v, o, lse, dO, dq, dk, dv};
  for (const void* ptr : ptrs)
    if (!ptr || !aligned16(ptr)) return FA_ERR_INVALID_ARG;
  fa::BwdParams p{};
  int num_sms = 0;
  fa_status st = bwd_setup(B, Hq, Hkv, N, d, causal, scale, workspace, workspace_bytes, &p, &num_sms, stream, true,
                           nullptr, 0, 0, Nk);
  if (st != FA_OK) return st;
  fa::BwdMaps m, m64;
  const long long BHq = static_cast<long long>(B) * Hq, BHkv = static_cast<long long>(B) * Hkv;
  if (!make_map(&m.q, q, 2, d, N, BHq) || !make_map(&m.k, k, 2, d, Nk, BHkv) || !make_map(&m.v, v, 2, d, Nk, BHkv) ||
      !make_map(&m.dO, dO, 2, d, N, BHq) || !make_map(&m.dk, dk, 2, d, Nk, BHkv) ||
      !make_map(&m.dv, dv, 2, d, Nk, BHkv) || !make_map(&m.dq, dq, 2, d, N, BHq) ||
      !make_map(&m64.q, q, 2, d, N, BHq, 64) || !make_map(&m64.dO, dO, 2, d, N, BHq, 64) ||
      !make_map(&m64.k, k, 2, d, Nk, BHkv, 64) || !make_map(&m64.v, v, 2, d, Nk, BHkv, 64))
    return FA_ERR_CUDA;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = fa::launch_bwd_pre(d, o, dO, lse, p, num_sms, s);
  if (e == cudaSuccess) e = fa::launch_bwd_wide(m, m64, p, s);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}
}  // namespace

extern "C" {

fa_status fa_bwd_dkdv(const void* q, const void* k, const void* v, const void* dO, void* dk, void* dv,
                      void* workspace, size_t workspace_bytes, int B, int Hq, int Hkv, int N, int d, int causal,
                      float scale, void* stream) {
  return bwd_dkdv_common(q, k, v, dO, dk, dv, workspace, workspace_bytes, B, Hq, Hkv, N, N, d, causal, scale,
                         stream);
}

fa_status fa_bwd_dq(void* dq, void* workspace, size_t workspace_bytes, int B, int Hq, int Hkv, int N, int d,
                    float scale, void* stream) {
  if (!dq || !aligned16(dq)) return FA_ERR_INVALID_ARG;
  fa::BwdParams p{};
  int num_sms = 0;
  fa_status st = bwd_setup(B, Hq, Hkv, N, d, 0, scale, workspace, workspace_bytes, &p, &num_sms, stream);
  if (st != FA_OK) return st;
  const cudaError_t e = fa::launch_bwd_dq(d, dq, p, num_sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO,
                 void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes, int B, int Hq, int Hkv,
                 int N, int d, int causal, float scale, void* stream) {
  if (d > 128)
    return bwd_wide(q, k, v, o, lse, dO, dq, dk, dv, workspace, workspace_bytes, B, Hq, Hkv, N, N, d, causal, scale,
                    stream);
  const void* ptrs[] = {q, k, v, o, lse, dO, dq, dk, dv};
  for (const void* ptr : ptrs)
    if (!ptr || !aligned16(ptr)) return FA_ERR_INVALID_ARG;
  fa_status st = fa_bwd_preprocess(o, lse, dO, workspace, workspace_bytes, B, Hq, Hkv, N, d, stream);
  if (st != FA_OK) return st;
  st = fa_bwd_dkdv(q, k, v, dO, dk, dv, workspace, workspace_bytes, B, Hq, Hkv, N, d, causal, scale, stream);
  if (st != FA_OK) return st;
  return fa_bwd_dq(dq, workspace, workspace_bytes, B, Hq, Hkv, N, d, scale, stream);
}

fa_status fa_bwd_kv(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO,
                    void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes, int B, int Hq, int Hkv,
                    int Nq, int Nk, int d, int causal, float scale, void* stream) {
  if (Nk < 1) return FA_ERR_INVALID_ARG;
  if (d > 128)
    return bwd_wide(q, k, v, o, lse, dO, dq, dk, dv, workspace, workspace_bytes, B, Hq, Hkv, Nq, Nk, d, causal,
                    scale, stream);
  const void* ptrs[] = {q, k, v, o, lse, dO, dq, dk, dv};
  for (const void* ptr : ptrs)
    if (!ptr || !aligned16(ptr)) return FA_ERR_INVALID_ARG;
  fa_status st = fa_bwd_preprocess(o, lse, dO, workspace, workspace_bytes, B, Hq, Hkv, Nq, d, stream);
  if (st != FA_OK) return st;
  st = bwd_dkdv_common(q, k, v, dO, dk, dv, workspace, workspace_bytes, B, Hq, Hkv, Nq, Nk, d, causal, scale, stream);
  if (st != FA_OK) return st;
  return fa_bwd_dq(dq, workspace, workspace_bytes, B, Hq, Hkv, Nq, d, scale, stream);
}

fa_status fa_bwd_deterministic(const void* q, const void* k, const void* v, const void* o, const float* lse,
                               const void* dO, void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes,
                               int B, int Hq, int Hkv, int N, int d, int causal, float scale, void* stream) {
  if (d > 128)       // the three-pass backward is bit reproducible too
    return bwd_wide(q, k, v, o, lse, dO, dq, dk, dv, workspace, workspace_bytes, B, Hq, Hkv, N, N, d, causal, scale,
                    stream);
  const void* ptrs[] = {q, k, v, o, lse, dO, dq, dk, dv};
  for (const void* ptr : ptrs)
    if (!ptr || !aligned16(ptr)) return FA_ERR_INVALID_ARG;
  fa::BwdParams p{};
  int num_sms = 0;
  fa_status st = bwd_setup(B, Hq, Hkv, N, d, causal, scale, workspace, workspace_bytes, &p, &num_sms, stream, true);
  if (st != FA_OK) return st;
  fa::BwdMaps m;
  const long long BHq = static_cast<long long>(B) * Hq, BHkv = static_cast<long long>(B) * Hkv;
  if (!make_map(&m.q, q, 2, d, N, BHq) || !make_map(&m.k, k, 2, d, N, BHkv) || !make_map(&m.v, v, 2, d, N, BHkv) ||
      !make_map(&m.dO, dO, 2, d, N, BHq) || !make_map(&m.dk, dk, 2, d, N, BHkv) || !make_map(&m.dv, dv, 2, d, N, BHkv) ||
      !make_map(&m.dq, dq, 2, d, N, BHq))
    return FA_ERR_CUDA;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = fa::launch_bwd_pre(d, o, dO, lse, p, num_sms, s);
  if (e == cudaSuccess) e = fa::launch_bwd_deterministic(d, m, p, s);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq, int Hkv, int N,
                 int d, int causal, float scale, void* stream) {
  return fwd_common(2, q, k, v, o, lse, B, Hq, Hkv, N, d, causal, scale, stream);
}

fa_status fa_fwd_kv(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq, int Hkv, int Nq,
                    int Nk, int d, int causal, float scale, void* stream) {
  if (Nk < 1) return FA_ERR_INVALID_ARG;
  return fwd_common(2, q, k, v, o, lse, B, Hq, Hkv, Nq, d, causal, scale, stream, nullptr, 0, 0, Nk);
}

fa_status fa_fwd_packed(const void* q, long long q_stride_h, long long q_stride_t, const void* k, long long k_stride_h,
                        long long k_stride_t, const void* v, long long v_stride_h, long long v_stride_t, void* o,
                        long long o_stride_h, long long o_stride_t, float* lse, const int* cu_seqlens, int S, int T,
                        int Hq, int Hkv, int d, int causal, float scale, void* stream) {
  if (!q || !k || !v || !o || !lse || !cu_seqlens) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse)) return FA_ERR_INVALID_ARG;
  fa_status st = check_sizes(1, Hq, Hkv, T, d, scale);
  if (st != FA_OK) return st;
  if (S < 1) return FA_ERR_INVALID_ARG;
  // rows and heads apart (no broadcast), 16-byte rows, within a tensor map's strides
  const long long strides[] = {q_stride_h, q_stride_t, k_stride_h, k_stride_t,
                               v_stride_h, v_stride_t, o_stride_h, o_stride_t};
  for (long long s : strides)
    if (s < d || s % 8 != 0 || s >= (1LL << 39)) return FA_ERR_INVALID_ARG;
  // (past 2^24 sequences the look for an item could outlast the waits for it)
  if (d > 128 || S > (1 << 24)) return FA_ERR_UNSUPPORTED;
  unsigned* status = nullptr;
  unsigned long long* clock_acc = nullptr;
  int num_sms = 0;
  st = device_state(stream, &status, &num_sms, &clock_acc);
  if (st != FA_OK) return st;
  CUtensorMap mq, mk, mv, mo;
  if (!make_map_strided(&mq, q, 2, d, T, Hq, q_stride_t, q_stride_h, 128) ||
      !make_map_strided(&mk, k, 2, d, T, Hkv, k_stride_t, k_stride_h, 128) ||
      !make_map_strided(&mv, v, 2, d, T, Hkv, v_stride_t, v_stride_h, 128) ||
      !make_map_strided(&mo, o, 2, d, T, Hq, o_stride_t, o_stride_h, 32))
    return FA_ERR_CUDA;
  fa::FwdParams p{};
  p.lse = lse;
  p.status = status;
  p.clock_acc = clock_acc;
  p.N = p.Nk = p.T = T;
  p.S = S;
  p.cu = cu_seqlens;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.o_sh = o_stride_h;
  p.o_st = o_stride_t;
  p.head_dim = d;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.causal = causal ? 1 : 0;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.timeout_ns = wait_limit_ns();
  p.test_stall = test_stall();
  return fa::launch_fwd_packed(d, mq, mk, mv, mo, p, num_sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_fwd_pair(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq, int Hkv,
                      int Nq, int Nk, int d, int causal, float scale, void* stream) {
  if (Nk < 1) return FA_ERR_INVALID_ARG;
  return fwd_common(2, q, k, v, o, lse, B, Hq, Hkv, Nq, d, causal, scale, stream, nullptr, 0, 0, Nk, true);
}

fa_status fa_fwd_blocksparse(const void* q, const void* k, const void* v, void* o, float* lse,
                             const unsigned char* block_mask, long long mask_stride_b, long long mask_stride_h, int B,
                             int Hq, int Hkv, int N, int d, int causal, float scale, void* stream) {
  if (!block_mask || mask_stride_b < 0 || mask_stride_h < 0) return FA_ERR_INVALID_ARG;
  if ((N + 127) / 128 > fa::kMaskMaxTiles) return FA_ERR_UNSUPPORTED;
  return fwd_common(2, q, k, v, o, lse, B, Hq, Hkv, N, d, causal, scale, stream, block_mask, mask_stride_b,
                    mask_stride_h);
}

fa_status fa_fwd_f32(const float* q, const float* k, const float* v, float* o, float* lse, int B, int Hq, int Hkv,
                     int N, int d, int causal, float scale, void* stream) {
  return fwd_common(4, q, k, v, o, lse, B, Hq, Hkv, N, d, causal, scale, stream);
}

size_t fa_fp8_row_scales(int N) { return N >= 1 ? static_cast<size_t>((N + 63) / 64) : 0; }

size_t fa_fp8_vt_keys(int N) { return N >= 1 ? static_cast<size_t>((N + 127) / 128 * 128) : 0; }

fa_status fa_fp8_quantize_rows(const void* x, void* out, float* scales, int BH, int N, int d, void* stream) {
  if (!x || !out || !scales || !aligned16(x) || !aligned16(out) || !aligned16(scales)) return FA_ERR_INVALID_ARG;
  if (BH < 1 || N < 1 || d < 1) return FA_ERR_INVALID_ARG;
  if (!fp8_dim(d)) return FA_ERR_UNSUPPORTED;
  unsigned* status = nullptr;
  const fa_status st = device_state(stream, &status);
  if (st != FA_OK) return st;
  return fa::launch_fp8_quant_rows(x, out, scales, BH, N, d, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_fp8_quantize_v(const void* v, void* vt, float* scales, int BH, int N, int d, void* stream) {
  if (!v || !vt || !scales || !aligned16(v) || !aligned16(vt) || !aligned16(scales)) return FA_ERR_INVALID_ARG;
  if (BH < 1 || N < 1 || d < 1) return FA_ERR_INVALID_ARG;
  if (!fp8_dim(d)) return FA_ERR_UNSUPPORTED;
  unsigned* status = nullptr;
  const fa_status st = device_state(stream, &status);
  if (st != FA_OK) return st;
  return fa::launch_fp8_quant_v(v, vt, scales, BH, N, d, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"

namespace {
fa_status fwd_fp8_common(const void* q, const float* q_scale, const void* k, const float* k_scale, const void* vt,
                         const float* v_scale, void* o, float* lse, int B, int Hq, int Hkv, int N, int Nk, int d,
                         int causal, float scale, void* stream) {
  const void* ptrs[] = {q, q_scale, k, k_scale, vt, v_scale, o, lse};
  for (const void* ptr : ptrs)
    if (!ptr || !aligned16(ptr)) return FA_ERR_INVALID_ARG;
  fa_status st = check_sizes(B, Hq, Hkv, N, d, scale);
  if (st != FA_OK) return st;
  if (Nk < 1 || check_sizes(B, Hq, Hkv, Nk, d, scale) != FA_OK) return FA_ERR_INVALID_ARG;
  if (!fp8_dim(d)) return FA_ERR_UNSUPPORTED;
  unsigned* status = nullptr;
  st = device_state(stream, &status);
  if (st != FA_OK) return st;
  CUtensorMap mq, mk, mvt, mo;
  const long long BHq = static_cast<long long>(B) * Hq, BHkv = static_cast<long long>(B) * Hkv;
  const int NP = (Nk + 127) / 128 * 128;
  if (!make_map(&mq, q, 1, d, N, BHq) || !make_map(&mk, k, 1, d, Nk, BHkv) ||
      !make_map(&mvt, vt, 1, NP, d, BHkv) || !make_map(&mo, o, 2, d, N, BHq))
    return FA_ERR_CUDA;
  fa::FwdParams p{};
  p.lse = lse;
  p.status = status;
  p.N = N;
  p.Nk = Nk;
  p.causal_off = Nk - N;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.BH = static_cast<int>(BHq);
  p.causal = causal ? 1 : 0;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.timeout_ns = wait_limit_ns();
  p.test_stall = test_stall();
  p.head_dim = d;
  p.q_scale = q_scale;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = d <= 128 ? fa::launch_fwd_fp8(mq, mk, mvt, mo, p, s) : fa::launch_fwd_fp8_wide(mq, mk, mvt, mo, p, s);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}
}  // namespace

extern "C" {

fa_status fa_fwd_fp8(const void* q, const float* q_scale, const void* k, const float* k_scale, const void* vt,
                     const float* v_scale, void* o, float* lse, int B, int Hq, int Hkv, int N, int d, int causal,
                     float scale, void* stream) {
  return fwd_fp8_common(q, q_scale, k, k_scale, vt, v_scale, o, lse, B, Hq, Hkv, N, N, d, causal, scale, stream);
}

fa_status fa_fwd_fp8_kv(const void* q, const float* q_scale, const void* k, const float* k_scale, const void* vt,
                        const float* v_scale, void* o, float* lse, int B, int Hq, int Hkv, int Nq, int Nk, int d,
                        int causal, float scale, void* stream) {
  return fwd_fp8_common(q, q_scale, k, k_scale, vt, v_scale, o, lse, B, Hq, Hkv, Nq, Nk, d, causal, scale, stream);
}

}  // extern "C"

namespace {
// The cache's own rules, and its arrays as the kernels take them.
fa_status cache8_pools(const fa_cache8* c, int B, int max_blocks, const void* block_table, bool need_weight,
                       fa::Cache8Pools* out) {
  if (!c || !block_table) return FA_ERR_INVALID_ARG;
  const void* ptrs[] = {c->k, c->v, c->k_scale, c->v_scale};
  for (const void* ptr : ptrs)
    if (!ptr || !aligned16(ptr)) return FA_ERR_INVALID_ARG;
  if (!aligned16(c->weight) || (need_weight && !c->weight)) return FA_ERR_INVALID_ARG;
  if (c->num_blocks < 1 || c->Hkv < 1 || c->Hkv > 65535 || c->d < 1 || B < 1 || B > 65535 || max_blocks < 1 ||
      max_blocks > (1 << 24))
    return FA_ERR_INVALID_ARG;
  if (!fp8_dim(c->d) || static_cast<long long>(c->num_blocks) * c->Hkv >= (1LL << 31)) return FA_ERR_UNSUPPORTED;
  *out = fa::Cache8Pools{c->k, c->v, c->k_scale, c->v_scale, c->weight, c->num_blocks, c->Hkv, c->d};
  return FA_OK;
}

// Bytes of fa_fwd_cache8's workspace: partial results, their statistics (off_s)
// and, with weights, the scores of every token and row (off_x).
constexpr size_t kNoWorkspace = 256;   // what is said where none is needed (0 says that the call refuses; all others are larger)
struct Cache8Workspace {
  size_t off_s, off_x, total;
  int score_row;                       // floats per token in the scores
};
Cache8Workspace cache8_workspace(int B, int Hkv, int R, int d, int max_blocks, bool weights) {
  const int cols = fa::cache8_columns(R), chunks = (R + cols - 1) / cols;
  const size_t D = d <= 128 ? 128 : 256;
  const size_t rows = fa::cache8_whole(B, Hkv, d, R, max_blocks)
                          ? 0
                          : 2 * static_cast<size_t>(fa::cache8_parts(B, Hkv, d, R, max_blocks)) * cols;
  const size_t units = static_cast<size_t>(B) * Hkv * chunks * max_blocks;
  Cache8Workspace w;
  w.off_s = align256(rows * D * 4);
  w.off_x = w.off_s + align256(rows * 3 * 4);
  w.score_row = R < cols ? (R + 3) / 4 * 4 : cols;
  w.total = w.off_x + (weights ? units * FA_CACHE8_BLOCK * w.score_row * 4 : 0);
  if (w.total == 0) w.total = kNoWorkspace;
  return w;
}

fa_status cache8_rows(int B, int Hq, int Hkv, int Nq, int d, int max_blocks) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Nq < 1 || Hq % Hkv != 0 || d < 1 || max_blocks < 1) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(Hq / Hkv) * Nq > fa::kCache8MaxRows || !fp8_dim(d)) return FA_ERR_UNSUPPORTED;
  // units of work (row groups x blocks) are counted in 32 bits
  const int R = Hq / Hkv * Nq, cols = fa::cache8_columns(R), chunks = (R + cols - 1) / cols;
  if (static_cast<double>(B) * Hkv * chunks * max_blocks >= 2147483648.0 ||
      static_cast<double>(B) * Hq * Nq >= 2147483648.0)
    return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// Bytes of fa_fwd_cache8_packed's workspace: two partial results per CTA, their statistics (off_s) and what is to be
// joined (off_j).
struct ChunkWorkspace {
  size_t off_s, off_j, total;
};
ChunkWorkspace chunk_workspace(int d, int max_blocks) {
  if (max_blocks <= 2) return {0, 0, kNoWorkspace};    // one key tile: nothing is split
  const size_t D = d <= 128 ? 128 : 256, rows = 2 * static_cast<size_t>(fa::kCache8Sms) * fa::chunk_rows(d);
  const size_t off_s = align256(rows * D * 4), off_j = off_s + align256(rows * 3 * 4);
  return {off_s, off_j, off_j + align256(fa::kCache8Sms * 8 * 4)};
}
// scale log2(e) = digits power, digits from 1 to 2.
void split_scale(float scale, float* digits, float* power) {
  int e = 0;
  *digits = 2.f * std::frexp(scale * 1.4426950408889634f, &e);
  *power = std::ldexp(1.f, e - 1);
}
fa_status chunk_sizes(int B, int T, int Hq, int Hkv, int d, int max_blocks) {
  if (B < 1 || B > 65535 || T < 1 || Hq < 1 || Hkv < 1 || Hkv > 65535 || Hq % Hkv != 0 || d < 1 || max_blocks < 1 ||
      max_blocks > (1 << 24))
    return FA_ERR_INVALID_ARG;
  if (!fp8_dim(d) || Hq / Hkv > 128 || T > (1 << 30)) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}
// A rotation's table for heads of d columns; its positions are the caller's to set.
fa_status rope_plan(const fa_rope_plan* r, int d, fa::RopePlan* out) {
  if (!r || !r->turns || r->axes < 1 || r->pairs < 1 || 2LL * r->pairs > d) return FA_ERR_INVALID_ARG;
  if (r->pairs % 4 != 0) return FA_ERR_UNSUPPORTED;
  *out = fa::RopePlan{};
  out->turns = r->turns;
  out->axis = r->axis;
  out->pairs = r->pairs;
  out->axes = r->axes;
  out->interleaved = r->interleaved ? 1 : 0;
  return FA_OK;
}

fa_status append_common(const void* k, long long k_stride_h, long long k_stride_t, const void* v, long long v_stride_h,
                        long long v_stride_t, const int* cu_seqlens, const int* start, int B, int T,
                        const fa_cache8* cache, const int* block_table, int max_blocks, const fa::RopePlan& rope,
                        void* stream) {
  if (!k || !v || !cu_seqlens || !start || !aligned16(k) || !aligned16(v)) return FA_ERR_INVALID_ARG;
  const long long strides[] = {k_stride_h, k_stride_t, v_stride_h, v_stride_t};
  for (long long s : strides)
    if (s < 0 || s % 8 != 0) return FA_ERR_INVALID_ARG;
  if (T < 1) return FA_ERR_INVALID_ARG;
  fa::Cache8AppendParams p{};
  fa_status st = cache8_pools(cache, B, max_blocks, block_table, false, &p.c);
  if (st != FA_OK) return st;
  unsigned* status = nullptr;
  st = device_state(stream, &status);
  if (st != FA_OK) return st;
  p.k = k;
  p.v = v;
  p.k_sh = k_stride_h;
  p.k_st = k_stride_t;
  p.v_sh = v_stride_h;
  p.v_st = v_stride_t;
  p.cu = cu_seqlens;
  p.start = start;
  p.table = block_table;
  p.B = B;
  p.T = T;
  p.max_blocks = max_blocks;
  p.rope = rope;
  return fa::launch_cache8_append(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}
}  // namespace

extern "C" {

fa_status fa_cache8_append(const void* k, long long k_stride_h, long long k_stride_t, const void* v,
                           long long v_stride_h, long long v_stride_t, const int* cu_seqlens, const int* start, int B,
                           int T, const fa_cache8* cache, const int* block_table, int max_blocks, void* stream) {
  return append_common(k, k_stride_h, k_stride_t, v, v_stride_h, v_stride_t, cu_seqlens, start, B, T, cache, block_table,
                       max_blocks, fa::RopePlan{}, stream);
}

fa_status fa_cache8_append_rope(const void* k, long long k_stride_h, long long k_stride_t, const void* v,
                                long long v_stride_h, long long v_stride_t, const int* cu_seqlens, const int* start, int B,
                                int T, const fa_cache8* cache, const int* block_table, int max_blocks,
                                const fa_rope_plan* rope, const int* positions, long long pos_stride_axis, void* stream) {
  if (!cache) return FA_ERR_INVALID_ARG;
  fa::RopePlan plan{};
  const fa_status st = rope_plan(rope, cache->d, &plan);
  if (st != FA_OK) return st;
  if (pos_stride_axis < 0) return FA_ERR_INVALID_ARG;
  plan.positions = positions;
  plan.pos_sa = pos_stride_axis;
  return append_common(k, k_stride_h, k_stride_t, v, v_stride_h, v_stride_t, cu_seqlens, start, B, T, cache, block_table,
                       max_blocks, plan, stream);
}

fa_status fa_rope(const void* q, long long q_stride_b, long long q_stride_h, long long q_stride_t, void* q_out,
                  long long q_out_stride_b, long long q_out_stride_h, long long q_out_stride_t, int Hq, const void* k,
                  long long k_stride_b, long long k_stride_h, long long k_stride_t, void* k_out,
                  long long k_out_stride_b, long long k_out_stride_h, long long k_out_stride_t, int Hkv, int B, int T,
                  int d, int elt_bytes, const fa_rope_plan* rope, const int* positions, long long pos_stride_axis,
                  long long pos_stride_b, int inverse, void* stream) {
  if (B < 1 || T < 1 || d < 8 || d > 256 || d % 8 != 0 || (elt_bytes != 2 && elt_bytes != 4) || !positions ||
      pos_stride_axis < 0 || pos_stride_b < 0)
    return FA_ERR_INVALID_ARG;
  fa::RopeParams p{};
  const fa_status st = rope_plan(rope, d, &p.rope);
  if (st != FA_OK) return st;
  p.x[0] = {q, q_out, q_stride_b, q_stride_h, q_stride_t, q_out_stride_b, q_out_stride_h, q_out_stride_t, Hq};
  p.x[1] = {k, k_out, k_stride_b, k_stride_h, k_stride_t, k_out_stride_b, k_out_stride_h, k_out_stride_t, Hkv};
  for (int i = 0; i < 2; ++i) {
    const fa::RopeTensor& x = p.x[i];
    if (i == 1 && x.H == 0) continue;                  // no K
    if (!x.in || !x.out || !aligned16(x.in) || !aligned16(x.out) || x.H < 1) return FA_ERR_INVALID_ARG;
    const long long strides[] = {x.in_sb, x.in_sh, x.in_st, x.out_sb, x.out_sh, x.out_st};
    for (long long s : strides)
      if (s < 0 || s % (16 / elt_bytes) != 0) return FA_ERR_INVALID_ARG;
    // no broadcast output: rows would be written by several threads
    if ((B > 1 && x.out_sb < d) || (x.H > 1 && x.out_sh < d) || (T > 1 && x.out_st < d)) return FA_ERR_INVALID_ARG;
  }
  if (static_cast<long long>(B) * T >= (1LL << 31) || static_cast<long long>(Hq) + Hkv > 65535) return FA_ERR_UNSUPPORTED;
  // An output where an input begins is that tensor's own, row for row: threads that read other rows than they write
  // would race.
  for (int i = 0; i < 2; ++i) {
    const fa::RopeTensor& x = p.x[i];
    if (x.H == 0) continue;
    if (i == 1 && x.out == p.x[0].out) return FA_ERR_INVALID_ARG;
    if (p.x[1 - i].H > 0 && x.out == p.x[1 - i].in) return FA_ERR_INVALID_ARG;
    if (x.out == x.in &&
        ((B > 1 && x.out_sb != x.in_sb) || (x.H > 1 && x.out_sh != x.in_sh) || (T > 1 && x.out_st != x.in_st)))
      return FA_ERR_INVALID_ARG;
  }
  unsigned* status = nullptr;
  const fa_status dev = device_state(stream, &status);
  if (dev != FA_OK) return dev;
  p.rope.positions = positions;
  p.rope.pos_sa = pos_stride_axis;
  p.rope.pos_sb = pos_stride_b;
  p.B = B;
  p.T = T;
  p.d = d;
  p.inverse = inverse ? 1 : 0;
  return fa::launch_rope(elt_bytes, p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t fa_fwd_cache8_workspace_bytes(int B, int Hq, int Hkv, int Nq, int d, int max_blocks, int add_weights) {
  if (cache8_rows(B, Hq, Hkv, Nq, d, max_blocks) != FA_OK) return 0;
  return cache8_workspace(B, Hkv, Hq / Hkv * Nq, d, max_blocks, add_weights != 0).total;
}

fa_status fa_fwd_cache8(const void* q, const fa_cache8* cache, const int* block_table, int max_blocks,
                        const int* lengths, void* o, float* lse, void* workspace, size_t workspace_bytes, int B, int Hq,
                        int Nq, int causal, float scale, int add_weights, float weight_decay, void* stream) {
  if (!q || !o || q == o || !lse || !lengths || !aligned16(q) || !aligned16(o) || !aligned16(lse)) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_INVALID_ARG;
  if (add_weights && (!std::isfinite(weight_decay) || !(weight_decay >= 0.f))) return FA_ERR_INVALID_ARG;
  fa::Cache8Params p{};
  fa_status st = cache8_pools(cache, B, max_blocks, block_table, add_weights != 0, &p.c);
  if (st == FA_OK) st = cache8_rows(B, Hq, p.c.Hkv, Nq, p.c.d, max_blocks);
  if (st != FA_OK) return st;
  p.G = Hq / p.c.Hkv;
  p.R = p.G * Nq;
  const int cols = fa::cache8_columns(p.R);
  p.chunks = (p.R + cols - 1) / cols;
  const Cache8Workspace w = cache8_workspace(B, p.c.Hkv, p.R, p.c.d, max_blocks, add_weights != 0);
  if (w.total > kNoWorkspace &&
      (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || workspace_bytes < w.total))
    return FA_ERR_WORKSPACE;
  unsigned* status = nullptr;
  st = device_state(stream, &status);
  if (st != FA_OK) return st;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.table = block_table;
  p.lengths = lengths;
  p.B = B;
  p.max_blocks = max_blocks;
  p.Hq = Hq;
  p.Nq = Nq;
  p.causal = causal ? 1 : 0;
  p.add_weights = add_weights ? 1 : 0;
  split_scale(scale, &p.scale_digits, &p.scale_power);
  p.decay = weight_decay;
  p.part_o = static_cast<float*>(workspace);
  p.part_s = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + w.off_s);
  p.scores = add_weights ? reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + w.off_x) : nullptr;
  p.score_row = w.score_row;
  p.status = status;
  p.timeout_ns = wait_limit_ns();
  p.test_stall = test_stall();
  CUtensorMap mk, mv;
  const long long rows = static_cast<long long>(p.c.num_blocks) * p.c.Hkv;
  if (!make_map(&mk, p.c.k, 1, p.c.d, FA_CACHE8_BLOCK, rows, 64) || !make_map(&mv, p.c.v, 1, p.c.d, FA_CACHE8_BLOCK, rows, 64))
    return FA_ERR_CUDA;
  return fa::launch_cache8_fwd(mk, mv, p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t fa_fwd_cache8_packed_workspace_bytes(int B, int T, int Hq, int Hkv, int d, int max_blocks) {
  if (chunk_sizes(B, T, Hq, Hkv, d, max_blocks) != FA_OK) return 0;
  return chunk_workspace(d, max_blocks).total;
}

fa_status fa_fwd_cache8_packed(const void* q, long long q_stride_h, long long q_stride_t, const fa_cache8* cache,
                               const int* block_table, int max_blocks, const int* cu_seqlens, const int* lengths, void* o,
                               long long o_stride_h, long long o_stride_t, float* lse, void* workspace,
                               size_t workspace_bytes, int B, int T, int Hq, int causal, float scale, void* stream) {
  if (!q || !o || q == o || !lse || !cu_seqlens || !lengths || !aligned16(q) || !aligned16(o) || !aligned16(lse))
    return FA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_INVALID_ARG;
  fa::ChunkParams p{};
  fa_status st = cache8_pools(cache, B, max_blocks, block_table, false, &p.c);
  if (st == FA_OK) st = chunk_sizes(B, T, Hq, p.c.Hkv, p.c.d, max_blocks);
  if (st != FA_OK) return st;
  const long long strides[] = {q_stride_h, q_stride_t, o_stride_h, o_stride_t};
  for (long long s : strides)
    if (s < p.c.d || s % 8 != 0) return FA_ERR_INVALID_ARG;
  const ChunkWorkspace w = chunk_workspace(p.c.d, max_blocks);
  if (w.total > kNoWorkspace &&
      (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || workspace_bytes < w.total))
    return FA_ERR_WORKSPACE;
  unsigned* status = nullptr;
  int num_sms = 0;
  st = device_state(stream, &status, &num_sms);
  if (st != FA_OK) return st;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.q_sh = q_stride_h;
  p.q_st = q_stride_t;
  p.o_sh = o_stride_h;
  p.o_st = o_stride_t;
  p.lse = lse;
  p.cu = cu_seqlens;
  p.lengths = lengths;
  p.table = block_table;
  p.B = B;
  p.T = T;
  p.max_blocks = max_blocks;
  p.G = Hq / p.c.Hkv;
  p.tt = 128 / p.G;
  p.causal = causal ? 1 : 0;
  p.ctas = num_sms < fa::kCache8Sms ? num_sms : fa::kCache8Sms;
  split_scale(scale, &p.scale_digits, &p.scale_power);
  p.status = status;
  p.timeout_ns = wait_limit_ns();
  p.test_stall = test_stall();
  p.part_o = static_cast<float*>(workspace);               // (offsets into nothing where none is needed: never read)
  p.part_s = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + w.off_s);
  p.joins = w.total > kNoWorkspace ? reinterpret_cast<int*>(static_cast<uint8_t*>(workspace) + w.off_j) : nullptr;
  CUtensorMap mk, mv;
  const long long rows = static_cast<long long>(p.c.num_blocks) * p.c.Hkv;
  if (!make_map(&mk, p.c.k, 1, p.c.d, FA_CACHE8_BLOCK, rows, 64) || !make_map(&mv, p.c.v, 1, p.c.d, FA_CACHE8_BLOCK, rows, 64))
    return FA_ERR_CUDA;
  return fa::launch_cache8_chunk(mk, mv, p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_cache8_evict(const fa_cache8* cache, const int* block_table, int max_blocks, const int* lengths, int B,
                          int keep, int recent, const int* to_table, int to_blocks, int* kept, int* new_lengths,
                          void* stream) {
  if (!lengths || !to_table || !kept || !new_lengths || new_lengths == lengths) return FA_ERR_INVALID_ARG;
  if (keep < 1 || recent < 0 || recent > keep || to_blocks < 1 ||
      static_cast<long long>(to_blocks) * FA_CACHE8_BLOCK < keep)
    return FA_ERR_INVALID_ARG;
  fa::Cache8EvictParams p{};
  fa_status st = cache8_pools(cache, B, max_blocks, block_table, true, &p.c);
  if (st != FA_OK) return st;
  // one CTA per destination block that is used
  if (static_cast<long long>(B) * ((keep - 1) / FA_CACHE8_BLOCK + 1) >= (1LL << 31)) return FA_ERR_UNSUPPORTED;
  unsigned* status = nullptr;
  st = device_state(stream, &status);
  if (st != FA_OK) return st;
  p.table = block_table;
  p.lengths = lengths;
  p.to_table = to_table;
  p.kept = kept;
  p.new_lengths = new_lengths;
  p.B = B;
  p.max_blocks = max_blocks;
  p.to_blocks = to_blocks;
  p.keep = keep;
  p.recent = recent;
  return fa::launch_cache8_evict(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_ex2_throughput(double* per_sm_per_cycle, void* stream) {
  if (!per_sm_per_cycle) return FA_ERR_INVALID_ARG;
  unsigned* status = nullptr;
  int num_sms = 0;
  const fa_status st = device_state(stream, &status, &num_sms);
  if (st != FA_OK) return st;
  if (num_sms > fa::kEx2MaxSms) return FA_ERR_UNSUPPORTED;
  return fa::measure_ex2_rate(num_sms, 4096, per_sm_per_cycle, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_device_status(void* stream) {
  unsigned* status = nullptr;
  fa_status st = device_state(stream, &status);
  if (st != FA_OK) return st;
  // read and clear this stream's word in the stream's own order: work on
  // other streams is neither waited for nor reported here
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  unsigned host = 0;
  if (cudaMemcpyAsync(&host, status, sizeof(host), cudaMemcpyDeviceToHost, s) != cudaSuccess) return FA_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return FA_ERR_CUDA;
  if (host != 0) {
    if (cudaMemsetAsync(status, 0, sizeof(unsigned), s) != cudaSuccess) return FA_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return FA_ERR_CUDA;
    return (host & 1u) ? FA_ERR_TIMEOUT : FA_ERR_DEVICE;
  }
  return FA_OK;
}

fa_status fa_sm_clock_mhz(double* mhz, void* stream) {
  if (!mhz) return FA_ERR_INVALID_ARG;
  unsigned* status = nullptr;
  unsigned long long* acc = nullptr;
  const fa_status st = device_state(stream, &status, nullptr, &acc);
  if (st != FA_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaDeviceSynchronize() != cudaSuccess) return FA_ERR_CUDA;
  unsigned long long host[2] = {0, 0};
  if (cudaMemcpyAsync(host, acc, sizeof(host), cudaMemcpyDeviceToHost, s) != cudaSuccess) return FA_ERR_CUDA;
  if (cudaMemsetAsync(acc, 0, sizeof(host), s) != cudaSuccess) return FA_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return FA_ERR_CUDA;
  *mhz = host[1] > 0 ? static_cast<double>(host[0]) * 1e3 / static_cast<double>(host[1]) : 0.0;
  return FA_OK;
}

const char* fa_status_string(fa_status s) {
  switch (s) {
    case FA_OK: return "ok";
    case FA_ERR_INVALID_ARG: return "invalid argument (null or misaligned pointer, or bad size)";
    case FA_ERR_UNSUPPORTED: return "unsupported combination of sizes or types";
    case FA_ERR_ARCH: return "current device is not compute capability 10.3 (sm_103)";
    case FA_ERR_CUDA: return "CUDA error";
    case FA_ERR_TIMEOUT: return "a bounded wait inside a kernel ran out; outputs of that call are invalid";
    case FA_ERR_WORKSPACE: return "workspace too small or misaligned";
    case FA_ERR_DEVICE: return "a kernel refused to run on this device's shared-memory layout; outputs invalid";
  }
  return "unknown status";
}

int fa_version(void) { return 500; }

}  // extern "C"
