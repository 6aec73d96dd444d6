// C-ABI host layer: argument validation, workspace, dispatch and error mapping.
// Nothing here computes on logits; every step of the path runs in kernels.hip.
#include <math.h>
#include <stddef.h>
#include <stdint.h>
#include <stdlib.h>

#include <mutex>

#include <hip/hip_runtime.h>

#include "tsr.h"
#include "kernels.hpp"
#if TSR_TRACE
#include "tsr_trace.h"
#endif

struct tsr_ctx {
  int device;
  int max_rows;
  int max_vocab;
  int max_k;
  uint64_t seed;
  tsr::VerifyWs ws;
  tsr::BeamWs bws;
  void* pws;   // verify_probs' workspace
  void* ws_block;
#if TSR_TRACE
  unsigned long long* trace;   // phase stamps (tracing build)
#endif
};

namespace {

// Per-row parameters are read on the device with this layout.
static_assert(sizeof(tsr::RowParams) == sizeof(tsr_params), "tsr_params layout");
static_assert(offsetof(tsr::RowParams, temperature) == offsetof(tsr_params, temperature) &&
                  offsetof(tsr::RowParams, top_k) == offsetof(tsr_params, top_k) &&
                  offsetof(tsr::RowParams, top_p) == offsetof(tsr_params, top_p) &&
                  offsetof(tsr::RowParams, min_p) == offsetof(tsr_params, min_p) &&
                  offsetof(tsr::RowParams, filter_mode) == offsetof(tsr_params, filter_mode),
              "tsr_params layout");

constexpr double kTemperatureMin = 1e-30;
constexpr double kTemperatureMax = 1e30;   // of the scoring calls
constexpr int kMaxDraft = 32;
constexpr int kMaxTreeNodes = 32;

// Runs f with the handle's device current and restores the caller's device.
template <class F>
int on_device(int device, F&& f) {
  int prev = -1;
  if (hipGetDevice(&prev) != hipSuccess) return TSR_EDEVICE;
  if (prev != device && hipSetDevice(device) != hipSuccess) return TSR_EDEVICE;
  const int rc = f();
  if (prev != device) (void)hipSetDevice(prev);
  return rc;
}

int check_params(const tsr_params* p) {
  if (!p) return TSR_EINVAL;
  if (!isfinite(p->temperature) || !isfinite(p->top_p) || !isfinite(p->min_p))
    return TSR_EINVAL;
  if (p->temperature < 0.0) return TSR_EINVAL;
  if (p->temperature > 0.0 && p->temperature < kTemperatureMin) return TSR_EINVAL;
  if (p->top_p < 0.0) return TSR_EINVAL;
  if (p->filter_mode != TSR_JOINT && p->filter_mode != TSR_SEQUENTIAL) return TSR_EINVAL;
  return TSR_OK;
}

tsr::KParams make_kparams(uint64_t seed, const tsr_params* p, int vocab, uint64_t step,
                          bool want_z) {
  tsr::KParams kp{};
  const double T = p->temperature;
  if (T == 0.0) {
    kp.flags = tsr::F_GREEDY;
    kp.c = 1.0f;
  } else {
    kp.c = (float)(1.4426950408889634 / T);
    kp.cR = kp.c * 16.0f;
    if (p->top_k > 0 && p->top_k < vocab) {
      kp.top_k = p->top_k;
      kp.flags |= tsr::F_K;
    }
    if (p->top_p < 1.0) {
      kp.top_p = p->top_p;
      kp.flags |= tsr::F_P;
    }
    if (p->min_p > 0.0 && p->min_p < 1.0) {
      kp.minp_off = T * log(p->min_p);
      kp.flags |= tsr::F_M;
    }
    if (p->filter_mode == TSR_SEQUENTIAL) kp.flags |= tsr::F_SEQ;
    if (want_z) kp.flags |= tsr::F_Z;
  }
  kp.key0 = (uint32_t)(seed & 0xFFFFFFFFu);
  kp.key1 = (uint32_t)(seed >> 32);
  kp.step_lo = (uint32_t)(step & 0xFFFFFFFFu);
  kp.step_hi = (uint32_t)(step >> 32);
  return kp;
}

int esize(int dtype) { return dtype == TSR_F32 ? 4 : 2; }

bool elem_aligned(const void* p, int dtype) {
  return ((uintptr_t)p % (uintptr_t)esize(dtype)) == 0;
}

bool word_aligned(const void* p) { return ((uintptr_t)p % 4) == 0; }

constexpr int kMaxQuantWidth = 1 << 30;
constexpr int kMaxQuantRows = (1 << 24) - 1;   // 256 threads a row: fewer than 2^32 in a launch
// sums of products of 8-bit integers fit 32 bits: 2^17 - 1 times (-128)^2
constexpr int kMaxInt8Width = (1 << 17) - 1;
constexpr int64_t kMaxInt8Stride = 1 << 22;   // a tile's 320 rows within 2^31 bytes
constexpr int kMaxInt8Vocab = 1 << 29;        // 256 threads to 64 channels: fewer than 2^32
constexpr int kMaxWideVocab = 1 << 30;          // ids past the last one stay whole numbers
constexpr int kMaxVprobsRows = (1 << 22) - 1;   // 1024 threads a sequence: fewer than 2^32

int check_quantize(const void* x, int dtype, int rows, int width, int64_t row_stride,
                   const int8_t* out_codes, int64_t codes_stride, const float* out_scale) {
  if (!x || !out_codes || !out_scale) return TSR_EINVAL;
  if (dtype != TSR_F32 && dtype != TSR_BF16) return TSR_EINVAL;
  if (rows < 0 || width < 1 || row_stride < width || codes_stride < width) return TSR_EINVAL;
  if (!elem_aligned(x, dtype) || !word_aligned(out_scale)) return TSR_EINVAL;
  if (width > kMaxQuantWidth || rows > kMaxQuantRows) return TSR_EUNSUPPORTED;
  return TSR_OK;
}

int check_int8(tsr_handle h, const int8_t* codes, int64_t codes_stride, const float* code_scale,
               int rows, const tsr_head* head, const void* out_logits, int dtype,
               int64_t out_stride) {
  if (!codes || !code_scale || !head || !out_logits) return TSR_EINVAL;
  if (!head->weight || !head->scale) return TSR_EINVAL;
  if (dtype != TSR_F32 && dtype != TSR_BF16) return TSR_EINVAL;
  if (rows < 0 || rows > h->max_rows || head->vocab < 1 || head->vocab > h->max_vocab ||
      head->width < 1)
    return TSR_EINVAL;
  if (codes_stride < head->width || head->weight_stride < head->width || out_stride < head->vocab)
    return TSR_EINVAL;
  if (!word_aligned(code_scale) || !word_aligned(head->scale) || !word_aligned(head->bias) ||
      !elem_aligned(out_logits, dtype))
    return TSR_EINVAL;
  if (head->width > kMaxInt8Width || head->vocab > kMaxInt8Vocab) return TSR_EUNSUPPORTED;
  // a single row has no next one
  if ((rows > 1 && codes_stride >= kMaxInt8Stride) ||
      (head->vocab > 1 && head->weight_stride >= kMaxInt8Stride))
    return TSR_EUNSUPPORTED;
  return TSR_OK;
}

constexpr int kMaxScoreRows = (1 << 22) - 1;    // 256 threads a slice of a row, 64 slices at most
constexpr int64_t kMaxScoreStride = 1ll << 36;   // rows times it, in bytes, within 2^63
constexpr int kMaxScoreTokens = 1024;           // the gradient compares a row's tokens in pairs

// Memory of `rows` rows of `width` bytes, `stride` bytes apart.
struct Rows {
  const void* at;
  int64_t stride, width;
  int rows;
};

// Whether a and b have a byte in common. Rows of the same stride may lie between each
// other's (columns of one larger matrix); of other strides, what lies from the first byte
// to the last counts.
bool overlap(Rows a, Rows b) {
  if (!a.at || !b.at || a.rows < 1 || b.rows < 1 || a.width < 1 || b.width < 1) return false;
  const uintptr_t x = (uintptr_t)a.at, y = (uintptr_t)b.at;
  const uint64_t xs = (uint64_t)((a.rows - 1) * a.stride + a.width);
  const uint64_t ys = (uint64_t)((b.rows - 1) * b.stride + b.width);
  if (x >= y + ys || y >= x + xs) return false;
  if (a.rows == 1) a.stride = b.stride;
  if (b.rows == 1) b.stride = a.stride;
  if (a.stride != b.stride || a.stride < 1) return true;
  const int64_t s = a.stride;
  const int64_t d = y >= x ? (int64_t)((y - x) % (uint64_t)s)
                           : (s - (int64_t)((x - y) % (uint64_t)s)) % s;
  return d < a.width || d + b.width > s;   // b's rows between a's end and its next
}

// Memory without gaps.
Rows block_of(const void* at, int64_t bytes) { return Rows{at, bytes, bytes, 1}; }

// Whether an output lies over an input or another output.
template <size_t O, size_t I>
bool clash(const Rows (&outs)[O], const Rows (&ins)[I]) {
  for (size_t i = 0; i < O; ++i) {
    for (size_t j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return true;
    for (size_t j = 0; j < I; ++j)
      if (overlap(outs[i], ins[j])) return true;
  }
  return false;
}

// Arguments of rows of logits that the scoring calls share. Strides times rows stay
// within 64 bits.
int check_scores(const void* logits, int dtype, int rows, int vocab, int64_t row_stride,
                 double temperature) {
  if (!logits) return TSR_EINVAL;
  if (dtype != TSR_F32 && dtype != TSR_BF16) return TSR_EINVAL;
  if (rows < 0 || vocab < 1 || row_stride < vocab || !elem_aligned(logits, dtype))
    return TSR_EINVAL;
  // log2(e) / T stays a float32 number
  if (!(temperature >= kTemperatureMin && temperature <= kTemperatureMax))
    return TSR_EINVAL;
  if (vocab > kMaxWideVocab || rows > kMaxScoreRows || row_stride >= kMaxScoreStride)
    return TSR_EUNSUPPORTED;
  return TSR_OK;
}

// Arguments every verify entry point checks (the handle's limits aside).
int check_verify(const void* target_logits, const void* draft_logits, int dtype,
                 const int32_t* draft_tokens, int rows, int K, int vocab,
                 const tsr_params* params, const int32_t* out_tokens,
                 const int32_t* out_accepted) {
  if (!target_logits || !draft_tokens || !out_tokens || !out_accepted) return TSR_EINVAL;
  if (dtype != TSR_F32 && dtype != TSR_BF16) return TSR_EINVAL;
  if (rows < 0 || vocab < 1 || K < 1 || K > kMaxDraft) return TSR_EINVAL;
  const int prc = check_params(params);
  if (prc != TSR_OK) return prc;
  if (params->temperature > 0.0 && !draft_logits) return TSR_EINVAL;
  if (!elem_aligned(target_logits, dtype) || (draft_logits && !elem_aligned(draft_logits, dtype)))
    return TSR_EINVAL;
  if (vocab > tsr::max_vocab_verify(dtype)) return TSR_EUNSUPPORTED;
  return TSR_OK;
}

// The verify launch once the arguments are checked (the device is current).
int launch_verify_checked(const void* target_logits, const void* draft_logits, int dtype,
                          const int32_t* draft_tokens, int rows, int K, int vocab,
                          const tsr::KParams& kp, const tsr::VerifyWs& ws, int32_t* out_tokens,
                          int32_t* out_accepted, int32_t* out_status, void* hip_stream) {
  // a row of a whole number of 16-byte chunks has no partial one (rows may
  // start at any element boundary)
  const int ragged = (vocab % (dtype == TSR_F32 ? 4 : 8)) != 0;
  const hipError_t e = tsr::launch_verify(target_logits, draft_logits, dtype, draft_tokens, rows,
                                          K, vocab, ragged, kp, ws, out_tokens,
                                          out_accepted, out_status, (hipStream_t)hip_stream);
  return e == hipSuccess ? TSR_OK : TSR_EDEVICE;
}

// spec_verify_noalloc's workspace: the per-(sequence, position) results (four
// int32 arrays of kStaticSlots), in `scratch` below: one copy per device,
// held until the process ends, shared by every call on that device. Every
// call writes each slot it reads, so nothing needs clearing.
constexpr int kStaticSlots = 1 << 16;   // sequences x (K + 1) positions
constexpr int kStaticSeqs = 1 << 14;    // sequences per call
constexpr size_t kStaticBytes = 4 * (size_t)kStaticSlots * sizeof(int32_t);
constexpr int kMaxDevices = 64;
std::mutex g_static_mu;
void* g_static_ptr[kMaxDevices];   // device address of `scratch` on each device, once looked up

}  // namespace

// In host code `scratch` names a host-side stand-in, not device memory: only
// its address from hipGetSymbolAddress (static_workspace) reaches kernels.
static __device__ __align__(256) unsigned char scratch[kStaticBytes];

namespace {

// The device address of `scratch` on `device` (the current device), looked up
// once per device and kept.
int static_workspace(int device, void** out) {
  if (device >= kMaxDevices) return TSR_EUNSUPPORTED;
  std::lock_guard<std::mutex> lock(g_static_mu);
  if (!g_static_ptr[device]) {
    void* p = nullptr;
    if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || !p) return TSR_EDEVICE;
    g_static_ptr[device] = p;
  }
  *out = g_static_ptr[device];
  return TSR_OK;
}

}  // namespace

extern "C" {

const char* sampler_strerror(int code) {
  switch (code) {
    case TSR_OK: return "ok";
    case TSR_EINVAL: return "invalid argument";
    case TSR_ENOMEM: return "out of device memory";
    case TSR_EDEVICE: return "HIP runtime error";
    case TSR_EUNSUPPORTED: return "size not supported by this build";
    default: return "unknown error code";
  }
}

int sampler_init(tsr_handle* out, int device, int max_rows, int max_vocab, int max_k,
                 uint64_t seed) {
  if (!out) return TSR_EINVAL;
  *out = nullptr;
  if (max_rows < 1 || max_vocab < 1 || max_k < 0 || max_k > kMaxDraft) return TSR_EINVAL;
  int ndev = 0;
  if (hipGetDeviceCount(&ndev) != hipSuccess) return TSR_EDEVICE;
  if (device < 0 || device >= ndev) return TSR_EINVAL;
  tsr_ctx* h = (tsr_ctx*)calloc(1, sizeof(tsr_ctx));
  if (!h) return TSR_ENOMEM;
  h->device = device;
  h->max_rows = max_rows;
  h->max_vocab = max_vocab;
  h->max_k = max_k;
  h->seed = seed;
  const int rc = on_device(device, [&]() -> int {
    const size_t slots = (size_t)max_rows * (size_t)(max_k + 1);
    const size_t vbytes = 4 * slots * sizeof(int32_t) + (size_t)max_rows * sizeof(uint32_t);
    const size_t bslots = (size_t)max_rows * tsr::kBeamMax;
    const size_t rbytes = (size_t)max_rows * 2 * (size_t)(max_k + 1) * sizeof(tsr::RowRec) +
                          (size_t)max_rows * 2 * tsr::kMaxSlices * sizeof(unsigned long long);
    const size_t bbytes = bslots * (sizeof(double) + sizeof(int32_t));
    const size_t pat = (((vbytes + 7) & ~(size_t)7) + rbytes + bbytes + 15) & ~(size_t)15;
    const size_t bytes = pat + tsr::vprobs_ws_most(max_rows, max_vocab);
    if (hipMalloc(&h->ws_block, bytes) != hipSuccess) return TSR_ENOMEM;
    if (hipMemset(h->ws_block, 0, bytes) != hipSuccess) return TSR_EDEVICE;
    if (hipDeviceSynchronize() != hipSuccess) return TSR_EDEVICE;
    int32_t* base = (int32_t*)h->ws_block;
    h->ws.acc = base;
    h->ws.tok = base + slots;
    h->ws.st_t = base + 2 * slots;
    h->ws.st_d = base + 3 * slots;
    h->ws.counter = (uint32_t*)(base + 4 * slots);
    h->ws.kmax1 = max_k + 1;
    // wide verify: per sequence 2 (max_k + 1) row records
    h->ws.rec = (tsr::RowRec*)((char*)h->ws_block + ((vbytes + 7) & ~(size_t)7));
    h->ws.recs = 2 * (max_k + 1);
    h->ws.part = (unsigned long long*)(h->ws.rec + (size_t)max_rows * 2 * (max_k + 1));
    // beam step: per row kBeamMax (score, token)
    char* bb = (char*)h->ws_block + ((vbytes + 7) & ~(size_t)7) + rbytes;
    h->bws.score = (double*)bb;
    h->bws.tok = (int32_t*)(bb + bslots * sizeof(double));
    h->pws = (char*)h->ws_block + pat;
#if TSR_TRACE
    if (hipMalloc(&h->trace, TSR_TRACE_WORDS * sizeof(uint64_t)) != hipSuccess) return TSR_ENOMEM;
    if (hipMemset(h->trace, 0, TSR_TRACE_WORDS * sizeof(uint64_t)) != hipSuccess) return TSR_EDEVICE;
    if (hipDeviceSynchronize() != hipSuccess) return TSR_EDEVICE;
#endif
    return TSR_OK;
  });
  if (rc != TSR_OK) {
    if (h->ws_block) (void)hipFree(h->ws_block);
#if TSR_TRACE
    if (h->trace) (void)hipFree(h->trace);
#endif
    free(h);
    return rc;
  }
  *out = h;
  return TSR_OK;
}

int sampler_destroy(tsr_handle h) {
  if (!h) return TSR_OK;
  const int rc = on_device(h->device, [&]() -> int {
    if (hipDeviceSynchronize() != hipSuccess) return TSR_EDEVICE;
    if (h->ws_block && hipFree(h->ws_block) != hipSuccess) return TSR_EDEVICE;
#if TSR_TRACE
    if (h->trace && hipFree(h->trace) != hipSuccess) return TSR_EDEVICE;
#endif
    return TSR_OK;
  });
  free(h);
  return rc;
}

int greedy_argmax(tsr_handle h, const void* logits, int dtype, int rows, int vocab,
                  int64_t row_stride, int32_t* out_tokens, int32_t* out_status,
                  void* hip_stream) {
  if (!h || !logits || !out_tokens) return TSR_EINVAL;
  if (dtype != TSR_F32 && dtype != TSR_BF16) return TSR_EINVAL;
  if (rows < 0 || rows > h->max_rows || vocab < 1 || vocab > h->max_vocab) return TSR_EINVAL;
  if (row_stride < vocab || !elem_aligned(logits, dtype)) return TSR_EINVAL;
  if (vocab > tsr::max_vocab_sample(dtype)) return TSR_EUNSUPPORTED;
  if (rows == 0) return TSR_OK;
  const long long sb = (long long)row_stride * esize(dtype);
  const int ragged = (vocab % (dtype == TSR_F32 ? 4 : 8)) != 0;   // a partial last chunk
  return on_device(h->device, [&]() -> int {
    const hipError_t e = tsr::launch_greedy(logits, dtype, rows, vocab, sb, ragged,
                                            out_tokens, out_status, (hipStream_t)hip_stream);
    return e == hipSuccess ? TSR_OK : TSR_EDEVICE;
  });
}

int sample_rows_ex(tsr_handle h, const void* logits, int dtype, int rows, int vocab,
                   int64_t row_stride, const tsr_constraints* cons, const tsr_params* params,
                   uint64_t step, int32_t* out_tokens, float* out_logprob, const tsr_diag* diag,
                   void* hip_stream) {
  if (!h || !logits || !out_tokens) return TSR_EINVAL;
  if (dtype != TSR_F32 && dtype != TSR_BF16) return TSR_EINVAL;
  if (rows < 0 || rows > h->max_rows || vocab < 1 || vocab > h->max_vocab) return TSR_EINVAL;
  if (row_stride < vocab || !elem_aligned(logits, dtype)) return TSR_EINVAL;
  const tsr_constraints none{};
  const tsr_constraints& cs = cons ? *cons : none;
  if (cs.allowed) {
    const int64_t words = ((int64_t)vocab + 31) / 32;
    if (cs.allowed_stride < words || ((uintptr_t)cs.allowed % 4) != 0) return TSR_EINVAL;
  }
  if (!cs.history && cs.history_len > 0) return TSR_EINVAL;   // a window length without ids
  const bool rep_given = cs.history && cs.history_len > 0;
  if (rep_given) {
    if (cs.history_len > tsr::kHistMax || cs.history_stride < cs.history_len ||
        ((uintptr_t)cs.history % 4) != 0)
      return TSR_EINVAL;
    if (!isfinite(cs.repetition_penalty) || cs.repetition_penalty < 1.0) return TSR_EINVAL;
  } else if (cs.history_len < 0) {
    return TSR_EINVAL;
  }
  if (cs.row_params && ((uintptr_t)cs.row_params % alignof(tsr_params)) != 0) return TSR_EINVAL;
  const tsr_params unit{1.0, 0, 1.0, 0.0, TSR_JOINT};
  if (!params && cs.row_params) params = &unit;   // the rows carry their own
  const int prc = check_params(params);
  if (prc != TSR_OK) return prc;
  if (vocab > tsr::max_vocab_sample(dtype)) return TSR_EUNSUPPORTED;
  if (rows == 0) return TSR_OK;
  tsr::DiagPtrs dg{};
  if (diag) {
    dg.status = diag->status;
    dg.kept_count = diag->kept_count;
    dg.threshold = diag->threshold;
    dg.kept_mass = diag->kept_mass;
    dg.probs = diag->probs;
  }
  dg.logprob = out_logprob;
  tsr::KParams kp = make_kparams(h->seed, params, vocab, step, dg.kept_mass != nullptr);
#if TSR_TRACE
  kp.trace = h->trace;
#endif
  if (cs.row_params) {
    kp.rowp = reinterpret_cast<const tsr::RowParams*>(cs.row_params);
    kp.flags |= tsr::F_ROWP;
    if (dg.kept_mass) kp.flags |= tsr::F_Z;
  }
  if (cs.allowed) {
    kp.allowed = cs.allowed;
    kp.allowed_stride = (long long)cs.allowed_stride;
    kp.flags |= tsr::F_MASK;
  }
  if (rep_given && cs.repetition_penalty != 1.0) {
    kp.hist = cs.history;
    kp.hist_stride = (long long)cs.history_stride;
    kp.hist_len = cs.history_len;
    kp.rpen = cs.repetition_penalty;
    kp.flags |= tsr::F_REP;
  }
  const long long sb = (long long)row_stride * esize(dtype);
  const int ragged = (vocab % (dtype == TSR_F32 ? 4 : 8)) != 0;   // a partial last chunk
  return on_device(h->device, [&]() -> int {
    const hipError_t e = tsr::launch_sample(logits, dtype, rows, vocab, sb, ragged, kp,
                                            out_tokens, dg, (hipStream_t)hip_stream);
    return e == hipSuccess ? TSR_OK : TSR_EDEVICE;
  });
}

int sample_rows_masked(tsr_handle h, const void* logits, int dtype, int rows, int vocab,
                       int64_t row_stride, const uint32_t* allowed, int64_t allowed_stride,
                       const tsr_params* params, uint64_t step, int32_t* out_tokens,
                       float* out_logprob, const tsr_diag* diag, void* hip_stream) {
  tsr_constraints cs{};
  cs.allowed = allowed;
  cs.allowed_stride = allowed_stride;
  return sample_rows_ex(h, logits, dtype, rows, vocab, row_stride, &cs, params, step, out_tokens,
                        out_logprob, diag, hip_stream);
}

int sample_rows(tsr_handle h, const void* logits, int dtype, int rows, int vocab,
                int64_t row_stride, const tsr_params* params, uint64_t step,
                int32_t* out_tokens, const tsr_diag* diag, void* hip_stream) {
  return sample_rows_masked(h, logits, dtype, rows, vocab, row_stride, nullptr, 0, params, step,
                            out_tokens, nullptr, diag, hip_stream);
}

int spec_verify(tsr_handle h, const void* target_logits, const void* draft_logits, int dtype,
                const int32_t* draft_tokens, int rows, int K, int vocab,
                const tsr_params* params, uint64_t step, int32_t* out_tokens,
                int32_t* out_accepted, int32_t* out_status, void* hip_stream) {
  if (!h) return TSR_EINVAL;
  if (rows > h->max_rows || vocab > h->max_vocab || K > h->max_k) return TSR_EINVAL;
  const int rc = check_verify(target_logits, draft_logits, dtype, draft_tokens, rows, K, vocab,
                              params, out_tokens, out_accepted);
  if (rc != TSR_OK || rows == 0) return rc;
  tsr::KParams kp = make_kparams(h->seed, params, vocab, step, false);
#if TSR_TRACE
  kp.trace = h->trace;
#endif
  return on_device(h->device, [&]() -> int {
    return launch_verify_checked(target_logits, draft_logits, dtype, draft_tokens, rows, K, vocab,
                                 kp, h->ws, out_tokens, out_accepted, out_status, hip_stream);
  });
}

int spec_verify_noalloc(int device, uint64_t seed, const void* target_logits,
                        const void* draft_logits, int dtype, const int32_t* draft_tokens,
                        int rows, int K, int vocab, const tsr_params* params, uint64_t step,
                        int32_t* out_tokens, int32_t* out_accepted, int32_t* out_status,
                        void* hip_stream) {
  if (rows > kStaticSeqs || (int64_t)rows * (K + 1) > kStaticSlots) return TSR_EINVAL;
  const int rc = check_verify(target_logits, draft_logits, dtype, draft_tokens, rows, K, vocab,
                              params, out_tokens, out_accepted);
  if (rc != TSR_OK) return rc;
  if (vocab > tsr::max_vocab_verify_narrow(dtype)) return TSR_EUNSUPPORTED;
  int ndev = 0;
  if (hipGetDeviceCount(&ndev) != hipSuccess) return TSR_EDEVICE;
  if (device < 0 || device >= ndev) return TSR_EINVAL;
  if (rows == 0) return TSR_OK;
  const tsr::KParams kp = make_kparams(seed, params, vocab, step, false);
  return on_device(device, [&]() -> int {
    void* base = nullptr;
    const int src = static_workspace(device, &base);
    if (src != TSR_OK) return src;
    int32_t* b = (int32_t*)base;
    tsr::VerifyWs ws;
    ws.acc = b;
    ws.tok = b + kStaticSlots;
    ws.st_t = b + 2 * kStaticSlots;
    ws.st_d = b + 3 * kStaticSlots;
    ws.counter = nullptr;   // the two-row verify keeps no arrival counters
    ws.kmax1 = K + 1;
    ws.rec = nullptr;   // the array holds no row records: register-pair rows only
    ws.recs = 0;
    ws.part = nullptr;
    return launch_verify_checked(target_logits, draft_logits, dtype, draft_tokens, rows, K, vocab,
                                 kp, ws, out_tokens, out_accepted, out_status, hip_stream);
  });
}

int tree_verify(tsr_handle h, const void* target_logits, const void* draft_logits, int dtype,
                const int32_t* parent, const int32_t* tokens, int rows, int nodes, int vocab,
                const tsr_params* params, uint64_t step, int32_t* out_tokens, int32_t* out_path,
                int32_t* out_accepted, int32_t* out_status, void* hip_stream) {
  if (!h || !target_logits || !parent || !tokens || !out_tokens || !out_path || !out_accepted)
    return TSR_EINVAL;
  if (dtype != TSR_F32 && dtype != TSR_BF16) return TSR_EINVAL;
  if (rows < 0 || rows > h->max_rows || vocab < 1 || vocab > h->max_vocab) return TSR_EINVAL;
  if (nodes < 1 || nodes > kMaxTreeNodes || nodes > h->max_k + 1) return TSR_EINVAL;
  const int prc = check_params(params);
  if (prc != TSR_OK) return prc;
  if (params->temperature > 0.0 && !draft_logits) return TSR_EINVAL;
  if (!elem_aligned(target_logits, dtype) || (draft_logits && !elem_aligned(draft_logits, dtype)))
    return TSR_EINVAL;
  if (vocab > tsr::max_vocab_verify(dtype)) return TSR_EUNSUPPORTED;
  if (rows == 0) return TSR_OK;
  tsr::KParams kp = make_kparams(h->seed, params, vocab, step, false);
#if TSR_TRACE
  kp.trace = h->trace;
#endif
  // a row of a whole number of 16-byte chunks has no partial one (rows may
  // start at any element boundary)
  const int ragged = (vocab % (dtype == TSR_F32 ? 4 : 8)) != 0;
  return on_device(h->device, [&]() -> int {
    const hipError_t e = tsr::launch_tree(target_logits, draft_logits, dtype, parent, tokens, rows,
                                          nodes, vocab, ragged, kp, h->ws, out_tokens,
                                          out_path, out_accepted, out_status,
                                          (hipStream_t)hip_stream);
    return e == hipSuccess ? TSR_OK : TSR_EDEVICE;
  });
}

int beam_step(tsr_handle h, const void* logits, int dtype, int groups, int beam, int vocab,
              int64_t row_stride, const double* beam_scores, int32_t* out_parent,
              int32_t* out_token, double* out_score, int32_t* out_status, void* hip_stream) {
  if (!h || !logits || !beam_scores || !out_parent || !out_token || !out_score) return TSR_EINVAL;
  if (dtype != TSR_F32 && dtype != TSR_BF16) return TSR_EINVAL;
  if (beam < 1 || beam > tsr::kBeamMax || groups < 0) return TSR_EINVAL;
  if ((int64_t)groups * beam > h->max_rows || vocab < 1 || vocab > h->max_vocab) return TSR_EINVAL;
  if (row_stride < vocab || !elem_aligned(logits, dtype) || ((uintptr_t)beam_scores % 8) != 0)
    return TSR_EINVAL;
  if (vocab > tsr::max_vocab_beam(dtype)) return TSR_EUNSUPPORTED;
  const long long sb = (long long)row_stride * esize(dtype);
  if (groups == 0) return TSR_OK;
  const int ragged = (vocab % (dtype == TSR_F32 ? 4 : 8)) != 0;   // a partial last chunk
  return on_device(h->device, [&]() -> int {
    const hipError_t e = tsr::launch_beam(logits, dtype, groups, beam, vocab, sb, ragged,
                                          beam_scores, h->bws, out_parent, out_token, out_score,
                                          out_status, (hipStream_t)hip_stream);
    return e == hipSuccess ? TSR_OK : TSR_EDEVICE;
  });
}

int quantize_rows(tsr_handle h, const void* x, int dtype, int rows, int width, int64_t row_stride,
                  int8_t* out_codes, int64_t codes_stride, float* out_scale, void* hip_stream) {
  if (!h) return TSR_EINVAL;
  const int rc = check_quantize(x, dtype, rows, width, row_stride, out_codes, codes_stride,
                                out_scale);
  if (rc != TSR_OK || rows == 0) return rc;
  return on_device(h->device, [&]() -> int {
    const hipError_t e = tsr::launch_quantize(x, dtype, rows, width,
                                              (long long)row_stride * esize(dtype), out_codes,
                                              (long long)codes_stride, out_scale,
                                              (hipStream_t)hip_stream);
    return e == hipSuccess ? TSR_OK : TSR_EDEVICE;
  });
}

int int8_logits(tsr_handle h, const int8_t* codes, int64_t codes_stride, const float* code_scale,
                int rows, const tsr_head* head, void* out_logits, int dtype, int64_t out_stride,
                void* hip_stream) {
  if (!h) return TSR_EINVAL;
  const int rc = check_int8(h, codes, codes_stride, code_scale, rows, head, out_logits, dtype,
                            out_stride);
  if (rc != TSR_OK || rows == 0) return rc;
  tsr::Int8Args a{};
  a.x = codes;
  a.x_stride = rows > 1 ? (long long)codes_stride : 0;   // no next row: any alignment and distance
  a.x_scale = code_scale;
  a.w = head->weight;
  a.w_stride = head->vocab > 1 ? (long long)head->weight_stride : 0;
  a.w_scale = head->scale;
  a.bias = head->bias;
  a.out = static_cast<unsigned char*>(out_logits);
  a.out_stride_bytes = (long long)out_stride * esize(dtype);
  a.rows = rows;
  a.vocab = head->vocab;
  a.width = head->width;
  return on_device(h->device, [&]() -> int {
    const hipError_t e = tsr::launch_int8(a, dtype, (hipStream_t)hip_stream);
    return e == hipSuccess ? TSR_OK : TSR_EDEVICE;
  });
}

int sample_hidden(tsr_handle h, const void* hidden, int hidden_dtype, int rows,
                  int64_t hidden_stride, const tsr_head* head, int8_t* codes,
                  int64_t codes_stride, float* code_scale, void* logits, int dtype,
                  const tsr_params* params, uint64_t step, int32_t* out_tokens,
                  const tsr_diag* diag, void* hip_stream) {
  // every argument of the three steps first: an error leaves nothing enqueued
  if (!h || !head || !out_tokens) return TSR_EINVAL;
  int rc = check_quantize(hidden, hidden_dtype, rows, head->width, hidden_stride, codes,
                          codes_stride, code_scale);
  if (rc == TSR_OK)
    rc = check_int8(h, codes, codes_stride, code_scale, rows, head, logits, dtype, head->vocab);
  if (rc == TSR_OK) rc = check_params(params);
  if (rc == TSR_OK && head->vocab > tsr::max_vocab_sample(dtype)) rc = TSR_EUNSUPPORTED;
  if (rc != TSR_OK || rows == 0) return rc;
  rc = quantize_rows(h, hidden, hidden_dtype, rows, head->width, hidden_stride, codes,
                     codes_stride, code_scale, hip_stream);
  if (rc == TSR_OK)
    rc = int8_logits(h, codes, codes_stride, code_scale, rows, head, logits, dtype, head->vocab,
                     hip_stream);
  if (rc == TSR_OK)
    rc = sample_rows(h, logits, dtype, rows, head->vocab, head->vocab, params, step, out_tokens,
                     diag, hip_stream);
  return rc;
}

int verify_probs_workspace(int dtype, int rows, int vocab) {
  if ((dtype != TSR_F32 && dtype != TSR_BF16) || rows < 1 || vocab < 1) return 0;
  return (int)tsr::vprobs_ws_bytes(dtype, rows, vocab);
}

int verify_probs_ex(tsr_handle h, const void* target_probs, int64_t target_seq_stride,
                    int64_t target_row_stride, const void* draft_probs, int64_t draft_seq_stride,
                    int64_t draft_row_stride, int dtype, const int32_t* draft_tokens,
                    const int32_t* draft_lens, const float* accept_u, const float* draw_u, int rows,
                    int K, int vocab, int32_t* out_tokens, int32_t* out_accepted,
                    int32_t* out_status, void* workspace, int64_t workspace_bytes,
                    void* hip_stream) {
  if (!h || !target_probs || !draft_tokens || !accept_u || !draw_u || !out_tokens || !out_accepted)
    return TSR_EINVAL;
  if (dtype != TSR_F32 && dtype != TSR_BF16) return TSR_EINVAL;
  if (rows < 0 || rows > h->max_rows || vocab < 1 || vocab > h->max_vocab) return TSR_EINVAL;
  if (K < 1 || K > kMaxDraft || K > h->max_k) return TSR_EINVAL;
  if (target_seq_stride < 0 || target_row_stride < 0) return TSR_EINVAL;
  if (draft_probs && (draft_seq_stride < 0 || draft_row_stride < 0)) return TSR_EINVAL;
  if (!elem_aligned(target_probs, dtype) || (draft_probs && !elem_aligned(draft_probs, dtype)))
    return TSR_EINVAL;
  if (!word_aligned(draft_tokens) || !word_aligned(draft_lens) || !word_aligned(accept_u) ||
      !word_aligned(draw_u) || !word_aligned(out_tokens) || !word_aligned(out_accepted) ||
      !word_aligned(out_status))
    return TSR_EINVAL;
  if (vocab > kMaxWideVocab || rows > kMaxVprobsRows) return TSR_EUNSUPPORTED;
  if (rows == 0) return TSR_OK;
  if (workspace && (((uintptr_t)workspace % 16) != 0 ||
                    workspace_bytes < (int64_t)tsr::vprobs_ws_bytes(dtype, rows, vocab)))
    return TSR_EINVAL;
  const long long es = esize(dtype);
  tsr::VprobsArgs a{};
  a.target = static_cast<const unsigned char*>(target_probs);
  a.t_seq = (long long)target_seq_stride * es;
  a.t_row = (long long)target_row_stride * es;
  a.draft = static_cast<const unsigned char*>(draft_probs);
  a.d_seq = (long long)draft_seq_stride * es;
  a.d_row = (long long)draft_row_stride * es;
  a.tokens = draft_tokens;
  a.lens = draft_lens;
  a.accept_u = accept_u;
  a.draw_u = draw_u;
  a.rows = rows;
  a.K = K;
  a.V = vocab;
  a.out_tokens = out_tokens;
  a.out_accepted = out_accepted;
  a.out_status = out_status;
  return on_device(h->device, [&]() -> int {
    const hipError_t e = tsr::launch_vprobs(a, dtype, workspace ? workspace : h->pws,
                                            (hipStream_t)hip_stream);
    return e == hipSuccess ? TSR_OK : TSR_EDEVICE;
  });
}

int verify_probs(tsr_handle h, const void* target_probs, int64_t target_seq_stride,
                 int64_t target_row_stride, const void* draft_probs, int64_t draft_seq_stride,
                 int64_t draft_row_stride, int dtype, const int32_t* draft_tokens,
                 const int32_t* draft_lens, const float* accept_u, const float* draw_u, int rows,
                 int K, int vocab, int32_t* out_tokens, int32_t* out_accepted,
                 int32_t* out_status, void* hip_stream) {
  return verify_probs_ex(h, target_probs, target_seq_stride, target_row_stride, draft_probs,
                         draft_seq_stride, draft_row_stride, dtype, draft_tokens, draft_lens,
                         accept_u, draw_u, rows, K, vocab, out_tokens, out_accepted, out_status,
                         nullptr, 0, hip_stream);
}

int norm_quantize_rows(tsr_handle h, const void* x, int64_t x_stride, const void* residual,
                       int64_t residual_stride, int dtype, const void* weight, int weight_dtype,
                       double eps, int rows, int width, void* out_residual,
                       int64_t out_residual_stride, int8_t* out_codes, int64_t codes_stride,
                       float* out_scale, void* hip_stream) {
  if (!h) return TSR_EINVAL;
  const int rc = check_quantize(x, dtype, rows, width, x_stride, out_codes, codes_stride,
                                out_scale);
  if (rc != TSR_OK) return rc;
  if (!isfinite(eps) || eps < 0.0) return TSR_EINVAL;
  if (weight && ((weight_dtype != TSR_F32 && weight_dtype != TSR_BF16) ||
                 !elem_aligned(weight, weight_dtype)))
    return TSR_EINVAL;
  if (residual && (residual_stride < width || !elem_aligned(residual, dtype))) return TSR_EINVAL;
  if (out_residual && (!residual || out_residual_stride < width ||
                       !elem_aligned(out_residual, dtype)))
    return TSR_EINVAL;
  if (x_stride >= kMaxScoreStride || codes_stride >= kMaxScoreStride ||
      (residual && residual_stride >= kMaxScoreStride) ||
      (out_residual && out_residual_stride >= kMaxScoreStride))
    return TSR_EUNSUPPORTED;
  if (rows == 0) return TSR_OK;
  const int es = esize(dtype);
  const Rows mx{x, x_stride * es, (int64_t)width * es, rows};
  const Rows mr{residual, residual_stride * es, (int64_t)width * es, rows};
  const Rows mh{out_residual, out_residual_stride * es, (int64_t)width * es, rows};
  const Rows mq{out_codes, codes_stride, width, rows};
  const Rows mw{weight, 0, (int64_t)width * esize(weight_dtype), 1};
  const Rows ms{out_scale, 0, (int64_t)rows * 4, 1};
  // the sum may take the place of x or of the residual, row for row
  const bool on_x = out_residual == x && (rows == 1 || out_residual_stride == x_stride);
  const bool on_r =
      out_residual == residual && (rows == 1 || out_residual_stride == residual_stride);
  if ((!on_x && overlap(mh, mx)) || (!on_r && overlap(mh, mr)) || overlap(mh, mw) ||
      overlap(mh, ms) || overlap(mh, mq))
    return TSR_EINVAL;
  if (overlap(mq, mx) || overlap(mq, mr) || overlap(mq, mw) || overlap(mq, ms)) return TSR_EINVAL;
  if (overlap(ms, mx) || overlap(ms, mr) || overlap(ms, mw)) return TSR_EINVAL;
  tsr::NormArgs a{};
  a.x = static_cast<const unsigned char*>(x);
  a.x_stride = (long long)x_stride * es;
  a.residual = static_cast<const unsigned char*>(residual);
  a.r_stride = (long long)residual_stride * es;
  a.weight = static_cast<const unsigned char*>(weight);
  a.eps = eps;
  a.rows = rows;
  a.width = width;
  a.out_h = static_cast<unsigned char*>(out_residual);
  a.h_stride = (long long)out_residual_stride * es;
  a.codes = out_codes;
  a.q_stride = (long long)codes_stride;
  a.scale = out_scale;
  return on_device(h->device, [&]() -> int {
    const hipError_t e =
        tsr::launch_norm_quantize(a, dtype, weight ? weight_dtype : dtype, (hipStream_t)hip_stream);
    return e == hipSuccess ? TSR_OK : TSR_EDEVICE;
  });
}

int token_logprobs_workspace(int dtype, int rows, int vocab, int top_k) {
  if ((dtype != TSR_F32 && dtype != TSR_BF16) || rows < 1 || vocab < 1 || top_k < 0 ||
      top_k > tsr::kMaxTop || rows > kMaxScoreRows || vocab > kMaxWideVocab)
    return 0;
  return (int)tsr::logprobs_ws_bytes(dtype, rows, vocab, top_k);
}

int token_logprobs(tsr_handle h, const void* logits, int dtype, int rows, int vocab,
                   int64_t row_stride, double temperature, const int32_t* tokens, int n_tokens,
                   int top_k, const tsr_logprobs* out, void* workspace, int64_t workspace_bytes,
                   void* hip_stream) {
  if (!h || !out) return TSR_EINVAL;
  const int rc = check_scores(logits, dtype, rows, vocab, row_stride, temperature);
  if (rc != TSR_OK) return rc;
  if (n_tokens < 0 || top_k < 0 || (n_tokens > 0 && (!tokens || !out->logprob)) ||
      (top_k > 0 && (!out->top_ids || !out->top_logprob)))
    return TSR_EINVAL;
  if (!word_aligned(tokens) || !word_aligned(out->logprob) || !word_aligned(out->entropy) ||
      !word_aligned(out->top_ids) || !word_aligned(out->top_logprob) ||
      !word_aligned(out->norm) || !word_aligned(out->status))
    return TSR_EINVAL;
  if (n_tokens > kMaxScoreTokens || top_k > tsr::kMaxTop) return TSR_EUNSUPPORTED;
  if (rows == 0) return TSR_OK;
  const int64_t need = (int64_t)tsr::logprobs_ws_bytes(dtype, rows, vocab, top_k);
  if (need && (!workspace || ((uintptr_t)workspace % 16) != 0 || workspace_bytes < need))
    return TSR_EINVAL;
  const int es = esize(dtype);
  const int64_t words = (int64_t)rows * 4;
  const Rows outs[] = {block_of(out->logprob, words * n_tokens), block_of(out->entropy, words),
                       block_of(out->top_ids, words * top_k),
                       block_of(out->top_logprob, words * top_k), block_of(out->norm, words * 2),
                       block_of(out->status, words), block_of(workspace, need)};
  const Rows ins[] = {Rows{logits, row_stride * es, (int64_t)vocab * es, rows},
                      block_of(tokens, words * n_tokens)};
  if (clash(outs, ins)) return TSR_EINVAL;
  tsr::LogprobArgs a{};
  a.logits = static_cast<const unsigned char*>(logits);
  a.stride_bytes = (long long)row_stride * esize(dtype);
  a.rows = rows;
  a.V = vocab;
  a.c = (float)(1.4426950408889634 / temperature);
  a.inv_t = 1.0 / temperature;
  a.tokens = tokens;
  a.n = n_tokens;
  a.k = top_k;
  a.logprob = out->logprob;
  a.entropy = out->entropy;
  a.top_ids = out->top_ids;
  a.top_logprob = out->top_logprob;
  a.norm = out->norm;
  a.status = out->status;
  return on_device(h->device, [&]() -> int {
    const hipError_t e = tsr::launch_logprobs(a, dtype, workspace, (hipStream_t)hip_stream);
    return e == hipSuccess ? TSR_OK : TSR_EDEVICE;
  });
}

int token_logprobs_grad(tsr_handle h, const void* logits, int dtype, int rows, int vocab,
                        int64_t row_stride, double temperature, const int32_t* tokens,
                        int n_tokens, const float* norm, const float* grad_logprob,
                        const float* entropy, const float* grad_entropy, void* out_grad,
                        int64_t grad_stride, void* hip_stream) {
  if (!h) return TSR_EINVAL;
  const int rc = check_scores(logits, dtype, rows, vocab, row_stride, temperature);
  if (rc != TSR_OK) return rc;
  if (!norm || !out_grad || n_tokens < 0 || (n_tokens > 0 && (!tokens || !grad_logprob)) ||
      (grad_entropy && !entropy) || grad_stride < vocab || !elem_aligned(out_grad, dtype))
    return TSR_EINVAL;
  if (!word_aligned(tokens) || !word_aligned(norm) || !word_aligned(grad_logprob) ||
      !word_aligned(entropy) || !word_aligned(grad_entropy))
    return TSR_EINVAL;
  if (n_tokens > kMaxScoreTokens || grad_stride >= kMaxScoreStride) return TSR_EUNSUPPORTED;
  if (rows == 0) return TSR_OK;
  // the logits are read again where the tokens are: the gradient has memory of its own
  const int es = esize(dtype);
  const int64_t words = (int64_t)rows * 4;
  const Rows outs[] = {Rows{out_grad, grad_stride * es, (int64_t)vocab * es, rows}};
  const Rows ins[] = {Rows{logits, row_stride * es, (int64_t)vocab * es, rows},
                      block_of(tokens, words * n_tokens), block_of(grad_logprob, words * n_tokens),
                      block_of(norm, words * 2), block_of(entropy, words),
                      block_of(grad_entropy, words)};
  if (clash(outs, ins)) return TSR_EINVAL;
  tsr::LogprobGradArgs a{};
  a.logits = static_cast<const unsigned char*>(logits);
  a.stride_bytes = (long long)row_stride * esize(dtype);
  a.rows = rows;
  a.V = vocab;
  a.c = (float)(1.4426950408889634 / temperature);
  a.inv_t = 1.0 / temperature;
  a.tokens = tokens;
  a.n = n_tokens;
  a.norm = norm;
  a.g = grad_logprob;
  a.entropy = entropy;
  a.ge = grad_entropy;
  a.out = static_cast<unsigned char*>(out_grad);
  a.out_stride_bytes = (long long)grad_stride * esize(dtype);
  return on_device(h->device, [&]() -> int {
    const hipError_t e = tsr::launch_logprobs_grad(a, dtype, (hipStream_t)hip_stream);
    return e == hipSuccess ? TSR_OK : TSR_EDEVICE;
  });
}

int distill_topk_workspace(int dtype, int rows, int vocab, int want_grad) {
  if ((dtype != TSR_F32 && dtype != TSR_BF16) || rows < 1 || vocab < 1 || rows > kMaxScoreRows ||
      vocab > kMaxWideVocab)
    return 0;
  return (int)tsr::distill_ws_bytes(dtype, rows, vocab, want_grad != 0);
}

int distill_topk(tsr_handle h, const void* logits, int dtype, int rows, int vocab,
                 int64_t row_stride, double temperature, const int32_t* ids,
                 const float* teacher_logprob, int k, int tail, const float* row_weight,
                 float* out_loss, void* out_grad, int64_t grad_stride, int32_t* out_status,
                 void* workspace, int64_t workspace_bytes, void* hip_stream) {
  if (!h) return TSR_EINVAL;
  const int rc = check_scores(logits, dtype, rows, vocab, row_stride, temperature);
  if (rc != TSR_OK) return rc;
  if (!ids || !teacher_logprob || !out_loss || k < 1 || (tail != 0 && tail != 1)) return TSR_EINVAL;
  if (out_grad && (grad_stride < vocab || !elem_aligned(out_grad, dtype))) return TSR_EINVAL;
  if (!word_aligned(ids) || !word_aligned(teacher_logprob) || !word_aligned(row_weight) ||
      !word_aligned(out_loss) || !word_aligned(out_status))
    return TSR_EINVAL;
  if (k > tsr::kMaxTop || (out_grad && grad_stride >= kMaxScoreStride)) return TSR_EUNSUPPORTED;
  if (rows == 0) return TSR_OK;
  const int64_t need = (int64_t)tsr::distill_ws_bytes(dtype, rows, vocab, out_grad != nullptr);
  if (need && (!workspace || ((uintptr_t)workspace % 16) != 0 || workspace_bytes < need))
    return TSR_EINVAL;
  // inputs are read more than once, and by several workgroups: outputs have memory of their own
  const int es = esize(dtype);
  const int64_t words = (int64_t)rows * 4;
  const Rows outs[] = {Rows{out_grad, grad_stride * es, (int64_t)vocab * es, rows},
                       block_of(out_loss, words), block_of(out_status, words),
                       block_of(workspace, need)};
  const Rows ins[] = {Rows{logits, row_stride * es, (int64_t)vocab * es, rows},
                      block_of(ids, words * k), block_of(teacher_logprob, words * k),
                      block_of(row_weight, words)};
  if (clash(outs, ins)) return TSR_EINVAL;
  tsr::DistillArgs a{};
  a.logits = static_cast<const unsigned char*>(logits);
  a.stride_bytes = (long long)row_stride * esize(dtype);
  a.rows = rows;
  a.V = vocab;
  a.c = (float)(1.4426950408889634 / temperature);
  a.inv_t = 1.0 / temperature;
  a.ids = ids;
  a.teacher = teacher_logprob;
  a.k = k;
  a.tail = tail;
  a.weight = row_weight;
  a.loss = out_loss;
  a.grad = static_cast<unsigned char*>(out_grad);
  a.grad_stride_bytes = (long long)grad_stride * esize(dtype);
  a.status = out_status;
  return on_device(h->device, [&]() -> int {
    const hipError_t e = tsr::launch_distill(a, dtype, workspace, (hipStream_t)hip_stream);
    return e == hipSuccess ? TSR_OK : TSR_EDEVICE;
  });
}

int sampler_philox(tsr_handle h, const uint32_t* counters, int n, uint32_t* out_words,
                   void* hip_stream) {
  if (!h || !counters || !out_words || n < 0) return TSR_EINVAL;
  if (n == 0) return TSR_OK;
  return on_device(h->device, [&]() -> int {
    const hipError_t e = tsr::launch_philox(counters, n, (uint32_t)(h->seed & 0xFFFFFFFFu),
                                            (uint32_t)(h->seed >> 32), out_words,
                                            (hipStream_t)hip_stream);
    return e == hipSuccess ? TSR_OK : TSR_EDEVICE;
  });
}

#if TSR_TRACE
int sampler_trace_read(tsr_handle h, uint64_t* out, int64_t n) {
  if (!h || !out || n < 0 || n > TSR_TRACE_WORDS) return TSR_EINVAL;
  return on_device(h->device, [&]() -> int {
    if (hipDeviceSynchronize() != hipSuccess) return TSR_EDEVICE;
    if (n && hipMemcpy(out, h->trace, (size_t)n * sizeof(uint64_t), hipMemcpyDeviceToHost) !=
                 hipSuccess)
      return TSR_EDEVICE;
    return TSR_OK;
  });
}

int sampler_trace_clear(tsr_handle h) {
  if (!h) return TSR_EINVAL;
  return on_device(h->device, [&]() -> int {
    if (hipDeviceSynchronize() != hipSuccess) return TSR_EDEVICE;
    if (hipMemset(h->trace, 0, TSR_TRACE_WORDS * sizeof(uint64_t)) != hipSuccess)
      return TSR_EDEVICE;
    return hipDeviceSynchronize() == hipSuccess ? TSR_OK : TSR_EDEVICE;
  });
}
#endif

}  // extern "C"
