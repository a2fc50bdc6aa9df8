// C ABI of the library (declarations and contracts: include/mxfp4.h).
//
// Conventions follow the C-API review on "Initial integration of a4w4 GEMM"
// (ROCm/TransformerEngine #663): an int status per call with distinct
// negative codes and an availability probe; and the stride/arch contract of
// "feat(ck-tile): aquant GEMM TE to dispatcher bridge" (ROCm/rocm-libraries
// #9980): packed strides only, the architecture checked at run time, every
// argument validated before anything is launched.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <vector>

#include "decode.h"
#include "few_tokens.h"
#include "mx_internal.h"
#include "mxfp4.h"

#define MX_API extern "C" __attribute__((visibility("default")))

namespace {

// Detail of the last rejection or failure on this thread (mx_last_error_string):
// which call, which argument and which constraint.  Every entry point that
// returns a status clears it first, so it always describes the latest call.
thread_local char t_detail[256] = "";

void clear_detail() { t_detail[0] = '\0'; }

// Leaves the detail as it was (for checks in calls that return no status).
struct KeepDetail {
  char was[sizeof t_detail];
  KeepDetail() { memcpy(was, t_detail, sizeof was); }
  ~KeepDetail() { memcpy(t_detail, was, sizeof was); }
};

__attribute__((format(printf, 2, 3))) int fail(int code, const char *fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(t_detail, sizeof t_detail, fmt, ap);
  va_end(ap);
  return code;
}

int fail_cuda(const char *what, cudaError_t e) {
  cudaGetLastError();  // clear the runtime's sticky copy of a non-fatal error
  return fail(MX_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

// Device status word (bit 0: a bounded wait ran out).  One copy per device
// that loads the library; kernels get its device address as an argument.
__device__ uint32_t g_status_word;

__global__ void probe_kernel() {}

// Per device: the architecture check (done once) and the device addresses of
// the library's arrays.  Those addresses belong to the CUDA context they were
// looked up in: after cudaDeviceReset (or when the caller makes another
// context current) the module is loaded again, possibly elsewhere, so they
// are looked up again whenever the current context differs from the one
// they came from.  The lookup happens on the first call of any entry point
// in a context, which also loads the module of the static split-K array
// (mxfp4_gemm_static_workspace), so no later call has to load a module
// while the caller may be capturing a stream.
struct DeviceInfo {
  bool checked = false;
  int rc = MX_OK;
  char why[160] = "";
  int num_sms = 0;
  CUcontext ctx = nullptr;
  uint32_t *status = nullptr;
  void *static_ws = nullptr;
};

constexpr int kMaxDevices = 64;
DeviceInfo g_devices[kMaxDevices];
std::mutex g_mutex;

using CtxGetCurrentFn = CUresult (*)(CUcontext *);

CUcontext current_context() {
  static CtxGetCurrentFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess) {
      fn = reinterpret_cast<CtxGetCurrentFn>(p);
    }
  });
  CUcontext c = nullptr;
  if (fn == nullptr || fn(&c) != CUDA_SUCCESS) return nullptr;
  return c;
}

int device_info(DeviceInfo **out) {
  int dev = 0;
  const cudaError_t ge = cudaGetDevice(&dev);
  if (ge != cudaSuccess) return fail_cuda("cudaGetDevice", ge);
  if (dev < 0 || dev >= kMaxDevices)
    return fail(MX_ERR_CUDA, "device index %d is outside the library's table of %d devices", dev,
                kMaxDevices);
  std::lock_guard<std::mutex> lock(g_mutex);
  DeviceInfo &d = g_devices[dev];
  if (!d.checked) {
    int major = 0, minor = 0;
    cudaError_t e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&d.num_sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return fail_cuda("cudaDeviceGetAttribute", e);
    if (major != 10 || minor != 3) {
      d.rc = MX_ERR_UNSUPPORTED_ARCH;
      snprintf(d.why, sizeof d.why, "device %d has compute capability %d.%d; the library runs on 10.3 (sm_103)",
               dev, major, minor);
    } else {
      cudaFuncAttributes attr;
      e = cudaFuncGetAttributes(&attr, probe_kernel);
      if (e != cudaSuccess) {
        cudaGetLastError();
        d.rc = MX_ERR_NOT_COMPILED;
        snprintf(d.why, sizeof d.why, "no sm_103a kernel image usable on device %d: %s", dev,
                 cudaGetErrorString(e));
      }
    }
    d.checked = true;
  }
  if (d.rc != MX_OK) return fail(d.rc, "%s", d.why);
  const CUcontext ctx = current_context();
  if (ctx == nullptr || ctx != d.ctx || d.status == nullptr) {
    void *p = nullptr, *w = nullptr;
    cudaError_t e = cudaGetSymbolAddress(&p, g_status_word);
    if (e != cudaSuccess) return fail_cuda("device address of the status word", e);
    e = mx::static_workspace_symbol(&w);
    if (e != cudaSuccess) return fail_cuda("device address of the static split-K array", e);
    d.status = static_cast<uint32_t *>(p);
    d.static_ws = w;
    d.ctx = current_context();  // made current by the lookups if it was not yet
  }
  *out = &d;
  return MX_OK;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int block_of(int format) { return format == MX_FMT_MXFP4 ? 32 : 16; }

bool valid_format(int f) { return f == MX_FMT_MXFP4 || f == MX_FMT_NVFP4; }

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess) {
      fn = reinterpret_cast<EncodeTiledFn>(p);
    }
  });
  return fn;
}

// Tensor map over packed FP4 codes [rows, k/2] bytes: boxes of 128 bytes
// (256 codes along K) x box_rows rows, 128-byte swizzle, zero fill past the
// last row.
int encode_codes_map(CUtensorMap *tm, const void *base, int64_t rows, int64_t k, int box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return MX_ERR_CUDA;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(k / 2), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(k / 2)};
  const cuuint32_t box[2] = {128u, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1u, 1u};
  const CUresult r = fn(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MX_OK : MX_ERR_CUDA;
}

// Tensor map over the output (or the split-K partials [splits * M, N]):
// boxes of 32 rows x 64 bytes, 64-byte swizzle.
int encode_out_map(CUtensorMap *tm, void *base, int64_t rows, int64_t cols, bool f32,
                   int box_cols) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return MX_ERR_CUDA;
  const int esize = f32 ? 4 : 2;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols * esize)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), 32u};
  const cuuint32_t estr[2] = {1u, 1u};
  const CUresult r = fn(tm, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                        2, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MX_OK : MX_ERR_CUDA;
}

// Tensor map over a tile-ordered scale buffer viewed as [atoms, 512 bytes]
// (32-bit elements, one 512-byte row per 128x4 atom): boxes of box_atoms
// rows, zero past the end.
int encode_scale_map(CUtensorMap *tm, const void *base, size_t bytes, int box_atoms) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return MX_ERR_CUDA;
  const cuuint64_t dims[2] = {128u, static_cast<cuuint64_t>(bytes / 512)};
  const cuuint64_t strides[1] = {512u};
  const cuuint32_t box[2] = {128u, static_cast<cuuint32_t>(box_atoms)};
  const cuuint32_t estr[2] = {1u, 1u};
  const CUresult r = fn(tm, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void *>(base), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MX_OK : MX_ERR_CUDA;
}

int launch_rc(const char *fn, cudaError_t e) {
  return e == cudaSuccess ? MX_OK : fail_cuda(fn, e);
}

int num_sms_or_default() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) == cudaSuccess &&
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && sms > 0)
    return sms;
  cudaGetLastError();
  return 152;
}

// Byte range [lo, hi) of a buffer, for the checks that inputs and outputs
// written concurrently do not overlap.
struct Range {
  uintptr_t lo, hi;
};

bool overlap(const Range &p, const Range &q) { return p.lo < q.hi && q.lo < p.hi; }

// Every check of a GEMM call's own arguments (no device, no workspace).
int gemm_check_args(const char *fn, int fmt, const void *a_codes, const void *a_scales,
                    const void *b_codes, const void *b_scales, const float *a_ts,
                    const float *b_ts, const void *d, int64_t m, int64_t n, int64_t k, int layout,
                    int out_dtype, int split_k, const mx_gemm_epilogue *epi) {
  if (!a_codes || !a_scales || !b_codes || !b_scales || !d)
    return fail(MX_ERR_INVALID_ARG, "%s: %s is null", fn,
                !a_codes ? "a_codes" : !a_scales ? "a_scales" : !b_codes ? "b_codes"
                : !b_scales ? "b_scales" : "d");
  if (epi && epi->gelu != 0 && epi->gelu != 1)
    return fail(MX_ERR_INVALID_ARG, "%s: epilogue gelu = %d (0 or 1)", fn, epi->gelu);
  if (epi && epi->bias && !aligned16(epi->bias))
    return fail(MX_ERR_ALIGNMENT, "%s: bias %p is not 16-byte aligned", fn,
                static_cast<const void *>(epi->bias));
  if (fmt == MX_FMT_NVFP4 && (!a_ts || !b_ts))
    return fail(MX_ERR_INVALID_ARG, "%s: %s is null (NVFP4 needs both tensor scales)", fn,
                !a_ts ? "a_tensor_scale" : "b_tensor_scale");
  if (split_k < 0) return fail(MX_ERR_INVALID_ARG, "%s: split_k = %d (0 = auto, or >= 1)", fn, split_k);
  if (layout != MX_LAYOUT_TN)
    return fail(MX_ERR_UNSUPPORTED_FEATURE, "%s: layout %d (only MX_LAYOUT_TN = 0)", fn, layout);
  if (out_dtype != MX_OUT_BF16 && out_dtype != MX_OUT_FP32)
    return fail(MX_ERR_UNSUPPORTED_FEATURE, "%s: out_dtype %d (MX_OUT_BF16 = 0 or MX_OUT_FP32 = 1)",
                fn, out_dtype);
  if (m <= 0 || n <= 0 || k <= 0)
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: M, N, K = %lld, %lld, %lld (all must be positive)",
                fn, static_cast<long long>(m), static_cast<long long>(n), static_cast<long long>(k));
  if (k % 256 != 0)
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: K = %lld is not a multiple of 256", fn,
                static_cast<long long>(k));
  if (m % 32 != 0 || n % 32 != 0)
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: %s = %lld is not a multiple of 32", fn,
                m % 32 ? "M" : "N", static_cast<long long>(m % 32 ? m : n));
  if (m >= (int64_t(1) << 31) || n >= (int64_t(1) << 31) || k >= (int64_t(1) << 31))
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: M, N and K must each be below 2^31", fn);
  if (!aligned16(a_codes) || !aligned16(b_codes) || !aligned16(a_scales) || !aligned16(b_scales) ||
      !aligned16(d))
    return fail(MX_ERR_ALIGNMENT, "%s: %s is not 16-byte aligned", fn,
                !aligned16(a_codes) ? "a_codes" : !aligned16(b_codes) ? "b_codes"
                : !aligned16(a_scales) ? "a_scales" : !aligned16(b_scales) ? "b_scales" : "d");
  if (fmt == MX_FMT_NVFP4 &&
      ((reinterpret_cast<uintptr_t>(a_ts) & 3u) || (reinterpret_cast<uintptr_t>(b_ts) & 3u)))
    return fail(MX_ERR_ALIGNMENT, "%s: a tensor scale pointer is not 4-byte aligned", fn);
  if (epi && epi->bias) {
    // the bias is read while D is written
    const size_t d_bytes = static_cast<size_t>(m) * static_cast<size_t>(n) *
                           (out_dtype == MX_OUT_FP32 ? 4u : 2u);
    const Range d_range{reinterpret_cast<uintptr_t>(d), reinterpret_cast<uintptr_t>(d) + d_bytes};
    const uintptr_t bb = reinterpret_cast<uintptr_t>(epi->bias);
    if (overlap(Range{bb, bb + static_cast<uintptr_t>(n) * sizeof(float)}, d_range))
      return fail(MX_ERR_INVALID_ARG, "%s: the bias overlaps D", fn);
  }
  return MX_OK;
}

int gemm_common(const char *fn, int fmt, const void *a_codes, const void *a_scales,
                const void *b_codes, const void *b_scales, const float *a_ts, const float *b_ts,
                void *d, int64_t m, int64_t n, int64_t k, int layout, int out_dtype, int split_k,
                const mx_gemm_epilogue *epi, void *workspace, size_t workspace_bytes,
                void *stream) {
  const int arc = gemm_check_args(fn, fmt, a_codes, a_scales, b_codes, b_scales, a_ts, b_ts, d, m,
                                  n, k, layout, out_dtype, split_k, epi);
  if (arc != MX_OK) return arc;
  DeviceInfo *dev = nullptr;
  const int drc = device_info(&dev);
  if (drc != MX_OK) return drc;
  const mx::GemmPlan plan = mx::gemm_plan(m, n, k, split_k, dev->num_sms);
  const int bn = plan.bn, splits = plan.splits;
  const bool pair = plan.kind == mx::kGemmPair, swap = plan.kind == mx::kGemmSwap;
  const size_t d_bytes = static_cast<size_t>(m) * static_cast<size_t>(n) *
                         (out_dtype == MX_OUT_FP32 ? 4u : 2u);
  const Range d_range{reinterpret_cast<uintptr_t>(d), reinterpret_cast<uintptr_t>(d) + d_bytes};
  if (plan.workspace()) {
    const size_t need = static_cast<size_t>(splits) * static_cast<size_t>(m) *
                        static_cast<size_t>(n) * sizeof(float);
    if (!workspace || workspace_bytes < need)
      return fail(MX_ERR_WORKSPACE, "%s: %d splits of K need a workspace of %zu bytes, got %zu%s",
                  fn, splits, need, workspace ? workspace_bytes : size_t(0),
                  workspace ? "" : " (null)");
    if (!aligned16(workspace))
      return fail(MX_ERR_ALIGNMENT, "%s: workspace is not 16-byte aligned", fn);
    const uintptr_t w = reinterpret_cast<uintptr_t>(workspace);
    if (overlap(Range{w, w + need}, d_range))
      return fail(MX_ERR_INVALID_ARG, "%s: the workspace overlaps D", fn);
  }
  CUtensorMap tma, tmb, tmd, tmsa, tmsb;
  // the single-CTA and swapped kernels (M <= 128) load the M rows of A, the
  // pair kernel 128 per CTA
  if (encode_codes_map(&tma, a_codes, m, k, pair ? 128 : static_cast<int>(m)) != MX_OK)
    return fail(MX_ERR_CUDA, "%s: tensor map of A could not be encoded", fn);
  // the pair kernel stages half of each 256-row B tile per CTA, the swapped
  // kernel its 128, 64 or 32 rows of B (plan.bn)
  if (encode_codes_map(&tmb, b_codes, n, k, pair ? 128 : bn) != MX_OK)
    return fail(MX_ERR_CUDA, "%s: tensor map of B could not be encoded", fn);
  if (pair) {
    const int atoms_per_stage = fmt == MX_FMT_MXFP4 ? 2 : 4;
    if (encode_scale_map(&tmsa, a_scales, mx_scale_bytes(m, k, fmt, MX_SCALE_TCGEN05),
                         atoms_per_stage) != MX_OK ||
        encode_scale_map(&tmsb, b_scales, mx_scale_bytes(n, k, fmt, MX_SCALE_TCGEN05),
                         atoms_per_stage) != MX_OK)
      return fail(MX_ERR_CUDA, "%s: tensor map of the scales could not be encoded", fn);
  }
  const int box_cols = mx::gemm_out_box_cols(out_dtype == MX_OUT_FP32, plan.workspace() ? splits : 1);
  // (the swapped kernel writes D with plain stores: no output map)
  const int orc = swap ? MX_OK
                  : plan.workspace()
                      ? encode_out_map(&tmd, workspace, static_cast<int64_t>(splits) * m, n, true,
                                       box_cols)
                      : encode_out_map(&tmd, d, m, n, out_dtype == MX_OUT_FP32, box_cols);
  if (orc != MX_OK) return fail(MX_ERR_CUDA, "%s: tensor map of the output could not be encoded", fn);
  mx::GemmArgs g{};
  g.fmt = fmt;
  g.tmap_a = &tma;
  g.tmap_b = &tmb;
  g.tmap_d = &tmd;
  g.tmap_sfa = pair ? &tmsa : nullptr;
  g.tmap_sfb = pair ? &tmsb : nullptr;
  g.pair = pair ? 1 : 0;
  g.swap = swap ? 1 : 0;
  g.a_scales = a_scales;
  g.b_scales = b_scales;
  g.a_ts = a_ts;
  g.b_ts = b_ts;
  g.d = d;
  g.out_fp32 = out_dtype == MX_OUT_FP32;
  g.m = m;
  g.n = n;
  g.k = k;
  g.split_k = splits;
  g.bn = bn;
  g.workspace = static_cast<float *>(workspace);
  g.status = dev->status;
  g.num_sms = dev->num_sms;
  if (epi) {
    g.epi.bias = epi->bias;
    g.epi.gelu = epi->gelu;
    g.epi.beta = epi->beta;
    g.epi.c = epi->beta != 0.0f ? d : nullptr;  // beta == 0: D stays write-only
  }
  g.epi.c_elems = m * n;
  g.epi.bias_elems = n;
  g.epi.status = dev->status;
  return launch_rc(fn, mx::launch_gemm(g, static_cast<cudaStream_t>(stream)));
}

}  // namespace

MX_API const char *mx_error_string(int code) {
  switch (code) {
    case MX_OK: return "success";
    case MX_ERR_INVALID_ARG: return "invalid argument (null pointer, bad enum or leading dim)";
    case MX_ERR_NOT_COMPILED: return "library built without sm_103a kernels";
    case MX_ERR_UNSUPPORTED_ARCH: return "current device is not an sm_103 GPU";
    case MX_ERR_UNSUPPORTED_SHAPE: return "unsupported shape (K % 256, M % 32, N % 32, block size)";
    case MX_ERR_UNSUPPORTED_FEATURE: return "unsupported feature (layout or output dtype)";
    case MX_ERR_ALIGNMENT: return "pointer or leading dimension not 16-byte aligned";
    case MX_ERR_WORKSPACE: return "workspace missing or too small";
    case MX_ERR_CUDA: return "CUDA runtime, driver or launch error";
    case MX_ERR_DEVICE_TIMEOUT: return "a bounded device-side wait ran out";
    case MX_ERR_DEVICE_BOUNDS: return "bounds-checked build: a kernel access outside its buffer";
    case MX_ERR_DEVICE_INDEX: return "a page, length or row number in device memory is out of range";
    default: return "unknown status code";
  }
}

MX_API const char *mx_last_error_string(void) {
  return t_detail[0] != '\0' ? t_detail : "no error recorded by the last call on this thread";
}

MX_API int mx_build_flags(void) {
#ifdef MX_BOUNDS_CHECK
  return MX_BUILD_BOUNDS_CHECK;
#else
  return 0;
#endif
}

MX_API int mx_available(void) {
  clear_detail();
  DeviceInfo *d = nullptr;
  const int rc = device_info(&d);
  if (rc == MX_ERR_CUDA) cudaGetLastError();
  return rc == MX_OK ? 1 : 0;
}

MX_API size_t mx_scale_bytes(int64_t rows, int64_t cols, int format, int scale_layout) {
  if (rows <= 0 || cols <= 0 || !valid_format(format)) return 0;
  const int blk = block_of(format);
  if (cols % blk != 0) return 0;
  const int64_t kb = cols / blk;
  if (scale_layout == MX_SCALE_PLAIN) return static_cast<size_t>(rows * kb);
  if (scale_layout == MX_SCALE_TCGEN05)
    return static_cast<size_t>((rows + 127) / 128 * 128 * ((kb + 3) / 4 * 4));
  return 0;
}

MX_API size_t mx_quantize_workspace_bytes(int64_t rows, int64_t cols, int format) {
  (void)rows;
  (void)cols;
  return format == MX_FMT_NVFP4 ? static_cast<size_t>(mx::kAmaxPartials) * sizeof(uint32_t) : 0;
}

namespace {

const char *fmt_name(int format) { return format == MX_FMT_MXFP4 ? "MXFP4" : "NVFP4"; }

// Checks one tensor of a quantize call (everything but the workspace) and
// fills its launch arguments.
int quantize_tensor_args(const char *fn, const void *x, int64_t rows, int64_t cols, int64_t ld_x,
                         int format, int scale_layout, void *codes, void *scales,
                         float *tensor_scale, mx::QuantizeArgs *a) {
  if (!x || !codes || !scales)
    return fail(MX_ERR_INVALID_ARG, "%s: %s is null", fn, !x ? "x" : !codes ? "codes" : "scales");
  if (!valid_format(format))
    return fail(MX_ERR_INVALID_ARG, "%s: format %d (MX_FMT_MXFP4 = 0 or MX_FMT_NVFP4 = 1)", fn,
                format);
  if (scale_layout != MX_SCALE_PLAIN && scale_layout != MX_SCALE_TCGEN05)
    return fail(MX_ERR_INVALID_ARG, "%s: scale_layout %d (MX_SCALE_PLAIN = 0 or MX_SCALE_TCGEN05 = 1)",
                fn, scale_layout);
  if (rows <= 0 || cols <= 0 || ld_x < cols)
    return fail(MX_ERR_INVALID_ARG, "%s: rows, cols, ld_x = %lld, %lld, %lld (positive, ld_x >= cols)",
                fn, static_cast<long long>(rows), static_cast<long long>(cols),
                static_cast<long long>(ld_x));
  if (format == MX_FMT_MXFP4 && tensor_scale != nullptr)
    return fail(MX_ERR_INVALID_ARG, "%s: tensor_scale must be null for MXFP4", fn);
  if (format == MX_FMT_NVFP4 && tensor_scale == nullptr)
    return fail(MX_ERR_INVALID_ARG, "%s: tensor_scale is null (NVFP4 writes s_t there)", fn);
  if (cols % block_of(format) != 0)
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: cols = %lld is not a multiple of the %s block %d", fn,
                static_cast<long long>(cols), fmt_name(format), block_of(format));
  if (rows >= (int64_t(1) << 31) || cols >= (int64_t(1) << 31))
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: rows and cols must each be below 2^31", fn);
  // the kernels index scale blocks of the (row-padded) tensor with 32 bits
  if ((rows + 127) / 128 * 128 * (cols / block_of(format)) >= (int64_t(1) << 31))
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: %lld x %lld has 2^31 or more scale blocks", fn,
                static_cast<long long>(rows), static_cast<long long>(cols));
  if (!aligned16(x) || (ld_x % 8) != 0 || !aligned16(codes) || !aligned16(scales))
    return fail(MX_ERR_ALIGNMENT, "%s: %s", fn,
                !aligned16(x) ? "x is not 16-byte aligned"
                : (ld_x % 8) ? "ld_x is not a multiple of 8 elements (16 bytes)"
                : !aligned16(codes) ? "codes is not 16-byte aligned" : "scales is not 16-byte aligned");
  if (format == MX_FMT_NVFP4 && (reinterpret_cast<uintptr_t>(tensor_scale) & 3u) != 0)
    return fail(MX_ERR_ALIGNMENT, "%s: tensor_scale is not 4-byte aligned", fn);
  *a = mx::QuantizeArgs{};
  a->x = x;
  a->rows = rows;
  a->cols = cols;
  a->ld = ld_x;
  a->tiled = scale_layout == MX_SCALE_TCGEN05;
  a->codes = codes;
  a->scales = scales;
  a->tensor_scale = tensor_scale;
  return MX_OK;
}

int check_amax_workspace(const char *fn, const void *workspace, size_t workspace_bytes,
                         size_t need) {
  if (!workspace || workspace_bytes < need)
    return fail(MX_ERR_WORKSPACE, "%s: NVFP4 needs a workspace of %zu bytes, got %zu%s", fn, need,
                workspace ? workspace_bytes : size_t(0), workspace ? "" : " (null)");
  if (!aligned16(workspace)) return fail(MX_ERR_ALIGNMENT, "%s: workspace is not 16-byte aligned", fn);
  return MX_OK;
}

}  // namespace

MX_API int mx_quantize_bf16(const void *x, int64_t rows, int64_t cols, int64_t ld_x, int format,
                            int scale_layout, void *codes, void *scales, float *tensor_scale,
                            void *workspace, size_t workspace_bytes, void *stream) {
  clear_detail();
  const char *fn = "mx_quantize_bf16";
  mx::QuantizeArgs a;
  int rc = quantize_tensor_args(fn, x, rows, cols, ld_x, format, scale_layout, codes, scales,
                                tensor_scale, &a);
  if (rc != MX_OK) return rc;
  if (format == MX_FMT_NVFP4) {
    rc = check_amax_workspace(fn, workspace, workspace_bytes,
                              mx_quantize_workspace_bytes(rows, cols, format));
    if (rc != MX_OK) return rc;
    a.partials = static_cast<uint32_t *>(workspace);
  }
  DeviceInfo *dev = nullptr;
  rc = device_info(&dev);
  if (rc != MX_OK) return rc;
  a.num_sms = dev->num_sms;
  a.status = dev->status;
  return launch_rc(fn, mx::launch_quantize_group(format == MX_FMT_MXFP4 ? 0 : 1, &a, 1,
                                                 static_cast<cudaStream_t>(stream)));
}

static_assert(MX_PHILOX_MAX_ROUNDS == mx::kPhiloxMaxRounds, "Philox round limit");

MX_API int nvfp4_quantize_bf16_sr(const void *x, int64_t rows, int64_t cols, int64_t ld_x,
                                  int scale_layout, void *codes, void *scales,
                                  float *tensor_scale, uint64_t seed, int philox_rounds,
                                  void *workspace, size_t workspace_bytes, void *stream) {
  clear_detail();
  const char *fn = "nvfp4_quantize_bf16_sr";
  if (philox_rounds < 1 || philox_rounds > MX_PHILOX_MAX_ROUNDS)
    return fail(MX_ERR_INVALID_ARG, "%s: philox_rounds = %d (1..%d)", fn, philox_rounds,
                MX_PHILOX_MAX_ROUNDS);
  mx::QuantizeArgs a;
  int rc = quantize_tensor_args(fn, x, rows, cols, ld_x, MX_FMT_NVFP4, scale_layout, codes, scales,
                                tensor_scale, &a);
  if (rc != MX_OK) return rc;
  rc = check_amax_workspace(fn, workspace, workspace_bytes,
                            mx_quantize_workspace_bytes(rows, cols, MX_FMT_NVFP4));
  if (rc != MX_OK) return rc;
  a.partials = static_cast<uint32_t *>(workspace);
  DeviceInfo *dev = nullptr;
  rc = device_info(&dev);
  if (rc != MX_OK) return rc;
  a.num_sms = dev->num_sms;
  a.status = dev->status;
  const mx::SrArgs sr{seed, philox_rounds, 0u};
  return launch_rc(fn, mx::launch_quantize_group(1, &a, 1, static_cast<cudaStream_t>(stream), &sr));
}

MX_API size_t mx_quantize_group_workspace_bytes(int count, int format) {
  if (count < 1 || count > MX_QUANTIZE_GROUP_MAX || !valid_format(format)) return 0;
  return static_cast<size_t>(count) * mx_quantize_workspace_bytes(1, block_of(format), format);
}

MX_API int mx_quantize_bf16_group(const mx_quantize_tensor *tensors, int count, int format,
                                  int scale_layout, void *workspace, size_t workspace_bytes,
                                  void *stream) {
  clear_detail();
  const char *fn = "mx_quantize_bf16_group";
  static_assert(MX_QUANTIZE_GROUP_MAX == mx::kQuantizeGroupMax, "group size");
  if (!tensors || count < 1 || count > MX_QUANTIZE_GROUP_MAX)
    return fail(MX_ERR_INVALID_ARG, "%s: %s", fn,
                !tensors ? "tensors is null" : "count must be in 1..MX_QUANTIZE_GROUP_MAX (8)");
  mx::QuantizeArgs a[MX_QUANTIZE_GROUP_MAX];
  Range in[MX_QUANTIZE_GROUP_MAX], out[3 * MX_QUANTIZE_GROUP_MAX];
  int nout = 0;
  for (int i = 0; i < count; ++i) {
    const mx_quantize_tensor &t = tensors[i];
    char who[48];
    snprintf(who, sizeof who, "%s (tensor %d)", fn, i);
    const int rc = quantize_tensor_args(who, t.x, t.rows, t.cols, t.ld_x, format, scale_layout,
                                        t.codes, t.scales, t.tensor_scale, &a[i]);
    if (rc != MX_OK) return rc;
    const uintptr_t x = reinterpret_cast<uintptr_t>(t.x);
    in[i] = Range{x, x + static_cast<uintptr_t>(((t.rows - 1) * t.ld_x + t.cols) * 2)};
    const uintptr_t c = reinterpret_cast<uintptr_t>(t.codes);
    out[nout++] = Range{c, c + static_cast<uintptr_t>(t.rows * t.cols / 2)};
    const uintptr_t sc = reinterpret_cast<uintptr_t>(t.scales);
    out[nout++] = Range{sc, sc + mx_scale_bytes(t.rows, t.cols, format, scale_layout)};
    if (t.tensor_scale) {
      const uintptr_t ts = reinterpret_cast<uintptr_t>(t.tensor_scale);
      out[nout++] = Range{ts, ts + sizeof(float)};
    }
  }
  // The tensors are quantized concurrently: no output may overlap an input
  // or another output.
  for (int o = 0; o < nout; ++o) {
    for (int i = 0; i < count; ++i)
      if (overlap(out[o], in[i]))
        return fail(MX_ERR_INVALID_ARG, "%s: an output overlaps the input of tensor %d", fn, i);
    for (int p = o + 1; p < nout; ++p)
      if (overlap(out[o], out[p])) return fail(MX_ERR_INVALID_ARG, "%s: two outputs overlap", fn);
  }
  if (format == MX_FMT_NVFP4) {
    const int rc = check_amax_workspace(fn, workspace, workspace_bytes,
                                        mx_quantize_group_workspace_bytes(count, format));
    if (rc != MX_OK) return rc;
    const Range ws{reinterpret_cast<uintptr_t>(workspace),
                   reinterpret_cast<uintptr_t>(workspace) +
                       mx_quantize_group_workspace_bytes(count, format)};
    for (int o = 0; o < nout; ++o)
      if (overlap(ws, out[o])) return fail(MX_ERR_INVALID_ARG, "%s: the workspace overlaps an output", fn);
    for (int i = 0; i < count; ++i) {
      if (overlap(ws, in[i])) return fail(MX_ERR_INVALID_ARG, "%s: the workspace overlaps an input", fn);
      a[i].partials = static_cast<uint32_t *>(workspace) + static_cast<size_t>(i) * mx::kAmaxPartials;
    }
  }
  DeviceInfo *dev = nullptr;
  const int rc = device_info(&dev);
  if (rc != MX_OK) return rc;
  for (int i = 0; i < count; ++i) {
    a[i].num_sms = dev->num_sms;
    a[i].status = dev->status;
  }
  return launch_rc(fn, mx::launch_quantize_group(format == MX_FMT_MXFP4 ? 0 : 1, a, count,
                                                 static_cast<cudaStream_t>(stream)));
}

namespace {

// Shared checks of the two bidimensional quantizers, in two phases: the
// arguments themselves (pointers, enum, sizes), then the shape limits of the
// format and the alignments.
int quantize_2d_basic(const char *fn, const void *x, int64_t rows, int64_t cols, int64_t ld_x,
                      int scale_layout, const void *codes, const void *scales,
                      const void *codes_t, const void *scales_t) {
  // codes and scales may both be null (columnwise output only)
  const bool rowwise = codes != nullptr || scales != nullptr;
  if (!x || !codes_t || !scales_t || (rowwise && (!codes || !scales)))
    return fail(MX_ERR_INVALID_ARG, "%s: %s", fn,
                !x ? "x is null" : !codes_t ? "codes_t is null" : !scales_t ? "scales_t is null"
                : "codes and scales must both be set or both be null");
  if (scale_layout != MX_SCALE_PLAIN && scale_layout != MX_SCALE_TCGEN05)
    return fail(MX_ERR_INVALID_ARG, "%s: scale_layout %d (MX_SCALE_PLAIN = 0 or MX_SCALE_TCGEN05 = 1)",
                fn, scale_layout);
  if (rows <= 0 || cols <= 0 || ld_x < cols)
    return fail(MX_ERR_INVALID_ARG, "%s: rows, cols, ld_x = %lld, %lld, %lld (positive, ld_x >= cols)",
                fn, static_cast<long long>(rows), static_cast<long long>(cols),
                static_cast<long long>(ld_x));
  return MX_OK;
}

int quantize_2d_shape(const char *fn, int format, const void *x, int64_t rows, int64_t cols,
                      int64_t ld_x, const void *codes, const void *scales, const void *codes_t,
                      const void *scales_t) {
  const int blk = block_of(format);
  if (rows % blk != 0 || cols % blk != 0)
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: %s = %lld is not a multiple of the %s block %d", fn,
                rows % blk ? "rows" : "cols", static_cast<long long>(rows % blk ? rows : cols),
                fmt_name(format), blk);
  if (rows >= (int64_t(1) << 31) || cols >= (int64_t(1) << 31))
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: rows and cols must each be below 2^31", fn);
  if ((rows + 127) / 128 * 128 * (cols / blk) >= (int64_t(1) << 31) ||
      (cols + 127) / 128 * 128 * (rows / blk) >= (int64_t(1) << 31))
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: %lld x %lld has 2^31 or more scale blocks", fn,
                static_cast<long long>(rows), static_cast<long long>(cols));
  if (!aligned16(x) || (ld_x % 8) != 0 || !aligned16(codes) || !aligned16(scales) ||
      !aligned16(codes_t) || !aligned16(scales_t))  // (a null pointer is aligned)
    return fail(MX_ERR_ALIGNMENT, "%s: %s", fn,
                !aligned16(x) ? "x is not 16-byte aligned"
                : (ld_x % 8) ? "ld_x is not a multiple of 8 elements (16 bytes)"
                : "an output pointer is not 16-byte aligned");
  return MX_OK;
}

}  // namespace

MX_API int mx_quantize_bf16_2d(const void *x, int64_t rows, int64_t cols, int64_t ld_x,
                               int format, int scale_layout, void *codes, void *scales,
                               void *codes_t, void *scales_t, void *stream) {
  clear_detail();
  const char *fn = "mx_quantize_bf16_2d";
  int rc = quantize_2d_basic(fn, x, rows, cols, ld_x, scale_layout, codes, scales, codes_t,
                             scales_t);
  if (rc != MX_OK) return rc;
  if (!valid_format(format))
    return fail(MX_ERR_INVALID_ARG, "%s: format %d (MX_FMT_MXFP4 = 0 or MX_FMT_NVFP4 = 1)", fn,
                format);
  if (format != MX_FMT_MXFP4)
    return fail(MX_ERR_UNSUPPORTED_FEATURE, "%s: NVFP4 takes nvfp4_quantize_bf16_2d", fn);
  rc = quantize_2d_shape(fn, format, x, rows, cols, ld_x, codes, scales, codes_t, scales_t);
  if (rc != MX_OK) return rc;
  const bool rowwise = codes != nullptr || scales != nullptr;
  // The two outputs are written concurrently from the same input: no output
  // may overlap the input or another output.
  const uintptr_t xb = reinterpret_cast<uintptr_t>(x);
  const Range in{xb, xb + static_cast<uintptr_t>(((rows - 1) * ld_x + cols) * 2)};
  const Range out[4] = {
      {reinterpret_cast<uintptr_t>(codes), reinterpret_cast<uintptr_t>(codes) + static_cast<uintptr_t>(rows * cols / 2)},
      {reinterpret_cast<uintptr_t>(scales), reinterpret_cast<uintptr_t>(scales) + mx_scale_bytes(rows, cols, format, scale_layout)},
      {reinterpret_cast<uintptr_t>(codes_t), reinterpret_cast<uintptr_t>(codes_t) + static_cast<uintptr_t>(rows * cols / 2)},
      {reinterpret_cast<uintptr_t>(scales_t), reinterpret_cast<uintptr_t>(scales_t) + mx_scale_bytes(cols, rows, format, scale_layout)}};
  for (int o = rowwise ? 0 : 2; o < 4; ++o) {
    if (overlap(out[o], in)) return fail(MX_ERR_INVALID_ARG, "%s: an output overlaps x", fn);
    for (int p = o + 1; p < 4; ++p)
      if (overlap(out[o], out[p])) return fail(MX_ERR_INVALID_ARG, "%s: two outputs overlap", fn);
  }
  DeviceInfo *dev = nullptr;
  rc = device_info(&dev);
  if (rc != MX_OK) return rc;
  return launch_rc(fn, mx::launch_mx_quantize_2d(x, rows, cols, ld_x,
                                                 scale_layout == MX_SCALE_TCGEN05, codes, scales,
                                                 codes_t, scales_t, dev->status,
                                                 static_cast<cudaStream_t>(stream)));
}

MX_API int nvfp4_quantize_bf16_2d(const void *x, int64_t rows, int64_t cols, int64_t ld_x,
                                  int scale_layout, void *codes, void *scales, void *codes_t,
                                  void *scales_t, float *tensor_scale, int stochastic,
                                  uint64_t seed, int philox_rounds, void *workspace,
                                  size_t workspace_bytes, void *stream) {
  clear_detail();
  const char *fn = "nvfp4_quantize_bf16_2d";
  const int fmt = MX_FMT_NVFP4;
  if (!tensor_scale) return fail(MX_ERR_INVALID_ARG, "%s: tensor_scale is null", fn);
  if (stochastic != 0 && stochastic != 1)
    return fail(MX_ERR_INVALID_ARG, "%s: stochastic = %d (0 or 1)", fn, stochastic);
  if (stochastic && (philox_rounds < 1 || philox_rounds > MX_PHILOX_MAX_ROUNDS))
    return fail(MX_ERR_INVALID_ARG, "%s: philox_rounds = %d (1..%d)", fn, philox_rounds,
                MX_PHILOX_MAX_ROUNDS);
  int rc = quantize_2d_basic(fn, x, rows, cols, ld_x, scale_layout, codes, scales, codes_t,
                             scales_t);
  if (rc == MX_OK)
    rc = quantize_2d_shape(fn, fmt, x, rows, cols, ld_x, codes, scales, codes_t, scales_t);
  if (rc != MX_OK) return rc;
  if ((reinterpret_cast<uintptr_t>(tensor_scale) & 3u) != 0)
    return fail(MX_ERR_ALIGNMENT, "%s: tensor_scale is not 4-byte aligned", fn);
  rc = check_amax_workspace(fn, workspace, workspace_bytes,
                            mx_quantize_workspace_bytes(rows, cols, fmt));
  if (rc != MX_OK) return rc;
  const bool rowwise = codes != nullptr || scales != nullptr;
  // Both outputs are written concurrently from the same input: no output may
  // overlap the input, the workspace or another output.
  const uintptr_t xb = reinterpret_cast<uintptr_t>(x);
  const Range in{xb, xb + static_cast<uintptr_t>(((rows - 1) * ld_x + cols) * 2)};
  const uintptr_t wsb = reinterpret_cast<uintptr_t>(workspace);
  const Range out[6] = {
      {reinterpret_cast<uintptr_t>(codes), reinterpret_cast<uintptr_t>(codes) + static_cast<uintptr_t>(rows * cols / 2)},
      {reinterpret_cast<uintptr_t>(scales), reinterpret_cast<uintptr_t>(scales) + mx_scale_bytes(rows, cols, fmt, scale_layout)},
      {reinterpret_cast<uintptr_t>(codes_t), reinterpret_cast<uintptr_t>(codes_t) + static_cast<uintptr_t>(rows * cols / 2)},
      {reinterpret_cast<uintptr_t>(scales_t), reinterpret_cast<uintptr_t>(scales_t) + mx_scale_bytes(cols, rows, fmt, scale_layout)},
      {reinterpret_cast<uintptr_t>(tensor_scale), reinterpret_cast<uintptr_t>(tensor_scale) + sizeof(float)},
      {wsb, wsb + mx_quantize_workspace_bytes(rows, cols, fmt)}};
  for (int o = rowwise ? 0 : 2; o < 6; ++o) {
    if (overlap(out[o], in)) return fail(MX_ERR_INVALID_ARG, "%s: an output overlaps x", fn);
    for (int p = o + 1; p < 6; ++p)
      if (overlap(out[o], out[p]))
        return fail(MX_ERR_INVALID_ARG, "%s: two outputs (or an output and the workspace) overlap",
                    fn);
  }
  DeviceInfo *dev = nullptr;
  rc = device_info(&dev);
  if (rc != MX_OK) return rc;
  const mx::SrArgs sr{seed, philox_rounds, 0u};
  return launch_rc(fn, mx::launch_nvfp4_quantize_2d(
      x, rows, cols, ld_x, scale_layout == MX_SCALE_TCGEN05, codes, scales, codes_t, scales_t,
      tensor_scale, static_cast<uint32_t *>(workspace), stochastic ? &sr : nullptr, dev->num_sms,
      dev->status, static_cast<cudaStream_t>(stream)));
}

MX_API int mx_scale_relayout(const void *plain, int64_t rows, int64_t cols, int format,
                             void *tiled, void *stream) {
  clear_detail();
  const char *fn = "mx_scale_relayout";
  if (!plain || !tiled)
    return fail(MX_ERR_INVALID_ARG, "%s: %s is null", fn, !plain ? "plain" : "tiled");
  if (!valid_format(format))
    return fail(MX_ERR_INVALID_ARG, "%s: format %d (MX_FMT_MXFP4 = 0 or MX_FMT_NVFP4 = 1)", fn,
                format);
  if (rows <= 0 || cols <= 0)
    return fail(MX_ERR_INVALID_ARG, "%s: rows, cols = %lld, %lld (both positive)", fn,
                static_cast<long long>(rows), static_cast<long long>(cols));
  if (cols % block_of(format) != 0)
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: cols = %lld is not a multiple of the %s block %d", fn,
                static_cast<long long>(cols), fmt_name(format), block_of(format));
  if (rows >= (int64_t(1) << 31) || cols >= (int64_t(1) << 31))
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: rows and cols must each be below 2^31", fn);
  DeviceInfo *dev = nullptr;
  const int rc = device_info(&dev);
  if (rc != MX_OK) return rc;
  return launch_rc(fn, mx::launch_scale_relayout(plain, rows, cols / block_of(format), tiled,
                                                 dev->status, static_cast<cudaStream_t>(stream)));
}

MX_API int mx_fp4_transpose(const void *codes, int64_t rows, int64_t cols, void *out,
                            void *stream) {
  clear_detail();
  const char *fn = "mx_fp4_transpose";
  if (!codes || !out)
    return fail(MX_ERR_INVALID_ARG, "%s: %s is null", fn, !codes ? "codes" : "out");
  if (rows <= 0 || cols <= 0)
    return fail(MX_ERR_INVALID_ARG, "%s: rows, cols = %lld, %lld (both positive)", fn,
                static_cast<long long>(rows), static_cast<long long>(cols));
  if (rows % 32 != 0 || cols % 32 != 0)
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: rows, cols = %lld, %lld (both multiples of 32)",
                fn, static_cast<long long>(rows), static_cast<long long>(cols));
  if (rows >= (int64_t(1) << 31) || cols >= (int64_t(1) << 31) ||
      (rows + 63) / 64 > 65535)
    return fail(MX_ERR_UNSUPPORTED_SHAPE,
                "%s: cols must be below 2^31 and rows below 64 * 65536", fn);
  if (!aligned16(codes) || !aligned16(out))
    return fail(MX_ERR_ALIGNMENT, "%s: %s is not 16-byte aligned", fn,
                !aligned16(codes) ? "codes" : "out");
  const uintptr_t ci = reinterpret_cast<uintptr_t>(codes), oi = reinterpret_cast<uintptr_t>(out);
  const uintptr_t bytes = static_cast<uintptr_t>(rows) * static_cast<uintptr_t>(cols) / 2;
  if (overlap(Range{ci, ci + bytes}, Range{oi, oi + bytes}))
    return fail(MX_ERR_INVALID_ARG, "%s: out overlaps codes", fn);
  DeviceInfo *dev = nullptr;
  const int rc = device_info(&dev);
  if (rc != MX_OK) return rc;
  return launch_rc(fn, mx::launch_fp4_transpose(codes, rows, cols, out, dev->status,
                                                static_cast<cudaStream_t>(stream)));
}

MX_API size_t mx_gemm_workspace_bytes(int64_t m, int64_t n, int64_t k, int split_k) {
  if (m <= 0 || n <= 0 || k <= 0 || k % 256 != 0 || split_k < 0) return 0;
  const mx::GemmPlan plan = mx::gemm_plan(m, n, k, split_k, num_sms_or_default());
  if (!plan.workspace()) return 0;
  return static_cast<size_t>(plan.splits) * static_cast<size_t>(m) * static_cast<size_t>(n) *
         sizeof(float);
}

MX_API int mxfp4_gemm(const void *a_codes, const void *a_scales, const void *b_codes,
                      const void *b_scales, void *d, int64_t m, int64_t n, int64_t k, int layout,
                      int out_dtype, int split_k, void *workspace, size_t workspace_bytes,
                      void *stream) {
  clear_detail();
  return gemm_common("mxfp4_gemm", MX_FMT_MXFP4, a_codes, a_scales, b_codes, b_scales, nullptr,
                     nullptr, d, m, n, k, layout, out_dtype, split_k, nullptr, workspace,
                     workspace_bytes, stream);
}

MX_API int nvfp4_gemm(const void *a_codes, const void *a_scales, const void *b_codes,
                      const void *b_scales, const float *a_tensor_scale,
                      const float *b_tensor_scale, void *d, int64_t m, int64_t n, int64_t k,
                      int layout, int out_dtype, int split_k, void *workspace,
                      size_t workspace_bytes, void *stream) {
  clear_detail();
  return gemm_common("nvfp4_gemm", MX_FMT_NVFP4, a_codes, a_scales, b_codes, b_scales,
                     a_tensor_scale, b_tensor_scale, d, m, n, k, layout, out_dtype, split_k,
                     nullptr, workspace, workspace_bytes, stream);
}

MX_API int mxfp4_gemm_ex(const void *a_codes, const void *a_scales, const void *b_codes,
                         const void *b_scales, void *d, int64_t m, int64_t n, int64_t k,
                         int layout, int out_dtype, int split_k,
                         const mx_gemm_epilogue *epilogue, void *workspace,
                         size_t workspace_bytes, void *stream) {
  clear_detail();
  return gemm_common("mxfp4_gemm_ex", MX_FMT_MXFP4, a_codes, a_scales, b_codes, b_scales, nullptr,
                     nullptr, d, m, n, k, layout, out_dtype, split_k, epilogue, workspace,
                     workspace_bytes, stream);
}

MX_API int nvfp4_gemm_ex(const void *a_codes, const void *a_scales, const void *b_codes,
                         const void *b_scales, const float *a_tensor_scale,
                         const float *b_tensor_scale, void *d, int64_t m, int64_t n, int64_t k,
                         int layout, int out_dtype, int split_k,
                         const mx_gemm_epilogue *epilogue, void *workspace,
                         size_t workspace_bytes, void *stream) {
  clear_detail();
  return gemm_common("nvfp4_gemm_ex", MX_FMT_NVFP4, a_codes, a_scales, b_codes, b_scales,
                     a_tensor_scale, b_tensor_scale, d, m, n, k, layout, out_dtype, split_k,
                     epilogue, workspace, workspace_bytes, stream);
}

// ---- products of a few tokens

namespace {

Range span(const void *p, uint64_t bytes) {
  const uintptr_t b = reinterpret_cast<uintptr_t>(p);
  return p ? Range{b, b + static_cast<uintptr_t>(bytes)} : Range{0, 0};
}

// Bytes from the first to the last element of `rows` rows.
uint64_t row_bytes(int64_t rows, int64_t cols, int64_t ld, uint64_t elem) {
  return rows <= 0 ? 0 : static_cast<uint64_t>((rows - 1) * ld + cols) * elem;
}

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// x of the few-token calls: BF16 [tokens, k].  `cols` names k in messages.
int few_check_x(const char *fn, const void *x, int64_t tokens, int64_t max_tokens, int64_t k,
                int64_t ld_x, const char *cols) {
  if (!x) return fail(MX_ERR_INVALID_ARG, "%s: x is null", fn);
  if (tokens < 0 || tokens > max_tokens)
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: tokens = %lld (0..%lld)", fn,
                static_cast<long long>(tokens), static_cast<long long>(max_tokens));
  if (k <= 0 || k % 32 != 0 || k >= (int64_t(1) << 31))
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: %s = %lld (a positive multiple of 32 below 2^31)", fn,
                cols, static_cast<long long>(k));
  if (ld_x < k || ld_x >= (int64_t(1) << 40))
    return fail(MX_ERR_INVALID_ARG, "%s: ld_x = %lld (>= %s = %lld, below 2^40)", fn,
                static_cast<long long>(ld_x), cols, static_cast<long long>(k));
  if (!aligned16(x) || ld_x % 8 != 0)
    return fail(MX_ERR_ALIGNMENT, "%s: %s", fn,
                !aligned16(x) ? "x is not 16-byte aligned"
                              : "ld_x is not a multiple of 8 elements (16 bytes)");
  return MX_OK;
}

// Scale blocks of a matrix [rows, k], its rows in whole tiles: 2^31 or more.
bool too_many_blocks(int format, int64_t rows, int64_t k) {
  return (rows + 127) / 128 * 128 * (k / block_of(format)) >= (int64_t(1) << 31);
}

// A stack of `count` FP4 matrices [rows, k] (rows, k already checked).
int few_check_matrix(const char *fn, const char *name, int format, const void *codes,
                     const void *scales, const float *ts, int64_t rows, int64_t k) {
  if (!codes || !scales)
    return fail(MX_ERR_INVALID_ARG, "%s: %s %s is null", fn, name, !codes ? "codes" : "scales");
  if ((format == MX_FMT_NVFP4) != (ts != nullptr))
    return fail(MX_ERR_INVALID_ARG, "%s: %s tensor scale %s", fn, name,
                ts ? "must be null for MXFP4" : "is null (NVFP4 needs it)");
  if (!aligned16(codes) || !aligned16(scales) || !aligned4(ts))
    return fail(MX_ERR_ALIGNMENT, "%s: %s %s", fn, name,
                !aligned16(codes) ? "codes are not 16-byte aligned"
                : !aligned16(scales) ? "scales are not 16-byte aligned"
                                     : "tensor scale is not 4-byte aligned");
  if (too_many_blocks(format, rows, k))
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: %s [%lld, %lld] has 2^31 or more scale blocks", fn,
                name, static_cast<long long>(rows), static_cast<long long>(k));
  return MX_OK;
}

// The ranges of a stack of matrices: codes, scales, tensor scales.
void matrix_ranges(const mx::FewMatrix &m, int format, int64_t count, int64_t rows, int64_t k,
                   Range *out) {
  out[0] = span(m.codes, static_cast<uint64_t>(count) * static_cast<uint64_t>(rows * (k / 2)));
  out[1] = span(m.scales, static_cast<uint64_t>(count) *
                              mx_scale_bytes(rows, k, format, MX_SCALE_TCGEN05));
  out[2] = span(m.ts, static_cast<uint64_t>(count) * sizeof(float));
}

// No output overlaps an input or another output.
int check_disjoint(const char *fn, const Range *out, int nout, const Range *in, int nin) {
  for (int o = 0; o < nout; ++o) {
    for (int i = 0; i < nin; ++i)
      if (overlap(out[o], in[i]))
        return fail(MX_ERR_INVALID_ARG, "%s: an output or the workspace overlaps an input", fn);
    for (int p = o + 1; p < nout; ++p)
      if (overlap(out[o], out[p]))
        return fail(MX_ERR_INVALID_ARG, "%s: two outputs (or an output and the workspace) overlap",
                    fn);
  }
  return MX_OK;
}

static_assert(MX_LINEAR_MAX_TOKENS == mx::kLinearMaxTokens, "few-token limits");
static_assert(MX_MOE_MAX_TOKENS == mx::kMoeMaxTokens && MX_MOE_MAX_EXPERTS == mx::kMoeMaxExperts &&
                  MX_MOE_MAX_TOP_K == mx::kMoeMaxTopK,
              "few-token limits");

constexpr size_t round256(size_t n) { return (n + 255) / 256 * 256; }

size_t moe_h_bytes(int64_t pairs, int64_t inter) {
  return round256(static_cast<size_t>(2 * mx::moe_max_parts(pairs) * pairs) *
                  static_cast<size_t>(inter) * sizeof(float));
}
size_t moe_z_bytes(int64_t pairs, int64_t hidden) {
  return round256(static_cast<size_t>(mx::moe_max_parts(pairs) * pairs) *
                  static_cast<size_t>(hidden) * sizeof(float));
}
size_t moe_images_bytes(int64_t tokens, int64_t hidden, int64_t inter, int top_k) {
  return round256(mx::moe_image_bytes(tokens * top_k, hidden) +
                  mx::moe_image_bytes(tokens * top_k, inter));
}

int route_check(const char *fn, const void *x, int64_t tokens, int64_t hidden, int64_t ld_x,
                const void *router, int64_t experts, const float *bias, int top_k, int normalize,
                const int32_t *ids, const float *weights) {
  const int rc = few_check_x(fn, x, tokens, MX_MOE_MAX_TOKENS, hidden, ld_x, "hidden");
  if (rc != MX_OK) return rc;
  if (!router || !ids || !weights)
    return fail(MX_ERR_INVALID_ARG, "%s: %s is null", fn,
                !router ? "router" : !ids ? "ids" : "weights");
  if (normalize != 0 && normalize != 1)
    return fail(MX_ERR_INVALID_ARG, "%s: normalize = %d (0 or 1)", fn, normalize);
  if (experts < 1 || experts > MX_MOE_MAX_EXPERTS)
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: experts = %lld (1..%d)", fn,
                static_cast<long long>(experts), MX_MOE_MAX_EXPERTS);
  if (top_k < 1 || top_k > MX_MOE_MAX_TOP_K || top_k > experts)
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: top_k = %d (1..%d and at most %lld experts)", fn,
                top_k, MX_MOE_MAX_TOP_K, static_cast<long long>(experts));
  if (!aligned16(router)) return fail(MX_ERR_ALIGNMENT, "%s: router is not 16-byte aligned", fn);
  if (!aligned4(bias) || !aligned4(ids) || !aligned4(weights))
    return fail(MX_ERR_ALIGNMENT, "%s: %s is not 4-byte aligned", fn,
                !aligned4(bias) ? "bias" : !aligned4(ids) ? "ids" : "weights");
  const Range in[3] = {span(x, row_bytes(tokens, hidden, ld_x, 2)),
                       span(router, static_cast<uint64_t>(experts * hidden) * 2),
                       span(bias, static_cast<uint64_t>(experts) * 4)};
  const uint64_t slots = static_cast<uint64_t>(tokens) * static_cast<uint64_t>(top_k) * 4;
  const Range out[2] = {span(ids, slots), span(weights, slots)};
  return check_disjoint(fn, out, 2, in, 3);
}

mx::FewMatrix few_matrix(const mx_moe_matrix &m) {
  return mx::FewMatrix{static_cast<const uint8_t *>(m.codes), static_cast<const uint8_t *>(m.scales),
                       m.tensor_scales};
}

// Checks of the experts' part of a call; fills its launch arguments.
int experts_check(const char *fn, const void *x, int64_t tokens, int64_t ld_x, const int32_t *ids,
                  const float *weights, int top_k, const mx_moe_weights *moe, const void *y,
                  int64_t ld_y, const void *workspace, size_t workspace_bytes, mx::MoeArgs *a) {
  if (!moe) return fail(MX_ERR_INVALID_ARG, "%s: the experts' descriptor is null", fn);
  if (!valid_format(moe->format))
    return fail(MX_ERR_INVALID_ARG, "%s: format %d (MX_FMT_MXFP4 = 0 or MX_FMT_NVFP4 = 1)", fn,
                moe->format);
  if (moe->activation != MX_ACT_SILU && moe->activation != MX_ACT_GELU)
    return fail(MX_ERR_INVALID_ARG, "%s: activation %d (MX_ACT_SILU = 0 or MX_ACT_GELU = 1)", fn,
                moe->activation);
  int rc = few_check_x(fn, x, tokens, MX_MOE_MAX_TOKENS, moe->hidden, ld_x, "hidden");
  if (rc != MX_OK) return rc;
  if (!ids || !weights || !y)
    return fail(MX_ERR_INVALID_ARG, "%s: %s is null", fn, !ids ? "ids" : !weights ? "weights" : "y");
  if (moe->inter <= 0 || moe->inter % 32 != 0 || moe->inter >= (int64_t(1) << 31))
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: inter = %lld (a positive multiple of 32 below 2^31)",
                fn, static_cast<long long>(moe->inter));
  if (moe->experts < 1 || moe->experts > MX_MOE_MAX_EXPERTS)
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: experts = %lld (1..%d)", fn,
                static_cast<long long>(moe->experts), MX_MOE_MAX_EXPERTS);
  if (moe->experts * moe->hidden >= (int64_t(1) << 31) ||
      moe->experts * moe->inter >= (int64_t(1) << 31))
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: a stack of 2^31 or more rows", fn);
  if (top_k < 1 || top_k > MX_MOE_MAX_TOP_K)
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: top_k = %d (1..%d)", fn, top_k, MX_MOE_MAX_TOP_K);
  if (ld_y < moe->hidden || ld_y >= (int64_t(1) << 40))
    return fail(MX_ERR_INVALID_ARG, "%s: ld_y = %lld (>= hidden = %lld, below 2^40)", fn,
                static_cast<long long>(ld_y), static_cast<long long>(moe->hidden));
  const struct {
    const char *name;
    const mx_moe_matrix *m;
    int64_t rows, k;
  } mats[3] = {{"gate", &moe->gate, moe->inter, moe->hidden},
               {"up", &moe->up, moe->inter, moe->hidden},
               {"down", &moe->down, moe->hidden, moe->inter}};
  for (const auto &m : mats) {
    rc = few_check_matrix(fn, m.name, moe->format, m.m->codes, m.m->scales, m.m->tensor_scales,
                          m.rows, m.k);
    if (rc != MX_OK) return rc;
  }
  if (!aligned16(y) || !aligned4(ids) || !aligned4(weights))
    return fail(MX_ERR_ALIGNMENT, "%s: %s", fn,
                !aligned16(y) ? "y is not 16-byte aligned"
                : !aligned4(ids) ? "ids is not 4-byte aligned" : "weights is not 4-byte aligned");
  const size_t need = mx_moe_workspace_bytes(tokens, moe->hidden, moe->inter, top_k);
  if (need > 0) {
    if (!workspace || workspace_bytes < need)
      return fail(MX_ERR_WORKSPACE, "%s: needs a workspace of %zu bytes, got %zu%s", fn, need,
                  workspace ? workspace_bytes : size_t(0), workspace ? "" : " (null)");
    if (!aligned16(workspace))
      return fail(MX_ERR_ALIGNMENT, "%s: workspace is not 16-byte aligned", fn);
  }
  *a = mx::MoeArgs{};
  a->x = x;
  a->ld_x = ld_x;
  a->tokens = static_cast<int>(tokens);
  a->top_k = top_k;
  a->experts = static_cast<int>(moe->experts);
  a->hidden = static_cast<int>(moe->hidden);
  a->inter = static_cast<int>(moe->inter);
  a->fmt = moe->format == MX_FMT_MXFP4 ? 0 : 1;
  a->gelu = moe->activation == MX_ACT_GELU;
  a->ids = ids;
  a->weights = weights;
  a->gate = few_matrix(moe->gate);
  a->up = few_matrix(moe->up);
  a->down = few_matrix(moe->down);
  a->y = const_cast<void *>(y);
  a->ld_y = ld_y;
  const int64_t pairs = tokens * top_k;
  char *ws = static_cast<char *>(const_cast<void *>(workspace));
  a->h = reinterpret_cast<float *>(ws);
  a->z = reinterpret_cast<float *>(ws + moe_h_bytes(pairs, moe->inter));
  a->image = reinterpret_cast<uint8_t *>(a->z) + moe_z_bytes(pairs, moe->hidden);
  a->factors = reinterpret_cast<float *>(
      a->image + moe_images_bytes(tokens, moe->hidden, moe->inter, top_k));
  a->counts = reinterpret_cast<uint32_t *>(
      reinterpret_cast<char *>(a->factors) + round256(static_cast<size_t>(2 * pairs) * sizeof(float)));
  Range in[12];
  in[0] = span(x, row_bytes(tokens, moe->hidden, ld_x, 2));
  in[1] = span(ids, static_cast<uint64_t>(pairs) * 4);
  in[2] = span(weights, static_cast<uint64_t>(pairs) * 4);
  matrix_ranges(a->gate, moe->format, moe->experts, moe->inter, moe->hidden, in + 3);
  matrix_ranges(a->up, moe->format, moe->experts, moe->inter, moe->hidden, in + 6);
  matrix_ranges(a->down, moe->format, moe->experts, moe->hidden, moe->inter, in + 9);
  const Range out[2] = {span(y, row_bytes(tokens, moe->hidden, ld_y, 2)), span(workspace, need)};
  return check_disjoint(fn, out, 2, in, 12);
}

void moe_device(mx::MoeArgs *a, const DeviceInfo *dev) {
  a->num_sms = dev->num_sms;
  a->status = dev->status;
  const int64_t pairs = static_cast<int64_t>(a->tokens) * a->top_k;
  a->up_parts = mx::moe_parts(pairs, a->experts, a->inter, a->hidden, dev->num_sms);
  a->down_parts = mx::moe_parts(pairs, a->experts, a->hidden, a->inter, dev->num_sms);
}

}  // namespace

namespace {

// The arguments of a linear call; workspace_used: the bytes that the call writes there.
int linear_check(const char *fn, const void *x, int64_t tokens, int64_t k, int64_t ld_x, int format,
                 const void *w_codes, const void *w_scales, const float *w_tensor_scale, int64_t n,
                 void *y, int64_t ld_y, int out_dtype, const mx_gemm_epilogue *epilogue,
                 const void *workspace, size_t workspace_used, mx::LinearArgs *out_args) {
  if (!valid_format(format))
    return fail(MX_ERR_INVALID_ARG, "%s: format %d (MX_FMT_MXFP4 = 0 or MX_FMT_NVFP4 = 1)", fn,
                format);
  int rc = few_check_x(fn, x, tokens, MX_LINEAR_MAX_TOKENS, k, ld_x, "k");
  if (rc != MX_OK) return rc;
  if (!y) return fail(MX_ERR_INVALID_ARG, "%s: y is null", fn);
  if (n <= 0 || n % 32 != 0 || n >= (int64_t(1) << 31))
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: n = %lld (a positive multiple of 32 below 2^31)", fn,
                static_cast<long long>(n));
  rc = few_check_matrix(fn, "weight", format, w_codes, w_scales, w_tensor_scale, n, k);
  if (rc != MX_OK) return rc;
  if (out_dtype != MX_OUT_BF16 && out_dtype != MX_OUT_FP32)
    return fail(MX_ERR_UNSUPPORTED_FEATURE, "%s: out_dtype %d (MX_OUT_BF16 = 0 or MX_OUT_FP32 = 1)",
                fn, out_dtype);
  if (ld_y < n || ld_y >= (int64_t(1) << 40))
    return fail(MX_ERR_INVALID_ARG, "%s: ld_y = %lld (>= n = %lld, below 2^40)", fn,
                static_cast<long long>(ld_y), static_cast<long long>(n));
  if (!aligned16(y)) return fail(MX_ERR_ALIGNMENT, "%s: y is not 16-byte aligned", fn);
  if (epilogue && epilogue->gelu != 0 && epilogue->gelu != 1)
    return fail(MX_ERR_INVALID_ARG, "%s: epilogue gelu = %d (0 or 1)", fn, epilogue->gelu);
  if (epilogue && epilogue->bias && !aligned16(epilogue->bias))
    return fail(MX_ERR_ALIGNMENT, "%s: bias is not 16-byte aligned", fn);
  mx::LinearArgs &a = *out_args;
  a = mx::LinearArgs{};
  a.x = x;
  a.ld_x = ld_x;
  a.tokens = static_cast<int>(tokens);
  a.n = n;
  a.k = k;
  a.fmt = format == MX_FMT_MXFP4 ? 0 : 1;
  a.w = mx::FewMatrix{static_cast<const uint8_t *>(w_codes), static_cast<const uint8_t *>(w_scales),
                      w_tensor_scale};
  a.y = y;
  a.ld_y = ld_y;
  a.out_fp32 = out_dtype == MX_OUT_FP32;
  if (epilogue) {
    a.bias = epilogue->bias;
    a.beta = epilogue->beta;
    a.gelu = epilogue->gelu;
  }
  Range in[5];
  in[0] = span(x, row_bytes(tokens, k, ld_x, 2));
  in[1] = span(a.bias, static_cast<uint64_t>(n) * sizeof(float));
  matrix_ranges(a.w, format, 1, n, k, in + 2);
  const Range out[2] = {span(y, row_bytes(tokens, n, ld_y, a.out_fp32 ? 4 : 2)),
                        span(workspace, workspace ? workspace_used : 0)};
  return check_disjoint(fn, out, workspace ? 2 : 1, in, 5);
}

int linear_run(const char *fn, mx::LinearArgs *a, void *workspace, void *stream) {
  DeviceInfo *dev = nullptr;
  const int rc = device_info(&dev);
  if (rc != MX_OK) return rc;
  if (a->tokens == 0) return MX_OK;
  a->num_sms = dev->num_sms;
  a->status = dev->status;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launch_rc(fn, workspace ? mx::launch_linear_mma(*a, workspace, s) : mx::launch_linear(*a, s));
}

}  // namespace

MX_API int mx_linear_bf16(const void *x, int64_t tokens, int64_t k, int64_t ld_x, int format,
                          const void *w_codes, const void *w_scales, const float *w_tensor_scale,
                          int64_t n, void *y, int64_t ld_y, int out_dtype,
                          const mx_gemm_epilogue *epilogue, void *stream) {
  clear_detail();
  const char *fn = "mx_linear_bf16";
  mx::LinearArgs a;
  const int rc = linear_check(fn, x, tokens, k, ld_x, format, w_codes, w_scales, w_tensor_scale, n,
                              y, ld_y, out_dtype, epilogue, nullptr, 0, &a);
  return rc != MX_OK ? rc : linear_run(fn, &a, nullptr, stream);
}

MX_API size_t mx_linear_workspace_bytes(int64_t tokens, int64_t k, int64_t n, int format) {
  if (!valid_format(format) || tokens < 1 || tokens > MX_LINEAR_MAX_TOKENS || k <= 0 || k % 32 != 0 ||
      n <= 0 || n % 32 != 0 || k >= (int64_t(1) << 31) || n >= (int64_t(1) << 31) ||
      too_many_blocks(format, n, k))
    return 0;
  const int fmt = format == MX_FMT_MXFP4 ? 0 : 1;
  return mx::linear_mma_better(tokens, n, k) ? mx::linear_workspace_bytes(fmt, tokens, n, k) : 0;
}

MX_API int mx_linear_bf16_workspace(const void *x, int64_t tokens, int64_t k, int64_t ld_x,
                                    int format, const void *w_codes, const void *w_scales,
                                    const float *w_tensor_scale, int64_t n, void *y, int64_t ld_y,
                                    int out_dtype, const mx_gemm_epilogue *epilogue,
                                    void *workspace, size_t workspace_bytes, void *stream) {
  clear_detail();
  const char *fn = "mx_linear_bf16_workspace";
  const size_t need = mx_linear_workspace_bytes(tokens, k, n, format);
  if (need == 0) workspace = nullptr;
  mx::LinearArgs a;
  int rc = linear_check(fn, x, tokens, k, ld_x, format, w_codes, w_scales, w_tensor_scale, n, y,
                        ld_y, out_dtype, epilogue, workspace, need, &a);
  if (rc != MX_OK) return rc;
  if (need > 0 && (workspace == nullptr || workspace_bytes < need))
    return fail(MX_ERR_WORKSPACE, "%s: needs a workspace of %zu bytes, got %zu%s", fn, need,
                workspace ? workspace_bytes : size_t(0), workspace ? "" : " (null)");
  if (!aligned16(workspace))
    return fail(MX_ERR_ALIGNMENT, "%s: workspace is not 16-byte aligned", fn);
  return linear_run(fn, &a, workspace, stream);
}

MX_API int mx_moe_route_bf16(const void *x, int64_t tokens, int64_t hidden, int64_t ld_x,
                             const void *router, int64_t experts, const float *bias, int top_k,
                             int normalize, int32_t *ids, float *weights, void *stream) {
  clear_detail();
  const char *fn = "mx_moe_route_bf16";
  int rc = route_check(fn, x, tokens, hidden, ld_x, router, experts, bias, top_k, normalize, ids,
                       weights);
  if (rc != MX_OK) return rc;
  DeviceInfo *dev = nullptr;
  rc = device_info(&dev);
  if (rc != MX_OK) return rc;
  if (tokens == 0) return MX_OK;
  const mx::RouteArgs a{x,     ld_x,  static_cast<int>(tokens), static_cast<int>(hidden),
                        static_cast<int>(experts), top_k, normalize, router, bias, ids, weights,
                        dev->status};
  return launch_rc(fn, mx::launch_moe_route(a, nullptr, static_cast<cudaStream_t>(stream)));
}

MX_API size_t mx_moe_workspace_bytes(int64_t tokens, int64_t hidden, int64_t inter, int top_k) {
  if (tokens < 1 || tokens > MX_MOE_MAX_TOKENS || top_k < 1 || top_k > MX_MOE_MAX_TOP_K ||
      hidden <= 0 || inter <= 0 || hidden % 32 != 0 || inter % 32 != 0 ||
      hidden >= (int64_t(1) << 31) || inter >= (int64_t(1) << 31))
    return 0;
  const int64_t pairs = tokens * top_k;
  return moe_h_bytes(pairs, inter) + moe_z_bytes(pairs, hidden) +
         moe_images_bytes(tokens, hidden, inter, top_k) +
         round256(static_cast<size_t>(2 * pairs) * sizeof(float)) +
         round256(static_cast<size_t>(mx::moe_counts(static_cast<int>(pairs))) * sizeof(uint32_t));
}

MX_API int mx_moe_experts_bf16(const void *x, int64_t tokens, int64_t ld_x, const int32_t *ids,
                               const float *weights, int top_k, const mx_moe_weights *moe, void *y,
                               int64_t ld_y, void *workspace, size_t workspace_bytes,
                               void *stream) {
  clear_detail();
  const char *fn = "mx_moe_experts_bf16";
  mx::MoeArgs a;
  int rc = experts_check(fn, x, tokens, ld_x, ids, weights, top_k, moe, y, ld_y, workspace,
                         workspace_bytes, &a);
  if (rc != MX_OK) return rc;
  DeviceInfo *dev = nullptr;
  rc = device_info(&dev);
  if (rc != MX_OK) return rc;
  if (tokens == 0) return MX_OK;
  moe_device(&a, dev);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = mx::launch_moe_prepare(a, s);
  return launch_rc(fn, e != cudaSuccess ? e : mx::launch_moe_experts(a, s));
}

MX_API int mx_moe_layer_bf16(const void *x, int64_t tokens, int64_t ld_x, const void *router,
                             const float *router_bias, int top_k, int normalize,
                             const mx_moe_weights *moe, int32_t *ids, float *weights, void *y,
                             int64_t ld_y, void *workspace, size_t workspace_bytes,
                             void *stream) {
  clear_detail();
  const char *fn = "mx_moe_layer_bf16";
  mx::MoeArgs a;
  int rc = experts_check(fn, x, tokens, ld_x, ids, weights, top_k, moe, y, ld_y, workspace,
                         workspace_bytes, &a);
  if (rc != MX_OK) return rc;
  rc = route_check(fn, x, tokens, moe->hidden, ld_x, router, moe->experts, router_bias, top_k,
                   normalize, ids, weights);
  if (rc != MX_OK) return rc;
  {
    // what the router reads and writes against the experts' inputs and outputs
    const uint64_t slots = static_cast<uint64_t>(tokens) * static_cast<uint64_t>(top_k) * 4;
    const Range choice[2] = {span(ids, slots), span(weights, slots)};
    Range fixed[9];
    matrix_ranges(a.gate, moe->format, moe->experts, moe->inter, moe->hidden, fixed);
    matrix_ranges(a.up, moe->format, moe->experts, moe->inter, moe->hidden, fixed + 3);
    matrix_ranges(a.down, moe->format, moe->experts, moe->hidden, moe->inter, fixed + 6);
    rc = check_disjoint(fn, choice, 2, fixed, 9);
    if (rc != MX_OK) return rc;
    const Range gate_in[2] = {span(router, static_cast<uint64_t>(moe->experts * moe->hidden) * 2),
                              span(router_bias, static_cast<uint64_t>(moe->experts) * 4)};
    const Range out[2] = {span(y, row_bytes(tokens, moe->hidden, ld_y, 2)),
                          span(workspace, mx_moe_workspace_bytes(tokens, moe->hidden, moe->inter,
                                                                 top_k))};
    rc = check_disjoint(fn, out, 2, gate_in, 2);
    if (rc != MX_OK) return rc;
  }
  DeviceInfo *dev = nullptr;
  rc = device_info(&dev);
  if (rc != MX_OK) return rc;
  if (tokens == 0) return MX_OK;
  moe_device(&a, dev);
  const mx::RouteArgs r{x,      ld_x,        a.tokens, a.hidden, a.experts, top_k,     normalize,
                        router, router_bias, ids,      weights,  dev->status};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = mx::launch_moe_route(r, &a, s);
  return launch_rc(fn, e != cudaSuccess ? e : mx::launch_moe_experts(a, s));
}

// ---- the rest of a decoding step

namespace {

// A strided block of rows in device memory.
struct Rows {
  const char *name;
  const void *p;
  int64_t rows, cols, ld;
};

// Do two blocks of 2-byte elements share an element?  Blocks of one stride may lie in each
// other's gaps; otherwise their whole ranges count.
bool rows_overlap(const Rows &a, const Rows &b) {
  const Range ra = span(a.p, row_bytes(a.rows, a.cols, a.ld, 2)), rb = span(b.p, row_bytes(b.rows, b.cols, b.ld, 2));
  if (!a.p || !b.p || !overlap(ra, rb)) return false;
  if (a.ld != b.ld) return true;
  const uint64_t pitch = static_cast<uint64_t>(a.ld) * 2, wa = static_cast<uint64_t>(a.cols) * 2,
                 wb = static_cast<uint64_t>(b.cols) * 2;
  const uint64_t d = rb.lo >= ra.lo ? (rb.lo - ra.lo) % pitch : (pitch - (ra.lo - rb.lo) % pitch) % pitch;
  return d < wa || d + wb > pitch;
}

// A block of `heads` heads: present iff there are heads, aligned, its stride wide enough.
int rows_check(const char *fn, const Rows &r) {
  if (r.cols == 0) {
    if (r.p) return fail(MX_ERR_INVALID_ARG, "%s: %s must be null: it has no heads", fn, r.name);
    return MX_OK;
  }
  if (!r.p) return fail(MX_ERR_INVALID_ARG, "%s: %s is null", fn, r.name);
  if (r.ld < r.cols || r.ld >= (int64_t(1) << 31))
    return fail(MX_ERR_INVALID_ARG, "%s: row stride %lld of %s (%lld .. 2^31 - 1)", fn,
                static_cast<long long>(r.ld), r.name, static_cast<long long>(r.cols));
  if (!aligned16(r.p) || r.ld % 8 != 0)
    return fail(MX_ERR_ALIGNMENT, "%s: %s %s", fn, r.name,
                !aligned16(r.p) ? "is not 16-byte aligned"
                                : "has a row stride that is not a multiple of 8 elements (16 bytes)");
  return MX_OK;
}

int qk_norm_check(const char *fn, const mx_qk_norm *n, int64_t tokens) {
  if (!n) return fail(MX_ERR_INVALID_ARG, "%s: the norm's descriptor is null", fn);
  if (tokens < 0 || tokens >= (int64_t(1) << 31))
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: tokens = %lld (0 .. 2^31 - 1)", fn, static_cast<long long>(tokens));
  if (n->q_heads < 0 || n->k_heads < 0 || n->q_heads > 65535 || n->k_heads > 65535 || n->q_heads + n->k_heads == 0)
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: %lld query and %lld key heads (0..65535, one at least)", fn,
                static_cast<long long>(n->q_heads), static_cast<long long>(n->k_heads));
  if (n->head_dim < 16 || n->head_dim > mx::kRopeMaxDim || n->head_dim % 16 != 0)
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: head_dim = %lld (a multiple of 16, 16..%d)", fn,
                static_cast<long long>(n->head_dim), mx::kRopeMaxDim);
  if (n->rotary_dim < 0 || n->rotary_dim > n->head_dim || n->rotary_dim % 16 != 0)
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: rotary_dim = %lld (a multiple of 16, 0..head_dim)", fn,
                static_cast<long long>(n->rotary_dim));
  if (n->interleaved != 0 && n->interleaved != 1)
    return fail(MX_ERR_INVALID_ARG, "%s: interleaved = %d (0 or 1)", fn, n->interleaved);
  if (!(n->eps >= 0.0f) || n->eps > FLT_MAX)
    return fail(MX_ERR_INVALID_ARG, "%s: eps = %g (0 or more, finite)", fn, static_cast<double>(n->eps));
  if ((n->rotary_dim > 0) != (n->inv_freq != nullptr))
    return fail(MX_ERR_INVALID_ARG, "%s: inv_freq %s", fn,
                n->inv_freq ? "must be null when rotary_dim is 0" : "is null");
  if (!aligned16(n->q_weight) || !aligned16(n->k_weight))
    return fail(MX_ERR_ALIGNMENT, "%s: %s is not 16-byte aligned", fn, aligned16(n->q_weight) ? "k_weight" : "q_weight");
  if (!aligned4(n->inv_freq)) return fail(MX_ERR_ALIGNMENT, "%s: inv_freq is not 4-byte aligned", fn);
  return MX_OK;
}

// Outputs (and plain ranges among them) against inputs and one another.
int rows_disjoint(const char *fn, const Rows *out, int nout, const Rows *in, int nin, const Range *small_out,
                  int nsmall_out, const Range *small_in, int nsmall_in, bool in_place) {
  auto range = [](const Rows &r) { return span(r.p, row_bytes(r.rows, r.cols, r.ld, 2)); };
  for (int o = 0; o < nout; ++o) {
    for (int i = 0; i < nin; ++i) {
      if (in_place && i == o && out[o].p == in[i].p && out[o].ld == in[i].ld) continue;
      if (rows_overlap(out[o], in[i]))
        return fail(MX_ERR_INVALID_ARG, "%s: %s overlaps %s", fn, out[o].name, in[i].name);
    }
    for (int p = o + 1; p < nout; ++p)
      if (rows_overlap(out[o], out[p]))
        return fail(MX_ERR_INVALID_ARG, "%s: %s overlaps %s", fn, out[o].name, out[p].name);
    for (int i = 0; i < nsmall_in; ++i)
      if (overlap(range(out[o]), small_in[i]))
        return fail(MX_ERR_INVALID_ARG, "%s: %s overlaps an input", fn, out[o].name);
    for (int p = 0; p < nsmall_out; ++p)
      if (overlap(range(out[o]), small_out[p]))
        return fail(MX_ERR_INVALID_ARG, "%s: %s overlaps another output or the workspace", fn, out[o].name);
  }
  for (int p = 0; p < nsmall_out; ++p)
    for (int i = 0; i < nin; ++i)
      if (overlap(small_out[p], range(in[i])))
        return fail(MX_ERR_INVALID_ARG, "%s: an output or the workspace overlaps %s", fn, in[i].name);
  return check_disjoint(fn, small_out, nsmall_out, small_in, nsmall_in);
}

mx::Heads heads_of(const void *x, int64_t ld, const void *dy, int64_t ld_dy, void *y, int64_t ld_y,
                   const void *weight, float *dweight, int64_t heads) {
  mx::Heads h;
  h.x = static_cast<const uint16_t *>(x);
  h.ld = ld;
  h.dy = static_cast<const uint16_t *>(dy);
  h.ld_dy = ld_dy;
  h.y = static_cast<uint16_t *>(y);
  h.ld_y = ld_y;
  h.weight = static_cast<const uint16_t *>(weight);
  h.dweight = dweight;
  h.heads = static_cast<int>(heads);
  return h;
}

void rope_args(mx::RopeArgs *a, int64_t tokens, const int32_t *positions, const mx_qk_norm *norm,
               const DeviceInfo *dev) {
  a->tokens = tokens;
  a->positions = positions;
  a->inv_freq = norm->inv_freq;
  a->head_dim = static_cast<int>(norm->head_dim);
  a->rotary_dim = static_cast<int>(norm->rotary_dim);
  a->interleaved = norm->interleaved;
  a->eps = norm->eps;
  a->partials = nullptr;
  a->num_sms = dev->num_sms;
  a->status = dev->status;
}

int positions_check(const char *fn, const int32_t *positions) {
  if (!positions) return fail(MX_ERR_INVALID_ARG, "%s: positions is null", fn);
  if (!aligned4(positions)) return fail(MX_ERR_ALIGNMENT, "%s: positions is not 4-byte aligned", fn);
  return MX_OK;
}

void norm_ranges(const mx_qk_norm *n, const int32_t *positions, int64_t tokens, Range *out) {
  out[0] = span(positions, static_cast<uint64_t>(tokens) * 4);
  out[1] = span(n->inv_freq, static_cast<uint64_t>(n->rotary_dim / 2) * 4);
  out[2] = span(n->q_weight, static_cast<uint64_t>(n->head_dim) * 2);
  out[3] = span(n->k_weight, static_cast<uint64_t>(n->head_dim) * 2);
}

}  // namespace

MX_API int mx_qk_norm_rope_bf16(const void *q, int64_t ld_q, const void *k, int64_t ld_k, int64_t tokens,
                                const int32_t *positions, const mx_qk_norm *norm, void *q_out,
                                int64_t ld_q_out, void *k_out, int64_t ld_k_out, void *stream) {
  clear_detail();
  const char *fn = "mx_qk_norm_rope_bf16";
  int rc = qk_norm_check(fn, norm, tokens);
  if (rc == MX_OK) rc = positions_check(fn, positions);
  if (rc != MX_OK) return rc;
  const int64_t qc = norm->q_heads * norm->head_dim, kc = norm->k_heads * norm->head_dim;
  const Rows in[2] = {{"q", q, tokens, qc, ld_q}, {"k", k, tokens, kc, ld_k}};
  const Rows out[2] = {{"q_out", q_out, tokens, qc, ld_q_out}, {"k_out", k_out, tokens, kc, ld_k_out}};
  for (int i = 0; i < 2 && rc == MX_OK; ++i) rc = rows_check(fn, in[i]);
  for (int i = 0; i < 2 && rc == MX_OK; ++i) rc = rows_check(fn, out[i]);
  if (rc != MX_OK) return rc;
  Range small[4];
  norm_ranges(norm, positions, tokens, small);
  rc = rows_disjoint(fn, out, 2, in, 2, nullptr, 0, small, 4, true);
  if (rc != MX_OK) return rc;
  DeviceInfo *dev = nullptr;
  rc = device_info(&dev);
  if (rc != MX_OK) return rc;
  if (tokens == 0) return MX_OK;
  mx::RopeArgs a;
  rope_args(&a, tokens, positions, norm, dev);
  a.part[0] = heads_of(q, ld_q, nullptr, 0, q_out, ld_q_out, norm->q_weight, nullptr, norm->q_heads);
  a.part[1] = heads_of(k, ld_k, nullptr, 0, k_out, ld_k_out, norm->k_weight, nullptr, norm->k_heads);
  return launch_rc(fn, mx::launch_qk_rope(a, static_cast<cudaStream_t>(stream)));
}

MX_API size_t mx_qk_norm_rope_backward_workspace_bytes(int64_t tokens, const mx_qk_norm *norm) {
  const KeepDetail keep;
  if (qk_norm_check("mx_qk_norm_rope_backward_workspace_bytes", norm, tokens) != MX_OK) return 0;
  return static_cast<size_t>(mx::kRopeBackCtas) * 2 * static_cast<size_t>(norm->head_dim) * sizeof(float);
}

MX_API int mx_qk_norm_rope_backward_bf16(const void *q, int64_t ld_q, const void *k, int64_t ld_k,
                                         const void *dq_out, int64_t ld_dq_out, const void *dk_out,
                                         int64_t ld_dk_out, int64_t tokens, const int32_t *positions,
                                         const mx_qk_norm *norm, void *dq, int64_t ld_dq, void *dk,
                                         int64_t ld_dk, float *dq_weight, float *dk_weight,
                                         void *workspace, size_t workspace_bytes, void *stream) {
  const char *fn = "mx_qk_norm_rope_backward_bf16";
  clear_detail();
  const size_t need = mx_qk_norm_rope_backward_workspace_bytes(tokens, norm);
  int rc = qk_norm_check(fn, norm, tokens);
  if (rc == MX_OK) rc = positions_check(fn, positions);
  if (rc != MX_OK) return rc;
  const int64_t qc = norm->q_heads * norm->head_dim, kc = norm->k_heads * norm->head_dim;
  const Rows in[4] = {{"q", q, tokens, qc, ld_q},
                      {"k", k, tokens, kc, ld_k},
                      {"dq_out", dq_out, tokens, qc, ld_dq_out},
                      {"dk_out", dk_out, tokens, kc, ld_dk_out}};
  const Rows out[2] = {{"dq", dq, tokens, qc, ld_dq}, {"dk", dk, tokens, kc, ld_dk}};
  for (int i = 0; i < 4 && rc == MX_OK; ++i) rc = rows_check(fn, in[i]);
  for (int i = 0; i < 2 && rc == MX_OK; ++i) rc = rows_check(fn, out[i]);
  if (rc != MX_OK) return rc;
  if ((dq_weight && !norm->q_weight) || (dk_weight && !norm->k_weight))
    return fail(MX_ERR_INVALID_ARG, "%s: %s must be null: there is no such weight", fn,
                dq_weight && !norm->q_weight ? "dq_weight" : "dk_weight");
  if (!aligned4(dq_weight) || !aligned4(dk_weight))
    return fail(MX_ERR_ALIGNMENT, "%s: %s is not 4-byte aligned", fn, aligned4(dq_weight) ? "dk_weight" : "dq_weight");
  const bool weights = dq_weight || dk_weight;
  if (weights) {
    if (!workspace || workspace_bytes < need)
      return fail(MX_ERR_WORKSPACE, "%s: needs a workspace of %zu bytes, got %zu%s", fn, need,
                  workspace ? workspace_bytes : size_t(0), workspace ? "" : " (null)");
    if (!aligned16(workspace)) return fail(MX_ERR_ALIGNMENT, "%s: workspace is not 16-byte aligned", fn);
  }
  Range small_in[4];
  norm_ranges(norm, positions, tokens, small_in);
  const uint64_t dw = static_cast<uint64_t>(norm->head_dim) * 4;
  const Range small_out[3] = {span(dq_weight, dw), span(dk_weight, dw), span(weights ? workspace : nullptr, need)};
  rc = rows_disjoint(fn, out, 2, in, 4, small_out, 3, small_in, 4, false);
  if (rc != MX_OK) return rc;
  DeviceInfo *dev = nullptr;
  rc = device_info(&dev);
  if (rc != MX_OK) return rc;
  if (tokens == 0 && !weights) return MX_OK;
  mx::RopeArgs a;
  rope_args(&a, tokens, positions, norm, dev);
  a.part[0] = heads_of(q, ld_q, dq_out, ld_dq_out, dq, ld_dq, norm->q_weight, dq_weight, norm->q_heads);
  a.part[1] = heads_of(k, ld_k, dk_out, ld_dk_out, dk, ld_dk, norm->k_weight, dk_weight, norm->k_heads);
  if (weights) a.partials = static_cast<float *>(workspace);
  return launch_rc(fn, mx::launch_qk_rope_backward(a, static_cast<cudaStream_t>(stream)));
}

namespace {

static_assert(MX_CACHE_BLOCK == mx::kCacheBlock && MX_ATTENTION_MAX_QUERY == mx::kAttentionMaxQuery &&
                  MX_ATTENTION_MAX_SEQUENCES == mx::kAttentionMaxSequences &&
                  MX_SAMPLE_MAX_VOCAB == mx::kSampleMaxVocab,
              "limits of the decoding step");

int cache_shape_check(const char *fn, const mx_kv_cache *c) {
  if (!c) return fail(MX_ERR_INVALID_ARG, "%s: the cache's descriptor is null", fn);
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: head_dim = %lld (64, 128 or 256)", fn,
                static_cast<long long>(c->head_dim));
  if (c->kv_heads < 1 || c->kv_heads > 1024)
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: kv_heads = %lld (1..1024)", fn, static_cast<long long>(c->kv_heads));
  if (c->page_tokens < MX_CACHE_BLOCK || c->page_tokens > (1 << 20) || c->page_tokens % MX_CACHE_BLOCK != 0)
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: page_tokens = %lld (a multiple of %d up to 2^20)", fn,
                static_cast<long long>(c->page_tokens), MX_CACHE_BLOCK);
  if (c->pages < 1 || c->pages >= (int64_t(1) << 31))
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: pages = %lld (1 .. 2^31 - 1)", fn, static_cast<long long>(c->pages));
  // (page_tokens * head_dim <= 2^28, pages * kv_heads < 2^41)
  if (c->pages * c->kv_heads > (int64_t(1) << 48) / (c->page_tokens * c->head_dim))
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: %lld pages of %lld x %lld x %lld codes (2^48 in all)", fn,
                static_cast<long long>(c->pages), static_cast<long long>(c->kv_heads),
                static_cast<long long>(c->page_tokens), static_cast<long long>(c->head_dim));
  return MX_OK;
}

// The cache, the page table and the lengths; fills the kernels' view and the six ranges
// (codes and scales of keys and values, page table, lengths).
int cache_check(const char *fn, const mx_kv_cache *c, const int32_t *page_table, int64_t max_pages,
                const int32_t *lengths, int64_t sequences, int64_t most, mx::CacheArgs *a, Range *ranges) {
  const int rc = cache_shape_check(fn, c);
  if (rc != MX_OK) return rc;
  if (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales)
    return fail(MX_ERR_INVALID_ARG, "%s: the cache's codes or scales are null", fn);
  if (!aligned16(c->k_codes) || !aligned16(c->k_scales) || !aligned16(c->v_codes) || !aligned16(c->v_scales))
    return fail(MX_ERR_ALIGNMENT, "%s: the cache's codes or scales are not 16-byte aligned", fn);
  if (!page_table || !lengths)
    return fail(MX_ERR_INVALID_ARG, "%s: %s is null", fn, !page_table ? "page_table" : "lengths");
  if (!aligned4(page_table) || !aligned4(lengths))
    return fail(MX_ERR_ALIGNMENT, "%s: %s is not 4-byte aligned", fn, !aligned4(page_table) ? "page_table" : "lengths");
  if (sequences < 0 || sequences > most)
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: sequences = %lld (0..%lld)", fn, static_cast<long long>(sequences),
                static_cast<long long>(most));
  if (max_pages < 1 || max_pages > (int64_t(1) << 24))
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: max_pages = %lld (1 .. 2^24)", fn, static_cast<long long>(max_pages));
  a->codes[0] = static_cast<uint8_t *>(c->k_codes);
  a->codes[1] = static_cast<uint8_t *>(c->v_codes);
  a->scales[0] = static_cast<uint8_t *>(c->k_scales);
  a->scales[1] = static_cast<uint8_t *>(c->v_scales);
  a->pages = c->pages;
  a->page_tokens = static_cast<int>(c->page_tokens);
  a->heads = static_cast<int>(c->kv_heads);
  a->head_dim = static_cast<int>(c->head_dim);
  a->table = page_table;
  a->max_pages = max_pages;
  a->lengths = lengths;
  a->sequences = static_cast<int>(sequences);
  a->status = nullptr;
  const uint64_t rows = static_cast<uint64_t>(c->pages) * static_cast<uint64_t>(c->kv_heads);
  const uint64_t codes = rows * static_cast<uint64_t>(c->page_tokens * c->head_dim);
  const uint64_t scales = rows * static_cast<uint64_t>(c->page_tokens / MX_CACHE_BLOCK);
  ranges[0] = span(c->k_codes, codes);
  ranges[1] = span(c->k_scales, scales);
  ranges[2] = span(c->v_codes, codes);
  ranges[3] = span(c->v_scales, scales);
  ranges[4] = span(page_table, static_cast<uint64_t>(sequences) * static_cast<uint64_t>(max_pages) * 4);
  ranges[5] = span(lengths, static_cast<uint64_t>(sequences) * 4);
  return MX_OK;
}

}  // namespace

MX_API int mx_kv_append_bf16(const void *k, int64_t ld_k, const void *v, int64_t ld_v, int64_t tokens,
                             const int32_t *starts, const int32_t *page_table, int64_t max_pages,
                             const int32_t *lengths, int64_t sequences, const mx_kv_cache *cache,
                             void *stream) {
  clear_detail();
  const char *fn = "mx_kv_append_bf16";
  mx::AppendArgs a;
  Range ranges[6];
  int rc = cache_check(fn, cache, page_table, max_pages, lengths, sequences, 65535, &a.c, ranges);
  if (rc != MX_OK) return rc;
  if (tokens < 0 || tokens > (int64_t(1) << 30))
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: tokens = %lld (0 .. 2^30)", fn, static_cast<long long>(tokens));
  if (!starts && sequences > 0 && tokens % sequences != 0)
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: %lld tokens for %lld sequences without starts", fn,
                static_cast<long long>(tokens), static_cast<long long>(sequences));
  const int64_t cols = cache->kv_heads * cache->head_dim;
  const Rows in[2] = {{"k", k, tokens, cols, ld_k}, {"v", v, tokens, cols, ld_v}};
  for (int i = 0; i < 2 && rc == MX_OK; ++i) rc = rows_check(fn, in[i]);
  if (rc != MX_OK) return rc;
  if (!aligned4(starts)) return fail(MX_ERR_ALIGNMENT, "%s: starts is not 4-byte aligned", fn);
  const Range inputs[5] = {span(k, row_bytes(tokens, cols, ld_k, 2)), span(v, row_bytes(tokens, cols, ld_v, 2)),
                           ranges[4], ranges[5], span(starts, static_cast<uint64_t>(sequences + 1) * 4)};
  rc = check_disjoint(fn, ranges, 4, inputs, 5);
  if (rc != MX_OK) return rc;
  DeviceInfo *dev = nullptr;
  rc = device_info(&dev);
  if (rc != MX_OK) return rc;
  if (tokens == 0 || sequences == 0) return MX_OK;
  a.c.status = dev->status;
  a.x[0] = static_cast<const uint16_t *>(k);
  a.x[1] = static_cast<const uint16_t *>(v);
  a.ld[0] = ld_k;
  a.ld[1] = ld_v;
  a.tokens = tokens;
  a.starts = starts;
  return launch_rc(fn, mx::launch_kv_append(a, static_cast<cudaStream_t>(stream)));
}

namespace {

int attention_shape_check(const char *fn, int64_t sequences, int64_t q_tokens, int64_t q_heads,
                          const mx_kv_cache *cache) {
  const int rc = cache_shape_check(fn, cache);
  if (rc != MX_OK) return rc;
  if (sequences < 0 || sequences > MX_ATTENTION_MAX_SEQUENCES)
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: sequences = %lld (0..%d)", fn, static_cast<long long>(sequences),
                MX_ATTENTION_MAX_SEQUENCES);
  if (q_tokens < 1 || q_tokens > MX_ATTENTION_MAX_QUERY)
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: q_tokens = %lld (1..%d)", fn, static_cast<long long>(q_tokens),
                MX_ATTENTION_MAX_QUERY);
  if (q_heads < cache->kv_heads || q_heads % cache->kv_heads != 0 ||
      q_heads / cache->kv_heads > mx::kAttentionMaxGroup)
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: q_heads = %lld (a multiple of kv_heads = %lld, at most %d times)", fn,
                static_cast<long long>(q_heads), static_cast<long long>(cache->kv_heads), mx::kAttentionMaxGroup);
  return MX_OK;
}

}  // namespace

MX_API size_t mx_attention_workspace_bytes(int64_t sequences, int64_t q_tokens, int64_t q_heads,
                                           const mx_kv_cache *cache) {
  const KeepDetail keep;
  if (attention_shape_check("mx_attention_workspace_bytes", sequences, q_tokens, q_heads, cache) != MX_OK) return 0;
  return mx::attention_workspace_bytes(q_heads / cache->kv_heads * q_tokens, static_cast<int>(cache->head_dim));
}

MX_API int mx_attention_bf16(const void *q, int64_t ld_q, int64_t q_heads, int64_t sequences,
                             int64_t q_tokens, const int32_t *page_table, int64_t max_pages,
                             const int32_t *lengths, const mx_kv_cache *cache, float scale,
                             int64_t window, void *out, int64_t ld_out, float *lse, void *workspace,
                             size_t workspace_bytes, void *stream) {
  const char *fn = "mx_attention_bf16";
  clear_detail();
  const size_t need = mx_attention_workspace_bytes(sequences, q_tokens, q_heads, cache);
  int rc = attention_shape_check(fn, sequences, q_tokens, q_heads, cache);
  if (rc != MX_OK) return rc;
  mx::AttentionArgs a;
  Range ranges[6];
  rc = cache_check(fn, cache, page_table, max_pages, lengths, sequences, MX_ATTENTION_MAX_SEQUENCES, &a.c, ranges);
  if (rc != MX_OK) return rc;
  if (!(scale >= -FLT_MAX && scale <= FLT_MAX))
    return fail(MX_ERR_INVALID_ARG, "%s: scale = %g (finite)", fn, static_cast<double>(scale));
  if (window < 0 || window >= (int64_t(1) << 31))
    return fail(MX_ERR_INVALID_ARG, "%s: window = %lld (0 .. 2^31 - 1)", fn, static_cast<long long>(window));
  const int64_t rows = sequences * q_tokens, cols = q_heads * cache->head_dim;
  const Rows in{"q", q, rows, cols, ld_q}, o{"out", out, rows, cols, ld_out};
  rc = rows_check(fn, in);
  if (rc == MX_OK) rc = rows_check(fn, o);
  if (rc != MX_OK) return rc;
  if (!aligned4(lse)) return fail(MX_ERR_ALIGNMENT, "%s: lse is not 4-byte aligned", fn);
  if (!workspace || workspace_bytes < need)
    return fail(MX_ERR_WORKSPACE, "%s: needs a workspace of %zu bytes, got %zu%s", fn, need,
                workspace ? workspace_bytes : size_t(0), workspace ? "" : " (null)");
  if (!aligned16(workspace)) return fail(MX_ERR_ALIGNMENT, "%s: workspace is not 16-byte aligned", fn);
  const Range outputs[2] = {span(lse, static_cast<uint64_t>(rows * q_heads) * 4), span(workspace, need)};
  rc = rows_disjoint(fn, &o, 1, &in, 1, outputs, 2, ranges, 6, false);
  if (rc != MX_OK) return rc;
  DeviceInfo *dev = nullptr;
  rc = device_info(&dev);
  if (rc != MX_OK) return rc;
  if (sequences == 0) return MX_OK;
  a.c.status = dev->status;
  a.q = static_cast<const uint16_t *>(q);
  a.ld_q = ld_q;
  a.q_heads = static_cast<int>(q_heads);
  a.q_tokens = static_cast<int>(q_tokens);
  a.scale = scale;
  a.window = window;
  a.out = static_cast<uint16_t *>(out);
  a.ld_out = ld_out;
  a.lse = lse;
  a.workspace = workspace;
  a.num_sms = dev->num_sms;
  return launch_rc(fn, mx::launch_attention(a, static_cast<cudaStream_t>(stream)));
}

MX_API int mx_sample(const void *logits, int64_t rows, int64_t vocab, int64_t ld, int dtype,
                     const float *temperature, const int32_t *top_k, const float *top_p,
                     const float *min_p, const float *uniform, int32_t *ids, float *probability,
                     void *stream) {
  clear_detail();
  const char *fn = "mx_sample";
  if (!logits || !uniform || !ids)
    return fail(MX_ERR_INVALID_ARG, "%s: %s is null", fn, !logits ? "logits" : !uniform ? "uniform" : "ids");
  if (dtype != MX_OUT_BF16 && dtype != MX_OUT_FP32)
    return fail(MX_ERR_UNSUPPORTED_FEATURE, "%s: dtype %d (MX_OUT_BF16 = 0 or MX_OUT_FP32 = 1)", fn, dtype);
  if (rows < 0 || rows > (1 << 20))
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: rows = %lld (0 .. 2^20)", fn, static_cast<long long>(rows));
  if (vocab < 1 || vocab > MX_SAMPLE_MAX_VOCAB)
    return fail(MX_ERR_UNSUPPORTED_SHAPE, "%s: vocab = %lld (1..%d)", fn, static_cast<long long>(vocab),
                MX_SAMPLE_MAX_VOCAB);
  if (ld < vocab || ld >= (int64_t(1) << 40))
    return fail(MX_ERR_INVALID_ARG, "%s: ld = %lld (>= vocab = %lld, below 2^40)", fn, static_cast<long long>(ld),
                static_cast<long long>(vocab));
  if (!aligned16(logits)) return fail(MX_ERR_ALIGNMENT, "%s: logits is not 16-byte aligned", fn);
  const struct {
    const char *name;
    const void *p;
  } small[7] = {{"temperature", temperature}, {"top_k", top_k}, {"top_p", top_p}, {"min_p", min_p},
                {"uniform", uniform},         {"ids", ids},     {"probability", probability}};
  for (const auto &v : small)
    if (!aligned4(v.p)) return fail(MX_ERR_ALIGNMENT, "%s: %s is not 4-byte aligned", fn, v.name);
  const uint64_t n = static_cast<uint64_t>(rows) * 4;
  const Range in[6] = {span(logits, row_bytes(rows, vocab, ld, dtype == MX_OUT_FP32 ? 4 : 2)),
                       span(temperature, n), span(top_k, n), span(top_p, n), span(min_p, n), span(uniform, n)};
  const Range out[2] = {span(ids, n), span(probability, n)};
  int rc = check_disjoint(fn, out, 2, in, 6);
  if (rc != MX_OK) return rc;
  DeviceInfo *dev = nullptr;
  rc = device_info(&dev);
  if (rc != MX_OK) return rc;
  if (rows == 0) return MX_OK;
  mx::SampleArgs a;
  a.logits = logits;
  a.ld = ld;
  a.rows = static_cast<int>(rows);
  a.vocab = static_cast<int>(vocab);
  a.fp32 = dtype == MX_OUT_FP32;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.uniform = uniform;
  a.ids = ids;
  a.probability = probability;
  a.num_sms = dev->num_sms;
  a.status = dev->status;
  return launch_rc(fn, mx::launch_sample(a, static_cast<cudaStream_t>(stream)));
}

MX_API int mx_device_status(void *stream) {
  clear_detail();
  DeviceInfo *dev = nullptr;
  const int rc = device_info(&dev);
  if (rc != MX_OK) return rc;
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail_cuda("mx_device_status: cudaStreamSynchronize", e);
  uint32_t word = 0;
  e = cudaMemcpy(&word, dev->status, sizeof word, cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return fail_cuda("mx_device_status: reading the status word", e);
  if (word != 0) {
    const uint32_t zero = 0;
    e = cudaMemcpy(dev->status, &zero, sizeof zero, cudaMemcpyHostToDevice);
    if (e != cudaSuccess) return fail_cuda("mx_device_status: clearing the status word", e);
  }
  if (word & mx::kStatusTimeoutBit)
    return fail(MX_ERR_DEVICE_TIMEOUT,
                "mx_device_status: a kernel's bounded wait ran out and it abandoned its work");
  if (word & mx::kStatusBoundsBit)
    return fail(MX_ERR_DEVICE_BOUNDS,
                "mx_device_status: a kernel of the bounds-checked build skipped an access outside "
                "its buffer");
  if (word & mx::kStatusIndexBit)
    return fail(MX_ERR_DEVICE_INDEX,
                "mx_device_status: a page, length or row number in device memory was out of range; "
                "what it names was left out");
  return MX_OK;
}

MX_API int mx_selftest_wait_timeout(uint64_t timeout_ns, void *stream) {
  clear_detail();
  const char *fn = "mx_selftest_wait_timeout";
  if (timeout_ns == 0 || timeout_ns > 10000000000ull)
    return fail(MX_ERR_INVALID_ARG, "%s: timeout_ns = %llu (1 .. 1e10)", fn,
                static_cast<unsigned long long>(timeout_ns));
  DeviceInfo *dev = nullptr;
  const int rc = device_info(&dev);
  if (rc != MX_OK) return rc;
  return launch_rc(fn, mx::launch_wait_selftest(dev->status, timeout_ns,
                                                static_cast<cudaStream_t>(stream)));
}

MX_API int mx_calibrate_mma(int form, int pair, int64_t steps, unsigned long long *cycles,
                            int cycles_capacity, double *flops, int *units, void *stream) {
  clear_detail();
  const char *fn = "mx_calibrate_mma";
  if (form < MX_MMA_MXF4 || form > MX_MMA_MXF4NVF4_4X)
    return fail(MX_ERR_INVALID_ARG, "%s: form %d (MX_MMA_* = 0..2)", fn, form);
  if (pair != 0 && pair != 1) return fail(MX_ERR_INVALID_ARG, "%s: pair = %d (0 or 1)", fn, pair);
  if (steps < 1 || steps > MX_CALIBRATE_MAX_STEPS)
    return fail(MX_ERR_INVALID_ARG, "%s: steps = %lld (1..MX_CALIBRATE_MAX_STEPS)", fn,
                static_cast<long long>(steps));
  if (!flops || !units)
    return fail(MX_ERR_INVALID_ARG, "%s: %s is null", fn, !flops ? "flops" : "units");
  if (cycles && (reinterpret_cast<uintptr_t>(cycles) & 7u))
    return fail(MX_ERR_ALIGNMENT, "%s: cycles is not 8-byte aligned", fn);
  DeviceInfo *dev = nullptr;
  const int rc = device_info(&dev);
  if (rc != MX_OK) return rc;
  if (cycles && cycles_capacity < dev->num_sms)
    return fail(MX_ERR_INVALID_ARG, "%s: cycles_capacity = %d, below the %d SMs", fn,
                cycles_capacity, dev->num_sms);
  int u = 0;
  const cudaError_t e = mx::launch_calibrate_mma(form, pair, steps, cycles, dev->status,
                                                 dev->num_sms, static_cast<cudaStream_t>(stream),
                                                 &u);
  if (e != cudaSuccess) return fail_cuda(fn, e);
  *units = u;
  *flops = static_cast<double>(u) * static_cast<double>(steps) * 4.0 * 2.0 *
           (pair ? 256.0 : 128.0) * 256.0 * 64.0;
  return MX_OK;
}

namespace mx {

namespace {
struct SetupRecord {
  const void *func;
  CUcontext ctx;
  int value;
};
std::mutex g_setup_mutex;
std::vector<SetupRecord> g_setup;  // one per kernel instance and context: a few dozen
}  // namespace

bool encode_codes_window_map(CUtensorMap *tm, const void *codes, int64_t rows, int64_t k,
                             int box_rows) {
  return encode_codes_map(tm, codes, rows, k, box_rows) == MX_OK;
}

bool kernel_setup_get(const void *func, int *value) {
  const CUcontext ctx = current_context();
  if (ctx == nullptr) return false;
  std::lock_guard<std::mutex> lock(g_setup_mutex);
  for (const SetupRecord &r : g_setup) {
    if (r.func == func && r.ctx == ctx) {
      if (value) *value = r.value;
      return true;
    }
  }
  return false;
}

void kernel_setup_put(const void *func, int value) {
  const CUcontext ctx = current_context();
  if (ctx == nullptr) return;
  std::lock_guard<std::mutex> lock(g_setup_mutex);
  for (SetupRecord &r : g_setup) {
    if (r.func == func && r.ctx == ctx) {
      r.value = value;
      return;
    }
  }
  g_setup.push_back(SetupRecord{func, ctx, value});
}

int gemm_static_workspace_call(const void *a_codes, const void *a_scales, const void *b_codes,
                               const void *b_scales, void *d, int64_t m, int64_t n, int64_t k,
                               int layout, int out_dtype, int split_k, void *stream) {
  clear_detail();
  const char *fn = "mxfp4_gemm_static_workspace";
  // every argument check of mxfp4_gemm first, so that the codes match it,
  // then the size of the partials against the array, before the device is
  // touched
  const int arc = gemm_check_args(fn, MX_FMT_MXFP4, a_codes, a_scales, b_codes, b_scales, nullptr,
                                  nullptr, d, m, n, k, layout, out_dtype, split_k, nullptr);
  if (arc != MX_OK) return arc;
  const mx::GemmPlan plan = mx::gemm_plan(m, n, k, split_k, num_sms_or_default());
  const int splits = plan.splits;
  const size_t need = plan.workspace() ? static_cast<size_t>(splits) * static_cast<size_t>(m) *
                                             static_cast<size_t>(n) * sizeof(float)
                                       : 0;
  if (need > static_cast<size_t>(MX_STATIC_WORKSPACE_BYTES))
    return fail(MX_ERR_WORKSPACE,
                "%s: %d splits of K need %zu bytes of partial sums, more than the %u bytes of the "
                "static array",
                fn, splits, need, static_cast<unsigned>(MX_STATIC_WORKSPACE_BYTES));
  DeviceInfo *dev = nullptr;
  const int drc = device_info(&dev);
  if (drc != MX_OK) return drc;
  return gemm_common(fn, MX_FMT_MXFP4, a_codes, a_scales, b_codes, b_scales, nullptr, nullptr, d,
                     m, n, k, layout, out_dtype, split_k, nullptr,
                     need > 0 ? dev->static_ws : nullptr,
                     need > 0 ? static_cast<size_t>(MX_STATIC_WORKSPACE_BYTES) : 0, stream);
}

}  // namespace mx
