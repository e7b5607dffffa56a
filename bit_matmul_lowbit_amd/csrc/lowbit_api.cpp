// C ABI of liblowbit.so: argument validation on the host, then kernel
// dispatch.  The contract of every entry point is in include/lowbit.h.
#include "../../include/lowbit.h"

#include "common.h"

#include <atomic>

namespace lowbit {

int device_cu_count() {
  // atomics: first calls may race from several host threads (they store the
  // same value)
  static std::atomic<int> cached[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
  int v = cached[dev].load(std::memory_order_relaxed);
  if (v == 0) {
    if (hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
        v <= 0)
      v = 256;
    cached[dev].store(v, std::memory_order_relaxed);
  }
  return v;
}

}  // namespace lowbit

namespace {

constexpr int64_t kMaxElems = int64_t(1) << 40;
constexpr int64_t kMaxK = int64_t(1) << 22;
constexpr int64_t kMaxRows = int64_t(1) << 22;

bool fmt_ok(int fmt) { return fmt == LOWBIT_FMT_Q1_G128 || fmt == LOWBIT_FMT_T2_G128; }

bool shape_ok(int64_t n, int64_t k) {
  if (n < 1 || k < 128 || k % 128 != 0 || k > kMaxK) return false;
  if (n > kMaxElems / k) return false;
  return ((n + 15) / 16) < (int64_t(1) << 31);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool type_ok(int t) { return t == LOWBIT_F32 || t == LOWBIT_F16 || t == LOWBIT_BF16; }

bool aligned_to_elem(const void* p, int type) {
  return (reinterpret_cast<uintptr_t>(p) & (type == LOWBIT_F32 ? 3u : 1u)) == 0;
}

// rows of k elements at stride ld: no overlap, and every offset below 2^40
bool rows_ok(int64_t m, int64_t k, int64_t ld) { return ld >= k && ld <= kMaxElems / m; }

int64_t padded(int64_t n) { return (n + 15) / 16 * 16; }

int hip_status(hipError_t e) { return e == hipSuccess ? LOWBIT_OK : LOWBIT_ERR_HIP; }

bool logits_shape_ok(int64_t n, int64_t b) {
  // the grid's threads (one per 16 logits) stay below 2^32
  return n >= 1 && n <= (int64_t(1) << 31) - 1 && b >= 1 && b <= 65535 && n <= (int64_t(1) << 35) / b;
}

bool lora_shape_ok(int64_t m, int64_t n, int64_t k, int64_t r, int64_t slots) {
  return m >= 1 && m <= kMaxRows && n >= 1 && n <= (int64_t(1) << 31) - 1 && k >= 8 && k <= kMaxK &&
         k % 8 == 0 && r >= 8 && r <= 256 && r % 8 == 0 && slots >= 1 && slots <= 4096 &&
         n <= kMaxElems / m && k <= kMaxElems / m && r * n <= kMaxElems / slots &&
         r * k <= kMaxElems / slots;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace

extern "C" {

int lowbit_version(void) { return 1; }

const char* lowbit_status_str(int status) {
  switch (status) {
    case LOWBIT_OK: return "ok";
    case LOWBIT_ERR_ARG: return "invalid argument (null pointer, format, batch or m)";
    case LOWBIT_ERR_SHAPE: return "invalid shape (n >= 1, k >= 128, k % 128 == 0, size limits)";
    case LOWBIT_ERR_ALIGN: return "pointer not 16-byte aligned";
    case LOWBIT_ERR_UNSUPPORTED: return "unsupported request";
    case LOWBIT_ERR_HIP: return "HIP launch failed";
    case LOWBIT_ERR_WORKSPACE: return "workspace missing or too small";
    case LOWBIT_ERR_SCRATCH: return "request needs more than the static scratch (1 MiB)";
    default: return "unknown status";
  }
}

size_t lowbit_codes_bytes(int fmt, int64_t n, int64_t k) {
  if (!fmt_ok(fmt) || !shape_ok(n, k)) return 0;
  return (size_t)(padded(n) * k / (fmt == LOWBIT_FMT_Q1_G128 ? 8 : 4));
}

size_t lowbit_scales_bytes(int fmt, int64_t n, int64_t k) {
  if (!fmt_ok(fmt) || !shape_ok(n, k)) return 0;
  return (size_t)(padded(n) * (k / 128) * 2);
}

int lowbit_quantize_q1(const uint16_t* w_fp16, int64_t n, int64_t k, void* codes,
                       uint16_t* scales, hipStream_t stream) {
  if (!w_fp16 || !codes || !scales) return LOWBIT_ERR_ARG;
  if (!shape_ok(n, k)) return LOWBIT_ERR_SHAPE;
  if (!aligned16(w_fp16) || !aligned16(codes) || !aligned16(scales)) return LOWBIT_ERR_ALIGN;
  return hip_status(lowbit::launch_quantize_q1(w_fp16, n, k, static_cast<uint8_t*>(codes),
                                               scales, stream));
}

int lowbit_pack_t2(const int8_t* t, const uint16_t* s_fp16, int64_t n, int64_t k, void* codes,
                   uint16_t* scales, hipStream_t stream) {
  if (!t || !s_fp16 || !codes || !scales) return LOWBIT_ERR_ARG;
  if (!shape_ok(n, k)) return LOWBIT_ERR_SHAPE;
  // t rows are read 8 bytes at a time; s is read element-wise
  if (!aligned16(t) || !aligned16(codes) || !aligned16(scales) ||
      (reinterpret_cast<uintptr_t>(s_fp16) & 1u))
    return LOWBIT_ERR_ALIGN;
  return hip_status(lowbit::launch_pack_t2(t, s_fp16, n, k, static_cast<uint8_t*>(codes), scales,
                                           stream));
}

int lowbit_pack(int fmt, const void* src, const uint16_t* src_scales, int64_t n, int64_t k,
                void* codes, uint16_t* scales, hipStream_t stream) {
  if (fmt == LOWBIT_FMT_Q1_G128) {
    if (src_scales) return LOWBIT_ERR_ARG;
    return lowbit_quantize_q1(static_cast<const uint16_t*>(src), n, k, codes, scales, stream);
  }
  if (fmt == LOWBIT_FMT_T2_G128)
    return lowbit_pack_t2(static_cast<const int8_t*>(src), src_scales, n, k, codes, scales,
                          stream);
  return LOWBIT_ERR_ARG;
}

int lowbit_unpack(int fmt, const void* codes, const uint16_t* scales, int64_t n, int64_t k,
                  uint16_t* w_fp16, hipStream_t stream) {
  if (!fmt_ok(fmt) || !codes || !scales || !w_fp16) return LOWBIT_ERR_ARG;
  if (!shape_ok(n, k)) return LOWBIT_ERR_SHAPE;
  if (!aligned16(codes) || !aligned16(scales) || !aligned16(w_fp16)) return LOWBIT_ERR_ALIGN;
  return hip_status(lowbit::launch_unpack(fmt, static_cast<const uint8_t*>(codes), scales, n, k,
                                          w_fp16, stream));
}

size_t lowbit_gemv_workspace_bytes(int fmt, int64_t n, int64_t k, int64_t b) {
  if (!fmt_ok(fmt) || !shape_ok(n, k) || b < 1 || b > 8) return 0;
  return lowbit::gemv_workspace_bytes(k, b);
}

int lowbit_gemv_prepare(int64_t n, int64_t k, const uint16_t* x_fp16, int64_t b, float* y_f32,
                        void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!x_fp16 || !y_f32) return LOWBIT_ERR_ARG;
  if (b < 1 || b > 8) return LOWBIT_ERR_ARG;
  if (!shape_ok(n, k)) return LOWBIT_ERR_SHAPE;
  if (!aligned16(x_fp16) || !aligned16(y_f32)) return LOWBIT_ERR_ALIGN;
  if (!workspace || workspace_bytes < lowbit::gemv_workspace_bytes(k, b))
    return LOWBIT_ERR_WORKSPACE;
  if (!aligned16(workspace)) return LOWBIT_ERR_ALIGN;
  return hip_status(lowbit::launch_gemv_prepare(n, k, x_fp16, b, y_f32, workspace, stream));
}

int lowbit_gemv_accumulate(int fmt, const void* codes, const uint16_t* scales, int64_t n,
                           int64_t k, int64_t b, float* y_f32, const void* workspace,
                           size_t workspace_bytes, hipStream_t stream) {
  if (!fmt_ok(fmt) || !codes || !scales || !y_f32) return LOWBIT_ERR_ARG;
  if (b < 1 || b > 8) return LOWBIT_ERR_ARG;
  if (!shape_ok(n, k)) return LOWBIT_ERR_SHAPE;
  if (!aligned16(codes) || !aligned16(scales) || !aligned16(y_f32)) return LOWBIT_ERR_ALIGN;
  if (!workspace || workspace_bytes < lowbit::gemv_workspace_bytes(k, b))
    return LOWBIT_ERR_WORKSPACE;
  if (!aligned16(workspace)) return LOWBIT_ERR_ALIGN;
  return hip_status(lowbit::launch_gemv_accumulate(fmt, static_cast<const uint8_t*>(codes),
                                                   scales, n, k, b, y_f32, workspace, stream));
}

int lowbit_gemv(int fmt, const void* codes, const uint16_t* scales, int64_t n, int64_t k,
                const uint16_t* x_fp16, int64_t b, float* y_f32, void* workspace,
                size_t workspace_bytes, hipStream_t stream) {
  if (!fmt_ok(fmt) || !codes || !scales || !x_fp16 || !y_f32) return LOWBIT_ERR_ARG;
  if (b < 1 || b > 8) return LOWBIT_ERR_ARG;
  if (!shape_ok(n, k)) return LOWBIT_ERR_SHAPE;
  if (!aligned16(codes) || !aligned16(scales) || !aligned16(x_fp16) || !aligned16(y_f32))
    return LOWBIT_ERR_ALIGN;
  if (!workspace || workspace_bytes < lowbit::gemv_workspace_bytes(k, b))
    return LOWBIT_ERR_WORKSPACE;
  if (!aligned16(workspace)) return LOWBIT_ERR_ALIGN;
  // small matrices: one kernel writes y (the workspace is not touched)
  if (lowbit::gemv_direct_ok(n, k, b))
    return hip_status(lowbit::launch_gemv_direct(fmt, static_cast<const uint8_t*>(codes), scales,
                                                 n, k, x_fp16, b, y_f32, stream));
  const int st = lowbit_gemv_prepare(n, k, x_fp16, b, y_f32, workspace, workspace_bytes, stream);
  if (st != LOWBIT_OK) return st;
  return lowbit_gemv_accumulate(fmt, codes, scales, n, k, b, y_f32, workspace, workspace_bytes,
                                stream);
}

int lowbit_gemv_noalloc(int fmt, const void* codes, const uint16_t* scales, int64_t n,
                        int64_t k, const uint16_t* x_fp16, int64_t b, float* y_f32,
                        hipStream_t stream) {
  if (!fmt_ok(fmt) || !codes || !scales || !x_fp16 || !y_f32) return LOWBIT_ERR_ARG;
  if (b < 1 || b > 8) return LOWBIT_ERR_ARG;
  if (!shape_ok(n, k)) return LOWBIT_ERR_SHAPE;
  if (!aligned16(codes) || !aligned16(scales) || !aligned16(x_fp16) || !aligned16(y_f32))
    return LOWBIT_ERR_ALIGN;
  if (lowbit::gemv_workspace_bytes(k, b) > lowbit::gemv_noalloc_scratch_bytes())
    return LOWBIT_ERR_SCRATCH;
  return hip_status(lowbit::launch_gemv_noalloc(fmt, static_cast<const uint8_t*>(codes), scales,
                                                n, k, x_fp16, b, y_f32, stream));
}

static int gemm_common(int fmt, const void* codes, const uint16_t* scales, int64_t n, int64_t k,
                       const uint16_t* x_bf16, int64_t m, void* y, bool out_f32,
                       hipStream_t stream) {
  if (!fmt_ok(fmt) || !codes || !scales || !x_bf16 || !y) return LOWBIT_ERR_ARG;
  if (m < 1 || m > (int64_t(1) << 22)) return LOWBIT_ERR_ARG;
  if (!shape_ok(n, k)) return LOWBIT_ERR_SHAPE;
  if (m > kMaxElems / k || m > kMaxElems / n) return LOWBIT_ERR_SHAPE;
  if (!aligned16(codes) || !aligned16(scales) || !aligned16(x_bf16) || !aligned16(y))
    return LOWBIT_ERR_ALIGN;
  return hip_status(lowbit::launch_gemm(fmt, static_cast<const uint8_t*>(codes), scales, n, k,
                                        x_bf16, m, y, out_f32, stream));
}

int lowbit_gemm(int fmt, const void* codes, const uint16_t* scales, int64_t n, int64_t k,
                const uint16_t* x_bf16, int64_t m, uint16_t* y_bf16, hipStream_t stream) {
  return gemm_common(fmt, codes, scales, n, k, x_bf16, m, y_bf16, false, stream);
}

int lowbit_gemm_f32(int fmt, const void* codes, const uint16_t* scales, int64_t n, int64_t k,
                    const uint16_t* x_bf16, int64_t m, float* y_f32, hipStream_t stream) {
  return gemm_common(fmt, codes, scales, n, k, x_bf16, m, y_f32, true, stream);
}

int lowbit_silu_mul(const float* h_f32, int64_t f, int64_t b, uint16_t* z_fp16,
                    hipStream_t stream) {
  if (!h_f32 || !z_fp16) return LOWBIT_ERR_ARG;
  if (b < 1 || b > (int64_t(1) << 20)) return LOWBIT_ERR_ARG;
  if (f < 8 || f % 8 != 0 || f > kMaxElems / (2 * b)) return LOWBIT_ERR_SHAPE;
  if (!aligned16(h_f32) || !aligned16(z_fp16)) return LOWBIT_ERR_ALIGN;
  return hip_status(lowbit::launch_silu_mul(h_f32, f, b, z_fp16, stream));
}

size_t lowbit_ffn_workspace_bytes(int fmt, int64_t k, int64_t f, int64_t b) {
  if (!fmt_ok(fmt) || f < 1 || f > kMaxElems || !shape_ok(2 * f, k) || !shape_ok(k, f) ||
      b < 1 || b > 8)
    return 0;
  return lowbit::ffn_workspace_bytes(k, f, b);
}

int lowbit_ffn(int fmt, const void* gu_codes, const uint16_t* gu_scales, const void* dn_codes,
               const uint16_t* dn_scales, int64_t k, int64_t f, const uint16_t* x_fp16,
               int64_t b, float* y_f32, void* workspace, size_t workspace_bytes,
               hipStream_t stream) {
  if (!fmt_ok(fmt) || !gu_codes || !gu_scales || !dn_codes || !dn_scales || !x_fp16 || !y_f32)
    return LOWBIT_ERR_ARG;
  if (b < 1 || b > 8) return LOWBIT_ERR_ARG;
  if (f < 1 || f > kMaxElems || !shape_ok(2 * f, k) || !shape_ok(k, f)) return LOWBIT_ERR_SHAPE;
  if (!aligned16(gu_codes) || !aligned16(gu_scales) || !aligned16(dn_codes) ||
      !aligned16(dn_scales) || !aligned16(x_fp16) || !aligned16(y_f32))
    return LOWBIT_ERR_ALIGN;
  if (!workspace || workspace_bytes < lowbit::ffn_workspace_bytes(k, f, b))
    return LOWBIT_ERR_WORKSPACE;
  if (!aligned16(workspace)) return LOWBIT_ERR_ALIGN;
  return hip_status(lowbit::launch_ffn(fmt, static_cast<const uint8_t*>(gu_codes), gu_scales,
                                       static_cast<const uint8_t*>(dn_codes), dn_scales, k, f,
                                       x_fp16, b, y_f32, workspace, stream));
}

int lowbit_embed(int fmt, const void* codes, const uint16_t* scales, int64_t n, int64_t k,
                 const int32_t* ids, int64_t count, uint16_t* out_fp16, hipStream_t stream) {
  if (!fmt_ok(fmt) || !codes || !scales || !ids || !out_fp16) return LOWBIT_ERR_ARG;
  if (count < 1 || count > (int64_t(1) << 31) - 1) return LOWBIT_ERR_ARG;
  if (!shape_ok(n, k) || n > (int64_t(1) << 31) - 1) return LOWBIT_ERR_SHAPE;
  if (count > kMaxElems / k) return LOWBIT_ERR_SHAPE;
  if (!aligned16(codes) || !aligned16(out_fp16) || (reinterpret_cast<uintptr_t>(scales) & 1u) ||
      (reinterpret_cast<uintptr_t>(ids) & 3u))
    return LOWBIT_ERR_ALIGN;
  return hip_status(lowbit::launch_embed(fmt, static_cast<const uint8_t*>(codes), scales, n, k,
                                         ids, count, out_fp16, stream));
}

size_t lowbit_argmax_workspace_bytes(int64_t n, int64_t b) {
  if (n < 1 || n > (int64_t(1) << 31) - 1 || b < 1 || b > 65535) return 0;
  return lowbit::argmax_workspace_bytes(n, b);
}

int lowbit_argmax(const float* y_f32, int64_t n, int64_t b, int32_t* idx_out, float* val_out,
                  void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!y_f32 || !idx_out) return LOWBIT_ERR_ARG;
  if (b < 1 || b > 65535) return LOWBIT_ERR_ARG;
  if (n < 1 || n > (int64_t(1) << 31) - 1 || n > kMaxElems / b) return LOWBIT_ERR_SHAPE;
  if ((reinterpret_cast<uintptr_t>(y_f32) & 3u) || (reinterpret_cast<uintptr_t>(idx_out) & 3u) ||
      (reinterpret_cast<uintptr_t>(val_out) & 3u))
    return LOWBIT_ERR_ALIGN;
  if (!workspace || workspace_bytes < lowbit::argmax_workspace_bytes(n, b))
    return LOWBIT_ERR_WORKSPACE;
  if (!aligned16(workspace)) return LOWBIT_ERR_ALIGN;
  return hip_status(lowbit::launch_argmax(y_f32, n, b, idx_out, val_out, workspace, stream));
}

size_t lowbit_lm_head_workspace_bytes(int fmt, int64_t n, int64_t k, int64_t b) {
  if (!fmt_ok(fmt) || !shape_ok(n, k) || n > (int64_t(1) << 31) - 1 || b < 1 || b > 8) return 0;
  return lowbit::lm_head_workspace_bytes(n, k, b);
}

int lowbit_lm_head(int fmt, const void* codes, const uint16_t* scales, int64_t n, int64_t k,
                   const uint16_t* x_fp16, int64_t b, float* y_f32, int32_t* idx_out,
                   float* val_out, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!fmt_ok(fmt) || !codes || !scales || !x_fp16 || !y_f32 || !idx_out) return LOWBIT_ERR_ARG;
  if (b < 1 || b > 8) return LOWBIT_ERR_ARG;
  if (!shape_ok(n, k) || n > (int64_t(1) << 31) - 1) return LOWBIT_ERR_SHAPE;
  if (!aligned16(codes) || !aligned16(scales) || !aligned16(x_fp16) || !aligned16(y_f32) ||
      (reinterpret_cast<uintptr_t>(idx_out) & 3u) || (reinterpret_cast<uintptr_t>(val_out) & 3u))
    return LOWBIT_ERR_ALIGN;
  if (!workspace || workspace_bytes < lowbit::lm_head_workspace_bytes(n, k, b))
    return LOWBIT_ERR_WORKSPACE;
  if (!aligned16(workspace)) return LOWBIT_ERR_ALIGN;
  return hip_status(lowbit::launch_lm_head(fmt, static_cast<const uint8_t*>(codes), scales, n, k,
                                           x_fp16, b, y_f32, idx_out, val_out, workspace,
                                           stream));
}

int lowbit_quantize_t2(const uint16_t* w_fp16, int64_t n, int64_t k, void* codes,
                       uint16_t* scales, hipStream_t stream) {
  if (!w_fp16 || !codes || !scales) return LOWBIT_ERR_ARG;
  if (!shape_ok(n, k)) return LOWBIT_ERR_SHAPE;
  if (!aligned16(w_fp16) || !aligned16(codes) || !aligned16(scales)) return LOWBIT_ERR_ALIGN;
  return hip_status(lowbit::launch_quantize_t2(w_fp16, n, k, static_cast<uint8_t*>(codes),
                                               scales, stream));
}

size_t lowbit_base3_bytes(int64_t n, int64_t k) {
  if (!shape_ok(n, k)) return 0;
  return (size_t)(n * ((k + 4) / 5));
}

int lowbit_t2_to_base3(const void* codes, const uint16_t* scales, int64_t n, int64_t k,
                       uint8_t* base3_out, uint16_t* scales_out, hipStream_t stream) {
  if (!codes || !scales || !base3_out || !scales_out) return LOWBIT_ERR_ARG;
  if (!shape_ok(n, k)) return LOWBIT_ERR_SHAPE;
  if (!aligned16(codes) || (reinterpret_cast<uintptr_t>(scales) & 1u) ||
      (reinterpret_cast<uintptr_t>(scales_out) & 1u))
    return LOWBIT_ERR_ALIGN;
  return hip_status(lowbit::launch_t2_to_base3(static_cast<const uint8_t*>(codes), scales, n, k,
                                               base3_out, scales_out, stream));
}

int lowbit_base3_to_t2(const uint8_t* base3, const uint16_t* scales_rm, int64_t n, int64_t k,
                       void* codes, uint16_t* scales, hipStream_t stream) {
  if (!base3 || !scales_rm || !codes || !scales) return LOWBIT_ERR_ARG;
  if (!shape_ok(n, k)) return LOWBIT_ERR_SHAPE;
  if (!aligned16(codes) || (reinterpret_cast<uintptr_t>(scales) & 1u) ||
      (reinterpret_cast<uintptr_t>(scales_rm) & 1u))
    return LOWBIT_ERR_ALIGN;
  return hip_status(lowbit::launch_base3_to_t2(base3, scales_rm, n, k,
                                               static_cast<uint8_t*>(codes), scales, stream));
}

int lowbit_norm_residual(const void* y, int y_type, int64_t ldy, const void* r, int r_type,
                         int64_t ldr, void* r_out, int64_t ldro, void* x_out, int x_type,
                         int64_t ldx, int64_t m, int64_t k, int post, const float* post_w,
                         const float* post_b, const void* gate, int gate_type, int64_t ldg,
                         float scale, int pre, const float* pre_w, const float* pre_b, float eps,
                         hipStream_t stream) {
  if (!r || (!r_out && !x_out) || !type_ok(r_type)) return LOWBIT_ERR_ARG;
  if (y && (!type_ok(y_type) || post < LOWBIT_NORM_NONE || post > LOWBIT_NORM_LAYER))
    return LOWBIT_ERR_ARG;
  if (x_out && (!type_ok(x_type) || pre < LOWBIT_NORM_NONE || pre > LOWBIT_NORM_LAYER))
    return LOWBIT_ERR_ARG;
  if (y && gate && !type_ok(gate_type)) return LOWBIT_ERR_ARG;
  if (!(eps >= 0.0f)) return LOWBIT_ERR_ARG;
  // a work-group of up to 1024 threads per row: the grid's threads stay below 2^32
  if (m < 1 || m > kMaxRows / 2 || k < 1 || k > kMaxK) return LOWBIT_ERR_SHAPE;
  if (!rows_ok(m, k, ldr) || (y && !rows_ok(m, k, ldy)) || (r_out && !rows_ok(m, k, ldro)) ||
      (x_out && !rows_ok(m, k, ldx)) || (y && gate && ldg != 0 && !rows_ok(m, k, ldg)))
    return LOWBIT_ERR_SHAPE;
  // in place means row on row: another stride would write rows not yet read
  if (r_out == r && ldro != ldr && m > 1) return LOWBIT_ERR_ARG;
  if (x_out && (x_out == r || x_out == y || x_out == r_out)) return LOWBIT_ERR_ARG;
  if (r_out && r_out == y) return LOWBIT_ERR_ARG;
  if (!aligned_to_elem(r, r_type) || (y && !aligned_to_elem(y, y_type)) ||
      (r_out && !aligned_to_elem(r_out, r_type)) || (x_out && !aligned_to_elem(x_out, x_type)) ||
      (y && gate && !aligned_to_elem(gate, gate_type)) || !aligned_to_elem(post_w, LOWBIT_F32) ||
      !aligned_to_elem(post_b, LOWBIT_F32) || !aligned_to_elem(pre_w, LOWBIT_F32) ||
      !aligned_to_elem(pre_b, LOWBIT_F32))
    return LOWBIT_ERR_ALIGN;
  lowbit::NormArgs a = {};
  a.y = y;
  a.r = r;
  a.r_out = r_out;
  a.x_out = x_out;
  // what is not used is cleared, so that the kernels see one form of it
  a.post = y ? post : LOWBIT_NORM_NONE;
  a.pre = x_out ? pre : LOWBIT_NORM_NONE;
  a.post_w = a.post ? post_w : nullptr;
  a.post_b = a.post ? post_b : nullptr;
  a.pre_w = a.pre ? pre_w : nullptr;
  a.pre_b = a.pre ? pre_b : nullptr;
  a.gate = y ? gate : nullptr;
  a.ldy = ldy;
  a.ldr = ldr;
  a.ldro = ldro;
  a.ldx = ldx;
  a.ldg = ldg;
  a.m = m;
  a.k = k;
  a.y_type = y ? y_type : r_type;
  a.r_type = r_type;
  a.x_type = x_out ? x_type : LOWBIT_F32;
  a.gate_type = a.gate ? gate_type : LOWBIT_F32;
  a.scale = scale;
  a.eps = eps;
  return hip_status(lowbit::launch_norm_residual(a, stream));
}

size_t lowbit_logits_workspace_bytes(int64_t n, int64_t b) {
  return logits_shape_ok(n, b) ? lowbit::logits_workspace_bytes(n, b) : 0;
}

int lowbit_logits_process(const void* y, int y_type, int64_t ldy, int64_t n, int64_t b,
                          const int32_t* tokens, int64_t tcap, int64_t ldt,
                          const int32_t* prompt_len, const int32_t* total_len,
                          const float* repetition, const float* frequency, const float* presence,
                          const int32_t* bias_ids, const float* bias_vals, int64_t bcap, int64_t ldb,
                          const int32_t* bias_len, const int32_t* mask, int64_t mask_rows,
                          int64_t ldm, const int32_t* mask_row, float* out, int64_t ldo,
                          int32_t* idx, float* val, void* workspace, size_t workspace_bytes,
                          hipStream_t stream) {
  if (!y || !type_ok(y_type) || (!out && !idx) || (val && !idx)) return LOWBIT_ERR_ARG;
  if (!bias_ids != !bias_vals) return LOWBIT_ERR_ARG;
  if (!logits_shape_ok(n, b) || !rows_ok(b, n, ldy) || (out && !rows_ok(b, n, ldo)))
    return LOWBIT_ERR_SHAPE;
  constexpr int64_t kMaxList = int64_t(1) << 30;
  if (tokens && (tcap < 0 || tcap >= kMaxList || !rows_ok(b, tcap, ldt))) return LOWBIT_ERR_SHAPE;
  // where many ids fall together the list is walked for every 256 tokens: a bound on that work
  constexpr int64_t kMaxBiases = 16384;
  if (bias_ids && (bcap < 0 || bcap > kMaxBiases || !rows_ok(b, bcap, ldb))) return LOWBIT_ERR_SHAPE;
  if (mask) {
    if (mask_rows < 1 || mask_rows > kMaxElems || !rows_ok(mask_rows, (n + 31) / 32, ldm))
      return LOWBIT_ERR_SHAPE;
  }
  // in place means row on row, in one type
  if (out && out == y && (y_type != LOWBIT_F32 || (ldo != ldy && b > 1))) return LOWBIT_ERR_ARG;
  if (!aligned_to_elem(y, y_type) || !aligned4(tokens) || !aligned4(prompt_len) ||
      !aligned4(total_len) || !aligned4(repetition) || !aligned4(frequency) || !aligned4(presence) ||
      !aligned4(bias_ids) || !aligned4(bias_vals) || !aligned4(bias_len) || !aligned4(mask) ||
      !aligned4(mask_row) || !aligned4(out) || !aligned4(idx) || !aligned4(val))
    return LOWBIT_ERR_ALIGN;
  if (idx) {
    if (!workspace || workspace_bytes < lowbit::logits_workspace_bytes(n, b))
      return LOWBIT_ERR_WORKSPACE;
    if (!aligned16(workspace)) return LOWBIT_ERR_ALIGN;
  }
  lowbit::LogitsArgs a = {};
  a.y = y;
  // an empty list is no list
  if (tokens && tcap > 0) {
    a.tokens = tokens;
    a.prompt_len = prompt_len;
    a.total_len = total_len;
    a.tcap = tcap;
    a.ldt = ldt;
  }
  a.repetition = repetition;
  a.frequency = frequency;
  a.presence = presence;
  if (bias_ids && bcap > 0) {
    a.bias_ids = bias_ids;
    a.bias_vals = bias_vals;
    a.bias_len = bias_len;
    a.bcap = bcap;
    a.ldb = ldb;
  }
  a.mask = mask;
  a.mask_row = mask_row;
  a.mask_rows = mask_rows;
  a.ldm = ldm;
  a.out = out;
  a.ldo = ldo;
  a.idx = idx;
  a.val = val;
  a.y_type = y_type;
  a.ldy = ldy;
  a.n = n;
  a.b = b;
  return hip_status(lowbit::launch_logits_process(a, workspace, stream));
}

size_t lowbit_lora_workspace_bytes(int64_t m, int64_t n, int64_t k, int64_t r, int64_t slots) {
  return lora_shape_ok(m, n, k, r, slots) ? lowbit::lora_workspace_bytes(m, n, k, r, slots) : 0;
}

int lowbit_lora_accumulate(const void* x, int x_type, int64_t ldx, const int32_t* ids, int64_t m,
                           int64_t n, int64_t k, int64_t r, int64_t slots, const void* a,
                           const void* b, const int32_t* ranks, const float* scales, void* y,
                           int y_type, int64_t ldy, void* workspace, size_t workspace_bytes,
                           hipStream_t stream) {
  if (!x || !ids || !a || !b || !y) return LOWBIT_ERR_ARG;
  if (x_type != LOWBIT_F16 && x_type != LOWBIT_BF16) return LOWBIT_ERR_ARG;
  if (y_type != LOWBIT_F32 && !(y_type == LOWBIT_BF16 && x_type == LOWBIT_BF16)) return LOWBIT_ERR_ARG;
  if (!lora_shape_ok(m, n, k, r, slots) || !rows_ok(m, k, ldx) || !rows_ok(m, n, ldy))
    return LOWBIT_ERR_SHAPE;
  if (!aligned16(x) || ldx % 8 != 0 || !aligned16(a) || !aligned16(b) || !aligned4(ids) ||
      !aligned4(ranks) || !aligned4(scales) || !aligned_to_elem(y, y_type))
    return LOWBIT_ERR_ALIGN;
  if (!workspace || workspace_bytes < lowbit::lora_workspace_bytes(m, n, k, r, slots))
    return LOWBIT_ERR_WORKSPACE;
  if (!aligned16(workspace)) return LOWBIT_ERR_ALIGN;
  lowbit::LoraArgs q = {};
  q.x = x;
  q.ids = ids;
  q.a = a;
  q.b = b;
  q.ranks = ranks;
  q.scales = scales;
  q.y = y;
  q.ldx = ldx;
  q.ldy = ldy;
  q.m = m;
  q.n = n;
  q.k = k;
  q.r = r;
  q.slots = slots;
  q.x_type = x_type;
  q.y_type = y_type;
  return hip_status(lowbit::launch_lora_accumulate(q, workspace, stream));
}

}  // extern "C"
