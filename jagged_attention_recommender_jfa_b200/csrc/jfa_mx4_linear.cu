// A linear layer over MXFP4 operands: the quantisations and products of its
// forward and backward pass behind one call each.  The launches are those of
// jfa_quantize_mxfp4*, jfa_matmul_mxfp4 on one stream; what the call saves is
// host time, which is what a layer of few tokens takes (a call from Python 2 us
// beside the 2.5 us of its launch).
#include "jfa_common.cuh"
#include "jfa_mx4.cuh"

namespace jfa {
namespace {

bool in_range(int64_t v) { return v >= 0 && v <= kMx4MaxDim; }

size_t operand_bytes(int64_t rows, int64_t cols) { return jfa_mxfp4_code_bytes(rows, cols) + jfa_mxfp4_scale_bytes(rows, cols); }

// An operand's place in the scratch buffer.
struct Operand {
    uint8_t *codes, *scales;
    Operand(uint8_t*& at, int64_t rows, int64_t cols) {
        codes = at;
        scales = codes + jfa_mxfp4_code_bytes(rows, cols);
        at = scales + jfa_mxfp4_scale_bytes(rows, cols);
    }
};

// What both passes ask of their arguments; the pointers of empty tensors are not looked at.
jfa_status check_linear(const char* who, int64_t m, int64_t n, int64_t k, jfa_dtype dtype, jfa_dtype dtype2, int backward,
                        const void* scratch, size_t scratch_bytes, const void* workspace, size_t ws_bytes) {
    if ((dtype != JFA_F32 && dtype != JFA_BF16) || (dtype2 != JFA_F32 && dtype2 != JFA_BF16))
        return set_last_error(JFA_ERR_INVALID_ARGUMENT, "%s: dtypes must be JFA_F32 or JFA_BF16", who);
    if (!in_range(m) || !in_range(n) || !in_range(k))
        return set_last_error(JFA_ERR_INVALID_ARGUMENT, "%s: m, n and k in [0, 2^30]", who);
    if (!workspace || ((uintptr_t)workspace & 15))
        return set_last_error(JFA_ERR_INVALID_ARGUMENT, "%s: workspace must be non-NULL and 16-byte aligned", who);
    if (ws_bytes < jfa_mxfp4_workspace_bytes())
        return set_last_error(JFA_ERR_WORKSPACE, "%s: workspace %zu < %zu bytes", who, ws_bytes, jfa_mxfp4_workspace_bytes());
    const size_t need = jfa_linear_mxfp4_scratch_bytes(m, n, k, backward);
    if (need > 0 && (!scratch || ((uintptr_t)scratch & 15)))
        return set_last_error(JFA_ERR_INVALID_ARGUMENT, "%s: scratch must be non-NULL and 16-byte aligned", who);
    if (scratch_bytes < need)
        return set_last_error(JFA_ERR_WORKSPACE, "%s: scratch %zu < %zu bytes", who, scratch_bytes, need);
    return JFA_OK;
}

jfa_status check_tensor(const char* who, const char* name, const void* p, int64_t rows, int64_t cols) {
    if (rows > 0 && cols > 0 && (!p || ((uintptr_t)p & 15)))
        return set_last_error(JFA_ERR_INVALID_ARGUMENT, "%s: %s must be non-NULL and 16-byte aligned", who, name);
    return JFA_OK;
}

}  // namespace
}  // namespace jfa

extern "C" {

size_t jfa_linear_mxfp4_scratch_bytes(int64_t m, int64_t n, int64_t k, int backward) {
    using namespace jfa;
    if (!in_range(m) || !in_range(n) || !in_range(k)) return 0;
    return backward ? operand_bytes(m, n) + operand_bytes(n, m) + operand_bytes(k, m) : operand_bytes(m, k);
}

jfa_status jfa_linear_mxfp4_forward(const void* x, jfa_dtype dtype, int64_t m, int64_t n, int64_t k, const uint8_t* w_codes,
                                    const uint8_t* w_scales, const float* bias, void* y, void* scratch, size_t scratch_bytes,
                                    void* workspace, size_t ws_bytes, jfa_stream_t stream) {
    using namespace jfa;
    const char* const who = "linear_mxfp4_forward";
    jfa_status s = check_linear(who, m, n, k, dtype, dtype, 0, scratch, scratch_bytes, workspace, ws_bytes);
    if (s == JFA_OK) s = check_tensor(who, "x", x, m, k);
    if (s == JFA_OK && m > 0) s = check_tensor(who, "w_codes", w_codes, n, k);
    if (s == JFA_OK && m > 0) s = check_tensor(who, "w_scales", w_scales, n, k);
    if (s == JFA_OK) s = check_tensor(who, "y", y, m, n);
    if (s != JFA_OK) return s;
    if ((uintptr_t)bias & 3) return set_last_error(JFA_ERR_INVALID_ARGUMENT, "%s: bias must be 4-byte aligned", who);
    if (m == 0 || n == 0) return JFA_OK;
    uint8_t* at = reinterpret_cast<uint8_t*>(scratch);
    const Operand a(at, m, k);
    s = jfa_quantize_mxfp4(x, dtype, m, k, 0, a.codes, a.scales, stream);
    return s != JFA_OK ? s : jfa_matmul_mxfp4(m, n, k, a.codes, a.scales, w_codes, w_scales, bias, y, dtype, 0, workspace,
                                              ws_bytes, stream);
}

jfa_status jfa_linear_mxfp4_backward(const void* dy, jfa_dtype dtype, const void* x, jfa_dtype x_dtype, int64_t m, int64_t n,
                                     int64_t k, const uint8_t* wt_codes, const uint8_t* wt_scales, void* dx, float* dw,
                                     int accumulate, void* scratch, size_t scratch_bytes, void* workspace, size_t ws_bytes,
                                     jfa_stream_t stream) {
    using namespace jfa;
    const char* const who = "linear_mxfp4_backward";
    jfa_status s = check_linear(who, m, n, k, dtype, x_dtype, 1, scratch, scratch_bytes, workspace, ws_bytes);
    if (s == JFA_OK) s = check_tensor(who, "dy", dy, m, n);
    if (s == JFA_OK) s = check_tensor(who, "x", x, m, k);
    if (s == JFA_OK && m > 0) s = check_tensor(who, "wt_codes", wt_codes, k, n);
    if (s == JFA_OK && m > 0) s = check_tensor(who, "wt_scales", wt_scales, k, n);
    if (s == JFA_OK) s = check_tensor(who, "dx", dx, m, k);
    if (s == JFA_OK) s = check_tensor(who, "dw", dw, n, k);
    if (s != JFA_OK) return s;
    uint8_t* at = reinterpret_cast<uint8_t*>(scratch);
    const Operand g(at, m, n), gt(at, n, m), xt(at, k, m);
    if (k == 0) return JFA_OK;   // both results are empty
    s = jfa_quantize_mxfp4_both(dy, dtype, m, n, g.codes, g.scales, gt.codes, gt.scales, stream);
    if (s == JFA_OK)
        s = jfa_matmul_mxfp4(m, k, n, g.codes, g.scales, wt_codes, wt_scales, nullptr, dx, dtype, 0, workspace, ws_bytes, stream);
    if (s == JFA_OK && n > 0) s = jfa_quantize_mxfp4(x, x_dtype, m, k, 1, xt.codes, xt.scales, stream);
    if (s == JFA_OK)
        s = jfa_matmul_mxfp4(n, k, m, gt.codes, gt.scales, xt.codes, xt.scales, nullptr, dw, JFA_F32, accumulate, workspace,
                             ws_bytes, stream);
    return s;
}

}  // extern "C"
