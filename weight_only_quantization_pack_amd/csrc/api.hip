// C ABI of libawq: argument validation on the host, then dispatch to the
// kernel launchers.  Nothing here touches the GPU before every argument has
// been checked, so invalid calls never launch and never write an output.
#include "cache.h"

#include <math.h>
#include <mutex>

namespace {

constexpr int kMaxGemvM = 16;
constexpr int kMaxT = 8192;        // exact fp64 |x| sums need T < 2^13
constexpr int kMaxAlpha = 64;

int check_ptr(const void* p) {
    if (p == nullptr) return AWQ_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(p) & 15u) return AWQ_ERR_ALIGN;
    return AWQ_OK;
}

// First non-OK status of a list of required pointers; NULL errors are
// reported before alignment errors.
int check_ptrs(std::initializer_list<const void*> ps) {
    for (const void* p : ps) if (p == nullptr) return AWQ_ERR_NULL;
    for (const void* p : ps) if (check_ptr(p) != AWQ_OK) return AWQ_ERR_ALIGN;
    return AWQ_OK;
}

int check_quant_params(int bits, int group_size, int zero_point) {
    if (bits != 3 && bits != 4) return AWQ_ERR_UNSUPPORTED;
    if (group_size != 128 && group_size != 64) return AWQ_ERR_UNSUPPORTED;
    if (zero_point != 0 && zero_point != 1) return AWQ_ERR_UNSUPPORTED;
    return AWQ_OK;
}

int check_nk(int N, int K) {
    if (N < 0 || K <= 0) return AWQ_ERR_SHAPE;
    if (K % awq::kGroup != 0) return AWQ_ERR_SHAPE;
    return AWQ_OK;
}

awq_status hip_status(int err) { return err == 0 ? AWQ_OK : AWQ_ERR_HIP; }

// the checks above return awq_status values as int
awq_status as_status(int st) { return static_cast<awq_status>(st); }
static_assert(sizeof(awq_status) == sizeof(int), "awq_status is passed as a C int");

}  // namespace

extern "C" {

const char* awq_status_str(awq_status status) {
    switch (status) {
        case AWQ_OK: return "AWQ_OK";
        case AWQ_ERR_NULL: return "AWQ_ERR_NULL";
        case AWQ_ERR_SHAPE: return "AWQ_ERR_SHAPE";
        case AWQ_ERR_UNSUPPORTED: return "AWQ_ERR_UNSUPPORTED";
        case AWQ_ERR_ALIGN: return "AWQ_ERR_ALIGN";
        case AWQ_ERR_WORKSPACE: return "AWQ_ERR_WORKSPACE";
        case AWQ_ERR_HIP: return "AWQ_ERR_HIP";
        default: return "AWQ_ERR_UNKNOWN";
    }
}

int awq_pack_format_version(void) { return 3; }

size_t awq_packed_words_per_row(int K, int bits) {
    if (K <= 0) return 0;
    if (bits == 4) return (size_t)K / 8;
    if (bits == 3) return 3 * ((size_t)K / 32);
    return 0;
}

size_t awq_packed_words(int N, int K, int bits) {
    if (N < 0) return 0;
    return 16 * (((size_t)N + 15) / 16) * awq_packed_words_per_row(K, bits);
}

awq_status awq_quantize_pack(const void* W, const float* s, int N, int K, int bits, int group_size,
                      int zero_point, void* qweight, void* scales, void* zeros, hipStream_t stream) {
    int st = check_quant_params(bits, group_size, zero_point);
    if (st) return as_status(st);
    if ((st = check_nk(N, K))) return as_status(st);
    if (N == 0) return AWQ_OK;
    if ((st = check_ptrs({W, qweight, scales, zeros}))) return as_status(st);
    if (s != nullptr && (st = check_ptr(s))) return as_status(st);
    return hip_status(awq::launch_quantize_pack(W, s, N, K, bits, group_size, zero_point, qweight, scales, zeros,
                                                stream));
}

awq_status awq_dequantize(const void* qweight, const void* scales, const void* zeros, void* W_hat, int N,
                   int K, int bits, int group_size, hipStream_t stream) {
    int st = check_quant_params(bits, group_size, 1);
    if (st) return as_status(st);
    if ((st = check_nk(N, K))) return as_status(st);
    if ((long long)N * K >= (1LL << 40)) return AWQ_ERR_SHAPE;
    if (N == 0) return AWQ_OK;
    if ((st = check_ptrs({qweight, scales, zeros, W_hat}))) return as_status(st);
    return hip_status(awq::launch_dequantize(qweight, scales, zeros, W_hat, N, K, bits, group_size,
                                             stream));
}

awq_status awq_scale_activations(const void* x, const float* s, void* x_out, int M, int K, hipStream_t stream) {
    if (M < 0 || K <= 0 || K % awq::kGroup != 0) return AWQ_ERR_SHAPE;
    if (M == 0) return AWQ_OK;
    int st = check_ptrs({x, s, x_out});
    if (st) return as_status(st);
    return hip_status(awq::launch_scale_activations(x, s, x_out, M, K, stream));
}

size_t awq_search_workspace_bytes(int T, int N, int K, int n_alpha) {
    if (T <= 0 || N <= 0 || K <= 0 || n_alpha <= 0) return 0;
    return awq::search_workspace_bytes(T, N, K, n_alpha, false);
}

size_t awq_search_workspace_bytes_fused(int T, int N, int K, int n_alpha) {
    if (T <= 0 || N <= 0 || K <= 0 || n_alpha <= 0) return 0;
    return awq::search_workspace_bytes(T, N, K, n_alpha, true);
}

namespace {
// the search path a workspace of this size takes: 0 = D buffered (the
// default), 1 = fused loss, -1 = too small for either
int search_path(int T, int N, int K, int n_alpha, size_t workspace_bytes) {
    if (workspace_bytes >= awq::search_workspace_bytes(T, N, K, n_alpha, false)) return 0;
    if (workspace_bytes >= awq::search_workspace_bytes(T, N, K, n_alpha, true)) return 1;
    return -1;
}
}  // namespace

awq_status awq_search_scale(const void* W, const void* X_cal, int T, int N, int K, const float* alphas,
                     int n_alpha, int bits, int group_size, int zero_point, float* s_out,
                     float* loss_out, int* best_out, void* workspace, size_t workspace_bytes,
                     hipStream_t stream) {
    int st = check_quant_params(bits, group_size, zero_point);
    if (st) return as_status(st);
    if (n_alpha < 1 || n_alpha > kMaxAlpha) return AWQ_ERR_UNSUPPORTED;
    if (T > kMaxT) return AWQ_ERR_UNSUPPORTED;
    if (T <= 0 || N <= 0) return AWQ_ERR_SHAPE;
    if ((st = check_nk(N, K))) return as_status(st);
    if ((long long)T * K >= (1LL << 31)) return AWQ_ERR_SHAPE;   // 32-bit offsets into X_cal
    if (alphas == nullptr) return AWQ_ERR_NULL;
    if ((st = check_ptrs({W, X_cal, s_out, workspace}))) return as_status(st);
    if (loss_out != nullptr && (st = check_ptr(loss_out))) return as_status(st);
    if (best_out != nullptr && (st = check_ptr(best_out))) return as_status(st);
    const int path = search_path(T, N, K, n_alpha, workspace_bytes);
    if (path < 0) return AWQ_ERR_WORKSPACE;
    return hip_status(awq::launch_search(&W, &N, 1, X_cal, T, K, alphas, n_alpha, bits, group_size,
                                         zero_point, s_out, loss_out, best_out, workspace,
                                         path == 1, stream));
}

awq_status awq_search_scale_shared(const void* const* Ws, const int* Ns, int n_layers, const void* X_cal,
                            int T, int K, const float* alphas, int n_alpha, int bits, int group_size,
                            int zero_point, float* s_out, float* loss_out, int* best_out,
                            void* workspace, size_t workspace_bytes, hipStream_t stream) {
    int st = check_quant_params(bits, group_size, zero_point);
    if (st) return as_status(st);
    if (n_alpha < 1 || n_alpha > kMaxAlpha) return AWQ_ERR_UNSUPPORTED;
    if (n_layers < 1 || n_layers > awq::kMaxSearchLayers) return AWQ_ERR_UNSUPPORTED;
    if (T > kMaxT) return AWQ_ERR_UNSUPPORTED;
    if (Ws == nullptr || Ns == nullptr || alphas == nullptr) return AWQ_ERR_NULL;
    long long N = 0;
    for (int l = 0; l < n_layers; ++l) {
        if (Ns[l] <= 0) return AWQ_ERR_SHAPE;
        N += Ns[l];
    }
    if (T <= 0 || N > (1LL << 30)) return AWQ_ERR_SHAPE;
    if ((st = check_nk((int)N, K))) return as_status(st);
    if ((long long)T * K >= (1LL << 31)) return AWQ_ERR_SHAPE;   // 32-bit offsets into X_cal
    for (int l = 0; l < n_layers; ++l)
        if (Ws[l] == nullptr) return AWQ_ERR_NULL;
    if ((st = check_ptrs({X_cal, s_out, workspace}))) return as_status(st);
    for (int l = 0; l < n_layers; ++l)
        if ((st = check_ptr(Ws[l]))) return as_status(st);
    if (loss_out != nullptr && (st = check_ptr(loss_out))) return as_status(st);
    if (best_out != nullptr && (st = check_ptr(best_out))) return as_status(st);
    const int path = search_path(T, (int)N, K, n_alpha, workspace_bytes);
    if (path < 0) return AWQ_ERR_WORKSPACE;
    return hip_status(awq::launch_search(Ws, Ns, n_layers, X_cal, T, K, alphas, n_alpha, bits,
                                         group_size, zero_point, s_out, loss_out, best_out,
                                         workspace, path == 1, stream));
}

size_t awq_search_mlp_workspace_bytes(int T, int K, int I, int K_out, int n_alpha) {
    if (T <= 0 || K <= 0 || I <= 0 || K_out <= 0 || n_alpha <= 0) return 0;
    if (K % awq::kGroup != 0 || I % awq::kGroup != 0) return 0;
    return awq::search_mlp_workspace_bytes(T, K, I, K_out, n_alpha);
}

awq_status awq_search_scale_mlp(const void* W_gate, const void* W_up, const void* W_down,
                                const void* X_cal, int T, int K, int I, int K_out,
                                const float* alphas, int n_alpha, int bits, int group_size,
                                int zero_point, float* s_out, float* loss_out, int* best_out,
                                void* workspace, size_t workspace_bytes, hipStream_t stream) {
    int st = check_quant_params(bits, group_size, zero_point);
    if (st) return as_status(st);
    if (n_alpha < 1 || n_alpha > kMaxAlpha) return AWQ_ERR_UNSUPPORTED;
    if (T > kMaxT) return AWQ_ERR_UNSUPPORTED;
    if (T <= 0 || I <= 0 || K_out <= 0) return AWQ_ERR_SHAPE;
    if ((st = check_nk(I, K))) return as_status(st);
    if (I % awq::kGroup != 0) return AWQ_ERR_SHAPE;            // I is the down projection's K
    // 32-bit offsets into X_cal and into the intermediate activations
    if ((long long)T * K >= (1LL << 31) || (long long)T * I >= (1LL << 31)) return AWQ_ERR_SHAPE;
    if ((long long)K_out * I >= (1LL << 40) || (long long)I * K >= (1LL << 40)) return AWQ_ERR_SHAPE;
    if (alphas == nullptr) return AWQ_ERR_NULL;
    if ((st = check_ptrs({W_gate, W_up, W_down, X_cal, s_out, workspace}))) return as_status(st);
    if (loss_out != nullptr && (st = check_ptr(loss_out))) return as_status(st);
    if (best_out != nullptr && (st = check_ptr(best_out))) return as_status(st);
    if (workspace_bytes < awq::search_mlp_workspace_bytes(T, K, I, K_out, n_alpha)) return AWQ_ERR_WORKSPACE;
    return hip_status(awq::launch_search_mlp(W_gate, W_up, W_down, K_out, X_cal, T, K, I, alphas, n_alpha,
                                             bits, group_size, zero_point, s_out, loss_out, best_out,
                                             workspace, stream));
}

namespace {
// shared checks of the decode entry points; 1 = nothing to do (M or N is 0)
int check_gemv(int M, int N, int K, int bits, int group_size) {
    int st = check_quant_params(bits, group_size, 1);
    if (st) return as_status(st);
    if (M > kMaxGemvM) return AWQ_ERR_UNSUPPORTED;
    if (M < 0) return AWQ_ERR_SHAPE;
    if ((st = check_nk(N, K))) return as_status(st);
    // the decode kernels address x and the packed tiles with 32-bit offsets
    if ((long long)M * K * 2 >= (1LL << 31) ||
        16LL * ((N + 15) / 16) * K / 8 * bits >= (1LL << 31))
        return AWQ_ERR_SHAPE;
    return (M == 0 || N == 0) ? -1 : AWQ_OK;
}
}  // namespace

awq_status awq_gemv(const void* x, const void* qweight, const void* scales, const void* zeros, void* y,
             int M, int N, int K, int bits, int group_size, hipStream_t stream) {
    int st = check_gemv(M, N, K, bits, group_size);
    if (st) return st < 0 ? AWQ_OK : as_status(st);
    if ((st = check_ptrs({x, qweight, scales, zeros, y}))) return as_status(st);
    return hip_status(awq::launch_gemv(x, nullptr, qweight, scales, zeros, nullptr, nullptr, nullptr,
                                       y, M, N, K, bits, group_size, stream));
}

awq_status awq_gemv_scaled(const void* x, const float* inv_s, const void* qweight, const void* scales,
                    const void* zeros, void* y, int M, int N, int K, int bits, int group_size,
                    hipStream_t stream) {
    int st = check_gemv(M, N, K, bits, group_size);
    if (st) return st < 0 ? AWQ_OK : as_status(st);
    if ((st = check_ptrs({x, inv_s, qweight, scales, zeros, y}))) return as_status(st);
    return hip_status(awq::launch_gemv(x, inv_s, qweight, scales, zeros, nullptr, nullptr, nullptr,
                                       y, M, N, K, bits, group_size, stream));
}

awq_status awq_gemv_gate_up(const void* x, const float* inv_s, const void* gate_qweight,
                     const void* gate_scales, const void* gate_zeros, const void* up_qweight,
                     const void* up_scales, const void* up_zeros, void* h, int M, int N, int K,
                     int bits, int group_size, hipStream_t stream) {
    int st = check_gemv(M, N, K, bits, group_size);
    if (st) return st < 0 ? AWQ_OK : as_status(st);
    if ((st = check_ptrs({x, gate_qweight, gate_scales, gate_zeros, up_qweight, up_scales, up_zeros, h})))
        return as_status(st);
    if (inv_s && (st = check_ptr(inv_s))) return as_status(st);
    return hip_status(awq::launch_gemv(x, inv_s, gate_qweight, gate_scales, gate_zeros, up_qweight,
                                       up_scales, up_zeros, h, M, N, K, bits, group_size,
                                       stream));
}

awq_status awq_gemm(const void* x, const void* qweight, const void* scales, const void* zeros, void* y,
             int M, int N, int K, int bits, int group_size, hipStream_t stream) {
    int st = check_quant_params(bits, group_size, 1);
    if (st) return as_status(st);
    if (M < 0) return AWQ_ERR_SHAPE;
    if ((st = check_nk(N, K))) return as_status(st);
    // the prefill kernel addresses x and the packed tiles with 32-bit offsets
    if ((long long)M * K >= (1LL << 31) || (long long)N * K / 8 >= (1LL << 31)) return AWQ_ERR_SHAPE;
    if (M == 0 || N == 0) return AWQ_OK;
    if ((st = check_ptrs({x, qweight, scales, zeros, y}))) return as_status(st);
    return hip_status(awq::launch_gemm(x, nullptr, qweight, scales, zeros, y, M, N, K, bits, group_size,
                                       stream));
}

size_t awq_gemm_splitk_workspace_bytes(int M, int N, int K) {
    if (M <= 0 || N <= 0 || K <= 0 || K % awq::kGroup != 0) return 0;
    return awq::gemm_splitk_workspace_bytes(M, N, K);
}

awq_status awq_gemm_splitk(const void* x, const void* qweight, const void* scales, const void* zeros,
                    void* y, int M, int N, int K, int bits, int group_size, void* workspace,
                    size_t workspace_bytes, hipStream_t stream) {
    int st = check_quant_params(bits, group_size, 1);
    if (st) return as_status(st);
    if (M < 0) return AWQ_ERR_SHAPE;
    if ((st = check_nk(N, K))) return as_status(st);
    if ((long long)M * K >= (1LL << 31) || (long long)N * K / 8 >= (1LL << 31)) return AWQ_ERR_SHAPE;
    if (M == 0 || N == 0) return AWQ_OK;
    if ((st = check_ptrs({x, qweight, scales, zeros, y}))) return as_status(st);
    const size_t need = awq::gemm_splitk_workspace_bytes(M, N, K);
    if (need > 0) {
        if (workspace == nullptr) return AWQ_ERR_NULL;
        if ((st = check_ptr(workspace))) return as_status(st);
        if (workspace_bytes < need) return AWQ_ERR_WORKSPACE;
    }
    return hip_status(awq::launch_gemm_splitk(x, nullptr, qweight, scales, zeros, y, M, N, K, bits,
                                              group_size, workspace, stream));
}

awq_status awq_gemm_scaled(const void* x, const float* inv_s, const void* qweight,
                           const void* scales, const void* zeros, void* y, int M, int N, int K,
                           int bits, int group_size, void* workspace, size_t workspace_bytes,
                           hipStream_t stream) {
    int st = check_quant_params(bits, group_size, 1);
    if (st) return as_status(st);
    if (M < 0) return AWQ_ERR_SHAPE;
    if ((st = check_nk(N, K))) return as_status(st);
    if ((long long)M * K >= (1LL << 31) || (long long)N * K / 8 >= (1LL << 31)) return AWQ_ERR_SHAPE;
    if (M == 0 || N == 0) return AWQ_OK;
    if ((st = check_ptrs({x, inv_s, qweight, scales, zeros, y}))) return as_status(st);
    if (workspace == nullptr || workspace_bytes == 0)
        return hip_status(awq::launch_gemm(x, inv_s, qweight, scales, zeros, y, M, N, K, bits,
                                           group_size, stream));
    if ((st = check_ptr(workspace))) return as_status(st);
    if (workspace_bytes < awq::gemm_splitk_workspace_bytes(M, N, K)) return AWQ_ERR_WORKSPACE;
    return hip_status(awq::launch_gemm_splitk(x, inv_s, qweight, scales, zeros, y, M, N, K, bits,
                                              group_size, workspace, stream));
}

}  // extern "C"

// ---------------------------------------------------------------------------
// awq_gemm_splitk_noalloc: awq_gemm_splitk with the fp32 partial sums in a
// fixed device array instead of a caller workspace.  Split K runs only while
// the output tiles (at most 128 x 256) occupy at most half the CUs, so the
// partials take at most CUs x 128 x 256 x 4 bytes: 32 MiB on a 256-CU MI355X.
// Each GPU the library runs on holds its own copy of the array until the
// process ends.  Host code never passes the array's name to a kernel (on the
// host it is only a stand-in for the symbol): the device address of each
// GPU's copy is asked of the runtime once, with that device current, and kept.
// ---------------------------------------------------------------------------
namespace {
constexpr size_t kScratchBytes = (size_t)32 << 20;
constexpr int kMaxDevices = 64;
}  // namespace

static __device__ __align__(256) unsigned char scratch[kScratchBytes];

namespace {
std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices];

// the current device's copy of `scratch` (nullptr if the runtime cannot say)
void* device_scratch() {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    if (g_scratch_ptr[dev] == nullptr) {
        void* p = nullptr;
        if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || p == nullptr) return nullptr;
        g_scratch_ptr[dev] = p;
    }
    return g_scratch_ptr[dev];
}
}  // namespace

extern "C" {

size_t awq_gemm_splitk_noalloc_max_bytes(void) { return kScratchBytes; }

awq_status awq_gemm_splitk_noalloc(const void* x, const void* qweight, const void* scales,
                                   const void* zeros, void* y, int M, int N, int K, int bits,
                                   int group_size, hipStream_t stream) {
    int st = check_quant_params(bits, group_size, 1);
    if (st) return as_status(st);
    if (M < 0) return AWQ_ERR_SHAPE;
    if ((st = check_nk(N, K))) return as_status(st);
    if ((long long)M * K >= (1LL << 31) || (long long)N * K / 8 >= (1LL << 31)) return AWQ_ERR_SHAPE;
    if (M == 0 || N == 0) return AWQ_OK;
    if ((st = check_ptrs({x, qweight, scales, zeros, y}))) return as_status(st);
    const size_t need = awq::gemm_splitk_workspace_bytes(M, N, K);
    if (need > kScratchBytes) return AWQ_ERR_WORKSPACE;
    void* ws = nullptr;
    if (need > 0 && (ws = device_scratch()) == nullptr) return AWQ_ERR_HIP;
    // every split writes all M x N entries of its partial tile, so nothing in
    // the array needs clearing between calls
    return hip_status(awq::launch_gemm_splitk(x, nullptr, qweight, scales, zeros, y, M, N, K, bits,
                                              group_size, ws, stream));
}

}  // extern "C"

// ---------------------------------------------------------------------------
// operators beside the packed products
// ---------------------------------------------------------------------------
namespace {
constexpr int kMaxNormWidth = 32768;      // a row lives in one workgroup's registers
constexpr int kMaxW8a8K = 1 << 17;        // 128 * 128 * K < 2^31: exact int32 sums

int check_dtype(int dtype) { return dtype == AWQ_F16 || dtype == AWQ_BF16 ? AWQ_OK : AWQ_ERR_UNSUPPORTED; }

// null pointers pass
int check_optional(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (p != nullptr && check_ptr(p) != AWQ_OK) return AWQ_ERR_ALIGN;
    return AWQ_OK;
}

int check_rows(int M, int K, int dtype) {
    if (int st = check_dtype(dtype)) return st;
    return M < 0 || K <= 0 || K % 16 != 0 || K >= kMaxW8a8K ? AWQ_ERR_SHAPE : AWQ_OK;
}

// A launch counts its threads in 32 bits.  The most: 32 a column with up to 4
// rows, 4 a row for narrow products on 128 x 128 tiles (wider ones of that many
// tiles go to the 256 x 256 kernel, which launches one workgroup a compute unit).
int check_w8a8(int M, int N, int K, int dtype) {
    if (int st = check_rows(M, K, dtype)) return st;
    if (N < 0 || M >= 1 << 29 || N >= 1 << 26) return AWQ_ERR_SHAPE;
    if ((long long)M * N >= (1LL << 40)) return AWQ_ERR_SHAPE;
    return AWQ_OK;
}

int check_workspace(const void* workspace, size_t bytes, size_t need) {
    if (need == 0) return AWQ_OK;
    if (workspace == nullptr) return AWQ_ERR_NULL;
    if (int st = check_ptr(workspace)) return st;
    return bytes < need ? AWQ_ERR_WORKSPACE : AWQ_OK;
}
}  // namespace

extern "C" {

awq_status awq_norm_gate_residual(const void* block, const void* residual, const void* post_weight,
                                  const void* post_bias, const void* gate, int gate_rows,
                                  float residual_scale, const void* pre_weight, const void* pre_bias,
                                  int kind, float eps, int T, int H, int dtype, void* residual_out,
                                  void* h, float* h_scales, hipStream_t stream) {
    int st = check_dtype(dtype);
    if (st) return as_status(st);
    if (kind != AWQ_NORM_RMS && kind != AWQ_NORM_LAYER) return AWQ_ERR_UNSUPPORTED;
    if (!(eps >= 0.0f)) return AWQ_ERR_UNSUPPORTED;
    if (T < 0 || H <= 0 || H % 8 != 0 || H > kMaxNormWidth) return AWQ_ERR_SHAPE;
    if (gate != nullptr && (gate_rows <= 0 || T % gate_rows != 0)) return AWQ_ERR_SHAPE;
    if (T == 0) return AWQ_OK;
    if ((st = check_ptrs({block, residual, pre_weight, residual_out, h}))) return as_status(st);
    if (post_bias != nullptr && post_weight == nullptr) return AWQ_ERR_NULL;
    if ((st = check_optional({post_weight, post_bias, gate, pre_bias, h_scales}))) return as_status(st);
    awq::NormProblem p{block, residual, post_weight, post_bias, gate, pre_weight, pre_bias, residual_out, h,
                       h_scales, residual_scale, eps, gate_rows, kind, T, H, dtype};
    return hip_status(awq::launch_norm(p, stream));
}

awq_status awq_quantize_rows(const void* x, int M, int K, int dtype, void* q, float* scales,
                             hipStream_t stream) {
    int st = check_rows(M, K, dtype);
    if (st) return as_status(st);
    if (M == 0) return AWQ_OK;
    if ((st = check_ptrs({x, q, scales}))) return as_status(st);
    return hip_status(awq::launch_quantize_rows(x, M, K, dtype, q, scales, stream));
}

size_t awq_gemm_w8a8_workspace_bytes(int M, int N, int K) {
    if (M <= 0 || N <= 0 || check_w8a8(M, N, K, AWQ_F16) != AWQ_OK) return 0;
    return awq::w8a8_workspace_bytes(M, N, K);
}

size_t awq_linear_w8a8_workspace_bytes(int M, int N, int K) {
    if (M <= 0 || N <= 0 || check_w8a8(M, N, K, AWQ_F16) != AWQ_OK) return 0;
    return awq::linear_w8a8_workspace_bytes(M, N, K);
}

awq_status awq_gemm_w8a8(const void* x, const float* x_scales, const void* weight,
                         const float* weight_scales, const float* bias, void* y, int M, int N, int K,
                         int dtype, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    int st = check_w8a8(M, N, K, dtype);
    if (st) return as_status(st);
    if (M == 0 || N == 0) return AWQ_OK;
    if ((st = check_ptrs({x, x_scales, weight, weight_scales, y}))) return as_status(st);
    if ((st = check_optional({bias}))) return as_status(st);
    if ((st = check_workspace(workspace, workspace_bytes, awq::w8a8_workspace_bytes(M, N, K))))
        return as_status(st);
    awq::W8a8Problem p{x, nullptr, weight, x_scales, weight_scales, bias, y, M, N, K, dtype};
    return hip_status(awq::launch_w8a8(p, workspace, stream));
}

awq_status awq_linear_w8a8(const void* x, const void* weight, const float* weight_scales, const float* bias,
                           void* y, int M, int N, int K, int dtype, void* workspace,
                           size_t workspace_bytes, hipStream_t stream) {
    int st = check_w8a8(M, N, K, dtype);
    if (st) return as_status(st);
    if (M == 0 || N == 0) return AWQ_OK;
    if ((st = check_ptrs({x, weight, weight_scales, y}))) return as_status(st);
    if ((st = check_optional({bias}))) return as_status(st);
    if ((st = check_workspace(workspace, workspace_bytes, awq::linear_w8a8_workspace_bytes(M, N, K))))
        return as_status(st);
    awq::W8a8Problem p{nullptr, x, weight, nullptr, weight_scales, bias, y, M, N, K, dtype};
    return hip_status(awq::launch_w8a8(p, workspace, stream));
}

namespace {
int check_moe(int M, int K, int I, int E, int top_k) {
    if (M > awq::kMoeMaxTokens || E > awq::kMoeMaxExperts || top_k < 1 || top_k > awq::kMoeMaxTopK || top_k > E)
        return AWQ_ERR_UNSUPPORTED;
    if (M < 0 || K <= 0 || I <= 0 || K % awq::kGroup != 0 || I % awq::kGroup != 0) return AWQ_ERR_SHAPE;
    // a token's operand row is held in LDS (as two fp16 planes)
    if (K > awq::kMoeMaxWidth || I > awq::kMoeMaxWidth) return AWQ_ERR_SHAPE;
    return AWQ_OK;
}
}  // namespace

size_t awq_moe_workspace_bytes(int M, int K, int I, int E, int top_k) {
    if (M <= 0 || check_moe(M, K, I, E, top_k) != AWQ_OK) return 0;
    return awq::moe_workspace_bytes(M, K, I, E, top_k);
}

awq_status awq_moe(const void* x, const float* inv_s, const void* router, const void* gate_qweight,
                   const void* gate_scales, const void* gate_zeros, const void* up_qweight,
                   const void* up_scales, const void* up_zeros, const void* down_qweight,
                   const void* down_scales, const void* down_zeros, void* y, int M, int K, int I, int E,
                   int top_k, int bits, int group_size, int renormalize, void* workspace,
                   size_t workspace_bytes, hipStream_t stream) {
    int st = check_quant_params(bits, group_size, 1);
    if (st) return as_status(st);
    if (renormalize != 0 && renormalize != 1) return AWQ_ERR_UNSUPPORTED;
    if ((st = check_moe(M, K, I, E, top_k))) return as_status(st);
    if (M == 0) return AWQ_OK;
    if ((st = check_ptrs({x, router, gate_qweight, gate_scales, gate_zeros, up_qweight, up_scales, up_zeros,
                          down_qweight, down_scales, down_zeros, y})))
        return as_status(st);
    if ((st = check_optional({inv_s}))) return as_status(st);
    if ((st = check_workspace(workspace, workspace_bytes, awq::moe_workspace_bytes(M, K, I, E, top_k))))
        return as_status(st);
    awq::MoeProblem p{x, router, inv_s, {gate_qweight, up_qweight, down_qweight},
                      {gate_scales, up_scales, down_scales}, {gate_zeros, up_zeros, down_zeros}, y, M, K, I, E,
                      top_k, bits, group_size, renormalize};
    return hip_status(awq::launch_moe(p, workspace, stream));
}

}  // extern "C"

// ---------------------------------------------------------------------------
// rotary positions and the paged 8-bit cache
// ---------------------------------------------------------------------------
namespace {
constexpr int kMaxRopeDim = 512;
constexpr long long kMaxGroups = 1LL << 24;      // workgroups of 256 threads: a launch counts threads in 32 bits
constexpr int kMaxCacheRows = 1 << 20;           // rows (tokens) and sequences of a call
constexpr int kMaxBookRows = 65535;              // table rows are a launch's second dimension
constexpr int kMaxPages = 1 << 30;
constexpr int kMaxHeads = 65535;
// cap tanh(x / cap) comes from cap - 2 cap / (exp(2 x / cap) + 1): right to cap 2^-21
constexpr float kMinCap = 0x1p-10f, kMaxCap = 1024.0f;
constexpr float kMaxScale = 0x1p100f;            // times 2^24, the unit of a product's operands, it stays in fp32
constexpr int kMaxWindow = 1 << 30;              // positions less a window stay in 31 bits

// index arrays are int32 and need no more than their own alignment
int check_index(std::initializer_list<const void*> ps) {
    for (const void* p : ps) if (p == nullptr) return AWQ_ERR_NULL;
    for (const void* p : ps) if (reinterpret_cast<uintptr_t>(p) & 3u) return AWQ_ERR_ALIGN;
    return AWQ_OK;
}

// rows of `heads` heads, `stride` elements apart
int check_stride(long long stride, int heads, int dim) {
    return stride < (long long)heads * dim || stride % 8 != 0 ? AWQ_ERR_SHAPE : AWQ_OK;
}

int check_rotation(const float* inv_freq, int rotary_dim, int dim, int layout, float magnitude) {
    if (inv_freq == nullptr) return AWQ_OK;
    if (layout != AWQ_ROPE_HALF && layout != AWQ_ROPE_INTERLEAVED) return AWQ_ERR_UNSUPPORTED;
    if (!isfinite(magnitude)) return AWQ_ERR_UNSUPPORTED;
    if (rotary_dim <= 0 || rotary_dim % 16 != 0 || rotary_dim > dim) return AWQ_ERR_SHAPE;
    return reinterpret_cast<uintptr_t>(inv_freq) & 3u ? AWQ_ERR_ALIGN : AWQ_OK;
}

awq::Rotation rotation(const float* inv_freq, int rotary_dim, int layout, float magnitude, int inverse) {
    return {inv_freq, magnitude, inv_freq ? rotary_dim / 2 : 0, layout == AWQ_ROPE_INTERLEAVED, inverse};
}

int check_page(int page_size) {
    return page_size == 16 || page_size == 32 || page_size == 64 || page_size == 128 ? AWQ_OK : AWQ_ERR_UNSUPPORTED;
}

int check_cache(int kv_heads, int dim, int pages, int page_size) {
    if (int st = check_page(page_size)) return st;
    if (dim != 64 && dim != 96 && dim != 128 && dim != 192 && dim != 256) return AWQ_ERR_UNSUPPORTED;
    // a page of all heads stays below 2^31 codes
    return kv_heads <= 0 || kv_heads > kMaxHeads || pages <= 0 || pages > kMaxPages ? AWQ_ERR_SHAPE : AWQ_OK;
}

// T rows of B sequences with tables of W pages; without starts every sequence has one row
int check_sequences(const int* starts, int T, int B, int W) {
    if (T < 0 || B < 0 || W <= 0 || T > kMaxCacheRows || B > kMaxCacheRows) return AWQ_ERR_SHAPE;
    return starts == nullptr && T != B ? AWQ_ERR_SHAPE : AWQ_OK;
}

int log2_of(int page_size) { return __builtin_ctz((unsigned)page_size); }

awq::Cache cache_of(const void* k, const float* ks, const void* v, const float* vs, int pages, int kv, int page_size,
                    int dim) {
    return {{(int8_t*)k, (int8_t*)v}, {(float*)ks, (float*)vs}, pages, kv, log2_of(page_size), dim};
}

int check_attention(int T, int B, int W, int heads, int kv_heads, int dim, int pages, int page_size, int max_new,
                    int max_len) {
    if (int st = check_cache(kv_heads, dim, pages, page_size)) return st;
    if (T < 0 || B < 0 || W <= 0 || T > kMaxCacheRows || B > kMaxCacheRows) return AWQ_ERR_SHAPE;
    if (heads <= 0 || heads % kv_heads != 0 || max_new <= 0 || max_len <= 0) return AWQ_ERR_SHAPE;
    // a wave for each row and head joins, a workgroup of up to 512 threads for each tile of rows computes
    return (long long)T * heads >= kMaxGroups || ((long long)T * (heads / kv_heads) / 16 + B) * kv_heads >= kMaxGroups / 2
               ? AWQ_ERR_SHAPE : AWQ_OK;
}

int check_book(int B, int W, int pages, int page_size) {
    if (int st = check_page(page_size)) return st;
    if (B < 0 || B > kMaxBookRows || W <= 0 || pages <= 0 || pages > kMaxPages) return AWQ_ERR_SHAPE;
    return (long long)B * W >= 1LL << 31 ? AWQ_ERR_SHAPE : AWQ_OK;       // pages of all rows are summed in 31 bits
}
}  // namespace

extern "C" {

awq_status awq_rope_frequencies(int rotary_dim, double base, int scaling, double factor, double original_length,
                                double low, double high, float* inv_freq, float* magnitude) {
    if (inv_freq == nullptr || magnitude == nullptr) return AWQ_ERR_NULL;
    if (rotary_dim <= 0 || rotary_dim % 2 != 0 || rotary_dim > kMaxRopeDim) return AWQ_ERR_SHAPE;
    if (!(base > 1.0) || !isfinite(base)) return AWQ_ERR_UNSUPPORTED;
    const bool rounded = scaling == AWQ_ROPE_YARN_ROUNDED;
    if (rounded) scaling = AWQ_ROPE_YARN;
    if (scaling < AWQ_ROPE_PLAIN || scaling > AWQ_ROPE_BANDS) return AWQ_ERR_UNSUPPORTED;
    if (scaling != AWQ_ROPE_PLAIN && (!(factor >= 1.0) || !isfinite(factor))) return AWQ_ERR_UNSUPPORTED;
    if (scaling == AWQ_ROPE_BASE && rotary_dim <= 2) return AWQ_ERR_SHAPE;
    const bool parts = scaling == AWQ_ROPE_YARN || scaling == AWQ_ROPE_BANDS;
    if (parts && (!(original_length > 0.0) || !isfinite(original_length) || !(low > 0.0) || !(high > low) || !isfinite(high)))
        return AWQ_ERR_UNSUPPORTED;
    const int n = rotary_dim / 2;
    const double two_pi = 6.283185307179586476925;
    if (scaling == AWQ_ROPE_BASE) base *= pow(factor, (double)rotary_dim / (rotary_dim - 2));
    *magnitude = scaling == AWQ_ROPE_YARN ? (float)(0.1 * log(factor) + 1.0) : 1.0f;
    for (int i = 0; i < n; ++i) {
        const double f = pow(base, -(double)i / n);
        double keep = 1.0;                       // the share of the unscaled frequency
        if (scaling == AWQ_ROPE_LINEAR) keep = 0.0;
        if (scaling == AWQ_ROPE_BANDS) keep = (original_length * f / two_pi - low) / (high - low);
        if (scaling == AWQ_ROPE_YARN) {          // a ramp over the channels between those that turn high and low times
            double from = n * log(original_length / (high * two_pi)) / log(base);
            double to = n * log(original_length / (low * two_pi)) / log(base);
            if (rounded) {
                from = fmin(fmax(floor(from), 0.0), rotary_dim - 1.0);
                to = fmin(fmax(ceil(to), 0.0), rotary_dim - 1.0);
                if (to <= from) to = from + 0.5;           // no channel between: a step behind `from`
            }
            keep = 1.0 - (i - from) / (to - from);
        }
        keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
        inv_freq[i] = (float)(f * keep + (keep < 1.0 ? f / factor * (1.0 - keep) : 0.0));
    }
    return AWQ_OK;
}

awq_status awq_rope(const void* x, long long x_stride, const int* positions, const float* inv_freq, float magnitude,
                    void* out, long long out_stride, int T, int heads, int head_dim, int rotary_dim, int layout,
                    int inverse, int dtype, hipStream_t stream) {
    int st = check_dtype(dtype);
    if (st) return as_status(st);
    if (T < 0 || heads <= 0 || heads > kMaxHeads || head_dim <= 0 || head_dim % 16 != 0 || head_dim > kMaxRopeDim)
        return AWQ_ERR_SHAPE;
    if (T / 4 + 1 >= kMaxGroups) return AWQ_ERR_SHAPE;
    if (inverse != 0 && inverse != 1) return AWQ_ERR_UNSUPPORTED;
    if (inv_freq == nullptr && T > 0) return AWQ_ERR_NULL;
    if ((st = check_rotation(inv_freq, rotary_dim, head_dim, layout, magnitude))) return as_status(st);
    if ((st = check_stride(x_stride, heads, head_dim)) || (st = check_stride(out_stride, heads, head_dim)))
        return as_status(st);
    if (T == 0) return AWQ_OK;
    if (x != nullptr && x == out && T > 1 && x_stride != out_stride) return AWQ_ERR_UNSUPPORTED;
    if ((st = check_ptrs({x, out})) || (st = check_index({positions}))) return as_status(st);
    const awq::RopeProblem p{x, x_stride, positions, out, out_stride,
                             rotation(inv_freq, rotary_dim, layout, magnitude, inverse), T, heads, head_dim, dtype};
    return hip_status(awq::launch_rope(p, stream));
}

awq_status awq_cache_append(const void* q, long long q_stride, const void* k, long long k_stride, const void* v,
                            long long v_stride, void* q_out, const float* inv_freq, float magnitude, int rotary_dim,
                            int layout, void* k_codes, float* k_scales, void* v_codes, float* v_scales,
                            const int* tables, const int* lens, const int* starts, int T, int B, int W, int heads,
                            int kv_heads, int head_dim, int pages, int page_size, int dtype, hipStream_t stream) {
    int st = check_dtype(dtype);
    if (st) return as_status(st);
    if ((st = check_cache(kv_heads, head_dim, pages, page_size)) || (st = check_sequences(starts, T, B, W)))
        return as_status(st);
    if (q != nullptr && (heads <= 0 || heads > kMaxHeads)) return AWQ_ERR_SHAPE;
    if ((st = check_rotation(inv_freq, rotary_dim, head_dim, layout, magnitude))) return as_status(st);
    if (q != nullptr && (st = check_stride(q_stride, heads, head_dim))) return as_status(st);
    if ((st = check_stride(k_stride, kv_heads, head_dim)) || (st = check_stride(v_stride, kv_heads, head_dim)))
        return as_status(st);
    // workgroups: rows by four for q, and two a kv head for every page that is reached
    const long long items = starts ? (long long)T / page_size + 2LL * B : B;
    if (T / 4 + 1 + 2 * (items < T ? items : T) * kv_heads >= kMaxGroups) return AWQ_ERR_SHAPE;
    if (T == 0 || B == 0) return AWQ_OK;
    if ((st = check_ptrs({k, v, k_codes, v_codes})) || (st = check_index({k_scales, v_scales, tables, lens})))
        return as_status(st);
    if (q != nullptr && (st = check_ptrs({q, q_out}))) return as_status(st);
    if (q != nullptr && q == q_out && T > 1 && q_stride != (long long)heads * head_dim) return AWQ_ERR_UNSUPPORTED;
    if (starts != nullptr && (st = check_index({starts}))) return as_status(st);
    const awq::AppendProblem p{q, k, v, q_stride, k_stride, v_stride, q_out,
                               rotation(inv_freq, rotary_dim, layout, magnitude, 0),
                               cache_of(k_codes, k_scales, v_codes, v_scales, pages, kv_heads, page_size, head_dim),
                               awq::Sequences{tables, lens, starts, T, B, W}, heads, dtype};
    return hip_status(awq::launch_cache_append(p, stream));
}

awq_status awq_cache_read(const void* k_codes, const float* k_scales, const void* v_codes, const float* v_scales,
                          const int* tables, const int* lens, const int* starts, int T, int B, int W, int kv_heads,
                          int head_dim, int pages, int page_size, int dtype, void* k_out, void* v_out,
                          hipStream_t stream) {
    int st = check_dtype(dtype);
    if (st) return as_status(st);
    if ((st = check_cache(kv_heads, head_dim, pages, page_size)) || (st = check_sequences(starts, T, B, W)))
        return as_status(st);
    if (T == 0 || B == 0) return AWQ_OK;
    if ((st = check_ptrs({k_codes, v_codes, k_out, v_out})) || (st = check_index({k_scales, v_scales, tables, lens})))
        return as_status(st);
    if (starts != nullptr && (st = check_index({starts}))) return as_status(st);
    const awq::ReadProblem p{cache_of(k_codes, k_scales, v_codes, v_scales, pages, kv_heads, page_size, head_dim),
                             awq::Sequences{tables, lens, starts, T, B, W}, k_out, v_out, dtype};
    return hip_status(awq::launch_cache_read(p, stream));
}

size_t awq_cache_attention_workspace_bytes(int T, int B, int heads, int kv_heads, int head_dim, int max_new,
                                           int max_len) {
    if (T <= 0 || B <= 0 || check_attention(T, B, 1, heads, kv_heads, head_dim, 1, 16, max_new, max_len) != AWQ_OK)
        return 0;
    return awq::attend_workspace_bytes(T, B, heads, kv_heads, head_dim, max_new, max_len);
}

awq_status awq_cache_attention(const void* q, long long q_stride, const void* k_codes, const float* k_scales,
                               const void* v_codes, const float* v_scales, const int* tables, const int* lens,
                               const int* starts, void* out, float* lse, float scale, int window, float softcap, int T,
                               int B, int W, int heads, int kv_heads, int head_dim, int pages, int page_size,
                               int max_new, int max_len, int dtype, void* workspace, size_t workspace_bytes,
                               hipStream_t stream) {
    int st = check_dtype(dtype);
    if (st) return as_status(st);
    if ((st = check_attention(T, B, W, heads, kv_heads, head_dim, pages, page_size, max_new, max_len)) ||
        (st = check_sequences(starts, T, B, W)) || (st = check_stride(q_stride, heads, head_dim)))
        return as_status(st);
    if (!(fabsf(scale) < kMaxScale) || window < 0) return AWQ_ERR_UNSUPPORTED;
    if (softcap != 0.0f && !(softcap >= kMinCap && softcap <= kMaxCap)) return AWQ_ERR_UNSUPPORTED;
    if (T == 0 || B == 0) return AWQ_OK;
    if ((st = check_ptrs({q, k_codes, v_codes, out})) || (st = check_index({k_scales, v_scales, tables, lens})))
        return as_status(st);
    if (q == out) return AWQ_ERR_UNSUPPORTED;
    if (starts != nullptr && (st = check_index({starts}))) return as_status(st);
    if (lse != nullptr && (st = check_index({lse}))) return as_status(st);
    if ((st = check_workspace(workspace, workspace_bytes,
                              awq::attend_workspace_bytes(T, B, heads, kv_heads, head_dim, max_new, max_len))))
        return as_status(st);
    const awq::AttendProblem p{q, q_stride, out, lse,
                               cache_of(k_codes, k_scales, v_codes, v_scales, pages, kv_heads, page_size, head_dim),
                               awq::Sequences{tables, lens, starts, T, B, W}, scale, softcap, heads,
                               window < kMaxWindow ? window : kMaxWindow, max_new,
                               max_len, dtype};
    return hip_status(awq::launch_cache_attention(p, workspace, stream));
}

awq_status awq_cache_fork(const int* tables, const int* lens, int* refs, const int* parents, int* out_tables,
                          int* out_lens, int B, int B_out, int W, int pages, int page_size, hipStream_t stream) {
    int st = check_book(B, W, pages, page_size);
    if (st) return as_status(st);
    if ((st = check_book(B_out, W, pages, page_size))) return as_status(st);
    if (B == 0 && B_out == 0) return AWQ_OK;
    if ((st = check_index({refs}))) return as_status(st);
    if (B > 0 && (st = check_index({tables, lens}))) return as_status(st);
    if (B_out > 0 && (st = check_index({parents, out_tables, out_lens}))) return as_status(st);
    if (B > 0 && B_out > 0 && (out_tables == tables || out_lens == lens)) return AWQ_ERR_UNSUPPORTED;
    return hip_status(awq::launch_cache_fork(tables, lens, refs, parents, out_tables, out_lens, B, B_out, W, pages,
                                             log2_of(page_size), stream));
}

awq_status awq_cache_reserve(int* tables, int* lens, int* refs, const int* counts, int* pairs, int* status, int B,
                             int W, int pages, int page_size, hipStream_t stream) {
    int st = check_book(B, W, pages, page_size);
    if (st) return as_status(st);
    if (B > awq::kMaxReserveRows) return AWQ_ERR_UNSUPPORTED;
    if ((st = check_index({status}))) return as_status(st);
    if (B > 0 && (st = check_index({tables, lens, refs, counts, pairs}))) return as_status(st);
    return hip_status(awq::launch_cache_reserve(tables, lens, refs, counts, pairs, status, B, W, pages,
                                                log2_of(page_size), stream));
}

awq_status awq_cache_compact(int* tables, const int* lens, int* refs, int* moves, int* count, int B, int W, int pages,
                             int page_size, hipStream_t stream) {
    int st = check_book(B, W, pages, page_size);
    if (st) return as_status(st);
    if ((st = check_index({refs, moves, count}))) return as_status(st);
    if (B > 0 && (st = check_index({tables, lens}))) return as_status(st);
    return hip_status(awq::launch_cache_compact(tables, lens, refs, moves, count, B, W, pages, log2_of(page_size), stream));
}

awq_status awq_cache_copy_pages(void* const* tensors, const size_t* page_bytes, int n_tensors, int layers,
                                const int* pairs, const int* count, int max_pairs, int pages, hipStream_t stream) {
    if (n_tensors < 1 || n_tensors > awq::kMaxCopyTensors) return AWQ_ERR_UNSUPPORTED;
    if (layers <= 0 || max_pairs < 0 || pages <= 0 || pages > kMaxPages) return AWQ_ERR_SHAPE;
    if (tensors == nullptr || page_bytes == nullptr) return AWQ_ERR_NULL;
    awq::CopyProblem p{};
    for (int t = 0; t < n_tensors; ++t) {
        if (page_bytes[t] == 0 || page_bytes[t] % 4 != 0 || page_bytes[t] > (size_t)1 << 30) return AWQ_ERR_SHAPE;
        p.tensors[t] = (char*)tensors[t];
        p.page_bytes[t] = page_bytes[t];
    }
    if (max_pairs == 0) return AWQ_OK;
    int st = AWQ_OK;
    for (int t = 0; t < n_tensors; ++t) if (tensors[t] == nullptr) return AWQ_ERR_NULL;
    // pages of whole 16 bytes are copied in these, others (scales, in layers of any number) in words of 4
    for (int t = 0; t < n_tensors; ++t)
        if ((st = page_bytes[t] % 16 == 0 ? check_ptr(tensors[t]) : check_index({tensors[t]}))) return as_status(st);
    if ((st = check_index({pairs}))) return as_status(st);
    if (count != nullptr && (st = check_index({count}))) return as_status(st);
    p.n = n_tensors;
    p.layers = layers;
    p.max_pairs = max_pairs;
    p.pages = pages;
    p.pairs = pairs;
    p.count = count;
    return hip_status(awq::launch_cache_copy_pages(p, stream));
}

}  // extern "C"
