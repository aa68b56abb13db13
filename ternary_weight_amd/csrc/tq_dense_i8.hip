// libtq: tq_gemm_dense_i8 -- int8 activations times a dense int8 weight, a
// scale per token and per output channel, on the int8 matrix cores.
//
//   acc[m][n] = sum_i xq[m][i] w[n][i] (int32, exact);
//   y = fl(float(acc) fl(x_scale[m] w_scale[n])).
//
// |acc| <= 128 * 128 * 65536 = 2^30, so int32 never wraps.
#include "tq_internal.h"
#include "tq_decode.h"

namespace {

using namespace tqk;

typedef int i32x4 __attribute__((ext_vector_type(4)));

struct Args {
    const int8_t* x;
    const float* xs;
    const int8_t* w;
    const float* ws;
    void* y;
    int32_t M, N, Kin;
};

template <int YT>
__device__ __forceinline__ void store_y(const Args& A, int m, int n, int acc)
{
    if (m >= A.M || n >= A.N) return;
    const float v = (float)acc * (A.xs[m] * A.ws[n]);
    const int64_t at = (int64_t)m * A.N + n;
    if (YT == TQ_F32) ((float*)A.y)[at] = v;
    else ((__bf16*)A.y)[at] = (__bf16)v;
}

// A workgroup of 4 waves: 16 tokens by 64 rows of w, a 16 x 16 tile per wave.
// Lane l holds 16 columns of row l % 16 per operand and step of 64 columns.
// Buffer resources: rows past M and N, and columns past Kin, read zeros.
template <int YT>
__global__ __launch_bounds__(256) void k_dense_i8(Args A, int tiles_m)
{
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int m0 = (int)(blockIdx.x % tiles_m) * 16, n0 = (int)(blockIdx.x / tiles_m) * 64 + (threadIdx.x >> 6) * 16;
    if (n0 >= A.N) return;
    const int K = A.Kin;
    const int64_t mrows = A.M - m0 < 16 ? A.M - m0 : 16, nrows = A.N - n0 < 16 ? A.N - n0 : 16;
    const __amdgpu_buffer_rsrc_t rx = rsrc(A.x + (int64_t)m0 * K, mrows * K);
    const __amdgpu_buffer_rsrc_t rw = rsrc(A.w + (int64_t)n0 * K, nrows * K);
    i32x4 acc = {0, 0, 0, 0};
    for (int k = 0; k < K; k += 64) {
        const int c = k + 16 * q;
        const uint32_t off = c < K ? (uint32_t)(r * K + c) : kOffNone;
        const u32x4 a = buffer_load<u32x4, 0>(rx, off, 0), b = buffer_load<u32x4, 0>(rw, off, 0);
        acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), acc, 0,
                                                    0, 0);
    }
    // lane l holds column l % 16 (n) of rows 4 (l / 16) + e (m)
#pragma unroll
    for (int e = 0; e < 4; ++e) store_y<YT>(A, m0 + 4 * q + e, n0 + r, acc[e]);
}

}  // namespace

TQ_EXPORT tq_status tq_gemm_dense_i8(int64_t M, int64_t N, int64_t Kin, const int8_t* xq, const float* x_scale,
                                     const int8_t* w, const float* w_scale, int32_t y_type, void* y, void* stream)
{
    tq_status s;
    if (M < 0 || N < 0 || Kin < 0)
        return tq_fail(TQ_ERR_ARG, "negative size M = %lld, N = %lld, Kin = %lld", (long long)M, (long long)N,
                       (long long)Kin);
    if (y_type != TQ_F32 && y_type != TQ_BF16)
        return tq_fail(TQ_ERR_ARG, "y_type = %d, must be TQ_F32 or TQ_BF16", y_type);
    if (Kin % 16 || Kin > TQ_MAX_KIN || M > TQ_MAX_N || N > TQ_MAX_N)
        return tq_fail(TQ_ERR_SHAPE, "M = %lld, N = %lld, in_features = %lld: M and N up to %d, Kin a multiple of 16 up to %d",
                       (long long)M, (long long)N, (long long)Kin, TQ_MAX_N, TQ_MAX_KIN);
    if (M == 0 || N == 0) return tq_ok();
    if ((s = tq_check_ptr(xq, "xq", Kin == 0))) return s;
    if ((s = tq_check_ptr(w, "w", Kin == 0))) return s;
    if ((s = tq_check_ptr(x_scale, "x_scale", false, 4))) return s;
    if ((s = tq_check_ptr(w_scale, "w_scale", false, 4))) return s;
    if ((s = tq_check_ptr(y, "y", false, 4))) return s;
    const int64_t yb = M * N * (y_type == TQ_F32 ? 4 : 2);
    if ((s = tq_check_overlap(y, yb, "y", xq, M * Kin, "xq"))) return s;
    if ((s = tq_check_overlap(y, yb, "y", w, N * Kin, "w"))) return s;
    if ((s = tq_check_overlap(y, yb, "y", x_scale, M * 4, "x_scale"))) return s;
    if ((s = tq_check_overlap(y, yb, "y", w_scale, N * 4, "w_scale"))) return s;
    const Args A{xq, x_scale, w, w_scale, y, (int32_t)M, (int32_t)N, (int32_t)Kin};
    const int64_t tm = (M + 15) / 16, tn = (N + 63) / 64;
    if (tm * tn > (1 << 24) - 1)
        return tq_fail(TQ_ERR_UNSUPPORTED, "%lld tiles exceed one launch", (long long)(tm * tn));
    if (y_type == TQ_F32)
        hipLaunchKernelGGL(k_dense_i8<TQ_F32>, dim3((unsigned)(tm * tn)), dim3(256), 0, (hipStream_t)stream, A, (int)tm);
    else
        hipLaunchKernelGGL(k_dense_i8<TQ_BF16>, dim3((unsigned)(tm * tn)), dim3(256), 0, (hipStream_t)stream, A, (int)tm);
    if ((s = tq_check_launch("tq_gemm_dense_i8"))) return s;
    return tq_ok();
}
