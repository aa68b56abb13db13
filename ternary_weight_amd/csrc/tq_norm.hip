// libtq: tq_rmsnorm -- residual addition, RMSNorm and the cast to the type
// the next product reads, one pass over the row.
//
//   h = x + residual;  r = 1 / sqrt(mean(h^2) + eps);  n = h r w;  y = n, or
//   q = rne(n 127 / max|n|) with the scale max|n| / 127.
//
// Two reductions per row (the sum of squares, then max|n|, which needs r)
// stand between reading x and writing y, so the row stays in registers
// between them: a thread keeps V units of U consecutive elements, and the
// row is read once, so memory bounds it (16381 x 4096, bf16 throughout with
// the residual: 89.6 us, 5.99 TB/s, where a copy of 1 GiB reaches 5.15).
// The sum of squares is fp64 (an fp64 fma per element is far below the memory
// time), rounded once to fp32; every other step is one IEEE fp32 operation
// (this file is built with -ffp-contract=off), so the int8 codes equal
// tq_act_quant_int8's of the same n, bit for bit.
#include <math.h>

#include "tq_internal.h"

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kNone = -1;                 // RT: no residual
constexpr int kMaxGrid = 1 << 20;         // workgroups of one launch; more rows are walked in a loop

struct Args {
    const void* x;
    const void* res;
    void* res_out;
    const float* w;
    void* y;
    float* ys;
    int64_t M;
    int32_t Kin;
    float eps;
};

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// U consecutive elements (a unit) as fp32, and back: 16 bytes per load or
// store where the type allows (U = 8 for bf16, 4 for fp32).  Outputs are
// stored non-temporally (2048 x 2560, residual, int8: 16.6 -> 11.9 us;
// 16381 x 4096 bf16: 93.8 -> 89.8 us), inputs are not loaded so (10% slower).
template <int TYPE, int U>
__device__ __forceinline__ void load_u(const void* row, int i, float (&v)[U])
{
    if (TYPE == TQ_F32) {
#pragma unroll
        for (int k = 0; k < U / 4; ++k) {
            const f32x4 f = reinterpret_cast<const f32x4*>(row)[i * (U / 4) + k];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[4 * k + e] = f[e];
        }
    } else {
        uint32_t w[U / 2];
        if constexpr (U == 8) {
            const u32x4 q = reinterpret_cast<const u32x4*>(row)[i];
            w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
        } else {
            const u32x2 q = reinterpret_cast<const u32x2*>(row)[i];
            w[0] = q.x, w[1] = q.y;
        }
#pragma unroll
        for (int k = 0; k < U / 2; ++k) {
            v[2 * k] = __uint_as_float(w[k] << 16);
            v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
        }
    }
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b)
{
    const uint16_t lo = __builtin_bit_cast(uint16_t, (__bf16)a), hi = __builtin_bit_cast(uint16_t, (__bf16)b);
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

template <int TYPE, int U>
__device__ __forceinline__ void store_u(void* row, int i, const float (&v)[U])
{
    if constexpr (TYPE == TQ_F32) {
#pragma unroll
        for (int k = 0; k < U / 4; ++k)
            __builtin_nontemporal_store(f32x4{v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]},
                                        &reinterpret_cast<f32x4*>(row)[i * (U / 4) + k]);
    } else if constexpr (U == 8) {
        __builtin_nontemporal_store(u32x4{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]),
                                          bf16_pair(v[6], v[7])},
                                    &reinterpret_cast<u32x4*>(row)[i]);
    } else {
        __builtin_nontemporal_store(u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])},
                                    &reinterpret_cast<u32x2*>(row)[i]);
    }
}

__device__ __forceinline__ uint32_t quant1(float v, float inv)
{
    const float r = fminf(fmaxf(rintf(v * inv), -127.0f), 127.0f);
    return (uint32_t)(uint8_t)(int8_t)(int)r;
}

__device__ __forceinline__ double wave_sum(double v)
{
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}

__device__ __forceinline__ float wave_max(float v)
{
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, 64));
    return v;
}

// One row per workgroup of T threads, V units of U elements per thread; the
// weight stays in registers over the workgroup's rows, except where a row
// alone takes half of a thread's 128 registers (Kin > 32768): there it is read
// from L2 again for each row, since keeping it spills (2048 x 65536, bf16
// throughout with the residual: 213 us, 422 us with the weight kept).
// Two reductions use two LDS arrays: a wave writes the first again only
// after the second's barrier, which every wave reaches after reading the
// first, so the loop over rows needs no further barrier.
template <int XT, int RT, int YT, int U, int T, int V>
__global__ __launch_bounds__(T) void k_rmsnorm(Args A)
{
    constexpr int W = T / 64;
    constexpr bool kKeep = V * U <= 32;
    __shared__ double red_s[W];
    __shared__ float red_a[W];
    const int tid = threadIdx.x, nu = A.Kin / U;
    float w[kKeep ? V : 1][U];
    if constexpr (kKeep)
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (tid + j * T < nu) load_u<TQ_F32, U>(A.w, tid + j * T, w[j]);
    for (int64_t m = blockIdx.x; m < A.M; m += gridDim.x) {
        const int64_t at = m * A.Kin;
        const uint8_t* xr = (const uint8_t*)A.x + at * (XT == TQ_F32 ? 4 : 2);
        const uint8_t* rr = RT == kNone ? nullptr : (const uint8_t*)A.res + at * (RT == TQ_F32 ? 4 : 2);
        float h[V][U];
#pragma unroll
        for (int j = 0; j < V; ++j) {
#pragma unroll
            for (int e = 0; e < U; ++e) h[j][e] = 0.0f;
            if (tid + j * T < nu) load_u<XT, U>(xr, tid + j * T, h[j]);
        }
        if constexpr (RT != kNone)
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (tid + j * T < nu) {
                    float r[U];
                    load_u<RT, U>(rr, tid + j * T, r);
#pragma unroll
                    for (int e = 0; e < U; ++e) h[j][e] += r[e];
                }
        double s = 0.0;
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int e = 0; e < U; ++e) s = fma((double)h[j][e], (double)h[j][e], s);
        s = wave_sum(s);
        if (W > 1) {
            if ((tid & 63) == 0) red_s[tid >> 6] = s;
            __syncthreads();
            s = 0.0;
#pragma unroll
            for (int k = 0; k < W; ++k) s += red_s[k];
        }
        if constexpr (RT != kNone)
            if (A.res_out) {
                uint8_t* ro = (uint8_t*)A.res_out + at * (RT == TQ_F32 ? 4 : 2);
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (tid + j * T < nu) store_u<RT, U>(ro, tid + j * T, h[j]);
            }
        const float mean = (float)(s / (double)A.Kin);
        const float r = 1.0f / sqrtf(mean + A.eps);
        float a = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (tid + j * T < nu) {
                if constexpr (!kKeep) load_u<TQ_F32, U>(A.w, tid + j * T, w[0]);
#pragma unroll
                for (int e = 0; e < U; ++e) h[j][e] = (h[j][e] * r) * w[kKeep ? j : 0][e];
                if constexpr (YT != TQ_I8) {
                    store_u<YT, U>((uint8_t*)A.y + at * (YT == TQ_F32 ? 4 : 2), tid + j * T, h[j]);
                } else {
#pragma unroll
                    for (int e = 0; e < U; ++e) a = fmaxf(a, fabsf(h[j][e]));
                }
            }
        if constexpr (YT == TQ_I8) {
            a = wave_max(a);
            if (W > 1) {
                if ((tid & 63) == 0) red_a[tid >> 6] = a;
                __syncthreads();
                a = red_a[0];
#pragma unroll
                for (int k = 1; k < W; ++k) a = fmaxf(a, red_a[k]);
            }
            const float inv = a > 0.0f ? 127.0f / a : 0.0f;
            uint32_t* q = (uint32_t*)((uint8_t*)A.y + at);
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (tid + j * T < nu) {
                    uint32_t c[U / 4];
#pragma unroll
                    for (int k = 0; k < U / 4; ++k)
                        c[k] = quant1(h[j][4 * k], inv) | (quant1(h[j][4 * k + 1], inv) << 8) |
                               (quant1(h[j][4 * k + 2], inv) << 16) | (quant1(h[j][4 * k + 3], inv) << 24);
                    if constexpr (U == 8)
                        __builtin_nontemporal_store(u32x2{c[0], c[1]}, &reinterpret_cast<u32x2*>(q)[tid + j * T]);
                    else __builtin_nontemporal_store(c[0], &q[tid + j * T]);
                }
            if (tid == 0) A.ys[m] = a > 0.0f ? a / 127.0f : 0.0f;
        } else if (W > 1) {
            __syncthreads();   // red_s is read before the next row writes it
        }
    }
}

template <int XT, int RT, int YT, int U, int T, int V>
void launch_as(const Args& A, hipStream_t st)
{
    const unsigned grid = (unsigned)(A.M < kMaxGrid ? A.M : kMaxGrid);
    hipLaunchKernelGGL((k_rmsnorm<XT, RT, YT, U, T, V>), dim3(grid), dim3(T), 0, st, A);
}

// The threads of a row: as few as hold it in registers (fewer, fuller
// workgroups hide each other's reductions; 2048 x 6912 fp32 to int8 with 256
// threads of 8 units 16.6 us, with 1024 threads of 2 to 4 units 30 us).
template <int XT, int RT, int YT>
void launch(const Args& A, hipStream_t st)
{
    // 8 elements per unit where x and the residual are bf16
    if constexpr (XT == TQ_BF16 && RT != TQ_F32) {
        if (A.Kin <= 1024) launch_as<XT, RT, YT, 8, 64, 2>(A, st);
        else if (A.Kin <= 4096) launch_as<XT, RT, YT, 8, 256, 2>(A, st);
        else if (A.Kin <= 8192) launch_as<XT, RT, YT, 8, 256, 4>(A, st);
        else if (A.Kin <= 16384) launch_as<XT, RT, YT, 8, 512, 4>(A, st);
        else if (A.Kin <= 32768) launch_as<XT, RT, YT, 8, 1024, 4>(A, st);
        else launch_as<XT, RT, YT, 8, 1024, 8>(A, st);
    } else {
        if (A.Kin <= 1024) launch_as<XT, RT, YT, 4, 64, 4>(A, st);
        else if (A.Kin <= 4096) launch_as<XT, RT, YT, 4, 256, 4>(A, st);
        else if (A.Kin <= 8192) launch_as<XT, RT, YT, 4, 256, 8>(A, st);
        else if (A.Kin <= 16384) launch_as<XT, RT, YT, 4, 512, 8>(A, st);
        else if (A.Kin <= 32768) launch_as<XT, RT, YT, 4, 1024, 8>(A, st);
        else launch_as<XT, RT, YT, 4, 1024, 16>(A, st);
    }
}

template <int XT, int RT>
void launch_y(int y_type, const Args& A, hipStream_t st)
{
    if (y_type == TQ_F32) launch<XT, RT, TQ_F32>(A, st);
    else if (y_type == TQ_BF16) launch<XT, RT, TQ_BF16>(A, st);
    else launch<XT, RT, TQ_I8>(A, st);
}

template <int XT>
void launch_r(int rt, int y_type, const Args& A, hipStream_t st)
{
    if (rt == kNone) launch_y<XT, kNone>(y_type, A, st);
    else if (rt == TQ_F32) launch_y<XT, TQ_F32>(y_type, A, st);
    else launch_y<XT, TQ_BF16>(y_type, A, st);
}

int64_t size_of(int t) { return t == TQ_F32 ? 4 : t == TQ_BF16 ? 2 : 1; }

}  // namespace

TQ_EXPORT tq_status tq_rmsnorm(int64_t M, int64_t Kin, int32_t x_type, const void* x, int32_t residual_type,
                               const void* residual, void* residual_out, const float* weight, float eps,
                               int32_t y_type, void* y, float* y_scale, void* stream)
{
    tq_status s;
    if (M < 0 || Kin < 0)
        return tq_fail(TQ_ERR_ARG, "negative size M = %lld, Kin = %lld", (long long)M, (long long)Kin);
    if (x_type != TQ_F32 && x_type != TQ_BF16)
        return tq_fail(TQ_ERR_ARG, "x_type = %d, must be TQ_F32 or TQ_BF16", x_type);
    if (residual && residual_type != TQ_F32 && residual_type != TQ_BF16)
        return tq_fail(TQ_ERR_ARG, "residual_type = %d, must be TQ_F32 or TQ_BF16", residual_type);
    if (y_type != TQ_F32 && y_type != TQ_BF16 && y_type != TQ_I8)
        return tq_fail(TQ_ERR_ARG, "y_type = %d, must be TQ_F32, TQ_BF16 or TQ_I8", y_type);
    if (Kin % 16 || Kin == 0 || Kin > TQ_MAX_KIN || M > (1ll << 31) - 1)
        return tq_fail(TQ_ERR_SHAPE, "M = %lld, in_features = %lld: a multiple of 16 in 16..%d, M up to 2^31 - 1",
                       (long long)M, (long long)Kin, TQ_MAX_KIN);
    if (!(eps >= 0.0f) || isinf(eps))
        return tq_fail(TQ_ERR_VALUE, "eps = %g, must be finite and not negative", (double)eps);
    if (residual_out && !residual) return tq_fail(TQ_ERR_ARG, "residual_out without a residual");
    if (M == 0) return tq_ok();
    if ((s = tq_check_ptr(x, "x", false))) return s;
    if ((s = tq_check_ptr(residual, "residual", true))) return s;
    if ((s = tq_check_ptr(residual_out, "residual_out", true))) return s;
    if ((s = tq_check_ptr(weight, "weight", false))) return s;
    if ((s = tq_check_ptr(y, "y", false))) return s;
    if (y_type == TQ_I8 && (s = tq_check_ptr(y_scale, "y_scale", false, 4))) return s;
    const int64_t xb = M * Kin * size_of(x_type), rb = M * Kin * size_of(residual_type), yb = M * Kin * size_of(y_type);
    const int64_t wb = Kin * 4, sb = y_type == TQ_I8 ? M * 4 : 0;
    if ((s = tq_check_overlap(y, yb, "y", x, xb, "x", y_type == x_type))) return s;
    if ((s = tq_check_overlap(y, yb, "y", residual, rb, "residual"))) return s;
    if ((s = tq_check_overlap(y, yb, "y", residual_out, rb, "residual_out"))) return s;
    if ((s = tq_check_overlap(y, yb, "y", weight, wb, "weight"))) return s;
    if ((s = tq_check_overlap(residual_out, rb, "residual_out", residual, rb, "residual", true))) return s;
    if ((s = tq_check_overlap(residual_out, rb, "residual_out", x, xb, "x"))) return s;
    if ((s = tq_check_overlap(residual_out, rb, "residual_out", weight, wb, "weight"))) return s;
    if ((s = tq_check_overlap(y_scale, sb, "y_scale", x, xb, "x"))) return s;
    if ((s = tq_check_overlap(y_scale, sb, "y_scale", y, yb, "y"))) return s;
    if ((s = tq_check_overlap(y_scale, sb, "y_scale", residual, rb, "residual"))) return s;
    if ((s = tq_check_overlap(y_scale, sb, "y_scale", residual_out, rb, "residual_out"))) return s;
    if ((s = tq_check_overlap(y_scale, sb, "y_scale", weight, wb, "weight"))) return s;
    const Args A{x, residual, residual_out, weight, y, y_scale, M, (int32_t)Kin, eps};
    const int rt = residual ? residual_type : kNone;
    if (x_type == TQ_F32) launch_r<TQ_F32>(rt, y_type, A, (hipStream_t)stream);
    else launch_r<TQ_BF16>(rt, y_type, A, (hipStream_t)stream);
    if ((s = tq_check_launch("tq_rmsnorm"))) return s;
    return tq_ok();
}
